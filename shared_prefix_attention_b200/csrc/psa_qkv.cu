// The pass between the QKV projection and attention, and the cache rows it
// feeds.  Per (token, head) row x of d elements:
//   norm      xn = w * x * r,  r = rsqrt(mean(x^2) + eps)        (w given)
//   rotation  pairs (a, b) of the first rot elements turn by the token's
//             angle: a' = a c - b s, b' = a s + b c; the rest pass through
// Three forms share the row code:
//   forward   queries and keys in, normed and rotated queries and keys out
//   append    queries out as above; keys (normed and rotated) and values go
//             straight to their cache rows, as bf16 or as e4m3(x / scale)
//   backward  with g = the upstream gradient turned back by the angle:
//             dx = r (w g - x r^2 mean(w g x)),  dw = sum over rows of g x r
// and cache_read copies cache rows back to dense bf16 (e4m3 * scale).
//
// All of it is bound by memory: each input element is read once and each
// output element written once, in 16-byte lane accesses, with everything in
// between in fp32 registers and one rounding at the store.  A row is spread
// over d/8 lanes of 8 elements, so the norm's sum is log2(d/8) shuffles and
// the half-split rotation fetches its partner elements from the lane rot/16
// away.  A warp keeps one token's cos/sin and weights in registers over all
// the heads of its task.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "psa_device.cuh"
#include "psa_internal.h"

namespace psa {
namespace {

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kUnroll = 4;  // rows a lane group has in flight

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0];
  const float4 b = reinterpret_cast<const float4*>(p)[1];
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                            pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
// e4m3(x / scale), saturating at +-448 (NaN stays NaN).  The division is the
// exact one, so the code equals the rounding of the fp32 quotient.
__device__ __forceinline__ void store8_e4m3(uint8_t* p, const float (&x)[8], float scale) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(
        make_float2(__fdiv_rn(x[4 * i], scale), __fdiv_rn(x[4 * i + 1], scale)), __NV_SATFINITE,
        __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(
        make_float2(__fdiv_rn(x[4 * i + 2], scale), __fdiv_rn(x[4 * i + 3], scale)),
        __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | (hi << 16);
  }
  *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

// Sum over the LPR lanes of a row group (every lane gets it).
template <int LPR>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int off = LPR / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// One lane's share of a token's rotation.  Half-split form: the lane's 8
// elements pair with those of lane `src`, by 8 angles; interleaved form: 4
// pairs inside the lane.  `s` carries the sign of the lane's half, so both
// halves compute own * c + other * s.  Lanes behind rot (on == false) keep
// their elements, infinities included.
template <bool INTER>
struct Turn {
  float c[INTER ? 4 : 8], s[INTER ? 4 : 8];
  int src;
  bool on;
};

template <bool INTER>
__device__ __forceinline__ void load_turn(Turn<INTER>& t, const float* cos_sin, int rot, int l,
                                          int lane, float dir) {
  constexpr int N = INTER ? 4 : 8;
  t.src = lane;
  t.on = 8 * l < rot;
#pragma unroll
  for (int i = 0; i < N; ++i) t.c[i] = 1.f, t.s[i] = 0.f;
  if (!t.on) return;
  const int half = rot / 2;
  int a0;  // first angle of the lane
  float sign;
  if constexpr (INTER) {
    a0 = 4 * l;
    sign = dir;
  } else {
    const bool first = 8 * l < half;
    a0 = first ? 8 * l : 8 * l - half;
    t.src = first ? lane + half / 8 : lane - half / 8;
    sign = first ? -dir : dir;
  }
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(cos_sin + a0 + i));
    const float4 s = __ldg(reinterpret_cast<const float4*>(cos_sin + half + a0 + i));
    t.c[i] = c.x, t.c[i + 1] = c.y, t.c[i + 2] = c.z, t.c[i + 3] = c.w;
    t.s[i] = sign * s.x, t.s[i + 1] = sign * s.y, t.s[i + 2] = sign * s.z, t.s[i + 3] = sign * s.w;
  }
}

template <bool INTER>
__device__ __forceinline__ void turn8(const Turn<INTER>& t, float (&x)[8]) {
  if constexpr (INTER) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = t.on ? a * t.c[i] - b * t.s[i] : a;
      x[2 * i + 1] = t.on ? a * t.s[i] + b * t.c[i] : b;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float other = __shfl_sync(0xffffffffu, x[i], t.src);
      x[i] = t.on ? x[i] * t.c[i] + other * t.s[i] : x[i];
    }
  }
}

__device__ __forceinline__ void load_weight(const void* w, int dtype, int l, float (&x)[8]) {
  if (dtype == PSA_F32)
    load8(static_cast<const float*>(w) + 8 * l, x);
  else
    load8(static_cast<const __nv_bfloat16*>(w) + 8 * l, x);
}

struct RowParams {
  const void *x[3];      // q, k, v rows in
  int64_t xs[3];         // their token strides, elements
  void *y[3];            // q_out; k_out or k cache; v cache
  int32_t H[3];          // heads of each kind (0: the kind takes no part)
  int32_t slices[3];     // warps a token's heads of the kind are split over
  int32_t hs;            // heads per slice
  int32_t nslice;        // slices[0] + slices[1] + slices[2]
  int32_t T;
  const int32_t* pos;
  const float* cos_sin;
  int64_t n_pos;
  int32_t rot;           // 0: no rotation
  const void* w[2];      // nullptr: no norm of that kind
  int32_t w_dtype;
  float eps;
  const int32_t* slots;  // append form: cache row per token, negative: none
  int64_t n_cache;
  bool e4m3;
  float scale[2];        // k_scale, v_scale
  int32_t* status;
  // backward
  const void* dy[2];     // upstream gradients, dense
  int64_t dxs[2];        // token strides of dx (in y[0], y[1])
  float* part;           // [grid][2][D] partial weight gradients
};

// The token's row in the angle table; -1 (and a report) if it is outside.
__device__ __forceinline__ int64_t token_angle(const RowParams& p, int t, int lane) {
  if (p.rot == 0) return 0;
  const int32_t at = __ldg(p.pos + t);
  if (at < 0 || at >= p.n_pos) {
    if (lane == 0) report_status(p.status, PSA_ERR_INVALID_ARG);
    return -1;
  }
  return at;
}

// Task -> (token, kind, first head, end head).
struct Task {
  int t, kind, h0, h1;
};
__device__ __forceinline__ Task task_of(const RowParams& p, int64_t task) {
  Task k;
  k.t = int(task / p.nslice);
  int s = int(task - int64_t(k.t) * p.nslice);
  k.kind = 0;
  while (k.kind < 2 && s >= p.slices[k.kind]) s -= p.slices[k.kind++];
  k.h0 = s * p.hs;
  k.h1 = min(k.h0 + p.hs, p.H[k.kind]);
  return k;
}

// Forward and append: one warp per task, its rows kUnroll at a time.
template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kRowThreads) rows_kernel(RowParams p) {
  constexpr int LPR = D / 8, GROUPS = 32 / LPR;
  const int lane = threadIdx.x & 31, l = lane % LPR, g = lane / LPR;
  const int64_t task = int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  if (task >= int64_t(p.T) * p.nslice) return;
  const Task k = task_of(p, task);
  // where the rows go: dense by token, or the token's cache row
  int64_t out_row = k.t;
  if (p.slots && k.kind > 0) {
    const int32_t slot = __ldg(p.slots + k.t);
    if (slot < 0) return;  // a padded token: nothing is cached
    if (slot >= p.n_cache) {
      if (lane == 0) report_status(p.status, PSA_ERR_INVALID_ARG);
      return;
    }
    out_row = slot;
  }
  const int64_t at = token_angle(p, k.t, lane);
  if (at < 0) return;
  const bool turns = p.rot > 0 && k.kind < 2;
  const bool norms = k.kind < 2 && p.w[k.kind] != nullptr;
  Turn<INTER> turn;
  if (turns) load_turn<INTER>(turn, p.cos_sin + at * p.rot, p.rot, l, lane, 1.f);
  float w[8];
  if (norms) load_weight(p.w[k.kind], p.w_dtype, l, w);
  const T* x0 = static_cast<const T*>(p.x[k.kind]) + int64_t(k.t) * p.xs[k.kind] + 8 * l;
  const size_t y0 = size_t(out_row) * p.H[k.kind];

  for (int hb = k.h0; hb < k.h1; hb += GROUPS * kUnroll) {
    float x[kUnroll][8];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = hb + u * GROUPS + g;
      if (h < k.h1) load8(x0 + size_t(h) * D, x[u]);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = hb + u * GROUPS + g;
      if (hb + u * GROUPS >= k.h1) break;  // uniform: every lane takes part in the shuffles
      if (norms) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[u][i], x[u][i], ss);
        const float r = rsqrtf(group_sum<LPR>(ss) * (1.f / D) + p.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[u][i] *= r * w[i];
      }
      if (turns) turn8<INTER>(turn, x[u]);
      if (h >= k.h1) continue;
      const size_t off = (y0 + h) * D + 8 * l;
      if (k.kind > 0 && p.e4m3)
        store8_e4m3(static_cast<uint8_t*>(p.y[k.kind]) + off, x[u], p.scale[k.kind - 1]);
      else
        store8(static_cast<T*>(p.y[k.kind]) + off, x[u]);
    }
  }
}

// Backward: a fixed grid strides over the tasks, so that each block sums its
// rows' weight gradients in registers and writes one partial; the order of
// every sum is fixed by the sizes alone.
template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kRowThreads) rows_bwd_kernel(RowParams p) {
  constexpr int LPR = D / 8, GROUPS = 32 / LPR, U = 2;
  __shared__ float red[kRowWarps][2][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LPR, g = lane / LPR;
  float dw[2][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[0][i] = dw[1][i] = 0.f;
  const int64_t tasks = int64_t(p.T) * p.nslice;
  for (int64_t task = int64_t(blockIdx.x) * kRowWarps + warp; task < tasks;
       task += int64_t(gridDim.x) * kRowWarps) {
    const Task k = task_of(p, task);
    const int64_t at = token_angle(p, k.t, lane);
    if (at < 0) continue;
    Turn<INTER> turn;
    if (p.rot) load_turn<INTER>(turn, p.cos_sin + at * p.rot, p.rot, l, lane, -1.f);
    const bool norms = p.w[k.kind] != nullptr;
    float w[8];
    if (norms) load_weight(p.w[k.kind], p.w_dtype, l, w);
    const T* x0 = static_cast<const T*>(p.x[k.kind]) + int64_t(k.t) * p.xs[k.kind] + 8 * l;
    const T* g0 = static_cast<const T*>(p.dy[k.kind]) + int64_t(k.t) * p.H[k.kind] * D + 8 * l;
    T* d0 = static_cast<T*>(p.y[k.kind]) + int64_t(k.t) * p.dxs[k.kind] + 8 * l;
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    for (int hb = k.h0; hb < k.h1; hb += GROUPS * U) {
      float x[U][8], dy[U][8];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = hb + u * GROUPS + g;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[u][i] = dy[u][i] = 0.f;
        if (h < k.h1) {
          load8(g0 + size_t(h) * D, dy[u]);
          if (norms) load8(x0 + size_t(h) * D, x[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = hb + u * GROUPS + g;
        if (hb + u * GROUPS >= k.h1) break;
        if (p.rot) turn8<INTER>(turn, dy[u]);
        if (norms) {
          float ss = 0.f, dot = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            ss = fmaf(x[u][i], x[u][i], ss);
            dot = fmaf(w[i] * dy[u][i], x[u][i], dot);
          }
          ss = group_sum<LPR>(ss);
          dot = group_sum<LPR>(dot);
          const float r = rsqrtf(ss * (1.f / D) + p.eps);
          const float c = r * r * dot * (1.f / D);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            acc[i] = fmaf(dy[u][i], x[u][i] * r, acc[i]);
            dy[u][i] = r * (w[i] * dy[u][i] - x[u][i] * c);
          }
        }
        if (h < k.h1) store8(d0 + size_t(h) * D, dy[u]);
      }
    }
    // a selection, not an index: dw stays in registers
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      dw[0][i] += k.kind == 0 ? acc[i] : 0.f;
      dw[1][i] += k.kind == 1 ? acc[i] : 0.f;
    }
  }
  // the row groups of a warp, then the warps of the block
#pragma unroll
  for (int kd = 0; kd < 2; ++kd)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v = dw[kd][i];
#pragma unroll
      for (int off = LPR; off < 32; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
      if (g == 0) red[warp][kd][8 * l + i] = v;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kRowThreads) {
    float v = 0.f;
#pragma unroll
    for (int wi = 0; wi < kRowWarps; ++wi) v += (&red[wi][0][0])[i];
    p.part[size_t(blockIdx.x) * 2 * D + i] = v;
  }
}

// Sums the blocks' partials: one block per 32 weights, eight strided partial
// sums per weight, joined in shared memory in a fixed order.
__global__ void __launch_bounds__(256) weight_sum_kernel(const float* part, int nblocks, int D,
                                                         float* dqw, float* dkw) {
  __shared__ float red[8][32];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), j = threadIdx.x >> 5;
  float v = 0.f;
  for (int b = j; b < nblocks; b += 8) v += part[size_t(b) * 2 * D + c];
  red[j][threadIdx.x & 31] = v;
  __syncthreads();
  if (j == 0) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += red[i][threadIdx.x & 31];
    float* dst = c < D ? dqw : dkw;
    if (dst) dst[c < D ? c : c - D] = v;
  }
}

// Cache rows back to dense bf16: one 16-byte output chunk (8 elements) per
// lane and step.  A row outside the cache gives zeros and a report.
template <bool E4M3>
__global__ void __launch_bounds__(256) cache_read_kernel(
    const void* kc, const void* vc, const int32_t* rows, int64_t n, int64_t n_cache, int row_elems,
    float k_scale, float v_scale, __nv_bfloat16* k, __nv_bfloat16* v, int32_t* status) {
  const int per_row = row_elems / 8;
  const int64_t total = n * per_row;
  const int64_t step = int64_t(gridDim.x) * blockDim.x;
  for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < total; i += step) {
    const int64_t r = i / per_row;
    const int c = int(i - r * per_row);
    const int32_t row = __ldg(rows + r);
    const bool ok = row >= 0 && row < n_cache;
    if (!ok) report_status(status, PSA_ERR_INVALID_ARG);
    const size_t src = size_t(ok ? row : 0) * row_elems + 8 * c;
    const size_t dst = size_t(r) * row_elems + 8 * c;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const void* cache = which ? vc : kc;
      __nv_bfloat16* out = which ? v : k;
      uint4 w = make_uint4(0, 0, 0, 0);
      if (ok) {
        if constexpr (E4M3) {
          const float sc = which ? v_scale : k_scale;
          const uint2 b = __ldg(
              reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(cache) + src));
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                __nv_fp8x2_storage_t((j < 2 ? b.x : b.y) >> (16 * (j & 1))), __NV_E4M3);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
            o[j] = pack_bf16(f.x * sc, f.y * sc);
          }
          w = make_uint4(o[0], o[1], o[2], o[3]);
        } else {
          w = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(cache) + src));
        }
      }
      *reinterpret_cast<uint4*>(out + dst) = w;
    }
  }
}

// Heads per warp: a token's heads of a kind stay in one warp (its angles and
// weights are loaded once) unless the call has too few tokens to give every
// SM sixteen warps; then they are split until it has, or until each row
// group has one row.
void plan_rows(RowParams& p, int D) {
  const int groups = 32 / (D / 8);
  const int64_t want = 148 * 16;
  int64_t n = p.T > 0 ? (want + p.T - 1) / p.T : 1;
  const int hmax = p.H[0] > p.H[1] ? p.H[0] : p.H[1];
  int64_t hs = (hmax + n - 1) / n;
  hs = (hs + groups - 1) / groups * groups;
  if (hs < groups) hs = groups;
  p.hs = int32_t(hs);
  p.nslice = 0;
  for (int k = 0; k < 3; ++k) {
    p.slices[k] = (p.H[k] + p.hs - 1) / p.hs;
    p.nslice += p.slices[k];
  }
}

RowParams row_params(const RowsArgs& a) {
  RowParams p = {};
  p.x[0] = a.q, p.x[1] = a.k, p.x[2] = a.v;
  p.xs[0] = a.q_stride, p.xs[1] = a.k_stride, p.xs[2] = a.v_stride;
  p.y[0] = a.q_out, p.y[1] = a.k_out, p.y[2] = a.v_out;
  p.H[0] = a.q ? a.Hq : 0, p.H[1] = a.k ? a.Hkv : 0, p.H[2] = a.v ? a.Hkv : 0;
  p.T = a.T;
  p.pos = a.how.positions;
  p.cos_sin = a.how.cos_sin;
  p.n_pos = a.how.n_positions;
  p.rot = a.how.cos_sin ? a.how.rot_dim : 0;
  p.w[0] = a.how.q_weight, p.w[1] = a.how.k_weight;
  p.w_dtype = a.how.weight_dtype;
  p.eps = a.how.eps;
  p.slots = a.slots;
  p.n_cache = a.n_cache;
  p.e4m3 = a.e4m3;
  p.scale[0] = a.k_scale, p.scale[1] = a.v_scale;
  p.status = a.status;
  return p;
}

template <typename T, int D>
int launch_rows_d(const RowsArgs& a) {
  RowParams p = row_params(a);
  plan_rows(p, D);
  const int64_t tasks = int64_t(p.T) * p.nslice;
  const int64_t grid = (tasks + kRowWarps - 1) / kRowWarps;
  if (grid > INT32_MAX) return PSA_ERR_INVALID_ARG;
  if (a.how.interleaved)
    rows_kernel<T, D, true><<<uint32_t(grid), kRowThreads, 0, a.stream>>>(p);
  else
    rows_kernel<T, D, false><<<uint32_t(grid), kRowThreads, 0, a.stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? PSA_OK : PSA_ERR_CUDA;
}

template <typename T, int D>
int launch_rows_bwd_d(const RowsBwdArgs& b) {
  RowParams p = row_params(b.rows);
  plan_rows(p, D);
  p.dy[0] = b.dq_out, p.dy[1] = b.dk_out;
  p.dxs[0] = b.dq_stride, p.dxs[1] = b.dk_stride;
  p.part = b.part;
  const int64_t tasks = int64_t(p.T) * p.nslice;
  int64_t grid = (tasks + kRowWarps - 1) / kRowWarps;
  if (grid > kRowsBwdMaxBlocks) grid = kRowsBwdMaxBlocks;
  if (grid > 0) {  // without tokens the weight gradients are zero
    if (b.rows.how.interleaved)
      rows_bwd_kernel<T, D, true><<<uint32_t(grid), kRowThreads, 0, b.rows.stream>>>(p);
    else
      rows_bwd_kernel<T, D, false><<<uint32_t(grid), kRowThreads, 0, b.rows.stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return PSA_ERR_CUDA;
  }
  if (!b.dq_weight && !b.dk_weight) return PSA_OK;
  weight_sum_kernel<<<2 * D / 32, 256, 0, b.rows.stream>>>(b.part, int(grid), D, b.dq_weight,
                                                           b.dk_weight);
  return cudaGetLastError() == cudaSuccess ? PSA_OK : PSA_ERR_CUDA;
}

}  // namespace

int launch_rows(const RowsArgs& a) {
  const bool f32 = a.f32;
  switch (a.D) {
    case 64:
      return f32 ? launch_rows_d<float, 64>(a) : launch_rows_d<__nv_bfloat16, 64>(a);
    case 128:
      return f32 ? launch_rows_d<float, 128>(a) : launch_rows_d<__nv_bfloat16, 128>(a);
    case 256:
      return f32 ? launch_rows_d<float, 256>(a) : launch_rows_d<__nv_bfloat16, 256>(a);
    default:
      return PSA_ERR_UNSUPPORTED;
  }
}

int launch_rows_bwd(const RowsBwdArgs& b) {
  const bool f32 = b.rows.f32;
  switch (b.rows.D) {
    case 64:
      return f32 ? launch_rows_bwd_d<float, 64>(b) : launch_rows_bwd_d<__nv_bfloat16, 64>(b);
    case 128:
      return f32 ? launch_rows_bwd_d<float, 128>(b) : launch_rows_bwd_d<__nv_bfloat16, 128>(b);
    case 256:
      return f32 ? launch_rows_bwd_d<float, 256>(b) : launch_rows_bwd_d<__nv_bfloat16, 256>(b);
    default:
      return PSA_ERR_UNSUPPORTED;
  }
}

int launch_cache_read(const CacheReadArgs& a) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PSA_ERR_CUDA;
  const int sms = sm_count(dev);
  if (sms <= 0) return PSA_ERR_CUDA;
  const int row_elems = a.Hkv * a.D;
  const int64_t total = a.n * (row_elems / 8);
  int64_t grid = (total + 255) / 256;
  if (grid > int64_t(sms) * 8) grid = int64_t(sms) * 8;
  auto kern = a.e4m3 ? cache_read_kernel<true> : cache_read_kernel<false>;
  kern<<<uint32_t(grid), 256, 0, a.stream>>>(a.kc, a.vc, a.rows, a.n, a.n_cache, row_elems,
                                             a.k_scale, a.v_scale,
                                             static_cast<__nv_bfloat16*>(a.k),
                                             static_cast<__nv_bfloat16*>(a.v), a.status);
  return cudaGetLastError() == cudaSuccess ? PSA_OK : PSA_ERR_CUDA;
}

}  // namespace psa
