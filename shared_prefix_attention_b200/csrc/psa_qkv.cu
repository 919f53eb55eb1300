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
// output element written once, with everything in between in fp32 registers
// and one rounding at the store.  A row is spread over d/16 lanes of two
// 8-element pieces each.  In the half-split form a lane's pieces are partners
// of one another (pairs (i, i + rot/2)), in the interleaved form they are
// neighbours, so a rotation never leaves its lane; the norm's sum is
// log2(d/16) shuffles.  (One piece per lane, partners exchanged by eight
// shuffles a row, took two to three times as long.)  A warp keeps one token's
// cos/sin and weights in registers over the heads of its task and has kUnroll
// row groups' loads in flight.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "psa_device.cuh"
#include "psa_internal.h"

namespace psa {
namespace {

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;

// A lane's share of a row as it was loaded: two pieces of 8 elements.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  static constexpr int kUnroll = 4;  // row groups in flight
  uint4 v[2];
  __device__ __forceinline__ void load(const __nv_bfloat16* row, int a, int b) {
    v[0] = *reinterpret_cast<const uint4*>(row + a);
    v[1] = *reinterpret_cast<const uint4*>(row + b);
  }
  __device__ __forceinline__ void get(float (&x)[16]) const {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[8 * j + 2 * i] = __uint_as_float(w[i] << 16);
        x[8 * j + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
};
template <>
struct Raw<float> {
  static constexpr int kUnroll = 2;
  float4 v[4];
  __device__ __forceinline__ void load(const float* row, int a, int b) {
    v[0] = reinterpret_cast<const float4*>(row + a)[0];
    v[1] = reinterpret_cast<const float4*>(row + a)[1];
    v[2] = reinterpret_cast<const float4*>(row + b)[0];
    v[3] = reinterpret_cast<const float4*>(row + b)[1];
  }
  __device__ __forceinline__ void get(float (&x)[16]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      x[4 * j] = v[j].x, x[4 * j + 1] = v[j].y, x[4 * j + 2] = v[j].z, x[4 * j + 3] = v[j].w;
  }
};

__device__ __forceinline__ void store_row(__nv_bfloat16* row, int a, int b, const float (&x)[16]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float* y = x + 8 * j;
    *reinterpret_cast<uint4*>(row + (j ? b : a)) =
        make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]),
                   pack_bf16(y[6], y[7]));
  }
}
__device__ __forceinline__ void store_row(float* row, int a, int b, const float (&x)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    reinterpret_cast<float4*>(row + (j < 2 ? a : b))[j & 1] =
        make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
}
// e4m3(x * inv), inv = 1 / scale in fp32 (a step of fp32 from the quotient at
// most), saturating at +-448 (NaN stays NaN).
__device__ __forceinline__ void store_row_e4m3(uint8_t* row, int a, int b, const float (&x)[16],
                                               float inv) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float* y = x + 8 * j + 4 * i;
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0] * inv, y[1] * inv),
                                                   __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2] * inv, y[3] * inv),
                                                   __NV_SATFINITE, __NV_E4M3);
      w[i] = lo | (hi << 16);
    }
    *reinterpret_cast<uint2*>(row + (j ? b : a)) = make_uint2(w[0], w[1]);
  }
}

// Sum over the LPR lanes of a row (every lane gets it).
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int off = LPR / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// Where a lane's two pieces start.  Lanes before rot/16 hold the rotated
// elements: partners (half-split) or 16 neighbours (interleaved).  The others
// pass their 16 neighbours through, infinities included.
struct Pieces {
  int a, b;
  bool on;
};
template <bool INTER>
__device__ __forceinline__ Pieces pieces_of(int l, int rot) {
  Pieces s;
  s.on = 16 * l < rot;
  s.a = 16 * l, s.b = s.a + 8;
  if (!INTER && s.on) s.a = 8 * l, s.b = rot / 2 + 8 * l;
  return s;
}

// The lane's eight angles of one position; dir -1 turns back.
__device__ __forceinline__ void load_turn(float (&c)[8], float (&s)[8], const float* cos_sin,
                                          int rot, int l, float dir) {
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    const float4 x = __ldg(reinterpret_cast<const float4*>(cos_sin + 8 * l + i));
    const float4 y = __ldg(reinterpret_cast<const float4*>(cos_sin + rot / 2 + 8 * l + i));
    c[i] = x.x, c[i + 1] = x.y, c[i + 2] = x.z, c[i + 3] = x.w;
    s[i] = dir * y.x, s[i + 1] = dir * y.y, s[i + 2] = dir * y.z, s[i + 3] = dir * y.w;
  }
}
template <bool INTER>
__device__ __forceinline__ void turn_row(const float (&c)[8], const float (&s)[8],
                                         float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float& a = x[INTER ? 2 * i : i];
    float& b = x[INTER ? 2 * i + 1 : 8 + i];
    const float a0 = a, b0 = b;
    a = a0 * c[i] - b0 * s[i];
    b = a0 * s[i] + b0 * c[i];
  }
}

__device__ __forceinline__ void load_weight(const void* w, int dtype, const Pieces& pc,
                                            float (&x)[16]) {
  if (dtype == PSA_F32) {
    Raw<float> r;
    r.load(static_cast<const float*>(w), pc.a, pc.b);
    r.get(x);
  } else {
    Raw<__nv_bfloat16> r;
    r.load(static_cast<const __nv_bfloat16*>(w), pc.a, pc.b);
    r.get(x);
  }
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
  float inv_scale[2];    // of k_scale, v_scale
  int32_t* status;
  // backward
  const void* dy[2];     // upstream gradients, dense
  int64_t dxs[2];        // token strides of dx (in y[0], y[1])
  float* part;           // [grid][D] partial weight gradients
  int32_t blocks_q;      // the blocks below it work on q, the others on k
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

// Forward and append: one warp per task, its row groups kUnroll at a time.
template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kRowThreads) rows_kernel(RowParams p) {
  constexpr int LPR = D / 16, GROUPS = 32 / LPR, U = Raw<T>::kUnroll;
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
  const bool norms = k.kind < 2 && p.w[k.kind] != nullptr;
  const Pieces pc = pieces_of<INTER>(l, k.kind < 2 ? p.rot : 0);
  float c[8], s[8], w[16];
  if (pc.on) load_turn(c, s, p.cos_sin + at * p.rot, p.rot, l, 1.f);
  if (norms) load_weight(p.w[k.kind], p.w_dtype, pc, w);
  const T* x0 = static_cast<const T*>(p.x[k.kind]) + int64_t(k.t) * p.xs[k.kind];
  const size_t y0 = size_t(out_row) * p.H[k.kind];

  for (int hb = k.h0; hb < k.h1; hb += GROUPS * U) {
    Raw<T> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = hb + u * GROUPS + g;
      if (h < k.h1) raw[u].load(x0 + size_t(h) * D, pc.a, pc.b);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = hb + u * GROUPS + g;
      if (hb + u * GROUPS >= k.h1) break;  // uniform: every lane takes part in the shuffles
      float x[16];
      raw[u].get(x);
      if (norms) {
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          s0 = fmaf(x[i], x[i], s0);
          s1 = fmaf(x[8 + i], x[8 + i], s1);
        }
        const float r = rsqrtf(row_sum<LPR>(s0 + s1) * (1.f / D) + p.eps);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = x[i] * r * w[i];
      }
      if (pc.on) turn_row<INTER>(c, s, x);
      if (h >= k.h1) continue;
      const size_t off = (y0 + h) * D;
      if (k.kind > 0 && p.e4m3)
        store_row_e4m3(static_cast<uint8_t*>(p.y[k.kind]) + off, pc.a, pc.b, x,
                       p.inv_scale[k.kind - 1]);
      else
        store_row(static_cast<T*>(p.y[k.kind]) + off, pc.a, pc.b, x);
    }
  }
}

// Backward: every block works on one kind and strides over its tasks, so that
// it sums its rows' weight gradients in registers and writes one partial; the
// order of every sum is fixed by the sizes alone.
template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kRowThreads, 2) rows_bwd_kernel(RowParams p) {
  constexpr int LPR = D / 16, GROUPS = 32 / LPR, U = Raw<T>::kUnroll / 2;
  __shared__ float red[kRowWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LPR, g = lane / LPR;
  const int kind = int(blockIdx.x) < p.blocks_q ? 0 : 1;
  const int block = int(blockIdx.x) - (kind ? p.blocks_q : 0);
  const int blocks = kind ? int(gridDim.x) - p.blocks_q : p.blocks_q;
  const Pieces pc = pieces_of<INTER>(l, p.rot);
  const bool norms = p.w[kind] != nullptr;
  const int H = p.H[kind], slices = p.slices[kind];
  float w[16], dw[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) dw[i] = 0.f;
  if (norms) load_weight(p.w[kind], p.w_dtype, pc, w);
  const int64_t tasks = int64_t(p.T) * slices;
  for (int64_t task = int64_t(block) * kRowWarps + warp; task < tasks;
       task += int64_t(blocks) * kRowWarps) {
    const int t = int(task / slices);
    const int h0 = int(task - int64_t(t) * slices) * p.hs, h1 = min(h0 + p.hs, H);
    const int64_t at = token_angle(p, t, lane);
    if (at < 0) continue;
    float c[8], s[8];
    if (pc.on) load_turn(c, s, p.cos_sin + at * p.rot, p.rot, l, -1.f);
    const T* x0 = static_cast<const T*>(p.x[kind]) + int64_t(t) * p.xs[kind];
    const T* g0 = static_cast<const T*>(p.dy[kind]) + int64_t(t) * H * D;
    T* d0 = static_cast<T*>(p.y[kind]) + int64_t(t) * p.dxs[kind];
    for (int hb = h0; hb < h1; hb += GROUPS * U) {
      Raw<T> xr[U], gr[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = hb + u * GROUPS + g;
        // rows behind the last one: zeros, they add nothing to the sums
        xr[u] = Raw<T>{};
        gr[u] = Raw<T>{};
        if (h < h1) {
          gr[u].load(g0 + size_t(h) * D, pc.a, pc.b);
          if (norms) xr[u].load(x0 + size_t(h) * D, pc.a, pc.b);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = hb + u * GROUPS + g;
        if (hb + u * GROUPS >= h1) break;
        float dy[16];
        gr[u].get(dy);
        if (pc.on) turn_row<INTER>(c, s, dy);
        if (norms) {
          float x[16];
          xr[u].get(x);
          float ss = 0.f, dot = 0.f;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            ss = fmaf(x[i], x[i], ss);
            dot = fmaf(w[i] * dy[i], x[i], dot);
          }
          ss = row_sum<LPR>(ss);
          dot = row_sum<LPR>(dot);
          const float r = rsqrtf(ss * (1.f / D) + p.eps);
          const float e = r * r * dot * (1.f / D);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            dw[i] = fmaf(dy[i], x[i] * r, dw[i]);
            dy[i] = r * (w[i] * dy[i] - x[i] * e);
          }
        }
        if (h < h1) store_row(d0 + size_t(h) * D, pc.a, pc.b, dy);
      }
    }
  }
  // the row groups of a warp, then the warps of the block
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float v = dw[i];
#pragma unroll
    for (int off = LPR; off < 32; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (g == 0) red[warp][(i < 8 ? pc.a : pc.b) + (i & 7)] = v;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < D; i += kRowThreads) {
    float v = 0.f;
#pragma unroll
    for (int wi = 0; wi < kRowWarps; ++wi) v += red[wi][i];
    p.part[size_t(blockIdx.x) * D + i] = v;
  }
}

// Sums the blocks' partials, [0, blocks_q) for q and the rest for k: one block
// per 32 weights, eight strided partial sums per weight, joined in shared
// memory in a fixed order.
__global__ void __launch_bounds__(256) weight_sum_kernel(const float* part, int blocks_q,
                                                         int blocks, int D, float* dqw,
                                                         float* dkw) {
  __shared__ float red[8][32];
  const int kind = blockIdx.y, c = blockIdx.x * 32 + (threadIdx.x & 31), j = threadIdx.x >> 5;
  const int b0 = kind ? blocks_q : 0, b1 = kind ? blocks : blocks_q;
  float v = 0.f;
#pragma unroll 4
  for (int b = b0 + j; b < b1; b += 8) v += part[size_t(b) * D + c];
  red[j][threadIdx.x & 31] = v;
  __syncthreads();
  if (j == 0) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += red[i][threadIdx.x & 31];
    float* dst = kind ? dkw : dqw;
    if (dst) dst[c] = v;
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
  const int groups = 32 / (D / 16);
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
  p.inv_scale[0] = 1.f / a.k_scale, p.inv_scale[1] = 1.f / a.v_scale;
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
  // two blocks per SM in all, shared between the kinds by their rows
  int64_t need[2], blocks[2];
  for (int k = 0; k < 2; ++k)
    need[k] = (int64_t(p.T) * p.slices[k] + kRowWarps - 1) / kRowWarps;
  const int64_t H = int64_t(p.H[0]) + p.H[1];
  for (int k = 0; k < 2; ++k) {
    const int64_t share = H ? (kRowsBwdMaxBlocks * int64_t(p.H[k]) + H - 1) / H : 0;
    blocks[k] = need[k] < share ? need[k] : share;
  }
  if (blocks[0] + blocks[1] > kRowsBwdMaxBlocks) --blocks[blocks[0] > blocks[1] ? 0 : 1];
  p.blocks_q = int32_t(blocks[0]);
  const uint32_t grid = uint32_t(blocks[0] + blocks[1]);
  if (grid > 0) {  // without tokens the weight gradients are zero
    if (b.rows.how.interleaved)
      rows_bwd_kernel<T, D, true><<<grid, kRowThreads, 0, b.rows.stream>>>(p);
    else
      rows_bwd_kernel<T, D, false><<<grid, kRowThreads, 0, b.rows.stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return PSA_ERR_CUDA;
  }
  if (!b.dq_weight && !b.dk_weight) return PSA_OK;
  weight_sum_kernel<<<dim3(D / 32, 2), 256, 0, b.rows.stream>>>(
      b.part, p.blocks_q, int(grid), D, b.dq_weight, b.dk_weight);
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
