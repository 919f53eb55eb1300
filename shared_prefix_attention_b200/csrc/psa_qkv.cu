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
// and one rounding at the store.
//
// Loads.  The heads of a token are contiguous, so each warp keeps a ring of
// kDepth bulk copies (2 KB of rows each) of its own coming, whatever its
// registers hold: no other warp takes part, so there is nothing to wait for
// but one's own bytes.  (Loads into registers, the next batch ahead of the one
// at hand, reached 4.1 TB/s on the large layout's forward: the weights and
// angles leave too few registers to have more rows on the way.)
//
// Layout.  A row is spread over d/16 lanes of two 8-element pieces each.  In
// the half-split form a lane's pieces are partners of one another (pairs (i,
// i + rot/2)), in the interleaved form they are neighbours, so a rotation
// never leaves its lane; the norm's sum is log2(d/16) shuffles.  (One piece
// per lane, partners exchanged by eight shuffles a row, took twice as long.)
// A warp keeps one token's cos/sin and weights in registers over the heads of
// its task.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "psa_device.cuh"
#include "psa_internal.h"
#include "psa_pair.cuh"

namespace psa {
namespace {

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kStageBytes = 2048;  // of a warp's ring
constexpr int kDepth = 4;          // stages
constexpr uint32_t kRowSmem = kRowWarps * kDepth * kStageBytes;

// Plain (untiled) bulk copy of contiguous global bytes into shared memory;
// addresses and size are multiples of 16 bytes.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// A warp's ring: stages of shared memory and a barrier each.
struct Ring {
  uint8_t* base;
  uint64_t* bar;
  uint32_t put = 0, got = 0;  // stages filled and emptied so far
  __device__ __forceinline__ uint8_t* at(uint32_t n) const {
    return base + (n % kDepth) * kStageBytes;
  }
};
__device__ __forceinline__ Ring make_ring(uint8_t* smem, uint64_t (*bars)[kDepth]) {
  const int warp = threadIdx.x >> 5;
  Ring r;
  r.base = smem + warp * kDepth * kStageBytes;
  r.bar = bars[warp];
  if ((threadIdx.x & 31) == 0) {
    for (int i = 0; i < kDepth; ++i) mbar_init(r.bar + i, 1);
    fence_barrier_init();
  }
  __syncwarp();
  return r;
}

// A lane's share of a row as it was loaded: two pieces of 8 elements; get()
// gives them as eight pairs for the packed fp32 instructions.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 v[2];
  __device__ __forceinline__ void load(const __nv_bfloat16* row, int a, int b) {
    v[0] = *reinterpret_cast<const uint4*>(row + a);
    v[1] = *reinterpret_cast<const uint4*>(row + b);
  }
  __device__ __forceinline__ void get(uint64_t (&x)[8]) const {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[4 * j + i] = f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
  }
};
template <>
struct Raw<float> {
  float4 v[4];
  __device__ __forceinline__ void load(const float* row, int a, int b) {
    v[0] = reinterpret_cast<const float4*>(row + a)[0];
    v[1] = reinterpret_cast<const float4*>(row + a)[1];
    v[2] = reinterpret_cast<const float4*>(row + b)[0];
    v[3] = reinterpret_cast<const float4*>(row + b)[1];
  }
  __device__ __forceinline__ void get(uint64_t (&x)[8]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      x[2 * j] = f2_pack(v[j].x, v[j].y), x[2 * j + 1] = f2_pack(v[j].z, v[j].w);
  }
};

__device__ __forceinline__ uint32_t bf16_pair(uint64_t x) {
  float lo, hi;
  f2_unpack(x, lo, hi);
  return pack_bf16(lo, hi);
}
__device__ __forceinline__ void store_row(__nv_bfloat16* row, int a, int b,
                                          const uint64_t (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 2; ++j)
    *reinterpret_cast<uint4*>(row + (j ? b : a)) =
        make_uint4(bf16_pair(x[4 * j]), bf16_pair(x[4 * j + 1]), bf16_pair(x[4 * j + 2]),
                   bf16_pair(x[4 * j + 3]));
}
__device__ __forceinline__ void store_row(float* row, int a, int b, const uint64_t (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float4 v;
    f2_unpack(x[2 * j], v.x, v.y);
    f2_unpack(x[2 * j + 1], v.z, v.w);
    reinterpret_cast<float4*>(row + (j < 2 ? a : b))[j & 1] = v;
  }
}
// e4m3(x * inv), inv = 1 / scale in fp32 (a step of fp32 from the quotient at
// most), saturating at +-448 (NaN stays NaN).
__device__ __forceinline__ void store_row_e4m3(uint8_t* row, int a, int b,
                                               const uint64_t (&x)[8], float inv) {
  const uint64_t inv2 = f2_pack(inv, inv);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 y;
      f2_unpack(f2_mul(x[4 * j + i], inv2), y.x, y.y);
      h[i] = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
    }
    *reinterpret_cast<uint2*>(row + (j ? b : a)) =
        make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
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

// A rotation as x' = x k1 + partner(x) k2, element by element: k1 the cosines,
// k2 the sines with the partner's sign; dir -1 turns back.  Half-split: the
// partner of pair i (of 8) is pair i ^ 4; interleaved: the pair swapped.
struct Turn {
  uint64_t k1[8], k2[8];
};
template <bool INTER>
__device__ __forceinline__ void load_turn(Turn& t, const float* cos_sin, int rot, int l,
                                          float dir) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(cos_sin + 8 * l) + i);
    float4 s = __ldg(reinterpret_cast<const float4*>(cos_sin + rot / 2 + 8 * l) + i);
    s.x *= dir, s.y *= dir, s.z *= dir, s.w *= dir;
    if constexpr (INTER) {
      t.k1[4 * i] = f2_pack(c.x, c.x), t.k1[4 * i + 1] = f2_pack(c.y, c.y);
      t.k1[4 * i + 2] = f2_pack(c.z, c.z), t.k1[4 * i + 3] = f2_pack(c.w, c.w);
      t.k2[4 * i] = f2_pack(-s.x, s.x), t.k2[4 * i + 1] = f2_pack(-s.y, s.y);
      t.k2[4 * i + 2] = f2_pack(-s.z, s.z), t.k2[4 * i + 3] = f2_pack(-s.w, s.w);
    } else {
      t.k1[2 * i] = t.k1[4 + 2 * i] = f2_pack(c.x, c.y);
      t.k1[2 * i + 1] = t.k1[5 + 2 * i] = f2_pack(c.z, c.w);
      t.k2[2 * i] = f2_pack(-s.x, -s.y), t.k2[2 * i + 1] = f2_pack(-s.z, -s.w);
      t.k2[4 + 2 * i] = f2_pack(s.x, s.y), t.k2[5 + 2 * i] = f2_pack(s.z, s.w);
    }
  }
}
template <bool INTER>
__device__ __forceinline__ uint64_t partner(const uint64_t (&x)[8], int i) {
  if constexpr (INTER) {
    float lo, hi;
    f2_unpack(x[i], lo, hi);
    return f2_pack(hi, lo);
  } else {
    return x[i ^ 4];
  }
}
template <bool INTER>
__device__ __forceinline__ void turn_row(const Turn& t, uint64_t (&x)[8]) {
  uint64_t y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    y[i] = f2_fma(partner<INTER>(x, i), t.k2[i], f2_mul(x[i], t.k1[i]));
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = y[i];
}

__device__ __forceinline__ void load_weight(const void* w, int dtype, const Pieces& pc,
                                            uint64_t (&x)[8]) {
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
__device__ __forceinline__ float pair_sum(uint64_t x) {
  float lo, hi;
  f2_unpack(x, lo, hi);
  return lo + hi;
}
// sum of a[i] b[i] over the lane's 16 elements
__device__ __forceinline__ float dot16(const uint64_t (&a)[8], const uint64_t (&b)[8]) {
  uint64_t s0 = f2_mul(a[0], b[0]), s1 = f2_mul(a[1], b[1]);
#pragma unroll
  for (int i = 2; i < 8; i += 2) {
    s0 = f2_fma(a[i], b[i], s0);
    s1 = f2_fma(a[i + 1], b[i + 1], s1);
  }
  return pair_sum(f2_add(s0, s1));
}

// What each of a launch's warps takes: `stages` ring stages, and `more` of the
// warps, spread among them, one more.  (A stage is at least 128 bytes of its
// own memory, so that 32 bits hold the number of all.  With the first `more`
// warps taking it, the warps' rows lie one fixed step apart: 49152 tokens 182
// us against 172.)
struct Share {
  int32_t stages, more, warps;
};

struct RowParams {
  const void *x[3];      // q, k, v rows in
  int64_t xs[3];         // their token strides, elements
  void *y[3];            // q_out; k_out or k cache; v cache
  int32_t H[3];          // heads of each kind (0: the kind takes no part)
  int32_t stages[3];     // ring stages of a token's heads of the kind
  Share share[2];        // of all kinds; the backward: of q, of k
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

// What a token's rows need besides themselves: its position and cache row,
// read one task ahead so that a task does not start with their latency.
struct Place {
  int32_t at = 0, slot = 0;
};
__device__ __forceinline__ Place load_place(const RowParams& p, int t) {
  Place v;
  if (p.rot) v.at = __ldg(p.pos + t);
  if (p.slots) v.slot = __ldg(p.slots + t);
  return v;
}
// Whether the position lies in the angle table (reported if not).
__device__ __forceinline__ bool place_turns(const RowParams& p, const Place& v, int lane) {
  if (p.rot == 0 || (v.at >= 0 && v.at < p.n_pos)) return true;
  if (lane == 0) report_status(p.status, PSA_ERR_INVALID_ARG);
  return false;
}

// A warp's share of the work: an equal range of all stages (tokens in order,
// within a token its kinds), so the warps end together whatever the sizes.
// The host divides (Share).
struct Walk {
  int t, s;  // token, and stage within it
  int left;  // stages to go
  int step;  // to the next token
};
__device__ __forceinline__ Walk make_walk(int warp, const Share& share, int per_token) {
  auto extra = [&](int w) { return int(uint32_t(w) * share.more / uint32_t(share.warps)); };
  const int begin = warp * share.stages + extra(warp);
  Walk w;
  w.t = int(uint32_t(begin) / uint32_t(per_token));
  w.s = begin - w.t * per_token;
  w.left = share.stages + extra(warp + 1) - extra(warp);
  w.step = 1;
  return w;
}
// Or every warps-th token, whole.
__device__ __forceinline__ Walk make_strided_walk(int warp, int warps, int T, int per_token) {
  Walk w;
  w.t = warp;
  w.s = 0;
  w.left = warp < T ? ((T - 1 - warp) / warps + 1) * per_token : 0;
  w.step = warps;
  return w;
}
// The walk's next task, heads [h0, h1) of one kind of one token, `rows` of
// them to a stage; the walk moves behind it.
struct Task {
  int t, kind, h0, h1;
};
__device__ __forceinline__ Task next_task(const RowParams& p, Walk& w, int rows) {
  Task k;
  k.t = w.t;
  k.kind = 0;
  int s = w.s;
  while (k.kind < 2 && s >= p.stages[k.kind]) s -= p.stages[k.kind++];
  const int n = min(p.stages[k.kind] - s, w.left);
  k.h0 = s * rows;
  k.h1 = min(k.h0 + n * rows, p.H[k.kind]);
  w.left -= n;
  w.s += n;
  if (w.s == p.stages[0] + p.stages[1] + p.stages[2]) w.s = 0, w.t += w.step;
  return k;
}

// Forward and append.
template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kRowThreads, 2) rows_kernel(RowParams p) {
  constexpr int LPR = D / 16, GROUPS = 32 / LPR;
  constexpr int ROWS = kStageBytes / (D * int(sizeof(T)));  // rows of a stage
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[kRowWarps][kDepth];
  __shared__ int abort_flag;
  const int lane = threadIdx.x & 31, l = lane % LPR, g = lane / LPR;
  if (threadIdx.x == 0) abort_flag = 0;
  __syncthreads();
  Walk walk = make_walk(int(blockIdx.x) * kRowWarps + (threadIdx.x >> 5), p.share[0],
                        p.stages[0] + p.stages[1] + p.stages[2]);
  Ring ring = make_ring(smem, bars);

  // the copies run ahead: their own walk over the tasks
  Walk next = walk;
  Task n = {};
  int nh = 0;
  auto put = [&]() {
    if (nh >= n.h1) {
      if (next.left == 0) return;
      n = next_task(p, next, ROWS);
      nh = n.h0;
    }
    if (lane == 0) {
      const T* src = static_cast<const T*>(p.x[n.kind]) + int64_t(n.t) * p.xs[n.kind] +
                     size_t(nh) * D;
      const uint32_t bytes = uint32_t(min(ROWS, n.h1 - nh)) * D * sizeof(T);
      uint64_t* bar = ring.bar + ring.put % kDepth;
      mbar_arrive_expect_tx(bar, bytes);
      bulk_load(smem_u32(ring.at(ring.put)), src, bytes, bar);
    }
    nh += ROWS;
    ++ring.put;
  };
#pragma unroll 1
  for (int i = 0; i < kDepth; ++i) put();

  bool ok = true;
  Place place = {};
  if (walk.left > 0) place = load_place(p, walk.t);
  while (ok && walk.left > 0) {
    const Task k = next_task(p, walk, ROWS);
    const Place here = place;
    if (walk.left > 0) place = load_place(p, walk.t);
    // where the rows go: dense by token, or the token's cache row (a padded
    // token caches nothing)
    int64_t out_row = k.t;
    bool live = true;
    if (p.slots && k.kind > 0) {
      if (here.slot >= p.n_cache && lane == 0) report_status(p.status, PSA_ERR_INVALID_ARG);
      live = here.slot >= 0 && here.slot < p.n_cache;
      out_row = here.slot;
    }
    live = live && place_turns(p, here, lane);
    const bool norms = k.kind < 2 && p.w[k.kind] != nullptr;
    const Pieces pc = pieces_of<INTER>(l, k.kind < 2 ? p.rot : 0);
    // The weights are folded into the rotation: (x w r) k1 + (its partner) k2
    // = r (x (w k1) + partner(x) (partner(w) k2)); without a rotation k1 = w.
    Turn turn;
    uint64_t w[8];
    if (norms) load_weight(p.w[k.kind], p.w_dtype, pc, w);
    if (pc.on && live) {
      load_turn<INTER>(turn, p.cos_sin + int64_t(here.at) * p.rot, p.rot, l, 1.f);
      if (norms) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          turn.k1[i] = f2_mul(turn.k1[i], w[i]);
          turn.k2[i] = f2_mul(turn.k2[i], partner<INTER>(w, i));
        }
      }
    } else if (norms) {
#pragma unroll
      for (int i = 0; i < 8; ++i) turn.k1[i] = w[i];
    }
    const size_t y0 = size_t(out_row) * p.H[k.kind];

    for (int hb = k.h0; hb < k.h1; hb += ROWS) {
      ok = __all_sync(0xffffffffu, mbar_wait(ring.bar + ring.got % kDepth,
                                             (ring.got / kDepth) & 1, &abort_flag, p.status));
      if (!ok) break;
      const T* rows = reinterpret_cast<const T*>(ring.at(ring.got));
#pragma unroll
      for (int u = 0; u < ROWS / GROUPS; ++u) {
        const int h = hb + u * GROUPS + g;
        if (!live || hb + u * GROUPS >= k.h1) break;  // uniform: all lanes shuffle
        uint64_t x[8];
        Raw<T> raw;
        raw.load(rows + (u * GROUPS + g) * D, pc.a, pc.b);
        raw.get(x);
        float r = 1.f;
        if (norms) r = rsqrtf(row_sum<LPR>(dot16(x, x)) * (1.f / D) + p.eps);
        if (pc.on) {
          turn_row<INTER>(turn, x);
        } else if (norms) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = f2_mul(x[i], turn.k1[i]);
        }
        if (norms) {
          const uint64_t r2 = f2_pack(r, r);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = f2_mul(x[i], r2);
        }
        if (h < k.h1) {
          const size_t off = (y0 + h) * D;
          if (k.kind > 0 && p.e4m3)
            store_row_e4m3(static_cast<uint8_t*>(p.y[k.kind]) + off, pc.a, pc.b, x,
                           p.inv_scale[k.kind - 1]);
          else
            store_row(static_cast<T*>(p.y[k.kind]) + off, pc.a, pc.b, x);
        }
      }
      ++ring.got;
      __syncwarp();  // every lane has read the stage
      put();
    }
  }
  if (!ok && lane == 0) {
    // let copies in flight land before the block exits
    const uint64_t w0 = globaltimer();
    while (globaltimer() - w0 < 1000000ull) {
    }
  }
}

// Backward: every block works on one kind, so that it sums its rows' weight
// gradients in registers and writes one partial; the order of every sum is
// fixed by the sizes alone.  A stage holds rows of x and of the upstream
// gradient.  WHOLE: a warp takes every so many-th token, whole.  Side by side
// the warps read faster than in ranges (49152 tokens of 40 heads: 291 us
// against 309), but with few tokens each the last round is half empty (6144
// tokens of 32 heads: 37.4 us against 35.9 in equal ranges).
template <typename T, int D, bool INTER, bool WHOLE>
__global__ void __launch_bounds__(kRowThreads, 2) rows_bwd_kernel(RowParams p) {
  constexpr int LPR = D / 16, GROUPS = 32 / LPR;
  constexpr int HALF = kStageBytes / 2;
  // at least one row group; fp32 rows of 16 lanes fill the stage with less
  constexpr int ROWS = HALF / (D * int(sizeof(T)));
  extern __shared__ __align__(128) uint8_t smem[];
  let_next_launch();
  __shared__ float red[kRowWarps][D];
  __shared__ uint64_t bars[kRowWarps][kDepth];
  __shared__ int abort_flag;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LPR, g = lane / LPR;
  if (threadIdx.x == 0) abort_flag = 0;
  __syncthreads();
  const int kind = int(blockIdx.x) < p.blocks_q ? 0 : 1;
  const int block = int(blockIdx.x) - (kind ? p.blocks_q : 0);
  const int blocks = kind ? int(gridDim.x) - p.blocks_q : p.blocks_q;
  const Pieces pc = pieces_of<INTER>(l, p.rot);
  const bool norms = p.w[kind] != nullptr;
  const int H = p.H[kind], per_token = p.stages[kind];
  uint64_t w[8], dw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i] = 0ull;
  if (norms) load_weight(p.w[kind], p.w_dtype, pc, w);
  const int warps = blocks * kRowWarps;
  Walk walk = WHOLE
                  ? make_strided_walk(block * kRowWarps + warp, warps, p.T, per_token)
                  : make_walk(block * kRowWarps + warp, p.share[kind], per_token);
  Ring ring = make_ring(smem, bars);

  // heads [h0, h1) of a token; the walk moves behind them
  auto next_rows = [&](Walk& at, int& t, int& h0, int& h1) {
    t = at.t;
    if (WHOLE) {
      h0 = 0;
      h1 = H;
      at.left -= per_token;
      at.t += at.step;
      return;
    }
    const int n = min(per_token - at.s, at.left);
    h0 = at.s * ROWS;
    h1 = min(h0 + n * ROWS, H);
    at.left -= n;
    at.s += n;
    if (at.s == per_token) at.s = 0, at.t += at.step;
  };
  Walk next = walk;
  int nt = 0, nh = 0, nh1 = 0;
  auto put = [&]() {
    if (nh >= nh1) {
      if (next.left == 0) return;
      next_rows(next, nt, nh, nh1);
    }
    if (lane == 0) {
      const uint32_t bytes = uint32_t(min(ROWS, nh1 - nh)) * D * sizeof(T);
      uint64_t* bar = ring.bar + ring.put % kDepth;
      const uint32_t dst = smem_u32(ring.at(ring.put));
      mbar_arrive_expect_tx(bar, norms ? 2 * bytes : bytes);
      bulk_load(dst, static_cast<const T*>(p.dy[kind]) + (int64_t(nt) * H + nh) * D, bytes, bar);
      if (norms)
        bulk_load(dst + HALF, static_cast<const T*>(p.x[kind]) + int64_t(nt) * p.xs[kind] +
                                  size_t(nh) * D, bytes, bar);
    }
    nh += ROWS;
    ++ring.put;
  };
#pragma unroll 1
  for (int i = 0; i < kDepth; ++i) put();

  bool ok = true;
  Place place = {};
  if (walk.left > 0) place = load_place(p, walk.t);
  while (ok && walk.left > 0) {
    int t, h0, h1;
    next_rows(walk, t, h0, h1);
    const Place here = place;
    if (walk.left > 0) place = load_place(p, walk.t);
    const bool live = place_turns(p, here, lane);
    Turn turn;
    if (pc.on && live)
      load_turn<INTER>(turn, p.cos_sin + int64_t(here.at) * p.rot, p.rot, l, -1.f);
    T* d0 = static_cast<T*>(p.y[kind]) + int64_t(t) * p.dxs[kind];
    for (int hb = h0; hb < h1; hb += ROWS) {
      ok = __all_sync(0xffffffffu, mbar_wait(ring.bar + ring.got % kDepth,
                                             (ring.got / kDepth) & 1, &abort_flag, p.status));
      if (!ok) break;
      const T* gr = reinterpret_cast<const T*>(ring.at(ring.got));
      const T* xr = reinterpret_cast<const T*>(ring.at(ring.got) + HALF);
#pragma unroll
      for (int u = 0; u < (ROWS + GROUPS - 1) / GROUPS; ++u) {
        const int i0 = u * GROUPS + g, h = hb + i0;
        if (!live || hb + u * GROUPS >= h1) break;  // uniform: all lanes shuffle
        // rows behind the last one: zeros, they add nothing to the sums
        const bool row = i0 < ROWS && h < h1;
        uint64_t dy[8];
        Raw<T> raw = {};
        if (row) raw.load(gr + i0 * D, pc.a, pc.b);
        raw.get(dy);
        if (pc.on) turn_row<INTER>(turn, dy);
        if (norms) {
          uint64_t x[8];
          raw = Raw<T>{};
          if (row) raw.load(xr + i0 * D, pc.a, pc.b);
          raw.get(x);
          const float ms = row_sum<LPR>(dot16(x, x)) * (1.f / D);
          // (without an eps a row of zeros has no root)
          const float r = row ? rsqrtf(ms + p.eps) : 0.f;
          const uint64_t r2 = f2_pack(r, r);
          uint64_t wg[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            wg[i] = f2_mul(w[i], dy[i]);
            dw[i] = f2_fma(f2_mul(dy[i], x[i]), r2, dw[i]);
          }
          const float e = -r * r * row_sum<LPR>(dot16(wg, x)) * (1.f / D);
          const uint64_t e2 = f2_pack(e, e);
#pragma unroll
          for (int i = 0; i < 8; ++i) dy[i] = f2_mul(r2, f2_fma(x[i], e2, wg[i]));
        }
        if (row) store_row(d0 + size_t(h) * D, pc.a, pc.b, dy);
      }
      ++ring.got;
      __syncwarp();  // every lane has read the stage
      put();
    }
  }
  if (!ok && lane == 0) {
    // let copies in flight land before the block exits
    const uint64_t w0 = globaltimer();
    while (globaltimer() - w0 < 1000000ull) {
    }
  }
  // the row groups of a warp, then the warps of the block
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint64_t v = dw[i];
#pragma unroll
    for (int off = LPR; off < 32; off <<= 1) v = f2_add(v, __shfl_xor_sync(0xffffffffu, v, off));
    float* at = red[warp] + (i < 4 ? pc.a : pc.b) + 2 * (i & 3);
    if (g == 0) f2_unpack(v, at[0], at[1]);
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
  wait_for_previous();
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

// Cache rows back to dense bf16.  A group of lanes (a power of two that covers
// the row, 32 at most) takes a row of K and of V in pieces of 8 elements, kReadUnroll
// of them on the way, and has its next row's number already.  (Pieces of 16
// e4m3 codes load wider but store every other 16 bytes: 84 against 66 us for
// 65536 rows of 1 KB.)  A row outside the cache gives zeros and a report.
constexpr int kReadUnroll = 4;
template <bool E4M3>
__global__ void __launch_bounds__(256) cache_read_kernel(
    const void* kc, const void* vc, const int32_t* rows, int64_t n, int64_t n_cache, int pieces,
    int group_log2, float k_scale, float v_scale, uint4* k, uint4* v, int32_t* status) {
  using Piece = std::conditional_t<E4M3, uint2, uint4>;
  const int64_t thread = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t step = (int64_t(gridDim.x) * blockDim.x) >> group_log2;
  const int group = 1 << group_log2, lane = int(thread) & (group - 1);
  int64_t r = thread >> group_log2;
  int32_t next = r < n ? __ldg(rows + r) : 0;
  for (; r < n; r += step) {
    const int32_t row = next;
    if (r + step < n) next = __ldg(rows + r + step);
    const bool ok = row >= 0 && row < n_cache;
    if (!ok && lane == 0) report_status(status, PSA_ERR_INVALID_ARG);
    const Piece* src[2] = {static_cast<const Piece*>(kc) + size_t(ok ? row : 0) * pieces,
                           static_cast<const Piece*>(vc) + size_t(ok ? row : 0) * pieces};
    uint4* dst[2] = {k + size_t(r) * pieces, v + size_t(r) * pieces};
    for (int c0 = lane; c0 < pieces; c0 += kReadUnroll * group) {
      Piece in[kReadUnroll][2];
#pragma unroll
      for (int u = 0; u < kReadUnroll; ++u)
#pragma unroll
        for (int which = 0; which < 2; ++which) {
          in[u][which] = Piece{};
          if (ok && c0 + u * group < pieces) in[u][which] = __ldg(src[which] + c0 + u * group);
        }
#pragma unroll
      for (int u = 0; u < kReadUnroll; ++u)
#pragma unroll
        for (int which = 0; which < 2; ++which) {
          uint4 out;
          if constexpr (E4M3) {
            const float sc = which ? v_scale : k_scale;
            const uint32_t w[2] = {in[u][which].x, in[u][which].y};
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                  __nv_fp8x2_storage_t(w[j / 2] >> (16 * (j & 1))), __NV_E4M3);
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
              o[j] = pack_bf16(f.x * sc, f.y * sc);
            }
            out = make_uint4(o[0], o[1], o[2], o[3]);
          } else {
            out = in[u][which];
          }
          if (c0 + u * group < pieces) dst[which][c0 + u * group] = out;
        }
    }
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

// Launches with the ring's shared memory (opted in once per device).
template <void (*KERNEL)(RowParams)>
int launch_ring(uint32_t grid, cudaStream_t stream, const RowParams& p) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PSA_ERR_CUDA;
  if (dev >= 64 || !(done.load(std::memory_order_acquire) >> dev & 1)) {
    if (cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int(kRowSmem)) != cudaSuccess)
      return PSA_ERR_CUDA;
    if (dev < 64) done.fetch_or(uint64_t(1) << dev, std::memory_order_release);
  }
  KERNEL<<<grid, kRowThreads, kRowSmem, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? PSA_OK : PSA_ERR_CUDA;
}

// Stages of `rows` heads that a token has in each kind.
void count_stages(RowParams& p, int rows) {
  for (int k = 0; k < 3; ++k) p.stages[k] = int32_t((int64_t(p.H[k]) + rows - 1) / rows);
}

// `blocks` blocks' warps over n stages.
Share share_of(int64_t n, int64_t blocks) {
  const int64_t warps = blocks * kRowWarps;
  if (warps == 0) return {};
  return {int32_t(n / warps), int32_t(n % warps), int32_t(warps)};
}

template <typename T, int D>
int launch_rows_d(const RowsArgs& a) {
  RowParams p = row_params(a);
  count_stages(p, kStageBytes / (D * int(sizeof(T))));
  // two blocks per SM, or as many as give every warp a stage
  const int64_t all = int64_t(p.T) * (int64_t(p.stages[0]) + p.stages[1] + p.stages[2]);
  int64_t grid = (all + kRowWarps - 1) / kRowWarps;
  if (all > INT32_MAX) return PSA_ERR_INVALID_ARG;
  if (grid > kRowsBlocks) grid = kRowsBlocks;
  p.share[0] = share_of(all, grid);
  return a.how.interleaved ? launch_ring<rows_kernel<T, D, true>>(uint32_t(grid), a.stream, p)
                           : launch_ring<rows_kernel<T, D, false>>(uint32_t(grid), a.stream, p);
}

template <typename T, int D>
int launch_rows_bwd_d(const RowsBwdArgs& b) {
  RowParams p = row_params(b.rows);
  count_stages(p, kStageBytes / 2 / (D * int(sizeof(T))));
  p.dy[0] = b.dq_out, p.dy[1] = b.dk_out;
  p.dxs[0] = b.dq_stride, p.dxs[1] = b.dk_stride;
  p.part = b.part;
  // two blocks per SM in all, shared between the kinds by their rows
  int64_t need[2], blocks[2];
  for (int k = 0; k < 2; ++k) {
    if (int64_t(p.T) * p.stages[k] > INT32_MAX) return PSA_ERR_INVALID_ARG;
    need[k] = (int64_t(p.T) * p.stages[k] + kRowWarps - 1) / kRowWarps;
  }
  const int64_t H = int64_t(p.H[0]) + p.H[1];
  for (int k = 0; k < 2; ++k) {
    const int64_t share = H ? (kRowsBlocks * int64_t(p.H[k]) + H - 1) / H : 0;
    blocks[k] = need[k] < share ? need[k] : share;
  }
  if (blocks[0] + blocks[1] > kRowsBlocks) --blocks[blocks[0] > blocks[1] ? 0 : 1];
  p.blocks_q = int32_t(blocks[0]);
  for (int k = 0; k < 2; ++k) p.share[k] = share_of(int64_t(p.T) * p.stages[k], blocks[k]);
  const uint32_t grid = uint32_t(blocks[0] + blocks[1]);
  if (grid > 0) {  // without tokens the weight gradients are zero
    // sixteen tokens for every warp: the last round costs a few percent at most
    const bool whole = p.T >= 16 * int64_t(grid) * kRowWarps;
    const int rc =
        b.rows.how.interleaved
            ? (whole ? launch_ring<rows_bwd_kernel<T, D, true, true>>(grid, b.rows.stream, p)
                     : launch_ring<rows_bwd_kernel<T, D, true, false>>(grid, b.rows.stream, p))
            : (whole ? launch_ring<rows_bwd_kernel<T, D, false, true>>(grid, b.rows.stream, p)
                     : launch_ring<rows_bwd_kernel<T, D, false, false>>(grid, b.rows.stream, p));
    if (rc != PSA_OK) return rc;
  }
  if (!b.dq_weight && !b.dk_weight) return PSA_OK;
  return launch_behind(weight_sum_kernel, dim3(D / 32, 2), 256, b.rows.stream,
                       static_cast<const float*>(b.part), int(p.blocks_q), int(grid), D,
                       b.dq_weight, b.dk_weight) == cudaSuccess
             ? PSA_OK
             : PSA_ERR_CUDA;
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
  const int pieces = a.Hkv * a.D / 8;
  int group_log2 = 0;
  while (group_log2 < 5 && (1 << group_log2) < pieces) ++group_log2;
  // at most sixteen blocks of 256 threads per SM (two rounds), each group on
  // several rows; 65536 rows: 66 us, 70 with eight
  const int64_t blocks = ((a.n << group_log2) + 255) / 256;
  const uint32_t grid = uint32_t(blocks < int64_t(sms) * 16 ? blocks : int64_t(sms) * 16);
  auto kern = a.e4m3 ? cache_read_kernel<true> : cache_read_kernel<false>;
  kern<<<grid, 256, 0, a.stream>>>(a.kc, a.vc, a.rows, a.n, a.n_cache, pieces, group_log2,
                                   a.k_scale, a.v_scale, static_cast<uint4*>(a.k),
                                   static_cast<uint4*>(a.v), a.status);
  return cudaGetLastError() == cudaSuccess ? PSA_OK : PSA_ERR_CUDA;
}

}  // namespace psa
