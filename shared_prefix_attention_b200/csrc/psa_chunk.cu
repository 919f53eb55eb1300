// Chunk attention: each request's new tokens over its cached keys (the new
// tokens' own among them), read through a token-granular page table or from
// a contiguous range, bf16 or e4m3, optionally within a sliding window and
// with logits capped by a tanh:
//   s_ij = scale q_i.k_j           (capped: c tanh(s_ij / c))
//   p_ij = exp(s_ij) for the keys j in (pos_i - window, pos_i], else 0
//   o_i  = sum_j p_ij v_j / sum_j p_ij,   lse_i = log sum_j p_ij
//
// The work is 4 d FLOP per visible (query row, key) pair, and the cache is
// read once per block of query rows, so long chunks are bound by the tensor
// cores and the exponentials, and single tokens by the cache's bytes.
//
// A KV head's query rows are packed (token, head of the group) into 128-row
// tiles, so one K/V tile serves all heads of the group.  A CTA (one per SM)
// walks its list of units (query block, KV head, key range) with two row
// halves on one K/V tile stream, or, where the rows fit one half ("twin"),
// with both halves on the same rows and alternate tiles: then each half keeps
// its own running max and sum and writes its own partial.
//   warps 0, 2   loaders of K (and the query rows, by TMA) and of V, in the
//                wide form with two more each.  A page table scatters a tile's
//                keys, so their rows are gathered with 16-byte asynchronous
//                copies straight into the 128-byte-swizzled tiles the MMA
//                reads, zeros behind the key range (no unused cache row is
//                touched); whole tiles of a contiguous bf16 range come by TMA.
//                e4m3 rows go through a thread-private staging area and are
//                widened to f16 (exact) by the thread that copied them.  The
//                loaders share their schedulers with the softmax warps, which
//                leave few issue slots: an earlier form that computed each
//                copy's addresses took 7500 cycles per tile where this one
//                takes under 3000 (four-row TMA gathers move half as much as
//                these copies: 21 against 41 bytes per clock and SM).
//   warp 1       tcgen05 issuer: per half S = Q K^T into TMEM, O += P V with P
//                read from TMEM over the S columns.  The whole warp walks in
//                step so that descriptors stay in uniform registers (a single
//                lane in a divergent branch issued at half the rate), and
//                waits for everything but P first.
//   warps 4..11  softmax of the two halves, one row per thread, running max in
//                the log2 domain with lazy rescaling, and the epilogue: final
//                rows, or a partial (O / l and log2-sum-exp, fp32) for the
//                join kernel.
// What bounds it (one long prompt's piece, 2048 tokens over 16k keys: 470 us =
// 1.24 PFLOP/s in runs of a few ms; 546 us = 1.07 PFLOP/s in long ones, whose
// SM clock the power limit holds at 1.66 GHz): the special-function unit and
// the tensor pipe are each busy 60 % of the time; a tile's chain QK, softmax,
// PV (about 3400 cycles) is longer than either's share of it (2050), and two
// halves are all that TMEM holds.  Over a page table the gather of a tile takes
// nearly as long as that chain.
// P is rounded to bf16 (f16 over an e4m3 cache) for the tensor cores: at most
// half a step per weight, averaged over the keys; the sum l keeps fp32.  f16
// steps stop shrinking at 2^-14, so those weights are held 2^7 up (kLift): one
// far below the row's largest is off by at most 2^-32 of it.
// Every wait is bounded.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <atomic>

#include "psa_chunk.h"
#include "psa_debug.cuh"
#include "psa_device.cuh"
#include "psa_internal.h"
#include "psa_pair.cuh"
#include "psa_tmem_wide.cuh"

namespace psa {
namespace {

constexpr int BM = 128;            // query rows per half
constexpr int BN = kChunkTile;     // keys per tile
// The narrow form: 12 warps, 168 registers a thread at launch = 64512 = 128 x
// 104 (loaders, MMA) + 256 x 200 (softmax: a whole 128-column S row in
// registers); the launcher checks the compiled count before the first launch.
// The wide form: 16 warps of 128 registers, more loaders, and a softmax that
// reads its rows in halves.
constexpr int kRegsLaunch = 168;
constexpr int kRegsLow = 104, kRegsSoftmax = 200;
constexpr int kWideLoaders = 3, kWideParts = 8;
template <bool WIDE>
constexpr int threads() { return WIDE ? 512 : 384; }
static_assert(128 * kRegsLow + 256 * kRegsSoftmax <= threads<false>() * kRegsLaunch,
              "register split");
constexpr float kRescaleLog2 = 8.f;
// Weights are 2^(logit - max + kLift): with a max that lags by kRescaleLog2 at
// most 2^15, which f16 holds (65504).  Unlifted, 64k equal keys beside one with
// 99 % of the weight had weights of 2 to 4 steps each: o was 5.5 % off.
template <bool F16>
constexpr float kLift = F16 ? 7.f : 0.f;
constexpr uint32_t kTmemCols = 512;  // per half: S at X*256, O at X*256 + 128

template <int D, bool E4M3, bool WIDE>
struct Cfg {
  static constexpr int NPART = D / 64;  // 128-byte swizzle atoms across d
  static constexpr uint32_t Q_BYTES = BM * D * 2;  // one half
  static constexpr uint32_t KV_BYTES = BN * D * 2;
  static constexpr int ROWB = E4M3 ? D : 2 * D;    // bytes of a cached row
  static constexpr int CPR = ROWB / 16;            // 16-byte copies of a row
  static constexpr int RPI = 32 / CPR;             // rows per warp instruction
  static constexpr int RG = 8 / RPI;               // instructions per 8 rows
  static constexpr int PARTS = WIDE ? kWideParts : 4;  // a tile is loaded in parts
  static constexpr int NPP = BN / 8 * RG / PARTS;  // instructions per part
  static constexpr int LOADERS = WIDE ? kWideLoaders : 1;  // warps of K, and of V
  static constexpr int MINE = (PARTS + LOADERS - 1) / LOADERS;  // parts of a warp at most
  static constexpr uint32_t STAGE_BYTES = E4M3 ? BN * D : 0;  // raw K (or V) tile
  static constexpr int NSK = D == 64 ? 4 : (E4M3 ? 2 : 3);
  static constexpr int NSV = D == 64 ? 4 : 2;
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_K = OFF_Q + 2 * Q_BYTES;
  static constexpr uint32_t OFF_V = OFF_K + NSK * KV_BYTES;
  static constexpr uint32_t OFF_STAGE = OFF_V + NSV * KV_BYTES;
  static constexpr uint32_t OFF_BAR = OFF_STAGE + 2 * STAGE_BYTES;
  static constexpr uint32_t NBAR = 3 + 2 * NSK + 2 * NSV + 8;
  static constexpr uint32_t SMEM = 1024 + OFF_BAR + NBAR * 8 + 16;
};

struct Params {
  const int32_t* plan;
  int32_t n_ctas, n_units, n_joins;
  const uint8_t* kc;
  const uint8_t* vc;
  int64_t n_cache;
  const int32_t* kv_indices;
  int64_t n_keys;
  __nv_bfloat16* o;
  bool o_wide;  // o is 32-byte aligned
  float* lse;
  int32_t n_rows, Hq, Hkv, G, TPH, window;
  float scale_log2;  // logits in the log2 domain; capped: 2 log2e scale / cap
  float cap_log2;    // cap * log2e
  float v_scale;
  float* part_o;
  float* part_lse;
  int64_t part_rows;
  int32_t* status;
};

// One unit of the plan as every role sees it.
struct Unit {
  int q0, ntok, pos0, kvh, kv0, t0, t1, twin, part;
  bool ok;  // inside the buffers (debug build); otherwise every role skips it
};

__device__ __forceinline__ Unit load_unit(const Params& p, const int4* units, int u) {
  const int4 a = __ldg(units + 3 * u), b = __ldg(units + 3 * u + 1);
  Unit x;
  x.q0 = a.x, x.ntok = a.y, x.pos0 = a.z, x.kvh = a.w;
  x.kv0 = b.x, x.t0 = b.y, x.t1 = b.z, x.twin = b.w;
  x.part = __ldg(reinterpret_cast<const int32_t*>(units + 3 * u + 2));
  x.ok = psa_in_bounds(
      x.q0 >= 0 && x.ntok > 0 && x.ntok <= (x.twin ? 1 : 2) * p.TPH &&
          int64_t(x.q0) + x.ntok <= p.n_rows && x.kvh >= 0 && x.kvh < p.Hkv && x.kv0 >= 0 &&
          x.t0 >= 0 && x.t1 > x.t0 && int64_t(x.kv0) + x.t1 <= p.n_keys && x.part >= -1 &&
          (x.part < 0 || x.part + int64_t(x.twin ? 2 : 1) * x.ntok * p.G <= p.part_rows),
      p.status);
  return x;
}

// Tokens and first position of half x (both halves have the same in a twin).
__device__ __forceinline__ int half_tokens(const Unit& u, int x, int TPH) {
  return u.twin ? u.ntok : (x ? u.ntok - TPH : min(u.ntok, TPH));
}
__device__ __forceinline__ int half_pos(const Unit& u, int x, int TPH) {
  return u.pos0 + (u.twin ? 0 : x * TPH);
}

// Whether half x takes part in the tile at key t.
__device__ __forceinline__ bool half_sees(const Unit& u, int x, int t, int TPH, int window) {
  if (u.twin) return (((t - u.t0) >> 7) & 1) == x;
  const int first = half_pos(u, x, TPH), n = half_tokens(u, x, TPH);
  return t <= first + n - 1 && (window == 0 || min(t + BN, u.t1) - 1 > first - window);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(live ? 16u : 0u)
               : "memory");
}
// Arrives on `bar` once every cp.async this thread issued so far has landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Four e4m3 codes to two f16 pairs (exact).
__device__ __forceinline__ uint2 e4m3x4_to_f16(uint32_t w) {
  uint2 r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(r.x), "=r"(r.y)
      : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w) {
  const __half2 h = __floats2half2_rn(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <bool F16>
__device__ __forceinline__ uint32_t pack_p(float lo, float hi) {
  if constexpr (F16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    return pack_bf16(lo, hi);
  }
}
// 32 bytes in one store: half the store instructions of 16-byte ones (a warp's
// store touches 32 rows).
__device__ __forceinline__ void store32(void* dst, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Logits outside [lo, hi) become the mark of a masked one, whose weight is
// exactly 0: -inf, or with a cap the lowest finite number, since a logit of
// -inf (an infinite key) has the weight of -c there.  (Finding the masked ones
// by their positions again took 2 % longer than comparing with the mark.)
template <bool CAP>
constexpr uint32_t kMasked = CAP ? 0xff7fffffu : 0xff800000u;
template <bool CAP, int N>
__device__ __forceinline__ void mask_row(uint32_t (&s)[N], int lo, int hi) {
#pragma unroll
  for (int w = 0; w < N / 32; ++w) {
    const int a = min(max(lo - 32 * w, 0), 32), b = min(max(hi - 32 * w, 0), 32);
    const uint32_t below_b = b == 32 ? 0xffffffffu : ((1u << b) - 1u);
    const uint32_t below_a = a == 32 ? 0xffffffffu : ((1u << a) - 1u);
    const uint32_t keep = below_b & ~below_a;
#pragma unroll
    for (int k = 0; k < 32; ++k)
      if (!((keep >> k) & 1u)) s[32 * w + k] = kMasked<CAP>;
  }
}

__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }
template <int N>
__device__ __forceinline__ float max_of_row(const uint32_t (&s)[N]) {
  float v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(s[k]);
#pragma unroll
  for (int k = 8; k < N - 8; k += 16)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = max3(v[i], __uint_as_float(s[k + i]), __uint_as_float(s[k + 8 + i]));
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = max3(v[i], v[i + 4], __uint_as_float(s[N - 8 + i]));
  v[0] = max3(v[0], v[1], __uint_as_float(s[N - 4]));
  v[2] = max3(v[2], v[3], __uint_as_float(s[N - 3]));
  return fmaxf(max3(v[0], v[2], __uint_as_float(s[N - 2])), __uint_as_float(s[N - 1]));
}

// kind::f16 with f16 or bf16 operands and fp32 accumulation.
template <bool F16>
__host__ __device__ constexpr uint32_t idesc_of(uint32_t M, uint32_t N, bool b_mn) {
  return (1u << 4) | (F16 ? 0u : (1u << 7) | (1u << 10)) | (uint32_t(b_mn) << 16) |
         ((N >> 3) << 17) | ((M >> 4) << 24);
}

// The log2-domain logit of a raw one.  Capped: c tanh(s / c) = c - 2 c / (1 +
// exp(2 s / c)); its error is absolute (1.4e-6 c at most), as a weight needs it.
template <bool CAP>
__device__ __forceinline__ float to_log2(float s, const Params& p) {
  if constexpr (CAP)
    return s == -INFINITY ? s
                          : fmaf(fast_rcp(1.f + fast_exp2(s * p.scale_log2)), -2.f * p.cap_log2,
                                 p.cap_log2);
  else
    return s * p.scale_log2;
}

// Weights of a row of logits, 2^(logit + neg_m), packed in pairs into the
// row's first half (pair k over logit k <= 2 k, which is done by then);
// returns their fp32 sum.
template <bool F16, int N, int K0 = 0, int K1 = N / 2>
__device__ __forceinline__ float weights_row(uint32_t (&s)[N], float neg_m, const Params& p) {
  const uint64_t sc2 = f2_pack(p.scale_log2, p.scale_log2), nm2 = f2_pack(neg_m, neg_m);
  uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
  for (int k = K0; k < K1; ++k) {
    float x0, x1;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])), sc2, nm2),
              x0, x1);
    const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
    acc[k & 3] = f2_add(acc[k & 3], f2_pack(p0, p1));
    s[k] = pack_p<F16>(p0, p1);
  }
  float v[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) f2_unpack(acc[k], v[2 * k], v[2 * k + 1]);
  return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
}

// min(a, b), NaN if either is (a NaN logit must not become a capped one).
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// The same of capped logits.  With e = exp(2 s / c) a weight is 2^(c' - m - 2
// c' / (1 + e)), c' = c log2(e): two exponentials and a reciprocal, which would
// leave the special-function unit a third of the uncapped rate.  So four
// reciprocals come from that of the four's product (e is held below 2^30,
// where the cap is reached to 1e-9, so the product stays finite).  With U half a
// step of fp32, 1 / (1 + e) is off by 7 U of itself (sum, two products, 2 U of
// the reciprocal, two products) and 2 U (a quarter of the exponential's and its
// argument's), which counts twice c'; c', the offset, the last sum: 24 U c' in
// all (test: logits to 4.5 c at c = 1000).  (A part of the first exponentials
// by a polynomial on the FMA pipe changed the time by 2 %; not kept.)
template <bool F16, bool MASKED, int N>
__device__ __forceinline__ float weights_row_capped(uint32_t (&s)[N], float neg_m,
                                                    const Params& p) {
  const uint64_t sc2 = f2_pack(p.scale_log2, p.scale_log2), one = f2_pack(1.f, 1.f);
  const uint64_t cap2 = f2_pack(-2.f * p.cap_log2, -2.f * p.cap_log2);
  const uint64_t top = f2_pack(neg_m + p.cap_log2, neg_m + p.cap_log2);
  uint64_t acc[2] = {0ull, 0ull};
#pragma unroll
  for (int k = 0; k < N / 4; ++k) {
    uint64_t e[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float x0, x1;
      f2_unpack(f2_mul(f2_pack(__uint_as_float(s[4 * k + 2 * j]),
                               __uint_as_float(s[4 * k + 2 * j + 1])), sc2), x0, x1);
      x0 = min_nan(x0, 30.f), x1 = min_nan(x1, 30.f);
      e[j] = f2_pack(fast_exp2(x0), fast_exp2(x1));
    }
    const uint64_t ab = f2_add(e[0], one), cd = f2_add(e[1], one);  // (a, b), (c, d)
    const uint64_t ac_bd = f2_mul(ab, cd);                          // (a c, b d)
    float ac, bd;
    f2_unpack(ac_bd, ac, bd);
    const float r = fast_rcp(ac * bd);
    const uint64_t rr = f2_mul(f2_pack(r, r), f2_pack(bd, ac));     // 1 / (a c), 1 / (b d)
    const uint64_t y[2] = {f2_fma(f2_mul(rr, cd), cap2, top), f2_fma(f2_mul(rr, ab), cap2, top)};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float x0, x1;
      f2_unpack(y[j], x0, x1);
      float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
      if (MASKED) {
        p0 = s[4 * k + 2 * j] == kMasked<true> ? 0.f : p0;
        p1 = s[4 * k + 2 * j + 1] == kMasked<true> ? 0.f : p1;
      }
      acc[j] = f2_add(acc[j], f2_pack(p0, p1));
      // packed behind the four's last use of its logits
      e[j] = pack_p<F16>(p0, p1);
    }
    s[2 * k] = uint32_t(e[0]);
    s[2 * k + 1] = uint32_t(e[1]);
  }
  float v[4];
  f2_unpack(acc[0], v[0], v[1]);
  f2_unpack(acc[1], v[2], v[3]);
  return (v[0] + v[1]) + (v[2] + v[3]);
}

template <int D, bool E4M3, bool CAP, bool WIDE>
__global__ void __launch_bounds__(threads<WIDE>(), 1)
    chunk_kernel(const __grid_constant__ CUtensorMap tmap_q,
                 const __grid_constant__ CUtensorMap tmap_k,
                 const __grid_constant__ CUtensorMap tmap_v, Params p) {
  using C = Cfg<D, E4M3, WIDE>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  __shared__ uint32_t tmem_base_slot;
  __shared__ int abort_flag;

  let_next_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const ChunkPlanView view(p.n_ctas, p.n_units, p.n_joins);
  if (__ldg(p.plan) != kChunkMagic || __ldg(p.plan + 1) != p.n_ctas ||
      __ldg(p.plan + 2) != p.n_units || __ldg(p.plan + 3) != p.n_joins) {
    if (threadIdx.x == 0) report_status(p.status, PSA_ERR_INVALID_ARG);
    return;
  }
  const int4* units = reinterpret_cast<const int4*>(p.plan + view.units);
  int u_first = __ldg(p.plan + view.lists + blockIdx.x);
  int u_end = __ldg(p.plan + view.lists + blockIdx.x + 1);
  if (!psa_in_bounds(u_first >= 0 && u_first <= u_end && u_end <= p.n_units, p.status))
    u_first = u_end = 0;

  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* q_full = bar;       // TMA bytes
  uint64_t* q_conv = bar + 1;   // e4m3: the softmax warps have widened Q to f16
  uint64_t* q_empty = bar + 2;  // MMA commit
  uint64_t* k_full = bar + 3;
  uint64_t* k_empty = k_full + C::NSK;
  uint64_t* v_full = k_empty + C::NSK;
  uint64_t* v_empty = v_full + C::NSV;
  uint64_t* s_full = v_empty + C::NSV;  // [2] each, one per half
  uint64_t* p_full = s_full + 2;
  uint64_t* pv_done = p_full + 2;
  uint64_t* o_free = pv_done + 2;

  if (threadIdx.x == 0) {
    abort_flag = 0;
    mbar_init(q_full, 1);
    mbar_init(q_conv, 8);
    mbar_init(q_empty, 1);
    for (int i = 0; i < C::NSK; ++i) {
      mbar_init(k_full + i, C::LOADERS * 32);
      mbar_init(k_empty + i, 1);
    }
    for (int i = 0; i < C::NSV; ++i) {
      mbar_init(v_full + i, C::LOADERS * 32);
      mbar_init(v_empty + i, 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(s_full + x, 1);
      mbar_init(p_full + x, 4);
      mbar_init(pv_done + x, 1);
      mbar_init(o_free + x, 4);
    }
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_slot;

  if (warp < 4 || warp >= 12) {
    if constexpr (!WIDE)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow) : "memory");
    if (warp == 0 || warp == 2 || (warp >= 12 && warp < 10 + 2 * C::LOADERS)) {
      // ================================================================ loaders
      // Warp 0 loads K (and the query rows), warp 2 loads V, in the wide form
      // with the help of warps 12, 14 and 13, 15; the rings advance on their
      // own.  A tile is made in parts: of the groups of 8 rows, part v takes
      // the RPI ones at (v % RG) * RPI.  A lane's rows of a part then all have
      // the same place in the swizzle, so its copies differ by constant
      // offsets, and one page-table entry per lane covers the part.
      const bool is_k = (warp & 1) == 0 && warp != 2;
      const int v0 = (warp < 12 ? 0 : (warp - 10) / 2) * C::MINE;
      const int n_mine = min(C::MINE, C::PARTS - v0);
      const int sub = lane / C::CPR, chunk = lane % C::CPR;
      if (lane == 0) {
        if (warp == 0) tma_prefetch_desc(&tmap_q);
        if (!E4M3 && !p.kv_indices) tma_prefetch_desc(is_k ? &tmap_k : &tmap_v);
      }
      const uint8_t* cache = (is_k ? p.kc : p.vc) + chunk * 16;
      uint64_t* full = is_k ? k_full : v_full;
      uint64_t* empty = is_k ? k_empty : v_empty;
      const uint32_t n_slots = is_k ? C::NSK : C::NSV;
      uint8_t* ring = smem + (is_k ? C::OFF_K : C::OFF_V);
      uint8_t* stage = smem + C::OFF_STAGE + (is_k ? 0 : C::STAGE_BYTES) + lane * 16;
      const size_t row_bytes = size_t(p.Hkv) * C::ROWB;
      auto first_row = [](int v) { return v / C::RG * C::NPP * 8 + v % C::RG * C::RPI; };
      const int lane_row = lane / C::RPI * 8 + lane % C::RPI;  // of a lane's table entry

      int u = u_first - 1, t = 0;
      Unit cur = {};  // the unit of the tile whose rows are at hand
      bool more = true, all = false;
      int32_t entry[C::MINE] = {};  // cache rows of this lane's table entries, -1: zeros
      const uint8_t* head = nullptr;
      // Moves on to the next tile and reads its page-table entries.
      auto advance = [&]() {
        t += BN;
        if (u < u_first || t >= cur.t1) {
          do {
            if (++u >= u_end) {
              more = false;
              return;
            }
            cur = load_unit(p, units, u);
          } while (!cur.ok);
          t = cur.t0;
          head = cache + size_t(cur.kvh) * C::ROWB;
        }
#pragma unroll
        for (int v = 0; v < C::MINE; ++v) {
          const int pos = t + first_row(v0 + v) + lane_row;
          entry[v] = -1;
          if (v < n_mine && lane < C::NPP * C::RPI && pos < cur.t1) {
            const int64_t flat = int64_t(cur.kv0) + pos;
            entry[v] = p.kv_indices ? __ldg(p.kv_indices + flat) : int32_t(flat);
          }
        }
      };
      // Rows outside the cache become zeros and a report.
      auto check = [&]() {
        bool good = true;
#pragma unroll
        for (int v = 0; v < C::MINE; ++v) {
          if (v < n_mine && lane < C::NPP * C::RPI && (entry[v] < 0 || entry[v] >= p.n_cache)) {
            if (t + first_row(v0 + v) + lane_row < cur.t1) report_status(p.status, PSA_ERR_INVALID_ARG);
            entry[v] = -1;
            good = false;
          }
        }
        all = __all_sync(0xffffffffu, good);
      };
      // one part: asynchronous copies of this lane's pieces, `step` bytes apart
      auto copy_part = [&](int v, uint32_t dst, uint32_t step) {
        if (all) {
#pragma unroll
          for (int n = 0; n < C::NPP; ++n)
            cp_async16(dst + n * step,
                       head + uint32_t(__shfl_sync(0xffffffffu, entry[v], n * C::RPI + sub)) *
                                  row_bytes);
        } else {
#pragma unroll 1
          for (int n = 0; n < C::NPP; ++n) {
            const int32_t e = __shfl_sync(0xffffffffu, entry[v], n * C::RPI + sub);
            cp_async16_or_zero(dst + n * step, head + size_t(max(e, 0)) * row_bytes, e >= 0);
          }
        }
      };
      // e4m3: this lane's staged pieces of a part (16 codes each) to f16
      auto widen_part = [&](int v, uint8_t* dst) {
        const uint32_t row = uint32_t(first_row(v0 + v) + sub), c0 = 2 * (chunk & 3);
        dst += uint32_t(chunk >> 2) * (BN * 128);
        uint8_t* at0 = dst + sw128(row, c0);
        uint8_t* at1 = dst + sw128(row, c0 + 1);
        const uint8_t* src = stage + (v0 + v) * C::NPP * 512;
#pragma unroll
        for (int n = 0; n < C::NPP; ++n) {
          const uint4 w = *reinterpret_cast<const uint4*>(src + n * 512);
          const uint2 a = e4m3x4_to_f16(w.x), b = e4m3x4_to_f16(w.y);
          const uint2 c = e4m3x4_to_f16(w.z), d = e4m3x4_to_f16(w.w);
          *reinterpret_cast<uint4*>(at0 + n * 1024) = make_uint4(a.x, a.y, b.x, b.y);
          *reinterpret_cast<uint4*>(at1 + n * 1024) = make_uint4(c.x, c.y, d.x, d.y);
        }
      };
      auto stage_part = [&](int v) {
        if (more) copy_part(v, smem_u32(stage) + (v0 + v) * C::NPP * 512, 512);
        cp_async_commit();
      };

      bool ok = true;
      advance();
      // the tile being made: whether there is one, and its unit's query rows
      // when it is the unit's first (e4m3 runs a tile ahead with its copies)
      bool now = more, first = true;
      int4 qbox = make_int4(cur.q0, cur.kvh, cur.twin, 0);
      if (E4M3 && more) {
        check();
#pragma unroll
        for (int v = 0; v < C::MINE; ++v)
          if (v < n_mine) stage_part(v);
        advance();
      }
      uint32_t slot = 0, phase = 0, uc = 0;
      while (now) {
        ok = __all_sync(0xffffffffu, mbar_wait(empty + slot, phase ^ 1, &abort_flag, p.status));
        if (!ok) break;
        uint8_t* dst = ring + slot * C::KV_BYTES;
        if constexpr (E4M3) {
          if (more) check();
#pragma unroll
          for (int v = 0; v < C::MINE; ++v) {
            if (v >= n_mine) break;
            // this part's copies: the oldest group
            if (n_mine == C::MINE)
              cp_async_wait<C::MINE - 1>();
            else
              cp_async_wait<C::MINE - 2>();
            widen_part(v, dst);
            stage_part(v);
          }
          fence_proxy_async_smem();
          mbar_arrive(full + slot);
        } else {
          if (!p.kv_indices && t + BN <= cur.t1) {
            // a whole tile of a contiguous range: one TMA copy
            if (lane == 0 && warp < 12) {
              mbar_arrive_expect_tx(full + slot, C::KV_BYTES);
#pragma unroll
              for (int part = 0; part < C::NPART; ++part)
                tma_load_3d(dst + part * BN * 128, is_k ? &tmap_k : &tmap_v, full + slot,
                            part * 64, cur.kvh, cur.kv0 + t);
            } else {
              mbar_arrive(full + slot);
            }
          } else {
            check();
#pragma unroll
            for (int v = 0; v < C::MINE; ++v)
              if (v < n_mine)
                copy_part(v, smem_u32(dst) + uint32_t(chunk >> 3) * (BN * 128) +
                                 sw128(uint32_t(first_row(v0 + v) + sub), chunk & 7), 1024);
            cp_async_arrive(full + slot);
          }
        }
        if (first && warp == 0) {
          // the query rows, behind the unit's first K tile
          if (lane == 0) {
            ok = mbar_wait(q_empty, (uc & 1) ^ 1, &abort_flag, p.status);
            if (ok) {
              mbar_arrive_expect_tx(q_full, 2 * C::NPART * uint32_t(p.TPH) * p.G * 128);
#pragma unroll
              for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int part = 0; part < C::NPART; ++part)
                  tma_load_3d(smem + C::OFF_Q + x * C::Q_BYTES + part * BM * 128, &tmap_q, q_full,
                              part * 64, qbox.y * p.G, qbox.x + (qbox.z ? 0 : x * p.TPH));
            }
          }
          ++uc;
          ok = __shfl_sync(0xffffffffu, int(ok), 0);
          if (!ok) break;
        }
        if constexpr (E4M3) {
          now = more;
          first = more && t == cur.t0;
          if (first) qbox = make_int4(cur.q0, cur.kvh, cur.twin, 0);
          if (more) advance();
        } else {
          advance();
          now = more;
          first = more && t == cur.t0;
          if (first) qbox = make_int4(cur.q0, cur.kvh, cur.twin, 0);
        }
        if (++slot == n_slots) slot = 0, phase ^= 1;
      }
      // every copy this thread issued lands before the CTA can exit
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (!ok || abort_flag) {
        const uint64_t w0 = globaltimer();
        while (globaltimer() - w0 < 1000000ull) {
        }
      }
    } else if (warp == 1) {
      // ================================================================ MMA issuer
      // The whole warp walks the units and waits (every value below is the
      // same in all lanes, so descriptors and branches stay in uniform
      // registers); one elected lane issues.
      const uint32_t idesc_qk = idesc_of<E4M3>(BM, BN, false);
      const uint32_t idesc_pv = idesc_of<E4M3>(BM, D, true);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint64_t dQ = umma_desc_sw128(smem_u32(smem + C::OFF_Q), 16, 1024);
      const uint64_t dK = umma_desc_sw128(smem_u32(smem + C::OFF_K), 16, 1024);
      const uint64_t dV = umma_desc_sw128(smem_u32(smem + C::OFF_V), BN * 128, 1024);
      uint32_t sk = 0, kph = 0, sv = 0, vph = 0;  // ring slots of the next K / V tile
      uint32_t uc = 0;
      uint32_t pvc[2] = {0, 0};  // PVs issued per half (all units)
      uint32_t uhc[2] = {0, 0};  // units in which the half had work
      bool ok = true;

      auto wait = [&](uint64_t* b, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(b, parity, &abort_flag, p.status));
      };
      // Called by one lane.  S_X = Q_X K^T into the S columns of half x:
      auto mma_qk = [&](int x) {
        const uint64_t a = dQ + x * (C::Q_BYTES >> 4), b = dK + sk * (C::KV_BYTES >> 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = ((ks >> 2) * (BM * 128) + (ks & 3) * 32) >> 4;
          umma_ss(tm + x * 256, a + off, b + off, idesc_qk, ks > 0 ? 1u : 0u);
        }
        umma_commit(s_full + x);
      };
      // O_X += P_X V, P_X in TMEM over the first 64 columns of S_X:
      auto mma_pv = [&](int x, bool first) {
        const uint64_t b = dV + sv * (C::KV_BYTES >> 4);
#pragma unroll
        for (int ks = 0; ks < BN / 16; ++ks)
          umma_ts(tm + x * 256 + 128, tm + x * 256 + ks * 8, b + ks * (2048 >> 4), idesc_pv,
                  (first && ks == 0) ? 0u : 1u);
        umma_commit(pv_done + x);
      };

      const int last = __shfl_sync(0xffffffffu, u_end, 0);
      for (int u = __shfl_sync(0xffffffffu, u_first, 0); u < last && ok; ++u) {
        const Unit w = load_unit(p, units, u);
        if (!w.ok) continue;
        const int n = __shfl_sync(0xffffffffu, (w.t1 - w.t0 + BN - 1) / BN, 0);
        const bool twin = __any_sync(0xffffffffu, w.twin);
        bool started[2] = {false, false};
        bool see[2];
#pragma unroll
        for (int x = 0; x < 2; ++x)
          see[x] = __any_sync(0xffffffffu, half_sees(w, x, w.t0, p.TPH, p.window));
        ok = wait(k_full + sk, kph) && wait(E4M3 ? q_conv : q_full, uc & 1);
        if (!ok) break;
        fence_proxy_async_smem();  // the loaders' copies, before the MMAs read them
        tc_fence_after();
        if (elect_one()) {
          if (see[0]) mma_qk(0);
          if (see[1]) mma_qk(1);
          umma_commit(k_empty + sk);
          if (n == 1) umma_commit(q_empty);
        }
        if (++sk == C::NSK) sk = 0, kph ^= 1;
        for (int j = 0; j < n; ++j) {
          // Everything but P is at hand before P is waited for, so that a
          // half's PV and its next QK follow its softmax at once.
          const bool more = j + 1 < n;
          bool next[2];
#pragma unroll
          for (int x = 0; x < 2; ++x)
            next[x] = more && __any_sync(0xffffffffu, half_sees(w, x, w.t0 + (j + 1) * BN, p.TPH,
                                                                p.window));
          ok = wait(v_full + sv, vph) && (!more || wait(k_full + sk, kph));
          if (!ok) break;
          fence_proxy_async_smem();
          // the other half of a twin has no P to come: it starts at once
          if (twin && more) {
            tc_fence_after();
            if (elect_one()) mma_qk(next[1]);
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (see[x]) {
              ok = (started[x] || wait(o_free + x, (uhc[x] & 1) ^ 1)) &&
                   wait(p_full + x, pvc[x] & 1);
              if (!ok) break;
              ++pvc[x];
            }
            tc_fence_after();
            if (elect_one()) {
              if (see[x]) mma_pv(x, !started[x]);
              if (next[x] && !twin) mma_qk(x);
              if (x == 1) {
                umma_commit(v_empty + sv);
                if (more) umma_commit(k_empty + sk);
                if (j + 2 == n) umma_commit(q_empty);
              }
            }
            started[x] = started[x] || see[x];
            see[x] = next[x];
          }
          if (!ok) break;
          if (++sv == C::NSV) sv = 0, vph ^= 1;
          if (more && ++sk == C::NSK) sk = 0, kph ^= 1;
        }
        if (!ok) break;
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (started[x]) ++uhc[x];
        ++uc;
      }
      if (!ok || abort_flag) {
        // give MMAs already issued time to finish before TMEM is freed
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 1000000ull) {
        }
      }
    }
  } else {
    if constexpr (!WIDE)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax) : "memory");
    // ================================================================ softmax + epilogue
    const int x = (warp - 4) >> 2;      // half
    const int quarter = warp & 3;       // TMEM lane quarter
    const int r = quarter * 32 + lane;  // row within the half
    const int tok = r / p.G, g = r - tok * p.G;
    const uint32_t trow = tmem + (uint32_t(quarter * 32) << 16) + x * 256;
    const uint32_t tS = trow, tO = trow + 128;
    uint32_t sc_count = 0;  // S tiles of this half consumed (all units)
    uint32_t uc = 0;
    for (int u = u_first; u < u_end; ++u) {
      const Unit w = load_unit(p, units, u);
      if (!w.ok) continue;
      if constexpr (E4M3) {
        // widen this thread's query row to f16, in place
        if (!mbar_wait(q_full, uc & 1, &abort_flag, p.status)) break;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          uint4* at = reinterpret_cast<uint4*>(smem + C::OFF_Q + x * C::Q_BYTES +
                                               (c >> 3) * (BM * 128) + sw128(r, c & 7));
          const uint4 v = *at;
          *at = make_uint4(bf16x2_to_f16x2(v.x), bf16x2_to_f16x2(v.y), bf16x2_to_f16x2(v.z),
                           bf16x2_to_f16x2(v.w));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_conv);
      }
      ++uc;
      const int ntok = half_tokens(w, x, p.TPH), pos_first = half_pos(w, x, p.TPH);
      const bool valid = tok < p.TPH && tok < ntok;
      const int pos = pos_first + tok;

      float m_run = -INFINITY, l_run = 0.f;
      int nt = 0;  // tiles of this half in this unit
      bool ok = true;
      for (int t = w.t0; t < w.t1; t += BN) {
        if (!half_sees(w, x, t, p.TPH, p.window)) continue;
        if (!mbar_wait(s_full + x, sc_count & 1, &abort_flag, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // some row of the half does not see the whole tile
        const bool masked = t + BN > w.t1 || t + BN - 1 > pos_first ||
                            (p.window && t <= pos_first + ntok - 1 - p.window);
        const int lo = p.window ? max(pos - p.window + 1 - t, 0) : 0;
        const int hi = min(pos + 1, w.t1) - t;

        // lazy rescaling: the max is raised when it grew by more than 2^8.  O
        // (the PVs of earlier tiles) is rescaled after P is stored, when the S
        // row no longer occupies registers; it only has to happen before this
        // tile's PV, which waits for p_full.
        float alpha = 1.f;
        auto raise = [&](float m_tile) {
          if (m_tile > m_run + kRescaleLog2) {
            alpha = fast_exp2(m_run - m_tile);
            l_run *= alpha;
            m_run = m_tile;
          }
          return m_run == -INFINITY ? 0.f : kLift<E4M3> - m_run;
        };
        if constexpr (CAP || WIDE) {
          // half a row at a time, read twice: a capped weight needs more
          // registers than a whole row leaves, and the wide form has fewer
          uint32_t sr[BN / 2];
          float mx = -INFINITY;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            tmem_ld64(tS + c * (BN / 2), sr);
            tmem_wait_ld();
            if (masked) mask_row<CAP>(sr, lo - c * (BN / 2), hi - c * (BN / 2));
            mx = fmaxf(mx, max_of_row(sr));
          }
          if constexpr (CAP) {
            // no logit above the lowest: none is seen, or those seen are at -c
            const float lowest = __uint_as_float(kMasked<true>);
            if (mx <= lowest) mx = lo < min(hi, BN) ? lowest : -INFINITY;
          }
          const float neg_m = raise(to_log2<CAP>(mx, p));
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            tmem_ld64(tS + c * (BN / 2), sr);
            tmem_wait_ld();
            if (masked) mask_row<CAP>(sr, lo - c * (BN / 2), hi - c * (BN / 2));
            if constexpr (!CAP)
              l_run += weights_row<E4M3>(sr, neg_m, p);
            else if (masked)
              l_run += weights_row_capped<E4M3, true>(sr, neg_m, p);
            else
              l_run += weights_row_capped<E4M3, false>(sr, neg_m, p);
            tmem_st32(tS + c * (BN / 4), *reinterpret_cast<uint32_t(*)[BN / 4]>(sr));
          }
        } else {
          // the whole S row in one TMEM load
          uint32_t sr[BN];
          tmem_ld128(tS, sr);
          tmem_wait_ld();
          if (masked) mask_row<CAP>(sr, lo, hi);
          const float neg_m = raise(to_log2<CAP>(max_of_row(sr), p));
          l_run += weights_row<E4M3, BN, 0, BN / 4>(sr, neg_m, p);
          tmem_st32(tS, *reinterpret_cast<uint32_t(*)[BN / 4]>(sr));
          l_run += weights_row<E4M3, BN, BN / 4, BN / 2>(sr, neg_m, p);
          tmem_st32(tS + 32, *reinterpret_cast<uint32_t(*)[BN / 4]>(sr + BN / 4));
        }
        if (nt > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          // wait for the latest PV into O, then scale O by alpha in place
          if (!mbar_wait(pv_done + x, (sc_count - 1) & 1, &abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t rr[32];
            tmem_ld32(tO + c * 32, rr);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) rr[k] = __float_as_uint(__uint_as_float(rr[k]) * alpha);
            tmem_st32(tO + c * 32, rr);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + x);
        ++sc_count;
        ++nt;
      }
      if (!ok) break;

      // this thread's row among the block's, and its partial
      const int brow = (w.twin ? 0 : x * p.TPH * p.G) + r, rows = w.ntok * p.G;
      const size_t part = size_t(w.part) + (w.twin ? x * rows : 0);
      if (nt == 0) {
        // no tile of this piece is this half's: an empty partial
        if (valid && w.part >= 0) p.part_lse[part + brow] = -INFINITY;
        continue;
      }
      // ---- epilogue: O / l straight from TMEM, LSE
      if (!mbar_wait(pv_done + x, (sc_count - 1) & 1, &abort_flag, p.status)) break;
      tc_fence_after();
      const float inv = l_run == 0.f ? 0.f : p.v_scale / l_run;
      const float lse2 = l_run == 0.f ? -INFINITY : m_run - kLift<E4M3> + __log2f(l_run);
      const size_t row = size_t(w.q0 + (w.twin ? 0 : x * p.TPH) + tok) * p.Hq + w.kvh * p.G + g;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t orr[32];
        tmem_ld32(tO + c * 32, orr);
        tmem_wait_ld();
        if (valid && w.part >= 0) {
          // partials are laid out [D / 4][rows][4]: the rows of a warp store
          // next to each other (row-major, 32 rows apart, a unit's epilogue
          // took 24000 cycles)
          float4* dst = reinterpret_cast<float4*>(p.part_o + part * D) + size_t(c) * 8 * rows + brow;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            dst[size_t(k) * rows] = make_float4(
                __uint_as_float(orr[4 * k]) * inv, __uint_as_float(orr[4 * k + 1]) * inv,
                __uint_as_float(orr[4 * k + 2]) * inv, __uint_as_float(orr[4 * k + 3]) * inv);
        } else if (valid) {
          uint32_t o[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            o[i] = pack_bf16(__uint_as_float(orr[2 * i]) * inv,
                             __uint_as_float(orr[2 * i + 1]) * inv);
          __nv_bfloat16* dst = p.o + row * D + c * 32;
          if (p.o_wide) {
            store32(dst, o);
            store32(dst + 16, o + 8);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              reinterpret_cast<uint4*>(dst)[k] =
                  make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          }
        }
      }
      if (valid && w.part >= 0) p.part_lse[part + brow] = lse2;
      if (valid && w.part < 0 && p.lse) p.lse[row] = lse2 * kLn2;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free + x);
    }
  }

  // ---- teardown: every role has finished issuing; free TMEM
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

// Joins the partials of split blocks by their log2-sum-exp.  A block of
// threads has 32 rows, one per lane (as the partials lie); its warps share the
// columns, and the rows go out through shared memory.  It starts as the chunk
// kernel's blocks leave: with the loads ahead of the maximum 3.5 to 5 us less
// per call (14 MB of partials: 133.7 us to 130.3; 68 MB: 414 to 410).
template <int D>
__global__ void __launch_bounds__(256) chunk_join_kernel(Params p) {
  constexpr int N = D / 32;  // groups of four columns of a warp: warp, warp + 8, ...
  constexpr int PITCH = D * 2 + 16;
  __shared__ __align__(16) uint8_t out[32 * PITCH];
  const ChunkPlanView view(p.n_ctas, p.n_units, p.n_joins);
  const bool fits = __ldg(p.plan) == kChunkMagic && __ldg(p.plan + 1) == p.n_ctas &&
                    __ldg(p.plan + 2) == p.n_units && __ldg(p.plan + 3) == p.n_joins;
  const int4* join = reinterpret_cast<const int4*>(p.plan + view.joins + 8 * blockIdx.x);
  int4 a = {};
  int count = 0;
  if (fits) {
    a = __ldg(join);
    count = __ldg(reinterpret_cast<const int32_t*>(join + 1));
  }
  wait_for_previous();
  if (!fits) return;  // reported by the chunk kernel
  const int q0 = a.x, rows = a.y, kvh = a.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row0 = blockIdx.y * 32;
  if (row0 >= rows) return;
  if (!psa_in_bounds(q0 >= 0 && rows > 0 && kvh >= 0 && kvh < p.Hkv && a.w >= 0 && count > 0 &&
                         int64_t(q0) + (rows - 1) / p.G < p.n_rows &&
                         a.w + int64_t(count) * rows <= p.part_rows,
                     threadIdx.x == 0 ? p.status : nullptr))
    return;
  const int r = min(row0 + lane, rows - 1);
  const float* lse = p.part_lse + a.w + r;
  const float4* o0 =
      reinterpret_cast<const float4*>(p.part_o + size_t(a.w) * D) + size_t(warp) * rows + r;
  // Four partials at a time, their loads together; the first four go out
  // ahead of the maximum over all.  (No read-only loads: the chunk kernel may
  // still have been writing when this one began.)
  float l[4];
  float4 v[4][N];
  auto load = [&](int i0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      l[j] = -INFINITY;
      if (i0 + j < count) {
        l[j] = __ldcg(lse + size_t(i0 + j) * rows);
        const float4* src = o0 + size_t(i0 + j) * rows * (D / 4);
#pragma unroll
        for (int n = 0; n < N; ++n) v[j][n] = __ldcg(src + size_t(n) * 8 * rows);
      }
    }
  };
  load(0);
  float m = fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3]));
#pragma unroll 8
  for (int i = 4; i < count; ++i) m = fmaxf(m, __ldcg(lse + size_t(i) * rows));
  float4 acc[N];
#pragma unroll
  for (int n = 0; n < N; ++n) acc[n] = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  for (int i0 = 0; i0 < count; i0 += 4) {
    if (i0 > 0) load(i0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // an empty partial's rows were not written: whatever they hold stays out
      if (l[j] == -INFINITY) continue;
      const float w = fast_exp2(l[j] - m);
      sum += w;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        acc[n].x = fmaf(w, v[j][n].x, acc[n].x), acc[n].y = fmaf(w, v[j][n].y, acc[n].y);
        acc[n].z = fmaf(w, v[j][n].z, acc[n].z), acc[n].w = fmaf(w, v[j][n].w, acc[n].w);
      }
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int n = 0; n < N; ++n)
    *reinterpret_cast<uint2*>(out + lane * PITCH + (warp + 8 * n) * 8) =
        make_uint2(pack_bf16(acc[n].x * inv, acc[n].y * inv),
                   pack_bf16(acc[n].z * inv, acc[n].w * inv));
  auto out_row = [&](int i) {
    return size_t(q0 + i / p.G) * p.Hq + kvh * p.G + i % p.G;
  };
  if (warp == 0 && p.lse && row0 + lane < rows)
    p.lse[out_row(r)] = sum == 0.f ? -INFINITY : (m + __log2f(sum)) * kLn2;
  __syncthreads();
  constexpr int CPR = D / 8;  // 16-byte pieces of a row
  for (int i = threadIdx.x; i < 32 * CPR; i += 256) {
    const int k = i / CPR, c = i % CPR;
    if (row0 + k < rows)
      reinterpret_cast<uint4*>(p.o + out_row(row0 + k) * D)[c] =
          *reinterpret_cast<const uint4*>(out + k * PITCH + c * 16);
  }
}

// Opt-in shared memory and the register count of one instantiation, looked up
// once per device.
template <int D, bool E4M3, bool CAP, bool WIDE>
int prepare_kernel(int dev) {
  static std::atomic<uint64_t> done{0};
  if (dev < 64 && (done.load(std::memory_order_acquire) >> dev & 1)) return PSA_OK;
  auto kern = chunk_kernel<D, E4M3, CAP, WIDE>;
  cudaFuncAttributes at;
  if (cudaFuncGetAttributes(&at, kern) != cudaSuccess) return PSA_ERR_CUDA;
  // setmaxnreg hands out what the launch reserved: fewer would never return
  if (!WIDE && at.numRegs != kRegsLaunch) return PSA_ERR_UNSUPPORTED;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           int(Cfg<D, E4M3, WIDE>::SMEM)) != cudaSuccess)
    return PSA_ERR_CUDA;
  if (dev < 64) done.fetch_or(uint64_t(1) << dev, std::memory_order_release);
  return PSA_OK;
}

template <int D, bool E4M3, bool CAP, bool WIDE>
int launch_chunk_d(const ChunkArgs& a) {
  using C = Cfg<D, E4M3, WIDE>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PSA_ERR_CUDA;
  int rc = prepare_kernel<D, E4M3, CAP, WIDE>(dev);
  if (rc != PSA_OK) return rc;
  const int G = a.info.Hq / a.info.Hkv, TPH = BM / G;
  CUtensorMap tq;
  {
    const uint64_t dims[3] = {uint64_t(D), uint64_t(a.info.Hq), uint64_t(a.T)};
    const uint64_t strides[2] = {uint64_t(D) * 2, uint64_t(a.info.Hq) * D * 2};
    const uint32_t box[3] = {64u, uint32_t(G), uint32_t(TPH)};
    rc = encode_tmap(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.q, dims, strides, box,
                     CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc != PSA_OK) return rc;
  }
  CUtensorMap tk = tq, tv = tq;  // only read for a contiguous bf16 range
  if (!E4M3 && !a.kv_indices) {
    const uint64_t dims[3] = {uint64_t(D), uint64_t(a.info.Hkv), uint64_t(a.n_cache)};
    const uint64_t strides[2] = {uint64_t(D) * 2, uint64_t(a.info.Hkv) * D * 2};
    const uint32_t box[3] = {64u, 1u, uint32_t(BN)};
    rc = encode_tmap(&tk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.kc, dims, strides, box,
                     CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc != PSA_OK) return rc;
    rc = encode_tmap(&tv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.vc, dims, strides, box,
                     CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc != PSA_OK) return rc;
  }
  Params p = {};
  p.plan = a.plan;
  p.n_ctas = a.info.n_ctas, p.n_units = a.info.n_units, p.n_joins = a.info.n_joins;
  p.kc = static_cast<const uint8_t*>(a.kc);
  p.vc = static_cast<const uint8_t*>(a.vc);
  p.n_cache = a.n_cache;
  p.kv_indices = a.kv_indices;
  p.n_keys = a.info.n_keys;
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.o_wide = (reinterpret_cast<uintptr_t>(a.o) & 31u) == 0;
  p.lse = a.lse;
  p.n_rows = a.info.n_rows, p.Hq = a.info.Hq, p.Hkv = a.info.Hkv, p.G = G, p.TPH = TPH;
  p.window = a.info.window;
  const float scale = a.scale * a.k_scale;
  p.scale_log2 = CAP ? 2.f * kLog2e * scale / a.cap : scale * kLog2e;
  p.cap_log2 = a.cap * kLog2e;
  p.v_scale = a.v_scale;
  p.part_o = a.part_o, p.part_lse = a.part_lse;
  p.part_rows = a.info.part_rows;
  p.status = a.status;
  chunk_kernel<D, E4M3, CAP, WIDE><<<a.info.n_ctas, threads<WIDE>(), C::SMEM, a.stream>>>(tq, tk, tv, p);
  if (cudaGetLastError() != cudaSuccess) return PSA_ERR_CUDA;
  if (a.info.n_joins > 0) {
    const dim3 grid(a.info.n_joins, (a.info.max_join_rows + 31) / 32);
    if (launch_behind(chunk_join_kernel<D>, grid, 256, a.stream, p) != cudaSuccess)
      return PSA_ERR_CUDA;
  }
  return PSA_OK;
}

template <int D, bool E4M3, bool WIDE>
int launch_chunk_cap(const ChunkArgs& a) {
  return a.cap > 0.f ? launch_chunk_d<D, E4M3, true, WIDE>(a)
                     : launch_chunk_d<D, E4M3, false, WIDE>(a);
}

template <int D>
int launch_chunk_of(const ChunkArgs& a) {
  // The wide form over an e4m3 cache (widening a tile keeps the loaders busy:
  // 418 us against 311 for pieces of 1024 tokens over 8k histories), and for
  // few rows through a page table, where gathering sets the pace (18 requests'
  // single tokens over 16k keys: 243 us against 211; contiguous, by TMA, 186
  // against 188).  For full blocks over bf16 its softmax costs more than its
  // loaders gain: 410 us against 425 on 16k paged histories.  The form is the
  // whole batch's: single tokens beside a prompt's piece go through the narrow one.
  if (a.e4m3) return launch_chunk_cap<D, true, true>(a);
  return a.info.all_twin && a.kv_indices ? launch_chunk_cap<D, false, true>(a)
                                         : launch_chunk_cap<D, false, false>(a);
}

}  // namespace

int launch_chunk(const ChunkArgs& a) {
  switch (a.info.head_dim) {
    case 64:
      return launch_chunk_of<64>(a);
    case 128:
      return launch_chunk_of<128>(a);
    default:
      return PSA_ERR_UNSUPPORTED;
  }
}

}  // namespace psa
