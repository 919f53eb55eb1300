// Host-side work plan of the chunk attention: query blocks x KV heads, the
// keys of each cut into pieces, the pieces handed to one list per CTA.
//
// The lists are made on the host, where the lengths are known, so the kernel
// needs no counter in device memory (nothing to zero before a launch, nothing
// for two launches to share) and every sum has a fixed order.
#include <algorithm>
#include <cstdint>
#include <queue>
#include <utility>
#include <vector>

#include "psa.h"
#include "psa_chunk.h"

namespace {

constexpr int kTile = psa::kChunkTile;

// Costs in units of one 128-key tile of a full block (both 128-row halves).
// A block whose rows fit one half runs "twin": the halves take alternate
// tiles of the same rows, so a tile costs about half as much.  A piece pays
// for its first tile's latency and its epilogue, a split block for its
// partial rows and the join launch.
constexpr double kTwinTile = 0.6, kPieceCost = 1.2, kSplitCost = 0.4, kJoinCost = 1.0;

struct Block {
  int32_t q0, ntok, pos0, kv0, lo, hi;  // keys [lo, hi) are seen by some row
  bool twin;
  int64_t tiles() const { return (int64_t(hi) - lo + kTile - 1) / kTile; }
  double tile_cost() const { return twin ? kTwinTile : 1.0; }
  // pieces for a budget of `len` full tiles per piece
  int64_t pieces(double len) const {
    const int64_t per = std::max<int64_t>(1, int64_t(len / tile_cost()));
    return (tiles() + per - 1) / per;
  }
};

struct Piece {
  int32_t block, kvh, index;
  double cost;
};

// Longest first, ties in listing order (a KV head's pieces of one key range
// stay together, so the CTAs in flight share their K/V in L2).
void list_pieces(const std::vector<Block>& blocks, int32_t Hkv, double len,
                 const std::vector<int32_t>& first_of_request, std::vector<Piece>& out) {
  out.clear();
  for (size_t r = 0; r + 1 < first_of_request.size(); ++r) {
    const int32_t b0 = first_of_request[r], b1 = first_of_request[r + 1];
    int64_t most = 0;
    for (int32_t b = b0; b < b1; ++b) most = std::max(most, blocks[b].pieces(len));
    for (int32_t h = 0; h < Hkv; ++h)
      for (int64_t s = 0; s < most; ++s)
        for (int32_t b = b0; b < b1; ++b) {
          const int64_t n = blocks[b].pieces(len);
          if (s >= n) continue;
          const int64_t t = blocks[b].tiles();
          const int64_t mine = t * (s + 1) / n - t * s / n;
          const double c = mine * blocks[b].tile_cost() + kPieceCost +
                           (n > 1 || (blocks[b].twin && t > 1) ? kSplitCost : 0.0);
          out.push_back({b, h, int32_t(s), c});
        }
  }
  std::stable_sort(out.begin(), out.end(),
                   [](const Piece& a, const Piece& b) { return a.cost > b.cost; });
}

// Greedy assignment; returns the longest list's cost.
double assign(const std::vector<Piece>& pieces, int32_t n_ctas, std::vector<int32_t>* cta_of) {
  using Load = std::pair<double, int32_t>;
  std::priority_queue<Load, std::vector<Load>, std::greater<Load>> heap;
  for (int32_t c = 0; c < n_ctas; ++c) heap.push({0.0, c});
  double longest = 0.0;
  for (size_t i = 0; i < pieces.size(); ++i) {
    Load l = heap.top();
    heap.pop();
    if (cta_of) (*cta_of)[i] = l.second;
    l.first += pieces[i].cost;
    longest = std::max(longest, l.first);
    heap.push(l);
  }
  return longest;
}

int build(const int32_t* qo_lens, const int32_t* kv_lens, int32_t B, int32_t Hq, int32_t Hkv,
          int32_t head_dim, int32_t window, int32_t n_ctas, int32_t* out, int64_t cap,
          psa_chunk_info* info) {
  const int32_t G = Hq / Hkv, tph = 128 / G;  // tokens per 128-row half
  std::vector<Block> blocks;
  std::vector<int32_t> first;  // first block of each request
  int64_t q0 = 0, kv0 = 0;
  for (int32_t b = 0; b < B; ++b) {
    const int32_t n = qo_lens[b], L = kv_lens[b];
    if (n < 0 || L < n) return PSA_ERR_INVALID_ARG;
    first.push_back(int32_t(blocks.size()));
    if (q0 + n > INT32_MAX / int64_t(Hq) || kv0 + L > INT32_MAX) return PSA_ERR_INVALID_ARG;
    for (int32_t i = 0; i < n; i += 2 * tph) {
      Block k;
      k.q0 = int32_t(q0 + i);
      k.ntok = std::min(n - i, 2 * tph);
      k.pos0 = L - n + i;
      k.kv0 = int32_t(kv0);
      k.lo = window > 0 ? std::max(0, k.pos0 - window + 1) : 0;
      k.hi = k.pos0 + k.ntok;
      k.twin = k.ntok <= tph;
      blocks.push_back(k);
    }
    q0 += n;
    kv0 += L;
  }
  first.push_back(int32_t(blocks.size()));

  double total = 0.0;
  for (const Block& k : blocks) total += k.tiles() * k.tile_cost() * Hkv;
  std::vector<Piece> pieces;
  double best_len = 0.0, best = 0.0;
  // whole blocks, then pieces of the mean list's length over `rounds`
  for (double rounds : {0.0, 0.5, 0.6, 0.7, 0.8, 0.9, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5,
                        4.0, 5.0, 6.0, 7.0, 8.0}) {
    const double len = rounds == 0 ? 1e18 : std::max(0.5, total / (double(n_ctas) * rounds));
    int64_t count = 0;
    double part_rows = 0.0;
    for (const Block& k : blocks) {
      const int64_t n = k.pieces(len) * (k.twin ? 2 : 1);
      count += n * Hkv;
      if (n > 1) part_rows += double(n) * k.ntok * G * Hkv;
    }
    if (rounds > 0 && count > 65536) break;
    list_pieces(blocks, Hkv, len, first, pieces);
    // a join reads its partials at memory speed, spread over the CTAs
    const double c = assign(pieces, n_ctas, nullptr) +
                     (part_rows > 0.0 ? kJoinCost + part_rows / (n_ctas * 256.0) * 0.25 : 0.0);
    if (rounds == 0 || c < best) {
      best = c;
      best_len = len;
    }
    if (len <= 0.5) break;
  }
  list_pieces(blocks, Hkv, best_len, first, pieces);
  const int32_t used = int32_t(std::min<int64_t>(n_ctas, std::max<size_t>(1, pieces.size())));
  std::vector<int32_t> cta_of(pieces.size());
  assign(pieces, used, &cta_of);

  // partial rows and joins of the blocks with more than one partial
  std::vector<int64_t> part_of(blocks.size() * size_t(Hkv), -1);
  std::vector<int32_t> joins;
  int64_t part_rows = 0;
  int32_t max_join_rows = 0;
  for (size_t b = 0; b < blocks.size(); ++b) {
    const Block& k = blocks[b];
    const int32_t rows = k.ntok * G;
    // a twin piece gives two partials (a single tile: the second is empty)
    const int64_t n = k.pieces(best_len) * (k.twin ? 2 : 1);
    if (n == 1 || k.tiles() == 1) continue;
    for (int32_t h = 0; h < Hkv; ++h) {
      part_of[b * Hkv + h] = part_rows;
      const int32_t j[8] = {k.q0, rows, h, int32_t(part_rows), int32_t(n), 0, 0, 0};
      joins.insert(joins.end(), j, j + 8);
      part_rows += n * rows;
      if (part_rows > INT32_MAX) return PSA_ERR_INVALID_ARG;
    }
    max_join_rows = std::max(max_join_rows, rows);
  }

  psa::ChunkPlanView view(used, int32_t(pieces.size()), int32_t(joins.size() / 8));
  *info = psa_chunk_info{B,    Hq,
                         Hkv,  head_dim,
                         window, int32_t(q0),
                         used, int32_t(pieces.size()),
                         int32_t(joins.size() / 8), max_join_rows,
                         kv0,  part_rows,
                         view.len};
  if (!out || cap < view.len) return PSA_ERR_CAPACITY;
  std::fill(out, out + view.len, 0);
  out[0] = psa::kChunkMagic;
  out[1] = used;
  out[2] = int32_t(pieces.size());
  out[3] = int32_t(joins.size() / 8);
  // units in list order: a CTA's pieces keep their longest-first order
  std::vector<int32_t> count(used + 1, 0);
  for (int32_t c : cta_of) ++count[c + 1];
  for (int32_t c = 0; c < used; ++c) count[c + 1] += count[c];
  std::copy(count.begin(), count.end(), out + view.lists);
  for (size_t i = 0; i < pieces.size(); ++i) {
    const Piece& p = pieces[i];
    const Block& k = blocks[p.block];
    const int64_t n = k.pieces(best_len), t = k.tiles();
    const int64_t t0 = t * p.index / n, t1 = t * (p.index + 1) / n;
    const int64_t part = part_of[size_t(p.block) * Hkv + p.kvh];
    int32_t* u = out + view.units + 12 * size_t(count[cta_of[i]]++);
    u[0] = k.q0;
    u[1] = k.ntok;
    u[2] = k.pos0;
    u[3] = p.kvh;
    u[4] = k.kv0;
    u[5] = int32_t(k.lo + t0 * kTile);
    u[6] = int32_t(std::min<int64_t>(k.lo + t1 * kTile, k.hi));
    u[7] = k.twin ? 1 : 0;
    u[8] = part < 0 ? -1 : int32_t(part + int64_t(p.index) * (k.twin ? 2 : 1) * k.ntok * G);
  }
  std::copy(joins.begin(), joins.end(), out + view.joins);
  return PSA_OK;
}

}  // namespace

extern "C" int psa_build_chunk_plan(const int32_t* qo_lens, const int32_t* kv_lens, int32_t B,
                                    int32_t Hq, int32_t Hkv, int32_t head_dim, int32_t window,
                                    int32_t n_ctas, int32_t* out, int64_t cap,
                                    psa_chunk_info* info) {
  if (!info || B < 0 || (B > 0 && (!qo_lens || !kv_lens)) || Hq <= 0 || Hkv <= 0 ||
      Hq % Hkv != 0 || window < 0 || n_ctas <= 0)
    return PSA_ERR_INVALID_ARG;
  if ((head_dim != 64 && head_dim != 128) || Hq / Hkv > 128) return PSA_ERR_UNSUPPORTED;
  try {
    return build(qo_lens, kv_lens, B, Hq, Hkv, head_dim, window, n_ctas, out, cap, info);
  } catch (...) {  // out of host memory
    return PSA_ERR_INVALID_ARG;
  }
}
