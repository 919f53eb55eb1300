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
// tiles of the same rows, so a tile costs less: the loaders set its pace, and
// 64-wide heads give them half the bytes (3 x 777 tokens of 16 such heads,
// capped: 132 us at 0.7 against 138 at 0.8; uncapped 74.5 / 76.8, and 79.8 at
// 0.6; e4m3 82.3 / 85.4; with four query heads to a KV head 135.5 / 133.9).
// A piece pays for its first tile's latency and its epilogue, a split block
// for its partial rows and the join launch.
constexpr double kTwinTile = 0.8, kTwinTile64 = 0.7;
constexpr double kPieceCost = 1.2, kSplitCost = 0.4, kJoinCost = 1.5;

struct Block {
  int32_t q0, ntok, pos0, kv0, lo, hi;  // keys [lo, hi) are seen by some row
  bool twin;
  double tile_cost;
  int32_t tiles() const { return int32_t((int64_t(hi) - lo + kTile - 1) / kTile); }
  double cost(int32_t n) const {  // of a piece of n tiles
    return n * tile_cost + kPieceCost + (n < tiles() || (twin && n > 1) ? kSplitCost : 0.0);
  }
};

// Tiles [t0, t1) of one block's range for one KV head, in one CTA's list.
struct Piece {
  int32_t block, kvh, t0, t1, cta;
  float cost;
};

struct Plan {
  std::vector<Piece> pieces;  // a CTA's pieces in its order
  double longest = 0.0;       // cost of the longest list
};

// Blocks cut into pieces of at most `len` full tiles, handed out longest
// first to the list that is shortest; ties in listing order (a KV head's
// pieces of one key range stay together, so the CTAs in flight share their
// K/V in L2).
Plan plan_pieces(const std::vector<Block>& blocks, const std::vector<int32_t>& first, int32_t Hkv,
                 int32_t n_ctas, double len) {
  Plan plan;
  auto count = [&](const Block& b) {
    const int32_t per = int32_t(std::min(1e9, std::max(1.0, len / b.tile_cost)));
    return (b.tiles() + per - 1) / per;
  };
  // the KV heads are alike: list and sort one head's pieces, then repeat them
  std::vector<Piece> one;
  for (size_t r = 0; r + 1 < first.size(); ++r) {
    int32_t most = 0;
    for (int32_t b = first[r]; b < first[r + 1]; ++b) most = std::max(most, count(blocks[b]));
    for (int32_t s = 0; s < most; ++s)
      for (int32_t b = first[r]; b < first[r + 1]; ++b) {
        const int64_t n = count(blocks[b]), t = blocks[b].tiles();
        if (s >= n) continue;
        const int32_t t0 = int32_t(t * s / n), t1 = int32_t(t * (s + 1) / n);
        one.push_back({b, 0, t0, t1, 0, float(blocks[b].cost(t1 - t0))});
      }
  }
  std::stable_sort(one.begin(), one.end(),
                   [](const Piece& a, const Piece& b) { return a.cost > b.cost; });
  // lists by (load, number), the shortest on top
  using Load = std::pair<double, int32_t>;
  std::priority_queue<Load, std::vector<Load>, std::greater<Load>> heap;
  for (int32_t c = 0; c < n_ctas; ++c) heap.push({0.0, c});
  plan.pieces.reserve(one.size() * size_t(Hkv));
  // pieces of one cost, head by head
  for (size_t i = 0, j = 0; i < one.size(); i = j) {
    while (j < one.size() && one[j].cost == one[i].cost) ++j;
    for (int32_t h = 0; h < Hkv; ++h)
      for (size_t k = i; k < j; ++k) {
        Piece p = one[k];
        Load l = heap.top();
        heap.pop();
        p.kvh = h;
        p.cta = l.second;
        l.first += p.cost;
        plan.longest = std::max(plan.longest, l.first);
        heap.push(l);
        plan.pieces.push_back(p);
      }
  }
  return plan;
}

// Lists filled one after another up to the load `most`, a block cut where a list is
// full: lists of equal cost with about one cut each.  Returns false if the
// lists do not hold all.
bool fill_lists(const std::vector<Block>& blocks, int32_t Hkv, int32_t n_ctas, double most,
                const std::vector<int32_t>& first, Plan& plan) {
  plan.pieces.clear();
  plan.longest = 0.0;
  int32_t cta = 0;
  double load = 0.0;
  for (size_t r = 0; r + 1 < first.size(); ++r)
    for (int32_t h = 0; h < Hkv; ++h)
      for (int32_t b = first[r]; b < first[r + 1]; ++b) {
        const Block& k = blocks[b];
        const int32_t n = k.tiles();
        for (int32_t t = 0; t < n;) {
          int32_t fit = n - t;
          if (load + k.cost(fit) > most) {
            const double left = most - load - kPieceCost - kSplitCost;
            fit = std::min(n - t, int32_t(left / k.tile_cost));
            // no stubs: a cut leaves at least two tiles on both sides
            if (n - t - fit < 2) fit = n - t - 2;
            if (fit < 2) {
              if (load == 0.0 || ++cta == n_ctas) return false;
              load = 0.0;
              continue;
            }
          }
          plan.pieces.push_back({b, h, t, t + fit, cta, 0.f});
          load += k.cost(fit);
          plan.longest = std::max(plan.longest, load);
          t += fit;
        }
      }
  return true;
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
    if (q0 + n > INT32_MAX / int64_t(Hq) || kv0 + L > INT32_MAX - 2 * kTile) return PSA_ERR_INVALID_ARG;
    for (int32_t i = 0; i < n; i += 2 * tph) {
      Block k;
      k.q0 = int32_t(q0 + i);
      k.ntok = std::min(n - i, 2 * tph);
      k.pos0 = L - n + i;
      k.kv0 = int32_t(kv0);
      k.lo = window > 0 ? std::max(0, k.pos0 - window + 1) : 0;
      k.hi = k.pos0 + k.ntok;
      k.twin = k.ntok <= tph;
      k.tile_cost = !k.twin ? 1.0 : head_dim == 64 ? kTwinTile64 : kTwinTile;
      blocks.push_back(k);
    }
    q0 += n;
    kv0 += L;
  }
  first.push_back(int32_t(blocks.size()));

  double total = 0.0;
  for (const Block& k : blocks) total += k.tiles() * k.tile_cost * Hkv;
  // a join reads its partials at memory speed, spread over the CTAs
  auto join_cost = [&](const Plan& plan) {
    double rows = 0.0;
    for (const Piece& p : plan.pieces) {
      const Block& k = blocks[p.block];
      if (p.t1 - p.t0 < k.tiles() || (k.twin && k.tiles() > 1))
        rows += (k.twin ? 2.0 : 1.0) * k.ntok * G;
    }
    return rows > 0.0 ? kJoinCost + rows / (n_ctas * 256.0) * 0.25 : 0.0;
  };
  Plan best;
  double best_cost = 0.0;
  auto offer = [&](Plan&& plan, double factor = 1.0) {
    const double c = factor * (plan.longest + join_cost(plan));
    if (best.pieces.empty() || c < best_cost) {
      best_cost = c;
      best = std::move(plan);
    }
  };
  if (!blocks.empty()) {
    // whole blocks, then pieces of the mean list's length over `rounds`
    for (double rounds : {0.0, 0.5, 0.75, 1.0, 1.5, 1.75, 2.0, 2.5, 3.0}) {
      const double len = rounds == 0 ? 1e18 : std::max(0.5, total / (double(n_ctas) * rounds));
      if (rounds > 0 && blocks.size() * double(Hkv) + total / len > 8192.0) break;
      offer(plan_pieces(blocks, first, Hkv, n_ctas, len));
      if (len <= 0.5) break;
    }
    // lists of at most one load, the smallest that holds all (to 1 %)
    Plan fill, tried;
    double low = total / n_ctas, high = 2.0 * low + 8.0;
    bool found = false;
    for (int i = 0; i < 20 && (!found || high - low > 0.01 * high); ++i) {
      const double mid = found || i > 0 ? 0.5 * (low + high) : high;
      if (fill_lists(blocks, Hkv, n_ctas, mid, first, tried)) {
        std::swap(fill, tried);
        high = mid;
        found = true;
      } else {
        low = mid;
        if (!found) high *= 2.0;
      }
    }
    // Filled lists keep fewer partials, but their CTAs are at different keys
    // of a head at any time: where the keys and values do not fit L2 they come
    // from memory more than once.  Measured, pieces against filled lists: 586
    // and 556 us with 75 MB of keys and values, 454 and 482 us with 290 MB.
    // (Counted as bf16 and whole: an e4m3 cache or a window may fit L2 where
    // this says that it does not; the plan is not told the cache's type.)
    const double kv_bytes = 4.0 * double(kv0) * Hkv * head_dim;
    if (found) offer(std::move(fill), kv_bytes > 120e6 ? 1.08 : 1.0);
  }
  const std::vector<Piece>& pieces = best.pieces;
  int32_t used = 1;
  for (const Piece& p : pieces) used = std::max(used, p.cta + 1);

  // pieces of each block and head: their partials lie back to back
  std::vector<int32_t> n_of(blocks.size() * size_t(Hkv), 0);
  for (const Piece& p : pieces) ++n_of[size_t(p.block) * Hkv + p.kvh];
  // partial rows and joins of the blocks with more than one partial
  std::vector<int64_t> part_of(blocks.size() * size_t(Hkv), -1);
  std::vector<int32_t> joins;
  int64_t part_rows = 0;
  int32_t max_join_rows = 0;
  for (size_t b = 0; b < blocks.size(); ++b) {
    const Block& k = blocks[b];
    const int32_t rows = k.ntok * G;
    for (int32_t h = 0; h < Hkv; ++h) {
      // a twin piece gives two partials (a single tile: the second is empty)
      const int64_t n = int64_t(n_of[b * Hkv + h]) * (k.twin ? 2 : 1);
      if (n == 1 || k.tiles() == 1) continue;
      part_of[b * Hkv + h] = part_rows;
      const int32_t j[8] = {k.q0, rows, h, int32_t(part_rows), int32_t(n), 0, 0, 0};
      joins.insert(joins.end(), j, j + 8);
      part_rows += n * rows;
      if (part_rows > INT32_MAX) return PSA_ERR_INVALID_ARG;
      max_join_rows = std::max(max_join_rows, rows);
    }
  }

  psa::ChunkPlanView view(used, int32_t(pieces.size()), int32_t(joins.size() / 8));
  *info = {};
  info->B = B, info->Hq = Hq, info->Hkv = Hkv, info->head_dim = head_dim, info->window = window;
  info->n_rows = int32_t(q0), info->n_keys = kv0;
  info->n_ctas = used, info->n_units = int32_t(pieces.size());
  info->n_joins = int32_t(joins.size() / 8), info->max_join_rows = max_join_rows;
  info->all_twin =
      std::all_of(blocks.begin(), blocks.end(), [](const Block& k) { return k.twin; });
  info->part_rows = part_rows, info->len = view.len;
  if (!out || cap < view.len) return PSA_ERR_CAPACITY;
  std::fill(out, out + view.len, 0);
  out[0] = psa::kChunkMagic;
  out[1] = used;
  out[2] = int32_t(pieces.size());
  out[3] = int32_t(joins.size() / 8);
  // units in list order
  std::vector<int32_t> count(used + 1, 0);
  for (const Piece& p : pieces) ++count[p.cta + 1];
  for (int32_t c = 0; c < used; ++c) count[c + 1] += count[c];
  std::copy(count.begin(), count.end(), out + view.lists);
  std::fill(n_of.begin(), n_of.end(), 0);  // now: partials placed so far
  for (const Piece& p : pieces) {
    const Block& k = blocks[p.block];
    const size_t at = size_t(p.block) * Hkv + p.kvh;
    const int32_t index = n_of[at]++;
    int32_t* u = out + view.units + 12 * size_t(count[p.cta]++);
    u[0] = k.q0;
    u[1] = k.ntok;
    u[2] = k.pos0;
    u[3] = p.kvh;
    u[4] = k.kv0;
    u[5] = k.lo + p.t0 * kTile;
    u[6] = int32_t(std::min<int64_t>(k.lo + int64_t(p.t1) * kTile, k.hi));
    u[7] = k.twin ? 1 : 0;
    u[8] = part_of[at] < 0 ? -1
                           : int32_t(part_of[at] + int64_t(index) * (k.twin ? 2 : 1) * k.ntok * G);
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
