// attend_plan.cuh -- how the work of one trie-attention call is cut (attend.cuh).
//
// Rows are (node, query head) pairs. The G query heads of one key head and kNpt = 128 / G
// consecutive nodes make a query tile of up to 128 rows; two consecutive tiles make a pair.
// Keys come in tiles of 128 tokens. The work falls into groups: the shared prefix, whose rows are
// all nodes of the batch whatever their request, and every request, whose rows are its own nodes
// and whose keys are its context and then its nodes. Where that takes no more units than sharing (the
// requests' rows fill their own tiles), there is no group of the prefix and every request's keys
// begin with it: one item where there were two, and no partial results to add. An item is one pair and key head of a group,
// over all key tiles of the group; it costs one unit (about a microsecond) per key tile and query
// tile, and item_cost units to begin and end (queries to load, products to wait for, partial
// results to write).
//
// The units of all items lie on one line, which C CTAs cut into equal contiguous pieces, at key
// tiles: a CTA owns the key tiles whose first unit lies in its piece. So every CTA has the same
// work whatever the lengths (one long request or hundreds of short ones), and an item spreads over
// as many CTAs as its length asks for. Every piece of an item leaves a partial result (output,
// maximum and sum per row), which a second kernel combines. Its place is R(item) + 256 c for CTA c,
// R the rows of the items before: along the line either the item or the CTA grows, and an item has
// at most 256 rows, so the places are disjoint and their number is bounded by the sizes alone.
#pragma once

#include <stdint.h>

namespace psi {

constexpr int kTileRows = 128;  // rows of a query tile
constexpr int kTileKeys = 128;  // tokens of a key tile
constexpr int kItemRows = 256;  // rows of a pair
constexpr int kMaxCtas = 148;   // CTAs of a call: one per SM

// Units to begin and end an item of w query tiles: measured on batches whose CTAs have only short
// items, or only long ones, until both kinds end together.
__host__ __device__ constexpr int item_cost(int w) { return 2 + 2 * w; }

struct AttendShape {
  int G, npt, Hkv;
};

// A group: nodes [lo, lo + n), `ctx_tiles` key tiles of cached tokens (`pre_tiles` of the shared prefix
// where the requests read it themselves, then those of `len` own tokens) and `node_tiles` of own
// nodes (none for the prefix). `bad`: its length is out of range, its rows become NaN.
struct AttendGroup {
  int lo, n, len, pre_tiles, ctx_tiles, node_tiles, bad;
  __host__ __device__ int key_tiles() const { return ctx_tiles + node_tiles; }
  __host__ __device__ int query_tiles(const AttendShape& s) const {
    return key_tiles() > 0 ? (n + s.npt - 1) / s.npt : 0;
  }
};

__host__ __device__ inline AttendGroup make_group(int lo, int n, int len, int64_t room, bool prefix, int pre_len = 0) {
  AttendGroup g;
  g.lo = lo;
  g.n = n;
  g.bad = len < 0 || len > room;
  g.len = g.bad ? 0 : len;
  g.pre_tiles = (pre_len + kTileKeys - 1) / kTileKeys;
  g.ctx_tiles = g.pre_tiles + (g.len + kTileKeys - 1) / kTileKeys;
  g.node_tiles = prefix ? 0 : (n + kTileKeys - 1) / kTileKeys;
  return g;
}

// Units, partial rows and items of a group. A pair of one query tile keeps two partial results per
// row: its key tiles alternate between two accumulators.
struct AttendSize {
  int64_t units, rows;
  int items;
};
__host__ __device__ inline AttendSize group_size(const AttendGroup& g, const AttendShape& s) {
  AttendSize z;
  const int t = g.query_tiles(s);
  z.units = (int64_t(t) * g.key_tiles() + t / 2 * item_cost(2) + (t & 1) * item_cost(1)) * s.Hkv;
  z.rows = t > 0 ? int64_t(s.Hkv) * s.G * (g.n + ((t & 1) ? g.n - (t - 1) * s.npt : 0)) : 0;
  z.items = (t + 1) / 2 * s.Hkv;
  return z;
}

// CTAs that share the line: at most one per key tile of the widest pairs, so that every CTA
// between an item's first and last owns a tile of it.
__host__ __device__ inline int active_ctas(int64_t units, bool wide, int ctas) {
  const int64_t most = wide ? units / 2 : units;
  return static_cast<int>(most < ctas ? (most > 0 ? most : (units > 0 ? 1 : 0)) : ctas);
}
// a / b of numbers that are not negative; most fit 32 bits, whose division is several times as fast.
__host__ __device__ inline int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}
__host__ __device__ inline int64_t cta_first_unit(int64_t units, int c, int C) { return quotient(units * c, C); }
__host__ __device__ inline int cta_of_unit(int64_t units, int64_t u, int C) {
  return static_cast<int>(quotient((u + 1) * C - 1, units));
}

// One CTA's piece of one item.
struct AttendSegment {
  AttendGroup g;
  int req;              // request, -1 for the prefix
  int kvh;              // key head
  int pair;             // pair of the group
  int q_tiles;          // 1 or 2
  int first_node;       // of the pair, in the group's numbering
  int t0, t1;           // key tiles
  int item;             // number of the item
  int64_t row;          // R(item)
  int64_t u0;           // the item's first key tile's first unit
};

// Walks a CTA's segments. Load: AttendGroup operator()(int req), for req = -1 .. B - 1.
struct AttendWalk {
  AttendShape s;
  int B;
  int64_t w0, w1;  // the CTA's units
  int req;
  AttendGroup g;
  int64_t gu, gr;  // units and rows before the group
  int gi;          // items before the group
  int q_tiles, pair, kvh;

  // Starts at group `first`, whose bases are given and whose units reach beyond w0.
  template <typename Load>
  __host__ __device__ void start(const AttendShape& shape, int nreq, int64_t from, int64_t to, int first, int64_t units,
                                 int64_t rows, int items, const Load& load) {
    s = shape;
    B = nreq;
    w0 = from;
    w1 = to;
    req = first;
    gu = units;
    gr = rows;
    gi = items;
    g = load(req);
    q_tiles = g.query_tiles(s);
    pair = kvh = 0;
    if (q_tiles > 0 && w0 > gu) {
      const int64_t per_pair = (int64_t(2) * g.key_tiles() + item_cost(2)) * s.Hkv;
      const int64_t p = quotient(w0 - gu, per_pair);
      pair = static_cast<int>(p < (q_tiles - 1) / 2 ? p : (q_tiles - 1) / 2);
      const int w = q_tiles - 2 * pair < 2 ? 1 : 2;
      const int64_t h = quotient(w0 - gu - pair * per_pair, int64_t(w) * g.key_tiles() + item_cost(w));
      kvh = static_cast<int>(h < s.Hkv - 1 ? h : s.Hkv - 1);
    }
  }

  template <typename Load>
  __host__ __device__ bool next(AttendSegment& seg, const Load& load) {
    for (;;) {
      if (2 * pair >= q_tiles) {
        const AttendSize z = group_size(g, s);
        gu += z.units;
        gr += z.rows;
        gi += z.items;
        if (++req >= B || gu >= w1) return false;
        g = load(req);
        q_tiles = g.query_tiles(s);
        pair = kvh = 0;
        continue;
      }
      const int T = g.key_tiles();
      const int w = q_tiles - 2 * pair < 2 ? 1 : 2;
      const int64_t u0 =
          gu + (int64_t(2) * T + item_cost(2)) * pair * s.Hkv + (int64_t(w) * T + item_cost(w)) * kvh + item_cost(w);
      if (u0 >= w1) return false;
      const int64_t a = w0 > u0 ? (w0 - u0 + w - 1) / w : 0, b = (w1 - u0 + w - 1) / w;
      const int t0 = static_cast<int>(a < T ? a : T), t1 = static_cast<int>(b < T ? b : T);
      const int rest = g.n - 2 * pair * s.npt;  // nodes from this pair on
      seg.g = g;
      seg.req = req;
      seg.kvh = kvh;
      seg.pair = pair;
      seg.q_tiles = w;
      seg.first_node = 2 * pair * s.npt;
      seg.t0 = t0;
      seg.t1 = t1;
      seg.item = gi + pair * s.Hkv + kvh;
      const int rows = s.G * (w == 2 ? (rest < 2 * s.npt ? rest : 2 * s.npt) : 2 * rest);
      seg.row = gr + int64_t(2) * pair * s.npt * s.G * s.Hkv + int64_t(kvh) * rows;
      seg.u0 = u0;
      if (++kvh == s.Hkv) {
        kvh = 0;
        ++pair;
      }
      if (t0 < t1) return true;
    }
  }
};

// Upper bounds over all node offsets of B requests with N nodes: partial rows and items.
inline int64_t max_partial_rows(int64_t N, int64_t Hq, int64_t Hkv, bool prefix) {
  return 2 * N * Hq + (prefix ? N * Hq + kTileRows * Hkv : 0) + int64_t(kItemRows) * kMaxCtas;
}
inline int64_t max_items(int64_t B, int64_t N, int npt, int64_t Hkv, bool prefix) {
  const int64_t pairs = N / (2 * npt) + 1;
  return Hkv * (pairs + (B < N ? B : N) + (prefix ? pairs : 0));
}
// Of units per CTA, for keys of `tokens` in any one request besides its nodes.
inline int64_t max_units(int64_t B, int64_t N, int npt, int64_t Hkv, int64_t tokens, int ctas) {
  const int64_t tiles = tokens / kTileKeys + N / kTileKeys + 3;  // (of the prefix, the context and the nodes)
  return (N / npt + (B < N ? B : N) + N / npt + 1) * Hkv * (tiles + item_cost(2)) / ctas + 2;
}

}  // namespace psi
