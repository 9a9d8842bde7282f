// attn_masked_tc.cuh -- the plan of the tensor-core attention whose rows read only
// some of the keys (attn_masked_tc.cu): which rows and keys a work item has, and how
// the items are shared out.  The same code on the device and, for the self-check, on
// the host.
//
// Rows.  The G = Hq / Hkv query heads of a kv head read the same keys, so a tile of
// 128 rows holds tpt = floor(128 / G) consecutive tokens of all G heads (row t G + g),
// and a window costs the W + tpt keys of that tile rather than the W + 128 of a tile
// of one head.  An item is a pair of tiles (a, b) of one sequence and kv head; both
// read the key tiles that are loaded for it.
//
// Keys.  An item's key tiles (128 keys each) are `lead` tiles from key 0 on, with the
// sinks, then tiles from `start` on, the beginning of its first row's window, up to
// its last row's position.
//
// Partition.  The key tiles of all items, end to end in the order (sequence, pair,
// head), are cut into one equal range per CTA.  Prompts take whole items (the border
// next to the cut), and an item counts as its tiles and kItemCost more, since what
// surrounds them (queries, first scores, output) takes that long; over a cache, where
// few items may have many tiles, an item is cut, the states of its pieces go to the
// workspace and a second kernel merges them; but where there are no more items than CTAs
// and none is much longer than an even range, each CTA takes one whole (keeps_items).
#pragma once

#include "rf_device.cuh"
#include "rf_internal.h"

namespace rf {
namespace masked {

constexpr int BQ = 128, BK = 128;
constexpr int kItemCost = 5;

struct Geo {
  const int* seq_lens;      // paged: [B] tokens of each sequence; else null
  const int* cu_q;          // packed: [B + 1] cumulative lengths, or null: equal ones
  const int* cu_k;
  int B, Hkv, G, tpt;       // tpt: tokens of a tile
  int npairs;               // pairs of a sequence, at most
  int max_q;                // paged: query tokens of each sequence (Tq)
  int total_q, total_k;     // packed
  int max_len;              // paged
  int window, sinks, tree;
  // What an item counts as beside its tiles (the first items of a long prompt have few;
  // 16k prompt 910 us at 2, 785 at 4, 775 at 6).
  __host__ __device__ __forceinline__ int extra() const { return seq_lens ? 0 : kItemCost; }
};

__host__ __device__ __forceinline__ int imin(int a, int b) { return a < b ? a : b; }
__host__ __device__ __forceinline__ int imax(int a, int b) { return a > b ? a : b; }

// Pair p of sequence b: its rows and its key tiles (of each kv head).
struct Group {
  int b, q0, k0;            // first query token, first key of the sequence (rows of Q, K)
  int lq, lk;               // the sequence's query tokens and keys
  int t0, t1;               // the pair's tokens t0 .. t1 - 1
  int start, lead, n;       // key tiles; n = 0: there are no rows
};

__host__ __device__ __forceinline__ Group group_of(const Geo& p, int g, bool report,
                                                   unsigned* err) {
  Group w;
  w.b = g / p.npairs;
  const int pair = g - w.b * p.npairs;
  if (p.seq_lens) {
    w.lk = ld_int(p.seq_lens, w.b, p.B, err);
    if (w.lk < 0 || w.lk > p.max_len) {
      if (report && pair == 0) note_error(err, kDevErrInput);
      w.lk = 0;
    }
    w.lq = p.max_q;
    w.q0 = w.b * p.max_q;
    w.k0 = 0;
  } else {
    int a0, a1, c0, c1;
    if (p.cu_q) {
      a0 = ld_int(p.cu_q, w.b, p.B + 1, err);
      a1 = ld_int(p.cu_q, w.b + 1, p.B + 1, err);
    } else {
      a0 = w.b * (p.total_q / p.B);
      a1 = a0 + p.total_q / p.B;
    }
    if (p.cu_k) {
      c0 = ld_int(p.cu_k, w.b, p.B + 1, err);
      c1 = ld_int(p.cu_k, w.b + 1, p.B + 1, err);
    } else {
      c0 = w.b * (p.total_k / p.B);
      c1 = c0 + p.total_k / p.B;
    }
    const bool ok = 0 <= a0 && a0 <= a1 && a1 <= p.total_q && a1 - a0 <= p.max_q && 0 <= c0 &&
                    c0 <= c1 && c1 <= p.total_k;
    if (!ok && report && pair == 0) note_error(err, kDevErrInput);
    w.q0 = ok ? a0 : 0;
    w.k0 = ok ? c0 : 0;
    w.lq = ok ? a1 - a0 : 0;
    w.lk = ok ? c1 - c0 : 0;
  }
  w.t0 = 2 * pair * p.tpt;
  w.t1 = imin(w.lq, w.t0 + 2 * p.tpt);
  w.start = w.lead = w.n = 0;
  if (w.t0 >= w.t1) return w;
  const int ctx = w.lk - w.lq;                        // position of token 0
  const int end = imax(0, imin(w.lk, p.tree ? w.lk : ctx + w.t1));      // behind the last key
  if (p.window > 0) {
    int lo = (p.tree ? ctx : ctx + w.t0) - p.window + 1;
    if (p.seq_lens) lo = lo > 0 ? lo & ~(BK - 1) : lo;       // whole pages lie in one tile
    if (lo > 0) {
      const int lead = (imin(p.sinks, end) + BK - 1) / BK;
      if (lead * BK < lo) {
        w.start = lo;
        w.lead = lead;
      }
    }
  }
  // rows that read nothing still take one (fully masked) tile, which writes their zeros
  w.n = imax(1, w.lead + (end - w.start + BK - 1) / BK);
  return w;
}

// The next group with rows from g on (B * npairs if there is none), left in w.
__host__ __device__ __forceinline__ int next_group(const Geo& p, int g, Group& w, unsigned* err) {
  const int ng = p.B * p.npairs;
  while (g < ng) {
    w = group_of(p, g, false, err);
    if (w.n > 0) return g;
    g = (w.b + 1) * p.npairs;                         // its later pairs have no rows either
  }
  return ng;
}

__host__ __device__ __forceinline__ int key0_of(const Group& w, int j) {
  return j < w.lead ? j * BK : w.start + (j - w.lead) * BK;
}

// What an item of the group counts as (0: it has no rows).
__host__ __device__ __forceinline__ int places(const Geo& p, const Group& w) {
  return w.n > 0 ? w.n + p.extra() : 0;
}

// T tiles over n ranges, the first T % n of them one longer.
struct Split64 {
  int64_t q, rem;
  __host__ __device__ __forceinline__ Split64(int64_t T, int n) : q(T / n), rem(T % n) {}
  __host__ __device__ __forceinline__ int64_t start(int c) const {
    return c * q + (c < rem ? c : rem);
  }
  __host__ __device__ __forceinline__ int owner(int64_t x) const {
    const int64_t big = rem * (q + 1);
    return (int)(x < big ? x / (q + 1) : rem + (x - big) / q);
  }
};

// Over a cache: items (most: the tiles of the longest) that are not cut.  A cut costs a
// second piece's start and output and the merge.  Trees of 16 nodes, 8 kv heads of 128, cut
// against whole, us: 16 sequences of 250 / 1000 / 2500 tokens 17 / 34 / 53 against 15 / 24 / 45,
// of 100 to 2000 41 against 31; one sequence (8 items) of 500 / 1000 14 / 15 against 17 / 23.
// 64 nodes, 8 sequences (64 items) of 1500 / 2000 tokens: 37 / 41 against 36 / 44.
__host__ __device__ __forceinline__ bool keeps_items(int64_t items, int most, int64_t total, int grid) {
  return items <= grid && most <= total / grid + (4 * items > grid ? 7 : 1);
}

// Where whole items are taken: the border next to place `off` of an item that counts
// as `all`; its tile there.
__host__ __device__ __forceinline__ bool snaps_up(int off, int all) { return 2 * off >= all; }

// A CTA's range, piece by piece.
struct Piece {
  Group w;
  int h, j0, j1;            // tiles j0 .. j1 - 1 of the item
  __host__ __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == w.n; }
};
struct Walk {
  int64_t left;             // what is still to take, as items count
  int g, h, j;              // the next tile; j may be behind the item's last: the next item's
  __host__ __device__ __forceinline__ Walk(int g_, int h_, int j_, int64_t count)
      : left(count), g(g_), h(h_), j(j_) {}
  __host__ __device__ __forceinline__ bool next(const Geo& p, Piece& out, unsigned* err) {
    if (left <= 0) return false;
    out.w = group_of(p, g, false, err);
    if (j >= out.w.n) {
      j = 0;
      if (++h >= p.Hkv) {
        h = 0;
        g = next_group(p, g + 1, out.w, err);
        if (g >= p.B * p.npairs) {                    // (on the device: the lengths changed)
          left = 0;
          return false;
        }
      }
    }
    left -= p.extra();
    out.h = h;
    out.j0 = j;
    out.j1 = p.extra() || (int64_t)(out.w.n - j) < left ? out.w.n : j + (int)left;
    left -= out.j1 - out.j0;
    j = out.j1;
    return true;
  }
};

// Tile x (0, 1) of a piece: its tokens, and which units it takes (unit u: the keys of
// half u & 1 of the item's key tile u / 2): those in which some row may read a key.  A
// prompt's tile that reads no key takes the first all the same: its scores tell the
// softmax warps, which write their output where the queries were loaded, that the load
// has ended (each waits for the scores of its own tiles only, every one in turn).
constexpr int kUnit = BK / 2;
struct Tile {
  int t0, t1;               // its tokens; t0 >= t1: it has no rows
  int sink, first, last;    // units 0 .. sink - 1 and first .. last
  __host__ __device__ __forceinline__ bool has() const { return t0 < t1; }
  __host__ __device__ __forceinline__ bool takes(int u) const {
    return u < sink || (u >= first && u <= last);
  }
};
__host__ __device__ __forceinline__ Tile tile_of(const Geo& p, const Group& w, int x) {
  Tile t;
  t.t0 = w.t0 + x * p.tpt;
  t.t1 = imin(w.t1, t.t0 + p.tpt);
  const int ctx = w.lk - w.lq;
  const int hi = p.tree ? w.lk - 1 : imin(w.lk - 1, ctx + t.t1 - 1);     // its last row's position
  const int lo = p.window > 0 ? (p.tree ? ctx : ctx + t.t0) - p.window + 1 : 0;
  t.sink = t.first = 0;
  t.last = t.has() && !p.seq_lens ? 0 : -1;
  if (hi < 0 || !t.has()) return t;
  t.first = 2 * w.lead + (lo > w.start ? (lo - w.start) / kUnit : 0);
  t.last = 2 * w.lead + (hi - w.start) / kUnit;
  if (p.window > 0)
    t.sink = imin((imin(p.sinks, w.lk) + kUnit - 1) / kUnit, w.lead > 0 ? 2 * w.lead : t.last + 1);
  return t;
}

// Whether some row of a pair may not read all of the n keys from key0 on: they are all
// read if they end at or before `end` and begin at or behind `begin` (or are sinks).
struct Whole {
  int end, begin;
  __host__ __device__ __forceinline__ bool partly(const Geo& p, int key0, int n) const {
    return key0 + n > end || (key0 < begin && key0 + n > p.sinks);
  }
};
__host__ __device__ __forceinline__ Whole whole_of(const Geo& p, const Group& w) {
  const int ctx = w.lk - w.lq;
  Whole a;
  a.end = p.tree ? ctx : ctx + w.t0 + 1;
  a.begin = p.window > 0 ? (p.tree ? w.lk : ctx + w.t1) - p.window : -2147483647;
  return a;
}

// Where a query tile is loaded: the place, and how many were there before.  Tiles come
// piece by piece, a before b, and not every piece has a b.  With kOwn each of the two
// has places of its own (where no piece has a b, a has all): whoever waits for the tiles
// of one of them only waits for every load of a place, in turn.  In places that both
// share it would pass over the other's loads, and a wait for the load behind one that has
// not ended yet goes by the same parity as the load before that, and returns at once.
struct QPlace {
  int slot, turn;
};
template <int S, bool kOwn>
struct QTurns {
  int na, nb;               // tiles so far: a's and b's, or (not kOwn) both in na
  bool pairs;
  __host__ __device__ __forceinline__ explicit QTurns(const Geo& p)
      : na(0), nb(0), pairs(p.max_q > p.tpt) {}
  __host__ __device__ __forceinline__ int places() const { return kOwn && pairs ? S / 2 : S; }
  __host__ __device__ __forceinline__ QPlace at(int x, int n) const {
    if (!kOwn || !pairs) return {n % S, n / S};
    return {x * (S / 2) + n % (S / 2), n / (S / 2)};
  }
  __host__ __device__ __forceinline__ QPlace next(int x) {
    return at(x, kOwn && x ? nb++ : na++);
  }
};

// The workspace slot of CTA c's piece of an item that begins at tile s0 (in the
// order of all tiles), of which the CTA's range begins at x0: only its first and
// its last item can be cut.
__host__ __device__ __forceinline__ int64_t slot_of(int c, int64_t s0, int64_t x0) {
  return 2 * (int64_t)c + (s0 < x0 ? 0 : 1);
}

}  // namespace masked
}  // namespace rf
