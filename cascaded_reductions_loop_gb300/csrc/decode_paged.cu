// decode_paged.cu -- the unmasked instances of the paged decode attention
// (decode_paged.cuh), its sizes and the host's walk of its plans.
#include "decode_paged.cuh"

#include <algorithm>
#include <vector>

namespace rf {
// Chunks of the fullest batch the cache can hold, over all tiles.
int64_t decode_paged_max_chunks(int B, int Hkv, int R, int max_pages, int page_size) {
  const int64_t tiles = (int64_t)B * Hkv * tiles_of(R);
  const int64_t chunks = ((int64_t)max_pages * page_size + kChunk - 1) / kChunk;
  return tiles >= (1ll << 31) ? (1ll << 31) : tiles * chunks;
}

// Workspace: tickets [B * HR], partial rows [2 * SMs][16][d], their (M, m, l).
size_t decode_paged_workspace_bytes(int B, int Hkv, int R, int d) {
  const int sms = sm_count();
  if (sms <= 0) return 0;
  const size_t rows = (size_t)2 * sms * kTileRows;
  return pad256((size_t)B * Hkv * tiles_of(R) * sizeof(unsigned)) +
         pad256(rows * d * sizeof(float)) + rows * sizeof(float4);
}

cudaError_t launch_decode_paged(const PagedKV& c, const void* Q, void* O, int Hq, int Tq,
                                float scale, void* workspace, unsigned* err, cudaStream_t s) {
  return launch_any<false>(c, Mask{}, Q, O, Hq, Tq, scale, workspace, err, s);
}

// Host-side walk of the partition (the functions above, shared by host and
// device) for `sms` CTAs of `W` warps; seq_lens is a host array.  Returns 0
// when every invariant holds, else the number of the first that fails:
//   1 no index leaves its array;
//   2 the warps' ranges, end to end, are all chunks, in order, once;
//   3 a warp leaves at most two unfinished tiles: its first and its last;
//   4 a CTA leaves at most two tiles to the workspace, in slots of their own;
//   5 a tile cut between CTAs has the parts that the merge counts, in the
//     slots that it reads, in key order.
//   6 the chunks are those that hold a key which some of the last Tq tokens reads
//     (and no other, but for those of the sinks and one at the window's beginning).
template <bool kExt>
static int plan_selfcheck(const Lens& lens, int W, int sms) {
  const int B = lens.B, HR = lens.HR;
  unsigned err = 0, total = 0, most = 0;
  std::vector<unsigned> pre((size_t)B + 1, 0);
  for (int b = 0; b < B; ++b) {
    const unsigned nck = num_chunks<kExt>(lens, seq_len(lens, b, true, &err));
    most = std::max(most, nck);
    total += nck * (unsigned)HR;
    pre[(size_t)b + 1] = total;
  }
  auto seq_of = [&](unsigned x) {
    return (int)(std::upper_bound(pre.begin(), pre.end(), x) - pre.begin()) - 1;
  };
  auto border = [&](unsigned x) {
    if (x == total) return total;
    const int b = seq_of(x);
    const unsigned nck = num_chunks<kExt>(lens, seq_len(lens, b, false, &err));
    return snap(x, (x - pre[(size_t)b]) % nck, nck);
  };
  if (total == 0) return 0;
  const unsigned grid = ctas_for(total, (unsigned)sms, (unsigned)W);
  const Split ctas(total, grid);
  Cursor<kExt> want = {-1, HR - 1, 0, 0, 0};
  unsigned x = 0;                                       // next chunk in the order of all
  std::vector<std::vector<int64_t>> parts((size_t)B * HR);
  std::vector<unsigned char> used((size_t)2 * sms, 0);
  for (unsigned c = 0; c < grid; ++c) {
    unsigned r0 = ctas.start(c), r1 = ctas.start(c + 1);
    if (keeps_tiles(most, (unsigned)W)) {
      r0 = border(r0);
      r1 = border(r1);
    }
    const Split warps(r1 - r0, (unsigned)W);
    int cut_tiles = 0;
    int64_t last_cut = -1;
    for (int w = 0; w < W; ++w) {
      const unsigned x0 = r0 + warps.start(w), n = warps.start(w + 1) - warps.start(w);
      if (n == 0) continue;
      if (x0 != x) return 2;
      const int b = seq_of(x0);
      Cursor<kExt> cur;
      if (!cur.init(lens, b, seq_len(lens, b, false, &err), x0 - pre[(size_t)b])) return 2;
      int left = 0;
      for (unsigned i = 0; i < n; ++i, ++x) {
        if (i > 0 && !cur.next(lens, &err)) return 2;
        if (err & kDevErrBounds) return 1;
        if (!want.next(lens, &err)) return 2;
        if (cur.b != want.b || cur.hr != want.hr || cur.ck != want.ck || cur.len != want.len)
          return 2;
        const bool tile_end = cur.ck + 1 == cur.nck;
        if (!tile_end && i + 1 != n) continue;
        const unsigned s0 = x0 + i - cur.ck, s1 = s0 + cur.nck;
        if (tile_end && s0 >= x0) continue;             // written by the warp itself
        if (left == 1 && i + 1 != n) return 3;          // the second state takes the ring
        if (++left > 2) return 3;
        const int64_t tile = (int64_t)cur.b * HR + cur.hr;
        if ((s0 < r0 || s1 > r1) && tile != last_cut) {
          if (keeps_tiles(most, (unsigned)W)) return 4;
          last_cut = tile;
          if (++cut_tiles > 2) return 4;
          const int64_t slot = slot_of(ctas, s0, c);
          if (slot < 0 || slot >= 2 * (int64_t)sms || used[(size_t)slot]++) return 4;
          const unsigned c0 = ctas.owner(s0);
          parts[(size_t)tile].push_back(slot);
          if (c0 + parts[(size_t)tile].size() - 1 != c) return 5;
          if (s1 <= r1 && parts[(size_t)tile].size() != ctas.owner(s1 - 1) - c0 + 1) return 5;
        }
      }
    }
  }
  if (x != total) return 2;
  for (int b = 0; kExt && b < B; ++b) {
    const int len = seq_len(lens, b, false, &err);
    const Span sp = span_of<kExt>(lens, len);
    const unsigned all = ((unsigned)len + kChunk - 1) / kChunk;
    if (sp.n + sp.skip != all || (sp.skip && sp.lead + sp.skip >= all)) return 6;
    // the keys left out: read by no token, and no whole chunk of such keys is in
    const int64_t lo = (int64_t)std::max(len - lens.Tq, 0) - lens.window + 1;
    if (sp.skip && ((int64_t)sp.lead * kChunk < std::min(lens.sinks, len) ||
                    ((int64_t)sp.lead + sp.skip) * kChunk > lo ||
                    ((int64_t)sp.lead + sp.skip + 1) * kChunk <= lo ||
                    ((int64_t)sp.lead - 1) * kChunk >= std::min(lens.sinks, len)))
      return 6;
    if (!sp.skip && lens.window != 0 && lo / kChunk > sp.lead && lo > 0) return 6;
  }
  return 0;
}

int decode_paged_plan_selfcheck(const int* seq_lens, int B, int HR, int max_len, int Tq, int window,
                                int sinks, int W, int sms) {
  const Lens lens = {seq_lens, B, HR, max_len, Tq, window, sinks};
  return window ? plan_selfcheck<true>(lens, W, sms) : plan_selfcheck<false>(lens, W, sms);
}

}  // namespace rf
