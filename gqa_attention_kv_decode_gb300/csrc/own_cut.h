// own_cut.h -- how the list of own-row tiles (own_rows.cuh) is cut into the
// ranges of its warps.  Whole numbers throughout, so that every CTA comes to
// the same ranges from the same few numbers.
#pragma once

#ifdef __CUDACC__
#define GQA_CUT_FN __host__ __device__ __forceinline__
#else
#define GQA_CUT_FN inline
#endif

namespace gqa {

// n ranges of `size` tiles, the first `longer` of them one longer.
struct OwnRanges {
  unsigned n, size, longer;
  GQA_CUT_FN static OwnRanges of(unsigned tiles, unsigned warps, unsigned min_tiles) {
    OwnRanges r;
    const unsigned most = tiles / min_tiles;
    r.n = most < 1u ? 1u : most < warps ? most : warps;
    r.size = tiles / r.n;
    r.longer = tiles - r.size * r.n;
    return r;
  }
  GQA_CUT_FN unsigned start(unsigned w) const { return w * size + (w < longer ? w : longer); }
  GQA_CUT_FN unsigned holder(unsigned x) const {  // the range with tile x
    const unsigned head = longer * (size + 1);
    return x < head ? x / (size + 1) : longer + (x - head) / size;
  }
};

// The list's first `head` tiles go to the `early` warps (those of the CTAs that
// begin with the grid), the rest to the `late` ones.  head is 0 where there are
// no early warps and N where there are no late ones (own_head).
struct OwnCut {
  unsigned head;
  OwnRanges a, b;
  GQA_CUT_FN static OwnCut of(unsigned N, unsigned head, unsigned early, unsigned late, unsigned min_tiles) {
    OwnCut c;
    c.head = head < N ? head : N;
    c.a = OwnRanges::of(c.head, early > 0u ? early : 1u, min_tiles);
    c.b = OwnRanges::of(N - c.head, late > 0u ? late : 1u, min_tiles);
    return c;
  }
  // The number, among all ranges in order, of the one with tile x.
  GQA_CUT_FN int holder(unsigned x) const {
    return int(x < head ? a.holder(x) : (head > 0u ? a.n : 0u) + b.holder(x - head));
  }
};

}  // namespace gqa
