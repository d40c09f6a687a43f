// Which sequence of a packed batch a token belongs to.
#pragma once

namespace cpattn {

// Sequence of token t: the last b with cu[b] <= t, found LG candidates at a
// time by the LG lanes of one row (B >= 1; c is the lane's number among them).
// Every lane of the warp executes it.
template <int LG>
__device__ __forceinline__ int find_seq(const int* cu, int B, int t, int c, int lane) {
  const int shift = (lane / LG) * LG;
  int lo = 0, n = B;  // the answer is in [lo, lo + n)
  while (__any_sync(0xffffffffu, n > 1)) {
    const int step = (n + LG - 1) / LG;
    const int i = lo + c * step;
    const bool le = c * step < n && (c == 0 || __ldg(cu + i) <= t);
    const unsigned hit =
        (__ballot_sync(0xffffffffu, le) >> shift) & ((LG == 32) ? 0xffffffffu : ((1u << LG) - 1));
    // Lengths are not negative in a valid batch, so the hits are a prefix; in
    // an invalid one the caller's check of the result rejects it.
    const int k = 31 - __clz(hit);
    const int off = k * step;
    n = min(step, n - off);
    lo += off;
  }
  return lo;
}

}  // namespace cpattn
