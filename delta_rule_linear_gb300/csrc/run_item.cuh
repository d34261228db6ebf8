// run_item.cuh -- which tokens of which sequence a warp or CTA has.
#pragma once

#include "linear_internal.cuh"

namespace kda {

// Sequences up to which runs are counted.  Counting goes over all sequences before the run's own, a warp 32 at a time, and leaves
// no run without tokens between the others; over all runs that is the square of the number of sequences.
// The convolution, 40,000 tokens of 2048 channels, counted and searched: 16 sequences 62.5 and 67.6 us, 512 sequences 89 and 85
// (gradients 200 both), 1024 128 and 99, 16,384 3826 and 317.  The scan's gradients, 16 states: 1024 sequences 5.8 and 4.2 ms, 16,384
// 288 and 34.
constexpr int kCounted = 512;

// Runs of L tokens: exact for equal lengths, a bound for both ways of numbering those of packed sequences with `total` rows.
inline long run_items(const LinSeqs &s, long total, int L) { return s.cu ? total / L + s.nseq : lin_items(s.nseq, s.T, s.T, false, L); }

// Of many sequences, n has its runs from this number on: the numbers rise with n and leave each sequence enough of them, so
// that a run's sequence can be searched for; some numbers have no run.
__device__ __forceinline__ int first_of_many(const LinSeqs &s, long total, int L, int n) {
    return min(max(s.cu[n], 0), (int)total) / L + n;
}
// Run `item` of many packed sequences, by a warp that looks at 32 places at a time; false: there is none.
__device__ __forceinline__ bool many_item(const LinSeqs &s, long total, int L, long item, LinItem &it) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = s.nseq, step;           // the sequence is among lo .. lo + n
    do {
        step = (n + 31) / 32;
        const int k = lane * step;
        const unsigned some = __ballot_sync(0xffffffffu, k < n && first_of_many(s, total, L, lo + k) <= item);
        if (!some) return false;
        const int last = (31 - __clz(some)) * step;
        lo += last;
        n = min(step, n - last);
    } while (step > 1);
    it.n = lo;
    it.first = first_of_many(s, total, L, lo);
    it.p = (int)item - it.first;
    it.start = min(max(s.cu[lo], 0), (int)total);
    it.len = max(min(s.cu[lo + 1], (int)total) - (int)it.start, 0);
    it.nseg = it.len > L ? (it.len + L - 1) / L : 1;
    return it.p < it.nseg;
}

// Run `item` of a batch, packed or not (whole warps call it together); false: there is none.  Whatever a prefix array says, no
// row outside the batch is in it.
__device__ __forceinline__ bool run_item(const LinSeqs &s, long total, int L, long item, LinItem &it) {
    if (!s.cu) return lin_item(s, L, (int)item, it);
    if (s.nseq > kCounted) return many_item(s, total, L, item, it);
    if (!lin_item(s, L, (int)item, it)) return false;
    it.start = min(max(it.start, 0L), total);
    it.len = (int)min((long)max(it.len, 0), total - it.start);
    return true;
}

}  // namespace kda
