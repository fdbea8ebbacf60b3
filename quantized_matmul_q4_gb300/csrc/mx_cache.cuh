// The paged MX cache and the batch of sequences that a call works on.
//
// Keys and values of a cache lie in pages of `page` tokens (a multiple of 16),
// for each key/value head apart: codes [pages][heads][page][D·bits/8] and
// scale bytes [pages][heads][page][4] (block b of the head in byte b, zeros
// past D / 32).  So the tokens of one head within a page are one contiguous
// run, which is what attention reads.
//
// Sequence i of a batch has the rows starts[i] .. starts[i + 1] of the dense
// tensors, the last of its lengths[i] cached tokens; its position p is slot
// p % page of page table[i · width + p / page].  All three arrays are device
// memory whose values no host check sees, so every index made from them is
// checked here: a page number or a position outside the cache or the table
// sets kStatusIndex in the status word, and its access is left out.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "kernels.h"

namespace q4mm {

// Entries of the ascending array key(0) .. key(n - 1) that are <= t, found by
// the whole warp, 32 at a time.
template <class F>
__device__ __forceinline__ int warp_count_le(F key, int n, long long t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, end = n;
    while (end - lo > 32) {
        const int step = (end - lo + 31) / 32, at = lo + (lane + 1) * step - 1;
        const unsigned le = __ballot_sync(0xFFFFFFFFu, at < end && key(at) <= t);
        const int whole = __popc(le);
        lo += whole * step;
        end = min(end, lo + step - 1);
    }
    const unsigned le = __ballot_sync(0xFFFFFFFFu, lo + lane < end && key(lo + lane) <= t);
    return lo + __popc(le);
}

// The sequence whose rows hold row t, or -1.
__device__ __forceinline__ int sequence_of_row(const MxBatchView &b, long long t) {
    const int i = warp_count_le([&](int j) { return (long long)b.starts[j]; }, b.seqs + 1, t) - 1;
    return i >= 0 && i < b.seqs ? i : -1;
}

// The page of sequence i that holds its page-sized piece `piece`, or -1.
__device__ __forceinline__ int page_of(const MxBatchView &b, const MxCacheView &c, int i, int piece, int *status) {
    if (piece >= 0 && piece < b.width) {
        const int p = b.table[(long long)i * b.width + piece];
        if (p >= 0 && p < c.pages) return p;
    }
    atomicOr(status, kStatusIndex);
    return -1;
}

// Slot number of the first token of (page p, head h): times D·bits/8 the place of its codes, times 4 of its scales.
__device__ __forceinline__ long long first_slot(const MxCacheView &c, int p, int h) {
    return ((long long)p * c.heads + h) * c.page;
}

}  // namespace q4mm
