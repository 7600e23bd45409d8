// kv8.cuh -- device helpers shared by the kernels of the paged 8-bit key / value cache.
//
// Cache layout: codes int8 [n_blocks][n_kv][block_size][d_h], one float32 scale
// for each (block, head): value = code * scale.  A request's tokens lie in the
// blocks its row of the block table names, block_size tokens to a block.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"

namespace rsq {

// Bits of the device status word set by these kernels (bit 1 is the bounded
// waits' timeout, 2 and 4 belong to the (Q, M) construction).
enum : int {
    kErrKvBlock = 8,   // a block id, slot or length outside the cache: those tokens were skipped
    kErrKvPool = 16,   // kv8_plan ran out of free blocks or of table columns
};

// One thread reports a bit (rare path).
__device__ __forceinline__ void kv8_report(int *status, int bits) {
    if (status) atomicOr(status, bits);
}

// A block's scale as the attention takes it: an infinite one reads as NaN.
__device__ __forceinline__ float kv8_scale(float v) {
    return fabsf(v) < __int_as_float(0x7F800000) ? v : __int_as_float(0x7FC00000);
}

// Entry i of the block table; -1 for an int64 one that is more than its lower half.
__device__ __forceinline__ int kv8_block(const Kv8Attention &p, long long i) {
    const int32_t *at = static_cast<const int32_t *>(p.table) + (i << p.wide_table);
    const int id = at[0], above = p.wide_table ? at[1] : 0;
    return above ? -1 : id;
}
// Its lower half alone, for where any block may be read in place of one that is none.
__device__ __forceinline__ int kv8_block_low(const Kv8Attention &p, long long i) {
    return static_cast<const int32_t *>(p.table)[i << p.wide_table];
}
// Entry i where the table's type is known.
template <bool kWide>
__device__ __forceinline__ int kv8_block(const Kv8Attention &p, long long i) {
    if (!kWide) return static_cast<const int32_t *>(p.table)[i];
    const int2 id = static_cast<const int2 *>(p.table)[i];
    return id.y ? -1 : id.x;
}

// The part of a request's state that every kernel clamps the same way: `n` new
// rows starting at row `first` of the T token rows, `pos0` the position of the
// first new token (negative when there are more new rows than tokens), `len`
// the tokens that the table can name.
struct Kv8Request {
    int first, n;
    long long pos0;
    int len;
};

__device__ __forceinline__ Kv8Request kv8_request(const int32_t *seq_len, const int32_t *cu_new, int b,
                                                  long long T, long long capacity) {
    Kv8Request r;
    const int seq = max(seq_len[b], 0);
    const int lo = max(cu_new[b], 0);
    const long long hi = min((long long)cu_new[b + 1], T);
    r.first = lo;
    r.n = hi > lo ? int(hi - lo) : 0;
    // positions follow the lengths as given, also when rows past T are cut off
    r.pos0 = (long long)seq - max((long long)cu_new[b + 1] - lo, 0ll);
    r.len = int(min((long long)seq, capacity));
    return r;
}

// Whether a batch has a long request (the CTA's answer, with a barrier), ...
__device__ __forceinline__ bool kv8_any_long(const int32_t *seq_len, const int32_t *cu_new, int B, int G, long long T,
                                             long long capacity) {
    bool any = false;
    for (int b = threadIdx.x; b < B; b += blockDim.x) {
        const Kv8Request r = kv8_request(seq_len, cu_new, b, T, capacity);
        const long long rows = (long long)r.n * G;
        any = any || (rows >= kKv8TcRows && rows * r.len >= kKv8TcWork);
    }
    return __syncthreads_or(any);
}
// ... and whether a request of it then goes to the tcgen05 kernel.
__device__ __forceinline__ bool kv8_goes_along(const Kv8Request &r, int G) { return (long long)r.n * G >= kKv8TcBeside; }

}  // namespace rsq
