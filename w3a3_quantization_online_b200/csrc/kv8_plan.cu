// kv8_plan.cu -- block tables and slot maps of the paged cache, from the requests' lengths.
//
// With c_b tokens in the cache and n_b new ones, request b needs the blocks
// [ceil(c_b / S), ceil((c_b + n_b) / S)) beyond those it holds.  They are taken
// from a list of free ids in request order, so request b's first fresh block
// is number cursor + sum_{i < b} need_i of the list, and new token t of it
// (row cu_b + t) gets position c_b + t and slot table[position / S] * S +
// position mod S.
//
// One launch: every CTA computes the two running sums over the requests for
// itself (at most 4096 of them, a few kilobytes out of L2), so no CTA waits for
// another, and then serves its share of requests and rows.  A row whose block
// is a fresh one reads its id from the free list, not from the table that
// another CTA may still be writing.  The call is a few microseconds of latency
// whatever its size: 3.0 us for a decode step of 64 requests (2 KB), 3.3 us for 27648
// rows of 48 prompts (0.35 MB).
#include "kv8.cuh"

namespace rsq {

namespace {

constexpr int kPlanThreads = 256;

template <class Id>
struct PlanArgs {
    const int32_t *ctx_len, *new_len;
    Id *table;
    const int32_t *free_blocks;
    const int32_t *cursor;
    int32_t *cursor_out, *cu_new, *seq_len, *positions;
    int64_t *slots;
    int *status;
    long long T;
    int B, width, shift, n_free;
};

__device__ __forceinline__ int clamp_i32(long long v) { return int(min(v, 2147483647ll)); }

// Id: of the block table's entries.
template <class Id>
__global__ void __launch_bounds__(kPlanThreads) k_kv8_plan(const PlanArgs<Id> p) {
    extern __shared__ int32_t psm[];
    int32_t *cu = psm;                    // B + 1: running sum of new tokens
    int32_t *start = psm + p.B + 1;       // B + 1: running sum of fresh blocks
    __shared__ long long wsum[2][kPlanThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int S = 1 << p.shift;

    // running sums, kPlanThreads requests at a time
    long long base_n = 0, base_f = 0;
    if (tid == 0) cu[0] = start[0] = 0;
    for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
        const int b = b0 + tid;
        long long n = 0, f = 0;
        if (b < p.B) {
            const long long c = max(p.ctx_len[b], 0);
            n = max(p.new_len[b], 0);
            const long long had = min((c + S - 1) >> p.shift, (long long)p.width);
            const long long has = min((c + n + S - 1) >> p.shift, (long long)p.width);
            f = has - had;
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long un = __shfl_up_sync(0xFFFFFFFFu, n, o), uf = __shfl_up_sync(0xFFFFFFFFu, f, o);
            if (lane >= o) n += un, f += uf;
        }
        if (lane == 31) wsum[0][warp] = n, wsum[1][warp] = f;
        __syncthreads();
        long long tn = 0, tf = 0;
#pragma unroll
        for (int w = 0; w < kPlanThreads / 32; ++w) {
            if (w < warp) n += wsum[0][w], f += wsum[1][w];
            tn += wsum[0][w], tf += wsum[1][w];
        }
        if (b < p.B) {
            cu[b + 1] = clamp_i32(base_n + n);
            start[b + 1] = clamp_i32(base_f + f);
        }
        base_n += tn, base_f += tf;
        __syncthreads();
    }

    const long long cursor = *p.cursor;
    auto fresh = [&](long long i) -> int {  // number i of the free list, -1 past its end
        return i >= 0 && i < p.n_free ? p.free_blocks[i] : -1;
    };

    // fresh table entries, one warp per request
    const int nwarps = gridDim.x * (kPlanThreads / 32);
    for (int b = blockIdx.x * (kPlanThreads / 32) + warp; b < p.B; b += nwarps) {
        const long long c = max(p.ctx_len[b], 0), n = max(p.new_len[b], 0);
        const int had = int(min((c + S - 1) >> p.shift, (long long)p.width));
        const int need = start[b + 1] - start[b];
        const long long from = cursor + start[b];
        for (int i = lane; i < need; i += 32) p.table[int64_t(b) * p.width + had + i] = fresh(from + i);
        if (lane == 0) {
            if (((c + n + S - 1) >> p.shift) > p.width || (need > 0 && (from < 0 || from + need > p.n_free)))
                kv8_report(p.status, kErrKvPool);
            p.seq_len[b] = clamp_i32(c + n);
            p.cu_new[b + 1] = cu[b + 1];
        }
    }
    if (blockIdx.x == 0 && tid == 0) {
        p.cu_new[0] = 0;
        *p.cursor_out = clamp_i32(cursor + base_f);
    }

    // positions and slots
    const int total = cu[p.B];
    for (long long t = (long long)blockIdx.x * kPlanThreads + tid; t < p.T; t += (long long)gridDim.x * kPlanThreads) {
        int32_t pos = -1;
        int64_t slot = -1;
        if (t < total) {
            int lo = 0, hi = p.B;  // the last request b with cu[b] <= t: cu[lo] <= t < cu[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cu[mid] <= t) lo = mid; else hi = mid;
            }
            const long long c = max(p.ctx_len[lo], 0);
            const long long at = c + (t - cu[lo]);
            const long long had = min((c + S - 1) >> p.shift, (long long)p.width);
            const long long col = at >> p.shift;
            pos = clamp_i32(at);
            if (col < p.width) {
                const Id id = col < had ? p.table[int64_t(lo) * p.width + col] : Id(fresh(cursor + start[lo] + (col - had)));
                // no cache has a block 2^31 - 1: larger ids become slots that kv8_append reports
                if (id >= 0) slot = (min(int64_t(id), int64_t(0x7FFFFFFF)) << p.shift) + (at & (S - 1));
            }
        }
        p.positions[t] = pos;
        p.slots[t] = slot;
    }
}

template <class Id>
cudaError_t launch(const PlanArgs<Id> &a, cudaStream_t s) {
    if (!a.status) return cudaErrorInvalidDevice;
    const long long by_rows = (a.T + kPlanThreads - 1) / kPlanThreads, by_req = (a.B + kPlanThreads / 32 - 1) / (kPlanThreads / 32);
    long long grid = by_rows > by_req ? by_rows : by_req;
    if (grid > num_sms()) grid = num_sms();
    if (grid < 1) grid = 1;
    k_kv8_plan<Id><<<unsigned(grid), kPlanThreads, 2 * (a.B + 1) * sizeof(int32_t), s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launch(1);
    return e;
}

}  // namespace

cudaError_t launch_kv8_plan(const int32_t *ctx_len, const int32_t *new_len, int B, void *block_table, bool wide_table,
                            int max_blocks, int block_size, const int32_t *free_blocks, int n_free, const int32_t *cursor,
                            int32_t *cursor_out, int32_t *cu_new, int32_t *seq_len, int32_t *positions, int64_t *slots,
                            long long T, cudaStream_t s) {
    int shift = 0;
    while ((1 << shift) < block_size) ++shift;
    int *status = device_status_word();
    if (wide_table)
        return launch(PlanArgs<int64_t>{ctx_len, new_len, static_cast<int64_t *>(block_table), free_blocks, cursor, cursor_out,
                                        cu_new, seq_len, positions, slots, status, T, B, max_blocks, shift, n_free}, s);
    return launch(PlanArgs<int32_t>{ctx_len, new_len, static_cast<int32_t *>(block_table), free_blocks, cursor, cursor_out,
                                    cu_new, seq_len, positions, slots, status, T, B, max_blocks, shift, n_free}, s);
}

}  // namespace rsq
