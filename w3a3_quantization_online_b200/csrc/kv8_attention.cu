// kv8_attention.cu -- attention over the paged cache of 8-bit codes, any head size.
//
// For new token i of a request with `len` tokens (the new ones are its last n)
// and query head h of the group of key head h / G:
//     s_j = sm_scale * k_scale[block(j)] * <q, k_codes[j]>,  j <= pos_i = len - n + i
//     o   = sum_j softmax(s)_j * v_scale[block(j)] * v_codes[j]
// with running maximum and sum; a row that sees no token gives zeros.
//
// This kernel serves the head sizes that the tensor-core kernels do not (16, 32
// and 256).  One CTA per (row, query head); its 16 warps take every sixteenth
// tile of 32 keys, 16 columns of a key to a lane, all in float32, and are joined through
// shared memory.  It is bound by instructions (a conversion and an fma for each code and query
// head: the heads of a group do not share them) and, for one long request, by the warps there are.
// Two CTAs to an SM, that is 64 registers a thread, are worth more than the few that then spill: d_h 32 68 and 103 us, d_h 256
// 281 and 352 us with 78.  For d_h 256 the compiler is left to find them (281 us; 323 with the bound written down, as it
// then keeps fewer loads on the way), which it does as long as little else lives through the loop: so the type of
// the block table is a template argument, and the check of the query touches one of its columns.
// Measured: 61 requests of up to 8192 tokens, 32 query over 8 key heads, d_h 32 68 us, d_h 256
// 282 us (4 warps: 102 and 801; a key to a lane for the scores and a few columns to a lane
// for the values, the codes loaded byte by byte: 890 and 1509).
#include "kv8.cuh"

namespace rsq {

namespace {

constexpr int kGenWarps = 16;
constexpr float kLog2e = 1.4426950408889634f;

// Sixteen codes as float32: the byte code ^ 0x80 is the low byte of a number in [2^23, 2^23 + 256).
__device__ __forceinline__ void codes16(const uint4 &u, float (&f)[16]) {
    const uint32_t w[4] = {u.x ^ 0x80808080u, u.y ^ 0x80808080u, u.z ^ 0x80808080u, u.w ^ 0x80808080u};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        f[i] = __uint_as_float(prmt(w[i >> 2], 0x4B000000u, 0x7650u | uint32_t(i & 3))) - 8388736.f;
}

template <class IO, int dh, bool kWide>
__global__ void __launch_bounds__(kGenWarps * 32, dh == 256 ? 0 : 2) k_kv8_attention_any(const Kv8Attention p) {
    using T = typename IO::T;
    __shared__ float s_o[kGenWarps][dh];
    __shared__ float s_m[kGenWarps], s_l[kGenWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long t = blockIdx.x;
    const int head = blockIdx.y, kvh = head / (p.n_heads / p.n_kv);
    const int S = 1 << p.shift;

    if (t >= p.cu_new[p.B]) return;               // behind the last sequence: left as it was
    int lo = 0, hi = p.B;                          // cu[lo] <= t < cu[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.cu_new[mid] <= t) lo = mid; else hi = mid;
    }
    const Kv8Request r = kv8_request(p.seq_len, p.cu_new, lo, p.T, (long long)p.width << p.shift);
    if (t < r.first || t >= r.first + r.n) return;
    const long long pos = r.pos0 + (t - r.first);
    const int seen = int(max(min(pos + 1, (long long)r.len), 0ll));
    if (pos + 1 > r.len && tid == 0) kv8_report(p.status, kErrKvBlock);

    const T *q = static_cast<const T *>(p.q) + t * p.ldq + (long long)head * dh;
    constexpr int kLanes = dh / 16, kKeys = 32 / kLanes;   // lanes to a key, keys at a time
    const int sub = lane % kLanes, own = lane / kLanes;
    float o[16], qs[16];
#pragma unroll
    for (int e = 0; e < 16; e += 8) load8(q + sub * 16 + e, *reinterpret_cast<float(*)[8]>(&qs[e]));
    // an infinity makes every score of the row infinite or NaN: a row whose scores are all -infinity is NaN too
    float most = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) most = fmaxf(most, fabsf(qs[e])), o[e] = 0.f;
    qs[0] += most < INFINITY ? 0.f : NAN;
    float m = -INFINITY, l = 0.f;
    for (int key0 = warp * 32; key0 < seen; key0 += kGenWarps * 32) {
        const int key = key0 + lane;
        bool vis = key < seen;
        long long row = 0, at = 0;                 // (block, head) of this lane's key, its first code
        if (vis) {
            const int id = kv8_block<kWide>(p, (long long)lo * p.width + (key >> p.shift));
            vis = id >= 0 && id < p.n_blocks;
            if (!vis) kv8_report(p.status, kErrKvBlock);
            else row = (long long)id * p.n_kv + kvh, at = ((row << p.shift) + (key & (S - 1))) * dh;
        }
        float dot = 0.f;                           // unseen keys: the first code of the cache
#pragma unroll 4
        for (int it = 0; it < kLanes; ++it) {
            float b[16], a = 0.f;
            codes16(*reinterpret_cast<const uint4 *>(p.k_cache + __shfl_sync(0xFFFFFFFFu, at, it * kKeys + own) + sub * 16), b);
#pragma unroll
            for (int e = 0; e < 16; ++e) a = fmaf(qs[e], b[e], a);
#pragma unroll
            for (int d = 1; d < kLanes; d <<= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, d);
            a = __shfl_sync(0xFFFFFFFFu, a, lane % kKeys * kLanes);
            if (lane / kKeys == it) dot = a;
        }
        float s = -INFINITY, vs = 0.f;
        if (vis) {
            s = dot * (p.sm_scale * kv8_scale(p.k_scale[row]) * kLog2e);
            vs = kv8_scale(p.v_scale[row]);
        }
        const float mt = warp_max(s);
        const float mn = fmaxf(m, mt);
        const float base = mn == -INFINITY ? 0.f : mn;
        const float c1 = m == -INFINITY ? 0.f : exp2f(m - base);
        const float pr = vis ? exp2f(s - base) : 0.f;
        float sum = pr;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        l = l * c1 + sum;
        m = mn;
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] *= c1;
        const float pv = vis ? pr * vs : 0.f;      // unseen keys: 0 times the first code of the cache
#pragma unroll 4
        for (int j0 = 0; j0 < 32; j0 += kKeys) {
            const float w = __shfl_sync(0xFFFFFFFFu, pv, j0 + own);
            const long long from = __shfl_sync(0xFFFFFFFFu, at, j0 + own);
            float b[16];
            codes16(*reinterpret_cast<const uint4 *>(p.v_cache + from + sub * 16), b);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = fmaf(w, b[e], o[e]);
        }
    }
#pragma unroll
    for (int d = kLanes; d < 32; d <<= 1)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] += __shfl_xor_sync(0xFFFFFFFFu, o[e], d);
    if (lane == 0) s_m[warp] = m, s_l[warp] = l;
    if (own == 0) {
#pragma unroll
        for (int e = 0; e < 16; ++e) s_o[warp][sub * 16 + e] = o[e];
    }
    __syncthreads();
    float mm = s_m[0];
    for (int w = 1; w < kGenWarps; ++w) mm = fmaxf(mm, s_m[w]);
    float f[kGenWarps], ll = 0.f;
    for (int w = 0; w < kGenWarps; ++w) {
        f[w] = s_m[w] == -INFINITY ? (s_l[w] != s_l[w] ? s_l[w] : 0.f) : exp2f(s_m[w] - mm);
        ll += s_l[w] * f[w];
    }
    T *out = static_cast<T *>(p.out) + t * (long long)p.n_heads * dh + (long long)head * dh;
    for (int i = tid; i < dh; i += kGenWarps * 32) {
        float a = 0.f;
        for (int w = 0; w < kGenWarps; ++w) a += s_o[w][i] * f[w];
        out[i] = IO::from_f(ll == 0.f ? 0.f : a / ll);
    }
}

template <class IO, int dh>
void launch(const Kv8Attention &p, dim3 grid, cudaStream_t s) {
    if (p.wide_table) k_kv8_attention_any<IO, dh, true><<<grid, kGenWarps * 32, 0, s>>>(p);
    else k_kv8_attention_any<IO, dh, false><<<grid, kGenWarps * 32, 0, s>>>(p);
}

template <class IO>
void launch_dh(const Kv8Attention &p, dim3 grid, cudaStream_t s) {
    if (p.dh == 16) launch<IO, 16>(p, grid, s);
    else if (p.dh == 32) launch<IO, 32>(p, grid, s);
    else launch<IO, 256>(p, grid, s);
}

}  // namespace

cudaError_t launch_kv8_attention_any(const Kv8Attention &p, int dtype, cudaStream_t s) {
    const dim3 grid(unsigned(p.T), unsigned(p.n_heads));
    if (dtype == 0) launch_dh<F32>(p, grid, s);
    else launch_dh<BF16>(p, grid, s);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launch(1);
    return e;
}

}  // namespace rsq
