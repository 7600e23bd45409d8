// kv8_attention_tc.cu -- attention of long chunks of new tokens over the paged 8-bit cache (bf16, d_h 64 and 128).
//
// Bound by arithmetic: 4 d_h flops and one exponential per visible (row, key)
// pair.  On an SM, 256 rows by 128 keys of d_h = 128 take 2048 clocks of the tensor core
// (two fp16 products) and 2048 clocks of the exponential unit, so the two have to overlap.
//
// An item is 256 rows (new token x query head of a group) of one request and key
// head, worked on as two tiles A and B of 128 rows that take turns: while the tensor core
// multiplies for one, the warps of the other do its softmax.  Every CTA (one to an SM)
// gets the same share of the (item, 128 keys) units, in order, an item counting six units
// more than it has; an item that is cut leaves its pieces (output, maximum and sum of each row)
// in the workspace, and a second kernel puts them together in their order.
// (With whole items, taken from a counter, the last ones ran alone: 562 us where this took
// 504 to 519, for 4312 new tokens of three requests on up to 5952 older ones, 32 heads over 8 of keys,
// d_h 128: 762 TFLOP/s.  Repeated for seconds the GPU reaches its 1000 W and takes 555 us.  256 rows by 128 keys
// take 4400 to 4600 clocks, two thirds of it the softmax of a tile (3000) and the products behind it one after the
// other.  Without older tokens an item has 1 to 16 tiles beside its six: 25321 tokens of 20 requests take 731 us,
// 0.24 of the tensor core's rate.)
//   * Warps 0-3 and 4-7, a thread to a row: read the scores S (fp32, TMEM) of 128
//     keys, find the maximum, form the probabilities and put them back into the same
//     TMEM columns as fp16, where they are the A operand of the next product.
//   * Warp 12, one elected lane: issues S = Q K^T (Q and K in shared memory) and
//     O += P V (P in TMEM, V in shared memory as it lies there, N contiguous).
//   * The other seven warps: codes from the cache, made fp16 (exact: the byte
//     code ^ 0x80 under the exponent of 1024, minus 1152), into two stages of K
//     and V tiles in the SWIZZLE_128B layout that both products read.  A code
//     is converted once for 256 rows.
// q is scaled by a power of two per row so that its largest value lies in
// [2^14, 2^15): exact in fp16 down to 2^-31 of the largest, below that off by at most half of fp16's smallest
// step, 2^-39 of the largest.  k_scale joins the scores after the product.  v_scale belongs to a block of keys, so it has to join P: with m
// the running maximum of the scores and R a reference per row,
//     x = 2^(s - m) (float32, summed into l),  P = x 2^(m - R + log2 v_scale),
// R kept within 15 of the largest s + log2 v_scale so far and put 12 below it when
// that is passed: O is then scaled down in TMEM, which happens a few times per row.
// The largest P so far lies in [2^12, 2^15]: fp16 keeps 11 bits of all that are above
// 2^-26 of it (off by 2^-11 of itself at most: an eighth of what rounding the output to bf16 costs).
// Every mbarrier wait is bounded; a timeout sets a bit in the device status
// word, no more products are issued, and the CTA drains before freeing TMEM.
#include <type_traits>

#include "kv8.cuh"
#include "sm100.cuh"

namespace rsq {

using namespace sm100;

namespace {

constexpr int kTcThreads = 512;
constexpr int kConvWarps = 7;
constexpr int kMmaWarp = 12;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kPad = 6;              // what an item costs beside its key tiles, in tiles (3: 570 us, 4: 513, 6: 504)
constexpr int kLeast = 8;            // key tiles that are worth a CTA
constexpr int kDesc = 8;             // int32s that describe a cut item
constexpr float kSlack = 15.f, kBelow = 12.f;   // bound - R at most, and when R is set

template <int DH>
struct TcCfg {
    static constexpr int kTile = 128 * DH * 2;           // bytes of 128 rows or keys in fp16
    static constexpr int kOffQ = 0;                      // tiles A and B
    static constexpr int kOffK = 2 * kTile;              // two stages
    static constexpr int kOffV = kOffK + 2 * kTile;
    static constexpr int kOffBar = kOffV + 2 * kTile;
    static constexpr int kKFull = 0, kKEmpty = 2, kVFull = 4, kVEmpty = 6, kSFull = 8, kPReady = 10, kOFull = 12,
                         kQReady = 14, kPHalf = 16, kBars = 18;
    static constexpr int kOffTm = kOffBar + kBars * 8;
    static constexpr int kOffPre = kOffTm + 8;           // B + 1 int64
    static constexpr int kSmem = kOffPre + 1024;         // and the batch
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// 32 lanes x 16 consecutive 32-bit TMEM columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
          "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// Waits for the loads of `v`, and ties every use of it to the wait.
__device__ __forceinline__ void tmem_wait(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
                   "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]),
                   "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]),
                   "+r"(v[30]), "+r"(v[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_wait(uint32_t (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
                 :
                 : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem desc], fp16 inputs.
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t is;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(is)::"memory");
    return is != 0;
}

// Instruction descriptor, kind::f16: fp16 x fp16 -> fp32.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major) {
    return (1u << 4) | (uint32_t(b_mn_major) << 16) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

// Sixteen codes (one 16-byte piece) -> sixteen fp16 values.
__device__ __forceinline__ void codes16(const uint4 &u, uint32_t (&h)[8]) {
    const uint32_t w[4] = {u.x ^ 0x80808080u, u.y ^ 0x80808080u, u.z ^ 0x80808080u, u.w ^ 0x80808080u};
    const __half2 off = __floats2half2_rn(1152.f, 1152.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t a = prmt(w[i], 0x64646464u, 0x4140u), b = prmt(w[i], 0x64646464u, 0x4342u);
        const __half2 x = __hsub2(*reinterpret_cast<__half2 *>(&a), off);
        const __half2 y = __hsub2(*reinterpret_cast<__half2 *>(&b), off);
        h[2 * i] = *reinterpret_cast<const uint32_t *>(&x);
        h[2 * i + 1] = *reinterpret_cast<const uint32_t *>(&y);
    }
}

// A piece of an item: key tiles j0 .. j1 - 1 of 256 rows of a request and key head.
struct Piece {
    Kv8Request rq;
    int b, h, tile, rows;    // rows: of the item
    int j0, j1, nt;          // nt: key tiles of the item
    int kend;
    long long start, cost, from;   // the item's place among all costs, its cost, where the CTA begins in it
    bool whole, none;              // all of the item, nothing to do
};

struct TcSplit {
    int32_t *desc;           // kDesc a CTA: the cut item that begins in it
    float *ml, *o;           // per CTA two places of 256 rows: maximum and sum, output of the piece
};

// Costs are in 1/64 of a key tile, and grow by the same amount from each item of a
// request to the next 256 rows of it (the heads of the same rows cost the same).
struct Costs {
    long long first;
    int step, tiles;
    __device__ __forceinline__ long long before(long long tile) const { return tile * first + step * (tile * (tile - 1) / 2); }
};
__device__ __forceinline__ Costs costs_of(const Kv8Request &rq, int G) {
    const long long rows = (long long)rq.n * G;
    const long long keys = max(rq.pos0, 0ll) + unsigned(rows < 256 ? rows : 256) / unsigned(G);
    return Costs{64 * kPad + 64 + keys / 2, 128 / G, int((rows + 255) / 256)};
}

// NB: blocks in a tile of 128 keys.
template <int DH, int NB>
__global__ void __launch_bounds__(kTcThreads, 1) k_kv8_attention_tc(const Kv8Attention p, const TcSplit sp) {
    using C = TcCfg<DH>;
    constexpr int W = 128 / NB;           // keys of a block
    extern __shared__ uint8_t tsm_raw[];
    uint8_t *base = smem_align1024(tsm_raw);
    const uint32_t bars = smem_u32(base + C::kOffBar);
    auto bar = [&](int i) { return bars + 8u * uint32_t(i); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(base + C::kOffTm);
    long long *pre = reinterpret_cast<long long *>(base + C::kOffPre);
    __shared__ long long s_sum[kTcThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = p.n_heads / p.n_kv;
    const long long capacity = (long long)p.width << p.shift;

    if (!kv8_any_long(p.seq_len, p.cu_new, p.B, G, p.T, capacity)) {
        if (tid == 0) sp.desc[blockIdx.x * kDesc + 4] = 0;
        return;
    }
    // running sum of the costs
    {
        long long sum = 0;
        if (tid == 0) pre[0] = 0;
        for (int b0 = 0; b0 < p.B; b0 += kTcThreads) {
            const int b = b0 + tid;
            long long n = 0;
            if (b < p.B) {
                const Kv8Request rq = kv8_request(p.seq_len, p.cu_new, b, p.T, capacity);
                if (kv8_goes_along(rq, G)) {
                    const Costs c = costs_of(rq, G);
                    n = c.before(c.tiles) * p.n_kv;
                }
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long u = __shfl_up_sync(0xFFFFFFFFu, n, o);
                if (lane >= o) n += u;
            }
            if (lane == 31) s_sum[warp] = n;
            __syncthreads();
            long long all = 0;
            for (int w = 0; w < kTcThreads / 32; ++w) {
                if (w < warp) n += s_sum[w];
                all += s_sum[w];
            }
            if (b < p.B) pre[b + 1] = sum + n;
            sum += all;
            __syncthreads();
        }
    }
    // the same share of the costs for each CTA
    const long long total = pre[p.B];
    const long long share = max((total + gridDim.x - 1) / gridDim.x, 64ll * kLeast);
    const long long begin = blockIdx.x * share, stop = min(begin + share, total);
    if (tid == 0) sp.desc[blockIdx.x * kDesc + 4] = 0;
    if (begin >= total) return;

    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(C::kKFull + s), kConvWarps);
            mbar_init(bar(C::kVFull + s), kConvWarps);
            mbar_init(bar(C::kKEmpty + s), 1);
            mbar_init(bar(C::kVEmpty + s), 1);
            mbar_init(bar(C::kSFull + s), 1);
            mbar_init(bar(C::kOFull + s), 1);
            mbar_init(bar(C::kPReady + s), 4);
            mbar_init(bar(C::kPHalf + s), 4);
            mbar_init(bar(C::kQReady + s), 4);
        }
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // TMEM columns: S (and P) of A, of B, O of A, of B
    auto col_s = [&](int t) { return tmem + uint32_t(128 * t); };
    auto col_o = [&](int t) { return tmem + uint32_t(256 + 128 * t); };

    int err = 0;
    auto wait = [&](int b, uint32_t ph) {      // few instructions: there are many of these in little loops
        if (err || mbar_try_wait(bar(b), ph)) return;
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(bar(b), ph))
            if (globaltimer_ns() - t0 > kWaitLimitNs) {
                err |= kErrMbarTimeout;
                break;
            }
    };
    // the piece at `at`, which moves on to the next item
    auto piece_at = [&](long long &at) -> Piece {
        Piece it;
        int lo = 0, hi = p.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (pre[mid] <= at) lo = mid; else hi = mid;
        }
        it.b = lo;
        it.rq = kv8_request(p.seq_len, p.cu_new, lo, p.T, capacity);
        const Costs c = costs_of(it.rq, G);
        const long long x = at - pre[lo];
        int t0 = 0, t1 = c.tiles;
        while (t1 - t0 > 1) {
            const int mid = (t0 + t1) >> 1;
            if (c.before(mid) * p.n_kv <= x) t0 = mid; else t1 = mid;
        }
        it.tile = t0;
        it.cost = c.first + (long long)c.step * t0;
        const long long y = x - c.before(t0) * p.n_kv;
        int h0 = 0, h1 = p.n_kv;                      // (a 64-bit division is a long piece of code)
        while (h1 - h0 > 1) {
            const int mid = (h0 + h1) >> 1;
            if (mid * it.cost <= y) h0 = mid; else h1 = mid;
        }
        it.h = h0;
        it.from = y - it.h * it.cost;
        const long long rows = (long long)it.rq.n * G - 256ll * t0;
        it.rows = rows < 256 ? int(rows) : 256;
        const long long last = it.rq.pos0 + (256u * t0 + it.rows - 1) / unsigned(G) + 1;
        it.kend = int(max(min(last, (long long)it.rq.len), 0ll));
        it.nt = (it.kend + 127) / 128;
        const long long to = min(it.cost, it.from + stop - at);
        auto tile_at = [&](long long z) -> int {      // key tiles that begin before z: the first kPad lie before them
            return z >= it.cost ? it.nt : int(min((max(z - 64 * kPad, 0ll) + 63) / 64, (long long)it.nt));
        };
        it.j0 = tile_at(it.from);
        it.j1 = tile_at(to);
        it.whole = it.nt == 0 ? it.from == 0 : it.j0 == 0 && it.j1 == it.nt;
        it.none = it.j0 == it.j1 && !it.whole;
        it.start = at - it.from;
        at += to - it.from;
        return it;
    };

    // 512 threads of 128 registers: 256 x 160 for the rows, 256 x 96 for the rest
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
        // ------------------------------------------------------------ softmax
        const int t = warp >> 2;                                   // tile A or B
        const int r128 = (warp & 3) * 32 + lane;                   // this thread's row, and its TMEM lane
        const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
        const uint32_t ts = col_s(t) + lanes, to = col_o(t) + lanes;
        int cnt = 0;                                               // key tiles so far
        for (long long at = begin; at < stop; ) {
            const Piece it = piece_at(at);
            if (tid == 0 && it.from == 0 && !it.whole) {
                // a cut item begins here: its pieces lie in this CTA's second place (if the CTA
                // reaches its first key tile) and in the first ones of the CTAs behind
                const int last = int((it.start + min(it.cost - 1, 64ll * (kPad + it.nt - 1))) / share);
                const int lead = it.j1 > 0;
                if (last - int(blockIdx.x) + lead > 1) {
                    int *d = sp.desc + blockIdx.x * kDesc;
                    d[0] = it.b, d[1] = it.h, d[2] = it.tile, d[3] = last, d[4] = 1, d[5] = lead;
                }
            }
            if (it.rows <= 128 * t || it.none) continue;
            const int r = 128 * t + r128;                          // row of the item
            const bool live = r < it.rows;
            // (rows of 128 bytes or more that lie in memory: their number stays below 2^31)
            const unsigned idx = it.tile * 256u + r, tok_u = idx / unsigned(G);
            const int tok = int(tok_u), head = it.h * G + int(idx - tok_u * G);
            auto limit = [&](unsigned row) -> int {
                return int(max(min(it.rq.pos0 + (it.tile * 256u + row) / unsigned(G) + 1, (long long)it.rq.len), 0ll));
            };
            const int lim = live ? limit(r) : 0;
            const int lim_min = limit(128 * t);                    // of the tile's first row
            if (live && it.rq.pos0 + tok + 1 > it.rq.len) kv8_report(p.status, kErrKvBlock);

            // Q: scaled, fp16, swizzled.  A few lanes to a row, so that whole lines are read.
            constexpr int LR = DH / 8, RI = 32 / LR;               // lanes to a row, rows at a time
            const int sub = lane % LR, rsub = lane / LR;
            uint8_t *mine = base + C::kOffQ + t * C::kTile + (warp & 3) * 32 * 128;   // the warp's rows
            auto chunk = [&](int row, int c) -> uint4 * {          // 8 columns of one of them
                return reinterpret_cast<uint4 *>(mine + row * 128 + (c >> 3) * 16384 + (((c & 7) ^ (row & 7)) << 4));
            };
            const unsigned alive = __ballot_sync(0xFFFFFFFFu, live);
            float qf;
            {
                const long long off = (long long)(it.rq.first + tok) * p.ldq + (long long)head * DH;
                const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) + 8 * sub;
                int ex = 0;
#pragma unroll 1
                for (int c0 = 0; c0 < LR; c0 += 4) {               // a longer body costs more to fetch than it hides
                    uint4 u[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int row = (c0 + c) * RI + rsub;
                        const long long from = __shfl_sync(0xFFFFFFFFu, off, row);
                        u[c] = alive >> row & 1 ? *reinterpret_cast<const uint4 *>(q + from) : make_uint4(0u, 0u, 0u, 0u);
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t w[4] = {u[c].x, u[c].y, u[c].z, u[c].w};
                        // bit patterns of |q|; with a NaN every score of the row is one, whatever the scale
                        const unsigned m2 = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                                                     __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
                        unsigned most = max(m2 & 0xFFFFu, m2 >> 16);
#pragma unroll
                        for (int o = 1; o < LR; o <<= 1) most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
                        const int up = min(14 - max(int(most >> 7) - 127, -100), 114);
                        const int own = __shfl_sync(0xFFFFFFFFu, up, (lane % RI) * LR);
                        if (lane / RI == c0 + c) ex = own;
                        float sg = __uint_as_float(uint32_t(127 + up) << 23);
                        if (p.sm_scale < 0.f) sg = -sg;            // the sign goes with q: factors stay positive
                        if (most >= 0x7F80u) sg = NAN;             // an infinity too: every score is infinite or NaN
                        uint32_t h[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            h[e] = pack_f16(__uint_as_float(w[e] << 16) * sg, __uint_as_float(w[e] & 0xFFFF0000u) * sg);
                        *chunk((c0 + c) * RI + rsub, sub) = make_uint4(h[0], h[1], h[2], h[3]);
                    }
                }
                qf = __uint_as_float(uint32_t(127 - ex) << 23) * (fabsf(p.sm_scale) * kLog2e);
                fence_proxy_async_cta();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::kQReady + t));
            }

            // block ids and scales, one block to a lane: the id is read two tiles
            // ahead, its scales one, so that nobody waits for either
            float ks = 0.f, vs = 0.f;
            bool there = false;
            auto id_at = [&](int j) -> int {                       // -2: no tokens there
                const int key = j * 128 + (lane % NB) * W;
                return key < it.kend ? kv8_block(p, (long long)it.b * p.width + (key >> p.shift)) : -2;
            };
            auto scales = [&](int id) {
                there = id >= 0 && id < p.n_blocks;
                const long long at = (long long)(there ? id : 0) * p.n_kv + it.h;
                ks = p.k_scale[at];
                vs = p.v_scale[at];
                if (id != -2 && !there) kv8_report(p.status, kErrKvBlock);
            };
            int ahead = -2;
            if (it.j0 < it.j1) {
                scales(id_at(it.j0));
                ahead = id_at(it.j0 + 1);
            }

            float m = -INFINITY, l = 0.f, R = -INFINITY;
            for (int j = it.j0; j < it.j1; ++j, ++cnt) {
                const float ks_j = there ? kv8_scale(ks) : 0.f, vs_j = there ? kv8_scale(vs) : 0.f;
                const bool fine = vs_j == vs_j;
                const float lv_j = !fine ? NAN : vs_j > 0.f ? lg2(vs_j) : -INFINITY;
                const unsigned here = __ballot_sync(0xFFFFFFFFu, there);
                const bool bad = !__all_sync(0xFFFFFFFFu, fine);
                scales(ahead);
                ahead = id_at(j + 2);
                const int key0 = j * 128;
                // with a scale that is no number, what is masked must not meet it
                const bool mask = key0 + 128 > lim_min || here != 0xFFFFFFFFu || bad;

                wait(C::kSFull + t, uint32_t(cnt & 1));
                __syncwarp();
                tc_fence_after();
                // The scores are read twice, 32 at a time: for the maximum and for the
                // probabilities.  All 128 at once would take most of the registers.
                constexpr int HB = W < 32 ? 32 / W : 1;             // blocks of 32 keys
                constexpr int HW = 32 / HB;                         // keys of them
                auto seen = [&](int q) -> unsigned {        // mask of the row's keys 32 q ..
                    const int end = min(lim - key0 - 32 * q, 32);
                    unsigned bits = end <= 0 ? 0u : 0xFFFFFFFFu >> (32 - end);
#pragma unroll
                    for (int b = 0; b < HB; ++b)
                        if (!(here >> (32 * q / W + b) & 1)) bits &= ~((HB == 1 ? 0xFFFFFFFFu : 0xFFFFu) << (HW * b));
                    return bits;
                };
                // factors of the blocks' scores, and the blocks' log2 v_scale
                float fb[NB], lv[NB];
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    fb[b] = qf * __shfl_sync(0xFFFFFFFFu, ks_j, b);
                    lv[b] = __shfl_sync(0xFFFFFFFFu, lv_j, b);
                }
                float mt = -INFINITY, bound = -INFINITY, lvm = -INFINITY;
                auto maxima = [&](auto masked) {
                    constexpr bool kMask = decltype(masked)::value;
                    float mg[NB];
#pragma unroll
                    for (int b = 0; b < NB; ++b) mg[b] = -INFINITY;
                    uint32_t v[2][32];
                    tmem_ld32(ts, v[0]);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t(&x)[32] = v[q & 1];
                        tmem_wait(x);
                        if (q < 3) tmem_ld32(ts + uint32_t(32 * (q + 1)), v[(q + 1) & 1]);
                        if (kMask) {
                            const unsigned bits = seen(q);
#pragma unroll
                            for (int c = 0; c < 32; ++c) x[c] = bits >> c & 1 ? x[c] : 0xFF800000u;
                        }
#pragma unroll
                        for (int h = 0; h < HB; ++h) {
                            float a[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) a[e] = fmaxf(__uint_as_float(x[HW * h + e]), __uint_as_float(x[HW * h + e + 4]));
#pragma unroll
                            for (int c = HW * h + 8; c < HW * h + HW; c += 8)
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    a[e] = max3(a[e], __uint_as_float(x[c + e]), __uint_as_float(x[c + e + 4]));
                            const int b = 32 * q / W + h;
                            mg[b] = max3(mg[b], fmaxf(a[0], a[1]), fmaxf(a[2], a[3]));
                        }
                    }
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const float a = kMask && mg[b] == -INFINITY ? mg[b] : mg[b] * fb[b];   // not 0 * infinity
                        mt = fmaxf(mt, a);
                        bound = fmaxf(bound, a + lv[b]);
                        lvm = kMask && a == -INFINITY ? lvm : fmaxf(lvm, lv[b]);
                    }
                };
                if (mask) maxima(std::true_type{});
                else maxima(std::false_type{});
                const float mn = fmaxf(m, mt);
                const float ms = mn == -INFINITY ? 0.f : mn;
                l *= m == -INFINITY ? 0.f : ex2(m - ms);
                m = mn;
                // the reference of P; the factor 2^(m - R + log2 v_scale) stays below 2^120
                bound = fmaxf(bound, ms + lvm - 105.f);
                float down = 1.f;
                if (bound > R + kSlack) {
                    const float rn = bound - kBelow;
                    if (R != -INFINITY) down = ex2(R - rn);
                    R = rn;
                }
                if (j > it.j0 && __any_sync(0xFFFFFFFFu, down != 1.f)) {
                    wait(C::kOFull + t, uint32_t((cnt - 1) & 1));   // the product before is done
                    __syncwarp();
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < DH; c += 16) {
                        uint32_t v[16];
                        tmem_ld16(to + uint32_t(c), v);
                        tmem_wait(v);
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * down);
                        tmem_st16(to + uint32_t(c), v);
                    }
                }
                auto tell = [&](int b) {                            // P is there: all of it, or its first 64 keys
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(b + t));
                };
                // probabilities: 2^(s - m) (in l) times w
                float w[NB];
                bool plain = !mask;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    w[b] = ms - R + lv[b];                          // log2; beyond 120 only where nothing is seen; NaN stays
                    plain = plain && fabsf(w[b]) < 60.f;
                }
                if (__all_sync(0xFFFFFFFFu, plain)) {
                    // w is of moderate size: it goes into the exponent, and out of the sums again
                    constexpr int H = W < 32 ? W : 32, NC = 128 / H;       // keys at a time
                    uint32_t v[2][H];
                    auto fetch = [&](int c) {
                        if constexpr (H == 32) tmem_ld32(ts + uint32_t(H * c), v[c & 1]);
                        else tmem_ld16(ts + uint32_t(H * c), v[c & 1]);
                    };
                    fetch(0);
                    float2 sum[2];
#pragma unroll
                    for (int q = 0; q < NC; ++q) {
                        const int b = q * H / W;
                        uint32_t(&y)[H] = v[q & 1];
                        uint32_t pk[H / 2];
                        tmem_wait(y);
                        if (q + 1 < NC) fetch(q + 1);
                        if (q * H % W == 0) sum[0] = sum[1] = make_float2(0.f, 0.f);
                        const float2 f2 = make_float2(fb[b], fb[b]), r2 = make_float2(lv[b] - R, lv[b] - R);
#pragma unroll
                        for (int c = 0; c < H; c += 2) {
                            float2 x = fma2(make_float2(__uint_as_float(y[c]), __uint_as_float(y[c + 1])), f2, r2);
                            x.x = ex2(x.x);
                            x.y = ex2(x.y);
                            sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], x);
                            pk[c >> 1] = pack_f16(x.x, x.y);
                        }
                        // into columns that have been read (those of q + 1 lie further on)
                        if constexpr (H == 32) tmem_st16(ts + uint32_t(H / 2 * q), pk);
                        else tmem_st8(ts + uint32_t(H / 2 * q), pk);
                        if ((q + 1) * H % W == 0) l += ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y)) * ex2(-w[b]);
                        if ((q + 1) * H == 64) tell(C::kPHalf);
                    }
                } else {
                    float sum = 0.f;
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        uint32_t v[32], pk[16];
                        tmem_ld32(ts + uint32_t(32 * q), v);
                        const unsigned bits = mask ? seen(q) : 0xFFFFFFFFu;
                        tmem_wait(v);
#pragma unroll
                        for (int h = 0; h < HB; ++h) {
                            const float f = qf * __shfl_sync(0xFFFFFFFFu, ks_j, 32 * q / W + h);
                            // a value scale that is no number does not raise R, and counts whatever R is
                            const float lvb = __shfl_sync(0xFFFFFFFFu, lv_j, 32 * q / W + h), up = ms - R + lvb;
                            const float wb = lvb != lvb ? lvb : R == -INFINITY ? 0.f : ex2(up > 120.f ? 120.f : up);
#pragma unroll
                            for (int c = HW * h; c < HW * h + HW; c += 2) {
                                float y[2];
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    float x = fmaf(__uint_as_float(v[c + e]), f, -ms);
                                    x = ex2(bits >> (c + e) & 1 ? x : -INFINITY);
                                    sum += x;
                                    y[e] = bits >> (c + e) & 1 ? x * wb : 0.f;    // not 0 times a NaN that is masked
                                }
                                pk[c >> 1] = pack_f16(y[0], y[1]);
                            }
                        }
                        tmem_st16(ts + uint32_t(16 * q), pk);
                        if (q == 1) tell(C::kPHalf);
                    }
                    l += sum;
                }
                tell(C::kPReady);
            }

            // out
            if (it.j0 < it.j1) {
                wait(C::kOFull + t, uint32_t((cnt - 1) & 1));
                __syncwarp();
                tc_fence_after();
            }
            // 2^(R - m) in two factors: R may lie more than 126 below m
            const float half = R == -INFINITY ? 0.f : ex2(0.5f * (R - m));
            const float inv = l == 0.f ? 0.f : half / l;
            const long long place = (2ll * blockIdx.x + (it.from == 0)) * 256 + r;
            if (!it.whole && live) *reinterpret_cast<float2 *>(sp.ml + place * 2) = make_float2(m, l);
#pragma unroll 1
            for (int c = 0; c < DH; c += 32) {
                uint32_t v[32];
                if (it.j0 < it.j1) {
                    tmem_ld32(to + uint32_t(c), v);
                    tmem_wait(v);
                }
                if (live || it.whole) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        float y[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) y[k] = it.j0 < it.j1 && l != 0.f ? __uint_as_float(v[e + k]) * inv * half : 0.f;
                        if (it.whole) {
                            // by way of the place of its queries, which are no longer needed
                            *chunk(lane, (c + e) / 8) = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                                                                   pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
                        } else {
                            float4 *o = reinterpret_cast<float4 *>(sp.o + place * DH + c + e);
                            o[0] = make_float4(y[0], y[1], y[2], y[3]);
                            o[1] = make_float4(y[4], y[5], y[6], y[7]);
                        }
                    }
                }
                __syncwarp();
            }
            if (it.whole) {
                const long long off = ((long long)(it.rq.first + tok) * p.n_heads + head) * DH;
                __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + 8 * sub;
#pragma unroll 2
                for (int c = 0; c < LR; ++c) {
                    const int row = c * RI + rsub;
                    const long long to_row = __shfl_sync(0xFFFFFFFFu, off, row);
                    if (alive >> row & 1) *reinterpret_cast<uint4 *>(out + to_row) = *chunk(row, sub);
                }
                __syncwarp();
            }
            tc_fence_before();
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
        if (warp == kMmaWarp) {
        // ------------------------------------------------------------ products
            // The whole warp walks along, so that addresses and descriptors are the same in
            // every lane and stay in uniform registers; one elected lane issues.  (With one
            // lane in the loop alone, a product took some 90 clocks to issue, more than the
            // 64 it takes to run: 618 us for 4312 tokens on up to 8000 where this takes 562.)
            const uint32_t id_qk = idesc_f16_f32(128, 128, false), id_pv = idesc_f16_f32(128, DH, true);
            const uint32_t sm = smem_u32(base);
            auto wait_all = [&](int b, uint32_t ph) {
                if (err || !__all_sync(0xFFFFFFFFu, mbar_try_wait(bar(b), ph))) {
                    wait(b, ph);
                    err = __any_sync(0xFFFFFFFFu, err != 0) ? kErrMbarTimeout : 0;
                }
                tc_fence_after();
            };
            auto qk = [&](int t, int st) {
                const uint64_t ad = smem_desc_sw128(sm + uint32_t(C::kOffQ + t * C::kTile), 1024);
                const uint64_t bd = smem_desc_sw128(sm + uint32_t(C::kOffK + st * C::kTile), 1024);
#pragma unroll
                for (int k = 0; k < DH / 16; ++k) {
                    const uint32_t off = uint32_t((k >> 2) * 16384 + (k & 3) * 32) >> 4;
                    umma_f16(col_s(t), ad + off, bd + off, id_qk, k != 0);
                }
                umma_commit(bar(C::kSFull + t));
            };
            auto pv = [&](int t, int st, int half, bool first) {   // 64 keys
                const uint64_t bd =
                    smem_desc_sw128_lbo(sm + uint32_t(C::kOffV + st * C::kTile), 16384, 1024) + uint64_t(half * 8192 >> 4);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    umma_f16_ts(col_o(t), col_s(t) + uint32_t(32 * half + 8 * k), bd + uint64_t((k * 2048) >> 4), id_pv,
                                !first || k != 0);
                if (half) umma_commit(bar(C::kOFull + t));
            };
            int g = 0, nq = 0, nqb = 0, cb = 0;   // stages (and tiles of A), items of A, of B, tiles of B
            for (long long at = begin; at < stop; ) {
                const Piece it = piece_at(at);
                if (__any_sync(0xFFFFFFFFu, it.none)) continue;
                const bool two = __any_sync(0xFFFFFFFFu, it.rows > 128);
                const int nt = __reduce_max_sync(0xFFFFFFFFu, it.j1 - it.j0);
                wait_all(C::kQReady, uint32_t(nq++ & 1));
                if (two) wait_all(C::kQReady + 1, uint32_t(nqb++ & 1));
                if (nt > 0) {
                    wait_all(C::kKFull + (g & 1), uint32_t((g >> 1) & 1));
                    if (!err && elect_one()) {
                        qk(0, g & 1);
                        if (two) qk(1, g & 1);
                        umma_commit(bar(C::kKEmpty + (g & 1)));
                    }
                    __syncwarp();
                }
                for (int j = 0; j < nt; ++j, ++g) {
                    const int st = g & 1, nx = st ^ 1;
                    const bool more = j + 1 < nt;
                    // V of this tile and K of the next (which every warp writes later)
                    wait_all(more ? C::kKFull + nx : C::kVFull + st, uint32_t(more ? (g + 1) >> 1 & 1 : g >> 1 & 1));
                    for (int t = 0; t < 2; ++t) {
                        if (t && !two) break;
                        const uint32_t ph = uint32_t((t ? cb++ : g) & 1);
                        wait_all(C::kPHalf + t, ph);
                        if (!err && elect_one()) pv(t, st, 0, j == 0);
                        __syncwarp();
                        wait_all(C::kPReady + t, ph);              // the other half of P
                        if (!err && elect_one()) {
                            pv(t, st, 1, false);
                            if (more) qk(t, nx);
                            if (t || !two) {
                                umma_commit(bar(C::kVEmpty + st));
                                if (more) umma_commit(bar(C::kKEmpty + nx));
                            }
                        }
                        __syncwarp();
                    }
                }
                if (err) break;
            }
        } else {
        // ------------------------------------------------------------ codes to fp16
        // A unit is 8 keys by 64 columns: a lane takes 16 of them, 4 lanes to a key.
        constexpr int kUnits = 16 * (DH / 64);
        constexpr int kPer = (kUnits + kConvWarps - 1) / kConvWarps;
        const int cw = warp < kMmaWarp ? warp - 8 : warp - 9;
        const int kr = lane >> 2, piece = lane & 3;
        int g = 0;
        for (long long at = begin; at < stop; ) {
            const Piece it = piece_at(at);
            if (it.none) continue;
            // lane r < 16: the cache row of keys 8 r of a tile; the table is read a tile ahead
            // (the lower half of an int64 id will do: the softmax masks what is no block; both halves took 527 us
            // where this takes 521)
            auto id_at = [&](int j) -> int {
                const int key = j * 128 + (lane & 15) * 8;
                return key < it.kend ? kv8_block_low(p, (long long)it.b * p.width + (key >> p.shift)) : 0;
            };
            const int in_block = ((lane & 15) * 8) & ((1 << p.shift) - 1);
            long long row = 0;
            auto place = [&](int id) {
                if (id < 0 || id >= p.n_blocks) id = 0;            // a missing block reads block 0 and is masked
                row = (((long long)id * p.n_kv + it.h) << p.shift) + in_block;
            };
            uint4 rk[kPer], rv[kPer];
            const int own = kr * DH + piece * 16;
            auto load = [&](const int8_t *cache, uint4 (&r)[kPer]) {
#pragma unroll
                for (int u = 0; u < kPer; ++u) {
                    const int unit = cw + u * kConvWarps;
                    const long long at = __shfl_sync(0xFFFFFFFFu, row, unit & 15);
                    if (unit >= kUnits) continue;
                    const int8_t *src = cache + at * DH + (own + (unit >> 4) * 64);
                    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(r[u].x), "=r"(r[u].y), "=r"(r[u].z), "=r"(r[u].w)
                                 : "l"(src));
                }
            };
            // unit u of a tile lies 1024 u bytes into it (8 rows of 128 bytes; 16 of them to 64 columns)
            const uint32_t d0 = uint32_t(cw * 1024 + kr * 128 + (((2 * piece) ^ kr) << 4));
            const uint32_t d1 = uint32_t(cw * 1024 + kr * 128 + (((2 * piece + 1) ^ kr) << 4));
            auto put = [&](uint8_t *tile, const uint4 (&r)[kPer]) {
#pragma unroll
                for (int u = 0; u < kPer; ++u) {
                    if (cw + u * kConvWarps >= kUnits) continue;
                    uint32_t h[8];
                    codes16(r[u], h);
                    *reinterpret_cast<uint4 *>(tile + d0 + u * kConvWarps * 1024) = make_uint4(h[0], h[1], h[2], h[3]);
                    *reinterpret_cast<uint4 *>(tile + d1 + u * kConvWarps * 1024) = make_uint4(h[4], h[5], h[6], h[7]);
                }
                fence_proxy_async_cta();
                __syncwarp();
            };
            int ahead = 0;
            if (it.j0 < it.j1) {
                place(id_at(it.j0));
                ahead = id_at(it.j0 + 1);
                load(p.k_cache, rk);
                load(p.v_cache, rv);
            }
            for (int j = it.j0; j < it.j1; ++j, ++g) {
                const int st = g & 1;
                const uint32_t ph = uint32_t((g >> 1) & 1);
                const bool more = j + 1 < it.j1;
                place(ahead);
                ahead = id_at(j + 2);
                wait(C::kKEmpty + st, ph ^ 1u);
                put(base + C::kOffK + st * C::kTile, rk);
                if (lane == 0) mbar_arrive(bar(C::kKFull + st));
                if (more) load(p.k_cache, rk);
                wait(C::kVEmpty + st, ph ^ 1u);
                put(base + C::kOffV + st * C::kTile, rv);
                if (lane == 0) mbar_arrive(bar(C::kVFull + st));
                if (more) load(p.v_cache, rv);
            }
        }
        }
    }
    if (err) {
        kv8_report(p.status, err);
        drain_delay();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// The pieces of a cut item put together: o = sum o_k w_k / sum w_k, w_k = l_k 2^(m_k - m).
// A block to 32 rows, a warp to a row at a time, the pieces in their order.
template <int DH>
__global__ void __launch_bounds__(256) k_kv8_attention_tc_join(const Kv8Attention p, const TcSplit sp) {
    constexpr int E = DH / 32;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int i = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int *d = sp.desc + i * kDesc;
    if (!d[4]) return;
    const int h = d[1], tile = d[2], lead = d[5];
    const int n = d[3] - i + lead;
    const int G = p.n_heads / p.n_kv;
    const Kv8Request rq = kv8_request(p.seq_len, p.cu_new, d[0], p.T, (long long)p.width << p.shift);
    using Vec = typename std::conditional<E == 4, float4, float2>::type;
    for (int row = blockIdx.y * 32 + warp; row < int(blockIdx.y) * 32 + 32; row += 8) {
        const unsigned idx = tile * 256u + row, tok = idx / unsigned(G);
        if ((long long)idx >= (long long)rq.n * G) return;
        auto at = [&](int k) -> int { return (lead && k == 0 ? 2 * i + 1 : 2 * (i + k + 1 - lead)) * 256 + row; };
        float mm = -INFINITY;
        for (int k = lane; k < n; k += 32) mm = fmaxf(mm, sp.ml[at(k) * 2]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xFFFFFFFFu, mm, o));
        float sum = 0.f, a[E];
#pragma unroll
        for (int e = 0; e < E; ++e) a[e] = 0.f;
#pragma unroll 2
        for (int k = 0; k < n; ++k) {
            const int r = at(k);
            const float2 ml = *reinterpret_cast<const float2 *>(sp.ml + r * 2);
            const Vec v = *reinterpret_cast<const Vec *>(sp.o + (size_t)r * DH + lane * E);
            const float w = ml.y == 0.f ? 0.f : ml.y * ex2(ml.x - mm);
            sum += w;
            a[0] += v.x * w;
            a[1] += v.y * w;
            if constexpr (E == 4) {
                a[2] += v.z * w;
                a[3] += v.w * w;
            }
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) +
                             ((long long)(rq.first + int(tok)) * p.n_heads + h * G + int(idx - tok * G)) * DH + lane * E;
        if constexpr (E == 4)
            *reinterpret_cast<uint2 *>(out) = make_uint2(pack_bf16x2(a[0] * inv, a[1] * inv), pack_bf16x2(a[2] * inv, a[3] * inv));
        else *reinterpret_cast<uint32_t *>(out) = pack_bf16x2(a[0] * inv, a[1] * inv);
    }
}

template <int DH, int NB>
cudaError_t launch(const Kv8Attention &p, const TcSplit &sp, cudaStream_t s) {
    using C = TcCfg<DH>;
    constexpr int kMaxBatch = 4096;
    auto *kern = k_kv8_attention_tc<DH, NB>;
    static bool configured[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= 64 || !configured[dev])) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem + (kMaxBatch + 1) * 8);
        if (e == cudaSuccess && dev < 64) configured[dev] = true;
    }
    if (e != cudaSuccess) return e;
    const unsigned n = unsigned(num_sms());
    kern<<<n, kTcThreads, C::kSmem + (p.B + 1) * 8, s>>>(p, sp);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    count_launch(1);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(n, 8);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_kv8_attention_tc_join<DH>, p, sp);
    if (e == cudaSuccess) count_launch(1);
    return e;
}

template <int DH>
cudaError_t launch_nb(const Kv8Attention &p, const TcSplit &sp, cudaStream_t s) {
    switch (p.shift) {
        case 4: return launch<DH, 8>(p, sp, s);
        case 5: return launch<DH, 4>(p, sp, s);
        case 6: return launch<DH, 2>(p, sp, s);
        default: return launch<DH, 1>(p, sp, s);
    }
}

}  // namespace

size_t kv8_attention_tc_workspace_bytes(int dh) {
    return size_t(num_sms()) * (kDesc * 4 + 2 * 256 * 8 + 2 * 256 * size_t(dh) * 4);
}

cudaError_t launch_kv8_attention_tc(const Kv8Attention &p, void *workspace, cudaStream_t s) {
    TcSplit sp;
    sp.desc = static_cast<int32_t *>(workspace);
    sp.ml = reinterpret_cast<float *>(sp.desc + num_sms() * kDesc);
    sp.o = sp.ml + size_t(num_sms()) * 2 * 256 * 2;
    return p.dh == 64 ? launch_nb<64>(p, sp, s) : launch_nb<128>(p, sp, s);
}

}  // namespace rsq
