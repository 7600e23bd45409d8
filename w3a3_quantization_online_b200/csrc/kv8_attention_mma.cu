// kv8_attention_mma.cu -- attention over the paged 8-bit cache for few rows (decode, checked guesses), d_h 64 and 128.
//
// Bound by reading the codes once: 2 n_kv d_h bytes per token and sequence.
//
// Work: the R = n G rows (new token x query head of a group) of a request that
// share a key head are cut into tiles of RT (8 or 16) rows; a tile of rows reads
// its request's keys in tiles of 32.  All (row tile, key tile) units of the batch,
// in one order and with kFixed units added to each row tile for what it costs to
// begin and end one, are dealt out evenly: first to the CTAs (one to an SM), then
// a CTA's range to its warps, whatever the lengths.  A warp works through its
// range alone.  A row tile that one warp does from end to end is written
// directly; the parts (m, l, O) of others meet in shared memory once the CTA's
// warps are through, and those of a row tile that lies in several CTAs in the
// workspace, where a second kernel joins them; every join has a fixed order.
// Row tiles of few keys are not cut between CTAs.
//
// A warp holds Q and O in registers and loads K and V straight
// from memory into the registers of m16n8k16 products.  The
// 16-wide side of a product belongs to the long dimension: S^T = K Q^T (16 keys by 8
// rows) and O^T = V^T P^T (16 columns by 8 rows); with 8 rows in the other place half
// of the products would be of zeros.
//   * codes are exact in fp16: the byte code ^ 0x80 under the exponent of 1024,
//     minus 1152; so no rounding there, and the block scales stay outside;
//   * K: the order of d inside a product is free, so a lane takes 16 consecutive
//     bytes of its keys; V: the order of the output columns is free, so a lane
//     takes 16 (8) consecutive bytes of four keys and pairs them bytewise;
//   * q is scaled by a power of two per row so that its largest value lies in
//     [2^14, 2^15): a bf16 q is then exact in fp16 down to 2^-31 of the largest,
//     a float32 q is taken as the sum of two fp16 parts (22 bits and a sign down to 2^-17);
//     what is smaller is off by at most half of fp16's smallest step, 2^-39 of the largest;
//   * probabilities go in relative to their 32 keys' maximum, times 2^15: fp16
//     keeps 11 bits of them down to 2^-29 (off by 2^-11 of itself at most: an eighth of what
//     rounding the output to bf16 costs); for float32, two fp16 parts (2^-23).  They are
//     transposed from the first product's layout to the second's by movmatrix;
//   * every 32 keys are accumulated from zero and join the float32 O with one
//     multiply and one fma, which carry the change of the maximum and v_scale.
// The loads of the next keys are issued as soon as the products that read the
// registers are done, so about 6 KB per warp are on the way.
//
// Measured (32 query over 8 key heads of 128, bf16): two requests of up to 131072 tokens, 269 MB,
// 65 us (4.1 TB/s; the key loops run at about 6 TB/s); 61 requests of up to 8192 tokens, 95 MB, 36.5 us;
// one request of 200 tokens, 32 heads, 11.5 us.  34 float32 tokens of 17 requests, 20 over 4 heads of 64: 16 to 18 us.
// What is not key loops is finding the range, loading queries and joining.
#include "kv8.cuh"

namespace rsq {

namespace {

constexpr int kFixed = 2;     // cost of a row tile besides its keys, in tiles of 32 keys
constexpr int kWhole = 12;    // row tiles of up to this many key tiles are not cut between CTAs
constexpr float kLog2e = 1.4426950408889634f;

struct Split {
    int32_t *desc;   // per CTA: {b, key head, row tile, last CTA, valid} of the one that it begins and a later CTA ends
    float *ml;       // [CTA][2][RT][2]: of the row tile that an earlier CTA began, of the one that a later CTA ends
    float *o;        // [CTA][2][RT][DH]
    bool skip_long;  // where a request is long, it and others of many rows are left to another kernel
};
constexpr int kDesc = 8;
constexpr int kMaxBatch = 4096, kCached = 1024;   // requests; those whose lengths are kept in shared memory

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Bytes `sel` picks out of w (code ^ 0x80 each), two at a time, as fp16 codes.
__device__ __forceinline__ uint32_t code_pair(uint32_t w, uint32_t sel) {
    uint32_t u = prmt(w, 0x64646464u, sel);
    const __half2 v = __hsub2(*reinterpret_cast<__half2 *>(&u), __floats2half2_rn(1152.f, 1152.f));
    return *reinterpret_cast<const uint32_t *>(&v);
}

template <int BYTES>
struct Vec;
template <>
struct Vec<16> {
    static __device__ __forceinline__ void load(const int8_t *p, uint32_t (&w)[4]) {
        asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "l"(p));
    }
};
template <>
struct Vec<8> {
    static __device__ __forceinline__ void load(const int8_t *p, uint32_t (&w)[2]) {
        asm volatile("ld.global.nc.L1::no_allocate.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
    }
};

// Over the four lanes that share g; over the eight that share t.
__device__ __forceinline__ float max_t(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
}
__device__ __forceinline__ float max_g(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 4));
    v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 8));
    return fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 16));
}
__device__ __forceinline__ float sum_g(float v) {
    v += __shfl_xor_sync(0xFFFFFFFFu, v, 4);
    v += __shfl_xor_sync(0xFFFFFFFFu, v, 8);
    return v + __shfl_xor_sync(0xFFFFFFFFu, v, 16);
}

// Transposes an 8 x 8 matrix of 16-bit values (lane (g, t) holds row g, columns 2t and 2t + 1).
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
    return d;
}

// Sixteen elements of a query as they lie in memory.
template <class IO>
struct RawQ;
template <>
struct RawQ<BF16> {
    uint4 a[2];
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        a[0] = *reinterpret_cast<const uint4 *>(p);
        a[1] = *reinterpret_cast<const uint4 *>(p + 8);
    }
    __device__ __forceinline__ void get(float (&v)[16]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t w[4] = {a[i].x, a[i].y, a[i].z, a[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[8 * i + 2 * e] = __uint_as_float(w[e] << 16);
                v[8 * i + 2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
            }
        }
    }
};
template <>
struct RawQ<F32> {
    float4 a[4];
    __device__ __forceinline__ void load(const float *p) {
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4 *>(p + 4 * i);
    }
    __device__ __forceinline__ void get(float (&v)[16]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * i] = a[i].x, v[4 * i + 1] = a[i].y, v[4 * i + 2] = a[i].z, v[4 * i + 3] = a[i].w;
    }
};

template <class IO>
struct Parts;
template <>
struct Parts<BF16> { static constexpr int k = 1; };
template <>
struct Parts<F32> { static constexpr int k = 2; };

// A part of a row tile's result.
template <int DH, int RT>
struct alignas(16) Part {
    float o[RT][DH + 4];
    float m[RT], l[RT];
};
// What a warp leaves: [0] of a row tile that an earlier warp began, [1] of one that it began and did not end.
template <int DH, int RT>
struct alignas(16) Left {
    Part<DH, RT> part[2];
    int valid[2], ends0, busy;     // ends0: part 0 is the row tile's last
    int b[2], h[2], tile[2], rows[2], first[2], keys[2];   // of the parts' row tiles; first row of the request, key tiles
    long long start;               // first unit of part 1's row tile
};

template <int RT>
constexpr int warps_of() { return RT == 8 ? 12 : 8; }   // 168 and 255 registers a thread

// a / b and what remains, in 32 bits where that will do.
struct Quot {
    long long q;
    int r;
};
__device__ __forceinline__ Quot divide(long long a, int b) {
    if (!(a >> 32)) {
        const unsigned q = unsigned(a) / unsigned(b);
        return Quot{(long long)q, int(unsigned(a) - q * unsigned(b))};
    }
    return Quot{a / b, int(a % b)};
}

template <class IO, int DH, int RT>
__global__ void __launch_bounds__(warps_of<RT>() * 32, 1)
k_kv8_attention_mma(const Kv8Attention p, const Split sp) {
    using T = typename IO::T;
    constexpr int NW = warps_of<RT>();
    constexpr int QP = Parts<IO>::k;
    constexpr int KS = DH / 16;        // products along d
    constexpr int KV4 = DH / 64;       // 16-byte loads of a key by a lane
    constexpr int VB = DH / 8;         // bytes of a value row taken by a lane
    constexpr int NH = RT / 8;         // groups of 8 rows
    extern __shared__ __align__(16) uint8_t asm_raw[];
    Left<DH, RT> *left = reinterpret_cast<Left<DH, RT> *>(asm_raw);
    int4 *cached = reinterpret_cast<int4 *>(left + NW);             // first row, rows, length, position of the first row
    long long *pre = reinterpret_cast<long long *>(cached + min(p.B, kCached));   // B + 1: running sum of units
    __shared__ long long s_sum[NW], s_cut[2], s_own[NW + 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int G = p.n_heads / p.n_kv, S = 1 << p.shift;
    const long long capacity = (long long)p.width << p.shift;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    auto request = [&](int b) -> Kv8Request {
        if (b >= kCached) return kv8_request(p.seq_len, p.cu_new, b, p.T, capacity);
        const int4 c = cached[b];
        return Kv8Request{c.x, c.y, (long long)c.w, int(min((long long)c.z, capacity))};
    };
    auto key_tiles = [](const Kv8Request &r) -> int { return max(1, (r.len + 31) / 32); };

    const bool any_long = sp.skip_long && kv8_any_long(p.seq_len, p.cu_new, p.B, G, p.T, capacity);
    // running sum of the units
    {
        long long base = 0;
        if (tid == 0) pre[0] = 0;
        for (int b0 = 0; b0 < p.B; b0 += NW * 32) {
            const int b = b0 + tid;
            long long n = 0;
            if (b < p.B) {
                const Kv8Request r = kv8_request(p.seq_len, p.cu_new, b, p.T, capacity);
                if (b < kCached) cached[b] = make_int4(r.first, r.n, r.len, int(r.pos0));
                const long long rows = (long long)r.n * G;
                const int tiles = any_long && kv8_goes_along(r, G) ? 0 : int((rows + RT - 1) / RT);
                n = (long long)tiles * p.n_kv * (key_tiles(r) + kFixed);
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long u = __shfl_up_sync(0xFFFFFFFFu, n, o);
                if (lane >= o) n += u;
            }
            if (lane == 31) s_sum[warp] = n;
            __syncthreads();
            long long all = 0;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                if (w < warp) n += s_sum[w];
                all += s_sum[w];
            }
            if (b < p.B) pre[b + 1] = base + n;
            base += all;
            __syncthreads();
        }
    }
    const long long total = pre[p.B];
    const int nc = int(min((long long)gridDim.x, total));
    const int me = blockIdx.x;
    if (tid == 0) sp.desc[me * kDesc + 4] = 0;
    if (me >= nc) return;

    auto request_of = [&](long long u) -> int {  // the request of unit u < total
        int lo = 0, hi = p.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (pre[mid] <= u) lo = mid; else hi = mid;
        }
        return lo;
    };
    // Where a cut at unit u really goes: not into a row tile's fixed units, nor into one of up to `whole` key tiles.
    auto cut = [&](long long u, int whole) -> long long {
        if (u >= total) return total;
        const int b = request_of(u), keys = key_tiles(request(b)), per = keys + kFixed;
        const int c = divide(u - pre[b], per).r;
        if (c <= kFixed) return u - c;
        return keys > whole ? u : 2 * c <= per ? u - c : u - c + per;
    };
    // The CTA's range, then its warps': from the cut range, which may be much longer
    // than an even share where row tiles are short.
    if (tid < 2) s_cut[tid] = me + tid >= nc ? total : cut(divide(total * (me + tid), nc).q, kWhole);
    __syncthreads();
    const long long cta0 = s_cut[0], cta1 = s_cut[1];
    if (tid <= NW)
        s_own[tid] = tid == 0 ? cta0 : tid == NW ? cta1 : max(cta0, min(cta1, cut(cta0 + divide((cta1 - cta0) * tid, NW).q, 1)));
    __syncthreads();
    long long u = s_own[warp];
    const long long u1 = s_own[warp + 1];
    Left<DH, RT> &mine = left[warp];
    if (lane == 0) mine.valid[0] = mine.valid[1] = 0, mine.ends0 = 0, mine.busy = u < u1;
    int b = u < u1 ? request_of(u) : 0;

    while (u < u1) {
        while (pre[b + 1] <= u) ++b;
        const Kv8Request rq = request(b);
        const int keys = key_tiles(rq), per = keys + kFixed;
        const Quot at = divide(u - pre[b], per);
        const int c0 = at.r, tile = int(at.q) / p.n_kv, h = int(at.q) - tile * p.n_kv;
        const int c1 = int(min((long long)per, c0 + (u1 - u)));
        const int k0 = max(0, c0 - kFixed), k1 = max(0, c1 - kFixed);                // key tiles
        const int rows = min(RT, int((long long)rq.n * G - (long long)tile * RT));   // rows of this tile
        // tokens that the first and the last row of the tile see, and this lane's rows
        auto limit = [&](int row) -> int {
            const long long pos = rq.pos0 + (tile * RT + row) / G;
            return int(max(min(pos + 1, (long long)rq.len), 0ll));
        };
        const int lim_min = limit(0), lim_max = limit(rows - 1);
        if (lane == 0 && c0 == 0 && rq.pos0 + (tile * RT + rows - 1) / G + 1 > rq.len) kv8_report(p.status, kErrKvBlock);

        // Q on its way first: this lane's row of a group of 8 is g
        RawQ<IO> raw[NH][KV4];
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            const int idx = tile * RT + min(g + 8 * n, rows - 1), tok = idx / G;
            const T *q = static_cast<const T *>(p.q) + (long long)(rq.first + tok) * p.ldq +
                         (long long)(h * G + idx - tok * G) * DH + 16 * t;
#pragma unroll
            for (int c = 0; c < KV4; ++c) raw[n][c].load(q + 64 * c);
        }

        float o[NH][VB][2];   // [rows][this lane's columns VB g + j][row 2t + e]
        float m[NH][2], l[NH][2];
#pragma unroll
        for (int n = 0; n < NH; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[n][e] = -INFINITY, l[n][e] = 0.f;
#pragma unroll
                for (int j = 0; j < VB; ++j) o[n][j][e] = 0.f;
            }

        const int key_first = 32 * k0;
        const int nt = lim_max > key_first ? min(k1 - k0, (lim_max - key_first + 31) / 32) : 0;
        // block ids and scales of up to 32 tiles, one tile to a lane
        int id[2];
        float ks[2], vs[2];
        auto look_up = [&](int j0) {
            const int key = key_first + (j0 + lane) * 32;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int k2 = key + 16 * s;
                id[s] = -1;
                ks[s] = vs[s] = 0.f;
                if (s && p.shift > 4) {
                    id[1] = id[0], ks[1] = ks[0], vs[1] = vs[0];
                } else if (j0 + lane < nt && k2 < lim_max) {
                    const int i = kv8_block(p, (long long)b * p.width + (k2 >> p.shift));
                    if (i >= 0 && i < p.n_blocks) {
                        id[s] = i;
                        ks[s] = p.k_scale[(long long)i * p.n_kv + h];
                        vs[s] = p.v_scale[(long long)i * p.n_kv + h];
                    } else {
                        kv8_report(p.status, kErrKvBlock);
                    }
                }
            }
        };
        // cache rows of the two halves of tile j (a missing block reads block 0 and is masked)
        auto rows_of = [&](int j, long long (&row)[2]) {
            const int key = key_first + j * 32;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int i = max(__shfl_sync(0xFFFFFFFFu, id[s], j & 31), 0);
                row[s] = (((long long)i * p.n_kv + h) << p.shift) + ((key + 16 * s) & (S - 1));
            }
        };
        uint32_t kr[4][KV4][4];
        uint32_t vr[2][4][VB / 4];
        auto load_k = [&](const long long (&row)[2]) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < KV4; ++c)
                    Vec<16>::load(p.k_cache + (row[i >> 1] + 8 * (i & 1) + g) * DH + 64 * c + 16 * t, kr[i][c]);
        };
        auto load_v = [&](const long long (&row)[2]) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    Vec<VB>::load(p.v_cache + (row[k] + 2 * t + (r & 1) + 8 * (r >> 1)) * DH + VB * g, vr[k][r]);
        };
        long long row[2];
        if (nt > 0) {
            look_up(0);
            rows_of(0, row);
            load_k(row);
            load_v(row);
        }
        // Q into the B operand; the rows of this lane's scores and outputs are 2t, 2t + 1
        uint32_t qb[QP][NH][KS][2];
        float qf[NH][2];     // what a product of the scaled row stands for, in units of log2
        int lim[NH][2];
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            const bool live = g + 8 * n < rows;
            float v[KV4][16];
            float most = 0.f;
#pragma unroll
            for (int c = 0; c < KV4; ++c) {
                raw[n][c].get(v[c]);
#pragma unroll
                for (int s = 0; s < 16; ++s) {
                    v[c][s] = live ? v[c][s] : 0.f;
                    most = fmaxf(most, fabsf(v[c][s]));
                }
            }
            most = max_t(most);
            // 2^(14 - exponent), from the bits; rows below 2^-100 keep that factor
            const int ex = max(int(__float_as_uint(most) >> 23) - 127, -100);
            // an infinity makes every score of the row infinite or NaN: a row whose scores are all -infinity is NaN too
            const float up = most < INFINITY ? __uint_as_float(uint32_t(127 + min(14 - ex, 114)) << 23) : NAN;
            const float f = __uint_as_float(uint32_t(127 - min(14 - ex, 114)) << 23) * (p.sm_scale * kLog2e);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                qf[n][e] = __shfl_sync(0xFFFFFFFFu, f, 4 * (2 * t + e));
                lim[n][e] = 8 * n + 2 * t + e < rows ? limit(8 * n + 2 * t + e) : 0;
            }
#pragma unroll
            for (int c = 0; c < KV4; ++c)
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    float x[4];
#pragma unroll
                    for (int s = 0; s < 4; ++s) x[s] = v[c][4 * w + s] * up;
                    const uint32_t lo = pack_f16(x[0], x[1]), hi = pack_f16(x[2], x[3]);
                    qb[0][n][4 * c + w][0] = lo;
                    qb[0][n][4 * c + w][1] = hi;
                    if (QP == 2) {
                        const float2 fl = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
                        const float2 fh = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
                        qb[QP - 1][n][4 * c + w][0] = pack_f16(x[0] - fl.x, x[1] - fl.y);
                        qb[QP - 1][n][4 * c + w][1] = pack_f16(x[2] - fh.x, x[3] - fh.y);
                    }
                }
        }

        for (int j = 0; j < nt; ++j) {
            const int key0 = key_first + j * 32;
            float ksj[2], vsj[2];
            bool there[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                ksj[s] = kv8_scale(__shfl_sync(0xFFFFFFFFu, ks[s], j & 31));
                vsj[s] = kv8_scale(__shfl_sync(0xFFFFFFFFu, vs[s], j & 31));
                there[s] = __shfl_sync(0xFFFFFFFFu, id[s], j & 31) >= 0;
            }
            // scores of 16 keys (g and g + 8 of them in this lane) by 8 rows
            float s[NH][2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int n = 0; n < NH; ++n)
#pragma unroll
                    for (int c = 0; c < 4; ++c) s[n][i][c] = 0.f;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    const uint32_t w0 = kr[2 * i][k >> 2][k & 3] ^ 0x80808080u;
                    const uint32_t w1 = kr[2 * i + 1][k >> 2][k & 3] ^ 0x80808080u;
                    const uint32_t a0 = code_pair(w0, 0x4140u), a2 = code_pair(w0, 0x4342u);
                    const uint32_t a1 = code_pair(w1, 0x4140u), a3 = code_pair(w1, 0x4342u);
#pragma unroll
                    for (int n = 0; n < NH; ++n)
#pragma unroll
                        for (int q = 0; q < QP; ++q)
                            mma_f16(s[n][i], a0, a1, a2, a3, qb[q][n][k][0], qb[q][n][k][1]);
                }
            }
            const bool more = j + 1 < nt;
            if (more) {
                if (((j + 1) & 31) == 0) look_up(j + 1);
                rows_of(j + 1, row);
                load_k(row);
            }
            // softmax of the tile
            const bool mask = key0 + 32 > lim_min || !there[0] || !there[1];
            uint32_t pb[QP][NH][2][2];    // probabilities as the B operand: [16 keys][8 keys]
            float co[NH][2], cn[NH][2];
#pragma unroll
            for (int n = 0; n < NH; ++n) {
                float x[2][2][2];         // [row][16 keys][8 keys]
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float fa = qf[n][e] * ksj[0], fb = qf[n][e] * ksj[1];
                    float mh[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float &v = s[n][i][2 * c + e];
                            v *= i ? fb : fa;
                            if (mask && (key0 + 16 * i + 8 * c + g >= lim[n][e] || !there[i])) v = -INFINITY;
                        }
                        mh[i] = fmaxf(s[n][i][e], s[n][i][2 + e]);
                    }
                    // factors of the probabilities of the two halves, and what a product of the row then stands for
                    float mt, vt, rs = 1.f, xa = 1.f, xb = 1.f;
                    if (p.shift > 4) {
                        mt = max_g(fmaxf(mh[0], mh[1]));
                        vt = vsj[0];
                    } else {
                        // two blocks: relative to the larger of the row's products of probability and value scale
                        mh[0] = max_g(mh[0]);
                        mh[1] = max_g(mh[1]);
                        mt = fmaxf(mh[0], mh[1]);
                        const float b2 = mt == -INFINITY ? 0.f : mt;
                        vt = 0x1p-100f;
                        if (fabsf(vsj[0]) < INFINITY) vt = fmaxf(vt, ex2(mh[0] - b2) * fabsf(vsj[0]));
                        if (fabsf(vsj[1]) < INFINITY) vt = fmaxf(vt, ex2(mh[1] - b2) * fabsf(vsj[1]));
                        rs = 32768.f / vt;
                        xa = fabsf(vsj[0]) < INFINITY ? vsj[0] : NAN;
                        xb = fabsf(vsj[1]) < INFINITY ? vsj[1] : NAN;
                    }
                    const float base = mt == -INFINITY ? 0.f : mt;
                    const float mn = fmaxf(m[n][e], mt);
                    co[n][e] = m[n][e] == -INFINITY ? 0.f : ex2(m[n][e] - mn);
                    cn[n][e] = mt == -INFINITY ? 0.f : ex2(mt - mn);
                    float sum = 0.f;
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float v = ex2(s[n][i][2 * c + e] - base);
                            sum += v;
                            if (p.shift > 4) v *= 32768.f;
                            else if (s[n][i][2 * c + e] != -INFINITY) v = v * (i ? xb : xa) * rs;   // masked: not 0 times a NaN
                            x[e][i][c] = v;
                        }
                    l[n][e] = l[n][e] * co[n][e] + sum * cn[n][e];
                    m[n][e] = mn;
                    cn[n][e] = mt == -INFINITY ? 0.f : cn[n][e] * (vt * 0x1p-15f);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint32_t w = pack_f16(x[0][i][c], x[1][i][c]);
                        pb[0][n][i][c] = transpose8(w);
                        if (QP == 2) {
                            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
                            pb[QP - 1][n][i][c] = transpose8(pack_f16(x[0][i][c] - f.x, x[1][i][c] - f.y));
                        }
                    }
            }
            // products with the values: 16 columns by 8 rows
#pragma unroll
            for (int w = 0; w < VB / 4; ++w) {
                uint32_t x[2][4];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    // bytes of two keys, interleaved: columns 0, 1 and 2, 3 of the word
                    const uint32_t r0 = vr[k][0][w] ^ 0x80808080u, r1 = vr[k][1][w] ^ 0x80808080u;
                    const uint32_t r2 = vr[k][2][w] ^ 0x80808080u, r3 = vr[k][3][w] ^ 0x80808080u;
                    x[k][0] = prmt(r0, r1, 0x5140u);
                    x[k][1] = prmt(r0, r1, 0x7362u);
                    x[k][2] = prmt(r2, r3, 0x5140u);
                    x[k][3] = prmt(r2, r3, 0x7362u);
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {    // columns 2c and 2c + 1 of the word
                    float acc[NH][4];
#pragma unroll
                    for (int n = 0; n < NH; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t a0 = code_pair(x[k][c], 0x4140u), a1 = code_pair(x[k][c], 0x4342u);
                        const uint32_t a2 = code_pair(x[k][2 + c], 0x4140u), a3 = code_pair(x[k][2 + c], 0x4342u);
#pragma unroll
                        for (int n = 0; n < NH; ++n)
#pragma unroll
                            for (int q = 0; q < QP; ++q) mma_f16(acc[n], a0, a1, a2, a3, pb[q][n][k][0], pb[q][n][k][1]);
                    }
#pragma unroll
                    for (int n = 0; n < NH; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float(&oo)[2] = o[n][4 * w + 2 * c + i];
                            const float2 v = fma2(make_float2(acc[n][2 * i], acc[n][2 * i + 1]),
                                                  make_float2(cn[n][0], cn[n][1]),
                                                  mul2(make_float2(oo[0], oo[1]), make_float2(co[n][0], co[n][1])));
                            oo[0] = v.x;
                            oo[1] = v.y;
                        }
                }
            }
            if (more) load_v(row);
        }

        const bool begins = c0 == 0, ends = c1 == per;
        if (begins && ends) {
            // the whole row tile: out directly, a lane's columns are contiguous
#pragma unroll
            for (int n = 0; n < NH; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = 8 * n + 2 * t + e;
                    const float ls = sum_g(l[n][e]);
                    if (row < rows) {
                        const int idx = tile * RT + row;
                        T *out = static_cast<T *>(p.out) +
                                 ((long long)(rq.first + idx / G) * p.n_heads + h * G + idx % G) * DH + VB * g;
                        const float inv = ls == 0.f ? 0.f : 1.f / ls;
#pragma unroll
                        for (int j = 0; j < VB; j += 8) {
                            float v[8];
#pragma unroll
                            for (int x = 0; x < 8; ++x) v[x] = o[n][j + x][e] * inv;
                            store8(out + j, v);
                        }
                    }
                }
        } else {
            const int slot = begins ? 1 : 0;
            Part<DH, RT> &pt = mine.part[slot];
#pragma unroll
            for (int n = 0; n < NH; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = 8 * n + 2 * t + e;
                    const float ls = sum_g(l[n][e]);
                    if (g == 0) pt.m[row] = m[n][e], pt.l[row] = ls;
#pragma unroll
                    for (int j = 0; j < VB; j += 4)
                        *reinterpret_cast<float4 *>(&pt.o[row][VB * g + j]) =
                            make_float4(o[n][j][e], o[n][j + 1][e], o[n][j + 2][e], o[n][j + 3][e]);
                }
            if (lane == 0) {
                mine.valid[slot] = 1;
                mine.b[slot] = b, mine.h[slot] = h, mine.tile[slot] = tile, mine.rows[slot] = rows;
                mine.first[slot] = rq.first, mine.keys[slot] = keys;
                if (begins) mine.start = u;
                else mine.ends0 = ends;
            }
        }
        u += c1 - c0;
    }

    // Join what the CTA's warps left.  A row tile that a warp began, or that the
    // first warp at work took over from an earlier CTA, goes on in the part 0 of the
    // warps behind it until one of them ends it.  A thread looks at one of these, then
    // the rows of all of them are shared out among the warps.
    __shared__ int s_last[2 * NW], s_done[2 * NW], s_any;   // last warp of it (-1: none); ends in this CTA
    if (tid == 0) s_any = 0;
    __syncthreads();
    if (tid < 2 * NW) {
        const int w0 = tid >> 1, slot = tid & 1;
        bool ours = left[w0].valid[slot] != 0;
#pragma unroll 1
        for (int w = 0; ours && slot == 0 && w < w0; ++w) ours = !left[w].busy;
        int last = w0;
        bool ended = slot == 0 && left[w0].ends0;
#pragma unroll 1
        for (int w = w0 + 1; ours && w < NW && !ended; ++w)
            if (left[w].busy) last = w, ended = left[w].ends0 && left[w].valid[0];
        if (ours) s_any = 1;
        s_last[tid] = ours ? last : -1;
        s_done[tid] = slot == 1 && ended;
        if (ours && slot == 1 && !ended) {
            // it ends in the last CTA whose range begins before its last unit
            const long long end = left[w0].start + left[w0].keys[1] + kFixed;
            int *d = sp.desc + me * kDesc;
            d[0] = left[w0].b[1], d[1] = left[w0].h[1], d[2] = left[w0].tile[1], d[3] = int((end * nc - 1) / total), d[4] = 1;
        }
    }
    __syncthreads();
    if (!s_any) return;
    int turn = 0;
#pragma unroll 1
    for (int k = 0; k < 2 * NW; ++k) {
        if (s_last[k] < 0) continue;
        const int w0 = k >> 1, slot = k & 1, last = s_last[k];
        const Left<DH, RT> &l0 = left[w0];
        const int c = lane * (DH / 32);
#pragma unroll 1
        for (int row = 0; row < l0.rows[slot]; ++row, turn = turn + 1 == NW ? 0 : turn + 1) {
            if (turn != warp) continue;
            float mm = l0.part[slot].m[row];
#pragma unroll 1
            for (int w = w0 + 1; w <= last; ++w)
                if (left[w].busy) mm = fmaxf(mm, left[w].part[0].m[row]);
            float ll = 0.f, a[DH / 32];
#pragma unroll
            for (int e = 0; e < DH / 32; ++e) a[e] = 0.f;
#pragma unroll 1
            for (int w = w0; w <= last; ++w) {
                if (!left[w].busy) continue;
                const Part<DH, RT> &pt = left[w].part[w == w0 ? slot : 0];
                const float f = pt.m[row] == -INFINITY ? 0.f : ex2(pt.m[row] - mm);
                ll += pt.l[row] * f;
#pragma unroll
                for (int e = 0; e < DH / 32; ++e) a[e] += pt.o[row][c + e] * f;
            }
            if (s_done[k]) {
                const int idx = l0.tile[slot] * RT + row, tok = idx / G;
                T *out = static_cast<T *>(p.out) +
                         ((long long)(l0.first[slot] + tok) * p.n_heads + l0.h[slot] * G + idx - tok * G) * DH + c;
                const float inv = ll == 0.f ? 0.f : 1.f / ll;
#pragma unroll
                for (int e = 0; e < DH / 32; ++e) out[e] = IO::from_f(a[e] * inv);
            } else {
                const long long r = (long long)(me * 2 + slot) * RT + row;
#pragma unroll
                for (int e = 0; e < DH / 32; ++e) sp.o[r * DH + c + e] = a[e];
                if (lane == 0) sp.ml[r * 2] = mm, sp.ml[r * 2 + 1] = ll;
            }
        }
    }
}

// Joins the parts of the tiles that were cut: CTA (i, y) takes two rows of the
// tile that CTA i of the kernel above began, four warps to a row.
template <class IO, int DH, int RT>
__global__ void __launch_bounds__(256) k_kv8_attention_join(const Kv8Attention p, const Split sp) {
    using T = typename IO::T;
    constexpr int E = DH / 32;
    __shared__ float s_o[8][DH];
    __shared__ float s_l[8];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int i = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int *d = sp.desc + i * kDesc;
    if (!d[4]) return;
    const int b = d[0], h = d[1], tile = d[2], last = d[3];
    const int row = blockIdx.y * 2 + (warp >> 2), part = warp & 3;
    // part 0 lies in this CTA's second place, the others in the first one of the CTAs behind it
    auto at = [&](int k) -> long long { return (long long)(k == 0 ? 2 * i + 1 : 2 * (i + k)) * RT + row; };
    const int n = last - i + 1;
    float mm = -INFINITY;
    for (int k = lane; k < n; k += 32) mm = fmaxf(mm, sp.ml[at(k) * 2]);
    mm = warp_max(mm);
    float ll = 0.f;
    float a[E];
#pragma unroll
    for (int e = 0; e < E; ++e) a[e] = 0.f;
#pragma unroll 4
    for (int k = part; k < n; k += 4) {
        const long long r = at(k);
        const float m = sp.ml[r * 2];
        const float f = m == -INFINITY ? 0.f : ex2(m - mm);
        ll += sp.ml[r * 2 + 1] * f;
#pragma unroll
        for (int e = 0; e < E; ++e) a[e] += sp.o[r * DH + lane + 32 * e] * f;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[warp][lane + 32 * e] = a[e];
    if (lane == 0) s_l[warp] = ll;
    __syncthreads();
    const Kv8Request rq = kv8_request(p.seq_len, p.cu_new, b, p.T, (long long)p.width << p.shift);
    const int G = p.n_heads / p.n_kv;
    for (int x = threadIdx.x; x < 2 * DH; x += 256) {
        const int rr = x / DH, dd = x % DH;
        const long long idx = (long long)tile * RT + blockIdx.y * 2 + rr;
        if (idx >= (long long)rq.n * G) continue;
        float o = 0.f, lsum = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) o += s_o[4 * rr + w][dd], lsum += s_l[4 * rr + w];
        static_cast<T *>(p.out)[((rq.first + idx / G) * p.n_heads + h * G + idx % G) * DH + dd] =
            IO::from_f(lsum == 0.f ? 0.f : o * (1.f / lsum));
    }
}

template <class IO, int DH, int RT>
cudaError_t launch(const Kv8Attention &p, void *workspace, bool skip_long, cudaStream_t s) {
    constexpr int NW = warps_of<RT>();
    const int n = num_sms();
    Split sp;
    sp.desc = static_cast<int32_t *>(workspace);
    sp.ml = reinterpret_cast<float *>(sp.desc + n * kDesc);
    sp.o = sp.ml + n * 2 * RT * 2;
    sp.skip_long = skip_long;
    const size_t parts = sizeof(Left<DH, RT>) * NW;
    auto *kern = k_kv8_attention_mma<IO, DH, RT>;
    static bool configured[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= 64 || !configured[dev])) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 int(parts + kCached * sizeof(int4) + size_t(kMaxBatch + 1) * sizeof(long long)));
        if (e == cudaSuccess && dev < 64) configured[dev] = true;
    }
    if (e != cudaSuccess) return e;
    kern<<<unsigned(n), NW * 32,
           parts + size_t(p.B < kCached ? p.B : kCached) * sizeof(int4) + size_t(p.B + 1) * sizeof(long long), s>>>(p, sp);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    count_launch(1);
    if (((long long)p.width << p.shift) <= 32 * kWhole) return e;   // nothing can be cut between CTAs
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(n), RT / 2);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_kv8_attention_join<IO, DH, RT>, p, sp);
    if (e == cudaSuccess) count_launch(1);
    return e;
}

template <class IO, int DH>
cudaError_t launch_rt(const Kv8Attention &p, void *workspace, bool skip_long, cudaStream_t s) {
    // Tiles of 8 rows where a request has that many or fewer on average: half the
    // registers and half the softmax of the 16-row tile.
    if (p.T * (p.n_heads / p.n_kv) <= 8ll * p.B) return launch<IO, DH, 8>(p, workspace, skip_long, s);
    return launch<IO, DH, 16>(p, workspace, skip_long, s);
}

}  // namespace

bool kv8_attention_mma_supports(int dh) { return dh == 64 || dh == 128; }

size_t kv8_attention_mma_workspace_bytes(int dh) {
    size_t most = 0;
    for (int rt = 8; rt <= 16; rt += 8) {
        const size_t n = size_t(num_sms());
        const size_t bytes = n * (kDesc * 4 + 2 * rt * 8 + 2 * size_t(rt) * dh * 4);
        if (bytes > most) most = bytes;
    }
    return most;
}

cudaError_t launch_kv8_attention_mma(const Kv8Attention &p, int dtype, void *workspace, bool skip_long, cudaStream_t s) {
    if (p.dh == 64)
        return dtype == 0 ? launch_rt<F32, 64>(p, workspace, skip_long, s) : launch_rt<BF16, 64>(p, workspace, skip_long, s);
    return dtype == 0 ? launch_rt<F32, 128>(p, workspace, skip_long, s) : launch_rt<BF16, 128>(p, workspace, skip_long, s);
}

}  // namespace rsq
