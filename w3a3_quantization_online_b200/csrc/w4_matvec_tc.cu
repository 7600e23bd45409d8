// w4_matvec_tc.cu -- products of token rows with 4-bit weights that carry group scales, on tcgen05.
//
//     y[t][n] = sum_k x[t][k] * (c[n][k] * s[n][k / group])
// for more than 24 rows, or 8 float32 ones (codes, scales and layouts as in w4_matvec.cu).  A CTA of 128 threads takes 128
// outputs, one to a thread, all tokens (up to 64) and a part of K, in spans of 64:
//   * TMA brings the codes of four spans at a time (128 rows of 128 bytes, swizzled;
//     a thread reading its own row from memory would touch a line per lane and load);
//     a thread makes bf16 of its row's 32 bytes of a span (exact) and stores them
//     as its lane of the A operand in TMEM, not in shared memory again;
//   * x, or the three bf16 parts of a float32 x as further rows, is the B operand in
//     shared memory (SWIZZLE_128B, K-major);
//   * one thread issues the four products of a span (M = 128, N = rows of x, K = 16)
//     into a fresh accumulator (two where groups are no multiple of 64), which every thread
//     reads back as its own row, multiplies by its scale and adds to its float32 sums.
// The products of a span run while the next codes are unpacked.  Up to 32 rows of x the
// A operand and the accumulators exist twice; beyond, four CTAs of an SM with one
// place each hide the products' latency better than two CTAs with two.  Unpacking and the
// float32 sums bound it, no longer the fragments of x that mma.sync needs for each
// 16 outputs (48 rows of 8192 x 8192, groups of 32, 39 us here; 57 us there).  Where the outputs alone do not fill the GPU a
// cluster of up to 8 CTAs splits K and joins its sums through distributed
// shared memory in a fixed order.
// Every mbarrier wait is bounded; a timeout sets a bit in the device status word.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace rsq {

using namespace sm100;

namespace {

constexpr int kTcThreads = 128;
constexpr int kSpan = 64;
constexpr int kStageSpans = 4;
constexpr int kCodes = 128 * kStageSpans * kSpan / 2;   // bytes of a stage of codes

struct MvTcArgs {
    const void *x;
    long long ldx;
    const uint8_t *codes;
    const float *scales;
    void *y;
    int *status;
    long long T;
    int N, K, group;
};

struct F16 {
    using T = __half;
    static __device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
};

// NX: rows of the B operand; TT: tokens (NX, or NX / 3 of a float32 x); G32: groups of
// 32 inputs or odd multiples of it, flushed every 32.
template <class IO, int NX, bool G32>
struct MvTcCfg {
    static constexpr int kParts = sizeof(typename IO::T) == 4 ? 3 : 1;
    static constexpr int TT = NX / kParts;
    static constexpr int kX = NX * 128;                    // bytes of x of a span
    static constexpr int kAcc = G32 ? 2 : 1;
    static constexpr int kBuf = 2 * (32 + NX * kAcc) <= 128 ? 2 : 1;       // places of codes and accumulators
    static constexpr int kRing = 2;                                        // stages of codes, four spans each
    static constexpr int kStages = kBuf + (kParts == 1 ? 2 : 1);           // of x
    static constexpr int kUsed = kBuf * (32 + NX * kAcc);                  // TMEM columns
    static constexpr int kCols = kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
    static_assert(kUsed <= 512, "TMEM columns");
    static constexpr int kSum = TT * 128 * 4;
    static constexpr int kOffX = kRing * kCodes;
    static constexpr int kData = kOffX + kStages * kX > kSum ? kOffX + kStages * kX : kSum;
    static constexpr int kOffBar = kData;
    static constexpr int kSmem = kOffBar + 48 + 1024;
    // CTAs to an SM: TMEM columns and registers (a sum per token)
    static constexpr int kMin = kCols > 256 ? 1 : kCols > 128 ? 2 : TT > 48 ? 3 : 4;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Eight codes of a word -> four bf16 pairs in order.
__device__ __forceinline__ void codes8(uint32_t w, uint32_t *o) {
    const __nv_bfloat162 off = __floats2bfloat162_rn(136.f, 136.f);
    uint32_t h[4];   // (e0, e4) (e1, e5) (e2, e6) (e3, e7): the exponent of 128 above code ^ 8
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t u = ((w >> (4 * i)) & 0x000F000Fu) ^ 0x43084308u;
        __nv_bfloat162 v = __hsub2(*reinterpret_cast<__nv_bfloat162 *>(&u), off);
        h[i] = *reinterpret_cast<uint32_t *>(&v);
    }
    o[0] = prmt(h[0], h[1], 0x5410u);
    o[1] = prmt(h[2], h[3], 0x5410u);
    o[2] = prmt(h[0], h[1], 0x7632u);
    o[3] = prmt(h[2], h[3], 0x7632u);
}

__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Loads of 16 columns; the wait ties the uses to it.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait(uint32_t (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
                 :
                 : "memory");
}

template <class IO, class OUT, int NX, bool G32>
__global__ void __launch_bounds__(kTcThreads, (MvTcCfg<IO, NX, G32>::kMin)) k_w4_matvec_tc(const __grid_constant__ CUtensorMap codes, const MvTcArgs p, int ks) {
    using C = MvTcCfg<IO, NX, G32>;
    using T = typename IO::T;
    constexpr int TT = C::TT, kBuf = C::kBuf, kRing = C::kRing;
    extern __shared__ uint8_t vsm_raw[];
    uint8_t *base = smem_align1024(vsm_raw);
    const uint32_t bar = smem_u32(base + C::kOffBar);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(base + C::kOffBar + 32);
    const int tid = threadIdx.x, warp = tid >> 5;
    const int n0 = blockIdx.x * 128;
    const long long tok0 = (long long)blockIdx.y * TT;
    const int n = min(n0 + tid, p.N - 1);
    const int groups = p.K / p.group;
    // stages of this CTA's part of K
    const int all = (p.K + kStageSpans * kSpan - 1) / (kStageSpans * kSpan);
    const int z = blockIdx.z, g0 = int((long long)all * z / ks), g1 = int((long long)all * (z + 1) / ks);
    const int s0 = g0 * kStageSpans, s1 = min(g1 * kStageSpans, (p.K + kSpan - 1) / kSpan);
    const float *srow = p.scales + (long long)n * groups;
    const T *x = static_cast<const T *>(p.x);
    int err = 0;

    // scales of a span: one, or one for each 32 inputs.  The group of the next one
    // is counted along, not divided for.
    // Four groups come with one load where rows of scales allow it.
    float sc[kStageSpans][C::kAcc];
    constexpr int kStep = G32 ? 32 : 64;
    int at_group = s0 * kSpan / p.group, in_group = s0 * kSpan - at_group * p.group;
    const bool four = groups % 4 == 0;
    float4 cur = make_float4(0.f, 0.f, 0.f, 0.f), ahead = cur;
    auto load_four = [&](int g) { return *reinterpret_cast<const float4 *>(srow + min(g & ~3, groups - 4)); };
    if (four) cur = load_four(at_group), ahead = load_four(at_group + 4);
    auto fetch_scales = [&](float (&f)[C::kAcc]) {
#pragma unroll
        for (int a = 0; a < C::kAcc; ++a) {
            const int e = at_group & 3;
            if (four) f[a] = e == 0 ? cur.x : e == 1 ? cur.y : e == 2 ? cur.z : cur.w;
            else f[a] = srow[min(at_group, groups - 1)];
            in_group += kStep;
            if (in_group >= p.group) {
                in_group -= p.group;
                ++at_group;
                if (four && (at_group & 3) == 0) cur = ahead, ahead = load_four(at_group + 4);
            }
        }
    };
    // x of a span: 16-byte chunk c of row r at c ^ (r & 7), 8-row groups of 1024 bytes
    const T *x_src = x + (tok0 + (tid >> 3)) * p.ldx + 8 * (tid & 7);
    const uint32_t x_dst = uint32_t((tid >> 3) * 128 + (((tid & 7) ^ ((tid >> 3) & 7)) << 4));
    auto fetch_x = [&](int s) {
        uint8_t *dst = base + C::kOffX + (s - s0) % C::kStages * C::kX;
        if constexpr (C::kParts == 1) {
            // a thread's chunks lie 16 rows apart
            const bool in = s < s1 && s * kSpan + 8 * (tid & 7) < p.K;
#pragma unroll
            for (int j = 0; j < NX / 16; ++j) {
                const bool live = in && tok0 + (tid >> 3) + 16 * j < p.T;
                cp16(smem_u32(dst) + x_dst + uint32_t(2048 * j), live ? x_src + s * kSpan + 16 * j * p.ldx : x, live);
            }
            cp_commit();
        } else {
            if (s >= s1) return;
#pragma unroll 2
            for (int i = tid; i < TT * 8; i += kTcThreads) {
                const int t = i >> 3, c = i & 7, k = s * kSpan + 8 * c;
                float r[8];
                if (tok0 + t < p.T && k < p.K) {
                    load8(reinterpret_cast<const float *>(x) + (tok0 + t) * p.ldx + k, r);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) r[e] = 0.f;
                }
                // parts cut off, not rounded: exact, and no finite value becomes an infinity; nothing is left of an infinity
#pragma unroll
                for (int q = 0; q < 3; ++q) {
                    const int row = q * TT + t;
                    uint32_t h[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) h[e] = prmt(__float_as_uint(r[2 * e]), __float_as_uint(r[2 * e + 1]), 0x7632u);
                    *reinterpret_cast<uint4 *>(dst + row * 128 + ((c ^ (row & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float left = r[e] - __uint_as_float(__float_as_uint(r[e]) & 0xFFFF0000u);
                        r[e] = q == 0 && fabsf(r[e]) == __int_as_float(0x7F800000) ? 0.f : left;
                    }
                }
            }
        }
    };

    const uint32_t full = bar + 16u;      // the codes' barriers, behind the products'
    auto fetch_codes = [&](int st) {      // one thread
        if (st >= g1) return;
        const int place = (st - g0) % kRing;
        mbar_expect_tx(full + 8u * uint32_t(place), uint32_t(kCodes));
        tma_load_2d(smem_u32(base + place * kCodes), &codes, st * (kStageSpans * kSpan / 2), n0, full + 8u * uint32_t(place));
    };
    if (tid == 0) {
        mbar_init(bar, 1);
        mbar_init(bar + 8u, 1);
        mbar_init(full, 1);
        mbar_init(full + 8u, 1);
        fence_mbar_init();
        prefetch_tmap(&codes);
        for (int st = 0; st < kRing; ++st) fetch_codes(g0 + st);
    }
    if constexpr (C::kParts == 1) {
        fetch_x(s0);
        fetch_x(s0 + 1);
    } else {
        fetch_x(s0);
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(tmem_slot), C::kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t lanes = uint32_t(warp * 32) << 16;
    // TMEM columns: the places of a span's codes (64 bf16 a lane), then of its accumulators
    auto col_a = [&](int i) { return tmem + uint32_t(32 * (i % kBuf)); };
    auto col_d = [&](int i) { return tmem + uint32_t(32 * kBuf + NX * C::kAcc * (i % kBuf)); };

    float y[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) y[t] = 0.f;
    auto flush = [&](int done, const float (&f)[C::kAcc]) {   // products of span number `done` of this CTA
        if (!mbar_wait(bar + 8u * uint32_t(done % kBuf), uint32_t((done / kBuf) & 1), err != 0)) err |= kErrMbarTimeout;
        __syncwarp();
        tc_fence_after();
        // up to 48 columns on the way together: a load alone takes longer than what is done with it
        constexpr int kCols = NX * C::kAcc, kBatch = kCols % 48 == 0 ? 48 : kCols % 32 == 0 ? 32 : 16;
#pragma unroll
        for (int c0 = 0; c0 < kCols; c0 += kBatch) {
            uint32_t v[kBatch / 16][16];
#pragma unroll
            for (int j = 0; j < kBatch / 16; ++j) tmem_ld16(col_d(done) + lanes + uint32_t(c0 + 16 * j), v[j]);
#pragma unroll
            for (int j = 0; j < kBatch / 16; ++j) {
                tmem_wait(v[j]);
                const int c = (c0 + 16 * j) % NX;
                const float fs = f[(c0 + 16 * j) / NX];
                if constexpr (C::kParts == 1) {
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const float2 r = fma2(make_float2(__uint_as_float(v[j][e]), __uint_as_float(v[j][e + 1])),
                                              make_float2(fs, fs), make_float2(y[c + e], y[c + e + 1]));
                        y[c + e] = r.x;
                        y[c + e + 1] = r.y;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if ((c + e) / TT < C::kParts) y[(c + e) % TT] = fmaf(__uint_as_float(v[j][e]), fs, y[(c + e) % TT]);
                }
            }
        }
    };

    const uint32_t idesc = idesc_bf16_f32(128, NX, false, false);
    int i = 0;
    for (int st = g0; st < g1; ++st) {
        const int place = (st - g0) % kRing, s = st * kStageSpans;
        if (!mbar_wait(full + 8u * uint32_t(place), uint32_t(((st - g0) / kRing) & 1), err != 0)) err |= kErrMbarTimeout;
        const uint8_t *row = base + place * kCodes + tid * 128;
#pragma unroll
        for (int u = 0; u < kStageSpans; ++u) {
            if (s + u >= s1) break;
            // with one place the sums are read first: there would be too many registers otherwise
            if constexpr (kBuf == 1) {
                if (i > 0) flush(i - 1, sc[(u + kStageSpans - 1) % kStageSpans]);
            }
            uint32_t pk[32];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint4 w = *reinterpret_cast<const uint4 *>(row + (((2 * u + h) ^ (tid & 7)) << 4));
                codes8(w.x, pk + 16 * h);
                codes8(w.y, pk + 16 * h + 4);
                codes8(w.z, pk + 16 * h + 8);
                codes8(w.w, pk + 16 * h + 12);
            }
            if constexpr (kBuf > 1) {
                if (i >= kBuf) flush(i - kBuf, sc[(u + kStageSpans - kBuf) % kStageSpans]);   // frees this span's place of codes, sums and x
            }
            fetch_scales(sc[u]);
            tmem_st32(col_a(i) + lanes, pk);
            if constexpr (C::kParts == 1) cp_wait<1>();     // x of this span is here (the next one's may not be)
            tmem_wait_st();
            fence_proxy_async_cta();
            tc_fence_before();
            __syncthreads();
            if (tid == 0) {
                tc_fence_after();
                const uint64_t bd = smem_desc_sw128(smem_u32(base + C::kOffX + i % C::kStages * C::kX), 1024);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (!err) umma_bf16_ts(col_d(i) + uint32_t(G32 ? (k >> 1) * NX : 0), col_a(i) + uint32_t(8 * k), bd + uint64_t(2 * k),
                                           idesc, G32 ? k & 1 : k != 0);
                if (!err) umma_commit(bar + 8u * uint32_t(i % kBuf));
                if (u == kStageSpans - 1 && !err) fetch_codes(st + kRing);    // everybody has read this stage
            }
            // into the place of the products that are done
            fetch_x(s + u + C::kStages - kBuf);
            ++i;
        }
    }
#pragma unroll
    for (int back = kBuf; back > 0; --back) {
        if (i < back) continue;
        float f[C::kAcc];
#pragma unroll
        for (int a = 0; a < C::kAcc; ++a) {
            f[a] = sc[0][a];
#pragma unroll
            for (int u = 1; u < kStageSpans; ++u) f[a] = (i - back) % kStageSpans == u ? sc[u][a] : f[a];
        }
        flush(i - back, f);
    }
    if (err) {
        if (p.status) atomicOr(p.status, err);
        drain_delay();
    }
    if constexpr (C::kParts == 1) cp_wait<0>();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, C::kCols);

    using O = typename OUT::T;
    if (ks == 1) {
        if (n0 + tid < p.N) {
#pragma unroll
            for (int t = 0; t < TT; ++t)
                if (tok0 + t < p.T) static_cast<O *>(p.y)[(tok0 + t) * p.N + n] = OUT::from_f(y[t]);
        }
        return;
    }
    float *sums = reinterpret_cast<float *>(base);     // [token][output], where x was
#pragma unroll
    for (int t = 0; t < TT; ++t) sums[t * 128 + tid] = y[t];
    cluster_sync();
    // this CTA's tokens z, z + ks, ...
    for (int t = z; t < TT; t += ks) {
        if (tok0 + t >= p.T) break;
        float v = 0.f;
        for (int r = 0; r < ks; ++r) v += ld_dsmem_f32(mapa(smem_u32(sums + t * 128 + tid), uint32_t(r)));
        if (n0 + tid < p.N) static_cast<O *>(p.y)[(tok0 + t) * p.N + n0 + tid] = OUT::from_f(v);
    }
    cluster_sync();    // nobody leaves while its sums are read
}

// The codes as N rows of K / 2 bytes, in boxes of 128 rows by 128 bytes; zeros outside.
bool make_codes_map(CUtensorMap *map, const uint8_t *codes, int N, int K) {
    using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static EncodeFn enc = nullptr;
    if (!enc) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess || !p) return false;
        enc = reinterpret_cast<EncodeFn>(p);
    }
    const cuuint64_t dims[2] = {cuuint64_t(K / 2), cuuint64_t(N)};
    const cuuint64_t strides[1] = {cuuint64_t(K / 2)};
    const cuuint32_t box[2] = {128, 128}, step[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(codes), dims, strides, box, step,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class IO, class OUT, int NX, bool G32>
cudaError_t launch_cfg(const MvTcArgs &a, cudaStream_t s) {
    using C = MvTcCfg<IO, NX, G32>;
    auto *kern = k_w4_matvec_tc<IO, OUT, NX, G32>;
    static bool configured[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= 64 || !configured[dev])) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e == cudaSuccess && dev < 64) configured[dev] = true;
    }
    if (e != cudaSuccess) return e;
    const long long tiles = (long long)((a.N + 127) / 128) * ((a.T + C::TT - 1) / C::TT);
    const int stages = (a.K + kStageSpans * kSpan - 1) / (kStageSpans * kSpan);
    // Split K as far as the GPU holds the CTAs.
    long long ks = (long long)num_sms() * C::kMin / tiles;
    ks = ks < 1 ? 1 : ks > 8 ? 8 : ks;
    if (ks > stages) ks = stages;
    CUtensorMap codes;
    if (!make_codes_map(&codes, a.codes, a.N, a.K)) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned((a.N + 127) / 128), unsigned((a.T + C::TT - 1) / C::TT), unsigned(ks));
    cfg.blockDim = dim3(kTcThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 1;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = unsigned(ks);
    cfg.attrs = at;
    cfg.numAttrs = ks > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, codes, a, int(ks));
}

template <class IO, class OUT, bool G32>
cudaError_t launch_nx(const MvTcArgs &a, cudaStream_t s) {
    if constexpr (sizeof(typename IO::T) == 4) {
        if (a.T <= 16) return launch_cfg<IO, OUT, 48, G32>(a, s);
        // 192 rows of x with two sums each would not fit TMEM
        if (a.T <= 32 || G32) return launch_cfg<IO, OUT, 96, G32>(a, s);
        return launch_cfg<IO, OUT, G32 ? 96 : 192, G32>(a, s);
    } else {
        if (a.T <= 32) return launch_cfg<IO, OUT, 32, G32>(a, s);
        if (a.T <= 48) return launch_cfg<IO, OUT, 48, G32>(a, s);
        return launch_cfg<IO, OUT, 64, G32>(a, s);
    }
}

template <class IO>
cudaError_t launch_out(const MvTcArgs &a, int out_dtype, cudaStream_t s) {
    const bool wide = a.group % 64 == 0;
    if (out_dtype == 0) return wide ? launch_nx<IO, F32, false>(a, s) : launch_nx<IO, F32, true>(a, s);
    if (out_dtype == 1) return wide ? launch_nx<IO, BF16, false>(a, s) : launch_nx<IO, BF16, true>(a, s);
    return wide ? launch_nx<IO, F16, false>(a, s) : launch_nx<IO, F16, true>(a, s);
}

}  // namespace

cudaError_t launch_w4_matvec_tc(const void *x, long long ldx, const uint8_t *codes_w, const float *scales_w, void *y,
                                long long T, int N, int K, int group, int dtype, int out_dtype, cudaStream_t s) {
    const MvTcArgs a{x, ldx, codes_w, scales_w, y, device_status_word(), T, N, K, group};
    if (!a.status) return cudaErrorInvalidDevice;
    const cudaError_t e = dtype == 0 ? launch_out<F32>(a, out_dtype, s) : launch_out<BF16>(a, out_dtype, s);
    if (e == cudaSuccess) count_launch(1);
    return e;
}

}  // namespace rsq
