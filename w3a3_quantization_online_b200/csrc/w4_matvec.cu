// w4_matvec.cu -- products of a few token rows with 4-bit weights that carry group scales.
//
//     y[t][n] = sum_k x[t][k] * (c[n][k] * s[n][k / group])
// c: 4-bit two's complement codes, packed as the activation codes are (element
// 2i in the low nibble of byte i); s: float32.  The weights are read once and
// are what bounds the call: N K / 2 bytes of codes and 4 N K / group of scales.
//
// The products run on the tensor cores in bf16 (m16n8k16: 16 outputs, 8 tokens):
// a 4-bit code is exact in bf16, and so is x, or the three bf16 parts of a
// float32 x (8 + 8 + 8 bits), which are taken as further rows of x, split when a stage
// is written (5 float32 rows are 15 columns, two tiles of 8).  32 or 64 inputs with one scale are accumulated
// from zero and then join the float32 sum times that scale, so nothing is
// rounded below 32 bits before the output.
//
// A CTA takes 32 RW outputs, all tokens (up to 24, or 8 float32 ones; more go to tcgen05) and a part of K, in stages of
// 8 KB of codes and the x that belongs to them, brought in by cp.async four
// stages deep.  RW warps share the outputs (two 16-row tiles each, so that a
// fragment of x serves both), the other factor KW = 8 / RW shares each stage's
// K, 64 to a warp.  Many tokens take RW = 4: x is read once per 128 outputs; few
// take RW = 1, which makes more CTAs.  Where the outputs alone do not fill the
// GPU, a cluster of up to 8 CTAs splits K and joins its sums through
// distributed shared memory, in a fixed order.
//
// The order of k inside a product is free as long as both operands agree: a lane
// takes the eight codes of a word, its pairs (e0, e4) (e1, e5) (e2, e6) (e3, e7)
// come out by shifts and masks with the exponent of 128 put above them, and one
// subtraction of 136 turns 128 + (code ^ 8) into the code; x is permuted alike.
//
// Measured: one bf16 row, 4096 x 4096, groups of 128 (8.9 MB) 7.6 to 8.2 us, latency; five float32 rows, 4096 x
// 12288, groups of 64 (29 MB) 22 to 23 us, issue slots 0.54 busy with unpacking and the products of the parts.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace rsq {

using namespace sm100;

namespace {

constexpr int kMvWarps = 8, kMvThreads = kMvWarps * 32;
constexpr int kWBytes = 8192;   // codes of a stage

struct MatvecArgs {
    const void *x;
    long long ldx;
    const uint8_t *codes;
    const float *scales;
    void *y;
    long long T;
    int N, K, group;
};

struct F16 {
    using T = __half;
    static __device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16 bytes into shared memory, zeros instead where `live` is false (the address is then not read).
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Eight codes of a word -> bf16 pairs (e0, e4), (e1, e5), (e2, e6), (e3, e7).
__device__ __forceinline__ void codes8(uint32_t w, uint32_t (&h)[4]) {
    const __nv_bfloat162 off = __floats2bfloat162_rn(136.f, 136.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t u = ((w >> (4 * i)) & 0x000F000Fu) ^ 0x43084308u;
        __nv_bfloat162 v = __hsub2(*reinterpret_cast<__nv_bfloat162 *>(&u), off);
        h[i] = *reinterpret_cast<uint32_t *>(&v);
    }
}

// Eight consecutive values of a row of x from shared memory -> the B registers of their two products.
__device__ __forceinline__ void load_x(const uint8_t *row, int chunk, int flip, uint32_t (&b)[4]) {
    const uint4 u = *reinterpret_cast<const uint4 *>(row + ((chunk ^ flip) << 4));
    b[0] = prmt(u.x, u.z, 0x5410u);
    b[1] = prmt(u.x, u.z, 0x7632u);
    b[2] = prmt(u.y, u.w, 0x5410u);
    b[3] = prmt(u.y, u.w, 0x7632u);
}

// RW: warps along the outputs; NT: tiles of eight rows of x (tokens, or parts of tokens).
template <class IO, int RW, int NT>
struct MvCfg {
    static constexpr int KW = kMvWarps / RW;
    static constexpr int BN = 32 * RW;              // outputs of a CTA
    static constexpr int KC = 64 * KW;              // inputs of a stage
    static constexpr int kParts = sizeof(typename IO::T) == 4 ? 3 : 1;
    static constexpr int TT = 8 * NT / kParts;      // tokens of a CTA
    static constexpr int kXRow = KC * 2;            // bytes of a row of x of a stage
    static constexpr int kLoads = kParts == 1 ? 1 : (TT * (KC / 4) + kMvThreads - 1) / kMvThreads;   // float4 a thread
    static constexpr int kStage = kWBytes + 8 * NT * kXRow;
    static constexpr int kStages = 4 * kStage <= 200 * 1024 ? 4 : 3;
    static constexpr int kSum = KW * BN * 8 * NT * 4;  // the warps' sums, over the stages when they are done
    static constexpr int kSmem = kStages * kStage > kSum ? kStages * kStage : kSum;
    static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
};

template <class IO, class OUT, bool G32, int RW, int NT>
__global__ void __launch_bounds__(kMvThreads) k_w4_matvec(const MatvecArgs p, int ks) {
    using C = MvCfg<IO, RW, NT>;
    using T = typename IO::T;
    constexpr int kParts = C::kParts;
    extern __shared__ __align__(128) uint8_t msm[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int rw = warp % RW, kw = warp / RW;
    const int n0 = blockIdx.x * C::BN;
    const long long tok0 = (long long)blockIdx.y * C::TT;
    const int groups = p.K / p.group;
    const int all = (p.K + C::KC - 1) / C::KC;
    const int z = blockIdx.z, st0 = int((long long)all * z / ks), st1 = int((long long)all * (z + 1) / ks);

    // stage st -> ring place.  Codes: rows of KC / 2 bytes, 16-byte chunk c of
    // row r at c ^ (r's pair); x: rows of KC elements, halves of 128 bytes
    // swapped in odd rows: both are then read without bank conflicts.
    constexpr int kWChunks = C::KC / 32;            // 16-byte chunks of a row of codes
    constexpr int kXChunks = C::kXRow / 16;
    auto wswz = [](int r, int c) { return kWChunks == 4 ? c ^ ((r >> 1) & 3) : c ^ (r & 7); };
    auto fetch = [&](int st, int place) {
        const uint32_t base = smem_u32(msm) + uint32_t(place * C::kStage);
        const int k0 = st * C::KC;
#pragma unroll
        for (int i = tid; i < C::BN * kWChunks; i += kMvThreads) {
            const int r = i / kWChunks, c = i % kWChunks;
            const bool live = k0 + 32 * c < p.K;
            const int n = min(n0 + r, p.N - 1);
            cp16(base + uint32_t(r * (C::KC / 2) + (wswz(r, c) << 4)),
                 p.codes + (live ? (long long)n * (p.K / 2) + k0 / 2 + 16 * c : 0), live);
        }
        if constexpr (kParts == 1) {
#pragma unroll
            for (int i = tid; i < 8 * NT * kXChunks; i += kMvThreads) {
                const int r = i / kXChunks, c = i % kXChunks;
                const int k = k0 + 8 * c;
                const bool live = tok0 + r < p.T && k < p.K;
                cp16(base + uint32_t(kWBytes + r * C::kXRow + ((c ^ ((r & 1) << 2)) << 4)),
                     static_cast<const T *>(p.x) + (live ? (tok0 + r) * p.ldx + k : 0), live);
            }
        }
    };
    // a float32 x goes through registers, a stage ahead of its place in the ring
    float4 ahead[C::kLoads];
    auto load_f32 = [&](int st) {
#pragma unroll
        for (int j = 0; j < C::kLoads; ++j) {
            const int i = tid + j * kMvThreads, t = i / (C::KC / 4), k = st * C::KC + 4 * (i % (C::KC / 4));
            ahead[j] = t < C::TT && tok0 + t < p.T && k < p.K
                           ? *reinterpret_cast<const float4 *>(static_cast<const float *>(p.x) + (tok0 + t) * p.ldx + k)
                           : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    };
    auto store_f32 = [&](int place) {
#pragma unroll
        for (int j = 0; j < C::kLoads; ++j) {
            const int i = tid + j * kMvThreads, t = i / (C::KC / 4), k4 = i % (C::KC / 4);
            if (t >= C::TT) continue;
            // (adding 0 sets the upper bits of every NaN)
            float r[4] = {__fadd_rn(ahead[j].x, 0.f), __fadd_rn(ahead[j].y, 0.f), __fadd_rn(ahead[j].z, 0.f),
                          __fadd_rn(ahead[j].w, 0.f)};
            // parts cut off, not rounded: exact, and no finite value becomes an infinity; the lower parts of an
            // infinity are NaN, and left out when the parts are joined
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                const int row = q * C::TT + t;
                *reinterpret_cast<uint2 *>(msm + place * C::kStage + kWBytes + row * C::kXRow +
                                           (((k4 >> 1) ^ ((row & 1) << 2)) << 4) + 8 * (k4 & 1)) =
                    make_uint2(prmt(__float_as_uint(r[0]), __float_as_uint(r[1]), 0x7632u),
                               prmt(__float_as_uint(r[2]), __float_as_uint(r[3]), 0x7632u));
#pragma unroll
                for (int e = 0; e < 4; ++e) r[e] -= __uint_as_float(__float_as_uint(r[e]) & 0xFFFF0000u);
            }
        }
    };

    float y[2][NT][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) y[m][i][e] = 0.f;

    // scales of this lane's rows (16 m + g, + 8) for the inputs of a stage
    constexpr int kF = G32 ? 2 : 1;
    const float *srow[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) srow[i] = p.scales + (long long)min(n0 + 32 * rw + 8 * i + g, p.N - 1) * groups;
    float sc[kF][4];
    auto scales_of = [&](int st) {
#pragma unroll
        for (int f = 0; f < kF; ++f) {
            const int gi = min((st * C::KC + 64 * kw + 32 * f) / p.group, groups - 1);
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[f][i] = srow[i][gi];
        }
    };

#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) {
        if (st0 + i < st1) fetch(st0 + i, i);
        cp_commit();
    }
    if (st0 < st1) scales_of(st0);
    if constexpr (kParts > 1) {
        // rows behind the parts stay zero
        constexpr int kRest = (8 * NT - 3 * C::TT) * kXChunks;
        if constexpr (kRest > 0)
            for (int i = tid; i < C::kStages * kRest; i += kMvThreads)
                *reinterpret_cast<uint4 *>(msm + i / kRest * C::kStage + kWBytes + 3 * C::TT * C::kXRow + i % kRest * 16) =
                    make_uint4(0u, 0u, 0u, 0u);
        load_f32(st0);
        store_f32(0);
        load_f32(st0 + 1);
    }
    int place = 0;
    for (int st = st0; st < st1; ++st) {
        cp_wait<C::kStages - 2>();
        __syncthreads();   // the stage is here, and the place of the one before is free
        {
            const int nx = st + C::kStages - 1;
            if (nx < st1) fetch(nx, (place + C::kStages - 1) % C::kStages);
            cp_commit();
            if constexpr (kParts > 1) {
                store_f32((place + 1) % C::kStages);
                load_f32(st + 2);
            }
        }
        const uint8_t *wst = msm + place * C::kStage;
        const uint8_t *xst = wst + kWBytes;
        float cur[kF][4];
#pragma unroll
        for (int f = 0; f < kF; ++f)
#pragma unroll
            for (int i = 0; i < 4; ++i) cur[f][i] = sc[f][i];
        if (st + 1 < st1) scales_of(st + 1);

        float acc[2][NT][4];
#pragma unroll
        for (int f = 0; f < 2; ++f) {      // 32 inputs: two products
            if (f == 0 || G32) {
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int i = 0; i < NT; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[m][i][e] = 0.f;
            }
            const int c = 2 * kw + f;      // 16-byte chunk of the codes
            uint32_t a[2][2][4];           // [16-row tile][product]
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int r0 = 32 * rw + 16 * m + g, r1 = r0 + 8;
                uint32_t h0[4], h1[4];
                codes8(*reinterpret_cast<const uint32_t *>(wst + r0 * (C::KC / 2) + (wswz(r0, c) << 4) + 4 * t), h0);
                codes8(*reinterpret_cast<const uint32_t *>(wst + r1 * (C::KC / 2) + (wswz(r1, c) << 4) + 4 * t), h1);
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    a[m][s][0] = h0[2 * s], a[m][s][1] = h1[2 * s];
                    a[m][s][2] = h0[2 * s + 1], a[m][s][3] = h1[2 * s + 1];
                }
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                uint32_t b[4];
                load_x(xst + (8 * i + g) * C::kXRow, 4 * c + t, (g & 1) << 2, b);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    mma_bf16(acc[m][i], a[m][0], b[0], b[1]);
                    mma_bf16(acc[m][i], a[m][1], b[2], b[3]);
                }
            }
            if (f == 1 || G32) {
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int i = 0; i < NT; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            y[m][i][e] = fmaf(acc[m][i][e], cur[G32 ? f : 0][2 * m + (e >> 1)], y[m][i][e]);
            }
        }
        place = place + 1 == C::kStages ? 0 : place + 1;
    }
    cp_wait<0>();
    __syncthreads();       // the stages are done with: their place holds the sums now

    // s_y[kw][token][output]
    float *s_y = reinterpret_cast<float *>(msm);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s_y[(kw * 8 * NT + 8 * i + 2 * t + (e & 1)) * C::BN + 32 * rw + 16 * m + g + 8 * (e >> 1)] = y[m][i][e];
    __syncthreads();
    constexpr int kOut = C::TT * C::BN, kAll = 8 * NT * C::BN;
    auto put = [&](int i, float v) {
        const long long tok = tok0 + i / C::BN;
        const int n = n0 + i % C::BN;
        if (tok < p.T && n < p.N) static_cast<typename OUT::T *>(p.y)[tok * p.N + n] = OUT::from_f(v);
    };
    for (int i = tid; i < kOut; i += kMvThreads) {
        // the parts of a float32 x from the smallest one up; where x has an infinity or NaN, the first part says all
        float v = 0.f, first = 0.f;
#pragma unroll
        for (int q = kParts - 1; q >= 0; --q)
#pragma unroll
            for (int w = 0; w < C::KW; ++w) {
                const float part = s_y[w * kAll + q * kOut + i];
                v += part;
                if (q == 0) first += part;
            }
        if (kParts > 1 && !(fabsf(first) < __int_as_float(0x7F800000))) v = first;
        if (ks == 1) put(i, v);
        else s_y[i] = v;
    }
    if (ks == 1) return;
    cluster_sync();
    // this CTA's share of the outputs, over the CTAs of the cluster
    const int o1 = kOut * (z + 1) / ks;
    for (int i = kOut * z / ks + tid; i < o1; i += kMvThreads) {
        float v = 0.f;
        for (int r = 0; r < ks; ++r) v += ld_dsmem_f32(mapa(smem_u32(s_y + i), uint32_t(r)));
        put(i, v);
    }
    cluster_sync();   // nobody leaves while its sums are read
}

template <class IO, class OUT, bool G32, int RW, int NT>
cudaError_t launch_cfg(const MatvecArgs &a, cudaStream_t s) {
    using C = MvCfg<IO, RW, NT>;
    auto *kern = k_w4_matvec<IO, OUT, G32, RW, NT>;
    const long long tiles = (long long)((a.N + C::BN - 1) / C::BN) * ((a.T + C::TT - 1) / C::TT);
    const int stages = (a.K + C::KC - 1) / C::KC;
    // Split K until there are CTAs for the whole GPU, but leave each at least two stages.
    int ks = 1;
    while (ks < 8 && tiles * ks < num_sms() && stages >= 4 * ks) ks *= 2;
    if (C::kSmem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned((a.N + C::BN - 1) / C::BN), unsigned((a.T + C::TT - 1) / C::TT), unsigned(ks));
    cfg.blockDim = dim3(kMvThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 1;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = unsigned(ks);
    cfg.attrs = at;
    cfg.numAttrs = ks > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, a, ks);
}

template <class IO, class OUT, bool G32>
cudaError_t launch_nt(const MatvecArgs &a, cudaStream_t s) {
    if constexpr (sizeof(typename IO::T) == 4) {
        if (a.T <= 2) return launch_cfg<IO, OUT, G32, 1, 1>(a, s);
        if (a.T <= 5) return launch_cfg<IO, OUT, G32, 1, 2>(a, s);
        return launch_cfg<IO, OUT, G32, 2, 3>(a, s);
    } else {
        if (a.T <= 8) return launch_cfg<IO, OUT, G32, 1, 1>(a, s);
        if (a.T <= 16) return launch_cfg<IO, OUT, G32, 2, 2>(a, s);
        return launch_cfg<IO, OUT, G32, 4, 3>(a, s);
    }
}

template <class IO, class OUT>
cudaError_t launch_group(const MatvecArgs &a, cudaStream_t s) {
    return a.group % 64 == 0 ? launch_nt<IO, OUT, false>(a, s) : launch_nt<IO, OUT, true>(a, s);
}

template <class IO>
cudaError_t launch_out(const MatvecArgs &a, int out_dtype, cudaStream_t s) {
    if (out_dtype == 0) return launch_group<IO, F32>(a, s);
    if (out_dtype == 1) return launch_group<IO, BF16>(a, s);
    return launch_group<IO, F16>(a, s);
}

}  // namespace

cudaError_t launch_w4_matvec(const void *x, long long ldx, const uint8_t *codes_w, const float *scales_w, void *y,
                             long long T, int N, int K, int group, int dtype, int out_dtype, cudaStream_t s) {
    const MatvecArgs a{x, ldx, codes_w, scales_w, y, T, N, K, group};
    const cudaError_t e = dtype == 0 ? launch_out<F32>(a, out_dtype, s) : launch_out<BF16>(a, out_dtype, s);
    if (e == cudaSuccess) count_launch(1);
    return e;
}

}  // namespace rsq
