// w4_gemv.cu -- Y = GELU(X W^T + bias) + R for a few tokens and a weight held in 4 bits with a scale
// per group of inputs (the decode form of a projection).
//
// w_nk = (q_nk - z) s with one z and s per `group` consecutive k.  Reading the weight bounds the time
// while the tokens are few: N K / 2 bytes and 2 N K / group of scales.  Each warp multiplies 16 weight
// rows (the 16-row operand of mma.sync m16n8k16) with 8 NT tokens.  q - z is an integer in -15..15 and
// exact in fp16 and bf16, so the tensor cores' products are exact; the sums of one group are
// multiplied by the scale in fp32 when the group ends.  Nothing but Y is rounded.
//
// Layout: no repacking.  The order of k within a matrix instruction is free as long as both operands
// agree, so lane 4 g + t takes consecutive k of its rows: one 128-k chunk gives it four 32-bit words of
// row g and of row g + 8 (eight k each), from one 16-byte, two 8-byte or four 4-byte pieces for groups
// of 128, 64 and 32, such that the four lanes of a row always work on the same group.
//
// A CTA of eight computing warps covers 16 WR rows and 128 WK inputs per stage (WR WK = 8): few tokens
// put the warps along K, which keeps the row tiles small and the grid large; many put them along N,
// which keeps the number of times that X is read from L2 down.  One producing thread fills a ring of
// stages by TMA (weights [WK][16 WR][64 B] and X [2 WK][M][64 elements, 128-byte swizzle], two copies
// per stage).  Where the row tiles alone leave SMs idle, a cluster splits K and sums through
// distributed shared memory in rank order.
#include <cudaTypedefs.h>

#include "fc_internal.cuh"
#include "fc_mma.cuh"
#include "fc_ptx.cuh"
#include "fc_tc.cuh"
#include "gemm_epi.cuh"

namespace fc {
namespace {

constexpr int kW4Warps = 8;
constexpr int kW4Threads = 32 * (kW4Warps + 1);   // warp 8 produces
constexpr int kW4MaxStages = 8;
constexpr int kAhead = 4;                         // stages that scales are loaded ahead

struct W4Args {
    int M, N, K;
    int nchunk;        // whole 128-k chunks
    int split;         // CTAs of a cluster along K
    int stages;
    uint32_t x_off;    // offset of X within a stage
    uint32_t stage_bytes;
    uint32_t off_bar, off_red;
    int gelu;
    const void *x, *wq, *s, *z, *bias, *R;
    void* y;
    int* flag;
};

template <typename T> struct Nib;   // 2^e + q pairs and their exact difference with 2^e + z
template <> struct Nib<__half> {
    static constexpr uint32_t MAGIC = 0x64006400u;   // 1024
    __device__ __forceinline__ static uint32_t sub(uint32_t v, uint32_t b) {
        __half2 r = __hsub2(*reinterpret_cast<__half2*>(&v), *reinterpret_cast<__half2*>(&b));
        return *reinterpret_cast<uint32_t*>(&r);
    }
};
template <> struct Nib<__nv_bfloat16> {
    static constexpr uint32_t MAGIC = 0x43004300u;   // 128
    __device__ __forceinline__ static uint32_t sub(uint32_t v, uint32_t b) {
        __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&v), *reinterpret_cast<__nv_bfloat162*>(&b));
        return *reinterpret_cast<uint32_t*>(&r);
    }
};

// The eight weights of a word as four pairs (k, k + 1), minus the zero point.
template <typename T>
__device__ __forceinline__ void unpack_word(uint32_t w, uint32_t zb, uint32_t (&p)[4]) {
    const uint32_t h = w >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t v = (__byte_perm(w, h, (i << 0) | (i << 4) | ((4 + i) << 8) | ((4 + i) << 12)) & 0x000F000Fu) | Nib<T>::MAGIC;
        p[i] = Nib<T>::sub(v, zb);
    }
}

template <typename T, int G, int NT>
__global__ void __launch_bounds__(kW4Threads) w4_gemv_kernel(const __grid_constant__ CUtensorMap mW,
                                                             const __grid_constant__ CUtensorMap mX,
                                                             const __grid_constant__ W4Args a) {
    constexpr int WR = NT, WK = kW4Warps / NT;
    constexpr int ROWS = 16 * WR, COLS = 8 * NT;
    constexpr int WPG = G / 32;         // words of a lane per group
    constexpr int NG = 4 / WPG;         // groups per 128-k chunk
    pdl_trigger();
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - smem_addr(smem_raw));
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = a.split > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int n0 = static_cast<int>(blockIdx.x) / a.split * ROWS;
    const int nblk = (a.nchunk + WK - 1) / WK;                       // stages' worth of K
    const int iters = rank < nblk ? (nblk - rank + a.split - 1) / a.split : 0;
    auto full = [&](int s) { return base + a.off_bar + 8u * s; };
    auto empty = [&](int s) { return base + a.off_bar + 8u * (kW4MaxStages + s); };
    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), kW4Warps);
        }
        fence_mbar_init();
    }
    __syncthreads();

    float acc[NT][4] = {};
    if (warp == kW4Warps) {
        if (lane == 0) {
            if (iters > 0) {
                prefetch_map(&mW);
                prefetch_map(&mX);
            }
            pdl_wait();
            const uint32_t bytes = WK * ROWS * 64u + 2u * WK * a.M * 128u;
            int it = 0, s = 0;
            uint32_t phase = 0;      // completions of the current stage's barriers so far, mod 2
            for (; it < iters; ++it) {
                if (it >= a.stages && !mbar_wait_bounded(empty(s), phase ^ 1u, a.flag)) break;
                const int kb = (it * a.split + rank) * WK;           // first chunk of the stage
                mbar_arrive_expect_tx(full(s), bytes);
                tma_load_3d(base + s * a.stage_bytes, &mW, 0, n0, kb, full(s));
                tma_load_3d(base + s * a.stage_bytes + a.x_off, &mX, 0, 0, 2 * kb, full(s));
                if (++s == a.stages) {
                    s = 0;
                    phase ^= 1u;
                }
            }
            if (it < iters)   // copies in flight land before the shared memory goes away
                for (int j = it - a.stages < 0 ? 0 : it - a.stages; j < it; ++j)
                    (void)mbar_wait_drain(full(j % a.stages), (j / a.stages) & 1);
        }
        __syncwarp();
    } else {
        pdl_wait();
        const int wr = warp % WR, wk = warp / WR;
        const int g = lane / 4, t = lane % 4;
        const int KG = a.K / G;
        const int nlo = n0 + 16 * wr + g, nhi = nlo + 8;
        // lane t of a row loads group t % NG of a chunk, the four lanes share by shuffles; kAhead stages
        // ahead of their use, each as one word of two scales and one of two zero points (rows g, g + 8)
        uint32_t sc_ring[kAhead], zp_ring[kAhead];
        const uint16_t* sc_lo = static_cast<const uint16_t*>(a.s) + static_cast<int64_t>(nlo < a.N ? nlo : 0) * KG;
        const uint16_t* sc_hi = static_cast<const uint16_t*>(a.s) + static_cast<int64_t>(nhi < a.N ? nhi : 0) * KG;
        const uint8_t* zp_lo = static_cast<const uint8_t*>(a.z) + static_cast<int64_t>(nlo < a.N ? nlo : 0) * KG;
        const uint8_t* zp_hi = static_cast<const uint8_t*>(a.z) + static_cast<int64_t>(nhi < a.N ? nhi : 0) * KG;
        auto load_scales = [&](int chunk, uint32_t& sc, uint32_t& zp) {
            const int gi = chunk * NG + t % NG;
            sc = 0u;
            zp = 0x00080008u;
            if (gi < KG) {   // past the last chunk: scale zero
                sc = __ldg(sc_lo + gi) | static_cast<uint32_t>(__ldg(sc_hi + gi)) << 16;
                if (a.z) zp = (__ldg(zp_lo + gi) & 15u) | (__ldg(zp_hi + gi) & 15u) << 16;
            }
        };
        // one group: WPG words of each row against the matching X pieces
        auto group = [&](int gi, const uint32_t* wl, const uint32_t* wh, auto&& xpiece, uint32_t sc, uint32_t zp) {
            float part[NT][4] = {};
            const uint32_t bl = Nib<T>::MAGIC | __byte_perm(zp, 0u, 0x1010), bh = Nib<T>::MAGIC | __byte_perm(zp, 0u, 0x3232);
            const float2 s2 = unpack2<T>(sc);
            const float sl = s2.x, sh = s2.y;
#pragma unroll
            for (int w = 0; w < WPG; ++w) {
                uint32_t pl[4], ph[4];
                unpack_word<T>(wl[w], bl, pl);
                unpack_word<T>(wh[w], bh, ph);
                const uint32_t a0[4] = {pl[0], ph[0], pl[1], ph[1]}, a1[4] = {pl[2], ph[2], pl[3], ph[3]};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint4 xv = xpiece(nt, gi, w);
                    mma16816<T>(part[nt], a0, xv.x, xv.y);
                    mma16816<T>(part[nt], a1, xv.z, xv.w);
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                acc[nt][0] += sl * part[nt][0];
                acc[nt][1] += sl * part[nt][1];
                acc[nt][2] += sh * part[nt][2];
                acc[nt][3] += sh * part[nt][3];
            }
        };
        // k of word w of group gi within the chunk
        auto kof = [&](int gi, int w) { return gi * G + t * (G / 4) + 8 * w; };
        bool ok = true;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) load_scales((i * a.split + rank) * WK + wk, sc_ring[i], zp_ring[i]);
        int s = 0;
        uint32_t phase = 0;
        for (int it0 = 0; ok && it0 < iters; it0 += kAhead)
#pragma unroll
          for (int i = 0; i < kAhead; ++i) {
            const int it = it0 + i;
            if (it >= iters || !ok) break;
            const uint32_t sc = sc_ring[i], zp = zp_ring[i];
            load_scales(((it + kAhead) * a.split + rank) * WK + wk, sc_ring[i], zp_ring[i]);
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(full(s), phase, a.flag))) {
                ok = false;
                break;
            }
            const uint32_t wbase = base + s * a.stage_bytes + static_cast<uint32_t>((wk * ROWS + 16 * wr + g) * 64);
            const uint32_t xbase = base + s * a.stage_bytes + a.x_off;
            auto xpiece = [&](int nt, int gi, int w) {
                const int k8 = kof(gi, w) / 8;                         // 16-byte piece of the chunk, 0..15
                const int m = min(8 * nt + g, a.M - 1);                // columns past M are never stored
                const uint32_t row = static_cast<uint32_t>((2 * wk + k8 / 8) * a.M + m);
                return lds128(xbase + row * 128u + ((static_cast<uint32_t>(k8 & 7) ^ (row & 7u)) << 4));
            };
#pragma unroll
            for (int gi = 0; gi < NG; ++gi) {
                uint32_t wl[WPG], wh[WPG];
                const uint32_t at = wbase + static_cast<uint32_t>(kof(gi, 0) / 2);
                if constexpr (WPG == 4) {
                    const uint4 l = lds128(at), h = lds128(at + 512u);
                    wl[0] = l.x; wl[1] = l.y; wl[2] = l.z; wl[3] = l.w;
                    wh[0] = h.x; wh[1] = h.y; wh[2] = h.z; wh[3] = h.w;
                } else if constexpr (WPG == 2) {
                    const uint2 l = lds64(at), h = lds64(at + 512u);
                    wl[0] = l.x; wl[1] = l.y;
                    wh[0] = h.x; wh[1] = h.y;
                } else {
                    wl[0] = lds32(at);
                    wh[0] = lds32(at + 512u);
                }
                const int src = (lane & 28) | gi;
                group(gi, wl, wh, xpiece, __shfl_sync(0xffffffffu, sc, src), __shfl_sync(0xffffffffu, zp, src));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty(s));
            if (++s == a.stages) {
                s = 0;
                phase ^= 1u;
            }
        }
        // the last K % 128 inputs (groups of 32 and 64), from global memory by the first K warps
        if (G < 128 && ok && rank == 0 && wk == 0 && a.nchunk * 128 < a.K) {
            const int k0 = a.nchunk * 128;
            uint32_t sc, zp;
            load_scales(a.nchunk, sc, zp);
            const T* x = static_cast<const T*>(a.x);
            const uint8_t* wq = static_cast<const uint8_t*>(a.wq);
            const int ng = (a.K - k0) / G;
            for (int gi = 0; gi < ng; ++gi) {
                uint32_t wl[WPG], wh[WPG];
#pragma unroll
                for (int w = 0; w < WPG; ++w) {
                    const int64_t at = (k0 + kof(gi, w)) / 2;
                    wl[w] = nlo < a.N ? *reinterpret_cast<const uint32_t*>(wq + static_cast<int64_t>(nlo) * (a.K / 2) + at) : 0u;
                    wh[w] = nhi < a.N ? *reinterpret_cast<const uint32_t*>(wq + static_cast<int64_t>(nhi) * (a.K / 2) + at) : 0u;
                }
                auto xpiece = [&](int nt, int gj, int w) {
                    const int m = min(8 * nt + g, a.M - 1);
                    return *reinterpret_cast<const uint4*>(x + static_cast<int64_t>(m) * a.K + k0 + kof(gj, w));
                };
                const int src = (lane & 28) | gi;
                group(gi, wl, wh, xpiece, __shfl_sync(0xffffffffu, sc, src), __shfl_sync(0xffffffffu, zp, src));
            }
        }
    }

    // sum over the K warps, then over the cluster, in fixed order; then the epilogue
    float* red = reinterpret_cast<float*>(gbase + a.off_red);   // [WK][COLS][ROWS + 4]
    constexpr int PITCH = ROWS + 4;
    __syncthreads();
    if (warp < kW4Warps) {
        const int wr = warp % WR, wk = warp / WR, g = lane / 4, t = lane % 4;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                red[(wk * COLS + 8 * nt + 2 * t + (e & 1)) * PITCH + 16 * wr + g + 8 * (e >> 1)] = acc[nt][e];
    }
    __syncthreads();
    const int per = ROWS * a.M;
    if (a.split > 1) {
        for (int i = threadIdx.x; i < per; i += kW4Threads) {
            const int m = i / ROWS, r = i % ROWS;
            float v = red[m * PITCH + r];
#pragma unroll
            for (int k = 1; k < WK; ++k) v += red[(k * COLS + m) * PITCH + r];
            red[m * PITCH + r] = v;
        }
        __syncwarp();
        cluster_sync();
    }
    const T* bias = static_cast<const T*>(a.bias);
    const T* R = static_cast<const T*>(a.R);
    for (int i = rank * kW4Threads + threadIdx.x; i < per; i += a.split * kW4Threads) {
        const int m = i / ROWS, r = i % ROWS, n = n0 + r;
        if (n >= a.N) continue;
        float v = 0.0f;
        if (a.split > 1) {
            const uint32_t at = smem_addr(red + m * PITCH + r);
            for (int c = 0; c < a.split; ++c) {
                float p;
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(p) : "r"(mapa_shared(at, c)) : "memory");
                v += p;
            }
        } else {
#pragma unroll
            for (int k = 0; k < WK; ++k) v += red[(k * COLS + m) * PITCH + r];
        }
        if (bias) v += to_f32(bias[n]);
        if (a.gelu) v = gelu_erf(v);
        const int64_t at = static_cast<int64_t>(m) * a.N + n;
        if (R) v += to_f32(R[at]);
        static_cast<T*>(a.y)[at] = from_f32<T>(v);
    }
    __syncwarp();
    if (a.split > 1) cluster_sync();   // the sums stay in place until every CTA has read them
}

template <typename T, int G, int NT>
int launch_w4(W4Args a, cudaStream_t st) {
    constexpr int WR = NT, WK = kW4Warps / NT, ROWS = 16 * WR;
    CUtensorMap mW{}, mX{};
    a.nchunk = a.K / 128;
    // a map needs a chunk to describe; without one (K < 128) no stage is loaded
    if (a.nchunk > 0) {
        const int64_t wd[3] = {64, a.N, a.nchunk}, ws[2] = {a.K / 2, 64};
        const int wb[3] = {64, ROWS, WK};
        const int64_t xd[3] = {64, a.M, 2 * static_cast<int64_t>(a.nchunk)}, xs[2] = {static_cast<int64_t>(a.K) * 2, 128};
        const int xb[3] = {64, a.M, 2 * WK};
        if (!make_map_3d(&mW, a.wq, kMapU8, wd, ws, wb, false) || !make_map_3d(&mX, a.x, kMap16, xd, xs, xb, true)) return FUSE_ECUDA;
    }
    a.x_off = WK * ROWS * 64;
    a.stage_bytes = static_cast<uint32_t>((a.x_off + 2 * WK * a.M * 128 + 1023) / 1024 * 1024);
    const uint32_t red = static_cast<uint32_t>(WK * 8 * NT * (ROWS + 4) * 4);
    const int row_tiles = static_cast<int>(ceil_div(a.N, ROWS));
    const int nblk = static_cast<int>(ceil_div(a.nchunk, WK));
    a.split = 1;
    while (a.split < 8 && row_tiles * a.split * 2 <= 2 * sm_count() && nblk >= 4 * a.split) a.split *= 2;
    const int iters = static_cast<int>(ceil_div(nblk > 0 ? nblk : 1, a.split));
    a.stages = iters < kW4MaxStages ? iters : kW4MaxStages;
    while (a.stages > 1 && a.stages * a.stage_bytes + red > 110 * 1024) --a.stages;
    a.off_red = a.stages * a.stage_bytes;
    a.off_bar = a.off_red + (red + 15) / 16 * 16;
    const uint32_t smem = a.off_bar + 16 * kW4MaxStages + 1024;
    const int rc = opt_in_smem((const void*)w4_gemv_kernel<T, G, NT>, 116 * 1024, true);
    if (rc != FUSE_OK) return rc;
    return launch_pdl(w4_gemv_kernel<T, G, NT>, dim3(static_cast<unsigned>(row_tiles * a.split)), dim3(kW4Threads), smem, st, a.split, mW, mX, a);
}

template <typename T, int G>
int run_w4_g(const W4Args& a, cudaStream_t st) {
    if (a.M <= 8) return launch_w4<T, G, 1>(a, st);
    if (a.M <= 16) return launch_w4<T, G, 2>(a, st);
    if (a.M <= 32) return launch_w4<T, G, 4>(a, st);
    return launch_w4<T, G, 8>(a, st);
}
template <typename T>
int run_w4(const W4Args& a, int group, cudaStream_t st) {
    if (group == 32) return run_w4_g<T, 32>(a, st);
    if (group == 64) return run_w4_g<T, 64>(a, st);
    return run_w4_g<T, 128>(a, st);
}

struct W4Entry {
    const void* kernel;
    const char* name;
};
template <typename T, int G>
void w4_entries(W4Entry* e, const char* const* names) {
    e[0] = {(const void*)w4_gemv_kernel<T, G, 1>, names[0]};
    e[1] = {(const void*)w4_gemv_kernel<T, G, 2>, names[1]};
    e[2] = {(const void*)w4_gemv_kernel<T, G, 4>, names[2]};
    e[3] = {(const void*)w4_gemv_kernel<T, G, 8>, names[3]};
}

}  // namespace

int w4_report_count() { return 24; }
int w4_report(int i, fuse_kernel_record* out) {
    if (i < 0 || i >= 24) return FUSE_EINVAL;
    static const char* const names[24] = {
        "w4_gemv_kernel<bf16, group 32, M <= 8>", "w4_gemv_kernel<bf16, group 32, M <= 16>", "w4_gemv_kernel<bf16, group 32, M <= 32>", "w4_gemv_kernel<bf16, group 32, M <= 64>",
        "w4_gemv_kernel<bf16, group 64, M <= 8>", "w4_gemv_kernel<bf16, group 64, M <= 16>", "w4_gemv_kernel<bf16, group 64, M <= 32>", "w4_gemv_kernel<bf16, group 64, M <= 64>",
        "w4_gemv_kernel<bf16, group 128, M <= 8>", "w4_gemv_kernel<bf16, group 128, M <= 16>", "w4_gemv_kernel<bf16, group 128, M <= 32>", "w4_gemv_kernel<bf16, group 128, M <= 64>",
        "w4_gemv_kernel<f16, group 32, M <= 8>", "w4_gemv_kernel<f16, group 32, M <= 16>", "w4_gemv_kernel<f16, group 32, M <= 32>", "w4_gemv_kernel<f16, group 32, M <= 64>",
        "w4_gemv_kernel<f16, group 64, M <= 8>", "w4_gemv_kernel<f16, group 64, M <= 16>", "w4_gemv_kernel<f16, group 64, M <= 32>", "w4_gemv_kernel<f16, group 64, M <= 64>",
        "w4_gemv_kernel<f16, group 128, M <= 8>", "w4_gemv_kernel<f16, group 128, M <= 16>", "w4_gemv_kernel<f16, group 128, M <= 32>", "w4_gemv_kernel<f16, group 128, M <= 64>"};
    W4Entry e[24];
    w4_entries<__nv_bfloat16, 32>(e, names);
    w4_entries<__nv_bfloat16, 64>(e + 4, names + 4);
    w4_entries<__nv_bfloat16, 128>(e + 8, names + 8);
    w4_entries<__half, 32>(e + 12, names + 12);
    w4_entries<__half, 64>(e + 16, names + 16);
    w4_entries<__half, 128>(e + 20, names + 20);
    return describe_kernel(e[i].kernel, e[i].name, kW4Threads, 110 * 1024, out);
}

}  // namespace fc

extern "C" int fuse_w4_gemv(const void* x, const void* wq, const void* scales, const void* zeros, const void* bias,
                            const void* R, void* y, int64_t M, int64_t N, int64_t K, int64_t group, int gelu,
                            int dtype, fuse_stream_t stream) {
    using namespace fc;
    if (M < 0 || N < 1 || K < 1 || (gelu != 0 && gelu != 1)) return FUSE_EINVAL;
    if (dtype != FUSE_F16 && dtype != FUSE_BF16) return FUSE_EINVAL;
    if (group != 32 && group != 64 && group != 128) return FUSE_EUNSUPPORTED;
    if (M > 64 || N > 0x7fffff00LL || K > 0x7fffff00LL || K % group != 0) return FUSE_EUNSUPPORTED;
    if (M == 0) return FUSE_OK;
    if (!x || !wq || !scales || !y) return FUSE_EINVAL;
    if (!is_aligned(x, 16) || !is_aligned(wq, 16) || !is_aligned(scales, 2) || !is_aligned(bias, 2) ||
        !is_aligned(R, 2) || !is_aligned(y, 2))
        return FUSE_EALIGN;
    const int64_t yb = M * N * 2;
    if (ranges_overlap(y, yb, x, M * K * 2) || ranges_overlap(y, yb, wq, N * (K / 2)) ||
        ranges_overlap(y, yb, scales, N * (K / group) * 2) || (zeros && ranges_overlap(y, yb, zeros, N * (K / group))) ||
        (bias && ranges_overlap(y, yb, bias, N * 2)) || (R && ranges_overlap(y, yb, R, yb)))
        return FUSE_EINVAL;
    W4Args a{};
    a.M = static_cast<int>(M);
    a.N = static_cast<int>(N);
    a.K = static_cast<int>(K);
    a.gelu = gelu;
    a.x = x;
    a.wq = wq;
    a.s = scales;
    a.z = zeros;
    a.bias = bias;
    a.R = R;
    a.y = y;
    a.flag = watchdog_flag();
    if (!a.flag) return FUSE_ECUDA;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return dtype == FUSE_F16 ? run_w4<__half>(a, static_cast<int>(group), st) : run_w4<__nv_bfloat16>(a, static_cast<int>(group), st);
}

extern "C" int64_t fuse_w4_gemv_bytes(int64_t M, int64_t N, int64_t K, int64_t group, int zeros, int bias,
                                      int residual) {
    if (M < 0 || N < 1 || K < 1 || group < 1 || K % group != 0 || K % 2 != 0) return FUSE_EINVAL;
    return N * (K / 2) + N * (K / group) * (zeros ? 3 : 2) + 2 * M * K + 2 * M * N + (bias ? 2 * N : 0) + (residual ? 2 * M * N : 0);
}
