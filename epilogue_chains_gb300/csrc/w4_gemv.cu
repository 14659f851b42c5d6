// w4_gemv.cu -- Y = GELU(X W^T + bias) + R for a few tokens and a weight held in 4 bits with a scale
// per group of inputs (the decode form of a projection).
//
// w_nk = (q_nk - z) s with one z and s per `group` consecutive k.  Reading the weight bounds the time
// while the tokens are few: N K / 2 bytes and 2 N K / group of scales.  q - z is an integer in -15..15 and
// exact in fp16 and bf16, so the tensor cores' products are exact; the sums of one group are multiplied
// by the scale in fp32 when the group ends.  Nothing but Y is rounded.  The weights are used as they are
// stored, without repacking.  Two kernels:
//
// w4_gemv_kernel, for few tokens.  Each warp multiplies 16 weight rows (the 16-row operand of mma.sync
// m16n8k16) with 8 tokens; more (where w4_tile_kernel cannot take them) are blocks of 8, the grid's
// second axis, and later blocks find the weights in L2.  The order of k within a matrix instruction is
// free as long as both operands agree, so lane 4 g + t takes consecutive k of its rows: one 128-k chunk
// gives it four 32-bit words of row g and of row g + 8 (eight k each), from one 16-byte, two 8-byte or
// four 4-byte pieces for groups of 128, 64 and 32, such that the four lanes of a row always work on the
// same group.  A warp takes two such chunks at a time: a row's 128 bytes, one request of the copy
// engine.
// A CTA of eight computing warps covers 16 rows and 2048 inputs per stage.  One producing thread fills a
// ring of stages by TMA (weights [8][16][128 B] and X [32][tokens][64 elements], 128-byte swizzle, scales
// and zero points); a CTA stays for several row tiles, so that the ring runs on while a tile is finished.
// Where the row tiles alone leave SMs idle, a cluster splits K and sums through distributed shared memory
// in rank order.  Scales that the copy engine cannot fetch (a row's are not whole 16-byte pieces) are
// loaded a block of stages ahead by the lanes instead: under load such a read takes microseconds, so the
// ring is used wherever it can be (5 x 4096 x 14336, groups of 32 with zero points: 18.9 -> 15.0 us).
// Two CTAs per SM with a ring of 112 KB each: three with 73 KB took 14.0 us where two take 12.9 (5 x 4096 x
// 14336) and 19.8 where two take 18.4 (1 x 28672 x 4096, 3.3 TB/s).  What bounds the large sizes is the
// work per weight between the ring and the tensor core (about 13 instructions per 8 weights to unpack);
// the same copies without any arithmetic take 12.4 us for 1 x 28672 x 4096.
//
// w4_tile_kernel, for more tokens: see below.
#include <cudaTypedefs.h>

#include <atomic>
#include <type_traits>

#include "fc_internal.cuh"
#include "fc_mma.cuh"
#include "fc_ptx.cuh"
#include "fc_tc.cuh"
#include "gemm_epi.cuh"

namespace fc {
namespace {

constexpr int kW4Warps = 8;
constexpr int kW4Threads = 32 * (kW4Warps + 1);   // warp 8 produces
constexpr int kW4Rows = 16, kW4Cols = 8;          // weight rows and tokens of a tile: one matrix instruction's
constexpr int kW4MaxStages = 8;
constexpr int kW4Smem = 200 * 1024;               // most dynamic shared memory of a CTA

struct W4Args {
    int M, N, K;
    int mbox;          // tokens of a tile in shared memory
    int nchunk;        // whole 256-k chunks
    int split;         // CTAs of a cluster along K
    int tiles;         // row tiles
    int stages;
    int x_resident;    // X is loaded once per CTA, not with every stage
    uint32_t x_off;    // offset of X within a stage, or of the resident X
    uint32_t s_off;    // of the scales within a stage
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
        uint32_t v = __byte_perm(w, h, (i << 0) | (i << 4) | ((4 + i) << 8) | ((4 + i) << 12));
        asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(v), "r"(0x000F000Fu), "r"(Nib<T>::MAGIC));   // (v & mask) | magic
        p[i] = Nib<T>::sub(v, zb);
    }
}

// Synchronize the computing warps (the loading warp goes on).
__device__ __forceinline__ void sync_compute() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kW4Warps) : "memory"); }

template <typename T, int G, bool TS>
__global__ void __launch_bounds__(kW4Threads, 2) w4_gemv_kernel(
    const __grid_constant__ CUtensorMap mW, const __grid_constant__ CUtensorMap mX, const __grid_constant__ CUtensorMap mS,
    const __grid_constant__ CUtensorMap mZ, const __grid_constant__ W4Args a) {
    constexpr int WK = kW4Warps, ROWS = kW4Rows, COLS = kW4Cols, PITCH = ROWS + 4;
    constexpr int WPG = G / 32;         // words of a lane per group
    constexpr int NG = 8 / WPG;         // groups per 256-k chunk
    constexpr int RED = WK * COLS * PITCH;      // floats of one buffer of partial sums
    constexpr uint32_t SROW = WK * NG * 2;      // bytes of a row's scales in a stage; half as many of zero points
    pdl_trigger();
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - smem_addr(smem_raw));
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = a.split > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int nblk = (a.nchunk + WK - 1) / WK;                       // stages' worth of K
    const int iters = rank < nblk ? (nblk - rank + a.split - 1) / a.split : 0;
    const int m0 = COLS * static_cast<int>(blockIdx.y), mrows = min(COLS, a.M - m0);      // this CTA's tokens
    // row tiles of this CTA: a split has one, else every gridDim.x-th
    const int tile0 = static_cast<int>(blockIdx.x) / a.split, tile_step = a.split > 1 ? a.tiles : static_cast<int>(gridDim.x);
    auto full = [&](int s) { return base + a.off_bar + 8u * s; };
    auto empty = [&](int s) { return base + a.off_bar + 8u * (kW4MaxStages + s); };
    const uint32_t x_full = base + a.off_bar + 8u * (2 * kW4MaxStages);
    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), kW4Warps);
        }
        mbar_init(x_full, 1);
        fence_mbar_init();
    }
    __syncthreads();

    if (warp == kW4Warps) {
        if (lane == 0) {
            if (iters > 0) {
                prefetch_map(&mW);
                prefetch_map(&mX);
                if (TS) prefetch_map(&mS);
                if (TS && a.z) prefetch_map(&mZ);
            }
            pdl_wait();
            const uint32_t x_bytes = 4u * WK * a.mbox * 128u;
            const uint32_t bytes = WK * ROWS * 128u + (a.x_resident ? 0u : x_bytes) + (TS ? ROWS * SROW : 0u) + (TS && a.z ? ROWS * SROW / 2 : 0u);
            int s = 0, loads = 0;
            uint32_t phase = 0;      // completions of the current stage's barriers so far, mod 2
            bool ok = true;
            const bool x_once = a.x_resident && iters > 0;
            if (x_once) {
                mbar_arrive_expect_tx(x_full, x_bytes * iters);
                for (int it = 0; it < iters; ++it)
                    tma_load_3d(base + a.x_off + it * x_bytes, &mX, 0, m0, 4 * (it * a.split + rank) * WK, x_full);
            }
            for (int tile = tile0; ok && tile < a.tiles; tile += tile_step) {
                for (int it = 0; it < iters; ++it) {
                    if (loads >= a.stages && !mbar_wait_bounded(empty(s), phase ^ 1u, a.flag)) {
                        ok = false;
                        break;
                    }
                    const int kb = (it * a.split + rank) * WK;           // first chunk of the stage
                    mbar_arrive_expect_tx(full(s), bytes);
                    tma_load_3d(base + s * a.stage_bytes, &mW, 0, tile * ROWS, kb, full(s));
                    if (!a.x_resident) tma_load_3d(base + s * a.stage_bytes + a.x_off, &mX, 0, m0, 4 * kb, full(s));
                    if (TS) tma_load_3d(base + s * a.stage_bytes + a.s_off, &mS, kb * NG, tile * ROWS, 0, full(s));
                    if (TS && a.z) tma_load_3d(base + s * a.stage_bytes + a.s_off + ROWS * SROW, &mZ, kb * NG, tile * ROWS, 0, full(s));
                    ++loads;
                    if (++s == a.stages) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) {   // copies in flight land before the shared memory goes away
                for (int j = max(0, loads - a.stages); j < loads; ++j) (void)mbar_wait_drain(full(j % a.stages), (j / a.stages) & 1);
                if (x_once) (void)mbar_wait_drain(x_full, 0);
            }
        }
        __syncwarp();
        if (a.split == 1) return;
    }

    float acc[4];
    const int wk = warp;
    const int g = lane / 4, t = lane % 4;
    const T* bias = static_cast<const T*>(a.bias);
    const T* R = static_cast<const T*>(a.R);
    float* red = reinterpret_cast<float*>(gbase + a.off_red);   // [2][WK][COLS][PITCH]
    auto write_red = [&](float* buf) {
#pragma unroll
        for (int e = 0; e < 4; ++e) buf[(wk * COLS + 2 * t + (e & 1)) * PITCH + g + 8 * (e >> 1)] = acc[e];
    };
    auto finish = [&](float v, int m, int n) {
        if (bias) v += to_f32(bias[n]);
        if (a.gelu) v = gelu_erf(v);
        const int64_t at = static_cast<int64_t>(m0 + m) * a.N + n;
        if (R) v += to_f32(R[at]);
        static_cast<T*>(a.y)[at] = from_f32<T>(v);
    };
    if (warp < kW4Warps) {
        pdl_wait();
        const int KG = a.K / G;
        // Scales and zero points: the four lanes of a row load one group each (two for groups of 32) and share by
        // shuffles; one word of two scales and one of two zero points (rows g, g + 8) per lane and group, a block
        // of stages ahead of its use (across row tiles).
        constexpr int SB = TS ? 1 : NG < 4 ? 4 / NG : 1;    // stages of a block
        constexpr int SW = NG < 4 ? 1 : NG / 4;    // words of a lane per block
        const int gstep = a.split * WK * NG;       // groups from a stage to the next
        const int gfirst = (rank * WK + wk) * NG + (NG < 4 ? t / NG * gstep + t % NG : t);
        auto load_scale = [&](int tile, int gi, uint32_t& sc, uint32_t& zp) {
            sc = 0u;
            zp = 0x00080008u;
            const int nlo = tile * ROWS + g, nhi = nlo + 8;
            if (gi < KG && nlo < a.N) {   // past the last chunk or row: scale zero
                const int64_t lo = static_cast<int64_t>(nlo) * KG + gi, hi = nhi < a.N ? lo + 8 * static_cast<int64_t>(KG) : lo;
                const uint16_t* sp = static_cast<const uint16_t*>(a.s);
                sc = sp[lo] | static_cast<uint32_t>(sp[hi]) << 16;
                if (a.z) {
                    const uint8_t* zq = static_cast<const uint8_t*>(a.z);
                    zp = (zq[lo] & 15u) | (zq[hi] & 15u) << 16;
                }
            }
        };
        auto load_scales = [&](int tile, int gi, uint32_t (&sc)[SW], uint32_t (&zp)[SW]) {
#pragma unroll
            for (int i = 0; i < SW; ++i) load_scale(tile, gi + 4 * i < a.nchunk * NG ? gi + 4 * i : KG, sc[i], zp[i]);
        };
        // one group: WPG words of each row against the matching X pieces
        auto group = [&](int gi, const uint32_t* wl, const uint32_t* wh, auto&& xpiece, float2 s2, uint32_t zl, uint32_t zh) {
            float part[4] = {};
            const uint32_t bl = Nib<T>::MAGIC | zl, bh = Nib<T>::MAGIC | zh;      // a row's zero point, twice
            const float sl = s2.x, sh = s2.y;
#pragma unroll
            for (int w = 0; w < WPG; ++w) {
                uint32_t pl[4], ph[4];
                unpack_word<T>(wl[w], bl, pl);
                unpack_word<T>(wh[w], bh, ph);
                const uint32_t a0[4] = {pl[0], ph[0], pl[1], ph[1]}, a1[4] = {pl[2], ph[2], pl[3], ph[3]};
                const uint4 xv = xpiece(gi, w);
                mma16816<T>(part, a0, xv.x, xv.y);
                mma16816<T>(part, a1, xv.z, xv.w);
            }
            acc[0] += sl * part[0];
            acc[1] += sl * part[1];
            acc[2] += sh * part[2];
            acc[3] += sh * part[3];
        };
        // k of word w of group gi within the chunk
        auto kof = [&](int gi, int w) { return gi * G + t * (G / 4) + 8 * w; };
        bool ok = true;
        // Where this lane's X pieces lie within a stage, of the chunk's eight words in the order of the groups:
        // row g is column g of the product.  Rows past M are other rows or unused space: those columns are never stored.
        // Words next to each other (or, in groups of 32, groups) share a row and differ in one or two bits of
        // the piece: XP of them come from one offset by exclusive or.
        constexpr int XP = G == 128 ? 4 : 2, XBIT = G == 32 ? 6 : 4;
        uint32_t xoff[8 / XP];
#pragma unroll
        for (int i = 0; i < 8 / XP; ++i) {
            const int k8 = kof(i * XP / WPG, i * XP % WPG) / 8;       // 16-byte piece of the chunk, 0..31
            const uint32_t row = static_cast<uint32_t>((4 * wk + k8 / 8) * a.mbox + g);
            xoff[i] = a.x_off + row * 128u + ((static_cast<uint32_t>(k8 & 7) ^ (row & 7u)) << 4);
        }
        // the weights of group gi: byte gi G / 2 + t G / 8 of the row's 128, swizzled by the row (gi by exclusive or)
        const uint32_t woff = static_cast<uint32_t>((wk * ROWS + g) * 128) + (static_cast<uint32_t>(t * (G / 8)) ^ (static_cast<uint32_t>(g & 7) << 4));
        const uint32_t x_step = a.x_resident ? 4u * WK * a.mbox * 128u : 0u;
        uint32_t sc_next[SW], zp_next[SW], sc[SW] = {}, zp[SW] = {};
        if (!TS) load_scales(tile0, gfirst, sc_next, zp_next);
        // this lane's scales within a stage: row g (rows of 128 and 64 bytes swizzled), the warp's first group
        const uint32_t srow = static_cast<uint32_t>(g) * SROW + wk * (NG * 2);
        int s = 0, turn = 0;
        uint32_t phase = 0;
        if (a.x_resident && iters > 0) ok = __all_sync(0xffffffffu, mbar_wait_bounded(x_full, 0, a.flag));
        for (int tile = tile0; tile < a.tiles; tile += tile_step) {
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = 0.0f;
            uint32_t xres = 0;
            for (int it0 = 0; ok && it0 < iters; it0 += SB)
#pragma unroll
              for (int i = 0; i < SB; ++i) {
                if (it0 + i >= iters || !ok) break;
                if (!TS && i == 0) {
#pragma unroll
                    for (int j = 0; j < SW; ++j) {
                        sc[j] = sc_next[j];
                        zp[j] = zp_next[j];
                    }
                    if (it0 + SB < iters) load_scales(tile, gfirst + (it0 + SB) * gstep, sc_next, zp_next);
                    else load_scales(tile + tile_step, gfirst, sc_next, zp_next);
                }
                if (!__all_sync(0xffffffffu, mbar_wait_bounded(full(s), phase, a.flag))) {
                    ok = false;
                    break;
                }
                // plain loads: the compiler keeps them behind the wait, and free to move among the rest
                const uint32_t stage = s * a.stage_bytes;
                const uint32_t xs = a.x_resident ? xres : stage;
                xres += x_step;
                auto xpiece = [&](int gi, int w) {
                    const int i = gi * WPG + w;
                    return *reinterpret_cast<const uint4*>(gbase + ((xs + xoff[i / XP]) ^ (i % XP << XBIT)));
                };
                // (TS) scales and zero points of up to four groups, rows g and g + 8
                constexpr int NS = NG < 4 ? NG : 4;
                uint32_t sl[2], sh[2], zl = 0x08080808u, zh = 0x08080808u;
#pragma unroll
                for (int gi = 0; gi < NG; ++gi) {
                    uint32_t wl[WPG], wh[WPG];
                    if (TS && gi % NS == 0) {
                        const uint32_t soff = srow ^ (G == 32 ? (srow >> 3) & 0x70u : G == 64 ? (srow >> 3) & 0x30u : 0u);
                        const uint8_t* sp = gbase + stage + a.s_off + soff + 2 * gi;
                        const uint8_t* zq = gbase + stage + a.s_off + ROWS * SROW + srow / 2 + gi;
                        if constexpr (NG < 4) {
                            sl[0] = *reinterpret_cast<const uint32_t*>(sp);
                            sh[0] = *reinterpret_cast<const uint32_t*>(sp + 8 * SROW);
                            if (a.z) {
                                zl = *reinterpret_cast<const uint16_t*>(zq);
                                zh = *reinterpret_cast<const uint16_t*>(zq + 4 * SROW);
                            }
                        } else {
                            const uint2 l = *reinterpret_cast<const uint2*>(sp), h = *reinterpret_cast<const uint2*>(sp + 8 * SROW);
                            sl[0] = l.x; sl[1] = l.y;
                            sh[0] = h.x; sh[1] = h.y;
                            if (a.z) {
                                zl = *reinterpret_cast<const uint32_t*>(zq) & 0x0F0F0F0Fu;
                                zh = *reinterpret_cast<const uint32_t*>(zq + 4 * SROW) & 0x0F0F0F0Fu;
                            }
                        }
                        if (NG < 4 && a.z) {
                            zl &= 0x0F0Fu;
                            zh &= 0x0F0Fu;
                        }
                    }
                    const uint8_t* at = gbase + ((stage + woff) ^ (gi * (G / 2)));
                    if constexpr (WPG == 4) {
                        const uint4 l = *reinterpret_cast<const uint4*>(at), h = *reinterpret_cast<const uint4*>(at + 1024);
                        wl[0] = l.x; wl[1] = l.y; wl[2] = l.z; wl[3] = l.w;
                        wh[0] = h.x; wh[1] = h.y; wh[2] = h.z; wh[3] = h.w;
                    } else if constexpr (WPG == 2) {
                        const uint2 l = *reinterpret_cast<const uint2*>(at), h = *reinterpret_cast<const uint2*>(at + 1024);
                        wl[0] = l.x; wl[1] = l.y;
                        wh[0] = h.x; wh[1] = h.y;
                    } else {
                        wl[0] = *reinterpret_cast<const uint32_t*>(at);
                        wh[0] = *reinterpret_cast<const uint32_t*>(at + 1024);
                    }
                    if constexpr (TS) {
                        const int w = gi % NS;
                        const uint32_t pair = __byte_perm(sl[w / 2], sh[w / 2], w & 1 ? 0x7632 : 0x5410);
                        group(gi, wl, wh, xpiece, unpack2<T>(pair), __byte_perm(zl, 0u, 0x4040 | w * 0x101), __byte_perm(zh, 0u, 0x4040 | w * 0x101));
                    } else {
                        const int src = (lane & 28) | (NG < 4 ? i * NG + gi : gi % 4);
                        const uint32_t z2 = a.z ? __shfl_sync(0xffffffffu, zp[NG < 4 ? 0 : gi / 4], src) : 0x00080008u;
                        group(gi, wl, wh, xpiece, unpack2<T>(__shfl_sync(0xffffffffu, sc[NG < 4 ? 0 : gi / 4], src)), __byte_perm(z2, 0u, 0x1010),
                              __byte_perm(z2, 0u, 0x3232));
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty(s));
                if (++s == a.stages) {
                    s = 0;
                    phase ^= 1u;
                }
            }
            // the last K % 256 inputs, from global memory by the first warp (scales that come through the ring have none)
            if (!TS && ok && rank == 0 && wk == 0 && a.nchunk * 256 < a.K) {
                const int k0 = a.nchunk * 256, nlo = tile * ROWS + g, nhi = nlo + 8;
                const T* x = static_cast<const T*>(a.x);
                const uint8_t* wq = static_cast<const uint8_t*>(a.wq);
                const int ng = (a.K - k0) / G;
                for (int gi = 0; gi < ng; ++gi) {
                    uint32_t wl[WPG], wh[WPG], tsc, tzp;
                    load_scale(tile, a.nchunk * NG + gi, tsc, tzp);
#pragma unroll
                    for (int w = 0; w < WPG; ++w) {
                        const int64_t at = (k0 + kof(gi, w)) / 2;
                        wl[w] = nlo < a.N ? *reinterpret_cast<const uint32_t*>(wq + static_cast<int64_t>(nlo) * (a.K / 2) + at) : 0u;
                        wh[w] = nhi < a.N ? *reinterpret_cast<const uint32_t*>(wq + static_cast<int64_t>(nhi) * (a.K / 2) + at) : 0u;
                    }
                    auto xpiece = [&](int gj, int w) {
                        return *reinterpret_cast<const uint4*>(x + static_cast<int64_t>(m0 + min(g, mrows - 1)) * a.K + k0 + kof(gj, w));
                    };
                    group(gi, wl, wh, xpiece, unpack2<T>(tsc), __byte_perm(tzp, 0u, 0x1010), __byte_perm(tzp, 0u, 0x3232));
                }
            }
            if (a.split > 1) break;
            // Sum over the K warps in fixed order, then the epilogue.  Two buffers: a warp writes one again only
            // after all have passed the next tile's barrier, having read it.
            float* buf = red + (turn & 1) * RED;
            ++turn;
            write_red(buf);
            sync_compute();
            for (int i = threadIdx.x; i < ROWS * mrows; i += 32 * kW4Warps) {
                const int m = i / ROWS, r = i % ROWS, n = tile * ROWS + r;
                if (n >= a.N) continue;
                float v = 0.0f;
#pragma unroll
                for (int k = 0; k < WK; ++k) v += buf[(k * COLS + m) * PITCH + r];
                finish(v, m, n);
            }
        }
    }
    if (a.split == 1) return;

    // a split: sums over the K warps, then over the cluster in rank order
    __syncthreads();
    if (warp < kW4Warps) write_red(red);
    __syncthreads();
    const int per = ROWS * mrows;
    for (int i = threadIdx.x; i < per; i += kW4Threads) {
        const int m = i / ROWS, r = i % ROWS;
        float v = red[m * PITCH + r];
#pragma unroll
        for (int k = 1; k < WK; ++k) v += red[(k * COLS + m) * PITCH + r];
        red[m * PITCH + r] = v;
    }
    __syncwarp();
    cluster_sync();
    for (int i = rank * kW4Threads + threadIdx.x; i < per; i += a.split * kW4Threads) {
        const int m = i / ROWS, r = i % ROWS, n = tile0 * ROWS + r;
        if (n >= a.N) continue;
        const uint32_t at = smem_addr(red + m * PITCH + r);
        float v = 0.0f;
        for (int c = 0; c < a.split; c += 2) {      // split is 2, 4 or 8
            float p0, p1;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(p0) : "r"(mapa_shared(at, c)) : "memory");
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(p1) : "r"(mapa_shared(at, c + 1)) : "memory");
            v = (v + p0) + p1;
        }
        finish(v, m, n);
    }
    __syncwarp();
    cluster_sync();   // the sums stay in place until every CTA has read them
}

template <typename T, int G, bool TS>
int launch_w4(W4Args a, cudaStream_t st) {
    constexpr int WK = kW4Warps, ROWS = kW4Rows;
    constexpr uint32_t SROW = WK * (256 / G) * 2;
    CUtensorMap mW{}, mX{}, mS{}, mZ{};
    a.mbox = a.M < kW4Cols ? a.M : kW4Cols;
    const int blocks = static_cast<int>(ceil_div(a.M, kW4Cols));
    a.nchunk = a.K / 256;
    // a map needs a chunk to describe; without one (K < 256) no stage is loaded
    if (a.nchunk > 0) {
        const int64_t wd[3] = {128, a.N, a.nchunk}, ws[2] = {a.K / 2, 128};
        const int wb[3] = {128, ROWS, WK};
        const int64_t xd[3] = {64, a.M, 4 * static_cast<int64_t>(a.nchunk)}, xs[2] = {static_cast<int64_t>(a.K) * 2, 128};
        const int xb[3] = {64, a.mbox, 4 * WK};
        if (!make_map_3d(&mW, a.wq, kMapU8, wd, ws, wb, 128) || !make_map_3d(&mX, a.x, kMap16, xd, xs, xb, 128)) return FUSE_ECUDA;
        if (TS) {
            const int64_t kg = a.K / G, sd[3] = {kg, a.N, 1}, ss[2] = {kg * 2, kg * 2 * a.N}, zs[2] = {kg, kg * a.N};
            const int sb[3] = {SROW / 2, ROWS, 1};
            if (!make_map_3d(&mS, a.s, kMap16, sd, ss, sb, G == 32 ? 128 : G == 64 ? 64 : 0)) return FUSE_ECUDA;
            if (a.z && !make_map_3d(&mZ, a.z, kMapU8, sd, zs, sb, 0)) return FUSE_ECUDA;
        }
    }
    a.tiles = static_cast<int>(ceil_div(a.N, ROWS));
    const int nblk = static_cast<int>(ceil_div(a.nchunk, WK));
    a.split = 1;
    // as long as all clusters run at once (two CTAs per SM; a GPC, an eighth of the SMs, takes whole clusters)
    while (a.split < 8 && static_cast<int64_t>(a.tiles) * blocks <= sm_count() / 8 / a.split * 8 && nblk >= 2 * a.split) a.split *= 2;
    const int iters = static_cast<int>(ceil_div(nblk > 0 ? nblk : 1, a.split));
    // X stays in shared memory for all of a CTA's tiles where it is small (whole stages of it keep the
    // swizzle's phase: 4 WK mbox rows are a multiple of 8), else it comes with every stage
    const int x_stage = 4 * WK * a.mbox * 128;
    a.x_resident = a.split == 1 && a.tiles > sm_count() && iters * x_stage <= 32 * 1024 ? 1 : 0;
    const uint32_t w_stage = WK * ROWS * 128;
    a.s_off = w_stage + (a.x_resident ? 0 : x_stage);
    a.stage_bytes = (a.s_off + (TS ? ROWS * SROW + (a.z ? ROWS * SROW / 2 : 0) : 0) + 1023) / 1024 * 1024;
    const uint32_t x_all = a.x_resident ? iters * x_stage : 0;
    const uint32_t pad = kW4Cols * 128;     // columns past M are read from behind the last rows of X
    const bool several = a.split == 1;     // row tiles per CTA, with two buffers of partial sums
    const uint32_t red = static_cast<uint32_t>((several ? 2 : 1) * WK * kW4Cols * (ROWS + 4) * 4);
    const uint32_t bars = 8 * (2 * kW4MaxStages + 1);
    constexpr uint32_t budget = 112 * 1024;     // two CTAs per SM
    const int want = a.split > 1 ? iters : kW4MaxStages;
    a.stages = want < kW4MaxStages ? want : kW4MaxStages;
    while (a.stages > 2 && a.stages * a.stage_bytes + x_all + red + pad + bars + 1024 > budget) --a.stages;
    a.x_off = a.x_resident ? a.stages * a.stage_bytes : w_stage;
    a.off_red = (a.stages * a.stage_bytes + x_all + pad + 15) / 16 * 16;
    a.off_bar = a.off_red + (red + 15) / 16 * 16;
    const uint32_t smem = a.off_bar + bars + 1024;
    if (smem > kW4Smem) return FUSE_EUNSUPPORTED;
    const int rc = opt_in_smem((const void*)w4_gemv_kernel<T, G, TS>, kW4Smem, true);
    if (rc != FUSE_OK) return rc;
    int64_t grid = static_cast<int64_t>(a.tiles) * a.split;
    if (several) {   // as many CTAs as are resident; each takes every grid-th row tile
        static std::atomic<uint32_t> known{0};    // shared memory (KB) and CTAs per SM of the last launch
        const uint32_t kb = (smem + 1023) / 1024;
        uint32_t k = known.load(std::memory_order_relaxed);
        if ((k >> 8) != kb) {
            k = (kb << 8) | static_cast<uint32_t>(blocks_per_sm(w4_gemv_kernel<T, G, TS>, kW4Threads, kb * 1024));
            known.store(k, std::memory_order_relaxed);
        }
        const int64_t resident = static_cast<int64_t>(sm_count()) * (k & 255u) / blocks > 0 ? static_cast<int64_t>(sm_count()) * (k & 255u) / blocks : 1;
        if (grid > resident) grid = resident;
    }
    return launch_pdl(w4_gemv_kernel<T, G, TS>, dim3(static_cast<unsigned>(grid), static_cast<unsigned>(blocks)), dim3(kW4Threads), smem, st, a.split, mW, mX, mS, mZ, a);
}

// ================================================================== tcgen05 tiles
// More than a few tokens make the matrix instructions count.  The integers q - z go from registers into
// tensor memory as the A operand of tcgen05.mma (128 weight rows x 128 k per unit, two 16-bit integers per
// TMEM column), X is the B operand from shared memory, and every group of k has its own fp32 accumulator
// in TMEM, which is read out, multiplied by the group's scale and added up in registers.
//
// Measured: 64 x 28672 x 4096 in groups of 64 36.9 us, 64 x 4096 x 4096 in groups of 128 11.5 us, 32 x 8192 x 8192 18.0 us.
// Not the loads (36.7 us with X loaded for the first stages only, 36.9 with the weights so) but the chain of a unit
// (unpack, MMAs, read-out) and its instructions bound it: the SMs issue half of the time.  Separate warps for unpacking
// and for reading out took 38.5 us when this form took 35.4.
//
// 320 threads: warps 0-7 work (TMEM lane quadrant warp % 4, i.e. 32 weight rows, one per lane; half
// warp / 4 of a unit's k when unpacking and of the tokens when reading out), warp 8 issues the MMAs, warp 9
// loads by TMA: weights (64-byte swizzle: the 16-byte reads of 8 consecutive rows are free of bank
// conflicts), X (128-byte swizzle), and scales and zero points for 16 groups at a time.  A worker unpacks
// unit u + 1 before it reads out unit u, so the MMAs of a unit run while the next one is unpacked.  Two
// CTAs share an SM (256 TMEM columns each): A 2 x 64, accumulators 128.  A cluster splits K; its sums meet
// in distributed shared memory in rank order.
constexpr int kTileWorkers = 8;
constexpr int kTileThreads = 32 * (kTileWorkers + 2);
constexpr int kTileStages = 4;
constexpr uint32_t kTileCols = 256, kTileD = 128;   // TMEM columns; first accumulator column

template <int NM>
struct TileLayout {
    static constexpr uint32_t W = 128 * 64;                          // weights of a stage
    static constexpr uint32_t X = NM * 128;                          // one 64-k atom of X
    static constexpr uint32_t STAGE = W + 2 * X;
    static constexpr uint32_t S = 2 * 128 * 16, Z = 128 * 16;        // scales and zeros of 16 groups
    static constexpr uint32_t OFF_S = kTileStages * STAGE;
    static constexpr uint32_t OFF_Z = OFF_S + 2 * S;
    static constexpr uint32_t OFF_BAR = OFF_Z + 2 * Z;
    static constexpr int N_BARS = 2 * kTileStages + 4 + 2 + 4 + 1;
    static constexpr uint32_t OFF_HOLD = OFF_BAR + N_BARS * 8;
    static constexpr uint32_t SMEM = OFF_HOLD + 16 + 1024;
    static_assert(SMEM <= 113 * 1024, "two CTAs per SM");
    static_assert(NM * 128 * 4 <= kTileStages * STAGE, "the sums of a split fit in the ring");
};

struct TileArgs {
    int M, N;
    int nchunk;        // 128-k chunks (whole ones: scales that the copy engine can load make K a multiple of 256)
    int per;           // chunks of a CTA
    int split, gelu, zeros;
    int y_vec;         // y is 8-byte aligned
    const void *bias, *R;
    void* y;
    int* flag;
};

template <typename T, int G, int NM>
__global__ void __launch_bounds__(kTileThreads, 2) w4_tile_kernel(
    const __grid_constant__ CUtensorMap mW, const __grid_constant__ CUtensorMap mX,
    const __grid_constant__ CUtensorMap mS, const __grid_constant__ CUtensorMap mZ,
    const __grid_constant__ TileArgs a) {
    using L = TileLayout<NM>;
    constexpr int NG = 128 / G;          // groups of a unit
    constexpr int UPB = 16 / NG;         // units of a block of scales
    constexpr int HT = NM / 2;           // tokens of a worker
    // The accumulators of a unit's groups form one set (two, one after the other, where a unit has more
    // groups than there are columns for); as many sets as fit, at most two.
    constexpr int SG = NG * NM <= 128 ? NG : 128 / NM;   // groups of a set
    constexpr int SETS = NG / SG;                        // sets of a unit
    constexpr int ND = 2 * SG * NM <= 128 ? 2 : 1;       // set buffers
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - smem_addr(smem_raw));
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    const int rank = a.split > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int n0 = static_cast<int>(blockIdx.x) / a.split * 128;
    const int c0 = rank * a.per;
    const int units = max(0, min(a.per, a.nchunk - c0));
    const uint32_t bar0 = base + L::OFF_BAR;
    // A ring of n buffers used for the 0th, 1st, ... time: parity of use i of a buffer is i & 1.
    auto full = [&](int i) { return bar0 + 8u * i; };
    auto empty = [&](int i) { return bar0 + 8u * (kTileStages + i); };
    auto s_full = [&](int i) { return bar0 + 8u * (2 * kTileStages + i); };
    auto s_empty = [&](int i) { return bar0 + 8u * (2 * kTileStages + 2 + i); };
    auto a_full = [&](int i) { return bar0 + 8u * (2 * kTileStages + 4 + i); };
    auto d_full = [&](int i) { return bar0 + 8u * (2 * kTileStages + 6 + i); };
    auto d_empty = [&](int i) { return bar0 + 8u * (2 * kTileStages + 8 + i); };
    const uint32_t drain = bar0 + 8u * (2 * kTileStages + 10);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kTileStages; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full(i), 1);
            mbar_init(s_empty(i), kTileWorkers);
            mbar_init(a_full(i), kTileWorkers);
            mbar_init(d_full(i), 1);
            mbar_init(d_empty(i), kTileWorkers);
        }
        mbar_init(drain, 1);
        fence_mbar_init();
    }
    if (warp == kTileWorkers) tmem_alloc(base + L::OFF_HOLD, kTileCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(gbase + L::OFF_HOLD), 0);
    // Only with its tensor memory in hand: a kernel that starts early and takes all of an SM's would wait for this one,
    // which would wait for the memory.
    pdl_trigger();
    pdl_wait();
    // the residual's lines of this tile, for the epilogue: 64 rows of a token each
    if (a.R && rank == 0)
        for (int l = threadIdx.x; l < 2 * a.M; l += kTileThreads) {
            const int n = n0 + 64 * (l & 1);
            if (n < a.N) asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const T*>(a.R) + static_cast<int64_t>(l >> 1) * a.N + n));
        }

    float acc[HT];
#pragma unroll
    for (int i = 0; i < HT; ++i) acc[i] = 0.0f;
    if (warp == kTileWorkers + 1) {
        // ---------------------------------------------------------------- loads
        if (lane == 0 && units > 0) {
            prefetch_map(&mW);
            prefetch_map(&mX);
            prefetch_map(&mS);
            if (a.zeros) prefetch_map(&mZ);
            const uint32_t bytes = L::W + 2u * a.M * 128u;
            int u = 0, blocks = 0;
            bool ok = true;
            for (; u < units; ++u) {
                const int st = u % kTileStages;
                if (u == 0 || (c0 + u) % UPB == 0) {
                    const int sb = blocks & 1;
                    if (blocks >= 2 && !mbar_wait_bounded(s_empty(sb), ((blocks >> 1) - 1) & 1, a.flag)) {
                        ok = false;
                        break;
                    }
                    const int g0 = (c0 + u) / UPB * 16;     // whole blocks, whatever chunk the CTA starts at
                    mbar_arrive_expect_tx(s_full(sb), L::S + (a.zeros ? L::Z : 0u));
                    tma_load_3d(base + L::OFF_S + sb * L::S, &mS, g0, n0, 0, s_full(sb));
                    tma_load_3d(base + L::OFF_S + sb * L::S + L::S / 2, &mS, g0 + 8, n0, 0, s_full(sb));
                    if (a.zeros) tma_load_3d(base + L::OFF_Z + sb * L::Z, &mZ, g0, n0, 0, s_full(sb));
                    ++blocks;
                }
                if (u >= kTileStages && !mbar_wait_bounded(empty(st), (u / kTileStages - 1) & 1, a.flag)) {
                    ok = false;
                    break;
                }
                const uint32_t at = base + st * L::STAGE;
                mbar_arrive_expect_tx(full(st), bytes);
                tma_load_3d(at, &mW, (c0 + u) * 64, n0, 0, full(st));
                tma_load_2d(at + L::W, &mX, (c0 + u) * 128, 0, full(st));
                tma_load_2d(at + L::W + L::X, &mX, (c0 + u) * 128 + 64, 0, full(st));
            }
            if (!ok) {   // copies in flight land before the shared memory goes away
                for (int j = max(0, u - kTileStages); j < u; ++j) (void)mbar_wait_drain(full(j % kTileStages), (j / kTileStages) & 1);
                for (int j = max(0, blocks - 2); j < blocks; ++j) (void)mbar_wait_drain(s_full(j & 1), (j >> 1) & 1);
            }
        }
        __syncwarp();
    } else if (warp == kTileWorkers) {
        // ---------------------------------------------------------------- MMA issue
        constexpr uint32_t idesc = idesc_f16(128, NM, false, false, std::is_same<T, __nv_bfloat16>::value);
        const uint32_t one = elect_one();
        const uint64_t desc0 = smem_desc_sw128(base + L::W, 16, 1024);
        bool ok = true, issued = false;
        auto wait = [&](uint32_t bar, uint32_t parity) {
            ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, a.flag));
            return ok;
        };
        int st = 0, d = 0;
        uint32_t st_par = 0, a_par = 0, d_par = 1;   // parities of the next waits; d_empty needs none at first
        bool d_again = false;
        for (int u = 0; ok && u < units; ++u) {
            const int ab = u & 1;
            if (!wait(a_full(ab), a_par) || !wait(full(st), st_par)) break;
            const uint64_t xd = desc0 + static_cast<uint64_t>(st * (L::STAGE >> 4));
            const uint32_t at = tmem + ab * 64;
#pragma unroll
            for (int h = 0; h < SETS; ++h) {
                if (d_again && !wait(d_empty(d), d_par)) break;
                tc_fence_after();
                const uint32_t dt = tmem + kTileD + d * (SG * NM);
#pragma unroll
                for (int g = 0; g < SG; ++g)
#pragma unroll
                    for (int k = 0; k < G / 16; ++k) {
                        const int s = (h * SG + g) * (G / 16) + k;
                        tc_mma_ts_if(one, dt + g * NM, at + s * 8, xd + ((s / 4) * (L::X >> 4) + (s % 4) * 2), idesc, k > 0 ? 1u : 0u);
                    }
                tc_commit_if(one, d_full(d));
                issued = true;
                if (++d == ND) {
                    d = 0;
                    d_par ^= 1u;
                    d_again = true;
                }
            }
            if (ok) tc_commit_if(one, empty(st));
            a_par ^= static_cast<uint32_t>(ab);
            if (++st == kTileStages) {
                st = 0;
                st_par ^= 1u;
            }
        }
        if (!ok && issued) {   // MMAs in flight finish before TMEM is freed
            tc_commit_if(one, drain);
            (void)mbar_wait_drain(drain, 0);
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- unpack and read out
        const int qd = warp % 4, hh = warp / 4, r = 32 * qd + lane;
        const uint32_t lanes = static_cast<uint32_t>(32 * qd) << 16;
        bool ok = true;
        auto wait = [&](uint32_t bar, uint32_t parity) {
            ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity & 1u, a.flag));
            return ok;
        };
        auto arrive = [&](uint32_t bar) {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        const uint32_t b0 = static_cast<uint32_t>(c0) / UPB;      // the CTA's first block of scales
        int d = 0, st = 0;
        uint32_t d_par = 0, st_par = 0;
        for (int u = 0; u <= units && ok; ++u) {
            if (u < units) {
                const uint32_t c = c0 + u, blk = c / UPB - b0, sb = blk & 1;
                const int ab = u & 1;
                if ((u == 0 || c % UPB == 0) && !wait(s_full(sb), blk >> 1)) break;
                if (!wait(full(st), st_par)) break;
                // A buffer ab is free: the accumulators of unit u - 2 have been waited for
                // this thread's row: 64 k from 64 hh on, two 16-byte pieces of the row's four
                const uint8_t* row = gbase + st * L::STAGE + r * 64;
                const uint32_t sw = static_cast<uint32_t>((r >> 1) & 3);
                const uint4 w0 = *reinterpret_cast<const uint4*>(row + (((2u * hh) ^ sw) << 4)), w1 = *reinterpret_cast<const uint4*>(row + (((2u * hh + 1u) ^ sw) << 4));
                const uint32_t words[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
                uint32_t zb[2] = {Nib<T>::MAGIC | 0x00080008u, Nib<T>::MAGIC | 0x00080008u};   // first and second 32 k
                if (a.zeros) {
                    const uint8_t* zp = gbase + L::OFF_Z + sb * L::Z + r * 16 + c % UPB * NG;
#pragma unroll
                    for (int i = 0; i < 2; ++i) zb[i] = Nib<T>::MAGIC | (zp[(64 * hh + 32 * i) / G] & 15u) * 0x00010001u;
                }
                float p[32];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint32_t q[4];
                    unpack_word<T>(words[i], zb[i / 4], q);
#pragma unroll
                    for (int e = 0; e < 4; ++e) p[4 * i + e] = __uint_as_float(q[e]);
                }
                tmem_st32(tmem + lanes + ab * 64 + 32 * hh, p);
                tmem_st_wait();
                tc_fence_before();
                arrive(a_full(ab));
                if (++st == kTileStages) {
                    st = 0;
                    st_par ^= 1u;
                }
            }
            if (u > 0) {
                const uint32_t v = c0 + u - 1, sb = (v / UPB - b0) & 1;      // chunk
                const uint8_t* sp = gbase + L::OFF_S + sb * L::S + r * 16;
#pragma unroll
                for (int h = 0; h < SETS; ++h) {
                    if (!wait(d_full(d), d_par)) break;
                    tc_fence_after();
#pragma unroll
                    for (int g = 0; g < SG; ++g) {
                        float x[HT];
                        const uint32_t at = tmem + lanes + kTileD + (d * SG + g) * NM + HT * hh;
                        if constexpr (HT == 32) tmem_ld32(at, x);
                        else if constexpr (HT == 16) tmem_ld16(at, x);
                        else tmem_ld8(at, x);
                        const uint32_t gb = v % UPB * NG + h * SG + g;      // group of the block
                        const float s = to_f32(*reinterpret_cast<const T*>(sp + (gb / 8) * (L::S / 2) + (gb % 8) * 2));
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < HT; i += 2) {
                            const float2 t = __ffma2_rn(make_float2(s, s), make_float2(x[i], x[i + 1]), make_float2(acc[i], acc[i + 1]));
                            acc[i] = t.x;
                            acc[i + 1] = t.y;
                        }
                    }
                    tc_fence_before();
                    arrive(d_empty(d));
                    if (++d == ND) {
                        d = 0;
                        d_par ^= 1u;
                    }
                }
                if (ok && v % UPB == UPB - 1) arrive(s_empty(sb));
            }
        }
    }

    // epilogue: thread (row r, tokens HT hh ..) of the workers; a split's sums in rank order
    const T* bias = static_cast<const T*>(a.bias);
    const T* R = static_cast<const T*>(a.R);
    T* y = static_cast<T*>(a.y);
    tc_fence_before();
    __syncthreads();      // every load has landed and every MMA is done: TMEM and the ring are free
    if (warp == kTileWorkers) {
        tc_fence_after();
        tmem_dealloc(tmem, kTileCols);
    }
    const int r = 32 * (warp % 4) + lane, t0 = HT * (warp / 4);
    if (a.split == 1) {
        const int n = n0 + r;
        if (warp < kTileWorkers && n < a.N) {
            const float b = bias ? to_f32(bias[n]) : 0.0f;
            float res[HT];        // all of them on their way before the first store
#pragma unroll
            for (int i = 0; i < HT; ++i)
                res[i] = R && t0 + i < a.M ? to_f32(R[static_cast<int64_t>(t0 + i) * a.N + n]) : 0.0f;
#pragma unroll
            for (int i = 0; i < HT; i += 2) {
                float2 v = make_float2(acc[i] + b, acc[i + 1] + b);
                if (a.gelu) v = gelu_erf2(v);
                if (t0 + i < a.M) y[static_cast<int64_t>(t0 + i) * a.N + n] = from_f32<T>(v.x + res[i]);
                if (t0 + i + 1 < a.M) y[static_cast<int64_t>(t0 + i + 1) * a.N + n] = from_f32<T>(v.y + res[i + 1]);
            }
        }
        return;
    }
    float* red = reinterpret_cast<float*>(gbase);   // [token][128]
    if (warp < kTileWorkers) {
#pragma unroll
        for (int i = 0; i < HT; ++i) red[(t0 + i) * 128 + r] = acc[i];
    }
    __syncwarp();
    cluster_sync();
    // four rows of one token at a time, two such pieces per thread with their loads together
    const int pieces = a.M * 32;
    for (int i0 = rank * kTileThreads + threadIdx.x; i0 < pieces; i0 += 2 * a.split * kTileThreads) {
        float v[2][4], b[2][4], res[2][4];
        int m[2], n[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int i = min(i0 + j * a.split * kTileThreads, pieces - 1);   // past the end: not stored
            m[j] = i / 32;
            n[j] = n0 + i % 32 * 4;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[j][e] = 0.0f;
                b[j][e] = bias && n[j] + e < a.N ? to_f32(bias[n[j] + e]) : 0.0f;
                res[j][e] = R && n[j] + e < a.N ? to_f32(R[static_cast<int64_t>(m[j]) * a.N + n[j] + e]) : 0.0f;
            }
        }
        for (int c = 0; c < a.split; c += 2) {      // split is 2, 4 or 8
            float p[2][2][4];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t at = mapa_shared(smem_addr(red + m[j] * 128 + (n[j] - n0)), c + k);
                    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                                 : "=f"(p[k][j][0]), "=f"(p[k][j][1]), "=f"(p[k][j][2]), "=f"(p[k][j][3]) : "r"(at) : "memory");
                }
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[j][e] += p[k][j][e];
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (i0 + j * a.split * kTileThreads >= pieces) break;
            float o[4];
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                float2 x = make_float2(v[j][e] + b[j][e], v[j][e + 1] + b[j][e + 1]);
                if (a.gelu) x = gelu_erf2(x);
                o[e] = x.x + res[j][e];
                o[e + 1] = x.y + res[j][e + 1];
            }
            T* dst = y + static_cast<int64_t>(m[j]) * a.N + n[j];
            if (n[j] >= a.N) continue;
            if (a.N % 4 == 0 && a.y_vec) {
                *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<T>(o[0], o[1]), pack2<T>(o[2], o[3]));
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n[j] + e < a.N) dst[e] = from_f32<T>(o[e]);
            }
        }
    }
    __syncwarp();
    cluster_sync();   // the sums stay in place until every CTA has read them
}

// Whether the copy engine can load the scales (and zero points): whole 16-byte pieces of a row.
bool scales_fit(const W4Args& a, int group) {
    const int kg = a.K / group;
    return kg % 8 == 0 && is_aligned(a.s, 16) && (!a.z || (kg % 16 == 0 && is_aligned(a.z, 16)));
}

template <typename T, int G, int NM>
int launch_tile(const W4Args& w, cudaStream_t st) {
    using L = TileLayout<NM>;
    TileArgs a{};
    a.M = w.M;
    a.N = w.N;
    a.nchunk = w.K / 128;
    a.gelu = w.gelu;
    a.zeros = w.z ? 1 : 0;
    a.y_vec = is_aligned(w.y, 8) ? 1 : 0;
    a.bias = w.bias;
    a.R = w.R;
    a.y = w.y;
    a.flag = w.flag;
    const int tiles = static_cast<int>(ceil_div(w.N, 128)), sms = sm_count();
    // The split with the least of (chunks of a CTA + 5 for its start and end) x waves.  A wave is two CTAs per SM in whole
    // clusters (a GPC, an eighth of the SMs, takes floor(38 / split) of them); a last wave that is not full counts half
    // and half its share, as its CTAs get an SM to themselves, and so does three quarters of a wave that all fits one CTA
    // per SM.  Measured for splits 1, 2, 4 and 8 (tiles of 128 rows x chunks of 128 inputs, us; best chosen but for 1 of
    // 29 sizes, by 6 %): 16 x 32 24.8, 14.3, 12.1, 10.6; 40 x 32 32, 18.6, 12.8, 16.9; 76 x 64 42, 23, 30, 32;
    // 32 x 112 78, 54, 31, 21; 140 x 32 40, 21, 26, 42; 224 x 32 42, 36, 45, 64; 300 x 32 41, 41, 55, 82.
    double best = 0.0;
    a.split = 0;
    for (int s = 1; s <= 8; s *= 2) {
        const int per = static_cast<int>(ceil_div(a.nchunk, s)), wave = sms / 4 / s * 8;
        if (wave < 1) break;
        const int full = tiles / wave, rest = tiles % wave;
        double waves = full + (rest > 0 ? full > 0 ? 0.5 + 0.5 * rest / wave : 1.0 : 0.0);
        if (static_cast<int64_t>(tiles) * s <= sms) waves = 0.75;
        const double cost = (per + 5) * waves;
        if (a.split == 0 || cost < best) {
            best = cost;
            a.split = s;
            a.per = per;
        }
    }
    CUtensorMap mW{}, mX{}, mS{}, mZ{};
    const int64_t KG = w.K / G;
    const int64_t wd[3] = {w.K / 2, w.N, 1}, ws[2] = {w.K / 2, static_cast<int64_t>(w.K / 2) * w.N};
    const int wb[3] = {64, 128, 1};
    const int64_t sd[3] = {KG, w.N, 1}, ss[2] = {KG * 2, KG * 2 * w.N};
    const int sbx[3] = {8, 128, 1};
    const int64_t zd[3] = {KG, w.N, 1}, zs[2] = {KG, KG * w.N};
    const int zbx[3] = {16, 128, 1};
    if (!make_map_3d(&mW, w.wq, kMapU8, wd, ws, wb, 64) || !make_map(&mX, w.x, w.M, w.K, 64, w.M, std::is_same<T, __nv_bfloat16>::value) ||
        !make_map_3d(&mS, w.s, kMap16, sd, ss, sbx, 0) || (w.z && !make_map_3d(&mZ, w.z, kMapU8, zd, zs, zbx, 0)))
        return FUSE_ECUDA;
    const int rc = opt_in_smem((const void*)w4_tile_kernel<T, G, NM>, L::SMEM, true);
    if (rc != FUSE_OK) return rc;
    return launch_pdl(w4_tile_kernel<T, G, NM>, dim3(static_cast<unsigned>(tiles * a.split)), dim3(kTileThreads), L::SMEM, st, a.split, mW, mX, mS, mZ, a);
}

template <typename T, int G>
int run_w4_g(const W4Args& a, cudaStream_t st) {
    const bool fits = scales_fit(a, G);
    // More than 8 tokens take another pass of w4_gemv_kernel over the weights.  At 9 tokens it takes 8.5 us for 4096 x
    // 4096 (tiles 8.2), 22.2 for 8192 x 8192 (17.2), 41 for 28672 x 4096 (29); at 8 7.8, 13.4 and 19.8.
    // Without scales that the copy engine can load it is those passes all the same: 64 x 4096 x 11008 in groups of 128
    // (86 scales a row) takes 51 us where 64 x 4096 x 11264 takes 17.8, 16 tokens 16.8 and 14.6, up to 8 are as fast.
    if (fits && a.M > 8) {
        if (a.M <= 16) return launch_tile<T, G, 16>(a, st);
        if (a.M <= 32) return launch_tile<T, G, 32>(a, st);
        return launch_tile<T, G, 64>(a, st);
    }
    return fits ? launch_w4<T, G, true>(a, st) : launch_w4<T, G, false>(a, st);
}
template <typename T>
int run_w4(const W4Args& a, int group, cudaStream_t st) {
    if (group == 32) return run_w4_g<T, 32>(a, st);
    if (group == 64) return run_w4_g<T, 64>(a, st);
    return run_w4_g<T, 128>(a, st);
}

template <typename T, int G>
int w4_entry(int i, const char* const* names, fuse_kernel_record* out) {
    switch (i) {
        case 0: return describe_kernel((const void*)w4_gemv_kernel<T, G, true>, names[0], kW4Threads, 110 * 1024, out);
        case 1: return describe_kernel((const void*)w4_gemv_kernel<T, G, false>, names[1], kW4Threads, 110 * 1024, out);
        case 2: return describe_kernel((const void*)w4_tile_kernel<T, G, 16>, names[2], kTileThreads, TileLayout<16>::SMEM, out, kTileCols);
        case 3: return describe_kernel((const void*)w4_tile_kernel<T, G, 32>, names[3], kTileThreads, TileLayout<32>::SMEM, out, kTileCols);
        default: return describe_kernel((const void*)w4_tile_kernel<T, G, 64>, names[4], kTileThreads, TileLayout<64>::SMEM, out, kTileCols);
    }
}

}  // namespace

int w4_report_count() { return 30; }
int w4_report(int i, fuse_kernel_record* out) {
    if (i < 0 || i >= 30) return FUSE_EINVAL;
#define FC_W4(T, G)                                                                                             \
    {"w4_gemv_kernel<" T ", group " G ">", "w4_gemv_kernel<" T ", group " G ", scales of any alignment>",       \
     "w4_tile_kernel<" T ", group " G ", M <= 16> (tcgen05)", "w4_tile_kernel<" T ", group " G ", M <= 32> (tcgen05)", \
     "w4_tile_kernel<" T ", group " G ", M <= 64> (tcgen05)"}
    static const char* const names[6][5] = {FC_W4("bf16", "32"), FC_W4("bf16", "64"), FC_W4("bf16", "128"),
                                            FC_W4("f16", "32"), FC_W4("f16", "64"), FC_W4("f16", "128")};
#undef FC_W4
    const int k = i / 5, v = i % 5;
    switch (k) {
        case 0: return w4_entry<__nv_bfloat16, 32>(v, names[k], out);
        case 1: return w4_entry<__nv_bfloat16, 64>(v, names[k], out);
        case 2: return w4_entry<__nv_bfloat16, 128>(v, names[k], out);
        case 3: return w4_entry<__half, 32>(v, names[k], out);
        case 4: return w4_entry<__half, 64>(v, names[k], out);
        default: return w4_entry<__half, 128>(v, names[k], out);
    }
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
