// mxfp4.cu -- microscaled 4-bit floating point: quantisation, and the product of two quantised operands.
//
// 32 consecutive values of a row share a scale 2^e, 2^(e + 2) <= max |v| < 2^(e + 3) (so the largest lies between 4
// and 8, and what exceeds 6 becomes 6); each value is v / 2^e rounded to 0, 1/2, 1, 3/2, 2, 3, 4 or 6, ties to the even
// code.  Dividing by a power of two is exact, so the codes are what the definition says, bit for bit.  Scales are
// held as bytes e + 127 (255: not a number) in tiles of 128 rows by 4 scales, 512 bytes each, in the order in which
// the tensor core takes them: byte (r % 32) 16 + (r / 32) 4 + s of a tile is row r's scale s.
//
//  * mxfp4_quantize_kernel, mxfp4_dequantize_kernel: bound by HBM.  A CTA takes a tile's 128 rows by 128 values.  28672 x 4096
//    in bf16: 45.3 us (6.57 TB/s) and 44.1 us (6.75 TB/s).
//  * mxfp4_gemm_kernel: Y = GELU(X W^T + bias) + R with X [M, K] and W [N, K] both quantised.  The weights are the
//    tensor core's 128 rows and the tokens its columns, so a warp's stores of a token are consecutive outputs and
//    few tokens cost few columns.  kind::mxf4 multiplies 64 values of a row at once, at four times the rate of 16-bit
//    operands; the scales go from shared memory to TMEM next to the accumulators.  K may be split over a
//    cluster of CTAs, whose sums meet in shared memory.  In a stream of equal calls, their weights in L2, one token of 4096 x 4096 4.2
//    us, 100 of 4096 x 14336 10.2 and 13.3 with their quantisation; with weights from HBM 4.4, and 18.6 with the quantisation: bound
//    by latency, the weights' way through a ring of stages and the join.
//  * mxfp4_pair_kernel: the same for many tokens, bound by the tensor cores and at short K by the change of accumulators.
#include <cudaTypedefs.h>
#include <math.h>

#include <mutex>
#include <type_traits>

#include "fc_internal.cuh"
#include "fc_mma.cuh"
#include "fc_ptx.cuh"
#include "fc_tc.cuh"
#include "gemm_epi.cuh"

namespace fc {
namespace {

constexpr int kQThreads = 256;

// ================================================================== quantisation
// Eight values to codes, the first in the lowest four bits.
__device__ __forceinline__ uint32_t to_e2m1(const float* v) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}
// The values of eight codes (exact in fp16).
__device__ __forceinline__ void from_e2m1(uint32_t c, float* v) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(c));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<__half>(h[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

struct QuantArgs {
    const void* x;
    int64_t ld;
    uint8_t *q, *s;
    int64_t rows, cols;
};

// Eight threads of 16 values (16-bit x) or sixteen of 8 (fp32) take a row's 128 values.
template <typename T>
__global__ void __launch_bounds__(kQThreads) mxfp4_quantize_kernel(const __grid_constant__ QuantArgs a) {
    constexpr int N = Vec32<T>::N, PER_ROW = 128 / N, ROWS = kQThreads / PER_ROW, GROUP = 32 / N, ITER = 128 / ROWS;
    __shared__ uint8_t tile[512];
    pdl_begin();
    const int tid = threadIdx.x, ch = tid % PER_ROW;
    const int64_t row0 = static_cast<int64_t>(blockIdx.y) * 128, col = static_cast<int64_t>(blockIdx.x) * 128 + ch * N;
    // (fp32: four vectors on their way at a time, 8192 x 4096 28.1 -> 23.8 us; the shorter 16-bit vectors gain nothing by it)
    constexpr int AHEAD = sizeof(T) == 4 ? 4 : 1;
#pragma unroll
    for (int i0 = 0; i0 < ITER; i0 += AHEAD) {
        float vs[AHEAD][N];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int r = tid / PER_ROW + (i0 + i) * ROWS;
#pragma unroll
            for (int e = 0; e < N; ++e) vs[i][e] = 0.0f;
            if (row0 + r < a.rows && col < a.cols) Vec32<T>::load(static_cast<const T*>(a.x) + (row0 + r) * a.ld + col, vs[i]);
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int r = tid / PER_ROW + (i0 + i) * ROWS;
            const bool in = row0 + r < a.rows && col < a.cols;
            float (&v)[N] = vs[i];
            uint32_t top = 0;                    // the largest magnitude's bits (infinity and NaN above all)
#pragma unroll
            for (int e = 0; e < N; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
#pragma unroll
            for (int o = 1; o < GROUP; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            const uint32_t field = top >> 23;    // max |v| >= 2^(field - 127)
            const uint32_t scale = field == 255u ? 255u : field > 2u ? field - 2u : 0u;
            const float inv = __uint_as_float((254u - min(scale, 253u)) << 23);
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] *= inv;
            if (in) {
                uint8_t* q = a.q + (row0 + r) * (a.cols / 2) + col / 2;
                if constexpr (N == 16) *reinterpret_cast<uint2*>(q) = make_uint2(to_e2m1(v), to_e2m1(v + 8));
                else *reinterpret_cast<uint32_t*>(q) = to_e2m1(v);
            }
            // (scales of rows and values past the matrix are 0: with codes of 0 they add nothing to a product)
            if (ch % GROUP == 0) tile[(r % 32) * 16 + (r / 32) * 4 + ch / GROUP] = static_cast<uint8_t>(in ? scale : 0u);
        }
    }
    __syncthreads();
    if (tid < 32)
        reinterpret_cast<uint4*>(a.s + (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * 512)[tid] = reinterpret_cast<uint4*>(tile)[tid];
}

template <typename T>
__global__ void __launch_bounds__(kQThreads) mxfp4_dequantize_kernel(const __grid_constant__ QuantArgs a, T* y) {
    constexpr int N = Vec32<T>::N, PER_ROW = 128 / N, ROWS = kQThreads / PER_ROW, GROUP = 32 / N, ITER = 128 / ROWS;
    __shared__ uint8_t tile[512];
    pdl_begin();
    const int tid = threadIdx.x, ch = tid % PER_ROW;
    if (tid < 32)
        reinterpret_cast<uint4*>(tile)[tid] = __ldcg(reinterpret_cast<const uint4*>(a.s + (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * 512) + tid);
    const int64_t row0 = static_cast<int64_t>(blockIdx.y) * 128, col = static_cast<int64_t>(blockIdx.x) * 128 + ch * N;
    uint2 w[ITER];
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        const int64_t row = row0 + tid / PER_ROW + i * ROWS;
        w[i] = make_uint2(0u, 0u);
        if (row < a.rows && col < a.cols) {
            const uint8_t* q = a.q + row * (a.cols / 2) + col / 2;
            if constexpr (N == 16) w[i] = __ldcg(reinterpret_cast<const uint2*>(q));
            else w[i].x = __ldcg(reinterpret_cast<const uint32_t*>(q));
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        const int r = tid / PER_ROW + i * ROWS;
        if (row0 + r >= a.rows || col >= a.cols) continue;
        const uint32_t s = tile[(r % 32) * 16 + (r / 32) * 4 + ch / GROUP];
        const float scale = __uint_as_float(s == 255u ? 0x7fc00000u : s == 0u ? 0x00400000u : s << 23);
        float v[N];
        from_e2m1(w[i].x, v);
        if constexpr (N == 16) from_e2m1(w[i].y, v + 8);
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] *= scale;
        Vec32<T>::store(y + (row0 + r) * a.cols + col, v);
    }
}

// ================================================================== product
// The accumulator's rows are weights (N), its columns tokens (M).
constexpr int kStageK = 256;                        // values of a row per stage: 128 bytes
// The product's K: a tile's scales (1024 bytes a stage) are counted in 32 bits, and the epilogue waits for all stages of an output in
// one bounded wait of a second.
constexpr int64_t kMostK = int64_t(1) << 29;
constexpr uint32_t kTileBytes = 128 * 128;          // 128 rows of a stage
constexpr int kGemmThreads = 32 * 6;                // warp 0: loads, 1: MMA issue, 2-5: epilogue

template <int NT>
struct GemmLayout {
    static constexpr uint32_t B_BYTES = NT * 128;
    static constexpr uint32_t STAGE = kTileBytes + B_BYTES + 2048;      // weights, tokens, the two operands' scales
    static constexpr int STAGES = NT <= 32 ? 5 : NT == 64 ? 4 : 6;      // up to 64 tokens two CTAs per SM
    static constexpr uint32_t OFF_BAR = STAGES * STAGE;
    static constexpr uint32_t OFF_HOLD = OFF_BAR + (2 * STAGES + 2) * 8;
    static constexpr uint32_t SMEM = OFF_HOLD + 16 + 1024;
    static constexpr uint32_t OFF_B = kTileBytes, OFF_SA = OFF_B + B_BYTES, OFF_SB = OFF_SA + 1024;
    static constexpr uint32_t TMEM_COLS = NT <= 32 ? 64 : NT == 64 ? 128 : 256;
    static constexpr uint32_t SFA_COL = NT, SFB_COL = NT + 8;           // two tiles of scales each
    static_assert(B_BYTES % 1024 == 0, "swizzle atoms");
    static_assert(SMEM <= 232448, "shared-memory budget");
    static_assert(SFB_COL + 8 <= TMEM_COLS, "TMEM");
    static_assert(128 * NT * 4 <= OFF_BAR, "partial sums fit over the stages");
};

struct GemmArgs {
    const uint8_t *xs, *ws;       // scale tiles
    const void *bias, *R;
    void* y;
    int M, N, K;
    int xtk;                      // scale tiles along K
    int stages;                   // of the whole K
    int split;                    // CTAs that share a tile
    int gelu;
    int* flag;
};

// D += (A sa) (B sb) with 4-bit operands of 64 values, scales per 32; `id` names the scale bytes in use.
__device__ __forceinline__ void tc_mma_mxf4_if(uint32_t one, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sa, uint32_t sb,
                                               uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate), "r"(one)
        : "memory");
}
// A tile of scales (512 bytes) from shared memory to four TMEM columns of every lane quadrant.
__device__ __forceinline__ void tc_cp_scales_if(uint32_t one, uint32_t tmem, uint64_t desc) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
        "@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(tmem), "l"(desc), "r"(one)
        : "memory");
}
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {   // no swizzle, 8 rows of 16 bytes after one another
    return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(128 >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
}
// Instruction descriptor, kind::mxf4: e2m1 operands, scales 2^e, fp32 sums; scale bytes `sf` and sf + 1.
__host__ __device__ constexpr uint32_t idesc_mxf4(int M, int N, int sf) {
    return (static_cast<uint32_t>(sf) << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) |
           (static_cast<uint32_t>(M >> 4) << 24) | (static_cast<uint32_t>(sf) << 29);
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// 32 tokens of one weight, N elements apart, `left` of them in the matrix: the residual, and the sums v finished and stored.
// (Whether there are GELU and residual is decided once for all 32: a branch for each keeps their chains of instructions
// from running next to one another, and took 8192 x 28672 x 4096 with GELU from 323 to 352 us.)
template <typename T>
__device__ __forceinline__ void load_32(const T* R, int64_t N, int left, T (&r)[32]) {
#pragma unroll
    for (int e = 0; e < 32; ++e) r[e] = e < left ? __ldcs(R + e * N) : from_f32<T>(0.0f);
}
template <typename T, bool GELU, bool ADD>
__device__ __forceinline__ void finish_pairs(T* y, int64_t N, int left, const float (&v)[32], float bias, const T (&r)[32]) {
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
        float2 x = __fadd2_rn(make_float2(v[e], v[e + 1]), f2(bias));
        if constexpr (GELU) x = gelu_erf2(x);
        if constexpr (ADD) x = __fadd2_rn(x, make_float2(to_f32(r[e]), to_f32(r[e + 1])));
        if (e < left) y[e * N] = from_f32<T>(x.x);
        if (e + 1 < left) y[(e + 1) * N] = from_f32<T>(x.y);
    }
}
template <typename T>
__device__ __forceinline__ void finish_32(T* y, int64_t N, int left, bool gelu, const float (&v)[32], float bias, const T (&r)[32], bool add) {
    if (gelu) {
        if (add) finish_pairs<T, true, true>(y, N, left, v, bias, r);
        else finish_pairs<T, true, false>(y, N, left, v, bias, r);
    } else {
        if (add) finish_pairs<T, false, true>(y, N, left, v, bias, r);
        else finish_pairs<T, false, false>(y, N, left, v, bias, r);
    }
}

// CTA `part` of the SPLIT that share a tile finishes every SPLIT-th of its tokens: a warp takes a token at a time, a lane four
// weights.  The parts are summed in order; sixteen reads of other CTAs' shared memory are on their way together (one token
// at a time, 200 tokens of 4096 x 4096 over two CTAs took 9.0 us, 2.2 more than unsplit).
template <typename T, int SPLIT>
__device__ __forceinline__ void join_tokens(const GemmArgs& a, uint32_t base, int m0, int n0, int part, int tokens, int warp, int lane) {
    constexpr int AHEAD = 16 / SPLIT;
    const int n = n0 + 4 * lane, wide = a.N - n;      // weights of this lane within the matrix, if below 4
    float bias[4] = {};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (a.bias && e < wide) bias[e] = to_f32(static_cast<const T*>(a.bias)[n + e]);
    uint32_t at[SPLIT];
#pragma unroll
    for (int p = 0; p < SPLIT; ++p) at[p] = mapa_shared(base + 16 * lane, p);
    const bool whole = a.N % 4 == 0 && (reinterpret_cast<uintptr_t>(a.y) & 7) == 0;
    for (int c0 = part + SPLIT * warp; c0 < tokens; c0 += 4 * SPLIT * AHEAD) {
        float x[AHEAD][SPLIT][4];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int c = min(c0 + 4 * SPLIT * i, tokens - 1);
#pragma unroll
            for (int p = 0; p < SPLIT; ++p)
                asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(x[i][p][0]), "=f"(x[i][p][1]), "=f"(x[i][p][2]), "=f"(x[i][p][3])
                             : "r"(at[p] + c * 512)
                             : "memory");
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int c = c0 + 4 * SPLIT * i;
            if (c >= tokens) break;
            const int64_t to = static_cast<int64_t>(m0 + c) * a.N + n;
            T* y = static_cast<T*>(a.y) + to;
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] = x[i][0][e];
#pragma unroll
                for (int p = 1; p < SPLIT; ++p) v[e] += x[i][p][e];
            }
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                float2 z = make_float2(v[e] + bias[e], v[e + 1] + bias[e + 1]);
                if (a.gelu) z = gelu_erf2(z);
                v[e] = z.x;
                v[e + 1] = z.y;
            }
            if (a.R)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (e < wide) v[e] += to_f32(static_cast<const T*>(a.R)[to + e]);
            if (whole) {
                if (wide > 0) *reinterpret_cast<uint2*>(y) = make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]));
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (e < wide) y[e] = from_f32<T>(v[e]);
            }
        }
    }
}

template <typename T, int NT>
__global__ void __launch_bounds__(kGemmThreads, NT <= 64 ? 2 : 1) mxfp4_gemm_kernel(const __grid_constant__ CUtensorMap mW,
                                                                                   const __grid_constant__ CUtensorMap mX,
                                                                                   const __grid_constant__ GemmArgs a) {
    using L = GemmLayout<NT>;
    constexpr int ST = L::STAGES;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - smem_addr(smem_raw));
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    auto full = [&](int i) { return base + L::OFF_BAR + 8u * i; };
    auto empty = [&](int i) { return base + L::OFF_BAR + 8u * (ST + i); };
    const uint32_t done = base + L::OFF_BAR + 8u * (2 * ST), drain = done + 8;
    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        mbar_init(done, 1);
        mbar_init(drain, 1);
        fence_mbar_init();
    }
    const uint32_t tmem = tmem_begin(base + L::OFF_HOLD, gbase + L::OFF_HOLD, L::TMEM_COLS, warp);
    const int split = a.split, part = static_cast<int>(blockIdx.x) % split, n_tile = static_cast<int>(blockIdx.x) / split;
    const int n0 = n_tile * 128, m0 = static_cast<int>(blockIdx.y) * NT;
    const int s0 = static_cast<int>(static_cast<int64_t>(a.stages) * part / split), s1 = static_cast<int>(static_cast<int64_t>(a.stages) * (part + 1) / split);
    // The first weights on their way into L2 while the kernel before (mostly the quantisation of X) runs out: 100 tokens of
    // 4096 x 14336 10.65 -> 10.25 us, 14.15 -> 13.4 with that kernel (in a stream of equal calls); more than the first six stages
    // gain less.
    if (warp == 0 && blockIdx.y == 0 && lane < 6 && s0 + lane < s1) {
        const int s = s0 + lane;
        tma_prefetch_2d(&mW, s * 64, n0);
        prefetch_l2_bulk(a.ws + static_cast<int64_t>(n_tile) * a.xtk * 512 + s * 1024, 512u * static_cast<uint32_t>(min(2, a.xtk - 2 * s)));
    }
    pdl_wait();

    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity & 1u, a.flag));
        return ok;
    };
    if (warp == 0) {
        if (lane == 0) {
            prefetch_map(&mW);
            prefetch_map(&mX);
        }
        const uint32_t one = elect_one();
        const uint8_t* sw = a.ws + static_cast<int64_t>(n_tile) * a.xtk * 512;
        const uint8_t* sx = a.xs + static_cast<int64_t>(m0 / 128) * a.xtk * 512;
        int i = 0;
        for (int s = s0; s < s1; ++s, ++i) {
            const int slot = i % ST;
            if (i >= ST && !wait(empty(slot), i / ST - 1)) break;
            const uint32_t at = base + slot * L::STAGE, bytes = 512u * static_cast<uint32_t>(min(2, a.xtk - 2 * s));
            if (lane == 0) mbar_arrive_expect_tx(full(slot), kTileBytes + L::B_BYTES + 2 * bytes);
            __syncwarp();
            tma_load_2d_if(one, at, &mW, s * 64, n0, full(slot));
            tma_load_2d_if(one, at + L::OFF_B, &mX, s * 64, m0, full(slot));
            if (one) {
                bulk_load(at + L::OFF_SA, sw + s * 1024, bytes, full(slot));
                bulk_load(at + L::OFF_SB, sx + s * 1024, bytes, full(slot));
            }
            __syncwarp();
        }
        if (!ok)   // copies in flight land before the shared memory goes away
            for (int j = max(0, i - ST); j < i; ++j) (void)mbar_wait_drain(full(j % ST), (j / ST) & 1);
    } else if (warp == 1) {
        const uint32_t one = elect_one();
        bool issued = false;
        int i = 0;
        for (int s = s0; s < s1; ++s, ++i) {
            const int slot = i % ST;
            if (!wait(full(slot), i / ST)) break;
            tc_fence_after();
            const uint32_t at = base + slot * L::STAGE;
            const int left = a.K - s * kStageK, steps = min(4, (left + 63) / 64);
#pragma unroll
            for (int t = 0; t < 2; ++t)
                if (2 * t < steps) {
                    tc_cp_scales_if(one, tmem + L::SFA_COL + 4 * t, scale_desc(at + L::OFF_SA + 512 * t));
                    tc_cp_scales_if(one, tmem + L::SFB_COL + 4 * t, scale_desc(at + L::OFF_SB + 512 * t));
                }
            const uint64_t da = smem_desc_sw128(at, 16, 1024), db = smem_desc_sw128(at + L::OFF_B, 16, 1024);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k < steps)
                    tc_mma_mxf4_if(one, tmem, da + 2 * k, db + 2 * k, k % 2 ? idesc_mxf4(128, NT, 2) : idesc_mxf4(128, NT, 0),
                                   tmem + L::SFA_COL + 4 * (k / 2), tmem + L::SFB_COL + 4 * (k / 2), i > 0 || k > 0 ? 1u : 0u);
            tc_commit_if(one, empty(slot));
            issued = true;
        }
        if (ok && issued) tc_commit_if(one, done);
        if (!ok && issued) {
            tc_commit_if(one, drain);
            (void)mbar_wait_drain(drain, 0);
        }
        __syncwarp();
    } else {
        const int quad = warp % 4, row = 32 * quad + lane, n = n0 + row;
        const bool in = n < a.N;
        const float bias = in && a.bias ? to_f32(static_cast<const T*>(a.bias)[n]) : 0.0f;
        const int tokens = min(NT, a.M - m0);
        float* part_sums = reinterpret_cast<float*>(gbase);          // [token][128], over the stages
        if (wait(done, 0)) {
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < tokens; c += 32) {
                float v[32] = {};      // (not read: without the zeros the compiler's order takes 100 tokens of 4096 x 14336 from 18.6 to 20.7 us)
                T r[32];
                const int64_t at = static_cast<int64_t>(m0 + c) * a.N + n;
                const int left = in ? tokens - c : 0;
                if (a.R && split == 1) load_32<T>(static_cast<const T*>(a.R) + at, a.N, left, r);
                tmem_ld32(tmem + (static_cast<uint32_t>(32 * quad) << 16) + c, v);
                tmem_ld_wait();
                if (split > 1) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) part_sums[(c + e) * 128 + row] = v[e];
                } else {
                    finish_32<T>(static_cast<T*>(a.y) + at, a.N, left, a.gelu != 0, v, bias, r, a.R != nullptr);
                }
            }
            tc_fence_before();
        }
    }
    if (split > 1) {
        // each CTA finishes its share of the tile's tokens, summing the parts in order
        cluster_sync();
        if (warp >= 2 && ok) {
            if (split == 2) join_tokens<T, 2>(a, base, m0, n0, part, min(NT, a.M - m0), warp - 2, lane);
            else if (split == 4) join_tokens<T, 4>(a, base, m0, n0, part, min(NT, a.M - m0), warp - 2, lane);
            else join_tokens<T, 8>(a, base, m0, n0, part, min(NT, a.M - m0), warp - 2, lane);
        }
        cluster_sync();
    } else {
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, L::TMEM_COLS);
    }
}

// ------------------------------------------------------------------ many tokens: CTA pairs
// Persistent clusters of two CTAs: M = 256 weights by N = 256 tokens (cta_group::2), each CTA holding its 128 weights, half of
// the tokens and, of the scales, its weights' and all tokens'.  Two accumulators of 256 columns and 24 columns of scales do
// not fit TMEM's 512, so the accumulators share 24 columns, which the epilogue reads first: the next tile's products
// start as soon as those are read, and run while the rest is finished and stored.
// 4096 x 4096 x 14336 70.8 us (6.8 PFLOP/s); 8192 x 28672 x 4096 with bias and GELU 323 us (6.0), of which the products are 240 and
// the change from one accumulator to the other 0.6 us a tile.  Stages, 4, 5 and 6, in us: that 324, 328 and 331, without GELU 311,
// 304 and 300, with a residual 385, 390 and 403, 4096 x 14336 x 4096 116, 110 and 120.
struct PairLayout {
    static constexpr int STAGES = 5;
    static constexpr uint32_t OFF_B = kTileBytes, OFF_SA = OFF_B + kTileBytes, OFF_SB = OFF_SA + 1024;
    static constexpr uint32_t STAGE = OFF_SB + 2048;
    static constexpr uint32_t OFF_BAR = STAGES * STAGE;
    static constexpr uint32_t OFF_HOLD = OFF_BAR + (2 * STAGES + 6) * 8;
    static constexpr uint32_t SMEM = OFF_HOLD + 16 + 1024;
    static constexpr uint32_t ACC1 = 232, SFA_COL = 488, SFB_COL = 496;    // accumulators at 0 and 232
    static_assert(STAGE % 1024 == 0, "swizzle atoms");
    static_assert(SMEM <= 232448, "shared-memory budget");
};
constexpr int kPairEpiWarps = 16;                      // four per TMEM lane quadrant
constexpr int kPairThreads = 32 * (4 + kPairEpiWarps); // warp 0: loads, 1: MMA issue, 4-19: epilogue
// Registers of a thread: 96 at the launch, then 40 and 104 (128 (40 + 4 x 104) = 58368 of the launch's 640 x 96 = 61440).
constexpr int kBand = 32;                              // token tiles of a band: 8192 tokens' values stay in L2

__device__ __forceinline__ void tc_mma_mxf4_pair_if(uint32_t one, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sa,
                                                    uint32_t sb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate), "r"(one)
        : "memory");
}
// (in each CTA of the pair from its own shared memory to its own TMEM)
__device__ __forceinline__ void tc_cp_scales_pair_if(uint32_t one, uint32_t tmem, uint64_t desc) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
        "@q tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(tmem), "l"(desc), "r"(one)
        : "memory");
}

struct PairArgs {
    GemmArgs g;
    int tiles_m, tiles_n;         // of 256 tokens, of 256 weights
};
// Tile t: bands of token tiles, weight by weight within a band.
__device__ __forceinline__ void tile_of(const PairArgs& a, int t, int& m0, int& n0) {
    const int per = kBand * a.tiles_n, band = t / per, first = band * kBand, wide = min(kBand, a.tiles_m - first), i = t - band * per;
    m0 = (first + i % wide) * 256;
    n0 = (i / wide) * 256;
}

template <typename T>
__global__ void __launch_bounds__(kPairThreads, 1) mxfp4_pair_kernel(const __grid_constant__ CUtensorMap mW, const __grid_constant__ CUtensorMap mX,
                                                                     const __grid_constant__ CUtensorMap mSW, const __grid_constant__ CUtensorMap mSX,
                                                                     const __grid_constant__ PairArgs a) {
    using L = PairLayout;
    constexpr int ST = L::STAGES;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - smem_addr(smem_raw));
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    auto full = [&](int i) { return base + L::OFF_BAR + 8u * i; };
    auto empty = [&](int i) { return base + L::OFF_BAR + 8u * (ST + i); };
    auto acc_full = [&](int i) { return base + L::OFF_BAR + 8u * (2 * ST + i); };
    auto acc_done = [&](int i) { return base + L::OFF_BAR + 8u * (2 * ST + 2 + i); };
    const uint32_t acc_read = base + L::OFF_BAR + 8u * (2 * ST + 4), drain = acc_read + 8;
    const uint32_t rank = cluster_rank();
    const int cid = static_cast<int>(blockIdx.x) / 2, clusters = static_cast<int>(gridDim.x) / 2;
    const int tiles = a.tiles_m * a.tiles_n, nk = a.g.stages;
    int* flag = a.g.flag;
    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        for (int i = 0; i < 2; ++i) mbar_init(acc_full(i), 1);
        for (int i = 0; i < 2; ++i) mbar_init(acc_done(i), 2 * kPairEpiWarps);
        mbar_init(acc_read, 2 * 4);
        mbar_init(drain, 1);
        fence_mbar_init();
    }
    const uint32_t tmem = tmem_begin_pair(base + L::OFF_HOLD, gbase + L::OFF_HOLD, 512, warp);
    pdl_wait();

    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity & 1u, flag));
        return ok;
    };
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 0) {
            // ---------------------------------------------------------------- loads; both CTAs' bytes count on the even one's barrier
            if (lane == 0) {
                prefetch_map(&mW);
                prefetch_map(&mX);
                prefetch_map(&mSW);
                prefetch_map(&mSX);
            }
            const uint32_t one = elect_one();
            int c = 0;
            for (int t = cid; ok && t < tiles; t += clusters) {
                int m0, n0;
                tile_of(a, t, m0, n0);
                for (int s = 0; s < nk; ++s, ++c) {
                    const int slot = c % ST;
                    if (c >= ST && !wait(empty(slot), c / ST - 1)) break;
                    if (rank == 0 && lane == 0) mbar_arrive_expect_tx(full(slot), 2 * L::STAGE);
                    __syncwarp();
                    const uint32_t at = base + slot * L::STAGE, bar = mapa_shared(full(slot), 0);
                    tma_load_2d_pair_if(one, at, &mW, s * 64, n0 + static_cast<int>(rank) * 128, bar);
                    tma_load_2d_pair_if(one, at + L::OFF_B, &mX, s * 64, m0 + static_cast<int>(rank) * 128, bar);
                    tma_load_3d_pair_if(one, at + L::OFF_SA, &mSW, s * 256, n0 / 128 + static_cast<int>(rank), 0, bar);
                    tma_load_3d_pair_if(one, at + L::OFF_SB, &mSX, s * 256, m0 / 128, 0, bar);
                }
            }
            if (!ok && rank == 0)   // both CTAs' copies in flight land before either's shared memory goes away
                for (int j = max(0, c - ST); j < c; ++j) (void)mbar_wait_drain(full(j % ST), (j / ST) & 1);
        } else if (warp == 1 && rank == 0) {
            // ---------------------------------------------------------------- MMA issue, for both CTAs
            const uint32_t one = elect_one();
            const int mine = tiles > cid ? (tiles - 1 - cid) / clusters + 1 : 0, total = mine * nk;
            int c = 0;
            for (int i = 0; ok && i < mine; ++i) {
                // this accumulator has been read (two tiles ago), and the columns that it shares with the other one
                if (i > 1 && !wait(acc_done(i % 2), i / 2 - 1)) break;
                if (i > 0 && !wait(acc_read, i - 1)) break;
                tc_fence_after();
                const uint32_t d = tmem + (i % 2 ? L::ACC1 : 0);
                for (int s = 0; s < nk; ++s, ++c) {
                    const int slot = c % ST;
                    if (!wait(full(slot), c / ST)) break;
                    tc_fence_after();
                    const uint32_t at = base + slot * L::STAGE;
                    const int steps = min(4, (a.g.K - s * kStageK + 63) / 64);
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        if (2 * t < steps) {
                            tc_cp_scales_pair_if(one, tmem + L::SFA_COL + 4 * t, scale_desc(at + L::OFF_SA + 512 * t));
                            tc_cp_scales_pair_if(one, tmem + L::SFB_COL + 8 * t, scale_desc(at + L::OFF_SB + 512 * t));
                            tc_cp_scales_pair_if(one, tmem + L::SFB_COL + 8 * t + 4, scale_desc(at + L::OFF_SB + 1024 + 512 * t));
                        }
                    const uint64_t da = smem_desc_sw128(at, 16, 1024), db = smem_desc_sw128(at + L::OFF_B, 16, 1024);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k < steps)
                            tc_mma_mxf4_pair_if(one, d, da + 2 * k, db + 2 * k, k % 2 ? idesc_mxf4(256, 256, 2) : idesc_mxf4(256, 256, 0),
                                                tmem + L::SFA_COL + 4 * (k / 2), tmem + L::SFB_COL + 8 * (k / 2), s > 0 || k > 0 ? 1u : 0u);
                    // frees the stage in both CTAs, unless no later load uses it
                    if (c + ST < total) tc_commit_pair_mc_if(one, empty(slot), 0x3);
                }
                if (ok) tc_commit_pair_mc_if(one, acc_full(i % 2), 0x3);
            }
            if (!ok && c > 0) {     // MMAs in flight finish before TMEM is freed
                if (one) tc_commit_pair(drain);
                __syncwarp();
                (void)mbar_wait_drain(drain, 0);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
        // ---------------------------------------------------------------- epilogue: 32 weights by 64 tokens of a tile
        // in two chunks, the one with the shared columns (tokens 232..255 of accumulator 0, 0..23 of 1) first.  The first
        // chunk's residual is on its way while the tile's products run.
        const int q = warp % 4, h = (warp - 4) / 4;
        const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
        const bool add = a.g.R != nullptr;
        for (int t = cid, i = 0; t < tiles; t += clusters, ++i) {
            int m0, n0;
            tile_of(a, t, m0, n0);
            const int b = i % 2, n = n0 + static_cast<int>(rank) * 128 + 32 * q + lane;
            const bool in = n < a.g.N;
            const float bias = in && a.g.bias ? to_f32(static_cast<const T*>(a.g.bias)[n]) : 0.0f;
            auto token = [&](int x) { return 64 * h + 32 * (b ? x : 1 - x); };
            auto at = [&](int x) { return static_cast<int64_t>(m0 + token(x)) * a.g.N + n; };
            auto left = [&](int x) { return in ? a.g.M - m0 - token(x) : 0; };
            T r[32];
            if (add) load_32<T>(static_cast<const T*>(a.g.R) + at(0), a.g.N, left(0), r);
            if (!wait(acc_full(b), i / 2)) break;
            tc_fence_after();
#pragma unroll 1
            for (int x = 0; x < 2; ++x) {
                float v[32];
                tmem_ld32(tmem + lanes + (b ? L::ACC1 : 0) + token(x), v);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (x == 0 && h == (b ? 0 : 3)) mbar_arrive_cluster(mapa_shared(acc_read, 0));
                    if (x == 1) mbar_arrive_cluster(mapa_shared(acc_done(b), 0));
                }
                if (x == 1 && add) load_32<T>(static_cast<const T*>(a.g.R) + at(1), a.g.N, left(1), r);
                finish_32<T>(static_cast<T*>(a.g.y) + at(x), a.g.N, left(x), a.g.gelu != 0, v, bias, r, add);
            }
        }
    }
    tc_fence_before();
    cluster_sync();  // neither CTA leaves while its peer may still signal it
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// A quantised matrix as rows of 16-bit elements (four values each), boxes of 128 bytes.
bool map_codes(CUtensorMap* map, const void* q, int64_t rows, int64_t K, int box_rows) { return make_map(map, q, rows, K / 4, 64, box_rows); }
// Its scale tiles: a row of tiles as 32-bit elements, boxes of two tiles' 1024 bytes.
bool map_scales(CUtensorMap* map, const void* s, int64_t rows, int64_t K, int box_rows) {
    const int64_t row = ceil_div(K, 128) * 512, n = ceil_div(rows, 128);
    const int64_t dims[3] = {row / 4, n, 1}, strides[2] = {row, row};
    const int box[3] = {256, box_rows, 1};
    return make_map_3d(map, s, kMap32, dims, strides, box, 0);
}

// Pairs that can be resident at once (both CTAs of one in one cluster of SMs).
int pairs() {
    static std::mutex mu;
    static int cached[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        (void)cudaGetLastError();
        return 1;
    }
    std::lock_guard<std::mutex> lock(mu);
    if (cached[dev] == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * static_cast<unsigned>(sm_count()));
        cfg.blockDim = dim3(kPairThreads);
        cfg.dynamicSmemBytes = PairLayout::SMEM;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = 2;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        int n = 0;
        if (opt_in_smem((const void*)mxfp4_pair_kernel<__half>, PairLayout::SMEM) != FUSE_OK ||
            cudaOccupancyMaxActiveClusters(&n, mxfp4_pair_kernel<__half>, &cfg) != cudaSuccess || n < 1) {
            (void)cudaGetLastError();
            n = sm_count() / 2;
        }
        cached[dev] = n > 0 ? n : 1;
    }
    return cached[dev];
}

template <typename T>
int launch_pair(const GemmArgs& g, const void* xq, const void* wq, cudaStream_t st) {
    CUtensorMap mW, mX, mSW, mSX;
    if (!map_codes(&mW, wq, g.N, g.K, 128) || !map_codes(&mX, xq, g.M, g.K, 128) || !map_scales(&mSW, g.ws, g.N, g.K, 1) ||
        !map_scales(&mSX, g.xs, g.M, g.K, 2))
        return FUSE_ECUDA;
    const int rc = opt_in_smem((const void*)mxfp4_pair_kernel<T>, PairLayout::SMEM);
    if (rc != FUSE_OK) return rc;
    const PairArgs a{g, static_cast<int>(ceil_div(g.M, 256)), static_cast<int>(ceil_div(g.N, 256))};
    const int64_t tiles = static_cast<int64_t>(a.tiles_m) * a.tiles_n;
    const int n = pairs();
    return launch_pdl(mxfp4_pair_kernel<T>, dim3(2 * static_cast<unsigned>(tiles < n ? tiles : n)), dim3(kPairThreads), PairLayout::SMEM, st, 2, mW, mX,
                      mSW, mSX, a);
}

template <typename T, int NT>
int launch_gemm(GemmArgs a, const void* xq, const void* wq, cudaStream_t st) {
    CUtensorMap mW, mX;
    if (!map_codes(&mW, wq, a.N, a.K, 128) || !map_codes(&mX, xq, a.M, a.K, NT)) return FUSE_ECUDA;
    const int rc = opt_in_smem((const void*)mxfp4_gemm_kernel<T, NT>, GemmLayout<NT>::SMEM);
    if (rc != FUSE_OK) return rc;
    const int64_t tn = ceil_div(a.N, 128), tm = ceil_div(a.M, NT);
    // K over up to eight CTAs while all of them are resident at once (two per SM up to 64 tokens) and each has two stages, so that none
    // is without.  Over two only from 24 stages on: joining them takes what 12 stages do (4096 weights, K = 4096, 16 stages, which lie
    // in L2: one token 4.2 us over eight, 4.6 over four, 5.7 unsplit, but 200 tokens 7.7 over two and 6.8 unsplit; K = 14336: 256 tokens
    // 12.7 over two, 15.1 unsplit).
    const int64_t room = sm_count() * (NT <= 64 ? 2 : 1);
    a.split = 1;
    while (a.split < 8 && tn * tm * a.split * 2 <= room && a.stages >= 2 * a.split * 2) a.split *= 2;
    if (a.split == 2 && a.stages < 24) a.split = 1;
    return launch_pdl(mxfp4_gemm_kernel<T, NT>, dim3(static_cast<unsigned>(tn * a.split), static_cast<unsigned>(tm)), dim3(kGemmThreads),
                      GemmLayout<NT>::SMEM, st, a.split, mW, mX, a);
}

// Tiles by the number of tokens, pairs of CTAs where their tiles are as many as half of those that can be resident.  In us, weights
// from HBM, K = 4096; tiles of 32, 64 and 128 tokens: one token of 4096 weights 4.4, 4.9 and 4.3, 32 of 14336 7.5, 8.0 and 7.5, 64 of
// 4096 -, 6.7 and 5.7, of 14336 -, 8.4 and 7.7, of 28672 -, 11.9 and 15.5.  128 tokens and pairs: 512 of 4096 6.6 and 9.4, 1024 of 4096
// 12.8 and 9.9, 256 of 14336 13.8 and 10.7, 128 of 28672 16.4 and 16.5; where pairs' tiles are half empty or few the rule takes the
// slower side, 128 of 14336 8.0 and 10.2, 256 of 9728 7.3 and 9.9.
template <typename T>
int run_gemm(const GemmArgs& a, const void* xq, const void* wq, cudaStream_t st) {
    if (a.M <= 32) return launch_gemm<T, 32>(a, xq, wq, st);
    if (a.M <= 64) return launch_gemm<T, 64>(a, xq, wq, st);
    if (ceil_div(a.M, 256) * ceil_div(a.N, 256) >= pairs() / 2) return launch_pair<T>(a, xq, wq, st);
    return launch_gemm<T, 128>(a, xq, wq, st);
}

int64_t scale_bytes(int64_t rows, int64_t cols) { return ceil_div(rows, 128) * ceil_div(cols, 128) * 512; }

// The rules on a quantised matrix that both directions share.
int check_matrix(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 1) return FUSE_EINVAL;
    if (cols % 32 != 0 || cols >= int64_t(1) << 31 || rows >= int64_t(1) << 22) return FUSE_EUNSUPPORTED;
    return FUSE_OK;
}

}  // namespace

int mxfp4_report_count() { return 14; }
int mxfp4_report(int i, fuse_kernel_record* out) {
    switch (i) {
        FC_REPORT(0, kQThreads, 0, 0, mxfp4_quantize_kernel<float>);
        FC_REPORT(1, kQThreads, 0, 0, mxfp4_quantize_kernel<__half>);
        FC_REPORT(2, kQThreads, 0, 0, mxfp4_quantize_kernel<__nv_bfloat16>);
        FC_REPORT(3, kQThreads, 0, 0, mxfp4_dequantize_kernel<float>);
        FC_REPORT(4, kQThreads, 0, 0, mxfp4_dequantize_kernel<__half>);
        FC_REPORT(5, kQThreads, 0, 0, mxfp4_dequantize_kernel<__nv_bfloat16>);
        FC_REPORT(6, kGemmThreads, GemmLayout<32>::SMEM, GemmLayout<32>::TMEM_COLS, mxfp4_gemm_kernel<__half, 32>);
        FC_REPORT(7, kGemmThreads, GemmLayout<64>::SMEM, GemmLayout<64>::TMEM_COLS, mxfp4_gemm_kernel<__half, 64>);
        FC_REPORT(8, kGemmThreads, GemmLayout<128>::SMEM, GemmLayout<128>::TMEM_COLS, mxfp4_gemm_kernel<__half, 128>);
        FC_REPORT(9, kGemmThreads, GemmLayout<32>::SMEM, GemmLayout<32>::TMEM_COLS, mxfp4_gemm_kernel<__nv_bfloat16, 32>);
        FC_REPORT(10, kGemmThreads, GemmLayout<64>::SMEM, GemmLayout<64>::TMEM_COLS, mxfp4_gemm_kernel<__nv_bfloat16, 64>);
        FC_REPORT(11, kGemmThreads, GemmLayout<128>::SMEM, GemmLayout<128>::TMEM_COLS, mxfp4_gemm_kernel<__nv_bfloat16, 128>);
        FC_REPORT(12, kPairThreads, PairLayout::SMEM, 512, mxfp4_pair_kernel<__half>);
        FC_REPORT(13, kPairThreads, PairLayout::SMEM, 512, mxfp4_pair_kernel<__nv_bfloat16>);
        default: return FUSE_EINVAL;
    }
}

}  // namespace fc

extern "C" int64_t fuse_mxfp4_scale_bytes(int64_t rows, int64_t cols) {
    const int rc = fc::check_matrix(rows, cols);
    return rc != FUSE_OK ? rc : fc::scale_bytes(rows, cols);
}

extern "C" int fuse_mxfp4_quantize(const void* x, int64_t ld, void* q, void* scales, int64_t rows, int64_t cols, int dtype, fuse_stream_t stream) {
    using namespace fc;
    int rc = check_matrix(rows, cols);
    if (rc != FUSE_OK) return rc;
    if (ld < cols || (dtype != FUSE_F32 && dtype != FUSE_F16 && dtype != FUSE_BF16)) return FUSE_EINVAL;
    if (ld >= int64_t(1) << 40) return FUSE_EUNSUPPORTED;
    if (rows == 0) return FUSE_OK;
    if (!x || !q || !scales) return FUSE_EINVAL;
    const int64_t size = dtype == FUSE_F32 ? 4 : 2;
    if (!is_aligned(x, 32) || ld * size % 32 != 0 || !is_aligned(q, 16) || !is_aligned(scales, 16)) return FUSE_EALIGN;
    const int64_t xb = ((rows - 1) * ld + cols) * size, qb = rows * cols / 2, sb = scale_bytes(rows, cols);
    if (ranges_overlap(x, xb, q, qb) || ranges_overlap(x, xb, scales, sb) || ranges_overlap(q, qb, scales, sb)) return FUSE_EINVAL;
    const QuantArgs a{x, ld, static_cast<uint8_t*>(q), static_cast<uint8_t*>(scales), rows, cols};
    const dim3 grid(static_cast<unsigned>(ceil_div(cols, 128)), static_cast<unsigned>(ceil_div(rows, 128)));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == FUSE_F32) return launch_pdl(mxfp4_quantize_kernel<float>, grid, dim3(kQThreads), 0, st, 1, a);
    if (dtype == FUSE_F16) return launch_pdl(mxfp4_quantize_kernel<__half>, grid, dim3(kQThreads), 0, st, 1, a);
    return launch_pdl(mxfp4_quantize_kernel<__nv_bfloat16>, grid, dim3(kQThreads), 0, st, 1, a);
}

extern "C" int fuse_mxfp4_dequantize(const void* q, const void* scales, void* y, int64_t rows, int64_t cols, int dtype, fuse_stream_t stream) {
    using namespace fc;
    int rc = check_matrix(rows, cols);
    if (rc != FUSE_OK) return rc;
    if (dtype != FUSE_F32 && dtype != FUSE_F16 && dtype != FUSE_BF16) return FUSE_EINVAL;
    if (rows == 0) return FUSE_OK;
    if (!y || !q || !scales) return FUSE_EINVAL;
    if (!is_aligned(y, 32) || !is_aligned(q, 16) || !is_aligned(scales, 16)) return FUSE_EALIGN;
    const int64_t yb = rows * cols * (dtype == FUSE_F32 ? 4 : 2), qb = rows * cols / 2, sb = scale_bytes(rows, cols);
    if (ranges_overlap(y, yb, q, qb) || ranges_overlap(y, yb, scales, sb)) return FUSE_EINVAL;
    const QuantArgs a{nullptr, 0, const_cast<uint8_t*>(static_cast<const uint8_t*>(q)), const_cast<uint8_t*>(static_cast<const uint8_t*>(scales)), rows, cols};
    const dim3 grid(static_cast<unsigned>(ceil_div(cols, 128)), static_cast<unsigned>(ceil_div(rows, 128)));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == FUSE_F32) return launch_pdl(mxfp4_dequantize_kernel<float>, grid, dim3(kQThreads), 0, st, 1, a, static_cast<float*>(y));
    if (dtype == FUSE_F16) return launch_pdl(mxfp4_dequantize_kernel<__half>, grid, dim3(kQThreads), 0, st, 1, a, static_cast<__half*>(y));
    return launch_pdl(mxfp4_dequantize_kernel<__nv_bfloat16>, grid, dim3(kQThreads), 0, st, 1, a, static_cast<__nv_bfloat16*>(y));
}

extern "C" int fuse_mxfp4_gemm(const void* xq, const void* xs, const void* wq, const void* ws, const void* bias, const void* R, void* y, int64_t M,
                               int64_t N, int64_t K, int gelu, int dtype, fuse_stream_t stream) {
    using namespace fc;
    int rc = check_matrix(M, K);
    if (rc == FUSE_OK) rc = check_matrix(N, K);
    if (rc != FUSE_OK) return rc;
    if (N < 1 || (gelu != 0 && gelu != 1) || (dtype != FUSE_F16 && dtype != FUSE_BF16)) return FUSE_EINVAL;
    if (K >= kMostK || ceil_div(M, 256) * ceil_div(N, 256) >= (int64_t(1) << 30) / ceil_div(K, kStageK)) return FUSE_EUNSUPPORTED;   // stages are counted in 32 bits
    if (M == 0) return FUSE_OK;
    if (!xq || !xs || !wq || !ws || !y) return FUSE_EINVAL;
    if (!is_aligned(xq, 16) || !is_aligned(xs, 16) || !is_aligned(wq, 16) || !is_aligned(ws, 16) || !is_aligned(y, 2) || !is_aligned(bias, 2) ||
        !is_aligned(R, 2))
        return FUSE_EALIGN;
    const int64_t yb = M * N * 2;
    struct { const void* p; int64_t n; } in[6] = {{xq, M * K / 2}, {xs, scale_bytes(M, K)}, {wq, N * K / 2}, {ws, scale_bytes(N, K)}, {bias, N * 2}, {R, yb}};
    for (const auto& x : in)
        if (x.p && ranges_overlap(y, yb, x.p, x.n)) return FUSE_EINVAL;
    GemmArgs a{};
    a.xs = static_cast<const uint8_t*>(xs);
    a.ws = static_cast<const uint8_t*>(ws);
    a.bias = bias;
    a.R = R;
    a.y = y;
    a.M = static_cast<int>(M);
    a.N = static_cast<int>(N);
    a.K = static_cast<int>(K);
    a.xtk = static_cast<int>(ceil_div(K, 128));
    a.stages = static_cast<int>(ceil_div(K, kStageK));
    a.gelu = gelu;
    a.flag = watchdog_flag();
    if (!a.flag) return FUSE_ECUDA;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return dtype == FUSE_F16 ? run_gemm<__half>(a, xq, wq, st) : run_gemm<__nv_bfloat16>(a, xq, wq, st);
}

extern "C" int64_t fuse_mxfp4_gemm_bytes(int64_t M, int64_t N, int64_t K, int bias, int residual) {
    if (M < 0 || N < 1 || K < 32 || K % 32 != 0) return FUSE_EINVAL;
    return (M + N) * (K / 2 + K / 32) + 2 * M * N * (residual ? 2 : 1) + (bias ? 2 * N : 0);
}
