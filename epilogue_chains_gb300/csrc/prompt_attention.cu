// prompt_attention.cu -- causal attention of packed prompts over a paged key/value cache.
//
//     o_ih = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m),   s_j = scale q_ih . k_j,   j <= keys - queries + i,
// for query i of a sequence's new tokens: its keys, old and new, are in the cache, and the new tokens are the
// last of them.  Scores are kept in base-2 units; a part of a row's keys gives (m, l, O) = (reference, sum of
// 2^(s - m), sum of 2^(s - m) v), and parts join as m = max m_i, l = sum 2^(m_i - m) l_i and O likewise.
//
// It is bound by the tensor cores: 4 D operations per query head and visible key.  An item is one key/value
// head and the query rows of its group of heads for some consecutive tokens, token by token, so a tile of 128
// rows spans few tokens where heads are grouped (less of the diagonal is computed in vain) and single tokens
// still fill rows with their group.  With D <= 128 an item has two tiles of 128 rows against the same K and V
// tiles, so that one tile's softmax runs while the tensor core works for the other.
//
// Work is dealt out in equal runs: all items of the batch lie in one line, each counting for its visible keys
// and an entry, and every CTA takes an equal run of it, whatever the lengths are.  What one CTA has of an item
// that several share goes through the workspace, and prompt_join_kernel joins it in the order of the keys.  The
// lengths are in device memory, so one launch configuration (and a captured graph) serves every batch.  All
// waits are bounded (watchdog).
#include <cudaTypedefs.h>
#include <math.h>

#include <type_traits>

#include "fc_internal.cuh"
#include "fc_mma.cuh"
#include "fc_ptx.cuh"
#include "fc_tc.cuh"

namespace fc {
namespace {

constexpr int kMaxBatch = 4096;
constexpr int kGrid = 160;                 // most CTAs (workspace bound)
// A running reference is replaced when a row's maximum exceeds it by more than 2^8, so weights stay
// within [0, 2^8]; for fp16 weights it is also set 2^7 below the maximum, which uses fp16's range
// upwards (2^15 at most) and keeps weights down to 2^-21 of the maximum at full precision.
constexpr float kLag = 8.0f;
template <typename T> struct Shift { static constexpr float V = 0.0f; };
template <> struct Shift<__half> { static constexpr float V = 7.0f; };
// What an item counts for apart from its keys, in keys: its entry and its output.
constexpr int kEntry = 192;
// A CTA's run is at least this many keys: shorter runs cost more to join than they save.
constexpr int kLeastRun = 512 + kEntry;

__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3f(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// A whole 32-byte sector per thread.
__device__ __forceinline__ void st_v8(float* p, const float* v) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])),
                 "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
                 "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
                 : "memory");
}

struct PromptArgs {
    const int32_t *table, *cu, *lens;
    int64_t table_ld;
    void* o;
    int batch, tokens, hq, hk, group;
    int tpt, tiles;                    // tokens of a tile of 128 rows; tiles of an item (1 or 2)
    int page_shift, num_pages, cache_rows;
    float c;                           // scale * log2(e)
    // workspace: where each CTA's run begins, and the parts of items that CTAs share: of CTA c slot 2 c has the part of
    // an item that began in an earlier CTA, slot 2 c + 1 that of one which begins here and goes on in a later one
    int4* start;                       // [kGrid + 1]
    float2* ml;                        // [2 kGrid][rows]
    float* po;                         // [2 kGrid][rows][D]
    int rows;
    int *flag, *bad;
};

// ================================================================== the line of items
struct Seq {
    int q0, n, L;      // first row and number of the new tokens; keys
};
// Sequence b, taken into range (`bad`: report what is out of range).
__device__ __forceinline__ Seq seq_of(const PromptArgs& a, int b, int* bad = nullptr) {
    const int c0 = a.cu[b], c1 = a.cu[b + 1], len = a.lens[b];
    Seq s;
    s.q0 = min(max(c0, 0), a.tokens);
    s.n = max(min(max(c1, 0), a.tokens) - s.q0, 0);
    const int64_t room = a.table_ld << a.page_shift;
    s.L = static_cast<int>(min(static_cast<int64_t>(max(len, 0)), room));
    if (bad && (c0 < 0 || c1 > a.tokens || c1 < c0 || len < 0 || len > room)) atomicExch(bad, 1);
    return s;
}
__device__ __forceinline__ int items_of(const PromptArgs& a, const Seq& s) {
    const int ti = a.tpt * a.tiles;
    return (s.n + ti - 1) / ti;
}
// Keys that the first `tokens` new tokens of a sequence see between them.
__device__ __forceinline__ int extent(const Seq& s, int tokens) { return max(s.L - s.n + min(tokens, s.n), 0); }
// Places of a head's first k items: sum over i < k of kEntry + extent((i + 1) ti).
__device__ __forceinline__ int64_t places(const PromptArgs& a, const Seq& s, int items, int k) {
    const int64_t ti = a.tpt * a.tiles, d = s.L - s.n;
    int64_t sum = static_cast<int64_t>(k) * kEntry;
    if (k == items && k > 0) {
        sum += extent(s, s.n);
        --k;
    }
    const int64_t i0 = d >= 0 ? 0 : -d / ti;          // the first item with d + (i + 1) ti > 0
    if (k > i0) sum += (k - i0) * d + ti * ((static_cast<int64_t>(k) * (k + 1) - i0 * (i0 + 1)) / 2);
    return sum;
}

// A place in the line: sequence, key/value head, item, 128-key block.
struct Pos {
    int b, h, i, t;
    __device__ __forceinline__ bool before(const Pos& o) const {
        if (b != o.b) return b < o.b;
        if (h != o.h) return h < o.h;
        if (i != o.i) return i < o.i;
        return t < o.t;
    }
};

// Place r of sequence b; within `snap` blocks of an item's end, that end.
__device__ __forceinline__ Pos pos_in(const PromptArgs& a, const Seq& s, int b, int64_t r, int snap) {
    const int items = items_of(a, s);
    const int64_t per = places(a, s, items, items);
    Pos p;
    p.b = b;
    p.h = static_cast<int>(r / per);
    r -= p.h * per;
    int lo = 0, hi = items - 1;                        // the last item that begins at or before r
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (places(a, s, items, mid) <= r) lo = mid;
        else hi = mid - 1;
    }
    const int64_t in = r - places(a, s, items, lo);
    const int blocks = (extent(s, (lo + 1) * a.tpt * a.tiles) + 127) / 128;
    p.i = lo;
    p.t = in <= kEntry ? 0 : static_cast<int>((in - kEntry) / 128);
    if (p.t <= snap) {
        p.t = 0;
    } else if (blocks - p.t <= snap) {
        p.i = lo + 1;
        p.t = 0;
    }
    return p;
}

// What a CTA does of one item: blocks t0 .. t1 - 1, of which tile 0 sees the first n0 and tile 1 the first n1.
struct Seg {
    int b, h, tok0;        // sequence, key/value head, first new token
    int q0, n, L;
    int t0, blocks, n0, n1;
    bool whole;
    __device__ __forceinline__ int steps() const { return max(n0, n1); }
};
// The walk along a run.
struct Walk {
    Pos p, end;
    Seq s;
    int items;
    __device__ __forceinline__ void begin(const PromptArgs& a, const Pos& from, const Pos& to) {
        p = from;
        end = to;
        items = 0;
        s = Seq{0, 0, 0};
        if (p.b < a.batch) load(a);
        settle(a);
    }
    __device__ __forceinline__ void load(const PromptArgs& a) {
        s = seq_of(a, p.b);
        items = items_of(a, s);
    }
    // To an item that exists.
    __device__ __forceinline__ void settle(const PromptArgs& a) {
        while (p.b < a.batch && p.i >= items) {
            p.i = 0;
            if (items == 0 || ++p.h == a.hk) {
                p.h = 0;
                if (++p.b < a.batch) load(a);
            }
        }
    }
    __device__ __forceinline__ bool next(const PromptArgs& a, Seg& g) {
        while (p.before(end)) {
            const int tok0 = p.i * a.tpt * a.tiles;
            const int b0 = (extent(s, tok0 + a.tpt) + 127) / 128;
            const int b1 = a.tiles == 2 && tok0 + a.tpt < s.n ? (extent(s, tok0 + 2 * a.tpt) + 127) / 128 : 0;
            g.blocks = max(b0, b1);
            const bool cut = p.b == end.b && p.h == end.h && p.i == end.i;
            const int t1 = cut ? min(end.t, g.blocks) : g.blocks;
            g.b = p.b;
            g.h = p.h;
            g.tok0 = tok0;
            g.q0 = s.q0;
            g.n = s.n;
            g.L = s.L;
            g.t0 = p.t;
            g.n0 = max(min(b0, t1) - p.t, 0);
            g.n1 = max(min(b1, t1) - p.t, 0);
            g.whole = p.t == 0 && t1 == g.blocks;
            p.t = 0;
            ++p.i;
            settle(a);
            if (g.n0 > 0 || g.n1 > 0 || g.whole) return true;
        }
        return false;
    }
};
// A softmax warp's walk and segment are in shared memory: kept in registers, next to a row's 128 scores, they spill.
struct WarpWalk {
    Walk walk;
    Seg seg;
};

// Where run `which` (0: this CTA's, 1: the next's) begins, for all threads; `scratch` is 64 * 8 bytes of shared memory.
template <int THREADS>
__device__ __forceinline__ void find_runs(const PromptArgs& a, int64_t* scratch, Pos (&run)[2]) {
    constexpr int WARPS = THREADS / 32;
    static_assert(WARPS <= 32, "scratch");
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int per = (a.batch + THREADS - 1) / THREADS;
    int64_t mine = 0;
    for (int i = 0; i < per; ++i) {
        const int b = tid * per + i;
        if (b >= a.batch) break;
        const Seq s = seq_of(a, b, blockIdx.x == 0 ? a.bad : nullptr);
        const int items = items_of(a, s);
        mine += a.hk * places(a, s, items, items);
    }
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    Pos* found = reinterpret_cast<Pos*>(scratch + 32);
    if (lane == 31) scratch[warp] = upto;
    if (tid < 2) found[tid] = Pos{a.batch, 0, 0, 0};
    __syncthreads();
    int64_t total = 0;
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) upto += scratch[w];
        total += scratch[w];
    }
    int64_t len = (total + gridDim.x - 1) / gridDim.x;
    if (len < kLeastRun) len = kLeastRun;
    const int snap = static_cast<int>(min(len / (128 * 32), static_cast<int64_t>(64)));
    for (int w = 0; w < 2; ++w) {
        const int64_t x = static_cast<int64_t>(blockIdx.x + w) * len;
        if (x >= upto || x < upto - mine) continue;
        int64_t at = upto - mine;                      // this thread's sequences have it
        for (int i = 0; i < per; ++i) {
            const int b = tid * per + i;
            if (b >= a.batch) break;
            const Seq s = seq_of(a, b);
            const int items = items_of(a, s);
            const int64_t here = a.hk * places(a, s, items, items);
            if (x < at + here) {
                found[w] = pos_in(a, s, b, x - at, snap);
                break;
            }
            at += here;
        }
    }
    __syncthreads();
    run[0] = found[0];
    run[1] = found[1];
}

// ================================================================== the kernel
constexpr int kSoftWarps = 8;                       // four per tile (one tile: the first four)
constexpr int kThreads = 32 * (4 + kSoftWarps);     // warp 0: Q, K, V loads, 1: S, 2: PV, 4-11: softmax
// Registers of a thread: 168 at the launch, then 96 for the first four warps and 200 for the softmax's, whose rows'
// 128 scores are in registers (128 (96 + 2 x 200) = 63488 of the launch's 384 x 168 = 64512).
constexpr int kFewRegs = 96, kManyRegs = 200;
constexpr int kFull = 4;                            // barriers of K tiles in turn, and of V tiles

template <int D>
struct Layout {
    static constexpr int TILES = D <= 128 ? 2 : 1;
    static constexpr int RING = D == 64 ? 6 : D == 128 ? 3 : 2;    // K and V tiles
    static constexpr uint32_t REGION = 128 * 128;              // one 64-column atom of 128 rows
    static constexpr uint32_t TILE = REGION * (D / 64);
    static constexpr uint32_t P_BYTES = 128 * 128 * 2;
    static constexpr uint32_t OFF_Q = 0;
    static constexpr uint32_t OFF_KV = TILES * TILE;
    static constexpr uint32_t OFF_P = OFF_KV + RING * TILE;
    static constexpr uint32_t OFF_BAR = OFF_P + TILES * P_BYTES;
    static constexpr int N_BARS = 2 + 2 * kFull + RING + 8 + 2;
    static constexpr uint32_t OFF_HOLD = OFF_BAR + N_BARS * 8;
    static constexpr uint32_t OFF_SCRATCH = (OFF_HOLD + 16 + 7) / 8 * 8;
    static constexpr uint32_t OFF_WALK = OFF_SCRATCH + 64 * 8;
    static constexpr uint32_t SMEM = OFF_WALK + 4 * TILES * sizeof(WarpWalk) + 1024;
    static constexpr uint32_t TMEM_COLS = 512, O_COL = 256;    // scores of tile t at 128 t, output at 256 + D t
    static_assert(SMEM <= 232448, "shared-memory budget");
    static_assert(SMEM > 116 * 1024, "one CTA per SM: each takes all of TMEM");
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1) prompt_attention_kernel(const __grid_constant__ CUtensorMap mQ,
                                                                       const __grid_constant__ CUtensorMap mK,
                                                                       const __grid_constant__ CUtensorMap mV,
                                                                       const __grid_constant__ PromptArgs a) {
    using L = Layout<D>;
    constexpr bool BF = std::is_same<T, __nv_bfloat16>::value;
    constexpr int RING = L::RING, TILES = L::TILES;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - smem_addr(smem_raw));
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    const uint32_t bar0 = base + L::OFF_BAR;
    const uint32_t q_full = bar0, q_free = bar0 + 8;
    auto k_full = [&](int i) { return bar0 + 8u * (2 + i); };
    auto v_full = [&](int i) { return bar0 + 8u * (2 + kFull + i); };
    auto empty = [&](int i) { return bar0 + 8u * (2 + 2 * kFull + i); };
    constexpr int X = 2 + 2 * kFull + RING;
    auto s_full = [&](int t) { return bar0 + 8u * (X + t); };
    auto s_free = [&](int t) { return bar0 + 8u * (X + 2 + t); };
    auto p_full = [&](int t) { return bar0 + 8u * (X + 4 + t); };
    auto o_done = [&](int t) { return bar0 + 8u * (X + 6 + t); };
    auto drain = [&](int w) { return bar0 + 8u * (X + 8 + w); };       // of warps 1 and 2
    int* flag = a.flag;
    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_free, 1);
        for (int i = 0; i < kFull; ++i) {
            mbar_init(k_full(i), 1);
            mbar_init(v_full(i), 1);
        }
        for (int i = 0; i < RING; ++i) mbar_init(empty(i), 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(s_full(t), 1);
            mbar_init(s_free(t), 4);
            mbar_init(p_full(t), 4);
            mbar_init(o_done(t), 1);
            mbar_init(drain(t), 1);
        }
        fence_mbar_init();
    }
    const uint32_t tmem = tmem_begin(base + L::OFF_HOLD, gbase + L::OFF_HOLD, L::TMEM_COLS, warp);
    pdl_wait();

    Pos run[2];
    find_runs<kThreads>(a, reinterpret_cast<int64_t*>(gbase + L::OFF_SCRATCH), run);
    if (threadIdx.x == 0) {
        a.start[blockIdx.x] = make_int4(run[0].b, run[0].h, run[0].i, run[0].t);
        if (blockIdx.x + 1 == gridDim.x) a.start[gridDim.x] = make_int4(run[1].b, run[1].h, run[1].i, run[1].t);
    }
    // Steps of an item: K(0), then K(j + 1) before V(j), through one ring.
    auto k_at = [](int j) { return j == 0 ? 0 : 2 * j - 1; };
    auto v_at = [](int j, int n) { return j + 1 < n ? 2 * j + 2 : 2 * j + 1; };
    Walk walk;
    walk.begin(a, run[0], run[1]);

    if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
    if (warp == 0) {
        // ---------------------------------------------------------------- Q, K and V loads
        if (lane == 0) {
            prefetch_map(&mQ);
            prefetch_map(&mK);
            prefetch_map(&mV);
        }
        const uint32_t one = elect_one();
        const int box_shift = min(a.page_shift, 7);
        const uint32_t q_box = static_cast<uint32_t>(a.group * a.tpt) * 128u;
        int c = 0, slot = 0, kc = 0, vc = 0, segs = 0;    // loads, the next one's slot, K and V tiles, items
        uint32_t phase = 1;
        bool ok = true;
        auto wait = [&](uint32_t bar, uint32_t parity) {
            ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity & 1u, flag));
            return ok;
        };
        Seg g;
        while (ok && walk.next(a, g)) {
            const int n = g.steps();
            if (n == 0) continue;
            if (segs > 0 && !wait(q_free, segs - 1)) break;
            const int tiles = g.n1 > 0 ? TILES : 1;
            if (lane == 0) mbar_arrive_expect_tx(q_full, tiles * (D / 64) * q_box);
            __syncwarp();
            for (int t = 0; t < tiles; ++t)
#pragma unroll
                for (int x = 0; x < D / 64; ++x)
                    tma_load_3d_if(one, base + L::OFF_Q + t * L::TILE + x * L::REGION, &mQ, 64 * x, g.h * a.group, g.q0 + g.tok0 + t * a.tpt, q_full);
            ++segs;
            const int32_t* table = a.table + static_cast<int64_t>(g.b) * a.table_ld;
            for (int x = 0; x < 2 * n; ++x, ++c) {
                // x-th load of the item: K for 0 and odd x below 2 n - 1, V for the others
                const bool is_k = x == 0 || (x % 2 == 1 && x < 2 * n - 1);
                const int j = is_k ? (x + 1) / 2 : (x == 2 * n - 1 ? n - 1 : x / 2 - 1);
                const int key0 = (g.t0 + j) * 128, nk = min(128, g.L - key0), nbox = (nk + (1 << box_shift) - 1) >> box_shift;
                const int key = key0 + (lane << box_shift);
                int row = a.cache_rows;         // past the cache: zeros
                if (lane < nbox) {
                    const int page = table[key >> a.page_shift];
                    if (page >= 0 && page < a.num_pages)
                        row = ((page * a.hk + g.h) << a.page_shift) + (key & ((1 << a.page_shift) - 1));
                    else
                        atomicExch(a.bad, 1);
                }
                if (c >= RING && !wait(empty(slot), phase)) break;
                const uint32_t full = is_k ? k_full(kc++ % kFull) : v_full(vc++ % kFull);
                const uint32_t dst = base + L::OFF_KV + slot * L::TILE;
                if (lane == 0) mbar_arrive_expect_tx(full, static_cast<uint32_t>(nbox << box_shift) * (D * 2));
                __syncwarp();
                for (int y = 0; y < nbox; ++y) {
                    const int r = __shfl_sync(0xffffffffu, row, y);
#pragma unroll
                    for (int e = 0; e < D / 64; ++e)
                        tma_load_2d_if(one, dst + e * L::REGION + ((static_cast<uint32_t>(y) << box_shift) * 128), is_k ? &mK : &mV, 64 * e, r, full);
                }
                if (++slot == RING) {
                    slot = 0;
                    phase ^= 1u;
                }
            }
        }
        if (!ok) {   // copies in flight land before the shared memory goes away
            if (segs > 0) (void)mbar_wait_drain(q_full, (segs - 1) & 1);
            for (int i = max(0, kc - kFull); i < kc; ++i) (void)mbar_wait_drain(k_full(i % kFull), (i / kFull) & 1);
            for (int i = max(0, vc - kFull); i < vc; ++i) (void)mbar_wait_drain(v_full(i % kFull), (i / kFull) & 1);
        }
        __syncwarp();
    } else if (warp == 1 || warp == 2) {
        // ---------------------------------------------------------------- MMA issue: S by warp 1, PV by warp 2
        const uint32_t one = elect_one();
        bool issued = false, ok = true;
        auto wait = [&](uint32_t bar, uint32_t parity) {
            ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity & 1u, flag));
            return ok;
        };
        int c = 0, kv = 0, segs = 0;      // loads and K (or V) tiles of the items before this one; items
        int i[2] = {0, 0};                // products of each tile so far
        Seg g;
        if (warp == 1) {
            constexpr uint32_t idS = idesc_f16(128, 128, false, false, BF);
            const uint64_t dq = smem_desc_sw128(base + L::OFF_Q, 16, 1024), dk = smem_desc_sw128(base + L::OFF_KV, 16, 1024);
            while (ok && walk.next(a, g)) {
                const int n = g.steps();
                if (n == 0) continue;
                if (!wait(q_full, segs)) break;
                for (int j = 0; ok && j < n; ++j) {
                    const int slot = (c + k_at(j)) % RING;
                    const uint64_t kd = dk + static_cast<uint64_t>(slot * (L::TILE >> 4));
                    if (!wait(k_full((kv + j) % kFull), (kv + j) / kFull)) break;
#pragma unroll
                    for (int t = 0; t < TILES; ++t) {
                        if (j >= (t == 0 ? g.n0 : g.n1)) continue;
                        if (i[t] > 0 && !wait(s_free(t), i[t] - 1)) break;
                        ++i[t];
                        tc_fence_after();
                        const uint64_t qd = dq + static_cast<uint64_t>(t * (L::TILE >> 4));
#pragma unroll
                        for (int s = 0; s < D / 16; ++s)
                            tc_mma_if(one, tmem + t * 128, qd + ((s / 4) * (L::REGION >> 4) + (s % 4) * 2),
                                      kd + ((s / 4) * (L::REGION >> 4) + (s % 4) * 2), idS, s > 0 ? 1u : 0u);
                        tc_commit_if(one, s_full(t));
                        issued = true;
                    }
                    if (ok) tc_commit_if(one, empty(slot));
                }
                if (ok) tc_commit_if(one, q_free);
                ++segs;
                kv += n;
                c += 2 * n;
            }
        } else {
            constexpr uint32_t idO = idesc_f16(128, D, false, true, BF);
            const uint64_t dp = smem_desc_sw128(base + L::OFF_P, 16, 1024), dv = smem_desc_sw128(base + L::OFF_KV, L::REGION, 1024);
            while (ok && walk.next(a, g)) {
                const int n = g.steps();
                for (int j = 0; ok && j < n; ++j) {
                    const int slot = (c + v_at(j, n)) % RING;
                    const uint64_t vd = dv + static_cast<uint64_t>(slot * (L::TILE >> 4));
                    if (!wait(v_full((kv + j) % kFull), (kv + j) / kFull)) break;
#pragma unroll
                    for (int t = 0; t < TILES; ++t) {
                        if (j >= (t == 0 ? g.n0 : g.n1)) continue;
                        if (!wait(p_full(t), i[t])) break;
                        ++i[t];
                        tc_fence_after();
                        const uint64_t pd = dp + static_cast<uint64_t>(t * (L::P_BYTES >> 4));
#pragma unroll
                        for (int s = 0; s < 8; ++s)   // 16 keys each
                            tc_mma_if(one, tmem + L::O_COL + t * D, pd + ((s / 4) * (L::REGION >> 4) + (s % 4) * 2), vd + s * (2048 >> 4), idO,
                                      j > 0 || s > 0 ? 1u : 0u);
                        tc_commit_if(one, o_done(t));
                        issued = true;
                    }
                    if (ok) tc_commit_if(one, empty(slot));
                }
                kv += n;
                c += 2 * n;
            }
        }
        if (!ok && issued) {   // MMAs in flight finish before TMEM is freed
            tc_commit_if(one, drain(warp - 1));
            (void)mbar_wait_drain(drain(warp - 1), 0);
        }
        __syncwarp();
    }
    } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
    if (warp < 4 + 4 * TILES) {
        // ---------------------------------------------------------------- softmax: thread r of tile t, one row
        const int t = (warp - 4) / 4, r = 32 * (warp % 4) + lane;
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp % 4)) << 16;
        const uint32_t st = tmem + lanes + t * 128, ot = tmem + lanes + L::O_COL + t * D;
        constexpr float SH = Shift<T>::V;
        bool ok = true;
        auto wait = [&](uint32_t bar, uint32_t parity) {
            ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity & 1u, flag));
            return ok;
        };
        int i = 0, c = 0, kv = 0;
        WarpWalk& w = *reinterpret_cast<WarpWalk*>(gbase + L::OFF_WALK + (warp - 4) * sizeof(WarpWalk));
        const Seg& g = w.seg;
        if (lane == 0) w.walk = walk;
        auto next = [&]() {
            bool more = false;
            if (lane == 0) {
                Walk mine = w.walk;
                Seg s;
                more = mine.next(a, s);
                w.walk = mine;
                w.seg = s;
            }
            return __shfl_sync(0xffffffffu, more, 0) != 0;
        };
        while (ok && next()) {
            __syncwarp();
            const int n = t == 0 ? g.n0 : g.n1;
            int left, kleft;         // keys from the block on: those that this row sees, those of the sequence
            {
                const int rt = r / a.group;
                kleft = g.L - g.t0 * 128;
                left = kleft - g.n + g.tok0 + t * a.tpt + rt + 1;
            }
            float m = -INFINITY, l = 0.0f;
            for (int j = 0; j < n; ++j, ++i, left -= 128, kleft -= 128) {
                if (!wait(s_full(t), i)) break;
                tc_fence_after();
                float x[128];
#pragma unroll
                for (int k = 0; k < 4; ++k) tmem_ld32(st + 32 * k, x + 32 * k);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_free(t));
                if (__any_sync(0xffffffffu, left < 128)) {
#pragma unroll
                    for (int k = 0; k < 128; ++k) x[k] = k >= left ? -INFINITY : x[k];
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int k = 0; k < 128; k += 2) mx[(k >> 1) & 3] = max3f(mx[(k >> 1) & 3], x[k], x[k + 1]);
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.c;
                float alpha = 1.0f;
                bool rescale = false;
                if (top > m + (SH + kLag)) {
                    if (j > 0) {
                        alpha = ex2f(m - (top - SH));
                        rescale = true;
                    }
                    m = top - SH;
                }
                // P and O are free once the previous PV has completed
                if (i > 0 && !wait(o_done(t), i - 1)) break;
                const float ref = m == -INFINITY ? 0.0f : m;
                const float2 c2 = make_float2(a.c, a.c), nm2 = make_float2(-ref, -ref);
                float2 sum2 = make_float2(0.0f, 0.0f);
                uint8_t* prow = gbase + L::OFF_P + t * L::P_BYTES + r * 128;
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    // The weights rounded to T, as the tensor core takes both operands of a product in one type.  Each is
                    // off by at most half a step of T, as the output's own rounding is.
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 e = __ffma2_rn(make_float2(x[8 * q + 2 * k], x[8 * q + 2 * k + 1]), c2, nm2);
                        const float2 p = make_float2(ex2f(e.x), ex2f(e.y));
                        sum2 = __fadd2_rn(sum2, p);
                        w[k] = pack2<T>(p.x, p.y);
                    }
                    *reinterpret_cast<uint4*>(prow + (q / 8) * L::REGION + (((q % 8) ^ (r & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
                l = l * alpha + (sum2.x + sum2.y);
                if (__any_sync(0xffffffffu, rescale)) {
                    tc_fence_after();
#pragma unroll 1
                    for (int k = 0; k < D / 32; ++k) {
                        float o[32];
                        tmem_ld32(ot + 32 * k, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= alpha;
                        tmem_st32(ot + 32 * k, o);
                    }
                    tmem_st_wait();
                }
                // V rows past the sequence's end: 0 x whatever lies there must be 0.  By the tile whose product with this
                // block is issued first.
                if (kleft < 128 && (t == 0 || j >= g.n0)) {
                    const int vi = kv + j;
                    if (!wait(v_full(vi % kFull), vi / kFull)) break;
                    uint8_t* vb = gbase + L::OFF_KV + ((c + v_at(j, g.steps())) % RING) * L::TILE;
                    for (int v = r; v < (128 - kleft) * (D / 8); v += 128) {
                        const int row = kleft + v / (D / 8), ch = v % (D / 8);
                        *reinterpret_cast<uint4*>(vb + (ch / 8) * L::REGION + row * 128 + (ch % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                fence_async_smem();      // the generic-proxy writes become visible to the tensor core
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full(t));
            }
            c += 2 * g.steps();
            kv += g.steps();
            if (!ok || (n > 0 && !wait(o_done(t), i - 1))) break;
            tc_fence_after();
            const int rt = r / a.group, head = r - rt * a.group, tok = g.tok0 + t * a.tpt + rt;
            const bool in = rt < a.tpt && tok < g.n;
            if (g.whole) {
                const float inv = l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l;
                T* dst = static_cast<T*>(a.o) + (static_cast<int64_t>(g.q0 + tok) * a.hq + g.h * a.group + head) * D;
#pragma unroll 1
                for (int k = 0; k < D / 32; ++k) {
                    float o[32];
                    uint32_t w[16];
                    if (n > 0) {
                        tmem_ld32(ot + 32 * k, o);
                        tmem_ld_wait();
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) w[e] = n == 0 || l == 0.0f ? 0u : pack2<T>(o[2 * e] * inv, o[2 * e + 1] * inv);
                    if (in) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            *reinterpret_cast<uint4*>(dst + 32 * k + 8 * e) = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
                    }
                }
            } else {
                const int64_t at = static_cast<int64_t>(2 * blockIdx.x + (g.t0 == 0 ? 1 : 0)) * a.rows + t * 128 + r;
                if (in) a.ml[at] = make_float2(m, l);
                float* dst = a.po + at * D;
                if (n > 0)
#pragma unroll 1
                    for (int k = 0; k < D / 32; ++k) {
                        float o[32];
                        tmem_ld32(ot + 32 * k, o);
                        tmem_ld_wait();
                        if (in)
#pragma unroll
                            for (int e = 0; e < 4; ++e) st_v8(dst + 32 * k + 8 * e, o + 8 * e);
                    }
            }
            tc_fence_before();
            __syncwarp();
        }
    }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, L::TMEM_COLS);
    }
}

// ================================================================== join
// The parts of an item that several CTAs share, one warp per row; blockIdx.y names the CTA whose run begins first within
// the item.  Lane c takes D / 32 columns.
constexpr int kJoinThreads = 128;
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) prompt_join_kernel(const __grid_constant__ PromptArgs a, int grid) {
    constexpr int W = D / 32;
    pdl_begin();
    const int c0 = blockIdx.y + 1;                 // run c0 begins within an item
    auto start = [&](int c) {
        const int4 v = __ldcg(a.start + c);
        return Pos{v.x, v.y, v.z, v.w};
    };
    auto same = [](const Pos& x, const Pos& y) { return x.b == y.b && x.h == y.h && x.i == y.i; };
    const Pos p = start(c0);
    if (p.t == 0 || p.b >= a.batch) return;
    const Pos q = start(c0 - 1);
    if (same(p, q) && q.t > 0) return;             // not the first
    const int row = blockIdx.x * (kJoinThreads / 32) + threadIdx.x / 32, lane = threadIdx.x % 32;
    const Seq s = seq_of(a, p.b);
    const int r = row % 128, rt = r / a.group, tok = (p.i * a.tiles + row / 128) * a.tpt + rt;
    if (row >= a.rows || rt >= a.tpt || tok >= s.n) return;
    float m = -INFINITY, l = 0.0f, acc[W] = {};
    // part 0 is CTA c0 - 1's; then that of each run that begins within the item and has something of it
    Pos at = p;
    for (int c = c0 - 1;; ++c) {
        bool has = true;
        if (c >= c0) {
            const Pos next = start(c + 1);
            has = at.before(next);
            at = next;
        }
        if (has) {
            const int64_t slot = static_cast<int64_t>(2 * c + (c < c0 ? 1 : 0)) * a.rows + row;
            const float2 x = __ldcg(a.ml + slot);
            if (x.x > -INFINITY || x.y != 0.0f) {        // (a part that this row sees nothing of has no output)
                const float nm = fmaxf(m, x.x), e0 = m == -INFINITY ? 0.0f : ex2f(m - nm), e1 = ex2f(x.x - nm);
                const float* src = a.po + slot * D + W * lane;
                l = l * e0 + x.y * e1;
#pragma unroll
                for (int e = 0; e < W; e += 2) {
                    const float2 v = __ldcg(reinterpret_cast<const float2*>(src + e));
                    acc[e] = acc[e] * e0 + v.x * e1;
                    acc[e + 1] = acc[e + 1] * e0 + v.y * e1;
                }
                m = nm;
            }
        }
        if (c >= c0 && !(same(at, p) && at.t > 0)) break;
        if (c + 1 >= grid) break;
    }
    const float inv = l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l;
    T* dst = static_cast<T*>(a.o) + (static_cast<int64_t>(s.q0 + tok) * a.hq + p.h * a.group + r % a.group) * D + W * lane;
#pragma unroll
    for (int e = 0; e < W; e += 2)
        *reinterpret_cast<uint32_t*>(dst + e) = l == 0.0f ? 0u : pack2<T>(acc[e] * inv, acc[e + 1] * inv);
}

// ================================================================== host side
struct Sizes {
    int64_t rows;
    size_t ml, po, bytes;
};
Sizes sizes(int64_t tokens, int64_t hq, int64_t hk, int64_t D) {
    Sizes s{};
    const int64_t group = hq / hk, tpt = 128 / group, tiles = D <= 128 ? 2 : 1;
    s.rows = tokens <= tpt ? tokens * group : tiles * 128;
    size_t at = (kGrid + 1) * sizeof(int4);
    auto part = [&](int64_t n) {
        at = (at + 255) / 256 * 256;
        const size_t was = at;
        at += static_cast<size_t>(n);
        return was;
    };
    s.ml = part(2 * kGrid * s.rows * 8);
    s.po = part(2 * kGrid * s.rows * D * 4);
    s.bytes = (at + 255) / 256 * 256;
    return s;
}

template <typename T, int D>
int run_prompt(PromptArgs a, const void* q, int64_t q_ld, const void* k, const void* v, cudaStream_t st) {
    using L = Layout<D>;
    const bool bf = std::is_same<T, __nv_bfloat16>::value;
    const int box = 1 << (a.page_shift < 7 ? a.page_shift : 7);
    CUtensorMap mQ, mK, mV;
    const int64_t dims[3] = {D, a.hq, a.tokens}, strides[2] = {D * 2, q_ld * 2};
    const int qbox[3] = {64, a.group, a.tpt};
    if (!make_map(&mK, k, a.cache_rows, D, 64, box, bf) || !make_map(&mV, v, a.cache_rows, D, 64, box, bf) ||
        !make_map_3d(&mQ, q, kMap16, dims, strides, qbox, 128))
        return FUSE_ECUDA;
    int rc = opt_in_smem((const void*)prompt_attention_kernel<T, D>, L::SMEM);
    if (rc != FUSE_OK) return rc;
    // no more CTAs than there can be runs
    const int64_t ti = static_cast<int64_t>(a.tpt) * a.tiles, room = a.table_ld << a.page_shift;
    const int64_t items = (ceil_div(a.tokens, ti) + (a.batch < a.tokens ? a.batch : a.tokens)) * a.hk;
    int64_t grid = sm_count() < kGrid ? sm_count() : kGrid;
    const int64_t runs = items * ceil_div(room + kEntry, kLeastRun);
    if (grid > runs) grid = runs;
    rc = launch_pdl(prompt_attention_kernel<T, D>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), L::SMEM, st, 1, mQ, mK, mV, a);
    // an item of at most one block of keys is nobody's to share
    if (rc != FUSE_OK || grid == 1 || room <= 128) return rc;
    return launch_pdl(prompt_join_kernel<T, D>, dim3(static_cast<unsigned>(ceil_div(a.rows, kJoinThreads / 32)), static_cast<unsigned>(grid - 1)),
                      dim3(kJoinThreads), 0, st, 1, a, static_cast<int>(grid));
}

}  // namespace

int prompt_report_count() { return 12; }
int prompt_report(int i, fuse_kernel_record* out) {
    switch (i) {
        FC_REPORT(0, kThreads, Layout<64>::SMEM, 512, prompt_attention_kernel<__nv_bfloat16, 64>);
        FC_REPORT(1, kThreads, Layout<128>::SMEM, 512, prompt_attention_kernel<__nv_bfloat16, 128>);
        FC_REPORT(2, kThreads, Layout<256>::SMEM, 512, prompt_attention_kernel<__nv_bfloat16, 256>);
        FC_REPORT(3, kThreads, Layout<64>::SMEM, 512, prompt_attention_kernel<__half, 64>);
        FC_REPORT(4, kThreads, Layout<128>::SMEM, 512, prompt_attention_kernel<__half, 128>);
        FC_REPORT(5, kThreads, Layout<256>::SMEM, 512, prompt_attention_kernel<__half, 256>);
        FC_REPORT(6, kJoinThreads, 0, 0, prompt_join_kernel<__nv_bfloat16, 64>);
        FC_REPORT(7, kJoinThreads, 0, 0, prompt_join_kernel<__nv_bfloat16, 128>);
        FC_REPORT(8, kJoinThreads, 0, 0, prompt_join_kernel<__nv_bfloat16, 256>);
        FC_REPORT(9, kJoinThreads, 0, 0, prompt_join_kernel<__half, 64>);
        FC_REPORT(10, kJoinThreads, 0, 0, prompt_join_kernel<__half, 128>);
        FC_REPORT(11, kJoinThreads, 0, 0, prompt_join_kernel<__half, 256>);
        default: return FUSE_EINVAL;
    }
}

}  // namespace fc

extern "C" size_t fuse_prompt_attention_workspace_bytes(int64_t tokens, int64_t q_heads, int64_t kv_heads, int64_t D) {
    if (tokens < 1 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0 || q_heads / kv_heads > 128 || D < 1) return 0;
    return fc::sizes(tokens, q_heads, kv_heads, D).bytes;
}

extern "C" int fuse_prompt_attention(const void* q, int64_t q_ld, const void* k_cache, const void* v_cache, const int32_t* block_table,
                                     int64_t table_ld, const int32_t* cu_queries, const int32_t* seq_lens, void* o, int64_t tokens,
                                     int64_t batch, int64_t q_heads, int64_t kv_heads, int64_t D, int64_t num_pages, int64_t page_size,
                                     float scale, int dtype, void* workspace, size_t ws_bytes, fuse_stream_t stream) {
    using namespace fc;
    if (tokens < 0 || batch < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0 || D < 1 || num_pages < 1 || page_size < 1 ||
        table_ld < 0 || !(scale > 0.0f) || !isfinite(scale))
        return FUSE_EINVAL;
    if (dtype != FUSE_F16 && dtype != FUSE_BF16) return FUSE_EINVAL;
    if (D != 64 && D != 128 && D != 256) return FUSE_EUNSUPPORTED;
    if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)) != 0) return FUSE_EUNSUPPORTED;
    const int64_t top = int64_t(1) << 31, group = q_heads / kv_heads;
    if (group > 128 || batch > kMaxBatch || q_heads > 65536 || tokens >= int64_t(1) << 24 || num_pages >= top / (kv_heads * page_size) ||
        table_ld >= (top - 4096) / page_size || q_ld >= int64_t(1) << 32)
        return FUSE_EUNSUPPORTED;
    // the line's places, times the CTAs, stay within 64 bits
    if ((tokens + batch) * kv_heads >= (int64_t(1) << 52) / (table_ld * page_size + kEntry)) return FUSE_EUNSUPPORTED;
    if (q_ld < q_heads * D) return FUSE_EINVAL;
    if (tokens == 0 || batch == 0) return FUSE_OK;
    if (!q || !k_cache || !v_cache || !o || !cu_queries || !seq_lens || (table_ld > 0 && !block_table)) return FUSE_EINVAL;
    if (!is_aligned(q, 16) || q_ld % 8 != 0 || !is_aligned(k_cache, 16) || !is_aligned(v_cache, 16) || !is_aligned(o, 16) ||
        !is_aligned(block_table, 4) || !is_aligned(cu_queries, 4) || !is_aligned(seq_lens, 4))
        return FUSE_EALIGN;
    const Sizes s = sizes(tokens, q_heads, kv_heads, D);
    if (!workspace || ws_bytes < s.bytes) return FUSE_EWORKSPACE;
    if (!is_aligned(workspace, 256)) return FUSE_EALIGN;
    const int64_t qb = ((tokens - 1) * q_ld + q_heads * D) * 2, ob = tokens * q_heads * D * 2, cb = num_pages * kv_heads * page_size * D * 2;
    struct { const void* p; int64_t n; } in[6] = {{q, qb}, {k_cache, cb}, {v_cache, cb}, {table_ld > 0 ? block_table : nullptr, batch * table_ld * 4},
                                                 {cu_queries, (batch + 1) * 4}, {seq_lens, batch * 4}};
    for (const auto& x : in)
        if (x.p && (ranges_overlap(o, ob, x.p, x.n) || ranges_overlap(workspace, static_cast<int64_t>(s.bytes), x.p, x.n))) return FUSE_EINVAL;
    if (ranges_overlap(workspace, static_cast<int64_t>(s.bytes), o, ob)) return FUSE_EINVAL;
    PromptArgs a{};
    a.table = block_table;
    a.cu = cu_queries;
    a.lens = seq_lens;
    a.table_ld = table_ld;
    a.o = o;
    a.batch = static_cast<int>(batch);
    a.tokens = static_cast<int>(tokens);
    a.hq = static_cast<int>(q_heads);
    a.hk = static_cast<int>(kv_heads);
    a.group = static_cast<int>(group);
    a.tpt = static_cast<int>(128 / group);
    a.tiles = D <= 128 ? 2 : 1;
    while ((1 << a.page_shift) < page_size) ++a.page_shift;
    a.num_pages = static_cast<int>(num_pages);
    a.cache_rows = static_cast<int>(num_pages * kv_heads * page_size);
    a.c = scale * 1.4426950408889634f;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.start = reinterpret_cast<int4*>(ws);
    a.ml = reinterpret_cast<float2*>(ws + s.ml);
    a.po = reinterpret_cast<float*>(ws + s.po);
    a.rows = static_cast<int>(s.rows);
    a.flag = watchdog_flag();
    a.bad = index_flag();
    if (!a.flag || !a.bad) return FUSE_ECUDA;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == FUSE_F16) {
        if (D == 64) return run_prompt<__half, 64>(a, q, q_ld, k_cache, v_cache, st);
        if (D == 128) return run_prompt<__half, 128>(a, q, q_ld, k_cache, v_cache, st);
        return run_prompt<__half, 256>(a, q, q_ld, k_cache, v_cache, st);
    }
    if (D == 64) return run_prompt<__nv_bfloat16, 64>(a, q, q_ld, k_cache, v_cache, st);
    if (D == 128) return run_prompt<__nv_bfloat16, 128>(a, q, q_ld, k_cache, v_cache, st);
    return run_prompt<__nv_bfloat16, 256>(a, q, q_ld, k_cache, v_cache, st);
}

extern "C" int64_t fuse_prompt_attention_bytes(int64_t tokens, int64_t keys, int64_t q_heads, int64_t kv_heads, int64_t D) {
    if (tokens < 0 || keys < 0 || q_heads < 1 || kv_heads < 1 || D < 1) return FUSE_EINVAL;
    return 4 * D * (kv_heads * keys + tokens * q_heads);   // K and V once; q and o
}

extern "C" int64_t fuse_prompt_attention_flops(int64_t pairs, int64_t q_heads, int64_t D) {
    if (pairs < 0 || q_heads < 1 || D < 1) return FUSE_EINVAL;
    return 4 * D * q_heads * pairs;
}
