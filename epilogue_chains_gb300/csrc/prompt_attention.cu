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
// still fill rows with their group.  An item has two tiles of 128 rows against the same K and V tiles: in one CTA,
// where one tile's softmax runs while the tensor core works for the other, or with D = 256 in a pair of CTAs.
//
// Work is dealt out in equal runs: all items of the batch lie in one line, each counting for its visible keys
// and an entry, and every CTA takes an equal run of it, whatever the lengths are.  What one CTA has of an item
// that several share goes through the workspace, and prompt_join_kernel joins it in the order of the keys.  The
// lengths are in device memory, so one launch configuration (and a captured graph) serves every batch.  All
// waits are bounded (watchdog).
//
// Measured (32 query heads on 8 for keys and values, D = 128, bf16): one prompt of 16384 1.43 ms, 1.54 PFLOP/s of the visible
// pairs, where the chip's power is the limit; 32 of up to 1024 (fp16) 126 us, 0.81; 64 new tokens after 65536 69 us, 1.0, of
// which the join is a fifth.  16 ungrouped heads of 256: 16384 1.40 ms, 1.57; 8 of up to 2048 108 to 111 us, 1.0.  D = 64 (32 heads
// on 8, bf16): 16384 1.10 ms, 1.0.
#include <cudaTypedefs.h>
#include <math.h>

#include <mutex>
#include <type_traits>

#include "fc_internal.cuh"
#include "fc_mma.cuh"
#include "fc_ptx.cuh"
#include "fc_tc.cuh"

namespace fc {
namespace {

constexpr int kMaxBatch = 4096;
constexpr int kTiles = 2;                  // of 128 rows, of an item
constexpr int kGrid = 160;                 // most CTAs (workspace bound); half as many pairs of them
// A running reference is replaced when a row's maximum exceeds it by more than 2^8, so weights stay
// within [0, 2^8]; for fp16 weights it is also set 2^7 below the maximum, which uses fp16's range
// upwards (2^15 at most) and keeps weights down to 2^-21 of the maximum at full precision.
constexpr float kLag = 8.0f;
template <typename T> struct Shift { static constexpr float V = 0.0f; };
template <> struct Shift<__half> { static constexpr float V = 7.0f; };
// What an item counts for apart from its keys, in keys: its entry and its output, of which D = 256 has the longer.  (8 prompts to
// 2048 109 -> 106 us, 100 to 300 with 16 heads on 4 110 -> 102.)
constexpr int kMostEntry = 352;
constexpr int entry_of(int D) { return D == 256 ? kMostEntry : 192; }
// A CTA's run is at least this many keys and an entry: shorter runs cost more to join than they save.
constexpr int kLeastRun = 512;
// Within this many blocks of an item's end a run ends there: so short a part costs more than it evens out.  (In us, from 0 to 2, 3
// and 4: D = 128, 32 prompts to 1024 126, 127, 121, 122, 64 to 200 52, 48, 48, 49, 16 to 500 44, 38, 37, 38, 8 to 2000 102, 98, 99,
// 101; D = 64, 20 to 600 53, 47, 51, 52; D = 256, 8 to 2048 109, 106, 107, 109.)
constexpr int snap_of(int D) { return D == 128 ? 3 : 2; }

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

__device__ __forceinline__ void st_shared_v4(uint32_t addr, const uint32_t (&v)[4]) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}

struct PromptArgs {
    const int32_t *table, *cu, *lens;
    int64_t table_ld;
    void* o;
    int batch, tokens, hq, hk, group;
    int recip;                         // row / group = row recip >> 16 for rows below 128
    int entry, snap;                   // entry_of(D), snap_of(D)
    uint64_t item_recip;               // ceil(2^32 / (tpt tiles))
    bool o_sectors;                    // o lies on a 32-byte boundary
    int tpt;                           // tokens of a tile of 128 rows
    int page_shift, num_pages, cache_rows;
    float c;                           // scale * log2(e)
    // workspace: where each CTA's run begins, and the parts of items that CTAs share: of CTA c slot 2 c has the part of
    // an item that began in an earlier CTA, slot 2 c + 1 that of one which begins here and goes on in a later one
    int4* start;                       // [kGrid + 1]
    float2* ml;                        // [2 for each run][rows]
    float* po;                         // [2 for each run][rows][D]
    int rows;
    int *flag, *bad;
    const void *q, *k, *v;             // for mend_row()
    int64_t q_ld;
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
// n / (tokens of an item), for n below 2^24 (a division takes several times as long).
__device__ __forceinline__ int over_item(const PromptArgs& a, int n) { return static_cast<int>(static_cast<uint64_t>(n) * a.item_recip >> 32); }
__device__ __forceinline__ int items_of(const PromptArgs& a, const Seq& s) { return over_item(a, s.n + a.tpt * kTiles - 1); }
// Keys that the first `tokens` new tokens of a sequence see between them.
__device__ __forceinline__ int extent(const Seq& s, int tokens) { return max(s.L - s.n + min(tokens, s.n), 0); }
// Places of a head's first k items: sum over i < k of entry + extent((i + 1) ti).
__device__ __forceinline__ int64_t places(const PromptArgs& a, const Seq& s, int items, int k) {
    const int64_t ti = a.tpt * kTiles, d = s.L - s.n;
    int64_t sum = static_cast<int64_t>(k) * a.entry;
    if (k == items && k > 0) {
        sum += extent(s, s.n);
        --k;
    }
    const int64_t i0 = d >= 0 ? 0 : over_item(a, static_cast<int>(-d));     // the first item with d + (i + 1) ti > 0
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

// x / y, both positive (64-bit divisions take several times as long as 32-bit ones).
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
    if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
    return x / y;
}
// Place r of sequence b; within `snap` blocks of an item's end, that end.
__device__ __forceinline__ Pos pos_in(const PromptArgs& a, const Seq& s, int b, int64_t r, int snap) {
    const int items = items_of(a, s);
    const int64_t per = places(a, s, items, items);
    Pos p;
    p.b = b;
    p.h = 0;
    if (r >= per) {
        p.h = static_cast<int>(quotient(r, per));
        r -= p.h * per;
    }
    int lo = 0, hi = items - 1;                        // the last item that begins at or before r
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (places(a, s, items, mid) <= r) lo = mid;
        else hi = mid - 1;
    }
    const int64_t in = r - places(a, s, items, lo);
    const int blocks = (extent(s, (lo + 1) * a.tpt * kTiles) + 127) / 128;
    p.i = lo;
    p.t = in <= a.entry ? 0 : static_cast<int>((in - a.entry) >> 7);
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
            const int tok0 = p.i * a.tpt * kTiles;
            const int b0 = (extent(s, tok0 + a.tpt) + 127) / 128;
            const int b1 = tok0 + a.tpt < s.n ? (extent(s, tok0 + 2 * a.tpt) + 127) / 128 : 0;
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
__device__ __forceinline__ Pos* found_at(int64_t* scratch) { return reinterpret_cast<Pos*>(scratch + 52); }
// Where run `me` of `runs` begins and where the next does, for all threads; `scratch` is 80 * 8 bytes of shared memory, in which both
// stay, at found_at().
template <int THREADS>
__device__ __forceinline__ void find_runs(const PromptArgs& a, int me, int runs, int64_t* scratch, Pos (&run)[2]) {
    constexpr int WARPS = THREADS / 32;
    static_assert(WARPS <= 24, "scratch");
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int per = (a.batch + THREADS - 1) / THREADS;
    int64_t mine = 0;
    int count = 0;                                     // items
    for (int i = 0; i < per; ++i) {
        const int b = tid * per + i;
        if (b >= a.batch) break;
        const Seq s = seq_of(a, b, me == 0 ? a.bad : nullptr);
        const int items = items_of(a, s);
        mine += a.hk * places(a, s, items, items);
        count += a.hk * items;
    }
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    count = __reduce_add_sync(0xffffffffu, count);
    // per warp its places and items; then for each target its thread and place there, and where it is found
    int64_t *sums = scratch, *counts = scratch + 24, *target = scratch + 48;
    Pos* found = found_at(scratch);
    if (lane == 31) {
        sums[warp] = upto;
        counts[warp] = count;
    }
    if (tid < 2) target[2 * tid] = -1;
    __syncthreads();
    int64_t total = 0, items = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) upto += sums[w];
        total += sums[w];
        items += counts[w];
    }
    // Equal runs, but none shorter than an item of kLeastRun keys or the average one: with few short items a CTA for each.
    int64_t len = quotient(total + runs - 1, runs), least = items > 0 ? quotient(total + items - 1, items) : 1;
    if (least > kLeastRun + a.entry) least = kLeastRun + a.entry;
    if (len < least) len = least;
    // Long runs snap further, as their parts are the longer for it: 1 / 4096 of a run (64 after 65536 70.1 us, without 71.8, 4 times
    // that 160 and 165; with 1 / 1024 8 of 512 after 16384 341 instead of 315).  Short ones as one likes: 2, 4 or 8 blocks take the same.
    const int snap = len < kLeastRun + a.entry ? 4 : max(a.snap, static_cast<int>(min(len >> 12, static_cast<int64_t>(64))));
    for (int w = 0; w < 2; ++w) {
        const int64_t x = static_cast<int64_t>(me + w) * len;
        if (x < upto && x >= upto - mine) {            // this thread's sequences have it
            target[2 * w] = tid;
            target[2 * w + 1] = x - (upto - mine);
        }
    }
    __syncthreads();
    if (warp < 2 && lane == 0) {
        Pos p{a.batch, 0, 0, 0};
        if (target[2 * warp] >= 0) {
            int64_t x = target[2 * warp + 1];
            for (int b = static_cast<int>(target[2 * warp]) * per;; ++b) {
                const Seq s = seq_of(a, b);
                const int n = items_of(a, s);
                const int64_t here = a.hk * places(a, s, n, n);
                if (x < here) {
                    p = pos_in(a, s, b, x, snap);
                    break;
                }
                x -= here;
            }
        }
        found[warp] = p;
    }
    __syncthreads();
    run[0] = found[0];
    run[1] = found[1];
}

// ================================================================== values that are not finite
// A weight of 0 is no mask in a product: 0 x infinity is NaN, in every row of a tile that does not see the key.  Of a tile's rows the
// first that sees a key sees the fewest, so its output tells whether that has happened.  Where it is not finite, the tile's rows for which
// one of the values that were multiplied with a weight of 0 is not finite are computed again, from the keys that they see alone:
// rare, and slow (a warp takes 8 ms to a row of 16384 keys).  CTAs of the join's launch look at the outputs of all whole items, which takes 2 to 3 us where the join is short
// (32 prompts to 1024 123.5 -> 126.5 us).  Code for it in prompt_attention_kernel costs more, there: looking the values over ahead of
// the products, by the softmax warps, 14 us, a look at the first row's sums by its softmax warp, before, with or after the output,
// or by the warp that issues PV, 7 to 13.  Where nothing is joined the kernel does it, in a form of its own (MEND).

// Whether one of eight values of type T is not finite: its exponent's bits are all ones.
template <typename T>
__device__ __forceinline__ bool not_finite(const uint4& v) {
    constexpr uint32_t MAG = 0x7fff7fffu, STEP = std::is_same<T, __half>::value ? 0x04000400u : 0x00800080u;
    return ((((v.x & MAG) + STEP) | ((v.y & MAG) + STEP) | ((v.z & MAG) + STEP) | ((v.w & MAG) + STEP)) & 0x80008000u) != 0;
}

// A key/value head of a sequence in the cache.
struct Keys {
    const int32_t* table;
    int h;
    __device__ __forceinline__ Keys(const PromptArgs& a, int b, int h) : table(a.table + static_cast<int64_t>(b) * a.table_ld), h(h) {}
    __device__ __forceinline__ int row(const PromptArgs& a, int key) const {        // -1: a page of zeros
        const int page = table[key >> a.page_shift];
        return page >= 0 && page < a.num_pages ? ((page * a.hk + h) << a.page_shift) + (key & ((1 << a.page_shift) - 1)) : -1;
    }
};

// By a warp: the last of the keys first .. end - 1 with a value that is not finite, or -1.
template <typename T, int D>
__device__ __forceinline__ int last_bad(const PromptArgs& a, const Keys& keys, int first, int end) {
    constexpr int LANES = D / 8;                    // threads that read a row in 16-byte vectors
    const int lane = threadIdx.x % 32;
    int last = -1;
#pragma unroll 2
    for (int key = first + lane / LANES; key < end; key += 32 / LANES) {
        const int row = keys.row(a, key);
        if (row >= 0 && not_finite<T>(__ldcg(static_cast<const uint4*>(a.v) + static_cast<int64_t>(row) * LANES + lane % LANES))) last = key;
    }
    return __reduce_max_sync(0xffffffffu, last);
}

// By a warp: f(j, x) for key key0 + j and the thread's columns x of its values, of 32 keys whose rows in the cache the threads have (-1: zeros).
// (No branch, so that the loads of AHEAD keys are on their way together.)
template <typename T, int D, int AHEAD, typename F>
__device__ __forceinline__ void for_values(const PromptArgs& a, int row, F&& f) {
    constexpr int W = D / 32;
    const int lane = threadIdx.x % 32;
#pragma unroll AHEAD
    for (int j = 0; j < 32; ++j) {
        const int rj = __shfl_sync(0xffffffffu, row, j);
        const uint32_t* v = reinterpret_cast<const uint32_t*>(static_cast<const T*>(a.v) + static_cast<int64_t>(max(rj, 0)) * D + W * lane);
        float x[W];
#pragma unroll
        for (int e = 0; e < W; e += 2) {
            const uint32_t w = __ldcg(v + e / 2);
            const float2 g = unpack2<T>(rj < 0 ? 0u : w);
            x[e] = g.x;
            x[e + 1] = g.y;
        }
        f(j, x);
    }
}
__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }

// By a warp: one row of the output again (sequence s's token tok, query head `head`).
template <typename T, int D, int AHEAD>
__device__ __forceinline__ void mend_row(const PromptArgs& a, const Keys& keys, const Seq& s, int tok, int head) {
    constexpr int W = D / 32, LANES = D / 8;        // columns of a thread; 16-byte vectors of a row
    const int lane = threadIdx.x % 32, seen = s.L - s.n + tok + 1;
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + (s.q0 + tok) * a.q_ld + head * D);
    float m = -INFINITY, l = 0.0f, acc[W];
#pragma unroll
    for (int e = 0; e < W; ++e) acc[e] = 0.0f;
#pragma unroll 1
    for (int key0 = 0; key0 < seen; key0 += 32) {
        // 32 scores, one to a thread; then the keys' values, of each W columns to a thread
        const int row = key0 + lane < seen ? keys.row(a, key0 + lane) : -1;
        const uint4* k = static_cast<const uint4*>(a.k) + static_cast<int64_t>(max(row, 0)) * LANES;
        float x = 0.0f;
#pragma unroll AHEAD
        for (int c = 0; c < LANES; ++c) {
            const uint4 kv = __ldcg(k + c), qv = __ldcg(q + c);
            const uint32_t kw[4] = {kv.x, kv.y, kv.z, kv.w}, qw[4] = {qv.x, qv.y, qv.z, qv.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 fk = unpack2<T>(kw[e]), fq = unpack2<T>(qw[e]);
                x = fmaf(fk.x, fq.x, x);
                x = fmaf(fk.y, fq.y, x);
            }
        }
        x = key0 + lane < seen ? (row >= 0 ? x * a.c : 0.0f) : -INFINITY;
        float top = x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (top > m) {
            const float alpha = ex2f(m - top);      // (0 from -inf, with sums of 0)
            m = top;
            l *= alpha;
#pragma unroll
            for (int e = 0; e < W; ++e) acc[e] *= alpha;
        }
        const float p = ex2f(x - (m == -INFINITY ? 0.0f : m));
        l += p;
        for_values<T, D, 2 * AHEAD>(a, row, [&](int j, const float (&v)[W]) {
            const float pj = __shfl_sync(0xffffffffu, p, j);
#pragma unroll
            for (int e = 0; e < W; ++e) acc[e] = fmaf(pj, v[e], acc[e]);
        });
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    const float inv = l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l;
    T* out = static_cast<T*>(a.o) + (static_cast<int64_t>(s.q0 + tok) * a.hq + head) * D + W * lane;
#pragma unroll
    for (int e = 0; e < W; e += 2) *reinterpret_cast<uint32_t*>(out + e) = l == 0.0f ? 0u : pack2<T>(acc[e] * inv, acc[e + 1] * inv);
}

// By a warp: of sequence b's item `at` (of all heads' in line) rows row, row + step .. below `end`, those that do not see a key by whose
// value, which is not finite, they have been multiplied.  A column in which a row sees such a value as well is the sum of those, whatever
// the weights are (so that a cache full of them, or a column of it, does not take long); only rows with another column to mend
// are computed again.  LONG false: all of them, as there are few keys.
template <typename T, int D, int AHEAD, bool LONG>
__device__ __forceinline__ void mend_rows(const PromptArgs& a, int b, int at, int row, int end, int step) {
    constexpr int W = D / 32;
    const int lane = threadIdx.x % 32;
    const Seq s = seq_of(a, b);
    const int items = items_of(a, s), h = at / items, tok0 = (at - h * items) * a.tpt * kTiles;
    const Keys keys(a, b, h);
    int tile = -1, first = 0, last = -1;            // keys that all rows of the tile see; the last one to mend
    float before[W];                                // the sum of what is not finite of those
    // adds what is not finite of keys from .. to - 1 to `sum`, or notes it from key `seen` on
    auto collect = [&](int from, int to, int seen, float (&sum)[W], uint32_t& unseen) {
#pragma unroll 1
        for (int key0 = from; key0 < to; key0 += 32)
            for_values<T, D, 2 * AHEAD>(a, key0 + lane < to ? keys.row(a, key0 + lane) : -1, [&](int j, const float (&v)[W]) {
#pragma unroll
                for (int e = 0; e < W; ++e)
                    if (!finite(v[e])) {
                        if (key0 + j < seen) sum[e] += v[e];
                        else unseen |= 1u << e;
                    }
            });
    };
#pragma unroll 1
    for (; row < end; row += step) {
        const int t = row / 128, r = row % 128, rt = r * a.recip >> 16, tok = tok0 + t * a.tpt + rt, seen = s.L - s.n + tok + 1;
        if (rt >= a.tpt || tok >= s.n || seen <= 0) continue;
        uint32_t unseen = 0;
        if (t != tile) {
            // the tile's blocks (a pair's tiles are multiplied with all of the item's; past the sequence's end there were zeros)
            tile = t;
            first = max(s.L - s.n + tok0 + t * a.tpt + 1, 0);
            last = last_bad<T, D>(a, keys, first, min(s.L, (extent(s, tok0 + (D == 256 ? kTiles : t + 1) * a.tpt) + 127) / 128 * 128));
#pragma unroll
            for (int e = 0; e < W; ++e) before[e] = 0.0f;
            if (LONG && last >= 0) collect(0, first, first, before, unseen);
        }
        if (seen > last) continue;
        const int head = h * a.group + r - rt * a.group;
        float sum[W];
        bool again = !LONG;
#pragma unroll
        for (int e = 0; e < W; ++e) sum[e] = before[e];
        if (LONG) collect(first, last + 1, seen, sum, unseen);
#pragma unroll
        for (int e = 0; e < W; ++e) again = again || ((unseen >> e & 1u) && finite(sum[e]));
        if (__any_sync(0xffffffffu, again)) {
            mend_row<T, D, AHEAD>(a, keys, s, tok, head);
        } else {
            T* out = static_cast<T*>(a.o) + (static_cast<int64_t>(s.q0 + tok) * a.hq + head) * D + W * lane;
#pragma unroll
            for (int e = 0; e < W; ++e)
                if (unseen >> e & 1u) out[e] = from_f32<T>(sum[e]);
        }
    }
}

// The same out of the way of the join's code.
template <typename T, int D>
__device__ __noinline__ void mend_apart(const PromptArgs& a, int b, int at, int row, int end, int step) {
    mend_rows<T, D, 2, true>(a, b, at, row, end, step);
}

// The items that a run (from..to) has whole, an item to each of `warps` warps, of which this is number `me`: mend(b, at) for
// each that has to be mended.
template <typename T, int D, typename Mend>
__device__ __forceinline__ void look_over(const PromptArgs& a, const Pos& from, const Pos& to, int me, int warps, Mend&& mend) {
    const int lane = threadIdx.x % 32;
    int before = 0;                                 // items of the run in the sequences before b0
    // (up to 32 sequences are read without waiting for where the run begins)
    for (int b0 = a.batch <= 32 ? 0 : from.b; b0 < a.batch && b0 <= to.b; b0 += 32) {
        // a sequence to each lane: its items in the run, all heads in line, from the lo-th on
        const int b = b0 + lane;
        Seq s{0, 0, 0};
        int items = 0, lo = 0, count = 0;
        if (b < a.batch) s = seq_of(a, b);
        if (b >= from.b && b <= to.b) {
            items = items_of(a, s);
            lo = b == from.b ? from.h * items + from.i + (from.t > 0 ? 1 : 0) : 0;
            count = max((b == to.b ? to.h * items + to.i : a.hk * items) - lo, 0);
        }
        int upto = count;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        const int all = __shfl_sync(0xffffffffu, upto, 31);
        for (int x = me >= before ? me - before : (warps - (before - me) % warps) % warps; x < all; x += warps) {
            const int from_lane = __popc(__ballot_sync(0xffffffffu, upto <= x));
            const int at = x - __shfl_sync(0xffffffffu, upto - count - lo, from_lane), per = __shfl_sync(0xffffffffu, items, from_lane);
            const int q0 = __shfl_sync(0xffffffffu, s.q0, from_lane), n = __shfl_sync(0xffffffffu, s.n, from_lane), unseen = n - __shfl_sync(0xffffffffu, s.L, from_lane);
            const int h = at / per, i = at - h * per;
            // of each tile the first token that sees a key: 16 bytes of its row by each of D / 8 lanes
            constexpr int LANES = D / 8, TILES = D == 256 ? 1 : kTiles;
            uint32_t bad = 0;
#pragma unroll
            for (int t0 = 0; t0 < kTiles; t0 += TILES) {
                const int t = t0 + lane / LANES, begin = (kTiles * i + t) * a.tpt, tok = max(begin, unseen);
                bool mine = false;
                if (t < t0 + TILES && tok < min(begin + a.tpt, n))
                    mine = not_finite<T>(__ldcg(static_cast<const uint4*>(a.o) + (static_cast<int64_t>(q0 + tok) * a.hq + h * a.group) * LANES + lane % LANES));
                bad |= __ballot_sync(0xffffffffu, mine);
            }
            if (bad != 0) mend(b0 + from_lane, at);
        }
        before += all;
    }
}
template <typename T, int D>
__device__ __noinline__ void mend_run(const PromptArgs& a, const Pos* run, int me, int warps) {
    look_over<T, D>(a, run[0], run[1], me, warps, [&](int b, int at) { mend_rows<T, D, 1, false>(a, b, at, 0, 128 * kTiles, 1); });
}

// Whether the thread's row of a tile's sums in tensor memory has one that is not finite: 0 times it is NaN.
template <int D>
__device__ __forceinline__ bool row_bad(uint32_t out) {
    float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll 1
    for (int y = 0; y < D; y += 64) {
        float o[32];
        tmem_ld_rows16(out + y, o);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) sum[e % 2] = __ffma2_rn(make_float2(o[2 * e], o[2 * e + 1]), make_float2(0.0f, 0.0f), sum[e % 2]);
    }
    return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y) != 0.0f;
}

// ================================================================== the kernel
// Warp 0: Q, K, V loads, 1: S, 2: PV, 3: the walk, from 4 on the softmax: eight warps for each tile, two threads to a row.
// A step of 256 rows by 128 keys takes, between one prompt of 8192 and one of 16384 (32 heads on 8): D = 128 1.66 us in either form, some
// 3000 cycles of the 1.75 to 1.9 GHz that the power limit leaves, of which the products would take 2048; D = 64 1.23 us in one
// piece (2550 cycles, products 1024), 1.42 as a loop.  It is bound by the softmax warps' instructions (600 a warp, four to a scheduler), of
// which 160 are the exponentials and their sums; without exponentials, or without loads, it takes as long.  An item's first step,
// output and diagonal cost 4000 cycles more, so short prompts are slower.  (A thread to a row, one warp per tile in each quarter of
// the SM, was slower: a softmax warp's own instructions, one after the other.)
constexpr int kTileWarps = 8;
constexpr int kFull = 4;                            // barriers of K tiles in turn, and of V tiles
constexpr uint32_t kMostTries = 1u << 18;
constexpr int kSegs = 4;                            // segments that the walk is ahead

template <int D>
struct Layout {
    static constexpr int TILES = kTiles;
    static constexpr int THREADS = 32 * (4 + kTileWarps * TILES);
    // Registers of a thread at the launch, and then of the first four warps and of the softmax's: within what the launch has.
    static constexpr int REGS = 96, FEW = 64, MANY = 104;
    static_assert(128 * (FEW + kTileWarps / 4 * TILES * MANY) <= THREADS * REGS, "registers");
    static constexpr int RING = D == 64 ? 6 : 3;                    // K and V tiles
    static constexpr uint32_t REGION = 128 * 128;              // one 64-column atom of 128 rows
    static constexpr uint32_t TILE = REGION * (D / 64);
    static constexpr uint32_t P_BYTES = 128 * 128 * 2;
    static constexpr uint32_t OFF_Q = 0;
    static constexpr uint32_t OFF_KV = TILES * TILE;
    static constexpr uint32_t OFF_P = OFF_KV + RING * TILE;
    static constexpr uint32_t OFF_BAR = OFF_P + TILES * P_BYTES;
    static constexpr int N_BARS = 2 + 2 * kFull + RING + 12 + 2 + 2 * kSegs + 4;
    static constexpr uint32_t OFF_HOLD = OFF_BAR + N_BARS * 8;
    static constexpr uint32_t OFF_SCRATCH = (OFF_HOLD + 16 + 7) / 8 * 8;
    static constexpr uint32_t OFF_SEG = OFF_SCRATCH + 80 * 8;
    static constexpr uint32_t OFF_NOTED = OFF_SEG + kSegs * sizeof(Seg);      // whether there may be something to mend
    static constexpr uint32_t SMEM = OFF_NOTED + 4 + 1024;
    static constexpr uint32_t TMEM_COLS = 512, O_COL = 256;    // scores of tile t at 128 t, output at 256 + D t
    static_assert(SMEM <= 232448, "shared-memory budget");
    static_assert(SMEM > 116 * 1024, "one CTA per SM: each takes all of TMEM");
};

// HALVES: the two halves of a block's weights as one piece of code (2), or as a loop (1).  MEND: no join comes after it.
template <typename T, int D, int HALVES, bool MEND>
__global__ void __launch_bounds__(Layout<D>::THREADS, 1) prompt_attention_kernel(const __grid_constant__ CUtensorMap mQ,
                                                                       const __grid_constant__ CUtensorMap mK,
                                                                       const __grid_constant__ CUtensorMap mV,
                                                                       const __grid_constant__ CUtensorMap mO,
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
    auto p_full = [&](int t, int h) { return bar0 + 8u * (X + 4 + 2 * t + h); };      // 64 keys' weights
    auto o_done = [&](int t, int h) { return bar0 + 8u * (X + 8 + 2 * t + h); };      // and their product with V
    auto drain = [&](int w) { return bar0 + 8u * (X + 12 + w); };       // of warps 1 and 2
    auto seg_full = [&](int i) { return bar0 + 8u * (X + 14 + i % kSegs); };
    auto seg_free = [&](int i) { return bar0 + 8u * (X + 14 + kSegs + i % kSegs); };
    auto out_full = [&](int t) { return bar0 + 8u * (X + 14 + 2 * kSegs + t); };      // a tile's output is in place of its P
    auto out_free = [&](int t) { return bar0 + 8u * (X + 16 + 2 * kSegs + t); };      // and has been taken
    int* flag = a.flag;
    if (threadIdx.x == 0) {
        if (MEND) *reinterpret_cast<int*>(gbase + L::OFF_NOTED) = 0;
        mbar_init(q_full, 1);
        mbar_init(q_free, 1);
        for (int i = 0; i < kFull; ++i) {
            mbar_init(k_full(i), 1);
            mbar_init(v_full(i), 1);
        }
        for (int i = 0; i < RING; ++i) mbar_init(empty(i), 1);
        for (int i = 0; i < kSegs; ++i) {
            mbar_init(seg_full(i), 1);
            mbar_init(seg_free(i), 3 + kTileWarps * TILES);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(s_full(t), 1);
            mbar_init(s_free(t), kTileWarps);
            mbar_init(out_full(t), kTileWarps);
            mbar_init(out_free(t), 1);
            for (int h = 0; h < 2; ++h) {
                mbar_init(p_full(t, h), kTileWarps);
                mbar_init(o_done(t, h), 1);
            }
            mbar_init(drain(t), 1);
        }
        fence_mbar_init();
    }
    if (threadIdx.x == 32 * 4) {
        prefetch_map(&mQ);
        prefetch_map(&mK);
        prefetch_map(&mV);
        prefetch_map(&mO);
    }
    const uint32_t tmem = tmem_begin(base + L::OFF_HOLD, gbase + L::OFF_HOLD, L::TMEM_COLS, warp);
    pdl_wait();

    Pos run[2];
    find_runs<L::THREADS>(a, blockIdx.x, gridDim.x, reinterpret_cast<int64_t*>(gbase + L::OFF_SCRATCH), run);
    if (threadIdx.x == 0) {
        a.start[blockIdx.x] = make_int4(run[0].b, run[0].h, run[0].i, run[0].t);
        if (blockIdx.x + 1 == gridDim.x) a.start[gridDim.x] = make_int4(run[1].b, run[1].h, run[1].i, run[1].t);
    }
    // Steps of an item: K(0), then K(j + 1) before V(j), through one ring.
    auto k_at = [](int j) { return j == 0 ? 0 : 2 * j - 1; };
    auto v_at = [](int j, int n) { return j + 1 < n ? 2 * j + 2 : 2 * j + 1; };
    Seg* segs_at = reinterpret_cast<Seg*>(gbase + L::OFF_SEG);
    bool ok = true;
    // (A bound by tries, each of which ends by itself after kTryWaitHintNs, together 5 s at most: mbar_wait_bounded()'s clock makes more code at each of
    // the many waits, which the warps fetch over and over: 32 prompts to 1024 142 -> 139 us.)
    auto wait = [&](uint32_t bar, uint32_t parity) {
        for (uint32_t n = 0; !__all_sync(0xffffffffu, mbar_try_wait(bar, parity & 1u)); ++n)
            if (n >= kMostTries || (n % 64 == 63 && *reinterpret_cast<volatile int*>(flag) != 0)) {
                atomicExch(flag, 1);
                ok = false;
                break;
            }
        return ok;
    };
    // Segment k of this CTA, for a warp that goes through them in order; it gives each back when it is done with it.
    auto segment = [&](int k) {
        if (!wait(seg_full(k), k / kSegs)) return false;
        return segs_at[k % kSegs].b >= 0;
    };
    auto leave = [&](int k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(seg_free(k));
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::FEW));
        if (warp == 0) {
            // ---------------------------------------------------------------- Q, K and V loads
            const uint32_t one = elect_one();
            const int box_shift = min(a.page_shift, 7);
            const uint32_t q_box = static_cast<uint32_t>(a.group * a.tpt) * 128u;
            int c = 0, slot = 0, kc = 0, vc = 0, segs = 0;    // loads, the next one's slot, K and V tiles, items
            uint32_t phase = 1;
            for (int k = 0; ok && segment(k); ++k) {
                const Seg g = segs_at[k % kSegs];
                leave(k);
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
            bool issued = false;
            int c = 0, kv = 0, segs = 0;      // loads and K (or V) tiles of the items before this one; items
            int i[2] = {0, 0};                // products of each tile so far
            if (warp == 1) {
                constexpr uint32_t idS = idesc_f16(128, 128, false, false, BF);
                const uint64_t dq = smem_desc_sw128(base + L::OFF_Q, 16, 1024), dk = smem_desc_sw128(base + L::OFF_KV, 16, 1024);
                for (int k = 0; ok && segment(k); ++k) {
                    const Seg g = segs_at[k % kSegs];
                    leave(k);
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
                for (int k = 0; ok && segment(k); ++k) {
                    const Seg g = segs_at[k % kSegs];
                    leave(k);
                    const int n = g.steps();
                    for (int j = 0; ok && j < n; ++j) {
                        const int slot = (c + v_at(j, n)) % RING;
                        const uint64_t vd = dv + static_cast<uint64_t>(slot * (L::TILE >> 4));
                        if (!wait(v_full((kv + j) % kFull), (kv + j) / kFull)) break;
#pragma unroll
                        for (int t = 0; t < TILES; ++t) {
                            if (j >= (t == 0 ? g.n0 : g.n1)) continue;
                            const uint64_t pd = dp + static_cast<uint64_t>(t * (L::P_BYTES >> 4));
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                if (!wait(p_full(t, h), i[t])) break;
                                tc_fence_after();
#pragma unroll
                                for (int s = 4 * h; s < 4 * h + 4; ++s)   // 16 keys each
                                    tc_mma_if(one, tmem + L::O_COL + t * D, pd + ((s / 4) * (L::REGION >> 4) + (s % 4) * 2), vd + s * (2048 >> 4), idO,
                                              j > 0 || s > 0 ? 1u : 0u);
                                tc_commit_if(one, o_done(t, h));
                                issued = true;
                            }
                            ++i[t];
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
        } else {
            // ---------------------------------------------------------------- the walk along the run, ahead of the others
            Walk walk;
            walk.begin(a, run[0], run[1]);
            Seg g;
            for (int k = 0;; ++k) {
                const bool more = walk.next(a, g);
                if (!more) g.b = -1;
                if (k >= kSegs && !wait(seg_free(k), k / kSegs - 1)) break;
                if (lane == 0) {
                    segs_at[k % kSegs] = g;
                    mbar_arrive(seg_full(k));
                }
                __syncwarp();
                if (!more) break;
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::MANY));
        // ---------------------------------------------------------------- softmax: threads l and l + 16 of a warp, one row
        const int t = (warp - 4) / kTileWarps, u = (warp - 4) % kTileWarps, r0 = 32 * (warp % 4) + 16 * (u / 4), r = r0 + lane % 16, hf = lane / 16;
        const uint32_t lanes = static_cast<uint32_t>(r0) << 16;
        const uint32_t st = tmem + lanes + t * 128, ot = tmem + lanes + L::O_COL + t * D;
        const bool stores = u == 0 && lane == 0;      // the thread that stores the tile's output
        // where the thread's weights go: chunk q of 16 bytes at this address with q 16 exchanged (128B swizzle)
        const uint32_t p_at = base + L::OFF_P + t * L::P_BYTES + r * 128 + (((4 * hf) ^ (r & 7)) << 4);
        constexpr float SH = Shift<T>::V;
        int i = 0, kv = 0, outs = 0;                  // steps of this tile; K (or V) tiles; outputs that P has held
        bool held = false;                            // P holds an output that is being stored
        // P may be written: what it held has been taken.
        auto p_ready = [&]() {
            if (!held) return true;
            held = false;
            if (stores) {
                bulk_wait_read0();
                mbar_arrive(out_free(t));
            }
            return wait(out_free(t), outs - 1);
        };
        for (int k = 0; ok && segment(k); ++k) {
            const Seg& g = segs_at[k % kSegs];       // (stays in shared memory: in registers, next to a row's scores, it spills)
            const int n = t == 0 ? g.n0 : g.n1;
            // the first block that some row of the tile does not see all of, and the one that the sequence's last key is in
            const int partial = ((g.L - g.n + g.tok0 + t * a.tpt + 1) >> 7) - g.t0, last = ((g.L - 1) >> 7) - g.t0;
            float m = -INFINITY, l = 0.0f;
            for (int j = 0; j < n; ++j, ++i) {
                if (!wait(s_full(t), i)) break;
                tc_fence_after();
                // 64 keys at a time, so that the weights of the first half are multiplied with V while those of the second are
                // computed, and half of P is free as soon as the last block's half has been multiplied.
#pragma unroll HALVES
                for (int h = 0; h < 2; ++h) {
                    // Asked here, needed below: a wait takes 200 cycles also where nothing is left to wait for (32 prompts to 1024
                    // 134 -> 128.5 us; one vote for both rare cases below: 127).
                    const bool taken = mbar_test(o_done(t, h), (i - 1) & 1);
                    float x[32];         // keys 64 h + 32 hf .. of the block
                    tmem_ld_rows16(st + 64 * h, x);
                    tmem_ld_wait();
                    if (h == 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(s_free(t));
                    }
                    if (j >= partial) {
                        // keys that this row sees, from the thread's first on
                        const int left = g.L - g.n + g.tok0 + t * a.tpt + (r * a.recip >> 16) + 1 - (g.t0 + j) * 128 - 64 * h - 32 * hf;
                        if (__any_sync(0xffffffffu, left < 32)) {
#pragma unroll
                            for (int y = 0; y < 32; ++y) x[y] = y >= left ? -INFINITY : x[y];
                        }
                    }
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int y = 0; y < 32; y += 2) mx[(y >> 1) & 3] = max3f(mx[(y >> 1) & 3], x[y], x[y + 1]);
                    float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.c;
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                    float alpha = 1.0f;
                    if (top > m + (SH + kLag)) {
                        if (j > 0 || h > 0) alpha = ex2f(m - (top - SH));     // (0 from -inf)
                        m = top - SH;
                    }
                    if (h == 0 && j == 0 && !p_ready()) break;
                    // (D = 64 in one piece: the second vote's alpha, kept for longer, spills)
                    const bool plain = __all_sync(0xffffffffu, taken && (HALVES == 2 || alpha == 1.0f));
                    if (!plain && !wait(o_done(t, h), i - 1)) break;
                    const float ref = m == -INFINITY ? 0.0f : m;
                    const float2 c2 = make_float2(a.c, a.c), nm2 = make_float2(-ref, -ref);
                    float2 sum2 = make_float2(0.0f, 0.0f);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        // Rounded to T, as the tensor core takes both operands of a product in one type.  Each is off by at most
                        // half a step of T, as the output's own rounding is.
                        uint32_t w[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const float2 e = __ffma2_rn(make_float2(x[8 * q + 2 * y], x[8 * q + 2 * y + 1]), c2, nm2);
                            const float2 p = make_float2(ex2f(e.x), ex2f(e.y));
                            sum2 = __fadd2_rn(sum2, p);
                            w[y] = pack2<T>(p.x, p.y);
                        }
                        st_shared_v4((p_at ^ (q << 4)) + h * L::REGION, w);
                    }
                    if ((HALVES == 2 || !plain) && __any_sync(0xffffffffu, alpha != 1.0f)) {      // rare: what has been issued of this tile's PV is waited for
                        if (!(h == 0 ? wait(o_done(t, 1), i - 1) : wait(o_done(t, 0), i))) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int y = 0; y < D / 64; ++y) {
                            float o[32];
                            tmem_ld_rows16(ot + 64 * y, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] *= alpha;
                            tmem_st_rows16(ot + 64 * y, o);
                        }
                        tmem_st_wait();
                    }
                    l = l * alpha + (sum2.x + sum2.y);
                    if (h == 0) {
                        // V rows past the sequence's end: 0 x whatever lies there must be 0.  By the tile whose product with
                        // this block is issued first.
                        if (j == last && (t == 0 || j >= g.n0)) {
                            const int vi = kv + j, kleft = g.L - (g.t0 + j) * 128;
                            if (!wait(v_full(vi % kFull), vi / kFull)) break;
                            uint8_t* vb = gbase + L::OFF_KV + ((2 * kv + v_at(j, g.steps())) % RING) * L::TILE;
                            for (int v = 32 * u + lane; v < (128 - kleft) * (D / 8); v += 32 * kTileWarps) {
                                const int row = kleft + v / (D / 8), ch = v % (D / 8);
                                *reinterpret_cast<uint4*>(vb + (ch / 8) * L::REGION + row * 128 + (ch % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
                            }
                        }
                    }
                    fence_async_smem();      // the generic-proxy writes become visible to the tensor core
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(p_full(t, h));
                }
                if (!ok) break;
            }
            kv += g.steps();
            if (!ok || (n > 0 && !wait(o_done(t, 1), i - 1))) break;
            tc_fence_after();
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            // Opaque copies: what depends on them is computed here, not kept in registers next to the scores (which spills).
            int er = r, eh = hf, el = lane, et = t;
            asm volatile("" : "+r"(er), "+r"(eh), "+r"(el), "+r"(et));
            const int tok0 = g.tok0 + et * a.tpt;
            if (MEND && u == 0 && n > 0 && row_bad<D>(ot) && el % 16 == 0) *reinterpret_cast<volatile int*>(gbase + L::OFF_NOTED) = 1;
            if (g.whole) {
                // Through P, which is free: a whole tile is stored from there by one copy while the warps go on; of one that ends
                // within the sequence each warp stores its rows, LANES lanes to a row.
                const float inv = l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l;
                uint8_t* mine = gbase + L::OFF_P + et * L::P_BYTES;
                constexpr int W = D < 128 ? D : 128, LANES = W / 8;      // columns at a time, lanes of a row
                const bool full = tok0 + a.tpt <= g.n;
#pragma unroll 1
                for (int w0 = 0; w0 < D && tok0 < g.n; w0 += W) {
                    if (!p_ready()) break;
#pragma unroll
                    for (int x = 0; x < W / 64; ++x) {
                        float o[32];
                        if (n > 0) {
                            tmem_ld_rows16(ot + w0 + 64 * x, o);
                            tmem_ld_wait();
                        }
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t v[4];
#pragma unroll
                            for (int y = 0; y < 4; ++y) v[y] = n == 0 || l == 0.0f ? 0u : pack2<T>(o[8 * q + 2 * y] * inv, o[8 * q + 2 * y + 1] * inv);
                            *reinterpret_cast<uint4*>(mine + x * L::REGION + er * 128 + (((4 * eh + q) ^ (er & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
                        }
                    }
                    if (full) {
                        fence_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(out_full(t));
                        if (u == 0) {
                            if (!wait(out_full(t), outs)) break;
                            if (lane == 0) {
#pragma unroll
                                for (int x = 0; x < W / 64; ++x)
                                    tma_store_3d(&mO, w0 + 64 * x, g.h * a.group, g.q0 + tok0, base + L::OFF_P + et * L::P_BYTES + x * L::REGION);
                                bulk_commit();
                            }
                            __syncwarp();
                        }
                        held = true;
                        ++outs;
                    } else {
                        __syncwarp();
                        const int ch = el % LANES;
                        T* out = static_cast<T*>(a.o) + (static_cast<int64_t>(g.q0 + tok0) * a.hq + g.h * a.group) * D + w0 + 8 * ch;
#pragma unroll
                        for (int x = 0; x < LANES / 2; ++x) {
                            const int row = er / 16 * 16 + x * (32 / LANES) + el / LANES, rt = row * a.recip >> 16;
                            if (rt < a.tpt && tok0 + rt < g.n)
                                *reinterpret_cast<uint4*>(out + (static_cast<int64_t>(rt) * a.hq + row - rt * a.group) * D) =
                                    *reinterpret_cast<const uint4*>(mine + (ch / 8) * L::REGION + row * 128 + (((ch % 8) ^ (row & 7)) << 4));
                        }
                        __syncwarp();
                    }
                }
            } else {
                const int rt = er * a.recip >> 16, tok = tok0 + rt;
                const bool in = rt < a.tpt && tok < g.n;
                const int64_t at = static_cast<int64_t>(2 * blockIdx.x + (g.t0 == 0 ? 1 : 0)) * a.rows + et * 128 + er;
                if (in && eh == 0) a.ml[at] = make_float2(m, l);
                float* dst = a.po + at * D + 32 * eh;
                if (n > 0)
#pragma unroll 1
                    for (int y = 0; y < D / 64; ++y) {
                        float o[32];
                        tmem_ld_rows16(ot + 64 * y, o);
                        tmem_ld_wait();
                        if (in)
#pragma unroll
                            for (int e = 0; e < 4; ++e) st_v8(dst + 64 * y + 8 * e, o + 8 * e);
                    }
            }
            tc_fence_before();
            leave(k);
        }
        if (stores) bulk_wait0();      // shared memory goes away
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, L::TMEM_COLS);
    }
    if constexpr (MEND) {      // (addresses anew: kept, they would take registers of the loops above)
        uint32_t raw = smem_addr(smem_raw), thread;
        asm volatile("mov.u32 %0, %%tid.x;" : "=r"(thread), "+r"(raw));
        uint8_t* at = smem_raw + (((raw + 1023u) & ~1023u) - raw);
        if (*reinterpret_cast<volatile int*>(at + L::OFF_NOTED) != 0 && thread >= 32 * 4)
            mend_run<T, D>(a, found_at(reinterpret_cast<int64_t*>(at + L::OFF_SCRATCH)), static_cast<int>(thread / 32) - 4, kTileWarps * TILES);
    }
}

// ================================================================== D = 256: a pair of CTAs
// TMEM holds one output of 256 columns next to a tile of scores, so the two tiles of an item lie in two CTAs, which act as one
// M = 256 unit (cta_group::2): CTA t of the pair has tile t's queries, weights and output, and of every block of K and V one half
// (64 keys; 128 columns), which leaves room for two blocks of each and takes half the bytes to every SM.  P is in TMEM, two
// blocks in turn.  CTA 0 issues all products; the bytes of both CTAs count on its barriers, its commits signal both.  The rest is
// as above.  (8 prompts to 2048 with 16 heads: 106 to 110 us.  One CTA by itself, a K or V tile of 64 KB at a time, took 151 us.)
struct PairLayout {
    static constexpr int THREADS = 32 * (4 + kTileWarps);
    static constexpr uint32_t Q_REGION = 128 * 128, K_REGION = 64 * 128, V_REGION = 128 * 128;   // 64-column atoms
    static constexpr uint32_t K_BYTES = 4 * K_REGION, V_BYTES = 2 * V_REGION;
    static constexpr uint32_t OFF_Q = 0, OFF_K = 4 * Q_REGION, OFF_V = OFF_K + 2 * K_BYTES;
    static constexpr uint32_t OFF_BAR = OFF_V + 2 * V_BYTES;
    static constexpr int N_BARS = 2 + 8 + 2 + 4 + 2 + 1 + 2 * kSegs + 2;
    static constexpr uint32_t OFF_HOLD = OFF_BAR + N_BARS * 8;
    static constexpr uint32_t OFF_SCRATCH = (OFF_HOLD + 16 + 7) / 8 * 8;
    static constexpr uint32_t OFF_SEG = OFF_SCRATCH + 80 * 8;
    static constexpr uint32_t OFF_NOTED = OFF_SEG + kSegs * sizeof(Seg);      // whether there may be something to mend
    static constexpr uint32_t SMEM = OFF_NOTED + 4 + 1024;
    static constexpr uint32_t P_COL = 128, O_COL = 256;        // scores at 0
    static_assert(SMEM <= 232448, "shared-memory budget");
    static_assert(SMEM > 116 * 1024, "one CTA per SM: each takes all of TMEM");
};

template <typename T, bool MEND>
__global__ void __launch_bounds__(PairLayout::THREADS, 1) prompt_pair_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
                                                                             const __grid_constant__ CUtensorMap mV,
                                                                             const __grid_constant__ PromptArgs a) {
    using L = PairLayout;
    constexpr int D = 256;
    constexpr bool BF = std::is_same<T, __nv_bfloat16>::value;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - smem_addr(smem_raw));
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    const int rank = static_cast<int>(cluster_rank()), pair = static_cast<int>(blockIdx.x) / 2, pairs = static_cast<int>(gridDim.x) / 2;
    const uint32_t bar0 = base + L::OFF_BAR;
    // of CTA 0: what is loaded, what both CTAs' softmax warps hand over
    const uint32_t q_full = bar0;
    auto k_full = [&](int i) { return bar0 + 8u * (1 + i % 2); };
    auto v_full = [&](int i) { return bar0 + 8u * (3 + i % 2); };
    const uint32_t s_free = bar0 + 8u * 5;
    auto p_full = [&](int i, int h) { return bar0 + 8u * (6 + 2 * (i % 2) + h); };      // block i's weights, 64 keys
    // of each CTA
    const uint32_t q_free = bar0 + 8u * 10, s_full = bar0 + 8u * 11;
    auto k_free = [&](int i) { return bar0 + 8u * (12 + i % 2); };
    auto v_free = [&](int i) { return bar0 + 8u * (14 + i % 2); };
    auto o_done = [&](int i) { return bar0 + 8u * (16 + i % 2); };                      // block i's product with V
    const uint32_t v_here = bar0 + 8u * 18;                                             // a V block that has to be patched has landed
    auto seg_full = [&](int i) { return bar0 + 8u * (19 + i % kSegs); };
    auto seg_free = [&](int i) { return bar0 + 8u * (19 + kSegs + i % kSegs); };
    auto drain = [&](int w) { return bar0 + 8u * (19 + 2 * kSegs + w); };
    static_assert(21 + 2 * kSegs <= L::N_BARS, "barriers");
    int* flag = a.flag;
    if (threadIdx.x == 0) {
        if (MEND) *reinterpret_cast<int*>(gbase + L::OFF_NOTED) = 0;
        mbar_init(q_full, 1);
        mbar_init(q_free, 1);
        mbar_init(s_full, 1);
        mbar_init(s_free, 2 * kTileWarps);
        mbar_init(v_here, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(k_full(i), 1);
            mbar_init(v_full(i), 1);
            mbar_init(k_free(i), 1);
            mbar_init(v_free(i), 1);
            mbar_init(o_done(i), 1);
            mbar_init(p_full(i, 0), 2 * kTileWarps);
            mbar_init(p_full(i, 1), 2 * kTileWarps);
            mbar_init(drain(i), 1);
        }
        for (int i = 0; i < kSegs; ++i) {
            mbar_init(seg_full(i), 1);
            mbar_init(seg_free(i), (rank == 0 ? 3 : 1) + kTileWarps);
        }
        fence_mbar_init();
    }
    if (threadIdx.x == 32 * 4) {
        prefetch_map(&mQ);
        prefetch_map(&mK);
        prefetch_map(&mV);
    }
    const uint32_t tmem = tmem_begin_pair(base + L::OFF_HOLD, gbase + L::OFF_HOLD, 512, warp);
    pdl_wait();

    Pos run[2];
    find_runs<L::THREADS>(a, pair, pairs, reinterpret_cast<int64_t*>(gbase + L::OFF_SCRATCH), run);
    if (threadIdx.x == 0 && rank == 0) {
        a.start[pair] = make_int4(run[0].b, run[0].h, run[0].i, run[0].t);
        if (pair + 1 == pairs) a.start[pairs] = make_int4(run[1].b, run[1].h, run[1].i, run[1].t);
    }
    Seg* segs_at = reinterpret_cast<Seg*>(gbase + L::OFF_SEG);
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        for (uint32_t n = 0; !__all_sync(0xffffffffu, mbar_try_wait(bar, parity & 1u)); ++n)
            if (n >= kMostTries || (n % 64 == 63 && *reinterpret_cast<volatile int*>(flag) != 0)) {
                atomicExch(flag, 1);
                ok = false;
                break;
            }
        return ok;
    };
    auto segment = [&](int k) {
        if (!wait(seg_full(k), k / kSegs)) return false;
        return segs_at[k % kSegs].b >= 0;
    };
    auto leave = [&](int k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(seg_free(k));
    };

    if (warp < 4) {
        if (warp == 0) {
            // ---------------------------------------------------------------- loads: this CTA's queries, keys and columns of V
            const uint32_t one = elect_one();
            const int k_shift = min(a.page_shift, 6), v_shift = min(a.page_shift, 7);
            const uint32_t q_box = static_cast<uint32_t>(a.group * a.tpt) * 128u;
            int kc = 0, vc = 0, segs = 0;
            const uint32_t q_bar = mapa_shared(q_full, 0);
            for (int k = 0; ok && segment(k); ++k) {
                const Seg g = segs_at[k % kSegs];
                leave(k);
                const int n = g.steps();
                if (n == 0) continue;
                if (segs > 0 && !wait(q_free, segs - 1)) break;
                if (rank == 0 && lane == 0) mbar_arrive_expect_tx(q_full, (g.n1 > 0 ? 2 : 1) * 4 * q_box);
                __syncwarp();
                if (rank == 0 || g.n1 > 0)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        tma_load_3d_pair_if(one, base + L::OFF_Q + x * L::Q_REGION, &mQ, 64 * x, g.h * a.group, g.q0 + g.tok0 + rank * a.tpt, q_bar);
                ++segs;
                const int32_t* table = a.table + static_cast<int64_t>(g.b) * a.table_ld;
                // the cache row of a key, or one past the cache: zeros
                auto row_of = [&](int key) {
                    const int page = table[key >> a.page_shift];
                    if (page >= 0 && page < a.num_pages) return ((page * a.hk + g.h) << a.page_shift) + (key & ((1 << a.page_shift) - 1));
                    atomicExch(a.bad, 1);
                    return a.cache_rows;
                };
                for (int x = 0; x < 2 * n; ++x) {
                    // K(0), then K(j + 1) before V(j)
                    const bool is_k = x == 0 || (x % 2 == 1 && x < 2 * n - 1);
                    const int j = is_k ? (x + 1) / 2 : (x == 2 * n - 1 ? n - 1 : x / 2 - 1);
                    const int key0 = (g.t0 + j) * 128, nk = min(128, g.L - key0);
                    if (is_k) {
                        const int mine = min(max(nk - 64 * rank, 0), 64), box = 1 << k_shift, boxes = (mine + box - 1) >> k_shift;
                        const int all = ((min(nk, 64) + box - 1) >> k_shift) + ((max(nk - 64, 0) + box - 1) >> k_shift);
                        const int row = lane < boxes ? row_of(key0 + 64 * rank + (lane << k_shift)) : 0;
                        if (kc >= 2 && !wait(k_free(kc), kc / 2 - 1)) break;
                        if (rank == 0 && lane == 0) mbar_arrive_expect_tx(k_full(kc), static_cast<uint32_t>(all << k_shift) * (D * 2));
                        __syncwarp();
                        const uint32_t dst = base + L::OFF_K + kc % 2 * L::K_BYTES, bar = mapa_shared(k_full(kc), 0);
                        for (int y = 0; y < boxes; ++y) {
                            const int r = __shfl_sync(0xffffffffu, row, y);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                tma_load_2d_pair_if(one, dst + e * L::K_REGION + ((static_cast<uint32_t>(y) << k_shift) * 128), &mK, 64 * e, r, bar);
                        }
                        ++kc;
                    } else {
                        const int box = 1 << v_shift, boxes = (nk + box - 1) >> v_shift;
                        const int row = lane < boxes ? row_of(key0 + (lane << v_shift)) : 0;
                        if (vc >= 2 && !wait(v_free(vc), vc / 2 - 1)) break;
                        if (rank == 0 && lane == 0) mbar_arrive_expect_tx(v_full(vc), static_cast<uint32_t>(boxes << v_shift) * (D * 2));
                        __syncwarp();
                        const uint32_t dst = base + L::OFF_V + vc % 2 * L::V_BYTES, bar = mapa_shared(v_full(vc), 0);
                        for (int y = 0; y < boxes; ++y) {
                            const int r = __shfl_sync(0xffffffffu, row, y);
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                tma_load_2d_pair_if(one, dst + e * L::V_REGION + ((static_cast<uint32_t>(y) << v_shift) * 128), &mV, 128 * rank + 64 * e, r, bar);
                        }
                        ++vc;
                    }
                }
            }
            if (!ok && rank == 0) {   // both CTAs' copies in flight land before either's shared memory goes away
                if (segs > 0) (void)mbar_wait_drain(q_full, (segs - 1) & 1);
                for (int i = max(0, kc - 2); i < kc; ++i) (void)mbar_wait_drain(k_full(i), (i / 2) & 1);
                for (int i = max(0, vc - 2); i < vc; ++i) (void)mbar_wait_drain(v_full(i), (i / 2) & 1);
            }
            __syncwarp();
        } else if (rank == 0 && warp < 3) {
            // ---------------------------------------------------------------- MMA issue for both CTAs: S by warp 1, PV by warp 2
            const uint32_t one = elect_one();
            bool issued = false;
            int i = 0, segs = 0;         // blocks and items so far
            if (warp == 1) {
                constexpr uint32_t idS = idesc_f16(256, 128, false, false, BF);
                const uint64_t dq = smem_desc_sw128(base + L::OFF_Q, 16, 1024);
                for (int k = 0; ok && segment(k); ++k) {
                    const Seg g = segs_at[k % kSegs];
                    leave(k);
                    const int n = g.steps();
                    if (n == 0) continue;
                    if (!wait(q_full, segs)) break;
                    for (int j = 0; j < n; ++j, ++i) {
                        if (!wait(k_full(i), i / 2) || (i > 0 && !wait(s_free, i - 1))) break;
                        tc_fence_after();
                        const uint64_t dk = smem_desc_sw128(base + L::OFF_K + i % 2 * L::K_BYTES, 16, 1024);
#pragma unroll
                        for (int s = 0; s < D / 16; ++s)
                            tc_mma_pair_if(one, tmem, dq + ((s / 4) * (L::Q_REGION >> 4) + (s % 4) * 2), dk + ((s / 4) * (L::K_REGION >> 4) + (s % 4) * 2), idS,
                                           s > 0 ? 1u : 0u);
                        tc_commit_pair_mc_if(one, s_full, 0x3);
                        tc_commit_pair_mc_if(one, k_free(i), 0x3);
                        issued = true;
                    }
                    if (ok) tc_commit_pair_mc_if(one, q_free, 0x3);
                    ++segs;
                }
            } else {
                constexpr uint32_t idO = idesc_f16(256, D, false, true, BF);
                for (int k = 0; ok && segment(k); ++k) {
                    const Seg g = segs_at[k % kSegs];
                    leave(k);
                    const int n = g.steps();
                    for (int j = 0; ok && j < n; ++j, ++i) {
                        if (!wait(v_full(i), i / 2)) break;
                        if (g.L - (g.t0 + j) * 128 < 128 && lane < 2) mbar_arrive_cluster_release(mapa_shared(v_here, lane));
                        __syncwarp();
                        const uint64_t dv = smem_desc_sw128(base + L::OFF_V + i % 2 * L::V_BYTES, L::V_REGION, 1024);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (!wait(p_full(i, h), i / 2)) break;
                            tc_fence_after();
#pragma unroll
                            for (int s = 4 * h; s < 4 * h + 4; ++s)   // 16 keys each
                                tc_mma_pair_ts_if(one, tmem + L::O_COL, tmem + L::P_COL + 64 * (i % 2) + 8 * s, dv + s * (2048 >> 4), idO, j > 0 || s > 0 ? 1u : 0u);
                            issued = true;
                        }
                        if (!ok) break;
                        tc_commit_pair_mc_if(one, v_free(i), 0x3);
                        tc_commit_pair_mc_if(one, o_done(i), 0x3);
                    }
                }
            }
            if (!ok && issued) {   // MMAs in flight finish before TMEM is freed
                if (one) tc_commit_pair(drain(warp - 1));
                __syncwarp();
                (void)mbar_wait_drain(drain(warp - 1), 0);
            }
            __syncwarp();
        } else if (warp == 3) {
            // ---------------------------------------------------------------- the walk along the run, ahead of the others
            Walk walk;
            walk.begin(a, run[0], run[1]);
            Seg g;
            for (int k = 0;; ++k) {
                const bool more = walk.next(a, g);
                if (!more) g.b = -1;
                if (k >= kSegs && !wait(seg_free(k), k / kSegs - 1)) break;
                if (lane == 0) {
                    segs_at[k % kSegs] = g;
                    mbar_arrive(seg_full(k));
                }
                __syncwarp();
                if (!more) break;
            }
        }
    } else {
        // ---------------------------------------------------------------- softmax: threads l and l + 16 of a warp, one row
        const int u = warp - 4, r0 = 32 * (warp % 4) + 16 * (u / 4), r = r0 + lane % 16, hf = lane / 16;
        const uint32_t st = tmem + (static_cast<uint32_t>(r0) << 16), ot = st + L::O_COL;
        const uint32_t s_free0 = mapa_shared(s_free, 0);
        constexpr float SH = Shift<T>::V;
        int i = 0, patched = 0;                       // blocks, and blocks with a patched V, so far
        for (int k = 0; ok && segment(k); ++k) {
            const Seg& g = segs_at[k % kSegs];
            const int n = rank == 0 ? g.n0 : g.n1, steps = g.steps();
            const int partial = ((g.L - g.n + g.tok0 + rank * a.tpt + 1) >> 7) - g.t0;
            float m = -INFINITY, l = 0.0f;
            for (int j = 0; j < steps; ++j, ++i) {
                if (!wait(s_full, i)) break;
                tc_fence_after();
                const bool taken = mbar_test(o_done(i), (i / 2 - 1) & 1);      // this block's place in P is free
                float x[64];         // keys 32 hf .. and 64 + 32 hf .. of the block
                tmem_ld_rows16(st, x);
                tmem_ld_rows16(st + 64, x + 32);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(s_free0);
                float alpha = 1.0f;
                if (j < n) {
                    if (j >= partial) {
                        const int left = g.L - g.n + g.tok0 + rank * a.tpt + (r * a.recip >> 16) + 1 - (g.t0 + j) * 128 - 32 * hf;
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (__any_sync(0xffffffffu, left - 64 * h < 32)) {
#pragma unroll
                                for (int y = 0; y < 32; ++y) x[32 * h + y] = y >= left - 64 * h ? -INFINITY : x[32 * h + y];
                            }
                    }
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int y = 0; y < 64; y += 2) mx[(y >> 1) & 3] = max3f(mx[(y >> 1) & 3], x[y], x[y + 1]);
                    float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.c;
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                    if (top > m + (SH + kLag)) {
                        if (j > 0) alpha = ex2f(m - (top - SH));
                        m = top - SH;
                    }
                }
                const bool plain = __all_sync(0xffffffffu, taken && alpha == 1.0f);
                if (!plain && !wait(o_done(i), i / 2 - 1)) break;
                if (!plain && __any_sync(0xffffffffu, alpha != 1.0f)) {    // rare: the last block's product is waited for
                    if (!wait(o_done(i - 1), (i - 1) / 2)) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int y = 0; y < D / 64; ++y) {
                        float o[32];
                        tmem_ld_rows16(ot + 64 * y, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= alpha;
                        tmem_st_rows16(ot + 64 * y, o);
                    }
                    tmem_st_wait();
                }
                tc_fence_after();
                const float ref = m == -INFINITY ? 0.0f : m;
                const float2 c2 = make_float2(a.c, a.c), nm2 = make_float2(-ref, -ref);
                float2 sum2 = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t w[16];      // rounded to T, as in the kernel above; a tile that sees nothing of the block: 0
#pragma unroll
                    for (int y = 0; y < 16; ++y) w[y] = 0u;
                    if (j < n)
#pragma unroll
                        for (int y = 0; y < 16; ++y) {
                            const float2 e = __ffma2_rn(make_float2(x[32 * h + 2 * y], x[32 * h + 2 * y + 1]), c2, nm2);
                            const float2 p = make_float2(ex2f(e.x), ex2f(e.y));
                            sum2 = __fadd2_rn(sum2, p);
                            w[y] = pack2<T>(p.x, p.y);
                        }
                    tmem_st_pairs16(st + L::P_COL + 64 * (i % 2) + 32 * h, w);
                    tmem_st_wait();
                    bool far = false;    // what is handed over is in shared memory as well
                    if (h == 0) {
                        const int kleft = g.L - (g.t0 + j) * 128;
                        if (kleft < 128) {       // V rows past the sequence's end: 0 x whatever lies there must be 0
                            if (!wait(v_here, patched)) break;
                            ++patched;
                            uint8_t* vb = gbase + L::OFF_V + i % 2 * L::V_BYTES;
                            for (int v = 32 * u + lane; v < (128 - kleft) * 16; v += 32 * kTileWarps) {
                                const int row = kleft + v / 16, ch = v % 16;
                                *reinterpret_cast<uint4*>(vb + (ch / 8) * L::V_REGION + row * 128 + (ch % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
                            }
                            fence_async_smem();
                            far = true;
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (far) mbar_arrive_cluster_release(mapa_shared(p_full(i, h), 0));
                        else mbar_arrive_cluster(mapa_shared(p_full(i, h), 0));
                    }
                }
                if (!ok) break;
                l = l * alpha + (sum2.x + sum2.y);
            }
            if (!ok || (steps > 0 && !wait(o_done(i - 1), (i - 1) / 2))) break;
            tc_fence_after();
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            const int tok0 = g.tok0 + rank * a.tpt;
            if (g.whole) {
                // A row's two threads store whole 32-byte sectors, if o lies on one.  (Through shared memory and a copy, 128 columns or twice 64 at a
                // time, it takes 4000 cycles too: 64 KB from each CTA of the pair at once.)
                const float inv = l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l;
                const int rt = r * a.recip >> 16;
                const bool in = rt < a.tpt && tok0 + rt < g.n;
                T* out = static_cast<T*>(a.o) + (static_cast<int64_t>(g.q0 + tok0 + rt) * a.hq + g.h * a.group + r - rt * a.group) * D + 32 * hf;
#pragma unroll 1
                for (int y = 0; y < D / 64 && tok0 < g.n; ++y) {
                    float o[32];
                    if (n > 0) {
                        tmem_ld_rows16(ot + 64 * y, o);
                        tmem_ld_wait();
                    }
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        float v[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(n == 0 || l == 0.0f ? 0u : pack2<T>(o[16 * q + 2 * e] * inv, o[16 * q + 2 * e + 1] * inv));
                        float* dst = reinterpret_cast<float*>(out + 64 * y + 16 * q);
                        if (in && a.o_sectors) st_v8(dst, v);
                        if (in && !a.o_sectors) {
                            *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
                            *reinterpret_cast<float4*>(dst + 4) = make_float4(v[4], v[5], v[6], v[7]);
                        }
                    }
                }
            } else {
                const int rt = r * a.recip >> 16, tok = tok0 + rt;
                const bool in = rt < a.tpt && tok < g.n;
                const int64_t at = static_cast<int64_t>(2 * pair + (g.t0 == 0 ? 1 : 0)) * a.rows + rank * 128 + r;
                if (in && hf == 0) a.ml[at] = make_float2(m, l);
                float* dst = a.po + at * D + 32 * hf;
                if (n > 0)
#pragma unroll 1
                    for (int y = 0; y < D / 64; ++y) {
                        float o[32];
                        tmem_ld_rows16(ot + 64 * y, o);
                        tmem_ld_wait();
                        if (in)
#pragma unroll
                            for (int e = 0; e < 4; ++e) st_v8(dst + 64 * y + 8 * e, o + 8 * e);
                    }
            }
            if (MEND && u == 0 && n > 0 && row_bad<D>(ot) && lane % 16 == 0) *reinterpret_cast<volatile int*>(gbase + L::OFF_NOTED) = 1;
            tc_fence_before();
            leave(k);
        }
    }
    tc_fence_before();
    cluster_sync();  // neither CTA leaves while its peer may still signal it
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
    // (each CTA has its own tile's word; what one mends again the other has mended alike)
    if (MEND && warp >= 4 && *reinterpret_cast<volatile int*>(gbase + L::OFF_NOTED) != 0)
        mend_run<T, D>(a, found_at(reinterpret_cast<int64_t*>(gbase + L::OFF_SCRATCH)), warp - 4, kTileWarps);
}

// ================================================================== join
// The parts of an item that several CTAs share.  Every run that begins within an item brings join_warps() warps, among which the
// item's rows are shared out: four or eight rows to a warp where two CTAs share the item, one where many do.  It is bound by
// latency: of its launch (about 3 us: the kernel before leaves no room for it), of where the runs begin, then of the parts, so a
// warp reads all it can at once.
constexpr int kJoinThreads = 128, kJoinWords = (kGrid + 1 + 31) / 32;
// Warps for each run that begins within an item.  (32 and 64, in us: D = 128, 32 prompts to 1024 119.4 and 120.7, 2 to 700 24.2 and
// 25.5; D = 256, 8 to 2048 111.6 and 105.9; 16 for D = 128, one of 4096 131 where 32 take 122.)
constexpr int join_warps(int D) { return D == 256 ? 64 : 32; }
// CTAs of each run that look at its whole items' outputs (look_over()), behind those that join.
constexpr int kMendCtas = 2;
// Returns whether some of the rows' sums are not finite.
template <typename T, int D, int ROWS, int AHEAD>
__device__ __forceinline__ bool join_rows(const PromptArgs& a, const Pos& p, const Seq& s, int row0, int rows, int c0, const uint32_t (&has)[kJoinWords], int lane) {
    constexpr int W = D / 32;
    bool bad = false;
    float m[ROWS], l[ROWS], acc[ROWS][W];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.0f;
#pragma unroll
        for (int y = 0; y < W; ++y) acc[i][y] = 0.0f;
    }
    // parts in the order of the keys: CTA c0 - 1's, then those of the runs in `has`
    int word = 0;
    uint32_t left = has[0];
    bool first = true;
    for (;;) {
        int slot[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            slot[j] = -1;
            if (first) {
                first = false;
                slot[j] = 2 * (c0 - 1) + 1;
                continue;
            }
            while (left == 0 && word + 1 < kJoinWords) {
                ++word;
#pragma unroll
                for (int k = 1; k < kJoinWords; ++k)
                    if (word == k) left = has[k];
            }
            if (left != 0) {
                slot[j] = 2 * (32 * word + __ffs(left) - 1);
                left &= left - 1;
            }
        }
        if (slot[0] < 0) break;
        float2 ml[ROWS][AHEAD];
        float v[ROWS][AHEAD][W];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                ml[i][j] = make_float2(-INFINITY, 0.0f);
                if (slot[j] < 0 || i >= rows) continue;
                const int64_t at = static_cast<int64_t>(slot[j]) * a.rows + row0 + i;
                ml[i][j] = __ldcg(a.ml + at);
#pragma unroll
                for (int y = 0; y < W; y += 2) {
                    const float2 x = __ldcg(reinterpret_cast<const float2*>(a.po + at * D + W * lane + y));
                    v[i][j][y] = x.x;
                    v[i][j][y + 1] = x.y;
                }
            }
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                if (ml[i][j].x == -INFINITY && ml[i][j].y == 0.0f) continue;      // (a part that the row sees nothing of has no output)
                const float top = fmaxf(m[i], ml[i][j].x), e0 = m[i] == -INFINITY ? 0.0f : ex2f(m[i] - top), e1 = ex2f(ml[i][j].x - top);
                l[i] = l[i] * e0 + ml[i][j].y * e1;
                m[i] = top;
#pragma unroll
                for (int y = 0; y < W; ++y) acc[i][y] = acc[i][y] * e0 + v[i][j][y] * e1;
            }
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int row = row0 + i, r = row % 128, rt = r * a.recip >> 16, tok = (p.i * kTiles + row / 128) * a.tpt + rt;
        if (i >= rows || rt >= a.tpt || tok >= s.n) continue;
        const float inv = l[i] > 0.0f ? 1.0f / l[i] : l[i] == 0.0f ? 0.0f : l[i];
        float look = 0.0f;                                 // 0 times what is not finite is NaN
#pragma unroll
        for (int y = 0; y < W; ++y) look = fmaf(acc[i][y], 0.0f, look);
        bad = bad || __any_sync(0xffffffffu, look != 0.0f);
        T* dst = static_cast<T*>(a.o) + (static_cast<int64_t>(s.q0 + tok) * a.hq + p.h * a.group + r - rt * a.group) * D + W * lane;
#pragma unroll
        for (int y = 0; y < W; y += 2)
            *reinterpret_cast<uint32_t*>(dst + y) = l[i] == 0.0f ? 0u : pack2<T>(acc[i][y] * inv, acc[i][y + 1] * inv);
    }
    return bad;
}

template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads, 5) prompt_join_kernel(const __grid_constant__ PromptArgs a, int grid) {
    pdl_begin();
    const int lane = threadIdx.x % 32, run = blockIdx.y, unit = blockIdx.x * (kJoinThreads / 32) + threadIdx.x / 32;
    auto start = [&](int c) {
        const int4 v = __ldcg(a.start + min(c, grid));
        return Pos{v.x, v.y, v.z, v.w};
    };
    const Pos p = start(run);
    if (unit >= join_warps(D)) {
        // what has to be mended is listed, so that all of the CTA's warps share its rows
        constexpr int WARPS = kJoinThreads / 32, MOST = 64;
        __shared__ int count, list[MOST][2];
        if (threadIdx.x == 0) count = 0;
        __syncthreads();
        look_over<T, D>(a, p, start(run + 1), unit - join_warps(D), kMendCtas * WARPS, [&](int b, int at) {
            int n = 0;
            if (lane == 0) {
                n = atomicAdd(&count, 1);
                if (n < MOST) {
                    list[n][0] = b;
                    list[n][1] = at;
                }
            }
            if (__shfl_sync(0xffffffffu, n, 0) >= MOST) mend_apart<T, D>(a, b, at, 0, 128 * kTiles, 1);
        });
        __syncthreads();
        for (int n = 0; n < min(count, MOST); ++n) mend_apart<T, D>(a, list[n][0], list[n][1], unit % WARPS, 128 * kTiles, WARPS);
        return;
    }
    if (p.t == 0 || p.b >= a.batch) return;            // this run begins with an item
    // The runs that begin within the same item, and of them those that have something of it (runs may be empty), as bits; the
    // first warp looks from this run on both ways.
    __shared__ uint32_t bits[2][kJoinWords];
    if (threadIdx.x < 2 * kJoinWords) bits[threadIdx.x / kJoinWords][threadIdx.x % kJoinWords] = 0;
    if (threadIdx.x < 32) {
        __syncwarp();
        auto look = [&](int k) {
            const Pos x = start(32 * k + lane), next = start(32 * k + lane + 1);
            const bool in = 32 * k + lane < grid && x.b == p.b && x.h == p.h && x.i == p.i && x.t > 0;
            const uint32_t w = __ballot_sync(0xffffffffu, in), h = __ballot_sync(0xffffffffu, in && x.before(next));
            if (lane == 0) {
                bits[0][k] = w;
                bits[1][k] = h;
            }
            return w;
        };
        const uint32_t w = look(run / 32);
        if (w & 1u)
            for (int k = run / 32 - 1; k >= 0 && (look(k) & 1u); --k) {}
        if (w >> 31)
            for (int k = run / 32 + 1; k < kJoinWords && (look(k) >> 31); ++k) {}
    }
    const Seq s = seq_of(a, p.b);
    __syncthreads();
    uint32_t has[kJoinWords];
    int runs = 0, rank = 0, c0 = 0;
#pragma unroll
    for (int k = 0; k < kJoinWords; ++k) {
        const uint32_t within = bits[0][k];
        has[k] = bits[1][k];
        if (runs == 0 && within != 0) c0 = 32 * k + __ffs(within) - 1;
        runs += __popc(within);
        rank += __popc(run >= 32 * k + 32 ? within : run > 32 * k ? within & ((1u << (run - 32 * k)) - 1u) : 0u);
    }
    int rows = 1;                                      // of a warp, so that all of an item's are someone's
    while (rows * runs * join_warps(D) < 256) rows *= 2;
    const int row0 = (rank * join_warps(D) + unit) * rows;
    if (row0 >= a.rows) return;
    bool bad = false;
    if (rows == 1) {
        bad = join_rows<T, D, 1, 4>(a, p, s, row0, 1, c0, has, lane);
    } else {
        for (int i = 0; i < rows && row0 + i < a.rows; i += 2) bad |= join_rows<T, D, 2, 2>(a, p, s, row0 + i, min(2, a.rows - row0 - i), c0, has, lane);
    }
    if (bad) mend_apart<T, D>(a, p.b, p.h * items_of(a, s) + p.i, row0, min(row0 + rows, a.rows), 1);
}

// ================================================================== host side
struct Sizes {
    int64_t rows;
    size_t ml, po, bytes;
};
Sizes sizes(int64_t tokens, int64_t hq, int64_t hk, int64_t D) {
    Sizes s{};
    const int64_t group = hq / hk, tpt = 128 / group;
    s.rows = tokens <= tpt ? tokens * group : 256;
    size_t at = (kGrid + 1) * sizeof(int4);
    auto part = [&](int64_t n) {
        at = (at + 255) / 256 * 256;
        const size_t was = at;
        at += static_cast<size_t>(n);
        return was;
    };
    const int64_t runs = D == 256 ? kGrid / 2 : kGrid;
    s.ml = part(2 * runs * s.rows * 8);
    s.po = part(2 * runs * s.rows * D * 4);
    s.bytes = (at + 255) / 256 * 256;
    return s;
}

// Pairs of CTAs that can be resident at once.
int pairs_resident() {
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
        cfg.blockDim = dim3(PairLayout::THREADS);
        cfg.dynamicSmemBytes = PairLayout::SMEM;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = 2;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        int n = 0;
        if (opt_in_smem((const void*)prompt_pair_kernel<__half, false>, PairLayout::SMEM) != FUSE_OK ||
            cudaOccupancyMaxActiveClusters(&n, prompt_pair_kernel<__half, false>, &cfg) != cudaSuccess || n < 1) {
            (void)cudaGetLastError();
            n = sm_count() / 2;
        }
        cached[dev] = n > 0 ? n : 1;
    }
    return cached[dev];
}

template <typename T, int D>
int run_prompt(PromptArgs a, const void* q, int64_t q_ld, const void* k, const void* v, cudaStream_t st) {
    constexpr bool bf = std::is_same<T, __nv_bfloat16>::value;
    const int box = 1 << (a.page_shift < 7 ? a.page_shift : 7), k_box = D == 256 && box > 64 ? 64 : box;
    CUtensorMap mQ, mK, mV;
    const int64_t dims[3] = {D, a.hq, a.tokens}, strides[2] = {D * 2, q_ld * 2};
    const int qbox[3] = {64, a.group, a.tpt};
    if (!make_map(&mK, k, a.cache_rows, D, 64, k_box, bf) || !make_map(&mV, v, a.cache_rows, D, 64, box, bf) ||
        !make_map_3d(&mQ, q, kMap16, dims, strides, qbox, 128))
        return FUSE_ECUDA;
    // no more runs than there can be
    const int64_t ti = static_cast<int64_t>(a.tpt) * kTiles, room = a.table_ld << a.page_shift;
    const int64_t items = (ceil_div(a.tokens, ti) + (a.batch < a.tokens ? a.batch : a.tokens)) * a.hk;
    const int64_t most = items * ceil_div(room + a.entry, kLeastRun + a.entry);
    const int64_t resident = D == 256 ? pairs_resident() : sm_count(), limit = D == 256 ? kGrid / 2 : kGrid;
    int64_t runs = resident < limit ? resident : limit;
    if (runs > most) runs = most;
    const bool join = runs > 1 && room > 128;      // an item of at most one block of keys is nobody's to share
    int rc;
    if constexpr (D == 256) {
        const auto kernel = join ? prompt_pair_kernel<T, false> : prompt_pair_kernel<T, true>;
        rc = opt_in_smem((const void*)kernel, PairLayout::SMEM);
        if (rc != FUSE_OK) return rc;
        rc = launch_pdl(kernel, dim3(static_cast<unsigned>(2 * runs)), dim3(PairLayout::THREADS), PairLayout::SMEM, st, 2, mQ, mK, mV, a);
    } else {
        using L = Layout<D>;
        CUtensorMap mO;
        const int64_t o_strides[2] = {D * 2, static_cast<int64_t>(a.hq) * D * 2};
        if (!make_map_3d(&mO, a.o, kMap16, dims, o_strides, qbox, 128)) return FUSE_ECUDA;
        // Short prompts: the loop, whose instructions the warps fetch half of.  In us, loop and one piece: D = 128, 32 prompts to 1024
        // 120 and 143, 8 to 2000 (28 heads on 4) 107 and 122, one of 4096 120 and 120, of 8192 400 and 366, of 16384 1450 and 1415;
        // D = 64 (32 heads on 4), 20 to 600 45 and 47, 8 to 2000 100 and 102, 8 to 3000 180 and 178, 16 to 4096 580 and 538.  Tokens with
        // those behind the last sequence, as the lengths are in device memory; keys of earlier turns are not counted, where the forms
        // differ less: 64 after 65536 70.5 and 70.1, 8 of 512 after 16384 322 and 318 (D = 128), 64 after 65536 57 and 53 (D = 64).
        constexpr int64_t LONG = D == 64 ? 1200 : 3000;    // tokens of a sequence
        const auto kernel = !join                        ? prompt_attention_kernel<T, D, 1, true>
                            : a.tokens >= LONG * a.batch ? prompt_attention_kernel<T, D, 2, false>
                                                         : prompt_attention_kernel<T, D, 1, false>;
        rc = opt_in_smem((const void*)kernel, L::SMEM);
        if (rc != FUSE_OK) return rc;
        rc = launch_pdl(kernel, dim3(static_cast<unsigned>(runs)), dim3(L::THREADS), L::SMEM, st, 1, mQ, mK, mV, mO, a);
    }
    if (rc != FUSE_OK || !join) return rc;
    return launch_pdl(prompt_join_kernel<T, D>, dim3(join_warps(D) / (kJoinThreads / 32) + kMendCtas, static_cast<unsigned>(runs)), dim3(kJoinThreads), 0, st, 1, a,
                      static_cast<int>(runs));
}

}  // namespace

int prompt_report_count() { return 22; }
int prompt_report(int i, fuse_kernel_record* out) {
    switch (i) {
        FC_REPORT(0, Layout<64>::THREADS, Layout<64>::SMEM, 512, prompt_attention_kernel<__nv_bfloat16, 64, 1, true>);
        FC_REPORT(1, Layout<64>::THREADS, Layout<64>::SMEM, 512, prompt_attention_kernel<__nv_bfloat16, 64, 1, false>);
        FC_REPORT(2, Layout<64>::THREADS, Layout<64>::SMEM, 512, prompt_attention_kernel<__nv_bfloat16, 64, 2, false>);
        FC_REPORT(3, Layout<128>::THREADS, Layout<128>::SMEM, 512, prompt_attention_kernel<__nv_bfloat16, 128, 1, true>);
        FC_REPORT(4, Layout<128>::THREADS, Layout<128>::SMEM, 512, prompt_attention_kernel<__nv_bfloat16, 128, 1, false>);
        FC_REPORT(5, Layout<128>::THREADS, Layout<128>::SMEM, 512, prompt_attention_kernel<__nv_bfloat16, 128, 2, false>);
        FC_REPORT(6, PairLayout::THREADS, PairLayout::SMEM, 512, prompt_pair_kernel<__nv_bfloat16, true>);
        FC_REPORT(7, PairLayout::THREADS, PairLayout::SMEM, 512, prompt_pair_kernel<__nv_bfloat16, false>);
        FC_REPORT(8, Layout<64>::THREADS, Layout<64>::SMEM, 512, prompt_attention_kernel<__half, 64, 1, true>);
        FC_REPORT(9, Layout<64>::THREADS, Layout<64>::SMEM, 512, prompt_attention_kernel<__half, 64, 1, false>);
        FC_REPORT(10, Layout<64>::THREADS, Layout<64>::SMEM, 512, prompt_attention_kernel<__half, 64, 2, false>);
        FC_REPORT(11, Layout<128>::THREADS, Layout<128>::SMEM, 512, prompt_attention_kernel<__half, 128, 1, true>);
        FC_REPORT(12, Layout<128>::THREADS, Layout<128>::SMEM, 512, prompt_attention_kernel<__half, 128, 1, false>);
        FC_REPORT(13, Layout<128>::THREADS, Layout<128>::SMEM, 512, prompt_attention_kernel<__half, 128, 2, false>);
        FC_REPORT(14, PairLayout::THREADS, PairLayout::SMEM, 512, prompt_pair_kernel<__half, true>);
        FC_REPORT(15, PairLayout::THREADS, PairLayout::SMEM, 512, prompt_pair_kernel<__half, false>);
        FC_REPORT(16, kJoinThreads, 0, 0, prompt_join_kernel<__nv_bfloat16, 64>);
        FC_REPORT(17, kJoinThreads, 0, 0, prompt_join_kernel<__nv_bfloat16, 128>);
        FC_REPORT(18, kJoinThreads, 0, 0, prompt_join_kernel<__nv_bfloat16, 256>);
        FC_REPORT(19, kJoinThreads, 0, 0, prompt_join_kernel<__half, 64>);
        FC_REPORT(20, kJoinThreads, 0, 0, prompt_join_kernel<__half, 128>);
        FC_REPORT(21, kJoinThreads, 0, 0, prompt_join_kernel<__half, 256>);
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
    // items are counted in 32 bits, the line's places, times the CTAs, in 64
    if ((tokens + batch) * kv_heads >= top || (tokens + batch) * kv_heads >= (int64_t(1) << 52) / (table_ld * page_size + kMostEntry)) return FUSE_EUNSUPPORTED;
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
    a.recip = static_cast<int>((65536 + group - 1) / group);
    a.tpt = static_cast<int>(128 / group);
    a.entry = entry_of(static_cast<int>(D));
    a.snap = snap_of(static_cast<int>(D));
    a.o_sectors = is_aligned(o, 32);
    a.item_recip = ((uint64_t(1) << 32) + a.tpt * kTiles - 1) / (a.tpt * kTiles);
    while ((1 << a.page_shift) < page_size) ++a.page_shift;
    a.num_pages = static_cast<int>(num_pages);
    a.cache_rows = static_cast<int>(num_pages * kv_heads * page_size);
    a.c = scale * 1.4426950408889634f;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.start = reinterpret_cast<int4*>(ws);
    a.ml = reinterpret_cast<float2*>(ws + s.ml);
    a.po = reinterpret_cast<float*>(ws + s.po);
    a.rows = static_cast<int>(s.rows);
    a.q = q;
    a.k = k_cache;
    a.v = v_cache;
    a.q_ld = q_ld;
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
