// paged_attention.cu -- attention of one new token per sequence over a paged key/value cache, with a
// prefix that the whole batch shares.
//
//     o_bh = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m),   s_j = scale q_bh . k_j
// over the prefix's keys and the sequence's own.  A part of the keys gives (m, l, O) = (reference, sum of
// 2^(s - m), sum of 2^(s - m) v), s in base-2 units; parts join as m = max m_i, l = sum 2^(m_i - m) l_i
// and O likewise, so any split of the key axis gives the same result up to fp32 rounding.
//
//  * paged_own_kernel: the sequences' own keys.  Every key and value is used by one group of query heads
//    only (q_heads / kv_heads rows), so reading them bounds the time.  The work is cut into units of 64
//    keys of one (sequence, key/value head), numbered in one line, and the CTAs take equal runs of it,
//    whatever the lengths are: a long sequence is shared by many CTAs, a CTA covers many short ones.  One
//    warp loads units by TMA into a ring, four compute: each multiplies its 16 keys of a unit with the
//    query rows by mma.sync (16 rows, mostly one group), and the warps' parts meet in shared memory when
//    a run ends.  Parts of a sequence that several CTAs share go through the workspace: the CTA that
//    arrives last joins them, in the order of the keys (with a prefix, paged_join_kernel does).  3 x 65536 keys (D = 128) take 109 us, 0.97 of
//    the copy rate; 32 sequences of up to 4096 keys 50 us, 0.83.
//  * paged_prefix_kernel, paged_prefix2_kernel: the shared prefix.  Here all batch * group query rows of a
//    key/value head meet the same keys: tcgen05 tiles of 128 or 256 rows by 128 keys, scores and output
//    in TMEM, the key axis split over the SMs.  1024 rows per head over 16384 keys (8 heads, D = 128) take
//    49 us of the call's 91, 1.4 PFLOP/s.
//  * paged_join_kernel, with a prefix: a row's own parts and the prefix's.
//
// The lengths are in device memory, so one launch configuration (and a captured graph) serves every
// length.  All waits are bounded (watchdog).
#include <cudaTypedefs.h>
#include <math.h>

#include <type_traits>

#include "fc_internal.cuh"
#include "fc_mma.cuh"
#include "fc_ptx.cuh"
#include "fc_tc.cuh"

namespace fc {
namespace {

constexpr int kOwnWarps = 4;
constexpr int kOwnThreads = 32 * (kOwnWarps + 1); // the last warp loads
constexpr int kChunk = 16;                        // keys of a warp per unit
constexpr int kUnit = kChunk * kOwnWarps;         // keys of a unit
constexpr int kOwnSlots = 8;                       // most ring slots
constexpr int kOwnGrid = 320;                     // most CTAs of paged_own_kernel (workspace bound)
constexpr int kCounterBytes = 8192;
static_assert(kOwnGrid * kOwnWarps * 4 + 4 <= kCounterBytes, "one counter per CTA and warp, and `ready`");
constexpr int kPrefixGrid = 160;                  // most CTAs of paged_prefix_kernel (workspace bound)
constexpr int kMaxBatch = 4096;
constexpr int kOwnSmem = 226 * 1024;              // dynamic shared memory at most, next to a few static words
// A running reference is replaced when a row's maximum exceeds it by more than 2^8, so weights stay
// within [0, 2^8]; for fp16 weights it is also set 2^7 below the maximum, which uses fp16's range
// upwards (2^15 at most) and keeps weights down to 2^-21 of the maximum at full precision.
constexpr float kLag = 8.0f;
template <typename T> struct Shift { static constexpr float V = 0.0f; };
template <> struct Shift<__half> { static constexpr float V = 7.0f; };

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

struct PagedArgs {
    const void* q;
    void* o;
    const int32_t *table, *lens, *ptable;
    int64_t table_ld;
    int batch, hq, hk, group, rt;      // rt = ceil(group / 16) row tiles of a key/value head
    int rows;                          // query rows of a tile, at most 16
    int page_shift, num_pages;
    int cache_rows;                    // num_pages hk page_size: a row past the cache reads zeros
    float c;                           // scale * log2(e)
    int slots;                         // of the ring
    uint32_t off_q, off_om, off_ml, off_bar, off_pre;
    // workspace
    // A CTA's units have at most one item that began in an earlier CTA (its part has slot 2 c) and one
    // that goes on in a later one (slot 2 c + 1 if it begins here; an item begins in one CTA, which
    // names its counter).
    int* count;                        // [kOwnGrid][kOwnWarps] parts that have arrived, by the item's first CTA
    int* ready;                        // with a prefix: 1 from the prefix kernel's grid-dependency wait to the join
    float *oml, *oo;                   // [2 kOwnGrid][rows] (m, l) and [..][rows][D]
    // with a prefix: where the own parts of an item (sequence, row tile of a key/value head) are, -1: in rml and ro
    // (it has one), else the CTAs that have them, first | last << 16; [batch hk rt]
    int* where;
    float *rml, *ro;                   // [batch hq] (m, l) and [..][D]
    float *pml, *po;                   // [kPrefixGrid + pitems][prow] (m, l, l', -) and [..][prow][D]
    // prefix
    int plen, ptiles, prow, prt, pgrid; // keys, 128-key tiles, rows of an item (128 or 256), a head's items, CTAs
    int pent;                          // places that an item's entry counts for (see PrefixSeg)
    int *flag, *bad;
};

// The CTA of `grid` that place u belongs to when CTA c takes places [c U / grid, (c + 1) U / grid).
__device__ __forceinline__ int cta_of(int64_t u, int64_t U, int grid) {
    const uint64_t n = static_cast<uint64_t>(u + 1) * static_cast<uint32_t>(grid) - 1;
    if (((n | static_cast<uint64_t>(U)) >> 32) == 0)   // a 64-bit division takes several times as long
        return static_cast<int>(static_cast<uint32_t>(n) / static_cast<uint32_t>(U));
    return static_cast<int>(n / static_cast<uint64_t>(U));
}

// Join (m, l, acc) with another part; a part without keys has m = -inf, l = 0.
__device__ __forceinline__ void join(float& m, float& l, float4& acc, float m2, float l2, const float4& o2) {
    const float nm = fmaxf(m, m2);
    const float a = m == -INFINITY ? 0.0f : ex2f(m - nm), b = m2 == -INFINITY ? 0.0f : ex2f(m2 - nm);
    l = l * a + l2 * b;
    acc.x = acc.x * a + o2.x * b;
    acc.y = acc.y * a + o2.y * b;
    acc.z = acc.z * a + o2.z * b;
    acc.w = acc.w * a + o2.w * b;
    m = nm;
}

// Join the parts c0 .. c1 of four output columns that lie in memory, in order; part(c, &m, &l) gives the
// address of part c's columns.  Eight parts are loaded at a time, so that their memory latencies overlap.
template <typename F>
__device__ __forceinline__ void join_parts(int c0, int c1, float& m, float& l, float4& acc, F&& part) {
    for (int c = c0; c <= c1; c += 8) {
        float pm[8], pl[8];
        float4 po[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) po[i] = __ldcg(part(min(c + i, c1), pm[i], pl[i]));
#pragma unroll
        for (int i = 0; i < 8; ++i)     // (past the last part nothing: an infinite sum once more, times zero, would be NaN)
            if (c + i <= c1) join(m, l, acc, pm[i], pl[i], po[i]);
    }
}

// ================================================================== the sequences' own keys
template <int D>
struct OwnLayout {
    static constexpr int ATOMS = D / 64;
    static constexpr uint32_t ATOM = kUnit * 128;                // 64 keys x 64 components
    static constexpr uint32_t SLOT = ATOM * ATOMS;               // K or V of a unit
    static constexpr uint32_t QATOM = 16 * 128;                  // 16 query rows x 64 components
    static constexpr uint32_t QSLOT = QATOM * ATOMS;
    // CTAs per SM.  D = 256: one, whose 255 registers hold the query rows next to the output, and whose ring is
    // twice as long (two, with the rows read again from shared memory for every unit: 69 us where one takes 59)
    static constexpr int CTAS = D <= 128 ? 2 : 1;
    static constexpr int NQ = D <= 128 ? 4 : 2;                  // buffers of query rows
};

// What is dealt out to the CTAs are places in one line: per item, that is sequence and row tile of a key/value
// head, an entry and then its units.  The entry stands for what an item costs apart from its units (loading
// the query rows, joining the parts: about a unit's time).  Without it, CTAs that got sequences of one unit took
// up to 40 us where the median took 27 (256 sequences of 1 to 256 keys).
struct Cursor {
    int left;        // places left of the CTA's, this one included
    int b, hr;       // sequence; key/value head * rt + row tile
    int j, n, len;   // unit of the sequence (-1: the entry), their number, its keys
};
__device__ __forceinline__ int places_of(int len) { return 1 + (len > kUnit ? (len - 1) / kUnit + 1 : 1); }

// Four computing warps and one that loads.  The loading warp places 32 units at a time, one per lane (which
// sequence and head, which pages), a batch ahead of the loads, so that no table entry is waited for between
// two loads; it loads the query rows of a run, then K and V of every unit, each into the next slot of a ring.
// Under load a dependent read of global memory takes several microseconds (the ring keeps the memory queues
// full), which is why nothing else reads global memory inside the loop.
template <typename T, int D>
__global__ void __launch_bounds__(kOwnThreads, OwnLayout<D>::CTAS) paged_own_kernel(
    const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
    const __grid_constant__ CUtensorMap mV, const __grid_constant__ CUtensorMap mK16,
    const __grid_constant__ CUtensorMap mV16, const __grid_constant__ PagedArgs a) {
    using L = OwnLayout<D>;
    pdl_trigger();
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - smem_addr(smem_raw));
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    int* pre = reinterpret_cast<int*>(gbase + a.off_pre);        // [batch + 1] places of a head before a sequence
    int* slen = pre + a.batch + 1;                               // [batch]
    __shared__ int wsum[kOwnWarps + 1];
    const uint32_t bars = base + a.off_bar;
    auto full = [&](int i) { return bars + 8u * i; };
    auto empty = [&](int i) { return bars + 8u * (kOwnSlots + i); };
    auto q_full = [&](int i) { return bars + 8u * (2 * kOwnSlots + i); };
    auto q_empty = [&](int i) { return bars + 8u * (2 * kOwnSlots + L::NQ + i); };
    // parts of run r in buffer r % 2, filled and joined by all computing warps
    auto parts_full = [&](int i) { return bars + 8u * (2 * kOwnSlots + 2 * L::NQ + i); };
    auto parts_free = [&](int i) { return bars + 8u * (2 * kOwnSlots + 2 * L::NQ + 2 + i); };
    if (tid == 0) {
        for (int i = 0; i < a.slots; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), kOwnWarps);
        }
        for (int i = 0; i < L::NQ; ++i) {
            mbar_init(q_full(i), 1);
            mbar_init(q_empty(i), kOwnWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(parts_full(i), kOwnWarps);
            mbar_init(parts_free(i), kOwnWarps);
        }
        fence_mbar_init();
        prefetch_map(&mQ);
        prefetch_map(&mK);
        prefetch_map(&mV);
    }
    // With a prefix, the kernel before this one is the prefix's, of which nothing is read here.  It lets this one
    // start once it has itself waited for what came before, so CTAs of this kernel take over the SMs as the
    // prefix's CTAs leave them; the wait is made up for at the end, for paged_join_kernel's sake.  Starting early
    // does not make the writes of the kernels before the prefix's visible here: the prefix kernel's release of
    // `ready`, after its wait, and the acquire here do (it is there by then: nothing is waited for).
    if (a.plen == 0) {
        pdl_wait();
    } else {
        if (tid == 32) (void)flag_wait_bounded(a.ready, 1, a.flag);
        __syncthreads();
        fence_async_global();          // for the copy engine's reads as well
    }

    // ------------------------------------------------------------ places of every sequence
    {
        const int64_t most = a.table_ld << a.page_shift;
        const int per = (a.batch + kOwnThreads - 1) / kOwnThreads, b0 = tid * per;
        int sum = 0;
        for (int b = b0; b < b0 + per && b < a.batch; ++b) {
            int n = __ldcg(a.lens + b);
            if (n < 0 || n > most) {
                if (blockIdx.x == 0) atomicExch(a.bad, 1);
                n = n < 0 ? 0 : static_cast<int>(most);
            }
            slen[b] = n;
            sum += places_of(n);
        }
        int scan = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, scan, o);
            if (lane >= o) scan += v;
        }
        if (lane == 31) wsum[warp] = scan;
        __syncthreads();
        int at = scan - sum;
        for (int w = 0; w < warp; ++w) at += wsum[w];
        for (int b = b0; b < b0 + per && b < a.batch; ++b) {
            pre[b] = at;
            at += places_of(slen[b]);
            if (b == a.batch - 1) pre[a.batch] = at;
        }
        __syncthreads();
    }
    const int HR = a.hk * a.rt;
    const int64_t U = static_cast<int64_t>(pre[a.batch]) * HR;
    // CTAs with work: two places each at least, as every further one makes the joins longer (one sequence of 3000 keys
    // 12.4 -> 11.0 us, two of 5000 13.8 -> 10.9, with three 11.1 and 10.7, but four of 1000 10.1 -> 12.4)
    const int G = static_cast<int>(min(static_cast<int64_t>(gridDim.x), (U + 1) / 2));
    if (static_cast<int>(blockIdx.x) >= G) return;
    const int64_t u0 = blockIdx.x * U / G;
    const int total = static_cast<int>((blockIdx.x + 1) * U / G - u0);

    auto locate = [&](int64_t u, Cursor& k) {
        int lo = 0, hi = a.batch - 1;   // the last sequence that starts at or before u
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (static_cast<int64_t>(pre[mid]) * HR <= u) lo = mid; else hi = mid - 1;
        }
        k.b = lo;
        const int places = pre[lo + 1] - pre[lo];
        k.n = places - 1;
        k.len = slen[lo];
        const int64_t in = u - static_cast<int64_t>(pre[lo]) * HR;
        if ((in >> 32) == 0) {
            k.hr = static_cast<int>(static_cast<uint32_t>(in) / static_cast<uint32_t>(places));
            k.j = static_cast<int>(static_cast<uint32_t>(in) % static_cast<uint32_t>(places)) - 1;
        } else {
            k.hr = static_cast<int>(in / places);
            k.j = static_cast<int>(in % places) - 1;
        }
    };

    if (warp == kOwnWarps) {
        // ---------------------------------------------------------------- loads
        // Whole units come in boxes of a page (64 keys at most), the last one of a sequence in boxes of 16, so
        // that hardly more is read than there is.
        const int big_shift = min(a.page_shift, 6);
        struct Place {
            int page[4];     // of the unit's boxes, as the table has them
            int in[4];       // row of a box within its page, all heads counted
            int boxes;       // boxes with keys; 0 where the sequence has none
            int shift;       // keys of a box
            int qrow;        // first query row if a part begins here, else -1
        };
        // The table is read for 32 units, one per lane, and the entries are used only when the 32 before them
        // have been loaded.
        auto place = [&](int i, Place& p) {   // place u0 + i
            p.boxes = 0;
            p.shift = 4;
            p.qrow = -1;
            if (i >= total) return;
            Cursor k;
            locate(u0 + i, k);
            if (a.plen > 0 && k.j == 0) {
                const int c0 = static_cast<int>(blockIdx.x), c1 = cta_of(u0 + i + k.n - 1, U, G);
                a.where[k.b * HR + k.hr] = c1 == c0 ? -1 : c0 | c1 << 16;
            }
            const int head = k.hr / a.rt, nk = min(kUnit, k.len - k.j * kUnit);
            if (k.j < 0 || nk <= 0) return;
            p.shift = nk == kUnit ? big_shift : 4;
            p.boxes = (nk + (1 << p.shift) - 1) >> p.shift;
            if (i == 0 || k.j == 0) p.qrow = k.b * a.hq + head * a.group + (k.hr % a.rt) * 16;
#pragma unroll
            for (int x = 0; x < 4; ++x)
                if (x < p.boxes) {
                    const int key = k.j * kUnit + (x << p.shift);
                    p.page[x] = __ldcg(a.table + k.b * a.table_ld + (key >> a.page_shift));
                    p.in[x] = (head << a.page_shift) + (key & ((1 << a.page_shift) - 1));
                }
        };
        const int page_rows = a.hk << a.page_shift;
        auto row_of = [&](const Place& p, int x) {
            if (x >= p.boxes) return 0;
            if (p.page[x] >= 0 && p.page[x] < a.num_pages) return p.page[x] * page_rows + p.in[x];
            atomicExch(a.bad, 1);
            return a.cache_rows;         // past the cache: zeros
        };
        const uint32_t one = elect_one();
        const uint64_t once = policy_evict_first();      // ragged batch 51.8 -> 49.4 us then: what else lies in L2 stays there
        int slot = 0, loads = 0, qs = 0, qloads = 0;
        uint32_t phase = 0, qphase = 0;          // completions of the current slot's barriers so far, mod 2
        bool ok = true;
        auto wait = [&](uint32_t bar, uint32_t parity) {
            ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, a.flag));
            return ok;
        };
        Place cur{}, ahead{};
        place(lane, cur);
        for (int i0 = 0; ok && i0 < total; i0 += 32) {
            int row[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) row[x] = row_of(cur, x);
            const int n = min(32, total - i0);
            for (int x = 0; ok && x < n; ++x) {
                const int boxes = __shfl_sync(0xffffffffu, cur.boxes, x);
                if (boxes > 0) {
                    const int qrow = __shfl_sync(0xffffffffu, cur.qrow, x), shift = __shfl_sync(0xffffffffu, cur.shift, x);
                    if (qrow >= 0) {
                        if (qloads >= L::NQ && !wait(q_empty(qs), qphase ^ 1u)) break;
                        if (lane == 0) mbar_arrive_expect_tx(q_full(qs), static_cast<uint32_t>(a.rows) * (D * 2));
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < L::ATOMS; ++i) tma_load_2d_if(one, base + a.off_q + qs * L::QSLOT + i * L::QATOM, &mQ, 64 * i, qrow, q_full(qs));
                        ++qloads;
                        if (++qs == L::NQ) {
                            qs = 0;
                            qphase ^= 1u;
                        }
                    }
                    int r[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y) r[y] = __shfl_sync(0xffffffffu, row[y], x);
                    auto load = [&](const CUtensorMap* map) {
                        if (loads >= a.slots && !wait(empty(slot), phase ^ 1u)) return;
                        if (lane == 0) mbar_arrive_expect_tx(full(slot), static_cast<uint32_t>(boxes << shift) * (D * 2));
                        __syncwarp();
                        const uint32_t dst = base + slot * L::SLOT;
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            if (y < boxes)
#pragma unroll
                                for (int i = 0; i < L::ATOMS; ++i)
                                    tma_load_2d_once_if(one, dst + i * L::ATOM + ((static_cast<uint32_t>(y) << shift) * 128), map, 64 * i, r[y], full(slot), once);
                        ++loads;
                        if (++slot == a.slots) {
                            slot = 0;
                            phase ^= 1u;
                        }
                    };
                    if (shift == big_shift) {
                        load(&mK);
                        if (ok) load(&mV);
                    } else {
                        load(&mK16);
                        if (ok) load(&mV16);
                    }
                }
                if (x == min(3, n - 1)) place(i0 + 32 + lane, ahead);   // once the ring has something to load
            }
            cur = ahead;
        }
        if (!ok) {   // after a wait that ran out: copies in flight land before the shared memory goes away
            for (int j = max(0, loads - a.slots); j < loads; ++j) (void)mbar_wait_drain(full(j % a.slots), (j / a.slots) & 1);
            for (int j = max(0, qloads - L::NQ); j < qloads; ++j) (void)mbar_wait_drain(q_full(j % L::NQ), (j / L::NQ) & 1);
        }
        if (a.plen > 0 && blockIdx.x == 0) pdl_wait();      // this kernel is not over before the prefix's is
        return;
    }

    // -------------------------------------------------------------------- joining a run's parts
    const int g = lane / 4, t = lane % 4;
    float* om = reinterpret_cast<float*>(gbase + a.off_om);      // [2][warp][rows][D]
    float* ml = reinterpret_cast<float*>(gbase + a.off_ml);      // [2][warp][16][2]
    // Every warp joins its share of the run's pieces of four output columns (and counts arrivals of its share).
    struct Run {
        int b, hr, j0, j1, n, buf;
    };
    auto join_run = [&](const Run& k) {
        const int head = k.hr / a.rt, row0 = (k.hr % a.rt) * 16, rows = min(a.rows, a.group - row0);
        if (warp * 32 >= rows * (D / 4)) return;
        const float* omb = om + k.buf * (kOwnWarps * a.rows * D);
        const float* mlb = ml + k.buf * (kOwnWarps * 32);
        int c0 = 0, c1 = 0;
        bool last = k.j0 == 0 && k.j1 == k.n;
        if (!last) {
            const int64_t first = static_cast<int64_t>(pre[k.b]) * HR + static_cast<int64_t>(k.hr) * (k.n + 1) + 1;
            c0 = cta_of(first, U, G);
            c1 = cta_of(first + k.n - 1, U, G);
        }
        const int64_t orow = static_cast<int64_t>(k.b) * a.hq + head * a.group + row0;
        for (int pass = 0; pass < 2; ++pass) {
            // pass 0: the warps' parts, to the output if this is all of the item, else to the workspace;
            // pass 1 (where the CTA's warp arrives last): the CTAs' parts, to the output
            for (int i = warp * 32 + lane; i < rows * (D / 4); i += 32 * kOwnWarps) {
                const int r = i / (D / 4), col = i % (D / 4);
                float m = -INFINITY, l = 0.0f;
                float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (pass == 0) {
#pragma unroll
                    for (int w = 0; w < kOwnWarps; ++w) {
                        const float2 x = *reinterpret_cast<const float2*>(mlb + (w * 16 + r) * 2);
                        join(m, l, acc, x.x, x.y, *reinterpret_cast<const float4*>(omb + (w * a.rows + r) * D + 4 * col));
                    }
                } else {
                    join_parts(c0, c1, m, l, acc, [&](int c, float& pm, float& pl) {
                        const int64_t at = static_cast<int64_t>(2 * c + (c == c0 ? 1 : 0)) * a.rows + r;
                        const float2 x = __ldcg(reinterpret_cast<const float2*>(a.oml + 2 * at));
                        pm = x.x;
                        pl = x.y;
                        return reinterpret_cast<const float4*>(a.oo + at * D + 4 * col);
                    });
                }
                if (last && a.plen == 0) {
                    // l == 0: no key (or none with a score above -inf): zeros
                    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                    uint2 w;
                    w.x = l == 0.0f ? 0u : pack2<T>(acc.x * inv, acc.y * inv);
                    w.y = l == 0.0f ? 0u : pack2<T>(acc.z * inv, acc.w * inv);
                    *reinterpret_cast<uint2*>(static_cast<T*>(a.o) + (orow + r) * D + 4 * col) = w;
                } else {   // a part for the item's last CTA, or for paged_join_kernel
                    const int64_t at = last ? orow + r : static_cast<int64_t>(2 * blockIdx.x + (k.j0 == 0 ? 1 : 0)) * a.rows + r;
                    // (m, l) of a row goes with the first of its columns that this warp holds: every warp's
                    // share is read back by the same warp of another CTA
                    if (col == 0 || lane == 0) *reinterpret_cast<float2*>((last ? a.rml : a.oml) + 2 * at) = make_float2(m, l);
                    *reinterpret_cast<float4*>((last ? a.ro : a.oo) + at * D + 4 * col) = acc;
                }
            }
            if (last || a.plen > 0) return;
            __threadfence();
            __syncwarp();
            int* count = a.count + c0 * kOwnWarps + warp;
            int arrived = 0;
            if (lane == 0) arrived = atomicAdd(count, 1);
            last = __shfl_sync(0xffffffffu, arrived, 0) == c1 - c0;
            if (!last) return;
            __threadfence();
            if (lane == 0) *count = 0;
        }
    };

    // -------------------------------------------------------------------- units
    Cursor cur;
    locate(u0, cur);
    cur.left = total;
    auto next = [&](Cursor& k) {
        --k.left;
        if (++k.j < k.n) return;
        k.j = -1;
        if (++k.hr < HR) return;
        k.hr = 0;
        if (++k.b < a.batch) {
            k.n = pre[k.b + 1] - pre[k.b] - 1;
            k.len = slen[k.b];
        }
    };
    int slot = 0, qs = 0, runs = 0;
    uint32_t phase = 0, qphase = 0;
    bool ok = true;
    // Wait for a barrier; done() gives a slot back.
    auto wait_full = [&](uint32_t bar, uint32_t ph) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(bar, ph, a.flag));
        return ok;
    };
    auto done = [&] {
        __syncwarp();
        if (lane == 0) mbar_arrive(empty(slot));
        if (++slot == a.slots) {
            slot = 0;
            phase ^= 1u;
        }
    };
    // The parts of run r are joined once those of run r + 1 have been written (or at the end): by then all
    // warps have written them, and nothing is waited for.
    Run before{};
    auto join_before = [&] {
        if (wait_full(parts_full(before.buf), ((runs - 1) >> 1) & 1)) join_run(before);
        __syncwarp();
        if (lane == 0) mbar_arrive(parts_free(before.buf));
    };
    // ldmatrix addresses: row and 16-byte column of this lane's matrix row, for Q, K and V (transposed)
    const int qrow = lane & 15, qcol = lane >> 4;
    const int kkey = warp * kChunk + (((lane >> 4) << 3) | (lane & 7)), kcol = (lane >> 3) & 1;
    const int vkey = warp * kChunk + ((((lane >> 3) & 1) << 3) | (lane & 7)), vcol = lane >> 4;
    auto swz = [](int row, int col) { return static_cast<uint32_t>(row * 128 + (((col & 7) ^ (row & 7)) << 4)); };
    while (cur.left > 0) {
        if (cur.j < 0) {
            next(cur);
            continue;
        }
        // ---- a run of units of one sequence and head: this CTA's part of it
        const int b = cur.b, hr = cur.hr, j0 = cur.j, n = cur.n;
        const int j1 = min(n - j0, cur.left) + j0;
        const int rows = min(a.rows, a.group - (hr % a.rt) * 16);
        const bool any = cur.len > 0;
        const uint32_t qb = base + a.off_q + qs * L::QSLOT;
        auto free_q = [&] {
            __syncwarp();
            if (lane == 0) mbar_arrive(q_empty(qs));
            if (++qs == L::NQ) {
                qs = 0;
                qphase ^= 1u;
            }
        };
        uint32_t qf[D / 16][4];
        if (any && wait_full(q_full(qs), qphase)) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) ldsm4(qf[k], qb + (k / 4) * L::QATOM + swz(qrow, 2 * k + qcol));
            free_q();
        }
        float o[D / 8][4] = {};
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;   // rows g and g + 8
        for (int j = j0; j < j1; ++j, next(cur)) {
            if (!any) continue;
            const int nv = cur.len - j * kUnit - warp * kChunk;       // keys of this warp in use
            if (!wait_full(full(slot), phase)) continue;
            uint32_t p[4];
            if (nv > 0) {
                const uint32_t kb = base + slot * L::SLOT;
                float s[2][4] = {};
                {
                    // fragments are loaded kDeep steps ahead; even and odd steps add up apart
                    constexpr int kDeep = D <= 128 ? 4 : 2;
                    float s2[2][4] = {};
                    uint32_t f[kDeep][4];
                    auto load = [&](int k) { ldsm4(f[k % kDeep], kb + (k / 4) * L::ATOM + swz(kkey, 2 * k + kcol)); };
#pragma unroll
                    for (int k = 0; k < kDeep; ++k) load(k);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        mma16816<T>(k & 1 ? s2[0] : s[0], qf[k], f[k % kDeep][0], f[k % kDeep][1]);
                        mma16816<T>(k & 1 ? s2[1] : s[1], qf[k], f[k % kDeep][2], f[k % kDeep][3]);
                        if (k + kDeep < D / 16) load(k + kDeep);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[0][e] += s2[0][e];
                        s[1][e] += s2[1][e];
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[i][e] *= a.c;
                        if (8 * i + 2 * t + (e & 1) >= nv) s[i][e] = -INFINITY;
                    }
                float x0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
                float x1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
                constexpr float SH = Shift<T>::V;
                const bool up0 = x0 > m0 + (SH + kLag), up1 = x1 > m1 + (SH + kLag);
                if (__any_sync(0xffffffffu, up0 || up1)) {
                    const float n0 = up0 ? x0 - SH : m0, n1 = up1 ? x1 - SH : m1;
                    const float a0 = up0 ? ex2f(m0 - n0) : 1.0f, a1 = up1 ? ex2f(m1 - n1) : 1.0f;
                    m0 = n0;
                    m1 = n1;
                    l0 *= a0;
                    l1 *= a1;
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        o[i][0] *= a0;
                        o[i][1] *= a0;
                        o[i][2] *= a1;
                        o[i][3] *= a1;
                    }
                }
                const float r0 = m0 == -INFINITY ? 0.0f : m0, r1 = m1 == -INFINITY ? 0.0f : m1;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    s[i][0] = ex2f(s[i][0] - r0);
                    s[i][1] = ex2f(s[i][1] - r0);
                    s[i][2] = ex2f(s[i][2] - r1);
                    s[i][3] = ex2f(s[i][3] - r1);
                }
                l0 += (s[0][0] + s[0][1]) + (s[1][0] + s[1][1]);
                l1 += (s[0][2] + s[0][3]) + (s[1][2] + s[1][3]);
                // The weights rounded to T for the product with V, whose other operand has that type; the sums above are
                // of the unrounded ones.  It moves the output by as much as rounding it to T does (1.4 times the error
                // of the rounding alone, in all); carrying what is rounded off would take every product with V twice.
                p[0] = pack2<T>(s[0][0], s[0][1]);
                p[1] = pack2<T>(s[0][2], s[0][3]);
                p[2] = pack2<T>(s[1][0], s[1][1]);
                p[3] = pack2<T>(s[1][2], s[1][3]);
            }
            done();
            if (!wait_full(full(slot), phase)) continue;
            if (nv > 0) {
                const uint32_t vb = base + slot * L::SLOT;
                auto pv = [&](auto tail) {
                    // keys past the sequence's end: 0 x whatever lies in the page must be 0
                    const uint32_t k0 = tail ? (2 * t < nv ? 0xFFFFu : 0u) | (2 * t + 1 < nv ? 0xFFFF0000u : 0u) : 0u;
                    const uint32_t k1 = tail ? (2 * t + 8 < nv ? 0xFFFFu : 0u) | (2 * t + 9 < nv ? 0xFFFF0000u : 0u) : 0u;
                    constexpr int kDeep = D <= 128 ? 3 : 2;
                    uint32_t f[kDeep][4];
                    auto load = [&](int k) { ldsm4_t(f[k % kDeep], vb + (k / 4) * L::ATOM + swz(vkey, 2 * k + vcol)); };
#pragma unroll
                    for (int k = 0; k < kDeep; ++k) load(k);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        uint32_t (&r)[4] = f[k % kDeep];
                        if (tail) {
                            r[0] &= k0;
                            r[1] &= k1;
                            r[2] &= k0;
                            r[3] &= k1;
                        }
                        mma16816<T>(o[2 * k], p, r[0], r[1]);
                        mma16816<T>(o[2 * k + 1], p, r[2], r[3]);
                        if (k + kDeep < D / 16) load(k + kDeep);
                    }
                };
                if (nv >= kChunk) pv(std::false_type{});
                else pv(std::true_type{});
            }
            done();
        }
        // ---- the warps' parts
        l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
        l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
        const int buf = runs & 1;
        if (runs >= 2) wait_full(parts_free(buf), ((runs >> 1) - 1) & 1);
        float* omb = om + buf * (kOwnWarps * a.rows * D);
        float* mlb = ml + buf * (kOwnWarps * 32);
        if (ok) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                if (g < rows) *reinterpret_cast<float2*>(omb + (warp * a.rows + g) * D + 8 * i + 2 * t) = make_float2(o[i][0], o[i][1]);
                if (g + 8 < rows) *reinterpret_cast<float2*>(omb + (warp * a.rows + g + 8) * D + 8 * i + 2 * t) = make_float2(o[i][2], o[i][3]);
            }
            if (t == 0) {
                if (g < rows) *reinterpret_cast<float2*>(mlb + (warp * 16 + g) * 2) = make_float2(m0, l0);
                if (g + 8 < rows) *reinterpret_cast<float2*>(mlb + (warp * 16 + g + 8) * 2) = make_float2(m1, l1);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(parts_full(buf));
        if (runs > 0) join_before();
        before = Run{b, hr, j0, j1, n, buf};
        ++runs;
    }
    if (runs > 0) join_before();
}

// The prefix's items (row tiles of a key/value head) lie in one line and are cut into equal ranges, one per CTA:
// pent places that stand for what an item costs a CTA apart from its tiles (loading the query rows, filling and
// emptying the pipeline, writing its part), then a place per 128-key tile.  Measured with 0, 2, 4 and 6 of them:
// 256 sequences over 16384 shared keys (D = 128) 103.9, 101.7, 101.0 and 101.3 us, 8 over 2048 (D = 256) 54.4, 53.2,
// 52.6 and 49.2.  With at most a tile per CTA there is nothing to even out (pent = 0).
constexpr int kEntry = 6;
struct PrefixSeg {
    int item, t0, n;     // tiles t0 .. t0 + n - 1 of the item
};
// The next segment of places u .. u1 - 1, from which it is taken; false: none left.
__device__ __forceinline__ bool next_seg(const PagedArgs& a, int& u, int u1, PrefixSeg& s) {
    const int per = a.ptiles + a.pent;
    while (u < u1) {
        s.item = u / per;
        const int in = u - s.item * per, end = min(per, in + (u1 - u));
        u += end - in;
        s.t0 = max(in - a.pent, 0);
        s.n = end - a.pent - s.t0;
        if (s.n > 0) return true;
    }
    return false;
}

// With a shared prefix, the last step: the prefix's parts of a row and its own.  It is bound by latency: 48 rows per
// head and 8 heads take 6 us, 1024 rows per head 8.  One warp per query row, lane c
// taking D / 32 columns.
constexpr int kJoinThreads = 128;
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const __grid_constant__ PagedArgs a) {
    constexpr int W = D / 32;
    pdl_trigger();
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kJoinThreads / 32) + threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    if (row >= static_cast<int64_t>(a.batch) * a.hq) return;
    const int b = static_cast<int>(row / a.hq), h = static_cast<int>(row % a.hq);
    const int head = h / a.group, prow = b * a.group + h % a.group;
    const int rpi = a.prow;
    const int pit = head * a.prt + prow / rpi;
    const int64_t per = a.ptiles + a.pent, PU = a.hk * a.prt * per, u = pit * per + a.pent;
    const int c0 = cta_of(u, PU, a.pgrid), np = cta_of(u + a.ptiles - 1, PU, a.pgrid) - c0 + 1;
    pdl_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.ready = 0;
    // Lane 0 has what has been joined, lanes 1 .. kParts a part each: the prefix's, then the row's own.  The columns
    // of a batch are loaded next to its maxima and sums, so one memory latency is waited for, not three (two, where
    // the own parts have to be looked up; the prefix's are on their way by then).
    constexpr int kParts = 7;
    const int tile = h % a.group / 16, w = __ldcg(a.where + (b * a.hk + head) * a.rt + tile);
    // (after a wait that ran out `where` may hold anything: within the workspace all the same)
    const int o0 = w < 0 ? 0 : min(w & 0xffff, kOwnGrid - 1), own = w < 0 ? 1 : max(min(w >> 16, kOwnGrid - 1) - o0 + 1, 1), all = own + np;
    auto load = [&](float (&v)[W], const float* src) {
        if constexpr (W == 2) {
            const float2 x = __ldcg(reinterpret_cast<const float2*>(src));
            v[0] = x.x;
            v[1] = x.y;
        } else {
#pragma unroll
            for (int e = 0; e < W; e += 4) {
                const float4 x = __ldcg(reinterpret_cast<const float4*>(src + e));
                v[e] = x.x;
                v[e + 1] = x.y;
                v[e + 2] = x.z;
                v[e + 3] = x.w;
            }
        }
    };
    float m = -INFINITY, l = 0.0f, acc[W] = {};
    const int64_t pre0 = static_cast<int64_t>(c0 + pit) * rpi + prow % rpi;          // the prefix's parts are rpi rows apart
    auto own_at = [&](int p) { return static_cast<int64_t>(2 * (o0 + p) + (p == 0 ? 1 : 0)) * a.rows + h % a.group % 16; };
    for (int p0 = 0; p0 < all; p0 += kParts) {
        float v[kParts][W];
#pragma unroll
        for (int c = 0; c < kParts; ++c) {
            if (p0 + c < np) load(v[c], a.po + (pre0 + static_cast<int64_t>(rpi) * (p0 + c)) * D + W * lane);
            else load(v[c], (w < 0 ? a.ro + row * D : a.oo + own_at(min(p0 + c, all - 1) - np) * D) + W * lane);
        }
        float pm = lane == 0 ? m : -INFINITY, pl = lane == 0 ? l : 0.0f;
        const int p = p0 + lane - 1;
        if (lane >= 1 && lane <= kParts && p < np) {
            const float4 x = __ldcg(reinterpret_cast<const float4*>(a.pml + (pre0 + static_cast<int64_t>(rpi) * p) * 4));
            pm = x.x;
            pl = x.y + x.z;
        } else if (lane >= 1 && lane <= kParts && p < all) {
            const float2 x = __ldcg(reinterpret_cast<const float2*>(w < 0 ? a.rml + row * 2 : a.oml + own_at(p - np) * 2));
            pm = x.x;
            pl = x.y;
        }
        float top = pm;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float e = pm == -INFINITY ? 0.0f : ex2f(pm - top);
        float sum = pl * e;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float e0 = __shfl_sync(0xffffffffu, e, 0);
#pragma unroll
        for (int i = 0; i < W; ++i) acc[i] *= e0;
#pragma unroll
        for (int c = 0; c < kParts; ++c) {
            const float ec = __shfl_sync(0xffffffffu, e, c + 1);
            if (p0 + c < all)
#pragma unroll
                for (int i = 0; i < W; ++i) acc[i] += ec * v[c][i];
        }
        m = top;
        l = sum;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    T* dst = static_cast<T*>(a.o) + row * D + W * lane;
#pragma unroll
    for (int e = 0; e < W; e += 2)
        *reinterpret_cast<uint32_t*>(dst + e) = l == 0.0f ? 0u : pack2<T>(acc[e] * inv, acc[e + 1] * inv);
}

// ================================================================== the shared prefix
constexpr int kPreSoftmaxWarps = 8;                       // two per TMEM lane quadrant
constexpr int kPreThreads = 32 * (3 + kPreSoftmaxWarps);  // warp 0: K, 1: MMA issue, 2: V, 3-10: softmax

template <int D>
struct PrefixLayout {
    static constexpr int ATOMS = D / 64;
    static constexpr int KV = D == 64 ? 4 : D == 128 ? 2 : 1;  // K and V stages
    static constexpr uint32_t REGION = 128 * 128;              // one 64-column atom of 128 rows
    static constexpr uint32_t TILE = REGION * ATOMS;           // Q, K or V: 128 rows x D
    static constexpr uint32_t P_BYTES = 128 * 128 * 2;
    static constexpr uint32_t OFF_Q = 0;
    static constexpr uint32_t OFF_K = TILE;
    static constexpr uint32_t OFF_V = OFF_K + KV * TILE;
    static constexpr uint32_t OFF_P = OFF_V + KV * TILE;
    static constexpr uint32_t OFF_BAR = OFF_P + P_BYTES;
    static constexpr int N_BARS = 2 + 4 * KV + 2 + 4;
    static constexpr uint32_t OFF_HOLD = OFF_BAR + N_BARS * 8;
    static constexpr uint32_t SMEM = OFF_HOLD + 16 + 1024;
    static constexpr uint32_t TMEM_COLS = 512, O_COL = 256;    // two 128-column score buffers, then O
    static_assert(SMEM <= 232448, "shared-memory budget");
    static_assert(SMEM > 116 * 1024, "one CTA per SM: each takes all of TMEM");
};

// A whole 32-byte sector per thread.
__device__ __forceinline__ void st_v8(float* p, const float* v) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])),
                 "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
                 "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
                 : "memory");
}

// Query rows qrow0 .. qrow0 + 127 of a key/value head into a swizzled tile, by THREADS threads (tid their number).
// Row x of a head is query head `head * group + x % group` of sequence x / group; rows past the batch are zeros.
// All of a thread's loads are under way before the first is stored: one at a time, they took 10 us of a call.
template <typename T, int D, int THREADS>
__device__ __forceinline__ void load_q_tile(uint8_t* tile, int head, int qrow0, int tid, const PagedArgs& a) {
    constexpr int PER = 128 * (D / 8) / THREADS, STEP = THREADS / (D / 8);   // vectors of a thread, rows apart
    uint4 x[PER];
    // Opaque copies: what depends on them is computed here, not kept in registers between the tiles (which spills)
    int group = a.group;
    asm volatile("" : "+r"(tid), "+r"(group));
    int row = qrow0 + tid / (D / 8);
    const int b = row / group, step_b = STEP / group, step_g = STEP - step_b * group;      // no division per vector
    int g = row - b * group;
    const uint4* at = static_cast<const uint4*>(a.q) + ((static_cast<int64_t>(b) * a.hq + head * group + g) * (D / 8) + tid % (D / 8));
    const int64_t step = (static_cast<int64_t>(step_b) * a.hq + step_g) * (D / 8), wrap = static_cast<int64_t>(a.hq - group) * (D / 8);
    const int rows = a.batch * group;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        x[i] = row < rows ? __ldcg(at) : make_uint4(0u, 0u, 0u, 0u);
        row += STEP;
        at += step;
        g += step_g;
        if (g >= group) {
            g -= group;
            at += wrap;
        }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int v = tid + i * THREADS, k = v / (D / 8), ch = v % (D / 8);
        *reinterpret_cast<uint4*>(tile + (ch / 8) * (128 * 128) + k * 128 + (((ch % 8) ^ (k & 7)) << 4)) = x[i];
    }
}

// Loads 128-key K or V tiles, by one warp.  A tile is 128 / box boxes of one page each.
template <int D>
struct PrefixLoader {
    const PagedArgs& a;
    const int lane, box_shift;
    const uint32_t one;
    int head = 0, page = 0;
    __device__ __forceinline__ PrefixLoader(const PagedArgs& args, int l)
        : a(args), lane(l), box_shift(min(args.page_shift, 7)), one(elect_one()) {}
    // Read this lane's page of a tile from the table; load() uses it.
    __device__ __forceinline__ void look(int tile) {
        const int key = tile * 128 + (lane << box_shift);
        if (lane << box_shift < 128 && key < a.plen) page = a.ptable[key >> a.page_shift];
    }
    __device__ __forceinline__ void load(const CUtensorMap* map, uint32_t dst, uint32_t full, int tile) {
        const int nk = min(128, a.plen - tile * 128), nbox = (nk + (1 << box_shift) - 1) >> box_shift;
        int row = a.cache_rows;         // past the cache: zeros
        if (lane < nbox) {
            const int key = tile * 128 + (lane << box_shift);
            if (page >= 0 && page < a.num_pages)
                row = ((page * a.hk + head) << a.page_shift) + (key & ((1 << a.page_shift) - 1));
            else
                atomicExch(a.bad, 1);
        }
        if (lane == 0) mbar_arrive_expect_tx(full, static_cast<uint32_t>(nbox << box_shift) * (D * 2));
        __syncwarp();
        for (int y = 0; y < nbox; ++y) {
            const int r = __shfl_sync(0xffffffffu, row, y);
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
                tma_load_2d_if(one, dst + c * (128 * 128) + ((static_cast<uint32_t>(y) << box_shift) * 128), map, 64 * c, r, full);
        }
    }
};

// One CTA per SM walks an equal run of (128-row tile of a key/value head, 128-key tile) pairs.  Per row
// tile it loads Q (rows b * group + i of the head), then S_j = Q K_j^T into one of two TMEM buffers while
// the softmax warps work on the other, P_j = 2^(S_j c - m) into shared memory, O += P_j V_j in TMEM, and
// at the end of the run it writes (m, l, O) as the run's part.
template <typename T, int D>
__global__ void __launch_bounds__(kPreThreads, 1) paged_prefix_kernel(const __grid_constant__ CUtensorMap mK,
                                                                      const __grid_constant__ CUtensorMap mV,
                                                                      const __grid_constant__ PagedArgs a) {
    using L = PrefixLayout<D>;
    constexpr bool BF = std::is_same<T, __nv_bfloat16>::value;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - smem_addr(smem_raw));
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    constexpr int KV = L::KV;
    const uint32_t bar0 = base + L::OFF_BAR;
    // A ring of n buffers used by tiles i = 0, 1, ... of this CTA: buffer i % n, parity (i / n) & 1.
    const uint32_t q_full = bar0, drain = bar0 + 8;
    auto k_full = [&](int i) { return bar0 + 8u * (2 + i); };
    auto k_empty = [&](int i) { return bar0 + 8u * (2 + KV + i); };
    auto v_full = [&](int i) { return bar0 + 8u * (2 + 2 * KV + i); };
    auto v_empty = [&](int i) { return bar0 + 8u * (2 + 3 * KV + i); };
    const uint32_t p_full = bar0 + 8u * (2 + 4 * KV), o_done = p_full + 8;
    auto s_full = [&](int i) { return bar0 + 8u * (4 + 4 * KV + i); };
    auto s_free = [&](int i) { return bar0 + 8u * (6 + 4 * KV + i); };
    int* flag = a.flag;
    if (threadIdx.x == 0) {
        mbar_init(q_full, kPreSoftmaxWarps);
        mbar_init(drain, 1);
        for (int i = 0; i < KV; ++i) {
            mbar_init(k_full(i), 1);
            mbar_init(k_empty(i), 1);
            mbar_init(v_full(i), 1);
            mbar_init(v_empty(i), 1);
        }
        mbar_init(p_full, kPreSoftmaxWarps);
        mbar_init(o_done, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full(i), 1);
            mbar_init(s_free(i), kPreSoftmaxWarps);
        }
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(base + L::OFF_HOLD, L::TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(gbase + L::OFF_HOLD), 0);
    pdl_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) st_release_gpu(a.ready, 1);
    pdl_trigger();   // only now: paged_own_kernel relies on it

    const int64_t U = static_cast<int64_t>(a.hk) * a.prt * (a.ptiles + a.pent);     // below 2^31
    const int u0 = static_cast<int>(blockIdx.x * U / gridDim.x), u1 = static_cast<int>((blockIdx.x + 1) * U / gridDim.x);
    auto keys_of = [&](int tile) { return min(128, a.plen - tile * 128); };

    if (warp == 0 || warp == 2) {
        // ---------------------------------------------------------------- K loads; V loads
        const bool is_k = warp == 0;
        const CUtensorMap* map = is_k ? &mK : &mV;
        if (lane == 0) prefetch_map(map);
        PrefixLoader<D> ld(a, lane);
        int i = 0;
        bool ok = true;
        PrefixSeg seg;
        for (int u = u0; ok && next_seg(a, u, u1, seg);) {
            ld.head = seg.item / a.prt;
            for (int j = 0; j < seg.n; ++j, ++i) {
                const int tile = seg.t0 + j, st = i % KV;
                ld.look(tile);
                ok = i < KV || __all_sync(0xffffffffu, mbar_wait_bounded(is_k ? k_empty(st) : v_empty(st), ((i - KV) / KV) & 1, flag));
                if (!ok) break;
                ld.load(map, base + (is_k ? L::OFF_K : L::OFF_V) + st * L::TILE, is_k ? k_full(st) : v_full(st), tile);
            }
        }
        if (!ok)   // copies in flight land before the shared memory goes away
            for (int j = max(0, i - KV); j < i; ++j) (void)mbar_wait_drain(is_k ? k_full(j % KV) : v_full(j % KV), (j / KV) & 1);
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issue
        constexpr uint32_t idS = idesc_f16(128, 128, false, false, BF);
        constexpr uint32_t idO = idesc_f16(128, D, false, true, BF);
        const uint32_t one = elect_one();
        const uint64_t dq = smem_desc_sw128(base + L::OFF_Q, 16, 1024), dk = smem_desc_sw128(base + L::OFF_K, 16, 1024);
        const uint64_t dp = smem_desc_sw128(base + L::OFF_P, 16, 1024), dv = smem_desc_sw128(base + L::OFF_V, L::REGION, 1024);
        bool issued = false, ok = true;
        auto wait = [&](uint32_t bar, uint32_t parity) {
            ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity & 1u, flag));
            return ok;
        };
        auto issue_s = [&](int i) {
            const int st = i % KV, sb = i & 1;
            if (!wait(k_full(st), i / KV)) return;
            if (i >= 2 && !wait(s_free(sb), (i >> 1) - 1)) return;
            tc_fence_after();
            const uint64_t kd = dk + static_cast<uint64_t>(st * (L::TILE >> 4));
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
                tc_mma_if(one, tmem + sb * 128, dq + ((s / 4) * (L::REGION >> 4) + (s % 4) * 2), kd + ((s / 4) * (L::REGION >> 4) + (s % 4) * 2),
                          idS, s > 0 ? 1u : 0u);
            tc_commit_if(one, s_full(sb));
            tc_commit_if(one, k_empty(st));
            issued = true;
        };
        auto issue_pv = [&](int i, bool first) {
            const int st = i % KV;
            if (!wait(p_full, i) || !wait(v_full(st), i / KV)) return;
            tc_fence_after();
            const uint64_t vd = dv + static_cast<uint64_t>(st * (L::TILE >> 4));
#pragma unroll
            for (int s = 0; s < 8; ++s)   // 16 keys each: P atom s / 4; V rows 16 s ..
                tc_mma_if(one, tmem + L::O_COL, dp + ((s / 4) * (L::REGION >> 4) + (s % 4) * 2), vd + s * (2048 >> 4), idO,
                          !first || s > 0 ? 1u : 0u);
            tc_commit_if(one, o_done);
            tc_commit_if(one, v_empty(st));
            issued = true;
        };
        int i = 0, segs = 0;
        PrefixSeg seg;
        for (int u = u0; ok && next_seg(a, u, u1, seg); ++segs) {
            const int n = seg.n;
            if (!wait(q_full, segs)) break;
            issue_s(i);
            for (int j = 0; ok && j < n; ++j) {
                if (j + 1 < n) issue_s(i + j + 1);
                if (ok) issue_pv(i + j, j == 0);
            }
            i += n;
        }
        if (!ok && issued) {   // MMAs in flight finish before TMEM is freed
            tc_commit_if(one, drain);
            (void)mbar_wait_drain(drain, 0);
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- softmax
        // Warp w serves TMEM lane quadrant w % 4 (query rows 32 (w % 4) + lane) and half hh of each tile's
        // keys and of O's columns; both warps of a quadrant read the whole score row for its maximum.
        const int qd = warp % 4, hh = (warp - 3) / 4, r = 32 * qd + lane;
        const uint32_t lanes = static_cast<uint32_t>(32 * qd) << 16;
        const int sid = (warp - 3) * 32 + lane;     // 0..255
        const int total_rows = a.batch * a.group;
        constexpr float SH = Shift<T>::V;
        constexpr int HK = 64;
        bool ok = true;
        int i = 0;
        PrefixSeg seg;
        for (int u = u0; ok && next_seg(a, u, u1, seg);) {
            const int item = seg.item, t0 = seg.t0, n = seg.n;
            const int head = item / a.prt, qrow0 = (item % a.prt) * 128;
            // The MMAs that read the previous tile's Q have completed (its last O was waited for).
            load_q_tile<T, D, 32 * kPreSoftmaxWarps>(gbase + L::OFF_Q, head, qrow0, sid, a);
            fence_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
            float m = -INFINITY, l = 0.0f;
            for (int j = 0; j < n; ++j, ++i) {
                const int sb = i & 1, nk = keys_of(t0 + j);
                if (!__all_sync(0xffffffffu, mbar_wait_bounded(s_full(sb), (i / 2) & 1, flag))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                float s[HK], so[HK];
                const uint32_t sbase = tmem + lanes + sb * 128;
#pragma unroll
                for (int k = 0; k < HK / 32; ++k) {
                    tmem_ld32(sbase + HK * hh + 32 * k, s + 32 * k);
                    tmem_ld32(sbase + HK * (1 - hh) + 32 * k, so + 32 * k);
                }
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_free(sb));
                if (nk < 128) {   // keys past the prefix's end
                    const int ts = nk - HK * hh, to = nk - HK * (1 - hh);
#pragma unroll
                    for (int k = 0; k < HK; ++k) {
                        s[k] = k >= ts ? -INFINITY : s[k];
                        so[k] = k >= to ? -INFINITY : so[k];
                    }
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int k = 0; k < HK; ++k) mx[k & 3] = max3f(mx[k & 3], s[k], so[k]);
                const float x = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.c;
                float alpha = 1.0f;
                bool rescale = false;
                if (x > m + (SH + kLag)) {
                    if (j > 0) {
                        alpha = ex2f(m - (x - SH));
                        rescale = true;
                    }
                    m = x - SH;
                }
                const float ref = m == -INFINITY ? 0.0f : m;
                uint32_t pk[HK / 2];     // the weights rounded to T, as in paged_own_kernel
                const float2 c2 = make_float2(a.c, a.c), nm2 = make_float2(-ref, -ref);
                float2 sum2 = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int k = 0; k < HK; k += 2) {
                    const float2 e = __ffma2_rn(make_float2(s[k], s[k + 1]), c2, nm2);
                    const float2 p = make_float2(ex2f(e.x), ex2f(e.y));
                    sum2 = __fadd2_rn(sum2, p);
                    pk[k / 2] = pack2<T>(p.x, p.y);
                }
                l = l * alpha + (sum2.x + sum2.y);
                // P and O are free once the previous tile's PV has completed
                if (i > 0 && !__all_sync(0xffffffffu, mbar_wait_bounded(o_done, (i - 1) & 1, flag))) {
                    ok = false;
                    break;
                }
                if (__any_sync(0xffffffffu, rescale)) {
                    tc_fence_after();
#pragma unroll 1
                    for (int k = 0; k < D / 64; ++k) {
                        const uint32_t col = L::O_COL + (D / 2) * hh + 32 * k;
                        float o[32];
                        tmem_ld32(tmem + lanes + col, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= alpha;
                        tmem_st32(tmem + lanes + col, o);
                    }
                    tmem_st_wait();
                }
                uint8_t* prow = gbase + L::OFF_P + r * 128;
#pragma unroll
                for (int q = 0; q < HK / 8; ++q) {
                    const int ch = (HK / 8) * hh + q;
                    *reinterpret_cast<uint4*>(prow + (ch / 8) * L::REGION + (((ch % 8) ^ (r & 7)) << 4)) =
                        make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
                }
                if (nk < 128) {   // V rows past the end: 0 x whatever lies there must be 0
                    const int st = i % KV;
                    if (!__all_sync(0xffffffffu, mbar_wait_bounded(v_full(st), (i / KV) & 1, flag))) {
                        ok = false;
                        break;
                    }
                    uint8_t* vb = gbase + L::OFF_V + st * L::TILE;
                    for (int v = sid; v < (128 - nk) * L::ATOMS * 8; v += 32 * kPreSoftmaxWarps) {
                        const int row = nk + v / (L::ATOMS * 8), c = v % (L::ATOMS * 8);
                        *reinterpret_cast<uint4*>(vb + (c / 8) * L::REGION + row * 128 + (c % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                fence_async_smem();   // the generic-proxy writes become visible to the tensor core
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full);
            }
            if (ok && !__all_sync(0xffffffffu, mbar_wait_bounded(o_done, (i - 1) & 1, flag))) ok = false;
            if (ok) {
                tc_fence_after();
                const int64_t at = (static_cast<int64_t>(blockIdx.x) + item) * 128 + r;
                const bool in = qrow0 + r < total_rows;
                if (in) {
                    if (hh == 0) *reinterpret_cast<float2*>(a.pml + at * 4) = make_float2(m, l);
                    else a.pml[at * 4 + 2] = l;
                }
                float* dst = a.po + at * D + (D / 2) * hh;
#pragma unroll 1
                for (int k = 0; k < D / 64; ++k) {
                    float o[32];
                    tmem_ld32(tmem + lanes + L::O_COL + (D / 2) * hh + 32 * k, o);
                    tmem_ld_wait();
                    if (in)
#pragma unroll
                        for (int e = 0; e < 4; ++e) st_v8(dst + 32 * k + 8 * e, o + 8 * e);
                }
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

// ------------------------------------------------------------------ two row tiles at a time
// For more than 128 rows per key/value head and D <= 128: the CTA holds two row tiles (256 rows) against the
// same K and V tiles, so every K and V byte serves twice as many rows, and while the softmax warps of one row
// tile wait for the tensor core, those of the other work.  One softmax thread per row takes its 128 scores into
// registers and gives the score buffer back at once, so S_t(j + 1) is computed while the thread works on
// S_t(j).  P goes through shared memory.  K and V tiles share one ring of three tiles in the order of their use,
// K(0) K(1) V(0) K(2) V(1) ...; one warp issues S_0(j), S_1(j), the next step's and so on, another the PVs, and the
// row tiles fall half a step apart by themselves.
// (P in TMEM over the scores it was made from, which leaves room for two stages of K and of V: S_t(j + 1) then
// waits for PV_t(j), and a step of 256 x 128 took 3000 cycles.)
template <int D>
struct Prefix2Layout {
    static constexpr int ATOMS = D / 64;
    static constexpr int RING = D == 64 ? 6 : 3;               // K and V tiles
    static constexpr uint32_t REGION = 128 * 128;
    static constexpr uint32_t TILE = REGION * ATOMS;
    static constexpr uint32_t P_BYTES = 128 * 128 * 2;
    static constexpr uint32_t OFF_Q = 0;                       // two tiles
    static constexpr uint32_t OFF_KV = 2 * TILE;
    static constexpr uint32_t OFF_P = OFF_KV + RING * TILE;    // two tiles
    static constexpr uint32_t OFF_BAR = OFF_P + 2 * P_BYTES;
    static constexpr int N_BARS = 2 + 2 * RING + 10;
    static constexpr uint32_t OFF_HOLD = OFF_BAR + N_BARS * 8;
    static constexpr uint32_t SMEM = OFF_HOLD + 16 + 1024;
    static constexpr uint32_t TMEM_COLS = 512, O_COL = 256;    // scores of tile t at 128 t, output at 256 + D t
    static_assert(SMEM <= 232448, "shared-memory budget");
    static_assert(SMEM > 116 * 1024, "one CTA per SM: each takes all of TMEM");
};

template <typename T, int D>
__global__ void __launch_bounds__(kPreThreads, 1) paged_prefix2_kernel(const __grid_constant__ CUtensorMap mK,
                                                                       const __grid_constant__ CUtensorMap mV,
                                                                       const __grid_constant__ PagedArgs a) {
    using L = Prefix2Layout<D>;
    constexpr bool BF = std::is_same<T, __nv_bfloat16>::value;
    constexpr int RING = L::RING;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - smem_addr(smem_raw));
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    const uint32_t bar0 = base + L::OFF_BAR;
    const uint32_t q_full = bar0;
    auto drain = [&](int w) { return bar0 + 8u * (10 + 2 * RING + w); };     // of warps 1 and 2
    auto full = [&](int i) { return bar0 + 8u * (1 + i); };
    auto empty = [&](int i) { return bar0 + 8u * (1 + RING + i); };
    auto s_full = [&](int t) { return bar0 + 8u * (2 + 2 * RING + t); };
    auto s_free = [&](int t) { return bar0 + 8u * (4 + 2 * RING + t); };
    auto p_full = [&](int t) { return bar0 + 8u * (6 + 2 * RING + t); };
    auto o_done = [&](int t) { return bar0 + 8u * (8 + 2 * RING + t); };
    int* flag = a.flag;
    if (threadIdx.x == 0) {
        mbar_init(q_full, kPreSoftmaxWarps);
        mbar_init(drain(0), 1);
        mbar_init(drain(1), 1);
        for (int i = 0; i < RING; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(s_full(t), 1);
            mbar_init(s_free(t), kPreSoftmaxWarps / 2);
            mbar_init(p_full(t), kPreSoftmaxWarps / 2);
            mbar_init(o_done(t), 1);
        }
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(base + L::OFF_HOLD, L::TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(gbase + L::OFF_HOLD), 0);
    pdl_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) st_release_gpu(a.ready, 1);
    pdl_trigger();   // only now: paged_own_kernel relies on it

    const int64_t U = static_cast<int64_t>(a.hk) * a.prt * (a.ptiles + a.pent);     // below 2^31
    const int u0 = static_cast<int>(blockIdx.x * U / gridDim.x), u1 = static_cast<int>((blockIdx.x + 1) * U / gridDim.x);
    // Place of K tile j and V tile j of a segment of n in the segment's loads: K(0), then K(j + 1) before V(j).
    auto k_at = [](int j) { return j == 0 ? 0 : 2 * j - 1; };
    auto v_at = [](int j, int n) { return j + 1 < n ? 2 * j + 2 : 2 * j + 1; };

    if (warp == 0) {
        // ---------------------------------------------------------------- K and V loads
        if (lane == 0) {
            prefetch_map(&mK);
            prefetch_map(&mV);
        }
        PrefixLoader<D> ld(a, lane);
        int c = 0, slot = 0;             // loads so far, and the next one's slot
        uint32_t phase = 1;              // of the wait for it to be empty
        bool ok = true;
        PrefixSeg seg;
        for (int u = u0; ok && next_seg(a, u, u1, seg);) {
            const int t0 = seg.t0, n = seg.n;
            ld.head = seg.item / a.prt;
            for (int x = 0; x < 2 * n; ++x, ++c) {
                // x-th load of the segment: K for 0 and odd x below 2 n - 1, V for the others
                const bool is_k = x == 0 || (x % 2 == 1 && x < 2 * n - 1);
                const int j = is_k ? (x + 1) / 2 : (x == 2 * n - 1 ? n - 1 : x / 2 - 1);
                ld.look(t0 + j);
                if (c >= RING) {
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(empty(slot), phase, flag));
                    if (!ok) break;
                }
                ld.load(is_k ? &mK : &mV, base + L::OFF_KV + slot * L::TILE, full(slot), t0 + j);
                if (++slot == RING) {
                    slot = 0;
                    phase ^= 1u;
                }
            }
        }
        if (!ok)   // copies in flight land before the shared memory goes away
            for (int j = max(0, c - RING); j < c; ++j) (void)mbar_wait_drain(full(j % RING), (j / RING) & 1);
        __syncwarp();
    } else if (warp < 3) {
        // ---------------------------------------------------------------- MMA issue: S by warp 1, PV by warp 2
        // One warp for both took 3150 cycles for a step whose MMAs take 2270: each of its waits, even for what had long
        // happened, left the tensor core idle for 150 to 200 cycles (16384 keys, 1024 rows of 8 heads: 59 us, with
        // two warps 49, 1.4 PFLOP/s).
        // The order of the waits matters: K and V tiles take turns in a ring slot, and a wait for a slot's use u tells
        // it from use u - 2 by parity alone, so use u - 1, which may be the other warp's, must be known to have
        // landed.  S(j) knows by s_free(j - 1): the thread that took S(j - 1) has stored P(j - 2) before, for which
        // it waited for PV(j - 3), so V(j - 3) has landed (and q_full says so of the segments before).  PV(j) knows
        // by p_full(j): S(j) is done, so K(j) and the tiles before it have landed.
        const uint32_t one = elect_one();
        bool issued = false, ok = true;
        auto wait = [&](uint32_t bar, uint32_t parity) {
            ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity & 1u, flag));
            return ok;
        };
        int i = 0, c = 0, segs = 0;      // steps and loads of the segments before this one, their number
        PrefixSeg seg;
        if (warp == 1) {
            constexpr uint32_t idS = idesc_f16(128, 128, false, false, BF);
            const uint64_t dq = smem_desc_sw128(base + L::OFF_Q, 16, 1024), dk = smem_desc_sw128(base + L::OFF_KV, 16, 1024);
            for (int u = u0; ok && next_seg(a, u, u1, seg); ++segs, i += seg.n, c += 2 * seg.n) {
                if (!wait(q_full, segs)) break;
                for (int j = 0; ok && j < seg.n; ++j) {
                    const int ck = c + k_at(j), slot = ck % RING;
                    const uint64_t kd = dk + static_cast<uint64_t>(slot * (L::TILE >> 4));
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (i + j > 0 && !wait(s_free(t), i + j - 1)) break;
                        if (t == 0 && !wait(full(slot), ck / RING)) break;
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
            }
        } else {
            constexpr uint32_t idO = idesc_f16(128, D, false, true, BF);
            const uint64_t dp = smem_desc_sw128(base + L::OFF_P, 16, 1024), dv = smem_desc_sw128(base + L::OFF_KV, L::REGION, 1024);
            for (int u = u0; ok && next_seg(a, u, u1, seg); i += seg.n, c += 2 * seg.n) {
                for (int j = 0; ok && j < seg.n; ++j) {
                    const int cv = c + v_at(j, seg.n), slot = cv % RING;
                    const uint64_t vd = dv + static_cast<uint64_t>(slot * (L::TILE >> 4));
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (!wait(p_full(t), i + j)) break;
                        if (t == 0 && !wait(full(slot), cv / RING)) break;
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
            }
        }
        if (!ok && issued) {   // MMAs in flight finish before TMEM is freed
            tc_commit_if(one, drain(warp - 1));
            (void)mbar_wait_drain(drain(warp - 1), 0);
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- softmax: thread r of tile t, one row
        const int t = (warp - 3) / 4, r = 32 * (warp % 4) + lane;
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp % 4)) << 16;
        const uint32_t st = tmem + lanes + t * 128, ot = tmem + lanes + L::O_COL + t * D;
        constexpr float SH = Shift<T>::V;
        bool ok = true;
        auto wait = [&](uint32_t bar, uint32_t parity) {
            ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity & 1u, flag));
            return ok;
        };
        int i = 0;
        PrefixSeg seg;
        for (int u = u0; ok && next_seg(a, u, u1, seg);) {
            const int item = seg.item, n = seg.n;
            int left = a.plen - seg.t0 * 128;        // keys from the tile on
            // this tile's Q, by its own warps: the MMAs that read the last one have completed
            load_q_tile<T, D, 32 * kPreSoftmaxWarps / 2>(gbase + L::OFF_Q + t * L::TILE, item / a.prt, item % a.prt * 256 + t * 128, r, a);
            fence_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
            float m = -INFINITY, l = 0.0f;
            for (int j = 0; j < n; ++j, ++i, left -= 128) {
                if (!wait(s_full(t), i)) break;
                tc_fence_after();
                float x[128];
#pragma unroll
                for (int k = 0; k < 4; ++k) tmem_ld32(st + 32 * k, x + 32 * k);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_free(t));
                if (left < 128) {        // keys past the prefix's end
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
                    uint32_t w[4];       // the weights rounded to T, as in paged_own_kernel
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
                if (left < 128 && t == 0) {   // V rows past the end: 0 x whatever lies there must be 0
                    const int cv = 2 * (i - j) + v_at(j, n);      // (row tile 1's PV is issued after row tile 0's)
                    if (!wait(full(cv % RING), cv / RING)) break;
                    uint8_t* vb = gbase + L::OFF_KV + (cv % RING) * L::TILE;
                    for (int v = r; v < (128 - left) * L::ATOMS * 8; v += 128) {
                        const int row = left + v / (L::ATOMS * 8), ch = v % (L::ATOMS * 8);
                        *reinterpret_cast<uint4*>(vb + (ch / 8) * L::REGION + row * 128 + (ch % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                fence_async_smem();      // the generic-proxy writes become visible to the tensor core
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full(t));
            }
            if (ok && wait(o_done(t), i - 1)) {
                tc_fence_after();
                const int64_t at = (static_cast<int64_t>(blockIdx.x) + item) * 256 + t * 128 + r;
                const bool in = item % a.prt * 256 + t * 128 + r < a.batch * a.group;
                if (in) *reinterpret_cast<float4*>(a.pml + at * 4) = make_float4(m, l, 0.0f, 0.0f);
                float* dst = a.po + at * D;
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
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, L::TMEM_COLS);
    }
}

// ================================================================== host side
// Rows of the prefix kernel's items: two tiles where there are more rows than one tile's and TMEM holds two outputs
// next to two tiles of scores.
int64_t prefix_rows(int64_t rows, int64_t D) { return rows > 128 && D <= 128 ? 256 : 128; }

struct Sizes {
    int64_t rows, prow, pitems;      // rows per part of own keys; of the prefix, and its items
    size_t count, oml, oo, where, rml, ro, pml, po;  // byte offsets of the workspace's parts
    size_t bytes;
};
Sizes sizes(int64_t batch, int64_t hq, int64_t hk, int64_t D, int64_t plen) {
    Sizes s{};
    const int64_t group = hq / hk;
    s.rows = group < 16 ? group : 16;
    s.prow = prefix_rows(batch * group, D);
    s.pitems = plen > 0 ? hk * ceil_div(batch * group, s.prow) : 0;
    size_t at = 0;
    auto part = [&](int64_t n) {
        const size_t was = at;
        at += (static_cast<size_t>(n) + 255) / 256 * 256;
        return was;
    };
    s.count = part(kCounterBytes);   // at the same place whatever the sizes
    s.oml = part(2 * kOwnGrid * s.rows * 8);
    s.oo = part(2 * kOwnGrid * s.rows * D * 4);
    if (plen > 0) {
        s.where = part(batch * hk * ceil_div(group, 16) * 4);
        s.rml = part(batch * hq * 8);
        s.ro = part(batch * hq * D * 4);
        s.pml = part((kPrefixGrid + s.pitems) * s.prow * 16);
        s.po = part((kPrefixGrid + s.pitems) * s.prow * D * 4);
    }
    s.bytes = at;
    return s;
}

// Ring slots, shared memory and CTAs per SM of paged_own_kernel: two CTAs with 64 KB of loads in flight each
// where that fits, else one with as many as fit.
template <int D>
int own_smem(PagedArgs* a, uint32_t* bytes, int* ctas) {
    using L = OwnLayout<D>;
    const uint32_t om = static_cast<uint32_t>(2 * kOwnWarps * a->rows * D * 4), ml = 2 * kOwnWarps * 16 * 8;
    const uint32_t bars = 8u * (2 * kOwnSlots + 2 * L::NQ + 4);
    const uint32_t pre = static_cast<uint32_t>(2 * a->batch + 1) * 4, q = L::NQ * L::QSLOT;
    const uint32_t fixed = q + om + ml + bars + pre + 1024;
    int n = 0;
    for (*ctas = L::CTAS;; --*ctas) {
        const uint32_t budget = *ctas == 2 ? 112u * 1024u : static_cast<uint32_t>(kOwnSmem);
        n = fixed < budget ? static_cast<int>((budget - fixed) / L::SLOT) : 0;
        if (n * L::SLOT >= 64u * 1024u || *ctas == 1) break;
    }
    if (n < 1) return FUSE_EUNSUPPORTED;
    a->slots = n < kOwnSlots ? n : kOwnSlots;
    a->off_q = a->slots * L::SLOT;
    a->off_om = a->off_q + q;
    a->off_ml = a->off_om + om;
    a->off_bar = a->off_ml + ml;
    a->off_pre = a->off_bar + bars;
    *bytes = a->off_pre + pre + 1024;
    return FUSE_OK;
}

// What the report gives as shared memory of paged_own_kernel: a launch's for one sequence and groups of four heads.
template <int D>
int own_report_smem() {
    PagedArgs a{};
    a.batch = 1;
    a.rows = 4;
    uint32_t bytes = 0;
    int ctas = 0;
    return own_smem<D>(&a, &bytes, &ctas) == FUSE_OK ? static_cast<int>(bytes) : 0;
}

template <typename T, int D>
int prefix_opt_in(const PagedArgs& a) {
    if constexpr (D <= 128)
        if (a.prow == 256) return opt_in_smem((const void*)paged_prefix2_kernel<T, D>, Prefix2Layout<D>::SMEM);
    return opt_in_smem((const void*)paged_prefix_kernel<T, D>, PrefixLayout<D>::SMEM);
}

template <typename T, int D>
int launch_prefix(const CUtensorMap& mK, const CUtensorMap& mV, const PagedArgs& a, cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>(a.pgrid));
    if constexpr (D <= 128)
        if (a.prow == 256) return launch_pdl(paged_prefix2_kernel<T, D>, grid, dim3(kPreThreads), Prefix2Layout<D>::SMEM, st, 1, mK, mV, a);
    return launch_pdl(paged_prefix_kernel<T, D>, grid, dim3(kPreThreads), PrefixLayout<D>::SMEM, st, 1, mK, mV, a);
}

// Everything that can refuse a call comes before the first launch.
template <typename T, int D>
int run_paged(PagedArgs a, const void* k, const void* v, cudaStream_t st) {
    const bool bf = std::is_same<T, __nv_bfloat16>::value;
    // A map costs the host about as much as everything else of a call but the launches, so equal ones are made once.
    CUtensorMap mQ, mK, mV, mK16, mV16, pK, pV;
    auto maps = [&](int box, CUtensorMap* k_map, CUtensorMap* v_map) {
        return make_map(k_map, k, a.cache_rows, D, 64, box, bf) && make_map(v_map, v, a.cache_rows, D, 64, box, bf);
    };
    const int page = 1 << a.page_shift, box = page < 64 ? page : 64;
    if (!maps(box, &mK, &mV) || !make_map(&mQ, a.q, static_cast<int64_t>(a.batch) * a.hq, D, 64, a.rows, bf)) return FUSE_ECUDA;
    mK16 = pK = mK;
    mV16 = pV = mV;
    if (box != 16 && !maps(16, &mK16, &mV16)) return FUSE_ECUDA;
    if (a.plen > 0 && page > 64 && !maps(128, &pK, &pV)) return FUSE_ECUDA;
    uint32_t smem = 0;
    int ctas = 0;
    int rc = own_smem<D>(&a, &smem, &ctas);
    if (rc != FUSE_OK) return rc;
    rc = opt_in_smem((const void*)paged_own_kernel<T, D>, kOwnSmem, true);
    if (rc != FUSE_OK) return rc;
    if (a.plen > 0) {
        rc = prefix_opt_in<T, D>(a);
        if (rc != FUSE_OK) return rc;
    }
    // every CTA is resident at once; more than there can be units would have nothing to do
    int64_t grid = static_cast<int64_t>(sm_count()) * ctas;
    const int64_t units = static_cast<int64_t>(a.batch) * a.hk * a.rt * (ceil_div(a.table_ld << a.page_shift, kUnit) + 2);
    if (grid > units) grid = units;
    if (grid > kOwnGrid) grid = kOwnGrid;
    if (units / grid >= 0x7fffffffLL) return FUSE_EUNSUPPORTED;   // a CTA counts its places in 32 bits

    if (a.plen > 0) {
        rc = launch_prefix<T, D>(pK, pV, a, st);
        if (rc != FUSE_OK) return rc;
    }
    rc = launch_pdl(paged_own_kernel<T, D>, dim3(static_cast<unsigned>(grid)), dim3(kOwnThreads), smem, st, 1, mQ, mK, mV, mK16, mV16, a);
    if (rc != FUSE_OK || a.plen == 0) return rc;
    const int64_t warps = static_cast<int64_t>(a.batch) * a.hq;
    return launch_pdl(paged_join_kernel<T, D>, dim3(static_cast<unsigned>(ceil_div(warps, kJoinThreads / 32))), dim3(kJoinThreads), 0, st, 1, a);
}

}  // namespace

int paged_report_count() { return 22; }
int paged_report(int i, fuse_kernel_record* out) {
    switch (i) {
#define FC_OWN(N, T, TN, D) case N: return describe_kernel((const void*)paged_own_kernel<T, D>, "paged_own_kernel<" TN ", D=" #D "> (own keys)", kOwnThreads, own_report_smem<D>(), out)
#define FC_PRE(N, T, TN, D) case N: return describe_kernel((const void*)paged_prefix_kernel<T, D>, "paged_prefix_kernel<" TN ", D=" #D "> (shared prefix, tcgen05)", kPreThreads, PrefixLayout<D>::SMEM, out, PrefixLayout<D>::TMEM_COLS)
        FC_OWN(0, __nv_bfloat16, "bf16", 64);
        FC_OWN(1, __nv_bfloat16, "bf16", 128);
        FC_OWN(2, __nv_bfloat16, "bf16", 256);
        FC_OWN(3, __half, "f16", 64);
        FC_OWN(4, __half, "f16", 128);
        FC_OWN(5, __half, "f16", 256);
        FC_PRE(6, __nv_bfloat16, "bf16", 64);
        FC_PRE(7, __nv_bfloat16, "bf16", 128);
        FC_PRE(8, __nv_bfloat16, "bf16", 256);
        FC_PRE(9, __half, "f16", 64);
        FC_PRE(10, __half, "f16", 128);
        FC_PRE(11, __half, "f16", 256);
#define FC_JOIN(N, T, TN, D) case N: return describe_kernel((const void*)paged_join_kernel<T, D>, "paged_join_kernel<" TN ", D=" #D "> (own part and prefix)", kJoinThreads, 0, out)
        FC_JOIN(12, __nv_bfloat16, "bf16", 64);
        FC_JOIN(13, __nv_bfloat16, "bf16", 128);
        FC_JOIN(14, __nv_bfloat16, "bf16", 256);
        FC_JOIN(15, __half, "f16", 64);
        FC_JOIN(16, __half, "f16", 128);
        FC_JOIN(17, __half, "f16", 256);
#undef FC_JOIN
#define FC_PRE2(N, T, TN, D) case N: return describe_kernel((const void*)paged_prefix2_kernel<T, D>, "paged_prefix2_kernel<" TN ", D=" #D "> (shared prefix, 256 rows)", kPreThreads, Prefix2Layout<D>::SMEM, out, Prefix2Layout<D>::TMEM_COLS)
        FC_PRE2(18, __nv_bfloat16, "bf16", 64);
        FC_PRE2(19, __nv_bfloat16, "bf16", 128);
        FC_PRE2(20, __half, "f16", 64);
        FC_PRE2(21, __half, "f16", 128);
#undef FC_PRE2
#undef FC_OWN
#undef FC_PRE
        default: return FUSE_EINVAL;
    }
}

}  // namespace fc

extern "C" size_t fuse_paged_attention_workspace_bytes(int64_t batch, int64_t q_heads, int64_t kv_heads, int64_t D,
                                                       int64_t prefix_len) {
    if (batch < 1 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0 || D < 1 || prefix_len < 0) return 0;
    return fc::sizes(batch, q_heads, kv_heads, D, prefix_len).bytes;
}

extern "C" int fuse_paged_attention(const void* q, const void* k_cache, const void* v_cache,
                                    const int32_t* block_table, int64_t table_ld, const int32_t* seq_lens,
                                    const int32_t* prefix_table, int64_t prefix_len, void* o, int64_t batch,
                                    int64_t q_heads, int64_t kv_heads, int64_t D, int64_t num_pages,
                                    int64_t page_size, float scale, int dtype, void* workspace, size_t ws_bytes,
                                    fuse_stream_t stream) {
    using namespace fc;
    if (batch < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0 || D < 1 || num_pages < 1 ||
        page_size < 1 || table_ld < 0 || prefix_len < 0 || !(scale > 0.0f) || !isfinite(scale))
        return FUSE_EINVAL;
    if (dtype != FUSE_F16 && dtype != FUSE_BF16) return FUSE_EINVAL;
    if (D != 64 && D != 128 && D != 256) return FUSE_EUNSUPPORTED;
    if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)) != 0) return FUSE_EUNSUPPORTED;
    const int64_t top = int64_t(1) << 31;
    if (batch > kMaxBatch || q_heads > 65536 || batch * q_heads >= top || num_pages >= top / (kv_heads * page_size) ||
        table_ld >= (top - 4096) / page_size || prefix_len >= top - 4096)
        return FUSE_EUNSUPPORTED;
    // places of the whole batch, and tiles of the prefix, stay below 2^31 (and a CTA's places: see run_paged())
    if ((table_ld * page_size / kUnit + 2) * batch >= top) return FUSE_EUNSUPPORTED;
    const int64_t group = q_heads / kv_heads;
    if (prefix_len > 0 && (ceil_div(prefix_len, 128) + kEntry) * kv_heads * ceil_div(batch * group, 128) >= top) return FUSE_EUNSUPPORTED;
    if (batch == 0) return FUSE_OK;
    if (!q || !k_cache || !v_cache || !o || !seq_lens || (table_ld > 0 && !block_table) || (prefix_len > 0 && !prefix_table))
        return FUSE_EINVAL;
    if (!is_aligned(q, 16) || !is_aligned(k_cache, 16) || !is_aligned(v_cache, 16) || !is_aligned(o, 16) ||
        !is_aligned(block_table, 4) || !is_aligned(seq_lens, 4) || !is_aligned(prefix_table, 4))
        return FUSE_EALIGN;
    const Sizes s = sizes(batch, q_heads, kv_heads, D, prefix_len);
    if (!workspace || ws_bytes < s.bytes) return FUSE_EWORKSPACE;
    if (!is_aligned(workspace, 256)) return FUSE_EALIGN;
    const int64_t qb = batch * q_heads * D * 2, cb = num_pages * kv_heads * page_size * D * 2;
    struct { const void* p; int64_t n; } in[6] = {{q, qb}, {k_cache, cb}, {v_cache, cb}, {table_ld > 0 ? block_table : nullptr, batch * table_ld * 4},
                                                 {seq_lens, batch * 4}, {prefix_len > 0 ? prefix_table : nullptr, ceil_div(prefix_len, page_size) * 4}};
    for (const auto& x : in)
        if (x.p && (ranges_overlap(o, qb, x.p, x.n) || ranges_overlap(workspace, static_cast<int64_t>(s.bytes), x.p, x.n))) return FUSE_EINVAL;
    if (ranges_overlap(workspace, static_cast<int64_t>(s.bytes), o, qb)) return FUSE_EINVAL;
    PagedArgs a{};
    a.q = q;
    a.o = o;
    a.table = block_table;
    a.lens = seq_lens;
    a.ptable = prefix_table;
    a.table_ld = table_ld;
    a.batch = static_cast<int>(batch);
    a.hq = static_cast<int>(q_heads);
    a.hk = static_cast<int>(kv_heads);
    a.group = static_cast<int>(group);
    a.rt = static_cast<int>(ceil_div(group, 16));
    a.rows = static_cast<int>(s.rows);
    while ((1 << a.page_shift) < page_size) ++a.page_shift;
    a.num_pages = static_cast<int>(num_pages);
    a.cache_rows = static_cast<int>(num_pages * kv_heads * page_size);
    a.c = scale * 1.4426950408889634f;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.count = reinterpret_cast<int*>(ws + s.count);
    a.ready = a.count + kOwnGrid * kOwnWarps;
    a.oml = reinterpret_cast<float*>(ws + s.oml);
    a.oo = reinterpret_cast<float*>(ws + s.oo);
    a.where = reinterpret_cast<int*>(ws + s.where);
    a.rml = reinterpret_cast<float*>(ws + s.rml);
    a.ro = reinterpret_cast<float*>(ws + s.ro);
    a.pml = reinterpret_cast<float*>(ws + s.pml);
    a.po = reinterpret_cast<float*>(ws + s.po);
    a.plen = static_cast<int>(prefix_len);
    if (prefix_len > 0) {
        a.ptiles = static_cast<int>(ceil_div(prefix_len, 128));
        a.prow = static_cast<int>(s.prow);
        a.prt = static_cast<int>(ceil_div(batch * group, s.prow));
        const int64_t units = static_cast<int64_t>(a.hk) * a.prt * a.ptiles;
        int64_t grid = sm_count() < kPrefixGrid ? sm_count() : kPrefixGrid;
        a.pgrid = static_cast<int>(grid < units ? grid : units);
        a.pent = units > grid ? kEntry : 0;
    }
    a.flag = watchdog_flag();
    a.bad = index_flag();
    if (!a.flag || !a.bad) return FUSE_ECUDA;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == FUSE_F16) {
        if (D == 64) return run_paged<__half, 64>(a, k_cache, v_cache, st);
        if (D == 128) return run_paged<__half, 128>(a, k_cache, v_cache, st);
        return run_paged<__half, 256>(a, k_cache, v_cache, st);
    }
    if (D == 64) return run_paged<__nv_bfloat16, 64>(a, k_cache, v_cache, st);
    if (D == 128) return run_paged<__nv_bfloat16, 128>(a, k_cache, v_cache, st);
    return run_paged<__nv_bfloat16, 256>(a, k_cache, v_cache, st);
}

extern "C" int64_t fuse_paged_attention_bytes(int64_t batch, int64_t q_heads, int64_t kv_heads, int64_t D,
                                              int64_t prefix_len, int64_t keys) {
    if (batch < 0 || q_heads < 1 || kv_heads < 1 || D < 1 || prefix_len < 0 || keys < 0) return FUSE_EINVAL;
    return 4 * D * (kv_heads * (prefix_len + keys) + batch * q_heads);   // K and V once; q and o
}

extern "C" int64_t fuse_paged_attention_flops(int64_t batch, int64_t q_heads, int64_t D, int64_t prefix_len,
                                              int64_t keys) {
    if (batch < 0 || q_heads < 1 || D < 1 || prefix_len < 0 || keys < 0) return FUSE_EINVAL;
    return 4 * D * q_heads * (batch * prefix_len + keys);
}
