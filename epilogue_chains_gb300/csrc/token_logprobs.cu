// token_logprobs.cu -- log probabilities of given tokens, the entropy of each row's distribution and its
// best alternatives, from logits that are read from HBM once.
//
//     z_j = scale x_j,   lse = log sum_j e^(z_j),   log p_j = z_j - lse,   H = lse - sum_j p_j z_j.
// A part of a row gives (m, S, T) = (max x, sum 2^d, sum 2^d d) with d = (x - m) scale log2(e) <= 0; parts join
// over M = max m_i as S = sum a_i S_i, T = sum a_i (T_i + S_i (m_i - M) scale log2(e)), a_i = 2^((m_i - M) scale log2(e)).
// Then log p_j = (x_j - M) scale - ln S and H = ln S - ln 2 T / S.  Differences from the maximum are taken before
// the scale multiplies them, so a large logit costs no digits.
//
// Alternatives without a second pass: each thread's m is the largest of the logits it has read, so the k-th
// largest of the threads' m bounds the k-th largest logit from below, and whatever reaches the bound was read
// by a thread whose m reaches it.  Only those threads' logits (k threads' worth, mostly) are read again, out of
// L2, and what reaches the bound is ranked by (logit, lower index first).  Many equal logits overflow the list
// of candidates; then k scans of the row find them one by one.
//
// A row is read by a cluster of 1, 2, 4 or 8 CTAs (few rows: more CTAs for each), whose parts and alternatives
// meet in the first CTA's shared memory.  It is bound by HBM: 4096 x 131072 in bf16, the best five of each, 167 us (6.4 TB/s);
// one row or a few by latency: 128000 fp32 logits of one row 4.2 us, with the best twenty 6.5 us (in a captured graph; a call
// takes 7.1).
#include <math.h>

#include <type_traits>

#include "fc_internal.cuh"
#include "fc_mma.cuh"
#include "fc_ptx.cuh"
#include "fc_tc.cuh"

namespace fc {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxTop = 32;
constexpr int kCand = 512;                  // candidates that the list holds
constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct LogprobArgs {
    const void* x;
    int64_t ld, rows;
    int vocab, top;
    const int32_t* tokens;
    float *logprob, *entropy, *top_logprob;
    int32_t* top_index;
    float scale, c;                         // c = scale log2(e)
    int* bad;
};

__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
// An alternative as one number: the larger logit, of equal ones the lower index, has the larger.  0 is none (a logit above
// -inf has a larger one).
__device__ __forceinline__ uint64_t key_of(float x, int i) {
    const uint32_t b = __float_as_uint(x + 0.0f);        // (zeros of both signs are equal)
    return static_cast<uint64_t>(b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u)) << 32 | (0xffffffffu - static_cast<uint32_t>(i));
}
__device__ __forceinline__ float logit_of(uint64_t k) {
    const uint32_t b = static_cast<uint32_t>(k >> 32);
    return __uint_as_float(b ^ ((b >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ int index_of(uint64_t k) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(k)); }
__device__ __forceinline__ uint64_t shfl_xor_u64(uint64_t v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }
// One comparison step of a bitonic network over the warp: the larger value goes to the lane with (lane & o) == 0 where `down`,
// else to the other.
__device__ __forceinline__ float exchange(float v, int o, bool down) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    return (((threadIdx.x & o) == 0) == down) ? fmaxf(v, u) : fminf(v, u);
}
__device__ __forceinline__ uint64_t exchange(uint64_t v, int o, bool down) {
    const uint64_t u = shfl_xor_u64(v, o);
    return ((((threadIdx.x & o) == 0) == down) == (v > u)) ? v : u;
}
// Sorted over the warp, largest first.
template <typename V>
__device__ __forceinline__ V sort_down(V v) {
#pragma unroll
    for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
        for (int j = k >> 1; j > 0; j >>= 1) v = exchange(v, j, (threadIdx.x & 31 & k) == 0);
    return v;
}
// The 32 largest of two sorted lists, `other` given back to front.
template <typename V>
__device__ __forceinline__ V merge_down(V v, V other) {
    v = v > other ? v : other;
#pragma unroll
    for (int j = 16; j > 0; j >>= 1) v = exchange(v, j, true);
    return v;
}

// A 32-byte vector of logits: whole sectors, also of the few that are read again.
struct Vec {
    uint4 lo, hi;
};
__device__ __forceinline__ Vec load(const Vec* p) {
    Vec v;
    asm volatile("ld.global.cg.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v.lo.x), "=r"(v.lo.y), "=r"(v.lo.z), "=r"(v.lo.w), "=r"(v.hi.x), "=r"(v.hi.y), "=r"(v.hi.z), "=r"(v.hi.w)
                 : "l"(p));
    return v;
}
template <typename T> __device__ __forceinline__ void unpack(const Vec& v, float* f) {
    Vec16<T>::unpack(v.lo, f);
    Vec16<T>::unpack(v.hi, f + Vec16<T>::N);
}
// Largest of its values (NaN left out).
template <typename T> __device__ __forceinline__ float vec_max(const Vec& v) {
    if constexpr (std::is_same<T, float>::value) {
        float f[8];
        unpack<T>(v, f);
        return fmaxf(fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3])), fmaxf(fmaxf(f[4], f[5]), fmaxf(f[6], f[7])));
    } else {
        using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
        const T2 *a = reinterpret_cast<const T2*>(&v.lo), *b = reinterpret_cast<const T2*>(&v.hi);
        const T2 m = __hmax2(__hmax2(__hmax2(a[0], a[1]), __hmax2(a[2], a[3])), __hmax2(__hmax2(b[0], b[1]), __hmax2(b[2], b[3])));
        return fmaxf(to_f32(m.x), to_f32(m.y));
    }
}

struct Shared {
    float sorted[kWarps][32];               // each warp's thread maxima, descending
    float merged[kWarps / 4][32];           // the largest of four warps'
    float s[kWarps], t[kWarps], bound;
    float part[3];                          // this CTA's (m, S, T)
    int flagged, cands;
    int list[kThreads];
    uint64_t cand[kCand];
    uint64_t best[kMaxTop];                 // this CTA's alternatives, best first, then 0
    uint64_t scan[kWarps];                  // one scan's best, by warp
};

// The part of a row that one CTA reads: vectors v0 .. v0 + nv - 1 of the aligned middle, and, in the cluster's
// first CTA, the `head` elements before the middle and those from `tail` on.
template <typename T>
struct Slice {
    static constexpr int N = 32 / sizeof(T);
    const T* row;
    const Vec* mid;
    int head, tail, vocab, v0, nv;
    bool first;
    __device__ __forceinline__ int peeled() const { return first ? head + (vocab - tail) : 0; }
    __device__ __forceinline__ int peel_at(int i) const { return i < head ? i : tail + (i - head); }
    __device__ __forceinline__ int index(int vec, int e) const { return head + (v0 + vec) * N + e; }
};

// Calls f(value, index) for every element of the slice.
template <typename T, typename F>
__device__ __forceinline__ void for_each(const Slice<T>& s, F&& f) {
    for (int v = threadIdx.x; v < s.nv; v += kThreads) {
        float x[Slice<T>::N];
        unpack<T>(load(s.mid + v), x);
#pragma unroll
        for (int e = 0; e < Slice<T>::N; ++e) f(x[e], s.index(v, e));
    }
    if (static_cast<int>(threadIdx.x) < s.peeled()) {
        const int i = s.peel_at(threadIdx.x);
        f(to_f32(s.row[i]), i);
    }
}

// The slice's alternatives in sh.best by one scan for each: the best that comes after the one before.  Logits of -inf (and
// NaN, which counts as -inf) are left out.
template <typename T>
__device__ __noinline__ void scan_top(Shared& sh, Slice<T> s, int top) {
    uint64_t last = ~uint64_t(0);
    for (int n = 0; n < top; ++n) {
        uint64_t best = 0;
        for_each<T>(s, [&](float x, int i) {
            const uint64_t k = key_of(x, i);
            if (x > -INFINITY && k < last && k > best) best = k;
        });
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const uint64_t k = shfl_xor_u64(best, o);
            best = k > best ? k : best;
        }
        __syncthreads();
        if (threadIdx.x % 32 == 0) sh.scan[threadIdx.x / 32] = best;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) best = sh.scan[w] > best ? sh.scan[w] : best;
        if (threadIdx.x == 0) sh.best[n] = best;
        last = best;              // (0: none is left, and none will be found)
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 6) token_logprobs_kernel(const __grid_constant__ LogprobArgs a, int cluster) {
    constexpr int N = Slice<T>::N, U = 2;
    __shared__ Shared sh;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const uint32_t rank = cluster > 1 ? cluster_rank() : 0u;
    const int64_t row = blockIdx.x / static_cast<unsigned>(cluster);
    pdl_begin();

    Slice<T> s;
    s.row = static_cast<const T*>(a.x) + row * a.ld;
    s.vocab = a.vocab;
    s.first = rank == 0;
    {
        const int lead = static_cast<int>((32u - (reinterpret_cast<uintptr_t>(s.row) & 31u)) & 31u) / static_cast<int>(sizeof(T));
        s.head = min(lead, a.vocab);
        const int vecs = (a.vocab - s.head) / N, per = (vecs + cluster - 1) / cluster;
        s.tail = s.head + vecs * N;
        s.v0 = min(static_cast<int>(rank) * per, vecs);
        s.nv = min(per, vecs - s.v0);
        s.mid = reinterpret_cast<const Vec*>(s.row + s.head) + s.v0;
    }
    if (tid == 0) sh.flagged = sh.cands = 0;

    // ---------------------------------------------------------------- one pass
    float m = -INFINITY, S = 0.0f, Tz = 0.0f;
    const float c = a.c;
    auto add = [&](float mx, auto&& values) {          // values(f): calls f for each value
        if (mx > m) {
            const float d = fmaxf((m - mx) * c, -200.0f), r = ex2f(d);
            Tz = r * (Tz + S * d);
            S *= r;
            m = mx;
        }
        // (-inf while nothing is finite: against 0 such logits give 2^-inf = 0)
        const float ref = m == -INFINITY ? 0.0f : m;
        values([&](float x) {
            const float d = max_nan((x - ref) * c, -200.0f);   // 0 x -inf would be NaN
            const float e = ex2f(d);
            S += e;
            Tz += e * d;
        });
    };
    int v = tid;
    for (; v + (U - 1) * kThreads < s.nv; v += U * kThreads) {
        Vec r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) r[u] = load(s.mid + v + u * kThreads);
        float mx = vec_max<T>(r[0]);
#pragma unroll
        for (int u = 1; u < U; ++u) mx = fmaxf(mx, vec_max<T>(r[u]));
        add(mx, [&](auto&& f) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float x[N];
                unpack<T>(r[u], x);
#pragma unroll
                for (int e = 0; e < N; ++e) f(x[e]);
            }
        });
    }
    for (; v < s.nv; v += kThreads) {
        const Vec r = load(s.mid + v);
        add(vec_max<T>(r), [&](auto&& f) {
            float x[N];
            unpack<T>(r, x);
#pragma unroll
            for (int e = 0; e < N; ++e) f(x[e]);
        });
    }
    if (tid < s.peeled()) {
        const float x = to_f32(s.row[s.peel_at(tid)]);
        add(x, [&](auto&& f) { f(x); });
    }

    // ---------------------------------------------------------------- the CTA's sums, and the bound
    if (a.top > 0) {
        sh.sorted[warp][lane] = sort_down(m);
    } else {
        float o = m;
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) o = fmaxf(o, __shfl_xor_sync(0xffffffffu, o, k));
        if (lane == 0) sh.sorted[warp][0] = o;
    }
    __syncthreads();
    float M = sh.sorted[0][0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) M = fmaxf(M, sh.sorted[w][0]);
    if (a.top > 0) {         // the warps' lists into one, four at a time
        if (warp < kWarps / 4) {
            float best = sh.sorted[4 * warp][lane];
#pragma unroll
            for (int w = 1; w < 4; ++w) best = merge_down(best, sh.sorted[4 * warp + w][31 - lane]);
            sh.merged[warp][lane] = best;
        }
        __syncthreads();
    }
    if (warp == 0 && a.top > 0) {
        float best = sh.merged[0][lane];
#pragma unroll
        for (int w = 1; w < kWarps / 4; ++w) best = merge_down(best, sh.merged[w][31 - lane]);
        if (lane == a.top - 1) sh.bound = best;
    }
    const bool some = m > -INFINITY;
    const float dm = some ? fmaxf((m - M) * c, -200.0f) : 0.0f, r = ex2f(dm);
    float Sw = some ? r * S : S, Tw = some ? r * (Tz + S * dm) : Tz;    // (of a thread that saw nothing finite, NaN or 0)
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) {
        Sw += __shfl_xor_sync(0xffffffffu, Sw, k);
        Tw += __shfl_xor_sync(0xffffffffu, Tw, k);
    }
    if (lane == 0) {
        sh.s[warp] = Sw;
        sh.t[warp] = Tw;
    }
    __syncthreads();
    if (tid == 0) {
        float St = 0.0f, Tt = 0.0f;
        for (int w = 0; w < kWarps; ++w) {
            St += sh.s[w];
            Tt += sh.t[w];
        }
        sh.part[0] = M;
        sh.part[1] = St;
        sh.part[2] = Tt;
    }

    // ---------------------------------------------------------------- the CTA's alternatives
    if (a.top > 0) {
        const float bound = sh.bound;
        if (some && m >= bound) sh.list[atomicAdd(&sh.flagged, 1)] = tid;
        __syncthreads();
        const int flagged = sh.flagged;
        auto take = [&](float x, int i) {
            if (x >= bound && x > -INFINITY) {
                const int at = atomicAdd(&sh.cands, 1);
                if (at < kCand) sh.cand[at] = key_of(x, i);
            }
        };
        // a power of two of threads to each flagged one's vectors, as many as these are, at most a warp
        const int each = (s.nv + kThreads - 1) / kThreads, shift = each > 1 ? min(5, 32 - __clz(each - 1)) : 0;
        for (int f = tid >> shift; f < flagged; f += kThreads >> shift)
            for (int w = sh.list[f] + (tid & ((1 << shift) - 1)) * kThreads; w < s.nv; w += kThreads << shift) {
                float x[N];
                unpack<T>(load(s.mid + w), x);
#pragma unroll
                for (int e = 0; e < N; ++e) take(x[e], s.index(w, e));
            }
        if (tid < s.peeled()) take(to_f32(s.row[s.peel_at(tid)]), s.peel_at(tid));
        __syncthreads();
        const int n = sh.cands;
        if (n > kCand) {
            scan_top<T>(sh, s, a.top);
        } else {
            // each candidate's place is the number of larger ones (no two are equal)
            for (int i = tid; i < n; i += kThreads) {
                const uint64_t k = sh.cand[i];
                int place = 0;
                for (int j = 0; j < n; ++j) place += sh.cand[j] > k;
                if (place < a.top) sh.best[place] = k;
            }
            if (tid >= n && tid < a.top) sh.best[tid] = 0;
        }
    }

    // ---------------------------------------------------------------- the row
    if (cluster > 1) cluster_sync();
    else __syncthreads();
    if (rank == 0 && warp == 0) {
        // lane i has CTA i's part
        float pm = -INFINITY, ps = 0.0f, pt = 0.0f;
        if (lane < cluster) {
            if (cluster == 1) {
                pm = sh.part[0];
                ps = sh.part[1];
                pt = sh.part[2];
            } else {
                const uint32_t at = mapa_shared(smem_addr(sh.part), lane);
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(pm) : "r"(at) : "memory");
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(ps) : "r"(at + 4) : "memory");
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(pt) : "r"(at + 8) : "memory");
            }
        }
        float top = pm;
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
        const float d = pm > -INFINITY ? fmaxf((pm - top) * c, -200.0f) : 0.0f, e = ex2f(d);
        float Sr = e * ps, Tr = e * (pt + ps * d);
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) {
            Sr += __shfl_xor_sync(0xffffffffu, Sr, k);
            Tr += __shfl_xor_sync(0xffffffffu, Tr, k);
        }
        // a row without a finite logit: log 0 for every token, and no entropy (NaN stays NaN)
        const bool empty = top == -INFINITY && Sr == 0.0f;
        const float ln = logf(Sr);
        auto log_p = [&](float x) { return empty ? -INFINITY : (x - top) * a.scale - ln; };
        if (lane == 0) {
            const int t = a.tokens ? a.tokens[row] : -1;
            float lp = 0.0f;
            if (t >= a.vocab) {
                atomicExch(a.bad, 1);
                lp = __int_as_float(0x7fc00000);
            } else if (t >= 0) {
                lp = log_p(to_f32(s.row[t]));
            }
            if (a.logprob) a.logprob[row] = lp;
            if (a.entropy) a.entropy[row] = empty ? 0.0f : ln - kLn2 * (Tr / Sr);
        }
        if (a.top > 0) {
            // the CTAs' lists, each of them sorted, into one
            float* ov = a.top_logprob ? a.top_logprob + row * a.top : nullptr;
            int32_t* oi = a.top_index ? a.top_index + row * a.top : nullptr;
            uint64_t part[kMaxCluster];      // odd ones back to front
            part[0] = lane < a.top ? sh.best[lane] : uint64_t(0);
#pragma unroll
            for (int q = 1; q < kMaxCluster; ++q) {
                const int i = q % 2 ? 31 - lane : lane;
                part[q] = 0;
                if (q < cluster && i < a.top)
                    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(*reinterpret_cast<unsigned long long*>(&part[q])) : "r"(mapa_shared(smem_addr(sh.best + i), q)) : "memory");
            }
#pragma unroll
            for (int step = 1; step < kMaxCluster; step *= 2)
                if (step < cluster)
#pragma unroll
                    for (int q = 0; q < kMaxCluster; q += 2 * step)
                        part[q] = merge_down(part[q], step == 1 ? part[q + step] : static_cast<uint64_t>(__shfl_sync(0xffffffffu, part[q + step], 31 - lane)));
            const uint64_t best = part[0];
            const int n = __popc(__ballot_sync(0xffffffffu, lane < a.top && best != 0));
            if (lane < n) {
                if (ov) ov[lane] = log_p(logit_of(best));
                if (oi) oi[lane] = index_of(best);
            }
            // Fewer than `top` logits above -inf: then the first tokens of the others, which are among the first `top`.
            if (n < a.top) {
                const float x = lane < a.top ? to_f32(s.row[lane]) : 0.0f;
                const bool none = lane < a.top && !(x > -INFINITY);
                const int at = n + __popc(__ballot_sync(0xffffffffu, none) & ((1u << lane) - 1u));
                if (none && at < a.top) {
                    if (ov) ov[at] = Sr == Sr ? -INFINITY : Sr;
                    if (oi) oi[at] = lane;
                }
            }
        }
    }
    if (cluster > 1) cluster_sync();      // the first CTA has read the others' shared memory
}

// CTAs of a row: twice as many while there are fewer than two for each SM and 2048 logits are left to each.  In us, over 1, 2, 4 and 8
// (bf16, the best five): 128000 logits of one row 10.6, 8.3, 7.2, 6.5, of 38 17.2, 11.9, 10.1, 10.9, of 152 17.9, 13.8, 16.2, 20.5, of
// 303 22.7, 23.7, 26.2, 32.9; 32000 of one row 6.2, 6.2, 5.9, 5.5, 8000 5.1, 5.2, 5.3, 5.5, 4000 4.6, 5.2, 5.3, 5.4.  Between such numbers
// of rows the last CTAs run alone, and the rule is off by up to a third: 200 rows 26.5, 22.1 (its choice), 16.4, 23.1.
int cluster_of(int64_t rows, int64_t vocab) {
    int c = 1;
    while (c < kMaxCluster && rows * c < 2 * static_cast<int64_t>(sm_count()) && vocab >= 4096 * c) c *= 2;
    return c;
}

template <typename T>
int run_logprobs(const LogprobArgs& a, cudaStream_t st) {
    const int c = cluster_of(a.rows, a.vocab);
    return launch_pdl(token_logprobs_kernel<T>, dim3(static_cast<unsigned>(a.rows * c)), dim3(kThreads), 0, st, c, a, c);
}

}  // namespace

int logprob_report_count() { return 3; }
int logprob_report(int i, fuse_kernel_record* out) {
    switch (i) {
        FC_REPORT(0, kThreads, 0, 0, token_logprobs_kernel<float>);
        FC_REPORT(1, kThreads, 0, 0, token_logprobs_kernel<__half>);
        FC_REPORT(2, kThreads, 0, 0, token_logprobs_kernel<__nv_bfloat16>);
        default: return FUSE_EINVAL;
    }
}

}  // namespace fc

extern "C" int fuse_token_logprobs(const void* logits, int64_t ld, const int32_t* tokens, float* logprob, float* entropy,
                                   float* top_logprob, int32_t* top_index, int64_t rows, int64_t vocab, int64_t top,
                                   float scale, int dtype, fuse_stream_t stream) {
    using namespace fc;
    if (rows < 0 || vocab < 1 || top < 0 || top > vocab || ld < vocab || !(scale > 0.0f) || !isfinite(scale * kLog2e)) return FUSE_EINVAL;
    if (dtype != FUSE_F32 && dtype != FUSE_F16 && dtype != FUSE_BF16) return FUSE_EINVAL;
    const int64_t size = dtype == FUSE_F32 ? 4 : 2, most = int64_t(1) << 31;
    if (top > kMaxTop || vocab >= most - 64 || rows >= most / kMaxCluster || ld >= (int64_t(1) << 40)) return FUSE_EUNSUPPORTED;
    if (rows == 0) return FUSE_OK;
    if (!logits || (!logprob && !entropy && top == 0) || (logprob && !tokens) || (top > 0 && !top_logprob && !top_index)) return FUSE_EINVAL;
    if (!is_aligned(logits, size) || !is_aligned(tokens, 4) || !is_aligned(logprob, 4) || !is_aligned(entropy, 4) ||
        !is_aligned(top_logprob, 4) || !is_aligned(top_index, 4))
        return FUSE_EALIGN;
    struct { const void* p; int64_t n; bool out; } op[6] = {
        {logits, ((rows - 1) * ld + vocab) * size, false}, {tokens, rows * 4, false}, {logprob, rows * 4, true}, {entropy, rows * 4, true},
        {top > 0 ? top_logprob : nullptr, rows * top * 4, true}, {top > 0 ? top_index : nullptr, rows * top * 4, true}};
    for (int i = 0; i < 6; ++i)
        for (int j = 0; j < i; ++j)
            if (op[i].out && op[i].p && op[j].p && ranges_overlap(op[i].p, op[i].n, op[j].p, op[j].n)) return FUSE_EINVAL;
    LogprobArgs a{};
    a.x = logits;
    a.ld = ld;
    a.rows = rows;
    a.vocab = static_cast<int>(vocab);
    a.top = static_cast<int>(top);
    a.tokens = tokens;
    a.logprob = logprob;
    a.entropy = entropy;
    a.top_logprob = top_logprob;
    a.top_index = top_index;
    a.scale = scale;
    a.c = scale * kLog2e;
    a.bad = index_flag();
    if (!a.bad) return FUSE_ECUDA;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == FUSE_F32) return run_logprobs<float>(a, st);
    return dtype == FUSE_F16 ? run_logprobs<__half>(a, st) : run_logprobs<__nv_bfloat16>(a, st);
}

extern "C" int64_t fuse_token_logprobs_bytes(int64_t rows, int64_t vocab, int64_t top, int dtype) {
    if (rows < 0 || vocab < 1 || top < 0 || (dtype != FUSE_F32 && dtype != FUSE_F16 && dtype != FUSE_BF16)) return FUSE_EINVAL;
    return rows * (vocab * (dtype == FUSE_F32 ? 4 : 2) + 12 + 8 * top);
}
