// rope_append.cu -- rotate the new queries and keys and append keys and values to a paged cache.
//
// Per token with position n and slot page * page_size + offset, for every pair (a, b) of the first
// `rot` components of each query and key head:  a' = a cos - b sin,  b' = b cos + a sin,  with the
// pair's cos and sin from row n of an fp32 table.  The rest of the head and the values are copied.
//
// The pass is a copy with six flops per pair, so bytes bound it: each component is read once and
// written once (2 (q_heads + 2 kv_heads) D elements per token).  A thread owns one pair of 16-byte
// vectors of kHeads consecutive heads of one token.  For half-split pairs the two vectors are the two
// halves of eight pairs, for interleaved pairs two neighbouring vectors, so both styles rotate within
// the thread; a thread's cosines and sines are loaded once for its kHeads heads.
#include "fc_internal.cuh"

namespace fc {
namespace {

// Heads of a thread and threads of a CTA, at 8192 tokens of 48 heads (32 + 2 8, D = 128) in us: 3 heads in 64 threads 32.4
// (6.2 TB/s, 0.92 of the copy rate), in 128 32.5, 2 heads 33.4 / 33.0, 4 heads 33.1 / 33.4, in 256 threads 36 to 43, one
// head 39 to 51; the same order for 36 and 40 heads and for D = 64 and 256.
constexpr int kRopeBlock = 64;
constexpr int kHeads = 3;

struct RopeArgs {
    const void* qkv;
    const float* cs;
    const int32_t* pos;
    const int32_t* slot;
    void *q, *k, *v;
    int64_t ld, nitem;      // nitem = tokens * chunks * pairs
    int64_t max_pos, slots;
    int tokens, hq, hk, D, rot, page_shift;
    int chunks;             // ceil((hq + 2 hk) / kHeads)
    int pairs;              // D / 16
    int* bad;
};

template <bool INTER>
__device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8], const float (&c)[8], const float (&s)[8]) {
    if constexpr (INTER) {   // a holds pairs 0..3, b pairs 4..7
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x0 = a[2 * i], y0 = a[2 * i + 1], x1 = b[2 * i], y1 = b[2 * i + 1];
            a[2 * i] = x0 * c[i] - y0 * s[i];
            a[2 * i + 1] = y0 * c[i] + x0 * s[i];
            b[2 * i] = x1 * c[4 + i] - y1 * s[4 + i];
            b[2 * i + 1] = y1 * c[4 + i] + x1 * s[4 + i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = a[i], y = b[i];
            a[i] = x * c[i] - y * s[i];
            b[i] = y * c[i] + x * s[i];
        }
    }
}

template <typename T, bool INTER>
__global__ void __launch_bounds__(kRopeBlock) rope_append_kernel(const __grid_constant__ RopeArgs p) {
    pdl_trigger();
    const int64_t id = static_cast<int64_t>(blockIdx.x) * kRopeBlock + threadIdx.x;
    if (id >= p.nitem) return;
    int pair, chunk;
    int64_t t;
    if ((p.nitem >> 32) == 0) {          // a 64-bit division takes several times as long
        const uint32_t i = static_cast<uint32_t>(id), rest = i / static_cast<uint32_t>(p.pairs);
        pair = static_cast<int>(i - rest * p.pairs);
        t = rest / static_cast<uint32_t>(p.chunks);
        chunk = static_cast<int>(rest - static_cast<uint32_t>(t) * p.chunks);
    } else {
        const int64_t rest = id / p.pairs;
        pair = static_cast<int>(id - rest * p.pairs);
        t = rest / p.chunks;
        chunk = static_cast<int>(rest - t * p.chunks);
    }
    pdl_wait();  // before any global-memory access (programmatic dependent launch)
    const int heads = p.hq + 2 * p.hk, h0 = chunk * kHeads;
    const bool turn = pair < p.rot / 16;
    // vectors (of eight components) of this pair within a head
    const int va = turn && !INTER ? pair : 2 * pair;
    const int vb = turn && !INTER ? pair + p.rot / 16 : 2 * pair + 1;
    const int vph = p.D / 8;   // vectors per head

    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(p.qkv) + t * p.ld) + h0 * vph;
    uint4 ra[kHeads], rb[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
        if (h0 + i < heads) {
            ra[i] = ld_stream(src + i * vph + va);
            rb[i] = ld_stream(src + i * vph + vb);
        }
    const int64_t slot = p.slot[t];
    const int64_t pos = p.rot > 0 ? p.pos[t] : 0;
    const bool pos_ok = p.rot == 0 || (pos >= 0 && pos < p.max_pos);
    const bool append = slot >= 0 && slot < p.slots && pos_ok;
    if (slot >= 0 && !append && pair == 0 && chunk == 0) atomicExch(p.bad, 1);

    float c[8], s[8];
    if (turn && pos_ok && h0 < p.hq + p.hk) {
        const float4* row = reinterpret_cast<const float4*>(p.cs + pos * p.rot) + 2 * pair;
        const float4* rs = row + p.rot / 8;
        const float4 c0 = row[0], c1 = row[1], s0 = rs[0], s1 = rs[1];
        c[0] = c0.x; c[1] = c0.y; c[2] = c0.z; c[3] = c0.w;
        c[4] = c1.x; c[5] = c1.y; c[6] = c1.z; c[7] = c1.w;
        s[0] = s0.x; s[1] = s0.y; s[2] = s0.z; s[3] = s0.w;
        s[4] = s1.x; s[5] = s1.y; s[6] = s1.z; s[7] = s1.w;
    }
    const int64_t page = slot >> p.page_shift;
    const int off = static_cast<int>(slot & ((1 << p.page_shift) - 1));
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        const int h = h0 + i;
        if (h >= heads) break;
        if (turn && h < p.hq + p.hk) {
            float a[8], b[8];
            Vec16<T>::unpack(ra[i], a);
            Vec16<T>::unpack(rb[i], b);
            if (pos_ok) rotate<INTER>(a, b, c, s);
            ra[i] = Vec16<T>::pack(a);
            rb[i] = Vec16<T>::pack(b);
        }
        uint4* dst;
        if (h < p.hq) {
            dst = static_cast<uint4*>(p.q) + (t * p.hq + h) * vph;
            if (!pos_ok) ra[i] = rb[i] = make_uint4(0u, 0u, 0u, 0u);
        } else {
            if (!append) continue;
            const int kh = h - p.hq;
            uint4* cache = static_cast<uint4*>(kh < p.hk ? p.k : p.v);
            const int64_t hh = kh < p.hk ? kh : kh - p.hk;
            dst = cache + (((page * p.hk + hh) << p.page_shift) + off) * vph;
        }
        dst[va] = ra[i];
        dst[vb] = rb[i];
    }
}

template <typename T>
int run_rope(const RopeArgs& a, bool inter, cudaStream_t st) {
    const int64_t grid = ceil_div(a.nitem, kRopeBlock);
    if (grid > 0x7fffffffLL) return FUSE_EUNSUPPORTED;
    if (inter) return launch_pdl(rope_append_kernel<T, true>, dim3(static_cast<unsigned>(grid)), dim3(kRopeBlock), 0, st, 1, a);
    return launch_pdl(rope_append_kernel<T, false>, dim3(static_cast<unsigned>(grid)), dim3(kRopeBlock), 0, st, 1, a);
}

}  // namespace

int rope_report_count() { return 4; }
int rope_report(int i, fuse_kernel_record* out) {
    switch (i) {
        case 0: return describe_kernel((const void*)rope_append_kernel<__nv_bfloat16, false>, "rope_append_kernel<bf16> (half-split pairs)", kRopeBlock, 0, out);
        case 1: return describe_kernel((const void*)rope_append_kernel<__nv_bfloat16, true>, "rope_append_kernel<bf16> (interleaved pairs)", kRopeBlock, 0, out);
        case 2: return describe_kernel((const void*)rope_append_kernel<__half, false>, "rope_append_kernel<f16> (half-split pairs)", kRopeBlock, 0, out);
        case 3: return describe_kernel((const void*)rope_append_kernel<__half, true>, "rope_append_kernel<f16> (interleaved pairs)", kRopeBlock, 0, out);
        default: return FUSE_EINVAL;
    }
}

}  // namespace fc

extern "C" int fuse_rope_append(const void* qkv, int64_t ld, const float* cos_sin, int64_t max_pos, int64_t rot,
                                const int32_t* positions, const int32_t* slots, void* q_out, void* k_cache,
                                void* v_cache, int64_t tokens, int64_t q_heads, int64_t kv_heads, int64_t D,
                                int64_t num_pages, int64_t page_size, int dtype, uint32_t flags,
                                fuse_stream_t stream) {
    using namespace fc;
    if (tokens < 0 || q_heads < 1 || kv_heads < 1 || D < 1 || num_pages < 0 || page_size < 1 || rot < 0 || rot > D ||
        max_pos < 0)
        return FUSE_EINVAL;
    if ((dtype != FUSE_F16 && dtype != FUSE_BF16) || (flags & ~FUSE_ROPE_INTERLEAVED) != 0) return FUSE_EINVAL;
    if (D % 16 != 0 || D > 512 || rot % 16 != 0) return FUSE_EUNSUPPORTED;
    if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)) != 0) return FUSE_EUNSUPPORTED;
    if (q_heads > 65536 || kv_heads > 65536) return FUSE_EUNSUPPORTED;
    if (num_pages >= (int64_t(1) << 31) / (kv_heads * page_size)) return FUSE_EUNSUPPORTED;
    const int64_t heads = q_heads + 2 * kv_heads, width = heads * D;
    if (ld < width) return FUSE_EINVAL;
    if (tokens == 0) return FUSE_OK;
    if (tokens > 0x7fffffffLL || ld > (int64_t(1) << 40) / tokens) return FUSE_EUNSUPPORTED;
    if (!qkv || !slots || !q_out || !k_cache || !v_cache || (rot > 0 && (!cos_sin || !positions))) return FUSE_EINVAL;
    if (ld % 8 != 0 || !is_aligned(qkv, 16) || !is_aligned(q_out, 16) || !is_aligned(k_cache, 16) ||
        !is_aligned(v_cache, 16) || !is_aligned(cos_sin, 16) || !is_aligned(positions, 4) || !is_aligned(slots, 4))
        return FUSE_EALIGN;
    struct { const void* p; int64_t n; } in[4] = {{qkv, ((tokens - 1) * ld + width) * 2}, {cos_sin, max_pos * rot * 4},
                                                 {rot > 0 ? positions : nullptr, tokens * 4}, {slots, tokens * 4}},
        out[3] = {{q_out, tokens * q_heads * D * 2}, {k_cache, num_pages * kv_heads * page_size * D * 2},
                  {v_cache, num_pages * kv_heads * page_size * D * 2}};
    for (int o = 0; o < 3; ++o) {
        for (int i = 0; i < 4; ++i)
            if (in[i].p && ranges_overlap(out[o].p, out[o].n, in[i].p, in[i].n)) return FUSE_EINVAL;
        for (int i = 0; i < o; ++i)
            if (ranges_overlap(out[o].p, out[o].n, out[i].p, out[i].n)) return FUSE_EINVAL;
    }
    RopeArgs a{};
    a.qkv = qkv;
    a.cs = cos_sin;
    a.pos = positions;
    a.slot = slots;
    a.q = q_out;
    a.k = k_cache;
    a.v = v_cache;
    a.ld = ld;
    a.max_pos = max_pos;
    a.slots = num_pages * page_size;
    a.tokens = static_cast<int>(tokens);
    a.hq = static_cast<int>(q_heads);
    a.hk = static_cast<int>(kv_heads);
    a.D = static_cast<int>(D);
    a.rot = static_cast<int>(rot);
    while ((1 << a.page_shift) < page_size) ++a.page_shift;
    a.chunks = static_cast<int>(ceil_div(heads, kHeads));
    a.pairs = static_cast<int>(D / 16);
    a.nitem = tokens * a.chunks * a.pairs;
    a.bad = index_flag();
    if (!a.bad) return FUSE_ECUDA;
    const bool inter = (flags & FUSE_ROPE_INTERLEAVED) != 0;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return dtype == FUSE_F16 ? run_rope<__half>(a, inter, st) : run_rope<__nv_bfloat16>(a, inter, st);
}

extern "C" int64_t fuse_rope_append_bytes(int64_t tokens, int64_t appended, int64_t q_heads, int64_t kv_heads,
                                          int64_t D, int64_t rot) {
    if (tokens < 0 || appended < 0 || appended > tokens || q_heads < 1 || kv_heads < 1 || D < 1 || rot < 0 || rot > D)
        return FUSE_EINVAL;
    return 4 * D * (tokens * q_heads + 2 * appended * kv_heads) + 4 * rot * appended + 8 * tokens;
}
