// Rotary positions, alone or with the write of new keys and values to a paged
// cache.  Elementwise and bound by memory: one pass, 16-byte vectors, each
// angle worked out once per thread for up to kHeads heads of a token.
//
// Angles.  Word i of `turns` is 2^64 times the fraction of a turn that pair i
// moves per position; word * position in 64-bit arithmetic drops whole turns
// exactly, so an angle is as good at position 10^6 as at 1.  Its top 32 bits
// are cut into a quadrant and a remainder within an eighth of a turn, which
// fp32 holds to 2^-28 turns, and sincospif takes the remainder.
//
// What bounds it: memory.  25,119 x 28 heads of 128 (bf16, read and written once,
// 360 MB) take 57 us, 6.3 TB/s, 0.93 of a plain copy's rate; the same with the
// cache write (463 MB) 75 us, 6.2 TB/s; in fp32 105 and 132 us, 6.9 and 7.0 TB/s.  A
// block of tokens takes 2.5 us, a launch.  Rows off 16 bytes, or a rotated part that
// is no whole vectors, take single elements, bound by their load and store
// instructions: the same in bf16 144 us, with 20 of 128 elements rotated 233 us.
#include "common.cuh"

namespace sdv {

namespace {

// 128 threads and at least six CTAs per SM (80 registers): 25,119 tokens of 28 heads
// turn in 57 us and enter the cache (with 4 + 4 heads of K and V) in 76, against
// 59 and 91 with 256 threads and two CTAs
constexpr int kRopeThreads = 128;
constexpr int kHeads = 4;       // heads per thread: their loads are in flight together, the angles shared

// cos and sin of 2 pi * frac(word * pos), times m
__device__ __forceinline__ float2 rope_cs(uint64_t word, int pos, float m) {
    const uint64_t a = word * (uint64_t)(int64_t)pos;
    const int32_t hi = (int32_t)((a + 0x80000000ull) >> 32);
    const int32_t q = (int32_t)(((uint32_t)hi + 0x20000000u) >> 30);       // nearest quarter turn
    const int32_t rem = (int32_t)((uint32_t)hi - ((uint32_t)q << 30));     // [-2^29, 2^29)
    float s, c;
    sincospif((float)rem * 0x1p-31f, &s, &c);
    if (q & 1) { const float t = c; c = -s; s = t; }
    if (q & 2) { c = -c; s = -s; }
    return make_float2(c * m, s * m);
}

// V elements as loaded: a 16-byte vector, or one element
template <typename T> constexpr int kVec = 16 / (int)sizeof(T);
template <typename T, int V> struct Raw {
    uint4 w;
    __device__ __forceinline__ void load(const T *p) { w = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<uint4 *>(p) = w; }
    __device__ __forceinline__ void unpack(float (&f)[8]) const { unpack_bf16x8(w, f); }
    __device__ __forceinline__ void unpack(float (&f)[4]) const {
        f[0] = __uint_as_float(w.x); f[1] = __uint_as_float(w.y);
        f[2] = __uint_as_float(w.z); f[3] = __uint_as_float(w.w);
    }
    __device__ __forceinline__ static uint32_t two(float a, float b) {      // rounded once, to nearest
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    __device__ __forceinline__ void pack(const float (&f)[8]) {
        w = make_uint4(two(f[0], f[1]), two(f[2], f[3]), two(f[4], f[5]), two(f[6], f[7]));
    }
    __device__ __forceinline__ void pack(const float (&f)[4]) {
        w = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};
template <typename T> struct Raw<T, 1> {
    T w;
    __device__ __forceinline__ void load(const T *p) { w = *p; }
    __device__ __forceinline__ void store(T *p) const { *p = w; }
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float *p, float x) { *p = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// where token n's key and value rows go: the offset of its slot in the pages,
// or -1; `pos` becomes the cache position
__device__ long append_slot(const RopeParams &p, int n, int &pos) {
    // the last sequence that begins at or before n (empty ones before it are
    // skipped by taking the last): cu is non-decreasing
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.cu[mid] <= n) lo = mid;
        else hi = mid - 1;
    }
    // clamped as the attention clamps them, so that a bad offset puts its tokens where the attention looks
    const int c0 = max(0, min(p.cu[lo], p.N)), c1 = max(c0, min(p.cu[lo + 1], p.N));
    if (n < c0 || n >= c1) return -2;              // behind the last sequence
    const long ps = (long)p.kv_len[lo] - (c1 - c0) + (n - c0);
    pos = (int)ps;
    if (ps < 0 || ps >= (long)p.table_cols * p.page_size) {
        set_fault(p.fault, FAULT_BAD_LENGTH);
        return -1;
    }
    const unsigned col = (unsigned)ps / (unsigned)p.page_size;       // a position fits 31 bits: kv_len does
    const int pg = p.table[(long)lo * p.table_stride + col];
    if (pg < 0 || pg >= p.n_pages) {
        set_fault(p.fault, FAULT_BAD_PAGE);
        return -1;
    }
    return (long)pg * p.pages.b + (long)((unsigned)ps - col * (unsigned)p.page_size) * p.pages.s;
}

// Sequence b's offsets and length, reported where they are none: by threads of
// their own, since a token meets only its own sequence's.
__device__ __forceinline__ void append_check(const RopeParams &p, int b) {
    const int a = p.cu[b], e = p.cu[b + 1], len = p.kv_len[b];
    if (a < 0 || a > p.N || e < a || e > p.N || len < 0 || (long)len > (long)p.table_cols * p.page_size)
        set_fault(p.fault, FAULT_BAD_LENGTH);
}

// q and the remainder of a / b, in 32 bits where a fits (a 64-bit division is a
// hundred instructions)
__device__ __forceinline__ long divide(long a, int b, int &rem) {
    if (a >> 32) {
        const long q = a / b;
        rem = (int)(a - q * b);
        return q;
    }
    const unsigned q = (unsigned)a / (unsigned)b;
    rem = (int)((unsigned)a - q * (unsigned)b);
    return q;
}

// One thread: one chunk of a token for up to kHeads heads.  A chunk is NP
// pairs (two vectors of V in the half layout, one in the interleaved), or V
// elements past the rotated ones, which are copied.  V = 1: single elements.
// Chunks of x and k come first, then the values' (copied whole).  Of an append,
// the first `checks` CTAs look over the offsets and lengths instead.
template <typename T, int V, bool kInter, bool kAppend>
__global__ void __launch_bounds__(kRopeThreads, 6)
rope_kernel(const RopeParams p, const int rot_chunks, const int chunks, const int groups, const int val_chunks,
            const int val_groups, const long items, const long val_items, const int checks) {
    constexpr int NP = kInter ? (V > 1 ? V / 2 : 1) : V;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (kAppend && (int)blockIdx.x < checks) {
        const int b = (int)blockIdx.x * kRopeThreads + (int)threadIdx.x;
        if (b < p.B) append_check(p, b);
        return;
    }
    const long id = (long)((int)blockIdx.x - (kAppend ? checks : 0)) * kRopeThreads + threadIdx.x;
    const T *x = static_cast<const T *>(p.x);
    T *y = static_cast<T *>(p.y);
    if (id < items) {
        // consecutive threads: consecutive chunks, then head groups, then tokens
        int c, grp;
        const int n = (int)divide(divide(id, chunks, c), groups, grp);
        const int h0 = grp * kHeads, h1 = min(h0 + kHeads, p.Hq + (kAppend ? p.Hk : 0));
        // the rows' loads go out first: neither the slot nor the angles hold them up
        const T *src[kHeads];
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
            const int h = h0 + i;
            src[i] = h >= h1 ? nullptr
                     : h < p.Hq ? x + (long)n * p.x_tok + (long)h * p.x_head
                                : static_cast<const T *>(p.k) + (long)n * p.kv_tok + (long)(h - p.Hq) * p.kv_head;
        }
        const bool turned = c < rot_chunks;
        // a chunk's elements: [oa, oa + V) and, of a pair in the half layout, [ob, ob + V)
        const int oa = !turned ? p.rot + (c - rot_chunks) * V : kInter ? c * (V > 1 ? V : 2) : c * V;
        const int ob = kInter ? oa + 1 : oa + p.rot / 2;
        const bool two = turned && (!kInter || V == 1);
        Raw<T, V> a[kHeads], b[kHeads];
#pragma unroll
        for (int i = 0; i < kHeads; ++i)
            if (src[i]) {
                a[i].load(src[i] + oa);
                if (two) b[i].load(src[i] + ob);
            }
        int pos = p.positions ? p.positions[n] : 0;
        long slot = 0;
        if (kAppend) {
            if (h1 <= p.Hq && p.positions) {           // queries with their positions: only whether n is anyone's
                if (n < p.cu[0] || n >= p.cu[p.B]) return;
            } else {
                int cached = 0;
                slot = append_slot(p, n, cached);
                if (slot == -2) return;
                if (!p.positions) pos = cached;
            }
        }
        float2 cs[NP];
        if (turned) {
#pragma unroll
            for (int i = 0; i < NP; ++i) cs[i] = rope_cs(__ldg(p.turns + c * NP + i), pos, p.magnitude);
        }
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
            const int h = h0 + i;
            if (!src[i] || (h >= p.Hq && slot < 0)) continue;
            T *dst = h < p.Hq ? y + (long)n * p.y_tok + (long)h * p.y_head
                              : static_cast<T *>(p.k_pages) + slot + (long)(h - p.Hq) * p.pages.h;
            if (turned) {
                if constexpr (V > 1) {
                    float fa[V], fb[V];
                    a[i].unpack(fa);
                    if (!kInter) b[i].unpack(fb);
#pragma unroll
                    for (int e = 0; e < NP; ++e) {
                        float &u = kInter ? fa[2 * e] : fa[e];
                        float &v = kInter ? fa[2 * e + 1] : fb[e];
                        const float u0 = u, v0 = v;
                        u = u0 * cs[e].x - v0 * cs[e].y;
                        v = v0 * cs[e].x + u0 * cs[e].y;
                    }
                    a[i].pack(fa);
                    if (!kInter) b[i].pack(fb);
                } else {
                    const float u0 = to_f(a[i].w), v0 = to_f(b[i].w);
                    from_f(&a[i].w, u0 * cs[0].x - v0 * cs[0].y);
                    from_f(&b[i].w, v0 * cs[0].x + u0 * cs[0].y);
                }
            } else if (dst == src[i]) {
                continue;                              // in place: what is not turned stays
            }
            a[i].store(dst + oa);
            if (two) b[i].store(dst + ob);
        }
    } else if (kAppend && id < items + val_items) {
        const long v = id - items;
        int c, grp;
        const int n = (int)divide(divide(v, val_chunks, c), val_groups, grp);
        const int h0 = grp * kHeads;
        Raw<T, V> a[kHeads];
#pragma unroll
        for (int i = 0; i < kHeads; ++i)
            if (h0 + i < p.Hk)
                a[i].load(static_cast<const T *>(p.v) + (long)n * p.kv_tok + (long)(h0 + i) * p.kv_head + c * V);
        int pos = 0;
        const long slot = append_slot(p, n, pos);
        if (slot < 0) return;
#pragma unroll
        for (int i = 0; i < kHeads; ++i)
            if (h0 + i < p.Hk)
                a[i].store(static_cast<T *>(p.v_pages) + slot + (long)(h0 + i) * p.pages.h + c * V);
    }
}

template <typename T, int V, bool kInter, bool kAppend>
cudaError_t launch_one(const RopeParams &p, cudaStream_t st) {
    const int np = kInter ? (V > 1 ? V / 2 : 1) : V;
    const int rot_chunks = p.rot / 2 / np;
    const int chunks = rot_chunks + (p.copy_rest ? (p.D - p.rot) / V : 0);
    const int heads = p.Hq + (kAppend ? p.Hk : 0);
    const int groups = (heads + kHeads - 1) / kHeads;
    const int val_chunks = p.D / V, val_groups = (p.Hk + kHeads - 1) / kHeads;
    const long items = (long)p.N * groups * chunks;
    const long val_items = kAppend ? (long)p.N * val_groups * val_chunks : 0;
    const int checks = kAppend ? (p.B + kRopeThreads - 1) / kRopeThreads : 0;    // CTAs that look over the sequences
    const long blocks = checks + (items + val_items + kRopeThreads - 1) / kRopeThreads;
    if (blocks > 0x7fffffffL) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rope_kernel<T, V, kInter, kAppend>, p, rot_chunks, chunks, groups, val_chunks,
                              val_groups, items, val_items, checks);
}

template <typename T, int V>
cudaError_t launch_v(const RopeParams &p, cudaStream_t st) {
    const bool app = p.k != nullptr;
    if (p.interleaved) return app ? launch_one<T, V, true, true>(p, st) : launch_one<T, V, true, false>(p, st);
    return app ? launch_one<T, V, false, true>(p, st) : launch_one<T, V, false, false>(p, st);
}

// 16-byte vectors: whole vectors of rotated pairs and of the rest, every row on a 16-byte boundary
template <typename T>
bool vectors_fit(const RopeParams &p) {
    constexpr int V = kVec<T>;
    auto al = [](const void *q) { return (reinterpret_cast<uintptr_t>(q) & 15u) == 0; };
    if (p.D % V || p.rot % (p.interleaved ? V : 2 * V)) return false;
    if (p.Hq && (!al(p.x) || !al(p.y) || p.x_tok % V || p.x_head % V || p.y_tok % V || p.y_head % V)) return false;
    if (p.k && (!al(p.k) || !al(p.v) || !al(p.k_pages) || !al(p.v_pages) || p.kv_tok % V || p.kv_head % V ||
                p.pages.b % V || p.pages.s % V || p.pages.h % V))
        return false;
    return true;
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p, cudaStream_t st) {
    if (p.dt == SD_BF16)
        return vectors_fit<__nv_bfloat16>(p) ? launch_v<__nv_bfloat16, 8>(p, st) : launch_v<__nv_bfloat16, 1>(p, st);
    return vectors_fit<float>(p) ? launch_v<float, 4>(p, st) : launch_v<float, 1>(p, st);
}

}  // namespace sdv
