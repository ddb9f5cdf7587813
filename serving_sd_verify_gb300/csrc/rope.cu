// Rotary positions, alone or with the write of new keys and values to a paged
// cache.  Elementwise and bound by memory: one pass, 16-byte vectors, each
// angle worked out once per thread for up to kHeads heads of a token.
//
// Angles.  Word i of `turns` is 2^64 times the fraction of a turn that pair i
// moves per position; word * position in 64-bit arithmetic drops whole turns
// exactly, so an angle is as good at position 10^6 as at 1.  Its top 32 bits
// are cut into a quadrant and a remainder within an eighth of a turn, which
// fp32 holds to 2^-28 turns, and sincospif takes the remainder.
#include "common.cuh"

namespace sdv {

namespace {

constexpr int kRopeThreads = 256;
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

template <typename T> struct Vec;
template <> struct Vec<float> {
    static constexpr int n = 4;
    float f[4];
    __device__ __forceinline__ void load(const float *p) {
        const float4 v = *reinterpret_cast<const float4 *>(p);
        f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
    }
    __device__ __forceinline__ void store(float *p) const {
        *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
    }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int n = 8;
    float f[8];
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        unpack_bf16x8(*reinterpret_cast<const uint4 *>(p), f);
    }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const {
        uint4 v;
        uint32_t *w = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);   // rounded once, to nearest
            w[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
        *reinterpret_cast<uint4 *>(p) = v;
    }
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
    const int a = p.cu[lo], e = p.cu[lo + 1];
    if (n < a || n >= e) {      // behind the last sequence (or an offset that is no offset)
        if (e > p.N || a < 0) set_fault(p.fault, FAULT_BAD_LENGTH);
        return -2;
    }
    const long ps = (long)p.kv_len[lo] - (e - a) + (n - a);
    pos = (int)ps;
    if (ps < 0 || ps >= (long)p.table_cols * p.page_size) {
        set_fault(p.fault, FAULT_BAD_LENGTH);
        return -1;
    }
    const int pg = p.table[(long)lo * p.table_stride + ps / p.page_size];
    if (pg < 0 || pg >= p.n_pages) {
        set_fault(p.fault, FAULT_BAD_PAGE);
        return -1;
    }
    return (long)pg * p.pages.b + (ps % p.page_size) * p.pages.s;
}

// One thread: one chunk of a token for up to kHeads heads.  A chunk is NP
// pairs (two vectors of V in the half layout, one in the interleaved), or V
// elements past the rotated ones, which are copied.  V = 1: single elements.
// Chunks of x and k come first, then the values' (copied whole).
template <typename T, int V, bool kInter, bool kAppend>
__global__ void __launch_bounds__(kRopeThreads)
rope_kernel(const RopeParams p, const int rot_chunks, const int chunks, const int groups, const int val_chunks,
            const int val_groups, const long items, const long val_items) {
    constexpr int NP = kInter ? (V > 1 ? V / 2 : 1) : V;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const long id = (long)blockIdx.x * kRopeThreads + threadIdx.x;
    const T *x = static_cast<const T *>(p.x);
    T *y = static_cast<T *>(p.y);
    if (id < items) {
        // consecutive threads: consecutive chunks, then head groups, then tokens
        const int c = (int)(id % chunks);
        const long t = id / chunks;
        const int grp = (int)(t % groups), n = (int)(t / groups);
        const int h0 = grp * kHeads, h1 = min(h0 + kHeads, p.Hq + (kAppend ? p.Hk : 0));
        int pos = 0;
        long slot = 0;
        if (kAppend) {
            slot = append_slot(p, n, pos);
            if (slot == -2) return;
        }
        if (p.positions) pos = p.positions[n];
        const T *src[kHeads];
        T *dst[kHeads];
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
            const int h = h0 + i;
            src[i] = nullptr;
            if (h >= h1) continue;
            if (h < p.Hq) {
                src[i] = x + (long)n * p.x_tok + (long)h * p.x_head;
                dst[i] = y + (long)n * p.y_tok + (long)h * p.y_head;
            } else if (slot >= 0) {
                src[i] = static_cast<const T *>(p.k) + (long)n * p.kv_tok + (long)(h - p.Hq) * p.kv_head;
                dst[i] = static_cast<T *>(p.k_pages) + slot + (long)(h - p.Hq) * p.pages.h;
            }
        }
        if (c < rot_chunks) {
            float2 cs[NP];
#pragma unroll
            for (int i = 0; i < NP; ++i) cs[i] = rope_cs(__ldg(p.turns + c * NP + i), pos, p.magnitude);
            if constexpr (V > 1) {
                Vec<T> a[kHeads], b[kHeads];
                const int oa = c * V, ob = oa + p.rot / 2;
#pragma unroll
                for (int i = 0; i < kHeads; ++i)
                    if (src[i]) {
                        a[i].load(src[i] + oa);
                        if (!kInter) b[i].load(src[i] + ob);
                    }
#pragma unroll
                for (int i = 0; i < kHeads; ++i)
                    if (src[i]) {
#pragma unroll
                        for (int e = 0; e < NP; ++e) {
                            float &u = kInter ? a[i].f[2 * e] : a[i].f[e];
                            float &v = kInter ? a[i].f[2 * e + 1] : b[i].f[e];
                            const float u0 = u, v0 = v;
                            u = u0 * cs[e].x - v0 * cs[e].y;
                            v = v0 * cs[e].x + u0 * cs[e].y;
                        }
                        a[i].store(dst[i] + oa);
                        if (!kInter) b[i].store(dst[i] + ob);
                    }
            } else {
                const int oa = kInter ? 2 * c : c, ob = kInter ? 2 * c + 1 : c + p.rot / 2;
#pragma unroll
                for (int i = 0; i < kHeads; ++i)
                    if (src[i]) {
                        const float u0 = to_f(src[i][oa]), v0 = to_f(src[i][ob]);
                        from_f(dst[i] + oa, u0 * cs[0].x - v0 * cs[0].y);
                        from_f(dst[i] + ob, v0 * cs[0].x + u0 * cs[0].y);
                    }
            }
        } else {
            const int o = p.rot + (c - rot_chunks) * V;
#pragma unroll
            for (int i = 0; i < kHeads; ++i)
                if (src[i] && dst[i] != src[i]) {
                    if constexpr (V > 1)
                        *reinterpret_cast<uint4 *>(dst[i] + o) = *reinterpret_cast<const uint4 *>(src[i] + o);
                    else
                        dst[i][o] = src[i][o];
                }
        }
    } else if (kAppend && id < items + val_items) {
        const long v = id - items;
        const int c = (int)(v % val_chunks);
        const long t = v / val_chunks;
        const int grp = (int)(t % val_groups), n = (int)(t / val_groups);
        int pos = 0;
        const long slot = append_slot(p, n, pos);
        if (slot < 0) return;
        for (int h = grp * kHeads; h < min(grp * kHeads + kHeads, p.Hk); ++h) {
            const T *src = static_cast<const T *>(p.v) + (long)n * p.kv_tok + (long)h * p.kv_head + c * V;
            T *dst = static_cast<T *>(p.v_pages) + slot + (long)h * p.pages.h + c * V;
            if constexpr (V > 1) *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<const uint4 *>(src);
            else *dst = *src;
        }
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
    const long blocks = (items + val_items + kRopeThreads - 1) / kRopeThreads;
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
                              val_groups, items, val_items);
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
    constexpr int V = Vec<T>::n;
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
