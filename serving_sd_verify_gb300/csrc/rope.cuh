// What the two rotary kernel files share: angles, vectors of elements, and the
// place of a new token in a paged cache.
#pragma once

#include "common.cuh"

namespace sdv {
namespace {

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

// where token n's key and value rows go: 0 and page and slot, -1 where nothing can
// be written, -2 for a token behind the last sequence; `pos` becomes the cache position
template <typename P> __device__ __forceinline__ int append_place(const P &p, int n, int &pos, int &page, int &slot) {
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
    page = pg;
    slot = (int)((unsigned)ps - col * (unsigned)p.page_size);
    return 0;
}
// the same as the offset of the slot in the pages
template <typename P> __device__ long append_slot(const P &p, int n, int &pos) {
    int page = 0, slot = 0;
    const int r = append_place(p, n, pos, page, slot);
    return r < 0 ? r : (long)page * p.pages.b + (long)slot * p.pages.s;
}

// Sequence b's offsets and length, reported where they are none: by threads of
// their own, since a token meets only its own sequence's.
template <typename P> __device__ __forceinline__ void append_check(const P &p, int b) {
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

}  // namespace
}  // namespace sdv
