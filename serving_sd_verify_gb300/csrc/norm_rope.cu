// Norms of query and key heads with rotary positions of several axes, alone or
// with the write of keys and values to a paged cache, as they are or as e4m3 with
// a scale per row.
//
// For a row x of D elements (one head of a token), weight w:
//   u = w x / sqrt(mean(x^2) + eps);  (u_a, u_b) -> (u_a c - u_b s, u_b c + u_a s)
// with c, s of positions[axis(i)] * w_i for pair i; a cached row then as codes
// u (448 / max |u|).  All in fp32 registers, each row read once.
#include "e4m3.cuh"
#include "rope.cuh"

namespace sdv {

namespace {

constexpr int kRowThreads = 128;

__device__ __forceinline__ int pair_axis(const NormRopeParams &p, int i) { return (int)(p.axis[i >> 4] >> (2 * (i & 15))) & 3; }

// One warp per row, single elements: any size, stride and alignment.  A row is
// read again where its values are needed again.
template <typename T>
__global__ void __launch_bounds__(kRowThreads)
norm_rope_row_kernel(const __grid_constant__ NormRopeParams p, const long rows, const int checks) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const bool append = p.v != nullptr;
    if ((int)blockIdx.x < checks) {
        const int b = (int)blockIdx.x * kRowThreads + (int)threadIdx.x;
        if (b < p.B) append_check(p, b);
        return;
    }
    const int lane = threadIdx.x & 31;
    const long id = (long)((int)blockIdx.x - checks) * (kRowThreads / 32) + (threadIdx.x >> 5);
    if (id >= rows) return;
    int h;
    const int n = (int)divide(id, p.Hq + p.Hk * (append ? 2 : 1), h);
    const int role = h < p.Hq ? 0 : h < p.Hq + p.Hk ? 1 : 2;         // query, key, value
    if (role) h -= p.Hq + (role - 1) * p.Hk;
    const T *x = static_cast<const T *>(role == 0 ? p.q : role == 1 ? p.k : p.v) +
                 (role == 0 ? (long)n * p.q_tok + (long)h * p.q_head : (long)n * p.k_tok + (long)h * p.k_head);
    int cached = 0, page = 0, slot = 0;
    if (append) {
        const int r = append_place(p, n, cached, page, slot);
        if (r == -2 || (r < 0 && role)) return;
    }
    T *y = nullptr;
    long at = 0;                     // of the row in the pages
    if (role == 0) y = static_cast<T *>(p.q_out) + (long)n * p.qo_tok + (long)h * p.qo_head;
    else if (!append) y = static_cast<T *>(p.k_out) + (long)n * p.ko_tok + (long)h * p.ko_head;
    else {
        at = (long)page * p.pages.b + (long)slot * p.pages.s + (long)h * p.pages.h;
        if (!p.k_scale) y = static_cast<T *>(role == 1 ? p.k_pages : p.v_pages) + at;
    }
    const T *w = static_cast<const T *>(role == 0 ? p.wq : role == 1 ? p.wk : nullptr);
    float inv = 1.f;
    if (w) {
        float sum = 0.f;
        for (int i = lane; i < p.D; i += 32) sum = fmaf(to_f(x[i]), to_f(x[i]), sum);
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        inv = __fdiv_rn(1.f, __fsqrt_rn(sum / (float)p.D + p.eps));
    }
    __syncwarp();                    // in place: every element has been read
    auto normed = [&](int i) { return w ? to_f(x[i]) * inv * to_f(w[i]) : to_f(x[i]); };
    // f(element, value) for the lane's elements; a pair's two are read before either is passed on
    auto visit = [&](auto f) {
        const int rot = role == 2 ? 0 : p.rot;
        for (int i = lane; i < rot / 2; i += 32) {
            const int a = p.interleaved ? 2 * i : i, b = p.interleaved ? a + 1 : i + p.rot / 2;
            const int pos = p.positions ? p.positions[pair_axis(p, i) * p.pos_stride + n] : cached;
            const float2 cs = rope_cs(p.turns[i], pos, p.magnitude);
            const float u = normed(a), v = normed(b);
            f(a, u * cs.x - v * cs.y);
            f(b, v * cs.x + u * cs.y);
        }
        for (int i = rot + lane; i < p.D; i += 32) f(i, normed(i));
    };
    if (y) {
        visit([&](int i, float v) { from_f(y + i, v); });
        return;
    }
    float amax = 0.f;
    visit([&](int, float v) { amax = fmaxf(amax, fabsf(v)); });
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    uint8_t *codes = static_cast<uint8_t *>(role == 1 ? p.k_pages : p.v_pages) + at;
    const float mul = e4m3_inverse(amax);
    visit([&](int i, float v) { codes[i] = (uint8_t)e4m3x2(v * mul, 0.f); });
    if (lane == 0)
        (role == 1 ? p.k_scale : p.v_scale)[((long)page * p.Hk + h) * p.page_size + slot] = e4m3_scale(amax);
}

template <typename T> cudaError_t launch_rows(const NormRopeParams &p, cudaStream_t st) {
    const bool append = p.v != nullptr;
    const long rows = (long)p.N * (p.Hq + p.Hk * (append ? 2 : 1));
    const int checks = append ? (p.B + kRowThreads - 1) / kRowThreads : 0;      // CTAs that look over the sequences
    const long blocks = checks + (rows + kRowThreads / 32 - 1) / (kRowThreads / 32);
    if (blocks > 0x7fffffffL) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kRowThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, norm_rope_row_kernel<T>, p, rows, checks);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams &p, cudaStream_t st) {
    return p.dt == SD_BF16 ? launch_rows<__nv_bfloat16>(p, st) : launch_rows<float>(p, st);
}

}  // namespace sdv
