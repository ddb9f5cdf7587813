// Norms of query and key heads with rotary positions of several axes, alone or
// with the write of keys and values to a paged cache, as they are or as e4m3 with
// a scale per row.
//
// For a row x of D elements (one head of a token), weight w:
//   u = w x / sqrt(mean(x^2) + eps);  (u_a, u_b) -> (u_a c - u_b s, u_b c + u_a s)
// with c, s of positions[axis(i)] * w_i for pair i; a cached row then as codes
// u 448 / max |u|.  All in fp32 registers, each row read once.
#include "e4m3.cuh"
#include "rope.cuh"

#include <algorithm>

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
        if (role == 2)
            for (int i = lane; i < p.D; i += 32) y[i] = x[i];        // bit for bit
        else
            visit([&](int i, float v) { from_f(y + i, v); });
        return;
    }
    float amax = 0.f;
    visit([&](int, float v) { amax = fmaxf(amax, fabsf(v)); });
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    uint8_t *codes = static_cast<uint8_t *>(role == 1 ? p.k_pages : p.v_pages) + at;
    const RowCodes code(amax);
    visit([&](int i, float v) { codes[i] = (uint8_t)e4m3x2(code(v), 0.f); });
    if (lane == 0)
        (role == 1 ? p.k_scale : p.v_scale)[((long)page * p.Hk + h) * p.page_size + slot] = e4m3_scale(amax);
}

// Whole 16-byte vectors.  A CTA takes `tokens` tokens with all their heads: it works
// out their angles and their places in the cache once, in shared memory, then 2^log_p
// lanes of a warp hold a row at a time, a lane one chunk of it -- the two vectors of
// V pairs in the half layout, the one of V / 2 pairs in the interleaved, or V elements
// past the turned ones.  The next rows' loads are in flight while a row's sums meet by
// shuffles among its lanes.  Arithmetic comes two elements an instruction: what bounds
// the kernel besides memory is the instructions it issues.
// Measured (bf16, three axes): 25,119 tokens of 32 heads of 128 69.3 us (5.9 TB/s of 6.8),
// of 28 with 8 written as e4m3 80.2 us (5.5 TB/s), 2,048 tokens of 80 into a bf16 cache
// 17.4 us (4.8 TB/s).  A lane group with angles of its own for four heads took 97, 171 and
// 26 us, two rows in flight a lane 99, 126 and 26 (registers for five CTAs an SM only), one
// warp a token with loads ahead in registers or in a ring of cp.async 76 to 101 and 92;
// seven CTAs an SM are as many as fit without spills in the loop (six: 74.3, 87.4 and
// 22.6, eight: 72.6, 84.1 and 18.4 with four tokens a CTA, which seven do in 69.9, 83.2
// and 17.4).
constexpr int kVecThreads = 128;
constexpr int kTokens = 8;           // of a CTA at most
constexpr int kVecPairs = 256;       // of a row at most: 32 chunks of 8

// the two elements of each 32-bit word of a vector, or its words two and two
__device__ __forceinline__ void unpack2(const uint4 &w, float2 (&f)[4]) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(x[i] << 16), __uint_as_float(x[i] & 0xffff0000u));
}
__device__ __forceinline__ void unpack2(const uint4 &w, float2 (&f)[2]) {
    f[0] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
    f[1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
}
__device__ __forceinline__ uint4 pack2(const float2 (&f)[4]) {
    return make_uint4(Raw<__nv_bfloat16, 8>::two(f[0].x, f[0].y), Raw<__nv_bfloat16, 8>::two(f[1].x, f[1].y),
                      Raw<__nv_bfloat16, 8>::two(f[2].x, f[2].y), Raw<__nv_bfloat16, 8>::two(f[3].x, f[3].y));
}
__device__ __forceinline__ uint4 pack2(const float2 (&f)[2]) {
    return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x), __float_as_uint(f[1].y));
}
__device__ __forceinline__ float2 neg2(float2 a) { return make_float2(-a.x, -a.y); }

struct VecShared {
    // cos and sin of two pairs, (c, c', s, s'); piece j of chunk c at j * rot_chunks + c, so that the lanes
    // of a row read without conflicts
    float4 angles[kTokens][kVecPairs / 2];
    int place[kTokens][4];           // status (append_place), page, slot, position
};

// The rows of one role (0 query, 1 key, 2 value) of the CTA's tokens.
template <typename T, bool kInter, int kCache, int kRole> struct Rows {
    static constexpr int V = kVec<T>, H = V / 2;
    const T *x;                      // token n0
    long x_tok, x_head;
    int heads, rows, step;
    int row, t, h;                   // the next to load
    uint4 a, b;                      // the loaded one: its vectors, its token (-1 behind the last row) and head
    int rt, rh;

    __device__ __forceinline__ void load(bool live, bool two, int oa, int ob) {
        rt = row < rows ? t : -1;
        rh = h;
        if (row < rows) {
            const T *src = x + t * x_tok + h * x_head;
            if (live) a = *reinterpret_cast<const uint4 *>(src + oa);
            if (two) b = *reinterpret_cast<const uint4 *>(src + ob);
        }
        row += step;
        h += step;
        if (h >= heads) {
            h -= heads;
            ++t;
            if (h >= heads) {
                const int q = (int)((unsigned)h / (unsigned)heads);
                t += q;
                h -= q * heads;
            }
        }
    }
    __device__ __forceinline__ Rows(const NormRopeParams &p, int n0, int nt, int first, int step_) {
        x = static_cast<const T *>(kRole == 0 ? p.q : kRole == 1 ? p.k : p.v) + (long)n0 * (kRole == 0 ? p.q_tok : p.k_tok);
        x_tok = kRole == 0 ? p.q_tok : p.k_tok;
        x_head = kRole == 0 ? p.q_head : p.k_head;
        heads = kRole ? p.Hk : kCache ? max(1, p.Hq) : p.Hq;      // (an append may have no queries: no rows, but a walk that divides)
        rows = nt * (kRole == 0 ? p.Hq : p.Hk);
        step = step_;
        row = first;
        t = (int)((unsigned)row / (unsigned)heads);
        h = row - t * heads;
        a = b = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void run(const NormRopeParams &p, const VecShared &sh, int n0, int log_p, int rot_chunks, int c,
                                        bool live, bool two, int oa, int ob) {
        const T *w = static_cast<const T *>(kRole == 0 ? p.wq : kRole == 1 ? p.wk : nullptr);
        float2 ga[H], gb[H];
        if (kRole < 2) {
            uint4 wa = make_uint4(0u, 0u, 0u, 0u), wb = wa;
            if (w && live) wa = __ldg(reinterpret_cast<const uint4 *>(w + oa));
            if (w && two) wb = __ldg(reinterpret_cast<const uint4 *>(w + ob));
            unpack2(wa, ga);
            unpack2(wb, gb);
        }
        const bool turned = kRole < 2 && c < rot_chunks;
        // whole warps go through the loop, rows or not: sums over some of a warp's lanes under a mask of their
        // own would cost a synchronisation each (25,119 x 32 heads 77.7 us)
        const int width = 1 << log_p;
        while (__any_sync(0xffffffffu, rt >= 0)) {
            const uint4 ca = a, cb = b;
            const int ct = rt, ch = rh;
            load(live, two, oa, ob);
            const int tok = max(ct, 0);
            const int *at = sh.place[tok];
            const bool write = ct >= 0 && !(kCache && (kRole ? at[0] < 0 : at[0] == -2));
            float2 fa[H], fb[H];
            unpack2(ca, fa);
            unpack2(cb, fb);
            if (kRole < 2 && w) {
                float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
                for (int e = 0; e < H; ++e) s2 = __ffma2_rn(fa[e], fa[e], s2);
                if (!kInter)
#pragma unroll
                    for (int e = 0; e < H; ++e) s2 = __ffma2_rn(fb[e], fb[e], s2);
                float sum = s2.x + s2.y;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1)
                    if (o < width) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                const float inv = rsqrtf(fmaf(sum, p.inv_dim, p.eps));
                const float2 i2 = make_float2(inv, inv);
#pragma unroll
                for (int e = 0; e < H; ++e) fa[e] = __fmul2_rn(__fmul2_rn(fa[e], i2), ga[e]);
                if (!kInter)
#pragma unroll
                    for (int e = 0; e < H; ++e) fb[e] = __fmul2_rn(__fmul2_rn(fb[e], i2), gb[e]);
            }
            if (turned) {
                const float4 *angle = sh.angles[tok] + c;
                if constexpr (kInter) {            // element pairs (a, b) side by side
#pragma unroll
                    for (int e = 0; e < H; e += 2) {
                        const float4 cs = angle[(e >> 1) * rot_chunks];
                        const float2 u = fa[e], v = fa[e + 1];
                        fa[e] = make_float2(u.x * cs.x - u.y * cs.z, u.y * cs.x + u.x * cs.z);
                        fa[e + 1] = make_float2(v.x * cs.y - v.y * cs.w, v.y * cs.y + v.x * cs.w);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < H; ++e) {
                        const float4 cs = angle[e * rot_chunks];
                        const float2 co = make_float2(cs.x, cs.y), si = make_float2(cs.z, cs.w), u = fa[e], v = fb[e];
                        fa[e] = __ffma2_rn(u, co, neg2(__fmul2_rn(v, si)));
                        fb[e] = __ffma2_rn(u, si, __fmul2_rn(v, co));
                    }
                }
            }
            if constexpr (kCache == 2 && kRole > 0) {
                float amax = 0.f;
                if (live)
#pragma unroll
                    for (int e = 0; e < H; ++e) amax = fmaxf(amax, fmaxf(fabsf(fa[e].x), fabsf(fa[e].y)));
                if (two)
#pragma unroll
                    for (int e = 0; e < H; ++e) amax = fmaxf(amax, fmaxf(fabsf(fb[e].x), fabsf(fb[e].y)));
#pragma unroll
                for (int o = 1; o < 32; o <<= 1)
                    if (o < width) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                const RowCodes code(amax);
                uint8_t *codes = static_cast<uint8_t *>(kRole == 1 ? p.k_pages : p.v_pages) + (long)at[1] * p.pages.b +
                                 (long)at[2] * p.pages.s + (long)ch * p.pages.h;
                auto put = [&](int o, const float2 (&f)[H]) {
                    uint32_t q[V / 4];
#pragma unroll
                    for (int e = 0; e < V / 4; ++e) {
                        const float2 x = code(f[2 * e]), y = code(f[2 * e + 1]);
                        q[e] = e4m3x4(x.x, x.y, y.x, y.y);
                    }
                    if constexpr (V == 8) *reinterpret_cast<uint2 *>(codes + o) = make_uint2(q[0], q[1]);
                    else *reinterpret_cast<uint32_t *>(codes + o) = q[0];
                };
                if (live && write) put(oa, fa);
                if (two && write) put(ob, fb);
                if (c == 0 && write)
                    (kRole == 1 ? p.k_scale : p.v_scale)[((long)at[1] * p.Hk + ch) * p.page_size + at[2]] = e4m3_scale(amax);
            } else {
                const long n = n0 + tok;
                T *y = kRole == 0  ? static_cast<T *>(p.q_out) + n * p.qo_tok + ch * p.qo_head
                       : !kCache ? static_cast<T *>(p.k_out) + n * p.ko_tok + ch * p.ko_head
                                 : static_cast<T *>(kRole == 1 ? p.k_pages : p.v_pages) + (long)at[1] * p.pages.b +
                                       (long)at[2] * p.pages.s + (long)ch * p.pages.h;
                // (values bit for bit)
                if (live && write) *reinterpret_cast<uint4 *>(y + oa) = kRole == 2 ? ca : pack2(fa);
                if (two && write) *reinterpret_cast<uint4 *>(y + ob) = kRole == 2 ? cb : pack2(fb);
            }
        }
    }
};

template <typename T, bool kInter, int kCache>       // kCache: 0 no cache, 1 pages of T, 2 of codes
__global__ void __launch_bounds__(kVecThreads, 7)
norm_rope_vec_kernel(const __grid_constant__ NormRopeParams p, const int log_p, const int rot_chunks, const int chunks,
                     const int tokens, const int checks) {
    constexpr int V = kVec<T>, NP = kInter ? V / 2 : V;
    __shared__ VecShared sh;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x;
    if (kCache && (int)blockIdx.x < checks) {
        const int b = (int)blockIdx.x * kVecThreads + tid;
        if (b < p.B) append_check(p, b);
        return;
    }
    const int n0 = ((int)blockIdx.x - checks) * tokens, nt = min(tokens, p.N - n0);
    const int lane = tid & 31, c = lane & ((1 << log_p) - 1);
    const bool turned = c < rot_chunks, live = c < chunks;
    // a chunk's elements: [oa, oa + V) and, of pairs in the half layout, [ob, ob + V)
    const int oa = turned ? c * V : p.rot + (c - rot_chunks) * V;
    const int ob = oa + p.rot / 2;
    const bool two = turned && !kInter;
    const int first = tid >> log_p, step = kVecThreads >> log_p;
    Rows<T, kInter, kCache, 0> q(p, n0, nt, first, step);
    q.load(live, two, oa, ob);
    if (kCache) {
        if (tid < nt) {
            int pos = 0, page = 0, slot = 0;
            sh.place[tid][0] = append_place(p, n0 + tid, pos, page, slot);
            sh.place[tid][1] = page;
            sh.place[tid][2] = slot;
            sh.place[tid][3] = pos;
        }
        if (!p.positions) __syncthreads();
    }
    const int half = p.rot / 2;
    for (int i = tid; i < nt * half; i += kVecThreads) {
        const int k = (int)((unsigned)i / (unsigned)half), pair = i - k * half;
        const int pos = p.positions ? __ldg(p.positions + (long)pair_axis(p, pair) * p.pos_stride + n0 + k) : sh.place[k][3];
        const int e = pair % NP;
        const float2 cs = rope_cs(__ldg(p.turns + pair), pos, p.magnitude);
        float *to = reinterpret_cast<float *>(&sh.angles[k][(e >> 1) * rot_chunks + pair / NP]) + (e & 1);
        to[0] = cs.x;
        to[2] = cs.y;
    }
    __syncthreads();
    q.run(p, sh, n0, log_p, rot_chunks, c, live, two, oa, ob);
    if (p.Hk) {
        Rows<T, kInter, kCache, 1> k(p, n0, nt, first, step);
        k.load(live, two, oa, ob);
        k.run(p, sh, n0, log_p, rot_chunks, c, live, two, oa, ob);
    }
    if (kCache) {
        Rows<T, kInter, kCache, 2> v(p, n0, nt, first, step);
        v.load(live, two, oa, ob);
        v.run(p, sh, n0, log_p, rot_chunks, c, live, two, oa, ob);
    }
}

// whole vectors of turned pairs and of the rest, at most one warp of chunks, every row on a 16-byte boundary
template <typename T> int vec_chunks(const NormRopeParams &p) {
    constexpr int V = kVec<T>;
    auto al = [](const void *q) { return (reinterpret_cast<uintptr_t>(q) & 15u) == 0; };
    if (p.D % V || p.rot % (p.interleaved ? V : 2 * V)) return 0;
    if (!al(p.wq) || !al(p.wk)) return 0;
    if (p.Hq && (!al(p.q) || !al(p.q_out) || p.q_tok % V || p.q_head % V || p.qo_tok % V || p.qo_head % V)) return 0;
    if (p.Hk && (!al(p.k) || p.k_tok % V || p.k_head % V)) return 0;
    if (p.Hk && !p.v && (!al(p.k_out) || p.ko_tok % V || p.ko_head % V)) return 0;
    // (rows of codes need V bytes, which the strides' V elements are; and no more of their bases)
    auto fits = [&](const void *q) { return reinterpret_cast<uintptr_t>(q) % (p.k_scale ? V : 16) == 0; };
    if (p.v && (!al(p.v) || !fits(p.k_pages) || !fits(p.v_pages) || p.pages.b % V || p.pages.s % V || p.pages.h % V)) return 0;
    const int chunks = p.rot / (p.interleaved ? V : 2 * V) + (p.D - p.rot) / V;
    return chunks <= 32 ? chunks : 0;
}

template <typename T, bool kInter, int kCache>
cudaError_t launch_vec(NormRopeParams p, int chunks, cudaStream_t st) {
    constexpr int V = kVec<T>;
    int log_p = 0;
    while (1 << log_p < chunks) ++log_p;
    p.inv_dim = 1.f / (float)p.D;
    const int checks = kCache ? (p.B + kVecThreads - 1) / kVecThreads : 0;      // CTAs that look over the sequences
    // several tokens to a CTA, as long as every SM gets six CTAs (2,048 tokens of 80 heads into a bf16 cache:
    // 17.4 us with two, 19.7 with one; 25,119 of 36 into one of 8 bits: 81.4 with eight, 83.2 with four, 95.6 with two)
    const int tokens = std::max(1, std::min(kTokens, p.N / (6 * std::max(1, device_sm_count()))));
    const long blocks = checks + ((long)p.N + tokens - 1) / tokens;
    if (blocks > 0x7fffffffL) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kVecThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, norm_rope_vec_kernel<T, kInter, kCache>, p, log_p, p.rot / (kInter ? V : 2 * V), chunks,
                              tokens, checks);
}

template <typename T, bool kInter> cudaError_t launch_cache(const NormRopeParams &p, int chunks, cudaStream_t st) {
    if (!p.v) return launch_vec<T, kInter, 0>(p, chunks, st);
    return p.k_scale ? launch_vec<T, kInter, 2>(p, chunks, st) : launch_vec<T, kInter, 1>(p, chunks, st);
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

template <typename T> cudaError_t launch_type(const NormRopeParams &p, cudaStream_t st) {
    const int chunks = vec_chunks<T>(p);
    if (!chunks) return launch_rows<T>(p, st);
    return p.interleaved ? launch_cache<T, true>(p, chunks, st) : launch_cache<T, false>(p, chunks, st);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams &p, cudaStream_t st) {
    return p.dt == SD_BF16 ? launch_type<__nv_bfloat16>(p, st) : launch_type<float>(p, st);
}

}  // namespace sdv
