// Attention of packed new tokens on CUDA cores: fp32 or bf16 storage, any page
// size, fp32 arithmetic throughout.  The tensor-core kernel takes the bf16
// calls it can (attn_varlen_tc.cu); this one takes the rest.
//
// A unit is R query rows (64, or 16 where no sequence has more rows per kv
// head than that) and its keys come in tiles of 64; units and tiles are dealt
// out as in varlen.cuh.  256 threads as 16 x 16: thread (ty, tx) computes
// R / 16 rows x 4 keys of S = Q K^T from transposed tiles in shared memory,
// the 16 threads of a row find its maximum and sum by shuffles, and the same
// thread adds P V for its rows and D / 16 of the columns, O in registers.
// The keys lie transposed and swizzled in shared memory, the weights go over
// them, and multiply-adds come two an instruction.  What bounds it: with 64 rows
// the shared-memory reads that feed the FMA pipe (410 tokens of 64 heads over 544
// keys, fp32: 394 us, 32 TFLOP/s), with 16 the latency of a tile's load, product
// and softmax one after the other (16 rows of 4 heads over 527 keys: 14 to 18 us).
// Causal fp32 prompts of 2,048 and 8,192 tokens, 28 / 4 heads of 128: 0.82 and 11.9
// ms, 37 and 41 TFLOP/s.
// Codes of an 8-bit cache (fp32 queries, or pages that are no multiple of 8 slots) are
// multiplied by their row's scale in fp32 where a tile is loaded, and a tree's words
// are looked at where a causal edge is; the rest is the same.
#include "e4m3.cuh"
#include "varlen.cuh"

#include <math.h>
#include <atomic>

namespace sdv {

namespace {

constexpr int kGThreads = 256;
constexpr int kGTile = 1 << kVarlenGenTileLog2;      // 64 keys
constexpr float kGLog2e = 1.4426950408889634f;

template <int D, int R> struct GLay {
    static constexpr int kQs = R + 4;               // transposed rows, padded: 16-byte aligned, bank-shifted
    static constexpr int kKs = kGTile;              // transposed keys, swizzled (key_at)
    static constexpr int kQ = D * kQs;              // floats
    static constexpr int kK = D * kKs;              // P overlays K: [kGTile][kQs]
    static constexpr int kV = kGTile * D;
    static constexpr int kP = kGTile * kQs;         // P has its own room where K's is too small
    static constexpr int kSmem = (kQ + (kK > kP ? kK : kP) + kV) * 4;
};

// Element (d, key) of the transposed keys: groups of 4 keys, exchanged within a
// row by d / 4, so that a warp that stores 8 vectors of 4 keys hits 32 banks and
// one that reads 64 keys of a row does too.
__device__ __forceinline__ int key_at(int d, int key4) { return d * kGTile + ((key4 ^ ((d >> 2) & 15)) << 2); }

// offset of key `key`'s row of the unit's kv head, or -1 for a bad page; `scale_at` that of its scales
__device__ __forceinline__ long key_offset(const VarlenParams &p, const VlUnit &u, int key, long &scale_at) {
    if (!p.table) return (long)(u.row0 - u.tok0 + key) * p.kv.s + (long)u.g * p.kv.h;
    const unsigned pi = p.page_log2 >= 0 ? (unsigned)key >> p.page_log2 : (unsigned)key / (unsigned)p.page_size;
    const int pg = __ldg(p.table + (long)u.b * p.table_stride + pi);
    if (pg < 0 || pg >= p.n_pages) { set_fault(p.fault, FAULT_BAD_PAGE); return -1; }
    const int slot = key - (int)pi * p.page_size;
    scale_at = ((long)pg * p.Hkv + u.g) * p.page_size + slot;
    return (long)pg * p.kv.b + (long)slot * p.kv.s + (long)u.g * p.kv.h;
}

// T: the queries' type, C: the cache's (T itself, or e4m3 codes with a scale per row)
template <typename T, typename C, int D, int R>
__global__ void __launch_bounds__(kGThreads, 2)
attn_varlen_generic_kernel(const VarlenParams p) {
    using L = GLay<D, R>;
    constexpr int TM = R / 16, TN = D / 16;          // rows and output columns of a thread
    constexpr int VP = Elem<T>::kPerVec, VPR = D / VP;
    constexpr int CP = Elem<C>::kPerVec, CPR = D / CP;
    constexpr bool kScaled = sizeof(C) == 1;
    extern __shared__ float4 smem4[];
    float *Qs = reinterpret_cast<float *>(smem4);    // [D][R + 4]
    float *Ks = Qs + L::kQ;                          // [D][64], swizzled
    float *Ps = Ks;                                  // [64][R + 4]
    float *Vs = Ks + (L::kK > L::kP ? L::kK : L::kP);  // [64][D]
    __shared__ VlPlan pl;
    __shared__ VlEnds ends;
    __shared__ int join_flag;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int cta = (int)blockIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (tid < 32) {
        const VlPlan q = vl_plan(p, cta);
        vl_plan_store(q, &pl);
    }
    __syncthreads();
    if (pl.idle) return;
    const int G = p.Hq / p.Hkv;
    const float qk = p.scale * kGLog2e;

    VlWalk walk(pl);
    VlUnit u;
    while (walk.next(p, pl, u)) {
        const int rows = u.ntok * G;
        __syncthreads();
        for (int i = tid; i < R * VPR; i += kGThreads) {       // Q, scaled, transposed
            const int r = i % R, v = i / R;
            float f[VP];
            if (r < rows) {
                const T *src = static_cast<const T *>(p.q) + (long)(u.row0 + r / G) * p.q_tok +
                               (long)(u.g * G + r % G) * p.q_head + v * VP;
                Elem<T>::load_vec(src, f);
            } else {
#pragma unroll
                for (int e = 0; e < VP; ++e) f[e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < VP; ++e) Qs[(v * VP + e) * L::kQs + r] = f[e] * qk;
        }
        float o[TM][TN], m[TM], l[TM];
        int lim[TM];
        uint64_t seen[TM];                             // of a tree: the block's slots that the row sees
#pragma unroll
        for (int a = 0; a < TM; ++a) {
            const int r = ty * TM + a;
            lim[a] = r < rows ? vl_limit(p, u, u.tok0 + r / G) : 0;
            seen[a] = p.tree && r < rows ? vl_tree_word(p, u, r / G) : 0;
            m[a] = -INFINITY;
            l[a] = 0.f;
#pragma unroll
            for (int e = 0; e < TN; ++e) o[a][e] = 0.f;
        }
        for (int t = u.t0; t < u.t1; ++t) {
            const int key0 = t * kGTile;
            __syncthreads();
            // a warp takes 8 vectors of 4 keys at a time
            for (int i = tid >> 5; i < (kGTile / 4) * (CPR / 8); i += kGThreads / 32) {
                const int kk = 4 * (i / (CPR / 8)) + ((tid >> 3) & 3), v = 8 * (i % (CPR / 8)) + (tid & 7);
                float kf[CP], vf[CP];
                const C *kp = nullptr, *vp = nullptr;
                float ks = 1.f, vs = 1.f;
                if (key0 + kk < u.kv) {
                    long scale_at = 0;
                    const long at = key_offset(p, u, key0 + kk, scale_at);
                    if (at >= 0) {
                        kp = static_cast<const C *>(p.k) + at;
                        vp = static_cast<const C *>(p.v) + at;
                        if constexpr (kScaled) {
                            ks = __ldg(p.k_scale + scale_at);
                            vs = __ldg(p.v_scale + scale_at);
                        }
                    }
                }
                if (kp) {
                    Elem<C>::load_vec(kp + v * CP, kf);
                    Elem<C>::load_vec(vp + v * CP, vf);
                    if constexpr (kScaled) {
#pragma unroll
                        for (int e = 0; e < CP; ++e) { kf[e] *= ks; vf[e] *= vs; }
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < CP; ++e) { kf[e] = 0.f; vf[e] = 0.f; }
                }
#pragma unroll
                for (int e = 0; e < CP; ++e) Ks[key_at(v * CP + e, kk >> 2) + (kk & 3)] = kf[e];
#pragma unroll
                for (int e = 0; e < CP; e += 4)
                    *reinterpret_cast<float4 *>(Vs + kk * D + v * CP + e) = make_float4(vf[e], vf[e + 1], vf[e + 2], vf[e + 3]);
            }
            __syncthreads();
            float2 s2[TM][2];
#pragma unroll
            for (int a = 0; a < TM; ++a) s2[a][0] = s2[a][1] = make_float2(0.f, 0.f);
#pragma unroll 8
            for (int d = 0; d < D; ++d) {
                const float4 k4 = *reinterpret_cast<const float4 *>(Ks + key_at(d, tx));
                float q[TM];
                if constexpr (TM == 4) {
                    const float4 q4 = *reinterpret_cast<const float4 *>(Qs + d * L::kQs + 4 * ty);
                    q[0] = q4.x; q[1] = q4.y; q[2] = q4.z; q[3] = q4.w;
                } else {
                    q[0] = Qs[d * L::kQs + ty];
                }
#pragma unroll
                for (int a = 0; a < TM; ++a) {       // two multiply-adds an instruction
                    s2[a][0] = __ffma2_rn(make_float2(q[a], q[a]), make_float2(k4.x, k4.y), s2[a][0]);
                    s2[a][1] = __ffma2_rn(make_float2(q[a], q[a]), make_float2(k4.z, k4.w), s2[a][1]);
                }
            }
            float s[TM][4];
#pragma unroll
            for (int a = 0; a < TM; ++a) {
                s[a][0] = s2[a][0].x; s[a][1] = s2[a][0].y;
                s[a][2] = s2[a][1].x; s[a][3] = s2[a][1].y;
            }
            __syncthreads();       // K has been read; P goes over it
#pragma unroll
            for (int a = 0; a < TM; ++a) {
                float mx = -INFINITY;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int key = key0 + 4 * tx + c;
                    if (key >= lim[a] || (p.tree && key >= u.off && !(seen[a] >> (key - u.off) & 1))) s[a][c] = -INFINITY;
                    mx = fmaxf(mx, s[a][c]);
                }
#pragma unroll
                for (int x = 1; x < 16; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
                const float m_new = fmaxf(m[a], mx);
                const float ref = m_new == -INFINITY ? 0.f : m_new;
                const float alpha = exp2f(m[a] - ref);         // 0 while nothing is held
                m[a] = m_new;
                float sum = 0.f;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    s[a][c] = exp2f(s[a][c] - ref);
                    sum += s[a][c];
                }
#pragma unroll
                for (int x = 1; x < 16; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
                l[a] = fmaf(l[a], alpha, sum);
#pragma unroll
                for (int e = 0; e < TN; ++e) o[a][e] *= alpha;
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float *to = Ps + (4 * tx + c) * L::kQs + ty * TM;
                if constexpr (TM == 4) *reinterpret_cast<float4 *>(to) = make_float4(s[0][c], s[1][c], s[2][c], s[3][c]);
                else *to = s[0][c];
            }
            __syncthreads();
#pragma unroll 4
            for (int kk = 0; kk < kGTile; ++kk) {
                float q[TM];
                if constexpr (TM == 4) {
                    const float4 q4 = *reinterpret_cast<const float4 *>(Ps + kk * L::kQs + 4 * ty);
                    q[0] = q4.x; q[1] = q4.y; q[2] = q4.z; q[3] = q4.w;
                } else {
                    q[0] = Ps[kk * L::kQs + ty];
                }
#pragma unroll
                for (int c = 0; c < TN; c += 4) {              // columns 64 (c / 4) + 4 tx ..: neighbours read 16 bytes each
                    const float4 v4 = *reinterpret_cast<const float4 *>(Vs + kk * D + 16 * c + 4 * tx);
#pragma unroll
                    for (int a = 0; a < TM; ++a) {
                        const float2 w = make_float2(q[a], q[a]);
                        float2 lo = make_float2(o[a][c], o[a][c + 1]), hi = make_float2(o[a][c + 2], o[a][c + 3]);
                        lo = __ffma2_rn(w, make_float2(v4.x, v4.y), lo);
                        hi = __ffma2_rn(w, make_float2(v4.z, v4.w), hi);
                        o[a][c] = lo.x; o[a][c + 1] = lo.y; o[a][c + 2] = hi.x; o[a][c + 3] = hi.y;
                    }
                }
            }
        }
        const bool whole = u.t0 == 0 && u.t1 == u.tiles;
        const long slot = u.t0 == 0 ? 2L * cta + 1 : 2L * cta;
#pragma unroll
        for (int a = 0; a < TM; ++a) {
            const int r = ty * TM + a;
            if (r >= rows) continue;
            const float inv = l[a] > 0.f ? 1.f / l[a] : 0.f;
#pragma unroll
            for (int c = 0; c < TN; c += 4) {
                const float4 v = make_float4(o[a][c], o[a][c + 1], o[a][c + 2], o[a][c + 3]);
                const int c4 = 4 * c + tx;
                if (whole)
                    vl_store4(p, (long)(u.row0 + r / G) * p.Hq + u.g * G + r % G, c4,
                              make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
                else
                    __stcg(reinterpret_cast<float4 *>(p.o_part) + (slot * (D / 4) + c4) * p.rows + r, v);
            }
            if (!whole && tx == 0) __stcg(p.ml_part + slot * p.rows + r, make_float2(m[a], l[a]));
        }
    }
    if (tid < 32) {
        vl_ends(p, pl, cta, &ends);
    }
    __threadfence();
    __syncthreads();
    if (tid < ends.n) vl_arrive(p, ends.u[tid]);
    for (int i = 0; i < ends.n; ++i) vl_join(p, ends.u[i], p.tb, 0, &join_flag, tid, kGThreads, 0);
}

template <typename T, typename C, int D, int R>
int grid_of() {
    using L = GLay<D, R>;
    static std::atomic<int> per_sm[kMaxDevices];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev >= 0 && dev < kMaxDevices) n = per_sm[dev].load(std::memory_order_acquire);
    if (n == 0) {
        if (cudaFuncSetAttribute(attn_varlen_generic_kernel<T, C, D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 L::kSmem) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, attn_varlen_generic_kernel<T, C, D, R>, kGThreads,
                                                          L::kSmem) != cudaSuccess)
            return 0;
        n = n < kVarlenGenPerSm ? n : kVarlenGenPerSm;
        if (dev >= 0 && dev < kMaxDevices) per_sm[dev].store(n, std::memory_order_release);
    }
    return n * device_sm_count();
}

template <typename T, typename C, int D, int R>
cudaError_t launch_gen(const VarlenParams &p, int grid, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kGThreads);
    cfg.dynamicSmemBytes = GLay<D, R>::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeCooperative;     // the CTAs of a shared unit wait for one another
    attr[1].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, attn_varlen_generic_kernel<T, C, D, R>, p);
}

template <typename T, typename C, typename F> auto by_size(const VarlenParams &p, F f) {
    const bool big = varlen_generic_rows(p) == 64;
    if (p.D == 128) return big ? f.template run<T, C, 128, 64>() : f.template run<T, C, 128, 16>();
    return big ? f.template run<T, C, 64, 64>() : f.template run<T, C, 64, 16>();
}
template <typename F> auto dispatch(const VarlenParams &p, F f) {
    using bf = __nv_bfloat16;
    if (p.k_scale) return p.dt == SD_BF16 ? by_size<bf, E4m3>(p, f) : by_size<float, E4m3>(p, f);
    return p.dt == SD_BF16 ? by_size<bf, bf>(p, f) : by_size<float, float>(p, f);
}

struct GridOf {
    template <typename T, typename C, int D, int R> int run() const { return grid_of<T, C, D, R>(); }
};
struct Launch {
    const VarlenParams &p;
    int grid;
    cudaStream_t st;
    template <typename T, typename C, int D, int R> cudaError_t run() const { return launch_gen<T, C, D, R>(p, grid, st); }
};

}  // namespace

// 16 rows where they hold every sequence's rows of a kv head: a tile then costs a
// quarter of the multiply-adds
int varlen_generic_rows(const VarlenParams &p) { return (long)p.max_q * (p.Hq / p.Hkv) <= 16 ? 16 : 64; }

int varlen_max_grid(int path, const VarlenParams &p) {
    return path >= 2 ? device_sm_count() : dispatch(p, GridOf{});
}

cudaError_t launch_varlen_generic(const VarlenParams &p, int grid, cudaStream_t st) {
    return dispatch(p, Launch{p, grid, st});
}

}  // namespace sdv
