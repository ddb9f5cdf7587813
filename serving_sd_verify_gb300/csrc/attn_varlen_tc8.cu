// Attention of packed new tokens over a paged cache in 8 bits (e4m3 codes with a
// scale per row) on the tensor cores, for sm_103a: bf16 queries and outputs, pages
// of a multiple of 8 slots, D of 64 or 128.
//
// The products run in e4m3 on the codes as they lie in the cache: no key or value is
// ever widened, so a tile of 128 keys is 16 KB to copy and to read instead of 32.
// With k_n, v_n the scales of key n, and for a unit (up to 256 query rows, as in
// attn_varlen_tc.cu, whose tiles, streams and joins these are):
//   S = (Q1 + Q2) K^T,  x_n = S_n k_n c,  m = max(x_n + log2 v_n) of the keys that the row sees
//   P_n = 2^u exp2(x_n - m),  l = sum P_n,  W_n = P_n v_n,  O = (W1 + W2 + W3) V,  out = O / l
//   Q: a row times a power of two that brings its largest element to [128, 256), as
//     a first e4m3 term and, exactly, what that leaves: a bf16 element has 8 bits and
//     each term holds 4, so the two are the element itself where it is above 2^-9
//     of the row's largest, and off by 2^-17 of the largest where not.  c is that
//     power's inverse times scale log2(e).
//   m: of what the keys contribute, their values' scales among it: a row's weights are
//     written against nothing but what the row itself sees, and neither a value that it
//     does not see, however large, nor one that it sees of small values, however large
//     its score, takes precision from the others.  It moves where a weight would pass
//     what the terms hold (max x and the part's largest scale tell that none does, mostly),
//     to max x and that scale where all the part's keys are seen and their scales are alike,
//     else to the keys' own (with two e4m3 terms, 2,048 over 32,768 2.17 ms; the keys' own
//     always, a third reading of each key's scales, 2.77; weights made first and looked
//     over behind 2.7 to 2.9).
//   W: in f16, and that in three e5m2 terms of 3 bits each (an e5m2 code is the upper
//     byte of an f16 value): off by 2^-9 of itself, or by 2^-17 where it is small.  With u
//     of 9 that is 2^-24 of the row's largest, so that a long rest far below one large
//     weight is kept: the 65,536 keys that it holds for lose 2^-8 of the sum of the weights
//     together at most, and for longer caches u grows with them.  (Two e4m3 terms end
//     at 2^-10 and 2^-14 of the largest: with one key 12 nats above 32,768 others a third
//     of the output went; one in e4m3 and one in e5m2 with m moved down where the
//     small ones had lost too much: 2.69 ms, error 2.1e-3 for 1.73e-3.)
// l takes P before any rounding.
//
// Warps as in attn_varlen_tc.cu, except that the softmax warps split and write Q
// (thread = row, which keeps its power of two), warp 2 reads the scales ahead and
// hands them over in a ring of kScaleSlots tiles, and warp 3 works out the units for
// all of them.
// Tensor memory: S_0 [0,128), S_1 [128,256), O_0 [256,256+D), O_1 [384,384+D).  A
// tile's scores come in two parts of 64 keys, whose weights go over the first 48 of
// their 64 columns: while a stream's softmax has one part, the tensor pipe adds the
// other's weights to O and makes the next tile's scores there, so that a warp does not
// wait for its own products (with two terms, 2,048 over 32,768: 5,400 clocks a pair of
// tiles, in one part 6,000).  Where a call's rows fit 32 of a tile's 128
// (decoding), Q's tile holds them four times and warp w of a stream takes keys
// [32 w, 32 w + 32) of a tile for all of them (64 sequences of one token: 119 -> 90 us).
//
// Measured.  2,048 tokens over 32,768 (64 / 8 heads): 2.43 ms, 0.88 PFLOP/s, against
// 1.49 in bf16; one token over 25,119 (28 / 4) 22.2 us for 26.5 MB; 64 sequences of one
// over 1,000 to 9,000, pages of 16, 86 us for 249 MB; 8 trees of 60 nodes 159 us.  With
// two e4m3 terms a weight 2.17 ms, 20.6, 86 and 164 us, and a tail that gets lost.
// What bounds it: the one warp that issues the products -- a part of 64 keys costs it
// 8 products for the scores (64 columns wide, each reads Q's 128 rows again) and 6 for O,
// and waits and commits -- and the chain of a part's scores, softmax and second
// product; in calls of few rows also a unit's start and end (9,000 clocks).  With
// two e4m3 terms were measured: a second issuing warp, 2.2 to 4.2 ms; four softmax
// warpgroups, 2.5 to 3.6 (104 registers a thread spill).
//
// Every wait is bounded; one that gives up sets the fault word, and the CTA
// drains its copies and MMAs before it returns.
#include "e4m3.cuh"
#include "varlen_tc.cuh"

namespace sdv {

namespace {

// In log2 units: the largest weight when m has been chosen, for up to 2^16 keys, and for any number; what a weight
// may be (f16 and e5m2 end at 2^16 and 2^15.8); what P may be (so that 2^26 of them, with rows of zeros beside others,
// stay finite); by how much scales that are alike differ.
constexpr float kWeightLog = 9.0f, kWeightLogMost = 14.0f, kWeightTop = 15.7f, kSumTop = 90.0f, kAlike = 1.5f;
constexpr int kScaleSlots = 4;

// a tile's scales, V's logarithms, and the largest and the smallest of those of each 32 keys
struct Scales {
    float k[128], v[128], log_v[128];
    float2 range[4];
};
// log2 of a scale, of no less than 2^-80: a row of zeros has a scale of 2^-109, and its P should stay finite
__device__ __forceinline__ float log_scale(float v) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(fmaxf(v, 0x1p-80f)));
    return y;
}

// The CTA's units, worked out by warp 3 ahead of everyone (each role's own walk would be on its way at
// every unit, and four copies of its code in the instruction cache).  Softmax warps read theirs here
// throughout: registers it would hold are spilled within the tiles' loop, to L2 (shared memory leaves
// L1 little).
struct Unit8 {
    VlUnit u;
    int more;           // 0: the last unit was the one before
    int alone;          // its sequence's only unit of a kv head
};
constexpr int kUnitSlots = 4, kUnitReaders = 3 + 8;      // warps 0 to 2, and the softmax warps

template <int D> struct Lay8 {
    static constexpr int kTile = 128 * D;                  // one term of Q, K or V: 128 rows of D bytes
    static constexpr int kSlots = D == 128 ? 9 : 16;
    static constexpr int kOffQ = 0;                        // two row tiles of two terms
    static constexpr int kOffRing = 4 * kTile;
    static constexpr int kMaxSlots = kSlots + 2;           // where no unit has a second row tile, its room too
    static constexpr int kOffScale = kOffRing + kSlots * kTile;
    static constexpr int kOffBar = kOffScale + kScaleSlots * (int)sizeof(Scales);
    // full[max] empty[max] qfull drain sfull[2][2] pfull[2][2] ofull[2] ofree[2] oadd[2] scfull[] scempty[] ufull[] uempty[]
    static constexpr int kBars = 2 * kMaxSlots + 2 + 4 + 4 + 2 + 2 + 2 + 2 * kScaleSlots + 2 * kUnitSlots;
    static constexpr int kOffMl = kOffBar + 8 * kBars;     // [2][128] exchange between the streams
    static constexpr int kOffMisc = kOffMl + 2 * 128 * 4;
    static constexpr int kOffUnits = kOffMisc + 512;
    static constexpr int kSmem = kOffUnits + kUnitSlots * (int)sizeof(Unit8) + 1024;    // + alignment slack
    static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
    static_assert(kOffBar % 16 == 0 && kOffMl % 16 == 0, "aligned parts");
};

// K or V of `box` slots of one page, with an L2 policy
__device__ __forceinline__ void load_page(uint32_t dst, const CUtensorMap *map, uint32_t bar, uint64_t policy, int slot,
                                          int g, int page) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(slot), "r"(g), "r"(page), "r"(bar), "l"(policy)
        : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), SDV_S8(0)
                 : "memory");
}
__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}

// instruction descriptor, kind::f8f6f4: A e4m3 or e5m2, K-major; B e4m3; fp32 D
__host__ __device__ constexpr uint32_t idesc_8(int M, int N, bool a_e5m2, bool b_mn_major) {
    return (1u << 4) | ((a_e5m2 ? 1u : 0u) << 7) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void umma8_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void umma8_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// descriptor of rows of D bytes in 8-row groups, swizzled within their D bytes
template <int D> __device__ __forceinline__ uint64_t row_desc(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)1 << 16;
    d |= (uint64_t)(8 * D / 16) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)(D == 128 ? 2 : 4) << 61;       // 128-byte or 64-byte swizzle
    return d;
}
// byte offset of 16-byte chunk c of row r in such a tile
template <int D> __device__ __forceinline__ uint32_t row_off(int r, int c) {
    return D == 128 ? sw128_off(r, c) : (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

// Row r of the Q tile at `tile` (the second term's tile behind the first's): the
// part-th of `parts` equal shares of its columns, in two terms.
// Returns what the products have to be multiplied by.
template <int D>
__device__ __forceinline__ float put_query(const __nv_bfloat16 *q, uint8_t *tile, int r, int part, int parts) {
    uint32_t top = 0;                                  // the largest magnitudes, as pairs of bit patterns
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(q) + i);
        top = __vmaxu2(__vmaxu2(__vmaxu2(top, v.x & 0x7fff7fffu), __vmaxu2(v.y & 0x7fff7fffu, v.z & 0x7fff7fffu)),
                       v.w & 0x7fff7fffu);
    }
    const int e = (int)(max(top & 0xffffu, top >> 16) >> 7);          // the largest element's biased exponent
    const int ec = max(e, 8);                          // (rows below 2^-119 keep their order of size, not their last bits)
    const float mul = __uint_as_float((uint32_t)(261 - ec) << 23);    // 2^(134 - ec): the largest to [2^7, 2^8)
    const int per = (D / 16) / parts;                  // chunks of 16 elements, read again from L1
#pragma unroll 1
    for (int i = part * per; i < (part + 1) * per; ++i) {
        const uint4 a = __ldg(reinterpret_cast<const uint4 *>(q) + 2 * i), b = __ldg(reinterpret_cast<const uint4 *>(q) + 2 * i + 1);
        const uint32_t src[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float f[4] = {__uint_as_float(src[2 * j] << 16) * mul, __uint_as_float(src[2 * j] & 0xffff0000u) * mul,
                                __uint_as_float(src[2 * j + 1] << 16) * mul, __uint_as_float(src[2 * j + 1] & 0xffff0000u) * mul};
            hi[j] = e4m3x4(f[0], f[1], f[2], f[3]);
            const float4 h = from_e4m3x4(hi[j]);
            lo[j] = e4m3x4(f[0] - h.x, f[1] - h.y, f[2] - h.z, f[3] - h.w);
        }
        *reinterpret_cast<uint4 *>(tile + row_off<D>(r, i)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(tile + 128 * D + row_off<D>(r, i)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    return e == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)(ec - 7) << 23);
}

// Two pairs of weights in f16 as e5m2 codes: the first two terms are cut off, what they leave is exact, and the
// third is rounded.
__device__ __forceinline__ void three_terms(__half2 a, __half2 b, uint32_t &t1, uint32_t &t2, uint32_t &t3) {
    auto bits = [](const __half2 &x) { return *reinterpret_cast<const uint32_t *>(&x); };
    auto upper = [&](__half2 x) {
        const uint32_t u = bits(x) & 0xff00ff00u;
        return *reinterpret_cast<const __half2 *>(&u);
    };
    t1 = __byte_perm(bits(a), bits(b), 0x7531);
    a = __hsub2(a, upper(a));
    b = __hsub2(b, upper(b));
    t2 = __byte_perm(bits(a), bits(b), 0x7531);
    a = __hsub2(a, upper(a));
    b = __hsub2(b, upper(b));
    t3 = __byte_perm(bits(a) + 0x00800080u, bits(b) + 0x00800080u, 0x7531);
}

// A row's m: what is added to x; whether one of a part's weights may pass what it may be, by the largest x and the
// largest of the part's scales (or the row has no m yet); and the move to `top`, the largest of what the part's keys
// contribute, where one does.  Returns what the row's sums have to be multiplied by.
__device__ __forceinline__ float weight_unit(float log_w, float m) { return m == -INFINITY ? 0.f : log_w - m; }
__device__ __forceinline__ bool may_pass(float xmax, float neg_m, float log_top, float m) {
    return (m == -INFINITY && xmax > -INFINITY) || xmax + neg_m > fminf(kWeightTop - log_top, kSumTop) - 0.02f;   // (roundings aside)
}
__device__ __forceinline__ float move_unit(bool row_ok, float xmax, float top, float log_w, float &m) {
    if (!row_ok || !(top > m + (kWeightTop - log_w) || xmax > m + (kSumTop - log_w))) return 1.f;
    const float alpha = ex2(m - top);
    m = top;
    return alpha;
}

// kRows: what one unit holds.  kPairs: up to 256 rows.  kSmall: no sequence has more
// rows of a kv head than one tile holds, and the second row tile's room is ring
// slots.  kQuad: none has more than 32 (decoding).  Four copies of the rows then lie
// in the tile's four quarters, and the warp of a quarter sees to 32 of a tile's 128
// keys: its copies' weights of the others are zero, each copy has a maximum and a sum
// of its own, and the copies are joined as the streams are.  One warp of a stream
// would work through 128 keys otherwise, and three sleep.
// kTree: a row sees of its sequence's new tokens those that its mask says.
enum Rows8 { kPairs, kSmall8, kQuad8 };
template <int D, Rows8 kRows, bool kTree>
__global__ void __launch_bounds__(kThreads, 1)
attn_varlen_tc8_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                       const VarlenParams p, const int tpt, const int box) {
    using L = Lay8<D>;
    constexpr bool kSmall = kRows != kPairs, kQuad = kRows == kQuad8;
    constexpr int kSubs = kQuad ? 1 : 2;               // parts of a tile's keys that go around by themselves
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u32 = smem_u32(smem_raw);
    const uint32_t base = (raw_u32 + 1023u) & ~1023u;
    uint8_t *sbase = smem_raw + (base - raw_u32);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = (int)blockIdx.x;

    const uint32_t sQ = base + L::kOffQ, sRing = base + L::kOffRing - (kSmall ? 2 * L::kTile : 0), bar0 = base + L::kOffBar;
    constexpr int slots = kSmall ? L::kMaxSlots : L::kSlots;
    auto full_bar = [&](int i) { return bar0 + 8u * i; };
    auto empty_bar = [&](int i) { return bar0 + 8u * (L::kMaxSlots + i); };
    const uint32_t bar1 = bar0 + 8u * (2 * L::kMaxSlots);
    const uint32_t qfull_bar = bar1, drain_bar = bar1 + 8u;                  // Q written (8 warps); see the end
    auto sfull_bar = [&](int i, int h) { return bar1 + 8u * (2 + 2 * i + h); };   // part h of S_i computed
    auto pfull_bar = [&](int i, int h) { return bar1 + 8u * (6 + 2 * i + h); };   // part h of W_i written (4 warps)
    auto ofull_bar = [&](int i) { return bar1 + 8u * (10 + i); };            // O_i complete for the unit
    auto ofree_bar = [&](int i) { return bar1 + 8u * (12 + i); };            // O_i read out (4 warps)
    auto oadd_bar = [&](int i) { return bar1 + 8u * (14 + i); };             // one more part added to O_i
    auto scfull_bar = [&](int i) { return bar1 + 8u * (16 + i); };           // scales written
    auto scempty_bar = [&](int i) { return bar1 + 8u * (16 + kScaleSlots + i); };   // and read (8 warps, or 4 twice)
    auto ufull_bar = [&](int i) { return bar1 + 8u * (16 + 2 * kScaleSlots + i); };
    auto uempty_bar = [&](int i) { return bar1 + 8u * (16 + 2 * kScaleSlots + kUnitSlots + i); };
    Unit8 *units = reinterpret_cast<Unit8 *>(sbase + L::kOffUnits);
    // The next unit, false behind the last.  Every warp goes through all of them, whatever it gave up:
    // these waits end because the others' do.
    int uslot = 0;
    uint32_t uphase = 0;
    auto next_unit = [&]() { return wait_bar(ufull_bar(uslot), uphase, nullptr, p.fault) && units[uslot].more != 0; };
    auto done_unit = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(uempty_bar(uslot));
        if (++uslot == kUnitSlots) { uslot = 0; uphase ^= 1u; }
    };
    Scales *scales = reinterpret_cast<Scales *>(sbase + L::kOffScale);
    float *xrow = reinterpret_cast<float *>(sbase + L::kOffMl);      // [2][128]: one value per stream and row
    Misc *misc = reinterpret_cast<Misc *>(sbase + L::kOffMisc);
    volatile int *abort_flag = &misc->abort_flag;

    if (tid == 0) {
        for (int i = 0; i < L::kMaxSlots; ++i) { mbar_init(full_bar(i), 1); mbar_init(empty_bar(i), 1); }
        mbar_init(qfull_bar, 8);
        for (int i = 0; i < kUnitSlots; ++i) { mbar_init(ufull_bar(i), 1); mbar_init(uempty_bar(i), kUnitReaders); }
        for (int i = 0; i < kScaleSlots; ++i) { mbar_init(scfull_bar(i), 1); mbar_init(scempty_bar(i), 8); }
        for (int i = 0; i < 2; ++i) {
            for (int h = 0; h < 2; ++h) { mbar_init(sfull_bar(i, h), 1); mbar_init(pfull_bar(i, h), 4); }
            mbar_init(oadd_bar(i), 1);
            mbar_init(ofull_bar(i), 1);
            mbar_init(ofree_bar(i), 4);
        }
        misc->abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_k)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_v)) : "memory");
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&misc->tmem)), "r"(512u) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (warp == 0) {
        const VlPlan q = vl_plan(p, cta);
        vl_plan_store(q, &misc->plan);
        // the producer goes straight on to its copies (it set up the barriers itself); the others wait for the plan
        asm volatile("bar.arrive 15, %0;" ::"n"(kThreads) : "memory");
    } else {
        tc_fence_before();
        named_sync(15, kThreads);
        tc_fence_after();
    }
    const uint32_t tmem = warp == 0 ? 0u : misc->tmem;
    const VlPlan &pl = misc->plan;
    const int G = p.Hq / p.Hkv;

    if (!pl.idle) {
        if (warp < 4) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
            if (warp == 0) {
                // ---------------------------------------------------------- TMA producer
                // the whole warp: the lanes share a tile's page look-ups and copies
                RingPos rp;
                long loads = 0;
                bool ok = true;
                // K and V that one unit alone reads leave L2 first; what several units read stays as usual
                uint64_t once, again;
                asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
                asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(again));
                const int copies = 128 / box;          // of a tile
                while (next_unit()) {
                    const VlUnit u = units[uslot].u;
                    const uint64_t policy = units[uslot].alone ? once : again;
                    done_unit();
                    const int n = u.t1 - u.t0;
                    if (n <= 0 || !ok) continue;
                    const int la = kSmall || u.ntok <= tpt ? 2 : 1;
                    const int32_t *trow = p.table + (long)u.b * p.table_stride;
                    // the lane's page of tile t: looked up a tile ahead, first used (and checked) by its copy
                    auto page_of = [&](int t) {
                        const int key = t * 128 + (lane % copies) * box;
                        return key < u.kv ? __ldg(trow + (p.page_log2 >= 0 ? key >> p.page_log2 : key / p.page_size)) : -1;
                    };
                    auto load_tile = [&](bool is_v, int t, int pg) {
                        if (ok && loads >= slots)
                            ok = wait_bar(empty_bar(rp.slot), rp.phase ^ 1u, abort_flag, p.fault);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) return;
                        const uint32_t dst = sRing + rp.slot * L::kTile, bar = full_bar(rp.slot);
                        const int boxes = min(copies, (u.kv - t * 128 + box - 1) / box);
                        if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(boxes * box * D));
                        __syncwarp();
                        if (lane < boxes) {
                            const int key = t * 128 + lane * box;
                            if (pg < 0 || pg >= p.n_pages) {      // read as zeros: the copy's fill
                                set_fault(p.fault, FAULT_BAD_PAGE);
                                pg = p.n_pages;
                            }
                            load_page(dst + lane * box * D, is_v ? &tmap_v : &tmap_k, bar, policy,
                                      p.page_log2 >= 0 ? key & (p.page_size - 1) : key % p.page_size, u.g, pg);
                        }
                        rp.step(slots);
                        ++loads;
                    };
                    int pk = page_of(u.t0), pv = pk;      // pages of the next K tile, of the V tile behind it
                    int pk2 = 0;
                    load_tile(false, u.t0, pk);
                    if (n > 1) pk = page_of(u.t0 + 1);
                    // V of tile j and K of tile j + la, in the order of use
                    if (la == 2 && n > 1) {
                        load_tile(false, u.t0 + 1, pk);
                        pk2 = pk;
                        if (n > 2) pk = page_of(u.t0 + 2);
                    }
                    for (int j = 0; ok && j < n; ++j) {
                        load_tile(true, u.t0 + j, pv);
                        if (la == 2) {
                            pv = pk2;
                            if (j + 2 < n) {
                                load_tile(false, u.t0 + j + 2, pk);
                                pk2 = pk;
                                if (j + 3 < n) pk = page_of(u.t0 + j + 3);
                            }
                        } else if (j + 1 < n) {
                            load_tile(false, u.t0 + j + 1, pk);
                            pv = pk;
                            if (j + 2 < n) pk = page_of(u.t0 + j + 2);
                        }
                    }
                }
                // the copies still in flight land before the CTA's shared memory goes
                if (*abort_flag) {
                    const int m = (int)min(loads, (long)slots);
                    RingPos a = rp;
                    for (int i = 0; i < m; ++i) {
                        if (a.slot == 0) { a.slot = slots - 1; a.phase ^= 1u; } else --a.slot;
                        wait_bar(full_bar(a.slot), a.phase, nullptr, p.fault);
                    }
                }
            } else if (warp == 1) {
                // ---------------------------------------------------------- MMA issuer
                // the whole warp runs the loop and one elected lane issues: the descriptors are then the
                // same in every lane for the compiler too and stay in uniform registers (issued from inside
                // a one-lane branch, the products took twice as long: 4.49 ms against 3.10 for the
                // 25,119-token prompt)
                {
                    const bool el = elect_one();
                    RingPos rp;
                    uint32_t qphase = 0, pphase = 0, fphase = 0, used = 0;        // (bit i: of stream i)
                    bool ok = true;
                    const uint32_t idS = idesc_8(128, 128 / kSubs, false, false), idO = idesc_8(128, D, true, true);
                    // the next tile of the ring: its slot
                    auto take = [&]() {
                        ok = ok && wait_bar(full_bar(rp.slot), rp.phase, abort_flag, p.fault);
                        tc_fence_after();
                        const int slot = rp.slot;
                        rp.step(slots);
                        return slot;
                    };
                    // descriptors by their first tile's, moved on by whole 16-byte units: rows of D bytes, 8-row
                    // groups 8 D bytes apart whatever the copies' size; the products take 32 of their columns
                    // (Q, K) or 32 of their rows (V) at a time
                    const uint64_t qd0 = row_desc<D>(sQ), kd0 = row_desc<D>(sRing);
                    // part h of S_i from row tile qt and the K tile in `slot`
                    auto issue_s = [&](int i, int qt, int slot, int h) {
                        const uint64_t qd = qd0 + (uint64_t)(qt * (2 * L::kTile / 16)),
                                       kd = kd0 + (uint64_t)(slot * (L::kTile / 16) + h * (64 * D / 16));
                        if (el) {
#pragma unroll
                            for (int term = 0; term < 2; ++term)
#pragma unroll
                                for (int kk = 0; kk < D / 32; ++kk)
                                    umma8_ss(tmem + 128u * i + 64u * h, qd + term * (L::kTile / 16) + 2 * kk, kd + 2 * kk, idS,
                                             term + kk > 0 ? 1u : 0u);
                            umma_commit(sfull_bar(i, h));
                        }
                    };
                    // W_i V for part h of the V tile in `slot`
                    auto issue_pv = [&](int i, int slot, bool first, int steps, int h) {
                        const uint64_t vd = kd0 + (uint64_t)(slot * (L::kTile / 16) + h * (64 * D / 16));
                        ok = ok && wait_bar(pfull_bar(i, h), pphase >> i & 1u, abort_flag, p.fault);
                        if (!ok) return;
                        tc_fence_after();
                        if (el) {
#pragma unroll
                            for (int kk = 0; kk < 4 / kSubs; ++kk) {
                                if (kSmall && kk + 2 * h >= steps) continue;
#pragma unroll
                                for (int term = 0; term < 3; ++term)
                                    umma8_ts(tmem + 256u + 128u * i, tmem + 128u * i + 64u * h + 32u / kSubs * term + 8u * kk,
                                             vd + kk * (32 * D / 16), idO, (!first || kk + term > 0) ? 1u : 0u);
                            }
                            if (kSubs > 1) umma_commit(oadd_bar(i));
                        }
                        if (h == kSubs - 1) pphase ^= 1u << i;
                    };
                    // O_i free for a new unit
                    auto claim = [&](int i) {
                        if (used >> i & 1u) {
                            ok = ok && wait_bar(ofree_bar(i), fphase >> i & 1u, abort_flag, p.fault);
                            tc_fence_after();
                            fphase ^= 1u << i;
                        }
                        used |= 1u << i;
                    };
                    while (next_unit()) {
                        const VlUnit u = units[uslot].u;
                        done_unit();
                        const int n = u.t1 - u.t0;
                        if (n <= 0 || !ok) continue;
                        const bool pair = !kSmall && u.ntok > tpt;
                        // the small form's second products stop at the step of 32 that holds the last key
                        auto steps = [&](int j) { return kSmall ? (u.kv - (u.t0 + j) * 128 + 31) >> 5 : 4; };
                        ok = wait_bar(qfull_bar, qphase, abort_flag, p.fault);
                        qphase ^= 1u;
                        if constexpr (kQuad) {         // (88 us for 64 sequences of one token; the loops below with one part 95)
                            int k = take();
                            if (!ok) continue;
                            issue_s(0, 0, k, 0);
                            if (el) umma_commit(empty_bar(k));
                            if (n > 1) {
                                k = take();
                                if (!ok) continue;
                                issue_s(1, 0, k, 0);
                                if (el) umma_commit(empty_bar(k));
                            }
                            for (int j = 0; ok && j < n; ++j) {
                                const int i = j & 1, v = take();
                                if (!ok) break;
                                if (j < 2) claim(i);
                                issue_pv(i, v, j < 2, steps(j), 0);
                                if (!ok) break;
                                if (el) umma_commit(empty_bar(v));
                                if (j + 2 < n) {
                                    k = take();
                                    if (!ok) break;
                                    issue_s(i, 0, k, 0);
                                    if (el) umma_commit(empty_bar(k));
                                } else {
                                    if (el) umma_commit(ofull_bar(i));
                                }
                            }
                            continue;
                        }
                        // Both parts of the first tiles' scores; then, as each part's weights come, their product and
                        // the same part of the stream's next tile: a stream's other part is with its softmax meanwhile.
                        int kt[2], vt[2] = {0, 0};
                        kt[0] = kt[1] = take();
                        if (!ok) continue;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            issue_s(0, 0, kt[0], h);
                            if (pair) issue_s(1, 1, kt[0], h);
                        }
                        if (el) umma_commit(empty_bar(kt[0]));
                        if (!pair && n > 1) {
                            kt[1] = take();
                            if (!ok) continue;
#pragma unroll
                            for (int h = 0; h < 2; ++h) issue_s(1, 0, kt[1], h);
                            if (el) umma_commit(empty_bar(kt[1]));
                        }
                        const int step = pair ? 1 : 2;
                        for (int jj = 0; ok && jj < n; jj += step) {
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                // (both unrolled, this warp's registers are too few for it: 2.80 ms against 2.47)
#pragma unroll 1
                                for (int i = 0; i < 2; ++i) {
                                    const int j = pair ? jj : jj + i;
                                    if (!ok || j >= n) continue;
                                    const bool odd = !pair && i;
                                    const bool fetch = h == 0 && (!pair || i == 0), last = h == 1 && (!pair || i == 1);
                                    if (fetch) {
                                        const int t = take();
                                        if (odd) vt[1] = t;
                                        else vt[0] = t;
                                    }
                                    const int v = odd ? vt[1] : vt[0];
                                    if (jj == 0 && h == 0) claim(i);
                                    issue_pv(i, v, jj == 0 && h == 0, steps(j), h);
                                    if (!ok) continue;
                                    if (last && el) umma_commit(empty_bar(v));
                                    if (j + step < n) {
                                        if (fetch) {
                                            const int t = take();
                                            if (odd) kt[1] = t;
                                            else kt[0] = t;
                                        }
                                        if (!ok) continue;
                                        const int k = odd ? kt[1] : kt[0];
                                        issue_s(i, pair ? i : 0, k, h);
                                        if (last && el) umma_commit(empty_bar(k));
                                    } else if (h == 1) {
                                        if (el) umma_commit(ofull_bar(i));
                                    }
                                }
                        }
                    }
                }
                __syncwarp();
            } else if (warp == 2) {
                // ---------------------------------------------------------- scales
                // a tile's scales: four keys a lane, pages looked up two tiles ahead and scales read one ahead
                unsigned done = 0;
                bool ok = true;
                while (next_unit()) {
                    const VlUnit u = units[uslot].u;
                    done_unit();
                    const int n = u.t1 - u.t0;
                    if (n <= 0 || !ok) continue;
                    const int32_t *trow = p.table + (long)u.b * p.table_stride;
                    auto page_of = [&](int j) {
                        const int key = (u.t0 + j) * 128 + 4 * lane;
                        return j < n && key < u.kv ? __ldg(trow + (p.page_log2 >= 0 ? key >> p.page_log2 : key / p.page_size)) : -1;
                    };
                    float4 ks, vs;
                    auto fetch = [&](int j, int pg) {
                        ks = vs = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (pg >= 0 && pg < p.n_pages) {
                            const int key = (u.t0 + j) * 128 + 4 * lane;
                            const int in = p.page_log2 >= 0 ? key & (p.page_size - 1) : key % p.page_size;
                            const long at = ((long)pg * p.Hkv + u.g) * p.page_size + in;
                            ks = __ldg(reinterpret_cast<const float4 *>(p.k_scale + at));
                            vs = __ldg(reinterpret_cast<const float4 *>(p.v_scale + at));
                        }
                    };
                    int pg = page_of(1);
                    fetch(0, page_of(0));
                    for (int j = 0; j < n; ++j, ++done) {
                        float4 k4 = ks, v4 = vs;
                        if (j + 1 < n) fetch(j + 1, pg);
                        pg = page_of(j + 2);
                        const int left = u.kv - (u.t0 + j) * 128 - 4 * lane;       // keys of the lane inside the sequence
                        if (left < 4) {
                            k4.w = v4.w = 0.f;
                            if (left < 3) k4.z = v4.z = 0.f;
                            if (left < 2) k4.y = v4.y = 0.f;
                            if (left < 1) k4.x = v4.x = 0.f;
                        }
                        const float4 lv = make_float4(log_scale(v4.x), log_scale(v4.y), log_scale(v4.z), log_scale(v4.w));
                        float top = fmaxf(max3(lv.x, lv.y, lv.z), lv.w), low = fminf(fminf(lv.x, lv.y), fminf(lv.z, lv.w));
#pragma unroll
                        for (int o = 4; o; o >>= 1) {
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                            low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
                        }
                        const unsigned slot = done % kScaleSlots;
                        if (done >= kScaleSlots)
                            ok = wait_bar(scempty_bar(slot), (done / kScaleSlots - 1) & 1u, abort_flag, p.fault);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        Scales &to = scales[slot];
                        reinterpret_cast<float4 *>(to.k)[lane] = k4;
                        reinterpret_cast<float4 *>(to.v)[lane] = v4;
                        reinterpret_cast<float4 *>(to.log_v)[lane] = lv;
                        if ((lane & 7) == 0) to.range[lane >> 3] = make_float2(top, low);
                        __syncwarp();
                        if (lane == 0) mbar_arrive(scfull_bar(slot));
                    }
                }
            } else if (warp == 3) {
                VlWalk walk(pl);
                bool more = true;
                for (int i = 0; more; ++i) {
                    if (i == kUnitSlots) {         // (the first units go out first)
                        vl_ends(p, pl, cta, &misc->ends);
                        asm volatile("bar.arrive 14, 288;" ::: "memory");
                    }
                    VlUnit u;
                    more = walk.next(p, pl, u);
                    if (i >= kUnitSlots) wait_bar(uempty_bar(uslot), uphase ^ 1u, nullptr, p.fault);
                    Unit8 &to = units[uslot];
                    if (lane == 0) {
                        to.u = u;
                        to.more = more;
                        to.alone = walk.s.nr == 1;
                        mbar_arrive(ufull_bar(uslot));
                    }
                    __syncwarp();
                    if (++uslot == kUnitSlots) { uslot = 0; uphase ^= 1u; }
                    if (!more && i < kUnitSlots) {
                        vl_ends(p, pl, cta, &misc->ends);
                        asm volatile("bar.arrive 14, 288;" ::: "memory");
                    }
                }
            }
        } else {
            // -------------------------------------------------------------- softmax
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
            const int w = (warp - 4) >> 2;             // stream
            const int r = (tid - 128) & 127;           // row of the tile = tensor-memory lane
            const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t s_col = tmem + lane_off + 128u * w, o_col = tmem + lane_off + 256u + 128u * w;
            const int quarter = warp & 3;
            const int ur = kQuad ? lane : r;           // row of the unit's tile
            const int tr = ur / G;                     // and its token
            // u: one more for every doubling of what a sequence may hold past 2^16
            const float log_w = fminf(kWeightLogMost, kWeightLog + (float)max(0, 16 - __clz(p.max_kv - 1)));
            uint32_t sphase = 0, ophase0 = 0, ophase1 = 0;
            bool have_ends = false;
            unsigned ring = 0;                         // tiles that went through the ring before this unit
            unsigned before = 0;                       // and key tiles
            uint32_t added = 0;                        // parts added to this stream's accumulator, announced by oadd
            bool was_pair = false;
            bool ok = true;
            while (next_unit()) {
                const VlUnit &u = units[uslot].u;
                const int n = u.t1 - u.t0;
                const bool pair = !kSmall && u.ntok > tpt;
                const int tl = tr + (pair && w ? tpt : 0);             // token within the unit
                const bool row_ok = tr < tpt && tl < u.ntok;
                const int lim = row_ok ? vl_limit(p, u, u.tok0 + tl) : 0;
                const uint64_t word = kTree && row_ok ? vl_tree_word(p, u, tl) : 0;
                // rows this warp has to do anything for
                const bool warp_live = __any_sync(0xffffffffu, row_ok);
                float m_used = -INFINITY, l = 0.f, qk = 0.f;
                // Q in two e4m3 terms.  The tile's last readers are done: a stream's own products have been
                // waited for, and where both write one tile behind a pair of them, they meet first.
                if (!pair && was_pair) named_sync(2, 256);
                was_pair = pair;
                if (n > 0) {
                    if (row_ok)
                        qk = put_query<D>(static_cast<const __nv_bfloat16 *>(p.q) + (long)(u.row0 + tl) * p.q_tok +
                                              (long)(u.g * G + (ur - tr * G)) * p.q_head,
                                          sbase + (sQ - base) + (pair && w ? 2 * L::kTile : 0), r, pair ? 0 : w, pair ? 1 : 2) *
                             (p.scale * kLog2e);
                    qk = qk < 0x1p-126f ? 0x1p-126f : qk;       // (NaN, a row that is not finite, stays)
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(qfull_bar);
                }
                const int step = pair ? 1 : 2, la = pair ? 1 : 2;
                const int j0 = pair ? 0 : w;
                for (int j = j0; j < n; j += step) {
                    const int key0 = (u.t0 + j) * 128;
                    ok = __all_sync(0xffffffffu, wait_bar(sfull_bar(w, 0), sphase, abort_flag, p.fault)) && ok;
                    tc_fence_after();
                    if (key0 + 128 > u.kv && (!pair || w == 0)) {
                        // slots past the sequence may hold anything, and 0 times that is not 0:
                        // one stream, all its warps, clears those rows of the last V tile that its
                        // product reads before that begins
                        const int nk = min(la, n);
                        const unsigned idx = ring + nk + j + min(j, n - nk);
                        const int slot = (int)(idx % (unsigned)slots);
                        ok = __all_sync(0xffffffffu, wait_bar(full_bar(slot), (idx / (unsigned)slots) & 1u,
                                                               abort_flag, p.fault)) && ok;
                        uint8_t *vt = sbase + (sRing - base) + slot * L::kTile;
                        const int v0 = u.kv - key0, v1 = kSmall ? (v0 + 31) & ~31 : 128;
                        for (int i = v0 * (D / 16) + r; i < v1 * (D / 16); i += 128)       // whole rows, in any order
                            reinterpret_cast<uint4 *>(vt)[i] = make_uint4(0u, 0u, 0u, 0u);
                        fence_proxy_async_smem();
                        // every warp's rows, before any arrival lets the product start
                        named_sync(3 + w, 128);
                    }
                    const unsigned tile = before + j, sc = tile % kScaleSlots;
                    ok = __all_sync(0xffffffffu, wait_bar(scfull_bar(sc), (tile / kScaleSlots) & 1u, abort_flag, p.fault)) && ok;
                    const Scales &ts = scales[sc];
                    if constexpr (kQuad) {
                        uint32_t s[32];
                        tmem_ld32_async(s_col + 32u * quarter, s);
                        tmem_ld_wait();
                        tmem_ld_bind(s);
                        const int from = key0 + 32 * quarter;
                        uint32_t seen = 0xffffffffu;
                        if constexpr (kTree) {
                            seen = (uint32_t)tree_seen(word, from - u.off);
                        } else {
                            const int vis = lim - from;
                            if (vis < 32) seen = vis <= 0 ? 0u : (1u << vis) - 1u;
                        }
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float4 f = reinterpret_cast<const float4 *>(ts.k)[8 * quarter + e / 4];
                            s[e] = __float_as_uint(__uint_as_float(s[e]) * f.x);
                            s[e + 1] = __float_as_uint(__uint_as_float(s[e + 1]) * f.y);
                            s[e + 2] = __float_as_uint(__uint_as_float(s[e + 2]) * f.z);
                            s[e + 3] = __float_as_uint(__uint_as_float(s[e + 3]) * f.w);
                        }
                        const bool edge = !__all_sync(0xffffffffu, seen == 0xffffffffu || !row_ok);
                        if (edge) {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!(seen >> e & 1)) s[e] = 0xff800000u;
                        }
                        float m = max3(__uint_as_float(s[0]), __uint_as_float(s[1]), __uint_as_float(s[2]));
                        float m2 = fmaxf(__uint_as_float(s[3]), __uint_as_float(s[31]));
#pragma unroll
                        for (int e = 4; e < 16; e += 2) m = max3(m, __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
#pragma unroll
                        for (int e = 16; e < 30; e += 2) m2 = max3(m2, __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
                        const float xmax = qk * max3(m, m2, __uint_as_float(s[30]));
                        float neg_m = weight_unit(log_w, m_used);
                        const float2 range = ts.range[quarter];
                        if (__any_sync(0xffffffffu, row_ok && may_pass(xmax, neg_m, range.x, m_used))) {
                            float top = xmax + range.x;
                            if (edge || range.x > range.y + kAlike) {
                                float t[2] = {-INFINITY, -INFINITY};
#pragma unroll
                                for (int g = 0; g < 8; ++g) {
                                    const float4 f = reinterpret_cast<const float4 *>(ts.log_v)[8 * quarter + g];
                                    t[0] = max3(t[0], fmaf(__uint_as_float(s[4 * g]), qk, f.x), fmaf(__uint_as_float(s[4 * g + 1]), qk, f.y));
                                    t[1] = max3(t[1], fmaf(__uint_as_float(s[4 * g + 2]), qk, f.z), fmaf(__uint_as_float(s[4 * g + 3]), qk, f.w));
                                }
                                top = fmaxf(t[0], t[1]);
                            }
                            const float alpha = move_unit(row_ok, xmax, top, log_w, m_used);
                            neg_m = weight_unit(log_w, m_used);
                            l *= alpha;
                            if (j > j0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                                uint32_t o[D / 32][32];
#pragma unroll
                                for (int c = 0; c < D / 32; ++c) tmem_ld32_async(o_col + 32u * c, o[c]);
                                tmem_ld_wait();
#pragma unroll
                                for (int c = 0; c < D / 32; ++c) {
                                    tmem_ld_bind(o[c]);
#pragma unroll
                                    for (int e = 0; e < 32; ++e) o[c][e] = __float_as_uint(__uint_as_float(o[c][e]) * alpha);
                                    tmem_st32(o_col + 32u * c, o[c]);
                                }
                            }
                        }
                        float ls[2] = {0.f, 0.f};
                        uint32_t t1[8], t2[8], t3[8];
                        const uint32_t none[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
                        for (int c = 0; c < 4; ++c)
                            if (c != quarter) {
                                tmem_st8(s_col + 8u * c, none);
                                tmem_st8(s_col + 32u + 8u * c, none);
                                tmem_st8(s_col + 64u + 8u * c, none);
                            }
#pragma unroll
                        for (int g = 0; g < 8; ++g) {
                            const float4 f = reinterpret_cast<const float4 *>(ts.v)[8 * quarter + g];
                            float x[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) x[e] = ex2(fmaf(__uint_as_float(s[4 * g + e]), qk, neg_m));
                            ls[0] += x[0] + x[2];
                            ls[1] += x[1] + x[3];
                            const __half2 v0 = __floats2half2_rn(x[0] * f.x, x[1] * f.y), v1 = __floats2half2_rn(x[2] * f.z, x[3] * f.w);
                            three_terms(v0, v1, t1[g], t2[g], t3[g]);
                        }
                        tmem_st8(s_col + 8u * quarter, t1);
                        tmem_st8(s_col + 32u + 8u * quarter, t2);
                        tmem_st8(s_col + 64u + 8u * quarter, t3);
                        l += ls[0] + ls[1];
                        tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(pfull_bar(w, 0));
                            mbar_arrive_n(scempty_bar(sc), 2);
                        }
                    } else {
                        // 64 keys at a time
#pragma unroll 1
                        for (int h = 0; h < 2; ++h, ++added) {
                            if (h) {
                                ok = __all_sync(0xffffffffu, wait_bar(sfull_bar(w, 1), sphase, abort_flag, p.fault)) && ok;
                                tc_fence_after();
                            }
                            if (warp_live) {
                                const uint32_t at = s_col + 64u * h;
                                uint32_t s[2][32];
#pragma unroll
                                for (int c = 0; c < 2; ++c) tmem_ld32_async(at + 32u * c, s[c]);
                                tmem_ld_wait();
#pragma unroll
                                for (int c = 0; c < 2; ++c) tmem_ld_bind(s[c]);
                                // the keys' scales
                                const float4 *ks = reinterpret_cast<const float4 *>(ts.k) + 16 * h, *vs = reinterpret_cast<const float4 *>(ts.v) + 16 * h;
#pragma unroll
                                for (int c = 0; c < 2; ++c)
#pragma unroll
                                    for (int e = 0; e < 32; e += 4) {
                                        const float4 f = ks[8 * c + e / 4];
                                        const float2 x = __fmul2_rn(make_float2(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])),
                                                                    make_float2(f.x, f.y));
                                        const float2 y = __fmul2_rn(make_float2(__uint_as_float(s[c][e + 2]), __uint_as_float(s[c][e + 3])),
                                                                    make_float2(f.z, f.w));
                                        s[c][e] = __float_as_uint(x.x); s[c][e + 1] = __float_as_uint(x.y);
                                        s[c][e + 2] = __float_as_uint(y.x); s[c][e + 3] = __float_as_uint(y.y);
                                    }
                                const int from = key0 + 64 * h;
                                uint64_t seen = ~0ull;
                                if constexpr (kTree) {                  // nodes among the keys, or what lies behind them
                                    seen = tree_seen(word, from - u.off);
                                } else {
                                    const int vis = lim - from;         // this row sees the first `vis` of the keys
                                    if (vis < 64) seen = vis <= 0 ? 0ull : (1ull << vis) - 1;
                                }
                                const bool edge = !__all_sync(0xffffffffu, seen == ~0ull || !row_ok);
                                if (edge) {
#pragma unroll
                                    for (int c = 0; c < 2; ++c)
#pragma unroll
                                        for (int e = 0; e < 32; ++e)
                                            if (!(seen >> (32 * c + e) & 1)) s[c][e] = 0xff800000u;
                                }
                                float m4[4];
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const uint32_t *x = s[i >> 1] + 16 * (i & 1);
                                    float m = max3(__uint_as_float(x[0]), __uint_as_float(x[1]), __uint_as_float(x[2]));
#pragma unroll
                                    for (int e = 3; e < 15; e += 2) m = max3(m, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                                    m4[i] = fmaxf(m, __uint_as_float(x[15]));
                                }
                                const float xmax = qk * fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]);
                                float neg_m = weight_unit(log_w, m_used);
                                const float4 range = reinterpret_cast<const float4 *>(ts.range)[h];
                                const float log_top = fmaxf(range.x, range.z);
                                if (__any_sync(0xffffffffu, row_ok && may_pass(xmax, neg_m, log_top, m_used))) {
                                    float top = xmax + log_top;
                                    if (edge || log_top > fminf(range.y, range.w) + kAlike) {
                                        const float4 *lv = reinterpret_cast<const float4 *>(ts.log_v) + 16 * h;
                                        float t[2] = {-INFINITY, -INFINITY};
#pragma unroll
                                        for (int g = 0; g < 16; ++g) {
                                            const uint32_t *x = s[g >> 3] + 4 * (g & 7);
                                            const float4 y = lv[g];
                                            t[0] = max3(t[0], fmaf(__uint_as_float(x[0]), qk, y.x), fmaf(__uint_as_float(x[1]), qk, y.y));
                                            t[1] = max3(t[1], fmaf(__uint_as_float(x[2]), qk, y.z), fmaf(__uint_as_float(x[3]), qk, y.w));
                                        }
                                        top = fmaxf(t[0], t[1]);
                                    }
                                    const float alpha = move_unit(row_ok, xmax, top, log_w, m_used);
                                    neg_m = weight_unit(log_w, m_used);
                                    l *= alpha;
                                    if ((j > j0 || h) && __any_sync(0xffffffffu, alpha != 1.f)) {
                                        // the part before this one has to be in O: the others are, their products went
                                        // out before this part's scores and complete in order
                                        ok = __all_sync(0xffffffffu, wait_bar(oadd_bar(w), (added - 1) & 1u, abort_flag, p.fault)) && ok;
                                        tc_fence_after();
#pragma unroll 1
                                        for (int c = 0; c < D / 32; ++c) {
                                            uint32_t o[32];
                                            tmem_ld32_async(o_col + 32u * c, o);
                                            tmem_ld_wait();
                                            tmem_ld_bind(o);
#pragma unroll
                                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                                            tmem_st32(o_col + 32u * c, o);
                                        }
                                    }
                                }
                                const float2 qk2 = make_float2(qk, qk), nm2 = make_float2(neg_m, neg_m);
                                float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                                // the weights go over scores that have been read: the first terms in the part's
                                // columns 0-15, the second in 16-31, the third in 32-47
                                uint32_t t1[16], t2[16], t3[16];
#pragma unroll
                                for (int g = 0; g < 16; ++g) {
                                    const uint32_t *x = s[g >> 3] + 4 * (g & 7);
                                    const float4 y = vs[g];
                                    const float2 x0 = __ffma2_rn(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])), qk2, nm2);
                                    const float2 x1 = __ffma2_rn(make_float2(__uint_as_float(x[2]), __uint_as_float(x[3])), qk2, nm2);
                                    const float2 p0 = make_float2(ex2(x0.x), ex2(x0.y)), p1 = make_float2(ex2(x1.x), ex2(x1.y));
                                    ls[0] = __fadd2_rn(ls[0], p0);
                                    ls[1] = __fadd2_rn(ls[1], p1);
                                    const float2 w0 = __fmul2_rn(p0, make_float2(y.x, y.y)), w1 = __fmul2_rn(p1, make_float2(y.z, y.w));
                                    three_terms(__floats2half2_rn(w0.x, w0.y), __floats2half2_rn(w1.x, w1.y), t1[g], t2[g], t3[g]);
                                }
                                tmem_st16(at, t1);
                                tmem_st16(at + 16u, t2);
                                tmem_st16(at + 32u, t3);
                                l += (ls[0].x + ls[1].x) + (ls[0].y + ls[1].y);
                                tmem_st_wait();
                            }
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) {
                                mbar_arrive(pfull_bar(w, h));
                                if (h) mbar_arrive_n(scempty_bar(sc), pair ? 1 : 2);
                            }
                        }
                    }
                    sphase ^= 1u;
                }
                // ---- end of the unit: this CTA's rows, normalised, or its part of them
                const bool whole = u.t0 == 0 && u.t1 == u.tiles;
                const bool had0 = n > 0, had1 = pair ? n > 0 : n > 1;     // streams that hold anything
                // A unit of two CTAs: the one that opens it has it last and keeps its part in tensor
                // memory; the other had it first and left its part in the workspace long ago.  So one
                // part is written and read instead of two (a batch of prompts shares about two units
                // per CTA: 256 KB each way).  Units of more CTAs are joined at the end, by all of them.
                const VlShared *sh = nullptr;
                if (!whole) {
                    if (!have_ends) asm volatile("bar.sync 14, 288;" ::: "memory");      // warp 3's answer
                    have_ends = true;
                    sh = misc->ends.u + (u.t0 > 0 ? 0 : misc->ends.n - 1);
                }
                const bool two = sh && sh->n == 2, keeper = two && u.t0 == 0;
                const long slot = keeper ? 2L * sh->last : u.t0 == 0 ? 2L * cta + 1 : 2L * cta;
                unsigned ticket = 0;
                if (keeper) {
                    if (tid == 128) {
                        const bool got = vl_wait(p.ctr + sh->first, 1u + p.wt.extra, p.wt.limit_ns);
                        if (!got) set_fault(p.fault, FAULT_WAIT_TIMEOUT);
                        misc->join_flag = got;
                        ticket = atomicAdd(p.ctr + sh->first, 1u);
                    }
                    named_sync(1, 256);
                    if (tid == 128 && ticket == 1u) atomicExch(p.ctr + sh->first, 0u);
                }
                ring += 2 * max(n, 0);
                before += max(n, 0);
                float a0 = 1.f, a1 = 0.f;
                if (!pair) {
                    // join the two streams of the one row tile: they exchange the row's maximum, then
                    // its sum, and each takes half of the columns of both accumulators
                    xrow[128 * w + r] = m_used;
                    named_sync(1, 256);
                    const float mo = xrow[128 * (w ^ 1) + r];
                    float m = fmaxf(m_used, mo);
                    if (kQuad) {                       // and of the other copies
#pragma unroll
                        for (int c = 0; c < 8; ++c) m = fmaxf(m, xrow[32 * c + lane]);
                    }
                    const float ref = m == -INFINITY ? 0.f : m;
                    const float own = ex2(m_used - ref), other = ex2(mo - ref);
                    l *= own;
                    m_used = m;
                    a0 = w == 0 ? own : other;
                    a1 = w == 0 ? other : own;
                    named_sync(2, 256);
                    xrow[128 * w + r] = l;
                    named_sync(1, 256);
                    if (kQuad) {
                        l = 0.f;
#pragma unroll
                        for (int c = 0; c < 8; ++c) l += xrow[32 * c + lane];
                    } else {
                        l += xrow[128 * (w ^ 1) + r];
                    }
                }
                // each warpgroup follows both barriers' phases; past the exchange above neither can be a unit behind
                if (pair ? n > 0 && w == 0 : had0)
                    ok = __all_sync(0xffffffffu, wait_bar(ofull_bar(0), ophase0, abort_flag, p.fault)) && ok;
                if (pair ? n > 0 && w == 1 : had1)
                    ok = __all_sync(0xffffffffu, wait_bar(ofull_bar(1), ophase1, abort_flag, p.fault)) && ok;
                if (had0) ophase0 ^= 1u;
                if (had1) ophase1 ^= 1u;
                tc_fence_after();
                if (warp_live) {
                    const int c0 = pair ? 0 : w * (D / 64), c1 = pair ? D / 32 : c0 + D / 64;
                    const uint32_t o0 = tmem + lane_off + 256u + (pair ? 128u * w : 0u);
                    const long prow = 128 * (pair ? w : 0) + ur;
                    const long orow = (long)(u.row0 + tl) * p.Hq + u.g * G + (ur - tr * G);
                    const bool dead = n <= 0;
                    float a2 = 0.f;                    // weight of the other CTA's part
                    if (keeper && row_ok) {
                        const float2 other = __ldcg(p.ml_part + slot * kVarlenTcRows + prow);
                        const float m = fmaxf(m_used, other.x), ref = m == -INFINITY ? 0.f : m;
                        const float f = ex2(m_used - ref);
                        a0 *= f;
                        a1 *= f;
                        a2 = ex2(other.x - ref);
                        l = l * f + a2 * other.y;
                        if (!misc->join_flag) l = 0.f;
                    }
                    const bool write = whole || keeper;
                    const float inv = write ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
                    if constexpr (kQuad) {
                        // 16 columns at a time: the copies' shares meet in the room of Q (its last product is
                        // done), and the warp of a quarter sums and writes four of the columns
                        float4 *meet = reinterpret_cast<float4 *>(sbase + (sQ - base)) + w * (4 * 4 * 32);
#pragma unroll 1
                        for (int c = w * (D / 32); c < (w + 1) * (D / 32); ++c) {
                            float f[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) f[e] = 0.f;
                            uint32_t o[16];
                            if (!dead) {
                                tmem_ld16_async(o0 + 16u * c, o);
                                tmem_ld_wait();
                                tmem_ld_bind16(o);
#pragma unroll
                                for (int e = 0; e < 16; ++e) f[e] = __uint_as_float(o[e]) * a0;
                            }
                            if (had1) {
                                tmem_ld16_async(o0 + 128u + 16u * c, o);
                                tmem_ld_wait();
                                tmem_ld_bind16(o);
#pragma unroll
                                for (int e = 0; e < 16; ++e) f[e] = fmaf(__uint_as_float(o[e]), a1, f[e]);
                            }
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                meet[(quarter * 4 + e) * 32 + lane] = make_float4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]);
                            named_sync(3 + w, 128);
                            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float4 y = meet[(e * 4 + quarter) * 32 + lane];
                                x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
                            }
                            named_sync(3 + w, 128);    // read, before the next columns go there
                            if (row_ok && ok) {
                                float4 *at = reinterpret_cast<float4 *>(p.o_part) + (slot * (D / 4) + 4 * c + quarter) * kVarlenTcRows + prow;
                                if (keeper) {
                                    const float4 y = __ldcg(at);
                                    x.x = fmaf(y.x, a2, x.x); x.y = fmaf(y.y, a2, x.y);
                                    x.z = fmaf(y.z, a2, x.z); x.w = fmaf(y.w, a2, x.w);
                                }
                                if (write) vl_store4(p, orow, 4 * c + quarter, make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
                                else __stcg(at, x);
                            }
                        }
                    } else
                    // (a loop, not unrolled: the code that runs once per unit is fetched once)
#pragma unroll 1
                    for (int c = c0; c < c1; ++c) {
                        uint32_t o[32];
                        if (!dead) {
                            tmem_ld32_async(o0 + 32u * c, o);
                            tmem_ld_wait();
                            tmem_ld_bind(o);
                        }
                        float f[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) f[e] = dead ? 0.f : __uint_as_float(o[e]) * (a0 * inv);
                        if (!pair && had1) {
                            tmem_ld32_async(o0 + 128u + 32u * c, o);
                            tmem_ld_wait();
                            tmem_ld_bind(o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) f[e] = fmaf(__uint_as_float(o[e]), a1 * inv, f[e]);
                        }
                        if (row_ok && ok) {
                            float4 *part = reinterpret_cast<float4 *>(p.o_part) +
                                           (slot * (D / 4) + 8 * c) * kVarlenTcRows + prow;
                            if (keeper) {
                                float4 v[8];
#pragma unroll
                                for (int e = 0; e < 8; ++e) v[e] = __ldcg(part + e * kVarlenTcRows);
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    f[4 * e] = fmaf(v[e].x, a2 * inv, f[4 * e]);
                                    f[4 * e + 1] = fmaf(v[e].y, a2 * inv, f[4 * e + 1]);
                                    f[4 * e + 2] = fmaf(v[e].z, a2 * inv, f[4 * e + 2]);
                                    f[4 * e + 3] = fmaf(v[e].w, a2 * inv, f[4 * e + 3]);
                                }
                            }
                            if (write) {
                                __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) + orow * D + 32 * c;
                                uint32_t v[16];
#pragma unroll
                                for (int q = 0; q < 16; ++q) {
                                    const __nv_bfloat162 b2 = __floats2bfloat162_rn(f[2 * q], f[2 * q + 1]);
                                    v[q] = *reinterpret_cast<const uint32_t *>(&b2);
                                }
                                // whole 32-byte sectors where the rows allow it
                                if (p.out32) {
                                    store_32b(dst, v);
                                    store_32b(dst + 16, v + 8);
                                } else {
#pragma unroll
                                    for (int q = 0; q < 4; ++q)
                                        *reinterpret_cast<uint4 *>(dst + 8 * q) =
                                            make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                                }
                            } else {
#pragma unroll
                                for (int e = 0; e < 32; e += 4)
                                    __stcg(part + (e / 4) * kVarlenTcRows, make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]));
                            }
                        }
                    }
                    if (row_ok && !write && (pair || w == 0) && (!kQuad || quarter == 0))
                        __stcg(p.ml_part + slot * kVarlenTcRows + prow,
                               make_float2(ok ? m_used : -INFINITY, ok ? l : 0.f));
                }
                if (two && !keeper) {
                    // announced at once, for the CTA that keeps the other part; should that one have
                    // given up waiting, the counter goes back to zero here
                    named_sync(1, 256);
                    if (tid == 128) {
                        __threadfence();
                        unsigned old;
                        asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(old) : "l"(p.ctr + sh->first)
                                     : "memory");
                        if (old == 1u) atomicExch(p.ctr + sh->first, 0u);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (pair) {
                    if (lane == 0 && n > 0) mbar_arrive(ofree_bar(w));
                } else {
                    named_sync(2, 256);                // both warpgroups have read both accumulators
                    if (lane == 0 && (w == 0 ? had0 : had1)) mbar_arrive(ofree_bar(w));
                }
                done_unit();
            }
            // the softmax warps (they hold the registers) join the shared units
            if (!have_ends) asm volatile("bar.sync 14, 288;" ::: "memory");
            const VlEnds &ends = misc->ends;
            named_sync(1, 256);                        // every part of this CTA is written
            if (tid - 128 < ends.n && ends.u[tid - 128].n > 2) vl_arrive(p, ends.u[tid - 128]);
            for (int i = 0; i < ends.n; ++i)
                if (ends.u[i].n > 2) vl_join(p, ends.u[i], tpt, 128, &misc->join_flag, tid - 128, 256, 1);
        }
    }

    // every product has been waited for by a softmax warp (or the CTA aborted:
    // then drain the pipe): free tensor memory
    __syncthreads();
    if (warp == 1 && lane == 0 && *abort_flag) {
        mbar_init(drain_bar, 1);       // used here alone
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        umma_commit(drain_bar);
        wait_bar(drain_bar, 0, nullptr, p.fault);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
template <int D, Rows8 kRows, bool kTree>
cudaError_t configure8() {
    // the shared-memory limit, and the registers that the warps share out
    static std::atomic<bool> done[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    cudaFuncAttributes a;
    e = cudaFuncGetAttributes(&a, attn_varlen_tc8_kernel<D, kRows, kTree>);
    if (e != cudaSuccess) return e;
    if (a.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;   // setmaxnreg would wait for registers that are not there
    e = cudaFuncSetAttribute(attn_varlen_tc8_kernel<D, kRows, kTree>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Lay8<D>::kSmem);
    if (e == cudaSuccess && dev >= 0 && dev < kMaxDevices) done[dev].store(true, std::memory_order_release);
    return e;
}

template <int D, Rows8 kRows, bool kTree>
cudaError_t launch_tc8(const VarlenParams &p, int grid, cudaStream_t st) {
    const int tpt = 128 / (p.Hq / p.Hkv), box_rows = page_box(p.page_size);
    alignas(64) CUtensorMap m[2];
    PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn_vl();
    if (!fn) return cudaErrorInvalidValue;
    for (int i = 0; i < 2; ++i) {       // (d, slot, kv head, page): a copy per page
        const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)p.page_size, (cuuint64_t)p.Hkv, (cuuint64_t)p.n_pages};
        const cuuint64_t strides[3] = {(cuuint64_t)p.kv.s, (cuuint64_t)p.kv.h, (cuuint64_t)p.kv.b};
        const cuuint32_t box[4] = {(cuuint32_t)D, (cuuint32_t)box_rows, 1, 1}, one[4] = {1, 1, 1, 1};
        if (fn(&m[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(i ? p.v : p.k), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               // a row's own bytes: 256 would fetch the next heads' with them, for CTAs that come much later (64
               // sequences of one token: 315 MB from memory against 249)
               D == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_64B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    cudaError_t e = configure8<D, kRows, kTree>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Lay8<D>::kSmem;
    cfg.stream = st;
    // the CTAs of a shared unit wait for one another: a cooperative launch makes
    // them resident together
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeCooperative;
    attr[1].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, attn_varlen_tc8_kernel<D, kRows, kTree>, m[0], m[1], p, tpt, box_rows);
}

template <int D, bool kTree> cudaError_t launch_rows8(const VarlenParams &p, int grid, cudaStream_t st) {
    const int G = p.Hq / p.Hkv;
    if (p.max_q * G <= 32) return launch_tc8<D, kQuad8, kTree>(p, grid, st);
    return p.max_q <= 128 / G ? launch_tc8<D, kSmall8, kTree>(p, grid, st) : launch_tc8<D, kPairs, kTree>(p, grid, st);
}
template <int D> cudaError_t launch_d(const VarlenParams &p, int grid, cudaStream_t st) {
    return p.tree ? launch_rows8<D, true>(p, grid, st) : launch_rows8<D, false>(p, grid, st);
}

}  // namespace

cudaError_t launch_varlen_tc8(const VarlenParams &p, int grid, cudaStream_t st) {
    return p.D == 128 ? launch_d<128>(p, grid, st) : launch_d<64>(p, grid, st);
}

}  // namespace sdv
