// Attention of packed new tokens on the tensor cores, for sm_103a: bf16, over
// the prompts' own keys or a paged cache whose pages are a multiple of 8 slots.
//
// For a unit (up to 256 query rows: 2 tiles of 128, each of 128 / G whole
// tokens with their G query heads) and key tile t of 128 keys:
//   S_t = Q K_t^T,  m = max(m, max S_t),  P_t = exp2((S_t - m) scale log2 e)
//   O = O + P_t V_t,  l = l + sum P_t,  out = O / l
// one pass over the keys, S and P in tensor memory, P rounded to bf16 for the
// second product (the running sum takes P before that rounding).  The heads of
// a group share a tile, so K and V are read once per 256 rows whatever G is,
// and a causal edge is 128 / G tokens wide instead of 128.
//
// Persistent, one CTA per SM; the units' tiles are dealt out evenly (varlen.cuh).
// Warp roles (384 threads; the softmax warps take over registers of the others):
//   warp 0            TMA: Q, and K and V tiles in the order of their use through
//                     a ring of tiles (a page at a time for a paged cache)
//   warp 1            issues the MMAs; warp 2 allocates tensor memory; warp 3 works
//                     out which units the CTA shares
//   warps 4-7, 8-11   softmax, thread = row: warpgroup i owns S_i and O_i
// The two warpgroups are two streams that alternate on the tensor pipe: while
// one does its softmax, the other's products run.  In a unit of more than 128
// rows stream i is row tile i and both read every K/V tile; in a smaller one
// (decoding, block verification) the streams take the even and the odd key
// tiles of the one row tile, and are joined at its end.
// The reference of a row's weights moves only where its maximum grows by more
// than 2^16 (bf16 and fp32 hold weights above 1 as well as those below), and O is
// rescaled then; P and l use the same reference, so it is exact either way.
// P is rounded to nearest bf16 for the second product, the running sum takes it
// before that: an output is off by about as much again as by its own rounding.
// Tensor memory: S_0 [0,128), S_1 [128,256), O_0 [256,256+D), O_1 [384,384+D);
// P_i overlays the first 64 columns of S_i (its second term, in the small form,
// the others).
//
// Measured.  A causal prompt of 25,119 tokens (28 / 4 heads of 128) takes 2.88 to
// 2.98 ms by the box's power, 1.52 to 1.57 PFLOP/s, 0.90 to 0.93 of what a large
// library product sustains on this part: the tensor pipe and its power.  The
// products read Q and K from shared
// memory at its full rate, 128 bytes a clock, so a pair of tiles takes 2,300
// clocks of the pipe instead of 2,050.  2,048 new tokens over 32,768 (64 / 8) take
// 1.49 ms.  One token over 25,119 takes 20.5 us for its 51 MB: 7.6 us of memory
// time between 6 us of start (the plan, the page table, the first tile) and 6 us
// of end (the last product, the join over 38 CTAs).  One token each of 64 and 256
// sequences over 4,000 keys takes 90 and 336 us with pages of 64 (floors of memory
// 78 and 310), 102 and 373 with pages of 16; over 900 keys 44 and 137 (18 and 70).
// 16 rows each of 8 sequences of
// 4,096 to 32,768 take 55 us with pages of 64 slots, 58 with pages of 16 and 69 with
// pages of 8: a copy costs about 40 clocks besides the 4 of each 128-byte row.
// Short units are bound by what surrounds their tiles: about 9,000 clocks a unit
// against 2,800 a tile.
//
// Every wait is bounded; one that gives up sets the fault word, and the CTA
// drains its copies and MMAs before it returns.
#include "tcgen05.cuh"
#include "varlen.cuh"

#include <math.h>
#include <atomic>

namespace sdv {

namespace {

constexpr int kThreads = 384;
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;   // 216 * 256 + 72 * 128 = 168 * 384
constexpr int kLaunchRegs = 168;
static_assert(kSoftmaxRegs * 256 + kOtherRegs * 128 <= kLaunchRegs * kThreads, "register shares within the launch's");
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescale = 16.0f;           // log2 units
constexpr int kPFirst = 64;                 // keys of P announced first; P V of these runs while the others' weights are made

template <int D> struct Lay {
    static constexpr int kHalves = D / 64;
    static constexpr int kTile = kHalves * 128 * 128;      // Q, K or V tile: 64-column blocks of [128 rows x 128 B]
    static constexpr int kSlots = D == 128 ? 5 : 9;
    static constexpr int kOffQ = 0;                        // two row tiles
    static constexpr int kOffRing = 2 * kTile;
    static constexpr int kOffBar = kOffRing + kSlots * kTile;
    static constexpr int kMaxSlots = kSlots + 1;           // where no unit has a second row tile, its room too
    // full[max] empty[max] qfull qempty sfull[2] pfull[2][2] ofull[2] ofree[2]
    static constexpr int kBars = 2 * kMaxSlots + 2 + 2 + 4 + 2 + 2;
    static constexpr int kOffMl = kOffBar + 8 * kBars + 8; // [2][128] exchange between the streams
    static constexpr int kOffMisc = kOffMl + 2 * 128 * 4;
    static constexpr int kSmem = kOffMisc + 512 + 1024;    // + alignment slack
    static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
};

struct Misc {
    uint32_t tmem;
    int abort_flag;
    int join_flag;
    int pad;
    VlPlan plan;
    VlEnds ends;
};
static_assert(sizeof(Misc) <= 512, "the misc area");

struct RingPos {        // slot and phase of the next tile in a ring
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void step(int n) { if (++slot == n) { slot = 0; phase ^= 1u; } }
};

// mbar_wait, inlined: a call cannot be made where the warps' register counts differ
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int *abort_flag, unsigned int *fault) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = global_timer();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 63u) == 0) {
            if (abort_flag && *abort_flag) return false;
            if (global_timer() - t0 > kWaitLimitNs) {
                if (abort_flag) *abort_flag = 1;
                set_fault(fault, FAULT_WAIT_TIMEOUT);
                return false;
            }
        }
    }
}

// K or V of 128 keys of the packed rows, or one page's 64 columns, with an L2 policy
__device__ __forceinline__ void load_kv_4d(uint32_t dst, const CUtensorMap *map, uint32_t bar, uint64_t policy, int row,
                                           int g) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(0), "r"(g), "r"(bar), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void load_kv_5d(uint32_t dst, const CUtensorMap *map, uint32_t bar, uint64_t policy, int slot,
                                           int half, int g, int page) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(slot), "r"(half), "r"(g), "r"(page), "r"(bar), "l"(policy)
        : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ void tmem_ld16_async(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13,"
        " %14, %15}, [%16];"
        : SDV_R8(0), SDV_R8(8)
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_bind16(uint32_t (&r)[16]) { asm volatile("" : SDV_W8(0), SDV_W8(8)); }

__device__ __forceinline__ void store_32b(void *p, const uint32_t *v) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// true in one lane of a converged warp, the same one each time
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r != 0;
}

// kSmall: no sequence has more rows of a kv head than one tile holds (decoding,
// block verification).  Those calls are bound by memory, so P goes into the
// second product as two bf16 terms, to 2^-16 of each weight, and the second row
// tile's room is a ring slot more.
// kFrom: where K and V are.  kPacked: the prompts' own rows.  kPages: a paged
// cache.  kPages16: one at D = 128 that is copied 16 slots at a time, with both
// 64-column blocks of those slots in one copy for K too.  K's 8-row groups then
// lie in two evenly spaced sets, the first and the second of each 16, and the
// scores come as two products of 64 columns: column c < 64 is key
// 16 (c / 8) + c % 8 of the tile, column 64 + c the key 8 further on; P and V
// follow that order.
template <bool kSets> __device__ __forceinline__ constexpr int key_of(int c) {
    return kSets ? 16 * ((c & 63) >> 3) + 8 * (c >> 6) + (c & 7) : c;
}
enum From { kPacked, kPages, kPages16 };
template <int D, From kFrom, bool kSmall>
__global__ void __launch_bounds__(kThreads, 1)
attn_varlen_tc_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                      const __grid_constant__ CUtensorMap tmap_v, const VarlenParams p, const int tpt, const int box) {
    using L = Lay<D>;
    constexpr bool kPaged = kFrom != kPacked, kSets = kFrom == kPages16;
    static_assert(!kSets || D == 128, "one 64-column block lies evenly anyway");
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u32 = smem_u32(smem_raw);
    const uint32_t base = (raw_u32 + 1023u) & ~1023u;
    uint8_t *sbase = smem_raw + (base - raw_u32);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = (int)blockIdx.x;

    const uint32_t sQ = base + L::kOffQ, sRing = base + L::kOffRing - (kSmall ? L::kTile : 0), bar0 = base + L::kOffBar;
    constexpr int slots = kSmall ? L::kMaxSlots : L::kSlots;
    auto full_bar = [&](int i) { return bar0 + 8u * i; };
    auto empty_bar = [&](int i) { return bar0 + 8u * (L::kMaxSlots + i); };
    const uint32_t bar1 = bar0 + 8u * (2 * L::kMaxSlots);
    const uint32_t qfull_bar = bar1, qempty_bar = bar1 + 8u;
    auto sfull_bar = [&](int i) { return bar1 + 8u * (2 + i); };             // S_i computed
    auto pfull_bar = [&](int i, int h) { return bar1 + 8u * (4 + 2 * i + h); };   // half h of P_i written (4 warps)
    auto ofull_bar = [&](int i) { return bar1 + 8u * (8 + i); };             // O_i complete for the unit
    auto ofree_bar = [&](int i) { return bar1 + 8u * (10 + i); };            // O_i read out (4 warps)
    float *xrow = reinterpret_cast<float *>(sbase + L::kOffMl);      // [2][128]: one value per stream and row
    Misc *misc = reinterpret_cast<Misc *>(sbase + L::kOffMisc);
    volatile int *abort_flag = &misc->abort_flag;

    if (tid == 0) {
        for (int i = 0; i < L::kMaxSlots; ++i) { mbar_init(full_bar(i), 1); mbar_init(empty_bar(i), 1); }
        mbar_init(qfull_bar, 1);
        mbar_init(qempty_bar, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(sfull_bar(i), 1);
            mbar_init(pfull_bar(i, 0), 4);
            mbar_init(pfull_bar(i, 1), 4);
            mbar_init(ofull_bar(i), 1);
            mbar_init(ofree_bar(i), 4);
        }
        misc->abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_q)) : "memory");
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
                VlWalk walk(pl);
                VlUnit u;
                RingPos rp;
                uint32_t qphase = 0;
                long loads = 0, units = 0;
                bool ok = true;
                // K and V that one unit alone reads leave L2 first (one token over 25,119: 22.2 -> 20.2 us);
                // what several units read stays as usual
                uint64_t once, again;
                asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
                asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(again));
                const int per_half = 128 / box;        // copies per 64-column block of a tile
                while (ok && walk.next(p, pl, u)) {
                    const int n = u.t1 - u.t0;
                    if (n <= 0) continue;
                    const int la = kSmall || u.ntok <= tpt ? 2 : 1;
                    const uint64_t policy = walk.s.nr == 1 ? once : again;
                    const int32_t *trow = kPaged ? p.table + (long)u.b * p.table_stride : nullptr;
                    // the lane's page of tile t: looked up a tile ahead, first used (and checked) by its copy
                    auto page_of = [&](int t) {
                        if (!kPaged) return 0;
                        const int key = t * 128 + (lane % per_half) * box;
                        int pg = -1;
                        if (key < u.kv) {
                            pg = __ldg(trow + (p.page_log2 >= 0 ? key >> p.page_log2 : key / p.page_size));
                        }
                        return pg;
                    };
                    auto load_tile = [&](bool is_v, int t, int pg) {
                        if (ok && loads >= slots)
                            ok = wait_bar(empty_bar(rp.slot), rp.phase ^ 1u, abort_flag, p.fault);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) return;
                        const uint32_t dst = sRing + rp.slot * L::kTile, bar = full_bar(rp.slot);
                        const CUtensorMap *map = is_v ? &tmap_v : &tmap_k;
                        if (!kPaged) {
                            if (lane == 0) {
                                mbar_arrive_expect_tx(bar, (uint32_t)L::kTile);
                                load_kv_4d(dst, map, bar, policy, u.row0 - u.tok0 + t * 128, u.g);
                            }
                        } else {
                            // V comes with both 64-column blocks of a page in one copy (a copy costs about
                            // 40 clocks besides the 4 of each 128-byte row), and K where its rows then lie
                            // evenly enough for the products: copies of 8 slots, and of 16 (From)
                            const int boxes = min(per_half, (u.kv - t * 128 + box - 1) / box);
                            if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(boxes * box * 128 * L::kHalves));
                            __syncwarp();
                            const bool both = kSets || is_v || box == 8;
                            const int i = lane % per_half, h = lane / per_half;
                            if (i < boxes && h < (both ? 1 : L::kHalves)) {
                                const int key = t * 128 + i * box;
                                if (pg < 0 || pg >= p.n_pages) {      // read as zeros: the copy's fill
                                    set_fault(p.fault, FAULT_BAD_PAGE);
                                    pg = p.n_pages;
                                }
                                load_kv_5d(dst + (both ? i * box * 128 * L::kHalves : h * (128 * 128) + i * box * 128),
                                           map, bar, policy,
                                           p.page_log2 >= 0 ? key & (p.page_size - 1) : key % p.page_size, h, u.g, pg);
                            }
                        }
                        rp.step(slots);
                        ++loads;
                    };
                    int pk = page_of(u.t0), pv = pk;      // pages of the next K tile, of the V tile behind it
                    int pk2 = 0;
                    // the first unit's Q at once; a later one's behind its first K tile, when the
                    // last unit's S products have read the old Q
                    if (units > 0) {
                        load_tile(false, u.t0, pk);
                        if (ok) ok = wait_bar(qempty_bar, qphase ^ 1u, abort_flag, p.fault);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                    }
                    if (lane == 0) {
                        const int nq = kSmall || u.ntok <= tpt ? 1 : 2;
                        mbar_arrive_expect_tx(qfull_bar, (uint32_t)(nq * L::kHalves * 128 * G * tpt));
                        for (int i = 0; i < nq; ++i)
                            for (int h = 0; h < L::kHalves; ++h)
                                tma_load_3d(sQ + i * L::kTile + h * (128 * 128), &tmap_q, qfull_bar, 64 * h, u.g * G,
                                            u.row0 + i * tpt);
                    }
                    __syncwarp();
                    if (units == 0) load_tile(false, u.t0, pk);
                    if (n > 1) pk = page_of(u.t0 + 1);
                    qphase ^= 1u;
                    ++units;
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
                    if (units > 0) wait_bar(qfull_bar, qphase ^ 1u, nullptr, p.fault);
                }
            } else if (warp == 1) {
                // ---------------------------------------------------------- MMA issuer
                // the whole warp runs the loop and one elected lane issues: the descriptors are then the
                // same in every lane for the compiler too and stay in uniform registers (issued from inside
                // a one-lane branch, the products took twice as long: 4.49 ms against 3.10 for the
                // 25,119-token prompt)
                {
                    const bool el = elect_one();
                    VlWalk walk(pl);
                    VlUnit u;
                    RingPos rp;
                    uint32_t qphase = 0, pphase[2] = {0, 0}, fphase[2] = {0, 0};
                    bool used[2] = {false, false};
                    bool ok = true;
                    const uint32_t idS = idesc_bf16(128, 128, false), idO = idesc_bf16(128, D, true);
                    auto wait_tile = [&]() {
                        ok = ok && wait_bar(full_bar(rp.slot), rp.phase, abort_flag, p.fault);
                        tc_fence_after();
                    };
                    // descriptors by their first tile's, moved on by whole 16-byte units
                    // K: its 8-row groups 1024 bytes apart, the 64-column blocks one after the other; from
                    // copies of 8 slots the blocks alternate every group, from copies of 16 as `From` says.
                    // V: 64-column blocks alternate every `box` rows (128 where K and V are not paged).
                    const uint32_t eight = box == 8 ? L::kHalves : 1;
                    const uint32_t khalf = (box == 8 ? 1024 : 128 * 128) / 16;
                    const uint64_t qd0 = sw128_desc(sQ, 16, 1024), kd0 = sw128_desc(sRing, 16, 1024 * eight),
                                   vd0 = sw128_desc(sRing, (uint32_t)box * 128, kSets ? 4096 : 1024 * eight);
                    const uint64_t ksets = sw128_desc(sRing, 16, 4096);       // a set's groups, one per 16 slots
                    uint32_t vrow[8];              // where the 16 keys of step kk begin in a V tile, in 16 bytes
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        vrow[kk] = kSets ? (kk & 3) * (8192 / 16) + (kk >> 2) * (1024 / 16)
                                         : (((16 * kk) & ~(box - 1)) * L::kHalves + ((16 * kk) & (box - 1))) * (128 / 16);
                    auto issue_s = [&](int i, int qt, int slot) {
                        const uint64_t qd = qd0 + (uint64_t)(qt * (L::kTile / 16)),
                                       kd = kd0 + (uint64_t)(slot * (L::kTile / 16));
                        if (el) {
                            if constexpr (kSets) {
                                const uint64_t kb = ksets + (uint64_t)(slot * (L::kTile / 16));
#pragma unroll
                                for (int set = 0; set < 2; ++set)
#pragma unroll
                                    for (int kk = 0; kk < D / 16; ++kk)
                                        umma_ss(tmem + 128u * i + 64u * set,
                                                qd + (kk & 3) * 2 + (kk >> 2) * (128 * 128 / 16),
                                                kb + set * (1024 / 16) + (kk & 3) * 2 + (kk >> 2) * (2048 / 16),
                                                idesc_bf16(128, 64, false), kk > 0 ? 1u : 0u);
                            } else {
#pragma unroll
                                for (int kk = 0; kk < D / 16; ++kk) {
                                    const uint64_t off = (kk & 3) * 2;
                                    umma_ss(tmem + 128u * i, qd + off + (kk >> 2) * (128 * 128 / 16),
                                            kd + off + (kk >> 2) * khalf, idS, kk > 0 ? 1u : 0u);
                                }
                            }
                            umma_commit(sfull_bar(i));
                        }
                    };
                    auto issue_pv = [&](int i, int slot, bool first, int steps) {
                        const uint64_t vd = vd0 + (uint64_t)(slot * (L::kTile / 16));
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            ok = ok && wait_bar(pfull_bar(i, h), pphase[i], abort_flag, p.fault);
                            if (!ok) return;
                            tc_fence_after();
                            if (el) {
#pragma unroll
                                for (int kk = h ? kPFirst / 16 : 0; kk < (h ? 8 : kPFirst / 16); ++kk) {
                                    if (kSmall && (kSets ? 2 * (kk & 3) : kk) >= steps) continue;
                                    umma_ts(tmem + 256u + 128u * i, tmem + 128u * i + 8u * kk, vd + vrow[kk], idO,
                                            (!first || kk > 0) ? 1u : 0u);
                                    if (kSmall)
                                        umma_ts(tmem + 256u + 128u * i, tmem + 128u * i + 64u + 8u * kk, vd + vrow[kk],
                                                idO, 1u);
                                }
                            }
                        }
                        pphase[i] ^= 1u;
                    };
                    // O_i free for a new unit
                    auto claim = [&](int i) {
                        if (used[i]) {
                            ok = ok && wait_bar(ofree_bar(i), fphase[i], abort_flag, p.fault);
                            tc_fence_after();
                            fphase[i] ^= 1u;
                        }
                        used[i] = true;
                    };
                    while (ok && walk.next(p, pl, u)) {
                        const int n = u.t1 - u.t0;
                        if (n <= 0) continue;
                        const bool pair = !kSmall && u.ntok > tpt;
                        // the small form's second products stop at the step of 16 that holds the last key
                        auto steps = [&](int j) { return kSmall ? (u.kv - (u.t0 + j) * 128 + 15) >> 4 : 8; };
                        ok = wait_bar(qfull_bar, qphase, abort_flag, p.fault);
                        if (!ok) break;
                        qphase ^= 1u;
                        wait_tile();
                        if (!ok) break;
                        issue_s(0, 0, rp.slot);
                        if (pair) issue_s(1, 1, rp.slot);
                        if (el) umma_commit(empty_bar(rp.slot));
                        rp.step(slots);
                        if (pair) {
                            if (n == 1) if (el) umma_commit(qempty_bar);
                            for (int j = 0; ok && j < n; ++j) {
                                wait_tile();
                                if (!ok) break;
                                const RingPos vp = rp;
                                rp.step(slots);
                                if (j == 0) claim(0);
                                issue_pv(0, vp.slot, j == 0, 8);
                                if (!ok) break;
                                if (j + 1 < n) {
                                    wait_tile();
                                    if (!ok) break;
                                    issue_s(0, 0, rp.slot);
                                } else {
                                    if (el) umma_commit(ofull_bar(0));
                                }
                                if (j == 0) claim(1);
                                issue_pv(1, vp.slot, j == 0, 8);
                                if (!ok) break;
                                if (el) umma_commit(empty_bar(vp.slot));
                                if (j + 1 < n) {
                                    issue_s(1, 1, rp.slot);
                                    if (el) umma_commit(empty_bar(rp.slot));
                                    rp.step(slots);
                                    if (j + 2 == n) if (el) umma_commit(qempty_bar);
                                } else {
                                    if (el) umma_commit(ofull_bar(1));
                                }
                            }
                        } else {
                            if (n > 1) {
                                wait_tile();
                                if (!ok) break;
                                issue_s(1, 0, rp.slot);
                                if (el) umma_commit(empty_bar(rp.slot));
                                rp.step(slots);
                            }
                            if (n <= 2) if (el) umma_commit(qempty_bar);
                            for (int j = 0; ok && j < n; ++j) {
                                const int i = j & 1;
                                wait_tile();
                                if (!ok) break;
                                if (j < 2) claim(i);
                                issue_pv(i, rp.slot, j < 2, steps(j));
                                if (!ok) break;
                                if (el) umma_commit(empty_bar(rp.slot));
                                rp.step(slots);
                                if (j + 2 < n) {
                                    wait_tile();
                                    if (!ok) break;
                                    issue_s(i, 0, rp.slot);
                                    if (el) umma_commit(empty_bar(rp.slot));
                                    rp.step(slots);
                                    if (j + 3 == n) if (el) umma_commit(qempty_bar);
                                } else {
                                    if (el) umma_commit(ofull_bar(i));
                                }
                            }
                        }
                    }
                    if (!ok) *abort_flag = 1;
                }
                __syncwarp();
            } else if (warp == 3) {
                vl_ends(p, pl, cta, &misc->ends);
                asm volatile("bar.arrive 14, 288;" ::: "memory");
            }
        } else {
            // -------------------------------------------------------------- softmax
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
            const int w = (warp - 4) >> 2;             // stream
            const int r = (tid - 128) & 127;           // row of the tile = tensor-memory lane
            const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t s_col = tmem + lane_off + 128u * w, o_col = tmem + lane_off + 256u + 128u * w;
            const float qk = p.scale * kLog2e;
            const int tr = r / G;                      // token of the row within its tile
            VlWalk walk(pl);
            VlUnit u;
            uint32_t sphase = 0, ophase0 = 0, ophase1 = 0;
            bool have_ends = false;
            unsigned ring = 0;                         // tiles that went through the ring before this unit
            bool ok = true;
            while (walk.next(p, pl, u)) {
                const int n = u.t1 - u.t0;
                const bool pair = !kSmall && u.ntok > tpt;
                const int tl = tr + (pair && w ? tpt : 0);             // token within the unit
                const bool row_ok = tr < tpt && tl < u.ntok;
                const int lim = row_ok ? vl_limit(p, u, u.tok0 + tl) : 0;
                // rows this warp has to do anything for
                const bool warp_live = __any_sync(0xffffffffu, row_ok);
                float m_used = -INFINITY, l = 0.f;
                const int step = pair ? 1 : 2, la = pair ? 1 : 2;
                const int j0 = pair ? 0 : w;
                for (int j = j0; j < n; j += step) {
                    const int key0 = (u.t0 + j) * 128;
                    ok = __all_sync(0xffffffffu, wait_bar(sfull_bar(w), sphase, abort_flag, p.fault)) && ok;
                    sphase ^= 1u;
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
                        const int v0 = u.kv - key0, v1 = !kSmall ? 128 : kSets ? (v0 + 31) & ~31 : (v0 + 15) & ~15;
                        for (int i = r; i < (v1 - v0) * 8 * L::kHalves; i += 128) {
                            const int row = v0 + i / (8 * L::kHalves), ch = i % (8 * L::kHalves);
                            const int in = row & (box - 1);
                            *reinterpret_cast<uint4 *>(vt + ((row - in) * L::kHalves + (ch >> 3) * box) * 128 +
                                                       sw128_off(in, ch & 7)) =
                                make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                        // every warp's rows, before any arrival lets the product start
                        named_sync(3 + w, 128);
                    }
                    if (warp_live) {
                        uint32_t s[4][32];
#pragma unroll
                        for (int c = 0; c < 4; ++c) tmem_ld32_async(s_col + 32u * c, s[c]);
                        tmem_ld_wait();
#pragma unroll
                        for (int c = 0; c < 4; ++c) tmem_ld_bind(s[c]);
                        const int vis = lim - key0;                     // this row sees keys [0, vis) of the tile
                        if (!__all_sync(0xffffffffu, vis >= 128 || !row_ok)) {
#pragma unroll
                            for (int c = 0; c < 4; ++c)
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (key_of<kSets>(32 * c + e) >= vis) s[c][e] = 0xff800000u;
                        }
                        const float2 qk2 = make_float2(qk, qk);
                        float2 ls[2], nm2;
                        uint32_t pk[16], lo[kSmall ? 16 : 1];
                        // weights of 16 keys: 8 words from `at`
                        auto weights = [&](int at) {
#pragma unroll
                            for (int c = at; c < at + 16; ++c) {
                                const uint32_t *src = s[c >> 4] + 2 * (c & 15);
                                const float2 x = __ffma2_rn(make_float2(__uint_as_float(src[0]), __uint_as_float(src[1])),
                                                            qk2, nm2);
                                const float p0 = ex2(x.x), p1 = ex2(x.y);
                                ls[c & 1] = __fadd2_rn(ls[c & 1], make_float2(p0, p1));
                                const __nv_bfloat162 b2 = __floats2bfloat162_rn(p0, p1);
                                const uint32_t hi = *reinterpret_cast<const uint32_t *>(&b2);
                                pk[c & 15] = hi;
                                if constexpr (kSmall) {       // what the rounding left, exact in fp32
                                    const __nv_bfloat162 r2 = __floats2bfloat162_rn(
                                        p0 - __uint_as_float(hi << 16), p1 - __uint_as_float(hi & 0xffff0000u));
                                    lo[c & 15] = *reinterpret_cast<const uint32_t *>(&r2);
                                }
                            }
                        };
                        float m4[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float m = max3(__uint_as_float(s[i][0]), __uint_as_float(s[i][1]), __uint_as_float(s[i][2]));
#pragma unroll
                            for (int e = 3; e < 31; e += 2)
                                m = max3(m, __uint_as_float(s[i][e]), __uint_as_float(s[i][e + 1]));
                            m4[i] = fmaxf(m, __uint_as_float(s[i][31]));
                        }
                        const float tmax = qk * fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]);
                        const bool need = tmax > m_used + kRescale;     // true at first while m_used = -inf
                        float alpha = 1.f;
                        if (need) {
                            alpha = ex2(m_used - tmax);                 // 0 while nothing is held
                            m_used = tmax;
                        }
                        if (j > j0 && __any_sync(0xffffffffu, need)) {
                            // S_j is complete, hence every earlier product of this stream too
                            // (they were issued before it and complete in order)
#pragma unroll 1
                            for (int c = 0; c < D / 16; ++c) {
                                uint32_t o[16];
                                tmem_ld16_async(o_col + 16u * c, o);
                                tmem_ld_wait();
                                tmem_ld_bind16(o);
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                                tmem_st16(o_col + 16u * c, o);
                            }
                        }
                        const float neg_m = m_used == -INFINITY ? 0.f : -m_used;
                        nm2 = make_float2(neg_m, neg_m);
                        ls[0] = ls[1] = make_float2(0.f, 0.f);
                        weights(0);
                        l *= alpha;
                        // 32 keys' weights, over the scores' first 64 columns (what is left of them over the others)
                        auto put = [&](uint32_t q) {
                            tmem_st16(s_col + 16u * q, pk);
                            if constexpr (kSmall) tmem_st16(s_col + 64u + 16u * q, lo);
                        };
                        put(0);
                        weights(16);
                        put(1);
                        if (!kSmall) weights(32);      // while the stores run (the small form has no registers for it)
                        tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(pfull_bar(w, 0));
                        if (kSmall) weights(32);
                        put(2);
                        weights(48);
                        put(3);
                        tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(pfull_bar(w, 1));
                        l += (ls[0].x + ls[1].x) + (ls[0].y + ls[1].y);
                    } else {
                        tc_fence_before();
                        if (lane == 0) { mbar_arrive(pfull_bar(w, 0)); mbar_arrive(pfull_bar(w, 1)); }
                    }
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
                ring += 2 * n;
                float a0 = 1.f, a1 = 0.f;
                if (!pair) {
                    // join the two streams of the one row tile: they exchange the row's maximum, then
                    // its sum, and each takes half of the columns of both accumulators
                    xrow[128 * w + r] = m_used;
                    named_sync(1, 256);
                    const float mo = xrow[128 * (w ^ 1) + r];
                    const float m = fmaxf(m_used, mo), ref = m == -INFINITY ? 0.f : m;
                    const float own = ex2(m_used - ref), other = ex2(mo - ref);
                    l *= own;
                    m_used = m;
                    a0 = w == 0 ? own : other;
                    a1 = w == 0 ? other : own;
                    named_sync(2, 256);
                    xrow[128 * w + r] = l;
                    named_sync(1, 256);
                    l += xrow[128 * (w ^ 1) + r];
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
                    const long prow = 128 * (pair ? w : 0) + r;
                    const long orow = (long)(u.row0 + tl) * p.Hq + u.g * G + (r - tr * G);
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
                    if (row_ok && !write && (pair || w == 0))
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
        // the barrier's phase may be anything: re-initialise one that nobody uses any more
        mbar_init(qempty_bar, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        umma_commit(qempty_bar);
        wait_bar(qempty_bar, 0, nullptr, p.fault);
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
PFN_cuTensorMapEncodeTiled_v12000 encode_fn_vl() {
    // looked up once; the initialisation of a function-local static is thread-safe
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess && q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
        return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
    }();
    return fn;
}

bool encode_vl(CUtensorMap *m, const void *ptr, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
               const cuuint32_t *box) {
    PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn_vl();
    if (!fn) return false;
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int page_box(int page_size) {       // slots per copy: the largest power of two that divides the page, up to 128
    int b = 128;
    while (page_size % b) b >>= 1;
    return b;
}

template <int D, From kFrom, bool kSmall>
cudaError_t configure() {
    // the shared-memory limit, and the registers that the warps share out
    static std::atomic<bool> done[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    cudaFuncAttributes a;
    e = cudaFuncGetAttributes(&a, attn_varlen_tc_kernel<D, kFrom, kSmall>);
    if (e != cudaSuccess) return e;
    if (a.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;   // setmaxnreg would wait for registers that are not there
    e = cudaFuncSetAttribute(attn_varlen_tc_kernel<D, kFrom, kSmall>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Lay<D>::kSmem);
    if (e == cudaSuccess && dev >= 0 && dev < kMaxDevices) done[dev].store(true, std::memory_order_release);
    return e;
}

template <int D, From kFrom, bool kSmall>
cudaError_t launch_tc(const VarlenParams &p, int grid, cudaStream_t st) {
    const int G = p.Hq / p.Hkv, tpt = 128 / G;
    alignas(64) CUtensorMap mq, mk, mv;
    {   // (d, head, token): box 64 d x G heads x tpt tokens = rows token * G + head of 128 bytes
        const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)p.Hq, (cuuint64_t)p.N};
        const cuuint64_t strides[2] = {(cuuint64_t)p.q_head * 2, (cuuint64_t)p.q_tok * 2};
        const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)tpt};
        if (!encode_vl(&mq, p.q, 3, dims, strides, box)) return cudaErrorInvalidValue;
    }
    int box_rows = 128;
    for (int i = 0; i < 2; ++i) {
        const void *t = i ? p.v : p.k;
        CUtensorMap *m = i ? &mv : &mk;
        if (kFrom != kPacked) {   // (d % 64, slot, d / 64, kv head, page): a copy per page and 64-column block
            box_rows = page_box(p.page_size);
            const cuuint64_t dims[5] = {64, (cuuint64_t)p.page_size, (cuuint64_t)(D / 64), (cuuint64_t)p.Hkv,
                                        (cuuint64_t)p.n_pages};
            const cuuint64_t strides[4] = {(cuuint64_t)p.kv.s * 2, 128, (cuuint64_t)p.kv.h * 2, (cuuint64_t)p.kv.b * 2};
            const cuuint32_t both = i == 1 || kFrom == kPages16 || box_rows == 8 ? D / 64 : 1;
            const cuuint32_t box[5] = {64, (cuuint32_t)box_rows, both, 1, 1};
            if (!encode_vl(m, t, 5, dims, strides, box)) return cudaErrorInvalidValue;
        } else {        // (d % 64, token, d / 64, kv head): one copy per tile
            const cuuint64_t dims[4] = {64, (cuuint64_t)p.N, (cuuint64_t)(D / 64), (cuuint64_t)p.Hkv};
            const cuuint64_t strides[3] = {(cuuint64_t)p.kv.s * 2, 128, (cuuint64_t)p.kv.h * 2};
            const cuuint32_t box[4] = {64, 128, (cuuint32_t)(D / 64), 1};
            if (!encode_vl(m, t, 4, dims, strides, box)) return cudaErrorInvalidValue;
        }
    }
    cudaError_t e = configure<D, kFrom, kSmall>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Lay<D>::kSmem;
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
    return cudaLaunchKernelEx(&cfg, attn_varlen_tc_kernel<D, kFrom, kSmall>, mq, mk, mv, p, tpt, box_rows);
}

}  // namespace

bool varlen_tc_supported(const VarlenParams &p) {
    if (p.dt != SD_BF16 || (p.D != 64 && p.D != 128) || p.Hq / p.Hkv > kVarlenMaxGroup) return false;
    if (p.table && p.page_size % 8) return false;      // a copy's rows start on the swizzle's 8-row period
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
    static std::atomic<int> known[kMaxDevices];       // per device: 0 not asked, 1 no, 2 yes
    int k = known[dev].load(std::memory_order_acquire);
    if (k == 0) {
        int optin = 0, major = 0, minor = 0;
        if (cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess) return false;
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
        k = encode_fn_vl() && optin >= Lay<128>::kSmem && optin >= Lay<64>::kSmem && major == 10 && minor == 3 ? 2 : 1;
        known[dev].store(k, std::memory_order_release);
    }
    return k == 2;
}

cudaError_t launch_varlen_tc(const VarlenParams &p, int grid, cudaStream_t st) {
    const bool small = p.max_q <= 128 / (p.Hq / p.Hkv);
    if (p.D == 128) {
        if (!p.table) return small ? launch_tc<128, kPacked, true>(p, grid, st) : launch_tc<128, kPacked, false>(p, grid, st);
        if (page_box(p.page_size) == 16)
            return small ? launch_tc<128, kPages16, true>(p, grid, st) : launch_tc<128, kPages16, false>(p, grid, st);
        return small ? launch_tc<128, kPages, true>(p, grid, st) : launch_tc<128, kPages, false>(p, grid, st);
    }
    if (!p.table) return small ? launch_tc<64, kPacked, true>(p, grid, st) : launch_tc<64, kPacked, false>(p, grid, st);
    return small ? launch_tc<64, kPages, true>(p, grid, st) : launch_tc<64, kPages, false>(p, grid, st);
}

}  // namespace sdv
