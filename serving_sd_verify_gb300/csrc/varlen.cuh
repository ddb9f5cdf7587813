// What the two kernels of packed (varlen) attention share: how the work of a
// ragged batch is divided, and how partial results are joined.
//
// Work.  Unit (b, g, r) is tokens [r tb, (r + 1) tb) of sequence b's new tokens
// for kv head g, with every query head that reads it; its keys are those its
// last token sees.  Units in the order (b, g, r) form one line whose length is
// counted in keys (a unit's visible keys plus a fixed cost); CTA c of n takes
// the c-th n-th of it, cut at whole key tiles.  So every CTA has the same load
// whatever the lengths are -- one token over a long cache, a causal prompt, a
// mixture -- and at most its first and its last unit are shared with its
// neighbours.  Lengths are read on the device, so the host needs only bounds;
// the whole plan costs a warp two passes over the sequences.
//
// Join.  A CTA that has only some of a unit's tiles leaves its weighted sums,
// running max and running sum in a slot of the workspace; when all n CTAs of
// the unit have arrived, each joins its n-th of the rows.  The order of the
// sum is the order of the tiles, whoever arrives when.
#pragma once

#include "common.cuh"

namespace sdv {
namespace {

struct VlSeq {
    int c0, q, kv;      // first packed row, new tokens, keys
    int off;            // causal: row i sees off + i + 1 keys
    int nr;             // units per kv head
};

__device__ __forceinline__ VlSeq vl_seq(const VarlenParams &p, int b, bool report) {
    VlSeq s;
    const int a = p.cu[b], e = p.cu[b + 1];
    const int len = p.kv_len ? p.kv_len[b] : 0;
    s.c0 = max(0, min(a, p.N));
    const int c1 = max(s.c0, min(e, p.N));
    s.q = min(c1 - s.c0, p.max_q);
    bool bad = a != s.c0 || e != s.c0 + s.q;
    if (p.kv_len) {
        const long slots = (long)p.table_cols * p.page_size;
        s.kv = max(0, (int)min((long)len, min((long)p.max_kv, slots)));
        bad = bad || s.kv != len;
    } else {
        s.kv = s.q;
    }
    if (bad && report) set_fault(p.fault, FAULT_BAD_LENGTH);
    s.off = s.kv - s.q;
    s.nr = s.q <= p.tb ? (s.q > 0 ? 1 : 0) : (int)((unsigned)(s.q + p.tb - 1) / (unsigned)p.tb);
    return s;
}

// keys the last token of unit r sees
__device__ __forceinline__ int vl_keys(const VarlenParams &p, const VlSeq &s, int r) {
    if (!p.causal) return s.kv;
    return max(0, s.off + min(s.q, (r + 1) * p.tb));
}

// Length of units [0, r) of one kv head on the work line, r <= nr, in keys >>
// line_shift: the exact sum, shifted, so that it never decreases with r.
__device__ __forceinline__ int vl_before(const VarlenParams &p, const VlSeq &s, int r) {
    if (r == 0) return 0;
    const int full = (p.causal ? max(s.kv, s.q) : s.kv) + p.fixed;   // the last unit's
    if (s.nr == 1) return full >> p.line_shift;
    long w = (long)r * full;
    if (p.causal) {
        const int r1 = r == s.nr ? r - 1 : r;      // units of tb tokens among them
        w = (long)r1 * (max(0, s.off) + p.fixed) + (long)p.tb * ((long)r1 * (r1 + 1) / 2);
        if (r == s.nr) w += full;
    }
    return (int)(w >> p.line_shift);
}

struct VlPos {          // a place on the work line: tile t of unit (b, g, r)
    int b, g, r, t;
    int x, len, tiles;  // where t > 0: the unit's beginning and length on the line, its tiles
    int row0, ntok;     // and its first packed row and tokens
};

struct VlUnit {
    int b, g, r;
    int row0, ntok;     // first packed row, tokens
    int tok0;           // the first one's number within the sequence
    int off, kv;
    int t0, t1, tiles;  // this CTA's tiles of all
};

// A unit shared by `n` CTAs: bit k of the mask is set where CTA base + k has a
// part (a share can fall between two cuts and have none).  The first opens the
// unit, this CTA's is the s-th.
struct VlShared {
    int base, first, last, n, s;
    int g, row0, ntok;
    unsigned mask[(kVarlenMaxGrid + 31) / 32];
};

struct VlPlan {
    int idle;
    VlPos begin, end;
    VlSeq s;            // the sequence of `begin`
    int share, total;   // CTA c takes [c share, (c + 1) share) of the line
    int group;          // and units are cut at multiples of this many tiles
};

__device__ __forceinline__ int vl_tiles(const VarlenParams &p, int keys) {
    return (keys + (1 << p.tile_log2) - 1) >> p.tile_log2;
}

// cut of a unit of length len and `tiles` tiles at `off` (0 <= off <= len): the
// tiles before it, in whole groups (a unit of p.group tiles or fewer is
// not cut); non-decreasing in off
__device__ __forceinline__ int vl_cut(const VarlenParams &p, int off, int len, int tiles, bool splittable, int group) {
    const int groups = (tiles + group - 1) / group;
    if (!splittable || tiles <= p.group) return 2 * off >= len ? tiles : 0;
    const int g = (int)((float)off * ((float)groups / (float)len) + 0.5f);
    return min(tiles, g * group);
}
__device__ __forceinline__ bool vl_splittable(const VarlenParams &p, const VlSeq &s) {
    return !p.causal || s.off >= 0;
}

// the place of boundary x, `o` past the beginning of sequence b's part of the line
__device__ __forceinline__ VlPos vl_locate(const VarlenParams &p, int b, const VlSeq &s, int x, int o, int group) {
    const int head = vl_before(p, s, s.nr);
    int g = min((int)((float)o / (float)head), p.Hkv - 1);     // at most 4096 heads: one off at most
    o -= g * head;
    if (o < 0) { --g; o += head; }
    else if (o >= head && g < p.Hkv - 1) { ++g; o -= head; }
    int r = 0, hi = s.nr - 1;                                  // the last unit that begins at or before o
    while (r < hi) {
        const int mid = (r + hi + 1) >> 1;
        if (vl_before(p, s, mid) <= o) r = mid;
        else hi = mid - 1;
    }
    const int u0 = vl_before(p, s, r), len = vl_before(p, s, r + 1) - u0;
    const int tiles = vl_tiles(p, vl_keys(p, s, r));
    int t = vl_cut(p, o - u0, len, tiles, vl_splittable(p, s), group);
    const VlPos in = {b, g, r, t, x - (o - u0), len, tiles, s.c0 + r * p.tb, min(p.tb, s.q - r * p.tb)};
    if (t < tiles || (tiles == 0 && 2 * (o - u0) < len)) return in;
    if (++r == s.nr) {                                         // at its end: the next unit's beginning
        r = 0;
        if (++g == p.Hkv) { g = 0; ++b; }
    }
    return {b, g, r, 0};
}

// The share of CTA `c` (one full warp).  The code runs once per CTA, so it is
// kept short: most of its time is instruction fetch.  The line's length stays
// within kVarlenLine (the host picks line_shift by its bounds); offsets that are
// no offsets (sequences that overlap) could exceed it and wrap the 32-bit sums,
// so the lengths' high bits are summed as well, each shifted before it is added,
// and where that is too large nothing is computed.
// Up to 32 sequences a lane holds one each.  More go in blocks of 32 whose
// lengths the lanes hold (32 blocks at a time), so that only the two blocks in
// which the share begins and ends are read again.
__device__ __forceinline__ VlPlan vl_plan(const VarlenParams &p, int c) {
    const int lane = threadIdx.x & 31;
    constexpr unsigned kAll = 0xffffffffu;
    constexpr int kHigh = 8;
    // what the shifts drop, 65,535 sequences' at most, does not carry a line past 2^31
    static_assert(kVarlenLine + 65536ll * (1 << kHigh) < (1ll << 31), "prefix sums in 32 bits");
    VlPlan pl = {};
    VlSeq s = {};
    unsigned w = 0, total = 0, coarse = 0;
    auto read = [&](int b, bool report) {
        w = 0;
        if (b < p.B) {
            s = vl_seq(p, b, report);
            w = (unsigned)p.Hkv * (unsigned)vl_before(p, s, s.nr);
        }
        return w;
    };
    auto scan = [&](unsigned v) {
        int e = (int)v;
#pragma unroll 1
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(kAll, e, d);
            if (lane >= d) e += y;
        }
        return e;
    };
    // the lengths of blocks s0 / 32 .. s0 / 32 + 31, one per lane
    auto blocks = [&](int s0, bool report) {
        unsigned mine = 0;
#pragma unroll 4
        for (int k = 0; k < 32; ++k) {
            const int b0 = s0 + 32 * k;
            if (b0 >= p.B) break;
            const unsigned t = __reduce_add_sync(kAll, read(b0 + lane, report));
            if (lane == k) mine = t;
            coarse = min(coarse + (w >> kHigh), 1u << 26);     // this lane's sequences'
        }
        return mine;
    };
    unsigned held = 0;
    if (p.B <= 32) {
        held = read(lane, c == 0);
        total = __reduce_add_sync(kAll, held);
        coarse = __reduce_add_sync(kAll, held >> kHigh);
    } else {
#pragma unroll 1
        for (int s0 = 0; s0 < p.B; s0 += 1024) {
            held = blocks(s0, c == 0);
            total += __reduce_add_sync(kAll, held);
        }
        coarse = __reduce_add_sync(kAll, coarse);
    }
    pl.total = (int)total;
    if (coarse > (unsigned)(kVarlenLine >> kHigh)) {
        if (c == 0 && lane == 0) set_fault(p.fault, FAULT_BAD_LENGTH);
        pl.total = 0;
    }
    // the smallest share the grid covers the line with (rounded up past fp32's error)
    pl.share = max(p.min_share, (int)((float)pl.total * p.inv_grid * (1.0f + 0x1p-20f)) + 1);
    // joining parts costs about what p.group tiles cost: a part this short is not worth it
    pl.group = pl.share > p.min_share ? 1 : p.group;
    const int x0 = c * pl.share, x1 = x0 + pl.share;
    pl.idle = x0 >= pl.total;
    if (pl.idle) return pl;
    // the sequences in which the share begins and ends: lane 0 then places the
    // beginning and lane 1 the end, side by side
    const int x = lane == 0 ? x0 : x1;
    int o = 0, found = p.B;
    // among 32 sequences from b0 whose first begins at `base`
    auto find = [&](int b0, int base) {
        const int e = base + (p.B > 1 ? scan(w) : (int)w), a = e - (int)w;
        const unsigned ms = __ballot_sync(kAll, x0 >= a && x0 < e), me = __ballot_sync(kAll, x1 >= a && x1 < e);
        const unsigned m = lane == 0 ? ms : me;
        const int src = __ffs((int)m) - 1;         // -1 where there is none: lane 31, not used
        VlSeq t;
        t.c0 = __shfl_sync(kAll, s.c0, src);
        t.q = __shfl_sync(kAll, s.q, src);
        t.kv = __shfl_sync(kAll, s.kv, src);
        t.nr = __shfl_sync(kAll, s.nr, src);
        const int ta = __shfl_sync(kAll, a, src);
        if (m && found == p.B) {
            t.off = t.kv - t.q;
            pl.s = t;
            o = x - ta;
            found = b0 + src;
        }
    };
    if (p.B <= 32) {
        find(0, 0);
    } else {
        int base = 0;
#pragma unroll 1
        for (int s0 = 0; s0 < p.B; s0 += 1024) {
            if (p.B > 1024) held = blocks(s0, false);
            const int e = base + scan(held), a = e - (int)held;
            unsigned at = __ballot_sync(kAll, x0 >= a && x0 < e) | __ballot_sync(kAll, x1 >= a && x1 < e);
            while (at) {                           // one block or two
                const int k = __ffs((int)at) - 1;
                at &= at - 1;
                read(s0 + 32 * k + lane, false);
                find(s0 + 32 * k, __shfl_sync(kAll, a, k));
            }
            base = __shfl_sync(kAll, e, 31);
            if (x1 < base) break;
        }
    }
    VlPos at = {p.B, 0, 0, 0};
    if (lane < 2 && found < p.B) at = vl_locate(p, found, pl.s, x, o, pl.group);
    if (at.b != found) pl.s.nr = 0;   // the next sequence's beginning: not yet read
    pl.begin = at;      // lane 0's; lane 1 holds the end
    pl.end = at;
    return pl;
}

// writes the plan that lanes 0 and 1 hold
__device__ __forceinline__ void vl_plan_store(const VlPlan &q, VlPlan *to) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) {
        to->idle = q.idle;
        to->begin = q.begin;
        to->s = q.s;
        to->share = q.share;
        to->total = q.total;
        to->group = q.group;
    } else if (lane == 1) {
        to->end = q.end;
    }
    __syncwarp();
}

// Walks a CTA's units in order; every warp role runs its own copy.
struct VlWalk {
    VlPos at;
    VlSeq s;
    bool fresh;         // s is that of at.b

    __device__ __forceinline__ explicit VlWalk(const VlPlan &pl) : at(pl.begin), s(pl.s), fresh(pl.s.nr > 0) {}

    __device__ __forceinline__ bool next(const VarlenParams &p, const VlPlan &pl, VlUnit &u) {
        for (;;) {
            if (at.b >= p.B) return false;
            if (at.b == pl.end.b && at.g == pl.end.g && at.r == pl.end.r && at.t >= pl.end.t) return false;
            if (at.b > pl.end.b) return false;
            if (!fresh) { s = vl_seq(p, at.b, false); fresh = true; }
            if (s.nr == 0) {
                ++at.b; at.g = at.r = at.t = 0; fresh = false;
                continue;
            }
            u.b = at.b; u.g = at.g; u.r = at.r;
            u.tok0 = at.r * p.tb;
            u.row0 = s.c0 + u.tok0;
            u.ntok = min(p.tb, s.q - u.tok0);
            u.off = s.off;
            u.kv = s.kv;
            u.tiles = vl_tiles(p, vl_keys(p, s, at.r));
            u.t0 = at.t;
            const bool last = at.b == pl.end.b && at.g == pl.end.g && at.r == pl.end.r;
            u.t1 = last ? pl.end.t : u.tiles;
            if (last) {
                at.t = pl.end.t;                 // next() ends here
            } else {
                at.t = 0;
                if (++at.r == s.nr) { at.r = 0; ++at.g; }
                if (at.g == p.Hkv) { at.g = 0; ++at.b; fresh = false; }
            }
            return true;
        }
    }
};

// keys that token i (within the sequence) of the unit sees
__device__ __forceinline__ int vl_limit(const VarlenParams &p, const VlUnit &u, int i) {
    return p.causal ? max(0, min(u.kv, u.off + i + 1)) : u.kv;
}

// the units that CTA c shares with others (one full warp): the one its share
// begins in the middle of, and the one it opens and leaves unfinished
struct VlEnds {
    int n;              // 0 to 2
    VlShared u[2];
};
__device__ void vl_ends(const VarlenParams &p, const VlPlan &pl, int c, VlEnds *to) {
    const int lane = threadIdx.x & 31;
    const bool same = pl.begin.b == pl.end.b && pl.begin.g == pl.end.g && pl.begin.r == pl.end.r;
    int found = 0;
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
        const VlPos at = i == 0 ? pl.begin : pl.end;
        if (at.t == 0 || (i == 1 && same && pl.begin.t > 0)) continue;
        if (same && pl.begin.t == pl.end.t) continue;       // between two boundaries cut alike: no part
        // (a unit that is cut is one that can be)
        auto cut = [&](int k) {       // tiles of the unit before boundary k
            const int x = k * pl.share;
            if (x <= at.x) return 0;
            if (x >= at.x + at.len || x >= pl.total) return at.tiles;
            return vl_cut(p, x - at.x, at.len, at.tiles, true, pl.group);
        };
        VlShared *r = to->u + found++;
        const int k0 = at.x / pl.share, k1 = min((at.x + at.len) / pl.share + 1, k0 + kVarlenMaxGrid);
        int first = -1, last = -1, n = 0, mine = 0;
#pragma unroll 1
        for (int k = k0; k < k1; k += 32) {
            const unsigned m = __ballot_sync(0xffffffffu, k + lane < k1 && cut(k + lane) < cut(k + lane + 1));
            if (first < 0 && m) first = k + __ffs((int)m) - 1;
            if (m) last = k + 31 - __clz((int)m);
            n += __popc(m);
            const int below = c - k;
            mine += below >= 32 ? __popc(m) : below > 0 ? __popc(m & ((1u << below) - 1u)) : 0;
            if (lane == 0) r->mask[(k - k0) >> 5] = m;
        }
        if (lane == 0) {
            r->base = k0;
            r->first = first;
            r->last = last;
            r->n = n;
            r->s = mine;
            r->g = at.g;
            r->row0 = at.row0;
            r->ntok = at.ntok;
        }
    }
    if (lane == 0) to->n = found;
    __syncwarp();
}

// Bounded wait until the counter reaches `target`.
__device__ __noinline__ bool vl_wait(const unsigned int *ctr, unsigned int target, unsigned long long limit_ns) {
    unsigned long long t0, t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    for (uint32_t it = 0;; ++it) {
        unsigned int v;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(ctr) : "memory");
        if (v >= target) return true;
        if ((it & 15u) == 15u) {
            asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
            if (t - t0 > limit_ns) return false;
        }
    }
}

// Four output values of one row, in the output's type.
__device__ __forceinline__ void vl_store4(const VarlenParams &p, long row, int c4, float4 o) {
    if (p.dt == SD_BF16) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(o.x, o.y), b = __floats2bfloat162_rn(o.z, o.w);
        uint2 w;
        w.x = *reinterpret_cast<const uint32_t *>(&a);
        w.y = *reinterpret_cast<const uint32_t *>(&b);
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + row * p.D + 4 * c4) = w;
    } else {
        *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + row * p.D + 4 * c4) = o;
    }
}

__device__ __forceinline__ float vl_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Joins this CTA's n-th of a shared unit's rows (`nt` threads, numbered by
// `tid`, that meet at barrier `bar`).  Row k of the
// unit is query head k % G of token k / G; in a slot the first `tpt` tokens'
// rows begin at 0 and the others' at `trows`.  Where a CTA has fewer items than threads, `lanes` threads share an item's parts, each taking every lanes-th,
// and combine by shuffles: always in the same order.
__device__ void vl_join(const VarlenParams &p, const VlShared &sh, int tpt, int trows, int *flag, int tid, int nt,
                        int bar) {
    auto meet = [&] { asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(nt) : "memory"); };
    unsigned int *ctr = p.ctr + sh.first;
    unsigned int ticket = 0;
    if (tid == 0) {
        const bool ok = vl_wait(ctr, (unsigned)sh.n + p.wt.extra, p.wt.limit_ns);
        if (!ok) set_fault(p.fault, FAULT_WAIT_TIMEOUT);
        *flag = ok;
        // second ticket, whether or not the wait succeeded: the CTA with the last
        // of the 2 n increments returns the counter to zero (nobody reads it then)
        ticket = atomicAdd(ctr, 1u);
    }
    meet();
    if (*flag) {
        // an item: 8 columns of a row; rows fastest, as the slots hold them
        const int G = p.Hq / p.Hkv, R = sh.ntok * G, items = R * (p.D / 8);
        const int ia = sh.s * items / sh.n, ie = (sh.s + 1) * items / sh.n;   // at most 1024 * 64 * 16
        int lanes = 1;
        while (lanes < 32 && 2 * lanes <= sh.n && (ie - ia) * lanes * 2 <= nt) lanes *= 2;
        const int sub = tid & (lanes - 1);
        const bool holes = sh.last - sh.first + 1 > sh.n;
        const long cstep = p.rows, sstep = (long)(p.D / 4) * p.rows;
        // kJoinItems items and kJoinParts parts of each at a time, so that their loads
        // are in flight together; the loops run the same number of times in every
        // thread, so that whole warps meet at the shuffles
        constexpr int kJoinItems = 2, kJoinParts = 4;
        const int stride = nt / lanes;
#pragma unroll 1
        for (int i0 = ia + tid / lanes; __any_sync(0xffffffffu, i0 < ie); i0 += kJoinItems * stride) {
            float M[kJoinItems], l[kJoinItems], acc[kJoinItems][8];
            int c8[kJoinItems], kr[kJoinItems];
            const float4 *src[kJoinItems];
            const float2 *mls[kJoinItems];
#pragma unroll
            for (int q = 0; q < kJoinItems; ++q) {
                const unsigned i = (unsigned)min(i0 + q * stride, items - 1);
                c8[q] = (int)(i / (unsigned)R);
                kr[q] = (int)i - c8[q] * R;
                const int row = kr[q] < tpt * G ? kr[q] : trows + kr[q] - tpt * G;
                src[q] = reinterpret_cast<const float4 *>(p.o_part) + 2 * c8[q] * cstep + row;
                mls[q] = p.ml_part + row;
                M[q] = -INFINITY;
                l[q] = 0.f;
#pragma unroll
                for (int x = 0; x < 8; ++x) acc[q][x] = 0.f;
            }
#pragma unroll 1
            for (int k0 = sh.first + sub; k0 <= sh.last; k0 += kJoinParts * lanes) {
                float4 va[kJoinItems][kJoinParts], vb[kJoinItems][kJoinParts];
                float2 ml[kJoinItems][kJoinParts];
#pragma unroll
                for (int e = 0; e < kJoinParts; ++e) {
                    const int k = k0 + e * lanes;
                    const bool part = k <= sh.last &&
                                      (!holes || ((sh.mask[(k - sh.base) >> 5] >> ((k - sh.base) & 31)) & 1u));
                    const long slot = k == sh.first ? 2L * k + 1 : 2L * k;
#pragma unroll
                    for (int q = 0; q < kJoinItems; ++q) {
                        const bool live = part && i0 + q * stride < ie;
                        va[q][e] = live ? __ldcg(src[q] + slot * sstep) : make_float4(0.f, 0.f, 0.f, 0.f);
                        vb[q][e] = live ? __ldcg(src[q] + slot * sstep + cstep) : make_float4(0.f, 0.f, 0.f, 0.f);
                        ml[q][e] = live ? __ldcg(mls[q] + slot * p.rows) : make_float2(-INFINITY, 0.f);
                    }
                }
#pragma unroll
                for (int q = 0; q < kJoinItems; ++q) {
                    float m = M[q];
#pragma unroll
                    for (int e = 0; e < kJoinParts; ++e) m = fmaxf(m, ml[q][e].x);
                    const float ref = m == -INFINITY ? 0.f : m;
                    const float f = vl_ex2(M[q] - ref);                // 0 for what saw nothing
                    M[q] = m;
                    l[q] *= f;
#pragma unroll
                    for (int x = 0; x < 8; ++x) acc[q][x] *= f;
#pragma unroll
                    for (int e = 0; e < kJoinParts; ++e) {
                        const float w = vl_ex2(ml[q][e].x - ref);
                        const float v[8] = {va[q][e].x, va[q][e].y, va[q][e].z, va[q][e].w,
                                            vb[q][e].x, vb[q][e].y, vb[q][e].z, vb[q][e].w};
                        l[q] = fmaf(w, ml[q][e].y, l[q]);
#pragma unroll
                        for (int x = 0; x < 8; ++x) acc[q][x] = fmaf(w, v[x], acc[q][x]);
                    }
                }
            }
#pragma unroll
            for (int q = 0; q < kJoinItems; ++q) {
                if (!__any_sync(0xffffffffu, i0 + q * stride < ie)) break;
#pragma unroll 1
                for (int o = 1; o < lanes; o <<= 1) {
                    const float M2 = __shfl_xor_sync(0xffffffffu, M[q], o), l2 = __shfl_xor_sync(0xffffffffu, l[q], o);
                    const float m = fmaxf(M[q], M2), ref = m == -INFINITY ? 0.f : m;
                    const float f1 = vl_ex2(M[q] - ref), f2 = vl_ex2(M2 - ref);
                    l[q] = f1 * l[q] + f2 * l2;
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        acc[q][x] = f1 * acc[q][x] + f2 * __shfl_xor_sync(0xffffffffu, acc[q][x], o);
                    M[q] = m;
                }
                if (i0 + q * stride < ie && sub == 0) {
                    const float inv = l[q] > 0.f ? 1.f / l[q] : 0.f;
                    const int tok = (int)((unsigned)kr[q] / (unsigned)G);
                    const long orow = (long)(sh.row0 + tok) * p.Hq + sh.g * G + (kr[q] - tok * G);
                    vl_store4(p, orow, 2 * c8[q],
                              make_float4(acc[q][0] * inv, acc[q][1] * inv, acc[q][2] * inv, acc[q][3] * inv));
                    vl_store4(p, orow, 2 * c8[q] + 1,
                              make_float4(acc[q][4] * inv, acc[q][5] * inv, acc[q][6] * inv, acc[q][7] * inv));
                }
            }
        }
    }
    if (tid == 0 && ticket == 2u * (unsigned)sh.n - 1u) atomicExch(ctr, 0u);
    meet();
}

// announces this CTA's part of a shared unit (one thread, after a barrier that
// follows every thread's writes of it)
__device__ __forceinline__ void vl_arrive(const VarlenParams &p, const VlShared &sh) {
    __threadfence();
    asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p.ctr + sh.first) : "memory");
}

}  // namespace
}  // namespace sdv
