// Runs the work plan of packed attention (varlen.cuh) on the host, the 32 lanes
// of a warp as coroutines that meet at every warp intrinsic, and checks how it
// deals out a batch.  Batches come on stdin, one after the other:
//   B Hkv G tensor causal prompt N max_q max_kv table_slots grid rows line_shift
//   cu_q[0 .. B]   kv_len[0 .. B-1] (not for prompts)
// with grid 0 for the default number of CTAs, rows 0 for the default form, and
// line_shift -1 for what the bounds ask for.  One line per batch on stdout:
//   fault word, length of the line, line_shift, CTAs with work, parts of tiles,
//   the most CTAs that share a unit, and "ok" or what is wrong.
#include <math.h>
#include <setjmp.h>
#include <ucontext.h>

#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <map>
#include <string>
#include <tuple>
#include <vector>

using std::max;
using std::min;

// ---- a warp
struct Lane { int x; };
static Lane lane_id;                      // the lane that runs
#define threadIdx lane_id
#ifndef __noinline__
#define __noinline__ __attribute__((noinline))
#endif
static jmp_buf at[33];                    // the lanes, and the main program
static ucontext_t start[32], home;
static bool begun[32];
static long exchange[32];

static void resume(int lane) {
    lane_id.x = lane;
    if (begun[lane]) _longjmp(at[lane], 1);
    begun[lane] = true;
    setcontext(&start[lane]);
}
// every lane up to here: the others run until they meet, in turn
static void __attribute__((noinline)) meet() {
    const int me = lane_id.x;
    if (_setjmp(at[me]) == 0) resume((me + 1) & 31);
}

template <class T> T __shfl_sync(unsigned, T v, int src) {
    exchange[lane_id.x] = (long)v;
    meet();
    const long r = exchange[src & 31];
    meet();
    return (T)r;
}
template <class T> T __shfl_up_sync(unsigned m, T v, int d) {
    return __shfl_sync(m, v, lane_id.x >= d ? lane_id.x - d : lane_id.x);
}
static unsigned __reduce_add_sync(unsigned, unsigned v) {
    exchange[lane_id.x] = v;
    meet();
    unsigned r = 0;
    for (long x : exchange) r += (unsigned)x;
    meet();
    return r;
}
static unsigned __ballot_sync(unsigned, bool p) {
    exchange[lane_id.x] = p;
    meet();
    unsigned r = 0;
    for (int i = 0; i < 32; ++i) r |= exchange[i] ? 1u << i : 0u;
    meet();
    return r;
}
static void __syncwarp() { meet(); }
static int __clz(int x) { return x ? __builtin_clz((unsigned)x) : 32; }
static int __popc(unsigned x) { return __builtin_popcount(x); }
static int __ffs(int x) { return __builtin_ffs(x); }
static unsigned atomicOr(unsigned *p, unsigned v) { const unsigned o = *p; *p |= v; return o; }
// named by functions that the plan does not call
template <class T> T __shfl_xor_sync(unsigned, T, int) { abort(); }
static bool __any_sync(unsigned, bool) { abort(); }
static unsigned atomicAdd(unsigned *, unsigned) { abort(); }
static unsigned atomicExch(unsigned *, unsigned) { abort(); }
static void __threadfence() { abort(); }
static float __uint_as_float(unsigned) { abort(); }
template <class T> T __ldcg(const T *) { abort(); }
template <class T> T __ldg(const T *) { abort(); }

#include "varlen.cuh"

using namespace sdv;

static VarlenParams P;
static int cta;
static VlPlan plan;
static VlEnds ends;

static void lane_main() {
    const VlPlan q = vl_plan(P, cta);
    vl_plan_store(q, &plan);
    if (!plan.idle) vl_ends(P, plan, cta, &ends);
    else ends.n = 0;
    meet();
    _longjmp(at[32], 1);                  // lane 0 is the first to come back
}

static void run_cta(int c) {
    static std::vector<char> stack(32 << 18);
    cta = c;
    memset(&plan, 0, sizeof plan);
    memset(&ends, 0, sizeof ends);
    for (int i = 0; i < 32; ++i) {
        begun[i] = false;
        getcontext(&start[i]);
        start[i].uc_stack.ss_sp = stack.data() + ((size_t)i << 18);
        start[i].uc_stack.ss_size = 1 << 18;
        start[i].uc_link = &home;
        makecontext(&start[i], lane_main, 0);
    }
    if (_setjmp(at[32]) == 0) resume(0);
}

struct Part { int t0, t1, c, tiles; };

static std::string check(int grid, long &parts, int &active, int &most) {
    std::map<std::tuple<int, int, int>, std::vector<Part>> dealt;
    std::vector<VlEnds> all((size_t)grid);
    char msg[200];
    auto wrong = [&](const char *what, int c, int b) {
        snprintf(msg, sizeof msg, "%s (CTA %d, sequence %d)", what, c, b);
        return std::string(msg);
    };
    for (int c = 0; c < grid; ++c) {
        run_cta(c);
        all[c] = ends;
        if (plan.idle) continue;
        ++active;
        VlWalk w(plan);
        VlUnit u;
        int shared = 0;
        while (w.next(P, plan, u)) {
            if (u.t1 < u.t0 || (u.t1 == u.t0 && u.tiles > 0)) return wrong("an empty part", c, u.b);
            dealt[{u.b, u.g, u.r}].push_back({u.t0, u.t1, c, u.tiles});
            ++parts;
            if (u.t0 == 0 && u.t1 == u.tiles) continue;
            // the kernels take the unit they begin in the middle of as the first, the one they leave as the last
            const int i = u.t0 > 0 ? 0 : ends.n - 1;
            if (i < 0 || ends.u[i].row0 != u.row0 || ends.u[i].g != u.g || ends.u[i].ntok != u.ntok ||
                (u.t0 == 0) != (ends.u[i].first == c))
                return wrong("a shared unit that is not among the ends", c, u.b);
            ++shared;
        }
        if (shared != ends.n) return wrong("ends that are no parts", c, plan.begin.b);
    }
    size_t units = 0;
    for (int b = 0; b < P.B; ++b) {
        const VlSeq s = vl_seq(P, b, false);
        for (int g = 0; g < P.Hkv; ++g)
            for (int r = 0; r < s.nr; ++r, ++units) {
                const auto f = dealt.find({b, g, r});
                if (f == dealt.end()) return wrong("a unit that nobody has", r, b);
                const auto &v = f->second;
                int t = 0, k = 0;
                const int n = (int)v.size();
                most = max(most, n);
                for (const Part &q : v) {
                    if (q.t0 != t) return wrong("tiles dealt twice or not at all", q.c, b);
                    t = q.t1;
                    if (n > 1) {
                        bool known = false;
                        for (int i = 0; i < all[q.c].n; ++i) {
                            const VlShared &e = all[q.c].u[i];
                            if (e.first != v[0].c || e.last != v[n - 1].c || e.n != n || e.s != k) continue;
                            known = true;
                            for (int c = e.first, j = 0; c <= e.last; ++c) {
                                const bool has = (e.mask[(c - e.base) >> 5] >> ((c - e.base) & 31)) & 1u;
                                if (has != (j < n && v[j].c == c)) known = false;
                                if (j < n && v[j].c == c) ++j;
                            }
                        }
                        if (!known) return wrong("a shared unit whose CTAs disagree", q.c, b);
                    }
                    ++k;
                }
                if (t != v[0].tiles) return wrong("a unit left unfinished", v[n - 1].c, b);
            }
    }
    if (units != dealt.size()) return wrong("units that are none", -1, -1);
    return "ok";
}

int main() {
    int B, Hkv, G, tensor, causal, prompt, N, max_q, max_kv, slots, grid, rows, shift;
    while (scanf("%d %d %d %d %d %d %d %d %d %d %d %d %d", &B, &Hkv, &G, &tensor, &causal, &prompt, &N, &max_q, &max_kv,
                 &slots, &grid, &rows, &shift) == 13) {
        std::vector<int> cu((size_t)B + 1), kv((size_t)B);
        for (int &x : cu) if (scanf("%d", &x) != 1) return 1;
        if (!prompt) for (int &x : kv) if (scanf("%d", &x) != 1) return 1;
        // as the host sets a call up
        static unsigned fault;
        fault = 0;
        memset(&P, 0, sizeof P);
        P.fault = &fault;
        P.B = B; P.Hkv = Hkv; P.Hq = Hkv * G; P.causal = causal;
        P.N = N; P.max_q = min(max_q, N); P.max_kv = max_kv;
        P.cu = cu.data();
        P.kv_len = prompt ? nullptr : kv.data();
        P.table_cols = slots / 8; P.page_size = 8;
        P.rows = rows ? rows : tensor ? kVarlenTcRows : (long)P.max_q * G <= 16 ? 16 : 64;
        P.tb = max(1, tensor ? 2 * (128 / G) : P.rows / G);
        P.tile_log2 = tensor ? kVarlenTcTileLog2 : kVarlenGenTileLog2;
        P.fixed = tensor ? kVarlenTcFixed : kVarlenGenFixed;
        P.group = tensor ? kVarlenTcGroup : kVarlenGenGroup;
        const double units = (double)Hkv * min((double)N / P.tb + B, (double)B * ((P.max_q + P.tb - 1) / P.tb));
        const double line = units * ((double)max(P.max_kv, P.max_q) + P.fixed);
        while (ldexp(line, -P.line_shift) > (double)kVarlenLine) ++P.line_shift;
        P.line_shift = max(P.line_shift, shift);
        P.min_share = max(1, (tensor ? kVarlenTcMinShare : kVarlenGenMinShare) >> P.line_shift);
        const int cap = tensor ? 152 : 4 * 152;
        if (!grid) grid = (int)max(1.0, min((double)cap, line / P.min_share + 1.0));
        P.inv_grid = 1.0f / (float)grid;
        if (P.fixed >> P.line_shift < 1) { printf("0 0 %d 0 0 0 refused\n", P.line_shift); continue; }
        long parts = 0;
        int active = 0, most = 0;
        const std::string what = check(grid, parts, active, most);
        run_cta(0);
        printf("%u %d %d %d %ld %d %s\n", fault, plan.total, P.line_shift, active, parts, most, what.c_str());
    }
    return 0;
}
