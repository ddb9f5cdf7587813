// What the tensor-core kernels of packed attention share: the tiles' ring, waits
// that give up, small wrappers, and the host side of their tensor maps.
#pragma once

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

// Of a tree's node with word `word` (vl_tree_word): which of the 64 keys from
// `from` past the tree's first position on it sees; those before that position all.
__device__ __forceinline__ uint64_t tree_seen(uint64_t word, int from) {
    if (from <= -64) return ~0ull;
    if (from < 0) return (word << -from) | ((1ull << -from) - 1);
    return from < 64 ? word >> from : 0ull;
}

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

int page_box(int page_size) {       // slots per copy: the largest power of two that divides the page, up to 128
    int b = 128;
    while (page_size % b) b >>= 1;
    return b;
}

}  // namespace
}  // namespace sdv
