// Device helpers of the attention kernels: barriers with bounded waits, asynchronous copies, tensor
// memory and the 16-bit matrix instruction (tcgen05, kind::f16).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "elem.h"

namespace uvu {
namespace tc {

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return uint32_t(__cvta_generic_to_shared(p)); }

// A value that is the same in all lanes, as the compiler can see it too: addresses, loop bounds and descriptors
// formed from it stay in uniform registers.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __reduce_or_sync(0xffffffffu, x); }
__device__ __forceinline__ int uniform(int x) { return int(uniform(uint32_t(x))); }

// ---------------------------------------------------------------------------------- barriers

__device__ __forceinline__ void bar_init(uint32_t b, uint32_t n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(b), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t b) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(b) : "memory");
}
__device__ __forceinline__ bool bar_test(uint32_t b, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(b), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ unsigned long long timer_ns() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
// The same, asleep for up to 20 us where the phase has not ended: a polling warp takes issue slots from
// the others (a third of all instructions, before).
__device__ __forceinline__ bool bar_sleep(uint32_t b, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(b), "r"(parity), "r"(20000u)
        : "memory");
    return ok != 0;
}
// Waits for the phase of `parity` to end.  False when another role has given up (*dead) or after
// about two seconds, which sets *dead and the status word; the caller then leaves its loop.  The global
// timer is far away (a read costs as much as several matrix instructions), so it is looked at rarely.
static __device__ __noinline__ bool bar_wait_slow(uint32_t b, uint32_t parity, volatile int* dead, unsigned* status) {
    unsigned long long t0 = 0;
    for (;;) {
        for (int i = 0; i < 64; ++i) {
            if (bar_sleep(b, parity)) return true;
            if (*dead) return false;
        }
        const unsigned long long now = timer_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > 2000000000ull) {
            *dead = 1;
            atomicOr(status, 1u);
            return false;
        }
    }
}
// The last wait before a role returns what others still use: bounded, whatever *dead says.
static __device__ __noinline__ void bar_wait_last(uint32_t b, uint32_t parity, unsigned* status) {
    unsigned long long t0 = 0;
    for (;;) {
        for (int i = 0; i < 64; ++i)
            if (bar_sleep(b, parity)) return;
        const unsigned long long now = timer_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > 2000000000ull) {
            atomicOr(status, 1u);
            return;
        }
    }
}
__device__ __forceinline__ bool bar_wait(uint32_t b, uint32_t parity, volatile int* dead, unsigned* status) {
    return bar_test(b, parity) || bar_wait_slow(b, parity, dead, status);
}
// By a whole warp.
__device__ __forceinline__ bool warp_wait(uint32_t b, uint32_t parity, volatile int* dead, unsigned* status) {
    return __all_sync(0xffffffffu, bar_wait(b, parity, dead, status));
}

// ------------------------------------------------------------------------------------- copies

// 16 bytes to shared memory, of which the first `bytes` are read and the others are zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// The barrier gets this thread's arrival when its copies issued so far have landed.
__device__ __forceinline__ void copy_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void copy_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// Ordinary and cp.async writes to shared memory that this thread has seen come before its matrix instructions.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// --------------------------------------------------------------------------- operand tiles

// An operand tile is [rows][64 columns] panels of 16-bit values: 128 bytes a row, groups of 8 rows
// (1024 bytes), the 16-byte chunk index XORed with the row within its group (128-byte swizzle).
// One panel of 128 rows is 16 KB; wider tiles are panels one after the other.
constexpr int kPanelBytes = 16384;
__device__ __forceinline__ uint32_t tile_offset(int row, int chunk) {  // chunk: 8 columns
    return uint32_t((chunk >> 3) * kPanelBytes + (row >> 3) * 1024 + (row & 7) * 128 + (((chunk ^ row) & 7) << 4));
}

// Shared-memory descriptors.  The lower word is the start address and the panel stride in units of 16
// bytes; the upper one the stride of 8-row groups (1024 bytes), version bits and the 128-byte swizzle.
// Tiles begin on 1024 bytes, so a step inside one is an addition to the lower word.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint64_t desc_of(uint32_t low) { return (uint64_t(kDescHigh) << 32) | low; }
// The tile's columns are the summed index (16 of them, beginning at column 16 k).  `panel`: bytes of a panel.
__device__ __forceinline__ uint64_t desc_cols(uint32_t tile, int k, int panel = kPanelBytes) {
    return desc_of((tile >> 4) + uint32_t(((k >> 2) * panel + (k & 3) * 32) >> 4) + (1u << 16));
}
// The tile's rows are the summed index (16 of them, beginning at row 16 k); panels of 64 columns are
// `panel` bytes apart.  col: first column; columns from a col that is not a multiple of 64 must end within
// its panel.
__device__ __forceinline__ uint64_t desc_rows(uint32_t tile, int k, int panel = kPanelBytes, int col = 0) {
    return desc_of((tile >> 4) + uint32_t((k * 2048 + (col >> 6) * panel + (col & 63) * 2) >> 4) + (uint32_t(panel >> 4) << 16));
}

// Instruction descriptor of kind::f16 with fp32 sums: M = 128, N = n; B's rows (true) or columns are the summed index.
template <typename T>
__device__ __forceinline__ uint32_t mma_desc(int n, bool b_rows) {
    constexpr uint32_t type = sizeof(T) == 2 && __is_same(T, __nv_bfloat16) ? 1u : 0u;
    return (1u << 4) | (type << 7) | (type << 10) | (uint32_t(b_rows) << 16) | (uint32_t(n >> 3) << 17) | (8u << 24);
}

// ------------------------------------------------------------------------------- tensor cores

// The issuing warp runs whole, so that addresses and descriptors stay in uniform registers, and one
// elected lane issues: with one lane alone in a branch, forming the operands cost twice the time of the products.
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
    return r;
}
// D (tensor memory) = [D +] A B, A from shared memory (SS) or tensor memory (TS).
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool add) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %3, 0;\n setp.ne.b32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %4, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(uint32_t(add)), "r"(id), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool add) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %3, 0;\n setp.ne.b32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %4, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(uint32_t(add)), "r"(id), "r"(lead)
        : "memory");
}
// The barrier gets an arrival when all matrix instructions issued so far are done.
__device__ __forceinline__ void mma_commit(uint32_t lead, uint32_t bar) {
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
        " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar),
        "r"(lead)
        : "memory");
}
__device__ __forceinline__ void tmem_alloc(uint32_t dst, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// The loads into r are done.  The registers pass through the wait, so that no use can be moved before it.
__device__ __forceinline__ void tmem_wait_ld(float (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]), "+f"(r[8]),
                   "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15])::"memory");
    asm volatile("" : "+f"(r[16]), "+f"(r[17]), "+f"(r[18]), "+f"(r[19]), "+f"(r[20]), "+f"(r[21]), "+f"(r[22]), "+f"(r[23]),
                      "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27]), "+f"(r[28]), "+f"(r[29]), "+f"(r[30]), "+f"(r[31])
                 ::"memory");
}
__device__ __forceinline__ void tmem_wait_ld(float (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]), "+f"(r[8]),
                   "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15])::"memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of the warp's 32 lanes (lane = row), as fp32.
__device__ __forceinline__ void tmem_ld32(uint32_t a, float (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
          "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
          "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(a));
}
__device__ __forceinline__ void tmem_ld8(uint32_t a, float (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
                 : "r"(a));
}
__device__ __forceinline__ void tmem_wait_ld(float (&r)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7])::"memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t a, float (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
        : "r"(a));
}
__device__ __forceinline__ void tmem_st8(uint32_t a, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(a), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(a),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t a, const float (&r)[16]) {
    uint32_t u[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(r[i]);
    tmem_st16(a, u);
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
using uvu::pack2;

}  // namespace tc
}  // namespace uvu
