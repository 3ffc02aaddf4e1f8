// lmkv_tcgen05.cuh -- the fifth-generation tensor core from one CTA: mbarriers
// with bounded waits, tensor memory, shared-memory operand descriptors and
// tcgen05.mma of 128 x N x 16 on 16-bit types with fp32 accumulators.
#pragma once

#include <type_traits>

#include "lmkv_mma.cuh"

namespace lmkv_tc {

// ---- mbarriers ----------------------------------------------------------
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// One arrival once this thread's asynchronous copies so far have landed.
__device__ __forceinline__ void mbar_arrive_copies(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ uint64_t now_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
// Waits for the phase of this parity, at most a second (or until another
// thread of the CTA gave up).  False: gave up; every role then leaves its loop.
// The clock is read once in kPolls polls: reading it takes longer than the
// waits of a running pipeline do.
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr int kPolls = 512;
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* gave_up) {
    if (mbar_test(bar, parity)) return true;
    uint64_t t0 = 0;
    while (true) {
#pragma unroll 1
        for (int i = 0; i < kPolls; ++i)
            if (mbar_test(bar, parity)) return true;
        const uint64_t t = now_ns();
        if (t0 == 0) t0 = t;
        if (*gave_up || t - t0 > kWaitNs) {
            *gave_up = 1;
            return false;
        }
    }
}

__device__ __forceinline__ void fence_async_shared() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ---- tensor memory ------------------------------------------------------
template <int kColumns>
__device__ __forceinline__ void tmem_alloc(uint32_t smem_result) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_result), "n"(kColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
template <int kColumns>
__device__ __forceinline__ void tmem_free(uint32_t tmem) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kColumns) : "memory");
}
__device__ __forceinline__ void fence_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of this warp's 32 lanes: register i is column i of the thread's lane.
__device__ __forceinline__ void tmem_ld32(uint32_t (&r)[32], uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// After wait_ld: what was loaded may be used from here on.
__device__ __forceinline__ void loaded(uint32_t (&r)[32]) {
#pragma unroll
    for (int i = 0; i < 32; i += 8)
        asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                     "+r"(r[i + 6]), "+r"(r[i + 7]));
}
// The same of 16 columns: load, multiply by f, store.
__device__ __forceinline__ void tmem_scale16(uint32_t addr, float f) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr) : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
    tmem_st16(addr, r);
}

// ---- products -----------------------------------------------------------
// Shared-memory tiles are kept as [column half of 64 elements][row][128 bytes],
// the eight 16-byte pieces of a row exchanged by the row number (128-byte
// swizzle): atoms of 8 rows x 128 bytes, 1024-byte aligned.
// An operand's descriptor, as its two words: the low one holds the address
// (in 16 bytes) and the lead offset, so a step along the tile is one addition.
struct Desc {
    uint32_t lo, hi;
    __device__ __forceinline__ Desc at(uint32_t bytes) const { return Desc{lo + (bytes >> 4), hi}; }
};
__device__ __forceinline__ Desc smem_desc(uint32_t addr, uint32_t lead_bytes, uint32_t stride_bytes) {
    return Desc{((addr & 0x3FFFF) >> 4) | ((lead_bytes >> 4) << 16), (stride_bytes >> 4) | (1u << 14) | (2u << 29)};
}
// Rows of the tile are the operand's M or N, columns its K.
__device__ __forceinline__ Desc desc_k_major(uint32_t addr) { return smem_desc(addr, 16, 1024); }
// Rows of the tile are the operand's K, columns its N (half_bytes from one
// half of 64 columns to the next).
__device__ __forceinline__ Desc desc_n_major(uint32_t addr, uint32_t half_bytes) {
    return smem_desc(addr, half_bytes, 1024);
}
// A tile of 16 columns without swizzle: groups of 8 rows, in each the first 8
// columns of its rows (16 bytes a row), then the other 8.
__device__ __forceinline__ uint32_t plain16_offset(int row, int piece) {
    return (uint32_t)((row >> 3) * 256 + piece * 128 + (row & 7) * 16);
}
__device__ __forceinline__ Desc desc_plain16(uint32_t addr) {
    return Desc{((addr & 0x3FFFF) >> 4) | ((128u >> 4) << 16), (256u >> 4) | (1u << 14)};
}
// Instruction descriptor: fp32 accumulator, A and B of one 16-bit type.
template <class T, int kN, bool kBNMajor>
__device__ __forceinline__ constexpr uint32_t instr_desc() {
    const uint32_t type = sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
    return (1u << 4) | (type << 7) | (type << 10) | ((kBNMajor ? 1u : 0u) << 16) | ((uint32_t)(kN >> 3) << 17) |
           ((uint32_t)(128 >> 4) << 24);
}
// The products are issued by one thread.  The whole warp runs through the
// issuing code, so that descriptors are computed once a warp (in uniform
// registers, where the instruction wants them), and `lead` (one lane's true)
// predicates the instruction alone.
__device__ __forceinline__ uint32_t elect_lead() {
    uint32_t lead;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(lead));
    return lead;
}
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, Desc a, Desc b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.u32 p, %6, 0;\n\tsetp.ne.u32 q, %7, 0;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
        "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"((uint32_t)add), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, Desc b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
        "setp.ne.u32 p, %5, 0;\n\tsetp.ne.u32 q, %6, 0;\n\tmov.b64 b, {%2, %3};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"((uint32_t)add), "r"(lead)
        : "memory");
}
// The barrier's next arrival is when all products issued by this thread so far are done.
__device__ __forceinline__ void mma_commit(uint32_t lead, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(lead)
        : "memory");
}

__device__ __forceinline__ void bar_sync(int id, int threads) {
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// The largest of three (a NaN gives way to a number).
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// ---- pairs of fp32 ------------------------------------------------------
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

}  // namespace lmkv_tc
