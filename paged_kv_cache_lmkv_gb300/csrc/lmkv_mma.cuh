// lmkv_mma.cuh -- warp-level pieces of the attention-side kernels: 16-byte
// asynchronous copies into swizzled shared memory, matrix fragments, and
// mma.sync products of 16 x 8 x 16 with fp32 accumulators.
#pragma once

#include "lmkv_paged.cuh"

namespace lmkv_mma {

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}

// 16 bytes global -> shared; zeros when !there (src is then not read).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
    const int n = there ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

template <class T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                                        uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 2^x: relative error at most 2^-22, 2^-inf = 0, NaN stays NaN.
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Byte offset of 16-byte piece `c` of row `r` in a tile of kRowBytes rows
// (128 or 256): pieces are exchanged within 128 bytes by the row number, so
// the eight rows an ldmatrix reads lie in different banks.
template <int kRowBytes>
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
    return (uint32_t)(r * kRowBytes + ((c ^ (r & 7)) << 4));
}

// Chunks of 16 cached tokens' rows of one head (K, or K and V) by one warp into
// its own shared memory, swizzled; rows that are not there are zeros.  In
// pages of a multiple of 16 tokens a chunk that begins at a multiple of 16
// lies in one page: its entry is fetched a chunk ahead, and a copy's address is
// an addition.
template <int D, bool kValues>
struct ChunkCopy {
    static constexpr int kRowBytes = D * 2;
    static constexpr int kVecs = kRowBytes / 16;
    static constexpr int kTileBytes = 16 * kRowBytes;
    static constexpr int kRowsPer = 32 / kVecs;
    static constexpr int kPatterns = 8 / kRowsPer;

    const lmkv_paged::Layer& layer;
    const int32_t* table;
    const uint8_t* base;         // the layer's K half
    const uint8_t* mine;         // with this lane's row and piece of a chunk of the head
    int64_t half_bytes;
    uint32_t row_bytes;
    int32_t end;                 // keys
    bool runs;
    uint32_t pattern[kPatterns];
    int32_t next_blk;

    __device__ __forceinline__ ChunkCopy(const lmkv_paged::Layer& l, const int32_t* t, const uint8_t* layer_base,
                                         int32_t head, int32_t last)
        : layer(l), table(t), base(layer_base), half_bytes(l.half_bytes()), row_bytes((uint32_t)l.row_bytes), end(last) {
        const int lane = threadIdx.x & 31, rsub = lane / kVecs, c = lane % kVecs;
        mine = base + (int64_t)head * kRowBytes + c * 16 + (int64_t)rsub * row_bytes;
        runs = l.block_size % 16 == 0;
#pragma unroll
        for (int k = 0; k < kPatterns; ++k) pattern[k] = swizzled<kRowBytes>(k * kRowsPer + rsub, c);
        next_blk = -1;
    }
    __device__ __forceinline__ void lookup(int32_t key0) {
        next_blk = runs && key0 < end ? table[layer.column(key0)] : -1;
    }
    // The chunk at key0 (looked up before) to dst; then looks up the one at
    // after.  Returns which of the 16 keys there are.
    __device__ __forceinline__ uint32_t copy(int32_t key0, uint32_t dst, int32_t after, int32_t* status) {
        const int lane = threadIdx.x & 31;
        const int32_t blk = next_blk;
        lookup(after);
        if (runs && key0 + 16 <= end && blk >= 0 && blk < layer.num_blocks) {
            const uint8_t* src = mine + (uint64_t)layer.row_of(blk, key0, layer.column(key0)) * row_bytes;
#pragma unroll
            for (int v = 0; v < kVecs / 2; ++v) {
                const uint32_t at = dst + pattern[v % kPatterns] + v / kPatterns * 8 * kRowBytes;
                cp_async16(at, src + v * (kRowsPer * row_bytes));
                if (kValues) cp_async16(at + kTileBytes, src + v * (kRowsPer * row_bytes) + half_bytes);
            }
            return 0xFFFFu;
        }
        const int32_t tok = key0 + (lane & 15);
        int64_t off = -1;
        if (tok < end) {
            off = layer.token_offset(table, tok);
            if (off < 0 && lane < 16) lmkv_paged::report(status, LMKV_ERR_BAD_BLOCK);
        }
        const uint32_t mask = __ballot_sync(0xFFFFFFFFu, off >= 0) & 0xFFFFu;
        const uint8_t* const piece = mine - (int64_t)(lane / kVecs) * row_bytes;
#pragma unroll
        for (int v = 0; v < kVecs / 2; ++v) {
            const int row = v * kRowsPer + lane / kVecs;
            const int64_t o = __shfl_sync(0xFFFFFFFFu, off, row);
            const uint32_t at = dst + pattern[v % kPatterns] + v / kPatterns * 8 * kRowBytes;
            const uint8_t* src = o >= 0 ? piece + o : base;
            cp_async16(at, src, o >= 0);
            if (kValues) cp_async16(at + kTileBytes, src + (o >= 0 ? half_bytes : 0), o >= 0);
        }
        return mask;
    }
};

// Two consecutive elements as one word (low half first); one load if `pairs`
// (4-byte aligned rows).
template <class T>
__device__ __forceinline__ uint32_t load_pair(const T* p, bool pairs) {
    if (pairs) return *reinterpret_cast<const uint32_t*>(p);
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
    return (uint32_t)h[0] | ((uint32_t)h[1] << 16);
}

}  // namespace lmkv_mma
