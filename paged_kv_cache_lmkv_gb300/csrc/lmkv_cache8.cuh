// lmkv_cache8.cuh -- pages of e4m3 codes with a power of two for each page and
// head: what the append and the attention share.
#pragma once

#include "lmkv_paged.cuh"

namespace lmkv_cache8 {

// One layer's scales, uint8 [2][num_blocks][kv_heads]: an element is code *
// 2^(byte - 127); a byte of 255 is NaN.
struct Scales {
    uint8_t* const* layer_base;     // DEVICE array; null: a 16-bit pool
    int32_t layer, kv_heads;
    int64_t num_blocks;

    __host__ static Scales of(const lmkv_pool_t* pool, void* const* scales, int32_t layer) {
        return Scales{reinterpret_cast<uint8_t* const*>(scales), layer, pool->num_kv_heads, pool->num_blocks};
    }
    __device__ __forceinline__ uint8_t* base() const { return layer_base[layer]; }
    __device__ __forceinline__ int64_t at(int kv, int64_t blk, int32_t h) const {
        return (kv * num_blocks + blk) * kv_heads + h;
    }
};

// 2^e for -149 <= e <= 127 (0 below), e = 128: NaN.
__device__ __forceinline__ float power_of_two(int e) {
    if (e >= 128) return __int_as_float(0x7FC00000);
    if (e >= -126) return __int_as_float((e + 127) << 23);
    return e >= -149 ? __int_as_float(1 << (e + 149)) : 0.f;
}

// Two codes (low byte first) as fp16, exactly.
__device__ __forceinline__ uint32_t codes_to_half2(uint16_t codes) {
    uint32_t w;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(w) : "h"(codes));
    return w;
}
// Two values as codes, lo in the low byte: to nearest even, beyond 448 to 448, NaN to NaN.
__device__ __forceinline__ uint16_t floats_to_codes(float lo, float hi) {
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
    return c;
}

// Scales come with an 8-bit pool and with no other.
inline int check_scales(const lmkv_pool_t* pool, void* const* scales, int32_t dtype) {
    if (dtype != LMKV_BF16 && dtype != LMKV_FP16) return LMKV_ERR_UNSUPPORTED;
    if (pool->elem_bytes != 1 && pool->elem_bytes != 2) return LMKV_ERR_UNSUPPORTED;
    if (pool->head_dim != 64 && pool->head_dim != 128) return LMKV_ERR_UNSUPPORTED;
    return (pool->elem_bytes == 1) == (scales != nullptr) ? LMKV_OK : LMKV_ERR_INVALID_ARG;
}

}  // namespace lmkv_cache8
