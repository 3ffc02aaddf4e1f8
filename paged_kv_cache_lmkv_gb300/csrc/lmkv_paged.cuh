// lmkv_paged.cuh -- what the attention-side operators share: one layer of the
// pool as the kernels see it, ragged batches, and the launch.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "lmkv.h"
#include "lmkv_internal.h"

namespace lmkv_paged {

__device__ __forceinline__ void pdl_launch_dependents() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// x / d for 0 <= x < 2^31 by a multiplication: with s = ceil(log2 d) and
// m = ceil(2^(31+s) / d) the product's error is below 1/d for every such x
// (Granlund and Montgomery, "Division by Invariant Integers using
// Multiplication", 1994).
struct FastDiv {
    uint32_t d, m, s;
    __host__ __device__ FastDiv() : d(1), m(0), s(0) {}
    __host__ explicit FastDiv(uint32_t dv) : d(dv), m(0), s(0) {
        while ((1ull << s) < dv) ++s;
        if (dv > 1) m = (uint32_t)(((1ull << (31 + s)) + dv - 1) / dv);
    }
    __device__ __forceinline__ uint32_t div(uint32_t x) const {
        return d == 1 ? x : __umulhi(x, m) >> (s - 1);
    }
};

// One layer of the pool.
struct Layer {
    const uint8_t* const* layer_base;   // DEVICE array; entry `layer` is this layer's base
    int32_t layer;
    int32_t block_size;
    int64_t num_blocks;
    int64_t row_bytes;                  // num_kv_heads * head_dim * elem_bytes
    FastDiv by_block;

    __host__ static Layer of(const lmkv_pool_t* pool, int32_t layer) {
        Layer l;
        l.layer_base = reinterpret_cast<const uint8_t* const*>(pool->layer_base);
        l.layer = layer;
        l.block_size = pool->block_size;
        l.num_blocks = pool->num_blocks;
        l.row_bytes = (int64_t)pool->num_kv_heads * pool->head_dim * pool->elem_bytes;
        l.by_block = FastDiv((uint32_t)pool->block_size);
        return l;
    }
    // Bytes from a layer's K half to its V half.
    __device__ __forceinline__ int64_t half_bytes() const { return num_blocks * block_size * row_bytes; }
    // The layer's base, or null (null or misaligned entry).
    __device__ __forceinline__ uint8_t* base() const {
        const uint8_t* b = layer_base[layer];
        return (reinterpret_cast<uintptr_t>(b) & 15) ? nullptr : const_cast<uint8_t*>(b);
    }
    // Byte offset in the K half of token `tok`'s row in table row `table`, or
    // -1 (the block id is out of range).
    __device__ __forceinline__ int64_t token_offset(const int32_t* table, int32_t tok) const {
        const uint32_t col = by_block.div((uint32_t)tok);
        const int64_t blk = table[col];
        if (blk < 0 || blk >= num_blocks) return -1;
        return (blk * block_size + (tok - (int32_t)(col * (uint32_t)block_size))) * row_bytes;
    }
    // The same in two steps, so that the table entry's load need not be waited
    // for at once: its place, then the row's number in the K half (below 2^32
    // in any memory: rows of 128 bytes and more), or kNoRow.
    __device__ __forceinline__ uint32_t column(int32_t tok) const { return by_block.div((uint32_t)tok); }
    __device__ __forceinline__ uint32_t row_of(int32_t blk, int32_t tok, uint32_t col) const {
        if (blk < 0 || blk >= num_blocks) return kNoRow;
        return (uint32_t)blk * (uint32_t)block_size + ((uint32_t)tok - col * (uint32_t)block_size);
    }
    static constexpr uint32_t kNoRow = 0xFFFFFFFFu;
};

__device__ __forceinline__ void report(int32_t* status, int code) {
    if (status != nullptr) atomicCAS(status, 0, code);
}

// A ragged batch as the kernels see it (lmkv_batch_t).
struct Seqs {
    const int32_t* q_start;
    const int32_t* kv_len;
    const int32_t* table;
    int32_t table_stride;
    int32_t num_req;
    int32_t num_tokens;
    int32_t max_new;
    int32_t max_kv_len;

    __host__ static Seqs of(const lmkv_batch_t* b) {
        return Seqs{b->q_start, b->kv_len, b->block_table, b->max_blocks, b->num_req, b->num_tokens,
                    b->max_new, b->max_kv_len};
    }
};

// One request: its rows and its cached tokens, clamped to the call's bounds.
struct Req {
    int32_t r;
    int32_t q0;       // first row
    int32_t n;        // new tokens
    int32_t len;      // cached tokens, new ones included
    bool ok;          // nothing was clamped
};

__device__ __forceinline__ Req load_req(const Seqs& s, int32_t r) {
    const int32_t a = s.q_start[r], b = s.q_start[r + 1], len = s.kv_len[r];
    Req q;
    q.r = r;
    q.q0 = min(max(a, 0), s.num_tokens);
    const int32_t end = min(max(b, q.q0), s.num_tokens);
    q.n = min(end - q.q0, s.max_new);
    q.len = min(max(len, 0), s.max_kv_len);
    q.ok = q.q0 == a && q.q0 + q.n == b && q.len == len;
    return q;
}

// The last request r of [0, num_req) with key(r) <= x, key ascending and
// key(0) <= x taken as given; called by a whole warp, 32 candidates a step.
template <class Key>
__device__ __forceinline__ int32_t find_request(int32_t num_req, int32_t x, Key key) {
    const int lane = threadIdx.x & 31;
    int32_t lo = 0, n = num_req;
    while (n > 1) {
        const int32_t step = (n + 31) >> 5;
        const int32_t at = lane * step;
        const bool below = at < n && (at == 0 || key(lo + at) <= x);
        const uint32_t votes = __ballot_sync(0xFFFFFFFFu, below);
        const int32_t k = 31 - __clz(votes);
        lo += k * step;
        n = min(step, n - k * step);
    }
    return lo;
}

// An equal share of a batch's cached tokens, in units (of some tokens; a
// request's last one may be short) counted over the requests in turn: units
// [all * part / parts, all * (part + 1) / parts).  Whatever the lengths are,
// CTAs that take a share each end together.  No share before the last ones is
// empty, so a request's units lie in shares that follow one another.
struct Share {
    int32_t r;          // request of the first unit
    int64_t first;      // that unit, counted from the request's first
    int64_t n;          // units
};
// Called by a whole warp, which goes over all requests; units(i): request i's.
template <class Units>
__device__ __forceinline__ Share find_share(int32_t num_req, int32_t part, int32_t parts, Units units) {
    const int lane = threadIdx.x & 31;
    int64_t all = 0;
    for (int32_t i = lane; i < num_req; i += 32) all += units(i);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, d);
    // fewer units than shares: one each, the last shares have none
    const int64_t use = min((int64_t)parts, all);
    Share x{0, 0, 0};
    if (part >= use) return x;
    const int64_t begin = all * part / use, end = all * (part + 1) / use;
    x.n = end - begin;
    int64_t before = 0;
    for (int32_t r0 = 0; r0 < num_req; r0 += 32) {
        const int32_t i = r0 + lane;
        const int64_t own = i < num_req ? (int64_t)units(i) : 0;
        int64_t upto = own;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(0xFFFFFFFFu, upto, d);
            if (lane >= d) upto += y;
        }
        upto += before;
        const uint32_t votes = __ballot_sync(0xFFFFFFFFu, begin < upto);
        if (votes != 0) {
            const int k = __ffs(votes) - 1;
            x.r = r0 + k;
            x.first = begin - __shfl_sync(0xFFFFFFFFu, upto - own, k);
            return x;
        }
        before = __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
    x.n = 0;      // not reached: begin < all
    return x;
}
// Units of a request's cached tokens; lengths of the request that had to be clamped are reported.
__device__ __forceinline__ int64_t units_of(const Seqs& s, int32_t i, int32_t unit, int32_t* status) {
    const Req q = load_req(s, i);
    if (!q.ok) report(status, LMKV_ERR_BAD_LENGTH);
    return (q.len + unit - 1) / unit;
}

// ---- element types ------------------------------------------------------
template <class T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
    static __device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __forceinline__ __nv_bfloat16 from_float(float x) { return __float2bfloat16_rn(x); }
    // Two values as one word, lo in the low half.
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        uint32_t w;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
        return w;
    }
};
template <>
struct Elem<__half> {
    static __device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
    static __device__ __forceinline__ __half from_float(float x) { return __float2half_rn(x); }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        uint32_t w;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
        return w;
    }
};
template <>
struct Elem<float> {
    static __device__ __forceinline__ float to_float(float x) { return x; }
    static __device__ __forceinline__ float from_float(float x) { return x; }
};

// ---- launch -------------------------------------------------------------
constexpr int32_t kSms = 152;

// Launch with programmatic stream serialization: every kernel here waits for
// its predecessors (griddepcontrol.wait) before it touches global memory.
template <class Kernel, class... Args>
int launch(Kernel kernel, int64_t grid, int threads, size_t smem, void* stream, int cluster, Args... args) {
    if (grid <= 0) return LMKV_OK;
    if (grid > INT32_MAX) return LMKV_ERR_INVALID_ARG;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cluster > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)cluster;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, args...);
    lmkv_internal_add_launches(1);
    return lmkv_internal_cuda_status(err);
}

// Raises a kernel's dynamic shared memory limit to kBytes, once per device (the
// first call, made outside any capture).
template <auto kKernel, int kBytes>
int allow_smem() {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    const cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return lmkv_internal_cuda_status(err);
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return LMKV_OK;
    const int rc = lmkv_internal_cuda_status(
        cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes));
    if (rc == LMKV_OK) done.fetch_or(bit, std::memory_order_relaxed);
    return rc;
}

// Checks of the host arguments that the operators have in common.
inline bool type_fits(const lmkv_pool_t* pool, int32_t dtype) {
    return ((dtype == LMKV_BF16 || dtype == LMKV_FP16) && pool->elem_bytes == 2) ||
           (dtype == LMKV_FP32 && pool->elem_bytes == 4);
}
inline bool rows_ok(const lmkv_rows_t* x, int32_t elem_bytes) {
    return x != nullptr && x->data != nullptr && reinterpret_cast<uintptr_t>(x->data) % elem_bytes == 0;
}
inline int check_batch(const lmkv_pool_t* pool, const lmkv_batch_t* b, int32_t num_q_heads) {
    if (b == nullptr || b->num_req < 0 || b->num_tokens < 0 || b->max_blocks < 0 || b->max_kv_len < 0 ||
        b->max_new < 0)
        return LMKV_ERR_INVALID_ARG;
    if (num_q_heads <= 0 || num_q_heads % pool->num_kv_heads != 0 || num_q_heads > (1 << 20))
        return LMKV_ERR_INVALID_ARG;
    if (b->max_kv_len > (int64_t)b->max_blocks * pool->block_size) return LMKV_ERR_INVALID_ARG;
    if (b->num_req > 0 && b->num_tokens > 0 && (b->q_start == nullptr || b->kv_len == nullptr ||
                                                (b->max_kv_len > 0 && b->block_table == nullptr)))
        return LMKV_ERR_INVALID_ARG;
    // rows are numbered (token, query head) with 32 bits
    if ((int64_t)b->num_tokens * num_q_heads > (int64_t)1 << 30 || b->num_req > (1 << 24))
        return LMKV_ERR_INVALID_ARG;
    return LMKV_OK;
}

}  // namespace lmkv_paged
