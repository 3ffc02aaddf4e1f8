// lmkv_blocks.cuh -- blocks of 128 cached tokens' rows of one head from pages
// into shared memory, as operands of the tensor core.
#pragma once

#include "lmkv_tcgen05.cuh"

namespace lmkv_tc {

constexpr int kBlock = 128;           // keys of a block
constexpr int kLoadWarps = 2;         // two groups of 32 rows each

// A tile of 128 rows in shared memory.
template <int D>
struct BlockShape {
    static constexpr int kHalves = D / 64;
    static constexpr int kHalfBytes = 128 * 128;
    static constexpr int kBytes = kHalves * kHalfBytes;
};

// One of the kLoadWarps warps that copy blocks by cp.async, 16 bytes a lane.
// Pages may end anywhere.  The addresses are what such a copy costs, so they
// are kept to an addition where they can be: table entries are fetched a block
// ahead, and in pages of a multiple of 16 tokens 16 rows follow one another.
template <int D>
struct BlockCopy {
    static constexpr int kVecs = D / 8;             // 16-byte pieces of a row
    static constexpr int kRowsPer = 32 / kVecs;     // rows of a warp-wide copy
    static constexpr int kGroups = kBlock / 32 / kLoadWarps;
    static constexpr int kPatterns = 8 / kRowsPer;  // copies until the swizzle repeats
    static constexpr uint32_t kNoRow = lmkv_paged::Layer::kNoRow, kPast = kNoRow - 1;

    const lmkv_paged::Layer& layer;
    const uint8_t* base;
    int w, lane, c, rsub;
    uint32_t row_bytes, step;
    bool runs;
    uint32_t pattern[kPatterns];
    int32_t next_tok[kGroups], next_blk[kGroups];
    uint32_t next_col[kGroups];
    uint32_t rows[kGroups], there[kGroups], all;

    __device__ __forceinline__ BlockCopy(const lmkv_paged::Layer& l, const uint8_t* layer_base, uint32_t ring, int warp)
        : layer(l), base(layer_base), w(warp), lane(threadIdx.x & 31) {
        c = lane % kVecs;
        rsub = lane / kVecs;
        row_bytes = (uint32_t)l.row_bytes;
        step = row_bytes * kRowsPer;
        runs = l.block_size % 16 == 0;
#pragma unroll
        for (int k = 0; k < kPatterns; ++k) {
            const int row = k * kRowsPer + rsub;
            pattern[k] = ring + (c >> 3) * BlockShape<D>::kHalfBytes + (w * kGroups * 32 + row) * 128 +
                         (((c & 7) ^ (row & 7)) << 4);
        }
    }
    // This lane's piece of head h's row 0 of the K half.
    __device__ __forceinline__ const uint8_t* piece(int32_t h) const { return base + (int64_t)h * (D * 2) + c * 16; }

    // Fetches the table entries of the block at key k, of a sequence of `end` keys.
    __device__ __forceinline__ void lookup(const int32_t* table, int32_t k, int32_t end) {
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            const int32_t tok = k + (w * kGroups + g) * 32 + lane;
            const bool on = tok < end;
            next_tok[g] = on ? tok : -1;
            next_col[g] = layer.column(on ? tok : 0);
            next_blk[g] = on ? table[next_col[g]] : 0;
        }
    }
    // Takes the fetched entries as the block to copy.
    __device__ __forceinline__ void take(int32_t* status) {
        all = ~0u;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            rows[g] = next_tok[g] < 0 ? kPast : layer.row_of(next_blk[g], next_tok[g], next_col[g]);
            if (rows[g] == kNoRow) lmkv_paged::report(status, LMKV_ERR_BAD_BLOCK);
            there[g] = __ballot_sync(0xFFFFFFFFu, rows[g] < kPast);
            all &= there[g];
        }
    }
    // Which of the block's 128 keys there are, this warp's words of it.
    __device__ __forceinline__ void put_mask(uint32_t* words) const {
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
            if ((threadIdx.x & 31) == 0) words[w * kGroups + g] = there[g];
    }
    // Copies the block's rows (zeros for keys that are not there) to `stage`
    // bytes into the ring.
    __device__ __forceinline__ void copy(const uint8_t* from, uint32_t stage) const {
        if (all == ~0u && runs) {
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint32_t row = __shfl_sync(0xFFFFFFFFu, rows[g], u * 16) + rsub;
                    const uint8_t* src = from + (uint64_t)row * row_bytes;
#pragma unroll
                    for (int v = 0; v < kVecs / 2; ++v)
                        lmkv_mma::cp_async16(pattern[(u * (kVecs / 2) + v) % kPatterns] + stage +
                                                 (g * 32 + (u * (kVecs / 2) + v) / kPatterns * 8) * 128,
                                             src + v * step);
                }
        } else if (all == ~0u) {
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
#pragma unroll
                for (int v = 0; v < kVecs; ++v) {
                    const uint32_t row = __shfl_sync(0xFFFFFFFFu, rows[g], v * kRowsPer + rsub);
                    lmkv_mma::cp_async16(pattern[v % kPatterns] + stage + (g * 32 + v / kPatterns * 8) * 128,
                                         from + (uint64_t)row * row_bytes);
                }
        } else {
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
#pragma unroll
                for (int v = 0; v < kVecs; ++v) {
                    const uint32_t row = __shfl_sync(0xFFFFFFFFu, rows[g], v * kRowsPer + rsub);
                    const bool on = row < kPast;
                    lmkv_mma::cp_async16(pattern[v % kPatterns] + stage + (g * 32 + v / kPatterns * 8) * 128,
                                         from + (on ? (uint64_t)row * row_bytes : 0), on);
                }
        }
    }
};
// Arrivals on a stage's barrier: a thread each when its copies have landed,
// and one a warp for what it wrote besides.
constexpr int kCopyArrivals = kLoadWarps * 33;
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
    mbar_arrive_copies(bar);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

}  // namespace lmkv_tc
