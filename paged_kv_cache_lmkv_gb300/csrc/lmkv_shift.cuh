// lmkv_shift.cuh -- scatter of chunks into pages with the keys turned by a
// whole number of positions per request (lmkv_scatter_chunks_shifted).
//
// The same items as the plain scatter (lmkv_kernels.cuh): a CTA takes one
// page run.  Runs of V, and of K under shift 0, are copied.  A run of K is
// turned: the angle of a pair is the same for every token and head of the
// request, so the CTA computes rot_dim / 2 (cos, sin) once, while its first
// rows are on their way.  Bound, as the scatter, by reading and writing every
// row once.  (16 layers of 5 documents, 8 heads of 128: 494 us, 6.5 TB/s, 0.96 of the copy rate;
// one layer of 10240 tokens: 16.3 us, 0.76, the plain scatter's 14.7.)
#pragma once

#include "lmkv_kernels.cuh"
#include "lmkv_rotary.cuh"

namespace lmkv {

template <int kCap>
struct ShiftBatchT : BatchT<kCap> {
    lmkv_rotary_detail::Rotary rot;
    lmkv_paged::FastDiv by_head;         // units per head
    int32_t row_units;                   // units per row
    int32_t head_dim;
    int64_t shift[kCap];                 // of packed request i
};

template <class B, class T, int V, bool kInterleaved, int kThreads, int kUnroll>
__global__ void __launch_bounds__(kThreads)
shift_scatter_kernel(const __grid_constant__ B p, int64_t num_items) {
    using U = lmkv_rotary_detail::Units<T, V, kInterleaved, true>;
    __shared__ float2 cs[LMKV_ROTARY_MAX_PAIRS];
    pdl_launch_dependents();
    pdl_wait();
    const int64_t item = blockIdx.x;
    if (p.prefetch_ahead > 0 && threadIdx.x == 0 && item + p.prefetch_ahead < num_items) {
        Run ahead;
        if (item_run<B, false>(p, item + p.prefetch_ahead, ahead)) bulk_prefetch_l2(ahead.chunk, ahead.bytes);
    }
    Run run;
    if (!item_run(p, item, run)) return;              // the same for the whole CTA
    const int64_t shift = p.shift[resolve_chunk(p, run.gl).req];
    if (run.kv == 1 || shift == 0) {
        cta_copy<kThreads, 8>(run.chunk, run.pool, run.bytes);
        return;
    }
    const int half = p.rot.half;
    const int units = (int)(run.bytes / (uint32_t)p.row_bytes) * p.row_units;
    const T* src = reinterpret_cast<const T*>(run.chunk);
    T* dst = reinterpret_cast<T*>(run.pool);
    // unit -> (row, head, unit of the head): the rows of a run are contiguous
    // and heads fill a row, so (row, head) is one running number of heads
    auto at = [&](int i, int& u) {
        const int head = (int)p.by_head.div((uint32_t)i);
        u = i - head * (int)p.by_head.d;
        return (int64_t)head * p.head_dim;
    };
    bool first = true;
    for (int i0 = threadIdx.x; i0 - (int)threadIdx.x < units; i0 += kThreads * kUnroll) {
        U x[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int i = i0 + k * kThreads;
            if (i < units) {
                int u;
                const int64_t o = at(i, u);
                x[k].load(src + o, u, half);
            }
        }
        if (first) {
            for (int i = threadIdx.x; i < half; i += kThreads)
                cs[U::place(i, half)] = lmkv_rotary_detail::cos_sin<T>(p.rot.turns[i], shift);
            __syncthreads();
            first = false;
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int i = i0 + k * kThreads;
            if (i < units) {
                int u;
                const int64_t o = at(i, u);
                x[k].turn(cs, u, half);
                x[k].store(dst + o, u, half);
            }
        }
    }
}

}  // namespace lmkv
