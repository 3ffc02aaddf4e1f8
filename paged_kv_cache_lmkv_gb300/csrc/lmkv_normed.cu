// lmkv_normed.cu -- append of new tokens whose heads of q and k are normed and
// turned in one pass, to 16-bit pages or to pages of e4m3 codes.
#include "lmkv_cache8.cuh"
#include "lmkv_rotary.cuh"

#include <cmath>

namespace {

using namespace lmkv_paged;
using namespace lmkv_rotary_detail;
using namespace lmkv_cache8;

struct Rows {
    void* data;
    int64_t token_stride;
    int64_t head_stride;
    static Rows of(const lmkv_rows_t* x) { return Rows{x->data, x->token_stride, x->head_stride}; }
    template <class T>
    __device__ __forceinline__ T* row(int32_t token, int32_t head) const {
        return static_cast<T*>(data) + (int64_t)token * token_stride + (int64_t)head * head_stride;
    }
};

struct NormedParams {
    Layer layer;
    Seqs seqs;
    Scales scales;
    Rows q, k, v, q_out;
    const int64_t* positions;
    const float *q_norm, *k_norm;
    int32_t* status;
    int32_t q_heads, kv_heads;
    int32_t kv_ctas;           // CTAs of pages; those after them: a token's q
    int32_t head_sets;         // of kHeads heads, of K and of V
    float eps;
    bool vec_q, vec_out, vec_k, vec_v;      // rows of 16-byte vectors
    bool shuffles;             // a turned element's partner is a whole number of vectors away
    FastDiv by_sets;
    Rotary rot;                // half == 0: none
};

constexpr int kThreads = 256;
constexpr int kHeads = 4;      // heads of a page's CTA
constexpr int kPer = 4;        // rows of a thread on their way together

// A row of D elements lies with D / 8 neighbouring lanes, eight elements each.
template <class T, int D>
struct RowOf {
    T raw[8];

    __device__ __forceinline__ void load(const T* row, int e0, bool vec) {
        if (vec) {
            int4& r = *reinterpret_cast<int4*>(raw);
            asm volatile("ld.global.L1::no_allocate.v4.s32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(row + e0) : "memory");
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) raw[i] = row[e0 + i];
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 8; ++i) raw[i] = Elem<T>::from_float(0.f);
    }
};

// x / sqrt(mean(x^2) + eps) * norm, then turned by (cos, sin) cs[pair]; called by whole
// warps.  row: the row in memory, for partners that no shuffle reaches.
template <class T, int D>
__device__ __forceinline__ void norm_and_turn(const NormedParams& p, const RowOf<T, D>& in, const T* row, const float* norm,
                                              const float2* cs, float (&x)[8]) {
    constexpr int kLanes = D / 8;
    const int lane = threadIdx.x & 31, sub = lane % kLanes, e0 = sub * 8;
    float r = 1.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = Elem<T>::to_float(in.raw[i]);
    if (norm != nullptr) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int d = kLanes / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
        r = 1.f / sqrtf(ss * (1.f / D) + p.eps);
        const float4 a = *reinterpret_cast<const float4*>(norm + e0), b = *reinterpret_cast<const float4*>(norm + e0 + 4);
        const float w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= r * w[i];
    }
    const int half = p.rot.half;
    if (half == 0) return;
    if (p.rot.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            if (e0 + i >= 2 * half) break;
            const float2 w = cs[(e0 + i) >> 1];
            const float a = x[i], b = x[i + 1];
            x[i] = a * w.x - b * w.y;
            x[i + 1] = a * w.y + b * w.x;
        }
    } else {
        float y[8];            // the partners
        if (p.shuffles) {
            const int from = e0 < half ? lane + half / 8 : e0 < 2 * half ? lane - half / 8 : lane;
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xFFFFFFFFu, x[i], from);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = e0 + i, to = e < half ? e + half : e < 2 * half ? e - half : e;
                y[i] = row == nullptr ? 0.f : Elem<T>::to_float(row[to]) * (norm != nullptr ? r * norm[to] : 1.f);
            }
            __syncwarp();      // read before the row is written in place
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = e0 + i;
            if (e >= 2 * half) break;
            const float2 w = cs[e < half ? e : e - half];
            x[i] = e < half ? x[i] * w.x - y[i] * w.y : y[i] * w.y + x[i] * w.x;
        }
    }
}

template <class T>
__device__ __forceinline__ void store_row(T* dst, const float (&x)[8], bool vec) {
    if (vec) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(Elem<T>::pack(x[0], x[1]), Elem<T>::pack(x[2], x[3]),
                                                    Elem<T>::pack(x[4], x[5]), Elem<T>::pack(x[6], x[7]));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) dst[i] = Elem<T>::from_float(x[i]);
    }
}

// A token's request, cached number and position.
struct Place {
    int32_t index;
    int64_t position;
    bool live;         // not a padded row
};

// One token's heads of q.
template <class T, int D>
__device__ __forceinline__ void append_q(const NormedParams& p, int32_t t, float2* cs) {
    constexpr int kLanes = D / 8, kGroups = kThreads / kLanes;
    __shared__ Place place;
    const int sub = threadIdx.x % kLanes, g = threadIdx.x / kLanes;
    RowOf<T, D> x[kPer];
    auto load = [&](int32_t h0) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int32_t h = h0 + j * kGroups + g;
            if (h < p.q_heads) x[j].load(p.q.row<T>(t, h), sub * 8, p.vec_q);
            else x[j].clear();
        }
    };
    load(0);
    if (threadIdx.x < 32) {
        const int32_t r = find_request(p.seqs.num_req, t, [&](int32_t i) { return p.seqs.q_start[i]; });
        if (threadIdx.x == 0) {
            const Req q = load_req(p.seqs, r);
            const int32_t end = min(max(p.seqs.q_start[r + 1], q.q0), p.seqs.num_tokens);
            Place x{0, 0, t >= q.q0 && t < end};
            if (x.live) {
                x.index = q.len - (end - q.q0) + (t - q.q0);
                x.position = p.positions != nullptr ? p.positions[t] : (int64_t)x.index;
                const bool whole = q.len == p.seqs.kv_len[r] && q.q0 == p.seqs.q_start[r] && end == p.seqs.q_start[r + 1];
                if (!whole || x.index < 0) report(p.status, LMKV_ERR_BAD_LENGTH);
            }
            place = x;
        }
    }
    __syncthreads();
    if (!place.live) return;
    for (int i = threadIdx.x; i < p.rot.half; i += kThreads) {
        const float2 w = cos_sin<T>(p.rot.turns[i], place.position);
        cs[i] = make_float2(w.x * p.rot.magnitude, w.y * p.rot.magnitude);
    }
    __syncthreads();
    for (int32_t h0 = 0; h0 < p.q_heads; h0 += kPer * kGroups) {
        if (h0 > 0) load(h0);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int32_t h = h0 + j * kGroups + g;
            if (h0 + j * kGroups >= p.q_heads) break;
            const bool on = h < p.q_heads;
            float y[8];
            norm_and_turn<T, D>(p, x[j], on ? p.q.row<T>(t, h) : nullptr, p.q_norm, cs, y);
            if (on) store_row<T>(p.q_out.row<T>(t, h) + sub * 8, y, p.vec_out);
        }
    }
}

// The least e with a <= 448 * 2^e, a finite and > 0: a = m 2^k with 1 <= m < 2, 448 = 1.75 * 2^8.
__device__ __forceinline__ int least_exponent(float a) {
    const uint32_t bits = __float_as_uint(a);
    const int k = (int)(bits >> 23) - 127;
    return (bits & 0x7FFFFFu) > 0x600000u ? k - 7 : k - 8;
}
constexpr int kLowest = -60, kHighest = 60;

// The new tokens of one page: kHeads heads of K or of V.  A page's tokens of a head have to be seen
// before the first is written, as they share a scale, so kHeads heads are spread over the
// CTA token by token and meet in shared memory.  Pages of more tokens than fit its registers are read twice.
template <class T, int D, bool kCodes>
__device__ __forceinline__ void append_page(const NormedParams& p, int32_t cta, float2* cs) {
    constexpr int kLanes = D / 8, kGroups = kThreads / kLanes;
    constexpr int kRows = kGroups / kHeads;         // tokens side by side
    constexpr int kRound = kRows * kPer;            // tokens of a round
    constexpr int kPairs = D / 2;
    __shared__ int32_t first[5];                    // page's first new token's row, its place in the page, the end's, block id, page's first token
    __shared__ int64_t position[kRound];
    __shared__ uint32_t amax[kHeads];
    const int32_t slot = (int32_t)p.by_sets.div((uint32_t)cta), set = cta - slot * p.head_sets;
    const int32_t sets = p.head_sets / 2;
    const int kv = set >= sets ? 1 : 0;
    const int32_t B = p.layer.block_size;
    uint8_t* const base = p.layer.base();
    if (threadIdx.x < 32) {
        // Slots q_start[r] / B + 2 r and on are request r's pages: n tokens come into n / B + 2
        // pages at most, and there are as many up to the next request's.
        auto key = [&](int32_t i) { return (int32_t)p.layer.by_block.div((uint32_t)max(p.seqs.q_start[i], 0)) + 2 * i; };
        const int32_t r = find_request(p.seqs.num_req, slot, key);
        if (threadIdx.x == 0) {
            const Req q = load_req(p.seqs, r);
            const int32_t end = min(max(p.seqs.q_start[r + 1], q.q0), p.seqs.num_tokens), n = end - q.q0;
            const bool whole = q.len == p.seqs.kv_len[r] && q.q0 == p.seqs.q_start[r] && end == p.seqs.q_start[r + 1];
            const int32_t old = q.len - n;          // (below 0: tokens without a place)
            const int32_t col = (int32_t)p.layer.by_block.div((uint32_t)max(old, 0)) + slot - key(r);
            const int64_t page0 = (int64_t)col * B;
            int32_t blk = -1, a = 0, b = 0;
            if (whole && n > 0 && slot >= key(r) && page0 < q.len) {
                a = (int32_t)(max((int64_t)max(old, 0), page0) - page0);
                b = (int32_t)(min((int64_t)q.len, page0 + B) - page0);
                blk = p.seqs.table[(int64_t)r * p.seqs.table_stride + col];
                if (base == nullptr || (kCodes && p.scales.base() == nullptr)) {
                    report(p.status, LMKV_ERR_BAD_POINTER);
                    blk = -1;
                } else if (blk < 0 || blk >= p.layer.num_blocks) {
                    report(p.status, LMKV_ERR_BAD_BLOCK);
                    blk = -1;
                }
            }
            first[0] = q.q0 + (int32_t)(page0 + a - old);      // row of token a of the page
            first[1] = a;
            first[2] = b;
            first[3] = blk;
            first[4] = (int32_t)page0;
        }
    }
    if (threadIdx.x < kHeads) amax[threadIdx.x] = 0;
    __syncthreads();
    const int32_t t0 = first[0], a = first[1], b = first[2], blk = first[3], page0 = first[4];
    if (blk < 0) return;
    const int sub = threadIdx.x % kLanes, g = threadIdx.x / kLanes;
    const int hs = g % kHeads, row0 = g / kHeads;
    const int32_t h = (kv ? set - sets : set) * kHeads + hs;
    const bool head = h < p.kv_heads;
    const Rows& in = kv ? p.v : p.k;
    const bool vec = kv ? p.vec_v : p.vec_k;
    // the page's row of token i of it, this lane's part
    auto place = [&](int32_t i) {
        return base + kv * p.layer.half_bytes() + ((int64_t)blk * B + i) * p.layer.row_bytes +
               ((int64_t)h * D + sub * 8) * (kCodes ? 1 : 2);
    };
    uint8_t* scale = nullptr;
    int before = kLowest;                           // exponent of the page's earlier tokens
    if constexpr (kCodes) {
        if (head) {
            scale = p.scales.base() + p.scales.at(kv, blk, h);
            if (a > 0) before = (int)*scale - 127;
        }
    }
    const int rounds = (b - a + kRound - 1) / kRound;
    float x[kPer][8];
    auto take = [&](int round) {
        const int32_t i0 = a + round * kRound;
        RowOf<T, D> raw[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int32_t i = i0 + j * kRows + row0;
            if (head && i < b) raw[j].load(in.row<T>(t0 + (i - a), h), sub * 8, vec);
            else raw[j].clear();
        }
        if (!kv && p.rot.half > 0) {
            __syncthreads();                        // the last round's are not read any more
            for (int i = threadIdx.x; i < kRound; i += kThreads) {
                const int32_t at = min(i0 + i, b - 1);
                position[i] = p.positions != nullptr ? p.positions[t0 + at - a] : (int64_t)page0 + at;
            }
            __syncthreads();
            const int half = p.rot.half, tokens = min(kRound, b - i0);
            for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
                const int tok = i / half, pair = i - tok * half;
                const float2 w = cos_sin<T>(p.rot.turns[pair], position[tok]);
                cs[tok * kPairs + pair] = make_float2(w.x * p.rot.magnitude, w.y * p.rot.magnitude);
            }
            __syncthreads();
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int32_t i = i0 + j * kRows + row0;
            const bool on = head && i < b;
            if (kv) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[j][e] = Elem<T>::to_float(raw[j].raw[e]);
            } else {
                norm_and_turn<T, D>(p, raw[j], on ? in.row<T>(t0 + (i - a), h) : nullptr, p.k_norm,
                                    cs + min((int)(i - i0), kRound - 1) * kPairs, x[j]);
            }
        }
    };
    float factor = 1.f;
    if constexpr (kCodes) {
        for (int round = 0; round < rounds; ++round) {
            take(round);
            float top = 0.f;
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if (head && a + round * kRound + j * kRows + row0 < b) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (fabsf(x[j][e]) < INFINITY) top = fmaxf(top, fabsf(x[j][e]));
                }
#pragma unroll
            for (int d = kLanes / 2; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
            // magnitudes order as their bits do
            if (sub == 0 && top > 0.f) atomicMax(&amax[hs], __float_as_uint(top));
        }
        __syncthreads();
        const float top = __uint_as_float(amax[hs]);
        const int e = max(before, top > 0.f ? min(max(least_exponent(top), kLowest), kHighest) : kLowest);
        if (head && a > 0 && e > before) {
            // the earlier tokens' codes, to the new scale
            const float by = power_of_two(before - e);
            for (int32_t i = row0; i < a; i += kRows) {
                uint2* const at = reinterpret_cast<uint2*>(place(i));
                const uint2 c = *at;
                uint32_t w[2] = {c.x, c.y};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t lo = codes_to_half2((uint16_t)w[k]), hi = codes_to_half2((uint16_t)(w[k] >> 16));
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&lo)),
                                 s = __half22float2(*reinterpret_cast<const __half2*>(&hi));
                    w[k] = (uint32_t)floats_to_codes(f.x * by, f.y * by) | ((uint32_t)floats_to_codes(s.x * by, s.y * by) << 16);
                }
                *at = make_uint2(w[0], w[1]);
            }
        }
        if (head && row0 == 0 && sub == 0) *scale = (uint8_t)(e + 127);
        factor = power_of_two(-e);
    }
    for (int round = 0; round < rounds; ++round) {
        if (!kCodes || rounds > 1) take(round);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int32_t i = a + round * kRound + j * kRows + row0;
            if (!head || i >= b) continue;
            if constexpr (kCodes) {
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = fabsf(x[j][e]) < INFINITY ? x[j][e] * factor : NAN;
                const uint32_t lo = (uint32_t)floats_to_codes(y[0], y[1]) | ((uint32_t)floats_to_codes(y[2], y[3]) << 16);
                const uint32_t hi = (uint32_t)floats_to_codes(y[4], y[5]) | ((uint32_t)floats_to_codes(y[6], y[7]) << 16);
                *reinterpret_cast<uint2*>(place(i)) = make_uint2(lo, hi);
            } else {
                store_row<T>(reinterpret_cast<T*>(place(i)), x[j], true);
            }
        }
    }
}

// The CTAs of the pages come first, as theirs is the longer chain of waits, then a
// CTA a token for q.
template <class T, int D, bool kCodes>
__global__ void __launch_bounds__(kThreads) append_normed_kernel(const __grid_constant__ NormedParams p) {
    constexpr int kRound = kThreads / (D / 8) / kHeads * kPer;
    __shared__ float2 cs[kRound * (D / 2)];
    pdl_launch_dependents();
    pdl_wait();
    if ((int32_t)blockIdx.x < p.kv_ctas) append_page<T, D, kCodes>(p, blockIdx.x, cs);
    else append_q<T, D>(p, blockIdx.x - p.kv_ctas, cs);
}

template <class T, int D, bool kCodes>
int launch_normed(const NormedParams& p, void* stream) {
    return launch(append_normed_kernel<T, D, kCodes>, (int64_t)p.kv_ctas + p.seqs.num_tokens, kThreads, 0, stream, 1, p);
}
template <class T>
int normed_typed(const NormedParams& p, int32_t head_dim, bool codes, void* stream) {
    if (head_dim == 64) return codes ? launch_normed<T, 64, true>(p, stream) : launch_normed<T, 64, false>(p, stream);
    return codes ? launch_normed<T, 128, true>(p, stream) : launch_normed<T, 128, false>(p, stream);
}

}  // namespace

extern "C" int lmkv_append_layer_normed(const lmkv_pool_t* pool, void* const* scales, int32_t dtype, int32_t layer,
                                        const lmkv_batch_t* batch, int32_t num_q_heads, const lmkv_rows_t* q,
                                        const lmkv_rows_t* k, const lmkv_rows_t* v, const lmkv_rows_t* q_out,
                                        const int64_t* positions, const lmkv_rotary_t* rotary, const float* q_norm,
                                        const float* k_norm, float eps, int32_t* d_status, void* stream) {
    int rc = lmkv_internal_check_pool(pool);
    if (rc == LMKV_OK) rc = check_scales(pool, scales, dtype);
    if (rc != LMKV_OK) return rc;
    if (layer < 0 || layer >= pool->num_layers || !(eps >= 0.f) || !std::isfinite(eps)) return LMKV_ERR_INVALID_ARG;
    rc = check_batch(pool, batch, num_q_heads);
    if (rc != LMKV_OK) return rc;
    NormedParams p = {};
    if (rotary != nullptr) rc = make_rotary(rotary, pool->head_dim, &p.rot);
    if (rc != LMKV_OK) return rc;
    if (batch->num_req == 0 || batch->num_tokens == 0) return LMKV_OK;
    if (!rows_ok(q, 2) || !rows_ok(k, 2) || !rows_ok(v, 2) || !rows_ok(q_out, 2)) return LMKV_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(q_norm) | reinterpret_cast<uintptr_t>(k_norm)) & 15) return LMKV_ERR_MISALIGNED;
    p.layer = Layer::of(pool, layer);
    p.seqs = Seqs::of(batch);
    p.scales = Scales::of(pool, scales, layer);
    p.q = Rows::of(q);
    p.k = Rows::of(k);
    p.v = Rows::of(v);
    p.q_out = Rows::of(q_out);
    p.positions = positions;
    p.q_norm = q_norm;
    p.k_norm = k_norm;
    p.status = d_status;
    p.q_heads = num_q_heads;
    p.kv_heads = pool->num_kv_heads;
    p.eps = eps;
    auto vec = [](const lmkv_rows_t* x) {
        return reinterpret_cast<uintptr_t>(x->data) % 16 == 0 && x->token_stride % 8 == 0 && x->head_stride % 8 == 0;
    };
    p.vec_q = vec(q);
    p.vec_out = vec(q_out);
    p.vec_k = vec(k);
    p.vec_v = vec(v);
    p.shuffles = p.rot.half % 8 == 0;
    p.head_sets = 2 * ((p.kv_heads + kHeads - 1) / kHeads);
    p.by_sets = FastDiv((uint32_t)p.head_sets);
    const int64_t slots = (int64_t)batch->num_tokens / pool->block_size + 2 * (int64_t)batch->num_req;
    const int64_t ctas = slots * p.head_sets;
    if (ctas + batch->num_tokens > INT32_MAX) return LMKV_ERR_INVALID_ARG;
    p.kv_ctas = (int32_t)ctas;
    const bool codes = pool->elem_bytes == 1;
    return dtype == LMKV_BF16 ? normed_typed<__nv_bfloat16>(p, pool->head_dim, codes, stream)
                              : normed_typed<__half>(p, pool->head_dim, codes, stream);
}
