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
    bool vectors;              // a lane's pairs are two vectors of eight elements
    FastDiv by_sets;
    Rotary rot;                // half == 0: none
};

constexpr int kThreads = 128;
constexpr int kHeads = 4;      // heads of a page's CTA
constexpr int kPer = 4;        // rows of a thread on their way together

// A row of D elements lies with D / 16 neighbouring lanes, eight pairs each: pair n = 8 l + i is lane l's i-th.
// The pairs that turn come first, then the other elements two by two.  In the half layout pair n is elements
// (n, n + half), so where half is a multiple of 8 a lane's pairs are two vectors, the i-th of one with the i-th of
// the other, and no lane needs another's elements; interleaved it is (2n, 2n + 1), in two vectors too.
template <int D, bool kInterleaved>
struct Pairs {
    static constexpr int kLanes = D / 16;
    static __device__ __forceinline__ int first(const NormedParams& p, int n) {
        if (kInterleaved) return 2 * n;
        if (n < p.rot.half) return n;
        return p.vectors ? (n & ~7) * 2 + (n & 7) : 2 * n;
    }
    static __device__ __forceinline__ int second(const NormedParams& p, int n) {
        if (kInterleaved) return 2 * n + 1;
        if (n < p.rot.half) return n + p.rot.half;
        return p.vectors ? (n & ~7) * 2 + 8 + (n & 7) : 2 * n + 1;
    }
    // Where lane l's two vectors begin.
    static __device__ __forceinline__ int first_vector(const NormedParams& p, int l) {
        return !kInterleaved && 8 * l < p.rot.half ? 8 * l : 16 * l;
    }
    static __device__ __forceinline__ int second_vector(const NormedParams& p, int l) {
        return !kInterleaved && 8 * l < p.rot.half ? 8 * l + p.rot.half : 16 * l + 8;
    }
    // Pair n's place in a token's table: lanes side by side.
    static __device__ __forceinline__ int place(int n) { return (n & 7) * kLanes + (n >> 3); }
};

// A lane's 16 elements of a row as they were loaded: the half layout's a_i, then its b_i; interleaved, pair by pair.
template <class T, int D, bool kInterleaved>
struct RowOf {
    using P = Pairs<D, kInterleaved>;
    uint32_t raw[8];

    static __device__ __forceinline__ void ld16(const T* at, uint32_t& x, uint32_t& y, uint32_t& z, uint32_t& w) {
        asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x), "=r"(y), "=r"(z), "=r"(w)
                     : "l"(at) : "memory");
    }
    template <bool kVec>
    __device__ __forceinline__ void load(const NormedParams& p, const T* row, int l) {
        if constexpr (kVec) {
            ld16(row + P::first_vector(p, l), raw[0], raw[1], raw[2], raw[3]);
            ld16(row + P::second_vector(p, l), raw[4], raw[5], raw[6], raw[7]);
        } else {
            const uint16_t* const e = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const uint32_t a = e[P::first(p, 8 * l + i)], b = e[P::second(p, 8 * l + i)];
                const uint32_t c = e[P::first(p, 8 * l + i + 1)], d = e[P::second(p, 8 * l + i + 1)];
                raw[kInterleaved ? i : i / 2] = a | ((kInterleaved ? b : c) << 16);
                raw[kInterleaved ? i + 1 : 4 + i / 2] = (kInterleaved ? c : b) | (d << 16);
            }
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 8; ++i) raw[i] = 0u;
    }
    __device__ __forceinline__ void take(float (&a)[8], float (&b)[8]) const {
        const T* const x = reinterpret_cast<const T*>(raw);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            a[i] = Elem<T>::to_float(x[kInterleaved ? 2 * i : i]);
            b[i] = Elem<T>::to_float(x[kInterleaved ? 2 * i + 1 : 8 + i]);
        }
    }
};

// A token's table: pair n as (cos w_a, sin w_b, sin w_a, cos w_b), w the norm's weights.
template <class T, int D, bool kInterleaved>
__device__ __forceinline__ float4 table_entry(const NormedParams& p, const float* norm, int n, int64_t position) {
    using P = Pairs<D, kInterleaved>;
    const float wa = norm != nullptr ? norm[P::first(p, n)] : 1.f, wb = norm != nullptr ? norm[P::second(p, n)] : 1.f;
    if (n >= p.rot.half) return make_float4(wa, 0.f, 0.f, wb);
    float2 w = cos_sin<T>(p.rot.turns[n], position);
    w.x *= p.rot.magnitude;
    w.y *= p.rot.magnitude;
    return make_float4(w.x * wa, w.y * wb, w.y * wa, w.x * wb);
}

// x / sqrt(mean(x^2) + eps) * norm, turned; called by whole warps.  table: the token's, from this lane's place on.
template <class T, int D, bool kInterleaved>
__device__ __forceinline__ void norm_and_turn(const NormedParams& p, const RowOf<T, D, kInterleaved>& in, int l, bool normed,
                                              const float4* table, float (&a)[8], float (&b)[8]) {
    constexpr int kLanes = D / 16;
    in.take(a, b);
    float r = 1.f;
    if (normed) {
        float s = 0.f, t = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s = fmaf(a[i], a[i], s);
            t = fmaf(b[i], b[i], t);
        }
        s += t;
#pragma unroll
        for (int d = kLanes / 2; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
        r = rsqrtf(s * (1.f / D) + p.eps);        // (within 2^-22)
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float4 w = table[i * kLanes];
        const bool turns = 8 * l + i < p.rot.half;         // others stay apart, whatever they hold
        const float x = a[i], y = b[i];
        a[i] = (turns ? x * w.x - y * w.y : x * w.x) * r;
        b[i] = (turns ? x * w.z + y * w.w : y * w.w) * r;
    }
}

// The lane's 16 values to a row of T.
template <class T, int D, bool kInterleaved, bool kVec>
__device__ __forceinline__ void store_row(const NormedParams& p, T* row, int l, const float (&a)[8], const float (&b)[8]) {
    using P = Pairs<D, kInterleaved>;
    if constexpr (kVec) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (kInterleaved) w[i] = Elem<T>::pack(a[i], b[i]);
            else w[i] = i < 4 ? Elem<T>::pack(a[2 * i], a[2 * i + 1]) : Elem<T>::pack(b[2 * (i & 3)], b[2 * (i & 3) + 1]);
        }
        *reinterpret_cast<uint4*>(row + P::first_vector(p, l)) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(row + P::second_vector(p, l)) = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            row[P::first(p, 8 * l + i)] = Elem<T>::from_float(a[i]);
            row[P::second(p, 8 * l + i)] = Elem<T>::from_float(b[i]);
        }
    }
}
// As codes of value * factor.
template <int D, bool kInterleaved, bool kVec>
__device__ __forceinline__ void store_codes(const NormedParams& p, uint8_t* row, int l, float (&a)[8], float (&b)[8], float factor) {
    using P = Pairs<D, kInterleaved>;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        a[i] = fabsf(a[i]) < INFINITY ? a[i] * factor : NAN;
        b[i] = fabsf(b[i]) < INFINITY ? b[i] * factor : NAN;
    }
    if constexpr (kVec) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (kInterleaved)
                w[i] = (uint32_t)floats_to_codes(a[2 * i], b[2 * i]) | ((uint32_t)floats_to_codes(a[2 * i + 1], b[2 * i + 1]) << 16);
            else if (i < 2)
                w[i] = (uint32_t)floats_to_codes(a[4 * i], a[4 * i + 1]) | ((uint32_t)floats_to_codes(a[4 * i + 2], a[4 * i + 3]) << 16);
            else
                w[i] = (uint32_t)floats_to_codes(b[4 * i - 8], b[4 * i - 7]) | ((uint32_t)floats_to_codes(b[4 * i - 6], b[4 * i - 5]) << 16);
        }
        *reinterpret_cast<uint2*>(row + P::first_vector(p, l)) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2*>(row + P::second_vector(p, l)) = make_uint2(w[2], w[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint16_t c = floats_to_codes(a[i], b[i]);
            row[P::first(p, 8 * l + i)] = (uint8_t)c;
            row[P::second(p, 8 * l + i)] = (uint8_t)(c >> 8);
        }
    }
}

// A token's position.
struct Place {
    int64_t position;
    bool live;         // not a padded row
};

// One token's heads of q.
template <class T, int D, bool kInterleaved, bool kVec>
__device__ __forceinline__ void append_q(const NormedParams& p, int32_t t, float4* table) {
    using P = Pairs<D, kInterleaved>;
    constexpr int kGroups = kThreads / P::kLanes;
    __shared__ Place place;
    const int l = threadIdx.x % P::kLanes, g = threadIdx.x / P::kLanes;
    RowOf<T, D, kInterleaved> x[kPer];
    auto load = [&](int32_t h0) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int32_t h = h0 + j * kGroups + g;
            if (h < p.q_heads) x[j].template load<kVec>(p, p.q.row<T>(t, h), l);
            else x[j].clear();
        }
    };
    // the first rows are on their way before the look-ups
    load(0);
    // The position, where it is given, needs no request; what another warp finds out about that is only reported.
    const bool given = p.positions != nullptr;
    if (given && threadIdx.x == 0)
        place = Place{p.positions[t], t >= p.seqs.q_start[0] && t < p.seqs.q_start[p.seqs.num_req]};
    if (threadIdx.x >= 32 && threadIdx.x < 64) {
        const int32_t r = find_request(p.seqs.num_req, t, [&](int32_t i) { return p.seqs.q_start[i]; });
        if (threadIdx.x == 32) {
            const Req q = load_req(p.seqs, r);
            const int32_t end = min(max(p.seqs.q_start[r + 1], q.q0), p.seqs.num_tokens);
            const bool live = t >= q.q0 && t < end;
            const int32_t index = q.len - (end - q.q0) + (t - q.q0);
            if (live) {
                const bool whole = q.len == p.seqs.kv_len[r] && q.q0 == p.seqs.q_start[r] && end == p.seqs.q_start[r + 1];
                if (!whole || index < 0) report(p.status, LMKV_ERR_BAD_LENGTH);
            }
            if (!given) place = Place{index, live};
        }
    }
    __syncthreads();
    if (!place.live) return;
    for (int n = threadIdx.x; n < D / 2; n += kThreads)
        table[P::place(n)] = table_entry<T, D, kInterleaved>(p, p.q_norm, n, place.position);
    __syncthreads();
#pragma unroll 1
    for (int32_t h0 = 0; h0 < p.q_heads; h0 += kPer * kGroups) {
        if (h0 > 0) load(h0);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int32_t h = h0 + j * kGroups + g;
            if (h0 + j * kGroups >= p.q_heads) break;
            float a[8], b[8];
            norm_and_turn<T, D, kInterleaved>(p, x[j], l, p.q_norm != nullptr, table + l, a, b);
            if (h < p.q_heads) store_row<T, D, kInterleaved, kVec>(p, p.q_out.row<T>(t, h), l, a, b);
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
template <class T, int D, bool kCodes, bool kInterleaved, bool kVec>
__device__ __forceinline__ void append_page(const NormedParams& p, int32_t cta, float4* table) {
    using P = Pairs<D, kInterleaved>;
    constexpr int kGroups = kThreads / P::kLanes;
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
    const int l = threadIdx.x % P::kLanes, g = threadIdx.x / P::kLanes;
    const int hs = g % kHeads, row0 = g / kHeads;
    const int32_t h = (kv ? set - sets : set) * kHeads + hs;
    const bool head = h < p.kv_heads;
    const Rows& in = kv ? p.v : p.k;
    // the page's row of its token i
    auto place = [&](int32_t i) {
        return base + kv * p.layer.half_bytes() + ((int64_t)blk * B + i) * p.layer.row_bytes + (int64_t)h * D * (kCodes ? 1 : 2);
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
    RowOf<T, D, kInterleaved> raw[kPer];
    // A round's rows, and its tokens' tables.
    auto take = [&](int round) {
        const int32_t i0 = a + round * kRound;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int32_t i = i0 + j * kRows + row0;
            if (head && i < b) raw[j].template load<kVec>(p, in.row<T>(t0 + (i - a), h), l);
            else raw[j].clear();
        }
        if (!kv) {
            const int tokens = min(kRound, b - i0);
            if (round > 0) __syncthreads();         // the last round's are not read any more
            for (int i = threadIdx.x; i < tokens; i += kThreads)
                position[i] = p.positions != nullptr ? p.positions[t0 + i0 + i - a] : (int64_t)page0 + i0 + i;
            __syncthreads();
            for (int i = threadIdx.x; i < tokens * kPairs; i += kThreads) {
                const int tok = i / kPairs, n = i % kPairs;
                table[tok * kPairs + P::place(n)] = table_entry<T, D, kInterleaved>(p, p.k_norm, n, position[tok]);
            }
            __syncthreads();
        }
    };
    // Row j of the round as it goes to the page.  (Worked out twice, for the scale and for the codes: held,
    // the values of all rows would cost half the warps of an SM.)
    auto value = [&](int j, float (&x)[8], float (&y)[8]) {
        if (kv) raw[j].take(x, y);
        else
            norm_and_turn<T, D, kInterleaved>(p, raw[j], l, p.k_norm != nullptr, table + (j * kRows + row0) * kPairs + l, x, y);
    };
    float factor = 1.f;
    if constexpr (kCodes) {
        for (int round = 0; round < rounds; ++round) {
            take(round);
            float top = 0.f;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int32_t i = a + round * kRound + j * kRows;
                if (i >= b) break;
                float x[8], y[8];
                value(j, x, y);
                if (head && i + row0 < b) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if (fabsf(x[e]) < INFINITY) top = fmaxf(top, fabsf(x[e]));
                        if (fabsf(y[e]) < INFINITY) top = fmaxf(top, fabsf(y[e]));
                    }
                }
            }
#pragma unroll
            for (int d = P::kLanes / 2; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
            // magnitudes order as their bits do
            if (l == 0 && top > 0.f) atomicMax(&amax[hs], __float_as_uint(top));
        }
        __syncthreads();
        const float top = __uint_as_float(amax[hs]);
        const int e = max(before, top > 0.f ? min(max(least_exponent(top), kLowest), kHighest) : kLowest);
        if (head && a > 0 && e > before) {
            // the earlier tokens' codes, to the new scale
            const float by = power_of_two(before - e);
            for (int32_t i = row0; i < a; i += kRows) {
                uint4* const at = reinterpret_cast<uint4*>(place(i) + l * 16);
                const uint4 c = *at;
                uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t lo = codes_to_half2((uint16_t)w[k]), hi = codes_to_half2((uint16_t)(w[k] >> 16));
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&lo)),
                                 s = __half22float2(*reinterpret_cast<const __half2*>(&hi));
                    w[k] = (uint32_t)floats_to_codes(f.x * by, f.y * by) | ((uint32_t)floats_to_codes(s.x * by, s.y * by) << 16);
                }
                *at = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        if (head && row0 == 0 && l == 0) *scale = (uint8_t)(e + 127);
        factor = power_of_two(-e);
    }
    for (int round = 0; round < rounds; ++round) {
        if (!kCodes || rounds > 1) take(round);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int32_t i = a + round * kRound + j * kRows;
            if (i >= b) break;
            float x[8], y[8];
            value(j, x, y);
            if (!head || i + row0 >= b) continue;
            if constexpr (kCodes) store_codes<D, kInterleaved, kVec>(p, place(i + row0), l, x, y, factor);
            else store_row<T, D, kInterleaved, kVec>(p, reinterpret_cast<T*>(place(i + row0)), l, x, y);
        }
    }
}

// The CTAs of the pages come first, as theirs is the longer chain of waits, then a
// CTA a token for q.  (Rows that do not go by vectors have a kernel of their own: their loads, one by one, would
// take its registers.)  Bound by the bytes, q's rows both ways above all: 8948 tokens of 80 heads into 8 bits take 70 us,
// 5.0 TB/s; 64 tokens 11, which is the launch and one chain of loads.
template <class T, int D, bool kCodes, bool kInterleaved, bool kVec>
__global__ void __launch_bounds__(kThreads, kVec ? 5 : 4) append_normed_kernel(const __grid_constant__ NormedParams p) {
    constexpr int kRound = kThreads / (D / 16) / kHeads * kPer;
    __shared__ float4 table[kRound * (D / 2)];
    pdl_launch_dependents();
    pdl_wait();
    if ((int32_t)blockIdx.x < p.kv_ctas) append_page<T, D, kCodes, kInterleaved, kVec>(p, blockIdx.x, table);
    else append_q<T, D, kInterleaved, kVec>(p, blockIdx.x - p.kv_ctas, table);
}

template <class T, int D, bool kCodes>
int launch_normed(const NormedParams& p, bool vec, void* stream) {
    const int64_t ctas = (int64_t)p.kv_ctas + p.seqs.num_tokens;
    if (vec)
        return p.rot.interleaved ? launch(append_normed_kernel<T, D, kCodes, true, true>, ctas, kThreads, 0, stream, 1, p)
                                 : launch(append_normed_kernel<T, D, kCodes, false, true>, ctas, kThreads, 0, stream, 1, p);
    return p.rot.interleaved ? launch(append_normed_kernel<T, D, kCodes, true, false>, ctas, kThreads, 0, stream, 1, p)
                             : launch(append_normed_kernel<T, D, kCodes, false, false>, ctas, kThreads, 0, stream, 1, p);
}
template <class T>
int normed_typed(const NormedParams& p, int32_t head_dim, bool codes, bool vec, void* stream) {
    if (head_dim == 64) return codes ? launch_normed<T, 64, true>(p, vec, stream) : launch_normed<T, 64, false>(p, vec, stream);
    return codes ? launch_normed<T, 128, true>(p, vec, stream) : launch_normed<T, 128, false>(p, vec, stream);
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
    p.vectors = p.rot.half % 8 == 0;
    // 16-byte vectors where a lane's pairs are such and every row starts on 16 bytes
    bool vec = p.vectors || p.rot.interleaved;
    for (const lmkv_rows_t* x : {q, k, v, q_out})
        vec = vec && reinterpret_cast<uintptr_t>(x->data) % 16 == 0 && x->token_stride % 8 == 0 && x->head_stride % 8 == 0;
    p.head_sets = 2 * ((p.kv_heads + kHeads - 1) / kHeads);
    p.by_sets = FastDiv((uint32_t)p.head_sets);
    const int64_t slots = (int64_t)batch->num_tokens / pool->block_size + 2 * (int64_t)batch->num_req;
    const int64_t ctas = slots * p.head_sets;
    if (ctas + batch->num_tokens > INT32_MAX) return LMKV_ERR_INVALID_ARG;
    p.kv_ctas = (int32_t)ctas;
    const bool codes = pool->elem_bytes == 1;
    return dtype == LMKV_BF16 ? normed_typed<__nv_bfloat16>(p, pool->head_dim, codes, vec, stream)
                              : normed_typed<__half>(p, pool->head_dim, codes, vec, stream);
}
