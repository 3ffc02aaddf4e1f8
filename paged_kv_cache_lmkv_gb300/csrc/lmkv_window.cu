// lmkv_window.cu -- attention of a batch's new tokens to their own pages, of 16
// or 8 bits, with a sliding window and sinks.
//
// With y_j = scale * q.k_j + log v_scale_j (powers of 2), and codes c_j of v,
//   o = sum_j 2^(y_j) c_j / sum_j 2^(y_j) / v_scale_j,
// which splits over any partition of the keys: a part keeps what its weights are
// relative to (m), l = sum 2^(y - m) / v_scale and sum 2^(y - m) c; parts are joined by
//   M = max m,  l = sum l 2^(m - M),  o = sum o 2^(m - M) / l
// (the running maximum and sum of Milakov and Gimelshein, "Online normalizer
// calculation for softmax", 2018).  So a page's scale of v costs its keys an
// addition in the exponent, and its scale of k a factor of the score; codes go to the products as they are.
// (The weights' product with v is of fp16, whose range y's maximum makes good use of whatever the scales are.)
// 16-bit pages are the same with scales of 1.
#include "lmkv_blocks.cuh"
#include "lmkv_cache8.cuh"

#include <cmath>

namespace {

using namespace lmkv_paged;
using namespace lmkv_mma;
using namespace lmkv_cache8;

struct Rows {
    uint8_t* data;
    int64_t token_stride;
    int64_t head_stride;
    static Rows of(const lmkv_rows_t* x) {
        return Rows{static_cast<uint8_t*>(x->data), x->token_stride, x->head_stride};
    }
    template <class T>
    __device__ __forceinline__ T* row(int32_t token, int32_t head) const {
        return reinterpret_cast<T*>(data) + (int64_t)token * token_stride + (int64_t)head * head_stride;
    }
};

// A request whose rows per KV head (new tokens x heads of the group) reach
// big_rows goes by the tile kernel, the others by streams.
struct WindowParams {
    Layer layer;
    Seqs seqs;
    Scales scales;
    Rows q, out;
    float* lse;
    int32_t* status;
    // Partial results: m (powers of 2), l and the weighted sum of codes.  Of the tiles
    // [part][row], row = token * q_heads + head; then of the streams [stream + row tile of the batch's
    // requests][row of the tile][KV head] (a stream's and a tile's number rise from
    // part to part, so their sum names it).
    float* part_o;
    float2* part_ml;
    int2* own_range;        // [request][row tile]: first and last stream that has some of it
    float scale_log2;       // of |scale|
    int32_t scale_sign;     // -1, 0 or 1
    int32_t window;         // INT32_MAX: none
    int32_t sinks;
    int32_t q_heads, kv_heads;
    int32_t rows;           // num_tokens * q_heads
    int32_t big_rows;       // INT32_MAX: no tiles
    int32_t own_cap;        // rows of a request that streams take at most
    int32_t own_tiles;      // row tiles of that many rows
    int32_t tile_rows;      // rows of a tile
    int32_t streams;        // warps that share the keys of a KV head
    int32_t slots;          // tile kernel: row tiles that there may be
    int32_t parts;          // its parts of the keys
    int32_t items;          // its items: row tiles x KV heads x parts
    int32_t* next_item;     // those taken (beyond one for each CTA); the streams begin it
    int64_t own_base;       // rows of partial results before the streams'
    bool q_pairs;           // q rows are 4-byte aligned
    bool q_vec;             // 16-byte aligned
    bool out_wide;          // out rows are 32-byte aligned
    FastDiv by_group;

    __device__ __forceinline__ int64_t own_part(int32_t stream, int32_t tile_no, int32_t row, int32_t h) const {
        return own_base + (((int64_t)stream + tile_no) * tile_rows + row) * kv_heads + h;
    }
};

constexpr float kLn2 = 0.69314718055994530942f, kLog2e = 1.44269504088896340736f;
// Weights are relative to 2^kBelow less than a maximum that may lag by 2^kLag, so they are 2^14
// at most, and those of 2^-20 of the largest are still normal fp16 numbers.
constexpr float kBelow = 6.f, kLag = 8.f;
// V's scales are at least 2^-90: the sum of weights holds their inverse.
constexpr uint32_t kLeastScale = 127 - 90;
// A finite number below every score, so that the first keys need no case of their own.
constexpr float kNone = -0x1p126f;

// The keys that some row of tokens t0 .. t1 (cached numbers) sees, in units of
// kUnit keys: first the sinks' units, then the window's.
struct Seen {
    int32_t first_units;      // units 0 .. first_units - 1
    int32_t then;             // number of the unit after them
    int32_t units;            // in all
    int32_t sink_end, lo, end;      // keys [0, sink_end) and [lo, end)

    __device__ __forceinline__ int32_t unit(int32_t i) const { return i < first_units ? i : i - first_units + then; }
    __device__ __forceinline__ bool some(int32_t j) const { return j < end && (j < sink_end || j >= lo); }
};
// The first key that token t's window has, t < 0 too: a difference of the two would not fit 32 bits for every window.
__device__ __forceinline__ int32_t first_in_window(const WindowParams& p, int32_t t) {
    return p.window == INT32_MAX ? 0 : max(t + 1, p.window) - p.window;
}
__device__ __forceinline__ Seen seen_by(const WindowParams& p, int32_t t0, int32_t t1, int32_t unit) {
    Seen s;
    s.end = max(t1 + 1, 0);
    s.lo = first_in_window(p, t0);
    s.sink_end = min(p.sinks, s.end);
    if (s.lo <= s.sink_end) s.lo = s.sink_end = 0;      // one stretch
    s.first_units = (s.sink_end + unit - 1) / unit;
    s.then = max(s.lo / unit, s.first_units);
    s.units = s.first_units + max((s.end + unit - 1) / unit - s.then, 0);
    return s;
}

// ---- streams ------------------------------------------------------------

constexpr int kWarps = 4;
constexpr int kChunk = 16;        // keys a warp takes at a time

// How KV rows of D elements lie in shared memory and come out as fragments.
// A chunk's 16 rows of K are the first operand of S^T = K q^T, and V^T that of O^T =
// V^T P^T, so that up to eight queries are the products' narrow side.  Either product's
// order of elements is free: thread (g, c) = (lane / 4, lane % 4) takes K's 16-byte
// pieces c, c + 4, .. of rows tau(g) and tau(g) + 8 whole, and D / 8 neighbouring elements of V's
// rows c, c + 4, c + 8, c + 12, with tau(g) = g / 2 + 4 (g % 2) the row that the weights' fragment has
// there.  Pieces are exchanged within a row so that neither read meets a bank twice.
template <class KV, int D>
struct Fragments {
    static constexpr bool kCodes = sizeof(KV) == 1;
    static constexpr int kRowBytes = D * (int)sizeof(KV);
    static constexpr int kPieces = kRowBytes / 16;
    static constexpr int kTileBytes = kChunk * kRowBytes;
    static constexpr int kPer = 16 / (int)sizeof(KV);     // elements of a piece
    static constexpr int kSteps = D / 16;

    static __device__ __forceinline__ uint32_t place(int row, int piece) {
        if constexpr (kRowBytes >= 128) {
            return (uint32_t)(row * kRowBytes + ((piece ^ (((row & 3) << 1) ^ (row & 4))) << 4));
        } else {        // two rows in 128 bytes
            return (uint32_t)((row ^ ((row >> 2) & 1)) * kRowBytes + ((piece ^ (row & 2)) << 4));
        }
    }
    // The element of V that row `half` (0, 1) of tile j of the product is, of lane group g.
    static __device__ __forceinline__ int element(int j, int g) {
        if constexpr (!kCodes && D == 128) return (j >> 2) * 64 + g * 8 + 2 * (j & 3);
        return g * (D / 8) + 2 * j;
    }
};

__device__ __forceinline__ uint4 lds128(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void sts128(uint32_t at, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) { return __byte_perm(a, b, sel); }
// The 8 x 8 matrix of 16-bit elements whose row lane / 4 has this word at columns 2 (lane % 4), transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t w) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(w));
    return r;
}

// What a chunk is besides its rows: which of its keys some row sees, and the scale bytes
// (k, v of row tau(g), then of row tau(g) + 8).
struct ChunkInfo {
    uint32_t mask, scales;
};

// Copies chunks of 16 keys' rows of one head, K and V, into a warp's ring.
template <class KV, int D>
struct ChunkLoad {
    using F = Fragments<KV, D>;
    static constexpr int kRowsPer = 32 / F::kPieces > 16 ? 16 : 32 / F::kPieces;     // rows of a warp-wide copy
    const WindowParams& p;
    const int32_t* table;
    const uint8_t* base;
    const uint8_t* scale_base;
    int64_t half_bytes, v_scales;
    uint32_t row_bytes;
    int32_t h;
    bool runs;
    Seen seen;
    int32_t next_blk;

    __device__ __forceinline__ ChunkLoad(const WindowParams& wp, const int32_t* t, const uint8_t* layer_base,
                                         const uint8_t* scales, int32_t head, const Seen& s)
        : p(wp), table(t), base(layer_base), half_bytes(wp.layer.half_bytes()),
          row_bytes((uint32_t)wp.layer.row_bytes), h(head), runs(wp.layer.block_size % kChunk == 0), seen(s), next_blk(-1) {
        scale_base = F::kCodes ? scales + head : nullptr;
        v_scales = wp.scales.num_blocks * wp.kv_heads;
    }
    __device__ __forceinline__ void lookup(int32_t i, int32_t n) {
        next_blk = runs && i < n ? table[p.layer.column(seen.unit(i) * kChunk)] : -1;
    }
    __device__ __forceinline__ uint32_t bytes_of(int32_t blk) const {
        if constexpr (!F::kCodes) return 0;
        const uint8_t* const at = scale_base + (int64_t)blk * p.kv_heads;
        return (uint32_t)at[0] | ((uint32_t)at[v_scales] << 8);
    }
    // Unit i (looked up before) to dst; then looks up the next, of n.
    __device__ __forceinline__ ChunkInfo copy(int32_t i, uint32_t dst, int32_t n) {
        const int lane = threadIdx.x & 31, piece = lane % F::kPieces, rsub = lane / F::kPieces;
        const int32_t blk = next_blk, key0 = seen.unit(i) * kChunk;
        lookup(i + 1, n);
        const uint8_t* const mine = base + (int64_t)h * F::kRowBytes + piece * 16;
        const bool whole = key0 + kChunk <= seen.end && (key0 >= seen.lo || key0 + kChunk <= seen.sink_end);
        if (runs && whole && blk >= 0 && blk < p.layer.num_blocks) {
            const uint8_t* src = mine + ((uint64_t)p.layer.row_of(blk, key0, p.layer.column(key0)) + rsub) * row_bytes;
#pragma unroll
            for (int r = 0; r < kChunk; r += kRowsPer) {
                const uint32_t at = dst + F::place(r + rsub, piece);
                cp_async16(at, src + r * row_bytes);
                cp_async16(at + F::kTileBytes, src + r * row_bytes + half_bytes);
            }
            const uint32_t s = bytes_of(blk);
            return ChunkInfo{0xFFFFu, s | (s << 16)};
        }
        const int32_t tok = key0 + (lane & 15);
        uint32_t row = Layer::kNoRow;
        int32_t b = 0;
        if (seen.some(tok)) {
            const uint32_t col = p.layer.column(tok);
            b = table[col];
            row = p.layer.row_of(b, tok, col);
            if (row == Layer::kNoRow && lane < 16) report(p.status, LMKV_ERR_BAD_BLOCK);
        }
        const uint32_t mask = __ballot_sync(0xFFFFFFFFu, row != Layer::kNoRow) & 0xFFFFu;
#pragma unroll
        for (int r = 0; r < kChunk; r += kRowsPer) {
            const uint32_t from = __shfl_sync(0xFFFFFFFFu, row, r + rsub);
            const bool on = from != Layer::kNoRow;
            const uint32_t at = dst + F::place(r + rsub, piece);
            const uint8_t* const src = mine + (on ? (uint64_t)from * row_bytes : 0);
            cp_async16(at, src, on);
            cp_async16(at + F::kTileBytes, src + (on ? half_bytes : 0), on);
        }
        uint32_t s = 0x7F7F7F7Fu;
        if constexpr (F::kCodes) {
            const int g = lane >> 2, ta = (g >> 1) + 4 * (g & 1);
            const int32_t ba = __shfl_sync(0xFFFFFFFFu, b, ta), bb = __shfl_sync(0xFFFFFFFFu, b, ta + 8);
            const uint32_t sa = (mask >> ta) & 1 ? bytes_of(ba) : 0x7F7Fu, sb = (mask >> (ta + 8)) & 1 ? bytes_of(bb) : 0x7F7Fu;
            s = sa | (sb << 16);
        }
        return ChunkInfo{mask, s};
    }
};

// One warp's 8 * NT rows against chunks of 16 keys.  Thread (g, c) holds of every tile of 8
// queries those numbered 2 c and 2 c + 1, and D / 8 elements of their output.
template <class T, class KV, int D, int NT>
struct StreamRows {
    using F = Fragments<KV, D>;
    using M = typename std::conditional<F::kCodes, __half, T>::type;       // of the products
    uint32_t qf[NT][F::kSteps][2];
    float o[NT][F::kSteps][4];
    float ref[NT][2], l[NT][2];    // what weights are relative to (kNone: no key yet); sums
    float factor[NT][2];           // of raw scores
    int32_t tok[NT][2];            // cached number of the row's token; -1: no row
    int32_t t_first, t_last;       // of the tile's rows

    // Rows row0 .. row0 + nrows - 1 of the request (token * group + head of the group).
    __device__ __forceinline__ void begin(const WindowParams& p, const Req& r, int32_t h, int32_t row0, int32_t nrows) {
        const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
        const int32_t group = (int32_t)p.by_group.d;
        const int32_t old = r.len - r.n;
        t_first = old + (int32_t)p.by_group.div((uint32_t)row0);
        t_last = old + (int32_t)p.by_group.div((uint32_t)(row0 + min(nrows, NT * 8) - 1));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int32_t rr = nt * 8 + g;
            const bool on = rr < nrows;
            const int32_t i = (int32_t)p.by_group.div((uint32_t)(row0 + (on ? rr : 0)));
            const T* src = p.q.row<T>(r.q0 + i, h * group + (row0 + (on ? rr : 0) - i * group));
#pragma unroll
            for (int s = 0; s < F::kSteps; ++s) {
                constexpr int kStepsPer = F::kPer / 4;
                const int e = (c + 4 * (s / kStepsPer)) * F::kPer + 4 * (s % kStepsPer);
                qf[nt][s][0] = on ? load_pair(src + e, p.q_pairs) : 0u;
                qf[nt][s][1] = on ? load_pair(src + e + 2, p.q_pairs) : 0u;
            }
        }
        const uint32_t flip = p.scale_sign < 0 ? 0x80008000u : 0u, all = p.scale_sign == 0 ? 0u : ~0u;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float f = p.scale_log2;
#pragma unroll
            for (int s = 0; s < F::kSteps; ++s)
#pragma unroll
                for (int k = 0; k < 2; ++k) qf[nt][s][k] = (qf[nt][s][k] ^ flip) & all;
            if constexpr (F::kCodes) {
                // the row's q as fp16 with its largest element between 2^14 and 2^15: exact but for elements
                // below 2^-28 of that
                float top = 0.f;
#pragma unroll
                for (int s = 0; s < F::kSteps; ++s)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const T* const x = reinterpret_cast<const T*>(&qf[nt][s][k]);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float a = fabsf(Elem<T>::to_float(x[i]));
                            if (a < INFINITY) top = fmaxf(top, a);
                        }
                    }
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                const int e = top > 0.f ? max((int)(__float_as_uint(top) >> 23) - 127, -100) : 0;
                const float by = power_of_two(14 - e);
                f *= power_of_two(e - 14);
#pragma unroll
                for (int s = 0; s < F::kSteps; ++s)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const T* const x = reinterpret_cast<const T*>(&qf[nt][s][k]);
                        qf[nt][s][k] = Elem<__half>::pack(Elem<T>::to_float(x[0]) * by, Elem<T>::to_float(x[1]) * by);
                    }
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                factor[nt][k] = __shfl_sync(0xFFFFFFFFu, f, (2 * c + k) * 4);
                const int32_t rr = nt * 8 + 2 * c + k;
                tok[nt][k] = rr < nrows ? old + (int32_t)p.by_group.div((uint32_t)(row0 + rr)) : -1;
                ref[nt][k] = kNone;
                l[nt][k] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < F::kSteps; ++j) o[nt][j][0] = o[nt][j][1] = o[nt][j][2] = o[nt][j][3] = 0.f;
        }
    }

    // The chunk at key0 whose K rows are at kt and V rows behind them.
    __device__ __forceinline__ void chunk(const WindowParams& p, uint32_t kt, int32_t key0, ChunkInfo info) {
        const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
        const int ta = (g >> 1) + 4 * (g & 1);
        float sc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
#pragma unroll
        for (int i = 0; i < F::kPieces / 4; ++i) {
            const uint4 a = lds128(kt + F::place(ta, c + 4 * i)), b = lds128(kt + F::place(ta + 8, c + 4 * i));
            const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
            if constexpr (F::kCodes) {
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const uint32_t k[4] = {codes_to_half2((uint16_t)aw[w]), codes_to_half2((uint16_t)bw[w]),
                                           codes_to_half2((uint16_t)(aw[w] >> 16)), codes_to_half2((uint16_t)(bw[w] >> 16))};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma16816<M>(sc[nt], k, qf[nt][i * 4 + w][0], qf[nt][i * 4 + w][1]);
                }
            } else {
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const uint32_t k[4] = {aw[2 * w], bw[2 * w], aw[2 * w + 1], bw[2 * w + 1]};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma16816<M>(sc[nt], k, qf[nt][i * 2 + w][0], qf[nt][i * 2 + w][1]);
                }
            }
        }
        // scores to powers of 2
        float k_scale[2] = {1.f, 1.f}, v_power[2] = {0.f, 0.f}, v_back[2] = {1.f, 1.f};
        if constexpr (F::kCodes) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                // 2^(byte - 127), byte - 127 and 2^(127 - byte) by their bits (2^-127 is not a normal number)
                const uint32_t kb = (info.scales >> (16 * i)) & 0xFF, vb = max((info.scales >> (16 * i + 8)) & 0xFF, kLeastScale);
                k_scale[i] = __uint_as_float(max(kb << 23, 0x00400000u));
                v_power[i] = __uint_as_float(0x4B000000u | vb) - (8388608.f + 127.f);
                v_back[i] = __uint_as_float(max((254u - vb) << 23, 0x00400000u));
            }
            // a scale of NaN makes its keys' exponents NaN
            if (__any_sync(0xFFFFFFFFu, __vcmpeq4(info.scales, 0xFFFFFFFFu) != 0u)) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (((info.scales >> (16 * i)) & 0xFF) == 0xFF || ((info.scales >> (16 * i + 8)) & 0xFF) == 0xFF)
                        v_power[i] = NAN, v_back[i] = 1.f;
            }
        }
        const bool whole = info.mask == 0xFFFFu && key0 + kChunk - 1 <= t_first &&
                           (p.window == INT32_MAX || key0 > t_last - p.window || key0 + kChunk <= p.sinks);
        bool grow = false;
        float d[NT][4];            // what the weights are powers of
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = i & 1, row = i >> 1;
                float& x = sc[nt][i];
                x = F::kCodes ? fmaf(x, factor[nt][k] * k_scale[row], v_power[row]) : x * factor[nt][k];
                if (!whole) {
                    const int32_t j = key0 + ta + 8 * row, t = tok[nt][k];
                    const bool see = ((info.mask >> (ta + 8 * row)) & 1) && j <= t &&
                                     (p.window == INT32_MAX || j > t - p.window || j < p.sinks);
                    if (!see) x = -INFINITY;
                }
                d[nt][i] = x - ref[nt][k];
                grow = grow || d[nt][i] > kBelow + kLag;
            }
        if (__any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float top = fmaxf(sc[nt][k], sc[nt][2 + k]);
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 4));
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 8));
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16));
                    const float to = fmaxf(ref[nt][k], top - kBelow);
                    const float f = exp2_fast(ref[nt][k] - to);
                    ref[nt][k] = to;
                    l[nt][k] *= f;
                    d[nt][k] = sc[nt][k] - to;
                    d[nt][2 + k] = sc[nt][2 + k] - to;
#pragma unroll
                    for (int j = 0; j < F::kSteps; ++j) {
                        o[nt][j][k] *= f;
                        o[nt][j][2 + k] *= f;
                    }
                }
        }
        uint32_t pf[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[i] = exp2_fast(d[nt][i]);
                l[nt][i & 1] = F::kCodes ? fmaf(w[i], v_back[i >> 1], l[nt][i & 1]) : l[nt][i & 1] + w[i];
            }
            // weights are rounded to 16 bits for the product with V, the sum takes them whole
            pf[nt][0] = transposed(Elem<M>::pack(w[0], w[1]));
            pf[nt][1] = transposed(Elem<M>::pack(w[2], w[3]));
        }
        const uint32_t vt = kt + F::kTileBytes;
        auto product = [&](int j, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
            const uint32_t a[4] = {a0, a1, a2, a3};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816<M>(o[nt][j], a, pf[nt][0], pf[nt][1]);
        };
        if constexpr (F::kCodes) {
            constexpr int kWords = D / 32;
            uint32_t v[4][kWords];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (D == 128) {
                    const uint4 x = lds128(vt + F::place(c + 4 * i, g));
                    v[i][0] = x.x, v[i][1] = x.y, v[i][kWords - 2] = x.z, v[i][kWords - 1] = x.w;
                } else {
                    const uint2 x = lds64(vt + F::place(c + 4 * i, g >> 1) + (g & 1) * 8);
                    v[i][0] = x.x, v[i][1] = x.y;
                }
            }
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint32_t sel = u ? 0x7362u : 0x5140u;
                    const uint32_t x = prmt(v[0][w], v[1][w], sel), y = prmt(v[2][w], v[3][w], sel);
                    product(2 * w + u, codes_to_half2((uint16_t)x), codes_to_half2((uint16_t)(x >> 16)),
                            codes_to_half2((uint16_t)y), codes_to_half2((uint16_t)(y >> 16)));
                }
            }
        } else {
#pragma unroll
            for (int piece = 0; piece < D / 64; ++piece) {
                uint32_t v[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 x = lds128(vt + F::place(c + 4 * i, g + 8 * piece));
                    v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
                }
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    product(piece * 4 + w, prmt(v[0][w], v[1][w], 0x5410), prmt(v[0][w], v[1][w], 0x7632),
                            prmt(v[2][w], v[3][w], 0x5410), prmt(v[2][w], v[3][w], 0x7632));
            }
        }
    }

    // This stream's part of the rows.
    __device__ __forceinline__ void end(const WindowParams& p, int32_t stream, int32_t tile_no, int32_t h, int32_t nrows) {
        const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float s = l[nt][k];
                s += __shfl_xor_sync(0xFFFFFFFFu, s, 4);
                s += __shfl_xor_sync(0xFFFFFFFFu, s, 8);
                s += __shfl_xor_sync(0xFFFFFFFFu, s, 16);
                const int32_t rr = nt * 8 + 2 * c + k;
                if (rr >= nrows) continue;
                const int64_t at = p.own_part(stream, tile_no, rr, h);
                if (g == 0) p.part_ml[at] = make_float2(ref[nt][k] == kNone ? -INFINITY : ref[nt][k], s);
                float* const row = p.part_o + at * D;
#pragma unroll
                for (int j = 0; j < F::kSteps; j += 2)
                    *reinterpret_cast<float4*>(row + F::element(j, g)) =
                        make_float4(o[nt][j][k], o[nt][j][2 + k], o[nt][j + 1][k], o[nt][j + 1][2 + k]);
            }
    }
};

// (128 KB of an SM's shared memory are taken at most: behind a kernel that needs less of it, as the join, a launch that
// depends on it did not get its blocks beside one another.  64 users of 1000 to 9000 tokens, 8 bits, 16 warps an SM: rings of
// three, 192 KB, 124 us by themselves and 198 in a row, of two, 128 KB, 123 in a row.  48 users with a window of 4096, 16 bits: 12 warps
// an SM, 192 KB, 135 us, 8 warps, 128 KB, 114.)
template <class KV, int D, int NT>
struct StreamShape {
    static constexpr int kTile = Fragments<KV, D>::kTileBytes;             // 1, 2 or 4 KB
    static constexpr int kStages = kTile >= 2048 ? 2 : 4;
    static constexpr int kWarpBytes = kStages * 2 * kTile;
    static constexpr int kSmem = kWarps * kWarpBytes;
    static constexpr int kCtas = kTile >= 4096 ? 2 : NT > 1 ? 3 : 4;       // an SM
};

// The chunks of all small requests' row tiles, one after the other, are shared
// equally among warps, whatever the lengths are; a warp runs through its share by itself, with
// no barrier, a ring of its own in shared memory filled by cp.async, and leaves a partial result for each row
// tile that it had some of.  Stream s of KV head h is warp s * kv_heads + h: the heads' warps of the same tokens run
// side by side and read the same pages' rows.  Bound by the bytes of the pages (with the join: 64 users of 1000 to 9000
// tokens, 8 bits, 125 us, 5.3 TB/s; 48 users with a window of 4096, 16 bits, 115 us, 6.2 TB/s).
template <class T, class KV, int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, StreamShape<KV, D, NT>::kCtas)
window_streams_kernel(const __grid_constant__ WindowParams p) {
    using X = StreamRows<T, KV, D, NT>;
    using F = Fragments<KV, D>;
    using Sh = StreamShape<KV, D, NT>;
    extern __shared__ __align__(1024) uint8_t smem[];
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t worker = blockIdx.x * kWarps + warp, stream = worker / p.kv_heads, h = worker - stream * p.kv_heads;
    if (stream >= p.streams) return;
    if (worker == 0 && lane == 0 && p.next_item != nullptr) *p.next_item = 0;
    const uint32_t ring = smem_u32(smem) + warp * Sh::kWarpBytes;
    const int32_t group = (int32_t)p.by_group.d;
    const uint8_t* const base = p.layer.base();
    const uint8_t* const scales = F::kCodes ? p.scales.base() : nullptr;
    const bool there = base != nullptr && (!F::kCodes || scales != nullptr);
    if (!there && worker == 0 && lane == 0) report(p.status, LMKV_ERR_BAD_POINTER);
    auto tiles_of = [&](const Req& r) {
        const int32_t n = r.n * group;
        return n >= p.big_rows ? 0 : (n + NT * 8 - 1) / (NT * 8);
    };
    auto seen_of = [&](const Req& r, int32_t tile) {
        const int32_t old = r.len - r.n, row0 = tile * NT * 8, row1 = min(row0 + NT * 8, r.n * group) - 1;
        return seen_by(p, old + (int32_t)p.by_group.div((uint32_t)row0), old + (int32_t)p.by_group.div((uint32_t)row1), kChunk);
    };
    // The tiles of a request see nearly the same keys: its units are the last tile's, which are at least as many.
    auto units_of = [&](const Req& r, int32_t tiles) {
        int32_t most = 0;
        if (tiles > 0) most = seen_of(r, tiles - 1).units;
        for (int32_t i = 0; i + 1 < tiles; ++i) most = max(most, seen_of(r, i).units);
        return most;
    };
    Share share = find_share(p.seqs.num_req, stream, p.streams, [&](int32_t i) -> int64_t {
        const Req r = load_req(p.seqs, i);
        if (!r.ok) report(p.status, LMKV_ERR_BAD_LENGTH);
        const int32_t tiles = tiles_of(r);
        return (int64_t)tiles * units_of(r, tiles);
    });
    X x;
    while (share.n > 0 && share.r < p.seqs.num_req) {
        const Req r = load_req(p.seqs, share.r);
        const int32_t tiles = tiles_of(r), units = units_of(r, tiles);
        const int32_t tile = units > 0 ? (int32_t)(share.first / units) : 0;
        if (units == 0 || tile >= tiles) {
            ++share.r;
            share.first = 0;
            continue;
        }
        const int32_t u0 = (int32_t)(share.first - (int64_t)tile * units);
        const int32_t n = (int32_t)min((int64_t)(units - u0), share.n);
        share.first += n;
        share.n -= n;
        const int32_t tile_no = share.r * p.own_tiles + tile, row0 = tile * NT * 8, nrows = r.n * group - row0;
        if (h == 0 && lane == 0) {
            if (u0 == 0) p.own_range[tile_no].x = stream;
            if (u0 + n == units) p.own_range[tile_no].y = stream;
        }
        const Seen seen = seen_of(r, tile);
        const int32_t u1 = there ? min(u0 + n, seen.units) : u0;
        ChunkLoad<KV, D> load(p, p.seqs.table + (int64_t)share.r * p.seqs.table_stride, base, scales, h, seen);
        ChunkInfo info[Sh::kStages];
        auto fill = [&](int32_t u) { return load.copy(u, ring + (u - u0) % Sh::kStages * (2 * F::kTileBytes), u1); };
        __syncwarp();
        load.lookup(u0, u1);
#pragma unroll
        for (int s = 0; s < Sh::kStages - 1; ++s) {
            info[s] = u0 + s < u1 ? fill(u0 + s) : ChunkInfo{0, 0};
            cp_commit();
        }
        x.begin(p, r, h, row0, nrows);
        for (int32_t b = u0; b < u1; b += Sh::kStages) {
#pragma unroll
            for (int s = 0; s < Sh::kStages; ++s) {
                const int32_t u = b + s;
                if (u >= u1) break;
                __syncwarp();      // the stage filled next was read by every lane
                constexpr int kAhead = Sh::kStages - 1;
                info[(s + kAhead) % Sh::kStages] = u + kAhead < u1 ? fill(u + kAhead) : ChunkInfo{0, 0};
                cp_commit();
                cp_wait<kAhead>();
                __syncwarp();
                x.chunk(p, ring + s * (2 * F::kTileBytes), seen.unit(u) * kChunk, info[s]);
            }
        }
        cp_wait<0>();
        x.end(p, stream, tile_no, h, nrows);
    }
}

// Joins the parts of rows that have them: of the small requests' rows (kTiles false: a
// stream's parts each) or of the big ones' (the tile kernel's parts).  kRowWarps warps a row: one where there are many rows, of few parts
// each, and all of a CTA's where few rows have many.  (One request of 131072 tokens, 8 heads on one KV head: 214 us in all
// with a warp a row, 33 with a CTA.)  Bound by waits for the parts, a load or two a warp.
template <class T, int D, bool kTiles, int kRowWarps>
__global__ void __launch_bounds__(kRowWarps == 1 ? 256 : kRowWarps * 32) window_join_kernel(const __grid_constant__ WindowParams p) {
    constexpr int kPer = D / 32;
    constexpr int kGroup = kRowWarps == 1 ? 32 : 8;        // parts at a time
    __shared__ float sums[kRowWarps == 1 ? 1 : kRowWarps][kRowWarps == 1 ? 1 : D];
    __shared__ float2 tops[kRowWarps];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = kRowWarps == 1 ? 0 : threadIdx.x >> 5;
    const int32_t group = (int32_t)p.by_group.d;
    int64_t i = kRowWarps == 1 ? (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
    int32_t tok, head, parts;
    int64_t first, stride;
    if constexpr (kTiles) {
        if (i >= p.rows) return;
        tok = (int32_t)(i / p.q_heads), head = (int32_t)(i - (int64_t)tok * p.q_heads);
        const Req q = load_req(p.seqs, find_request(p.seqs.num_req, tok, [&](int32_t k) { return p.seqs.q_start[k]; }));
        if (tok < q.q0 || tok >= q.q0 + q.n || q.n * group < p.big_rows) return;
        first = i, stride = p.rows, parts = p.parts;
    } else {
        if (i >= (int64_t)p.seqs.num_req * p.own_cap * p.kv_heads) return;
        const int32_t h = (int32_t)(i % p.kv_heads);
        i /= p.kv_heads;
        const int32_t r = (int32_t)(i / p.own_cap), row = (int32_t)(i % p.own_cap);
        const Req q = load_req(p.seqs, r);
        if (row >= q.n * group || q.n * group >= p.big_rows) return;
        const int32_t n = (int32_t)p.by_group.div((uint32_t)row);
        tok = q.q0 + n, head = h * group + (row - n * group);
        // streams g, g + 1, .. have some of the row's tile (clamped: lengths that change while the call
        // runs give a wrong sum, not a wild address); a request of no keys has none
        const int32_t tile_no = r * p.own_tiles + row / p.tile_rows;
        int32_t g = 0;
        parts = 0;
        if (q.len > 0) {
            const int2 range = p.own_range[tile_no];
            g = min(max(range.x, 0), p.streams - 1);
            parts = min(max(range.y, g), p.streams - 1) - g + 1;
        }
        first = p.own_part(g, tile_no, row % p.tile_rows, h);
        stride = (int64_t)p.tile_rows * p.kv_heads;
    }
    // m and l of some parts at a time, one a lane; then the parts' sums, whose loads
    // do not wait for one another
    float top = -INFINITY, sum = 0.f, acc[kPer] = {};
    for (int32_t s0 = warp * kGroup; s0 < parts; s0 += kGroup * kRowWarps) {
        const int32_t n = min(kGroup, parts - s0);
        const float2 v = lane < n ? p.part_ml[first + (s0 + lane) * stride] : make_float2(-INFINITY, 0.f);
        constexpr int kAhead = 8;
        float x[kAhead][kPer];
        auto load = [&](int32_t s) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const float* src = p.part_o + (first + min(s0 + s + u, parts - 1) * stride) * D + lane * kPer;
                if constexpr (kPer == 4) *reinterpret_cast<float4*>(x[u]) = *reinterpret_cast<const float4*>(src);
                else *reinterpret_cast<float2*>(x[u]) = *reinterpret_cast<const float2*>(src);
            }
        };
        load(0);
        float mn = v.x;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, d));
        mn = fmaxf(mn, top);
        const float mu = mn == -INFINITY ? 0.f : mn;
        const float f = exp2_fast(v.x - mu), before = exp2_fast(top - mu);
        top = mn;
        float l = v.y * f;             // (a NaN stays one)
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
        sum = sum * before + l;
#pragma unroll
        for (int k = 0; k < kPer; ++k) acc[k] *= before;
        for (int32_t s = 0; s < n; s += kAhead) {
            if (s > 0) load(s);
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const float fs = __shfl_sync(0xFFFFFFFFu, f, (s + u) & 31);
                if (s + u < n && fs != 0.f) {        // (a part of no keys has written no sums)
#pragma unroll
                    for (int k = 0; k < kPer; ++k) acc[k] += x[u][k] * fs;
                }
            }
        }
    }
    if constexpr (kRowWarps > 1) {
        if (lane == 0) tops[warp] = make_float2(top, sum);
#pragma unroll
        for (int k = 0; k < kPer; ++k) sums[warp][lane * kPer + k] = acc[k];
        __syncthreads();
        if (warp != 0) return;
        const float2 v = lane < kRowWarps ? tops[lane] : make_float2(-INFINITY, 0.f);
        top = v.x;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        const float f = exp2_fast(v.x - (top == -INFINITY ? 0.f : top));
        sum = v.y * f;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
#pragma unroll
        for (int k = 0; k < kPer; ++k) acc[k] = 0.f;
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) {
            const float fw = __shfl_sync(0xFFFFFFFFu, f, w);
#pragma unroll
            for (int k = 0; k < kPer; ++k) acc[k] += sums[w][lane * kPer + k] * fw;
        }
    }
    const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
    T* dst = p.out.row<T>(tok, head) + lane * kPer;
#pragma unroll
    for (int k = 0; k < kPer; ++k) dst[k] = Elem<T>::from_float(acc[k] * inv);
    if (lane == 0 && p.lse != nullptr)
        p.lse[(int64_t)tok * p.q_heads + head] = ((top == -INFINITY ? 0.f : top) + log2f(sum)) * kLn2;
}

// ---- tiles of 128 rows on the tensor core -------------------------------

using namespace lmkv_tc;

constexpr int kTileRows = 256;        // two tiles of 128 rows share every K and V block
constexpr int kLoaders = 6;           // warps that bring K and V
// Registers of a softmax thread and of the others: 256 of each share the launch's 512 x 128.
constexpr int kSoftmaxRegs = 192, kOtherRegs = 64;
static_assert(kSoftmaxRegs + kOtherRegs == 2 * 128, "what one half gives, the other takes");
constexpr int kTileThreads = (8 + kLoaders + 2) * 32;
constexpr int kUnits = kBlock / kChunk;         // of 16 keys, in a block
constexpr int kInfoSlots = 8;

template <int D>
struct WindowTile {
    static constexpr int kHalfBytes = BlockShape<D>::kHalfBytes;
    static constexpr int kStageBytes = BlockShape<D>::kBytes;      // 128 rows of K, V or q in 16 bits
    static constexpr int kStages = D == 128 ? 5 : 8;
    static constexpr int kSmem = (2 + kStages) * kStageBytes;
};

// 256 rows of a request and KV head, or a part of their keys.
struct Item {
    int32_t h;               // KV head; -1: there are no more items
    int32_t q0, n, old;      // the request's first row, new tokens, and tokens before them
    int32_t row0;            // the first of the 256 rows
    int32_t b0, b1;          // blocks of the keys that its rows see
    int32_t part;
    const int32_t* table;
    Seen seen;
};
constexpr int kItems = 4;    // on their way

// Rows of one request, (token, head of the group) in token order, 256 at a time,
// against the keys that they see, in blocks of 128.  Products and powers are both near their limits, so the two
// tiles of 128 rows take turns: while the tensor core works on one tile's
// weights x V and next q x K, the other tile's softmax runs.
//   warps 0-3, 4-7   softmax of tile 0, 1: a thread holds a row.  Scores come
//                    from tensor memory, weights go back over them as the next
//                    product's first operand; the output stays in tensor memory until the end.
//   warps 8-13       K and V in units of 16 rows (one page's) into a ring in shared memory that
//                    both tiles read: codes through registers, where they become fp16, 16-bit rows by cp.async
//   warp 14          takes the next items, looks up what they are, and of their blocks the pages and scales
//   warp 15          one thread issues every product
// A CTA an SM goes from item to item, whichever is next (what comes of them does not depend on who takes
// them).  K and V of the next are on their way while the last products run, and its q while the output is
// written: by themselves, with their first loads and their output waited for, items of ten blocks took 53,000 cycles of
// which 18,000 were that.
// A unit's scales are the same for its 16 keys: a factor and an addend of the exponent's multiply-add.
// Tensor memory: scores of tile 0, 1 at columns 0, 128; outputs at 256, 384.
// Bound by the softmax's instructions between two products.  (4 prompts of 65 to 1200 tokens behind 1500 to 8000 on an
// 8-bit cache, 64 heads: 351 us, 1.05 PFLOP/s.)
template <class T, class KV, int D>
__global__ void __launch_bounds__(kTileThreads, 1)
window_tiles_kernel(const __grid_constant__ WindowParams p) {
    constexpr bool kCodes = sizeof(KV) == 1;
    using S = WindowTile<D>;
    using M = typename std::conditional<kCodes, __half, T>::type;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ uint64_t bars[2 * S::kStages + 8 + 2 * kItems + 2 * kInfoSlots];
    __shared__ uint32_t tmem_base;
    __shared__ int gave_up;
    __shared__ Item items[kItems];
    __shared__ uint2 infos[kInfoSlots][kUnits];      // of a block's units: first row of the K half, which of its rows there are
    __shared__ __align__(16) uint16_t masks[kInfoSlots][kUnits];      // which of a unit's keys there are
    __shared__ float4 powers[kCodes ? kInfoSlots : 1][kUnits];        // its scale of K; V's as power, and inverse
    pdl_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t full = smem_u32(bars), empty = full + 8 * S::kStages, s_full = empty + 8 * S::kStages,
                   p_ready = s_full + 16, o_full = p_ready + 32, item_full = o_full + 16,
                   item_empty = item_full + 8 * kItems, info_full = item_empty + 8 * kItems,
                   info_empty = info_full + 8 * kInfoSlots;
    const uint32_t q_smem = smem_u32(smem), kv_smem = q_smem + 2 * S::kStageBytes;
    if (tid == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(full + 8 * i, kCodes ? kUnits : kUnits * 33);
            mbar_init(empty + 8 * i, 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(s_full + 8 * t, 1);
            mbar_init(p_ready + 16 * t, 4);
            mbar_init(p_ready + 16 * t + 8, 4);
            mbar_init(o_full + 8 * t, 1);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(item_full + 8 * i, 1);
            mbar_init(item_empty + 8 * i, 8 + kLoaders + 1);
        }
        for (int i = 0; i < kInfoSlots; ++i) {
            mbar_init(info_full + 8 * i, 1);
            mbar_init(info_empty + 8 * i, 1);
        }
        gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8 + kLoaders + 1) tmem_alloc<512>(smem_u32(&tmem_base));
    pdl_wait();
    const int32_t group = (int32_t)p.by_group.d;
    uint8_t* const base = p.layer.base();
    const uint8_t* const scales = kCodes ? p.scales.base() : nullptr;
    const bool there = base != nullptr && (!kCodes || scales != nullptr);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    // The it-th item of this CTA, once it is known; its place is free again when all warps but the one that takes
    // items have read it.
    auto get = [&](int32_t it, Item& x) {
        const int slot = it % kItems;
        if (!mbar_wait(item_full + 8 * slot, it / kItems & 1, &gave_up)) return false;
        x = items[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(item_empty + 8 * slot);
        return x.h >= 0;
    };
    // (Stages of the ring are counted on from item to item, K and V of a block in turn.)
    {
        if (warp < 8) {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
            const int t = warp >> 2;
            const uint32_t lane_base = tmem_base + ((uint32_t)(warp & 3) << 21);     // lane 32 * (warp % 4)
            const uint32_t s_at = lane_base + t * 128, o_at = lane_base + 256 + t * 128;
            const uint32_t dst = q_smem + t * S::kStageBytes + (warp & 3) * (32 * 128);
            constexpr int kRowLanes = D / 8, kSide = 32 / kRowLanes;
            const int piece = lane % kRowLanes;
            float m = -INFINITY;              // the maximum (lagging), in powers of 2
            float2 l2 = make_float2(0.f, 0.f);
            // of the item before: my row, whose result is still to be written
            int32_t row_tok = -1, row_head = 0, row_part = 0, last_block = -1;
            bool row_left = false, row_blocks = false;
            uint32_t blocks_before = 0, scores_phase = 0, out_phase = 0;
            auto finish = [&] {
                row_left = false;
                if (row_blocks) {
                    if (!mbar_wait(o_full + 8 * t, out_phase, &gave_up)) return false;
                    out_phase ^= 1;
                    fence_after_sync();
                    if (last_block >= 0 && (tid & 127) == 0) {
                        mbar_arrive(empty + 8 * ((2 * (uint32_t)last_block + 1) % S::kStages));
                        mbar_arrive(info_empty + 8 * (last_block % kInfoSlots));
                    }
                }
                const float l = l2.x + l2.y;
                const bool final = p.parts == 1, live = row_tok >= 0;
                const int64_t row = (int64_t)(live ? row_tok : 0) * p.q_heads + row_head;
                const int64_t at = (int64_t)row_part * p.rows + row;
                const float ref = m == -INFINITY ? -INFINITY : m - kBelow;
                const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
                T* const to = p.out.row<T>(live ? row_tok : 0, row_head);
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                    uint32_t y[16];
                    if (row_blocks) {
                        tmem_ld16(y, o_at + c);
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) y[j] = 0u;
                    }
                    if (live && final) {
                        // (a lane writes 32 bytes of its row at once: rows lie apart, and every part of one takes its own turn)
                        uint32_t w[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            w[i] = Elem<T>::pack(__uint_as_float(y[2 * i]) * inv, __uint_as_float(y[2 * i + 1]) * inv);
                        if (p.out_wide) {
                            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to + c), "r"(w[0]),
                                         "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
                        } else {
                            uint16_t* const e = reinterpret_cast<uint16_t*>(to + c);
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                e[2 * i] = (uint16_t)w[i];
                                e[2 * i + 1] = (uint16_t)(w[i] >> 16);
                            }
                        }
                    } else if (live) {
#pragma unroll
                        for (int j = 0; j < 16; j += 4)
                            *reinterpret_cast<uint4*>(p.part_o + at * D + c + j) = make_uint4(y[j], y[j + 1], y[j + 2], y[j + 3]);
                    }
                }
                if (live && final && p.lse != nullptr) p.lse[row] = ((m == -INFINITY ? 0.f : ref) + log2f(l)) * kLn2;
                if (live && !final) p.part_ml[at] = make_float2(ref, l);
                return true;
            };
            bool ok = true;
            for (int32_t it = 0; ok; ++it) {
                Item item;
                const bool some = get(it, item);
                const int32_t req_rows = item.n * group;
                const int tiles = min(item.row0 + kTileRows, req_rows) - item.row0 > 128 ? 2 : 1;
                const bool mine = some && t < tiles;
                const int32_t blocks = some ? item.b1 - item.b0 : 0;
                if (mine) {
                // The warp's rows of q into shared memory, 16 bytes a lane side by side.  (This and the end run once,
                // out of memory that holds no instructions of theirs any more: loops, not lines, keep them
                // short.  Unrolled, the rows took 31,000 cycles.)
                // (no product reads the last item's any more: its scores were all there)
                auto row_at = [&](int i, int32_t& token, int32_t& hd) {      // the i-th row of this lane's; its place in dst
                    const int r = i * kSide + lane / kRowLanes;
                    const int32_t at = item.row0 + warp * 32 + r;
                    const int32_t of = (int32_t)p.by_group.div((uint32_t)at);
                    token = at < req_rows ? item.q0 + of : -1;
                    hd = item.h * group + (at - of * group);
                    return dst + (piece >> 3) * S::kHalfBytes + r * 128 + (((piece & 7) ^ (r & 7)) << 4);
                };
#pragma unroll 1
                for (int i = 0; i < kRowLanes; ++i) {
                    int32_t token, hd;
                    const uint32_t at = row_at(i, token, hd);
                    const bool on = token >= 0 && p.scale_sign != 0;
                    const T* const src = p.q.row<T>(on ? token : item.q0, hd) + piece * 8;
                    if (p.q_vec) {
                        cp_async16(at, src, on);
                    } else {
                        uint4 v = make_uint4(0u, 0u, 0u, 0u);
                        if (on) v = make_uint4(load_pair(src, p.q_pairs), load_pair(src + 2, p.q_pairs),
                                               load_pair(src + 4, p.q_pairs), load_pair(src + 6, p.q_pairs));
                        sts128(at, v);
                    }
                }
                cp_commit();
                }
                if (row_left) ok = finish();
                if (!some || !ok) break;
                if (mine) {
                cp_wait<0>();
                __syncwarp();
                float factor = p.scale_log2;
                auto my_piece = [&](int c) { return dst + (c >> 3) * S::kHalfBytes + lane * 128 + (((c & 7) ^ (lane & 7)) << 4); };
                if (kCodes || p.scale_sign < 0) {
                    // my row: negated for a negative scale, and beside codes as fp16 with its largest element
                    // between 2^14 and 2^15
                    float by = p.scale_sign < 0 ? -1.f : 1.f;
                    if constexpr (kCodes) {
                        float top = 0.f;
#pragma unroll 1
                        for (int c = 0; c < kRowLanes; ++c) {
                            const uint4 v = lds128(my_piece(c));
                            const T* const e = reinterpret_cast<const T*>(&v);
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const float a = fabsf(Elem<T>::to_float(e[j]));
                                if (a < INFINITY) top = fmaxf(top, a);
                            }
                        }
                        const int x = top > 0.f ? max((int)(__float_as_uint(top) >> 23) - 127, -100) : 0;
                        by *= power_of_two(14 - x);
                        factor *= power_of_two(x - 14);
                    }
#pragma unroll 1
                    for (int c = 0; c < kRowLanes; ++c) {
                        const uint4 v = lds128(my_piece(c));
                        const T* const e = reinterpret_cast<const T*>(&v);
                        sts128(my_piece(c), make_uint4(Elem<M>::pack(Elem<T>::to_float(e[0]) * by, Elem<T>::to_float(e[1]) * by),
                                                       Elem<M>::pack(Elem<T>::to_float(e[2]) * by, Elem<T>::to_float(e[3]) * by),
                                                       Elem<M>::pack(Elem<T>::to_float(e[4]) * by, Elem<T>::to_float(e[5]) * by),
                                                       Elem<M>::pack(Elem<T>::to_float(e[6]) * by, Elem<T>::to_float(e[7]) * by)));
                    }
                }
                fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_ready + 16 * t + 8);     // its phase 0: q is there

                const int32_t R = item.row0 + tid;
                const bool live = R < req_rows;
                const int32_t n = (int32_t)p.by_group.div((uint32_t)(live ? R : item.row0));
                // my row sees keys below end, from begin on or below the sinks
                const int32_t end = live ? item.old + n + 1 : 0, begin = first_in_window(p, end - 1);
                m = -INFINITY;
                l2 = make_float2(0.f, 0.f);
                row_left = true;
                row_tok = live ? item.q0 + n : -1;
                row_head = item.h * group + ((live ? R : item.row0) - n * group);
                row_part = item.part;
                row_blocks = blocks > 0;
                last_block = t == tiles - 1 ? (int32_t)(blocks_before + blocks) - 1 : -1;
                for (int32_t j = 0; j < blocks; ++j) {
                    const int32_t k = item.seen.unit(item.b0 + j) * kBlock;
                    if (!mbar_wait(s_full + 8 * t, scores_phase, &gave_up)) {
                        ok = false;
                        break;
                    }
                    scores_phase ^= 1;
                    if (t == tiles - 1 && (tid & 127) == 0) {
                        // every product up to these scores is done: K of this block and V of the last are free
                        const uint32_t kv = (blocks_before + j) * 2;
                        mbar_arrive(empty + 8 * (kv % S::kStages));
                        if (j > 0) {
                            mbar_arrive(empty + 8 * ((kv - 1) % S::kStages));
                            mbar_arrive(info_empty + 8 * ((blocks_before + j - 1) % kInfoSlots));
                        }
                    }
                    fence_after_sync();
                    const int slot_of = (blocks_before + j) % kInfoSlots;
                    const uint4 words = *reinterpret_cast<const uint4*>(masks[slot_of]);
                    const bool whole = __all_sync(0xFFFFFFFFu, end - k >= kBlock && (begin <= k || k + kBlock <= p.sinks)) &&
                                       (words.x & words.y & words.z & words.w) == ~0u;
                    // scores of 32 keys, those not seen as -infinity
                    auto below = [](int32_t n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u; };
                    auto take = [&](uint32_t (&x)[32], int i) {
                        if (whole) return;
                        const int32_t at = k + 32 * i;
                        const uint32_t bits = (i == 0 ? words.x : i == 1 ? words.y : i == 2 ? words.z : words.w) &
                                              below(end - at) & (~below(begin - at) | below(p.sinks - at));
                        if (__all_sync(0xFFFFFFFFu, bits == ~0u)) return;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!((bits >> e) & 1)) x[e] = 0xFF800000u;
                    };
                    // a unit's factor (never 0: -infinity is to stay that)
                    auto factor_of = [&](const float4& u) { return kCodes ? fmaxf(factor * u.x, 0x1p-126f) : factor; };
                    auto powers_of = [&](int u) {
                        return kCodes ? powers[kCodes ? slot_of : 0][u] : make_float4(1.f, 0.f, 1.f, 0.f);
                    };
                    uint32_t x[4][32];
                    float mx = -INFINITY;
                    tmem_ld32(x[0], s_at);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 of[2] = {powers_of(2 * i), powers_of(2 * i + 1)};
                        wait_ld();
                        loaded(x[i]);
                        if (i < 3) tmem_ld32(x[i + 1], s_at + 32 * (i + 1));
                        take(x[i], i);
                        if constexpr (kCodes) {
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                float a = -INFINITY, c = -INFINITY;
#pragma unroll
                                for (int j = 16 * u; j < 16 * u + 16; j += 4) {
                                    a = max3(a, __uint_as_float(x[i][j]), __uint_as_float(x[i][j + 1]));
                                    c = max3(c, __uint_as_float(x[i][j + 2]), __uint_as_float(x[i][j + 3]));
                                }
                                mx = fmaxf(mx, fmaf(fmaxf(a, c), factor_of(of[u]), of[u].y));
                            }
                        } else {
                            float a = -INFINITY, c = -INFINITY;
#pragma unroll
                            for (int j = 0; j < 32; j += 4) {
                                a = max3(a, __uint_as_float(x[i][j]), __uint_as_float(x[i][j + 1]));
                                c = max3(c, __uint_as_float(x[i][j + 2]), __uint_as_float(x[i][j + 3]));
                            }
                            mx = fmaxf(mx, fmaxf(a, c));
                        }
                    }
                    if constexpr (!kCodes) mx *= factor;
                    // the output is rescaled when the maximum has grown by more than 2^kLag
                    const bool grow = mx > m + kLag;
                    if (__any_sync(0xFFFFFFFFu, grow)) {
                        const float f = grow ? exp2_fast(m - mx) : 1.f;
                        if (grow) m = mx;
                        l2.x *= f;
                        l2.y *= f;
                        if (j > 0) {
                            // the scores were there, so the product before them, into the output, is done
#pragma unroll 1
                            for (int c = 0; c < D; c += 16) tmem_scale16(o_at + c, f);
                        }
                    }
                    const float neg = m == -INFINITY ? 0.f : kBelow - m;
                    float4 next = powers_of(0);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t w[16];
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const float4 of = next;
                            if (2 * i + u + 1 < kUnits) next = powers_of(2 * i + u + 1);
                            const float f = factor_of(of), a = neg + of.y;
                            const float2 f2 = make_float2(f, f), a2 = make_float2(a, a);
                            float2 s0 = make_float2(0.f, 0.f), s1 = s0;
#pragma unroll
                            for (int j = 8 * u; j < 8 * u + 8; ++j) {
                                float2 e = fma2(make_float2(__uint_as_float(x[i][2 * j]), __uint_as_float(x[i][2 * j + 1])),
                                                f2, a2);
                                e.x = exp2_fast(e.x);
                                e.y = exp2_fast(e.y);
                                if (j & 1) s1 = add2(s1, e);
                                else s0 = add2(s0, e);
                                // weights are rounded to 16 bits for the product with V, the sum takes them whole
                                w[j] = Elem<M>::pack(e.x, e.y);
                            }
                            if constexpr (kCodes) {
                                l2 = fma2(add2(s0, s1), make_float2(of.z, of.z), l2);
                            } else {
                                l2 = add2(l2, add2(s0, s1));
                            }
                        }
                        tmem_st16(s_at + 16 * i, w);       // over scores that have been read
                        if (i & 1) {                       // 64 keys' weights are there
                            wait_st();
                            fence_before_sync();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(p_ready + 16 * t + 8 * (i >> 1));
                        }
                    }
                }
                }
                blocks_before += blocks;
            }
            if (row_left && ok) finish();
            cp_wait<0>();
        } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp < 8 + kLoaders) {
            // Unit u of an item is rows 16 (u % 8) .. of its u / 8-th stage (K, V of a block in turn); warp
            // 8 + i takes units i, i + kLoaders, ..
            const uint32_t row_bytes = (uint32_t)p.layer.row_bytes;
            const int64_t half_bytes = p.layer.half_bytes();
            constexpr int kRowBytes = D * (int)sizeof(KV), kPieces = kRowBytes / 16, kRowsPer = 32 / kPieces;
            constexpr int kCopies = kChunk / kRowsPer;
            const int c = lane % kPieces, rsub = lane / kPieces;
            uint32_t blocks_before = 0;
            bool ok = true;
            for (int32_t it = 0; ok; ++it) {
            const uint8_t* mine;
            int32_t all_units;
            {
                Item item;
                if (!get(it, item)) break;
                mine = base + (int64_t)item.h * kRowBytes + c * 16 + (int64_t)rsub * row_bytes;
                all_units = (item.b1 - item.b0) * 2 * kUnits;
            }
            // What there is to know of unit u, and where this lane's part of it is.
            struct Unit {
                uint32_t held;
                const uint8_t* src;
                __device__ __forceinline__ bool on(int row) const { return (held >> row) & 1; }
            };
            auto find = [&](int32_t u) {
                const uint32_t block = blocks_before + u / (2 * kUnits);
                ok = ok && mbar_wait(info_full + 8 * (block % kInfoSlots), (block / kInfoSlots) & 1, &gave_up);
                const uint2 x = infos[block % kInfoSlots][u % kUnits];
                return Unit{ok ? x.y : 0u, mine + (u / kUnits % 2 != 0 ? half_bytes : 0) + (uint64_t)x.x * row_bytes};
            };
            auto enter = [&](int32_t u) {      // the unit's stage is free
                const uint32_t kv = blocks_before * 2 + u / kUnits, st = kv % S::kStages;
                return kv < S::kStages || mbar_wait(empty + 8 * st, (kv / S::kStages - 1) & 1, &gave_up);
            };
            auto stage_of = [&](int32_t u) { return (blocks_before * 2 + u / kUnits) % S::kStages; };
            const int32_t u_first = warp - 8;
            if constexpr (kCodes) {
                // Registers that a part of a unit has left take that part of the warp's next.  (Prompts on an 8-bit cache: one unit at a time
                // 371 us, two in registers of their own, which spill, 395; by cp.async into the unit's own place, and from
                // there, 402, for shared memory's bandwidth.)
                // Of a lane's 16 codes the fp16 values are two pieces of a row: those of its two halves in turn, so
                // that they meet no bank twice; the other piece is the next or the one before, and rows r * kRowsPer
                // further exchange by the next bits.
                const bool odd = D == 128 && (c >> 2) != 0;
                const uint32_t first_piece = kv_smem + (D == 128 ? (c >> 2) * S::kHalfBytes : 0) + rsub * 128 +
                                             ((((2 * c + (odd ? 1 : 0)) & 7) ^ (rsub & 7)) << 4);
                uint4 codes[kCopies];
                auto load = [&](const Unit& x, int r) {
                    codes[r] = make_uint4(0u, 0u, 0u, 0u);
                    if (x.on(r * kRowsPer + rsub)) codes[r] = *reinterpret_cast<const uint4*>(x.src + r * kRowsPer * row_bytes);
                };
                if (u_first < all_units) {
                    const Unit x = find(u_first);
#pragma unroll
                    for (int r = 0; r < kCopies; ++r) load(x, r);
                }
#pragma unroll 1
                for (int32_t u = u_first; u < all_units; u += kLoaders) {
                    Unit next{0u, mine};
                    if (u + kLoaders < all_units) next = find(u + kLoaders);
                    ok = ok && enter(u);
                    if (!ok) break;
                    const uint32_t dst = stage_of(u) * S::kStageBytes + u % kUnits * (kChunk * 128);
#pragma unroll
                    for (int r = 0; r < kCopies; ++r) {
                        const uint4 v = codes[r];
                        const uint32_t w[4] = {odd ? v.z : v.x, odd ? v.w : v.y, odd ? v.x : v.z, odd ? v.y : v.w};
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            sts128(((first_piece ^ (i << 4)) ^ ((r * kRowsPer & 7) << 4)) + dst + r * (kRowsPer * 128),
                                   make_uint4(codes_to_half2((uint16_t)w[2 * i]), codes_to_half2((uint16_t)(w[2 * i] >> 16)),
                                              codes_to_half2((uint16_t)w[2 * i + 1]),
                                              codes_to_half2((uint16_t)(w[2 * i + 1] >> 16))));
                        load(next, r);
                    }
                    __syncwarp();
                    // (the products' thread has the writes seen by the tensor core, once for an item)
                    if (lane == 0) mbar_arrive(full + 8 * stage_of(u));
                }
            } else {
#pragma unroll 1
                for (int32_t u = u_first; u < all_units; u += kLoaders) {
                    ok = enter(u);
                    if (!ok) break;
                    const uint32_t stage = stage_of(u);
                    const uint32_t dst = kv_smem + stage * S::kStageBytes + u % kUnits * (kChunk * 128) + (c >> 3) * S::kHalfBytes;
                    const Unit x = find(u);
                    const bool all = (x.held & 0xFFFFu) == 0xFFFFu;
#pragma unroll
                    for (int r = 0; r < kCopies; ++r) {
                        const int i = r * kRowsPer + rsub;
                        const uint32_t at = dst + i * 128 + (((c & 7) ^ (i & 7)) << 4);
                        if (all) cp_async16(at, x.src + r * kRowsPer * row_bytes);
                        else cp_async16(at, x.on(i) ? x.src + r * kRowsPer * row_bytes : base, x.on(i));
                    }
                    copies_arrive(full + 8 * stage);
                }
            }
            blocks_before += all_units / (2 * kUnits);
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        } else if (warp == 8 + kLoaders) {
            // Where the requests are few: those with the most keys before others, lane r's row tiles from the
            // first_tile-th on.
            const bool sorted = p.seqs.num_req <= 32;
            int32_t tiles = 0, first_tile = 0, all_tiles = p.slots;
            if (sorted) {
                int32_t keys = -1;
                if (lane < p.seqs.num_req) {
                    const Req r = load_req(p.seqs, lane);
                    if (r.n * group >= p.big_rows) tiles = (r.n * group + kTileRows - 1) / kTileRows;
                    keys = r.len;
                }
                all_tiles = 0;
                for (int i = 0; i < 32; ++i) {
                    const int32_t t = __shfl_sync(0xFFFFFFFFu, tiles, i), k = __shfl_sync(0xFFFFFFFFu, keys, i);
                    if (k > keys || (k == keys && i < lane)) first_tile += t;
                    all_tiles += t;
                }
            }
            uint32_t blocks_before = 0;
            for (int32_t it = 0, next = blockIdx.x;; ) {
                Item x = {};
                x.h = -1;
                if (next < (int64_t)all_tiles * p.kv_heads * p.parts) {
                    const int32_t h = next % p.kv_heads;
                    const int32_t of = next / p.kv_heads, at = of % all_tiles;
                    int32_t r, req_rows;
                    Req req;
                    x.part = of / all_tiles;
                    // the last row tiles of a request see the most keys: they begin first
                    if (sorted) {
                        r = __ffs(__ballot_sync(0xFFFFFFFFu, at >= first_tile && at < first_tile + tiles)) - 1;
                        req = load_req(p.seqs, r);
                        req_rows = req.n * group;
                        x.row0 = (__shfl_sync(0xFFFFFFFFu, first_tile + tiles, r) - 1 - at) * kTileRows;
                    } else {
                        // slots q_start[r] * group / 256 + r and on are request r's row tiles
                        const int32_t slot = p.slots - 1 - at;
                        auto key = [&](int32_t i) { return (int32_t)((int64_t)max(p.seqs.q_start[i], 0) * group / kTileRows) + i; };
                        r = find_request(p.seqs.num_req, slot, key);
                        req = load_req(p.seqs, r);
                        req_rows = req.n * group;
                        x.row0 = slot >= key(r) ? (slot - key(r)) * kTileRows : req_rows;
                    }
                    int32_t taken = 0;
                    if (lane == 0) taken = atomicAdd(p.next_item, 1);
                    next = (int32_t)gridDim.x + __shfl_sync(0xFFFFFFFFu, taken, 0);
                    if (x.row0 >= req_rows || req_rows < p.big_rows) continue;       // a place of no rows
                    if (lane == 0) {
                        if (!req.ok) report(p.status, LMKV_ERR_BAD_LENGTH);
                        if (!there) report(p.status, LMKV_ERR_BAD_POINTER);
                    }
                    x.h = h;
                    x.q0 = req.q0;
                    x.n = req.n;
                    x.old = req.len - req.n;
                    x.table = p.seqs.table + (int64_t)r * p.seqs.table_stride;
                    const int32_t last = min(x.row0 + kTileRows, req_rows) - 1;
                    x.seen = seen_by(p, x.old + (int32_t)p.by_group.div((uint32_t)x.row0),
                                     x.old + (int32_t)p.by_group.div((uint32_t)last), kBlock);
                    const int32_t units = there ? x.seen.units : 0;
                    x.b0 = (int32_t)((int64_t)units * x.part / p.parts);
                    x.b1 = (int32_t)((int64_t)units * (x.part + 1) / p.parts);
                }
                const int slot = it % kItems;
                if (it >= kItems && !mbar_wait(item_empty + 8 * slot, (it / kItems - 1) & 1, &gave_up)) break;
                if (lane == 0) {
                    items[slot] = x;
                    mbar_arrive(item_full + 8 * slot);
                }
                __syncwarp();
                ++it;
                if (x.h < 0) break;
                // the units of four blocks at a time, one a lane
                bool ok = true;
                const int32_t blocks = x.b1 - x.b0;
                for (int32_t j0 = 0; j0 < blocks && ok; j0 += 4) {
                    const int32_t j = j0 + lane / kUnits, i = lane % kUnits;
                    uint32_t row = 0, rows = 0, kb = 127, vb = 127;
                    if (j < blocks) {
                        const int32_t k = x.seen.unit(x.b0 + j) * kBlock + i * kChunk;
                        // keys [0, sink_end) and [lo, end) are seen
                        auto below = [](int32_t n) { return n >= 16 ? 0xFFFFu : n <= 0 ? 0u : (1u << n) - 1u; };
                        rows = below(x.seen.end - k) & (below(x.seen.sink_end - k) | ~below(x.seen.lo - k));
                        if (rows != 0) {
                            const uint32_t col = p.layer.column(k);
                            const int32_t blk = x.table[col];
                            row = p.layer.row_of(blk, k, col);
                            if (row == Layer::kNoRow) {
                                report(p.status, LMKV_ERR_BAD_BLOCK);
                                row = rows = 0;
                            } else if (kCodes) {
                                kb = scales[p.scales.at(0, blk, x.h)];
                                vb = max((uint32_t)scales[p.scales.at(1, blk, x.h)], kLeastScale);
                            }
                        }
                    }
                    for (int32_t f = 0; f < 4 && j0 + f < blocks && ok; ++f) {
                        const uint32_t block = blocks_before + j0 + f, at = block % kInfoSlots;
                        if (block >= kInfoSlots)
                            ok = mbar_wait(info_empty + 8 * at, (block / kInfoSlots - 1) & 1, &gave_up);
                        if (ok && lane / kUnits == f) {
                            infos[at][i] = make_uint2(row, rows);
                            masks[at][i] = (uint16_t)rows;
                            // (a scale of NaN makes its keys' exponents NaN)
                            if (kCodes)
                                powers[kCodes ? at : 0][i] =
                                    make_float4(power_of_two((int)kb - 127), kb == 255 || vb == 255 ? NAN : (float)((int)vb - 127),
                                                power_of_two(127 - (int)vb), 0.f);
                        }
                        __syncwarp();
                        if (ok && lane == 0) mbar_arrive(info_full + 8 * at);
                    }
                }
                if (!ok) break;
                blocks_before += blocks;
            }
        } else {
            constexpr uint32_t qk = instr_desc<M, kBlock, false>(), pv = instr_desc<M, D, true>();
            // all of tensor memory is this CTA's, so its columns count from 0
            constexpr uint32_t kScores = 0, kOut = 256;
            const uint32_t lead = elect_lead();
            const Desc q0 = desc_k_major(q_smem), k0 = desc_k_major(kv_smem), v0 = desc_n_major(kv_smem, S::kHalfBytes);
            // places of the next K and V items in the ring, and their phases
            int32_t ks = 0, vs = 1;
            uint32_t kph = 0, vph = 0;
            auto advance = [](int32_t& st, uint32_t& ph) {
                st += 2;
                if (st >= S::kStages) {
                    st -= S::kStages;
                    ph ^= 1;
                }
            };
            auto scores = [&](int t, int32_t st) {         // tile t's q x K
                const Desc a = q0.at(t * S::kStageBytes), k = k0.at(st * S::kStageBytes);
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const uint32_t at = (s >> 2) * S::kHalfBytes + (s & 3) * 32;
                    mma_ss(lead, kScores + t * 128, a.at(at), k.at(at), qk, s > 0);
                }
                mma_commit(lead, s_full + 8 * t);
            };
            // the copies of an item, before the products that read them
            auto landed = [&](int32_t st, uint32_t ph) {
                const bool there = mbar_wait(full + 8 * st, ph, &gave_up);
                fence_async_shared();
                return there;
            };
            bool ok = true;
            uint32_t ready[2][2] = {};            // phases of the weights' halves (the second's first: q)
            auto weights = [&](int t, int half) {
                const bool there = mbar_wait(p_ready + 16 * t + 8 * half, ready[t][half], &gave_up);
                ready[t][half] ^= 1;
                return there;
            };
            Item item;
            for (int32_t it = 0; ok && get(it, item); ++it) {
            const int32_t blocks = item.b1 - item.b0;
            const int tiles = min(item.row0 + kTileRows, item.n * group) - item.row0 > 128 ? 2 : 1;
            // (q of items without keys is not waited for with any product, but its phase passes)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (t >= tiles || !ok) break;
                ok = weights(t, 1);
                if (ok && t == 0 && blocks > 0) ok = landed(ks, kph);
                if (ok && blocks > 0) scores(t, ks);
            }
            if (blocks == 0 || !ok) continue;
            advance(ks, kph);
            ok = landed(vs, vph);
            for (int32_t j = 0; j < blocks && ok; ++j) {
                const bool more = j + 1 < blocks;
                const Desc v = v0.at(vs * S::kStageBytes);
                advance(vs, vph);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (t >= tiles || !ok) break;
                    // the weights come in two halves of 64 keys, a barrier each
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        ok = ok && weights(t, half);
                        if (!ok) break;
                        fence_after_sync();
#pragma unroll
                        for (int s = half * 4; s < half * 4 + 4; ++s)
                            mma_ts(lead, kOut + t * 128, kScores + t * 128 + 8 * s, v.at(s * 2048), pv, j > 0 || s > 0);
                    }
                    if (!ok) break;
                    // waits for loads stand where the tensor core has work
                    if (more) {
                        if (t == 0) ok = landed(ks, kph);
                        // issued behind the product that reads the weights from the same columns
                        if (ok) scores(t, ks);
                        if (t == 0) ok = ok && landed(vs, vph);
                    } else {
                        mma_commit(lead, o_full + 8 * t);
                    }
                }
                if (more) advance(ks, kph);
            }
            }
        }
        }
    }
    __syncwarp();
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (tid == 0 && gave_up) report(p.status, LMKV_ERR_TIMEOUT);
    if (warp == 8 + kLoaders + 1) tmem_free<512>(tmem_base);
}


// ---- host ---------------------------------------------------------------

// Rows of a request from which tiles take it.  (Tiles against streams, us, 8 KV heads of 128, by rows: 8 bits, 8 requests of 4000
// keys 24: 59 : 48, 32: 57 : 49, 48: 59 : 62; 64 of 1000 24: 100 : 85, 32: 94 : 89, 48: 98 : 122; 16 bits 8 of 4000 16: 54 : 53, 48: 53 : 80;
// 64 of 1000 16: 86 : 68, 48: 85 : 147.  Between, tiles gain where all requests are alike and lose where few of them
// are so big, as they then have the SMs to themselves for as long: 12 requests of 16 to 40 rows, 700 to 7000 keys, all in streams 60 and 71 us
// for 8 and 16 bits, those of 40 in tiles 96 and 95.)
constexpr int kBigRows = 48;
// CTAs of the tile kernel up to which it splits the keys: two rounds of one an SM.
constexpr int64_t kMostTileCtas = 2 * kSms;

// Rows up to which a CTA joins each.
constexpr int kJoinWarps = 32;
constexpr int64_t kFewRows = 4 * kSms;

struct Plan {
    int32_t big_rows, own_cap, own_tiles, tile_rows, streams, slots, parts;
    int64_t tile_part_rows, own_rows;
    uint64_t bytes;
};

// What a call within these bounds takes; most: room for every smaller one too.
Plan make_plan(const lmkv_pool_t* pool, int32_t q_heads, int32_t num_tokens, int32_t num_req, int32_t max_new,
               int32_t max_kv_len, bool most) {
    Plan x = {};
    const int64_t heads = pool->num_kv_heads, group = q_heads / heads;
    const int64_t rows = (int64_t)num_tokens * q_heads;
    // (a bound of 0 still has rows to look at: lengths beyond it are reported)
    const int64_t req_rows = (int64_t)(max_new < 1 ? 1 : max_new < num_tokens ? max_new : num_tokens) * group;
    // tiles take a unit of 16 keys from one page
    const bool big = req_rows >= kBigRows && pool->block_size % kChunk == 0;
    x.big_rows = big ? kBigRows : INT32_MAX;
    x.own_cap = (int32_t)(big ? kBigRows - 1 : req_rows);
    x.tile_rows = x.own_cap <= 8 ? 8 : 16;
    x.own_tiles = (x.own_cap + x.tile_rows - 1) / x.tile_rows;
    const bool wide = pool->elem_bytes == 2 && pool->head_dim == 128;
    const int64_t warps = (int64_t)kSms * kWarps * (most ? 4 : wide ? 2 : x.tile_rows > 8 ? 3 : 4);
    int64_t streams = warps / heads > 0 ? warps / heads : 1;
    x.streams = (int32_t)streams;
    // (smaller batches may have tiles of fewer rows, and so of more in number)
    const int64_t per_req = most ? ((int64_t)x.own_tiles * x.tile_rows + 8) : (int64_t)x.own_tiles * x.tile_rows;
    x.own_rows = (x.streams * (int64_t)x.tile_rows + num_req * per_req) * heads;
    x.parts = 1;
    if (big) {
        const int64_t slots = (int64_t)num_tokens * group / kTileRows + num_req;
        const int64_t blocks = ((int64_t)max_kv_len + kBlock - 1) / kBlock;
        x.slots = (int32_t)slots;
        if (slots * heads < kSms) {
            const int64_t n = kMostTileCtas / (slots * heads);
            x.parts = (int32_t)(n < blocks ? n : blocks < 1 ? 1 : blocks);
        }
        x.tile_part_rows = x.parts > 1 ? x.parts * rows : 0;
        if (most) x.tile_part_rows = kMostTileCtas * kTileRows;        // a split call's rows are fewer
    }
    x.bytes = (uint64_t)(x.tile_part_rows + x.own_rows) * (pool->head_dim * 4 + 8) +
              (uint64_t)num_req * (most ? (x.own_cap + 7) / 8 : x.own_tiles) * 8 + 8;
    return x;
}

template <class T, class KV, int D, int NT>
int launch_streams(const WindowParams& p, void* stream) {
    return launch(window_streams_kernel<T, KV, D, NT>, ((int64_t)p.streams * p.kv_heads + kWarps - 1) / kWarps, kWarps * 32,
                  StreamShape<KV, D, NT>::kSmem, stream, 1, p);
}

// What the kernels of one type need before their first launch, all at once (once per device; the first call,
// made outside any capture).
template <class T, class KV, int D>
int get_ready() {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    const cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return lmkv_internal_cuda_status(err);
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return LMKV_OK;
    int rc = allow_smem<window_streams_kernel<T, KV, D, 1>, StreamShape<KV, D, 1>::kSmem>();
    if (rc == LMKV_OK) rc = allow_smem<window_streams_kernel<T, KV, D, 2>, StreamShape<KV, D, 2>::kSmem>();
    if (rc == LMKV_OK) rc = allow_smem<window_tiles_kernel<T, KV, D>, WindowTile<D>::kSmem>();
    if (rc == LMKV_OK) rc = keep_carveout<window_streams_kernel<T, KV, D, 1>>();
    if (rc == LMKV_OK) rc = keep_carveout<window_streams_kernel<T, KV, D, 2>>();
    if (rc == LMKV_OK) rc = keep_carveout<window_join_kernel<T, D, false, 1>>();
    if (rc == LMKV_OK) rc = keep_carveout<window_join_kernel<T, D, false, kJoinWarps>>();
    if (rc == LMKV_OK) rc = keep_carveout<window_join_kernel<T, D, true, 1>>();
    if (rc == LMKV_OK) done.fetch_or(bit, std::memory_order_relaxed);
    return rc;
}

template <class T, class KV, int D>
int window_typed(const WindowParams& p, const Plan& x, void* stream) {
    int rc = get_ready<T, KV, D>();
    if (rc == LMKV_OK) rc = x.tile_rows == 8 ? launch_streams<T, KV, D, 1>(p, stream) : launch_streams<T, KV, D, 2>(p, stream);
    if (rc == LMKV_OK && x.big_rows < INT32_MAX)
        rc = launch(window_tiles_kernel<T, KV, D>, p.items < kSms ? p.items : kSms, kTileThreads, WindowTile<D>::kSmem, stream, 1,
                    p);
    const int64_t rows = (int64_t)p.seqs.num_req * x.own_cap * p.kv_heads;
    if (rc == LMKV_OK)
        rc = rows <= kFewRows ? launch(window_join_kernel<T, D, false, kJoinWarps>, rows, kJoinWarps * 32, 0, stream, 1, p)
                              : launch(window_join_kernel<T, D, false, 1>, (rows + 7) / 8, 256, 0, stream, 1, p);
    if (rc == LMKV_OK && x.parts > 1)
        rc = launch(window_join_kernel<T, D, true, 1>, ((int64_t)p.rows + 7) / 8, 256, 0, stream, 1, p);
    return rc;
}

template <class T>
int window_dims(const WindowParams& p, const Plan& x, const lmkv_pool_t* pool, void* stream) {
    if (pool->elem_bytes == 1)
        return pool->head_dim == 64 ? window_typed<T, uint8_t, 64>(p, x, stream) : window_typed<T, uint8_t, 128>(p, x, stream);
    return pool->head_dim == 64 ? window_typed<T, T, 64>(p, x, stream) : window_typed<T, T, 128>(p, x, stream);
}

}  // namespace

extern "C" {

int lmkv_attend_window_workspace_bytes(const lmkv_pool_t* pool, int32_t num_q_heads, int32_t num_tokens, int32_t num_req,
                                       int32_t max_new, int32_t max_kv_len, uint64_t* bytes) {
    const int rc = lmkv_internal_check_pool(pool);
    if (rc != LMKV_OK) return rc;
    if ((pool->elem_bytes != 1 && pool->elem_bytes != 2) || (pool->head_dim != 64 && pool->head_dim != 128))
        return LMKV_ERR_UNSUPPORTED;
    if (bytes == nullptr || num_q_heads <= 0 || num_q_heads % pool->num_kv_heads != 0 || num_q_heads > (1 << 20) ||
        num_tokens < 0 || num_req < 0 || num_req > (1 << 24) || max_new < 0 || max_kv_len < 0 ||
        (int64_t)num_tokens * num_q_heads > (int64_t)1 << 30)
        return LMKV_ERR_INVALID_ARG;
    *bytes = num_tokens == 0 || num_req == 0
                 ? 0 : make_plan(pool, num_q_heads, num_tokens, num_req, max_new, max_kv_len, true).bytes;
    return LMKV_OK;
}

int lmkv_attend_layer_window(const lmkv_pool_t* pool, void* const* scales, int32_t dtype, int32_t layer,
                             const lmkv_batch_t* batch, int32_t num_q_heads, const lmkv_rows_t* q, float scale,
                             int32_t window, int32_t sinks, const lmkv_rows_t* out, float* lse, void* workspace,
                             uint64_t workspace_bytes, int32_t* d_status, void* stream) {
    int rc = lmkv_internal_check_pool(pool);
    if (rc == LMKV_OK) rc = check_scales(pool, scales, dtype);
    if (rc != LMKV_OK) return rc;
    if (layer < 0 || layer >= pool->num_layers || !std::isfinite(scale * kLog2e) || window < 0 || sinks < 0)
        return LMKV_ERR_INVALID_ARG;
    rc = check_batch(pool, batch, num_q_heads);
    if (rc != LMKV_OK) return rc;
    if (batch->max_kv_len > INT32_MAX - 65536) return LMKV_ERR_INVALID_ARG;
    if (batch->num_req == 0 || batch->num_tokens == 0) return LMKV_OK;
    if (!rows_ok(q, 2) || !rows_ok(out, 2)) return LMKV_ERR_INVALID_ARG;
    const Plan x = make_plan(pool, num_q_heads, batch->num_tokens, batch->num_req, batch->max_new, batch->max_kv_len, false);
    if ((int64_t)x.slots * pool->num_kv_heads * x.parts > INT32_MAX / 2) return LMKV_ERR_INVALID_ARG;
    if (workspace == nullptr || workspace_bytes < x.bytes) return LMKV_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(workspace) & 15) return LMKV_ERR_MISALIGNED;
    if (out->data == q->data) return LMKV_ERR_INVALID_ARG;
    WindowParams p = {};
    p.layer = Layer::of(pool, layer);
    p.seqs = Seqs::of(batch);
    p.scales = Scales::of(pool, scales, layer);
    p.q = Rows::of(q);
    p.out = Rows::of(out);
    p.lse = lse;
    p.status = d_status;
    const uint64_t parts = (uint64_t)(x.tile_part_rows + x.own_rows);
    p.part_o = static_cast<float*>(workspace);
    p.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + parts * pool->head_dim * 4);
    p.own_range = reinterpret_cast<int2*>(p.part_ml + parts);
    p.next_item = x.big_rows < INT32_MAX ? reinterpret_cast<int32_t*>(p.own_range + (int64_t)batch->num_req * x.own_tiles) : nullptr;
    p.items = x.slots * pool->num_kv_heads * x.parts;
    p.own_base = x.tile_part_rows;
    p.scale_sign = scale > 0.f ? 1 : scale < 0.f ? -1 : 0;
    p.scale_log2 = scale == 0.f ? 1.f : std::fabs(scale) * kLog2e;
    p.window = window == 0 ? INT32_MAX : window;
    p.sinks = sinks;
    p.q_heads = num_q_heads;
    p.kv_heads = pool->num_kv_heads;
    p.rows = batch->num_tokens * num_q_heads;
    p.big_rows = x.big_rows;
    p.own_cap = x.own_cap;
    p.own_tiles = x.own_tiles;
    p.tile_rows = x.tile_rows;
    p.streams = x.streams;
    p.slots = x.slots;
    p.parts = x.parts;
    auto aligned = [](const lmkv_rows_t* r, int64_t to) {
        return reinterpret_cast<uintptr_t>(r->data) % to == 0 && r->token_stride * 2 % to == 0 && r->head_stride * 2 % to == 0;
    };
    p.q_vec = aligned(q, 16);
    p.out_wide = aligned(out, 32);
    p.q_pairs = aligned(q, 4);
    p.by_group = FastDiv((uint32_t)(num_q_heads / pool->num_kv_heads));
    return dtype == LMKV_BF16 ? window_dims<__nv_bfloat16>(p, x, pool, stream) : window_dims<__half>(p, x, pool, stream);
}

}  // extern "C"
