// lmkv_attend.cu -- attention of a batch's new tokens to one layer's pages,
// behind a prefix that all requests share.
//
// With x = scale * q.k, o = sum_j e^(x_j) v_j / sum_j e^(x_j) splits over any
// partition of the keys: a part keeps its largest x (m), l = sum e^(x - m) and
// sum e^(x - m) v, and parts are joined by
//   M = max m,  l = sum l e^(m - M),  o = sum o e^(m - M) / l
// (the running maximum and sum of Milakov and Gimelshein, "Online normalizer
// calculation for softmax", 2018, which is also how a part takes its keys one
// block at a time).  So the prefix is attended to by the rows of all requests
// at once, tile by tile, and read once for the batch; a request's own pages by
// its own rows; and a last kernel joins the parts.  Powers are of 2, with
// scale * log2(e) folded into x.
#include "lmkv_blocks.cuh"

#include <cmath>

namespace {

using namespace lmkv_paged;
using namespace lmkv_mma;

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
// kBigRows has its own pages attended to by the tile kernel, after the prefix
// and in the same pass; the others', with too few rows for a tile of 128, by
// the row kernel.  (Tiles against rows, us: 64 requests of 1000 keys, 48 rows 120 :
// 152, 64 rows 96 : 160; of 300 keys, 48 rows 61 : 50, 64 rows 50 : 58.)
constexpr int kBigRows = 64;

struct AttendParams {
    Layer layer;
    Seqs seqs;
    Rows q, out;
    float* lse;
    const int32_t* prefix_table;
    int32_t* status;
    // Partial results: m (powers of 2), l and the weighted sum of v.  First
    // [prefix_parts][rows], row = token * q_heads + head, then the own parts:
    // [stream + row tile of the batch's requests][row of the tile][KV head] (a
    // stream's and a tile's number rise from part to part, so their sum names it).
    float* part_o;
    float2* part_ml;
    float scale_log2;       // of |scale|
    float lowest;           // least raw score that a tile's weights are relative to (kFarScore)
    int32_t scale_sign;     // -1, 0 or 1
    int32_t prefix_len;
    int32_t q_heads, kv_heads;
    int32_t rows;           // num_tokens * q_heads
    int32_t row_tiles;      // row kernel: row tiles of the prefix part (0: the tile kernel has it)
    int32_t prefix_parts, prefix_span;    // parts of the prefix (row kernel: keys in each)
    int32_t tiles;          // tile kernel: row tiles (0: not launched)
    int32_t tile_ctas;      // its CTAs that take tiles; those after them run streams
    int32_t own_cap;        // rows of a request that the row kernel takes at most
    int32_t own_tiles;      // row tiles of that many rows
    int32_t tile_rows;      // rows of a tile that there may be
    int32_t streams;        // warps that share the own tokens for a KV head; 0: a CTA per row tile
    int2* own_range;        // [request][row tile]: first and last stream that has some of it
    uint32_t* again;        // [tile kernel's CTA][8]: its rows to take again (where a request may be big)
    int32_t again_cta;      // first CTA of the row kernel that does so
    bool big;               // a request may have kBigRows rows
    bool own_final;         // the own part is all of a small request: no join
    bool q_pairs;           // q rows are 4-byte aligned
    bool q_vec;             // q rows are 16-byte aligned
    bool out_vec;           // out rows are 16-byte aligned
    FastDiv by_group;

    __device__ __forceinline__ int64_t own_part(int32_t stream, int32_t tile_no, int32_t row, int32_t h) const {
        return (int64_t)prefix_parts * rows + (((int64_t)stream + tile_no) * tile_rows + row) * kv_heads + h;
    }
};

constexpr int kTileRows = 256;    // of the tile kernel: two tiles of 128 rows share every K and V block
constexpr int kRowTile = 16;      // rows of a tile: one mma.sync operand
constexpr int kWarps = 4;
constexpr int kChunk = 16;        // keys a warp takes at a time
constexpr int kStages = 2;
constexpr int kRowCtas = 3;       // CTAs an SM: more in flight than with three stages and two CTAs
constexpr float kLn2 = 0.69314718055994530942f, kLog2e = 1.44269504088896340736f;

// A row tile's place in the batch.
struct Tile {
    const int32_t* table;
    int32_t k0, k1;        // keys of this part
    int32_t h;             // KV head
    int32_t part;
    int32_t r;             // request, or -1: rows of the whole batch
    int32_t t0, row0;      // row i of the tile is row row0 + i of the rows that begin at token t0
    int32_t nrows;         // rows from row0 on (may exceed the tile)
    int32_t limit0;        // row row0 + i sees keys below limit0 + (row0 + i) / group * causal
    int32_t causal;
};

// The row tile of CTA `bid`; false when it has none.
__device__ __forceinline__ bool find_tile(const AttendParams& p, int32_t bid, Tile& t) {
    const int32_t group = (int32_t)p.by_group.d;
    const int32_t prefix_ctas = p.row_tiles * p.kv_heads * p.prefix_parts;
    if (bid < prefix_ctas) {
        const int32_t tile = bid % p.row_tiles;
        const int32_t x = bid / p.row_tiles;
        t.h = x % p.kv_heads;
        t.part = x / p.kv_heads;
        t.r = -1;
        t.table = p.prefix_table;
        t.k0 = t.part * p.prefix_span;
        t.k1 = min(t.k0 + p.prefix_span, p.prefix_len);
        t.t0 = 0;
        t.row0 = tile * kRowTile;
        const int32_t end = min(max(p.seqs.q_start[p.seqs.num_req], 0), p.seqs.num_tokens);
        t.nrows = end * group - t.row0;
        t.limit0 = p.prefix_len;
        t.causal = 0;
        return t.nrows > 0;
    }
    bid -= prefix_ctas;
    // heads change fastest: the heads' CTAs of the same tokens read the same pages' rows
    t.h = bid % p.kv_heads;
    int32_t x = bid / p.kv_heads;
    const int32_t tile = x % p.own_tiles;
    x /= p.own_tiles;
    t.r = x;
    t.part = 0;
    const Req q = load_req(p.seqs, t.r);
    if (!q.ok && threadIdx.x == 0) report(p.status, LMKV_ERR_BAD_LENGTH);
    t.row0 = tile * kRowTile;
    t.nrows = q.n * group - t.row0;
    if (t.nrows <= 0 || (p.big && q.n * group >= kBigRows)) return false;
    t.table = p.seqs.table + (int64_t)t.r * p.seqs.table_stride;
    t.t0 = q.q0;
    t.limit0 = q.len - q.n + 1;
    t.causal = 1;
    const int32_t last = (int32_t)p.by_group.div((uint32_t)(t.row0 + min(t.nrows, kRowTile) - 1));
    t.k0 = 0;
    t.k1 = max(0, min(q.len, t.limit0 + last));
    return true;
}

// One warp's 16 rows against chunks of 16 keys, by mma.sync: q, and the running
// maximum, sum and output.
template <class T, int D>
struct WarpRows {
    static constexpr int kRowBytes = D * 2;
    static constexpr int kTileBytes = kChunk * kRowBytes;   // K (or V) rows of a stage
    static constexpr int kSteps = D / 16;

    // this thread's two rows: lane / 4 and lane / 4 + 8
    int32_t limit[2];
    uint32_t qf[kSteps][4];
    float o[D / 8][4];
    float m[2], l[2];

    __device__ __forceinline__ void begin(const AttendParams& p, const Tile& t) {
        const int lane = threadIdx.x & 31;
        const int32_t group = (int32_t)p.by_group.d;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int32_t rr = (lane >> 2) + 8 * i;
            const bool on = rr < t.nrows;
            const int32_t n = (int32_t)p.by_group.div((uint32_t)(t.row0 + (on ? rr : 0)));
            limit[i] = on ? t.limit0 + t.causal * n : 0;
            const T* src = p.q.row<T>(t.t0 + n, t.h * group + (t.row0 + rr - n * group));
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const int e = s * 16 + (lane & 3) * 2;
                qf[s][i] = on ? load_pair(src + e, p.q_pairs) : 0u;
                qf[s][2 + i] = on ? load_pair(src + e + 8, p.q_pairs) : 0u;
            }
            m[i] = -INFINITY;
            l[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    }

    // The chunk at key `key0` whose K rows are at kt and V rows behind them;
    // mask: which of its keys there are.
    __device__ __forceinline__ void chunk(uint32_t kt, int32_t key0, uint32_t mask, float scale) {
        const int lane = threadIdx.x & 31;
        const uint32_t vt = kt + kTileBytes;
        float sc[2][4] = {};
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            uint32_t b[4];
            // matrices: keys 0-7 x d 0-7, keys 0-7 x d 8-15, keys 8-15 x d 0-7, keys 8-15 x d 8-15
            ldmatrix4(b, kt + swizzled<kRowBytes>((lane & 7) + ((lane >> 4) << 3), 2 * s + ((lane >> 3) & 1)));
            mma16816<T>(sc[0], qf[s], b[0], b[1]);
            mma16816<T>(sc[1], qf[s], b[2], b[3]);
        }
        key0 += (lane & 3) * 2;
        float pr[2][4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float top = -INFINITY;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int at = n * 8 + j;
                    const bool seen = key0 + at < limit[r] && ((mask >> (at + (lane & 3) * 2)) & 1);
                    float& x = sc[n][2 * r + j];
                    x = seen ? x * scale : -INFINITY;
                    top = fmaxf(top, x);
                }
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            const float mn = fmaxf(m[r], top);
            const float mu = mn == -INFINITY ? 0.f : mn;      // nothing seen yet: every power is 0
            const float corr = exp2_fast(m[r] - mu);
            m[r] = mn;
            float sum = 0.f;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) sum += pr[n][2 * r + j] = exp2_fast(sc[n][2 * r + j] - mu);
            l[r] = l[r] * corr + sum;
            if (corr != 1.f) {
#pragma unroll
                for (int d = 0; d < D / 8; ++d) {
                    o[d][2 * r] *= corr;
                    o[d][2 * r + 1] *= corr;
                }
            }
        }
        // Weights are rounded to T for the product with V (relative error at
        // most half a step of T each, of either sign, against the sums in fp32).  A second product with what the
        // rounding leaves over would leave the result's own rounding alone (0.0023 for 0.0017 on 64 users behind 16384
        // tokens, bf16), at 4 to 11 % of a call: 50.3 : 52.6 us there, 65 : 72 with 600 own tokens each, 9.9 : 10.9
        // for 4 requests of 512.
        const uint32_t pf[4] = {Elem<T>::pack(pr[0][0], pr[0][1]), Elem<T>::pack(pr[0][2], pr[0][3]),
                                Elem<T>::pack(pr[1][0], pr[1][1]), Elem<T>::pack(pr[1][2], pr[1][3])};
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
            uint32_t b[4];
            ldmatrix4_trans(b, vt + swizzled<kRowBytes>(lane & 15, 2 * d + (lane >> 4)));
            mma16816<T>(o[2 * d], pf, b[0], b[1]);
            mma16816<T>(o[2 * d + 1], pf, b[2], b[3]);
        }
    }

    // l becomes the whole row's.
    __device__ __forceinline__ void end() {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 1);
            l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 2);
        }
    }
};

// Joins the results of a CTA's warps for the same rows in shared
// memory; put(row, first of four elements, m, l, their sums) takes what comes of it.  (As the row kernel's end
// does; with one function for both, calls of one tile a request took 5 % longer.)
template <class T, int D, class Put>
__device__ __forceinline__ void join_warps(const WarpRows<T, D>& x, uint8_t* smem, float2 (*ml)[kRowTile], Put put) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* const wo = reinterpret_cast<float*>(smem) + warp * kRowTile * D;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int rr = (lane >> 2) + 8 * r;
        if ((lane & 3) == 0) ml[warp][rr] = make_float2(x.m[r], x.l[r]);
#pragma unroll
        for (int d = 0; d < D / 8; ++d)
            *reinterpret_cast<float2*>(wo + rr * D + d * 8 + (lane & 3) * 2) =
                make_float2(x.o[d][2 * r], x.o[d][2 * r + 1]);
    }
    __syncthreads();
    const float* const all = reinterpret_cast<const float*>(smem);
    for (int i = threadIdx.x; i < kRowTile * (D / 4); i += kWarps * 32) {
        const int rr = i / (D / 4), c = (i % (D / 4)) * 4;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w][rr].x);
        const float mu = top == -INFINITY ? 0.f : top;
        float sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = exp2_fast(ml[w][rr].x - mu);
            const float4 y = *reinterpret_cast<const float4*>(all + (w * kRowTile + rr) * D + c);
            sum += f * ml[w][rr].y;
            acc.x += f * y.x;
            acc.y += f * y.y;
            acc.z += f * y.z;
            acc.w += f * y.w;
        }
        put(rr, c, top, sum, acc);
    }
}

// Four elements of a row whose sums are complete, and its lse.
template <class T>
__device__ __forceinline__ void put_final(const AttendParams& p, int32_t tok, int32_t head, int c, float top, float sum,
                                          float4 acc) {
    const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
    T* dst = p.out.row<T>(tok, head) + c;
    dst[0] = Elem<T>::from_float(acc.x * inv);
    dst[1] = Elem<T>::from_float(acc.y * inv);
    dst[2] = Elem<T>::from_float(acc.z * inv);
    dst[3] = Elem<T>::from_float(acc.w * inv);
    if (c == 0 && p.lse != nullptr)
        p.lse[(int64_t)tok * p.q_heads + head] = ((top == -INFINITY ? 0.f : top) + log2f(sum)) * kLn2;
}

// Rows of the tile kernel are taken again where a request may be big.  Most are rows that a value
// of another request has spoiled: the tile's product multiplies every key's row of v, those a row
// does not see by a weight of 0, and 0 times infinity or NaN is NaN.  Others have scores far from 0
// (kFarScore).  The last CTAs of the row or stream kernel, which follow the tile kernel, share the
// windows of 16 rows that hold some; one goes over the prefix and the own keys of one request at
// a time, as the row kernel takes its rows.  What comes of the request's rows is the whole result of a
// big one and the prefix's of others, and stands for all parts.  Without any, which is the rule,
// 16 bits a window are looked at: 0 to 2 us.  (Requests of 70, 70, 70 and 30 tokens behind 12000 keys, 16
// heads of 128, one with a NaN: 0.34 ms, without it 0.057; a row a warp took 7.8.)

// The windows of a CTA: bits of the rows, those of window w0 + f * ctas in found[f].
template <class T, int D>
__device__ __noinline__ void take_windows(const AttendParams& p, const uint32_t* found, int32_t w0, int32_t ctas, uint8_t* smem,
                                          float2 (*ml)[kRowTile]) {
    using W = WarpRows<T, D>;
    constexpr int kWindows = kTileRows / kRowTile;      // of a tile
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t group = (int32_t)p.by_group.d;
    const int32_t live_rows = min(max(p.seqs.q_start[p.seqs.num_req], 0), p.seqs.num_tokens) * group;
    const uint32_t ring = smem_u32(smem) + warp * (kStages * 2 * W::kTileBytes);
    const float signed_scale = p.scale_log2 * (float)p.scale_sign;
    const uint8_t* const base = p.layer.base();
#pragma unroll 1
    for (int32_t f = 0; f < kWarps * 32; ++f) {
        uint32_t left = found[f];      // the same for all threads
        if (left == 0) continue;
        const int32_t at = w0 + f * ctas;
        Tile t;
        t.h = at / kWindows / p.tiles;
        t.t0 = 0;
        t.row0 = at / kWindows % p.tiles * kTileRows + at % kWindows * kRowTile;
        t.nrows = live_rows - t.row0;
        t.limit0 = t.causal = 0;                    // (limits below)
        while (left != 0) {
            // the request of the first row left, and its rows of the window
            const int32_t tok0 = (int32_t)p.by_group.div((uint32_t)(t.row0 + __ffs(left) - 1));
            const Req q = load_req(p.seqs, find_request(p.seqs.num_req, tok0, [&](int32_t i) { return p.seqs.q_start[i]; }));
            const bool big = q.n * group >= kBigRows;
            uint32_t now = 0;
            for (int r = 0; r < kRowTile; ++r) {
                const int32_t tok = (int32_t)p.by_group.div((uint32_t)(t.row0 + r));
                if (((left >> r) & 1) && tok >= q.q0 && tok < q.q0 + q.n) now |= 1u << r;
            }
            left &= ~(now | (left & -left));        // (a row of no request is left as it is)
            if (now == 0) continue;
            W x;
            x.begin(p, t);
#pragma unroll 1
            for (int own = 0; own < (big ? 2 : 1); ++own) {
                // (rows of other requests come to nothing that is kept)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int32_t rr = min((lane >> 2) + 8 * i, t.nrows - 1);
                    const int32_t tok = (int32_t)p.by_group.div((uint32_t)(t.row0 + rr));
                    x.limit[i] = own ? q.len - q.n + 1 + (tok - q.q0) : p.prefix_len;
                }
                const int32_t end = base == nullptr ? 0 : own ? q.len : p.prefix_len;
                const int32_t chunks = (end + kChunk - 1) / kChunk;
                const int32_t mine = chunks > warp ? (chunks - warp + kWarps - 1) / kWarps : 0;
                uint32_t there[kStages];
                ChunkCopy<D, true> rows(p.layer, own ? p.seqs.table + (int64_t)q.r * p.seqs.table_stride : p.prefix_table,
                                        base, t.h, end);
                auto key_of = [&](int32_t i) { return (i * kWarps + warp) * kChunk; };
                auto fill = [&](int32_t i) {        // (what is not there has been reported)
                    return rows.copy(key_of(i), ring + (i % kStages) * (2 * W::kTileBytes), key_of(i + 1), nullptr);
                };
                __syncwarp();
                rows.lookup(key_of(0));
#pragma unroll
                for (int s = 0; s < kStages - 1; ++s) {
                    there[s] = s < mine ? fill(s) : 0u;
                    cp_commit();
                }
                for (int32_t i0 = 0; i0 < mine; i0 += kStages) {
#pragma unroll
                    for (int u = 0; u < kStages; ++u) {
                        const int32_t i = i0 + u;
                        if (i >= mine) break;
                        __syncwarp();      // the stage filled next was read by every lane
                        constexpr int kAhead = kStages - 1;
                        there[(u + kAhead) % kStages] = i + kAhead < mine ? fill(i + kAhead) : 0u;
                        cp_commit();
                        cp_wait<kStages - 1>();
                        __syncwarp();
                        x.chunk(ring + u * (2 * W::kTileBytes), key_of(i), there[u], signed_scale);
                    }
                }
                cp_wait<0>();
            }
            __syncthreads();
            x.end();
            join_warps<T, D>(x, smem, ml, [&](int rr, int c, float top, float sum, float4 acc) {
                if (((now >> rr) & 1) == 0) return;
                const int32_t tok = (int32_t)p.by_group.div((uint32_t)(t.row0 + rr));
                const int32_t head = t.h * group + (t.row0 + rr - tok * group);
                if (big && p.prefix_parts == 1) {
                    put_final<T>(p, tok, head, c, top, sum, acc);
                    return;
                }
                for (int32_t part = 0; part < p.prefix_parts; ++part) {
                    const int64_t row = (int64_t)part * p.rows + (int64_t)tok * p.q_heads + head;
                    *reinterpret_cast<float4*>(p.part_o + row * D + c) = part == 0 ? acc : make_float4(0.f, 0.f, 0.f, 0.f);
                    if (c == 0) p.part_ml[row] = part == 0 ? make_float2(top, sum) : make_float2(-INFINITY, 0.f);
                }
            });
            __syncthreads();
        }
    }
}

// Looks for windows; the CTA is number `cta` of those that do.
template <class T, int D>
__device__ __forceinline__ void take_again(const AttendParams& p, int32_t cta, int32_t ctas, uint8_t* smem,
                                           float2 (*ml)[kRowTile]) {
    __shared__ uint32_t found[kWarps * 32];
    constexpr int kWindows = kTileRows / kRowTile;      // of a tile
    const int32_t windows = p.tiles * kWindows * p.kv_heads;
    // every thread looks at one of the CTA's windows, that many at a time
    for (int32_t w0 = cta; w0 < windows; w0 += kWarps * 32 * ctas) {
        const int32_t mine = w0 + (int32_t)threadIdx.x * ctas;
        uint32_t bits = 0;
        if (mine < windows) {
            const int32_t at = mine / kWindows, win = mine % kWindows;        // tile + p.tiles * head
            for (int32_t part = 0; part < p.prefix_parts; ++part)
                bits |= p.again[((int64_t)part * p.kv_heads * p.tiles + at) * 8 + (win >> 1)];
            bits = (bits >> ((win & 1) * kRowTile)) & 0xFFFFu;
        }
        if (!__syncthreads_or(bits != 0)) continue;
        found[threadIdx.x] = bits;
        __syncthreads();
        take_windows<T, D>(p, found, w0, ctas, smem, ml);
        __syncthreads();
    }
}

// Small batches and short contexts: a CTA per row tile (and part of the
// prefix).  Bound by the bytes of K and V: with a few rows per KV head the
// products are a fraction of the loads' time, so the four warps of a CTA share
// the rows, take 16 keys (a page) each in turn, and run by themselves: every
// warp has its own ring of kStages x 16 K and V rows, filled by cp.async, and
// its own running maximum, sum and output; they are joined in shared memory at
// the end.  (4 requests of up to 90 keys behind 512, 2 KV heads of 64: 6.3 us, all of it
// latency: a launch, three dependent look-ups, one round of rows.)
// kBig: a request may be big, and the CTAs from again_cta on take_again.
template <class T, int D, bool kBig>
__global__ void __launch_bounds__(kWarps * 32, kRowCtas)
attend_rows_kernel(const __grid_constant__ AttendParams p) {
    using W = WarpRows<T, D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ float2 ml[kWarps][kRowTile];
    pdl_launch_dependents();
    pdl_wait();
    if (kBig && (int32_t)blockIdx.x >= p.again_cta) {
        take_again<T, D>(p, blockIdx.x - p.again_cta, gridDim.x - p.again_cta, smem, ml);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Tile t;
    if (!find_tile(p, blockIdx.x, t)) return;
    const uint8_t* base = p.layer.base();
    if (base == nullptr) {
        if (threadIdx.x == 0) report(p.status, LMKV_ERR_BAD_POINTER);
        t.k1 = t.k0;
    }
    const int32_t group = (int32_t)p.by_group.d;
    const uint32_t ring = smem_u32(smem) + warp * (kStages * 2 * W::kTileBytes);
    const int32_t chunks = (t.k1 - t.k0 + kChunk - 1) / kChunk;
    const int32_t mine = chunks > warp ? (chunks - warp + kWarps - 1) / kWarps : 0;
    uint32_t there[kStages];       // key masks of the stages (constant indices after unrolling)
    ChunkCopy<D, true> rows(p.layer, t.table, base, t.h, t.k1);
    auto key_of = [&](int32_t i) { return t.k0 + (i * kWarps + warp) * kChunk; };       // my i-th chunk
    auto fill = [&](int32_t i) {                       // into its stage
        return rows.copy(key_of(i), ring + (i % kStages) * (2 * W::kTileBytes), key_of(i + 1), p.status);
    };
    // the first rows are on their way while q comes
    rows.lookup(key_of(0));
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
        there[s] = s < mine ? fill(s) : 0u;
        cp_commit();
    }
    W x;
    x.begin(p, t);
    const float signed_scale = p.scale_log2 * (float)p.scale_sign;
    for (int32_t i0 = 0; i0 < mine; i0 += kStages) {
#pragma unroll
        for (int u = 0; u < kStages; ++u) {
            const int32_t i = i0 + u;
            if (i >= mine) break;
            __syncwarp();      // the stage filled next was read by every lane
            constexpr int kAhead = kStages - 1;
            there[(u + kAhead) % kStages] = i + kAhead < mine ? fill(i + kAhead) : 0u;
            cp_commit();
            cp_wait<kStages - 1>();
            __syncwarp();
            x.chunk(ring + u * (2 * W::kTileBytes), key_of(i), there[u], signed_scale);
        }
    }
    cp_wait<0>();
    __syncthreads();

    // join the warps in shared memory
    x.end();
    float* const wo = reinterpret_cast<float*>(smem) + warp * kRowTile * D;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int rr = (lane >> 2) + 8 * r;
        if ((lane & 3) == 0) ml[warp][rr] = make_float2(x.m[r], x.l[r]);
#pragma unroll
        for (int d = 0; d < D / 8; ++d)
            *reinterpret_cast<float2*>(wo + rr * D + d * 8 + (lane & 3) * 2) =
                make_float2(x.o[d][2 * r], x.o[d][2 * r + 1]);
    }
    __syncthreads();
    const float* const all = reinterpret_cast<const float*>(smem);
    for (int i = threadIdx.x; i < kRowTile * (D / 4); i += kWarps * 32) {
        const int rr = i / (D / 4), c = (i % (D / 4)) * 4;
        if (rr >= t.nrows) break;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w][rr].x);
        const float mu = top == -INFINITY ? 0.f : top;
        float sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = exp2_fast(ml[w][rr].x - mu);
            const float4 y = *reinterpret_cast<const float4*>(all + (w * kRowTile + rr) * D + c);
            sum += f * ml[w][rr].y;
            acc.x += f * y.x;
            acc.y += f * y.y;
            acc.z += f * y.z;
            acc.w += f * y.w;
        }
        const int32_t n = (int32_t)p.by_group.div((uint32_t)(t.row0 + rr));
        const int32_t tok = t.t0 + n, head = t.h * group + (t.row0 + rr - n * group);
        const int32_t row = tok * p.q_heads + head;
        if (t.r >= 0 && p.own_final) {
            const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
            T* dst = p.out.row<T>(tok, head) + c;
            dst[0] = Elem<T>::from_float(acc.x * inv);
            dst[1] = Elem<T>::from_float(acc.y * inv);
            dst[2] = Elem<T>::from_float(acc.z * inv);
            dst[3] = Elem<T>::from_float(acc.w * inv);
            if (c == 0 && p.lse != nullptr) p.lse[row] = (mu + log2f(sum)) * kLn2;
        } else {
            const int64_t at = t.r < 0 ? (int64_t)t.part * p.rows + row
                                       : p.own_part(0, t.r * p.own_tiles + t.row0 / kRowTile, rr, t.h);
            *reinterpret_cast<float4*>(p.part_o + at * D + c) = acc;
            if (c == 0) p.part_ml[at] = make_float2(top, sum);
        }
    }
}

// Longer own contexts: streams.  The chunks of all small requests' row tiles,
// one after the other, are shared equally among warps, whatever the lengths
// are; a warp runs through its share by itself, with no barrier, and leaves a
// partial result for each row tile that it had some of.  Stream g of KV head h
// is warp `g * kv_heads + h` of the launch: the heads' warps of the same tokens run
// side by side and read the same pages' rows.  (128 requests of 2048 keys, 8 KV heads of
// 128: 189 us with launch and join, 5.7 TB/s.)
template <class T, int D>
__device__ __forceinline__ void run_stream(const AttendParams& p, int32_t worker, uint32_t ring) {
    using W = WarpRows<T, D>;
    const int lane = threadIdx.x & 31;
    const int32_t group = (int32_t)p.by_group.d;
    const int32_t g = worker / p.kv_heads;
    if (g >= p.streams) return;
    Tile t;
    t.h = worker - g * p.kv_heads;
    t.causal = 1;
    const uint8_t* const base = p.layer.base();
    if (base == nullptr && worker == 0 && lane == 0) report(p.status, LMKV_ERR_BAD_POINTER);
    // row tiles of a request, and chunks of each
    auto tiles_of = [&](const Req& q) {
        const int32_t n = q.n * group;
        return p.big && n >= kBigRows ? 0 : (n + kRowTile - 1) / kRowTile;
    };
    Share share = find_share(p.seqs.num_req, g, p.streams, [&](int32_t i) -> int64_t {
        const Req q = load_req(p.seqs, i);
        if (!q.ok) report(p.status, LMKV_ERR_BAD_LENGTH);
        return (int64_t)tiles_of(q) * ((q.len + kChunk - 1) / kChunk);
    });
    const float signed_scale = p.scale_log2 * (float)p.scale_sign;
    W x;
    while (share.n > 0 && share.r < p.seqs.num_req) {
        const Req q = load_req(p.seqs, share.r);
        const int32_t per_tile = (q.len + kChunk - 1) / kChunk;
        const int32_t tile = per_tile > 0 ? (int32_t)(share.first / per_tile) : 0;
        if (per_tile == 0 || tile >= tiles_of(q)) {
            ++share.r;
            share.first = 0;
            continue;
        }
        const int32_t c0 = (int32_t)(share.first - (int64_t)tile * per_tile);
        const int32_t n = (int32_t)min((int64_t)(per_tile - c0), share.n);
        share.first += n;
        share.n -= n;
        t.r = share.r;
        t.table = p.seqs.table + (int64_t)share.r * p.seqs.table_stride;
        t.t0 = q.q0;
        t.limit0 = q.len - q.n + 1;
        t.row0 = tile * kRowTile;
        t.nrows = q.n * group - t.row0;
        const int32_t tile_no = share.r * p.own_tiles + tile;
        if (t.h == 0 && lane == 0) {
            if (c0 == 0) p.own_range[tile_no].x = g;
            if (c0 + n == per_tile) p.own_range[tile_no].y = g;
        }
        // keys that the tile's last row does not see are left out
        const int32_t last = (int32_t)p.by_group.div((uint32_t)(t.row0 + min(t.nrows, kRowTile) - 1));
        const int32_t k0 = c0 * kChunk;
        const int32_t k1 = base == nullptr ? k0 : max(k0, min(min(k0 + n * kChunk, q.len), t.limit0 + last));
        const int32_t mine = (k1 - k0 + kChunk - 1) / kChunk;
        uint32_t there[kStages];
        ChunkCopy<D, true> rows(p.layer, t.table, base, t.h, k1);
        auto fill = [&](int32_t i) {
            return rows.copy(k0 + i * kChunk, ring + (i % kStages) * (2 * W::kTileBytes), k0 + (i + 1) * kChunk, p.status);
        };
        __syncwarp();
        rows.lookup(k0);
#pragma unroll
        for (int s = 0; s < kStages - 1; ++s) {
            there[s] = s < mine ? fill(s) : 0u;
            cp_commit();
        }
        x.begin(p, t);
        for (int32_t i0 = 0; i0 < mine; i0 += kStages) {
#pragma unroll
            for (int u = 0; u < kStages; ++u) {
                const int32_t i = i0 + u;
                if (i >= mine) break;
                __syncwarp();      // the stage filled next was read by every lane
                constexpr int kAhead = kStages - 1;
                there[(u + kAhead) % kStages] = i + kAhead < mine ? fill(i + kAhead) : 0u;
                cp_commit();
                cp_wait<kStages - 1>();
                __syncwarp();
                x.chunk(ring + u * (2 * W::kTileBytes), k0 + i * kChunk, there[u], signed_scale);
            }
        }
        cp_wait<0>();
        x.end();
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int rr = (lane >> 2) + 8 * r;
            if (rr >= t.nrows) continue;
            const int64_t at = p.own_part(g, tile_no, rr, t.h);
            if ((lane & 3) == 0) p.part_ml[at] = make_float2(x.m[r], x.l[r]);
#pragma unroll
            for (int d = 0; d < D / 8; ++d)
                *reinterpret_cast<float2*>(p.part_o + at * D + d * 8 + (lane & 3) * 2) =
                    make_float2(x.o[d][2 * r], x.o[d][2 * r + 1]);
        }
    }
}

template <class T, int D, bool kBig>
__global__ void __launch_bounds__(kWarps * 32, kRowCtas)
attend_streams_kernel(const __grid_constant__ AttendParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    pdl_launch_dependents();
    pdl_wait();
    if constexpr (kBig) {
        __shared__ float2 ml[kWarps][kRowTile];
        if ((int32_t)blockIdx.x >= p.again_cta) {
            take_again<T, D>(p, blockIdx.x - p.again_cta, gridDim.x - p.again_cta, smem, ml);
            return;
        }
    }
    const int warp = threadIdx.x >> 5;
    run_stream<T, D>(p, blockIdx.x * kWarps + warp,
                              smem_u32(smem) + warp * (kStages * 2 * WarpRows<T, D>::kTileBytes));
}

// ---- tiles of 128 rows on the tensor core -------------------------------

using namespace lmkv_tc;

constexpr int kTileThreads = 352;     // softmax 2 x 128, loads 64, products 1 (of 32)
constexpr int kMaxSegs = 8;           // the prefix and every big request that 256 rows can touch
constexpr int kMaskSlots = 8;
// The main loop takes x * scale - m * scale as one product and sum, with m * scale rounded: all
// weights of a row are off by the same power of that rounding (as is the part's m), which is harmless until it
// leaves their range.  Rows of scores beyond this (in powers of 2), where it is 2^-8 of a power yet, are taken
// again by differences.  No weights are relative to less than its negative, so that keys that far down come to nothing
// beside others.
constexpr float kFarScore = 0x1p16f;
constexpr int kStreamWarps = 8;       // streams of a CTA that has no tiles (with rings of three, or 9 to 11, slower)

// Keys in a row's order: the prefix, then each big request of the tile.
struct Seg {
    const int32_t* table;
    int32_t end;       // keys [0, end)
    int32_t first;     // number of its first block
    int32_t q0, n;     // its tokens; the prefix: n < 0
    int32_t limit0;    // token q0 + i sees keys below limit0 + i
};

template <int D>
struct TileShape {
    static constexpr int kHalfBytes = BlockShape<D>::kHalfBytes;
    static constexpr int kStageBytes = BlockShape<D>::kBytes;      // 128 rows of K, V or q
    static constexpr int kStages = D == 128 ? 5 : 8;
    static constexpr int kSmem = (2 + kStages) * kStageBytes;
};

// Takes a row of a part again, by one warp, or leaves it to take_again where a request may
// be big.  Only rows whose scores are far from 0 (kFarScore) need it where none is.  32 keys a step, a key
// a lane for the weights, D / 32 elements a lane for the sums.  (As a function of its own, and
// over the tile's segments, it leaves the main loop its registers: with the prefix alone
// as its keys 635 us for 586.)
template <class T, int D>
__device__ __noinline__ void take_row(const AttendParams& p, const Seg* segs, int32_t nseg, int32_t num_blocks,
                                       const uint8_t* base, int32_t h, int32_t part, int32_t tile_row) {
    if (p.big) {
        if ((threadIdx.x & 31) == 0) p.again[(int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)] |= 1u << (tile_row & 31);
        return;
    }
    const int32_t group = (int32_t)p.by_group.d;
    const int32_t tok = (int32_t)p.by_group.div((uint32_t)tile_row), head = h * group + (tile_row - tok * group);
    const int32_t b0 = (int32_t)((int64_t)num_blocks * part / p.prefix_parts);
    const int32_t b1 = (int32_t)((int64_t)num_blocks * (part + 1) / p.prefix_parts);
    constexpr int kPer = D / 32;
    const int lane = threadIdx.x & 31;
    const T* const q = p.q.row<T>(tok, head);
    const uint8_t* const k_rows = base + (int64_t)h * (D * 2);
    const uint8_t* const v_rows = k_rows + p.layer.half_bytes();
    const float scale = p.scale_log2 * (float)p.scale_sign;
    float m = -INFINITY, l = 0.f, acc[kPer] = {};
    for (int32_t si = 0; si < nseg; ++si) {
        const Seg& sg = segs[si];
        if (sg.n >= 0 && (tok < sg.q0 || tok >= sg.q0 + sg.n)) continue;
        int64_t end = min((int64_t)sg.end, (int64_t)(b1 - sg.first) * kBlock);
        if (sg.n >= 0) end = min(end, (int64_t)sg.limit0 + (tok - sg.q0));
        for (int64_t k0 = (int64_t)max(b0 - sg.first, 0) * kBlock; k0 < end; k0 += 32) {
            const int64_t at = k0 + lane < end ? p.layer.token_offset(sg.table, (int32_t)k0 + lane) : -1;
            float x = -INFINITY;
            if (at >= 0) {
                x = 0.f;
#pragma unroll 4
                for (int c = 0; c < D / 8; ++c) {
                    const int4 k = *reinterpret_cast<const int4*>(k_rows + at + c * 16);
                    const T* const e = reinterpret_cast<const T*>(&k);
#pragma unroll
                    for (int i = 0; i < 8; ++i) x = fmaf(Elem<T>::to_float(q[c * 8 + i]), Elem<T>::to_float(e[i]), x);
                }
                x *= scale;
            }
            float top = x;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
            const float mn = fmaxf(m, top), mu = mn == -INFINITY ? 0.f : mn;
            const float f = exp2_fast(m - mu), w = exp2_fast(x - mu);
            m = mn;
            l = l * f + w;
#pragma unroll
            for (int i = 0; i < kPer; ++i) acc[i] *= f;
            for (int j = 0; j < 32; ++j) {
                const int64_t from = __shfl_sync(0xFFFFFFFFu, at, j);
                const float wj = __shfl_sync(0xFFFFFFFFu, w, j);
                if (from < 0) continue;
                const T* const v = reinterpret_cast<const T*>(v_rows + from) + lane * kPer;
#pragma unroll
                for (int i = 0; i < kPer; ++i) acc[i] = fmaf(wj, Elem<T>::to_float(v[i]), acc[i]);
            }
        }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
    const int64_t row = (int64_t)tok * p.q_heads + head, at = (int64_t)part * p.rows + row;
    float* const sum = p.part_o + at * D + lane * kPer;
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum[i] = acc[i];
    if (lane == 0) p.part_ml[at] = make_float2(m, l);
}

// Rows of all requests, (token, head of the group) in token order, 256 to a
// CTA, against the prefix and then against the own pages of the big requests
// among them.  Products and powers are both near their limits, so the two
// tiles of 128 rows take turns: while the tensor core works on one tile's
// weights x V and next q x K, the other tile's softmax runs.
//   warps 0-3, 4-7   softmax of tile 0, 1: a thread holds a row.  Scores come
//                    from tensor memory, weights go back over them as the next
//                    product's first operand; the output stays in tensor
//                    memory until the end.
//   warps 8-9        K and V blocks of 128 keys, cp.async row by row (pages
//                    may end anywhere), through a ring in shared memory that
//                    both tiles read
//   warp 10          one thread issues every product
// The running maximum may lag: an output is rescaled only when a row's
// maximum has grown by more than 2^8 since, else weights simply exceed 1 (by
// 2^8 at most), which costs nothing in fp32 sums or floating-point weights.
// Tensor memory: scores of tile 0, 1 at columns 0, 128; outputs at 256, 384.
// Bound by the turn of the two tiles: a block of 128 keys takes 2830 cycles for 256
// rows, of which the products are 2048 of the tensor core (and of shared memory's
// bandwidth) and the powers 1024.  (12 prompts of 65 to 400 tokens, 64 heads of 128 behind 8192
// keys: 547 us, 1.45 PFLOP/s.)  q and the results moved in pieces side by side, as the
// weights' kernel reads q, take registers from the main loop: 598 us a call for 585.
// Few tiles (a decode step's) do not fill the SMs for long and leave the memory
// idle that the own pages' streams are bound by: then some of the SMs' CTAs take the
// tiles and the others run the streams at the same time.
template <class T, int D>
__global__ void __launch_bounds__(kTileThreads, 1)
attend_tiles_kernel(const __grid_constant__ AttendParams p) {
    using S = TileShape<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ uint64_t bars[2 * S::kStages + 8];
    __shared__ uint32_t tmem_base;
    __shared__ int gave_up;
    __shared__ Seg segs[kMaxSegs];
    __shared__ int32_t num_segs, num_blocks;
    __shared__ uint4 key_mask[kMaskSlots];
    __shared__ uint32_t spoiled[8];       // rows to take again, of each softmax warp
    pdl_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if ((int32_t)blockIdx.x >= p.tile_ctas) {
        pdl_wait();
        constexpr int kBytes = kStages * 2 * WarpRows<T, D>::kTileBytes;
        static_assert(kStreamWarps * kBytes <= S::kSmem, "the streams' rings fit");
        if (warp < kStreamWarps)
            run_stream<T, D>(p, ((int32_t)blockIdx.x - p.tile_ctas) * kStreamWarps + warp, smem_u32(smem) + warp * kBytes);
        return;
    }
    const uint32_t full = smem_u32(bars), empty = full + 8 * S::kStages, s_full = empty + 8 * S::kStages,
                   p_ready = s_full + 16, o_full = p_ready + 32;
    const uint32_t q_smem = smem_u32(smem), kv_smem = q_smem + 2 * S::kStageBytes;
    if (tid == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(full + 8 * i, kCopyArrivals);
            mbar_init(empty + 8 * i, 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(s_full + 8 * t, 1);
            mbar_init(p_ready + 16 * t, 4);
            mbar_init(p_ready + 16 * t + 8, 4);
            mbar_init(o_full + 8 * t, 1);
        }
        gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (tid < 8) spoiled[tid] = 0;
    if (warp == 10) tmem_alloc<512>(smem_u32(&tmem_base));
    pdl_wait();

    const int32_t group = (int32_t)p.by_group.d;
    const int32_t tile = blockIdx.x % p.tiles;
    const int32_t h = blockIdx.x / p.tiles % p.kv_heads;
    const int32_t part = blockIdx.x / p.tiles / p.kv_heads;
    const int32_t live_tokens = min(max(p.seqs.q_start[p.seqs.num_req], 0), p.seqs.num_tokens);
    const int32_t row0 = tile * kTileRows;
    const int32_t live_rows = live_tokens * group;
    uint8_t* const base = p.layer.base();
    if (p.big && warp == 10 && lane < 8) p.again[(int64_t)blockIdx.x * 8 + lane] = 0;
    if (warp == 0 && row0 < live_rows) {
        const int32_t t_first = (int32_t)p.by_group.div((uint32_t)row0);
        const int32_t t_last = (int32_t)p.by_group.div((uint32_t)(min(row0 + kTileRows, live_rows) - 1));
        int32_t count = 0;
        if (p.prefix_len > 0) {
            if (lane == 0) segs[0] = Seg{p.prefix_table, p.prefix_len, 0, 0, -1, 0};
            count = 1;
        }
        if (p.big) {
            auto key = [&](int32_t i) { return p.seqs.q_start[i]; };
            const int32_t r_first = find_request(p.seqs.num_req, t_first, key);
            const int32_t r_last = find_request(p.seqs.num_req, t_last, key);
            for (int32_t r0 = r_first; r0 <= r_last; r0 += 32) {
                const int32_t r = r0 + lane;
                bool on = false;
                Seg s = {};
                if (r <= r_last) {
                    const Req q = load_req(p.seqs, r);
                    if (!q.ok) report(p.status, LMKV_ERR_BAD_LENGTH);
                    on = q.n * group >= kBigRows && q.q0 <= t_last && q.q0 + q.n > t_first;
                    s.table = p.seqs.table + (int64_t)r * p.seqs.table_stride;
                    s.q0 = q.q0;
                    s.n = q.n;
                    s.limit0 = q.len - q.n + 1;
                    s.end = max(0, s.limit0 + min(q.n - 1, t_last - q.q0));
                }
                const uint32_t votes = __ballot_sync(0xFFFFFFFFu, on);
                const int32_t at = count + __popc(votes & ((1u << lane) - 1));
                if (on && at < kMaxSegs) segs[at] = s;       // lengths that overlap could give more
                count = min(count + __popc(votes), kMaxSegs);
            }
        }
        __syncwarp();
        if (lane == 0) {
            int32_t blocks = 0;
            for (int32_t i = 0; i < count; ++i) {
                segs[i].first = blocks;
                blocks += (segs[i].end + kBlock - 1) / kBlock;
            }
            num_segs = count;
            num_blocks = base == nullptr ? 0 : blocks;
            if (base == nullptr) report(p.status, LMKV_ERR_BAD_POINTER);
        }
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = tmem_base;
    if (row0 < live_rows) {
        const int32_t nseg = num_segs;
        const int32_t b0 = (int32_t)((int64_t)num_blocks * part / p.prefix_parts);
        const int32_t b1 = (int32_t)((int64_t)num_blocks * (part + 1) / p.prefix_parts);
        const int tiles = live_rows - row0 > 128 ? 2 : 1;

        if (warp < 8) {
            const int t = warp >> 2;
            const int32_t R = row0 + tid;
            const bool live = R < live_rows;
            const int32_t tok = (int32_t)p.by_group.div((uint32_t)(live ? R : 0));
            const int32_t head = h * group + (live ? R - tok * group : 0);
            if (t < tiles) {
                // my row of q, negated for a negative scale, into shared memory
                const T* src = p.q.row<T>(tok, head);
                const uint32_t dst = q_smem + t * S::kStageBytes + (tid & 127) * 128;
                const uint32_t flip = p.scale_sign < 0 ? 0x80008000u : 0u, all = p.scale_sign == 0 || !live ? 0u : ~0u;
                int4 qv[D / 8];              // all loads on their way before the first is waited for
                if (p.q_vec) {
#pragma unroll
                    for (int c = 0; c < D / 8; ++c) qv[c] = *reinterpret_cast<const int4*>(src + c * 8);
                } else {
#pragma unroll
                    for (int c = 0; c < D / 8; ++c)
                        qv[c] = make_int4((int)load_pair(src + c * 8, p.q_pairs), (int)load_pair(src + c * 8 + 2, p.q_pairs),
                                          (int)load_pair(src + c * 8 + 4, p.q_pairs), (int)load_pair(src + c * 8 + 6, p.q_pairs));
                }
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    const int4 v = qv[c];
                    const uint32_t at = dst + (c >> 3) * S::kHalfBytes + (((c & 7) ^ (tid & 7)) << 4);
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"((v.x ^ flip) & all),
                                 "r"((v.y ^ flip) & all), "r"((v.z ^ flip) & all), "r"((v.w ^ flip) & all)
                                 : "memory");
                }
                fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_ready + 16 * t + 8);     // its phase 0: q is there

                int32_t own = -1;
                for (int32_t i = 0; i < nseg; ++i)
                    if (segs[i].n >= 0 && tok >= segs[i].q0 && tok < segs[i].q0 + segs[i].n) own = i;
                const uint32_t lane_base = tmem + ((uint32_t)(warp & 3) << 21);     // lane 32 * (warp % 4)
                const uint32_t s_at = lane_base + t * 128, o_at = lane_base + 256 + t * 128;
                const float scale = p.scale_log2;
                float m = -INFINITY;              // what weights are relative to, in units of raw scores
                float2 l2 = make_float2(0.f, 0.f);
                int32_t si = 0;
                bool ok = true;
                for (int32_t b = b0; b < b1; ++b) {
                    while (si + 1 < nseg && b >= segs[si + 1].first) ++si;
                    const Seg& sg = segs[si];
                    const int32_t k = (b - sg.first) * kBlock;
                    int32_t seen = min(sg.end - k, kBlock);
                    if (sg.n >= 0) seen = si == own ? min(seen, sg.limit0 + (tok - sg.q0) - k) : 0;
                    if (!mbar_wait(s_full + 8 * t, (b - b0) & 1, &gave_up)) {
                        ok = false;
                        break;
                    }
                    if (t == tiles - 1 && (tid & 127) == 0) {
                        // every product up to these scores is done: K of this block and V of the last are free
                        const int32_t j = b - b0;
                        mbar_arrive(empty + 8 * (2 * j % S::kStages));
                        if (j > 0) mbar_arrive(empty + 8 * ((2 * j - 1) % S::kStages));
                    }
                    fence_after_sync();
                    const uint32_t* const words = reinterpret_cast<const uint32_t*>(&key_mask[(b - b0) % kMaskSlots]);
                    const bool whole = __all_sync(0xFFFFFFFFu, seen >= kBlock && (words[0] & words[1] & words[2] & words[3]) == ~0u);
                    // scores of 32 keys, those not seen as -infinity
                    auto take = [&](uint32_t (&x)[32], int i) {
                        if (whole) return;
                        const int32_t n = seen - 32 * i;
                        const uint32_t bits = words[i] & (n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (!((bits >> j) & 1)) x[j] = 0xFF800000u;
                    };
                    uint32_t x[4][32];
                    float mx = -INFINITY, my = -INFINITY;
                    tmem_ld32(x[0], s_at);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        wait_ld();
                        loaded(x[i]);
                        if (i < 3) tmem_ld32(x[i + 1], s_at + 32 * (i + 1));
                        take(x[i], i);
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            mx = max3(mx, __uint_as_float(x[i][j]), __uint_as_float(x[i][j + 1]));
                            my = max3(my, __uint_as_float(x[i][j + 2]), __uint_as_float(x[i][j + 3]));
                        }
                    }
                    mx = fmaxf(mx, my);
                    // weights are relative to m; m moves when it would be exceeded by more than 2^8
                    const bool grow = mx > m && !((mx - m) * scale <= 8.f);
                    if (__any_sync(0xFFFFFFFFu, grow)) {
                        const float mn = grow ? fmaxf(mx, p.lowest) : m;
                        const float f = grow && m != -INFINITY ? exp2_fast((m - mn) * scale) : grow ? 0.f : 1.f;
                        m = mn;
                        l2.x *= f;
                        l2.y *= f;
                        if (b > b0) {
                            // the scores were there, so the product before them, into the output, is done
#pragma unroll 1
                            for (int c = 0; c < D; c += 16) tmem_scale16(o_at + c, f);
                        }
                    }
                    const float neg = m == -INFINITY ? 0.f : -m * scale;
                    const float2 sc2 = make_float2(scale, scale), ng2 = make_float2(neg, neg);
                    float2 sums[4] = {l2, make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t w[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            float2 e = fma2(make_float2(__uint_as_float(x[i][2 * j]), __uint_as_float(x[i][2 * j + 1])),
                                            sc2, ng2);
                            e.x = exp2_fast(e.x);
                            e.y = exp2_fast(e.y);
                            sums[j & 3] = add2(sums[j & 3], e);
                            // weights are rounded to T for the product with V, the sum takes them whole
                            w[j] = Elem<T>::pack(e.x, e.y);
                        }
                        tmem_st16(s_at + 16 * i, w);       // over scores that have been read
                        if (i & 1) {                       // 64 keys' weights are there
                            wait_st();
                            fence_before_sync();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(p_ready + 16 * t + 8 * (i >> 1));
                        }
                    }
                    l2 = add2(add2(sums[0], sums[1]), add2(sums[2], sums[3]));
                }
                // my row of the result
                const float l = l2.x + l2.y;
                if (ok && b1 > b0) ok = mbar_wait(o_full + 8 * t, 0, &gave_up);
                if (ok) {
                    fence_after_sync();
                    // without a prefix a small request's rows have nothing here
                    const bool wanted = live && (own >= 0 || p.prefix_len > 0);
                    const bool final = own >= 0 && p.prefix_parts == 1;
                    const int64_t row = (int64_t)tok * p.q_heads + head;
                    const int64_t at = (int64_t)part * p.rows + row;
                    const float m2 = m == -INFINITY ? -INFINITY : m * scale;
                    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
                    T* const out = p.out.row<T>(tok, head);
                    float z = 0.f;                    // NaN once a sum is not finite
                    // (rolled: its addresses would take registers from the main loop, 614 : 580 us)
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t y[32];
                        if (b1 > b0) {
                            tmem_ld32(y, o_at + 32 * c);
                            wait_ld();
                            loaded(y);
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; ++j) y[j] = 0u;
                        }
#pragma unroll
                        for (int j = 0; j < 32; ++j) z = fmaf(__uint_as_float(y[j]), 0.f, z);
                        if (!wanted) continue;
                        if (final) {
#pragma unroll
                            for (int j = 0; j < 32; j += 8) {
                                uint32_t w[4];
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    w[i] = Elem<T>::pack(__uint_as_float(y[j + 2 * i]) * inv,
                                                         __uint_as_float(y[j + 2 * i + 1]) * inv);
                                T* dst = out + 32 * c + j;
                                if (p.out_vec) {
                                    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
                                } else {
                                    uint16_t* d16 = reinterpret_cast<uint16_t*>(dst);
#pragma unroll
                                    for (int i = 0; i < 4; ++i) {
                                        d16[2 * i] = (uint16_t)w[i];
                                        d16[2 * i + 1] = (uint16_t)(w[i] >> 16);
                                    }
                                }
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; j += 4)
                                *reinterpret_cast<uint4*>(p.part_o + at * D + 32 * c + j) =
                                    make_uint4(y[j], y[j + 1], y[j + 2], y[j + 3]);
                        }
                    }
                    if (wanted && final && p.lse != nullptr)
                        p.lse[row] = ((m == -INFINITY ? 0.f : m2) + log2f(l)) * kLn2;
                    if (wanted && !final) p.part_ml[at] = make_float2(m2, l);
                    // rows to take again: spoiled ones (keys of other requests, and a sum that is not finite), and those
                    // whose scores are far from 0
                    const bool others = nseg > (p.prefix_len > 0 ? 1 : 0) + (own >= 0 ? 1 : 0);
                    const bool spoilt = others && z != 0.f && l < INFINITY;
                    const bool far = m != -INFINITY && (m <= p.lowest || m2 > kFarScore);
                    const uint32_t again = __ballot_sync(0xFFFFFFFFu, wanted && (spoilt || far));
                    if (lane == 0) spoiled[warp] = again;
                }
            }
        } else if (warp < 8 + kLoadWarps) {
            BlockCopy<D> rows(p.layer, base, kv_smem, warp - 8);
            const uint8_t* const from_k = rows.piece(h);
            const uint8_t* const from_v = from_k + p.layer.half_bytes();
            int32_t si = 0, item = 0;
            auto lookup = [&](int32_t b) {
                while (si + 1 < nseg && b >= segs[si + 1].first) ++si;
                rows.lookup(segs[si].table, (b - segs[si].first) * kBlock, segs[si].end);
            };
            bool ok = true;
            if (b0 < b1) lookup(b0);
            for (int32_t b = b0; b < b1 && ok; ++b) {
                rows.take(p.status);
                if (b + 1 < b1) lookup(b + 1);
#pragma unroll 1
                for (int kv = 0; kv < 2; ++kv, ++item) {
                    const int st = item % S::kStages;
                    if (item >= S::kStages && !mbar_wait(empty + 8 * st, (item / S::kStages - 1) & 1, &gave_up)) {
                        ok = false;
                        break;
                    }
                    if (kv == 0) rows.put_mask(reinterpret_cast<uint32_t*>(&key_mask[(b - b0) % kMaskSlots]));
                    rows.copy(kv ? from_v : from_k, st * S::kStageBytes);
                    copies_arrive(full + 8 * st);
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        } else {
            if (warp == 10 && b1 > b0) {
                constexpr uint32_t qk = instr_desc<T, kBlock, false>(), pv = instr_desc<T, D, true>();
                // all of tensor memory is this CTA's, so its columns count from 0
                constexpr uint32_t kScores = 0, kOut = 256;
                const int32_t blocks = b1 - b0;
                const uint32_t lead = elect_lead();
                const Desc q0 = desc_k_major(q_smem), k0 = desc_k_major(kv_smem),
                           v0 = desc_n_major(kv_smem, S::kHalfBytes);
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
                bool ok = landed(0, 0);
                for (int t = 0; t < tiles && ok; ++t) {
                    ok = mbar_wait(p_ready + 16 * t + 8, 0, &gave_up);
                    if (ok) scores(t, 0);
                }
                advance(ks, kph);
                ok = ok && landed(vs, vph);
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
                            ok = ok && mbar_wait(p_ready + 16 * t + 8 * half, (j + half) & 1, &gave_up);
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
                    advance(ks, kph);
                }
            }
        }
    }
    __syncwarp();
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (tid == 0 && gave_up) report(p.status, LMKV_ERR_TIMEOUT);
    if (warp == 10) tmem_free<512>(tmem);
    if (warp < 8) {
        for (uint32_t left = spoiled[warp]; left != 0; left &= left - 1)
            take_row<T, D>(p, segs, num_segs, num_blocks, base, h, part, row0 + warp * 32 + __ffs(left) - 1);
    }
}

// Joins the parts of the rows that have more than one: a warp per row, of all
// rows (kOwnRows false) or of the small requests' only.  (2048 rows of 128 in about ten
// parts: 7.7 us.)
template <class T, int D, bool kOwnRows>
__global__ void __launch_bounds__(256) attend_join_kernel(const __grid_constant__ AttendParams p) {
    constexpr int kPer = D / 32;
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int32_t group = (int32_t)p.by_group.d;
    int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    int32_t r, row_of_r, h;
    Req q;
    if (kOwnRows) {
        if (i >= (int64_t)p.seqs.num_req * p.own_cap * p.kv_heads) return;
        h = (int32_t)(i % p.kv_heads);
        i /= p.kv_heads;
        r = (int32_t)(i / p.own_cap);
        row_of_r = (int32_t)(i % p.own_cap);
        q = load_req(p.seqs, r);
        if (row_of_r >= q.n * group) return;
    } else {
        if (i >= p.rows) return;
        const int32_t tok = (int32_t)(i / p.q_heads), head = (int32_t)(i % p.q_heads);
        r = find_request(p.seqs.num_req, tok, [&](int32_t k) { return p.seqs.q_start[k]; });
        q = load_req(p.seqs, r);
        if (!q.ok && lane == 0) report(p.status, LMKV_ERR_BAD_LENGTH);
        if (tok < q.q0 || tok >= q.q0 + q.n) return;       // a padded row
        h = head / group;
        row_of_r = (tok - q.q0) * group + (head - h * group);
    }
    const bool big = p.big && q.n * group >= kBigRows;
    if (big ? p.prefix_parts == 1 : p.own_final) return;   // written already
    const int32_t n = (int32_t)p.by_group.div((uint32_t)row_of_r);
    const int32_t tok = q.q0 + n, head = h * group + (row_of_r - n * group);
    const int64_t row = (int64_t)tok * p.q_heads + head;
    const int32_t shared = big || p.prefix_len > 0 ? p.prefix_parts : 0;
    const int32_t tile_no = r * p.own_tiles + row_of_r / kRowTile, row_of_tile = row_of_r % kRowTile;
    int32_t g = 0, own = 0;                // the tile's own parts: streams g, g + 1, ...
    if (!big && q.len > 0) {
        own = 1;
        if (p.streams > 0) {
            // (clamped: lengths that change while the call runs give a wrong sum, not a wild address)
            const int2 range = p.own_range[tile_no];
            g = min(max(range.x, 0), p.streams - 1);
            own = min(max(range.y, g), p.streams - 1) - g + 1;
        }
    }
    const int32_t parts = shared + own;
    // m and l of 32 parts at a time, one a lane; then the parts' sums, whose loads
    // no longer wait for one another
    const int64_t own_stride = (int64_t)p.tile_rows * p.kv_heads;
    const int64_t own0 = p.own_part(g, tile_no, row_of_tile, h);
    auto place = [&](int32_t s) { return s < shared ? (int64_t)s * p.rows + row : own0 + (s - shared) * own_stride; };
    float top = -INFINITY, sum = 0.f, acc[kPer] = {};
    for (int32_t s0 = 0; s0 < parts; s0 += 32) {
        const int32_t n = min(32, parts - s0);
        const float2 v = lane < n ? p.part_ml[place(s0 + lane)] : make_float2(-INFINITY, 0.f);
        float mn = v.x;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, d));
        mn = fmaxf(mn, top);
        const float mu = mn == -INFINITY ? 0.f : mn;
        const float f = exp2_fast(v.x - mu), before = exp2_fast(top - mu);
        top = mn;
        float l = v.y * f;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
        sum = sum * before + l;
#pragma unroll
        for (int k = 0; k < kPer; ++k) acc[k] *= before;
        constexpr int kAhead = 8;
        for (int32_t s = 0; s < n; s += kAhead) {
            float x[kAhead][kPer];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const float* src = p.part_o + place(min(s0 + s + u, parts - 1)) * D + lane * kPer;
                if constexpr (kPer == 4) *reinterpret_cast<float4*>(x[u]) = *reinterpret_cast<const float4*>(src);
                else *reinterpret_cast<float2*>(x[u]) = *reinterpret_cast<const float2*>(src);
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const float fs = __shfl_sync(0xFFFFFFFFu, f, (s + u) & 31);
                if (s + u < n) {
#pragma unroll
                    for (int k = 0; k < kPer; ++k) acc[k] += x[u][k] * fs;
                }
            }
        }
    }
    const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
    T* dst = p.out.row<T>(tok, head) + lane * kPer;
#pragma unroll
    for (int k = 0; k < kPer; ++k) dst[k] = Elem<T>::from_float(acc[k] * inv);
    if (lane == 0 && p.lse != nullptr)
        p.lse[row] = ((top == -INFINITY ? 0.f : top) + log2f(sum)) * kLn2;
}

// ---- host ---------------------------------------------------------------

struct Plan {
    int32_t row_tiles, tiles, prefix_parts, prefix_span;
    int32_t own_cap, own_tiles, tile_rows, streams;
    bool big, own_final, join;
    int32_t stream_ctas;      // of the tile kernel; 0: the streams have their own launch
    int64_t rows;
    uint64_t o_bytes, ml_bytes, range_bytes, bytes;
};

constexpr int32_t kStreamKeys = 16 * kWarps * kChunk;     // own contexts longer than this go by streams

// Scores of a prefix (rows x keys x KV heads) from which its rows are taken by tiles.
// Below, the row kernel's 16 rows at a time read the prefix again from L2 in
// less time than tiles take to begin and to be joined.  (Rows against tiles,
// us, 8 heads: 128 rows x 1000 keys 25 : 43, x 8192 48 : 51; 256 x 3000 48 : 57, x 8192
// 72 : 63; 512 x 1000 50 : 63, x 3000 67 : 69, x 8192 117 : 78; 2 heads, 2048 x 3000 66 : 69; 32
// heads, 128 x 3000 68 : 70, 256 x 3000 108 : 95.)
constexpr double kTileScores = 12 << 20;

// Splits of `keys` keys over `ctas` CTAs each: enough for six on every SM (two rounds of three),
// none below 128 keys.
void split(int64_t ctas, int32_t keys, int32_t* splits, int32_t* span) {
    const int64_t want = (6 * kSms + ctas - 1) / ctas;
    const int64_t most = (keys + 127) / 128;
    const int64_t n = want < most ? want : most;
    int64_t s = (keys + n - 1) / n;
    s = (s + 63) / 64 * 64;
    *span = (int32_t)s;
    *splits = (int32_t)((keys + s - 1) / s);
}

// Parts of the tile kernel's blocks: the number that leaves the fewest rounds
// of one CTA per SM, a part's cost being its blocks and the writing and
// joining of its rows (about two blocks' time).  More than kMostRounds rounds would gain 3 % at most,
// for more workspace.
constexpr int32_t kMostParts = 64, kMostRounds = 16;
int32_t tile_parts(int64_t ctas, int64_t blocks) {
    int32_t best = 1;
    double best_cost = 0;
    for (int32_t n = 1; n <= kMostParts && n <= blocks; ++n) {
        const int64_t rounds = (ctas * n + kSms - 1) / kSms;
        if (n > 1 && rounds > kMostRounds) break;
        const double cost = (double)rounds * ((double)((blocks + n - 1) / n) + (n > 1 ? 2.0 : 0.0)) + (n > 1 ? 1.0 : 0.0);
        if (n == 1 || cost < best_cost) {
            best = n;
            best_cost = cost;
        }
    }
    return best;
}

// The most CTAs that tile_parts makes of `ctas` for any number of blocks up to this.  With x =
// ctas / kSms and b blocks, n parts cost more than x (b + 2 n) + 1; so n is not taken unless that is
// below the cost of a single part, ceil(x) b, nor, where some n1 parts fill one round, unless it
// is below theirs, b / n1 + 4.
int64_t most_tile_ctas(int64_t ctas, int64_t blocks) {
    const double x = (double)ctas / kSms, b = (double)blocks;
    const int64_t n1 = kSms / ctas;
    const double bound = n1 <= 1 ? (std::ceil(x) - x) * b : (1.0 / (double)n1 - x) * b + 3.0;
    int64_t most = (int64_t)(bound * kSms / 2) + 1;
    if (most < n1 * ctas) most = n1 * ctas;             // (and those beside streams)
    if (most > kMostRounds * kSms) most = kMostRounds * kSms;
    if (most > ctas * blocks) most = ctas * blocks;
    return most < ctas ? ctas : most;
}

Plan make_plan(const lmkv_pool_t* pool, int32_t q_heads, int32_t num_tokens, int32_t num_req, int32_t max_new,
               int32_t prefix_len, int32_t max_kv_len) {
    Plan x = {};
    const int64_t group = q_heads / pool->num_kv_heads;
    const int64_t batch_rows = (int64_t)num_tokens * group;            // per KV head
    // (a bound of 0 still has rows to look at: lengths beyond it are reported)
    const int64_t req_rows = (int64_t)(max_new < 1 ? 1 : max_new < num_tokens ? max_new : num_tokens) * group;
    x.rows = (int64_t)num_tokens * q_heads;
    x.big = req_rows >= kBigRows;
    if (x.big || (batch_rows > kRowTile && (double)batch_rows * prefix_len * pool->num_kv_heads > kTileScores)) {
        x.tiles = (int32_t)((batch_rows + kTileRows - 1) / kTileRows);
        const int64_t blocks = ((int64_t)prefix_len + kBlock - 1) / kBlock +
                               (x.big ? ((int64_t)max_kv_len + kBlock - 1) / kBlock : 0);
        x.prefix_parts = tile_parts((int64_t)x.tiles * pool->num_kv_heads, blocks);
    } else if (prefix_len > 0) {
        x.row_tiles = (int32_t)((batch_rows + kRowTile - 1) / kRowTile);
        split((int64_t)x.row_tiles * pool->num_kv_heads, prefix_len, &x.prefix_parts, &x.prefix_span);
    }
    x.own_cap = (int32_t)(x.big ? kBigRows - 1 : req_rows);
    x.own_tiles = (x.own_cap + kRowTile - 1) / kRowTile;
    x.tile_rows = x.own_cap < kRowTile ? x.own_cap : kRowTile;
    // A CTA per row tile while that is at most 16 chunks a warp, else streams: as many warps
    // as fit at once.  (CTAs against streams, us: 4 requests of 512 keys 15 : 19, 1024 23 : 23,
    // 2048 35 : 26; 32 requests 23 : 30, 37 : 44, 62 : 67, all of the same length, which is where
    // streams gain least.)  Streams that run beside the tiles gain at any length.  (One launch
    // after the other against beside: 64 requests behind 16384 keys, of 32 keys 64 : 51, 512 100 :
    // 68, 2048 178 : 132; 128 behind 8192, 65 : 46, 118 : 80, 239 : 205.)
    const int64_t heads = pool->num_kv_heads, tile_heads = x.tiles * heads;
    const bool beside = !x.big && x.tiles > 0 && tile_heads <= kSms / 2;
    if (max_kv_len > (beside ? 0 : kStreamKeys)) {
        int64_t warps = kRowCtas * kSms * kWarps;
        if (beside) {
            // The SMs are divided by what each side would take of them: 2.3 us for 256 rows x 128
            // keys with its share of start and end, 45 GB/s of an SM for the own pages, half of
            // whose bound is there; the tiles get three eighths at least, as the bound may be
            // far off.  (64 users behind 16384 tokens, us by SMs for the tiles: 64: 52, 72: 50, 80: 53,
            // 88: 57; one launch after the other: 70.)
            const double tile_us = 2.3 * (double)tile_heads * (double)((prefix_len + kBlock - 1) / kBlock);
            const double own_us = (double)num_req * heads * max_kv_len * 0.5 * pool->head_dim * 4 / 45e3;
            int64_t n = (int64_t)(kSms * tile_us / (tile_us + own_us));
            n = n < kSms * 3 / 8 ? kSms * 3 / 8 : n > kSms - 16 ? kSms - 16 : n;
            const int64_t blocks = (prefix_len + kBlock - 1) / kBlock;
            int64_t parts = n / tile_heads > 0 ? n / tile_heads : 1;
            parts = parts > blocks ? blocks : parts;
            x.prefix_parts = (int32_t)parts;
            x.stream_ctas = (int32_t)(kSms - tile_heads * parts);
            warps = (int64_t)x.stream_ctas * kStreamWarps;
        }
        x.streams = (int32_t)(warps / heads > 0 ? warps / heads : 1);
        if (x.stream_ctas > 0) x.stream_ctas = (int32_t)((x.streams * heads + kStreamWarps - 1) / kStreamWarps);
    }
    x.own_final = prefix_len == 0 && x.streams == 0;
    x.join = x.prefix_parts > 1 || !x.own_final;
    const uint64_t own_rows = ((uint64_t)x.streams + (uint64_t)num_req * x.own_tiles) * x.tile_rows * pool->num_kv_heads;
    const uint64_t parts = x.join ? (uint64_t)x.prefix_parts * x.rows + own_rows : 0;
    x.o_bytes = parts * pool->head_dim * 4;
    x.ml_bytes = parts * 8;
    x.range_bytes = x.join ? (uint64_t)num_req * x.own_tiles * 8 : 0;
    x.bytes = x.o_bytes + x.ml_bytes + x.range_bytes +
              (x.big ? (uint64_t)x.tiles * pool->num_kv_heads * x.prefix_parts * 32 : 0);
    return x;
}

// Bytes that hold the plan of any call within these bounds (a plan's own need falls where
// a larger batch needs no parts).
uint64_t most_bytes(const lmkv_pool_t* pool, int32_t q_heads, int32_t num_tokens, int32_t num_req, int32_t max_new,
                    int32_t prefix_len, int32_t max_kv_len) {
    const int64_t heads = pool->num_kv_heads, group = q_heads / heads;
    const int64_t rows = (int64_t)num_tokens * q_heads;
    const int64_t req_rows = (int64_t)(max_new < 1 ? 1 : max_new < num_tokens ? max_new : num_tokens) * group;
    const bool big = req_rows >= kBigRows;
    const bool far = max_kv_len > kStreamKeys;
    if (!big && !far && prefix_len == 0) return 0;              // one part, written at once
    // the prefix's parts, by tiles (of every number of them up to the call's) and by rows
    uint64_t parts = 0, again = 0;
    if (big || prefix_len > 0) {
        const int64_t blocks = ((int64_t)prefix_len + kBlock - 1) / kBlock +
                               (big ? ((int64_t)max_kv_len + kBlock - 1) / kBlock : 0);
        const int64_t tiles = ((int64_t)num_tokens * group + kTileRows - 1) / kTileRows;
        int64_t ctas = tiles * heads;
        for (int64_t t = 1; t <= tiles && t * heads <= kMostRounds * kSms; ++t) {
            const int64_t most = most_tile_ctas(t * heads, blocks < 1 ? 1 : blocks);
            const int64_t tile_rows = t * kTileRows * heads < rows ? t * kTileRows * heads : rows;
            const uint64_t n = (uint64_t)(most / (t * heads)) * tile_rows;
            if (n > parts) parts = n;
            if (most > ctas) ctas = most;
        }
        if ((uint64_t)rows > parts) parts = rows;
        if (big) again = (uint64_t)ctas * 32;
    }
    if (prefix_len > 0) {
        // split() makes two rounds of kRowCtas an SM, and as many again by rounding up
        const int64_t by_keys = ((int64_t)prefix_len + 127) / 128 * rows, by_ctas = (int64_t)4 * kRowCtas * kSms * kRowTile;
        const uint64_t n = by_keys < by_ctas ? by_keys : by_ctas;
        if (n > parts) parts = n;
    }
    const int64_t warps = far ? kRowCtas * kSms * kWarps : prefix_len > 0 && max_kv_len > 0 ? kSms * kStreamWarps : 0;
    const int64_t streams = warps == 0 ? 0 : warps / heads > 0 ? warps / heads : 1;
    const int64_t own_cap = big ? kBigRows - 1 : req_rows, own_tiles = (own_cap + kRowTile - 1) / kRowTile;
    const uint64_t own_rows = ((uint64_t)streams + (uint64_t)num_req * own_tiles) *
                              (own_cap < kRowTile ? own_cap : kRowTile) * heads;
    return (parts + own_rows) * ((uint64_t)pool->head_dim * 4 + 8) + (uint64_t)num_req * own_tiles * 8 + again;
}

int check_shape(const lmkv_pool_t* pool) {
    const int rc = lmkv_internal_check_pool(pool);
    if (rc != LMKV_OK) return rc;
    if (pool->elem_bytes != 2 || (pool->head_dim != 64 && pool->head_dim != 128)) return LMKV_ERR_UNSUPPORTED;
    return LMKV_OK;
}

template <class T, int D, bool kBig>
int attend_launches(AttendParams& p, const Plan& x, void* stream) {
    constexpr int smem = kWarps * kStages * 2 * kChunk * D * 2;
    int rc = allow_smem<attend_rows_kernel<T, D, kBig>, smem>();
    if (rc == LMKV_OK) rc = allow_smem<attend_streams_kernel<T, D, kBig>, smem>();
    if (rc == LMKV_OK) rc = allow_smem<attend_tiles_kernel<T, D>, TileShape<D>::kSmem>();
    if (rc == LMKV_OK)
        rc = launch(attend_tiles_kernel<T, D>, (int64_t)x.tiles * p.kv_heads * x.prefix_parts + x.stream_ctas, kTileThreads,
                    TileShape<D>::kSmem, stream, 1, p);
    if (rc != LMKV_OK) return rc;
    // the own pages, and the prefix where tiles do not have it; beside them the rows to take again
    const int64_t windows = kBig ? (int64_t)x.tiles * (kTileRows / kRowTile) * p.kv_heads : 0;
    // (CTAs for them: what the first round has left)
    auto again = [&](int64_t ctas) {
        const int64_t left = kRowCtas * kSms - ctas, most = left > kSms / 2 ? left : kSms / 2;
        return windows < most ? windows : most;
    };
    if (x.streams == 0 || x.stream_ctas > 0) {
        // (with no room for cached tokens too: lengths beyond that bound are reported)
        const int64_t ctas = ((int64_t)x.row_tiles * x.prefix_parts +
                              (x.streams == 0 ? (int64_t)x.own_tiles * p.seqs.num_req : 0)) * p.kv_heads;
        p.again_cta = (int32_t)ctas;
        rc = launch(attend_rows_kernel<T, D, kBig>, ctas + again(ctas), kWarps * 32, smem, stream, 1, p);
    } else {
        rc = launch(attend_rows_kernel<T, D, kBig>, (int64_t)x.row_tiles * x.prefix_parts * p.kv_heads, kWarps * 32, smem,
                    stream, 1, p);
        const int64_t ctas = ((int64_t)x.streams * p.kv_heads + kWarps - 1) / kWarps;
        p.again_cta = (int32_t)ctas;
        if (rc == LMKV_OK)
            rc = launch(attend_streams_kernel<T, D, kBig>, ctas + again(ctas), kWarps * 32, smem, stream, 1, p);
    }
    if (rc != LMKV_OK || !x.join) return rc;
    // the small requests' rows, where there are no others or those are done already
    if (!x.big || x.prefix_parts <= 1)
        return launch(attend_join_kernel<T, D, true>, ((int64_t)p.seqs.num_req * x.own_cap * p.kv_heads + 7) / 8, 256, 0,
                      stream, 1, p);
    return launch(attend_join_kernel<T, D, false>, (x.rows + 7) / 8, 256, 0, stream, 1, p);
}

template <class T, int D>
int attend_typed(AttendParams& p, const Plan& x, void* stream) {
    return x.big ? attend_launches<T, D, true>(p, x, stream) : attend_launches<T, D, false>(p, x, stream);
}

}  // namespace

extern "C" {

int lmkv_attend_workspace_bytes(const lmkv_pool_t* pool, int32_t num_q_heads, int32_t num_tokens, int32_t num_req,
                                int32_t max_new, int64_t prefix_len, int32_t max_kv_len, uint64_t* bytes) {
    const int rc = check_shape(pool);
    if (rc != LMKV_OK) return rc;
    if (bytes == nullptr || num_q_heads <= 0 || num_q_heads % pool->num_kv_heads != 0 || num_tokens < 0 ||
        num_req < 0 || max_new < 0 || max_kv_len < 0 || prefix_len < 0 || prefix_len > INT32_MAX - 65536 ||
        (int64_t)num_tokens * num_q_heads > (int64_t)1 << 30)
        return LMKV_ERR_INVALID_ARG;
    *bytes = num_tokens == 0 || num_req == 0
                 ? 0 : most_bytes(pool, num_q_heads, num_tokens, num_req, max_new, (int32_t)prefix_len, max_kv_len);
    return LMKV_OK;
}

int lmkv_attend_layer(const lmkv_pool_t* pool, int32_t dtype, int32_t layer, const lmkv_batch_t* batch,
                      int32_t num_q_heads, const lmkv_rows_t* q, const int32_t* prefix_table, int64_t prefix_len,
                      float scale, const lmkv_rows_t* out, float* lse, void* workspace, uint64_t workspace_bytes,
                      int32_t* d_status, void* stream) {
    int rc = check_shape(pool);
    if (rc != LMKV_OK) return rc;
    if (!type_fits(pool, dtype)) return LMKV_ERR_UNSUPPORTED;
    if (layer < 0 || layer >= pool->num_layers || !std::isfinite(scale * kLog2e)) return LMKV_ERR_INVALID_ARG;
    rc = check_batch(pool, batch, num_q_heads);
    if (rc != LMKV_OK) return rc;
    if (prefix_len < 0 || prefix_len > INT32_MAX - 65536 || batch->max_kv_len > INT32_MAX - 65536 ||
        (prefix_len > 0 && prefix_table == nullptr))
        return LMKV_ERR_INVALID_ARG;
    if (batch->num_req == 0 || batch->num_tokens == 0) return LMKV_OK;
    if (!rows_ok(q, 2) || !rows_ok(out, 2)) return LMKV_ERR_INVALID_ARG;
    const Plan x = make_plan(pool, num_q_heads, batch->num_tokens, batch->num_req, batch->max_new,
                             (int32_t)prefix_len, batch->max_kv_len);
    if (x.bytes > 0 && (workspace == nullptr || workspace_bytes < x.bytes)) return LMKV_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(workspace) & 15) return LMKV_ERR_MISALIGNED;
    if (out->data == q->data) return LMKV_ERR_INVALID_ARG;
    AttendParams p = {};
    p.layer = Layer::of(pool, layer);
    p.seqs = Seqs::of(batch);
    p.q = Rows::of(q);
    p.out = Rows::of(out);
    p.lse = lse;
    p.prefix_table = prefix_table;
    p.status = d_status;
    p.part_o = static_cast<float*>(workspace);
    p.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + x.o_bytes);
    p.own_range = reinterpret_cast<int2*>(static_cast<uint8_t*>(workspace) + x.o_bytes + x.ml_bytes);
    p.again = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(workspace) + x.o_bytes + x.ml_bytes + x.range_bytes);
    p.scale_sign = scale > 0.f ? 1 : scale < 0.f ? -1 : 0;
    p.scale_log2 = scale == 0.f ? 1.f : std::fabs(scale) * kLog2e;
    p.lowest = -kFarScore / p.scale_log2;
    p.prefix_len = (int32_t)prefix_len;
    p.q_heads = num_q_heads;
    p.kv_heads = pool->num_kv_heads;
    p.rows = (int32_t)x.rows;
    p.row_tiles = x.row_tiles;
    p.tiles = x.tiles;
    p.tile_ctas = x.tiles * p.kv_heads * x.prefix_parts;
    p.prefix_parts = x.prefix_parts;
    p.prefix_span = x.prefix_span;
    p.own_cap = x.own_cap;
    p.own_tiles = x.own_tiles;
    p.tile_rows = x.tile_rows;
    p.streams = x.streams;
    p.big = x.big;
    p.own_final = x.own_final;
    auto aligned = [](const lmkv_rows_t* r, int64_t to) {
        return reinterpret_cast<uintptr_t>(r->data) % to == 0 && r->token_stride * 2 % to == 0 && r->head_stride * 2 % to == 0;
    };
    p.q_vec = aligned(q, 16);
    p.out_vec = aligned(out, 16);
    p.q_pairs = aligned(q, 4);
    p.by_group = FastDiv((uint32_t)(num_q_heads / pool->num_kv_heads));
    if (dtype == LMKV_BF16)
        return pool->head_dim == 64 ? attend_typed<__nv_bfloat16, 64>(p, x, stream)
                                    : attend_typed<__nv_bfloat16, 128>(p, x, stream);
    return pool->head_dim == 64 ? attend_typed<__half, 64>(p, x, stream) : attend_typed<__half, 128>(p, x, stream);
}

}  // extern "C"
