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
#include "lmkv_mma.cuh"

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

struct AttendParams {
    Layer layer;
    Seqs seqs;
    Rows q, out;
    float* lse;
    const int32_t* prefix_table;
    int32_t* status;
    float* part_o;          // [splits][rows][D]
    float2* part_ml;        // [splits][rows]: m (powers of 2), l
    float scale_log2;
    int32_t prefix_len;
    int32_t q_heads, kv_heads;
    int32_t rows;           // num_tokens * q_heads
    int32_t prefix_tiles;   // row tiles of the prefix part
    int32_t prefix_splits, prefix_span;   // splits of the prefix, keys in each
    int32_t own_slots;      // row tile slots of the own part
    int32_t own_splits, own_span;
    bool direct;            // one part in all: it writes out and lse itself
    bool q_pairs;           // q rows are 4-byte aligned
    FastDiv by_group;
};

constexpr int kRowTile = 16;      // rows of a tile: one mma.sync operand
constexpr int kWarps = 4;
constexpr int kChunk = 16;        // keys a warp takes at a time
constexpr int kStages = 3;
constexpr float kLn2 = 0.69314718055994530942f;

// A tile's place in the batch.
struct Tile {
    const int32_t* table;
    int32_t k0, k1;        // keys of this part
    int32_t h;             // KV head
    int32_t part;          // index into the partial results
    int32_t t0, row0;      // row i of the tile is row row0 + i of the rows that begin at token t0
    int32_t nrows;         // rows from row0 on (may exceed the tile)
    int32_t limit0;        // row row0 + i sees keys below limit0 + (row0 + i) / group * causal
    int32_t causal;
};

// The tile of CTA `bid`; false when it has none.  Called by whole warps.
// Row tiles of the own part: request r's rows begin at slot
// floor(q_start[r] * group / 16) + r, which leaves room for every request's
// last partial tile, so the slots need no scan over the requests.
__device__ __forceinline__ bool find_tile(const AttendParams& p, int32_t bid, int rows_per_tile, Tile& t) {
    const int32_t group = (int32_t)p.by_group.d;
    const int32_t prefix_ctas = p.prefix_tiles * p.kv_heads * p.prefix_splits;
    if (bid < prefix_ctas) {
        const int32_t tile = bid % p.prefix_tiles;
        const int32_t x = bid / p.prefix_tiles;
        t.h = x % p.kv_heads;
        t.part = x / p.kv_heads;
        t.table = p.prefix_table;
        t.k0 = t.part * p.prefix_span;
        t.k1 = min(t.k0 + p.prefix_span, p.prefix_len);
        t.t0 = 0;
        t.row0 = tile * rows_per_tile;
        const int32_t end = min(max(p.seqs.q_start[p.seqs.num_req], 0), p.seqs.num_tokens);
        t.nrows = end * group - t.row0;
        t.limit0 = p.prefix_len;
        t.causal = 0;
        return t.nrows > 0;
    }
    bid -= prefix_ctas;
    t.h = bid % p.kv_heads;
    const int32_t x = bid / p.kv_heads;
    const int32_t slot = x % p.own_slots;
    const int32_t split = x / p.own_slots;
    auto first_slot = [&](int32_t i) { return (int32_t)((int64_t)p.seqs.q_start[i] * group / rows_per_tile) + i; };
    const int32_t r = find_request(p.seqs.num_req, slot, first_slot);
    const Req q = load_req(p.seqs, r);
    if (!q.ok && (threadIdx.x & 31) == 0) report(p.status, LMKV_ERR_BAD_LENGTH);
    t.part = p.prefix_splits + split;
    t.row0 = (slot - first_slot(r)) * rows_per_tile;
    t.nrows = q.n * group - t.row0;
    if (t.row0 < 0 || t.nrows <= 0) return false;
    t.table = p.seqs.table + (int64_t)r * p.seqs.table_stride;
    t.t0 = q.q0;
    t.limit0 = q.len - q.n + 1;
    t.causal = 1;
    const int32_t last = (int32_t)p.by_group.div((uint32_t)(t.row0 + min(t.nrows, rows_per_tile) - 1));
    t.k0 = split * p.own_span;
    t.k1 = max(t.k0, min(t.k0 + p.own_span, t.limit0 + last));
    return p.direct || t.k0 < q.len;
}

// Row tiles of 16 by mma.sync.  Bound by the bytes of K and V: with a few rows
// per KV head the products are a fraction of the loads' time, so the four
// warps of a CTA share the rows, take 16 keys (a page) each in turn, and run
// by themselves: every warp has its own ring of kStages x 16 K and V rows,
// filled by cp.async, and its own running maximum, sum and output; they are
// joined in shared memory at the end.
template <class T, int D>
__global__ void __launch_bounds__(kWarps * 32)
attend_rows_kernel(const __grid_constant__ AttendParams p) {
    constexpr int kRowBytes = D * 2;
    constexpr int kVecs = kRowBytes / 16;            // 16-byte pieces of a row
    constexpr int kTileBytes = kChunk * kRowBytes;   // K (or V) rows of a stage
    constexpr int kSteps = D / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float2 ml[kWarps][kRowTile];
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Tile t;
    if (!find_tile(p, blockIdx.x, kRowTile, t)) return;
    const uint8_t* base = p.layer.base();
    if (base == nullptr) {
        if (threadIdx.x == 0) report(p.status, LMKV_ERR_BAD_POINTER);
        t.k1 = t.k0;
    }
    const int32_t group = (int32_t)p.by_group.d;
    const int64_t half_bytes = p.layer.half_bytes();
    const int64_t head_bytes = (int64_t)t.h * kRowBytes;
    uint8_t* const ring = smem + warp * (kStages * 2 * kTileBytes);
    const uint32_t ring_u = smem_u32(ring);

    // this thread's two rows: lane / 4 and lane / 4 + 8
    int32_t limit[2];
    uint32_t qf[kSteps][4];
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
    }

    const int32_t chunks = (t.k1 - t.k0 + kChunk - 1) / kChunk;
    const int32_t mine = chunks > warp ? (chunks - warp + kWarps - 1) / kWarps : 0;
    uint32_t there[kStages];       // key masks of the stages (constant indices after unrolling)

    auto fill = [&](int32_t i) -> uint32_t {           // my i-th chunk into its stage
        const int32_t tok = t.k0 + (i * kWarps + warp) * kChunk + (lane & 15);
        int64_t off = -1;
        if (tok < t.k1) {
            off = p.layer.token_offset(t.table, tok);
            if (off < 0 && lane < 16) report(p.status, LMKV_ERR_BAD_BLOCK);
        }
        const uint32_t mask = __ballot_sync(0xFFFFFFFFu, off >= 0) & 0xFFFFu;
        const uint32_t dst = ring_u + (i % kStages) * (2 * kTileBytes);
#pragma unroll
        for (int v = 0; v < kChunk * kVecs / 32; ++v) {
            const int row = (v * 32 + lane) / kVecs, c = (v * 32 + lane) % kVecs;
            const int64_t o = __shfl_sync(0xFFFFFFFFu, off, row);
            const uint8_t* src = o >= 0 ? base + o + head_bytes + c * 16 : base;
            const uint32_t at = dst + swizzled<kRowBytes>(row, c);
            cp_async16(at, src, o >= 0);
            cp_async16(at + kTileBytes, src + (o >= 0 ? half_bytes : 0), o >= 0);
        }
        return mask;
    };

    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

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
            {
                constexpr int kAhead = kStages - 1;
                there[(u + kAhead) % kStages] = i + kAhead < mine ? fill(i + kAhead) : 0u;
                cp_commit();
            }
            cp_wait<kStages - 1>();
            __syncwarp();
            const uint32_t kt = ring_u + u * (2 * kTileBytes), vt = kt + kTileBytes;
            const uint32_t mask = there[u];
            float sc[2][4] = {};
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                uint32_t b[4];
                // matrices: keys 0-7 x d 0-7, keys 0-7 x d 8-15, keys 8-15 x d 0-7, keys 8-15 x d 8-15
                ldmatrix4(b, kt + swizzled<kRowBytes>((lane & 7) + ((lane >> 4) << 3), 2 * s + ((lane >> 3) & 1)));
                mma16816<T>(sc[0], qf[s], b[0], b[1]);
                mma16816<T>(sc[1], qf[s], b[2], b[3]);
            }
            const int32_t key0 = t.k0 + (i * kWarps + warp) * kChunk + (lane & 3) * 2;
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
                        x = seen ? x * p.scale_log2 : -INFINITY;
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
            // most half a step of T each, of either sign, against the sums in fp32).
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
    }
    cp_wait<0>();
    __syncthreads();

    // join the warps: sums over the quad first, then over warps in shared memory
    float* const wo = reinterpret_cast<float*>(smem) + warp * kRowTile * D;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 1);
        l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 2);
        const int rr = (lane >> 2) + 8 * r;
        if ((lane & 3) == 0) ml[warp][rr] = make_float2(m[r], l[r]);
#pragma unroll
        for (int d = 0; d < D / 8; ++d)
            *reinterpret_cast<float2*>(wo + rr * D + d * 8 + (lane & 3) * 2) =
                make_float2(o[d][2 * r], o[d][2 * r + 1]);
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
            const float4 x = *reinterpret_cast<const float4*>(all + (w * kRowTile + rr) * D + c);
            sum += f * ml[w][rr].y;
            acc.x += f * x.x;
            acc.y += f * x.y;
            acc.z += f * x.z;
            acc.w += f * x.w;
        }
        const int32_t n = (int32_t)p.by_group.div((uint32_t)(t.row0 + rr));
        const int32_t tok = t.t0 + n, head = t.h * group + (t.row0 + rr - n * group);
        const int32_t row = tok * p.q_heads + head;
        if (p.direct) {
            const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
            T* dst = p.out.row<T>(tok, head) + c;
            dst[0] = Elem<T>::from_float(acc.x * inv);
            dst[1] = Elem<T>::from_float(acc.y * inv);
            dst[2] = Elem<T>::from_float(acc.z * inv);
            dst[3] = Elem<T>::from_float(acc.w * inv);
            if (c == 0 && p.lse != nullptr) p.lse[row] = (mu + log2f(sum)) * kLn2;
        } else {
            const int64_t at = (int64_t)t.part * p.rows + row;
            *reinterpret_cast<float4*>(p.part_o + at * D + c) = acc;
            if (c == 0) p.part_ml[at] = make_float2(top, sum);
        }
    }
}

// Joins the parts of every row: a warp per (token, query head).
template <class T, int D>
__global__ void __launch_bounds__(256) attend_join_kernel(const __grid_constant__ AttendParams p) {
    constexpr int kPer = D / 32;
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int32_t row = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= p.rows) return;
    const int32_t tok = row / p.q_heads, head = row - tok * p.q_heads;
    const int32_t r = find_request(p.seqs.num_req, tok, [&](int32_t i) { return p.seqs.q_start[i]; });
    const Req q = load_req(p.seqs, r);
    if (!q.ok && lane == 0) report(p.status, LMKV_ERR_BAD_LENGTH);
    if (tok < q.q0 || tok >= q.q0 + q.n) return;       // a padded row
    const int32_t parts = p.prefix_splits + (q.len + p.own_span - 1) / p.own_span;
    float top = -INFINITY, sum = 0.f, acc[kPer] = {};
    for (int32_t s = 0; s < parts; ++s) {
        const int64_t at = (int64_t)s * p.rows + row;
        const float2 v = p.part_ml[at];
        float x[kPer];
        const float* src = p.part_o + at * D + lane * kPer;
        if constexpr (kPer == 4) *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(src);
        else *reinterpret_cast<float2*>(x) = *reinterpret_cast<const float2*>(src);
        const float mn = fmaxf(top, v.x);
        const float mu = mn == -INFINITY ? 0.f : mn;
        const float fa = exp2_fast(top - mu), fb = exp2_fast(v.x - mu);
        top = mn;
        sum = sum * fa + v.y * fb;
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] = acc[i] * fa + x[i] * fb;
    }
    const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
    T* dst = p.out.row<T>(tok, head) + lane * kPer;
#pragma unroll
    for (int i = 0; i < kPer; ++i) dst[i] = Elem<T>::from_float(acc[i] * inv);
    if (lane == 0 && p.lse != nullptr)
        p.lse[row] = ((top == -INFINITY ? 0.f : top) + log2f(sum)) * kLn2;
}

// ---- host ---------------------------------------------------------------

struct Plan {
    int32_t prefix_tiles, prefix_splits, prefix_span;
    int32_t own_slots, own_splits, own_span;
    bool direct;
    int64_t rows;
    uint64_t o_bytes, bytes;
};

constexpr int32_t kSms = 152;

// Splits: enough CTAs for two on every SM, none below 128 keys.
void split(int64_t ctas, int32_t keys, int32_t* splits, int32_t* span) {
    const int64_t want = (4 * kSms + ctas - 1) / ctas;
    const int64_t most = (keys + 127) / 128;
    const int64_t n = want < most ? want : most;
    int64_t s = (keys + n - 1) / n;
    s = (s + 63) / 64 * 64;
    *span = (int32_t)s;
    *splits = (int32_t)((keys + s - 1) / s);
}

Plan make_plan(const lmkv_pool_t* pool, int32_t q_heads, int32_t num_tokens, int32_t num_req, int32_t prefix_len,
               int32_t max_kv_len) {
    Plan x = {};
    const int64_t group = q_heads / pool->num_kv_heads;
    x.rows = (int64_t)num_tokens * q_heads;
    if (prefix_len > 0) {
        x.prefix_tiles = (int32_t)((num_tokens * group + kRowTile - 1) / kRowTile);
        split((int64_t)x.prefix_tiles * pool->num_kv_heads, prefix_len, &x.prefix_splits, &x.prefix_span);
    }
    x.own_span = 1;
    if (max_kv_len > 0 || prefix_len == 0) {
        x.own_slots = (int32_t)(num_tokens * group / kRowTile) + num_req;
        split((int64_t)x.own_slots * pool->num_kv_heads, max_kv_len > 0 ? max_kv_len : 1, &x.own_splits, &x.own_span);
    }
    x.direct = x.prefix_splits + x.own_splits == 1 && x.own_splits == 1;
    const uint64_t parts = x.direct ? 0 : (uint64_t)(x.prefix_splits + x.own_splits);
    x.o_bytes = parts * x.rows * pool->head_dim * 4;
    x.bytes = x.o_bytes + parts * x.rows * 8;
    return x;
}

int check_shape(const lmkv_pool_t* pool) {
    const int rc = lmkv_internal_check_pool(pool);
    if (rc != LMKV_OK) return rc;
    if (pool->elem_bytes != 2 || (pool->head_dim != 64 && pool->head_dim != 128)) return LMKV_ERR_UNSUPPORTED;
    return LMKV_OK;
}

template <class T, int D>
int attend_typed(AttendParams& p, const Plan& x, void* stream) {
    constexpr int smem = kWarps * kStages * 2 * kChunk * D * 2;
    int rc = allow_smem<attend_rows_kernel<T, D>, smem>();
    if (rc != LMKV_OK) return rc;
    const int64_t grid = ((int64_t)x.prefix_tiles * x.prefix_splits + (int64_t)x.own_slots * x.own_splits) * p.kv_heads;
    rc = launch(attend_rows_kernel<T, D>, grid, kWarps * 32, smem, stream, 1, p);
    if (rc != LMKV_OK || x.direct) return rc;
    return launch(attend_join_kernel<T, D>, (x.rows + 7) / 8, 256, 0, stream, 1, p);
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
                 ? 0 : make_plan(pool, num_q_heads, num_tokens, num_req, (int32_t)prefix_len, max_kv_len).bytes;
    return LMKV_OK;
}

int lmkv_attend_layer(const lmkv_pool_t* pool, int32_t dtype, int32_t layer, const lmkv_batch_t* batch,
                      int32_t num_q_heads, const lmkv_rows_t* q, const int32_t* prefix_table, int64_t prefix_len,
                      float scale, const lmkv_rows_t* out, float* lse, void* workspace, uint64_t workspace_bytes,
                      int32_t* d_status, void* stream) {
    int rc = check_shape(pool);
    if (rc != LMKV_OK) return rc;
    if (!type_fits(pool, dtype)) return LMKV_ERR_UNSUPPORTED;
    if (layer < 0 || layer >= pool->num_layers || !std::isfinite(scale)) return LMKV_ERR_INVALID_ARG;
    rc = check_batch(pool, batch, num_q_heads);
    if (rc != LMKV_OK) return rc;
    if (prefix_len < 0 || prefix_len > INT32_MAX - 65536 || batch->max_kv_len > INT32_MAX - 65536 ||
        (prefix_len > 0 && prefix_table == nullptr))
        return LMKV_ERR_INVALID_ARG;
    if (batch->num_req == 0 || batch->num_tokens == 0) return LMKV_OK;
    if (!rows_ok(q, 2) || !rows_ok(out, 2)) return LMKV_ERR_INVALID_ARG;
    const Plan x = make_plan(pool, num_q_heads, batch->num_tokens, batch->num_req, (int32_t)prefix_len,
                             batch->max_kv_len);
    if (x.bytes > 0 && (workspace == nullptr || workspace_bytes < x.bytes)) return LMKV_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(workspace) & 15) return LMKV_ERR_MISALIGNED;
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
    p.scale_log2 = scale * 1.44269504088896340736f;
    p.prefix_len = (int32_t)prefix_len;
    p.q_heads = num_q_heads;
    p.kv_heads = pool->num_kv_heads;
    p.rows = (int32_t)x.rows;
    p.prefix_tiles = x.prefix_tiles;
    p.prefix_splits = x.prefix_splits;
    p.prefix_span = x.prefix_span;
    p.own_slots = x.own_slots;
    p.own_splits = x.own_splits;
    p.own_span = x.own_span;
    p.direct = x.direct;
    p.q_pairs = reinterpret_cast<uintptr_t>(q->data) % 4 == 0 && q->token_stride % 2 == 0 && q->head_stride % 2 == 0;
    p.by_group = FastDiv((uint32_t)(num_q_heads / pool->num_kv_heads));
    if (dtype == LMKV_BF16)
        return pool->head_dim == 64 ? attend_typed<__nv_bfloat16, 64>(p, x, stream)
                                    : attend_typed<__nv_bfloat16, 128>(p, x, stream);
    return pool->head_dim == 64 ? attend_typed<__half, 64>(p, x, stream) : attend_typed<__half, 128>(p, x, stream);
}

}  // extern "C"
