// lmkv_evict.cu -- accumulated attention weight per cached token, and eviction
// of the tokens that received least of it ("H2O: Heavy-Hitter Oracle for
// Efficient Generative Inference of Large Language Models", Zhang et al.,
// 2023).
#include "lmkv_mma.cuh"

#include <cmath>

namespace {

using namespace lmkv_paged;
using namespace lmkv_mma;

constexpr float kLog2e = 1.44269504088896340736f;

// ---- weights ------------------------------------------------------------

struct WeighParams {
    Layer layer;
    Seqs seqs;
    const uint8_t* q;
    int64_t q_token_stride, q_head_stride;
    const float* lse;
    const float* scores;
    float* scores_out;
    int64_t score_stride;
    int32_t* status;
    float scale_log2, decay;
    int32_t q_heads, kv_heads;
    int32_t splits, span;          // key splits of a request, keys in each (a multiple of 64)
    int32_t row_cap;               // rows of a shared-memory row tile (a multiple of 8)
    bool q_vec;                    // q rows start on 16 bytes
    FastDiv by_group;
};

constexpr int kWarps = 4;
constexpr int kChunk = 16;         // keys a warp takes at a time
constexpr int kStages = 4;
constexpr int kMaxRowCap = 128;    // rows of a row tile at most
constexpr int kSpan = 256;         // keys of a CTA

// scores_out = decay * scores + column sums of e^(scale q.k - lse).
// The products are taken transposed, keys x rows: a warp holds 16 keys as the
// first operand and runs over the rows (new tokens x heads of the group),
// eight at a time, so a key's sum stays in one quad's registers and its order
// is fixed.  K is read once from HBM; a request with more rows than row_cap
// goes over its CTA's keys again from L2.  With few rows bound by the bytes of K.
template <class T, int D>
__global__ void __launch_bounds__(kWarps * 32)
weigh_kernel(const __grid_constant__ WeighParams p) {
    constexpr int kRowBytes = D * 2;
    constexpr int kVecs = kRowBytes / 16;
    constexpr int kTileBytes = kChunk * kRowBytes;
    constexpr int kSteps = D / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // heads change fastest: the heads' CTAs of the same tokens read the same pages' rows
    const int32_t h = blockIdx.x % p.kv_heads;
    const int32_t x = blockIdx.x / p.kv_heads;
    const int32_t r = x % p.seqs.num_req;
    const int32_t k0 = x / p.seqs.num_req * p.span;
    const Req q = load_req(p.seqs, r);
    if (!q.ok && threadIdx.x == 0) report(p.status, LMKV_ERR_BAD_LENGTH);
    const int32_t k1 = min(k0 + p.span, q.len);
    if (k0 >= k1) return;
    const uint8_t* base = p.layer.base();
    if (base == nullptr && threadIdx.x == 0) report(p.status, LMKV_ERR_BAD_POINTER);
    const int32_t* table = p.seqs.table + (int64_t)r * p.seqs.table_stride;
    const int32_t group = (int32_t)p.by_group.d;
    const int32_t rows = base == nullptr ? 0 : q.n * group;

    uint8_t* const ring = smem + warp * (kStages * kTileBytes);
    const uint32_t ring_u = smem_u32(ring);
    uint8_t* const qt = smem + kWarps * kStages * kTileBytes;                  // [row_cap][D] swizzled
    const uint32_t qt_u = smem_u32(qt);
    float* const row_lse = reinterpret_cast<float*>(qt + p.row_cap * kRowBytes);    // times log2 e
    int32_t* const row_limit = reinterpret_cast<int32_t*>(row_lse + p.row_cap);
    float* const acc = reinterpret_cast<float*>(row_limit + p.row_cap);             // [span]

    for (int i = threadIdx.x; i < p.span; i += kWarps * 32) acc[i] = 0.f;
    const int32_t chunks = (k1 - k0 + kChunk - 1) / kChunk;
    const int32_t mine = chunks > warp ? (chunks - warp + kWarps - 1) / kWarps : 0;

    auto fill = [&](int32_t i) {
        const int32_t tok = k0 + (i * kWarps + warp) * kChunk + (lane & 15);
        int64_t off = -1;
        if (tok < k1) {
            off = p.layer.token_offset(table, tok);
            if (off < 0 && lane < 16) report(p.status, LMKV_ERR_BAD_BLOCK);
        }
        const uint32_t mask = __ballot_sync(0xFFFFFFFFu, off >= 0) & 0xFFFFu;
        const uint32_t dst = ring_u + (i % kStages) * kTileBytes;
#pragma unroll
        for (int v = 0; v < kChunk * kVecs / 32; ++v) {
            const int row = (v * 32 + lane) / kVecs, c = (v * 32 + lane) % kVecs;
            const int64_t o = __shfl_sync(0xFFFFFFFFu, off, row);
            cp_async16(dst + swizzled<kRowBytes>(row, c),
                       o >= 0 ? base + o + (int64_t)h * kRowBytes + c * 16 : base, o >= 0);
        }
        return mask;
    };

    for (int32_t row0 = 0; row0 < rows; row0 += p.row_cap) {
        const int32_t nrows = min(p.row_cap, rows - row0);
        const int32_t padded = (nrows + 7) & ~7;
        __syncthreads();
        for (int i = threadIdx.x; i < padded * kVecs; i += kWarps * 32) {
            const int rr = i / kVecs, c = i % kVecs;
            int4 v = make_int4(0, 0, 0, 0);
            if (rr < nrows) {
                const int32_t n = (int32_t)p.by_group.div((uint32_t)(row0 + rr));
                const int32_t head = h * group + (row0 + rr - n * group);
                const T* src = reinterpret_cast<const T*>(p.q) + (int64_t)(q.q0 + n) * p.q_token_stride +
                               (int64_t)head * p.q_head_stride + c * 8;
                if (p.q_vec) {
                    v = *reinterpret_cast<const int4*>(src);
                } else {
                    v.x = (int)load_pair(src, false);
                    v.y = (int)load_pair(src + 2, false);
                    v.z = (int)load_pair(src + 4, false);
                    v.w = (int)load_pair(src + 6, false);
                }
                if (c == 0) {
                    const float e = p.lse[(int64_t)(q.q0 + n) * p.q_heads + head];
                    row_lse[rr] = e * kLog2e;
                    row_limit[rr] = e == -INFINITY ? 0 : q.len - q.n + n + 1;
                }
            } else if (c == 0) {
                row_lse[rr] = 0.f;
                row_limit[rr] = 0;
            }
            *reinterpret_cast<int4*>(qt + swizzled<kRowBytes>(rr, c)) = v;
        }
        __syncthreads();
        uint32_t there[kStages];
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
                __syncwarp();
                constexpr int kAhead = kStages - 1;
                there[(u + kAhead) % kStages] = i + kAhead < mine ? fill(i + kAhead) : 0u;
                cp_commit();
                cp_wait<kStages - 1>();
                __syncwarp();
                const uint32_t kt = ring_u + u * kTileBytes;
                uint32_t kf[kSteps][4];
#pragma unroll
                for (int s = 0; s < kSteps; ++s)       // keys 0-7 / 8-15 x d 0-7, then x d 8-15
                    ldmatrix4(kf[s], kt + swizzled<kRowBytes>(lane & 15, 2 * s + (lane >> 4)));
                const int32_t local = (i * kWarps + warp) * kChunk + (lane >> 2);
                const bool ok0 = (there[u] >> (lane >> 2)) & 1, ok1 = (there[u] >> ((lane >> 2) + 8)) & 1;
                float s0 = 0.f, s1 = 0.f;
                for (int32_t g = 0; g < padded; g += 8) {
                    float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int s = 0; s < kSteps; s += 2) {
                        uint32_t b[4];                 // rows x d of two steps
                        ldmatrix4(b, qt_u + swizzled<kRowBytes>(g + (lane & 7), 2 * s + (lane >> 3)));
                        mma16816<T>(c, kf[s], b[0], b[1]);
                        mma16816<T>(c, kf[s + 1], b[2], b[3]);
                    }
                    const int rr = g + (lane & 3) * 2;
                    const float2 e = *reinterpret_cast<const float2*>(row_lse + rr);
                    const int2 lim = *reinterpret_cast<const int2*>(row_limit + rr);
                    const int32_t key = k0 + local;
                    if (key < lim.x) s0 += exp2_fast(fmaf(c[0], p.scale_log2, -e.x));
                    if (key < lim.y) s0 += exp2_fast(fmaf(c[1], p.scale_log2, -e.y));
                    if (key + 8 < lim.x) s1 += exp2_fast(fmaf(c[2], p.scale_log2, -e.x));
                    if (key + 8 < lim.y) s1 += exp2_fast(fmaf(c[3], p.scale_log2, -e.y));
                }
                s0 += __shfl_xor_sync(0xFFFFFFFFu, s0, 1);
                s1 += __shfl_xor_sync(0xFFFFFFFFu, s1, 1);
                s0 += __shfl_xor_sync(0xFFFFFFFFu, s0, 2);
                s1 += __shfl_xor_sync(0xFFFFFFFFu, s1, 2);
                if ((lane & 3) == 0) {
                    if (ok0) acc[local] += s0;
                    if (ok1) acc[local + 8] += s1;
                }
            }
        }
        cp_wait<0>();
    }
    __syncthreads();
    const int64_t at = ((int64_t)r * p.kv_heads + h) * p.score_stride + k0;
    for (int i = threadIdx.x; i < k1 - k0; i += kWarps * 32)
        p.scores_out[at + i] = p.decay == 0.f ? acc[i] : fmaf(p.decay, p.scores[at + i], acc[i]);
}

// ---- selection ----------------------------------------------------------

struct EvictParams {
    Layer layer;
    const int32_t* table;
    const int32_t* kv_len;
    const float* scores;
    int32_t* keep;
    int32_t* new_len;
    float* kept_scores;
    int32_t* status;
    int64_t score_stride, kept_stride;
    int32_t table_stride, num_req, max_kv_len, kv_heads;
    int32_t budget, sinks, recent;
    int32_t head_bytes;
};

__device__ __forceinline__ int32_t clamped_len(const EvictParams& p, int32_t r) {
    return min(max(p.kv_len[r], 0), p.max_kv_len);
}

// Order of the scores as unsigned numbers: NaN lowest, then -inf up to +inf,
// -0 equal to +0.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0u;
    const uint32_t b = __float_as_uint(x + 0.f);      // -0 + 0 = +0
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

constexpr int kSelectThreads = 1024;
constexpr int kBins = 2048;
constexpr int kSelectTokens = 50 * 1024;      // keys that fit in shared memory

// Exclusive sums over the CTA of two counts a thread, in thread order.
__device__ __forceinline__ int2 scan_pairs(int2 mine, int2* warp_sums) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int2 v = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, v.x, d), y = __shfl_up_sync(0xFFFFFFFFu, v.y, d);
        if (lane >= d) {
            v.x += x;
            v.y += y;
        }
    }
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    int2 t = warp_sums[lane];
    const int2 t0 = t;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, t.x, d), y = __shfl_up_sync(0xFFFFFFFFu, t.y, d);
        if (lane >= d) {
            t.x += x;
            t.y += y;
        }
    }
    const int bx = __shfl_sync(0xFFFFFFFFu, t.x - t0.x, warp), by = __shfl_sync(0xFFFFFFFFu, t.y - t0.y, warp);
    return make_int2(bx + v.x - mine.x, by + v.y - mine.y);
}

// A CTA per (request, head).  The need-th largest key of the candidates
// (tokens that are neither sinks nor recent) is found digit by digit (11, 11
// and 10 bits), most significant first, with a histogram over the candidates
// that share the digits found so far; then every thread counts what it keeps
// of a run of consecutive tokens, one scan places the runs, and the kept
// tokens are written in order, the first ties among them.  The keys are read
// once, into shared memory (kStaged; more than kSelectTokens are read again
// from L2 instead).  Wide digits are for the counters: scores crowd into few
// exponents, and threads that meet on a counter take turns.
template <bool kStaged>
__global__ void __launch_bounds__(kSelectThreads)
select_kernel(const __grid_constant__ EvictParams p) {
    __shared__ uint32_t hist[kBins];
    __shared__ uint32_t digit_s, above_s;
    __shared__ int2 warp_sums[32];
    extern __shared__ uint32_t keys[];
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x;
    const int32_t h = blockIdx.x % p.kv_heads, r = blockIdx.x / p.kv_heads;
    const int32_t len = clamped_len(p, r);
    if (tid == 0 && h == 0) {
        if (len != p.kv_len[r]) report(p.status, LMKV_ERR_BAD_LENGTH);
        p.new_len[r] = min(len, p.budget);
    }
    const float* const w = p.scores + ((int64_t)r * p.kv_heads + h) * p.score_stride;
    int32_t* const keep = p.keep + ((int64_t)r * p.kv_heads + h) * p.budget;
    float* const kept = p.kept_scores == nullptr
                            ? nullptr : p.kept_scores + ((int64_t)r * p.kv_heads + h) * p.kept_stride;
    if (len <= p.budget) {
        for (int32_t i = tid; i < p.budget; i += kSelectThreads) {
            keep[i] = i < len ? i : -1;
            if (kept != nullptr) kept[i] = i < len ? w[i] : 0.f;
        }
        return;
    }
    const int32_t lo = p.sinks, hi = len - p.recent;
    const int32_t need = p.budget - p.sinks - p.recent;       // < hi - lo
    uint32_t prefix = 0, want = (uint32_t)need;               // want: still to take among the prefix's
    if (kStaged)
        for (int32_t i = tid; i < len; i += kSelectThreads) keys[i] = order_key(w[i]);
    auto key_of = [&](int32_t i) { return kStaged ? keys[i] : order_key(w[i]); };
    int top = 32;                                             // bits above are found
    while (top > 0 && need > 0) {
        const int low = top > 11 ? top - 11 : 0;
        const uint32_t digits = (1u << (top - low)) - 1u;
        for (int i = tid; i < kBins; i += kSelectThreads) hist[i] = 0;
        __syncthreads();
        for (int32_t i = lo + tid; i < hi; i += kSelectThreads) {
            const uint32_t k = key_of(i);
            if (top == 32 || (k >> top) == (prefix >> top)) atomicAdd(&hist[(k >> low) & digits], 1u);
        }
        __syncthreads();
        // thread t holds the t-th pair of counters from the top
        const int hi_bin = kBins - 1 - 2 * tid;
        const int c0 = (int)hist[hi_bin], c1 = (int)hist[hi_bin - 1];
        const int2 before = scan_pairs(make_int2(c0 + c1, 0), warp_sums);
        const uint32_t b0 = (uint32_t)before.x, b1 = b0 + c0;
        if (b0 < want && want <= b0 + c0) {
            digit_s = hi_bin;
            above_s = b0;
        }
        if (b1 < want && want <= b1 + c1) {
            digit_s = hi_bin - 1;
            above_s = b1;
        }
        __syncthreads();
        prefix |= digit_s << low;
        want -= above_s;
        top = low;
        __syncthreads();
    }
    // `want` of the keys equal to prefix are kept, all larger ones.  A run is an odd
    // number of tokens, so that the threads' places lie in different banks.
    const int32_t run = ((len + kSelectThreads - 1) / kSelectThreads) | 1;
    const int32_t from = min(tid * run, len), to = min(from + run, len);
    int2 count = make_int2(0, 0);                             // kept for certain, ties
    __syncthreads();
    for (int32_t i = from; i < to; ++i) {
        if (i < lo || i >= hi) {
            ++count.x;
        } else if (need > 0) {
            const uint32_t k = key_of(i);
            count.x += k > prefix;
            count.y += k == prefix;
        }
    }
    int2 at = scan_pairs(count, warp_sums);
    for (int32_t i = from; i < to; ++i) {
        bool keeps = i < lo || i >= hi, tie = false;
        if (!keeps && need > 0) {
            const uint32_t k = key_of(i);
            keeps = k > prefix;
            tie = k == prefix;
        }
        if (keeps || (tie && at.y < (int32_t)want)) {
            const int32_t slot = at.x + min(at.y, (int32_t)want);
            if (slot < p.budget) {
                keep[slot] = i;
                if (kept != nullptr) kept[slot] = w[i];
            }
        }
        at.x += keeps;
        at.y += tie;
    }
}

// ---- compaction ---------------------------------------------------------

constexpr int kMoveThreads = 256;
constexpr int kMoveDepth = 8;              // batches of rows on their way

// Moves the kept rows of one (request, head, K or V, column piece) to the
// front of the request's pages, in place.  keep is ascending, so keep[i] >= i
// and a batch of slots in order may be written once its own rows, and those of
// the batches before it, have been read: what later batches read lies behind.
// So rows may be fetched as early as one likes: kMoveDepth batches are under
// way in shared memory (cp.async), each thread storing what it fetched itself,
// with one barrier a batch, and the tokens and pages of the next ones are
// looked up before they are needed.  Slots whose token stays (a leading run,
// as keep[i] - i never falls) are skipped.  Bound by reading and writing the
// moved rows.
template <int kBytes>
__global__ void __launch_bounds__(kMoveThreads)
compact_kernel(const __grid_constant__ EvictParams p, int32_t pieces, int32_t piece_vecs) {
    __shared__ __align__(16) uint8_t ring[kMoveDepth][kMoveThreads * kBytes];
    pdl_launch_dependents();
    pdl_wait();
    int32_t x = blockIdx.x;
    const int32_t piece = x % pieces;
    x /= pieces;
    const int32_t h = x % p.kv_heads;
    x /= p.kv_heads;
    const int32_t kv = x & 1, r = x >> 1;
    const int32_t len = clamped_len(p, r);
    if (len <= p.budget) return;
    uint8_t* base = p.layer.base();
    if (base == nullptr) {
        if (threadIdx.x == 0) report(p.status, LMKV_ERR_BAD_POINTER);
        return;
    }
    const int32_t vecs = min(piece_vecs, p.head_bytes / kBytes - piece * piece_vecs);
    const int32_t* table = p.table + (int64_t)r * p.table_stride;
    const int32_t* keep = p.keep + ((int64_t)r * p.kv_heads + h) * p.budget;
    int32_t first = 0, end = p.budget;                 // first slot that moves
    while (first < end) {
        const int32_t mid = (first + end) >> 1;
        if (keep[mid] == mid) first = mid + 1;
        else end = mid;
    }
    // thread -> (slot of the batch, vector of the piece)
    const int32_t per_batch = kMoveThreads / vecs;
    const int32_t mine = threadIdx.x / vecs, vec = threadIdx.x - mine * vecs;
    const bool idle = mine >= per_batch;
    base += kv * p.layer.half_bytes() + (int64_t)h * p.head_bytes + ((int64_t)piece * piece_vecs + vec) * kBytes;
    const int32_t batches = (p.budget - first + per_batch - 1) / per_batch;
    auto slot_of = [&](int32_t i) {                    // my slot in batch i, or -1
        const int32_t s = first + i * per_batch + mine;
        return idle || s >= p.budget ? -1 : s;
    };
    uint32_t came = 0;                                 // bit i % 32: batch i's row is on its way
    auto fetch = [&](int32_t i, int32_t tok) {
        came &= ~(1u << (i & 31));
        if (tok >= 0) {
            const int64_t from = p.layer.token_offset(table, tok);
            if (from < 0) report(p.status, LMKV_ERR_BAD_BLOCK);
            else came |= 1u << (i & 31);
            uint8_t* const to = &ring[i % kMoveDepth][threadIdx.x * kBytes];
            if (from >= 0) {
                if constexpr (kBytes == 16) cp_async16(smem_u32(to), base + from);
                else if constexpr (kBytes == 4)
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(to)), "l"(base + from) : "memory");
                else *to = base[from];
            }
        }
        cp_commit();
    };
    auto token_of = [&](int32_t i) {                   // the token that batch i's slot receives
        const int32_t s = i < batches ? slot_of(i) : -1;
        return s >= 0 ? keep[s] : -1;
    };
    int32_t ahead[2] = {token_of(0), token_of(1)};     // tokens of the next batches to fetch
#pragma unroll 1
    for (int32_t i = 0; i < kMoveDepth - 1; ++i) {
        const int32_t tok = ahead[0];
        ahead[0] = ahead[1];
        ahead[1] = token_of(i + 2);
        fetch(i, tok);
    }
#pragma unroll 1
    for (int32_t i = 0; i < batches; ++i) {
        int64_t to = -1;
        if ((came >> (i & 31)) & 1) {
            to = p.layer.token_offset(table, slot_of(i));
            if (to < 0) report(p.status, LMKV_ERR_BAD_BLOCK);
        }
        cp_wait<kMoveDepth - 2>();
        __syncthreads();               // batch i and those before it have been read by every thread
        if (to >= 0) {
            const uint8_t* const src = &ring[i % kMoveDepth][threadIdx.x * kBytes];
            if constexpr (kBytes == 16) *reinterpret_cast<int4*>(base + to) = *reinterpret_cast<const int4*>(src);
            else if constexpr (kBytes == 4) *reinterpret_cast<int32_t*>(base + to) = *reinterpret_cast<const int32_t*>(src);
            else base[to] = *src;
        }
        const int32_t tok = ahead[0];
        ahead[0] = ahead[1];
        ahead[1] = token_of(i + kMoveDepth + 1);
        fetch(i + kMoveDepth - 1, tok);
    }
    cp_wait<0>();
}

template <int kBytes>
int launch_compact(const EvictParams& p, void* stream) {
    const int32_t vecs = p.head_bytes / kBytes;
    const int32_t most = 64 / kBytes;                  // 64-byte pieces: more CTAs, whole sectors
    const int32_t piece = vecs < most ? vecs : most;
    const int32_t pieces = (vecs + piece - 1) / piece;
    return launch(compact_kernel<kBytes>, (int64_t)p.num_req * p.kv_heads * 2 * pieces, kMoveThreads, 0, stream, 1, p,
                  pieces, piece);
}

template <class T, int D>
int weigh_typed(const WeighParams& p, void* stream) {
    const size_t smem = (size_t)kWarps * kStages * kChunk * D * 2 + (size_t)p.row_cap * (D * 2 + 8) + (size_t)p.span * 4;
    constexpr int most = kWarps * kStages * kChunk * D * 2 + kMaxRowCap * (D * 2 + 8) + kSpan * 4;
    const int rc = allow_smem<weigh_kernel<T, D>, most>();
    if (rc != LMKV_OK) return rc;
    return launch(weigh_kernel<T, D>, (int64_t)p.seqs.num_req * p.kv_heads * p.splits, kWarps * 32, smem, stream, 1, p);
}

}  // namespace

extern "C" {

int lmkv_weigh_layer(const lmkv_pool_t* pool, int32_t dtype, int32_t layer, const lmkv_batch_t* batch,
                     int32_t num_q_heads, const lmkv_rows_t* q, const float* lse, float scale, float decay,
                     const float* scores, float* scores_out, int64_t score_stride, int32_t* d_status, void* stream) {
    int rc = lmkv_internal_check_pool(pool);
    if (rc != LMKV_OK) return rc;
    if (pool->elem_bytes != 2 || (pool->head_dim != 64 && pool->head_dim != 128) || !type_fits(pool, dtype))
        return LMKV_ERR_UNSUPPORTED;
    if (layer < 0 || layer >= pool->num_layers || !std::isfinite(scale) || !std::isfinite(decay))
        return LMKV_ERR_INVALID_ARG;
    rc = check_batch(pool, batch, num_q_heads);
    if (rc != LMKV_OK) return rc;
    if (batch->max_kv_len > INT32_MAX - 65536 || score_stride < batch->max_kv_len) return LMKV_ERR_INVALID_ARG;
    if (batch->num_req == 0 || batch->max_kv_len == 0) return LMKV_OK;
    if (batch->q_start == nullptr || batch->kv_len == nullptr || batch->block_table == nullptr ||
        scores_out == nullptr || (decay != 0.f && scores == nullptr))
        return LMKV_ERR_INVALID_ARG;
    if (batch->num_tokens > 0 && (!rows_ok(q, 2) || lse == nullptr)) return LMKV_ERR_INVALID_ARG;
    WeighParams p = {};
    p.layer = Layer::of(pool, layer);
    p.seqs = Seqs::of(batch);
    if (batch->num_tokens > 0) {
        p.q = static_cast<const uint8_t*>(q->data);
        p.q_token_stride = q->token_stride;
        p.q_head_stride = q->head_stride;
        p.q_vec = reinterpret_cast<uintptr_t>(q->data) % 16 == 0 && q->token_stride % 8 == 0 && q->head_stride % 8 == 0;
    }
    p.lse = lse;
    p.scores = scores;
    p.scores_out = scores_out;
    p.score_stride = score_stride;
    p.status = d_status;
    p.scale_log2 = scale * kLog2e;
    p.decay = decay;
    p.q_heads = num_q_heads;
    p.kv_heads = pool->num_kv_heads;
    p.by_group = FastDiv((uint32_t)(num_q_heads / pool->num_kv_heads));
    const int64_t rows = (int64_t)batch->max_new * p.by_group.d;
    p.row_cap = rows < 8 ? 8 : rows > kMaxRowCap ? kMaxRowCap : (int32_t)((rows + 7) / 8 * 8);
    p.span = kSpan;
    p.splits = (batch->max_kv_len + p.span - 1) / p.span;
    if (dtype == LMKV_BF16)
        return pool->head_dim == 64 ? weigh_typed<__nv_bfloat16, 64>(p, stream) : weigh_typed<__nv_bfloat16, 128>(p, stream);
    return pool->head_dim == 64 ? weigh_typed<__half, 64>(p, stream) : weigh_typed<__half, 128>(p, stream);
}

int lmkv_evict_layer(const lmkv_pool_t* pool, int32_t layer, const int32_t* block_table, int32_t max_blocks,
                     const int32_t* kv_len, int32_t num_req, int32_t max_kv_len, const float* scores,
                     int64_t score_stride, int32_t budget, int32_t sinks, int32_t recent, int32_t* keep,
                     int32_t* new_len, float* kept_scores, int64_t kept_stride, int32_t* d_status, void* stream) {
    int rc = lmkv_internal_check_pool(pool);
    if (rc != LMKV_OK) return rc;
    if (layer < 0 || layer >= pool->num_layers || num_req < 0 || num_req > (1 << 24) || max_blocks < 0 ||
        max_kv_len < 0 || max_kv_len > INT32_MAX - 65536 || max_kv_len > (int64_t)max_blocks * pool->block_size)
        return LMKV_ERR_INVALID_ARG;
    if (budget < 1 || sinks < 0 || recent < 0 || (int64_t)sinks + recent > budget || score_stride < max_kv_len ||
        (kept_scores != nullptr && kept_stride < budget))
        return LMKV_ERR_INVALID_ARG;
    if (num_req == 0) return LMKV_OK;
    if (kv_len == nullptr || keep == nullptr || new_len == nullptr || new_len == kv_len || kept_scores == scores ||
        (max_kv_len > 0 && (block_table == nullptr || scores == nullptr)))
        return LMKV_ERR_INVALID_ARG;
    EvictParams p = {};
    p.layer = Layer::of(pool, layer);
    p.table = block_table;
    p.kv_len = kv_len;
    p.scores = scores;
    p.keep = keep;
    p.new_len = new_len;
    p.kept_scores = kept_scores;
    p.status = d_status;
    p.score_stride = score_stride;
    p.kept_stride = kept_stride;
    p.table_stride = max_blocks;
    p.num_req = num_req;
    p.max_kv_len = max_kv_len;
    p.kv_heads = pool->num_kv_heads;
    p.budget = budget;
    p.sinks = sinks;
    p.recent = recent;
    p.head_bytes = pool->head_dim * pool->elem_bytes;
    if (max_kv_len <= kSelectTokens) {
        rc = allow_smem<select_kernel<true>, kSelectTokens * 4>();
        if (rc == LMKV_OK)
            rc = launch(select_kernel<true>, (int64_t)num_req * p.kv_heads, kSelectThreads, (size_t)max_kv_len * 4, stream,
                        1, p);
    } else {
        rc = launch(select_kernel<false>, (int64_t)num_req * p.kv_heads, kSelectThreads, 0, stream, 1, p);
    }
    if (rc != LMKV_OK || max_kv_len <= budget) return rc;
    // a head's row starts on a multiple of its own bytes: the largest unit that divides them
    if (p.head_bytes % 16 == 0) return launch_compact<16>(p, stream);
    if (p.head_bytes % 4 == 0) return launch_compact<4>(p, stream);
    return launch_compact<1>(p, stream);
}

}  // extern "C"
