// lmkv_evict.cu -- accumulated attention weight per cached token, and eviction
// of the tokens that received least of it ("H2O: Heavy-Hitter Oracle for
// Efficient Generative Inference of Large Language Models", Zhang et al.,
// 2023).
#include "lmkv_blocks.cuh"

#include <cmath>

namespace {

using namespace lmkv_paged;
using namespace lmkv_mma;
using namespace lmkv_tc;

constexpr float kLog2e = 1.44269504088896340736f;

// ---- weights ------------------------------------------------------------
//
// scores_out = decay * scores + column sums of e^(scale q.k - lse).  Products
// are taken transposed, keys x rows, so that a key's sum stays in one thread
// (or quad), in an order that never changes.

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
    float lse_scale;               // 1 / scale (tile kernel)
    int32_t q_heads, kv_heads;
    int32_t splits;                // shares of the batch's tokens, a CTA each for every head
    bool q_vec;                    // q rows start on 16 bytes
    FastDiv by_group;

    // Row `row` of request q's rows, of KV head h.
    template <class T>
    __device__ __forceinline__ const T* q_row(int32_t tok, int32_t head) const {
        return reinterpret_cast<const T*>(q) + (int64_t)tok * q_token_stride + (int64_t)head * q_head_stride;
    }
};

// 16 bytes of a row of q.
template <class T>
__device__ __forceinline__ int4 load_q(const T* src, bool vec) {
    if (vec) return *reinterpret_cast<const int4*>(src);
    return make_int4((int)load_pair(src, false), (int)load_pair(src + 2, false), (int)load_pair(src + 4, false),
                     (int)load_pair(src + 6, false));
}

// A CTA's keys: its request, head and range.
struct WeighPart {
    Req q;
    int32_t h, k0, k1;
    const int32_t* table;
};

constexpr int kWarps = 4;
constexpr int kChunk = 16;         // keys a warp takes at a time
constexpr int kStages = 2;
constexpr int kRowTile = 64;       // rows whose q is in shared memory at a time
constexpr int kUnit = kWarps * kChunk;
constexpr int kRowCtas = 5;        // CTAs an SM

// Few rows (a decode step): mma.sync of 16 keys x 8 rows.  Bound by the bytes
// of K: every warp runs by itself, 16 keys (a page) at a time through its own
// ring, and keeps a chunk's keys as the first operand while it goes over the
// rows, eight at a time; kOne: no request has more than eight, whose q stays
// in registers.  One round of CTAs takes equal shares of the batch's tokens
// (find_share): with a CTA per 1024 tokens the last round's idle SMs cost up to a
// fifth (67 : 50 us).  24 requests of 1000 to 9000 tokens, 8 KV heads of 128: 49.6 us, 5.25
// TB/s, 0.78 of the copy rate; q in registers 62 : 65 us on 24 of 5000.  Heads change fastest: the heads' CTAs of the same tokens read the
// same pages' rows.
template <class T, int D, bool kOne>
__global__ void __launch_bounds__(kWarps * 32, kRowCtas)
weigh_rows_kernel(const __grid_constant__ WeighParams p) {
    constexpr int kRowBytes = D * 2;
    constexpr int kTileBytes = kChunk * kRowBytes;
    constexpr int kSteps = D / 16;
    constexpr int kRows = kOne ? 8 : kRowTile;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ __align__(128) uint8_t qt[kRows * kRowBytes];      // swizzled
    __shared__ float row_lse[kRows];         // times log2 e
    __shared__ int32_t row_limit[kRows];
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint8_t* const base = p.layer.base();
    if (base == nullptr && threadIdx.x == 0) report(p.status, LMKV_ERR_BAD_POINTER);
    const int32_t group = (int32_t)p.by_group.d;
    const uint32_t ring = smem_u32(smem) + warp * (kStages * kTileBytes), q_u = smem_u32(qt);
    WeighPart x;
    x.h = blockIdx.x % p.kv_heads;
    Share share = find_share(p.seqs.num_req, blockIdx.x / p.kv_heads, p.splits,
                             [&](int32_t i) { return units_of(p.seqs, i, kUnit, p.status); });
    for (; share.n > 0 && share.r < p.seqs.num_req; ++share.r, share.first = 0) {
        x.q = load_req(p.seqs, share.r);
        const int64_t here = min((int64_t)(x.q.len + kUnit - 1) / kUnit - share.first, share.n);
        if (here <= 0) continue;
        share.n -= here;
        x.k0 = (int32_t)share.first * kUnit;
        x.k1 = min(x.k0 + (int32_t)here * kUnit, x.q.len);
        x.table = p.seqs.table + (int64_t)share.r * p.seqs.table_stride;
        const int32_t rows = base == nullptr ? 0 : x.q.n * group;
        const int64_t at = ((int64_t)x.q.r * p.kv_heads + x.h) * p.score_stride;
        const int32_t chunks = (x.k1 - x.k0 + kChunk - 1) / kChunk;
        const int32_t mine = chunks > warp ? (chunks - warp + kWarps - 1) / kWarps : 0;
        auto key_of = [&](int32_t i) { return x.k0 + (i * kWarps + warp) * kChunk; };       // my i-th chunk
        ChunkCopy<D, false> copy(p.layer, x.table, base, x.h, x.k1);
        auto fill = [&](int32_t i) {
            return copy.copy(key_of(i), ring + (i % kStages) * kTileBytes, key_of(i + 1), p.status);
        };

        for (int32_t row0 = 0; row0 == 0 || row0 < rows; row0 += kRows) {
            const int32_t nrows = min(kRows, rows - row0);
            const int32_t padded = (nrows + 7) & ~7;
            uint32_t there[kStages];
            __syncthreads();
            copy.lookup(key_of(0));
    #pragma unroll
            for (int s = 0; s < kStages - 1; ++s) {
                there[s] = rows > 0 && s < mine ? fill(s) : 0u;
                cp_commit();
            }
            for (int i = threadIdx.x; i < padded * (D / 8); i += kWarps * 32) {
                const int rr = i / (D / 8), c = i % (D / 8);
                int4 v = make_int4(0, 0, 0, 0);
                float lse = INFINITY;
                int32_t limit = 0;
                if (rr < nrows) {
                    const int32_t n = (int32_t)p.by_group.div((uint32_t)(row0 + rr));
                    const int32_t head = x.h * group + (row0 + rr - n * group);
                    v = load_q(p.q_row<T>(x.q.q0 + n, head) + c * 8, p.q_vec);
                    if (c == 0) {
                        lse = p.lse[(int64_t)(x.q.q0 + n) * p.q_heads + head];
                        limit = lse == -INFINITY ? 0 : x.q.len - x.q.n + n + 1;
                    }
                }
                *reinterpret_cast<int4*>(qt + swizzled<kRowBytes>(rr, c)) = v;
                if (c == 0) {
                    row_lse[rr] = lse * kLog2e;
                    row_limit[rr] = limit;
                }
            }
            __syncthreads();
            uint32_t qf[kSteps / 2][4];                    // second operands of two steps
            if (kOne) {
    #pragma unroll
                for (int s = 0; s < kSteps / 2; ++s)
                    ldmatrix4(qf[s], q_u + swizzled<kRowBytes>(lane & 7, 4 * s + (lane >> 3)));
            }
            for (int32_t i0 = 0; i0 < mine; i0 += kStages) {
    #pragma unroll
                for (int u = 0; u < kStages; ++u) {
                    const int32_t i = i0 + u;
                    if (i >= mine) break;
                    __syncwarp();
                    constexpr int kAhead = kStages - 1;
                    there[(u + kAhead) % kStages] = rows > 0 && i + kAhead < mine ? fill(i + kAhead) : 0u;
                    cp_commit();
                    const int32_t key = key_of(i) + (lane >> 2);      // and key + 8
                    float old[2] = {0.f, 0.f};
    #pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if ((lane & 3) == 0 && key + 8 * k < x.k1) {
                            if (row0 > 0) old[k] = p.scores_out[at + key + 8 * k];
                            else if (p.decay != 0.f) old[k] = p.decay * p.scores[at + key + 8 * k];
                        }
                    cp_wait<kStages - 1>();
                    __syncwarp();
                    const uint32_t kt = ring + u * kTileBytes;
                    uint32_t kf[kSteps][4];
    #pragma unroll
                    for (int s = 0; s < kSteps; ++s)       // keys 0-7 / 8-15 x d 0-7, then x d 8-15
                        ldmatrix4(kf[s], kt + swizzled<kRowBytes>(lane & 15, 2 * s + (lane >> 4)));
                    float s0 = 0.f, s1 = 0.f;
    #pragma unroll 1
                    for (int32_t g = 0; g < padded; g += 8) {
                        float c[4] = {0.f, 0.f, 0.f, 0.f};
    #pragma unroll
                        for (int s = 0; s < kSteps / 2; ++s) {
                            if (!kOne) ldmatrix4(qf[s], q_u + swizzled<kRowBytes>(g + (lane & 7), 4 * s + (lane >> 3)));
                            mma16816<T>(c, kf[2 * s], qf[s][0], qf[s][1]);
                            mma16816<T>(c, kf[2 * s + 1], qf[s][2], qf[s][3]);
                        }
                        const int rr = g + (lane & 3) * 2;
                        const float2 e = *reinterpret_cast<const float2*>(row_lse + rr);
                        const int2 lim = *reinterpret_cast<const int2*>(row_limit + rr);
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
                        if (key < x.k1) p.scores_out[at + key] = old[0] + ((there[u] >> (lane >> 2)) & 1 ? s0 : 0.f);
                        if (key + 8 < x.k1)
                            p.scores_out[at + key + 8] = old[1] + ((there[u] >> ((lane >> 2) + 8)) & 1 ? s1 : 0.f);
                    }
                }
            }
            cp_wait<0>();
        }
    }
}

// Many rows (an observation window): tcgen05 products of 128 keys x 128 rows.
//   warps 0-15  a thread holds a key and sums over 128 rows, whose scores come
//               from tensor memory: of the even blocks and the odd in turn
//               (warps 0-7, 8-15), rows 0-127 and 128-255 (four warps each)
//   warps 16-17 K blocks through a ring in shared memory
//   warp 18     issues the products of a block with up to 256 rows, into the
//               half of tensor memory that the warps of that block have left
// The product brings -lse along: 16 more columns, of q the three parts of
// -lse / scale that the type can hold, of k what they count for (extra_parts),
// so that a thread needs nothing but the scores: reading 128 rows' lse from
// shared memory took as much of its bandwidth as the product's operands do,
// and bound the kernel (2350 cycles a block, of which the powers take 1024).
// Shares as the row kernel's, a CTA an SM, where a request counts kTileBegin blocks
// before its own; its rows beyond 256 go over the share again, from L2.  (4 windows of 64 tokens at 5000 to 16000, 32 heads on 8 of 128:
// 29.0 us a call.  With three quarters of the powers left out it was 31 of 37: what
// bounds it is the wait for a block's product, 1340 cycles, between two blocks of a
// parity, and the start.  Scores fetched ahead of their
// use, 16 or 32 a time, spill: 41 and 51.)
constexpr int kTileThreads = 608;
constexpr int kTileBegin = 3;      // blocks' time that beginning a request costs (0: 31.5 us, 2: 29.6, 3: 29.2, 6: 29.6)
constexpr int kTileRows = 256;

template <int D>
struct WeighShape {
    static constexpr int kStages = D == 128 ? 4 : 6;
    static constexpr int kQBytes = kTileRows * D * 2;              // [half of 64 columns][256 rows][128 bytes]
    static constexpr int kExtraQ = kQBytes + kStages * BlockShape<D>::kBytes;
    static constexpr int kExtraK = kExtraQ + kTileRows * 32;
    static constexpr int kSmem = kExtraK + kBlock * 32;
};

// x as a sum of three numbers of type T, each times its weight: hi 2^15 + mid 2^4 +
// lo 2^-7.  fp16 parts reach +-2^31 (half steps of 2^-3 there, of 2^-31 near 0), bf16
// parts hold 24 bits of any fp32.
constexpr float kHi = 0x1p15f, kMid = 0x1p4f, kLo = 0x1p-7f;
template <class T>
__device__ __forceinline__ void extra_parts(float x, uint32_t* hi_mid, uint32_t* lo) {
    const T hi = Elem<T>::from_float(x * (1.f / kHi));
    float rest = isfinite(x) ? x - Elem<T>::to_float(hi) * kHi : 0.f;
    const T mid = Elem<T>::from_float(rest * (1.f / kMid));
    rest -= Elem<T>::to_float(mid) * kMid;
    *hi_mid = Elem<T>::pack(Elem<T>::to_float(hi), Elem<T>::to_float(mid));
    *lo = Elem<T>::pack(rest * (1.f / kLo), 0.f);
}

// The share's parts in turn: keys of one request at a time.  Every role walks
// them alike.
struct WeighWalk {
    const WeighParams& p;
    Share share;
    WeighPart x;
    int32_t rows, blocks, passes;
    int64_t at;            // of the part's first key's score

    __device__ __forceinline__ bool next(bool there) {
        for (; share.n > 0 && share.r < p.seqs.num_req; ++share.r, share.first = 0) {
            x.q = load_req(p.seqs, share.r);
            // a request counts kTileBegin units before its blocks
            const int64_t all = x.q.len > 0 ? (int64_t)(x.q.len + kBlock - 1) / kBlock + kTileBegin : 0;
            const int64_t here = min(all - share.first, share.n);
            if (here <= 0) continue;
            share.n -= here;
            const int64_t b0 = max(share.first - kTileBegin, (int64_t)0), b1 = share.first + here - kTileBegin;
            if (b1 <= b0) continue;
            x.k0 = (int32_t)b0 * kBlock;
            x.k1 = (int32_t)min(b1 * kBlock, (int64_t)x.q.len);
            x.table = p.seqs.table + (int64_t)share.r * p.seqs.table_stride;
            rows = there ? x.q.n * (int32_t)p.by_group.d : 0;
            blocks = (int32_t)(b1 - b0);
            passes = (rows + kTileRows - 1) / kTileRows;
            at = ((int64_t)share.r * p.kv_heads + x.h) * p.score_stride + x.k0;
            ++share.r;
            share.first = 0;
            return true;
        }
        return false;
    }
};

template <class T, int D>
__global__ void __launch_bounds__(kTileThreads, 1)
weigh_tiles_kernel(const __grid_constant__ WeighParams p) {
    using S = WeighShape<D>;
    using B = BlockShape<D>;
    constexpr int kMaskSlots = 8;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ uint64_t bars[2 * S::kStages + 5];
    __shared__ uint32_t tmem_base;
    __shared__ int gave_up;
    __shared__ Share share_s;
    __shared__ int32_t least_limit[2];             // of the pass's rows, by its parity
    __shared__ uint4 key_mask[kMaskSlots];
    __shared__ __align__(16) int32_t row_limit[kTileRows];
    __shared__ float upper[2][2][kBlock];          // sums over rows 128-255, two blocks of each parity
    pdl_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t full = smem_u32(bars), empty = full + 8 * S::kStages, s_full = empty + 8 * S::kStages,
                   s_free = s_full + 16, q_ready = s_free + 16;
    const uint32_t q_smem = smem_u32(smem), k_smem = q_smem + S::kQBytes;
    if (tid < kBlock) {
        // every key's extra columns: what the parts of -lse / scale count for
        *reinterpret_cast<uint4*>(smem + S::kExtraK + plain16_offset(tid, 0)) =
            make_uint4(Elem<T>::pack(kHi, kMid), Elem<T>::pack(kLo, 0.f), 0u, 0u);
        *reinterpret_cast<uint4*>(smem + S::kExtraK + plain16_offset(tid, 1)) = make_uint4(0u, 0u, 0u, 0u);
    }
    if (tid == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(full + 8 * i, kCopyArrivals);
            mbar_init(empty + 8 * i, 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(s_full + 8 * t, 1);
            mbar_init(s_free + 8 * t, 8);
        }
        mbar_init(q_ready, 16);
        gave_up = 0;
        least_limit[0] = least_limit[1] = INT32_MAX;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 18) tmem_alloc<512>(smem_u32(&tmem_base));
    pdl_wait();
    uint8_t* const base = p.layer.base();
    if (base == nullptr && tid == 0) report(p.status, LMKV_ERR_BAD_POINTER);
    if (warp == 0) {
        const Share s = find_share(p.seqs.num_req, blockIdx.x / p.kv_heads, p.splits,
                                   [&](int32_t i) -> int64_t {
                                       const int64_t n = units_of(p.seqs, i, kBlock, p.status);
                                       return n > 0 ? n + kTileBegin : 0;
                                   });
        if (lane == 0) share_s = s;
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    WeighWalk walk{p, share_s};
    walk.x.h = blockIdx.x % p.kv_heads;
    const WeighPart& x = walk.x;
    const int32_t group = (int32_t)p.by_group.d;
    if (warp < 16) {
        const int parity = warp >> 3, high = (warp >> 2) & 1;
        const uint32_t s_at = tmem_base + ((uint32_t)(warp & 3) << 21) + parity * 256 + high * 128;
        const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
        // A wait that gave up (ok false) skips the work and not the barriers, which
        // the other warps may be waiting at.
        bool ok = true;
        int32_t it = 0, pass_no = 0;
        while (walk.next(base != nullptr)) {
            const int32_t keys = x.k1 - x.k0;
            if (walk.passes == 0) {                 // nothing but the decay
                for (int32_t k = tid; k < keys; k += 512)
                    p.scores_out[walk.at + k] = p.decay == 0.f ? 0.f : p.decay * p.scores[walk.at + k];
            }
            for (int32_t pass = 0; pass < walk.passes; ++pass, ++pass_no) {
                const int32_t row0 = pass * kTileRows, nrows = min(kTileRows, walk.rows - row0);
                if (it > 0) {
                    // every product with the q before is done once all scores have come, and what
                    // one thread has written to scores_out another may add to
                    bar_sync(1, 512);
                    if (tid == 0) least_limit[pass_no & 1] = INT32_MAX;
                    bar_sync(1, 512);
                }
                {
                    // q by pieces of 16 bytes, a row's side by side (half a row a thread took 3.5 us: 32
                    // lines a load), all on their way before the first is waited for; rows that are not
                    // there weigh nothing
                    constexpr int kPieces = D / 8, kMine = kTileRows * kPieces / 512;
                    int4 qv[kMine];
#pragma unroll
                    for (int i = 0; i < kMine; ++i) {
                        const int32_t at = i * 512 + tid, r = at / kPieces;
                        const int32_t n = (int32_t)p.by_group.div((uint32_t)(row0 + r));
                        const int32_t head = x.h * group + (row0 + r - n * group);
                        qv[i] = r < nrows ? load_q(p.q_row<T>(x.q.q0 + n, head) + at % kPieces * 8, p.q_vec)
                                          : make_int4(0, 0, 0, 0);
                    }
                    const int row = tid >> 1, part = tid & 1;
                    const bool on = row < nrows;
                    const int32_t n = (int32_t)p.by_group.div((uint32_t)(row0 + (on ? row : 0)));
                    const int32_t head = x.h * group + (on ? row0 + row - n * group : 0);
                    const float lse = on ? p.lse[(int64_t)(x.q.q0 + n) * p.q_heads + head] : INFINITY;
#pragma unroll
                    for (int i = 0; i < kMine; ++i) {
                        const int32_t at = i * 512 + tid, r = at / kPieces, c = at % kPieces;
                        const uint32_t to = q_smem + r * 128 + (c >> 3) * (kTileRows * 128) + (((c & 7) ^ (r & 7)) << 4);
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(qv[i].x), "r"(qv[i].y),
                                     "r"(qv[i].z), "r"(qv[i].w) : "memory");
                    }
                    const int32_t limit = !on || lse == -INFINITY ? 0 : x.q.len - x.q.n + n + 1;
                    {
                        // a row that sees nothing weighs nothing: as one of infinite lse
                        uint4 e = make_uint4(0u, 0u, 0u, 0u);
                        if (part == 0)
                            extra_parts<T>(-(lse == -INFINITY ? INFINITY : lse) * p.lse_scale, &e.x, &e.y);
                        *reinterpret_cast<uint4*>(smem + S::kExtraQ + plain16_offset(row, part)) = e;
                    }
                    if (part == 0) row_limit[row] = limit;
                    const int32_t least_here = __reduce_min_sync(0xFFFFFFFFu, on ? limit : INT32_MAX);
                    if (lane == 0) atomicMin(&least_limit[pass_no & 1], least_here);
                    fence_async_shared();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(q_ready);
                    bar_sync(1, 512);               // the limits are there
                }
                const int32_t least = least_limit[pass_no & 1];
                const int32_t chunks = min(max(nrows - high * 128, 0) + 31, 128) >> 5;
                for (int32_t i = 0; i < walk.blocks; ++i, ++it) {
                    if ((it & 1) != parity) continue;
                    const int32_t place = i * kBlock + (warp & 3) * 32 + lane, key = x.k0 + place;
                    float old = 0.f;
                    if (!high && place < keys) {
                        if (pass > 0) old = p.scores_out[walk.at + place];
                        else if (p.decay != 0.f) old = p.decay * p.scores[walk.at + place];
                    }
                    ok = ok && mbar_wait(s_full + 8 * parity, (it >> 1) & 1, &gave_up);
                    float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    bool there = false;
                    if (ok) {
                        if ((warp & 7) == 0 && lane == 0) mbar_arrive(empty + 8 * (it % S::kStages));    // K has been used
                        fence_after_sync();
                        there = (reinterpret_cast<const uint32_t*>(&key_mask[it % kMaskSlots])[warp & 3] >> lane) & 1;
                        const bool whole = x.k0 + i * kBlock + (warp & 3) * 32 + 31 < least;     // every row sees these keys
                        // one path a chunk: a choice within it would keep its powers from overlapping
                        auto add_rows = [&](const uint32_t (&v)[32], int32_t c, auto masked) {
#pragma unroll
                            for (int j = 0; j < 32; j += 4) {
                                float2 a = mul2(make_float2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), sc2);
                                float2 b = mul2(make_float2(__uint_as_float(v[j + 2]), __uint_as_float(v[j + 3])), sc2);
                                a.x = exp2_fast(a.x);
                                a.y = exp2_fast(a.y);
                                b.x = exp2_fast(b.x);
                                b.y = exp2_fast(b.y);
                                if constexpr (decltype(masked)::value) {
                                    const int4 lim = *reinterpret_cast<const int4*>(row_limit + high * 128 + 32 * c + j);
                                    a.x = key < lim.x ? a.x : 0.f;
                                    a.y = key < lim.y ? a.y : 0.f;
                                    b.x = key < lim.z ? b.x : 0.f;
                                    b.y = key < lim.w ? b.y : 0.f;
                                }
                                acc[0] = add2(acc[0], a);
                                acc[1] = add2(acc[1], b);
                            }
                        };
                        // what a chunk waits for the scheduler's other three warps fill
#pragma unroll 1
                        for (int32_t c = 0; c < chunks; ++c) {
                            uint32_t y[32];
                            tmem_ld32(y, s_at + 32 * c);
                            wait_ld();
                            loaded(y);
                            if (whole) add_rows(y, c, std::false_type());
                            else add_rows(y, c, std::true_type());
                        }
                        fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(s_free + 8 * parity);
                    }
                    float total = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
                    float* const other = &upper[parity][(it >> 1) & 1][(warp & 3) * 32 + lane];
                    if (high) *other = total;
                    bar_sync(2 + parity, 256);
                    if (!high && ok && place < keys) p.scores_out[walk.at + place] = old + (there ? total + *other : 0.f);
                }
            }
        }
    } else if (warp < 16 + kLoadWarps) {
        BlockCopy<D> k(p.layer, base, k_smem, warp - 16);
        const uint8_t* const from = k.piece(x.h);
        bool ok = true;
        int32_t it = 0;
        while (ok && walk.next(base != nullptr)) {
            const int32_t total = walk.blocks * walk.passes;
            int32_t i = 0;                               // block of the pass
            if (total > 0) k.lookup(x.table, x.k0, x.k1);
            for (int32_t n = 0; n < total; ++n, ++it) {
                k.take(p.status);
                if (++i == walk.blocks) i = 0;
                if (n + 1 < total) k.lookup(x.table, x.k0 + i * kBlock, x.k1);
                const int st = it % S::kStages;
                if (it >= S::kStages) ok = mbar_wait(empty + 8 * st, (it / S::kStages - 1) & 1, &gave_up);
                if (!ok) break;
                k.put_mask(reinterpret_cast<uint32_t*>(&key_mask[it % kMaskSlots]));
                k.copy(from, st * B::kBytes);
                copies_arrive(full + 8 * st);
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        constexpr uint32_t id128 = instr_desc<T, 128, false>(), id256 = instr_desc<T, 256, false>();
        const uint32_t lead = elect_lead();
        const Desc q0 = desc_k_major(q_smem), k0 = desc_k_major(k_smem);
        const Desc qx = desc_plain16(q_smem + S::kExtraQ), kx = desc_plain16(q_smem + S::kExtraK);
        bool ok = true;
        int32_t it = 0, pass_no = 0;
        while (ok && walk.next(base != nullptr)) {
            for (int32_t pass = 0; pass < walk.passes && ok; ++pass, ++pass_no) {
                const bool two = walk.rows - pass * kTileRows > 128;
                ok = mbar_wait(q_ready, pass_no & 1, &gave_up);
                for (int32_t i = 0; i < walk.blocks && ok; ++i, ++it) {
                    const int parity = it & 1, st = it % S::kStages;
                    ok = mbar_wait(full + 8 * st, (it / S::kStages) & 1, &gave_up) &&
                         (it < 2 || mbar_wait(s_free + 8 * parity, ((it >> 1) - 1) & 1, &gave_up));
                    if (!ok) break;
                    fence_async_shared();
                    fence_after_sync();
                    const Desc a = k0.at(st * B::kBytes);
                    const uint32_t id = two ? id256 : id128;
#pragma unroll
                    for (int s = 0; s < D / 16; ++s)
                        mma_ss(lead, parity * 256, a.at((s >> 2) * B::kHalfBytes + (s & 3) * 32),
                               q0.at((s >> 2) * (kTileRows * 128) + (s & 3) * 32), id, s > 0);
                    mma_ss(lead, parity * 256, kx, qx, id, true);
                    mma_commit(lead, s_full + 8 * parity);
                }
            }
        }
    }
    __syncwarp();
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (tid == 0 && gave_up) report(p.status, LMKV_ERR_TIMEOUT);
    if (warp == 18) tmem_free<512>(tmem_base);
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
constexpr uint32_t kNoKey = 0u;                // of places behind the last token
constexpr uint32_t kNanKey = 1u;
constexpr uint32_t kZeroKey = 0x80000000u;     // of a score of zero
constexpr uint32_t kKeepKey = 0xFFFFFFFFu;     // of tokens that are kept whatever their score
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return kNanKey;
    const uint32_t b = __float_as_uint(x + 0.f);      // -0 + 0 = +0
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

constexpr int kSelectThreads = 1024;
constexpr int kBins = 2048;
constexpr int kSelectTokens = 50 * 1024;      // scores that fit in shared memory

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

// A CTA per (request, head).  Sinks and recent tokens have the largest key of
// all, so what is kept is the budget largest.  The last of these is found
// digit by digit (11, 11 and 10 bits), most significant first, with a histogram
// over the keys that share the digits found so far; then every thread counts
// what it keeps of a run of consecutive tokens, one scan places the runs, and
// the kept tokens are written in order, the first ties among them.  The keys
// are made once, into shared memory (kStaged; more than kSelectTokens are made
// again from L2 instead), and taken four at a time: the kernel is bound by its
// instructions, on the SM of the longest request.  Wide digits are for the
// counters: scores crowd into few exponents, and threads that meet on a
// counter take turns; the score that most tokens may share, zero, is counted
// in registers.  (12 requests of 3500 to 20000 tokens, 8 heads: 17.7 us.  With the move of 12
// of 20000 staged 42 : 48 us not staged, of 48000 60 : 78.)
template <bool kStaged>
__global__ void __launch_bounds__(kSelectThreads)
select_kernel(const __grid_constant__ EvictParams p) {
    __shared__ uint32_t hist[kBins];
    __shared__ uint32_t digit_s, above_s;
    __shared__ int2 warp_sums[32];
    extern __shared__ __align__(16) uint32_t keys[];
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
    const int32_t lo = p.sinks, hi = len - p.recent, quads = (len + 3) >> 2;
    auto make_key = [&](int32_t i, float s) {
        return i >= len ? kNoKey : i < lo || i >= hi ? kKeepKey : order_key(s);
    };
    if (kStaged) {
        // every score of the thread on its way before the first is waited for
        for (int32_t i = tid; i < len; i += kSelectThreads)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(keys + i)), "l"(w + i) : "memory");
        cp_commit();
        cp_wait<0>();
    }
    // four tokens' keys; `raw`: from the scores, which the first pass over
    // shared memory turns into keys
    auto quad = [&](int32_t q, bool raw) {
        uint4* const place = reinterpret_cast<uint4*>(keys) + q;
        if (kStaged && !raw) return *place;
        uint32_t k[4];
        if (kStaged) {
            const uint4 s = *place;
            k[0] = s.x, k[1] = s.y, k[2] = s.z, k[3] = s.w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) k[j] = 4 * q + j < len ? __float_as_uint(w[4 * q + j]) : 0u;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) k[j] = make_key(4 * q + j, __uint_as_float(k[j]));
        const uint4 x = make_uint4(k[0], k[1], k[2], k[3]);
        if (kStaged) *place = x;
        return x;
    };
    uint32_t prefix = 0, want = (uint32_t)p.budget;       // want: still to take among the prefix's
    for (int top = 32; top > 0;) {                         // bits from top on are found
        const int low = top > 11 ? top - 11 : 0;
        const uint32_t digits = (1u << (top - low)) - 1u;
        for (int i = tid; i < kBins; i += kSelectThreads) hist[i] = 0;
        __syncthreads();
        uint32_t zeros = 0;
        auto count = [&](uint32_t k) {
            if (top < 32 && (k >> top) != (prefix >> top)) return;
            if (k == kZeroKey) ++zeros;
            else atomicAdd(&hist[(k >> low) & digits], 1u);
        };
        for (int32_t q = tid; q < quads; q += kSelectThreads) {
            const uint4 k = quad(q, top == 32);
            count(k.x);
            count(k.y);
            count(k.z);
            count(k.w);
        }
        zeros = __reduce_add_sync(0xFFFFFFFFu, zeros);
        if ((tid & 31) == 0 && zeros > 0) atomicAdd(&hist[(kZeroKey >> low) & digits], zeros);
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
    // number of quads, so that the threads' places lie in different banks.
    const int32_t run = ((quads + kSelectThreads - 1) / kSelectThreads) | 1;
    const int32_t from = min(tid * run, quads), to = min(from + run, quads);
    int2 mine = make_int2(0, 0);                              // kept for certain, ties
    for (int32_t q = from; q < to; ++q) {
        const uint4 k = quad(q, false);
        mine.x += (k.x > prefix) + (k.y > prefix) + (k.z > prefix) + (k.w > prefix);
        mine.y += (k.x == prefix) + (k.y == prefix) + (k.z == prefix) + (k.w == prefix);
    }
    int2 at = scan_pairs(mine, warp_sums);
    // 32 tokens at a time as bits, of which only the kept ones are gone through
    auto bits = [&](int32_t q0, uint32_t* more, uint32_t* tie) {
        *more = *tie = 0;
#pragma unroll
        for (int32_t u = 0; u < 8; ++u) {
            if (q0 + u >= to) break;
            const uint4 k = quad(q0 + u, false);
            *more |= ((k.x > prefix) | (k.y > prefix) << 1 | (k.z > prefix) << 2 | (k.w > prefix) << 3) << (4 * u);
            *tie |= ((k.x == prefix) | (k.y == prefix) << 1 | (k.z == prefix) << 2 | (k.w == prefix) << 3) << (4 * u);
        }
    };
    auto walk = [&](int32_t q0, uint32_t more, uint32_t tie, auto put) {
        for (uint32_t left = more | tie; left != 0; left &= left - 1) {
            const int bit = __ffs(left) - 1;
            const bool sure = (more >> bit) & 1;
            if (sure || at.y < (int32_t)want) {
                const int32_t slot = at.x + min(at.y, (int32_t)want);
                if (slot < p.budget) put(slot, 4 * q0 + bit);
            }
            at.x += sure;
            at.y += !sure;
        }
    };
    if (kStaged) {
        // the keys make room for the list of tokens, which is then written out side by side
        constexpr int kWords = (kSelectTokens / kSelectThreads + 4 + 31) / 32;
        uint32_t more[kWords], tie[kWords];
#pragma unroll
        for (int n = 0; n < kWords; ++n) bits(from + 8 * n, &more[n], &tie[n]);
        __syncthreads();
#pragma unroll
        for (int n = 0; n < kWords; ++n)
            walk(from + 8 * n, more[n], tie[n], [&](int32_t slot, int32_t i) { keys[slot] = (uint32_t)i; });
        __syncthreads();
#pragma unroll 4
        for (int32_t s = tid; s < p.budget; s += kSelectThreads) {
            const int32_t i = (int32_t)keys[s];
            keep[s] = i;
            if (kept != nullptr) kept[s] = w[i];
        }
    } else {
        for (int32_t q0 = from; q0 < to; q0 += 8) {
            uint32_t more, tie;
            bits(q0, &more, &tie);
            walk(q0, more, tie, [&](int32_t slot, int32_t i) {
                keep[slot] = i;
                if (kept != nullptr) kept[slot] = w[i];
            });
        }
    }
}

// ---- compaction ---------------------------------------------------------

constexpr int kMoveThreads = 128;
constexpr int kMoveSlots = kMoveThreads;   // slots of a batch
constexpr int kMoveDepth = 3;              // batches of rows on their way or being written
constexpr int kPieceBytes = 64;            // of a head's row: more CTAs, whole sectors

// Moves the kept rows of one (request, head, K or V, column piece) to the
// front of the request's pages, in place.  keep is ascending, so keep[i] >= i
// and a batch of slots in order may be written once its own rows, and those of
// the batches before it, have been read: what later batches read lies behind.
// So rows may be fetched as early as one likes: the next batches' are under
// way in shared memory (cp.async) while one is written, each thread writing
// what it fetched itself, with one barrier a batch.  Where rows come from and
// go to is looked up two batches ahead of the fetch, a slot a thread.  Slots whose token
// stays (a leading run, as keep[i] - i never falls) are skipped.  Bound by
// reading and writing the moved rows.  (The same batch to 4096 tokens: 76 us, 360 MB, 4.7
// TB/s, 0.70 of the copy rate: the rows are read in pieces of 64 bytes from all over the
// pages.  Pieces of 32 bytes 128 : 104 us a call, of 128 bytes 105; four batches on their way 103,
// five 130.)
template <int kBytes>
__global__ void __launch_bounds__(kMoveThreads)
compact_kernel(const __grid_constant__ EvictParams p, int32_t pieces) {
    extern __shared__ __align__(16) uint8_t move_smem[];       // [kMoveDepth][kMoveSlots][piece]
    constexpr int kPlaces = kMoveDepth + 1;
    __shared__ uint32_t from[kPlaces][kMoveSlots], to[kPlaces][kMoveSlots];     // rows of the K or V half
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
    const int32_t vecs = (p.head_bytes - piece * kPieceBytes) / kBytes;      // of this piece (kVecs at most are moved)
    const int32_t* table = p.table + (int64_t)r * p.table_stride;
    const int32_t* keep = p.keep + ((int64_t)r * p.kv_heads + h) * p.budget;
    int32_t first = 0, end = p.budget;                 // first slot that moves
    while (first < end) {
        const int32_t mid = (first + end) >> 1;
        if (keep[mid] == mid) first = mid + 1;
        else end = mid;
    }
    base += kv * p.layer.half_bytes() + (int64_t)h * p.head_bytes + piece * kPieceBytes;
    const int32_t batches = (p.budget - first + kMoveSlots - 1) / kMoveSlots;
    // unit k of thread t: vector t % kVecs of slot t / kVecs + k * kMoveThreads / kVecs
    constexpr int kVecs = kPieceBytes / kBytes, kUnits = kMoveSlots * kVecs / kMoveThreads;
    constexpr int kStep = kMoveThreads / kVecs;
    const int32_t v = threadIdx.x % kVecs, s0 = threadIdx.x / kVecs;
    const bool mine = v < vecs;
    uint8_t* const at = base + v * kBytes;
    uint8_t* const ring = move_smem + threadIdx.x * kBytes;

    // Batch i's slot of this thread: its token (-1: none), one batch ahead of the look-up.
    auto token_of = [&](int32_t i) {
        const int32_t s = first + i * kMoveSlots + (int32_t)threadIdx.x;
        return i < batches && s < p.budget ? keep[s] : -1;
    };
    auto look_up = [&](int32_t i, int32_t tok) {
        uint32_t a = Layer::kNoRow, b = Layer::kNoRow;
        if (tok >= 0) {
            const int32_t s = first + i * kMoveSlots + (int32_t)threadIdx.x;
            const uint32_t ca = p.layer.column(tok), cb = p.layer.column(s);
            a = p.layer.row_of(table[ca], tok, ca);
            b = p.layer.row_of(table[cb], s, cb);
            if (a == Layer::kNoRow || b == Layer::kNoRow) {
                report(p.status, LMKV_ERR_BAD_BLOCK);
                a = b = Layer::kNoRow;
            }
        }
        from[i % kPlaces][threadIdx.x] = a;
        to[i % kPlaces][threadIdx.x] = b;
    };
    auto fetch = [&](int32_t i) {
        if (i < batches && mine) {
            uint8_t* const stage = ring + i % kMoveDepth * (kMoveSlots * kPieceBytes);
#pragma unroll
            for (int k = 0; k < kUnits; ++k) {
                const uint32_t row = from[i % kPlaces][s0 + k * kStep];
                if (row == Layer::kNoRow) continue;
                const int64_t a = (int64_t)((uint64_t)row * (uint64_t)p.layer.row_bytes);
                uint8_t* const dst = stage + k * kMoveThreads * kBytes;
                if constexpr (kBytes == 16) cp_async16(smem_u32(dst), at + a);
                else if constexpr (kBytes == 4)
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(at + a) : "memory");
                else *dst = at[a];
            }
        }
        cp_commit();
    };
    for (int32_t i = 0; i < kMoveDepth; ++i) look_up(i, token_of(i));
    int32_t next = token_of(kMoveDepth);
    __syncthreads();
    for (int32_t i = 0; i < kMoveDepth - 1; ++i) fetch(i);
#pragma unroll 1
    for (int32_t i = 0; i < batches; ++i) {
        cp_wait<kMoveDepth - 2>();
        __syncthreads();               // batch i and those before it have been read by every thread
        fetch(i + kMoveDepth - 1);
        if (mine) {
            const uint8_t* const stage = ring + i % kMoveDepth * (kMoveSlots * kPieceBytes);
#pragma unroll
            for (int k = 0; k < kUnits; ++k) {
                const uint32_t row = to[i % kPlaces][s0 + k * kStep];
                if (row == Layer::kNoRow) continue;
                const int64_t b = (int64_t)((uint64_t)row * (uint64_t)p.layer.row_bytes);
                const uint8_t* const src = stage + k * kMoveThreads * kBytes;
                if constexpr (kBytes == 16) *reinterpret_cast<int4*>(at + b) = *reinterpret_cast<const int4*>(src);
                else if constexpr (kBytes == 4) *reinterpret_cast<int32_t*>(at + b) = *reinterpret_cast<const int32_t*>(src);
                else at[b] = *src;
            }
        }
        look_up(i + kMoveDepth, next);                 // the places of batch i - 1, which every thread has left
        next = token_of(i + kMoveDepth + 1);
    }
    cp_wait<0>();
}

template <int kBytes>
int launch_compact(const EvictParams& p, void* stream) {
    const int32_t pieces = (p.head_bytes + kPieceBytes - 1) / kPieceBytes;
    constexpr int ring = kMoveDepth * kMoveSlots * kPieceBytes;
    const int rc = allow_smem<compact_kernel<kBytes>, ring>();
    if (rc != LMKV_OK) return rc;
    return launch(compact_kernel<kBytes>, (int64_t)p.num_req * p.kv_heads * 2 * pieces, kMoveThreads, ring, stream, 1, p,
                  pieces);
}

// Rows per KV head from which the tile kernel takes a batch: beyond one second
// operand of the row kernel, whose products are then many for the keys that it
// reads.  (Rows against tiles, us: 8 requests of 8000 keys, 8 rows 40 : 42, 16 rows 58 : 42, 64
// rows 95 : 42; 2 of 3000, 13 : 17, 17 : 16, 25 : 17; 24 of 2000, 33 : 36, 48 : 36, 80 : 38;
// 300 of 500, 16 rows 132 : 95; only many requests of next to nothing lose: 1000 of 64 keys, 16 rows
// 124 : 176, 64 rows 232 : 203.)
constexpr int kTileMinRows = 9;

template <class T, int D>
int weigh_typed(WeighParams& p, void* stream) {
    const int64_t rows = (int64_t)(p.seqs.max_new < p.seqs.num_tokens ? p.seqs.max_new : p.seqs.num_tokens) * p.by_group.d;
    // (the tile kernel carries -lse / scale, in fp16 up to 2^31: lse up to 2^19 at the smallest scale it takes)
    // (with no room for cached tokens a CTA of the row kernel looks at the lengths and has no shares)
    const bool tiles = rows >= kTileMinRows && std::fabs(p.scale_log2) >= 0x1p-12f * kLog2e && p.seqs.max_kv_len > 0;
    p.lse_scale = kLog2e / p.scale_log2;
    const int64_t heads = p.kv_heads, req = p.seqs.num_req;
    // one round of CTAs
    const int64_t unit = tiles ? kBlock : kUnit;
    const int64_t want = (tiles ? 1 : kRowCtas) * kSms / heads, most = ((int64_t)p.seqs.max_kv_len + unit - 1) / unit * req;
    p.splits = (int32_t)(want < 1 || most < 1 ? 1 : want > most ? most : want);
    const int64_t grid = most < 1 ? 1 : heads * p.splits;
    if (!tiles) {
        constexpr int ring = kWarps * kStages * kChunk * D * 2;
        int rc = allow_smem<weigh_rows_kernel<T, D, true>, ring>();
        if (rc == LMKV_OK) rc = allow_smem<weigh_rows_kernel<T, D, false>, ring>();
        if (rc != LMKV_OK) return rc;
        return rows <= 8 ? launch(weigh_rows_kernel<T, D, true>, grid, kWarps * 32, ring, stream, 1, p)
                         : launch(weigh_rows_kernel<T, D, false>, grid, kWarps * 32, ring, stream, 1, p);
    }
    const int rc = allow_smem<weigh_tiles_kernel<T, D>, WeighShape<D>::kSmem>();
    if (rc != LMKV_OK) return rc;
    return launch(weigh_tiles_kernel<T, D>, grid, kTileThreads, WeighShape<D>::kSmem, stream, 1, p);
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
    if (layer < 0 || layer >= pool->num_layers || !std::isfinite(scale * kLog2e) || !std::isfinite(decay))
        return LMKV_ERR_INVALID_ARG;
    rc = check_batch(pool, batch, num_q_heads);
    if (rc != LMKV_OK) return rc;
    if (batch->max_kv_len > INT32_MAX - 65536 || score_stride < batch->max_kv_len) return LMKV_ERR_INVALID_ARG;
    if (batch->num_req == 0) return LMKV_OK;
    // (with no room for cached tokens only the lengths are looked at)
    const bool room = batch->max_kv_len > 0;
    if (!room && (batch->q_start == nullptr || batch->kv_len == nullptr)) return LMKV_OK;
    if (batch->q_start == nullptr || batch->kv_len == nullptr || (room && batch->block_table == nullptr) ||
        (room && (scores_out == nullptr || (decay != 0.f && scores == nullptr))))
        return LMKV_ERR_INVALID_ARG;
    if (room && batch->num_tokens > 0 && (!rows_ok(q, 2) || lse == nullptr)) return LMKV_ERR_INVALID_ARG;
    WeighParams p = {};
    p.layer = Layer::of(pool, layer);
    p.seqs = Seqs::of(batch);
    if (room && batch->num_tokens > 0) {
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
        max_kv_len < 0 || max_kv_len > INT32_MAX - 65536 || max_kv_len > (int64_t)max_blocks * pool->block_size ||
        pool->num_blocks * pool->block_size >= (int64_t)Layer::kNoRow)          // rows are numbered with 32 bits
        return LMKV_ERR_INVALID_ARG;
    if (budget < 1 || sinks < 0 || recent < 0 || (int64_t)sinks + recent > budget || score_stride < max_kv_len ||
        (kept_scores != nullptr && kept_stride < budget))
        return LMKV_ERR_INVALID_ARG;
    if (num_req == 0) return LMKV_OK;
    if (kv_len == nullptr || keep == nullptr || new_len == nullptr || new_len == kv_len ||
        (kept_scores != nullptr && kept_scores == scores) ||
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
            rc = launch(select_kernel<true>, (int64_t)num_req * p.kv_heads, kSelectThreads, ((size_t)max_kv_len + 3) / 4 * 16, stream,
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
