// lmkv_pages.cu -- pages of the pool: copied, forked, given, freed and moved
// together, with their bookkeeping on the device.
//
// What is counted is whole numbers, so the order of the atomic additions that
// count references changes nothing; what is given (free pages, in ascending
// order, row by row) is given by prefix sums in one CTA.
#include "lmkv_paged.cuh"

#include <climits>

namespace {

using namespace lmkv_paged;

// Rows of one page that go to another.
struct Move {
    int32_t src, dst;
    int32_t tokens;      // the first of the page; 0: nothing to do
};

struct PagesParams {
    const int32_t* table;
    int32_t* table_out;
    const int32_t* kv_len;
    const int32_t* new_len;       // resize
    const int32_t* parents;       // fork
    int32_t* len_out;             // fork
    const int32_t* refs;
    int32_t* refs_out;
    int32_t* page_map;            // compact
    int32_t* status;
    int32_t rows, rows_out, max_blocks, block_size;
    int32_t num_blocks;
    // workspace
    int32_t* count;               // moves
    int32_t* owner;               // [num_blocks] fork: first row that goes on with a page that is not full
    int32_t* list;                // [num_blocks] free pages in ascending order
    int32_t* held;                // [num_blocks] compact: held pages in ascending order
    int32_t* first;               // [rows] pages given to the rows before
    Move* moves;                  // [max(rows, num_blocks)]

    __device__ __forceinline__ int32_t length(const int32_t* lens, int32_t r) const {
        const int32_t n = lens[r], most = (int32_t)min((int64_t)max_blocks * block_size, (int64_t)INT32_MAX);
        if (n < 0 || n > most) report(status, LMKV_ERR_BAD_LENGTH);
        return min(max(n, 0), most);
    }
    __device__ __forceinline__ int32_t pages(int32_t len) const {
        return len / block_size + (len % block_size != 0 ? 1 : 0);
    }
    __device__ __forceinline__ bool valid(int32_t id) const { return id >= 0 && id < num_blocks; }
    // One reference more or less to a page that may be counted.
    __device__ __forceinline__ void add(int32_t id, int32_t by) const {
        if (!valid(id)) report(status, LMKV_ERR_BAD_BLOCK);
        else if (refs_out[id] >= 0 || refs[id] >= 0) atomicAdd(refs_out + id, by);
    }
};

constexpr int kThreads = 256;

// What a call counts and gives is worked out by one cluster of CTAs: its steps wait for
// one another at the cluster's barrier.  (Fork and grow of 16 requests of 8 beams 37 us, of 2 of 4 beams 33; with a
// launch for each step 42 and 43; clusters of 4 40 and 33, of 2 49 and 41.)
constexpr int kCluster = 8;
constexpr int kOne = 1024;         // threads of a CTA
constexpr int kWarps = kOne / 32;
constexpr int kAll = kCluster * kOne, kAllWarps = kCluster * kWarps;
// Pages that a pool may have here: the threads' counters go beyond the last one by less than kAll, and
// have 32 bits.
constexpr int64_t kMostPages = (int64_t)INT32_MAX - kAll;
// Entries of a table, whose columns a warp goes through 32 at a time.
constexpr int64_t kMostEntries = (int64_t)INT32_MAX - kAll;

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The references as they are, and what else starts from nothing.
__device__ __forceinline__ void begin_all(const PagesParams& p) {
    for (int32_t i = blockIdx.x * kOne + threadIdx.x; i < p.num_blocks; i += kAll) {
        if (p.refs_out != p.refs) p.refs_out[i] = p.refs[i];
        if (p.parents != nullptr) p.owner[i] = INT_MAX;
        if (p.page_map != nullptr) p.page_map[i] = i;
    }
}

// fork: rows give their pages back, and those of the new table begin; a warp a row.
__device__ __forceinline__ void fork_rows(const PagesParams& p) {
    const int lane = threadIdx.x & 31;
    for (int32_t b = blockIdx.x * kWarps + (threadIdx.x >> 5); b < p.rows + p.rows_out; b += kAllWarps) {
        if (b < p.rows) {
            const int32_t n = p.pages(p.length(p.kv_len, b));
            const int32_t* const row = p.table + (int64_t)b * p.max_blocks;
#pragma unroll 4
            for (int32_t c = lane; c < n; c += 32) p.add(row[c], -1);
            continue;
        }
        const int32_t i = b - p.rows, parent = p.parents[i];
        const bool on = parent >= 0 && parent < p.rows;
        const int32_t len = on ? p.length(p.kv_len, parent) : 0;
        const int32_t full = len / p.block_size, n = p.pages(len);
        const int32_t* const row = p.table + (int64_t)(on ? parent : 0) * p.max_blocks;
        int32_t* const out = p.table_out + (int64_t)i * p.max_blocks;
#pragma unroll 4
        for (int32_t c = lane; c < p.max_blocks; c += 32) {
            const int32_t id = c < n ? row[c] : -1;
            out[c] = id;
            if (c < full) p.add(id, 1);
            else if (c < n && p.valid(id)) atomicMin(p.owner + id, i);
        }
        if (lane == 0) p.len_out[i] = len;
    }
}

// resize: pages behind the rows' new lengths lose a reference.
__device__ __forceinline__ void resize_rows(const PagesParams& p) {
    const int lane = threadIdx.x & 31;
    for (int32_t r = blockIdx.x * kWarps + (threadIdx.x >> 5); r < p.rows; r += kAllWarps) {
        const int32_t had = p.pages(p.length(p.kv_len, r)), has = p.pages(p.length(p.new_len, r));
        const int32_t* const row = p.table + (int64_t)r * p.max_blocks;
        int32_t* const out = p.table_out + (int64_t)r * p.max_blocks;
#pragma unroll 4
        for (int32_t c = lane; c < p.max_blocks; c += 32) {
            const int32_t id = c < had ? row[c] : -1;
            if (c >= has && c < had) p.add(id, -1);
            out[c] = c < has ? id : -1;
        }
    }
}

// Exclusive prefix sum over the CTA's threads; *all: the sum of all.
__device__ __forceinline__ int32_t scan_cta(int32_t x, int32_t* warp_sums, int32_t* all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t upto = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t y = __shfl_up_sync(0xFFFFFFFFu, upto, d);
        if (lane >= d) upto += y;
    }
    if (lane == 31) warp_sums[warp] = upto;
    __syncthreads();
    int32_t s = warp_sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t y = __shfl_up_sync(0xFFFFFFFFu, s, d);
        if (lane >= d) s += y;
    }
    *all = __shfl_sync(0xFFFFFFFFu, s, 31);
    const int32_t before = __shfl_sync(0xFFFFFFFFu, s, (warp + 31) & 31);
    __syncthreads();           // warp_sums may be written again
    return (warp > 0 ? before : 0) + upto - x;
}

// Lists the pages whose reference count passes, in ascending order, up to `most` of them; returns how many pass.
// A warp takes a contiguous part: it counts, the CTA adds up, it writes.
template <class Pass>
__device__ __forceinline__ int32_t list_pages(const PagesParams& p, int32_t* out, int32_t most, int32_t* warp_sums, Pass pass) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t span = ((p.num_blocks + kWarps - 1) / kWarps + 127) / 128 * 128;
    const int64_t i0 = (int64_t)warp * span, i1 = min(i0 + span, (int64_t)p.num_blocks);
    auto bits_at = [&](int64_t i) {        // of four pages, this lane's
        uint32_t m = 0;
        const int64_t at = i + lane * 4;
        if (at + 3 < p.num_blocks) {
            const int4 v = *reinterpret_cast<const int4*>(p.refs_out + at);
            m = (pass(v.x) ? 1u : 0u) | (pass(v.y) ? 2u : 0u) | (pass(v.z) ? 4u : 0u) | (pass(v.w) ? 8u : 0u);
        } else {
            for (int k = 0; k < 4; ++k)
                if (at + k < p.num_blocks && pass(p.refs_out[at + k])) m |= 1u << k;
        }
        return m;
    };
    int32_t n = 0;
#pragma unroll 4
    for (int64_t i = i0; i < i1; i += 128) n += __popc(bits_at(i));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, d);
    int32_t all;
    int32_t at = scan_cta(lane == 0 ? n : 0, warp_sums, &all);
    at = __shfl_sync(0xFFFFFFFFu, at, 0);
#pragma unroll 4
    for (int64_t i = i0; i < i1; i += 128) {
        if (at >= most) break;
        const uint32_t m = bits_at(i);
        int32_t upto = __popc(m);
        const int32_t mine = upto;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t y = __shfl_up_sync(0xFFFFFFFFu, upto, d);
            if (lane >= d) upto += y;
        }
        int32_t to = at + upto - mine;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if ((m >> k) & 1) {
                if (to < most) out[to] = (int32_t)(i + lane * 4 + k);
                ++to;
            }
        at += __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
    return all;
}

// Gives the pages that rows want, the lowest free ones, row by row; by the cluster's first CTA.
// fork: a row wants a page for the tokens of its last page, if another goes on with
// that; resize: those of its new length that it does not have.
template <bool kFork>
__device__ __forceinline__ void give(const PagesParams& p, int32_t* warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t total = 0;
    for (int32_t r0 = 0; r0 < p.rows_out; r0 += kOne) {
        const int32_t r = r0 + (int32_t)threadIdx.x;
        int32_t n = 0;
        if (r < p.rows_out) {
            if constexpr (kFork) {
                const int32_t len = p.len_out[r];
                if (len % p.block_size != 0) {
                    const int32_t id = p.table_out[(int64_t)r * p.max_blocks + len / p.block_size];
                    if (!p.valid(id)) report(p.status, LMKV_ERR_BAD_BLOCK);
                    else if (p.owner[id] == r && p.refs_out[id] == 0) p.refs_out[id] = 1;     // (no other row's concern)
                    else n = 1;
                }
            } else {
                n = max(0, p.pages(p.length(p.new_len, r)) - p.pages(p.length(p.kv_len, r)));
            }
        }
        int32_t all;
        const int32_t before = scan_cta(n, warp_sums, &all);
        if (r < p.rows_out) p.first[r] = total + before;
        total += all;              // (a table has fewer than 2^31 entries)
    }
    __syncthreads();               // this CTA's references count
    const int32_t there = total > 0 ? list_pages(p, p.list, min(total, p.num_blocks), warp_sums, [](int32_t x) { return x == 0; }) : 0;
    __syncthreads();
    for (int32_t r = warp; r < p.rows_out && total > 0; r += kWarps) {
        const int32_t at = p.first[r], n = (r + 1 < p.rows_out ? p.first[r + 1] : total) - at;
        if (n == 0) continue;
        int32_t* const row = p.table_out + (int64_t)r * p.max_blocks;
        const int32_t col = kFork ? p.len_out[r] / p.block_size : p.pages(p.length(p.kv_len, r));
        for (int32_t i = lane; i < n; i += 32) {
            const int32_t id = at + i < there ? p.list[at + i] : -1;
            if (id < 0) report(p.status, LMKV_ERR_NO_PAGES);
            else p.refs_out[id] = 1;
            if constexpr (kFork) p.moves[at + i] = Move{row[col], id, id < 0 ? 0 : p.len_out[r] % p.block_size};
            row[col + i] = id;
        }
    }
    if (kFork && threadIdx.x == 0) *p.count = total;
}

// compact: the i-th free page from below takes the i-th held one from above, as
// long as that lies behind it; by the cluster's first CTA.
__device__ __forceinline__ void close_gaps(const PagesParams& p, int32_t* warp_sums) {
    __shared__ int32_t moved;
    if (threadIdx.x == 0) moved = 0;
    const int32_t gaps = list_pages(p, p.list, p.num_blocks, warp_sums, [](int32_t x) { return x == 0; });
    const int32_t held = list_pages(p, p.held, p.num_blocks, warp_sums, [](int32_t x) { return x > 0; });
    __syncthreads();
    const int32_t most = min(gaps, held);
    int32_t mine = 0;
    for (int32_t i = threadIdx.x; i < most; i += kOne) {
        const int32_t to = p.list[i], from = p.held[held - 1 - i];
        if (to >= from) break;     // so are all behind
        p.moves[i] = Move{from, to, p.block_size};
        p.page_map[from] = to;
        p.refs_out[to] = p.refs_out[from];
        p.refs_out[from] = 0;
        ++mine;
    }
    atomicAdd(&moved, mine);
    __syncthreads();
    if (threadIdx.x == 0) *p.count = moved;
}

__device__ __forceinline__ void follow_rows(const PagesParams& p) {
    const int lane = threadIdx.x & 31;
    for (int32_t r = blockIdx.x * kWarps + (threadIdx.x >> 5); r < p.rows; r += kAllWarps) {
        const int32_t n = p.pages(p.length(p.kv_len, r));
        const int32_t* const row = p.table + (int64_t)r * p.max_blocks;
        int32_t* const out = p.table_out + (int64_t)r * p.max_blocks;
#pragma unroll 4
        for (int32_t c = lane; c < p.max_blocks; c += 32) {
            int32_t id = c < n ? row[c] : -1;
            if (c < n) {
                if (p.valid(id)) id = p.page_map[id];
                else report(p.status, LMKV_ERR_BAD_BLOCK);
            }
            out[c] = id;
        }
    }
}

enum class Call { kFork, kResize, kCompact };

template <Call kCall>
__global__ void __launch_bounds__(kOne, 1) pages_plan_kernel(const __grid_constant__ PagesParams p) {
    __shared__ int32_t warp_sums[kWarps];
    pdl_launch_dependents();
    pdl_wait();
    if (kCall != Call::kResize || p.refs_out != p.refs) {
        begin_all(p);
        cluster_sync();
    }
    if constexpr (kCall == Call::kCompact) {
        if (blockIdx.x == 0) close_gaps(p, warp_sums);
        cluster_sync();
        follow_rows(p);
    } else {
        if constexpr (kCall == Call::kFork) fork_rows(p);
        else resize_rows(p);
        cluster_sync();
        if (blockIdx.x == 0) give<kCall == Call::kFork>(p, warp_sums);
    }
}

// ---- copies -------------------------------------------------------------

struct CopyParams {
    const uint8_t* const* layer_base;
    uint8_t* const* scales;
    const int32_t *src, *dst;      // or
    const Move* moves;
    const int32_t* count;
    int32_t* status;
    int64_t num_blocks, row_bytes, half_bytes;
    int32_t n, block_size, layers, kv_heads;
    FastDiv by_layers;
};

constexpr int kVecs = 8;           // 16-byte loads of a thread in flight

// A CTA an item, in turn: the tokens of one page, K or V of one layer, as one run
// of rows.  Bound by the bytes, both ways.  (650 pages of 16 layers, 680 MB both ways: 108 us, 6.3 TB/s.)
__global__ void __launch_bounds__(kThreads) pages_copy_kernel(const __grid_constant__ CopyParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int32_t n = p.moves != nullptr ? *p.count : p.n;
    const int64_t items = (int64_t)n * p.layers * 2;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        // K and V of a layer, then the next layer, then the next page
        const int kv = (int)(item & 1);
        int32_t i, layer;
        if (items <= INT32_MAX) {
            i = (int32_t)p.by_layers.div((uint32_t)(item >> 1));
            layer = (int32_t)(item >> 1) - i * p.layers;
        } else {
            i = (int32_t)((item >> 1) / p.layers);
            layer = (int32_t)((item >> 1) % p.layers);
        }
        Move m;
        if (p.moves != nullptr) m = p.moves[i];
        else m = Move{p.src[i], p.dst[i], p.block_size};
        const uint8_t* const base = p.layer_base[layer];
        uint8_t* const sc = p.scales != nullptr ? p.scales[layer] : nullptr;
        if (m.tokens == 0 || m.src == m.dst) continue;
        if (m.src < 0 || m.src >= p.num_blocks || m.dst < 0 || m.dst >= p.num_blocks) {
            if (threadIdx.x == 0) report(p.status, LMKV_ERR_BAD_BLOCK);
            continue;
        }
        if (base == nullptr || (reinterpret_cast<uintptr_t>(base) & 15) || (p.scales != nullptr && sc == nullptr)) {
            if (threadIdx.x == 0) report(p.status, LMKV_ERR_BAD_POINTER);
            continue;
        }
        const int64_t page = p.block_size * p.row_bytes;
        const int4* const from = reinterpret_cast<const int4*>(base + kv * p.half_bytes + m.src * page);
        int4* const to = reinterpret_cast<int4*>(const_cast<uint8_t*>(base) + kv * p.half_bytes + m.dst * page);
        const int64_t vecs = m.tokens * p.row_bytes / 16;
        for (int64_t v0 = threadIdx.x; v0 < vecs; v0 += kThreads * kVecs) {
            int4 x[kVecs];
#pragma unroll
            for (int u = 0; u < kVecs; ++u)
                if (v0 + u * kThreads < vecs)
                    asm volatile("ld.global.L1::no_allocate.v4.s32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(x[u].x), "=r"(x[u].y), "=r"(x[u].z), "=r"(x[u].w) : "l"(from + v0 + u * kThreads)
                                 : "memory");
#pragma unroll
            for (int u = 0; u < kVecs; ++u)
                if (v0 + u * kThreads < vecs)
                    asm volatile("st.global.cs.v4.s32 [%0], {%1, %2, %3, %4};" ::"l"(to + v0 + u * kThreads), "r"(x[u].x),
                                 "r"(x[u].y), "r"(x[u].z), "r"(x[u].w) : "memory");
        }
        if (sc != nullptr)
            for (int32_t h = threadIdx.x; h < p.kv_heads; h += kThreads)
                sc[(kv * p.num_blocks + m.dst) * p.kv_heads + h] = sc[(kv * p.num_blocks + m.src) * p.kv_heads + h];
    }
}

int launch_copy(const lmkv_pool_t* pool, void* const* scales, const int32_t* src, const int32_t* dst, const Move* moves,
                const int32_t* count, int64_t most, int32_t* d_status, void* stream) {
    CopyParams c = {};
    c.layer_base = reinterpret_cast<const uint8_t* const*>(pool->layer_base);
    c.scales = reinterpret_cast<uint8_t* const*>(scales);
    c.src = src;
    c.dst = dst;
    c.moves = moves;
    c.count = count;
    c.status = d_status;
    c.num_blocks = pool->num_blocks;
    c.row_bytes = (int64_t)pool->num_kv_heads * pool->head_dim * pool->elem_bytes;
    c.half_bytes = pool->num_blocks * pool->block_size * c.row_bytes;
    c.n = (int32_t)most;
    c.block_size = pool->block_size;
    c.layers = pool->num_layers;
    c.kv_heads = pool->num_kv_heads;
    c.by_layers = FastDiv((uint32_t)pool->num_layers);
    constexpr int64_t kCtas = 4 * kSms;
    const int64_t items = most * pool->num_layers * 2;
    return launch(pages_copy_kernel, items < kCtas ? items : kCtas, kThreads, 0, stream, 1, c);
}

// ---- host ---------------------------------------------------------------

constexpr int32_t kMostRows = 1 << 24;

uint64_t round16(uint64_t n) { return (n + 15) / 16 * 16; }

uint64_t workspace_need(const lmkv_pool_t* pool, int32_t rows) {
    const uint64_t blocks = (uint64_t)pool->num_blocks, moves = blocks > (uint64_t)rows ? blocks : (uint64_t)rows;
    return 16 + 3 * round16(blocks * 4) + round16((uint64_t)rows * 4) + round16(moves * sizeof(Move));
}

// What the calls check alike; fills what they have in common.
int begin(const lmkv_pool_t* pool, const int32_t* table, int32_t max_blocks, const int32_t* kv_len, int32_t rows,
          int32_t rows_out, const int32_t* refs, int32_t* table_out, int32_t* refs_out, void* workspace,
          uint64_t workspace_bytes, int32_t* d_status, PagesParams* p) {
    const int rc = lmkv_internal_check_pool(pool);
    if (rc != LMKV_OK) return rc;
    if (pool->num_blocks > kMostPages) return LMKV_ERR_UNSUPPORTED;
    if (rows < 0 || rows_out < 0 || rows > kMostRows || rows_out > kMostRows || max_blocks < 0 ||
        (int64_t)max_blocks * (rows > rows_out ? rows : rows_out) > kMostEntries ||
        refs == nullptr || refs_out == nullptr ||
        (rows > 0 && (kv_len == nullptr || (max_blocks > 0 && table == nullptr))) ||
        (rows_out > 0 && max_blocks > 0 && table_out == nullptr) || workspace == nullptr ||
        workspace_bytes < workspace_need(pool, rows_out))
        return LMKV_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(workspace) | reinterpret_cast<uintptr_t>(refs) | reinterpret_cast<uintptr_t>(refs_out)) & 15)
        return LMKV_ERR_MISALIGNED;
    *p = PagesParams{};
    p->table = table;
    p->table_out = table_out;
    p->kv_len = kv_len;
    p->refs = refs;
    p->refs_out = refs_out;
    p->status = d_status;
    p->rows = rows;
    p->rows_out = rows_out;
    p->max_blocks = max_blocks;
    p->block_size = pool->block_size;
    p->num_blocks = (int32_t)pool->num_blocks;
    uint8_t* at = static_cast<uint8_t*>(workspace);
    auto take = [&](uint64_t bytes) {
        uint8_t* const x = at;
        at += round16(bytes);
        return x;
    };
    const uint64_t ids = (uint64_t)pool->num_blocks * 4;
    p->count = reinterpret_cast<int32_t*>(take(4));
    p->owner = reinterpret_cast<int32_t*>(take(ids));
    p->list = reinterpret_cast<int32_t*>(take(ids));
    p->held = reinterpret_cast<int32_t*>(take(ids));
    p->first = reinterpret_cast<int32_t*>(take((uint64_t)rows_out * 4));
    p->moves = reinterpret_cast<Move*>(at);
    return LMKV_OK;
}

int scales_fit(const lmkv_pool_t* pool, void* const* scales) {
    return scales == nullptr || pool->elem_bytes == 1 ? LMKV_OK : LMKV_ERR_INVALID_ARG;
}

template <Call kCall>
int launch_plan(const PagesParams& p, void* stream) {
    return launch(pages_plan_kernel<kCall>, kCluster, kOne, 0, stream, kCluster, p);
}

}  // namespace

extern "C" {

int lmkv_pages_workspace_bytes(const lmkv_pool_t* pool, int32_t rows, uint64_t* bytes) {
    const int rc = lmkv_internal_check_pool(pool);
    if (rc != LMKV_OK) return rc;
    if (pool->num_blocks > kMostPages) return LMKV_ERR_UNSUPPORTED;
    if (bytes == nullptr || rows < 0 || rows > kMostRows) return LMKV_ERR_INVALID_ARG;
    *bytes = workspace_need(pool, rows);
    return LMKV_OK;
}

int lmkv_copy_pages(const lmkv_pool_t* pool, void* const* scales, const int32_t* src, const int32_t* dst, int32_t n,
                    int32_t* d_status, void* stream) {
    int rc = lmkv_internal_check_pool(pool);
    if (rc == LMKV_OK) rc = scales_fit(pool, scales);
    if (rc != LMKV_OK) return rc;
    if (n < 0 || (n > 0 && (src == nullptr || dst == nullptr))) return LMKV_ERR_INVALID_ARG;
    if (n == 0) return LMKV_OK;
    return launch_copy(pool, scales, src, dst, nullptr, nullptr, n, d_status, stream);
}

int lmkv_fork_pages(const lmkv_pool_t* pool, void* const* scales, const int32_t* block_table, int32_t max_blocks,
                    const int32_t* kv_len, int32_t rows, const int32_t* parents, int32_t rows_out, const int32_t* refs,
                    int32_t* table_out, int32_t* len_out, int32_t* refs_out, void* workspace, uint64_t workspace_bytes,
                    int32_t* d_status, void* stream) {
    PagesParams p;
    int rc = begin(pool, block_table, max_blocks, kv_len, rows, rows_out, refs, table_out, refs_out, workspace,
                   workspace_bytes, d_status, &p);
    if (rc == LMKV_OK) rc = scales_fit(pool, scales);
    if (rc != LMKV_OK) return rc;
    if ((rows_out > 0 && (parents == nullptr || len_out == nullptr || len_out == kv_len)) ||
        (table_out == block_table && rows > 0 && rows_out > 0 && max_blocks > 0))
        return LMKV_ERR_INVALID_ARG;
    p.parents = parents;
    p.len_out = len_out;
    rc = launch_plan<Call::kFork>(p, stream);
    if (rc == LMKV_OK && rows_out > 0) rc = launch_copy(pool, scales, nullptr, nullptr, p.moves, p.count, rows_out, d_status, stream);
    return rc;
}

int lmkv_resize_pages(const lmkv_pool_t* pool, const int32_t* block_table, int32_t max_blocks, const int32_t* kv_len,
                      const int32_t* new_len, int32_t rows, const int32_t* refs, int32_t* table_out, int32_t* refs_out,
                      void* workspace, uint64_t workspace_bytes, int32_t* d_status, void* stream) {
    PagesParams p;
    int rc = begin(pool, block_table, max_blocks, kv_len, rows, rows, refs, table_out, refs_out, workspace, workspace_bytes,
                   d_status, &p);
    if (rc != LMKV_OK) return rc;
    if (rows > 0 && new_len == nullptr) return LMKV_ERR_INVALID_ARG;
    p.new_len = new_len;
    return launch_plan<Call::kResize>(p, stream);
}

int lmkv_compact_pages(const lmkv_pool_t* pool, void* const* scales, const int32_t* block_table, int32_t max_blocks,
                       const int32_t* kv_len, int32_t rows, const int32_t* refs, int32_t* table_out, int32_t* refs_out,
                       int32_t* page_map, void* workspace, uint64_t workspace_bytes, int32_t* d_status, void* stream) {
    PagesParams p;
    int rc = begin(pool, block_table, max_blocks, kv_len, rows, rows, refs, table_out, refs_out, workspace, workspace_bytes,
                   d_status, &p);
    if (rc == LMKV_OK) rc = scales_fit(pool, scales);
    if (rc != LMKV_OK) return rc;
    if (page_map == nullptr) return LMKV_ERR_INVALID_ARG;
    p.page_map = page_map;
    rc = launch_plan<Call::kCompact>(p, stream);
    if (rc == LMKV_OK)
        rc = launch_copy(pool, scales, nullptr, nullptr, p.moves, p.count, pool->num_blocks / 2, d_status, stream);
    return rc;
}

}  // extern "C"
