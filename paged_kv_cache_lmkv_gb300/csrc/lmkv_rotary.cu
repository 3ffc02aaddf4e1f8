// lmkv_rotary.cu -- rotary set-up (host) and the append of new tokens to the
// pages of one layer.
#include "lmkv_rotary.cuh"

#include <cmath>

namespace lmkv_rotary_detail {

int make_rotary(const lmkv_rotary_t* in, int32_t head_dim, Rotary* out) {
    if (in == nullptr || in->rot_dim < 2 || in->rot_dim % 2 != 0 || in->rot_dim > head_dim ||
        in->rot_dim > 2 * LMKV_ROTARY_MAX_PAIRS || !std::isfinite(in->magnitude))
        return LMKV_ERR_INVALID_ARG;
    out->half = in->rot_dim / 2;
    out->interleaved = in->interleaved != 0;
    out->magnitude = (float)in->magnitude;
    for (int i = 0; i < LMKV_ROTARY_MAX_PAIRS; ++i) {
        out->turns[i] = 0;
        if (i >= out->half) continue;
        if (!std::isfinite(in->inv_freq[i])) return LMKV_ERR_INVALID_ARG;
        double t = in->inv_freq[i] * 0.15915494309189533577;    // 1 / 2 pi
        t -= std::floor(t);                                     // whole turns change nothing
        const double scaled = std::nearbyint(t * 18446744073709551616.0);     // 2^64
        out->turns[i] = scaled >= 18446744073709551616.0 ? 0 : (uint64_t)scaled;
    }
    return LMKV_OK;
}

}  // namespace lmkv_rotary_detail

namespace {

using namespace lmkv_paged;
using namespace lmkv_rotary_detail;

struct Rows {
    void* data;
    int64_t token_stride;
    int64_t head_stride;
    static Rows of(const lmkv_rows_t* x) { return Rows{x->data, x->token_stride, x->head_stride}; }
};

struct AppendParams {
    Layer layer;
    Seqs seqs;
    Rows q, k, v, q_out;
    const int64_t* positions;
    int32_t* status;
    int32_t q_heads, kv_heads, head_dim;
    FastDiv by_units, by_copies;       // units of a rotated head, vectors of a copied one
    Rotary rot;
};

constexpr int kThreads = 128;
constexpr int kAhead = 4;      // units of a thread on their way together

// A CTA per token.  Its rows need no look-up, so their first units are on
// their way while warp 0 finds the token's request, position and page row and
// the (cos, sin) of every pair, one for all heads, go to shared memory.  Bound
// by the rows' bytes: q read and written, k and v read and written into the
// pages.  (Two, four and eight tokens a CTA, whose loads wait for one
// another's look-ups, took 24-44% longer on 8948 tokens of 80 heads: 59 us, 6.2 TB/s,
// 0.92 of the copy rate.)
template <class T, int V, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendParams p) {
    using U = Units<T, V, kInterleaved>;
    __shared__ float2 cs[LMKV_ROTARY_MAX_PAIRS];
    __shared__ int64_t page_off, position;
    __shared__ int32_t live;
    pdl_launch_dependents();
    pdl_wait();
    const int32_t t = blockIdx.x;
    const int half = p.rot.half;
    const int units = U::count(half, p.head_dim), copies = p.head_dim / V;
    const int rotated = (p.q_heads + p.kv_heads) * units;
    const int slots = rotated + p.kv_heads * copies;
    uint8_t* const base = p.layer.base();

    // slot -> (q, k or v; head; unit)
    struct Slot {
        int what, h, u;
    };
    auto slot_of = [&](int i) {
        Slot s;
        if (i < rotated) {
            s.h = (int)p.by_units.div((uint32_t)i);
            s.u = i - s.h * units;
            s.what = s.h < p.q_heads ? 0 : 1;
            if (s.what) s.h -= p.q_heads;
        } else {
            s.what = 2;
            s.h = (int)p.by_copies.div((uint32_t)(i - rotated));
            s.u = i - rotated - s.h * copies;
        }
        return s;
    };
    U x[kAhead];
    auto load = [&](int i0) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = i0 + k * kThreads;
            if (i >= slots) break;
            const Slot s = slot_of(i);
            const Rows& in = s.what == 0 ? p.q : s.what == 1 ? p.k : p.v;
            const T* src = static_cast<const T*>(in.data) + (int64_t)t * in.token_stride + (int64_t)s.h * in.head_stride;
            if (s.what < 2) x[k].load(src, s.u, half);
            else x[k].a = ld_vec<T, V, false>(src + s.u * V);
        }
    };
    load(threadIdx.x);
    if (threadIdx.x < 32) {
        const int32_t r = find_request(p.seqs.num_req, t, [&](int32_t i) { return p.seqs.q_start[i]; });
        if (threadIdx.x == 0) {
            int64_t off = -1, pos = 0;
            int32_t on = 0;
            const Req q = load_req(p.seqs, r);
            const int32_t end = min(max(p.seqs.q_start[r + 1], q.q0), p.seqs.num_tokens);
            if (t >= q.q0 && t < end) {
                on = 1;
                const int32_t index = q.len - (end - q.q0) + (t - q.q0);
                pos = p.positions != nullptr ? p.positions[t] : (int64_t)index;
                const bool whole = q.len == p.seqs.kv_len[r] && q.q0 == p.seqs.q_start[r] && end == p.seqs.q_start[r + 1];
                if (base == nullptr) {
                    report(p.status, LMKV_ERR_BAD_POINTER);
                } else if (!whole || index < 0) {
                    // a clamped length says nothing about where the tokens go
                    report(p.status, LMKV_ERR_BAD_LENGTH);
                } else {
                    off = p.layer.token_offset(p.seqs.table + (int64_t)r * p.seqs.table_stride, index);
                    if (off < 0) report(p.status, LMKV_ERR_BAD_BLOCK);
                }
            }
            page_off = off;
            position = pos;
            live = on;
        }
    }
    __syncthreads();
    if (!live) return;                 // a padded row
    for (int i = threadIdx.x; i < half; i += kThreads) {
        const float2 w = cos_sin<T>(p.rot.turns[i], position);
        cs[U::place(i, half)] = make_float2(w.x * p.rot.magnitude, w.y * p.rot.magnitude);
    }
    __syncthreads();
    uint8_t* const page = page_off < 0 ? nullptr : base + page_off;
    for (int i0 = threadIdx.x; i0 < slots; i0 += kThreads * kAhead) {
        if (i0 >= kThreads) load(i0);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = i0 + k * kThreads;
            if (i >= slots) break;
            const Slot s = slot_of(i);
            if (s.what == 0) {
                x[k].turn(cs, s.u, half);
                x[k].store(static_cast<T*>(p.q_out.data) + (int64_t)t * p.q_out.token_stride +
                               (int64_t)s.h * p.q_out.head_stride, s.u, half);
            } else if (page != nullptr) {
                T* const out = reinterpret_cast<T*>(page) + (int64_t)s.h * p.head_dim;
                if (s.what == 1) {
                    x[k].turn(cs, s.u, half);
                    x[k].store(out, s.u, half);
                } else {
                    st_vec<T, V, false>(reinterpret_cast<T*>(page + p.layer.half_bytes()) + (int64_t)s.h * p.head_dim +
                                            s.u * V, x[k].a);
                }
            }
        }
    }
}

template <class T, int V, bool kInterleaved>
int launch_append(AppendParams& p, void* stream) {
    p.by_units = FastDiv((uint32_t)Units<T, V, kInterleaved>::count(p.rot.half, p.head_dim));
    p.by_copies = FastDiv((uint32_t)(p.head_dim / V));
    return launch(append_kernel<T, V, kInterleaved>, p.seqs.num_tokens, kThreads, 0, stream, 1, p);
}

template <class T>
int append_typed(AppendParams& p, bool vector, void* stream) {
    constexpr int V = 16 / sizeof(T);
    if (p.rot.interleaved)
        return vector ? launch_append<T, V, true>(p, stream) : launch_append<T, 1, true>(p, stream);
    return vector ? launch_append<T, V, false>(p, stream) : launch_append<T, 1, false>(p, stream);
}

bool finite_all(double a, double b, double c, double d, double e) {
    return std::isfinite(a) && std::isfinite(b) && std::isfinite(c) && std::isfinite(d) && std::isfinite(e);
}

}  // namespace

extern "C" {

int lmkv_rotary_init(lmkv_rotary_t* out, int32_t rot_dim, int32_t interleaved, double base, int32_t scaling,
                     double factor, double low, double high, double original) {
    const double two_pi = 6.283185307179586477;
    if (out == nullptr || rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > 2 * LMKV_ROTARY_MAX_PAIRS ||
        !finite_all(base, factor, low, high, original) || !(base > 1.0) || !(factor >= 1.0))
        return LMKV_ERR_INVALID_ARG;
    if (scaling < LMKV_ROTARY_PLAIN || scaling > LMKV_ROTARY_YARN) return LMKV_ERR_INVALID_ARG;
    const bool ramp = scaling == LMKV_ROTARY_RAMP || scaling == LMKV_ROTARY_YARN;
    if ((scaling == LMKV_ROTARY_BANDS || ramp) && (!(low > 0.0) || !(low < high) || !(original > 0.0)))
        return LMKV_ERR_INVALID_ARG;
    if (scaling == LMKV_ROTARY_BASE) {
        if (rot_dim <= 2) return LMKV_ERR_INVALID_ARG;
        base *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
        if (!std::isfinite(base)) return LMKV_ERR_INVALID_ARG;
    }
    lmkv_rotary_t r = {};
    r.rot_dim = rot_dim;
    r.interleaved = interleaved != 0;
    r.magnitude = ramp ? 0.1 * std::log(factor) + 1.0 : 1.0;
    // the (fractional) pair that makes n turns over `original` positions
    auto pair_of = [&](double n) { return rot_dim * std::log(original / (n * two_pi)) / (2.0 * std::log(base)); };
    double first = 0.0, last = 0.0;      // ends of the ramp
    if (ramp) {
        first = pair_of(high);
        last = pair_of(low);             // > first
        if (scaling == LMKV_ROTARY_YARN) {
            first = std::fmax(std::floor(first), 0.0);
            last = std::fmin(std::ceil(last), rot_dim - 1.0);
            if (last < first) return LMKV_ERR_INVALID_ARG;
            if (last == first) last += 0.001;
        }
    }
    for (int i = 0; i < rot_dim / 2; ++i) {
        const double f = std::pow(base, -2.0 * i / rot_dim);
        double keep = 1.0;      // share of the unscaled frequency
        if (scaling == LMKV_ROTARY_LINEAR) {
            keep = 0.0;
        } else if (scaling == LMKV_ROTARY_BANDS) {
            keep = (original * f / two_pi - low) / (high - low);
        } else if (ramp) {
            keep = 1.0 - (i - first) / (last - first);
        }
        keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
        r.inv_freq[i] = f * keep + f / factor * (1.0 - keep);
    }
    *out = r;
    return LMKV_OK;
}

int lmkv_append_layer(const lmkv_pool_t* pool, int32_t dtype, int32_t layer, const lmkv_batch_t* batch,
                      int32_t num_q_heads, const lmkv_rows_t* q, const lmkv_rows_t* k, const lmkv_rows_t* v,
                      const lmkv_rows_t* q_out, const int64_t* positions, const lmkv_rotary_t* rotary,
                      int32_t* d_status, void* stream) {
    int rc = lmkv_internal_check_pool(pool);
    if (rc != LMKV_OK) return rc;
    if (!type_fits(pool, dtype)) return LMKV_ERR_UNSUPPORTED;
    if (layer < 0 || layer >= pool->num_layers) return LMKV_ERR_INVALID_ARG;
    rc = check_batch(pool, batch, num_q_heads);
    if (rc != LMKV_OK) return rc;
    AppendParams p = {};
    rc = make_rotary(rotary, pool->head_dim, &p.rot);
    if (rc != LMKV_OK) return rc;
    if (batch->num_req == 0 || batch->num_tokens == 0) return LMKV_OK;
    const int32_t e = pool->elem_bytes;
    if (!rows_ok(q, e) || !rows_ok(k, e) || !rows_ok(v, e) || !rows_ok(q_out, e)) return LMKV_ERR_INVALID_ARG;
    p.layer = Layer::of(pool, layer);
    p.seqs = Seqs::of(batch);
    p.q = Rows::of(q);
    p.k = Rows::of(k);
    p.v = Rows::of(v);
    p.q_out = Rows::of(q_out);
    p.positions = positions;
    p.status = d_status;
    p.q_heads = num_q_heads;
    p.kv_heads = pool->num_kv_heads;
    p.head_dim = pool->head_dim;
    // 16-byte vectors where every row starts on 16 bytes and they divide a head
    bool vector = vector_fits(p.rot.half, p.rot.interleaved, p.head_dim, e);
    for (const lmkv_rows_t* x : {q, k, v, q_out})
        vector = vector && reinterpret_cast<uintptr_t>(x->data) % 16 == 0 && x->token_stride * e % 16 == 0 &&
                 x->head_stride * e % 16 == 0;
    if (dtype == LMKV_BF16) return append_typed<__nv_bfloat16>(p, vector, stream);
    if (dtype == LMKV_FP16) return append_typed<__half>(p, vector, stream);
    return append_typed<float>(p, vector, stream);
}

}  // extern "C"
