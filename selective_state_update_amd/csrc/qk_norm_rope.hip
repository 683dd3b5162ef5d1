// qk_norm_rope.hip -- norms of queries and keys for each head with the position
// rotation, optionally into a paged key-value cache, on MI355X (gfx950):
// ssu_qk_norm_rope. The operation is stated in include/ssu.h.

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "host_checks.h"
#include "internal.h"
#include "seq_common.h"

namespace ssu {
namespace {

constexpr int kMaxHeaddim = 512;

struct QkParams {
    const uint16_t *q, *k, *v;
    int64_t q_t, q_h, k_t, k_h, v_t, v_h;
    const void *q_weight, *k_weight;  // fp32 or the 16-bit type; NULL: 1
    const void *positions, *slots;
    const float *cos_sin;
    int64_t cs_row;
    uint16_t *q_out, *k_out, *k_cache, *v_cache;
    int64_t qo_t, qo_h, ko_t, ko_h;
    int64_t kc_page, kc_row, kc_h, vc_page, vc_row, vc_h;
    int64_t ntokens, max_pos, num_slots, total;  // total: head rows
    int32_t nq, nk, rows_per_token, headdim, rot, interleaved, page_size;
    int32_t pos64, slot64, qw32, kw32;
    int32_t q_groups, k_groups, groups_per_token;  // of kRows heads
    float eps;
};

template <typename T>
__device__ __forceinline__ float weight_at(const void *w, int is32, int i)
{
    if (!w)
        return 1.0f;
    return is32 ? static_cast<const float *>(w)[i] : T::lo(static_cast<const uint16_t *>(w)[i]);
}

// One wave per head row (a token's query, key and, with a cache, value heads),
// lane l holding elements l, l + 64, ... and, for the rotation, their pairs'
// other elements. Any headdim and rotation width: it takes the headdims that the
// kernel below does not, and few rows of a width that is no multiple of 8 (16 tokens
// of 32 + 8 heads of 128 into a cache, rot 94: 4.2 against 5.2 us; 128 tokens 5.8
// against 5.5, 4096 tokens 119 against 41).
template <typename T>
__global__ void __launch_bounds__(256) ssu_qk_rows_kernel(const QkParams p)
{
    constexpr int M = kMaxHeaddim / 64;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    const int lane = static_cast<int>(threadIdx.x) & 63;
    if (row >= p.total)
        return;
    const int64_t t = row / p.rows_per_token;
    const int r = static_cast<int>(row - t * p.rows_per_token);
    const int64_t pos = load_index(p.positions, p.pos64, t);
    if (pos < 0 || pos >= p.max_pos)
        return;  // padding
    const bool is_q = r < p.nq, is_v = r >= p.nq + p.nk;
    const int h = is_q ? r : is_v ? r - p.nq - p.nk : r - p.nq;
    uint16_t *cache = nullptr;
    if (!is_q && p.k_cache) {
        const int64_t slot = load_index(p.slots, p.slot64, t);
        if (slot >= 0 && slot < p.num_slots) {
            const int64_t page = slot / p.page_size, off = slot - page * p.page_size;
            cache = is_v ? p.v_cache + page * p.vc_page + off * p.vc_row + h * p.vc_h
                         : p.k_cache + page * p.kc_page + off * p.kc_row + h * p.kc_h;
        }
    }
    if (is_v) {
        const uint16_t *const x = p.v + t * p.v_t + h * p.v_h;
        if (cache)
            for (int i = lane; i < p.headdim; i += 64)
                cache[i] = x[i];
        return;
    }
    const uint16_t *const x = is_q ? p.q + t * p.q_t + h * p.q_h : p.k + t * p.k_t + h * p.k_h;
    const void *const w = is_q ? p.q_weight : p.k_weight;
    const int w32 = is_q ? p.qw32 : p.kw32, half = p.rot / 2;
    const float *const cs = p.cos_sin + pos * p.cs_row;
    float own[M], other[M], c[M], s[M], sum = 0.0f;
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const int i = lane + 64 * m;
        own[m] = other[m] = s[m] = 0.0f;
        c[m] = 1.0f;
        if (i < p.headdim) {
            own[m] = T::lo(x[i]);
            sum = fmaf(own[m], own[m], sum);
            own[m] *= weight_at<T>(w, w32, i);
            if (i < p.rot) {
                const int pair = p.interleaved ? i >> 1 : i < half ? i : i - half;
                const bool first = p.interleaved ? !(i & 1) : i < half;
                const int j = p.interleaved ? i ^ 1 : first ? i + half : i - half;
                other[m] = T::lo(x[j]) * weight_at<T>(w, w32, j);
                c[m] = cs[pair];
                s[m] = first ? -cs[half + pair] : cs[half + pair];
            }
        }
    }
#pragma unroll
    for (int m = 32; m >= 1; m /= 2)
        sum += __shfl_xor(sum, m);
    const float scale = 1.0f / sqrtf(sum / static_cast<float>(p.headdim) + p.eps);
    uint16_t y[M];
#pragma unroll
    for (int m = 0; m < M; ++m)
        y[m] = T::round((own[m] * c[m] + other[m] * s[m]) * scale);
    // in place: every element has been read before the first is written
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    uint16_t *const out = is_q ? p.q_out + t * p.qo_t + h * p.qo_h : p.k_out ? p.k_out + t * p.ko_t + h * p.ko_h : nullptr;
#pragma unroll
    for (int m = 0; m < M; ++m)
        if (lane + 64 * m < p.headdim) {
            if (out)
                out[lane + 64 * m] = y[m];
            if (cache)
                cache[lane + 64 * m] = y[m];
        }
}

constexpr int kRows = 4;  // heads of a token per group of lanes

// Which elements of a row a lane has, as two runs of up to four.
enum class Runs {
    halves,       // both elements of pairs (i, i + rot/2); rot a multiple of 8
    halves_edge,  // the same, any rot
    inter,        // pairs (2i, 2i + 1); rot a multiple of 8
    inter_edge,   // the same, any rot
};

// n elements of a row of d from `at` on, zeros behind them. EDGE: n < 4 or none;
// the four elements read lie in the row.
template <bool EDGE, bool STREAM>
__device__ __forceinline__ u32x2 load_run(const uint16_t *row, int at, int n, int d)
{
    const int from = EDGE ? min(at, d - 4) : at;
    const u32x2_a2 *const p = reinterpret_cast<const u32x2_a2 *>(row + from);
    u32x2 x;
    if constexpr (STREAM)
        x = __builtin_nontemporal_load(p);
    else
        x = *p;
    if constexpr (EDGE) {
        const uint64_t y = (static_cast<uint64_t>(x[1]) << 32 | x[0]) >> 16 * min(at - from, 3);
        const uint64_t kept = n <= 0 ? 0 : ~uint64_t(0) >> 16 * (4 - min(n, 4));
        x = u32x2{static_cast<uint32_t>(y & kept), static_cast<uint32_t>((y & kept) >> 32)};
    }
    return x;
}

template <bool EDGE>
__device__ __forceinline__ void store_run(uint16_t *p, int n, uint32_t x, uint32_t y)
{
    if (!EDGE || n == 4) {
        __builtin_nontemporal_store(u32x2{x, y}, reinterpret_cast<u32x2_a2 *>(p));
        return;
    }
    if (n > 0)
        p[0] = static_cast<uint16_t>(x);
    if (n > 1)
        p[1] = static_cast<uint16_t>(x >> 16);
    if (n > 2)
        p[2] = static_cast<uint16_t>(y);
}

// A lane's two runs of a row.
template <Runs RUNS>
__device__ __forceinline__ u32x4 load_runs(const uint16_t *p, int at, int n, int at2, int n2, int d)
{
    if constexpr (RUNS == Runs::inter || RUNS == Runs::inter_edge) {
        return __builtin_nontemporal_load(reinterpret_cast<const u32x4_a2 *>(p + at));
    } else {
        constexpr bool EDGE = RUNS == Runs::halves_edge;
        const u32x2 x = load_run<EDGE, true>(p, at, n, d), y = load_run<EDGE, true>(p, at2, n2, d);
        return u32x4{x[0], x[1], y[0], y[1]};
    }
}

template <Runs RUNS>
__device__ __forceinline__ void store_runs(uint16_t *p, int at, int n, int at2, int n2, u32x4 v)
{
    if constexpr (RUNS == Runs::inter || RUNS == Runs::inter_edge) {
        __builtin_nontemporal_store(v, reinterpret_cast<u32x4_a2 *>(p + at));
    } else {
        store_run<RUNS == Runs::halves_edge>(p + at, n, v[0], v[1]);
        store_run<RUNS == Runs::halves_edge>(p + at2, n2, v[2], v[3]);
    }
}

// Four values from element i on; PART: the last of `count` for what lies behind it.
template <bool PART>
__device__ __forceinline__ f32x4 load_floats(const float *p, int i, int count)
{
    if constexpr (PART)
        return f32x4{p[min(i, count - 1)], p[min(i + 1, count - 1)], p[min(i + 2, count - 1)], p[min(i + 3, count - 1)]};
    else
        return *reinterpret_cast<const f32x4_a4 *>(p + i);
}

// The weights of a run.
template <typename T, bool EDGE>
__device__ __forceinline__ f32x4 weights_at(const void *w, int is32, int i, int n, int d)
{
    if (!w)
        return f32x4{1.0f, 1.0f, 1.0f, 1.0f};
    if (is32)
        return load_floats<EDGE>(static_cast<const float *>(w), i, d);
    const u32x2 x = load_run<EDGE, false>(static_cast<const uint16_t *>(w), i, n, d);
    return f32x4{T::lo(x[0]), T::hi(x[0]), T::lo(x[1]), T::hi(x[1])};
}

// Rows of 16-byte runs: headdim a multiple of 8. LANES lanes take one head row, a
// lane 8 of its elements as two runs of 4: both elements of 4 pairs (runs at 4 l and
// rot / 2 + 4 l, or 8 consecutive elements when interleaved), or 8 elements behind the
// rotated part; at the end of either part fewer (halves_edge). So nothing is
// exchanged but the sum of squares. A group of lanes takes kRows heads of one token,
// all q, all k or all v, with the weights and the token's cosines and sines read once
// and the rows' loads on their way together: memory-bound, each element is read and
// written once, past the caches (16384 tokens of 32 + 8 heads of 128: 60 us, 5.6 TB/s;
// with cached accesses 69 us).
template <typename T, Runs RUNS, int LANES>
__global__ void __launch_bounds__(256) ssu_qk_groups_kernel(const QkParams p)
{
    constexpr bool INTER = RUNS == Runs::inter || RUNS == Runs::inter_edge, EDGE = RUNS == Runs::halves_edge;
    constexpr bool PART = EDGE || RUNS == Runs::inter_edge;  // a lane may have fewer than four pairs
    const uint32_t group = blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
    const int l = static_cast<int>(threadIdx.x) % LANES;
    const uint32_t t = group / static_cast<uint32_t>(p.groups_per_token);
    int j = static_cast<int>(group - t * static_cast<uint32_t>(p.groups_per_token));
    if (static_cast<int64_t>(t) >= p.ntokens)
        return;
    const int64_t pos = load_index(p.positions, p.pos64, t);
    if (pos < 0 || pos >= p.max_pos)
        return;  // padding
    const bool is_q = j < p.q_groups, is_v = j >= p.q_groups + p.k_groups;
    j -= is_q ? 0 : is_v ? p.q_groups + p.k_groups : p.q_groups;
    const int h0 = j * kRows, heads = min((is_q ? p.nq : p.nk) - h0, kRows);
    const uint16_t *x = is_q ? p.q + t * p.q_t + h0 * p.q_h : is_v ? p.v + t * p.v_t + h0 * p.v_h : p.k + t * p.k_t + h0 * p.k_h;
    const int64_t x_h = is_q ? p.q_h : is_v ? p.v_h : p.k_h;

    const int half = p.rot / 2, pairs = (half + 3) / 4;  // lanes with pairs in halves
    const bool turned = EDGE ? l < pairs : 8 * l < p.rot;
    const int at = INTER || (!EDGE && !turned) ? 8 * l : turned ? 4 * l : p.rot + 8 * (l - pairs);
    const int at2 = !INTER && turned ? half + 4 * l : at + 4;
    const int n = EDGE && turned ? min(half - at, 4) : min(p.headdim - at, 4), n2 = EDGE && turned ? n : min(p.headdim - at2, 4);
    const bool in = EDGE ? n > 0 : 8 * l < p.headdim;
    u32x4 v[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
        v[i] = in && i < heads ? load_runs<RUNS>(x + i * x_h, at, n, at2, n2, p.headdim) : u32x4{0, 0, 0, 0};

    uint16_t *cache = nullptr;
    int64_t c_h = 0;
    if (!is_q && p.k_cache) {
        const int64_t slot = load_index(p.slots, p.slot64, t);
        if (slot >= 0 && slot < p.num_slots) {
            const int64_t page = slot / p.page_size, off = slot - page * p.page_size;
            c_h = is_v ? p.vc_h : p.kc_h;
            cache = (is_v ? p.v_cache + page * p.vc_page + off * p.vc_row : p.k_cache + page * p.kc_page + off * p.kc_row) + h0 * c_h;
        }
    }
    uint16_t *out = is_q ? p.q_out + t * p.qo_t + h0 * p.qo_h : is_v || !p.k_out ? nullptr : p.k_out + t * p.ko_t + h0 * p.ko_h;
    const int64_t o_h = is_q ? p.qo_h : p.ko_h;

    if (!is_v) {
        const void *const w = is_q ? p.q_weight : p.k_weight;
        const int w32 = is_q ? p.qw32 : p.kw32;
        f32x4 wa = {0.0f, 0.0f, 0.0f, 0.0f}, wb = wa, c = wa, s = wa;
        if (in) {
            wa = weights_at<T, EDGE>(w, w32, at, n, p.headdim);
            wb = weights_at<T, EDGE>(w, w32, at2, n2, p.headdim);
        }
        const int m = half - 4 * l;  // this lane's pairs, from 4 l on, or more
        if (turned) {
            const float *const cs = p.cos_sin + pos * p.cs_row;
            c = load_floats<PART>(cs, 4 * l, half);
            s = load_floats<PART>(cs + half, 4 * l, half);
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            float a[4], b[4], sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                a[2 * e] = T::lo(v[i][e]);
                a[2 * e + 1] = T::hi(v[i][e]);
                b[2 * e] = T::lo(v[i][2 + e]);
                b[2 * e + 1] = T::hi(v[i][2 + e]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sum = fmaf(a[e], a[e], sum);
                sum = fmaf(b[e], b[e], sum);
            }
            const float scale = rsqrtf(sum_lanes<LANES>(sum) / static_cast<float>(p.headdim) + p.eps);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                a[e] *= wa[e] * scale;
                b[e] *= wb[e] * scale;
            }
            // the pairs: (a[e], b[e]), or neighbours when interleaved; the others are
            // left out, since a zero sine would carry infinities over
            if (turned) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float &first = INTER ? (e < 2 ? a[2 * e % 4] : b[2 * e % 4]) : a[e];
                    float &second = INTER ? (e < 2 ? a[2 * e % 4 + 1] : b[2 * e % 4 + 1]) : b[e];
                    const float u = first * c[e] - second * s[e], w = second * c[e] + first * s[e];
                    first = !PART || e < m ? u : first;
                    second = !PART || e < m ? w : second;
                }
            }
            v[i] = u32x4{pack2<T>(a[0], a[1]), pack2<T>(a[2], a[3]), pack2<T>(b[0], b[1]), pack2<T>(b[2], b[3])};
        }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i)
        if (in && i < heads) {
            if (out)
                store_runs<RUNS>(out + i * o_h, at, n, at2, n2, v[i]);
            if (cache)
                store_runs<RUNS>(cache + i * c_h, at, n, at2, n2, v[i]);
        }
}

using QkFn = void (*)(QkParams);

template <typename T, Runs RUNS>
QkFn groups_kernel(int lanes)
{
    if constexpr (RUNS != Runs::halves_edge)  // (a lane for each part at least)
        if (lanes == 1)
            return &ssu_qk_groups_kernel<T, RUNS, 1>;
    switch (lanes) {
    case 2: return &ssu_qk_groups_kernel<T, RUNS, 2>;
    case 4: return &ssu_qk_groups_kernel<T, RUNS, 4>;
    case 8: return &ssu_qk_groups_kernel<T, RUNS, 8>;
    case 16: return &ssu_qk_groups_kernel<T, RUNS, 16>;
    case 32: return &ssu_qk_groups_kernel<T, RUNS, 32>;
    default: return &ssu_qk_groups_kernel<T, RUNS, 64>;
    }
}

template <typename T>
QkFn groups_kernel(Runs runs, int lanes)
{
    return runs == Runs::inter ? groups_kernel<T, Runs::inter>(lanes)
         : runs == Runs::inter_edge ? groups_kernel<T, Runs::inter_edge>(lanes)
         : runs == Runs::halves ? groups_kernel<T, Runs::halves>(lanes) : groups_kernel<T, Runs::halves_edge>(lanes);
}

// ------------------------------------------------------------------ host --

ssu_status check_qk(const ssu_qk_args &a)
{
    const char *const who = "ssu_qk_norm_rope";
    if (a.ntokens < 0 || a.nq < 0 || a.nk < 0 || a.max_pos < 0 || a.num_pages < 0)
        return fail(SSU_ERR_INVALID_ARGUMENT, "%s: negative size", who);
    if (a.headdim < 1 || a.rot < 0 || a.rot > a.headdim || a.rot % 2)
        return fail(SSU_ERR_INVALID_ARGUMENT, "%s: headdim %d, rot %d: rot must be even, at most headdim", who,
                    a.headdim, a.rot);
    if (a.headdim > kMaxHeaddim)
        return fail(SSU_ERR_UNSUPPORTED, "%s: headdim %d > %d", who, a.headdim, kMaxHeaddim);
    if (a.interleaved != 0 && a.interleaved != 1)
        return fail(SSU_ERR_INVALID_ARGUMENT, "%s: interleaved must be 0 or 1", who);
    if (!(a.eps >= 0.0f) || !std::isfinite(a.eps))
        return fail(SSU_ERR_INVALID_ARGUMENT, "%s: eps must be finite and >= 0", who);
    const bool cache = a.k_cache.ptr || a.v_cache.ptr || a.slots.ptr || a.v.ptr;
    const int32_t type = a.nq > 0 ? a.q.dtype : a.k.dtype;
    if (type != SSU_BF16 && type != SSU_F16)
        return fail(SSU_ERR_INVALID_ARGUMENT, "%s: q and k must be BF16 or F16", who);
    if (a.ntokens == 0 || a.nq + a.nk == 0)
        return SSU_OK;
    const bool nq = a.nq == 0, nk = a.nk == 0;
    SSU_TRY(check_view(a.q, "q", type, 3, nq));
    SSU_TRY(check_view(a.q_out, "q_out", type, 3, nq));
    SSU_TRY(check_view(a.k, "k", type, 3, nk));
    SSU_TRY(check_view(a.k_out, "k_out", type, 3, nk || cache));
    SSU_TRY(check_view(a.positions, "positions", a.positions.dtype == SSU_I64 ? SSU_I64 : SSU_I32, 1, false));
    SSU_TRY(check_view(a.cos_sin, "cos_sin", SSU_F32, 2, a.rot == 0 || a.max_pos == 0));
    for (const ssu_view *w : {&a.q_weight, &a.k_weight})
        if (w->ptr) {
            SSU_TRY(check_view(*w, "weight", w->dtype == SSU_F32 ? SSU_F32 : type, 1, true));
            if (a.headdim > 1 && w->stride[0] != 1)
                return fail(SSU_ERR_UNSUPPORTED, "weight: stride must be 1");
            if (reinterpret_cast<uintptr_t>(w->ptr) % (w->dtype == SSU_F32 ? 4 : 2))
                return fail(SSU_ERR_MISALIGNED, "weight: pointer must be aligned to its element");
        }
    if (cache) {
        if (a.page_size < 1)
            return fail(SSU_ERR_INVALID_ARGUMENT, "%s: page_size %d", who, a.page_size);
        if (a.num_pages > INT64_MAX / a.page_size)
            return fail(SSU_ERR_INVALID_ARGUMENT, "%s: num_pages * page_size too large", who);
        const bool none = nk || a.num_pages == 0;
        SSU_TRY(check_view(a.v, "v", type, 3, nk));
        SSU_TRY(check_view(a.k_cache, "k_cache", type, 4, none));
        SSU_TRY(check_view(a.v_cache, "v_cache", type, 4, none));
        SSU_TRY(check_view(a.slots, "slots", a.slots.dtype == SSU_I64 ? SSU_I64 : SSU_I32, 1, false));
        if (a.headdim > 1 && ((a.k_cache.ptr && a.k_cache.stride[3] != 1) || (a.v_cache.ptr && a.v_cache.stride[3] != 1)))
            return fail(SSU_ERR_UNSUPPORTED, "k_cache/v_cache: inner stride must be 1");
        if (a.slots.stride[0] != 1 && a.ntokens > 1)
            return fail(SSU_ERR_UNSUPPORTED, "slots: stride must be 1");
    }
    SSU_TRY(check_written(a.q_out, "q_out", {a.ntokens, a.nq}));
    SSU_TRY(check_written(a.k_out, "k_out", {a.ntokens, a.nk}));
    SSU_TRY(check_written(a.k_cache, "k_cache", {a.num_pages, a.page_size, a.nk}));
    SSU_TRY(check_written(a.v_cache, "v_cache", {a.num_pages, a.page_size, a.nk}));
    for (const ssu_view *v : {&a.q, &a.k, &a.v, &a.q_out, &a.k_out})
        if (v->ptr && a.headdim > 1 && v->stride[2] != 1)
            return fail(SSU_ERR_UNSUPPORTED, "q/k/v/outputs: inner stride must be 1");
    if (a.positions.stride[0] != 1 && a.ntokens > 1)
        return fail(SSU_ERR_UNSUPPORTED, "positions: stride must be 1");
    if (a.rot > 1 && a.cos_sin.ptr && a.cos_sin.stride[1] != 1)
        return fail(SSU_ERR_UNSUPPORTED, "cos_sin: inner stride must be 1");
    for (const ssu_view *v : {&a.q, &a.k, &a.v, &a.q_out, &a.k_out, &a.k_cache, &a.v_cache})
        if (reinterpret_cast<uintptr_t>(v->ptr) % 2)
            return fail(SSU_ERR_MISALIGNED, "16-bit operand not 2-byte aligned");
    if (reinterpret_cast<uintptr_t>(a.cos_sin.ptr) % 4)
        return fail(SSU_ERR_MISALIGNED, "cos_sin: pointer must be 4-byte aligned");
    for (const ssu_view *v : {&a.positions, &a.slots})
        if (reinterpret_cast<uintptr_t>(v->ptr) % (v->dtype == SSU_I64 ? 8 : 4))
            return fail(SSU_ERR_MISALIGNED, "positions/slots: pointer must be aligned to its element");
    return SSU_OK;
}

}  // namespace
}  // namespace ssu

extern "C" ssu_status ssu_qk_norm_rope(const ssu_qk_args *args, hipStream_t stream)
{
    using namespace ssu;
    if (!args)
        return fail(SSU_ERR_INVALID_ARGUMENT, "ssu_qk_norm_rope: null args");
    const ssu_qk_args &a = *args;
    SSU_TRY(check_qk(a));
    if (a.ntokens == 0 || a.nq + a.nk == 0 || a.max_pos == 0)
        return SSU_OK;
    QkParams p{};
    p.q = static_cast<const uint16_t *>(a.q.ptr);
    p.q_t = a.q.stride[0];
    p.q_h = a.q.stride[1];
    p.k = static_cast<const uint16_t *>(a.k.ptr);
    p.k_t = a.k.stride[0];
    p.k_h = a.k.stride[1];
    p.v = static_cast<const uint16_t *>(a.v.ptr);
    p.v_t = a.v.stride[0];
    p.v_h = a.v.stride[1];
    p.q_weight = a.q_weight.ptr;
    p.qw32 = a.q_weight.dtype == SSU_F32;
    p.k_weight = a.k_weight.ptr;
    p.kw32 = a.k_weight.dtype == SSU_F32;
    p.positions = a.positions.ptr;
    p.pos64 = a.positions.dtype == SSU_I64;
    p.slots = a.slots.ptr;
    p.slot64 = a.slots.dtype == SSU_I64;
    p.cos_sin = static_cast<const float *>(a.cos_sin.ptr);
    p.cs_row = a.cos_sin.stride[0];
    p.q_out = static_cast<uint16_t *>(const_cast<void *>(a.q_out.ptr));
    p.qo_t = a.q_out.stride[0];
    p.qo_h = a.q_out.stride[1];
    p.k_out = static_cast<uint16_t *>(const_cast<void *>(a.k_out.ptr));
    p.ko_t = a.k_out.stride[0];
    p.ko_h = a.k_out.stride[1];
    p.k_cache = static_cast<uint16_t *>(const_cast<void *>(a.k_cache.ptr));
    p.kc_page = a.k_cache.stride[0];
    p.kc_row = a.k_cache.stride[1];
    p.kc_h = a.k_cache.stride[2];
    p.v_cache = static_cast<uint16_t *>(const_cast<void *>(a.v_cache.ptr));
    p.vc_page = a.v_cache.stride[0];
    p.vc_row = a.v_cache.stride[1];
    p.vc_h = a.v_cache.stride[2];
    p.ntokens = a.ntokens;
    p.max_pos = a.max_pos;
    p.num_slots = p.k_cache ? a.num_pages * a.page_size : 0;
    p.nq = a.nq;
    p.nk = a.nk;
    const int64_t rows = static_cast<int64_t>(a.nq) + static_cast<int64_t>(a.nk) * (p.k_cache ? 2 : 1);
    if (rows > INT32_MAX - kRows || a.ntokens > INT64_MAX / rows)
        return fail(SSU_ERR_UNSUPPORTED, "ssu_qk_norm_rope: 2^31 heads or 2^63 head rows");
    p.rows_per_token = static_cast<int32_t>(rows);
    p.headdim = a.headdim;
    p.rot = a.rot;
    p.interleaved = a.interleaved;
    p.page_size = a.page_size;
    p.eps = a.eps;
    p.total = a.ntokens * p.rows_per_token;
    const bool bf16 = (a.nq > 0 ? a.q.dtype : a.k.dtype) == SSU_BF16;
    p.q_groups = (a.nq + kRows - 1) / kRows;
    p.k_groups = (a.nk + kRows - 1) / kRows;
    p.groups_per_token = p.q_groups + p.k_groups * (p.k_cache ? 2 : 1);
    const int64_t groups = a.ntokens * p.groups_per_token;
    const Runs runs = a.rot % 8 == 0 ? (a.interleaved ? Runs::inter : Runs::halves) : a.interleaved ? Runs::inter_edge : Runs::halves_edge;
    const int need = runs == Runs::halves_edge ? (a.rot / 2 + 3) / 4 + (a.headdim - a.rot + 7) / 8 : (a.headdim + 7) / 8;
    int lanes = 1;
    while (lanes < need)
        lanes *= 2;
    const bool few = a.rot % 8 != 0 && p.total <= 2048;  // (the kernel of single rows starts sooner)
    const bool grouped = a.headdim % 8 == 0 && lanes <= 64 && !few;
    const int64_t workgroups = grouped ? groups / (256 / lanes) + (groups % (256 / lanes) != 0) : p.total / 4 + (p.total % 4 != 0);
    SSU_TRY(check_launch(workgroups, 256, "ssu_qk_norm_rope"));
    DeviceGuard guard;
    SSU_TRY(guard.enter(a.device));
    const QkFn fn = !grouped ? (bf16 ? &ssu_qk_rows_kernel<Bf16> : &ssu_qk_rows_kernel<F16>)
                             : bf16 ? groups_kernel<Bf16>(runs, lanes) : groups_kernel<F16>(runs, lanes);
    const hipError_t e = launch_kernel(fn, p, workgroups, 256, 0, stream);
    if (e != hipSuccess)
        return fail(SSU_ERR_HIP, "launch of the norm and rotation kernel failed: %s", hipGetErrorString(e));
    return SSU_OK;
}
