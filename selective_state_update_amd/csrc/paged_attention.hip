// paged_attention.hip -- attention of one new token per request over a paged
// key-value cache on MI355X (gfx950): ssu_paged_attention. The operation is
// stated in include/ssu.h.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "host_checks.h"
#include "internal.h"
#include "seq_common.h"

namespace ssu {
namespace {

constexpr int kWaves = 4;
constexpr int kTile = 32;               // tokens of one wave's step
constexpr int kRound = kWaves * kTile;  // tokens of one workgroup's step
constexpr int kMaxSplits = 128;

struct AttnParams {
    const uint16_t *q, *k, *v;
    int64_t q_b, q_h, k_page, k_row, k_h, v_page, v_row, v_h;
    const int32_t *table, *lens;
    int64_t t_b, num_pages, max_pages;
    uint16_t *out;
    int64_t o_b, o_h;
    float *lse;
    int64_t l_b, l_h;
    float *part;  // [batch, splits, nq, D] partial sums, then [batch, splits, nq, 2] (maximum, sum)
    float *stat;
    int32_t batch, nq, nk, heads_per_kv, row_tiles, page_size, splits, min_rounds, total;
    float scale_log2;  // scale * log2(e): weights are powers of 2
};

// The part of a request's tokens that one split takes: `per` rounds each, the
// same for all its splits, so that a request's own length is divided evenly
// whatever the table has room for.
struct Share {
    int64_t n, begin, end;  // visible tokens at most; this split's range
    int active;             // splits that have work (at least 1)
};

__device__ __forceinline__ Share share_of(const AttnParams &p, int b, int split)
{
    Share s;
    s.n = p.lens[b];
    if (s.n >= 0)
        s.n = p.num_pages == 0 ? 0 : min(s.n, p.max_pages * p.page_size);
    const int rounds = static_cast<int>((s.n + kRound - 1) / kRound);
    const int per = max((rounds + p.splits - 1) / p.splits, p.min_rounds);
    s.active = max((rounds + per - 1) / per, 1);
    s.begin = static_cast<int64_t>(split) * per * kRound;
    s.end = min(s.n, s.begin + static_cast<int64_t>(per) * kRound);
    return s;
}

// fp16 weights are scaled by 2^14 (at most 2^14, then): what lies 2^-28 below a
// row's largest weight is still a normal number.
template <typename T>
constexpr float kShift = 0.0f;
template <>
constexpr float kShift<F16> = 14.0f;

// One workgroup per (request, split, key/value head, 16 of its query heads).
// Memory-bound: every visible K and V row is read once per 16 query heads, so
// the loads decide, and the products are arranged for them:
//
//  - S^T = K Q^T with K's rows as they lie in memory: lane l reads 16 bytes of
//    token l % 16, which is a fragment of the product; no LDS.
//  - The result has one query head per lane column, so a row's statistics are
//    one value per lane (plus two exchanges for the maximum), and the weights
//    lie exactly as the second product's fragment wants them: the lane's 4
//    tokens of two 16-token tiles are its 8 places of the contracted axis.
//  - V's rows are read whole too: 16 lanes hold 16 runs of a token's D values,
//    and a lane has its run of 8 tokens. Output column c of product m stands
//    for value c * D/16 + m, so a product's fragment is a transposition inside
//    the lane (byte permutes), and the output comes back in runs of D/16.
//
// Every wave takes every fourth 32-token step with statistics of its own; K of
// the next step is requested before the softmax of this one. PAGE16: pages
// are a multiple of 16 tokens, a tile lies in one page and its address is
// uniform; otherwise every lane looks its own token up.
template <typename T, int D, bool PAGE16>
__global__ void __launch_bounds__(64 * kWaves) ssu_attn_split_kernel(const AttnParams p)
{
    constexpr int KS = D / 32;      // products along D of a score
    constexpr int E = D / 16;       // values of a V row per lane, products of an output row
    constexpr int EW = E / 2;       // the same in words
    using V = uint32_t __attribute__((ext_vector_type(EW)));
    typedef V V_a2 __attribute__((aligned(2)));
    __shared__ float part[kWaves][16][D];
    __shared__ float stat_m[kWaves][16], stat_l[kWaves][16];

    int id = xcd_order(static_cast<int>(blockIdx.x), p.total);
    const int rt = id % p.row_tiles;
    id /= p.row_tiles;
    const int kh = id % p.nk;
    id /= p.nk;
    const int split = id % p.splits, b = id / p.splits;
    const Share sh = share_of(p, b, split);
    if (sh.n < 0 || split >= sh.active)
        return;  // padding, or a length that needs fewer splits
    const int lane = static_cast<int>(threadIdx.x) & 63, c = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int rows = min(p.heads_per_kv - rt * 16, 16);  // query heads of this workgroup
    const int h0 = kh * p.heads_per_kv + rt * 16;

    u32x4 qf[KS];
#pragma unroll
    for (int i = 0; i < KS; ++i)
        qf[i] = c < rows ? *reinterpret_cast<const u32x4_a2 *>(p.q + b * p.q_b + (h0 + c) * p.q_h + (i * 4 + g) * 8)
                         : u32x4{0, 0, 0, 0};

    const int32_t *const table = p.table + b * p.t_b;
    const uint16_t *const kbase = p.k + kh * p.k_h + g * 8, *const vbase = p.v + kh * p.v_h + c * E;

    // A tile of 16 tokens: where it is, and which of its tokens are visible.
    struct Tile {
        const uint16_t *k, *v;  // PAGE16: this lane's K row and the tile's first V row
        int page, off;          // otherwise: this lane's token
        uint32_t seen;          // uniform, a bit per token
    };
    auto locate = [&](int64_t t0) {
        Tile t;
        if constexpr (PAGE16) {
            const int64_t at = min(t0, (sh.n - 1) & ~int64_t(15));
            const int col = static_cast<int>(at) / p.page_size;
            const int64_t off = at - static_cast<int64_t>(col) * p.page_size;
            int64_t page = table[col];
            const bool good = page >= 0 && page < p.num_pages;
            page = good ? page : 0;
            const int64_t left = sh.end - t0;
            t.seen = !good || left <= 0 ? 0u : left >= 16 ? 0xffffu : (1u << left) - 1u;
            t.k = kbase + page * p.k_page + (off + c) * p.k_row;
            t.v = vbase + page * p.v_page + off * p.v_row;
        } else {
            const int at = static_cast<int>(min(t0 + c, sh.n - 1));
            const int col = at / p.page_size;
            t.off = at - col * p.page_size;
            t.page = table[col];
            const bool good = t.page >= 0 && t.page < p.num_pages;
            t.page = good ? t.page : 0;
            t.seen = static_cast<uint32_t>(__ballot(good && t0 + c < sh.end)) & 0xffffu;
            t.k = kbase + t.page * p.k_page + t.off * p.k_row;
        }
        return t;
    };
    auto load_k = [&](const Tile &t, u32x4 (&f)[KS]) {
#pragma unroll
        for (int i = 0; i < KS; ++i)
            f[i] = *reinterpret_cast<const u32x4_a2 *>(t.k + i * 32);
    };
    auto load_v = [&](const Tile &t, V *f) {  // tokens 4g .. 4g+3
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (PAGE16) {
                f[i] = *reinterpret_cast<const V_a2 *>(t.v + (4 * g + i) * p.v_row);
            } else {
                const int64_t page = __shfl(t.page, 4 * g + i), off = __shfl(t.off, 4 * g + i);
                f[i] = *reinterpret_cast<const V_a2 *>(vbase + page * p.v_page + off * p.v_row);
            }
        }
    };

    f32x4 o[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
        o[e] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    float m = -INFINITY, l = 0.0f;  // of query head c (l: this lane's tokens)

    int64_t t0 = sh.begin + wave * kTile;
    Tile tile[2];
    u32x4 kf[2][KS];
    if (t0 < sh.end) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            tile[u] = locate(t0 + 16 * u);
            load_k(tile[u], kf[u]);
        }
    }
    while (t0 < sh.end) {
        V vf[8];
        load_v(tile[0], vf);
        load_v(tile[1], vf + 4);
        f32x4 s[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            s[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < KS; ++i)
                s[u] = Mma<T>::run(kf[u][i], qf[i], s[u]);
        }
        const uint32_t seen[2] = {tile[0].seen, tile[1].seen};
        t0 += kRound;
        if (t0 < sh.end) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                tile[u] = locate(t0 + 16 * u);
                load_k(tile[u], kf[u]);
            }
        }

        // softmax over the step's 32 tokens
        float top = m;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[u][i] *= p.scale_log2;
                if (seen[u] != 0xffffu)
                    s[u][i] = (seen[u] >> (4 * g + i)) & 1 ? s[u][i] : -INFINITY;
                top = fmaxf(top, s[u][i]);
            }
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float base = top == -INFINITY ? 0.0f : top;  // scores of -inf weigh nothing
        const float keep = __builtin_amdgcn_exp2f(m - base);
        m = top;
        float w[8], sum = 0.0f;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[4 * u + i] = __builtin_amdgcn_exp2f(s[u][i] - base + kShift<T>);
                sum += w[4 * u + i];
            }
        l = fmaf(l, keep, sum);
        if (__any(keep != 1.0f)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float f = __shfl(keep, 4 * g + i);  // of the output rows that this lane holds
#pragma unroll
                for (int e = 0; e < E; ++e)
                    o[e][i] *= f;
            }
        }
        // the weights as a 16-bit pair, value and remainder: rounded once they
        // would add an error of the output's own rounding's size
        u32x4 hi, lo;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            hi[i] = pack2<T>(w[2 * i], w[2 * i + 1]);
            lo[i] = pack2<T>(w[2 * i] - T::lo(hi[i]), w[2 * i + 1] - T::hi(hi[i]));
        }
        if (seen[0] != 0xffffu || seen[1] != 0xffffu) {  // what is not visible may be NaN
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (!((seen[i / 4] >> (4 * g + i % 4)) & 1))
                    vf[i] = V{};
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            u32x4 f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f[i] = e % 2 ? high_halves(vf[2 * i][e / 2], vf[2 * i + 1][e / 2])
                             : low_halves(vf[2 * i][e / 2], vf[2 * i + 1][e / 2]);
            o[e] = Mma<T>::run(hi, f, o[e]);
            o[e] = Mma<T>::run(lo, f, o[e]);
        }
    }

    // join the waves
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (g == 0) {
        stat_m[wave][c] = m;
        stat_l[wave][c] = l;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * g + i;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            top = fmaxf(top, stat_m[w][r]);
        const float f = __builtin_amdgcn_exp2f(stat_m[wave][r] - (top == -INFINITY ? 0.0f : top));
#pragma unroll
        for (int e = 0; e < E; ++e)
            part[wave][r][c * E + e] = o[e][i] * f;
    }
    __syncthreads();
    for (int at = static_cast<int>(threadIdx.x); at < rows * D; at += 64 * kWaves) {
        const int r = at / D, d = at % D, h = h0 + r;
        float top = -INFINITY, sum = 0.0f, y = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            top = fmaxf(top, stat_m[w][r]);
        const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            sum = fmaf(stat_l[w][r], __builtin_amdgcn_exp2f(stat_m[w][r] - base), sum);
            y += part[w][r][d];
        }
        if (sh.active == 1) {
            p.out[b * p.o_b + h * p.o_h + d] = T::round(sum == 0.0f ? 0.0f : y / sum);
            if (p.lse && d == 0)
                p.lse[b * p.l_b + h * p.l_h] = sum == 0.0f ? -INFINITY : (base - kShift<T> + log2f(sum)) * kLn2Hi;
        } else {
            const int64_t row = (static_cast<int64_t>(b) * p.splits + split) * p.nq + h;
            p.part[row * D + d] = y;
            if (d == 0) {
                p.stat[2 * row] = top;
                p.stat[2 * row + 1] = sum;
            }
        }
    }
}

// One workgroup per (request, query head): the splits' partial sums joined.
template <typename T, int D>
__global__ void __launch_bounds__(D) ssu_attn_join_kernel(const AttnParams p)
{
    const int b = static_cast<int>(blockIdx.x) / p.nq, h = static_cast<int>(blockIdx.x) % p.nq;
    const int d = static_cast<int>(threadIdx.x);
    const Share sh = share_of(p, b, 0);
    if (sh.n < 0 || sh.active == 1)
        return;  // padding, or written already
    const int64_t row0 = static_cast<int64_t>(b) * p.splits * p.nq + h;
    float top = -INFINITY, sum = 0.0f, y = 0.0f;
    for (int s = 0; s < sh.active; ++s)
        top = fmaxf(top, p.stat[2 * (row0 + static_cast<int64_t>(s) * p.nq)]);
    const float base = top == -INFINITY ? 0.0f : top;
    for (int s = 0; s < sh.active; ++s) {
        const int64_t row = row0 + static_cast<int64_t>(s) * p.nq;
        const float f = __builtin_amdgcn_exp2f(p.stat[2 * row] - base);
        sum = fmaf(p.stat[2 * row + 1], f, sum);
        y = fmaf(p.part[row * D + d], f, y);
    }
    p.out[b * p.o_b + h * p.o_h + d] = T::round(sum == 0.0f ? 0.0f : y / sum);
    if (p.lse && d == 0)
        p.lse[b * p.l_b + h * p.l_h] = sum == 0.0f ? -INFINITY : (base - kShift<T> + log2f(sum)) * kLn2Hi;
}

using AttnFn = void (*)(AttnParams);

struct AttnKernels {
    AttnFn split, join;
};

template <typename T, int D>
AttnKernels attn_kernels(bool page16)
{
    return {page16 ? &ssu_attn_split_kernel<T, D, true> : &ssu_attn_split_kernel<T, D, false>, &ssu_attn_join_kernel<T, D>};
}

template <typename T>
AttnKernels attn_kernels(int D, bool page16)
{
    return D == 64 ? attn_kernels<T, 64>(page16) : D == 128 ? attn_kernels<T, 128>(page16) : attn_kernels<T, 256>(page16);
}

// ------------------------------------------------------------------ host --

ssu_status check_sizes(const ssu_attn_args &a, const char *who)
{
    if (a.batch < 0 || a.num_pages < 0 || a.max_pages < 0 || a.page_size < 1)
        return fail(SSU_ERR_INVALID_ARGUMENT, "%s: bad size: batch %d, num_pages %lld, max_pages %lld, page_size %d", who,
                    a.batch, static_cast<long long>(a.num_pages), static_cast<long long>(a.max_pages), a.page_size);
    if (a.nk < 1 || a.nq < 1 || a.nq % a.nk)
        return fail(SSU_ERR_INVALID_ARGUMENT, "%s: %d key heads do not divide %d query heads", who, a.nk, a.nq);
    if (a.headdim != 64 && a.headdim != 128 && a.headdim != 256)
        return fail(SSU_ERR_UNSUPPORTED, "%s: headdim %d is not 64, 128 or 256", who, a.headdim);
    if (static_cast<int64_t>(a.batch) * a.nq > 0x7fffffff / kMaxSplits)
        return fail(SSU_ERR_UNSUPPORTED, "%s: batch * nq %lld too large", who, static_cast<long long>(a.batch) * a.nq);
    if (a.max_pages > INT64_MAX / a.page_size)
        return fail(SSU_ERR_INVALID_ARGUMENT, "%s: max_pages * page_size too large", who);
    return SSU_OK;
}

struct Plan {
    int row_tiles, splits, min_rounds;
    int64_t stat_at, bytes;  // workspace: floats before the statistics, bytes in all
};

// How many splits each request's length may take: enough workgroups to fill
// the chip several times over (lengths differ), no more than the table's room
// needs.
Plan plan_of(const ssu_attn_args &a)
{
    Plan p{};
    p.row_tiles = (a.nq / a.nk + 15) / 16;
    const int64_t units = static_cast<int64_t>(a.batch) * a.nk * p.row_tiles;
    const int64_t rounds = (a.max_pages * a.page_size + kRound - 1) / kRound;
    p.min_rounds = units >= kNumCUs ? 4 : 1;
    const int64_t want = units > 0 ? (16 * kNumCUs + units - 1) / units : 1;
    const int64_t most = (rounds + p.min_rounds - 1) / p.min_rounds;
    p.splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({want, most, kMaxSplits})));
    if (p.splits > 1) {
        const int64_t rows = static_cast<int64_t>(a.batch) * p.splits * a.nq;
        p.stat_at = rows * a.headdim;
        p.bytes = (p.stat_at + 2 * rows) * 4;
    }
    return p;
}

ssu_status check_attn(const ssu_attn_args &a)
{
    const char *const who = "ssu_paged_attention";
    if (a.reserved != 0)
        return fail(SSU_ERR_INVALID_ARGUMENT, "%s: reserved field must be 0", who);
    if (!std::isfinite(a.scale))
        return fail(SSU_ERR_INVALID_ARGUMENT, "%s: scale is not finite", who);
    SSU_TRY(check_sizes(a, who));
    if (a.batch == 0)
        return SSU_OK;
    const int32_t type = a.q.dtype;
    if (type != SSU_BF16 && type != SSU_F16)
        return fail(SSU_ERR_INVALID_ARGUMENT, "%s: q must be BF16 or F16", who);
    SSU_TRY(check_view(a.q, "q", type, 3, false));
    SSU_TRY(check_view(a.k_cache, "k_cache", type, 4, a.num_pages == 0));
    SSU_TRY(check_view(a.v_cache, "v_cache", type, 4, a.num_pages == 0));
    SSU_TRY(check_view(a.block_table, "block_table", SSU_I32, 2, a.max_pages == 0));
    SSU_TRY(check_view(a.seq_lens, "seq_lens", SSU_I32, 1, false));
    SSU_TRY(check_view(a.out, "out", type, 3, false));
    SSU_TRY(check_view(a.lse, "lse", SSU_F32, 2, true));
    SSU_TRY(check_written(a.out, "out", {a.batch, a.nq}));
    SSU_TRY(check_written(a.lse, "lse", {a.batch, a.nq}));
    if (a.q.stride[2] != 1 || a.out.stride[2] != 1 || (a.k_cache.ptr && a.k_cache.stride[3] != 1) ||
        (a.v_cache.ptr && a.v_cache.stride[3] != 1))
        return fail(SSU_ERR_UNSUPPORTED, "q/out/k_cache/v_cache: inner stride must be 1");
    if ((a.max_pages > 1 && a.block_table.stride[1] != 1) || (a.batch > 1 && a.seq_lens.stride[0] != 1))
        return fail(SSU_ERR_UNSUPPORTED, "block_table/seq_lens: inner stride must be 1");
    for (const ssu_view *v : {&a.q, &a.k_cache, &a.v_cache, &a.out})
        if (reinterpret_cast<uintptr_t>(v->ptr) % 2)
            return fail(SSU_ERR_MISALIGNED, "q/k_cache/v_cache/out: pointer must be 2-byte aligned");
    for (const ssu_view *v : {&a.block_table, &a.seq_lens, &a.lse})
        if (reinterpret_cast<uintptr_t>(v->ptr) % 4)
            return fail(SSU_ERR_MISALIGNED, "block_table/seq_lens/lse: pointer must be 4-byte aligned");
    return SSU_OK;
}

}  // namespace
}  // namespace ssu

extern "C" {

int64_t ssu_paged_attention_workspace(const ssu_attn_args *a)
{
    using namespace ssu;
    if (!a || check_sizes(*a, "ssu_paged_attention_workspace") != SSU_OK)
        return -1;
    return plan_of(*a).bytes;
}

ssu_status ssu_paged_attention(const ssu_attn_args *args, hipStream_t stream)
{
    using namespace ssu;
    if (!args)
        return fail(SSU_ERR_INVALID_ARGUMENT, "ssu_paged_attention: null args");
    const ssu_attn_args &a = *args;
    SSU_TRY(check_attn(a));
    if (a.batch == 0)
        return SSU_OK;
    const Plan plan = plan_of(a);
    if (plan.bytes > 0) {
        if (!a.workspace || a.workspace_bytes < plan.bytes)
            return fail(SSU_ERR_INVALID_ARGUMENT, "ssu_paged_attention: workspace of %lld bytes, %lld needed",
                        static_cast<long long>(a.workspace ? a.workspace_bytes : 0), static_cast<long long>(plan.bytes));
        if (reinterpret_cast<uintptr_t>(a.workspace) % 16)
            return fail(SSU_ERR_MISALIGNED, "ssu_paged_attention: workspace must be 16-byte aligned");
    }
    AttnParams p{};
    p.q = static_cast<const uint16_t *>(a.q.ptr);
    p.q_b = a.q.stride[0];
    p.q_h = a.q.stride[1];
    p.k = static_cast<const uint16_t *>(a.k_cache.ptr);
    p.k_page = a.k_cache.stride[0];
    p.k_row = a.k_cache.stride[1];
    p.k_h = a.k_cache.stride[2];
    p.v = static_cast<const uint16_t *>(a.v_cache.ptr);
    p.v_page = a.v_cache.stride[0];
    p.v_row = a.v_cache.stride[1];
    p.v_h = a.v_cache.stride[2];
    p.table = static_cast<const int32_t *>(a.block_table.ptr);
    p.t_b = a.block_table.stride[0];
    p.lens = static_cast<const int32_t *>(a.seq_lens.ptr);
    p.num_pages = a.num_pages;
    p.max_pages = a.max_pages;
    p.out = static_cast<uint16_t *>(const_cast<void *>(a.out.ptr));
    p.o_b = a.out.stride[0];
    p.o_h = a.out.stride[1];
    p.lse = static_cast<float *>(const_cast<void *>(a.lse.ptr));
    p.l_b = a.lse.stride[0];
    p.l_h = a.lse.stride[1];
    p.batch = a.batch;
    p.nq = a.nq;
    p.nk = a.nk;
    p.heads_per_kv = a.nq / a.nk;
    p.page_size = a.page_size;
    p.row_tiles = plan.row_tiles;
    p.splits = plan.splits;
    p.min_rounds = plan.min_rounds;
    p.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
    p.part = static_cast<float *>(a.workspace);
    p.stat = p.part + plan.stat_at;
    p.total = a.batch * a.nk * plan.row_tiles * plan.splits;
    const bool page16 = a.page_size % 16 == 0;
    const AttnKernels k = a.q.dtype == SSU_BF16 ? attn_kernels<Bf16>(a.headdim, page16) : attn_kernels<F16>(a.headdim, page16);
    DeviceGuard guard;
    SSU_TRY(guard.enter(a.device));
    hipError_t e = launch_kernel(k.split, p, p.total, 64 * kWaves, 0, stream);
    if (e == hipSuccess && plan.splits > 1)
        e = launch_kernel(k.join, p, static_cast<int64_t>(a.batch) * a.nq, a.headdim, 0, stream);
    if (e != hipSuccess)
        return fail(SSU_ERR_HIP, "launch of the paged attention kernels failed: %s", hipGetErrorString(e));
    return SSU_OK;
}

}  // extern "C"
