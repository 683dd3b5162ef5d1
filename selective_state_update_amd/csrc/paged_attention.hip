// paged_attention.hip -- attention of one new token per request over a paged
// key-value cache on MI355X (gfx950): ssu_paged_attention. The operation is
// stated in include/ssu.h.

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "host_checks.h"
#include "internal.h"
#include "seq_common.h"

namespace ssu {
namespace {

struct AttnParams {
    const uint16_t *q, *k, *v;
    int64_t q_b, q_h, k_page, k_row, k_h, v_page, v_row, v_h;
    const int32_t *table, *lens;
    int64_t t_b, num_pages, max_pages;
    uint16_t *out;
    int64_t o_b, o_h;
    float *lse;
    int64_t l_b, l_h;
    int32_t batch, nq, nk, heads_per_kv, page_size;
    float scale;
};

// One workgroup per (request, query head); its four waves take every fourth
// token, each with a running maximum and sum, and are joined at the end.
template <typename T, int D>
__global__ void __launch_bounds__(256) ssu_attn_rows_kernel(const AttnParams p)
{
    constexpr int E = D / 64;  // elements per lane
    __shared__ float part[4][D];
    __shared__ float stat[4][2];
    const int b = static_cast<int>(blockIdx.x) / p.nq, h = static_cast<int>(blockIdx.x) % p.nq;
    const int kh = h / p.heads_per_kv, lane = static_cast<int>(threadIdx.x) & 63, wave = static_cast<int>(threadIdx.x) >> 6;
    int64_t n = p.lens[b];
    if (n < 0)
        return;  // padding
    n = min(n, p.max_pages * p.page_size);
    float q[E], o[E], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = T::lo(p.q[b * p.q_b + h * p.q_h + lane + 64 * e]);
        o[e] = 0.0f;
    }
    for (int64_t j = wave; j < n; j += 4) {
        const int64_t col = j / p.page_size, page = p.table[b * p.t_b + col], off = j - col * p.page_size;
        if (page < 0 || page >= p.num_pages)
            continue;
        const uint16_t *const kr = p.k + page * p.k_page + off * p.k_row + kh * p.k_h;
        const uint16_t *const vr = p.v + page * p.v_page + off * p.v_row + kh * p.v_h;
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e)
            s = fmaf(q[e], T::lo(kr[lane + 64 * e]), s);
#pragma unroll
        for (int x = 32; x >= 1; x /= 2)
            s += __shfl_xor(s, x);
        s *= p.scale;
        const float top = fmaxf(m, s), base = top == -INFINITY ? 0.0f : top;  // -inf scores weigh nothing
        const float keep = expf(m - base), w = expf(s - base);
        m = top;
        l = fmaf(l, keep, w);
#pragma unroll
        for (int e = 0; e < E; ++e)
            o[e] = fmaf(o[e], keep, w * T::lo(vr[lane + 64 * e]));
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
        part[wave][lane + 64 * e] = o[e];
    if (lane == 0) {
        stat[wave][0] = m;
        stat[wave][1] = l;
    }
    __syncthreads();
    float top = -INFINITY, sum = 0.0f, f[4];
    for (int w = 0; w < 4; ++w)
        top = fmaxf(top, stat[w][0]);
    const float base = top == -INFINITY ? 0.0f : top;
    for (int w = 0; w < 4; ++w) {
        f[w] = expf(stat[w][0] - base);
        sum += stat[w][1] * f[w];
    }
    for (int i = static_cast<int>(threadIdx.x); i < D; i += 256) {
        float y = 0.0f;
        for (int w = 0; w < 4; ++w)
            y = fmaf(part[w][i], f[w], y);
        p.out[b * p.o_b + h * p.o_h + i] = T::round(sum == 0.0f ? 0.0f : y / sum);
    }
    if (p.lse && threadIdx.x == 0)
        p.lse[b * p.l_b + h * p.l_h] = sum == 0.0f ? -INFINITY : base + logf(sum);
}

using AttnFn = void (*)(AttnParams);

AttnFn rows_kernel(int32_t type, int D)
{
    if (type == SSU_BF16)
        return D == 64 ? &ssu_attn_rows_kernel<Bf16, 64> : D == 128 ? &ssu_attn_rows_kernel<Bf16, 128>
                                                                    : &ssu_attn_rows_kernel<Bf16, 256>;
    return D == 64 ? &ssu_attn_rows_kernel<F16, 64> : D == 128 ? &ssu_attn_rows_kernel<F16, 128>
                                                               : &ssu_attn_rows_kernel<F16, 256>;
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
    if (static_cast<int64_t>(a.batch) * a.nq > 0x7fffffff)
        return fail(SSU_ERR_UNSUPPORTED, "%s: more than 2^31 workgroups", who);
    return SSU_OK;
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
    return 0;
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
    p.scale = a.scale;
    DeviceGuard guard;
    SSU_TRY(guard.enter(a.device));
    const hipError_t e = launch_kernel(rows_kernel(a.q.dtype, a.headdim), p, static_cast<int64_t>(a.batch) * a.nq, 256, 0,
                                       stream);
    if (e != hipSuccess)
        return fail(SSU_ERR_HIP, "launch of the paged attention kernel failed: %s", hipGetErrorString(e));
    return SSU_OK;
}

}  // extern "C"
