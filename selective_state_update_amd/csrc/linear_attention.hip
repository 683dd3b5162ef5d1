// linear_attention.hip -- linear attention with a decay for each head on MI355X
// (gfx950): ssu_linear_attention over whole prompts, ssu_linear_attention_step
// for one token per request. The operation is stated in include/ssu.h.

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "host_checks.h"
#include "internal.h"
#include "seq_common.h"

namespace ssu {
namespace {

struct LinearParams {
    float *state;
    int64_t s_slot, s_head, s_row;
    const void *idx;
    int64_t pool_slots;
    const int32_t *cu;  // NULL: token b is request b's
    const uint16_t *q, *k, *v;
    int64_t q_t, q_g, k_t, k_g, v_t, v_h;
    const float *decay, *beta;
    int64_t d_t, d_h, b_t, b_h;
    uint16_t *out;
    int64_t o_t, o_h;
    int64_t ntokens;
    int32_t idx64, batch, nheads, heads_per_group, headdim, tiles, total;
    float scale;
};

// The recurrence, token after token, the state in registers. One wave owns
// RPI * R rows p of one (request, head): a row's N values are split over LPR =
// N / 4 lanes (N = 256: 32 lanes with two chunks), one dwordx4 each, so that
// one instruction moves 1 KiB of contiguous state.
template <int N, int R>
__global__ void __launch_bounds__(64) ssu_linear_recurrent_kernel(const LinearParams p)
{
    constexpr int VEC = N > 128 ? N / 128 : 1;
    constexpr int LPR = N / (4 * VEC);
    constexpr int RPI = 64 / LPR;
    static_assert(R <= LPR, "one writer lane per row");
    const int g = xcd_order(static_cast<int>(blockIdx.x), p.total);
    const int tile = g % p.tiles, bh = g / p.tiles;
    const int h = bh % p.nheads, b = bh / p.nheads, grp = h / p.heads_per_group;
    const int lane = static_cast<int>(threadIdx.x), c = lane % LPR, sub = lane / LPR;
    const int64_t slot = load_index(p.idx, p.idx64, b);
    if (slot < 0 || slot >= p.pool_slots)
        return;  // padding
    int64_t t = b, end = b + 1;
    if (p.cu) {
        t = max(static_cast<int64_t>(p.cu[b]), int64_t(0));
        end = min(static_cast<int64_t>(p.cu[b + 1]), p.ntokens);
    }
    if (t >= end)
        return;

    const int row0 = tile * RPI * R + sub;
    float *const sp = p.state + slot * p.s_slot + h * p.s_head + 4 * c;
    f32x4 s[R][VEC];
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (row0 + j * RPI < p.headdim)
                s[j][e] = load4<true>(sp + (row0 + j * RPI) * p.s_row + 128 * e);
            else
                s[j][e] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    for (; t < end; ++t) {
        const uint16_t *const qt = p.q + t * p.q_t + grp * p.q_g, *const kt = p.k + t * p.k_t + grp * p.k_g;
        const uint16_t *const vt = p.v + t * p.v_t + h * p.v_h;
        const float a = exp_f32(p.decay[t * p.d_t + h * p.d_h]);
        const float beta = p.beta ? p.beta[t * p.b_t + h * p.b_h] : 1.0f;
        float q[VEC][4], k[VEC][4];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const u32x2 qw = *reinterpret_cast<const u32x2_a2 *>(qt + 4 * c + 128 * e);
            const u32x2 kw = *reinterpret_cast<const u32x2_a2 *>(kt + 4 * c + 128 * e);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                q[e][2 * i] = Bf16::lo(qw[i]);
                q[e][2 * i + 1] = Bf16::hi(qw[i]);
                k[e][2 * i] = Bf16::lo(kw[i]);
                k[e][2 * i + 1] = Bf16::hi(kw[i]);
            }
        }
        float y[R];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const int row = row0 + j * RPI;
            const float v = beta * (row < p.headdim ? Bf16::lo(vt[row]) : 0.0f);
            float acc = 0.0f;
#pragma unroll
            for (int e = 0; e < VEC; ++e)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[j][e][i] = fmaf(s[j][e][i], a, v * k[e][i]);
                    acc = fmaf(s[j][e][i], q[e][i], acc);
                }
#pragma unroll
            for (int m = LPR / 2; m >= 1; m /= 2)
                acc += __shfl_xor(acc, m);
            y[j] = acc;
        }
#pragma unroll
        for (int j = 0; j < R; ++j)
            if (c == j && row0 + j * RPI < p.headdim)
                p.out[t * p.o_t + h * p.o_h + row0 + j * RPI] = Bf16::round(p.scale * y[j]);
    }

#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (row0 + j * RPI < p.headdim)
                store4<true>(sp + (row0 + j * RPI) * p.s_row + 128 * e, s[j][e]);
}

using LinearFn = void (*)(LinearParams);

struct LinearKernel {
    LinearFn fn;
    int rows;  // of the state per workgroup
};

template <int N, int R>
constexpr LinearKernel recurrent()
{
    constexpr int VEC = N > 128 ? N / 128 : 1;
    return {&ssu_linear_recurrent_kernel<N, R>, 64 / (N / (4 * VEC)) * R};
}

LinearKernel recurrent_kernel(int N)
{
    switch (N) {
    case 16: return recurrent<16, 4>();
    case 32: return recurrent<32, 4>();
    case 64: return recurrent<64, 4>();
    case 128: return recurrent<128, 4>();
    default: return recurrent<256, 4>();
    }
}

// ------------------------------------------------------------------ host --

ssu_status check_sizes(const ssu_linear_args &a, const char *who)
{
    if (a.batch < 0 || a.ntokens < 0 || a.pool_slots < 0 || a.nheads < 1)
        return fail(SSU_ERR_INVALID_ARGUMENT, "%s: bad size: batch %d, ntokens %lld, pool_slots %lld, nheads %d", who,
                    a.batch, static_cast<long long>(a.ntokens), static_cast<long long>(a.pool_slots), a.nheads);
    if (a.ngroups < 1 || a.nheads % a.ngroups)
        return fail(SSU_ERR_INVALID_ARGUMENT, "%s: ngroups %d does not divide nheads %d", who, a.ngroups, a.nheads);
    if (a.headdim < 16 || a.headdim > 256 || a.headdim % 16)
        return fail(SSU_ERR_UNSUPPORTED, "%s: headdim %d is not a multiple of 16 in 16 .. 256", who, a.headdim);
    if (a.dstate != 16 && a.dstate != 32 && a.dstate != 64 && a.dstate != 128 && a.dstate != 256)
        return fail(SSU_ERR_UNSUPPORTED, "%s: dstate %d is not 16, 32, 64, 128 or 256", who, a.dstate);
    if (a.ntokens > 0x7fffffff)
        return fail(SSU_ERR_UNSUPPORTED, "%s: more than 2^31 tokens", who);
    if (static_cast<int64_t>(a.batch) * a.nheads * (a.headdim / 16) > 0x7fffffff)
        return fail(SSU_ERR_UNSUPPORTED, "%s: batch * nheads too large", who);
    return SSU_OK;
}

ssu_status check_linear(const ssu_linear_args &a, const char *who, bool prompts)
{
    if (a.reserved != 0)
        return fail(SSU_ERR_INVALID_ARGUMENT, "%s: reserved field must be 0", who);
    if (!std::isfinite(a.scale))
        return fail(SSU_ERR_INVALID_ARGUMENT, "%s: scale is not finite", who);
    SSU_TRY(check_sizes(a, who));
    SSU_TRY(check_view(a.state, "state", SSU_F32, 4, a.pool_slots == 0));
    SSU_TRY(check_view(a.idx, "idx", a.idx.dtype == SSU_I64 ? SSU_I64 : SSU_I32, 1, a.batch == 0));
    if (prompts)
        SSU_TRY(check_view(a.cu_seqlens, "cu_seqlens", SSU_I32, 1, false));
    else if (a.cu_seqlens.ptr || a.workspace || a.ntokens != a.batch)
        return fail(SSU_ERR_INVALID_ARGUMENT, "%s: one token per request, cu_seqlens and workspace NULL", who);
    const bool none = a.ntokens == 0;
    SSU_TRY(check_view(a.q, "q", SSU_BF16, 3, none));
    SSU_TRY(check_view(a.k, "k", SSU_BF16, 3, none));
    SSU_TRY(check_view(a.v, "v", SSU_BF16, 3, none));
    SSU_TRY(check_view(a.log_decay, "log_decay", SSU_F32, 2, none));
    SSU_TRY(check_view(a.beta, "beta", SSU_F32, 2, true));
    SSU_TRY(check_view(a.out, "out", SSU_BF16, 3, none));
    SSU_TRY(check_written(a.state, "state", {a.pool_slots, a.nheads, a.headdim}));
    SSU_TRY(check_written(a.out, "out", {a.ntokens, a.nheads}));
    if (a.state.ptr && a.state.stride[3] != 1)
        return fail(SSU_ERR_UNSUPPORTED, "state: dstate stride must be 1");
    if (a.idx.ptr && a.idx.stride[0] != 1)
        return fail(SSU_ERR_UNSUPPORTED, "idx: stride must be 1");
    if (prompts && a.cu_seqlens.stride[0] != 1)
        return fail(SSU_ERR_UNSUPPORTED, "cu_seqlens: stride must be 1");
    for (const ssu_view *v : {&a.q, &a.k, &a.v, &a.out})
        if (v->ptr && v->stride[2] != 1)
            return fail(SSU_ERR_UNSUPPORTED, "q/k/v/out: inner stride must be 1");
    if (reinterpret_cast<uintptr_t>(a.state.ptr) % 16 ||
        (a.state.ptr && (a.state.stride[0] % 4 || a.state.stride[1] % 4 || a.state.stride[2] % 4)))
        return fail(SSU_ERR_MISALIGNED, "state: pointer and slot/head/row strides must be 16-byte multiples");
    for (const ssu_view *v : {&a.q, &a.k, &a.v, &a.out})
        if (reinterpret_cast<uintptr_t>(v->ptr) % 2)
            return fail(SSU_ERR_MISALIGNED, "q/k/v/out: pointer must be 2-byte aligned");
    for (const ssu_view *v : {&a.log_decay, &a.beta, &a.cu_seqlens})
        if (reinterpret_cast<uintptr_t>(v->ptr) % 4)
            return fail(SSU_ERR_MISALIGNED, "log_decay/beta/cu_seqlens: pointer must be 4-byte aligned");
    if (reinterpret_cast<uintptr_t>(a.idx.ptr) % (a.idx.dtype == SSU_I64 ? 8 : 4))
        return fail(SSU_ERR_MISALIGNED, "idx: pointer must be aligned to its element");
    return SSU_OK;
}

LinearParams linear_params(const ssu_linear_args &a)
{
    LinearParams p{};
    p.state = static_cast<float *>(const_cast<void *>(a.state.ptr));
    p.s_slot = a.state.stride[0];
    p.s_head = a.state.stride[1];
    p.s_row = a.state.stride[2];
    p.idx = a.idx.ptr;
    p.idx64 = a.idx.dtype == SSU_I64;
    p.pool_slots = a.pool_slots;
    p.cu = static_cast<const int32_t *>(a.cu_seqlens.ptr);
    p.q = static_cast<const uint16_t *>(a.q.ptr);
    p.q_t = a.q.stride[0];
    p.q_g = a.q.stride[1];
    p.k = static_cast<const uint16_t *>(a.k.ptr);
    p.k_t = a.k.stride[0];
    p.k_g = a.k.stride[1];
    p.v = static_cast<const uint16_t *>(a.v.ptr);
    p.v_t = a.v.stride[0];
    p.v_h = a.v.stride[1];
    p.decay = static_cast<const float *>(a.log_decay.ptr);
    p.d_t = a.log_decay.stride[0];
    p.d_h = a.log_decay.stride[1];
    p.beta = static_cast<const float *>(a.beta.ptr);
    p.b_t = a.beta.stride[0];
    p.b_h = a.beta.stride[1];
    p.out = static_cast<uint16_t *>(const_cast<void *>(a.out.ptr));
    p.o_t = a.out.stride[0];
    p.o_h = a.out.stride[1];
    p.ntokens = a.ntokens;
    p.batch = a.batch;
    p.nheads = a.nheads;
    p.heads_per_group = a.nheads / a.ngroups;
    p.headdim = a.headdim;
    p.scale = a.scale;
    return p;
}

ssu_status launch_recurrent(const ssu_linear_args &a, hipStream_t stream)
{
    DeviceGuard guard;
    SSU_TRY(guard.enter(a.device));
    const LinearKernel k = recurrent_kernel(a.dstate);
    LinearParams p = linear_params(a);
    p.tiles = (a.headdim + k.rows - 1) / k.rows;
    p.total = a.batch * a.nheads * p.tiles;
    const hipError_t e = launch_kernel(k.fn, p, p.total, 64, 0, stream);
    if (e != hipSuccess)
        return fail(SSU_ERR_HIP, "launch of the linear attention kernel failed: %s", hipGetErrorString(e));
    return SSU_OK;
}

}  // namespace
}  // namespace ssu

extern "C" {

int64_t ssu_linear_attention_workspace(const ssu_linear_args *a)
{
    using namespace ssu;
    if (!a || check_sizes(*a, "ssu_linear_attention_workspace") != SSU_OK)
        return -1;
    return 0;
}

ssu_status ssu_linear_attention(const ssu_linear_args *a, hipStream_t stream)
{
    using namespace ssu;
    if (!a)
        return fail(SSU_ERR_INVALID_ARGUMENT, "ssu_linear_attention: null args");
    SSU_TRY(check_linear(*a, "ssu_linear_attention", true));
    if (a->batch == 0 || a->ntokens == 0)
        return SSU_OK;
    return launch_recurrent(*a, stream);
}

ssu_status ssu_linear_attention_step(const ssu_linear_args *a, hipStream_t stream)
{
    using namespace ssu;
    if (!a)
        return fail(SSU_ERR_INVALID_ARGUMENT, "ssu_linear_attention_step: null args");
    SSU_TRY(check_linear(*a, "ssu_linear_attention_step", false));
    if (a->batch == 0)
        return SSU_OK;
    return launch_recurrent(*a, stream);
}

}  // extern "C"
