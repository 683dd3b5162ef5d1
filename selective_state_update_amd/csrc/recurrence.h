// recurrence.h -- what the operators on state slots share (linear_attention.hip,
// gated_delta.hip; not installed): their operands as a kernel takes them and the
// host's checks of them.
#ifndef SSU_RECURRENCE_H
#define SSU_RECURRENCE_H

#include <cmath>
#include <cstdint>

#include "host_checks.h"
#include "internal.h"
#include "seq_common.h"

namespace ssu {

constexpr int kChunk = 32;  // tokens of prompts that go through the recurrence at once
constexpr float kDecayFloor = -1.0e4f;  // exp is 0 far above it; sums of it stay finite

struct LinearParams {
    float *state;
    int64_t s_slot, s_head, s_row;
    const void *idx;
    int64_t pool_slots;
    const int32_t *cu;  // (prompts)
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

// Argument checks of ssu_linear_args and ssu_delta_args, whose operands are the same.
template <typename A>
ssu_status check_sizes(const A &a, const char *who)
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
    if (a.ntokens > 0x7ffff000)  // (a segment and two workgroups' tokens count in 32 bits)
        return fail(SSU_ERR_UNSUPPORTED, "%s: more than 2^31 tokens", who);
    if ((a.ntokens / kChunk + a.batch + 8) * a.nheads > 0x7fffffff / (a.headdim / 16))
        return fail(SSU_ERR_UNSUPPORTED, "%s: batch * nheads too large", who);
    return SSU_OK;
}

template <typename A>
ssu_status check_linear(const A &a, const char *who, bool prompts)
{
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
    if (prompts)
        for (const ssu_view *v : {&a.q, &a.k, &a.v, &a.out})
            if (v->stride[0] >= int64_t(1) << 24)  // 64 rows lie within 2^31 bytes
                return fail(SSU_ERR_UNSUPPORTED, "%s: a token stride of 2^24 elements or more", who);
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

template <typename A>
LinearParams linear_params(const A &a)
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

}  // namespace ssu

#endif  // SSU_RECURRENCE_H
