// paged_attention.hip -- attention of one new token per request over a paged
// key-value cache on MI355X (gfx950): ssu_paged_attention. The operation is
// stated in include/ssu.h, its kernels in attention_kernels.h.

#include "attention_kernels.h"

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
    SSU_TRY(check_attn(a, "ssu_paged_attention"));
    if (a.batch == 0)
        return SSU_OK;
    const Plan plan = plan_of(a);
    if (plan.bytes > 0 && (!a.workspace || a.workspace_bytes < plan.bytes))
        return fail(SSU_ERR_INVALID_ARGUMENT, "ssu_paged_attention: workspace of %lld bytes, %lld needed",
                    static_cast<long long>(a.workspace ? a.workspace_bytes : 0), static_cast<long long>(plan.bytes));
    if (reinterpret_cast<uintptr_t>(a.workspace) % 16)
        return fail(SSU_ERR_MISALIGNED, "ssu_paged_attention: workspace must be 16-byte aligned");
    SSU_TRY(check_launch(plan.groups, 64 * plan.waves, "ssu_paged_attention"));
    DeviceGuard guard;
    SSU_TRY(guard.enter(a.device));
    return launch_attn<false>(a, plan, attn_params(a, plan, a.workspace), "ssu_paged_attention", stream);
}

}  // extern "C"
