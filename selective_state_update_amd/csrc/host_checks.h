// host_checks.h -- host-side argument checks shared by libssu's entry points
// (not installed).
#ifndef SSU_HOST_CHECKS_H
#define SSU_HOST_CHECKS_H

#include <hip/hip_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "internal.h"
#include "ssu.h"

#define SSU_TRY(expr)                    \
    do {                                 \
        const ssu_status s_ = (expr);    \
        if (s_ != SSU_OK)                \
            return s_;                   \
    } while (0)

namespace ssu {

inline ssu_status check_view(const ssu_view &v, const char *name, int32_t dtype, int rank, bool nullable)
{
    if (!v.ptr && !nullable)
        return fail(SSU_ERR_INVALID_ARGUMENT, "%s: null pointer", name);
    if (!v.ptr)
        return SSU_OK;
    if (v.dtype != dtype)
        return fail(SSU_ERR_INVALID_ARGUMENT, "%s: dtype tag %d, expected %d", name, v.dtype, dtype);
    if (v.reserved != 0)
        return fail(SSU_ERR_INVALID_ARGUMENT, "%s: reserved field must be 0", name);
    for (int i = 0; i < rank; ++i)
        if (v.stride[i] < 0)
            return fail(SSU_ERR_INVALID_ARGUMENT, "%s: negative stride[%d]", name, i);
    return SSU_OK;
}

// A written view must give each element memory of its own: an axis of more than
// one element has a stride.
inline ssu_status check_written(const ssu_view &v, const char *name, std::initializer_list<int64_t> sizes)
{
    int i = 0;
    for (const int64_t n : sizes) {
        if (v.ptr && n > 1 && v.stride[i] == 0)
            return fail(SSU_ERR_INVALID_ARGUMENT, "%s: written with stride[%d] = 0", name, i);
        ++i;
    }
    return SSU_OK;
}

// A launch counts its threads in 32 bits.
inline ssu_status check_launch(int64_t groups, int threads, const char *who)
{
    if (groups > UINT32_MAX / threads)
        return fail(SSU_ERR_UNSUPPORTED, "%s: %lld workgroups of %d threads, 2^32 threads or more", who,
                    static_cast<long long>(groups), threads);
    return SSU_OK;
}

// Restores the caller's current device on every return path.
struct DeviceGuard {
    int prev = -1;
    bool switched = false;
    ssu_status enter(int device)
    {
        if (device < 0)
            return SSU_OK;
        if (hipGetDevice(&prev) != hipSuccess)
            return fail(SSU_ERR_HIP, "hipGetDevice failed");
        if (prev != device) {
            if (hipSetDevice(device) != hipSuccess)
                return fail(SSU_ERR_HIP, "hipSetDevice(%d) failed", device);
            switched = true;
        }
        return SSU_OK;
    }
    ~DeviceGuard()
    {
        if (switched)
            (void)hipSetDevice(prev);
    }
};

}  // namespace ssu

#endif  // SSU_HOST_CHECKS_H
