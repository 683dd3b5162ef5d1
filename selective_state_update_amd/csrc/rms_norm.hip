// rms_norm.hip -- root-mean-square norm with the residual's addition, to 16 bits
// or to 8 bits with scales, on MI355X (gfx950): ssu_add_rms_norm. The operation
// is stated in include/ssu.h.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "host_checks.h"
#include "internal.h"
#include "seq_common.h"

namespace ssu {
namespace {

constexpr int kMaxWidth = 32768;
constexpr float kLargest = 448.0f;  // of E4M3

struct NormParams {
    const uint16_t *x;
    void *residual;  // fp32 or x's type
    const void *weight;
    void *out;
    float *scales;
    int64_t x_t, r_t, o_t, s_t, s_g;
    int64_t ntokens;
    int32_t width, lanes, waves, group_lanes, w32;
    float eps;
};

enum class Residual { none, same, f32 };

// Bytes have no alignment of their own: rows of an odd width begin anywhere.
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));

// The sum and the largest bits over aligned groups of 1, 2, 4 .. 64 lanes. Bits of
// magnitudes order as the values do, NaN above infinity, so that NaN stays.
__device__ __forceinline__ float sum_over(float x, int lanes)
{
    if (lanes > 1)
        x = dpp_add<0xB1>(x);
    if (lanes > 2)
        x = dpp_add<0x4E>(x);
    if (lanes > 4)
        x = dpp_add<0x141>(x);
    if (lanes > 8)
        x = dpp_add<0x140>(x);
    if (lanes > 16)
        x += __shfl_xor(x, 16);
    if (lanes > 32)
        x += __shfl_xor(x, 32);
    return x;
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t x)
{
    return max(x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), CTRL, 0xf, 0xf, true)));
}

__device__ __forceinline__ uint32_t max_over(uint32_t x, int lanes)
{
    if (lanes > 1)
        x = dpp_max<0xB1>(x);
    if (lanes > 2)
        x = dpp_max<0x4E>(x);
    if (lanes > 4)
        x = dpp_max<0x141>(x);
    if (lanes > 8)
        x = dpp_max<0x140>(x);
    if (lanes > 16)
        x = max(x, static_cast<uint32_t>(__shfl_xor(static_cast<int>(x), 16)));
    if (lanes > 32)
        x = max(x, static_cast<uint32_t>(__shfl_xor(static_cast<int>(x), 32)));
    return x;
}

// y / unit for |y| <= 448 unit, rounded as a division is: the product with the rounded reciprocal
// and one correction by what it leaves, which is exact unless it is below fp32's least. That a
// quotient halfway between two 8-bit values stays there, and none beside it gets there, holds
// for all 2^23 significands of unit. 509 rows of 8192 9.3 us, 65536 of 512 in groups of 32 33:
// the product alone 8.9 and 31, divisions 10.2 and 37.
__device__ __forceinline__ void over(float (&y)[8], float unit)
{
    if (unit > 0x1p-90f && unit < INFINITY) {
        const float inv = 1.0f / unit;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q = y[i] * inv;
            y[i] = fmaf(-fmaf(q, unit, -y[i]), inv, q);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            y[i] /= unit;
    }
}

// n (8: all) 16-bit values from p on, zeros behind them. With RUNS they are all there.
template <typename T, bool RUNS>
__device__ __forceinline__ void load_halves(const uint16_t *p, int n, float (&f)[8])
{
    u32x4 w = {0, 0, 0, 0};
    if (RUNS || n == 8) {
        w = *reinterpret_cast<const u32x4_a2 *>(p);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                w[i / 2] |= static_cast<uint32_t>(p[i]) << 16 * (i % 2);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        f[i] = i % 2 ? T::hi(w[i / 2]) : T::lo(w[i / 2]);
}

template <bool RUNS>
__device__ __forceinline__ void load_floats(const float *p, int n, float (&f)[8])
{
    if (RUNS || n == 8) {
        const f32x4 a = *reinterpret_cast<const f32x4_a4 *>(p), b = *reinterpret_cast<const f32x4_a4 *>(p + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = a[i];
            f[i + 4] = b[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = i < n ? p[i] : 0.0f;
    }
}

template <typename T>
__device__ __forceinline__ void store_halves(uint16_t *p, int n, const float (&f)[8])
{
    if (n == 8) {
        const u32x4 w = {pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7])};
        __builtin_nontemporal_store(w, reinterpret_cast<u32x4_a2 *>(p));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                p[i] = T::round(f[i]);
    }
}

__device__ __forceinline__ void store_floats(float *p, int n, const float (&f)[8])
{
    if (n == 8) {
        __builtin_nontemporal_store(f32x4{f[0], f[1], f[2], f[3]}, reinterpret_cast<f32x4_a4 *>(p));
        __builtin_nontemporal_store(f32x4{f[4], f[5], f[6], f[7]}, reinterpret_cast<f32x4_a4 *>(p + 4));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                p[i] = f[i];
    }
}

// Rows of up to 64 runs of 8 values take `lanes` lanes (a power of two) of a wave, longer
// ones a workgroup of `waves` waves, M runs a lane, `64 * waves` runs apart: each
// value is read once, kept in fp32 and written once, past the L2 (its readers run on all
// XCDs; 16384 rows of 4096: 78 against 92 us). Memory-bound: 16384 rows of 5120 with an
// fp32 residual, to 8 bits, 171 us, 5.4 TB/s; a single row 4.5 us, which is the launch,
// one load's latency and the sum's way through the waves. RUNS: a width of whole runs,
// whose loads have no branches (a lane without a run reads the last) and whose weights
// are on their way while the sum is taken; 171 against 179 us.
template <typename T, Residual R, bool Q, int M, bool RUNS>
__global__ void __launch_bounds__(1024) ssu_rms_norm_kernel(const NormParams p)
{
    __shared__ float sums[16];
    __shared__ uint32_t tops[16];
    const int tid = static_cast<int>(threadIdx.x), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const bool shared = p.waves > 0;  // a row of several waves
    const int step = shared ? 64 * p.waves : p.lanes;
    const int first = shared ? tid : tid % p.lanes;
    const int64_t t = shared ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * (blockDim.x / p.lanes) + tid / p.lanes;
    const bool live = t < p.ntokens;
    const int64_t row = live ? t : p.ntokens - 1;

    float s[M][8], r[M][8], w[M][8], sum = 0.0f;
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const int run = (first + m * step) * 8, n = min(max(p.width - run, 0), 8), at = RUNS ? min(run, p.width - 8) : run;
        load_halves<T, RUNS>(p.x + row * p.x_t + at, n, s[m]);
        if constexpr (R == Residual::same)
            load_halves<T, RUNS>(static_cast<const uint16_t *>(p.residual) + row * p.r_t + at, n, r[m]);
        if constexpr (R == Residual::f32)
            load_floats<RUNS>(static_cast<const float *>(p.residual) + row * p.r_t + at, n, r[m]);
    }
    auto load_weights = [&] {
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int run = (first + m * step) * 8, n = min(max(p.width - run, 0), 8), at = RUNS ? min(run, p.width - 8) : run;
            if (!p.weight)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    w[m][i] = 1.0f;
            else if (p.w32)
                load_floats<RUNS>(static_cast<const float *>(p.weight) + at, n, w[m]);
            else
                load_halves<T, RUNS>(static_cast<const uint16_t *>(p.weight) + at, n, w[m]);
        }
    };
    if constexpr (RUNS)
        load_weights();  // on their way while the sum is taken
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const bool in = !RUNS || (first + m * step) * 8 < p.width;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (R != Residual::none)
                s[m][i] += r[m][i];
            s[m][i] = in ? s[m][i] : 0.0f;
            sum = fmaf(s[m][i], s[m][i], sum);
        }
    }
    sum = sum_over(sum, shared ? 64 : p.lanes);
    if (shared) {
        if (tid % 64 == 0)
            sums[wave] = sum;
        __syncthreads();
        sum = sums[0];
        for (int w = 1; w < p.waves; ++w)
            sum += sums[w];
    }
    const float scale = 1.0f / sqrtf(sum / static_cast<float>(p.width) + p.eps);

    if constexpr (!RUNS)
        load_weights();
    uint32_t top[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const int at = (first + m * step) * 8, n = min(max(p.width - at, 0), 8);
        if constexpr (R == Residual::same)
            if (live)
                store_halves<T>(static_cast<uint16_t *>(p.residual) + row * p.r_t + at, n, s[m]);
        if constexpr (R == Residual::f32)
            if (live)
                store_floats(static_cast<float *>(p.residual) + row * p.r_t + at, n, s[m]);
        top[m] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s[m][i] = s[m][i] * scale * w[m][i];
            if (i < n)
                top[m] = max(top[m], __float_as_uint(s[m][i]) & 0x7fffffffu);
        }
    }
    if constexpr (!Q) {
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int at = (first + m * step) * 8, n = min(max(p.width - at, 0), 8);
            if (live)
                store_halves<T>(static_cast<uint16_t *>(p.out) + row * p.o_t + at, n, s[m]);
        }
        return;
    }
    if (p.group_lanes > 0) {
#pragma unroll
        for (int m = 0; m < M; ++m)
            top[m] = max_over(top[m], p.group_lanes);
    } else {
#pragma unroll
        for (int m = 1; m < M; ++m)
            top[0] = max(top[0], top[m]);
        top[0] = max_over(top[0], shared ? 64 : p.lanes);
        if (shared) {
            if (tid % 64 == 0)
                tops[wave] = top[0];
            __syncthreads();
            for (int w = 0; w < p.waves; ++w)
                top[0] = max(top[0], tops[w]);
        }
#pragma unroll
        for (int m = 1; m < M; ++m)
            top[m] = top[0];
    }
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const int run = first + m * step, at = run * 8, n = min(max(p.width - at, 0), 8);
        const float most = __uint_as_float(top[m]) / kLargest;
        const float unit = most < 0x1p-126f ? 0x1p-126f : most;  // (NaN stays)
        over(s[m], unit);
        u32x2 q;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            int word = __builtin_amdgcn_cvt_pk_fp8_f32(s[m][4 * h], s[m][4 * h + 1], 0, false);
            word = __builtin_amdgcn_cvt_pk_fp8_f32(s[m][4 * h + 2], s[m][4 * h + 3], word, true);
            q[h] = static_cast<uint32_t>(word);
        }
        if (!live)
            continue;
        uint8_t *const out = static_cast<uint8_t *>(p.out) + row * p.o_t + at;
        if (n == 8) {
            __builtin_nontemporal_store(q, reinterpret_cast<u32x2_a1 *>(out));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n)
                    out[i] = static_cast<uint8_t>(q[i / 4] >> 8 * (i % 4));
        }
        const int lead = p.group_lanes > 0 ? p.group_lanes : 1 << 30;  // runs of a scale
        if (n > 0 && run % lead == 0)
            p.scales[row * p.s_t + run / lead * p.s_g] = unit;
    }
}

using NormFn = void (*)(NormParams);

template <typename T, Residual R, bool Q, bool RUNS>
NormFn norm_kernel(int m)
{
    return m == 1 ? &ssu_rms_norm_kernel<T, R, Q, 1, RUNS>
         : m == 2 ? &ssu_rms_norm_kernel<T, R, Q, 2, RUNS>
                  : &ssu_rms_norm_kernel<T, R, Q, 4, RUNS>;
}

template <typename T, Residual R>
NormFn norm_kernel(bool q, bool runs, int m)
{
    return q ? (runs ? norm_kernel<T, R, true, true>(m) : norm_kernel<T, R, true, false>(m))
             : (runs ? norm_kernel<T, R, false, true>(m) : norm_kernel<T, R, false, false>(m));
}

template <typename T>
NormFn norm_kernel(Residual r, bool q, bool runs, int m)
{
    return r == Residual::none ? norm_kernel<T, Residual::none>(q, runs, m)
         : r == Residual::same ? norm_kernel<T, Residual::same>(q, runs, m)
                               : norm_kernel<T, Residual::f32>(q, runs, m);
}

// ------------------------------------------------------------------ host --

ssu_status check_norm(const ssu_norm_args &a)
{
    const char *const who = "ssu_add_rms_norm";
    if (a.ntokens < 0 || a.width < 1 || a.group < 0)
        return fail(SSU_ERR_INVALID_ARGUMENT, "%s: bad size: ntokens %lld, width %d, group %d", who,
                    static_cast<long long>(a.ntokens), a.width, a.group);
    if (a.width > kMaxWidth)
        return fail(SSU_ERR_UNSUPPORTED, "%s: width %d above %d", who, a.width, kMaxWidth);
    if (!(a.eps >= 0.0f) || !std::isfinite(a.eps))
        return fail(SSU_ERR_INVALID_ARGUMENT, "%s: eps must be finite and not negative", who);
    const int32_t type = a.x.dtype;
    if (type != SSU_BF16 && type != SSU_F16)
        return fail(SSU_ERR_INVALID_ARGUMENT, "%s: x must be BF16 or F16", who);
    const bool eight = a.out.dtype == SSU_E4M3;
    if (a.group != 0) {
        if (!eight || a.width % a.group)
            return fail(SSU_ERR_INVALID_ARGUMENT, "%s: group %d: out is not E4M3 or the width %d no multiple", who, a.group, a.width);
        if (a.group != 32 && a.group != 64 && a.group != 128 && a.group != 256)
            return fail(SSU_ERR_UNSUPPORTED, "%s: group %d is not 32, 64, 128 or 256", who, a.group);
    }
    if (!eight && a.scales.ptr)
        return fail(SSU_ERR_INVALID_ARGUMENT, "%s: scales without an output in E4M3", who);
    const bool none = a.ntokens == 0;
    const int64_t groups = a.group ? a.width / a.group : 1;
    SSU_TRY(check_view(a.x, "x", type, 2, none));
    SSU_TRY(check_view(a.residual, "residual", a.residual.dtype == SSU_F32 ? SSU_F32 : type, 2, true));
    SSU_TRY(check_view(a.weight, "weight", a.weight.dtype == SSU_F32 ? SSU_F32 : type, 1, true));
    SSU_TRY(check_view(a.out, "out", eight ? SSU_E4M3 : type, 2, none));
    SSU_TRY(check_view(a.scales, "scales", SSU_F32, 2, none || !eight));
    SSU_TRY(check_written(a.residual, "residual", {a.ntokens}));
    SSU_TRY(check_written(a.out, "out", {a.ntokens}));
    SSU_TRY(check_written(a.scales, "scales", {a.ntokens, groups}));
    for (const ssu_view *v : {&a.x, &a.residual, &a.out})
        if (v->ptr && a.width > 1 && v->stride[1] != 1)
            return fail(SSU_ERR_UNSUPPORTED, "x/residual/out: inner stride must be 1");
    if (a.weight.ptr && a.width > 1 && a.weight.stride[0] != 1)
        return fail(SSU_ERR_UNSUPPORTED, "weight: stride must be 1");
    for (const ssu_view *v : {&a.x, &a.residual, &a.weight, &a.out, &a.scales}) {
        const uintptr_t size = v->dtype == SSU_F32 ? 4 : v->dtype == SSU_E4M3 ? 1 : 2;
        if (reinterpret_cast<uintptr_t>(v->ptr) % size)
            return fail(SSU_ERR_MISALIGNED, "x/residual/weight/out/scales: pointer must be aligned to its element");
    }
    return SSU_OK;
}

}  // namespace
}  // namespace ssu

extern "C" ssu_status ssu_add_rms_norm(const ssu_norm_args *args, hipStream_t stream)
{
    using namespace ssu;
    if (!args)
        return fail(SSU_ERR_INVALID_ARGUMENT, "ssu_add_rms_norm: null args");
    const ssu_norm_args &a = *args;
    SSU_TRY(check_norm(a));
    if (a.ntokens == 0)
        return SSU_OK;
    NormParams p{};
    p.x = static_cast<const uint16_t *>(a.x.ptr);
    p.x_t = a.x.stride[0];
    p.residual = const_cast<void *>(a.residual.ptr);
    p.r_t = a.residual.stride[0];
    p.weight = a.weight.ptr;
    p.w32 = a.weight.dtype == SSU_F32;
    p.out = const_cast<void *>(a.out.ptr);
    p.o_t = a.out.stride[0];
    p.scales = static_cast<float *>(const_cast<void *>(a.scales.ptr));
    p.s_t = a.scales.stride[0];
    p.s_g = a.scales.stride[1];
    p.ntokens = a.ntokens;
    p.width = a.width;
    p.eps = a.eps;
    p.group_lanes = a.group / 8;
    const int runs = (a.width + 7) / 8;
    int m = 1, threads = 256;
    int64_t groups;
    if (runs <= 64) {
        for (p.lanes = 1; p.lanes < runs; p.lanes *= 2) {
        }
        const int rows = 256 / p.lanes;
        groups = a.ntokens / rows + (a.ntokens % rows != 0);
    } else {
        // (16384 rows of 640 runs: m = 2 172 us, 1 182, 4 190; of 1024: 171, 186, 183; of 2048:
        // 395 (m = 2), 414 (4); 16384 rows of 512 runs 92 with 1, 90 with 2, but 509 of
        // them 6.1 against 6.2: few rows want many waves)
        m = runs <= 512 ? 1 : runs <= 2048 ? 2 : 4;
        p.waves = (runs + 64 * m - 1) / (64 * m);
        threads = 64 * p.waves;
        groups = a.ntokens;
    }
    SSU_TRY(check_launch(groups, threads, "ssu_add_rms_norm"));
    const Residual r = !p.residual ? Residual::none : a.residual.dtype == SSU_F32 ? Residual::f32 : Residual::same;
    const bool eight = a.out.dtype == SSU_E4M3, runs_only = a.width % 8 == 0;
    const NormFn fn = a.x.dtype == SSU_BF16 ? norm_kernel<Bf16>(r, eight, runs_only, m) : norm_kernel<F16>(r, eight, runs_only, m);
    DeviceGuard guard;
    SSU_TRY(guard.enter(a.device));
    const hipError_t e = launch_kernel(fn, p, groups, threads, 0, stream);
    if (e != hipSuccess)
        return fail(SSU_ERR_HIP, "launch of the norm kernel failed: %s", hipGetErrorString(e));
    return SSU_OK;
}
