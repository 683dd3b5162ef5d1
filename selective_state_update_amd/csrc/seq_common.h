// seq_common.h -- device helpers shared by the sequence operators
// (linear_attention.hip, qk_norm_rope.hip, paged_attention.hip; not installed).
#ifndef SSU_SEQ_COMMON_H
#define SSU_SEQ_COMMON_H

#include <hip/hip_runtime.h>

#include <cstdint>

#include "internal.h"

namespace ssu {

constexpr int kNumCUs = 256;  // MI355X

using u32x4 = uint32_t __attribute__((ext_vector_type(4)));

// Runs of 16-bit elements as one access. The type's alignment is the
// element's: gfx950 reads and writes 4, 8 and 16 bytes at any 2-byte address,
// at full speed where the address is a multiple of the size, so views need no
// alignment beyond their elements'.
typedef uint32_t u32_a2 __attribute__((aligned(2)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef f32x4 f32x4_a4 __attribute__((aligned(4)));

// 16-bit floating types: the fp32 value of bits, and bits rounded to nearest
// even from fp32 (the conversion is kept opaque to the compiler so that it is
// never fused with the operation that produces its operand).
struct Bf16 {
    using Native = __bf16;
    static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
    static __device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
    static __device__ __forceinline__ uint16_t round(float f)
    {
        asm volatile("" : "+v"(f));
        return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
    }
};

struct F16 {
    using Native = _Float16;
    static __device__ __forceinline__ float value(uint16_t b)
    {
        return static_cast<float>(__builtin_bit_cast(_Float16, b));
    }
    static __device__ __forceinline__ float lo(uint32_t w) { return value(static_cast<uint16_t>(w)); }
    static __device__ __forceinline__ float hi(uint32_t w) { return value(static_cast<uint16_t>(w >> 16)); }
    static __device__ __forceinline__ uint16_t round(float f)
    {
        asm volatile("" : "+v"(f));
        return __builtin_bit_cast(uint16_t, static_cast<_Float16>(f));
    }
};

// One wave's product of a 16 x 32 and a 32 x 16 tile on the matrix cores, fp32
// sums. Lane l holds row (column) l % 16 of a (of b), 8 consecutive places of
// the contracted axis from 8 * (l / 16); of the result it holds column l % 16,
// rows 4 * (l / 16) + 0..3. Which values share a place of the contracted axis
// is free as long as a and b agree.
template <typename T>
struct Mma;

template <>
struct Mma<Bf16> {
    using Frag = __bf16 __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ f32x4 run(u32x4 a, u32x4 b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(Frag, a), __builtin_bit_cast(Frag, b), c, 0, 0, 0);
    }
};

template <>
struct Mma<F16> {
    using Frag = _Float16 __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ f32x4 run(u32x4 a, u32x4 b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(Frag, a), __builtin_bit_cast(Frag, b), c, 0, 0, 0);
    }
};

// Two fp32 values as a word of two 16-bit ones, rounded to nearest even (one
// instruction).
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    using F = float __attribute__((ext_vector_type(2)));
    using H = typename T::Native __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((F{lo, hi}), H));
}

// The 16-bit halves of two words side by side: the low ones, the high ones.
__device__ __forceinline__ uint32_t low_halves(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); }
__device__ __forceinline__ uint32_t high_halves(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }

// Element i of an index array of 32- or 64-bit integers.
__device__ __forceinline__ int64_t load_index(const void *p, int is64, int64_t i)
{
    return is64 ? static_cast<const int64_t *>(p)[i] : static_cast<int64_t>(static_cast<const int32_t *>(p)[i]);
}

// The sum over aligned groups of LANES lanes, in every lane of a group: within 16
// lanes by DPP (quad permutes, half-row and row mirror), beyond by exchange.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float x)
{
    return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}

template <int LANES>
__device__ __forceinline__ float sum_lanes(float x)
{
    if constexpr (LANES >= 2)
        x = dpp_add<0xB1>(x);
    if constexpr (LANES >= 4)
        x = dpp_add<0x4E>(x);
    if constexpr (LANES >= 8)
        x = dpp_add<0x141>(x);
    if constexpr (LANES >= 16)
        x = dpp_add<0x140>(x);
    if constexpr (LANES >= 32)
        x += __shfl_xor(x, 16);
    if constexpr (LANES >= 64)
        x += __shfl_xor(x, 32);
    return x;
}

// Inclusive sums over the wave's lanes, by DPP: within 16 lanes (lane - 1, - 2,
// - 4, - 8), then the last of 16 to the next 16 and of 32 to the next 32.
template <int CTRL, int MASK>
__device__ __forceinline__ int dpp_up(int x)
{
    return x + __builtin_amdgcn_update_dpp(0, x, CTRL, MASK, 0xf, true);
}

__device__ __forceinline__ int scan_lanes(int x)
{
    x = dpp_up<0x111, 0xf>(x);
    x = dpp_up<0x112, 0xf>(x);
    x = dpp_up<0x114, 0xf>(x);
    x = dpp_up<0x118, 0xf>(x);
    x = dpp_up<0x142, 0xa>(x);
    return dpp_up<0x143, 0xc>(x);
}

// Launch a kernel and return its own status (a call that fails leaves no
// error behind for the caller's next runtime call).
template <typename P>
hipError_t launch_kernel(void (*fn)(P), const P &p, int64_t grid, int block, size_t lds, hipStream_t stream)
{
    P copy = p;
    void *args[] = {&copy};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void *>(fn), dim3(static_cast<uint32_t>(grid)),
                                         dim3(block), args, lds, stream);
    if (e != hipSuccess)
        (void)hipGetLastError();
    return e;
}

}  // namespace ssu

#endif  // SSU_SEQ_COMMON_H
