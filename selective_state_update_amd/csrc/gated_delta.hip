// gated_delta.hip -- the gated delta rule on MI355X (gfx950):
// ssu_gated_delta_rule over whole prompts, ssu_gated_delta_rule_step for one
// token per request. The operation is stated in include/ssu.h.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "host_checks.h"
#include "internal.h"
#include "recurrence.h"
#include "seq_common.h"

namespace ssu {
namespace {

constexpr float kFaint = 1e-6f;  // beside the squares of q and k that are normalized

__device__ __forceinline__ float inverse_length(float squares) { return 1.0f / sqrtf(squares + kFaint); }

struct StepParams {
    LinearParams a;
    int32_t normalize;
};

// One token per request. One wave owns RPI * R rows p of one (request, head): a
// row's N values are split over LPR = N / 4 lanes (N = 256: 32 lanes with two
// chunks), one dwordx4 each, so that one instruction moves 1 KiB of contiguous
// state. Memory-bound by the state, read and written once, past the caches; what
// does not depend on the slot is requested first, since vector loads return in order.
// What a row recalls of k has to be known before the row is written: two sums over
// its lanes, one behind the other, instead of the one of linear attention.
template <int N, int R>
__global__ void __launch_bounds__(64) ssu_delta_step_kernel(const StepParams sp)
{
    constexpr int VEC = N > 128 ? N / 128 : 1;
    constexpr int LPR = N / (4 * VEC);
    constexpr int RPI = 64 / LPR;
    static_assert(R <= LPR, "one writer lane per row");
    const LinearParams &p = sp.a;
    const int id = xcd_order(static_cast<int>(blockIdx.x), p.total);
    const int tile = id % p.tiles, bh = id / p.tiles;
    const int h = __builtin_amdgcn_readfirstlane(bh % p.nheads), b = __builtin_amdgcn_readfirstlane(bh / p.nheads);
    const int grp = __builtin_amdgcn_readfirstlane(h / p.heads_per_group);
    const int lane = static_cast<int>(threadIdx.x), c = lane % LPR, sub = lane / LPR;
    const int row0 = __builtin_amdgcn_readfirstlane(tile * RPI * R) + sub;

    const uint16_t *const qt = p.q + b * p.q_t + grp * p.q_g, *const kt = p.k + b * p.k_t + grp * p.k_g;
    const uint16_t *const vt = p.v + b * p.v_t + h * p.v_h;
    u32x2 qw[VEC], kw[VEC];
    uint16_t vw[R];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        qw[e] = *reinterpret_cast<const u32x2_a2 *>(qt + 4 * c + 128 * e);
        kw[e] = *reinterpret_cast<const u32x2_a2 *>(kt + 4 * c + 128 * e);
    }
#pragma unroll
    for (int j = 0; j < R; ++j)
        vw[j] = vt[min(row0 + j * RPI, p.headdim - 1)];

    const int64_t slot = p.idx64 ? load_ro(static_cast<const int64_t *>(p.idx) + b)
                                 : static_cast<int64_t>(load_ro(static_cast<const int32_t *>(p.idx) + b));
    if (slot < 0 || slot >= p.pool_slots)
        return;  // padding
    float *const state = p.state + slot * p.s_slot + h * p.s_head + row0 * p.s_row + 4 * c;
    f32x4 s[R][VEC];
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            s[j][e] = row0 + j * RPI < p.headdim ? load4<true>(state + j * RPI * p.s_row + 128 * e) : f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const float a = exp_f32(load_ro(p.decay + (b * p.d_t + h * p.d_h)));
    const float beta = p.beta ? load_ro(p.beta + (b * p.b_t + h * p.b_h)) : 1.0f;
    f32x4 q[VEC], k[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            q[e][i] = i % 2 ? Bf16::hi(qw[e][i / 2]) : Bf16::lo(qw[e][i / 2]);
            k[e][i] = i % 2 ? Bf16::hi(kw[e][i / 2]) : Bf16::lo(kw[e][i / 2]);
        }
    float qscale = p.scale;
    if (sp.normalize) {
        float qq = 0.0f, kk = 0.0f;
#pragma unroll
        for (int e = 0; e < VEC; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                qq = fmaf(q[e][i], q[e][i], qq);
                kk = fmaf(k[e][i], k[e][i], kk);
            }
        qscale *= inverse_length(sum_lanes<LPR>(qq));
        const float length = inverse_length(sum_lanes<LPR>(kk));
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            k[e] *= length;
    }
    float mine = 0.0f;  // row c of this lane's R
#pragma unroll
    for (int j = 0; j < R; ++j) {
        float x = 0.0f, y = 0.0f;
#pragma unroll
        for (int e = 0; e < VEC; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[j][e][i] *= a;
                x = fmaf(s[j][e][i], k[e][i], x);
            }
        const float u = beta * (Bf16::lo(vw[j]) - sum_lanes<LPR>(x));
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[j][e][i] = fmaf(u, k[e][i], s[j][e][i]);
                y = fmaf(s[j][e][i], q[e][i], y);
            }
            if (row0 + j * RPI < p.headdim)
                store4<true>(state + j * RPI * p.s_row + 128 * e, s[j][e]);
        }
        y = sum_lanes<LPR>(y);
        mine = c == j ? y : mine;
    }
    if (c < R && row0 + c * RPI < p.headdim)
        p.out[b * p.o_t + h * p.o_h + row0 + c * RPI] = Bf16::round(qscale * mine);
}

// Prompts, 32 tokens (a chunk) at a time. With L_i the decays' logarithms summed
// from the chunk's start, S the state before it and k, q normalized if asked:
//
//   u_i = beta_i (v_i - exp(L_i) S k_i - sum_{j < i} exp(L_i - L_j) (k_i . k_j) u_j)
//
// is a triangular system in the chunk's u, the same for all columns p of a head:
// with X its inverse, u = X diag(beta) (v - diag(exp(L)) S k), and
//
//   out_i = scale * ( exp(L_i) S q_i + sum_{j <= i} exp(L_i - L_j) (k_j . q_i) u_j )
//   S     = exp(L_31) S + sum_j exp(L_31 - L_j) u_j k_j^T
//
// What does not depend on the state (X diag(beta), the weights of u in out, the
// exponentials) comes from a first kernel, all chunks and heads at once, as
// fragments of the second kernel's products in bf16 pieces; the second kernel takes
// the chunks of a sequence in order.
//
// Of a chunk and head, in units of 16 bytes (8 KiB in all; what a call writes and reads of
// them is as much as its operands): X's second tile of 16 tokens in 3 pieces, a unit per
// lane, and its first, which has half the places, in 3 of half a unit per lane; the
// weights the same in 2; then 128 floats: exp(L_i) / |k_i|, exp(L_31 - L_i) / |k_i|,
// scale exp(L_i) / |q_i|, and Limits.
constexpr int kXUnits = 3 * 64 + 3 * 32, kSumsAt = kXUnits + 2 * 64 + 2 * 32, kUnits = kSumsAt + 32;

// A chunk's exp(L_31), and the bounds within which it is computed from its fragments: of the
// values that enter the triangle's right side (negative if a fragment is not finite), of the
// state before it, and what the state can gain of such values. Beyond them its tokens
// go one after the other, as infinities and NaN have to.
struct Limits {
    float whole, most, state, gain;
};

// The fragments of tile t, piece e.
__device__ __forceinline__ u32x4 first_half(u32x2 x) { return u32x4{x[0], x[1], 0, 0}; }

__device__ __forceinline__ u32x4 x_of(const u32x4 *x, int t, int e, int lane)
{
    return t ? x[64 * e + lane] : first_half(reinterpret_cast<const u32x2 *>(x + 192 + 32 * e)[lane]);
}

__device__ __forceinline__ u32x4 w_of(const u32x4 *x, int t, int e, int lane)
{
    return t ? x[kXUnits + 64 * e + lane] : first_half(reinterpret_cast<const u32x2 *>(x + kXUnits + 128 + 32 * e)[lane]);
}

struct DeltaParams {
    LinearParams a;
    u32x4 *chunks;  // [chunks, nheads, kUnits]
    int32_t normalize, dstate;
};

// Two values as three bf16 each (2^-24 relative; the last part fits and is cut off).
// (The rests as dot products of pairs, one instruction each, run where the matrix
// instructions do and hold them up; all parts cut off, not rounded, cost the two that
// enter out a bit each.)
__device__ __forceinline__ void split_triple(float x, float y, uint32_t &a, uint32_t &b, uint32_t &c)
{
    a = pack2<Bf16>(x, y);
    const float x1 = x - Bf16::lo(a), y1 = y - Bf16::hi(a);
    b = pack2<Bf16>(x1, y1);
    c = high_halves(__float_as_uint(x1 - Bf16::lo(b)), __float_as_uint(y1 - Bf16::hi(b)));
}

struct Pieces {
    u32x4 a, b, c;
};

__device__ __forceinline__ Pieces split_triple(const f32x4 &x, const f32x4 &y)
{
    Pieces p;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const f32x4 &f = e < 2 ? x : y;
        uint32_t a, b, c;
        split_triple(f[2 * e % 4], f[2 * e % 4 + 1], a, b, c);
        p.a[e] = a;
        p.b[e] = b;
        p.c[e] = c;
    }
    return p;
}

__device__ __forceinline__ f32x4 halves(u32x2 w) { return f32x4{Bf16::lo(w[0]), Bf16::hi(w[0]), Bf16::lo(w[1]), Bf16::hi(w[1])}; }

// The larger of two; of m and x's magnitudes; NaN stays.
__device__ __forceinline__ float larger(float x, float y) { return __builtin_elementwise_maximum(x, y); }

__device__ __forceinline__ float largest(const f32x4 &x, float m)
{
#pragma unroll
    for (int r = 0; r < 4; ++r)
        m = larger(m, fabsf(x[r]));
    return m;
}

template <int MT>
__device__ __forceinline__ float largest(const f32x4 (&x)[MT])
{
    float most = 0.0f;
#pragma unroll
    for (int m = 0; m < MT; ++m)
        most = largest(x[m], most);
    return most;
}

// acc * 0 added up: 0, or NaN if one is not finite.
__device__ __forceinline__ float unless_finite(const f32x4 &x, float zero)
{
#pragma unroll
    for (int r = 0; r < 4; ++r)
        zero = fmaf(x[r], 0.0f, zero);
    return zero;
}

// A wave per chunk and head. The scores of two tiles of 16 tokens come out of the
// products with 4 consecutive j per lane and i = its lane % 16, which is how a
// fragment with rows i wants them. The triangle's diagonal tiles are inverted by
// substitution (a product of powers would lose digits to keys that repeat), a column
// per lane; the tile below them is -X11 L10 X00, in fp32 matrix products, taken
// transposed so that it too comes out as a fragment. 16384 tokens, 32 heads of 128
// (16 of keys): 62 us for 268 MB, which a copy moves in 42; between the two are the vector
// instructions of the splitting, the decays and the substitution.
template <int N>
__global__ void __launch_bounds__(256, 2) ssu_delta_pairs_kernel(const DeltaParams p)
{
    constexpr int KS = N / 32, PITCH = 20;
    const LinearParams &a = p.a;
    __shared__ __attribute__((aligned(16))) float lower[4][2][16 * PITCH + 4], inverse[4][2][16 * PITCH + 4];
    __shared__ __attribute__((aligned(16))) float lsum[4][32], lrest[4][32], lbeta[4][32], lk[4][32], lq[4][32];
    __shared__ int owner;
    __shared__ int64_t found[2];

    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, c = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int blocks = (a.nheads + 3) / 4;
    const int f = static_cast<int>(blockIdx.x) / blocks, h = static_cast<int>(blockIdx.x) % blocks * 4 + wave;

    // chunk f of all: sequence b's are cu[b] / 32 + b and the following (distinct
    // for ordered sequences; otherwise the first to come has it)
    if (tid == 0)
        owner = -1;
    __syncthreads();
    for (int b = tid; b < a.batch; b += 256) {
        const int64_t slot = load_index(a.idx, a.idx64, b);
        const int64_t lo = min(max(static_cast<int64_t>(a.cu[b]), int64_t(0)), a.ntokens);
        const int64_t hi = min(max(static_cast<int64_t>(a.cu[b + 1]), lo), a.ntokens);
        const int64_t s = f - (lo / kChunk + b);
        if (s >= 0 && s * kChunk < hi - lo && slot >= 0 && slot < a.pool_slots && atomicCAS(&owner, -1, b) == -1) {
            found[0] = lo + s * kChunk;
            found[1] = min(hi - (lo + s * kChunk), int64_t(kChunk));
        }
    }
    __syncthreads();
    if (owner < 0 || h >= a.nheads)
        return;
    const int64_t begin = uniform(found[0]);
    const int rows = __builtin_amdgcn_readfirstlane(static_cast<int>(found[1]));
    const int grp = h / a.heads_per_group;

    // rows behind the sequence's end come from its last row and have no gain
    u32x4 kf[2][KS], qf[2][KS];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int64_t row = begin + min(16 * t + c, rows - 1);
        const uint16_t *const kr = a.k + row * a.k_t + grp * a.k_g + 8 * g, *const qr = a.q + row * a.q_t + grp * a.q_g + 8 * g;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const bool in = 32 * s + 8 * g < p.dstate;
            kf[t][s] = in ? *reinterpret_cast<const u32x4_a2 *>(kr + 32 * s) : u32x4{0, 0, 0, 0};
            qf[t][s] = in ? *reinterpret_cast<const u32x4_a2 *>(qr + 32 * s) : u32x4{0, 0, 0, 0};
        }
    }
    const int tok = lane % 32;
    const int64_t own = begin + min(tok, rows - 1);
    const float decay = a.decay[own * a.d_t + h * a.d_h];
    const float gain = a.beta ? a.beta[own * a.b_t + h * a.b_h] : 1.0f;

    // L in units of log 2 and fp64, kept as fp32 and what that leaves
    const bool in = tok < rows;
    double sum = in ? static_cast<double>(decay < kDecayFloor ? kDecayFloor : decay) * 1.4426950408889634 : 0.0;
    sum += lanes_up<0x111, 0xf>(sum);
    sum += lanes_up<0x112, 0xf>(sum);
    sum += lanes_up<0x114, 0xf>(sum);
    sum += lanes_up<0x118, 0xf>(sum);
    sum += lanes_up<0x142, 0xa>(sum);
    const double all = lane_of(sum, 31);
    if (lane < 32) {
        lsum[wave][lane] = static_cast<float>(sum);
        lrest[wave][lane] = static_cast<float>(sum - static_cast<double>(static_cast<float>(sum)));
        lbeta[wave][lane] = in ? gain : 0.0f;
    }

    // scores: rows j (4 g + r of its tile), columns i (c of its)
    f32x4 k00 = {}, k11 = {}, k10 = {}, q00 = {}, q01 = {}, q11 = {};  // k10: rows 16 + 4 g + r, columns c
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        k00 = Mma<Bf16>::run(kf[0][s], kf[0][s], k00);
        k11 = Mma<Bf16>::run(kf[1][s], kf[1][s], k11);
        k10 = Mma<Bf16>::run(kf[1][s], kf[0][s], k10);
        q00 = Mma<Bf16>::run(kf[0][s], qf[0][s], q00);
        q01 = Mma<Bf16>::run(kf[0][s], qf[1][s], q01);
        q11 = Mma<Bf16>::run(kf[1][s], qf[1][s], q11);
    }
    // the squares are the products' diagonals, in lanes c of 4 g .. 4 g + 3
    f32x4 qq0 = {}, qq1 = {};
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        qq0 = Mma<Bf16>::run(qf[0][s], qf[0][s], qq0);
        qq1 = Mma<Bf16>::run(qf[1][s], qf[1][s], qq1);
    }
    auto diagonal = [&](const f32x4 &x) { return c % 4 < 2 ? (c % 4 == 0 ? x[0] : x[1]) : c % 4 == 2 ? x[2] : x[3]; };
    const float kk0 = diagonal(k00), kk1 = diagonal(k11), q0 = diagonal(qq0), q1 = diagonal(qq1);
    const bool has = c / 4 == g;  // (other lanes: no token's)
    const float kk = has ? larger(kk0, kk1) : 0.0f, qq = has ? larger(q0, q1) : 0.0f;
    if (!p.normalize) {
        if (lane < 32)
            lk[wave][lane] = lq[wave][lane] = 1.0f;
    } else if (has) {
        lk[wave][c] = inverse_length(kk0);
        lk[wave][16 + c] = inverse_length(kk1);
        lq[wave][c] = inverse_length(q0);
        lq[wave][16 + c] = inverse_length(q1);
    }
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");

    struct Token {
        float sum, rest, beta, k, q;
    };
    auto token = [&](int i) { return Token{lsum[wave][i], lrest[wave][i], lbeta[wave][i], lk[wave][i], lq[wave][i]}; };
    auto decayed = [](const Token &i, const Token &j) { return __builtin_amdgcn_exp2f((i.sum - j.sum) + (i.rest - j.rest)); };
    const Token at0 = token(c), at1 = token(16 + c);  // i of the columns
    f32x4 beta0, beta1;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int j = 4 * g + r;
        const Token j0 = token(j), j1 = token(16 + j);
        beta0[r] = j0.beta;
        beta1[r] = j1.beta;
        const float d00 = decayed(at0, j0), d11 = decayed(at1, j1), d01 = decayed(at1, j0);
        float x = k00[r] * (at0.beta * d00) * (at0.k * j0.k), y = k11[r] * (at1.beta * d11) * (at1.k * j1.k);
        float z = q00[r] * d00 * (at0.q * j0.k), w = q11[r] * d11 * (at1.q * j1.k);
        asm("" : "+v"(x), "+v"(y), "+v"(z), "+v"(w));  // (selects, not branches around the exponentials)
        k00[r] = j < c ? x : 0.0f;
        k11[r] = j < c ? y : 0.0f;
        q00[r] = a.scale * (j <= c ? z : 0.0f);
        q11[r] = a.scale * (j <= c ? w : 0.0f);
        q01[r] = a.scale * (q01[r] * d01 * (at1.q * j0.k));
        k10[r] = k10[r] * (j1.beta * decayed(j1, at0)) * (j1.k * at0.k);
    }
    *reinterpret_cast<f32x4 *>(&lower[wave][0][c * PITCH + 4 * g]) = k00;
    *reinterpret_cast<f32x4 *>(&lower[wave][1][c * PITCH + 4 * g]) = k11;
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");

    // column c of the inverse of 1 + the tile (of tile g % 2)
    const float *const tile = lower[wave][g % 2];
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float acc = i == c ? 1.0f : 0.0f;
#pragma unroll
        for (int j = 0; j < i; j += 4) {
            const f32x4 l = *reinterpret_cast<const f32x4 *>(tile + i * PITCH + j);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (j + e < i)
                    acc = fmaf(-l[e], x[j + e], acc);
        }
        x[i] = acc;
    }
    if (g < 2)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            inverse[wave][g][i * PITCH + c] = x[i];
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    f32x4 x00 = *reinterpret_cast<const f32x4 *>(&inverse[wave][0][c * PITCH + 4 * g]);
    f32x4 x11 = *reinterpret_cast<const f32x4 *>(&inverse[wave][1][c * PITCH + 4 * g]);
    f32x4 m = {}, x10 = {};
#pragma unroll
    for (int r = 0; r < 4; ++r)
        m = __builtin_amdgcn_mfma_f32_16x16x4f32(k10[r], x11[r], m, 0, 0, 0);
#pragma unroll
    for (int r = 0; r < 4; ++r)
        x10 = __builtin_amdgcn_mfma_f32_16x16x4f32(inverse[wave][0][(4 * g + r) * PITCH + c], m[r], x10, 0, 0, 0);
    x00 *= beta0;
    x10 *= -beta0;
    x11 *= beta1;

    const int64_t id = static_cast<int64_t>(f) * a.nheads + h;
    u32x4 *const out = p.chunks + id * kUnits;
    auto half = [&](int at, uint32_t a, uint32_t b) { reinterpret_cast<u32x2 *>(out + at)[lane] = u32x2{a, b}; };
    const f32x4 none = {0.0f, 0.0f, 0.0f, 0.0f};
    const Pieces x0 = split_triple(x00, none), x1 = split_triple(x10, x11);
    out[lane] = x1.a;
    out[64 + lane] = x1.b;
    out[128 + lane] = x1.c;
    half(192, x0.a[0], x0.a[1]);
    half(192 + 32, x0.b[0], x0.b[1]);
    half(192 + 64, x0.c[0], x0.c[1]);
    u32x4 hi, lo;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const f32x4 &w = e < 2 ? q01 : q11;
        uint32_t wh, wl;
        split_pair(w[2 * e % 4], w[2 * e % 4 + 1], wh, wl);
        hi[e] = wh;
        lo[e] = wl;
    }
    out[kXUnits + lane] = hi;
    out[kXUnits + 64 + lane] = lo;
    uint32_t h0, h1, l0, l1;
    split_pair(q00[0], q00[1], h0, l0);
    split_pair(q00[2], q00[3], h1, l1);
    half(kXUnits + 128, h0, h1);
    half(kXUnits + 160, l0, l1);
    const float grow = __builtin_amdgcn_exp2f(static_cast<float>(sum)), whole = __builtin_amdgcn_exp2f(static_cast<float>(all));
    const float kept = grow * lk[wave][tok], late = in ? __builtin_amdgcn_exp2f(static_cast<float>(all - sum)) * lk[wave][tok] : 0.0f;
    const float asked = a.scale * grow * lq[wave][tok];
    float zero = fmaf(kept, 0.0f, fmaf(late, 0.0f, fmaf(asked, 0.0f, whole * 0.0f)));
    for (const f32x4 &v : {x00, x10, x11, q00, q01, q11})
        zero = unless_finite(v, zero);
    const bool finite = !__any(zero != 0.0f);

    // How large the state and r may be (Limits) so that whatever the recurrence computes of them, here
    // or token by token, stays below 2^127. With D the largest decay between two points of the
    // chunk (1 or more), K, Q the largest lengths of k and q, K' of normalized k, X the largest of
    // the inverse's values: |u| <= 32 X |r|, a state's value between two tokens is
    // D (|S| + 32 K' |u|) at most, a sum of N products of it with k or q 16 K or 16 Q times
    // that, and out |scale| / |q| times it. Of |S| that is 16 D W, of |r| 2^15 X D W K' (what an
    // inverse length of at most 1000 takes u to is less), W = max(1, K, Q, Q |scale| / |q|).
    // r has 2^10 less than that, and up to 8 times what is looked at.
    const float xs = largest(x00, largest(x10, largest(x11, 0.0f))), unit = fabsf(a.scale) * lq[wave][tok];
    // where no decay grows, K, Q <= 2^12, X, |scale| / |q| <= 2^10
    f32x4 limits = {whole, p.normalize ? 0x1p65f : 0x1p53f, 0x1p96f, 0x1p88f};
    if (!__all(!(in && decay > 0.0f) && kk <= 0x1p24f && qq <= 0x1p24f && xs <= 0x1p10f && unit <= 0x1p10f)) {
        auto of_wave = [](float x) {
#pragma unroll
            for (int m = 32; m >= 1; m /= 2)
                x = larger(x, __shfl_xor(x, m));
            return x;
        };
        float low = fminf(static_cast<float>(sum), 0.0f);  // the least sum of decays up to a token
#pragma unroll
        for (int m = 1; m < 32; m *= 2)
            low = fminf(low, __shfl_up(low, m, 32));
        const float D = __builtin_amdgcn_exp2f(of_wave(larger(static_cast<float>(sum) - low, 0.0f)));
        const float X = of_wave(larger(xs, 0x1p-10f));  // (r stays finite)
        const float K = sqrtf(of_wave(larger(kk, 1.0f))), normed = p.normalize ? 1.0f : K;
        const float W = larger(K, sqrtf(of_wave(qq)) * of_wave(larger(unit, 1.0f)));
        limits[1] = 0x1p112f / (0x1p15f * X * D * W * normed);
        limits[2] = 0x1p122f / (16.0f * D * W);
        limits[3] = 0x1p13f * normed * D * X * limits[1];
    }
    limits[1] = finite ? limits[1] : -1.0f;
    float *const s = reinterpret_cast<float *>(out + kSumsAt);
    if (lane < 32) {
        s[lane] = kept;
        s[32 + lane] = late;
        s[64 + lane] = asked;
    }
    if (lane == 0)
        *reinterpret_cast<f32x4 *>(s + 96) = limits;
}

// Where a token's row of k and q in LDS has its 16-byte runs: exchanged by row, so that
// neither 16 rows of one run nor 4 rows of 4 runs (read transposed) have bank conflicts.
template <int N>
__device__ __forceinline__ int run_of(int row, int run)
{
    const int f = N >= 128 ? (row & 3) << 2 | (row >> 2 & 3) : N == 64 ? (row & 2) << 1 | (row >> 2 & 3) : row >> 2 & 3;
    return row * (N / 8) + (run ^ f);
}

// Chunks in order. Waves hold the state in registers as the result tiles of the update's
// product: a lane has, of row p = lane % 16, n = 32 s + 8 g + 0 .. 7. Operands are arranged
// so that nothing is exchanged between lanes: a lane's 8 values are a fragment of the
// products with k and q, 16 bytes of a row of which are the other; S k comes out with 4
// consecutive tokens per lane, and those of two 16-token tiles are a fragment of the
// products with the inverse, as u is of those with k and the weights. Only k for the update
// and v are read transposed, from LDS.

// What a workgroup has of which sequence.
struct Stretch {
    int b, h, col0, total;  // sequence, head, first column, tokens
    int64_t slot, lo;       // its state, its first row
    const uint16_t *k, *q, *v;
    const u32x4 *x;  // its first chunk
};

// Workgroups go round the 8 XCDs: the columns of a head, which share its k, q and
// fragments, beside each other on one.
__device__ __forceinline__ bool stretch_of(const DeltaParams &p, int columns, Stretch &s)
{
    const LinearParams &a = p.a;
    const int id = static_cast<int>(blockIdx.x) / 8, unit = id / a.tiles * 8 + static_cast<int>(blockIdx.x) % 8;
    if (unit >= a.total)
        return false;
    s.b = unit / a.nheads;
    s.h = unit % a.nheads;
    s.col0 = id % a.tiles * columns;
    s.slot = uniform(load_index(a.idx, a.idx64, s.b));
    s.lo = min(max(static_cast<int64_t>(a.cu[s.b]), int64_t(0)), a.ntokens);
    const int64_t hi = min(max(static_cast<int64_t>(a.cu[s.b + 1]), s.lo), a.ntokens);
    s.total = __builtin_amdgcn_readfirstlane(static_cast<int>(hi - s.lo));
    const int grp = s.h / a.heads_per_group;
    s.k = a.k + s.lo * a.k_t + grp * a.k_g;
    s.q = a.q + s.lo * a.q_t + grp * a.q_g;
    s.v = a.v + s.lo * a.v_t + s.h * a.v_h;
    s.x = p.chunks + ((s.lo / kChunk + s.b) * a.nheads + s.h) * kUnits;
    return s.slot >= 0 && s.slot < a.pool_slots && s.total > 0;
}

__device__ __forceinline__ u32x4 at_bytes(const uint16_t *base, uint32_t off)
{
    return *reinterpret_cast<const u32x4_a2 *>(reinterpret_cast<const char *>(base) + off);
}

// What does not depend on the state of a chunk, as the first kernel left it.
__device__ __forceinline__ const float *sums_of(const u32x4 *x) { return reinterpret_cast<const float *>(x + kSumsAt); }

__device__ __forceinline__ Limits limits_of(const float *sums)
{
    const f32x4 x = *reinterpret_cast<const f32x4 *>(sums + 96);
    return {x[0], x[1], x[2], x[3]};
}

template <int N, int MT>
__device__ __forceinline__ void load_state(const DeltaParams &p, const Stretch &s, int p0, int n0, f32x4 (&st)[MT], bool store)
{
    const LinearParams &a = p.a;
    const int c = static_cast<int>(threadIdx.x) & 15;
    float *const pool = a.state + s.slot * a.s_slot + s.h * a.s_head + (p0 + c) * a.s_row + n0;
    const bool in = p0 < a.headdim && (N >= 64 || n0 < p.dstate);  // (N = 16 in a tile of 32)
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        float *const at = pool + 32 * (m / 2) + 4 * (m % 2);
        if (!store)
            st[m] = in ? *reinterpret_cast<const f32x4 *>(at) : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        else if (in)
            *reinterpret_cast<f32x4 *>(at) = st[m];
    }
}

// The tokens t0 .. of a chunk one after the other, as in the kernel of steps: where a
// value is not finite the pieces in 16 bits make NaN of infinities, and NaN of one token would
// reach those before it through the inverse's zeros. All WN waves of a column come here.
template <int N, int MT, int WN>
__device__ __forceinline__ void by_tokens(const DeltaParams &p, const Stretch &s, int t0, int p0, int n0, int wn, f32x4 (&st)[MT],
                                          float (*box)[WN][64])
{
    const LinearParams &a = p.a;
    const int lane = static_cast<int>(threadIdx.x) & 63, c = lane & 15, g = lane >> 4;
    const bool in_n = N >= 64 || n0 < p.dstate;
    const int t1 = min(t0 + kChunk, s.total);
    // the sum over this wave's n, then over the waves' (through box[turn])
    auto whole_sum = [&](float x, int turn) {
        x += __shfl_xor(x, 16);
        x += __shfl_xor(x, 32);
        if constexpr (WN > 1) {
            box[turn][wn][lane] = x;
            __syncthreads();
            x = box[turn][0][lane];
#pragma unroll
            for (int w = 1; w < WN; ++w)
                x += box[turn][w][lane];
        }
        return x;
    };
    // of all n of a row: every wave for itself, before anything is multiplied with the row
    auto length_of = [&](const uint16_t *row) {
        if (!p.normalize)
            return 1.0f;
        const f32x4 x = 4 * lane < p.dstate ? halves(*reinterpret_cast<const u32x2_a2 *>(row + 4 * lane)) : f32x4{};
        return inverse_length(sum_lanes<64>(fmaf(x[3], x[3], fmaf(x[2], x[2], fmaf(x[1], x[1], x[0] * x[0])))));
    };
#pragma unroll 1
    for (int t = t0; t < t1; ++t) {
        const int64_t tok = s.lo + t;
        const float keep = exp_f32(a.decay[tok * a.d_t + s.h * a.d_h]);
        const float beta = a.beta ? a.beta[tok * a.b_t + s.h * a.b_h] : 1.0f;
        const uint16_t *const kr = s.k + t * a.k_t, *const qr = s.q + t * a.q_t;
        auto values = [&](const uint16_t *row, int m) {
            return in_n ? halves(*reinterpret_cast<const u32x2_a2 *>(row + n0 + 32 * (m / 2) + 4 * (m % 2))) : f32x4{};
        };
        const float klength = length_of(kr), qlength = length_of(qr);
        float x = 0.0f, y = 0.0f;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const f32x4 k = klength * values(kr, m);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (in_n)  // (an infinite decay times the zeros behind N is NaN)
                    st[m][e] *= keep;
                x = fmaf(st[m][e], k[e], x);
            }
        }
        const float u = beta * (Bf16::lo(s.v[t * a.v_t + min(p0 + c, a.headdim - 1)]) - whole_sum(x, 0));
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const f32x4 k = klength * values(kr, m), q = values(qr, m);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (in_n)  // (as is an infinite u)
                    st[m][e] = fmaf(u, k[e], st[m][e]);
                y = fmaf(st[m][e], q[e], y);
            }
        }
        y = whole_sum(y, 1);
        if (wn == 0 && g == 0 && p0 < a.headdim)
            a.out[tok * a.o_t + s.h * a.o_h + p0 + c] = Bf16::round(a.scale * qlength * y);
    }
}

// The chunk's u (rows tokens, columns p) from r, and its pieces for the update.
__device__ __forceinline__ void solve(const u32x4 (&x)[2][3], const f32x4 (&r)[2], f32x4 (&u)[2])
{
    const Pieces f = split_triple(r[0], r[1]);
    u[0] = u[1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // the smallest products first, the two tiles in turn
#pragma unroll
    for (int e = 0; e < 6; ++e)
#pragma unroll
        for (int t = 0; t < 2; ++t)
            u[t] = Mma<Bf16>::run(x[t][e == 1 || e == 4 ? 1 : e == 2 ? 2 : 0], e == 0 ? f.c : e == 1 || e == 3 ? f.b : f.a, u[t]);
}

// 16 tokens of out (rows p, columns tokens) from S q and u, stored.
__device__ __forceinline__ void write_out(const DeltaParams &p, const Stretch &s, int row0, int p0, const f32x4 &sq, float asked,
                                          const f32x4 (&u)[2], u32x4 wh, u32x4 wl)
{
    const LinearParams &a = p.a;
    const int g = (static_cast<int>(threadIdx.x) & 63) >> 4, c = static_cast<int>(threadIdx.x) & 15;
    u32x4 uh, ul;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        uint32_t h, l;
        split_pair(u[e / 2][2 * e % 4], u[e / 2][2 * e % 4 + 1], h, l);
        uh[e] = h;
        ul[e] = l;
    }
    f32x4 o = asked * sq;
    o = Mma<Bf16>::run(ul, wh, o);
    o = Mma<Bf16>::run(uh, wl, o);
    o = Mma<Bf16>::run(uh, wh, o);
    if (row0 + c < s.total && p0 < a.headdim)
        *reinterpret_cast<u32x2_a2 *>(reinterpret_cast<char *>(a.out + (s.lo + row0) * a.o_t + s.h * a.o_h + p0) +
                                      2 * (c * static_cast<uint32_t>(a.o_t) + 4 * g)) =
            u32x2{pack2<Bf16>(o[0], o[1]), pack2<Bf16>(o[2], o[3])};
}

// Few columns of heads: a chunk's time is the length of its chain of instructions, one wave on
// a SIMD, so that what is not part of it is done by others. WN waves share the N of 16
// columns out; their shares of S k are added up through LDS, one barrier a chunk, and what
// follows every wave computes for itself. Two waves, a chunk behind, write out what u and the shares of S q
// give for a tile of 16 tokens each. Two more bring operands into LDS, requested three
// chunks ahead. One prompt of 16384 tokens, 32 heads of 128 x 128: 535 us, 1 us a chunk,
// about 2300 cycles of a chain wave's instructions, of which a wave alone on its SIMD starts one
// in 5.6 cycles; with the N on two waves 695 us, on one 878 (both with the first kernel).
template <int N, int WN>
__global__ void __launch_bounds__(64 * (WN + 4)) ssu_delta_narrow_kernel(const DeltaParams p)
{
    constexpr int NW = N / WN, KS = NW / 32, MT = NW / 16, VP = 32;
    constexpr int RK = 32 * N / 8, UK = (RK + 127) / 128, UX = (kXUnits + 127) / 128;
    struct Stage {
        u32x4 k[RK], q[RK], x[128 * UX];  // (x: as many as the loads; a branch would make their waits longer)
        float sums[128];
        uint16_t v[kChunk * VP];
    };
    __shared__ __attribute__((aligned(16))) Stage ring[2];
    __shared__ f32x4 shares_k[WN > 1 ? 2 : 1][WN][2][64], shares_q[3][WN][2][64], lu[2][2][64];
    __shared__ float bad[2][WN];
    __shared__ float box[2][WN][64];

    const LinearParams &a = p.a;
    Stretch s;
    if (!stretch_of(p, 16, s))
        return;
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, c = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), chunks = (s.total + kChunk - 1) / kChunk;
    const int64_t stride = static_cast<int64_t>(a.nheads) * kUnits;
    auto any_bad = [&](int i) {
        float y = bad[i & 1][0];
#pragma unroll
        for (int w = 1; w < WN; ++w)
            y += bad[i & 1][w];
        return __builtin_amdgcn_readfirstlane(__float_as_int(y)) != 0;
    };
    // the barriers of a chunk that goes token by token
    auto stand_by = [&](int i) {
        if (WN > 1)
            for (int n = 2 * min(s.total - i * kChunk, kChunk); n > 0; --n)
                __syncthreads();
    };

    if (wave >= WN + 2) {  // chunk i + 1 into LDS before barrier i
        const int lt = tid - 64 * (WN + 2);
        struct Load {
            u32x4 k[UK], q[UK], x[UX], v;
        } even, odd;
        // byte offsets from a chunk's first row; rows behind the end come from the last one
        uint32_t ok[UK], oq[UK], ov = 0;
        auto offsets = [&](int last) {
#pragma unroll
            for (int e = 0; e < UK; ++e) {
                const int u = lt + 128 * e, n = u % (N / 8) * 8, col = N >= 64 || n < p.dstate ? n : 0;
                const uint32_t row = min(u / (N / 8) % 32, last);
                ok[e] = 2 * (row * static_cast<uint32_t>(a.k_t) + col);
                oq[e] = 2 * (row * static_cast<uint32_t>(a.q_t) + col);
            }
            ov = 2 * (min(lt % 64 / 2, last) * static_cast<uint32_t>(a.v_t) + s.col0 + 8 * (lt % 2));
        };
        auto request = [&](int i, Load &l) {
            const int ci = min(i, chunks - 1);
            const int64_t row = static_cast<int64_t>(ci) * kChunk;
            if (s.total - ci * kChunk < kChunk)
                offsets(s.total - ci * kChunk - 1);
#pragma unroll
            for (int e = 0; e < UK; ++e) {
                l.k[e] = at_bytes(s.k + row * a.k_t, ok[e]);
                l.q[e] = at_bytes(s.q + row * a.q_t, oq[e]);
            }
            const u32x4 *const x = s.x + ci * stride;
#pragma unroll
            for (int e = 0; e < UX; ++e)
                l.x[e] = x[min(lt + 128 * e, kXUnits - 1)];
            // v by the first wave, the sums by the second
            l.v = wave == WN + 2 ? at_bytes(s.v + row * a.v_t, ov) : x[kSumsAt + lt % 32];
        };
        offsets(kChunk - 1);
        auto turn = [&](int i, Load &l) {
            Stage &to = ring[(i + 1) & 1];
#pragma unroll
            for (int e = 0; e < UK; ++e) {
                const int u = lt + 128 * e, row = u / (N / 8), run = u % (N / 8);
                const bool in = N >= 64 || run * 8 < p.dstate;
                if (RK % 128 == 0 || u < RK) {
                    to.k[run_of<N>(row, run)] = in ? l.k[e] : u32x4{0, 0, 0, 0};
                    to.q[run_of<N>(row, run)] = in ? l.q[e] : u32x4{0, 0, 0, 0};
                }
            }
#pragma unroll
            for (int e = 0; e < UX; ++e)
                to.x[lt + 128 * e] = l.x[e];
            if (lt < 64)
                *reinterpret_cast<u32x4 *>(&to.v[lt / 2 * VP + 8 * (lt % 2)]) = l.v;
            else if (lt < 96)
                reinterpret_cast<u32x4 *>(to.sums)[lt - 64] = l.v;
            request(i + 3, l);
            __syncthreads();
            if (i == chunks)
                return true;
            if (i >= 0 && any_bad(i))
                stand_by(i);
            return false;
        };
        request(0, odd);
        request(1, even);
#pragma unroll 1
        for (int i = -1; !turn(i, odd) && !turn(i + 1, even); i += 2) {
        }
        return;
    }
    if (wave >= WN) {  // out of chunk i - 1 behind barrier i
        const int t = wave - WN;
        struct Weights {
            float asked;
            u32x4 hi, lo;
        } even, odd;
        bool skip = true;
        auto turn = [&](int i, const Weights &last, Weights &now) {
            const u32x4 *const x = s.x + min(i, chunks - 1) * stride;
            // (both tiles by the same loads: a branch around them would be waited for)
            const char *const at = reinterpret_cast<const char *>(x + kXUnits + 128 * (1 - t)) + lane * (8 + 8 * t);
            const u32x2 h = *reinterpret_cast<const u32x2 *>(at), l = *reinterpret_cast<const u32x2 *>(at + 512 + 512 * t);
            const u32x2 h1 = *reinterpret_cast<const u32x2 *>(at + 8 * t), l1 = *reinterpret_cast<const u32x2 *>(at + 512 + 520 * t);
            now = {sums_of(x)[64 + 16 * t + c], u32x4{h[0], h[1], h1[0], h1[1]}, u32x4{l[0], l[1], l1[0], l1[1]}};
            __syncthreads();
            if (!skip) {
                const f32x4 u[2] = {lu[(i - 1) & 1][0][lane], lu[(i - 1) & 1][1][lane]};
                const int from = (i - 1) % 3;
                f32x4 sq = shares_q[from][0][t][lane];
#pragma unroll
                for (int w = 1; w < WN; ++w)
                    sq += shares_q[from][w][t][lane];
                write_out(p, s, (i - 1) * kChunk + 16 * t, s.col0, sq, last.asked, u, t ? last.hi : first_half(u32x2{last.hi[0], last.hi[1]}),
                          t ? last.lo : first_half(u32x2{last.lo[0], last.lo[1]}));
            }
            if (i == chunks)
                return true;
            skip = any_bad(i);
            if (skip)
                stand_by(i);
            return false;
        };
        __syncthreads();  // the first chunk's operands
#pragma unroll 1
        for (int i = 0; !turn(i, odd, even) && !turn(i + 1, even, odd); i += 2) {
        }
        return;
    }

    const int wn = wave, n0 = wn * NW + 8 * g;
    f32x4 st[MT];
    load_state<N>(p, s, s.col0, n0, st, false);
    __syncthreads();
    // what a chunk needs besides the state, read from LDS as soon as the chunk before no
    // longer needs the registers: nothing of it is waited for
    u32x4 kf[KS][2], qf[KS][2], xf[2][3], kt[MT];
    u32x2 vf[2];
    f32x4 kept[2], late[2];
    Limits limits;
    float whole, reach = INFINITY;  // (reach: no value of this wave's state is larger)
    auto read_first = [&](const Stage &at) {
#pragma unroll
        for (int e = 0; e < KS; ++e)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                kf[e][t] = at.k[run_of<N>(16 * t + c, wn * (NW / 8) + 4 * e + g)];
                qf[e][t] = at.q[run_of<N>(16 * t + c, wn * (NW / 8) + 4 * e + g)];
            }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            vf[t] = read_transposed(&at.v[(16 * t + 4 * g + c / 4) * VP + 4 * (c % 4)]);
            kept[t] = *reinterpret_cast<const f32x4 *>(&at.sums[16 * t + 4 * g]);
        }
        limits = limits_of(at.sums);
    };
    auto read_x = [&](const Stage &at) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 3; ++e)
                xf[t][e] = x_of(at.x, t, e, lane);
    };
    auto read_last = [&](const Stage &at) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
            late[t] = *reinterpret_cast<const f32x4 *>(&at.sums[32 + 16 * t + 4 * g]);
        whole = at.sums[96];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int row = 4 * g + c / 4, run = wn * (NW / 8) + 4 * (m / 2) + c % 4;
            auto of = [&](int r) { return reinterpret_cast<const uint16_t *>(&at.k[run_of<N>(r, run)]) + 4 * (m % 2); };
            const u32x2 x = read_transposed(of(row)), y = read_transposed(of(row + 16));
            kt[m] = u32x4{x[0], x[1], y[0], y[1]};
        }
    };
    read_first(ring[0]);
    read_x(ring[0]);
    read_last(ring[0]);
#pragma unroll 1
    for (int i = 0; i < chunks; ++i) {
        const Stage &next = ring[(i + 1) & 1];
        // S k (rows tokens, columns p) and S q (rows p, columns tokens), this wave's n
        f32x4 sk[2] = {}, sq[2] = {};
#pragma unroll
        for (int e = 0; e < KS; ++e) {
            const Pieces f = split_triple(st[2 * e], st[2 * e + 1]);
#pragma unroll
            for (int t = 0; t < 2; ++t)
                sk[t] = Mma<Bf16>::run(kf[e][t], f.c, sk[t]);
#pragma unroll
            for (int t = 0; t < 2; ++t)
                sk[t] = Mma<Bf16>::run(kf[e][t], f.b, sk[t]);
#pragma unroll
            for (int t = 0; t < 2; ++t)
                sk[t] = Mma<Bf16>::run(kf[e][t], f.a, sk[t]);
#pragma unroll
            for (int t = 0; t < 2; ++t)
                sq[t] = Mma<Bf16>::run(f.b, qf[e][t], sq[t]);
#pragma unroll
            for (int t = 0; t < 2; ++t)
                sq[t] = Mma<Bf16>::run(f.a, qf[e][t], sq[t]);
        }
        const f32x4 v[2] = {halves(vf[0]), halves(vf[1])};
        // whether all of it is within its limits (sk: this wave's share of up to 4), and its sums:
        // the other waves know of it as soon as these do
        float most = 0.0f;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            sk[t] *= kept[t];
            most = largest(sk[t], largest(v[t], most));
        }
        if (__any(!(reach <= limits.state))) {
            reach = largest(st);
            most = reach <= limits.state ? most : INFINITY;
        }
        bad[i & 1][wn] = __any(!(most <= limits.most)) ? 1.0f : 0.0f;
        reach = fmaf(reach, whole, limits.gain);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if (WN > 1)
                shares_k[i & 1][wn][t][lane] = sk[t];
            shares_q[i % 3][wn][t][lane] = sq[t];
        }
        __syncthreads();

        f32x4 r[2], u[2];
        const bool slow = any_bad(i);
        asm volatile("");  // (read here, not where it is asked)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if constexpr (WN > 1) {
                sk[t] = shares_k[i & 1][0][t][lane];
#pragma unroll
                for (int w = 1; w < WN; ++w)
                    sk[t] += shares_k[i & 1][w][t][lane];
            }
            r[t] = v[t] - sk[t];
        }
        solve(xf, r, u);
        read_first(next);
        read_x(next);
        if (__builtin_expect(!slow, 1)) {
            if (wn == 0) {
                lu[i & 1][0][lane] = u[0];
                lu[i & 1][1][lane] = u[1];
            }
            const Pieces f = split_triple(late[0] * u[0], late[1] * u[1]);
#pragma unroll
            for (int e = 0; e < 3; ++e)
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    if (e == 0)
                        st[m] *= whole;
                    st[m] = Mma<Bf16>::run(kt[m], e == 0 ? f.c : e == 1 ? f.b : f.a, st[m]);
                }
        } else {
            by_tokens<N, MT, WN>(p, s, i * kChunk, s.col0, n0, wn, st, box);
            reach = INFINITY;
        }
        read_last(next);
    }
    __syncthreads();  // the last u
    load_state<N>(p, s, s.col0, n0, st, true);
}

// Many columns: a wave has all N of 16 of them, kWideWaves waves as many of one head. They share
// a chunk's operands, which go through one stage in LDS, requested while the chunk before is
// worked on, two barriers a chunk: what covers a wave's waits is the other waves of its
// SIMD, two to four of them, and the one stage is what leaves room for them. 16 prompts of up to
// 2048 tokens, 32 heads of 128 x 128: 224 us. Two stages and two waves took 298, eight
// waves to a stage 337, 32 columns to a wave 373. What bounds it: vector instructions
// of three waves beside the matrix products (under which the clock falls to 1.7 GHz), and
// at the end the longest prompt, alone.
constexpr int kWideWaves = 4;

template <int N>
__global__ void __launch_bounds__(64 * kWideWaves, N == 256 ? 2 : N == 128 ? 3 : 4) ssu_delta_wide_kernel(const DeltaParams p)
{
    constexpr int THREADS = 64 * kWideWaves, KS = N / 32, MT = N / 16;
    constexpr int PC = 16 * kWideWaves, VP = PC + 16;  // columns, pitch in LDS
    constexpr int KP = N / 8 + (N == 32 ? 1 : 5);      // of k and q: a multiple of 16 runs and 5 (13)
    constexpr int RK = 32 * N / 8, RV = 32 * PC / 8;  // runs of 16 bytes
    constexpr int UK = (RK + THREADS - 1) / THREADS, UV = (RV + THREADS - 1) / THREADS, UX = (kUnits + THREADS - 1) / THREADS;
    struct Stage {
        u32x4 k[32 * KP], q[32 * KP], x[kUnits];
        uint16_t v[kChunk * VP];
    };
    __shared__ __attribute__((aligned(16))) Stage at;

    const LinearParams &a = p.a;
    Stretch s;
    if (!stretch_of(p, PC, s))
        return;
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, c = lane & 15, g = lane >> 4;
    const int wc = __builtin_amdgcn_readfirstlane(tid >> 6), chunks = (s.total + kChunk - 1) / kChunk;
    const int p0 = s.col0 + 16 * wc;

    // Requests of a chunk; rows behind the end come from the last one, columns behind P
    // and N from the first.
    u32x4 rk[UK], rq[UK], rv[UV], rx[UX];
    uint32_t ok[UK], oq[UK], ov[UV];  // byte offsets from a chunk's first row
    auto offsets = [&](int last) {     // of a chunk with rows 0 .. last
#pragma unroll
        for (int e = 0; e < UK; ++e) {
            const int u = tid + THREADS * e, n = u % (N / 8) * 8, col = N >= 64 || n < p.dstate ? n : 0;
            const uint32_t row = min(u / (N / 8), last);
            ok[e] = 2 * (row * static_cast<uint32_t>(a.k_t) + col);
            oq[e] = 2 * (row * static_cast<uint32_t>(a.q_t) + col);
        }
#pragma unroll
        for (int e = 0; e < UV; ++e) {
            const int u = tid + THREADS * e, col = s.col0 + u % (PC / 8) * 8;
            ov[e] = 2 * (min(u / (PC / 8), last) * static_cast<uint32_t>(a.v_t) + (col < a.headdim ? col : 0));
        }
    };
    auto request = [&](int i) {
        const int64_t row = static_cast<int64_t>(i) * kChunk;
        if (s.total - i * kChunk < kChunk)
            offsets(s.total - i * kChunk - 1);
#pragma unroll
        for (int e = 0; e < UK; ++e) {
            rk[e] = at_bytes(s.k + row * a.k_t, ok[e]);
            rq[e] = at_bytes(s.q + row * a.q_t, oq[e]);
        }
#pragma unroll
        for (int e = 0; e < UV; ++e)
            rv[e] = at_bytes(s.v + row * a.v_t, ov[e]);
#pragma unroll
        for (int e = 0; e < UX; ++e)
            rx[e] = s.x[static_cast<int64_t>(i) * a.nheads * kUnits + min(tid + THREADS * e, kUnits - 1)];
    };
    auto place = [&] {
#pragma unroll
        for (int e = 0; e < UK; ++e) {
            const int u = tid + THREADS * e, row = u / (N / 8), run = u % (N / 8);
            if (RK % THREADS == 0 || u < RK) {
                const bool in = N >= 64 || run * 8 < p.dstate;
                at.k[row * KP + run] = in ? rk[e] : u32x4{0, 0, 0, 0};
                at.q[row * KP + run] = in ? rq[e] : u32x4{0, 0, 0, 0};
            }
        }
#pragma unroll
        for (int e = 0; e < UV; ++e) {
            const int u = tid + THREADS * e;
            if (RV % THREADS == 0 || u < RV)
                *reinterpret_cast<u32x4 *>(at.v + u / (PC / 8) * VP + u % (PC / 8) * 8) = rv[e];
        }
#pragma unroll
        for (int e = 0; e < UX; ++e) {
            const int u = tid + THREADS * e;
            if (kUnits % THREADS == 0 || u < kUnits)
                at.x[u] = rx[e];
        }
    };
    offsets(kChunk - 1);
    request(0);
    f32x4 st[MT];
    load_state<N>(p, s, p0, 8 * g, st, false);
    float reach = INFINITY;  // no value of the state is larger
    place();
    __syncthreads();

#pragma unroll 1
    for (int i = 0; i < chunks; ++i) {
        const float *const sums = sums_of(at.x);

        // S k (rows tokens, columns p) and S q (rows p, columns tokens)
        f32x4 sk[2] = {}, sq[2] = {};
#pragma unroll
        for (int e = 0; e < KS; ++e) {
            u32x4 kf[2], qf[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                kf[t] = at.k[(16 * t + c) * KP + 4 * e + g];
                qf[t] = at.q[(16 * t + c) * KP + 4 * e + g];
            }
            const Pieces f = split_triple(st[2 * e], st[2 * e + 1]);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                sk[t] = Mma<Bf16>::run(kf[t], f.c, sk[t]);
                sq[t] = Mma<Bf16>::run(f.b, qf[t], sq[t]);
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                sk[t] = Mma<Bf16>::run(kf[t], f.b, sk[t]);
                sq[t] = Mma<Bf16>::run(f.a, qf[t], sq[t]);
            }
#pragma unroll
            for (int t = 0; t < 2; ++t)
                sk[t] = Mma<Bf16>::run(kf[t], f.a, sk[t]);
        }
        __builtin_amdgcn_sched_barrier(0);
        f32x4 r[2], u[2];
        float most = 0.0f;
        u32x4 xf[2][3];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 3; ++e)
                xf[t][e] = x_of(at.x, t, e, lane);
        const int vtr = (4 * g + c / 4) * VP + 4 * (c % 4) + 16 * wc;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const f32x4 kept = *reinterpret_cast<const f32x4 *>(sums + 16 * t + 4 * g);
            r[t] = halves(read_transposed(at.v + vtr + 16 * t * VP));
#pragma unroll
            for (int e = 0; e < 4; ++e)
                r[t][e] = fmaf(-kept[e], sk[t][e], r[t][e]);
            most = largest(r[t], most);
        }
        solve(xf, r, u);
        const Limits limits = limits_of(sums);
        if (__any(!(reach <= limits.state))) {
            reach = largest(st);
            most = reach <= limits.state ? most : INFINITY;
        }
        __builtin_amdgcn_sched_barrier(0);
        if (__builtin_expect(__all(most <= limits.most), 1)) {
            // the state behind the chunk
            const float whole = limits.whole;
            reach = fmaf(reach, whole, limits.gain);
            const Pieces f = split_triple(*reinterpret_cast<const f32x4 *>(sums + 32 + 4 * g) * u[0],
                                          *reinterpret_cast<const f32x4 *>(sums + 48 + 4 * g) * u[1]);
            constexpr int MB = MT < 4 ? MT : 4;  // tiles at a time
#pragma unroll
            for (int m0 = 0; m0 < MT; m0 += MB) {
                __builtin_amdgcn_sched_barrier(0);
                u32x4 kt[MB];
#pragma unroll
                for (int m = 0; m < MB; ++m) {
                    const int row = 4 * g + c / 4, run = 4 * ((m0 + m) / 2) + c % 4;
                    auto of = [&](int r) { return reinterpret_cast<const uint16_t *>(&at.k[r * KP + run]) + 4 * (m % 2); };
                    const u32x2 x = read_transposed(of(row)), y = read_transposed(of(row + 16));
                    kt[m] = u32x4{x[0], x[1], y[0], y[1]};
                }
#pragma unroll
                for (int e = 0; e < 3; ++e)
#pragma unroll
                    for (int m = 0; m < MB; ++m) {
                        if (e == 0)
                            st[m0 + m] *= whole;
                        st[m0 + m] = Mma<Bf16>::run(kt[m], e == 0 ? f.c : e == 1 ? f.b : f.a, st[m0 + m]);
                    }
            }
            __builtin_amdgcn_sched_barrier(0);
            request(min(i + 1, chunks - 1));
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                write_out(p, s, i * kChunk + 16 * t, p0, sq[t], sums[64 + 16 * t + c], u, w_of(at.x, t, 0, lane),
                          w_of(at.x, t, 1, lane));
                __builtin_amdgcn_sched_barrier(0);
            }
        } else {
            by_tokens<N, MT, 1>(p, s, i * kChunk, p0, 8 * g, 0, st, nullptr);
            reach = INFINITY;
            request(min(i + 1, chunks - 1));
        }
        __syncthreads();
        place();
        __syncthreads();
    }
    load_state<N>(p, s, p0, 8 * g, st, true);
}

using StepFn = void (*)(StepParams);

struct StepKernel {
    StepFn fn;
    int rows;  // of the state per workgroup
};

// LOADS dwordx4 of state per lane.
template <int N, int LOADS>
constexpr StepKernel step_kernel()
{
    constexpr int VEC = N > 128 ? N / 128 : 1;
    return {&ssu_delta_step_kernel<N, LOADS / VEC>, 64 / (N / (4 * VEC)) * LOADS / VEC};
}

template <int LOADS>
StepKernel step_kernel(int N)
{
    switch (N) {
    case 16: return step_kernel<16, LOADS>();
    case 32: return step_kernel<32, LOADS>();
    case 64: return step_kernel<64, LOADS>();
    case 128: return step_kernel<128, LOADS>();
    default: return step_kernel<256, LOADS>();
    }
}

using DeltaFn = void (*)(DeltaParams);

struct ChunkKernel {
    DeltaFn fn;
    int waves, columns;
};

template <int N, int WN>
constexpr ChunkKernel narrow_kernel()
{
    return {&ssu_delta_narrow_kernel<N, WN>, WN + 4, 16};
}

template <int N>
constexpr ChunkKernel wide_kernel()
{
    return {&ssu_delta_wide_kernel<N>, kWideWaves, 16 * kWideWaves};
}

// tiles: of 16 columns, of all sequences and heads. More than two for each compute unit
// fill the SIMDs with waves that have all N; fewer take the shortest chain for each (both
// kernels together, us, narrow against wide: N = 128, 512 tiles of ragged prompts 95 and 158,
// 1024 169 and 169, 1024 of equal ones 316 and 210; N = 64: 83 and 123, 147 and 126; N = 256,
// 512 tiles 114 and 218, 1024 209 and 226, 2048 413 and 296). The N of a column
// goes to as many waves as have 32 of them, at most 4 (16384 tokens, 32 heads of 128 x 128: 4
// waves 591, 2 695, 1 878).
ChunkKernel chunk_kernel(int N, int64_t tiles)
{
    const bool many = tiles > 2 * kNumCUs;
    if (N <= 32)
        return many ? wide_kernel<32>() : narrow_kernel<32, 1>();
    if (N == 64)
        return many ? wide_kernel<64>() : narrow_kernel<64, 2>();
    if (N == 128)
        return many ? wide_kernel<128>() : narrow_kernel<128, 4>();
    return many ? wide_kernel<256>() : narrow_kernel<256, 4>();
}

// ------------------------------------------------------------------ host --

ssu_status check_delta(const ssu_delta_args &a, const char *who, bool prompts)
{
    if (a.normalize != 0 && a.normalize != 1)
        return fail(SSU_ERR_INVALID_ARGUMENT, "%s: normalize must be 0 or 1", who);
    return check_linear(a, who, prompts);
}

// Launch of a step as linear attention's, by the bytes of state that it moves one way: 2 KiB
// of it a wave, 4 KiB from 8 MiB on, and from 40 and 128 MiB on 16 and 14 waves to a
// compute unit, no more. 253 requests, 32 heads of 128 x 128: 169 us, 6.3 TB/s, what a large
// copy reaches; one request 4.0 us, the launch and slot, then state, then the two sums.
ssu_status launch_step(const ssu_delta_args &a, hipStream_t stream)
{
    const int64_t mib = static_cast<int64_t>(a.batch) * a.nheads * a.headdim * a.dstate >> 18;
    const StepKernel k = mib < 8 ? step_kernel<2>(a.dstate) : step_kernel<4>(a.dstate);
    StepParams p{linear_params(a), a.normalize};
    p.a.tiles = (a.headdim + k.rows - 1) / k.rows;
    const int64_t groups = static_cast<int64_t>(a.batch) * a.nheads * p.a.tiles;
    SSU_TRY(check_launch(groups, 64, "ssu_gated_delta_rule_step"));
    p.a.total = static_cast<int>(groups);
    DeviceGuard guard;
    SSU_TRY(guard.enter(a.device));
    size_t lds = 0;
    if (mib >= 40) {
        int dev = 0;
        if (hipGetDevice(&dev) != hipSuccess)
            return fail(SSU_ERR_HIP, "hipGetDevice failed");
        const DeviceLimits lim = device_limits(dev);
        lds = lds_for_cap(mib < 128 ? 16 : 14, lim.lds_cu, lim.lds_block);
    }
    const hipError_t e = launch_kernel(k.fn, p, groups, 64, lds, stream);
    if (e != hipSuccess)
        return fail(SSU_ERR_HIP, "launch of the delta rule's step failed: %s", hipGetErrorString(e));
    return SSU_OK;
}

int64_t chunks_of(const ssu_delta_args &a) { return a.ntokens / kChunk + a.batch; }

int64_t workspace_of(const ssu_delta_args &a)
{
    return a.ntokens == 0 ? 0 : chunks_of(a) * a.nheads * kUnits * 16;
}

ssu_status launch_chunks(const ssu_delta_args &a, hipStream_t stream)
{
    const int64_t bytes = workspace_of(a);
    if (!a.workspace || a.workspace_bytes < bytes)
        return fail(SSU_ERR_INVALID_ARGUMENT, "ssu_gated_delta_rule: workspace of %lld bytes, %lld needed",
                    static_cast<long long>(a.workspace ? a.workspace_bytes : 0), static_cast<long long>(bytes));
    if (reinterpret_cast<uintptr_t>(a.workspace) % 16)
        return fail(SSU_ERR_MISALIGNED, "ssu_gated_delta_rule: workspace must be 16-byte aligned");
    const int64_t units = static_cast<int64_t>(a.batch) * a.nheads;
    const ChunkKernel k = chunk_kernel(a.dstate, units * (a.headdim / 16));
    DeltaParams p{};
    p.a = linear_params(a);
    p.a.tiles = (a.headdim + k.columns - 1) / k.columns;
    p.a.total = static_cast<int>(units);
    p.normalize = a.normalize;
    p.dstate = a.dstate;
    p.chunks = static_cast<u32x4 *>(a.workspace);
    const int64_t first = chunks_of(a) * ((a.nheads + 3) / 4), second = (units + 7) / 8 * 8 * p.a.tiles;
    SSU_TRY(check_launch(first, 256, "ssu_gated_delta_rule"));
    SSU_TRY(check_launch(second, 64 * k.waves, "ssu_gated_delta_rule"));
    const DeltaFn pairs = a.dstate <= 32 ? &ssu_delta_pairs_kernel<32> : a.dstate == 64 ? &ssu_delta_pairs_kernel<64>
                        : a.dstate == 128 ? &ssu_delta_pairs_kernel<128> : &ssu_delta_pairs_kernel<256>;
    DeviceGuard guard;
    SSU_TRY(guard.enter(a.device));
    hipError_t e = launch_kernel(pairs, p, first, 256, 0, stream);
    if (e == hipSuccess)
        e = launch_kernel(k.fn, p, second, 64 * k.waves, 0, stream);
    if (e != hipSuccess)
        return fail(SSU_ERR_HIP, "launch of the chunked delta rule failed: %s", hipGetErrorString(e));
    return SSU_OK;
}

}  // namespace
}  // namespace ssu

extern "C" {

int64_t ssu_gated_delta_rule_workspace(const ssu_delta_args *a)
{
    using namespace ssu;
    if (!a || check_sizes(*a, "ssu_gated_delta_rule_workspace") != SSU_OK)
        return -1;
    return workspace_of(*a);
}

ssu_status ssu_gated_delta_rule(const ssu_delta_args *a, hipStream_t stream)
{
    using namespace ssu;
    if (!a)
        return fail(SSU_ERR_INVALID_ARGUMENT, "ssu_gated_delta_rule: null args");
    SSU_TRY(check_delta(*a, "ssu_gated_delta_rule", true));
    if (a->batch == 0 || a->ntokens == 0)
        return SSU_OK;
    return launch_chunks(*a, stream);
}

ssu_status ssu_gated_delta_rule_step(const ssu_delta_args *a, hipStream_t stream)
{
    using namespace ssu;
    if (!a)
        return fail(SSU_ERR_INVALID_ARGUMENT, "ssu_gated_delta_rule_step: null args");
    SSU_TRY(check_delta(*a, "ssu_gated_delta_rule_step", false));
    if (a->batch == 0)
        return SSU_OK;
    return launch_step(*a, stream);
}

}  // extern "C"
