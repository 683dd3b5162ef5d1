// linear_attention.hip -- linear attention with a decay for each head on MI355X
// (gfx950): ssu_linear_attention over whole prompts, ssu_linear_attention_step
// for one token per request. The operation is stated in include/ssu.h.

#include <hip/hip_runtime.h>

#include <algorithm>
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

// One token per request. One wave owns RPI * R rows p of one (request, head): a
// row's N values are split over LPR = N / 4 lanes (N = 256: 32 lanes with two
// chunks), one dwordx4 each, so that one instruction moves 1 KiB of contiguous
// state. Memory-bound by the state, read and written once: what does not
// depend on the slot is requested first (vector loads return in order, so
// nothing may wait behind the state), the slot and the head's decay and gain go
// through the scalar cache, and the state goes past the caches.
template <int N, int R>
__global__ void __launch_bounds__(64) ssu_linear_step_kernel(const LinearParams p)
{
    constexpr int VEC = N > 128 ? N / 128 : 1;
    constexpr int LPR = N / (4 * VEC);
    constexpr int RPI = 64 / LPR;
    static_assert(R <= LPR, "one writer lane per row");
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
    float *const sp = p.state + slot * p.s_slot + h * p.s_head + row0 * p.s_row + 4 * c;
    f32x4 s[R][VEC];
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            s[j][e] = row0 + j * RPI < p.headdim ? load4<true>(sp + j * RPI * p.s_row + 128 * e) : f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const float a = exp_f32(load_ro(p.decay + (b * p.d_t + h * p.d_h)));
    const float beta = p.beta ? load_ro(p.beta + (b * p.b_t + h * p.b_h)) : 1.0f;
    float y[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const float v = beta * Bf16::lo(vw[j]);
        float acc = 0.0f;
#pragma unroll
        for (int e = 0; e < VEC; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float k = i % 2 ? Bf16::hi(kw[e][i / 2]) : Bf16::lo(kw[e][i / 2]);
                const float q = i % 2 ? Bf16::hi(qw[e][i / 2]) : Bf16::lo(qw[e][i / 2]);
                s[j][e][i] = fmaf(s[j][e][i], a, v * k);
                acc = fmaf(s[j][e][i], q, acc);
            }
        y[j] = acc;
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (row0 + j * RPI < p.headdim)
                store4<true>(sp + j * RPI * p.s_row + 128 * e, s[j][e]);
    }
    float mine = 0.0f;  // row c of this lane's R
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const float sum = sum_lanes<LPR>(y[j]);
        mine = c == j ? sum : mine;
    }
    if (c < R && row0 + c * RPI < p.headdim)
        p.out[b * p.o_t + h * p.o_h + row0 + c * RPI] = Bf16::round(p.scale * mine);
}

// Prompts, 32 tokens (a chunk) at a time. With L_i the decays' logarithms summed
// from the chunk's start, S the state before it:
//
//   out_i = scale * ( exp(L_i) S q_i + sum_{j <= i} exp(L_i - L_j) beta_j (k_j . q_i) v_j )
//   S     = exp(L_31) S + sum_j exp(L_31 - L_j) beta_j v_j k_j^T
//
// One workgroup of W waves takes a segment of a sequence, one head and 16 W
// columns of v (rows p of the state); wave w owns columns 16 w .. 16 w + 15,
// whose state stays in its registers as the result tiles of the second line's
// product. Places of a contracted axis may stand for any value as long as both
// operands agree, which is used so that nothing is exchanged between lanes:
//
//  - a lane's state values of two tiles, 4 consecutive n each, are a fragment of
//    S q (as a bf16 pair, value and remainder), against two 8-byte runs of q;
//  - the scores k_j . q_i come out with 4 consecutive j per lane, and those of
//    two 16-token tiles are a fragment of their product with v; the waves share
//    the tiles out and pass them on through LDS, also as a pair;
//  - k for the update and v for both products are read from LDS transposed
//    (ds_read_b64_tr_b16: 4 rows of 16 values become 4 values per lane).
//
// The update's operand exp(L_31 - L_j) beta_j v_j is split into three bf16 (2^-24
// relative): the state is fp32 and is handed on. L is summed in fp64 and in
// units of log 2: a difference of two sums keeps its digits behind a reset.
//
// Long sequences are cut into segments: a first kernel (FULL = false) computes
// every segment's own contribution to the state, a second the states in front
// of the segments from them, and the third starts every segment there.
constexpr int kChunk = 32;
constexpr int kTiles = kChunk / 16;  // of tokens: a product's 32 places hold both
constexpr float kDecayFloor = -1.0e4f;  // exp is 0 far above it; sums of it stay finite

struct ChunkParams {
    LinearParams a;
    float *states;  // [segments, nheads, headdim, dstate]
    float *decays;  // [segments, nheads]: a segment's whole decay, log2 of it
    int32_t seg_len, slices, dstate;
};

__device__ __forceinline__ void split_pair(float x, float y, uint32_t &hi, uint32_t &lo)
{
    hi = pack2<Bf16>(x, y);
    lo = pack2<Bf16>(x - Bf16::lo(hi), y - Bf16::hi(hi));
}

// A double from other lanes by DPP (zero where the lane has no source or its
// row is not in MASK), and one lane's in all.
template <int CTRL, int MASK>
__device__ __forceinline__ double lanes_up(double x)
{
    const uint64_t v = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, MASK, 0xf, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(v >> 32), CTRL, MASK, 0xf, true);
    return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

__device__ __forceinline__ double lane_of(double x, int lane)
{
    const uint64_t v = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(v), lane);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(v >> 32), lane);
    return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

__device__ __forceinline__ int64_t uniform(int64_t x)
{
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<int>(x));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<int>(x >> 32));
    return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}

// 4 rows of 16 16-bit values in LDS, the lane's address being that of values
// 4 (l % 4) .. of row (l % 16) / 4 of its 16 lanes' rows: the lane gets value
// l % 16 of each.
__device__ __forceinline__ u32x2 read_transposed(const uint16_t *p)
{
    using S4 = short __attribute__((ext_vector_type(4)));
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                         (__attribute__((address_space(3))) S4 *)(const_cast<uint16_t *>(p))));
}

// DENSE: four waves per SIMD, whose instructions are enough for each other's waits;
// otherwise three (N = 128), which read the operands of several products ahead
// (chunk_kernels says which).
template <int N, int W, bool FULL, bool DENSE>
__global__ void __launch_bounds__(64 * W, N == 256 ? 2 : FULL && !DENSE ? 3 : 4) ssu_linear_chunk_kernel(const ChunkParams p)
{
    constexpr int THREADS = 64 * W;
    constexpr int MT = N / 16;        // state tiles along n
    constexpr int KS = N / 32;        // products along n of a score
    constexpr int AHEAD = DENSE ? 1 : KS < 4 ? KS : 4;  // of them, read ahead
    constexpr int MAHEAD = DENSE ? 1 : MT < 8 ? MT : 8;  // the same of state tiles
    constexpr bool PART = N * kChunk / 8 < THREADS;  // not every thread has a run of q and k
    constexpr int PC = 16 * W;        // columns of v
    // pitches in LDS: 16 rows of 8 or 16 bytes, and 4 rows of 32, in banks of their own
    constexpr int ROW = N == 32 ? 56 : N == 64 ? 72 : N + 24;
    constexpr int VROW = W == 4 ? 72 : 152;
    constexpr int QU = (N * kChunk / 8 + THREADS - 1) / THREADS;  // 16-byte runs of q and of k per thread
    constexpr int VU = PC * kChunk / 8 / THREADS;                 // of v
    __shared__ __attribute__((aligned(16))) uint16_t lq[FULL ? kChunk * ROW : 8];
    __shared__ __attribute__((aligned(16))) uint16_t lk[kChunk * ROW];
    __shared__ __attribute__((aligned(16))) uint16_t lv[kChunk * VROW];
    __shared__ u32x4 lw[FULL ? kTiles : 1][2][64];  // scores: token tile, value / remainder, lane
    // of THREADS tokens: L in units of log 2, as fp32 and what that leaves, and what follows from it
    __shared__ __attribute__((aligned(16))) float lsum[THREADS], lrest[THREADS], lbeta[THREADS], lgrow[THREADS], llate[THREADS];
    __shared__ float lall[THREADS / kChunk];
    __shared__ double whole[W];  // the segment's log decay so far, of every wave's tokens
    __shared__ int owner;         // this segment's sequence
    __shared__ int64_t found[3];  // its slot and rows

    const LinearParams &a = p.a;
    // workgroups go round the 8 XCDs: XCD x has segments x, x + 8, ..., all heads
    // and slices of a segment (which share its q and k) beside each other
    const int inner = a.nheads * p.slices, id = static_cast<int>(blockIdx.x) / 8;
    const int f = id / inner * 8 + static_cast<int>(blockIdx.x) % 8;
    const int h = id % inner / p.slices, slice = id % p.slices, grp = h / a.heads_per_group;
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, c = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    // segment f of all: sequence b's are cu[b] / seg_len + b and the following
    // (distinct for ordered sequences; otherwise the first to come has it)
    if (tid == 0)
        owner = -1;
    __syncthreads();
    for (int b = tid; b < a.batch; b += THREADS) {
        const int64_t slot = load_index(a.idx, a.idx64, b);
        const int64_t lo = min(max(static_cast<int64_t>(a.cu[b]), int64_t(0)), a.ntokens);
        const int64_t hi = min(max(static_cast<int64_t>(a.cu[b + 1]), lo), a.ntokens);
        const int64_t s = f - (lo / p.seg_len + b);
        if (s >= 0 && s * p.seg_len < hi - lo && slot >= 0 && slot < a.pool_slots && atomicCAS(&owner, -1, b) == -1) {  // (padding: none)
            found[0] = slot;
            found[1] = lo;
            found[2] = hi;
        }
    }
    __syncthreads();
    const int b = __builtin_amdgcn_readfirstlane(owner);
    if (b < 0)
        return;
    const int64_t slot = uniform(found[0]), lo = uniform(found[1]), hi = uniform(found[2]);
    const int base = static_cast<int>(lo / p.seg_len) + b, seg = f - base;
    const int segs = static_cast<int>((hi - lo + p.seg_len - 1) / p.seg_len);
    const int64_t begin = lo + static_cast<int64_t>(seg) * p.seg_len;
    const int rows = __builtin_amdgcn_readfirstlane(static_cast<int>(min(hi - begin, static_cast<int64_t>(p.seg_len))));
    if (!FULL && seg == segs - 1)
        return;  // nothing comes behind it

    const int p0 = slice * PC + wave * 16;  // this wave's first column
    const bool live = p0 < a.headdim;
    const int prow = p0 + c;                // this lane's
    float *const pool = a.state + slot * a.s_slot + h * a.s_head;
    const int64_t plane = static_cast<int64_t>(a.headdim) * p.dstate;

    // the lane's values of row `prow`: n = 16 m + 4 g + 0 .. 3
    f32x4 st[MT];
    auto load_state = [&](const float *src, int64_t row) {
        if (!live)
            return;
        src += prow * row + 4 * g;
#pragma unroll
        for (int m = 0; m < MT; ++m)
            if (16 * m < p.dstate)
                st[m] = *reinterpret_cast<const f32x4 *>(src + 16 * m);
    };
    auto store_state = [&](float *dst, int64_t row) {
        if (!live)
            return;
        dst += prow * row + 4 * g;
#pragma unroll
        for (int m = 0; m < MT; ++m)
            if (16 * m < p.dstate)
                *reinterpret_cast<f32x4 *>(dst + 16 * m) = st[m];
    };

    // requests of a chunk: rows behind the segment's end come from its last row
    // and count as zeros
    u32x4 rq[QU], rk[QU], rv[VU];
    float rdecay = 0.0f, rbeta = 0.0f;
    const uint32_t oo = 2 * (c * static_cast<uint32_t>(a.o_t) + 4 * g);  // of out: this lane's 4 values of token c
    uint32_t oq[QU], ok[QU], ov[VU];  // byte offsets from a chunk's first row
    auto offsets = [&](int last) {     // of a chunk with rows 0 .. last
#pragma unroll
        for (int i = 0; i < QU; ++i) {
            const int u = tid + THREADS * i, n = u % (N / 8) * 8, col = n < p.dstate ? n : 0;
            const uint32_t t = min(u / (N / 8), last);
            oq[i] = 2 * (t * static_cast<uint32_t>(a.q_t) + col);
            ok[i] = 2 * (t * static_cast<uint32_t>(a.k_t) + col);
        }
#pragma unroll
        for (int i = 0; i < VU; ++i) {
            const int u = tid + THREADS * i, col = u % (PC / 8) * 8;
            ov[i] = 2 * (min(u / (PC / 8), last) * static_cast<uint32_t>(a.v_t) + (slice * PC + col < a.headdim ? col : 0));
        }
    };
    auto at = [](const uint16_t *base, uint32_t off) {
        return *reinterpret_cast<const u32x4_a2 *>(reinterpret_cast<const char *>(base) + off);
    };
    const uint16_t *qt = a.q + begin * a.q_t + grp * a.q_g, *kt = a.k + begin * a.k_t + grp * a.k_g;  // of the next request
    const uint16_t *vt = a.v + begin * a.v_t + h * a.v_h + slice * PC;
    auto request = [&](int t0) {
        if (rows - t0 < kChunk)
            offsets(rows - t0 - 1);
#pragma unroll
        for (int i = 0; i < QU; ++i) {
            if constexpr (FULL)
                rq[i] = at(qt, oq[i]);
            rk[i] = at(kt, ok[i]);
        }
#pragma unroll
        for (int i = 0; i < VU; ++i)
            rv[i] = at(vt, ov[i]);
        qt += kChunk * a.q_t;
        kt += kChunk * a.k_t;
        vt += kChunk * a.v_t;
    };
    // L and what follows from it for as many tokens as the workgroup has threads:
    // a wave has two chunks, and a chunk waits for its sums once in 2 W
    auto request_sums = [&](int t0) {  // (behind the segment's end: of its last token)
        const int64_t t = begin + min(t0 + tid, rows - 1);
        rdecay = a.decay[t * a.d_t + h * a.d_h];
        rbeta = a.beta ? a.beta[t * a.b_t + h * a.b_h] : 1.0f;
    };
    auto sums = [&](int t0) {
        const bool in = t0 + tid < rows;
        const float d = rdecay < kDecayFloor ? kDecayFloor : rdecay;  // (NaN stays)
        double sum = in ? static_cast<double>(d) * 1.4426950408889634 : 0.0;
        sum += lanes_up<0x111, 0xf>(sum);  // lane - 1, - 2, - 4, - 8 of each 16
        sum += lanes_up<0x112, 0xf>(sum);
        sum += lanes_up<0x114, 0xf>(sum);
        sum += lanes_up<0x118, 0xf>(sum);
        sum += lanes_up<0x142, 0xa>(sum);  // the last of 16 to the next 16
        const double first = lane_of(sum, 31), second = lane_of(sum, 63), all = lane < kChunk ? first : second;
        const float gain = in ? rbeta : 0.0f;
        lsum[tid] = static_cast<float>(sum);
        lrest[tid] = static_cast<float>(sum - static_cast<double>(static_cast<float>(sum)));
        lbeta[tid] = gain;
        lgrow[tid] = __builtin_amdgcn_exp2f(static_cast<float>(sum));
        llate[tid] = in ? gain * __builtin_amdgcn_exp2f(static_cast<float>(all - sum)) : 0.0f;
        if (lane % kChunk == 0)
            lall[tid / kChunk] = __builtin_amdgcn_exp2f(static_cast<float>(all));
        if (!FULL && lane == 0)
            whole[wave] = t0 == 0 ? first + second : whole[wave] + (first + second);
    };
    auto place = [&](int t0) {
        // zeros behind the segment's end, behind N (16 in a tile of 32) and behind P
        const bool cut = t0 + kChunk > rows || p.dstate < N || slice * PC + PC > a.headdim;
        if (cut) {
#pragma unroll
            for (int i = 0; i < QU; ++i) {
                const int u = tid + THREADS * i;
                if (t0 + u / (N / 8) >= rows || u % (N / 8) * 8 >= p.dstate) {
                    rk[i] = u32x4{0, 0, 0, 0};
                    if constexpr (FULL)
                        rq[i] = u32x4{0, 0, 0, 0};
                }
            }
#pragma unroll
            for (int i = 0; i < VU; ++i) {
                const int u = tid + THREADS * i;
                if (t0 + u / (PC / 8) >= rows || slice * PC + u % (PC / 8) * 8 >= a.headdim)
                    rv[i] = u32x4{0, 0, 0, 0};
            }
        }
#pragma unroll
        for (int i = 0; i < QU; ++i) {
            const int u = tid + THREADS * i, at = u / (N / 8) * ROW + u % (N / 8) * 8;
            if (PART && u >= N * kChunk / 8)
                break;
            if constexpr (FULL)
                *reinterpret_cast<u32x4 *>(lq + at) = rq[i];
            *reinterpret_cast<u32x4 *>(lk + at) = rk[i];
        }
#pragma unroll
        for (int i = 0; i < VU; ++i) {
            const int u = tid + THREADS * i;
            *reinterpret_cast<u32x4 *>(lv + u / (PC / 8) * VROW + u % (PC / 8) * 8) = rv[i];
        }
    };

    offsets(kChunk - 1);
    request_sums(0);
    request(0);
    auto start = [&] {  // the state before the segment
#pragma unroll
        for (int m = 0; m < MT; ++m)
            st[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if constexpr (FULL) {
            if (segs == 1)
                load_state(pool, a.s_row);
            else
                load_state(p.states + (static_cast<int64_t>(f) * a.nheads + h) * plane, p.dstate);
        }
    };
    start();
    if constexpr (FULL)  // (the tiles above the diagonal stay zero)
        for (int i = tid; i < kTiles * 2 * 64; i += THREADS)
            (&lw[0][0][0])[i] = u32x4{0, 0, 0, 0};
    sums(0);
    request_sums(THREADS);
    place(0);
    __syncthreads();

    float zero = 0.0f;  // or NaN: an output was not finite
    uint16_t *out = a.out + begin * a.o_t + h * a.o_h + p0;
    for (int t0 = 0; t0 < rows; t0 += kChunk) {
        const int next = t0 + kChunk;
        const bool more = next < rows;
        const int at0 = t0 % THREADS;  // of the chunk's sums
        if (more)
            request(next);

        // v of the wave's columns as fragments: 8 tokens of 32 per lane
        const int tr = (4 * g + c / 4) * ROW + 4 * (c % 4), vtr = (4 * g + c / 4) * VROW + 4 * (c % 4) + wave * 16;
        const u32x2 v0 = read_transposed(lv + vtr), v1 = read_transposed(lv + 16 * VROW + vtr);
        const u32x4 vf = {v0[0], v0[1], v1[0], v1[1]};

        if constexpr (FULL) {
            // weighted scores of the pairs of 16-token tiles (it, jt <= it), dealt
            // out to the waves; result rows j = 16 jt + 4g + r, columns
            // i = 16 it + c
            static_assert(kTiles == 2 && W >= 3, "three pairs, one for a wave");
            if (const int pair = wave; pair < 3) {
                const int it = pair >= 1 ? 1 : 0, jt = pair >= 2 ? 1 : 0;
                f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int e0 = 0; e0 < KS; e0 += AHEAD) {
                    u32x4 kf[AHEAD], qf[AHEAD];
#pragma unroll
                    for (int e = 0; e < AHEAD; ++e) {
                        kf[e] = *reinterpret_cast<const u32x4 *>(lk + (16 * jt + c) * ROW + 32 * (e0 + e) + 8 * g);
                        qf[e] = *reinterpret_cast<const u32x4 *>(lq + (16 * it + c) * ROW + 32 * (e0 + e) + 8 * g);
                    }
#pragma unroll
                    for (int e = 0; e < AHEAD; ++e)
                        x = Mma<Bf16>::run(kf[e], qf[e], x);
                }
                const float li = lsum[at0 + 16 * it + c], ri = lrest[at0 + 16 * it + c];
                const f32x4 lj = *reinterpret_cast<const f32x4 *>(&lsum[at0 + 16 * jt + 4 * g]);
                const f32x4 rj = *reinterpret_cast<const f32x4 *>(&lrest[at0 + 16 * jt + 4 * g]);
                const f32x4 bj = *reinterpret_cast<const f32x4 *>(&lbeta[at0 + 16 * jt + 4 * g]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float y = x[r] * (bj[r] * __builtin_amdgcn_exp2f((li - lj[r]) + (ri - rj[r])));
                    asm("" : "+v"(y));  // (a select, not a branch around the exponential)
                    x[r] = 16 * jt + 4 * g + r <= 16 * it + c ? y : 0.0f;
                }
                uint32_t h0, h1, l0, l1;
                split_pair(x[0], x[1], h0, l0);
                split_pair(x[2], x[3], h1, l1);
                *(reinterpret_cast<u32x2 *>(&lw[it][0][lane]) + jt) = u32x2{h0, h1};
                *(reinterpret_cast<u32x2 *>(&lw[it][1][lane]) + jt) = u32x2{l0, l1};
            }

            // S q, all tokens: result rows p, columns i
            f32x4 o[kTiles];
#pragma unroll
            for (int it = 0; it < kTiles; ++it)
                o[it] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            u32x4 qf[AHEAD][kTiles];
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                if (s % AHEAD == 0)
#pragma unroll
                    for (int e = 0; e < AHEAD; ++e)
#pragma unroll
                        for (int it = 0; it < kTiles; ++it) {
                            const uint16_t *const qrow = lq + (16 * it + c) * ROW + 32 * (s + e) + 4 * g;
                            const u32x2 x = *reinterpret_cast<const u32x2 *>(qrow), y = *reinterpret_cast<const u32x2 *>(qrow + 16);
                            qf[e][it] = u32x4{x[0], x[1], y[0], y[1]};
                        }
                u32x4 fh, fl;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t wh, wl;
                    split_pair(st[2 * s + e / 2][2 * (e % 2)], st[2 * s + e / 2][2 * (e % 2) + 1], wh, wl);
                    fh[e] = wh;
                    fl[e] = wl;
                }
#pragma unroll
                for (int it = 0; it < kTiles; ++it)
                    o[it] = Mma<Bf16>::run(fh, qf[s % AHEAD][it], o[it]);
#pragma unroll
                for (int it = 0; it < kTiles; ++it)
                    o[it] = Mma<Bf16>::run(fl, qf[s % AHEAD][it], o[it]);
            }
#pragma unroll
            for (int it = 0; it < kTiles; ++it)
                o[it] *= lgrow[at0 + 16 * it + c];
            __syncthreads();  // the scores are there
#pragma unroll
            for (int it = 0; it < kTiles; ++it) {
                o[it] = Mma<Bf16>::run(vf, lw[it][0][lane], o[it]);
                o[it] = Mma<Bf16>::run(vf, lw[it][1][lane], o[it]);
            }
#pragma unroll
            for (int it = 0; it < kTiles; ++it)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    zero = fmaf(o[it][r], 0.0f, zero);
            if (live) {
#pragma unroll
                for (int it = 0; it < kTiles; ++it)
                    if (t0 + 16 * it + c < rows)
                        *reinterpret_cast<u32x2_a2 *>(reinterpret_cast<char *>(out + it * 16 * a.o_t) + oo) =
                            u32x2{pack2<Bf16>(a.scale * o[it][0], a.scale * o[it][1]),
                                  pack2<Bf16>(a.scale * o[it][2], a.scale * o[it][3])};
                out += kChunk * a.o_t;
            }
        }

        // the state behind the chunk
        const float all = lall[at0 / kChunk];
#pragma unroll
        for (int m = 0; m < MT; ++m)
            st[m] *= all;
        u32x4 f1, f2, f3;
        const f32x4 late0 = *reinterpret_cast<const f32x4 *>(&llate[at0 + 4 * g]);
        const f32x4 late1 = *reinterpret_cast<const f32x4 *>(&llate[at0 + 16 + 4 * g]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const f32x4 &late = e < 2 ? late0 : late1;
            const float x = Bf16::lo(vf[e]) * late[2 * e % 4], y = Bf16::hi(vf[e]) * late[2 * e % 4 + 1];
            const uint32_t h1 = pack2<Bf16>(x, y);
            const float x1 = x - Bf16::lo(h1), y1 = y - Bf16::hi(h1);
            const uint32_t h2 = pack2<Bf16>(x1, y1);
            f1[e] = h1;
            f2[e] = h2;
            f3[e] = pack2<Bf16>(x1 - Bf16::lo(h2), y1 - Bf16::hi(h2));
        }
#pragma unroll
        for (int m0 = 0; m0 < MT; m0 += MAHEAD) {
            u32x4 kf[MAHEAD];
#pragma unroll
            for (int m = 0; m < MAHEAD; ++m) {
                const u32x2 x = read_transposed(lk + tr + 16 * (m0 + m)), y = read_transposed(lk + 16 * ROW + tr + 16 * (m0 + m));
                kf[m] = u32x4{x[0], x[1], y[0], y[1]};
            }
#pragma unroll
            for (const u32x4 &f : {f1, f2, f3})
#pragma unroll
                for (int m = 0; m < MAHEAD; ++m)
                    st[m0 + m] = Mma<Bf16>::run(kf[m], f, st[m0 + m]);
        }
        if (more) {
            __syncthreads();  // LDS is free again
            if (next % THREADS == 0) {
                sums(next);
                request_sums(next + THREADS);
            }
            place(next);
            __syncthreads();
        }
    }

    // Not finite: the pieces in 16 bits make NaN of infinities, a zero times the growth
    // of a chunk that fp32 does not hold is one too, and NaN stays. Then the segment
    // goes through the recurrence again, token by token, as in the kernel of steps
    // (finite data pays for the checks less than a measurement shows; a NaN in one of 16
    // prompts of 1 to 2048 tokens makes 81 us 1.5 ms).
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            zero = fmaf(st[m][e], 0.0f, zero);
    if (live && __any(zero != 0.0f)) {
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "agent");  // (behind this wave's own outputs)
        start();
#pragma unroll 1
        for (int64_t t = begin; t < begin + rows; ++t) {
            const float keep = exp_f32(a.decay[t * a.d_t + h * a.d_h]);
            const float x = (a.beta ? a.beta[t * a.b_t + h * a.b_h] : 1.0f) * Bf16::lo(a.v[t * a.v_t + h * a.v_h + prow]);
            const uint16_t *const kr = a.k + t * a.k_t + grp * a.k_g + 4 * g, *const qr = a.q + t * a.q_t + grp * a.q_g + 4 * g;
            float y = 0.0f;
#pragma unroll
            for (int m = 0; m < MT; ++m)
                if (16 * m < p.dstate) {
                    const u32x2 kw = *reinterpret_cast<const u32x2_a2 *>(kr + 16 * m), qw = *reinterpret_cast<const u32x2_a2 *>(qr + 16 * m);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        st[m][e] = fmaf(st[m][e], keep, x * (e % 2 ? Bf16::hi(kw[e / 2]) : Bf16::lo(kw[e / 2])));
                        y = fmaf(st[m][e], e % 2 ? Bf16::hi(qw[e / 2]) : Bf16::lo(qw[e / 2]), y);
                    }
                }
            if constexpr (FULL) {
                y += __shfl_xor(y, 16);
                y += __shfl_xor(y, 32);
                if (g == 0)
                    a.out[t * a.o_t + h * a.o_h + prow] = Bf16::round(a.scale * y);
            }
        }
    }

    if constexpr (FULL) {
        if (seg == segs - 1)
            store_state(pool, a.s_row);
    } else {
        store_state(p.states + (static_cast<int64_t>(f) * a.nheads + h) * plane, p.dstate);
        if (slice == 0 && tid == 0) {
            double log_decay = whole[0];
#pragma unroll
            for (int w = 1; w < W; ++w)
                log_decay += whole[w];
            p.decays[static_cast<int64_t>(f) * a.nheads + h] = static_cast<float>(log_decay);
        }
    }
}

// The states in front of a sequence's segments, in place of the segments' own
// contributions: four consecutive values of one head per thread.
__global__ void __launch_bounds__(256) ssu_linear_segments_kernel(const ChunkParams p)
{
    const LinearParams &a = p.a;
    const int plane = a.headdim * p.dstate, blocks = (plane + 1023) / 1024;
    const int id = static_cast<int>(blockIdx.x), h = id / blocks % a.nheads, b = id / blocks / a.nheads;
    const int i = (id % blocks * 256 + static_cast<int>(threadIdx.x)) * 4;
    const int64_t slot = load_index(a.idx, a.idx64, b);
    const int64_t lo = min(max(static_cast<int64_t>(a.cu[b]), int64_t(0)), a.ntokens);
    const int64_t hi = min(max(static_cast<int64_t>(a.cu[b + 1]), lo), a.ntokens);
    const int segs = static_cast<int>((hi - lo + p.seg_len - 1) / p.seg_len);
    if (slot < 0 || slot >= a.pool_slots || segs <= 1 || i >= plane)
        return;
    const int64_t first = (lo / p.seg_len + b) * a.nheads + h, step = static_cast<int64_t>(a.nheads) * plane;
    f32x4 s = *reinterpret_cast<const f32x4 *>(a.state + slot * a.s_slot + h * a.s_head + i / p.dstate * a.s_row + i % p.dstate);
    float *at = p.states + first * plane + i;
    const float *decay = p.decays + first;
    constexpr int U = 8;  // segments on their way at once
    for (int t = 0; t < segs; t += U) {
        f32x4 x[U];
        float d[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (t + u < segs - 1) {
                x[u] = *reinterpret_cast<const f32x4 *>(at + u * step);
                d[u] = decay[static_cast<int64_t>(t + u) * a.nheads];
            }
        const f32x4 s0 = s;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t + u < segs)
                *reinterpret_cast<f32x4 *>(at + u * step) = s;
            if (t + u < segs - 1)
                s = s * __builtin_amdgcn_exp2f(d[u]) + x[u];
        }
        // Not finite (and so it stays): a decay over a whole segment may have left fp32
        // where the tokens' own, one after the other, leave an infinity infinite, a zero
        // 0 and a tiny value finite.
        if (__builtin_expect(!__builtin_isfinite((s[0] + s[1]) + (s[2] + s[3])), 0)) {
            s = s0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (t + u < segs)
                    *reinterpret_cast<f32x4 *>(at + u * step) = s;
                if (t + u < segs - 1) {
                    bool reset = false;  // (a token's own decay is 0)
                    const int64_t r0 = lo + static_cast<int64_t>(t + u) * p.seg_len;
                    for (int r = 0; r < p.seg_len; ++r)
                        reset |= exp_f32(a.decay[(r0 + r) * a.d_t + h * a.d_h]) == 0.0f;
                    const float whole = __builtin_amdgcn_exp2f(d[u]), half = __builtin_amdgcn_exp2f(0.5f * d[u]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float kept = __builtin_isinf(s[e]) ? s[e] * (reset ? 0.0f : 1.0f) : whole < INFINITY ? s[e] * whole : s[e] * half * half;
                        s[e] = s[e] == 0.0f ? x[u][e] : kept + x[u][e];
                    }
                }
            }
        }
        at += U * step;
    }
}

using LinearFn = void (*)(LinearParams);

struct StepKernel {
    LinearFn fn;
    int rows;  // of the state per workgroup
};

// LOADS dwordx4 of state per lane.
template <int N, int LOADS>
constexpr StepKernel step_kernel()
{
    constexpr int VEC = N > 128 ? N / 128 : 1;
    return {&ssu_linear_step_kernel<N, LOADS / VEC>, 64 / (N / (4 * VEC)) * LOADS / VEC};
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

using ChunkFn = void (*)(ChunkParams);

struct ChunkKernels {
    ChunkFn states, full;
    int columns;  // of v per workgroup
};

template <int N, int W, bool DENSE>
constexpr ChunkKernels chunk_kernels()
{
    return {&ssu_linear_chunk_kernel<N, W, false, W == 8>, &ssu_linear_chunk_kernel<N, W, true, DENSE>, 16 * W};
}

// Eight waves where they share the products of q and k of whole heads and their
// states fit four waves per SIMD: N = 128, P in 80 .. 128 (one prompt of 16384
// tokens, 32 heads of 128 x 128: 226 us, 270 with four waves; a head of 64 x 128
// has columns for four only). Four elsewhere: more workgroups to hide each other's
// waits (4 prompts of 3000, 8 heads of 128 x 64: 34.5 us against 36.9; of
// 128 x 256: 68.7 against 92.2; of 224 x 128: 62.5 against 77.6).
//
// Those of four read ahead (a prompt of 37 tokens 9.1 us against 9.7 dense, 16 of 1
// to 2048 tokens 82 against 84.5), unless there are more of N = 128 than three waves
// per SIMD hold (32 prompts of 700 tokens, 16 heads of 224 x 128: 144 against 129);
// eight always are dense (the prompt of 16384 tokens 252 us otherwise).
ChunkKernels chunk_kernels(int N, int P, int64_t waves)
{
    if (N == 128 && P > 64 && P <= 128)
        return chunk_kernels<128, 8, true>();
    if (N == 128 && waves > 12 * kNumCUs)
        return chunk_kernels<128, 4, true>();
    return N <= 32 ? chunk_kernels<32, 4, false>() : N == 64 ? chunk_kernels<64, 4, false>()
         : N == 128 ? chunk_kernels<128, 4, false>() : chunk_kernels<256, 4, false>();
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
    if (a.ntokens > 0x7ffff000)  // (a segment and two workgroups' tokens count in 32 bits)
        return fail(SSU_ERR_UNSUPPORTED, "%s: more than 2^31 tokens", who);
    if ((a.ntokens / kChunk + a.batch + 8) * a.nheads > 0x7fffffff / (a.headdim / 16))
        return fail(SSU_ERR_UNSUPPORTED, "%s: batch * nheads too large", who);
    return SSU_OK;
}

// Segments of a prompt call.
struct Plan {
    int seg_len, segments, slices;
    int64_t waves;             // of all sequences, uncut
    int64_t decays_at, bytes;  // workspace (0: one segment per sequence)
};

// Sequences are cut where whole ones would leave most of the chip idle: at most
// one wave per SIMD (16 prompts of 1 to 2048 tokens, 16 heads of 64 x 128: 81 us
// cut, 129 uncut; 16 of 1024 tokens 89 and 70, but the host cannot tell them
// apart; with twice the waves uncut is faster for both, 131 against 155 us and 85
// against 126), and more than 256 tokens, or 64 of every sequence up to 1024 in
// all (256 tokens of one prompt: 23 us cut, 20 uncut; 19 prompts of 1 to 86, 8
// heads of 16 x 16: 11.0 and 7.0). Then segments are as long as fills the chip
// once, with three waves per SIMD (four in workgroups of eight, two at N = 256),
// half a segment of every sequence but one lost, but of 128 tokens at least and a
// 64th of all at most: one prompt of 4096 tokens takes 38 us in segments of 128,
// 44 in segments of 256.
Plan plan_of(const ssu_linear_args &a)
{
    Plan p{};
    const int columns = chunk_kernels(a.dstate, a.headdim, 0).columns, waves = columns / 16;
    p.slices = (a.headdim + columns - 1) / columns;
    const int64_t units = static_cast<int64_t>(a.nheads) * p.slices * waves;
    const int64_t chunks = (a.ntokens + kChunk - 1) / kChunk;
    p.waves = a.batch * units;
    const bool cuts = chunks > std::max(8, std::min(a.batch, 16) * 2) && p.waves <= 4 * kNumCUs;
    const int64_t room = (a.dstate == 256 ? 8 : waves == 4 ? 12 : 16) * kNumCUs - (cuts ? (a.batch - 1) * units / 2 : 0);
    const int64_t per = std::max<int64_t>({(chunks * units + room - 1) / room, (chunks + 63) / 64, 4});
    const bool cut = cuts && per < chunks;
    p.seg_len = static_cast<int>(cut ? per * kChunk : std::min<int64_t>(a.ntokens + 1, INT32_MAX));
    p.segments = static_cast<int>(a.ntokens / p.seg_len) + a.batch;
    if (cut) {
        p.decays_at = static_cast<int64_t>(p.segments) * a.nheads * a.headdim * a.dstate * 4;
        p.bytes = p.decays_at + static_cast<int64_t>(p.segments) * a.nheads * 4;
    }
    return p;
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

// Launch of a step by the bytes of state that it moves one way (H16 P64 N128 and
// others): two dwordx4 per lane below 8 MiB (more waves for the latency: one
// request 2.9 us), four above; residency capped (by unused LDS) at 16 workgroups per
// CU from 40 MiB and 14 from 128 MiB, since more state in flight only crowds
// the memory system (256 MiB: 88.5 us, 6.1 TB/s, at 14;
// 96.0 uncapped, 91.9 at 12, 89.0 at 16; 32 MiB: 13.5 us uncapped, 14.0 at 16).
ssu_status launch_step(const ssu_linear_args &a, hipStream_t stream)
{
    const int64_t mib = static_cast<int64_t>(a.batch) * a.nheads * a.headdim * a.dstate >> 18;
    const StepKernel k = mib < 8 ? step_kernel<2>(a.dstate) : step_kernel<4>(a.dstate);
    LinearParams p = linear_params(a);
    p.tiles = (a.headdim + k.rows - 1) / k.rows;
    const int64_t groups = static_cast<int64_t>(a.batch) * a.nheads * p.tiles;
    SSU_TRY(check_launch(groups, 64, "ssu_linear_attention_step"));
    p.total = static_cast<int>(groups);
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
    const hipError_t e = launch_kernel(k.fn, p, p.total, 64, lds, stream);
    if (e != hipSuccess)
        return fail(SSU_ERR_HIP, "launch of the linear attention step failed: %s", hipGetErrorString(e));
    return SSU_OK;
}

ssu_status launch_chunks(const ssu_linear_args &a, hipStream_t stream)
{
    const Plan plan = plan_of(a);
    if (plan.bytes > 0) {
        if (!a.workspace || a.workspace_bytes < plan.bytes)
            return fail(SSU_ERR_INVALID_ARGUMENT, "ssu_linear_attention: workspace of %lld bytes, %lld needed",
                        static_cast<long long>(a.workspace ? a.workspace_bytes : 0), static_cast<long long>(plan.bytes));
        if (reinterpret_cast<uintptr_t>(a.workspace) % 16)
            return fail(SSU_ERR_MISALIGNED, "ssu_linear_attention: workspace must be 16-byte aligned");
    }
    const ChunkKernels k = chunk_kernels(a.dstate, a.headdim, plan.bytes > 0 ? 0 : plan.waves);
    ChunkParams p{};
    p.a = linear_params(a);
    p.states = static_cast<float *>(a.workspace);
    p.decays = reinterpret_cast<float *>(static_cast<char *>(a.workspace) + plan.decays_at);
    p.seg_len = plan.seg_len;
    p.slices = plan.slices;
    p.dstate = a.dstate;
    const int64_t groups = (static_cast<int64_t>(plan.segments) + 7) / 8 * 8 * a.nheads * plan.slices;
    SSU_TRY(check_launch(groups, 4 * k.columns, "ssu_linear_attention"));
    DeviceGuard guard;
    SSU_TRY(guard.enter(a.device));
    hipError_t e = hipSuccess;
    if (plan.bytes > 0) {
        e = launch_kernel(k.states, p, groups, 4 * k.columns, 0, stream);
        const int64_t blocks = (static_cast<int64_t>(a.headdim) * a.dstate + 1023) / 1024;
        if (e == hipSuccess)
            e = launch_kernel(&ssu_linear_segments_kernel, p, blocks * a.nheads * a.batch, 256, 0, stream);
    }
    if (e == hipSuccess)
        e = launch_kernel(k.full, p, groups, 4 * k.columns, 0, stream);
    if (e != hipSuccess)
        return fail(SSU_ERR_HIP, "launch of the chunked linear attention failed: %s", hipGetErrorString(e));
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
    return plan_of(*a).bytes;
}

ssu_status ssu_linear_attention(const ssu_linear_args *a, hipStream_t stream)
{
    using namespace ssu;
    if (!a)
        return fail(SSU_ERR_INVALID_ARGUMENT, "ssu_linear_attention: null args");
    SSU_TRY(check_linear(*a, "ssu_linear_attention", true));
    if (a->batch == 0 || a->ntokens == 0)
        return SSU_OK;
    return launch_chunks(*a, stream);
}

ssu_status ssu_linear_attention_step(const ssu_linear_args *a, hipStream_t stream)
{
    using namespace ssu;
    if (!a)
        return fail(SSU_ERR_INVALID_ARGUMENT, "ssu_linear_attention_step: null args");
    SSU_TRY(check_linear(*a, "ssu_linear_attention_step", false));
    if (a->batch == 0)
        return SSU_OK;
    return launch_step(*a, stream);
}

}  // extern "C"
