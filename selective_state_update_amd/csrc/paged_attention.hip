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

constexpr int kTile = 32;     // tokens of one wave's step
constexpr int kJoinWaves = 4;  // of a workgroup of the join

// Waves of a workgroup. D = 256 needs half the register file per wave: two
// waves and two workgroups per CU instead of four and one keep one of them
// loading while the other joins (64 requests up to 4096 tokens, 8 heads of 256:
// 178 against 195 us).
constexpr int waves_for(int D) { return D == 256 ? 2 : 4; }

// Tokens of a step of a workgroup of so many waves.
constexpr int round_of(int waves) { return waves * kTile; }

struct AttnParams {
    const uint16_t *q, *k, *v;
    int64_t q_b, q_h, k_page, k_row, k_h, v_page, v_row, v_h;
    const int32_t *table, *lens;
    int64_t t_b, num_pages, max_pages;
    uint16_t *out;
    int64_t o_b, o_h;
    float *lse;
    int64_t l_b, l_h;
    // Workspace: for every workgroup, what the unit that it leaves unfinished
    // is (Open), and for its first and its last unit 16 rows of sums and of
    // (maximum, sum).
    struct Open *open;
    float *part, *stat;
    int32_t batch, nk, heads_per_kv, row_tiles, page_size, groups;
    int32_t cuts, cuts_half;  // runs of a unit's line, with all workgroups or one per CU; 0: too many would be left over
    float scale_log2;  // scale * log2(e): weights are powers of 2
};

// A unit (request, key/value head, 16 query heads) whose first steps a
// workgroup did and whose last ones workgroup `last` does; b < 0: none.
struct Open {
    int32_t b, unit, last, stride;  // (every stride-th workgroup up to `last`)
};

// The visible tokens of a request (negative: padding) and its steps; a request
// without a visible token has one, which writes its zeros.
__device__ __forceinline__ int64_t visible(const AttnParams &p, int b)
{
    const int64_t n = p.lens[b];
    return n < 0 ? n : p.num_pages == 0 ? 0 : min(n, p.max_pages * p.page_size);
}

__device__ __forceinline__ int64_t rounds_of(int64_t n, int round)
{
    return n < 0 ? 0 : n == 0 ? 1 : (n + round - 1) / round;
}

// fp16 weights are scaled by 2^14 (at most 2^14, then): what lies 2^-28 below a
// row's largest weight is still a normal number.
template <typename T>
constexpr float kShift = 0.0f;
template <>
constexpr float kShift<F16> = 14.0f;

// What a partial sum with maximum `own` is multiplied by under the maximum `top`:
// positive wherever the sum's weights are, so that infinities in it stay (2^-126 of
// a finite sum is nothing beside the largest weight's).
__device__ __forceinline__ float rescale(float own, float top)
{
    return __builtin_amdgcn_exp2f(fmaxf(own - (top == -INFINITY ? 0.0f : top), own == -INFINITY ? own : -126.0f));
}

template <typename T>
__device__ __forceinline__ void write_lse(const AttnParams &p, int b, int h, float sum, float top)
{
    if (p.lse)
        p.lse[b * p.l_b + h * p.l_h] = sum == 0.0f ? -INFINITY : (top - kShift<T> + log2f(sum)) * kLn2Hi;
}

// The steps of all units stand in one line (requests in order, a request's
// units in order, a unit's steps in order), and every workgroup takes an equal
// run of it: requests of very different lengths, one long request and many
// short ones all fill the chip with one set of resident workgroups. A unit
// that lies across two or more runs is joined by the second kernel; a
// workgroup leaves at most two of its units unfinished, its first and its last.
//
// With four steps or more for a workgroup (D of 128 and 256), and where hardly one is
// left over, there is a line for each unit of a request instead, all cut alike: the
// workgroups of a run read the same tokens' heads, which lie beside each other, at
// about the same time (64 requests up to 8192 tokens, 8 heads of 128: 175 against 181
// us; one of 100000: 71 against 76; D = 64, 64 up to 8192: 105 against 100).
//
// Memory-bound: every visible K and V row is read once per 16 query heads, so
// the loads decide, and the products are arranged for them:
//
//  - S^T = K Q^T. Whole rows of K are read, 1 KiB per load, and turned into the
//    product's fragments (lane l: 16 bytes of token l % 16) through LDS, runs
//    of a row swapped so that neither side has bank conflicts. Read as fragments, 64
//    bytes of each of 16 rows per load, they came at 6.1 to 6.3 TB/s at best.
//  - The result has one query head per lane column, so a row's statistics are
//    one value per lane (plus two exchanges for the maximum), and the weights
//    lie exactly as the second product's fragment wants them: the lane's 4
//    tokens of two 16-token tiles are its 8 places of the contracted axis.
//  - V's rows are read whole too: 16 lanes hold 16 runs of a token's D values,
//    and a lane has its run of 8 tokens. Output column c of product m stands
//    for value c * D/16 + m, so a product's fragment is a transposition inside
//    the lane (byte permutes), and the output comes back in runs of D/16.
//
// K and V are read past the caches (non-temporal; 64 requests of 1 to 1600 tokens 45.6
// against 46.3 us, 3 of 100003 tokens 113 against 115, and 116 without LDS). Each wave
// takes every W-th step of 32 tokens with statistics of its own. PAGE16:
// pages are a multiple of 16 tokens, a tile lies in one page and its address
// is uniform; otherwise every lane looks its own token up. WHOLE (short caches,
// see plan_of): no line, a workgroup per unit, nothing to join behind it.
template <typename T, int D, bool PAGE16, bool WHOLE, int W>
__global__ void __launch_bounds__(64 * W, D <= 128 ? 2 : 1) ssu_attn_split_kernel(const AttnParams p)
{
    constexpr int kWaves = W;
    constexpr int kRound = round_of(W);
    constexpr int KS = D / 32;      // products along D of a score
    constexpr int E = D / 16;       // values of a V row per lane, products of an output row
    constexpr int EW = E / 2;       // the same in words
    constexpr int CH = D / 8;       // 16-byte runs of a K row
    constexpr int RPI = 64 / CH;    // K rows that one load reads
    constexpr int SW = CH < 16 ? CH - 1 : 15;
    using V = uint32_t __attribute__((ext_vector_type(EW)));
    typedef V V_a2 __attribute__((aligned(2)));
    __shared__ __attribute__((aligned(16))) float part[kWaves][16][D];
    __shared__ __attribute__((aligned(16))) float stat_m[kWaves][16], stat_l[kWaves][16], row_top[16], row_sum[16];
    __shared__ int64_t scan[kWaves];
    __shared__ int64_t found[3];  // its request, the steps before it, its tokens

    int wg = static_cast<int>(blockIdx.x);
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, c = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int units = p.nk * p.row_tiles;  // of a request
    const int ch = lane % CH, ksub = lane / CH;
    u32x4 *const kbuf = reinterpret_cast<u32x4 *>(&part[wave][0][0]);  // a step's K; sums only behind the last step

    // this workgroup's run of the line, and the request that it begins in: the
    // steps of one unit of every request, summed over them
    int64_t per, pos, stop, n, before;  // (before: a unit's steps of all earlier requests)
    int b, lanes = 1, line = units, unit = -1, run = wg;  // lines; units of a request in one; the line's unit
    auto run_of = [&](int64_t steps) {
        const int64_t total = steps * units;
        const int64_t all = static_cast<int64_t>(p.batch) * units;  // of the batch
        const bool half = D == 128 && p.groups > kNumCUs && (all <= kNumCUs / 8 || total >= 6 * (kNumCUs + all));
        // (no more than steps: those with work are spread over all XCDs)
        const int groups = static_cast<int>(min(static_cast<int64_t>(half ? kNumCUs : p.groups), max(total, int64_t(1))));
        int runs = groups;
        int64_t length = total;
        bool in = wg < groups;
        const int cuts = half ? p.cuts_half : p.cuts;
        if (D > 64 && cuts > 0 && total >= 4 * groups) {
            asm volatile("");  // (a branch, not its divisions ahead of it)
            lanes = units;
            line = 1;
            length = steps;
            runs = cuts;
            run = wg / units;
            unit = wg - run * units;
            in = run < runs;
        } else if (in) {
            run = wg = xcd_order(wg, groups);
        }
        per = (length + runs - 1) / runs;
        pos = run * per;
        stop = in ? min(pos + per, length) : 0;
        if (tid == 0)
            p.open[wg] = Open{-1, 0, 0, 0};
    };
    if constexpr (WHOLE) {
        b = wg / units;
        n = visible(p, b);
        if (n < 0)
            return;
        before = 0;
        per = stop = rounds_of(n, kRound);
        pos = 0;
    } else if (p.batch <= 64) {  // every wave for itself: a request per lane (at most 2^25 steps each)
        const int64_t own_n = lane < p.batch ? visible(p, lane) : -1;
        const uint32_t own = static_cast<uint32_t>(rounds_of(own_n, kRound)), sum = scan_lanes(static_cast<int>(own));
        run_of(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(sum), 63)));
        if (pos >= stop)
            return;
        const uint64_t mine = __ballot(static_cast<int64_t>(sum - own) * line <= pos && pos < static_cast<int64_t>(sum) * line);
        b = static_cast<int>(__builtin_ctzll(mine));
        n = __builtin_amdgcn_readlane(static_cast<int>(own_n), b);
        before = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(sum - own), b));
    } else {
        int64_t total = 0;
        for (int i = tid; i < p.batch; i += 64 * kWaves)
            total += rounds_of(visible(p, i), kRound);
#pragma unroll
        for (int m = 32; m >= 1; m /= 2)
            total += __shfl_xor(total, m);
        if (lane == 0)
            scan[wave] = total;
        __syncthreads();
        total = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            total += scan[w];
        run_of(total);
        if (pos >= stop)
            return;
        before = 0;
        for (int b0 = 0; b0 < p.batch; b0 += 64 * kWaves) {
            const int i = b0 + tid;
            const int64_t own_n = i < p.batch ? visible(p, i) : -1, own = rounds_of(own_n, kRound);
            int64_t sum = own;
#pragma unroll
            for (int m = 1; m < 64; m *= 2) {
                const int64_t up = __shfl_up(sum, m);
                sum += lane >= m ? up : 0;
            }
            __syncthreads();
            if (lane == 63)
                scan[wave] = sum;
            __syncthreads();
            int64_t first = before + sum - own;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                first += w < wave ? scan[w] : 0;
                before += scan[w];
            }
            if (first * line <= pos && pos < (first + own) * line) {
                found[0] = i;
                found[1] = first;
                found[2] = own_n;
            }
            if (before * line > pos)
                break;
        }
        __syncthreads();
        b = __builtin_amdgcn_readfirstlane(static_cast<int>(found[0]));
        before = found[1];
        n = found[2];
    }
    int64_t rounds = rounds_of(n, kRound);
    int64_t step0 = 0;  // of the unit, where this workgroup begins
    if constexpr (WHOLE) {
        unit = wg % units;
    } else if (unit < 0) {
        unit = static_cast<int>((pos - before * units) / rounds);
        step0 = pos - before * units - unit * rounds;
    } else {
        step0 = pos - before;
    }

    for (;;) {
        const int64_t steps = min(rounds - step0, stop - pos);
        const struct {
            int64_t n, begin, end;
        } sh = {n, step0 * kRound, min(n, (step0 + steps) * kRound)};
        unit = __builtin_amdgcn_readfirstlane(unit);
        const int kh = unit / p.row_tiles, rt = unit - kh * p.row_tiles;
        const int rows = min(p.heads_per_kv - rt * 16, 16);  // query heads of this unit
        const int h0 = kh * p.heads_per_kv + rt * 16;

        u32x4 qf[KS];
#pragma unroll
        for (int i = 0; i < KS; ++i)
            qf[i] = c < rows ? *reinterpret_cast<const u32x4_a2 *>(p.q + b * p.q_b + (h0 + c) * p.q_h + (i * 4 + g) * 8)
                             : u32x4{0, 0, 0, 0};
        const int32_t *const table = p.table + b * p.t_b;
        const uint16_t *const kbase = p.k + kh * p.k_h + ch * 8, *const vbase = p.v + kh * p.v_h + c * E;

        // A tile of 16 tokens: its page id as the table has it (requested a step
        // before it is needed), then where it is and which of its tokens are
        // visible. Uniform with PAGE16 (through the scalar cache: a vector load
        // would make its reader wait for all K and V loads issued before it),
        // otherwise of this lane's token.
        struct Entry {
            int off;
            int page;
        };
        struct Tile {
            int64_t k, v;  // PAGE16: the tile's first rows; otherwise this lane's
            uint32_t seen;  // uniform, a bit per token
        };
        auto peek = [&](int64_t t0) {
            Entry e;
            if constexpr (PAGE16) {
                const int at = static_cast<int>(min(t0, (sh.end - 1) & ~int64_t(15)));
                const int col = __builtin_amdgcn_readfirstlane(at / p.page_size);
                e.off = at - col * p.page_size;
                e.page = load_ro(table + col);
            } else {
                const int at = static_cast<int>(min(t0 + c, sh.end - 1));
                const int col = at / p.page_size;
                e.off = at - col * p.page_size;
                e.page = table[col];
            }
            return e;
        };
        auto locate = [&](int64_t t0, const Entry &e) {
            Tile t;
            const bool good = e.page >= 0 && e.page < p.num_pages;
            const int64_t page = good ? e.page : 0;
            t.k = page * p.k_page + e.off * p.k_row;
            t.v = page * p.v_page + e.off * p.v_row;
            if constexpr (PAGE16) {
                const int64_t left = sh.end - t0;
                t.seen = !good || left <= 0 ? 0u : left >= 16 ? 0xffffu : (1u << left) - 1u;
            } else {
                t.seen = static_cast<uint32_t>(__ballot(good && t0 + c < sh.end)) & 0xffffu;
            }
            return t;
        };
        const uint16_t *const klane = kbase + (PAGE16 ? ksub * p.k_row : 0), *const vlane = vbase + (PAGE16 ? 4 * g * p.v_row : 0);
        auto load_k = [&](const Tile &t, u32x4 (&f)[KS]) {
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                const int64_t row = PAGE16 ? t.k + i * RPI * p.k_row : __shfl(t.k, RPI * i + ksub);
                f[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_a2 *>(klane + row));
            }
        };
        auto load_v = [&](const Tile &t, V *f) {  // tokens 4g .. 4g+3
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t row = PAGE16 ? t.v + i * p.v_row : __shfl(t.v, 4 * g + i);
                f[i] = __builtin_nontemporal_load(reinterpret_cast<const V_a2 *>(vlane + row));
            }
        };

        f32x4 o[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
            o[e] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        float m = -INFINITY, l = 0.0f;  // of query head c (l: this lane's tokens)

        // One step of 32 tokens, with K (kf) and V (vf) on their way: K of the next
        // step is requested once the scores have freed its registers, with the page
        // ids of the step behind it, and the next V after this one's product. Behind
        // the last step the loads go to the split's last tile again: a condition
        // around them would make every wait for older loads a wait for all.
        int64_t t0 = sh.begin + wave * kTile;
        Tile tile[2];
        Entry entry[2];
        u32x4 kf[2][KS];
        V vf[8];
        if (t0 < sh.end) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                tile[u] = locate(t0 + 16 * u, peek(t0 + 16 * u));
                load_k(tile[u], kf[u]);
                load_v(tile[u], vf + 4 * u);
                entry[u] = peek(t0 + kRound + 16 * u);
            }
        }
        while (t0 < sh.end) {
            const uint32_t seen[2] = {tile[0].seen, tile[1].seen};
            t0 += kRound;
            f32x4 s[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                s[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < KS; ++i)
                    kbuf[(u * 16 + RPI * i + ksub) * CH + (ch ^ ((RPI * i + ksub) & SW))] = kf[u][i];
            }
            __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");  // (the buffer is this wave's own)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
                for (int i = 0; i < KS; ++i)
                    kf[u][i] = kbuf[(u * 16 + c) * CH + ((4 * i + g) ^ (c & SW))];
#pragma unroll
                for (int i = 0; i < KS; ++i)
                    s[u] = Mma<T>::run(kf[u][i], qf[i], s[u]);
            }

#pragma unroll
            for (int u = 0; u < 2; ++u) {
                tile[u] = locate(t0 + 16 * u, entry[u]);
                entry[u] = peek(t0 + kRound + 16 * u);
                load_k(tile[u], kf[u]);
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
            load_v(tile[0], vf);
            load_v(tile[1], vf + 4);
        }

        // An infinity in V, times a weight's remainder or a weight that 16 bits round to
        // 0, is not what the formula has: such a wave's sums are taken again with whole
        // weights, token by token (the check costs a call 0.2 to 1 us).
        f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                zero[i] = fmaf(o[e][i], 0.0f, zero[i]);
        if (__any((zero[0] + zero[1]) + (zero[2] + zero[3]) != 0.0f)) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                o[e] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll 1
            for (int64_t j = sh.begin + wave * kTile; j < sh.end; j += (j + 1) % kTile ? 1 : 1 + kRound - kTile) {
                const int at = static_cast<int>(j), col = at / p.page_size, off = at - col * p.page_size;
                const int64_t page = table[col];
                if (page < 0 || page >= p.num_pages)
                    continue;
                const uint16_t *const kr = p.k + page * p.k_page + off * p.k_row + kh * p.k_h;
                const uint16_t *const qr = p.q + b * p.q_b + (h0 + min(c, rows - 1)) * p.q_h;
                float s = 0.0f;  // of query head c, this lane's quarter of D
#pragma unroll 1
                for (int d = g * (D / 4); d < (g + 1) * (D / 4); d += 8) {
                    const u32x4 kw = *reinterpret_cast<const u32x4_a2 *>(kr + d), qw = *reinterpret_cast<const u32x4_a2 *>(qr + d);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s = fmaf(T::hi(kw[i]), T::hi(qw[i]), fmaf(T::lo(kw[i]), T::lo(qw[i]), s));
                }
                s += __shfl_xor(s, 16);
                s += __shfl_xor(s, 32);
                s *= p.scale_log2;
                float w = __builtin_amdgcn_exp2f(s - base + kShift<T>);
                w = s > -INFINITY && w == 0.0f ? 0x1p-126f : w;
                const V x = *reinterpret_cast<const V_a2 *>(p.v + page * p.v_page + off * p.v_row + kh * p.v_h + c * E);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float wi = __shfl(w, 4 * g + i);
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        o[e][i] = fmaf(wi, e % 2 ? T::hi(x[e / 2]) : T::lo(x[e / 2]), o[e][i]);
                }
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
        f32x4 top = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, own;  // of rows 4g .. 4g+3
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            top = __builtin_elementwise_max(top, *reinterpret_cast<const f32x4 *>(&stat_m[w][4 * g]));
        own = *reinterpret_cast<const f32x4 *>(&stat_m[wave][4 * g]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float f = rescale(own[i], top[i]);
#pragma unroll
            for (int e = 0; e < E; ++e)
                part[wave][4 * g + i][c * E + e] = o[e][i] * f;
        }
        if (wave == 0 && c == 0) {
            f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const f32x4 x = *reinterpret_cast<const f32x4 *>(&stat_m[w][4 * g]);
                const f32x4 y = *reinterpret_cast<const f32x4 *>(&stat_l[w][4 * g]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sum[i] = fmaf(y[i], rescale(x[i], top[i]), sum[i]);
            }
            *reinterpret_cast<f32x4 *>(&row_top[4 * g]) = top;
            *reinterpret_cast<f32x4 *>(&row_sum[4 * g]) = sum;
        }
        __syncthreads();
        const bool whole = WHOLE || steps == rounds;
        const int64_t row0 = (2 * static_cast<int64_t>(wg) + (step0 == 0)) * 16;
        for (int at = 4 * tid; at < rows * D; at += 4 * 64 * kWaves) {
            const int r = at / D, d = at % D;
            f32x4 y = *reinterpret_cast<const f32x4 *>(&part[0][r][d]);
#pragma unroll
            for (int w = 1; w < kWaves; ++w)
                y += *reinterpret_cast<const f32x4 *>(&part[w][r][d]);
            const float most = row_top[r], sum = row_sum[r];
            if (whole) {
                y *= sum == 0.0f ? 0.0f : 1.0f / sum;
                *reinterpret_cast<u32x2_a2 *>(p.out + b * p.o_b + (h0 + r) * p.o_h + d) =
                    u32x2{pack2<T>(y[0], y[1]), pack2<T>(y[2], y[3])};
                if (d == 0)
                    write_lse<T>(p, b, h0 + r, sum, most);
            } else {
                *reinterpret_cast<f32x4 *>(p.part + (row0 + r) * D + d) = y;
                if (d == 0) {
                    p.stat[2 * (row0 + r)] = most;
                    p.stat[2 * (row0 + r) + 1] = sum;
                }
            }
        }
        if (!whole && step0 == 0 && tid == 0)
            p.open[wg] = Open{b, unit, wg + (static_cast<int32_t>((pos + rounds - 1) / per) - run) * lanes, lanes};

        // the next unit
        pos += steps;
        if (WHOLE || pos >= stop)
            return;
        step0 = 0;
        if (lanes > 1 || ++unit == units) {
            unit = lanes > 1 ? unit : 0;
            do
                n = visible(p, ++b);
            while (n < 0);  // (pos < stop: there is one)
            rounds = rounds_of(n, kRound);
        }
        __syncthreads();  // LDS is free again
    }
}

// A workgroup per unit that lies across several runs and row of it: the runs'
// partial sums joined, dealt out to its waves and several of them on their way at
// once (it is the latency of these reads that the kernel costs: with one wave per
// row attention of one request over 777 tokens takes 12.2 us instead of 11.0).
template <typename T, int D>
__global__ void __launch_bounds__(64 * kJoinWaves) ssu_attn_join_kernel(const AttnParams p)
{
    constexpr int E = D / 64;
    __shared__ float part[kJoinWaves][D], sums[kJoinWaves];
    const int most = min(p.heads_per_kv, 16);  // rows of a unit
    const int wg = static_cast<int>(blockIdx.x) / most, r = static_cast<int>(blockIdx.x) % most;
    const int wave = static_cast<int>(threadIdx.x) >> 6, lane = static_cast<int>(threadIdx.x) & 63;
    const Open u = p.open[wg];
    if (u.b < 0)
        return;
    const int kh = u.unit / p.row_tiles, rt = u.unit - kh * p.row_tiles;
    if (r >= p.heads_per_kv - rt * 16)
        return;
    // this workgroup's last unit, then the first ones of those up to u.last
    auto row_of = [&](int w) { return (2 * static_cast<int64_t>(w) + (w == wg)) * 16 + r; };
    float top = -INFINITY;
    for (int w = wg + lane * u.stride; w <= u.last; w += 64 * u.stride)
        top = fmaxf(top, p.stat[2 * row_of(w)]);
#pragma unroll
    for (int m = 32; m >= 1; m /= 2)
        top = fmaxf(top, __shfl_xor(top, m));
    float sum = 0.0f, y[E] = {};
#pragma unroll 8
    for (int w = wg + wave * u.stride; w <= u.last; w += kJoinWaves * u.stride) {
        const int64_t row = row_of(w);
        const float f = rescale(p.stat[2 * row], top);
        sum = fmaf(p.stat[2 * row + 1], f, sum);
#pragma unroll
        for (int e = 0; e < E; ++e)
            y[e] = fmaf(p.part[row * D + lane + 64 * e], f, y[e]);
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
        part[wave][lane + 64 * e] = y[e];
    if (lane == 0)
        sums[wave] = sum;
    __syncthreads();
    if (wave > 0)
        return;
#pragma unroll
    for (int k = 1; k < kJoinWaves; ++k) {
        sum += sums[k];
#pragma unroll
        for (int e = 0; e < E; ++e)
            y[e] += part[k][lane + 64 * e];
    }
    const int h = kh * p.heads_per_kv + rt * 16 + r;
#pragma unroll
    for (int e = 0; e < E; ++e)
        p.out[u.b * p.o_b + h * p.o_h + lane + 64 * e] = T::round(sum == 0.0f ? 0.0f : y[e] / sum);
    if (lane == 0)
        write_lse<T>(p, u.b, h, sum, top);
}

using AttnFn = void (*)(AttnParams);

struct AttnKernels {
    AttnFn split, join;
};

template <typename T, int D, bool WHOLE, int W>
AttnKernels attn_kernels(bool page16)
{
    return {page16 ? &ssu_attn_split_kernel<T, D, true, WHOLE, W> : &ssu_attn_split_kernel<T, D, false, WHOLE, W>,
            &ssu_attn_join_kernel<T, D>};
}

template <typename T>
AttnKernels attn_kernels(int D, bool page16, bool whole, int waves)
{
    if (!whole)
        return D == 64 ? attn_kernels<T, 64, false, waves_for(64)>(page16)
             : D == 128 ? attn_kernels<T, 128, false, waves_for(128)>(page16) : attn_kernels<T, 256, false, waves_for(256)>(page16);
    return D == 64 ? attn_kernels<T, 64, true, 4>(page16)
         : D == 128 ? attn_kernels<T, 128, true, 4>(page16)
         : waves == 4 ? attn_kernels<T, 256, true, 4>(page16) : attn_kernels<T, 256, true, 2>(page16);
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
        return fail(SSU_ERR_UNSUPPORTED, "%s: batch * nq %lld too large", who, static_cast<long long>(a.batch) * a.nq);
    if (a.max_pages > (INT64_MAX >> 1) / a.page_size)
        return fail(SSU_ERR_INVALID_ARGUMENT, "%s: max_pages * page_size too large", who);
    return SSU_OK;
}

struct Plan {
    int row_tiles, groups, waves;
    bool whole;  // a workgroup per unit, no workspace
    int64_t part_at, stat_at, bytes;  // workspace
};

// A workgroup of its own per unit where no unit has more than 512 tokens (256 at D =
// 256), or no more than 16 steps and there is at least one unit for every CU: no line
// to lay out, no partial sums, one launch, and as many workgroups per CU as fit,
// which load while others start and join (one request, 2 heads of 128: 100 tokens 6.1
// against 9.2 us, 400 tokens 9.0 against 10.3, 800 tokens 13.1 against 11.1; 32
// requests of 1 to 1600 tokens, 8 heads: 26 against 34 us; 64 of 1 to 1600: 46
// against 50; 64 of 1 to 8192: 218 against 184). At D = 256 with four waves while
// each has a CU to itself (32 requests of 1 to 1600 tokens, 8 heads: 52 us, 62 in a line;
// 64 of 1 to 200: 23 us with four waves, 18 with two). (All of these, and those below,
// from before the check for infinities, which costs either side 0.2 to 1 us.)
//
// Otherwise a line with two workgroups per CU; at D = 128 every second one leaves
// (the kernel knows the lengths) where the runs' pieces of units have 6 steps or more
// or are few: four waves' loads are enough then to fill the memory system, and more
// only crowd it (64 requests up to 8192 tokens, 8 heads: 174 against 180 us with two;
// 64 up to 4500: 104 against 110; one of 100000: 71 against 76; but in a table for 16384
// tokens 64 up to 800: 36 against 34, 256 up to 400: 76 against 67; D = 64, 64 up to
// 8192: 121 against 100). No more than there can be steps.
Plan plan_of(const ssu_attn_args &a)
{
    Plan p{};
    p.row_tiles = (a.nq / a.nk + 15) / 16;
    const int64_t units = static_cast<int64_t>(a.batch) * a.nk * p.row_tiles;
    const int64_t tokens = a.max_pages * a.page_size;
    p.waves = a.headdim == 256 && units > kNumCUs ? 2 : 4;
    p.whole = tokens <= (units < kNumCUs ? (a.headdim == 256 ? 256 : 512) : 16 * round_of(p.waves));
    if (p.whole) {
        p.groups = static_cast<int>(units);
        return p;
    }
    p.waves = waves_for(a.headdim);
    const int64_t rounds = (tokens + round_of(p.waves) - 1) / round_of(p.waves);
    const int64_t resident = 2 * kNumCUs;
    p.groups = static_cast<int>(units > resident / rounds ? resident : std::max<int64_t>(units * rounds, 1));
    p.part_at = static_cast<int64_t>(p.groups) * sizeof(Open);
    p.stat_at = p.part_at + static_cast<int64_t>(p.groups) * 32 * a.headdim * 4;
    p.bytes = p.stat_at + static_cast<int64_t>(p.groups) * 32 * 2 * 4;
    return p;
}

float log2_scale(const ssu_attn_args &a) { return static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634); }

ssu_status check_attn(const ssu_attn_args &a)
{
    const char *const who = "ssu_paged_attention";
    if (a.reserved != 0)
        return fail(SSU_ERR_INVALID_ARGUMENT, "%s: reserved field must be 0", who);
    if (!std::isfinite(log2_scale(a)))
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
    if (plan.bytes > 0 && (!a.workspace || a.workspace_bytes < plan.bytes))
        return fail(SSU_ERR_INVALID_ARGUMENT, "ssu_paged_attention: workspace of %lld bytes, %lld needed",
                    static_cast<long long>(a.workspace ? a.workspace_bytes : 0), static_cast<long long>(plan.bytes));
    if (reinterpret_cast<uintptr_t>(a.workspace) % 16)
        return fail(SSU_ERR_MISALIGNED, "ssu_paged_attention: workspace must be 16-byte aligned");
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
    p.nk = a.nk;
    p.heads_per_kv = a.nq / a.nk;
    p.page_size = a.page_size;
    p.row_tiles = plan.row_tiles;
    p.groups = plan.groups;
    const auto cuts = [units = a.nk * plan.row_tiles](int groups) { return groups % units * 16 <= groups ? groups / units : 0; };
    p.cuts = cuts(plan.groups);
    p.cuts_half = cuts(kNumCUs);
    p.scale_log2 = log2_scale(a);
    char *const ws = static_cast<char *>(a.workspace);
    p.open = reinterpret_cast<Open *>(ws);
    p.part = reinterpret_cast<float *>(ws + plan.part_at);
    p.stat = reinterpret_cast<float *>(ws + plan.stat_at);
    const bool page16 = a.page_size % 16 == 0;
    const AttnKernels k = a.q.dtype == SSU_BF16 ? attn_kernels<Bf16>(a.headdim, page16, plan.whole, plan.waves)
                                                : attn_kernels<F16>(a.headdim, page16, plan.whole, plan.waves);
    SSU_TRY(check_launch(plan.groups, 64 * plan.waves, "ssu_paged_attention"));
    DeviceGuard guard;
    SSU_TRY(guard.enter(a.device));
    hipError_t e = launch_kernel(k.split, p, plan.groups, 64 * plan.waves, 0, stream);
    if (e == hipSuccess && !plan.whole && plan.groups > 1)
        e = launch_kernel(k.join, p, plan.groups * std::min(p.heads_per_kv, 16), 64 * kJoinWaves, 0, stream);
    if (e != hipSuccess)
        return fail(SSU_ERR_HIP, "launch of the paged attention kernels failed: %s", hipGetErrorString(e));
    return SSU_OK;
}

}  // extern "C"
