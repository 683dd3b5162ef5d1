// shared_prefix_attention.hip -- attention of one new token per request behind a
// prefix that the whole batch shares, over a paged key-value cache on MI355X
// (gfx950): ssu_shared_prefix_attention. The operation is stated in include/ssu.h.

#include "attention_kernels.h"

namespace ssu {
namespace {

using f32x16 = float __attribute__((ext_vector_type(16)));

// One wave's product of a 32 x 16 and a 16 x 32 tile, fp32 sums. Lane l holds row
// (column) l % 32 of a (of b), 8 consecutive places of the contracted axis from
// 8 * (l / 32); of the result column l % 32, rows 8 * (r / 4) + 4 * (l / 32) + r % 4.
template <typename T>
__device__ __forceinline__ f32x16 mma32(u32x4 a, u32x4 b, f32x16 c)
{
    using Frag = typename Mma<T>::Frag;
    if constexpr (std::is_same_v<T, Bf16>)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(Frag, a), __builtin_bit_cast(Frag, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(Frag, a), __builtin_bit_cast(Frag, b), c, 0, 0, 0);
}

struct PrefixParams {
    AttnParams a;  // (its prefix_part and prefix_stat are written here)
    const int32_t *table;
    float *part, *stat;
    int32_t rows, row_tiles, units;  // rows: all requests' query heads of a key head
    uint32_t page_magic;             // t / page_size = t * page_magic >> page_shift, t < 2^31
    int32_t page_shift;
};

constexpr int kRowsOfWave = 32;

// Waves of a workgroup: two on each SIMD, or one where D = 256 needs all its registers.
constexpr int prefix_waves(int D) { return D == 256 ? 4 : 8; }

// Where row r of a tile has its 16-byte run: exchanged by row, so that neither 16 rows of one
// run (K) nor 4 rows of 4 runs (V, transposed) have bank conflicts.
template <int CH>
__device__ __forceinline__ int run_at(int r, int run)
{
    return r * CH + (run ^ (CH == 8 ? (r & 2) << 1 | (r >> 2 & 3) : (r & 3) << 2 | (r >> 2 & 3)));
}

// One workgroup takes 256 rows (a request's query head each; 128 at D = 256) of one key
// head and one piece of the prefix, a wave 32 of them; tiles of 64 tokens go through LDS, two
// buffers and one barrier a tile, requested three tiles ahead, or two where registers
// are short. S^T = K Q^T and O^T = V^T P^T: a row's statistics are
// one value per lane (and its other half's), its weights lie as the second product's
// fragment wants them (8 tokens of 16 per lane, whichever they are), and V is read
// transposed. The rows of LDS are whole rows of K and V.
// Weights are rounded to 16 bits once (half a step: 2^-8, fp16 2^-11, relative), while l adds up
// whole ones: products with their remainders too, as where a row's tokens are its own, take
// 256 requests of 64 heads behind 30011 tokens from 375 to 476 us, 64 of 32 behind 8192 from 69
// to 75, and the root mean square of out's error from 1.30 (fp16 1.38) times the one of its own
// rounding to 1.00.
template <typename T, int D>
__global__ void __launch_bounds__(64 * prefix_waves(D), D <= 128 ? 2 : 1) ssu_prefix_kernel(const PrefixParams p)
{
    constexpr int W = prefix_waves(D), WR = kPrefixTile / W, kRowsOfGroup = kRowsOfWave * W;  // (WR: rows of a tile that a wave loads)
    constexpr int KS = D / 16, DT = D / 32, CH = D / 8;
    constexpr bool DEEP = D <= 128;
    constexpr int RPI = 64 / CH, LI = WR / RPI;  // rows of one load, loads of a wave's rows
    __shared__ u32x4 lk[2][kPrefixTile * CH], lv[2][kPrefixTile * CH];
    __shared__ __attribute__((aligned(16))) uint32_t lseen[2][W], lbusy[W];

    const AttnParams &a = p.a;
    const PrefixCut cut = prefix_cut(a);
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, c = lane & 31, hl = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // workgroups go round the 8 XCDs: all rows of a head's piece, which read the same
    // K and V, beside each other on one
    const int id = static_cast<int>(blockIdx.x) / 8, unit = id / p.row_tiles * 8 + static_cast<int>(blockIdx.x) % 8;
    if (unit >= p.units)
        return;
    const int piece = unit / a.nk, kh = unit % a.nk;
    if (piece >= cut.pieces)
        return;
    const int begin = piece * cut.per * kPrefixTile;
    const int end = static_cast<int>(min(cut.tokens, static_cast<int64_t>(begin) + cut.per * kPrefixTile));
    const int tiles = (end - begin + kPrefixTile - 1) / kPrefixTile;

    // Rows of padding requests count as rows that are not there: whatever their q holds is not used.
    const int row = (id % p.row_tiles) * kRowsOfGroup + wave * kRowsOfWave + c;
    const int b = min(row, p.rows - 1) / a.heads_per_kv, h = kh * a.heads_per_kv + min(row, p.rows - 1) % a.heads_per_kv;
    const bool live = row < p.rows && a.lens[b] >= 0;
    const bool busy = __any(live);  // (uniform)
    // Scores stay unscaled, so that the scale is part of the exponent's one fma (2 to 3 %): with
    // its sign moved into Q, and scores of 0 instead of a scale of 0.
    const bool flat = a.scale_log2 == 0.0f;
    const float scale = flat ? 1.0f : fabsf(a.scale_log2);
    const uint32_t sign = a.scale_log2 < 0.0f ? 0x80008000u : 0u;
    u32x4 qf[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s)
        qf[s] = *reinterpret_cast<const u32x4_a2 *>(a.q + b * a.q_b + h * a.q_h + 16 * s + 8 * hl);
#pragma unroll
    for (int s = 0; s < KS; ++s)
        qf[s] = sign ^ (live ? qf[s] : u32x4{0, 0, 0, 0});

    // this wave's rows of a tile: the page ids a tile ahead of K and V (and requested before
    // the older tile's, since loads return in order), those three (D = 256: two) ahead
    // of the products; behind the end the last token again, as not visible
    const int sub = lane / CH, ch = lane % CH;
    int32_t page[LI];
    struct Rows {
        u32x4 k[LI], v[LI];
        bool good[LI];
    } even, odd;  // (odd only if DEEP)
    auto token = [&](int tile, int i) { return static_cast<uint32_t>(begin) + tile * kPrefixTile + WR * wave + RPI * i + sub; };
    auto place = [&](int tile, int i, int &col, int &off) {
        const uint32_t t = min(token(tile, i), static_cast<uint32_t>(end - 1));
        col = static_cast<int>(static_cast<uint64_t>(t) * p.page_magic >> p.page_shift);
        off = static_cast<int>(t) - col * a.page_size;
    };
    auto request_ids = [&](int tile, int32_t (&to)[LI]) {
#pragma unroll
        for (int i = 0; i < LI; ++i) {
            int col, off;
            place(min(tile, tiles - 1), i, col, off);
            to[i] = p.table[col];
        }
    };
    auto request = [&](int tile, Rows &to) {  // with the next one's page ids
        int32_t next[LI];
        request_ids(tile + 1, next);
#pragma unroll
        for (int i = 0; i < LI; ++i) {
            int col, off;
            place(min(tile, tiles - 1), i, col, off);
            const bool in = page[i] >= 0 && page[i] < a.num_pages;
            to.good[i] = in && token(min(tile, tiles - 1), i) < static_cast<uint32_t>(end);
            const int64_t pg = in ? page[i] : 0;
            to.k[i] = *reinterpret_cast<const u32x4_a2 *>(a.k + pg * a.k_page + off * a.k_row + kh * a.k_h + 8 * ch);
            to.v[i] = *reinterpret_cast<const u32x4_a2 *>(a.v + pg * a.v_page + off * a.v_row + kh * a.v_h + 8 * ch);
            page[i] = next[i];
        }
    };
    auto stage = [&](int buf, const Rows &from) {
        uint32_t seen = 0;
#pragma unroll
        for (int i = 0; i < LI; ++i) {
            const int r = WR * wave + RPI * i + sub, at = run_at<CH>(r, ch);
            const uint64_t ok = __ballot(from.good[i]);
#pragma unroll
            for (int j = 0; j < RPI; ++j)
                seen |= static_cast<uint32_t>(ok >> (CH * j) & 1) << (RPI * i + j);
            // what is not visible may be NaN
            lk[buf][at] = from.good[i] ? from.k[i] : u32x4{0, 0, 0, 0};
            lv[buf][at] = from.good[i] ? from.v[i] : u32x4{0, 0, 0, 0};
        }
        lseen[buf][wave] = seen;
    };

    f32x16 o[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d)
        o[d] = f32x16{};
    float m = -INFINITY, l = 0.0f;  // of this lane's row (m: unscaled until the end, l: this lane's tokens)

    request_ids(0, page);
    request(0, even);
    if constexpr (DEEP)
        request(1, odd);
    stage(0, even);
    request(DEEP ? 2 : 1, even);
    lbusy[wave] = busy;
    __syncthreads();
    uint32_t work = 0;
#pragma unroll
    for (int i = 0; i < W; ++i)
        work |= lbusy[i];
    if (__builtin_amdgcn_readfirstlane(static_cast<int>(work)) == 0)
        return;  // (all of them)
    auto turn = [&](int tile, Rows &next) {  // `next` holds tile + 1
        const int buf = tile & 1;
        // D = 256: places in LDS are computed for every tile, not kept in registers (they
        // would be spilled: 256 requests of 32 heads behind 8000 tokens 262 against 491 us)
        int at_lane = lane;
        if constexpr (!DEEP)
            asm volatile("" : "+v"(at_lane));
        f32x16 s[2];
        u32x4 w[4];
        if (busy) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                // products before the other wave's softmax, the halves one after the other: 1 to 3 %
                __builtin_amdgcn_s_setprio(1);
                s[t] = f32x16{};
#pragma unroll
                for (int k = 0; k < KS; ++k)
                    s[t] = mma32<T>(lk[buf][run_at<CH>(32 * t + at_lane % 32, 2 * k + at_lane / 32)], qf[k], s[t]);
            }
            __builtin_amdgcn_s_setprio(0);
            uint32_t seen[W], both = ~0u;
#pragma unroll
            for (int i = 0; i < W; ++i)
                both &= seen[i] = lseen[buf][i];
            const bool all = both == (WR == 8 ? 0xffu : 0xffffu);
            float top = m;
            if (flat)
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    s[t] *= 0.0f;
            if (!all)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int token = 32 * t + 8 * (r / 4) + r % 4;  // (and 4 hl)
                        s[t][r] = seen[token / WR] >> (token % WR + 4 * hl) & 1 ? s[t][r] : -INFINITY;
                    }
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    top = fmaxf(top, s[t][r]);
            top = fmaxf(top, __shfl_xor(top, 32));
            const float base = top == -INFINITY ? 0.0f : top;  // scores of -inf weigh nothing
            const float keep = __builtin_amdgcn_exp2f((m - base) * scale), shift = fmaf(-base, scale, kShift<T>);
            m = top;
            float sum = 0.0f;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    s[t][r] = __builtin_amdgcn_exp2f(fmaf(s[t][r], scale, shift));
                    sum += s[t][r];
                }
            l = fmaf(l, keep, sum);
            if (__any(keep != 1.0f))
#pragma unroll
                for (int d = 0; d < DT; ++d)
                    o[d] *= keep;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 16; r += 2)
                    w[2 * t + r / 8][r / 2 % 4] = pack2<T>(s[t][r], s[t][r + 1]);
        }
        stage(buf ^ 1, next);
        request(tile + (DEEP ? 3 : 2), next);
        if (busy) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int d = 0; d < DT; ++d) {
                    const int r0 = 16 * k + 4 * (at_lane / 32) + at_lane % 16 / 4, run = 4 * d + 2 * (at_lane / 16 % 2) + at_lane % 4 / 2;
                    auto at = [&](int r) {
                        return reinterpret_cast<const uint16_t *>(&lv[buf][run_at<CH>(r, run)]) + 4 * (at_lane % 2);
                    };
                    const u32x2 x = read_transposed(at(r0)), y = read_transposed(at(r0 + 8));
                    o[d] = mma32<T>(u32x4{x[0], x[1], y[0], y[1]}, w[k], o[d]);
                }
        }
        __syncthreads();
    };
#pragma unroll 1
    for (int tile = 0; tile < tiles; tile += 2) {
        turn(tile, DEEP ? odd : even);
        if (tile + 1 < tiles)
            turn(tile + 1, even);
    }
    if (!busy)
        return;
    m *= scale;

    // An infinity in V, times a weight that 16 bits round to 0, is not what the formula
    // has: such a row's sums are taken again with whole weights, token by token (the
    // other rows of its wave are other requests' and keep theirs: with a finite row all V is).
    // A row whose weights add up to NaN is NaN whatever V holds.
    l += __shfl_xor(l, 32);
    float zero = 0.0f;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r)
            zero = fmaf(o[d][r], 0.0f, zero);
    const bool again = live && l == l && zero + __shfl_xor(zero, 32) != 0.0f;
    if (__any(again)) {
#pragma unroll
        for (int d = 0; d < DT; ++d)
            o[d] = again ? f32x16{} : o[d];
        const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll 1
        for (int t = begin; t < end; ++t) {
            const int col = t / a.page_size, off = t - col * a.page_size;
            const int64_t pg = p.table[col];
            if (pg < 0 || pg >= a.num_pages)
                continue;
            const uint16_t *const kt = a.k + pg * a.k_page + off * a.k_row + kh * a.k_h, *const qt = a.q + b * a.q_b + h * a.q_h;
            float s = 0.0f;  // this lane's half of D
#pragma unroll 1
            for (int d = hl * (D / 2); d < (hl + 1) * (D / 2); d += 8) {
                const u32x4 kw = *reinterpret_cast<const u32x4_a2 *>(kt + d), qw = *reinterpret_cast<const u32x4_a2 *>(qt + d);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s = fmaf(T::hi(kw[i]), T::hi(qw[i]), fmaf(T::lo(kw[i]), T::lo(qw[i]), s));
            }
            s += __shfl_xor(s, 32);
            s *= a.scale_log2;
            float w = __builtin_amdgcn_exp2f(s - base + kShift<T>);
            w = !again ? 0.0f : s > -INFINITY && w == 0.0f ? 0x1p-126f : w;
            const uint16_t *const vt = a.v + pg * a.v_page + off * a.v_row + kh * a.v_h + 4 * hl;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int r = 0; r < 16; r += 4) {
                    const u32x2 x = *reinterpret_cast<const u32x2_a2 *>(vt + 32 * d + 2 * r);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        o[d][r + i] = fmaf(w, i % 2 ? T::hi(x[i / 2]) : T::lo(x[i / 2]), o[d][r + i]);
                }
        }
    }

    if (!live)
        return;
    const int64_t at = piece * a.prefix_rows + static_cast<int64_t>(b) * a.nk * a.heads_per_kv + h;
    if (hl == 0) {
        p.stat[2 * at] = m;
        p.stat[2 * at + 1] = l;
    }
    float *const part = p.part + at * D + 4 * hl;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int r = 0; r < 16; r += 4)
            *reinterpret_cast<f32x4 *>(part + 32 * d + 2 * r) = f32x4{o[d][r], o[d][r + 1], o[d][r + 2], o[d][r + 3]};
}

using PrefixFn = void (*)(PrefixParams);

template <typename T>
PrefixFn prefix_kernel(int D)
{
    return D == 64 ? &ssu_prefix_kernel<T, 64> : D == 128 ? &ssu_prefix_kernel<T, 128> : &ssu_prefix_kernel<T, 256>;
}

// ------------------------------------------------------------------ host --

struct PrefixPlan {
    Plan own;
    int waves, pieces, rows, row_tiles;
    int64_t part_at, stat_at, bytes;  // workspace, behind the own tokens'
};

// Pieces of the prefix, all of about the same length: as many as take the least time,
// counted in ns. A workgroup takes its tiles one after the other, each D * (10 + waves
// with rows) (D = 128: 1.4 us with one, 2.3 with eight; about 1.5 and 2.5 measured), and two more for its start and
// end, one workgroup to a compute unit; a piece more costs its sums, written and read at
// 3.3 TB/s, and 0.2 us of the join. 64 requests of 32 heads (8 of keys), 8192 tokens: 4
// pieces 115 us, 8 83, 16 70, 32 68, 64 85, the rule's 69; 2000 tokens: 37, 28, 27, 31, 31,
// 28; 256 requests of 64 heads behind 30011: 383, 393, 427, 488, 615, 382; 8 requests of
// 32 heads, 32000 tokens: 217, 118, 68, 45, 57, 46.
PrefixPlan prefix_plan_of(const ssu_shared_args &a)
{
    PrefixPlan p{};
    p.own = plan_of(a.attn);
    const int64_t rows = static_cast<int64_t>(a.attn.batch) * (a.attn.nq / a.attn.nk);
    p.rows = static_cast<int>(rows);
    p.waves = prefix_waves(a.attn.headdim);
    p.row_tiles = static_cast<int>((rows + kRowsOfWave * p.waves - 1) / (kRowsOfWave * p.waves));
    const int64_t tokens = std::min<int64_t>(a.prefix_pages > INT32_MAX ? INT32_MAX : a.prefix_pages * a.attn.page_size, INT32_MAX);
    const int64_t tiles = (tokens + kPrefixTile - 1) / kPrefixTile, groups = static_cast<int64_t>(p.row_tiles) * a.attn.nk;
    const int64_t tile_ns = a.attn.headdim * (10 + std::min<int64_t>((rows + kRowsOfWave - 1) / kRowsOfWave, p.waves));
    const int64_t piece_ns = 200 + rows * a.attn.nk * a.attn.headdim / 400;
    int64_t best = INT64_MAX;
    for (int n = 1; n <= 64 && n <= std::max<int64_t>(tiles, 1); ++n) {
        const int64_t time = (groups * n + kNumCUs - 1) / kNumCUs * ((tiles + n - 1) / n + 2) * tile_ns + n * piece_ns;
        if (time < best) {
            best = time;
            p.pieces = n;
        }
    }
    p.part_at = (p.own.bytes + 255) / 256 * 256;
    const int64_t sums = static_cast<int64_t>(p.pieces) * a.attn.batch * a.attn.nq;
    p.stat_at = p.part_at + sums * a.attn.headdim * 4;
    p.bytes = p.stat_at + sums * 8;
    return p;
}

ssu_status check_prefix_sizes(const ssu_shared_args &a, const char *who)
{
    SSU_TRY(check_sizes(a.attn, who));
    if (a.prefix_pages < 0 || a.prefix_pages > (INT64_MAX >> 1) / a.attn.page_size)
        return fail(SSU_ERR_INVALID_ARGUMENT, "%s: bad prefix_pages %lld", who, static_cast<long long>(a.prefix_pages));
    return SSU_OK;
}

}  // namespace
}  // namespace ssu

extern "C" {

int64_t ssu_shared_prefix_attention_workspace(const ssu_shared_args *a)
{
    using namespace ssu;
    if (!a || check_prefix_sizes(*a, "ssu_shared_prefix_attention_workspace") != SSU_OK)
        return -1;
    return a->attn.batch == 0 ? 0 : prefix_plan_of(*a).bytes;
}

ssu_status ssu_shared_prefix_attention(const ssu_shared_args *args, hipStream_t stream)
{
    using namespace ssu;
    const char *const who = "ssu_shared_prefix_attention";
    if (!args)
        return fail(SSU_ERR_INVALID_ARGUMENT, "%s: null args", who);
    const ssu_attn_args &a = args->attn;
    SSU_TRY(check_attn(a, who));
    SSU_TRY(check_prefix_sizes(*args, who));
    if (a.batch == 0)
        return SSU_OK;
    SSU_TRY(check_view(args->prefix_table, "prefix_table", SSU_I32, 1, args->prefix_pages == 0));
    SSU_TRY(check_view(args->prefix_len, "prefix_len", SSU_I32, 1, false));
    if (args->prefix_pages > 1 && args->prefix_table.stride[0] != 1)
        return fail(SSU_ERR_UNSUPPORTED, "prefix_table: stride must be 1");
    for (const ssu_view *v : {&args->prefix_table, &args->prefix_len})
        if (reinterpret_cast<uintptr_t>(v->ptr) % 4)
            return fail(SSU_ERR_MISALIGNED, "prefix_table/prefix_len: pointer must be 4-byte aligned");
    const PrefixPlan plan = prefix_plan_of(*args);
    if (!a.workspace || a.workspace_bytes < plan.bytes)
        return fail(SSU_ERR_INVALID_ARGUMENT, "%s: workspace of %lld bytes, %lld needed", who,
                    static_cast<long long>(a.workspace ? a.workspace_bytes : 0), static_cast<long long>(plan.bytes));
    if (reinterpret_cast<uintptr_t>(a.workspace) % 16)
        return fail(SSU_ERR_MISALIGNED, "%s: workspace must be 16-byte aligned", who);
    char *const ws = static_cast<char *>(a.workspace);
    PrefixParams p{};
    p.a = attn_params(a, plan.own, a.workspace);
    p.part = reinterpret_cast<float *>(ws + plan.part_at);
    p.stat = reinterpret_cast<float *>(ws + plan.stat_at);
    p.a.prefix_part = p.part;
    p.a.prefix_stat = p.stat;
    p.a.prefix_len = static_cast<const int32_t *>(args->prefix_len.ptr);
    p.a.prefix_pages = args->prefix_pages;
    p.a.prefix_rows = static_cast<int64_t>(a.batch) * a.nq;
    p.a.prefix_pieces = plan.pieces;
    p.table = static_cast<const int32_t *>(args->prefix_table.ptr);
    p.rows = plan.rows;
    p.row_tiles = plan.row_tiles;
    p.units = plan.pieces * a.nk;
    int bits = 0;  // 2^bits >= page_size
    while ((int64_t(1) << bits) < a.page_size)
        ++bits;
    p.page_shift = 31 + bits;
    p.page_magic = static_cast<uint32_t>(((uint64_t(1) << p.page_shift) + a.page_size - 1) / a.page_size);
    const int64_t groups = (static_cast<int64_t>(plan.pieces) * a.nk + 7) / 8 * 8 * plan.row_tiles;
    SSU_TRY(check_launch(groups, 64 * plan.waves, who));
    SSU_TRY(check_launch(plan.own.groups, 64 * plan.own.waves, who));
    DeviceGuard guard;
    SSU_TRY(guard.enter(a.device));
    if (args->prefix_pages > 0 && a.num_pages > 0) {
        const PrefixFn fn = a.q.dtype == SSU_BF16 ? prefix_kernel<Bf16>(a.headdim) : prefix_kernel<F16>(a.headdim);
        const hipError_t e = launch_kernel(fn, p, groups, 64 * plan.waves, 0, stream);
        if (e != hipSuccess)
            return fail(SSU_ERR_HIP, "%s: launch of the prefix kernel failed: %s", who, hipGetErrorString(e));
    }
    return launch_attn<true>(a, plan.own, p.a, who, stream);
}

}  // extern "C"
