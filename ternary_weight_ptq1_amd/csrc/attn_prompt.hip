// attn_prompt.hip -- attention over whole packed prompts (ptq1_attn_prompt).
//
//   out_i = sum_j p_ij V_j / sum_j p_ij,  p_ij = exp2(t_ij - m_i),
//   t_ij = scale log2(e) (q_i . K_j),     j over the keys that query i sees
//
// in one pass over the keys with a running maximum m_i.  Bounded by the
// matrix cores: 2 d multiply-adds for every visible pair, against 2 bytes of
// each operand.  Measured: 16384 tokens, 40 heads over 8 of 128, causal:
// 2.5 ms (1100 TFLOP/s of visible pairs; a library matrix product 1180 to
// 1350), matrix cores busy 60% of the cycles and vector units 49%, at a clock
// of 1.75 GHz; 9 prompts of 5 to 2500 tokens 87 us; 33 tokens 8.7 us.  64-wide
// heads have twice the exponentials for a product: 8192 tokens of 32 heads over
// 8 reach 920 TFLOP/s with the vector units 72% busy and the matrix cores 48%.
//
// The weights enter the second product as one 16-bit term, rounded once, and
// the rounded ones are summed, in fp32.  Values without a mean under many alike
// weights show it most: the rows' error against 64 bits, relative to their
// norm, is 2.15e-3 in bf16 for 16384 tokens (1.64e-3 the rounding of the result
// alone) and 2.6e-4 in fp16 (2.0e-4); with sharper weights or a mean of the
// values, 3 times their spread, it is that rounding's plus 1% (summed unrounded
// plus 9%).  A second term for the rest costs half of the matrix work again and
// more registers: 16384 tokens 2640 -> 3670 us, 9 prompts 98 -> 125, 33 tokens
// 8.8 -> 9.3 (one card); and of 256-wide heads the pairs' weights would not fit
// into LDS beside the tiles.
//
// Rows.  The query rows of a kv head are its group's heads of every token
// (row r = token r / group, head r % group): a tile of 128 rows then shares
// all its K and V, fills up for a few tokens already, and its causal border
// crosses few keys.
//
// One wave owns 32 rows, four a workgroup.  S^T = K Q^T and O^T = V^T P^T on
// 32x32x16 MFMA, so that a lane holds the scores of ONE row (column lane %
// 32): the maximum and sum of a row are in-lane but for one swap between lane
// l and l + 32.  The score registers of a lane are keys 8 b + 4 (lane / 32) +
// i, and any assignment of keys to the k-slots of the second product is as
// good as another if both operands follow it: slot j < 4 takes block 2 s and
// j >= 4 block 2 s + 1, so P needs no exchange at all, and the V operand is
// two transposing LDS reads of four keys each.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "ptq1_attn.h"
#include "ptq1_attn_tile.h"
#include "ptq1_launch.h"

namespace ptq1 {
namespace {

constexpr int kAhead = 4;               // K reads ahead of their products

// Query rows of a workgroup: 32 a wave, or a pair of waves (256-wide heads).
constexpr int kPrRows = 128;
// Waves of a workgroup.
constexpr int prompt_waves(int d) { return d == 256 ? 8 : 4; }

// The 16-byte piece p of key row r of a K or V tile lies at piece p ^ swizzle
// of that row.  K is read 16 rows at one piece at a time, V 4 rows at four
// pieces; the exclusive-or spreads either over the 64 banks.
template <int D>
__device__ __forceinline__ int k_swizzle(int r)
{
    return D >= 128 ? r & 15 : (r >> 1) & 7;
}
template <int D>
__device__ __forceinline__ int v_swizzle(int r)
{
    return D >= 128 ? (r & 3) << 2 : ((r >> 1) & 1) << 2;
}
template <int D>
__device__ __forceinline__ int k_place(int r, int p)
{
    return r * D + ((p ^ k_swizzle<D>(r)) << 3);
}
template <int D>
__device__ __forceinline__ int v_place(int r, int p)
{
    return r * D + ((p ^ v_swizzle<D>(r)) << 3);
}

// Keys that query `tok` of a sequence sees, with `off` keys before its first
// query and `lk` in all: the first so many.
__device__ __forceinline__ int visible(const PromptArgs &a, int tok, int off, int lk)
{
    const int n = a.causal ? tok + off + 1 : lk;
    return n > 0 ? n : 0;
}

// One tile of R query rows of one kv head, and the keys of one workgroup (all
// below 2^31: the host has seen to it).  The tiles of a kv head are numbered
// densely; those from plan.whole on have plan.splits workgroups each.
struct PromptTile {
    int q0, k0, lk, off;    // the sequence: its first rows, its keys, keys before its first query
    int rows, row0, end;    // its rows; this tile's first one and the one behind its last
    int group, kh;
    int reach;              // keys that some row of the tile sees; of them, this workgroup's:
    int first, any, all;    // the first one, the one behind the last, and where the first comes that not every row sees
    bool split;             // there are several workgroups
    int cut;                // its number among the tiles that may be cut, of all kv heads
};

// The place of a row's parts: by tile where only the last tiles are cut, else
// by row and head (tiles of few rows would leave much of theirs unused).
__device__ __forceinline__ int64_t part_row(const PromptArgs &a, const PromptPlan &plan, const PromptTile &t, int tok,
                                            int head, int row)
{
    return plan.whole > 0 ? static_cast<int64_t>(t.cut) * kPrRows + (row - t.row0)
                          : static_cast<int64_t>(t.q0 + tok) * a.hq + head;
}

// Workgroups go to the eight XCDs in turn, each with an L2 of its own: heads
// vary fastest, so that a head's tiles meet on as few XCDs as its number
// allows (eight heads: one each).  False: nothing (more) to do.  The rows of
// a sequence past its bounds, or with rows that are not there, become NaN.
template <typename T, int D>
__device__ __forceinline__ bool prompt_tile(const PromptArgs &a, const PromptPlan &plan, bool join, int &part, PromptTile &t)
{
    constexpr int R = kPrRows;
    t.group = a.hq / a.hkv;
    t.kh = static_cast<int>(blockIdx.x % static_cast<uint32_t>(a.hkv));
    int number = static_cast<int>(blockIdx.x / static_cast<uint32_t>(a.hkv));
    // all first parts of the tiles that are cut, then all second ones ...; no
    // branch, which would take another trip to the arguments (0.4 us of a
    // short prompt's 9); exact below 2^20 workgroups of a kv head
    part = 0;
    if (join)
        number += plan.whole;
    else {
        part = static_cast<int>(fmaxf((static_cast<float>(number - plan.whole) + 0.5f) * plan.per_cut, 0.0f));
        part = __builtin_amdgcn_readfirstlane(part);
        number -= part * (plan.tiles - plan.whole);
    }
    int64_t b, at, q0, k0, lq, lk;
    if (a.batch <= 64) {
        int qf = 0, qe = 0, kf = 0, ke = 0;  // the lane's sequence (all four at once: one trip to memory)
        if (!find_tile<true>(
                number, a.batch,
                [&](int64_t i) {
                    qf = a.cu_q[i];
                    qe = a.cu_q[i + 1];
                    kf = a.cu_k[i];
                    ke = a.cu_k[i + 1];
                    // only rows that exist count
                    const int64_t first = qf, end = qe;
                    const int64_t n = (end < a.q_rows ? end : a.q_rows) - (first > 0 ? first : 0);
                    return n > 0 ? (n * t.group + R - 1) / R : 0;
                },
                b, at))
            return false;
        const int who = static_cast<int>(b);
        q0 = __builtin_amdgcn_readlane(qf, who);
        lq = __builtin_amdgcn_readlane(qe, who) - q0;
        k0 = __builtin_amdgcn_readlane(kf, who);
        lk = __builtin_amdgcn_readlane(ke, who) - k0;
    } else {
        // Large batches in the order they come, without counting through all
        // sequences: 128 prompts of 512 tokens 592 us (801 counted, the longest
        // first), 4096 of 16 tokens 640 us (18400).  9 prompts of 5 to 2500
        // tokens: 92 to 95 us with the longest first, 94 to 100 as they come.
        if (!find_rows<R>(number, a.cu_q, a.batch, a.q_rows, t.group, b, at)) return false;
        b = __builtin_amdgcn_readfirstlane(static_cast<int>(b));
        at = __builtin_amdgcn_readfirstlane(static_cast<int>(at));
        q0 = a.cu_q[b];
        lq = a.cu_q[b + 1] - q0;
        k0 = a.cu_k[b];
        lk = a.cu_k[b + 1] - k0;
    }
    if (q0 < 0 || k0 < 0 || q0 + lq > a.q_rows || lk < 0 || k0 + lk > a.k_rows || lq > a.max_q || lk > a.max_k) {
        const int64_t r = (q0 < 0 ? -q0 * t.group : 0) + at * R + threadIdx.x, tok = q0 + r / t.group;
        if (!join && part == 0 && threadIdx.x < R && tok < q0 + lq && tok < a.q_rows) {
            T *dst = static_cast<T *>(a.out) + (tok * a.hq + t.kh * t.group + r % t.group) * D;
            const float n = __builtin_nanf("");
            for (int e = 0; e < D; e += 4) store4(dst + e, at_f32x4{n, n, n, n});
        }
        return false;
    }
    t.q0 = static_cast<int>(q0);
    t.k0 = static_cast<int>(k0);
    t.lk = static_cast<int>(lk);
    t.off = static_cast<int>(lk - lq);
    t.rows = static_cast<int>(lq) * t.group;
    // the last rows see the most keys: they start first
    t.row0 = ((t.rows + R - 1) / R - 1 - static_cast<int>(at)) * R;
    t.end = t.row0 + R < t.rows ? t.row0 + R : t.rows;
    t.reach = visible(a, (t.end - 1) / t.group, t.off, t.lk);
    t.split = number >= plan.whole && t.reach > plan.chunk;
    t.cut = (number - plan.whole) * a.hkv + t.kh;
    t.first = part * plan.chunk;
    if (t.first >= t.reach && part > 0) return false;
    t.any = t.split && t.reach - t.first > plan.chunk ? t.first + plan.chunk : t.reach;
    const int every = visible(a, t.row0 / t.group, t.off, t.lk);
    t.all = every < t.any ? every : t.any;
    return true;
}

// One lane's query row (column lane % 32 of its tile of 32).
struct PromptRow {
    bool is;
    int at, tok, head;
    int seen;  // keys that it sees
};
__device__ __forceinline__ PromptRow prompt_row(const PromptArgs &a, const PromptTile &t, int row)
{
    PromptRow r;
    r.is = row < t.rows;
    const int at = r.is ? row : t.rows - 1;
    r.at = at;
    r.tok = at / t.group;
    r.head = t.kh * t.group + at % t.group;
    r.seen = visible(a, r.tok, t.off, t.lk);
    return r;
}

// Adds to O^T, dimensions d0 + 32 i + ..., the NaNs and infinities among the
// values from key `border` on that the row sees (they were left out of the
// products, or a zero weight would have carried them to rows that do not).
template <typename T, int N>
__device__ __forceinline__ void add_non_finite(const PromptArgs &a, const PromptTile &t, const PromptRow &row, int border,
                                               int d, int d0, int half, at_f32x16 (&o)[N])
{
    for (int r = border; r < t.any; ++r) {
        const T *src = static_cast<const T *>(a.v) + static_cast<int64_t>(t.k0 + r) * a.vs + static_cast<int64_t>(t.kh) * d + d0 + 4 * half;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
                const at_f32x4 x = load4(src + 32 * i + 2 * j);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (r < row.seen && !(fabsf(x[e]) <= 3.4028235e38f)) o[i][j + e] += x[e];
            }
    }
}

// The row's dimensions d0 + 32 i + 8 b + 4 half + e, finished, or as one part of several.
template <typename T, int N>
__device__ __forceinline__ void store_rows(const PromptArgs &a, const PromptPlan &plan, const PromptTile &t, const PromptRow &row,
                                           int part, int d, int d0, int half, const at_f32x16 (&o)[N], float m, float l,
                                           float *parts)
{
    const int64_t at = static_cast<int64_t>(t.q0 + row.tok) * a.hq + row.head;
    if (!t.split) {
        T *dst = static_cast<T *>(a.out) + at * d + d0 + 4 * half;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < 16; j += 4)
                store4(dst + 32 * i + 2 * j, at_f32x4{o[i][j], o[i][j + 1], o[i][j + 2], o[i][j + 3]});
        return;
    }
    const int64_t slot = part_row(a, plan, t, row.tok, row.head, row.at) * plan.splits + part;
    float *dst = parts + slot * d + d0 + 4 * half;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 16; j += 4)
            store4(dst + 32 * i + 2 * j, at_f32x4{o[i][j], o[i][j + 1], o[i][j + 2], o[i][j + 3]});
    if (half == 0 && d0 == 0) {
        parts[plan.rows_floats + slot * 2] = m;
        parts[plan.rows_floats + slot * 2 + 1] = l;
    }
}

// A NaN or an infinity leaves a V tile in LDS (zeros in its place); true if there was one.
template <typename T, int D>
__device__ __forceinline__ bool clean_tile(T *vb)
{
    bool odd = false;
    for (int i = threadIdx.x; i < kKeys * (D / 8); i += 64 * prompt_waves(D)) {
        at_u32x4 w = *reinterpret_cast<const at_u32x4 *>(vb + 8 * i);
        if (clear_non_finite<T>(w)) {
            *reinterpret_cast<at_u32x4 *>(vb + 8 * i) = w;
            odd = true;
        }
    }
    return odd;
}

// A lane's share of copying tiles of 64 rows straight from memory into LDS:
// 64 pieces of 16 bytes per wave instruction at consecutive places; the lane
// picks the piece that belongs there.  The tile's address is in the (scalar)
// buffer descriptor, the lane's part a 32-bit offset that stays: piece i is
// i * RS rows further on, where the swizzle is the same.  The descriptor ends with row `rows` - 1: nothing behind it is read.
template <typename T, int D, bool V>
struct Staging {
    static constexpr int W = prompt_waves(D), P = D / 8, RS = 64 * W / P, N = kKeys / RS;
    static_assert(RS % 16 == 0 || (V && RS % 4 == 0), "the swizzle is the same RS rows further on");
    const char *base;
    int64_t stride;  // bytes
    uint32_t off;
    __device__ __forceinline__ Staging(const void *src, int64_t row, int64_t row_stride, int kh)
        : base(reinterpret_cast<const char *>(static_cast<const T *>(src) + row * row_stride + static_cast<int64_t>(kh) * D)),
          stride(row_stride * 2)
    {
        const uint32_t r = threadIdx.x / P, p = threadIdx.x % P;
        off = r * static_cast<uint32_t>(stride) + 16 * (p ^ (V ? v_swizzle<D>(r) : k_swizzle<D>(r)));
    }
    // rows n0 .. n0 + 63, of `rows`
    __device__ __forceinline__ void copy(T *dst, int n0, int rows) const
    {
        const uint32_t step = static_cast<uint32_t>(stride);
        const uint32_t more = rows - 1 - n0 < kKeys - 1 ? rows - 1 - n0 : kKeys - 1;  // rows behind the first
        const char *src = base + n0 * stride;
        const int wave = threadIdx.x >> 6;
#pragma unroll
        for (int i = 0; i < N; ++i)
            copy_to_lds(src, more * step + 2 * D, off + i * RS * step, dst + (i * W + wave) * 512);
    }
};

// The V operand of keys 16 u .. + 15, dimensions 32 i .. + 31: lane: key 16 u
// + 4 half + (lane % 16) / 4 (then + 8), dimensions 32 i + 16 ((lane / 16) %
// 2) + 4 (lane % 4) of two transposing reads.
template <typename T, int D>
__device__ __forceinline__ typename Op16<T>::x8 read_v(const T *vb, int u, int i)
{
    const int lane = threadIdx.x & 63;
    const int r = 16 * u + 4 * (lane >> 5) + ((lane & 15) >> 2);
    const int d = 32 * i + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
    const at_s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(vb + v_place<D>(r, d >> 3) + (d & 7)));
    const at_s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(vb + v_place<D>(r + 8, d >> 3) + (d & 7)));
    return __builtin_bit_cast(typename Op16<T>::x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

template <typename T, int D>
__global__ void __launch_bounds__(64 * prompt_waves(D), 2) k_attn_prompt(PromptArgs a, PromptPlan plan, float *parts)
{
    typedef typename Op16<T>::x8 x8;
    constexpr int BN = kKeys;
    constexpr int KT = BN / 32;             // score tiles
    constexpr int DT = D / 32;              // output tiles
    constexpr int KK = D / 16;              // MFMA steps over the head dimension

    // Two tiles each: separate objects, so that the copies into one need not
    // have ended before the other is read.
    __shared__ __attribute__((aligned(16))) T kt0[BN * D], kt1[BN * D], vt0[BN * D], vt1[BN * D];
    __shared__ int odd_values;  // a NaN or an infinity was met in a V tile on the causal border

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = lane & 31, half = lane >> 5;
    int piece;
    PromptTile t;
    if (!prompt_tile<T, D>(a, plan, false, piece, t)) return;
    const int any = t.any, all = t.all;
    int seen = 0;  // (set for the border tiles; the others use every key)

    // ---- queries: B operand, column = row, k = 16 kk + 8 half + j
    x8 qf[KK];
    {
        const PromptRow row = prompt_row(a, t, t.row0 + 32 * wave + col);
        const T *qp = static_cast<const T *>(a.q) + static_cast<int64_t>(t.q0 + row.tok) * a.qs + static_cast<int64_t>(row.head) * D;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) qf[kk] = *reinterpret_cast<const x8 *>(qp + 16 * kk + 8 * half);
    }
    const Staging<T, D, false> keys(a.k, t.k0, a.ks, t.kh);
    const Staging<T, D, true> values(a.v, t.k0, a.vs, t.kh);

    const float c = a.scale * kLog2e;
    at_f32x16 o[DT];
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] = 0.0f;
    float m = -__builtin_inff(), l = 0.0f, l2 = 0.0f;  // m: the reference, in units of log2
    bool large = false;

    // S^T of the tile in kb
    auto scores = [&](at_f32x16 (&s)[KT], const T *kb) {
#pragma unroll
        for (int t = 0; t < KT; ++t) {
#pragma unroll
            for (int j = 0; j < 16; ++j) s[t][j] = 0.0f;
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                const x8 kf = *reinterpret_cast<const x8 *>(kb + k_place<D>(32 * t + col, 2 * kk + half));
                s[t] = Op16<T>::mfma32(kf, qf[kk], s[t]);
            }
        }
    };
    auto hide = [&](at_f32x16 (&s)[KT], int n0) {
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (n0 + 32 * t + 8 * (j >> 2) + 4 * half + (j & 3) >= seen) s[t][j] = -__builtin_inff();
    };
    auto largest = [&](const at_f32x16 (&s)[KT]) {
        float top = s[0][0];
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int j = 0; j < 16; ++j) top = fmaxf(top, s[t][j]);
        return lane_pair_max<32>(top) * c;
    };
    // The reference in use may lag by 8 (weights up to 2^8 lose nothing in
    // either type): few tiles after the first rescale.
    auto raise = [&](float top) {
        const float mt = reference<T>(top);
        if (__ballot(mt > m + 8.0f) != 0) {
            const float mn = fmaxf(m, mt);
            const float f = m == mn ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
            l *= f;
            l2 *= f;
#pragma unroll
            for (int i = 0; i < DT; ++i) o[i] *= f;
            m = mn;
            large = large_scores(m);
        }
    };

    // One tile: its scores, weights and products, while the next one arrives
    // in the other buffers.
    auto step = [&](auto border, const T *kb, T *vb, T *kn, T *vn, int n0) {
        constexpr bool BORDER = decltype(border)::value;  // some row may not see some key of the tile
        if (n0 + BN < any) {
            keys.copy(kn, n0 + BN, any);
            values.copy(vn, n0 + BN, any);
        }
        at_f32x16 s[KT];
        scores(s, kb);
        // the K reads run ahead of the products
        __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
        for (int i = 0; i < KT * KK - kAhead; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x8, kAhead, 0);
        if constexpr (BORDER) hide(s, n0);
        raise(largest(s));
        const float ms = m == -__builtin_inff() ? 0.0f : m;
        float mul = c;
        if (large) {
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int j = 0; j < 16; ++j) s[t][j] *= c;
            mul = 1.0f;
        }
        x8 pf[2 * KT];
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                pf[2 * t + (j >> 3)][j & 7] = static_cast<T>(__builtin_amdgcn_exp2f(fmaf(s[t][j], mul, -ms)));
            }
#pragma unroll
        for (int u = 0; u < 2 * KT; u += 2) {
            l = add_weights<T>(pf[u], l);
            l2 = add_weights<T>(pf[u + 1], l2);
        }
        if constexpr (BORDER) {
            // Some rows do not see some of these keys, and a zero weight would
            // not keep a NaN or an infinity out of them: such values leave the
            // tile and are given to the rows that see them at the end.
            if (clean_tile<T, D>(vb)) odd_values = 1;
            __syncthreads();
        }
        // ---- O^T += V^T P^T
#pragma unroll
        for (int u = 0; u < 2 * KT; ++u) {
#pragma unroll
            for (int i = 0; i < DT; ++i) o[i] = Op16<T>::mfma32(read_v<T, D>(vb, u, i), pf[u], o[i]);
        }
        __syncthreads();
    };

    if (threadIdx.x == 0) odd_values = 0;
    if (t.first < any) {
        keys.copy(kt0, t.first, any);
        values.copy(vt0, t.first, any);
    }
    __syncthreads();
    int n0 = t.first;
    for (; n0 + 2 * BN <= all; n0 += 2 * BN) {
        step(std::false_type{}, kt0, vt0, kt1, vt1, n0);
        step(std::false_type{}, kt1, vt1, kt0, vt0, n0 + BN);
    }
    const int border = n0;
    // the row anew: kept through the loop it takes registers that the V reads run ahead in
    int again = col;
    asm volatile("" : "+v"(again));
    const PromptRow row = prompt_row(a, t, t.row0 + 32 * wave + again);
    seen = row.seen;
    for (; n0 < any; n0 += 2 * BN) {
        step(std::true_type{}, kt0, vt0, kt1, vt1, n0);
        if (n0 + BN >= any) break;
        step(std::true_type{}, kt1, vt1, kt0, vt0, n0 + BN);
    }
    l = lane_pair_sum<32>(l + l2);
    const float f = t.split ? 1.0f : seen == 0 ? 0.0f : 1.0f / l;
#pragma unroll
    for (int i = 0; i < DT; ++i) o[i] *= f;
    if (t.first < any && odd_values != 0) add_non_finite<T, DT>(a, t, row, border, D, 0, half, o);
    if (row.is) store_rows<T, DT>(a, plan, t, row, piece, D, 0, half, o, m, l, parts);
}

// The same for 256-wide heads, whose O^T and queries for 32 rows take 192
// registers of a lane: a pair of waves shares 32 rows.  Each makes the scores
// of one half of a tile's 64 keys and forms their weights, the pair exchanges
// maxima and weights through LDS, and each multiplies all 64 keys' weights
// with one half of the dimensions.  Eight waves, 128 rows, share the tiles: one
// workgroup a CU, two waves a SIMD.  4000 queries of 24 heads over as many
// keys: 238 us (826 TFLOP/s of visible pairs); one wave for 32 rows (one a
// SIMD) took 286, pairs in workgroups of four waves with one buffer each for K
// and V (two a CU; the copies have half a tile's time) 251, the next tile's
// scores taken beside this one's weights 266 (the matrix cores and the vector
// units then overlap in a wave, but the registers leave no reads ahead).  At
// 8192 tokens the matrix cores are 44% busy and the vector units 26%: the eight
// waves run in step, by three barriers a tile.  15 registers of a lane are
// spilled around the main loop (by the set-up, the border tiles and the end),
// none in it.
//
template <typename T>
__global__ void __launch_bounds__(64 * prompt_waves(256), 2) k_attn_prompt_wide(PromptArgs a, PromptPlan plan, float *parts)
{
    typedef typename Op16<T>::x8 x8;
    constexpr int D = 256, BN = kKeys, DT = 4, KK = D / 16;
    __shared__ __attribute__((aligned(16))) T kt0[BN * D], kt1[BN * D], vt0[BN * D], vt1[BN * D];
    __shared__ x8 weights[4][4][64];   // [pair][k-step of 16 keys][lane]
    __shared__ float tops[4][2][32];   // [pair][key half][row]
    __shared__ int odd_values;

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = lane & 31, half = lane >> 5;
    const int pair = wave >> 1, part = wave & 1;
    int piece;
    PromptTile t;
    if (!prompt_tile<T, D>(a, plan, false, piece, t)) return;
    const PromptRow row = prompt_row(a, t, t.row0 + 32 * pair + col);
    const int seen = row.seen, any = t.any, all = t.all;

    x8 qf[KK];
    {
        const T *qp = static_cast<const T *>(a.q) + static_cast<int64_t>(t.q0 + row.tok) * a.qs + static_cast<int64_t>(row.head) * D;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) qf[kk] = *reinterpret_cast<const x8 *>(qp + 16 * kk + 8 * half);
    }
    const Staging<T, D, false> keys(a.k, t.k0, a.ks, t.kh);
    const Staging<T, D, true> values(a.v, t.k0, a.vs, t.kh);
    const float c = a.scale * kLog2e;
    at_f32x16 o[DT];  // dimensions 128 part + 32 i + ...
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] = 0.0f;
    float m = -__builtin_inff(), l = 0.0f, l2 = 0.0f;  // l: of this wave's keys
    bool large = false;

    auto step = [&](auto border, const T *kb, T *vb, T *kn, T *vn, int n0) {
        constexpr bool BORDER = decltype(border)::value;
        if (n0 + BN < any) {
            keys.copy(kn, n0 + BN, any);
            values.copy(vn, n0 + BN, any);
        }
        // ---- S^T of keys 32 part ..
        at_f32x16 s;
#pragma unroll
        for (int j = 0; j < 16; ++j) s[j] = 0.0f;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
            s = Op16<T>::mfma32(*reinterpret_cast<const x8 *>(kb + k_place<D>(32 * part + col, 2 * kk + half)), qf[kk], s);
        __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
        for (int i = 0; i < KK - kAhead; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x8, kAhead, 0);
        if constexpr (BORDER) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (n0 + 32 * part + 8 * (j >> 2) + 4 * half + (j & 3) >= seen) s[j] = -__builtin_inff();
        }
        float top = s[0];
#pragma unroll
        for (int j = 1; j < 16; ++j) top = fmaxf(top, s[j]);
        top = lane_pair_max<32>(top) * c;
        if (half == 0) tops[pair][part][col] = top;
        barrier_lds();
        top = fmaxf(top, tops[pair][part ^ 1][col]);
        const float mt = reference<T>(top);
        if (__ballot(mt > m + 8.0f) != 0) {  // the same in both waves
            const float mn = fmaxf(m, mt);
            const float f = m == mn ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
            l *= f;
            l2 *= f;
#pragma unroll
            for (int i = 0; i < DT; ++i) o[i] *= f;
            m = mn;
            large = large_scores(m);
        }
        const float ms = m == -__builtin_inff() ? 0.0f : m;
        float mul = c;
        if (large) {
#pragma unroll
            for (int j = 0; j < 16; ++j) s[j] *= c;
            mul = 1.0f;
        }
        x8 pf[2];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            pf[j >> 3][j & 7] = static_cast<T>(__builtin_amdgcn_exp2f(fmaf(s[j], mul, -ms)));
        }
        l = add_weights<T>(pf[0], l);
        l2 = add_weights<T>(pf[1], l2);
        weights[pair][2 * part][lane] = pf[0];
        weights[pair][2 * part + 1][lane] = pf[1];
        if constexpr (BORDER) {
            if (clean_tile<T, D>(vb)) odd_values = 1;
        }
        barrier_lds();
        // ---- O^T of dimensions 128 part ..
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const x8 w = weights[pair][u][lane];
#pragma unroll
            for (int i = 0; i < DT; ++i) o[i] = Op16<T>::mfma32(read_v<T, D>(vb, u, DT * part + i), w, o[i]);
        }
        barrier_copies();  // all have read, the next tile is there
    };

    if (threadIdx.x == 0) odd_values = 0;
    if (t.first < any) {
        keys.copy(kt0, t.first, any);
        values.copy(vt0, t.first, any);
    }
    barrier_copies();
    int n0 = t.first;
    for (; n0 + 2 * BN <= all; n0 += 2 * BN) {
        step(std::false_type{}, kt0, vt0, kt1, vt1, n0);
        step(std::false_type{}, kt1, vt1, kt0, vt0, n0 + BN);
    }
    const int border = n0;
    for (; n0 < any; n0 += 2 * BN) {
        step(std::true_type{}, kt0, vt0, kt1, vt1, n0);
        if (n0 + BN >= any) break;
        step(std::true_type{}, kt1, vt1, kt0, vt0, n0 + BN);
    }

    // the pair's sums
    l = lane_pair_sum<32>(l + l2);
    __syncthreads();
    if (half == 0) tops[pair][part][col] = l;
    __syncthreads();
    l = tops[pair][0][col] + tops[pair][1][col];
    const float f = t.split ? 1.0f : seen == 0 ? 0.0f : 1.0f / l;
#pragma unroll
    for (int i = 0; i < DT; ++i) o[i] *= f;
    if (t.first < any && odd_values != 0) add_non_finite<T, DT>(a, t, row, border, D, 128 * part, half, o);
    if (row.is) store_rows<T, DT>(a, plan, t, row, piece, D, 128 * part, half, o, m, l, parts);
}

// Joins the chunks of the tiles that were split: D / 4 lanes per row, one row
// each (blockIdx.y: the part of a tile's rows).
constexpr int join_rows(int d) { return 256 / (d / 4); }

template <typename T, int D>
__global__ void __launch_bounds__(256) k_prompt_join(PromptArgs a, PromptPlan plan, const float *part)
{
    constexpr int LPR = D / 4;
    int piece;
    PromptTile t;
    if (!prompt_tile<T, D>(a, plan, true, piece, t) || !t.split) return;
    const int n = (t.reach + plan.chunk - 1) / plan.chunk;
    const int x = threadIdx.x % LPR;
    const int r = t.row0 + static_cast<int>(blockIdx.y * join_rows(D) + threadIdx.x / LPR);
    if (r >= t.end) return;
    const PromptRow row = prompt_row(a, t, r);
    const int64_t at = static_cast<int64_t>(t.q0 + row.tok) * a.hq + row.head;
    const int64_t place = part_row(a, plan, t, row.tok, row.head, r) * plan.splits;
    const float *ml = part + plan.rows_floats + place * 2, *src = part + place * D + 4 * x;
    float M = -__builtin_inff();
    for (int i = x; i < n; i += LPR) M = fmaxf(M, ml[2 * i]);
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) M = fmaxf(M, __shfl_xor(M, o, 64));
    if (M == -__builtin_inff()) M = 0.0f;
    float L = 0.0f;
    at_f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
        const float w = __builtin_amdgcn_exp2f(ml[2 * i] - M);
        L += w * ml[2 * i + 1];
        o += w * *reinterpret_cast<const at_f32x4 *>(src + static_cast<int64_t>(i) * D);
    }
    store4(static_cast<T *>(a.out) + at * D + 4 * x, o * (row.seen == 0 ? 0.0f : 1.0f / L));
}

template <typename T, int D>
hipError_t prompt_launch(const PromptArgs &a, const PromptPlan &plan, float *part, hipStream_t s)
{
    const int cut = plan.tiles - plan.whole;
    const dim3 grid(static_cast<uint32_t>((plan.whole + cut * plan.splits) * a.hkv));
    if constexpr (D == 256)
        hipLaunchKernelGGL((k_attn_prompt_wide<T>), grid, dim3(64 * prompt_waves(D)), 0, s, a, plan, part);
    else
        hipLaunchKernelGGL((k_attn_prompt<T, D>), grid, dim3(64 * prompt_waves(D)), 0, s, a, plan, part);
    if (plan.splits > 1)
        hipLaunchKernelGGL((k_prompt_join<T, D>), dim3(static_cast<uint32_t>(cut * a.hkv), kPrRows / join_rows(D)), dim3(256), 0, s, a, plan, part);
    return hipGetLastError();
}

template <typename T>
hipError_t prompt_d(const PromptArgs &a, int d, const PromptPlan &plan, float *part, hipStream_t s)
{
    return d == 64 ? prompt_launch<T, 64>(a, plan, part, s)
                   : d == 128 ? prompt_launch<T, 128>(a, plan, part, s) : prompt_launch<T, 256>(a, plan, part, s);
}

}  // namespace

// Whole tiles of all rows, and a part of one for every sequence.
int64_t prompt_tiles(int64_t batch, int64_t q_rows, int32_t hq, int32_t hkv)
{
    return q_rows * (hq / hkv) / kPrRows + batch;
}

// Bytes of parts above which nothing is cut: max_k may be a bound that no
// sequence comes near.
constexpr double kMaxParts = 1 << 28;

PromptPlan prompt_plan(int64_t batch, int64_t q_rows, int64_t max_k, int32_t hq, int32_t hkv, int32_t d, int64_t k_rows)
{
    // The time with tiles cut in n along their keys, in us: rounds of
    // workgroups, each of a key's time as measured with the GPU full, and from
    // n = 2 on the parts' rows in fp32 (written and read, at half of HBM's rate:
    // they come in bursts) and the join.  Either all tiles are cut, or only
    // those behind the last full round of whole ones, if the tiles reach about
    // equally far: few queries behind many keys, and these at least 0.6 of the
    // longest sequence's on average (`even`).  16 queries over 8016 keys: 146 us
    // uncut, 20 in chunks of 512; 1657 queries of 24 heads of 256 over 4000 and
    // more, 320 tiles: 307 uncut, 266 all cut in two, 229 the last 64 in three;
    // 40 batches of 1 to 16 chunks behind contexts 0.93 of the time uncut (0.81
    // to 1.03), at an evenness of 0.5 1.01 to 1.05 times it.
    // A ragged batch of whole prompts has few queries by their mean as well, but
    // not as many keys.  Its last tiles are the shortest and fill the gaps as
    // they are, so where its tiles fill the GPU none is cut: 40 batches of 5 to
    // 33 prompts of 840 to 7800 tokens and less 0.96 of the time with the last
    // tiles cut (0.83 to 1.00); 1272 tiles of up to 2500 keys of 128, 89 us, took
    // 115 all cut in two.
    PromptPlan p;
    const double slots = d == 256 ? 256 : 512, key = d == 256 ? 0.04 : 0.029;  // workgroups the GPU holds
    const int64_t tiles = prompt_tiles(batch, q_rows, hq, hkv);
    p.tiles = static_cast<int32_t>(tiles);
    const bool few = batch > 0 && max_k >= 4 * (q_rows / batch);
    const bool even = static_cast<double>(k_rows) >= 0.6 * static_cast<double>(batch) * static_cast<double>(max_k);
    const int64_t full = few && even ? static_cast<int64_t>(static_cast<double>(tiles * hkv) / slots) * static_cast<int64_t>(slots) / hkv : 0;
    const int most = few && !even && static_cast<double>(tiles * hkv) > slots ? 1 : 64;
    double best = 0.0;
    int n = 1;
    for (const int64_t whole : {int64_t{0}, full}) {
        if (whole == 0 && best > 0.0) break;  // the same again
        const double rest = static_cast<double>((tiles - whole) * hkv);
        const double before = __builtin_ceil(static_cast<double>(whole * hkv) / slots) * static_cast<double>(max_k) * key;
        const double rows = whole > 0 ? rest * kPrRows : static_cast<double>(q_rows) * hq;
        for (int i = whole > 0 ? 2 : 1; i <= most && max_k / i >= 256; ++i) {
            if (i > 1 && rows * i * (d + 2) * 4 > kMaxParts) break;
            double us = before + __builtin_ceil(rest * i / slots) * static_cast<double>(max_k) / i * key;
            if (i > 1) us += 6.0 + rest * i * kPrRows * d * 4 * 2 / 2.5e6;
            if (i == 1 || us < best * 0.95) {
                best = us;
                n = i;
                p.whole = static_cast<int32_t>(whole);
            }
        }
    }
    p.chunk = static_cast<int32_t>(((max_k + n - 1) / n + 127) / 128 * 128);
    if (p.chunk == 0) p.chunk = 128;
    p.splits = static_cast<int32_t>(max_k > 0 ? (max_k + p.chunk - 1) / p.chunk : 1);
    if (p.splits == 1) p.whole = 0;
    if (p.splits > 1) {
        p.per_cut = 1.0f / static_cast<float>(tiles - p.whole);
        const size_t rows = p.whole > 0 ? static_cast<size_t>(tiles - p.whole) * hkv * kPrRows : static_cast<size_t>(q_rows) * hq;
        p.rows_floats = rows * p.splits * d;
        p.part_floats = p.rows_floats + rows * p.splits * 2;
    }
    return p;
}

hipError_t launch_attn_prompt(const PromptArgs &a, int dtype, int32_t d, const PromptPlan &plan, float *part, hipStream_t s)
{
    return dtype == PTQ1_BF16 ? prompt_d<__bf16>(a, d, plan, part, s) : prompt_d<_Float16>(a, d, plan, part, s);
}

}  // namespace ptq1
