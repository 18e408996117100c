// attn_prompt.hip -- attention over whole packed prompts (ptq1_attn_prompt).
//
//   out_i = sum_j p_ij V_j / sum_j p_ij,  p_ij = exp2(t_ij - m_i),
//   t_ij = scale log2(e) (q_i . K_j),     j over the keys that query i sees
//
// in one pass over the keys with a running maximum m_i.  Bounded by the
// matrix cores: 4 d multiply-adds for every visible pair, against 2 bytes of
// each operand.
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
#include "ptq1_launch.h"

namespace ptq1 {
namespace {

constexpr int kPrWaves = 4;
constexpr int kPrThreads = 64 * kPrWaves;
constexpr int kPrRows = 32 * kPrWaves;  // query rows of a workgroup
constexpr int kJoinParts = 4;           // workgroups that join one tile
constexpr int kAhead = 4;               // K reads ahead of their products

typedef short at_s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) at_s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) void lds_void;
constexpr int kBufferFlags = 0x00027000;  // raw buffer of bytes

constexpr int prompt_keys(int d) { return d == 256 ? 32 : 64; }

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

// 16 bytes per lane from base + off to 1024 consecutive bytes of LDS; bytes
// from `bytes` on are not read.
__device__ __forceinline__ void copy_to_lds(const char *base, uint32_t bytes, uint32_t off, void *dst)
{
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(base), 0, static_cast<int>(bytes), kBufferFlags);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void *)dst, 16, static_cast<int>(off), 0, 0, 0);
}

// Zeros in the place of NaNs and infinities (an exponent of all ones) among
// eight values; true if there was one.
template <typename T>
__device__ __forceinline__ bool clear_non_finite(at_u32x4 &w)
{
    constexpr uint32_t E = std::is_same<T, __bf16>::value ? 0x7f80u : 0x7c00u;
    bool found = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool lo = (w[i] & E) == E, hi = (w[i] & (E << 16)) == (E << 16);
        w[i] &= (lo ? 0xffff0000u : ~0u) & (hi ? 0xffffu : ~0u);
        found |= lo || hi;
    }
    return found;
}

// The flat tile's sequence and its place there, counted from the end; only
// rows that exist count.
__device__ __forceinline__ bool prompt_tile(const PromptArgs &a, int64_t flat, int64_t &b, int64_t &at)
{
    return find_tile<true>(
        flat, a.batch,
        [&](int64_t i) {
            const int64_t first = a.cu_q[i], end = a.cu_q[i + 1];
            const int64_t n = (end < a.q_rows ? end : a.q_rows) - (first > 0 ? first : 0);
            return n > 0 ? (n * (a.hq / a.hkv) + kPrRows - 1) / kPrRows : 0;
        },
        b, at);
}

// A sequence past its bounds, or with rows that are not there: its rows are NaN.
__device__ __forceinline__ bool prompt_refused(const PromptArgs &a, int64_t q0, int64_t lq, int64_t k0, int64_t lk)
{
    return q0 < 0 || k0 < 0 || q0 + lq > a.q_rows || lk < 0 || k0 + lk > a.k_rows || lq > a.max_q || lk > a.max_k;
}

// Keys that query `tok` of a sequence sees: the first so many.
__device__ __forceinline__ int visible(const PromptArgs &a, int64_t tok, int64_t off, int64_t lk)
{
    const int64_t n = a.causal ? tok + off + 1 : lk;
    return static_cast<int>(n > 0 ? n : 0);
}

template <typename T, int D>
__global__ void __launch_bounds__(kPrThreads, D == 256 ? 1 : 2) k_attn_prompt(PromptArgs a, PromptPlan plan, float *part)
{
    typedef typename Op16<T>::x8 x8;
    constexpr int BN = prompt_keys(D);      // keys of a tile
    constexpr int KT = BN / 32;             // score tiles
    constexpr int DT = D / 32;              // output tiles
    constexpr int KK = D / 16;              // MFMA steps over the head dimension
    constexpr int P = D / 8;                // 16-byte pieces of a row
    constexpr int NLD = BN * P / kPrThreads;  // pieces a thread stages, of K and of V

    // Two tiles each: separate objects, so that the copies into one need not
    // have ended before the other is read.
    __shared__ __attribute__((aligned(16))) T kt0[BN * D], kt1[BN * D], vt0[BN * D], vt1[BN * D];
    __shared__ int odd_values;  // a NaN or an infinity was met in a V tile on the causal border

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = lane & 31, half = lane >> 5;

    // Workgroups go to the eight XCDs in turn, each with an L2 of its own.
    // Heads vary fastest, so that a head's tiles meet on as few XCDs as its
    // number allows (eight heads: one each).
    const int group = a.hq / a.hkv;
    const int kh = static_cast<int>(blockIdx.x % static_cast<uint32_t>(a.hkv));
    const int64_t flat = blockIdx.x / static_cast<uint32_t>(a.hkv);
    int64_t b, at;
    if (!prompt_tile(a, flat, b, at)) return;
    const int64_t q0 = a.cu_q[b], k0 = a.cu_k[b];
    const int64_t lq = a.cu_q[b + 1] - q0, lk = a.cu_k[b + 1] - k0;
    const int64_t rows = lq * group;
    if (prompt_refused(a, q0, lq, k0, lk)) {
        const int64_t r = (q0 < 0 ? -q0 * group : 0) + at * kPrRows + threadIdx.x, tok = q0 + r / group;
        if (blockIdx.y == 0 && threadIdx.x < kPrRows && r < rows && tok < a.q_rows) {
            T *dst = static_cast<T *>(a.out) + (tok * a.hq + kh * group + r % group) * D;
            const float n = __builtin_nanf("");
            for (int e = 0; e < D; e += 4) store4(dst + e, at_f32x4{n, n, n, n});
        }
        return;
    }
    // the last rows see the most keys: they start first
    const int64_t tile = (rows + kPrRows - 1) / kPrRows - 1 - at;

    const int64_t row = tile * kPrRows + 32 * wave + col;
    const int64_t rowc = row < rows ? row : rows - 1;
    const int32_t tok = static_cast<int32_t>(rowc / group), head = static_cast<int32_t>(rowc % group);
    const int64_t off = lk - lq;
    // keys below `seen` are visible to this lane's row
    const int seen = visible(a, tok, off, lk);
    const int64_t tok_first = tile * kPrRows / group;
    const int64_t row_last = (tile + 1) * kPrRows < rows ? (tile + 1) * kPrRows - 1 : rows - 1;
    // keys that some row of the tile sees; of them, this workgroup's
    const int reach = visible(a, row_last / group, off, lk);
    const int first = static_cast<int>(blockIdx.y * plan.chunk);
    if (first >= reach && blockIdx.y > 0) return;
    const bool split = reach > plan.chunk;
    const int any = split && reach - first > plan.chunk ? first + static_cast<int>(plan.chunk) : reach;
    // keys that every row sees
    const int every = visible(a, tok_first, off, lk), all = every < any ? every : any;

    // ---- queries: B operand, column = row, k = 16 kk + 8 half + j
    x8 qf[KK];
    {
        const T *qp = static_cast<const T *>(a.q) + (q0 + tok) * a.qs + static_cast<int64_t>(kh * group + head) * D;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) qf[kk] = *reinterpret_cast<const x8 *>(qp + 16 * kk + 8 * half);
    }

    // ---- staging: straight from memory into LDS, 64 pieces of 16 bytes per
    // wave instruction at consecutive places; the lane picks the piece that
    // belongs there.  The tile's address is in the (scalar) buffer
    // descriptor, the lane's part a 32-bit offset that stays.  The
    // descriptor ends with the last visible key's row: nothing behind it is read.
    const char *kbase = reinterpret_cast<const char *>(static_cast<const T *>(a.k) + k0 * a.ks + static_cast<int64_t>(kh) * D);
    const char *vbase = reinterpret_cast<const char *>(static_cast<const T *>(a.v) + k0 * a.vs + static_cast<int64_t>(kh) * D);
    const uint32_t kstep = static_cast<uint32_t>(a.ks) * 2, vstep = static_cast<uint32_t>(a.vs) * 2;
    // piece i of a lane: rows i * RS further on, where the swizzle is the
    // same again after KC pieces
    constexpr int RS = kPrThreads / P, KC = D == 256 ? 2 : 1;
    uint32_t koff[KC], voff;
#pragma unroll
    for (int i = 0; i < KC; ++i) {
        const uint32_t r = i * RS + threadIdx.x / P, p = threadIdx.x % P;
        koff[i] = r * kstep + 16 * (p ^ k_swizzle<D>(r));
        if (i == 0) voff = r * vstep + 16 * (p ^ v_swizzle<D>(r));
    }
    auto stage_k = [&](T *dst, int n0) {
        const uint32_t more = any - 1 - n0 < BN - 1 ? any - 1 - n0 : BN - 1;  // rows behind the first
        const char *src = kbase + n0 * (a.ks * 2);
#pragma unroll
        for (int i = 0; i < NLD; ++i)
            copy_to_lds(src, more * kstep + 2 * D, koff[i % KC] + (i / KC * KC * RS) * kstep, dst + (i * kPrWaves + wave) * 512);
    };
    auto stage_v = [&](T *dst, int n0) {
        const uint32_t more = any - 1 - n0 < BN - 1 ? any - 1 - n0 : BN - 1;
        const char *src = vbase + n0 * (a.vs * 2);
#pragma unroll
        for (int i = 0; i < NLD; ++i)
            copy_to_lds(src, more * vstep + 2 * D, voff + (i * RS) * vstep, dst + (i * kPrWaves + wave) * 512);
    };

    const float c = a.scale * kLog2e;
    at_f32x16 o[DT];
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] = 0.0f;
    float m = -__builtin_inff(), l = 0.0f;  // m: in units of log2

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
    // The maximum in use may lag by 8 (weights up to 2^8 lose nothing in
    // either type): few tiles after the first rescale.
    auto raise = [&](float top) {
        if (__ballot(top > m + 8.0f) != 0) {
            const float mn = fmaxf(m, top);
            const float f = m == mn ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
            l *= f;
#pragma unroll
            for (int i = 0; i < DT; ++i) o[i] *= f;
            m = mn;
        }
    };

    // One tile: its scores, weights and products, while the next one arrives
    // in the other buffers.
    auto step = [&](auto border, const T *kb, T *vb, T *kn, T *vn, int n0) {
        constexpr bool BORDER = decltype(border)::value;  // some row may not see some key of the tile
        if (n0 + BN < any) {
            stage_k(kn, n0 + BN);
            stage_v(vn, n0 + BN);
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
        x8 pf[2 * KT];
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float e = __builtin_amdgcn_exp2f(fmaf(s[t][j], c, -ms));
                l += e;
                pf[2 * t + (j >> 3)][j & 7] = static_cast<T>(e);
            }
        if constexpr (BORDER) {
            // Some rows do not see some of these keys, and a zero weight would
            // not keep a NaN or an infinity out of them: such values leave the
            // tile and are given to the rows that see them at the end.
            bool odd = false;
            for (int i = threadIdx.x; i < BN * P; i += kPrThreads) {
                at_u32x4 w = *reinterpret_cast<const at_u32x4 *>(vb + 8 * i);
                if (clear_non_finite<T>(w)) {
                    *reinterpret_cast<at_u32x4 *>(vb + 8 * i) = w;
                    odd = true;
                }
            }
            if (odd) odd_values = 1;
            __syncthreads();
        }
        // ---- O^T += V^T P^T
#pragma unroll
        for (int u = 0; u < 2 * KT; ++u) {
#pragma unroll
            for (int i = 0; i < DT; ++i) {
                // lane: key 16 u + 4 half + (lane % 16) / 4 (then + 8), dimensions 32 i + 16 ((lane / 16) % 2) + 4 (lane % 4)
                const int r = 16 * u + 4 * half + ((lane & 15) >> 2);
                const int d = 32 * i + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
                const at_s16x4 lo =
                    __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(vb + v_place<D>(r, d >> 3) + (d & 7)));
                const at_s16x4 hi =
                    __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(vb + v_place<D>(r + 8, d >> 3) + (d & 7)));
                const auto w = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
                o[i] = Op16<T>::mfma32(__builtin_bit_cast(x8, w), pf[u], o[i]);
            }
        }
        __syncthreads();
    };

    if (threadIdx.x == 0) odd_values = 0;
    if (first < any) {
        stage_k(kt0, first);
        stage_v(vt0, first);
    }
    __syncthreads();
    int n0 = first;
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
    l = lane_pair_sum<32>(l);
    const float f = split ? 1.0f : seen == 0 ? 0.0f : 1.0f / l;
#pragma unroll
    for (int i = 0; i < DT; ++i) o[i] *= f;
    if (first < any && odd_values != 0) {
        for (int r = border; r < any; ++r) {
            const T *src = static_cast<const T *>(a.v) + (k0 + r) * a.vs + static_cast<int64_t>(kh) * D + 4 * half;
#pragma unroll
            for (int i = 0; i < DT; ++i)
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const at_f32x4 x = load4(src + 32 * i + 2 * j);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (r < seen && !(fabsf(x[e]) <= 3.4028235e38f)) o[i][j + e] += x[e];
                }
        }
    }
    if (row >= rows) return;
    if (!split) {
        T *dst = static_cast<T *>(a.out) + ((q0 + tok) * a.hq + kh * group + head) * D;
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
            for (int j = 0; j < 16; j += 4)
                store4(dst + 32 * i + 2 * j + 4 * half, at_f32x4{o[i][j], o[i][j + 1], o[i][j + 2], o[i][j + 3]});
    } else {
        const int64_t slot = ((q0 + tok) * a.hq + kh * group + head) * plan.splits + blockIdx.y;
        float *dst = part + slot * D;
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
            for (int j = 0; j < 16; j += 4)
                store4(dst + 32 * i + 2 * j + 4 * half, at_f32x4{o[i][j], o[i][j + 1], o[i][j + 2], o[i][j + 3]});
        if (half == 0) {
            part[plan.rows_floats + slot * 2] = m;
            part[plan.rows_floats + slot * 2 + 1] = l;
        }
    }
}

// Joins the chunks of the tiles that were split: D / 4 lanes per row.
template <typename T, int D>
__global__ void __launch_bounds__(256) k_prompt_join(PromptArgs a, PromptPlan plan, const float *part)
{
    constexpr int LPR = D / 4;
    const int group = a.hq / a.hkv;
    const int kh = static_cast<int>(blockIdx.x % static_cast<uint32_t>(a.hkv));
    int64_t b, at;
    if (!prompt_tile(a, blockIdx.x / static_cast<uint32_t>(a.hkv), b, at)) return;
    const int64_t q0 = a.cu_q[b], k0 = a.cu_k[b];
    const int64_t lq = a.cu_q[b + 1] - q0, lk = a.cu_k[b + 1] - k0, rows = lq * group;
    if (prompt_refused(a, q0, lq, k0, lk)) return;
    const int64_t tile = (rows + kPrRows - 1) / kPrRows - 1 - at;
    const int64_t end = (tile + 1) * kPrRows < rows ? (tile + 1) * kPrRows : rows;
    const int reach = visible(a, (end - 1) / group, lk - lq, lk);
    if (reach <= plan.chunk) return;
    const int n = static_cast<int>((reach + plan.chunk - 1) / plan.chunk);
    const int e = (threadIdx.x % LPR) * 4;
    // blockIdx.y: a quarter of the tile's rows
    const int64_t r0 = tile * kPrRows + blockIdx.y * (kPrRows / kJoinParts);
    for (int64_t r = r0 + threadIdx.x / LPR; r < r0 + kPrRows / kJoinParts && r < end; r += 256 / LPR) {
        const int64_t tok = r / group, at_out = (q0 + tok) * a.hq + kh * group + r % group;
        const float *ml = part + plan.rows_floats + at_out * plan.splits * 2, *src = part + at_out * plan.splits * D + e;
        float M = -__builtin_inff();
        for (int i = 0; i < n; ++i) M = fmaxf(M, ml[2 * i]);
        if (M == -__builtin_inff()) M = 0.0f;
        float L = 0.0f;
        at_f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int i = 0; i < n; ++i) {
            const float w = __builtin_amdgcn_exp2f(ml[2 * i] - M);
            L += w * ml[2 * i + 1];
            o += w * *reinterpret_cast<const at_f32x4 *>(src + static_cast<int64_t>(i) * D);
        }
        const float f = visible(a, tok, lk - lq, lk) == 0 ? 0.0f : 1.0f / L;
        store4(static_cast<T *>(a.out) + at_out * D + e, o * f);
    }
}

template <typename T, int D>
hipError_t prompt_launch(const PromptArgs &a, const PromptPlan &plan, float *part, hipStream_t s)
{
    const uint32_t tiles = static_cast<uint32_t>(prompt_tiles(a.batch, a.q_rows, a.hq, a.hkv) * a.hkv);
    hipLaunchKernelGGL((k_attn_prompt<T, D>), dim3(tiles, static_cast<uint32_t>(plan.splits)), dim3(kPrThreads), 0, s, a,
                       plan, part);
    if (plan.splits > 1)
        hipLaunchKernelGGL((k_prompt_join<T, D>), dim3(tiles, kJoinParts), dim3(256), 0, s, a, plan, part);
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

PromptPlan prompt_plan(int64_t batch, int64_t q_rows, int64_t max_k, int32_t hq, int32_t hkv, int32_t d)
{
    PromptPlan p;
    p.chunk = max_k > 0 ? (max_k + 127) / 128 * 128 : 128;
    const int64_t slots = d == 256 ? 256 : 512;  // workgroups the GPU holds
    const int64_t tiles = prompt_tiles(batch, q_rows, hq, hkv) * hkv;
    // Chunks that fill the GPU about once (half of max_k: a causal tile's
    // reach on average), of 512 keys at least: a chunk costs its rows in fp32,
    // written and read.  Cut three times finer: 0.34 ms for 0.28 at 1657
    // queries of 24 heads of 256 over 4000 keys and more, and with many tiles
    // cutting costs more than the last workgroups' wait: 1272 tiles of
    // up to 2500 keys of 128 in two took 115 us for 88.
    if (tiles < 4 * slots) {
        int64_t chunk = (tiles * (max_k / 2) / slots + 127) / 128 * 128;
        if (chunk < 512) chunk = 512;
        if (chunk < max_k) {
            p.chunk = chunk;
            p.splits = (max_k + chunk - 1) / chunk;
            p.rows_floats = static_cast<size_t>(q_rows) * hq * p.splits * d;
            p.part_floats = p.rows_floats + static_cast<size_t>(q_rows) * hq * p.splits * 2;
        }
    }
    return p;
}

hipError_t launch_attn_prompt(const PromptArgs &a, int dtype, int32_t d, const PromptPlan &plan, float *part, hipStream_t s)
{
    return dtype == PTQ1_BF16 ? prompt_d<__bf16>(a, d, plan, part, s) : prompt_d<_Float16>(a, d, plan, part, s);
}

}  // namespace ptq1
