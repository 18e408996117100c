// attn_chunk_few.hip -- attention of chunks over the cache where no sequence has
// more than 32 query rows of a kv head (ptq1_attn_chunk): a few proposed tokens
// that are verified, single tokens among them.  The products and their layout
// are those of attn_chunk.hip.
#include "ptq1_attn_chunk.h"

namespace ptq1 {
namespace {

constexpr int kFewWaves = 4;

// Few rows of a sequence's (32 of a kv head at most): its keys' bytes bound it, as
// they do the single tokens' attention, and as there K and V come straight from
// memory into the operands' registers, a wave's next K requested as soon as the
// first product has consumed the current one, its next V after the second: no
// LDS, no barrier, and every wave has keys of its own (32 at a time), joined at
// the end.  The matrix cores are 11% busy, so the weights enter as two 16-bit terms
// for nothing (bf16: the error against 64 bits 2.1e-3 -> 1.7e-3, the rounding of
// the result).
//
// 5 queries behind 700 tokens (40 heads over 8 of 128, bf16): 12.3 us and 4.5 for the
// join, a chain of loads; the tiles of 128 rows in LDS took 13.7 and 4.5.  32
// sequences of 4000 to 8000 tokens with 4 to 8 (32 heads over 8): 157 us, and 13.5
// for the join, of 810 MB (5.2 TB/s); the tiles took 160.  Measured and not kept:
// eight waves (17.7 against 15.8 us behind 700 tokens, both launches).
//
// 256-wide heads hold one wave a SIMD and have 11 to 21 registers spilled, some of
// them read back in every step: 32 sequences of 4000 to 8000 tokens with 3 to 5
// (24 heads over 4) take 225 us for 800 MB (3.6 TB/s), over int8 160 for 407.
// 128-wide heads over int8, 32 sequences as above: 143 us for 419 MB (2.9 TB/s).
template <typename C, typename QT, int D>
__global__ void __launch_bounds__(64 * kFewWaves, D == 256 ? 1 : 2) k_attn_chunk_few(ChunkArgs a)
{
    typedef typename WeightOf<C>::type T;
    typedef typename Op16<QT>::x8 k8;
    typedef typename Op16<T>::x8 x8;
    constexpr bool I8 = std::is_same<C, int8_t>::value;
    constexpr int W = kFewWaves, DT = D / 32, KK = D / 16;
    constexpr int NL = I8 ? D / 32 : D / 16;  // 16-byte loads of a lane, for K and for V
    __shared__ __attribute__((aligned(16))) float rows[W * kFewRows * (D + 4)];
    __shared__ float ms[W][kFewRows], ls[W][kFewRows];
    __shared__ int us[W][kFewRows];
    __shared__ int64_t place[kFewRows];
    __shared__ int bad_page;

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 31, half = lane >> 5;
    ChunkTile t;
    if (!chunk_tile<QT, D>(a, blockIdx.x, false, t)) return;
    const ChunkRow row = chunk_row(a, t, col);
    const float c = a.scale * kLog2e;
    // ---- the steps of 32 keys: as many as some row sees keys of
    int n = 2 * (t.last - t.first);
    if (n > 0 && step_key(t.c, t.last - 1) + 32 >= t.c.reach) --n;
    const auto key_of = [&](int i) { return step_key(t.c, t.first + (i >> 1)) + 32 * (i & 1); };
    ChunkPages pages(a, t);
    const int shift = a.page_shift, mask = (1 << shift) - 1;
    const uint32_t page_cells = static_cast<uint32_t>(a.hkv) << shift, page_bytes = page_cells * (D * static_cast<uint32_t>(sizeof(C)));
    const int64_t first_cell = static_cast<int64_t>(t.kh) << shift;
    const char *kp = static_cast<const char *>(a.k_pages) + first_cell * (D * static_cast<int64_t>(sizeof(C)));
    const char *vp = static_cast<const char *>(a.v_pages) + first_cell * (D * static_cast<int64_t>(sizeof(C)));
    // the token of the lane's K row, and for int8 of its run of V and of steps
    const int k_token = I8 ? ((col & 4) << 2) | ((col & 16) >> 1) | ((col & 8) >> 1) | (col & 3) : token_of_row(col);
    at_u32x4 kr[NL], vr[NL];
    at_f32x4 ksr[I8 ? 4 : 1], vsr[I8 ? 4 : 1];
    const auto load_k = [&](int n0) {
        const int32_t pg = k_token & 16 ? pages.run[1] : pages.run[0];
        const char *src = kp + static_cast<uint64_t>(page_bytes) * static_cast<uint32_t>(pg) + ((n0 + k_token) & mask) * (D * static_cast<int>(sizeof(C))) + 16 * half;
#pragma unroll
        for (int i = 0; i < NL; ++i) kr[i] = *reinterpret_cast<const at_u32x4 *>(src + 32 * i);
    };
    const auto load_steps = [&](const float *steps, int n0, at_f32x4 (&to)[I8 ? 4 : 1]) {
        const float *src = steps + first_cell + static_cast<uint64_t>(page_cells) * static_cast<uint32_t>(half ? pages.run[1] : pages.run[0]) + ((n0 + 16 * half) & mask);
#pragma unroll
        for (int i = 0; i < (I8 ? 4 : 1); ++i) to[i] = *reinterpret_cast<const at_f32x4 *>(src + 4 * i);
    };
    const auto load_v = [&](int n0) {
        if constexpr (I8) {  // dimension 32 i + col, the 16 tokens of the half's run
            const char *src = vp + static_cast<uint64_t>(page_bytes) * static_cast<uint32_t>(half ? pages.run[1] : pages.run[0]) +
                              ((static_cast<uint32_t>(col) << shift) + ((n0 + 16 * half) & mask));
#pragma unroll
            for (int i = 0; i < NL; ++i) vr[i] = *reinterpret_cast<const at_u32x4 *>(src + (static_cast<uint32_t>(32 * i) << shift));
        } else {  // tokens 16 u + 8 half .., dimension 32 i + col at 2 i + u
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const char *src = vp + static_cast<uint64_t>(page_bytes) * static_cast<uint32_t>(pages.run[u]) +
                                  2 * ((static_cast<uint32_t>(col) << shift) + ((n0 + 16 * u + 8 * half) & mask));
#pragma unroll
                for (int i = 0; i < NL / 2; ++i) vr[2 * i + u] = *reinterpret_cast<const at_u32x4 *>(src + (static_cast<uint32_t>(64 * i) << shift));
            }
        }
    };

    if (threadIdx.x == 0) bad_page = 0;
    __syncthreads();
    int i = wave;
    if (i < n) {
        pages.find(key_of(i));
        pages.use();
        load_k(key_of(i));
        if constexpr (I8) load_steps(a.k_steps, key_of(i), ksr);
        load_v(key_of(i));
        if constexpr (I8) load_steps(a.v_steps, key_of(i), vsr);
        pages.find(key_of(min(i + W, n - 1)));
    }
    const ChunkQuery<QT, D, I8, I8> q(a, t, row, half);
    const bool lifted = I8 && __ballot(q.lift != 0) != 0;
    at_f32x16 o[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[d][j] = 0.0f;
    ChunkSoftmax<C, 1, 2, I8> w;
    ChunkNotes notes{0, 0};
    int steps_unit = -126;

    for (; i < n; i += W) {
        const int n0 = key_of(i), at = t.first + (i >> 1);
        const bool border = at < t.c.all_from || at >= t.c.all_to;  // some row may not see some key
        const bool more = i + W < n;
        at_f32x16 s[1];
#pragma unroll
        for (int j = 0; j < 16; ++j) s[0][j] = 0.0f;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            k8 kf;
            if constexpr (I8) {
                at_u32x2 codes = {kr[kk >> 1][2 * (kk & 1)], kr[kk >> 1][2 * (kk & 1) + 1]};
                asm volatile("" : "+v"(codes));  // keeps them packed up to here
                kf = codes_to<QT>(codes[0], codes[1]);
                if ((kk & 1) == 1) __builtin_amdgcn_sched_barrier(0);  // or all are converted up front
            } else
                kf = __builtin_bit_cast(k8, kr[kk]);
            s[0] = Op16<QT>::mfma32(kf, q.f[kk], s[0]);
        }
        if constexpr (I8) {
            if (lifted) w.by_power(s, q.lift >> 1);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float k = ksr[j >> 2][j & 3];
                s[0][j] *= k != k ? k : fminf(k * c, 3.4028235e38f);
            }
            if (lifted) w.by_power(s, (q.lift + 1) >> 1);
        }
        if (more) {
            pages.use();
            load_k(key_of(i + W));
            if constexpr (I8) load_steps(a.k_steps, key_of(i + W), ksr);
        }
        const HiddenKeys hidden(row.seen, t, n0);
        w.raise(w.top(border, s, hidden, n0, half, c, [](int, int) { return 1.0f; }, false, [] { return 0; }), o, w.unit);
        x8 pf[2][2];  // [term][16 keys]
        if constexpr (I8) {
            float most = 0.0f;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int key = n0 + 16 * half + j;
                const bool some = !border | ((key < t.c.reach) & ((key >= t.c.lo) | (key < t.c.sunk)));
                most = fmaxf(most, some ? vsr[j >> 2][j & 3] : 0.0f);
            }
            most = lane_pair_max<32>(most);
            steps_unit = unit_of_steps(steps_unit, __builtin_amdgcn_readfirstlane(static_cast<int>(__builtin_bit_cast(uint32_t, most) >> 23) - 126));
            w.products(border, s, hidden, n0, half, [&](int, int j) { return ldexpf(vsr[j >> 2][j & 3], -steps_unit); }, steps_unit, pf,
                                        [&](float f) {
#pragma unroll
                                            for (int d = 0; d < DT; ++d) o[d] *= f;
                                        });
        } else
            w.weights(s, c, pf);
        if (!I8 && border) {
            // (as in the tiles: what a row does not see must not meet its zero weight)
            uint32_t odd = 0;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const at_u32x4 seen = seen_halves(n0 + 16 * u + 8 * half, t.c.lo, t.c.reach, t.c.sunk);
#pragma unroll
                for (int k = u; k < NL; k += 2) {
                    vr[k] &= seen;
                    odd |= clear_non_finite<T>(vr[k]);
                    asm volatile("" : "+v"(odd), "+v"(vr[k]));  // (one after the other: all at once need registers)
                }
            }
            if (__ballot(odd != 0) != 0) notes.odd_steps |= step_bit(n0);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                x8 vf;
                if constexpr (I8) {
                    at_u32x2 codes = {vr[d][2 * u], vr[d][2 * u + 1]};
                    asm volatile("" : "+v"(codes));
                    vf = codes_to_f16(codes[0], codes[1]);
                    if ((d & 1) == 1) __builtin_amdgcn_sched_barrier(0);
                } else
                    vf = __builtin_bit_cast(x8, vr[2 * d + u]);
#pragma unroll
                for (int k = 0; k < 2; ++k) o[d] = Op16<T>::mfma32(vf, pf[k][u], o[d]);
            }
        if (more) {
            load_v(key_of(i + W));
            if constexpr (I8) load_steps(a.v_steps, key_of(i + W), vsr);
        }
        pages.find(key_of(min(i + 2 * W, n - 1)));
    }
    const float l = lane_pair_sum<32>(w.l + w.l2);
    if constexpr (!I8)
        if (notes.odd_steps != 0) add_odd_values<T, DT>(a, t, row, notes, D, 0, half, o);

    // ---- join the waves' rows: each row's weights of the waves first
    if (half == 0) {
        ms[wave][col] = w.m;
        ls[wave][col] = l;
        us[wave][col] = I8 ? w.unit : 0;
    }
    if (col < t.rows) {
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int j = 0; j < 16; j += 4)
                *reinterpret_cast<at_f32x4 *>(rows + (wave * kFewRows + col) * (D + 4) + 32 * d + 2 * j + 4 * half) = at_f32x4{o[d][j], o[d][j + 1], o[d][j + 2], o[d][j + 3]};
    }
    if (__ballot(pages.bad) != 0 && lane == 0) bad_page = 1;
    __syncthreads();
    if (wave == 0 && half == 0 && row.is) {
        float M = ms[0][col];
        int unit = us[0][col];
#pragma unroll
        for (int k = 1; k < W; ++k) {
            M = fmaxf(M, ms[k][col]);
            unit = max(unit, us[k][col]);
        }
        const float Ms = M == -__builtin_inff() ? 0.0f : M;
        float L = 0.0f, f[W];
#pragma unroll
        for (int k = 0; k < W; ++k) {
            f[k] = __builtin_amdgcn_exp2f(ms[k][col] - Ms);
            L += f[k] * ls[k][col];
        }
        const bool none = row.seen.hi == 0 || (t.pieces > 1 && L == 0.0f);
        float inv = none ? 0.0f : 1.0f / L;
        if (bad_page != 0 && sees_bad_page(a, t, row)) L = inv = __builtin_nanf("");
#pragma unroll
        for (int k = 0; k < W; ++k) ls[k][col] = (I8 ? ldexpf(f[k], us[k][col] - unit) : f[k]) * inv;
        us[0][col] = unit;
        if (t.pieces == 1)
            place[col] = (static_cast<int64_t>(t.q0) + row.tok) * a.hq + row.head;
        else {
            const int64_t slot = part_slot(a, t, col);
            place[col] = slot;
            a.parts[a.rows_floats + slot * 2] = M;
            a.parts[a.rows_floats + slot * 2 + 1] = L;
        }
    }
    __syncthreads();
    for (int x = threadIdx.x; x < t.rows * (D / 4); x += 64 * W) {
        const int r = x / (D / 4), e = (x % (D / 4)) * 4;
        at_f32x4 sum = ls[0][r] * *reinterpret_cast<const at_f32x4 *>(rows + r * (D + 4) + e);
#pragma unroll
        for (int k = 1; k < W; ++k) sum += ls[k][r] * *reinterpret_cast<const at_f32x4 *>(rows + (k * kFewRows + r) * (D + 4) + e);
        if constexpr (I8) {
            const int unit = us[0][r];
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[j] = ldexpf(sum[j], unit);
        }
        if (t.pieces == 1)
            store4(static_cast<QT *>(a.out) + place[r] * D + e, sum);
        else
            store4(a.parts + place[r] * D + e, sum);
    }
}

template <typename C, typename QT>
void few_launch(const ChunkArgs &a, int d, uint32_t groups, hipStream_t s)
{
    if (d == 64)
        hipLaunchKernelGGL((k_attn_chunk_few<C, QT, 64>), dim3(groups), dim3(64 * kFewWaves), 0, s, a);
    else if (d == 128)
        hipLaunchKernelGGL((k_attn_chunk_few<C, QT, 128>), dim3(groups), dim3(64 * kFewWaves), 0, s, a);
    else
        hipLaunchKernelGGL((k_attn_chunk_few<C, QT, 256>), dim3(groups), dim3(64 * kFewWaves), 0, s, a);
}

}  // namespace

hipError_t launch_chunk_few(const ChunkArgs &a, int cache_type, int q_type, int d, uint32_t groups, hipStream_t s)
{
    if (cache_type == PTQ1_BF16)
        few_launch<__bf16, __bf16>(a, d, groups, s);
    else if (cache_type == PTQ1_F16)
        few_launch<_Float16, _Float16>(a, d, groups, s);
    else if (q_type == PTQ1_F16)
        few_launch<int8_t, _Float16>(a, d, groups, s);
    else
        few_launch<int8_t, __bf16>(a, d, groups, s);
    return hipGetLastError();
}

}  // namespace ptq1
