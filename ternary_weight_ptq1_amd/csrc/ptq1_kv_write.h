// ptq1_kv_write.h -- the kernel that writes fresh tokens into the paged cache,
// with rotary positions on their keys and queries, and ahead of them (NORM)
// norms: ptq1_kv_write (kv_cache.hip) and ptq1_kv_write_norm (kv_norm.hip), a
// translation unit each.
#pragma once
#include <type_traits>

#include "ptq1_attn.h"
#include "ptq1_launch.h"

namespace ptq1 {
namespace {

constexpr int kKvThreads = 256;
constexpr int kVTok = 64;  // tokens of one V tile (write): a wave's lanes
// q and k rows a thread has in flight.  With norms, whose sums every row waits
// for, more workgroups hide more than more rows: 8191 tokens of 24 + 4 + 4 heads of
// 256 95 us with one, 101 with two, 151 with four.
template <bool NORM>
constexpr int kRowsPer = NORM ? 1 : 2;

struct KvWriteArgs {
    const void *q, *k, *v;
    int64_t qs, ks, vs;  // row strides in elements
    int64_t tokens;
    int32_t hq, hkv;
    const int32_t *positions;
    const float *cos_sin;
    int64_t n_positions;
    int32_t rot;
    const int64_t *slots;
    void *q_out;
    void *k_pages, *v_pages;
    float *k_steps, *v_steps;
    int64_t n_slots;
    int32_t page_shift;
    uint32_t v_blocks;  // blocks of V tiles (first: they take longest); q and k rows follow
    const float *q_gain, *k_gain;  // of the norms, [D] or null: ones
    float eps;
    uint32_t per_head;    // rows / heads is rows * per_head >> head_shift, for rows below 2^25
    int32_t head_shift;
};

// Largest magnitude over the N-lane group (N = 16, 32 or 64) of |v|; NaN or
// infinity when the group holds one (an integer maximum of the bit patterns
// with the sign cleared orders magnitudes, infinity and NaN last).
template <int N>
__device__ __forceinline__ float group_absmax(float m)
{
    uint32_t u = __builtin_bit_cast(uint32_t, m) & 0x7fffffffu;
#pragma unroll
    for (int o = 1; o < N; o <<= 1) {
        const uint32_t w = static_cast<uint32_t>(__shfl_xor(static_cast<int>(u), o, kWave));
        u = u > w ? u : w;
    }
    return __builtin_bit_cast(float, u);
}

// The sum over the N-lane group, in every lane.
template <int N>
__device__ __forceinline__ float group_sum(float v)
{
    static_assert(N == 16 || N == 32 || N == 64, "rows of 64, 128 or 256 elements");
    const auto add = [&](auto ctrl) {
        const int iv = __builtin_bit_cast(int, v);
        v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(iv, iv, decltype(ctrl)::value, 0xF, 0xF, false));
    };
    add(std::integral_constant<int, 0xB1>{});   // lane ^ 1
    add(std::integral_constant<int, 0x4E>{});   // lane ^ 2
    add(std::integral_constant<int, 0x141>{});  // half-row mirror
    add(std::integral_constant<int, 0x140>{});  // row mirror
    if constexpr (N >= 32) v = lane_pair_sum<16>(v);
    if constexpr (N >= 64) v = lane_pair_sum<32>(v);
    return v;
}

__device__ __forceinline__ float squares4(at_f32x4 x)
{
    return (x[0] * x[0] + x[1] * x[1]) + (x[2] * x[2] + x[3] * x[3]);
}

__device__ __forceinline__ float absmax4(at_f32x4 x)
{
    uint32_t u = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float xi = x[i];  // (a bit cast of a vector's element itself reads element 0)
        const uint32_t w = __builtin_bit_cast(uint32_t, xi) & 0x7fffffffu;
        u = u > w ? u : w;
    }
    return __builtin_bit_cast(float, u);
}

// The int8 quantiser of one row with largest magnitude `top`: step and the
// multiplier of its values.  A non-finite row: step NaN, codes 0.
__device__ __forceinline__ void row_quantiser(float top, float &step, float &mul)
{
    if (!(top <= 3.4028235e38f)) {
        step = __builtin_nanf("");
        mul = 0.0f;
    } else if (top < 0x1p-119f) {  // 127 / top would overflow
        step = 0.0f;
        mul = 0.0f;
    } else {
        step = fminf(top / 127.0f, 0x1.020406p121f);  // (times 127 it is finite)
        mul = 127.0f / top;
    }
}

__device__ __forceinline__ int8_t row_code(float x, float mul)
{
    const float r = rintf(x * mul);
    return mul == 0.0f ? int8_t{0} : static_cast<int8_t>(static_cast<int>(fminf(fmaxf(r, -127.0f), 127.0f)));
}

// Dimensions of a V tile.  int8 needs the whole row for its step; a 16-bit
// tile of 256 dimensions would take LDS that the q and k blocks beside it
// then lack (four blocks a CU instead of all: 8191 tokens of 32 heads of 256
// took 126 us for 89).
template <typename C>
constexpr int kv_write_dims(int d)
{
    return std::is_same<C, int8_t>::value ? d : 64;
}

// q and k rows: D / 4 lanes per row of four elements, rows token-major with
// a token's q heads, then its k heads, several rows of a thread in flight.
// V: a block takes 64 tokens of one head through LDS and stores runs of eight
// tokens per dimension where eight slots follow each other from a multiple
// of eight, so that the dimension-major pages are written in 16-byte pieces
// (int8: 8), single tokens elsewhere.
//
// NORM: q and k rows are normed ahead of the rotation, y = a gain x with a =
// (mean(x^2) + eps)^(-1/2) over the row, in fp32.
template <typename S, typename Q, typename C, int D, bool NORM>
__global__ void __launch_bounds__(kKvThreads) k_kv_write(KvWriteArgs a)
{
    constexpr bool I8 = std::is_same<C, int8_t>::value;
    constexpr int LPR = D / 4;               // lanes per row
    constexpr int RPB = kKvThreads / LPR;    // rows per block and pass
    constexpr int ROWS = kRowsPer<NORM>;
    const int sub = threadIdx.x / LPR, e = (threadIdx.x % LPR) * 4;
    const int64_t page = int64_t{1} << a.page_shift;

    if (blockIdx.x >= a.v_blocks) {
        const uint32_t heads = static_cast<uint32_t>(a.hq + a.hkv);
        const int half = a.rot >> 1;
        const bool turns = e < a.rot, upper = e >= half;
        const int lo = upper ? e - half : e, other = upper ? lo : lo + half;
        at_f32x4 x[ROWS], y[ROWS], c[ROWS], sn[ROWS];
        int64_t token[ROWS];
        int h[ROWS], pos[ROWS];
        bool there[ROWS], placed[ROWS];
#pragma unroll
        for (int u = 0; u < ROWS; ++u) {
            const uint32_t row = ((blockIdx.x - a.v_blocks) * ROWS + u) * RPB + sub;
            if constexpr (NORM) {
                // (of a 256-wide row a wave's lanes have one: its address is scalar)
                const uint32_t r = LPR == kWave ? __builtin_amdgcn_readfirstlane(row) : row;
                const uint32_t t = static_cast<uint32_t>((static_cast<uint64_t>(r) * a.per_head) >> a.head_shift);
                token[u] = t;
                h[u] = static_cast<int>(r - t * heads);
            } else {
                token[u] = row / heads;
                h[u] = static_cast<int>(row % heads);
            }
            there[u] = token[u] < a.tokens;
            if (!there[u]) continue;
            const S *src = h[u] < a.hq ? static_cast<const S *>(a.q) + token[u] * a.qs + static_cast<int64_t>(h[u]) * D
                                       : static_cast<const S *>(a.k) + token[u] * a.ks + static_cast<int64_t>(h[u] - a.hq) * D;
            x[u] = load4(src + e);
            if (turns) {
                y[u] = load4(src + other);
                pos[u] = a.positions[token[u]];
            }
        }
#pragma unroll
        for (int u = 0; u < ROWS; ++u) {
            placed[u] = there[u] && turns && pos[u] >= 0 && pos[u] < a.n_positions;
            if (!placed[u]) continue;
            const float *cs = a.cos_sin + static_cast<int64_t>(pos[u]) * a.rot + lo;
            c[u] = load4(cs);
            sn[u] = load4(cs + half);
        }
        if constexpr (NORM) {
#pragma unroll
            for (int u = 0; u < ROWS; ++u) {
                if (!there[u]) continue;  // (a row's lanes alike)
                const float sum = group_sum<LPR>(squares4(x[u]));
                float f = 1.0f, a_row = __builtin_amdgcn_rsqf(sum * (1.0f / D) + a.eps);
                if (!(sum <= 3.4028235e38f) && group_absmax<LPR>(absmax4(x[u])) <= 3.4028235e38f) {
                    // finite values whose squares are not: from 2^60 on, so that
                    // 2^-70 of them has ordinary squares
                    f = 0x1p-70f;
                    a_row = __builtin_amdgcn_rsqf(group_sum<LPR>(squares4(x[u] * f)) * (1.0f / D) + a.eps * f * f);
                }
                x[u] = x[u] * f * a_row;
                if (turns) y[u] = y[u] * f * a_row;
                // (a gain is in the caches: loaded ahead with the rows, it gains 2%
                // at some sizes and loses 3 at others)
                const float *gain = h[u] < a.hq ? a.q_gain : a.k_gain;
                if (gain != nullptr) {
                    x[u] *= load4(gain + e);
                    if (turns) y[u] *= load4(gain + other);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < ROWS; ++u) {
            if (!there[u]) continue;
            if (placed[u]) {
#pragma clang fp contract(off)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float xc = x[u][i] * c[u][i], ys = y[u][i] * sn[u][i];
                    x[u][i] = upper ? xc + ys : xc - ys;
                }
            } else if (turns) {
                const float n = __builtin_nanf("");
                x[u] = at_f32x4{n, n, n, n};
            }
            if (h[u] < a.hq) {
                store4(static_cast<Q *>(a.q_out) + (token[u] * a.hq + h[u]) * D + e, x[u]);
                continue;
            }
            const int kh = h[u] - a.hq;
            const int64_t slot = a.slots[token[u]];
            if (slot < 0 || slot >= a.n_slots) continue;
            const int64_t cell = ((slot >> a.page_shift) * a.hkv + kh) * page + (slot & (page - 1));
            if constexpr (I8) {
                const float top = group_absmax<LPR>(absmax4(x[u]));
                float step, mul;
                row_quantiser(top, step, mul);
                uint32_t w = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w |= static_cast<uint32_t>(static_cast<uint8_t>(row_code(x[u][i], mul))) << (8 * i);
                *reinterpret_cast<uint32_t *>(static_cast<int8_t *>(a.k_pages) + cell * D + e) = w;
                if (e == 0) a.k_steps[cell] = step;
            } else {
                store4(static_cast<C *>(a.k_pages) + cell * D + e, x[u]);
            }
        }
        return;
    }

    // ---- V tile, [token][dimension]: rows of an odd number of dwords
    constexpr int DV = kv_write_dims<C>(D), ROW = DV + 4 / static_cast<int>(sizeof(C));
    constexpr int LPV = DV / 4, RPV = kKvThreads / LPV, PER = kVTok / RPV;
    __shared__ __attribute__((aligned(16))) C tile[kVTok * ROW];
    __shared__ float row_step[kVTok];  // int8
    const uint32_t vb = blockIdx.x, hkv = static_cast<uint32_t>(a.hkv);
    const int kh = static_cast<int>(vb % hkv), d0 = static_cast<int>(vb / hkv % (D / DV)) * DV;
    const int64_t t0 = static_cast<int64_t>(vb / hkv / (D / DV)) * kVTok;
    const int n = static_cast<int>(a.tokens - t0 < kVTok ? a.tokens - t0 : kVTok);
    const int vsub = threadIdx.x / LPV, ve = (threadIdx.x % LPV) * 4;
    at_f32x4 x[PER];
#pragma unroll
    for (int u = 0; u < PER; ++u) {
        const int r = u * RPV + vsub;
        if (r < n) x[u] = load4(static_cast<const S *>(a.v) + (t0 + r) * a.vs + static_cast<int64_t>(kh) * D + d0 + ve);
    }
    // Every wave: lane = token.  Its place (of dimension d0, in v_pages),
    // whether a run of eight starts at it, and whether it is in none.
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int64_t slot = -1;
    if (lane < n) slot = a.slots[t0 + lane];
    const bool in = slot >= 0 && slot < a.n_slots;
    if (!in) slot = -1;
    const int64_t next = __shfl_down(slot, 1, 64);
    const uint64_t follows = __ballot(in && lane < kVTok - 1 && next == slot + 1);
    const uint64_t runs = __ballot(in && (slot & 7) == 0 && lane <= kVTok - 8 && ((follows >> lane) & 0x7f) == 0x7f);
    // a run starts at this token or at one of the seven before it
    const bool alone = in && ((lane >= 7 ? runs >> (lane - 7) : runs << (7 - lane)) & 0xff) == 0;
    const int64_t off = slot & (page - 1), block = (slot >> a.page_shift) * a.hkv + kh;
    const int64_t place = (block * D + d0) * page + off;
    float steps[PER];
#pragma unroll
    for (int u = 0; u < PER; ++u) {
        const int r = u * RPV + vsub;
        if (r >= n) continue;
        if constexpr (I8) {
            const float top = group_absmax<LPV>(absmax4(x[u]));
            float mul;
            row_quantiser(top, steps[u], mul);
            uint32_t w = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w |= static_cast<uint32_t>(static_cast<uint8_t>(row_code(x[u][i], mul))) << (8 * i);
            *reinterpret_cast<uint32_t *>(tile + r * ROW + ve) = w;
        } else {
            typedef C c2 __attribute__((ext_vector_type(2)));
            *reinterpret_cast<c2 *>(tile + r * ROW + ve) = c2{static_cast<C>(x[u][0]), static_cast<C>(x[u][1])};
            *reinterpret_cast<c2 *>(tile + r * ROW + ve + 2) = c2{static_cast<C>(x[u][2]), static_cast<C>(x[u][3])};
        }
    }
    if constexpr (I8) {
        if (ve == 0) {
#pragma unroll
            for (int u = 0; u < PER; ++u)
                if (u * RPV + vsub < n) row_step[u * RPV + vsub] = steps[u];
        }
    }
    __syncthreads();
    if constexpr (I8) {
        if (wave == 0 && in) a.v_steps[block * page + off] = row_step[lane];
    }
    C *vp = static_cast<C *>(a.v_pages);
    typedef C c8 __attribute__((ext_vector_type(8)));
    if (runs != 0) {
        // lane: run lane % 8, dimension lane / 8 of eight
        const int g = lane & 7;
        uint64_t m = runs;
#pragma unroll
        for (int k = 0; k < 7; ++k)
            if (k < g) m &= m - 1;
        const int r = m != 0 ? __builtin_ctzll(m) : 0;
        const int64_t to = __shfl(place, r, 64);
        if (m != 0) {
#pragma unroll
            for (int d = 0; d < DV; d += 8 * (kKvThreads / 64)) {
                const int at = d + 8 * wave + (lane >> 3);
                c8 w;
#pragma unroll
                for (int t = 0; t < 8; ++t) w[t] = tile[(r + t) * ROW + at];
                *reinterpret_cast<c8 *>(vp + to + at * page) = w;
            }
        }
    }
    if (alone) {
#pragma unroll 8
        for (int d = wave; d < DV; d += kKvThreads / 64) vp[place + d * page] = tile[lane * ROW + d];
    }
}

inline int log2_of(int32_t v) { return __builtin_ctz(static_cast<unsigned>(v)); }

template <bool NORM, typename S, typename Q, typename C, int D>
hipError_t write_launch(KvWriteArgs &a, hipStream_t s)
{
    constexpr int RPB = kKvThreads / (D / 4) * kRowsPer<NORM>;
    const int64_t heads = a.hq + a.hkv, rows = a.tokens * heads;
    int log = 0;
    while ((int64_t{1} << log) < heads) ++log;
    a.head_shift = 25 + log;  // the product is off by less than 2^log rows of 2^25
    a.per_head = static_cast<uint32_t>(((int64_t{1} << a.head_shift) + heads - 1) / heads);
    a.v_blocks = static_cast<uint32_t>((a.tokens + kVTok - 1) / kVTok * a.hkv * (D / kv_write_dims<C>(D)));
    hipLaunchKernelGGL((k_kv_write<S, Q, C, D, NORM>), dim3(a.v_blocks + static_cast<uint32_t>((rows + RPB - 1) / RPB)),
                       dim3(kKvThreads), 0, s, a);
    return hipGetLastError();
}

template <bool NORM, typename S, typename Q, typename C>
hipError_t write_d(KvWriteArgs &a, int d, hipStream_t s)
{
    return d == 64 ? write_launch<NORM, S, Q, C, 64>(a, s)
                   : d == 128 ? write_launch<NORM, S, Q, C, 128>(a, s) : write_launch<NORM, S, Q, C, 256>(a, s);
}

template <bool NORM, typename S, typename Q>
hipError_t write_c(KvWriteArgs &a, int d, int c, hipStream_t s)
{
    return c == PTQ1_F16 ? write_d<NORM, S, Q, _Float16>(a, d, s)
                         : c == PTQ1_BF16 ? write_d<NORM, S, Q, __bf16>(a, d, s) : write_d<NORM, S, Q, int8_t>(a, d, s);
}

template <bool NORM, typename S>
hipError_t write_q(KvWriteArgs &a, int d, int c, int q, hipStream_t s)
{
    return q == PTQ1_F32 ? write_c<NORM, S, float>(a, d, c, s)
                         : q == PTQ1_F16 ? write_c<NORM, S, _Float16>(a, d, c, s) : write_c<NORM, S, __bf16>(a, d, c, s);
}

}  // namespace
}  // namespace ptq1
