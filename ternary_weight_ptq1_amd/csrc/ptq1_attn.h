// ptq1_attn.h -- device helpers shared by the cache and attention kernels
// (kv_cache.hip, attn_decode.hip, attn_prompt.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <cstdint>

#include "ptq1_device.h"

namespace ptq1 {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float at_f32x4 __attribute__((ext_vector_type(4)));
typedef float at_f32x8 __attribute__((ext_vector_type(8)));
typedef float at_f32x16 __attribute__((ext_vector_type(16)));
typedef int at_i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t at_u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t at_u32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f;

// The 16-bit operand types of the matrix instructions.
template <typename T>
struct Op16;

template <>
struct Op16<__bf16> {
    typedef bf16x4 x4;
    typedef bf16x8 x8;
    static __device__ __forceinline__ at_f32x4 mfma16(x8 a, x8 b, at_f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ at_f32x16 mfma32(x8 a, x8 b, at_f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
};

template <>
struct Op16<_Float16> {
    typedef f16x4 x4;
    typedef f16x8 x8;
    static __device__ __forceinline__ at_f32x4 mfma16(x8 a, x8 b, at_f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ at_f32x16 mfma32(x8 a, x8 b, at_f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
};

// The larger of lane l's and lane l ^ H's value, in both lanes (H = 16, 32).
template <int H>
__device__ __forceinline__ float lane_pair_max(float v)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    uint32_t lo, hi;
    if constexpr (H == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
        lo = r[0];
        hi = r[1];
    } else {
        const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
        lo = r[0];
        hi = r[1];
    }
    return fmaxf(__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi));
}

// 4 contiguous elements of a source row, as fp32.
__device__ __forceinline__ at_f32x4 load4(const float *p) { return *reinterpret_cast<const at_f32x4 *>(p); }
__device__ __forceinline__ at_f32x4 load4(const __bf16 *p)
{
    return __builtin_convertvector(*reinterpret_cast<const bf16x4 *>(p), at_f32x4);
}
__device__ __forceinline__ at_f32x4 load4(const _Float16 *p)
{
    return __builtin_convertvector(*reinterpret_cast<const f16x4 *>(p), at_f32x4);
}

// 4 fp32 values to 4 contiguous elements, rounded to nearest even.
__device__ __forceinline__ void store4(float *p, at_f32x4 v) { *reinterpret_cast<at_f32x4 *>(p) = v; }
__device__ __forceinline__ void store4(__bf16 *p, at_f32x4 v)
{
    *reinterpret_cast<bf16x4 *>(p) = __builtin_convertvector(v, bf16x4);
}
__device__ __forceinline__ void store4(_Float16 *p, at_f32x4 v)
{
    *reinterpret_cast<f16x4 *>(p) = __builtin_convertvector(v, f16x4);
}

// 8 int8 codes (two dwords) as fp16, exact: the byte code + 128 put into the
// mantissa of 1024 is 1152 + code.
__device__ __forceinline__ f16x8 codes_to_f16(uint32_t a, uint32_t b)
{
    a ^= 0x80808080u;
    b ^= 0x80808080u;
    at_u32x4 w;
    w[0] = __builtin_amdgcn_perm(0x64646464u, a, 0x04010400u);
    w[1] = __builtin_amdgcn_perm(0x64646464u, a, 0x04030402u);
    w[2] = __builtin_amdgcn_perm(0x64646464u, b, 0x04010400u);
    w[3] = __builtin_amdgcn_perm(0x64646464u, b, 0x04030402u);
    return __builtin_bit_cast(f16x8, w) - static_cast<_Float16>(1152.0f);
}

// 2^e for e in [-126, 127]
__device__ __forceinline__ float pow2(int e) { return __builtin_bit_cast(float, static_cast<uint32_t>(127 + e) << 23); }

// The place of flat tile `flat` among the tiles of `batch` sequences, of which
// sequence i has tiles_of(i): dense, so that none of the workgroups that the
// engines take in turn is empty (with one tile index for all sequences, short
// sequences left whole engines idle).  SORTED: the longest of each 64
// sequences come first, for tiles of unlike cost.  Every lane of a wave takes
// part and gets the answer; false: there are fewer tiles.
template <bool SORTED, class F>
__device__ __forceinline__ bool find_tile(int64_t flat, int64_t batch, F tiles_of, int64_t &seq, int64_t &tile)
{
    const int lane = threadIdx.x & 63;
    for (int64_t base = 0; base < batch; base += 64) {
        const int n = static_cast<int>(batch - base < 64 ? batch - base : 64);
        // at most 2^31 - 1 tiles in all (the grid's limit)
        const int mine = lane < n ? static_cast<int>(tiles_of(base + lane)) : 0;
        int before = 0, total = 0;
        if constexpr (SORTED) {
            for (int j = 0; j < n; ++j) {
                const int other = __builtin_amdgcn_readlane(mine, j);
                total += other;
                if (other > mine || (other == mine && j < lane)) before += other;
            }
        } else {
            int sum = mine;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int up = __shfl_up(sum, o, 64);
                if (lane >= o) sum += up;
            }
            before = sum - mine;
            total = __builtin_amdgcn_readlane(sum, 63);
        }
        if (flat >= total) {
            flat -= total;
            continue;
        }
        const int at = static_cast<int>(flat);
        const uint64_t hit = __ballot(at >= before && at - before < mine);
        const int who = __builtin_ctzll(hit);
        seq = base + who;
        tile = at - __builtin_amdgcn_readlane(before, who);
        return true;
    }
    return false;
}

// find_tile<false> for large batches: a lane counts the tiles of a run of
// sequences, and only the run that holds the tile is searched.
template <class F>
__device__ __forceinline__ bool find_tile_in_runs(int64_t flat, int64_t batch, F tiles_of, int64_t &seq, int64_t &tile)
{
    const int64_t run = (batch + 63) / 64, from = (threadIdx.x & 63) * run;
    const int64_t to = from + run < batch ? from + run : batch;
    int mine = 0;
#pragma unroll 4
    for (int64_t i = from; i < to; ++i) mine += static_cast<int>(tiles_of(i));
    int64_t lane, rest;
    if (!find_tile<false>(flat, 64, [&](int64_t) { return mine; }, lane, rest)) return false;
    const int64_t first = __builtin_amdgcn_readfirstlane(static_cast<int>(lane)) * run;
    const int64_t n = first + run < batch ? run : batch - first;
    if (!find_tile<false>(rest, n, [&](int64_t i) { return tiles_of(first + i); }, seq, tile)) return false;
    seq += first;
    return true;
}

// The same for sequences that are consecutive rows cu[i] .. cu[i + 1] of
// `rows` (what lies outside does not count), `group` of a tile's R each, in
// any batch with one trip to memory for a factor of 64: sequence i's tiles
// are numbered from (rows before it) / R + i on, which leaves room for all of
// them and at most one number unused; the numbers end below rows * group / R
// + batch.
template <int R>
__device__ __forceinline__ bool find_rows(int64_t flat, const int32_t *cu, int64_t batch, int64_t rows, int64_t group,
                                          int64_t &seq, int64_t &tile)
{
    const auto row = [&](int64_t i) {
        const int64_t r = cu[i];
        return r < 0 ? 0 : r < rows ? r : rows;
    };
    int64_t lo = 0, n = batch;
    for (;;) {
        const int64_t step = (n + 63) / 64, at = (threadIdx.x & 63) * step;
        const uint64_t below = __ballot(at < n && row(lo + at) * group / R + lo + at <= flat);
        if (below == 0) return false;
        const int64_t skip = (63 - __builtin_clzll(below)) * step;
        lo += skip;
        n = n - skip < step ? n - skip : step;
        if (step == 1) break;
    }
    const int64_t first = row(lo), count = row(lo + 1) - first;
    seq = lo;
    tile = flat - (first * group / R + lo);
    return tile * R < count * group;
}

}  // namespace ptq1
