// ptq1_attn_tile.h -- what the attention kernels over tiles of 64 keys share
// (attn_prompt.hip, attn_chunk.hip): the reference that a row's weights are
// relative to, their sums, and copies into LDS.
#pragma once
#include <type_traits>

#include "ptq1_attn.h"

namespace ptq1 {
namespace {

typedef short at_s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) at_s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) void lds_void;
constexpr int kBufferFlags = 0x00027000;  // raw buffer of bytes

constexpr int kKeys = 64;  // keys of a tile

// fp16 weights are 2^7 times themselves (at most 2^15 with the maximum's lag,
// below), and the sums with them: fp16's smallest step, 2^-24, is then 2^-31
// of the largest weight at most, so that many small weights beside one large
// one do not vanish.  bf16 weights, which have fp32's exponents, are 2^-40
// times themselves: the sum over 2^31 keys is then in fp32's range whenever the
// values are.
//
// A row's reference, the number that its weights are powers relative to, is its
// largest score less that.  It is what the kernels keep and join by, so its
// rounding is no error; but from 2^23 on, where that could make a weight larger
// by more than 2^0.5 (and with the lag more than fp16 holds), it is the largest
// score itself.
template <typename T>
__device__ __forceinline__ float reference(float top)
{
    return fabsf(top) < 0x1p23f ? top - (std::is_same<T, _Float16>::value ? 7.0f : -40.0f) : top;
}

// Some row's reference is so large (2^20 in units of log2) that a product
// rounded and one fused into the exponent's sum would differ by too much of a
// weight: the products are then rounded first.
__device__ __forceinline__ bool large_scores(float m)
{
    constexpr uint32_t kFrom = 0x49800000u, kInf = 0x7f800000u;
    return __ballot((__builtin_bit_cast(uint32_t, m) & 0x7fffffffu) - kFrom < kInf - kFrom) != 0;
}

// l + the sum, in fp32, of eight weights as they enter the second product,
// rounded to T: a row's weights then make up one, and what a rounding adds to
// one value it takes from the others (with the sum over unrounded weights a row
// that sees one key only was off by that key's rounding).
template <typename T>
__device__ __forceinline__ float add_weights(typename Op16<T>::x8 p, float l)
{
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        if constexpr (std::is_same<T, _Float16>::value)
            l = __builtin_amdgcn_fdot2(f16x2{p[i], p[i + 1]}, f16x2{1.0f, 1.0f}, l, false);
        else
            l = __builtin_amdgcn_fdot2_f32_bf16(bf16x2{p[i], p[i + 1]}, bf16x2{1.0f, 1.0f}, l, false);
    }
    return l;
}

// 16 bytes per lane from base + off to 1024 consecutive bytes of LDS; bytes
// from `bytes` on are not read.
__device__ __forceinline__ void copy_to_lds(const char *base, uint32_t bytes, uint32_t off, void *dst)
{
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(base), 0, static_cast<int>(bytes), kBufferFlags);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void *)dst, 16, static_cast<int>(off), 0, 0, 0);
}

// Zeros in the place of NaNs and infinities (an exponent of all ones, to which a
// one in its last place carries into the sign's) among eight values; not zero if
// there was one.  (No comparisons: their masks, of a lane's whole tile at once,
// went through memory.)
template <typename T>
__device__ __forceinline__ uint32_t clear_non_finite(at_u32x4 &w)
{
    constexpr uint32_t E = std::is_same<T, __bf16>::value ? 0x7f807f80u : 0x7c007c00u, kLast = E & ~(E << 1);
    uint32_t found = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t hit = ((w[i] & E) + kLast) & 0x80008000u;
        w[i] &= ~(hit | (hit - (hit >> 15)));
        found |= hit;
    }
    return found;
}

// Barriers with waits of their own: __syncthreads would wait for the copies
// that have just been issued.  The wait for the copies is the builtin, so that
// the compiler knows of it; with one that it could not see it waited itself,
// for the newest copies too, where the weights are read (238 us: 250).
__device__ __forceinline__ void barrier_lds() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }
__device__ __forceinline__ void barrier_copies()
{
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

}  // namespace
}  // namespace ptq1
