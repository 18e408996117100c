// kv_cache.hip -- the paged key-value cache: write with rotary positions
// (ptq1_kv_write) and packed read-back (ptq1_kv_read).  Layout and
// semantics: include/ptq1.h.
//
// Both are one pass over their data, bounded by HBM for many tokens and by
// one launch's latency for a few.  Measured: 8191 tokens of 24 + 4 + 4 heads
// of 256, fp32 to bf16, written in 87 us (4.65 TB/s; a copy 5.4), one token
// of 40 + 8 + 8 heads of 128 in 3.0; 96 thousand tokens of 8 heads of 128
// read back from int8 to bf16 in 88 (4.5 TB/s, two thirds of it written).
#include <hip/hip_runtime.h>

#include "ptq1_attn.h"
#include "ptq1_kv_write.h"
#include "ptq1_launch.h"

namespace ptq1 {
namespace {

struct KvReadArgs {
    const void *k_pages, *v_pages;
    const float *k_steps, *v_steps;
    int64_t n_pages;
    int32_t page_shift, hkv;
    const int32_t *table;
    int64_t max_pages;
    const int32_t *cu;
    int64_t batch, rows;
    void *k_out, *v_out;
};

constexpr int kReadTok = 64;  // tokens of one tile

// 8 fp32 values to 8 contiguous elements, rounded to nearest even.
template <typename O>
__device__ __forceinline__ void store8(O *p, const float (&v)[8])
{
    store4(p, at_f32x4{v[0], v[1], v[2], v[3]});
    store4(p + 4, at_f32x4{v[4], v[5], v[6], v[7]});
}

// One block: 64 tokens (from a multiple of 64 in the sequence, so runs of
// tokens stay aligned in their pages) of one head of one sequence.  V's runs
// are requested first, K rows are copied meanwhile, then V goes through LDS
// from dimension-major to rows, 128 dimensions at a time.
template <typename C, typename O, int D>
__global__ void __launch_bounds__(kKvThreads) k_kv_read(KvReadArgs a)
{
    constexpr bool I8 = std::is_same<C, int8_t>::value;
    constexpr int EPL = 16 / sizeof(C);      // cache elements per 16-byte load
    constexpr int DB = D < 128 ? D : 128;    // dimensions of one pass
    constexpr int RUNS = kReadTok / EPL;
    constexpr int PER = DB * RUNS / kKvThreads;  // V loads of a thread and pass
    // rows of an odd number of dwords: the threads of a wave write eight
    // dimensions of eight runs, and read four rows
    constexpr int ROW = DB + (sizeof(O) == 4 ? 1 : 2);
    typedef C cvec __attribute__((ext_vector_type(EPL)));
    typedef C c8 __attribute__((ext_vector_type(8)));
    const int kh = static_cast<int>(blockIdx.x % static_cast<uint32_t>(a.hkv));
    int64_t b, at;
    if (!find_rows<kReadTok>(blockIdx.x / static_cast<uint32_t>(a.hkv), a.cu, a.batch, a.rows, 1, b, at) || a.cu[b] < 0)
        return;
    const int64_t first = a.cu[b], end = a.cu[b + 1] < a.rows ? a.cu[b + 1] : a.rows;
    const int64_t t0 = at * kReadTok, out0 = first + t0;
    const int n = static_cast<int>(end - out0 < kReadTok ? end - out0 : kReadTok);
    const int64_t page = int64_t{1} << a.page_shift;
    __shared__ int64_t cells[kReadTok];  // (page * heads + head) * page_size + place, -1: no such page
    __shared__ float steps[kReadTok];    // V's
    __shared__ __attribute__((aligned(16))) O tile[kReadTok * ROW];
    if (threadIdx.x < kReadTok) {
        const int64_t t = t0 + threadIdx.x, pi = t >> a.page_shift;
        int64_t c = -1;
        if (static_cast<int>(threadIdx.x) < n && pi < a.max_pages) {
            const int64_t pg = a.table[b * a.max_pages + pi];
            if (pg >= 0 && pg < a.n_pages) c = (pg * a.hkv + kh) * page + (t & (page - 1));
        }
        cells[threadIdx.x] = c;
        if (I8) steps[threadIdx.x] = c >= 0 ? a.v_steps[c] : 0.0f;
    }
    __syncthreads();
    const float nan = __builtin_nanf("");
#pragma unroll
    for (int d0 = 0; d0 < D; d0 += DB) {
        cvec v[PER];
        bool is[PER];
#pragma unroll
        for (int u = 0; u < PER; ++u) {
            const int i = u * kKvThreads + threadIdx.x, d = i / RUNS, r = (i % RUNS) * EPL;
            const int64_t c = cells[r];  // a page holds a multiple of 16 tokens and t0 is one of 64: a run is in one page
            is[u] = c >= 0;
            if (!is[u]) continue;
            const int64_t pgh = c >> a.page_shift, off = c & (page - 1);
            v[u] = *reinterpret_cast<const cvec *>(static_cast<const C *>(a.v_pages) + (pgh * D + d0 + d) * page + off);
        }
        if (d0 == 0) {
            // K: D / 8 lanes per row
            constexpr int LPR = D / 8, RPB = kKvThreads / LPR, KPER = kReadTok / RPB;
            const int e = (threadIdx.x % LPR) * 8;
            c8 k[KPER];
            float ks[KPER];
#pragma unroll
            for (int u = 0; u < KPER; ++u) {
                const int r = u * RPB + threadIdx.x / LPR;
                const int64_t c = cells[r];
                if (c < 0) continue;
                k[u] = *reinterpret_cast<const c8 *>(static_cast<const C *>(a.k_pages) + c * D + e);
                if constexpr (I8) ks[u] = a.k_steps[c];
            }
#pragma unroll
            for (int u = 0; u < KPER; ++u) {
                const int r = u * RPB + threadIdx.x / LPR;
                if (r >= n) continue;
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[i] = nan;
                    if (cells[r] >= 0) {
                        x[i] = static_cast<float>(k[u][i]);
                        if constexpr (I8) x[i] *= ks[u];
                    }
                }
                store8(static_cast<O *>(a.k_out) + ((out0 + r) * a.hkv + kh) * D + e, x);
            }
        }
        if (d0 > 0) __syncthreads();
#pragma unroll
        for (int u = 0; u < PER; ++u) {
            const int i = u * kKvThreads + threadIdx.x, d = i / RUNS, r = (i % RUNS) * EPL;
#pragma unroll
            for (int t = 0; t < EPL; ++t) {
                float x = nan;
                if (is[u]) {
                    x = static_cast<float>(v[u][t]);
                    if constexpr (I8) x *= steps[r + t];
                }
                tile[(r + t) * ROW + d] = static_cast<O>(x);
            }
        }
        __syncthreads();
        constexpr int VEC = 16 / static_cast<int>(sizeof(O));  // elements of a 16-byte store
        constexpr int LPV = DB / VEC;
        for (int i = threadIdx.x; i < kReadTok * LPV; i += kKvThreads) {
            const int r = i / LPV, e = (i % LPV) * VEC;
            if (r >= n) continue;
            const uint32_t *src = reinterpret_cast<const uint32_t *>(tile + r * ROW + e);
            const at_u32x4 w = {src[0], src[1], src[2], src[3]};
            *reinterpret_cast<at_u32x4 *>(static_cast<O *>(a.v_out) + ((out0 + r) * a.hkv + kh) * D + d0 + e) = w;
        }
    }
}

template <typename C, typename O, int D>
hipError_t read_launch(const KvReadArgs &a, hipStream_t s)
{
    // whole tiles of all rows, and a part of one for every sequence
    const int64_t tiles = a.rows / kReadTok + a.batch;
    hipLaunchKernelGGL((k_kv_read<C, O, D>), dim3(static_cast<uint32_t>(tiles * a.hkv)), dim3(kKvThreads), 0, s, a);
    return hipGetLastError();
}

template <typename C, typename O>
hipError_t read_d(const KvReadArgs &a, int d, hipStream_t s)
{
    return d == 64 ? read_launch<C, O, 64>(a, s)
                   : d == 128 ? read_launch<C, O, 128>(a, s) : read_launch<C, O, 256>(a, s);
}

template <typename C>
hipError_t read_o(const KvReadArgs &a, int d, int o, hipStream_t s)
{
    return o == PTQ1_F32 ? read_d<C, float>(a, d, s)
                         : o == PTQ1_F16 ? read_d<C, _Float16>(a, d, s) : read_d<C, __bf16>(a, d, s);
}

}  // namespace

hipError_t launch_kv_write(const void *q, int64_t qs, const void *k, int64_t ks, const void *v, int64_t vs, int src,
                           int64_t tokens, int32_t hq, const int32_t *positions, const float *cos_sin,
                           int64_t n_positions, int32_t rot, const int64_t *slots, void *q_out, int q_type,
                           const ptq1_kv_cache &c, hipStream_t s)
{
    KvWriteArgs a{q,     k,     v,         qs,          ks,        vs,        tokens, hq,
                  c.n_kv_heads, positions, cos_sin, n_positions, rot, slots, q_out, c.k_pages, c.v_pages,
                  c.k_steps, c.v_steps, c.n_pages * c.page_size, log2_of(c.page_size), 0, nullptr, nullptr, 0.0f, 0, 0};
    return src == PTQ1_F32 ? write_q<false, float>(a, c.head_dim, c.dtype, q_type, s)
                           : src == PTQ1_F16 ? write_q<false, _Float16>(a, c.head_dim, c.dtype, q_type, s)
                                             : write_q<false, __bf16>(a, c.head_dim, c.dtype, q_type, s);
}

hipError_t launch_kv_read(const ptq1_kv_cache &c, const int32_t *table, int64_t max_pages, const int32_t *cu,
                          int64_t batch, int64_t rows, void *k_out, void *v_out, int out_type, hipStream_t s)
{
    const KvReadArgs a{c.k_pages, c.v_pages, c.k_steps, c.v_steps, c.n_pages, log2_of(c.page_size),
                       c.n_kv_heads, table, max_pages, cu, batch, rows, k_out, v_out};
    return c.dtype == PTQ1_F16 ? read_o<_Float16>(a, c.head_dim, out_type, s)
                               : c.dtype == PTQ1_BF16 ? read_o<__bf16>(a, c.head_dim, out_type, s)
                                                      : read_o<int8_t>(a, c.head_dim, out_type, s);
}

}  // namespace ptq1
