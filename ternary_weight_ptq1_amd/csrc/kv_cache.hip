// kv_cache.hip -- the paged key-value cache: write with rotary positions
// (ptq1_kv_write) and packed read-back (ptq1_kv_read).  Layout and
// semantics: include/ptq1.h.
//
// Both are one pass over their data, bounded by HBM for many tokens and by
// one launch's latency for a few.
#include <hip/hip_runtime.h>

#include "ptq1_attn.h"
#include "ptq1_launch.h"

namespace ptq1 {
namespace {

constexpr int kKvThreads = 256;
constexpr int kVTok = 32;  // tokens of one V tile (write)

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
    int64_t qk_blocks;  // blocks of q and k rows; V tiles follow
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
        step = top / 127.0f;
        mul = 127.0f / top;
    }
}

__device__ __forceinline__ int8_t row_code(float x, float mul)
{
    const float r = rintf(x * mul);
    return mul == 0.0f ? int8_t{0} : static_cast<int8_t>(static_cast<int>(fminf(fmaxf(r, -127.0f), 127.0f)));
}

// Elements e .. e + 3 of a row at position pos, turned.
template <typename S>
__device__ __forceinline__ at_f32x4 load_turned(const S *row, int e, const KvWriteArgs &a, int64_t token)
{
    at_f32x4 x = load4(row + e);
    if (e < a.rot) {
        const int half = a.rot >> 1;
        const int64_t pos = a.positions[token];
        if (pos < 0 || pos >= a.n_positions) {
            const float n = __builtin_nanf("");
            return at_f32x4{n, n, n, n};
        }
        const float *cs = a.cos_sin + pos * a.rot;
        const bool upper = e >= half;
        const int lo = upper ? e - half : e;
        const at_f32x4 c = load4(cs + lo), s = load4(cs + half + lo);
        const at_f32x4 y = load4(row + (upper ? lo : lo + half));
        {
#pragma clang fp contract(off)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float xc = x[i] * c[i], ys = y[i] * s[i];
                x[i] = upper ? xc + ys : xc - ys;
            }
        }
    }
    return x;
}

// q and k rows: D / 4 lanes per row of four elements, rows token-major with
// a token's q heads, then its k heads.  V: a block takes 32 tokens of one
// head through LDS and stores runs of tokens per dimension, so that the
// dimension-major pages are written in 64-byte pieces where slots follow
// each other.
template <typename S, typename Q, typename C, int D>
__global__ void __launch_bounds__(kKvThreads) k_kv_write(KvWriteArgs a)
{
    constexpr bool I8 = std::is_same<C, int8_t>::value;
    constexpr int LPR = D / 4;               // lanes per row
    constexpr int RPB = kKvThreads / LPR;    // rows per block
    const int sub = threadIdx.x / LPR, e = (threadIdx.x % LPR) * 4;
    const int64_t page = int64_t{1} << a.page_shift;

    if (static_cast<int64_t>(blockIdx.x) < a.qk_blocks) {
        const int64_t row = static_cast<int64_t>(blockIdx.x) * RPB + sub;
        const uint32_t heads = static_cast<uint32_t>(a.hq + a.hkv);
        const int64_t token = static_cast<uint32_t>(row) / heads;
        if (token >= a.tokens) return;
        const int h = static_cast<int>(static_cast<uint32_t>(row) % heads);
        if (h < a.hq) {
            const S *src = static_cast<const S *>(a.q) + token * a.qs + static_cast<int64_t>(h) * D;
            store4(static_cast<Q *>(a.q_out) + (token * a.hq + h) * D + e, load_turned(src, e, a, token));
            return;
        }
        const int kh = h - a.hq;
        const int64_t slot = a.slots[token];
        if (slot < 0 || slot >= a.n_slots) return;
        const S *src = static_cast<const S *>(a.k) + token * a.ks + static_cast<int64_t>(kh) * D;
        const at_f32x4 x = load_turned(src, e, a, token);
        const int64_t cell = ((slot >> a.page_shift) * a.hkv + kh) * page + (slot & (page - 1));
        if constexpr (I8) {
            const float top = group_absmax<LPR>(absmax4(x));
            float step, mul;
            row_quantiser(top, step, mul);
            uint32_t w = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) w |= static_cast<uint32_t>(static_cast<uint8_t>(row_code(x[i], mul))) << (8 * i);
            *reinterpret_cast<uint32_t *>(static_cast<int8_t *>(a.k_pages) + cell * D + e) = w;
            if (e == 0) a.k_steps[cell] = step;
        } else {
            store4(static_cast<C *>(a.k_pages) + cell * D + e, x);
        }
        return;
    }

    // ---- V tile ----
    __shared__ C tile[D][kVTok + 4 / sizeof(C)];
    __shared__ int64_t cell0[kVTok];  // place of the token's dimension 0 in v_pages, -1: not written
    const int64_t vb = static_cast<int64_t>(blockIdx.x) - a.qk_blocks;
    const int kh = static_cast<int>(static_cast<uint32_t>(vb) % static_cast<uint32_t>(a.hkv));
    const int64_t t0 = static_cast<int64_t>(static_cast<uint32_t>(vb) / static_cast<uint32_t>(a.hkv)) * kVTok;
    const int n = static_cast<int>(a.tokens - t0 < kVTok ? a.tokens - t0 : kVTok);
    for (int r = sub; r < n; r += RPB) {
        const int64_t token = t0 + r;
        const int64_t slot = a.slots[token];
        const bool in = slot >= 0 && slot < a.n_slots;
        const at_f32x4 x = load4(static_cast<const S *>(a.v) + token * a.vs + static_cast<int64_t>(kh) * D + e);
        const int64_t pg = (slot >> a.page_shift) * a.hkv + kh, off = slot & (page - 1);
        if constexpr (I8) {
            const float top = group_absmax<LPR>(absmax4(x));
            float step, mul;
            row_quantiser(top, step, mul);
#pragma unroll
            for (int i = 0; i < 4; ++i) tile[e + i][r] = row_code(x[i], mul);
            if (e == 0 && in) a.v_steps[pg * page + off] = step;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) tile[e + i][r] = static_cast<C>(x[i]);
        }
        if (e == 0) cell0[r] = in ? pg * D * page + off : -1;
    }
    __syncthreads();
    C *vp = static_cast<C *>(a.v_pages);
    for (int i = threadIdx.x; i < D * kVTok; i += kKvThreads) {
        const int r = i % kVTok, d = i / kVTok;
        if (r < n && cell0[r] >= 0) vp[cell0[r] + static_cast<int64_t>(d) * page] = tile[d][r];
    }
}

struct KvReadArgs {
    const void *k_pages, *v_pages;
    const float *k_steps, *v_steps;
    int64_t n_pages;
    int32_t page_shift, hkv;
    const int32_t *table;
    int64_t max_pages;
    const int32_t *cu;
    int64_t rows;
    void *k_out, *v_out;
};

constexpr int kReadTok = 64;  // tokens of one tile

// One block: 64 tokens (from a multiple of 64 in the sequence, so runs of
// tokens stay aligned in their pages) of one head of one sequence.  K rows
// are copied; V goes through LDS from dimension-major to rows.
template <typename C, typename O, int D>
__global__ void __launch_bounds__(kKvThreads) k_kv_read(KvReadArgs a)
{
    constexpr bool I8 = std::is_same<C, int8_t>::value;
    constexpr int EPL = 16 / sizeof(C);  // cache elements per 16-byte load
    typedef C cvec __attribute__((ext_vector_type(EPL)));
    const int64_t b = blockIdx.y / a.hkv;
    const int kh = static_cast<int>(blockIdx.y % a.hkv);
    const int64_t first = a.cu[b], len = a.cu[b + 1] - first;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kReadTok;
    if (t0 >= len) return;
    const int n = static_cast<int>(len - t0 < kReadTok ? len - t0 : kReadTok);
    const int64_t page = int64_t{1} << a.page_shift;
    __shared__ int64_t cells[kReadTok];  // (page * heads + head) * page_size + place, -1: no such page
    __shared__ float tile[64][kReadTok + 1];
    if (threadIdx.x < kReadTok) {
        const int64_t t = t0 + threadIdx.x, at = t >> a.page_shift;
        int64_t c = -1;
        if (static_cast<int>(threadIdx.x) < n && at < a.max_pages) {
            const int64_t pg = a.table[b * a.max_pages + at];
            if (pg >= 0 && pg < a.n_pages) c = (pg * a.hkv + kh) * page + (t & (page - 1));
        }
        cells[threadIdx.x] = c;
    }
    __syncthreads();
    const float nan = __builtin_nanf("");
    // K: D / 4 lanes per row
    {
        constexpr int LPR = D / 4, RPB = kKvThreads / LPR;
        const int e = (threadIdx.x % LPR) * 4;
        for (int r = threadIdx.x / LPR; r < n; r += RPB) {
            const int64_t out = first + t0 + r;
            if (out < 0 || out >= a.rows) continue;
            const int64_t c = cells[r];
            at_f32x4 x = {nan, nan, nan, nan};
            if (c >= 0) {
                if constexpr (I8) {
                    const uint32_t w = *reinterpret_cast<const uint32_t *>(static_cast<const int8_t *>(a.k_pages) + c * D + e);
                    const float s = a.k_steps[c];
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = s * static_cast<float>(static_cast<int8_t>(w >> (8 * i)));
                } else {
                    x = load4(static_cast<const C *>(a.k_pages) + c * D + e);
                }
            }
            store4(static_cast<O *>(a.k_out) + (out * a.hkv + kh) * D + e, x);
        }
    }
    // V: 64 dimensions at a time; runs of EPL tokens are one load (a page
    // holds a multiple of 16 tokens and t0 is one of 64)
    for (int d0 = 0; d0 < D; d0 += 64) {
        constexpr int RUNS = kReadTok / EPL;
        for (int i = threadIdx.x; i < 64 * RUNS; i += kKvThreads) {
            const int d = i / RUNS, r = (i % RUNS) * EPL;
            const int64_t c = r < n ? cells[r] : -1;
            if (c >= 0) {
                // cells counts rows of D in K; in V the run starts at dimension d of the page's block
                const int64_t pgh = c >> a.page_shift, off = c & (page - 1);
                const cvec w = *reinterpret_cast<const cvec *>(static_cast<const C *>(a.v_pages) +
                                                               (pgh * D + d0 + d) * page + off);
#pragma unroll
                for (int j = 0; j < EPL; ++j) {
                    float x = static_cast<float>(w[j]);
                    if constexpr (I8) x = (r + j < n ? a.v_steps[c + j] : 0.0f) * x;
                    tile[d][r + j] = x;
                }
            } else {
#pragma unroll
                for (int j = 0; j < EPL; ++j) tile[d][r + j] = nan;
            }
        }
        __syncthreads();
        const int e = (threadIdx.x % 16) * 4;
        for (int r = threadIdx.x / 16; r < n; r += kKvThreads / 16) {
            const int64_t out = first + t0 + r;
            if (out < 0 || out >= a.rows) continue;
            const at_f32x4 x = {tile[e][r], tile[e + 1][r], tile[e + 2][r], tile[e + 3][r]};
            store4(static_cast<O *>(a.v_out) + (out * a.hkv + kh) * D + d0 + e, x);
        }
        __syncthreads();
    }
}

int log2_of(int32_t v) { return __builtin_ctz(static_cast<unsigned>(v)); }

template <typename S, typename Q, typename C, int D>
hipError_t write_launch(KvWriteArgs &a, hipStream_t s)
{
    constexpr int RPB = kKvThreads / (D / 4);
    const int64_t rows = a.tokens * (a.hq + a.hkv);
    a.qk_blocks = (rows + RPB - 1) / RPB;
    const int64_t vt = (a.tokens + kVTok - 1) / kVTok * a.hkv;
    hipLaunchKernelGGL((k_kv_write<S, Q, C, D>), dim3(static_cast<uint32_t>(a.qk_blocks + vt)), dim3(kKvThreads), 0, s,
                       a);
    return hipGetLastError();
}

template <typename S, typename Q, typename C>
hipError_t write_d(KvWriteArgs &a, int d, hipStream_t s)
{
    return d == 64 ? write_launch<S, Q, C, 64>(a, s)
                   : d == 128 ? write_launch<S, Q, C, 128>(a, s) : write_launch<S, Q, C, 256>(a, s);
}

template <typename S, typename Q>
hipError_t write_c(KvWriteArgs &a, int d, int c, hipStream_t s)
{
    return c == PTQ1_F16 ? write_d<S, Q, _Float16>(a, d, s)
                         : c == PTQ1_BF16 ? write_d<S, Q, __bf16>(a, d, s) : write_d<S, Q, int8_t>(a, d, s);
}

template <typename S>
hipError_t write_q(KvWriteArgs &a, int d, int c, int q, hipStream_t s)
{
    return q == PTQ1_F32 ? write_c<S, float>(a, d, c, s)
                         : q == PTQ1_F16 ? write_c<S, _Float16>(a, d, c, s) : write_c<S, __bf16>(a, d, c, s);
}

template <typename C, typename O, int D>
hipError_t read_launch(const KvReadArgs &a, int64_t batch, hipStream_t s)
{
    const int64_t cap = a.max_pages << a.page_shift;
    const int64_t longest = cap < a.rows ? cap : a.rows;
    // a sequence longer than its pages still has rows to fill (with NaN)
    const int64_t tiles = ((a.rows > longest ? a.rows : longest) + kReadTok - 1) / kReadTok;
    hipLaunchKernelGGL((k_kv_read<C, O, D>),
                       dim3(static_cast<uint32_t>(tiles), static_cast<uint32_t>(batch * a.hkv)), dim3(kKvThreads), 0, s,
                       a);
    return hipGetLastError();
}

template <typename C, typename O>
hipError_t read_d(const KvReadArgs &a, int64_t batch, int d, hipStream_t s)
{
    return d == 64 ? read_launch<C, O, 64>(a, batch, s)
                   : d == 128 ? read_launch<C, O, 128>(a, batch, s) : read_launch<C, O, 256>(a, batch, s);
}

template <typename C>
hipError_t read_o(const KvReadArgs &a, int64_t batch, int d, int o, hipStream_t s)
{
    return o == PTQ1_F32 ? read_d<C, float>(a, batch, d, s)
                         : o == PTQ1_F16 ? read_d<C, _Float16>(a, batch, d, s) : read_d<C, __bf16>(a, batch, d, s);
}

}  // namespace

hipError_t launch_kv_write(const void *q, int64_t qs, const void *k, int64_t ks, const void *v, int64_t vs, int src,
                           int64_t tokens, int32_t hq, const int32_t *positions, const float *cos_sin,
                           int64_t n_positions, int32_t rot, const int64_t *slots, void *q_out, int q_type,
                           const ptq1_kv_cache &c, hipStream_t s)
{
    KvWriteArgs a{q,     k,     v,         qs,          ks,        vs,        tokens, hq,
                  c.n_kv_heads, positions, cos_sin, n_positions, rot, slots, q_out, c.k_pages, c.v_pages,
                  c.k_steps, c.v_steps, c.n_pages * c.page_size, log2_of(c.page_size), 0};
    return src == PTQ1_F32 ? write_q<float>(a, c.head_dim, c.dtype, q_type, s)
                           : src == PTQ1_F16 ? write_q<_Float16>(a, c.head_dim, c.dtype, q_type, s)
                                             : write_q<__bf16>(a, c.head_dim, c.dtype, q_type, s);
}

hipError_t launch_kv_read(const ptq1_kv_cache &c, const int32_t *table, int64_t max_pages, const int32_t *cu,
                          int64_t batch, int64_t rows, void *k_out, void *v_out, int out_type, hipStream_t s)
{
    const KvReadArgs a{c.k_pages, c.v_pages, c.k_steps, c.v_steps, c.n_pages, log2_of(c.page_size),
                       c.n_kv_heads, table, max_pages, cu, rows, k_out, v_out};
    return c.dtype == PTQ1_F16 ? read_o<_Float16>(a, batch, c.head_dim, out_type, s)
                               : c.dtype == PTQ1_BF16 ? read_o<__bf16>(a, batch, c.head_dim, out_type, s)
                                                      : read_o<int8_t>(a, batch, c.head_dim, out_type, s);
}

}  // namespace ptq1
