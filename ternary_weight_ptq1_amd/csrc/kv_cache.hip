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
#include "ptq1_launch.h"

namespace ptq1 {
namespace {

constexpr int kKvThreads = 256;
constexpr int kVTok = 64;  // tokens of one V tile (write): a wave's lanes
constexpr int kRowsPer = 2;  // q and k rows a thread has in flight (write)

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
template <typename S, typename Q, typename C, int D>
__global__ void __launch_bounds__(kKvThreads) k_kv_write(KvWriteArgs a)
{
    constexpr bool I8 = std::is_same<C, int8_t>::value;
    constexpr int LPR = D / 4;               // lanes per row
    constexpr int RPB = kKvThreads / LPR;    // rows per block and pass
    const int sub = threadIdx.x / LPR, e = (threadIdx.x % LPR) * 4;
    const int64_t page = int64_t{1} << a.page_shift;

    if (blockIdx.x >= a.v_blocks) {
        const uint32_t heads = static_cast<uint32_t>(a.hq + a.hkv);
        const int half = a.rot >> 1;
        const bool turns = e < a.rot, upper = e >= half;
        const int lo = upper ? e - half : e, other = upper ? lo : lo + half;
        at_f32x4 x[kRowsPer], y[kRowsPer], c[kRowsPer], sn[kRowsPer];
        int64_t token[kRowsPer];
        int h[kRowsPer], pos[kRowsPer];
        bool there[kRowsPer], placed[kRowsPer];
#pragma unroll
        for (int u = 0; u < kRowsPer; ++u) {
            const uint32_t row = ((blockIdx.x - a.v_blocks) * kRowsPer + u) * RPB + sub;
            token[u] = row / heads;
            h[u] = static_cast<int>(row % heads);
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
        for (int u = 0; u < kRowsPer; ++u) {
            placed[u] = there[u] && turns && pos[u] >= 0 && pos[u] < a.n_positions;
            if (!placed[u]) continue;
            const float *cs = a.cos_sin + static_cast<int64_t>(pos[u]) * a.rot + lo;
            c[u] = load4(cs);
            sn[u] = load4(cs + half);
        }
#pragma unroll
        for (int u = 0; u < kRowsPer; ++u) {
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

int log2_of(int32_t v) { return __builtin_ctz(static_cast<unsigned>(v)); }

template <typename S, typename Q, typename C, int D>
hipError_t write_launch(KvWriteArgs &a, hipStream_t s)
{
    constexpr int RPB = kKvThreads / (D / 4) * kRowsPer;
    const int64_t rows = a.tokens * (a.hq + a.hkv);
    a.v_blocks = static_cast<uint32_t>((a.tokens + kVTok - 1) / kVTok * a.hkv * (D / kv_write_dims<C>(D)));
    hipLaunchKernelGGL((k_kv_write<S, Q, C, D>), dim3(a.v_blocks + static_cast<uint32_t>((rows + RPB - 1) / RPB)),
                       dim3(kKvThreads), 0, s, a);
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
                  c.k_steps, c.v_steps, c.n_pages * c.page_size, log2_of(c.page_size), 0};
    return src == PTQ1_F32 ? write_q<float>(a, c.head_dim, c.dtype, q_type, s)
                           : src == PTQ1_F16 ? write_q<_Float16>(a, c.head_dim, c.dtype, q_type, s)
                                             : write_q<__bf16>(a, c.head_dim, c.dtype, q_type, s);
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
