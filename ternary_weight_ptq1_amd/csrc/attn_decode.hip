// attn_decode.hip -- attention of one new token per sequence over the paged
// cache (ptq1_attn_decode).
//
//   out = sum_j p_j V[j] / sum_j p_j,  p_j = exp2(t_j - M),
//   t_j = scale log2(e) (q . K[j]),    M = max_j t_j
//
// in one pass with a running maximum: partial results (M, sum, rows) of
// disjoint token sets join by exp2(M_i - M) weights.  Every byte of K and V
// is read once and meets few operations, so HBM bounds it; what the design
// is about is keeping enough loads in flight and nothing else in their way:
//
//   - The products run on 16x16x32 MFMA with the tokens on the rows:
//     S^T = K Q^T (16 tokens x 16 query heads of one kv head), and O^T =
//     V^T P^T (16 dimensions x 16 heads).  The K pages are token-major and the
//     V pages dimension-major, so both A operands are 16 contiguous bytes per
//     lane straight from HBM: no LDS, no transposition, no barrier in the
//     loop.
//   - The rows of the S^T tiles are assigned to tokens so that the result
//     registers of a lane are 8 (int8 caches: 16) consecutive tokens of its
//     head: exactly the k-slots of the lane's V operand, so P goes from the
//     softmax into the second product without leaving its lane.
//   - A wave's next K is requested as soon as the first product has consumed
//     the current one, its next V after the second: one of the two is always
//     in flight.
//   - Sixteen heads cost the same as one here (the MFMA has 16 columns), and
//     the matrix cores are nearly idle, so fp32 queries and the weights enter
//     as two or three 16-bit terms: K and V are exact, so the result is that
//     of fp32 products.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "ptq1_attn.h"
#include "ptq1_launch.h"

namespace ptq1 {
namespace {

constexpr int kDecWaves = 4;
constexpr int kDecThreads = 64 * kDecWaves;
constexpr int kDecHeads = 16;       // query heads per workgroup (MFMA columns)
constexpr int kMaxChunks = 1024;    // chunks of one sequence (the join's LDS)
constexpr int64_t kMaxChunk = 4096; // tokens (page indices of a chunk in LDS: 256 pages of 16)

struct DecodeArgs {
    const void *q;
    int32_t hq, hkv, hblocks;  // hblocks: groups of 16 query heads per kv head
    const void *k_pages, *v_pages;
    const float *k_steps, *v_steps;
    int64_t n_pages;
    int32_t page_shift;
    const int32_t *table;
    int64_t max_pages;
    const int32_t *lens;
    int64_t max_len, chunk, chunks;
    float scale;
    void *out;
    float *part_rows, *part_ml;
};

// MFMA operand type of a cache type
template <typename C>
struct OpOf {
    typedef C type;
};
template <>
struct OpOf<int8_t> {
    typedef __bf16 type;
};

// The n-th 16-bit term of x: x = hi + mid + lo with each term the rounding
// of what the earlier ones left (bf16: 24 bits in three terms; fp16: 22 in two
// down to 2^-24, so values are near 1 there).
template <typename T, int N>
__device__ __forceinline__ void split_terms(const float (&x)[8], typename Op16<T>::x8 (&out)[N])
{
    float r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = x[j];
#pragma unroll
    for (int n = 0; n < N; ++n) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const T h = static_cast<T>(r[j]);
            out[n][j] = h;
            if (n + 1 < N) r[j] -= static_cast<float>(h);
        }
    }
}

// 8 int8 codes (two dwords) as bf16: exact.
__device__ __forceinline__ bf16x8 codes_to_bf16(uint32_t a, uint32_t b)
{
    bf16x8 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        o[j] = static_cast<__bf16>(static_cast<float>(static_cast<int8_t>(a >> (8 * j))));
        o[4 + j] = static_cast<__bf16>(static_cast<float>(static_cast<int8_t>(b >> (8 * j))));
    }
    return o;
}

// C: cache element, QT: type of q and out, D: head_dim, NQ / NP: 16-bit terms
// of the queries and the weights.
template <typename C, typename QT, int D, int NQ, int NP>
__global__ void __launch_bounds__(kDecThreads, D == 256 ? 1 : 2) k_attn_decode(DecodeArgs a)
{
    constexpr bool I8 = std::is_same<C, int8_t>::value;
    typedef typename OpOf<C>::type T;
    typedef typename Op16<T>::x8 x8;
    constexpr int TS = I8 ? 64 : 32;        // tokens of one step
    constexpr int NT = TS / 16;             // score tiles of one step
    constexpr int RUN = TS / 4;             // consecutive tokens of a lane
    constexpr int NL = D / 16;              // 16-byte loads per lane and step, for K and for V
    constexpr int KK = D / 32;              // MFMA steps over the head dimension
    constexpr int LPT = NL / NT;            // K loads per score tile

    extern __shared__ __attribute__((aligned(16))) char lds[];
    __shared__ int32_t pages[kMaxChunk / 16];
    __shared__ float wm[kDecWaves][kDecHeads], wl[kDecWaves][kDecHeads];
    __shared__ int bad_page;

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = lane & 15, grp = lane >> 4;
    const int64_t b = blockIdx.z;
    const int kh = static_cast<int>(blockIdx.y) / a.hblocks, hb = static_cast<int>(blockIdx.y) % a.hblocks;
    const int group = a.hq / a.hkv;
    const int h0 = kh * group + hb * kDecHeads;                                  // first query head
    const int nh = group - hb * kDecHeads < kDecHeads ? group - hb * kDecHeads : kDecHeads;
    const int64_t len = a.lens[b];
    const bool bad_len = len < 0 || len > a.max_len;
    const int64_t c0 = static_cast<int64_t>(blockIdx.x) * a.chunk;
    const int64_t c1 = bad_len ? c0 : (c0 + a.chunk < len ? c0 + a.chunk : len);
    if (c0 >= c1 && blockIdx.x != 0) return;  // the join reads the first chunk and those below the length
    const int ntok = static_cast<int>(c1 > c0 ? c1 - c0 : 0);
    const int page_mask = (1 << a.page_shift) - 1;

    // ---- the chunk's pages (a bad one: page 0 is read, and the rows end NaN)
    if (threadIdx.x == 0) bad_page = bad_len ? 1 : 0;
    __syncthreads();
    for (int i = threadIdx.x; i < (ntok + page_mask) >> a.page_shift; i += kDecThreads) {
        int32_t pg = a.table[b * a.max_pages + (c0 >> a.page_shift) + i];
        if (pg < 0 || pg >= a.n_pages) {
            bad_page = 1;
            pg = 0;
        }
        pages[i] = pg;
    }

    // ---- queries: B operand, column = head, k = 8 consecutive dimensions
    // (int8: dimension 64 p + 16 grp + 8 s of steps 2 p + s, the bytes a lane
    // loads at once; else 32 kk + 8 grp)
    float c = a.scale * kLog2e;  // scores in units of log2
    x8 qf[KK][NQ];
    {
        const QT *qp = static_cast<const QT *>(a.q) + (b * a.hq + h0 + (col < nh ? col : 0)) * D;
        float mul = 1.0f;
        if constexpr (std::is_same<T, _Float16>::value && std::is_same<QT, float>::value) {
            // fp16 terms: bring the head's largest magnitude to [1, 2)
            float m = 0.0f;
            for (int kk = 0; kk < KK; ++kk)
#pragma unroll
                for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(static_cast<float>(qp[32 * kk + 8 * grp + j])));
            m = lane_pair_max<32>(lane_pair_max<16>(m));
            if (m > 0x1p-120f && m < 0x1p120f) {
                const int e = static_cast<int>((__builtin_bit_cast(uint32_t, m) >> 23) & 255u) - 127;
                mul = __builtin_bit_cast(float, static_cast<uint32_t>(127 - e) << 23);
                c *= __builtin_bit_cast(float, static_cast<uint32_t>(127 + e) << 23);
            }
        }
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            const int d0 = I8 ? 64 * (kk >> 1) + 16 * grp + 8 * (kk & 1) : 32 * kk + 8 * grp;
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = static_cast<float>(qp[d0 + j]) * mul;
            split_terms<T, NQ>(x, qf[kk]);
        }
    }
    __syncthreads();

    // ---- one step's loads.  Tokens past the chunk's end are read from its
    // last token (K) or last run (V), and masked below.
    const int last = ntok - 1;
    const char *kp = static_cast<const char *>(a.k_pages), *vp = static_cast<const char *>(a.v_pages);
    auto load_k = [&](int base, at_u32x4 (&r)[NL]) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            int tok = base + RUN * (col >> 2) + 4 * t + (col & 3);
            tok = tok < last ? tok : last;
            const int64_t cell = ((static_cast<int64_t>(pages[tok >> a.page_shift]) * a.hkv + kh) << a.page_shift) +
                                 (tok & page_mask);
            const char *src = kp + cell * (D * static_cast<int64_t>(sizeof(C))) + 16 * grp;
#pragma unroll
            for (int i = 0; i < LPT; ++i) r[t * LPT + i] = *reinterpret_cast<const at_u32x4 *>(src + 64 * i);
        }
    };
    auto run_of = [&](int base) {
        const int tok = base + RUN * grp, lr = last & ~(RUN - 1);
        return tok < lr ? tok : lr;
    };
    auto load_v = [&](int base, at_u32x4 (&r)[NL]) {
        const int tok = run_of(base);
        const int64_t pgh = static_cast<int64_t>(pages[tok >> a.page_shift]) * a.hkv + kh;
        const char *src = vp + (((pgh * D + col) << a.page_shift) + (tok & page_mask)) * static_cast<int64_t>(sizeof(C));
        const int64_t stride = (static_cast<int64_t>(16) << a.page_shift) * sizeof(C);
#pragma unroll
        for (int i = 0; i < NL; ++i) r[i] = *reinterpret_cast<const at_u32x4 *>(src + i * stride);
    };
    auto load_steps = [&](int base, at_f32x4 (&ks)[NT], at_f32x4 (&vs)[NT]) {
        const int tok = run_of(base);
        const int64_t cell = ((static_cast<int64_t>(pages[tok >> a.page_shift]) * a.hkv + kh) << a.page_shift) +
                             (tok & page_mask);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            ks[t] = *reinterpret_cast<const at_f32x4 *>(a.k_steps + cell + 4 * t);
            vs[t] = *reinterpret_cast<const at_f32x4 *>(a.v_steps + cell + 4 * t);
        }
    };

    const at_f32x4 zero4 = {0.0f, 0.0f, 0.0f, 0.0f};
    at_f32x4 o[D / 16];
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[i] = zero4;
    float m = -__builtin_inff(), l = 0.0f;

    at_u32x4 kr[NL], vr[NL];
    at_f32x4 ks[NT], vs[NT];
    int base = wave * TS;
    if (base < ntok) {
        load_k(base, kr);
        if constexpr (I8) load_steps(base, ks, vs);
        load_v(base, vr);
    }
    for (; base < ntok; base += kDecWaves * TS) {
        const int next = base + kDecWaves * TS;
        // ---- scores: tile t, register i of lane: token base + RUN grp + 4 t + i, head col
        at_f32x4 s[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            s[t] = zero4;
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                x8 kf;
                if constexpr (I8) {
                    at_u32x4 w = kr[t * LPT + (kk >> 1)];
                    asm volatile("" : "+v"(w));  // keeps the codes packed up to here
                    kf = kk & 1 ? codes_to_bf16(w[2], w[3]) : codes_to_bf16(w[0], w[1]);
                } else {
                    kf = __builtin_bit_cast(x8, kr[t * LPT + kk]);
                }
#pragma unroll
                for (int n = 0; n < NQ; ++n) s[t] = Op16<T>::mfma16(kf, qf[kk][n], s[t]);
            }
            if constexpr (I8) __builtin_amdgcn_sched_barrier(0);  // or every code is converted up front, into spills
        }
        at_f32x4 vsc[NT];
        if constexpr (I8) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                s[t] *= ks[t];
                vsc[t] = vs[t];
            }
        }
        if (next < ntok) {
            load_k(next, kr);
            if constexpr (I8) load_steps(next, ks, vs);
        }
        const bool tail = base + TS > ntok;
        float top = -__builtin_inff();
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[t][i] *= c;
                if (tail && base + RUN * grp + 4 * t + i >= ntok) s[t][i] = -__builtin_inff();
                top = fmaxf(top, s[t][i]);
            }
        top = lane_pair_max<32>(lane_pair_max<16>(top));
        // a larger maximum rescales what is there (all lanes of a head alike)
        if (__ballot(top > m) != 0) {
            const float mn = fmaxf(m, top);
            const float f = m == mn ? 1.0f : exp2f(m - mn);
            l *= f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) o[i] *= f;
            m = mn;
        }
        const float ms = m == -__builtin_inff() ? 0.0f : m;
        float p[TS / 4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float e = exp2f(s[t][i] - ms);
                l += e;
                if constexpr (I8) e = tail && base + RUN * grp + 4 * t + i >= ntok ? 0.0f : e * vsc[t][i];
                p[4 * t + i] = e;
            }
        // ---- O^T += V^T P^T, slot j of step u: token base + RUN grp + 8 u + j
        if (tail) {
            // what lies past the end may hold anything; zero weights do not silence a NaN
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                constexpr int PER = 4 / sizeof(C);  // tokens per dword
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int left = ntok - (base + RUN * grp + PER * w);
                    const uint32_t keep = left >= PER ? 0xffffffffu
                                          : left <= 0 ? 0u
                                                      : (1u << (8 * static_cast<int>(sizeof(C)) * left)) - 1u;
                    vr[i][w] &= keep;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < NT / 2; ++u) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = p[8 * u + j];
            x8 pf[NP];
            split_terms<T, NP>(x, pf);
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                x8 vf;
                if constexpr (I8) {
                    at_u32x2 w = {vr[i][2 * u], vr[i][2 * u + 1]};
                    asm volatile("" : "+v"(w));
                    vf = codes_to_bf16(w[0], w[1]);
                } else
                    vf = __builtin_bit_cast(x8, vr[i]);
#pragma unroll
                for (int n = 0; n < NP; ++n) o[i] = Op16<T>::mfma16(vf, pf[n], o[i]);
                if constexpr (I8)
                    if ((i & 1) == 1) __builtin_amdgcn_sched_barrier(0);
            }
        }
        if (next < ntok) load_v(next, vr);
    }
    l = lane_pair_sum<32>(lane_pair_sum<16>(l));

    // ---- join the four waves: rows in LDS [wave][head][D + 4]
    float *rows = reinterpret_cast<float *>(lds);
    if (grp == 0) {
        wm[wave][col] = m;
        wl[wave][col] = l;
    }
    if (col < nh) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
            *reinterpret_cast<at_f32x4 *>(rows + (wave * nh + col) * (D + 4) + 16 * i + 4 * grp) = o[i];
    }
    __syncthreads();
    const bool bad = bad_page != 0;
    for (int i = threadIdx.x; i < nh * (D / 4); i += kDecThreads) {
        const int h = i / (D / 4), e = (i % (D / 4)) * 4;
        float M = wm[0][h];
#pragma unroll
        for (int w = 1; w < kDecWaves; ++w) M = fmaxf(M, wm[w][h]);
        const float Ms = M == -__builtin_inff() ? 0.0f : M;
        float L = 0.0f;
        at_f32x4 r = zero4;
#pragma unroll
        for (int w = 0; w < kDecWaves; ++w) {
            const float f = exp2f(wm[w][h] - Ms);
            L += f * wl[w][h];
            r += f * *reinterpret_cast<const at_f32x4 *>(rows + (w * nh + h) * (D + 4) + e);
        }
        if (bad) L = __builtin_nanf("");
        const int64_t row = b * a.hq + h0 + h;
        if (a.chunks == 1) {
            const float f = ntok == 0 && !bad ? 0.0f : 1.0f / L;
            store4(static_cast<QT *>(a.out) + row * D + e, r * f);
        } else {
            *reinterpret_cast<at_f32x4 *>(a.part_rows + (row * a.chunks + blockIdx.x) * D + e) = r;
            if (e == 0) {
                a.part_ml[(row * a.chunks + blockIdx.x) * 2] = M;
                a.part_ml[(row * a.chunks + blockIdx.x) * 2 + 1] = L;
            }
        }
    }
}

// Joins a row's chunks: one workgroup per (query head, sequence), its D / 4
// lanes wide groups taking every n-th chunk, then a sum over the groups in
// LDS.
template <typename QT, int D>
__global__ void __launch_bounds__(256) k_attn_join(DecodeArgs a)
{
    constexpr int LPR = D / 4, G = 256 / LPR;
    __shared__ float wgt[kMaxChunks];
    __shared__ float red[4];
    __shared__ at_f32x4 sums[G][LPR];
    const int64_t b = blockIdx.y;
    const int64_t row = b * a.hq + blockIdx.x;
    const int64_t len = a.lens[b];
    const int n = len <= 0 || len > a.max_len ? 1 : static_cast<int>((len + a.chunk - 1) / a.chunk);
    const float *ml = a.part_ml + row * a.chunks * 2;
    float M = -__builtin_inff();
    for (int i = threadIdx.x; i < n; i += 256) M = fmaxf(M, ml[2 * i]);
    M = wave_max(M);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = M;
    __syncthreads();
    M = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    if (M == -__builtin_inff()) M = 0.0f;
    __syncthreads();
    float L = 0.0f;
    for (int i = threadIdx.x; i < n; i += 256) {
        const float w = exp2f(ml[2 * i] - M);
        wgt[i] = w;
        L += w * ml[2 * i + 1];
    }
    L = wave_sum(L);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = L;
    __syncthreads();
    L = (red[0] + red[1]) + (red[2] + red[3]);
    const int g = threadIdx.x / LPR, x = threadIdx.x % LPR;
    at_f32x4 r = {0.0f, 0.0f, 0.0f, 0.0f};
    const float *pr = a.part_rows + row * a.chunks * D + 4 * x;
#pragma unroll 8
    for (int i = g; i < n; i += G) r += wgt[i] * *reinterpret_cast<const at_f32x4 *>(pr + static_cast<int64_t>(i) * D);
    sums[g][x] = r;
    __syncthreads();
    if (g == 0) {
#pragma unroll
        for (int i = 1; i < G; ++i) r += sums[i][x];
        store4(static_cast<QT *>(a.out) + row * D + 4 * x, r * (len == 0 ? 0.0f : 1.0f / L));
    }
}

template <typename C, typename QT, int D, int NQ, int NP>
hipError_t decode_launch(const DecodePlan &p, const DecodeArgs &a, int64_t batch, hipStream_t s)
{
    static std::atomic<uint64_t> lds_done{0};
    const auto kernel = k_attn_decode<C, QT, D, NQ, NP>;
    constexpr int kMaxLds = kDecWaves * kDecHeads * (D + 4) * 4;
    const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void *>(kernel), kMaxLds, lds_done);
    if (e != hipSuccess) return e;
    const int group = a.hq / a.hkv;
    const int lds = kDecWaves * (group < kDecHeads ? group : kDecHeads) * (D + 4) * 4;
    hipLaunchKernelGGL(kernel,
                       dim3(static_cast<uint32_t>(p.chunks), static_cast<uint32_t>(a.hkv * a.hblocks),
                            static_cast<uint32_t>(batch)),
                       dim3(kDecThreads), lds, s, a);
    if (p.chunks > 1)
        hipLaunchKernelGGL((k_attn_join<QT, D>), dim3(static_cast<uint32_t>(a.hq), static_cast<uint32_t>(batch)),
                           dim3(256), 0, s, a);
    return hipGetLastError();
}

template <typename C, typename QT, int NQ, int NP>
hipError_t decode_d(const DecodePlan &p, const DecodeArgs &a, int64_t batch, int d, hipStream_t s)
{
    return d == 64 ? decode_launch<C, QT, 64, NQ, NP>(p, a, batch, s)
                   : d == 128 ? decode_launch<C, QT, 128, NQ, NP>(p, a, batch, s)
                              : decode_launch<C, QT, 256, NQ, NP>(p, a, batch, s);
}

}  // namespace

DecodePlan decode_plan(int64_t batch, int32_t hq, int32_t hkv, int32_t d, int64_t max_len)
{
    DecodePlan p;
    const int64_t group = hq / hkv, hblocks = (group + kDecHeads - 1) / kDecHeads;
    const int64_t per = batch * hkv * hblocks;
    // about four workgroups per CU when every sequence is at its bound
    int64_t chunk = (max_len * per + 1023) / 1024;
    chunk = (chunk + 255) / 256 * 256;
    const int64_t least = ((max_len + kMaxChunks - 1) / kMaxChunks + 255) / 256 * 256;
    if (chunk > 1024) chunk = 1024;
    if (chunk < least) chunk = least;
    if (chunk < 256) chunk = 256;
    p.chunk = chunk;
    p.chunks = max_len > 0 ? (max_len + chunk - 1) / chunk : 1;
    if (p.chunks > 1) {
        p.rows_floats = static_cast<size_t>(batch) * hq * p.chunks * d;
        p.part_floats = p.rows_floats + static_cast<size_t>(batch) * hq * p.chunks * 2;
    }
    return p;
}

hipError_t launch_attn_decode(const DecodePlan &p, const void *q, int q_type, int64_t batch, int32_t hq,
                              const ptq1_kv_cache &c, const int32_t *table, int64_t max_pages, const int32_t *lens,
                              int64_t max_len, float scale, void *out, float *part, hipStream_t s)
{
    const int32_t group = hq / c.n_kv_heads;
    const DecodeArgs a{q, hq, c.n_kv_heads, (group + kDecHeads - 1) / kDecHeads, c.k_pages, c.v_pages, c.k_steps,
                       c.v_steps, c.n_pages, __builtin_ctz(static_cast<unsigned>(c.page_size)), table, max_pages, lens,
                       max_len, p.chunk, p.chunks, scale, out, part, part + p.rows_floats};
    const int d = c.head_dim;
    if (c.dtype == PTQ1_BF16)
        return q_type == PTQ1_F32 ? decode_d<__bf16, float, 3, 3>(p, a, batch, d, s)
                                  : decode_d<__bf16, __bf16, 1, 2>(p, a, batch, d, s);
    if (c.dtype == PTQ1_F16)
        return q_type == PTQ1_F32 ? decode_d<_Float16, float, 3, 2>(p, a, batch, d, s)
                                  : decode_d<_Float16, _Float16, 1, 2>(p, a, batch, d, s);
    return q_type == PTQ1_F32 ? decode_d<int8_t, float, 3, 3>(p, a, batch, d, s)
           : q_type == PTQ1_F16 ? decode_d<int8_t, _Float16, 2, 2>(p, a, batch, d, s)
                                : decode_d<int8_t, __bf16, 1, 2>(p, a, batch, d, s);
}

}  // namespace ptq1
