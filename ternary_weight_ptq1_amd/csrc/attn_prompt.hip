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

#include "ptq1_attn.h"
#include "ptq1_launch.h"

namespace ptq1 {
namespace {

constexpr int kPrWaves = 4;
constexpr int kPrThreads = 64 * kPrWaves;
constexpr int kPrRows = 32 * kPrWaves;  // query rows of a workgroup

typedef short at_s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) at_s16x4 lds_s16x4;

// Place (in elements) of the 16-byte piece p of key row r in a K or V tile of
// rows of D elements.  K is read 16 rows at one piece at a time, V 4 rows at
// four pieces; the exclusive-or spreads either over the 64 banks.
template <int D>
__device__ __forceinline__ int k_place(int r, int p)
{
    constexpr int P = D / 8;  // pieces of a row
    const int x = P >= 16 ? r & 15 : (r >> 1) & 7;
    return r * D + ((p ^ x) << 3);
}
template <int D>
__device__ __forceinline__ int v_place(int r, int p)
{
    const int x = D >= 128 ? (r & 3) << 2 : ((r >> 1) & 1) << 2;
    return r * D + ((p ^ x) << 3);
}

template <typename T, int D>
__global__ void __launch_bounds__(kPrThreads, D == 256 ? 1 : 2) k_attn_prompt(PromptArgs a, int32_t tiles)
{
    typedef typename Op16<T>::x8 x8;
    constexpr int BN = D == 256 ? 32 : 64;  // keys of a tile
    constexpr int KT = BN / 32;             // score tiles
    constexpr int DT = D / 32;              // output tiles
    constexpr int KK = D / 16;              // MFMA steps over the head dimension
    constexpr int P = D / 8;                // 16-byte pieces of a row
    constexpr int NLD = BN * P / kPrThreads;  // pieces a thread stages, of K and of V

    extern __shared__ __attribute__((aligned(16))) char lds[];
    T *kt = reinterpret_cast<T *>(lds);            // [2][BN * D]
    T *vt = kt + 2 * BN * D;                       // [2][BN * D]

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = lane & 31, half = lane >> 5;

    const int64_t pairs = a.batch * a.hkv;
    const int64_t pair = static_cast<int64_t>(blockIdx.x) % pairs;
    const int64_t b = pair / a.hkv;
    const int kh = static_cast<int>(pair % a.hkv);
    const int group = a.hq / a.hkv;
    const int64_t q0 = a.cu_q[b], k0 = a.cu_k[b];
    const int64_t lq = a.cu_q[b + 1] - q0, lk = a.cu_k[b + 1] - k0;
    if (lq <= 0) return;
    const int64_t rows = lq * group;
    const bool bad = q0 < 0 || k0 < 0 || q0 + lq > a.q_rows || lk < 0 || k0 + lk > a.k_rows || lq > a.max_q ||
                     lk > a.max_k;
    if (bad) {
        for (int64_t r = static_cast<int64_t>(blockIdx.x) / pairs * kPrRows + threadIdx.x; r < rows;
             r += static_cast<int64_t>(tiles) * kPrRows) {
            if (threadIdx.x >= kPrRows) break;
            const int64_t tok = q0 + r / group;
            if (tok < 0 || tok >= a.q_rows) continue;
            T *dst = static_cast<T *>(a.out) + (tok * a.hq + kh * group + r % group) * D;
            const float n = __builtin_nanf("");
            for (int e = 0; e < D; e += 4) store4(dst + e, at_f32x4{n, n, n, n});
        }
        return;
    }
    // the last rows see the most keys: they start first
    const int64_t nt = (rows + kPrRows - 1) / kPrRows;
    const int64_t tile = nt - 1 - static_cast<int64_t>(blockIdx.x) / pairs;
    if (tile < 0) return;

    const int64_t row = tile * kPrRows + 32 * wave + col;
    const int64_t rowc = row < rows ? row : rows - 1;
    const int32_t tok = static_cast<int32_t>(rowc / group), head = static_cast<int32_t>(rowc % group);
    // keys below `seen` are visible to this lane's row
    const int64_t off = lk - lq;
    int64_t seen64 = a.causal ? tok + off + 1 : lk;
    if (seen64 < 0) seen64 = 0;
    const int seen = static_cast<int>(seen64);
    const int64_t tok_first = tile * kPrRows / group;
    const int64_t row_last = (tile + 1) * kPrRows < rows ? (tile + 1) * kPrRows - 1 : rows - 1;
    int64_t all64 = a.causal ? tok_first + off + 1 : lk;                 // keys that every row of the tile sees
    int64_t any64 = a.causal ? row_last / group + off + 1 : lk;         // keys that some row sees
    const int all = static_cast<int>(all64 < 0 ? 0 : all64), any = static_cast<int>(any64 < 0 ? 0 : any64);

    // ---- queries: B operand, column = row, k = 16 kk + 8 half + j
    x8 qf[KK];
    {
        const T *qp = static_cast<const T *>(a.q) + (q0 + tok) * a.qs + static_cast<int64_t>(kh * group + head) * D;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) qf[kk] = *reinterpret_cast<const x8 *>(qp + 16 * kk + 8 * half);
    }

    // ---- staging: thread -> pieces (row i * RS + threadIdx.x / P, piece threadIdx.x % P)
    constexpr int RS = kPrThreads / P;
    const int sr = threadIdx.x / P, sp = threadIdx.x % P;
    const T *kp = static_cast<const T *>(a.k) + (k0 + sr) * a.ks + static_cast<int64_t>(kh) * D + 8 * sp;
    const T *vp = static_cast<const T *>(a.v) + (k0 + sr) * a.vs + static_cast<int64_t>(kh) * D + 8 * sp;
    at_u32x4 kr[NLD], vr[NLD];
    const at_u32x4 zero = {0u, 0u, 0u, 0u};
    auto load_tile = [&](int n0) {
#pragma unroll
        for (int i = 0; i < NLD; ++i) {
            const int r = n0 + i * RS;
            const bool in = r + sr < any;  // past the last visible key: zeros
            kr[i] = in ? *reinterpret_cast<const at_u32x4 *>(kp + r * a.ks) : zero;
            vr[i] = in ? *reinterpret_cast<const at_u32x4 *>(vp + r * a.vs) : zero;
        }
    };
    auto store_tile = [&](int buf) {
#pragma unroll
        for (int i = 0; i < NLD; ++i) {
            const int r = i * RS + sr;
            *reinterpret_cast<at_u32x4 *>(kt + buf * BN * D + k_place<D>(r, sp)) = kr[i];
            *reinterpret_cast<at_u32x4 *>(vt + buf * BN * D + v_place<D>(r, sp)) = vr[i];
        }
    };

    const float c = a.scale * kLog2e;
    at_f32x16 o[DT];
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] = 0.0f;
    float m = -__builtin_inff(), l = 0.0f;  // m: in units of log2

    if (any > 0) {
        load_tile(0);
        store_tile(0);
    }
    __syncthreads();
    int buf = 0;
    for (int n0 = 0; n0 < any; n0 += BN, buf ^= 1) {
        const bool more = n0 + BN < any;
        if (more) load_tile(n0 + BN);
        const T *kb = kt + buf * BN * D, *vb = vt + buf * BN * D;
        // ---- S^T
        at_f32x16 s[KT];
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
        if (n0 + BN > all) {
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (n0 + 32 * t + 8 * (j >> 2) + 4 * half + (j & 3) >= seen) s[t][j] = -__builtin_inff();
        }
        // ---- softmax
        float top = s[0][0];
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int j = 0; j < 16; ++j) top = fmaxf(top, s[t][j]);
        top = lane_pair_max<32>(top) * c;
        if (__ballot(top > m) != 0) {
            const float mn = fmaxf(m, top);
            const float f = m == mn ? 1.0f : exp2f(m - mn);
            l *= f;
#pragma unroll
            for (int i = 0; i < DT; ++i) o[i] *= f;
            m = mn;
        }
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
        // ---- O^T += V^T P^T
#pragma unroll
        for (int u = 0; u < 2 * KT; ++u) {
#pragma unroll
            for (int i = 0; i < DT; ++i) {
                // lane: key 16 u + 4 half + (lane % 16) / 4 (then + 8), dimensions 32 i + 16 ((lane / 16) % 2) + 4 (lane % 4)
                const int r = 16 * u + 4 * half + ((lane & 15) >> 2);
                const int d = 32 * i + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
                const at_s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (lds_s16x4 *)(vb + v_place<D>(r, d >> 3) + (d & 7)));
                const at_s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (lds_s16x4 *)(vb + v_place<D>(r + 8, d >> 3) + (d & 7)));
                const auto w = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
                o[i] = Op16<T>::mfma32(__builtin_bit_cast(x8, w), pf[u], o[i]);
            }
        }
        if (more) store_tile(buf ^ 1);
        __syncthreads();
    }
    l = lane_pair_sum<32>(l);
    if (row < rows) {
        const float f = seen == 0 ? 0.0f : 1.0f / l;
        T *dst = static_cast<T *>(a.out) + ((q0 + tok) * a.hq + kh * group + head) * D;
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
            for (int j = 0; j < 16; j += 4)
                store4(dst + 32 * i + 2 * j + 4 * half,
                       at_f32x4{o[i][j] * f, o[i][j + 1] * f, o[i][j + 2] * f, o[i][j + 3] * f});
    }
}

template <typename T, int D>
hipError_t prompt_launch(const PromptArgs &a, hipStream_t s)
{
    static std::atomic<uint64_t> lds_done{0};
    constexpr int BN = D == 256 ? 32 : 64;
    constexpr int lds = 4 * BN * D * 2;
    const auto kernel = k_attn_prompt<T, D>;
    const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void *>(kernel), lds, lds_done);
    if (e != hipSuccess) return e;
    const int64_t tiles = (a.max_q * (a.hq / a.hkv) + kPrRows - 1) / kPrRows;
    hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(tiles * a.batch * a.hkv)), dim3(kPrThreads), lds, s, a,
                       static_cast<int32_t>(tiles));
    return hipGetLastError();
}

template <typename T>
hipError_t prompt_d(const PromptArgs &a, int d, hipStream_t s)
{
    return d == 64 ? prompt_launch<T, 64>(a, s) : d == 128 ? prompt_launch<T, 128>(a, s) : prompt_launch<T, 256>(a, s);
}

}  // namespace

size_t prompt_part_floats(int64_t, int32_t, int32_t, int32_t, int64_t, int64_t) { return 0; }

hipError_t launch_attn_prompt(const PromptArgs &a, int dtype, int32_t d, float *, hipStream_t s)
{
    return dtype == PTQ1_BF16 ? prompt_d<__bf16>(a, d, s) : prompt_d<_Float16>(a, d, s);
}

}  // namespace ptq1
