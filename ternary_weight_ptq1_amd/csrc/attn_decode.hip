// attn_decode.hip -- attention of one new token per sequence over the paged
// cache (ptq1_attn_decode), or over a window of it (ptq1_attn_decode_window).
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
//   - The first K and V are requested before the queries are converted.
//   - A wave's next K is requested as soon as the first product has consumed
//     the current one, its next V after the second: one of the two is always
//     in flight.
//   - Sixteen heads cost the same as one here (the MFMA has 16 columns), and
//     the matrix cores are nearly idle, so fp32 queries and the weights enter
//     as two or three 16-bit terms: K and V are exact, so the result is that
//     of fp32 products.
//
// Measured: 64 sequences of 3 to 8190 tokens, 32 heads over 8 of 128, bf16:
// 55 us and 5 for the join (261 MB: 4.7 TB/s; a copy 5.4); 16 sequences of
// 900 to 5000 tokens, 24 heads over 4 of 256, fp16: 31 and 5.  77 tokens of
// one sequence: 4.7 us in one launch.  A kv head of more than 16 query heads is
// read once for every 16: 40 heads over one, those 64 sequences, 20 us and 5
// for 99 MB fetched of 33.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "ptq1_attn.h"
#include "ptq1_launch.h"
#include "ptq1_split.h"

namespace ptq1 {
namespace {

constexpr int kDecWaves = 4;
constexpr int kDecThreads = 64 * kDecWaves;
constexpr int kDecHeads = 16;       // query heads per workgroup (MFMA columns)
constexpr int kMaxShares = 512;     // a sequence's pieces are twice that at most (the join's LDS)

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
    int64_t batch, max_len;
    int32_t shares;  // workgroups that the GPU holds for one kv head (for 16 query heads of it)
    int32_t cut;     // some sequence may be cut
    int32_t lowered;  // the parts' rows are 2^sum_exponent of their sum of weights times lower (int8 caches)
    float scale;
    void *out;
    float *part_rows, *part_ml;
    int32_t window, sinks;  // of the windowed calls
};

__device__ __forceinline__ int wave_total(int v)
{
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
    return __builtin_amdgcn_readfirstlane(v);
}

// The lengths of sequences lane, lane + 64 ..., of which the first stays in a
// register: a batch of 64 makes one trip to memory for them.
struct LaneLens {
    int first;
    __device__ __forceinline__ LaneLens(const DecodeArgs &a)
    {
        const int64_t lane = threadIdx.x & 63;
        first = lane < a.batch ? a.lens[lane] : 0;
    }
    // the sum of f(length) over the sequences before `end`
    template <class F>
    __device__ __forceinline__ int sum(const DecodeArgs &a, int64_t end, F f) const
    {
        int v = 0;
        for (int64_t i = threadIdx.x & 63; i < end; i += 64) v += f(i < 64 ? first : a.lens[i]);
        return wave_total(v);
    }
};

// Tokens of a sequence of `len` that are read (of one that is refused: what it
// is refused for).
template <bool WIN>
__device__ __forceinline__ int tokens_read(const DecodeArgs &a, int len)
{
    if constexpr (WIN)
        if (len > 0 && len <= a.max_len) return window_of(len, a.window, a.sinks).tokens;
    return len;
}

// Steps of one workgroup's piece of a sequence.
template <bool WIN>
__device__ __forceinline__ int piece_steps(const DecodeArgs &a, const LaneLens &lens)
{
    const int total = lens.sum(a, a.batch, [&](int n) { return decode_steps(tokens_read<WIN>(a, n), a.max_len); });
    return steps_per_piece(total, wanted_pieces(a.batch, a.shares));
}

// MFMA operand type of a cache type
template <typename C>
struct OpOf {
    typedef C type;
};
template <>
struct OpOf<int8_t> {
    typedef _Float16 type;
};

// The n-th 16-bit term of x: x = hi + mid + lo with each term the rounding
// of what the earlier ones left (bf16: 24 bits in three terms; fp16: 22 in two
// down to 2^-24, so values are near 1 there).
template <typename T, int N>
__device__ __forceinline__ void split_terms(const float (&x)[8], typename Op16<T>::x8 (&out)[N])
{
    float r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        r[j] = x[j];
        // one rounding of x for all its uses: the product behind x, fused into
        // the first term alone, rounds the other way now and then, and the
        // second term then lacks 2^-11 of x
        if (N > 1) asm volatile("" : "+v"(r[j]));
    }
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

// The e of the power of two 2^e above a sum of weights (0 for 0, NaN and infinity).
__device__ __forceinline__ int sum_exponent(float l) { return __builtin_amdgcn_frexp_expf(l); }

// C: cache element, QT: type of q and out, D: head_dim, NQ: 16-bit terms of
// the queries (int8 caches: 8-bit digits), NP: 16-bit terms of the weights.
//
// int8 caches: K's codes are operands as they are, of the int8 MFMA; the
// queries are fixed-point numbers of NQ signed 8-bit digits, scaled by a
// power of two to the head's largest magnitude, and the digits' exact int32
// products are joined in fp32.  V's codes become fp16 (exactly), the token's
// step goes into its weight, relative to a running power of two that no such
// product exceeds.  Converting both to bf16 and taking the steps' whole range
// there spent 1300 vector instructions on 64 tokens instead of about 560: 93
// us for 131071 tokens of 8 heads of 128 where 60 are enough now.
//
// WIN: a sliding window and first tokens that stay visible.  The tokens that
// are read are numbered without the gap between them (WindowTokens): all of
// the above then works on these numbers, and a token's real number is needed
// for its page and its place in it alone.  What is read beside the tokens that
// are seen (the rest of two runs of 16) is masked like what lies past the end.
// 64 sequences of 3 to 131072 tokens (32 heads over 8 of 128, bf16), windows of
// 4096: 462 MB in 91 us (5.1 TB/s) and 6 for the join.
template <typename C, typename QT, int D, int NQ, int NP, bool WIN>
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
    __shared__ float wm[kDecWaves][kDecHeads], wl[kDecWaves][kDecHeads];

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = lane & 15, grp = lane >> 4;
    const int page_shift = a.page_shift, page_mask = (1 << page_shift) - 1;
    // heads vary fastest: the same number of chunks for each of the eight XCDs
    const uint32_t hgroups = static_cast<uint32_t>(a.hkv * a.hblocks);
    const int hg = static_cast<int>(blockIdx.x % hgroups);
    const int kh = hg / a.hblocks, hb = hg % a.hblocks;
    const int group = a.hq / a.hkv;
    const int h0 = kh * group + hb * kDecHeads;                                  // first query head
    const int nh = group - hb * kDecHeads < kDecHeads ? group - hb * kDecHeads : kDecHeads;
    // ---- this workgroup's piece: up to `per` steps of one sequence
    const int64_t piece = blockIdx.x / hgroups;
    // (every argument in one trip to memory: the branch would take more)
    asm volatile("" ::"s"(a.q), "s"(a.k_pages), "s"(a.v_pages), "s"(a.k_steps), "s"(a.v_steps), "s"(a.n_pages),
                 "s"(a.page_shift), "s"(a.table), "s"(a.max_pages), "s"(a.lens), "s"(a.batch), "s"(a.max_len),
                 "s"(a.shares), "s"(a.scale));
    int per = kMaxSteps, b = static_cast<int>(piece), first = 0, len;
    if (a.cut) {
        const LaneLens lens(a);
        per = piece_steps<WIN>(a, lens);
        int64_t seq, tile;
        int mine = 0;
        const auto pieces = [&](int n) { return pieces_of(decode_steps(tokens_read<WIN>(a, n), a.max_len), per); };
        const auto of_lane = [&](int64_t) { return pieces(mine = lens.first); };
        const auto of_any = [&](int64_t i) { return pieces(a.lens[i]); };
        if (!(a.batch <= 64 ? find_tile<false>(piece, a.batch, of_lane, seq, tile)
                            : find_tile_in_runs(piece, a.batch, of_any, seq, tile)))
            return;
        b = __builtin_amdgcn_readfirstlane(static_cast<int>(seq));
        first = __builtin_amdgcn_readfirstlane(static_cast<int>(tile));
        len = a.batch <= 64 ? __builtin_amdgcn_readlane(mine, b & 63) : a.lens[b];
    } else
        len = a.lens[b];
    const bool bad_len = len < 0 || len > a.max_len;
    const WindowTokens win = WIN ? window_of(len, a.window, a.sinks) : WindowTokens{};
    const int read = tokens_read<WIN>(a, len);
    const bool whole = decode_steps(read, a.max_len) <= per;
    const PieceTokens tokens = piece_tokens(first, per, read);
    const int begin = tokens.begin, end = bad_len ? begin : tokens.end;

    // ---- the queries' own loads, first of all: of column = head, dimensions
    // 32 kk + 8 grp .. (int8: for the magnitude; and of wave kk operand kk's
    // 64 kk + 16 grp ..)
    typedef QT q8 __attribute__((ext_vector_type(8)));
    constexpr int QK = I8 ? D / 64 : KK;
    const QT *qp = static_cast<const QT *>(a.q) + (static_cast<int64_t>(b) * a.hq + h0 + (col < nh ? col : 0)) * D;
    q8 raw[KK], own[2];
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) raw[kk] = *reinterpret_cast<const q8 *>(qp + 32 * kk + 8 * grp);
    if constexpr (I8) {
        const int at = 64 * (wave < QK ? wave : 0) + 16 * grp;
        own[0] = *reinterpret_cast<const q8 *>(qp + at);
        own[1] = *reinterpret_cast<const q8 *>(qp + at + 8);
    }

    // ---- one step's loads.  Tokens past the end are read from the last token
    // (K) or the last run (V), and masked below.  The pages of a lane's runs are
    // looked up a step ahead: K's run is that of its row, V's that of its
    // slots.  A page that does not exist: page 0 is read, and the rows end NaN.
    const int last = end - 1, last_run = last & ~(RUN - 1);
    const auto real = [&](int tok) { return WIN && tok >= win.sunk ? tok + win.gap : tok; };
    // (WIN: without branches; of those that && makes here, the compiler lost the
    // selected value)
    const uint32_t hole_size = win.hole_end > win.hole ? win.hole_end - win.hole : 0;
    const auto hidden = [&](bool tail, int tok) -> bool {
        if constexpr (WIN)
            return tail & ((tok >= end) | (static_cast<uint32_t>(tok - win.hole) < hole_size));
        else
            return tail && tok >= end;
    };
    const int32_t *table = a.table + static_cast<int64_t>(b) * a.max_pages;
    bool bad = bad_len;
    auto page_of = [&](int tok) {
        const int32_t pg = table[real(tok < last ? tok : last) >> page_shift];
        return pg;
    };
    auto checked = [&](int32_t pg) {
        const bool is = pg >= 0 && pg < a.n_pages;
        bad |= !is;
        return is ? pg : 0;
    };
    const char *kp = static_cast<const char *>(a.k_pages), *vp = static_cast<const char *>(a.v_pages);
    auto load_k = [&](int base, int32_t pg, at_u32x4 (&r)[NL]) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            int tok = base + RUN * (col >> 2) + 4 * t + (col & 3);
            tok = tok < last ? tok : last;
            const int64_t cell = ((static_cast<int64_t>(pg) * a.hkv + kh) << page_shift) + (real(tok) & page_mask);
            const char *src = kp + cell * (D * static_cast<int64_t>(sizeof(C))) + 16 * grp;
#pragma unroll
            for (int i = 0; i < LPT; ++i) r[t * LPT + i] = *reinterpret_cast<const at_u32x4 *>(src + 64 * i);
        }
    };
    auto run_of = [&](int base) {
        const int tok = base + RUN * grp;
        return real(tok < last_run ? tok : last_run);
    };
    auto load_v = [&](int base, int32_t pg, at_u32x4 (&r)[NL]) {
        const int64_t pgh = static_cast<int64_t>(pg) * a.hkv + kh;
        const char *src = vp + (((pgh * D + col) << page_shift) + (run_of(base) & page_mask)) * static_cast<int64_t>(sizeof(C));
        const int64_t stride = (static_cast<int64_t>(16) << page_shift) * sizeof(C);
#pragma unroll
        for (int i = 0; i < NL; ++i) r[i] = *reinterpret_cast<const at_u32x4 *>(src + i * stride);
    };
    auto load_steps = [&](const float *steps, int base, int32_t pg, at_f32x4 (&r)[NT]) {
        const int64_t cell = ((static_cast<int64_t>(pg) * a.hkv + kh) << page_shift) + (run_of(base) & page_mask);
#pragma unroll
        for (int t = 0; t < NT; ++t) r[t] = *reinterpret_cast<const at_f32x4 *>(steps + cell + 4 * t);
    };

    // ---- queries: B operand, column = head, k = 8 consecutive dimensions
    // (int8: dimension 64 p + 16 grp + 8 s of steps 2 p + s, the bytes a lane
    // loads at once; else 32 kk + 8 grp)
    float c = a.scale * kLog2e, far = 1.0f;  // scores in units of log2
    x8 qf[I8 ? 1 : QK][NQ];  // (int8: the digits stay in LDS)
    auto make_queries = [&] {
        int shift = 0;  // the queries enter times 2^shift
        if constexpr (I8 || (std::is_same<T, _Float16>::value && std::is_same<QT, float>::value)) {
            // the head's largest magnitude, whatever it is, brought to [2^14, 2^15)
            // (fp16 terms: what the third leaves is then 2^-39 of it) or below
            // 2^(8 NQ - 2) (digits)
            uint32_t mx = 0;  // of the bit patterns: NaN and infinity last
#pragma unroll
            for (int kk = 0; kk < KK; ++kk)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float x = static_cast<float>(raw[kk][j]);
                    const uint32_t u = __builtin_bit_cast(uint32_t, x) & 0x7fffffffu;
                    mx = mx > u ? mx : u;
                }
            mx = max(mx, static_cast<uint32_t>(__shfl_xor(static_cast<int>(mx), 16, 64)));
            mx = max(mx, static_cast<uint32_t>(__shfl_xor(static_cast<int>(mx), 32, 64)));
            const int e = __builtin_amdgcn_frexp_expf(__builtin_bit_cast(float, mx)) - 1;
            shift = (I8 ? 8 * NQ - 3 : 14) - e;
            if constexpr (I8) {
                // Products of digits and codes are whole numbers below 2^45.  c
                // comes first and a step (below 2^122) second, so c keeps what
                // makes the first factor neither overflow nor lose bits, and
                // `far` the rest of a power of two beyond that (none for scales
                // and queries of ordinary size).
                const int all = __builtin_amdgcn_frexp_expf(c) - shift, here = min(max(all, -125), 80);
                c = ldexpf(__builtin_amdgcn_frexp_mantf(c), here);
                far = ldexpf(1.0f, min(max(all - here, -126), 127));
            } else
                // finite, or it would make a NaN of a key of zeros: scores that
                // are not zero are then past 2^79 either way
                c = fminf(ldexpf(c, -shift), 3.4028235e38f);
            if (mx >= 0x7f800000u) c = __builtin_nanf("");  // a NaN or an infinity in the query
        }
        // (bf16 terms have fp32's exponents and are taken as they are, down to
        // 2^-133: to look for heads near that and scale them took 0.13 us of the
        // 4.73 of a sequence of 77 tokens)
        if constexpr (I8) {
            // the waves share the work: operand kk by wave kk, through LDS
            static_assert(QK <= kDecWaves, "an operand for each wave at most");
            at_i32x4 *shared = reinterpret_cast<at_i32x4 *>(lds);
            if (wave < QK) {
                at_i32x4 dig[NQ];
#pragma unroll
                for (int n = 0; n < NQ; ++n) dig[n] = at_i32x4{0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    int v = static_cast<int>(rintf(ldexpf(static_cast<float>(own[j >> 3][j & 7]), shift)));
#pragma unroll
                    for (int n = 0; n < NQ; ++n) {
                        dig[n][j >> 2] |= (v & 255) << (8 * (j & 3));
                        v = (v - static_cast<int8_t>(v)) >> 8;
                    }
                }
#pragma unroll
                for (int n = 0; n < NQ; ++n) shared[(wave * NQ + n) * 64 + lane] = dig[n];
            }
        } else {
#pragma unroll
            for (int kk = 0; kk < QK; ++kk) {
                float x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    x[j] = static_cast<float>(raw[kk][j]);
                    if constexpr (std::is_same<T, _Float16>::value) x[j] = ldexpf(x[j], shift);
                }
                split_terms<T, NQ>(x, qf[kk]);
            }
        }
    };

    // ---- the first step's loads, ahead of the queries' conversion (in the same
    // branch: behind it the compiler would wait for these loads as well)
    at_u32x4 kr[NL], vr[NL];
    at_f32x4 ks[NT], vs[NT];
    int base = begin + wave * TS;
    int32_t kpage = 0, vpage = 0;
    if (base < end) {
        kpage = page_of(base + RUN * (col >> 2));
        vpage = page_of(base + RUN * grp);
        const int32_t k0 = checked(kpage), v0 = checked(vpage);
        load_k(base, k0, kr);
        if constexpr (I8) load_steps(a.k_steps, base, v0, ks);
        if constexpr (I8) load_steps(a.v_steps, base, v0, vs);
        load_v(base, v0, vr);
        kpage = page_of(base + kDecWaves * TS + RUN * (col >> 2));
        vpage = page_of(base + kDecWaves * TS + RUN * grp);
        make_queries();
    } else if (I8)
        make_queries();
    // not __syncthreads: it would wait for the first K and V
    if constexpr (I8) asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    const bool any_far = I8 && __ballot(far != 1.0f) != 0;
    // fp16 weights, and sums, are 2^14 times themselves: small ones (many tokens
    // beside one that takes nearly all) would fall below fp16's smallest step,
    // 2^-24, otherwise.  bf16 weights, which have fp32's exponents, 2^-22 times
    // themselves: the sum over the 2^22 tokens that a sequence may have is then
    // in fp32's range whenever the values are.  (A product of its own: in the
    // exponent it costs the weights the low bits of the sum there: fp32
    // queries over 77 tokens are off by 4.9e-7 of the result then, 3.0e-7 so.)
    constexpr float kLift = I8 ? 1.0f : std::is_same<C, _Float16>::value ? 0x1p14f : 0x1p-22f;
    const at_f32x4 zero4 = {0.0f, 0.0f, 0.0f, 0.0f};
    at_f32x4 o[D / 16];
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[i] = zero4;
    float m = -__builtin_inff(), l = 0.0f;
    // int8: weights times steps enter in units of 2^(wexp - 14), wexp such that
    // they are below 2^14 in fp16; o is in these units
    int wexp = -112;

    for (; base < end; base += kDecWaves * TS) {
        const int next = base + kDecWaves * TS;
        // ---- scores: tile t, register i of lane: token base + RUN grp + 4 t + i, head col
        at_f32x4 s[NT];
        if constexpr (I8) {
            // digit by digit from the highest, each read from LDS anew: kept
            // in registers they make the kernel spill
            uint32_t place = lane;
            asm volatile("" : "+v"(place));
            const at_i32x4 *digits = reinterpret_cast<const at_i32x4 *>(lds) + place;
#pragma unroll
            for (int n = NQ - 1; n >= 0; --n) {
                at_i32x4 dig[QK];
#pragma unroll
                for (int kk = 0; kk < QK; ++kk) dig[kk] = digits[(kk * NQ + n) * 64];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    at_i32x4 acc = {0, 0, 0, 0};
#pragma unroll
                    for (int kk = 0; kk < QK; ++kk)
                        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(at_i32x4, kr[t * LPT + kk]), dig[kk],
                                                                    acc, 0, 0, 0);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float x = static_cast<float>(acc[i]);
                        s[t][i] = n == NQ - 1 ? x : fmaf(s[t][i], 256.0f, x);
                    }
                }
            }
        } else {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                s[t] = zero4;
#pragma unroll
                for (int kk = 0; kk < KK; ++kk)
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
                        s[t] = Op16<T>::mfma16(__builtin_bit_cast(x8, kr[t * LPT + kk]), qf[kk][n], s[t]);
            }
        }
        if constexpr (I8) {
#pragma unroll
            for (int t = 0; t < NT; ++t) s[t] = s[t] * c * ks[t];
            if (any_far) {
#pragma unroll
                for (int t = 0; t < NT; ++t) s[t] *= far;
            }
        }
        const int32_t kn = checked(kpage), vn = checked(vpage);
        if (next < end) {
            load_k(next, kn, kr);
            if constexpr (I8) load_steps(a.k_steps, next, vn, ks);
            kpage = page_of(next + kDecWaves * TS + RUN * (col >> 2));
            vpage = page_of(next + kDecWaves * TS + RUN * grp);
        }
        bool tail = base + TS > end;  // something is masked
        if constexpr (WIN) tail |= (base < win.hole_end) & (base + TS > win.hole);
        float top = -__builtin_inff();
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (!I8) s[t][i] *= c;
                if (hidden(tail, base + RUN * grp + 4 * t + i)) s[t][i] = -__builtin_inff();
                top = fmaxf(top, s[t][i]);
            }
        top = lane_pair_max<32>(lane_pair_max<16>(top));
        // a larger maximum rescales what is there (all lanes of a head alike)
        if (__ballot(top > m) != 0) {
            const float mn = fmaxf(m, top);
            float f = m == mn ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
            l *= f;
            if constexpr (I8) {
                // the units come down with the weights, or a large step whose
                // weight has become nothing would keep the resolution coarse
                int down = static_cast<int>(__builtin_bit_cast(uint32_t, f) >> 23) - 126;  // f < 2^down
                down = down > 0 ? 0 : down < -112 - wexp ? -112 - wexp : down;
                f *= pow2(-down);
                wexp += down;
            }
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
                float e = __builtin_amdgcn_exp2f(s[t][i] - ms) * kLift;
                l += e;
                if constexpr (I8) e *= hidden(tail, base + RUN * grp + 4 * t + i) ? 0.0f : vs[t][i];
                p[4 * t + i] = e;
            }
        if constexpr (I8) {
            float top = 0.0f;
#pragma unroll
            for (int j = 0; j < TS / 4; ++j) top = fmaxf(top, p[j]);
            top = lane_pair_max<32>(lane_pair_max<16>(top));
            int e = static_cast<int>(__builtin_bit_cast(uint32_t, top) >> 23) - 126;  // 2^e > top
            e = e > 126 ? 126 : e;
            if (e > wexp) {
                const float f = pow2(wexp - e > -126 ? wexp - e : -126);
#pragma unroll
                for (int i = 0; i < D / 16; ++i) o[i] *= f;
                wexp = e;
            }
            const float unit = pow2(14 - wexp);
#pragma unroll
            for (int j = 0; j < TS / 4; ++j) p[j] *= unit;
        }
        // ---- O^T += V^T P^T, slot j of step u: token base + RUN grp + 8 u + j
        if (tail) {
            // what lies past the end may hold anything; zero weights do not silence a NaN
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                constexpr int PER = 4 / sizeof(C);  // tokens per dword
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int left = end - (base + RUN * grp + PER * w);
                    uint32_t keep = left >= PER ? 0xffffffffu
                                    : left <= 0 ? 0u
                                                : (1u << (8 * static_cast<int>(sizeof(C)) * left)) - 1u;
                    if constexpr (WIN) {
                        constexpr uint32_t kOne = (1ull << (8 * sizeof(C))) - 1;
#pragma unroll
                        for (int t = 0; t < PER; ++t)
                            keep &= hidden(true, base + RUN * grp + PER * w + t) ? ~(kOne << (8 * static_cast<int>(sizeof(C)) * t)) : ~0u;
                    }
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
                    asm volatile("" : "+v"(w));  // keeps the codes packed up to here
                    vf = codes_to_f16(w[0], w[1]);
                } else
                    vf = __builtin_bit_cast(x8, vr[i]);
#pragma unroll
                for (int n = 0; n < NP; ++n) o[i] = Op16<T>::mfma16(vf, pf[n], o[i]);
                if constexpr (I8)
                    if ((i & 1) == 1) __builtin_amdgcn_sched_barrier(0);  // or every code is converted up front
            }
        }
        if (next < end) {
            if constexpr (I8) load_steps(a.v_steps, next, vn, vs);
            load_v(next, vn, vr);
        }
    }
    l = lane_pair_sum<32>(lane_pair_sum<16>(l));
    if constexpr (I8) {
        // out of the units, and divided by a power of two next to the weights'
        // sum: with the largest steps a sum may be past fp32's range when no
        // mean is
        const int down = wexp - 14 - sum_exponent(l);
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] = ldexpf(o[i][j], down);
    }

    // ---- join the four waves: rows in LDS [wave][head][D + 4]
    if constexpr (I8) __syncthreads();  // where the digits were
    float *rows = reinterpret_cast<float *>(lds);
    if (__ballot(bad) != 0) l = __builtin_nanf("");
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
    for (int i = threadIdx.x; i < nh * (D / 4); i += kDecThreads) {
        const int h = i / (D / 4), e = (i % (D / 4)) * 4;
        float M = wm[0][h];
#pragma unroll
        for (int w = 1; w < kDecWaves; ++w) M = fmaxf(M, wm[w][h]);
        const float Ms = M == -__builtin_inff() ? 0.0f : M;
        // (int8: the rows are below the waves' sums by a power of two)
        float L = 0.0f, f[kDecWaves];
#pragma unroll
        for (int w = 0; w < kDecWaves; ++w) {
            f[w] = __builtin_amdgcn_exp2f(wm[w][h] - Ms);
            L += f[w] * wl[w][h];
        }
        const float inv = whole ? 1.0f / L : I8 ? ldexpf(1.0f, -sum_exponent(L)) : 1.0f;
        at_f32x4 r = zero4;
#pragma unroll
        for (int w = 0; w < kDecWaves; ++w)
            r += (I8 ? ldexpf(f[w], sum_exponent(wl[w][h])) * inv : f[w] * inv) * *reinterpret_cast<const at_f32x4 *>(rows + (w * nh + h) * (D + 4) + e);
        if (whole) {
            if (len == 0) r = zero4;
            store4(static_cast<QT *>(a.out) + (static_cast<int64_t>(b) * a.hq + h0 + h) * D + e, r);
        } else {
            const int64_t slot = piece * a.hq + h0 + h;
            *reinterpret_cast<at_f32x4 *>(a.part_rows + slot * D + e) = r;
            if (e == 0) {
                a.part_ml[slot * 2] = M;
                a.part_ml[slot * 2 + 1] = L;
            }
        }
    }
}

// Joins the pieces of a sequence that was cut: one workgroup
// per (query head, sequence), its D / 4 lanes wide groups taking every n-th
// piece, then a sum over the groups in LDS.
template <typename QT, int D, bool WIN>
__global__ void __launch_bounds__(256) k_attn_join(DecodeArgs a)
{
    constexpr int LPR = D / 4, G = 256 / LPR;
    __shared__ float wgt[2 * kMaxShares];
    __shared__ float red[4];
    __shared__ at_f32x4 sums[G][LPR];
    const int64_t b = blockIdx.y, h = blockIdx.x;
    const LaneLens lens(a);
    const int per = piece_steps<WIN>(a, lens);
    const auto pieces = [&](int len) { return pieces_of(decode_steps(tokens_read<WIN>(a, len), a.max_len), per); };
    const int n = pieces(b < 64 ? __builtin_amdgcn_readlane(lens.first, static_cast<int>(b)) : a.lens[b]);
    if (n == 1) return;
    const int64_t before = lens.sum(a, b, pieces);
    auto slot = [&](int i) { return (before + i) * a.hq + h; };
    float M = -__builtin_inff();
    for (int i = threadIdx.x; i < n; i += 256) M = fmaxf(M, a.part_ml[slot(i) * 2]);
    M = wave_max(M);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = M;
    __syncthreads();
    M = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    if (M == -__builtin_inff()) M = 0.0f;
    __syncthreads();
    float L = 0.0f;
    for (int i = threadIdx.x; i < n; i += 256) {
        const float w = __builtin_amdgcn_exp2f(a.part_ml[slot(i) * 2] - M);
        const float l = w * a.part_ml[slot(i) * 2 + 1];
        wgt[i] = a.lowered ? ldexpf(w, sum_exponent(a.part_ml[slot(i) * 2 + 1])) : w;
        L += l;
    }
    L = wave_sum(L);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = L;
    __syncthreads();
    const float inv = 1.0f / ((red[0] + red[1]) + (red[2] + red[3]));
    const int g = threadIdx.x / LPR, x = threadIdx.x % LPR;
    at_f32x4 r = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
    for (int i = g; i < n; i += G) r += wgt[i] * inv * *reinterpret_cast<const at_f32x4 *>(a.part_rows + slot(i) * D + 4 * x);
    sums[g][x] = r;
    __syncthreads();
    if (g == 0) {
#pragma unroll
        for (int i = 1; i < G; ++i) r += sums[i][x];
        store4(static_cast<QT *>(a.out) + (b * a.hq + h) * D + 4 * x, r);
    }
}

template <bool WIN, typename C, typename QT, int D, int NQ, int NP>
hipError_t decode_launch(const DecodePlan &p, const DecodeArgs &a, int64_t batch, hipStream_t s)
{
    static std::atomic<uint64_t> lds_done{0};
    const auto kernel = k_attn_decode<C, QT, D, NQ, NP, WIN>;
    // the waves' rows at the end; int8: the queries' digits before
    constexpr int kMaxLds = kDecWaves * kDecHeads * (D + 4) * 4;
    constexpr int kDigits = std::is_same<C, int8_t>::value ? D / 64 * NQ * 1024 : 0;
    static_assert(kDigits <= kMaxLds, "the digits fit");
    const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void *>(kernel), kMaxLds, lds_done);
    if (e != hipSuccess) return e;
    const int group = a.hq / a.hkv;
    const int rows = kDecWaves * (group < kDecHeads ? group : kDecHeads) * (D + 4) * 4;
    const int lds = rows > kDigits ? rows : kDigits;
    hipLaunchKernelGGL(kernel,
                       dim3(static_cast<uint32_t>(p.pieces * a.hkv * a.hblocks)), dim3(kDecThreads), lds, s, a);
    if (p.join)
        hipLaunchKernelGGL((k_attn_join<QT, D, WIN>), dim3(static_cast<uint32_t>(a.hq), static_cast<uint32_t>(batch)),
                           dim3(256), 0, s, a);
    return hipGetLastError();
}

template <bool WIN, typename C, typename QT, int NQ, int NP>
hipError_t decode_d(const DecodePlan &p, const DecodeArgs &a, int64_t batch, int d, hipStream_t s)
{
    return d == 64 ? decode_launch<WIN, C, QT, 64, NQ, NP>(p, a, batch, s)
                   : d == 128 ? decode_launch<WIN, C, QT, 128, NQ, NP>(p, a, batch, s)
                              : decode_launch<WIN, C, QT, 256, NQ, NP>(p, a, batch, s);
}

template <bool WIN>
hipError_t decode_types(const DecodePlan &p, const DecodeArgs &a, int q_type, int cache_type, int d, hipStream_t s)
{
    if (cache_type == PTQ1_BF16)
        return q_type == PTQ1_F32 ? decode_d<WIN, __bf16, float, 3, 3>(p, a, a.batch, d, s)
                                  : decode_d<WIN, __bf16, __bf16, 1, 2>(p, a, a.batch, d, s);
    if (cache_type == PTQ1_F16)
        return q_type == PTQ1_F32 ? decode_d<WIN, _Float16, float, 3, 2>(p, a, a.batch, d, s)
                                  : decode_d<WIN, _Float16, _Float16, 1, 2>(p, a, a.batch, d, s);
    return q_type == PTQ1_F32 ? decode_d<WIN, int8_t, float, 4, 3>(p, a, a.batch, d, s)
           : q_type == PTQ1_F16 ? decode_d<WIN, int8_t, _Float16, 3, 2>(p, a, a.batch, d, s)
                                : decode_d<WIN, int8_t, __bf16, 3, 2>(p, a, a.batch, d, s);
}

}  // namespace

DecodePlan decode_plan(int64_t batch, int32_t hq, int32_t hkv, int32_t d, int64_t max_len, bool windowed)
{
    DecodePlan p;
    const int64_t group = hq / hkv, hgroups = hkv * ((group + kDecHeads - 1) / kDecHeads);
    const int64_t each = max_len > 0 ? (max_len + kStep - 1) / kStep : 1;  // steps of a sequence at its bound
    // two workgroups of four waves a CU; of 256-wide heads' registers, one
    int64_t shares = (d == 256 ? 256 : 512) / hgroups;
    if (shares < 1) shares = 1;
    if (shares > kMaxShares) shares = kMaxShares;
    p.shares = static_cast<int32_t>(shares);
    const int64_t want = wanted_pieces(batch, shares);
    // every sequence has a step, so a piece has at least so many: large
    // batches of short sequences are not cut (1024 of 512 tokens: 455 us with
    // the search for their pieces and the join's launch, 364 without)
    p.join = each > (batch + want - 1) / want;
    if (windowed && p.join && each <= 8) {
        // Windows are of one length, and mostly short: is the time of the steps
        // that cutting saves (1.9 us each, 3.6 of 256-wide heads) more than it
        // costs?  One sequence, 40 heads over 8 of 128: windows of 256, 700, 1024
        // and 2000 tokens 11.9, 12.3, 12.1, 12.1 us cut and 8.0, 11.0, 14.3, 22.0
        // uncut; 32 of 1024 and 2000 28.6, 45.4 and 22.6, 39.3; 200 of 700 over
        // int8, 64-wide, 39.6 and 16.5.
        const int64_t groups = batch * hgroups, slots = d == 256 ? 256 : 512;
        const int64_t saved = each * ((groups + slots - 1) / slots) - (each * groups + slots - 1) / slots;
        p.join = static_cast<double>(saved) * (d == 256 ? 3.6 : 1.9) > 6.0 + static_cast<double>(batch < 64 ? batch : 64) / 4;
    }
    p.pieces = p.join && want + batch < each * batch ? want + batch : p.join ? each * batch : batch;
    if (p.join) {
        p.rows_floats = static_cast<size_t>(p.pieces) * hq * d;
        p.part_floats = p.rows_floats + static_cast<size_t>(p.pieces) * hq * 2;
    }
    return p;
}

hipError_t launch_attn_decode(const DecodePlan &p, const void *q, int q_type, int64_t batch, int32_t hq,
                              const ptq1_kv_cache &c, const int32_t *table, int64_t max_pages, const int32_t *lens,
                              int64_t max_len, int32_t window, int32_t sinks, float scale, void *out, float *part,
                              hipStream_t s)
{
    const int32_t group = hq / c.n_kv_heads;
    const DecodeArgs a{q, hq, c.n_kv_heads, (group + kDecHeads - 1) / kDecHeads, c.k_pages, c.v_pages, c.k_steps,
                       c.v_steps, c.n_pages, __builtin_ctz(static_cast<unsigned>(c.page_size)), table, max_pages, lens,
                       batch, max_len, p.shares, p.join, c.dtype == PTQ1_I8, scale, out, part, part + p.rows_floats,
                       window, sinks};
    return window > 0 ? decode_types<true>(p, a, q_type, c.dtype, c.head_dim, s)
                      : decode_types<false>(p, a, q_type, c.dtype, c.head_dim, s);
}

}  // namespace ptq1
