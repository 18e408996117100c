// attn_chunk.hip -- attention of the last tokens of every sequence over the
// paged cache that holds them already (ptq1_attn_chunk).
//
//   out_i = sum_j p_ij V_j / sum_j p_ij,  p_ij = exp2(t_ij - m_i),
//   t_ij = scale log2(e) (q_i . K_j),     j over the keys that query i sees
//
// in one pass over the keys with a running maximum m_i.  Many rows are bounded
// by the matrix cores, few by the cache's bytes.
//
// Rows.  As in attn_prompt.hip: the query rows of a kv head are its group's
// heads of every token, a tile is 128 of them (32 a wave; of 256-wide heads a
// pair of waves), and steps are 64 keys, in two LDS buffers, through 32x32x16
// MFMA with one query row per lane.
//
// Layout.  K pages are token-major, V pages dimension-major, and both lie in
// LDS as in memory, so both A operands are 16 contiguous bytes per lane and
// nothing is transposed.  The rows of a score tile are assigned to tokens so
// that the score registers of a lane are eight consecutive tokens: exactly the
// k-slots of its V operand, so P needs no exchange.
//
// Pages.  A page holds whole runs of 16 tokens, of which a step has four.  A
// wave instruction copies pieces of one run of K (its page is in a scalar), and
// of V of all four (the lane picks its own).  The pages of a step are looked up
// a step before they are needed, two before they are read.
//
// int8 caches.  16-bit pieces cannot come from memory, so a step's codes pass
// through registers and become 16-bit operands in LDS, exactly, once for all
// waves: K's in the queries' type, V's in fp16.  K's step, with the scale,
// multiplies the scores; V's multiplies the weights, which then enter the second
// product in units of a power of two of their row.
//
// Measured (matrix work differs by up to 10% from card to card; these are the
// faster ones).  4096 tokens behind 28000 (40 heads over 8 of 128, bf16): 1480 to
// 1580 us, 980 to 1050 TFLOP/s; matrix cores 51% busy, vector units 54%.  8 x 256 to
// 512 tokens behind 6000 to 12000 over int8: 766 to 780 us, 780 TFLOP/s, the vector units
// (56%; the codes of a step cost 160 of 630 instructions of a wave) and LDS (stores
// of codes: on the layout of the 16-bit tiles they met two by two, 3% more).  4 x 350
// to 700 tokens behind 2000 to 4000, 256-wide heads, fp16: 233 us, 650 TFLOP/s, eight
// waves in step through three barriers (matrix cores 29%).  3 x 1000 to 2000 tokens
// in windows of 1024 (32 heads over 8 of 128): 131 us, 640 TFLOP/s: of a tile's 18
// steps three are on a border, and 158 tiles of a kv head run on 64 places.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "ptq1_attn_chunk.h"

namespace ptq1 {
namespace {

constexpr int kAhead = 4;  // K reads ahead of their products
constexpr int chunk_waves(int d) { return d == 256 ? 8 : 4; }

// The 16-byte piece p of row r of a tile in LDS lies at piece p ^ swizzle of
// that row: 16 rows at one piece spread over all banks.  (V's rows are
// dimensions, of 64 tokens: as K's of 64-wide heads.)
template <int W>
__device__ __forceinline__ int swizzle(int r)
{
    return W >= 128 ? r & 15 : (r >> 1) & 7;
}
// The byte offset of piece `half` of row r; piece 2 i + half is at it ^ kPair i.
//
// Of int8 caches a thread brings 16 codes, which are two pieces: the first
// pieces of a row fill its first half and the second ones the other, and the
// swizzle's bits are turned by one, so that 16 threads write 16 pieces on all
// banks too.
template <typename C, int W>
__device__ __forceinline__ int row_of(int r, int half)
{
    if constexpr (std::is_same<C, int8_t>::value) {
        const int x = swizzle<W>(r);
        return (r * (2 * W) + 16 * ((x >> 1) | (x & 1) * (W >= 128 ? 8 : 4))) ^ (W * half);
    }
    return (r * (2 * W) + 16 * swizzle<W>(r)) ^ (16 * half);
}
template <typename C>
constexpr int kPair = std::is_same<C, int8_t>::value ? 16 : 32;
// The value, which the compiler then makes anew where it is used: what every
// step makes of a lane's place it would keep in registers through all of them.
__device__ __forceinline__ int not_kept(int v)
{
    asm volatile("" : "+v"(v));
    return v;
}
// A step's buffers in LDS; int8 caches: with the steps of its tokens, K's times
// scale and log2 e, V's in units of 2^*unit, which none exceeds.
template <typename QT, typename T>
struct ChunkBuffer {
    QT *k;
    T *v;
    float *ks, *vs;
    int *unit;
};

// A lane's share of bringing a step's keys and values into LDS.
template <typename C, typename QT, int D>
struct ChunkStaging {
    static constexpr bool I8 = std::is_same<C, int8_t>::value;
    typedef typename WeightOf<C>::type T;
    typedef ChunkBuffer<QT, T> Buffer;
    static constexpr int W = chunk_waves(D), NT = 64 * W;
    static constexpr int NK = BN * D * static_cast<int>(sizeof(C)) / (16 * NT);  // 16-byte loads of a thread, for K and for V
    const char *kp, *vp;   // of this kv head
    const float *ksp, *vsp;
    uint32_t page_bytes, page_cells;
    int page_shift, mask;
    at_u32x4 kr[I8 ? NK : 1], vr[I8 ? NK : 1];
    float step = 0.0f, c;
    int lo, reach, sunk, unit = -126;

    __device__ __forceinline__ ChunkStaging(const ChunkArgs &a, const ChunkTile &t)
        : page_shift(a.page_shift), mask((1 << a.page_shift) - 1), c(a.scale * kLog2e), lo(t.c.lo), reach(t.c.reach), sunk(t.c.sunk)
    {
        const int kh = t.kh;
        page_cells = static_cast<uint32_t>(a.hkv) << page_shift;
        page_bytes = page_cells * (D * static_cast<uint32_t>(sizeof(C)));
        const int64_t first = (static_cast<int64_t>(kh) << page_shift) * (D * static_cast<int64_t>(sizeof(C)));
        kp = static_cast<const char *>(a.k_pages) + first;
        vp = static_cast<const char *>(a.v_pages) + first;
        ksp = a.k_steps + (static_cast<int64_t>(kh) << page_shift);
        vsp = a.v_steps + (static_cast<int64_t>(kh) << page_shift);
    }

    // 16-bit caches: straight into LDS
    __device__ __forceinline__ void copy(const ChunkPages &p, int n0, const Buffer &to) const
    {
        static_assert(!I8, "16 bits");
        constexpr int P = D / 8, RK = 64 / P;  // pieces of a row of K, rows of an instruction
        const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            const int r0 = (i * W + wave) * RK, r = (r0 & 15) + lane / P;  // (a run's row: the swizzle goes by it)
            const char *base = kp + static_cast<uint64_t>(page_bytes) * static_cast<uint32_t>(p.of(r0 >> 4)) +
                               ((n0 + (r0 & ~15)) & mask) * (2 * D);
            copy_to_lds(base, 16 * 2 * D, r * (2 * D) + 16 * ((lane % P) ^ swizzle<D>(r)), to.k + (i * W + wave) * 512);
        }
        // V: the piece of a lane is the same in every instruction
        const int d0 = wave * 8 + (lane >> 3), piece = (lane & 7) ^ swizzle<BN>(d0);
        const char *src = vp + static_cast<uint64_t>(page_bytes) * static_cast<uint32_t>(p.of(piece >> 1)) +
                          2 * ((static_cast<uint32_t>(d0) << page_shift) + ((n0 + 8 * piece) & mask));
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)src, (lds_void *)(to.v + (i * W + wave) * 512), 16, 0, 0);
            src += static_cast<uint32_t>(2 * 8 * W) << page_shift;
        }
    }

    // int8 caches: into registers ...
    __device__ __forceinline__ void load(const ChunkPages &p, int n0)
    {
        static_assert(I8, "8 bits");
        constexpr int L = D / 16;  // loads of a row of K
        const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            const int r0 = (i * W + wave) * (64 / L), r = (r0 & 15) + lane / L;
            const char *base = kp + static_cast<uint64_t>(page_bytes) * static_cast<uint32_t>(p.of(r0 >> 4)) +
                               ((n0 + (r0 & ~15)) & mask) * D;
            kr[i] = *reinterpret_cast<const at_u32x4 *>(base + (r * D + 16 * (lane % L)));
        }
        const char *src = vp + static_cast<uint64_t>(page_bytes) * static_cast<uint32_t>(p.of(lane & 3)) +
                          ((static_cast<uint32_t>(threadIdx.x >> 2) << page_shift) + ((n0 + 16 * (lane & 3)) & mask));
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            vr[i] = *reinterpret_cast<const at_u32x4 *>(src);
            src += static_cast<uint32_t>(NT / 4) << page_shift;
        }
        if (wave < 2)
            step = (wave == 0 ? ksp : vsp)[static_cast<uint64_t>(page_cells) * static_cast<uint32_t>(p.of(lane >> 4)) + ((n0 + lane) & mask)];
    }
    // ... and as 16-bit operands into LDS: K's in the queries' type, V's in fp16
    __device__ __forceinline__ void store(int n0, const Buffer &to)
    {
        constexpr int L = D / 16;
        const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int k_at = not_kept(row_of<C, D>(wave * (64 / L) + lane / L, 0) ^ (16 * (lane % L)));
        const int v_at = not_kept(row_of<C, BN>(static_cast<int>(threadIdx.x >> 2), 0) ^ (16 * (lane & 3)));
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            typedef typename Op16<QT>::x8 k8;
            char *at = reinterpret_cast<char *>(to.k) + i * W * 64 * 32;  // (64 rows or 16 on: the swizzle is the same)
            *reinterpret_cast<k8 *>(at + k_at) = codes_to<QT>(kr[i][0], kr[i][1]);
            *reinterpret_cast<k8 *>(at + (k_at ^ D)) = codes_to<QT>(kr[i][2], kr[i][3]);
            __builtin_amdgcn_sched_barrier(0);  // (or all codes are converted before the first are stored)
        }
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            char *at = reinterpret_cast<char *>(to.v) + i * (NT / 4) * (2 * BN);
            *reinterpret_cast<f16x8 *>(at + v_at) = codes_to_f16(vr[i][0], vr[i][1]);
            *reinterpret_cast<f16x8 *>(at + (v_at ^ BN)) = codes_to_f16(vr[i][2], vr[i][3]);
            __builtin_amdgcn_sched_barrier(0);
        }
        // (the product is finite, or it would make a NaN of a sum of zero)
        if (wave == 0) to.ks[lane] = step != step ? step : fminf(step * c, 3.4028235e38f);
        if (wave == 1) {
            const int key = n0 + lane;
            const bool some = (key < reach) & ((key >= lo) | (key < sunk));
            const float top = wave_max(some ? step : 0.0f);
            const int e = __builtin_amdgcn_readfirstlane(static_cast<int>(__builtin_bit_cast(uint32_t, top) >> 23) - 126);  // 2^e above
            unit = unit_of_steps(unit, e);
            to.vs[lane] = ldexpf(step, -unit);
            if (lane == 0) *to.unit = unit;
        }
    }
};

// NaNs and infinities leave a V tile in LDS (zeros in their place); one of a key
// that some row sees is noted.  (Were those of other keys noted too, what lies
// behind a sequence's end would decide the time: 84 us for 13 behind 161 and 130
// keys, and with first tokens and a window's begin 2890 for 90.)  Most tiles have
// none, which the largest magnitude among a thread's values tells.
template <typename T, int D>
__device__ __forceinline__ void clean_values(T *v, int n0, const ChunkSteps &seen, ChunkNotes *notes)
{
    constexpr int NT = 64 * chunk_waves(D), N = BN * D / 8 / NT;
    at_u32x4 w[N];
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = *reinterpret_cast<const at_u32x4 *>(v + 8 * (i * NT + threadIdx.x));
    LargestHalf<T> most;
#pragma unroll
    for (int i = 0; i < N; ++i) most.of(w[i]);
    if (!most.non_finite()) return;
    // (a thread's pieces are of the same eight keys, as in ChunkStaging)
    const int piece = static_cast<int>(threadIdx.x & 7) ^ swizzle<BN>(static_cast<int>(threadIdx.x >> 3));
    const at_u32x4 halves = seen_halves(n0 + 8 * piece, seen.lo, seen.reach, seen.sunk);
    uint32_t gone = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const at_u32x4 was = w[i];
        if (clear_non_finite<T>(w[i])) *reinterpret_cast<at_u32x4 *>(v + 8 * (i * NT + threadIdx.x)) = w[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) gone |= (was[j] ^ w[i][j]) & halves[j];
    }
    if (gone == 0) return;
    atomicOr(&notes->odd_steps, step_bit(n0));
}

// The row's dimensions d0 + 32 i + 8 b + 4 half + e, finished: as they are, or
// as one part of several (the mean over its keys, their reference and sum).
template <typename QT, int N>
__device__ __forceinline__ void store_rows(const ChunkArgs &a, const ChunkTile &t, const ChunkRow &row, int at, int d, int d0,
                                           int half, const at_f32x16 (&o)[N], float m, float l)
{
    if (t.pieces == 1) {
        QT *dst = static_cast<QT *>(a.out) + ((static_cast<int64_t>(t.q0) + row.tok) * a.hq + row.head) * d + d0 + 4 * half;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < 16; j += 4)
                store4(dst + 32 * i + 2 * j, at_f32x4{o[i][j], o[i][j + 1], o[i][j + 2], o[i][j + 3]});
        return;
    }
    const int64_t slot = part_slot(a, t, at);
    float *dst = a.parts + slot * d + d0 + 4 * half;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 16; j += 4)
            store4(dst + 32 * i + 2 * j, at_f32x4{o[i][j], o[i][j + 1], o[i][j + 2], o[i][j + 3]});
    if (half == 0 && d0 == 0) {
        a.parts[a.rows_floats + slot * 2] = m;
        a.parts[a.rows_floats + slot * 2 + 1] = l;
    }
}

// A lane's row at the end: the mean over its keys, 1 / l times the sums of
// products (int8 caches: and out of their units), with what was left aside on
// the way.  A row that sees no key is zero; of a piece's keys a row may see
// none.
template <typename C, typename QT, int N>
__device__ __forceinline__ void finish(const ChunkArgs &a, const ChunkTile &t, const ChunkRow &row, const ChunkNotes &notes,
                                       int at, int d, int d0, int half, at_f32x16 (&o)[N], float m, float l, int unit)
{
    const bool none = row.seen.hi == 0 || (t.pieces > 1 && l == 0.0f);
    float f = none ? 0.0f : 1.0f / l;
    if (notes.bad != 0 && sees_bad_page(a, t, row)) l = f = __builtin_nanf("");
#pragma unroll
    for (int i = 0; i < N; ++i) {
        o[i] *= f;
        if constexpr (std::is_same<C, int8_t>::value) {
#pragma unroll
            for (int j = 0; j < 16; ++j) o[i][j] = ldexpf(o[i][j], unit);
        }
    }
    if constexpr (!std::is_same<C, int8_t>::value)
        if (notes.odd_steps != 0) add_odd_values<C, N>(a, t, row, notes, d, d0, half, o);
    if (row.is) store_rows<QT, N>(a, t, row, at, d, d0, half, o, m, l);
}

// The steps first .. last in pairs (a buffer each): in the inner loops those
// whose keys every row sees, and the others.
template <class F>
__device__ __forceinline__ void run_steps(const ChunkTile &t, const F &step)
{
    int i = t.first;
    const int whole = t.c.all_to < t.last ? t.c.all_to : t.last;
    while (i < t.last) {
        for (; i < t.last && (i < t.c.all_from || i + 2 > whole); i += 2) {
            step(std::true_type{}, std::false_type{}, i);
            if (i + 1 < t.last) step(std::true_type{}, std::true_type{}, i + 1);
        }
        for (; i + 2 <= whole; i += 2) {
            step(std::false_type{}, std::false_type{}, i);
            step(std::false_type{}, std::true_type{}, i + 1);
        }
    }
}

template <typename C, typename QT, int D>
__global__ void __launch_bounds__(64 * chunk_waves(D), 2) k_attn_chunk(ChunkArgs a)
{
    typedef typename WeightOf<C>::type T;
    typedef typename Op16<T>::x8 x8;
    typedef ChunkBuffer<QT, T> Buffer;
    constexpr bool I8 = std::is_same<C, int8_t>::value;
    constexpr int KT = BN / 32, DT = D / 32, KK = D / 16;

    // two buffers: separate objects, so that the copies into one need not have
    // ended before the other is read
    __shared__ __attribute__((aligned(16))) QT kt0[BN * D], kt1[BN * D];
    __shared__ __attribute__((aligned(16))) T vt0[BN * D], vt1[BN * D];
    __shared__ float steps[I8 ? 4 * BN : 1];
    __shared__ int step_units[2];
    __shared__ SeenKeys seen_of[kChunkRows];  // (in registers it would be in the way of the inner steps)
    __shared__ int lift_of[I8 ? kChunkRows : 1];
    __shared__ ChunkNotes notes;

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 31, half = lane >> 5;
    __shared__ ChunkTile tile_note;  // for the end: in registers it would be in the way meanwhile
    ChunkTile t;
    if (!chunk_tile<QT, D>(a, blockIdx.x, false, t)) return;
    if (threadIdx.x == 0) tile_note = t;
    const bool idle = t.row0 + 32 * wave >= t.rows;  // no row of this wave's is there
    ChunkPages pages(a, t);
    ChunkStaging<C, QT, D> staging(a, t);
    if (t.first < t.last) pages.find(step_key(t.c, t.first));
    const float c = a.scale * kLog2e;
    const ChunkRow first_row = chunk_row(a, t, t.row0 + 32 * wave + col);
    seen_of[32 * wave + col] = first_row.seen;
    const ChunkQuery<QT, D, false, I8> q(a, t, first_row, half);
    if constexpr (I8) lift_of[32 * wave + col] = q.lift;
    const bool lifted = I8 && __ballot(q.lift != 0) != 0;
    if (threadIdx.x == 0) notes = {0, 0};

    at_f32x16 o[DT];
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] = 0.0f;
    ChunkSoftmax<C, KT, 1> w;

    // One step, while the next one's keys and values arrive in the other buffers.
    auto step = [&](auto border, auto odd, int i) __attribute__((always_inline)) {
        constexpr bool BORDER = decltype(border)::value;  // some row may not see some key of the step
        constexpr bool ODD = decltype(odd)::value;
        const Buffer b{ODD ? kt1 : kt0, ODD ? vt1 : vt0, steps + (ODD ? 2 * BN : 0), steps + (ODD ? 3 * BN : BN), step_units + ODD};
        const Buffer next{ODD ? kt0 : kt1, ODD ? vt0 : vt1, steps + (ODD ? 0 : 2 * BN), steps + (ODD ? BN : 3 * BN), step_units + !ODD};
        const int n0 = step_key(t.c, i);
        if (i + 1 < t.last) {
            pages.use();
            if constexpr (I8)
                staging.load(pages, step_key(t.c, i + 1));
            else
                staging.copy(pages, step_key(t.c, i + 1), next);
        }
        pages.find(step_key(t.c, min(i + 2, t.last - 1)));  // (in no branch, at whose end the compiler would wait for it)
        SeenKeys seen{0, 0};
        if constexpr (BORDER) seen = seen_of[32 * wave + col];
        x8 pf[1][2 * KT];
        if (!idle) {
            at_f32x16 s[KT];
            const int k_row = not_kept(row_of<C, D>(token_of_row(col), half));
#pragma unroll
            for (int k = 0; k < KT; ++k) {
#pragma unroll
                for (int j = 0; j < 16; ++j) s[k][j] = 0.0f;
#pragma unroll
                for (int kk = 0; kk < KK; ++kk) {
                    typedef typename Op16<QT>::x8 k8;
                    const k8 kf = *reinterpret_cast<const k8 *>(reinterpret_cast<const char *>(b.k) + (k_row ^ (kPair<C> * kk)) + 32 * k * (2 * D));
                    s[k] = Op16<QT>::mfma32(kf, q.f[kk], s[k]);
                }
            }
            // the K reads run ahead of the products
            __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
            for (int k = 0; k < KT * KK - kAhead; ++k) {
                __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
            __builtin_amdgcn_sched_group_barrier(0x8, kAhead, 0);
            w.raise(w.top(BORDER, s, HiddenKeys(seen, t, n0), n0, half, c, [&](int k, int j) { return b.ks[w.key(k, j, half)]; }, lifted, [&] { return lift_of[32 * wave + col]; }), o, w.unit);
            if constexpr (I8) {
                if constexpr (BORDER) asm volatile("" : "+v"(seen.lo), "+v"(seen.hi));  // (or the masks of 64 keys are kept)
                w.products(BORDER, s, HiddenKeys(seen, t, n0), n0, half, [&](int k, int j) { return b.vs[w.key(k, j, half)]; }, *b.unit, pf, [&](float f) {
#pragma unroll
                    for (int d = 0; d < DT; ++d) o[d] *= f;
                });
            } else
                w.weights(s, c, pf);
        }
        if constexpr (BORDER && !I8) {
            // a zero weight would not keep a NaN or an infinity out of the rows
            // that do not see it: such values leave the tile and are given to
            // the rows that see them at the end
            clean_values<T, D>(b.v, n0, tile_note.c, &notes);
            __syncthreads();
        }
        if (!idle) {
            const int v_row = not_kept(row_of<C, BN>(col, half));
#pragma unroll
            for (int u = 0; u < 2 * KT; ++u)
#pragma unroll
                for (int d = 0; d < DT; ++d)
                    o[d] = Op16<T>::mfma32(*reinterpret_cast<const x8 *>(reinterpret_cast<const char *>(b.v) + (v_row ^ (kPair<C> * u)) + 32 * d * (2 * BN)), pf[0][u], o[d]);
        }
        if constexpr (I8)
            if (i + 1 < t.last) staging.store(step_key(t.c, i + 1), next);
        __syncthreads();
    };

    if (t.first < t.last) {
        const int n0 = step_key(t.c, t.first);
        const Buffer b{kt0, vt0, steps, steps + BN, step_units};
        pages.use();
        if constexpr (I8) {
            staging.load(pages, n0);
            staging.store(n0, b);
        } else
            staging.copy(pages, n0, b);
        pages.find(step_key(t.c, min(t.first + 1, t.last - 1)));
    }
    __syncthreads();
    run_steps(t, step);
    if (__ballot(pages.bad) != 0 && lane == 0) notes.bad = 1;
    __syncthreads();
    if (idle) return;
    const ChunkTile end = tile_note;
    const int at = end.row0 + 32 * wave + col;
    finish<C, QT, DT>(a, end, chunk_row(a, end, at), notes, at, D, 0, half, o, w.m, lane_pair_sum<32>(w.l + w.l2), w.unit);
}

// The same for 256-wide heads, whose O^T and queries for 32 rows take 192
// registers of a lane: a pair of waves shares 32 rows.  Each makes the scores
// of one half of a step's 64 keys and forms their weights, the pair exchanges
// maxima and weights (int8 caches: and their units) through LDS, and each
// multiplies all 64 keys' weights with one half of the dimensions.
template <typename C, typename QT>
__global__ void __launch_bounds__(64 * chunk_waves(256), 2) k_attn_chunk_wide(ChunkArgs a)
{
    typedef typename WeightOf<C>::type T;
    typedef typename Op16<T>::x8 x8;
    typedef ChunkBuffer<QT, T> Buffer;
    constexpr bool I8 = std::is_same<C, int8_t>::value;
    constexpr int D = 256, DT = 4, KK = D / 16;
    __shared__ __attribute__((aligned(16))) QT kt0[BN * D], kt1[BN * D];
    __shared__ __attribute__((aligned(16))) T vt0[BN * D], vt1[BN * D];
    __shared__ x8 weights[4][4][64];   // [pair][k-step of 16 keys][lane]
    __shared__ float tops[4][2][32];   // [pair][key half][row]
    __shared__ int units[I8 ? 4 : 1][2][32];
    __shared__ float steps[I8 ? 4 * BN : 1];
    __shared__ int step_units[2];
    __shared__ SeenKeys seen_of[kChunkRows];
    __shared__ int lift_of[I8 ? kChunkRows : 1];
    __shared__ ChunkNotes notes;

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 31, half = lane >> 5;
    const int pair = wave >> 1, part = wave & 1;
    __shared__ ChunkTile tile_note;  // for the end: in registers it would be in the way meanwhile
    ChunkTile t;
    if (!chunk_tile<QT, D>(a, blockIdx.x, false, t)) return;
    if (threadIdx.x == 0) tile_note = t;
    const bool idle = t.row0 + 32 * pair >= t.rows;
    ChunkPages pages(a, t);
    ChunkStaging<C, QT, D> staging(a, t);
    if (t.first < t.last) pages.find(step_key(t.c, t.first));
    const float c = a.scale * kLog2e;
    const ChunkRow first_row = chunk_row(a, t, t.row0 + 32 * pair + col);
    seen_of[32 * pair + col] = first_row.seen;
    const ChunkQuery<QT, D, false, I8> q(a, t, first_row, half);
    if constexpr (I8) lift_of[32 * pair + col] = q.lift;
    const bool lifted = I8 && __ballot(q.lift != 0) != 0;
    if (threadIdx.x == 0) notes = {0, 0};

    at_f32x16 o[DT];  // dimensions 128 part + 32 i + ...
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] = 0.0f;
    ChunkSoftmax<C, 1, 1> w;  // l: of this wave's keys
    int o_unit = -126;

    auto step = [&](auto border, auto odd, int i) __attribute__((always_inline)) {
        constexpr bool BORDER = decltype(border)::value;
        constexpr bool ODD = decltype(odd)::value;
        const Buffer b{ODD ? kt1 : kt0, ODD ? vt1 : vt0, steps + (ODD ? 2 * BN : 0), steps + (ODD ? 3 * BN : BN), step_units + ODD};
        const Buffer next{ODD ? kt0 : kt1, ODD ? vt0 : vt1, steps + (ODD ? 0 : 2 * BN), steps + (ODD ? BN : 3 * BN), step_units + !ODD};
        const int n0 = step_key(t.c, i), mine = n0 + 32 * part;
        if (i + 1 < t.last) {
            pages.use();
            if constexpr (I8)
                staging.load(pages, step_key(t.c, i + 1));
            else
                staging.copy(pages, step_key(t.c, i + 1), next);
        }
        pages.find(step_key(t.c, min(i + 2, t.last - 1)));
        SeenKeys seen{0, 0};
        if constexpr (BORDER) seen = seen_of[32 * pair + col];
        at_f32x16 s[1];
        float top = 0.0f;
        if (!idle) {
#pragma unroll
            for (int j = 0; j < 16; ++j) s[0][j] = 0.0f;
            const int k_row = not_kept(row_of<C, D>(32 * part + token_of_row(col), half));
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                typedef typename Op16<QT>::x8 k8;
                s[0] = Op16<QT>::mfma32(*reinterpret_cast<const k8 *>(reinterpret_cast<const char *>(b.k) + (k_row ^ (kPair<C> * kk))), q.f[kk], s[0]);
            }
            __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
            for (int k = 0; k < KK - kAhead; ++k) {
                __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
            __builtin_amdgcn_sched_group_barrier(0x8, kAhead, 0);
            top = w.top(BORDER, s, HiddenKeys(seen, t, n0), mine, half, c, [&](int, int j) { return b.ks[32 * part + w.key(0, j, half)]; }, lifted, [&] { return lift_of[32 * pair + col]; });
            if (half == 0) tops[pair][part][col] = top;
        }
        barrier_lds();
        if (!idle) {
            top = fmaxf(top, tops[pair][part ^ 1][col]);
            w.raise(top, o, o_unit);  // the same in both waves
            x8 pf[1][2];
            if constexpr (I8) {
                if constexpr (BORDER) asm volatile("" : "+v"(seen.lo), "+v"(seen.hi));
                w.products(BORDER, s, HiddenKeys(seen, t, n0), mine, half, [&](int, int j) { return b.vs[32 * part + w.key(0, j, half)]; }, *b.unit, pf, [](float) {});
                if (half == 0) units[pair][part][col] = w.unit;
            } else
                w.weights(s, c, pf);
            weights[pair][2 * part][lane] = pf[0][0];
            weights[pair][2 * part + 1][lane] = pf[0][1];
        }
        if constexpr (BORDER && !I8) {
            clean_values<T, D>(b.v, n0, tile_note.c, &notes);
        }
        barrier_lds();
        if (!idle) {
            int behind[2] = {0, 0};  // of a half's unit behind o's
            if constexpr (I8) {
                const int u0 = units[pair][0][col], u1 = units[pair][1][col];
                const int now = max(o_unit, max(u0, u1));
                if (__ballot(now > o_unit) != 0) {
                    const float f = ldexpf(1.0f, o_unit - now);
#pragma unroll
                    for (int d = 0; d < DT; ++d) o[d] *= f;
                    o_unit = now;
                }
                behind[0] = u0 - now;
                behind[1] = u1 - now;
            }
            // ---- O^T of dimensions 128 part ..
            const int v_row = not_kept(row_of<C, BN>(128 * part + col, half));
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                x8 p = weights[pair][u][lane];
                if constexpr (I8)
                    if (__ballot(behind[u >> 1] != 0) != 0) p *= static_cast<T>(ldexpf(1.0f, behind[u >> 1]));
#pragma unroll
                for (int d = 0; d < DT; ++d)
                    o[d] = Op16<T>::mfma32(*reinterpret_cast<const x8 *>(reinterpret_cast<const char *>(b.v) + (v_row ^ (kPair<C> * u)) + 32 * d * (2 * BN)), p, o[d]);
            }
        }
        if constexpr (I8)
            if (i + 1 < t.last) staging.store(step_key(t.c, i + 1), next);
        barrier_copies();  // all have read, the next step is there
    };

    if (t.first < t.last) {
        const int n0 = step_key(t.c, t.first);
        const Buffer b{kt0, vt0, steps, steps + BN, step_units};
        pages.use();
        if constexpr (I8) {
            staging.load(pages, n0);
            staging.store(n0, b);
        } else
            staging.copy(pages, n0, b);
        pages.find(step_key(t.c, min(t.first + 1, t.last - 1)));
    }
    barrier_copies();
    run_steps(t, step);
    if (__ballot(pages.bad) != 0 && lane == 0) notes.bad = 1;
    // the pair's sums
    float l = lane_pair_sum<32>(w.l + w.l2);
    __syncthreads();
    if (half == 0) tops[pair][part][col] = l;
    __syncthreads();
    if (idle) return;
    l = tops[pair][0][col] + tops[pair][1][col];
    const ChunkTile end = tile_note;
    const int at = end.row0 + 32 * pair + col;
    finish<C, QT, DT>(a, end, chunk_row(a, end, at), notes, at, D, 128 * part, half, o, w.m, l, o_unit);
}

// Joins the parts of the tiles that were cut: D / 4 lanes hold a row, and where
// few tiles have many pieces, all groups of lanes share one row's (G > 1), each
// taking every G-th (blockIdx.y: which of a tile's rows).
constexpr int join_lanes(int d) { return d / 4; }
constexpr int64_t kJoinGroups = 2048;
constexpr int kJoinAhead = 4;

template <typename QT, int D, bool MANY>
__global__ void __launch_bounds__(256) k_chunk_join(ChunkArgs a)
{
    constexpr int LPR = join_lanes(D), GROUPS = 256 / LPR, G = MANY ? GROUPS : 1, ROWS = GROUPS / G;
    __shared__ at_f32x4 sums[MANY ? GROUPS : 1][LPR];
    ChunkTile t;
    if (!chunk_tile<QT, D>(a, blockIdx.x, true, t) || t.pieces == 1) return;
    const int x = threadIdx.x % LPR, g = threadIdx.x / LPR, part = MANY ? g : 0;
    const int64_t stride = static_cast<int64_t>(t.stride) * a.hkv * a.slot_rows;
    for (int r = t.row0 + static_cast<int>(blockIdx.y) * ROWS + (MANY ? 0 : g); r < t.end; r += gridDim.y * ROWS) {
        const ChunkRow row = chunk_row(a, t, r);
        const int64_t first = part_slot(a, t, r);
        const float2 *ml = reinterpret_cast<const float2 *>(a.parts + a.rows_floats) + first;
        const float *src = a.parts + first * D + 4 * x;
        // lane x has piece x's reference and sum (the first LPR of them), and
        // every lane its elements of its first rows: one trip to memory
        at_f32x4 ahead[kJoinAhead];
#pragma unroll
        for (int i = 0; i < kJoinAhead; ++i) ahead[i] = *reinterpret_cast<const at_f32x4 *>(src + (part + i * G < t.pieces ? part + i * G : 0) * stride * D);
        const float2 mine = x < t.pieces ? ml[x * stride] : float2{-__builtin_inff(), 0.0f};
        float M = mine.x;
        for (int i = x + LPR; i < t.pieces; i += LPR) M = fmaxf(M, ml[i * stride].x);
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) M = fmaxf(M, __shfl_xor(M, o, 64));
        if (M == -__builtin_inff()) M = 0.0f;
        const float weight = __builtin_amdgcn_exp2f(mine.x - M) * mine.y;
        float L = weight;
        for (int i = x + LPR; i < t.pieces; i += LPR) L += __builtin_amdgcn_exp2f(ml[i * stride].x - M) * ml[i * stride].y;
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) L += __shfl_xor(L, o, 64);
        const float inv = row.seen.hi == 0 ? 0.0f : 1.0f / L;
        const auto weight_of = [&](int i) {
            return (i < LPR ? __shfl(weight, (threadIdx.x & 63 & ~(LPR - 1)) + i, 64)
                            : __builtin_amdgcn_exp2f(ml[i * stride].x - M) * ml[i * stride].y) * inv;
        };
        at_f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < kJoinAhead; ++i)
            if (part + i * G < t.pieces) o += weight_of(part + i * G) * ahead[i];
#pragma unroll 4
        for (int i = part + kJoinAhead * G; i < t.pieces; i += G) o += weight_of(i) * *reinterpret_cast<const at_f32x4 *>(src + i * stride * D);
        if constexpr (MANY) {
            sums[g][x] = o;
            __syncthreads();
            if (g == 0) {
#pragma unroll
                for (int i = 1; i < GROUPS; ++i) o += sums[i][x];
            }
            __syncthreads();
        }
        if (!MANY || g == 0)
            store4(static_cast<QT *>(a.out) + ((static_cast<int64_t>(t.q0) + row.tok) * a.hq + row.head) * D + 4 * x, o);
    }
}

template <typename C, typename QT, int D>
hipError_t chunk_launch(const ChunkArgs &a, const ChunkPlan &p, int cache_type, int q_type, hipStream_t s)
{
    const dim3 grid(static_cast<uint32_t>(p.numbers * a.hkv));
    if (p.few) {
        const hipError_t e = launch_chunk_few(a, cache_type, q_type, D, grid.x, s);
        if (e != hipSuccess) return e;
    } else if constexpr (D == 256)
        hipLaunchKernelGGL((k_attn_chunk_wide<C, QT>), grid, dim3(64 * chunk_waves(D)), 0, s, a);
    else
        hipLaunchKernelGGL((k_attn_chunk<C, QT, D>), grid, dim3(64 * chunk_waves(D)), 0, s, a);
    if (p.cut) {
        // a workgroup for some rows of a tile each; many tiles are mostly uncut,
        // and their workgroups only find that out
        const int64_t tiles = p.tiles * a.hkv, each = kJoinGroups / tiles;
        const bool many = p.few && p.wanted >= 16 * p.tiles;
        const int64_t at_once = many ? 1 : 256 / join_lanes(D), rows = (p.slot_rows + at_once - 1) / at_once;
        const dim3 groups(static_cast<uint32_t>(tiles), static_cast<uint32_t>(each < 1 ? 1 : each < rows ? each : rows));
        if (many)
            hipLaunchKernelGGL((k_chunk_join<QT, D, true>), groups, dim3(256), 0, s, a);
        else
            hipLaunchKernelGGL((k_chunk_join<QT, D, false>), groups, dim3(256), 0, s, a);
    }
    return hipGetLastError();
}

template <typename C, typename QT>
hipError_t chunk_d(const ChunkArgs &a, const ChunkPlan &p, int cache_type, int q_type, int d, hipStream_t s)
{
    return d == 64 ? chunk_launch<C, QT, 64>(a, p, cache_type, q_type, s) : d == 128 ? chunk_launch<C, QT, 128>(a, p, cache_type, q_type, s) : chunk_launch<C, QT, 256>(a, p, cache_type, q_type, s);
}

}  // namespace

// Bytes of parts above which nothing is cut.
constexpr int64_t kMaxChunkParts = int64_t{1} << 28;

ChunkPlan chunk_plan(int64_t batch, int64_t q_rows, int64_t max_q, int32_t hq, int32_t hkv, int32_t d, int64_t max_len,
                     int64_t window, int64_t sinks)
{
    ChunkPlan p;
    const int64_t group = hq / hkv, rows = max_q * group;
    p.tiles = q_rows * group / kChunkRows + batch;
    p.numbers = p.tiles;
    p.few = rows <= kFewRows;
    p.slot_rows = static_cast<int32_t>(rows < kChunkRows ? rows : kChunkRows);
    // workgroups that the GPU holds (of 64-wide heads over 16-bit caches it holds
    // 768, three a CU: their last rounds are judged by a smaller GPU than it is)
    const int64_t slots = d == 256 ? 256 : 512;
    p.wanted = static_cast<int32_t>(slots / hkv > 1 ? slots / hkv : 1);
    const int most = steps_bound(static_cast<int>(max_len), static_cast<int>(window), static_cast<int>(sinks), static_cast<int>(group));
    // pieces: of all tiles wanted + tiles at most, or twice wanted in the place of
    // the last tiles; of those that are cut, which need a place, twice wanted
    const int64_t numbers = 2 * p.wanted + p.tiles, places = 2 * p.wanted, parts = places * hkv * p.slot_rows;
    p.cut = most > kChunkMinSteps && p.tiles * hkv <= 4 * slots && parts * (d + 2) * 4 <= kMaxChunkParts;
    if (p.cut) {
        // a step's time with the GPU full, a piece's rows written and read in
        // fp32 at half of HBM's rate (they come in bursts), and the join, in us
        const double step = p.few ? (d == 256 ? 2.7 : 1.35) : d == 256 ? 2.6 : d == 128 ? 1.9 : 1.1;
        p.join_cost = static_cast<float>((p.few ? 5.0 : 6.0) / step);
        p.piece_cost = static_cast<float>(static_cast<double>(hkv) * p.slot_rows * d * 4 * 2 / 2.5e6 / step);
        const int64_t pieces = p.tiles * ((most + kChunkMinSteps - 1) / kChunkMinSteps);
        p.numbers = pieces < numbers ? pieces : numbers;
        p.rows_floats = static_cast<size_t>(parts) * d;
        p.part_floats = p.rows_floats + static_cast<size_t>(parts) * 2;
    }
    return p;
}

hipError_t launch_attn_chunk(const ChunkPlan &p, const void *q, int64_t qs, int q_type, const int32_t *cu, int64_t batch,
                             int64_t q_rows, int64_t max_q, int32_t hq, const ptq1_kv_cache &c, const int32_t *table,
                             int64_t max_pages, const int32_t *lens, int64_t max_len, int32_t window, int32_t sinks,
                             float scale, void *out, float *parts, hipStream_t s)
{
    int head_shift = 24;  // the product is off by less than 2^head_shift / 2^24 heads of 2^24
    while ((1 << (head_shift - 24)) < c.n_kv_heads) ++head_shift;
    const uint32_t per_head = static_cast<uint32_t>(((int64_t{1} << head_shift) + c.n_kv_heads - 1) / c.n_kv_heads);
    const ChunkArgs a{q, qs, cu, lens, table, max_pages, batch, q_rows, max_q, max_len, hq, c.n_kv_heads, hq / c.n_kv_heads, per_head, head_shift, c.k_pages,
                      c.v_pages, c.k_steps, c.v_steps, c.n_pages, __builtin_ctz(static_cast<unsigned>(c.page_size)),
                      window, sinks, scale, out, p.wanted, p.cut, 2 * p.wanted, p.slot_rows,
                      p.join_cost, p.piece_cost, static_cast<int64_t>(p.rows_floats), parts};
    if (c.dtype == PTQ1_BF16) return chunk_d<__bf16, __bf16>(a, p, c.dtype, q_type, c.head_dim, s);
    if (c.dtype == PTQ1_F16) return chunk_d<_Float16, _Float16>(a, p, c.dtype, q_type, c.head_dim, s);
    return q_type == PTQ1_F16 ? chunk_d<int8_t, _Float16>(a, p, c.dtype, q_type, c.head_dim, s) : chunk_d<int8_t, __bf16>(a, p, c.dtype, q_type, c.head_dim, s);
}

}  // namespace ptq1
