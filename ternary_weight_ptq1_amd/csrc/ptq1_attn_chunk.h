// ptq1_attn_chunk.h -- what the kernels of the attention of chunks over the
// cache share (attn_chunk.hip, attn_chunk_few.hip): which rows and steps a
// workgroup takes, the pages of a step, and the softmax of its scores.
#pragma once
#include <hip/hip_runtime.h>

#include <type_traits>

#include "ptq1_attn.h"
#include "ptq1_attn_tile.h"
#include "ptq1_chunk.h"
#include "ptq1_launch.h"

namespace ptq1 {

struct ChunkArgs {
    const void *q;
    int64_t qs;  // row stride in elements
    const int32_t *cu, *lens, *table;
    int64_t max_pages, batch, q_rows, max_q, max_len;
    int32_t hq, hkv, group;
    uint32_t per_head;  // n / hkv is n * per_head >> head_shift, for n below 2^24
    int32_t head_shift;
    const void *k_pages, *v_pages;
    const float *k_steps, *v_steps;
    int64_t n_pages;
    int32_t page_shift;
    int32_t window, sinks;
    float scale;
    void *out;
    int32_t wanted, cut;       // pieces of one kv head that fill the GPU; tiles may be cut
    int32_t places, slot_rows; // of parts, of one kv head, and rows of one
    float join_cost, piece_cost;  // in steps
    int64_t rows_floats;
    float *parts;
};

// The kernels for few rows (plan.few).
hipError_t launch_chunk_few(const ChunkArgs &a, int cache_type, int q_type, int d, uint32_t groups, hipStream_t s);

namespace {

constexpr int BN = kChunkKeys;
static_assert(kKeys == kChunkKeys, "a step is a tile of keys");
constexpr int kFewRows = 32;  // of a kv head, that one set of columns holds

// The 16-bit type of the second product over a cache of C: int8 codes and the
// weights that meet them are fp16.  (The first product is in the queries' type.)
template <typename C>
struct WeightOf {
    typedef C type;
};
template <>
struct WeightOf<int8_t> {
    typedef _Float16 type;
};

// The token of row r of a score tile of 32: bits 2 and 3 change places.
__device__ __forceinline__ int token_of_row(int r) { return (r & 19) | ((r & 4) << 1) | ((r & 8) >> 1); }

// A sequence's rows and keys as the arguments give them.
struct ChunkSeq {
    int q0, lq, len;
};
__device__ __forceinline__ ChunkSeq chunk_seq(const ChunkArgs &a, int64_t b)
{
    return {a.cu[b], a.cu[b + 1] - a.cu[b], a.lens[b]};
}
__device__ __forceinline__ bool refused(const ChunkArgs &a, const ChunkSeq &s)
{
    return s.q0 < 0 || s.lq > a.max_q || s.q0 + static_cast<int64_t>(s.lq) > a.q_rows || s.len < 0 || s.len > a.max_len;
}
// Tiles of the rows that exist.
__device__ __forceinline__ int seq_tiles(const ChunkArgs &a, const ChunkSeq &s, int group)
{
    const int64_t first = s.q0 > 0 ? s.q0 : 0, end = s.q0 + static_cast<int64_t>(s.lq);
    const int64_t n = (end < a.q_rows ? end : a.q_rows) - first;
    return n > 0 ? static_cast<int>((n * group + kChunkRows - 1) / kChunkRows) : 0;
}
__device__ __forceinline__ int seq_steps(const ChunkArgs &a, const ChunkSeq &s, int group)
{
    return refused(a, s) ? 0 : steps_bound(s.len, a.window, a.sinks, group);
}

template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp(int v)
{
    return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);  // (0 where there is no such lane)
}
// The sum of the lanes up to and with this one's.
__device__ __forceinline__ int lanes_to(int v)
{
    v += dpp<0x111, 0xF>(v);  // one lane down its row of 16, two ...
    v += dpp<0x112, 0xF>(v);
    v += dpp<0x114, 0xF>(v);
    v += dpp<0x118, 0xF>(v);
    v += dpp<0x142, 0xA>(v);  // the last of row 0 to row 1, of 2 to 3
    v += dpp<0x143, 0xC>(v);  // of row 1 to rows 2 and 3
    return v;
}
__device__ __forceinline__ int wave_total(int v) { return __builtin_amdgcn_readlane(lanes_to(v), 63); }
// The largest, of numbers that are not negative.
__device__ __forceinline__ int wave_largest(int v)
{
    v = max(v, dpp<0x111, 0xF>(v));
    v = max(v, dpp<0x112, 0xF>(v));
    v = max(v, dpp<0x114, 0xF>(v));
    v = max(v, dpp<0x118, 0xF>(v));
    v = max(v, dpp<0x142, 0xA>(v));
    v = max(v, dpp<0x143, 0xC>(v));
    return __builtin_amdgcn_readlane(v, 63);
}
// The sum of f(sequence) over the first n.
template <class F>
__device__ __forceinline__ int sum_over(const ChunkArgs &a, int64_t n, F f)
{
    int v = 0;
    for (int64_t i = threadIdx.x & 63; i < n; i += 64) v += f(chunk_seq(a, i));
    return wave_total(v);
}

// One tile of query rows of one kv head, and the steps of one workgroup.
struct ChunkTile {
    int group, kh;
    int b;
    int q0, off;             // the sequence's first row; keys before its first query
    int rows, row0, end;     // its rows; this tile's first one and the one behind its last
    ChunkSteps c;
    int first, last;         // this workgroup's steps
    int pieces;              // of the tile
    int place, stride;       // of the piece's part (join: of the first one's), and between them
};

// The numbers of the lanes before this one, and all lanes' together.
__device__ __forceinline__ int lanes_before(int mine, int &total)
{
    const int sum = lanes_to(mine);
    total = __builtin_amdgcn_readlane(sum, 63);
    return sum - mine;
}

// Which tile and piece workgroup `number` of a kv head takes (join: which tile
// of those that were cut), by the sequences' tiles and steps; false: none.
//
// Up to 64 sequences (a lane each): tiles are numbered from the longest
// sequence on.  Where all are about equally long (0.6 of the longest on
// average), whole rounds of tiles run uncut, and those behind them are cut in
// the number that is estimated to end soonest: rounds of pieces, in steps, and
// what a piece's rows and the join cost, in steps too.  (3 x 1000 to 2000 tokens in
// windows of 1024: 30 tiles of 19 steps behind the last round, 132 us uncut, 147
// where the estimate is made to cut them.  4096 tokens behind 28000: 32 tiles of
// 322, cut in two, 1564 us, 1577 uncut: where they are one workgroup a CU, each is
// faster.)  Otherwise tiles are only cut that are longer than an even share, into
// pieces of that: shorter ones fill the gaps as they are.
// More sequences: in their order, all cut, or none.
struct ChunkPick {
    int q0, lq, len;
    int b, tiles, tile, piece, per, place, stride;
};
__device__ __forceinline__ bool pick_of_64(const ChunkArgs &a, int number, int group, bool join, ChunkPick &k)
{
    const int lane = threadIdx.x & 63, n = static_cast<int>(a.batch);
    ChunkSeq s{0, 0, 0};
    int tiles = 0, steps = 0;
    if (lane < n) {
        s = chunk_seq(a, lane);
        tiles = seq_tiles(a, s, group);
        steps = seq_steps(a, s, group);
    }
    int before = 0, all = 0;
    for (int j = 0; j < n; ++j) {
        const int t = __builtin_amdgcn_readlane(tiles, j), other = __builtin_amdgcn_readlane(steps, j);
        all += t;
        if (other > steps || (other == steps && j < lane)) before += t;
    }
    int whole = all, per = 1 << 30;
    if (a.cut) {
        const int total = wave_total(tiles * steps), longest = wave_largest(steps);
        const int full = all / a.wanted * a.wanted, mine = max(0, min(tiles, before + tiles - full));
        const int left = wave_total(mine * steps), last = wave_largest(mine > 0 ? steps : 0);
        if (10 * static_cast<int64_t>(total) < 6 * static_cast<int64_t>(all) * longest) {
            whole = 0;
            per = chunk_piece(total, a.wanted);
        } else if (all > full && 10 * static_cast<int64_t>(left) >= 6 * static_cast<int64_t>(all - full) * last) {
            // (a lane each: a loop over them took 10 us of a kernel's start)
            const float cost = chunk_cost(chunk_cut_of(lane), all - full, last, a.wanted, a.join_cost, a.piece_cost);
            const float least = -wave_max(cost < 0.0f ? -__builtin_inff() : -cost);
            const int n = chunk_cut_of(__builtin_ctzll(__ballot(cost == least)));
            if (n > 1) {
                whole = full;
                per = imax(kChunkMinSteps, (last + n - 1) / n);
            }
        }
    }
    const int rest = max(0, min(tiles, before + tiles - whole));  // its tiles that may be cut
    // (stores into k at the end alone: from both branches they went through memory)
    int who, tile, piece = 0, at = 0, stride = 0;
    if (!join && number < whole) {
        per = 1 << 30;
        who = __builtin_ctzll(__ballot(number >= before && number - before < tiles));
        tile = number - __builtin_amdgcn_readlane(before, who);
    } else {
        if (!join) number -= whole;
        // (places for parts: of the tiles that are cut alone)
        const int pieces = chunk_pieces(steps, per), numbers = rest * pieces;
        int total, places;
        const int place = lanes_before(pieces > 1 ? numbers : 0, places), from = lanes_before(join ? rest : numbers, total);
        if (number >= total || places > a.places) return false;
        who = __builtin_ctzll(__ballot(number >= from && number - from < (join ? rest : numbers)));
        const int r = number - __builtin_amdgcn_readlane(from, who);
        stride = __builtin_amdgcn_readlane(rest, who);
        piece = join ? 0 : r / stride;
        tile = __builtin_amdgcn_readlane(tiles, who) - stride + (join ? r : r - piece * stride);
        at = __builtin_amdgcn_readlane(place, who) + r;
    }
    k = {__builtin_amdgcn_readlane(s.q0, who), __builtin_amdgcn_readlane(s.lq, who), __builtin_amdgcn_readlane(s.len, who), who,
         __builtin_amdgcn_readlane(tiles, who), tile, piece, per, at, stride};
    return true;
}
__device__ __forceinline__ bool pick_of_many(const ChunkArgs &a, int number, int group, bool join, ChunkPick &k)
{
    int per = 1 << 30;
    if (a.cut)
        per = chunk_piece(sum_over(a, a.batch, [&](const ChunkSeq &s) { return seq_tiles(a, s, group) * seq_steps(a, s, group); }), a.wanted);
    const auto numbers = [&](const ChunkSeq &s) { return seq_tiles(a, s, group) * chunk_pieces(seq_steps(a, s, group), per); };
    const auto of = [&](int64_t i) {
        const ChunkSeq s = chunk_seq(a, i);
        return join ? seq_tiles(a, s, group) : numbers(s);
    };
    int64_t b64, at;
    if (!(a.cut ? find_tile_in_runs(number, a.batch, of, b64, at) : find_rows<kChunkRows>(number, a.cu, a.batch, a.q_rows, group, b64, at)))
        return false;
    const int b = __builtin_amdgcn_readfirstlane(static_cast<int>(b64));
    int tile = __builtin_amdgcn_readfirstlane(static_cast<int>(at)), piece = 0, place = 0;
    const ChunkSeq s = chunk_seq(a, b);
    const int tiles = seq_tiles(a, s, group), pieces = chunk_pieces(seq_steps(a, s, group), per);
    if (pieces > 1) {
        const int before = sum_over(a, b, [&](const ChunkSeq &s) { return chunk_pieces(seq_steps(a, s, group), per) > 1 ? numbers(s) : 0; });
        if (before + tiles * pieces > a.places) return false;
        place = before + tile;
        if (!join) {
            piece = tile / tiles;
            tile -= piece * tiles;
        }
    }
    k = {s.q0, s.lq, s.len, b, tiles, tile, piece, per, place, tiles};
    return true;
}

// False: nothing (more) to do.  The rows of a sequence that is refused become
// NaN.
template <typename QT, int D>
__device__ __forceinline__ bool chunk_tile(const ChunkArgs &a, uint32_t block, bool join, ChunkTile &t)
{
    t.group = a.group;
    const int number = static_cast<int>((static_cast<uint64_t>(block) * a.per_head) >> a.head_shift);
    t.kh = static_cast<int>(block) - number * a.hkv;
    ChunkPick k;
    if (!(a.batch <= 64 ? pick_of_64(a, number, t.group, join, k) : pick_of_many(a, number, t.group, join, k))) return false;
    const ChunkSeq s{k.q0, k.lq, k.len};
    if (refused(a, s)) {
        const int64_t r = (s.q0 < 0 ? -static_cast<int64_t>(s.q0) * t.group : 0) + static_cast<int64_t>(k.tile) * kChunkRows + threadIdx.x;
        const int64_t tok = s.q0 + r / t.group;
        if (!join && k.piece == 0 && threadIdx.x < kChunkRows && tok < s.q0 + static_cast<int64_t>(s.lq) && tok < a.q_rows) {
            QT *dst = static_cast<QT *>(a.out) + (tok * a.hq + t.kh * t.group + r % t.group) * D;
            const float n = __builtin_nanf("");
            for (int e = 0; e < D; e += 4) store4(dst + e, at_f32x4{n, n, n, n});
        }
        return false;
    }
    t.b = k.b;
    t.q0 = s.q0;
    t.off = s.len - s.lq;
    t.rows = s.lq * t.group;
    // the last rows see the most keys: they start first
    t.row0 = (k.tiles - 1 - k.tile) * kChunkRows;
    t.end = t.row0 + kChunkRows < t.rows ? t.row0 + kChunkRows : t.rows;
    t.c = chunk_steps(t.row0 / t.group + t.off, (t.end - 1) / t.group + t.off, a.window, a.sinks);
    t.pieces = chunk_pieces(t.c.steps, k.per);
    if (k.piece >= t.pieces) return false;
    t.first = k.piece * k.per;
    t.last = t.c.steps - t.first > k.per ? t.first + k.per : t.c.steps;
    t.place = k.place;
    t.stride = k.stride;
    return true;
}

// The place of a row's part.
__device__ __forceinline__ int64_t part_slot(const ChunkArgs &a, const ChunkTile &t, int row)
{
    return (static_cast<int64_t>(t.place) * a.hkv + t.kh) * a.slot_rows + (row - t.row0);
}

// One lane's query row.
struct ChunkRow {
    bool is;
    int tok, head;
    SeenKeys seen;
};
__device__ __forceinline__ ChunkRow chunk_row(const ChunkArgs &a, const ChunkTile &t, int row)
{
    ChunkRow r;
    r.is = row < t.rows;
    const int at = r.is ? row : t.rows - 1;
    r.tok = at / t.group;
    r.head = t.kh * t.group + at % t.group;
    r.seen = seen_keys(r.tok + t.off, a.window);
    return r;
}

// Where the keys of a step are: a wave's lanes hold the pages of the step's
// four runs of 16 tokens (lane % 4), looked up by `find` and checked by `use`,
// which leaves them in scalars.  A run that no row of the tile sees (behind the
// sequence, or between the first tokens and the windows, where pages may have
// been given back) reads another's page; all of it is masked.
struct ChunkPages {
    const int32_t *table;
    int page_shift, lo, reach, sunk;
    uint32_t n_pages;
    int32_t found = 0;
    int32_t run[4];
    bool bad = false;

    __device__ __forceinline__ ChunkPages(const ChunkArgs &a, const ChunkTile &t)
        : table(a.table + static_cast<int64_t>(t.b) * a.max_pages), page_shift(a.page_shift), lo(t.c.lo), reach(t.c.reach), sunk(t.c.sunk),
          n_pages(static_cast<uint32_t>(a.n_pages))
    {
        asm volatile("" : "+s"(n_pages));  // (kept, not loaded in every step)
    }
    __device__ __forceinline__ void find(int n0)
    {
        const int s = n0 + 16 * (threadIdx.x & 3);
        const int tok = s < sunk ? s : min(max(s, lo), reach - 1);
        found = table[tok >> page_shift];
    }
    __device__ __forceinline__ void use()
    {
        const bool is = static_cast<uint32_t>(found) < n_pages;
        bad |= !is;
        const int32_t pg = is ? found : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) run[i] = __builtin_amdgcn_readlane(pg, i);
    }
    __device__ __forceinline__ int32_t of(int i) const
    {
        const int32_t a = i & 1 ? run[1] : run[0], b = i & 1 ? run[3] : run[2];
        return i & 2 ? b : a;
    }
};

// int8 caches: the unit (its exponent) of values' steps of which those that some
// row sees are below 2^e: the last one as long as it is at most 2^12 more.
__device__ __forceinline__ int unit_of_steps(int unit, int e)
{
    return e > 125 || (e <= unit && e >= unit - 12) ? unit : e + 2;
}

// Byte B of x, signed, as fp32 (of a shift and a conversion the compiler makes
// two instructions).
template <int B>
__device__ __forceinline__ float code_of(uint32_t x)
{
    float f;
    if constexpr (B == 0)
        asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_0" : "=v"(f) : "v"(x));
    else if constexpr (B == 1)
        asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_1" : "=v"(f) : "v"(x));
    else if constexpr (B == 2)
        asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_2" : "=v"(f) : "v"(x));
    else
        asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_3" : "=v"(f) : "v"(x));
    return f;
}
// 8 int8 codes (two dwords) as bf16, exact: the upper halves of them as fp32.
__device__ __forceinline__ bf16x8 codes_to_bf16(uint32_t a, uint32_t b)
{
    const auto pair = [](float lo, float hi) {
        return __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, hi), __builtin_bit_cast(uint32_t, lo), 0x07060302u);
    };
    const at_u32x4 w = {pair(code_of<0>(a), code_of<1>(a)), pair(code_of<2>(a), code_of<3>(a)), pair(code_of<0>(b), code_of<1>(b)),
                        pair(code_of<2>(b), code_of<3>(b))};
    return __builtin_bit_cast(bf16x8, w);
}
template <typename T>
__device__ __forceinline__ typename Op16<T>::x8 codes_to(uint32_t a, uint32_t b)
{
    if constexpr (std::is_same<T, __bf16>::value)
        return codes_to_bf16(a, b);
    else
        return codes_to_f16(a, b);
}

// What was met on the way, for the end: the steps (modulo 32) whose V tile had a
// NaN or an infinity removed that some row sees, and whether a page was not there.
struct ChunkNotes {
    uint32_t odd_steps;
    int bad;
};
__device__ __forceinline__ uint32_t step_bit(int n0) { return 1u << ((n0 / kChunkKeys) & 31); }

// The largest magnitude among 16-bit values, as bits: a NaN's or an infinity's if there is one.
template <typename T>
struct LargestHalf {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u16x2 most = {0, 0};
    __device__ __forceinline__ void of(const at_u32x4 &w)
    {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t x = w[j] & 0x7fff7fffu;
            most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, x));
        }
    }
    __device__ __forceinline__ bool non_finite() const
    {
        constexpr uint16_t kNone = std::is_same<T, __bf16>::value ? 0x7f80u : 0x7c00u;
        return most[0] >= kNone || most[1] >= kNone;
    }
};

// Of the eight keys from `key` on, in 16 bits each: ones for those that some row
// of the tile sees.  The others hold anything (behind a sequence's end or ahead
// of its windows what no token was written to), and are no row's concern.
__device__ __forceinline__ at_u32x4 seen_halves(int key, int lo, int reach, int sunk)
{
    const auto below = [&](int end) { return (1 << min(max(end - key, 0), 8)) - 1; };  // a bit for each of the eight
    const int some = below(reach) & (~below(lo) | below(sunk));
    at_u32x4 m;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t a = __builtin_amdgcn_sbfe(some, 2 * j, 1), b = __builtin_amdgcn_sbfe(some, 2 * j + 1, 1);
        m[j] = (a & 0xffffu) | (b & 0xffff0000u);
    }
    return m;
}

// The page of a key, -1 if there is none.
__device__ __forceinline__ int64_t page_of_key(const ChunkArgs &a, const ChunkTile &t, int key)
{
    const int64_t pg = a.table[static_cast<int64_t>(t.b) * a.max_pages + (key >> a.page_shift)];
    return pg >= 0 && pg < a.n_pages ? pg : -1;
}

// Adds to O^T, dimensions d0 + 32 i + ..., the NaNs and infinities among the
// values that the row sees and that were left out of the products.
template <typename T, int N>
__device__ __forceinline__ void add_odd_values(const ChunkArgs &a, const ChunkTile &t, const ChunkRow &row,
                                               const ChunkNotes &notes, int d, int d0, int half, at_f32x16 (&o)[N])
{
    const int64_t page = int64_t{1} << a.page_shift;
    for (int step = t.first; step < t.last; ++step) {
        const int n0 = step_key(t.c, step);
        if ((notes.odd_steps & step_bit(n0)) == 0) continue;
        for (int j = n0; j < n0 + kChunkKeys && j < t.c.reach; ++j) {
            if (j >= t.c.sunk && j < t.c.lo) continue;
            const int64_t pg = page_of_key(a, t, j);
            if (pg < 0 || !(j < row.seen.hi && (j >= row.seen.lo || j < a.sinks))) continue;
            const T *src = static_cast<const T *>(a.v_pages) + ((pg * a.hkv + t.kh) * d + d0 + 4 * half) * page + (j & (page - 1));
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float x = static_cast<float>(src[(32 * i + 8 * (e >> 2) + (e & 3)) * page]);
                    if (!(fabsf(x) <= 3.4028235e38f)) o[i][e] += x;
                }
        }
    }
}

// The row sees a key whose page is not there.
__device__ __forceinline__ bool sees_bad_page(const ChunkArgs &a, const ChunkTile &t, const ChunkRow &row)
{
    bool bad = false;
    const int first = row.seen.lo >> a.page_shift, end = (row.seen.hi + (1 << a.page_shift) - 1) >> a.page_shift;
    for (int i = 0; i < end && i < first; ++i)
        if ((i << a.page_shift) < a.sinks) bad |= page_of_key(a, t, i << a.page_shift) < 0;
        else break;
    for (int i = first; i < end; ++i) bad |= page_of_key(a, t, i << a.page_shift) < 0;
    return bad;
}

// One lane's row as the products' B operand, k = 16 kk + 8 half + j (RUN16: 32
// (kk / 2) + 16 half + 8 (kk % 2) + j, the order of 16 int8 codes that a lane
// loads at once).
//
// int8 caches (LIFT): a score is the sum of query times code, times the key's
// step.  bf16 queries below 2^-80 or above 2^80, whose sums could leave fp32's
// range though the scores would not, enter divided by 2^lift, which brings the
// row's largest to about one.
template <typename QT, int D, bool RUN16 = false, bool LIFT = false>
struct ChunkQuery {
    typename Op16<QT>::x8 f[D / 16];
    int lift = 0;
    __device__ __forceinline__ ChunkQuery(const ChunkArgs &a, const ChunkTile &t, const ChunkRow &row, int half)
    {
        const QT *qp = static_cast<const QT *>(a.q) + (static_cast<int64_t>(t.q0) + row.tok) * a.qs + static_cast<int64_t>(row.head) * D;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
            f[kk] = *reinterpret_cast<const typename Op16<QT>::x8 *>(qp + (RUN16 ? 32 * (kk >> 1) + 16 * half + 8 * (kk & 1) : 16 * kk + 8 * half));
        if constexpr (LIFT && std::is_same<QT, __bf16>::value) {
            typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
            u16x2 most = {0, 0};
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t x = __builtin_bit_cast(at_u32x4, f[kk])[j] & 0x7fff7fffu;
                    most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, x));
                }
            const float top = lane_pair_max<32>(__builtin_bit_cast(float, static_cast<uint32_t>(most[0] > most[1] ? most[0] : most[1]) << 16));
            const int e = static_cast<int>(__builtin_bit_cast(uint32_t, top) >> 23) - 127;
            const bool far = (top > 0.0f) & (e < 128) & ((e > 80) | (e < -80));
            lift = far ? e : 0;
            if (__ballot(far) != 0) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[kk][j] = static_cast<QT>(ldexpf(static_cast<float>(f[kk][j]), -lift));
            }
        }
    }
};

// Which keys of a step a row does not see.
struct HiddenKeys {
    int hi, lo, sinks;
    bool gap;  // (of any row) first keys that are seen beside the window are among them
    __device__ __forceinline__ HiddenKeys(const SeenKeys &seen, const ChunkTile &t, int n0)
        : hi(seen.hi), lo(seen.lo), sinks(t.c.sunk), gap(n0 < t.c.sunk)
    {
    }
    // (no branches in these: a value that one selects is lost by the compiler)
    __device__ __forceinline__ bool beside_gap(int key) const { return (key >= hi) | ((key < lo) & (key >= sinks)); }
    __device__ __forceinline__ bool without_gap(int key) const
    {
        return static_cast<uint32_t>(key - lo) >= static_cast<uint32_t>(hi - lo);
    }
};

// The weights of KT * 32 keys from key n0 on, of one lane's row (score
// register j of tile t: key n0 + 32 t + 16 (j / 8) + 8 half + j % 8).
//
// int8 caches: a weight times its value's step, in the step's unit, is p vs; o
// is in units of 2^unit of its row.  Where the two units are the same in all
// rows, that is all; elsewhere (the first steps, after the reference has moved,
// where steps differ much, and on the border) the row's unit goes by the
// products themselves, so that they are below 2^15, by at most 2^12 more than
// they need: what is lost is below 2^-27 of the row's largest.
//
// RUN16: register j is key n0 + 32 t + 16 half + j instead.
// TERMS: 16-bit terms that a weight (int8: times its step) enters as, the second
// the rounding of what the first one leaves.  With one, the sum is that of the
// rounded weights.
template <typename C, int KT, int TERMS, bool RUN16 = false>
struct ChunkSoftmax {
    static constexpr bool I8 = std::is_same<C, int8_t>::value;
    typedef typename WeightOf<C>::type T;
    typedef typename Op16<T>::x8 x8;
    float m = -__builtin_inff(), l = 0.0f, l2 = 0.0f;  // m: the reference, in units of log2
    bool large = false;
    int unit = -126;
    // int8 caches: a step's scores are multiplied by their keys' steps and taken
    // from the reference at once, base; `shift` further where it moves (and all
    // of it where products are rounded first, base = 0: in a row's first step,
    // which has no reference yet, and among large or lifted scores)
    float base = 0.0f, shift = 0.0f;

    static __device__ __forceinline__ int key(int t, int j, int half)
    {
        return RUN16 ? 32 * t + 16 * half + j : 32 * t + 16 * (j >> 3) + 8 * half + (j & 7);
    }

    static __device__ __forceinline__ void by_power(at_f32x16 (&s)[KT], int e)
    {
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int j = 0; j < 16; ++j) s[t][j] = ldexpf(s[t][j], e);
    }

    // the largest score of the lane's pair (int8 caches: less base); on the border
    // hidden ones leave the scores (int8 caches: ks(t, j) is the step of score register j of tile t;
    // lifted: of some row the queries are, lift() is the lane's)
    template <class S, class L>
    __device__ __forceinline__ float top(bool border, at_f32x16 (&s)[KT], const HiddenKeys &hidden, int n0, int half, float c, S ks, bool lifted, L lift)
    {
        if constexpr (I8) {
            base = large || lifted || m == -__builtin_inff() ? 0.0f : m;
            if (lifted) by_power(s, lift() >> 1);
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    s[t][j] = fmaf(s[t][j], ks(t, j), -base);
                    if (!RUN16 && (j & 7) == 7) __builtin_amdgcn_sched_barrier(0);  // (or all steps are read up front)
                }
            if (lifted) by_power(s, (lift() + 1) >> 1);
        }
        if (border) {
            if (hidden.gap) {
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int j = 0; j < 16; ++j) s[t][j] = hidden.beside_gap(n0 + key(t, j, half)) ? -__builtin_inff() : s[t][j];
            } else {
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int j = 0; j < 16; ++j) s[t][j] = hidden.without_gap(n0 + key(t, j, half)) ? -__builtin_inff() : s[t][j];
            }
        }
        float top = s[0][0];
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int j = 0; j < 16; ++j) top = fmaxf(top, s[t][j]);
        top = lane_pair_max<32>(top);
        return I8 ? top : top * c;
    }

    // The reference follows the largest score, by 8 at most behind it (weights
    // up to 2^8 lose nothing): few steps after the first rescale.  units: o's.
    template <int N>
    __device__ __forceinline__ void raise(float top, at_f32x16 (&o)[N], int &units)
    {
        const float mt = reference<T>(top), was = I8 ? m - base : m;
        if constexpr (I8) shift = was;
        if (__ballot(mt > was + 8.0f) != 0) {
            float mn = fmaxf(was, mt);
            if constexpr (I8) {
                // whole numbers, of which sums are exact (below 2^24): rounded here alone,
                // a reference would be another for this step's keys than for the later ones'
                mn = ceilf(mn);
                m = base + mn;
            } else
                m = mn;
            float f = was == mn ? 1.0f : __builtin_amdgcn_exp2f(was - mn);
            l *= f;
            l2 *= f;
            if constexpr (I8) {
                // the units come down with the weights, or a large step whose
                // weight has become nothing would keep the resolution coarse
                int down = static_cast<int>(__builtin_bit_cast(uint32_t, f) >> 23) - 126;  // f < 2^down
                down = down > 0 ? 0 : down;
                f *= pow2(-down);
                if (&units != &unit) unit = max(unit + down, -300);
                units = max(units + down, -300);
            }
#pragma unroll
            for (int i = 0; i < N; ++i) o[i] *= f;
            if constexpr (I8) shift = mn;
            large = large_scores(m);
        }
    }

    // the terms of what is in s
    __device__ __forceinline__ void terms(const at_f32x16 (&s)[KT], x8 (&pf)[TERMS][2 * KT])
    {
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                float x = s[t][j];
                if constexpr (TERMS > 1) asm volatile("" : "+v"(x));  // (one rounding of a product behind it for both terms)
                const T first = static_cast<T>(x);
                pf[0][2 * t + (j >> 3)][j & 7] = first;
                if constexpr (TERMS > 1) pf[1][2 * t + (j >> 3)][j & 7] = static_cast<T>(x - static_cast<float>(first));
            }
    }

    // 16-bit caches
    __device__ __forceinline__ void weights(at_f32x16 (&s)[KT], float c, x8 (&pf)[TERMS][2 * KT])
    {
        const float ms = m == -__builtin_inff() ? 0.0f : m;
        float mul = c;
        if (large) {
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int j = 0; j < 16; ++j) s[t][j] *= c;
            mul = 1.0f;
        }
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                s[t][j] = __builtin_amdgcn_exp2f(fmaf(s[t][j], mul, -ms));
                if constexpr (TERMS > 1) {
                    if ((j & 1) == 0) l += s[t][j];
                    else l2 += s[t][j];
                }
            }
        terms(s, pf);
        if constexpr (TERMS == 1) {
#pragma unroll
            for (int u = 0; u < 2 * KT; u += 2) {
                l = add_weights<T>(pf[0][u], l);
                l2 = add_weights<T>(pf[0][u + 1], l2);
            }
        }
    }

    // int8 caches: weights times steps; rescale(f): o's unit has become 1 / f of what it was
    template <class S, class F>
    __device__ __forceinline__ void products(bool border, at_f32x16 (&s)[KT], const HiddenKeys &hidden, int n0, int half, S vs,
                                             int of_steps, x8 (&pf)[TERMS][2 * KT], F rescale)
    {
        if (shift == -__builtin_inff()) shift = 0.0f;
        if (__ballot(shift != 0.0f) != 0) {
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int j = 0; j < 16; ++j) s[t][j] -= shift;
        }
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float p = __builtin_amdgcn_exp2f(s[t][j]);
                if ((j & 1) == 0) l += p;
                else l2 += p;
                s[t][j] = p * vs(t, j);
                if (!RUN16 && (j & 7) == 7) __builtin_amdgcn_sched_barrier(0);
            }
        if (border) {
            // a weight of nothing leaves a NaN as it is: of a step that the row does not see
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int j = 0; j < 16; ++j) s[t][j] = hidden.beside_gap(n0 + key(t, j, half)) ? 0.0f : s[t][j];
        }
        if (border || __ballot(unit != of_steps) != 0) {
            float top = s[0][0];
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int j = 0; j < 16; ++j) top = fmaxf(top, s[t][j]);
            top = lane_pair_max<32>(top);
            // (2^e above the largest)
            const int need = static_cast<int>(__builtin_bit_cast(uint32_t, top) >> 23) - 126 - 15 + of_steps;
            const int next = max(need, min(of_steps, need + 12));
            if (next > unit) {
                rescale(ldexpf(1.0f, unit - next));
                unit = next;
            }
            const int by = of_steps - unit;
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int j = 0; j < 16; ++j) s[t][j] = ldexpf(s[t][j], by);
        }
        terms(s, pf);
    }
};

}  // namespace
}  // namespace ptq1
