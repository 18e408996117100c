// ptq1_chunk.h -- which keys the rows of a tile see in the attention of chunks
// over the cache, and how tiles are cut along them: plain arithmetic for the
// host, the kernels, and a test on the CPU.
#pragma once
#include <cstdint>

namespace ptq1 {

constexpr int kChunkRows = 128;   // query rows of a tile
constexpr int kChunkKeys = 64;    // keys of one step
constexpr int kChunkMinSteps = 4; // steps of a piece, at least (1 or 2 where rows are few: 705 keys 20.0 and 16.4 us for 16.1)

constexpr int imax(int a, int b) { return a > b ? a : b; }
constexpr int imin(int a, int b) { return a < b ? a : b; }

// What a query at position p sees, of `sinks` first tokens and a window (no
// window: one that is longer than any sequence): the keys j with j < hi and (j
// >= lo or j < sinks).
struct SeenKeys {
    int lo, hi;
};
constexpr SeenKeys seen_keys(int p, int window)
{
    return {imax(0, p + 1 - window), imax(0, p + 1)};
}

// The steps of a tile whose rows stand at positions first .. last: step i has
// the keys step_key(i) .., real ones numbered through with `gap` steps between
// the first tokens' and the windows' left out.
struct ChunkSteps {
    int lo, reach, sunk;   // keys that some row sees: [lo, reach), and below sunk
    int head, gap;         // from step `head` on, `gap` steps further
    int steps;
    int all_from, all_to;  // every row sees every key of these steps
};
constexpr ChunkSteps chunk_steps(int first, int last, int window, int sinks)
{
    constexpr int N = kChunkKeys;
    ChunkSteps c{};
    c.lo = seen_keys(first, window).lo;
    c.reach = seen_keys(last, window).hi;
    c.sunk = imin(sinks, c.reach);
    const int begin = c.lo / N;
    c.head = c.lo > 0 ? (c.sunk + N - 1) / N : 0;
    c.gap = imax(0, begin - c.head);
    c.steps = imax(0, (c.reach + N - 1) / N - c.gap);
    const SeenKeys late = seen_keys(last, window), early = seen_keys(first, window);
    c.all_from = (late.lo + N - 1) / N - c.gap;
    c.all_to = early.hi / N - c.gap;
    if (c.all_to < c.all_from) c.all_to = c.all_from;
    return c;
}
constexpr int step_key(const ChunkSteps &c, int i) { return kChunkKeys * (i < c.head ? i : i + c.gap); }

// No tile of a sequence of `len` tokens has more steps (a tile's rows are of
// (kChunkRows - 1) / group + 2 tokens at most).
constexpr int steps_bound(int len, int window, int sinks, int group)
{
    const int all = (len + kChunkKeys - 1) / kChunkKeys;
    const int64_t span = static_cast<int64_t>(window) + (kChunkRows - 1) / group + 1;
    const int64_t some = (span + 2 * kChunkKeys - 2) / kChunkKeys + (static_cast<int64_t>(sinks) + kChunkKeys - 1) / kChunkKeys;
    return len <= 0 ? 0 : some < all ? static_cast<int>(some) : all;
}

// Steps of one piece where the tiles' steps are `total` in all and `wanted`
// pieces fill the GPU.
constexpr int chunk_piece(int total, int wanted) { return imax(kChunkMinSteps, (total + wanted - 1) / wanted); }

// What `tiles` of `steps` each, cut in n pieces, take where `wanted` run side by
// side, in steps (join_cost and piece_cost too); negative: too many pieces (twice
// `wanted` at most), or too short ones.
constexpr float chunk_cost(int n, int tiles, int steps, int wanted, float join_cost, float piece_cost)
{
    const int per = (steps + n - 1) / n;
    if (n > 1 && (static_cast<int64_t>(tiles) * n > 2 * static_cast<int64_t>(wanted) || per < kChunkMinSteps)) return -1.0f;
    return static_cast<float>((tiles * n + wanted - 1) / wanted * per) + (n > 1 ? join_cost + piece_cost * static_cast<float>(tiles * n) : 0.0f);
}
// The numbers of pieces that are considered, by lane: 1 to 15, then eight of
// each power of two, up to 960.
constexpr int chunk_cut_of(int lane) { return lane < 8 ? lane + 1 : (8 + (lane & 7)) << ((lane >> 3) - 1); }

constexpr int chunk_pieces(int steps, int per) { return imax(1, (steps + per - 1) / per); }

}  // namespace ptq1
