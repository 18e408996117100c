// ptq1_split.h -- how the decode attention cuts sequences into pieces: plain
// arithmetic for the host, the kernels, and a test on the CPU.
#pragma once
#include <cstdint>

namespace ptq1 {

constexpr int kStep = 256;           // tokens of one step of the split (one page or several)
constexpr int kMaxSteps = 1 << 14;   // steps of a sequence (of 2^22 tokens)

// Steps of a sequence: one at least (an empty or refused one has its rows
// written too).  All sequences' together are at most 2^30 (2^16 times 2^14).
constexpr int decode_steps(int len, int64_t max_len)
{
    return len <= 0 || len > max_len ? 1 : (len + kStep - 1) / kStep;
}

// Few sequences: pieces that fill the GPU once (`shares` workgroups of a kv
// head).  Many: half of that, since their ends leave the pieces unequal (64
// sequences of 3 to 8190 tokens: 61 us with 512 tokens a piece, 71 with 256,
// 75 with 2048; one of 131071 over int8: 64 us in one round of 2048, 75 in
// two).
constexpr int64_t wanted_pieces(int64_t batch, int64_t shares)
{
    return batch * 2 <= shares ? shares : 2 * shares;
}

// Steps of one piece, of `total` in all sequences.  No sequence has more than
// kMaxSteps, so no piece needs to (and its tokens fit 32 bits).
constexpr int steps_per_piece(int total, int64_t wanted)
{
    const int want = static_cast<int>(wanted), per = (total + want - 1) / want;
    return per < kMaxSteps ? per : kMaxSteps;
}

constexpr int pieces_of(int steps, int per) { return (steps + per - 1) / per; }

// The tokens begin .. end of a sequence's `first`-th piece.
struct PieceTokens {
    int begin, end;
};
constexpr PieceTokens piece_tokens(int first, int per, int len)
{
    const int begin = first * per * kStep;
    return {begin, begin + per * kStep < len ? begin + per * kStep : len};
}

}  // namespace ptq1
