// The cache held in 4 bits: where a value's code, scale and lo lie.
//
// A value is scale * code + lo, with a scale and a lo (fp16) for each token, key
// head and 32 channels.  The pages of one key head are rows of blocks of 16
// tokens and C = min(head dim, 128) channels, codes first (8 C bytes), then
// scales and los (2 C bytes); a head of 256 is two of them side by side, so that
// 16 tokens always take 10 head_dim bytes.  A word is the codes of 8 channels,
// slots 0 to 7 (low bits first) those of channels 0 2 4 6 1 3 5 7: a shift and a
// mask give two neighbours as a pair.
//
//   keys    words [token][(channel / 8) % 4][channel / 32]
//           params [token][channel / 32][scale, lo]
//   values  words [token / 4][channel / 8][token % 4]
//           params [token / 4][channel / 32][scale, lo][token % 4]
//
// Both orders are what a lane of the attention's matrix instructions reads in 16
// bytes: of the keys, the four words whose channels it multiplies in four
// instructions, of the values, one column of 8 channels of four tokens, which it
// turns into pairs of tokens.  A word is one token's in both, so that a token is
// written without reading its neighbours.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ttq {

constexpr int kPackGroup = 32;       // channels of a scale
constexpr float kPackMost = 32768.f;  // larger values saturate: scale * 15 + lo stays an fp16 number

// Word of channels 8 v .. 8 v + 7 of token t (of 16) in the blocks of 16 tokens
// of a head: its byte.
template <bool KEYS>
__host__ __device__ inline int packed_word(int dim, int t, int v) {
  const int c = dim < 128 ? dim : 128, block = v / (c / 8) * 10 * c;
  v %= c / 8;
  return block + 4 * (KEYS ? t * (c / 8) + v % 4 * (c / 32) + v / 4 : (t / 4 * (c / 8) + v) * 4 + t % 4);
}
// Scale of the same channels; the lo lies kPackLo bytes further.
template <bool KEYS>
__host__ __device__ inline int packed_scale(int dim, int t, int v) {
  const int c = dim < 128 ? dim : 128, block = v / (c / 8) * 10 * c;
  v %= c / 8;
  return block + 8 * c + (KEYS ? (t * (c / 32) + v / 4) * 4 : (t / 4 * (c / 32) + v / 4) * 16 + t % 4 * 2);
}
template <bool KEYS>
constexpr int kPackLo = KEYS ? 2 : 8;

}  // namespace ttq
