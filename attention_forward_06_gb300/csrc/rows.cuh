// rows.cuh -- writing a warp's rows, one per lane, in whole cache lines.
#pragma once

#include <cstdint>

namespace attn {

// A warp store of one 16-byte chunk per lane touches 32 rows (32 cache lines) when each lane holds
// a row.  This transposes the chunks within each group of CH lanes (log2 CH butterfly stages of
// shuffles, each swapping one bit between lane and chunk index): lane m held its row's CH chunks in
// w[0 .. 4 CH); after it lane CH g + q holds chunk q of rows CH g .. CH g + CH - 1, so that each of CH
// stores writes 32 / CH whole rows.
template <int CH>
__device__ __forceinline__ void transpose_chunks(uint32_t (&w)[4 * CH], int lane) {
  const int q = lane % CH;
#pragma unroll
  for (int b = CH / 2; b >= 1; b /= 2) {
    const bool hi = (q & b) != 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (c & b) continue;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const uint32_t send = hi ? w[4 * c + h] : w[4 * (c ^ b) + h];
        const uint32_t recv = __shfl_xor_sync(0xffffffffu, send, b);
        if (hi)
          w[4 * c + h] = recv;
        else
          w[4 * (c ^ b) + h] = recv;
      }
    }
  }
}

// Stores 32 rows of a warp, one row per lane (lane m holds its row's CH 16-byte chunks in
// w[0 .. 4 CH)), row m at base + m * stride; rows m >= live_rows are skipped.
template <int CH>
__device__ __forceinline__ void store_warp_rows(uint32_t (&w)[4 * CH], uint8_t* base, int64_t stride, int live_rows,
                                                int lane) {
  transpose_chunks<CH>(w, lane);
  const int q = lane % CH;
  const int m0 = lane - q;
#pragma unroll
  for (int k = 0; k < CH; ++k)
    if (m0 + k < live_rows)
      *reinterpret_cast<uint4*>(base + (m0 + k) * stride + 16 * q) =
          make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
}

}  // namespace attn
