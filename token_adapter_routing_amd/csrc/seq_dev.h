// Device helpers of the kernels that work on packed sequences.
#pragma once

#include "molora_dev.h"

namespace molora {

typedef __attribute__((__vector_size__(16 * sizeof(float)))) float f32x16_t;
typedef __attribute__((__vector_size__(4 * sizeof(short)))) short s16x4_t;

// D = A B + C, A 32x16, B 16x32, D 32x32.  A: lane l row l % 32, B: lane l column l % 32, both
// k-slots 8 (l / 32) .. + 7; D: lane l column l % 32, register r row r % 4 + 8 (r / 4) + 4 (l / 32).
__device__ __forceinline__ f32x16_t mfma32x32x16(bf16x8_t a, bf16x8_t b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The largest s in [0, n) with key(s) <= x for a non-decreasing key, by the whole wave: every step
// looks at 64 places, so up to 4096 sequences take two loads.  -1 when key(0) > x.  With keys out
// of order (offsets that do not ascend) the result is some s in [-1, n).
template <typename Key>
__device__ __forceinline__ int wave_search(int n, long long x, Key key) {
  const int lane = threadIdx.x & 63;
  int lo = 0;
  for (;;) {
    const int stride = (n + kWave - 1) / kWave;
    const int at = lane * stride;
    const uint64_t below = __ballot(at < n && key(lo + at) <= x);
    const int cnt = __popcll(below);
    if (cnt == 0) return lo - 1 < 0 ? -1 : lo;
    lo += (cnt - 1) * stride;
    if (stride == 1) return lo;
    n = min(stride, n - (cnt - 1) * stride);
  }
}

// Tiles of up to 64 sequences, the longest sequence first: lane s holds sequence s's number of tiles
// (0 past the last).  The sequence of the rank-th tile, -1 past the last, and in *tile its place in
// the sequence.
__device__ __forceinline__ int ranked_tile(int n, int n_seq, long long rank, int* tile) {
  const int lane = threadIdx.x & 63;
  long long first = 0;  // tiles of the sequences before this one
  for (int s = 0; s < n_seq; ++s) {
    const int m = __builtin_amdgcn_readlane(n, s);
    if (m > n || (m == n && s < lane)) first += m;
  }
  const uint64_t mine = __ballot(n > 0 && first <= rank && rank < first + n);
  if (mine == 0) return -1;
  const int s = __builtin_ctzll(mine);
  *tile = __builtin_amdgcn_readlane((int)(rank - first), s);
  return s;
}

// Row range of sequence s, limited to [0, T].
struct SeqRange {
  int lo, n;
};
__device__ __forceinline__ SeqRange seq_range(const int32_t* __restrict__ off, int s, int T) {
  const int a = min(max(off[s], 0), T), b = min(max(off[s + 1], 0), T);
  return {__builtin_amdgcn_readfirstlane(a), __builtin_amdgcn_readfirstlane(max(b - a, 0))};
}

// What the queries of one sequence see.
struct Mask {
  int shift;   // position of query i: i + shift
  int window;  // 0: none
  int sinks;
  __device__ __forceinline__ bool sees(int p, int j) const {
    return j <= p && (window == 0 || j > p - window || j < sinks);
  }
};

}  // namespace molora
