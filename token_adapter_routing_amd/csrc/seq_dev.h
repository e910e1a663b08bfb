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

// Sum over lanes 0..15, uniform.
template <int CTRL>
__device__ __forceinline__ int row_ror(int v) {
  return __builtin_amdgcn_update_dpp(v, v, CTRL, 0xf, 0xf, true);
}
__device__ __forceinline__ int row_sum16(int v) {
  v += row_ror<0x128>(v);
  v += row_ror<0x124>(v);
  v += row_ror<0x122>(v);
  return __builtin_amdgcn_readfirstlane(v + row_ror<0x121>(v));
}

// Row range of one sequence, limited to [0, T].
struct SeqRange {
  int lo, n;
};
__device__ __forceinline__ SeqRange seq_range(const int32_t* __restrict__ off, int s, int T) {
  const int a = min(max(off[s], 0), T), b = min(max(off[s + 1], 0), T);
  return {a, max(b - a, 0)};
}

// The tile of one slot of a packed batch, tiles of `tile` rows of the first or the second of two
// offset arrays: sequence, first row in it, both row ranges.
struct SeqTile {
  int s, row0;
  SeqRange a, b;
  bool ok;
};

// Up to kLevels sequences: the longest tiles of all sequences come first, by how many tiles lie between a
// tile and its sequence's shortest end (workgroups start in slot order, so long ones do not come last and
// the first ones are spread over the CUs).  FROM_END: a sequence's last tile is its longest.  The level of
// a slot is found by halving, a sum over 16 lanes per step (4 x 2048 tokens, 16 heads of 64: 64 us
// forward and 182 us backward sequence by sequence, 55 and 156 us by level).
// With more, slots run through the sequences (attn_slot0), which are then short beside the batch, and the
// tiles of one, which read the same rows, run together (32 x 512 tokens, 16 heads of 128: 77 and 257 us, by
// level 85 and 279 us).  Up to 64 the lanes hold one each.
constexpr int kLevels = 16;
template <bool OF_A, bool FROM_END, int TILE>
__device__ __forceinline__ SeqTile find_tile(const int32_t* __restrict__ offa, int Ta, const int32_t* __restrict__ offb,
                                             int Tb, int n_seq, int slots, int slot) {
  SeqTile t{};
  if (n_seq > kWave) {
    if (FROM_END) slot = slots - 1 - slot;
    const int32_t* off = OF_A ? offa : offb;
    const int T = OF_A ? Ta : Tb;
    const int s = __builtin_amdgcn_readfirstlane(
        wave_search(n_seq, slot, [&](int i) { return attn_slot0(min(max(off[i], 0), T), i, TILE); }));
    if (s < 0) return t;
    const SeqRange a = seq_range(offa, s, Ta), b = seq_range(offb, s, Tb);
    t.a = {__builtin_amdgcn_readfirstlane(a.lo), __builtin_amdgcn_readfirstlane(a.n)};
    t.b = {__builtin_amdgcn_readfirstlane(b.lo), __builtin_amdgcn_readfirstlane(b.n)};
    t.s = s;
    const long long row0 = (slot - attn_slot0(OF_A ? t.a.lo : t.b.lo, s, TILE)) * TILE;
    t.ok = row0 >= 0 && row0 < (OF_A ? t.a.n : t.b.n);
    t.row0 = (int)row0;
    return t;
  }
  const int lane = threadIdx.x & 63;
  SeqRange a{0, 0}, b{0, 0};
  if (lane < n_seq) {
    a = seq_range(offa, lane, Ta);
    b = seq_range(offb, lane, Tb);
  }
  const SeqRange mine = OF_A ? a : b;
  const int n = (mine.n + TILE - 1) / TILE;
  int s, tile;
  if (n_seq <= kLevels) {
    // level l of a tile: how many of its sequence, itself included, are as long or shorter; above(l): how
    // many tiles of all have a higher one
    auto above = [&](int l) { return row_sum16(max(n - l, 0)); };
    if (slot >= above(0)) return t;
    int lo = 0, hi = 1;  // in the end above(lo) > slot >= above(hi), hi = lo + 1
    while (above(hi) > slot) {
      lo = hi;
      hi *= 2;
    }
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (above(mid) > slot) lo = mid;
      else hi = mid;
    }
    uint64_t here = __ballot(n >= hi);
    for (int skip = slot - above(hi); skip > 0; --skip) here &= here - 1;
    s = __builtin_ctzll(here);
    tile = FROM_END ? hi - 1 : __builtin_amdgcn_readlane(n, s) - hi;
  } else {
    if (FROM_END) slot = slots - 1 - slot;
    const int first = (int)attn_slot0(mine.lo, lane, TILE);
    const uint64_t here = __ballot(lane < n_seq && first <= slot && slot < first + n);
    if (here == 0) return t;
    s = __builtin_ctzll(here);
    tile = slot - __builtin_amdgcn_readlane(first, s);
  }
  t.s = s;
  t.row0 = tile * TILE;
  t.a = {__builtin_amdgcn_readlane(a.lo, s), __builtin_amdgcn_readlane(a.n, s)};
  t.b = {__builtin_amdgcn_readlane(b.lo, s), __builtin_amdgcn_readlane(b.n, s)};
  t.ok = true;
  return t;
}

// What the queries of one sequence see: the query at position p key j when j <= p and (window == 0 or
// j > p - window or j < sinks).
struct Mask {
  int shift;   // position of query i: i + shift
  int window;  // 0: none
  int sinks;
};

}  // namespace molora
