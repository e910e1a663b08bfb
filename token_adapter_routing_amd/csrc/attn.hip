// Causal attention over packed sequences with a window and sink tokens, forward and backward.
//
//   forward   S = scale Q K^T over the visible pairs, O = softmax(S) V, lse = log sum exp S
//   backward  P = exp(S - lse), dV = P^T dO, dP = dO V^T, dS = P (dP - rowsum(dO O)),
//             dQ = scale dS K, dK = scale dS^T Q
//
// One pass over the keys per query tile with the running maximum and sum of the softmax; S, P and
// dS exist only in registers.  Products run on 32x32x16 bf16 matrix instructions, arranged so
// that a product's result is the next one's operand as it stands: the forward computes S^T (keys
// down, queries across), so a lane holds 16 keys of one query, the softmax's maximum and sum are
// sums over registers and one exchange between the wave's halves, and P^T, rounded to bf16, is
// the right operand of O^T = V^T P^T.  The operand that has to be read along its columns (V, and
// in the backward K, Q, dO) comes from LDS through the transposing 8-byte read.
//
// Tiles lie in LDS as rows of D values whose 16-byte pieces are permuted by the row (Tile::off),
// so that both the row reads (32 rows, one piece each) and the transposing reads (4 rows, four
// neighbouring pieces each) touch every bank once.
#include <cmath>

#include "decoder_launch.h"
#include "seq_dev.h"

namespace molora {

namespace {

constexpr int kBN = 64;  // keys per LDS tile of the forward and the dq pass

template <int D>
struct Tile {
  static constexpr int kRow = 2 * D;        // bytes
  static constexpr int kPieces = D / 8;     // 16-byte pieces per row
  static __device__ __forceinline__ int swz(int row) {
    if constexpr (D == 128) return ((row & 3) << 2) | ((row >> 2) & 3);
    else return (((row >> 1) & 1) << 2) | ((row >> 2) & 3);
  }
  static __device__ __forceinline__ int off(int row, int piece) { return row * kRow + ((piece ^ swz(row)) << 4); }
};

// Asynchronous copy of ROWS rows of a packed tensor into an LDS tile, straight from global memory: an
// instruction fills 1 KiB of LDS in lane order, so the lanes pick the global pieces that the tile's
// permutation puts there.  Rows past `last` repeat row `last`.  The data is there after
// tiles_ready().
template <int D, int ROWS>
struct Fetch {
  static constexpr int kRows = 1024 / Tile<D>::kRow;    // rows per instruction
  static constexpr int kN = ROWS / kRows / 4;           // instructions per wave
  uint32_t row[kN], col[kN];
  __device__ __forceinline__ void init(int lane, int wave) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int r = (4 * i + wave) * kRows + lane / Tile<D>::kPieces;
      row[i] = r;
      col[i] = 16 * ((lane % Tile<D>::kPieces) ^ Tile<D>::swz(r));
    }
  }
  // stride in bytes
  __device__ __forceinline__ void operator()(char* __restrict__ lds, const uint16_t* base, long long stride, int row0,
                                             int last, int wave) const {
    const char* p = reinterpret_cast<const char*>(base) + row0 * stride;
    const uint32_t left = last - row0;
#pragma unroll
    for (int i = 0; i < kN; ++i)
      __builtin_amdgcn_global_load_lds(
          (const __attribute__((address_space(1))) void*)(p + (min(row[i], left) * (uint32_t)stride + col[i])),
          (__attribute__((address_space(3))) void*)(lds + (4 * i + wave) * 1024), 16, 0, 0);
  }
};

// This wave's copies into LDS have arrived, then everyone's.
__device__ __forceinline__ void tiles_ready() {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
}

// Lane's places in any tile.  The permutation XORs row bits 0..3 into the piece, so neighbouring
// operands are an XOR and a constant apart: row operands st differ in piece bits 1.., column operands
// in piece bits 2.. (mb) and, eight rows on, in piece bit 1.
struct LaneOff {
  uint32_t row, col;
};
template <int D>
__device__ __forceinline__ LaneOff lane_off(int lane) {
  const int h = lane >> 5, q = lane & 15, c = (lane & 16) + 4 * (q & 3);
  return {(uint32_t)Tile<D>::off(lane & 31, h), (uint32_t)(Tile<D>::off(4 * h + (q >> 2), c >> 3) + (c & 4) * 2)};
}

// Left operand (rows down): rows row0 + lane % 32 (row0 a multiple of 16), values 16 st + 8 h .. + 7.
template <int D>
__device__ __forceinline__ bf16x8_t row_frag(const char* lds, LaneOff o, int row0, int st) {
  return as_bf16x8(ld16(lds + ((o.row ^ (st << 5)) + row0 * Tile<D>::kRow)));
}

// Left operand (columns down): column 32 mb + lane % 32 of the tile; k-slots 0..3 are rows
// row0 + 4 h + 0..3 (row0 a multiple of 16), k-slots 4..7 rows row0 + 8 + 4 h + 0..3, the order in
// which a 32x32 result holds its rows.  Each group of 16 lanes reads a 4 x 16 block and gets its
// columns.
template <int D>
__device__ __forceinline__ bf16x8_t col_frag(const char* lds, LaneOff o, int row0, int mb) {
  typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;
  const char* a = lds + ((o.col ^ (mb << 6)) + row0 * Tile<D>::kRow);
  const char* b = lds + ((o.col ^ (mb << 6) ^ 32) + (row0 + 8) * Tile<D>::kRow);
  union {
    s16x4_t s[2];
    bf16x8_t v;
  } u;
  u.s[0] = __builtin_bit_cast(s16x4_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)a));
  u.s[1] = __builtin_bit_cast(s16x4_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)b));
  return u.v;
}

// Schedule of a run of N steps of M products, each step with R operand reads from LDS: the reads of A
// steps go ahead, so that a product does not wait for the read before it.
template <int N, int M, int R, int A>
__device__ __forceinline__ void reads_ahead() {
  __builtin_amdgcn_sched_group_barrier(0x100, A * R, 0);
#pragma unroll
  for (int i = 0; i < N - A; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, M, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, R, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, A * M, 0);
}

// Right operand from registers: rows 16 s .. + 15 of a 32x32 result, rounded to bf16.
__device__ __forceinline__ bf16x8_t acc_frag(const f32x16_t& v, int s) {
  u32x4_t u;
#pragma unroll
  for (int i = 0; i < 4; ++i) u[i] = pack_bf16x2(v[8 * s + 2 * i], v[8 * s + 2 * i + 1]);
  return as_bf16x8(u);
}

// What acc_frag rounded away, as bf16 again: together they hold 16 bits of the value.
__device__ __forceinline__ bf16x8_t acc_rest(const f32x16_t& v, int s, bf16x8_t hi) {
  u32x4_t u;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    u[i] = pack_bf16x2(v[8 * s + 2 * i] - (float)hi[2 * i], v[8 * s + 2 * i + 1] - (float)hi[2 * i + 1]);
  return as_bf16x8(u);
}

__device__ __forceinline__ int acc_row(int r, int h) { return (r & 3) + 8 * (r >> 2) + 4 * h; }

// Key tiles a query tile visits: the sinks' first, then the window's.
struct KeyTiles {
  int sink, lo, n;
  __device__ __forceinline__ int at(int i) const { return (i < sink ? i : lo + i - sink) * kBN; }
};
__device__ __forceinline__ KeyTiles key_tiles(const Mask& m, int p_lo, int p_hi, int Lk) {
  KeyTiles t;
  const int hi = min(p_hi + 1, Lk);  // keys below hi may be seen
  const int first = m.window ? max(p_lo - m.window + 1, 0) : 0;
  t.lo = first / kBN;
  t.sink = m.window ? min((min(m.sinks, max(hi, 0)) + kBN - 1) / kBN, t.lo) : 0;
  t.n = t.sink + max((hi + kBN - 1) / kBN - t.lo, 0);
  if (hi <= 0) t.n = 0;
  return t;
}

// Scores of one lane's query at position p against keys j0 + acc_row(i, h) of a 32x32 result: -inf
// where it does not see the key.  Everything is taken relative to the lane's first key, so that each
// score costs a comparison with a constant or three.
__device__ __forceinline__ void hide(f32x16_t& s, const Mask& m, int p, int j0, int h) {
  const int last = p - j0 - 4 * h;
  if (m.window == 0) {
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = acc_row(i, 0) <= last ? s[i] : -INFINITY;
  } else {
    const int first = last - m.window, sinks = m.sinks - j0 - 4 * h;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int r = acc_row(i, 0);
      s[i] = r <= last && (r > first || r < sinks) ? s[i] : -INFINITY;
    }
  }
}

// Whether rows at positions [p_lo, p_hi] see nothing, or everything, of keys [j0, j1].
__device__ __forceinline__ bool sees_none(const Mask& m, int p_lo, int p_hi, int j0, int j1) {
  return j0 > p_hi || (m.window && j1 <= p_lo - m.window && j0 >= m.sinks);
}
__device__ __forceinline__ bool sees_all(const Mask& m, int p_lo, int p_hi, int j0, int j1) {
  return j1 <= p_lo && (!m.window || j0 > p_hi - m.window || j1 < m.sinks);
}

// ---- Rows taken again.  A hidden pair has weight 0, but 0 times an infinity or a NaN is NaN, so a row of
// sums that is not finite may owe it to a row that it does not see and that shares a tile with one
// that it does.  Its columns that are not finite are summed again over the visible pairs alone, a lane
// per pair for the weights and then a lane per column.  Columns with such a value in a tile that the
// whole wave sees are lost for good: one pass over those tiles leaves them out, so that only the rows
// around a bad one are taken again.  Finite inputs never come here; the test itself is within the spread
// of the measurements (train batch 270 us without it, 268 us with it).

// The workgroup's number and the kernel's first argument, read afresh where rows are taken again:
// otherwise all they lead to would be kept in scalar registers, and spilled, while the products run (8192
// tokens, 32 / 8 heads of 128: dq and dk / dv 780 + 1254 us with it kept, 740 + 1144 us read afresh).
__device__ __forceinline__ unsigned group_again() {
  unsigned id = blockIdx.x;
  asm volatile("" : "+s"(id));
  return id;
}
template <typename Args>
__device__ __forceinline__ const Args& args_again() {
  auto p = __builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const Args*)(const void*)p;
}

// Rows of a 32 x D block held as D x 32 that are not finite (bit per row).
template <int D>
__device__ __forceinline__ uint32_t odd_rows(const f32x16_t* acc, bool mine) {
  float zero[D / 32];  // 0 times a finite value; NaN otherwise
#pragma unroll
  for (int mb = 0; mb < D / 32; ++mb) {
    zero[mb] = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) zero[mb] = fmaf(acc[mb][i], 0.f, zero[mb]);
  }
#pragma unroll
  for (int mb = 1; mb < D / 32; ++mb) zero[0] += zero[mb];
  const uint64_t b = __ballot(mine && zero[0] != zero[0]);
  return (uint32_t)(b | (b >> 32));
}

__device__ __forceinline__ bool sees(const Mask& m, int p, int j) {
  return j <= p && (!m.window || j > p - m.window || j < m.sinks);
}

template <int D>
__device__ __forceinline__ float dot_rows(const uint16_t* x, const uint16_t* y) {
  float s = 0.f;
#pragma unroll 4
  for (int i = 0; i < D; i += 8) {
    const u32x4_t u = ld16(x + i), v = ld16(y + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s = fmaf(bf16_to_f32(u[e] & 0xffffu), bf16_to_f32(v[e] & 0xffffu), s);
      s = fmaf(bf16_to_f32(u[e] >> 16), bf16_to_f32(v[e] >> 16), s);
    }
  }
  return s;
}

__device__ __forceinline__ float lane_value(float v, int i) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), i));
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }

// The lane's D / 64 columns (bits) in which one of the first n rows of `base` is not finite.
template <int D>
__device__ __forceinline__ uint32_t odd_columns(const uint16_t* base, long long stride, int n, int lane) {
  uint32_t odd = 0;
#pragma unroll 8
  for (int i = 0; i < n; ++i)
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      odd |= (uint32_t)((base[i * stride + D / 64 * lane + c] & 0x7f80) == 0x7f80) << c;
  return odd;
}

// The lane's columns of a stored row that are not finite and not lost.
template <int D, typename T>
__device__ __forceinline__ uint32_t to_repair(const T* row, uint32_t lost, int lane) {
  uint32_t odd = 0;
#pragma unroll
  for (int c = 0; c < D / 64; ++c) {
    const T v = row[D / 64 * lane + c];
    if constexpr (sizeof(T) == 2) odd |= (uint32_t)!finite(bf16_to_f32(v)) << c;
    else odd |= (uint32_t)!finite(v) << c;
  }
  return odd & ~lost;
}

// One row of sums, D / 64 columns per lane.
template <int D>
struct RowSum {
  float x[D / 64] = {};
  // Adds w times row i of `base` for every lane i of `who`.
  __device__ __forceinline__ void add(uint64_t who, float w, const uint16_t* base, long long stride, int lane) {
    for (; who; who &= who - 1) {
      const int i = __builtin_ctzll(who);
      const float f = lane_value(w, i);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) x[c] = fmaf(f, bf16_to_f32(base[i * stride + D / 64 * lane + c]), x[c]);
    }
  }
  // The columns of `odd`.
  __device__ __forceinline__ void store(uint16_t* row, float mul, uint32_t odd, int lane) const {
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      if (odd >> c & 1) row[D / 64 * lane + c] = (uint16_t)pack_bf16x2(x[c] * mul, 0.f);
  }
  __device__ __forceinline__ void store(float* row, float, uint32_t odd, int lane) const {
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      if (odd >> c & 1) row[D / 64 * lane + c] = x[c];
  }
};

// Workgroup -> (head, slot, chunk of the slot's key tiles): the heads of one key-value head follow each
// other on one XCD (consecutive workgroups go round the XCDs); the chunk is the slowest, so that
// workgroups without work lie together at the end.
struct Place {
  int hq, hk, slot, chunk;
};
__device__ __forceinline__ Place place(const AttnArgs& a, int slots, unsigned id) {
  const unsigned g = a.Hq / a.Hkv, rest = id / a.Hkv, hk = id % a.Hkv, at = rest / g;
  const unsigned chunk = at / slots;
  return {(int)(hk * g + rest % g), (int)hk, (int)(at - chunk * slots), (int)chunk};
}

// A query tile's key tiles split over up to `splits` workgroups, at least kAttnMinTiles each; without a
// window by the sequence's longest tile, so that its chunks are equally long.
struct Chunks {
  int per, n;
};
__device__ __forceinline__ Chunks key_chunks(const Mask& m, int tiles, int Lk, int splits) {
  const int longest = m.window ? tiles : (Lk + kBN - 1) / kBN;
  const int per = max((longest + splits - 1) / splits, kAttnMinTiles);
  return {per, max((tiles + per - 1) / per, 1)};
}

// A workgroup's query tile and its chunk of the key tiles.
struct QTile {
  Mask m;
  KeyTiles kt;
  int hq, hk, slot, chunk, chunks, it0, it1;
  int q0, k0, Lk, last, row0;  // first rows of the sequence, keys, last query, tile's first query
  bool ok;
  // The lane's columns of `base` that are not finite in a key tile which all of the wave's rows see.
  template <int D>
  __device__ __forceinline__ uint32_t lost_columns(const uint16_t* base, long long stride, int wave, int lane) const {
    const int r0 = row0 + 32 * wave, p_lo = r0 + m.shift, p_hi = min(r0 + 31, last) + m.shift;
    uint32_t odd = 0;
    for (int it = it0; it < it1; ++it) {
      const int j0 = kt.at(it);
      if (sees_all(m, p_lo, p_hi, j0, j0 + kBN - 1)) odd |= odd_columns<D>(base + j0 * stride, stride, kBN, lane);
    }
    return odd;
  }
};
__device__ __forceinline__ QTile q_tile(const AttnArgs& a, int slots, unsigned id, int splits) {
  QTile x{};
  const Place pl = place(a, slots, id);
  const SeqTile t = find_tile<true, true, kAttnQ>(a.q_off, a.Tq, a.kv_off, a.Tkv, a.n_seq, slots, pl.slot);
  if (!t.ok) return x;
  x.hq = pl.hq, x.hk = pl.hk, x.slot = pl.slot, x.chunk = pl.chunk;
  x.q0 = t.a.lo, x.k0 = t.b.lo, x.Lk = t.b.n, x.last = t.a.n - 1, x.row0 = t.row0;
  x.m = Mask{x.Lk - t.a.n, a.window, a.sinks};
  x.kt = key_tiles(x.m, x.row0 + x.m.shift, min(x.row0 + kAttnQ - 1, x.last) + x.m.shift, x.Lk);
  const Chunks ch = key_chunks(x.m, x.kt.n, x.Lk, splits);
  x.chunks = ch.n;
  x.it0 = x.chunk * ch.per;
  x.it1 = min(x.it0 + ch.per, x.kt.n);
  x.ok = x.chunk < ch.n;
  return x;
}

// Stores a 32 x D block held as D x 32 as fp32 rows of D.
template <int D>
__device__ __forceinline__ void store_part(float* row, const f32x16_t* acc, int h) {
#pragma unroll
  for (int mb = 0; mb < D / 32; ++mb)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      f32x4_t v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = acc[mb][4 * g + i];
      *reinterpret_cast<f32x4_t*>(row + 32 * mb + 8 * g + 4 * h) = v;
    }
}

// Stores the first `rows` rows of a wave's 32 x D block held as D x 32 (column = row of the output), times
// the lane's `mul`.  The rows are put together in LDS (the wave's own 32 rows of a tile, which nothing else
// uses any more): written as they are held, 16 bytes of 32 rows at a time, they would cost a pass of
// partial lines per instruction (16 ragged prompts of up to 512, 16 heads of 128: 24.7 us so, 22.3 us from LDS;
// the backward of 8 of up to 2048: 236 and 225 us).
template <int D>
__device__ __forceinline__ void store_rows(char* lds, uint16_t* base, long long token, int rows, const f32x16_t* acc,
                                           float mul, int lane) {
  const int h = lane >> 5, n = lane & 31;
#pragma unroll
  for (int mb = 0; mb < D / 32; ++mb)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      uint2 v;
      v.x = pack_bf16x2(acc[mb][4 * g] * mul, acc[mb][4 * g + 1] * mul);
      v.y = pack_bf16x2(acc[mb][4 * g + 2] * mul, acc[mb][4 * g + 3] * mul);
      *reinterpret_cast<uint2*>(lds + Tile<D>::off(n, 4 * mb + g) + 8 * h) = v;
    }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  constexpr int kPieces = Tile<D>::kPieces, kStep = kWave / kPieces;
  const int piece = lane % kPieces;
#pragma unroll
  for (int i = 0; i < 32 / kStep; ++i) {
    const int row = i * kStep + lane / kPieces;
    if (row < rows) st16(base + row * token + 8 * piece, ld16(lds + Tile<D>::off(row, piece)));
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

}  // namespace

namespace {

// attn_fwd_k's rows that are taken again: the wave's rows of the bits of `again`, with the reference
// maxima and the sums' inverses that the lanes hold.
template <int D>
__device__ __forceinline__ void fwd_again(const AttnArgs& a, int slots, uint32_t again, int wave, int lane, float mx,
                                          float inv) {
  const QTile t = q_tile(a, slots, group_again(), a.splits);
  const uint16_t* kb = a.k.p + (long long)t.k0 * a.k.token + t.hk * a.k.head;
  const uint16_t* vb = a.v.p + (long long)t.k0 * a.v.token + t.hk * a.v.head;
  const float c = a.scale * kLog2e;
  const uint32_t lost = t.lost_columns<D>(vb, a.v.token, wave, lane);
  __threadfence();  // the rows are stored
  for (uint32_t left = again; left; left &= left - 1) {
    const int i = __builtin_ctz(left), at = 32 * wave + i, p = t.row0 + at + t.m.shift;
    const long long row = t.q0 + t.row0 + at;
    const uint16_t* qr = a.q.p + row * a.q.token + t.hq * a.q.head;
    const float top = lane_value(mx, i), ref = top > -INFINITY ? top : 0.f;
    auto repair = [&](auto* out) {
      const uint32_t odd = to_repair<D>(out, lost, lane);
      if (!__any(odd)) return;
      RowSum<D> x;
      for (int it = t.it0; it < t.it1; ++it) {
        const int j0 = t.kt.at(it), j = j0 + lane;
        const bool see = sees(t.m, p, j);
        const float w = see ? exp2_hw(fmaf(dot_rows<D>(qr, kb + j * a.k.token), c, -ref)) : 0.f;
        x.add(__ballot(see), w, vb + j0 * a.v.token, a.v.token, lane);
      }
      x.store(out, lane_value(inv, i), odd, lane);
    };
    if (t.chunks > 1)
      repair(a.part + ((size_t)(t.chunk * slots + t.slot) * a.Hq + t.hq) * attn_fwd_part_floats(D) + (size_t)at * D);
    else repair(a.o.p + row * a.o.token + t.hq * a.o.head);
  }
}

}  // namespace

// A workgroup: 128 queries of one head, 32 per wave; tiles of 64 keys, double-buffered.  128 queries
// because a tile of keys then feeds four waves from LDS once, and the operands, sums and scores of 32
// queries by 128 values are the 223 registers that leave two waves per SIMD; 64 keys because two
// workgroups' double buffers of K and V (64 KiB each) then fit a CU.
//
// Bound by the matrix units at the clock they leave (54 % busy at 1.8 GHz; the library's product of 8192^3
// goes to 71 % at 1.5): 8192 tokens, 32 / 8 heads of 128, 532 us = 1033 TFLOP/s, no bank conflicts; without
// copies and barriers the rest takes 479 us.  Heads of 64 do half the products per softmax, whose vector
// instructions then bound them: 4 x 4096 tokens, 16 heads 166 us = 826 TFLOP/s.  Short calls: one tile
// 8.2 us, each further 64 keys about 1.07 us.
template <int D>
__global__ __launch_bounds__(256, 2) void attn_fwd_k(AttnArgs a, int slots) {
  constexpr int kTileB = kBN * Tile<D>::kRow;
  __shared__ __attribute__((aligned(16))) char ldsK0[kTileB], ldsK1[kTileB], ldsV0[kTileB], ldsV1[kTileB];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), h = lane >> 5,
            n = lane & 31;
  const QTile t = q_tile(a, slots, blockIdx.x, a.splits);
  if (!t.ok) return;
  const Mask m = t.m;
  const KeyTiles kt = t.kt;
  const int Lk = t.Lk, q0 = t.q0, k0 = t.k0, last = t.last;
  const int it0 = t.it0, it1 = t.it1;
  const int r0 = t.row0 + 32 * wave, r = min(r0 + n, last);
  const int p = r + m.shift, p_lo = r0 + m.shift, p_hi = min(r0 + 31, last) + m.shift;
  const uint16_t* kb = a.k.p + (long long)k0 * a.k.token + t.hk * a.k.head;
  const uint16_t* vb = a.v.p + (long long)k0 * a.v.token + t.hk * a.v.head;
  bf16x8_t q[D / 16];
  {
    const uint16_t* qr = a.q.p + (long long)(q0 + r) * a.q.token + t.hq * a.q.head + 8 * h;
#pragma unroll
    for (int st = 0; st < D / 16; ++st) q[st] = as_bf16x8(ld16(qr + 16 * st));
  }
  f32x16_t o[D / 32];
#pragma unroll
  for (int mb = 0; mb < D / 32; ++mb) o[mb] = f32x16_t{};
  const float c = a.scale * kLog2e;  // the softmax in base 2
  float mx = -INFINITY, sum = 0.f;   // reference maximum of c s; the lane's part of the sum
  Fetch<D, kBN> fetch;
  fetch.init(lane, wave);
  const LaneOff lo = lane_off<D>(lane);
  const long long ks = 2 * a.k.token, vs = 2 * a.v.token;
  auto step = [&](int it, const char* __restrict__ K, const char* __restrict__ V, char* __restrict__ nextK,
                  char* __restrict__ nextV) {
    const int j0 = kt.at(it);
    if (it + 1 < it1) {
      fetch(nextK, kb, ks, kt.at(it + 1), Lk - 1, wave);
      fetch(nextV, vb, vs, kt.at(it + 1), Lk - 1, wave);
    }
    if (r0 <= last && !sees_none(m, p_lo, p_hi, j0, j0 + kBN - 1)) {
      f32x16_t s[2] = {f32x16_t{}, f32x16_t{}};
#pragma unroll
      for (int st = 0; st < D / 16; ++st)
#pragma unroll
        for (int b = 0; b < 2; ++b) s[b] = mfma32x32x16(row_frag<D>(K, lo, 32 * b, st), q[st], s[b]);
      reads_ahead<D / 16, 2, 2, 3>();
      if (!sees_all(m, p_lo, p_hi, j0, j0 + kBN - 1)) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
          hide(s[b], m, p, j0 + 32 * b, h);
      }
      float top = s[0][0];
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, s[b][i]);
      top *= c;
      // The reference follows the maximum only when it is left behind by more than 2^8: until then the
      // weights stay below 2^8, which costs no precision in floating point.
      if (__any(top > mx + 8.f)) {
        const float up = fmaxf(mx, fmaxf(top, __shfl_xor(top, 32, kWave)));
        const float f = up > -INFINITY ? exp2_hw(mx - up) : 1.f;
        mx = up;
        sum *= f;
#pragma unroll
        for (int mb = 0; mb < D / 32; ++mb)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[mb][i] *= f;
      }
      const float ref = mx > -INFINITY ? mx : 0.f;
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[b][i] = exp2_hw(fmaf(s[b][i], c, -ref));
          sum += s[b][i];
        }
#pragma unroll
      for (int st = 0; st < kBN / 16; ++st) {
        const bf16x8_t pf = acc_frag(s[st >> 1], st & 1);
#pragma unroll
        for (int mb = 0; mb < D / 32; ++mb) o[mb] = mfma32x32x16(col_frag<D>(V, lo, 16 * st, mb), pf, o[mb]);
      }
    }
    tiles_ready();
  };
  if (it0 < it1) {
    fetch(ldsK0, kb, ks, kt.at(it0), Lk - 1, wave);
    fetch(ldsV0, vb, vs, kt.at(it0), Lk - 1, wave);
  }
  tiles_ready();
  for (int it = it0; it < it1; it += 2) {
    step(it, ldsK0, ldsV0, ldsK1, ldsV1);
    if (it + 1 < it1) step(it + 1, ldsK1, ldsV1, ldsK0, ldsV0);
  }
  sum += __shfl_xor(sum, 32, kWave);
  const bool mine = r0 + n <= last;
  const uint32_t again = odd_rows<D>(o, mine && sum < INFINITY);
  const float inv = sum > 0.f ? 1.f / sum : sum;
  if (t.chunks > 1) {  // sums [128][D], maxima [128], weights [128] of this chunk
    float* part = a.part + ((size_t)(t.chunk * slots + t.slot) * a.Hq + t.hq) * attn_fwd_part_floats(D);
    if (mine) store_part<D>(part + (size_t)(32 * wave + n) * D, o, h);
    if (h == 0) {
      part[(size_t)kAttnQ * D + 32 * wave + n] = mx;
      part[(size_t)kAttnQ * (D + 1) + 32 * wave + n] = sum;
    }
  } else {
    store_rows<D>(wave == 0 ? ldsK0 : wave == 1 ? ldsK1 : wave == 2 ? ldsV0 : ldsV1,
                  a.o.p + (long long)(q0 + r0) * a.o.token + t.hq * a.o.head, a.o.token, last + 1 - r0, o, inv, lane);
    if (mine && a.lse != nullptr && h == 0)
      a.lse[(size_t)t.hq * a.Tq + q0 + r] = sum > 0.f ? (mx + log2f(sum)) * kLn2 : (sum == 0.f ? -INFINITY : sum);
  }
  if (again) fwd_again<D>(args_again<AttnArgs>(), slots, again, wave, lane, mx, inv);
}

// Joins the chunks of the query tiles that were split, in order: a workgroup per 32 rows of a tile and
// head, eight threads per row.
template <int D>
__global__ __launch_bounds__(256) void attn_fwd_join_k(AttnArgs a, int slots) {
  const int hq = (int)(blockIdx.x % a.Hq), quarter = (int)(blockIdx.x / a.Hq & 3), slot = (int)(blockIdx.x / a.Hq / 4);
  const SeqTile t = find_tile<true, true, kAttnQ>(a.q_off, a.Tq, a.kv_off, a.Tkv, a.n_seq, slots, slot);
  if (!t.ok) return;
  const Mask m{t.b.n - t.a.n, a.window, a.sinks};
  const int last = t.a.n - 1;
  const KeyTiles kt = key_tiles(m, t.row0 + m.shift, min(t.row0 + kAttnQ - 1, last) + m.shift, t.b.n);
  const Chunks ch = key_chunks(m, kt.n, t.b.n, a.splits);
  const int row = 32 * quarter + (threadIdx.x >> 3), d0 = (threadIdx.x & 7) * (D / 8);
  if (ch.n == 1 || t.row0 + row > last) return;
  const size_t next = (size_t)slots * a.Hq * attn_fwd_part_floats(D);
  const float* part = a.part + ((size_t)slot * a.Hq + hq) * attn_fwd_part_floats(D);
  float mx = -INFINITY, sum = 0.f;
  f32x4_t o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) o[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  constexpr int kBatch = 4;  // chunks read side by side
  for (int c0 = 0; c0 < ch.n; c0 += kBatch) {
    float pm[kBatch], pl[kBatch];
    f32x4_t x[kBatch][D / 32];
#pragma unroll
    for (int c = 0; c < kBatch; ++c) {
      const float* p = part + min(c0 + c, ch.n - 1) * next;
      pm[c] = p[(size_t)kAttnQ * D + row];
      pl[c] = p[(size_t)kAttnQ * (D + 1) + row];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) x[c][i] = *reinterpret_cast<const f32x4_t*>(p + (size_t)row * D + d0 + 4 * i);
    }
    float up = mx;
#pragma unroll
    for (int c = 0; c < kBatch; ++c)
      if (c0 + c < ch.n) up = fmaxf(up, pm[c]);
    const float ref = up > -INFINITY ? up : 0.f, f0 = exp2_hw(mx - ref);
    mx = up;
    sum *= f0;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] *= f0;
#pragma unroll
    for (int c = 0; c < kBatch; ++c) {
      if (c0 + c >= ch.n) continue;
      const float f = exp2_hw(pm[c] - ref);
      sum = fmaf(pl[c], f, sum);
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] = fmaf(x[c][i][j], f, o[i][j]);
    }
  }
  const float inv = sum > 0.f ? 1.f / sum : sum;
  const long long r = t.a.lo + t.row0 + row;
  uint16_t* out = a.o.p + r * a.o.token + hq * a.o.head + d0;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    uint2 v;
    v.x = pack_bf16x2(o[i][0] * inv, o[i][1] * inv);
    v.y = pack_bf16x2(o[i][2] * inv, o[i][3] * inv);
    *reinterpret_cast<uint2*>(out + 4 * i) = v;
  }
  if (a.lse != nullptr && d0 == 0)
    a.lse[(size_t)hq * a.Tq + r] = sum > 0.f ? (mx + log2f(sum)) * kLn2 : (sum == 0.f ? -INFINITY : sum);
}

namespace {

// attn_dq_k's rows that are taken again (see fwd_again).
template <int D>
__device__ __forceinline__ void dq_again(const AttnBackwardArgs& b, int slots, uint32_t again, int wave, int lane,
                                         float lse2, float delta) {
  const AttnArgs& a = b.f;
  const QTile t = q_tile(a, slots, group_again(), b.q_splits);
  const uint16_t* kb = a.k.p + (long long)t.k0 * a.k.token + t.hk * a.k.head;
  const uint16_t* vb = a.v.p + (long long)t.k0 * a.v.token + t.hk * a.v.head;
  const float c = a.scale * kLog2e;
  const uint32_t lost = t.lost_columns<D>(kb, a.k.token, wave, lane);
  __threadfence();  // the rows are stored
  for (uint32_t left = again; left; left &= left - 1) {
    const int i = __builtin_ctz(left), at = 32 * wave + i, p = t.row0 + at + t.m.shift;
    const long long row = t.q0 + t.row0 + at;
    const uint16_t* qr = a.q.p + row * a.q.token + t.hq * a.q.head;
    const uint16_t* gr = b.dout.p + row * b.dout.token + t.hq * b.dout.head;
    const float li = lane_value(lse2, i), di = lane_value(delta, i);
    auto repair = [&](auto* out) {
      const uint32_t odd = to_repair<D>(out, lost, lane);
      if (!__any(odd)) return;
      RowSum<D> x;
      for (int it = t.it0; it < t.it1; ++it) {
        const int j0 = t.kt.at(it), j = j0 + lane;
        const bool see = sees(t.m, p, j);
        float w = 0.f;
        if (see) {
          w = exp2_hw(fmaf(dot_rows<D>(qr, kb + j * a.k.token), c, -li));
          w *= dot_rows<D>(gr, vb + j * a.v.token) - di;
        }
        x.add(__ballot(see), w, kb + j0 * a.k.token, a.k.token, lane);
      }
      x.store(out, a.scale, odd, lane);
    };
    if (t.chunks > 1) repair(b.q_part + (((size_t)(t.chunk * slots + t.slot) * a.Hq + t.hq) * kAttnQ + at) * D);
    else repair(b.dq.p + row * b.dq.token + t.hq * b.dq.head);
  }
}

}  // namespace

// dQ and the row sums of dO O: a workgroup holds 128 queries of one head, 32 per wave, and walks
// the keys as the forward does.  A kernel of its own, so that dQ is summed in registers in one order:
// together with dK and dV it would need atomics or a pass over partial sums.  The price is S and dP
// twice, seven products for five.
// Bound as the forward: 8192 tokens, 32 / 8 heads of 128, 730 us = 1129 TFLOP/s, the matrix units busy
// 61 % of the cycles (three products for one exponential); heads of 64, window 1024: 122 us.
template <int D, bool FINE>
__global__ __launch_bounds__(256, FINE ? 1 : D == 64 ? 3 : 2) void attn_dq_k(AttnBackwardArgs b, int slots) {
  constexpr int kTileB = kBN * Tile<D>::kRow;
  __shared__ __attribute__((aligned(16))) char ldsK0[kTileB], ldsK1[kTileB], ldsV0[kTileB], ldsV1[kTileB];
  const AttnArgs& a = b.f;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), h = lane >> 5,
            n = lane & 31;
  const QTile t = q_tile(a, slots, blockIdx.x, b.q_splits);
  if (!t.ok) return;
  const Mask m = t.m;
  const KeyTiles kt = t.kt;
  const int Lk = t.Lk, q0 = t.q0, k0 = t.k0, last = t.last;
  const int it0 = t.it0, it1 = t.it1;
  const int r0 = t.row0 + 32 * wave, r = min(r0 + n, last);
  const int p = r + m.shift, p_lo = r0 + m.shift, p_hi = min(r0 + 31, last) + m.shift;
  const uint16_t* kb = a.k.p + (long long)k0 * a.k.token + t.hk * a.k.head;
  const uint16_t* vb = a.v.p + (long long)k0 * a.v.token + t.hk * a.v.head;
  bf16x8_t q[D / 16], g[D / 16];
  float delta = 0.f;
  {
    const long long row = q0 + r;
    const uint16_t* qr = a.q.p + row * a.q.token + t.hq * a.q.head + 8 * h;
    const uint16_t* gr = b.dout.p + row * b.dout.token + t.hq * b.dout.head + 8 * h;
    const uint16_t* orow = a.o.p + row * a.o.token + t.hq * a.o.head + 8 * h;
#pragma unroll
    for (int st = 0; st < D / 16; ++st) {
      q[st] = as_bf16x8(ld16(qr + 16 * st));
      const u32x4_t gv = ld16(gr + 16 * st), ov = ld16(orow + 16 * st);
      g[st] = as_bf16x8(gv);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        delta = fmaf(bf16_to_f32(gv[i] & 0xffffu), bf16_to_f32(ov[i] & 0xffffu), delta);
        delta = fmaf(bf16_to_f32(gv[i] >> 16), bf16_to_f32(ov[i] >> 16), delta);
      }
    }
    delta += __shfl_xor(delta, 32, kWave);
  }
  const size_t stat = (size_t)t.hq * a.Tq + q0 + r;
  const float lse = a.lse[stat];
  const float lse2 = lse == -INFINITY ? 0.f : lse * kLog2e;  // a row that sees nothing: its scores are all -inf
  if (t.chunk == 0 && h == 0 && r0 + n <= last) {
    b.lse2[stat] = lse2;
    b.delta[stat] = -delta;
  }
  f32x16_t dq[D / 32];
#pragma unroll
  for (int mb = 0; mb < D / 32; ++mb) dq[mb] = f32x16_t{};
  const float c = a.scale * kLog2e;
  f32x16_t from;  // dP - delta is summed from here
#pragma unroll
  for (int i = 0; i < 16; ++i) from[i] = -delta;
  Fetch<D, kBN> fetch;
  fetch.init(lane, wave);
  const LaneOff lo = lane_off<D>(lane);
  const long long ks = 2 * a.k.token, vs = 2 * a.v.token;
  auto step = [&](int it, const char* __restrict__ K, const char* __restrict__ V, char* __restrict__ nextK,
                  char* __restrict__ nextV) {
    const int j0 = kt.at(it);
    if (it + 1 < it1) {
      fetch(nextK, kb, ks, kt.at(it + 1), Lk - 1, wave);
      fetch(nextV, vb, vs, kt.at(it + 1), Lk - 1, wave);
    }
    if (r0 <= last && !sees_none(m, p_lo, p_hi, j0, j0 + kBN - 1)) {
      const bool all = sees_all(m, p_lo, p_hi, j0, j0 + kBN - 1);
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) {
        f32x16_t s = f32x16_t{}, dp = from;
#pragma unroll
        for (int st = 0; st < D / 16; ++st) {
          s = mfma32x32x16(row_frag<D>(K, lo, 32 * blk, st), q[st], s);
          dp = mfma32x32x16(row_frag<D>(V, lo, 32 * blk, st), g[st], dp);
        }
        reads_ahead<D / 16, 2, 2, 3>();
        if (!all) hide(s, m, p, j0 + 32 * blk, h);
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = exp2_hw(fmaf(s[i], c, -lse2)) * dp[i];
        const bf16x8_t df[2] = {acc_frag(s, 0), acc_frag(s, 1)};
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int st = 0; st < 2; ++st)
#pragma unroll
          for (int mb = 0; mb < D / 32; ++mb)
            dq[mb] = mfma32x32x16(col_frag<D>(K, lo, 32 * blk + 16 * st, mb), df[st], dq[mb]);
        reads_ahead<D / 16, 1, 2, 4>();
        if constexpr (FINE) {
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            const bf16x8_t rest = acc_rest(s, st, df[st]);
#pragma unroll
            for (int mb = 0; mb < D / 32; ++mb)
              dq[mb] = mfma32x32x16(col_frag<D>(K, lo, 32 * blk + 16 * st, mb), rest, dq[mb]);
          }
        }
      }
    }
    tiles_ready();
  };
  if (it0 < it1) {
    fetch(ldsK0, kb, ks, kt.at(it0), Lk - 1, wave);
    fetch(ldsV0, vb, vs, kt.at(it0), Lk - 1, wave);
  }
  tiles_ready();
  for (int it = it0; it < it1; it += 2) {
    step(it, ldsK0, ldsV0, ldsK1, ldsV1);
    if (it + 1 < it1) step(it + 1, ldsK1, ldsV1, ldsK0, ldsV0);
  }
  const bool mine = r0 + n <= last;
  // a row that sees something and whose lse or delta is not finite has no other result
  const uint32_t again = odd_rows<D>(dq, mine && (lse == -INFINITY || finite(lse + delta)));
  if (mine && t.chunks > 1) {
    float* part = b.q_part + ((size_t)(t.chunk * slots + t.slot) * a.Hq + t.hq) * kAttnQ * D;
    store_part<D>(part + (size_t)(32 * wave + n) * D, dq, h);
  } else if (t.chunks == 1) {
    store_rows<D>(wave == 0 ? ldsK0 : wave == 1 ? ldsK1 : wave == 2 ? ldsV0 : ldsV1,
                  b.dq.p + (long long)(q0 + r0) * b.dq.token + t.hq * b.dq.head, b.dq.token, last + 1 - r0, dq, a.scale, lane);
  }
  if (again) dq_again<D>(args_again<AttnBackwardArgs>(), slots, again, wave, lane, lse2, delta);
}

// Adds the chunks of the query tiles that were split, in order (see attn_fwd_join_k).
template <int D>
__global__ __launch_bounds__(256) void attn_dq_join_k(AttnBackwardArgs b, int slots) {
  const AttnArgs& a = b.f;
  const int hq = (int)(blockIdx.x % a.Hq), quarter = (int)(blockIdx.x / a.Hq & 3), slot = (int)(blockIdx.x / a.Hq / 4);
  const SeqTile t = find_tile<true, true, kAttnQ>(a.q_off, a.Tq, a.kv_off, a.Tkv, a.n_seq, slots, slot);
  if (!t.ok) return;
  const Mask m{t.b.n - t.a.n, a.window, a.sinks};
  const int last = t.a.n - 1;
  const KeyTiles kt = key_tiles(m, t.row0 + m.shift, min(t.row0 + kAttnQ - 1, last) + m.shift, t.b.n);
  const Chunks ch = key_chunks(m, kt.n, t.b.n, b.q_splits);
  const int row = 32 * quarter + (threadIdx.x >> 3), d0 = (threadIdx.x & 7) * (D / 8);
  if (ch.n == 1 || t.row0 + row > last) return;
  const size_t next = (size_t)slots * a.Hq * kAttnQ * D;
  const float* part = b.q_part + ((size_t)slot * a.Hq + hq) * kAttnQ * D + (size_t)row * D + d0;
  uint16_t* out = b.dq.p + (long long)(t.a.lo + t.row0 + row) * b.dq.token + hq * b.dq.head + d0;
  f32x4_t sum[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) sum[i] = *reinterpret_cast<const f32x4_t*>(part + 4 * i);
#pragma unroll 4
  for (int c = 1; c < ch.n; ++c)
#pragma unroll
    for (int i = 0; i < D / 32; ++i) sum[i] += *reinterpret_cast<const f32x4_t*>(part + c * next + 4 * i);
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const f32x4_t x = sum[i];
    uint2 v;
    v.x = pack_bf16x2(x[0] * a.scale, x[1] * a.scale);
    v.y = pack_bf16x2(x[2] * a.scale, x[3] * a.scale);
    *reinterpret_cast<uint2*>(out + 4 * i) = v;
  }
}

namespace {

// A key tile of the dk / dv pass: 128 keys of one key-value head, the queries that see any of them
// in steps of attn_step() rows, taken for every query head that reads the head: `total` steps in `chunks`
// workgroups of `per` steps.  per comes from the longest tile's steps, so that chunks are about
// equally long and short tiles are not split.
struct KvTile {
  SeqRange q, k;
  int k0, t_lo, nt, total, chunks, per;
  long long part;  // of chunk 0
  bool ok;
};

// The tile of place `slot`, or with `sink` set of sinks' tile `slot`.
template <int kBQ>
__device__ __forceinline__ KvTile find_kv_tile(const AttnBackwardArgs& b, bool sink, int slots, int slot) {
  const AttnArgs& a = b.f;
  KvTile t{};
  if (sink) {
    const int s = slot / b.sink_tiles;
    const SeqRange q = seq_range(a.q_off, s, a.Tq), k = seq_range(a.kv_off, s, a.Tkv);
    t.q = {__builtin_amdgcn_readfirstlane(q.lo), __builtin_amdgcn_readfirstlane(q.n)};
    t.k = {__builtin_amdgcn_readfirstlane(k.lo), __builtin_amdgcn_readfirstlane(k.n)};
    t.k0 = slot % b.sink_tiles * kAttnK;
    if (t.k0 >= t.k.n) return t;
  } else {  // in a sequence the first keys, which the most queries see, come first
    const SeqTile f = find_tile<false, false, kAttnK>(a.q_off, a.Tq, a.kv_off, a.Tkv, a.n_seq, slots, slot);
    if (!f.ok || f.row0 < b.sink_tiles * kAttnK) return t;
    t.q = f.a;
    t.k = f.b;
    t.k0 = f.row0;
  }
  t.ok = true;
  const int shift = t.k.n - t.q.n, group = a.Hq / a.Hkv;
  const int i_lo = max(t.k0 - shift, 0);
  int i_hi = t.q.n;
  if (a.window && t.k0 >= a.sinks) {
    const long long end = (long long)min(t.k0 + kAttnK, t.k.n) - 1 + a.window - shift;
    i_hi = (int)max(0ll, min((long long)t.q.n, end));
  }
  t.t_lo = i_lo / kBQ;
  t.nt = max((i_hi + kBQ - 1) / kBQ - t.t_lo, 0);
  t.total = t.nt * group;
  const int steps = (t.q.n + kBQ - 1) / kBQ * group, splits = sink ? b.sink_splits : b.splits;
  t.per = max(((sink ? steps : min(steps, b.most)) + splits - 1) / splits, sink ? b.sink_min : b.min_steps);
  t.per = max(t.per, (t.total + splits - 1) / splits);  // never more chunks than there are places
  t.chunks = max((t.total + t.per - 1) / t.per, 1);
  const long long sink_parts = (long long)b.sink_tiles * a.n_seq * b.sink_splits;
  t.part = (sink ? 0 : sink_parts) + (long long)slot * splits;
  return t;
}

// Workgroup -> (key-value head, tile, chunk).  The sinks' tiles come first.  The chunk is the slowest index:
// workgroups without work then lie together at the end (spread between the others they would leave
// whole CUs idle).
struct KvPlace {
  int hk, chunk;
  KvTile t;
};
template <int kBQ>
__device__ __forceinline__ KvPlace kv_place(const AttnBackwardArgs& b, int slots, unsigned at) {
  const int sinks = b.sink_tiles * b.f.n_seq, first = sinks * b.sink_splits;
  int id = (int)(at / b.f.Hkv);
  const bool sink = id < first;
  if (!sink) id -= first;
  const int n_tiles = sink ? sinks : slots, chunk = id / n_tiles;
  return {(int)(at % b.f.Hkv), chunk, find_kv_tile<kBQ>(b, sink, slots, id - chunk * n_tiles)};
}

}  // namespace

namespace {

// attn_dkv_k's rows that are taken again: the wave's keys of the bits of `again`.
template <int D>
__device__ __forceinline__ void dkv_again(const AttnBackwardArgs& b, int slots, uint32_t again, int wave, int lane) {
  constexpr int kBQ = attn_step(D);
  const AttnArgs& a = b.f;
  const KvPlace pl = kv_place<kBQ>(b, slots, group_again());
  const KvTile& t = pl.t;
  const int group = a.Hq / a.Hkv, it0 = pl.chunk * t.per, it1 = min(it0 + t.per, t.total), jw = t.k0 + 32 * wave;
  const Mask m{t.k.n - t.q.n, a.window, a.sinks};
  const float c = a.scale * kLog2e;
  struct Step {
    const uint16_t *q, *g;
    const float *lse2, *delta;
    int i0;  // first row
  };
  auto at = [&](int it) {
    const int hq = pl.hk * group + it / t.nt, i0 = (t.t_lo + t.nt - 1 - it % t.nt) * kBQ;
    const long long row = t.q.lo + i0;
    const size_t stat = (size_t)hq * a.Tq + row;
    return Step{a.q.p + row * a.q.token + hq * a.q.head, b.dout.p + row * b.dout.token + hq * b.dout.head, b.lse2 + stat,
                b.delta + stat, i0};
  };
  uint32_t lost_k = 0, lost_v = 0;
  for (int it = it0; it < it1; ++it) {
    const Step s = at(it);
    const int p0 = s.i0 + m.shift;
    if (s.i0 + kBQ > t.q.n || !sees_all(m, p0, p0 + kBQ - 1, jw, jw + 31)) continue;
    const bool bad_p = __any(lane < kBQ && !finite(s.lse2[lane % kBQ]));
    const bool bad_ds = bad_p || __any(lane < kBQ && !finite(s.delta[lane % kBQ]));
    lost_v |= bad_p ? ~0u : odd_columns<D>(s.g, b.dout.token, kBQ, lane);
    lost_k |= bad_ds ? ~0u : odd_columns<D>(s.q, a.q.token, kBQ, lane);
  }
  __threadfence();  // the rows are stored
  for (uint32_t left = again; left; left &= left - 1) {
    const int j = jw + __builtin_ctz(left);
    const long long key = t.k.lo + j;
    const uint16_t* kp = a.k.p + key * a.k.token + pl.hk * a.k.head;
    const uint16_t* vp = a.v.p + key * a.v.token + pl.hk * a.v.head;
    auto repair = [&](auto* dk, auto* dv) {
      const uint32_t odd_k = to_repair<D>(dk, lost_k, lane), odd_v = to_repair<D>(dv, lost_v, lane);
      if (!__any(odd_k | odd_v)) return;
      RowSum<D> xk, xv;
      for (int it = it0; it < it1; ++it) {
        const Step s = at(it);
        const int row = s.i0 + lane;
        const bool see = lane < kBQ && row < t.q.n && sees(m, row + m.shift, j);
        float w = 0.f, ds = 0.f;
        if (see) {
          w = exp2_hw(fmaf(dot_rows<D>(s.q + lane * a.q.token, kp), c, -s.lse2[lane]));
          ds = w * (dot_rows<D>(s.g + lane * b.dout.token, vp) + s.delta[lane]);
        }
        const uint64_t who = __ballot(see);
        xv.add(who, w, s.g, b.dout.token, lane);
        xk.add(who, ds, s.q, a.q.token, lane);
      }
      xk.store(dk, a.scale, odd_k, lane);
      xv.store(dv, 1.f, odd_v, lane);
    };
    if (t.chunks > 1) {
      float* part = b.part + ((size_t)(t.part + pl.chunk) * a.Hkv + pl.hk) * attn_part_floats(D) + (size_t)(j - t.k0) * D;
      repair(part, part + (size_t)kAttnK * D);
    } else {
      repair(b.dk.p + key * b.dk.token + pl.hk * b.dk.head, b.dv.p + key * b.dv.token + pl.hk * b.dv.head);
    }
  }
}

}  // namespace

// dK and dV: a workgroup holds 128 keys of one key-value head, 32 per wave, and walks the queries
// of every query head that reads it (or one chunk of them, whose sums go to the workspace).  S and
// dP are computed with the queries down, so that P and dS are the right operands of dV^T = dO^T P
// and dK^T = Q^T dS.
// Bound as the forward, and by the waits between steps: 8192 tokens, 32 / 8 heads of 128, 1115 us = 986
// TFLOP/s, the matrix units busy 50 % of the cycles, waves waiting for copies and each other 28 %
// (with 128 values a step holds 32 rows: Q, dO and V fill the LDS of two workgroups); heads of 64,
// 64 rows per step, 4 x 4096 tokens, 16 heads 287 us = 957 TFLOP/s.
template <int D, bool FINE>
__global__ __launch_bounds__(256, FINE ? 1 : D == 64 ? 3 : 2) void attn_dkv_k(AttnBackwardArgs b, int slots) {
  constexpr int kBQ = attn_step(D), kTileB = kBQ * Tile<D>::kRow;
  // dP - delta is summed from -delta where vector instructions bound the pass (8192 tokens, 32 / 8 heads of
  // 64, window 1024: 186 -> 182 us; with 128 values the sums' start would wait for it: 1171 -> 1187 us).
  constexpr bool kFrom = D == 64;
  __shared__ __attribute__((aligned(16))) char ldsQ0[kTileB], ldsQ1[kTileB], ldsG0[kTileB], ldsG1[kTileB];
  __shared__ __attribute__((aligned(16))) float st0[2 * kBQ], st1[2 * kBQ];  // lse in base 2, -row sums
  // The workgroup's V stays in LDS: beside K's operands and the sums of dK and dV in registers it would
  // cost a wave per SIMD (4 x 4096 tokens, 16 heads, when it was moved: 64 values 451 us with V in
  // registers and two waves, 402 us with three; 128 values 1438 us with one wave, 794 us with two).
  __shared__ __attribute__((aligned(16))) char ldsV[kAttnK * Tile<D>::kRow];
  const AttnArgs& a = b.f;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), h = lane >> 5,
            n = lane & 31;
  const int group = a.Hq / a.Hkv;
  const KvPlace pl = kv_place<kBQ>(b, slots, blockIdx.x);
  const KvTile& t = pl.t;
  const int hk = pl.hk, chunk = pl.chunk;
  if (!t.ok || chunk >= t.chunks) return;
  const SeqRange qr = t.q, kr = t.k;
  const int k0 = t.k0, Lq = qr.n, Lk = kr.n, nt = t.nt;
  const int it0 = chunk * t.per, it1 = min(it0 + t.per, t.total);
  const Mask m{Lk - Lq, a.window, a.sinks};
  const int jw = k0 + 32 * wave, j = jw + n, jr = min(j, Lk - 1);  // wave's first key, lane's key
  bf16x8_t kf[D / 16];
  {
    const uint16_t* kp = a.k.p + (long long)(kr.lo + jr) * a.k.token + hk * a.k.head + 8 * h;
#pragma unroll
    for (int st = 0; st < D / 16; ++st) kf[st] = as_bf16x8(ld16(kp + 16 * st));
    Fetch<D, kAttnK> whole;
    whole.init(lane, wave);
    whole(ldsV, a.v.p + (long long)kr.lo * a.v.token + hk * a.v.head, 2 * a.v.token, k0, Lk - 1, wave);
  }
  f32x16_t dk[D / 32], dv[D / 32];
#pragma unroll
  for (int mb = 0; mb < D / 32; ++mb) dk[mb] = dv[mb] = f32x16_t{};
  const float c = a.scale * kLog2e;
  Fetch<D, kBQ> fetch;
  fetch.init(lane, wave);
  const LaneOff lo0 = lane_off<D>(lane);
  const long long qs = 2 * a.q.token, gs = 2 * b.dout.token;
  const uint16_t* qb = a.q.p + (long long)qr.lo * a.q.token;
  const uint16_t* gb = b.dout.p + (long long)qr.lo * b.dout.token;
  // The queries from the last on: every key tile of a causal sequence ends there, so the workgroups
  // that run together read the same rows.
  int head = it0 < it1 ? it0 / nt : 0, back = it0 - head * nt, i0 = 0;  // of the next request; rows requested last
  auto request = [&](char* __restrict__ Q, char* __restrict__ G, float* __restrict__ st) {
    const int hq = hk * group + head;
    i0 = (t.t_lo + nt - 1 - back) * kBQ;
    if (++back == nt) {
      back = 0;
      ++head;
    }
    fetch(Q, qb + hq * a.q.head, qs, i0, Lq - 1, wave);
    fetch(G, gb + hq * b.dout.head, gs, i0, Lq - 1, wave);
    if (wave < 2 * kBQ / kWave) {
      const int at = wave * kWave + lane;
      const float* src = (at < kBQ ? b.lse2 : b.delta) + (size_t)hq * a.Tq + qr.lo + min(i0 + (at & (kBQ - 1)), Lq - 1);
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                       (__attribute__((address_space(3))) void*)(st + wave * kWave), 4, 0, 0);
    }
  };
  auto step = [&](int it, const char* __restrict__ Q, const char* __restrict__ G, const float* __restrict__ ls,
                  char* __restrict__ nextQ, char* __restrict__ nextG, float* __restrict__ next_st) {
    const int s0 = i0;
    if (it + 1 < it1) request(nextQ, nextG, next_st);
    LaneOff lo = lo0;
    // opaque: the operands' addresses are made when needed; kept in registers they would spill others
    asm volatile("" : "+v"(lo.row), "+v"(lo.col));
#pragma unroll
    for (int sb = kBQ - 32; sb >= 0; sb -= 32) {
      const int r0 = s0 + sb;
      const int p_lo = r0 + m.shift, p_hi = min(r0 + 31, Lq - 1) + m.shift;
      if (jw < Lk && !sees_none(m, p_lo, p_hi, jw, jw + 31)) {
        const bool all = r0 + 32 <= Lq && sees_all(m, p_lo, p_hi, jw, jw + 31);
        f32x16_t s = f32x16_t{}, dp = f32x16_t{};
        if constexpr (kFrom) {
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const f32x4_t d4 = *reinterpret_cast<const f32x4_t*>(ls + kBQ + sb + 8 * g + 4 * h);
#pragma unroll
            for (int i = 0; i < 4; ++i) dp[4 * g + i] = d4[i];
          }
        }
#pragma unroll
        for (int st = 0; st < D / 16; ++st) {
          s = mfma32x32x16(row_frag<D>(Q, lo, sb, st), kf[st], s);
          dp = mfma32x32x16(row_frag<D>(G, lo, sb, st), row_frag<D>(ldsV, lo, 32 * wave, st), dp);
        }
        reads_ahead<D / 16, 2, 3, 3>();
        if (!all) {
          // the queries that see key j: a range of rows, here relative to the lane's first
          const int first = j - m.shift - r0 - 4 * h, rows = Lq - r0 - 4 * h;
          const int end = m.window == 0 || j < m.sinks ? rows : min(first + m.window, rows);
#pragma unroll
          for (int i = 0; i < 16; ++i) s[i] = acc_row(i, 0) >= first && acc_row(i, 0) < end ? s[i] : -INFINITY;
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x4_t l4 = *reinterpret_cast<const f32x4_t*>(ls + sb + 8 * g + 4 * h);
          f32x4_t d4{0.f, 0.f, 0.f, 0.f};
          if constexpr (!kFrom) d4 = *reinterpret_cast<const f32x4_t*>(ls + kBQ + sb + 8 * g + 4 * h);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float pv = exp2_hw(fmaf(s[4 * g + i], c, -l4[i]));
            s[4 * g + i] = pv;
            dp[4 * g + i] = pv * (kFrom ? dp[4 * g + i] : dp[4 * g + i] + d4[i]);
          }
        }
        const bf16x8_t pf[2] = {acc_frag(s, 0), acc_frag(s, 1)}, df[2] = {acc_frag(dp, 0), acc_frag(dp, 1)};
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int st = 0; st < 2; ++st)
#pragma unroll
          for (int mb = 0; mb < D / 32; ++mb) {
            dv[mb] = mfma32x32x16(col_frag<D>(G, lo, sb + 16 * st, mb), pf[st], dv[mb]);
            dk[mb] = mfma32x32x16(col_frag<D>(Q, lo, sb + 16 * st, mb), df[st], dk[mb]);
          }
        reads_ahead<D / 8, 1, 2, 4>();
        if constexpr (FINE) {
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            const bf16x8_t pr = acc_rest(s, st, pf[st]), dr = acc_rest(dp, st, df[st]);
#pragma unroll
            for (int mb = 0; mb < D / 32; ++mb) {
              dv[mb] = mfma32x32x16(col_frag<D>(G, lo, sb + 16 * st, mb), pr, dv[mb]);
              dk[mb] = mfma32x32x16(col_frag<D>(Q, lo, sb + 16 * st, mb), dr, dk[mb]);
            }
          }
        }
      }
    }
    tiles_ready();
  };
  if (it0 < it1) request(ldsQ0, ldsG0, st0);
  tiles_ready();
  for (int it = it0; it < it1; it += 2) {
    step(it, ldsQ0, ldsG0, st0, ldsQ1, ldsG1, st1);
    if (it + 1 < it1) step(it + 1, ldsQ1, ldsG1, st1, ldsQ0, ldsG0, st0);
  }
  const bool mine = j < Lk;
  const uint32_t again = odd_rows<D>(dk, mine) | odd_rows<D>(dv, mine);
  if (t.chunks > 1) {
    if (mine) {
      float* part = b.part + ((size_t)(t.part + chunk) * a.Hkv + hk) * attn_part_floats(D) + (size_t)(32 * wave + n) * D;
      store_part<D>(part, dk, h);
      store_part<D>(part + (size_t)kAttnK * D, dv, h);
    }
  } else {
    char* lds = wave == 0 ? ldsQ0 : wave == 1 ? ldsQ1 : wave == 2 ? ldsG0 : ldsG1;
    const long long key = kr.lo + jw;
    store_rows<D>(lds, b.dk.p + key * b.dk.token + hk * b.dk.head, b.dk.token, Lk - jw, dk, a.scale, lane);
    store_rows<D>(lds, b.dv.p + key * b.dv.token + hk * b.dv.head, b.dv.token, Lk - jw, dv, 1.f, lane);
  }
  if (again) dkv_again<D>(args_again<AttnBackwardArgs>(), slots, again, wave, lane);
}

// Adds the chunks of the key tiles that were split, in order: kJoinParts workgroups per tile.  Bound by
// the parts' bytes: 8192 tokens, 8 heads of 128 in 2 chunks, 134 MB in 19 us.
constexpr int kJoinParts = 16;
template <int D>
__global__ __launch_bounds__(256) void attn_dkv_join_k(AttnBackwardArgs b, int slots) {
  const AttnArgs& a = b.f;
  const int hk = (int)(blockIdx.x % a.Hkv), piece = (int)(blockIdx.x / a.Hkv % kJoinParts);
  const int id = (int)(blockIdx.x / a.Hkv / kJoinParts), sinks = b.sink_tiles * a.n_seq;
  const KvTile t = find_kv_tile<attn_step(D)>(b, id < sinks, slots, id < sinks ? id : id - sinks);
  if (!t.ok || t.chunks == 1) return;
  const float* part = b.part + ((size_t)t.part * a.Hkv + hk) * attn_part_floats(D);
  const size_t next = (size_t)a.Hkv * attn_part_floats(D);
  constexpr int kQuads = D / 4, kRows = kAttnK / kJoinParts;
  for (int i = threadIdx.x; i < 2 * kRows * kQuads; i += 256) {
    const int which = i / (kRows * kQuads), row = kRows * piece + i / kQuads % kRows, c = i % kQuads * 4;
    if (t.k0 + row >= t.k.n) continue;
    const float* at = part + (size_t)which * kAttnK * D + (size_t)row * D + c;
    f32x4_t x = *reinterpret_cast<const f32x4_t*>(at);
#pragma unroll 4
    for (int ch = 1; ch < t.chunks; ++ch) x += *reinterpret_cast<const f32x4_t*>(at + ch * next);
    const Rows& o = which ? b.dv : b.dk;
    const float mul = which ? 1.f : a.scale;
    uint2 v;
    v.x = pack_bf16x2(x[0] * mul, x[1] * mul);
    v.y = pack_bf16x2(x[2] * mul, x[3] * mul);
    *reinterpret_cast<uint2*>(o.p + (long long)(t.k.lo + t.k0 + row) * o.token + hk * o.head + c) = v;
  }
}

namespace {

template <int D>
hipError_t forward(const AttnArgs& a, hipStream_t s) {
  const int slots = (int)attn_slots(a.Tq, a.n_seq, kAttnQ);
  hipLaunchKernelGGL((attn_fwd_k<D>), dim3((unsigned)(slots * a.Hq * a.splits)), dim3(256), 0, s, a, slots);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  hipLaunchKernelGGL((attn_fwd_join_k<D>), dim3((unsigned)(slots * a.Hq * 4)), dim3(256), 0, s, a, slots);
  return hipGetLastError();
}

template <int D, bool FINE>
hipError_t backward(const AttnBackwardArgs& b, hipStream_t s) {
  const AttnArgs& a = b.f;
  const long long ks = attn_slots(a.Tkv, a.n_seq, kAttnK);
  if (a.Tq > 0) {
    const int qs = (int)attn_slots(a.Tq, a.n_seq, kAttnQ);
    hipLaunchKernelGGL((attn_dq_k<D, FINE>), dim3((unsigned)(qs * a.Hq * b.q_splits)), dim3(256), 0, s, b, qs);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (b.q_splits > 1) {
      hipLaunchKernelGGL((attn_dq_join_k<D>), dim3((unsigned)(qs * a.Hq * 4)), dim3(256), 0, s, b, qs);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
  }
  const long long sinks = (long long)b.sink_tiles * a.n_seq;
  const dim3 grid((unsigned)((sinks * b.sink_splits + ks * b.splits) * a.Hkv));
  hipLaunchKernelGGL((attn_dkv_k<D, FINE>), grid, dim3(256), 0, s, b, (int)ks);
  const hipError_t e = hipGetLastError();
  const long long joins = sinks + (b.splits > 1 ? ks : 0);
  if (e != hipSuccess || joins == 0) return e;
  hipLaunchKernelGGL((attn_dkv_join_k<D>), dim3((unsigned)(joins * a.Hkv * kJoinParts)), dim3(256), 0, s, b, (int)ks);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_forward(const AttnArgs& a, hipStream_t s) {
  return a.D == 64 ? forward<64>(a, s) : forward<128>(a, s);
}

// P and dS enter the second products rounded to bf16, which errs as much as the rounding of the result
// does.  In a batch of few rows single roundings show in the gradients (nothing averages), and the
// products are a small part of the time: there both go in as a rounded value and its rest (one head of 128,
// 64 rows: 16.1 us rounded, 17.9 us with the rest).
hipError_t launch_attn_backward(const AttnBackwardArgs& b, hipStream_t s) {
  constexpr int kFineRows = 64;
  if (b.f.Tq <= kFineRows) return b.f.D == 64 ? backward<64, true>(b, s) : backward<128, true>(b, s);
  return b.f.D == 64 ? backward<64, false>(b, s) : backward<128, false>(b, s);
}

}  // namespace molora
