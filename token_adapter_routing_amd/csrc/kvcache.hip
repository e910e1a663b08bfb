// Paged key-value cache: appending rows (16 bits as they are, 8 bits with a power-of-two factor
// per row) and the attention of one new token per sequence over the cache.
#include <cmath>

#include "decoder_launch.h"
#include "seq_dev.h"

namespace molora {

// ------------------------------------------------------------------------------- append
// A wave per token: the token's sequence by a search in q_off, its page and row, then its
// 2 Hkv rows of D values, D / 8 lanes per row (16-byte pieces), 64 / (D / 8) rows at a time.
// Memory-bound: every row is read once and written once, past the caches, which nothing that follows soon
// reads it from (15 prompts, 8 heads of 128, bf16, 126 MB of rows not in any cache: 27.5 us with ordinary
// stores, 21.8 us = 6.1 TB/s; 16384 tokens in 8 bits 25.4 and 24.4 us).  Several rows requested at once per
// lane gain nothing (28.4 us).  256 single tokens in 8 bits 5.5 us: the launch and three dependent loads.
//
// e4m3: the row's factor is the smallest power of two that brings its largest finite magnitude
// within 448 (a floating format keeps its relative precision under any factor, and a power of two
// makes both the scaling here and the product on the way back exact), so the row is rounded once.
template <int D, bool E4M3>
__global__ __launch_bounds__(256) void kv_append_k(KvAppendArgs a) {
  constexpr int kLanes = D / 8, kRows = kWave / kLanes;
  const int lane = threadIdx.x & 63;
  const int t = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  if (t >= a.T) return;
  int b = t, pos;
  if (a.q_off != nullptr) {
    b = __builtin_amdgcn_readfirstlane(wave_search(a.n_seq, t, [&](int i) { return (long long)a.q_off[i]; }));
    if (b < 0 || t >= a.q_off[b + 1]) return;  // before the first or behind the last sequence
    pos = a.lens[b] - (a.q_off[b + 1] - t);
  } else {
    pos = a.lens[b] - 1;
  }
  const int page_size = 1 << a.c.page_shift;
  if (pos < 0 || (pos >> a.c.page_shift) >= a.width) return;
  const int page = a.table[(long long)b * a.width + (pos >> a.c.page_shift)];
  if (page < 0 || page >= a.c.n_pages) return;
  const int piece = lane % kLanes, sub = lane / kLanes;
  const long long row0 = (long long)page * a.c.Hkv * page_size + (pos & (page_size - 1));
  for (int i = sub; i < 2 * a.c.Hkv; i += kRows) {
    const bool is_v = i >= a.c.Hkv;
    const int head = is_v ? i - a.c.Hkv : i;
    const Rows& src = is_v ? a.v : a.k;
    const u32x4_t x = ld16(src.p + t * src.token + head * src.head + 8 * piece);
    const long long row = row0 + (long long)head * page_size;
    if constexpr (!E4M3) {
      st16_nt(reinterpret_cast<uint16_t*>(is_v ? a.c.v : a.c.k) + row * D + 8 * piece, x);
    } else {
      float f[8], big = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[2 * j] = bf16_to_f32(x[j] & 0xffffu);
        f[2 * j + 1] = bf16_to_f32(x[j] >> 16);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float m = fabsf(f[j]);
        if (m < INFINITY) big = fmaxf(big, m);
      }
#pragma unroll
      for (int d = 1; d < kLanes; d <<= 1) big = fmaxf(big, __shfl_xor(big, d, kWave));
      // big = m 2^e with m in [1/2, 1); 448 = 7/8 2^9.  -112 keeps every factor and product normal.
      int e;
      const float m = frexpf(big, &e);
      const int n = big > 0.f ? max(e - (m > 0.875f ? 8 : 9), -112) : -112;
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float v = ldexpf(f[j], -n);
        y[j] = v == v ? fminf(fmaxf(v, -448.f), 448.f) : v;
      }
      int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
      lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], lo, true);
      int hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], 0, false);
      hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], hi, true);
      __builtin_nontemporal_store(
          (uint64_t)(uint32_t)hi << 32 | (uint32_t)lo,
          reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(is_v ? a.c.v : a.c.k) + row * D + 8 * piece));
      if (piece == 0) (is_v ? a.c.v_scale : a.c.k_scale)[row] = (uint8_t)(n + 127);
    }
  }
}

hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t s) {
  const dim3 grid((a.T + 3) / 4), block(256);
  if (a.c.D == 64) {
    if (a.c.e4m3) hipLaunchKernelGGL((kv_append_k<64, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((kv_append_k<64, false>), grid, block, 0, s, a);
  } else {
    if (a.c.e4m3) hipLaunchKernelGGL((kv_append_k<128, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((kv_append_k<128, false>), grid, block, 0, s, a);
  }
  return hipGetLastError();
}

// ------------------------------------------------------------------------------- decode
// S^T = K Q^T and O^T = V^T P^T on 16x16x32 instructions, the (up to 16) query heads of a
// key-value head across, straight from global memory: no LDS on the way.
//   K: lane l holds key l % 16 of a 16-key tile and values 64 i + 16 (l / 16) .. + 15: 32 contiguous
//      bytes (16 in 8 bits).
//   V: lane l holds values VW (l % 16) .. + VW - 1 (VW = D / 16) of the keys that S^T left in its
//      own registers, 4 (l / 16) .. + 3 of both 16-key tiles: 16 lanes read one row.  The 8 keys x
//      VW values are turned in registers, a byte permutation per pair, into VW operands.
// P, rounded to bf16, is then the right operand of the second product as it stands.
// Bound by the bytes of the visible rows.  A wave takes every fourth 32-key block of its split
// and requests the next block before it works on the current one.  Straight to registers, because a
// row is used by one wave only: LDS would add a copy and barriers and save no byte.
// 64 sequences of 4096 on average, 32 / 8 heads of 128: 184 us, 5.8 TB/s (a large copy reaches 5.2);
// 8 bits, 256 sequences with a window: 276 us, 5.9 TB/s; one sequence of 32768: 23.1 us and 5.0 us for
// the join.
namespace {

// The visible blocks of one sequence: blocks [0, sink) hold its sink tokens, the rest starts at
// block `first`; positions past `len`, and between the sinks and `lo`, are masked inside blocks.
struct DecSeq {
  int len, lo, sink, first, blocks;
  __device__ __forceinline__ int block(int i) const { return i < sink ? i : first + i - sink; }
};
__device__ __forceinline__ DecSeq dec_seq(const DecodeArgs& a, int b) {
  DecSeq s;
  s.len = __builtin_amdgcn_readfirstlane(min(max(a.lens[b], 0), a.width << a.c.page_shift));
  s.lo = a.window ? max(s.len - a.window, 0) : 0;
  s.first = s.lo / kDecBlock;
  s.sink = a.window ? min((min(a.sinks, s.len) + kDecBlock - 1) / kDecBlock, s.first) : 0;
  s.blocks = s.sink + (s.len + kDecBlock - 1) / kDecBlock - s.first;
  return s;
}

// One 32-key block of K and V in registers.
template <int D, bool E4M3>
struct DecTile {
  static constexpr int VW = D / 16;               // values of V per lane and key
  static constexpr int KB = E4M3 ? 1 : 2;         // bytes per value
  static constexpr int KV4 = 16 * KB / 16;        // 16-byte loads per lane, key tile and 64 values
  u32x4_t k[2][D / 64][KV4];
  uint32_t v[8][VW * KB / 4];
  uint32_t ks[2], vs[2];
  int pos0;
  bool ok[2];  // the halves' pages exist

  __device__ __forceinline__ void load(const DecodeArgs& a, const int32_t* table, int blk, int hk, int len, int lane) {
    pos0 = blk * kDecBlock;
    const int page_size = 1 << a.c.page_shift, m = lane & 15, g = lane >> 4;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int p = pos0 + 16 * t;
      int page = p < len ? table[p >> a.c.page_shift] : -1;
      page = __builtin_amdgcn_readfirstlane(page);
      ok[t] = page >= 0 && page < a.c.n_pages;
      // an absent page's place is taken by page 0: read, never used
      const long long row0 = ((long long)(ok[t] ? page : 0) * a.c.Hkv + hk) * page_size + (p & (page_size - 1));
      const char* kp = reinterpret_cast<const char*>(a.c.k) + row0 * D * KB;
      const char* vp = reinterpret_cast<const char*>(a.c.v) + row0 * D * KB;
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
#pragma unroll
        for (int q = 0; q < KV4; ++q) k[t][i][q] = ld16_nt(kp + (m * D + 64 * i + 16 * g) * KB + 16 * q);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const char* r = vp + ((4 * g + i) * D + VW * m) * KB;
        if constexpr (VW * KB == 16) {
          const u32x4_t x = ld16_nt(r);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[4 * t + i][j] = x[j];
        } else if constexpr (VW * KB == 8) {
          const uint64_t x = __builtin_nontemporal_load(reinterpret_cast<const uint64_t*>(r));
          v[4 * t + i][0] = (uint32_t)x;
          v[4 * t + i][1] = (uint32_t)(x >> 32);
        } else {
          v[4 * t + i][0] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(r));
        }
      }
      if constexpr (E4M3) {
        ks[t] = a.c.k_scale[row0 + m];
        vs[t] = *reinterpret_cast<const uint32_t*>(a.c.v_scale + row0 + 4 * g);
      }
    }
  }
};

// Two 8-bit values (half `hi` of w) times the power of two in `scale`, as packed bf16: exact.
__device__ __forceinline__ uint32_t cvt_e4m3(uint32_t w, float scale, bool hi) {
  typedef __attribute__((__vector_size__(2 * sizeof(__bf16)))) __bf16 bf16x2_t;
  return hi ? __builtin_bit_cast(uint32_t, (bf16x2_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, true))
            : __builtin_bit_cast(uint32_t, (bf16x2_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, false));
}

}  // namespace

template <int D, bool E4M3>
__global__ __launch_bounds__(256, 2) void attn_decode_k(DecodeArgs a, int head_tiles) {
  using T = DecTile<D, E4M3>;
  constexpr int VW = T::VW;
  __shared__ float so[4][kDecHeads][D + 4];
  __shared__ float sm[4][kDecHeads], sl[4][kDecHeads];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), n = lane & 15,
            g = lane >> 4;
  // consecutive workgroups take different sequences and heads: a long sequence's splits spread
  const unsigned units = (unsigned)a.n_seq * a.c.Hkv * head_tiles, unit = blockIdx.x % units;
  const int split = (int)(blockIdx.x / units), ht = (int)(unit % head_tiles), hk = (int)(unit / head_tiles % a.c.Hkv),
            b = (int)(unit / head_tiles / a.c.Hkv);
  const DecSeq sq = dec_seq(a, b);
  const int per = decode_blocks_per_split(sq.blocks, a.splits);
  const int i0 = split * per, i1 = min(i0 + per, sq.blocks);
  if (i0 >= i1 && split > 0) return;  // the first split writes an empty sequence's result
  const int group = a.Hq / a.c.Hkv, h0 = ht * kDecHeads, heads = min(kDecHeads, group - h0);
  const int hq = hk * group + h0 + min(n, heads - 1);
  const int32_t* table = a.table + (long long)b * a.width;
  bf16x8_t q[D / 64][2];
  {
    const uint16_t* qr = a.q.p + b * a.q.token + hq * a.q.head + 16 * g;
#pragma unroll
    for (int i = 0; i < D / 64; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) q[i][e] = as_bf16x8(ld16(qr + 64 * i + 8 * e));
  }
  const float c = a.scale * kLog2e;
  f32x4_t o[VW];
#pragma unroll
  for (int j = 0; j < VW; ++j) o[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  float mx = -INFINITY, sum = 0.f;

  auto work = [&](const T& x) {
    f32x4_t s[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      s[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        if constexpr (!E4M3) {
#pragma unroll
          for (int e = 0; e < 2; ++e) s[t] = mfma16x16x32(as_bf16x8(x.k[t][i][e]), q[i][e], s[t]);
        } else {
          const float f = __uint_as_float(x.ks[t] << 23);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            u32x4_t w;
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = cvt_e4m3(x.k[t][i][0][2 * e + (j >> 1)], f, j & 1);
            s[t] = mfma16x16x32(as_bf16x8(w), q[i][e], s[t]);
          }
        }
      }
    }
    uint32_t v[8][VW / 2];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (!E4M3) {
#pragma unroll
        for (int j = 0; j < VW / 2; ++j) v[i][j] = x.v[i][j];
      } else {
        const float f = __uint_as_float(((x.vs[i >> 2] >> (8 * (i & 3))) & 0xffu) << 23);
#pragma unroll
        for (int j = 0; j < VW / 2; ++j) v[i][j] = cvt_e4m3(x.v[i][j >> 1], f, j & 1);
      }
    }
    const bool whole = x.ok[0] && x.ok[1] && x.pos0 + kDecBlock <= sq.len &&
                       (x.pos0 >= sq.lo || x.pos0 + kDecBlock <= a.sinks);
    if (!whole) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int p = x.pos0 + 16 * t + 4 * g + i;
          if (!(x.ok[t] && p < sq.len && (p >= sq.lo || p < a.sinks))) {
            s[t][i] = -INFINITY;
#pragma unroll
            for (int j = 0; j < VW / 2; ++j) v[4 * t + i][j] = 0;
          }
        }
    }
    float top = s[0][0];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, s[t][i]);
    top *= c;
    if (__any(top > mx + 8.f)) {  // the reference maximum follows late: weights stay below 2^8
      float up = fmaxf(mx, fmaxf(top, __shfl_xor(top, 16, kWave)));
      up = fmaxf(up, __shfl_xor(up, 32, kWave));
      const float f = up > -INFINITY ? exp2_hw(mx - up) : 1.f;
      mx = up;
      sum *= f;
#pragma unroll
      for (int j = 0; j < VW; ++j) o[j] *= f;
    }
    const float ref = mx > -INFINITY ? mx : 0.f;
    float p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[i] = exp2_hw(fmaf(s[i >> 2][i & 3], c, -ref));
      sum += p[i];
    }
    u32x4_t pf;
#pragma unroll
    for (int i = 0; i < 4; ++i) pf[i] = pack_bf16x2(p[2 * i], p[2 * i + 1]);
#pragma unroll
    for (int j = 0; j < VW; ++j) {
      u32x4_t w;  // value VW m + j of the lane's eight keys
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = __builtin_amdgcn_perm(v[2 * i + 1][j >> 1], v[2 * i][j >> 1], (j & 1) ? 0x07060302u : 0x05040100u);
      o[j] = mfma16x16x32(as_bf16x8(w), as_bf16x8(pf), o[j]);
    }
  };

  int i = i0 + wave;
  if (i < i1) {
    T x, y;
    x.load(a, table, sq.block(i), hk, sq.len, lane);
    for (;;) {
      const bool two = i + 4 < i1, three = i + 8 < i1;
      if (two) y.load(a, table, sq.block(i + 4), hk, sq.len, lane);
      work(x);
      if (!two) break;
      if (three) x.load(a, table, sq.block(i + 8), hk, sq.len, lane);
      work(y);
      if (!three) break;
      i += 8;
    }
  }
  sum += __shfl_xor(sum, 16, kWave);
  sum += __shfl_xor(sum, 32, kWave);
  // the four waves' parts
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int j = 0; j < VW; ++j) so[wave][n][VW * (4 * g + r) + j] = o[j][r];
  if (g == 0) {
    sm[wave][n] = mx;
    sl[wave][n] = sum;
  }
  __syncthreads();
  const int head = tid >> 4, d0 = (tid & 15) * VW;
  if (head >= heads) return;
  float m = fmaxf(fmaxf(sm[0][head], sm[1][head]), fmaxf(sm[2][head], sm[3][head]));
  const float ref = m > -INFINITY ? m : 0.f;
  float l = 0.f, r[VW];
#pragma unroll
  for (int j = 0; j < VW; ++j) r[j] = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float f = exp2_hw(sm[w][head] - ref);
    l = fmaf(sl[w][head], f, l);
#pragma unroll
    for (int j = 0; j < VW; ++j) r[j] = fmaf(so[w][head][d0 + j], f, r[j]);
  }
  const int out = hk * group + h0 + head;
  if (a.splits == 1) {
    const float inv = l > 0.f ? 1.f / l : l;
    uint16_t* po = a.o.p + b * a.o.token + out * a.o.head + d0;
#pragma unroll
    for (int j = 0; j < VW; j += 2) *reinterpret_cast<uint32_t*>(po + j) = pack_bf16x2(r[j] * inv, r[j + 1] * inv);
    if (a.lse != nullptr && (tid & 15) == 0)
      a.lse[(size_t)b * a.Hq + out] = l > 0.f ? (m + log2f(l)) * kLn2 : (l == 0.f ? -INFINITY : l);
  } else {
    float* part = a.part + ((size_t)unit * a.splits + split) * decode_part_floats(D);
#pragma unroll
    for (int j = 0; j < VW; ++j) part[head * D + d0 + j] = r[j];
    if ((tid & 15) == 0) {
      part[kDecHeads * D + head] = m;
      part[kDecHeads * (D + 1) + head] = l;
    }
  }
}

// Joins the splits of one (sequence, query head): a workgroup each, D / 4 threads per part, so that 8
// or 16 parts are read side by side; each such group of threads adds its parts in order, then the
// groups' sums are added in order.
template <int D>
__global__ __launch_bounds__(256) void attn_decode_join_k(DecodeArgs a, int head_tiles) {
  constexpr int kThreads = D / 4, kGroups = 256 / kThreads;
  __shared__ __attribute__((aligned(16))) float sums[kGroups][D + 4];  // behind each l and m
  const int tid = threadIdx.x;
  const unsigned id = blockIdx.x;
  const int b = (int)(id / a.Hq), hq = (int)(id % a.Hq);
  const int group = a.Hq / a.c.Hkv, hk = hq / group, ht = hq % group / kDecHeads, head = hq % group % kDecHeads;
  const DecSeq sq = dec_seq(a, b);
  const int per = decode_blocks_per_split(sq.blocks, a.splits);
  const int parts = max(1, (sq.blocks + per - 1) / per);
  const size_t unit = ((size_t)b * a.c.Hkv + hk) * head_tiles + ht, next = decode_part_floats(D);
  const float* part = a.part + unit * a.splits * next;
  // a group's parts eight at a time, with their own reference maximum
  const int grp = tid / kThreads, d0 = tid % kThreads * 4;
  float m = -INFINITY, l = 0.f;
  f32x4_t r{0.f, 0.f, 0.f, 0.f};
  for (int s0 = grp; s0 < parts; s0 += 8 * kGroups) {
    float pm[8], pl[8];
    f32x4_t x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float* ps = part + min(s0 + i * kGroups, parts - 1) * next;
      pm[i] = ps[kDecHeads * D + head];
      pl[i] = ps[kDecHeads * (D + 1) + head];
      x[i] = *reinterpret_cast<const f32x4_t*>(ps + head * D + d0);
    }
    float up = m;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (s0 + i * kGroups >= parts) pm[i] = -INFINITY;
      up = fmaxf(up, pm[i]);
    }
    const float ref = up > -INFINITY ? up : 0.f, f0 = exp2_hw(m - ref);
    m = up;
    l *= f0;
    r *= f0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (s0 + i * kGroups >= parts) continue;  // a repeated part: whatever it holds stays out
      const float f = exp2_hw(pm[i] - ref);
      l = fmaf(pl[i], f, l);
#pragma unroll
      for (int j = 0; j < 4; ++j) r[j] = fmaf(x[i][j], f, r[j]);
    }
  }
  *reinterpret_cast<f32x4_t*>(&sums[grp][d0]) = r;
  if (d0 == 0) {
    sums[grp][D] = l;
    sums[grp][D + 1] = m;
  }
  __syncthreads();
  if (tid >= kThreads) return;
  m = -INFINITY;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) m = fmaxf(m, sums[g][D + 1]);
  const float ref = m > -INFINITY ? m : 0.f;
  l = 0.f;
  r = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const float f = exp2_hw(sums[g][D + 1] - ref);
    l = fmaf(sums[g][D], f, l);
    const f32x4_t x = *reinterpret_cast<const f32x4_t*>(&sums[g][d0]);
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = fmaf(x[j], f, r[j]);
  }
  const float inv = l > 0.f ? 1.f / l : l;
  uint2 v;
  v.x = pack_bf16x2(r[0] * inv, r[1] * inv);
  v.y = pack_bf16x2(r[2] * inv, r[3] * inv);
  *reinterpret_cast<uint2*>(a.o.p + b * a.o.token + hq * a.o.head + d0) = v;
  if (a.lse != nullptr && tid == 0)
    a.lse[(size_t)b * a.Hq + hq] = l > 0.f ? (m + log2f(l)) * kLn2 : (l == 0.f ? -INFINITY : l);
}

namespace {

template <int D>
hipError_t decode(const DecodeArgs& a, hipStream_t s) {
  const int group = a.Hq / a.c.Hkv, head_tiles = (group + kDecHeads - 1) / kDecHeads;
  const dim3 grid((unsigned)((long long)a.n_seq * a.c.Hkv * head_tiles * a.splits));
  if (a.c.e4m3) hipLaunchKernelGGL((attn_decode_k<D, true>), grid, dim3(256), 0, s, a, head_tiles);
  else hipLaunchKernelGGL((attn_decode_k<D, false>), grid, dim3(256), 0, s, a, head_tiles);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  hipLaunchKernelGGL((attn_decode_join_k<D>), dim3((unsigned)(a.n_seq * a.Hq)), dim3(256), 0, s, a, head_tiles);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_decode(const DecodeArgs& a, hipStream_t s) {
  return a.c.D == 64 ? decode<64>(a, s) : decode<128>(a, s);
}

}  // namespace molora
