// Routing by scores: softmax or sigmoid scores, a balance bias for the selection, adapter
// groups, top-k, (re)normalised weights; and its gradient.
//
//   s = softmax(l) | sigmoid(l);  c = s + bias;  mark_g = sum of group g's two largest c;
//   keep the topk_group largest marks; choose the k largest c; w = factor s / [renorm] sum s
//   dl_e = p_e (g_e - sum_j p_j g_j) [sigmoid: times 1 - s_e], g_j = factor dw_j of the chosen, else 0;
//   renorm: p the chosen's s over their sum, 0 for the others; else p = s, for sigmoid without the sum
//
// Layout: eight lanes per token, lane i holding adapters [i E, (i + 1) E), E = 2, 4 or 8 with
// 8 E >= K, so a wave takes eight tokens, a reduction over adapters is E register steps and
// three exchanges inside eight lanes, and each lane's logits are one contiguous piece.  One
// round of the selection per chosen adapter (k <= 8).  Eight lanes and not a wave per token: a
// reduction over 64 lanes is six dependent exchanges for one token, this is three for eight.
//
// Bound by the length of that chain, not by memory (16384 x 64 fp32 logits are 4.3 MB, 1 us):
//   scores  256 x 16, k 2: 3.0 us; 16384 x 64, k 8, 8 groups of which 4, bias: 8.8 us (10.1 us with
//           LDS exchanges for the register moves)
//   backward  16384 x 64, k 4: 4.9 us, 1.8 TB/s
#include <cfloat>
#include <cmath>

#include "decoder_launch.h"
#include "molora_dev.h"

namespace molora {

namespace {

constexpr int kLanes = 8;             // lanes per token
constexpr int kTok = kWave / kLanes;  // tokens per wave
constexpr int kWaves = 4;             // waves per workgroup

// The value of another lane of the eight: STEP 0 lane ^ 1, 1 lane ^ 2, 2 the mirrored lane (which after
// the first two steps holds what lane ^ 4 holds).  Register moves, no LDS exchange.
template <int STEP>
__device__ __forceinline__ int peer(int v) {
  constexpr int kCtrl = STEP == 0 ? 0xB1 : STEP == 1 ? 0x4E : 0x141;  // quad_perm 1032, 2301; row_half_mirror
  return __builtin_amdgcn_update_dpp(v, v, kCtrl, 0xf, 0xf, true);
}
template <int STEP>
__device__ __forceinline__ float peer(float v) {
  return __int_as_float(peer<STEP>(__float_as_int(v)));
}
template <int STEP>
__device__ __forceinline__ double peer(double v) {
  const uint64_t u = __double_as_longlong(v);
  const uint32_t lo = peer<STEP>((int)(uint32_t)u), hi = peer<STEP>((int)(uint32_t)(u >> 32));
  return __longlong_as_double(((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return fmax(a, b); }
__device__ __forceinline__ float smaller(float a, float b) { return fminf(a, b); }
__device__ __forceinline__ double smaller(double a, double b) { return fmin(a, b); }

// Reductions over the eight lanes of a token, the result in all of them.
template <typename F>
__device__ __forceinline__ F sum8(F v) {
  v += peer<0>(v);
  v += peer<1>(v);
  return v + peer<2>(v);
}
template <typename F>
__device__ __forceinline__ F max8(F v) {
  v = larger(v, peer<0>(v));
  v = larger(v, peer<1>(v));
  return larger(v, peer<2>(v));
}
__device__ __forceinline__ int min8(int v) {
  v = min(v, peer<0>(v));
  v = min(v, peer<1>(v));
  return min(v, peer<2>(v));
}

// Lane's E logits of token `tok`; absent adapters (NaN, -inf, past K) come as -inf, +inf as the
// largest finite number.
template <int E>
__device__ __forceinline__ void load_logits(const float* __restrict__ logits, int tok, bool mine, int K, int e0,
                                            float* l) {
  const float* row = logits + (size_t)tok * K + e0;
#pragma unroll
  for (int j = 0; j < E; ++j) l[j] = -INFINITY;
  if (mine) {
    if (K == kLanes * E) {  // whole rows: E a multiple of 2, so 8- or 16-byte pieces
      if constexpr (E >= 4) {
#pragma unroll
        for (int q = 0; q < E / 4; ++q) {
          const u32x4_t v = ld16(row + 4 * q);
#pragma unroll
          for (int j = 0; j < 4; ++j) l[4 * q + j] = __uint_as_float(v[j]);
        }
      } else {
        const float2 v = *reinterpret_cast<const float2*>(row);
        l[0] = v.x;
        l[1] = v.y;
      }
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (e0 + j < K) l[j] = row[j];
    }
  }
#pragma unroll
  for (int j = 0; j < E; ++j) l[j] = l[j] == l[j] ? fminf(l[j], FLT_MAX) : -INFINITY;
}

// Scores of the lane's adapters in F; exp(l - top) and 1 / (1 + exp(-l)) as written, so that an
// absent adapter (-inf) gets exactly 0.
template <typename F, int E>
__device__ __forceinline__ void scores(const float* l, int score, F* s) {
  if (score == kScoreSigmoid) {
#pragma unroll
    for (int j = 0; j < E; ++j) s[j] = F(1) / (F(1) + exp(-F(l[j])));
    return;
  }
  float top = -INFINITY;
#pragma unroll
  for (int j = 0; j < E; ++j) top = fmaxf(top, l[j]);
  top = max8(top);
  F total = 0;
#pragma unroll
  for (int j = 0; j < E; ++j) {
    s[j] = l[j] > -INFINITY ? exp(F(l[j]) - F(top)) : F(0);
    total += s[j];
  }
  total = sum8(total);
  const F inv = total > F(0) ? F(1) / total : F(0);
#pragma unroll
  for (int j = 0; j < E; ++j) s[j] *= inv;
}

// The scores s of the adapters in `sel` (bits of the lane's E) over their sum, 0 for the others.  With a
// bias, or sigmoid scores, the chosen ones can all be tiny: a sum below 2^-60 is made again in 64 bits,
// before fp32 loses bits to its smallest numbers and 1 / sum its range.  A single chosen adapter's share is
// exactly 1 (the quotient is corrected once), so that its weight has no gradient.
template <int E>
__device__ __forceinline__ void shares(const float* l, int score, uint32_t sel, bool mine, const float* s, float* p) {
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < E; ++j) {
    p[j] = (sel >> j) & 1u ? s[j] : 0.f;
    sum += p[j];
  }
  sum = sum8(sum);
  const bool tiny = sum < 0x1p-60f;
  const float inv = tiny ? 0.f : 1.f / sum;
#pragma unroll
  for (int j = 0; j < E; ++j) {
    const float q = p[j] * inv;
    p[j] = tiny ? 0.f : fmaf(fmaf(-q, sum, p[j]), inv, q);
  }
  if (!__any(mine && tiny)) return;
  double d[E], total = 0;
  scores<double, E>(l, score, d);
#pragma unroll
  for (int j = 0; j < E; ++j) {
    d[j] = (sel >> j) & 1u ? d[j] : 0.0;
    total += d[j];
  }
  total = sum8(total);
#pragma unroll
  for (int j = 0; j < E; ++j)
    if (tiny) p[j] = total > 0.0 ? (float)(d[j] / total) : 0.f;
}

// Rounds of "largest value, lowest index" over the n values spread over eight lanes (lane i's
// j-th has index base + j step; values of -inf are never taken).  Returns the taken indices;
// *gap is the distance between the last one taken and the largest left (inf where none is).
template <typename F, int E>
__device__ __forceinline__ uint64_t take_largest(F* v, int base, int step, int rounds, F* gap) {
  uint64_t taken = 0;
  F last = INFINITY;
  *gap = INFINITY;
  for (int r = 0; r <= rounds; ++r) {
    F best = v[0];
#pragma unroll
    for (int j = 1; j < E; ++j) best = larger(best, v[j]);
    best = max8(best);
    if (r == rounds) {
      if (best > -INFINITY) *gap = last - best;
      break;
    }
    last = best;
    int at = 64;
#pragma unroll
    for (int j = E - 1; j >= 0; --j) at = v[j] == best ? base + j * step : at;
    at = min8(at);
    if (best > -INFINITY) taken |= 1ull << at;
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] = base + j * step == at ? -INFINITY : v[j];
  }
  return taken;
}

// The chosen adapters of the lane's token.  c: the lane's selection values (destroyed).
// *margin: the narrowest of the decisions' distances.  mem: the wave's kTok * K values.
template <typename F, int E>
__device__ __forceinline__ uint64_t choose(F* c, const RouteScoresArgs& a, int t, int lane8, F* mem, F* margin) {
  *margin = INFINITY;
  if (a.n_group > 1) {
    const int gs = a.K / a.n_group;
    // a group's mark: its largest value plus its second largest where it has one
    auto add = [](F& m1, F& m2, F x) {
      m2 = larger(m2, smaller(m1, x));
      m1 = larger(m1, x);
    };
    auto mark_of = [](F m1, F m2) { return m2 > -INFINITY ? m1 + m2 : m1; };
    uint64_t kept;
    if (gs == E) {  // a lane's adapters are a group
      F m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
      for (int j = 0; j < E; ++j) add(m1, m2, c[j]);
      F mark[1] = {mark_of(m1, m2)};
      kept = take_largest<F, 1>(mark, lane8, 1, a.topk_group, margin);
    } else {
      F* row = mem + t * a.K;
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (lane8 * E + j < a.K) row[lane8 * E + j] = c[j];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      F mark[8];  // groups lane8, lane8 + 8, ...
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        F m1 = -INFINITY, m2 = -INFINITY;
        const int g = lane8 + kLanes * i;
        if (g < a.n_group)
          for (int j = 0; j < gs; ++j) add(m1, m2, row[g * gs + j]);
        mark[i] = mark_of(m1, m2);
      }
      kept = take_largest<F, 8>(mark, lane8, kLanes, a.topk_group, margin);
    }
    const uint32_t inv = (65536u + gs - 1) / gs;  // e / gs for e < 64
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const uint32_t e = lane8 * E + j;
      if (!((kept >> ((e * inv) >> 16)) & 1ull)) c[j] = -INFINITY;
    }
  }
  F gap;
  const uint64_t chosen = take_largest<F, E>(c, lane8 * E, 1, a.k, &gap);
  if (gap < *margin) *margin = gap;
  return chosen;
}

}  // namespace

template <int E>
__global__ __launch_bounds__(kWave * kWaves) void route_scores_k(RouteScoresArgs a) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t = lane / kLanes, lane8 = lane % kLanes;
  const int tok = (blockIdx.x * kWaves + wave) * kTok + t;
  const bool mine = tok < a.N;
  const int e0 = lane8 * E;
  float l[E], s[E], b[E];
  load_logits<E>(a.logits, tok, mine, a.K, e0, l);
#pragma unroll
  for (int j = 0; j < E; ++j) b[j] = a.bias != nullptr && e0 + j < a.K ? a.bias[e0 + j] : 0.f;
  scores<float, E>(l, a.score, s);
  double* mem = reinterpret_cast<double*>(lds) + (size_t)wave * kTok * a.K;
  auto can = [&](int j) { return l[j] > -INFINITY && b[j] > -INFINITY; };  // false for a NaN bias
  uint64_t chosen;
  if (a.bias == nullptr && a.n_group == 1) {
    float c[E];
#pragma unroll
    for (int j = 0; j < E; ++j) c[j] = l[j];
    float margin;
    chosen = choose<float, E>(c, a, t, lane8, nullptr, &margin);
  } else {
    float c[E], margin, scale = 0.f;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      c[j] = can(j) ? s[j] + b[j] : -INFINITY;
      if (can(j)) scale = fmaxf(scale, s[j] + fabsf(b[j]));
    }
    chosen = choose<float, E>(c, a, t, lane8, reinterpret_cast<float*>(mem), &margin);
    // s is within about 8 x 2^-24 of itself, s + bias rounds once and a mark is two of them: decisions
    // nearer than 2^-19 of the largest magnitude are taken again in 64 bits
    const float close = max8(scale) * 0x1p-19f;
    if (__any(mine && !(margin > close))) {
      double s64[E], gap;
      scores<double, E>(l, a.score, s64);
#pragma unroll
      for (int j = 0; j < E; ++j) s64[j] = can(j) ? s64[j] + (double)b[j] : -INFINITY;
      chosen = choose<double, E>(s64, a, t, lane8, mem, &gap);
    }
  }
  if (a.renorm) shares<E>(l, a.score, (uint32_t)(chosen >> e0), mine && chosen != 0, s, s);
  if (!mine) return;
  int32_t* idx = a.idx + (size_t)tok * a.k;
  float* w = a.w + (size_t)tok * a.k;
#pragma unroll
  for (int j = 0; j < E; ++j)
    if ((chosen >> (e0 + j)) & 1ull) {
      const int slot = __popcll(chosen & ((1ull << (e0 + j)) - 1));  // ascending adapter index
      idx[slot] = e0 + j;
      w[slot] = s[j] * a.factor;
    }
  if (lane8 >= __popcll(chosen) && lane8 < a.k) {
    idx[lane8] = -1;
    w[lane8] = 0.f;
  }
}

template <int E>
__global__ __launch_bounds__(kWave * kWaves) void route_scores_bwd_k(RouteScoresArgs a, const float* __restrict__ dw,
                                                                     float* __restrict__ dl) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t = lane / kLanes, lane8 = lane % kLanes;
  const int tok = (blockIdx.x * kWaves + wave) * kTok + t;
  const bool mine = tok < a.N;
  const int e0 = lane8 * E;
  float l[E], s[E], g[E];
  load_logits<E>(a.logits, tok, mine, a.K, e0, l);
  scores<float, E>(l, a.score, s);
  uint32_t sel = 0;
#pragma unroll
  for (int j = 0; j < E; ++j) g[j] = 0.f;
  if (mine)
    for (int i = 0; i < a.k; ++i) {
      const int e = a.idx[(size_t)tok * a.k + i];
      const float v = dw[(size_t)tok * a.k + i];
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (e == e0 + j) {
          g[j] = v * a.factor;
          sel |= 1u << j;
        }
    }
  // softmax: p (g - sum p g); sigmoid the same times 1 - s, the sum only with renorm.  p: s, or its share
  float p[E], dot = 0.f;
#pragma unroll
  for (int j = 0; j < E; ++j) p[j] = s[j];
  if (a.renorm) shares<E>(l, a.score, sel, mine, s, p);
#pragma unroll
  for (int j = 0; j < E; ++j) dot = fmaf(p[j], g[j], dot);
  dot = a.renorm || a.score == kScoreSoftmax ? sum8(dot) : 0.f;
  if (!mine) return;
  float* out = dl + (size_t)tok * a.K + e0;
  float r[E];
#pragma unroll
  for (int j = 0; j < E; ++j) {
    r[j] = p[j] * (g[j] - dot);
    if (a.score == kScoreSigmoid) r[j] *= 1.f - s[j];
    if (!(l[j] > -INFINITY)) r[j] = 0.f;
  }
  if (a.K == kLanes * E) {
    if constexpr (E >= 4) {
#pragma unroll
      for (int q = 0; q < E / 4; ++q)
        st16(out + 4 * q, u32x4_t{__float_as_uint(r[4 * q]), __float_as_uint(r[4 * q + 1]), __float_as_uint(r[4 * q + 2]),
                                  __float_as_uint(r[4 * q + 3])});
    } else {
      *reinterpret_cast<float2*>(out) = make_float2(r[0], r[1]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (e0 + j < a.K) out[j] = r[j];
  }
}

hipError_t launch_route_scores(const RouteScoresArgs& a, hipStream_t s) {
  const dim3 grid((a.N + kTok * kWaves - 1) / (kTok * kWaves)), block(kWave * kWaves);
  const size_t lds = a.n_group > 1 ? (size_t)kWaves * kTok * a.K * sizeof(double) : 0;
  if (a.K <= 16) hipLaunchKernelGGL((route_scores_k<2>), grid, block, lds, s, a);
  else if (a.K <= 32) hipLaunchKernelGGL((route_scores_k<4>), grid, block, lds, s, a);
  else hipLaunchKernelGGL((route_scores_k<8>), grid, block, lds, s, a);
  return hipGetLastError();
}

hipError_t launch_route_scores_backward(const RouteScoresArgs& a, const float* dw, float* dl, hipStream_t s) {
  const dim3 grid((a.N + kTok * kWaves - 1) / (kTok * kWaves)), block(kWave * kWaves);
  if (a.K <= 16) hipLaunchKernelGGL((route_scores_bwd_k<2>), grid, block, 0, s, a, dw, dl);
  else if (a.K <= 32) hipLaunchKernelGGL((route_scores_bwd_k<4>), grid, block, 0, s, a, dw, dl);
  else hipLaunchKernelGGL((route_scores_bwd_k<8>), grid, block, 0, s, a, dw, dl);
  return hipGetLastError();
}

}  // namespace molora
