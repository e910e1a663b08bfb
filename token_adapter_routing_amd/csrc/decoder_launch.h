// Host-side launchers of the decoder's operators (internal to the library).  Every launcher
// assumes its arguments were validated by the C-ABI layer and only enqueues work.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "decoder_plan.h"
#include "molora_launch.h"

namespace molora {

enum { kScoreSoftmax = 0, kScoreSigmoid = 1 };

struct RouteScoresArgs {
  const float* logits;
  const float* bias;  // or NULL
  int N, K, k, score, n_group, topk_group, renorm;
  float factor;
  int32_t* idx;  // the backward reads it
  float* w;
};
hipError_t launch_route_scores(const RouteScoresArgs& a, hipStream_t s);
hipError_t launch_route_scores_backward(const RouteScoresArgs& a, const float* dw, float* dl, hipStream_t s);

// Rows of packed tensors: element strides between tokens and heads.
struct Rows {
  uint16_t* p;
  long long token, head;
};
struct AttnArgs {
  Rows q, k, v, o;
  float* lse;  // [Hq][Tq] or NULL
  const int32_t* q_off;
  const int32_t* kv_off;
  int n_seq, Hq, Hkv, D, Tq, Tkv, window, sinks;
  float scale;
  int splits;   // attn_q_splits; the forward's parts in part
  float* part;  // splits > 1: [splits][query tile slots][Hq] x attn_fwd_part_floats
};
hipError_t launch_attn_forward(const AttnArgs& a, hipStream_t s);

struct AttnBackwardArgs {
  AttnArgs f;  // o and lse as the forward wrote them
  Rows dout, dq, dk, dv;
  float* lse2;   // workspace [Hq][Tq]: lse in base 2
  float* delta;  // workspace [Hq][Tq]: -rowsum(dO O)
  int q_splits;   // attn_q_splits
  float* q_part;  // workspace: the split query tiles' sums
  int splits, sink_splits, sink_tiles, most, min_steps, sink_min;  // attn_bwd_plan
  float* part;   // workspace: the split key tiles' sums
};
hipError_t launch_attn_backward(const AttnBackwardArgs& a, hipStream_t s);

struct KvCacheDev {
  void* k;
  void* v;
  uint8_t* k_scale;  // e4m3 only
  uint8_t* v_scale;
  int n_pages, Hkv, page_shift, D;
  bool e4m3;
};
struct KvAppendArgs {
  KvCacheDev c;
  Rows k, v;
  int T, n_seq;
  const int32_t* q_off;  // NULL: one row per sequence
  const int32_t* table;
  int width;
  const int32_t* lens;
};
hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t s);

struct DecodeArgs {
  KvCacheDev c;
  Rows q, o;
  float* lse;  // [n_seq][Hq] or NULL
  int n_seq, Hq;
  const int32_t* table;
  int width;
  const int32_t* lens;
  int window, sinks;
  float scale;
  int splits;   // decode_plan
  float* part;  // decode_plan, splits > 1
};
hipError_t launch_attn_decode(const DecodeArgs& a, hipStream_t s);

// The decoder over a paged cache per layer (xfmr.cpp): xf holds n_seq * seq_len = the new tokens.
struct XfServeLaunch {
  XfLaunch xf;
  const KvCacheDev* caches;  // [n_layers]
  int n_seq;
  const int32_t* q_off;  // prompts; NULL: one token per sequence
  const int32_t* table;
  int width;
  const int32_t* lens;
  int window, sinks;
  int splits;         // decode_plan, single tokens
  size_t part_bytes;  // its workspace
};
hipError_t launch_xf_serve(const XfServeLaunch& a, hipStream_t s);

}  // namespace molora
