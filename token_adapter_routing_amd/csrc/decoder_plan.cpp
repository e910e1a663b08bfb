// Workspace arithmetic of the decoder's operators (HIP-free).
#include "decoder_plan.h"

#include <algorithm>

namespace molora {

// Splits: enough workgroups (kDecTarget) that sequences of different lengths even out over the
// 256 CUs, no more than the longest possible sequence has pieces of kDecMinBlocks blocks.  64 ragged
// sequences of up to 8192, 8 key-value heads: 239 / 214 / 203 / 207 us with 512 / 1024 / 2048 / 4096; one
// of 32771: 31.4 / 30.2 / 30.0 / 29.8 us.
DecodePlan decode_plan(int n_seq, int n_heads, int n_kv_heads, int head_dim, int page_size, int table_width) {
  constexpr long long kDecTarget = 2048;
  DecodePlan p{};
  const int group = n_heads / n_kv_heads;
  p.head_tiles = (group + kDecHeads - 1) / kDecHeads;
  p.units = (long long)n_seq * n_kv_heads * p.head_tiles;
  const long long blocks = ((long long)page_size * table_width + kDecBlock - 1) / kDecBlock;
  const long long most = std::max(1ll, (blocks + kDecMinBlocks - 1) / kDecMinBlocks);
  const long long want = p.units > 0 ? (kDecTarget + p.units - 1) / p.units : 1;
  p.splits = (int)std::min(want, most);
  p.part_floats = p.splits > 1 ? (size_t)p.units * p.splits * decode_part_floats(head_dim) : 0;
  p.total = align256(p.part_floats * sizeof(float));
  return p;
}

// Splits: up to kQTarget workgroups, one for each of the 512 places, counted by the work of an average tile:
// with as many queries as keys it is half of the longest one, which then sets the time (8192 tokens, 4 heads
// of 128, 260 tiles: forward 155 us whole, 108 us split; 4096 tokens, 8 heads, 264 tiles: 79 and 62 us).
// Sequences of kQKeys keys on average (512 keys gain nothing: 15.8 us whole, 17.1 us split; 1024 keys
// 24.4 us whole, 18.4 us split); of more where the tiles alone give every CU a workgroup, whose parts have
// to be written and joined too (2048 tokens, 16 heads, 272 tiles: 43 and 41 us; 1024 tokens, 32 heads, 288
// tiles: 26 and 34 us).
constexpr long long kQTarget = 512, kQKeys = 768;
int attn_q_splits(int Tq, int Tkv, int n_seq, int n_heads, int window, int sinks) {
  const long long units = attn_slots(Tq, n_seq, kAttnQ) * n_heads;
  if (units <= 0 || Tkv == 0 || Tkv < n_seq * (units < kQTarget / 2 ? kQKeys : 7 * units)) return 1;
  long long keys = Tkv, target = kQTarget;
  if (window > 0 && window < Tkv) keys = std::min(keys, (long long)window + sinks + 2 * kAttnQ);
  else target = kQTarget * 2 * Tkv / (2ll * Tkv - std::min(Tq, Tkv));
  const long long tiles = (keys + 63) / 64;
  return (int)std::max(1ll, std::min({target / units, (tiles + kAttnMinTiles - 1) / kAttnMinTiles, 16ll}));
}

size_t attn_fwd_ws_bytes(int Tq, int Tkv, int n_seq, int n_heads, int head_dim, int window, int sinks) {
  const int splits = attn_q_splits(Tq, Tkv, n_seq, n_heads, window, sinks);
  if (splits == 1) return 0;
  return align256((size_t)splits * attn_slots(Tq, n_seq, kAttnQ) * n_heads * attn_fwd_part_floats(head_dim) * sizeof(float));
}

// A causal sequence's key tiles are seen by unequal numbers of queries, so with few tiles the longest
// one sets the time: chunks until there are kBwdTarget workgroups, two for each of the 512 places
// that two waves per SIMD leave (8192 tokens, 32 / 8 heads of 128: dk / dv 1575 us unsplit, 1162 us
// and 19 us for the join in 2 chunks).  Few tiles of long sequences (kQKeys): one workgroup for each place,
// in chunks down to 384 rows (1024 tokens, 4 heads of 128: backward 71 us with whole tiles, 52 us).
// With a window a tile sees a window's worth, but the sinks' tiles every query: those are taken apart, in
// chunks half as long as the others' (8192 tokens, 32 / 8 heads of 64, window 1024, 16 sinks: dk / dv
// 1008 us unsplit, 198 us and 5 us for the join in 14 chunks; 4096 tokens, 16 / 1 heads of 64, window 512,
// 4 sinks: backward 172 us in 16 chunks, 87 us in 64).
AttnBwdPlan attn_bwd_plan(int Tq, int Tkv, int n_seq, int n_heads, int n_kv_heads, int head_dim, int window, int sinks) {
  constexpr long long kBwdTarget = 1024, kBwdPartBytes = 512ll << 20;
  AttnBwdPlan p{};
  const long long slots = attn_slots(Tkv, n_seq, kAttnK), units = slots * n_kv_heads, group = n_heads / n_kv_heads;
  const long long rows = attn_step(head_dim), steps = ((long long)Tq + rows - 1) / rows * group;
  const long long bytes = (long long)(attn_part_floats(head_dim) * sizeof(float));
  const bool few = units > 0 && units < kQTarget / 2 && Tq >= kQKeys * n_seq;
  const long long min_steps = (few ? 384 : 1024) / rows;
  p.sink_min = (int)(1024 / rows);
  p.min_steps = (int)min_steps;
  const bool windowed = window > 0 && window < Tq;
  p.most = (int)std::min(steps, windowed ? ((long long)window + kAttnK + 2 * rows - 2) / rows * group : steps);
  p.splits = p.sink_splits = 1;
  if (units > 0) {
    const long long target = windowed || few ? kBwdTarget / 2 : kBwdTarget;  // a window's tiles are equally long
    p.splits = (int)std::max(1ll, std::min({(target + units - 1) / units, 16ll,
                                            ((long long)p.most + min_steps - 1) / min_steps,
                                            kBwdPartBytes / (units * bytes)}));
    if (windowed && sinks > 0) {
      const long long per_seq = (std::min((long long)sinks, (long long)Tkv) + kAttnK - 1) / kAttnK;
      const long long tiles = per_seq * n_seq;
      const long long per = std::max((long long)p.sink_min, ((long long)p.most / p.splits + 1) / 2);
      const long long n = tiles <= 0 ? 1
                                     : std::min({2 * kBwdTarget / (tiles * n_kv_heads), 64ll, (steps + per - 1) / per,
                                                 kBwdPartBytes / (tiles * n_kv_heads * bytes)});
      if (n > 1) {
        p.sink_splits = (int)n;
        p.sink_tiles = (int)per_seq;
      }
    }
  }
  const size_t stat = align256((size_t)Tq * n_heads * sizeof(float));
  const long long parts = (p.sink_tiles > 0 ? (long long)p.sink_tiles * n_seq * p.sink_splits : 0) +
                          (p.splits > 1 ? slots * p.splits : 0);
  p.lse_off = 0;
  p.delta_off = stat;
  p.part_off = 2 * stat;
  p.q_splits = attn_q_splits(Tq, Tkv, n_seq, n_heads, window, sinks);
  p.q_part_off = p.part_off + (size_t)(parts * n_kv_heads * bytes);
  p.total = p.q_part_off;
  if (p.q_splits > 1)
    p.total += align256((size_t)p.q_splits * attn_slots(Tq, n_seq, kAttnQ) * n_heads * kAttnQ * head_dim * sizeof(float));
  return p;
}

XfServePlan xf_serve_plan(int N, int d, int f, size_t lora_bytes, size_t part_bytes) {
  XfServePlan p{};
  const size_t nd = align256((size_t)N * d * sizeof(uint16_t)), nf = align256((size_t)N * f * sizeof(uint16_t));
  size_t off = 0;
  for (size_t* at : {&p.h_off, &p.q_off, &p.k_off, &p.v_off, &p.att_off, &p.o_off}) {
    *at = off;
    off += nd;
  }
  for (size_t* at : {&p.g_off, &p.u_off}) {
    *at = off;
    off += nf;
  }
  p.part_off = off;
  off += align256(part_bytes);
  p.lora_off = off;
  off += align256(lora_bytes);
  p.blas_off = off;
  p.blas_bytes = kXfBlasBytes;
  p.total = off + p.blas_bytes;
  return p;
}

}  // namespace molora
