// Sizes and index formulas shared by the host layer and the kernels of the decoder's operators.
// Plain C++ without HIP types (see molora_plan.h).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "molora_plan.h"

namespace molora {

// ---- attention over packed sequences: query tiles of kAttnQ rows.  Sequence s owns the tile
// slots from q_off[s] / kAttnQ + s on: floor((a + L) / t) + 1 >= floor(a / t) + ceil(L / t), so
// the slots of two sequences never meet, a slot's sequence is found by search in q_off itself,
// and T / kAttnQ + n_seq slots cover every tile.
constexpr int kAttnQ = 128;   // query rows per workgroup of the forward and the dq pass
constexpr int kAttnK = 128;   // key rows per workgroup of the dk / dv pass
MOLORA_HD inline long long attn_slot0(int off, int s, int tile) { return (long long)(off / tile) + s; }
MOLORA_HD inline long long attn_slots(int T, int n_seq, int tile) { return (long long)(T / tile) + n_seq; }

// Few query tiles before many keys: the forward and the dq pass split a tile's key tiles over up to
// attn_q_splits() workgroups, at least kAttnMinTiles of 64 keys each, and join the parts.
constexpr int kAttnMinTiles = 6;
int attn_q_splits(int Tq, int Tkv, int n_seq, int n_heads, int window, int sinks);
MOLORA_HD inline size_t attn_fwd_part_floats(int head_dim) { return (size_t)kAttnQ * (head_dim + 2); }
size_t attn_fwd_ws_bytes(int Tq, int Tkv, int n_seq, int n_heads, int head_dim, int window, int sinks);

// Backward: lse in base 2 and rowsum(dO O), fp32 [heads][Tq] each, then the sums of the key tiles that
// are split into chunks, [2][kAttnK][head_dim] fp32 per (tile, chunk, kv head): first the sinks' tiles
// (sink_tiles > 0: that many of every sequence, in sink_splits chunks), then the others (splits > 1).
// Query rows per step of the dk / dv pass: with heads of 64 twice as many fit in LDS beside three
// waves per SIMD, which halves the waits between steps.
MOLORA_HD constexpr int attn_step(int head_dim) { return head_dim == 64 ? 64 : 32; }
struct AttnBwdPlan {
  int splits, sink_splits, sink_tiles;
  int most;       // steps of the longest tile that is not a sinks' tile
  int min_steps;  // per chunk of it
  int sink_min;   // per chunk of a sinks' tile
  int q_splits;
  size_t lse_off, delta_off, part_off, q_part_off, total;
};
AttnBwdPlan attn_bwd_plan(int Tq, int Tkv, int n_seq, int n_heads, int n_kv_heads, int head_dim, int window, int sinks);
MOLORA_HD inline size_t attn_part_floats(int head_dim) { return (size_t)2 * kAttnK * head_dim; }

// ---- decode attention: blocks of kDecBlock positions; a sequence's visible blocks are split
// evenly over `splits` workgroups, at least kDecMinBlocks each.  Partial results per (sequence,
// head tile, split): kDecHeads rows of head_dim sums (fp32), then the maxima and the sums of
// weights.
constexpr int kDecBlock = 32;
constexpr int kDecHeads = 16;     // query heads per workgroup (one matrix-instruction column block)
constexpr int kDecMinBlocks = 8;  // two per wave
struct DecodePlan {
  int head_tiles;  // workgroups per key-value head: ceil(query heads per kv head / kDecHeads)
  long long units;  // n_seq * n_kv_heads * head_tiles
  int splits;
  size_t part_floats, total;
};
DecodePlan decode_plan(int n_seq, int n_heads, int n_kv_heads, int head_dim, int page_size, int table_width);
MOLORA_HD inline size_t decode_part_floats(int head_dim) { return (size_t)kDecHeads * (head_dim + 2); }
MOLORA_HD inline int decode_blocks_per_split(int blocks, int splits) {
  const int per = ((blocks + splits - 1) / splits + 3) / 4 * 4;  // the four waves take as many each
  return per < kDecMinBlocks ? kDecMinBlocks : per;
}

// ---- the synthetic decoder's serving form over N new tokens: the activations of xf_plan without
// scores and probabilities, the decode attention's parts, the applies' and the GEMM library's
// workspaces.
struct XfServePlan {
  size_t h_off, q_off, k_off, v_off, att_off, o_off, g_off, u_off;
  size_t part_off, lora_off, blas_off, blas_bytes, total;
};
XfServePlan xf_serve_plan(int N, int d, int f, size_t lora_bytes, size_t part_bytes);

}  // namespace molora
