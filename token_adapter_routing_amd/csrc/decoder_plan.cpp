// Workspace arithmetic of the decoder's operators (HIP-free).
#include "decoder_plan.h"

#include <algorithm>

namespace molora {

// Splits: enough workgroups (kDecTarget) that sequences of different lengths even out over the
// 256 CUs, no more than the longest possible sequence has pieces of kDecMinBlocks blocks.
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
