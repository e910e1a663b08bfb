// CPU test of the decoder operators' host layer (capi_decoder.cpp, decoder_plan.cpp), built with
// AddressSanitizer and UndefinedBehaviorSanitizer on top of the stand-ins of capi_host_test.cpp:
// each launcher here performs, on host memory, every workspace write of the kernels it replaces,
// tile by tile as they place them, on buffers of exactly the queried size.
#define main capi_host_main
#include "capi_host_test.cpp"
#undef main

#include "decoder_launch.h"
#include "molora_decoder.h"

static int g_splits = 0;  // of the last call

namespace molora {

hipError_t launch_route_scores(const RouteScoresArgs&, hipStream_t) {
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_route_scores_backward(const RouteScoresArgs&, const float*, float*, hipStream_t) {
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_kv_append(const KvAppendArgs&, hipStream_t) {
  ++g_launches;
  return hipSuccess;
}

hipError_t launch_attn_forward(const AttnArgs& a, hipStream_t) {
  ++g_launches;
  g_splits = a.splits;
  const long long slots = attn_slots(a.Tq, a.n_seq, kAttnQ);
  if (a.splits > 1)
    for (int c = 0; c < a.splits; ++c)
      for (long long s = 0; s < slots; ++s)
        for (int h = 0; h < a.Hq; ++h)
          write_span<float>(a.part, (size_t)((c * slots + s) * a.Hq + h) * attn_fwd_part_floats(a.D),
                            attn_fwd_part_floats(a.D), "forward parts");
  return hipSuccess;
}

hipError_t launch_attn_backward(const AttnBackwardArgs& b, hipStream_t) {
  ++g_launches;
  const AttnArgs& a = b.f;
  g_splits = b.splits;
  write_span<float>(b.lse2, 0, (size_t)a.Hq * a.Tq, "lse2");
  write_span<float>(b.delta, 0, (size_t)a.Hq * a.Tq, "delta");
  const long long qs = attn_slots(a.Tq, a.n_seq, kAttnQ), ks = attn_slots(a.Tkv, a.n_seq, kAttnK);
  if (b.q_splits > 1)
    for (int c = 0; c < b.q_splits; ++c)
      for (long long s = 0; s < qs; ++s)
        for (int h = 0; h < a.Hq; ++h)
          write_span<float>(b.q_part, (size_t)((c * qs + s) * a.Hq + h) * kAttnQ * a.D, (size_t)kAttnQ * a.D, "dq parts");
  // a key tile's chunks: the sinks' tiles first, then every place's
  const long long sinks = (long long)b.sink_tiles * a.n_seq;
  CHECK(b.sink_tiles == 0 || b.sink_splits > 1, "sinks' tiles apart without a split");
  CHECK((sinks * b.sink_splits + ks * b.splits) * a.Hkv < (1ll << 31), "grid");
  auto part = [&](long long p, int h) {
    write_span<float>(b.part, (size_t)(p * a.Hkv + h) * attn_part_floats(a.D), attn_part_floats(a.D), "key tile parts");
  };
  for (int h = 0; h < a.Hkv; ++h) {
    for (long long p = 0; p < sinks * b.sink_splits; ++p) part(p, h);
    if (b.splits > 1)
      for (long long p = 0; p < ks * b.splits; ++p) part(sinks * b.sink_splits + p, h);
  }
  return hipSuccess;
}

static void decode_writes(int n_seq, int Hq, int Hkv, int D, int splits, float* part) {
  const int head_tiles = (Hq / Hkv + kDecHeads - 1) / kDecHeads;
  if (splits > 1)
    for (long long u = 0; u < (long long)n_seq * Hkv * head_tiles; ++u)
      for (int s = 0; s < splits; ++s)
        write_span<float>(part, (size_t)(u * splits + s) * decode_part_floats(D), decode_part_floats(D), "decode parts");
}
hipError_t launch_attn_decode(const DecodeArgs& a, hipStream_t) {
  ++g_launches;
  g_splits = a.splits;
  decode_writes(a.n_seq, a.Hq, a.c.Hkv, a.c.D, a.splits, a.part);
  return hipSuccess;
}

hipError_t launch_xf_serve(const XfServeLaunch& v, hipStream_t) {
  ++g_launches;
  const XfLaunch& a = v.xf;
  const int N = a.n_seq * a.seq_len, H = a.d / kXfHeadDim;
  const XfServePlan p = xf_serve_plan(N, a.d, a.f, a.lora_bytes, v.part_bytes);
  const size_t nd = (size_t)N * a.d, nf = (size_t)N * a.f;
  write_span<uint16_t>(a.ws + p.h_off, 0, nd, "serve h");
  write_span<uint16_t>(a.ws + p.q_off, 0, nd, "serve q");
  write_span<uint16_t>(a.ws + p.k_off, 0, nd, "serve k");
  write_span<uint16_t>(a.ws + p.v_off, 0, nd, "serve v");
  write_span<uint16_t>(a.ws + p.att_off, 0, nd, "serve att");
  write_span<uint16_t>(a.ws + p.o_off, 0, nd, "serve o");
  write_span<uint16_t>(a.ws + p.g_off, 0, nf, "serve gate");
  write_span<uint16_t>(a.ws + p.u_off, 0, nf, "serve up");
  write_span<char>(a.ws + p.blas_off, 0, p.blas_bytes, "serve blas");
  write_span<char>(a.ws + p.lora_off, 0, a.lora_bytes, "serve lora");
  if (v.q_off == nullptr) decode_writes(v.n_seq, H, H, kXfHeadDim, v.splits, reinterpret_cast<float*>(a.ws + p.part_off));
  return hipSuccess;
}

}  // namespace molora

static molora_rows rows(int heads, int D) { return {fake(0x10000), (long long)heads * D, D}; }

static void with_workspace(size_t need, const char* name, int launches,
                           int (*call)(void*, size_t, void*), void* ctx) {
  if (need > kMaxBuf) return;
  char* ws = static_cast<char*>(exact_alloc(need));
  g_ws_base = ws;
  g_ws_bytes = need;
  g_ranges.clear();
  const int l0 = g_launches;
  int rc = call(need > 0 ? ws : nullptr, need, ctx);
  CHECK(rc == MOLORA_OK && g_launches == l0 + launches, "%s", name);
  check_disjoint(name);
  if (need > 0) {
    CHECK(call(ws, need - 1, ctx) == MOLORA_ENOSPC && call(nullptr, need, ctx) == MOLORA_ENOSPC, "%s: short workspace", name);
    CHECK(g_launches == l0 + launches, "%s launched without its workspace", name);
  }
  g_ws_base = nullptr;
  free(ws);
}

static void test_attention(int n_seq, int Hq, int Hkv, int D, int Tq, int Tkv, int window, int sinks) {
  molora_attn_shape s{n_seq, Hq, Hkv, D, Tq, Tkv, (const int32_t*)fake(0x1000), nullptr, window, sinks, 0.1f};
  const int some = n_seq > 0 && Tq > 0, any = n_seq > 0 && (Tq > 0 || Tkv > 0);
  size_t need = 0;
  CHECK(molora_attn_forward_workspace(&s, &need) == MOLORA_OK, "forward workspace");
  auto fwd = [](void* ws, size_t n, void* c) {
    const molora_attn_shape* s = static_cast<molora_attn_shape*>(c);
    const molora_rows q = rows(s->n_heads, s->head_dim), k = rows(s->n_kv_heads, s->head_dim);
    return molora_attn_forward(s, &q, &k, &k, &q, (float*)fake(0x2000), ws, n, nullptr);
  };
  if (some) with_workspace(need, "attn_forward", 1, fwd, &s);
  CHECK(molora_attn_backward_workspace(&s, &need) == MOLORA_OK, "backward workspace");
  auto bwd = [](void* ws, size_t n, void* c) {
    const molora_attn_shape* s = static_cast<molora_attn_shape*>(c);
    const molora_rows q = rows(s->n_heads, s->head_dim), k = rows(s->n_kv_heads, s->head_dim);
    return molora_attn_backward(s, &q, &q, &k, &k, &q, (float*)fake(0x2000), &q, &k, &k, ws, n, nullptr);
  };
  if (any) with_workspace(need, "attn_backward", 1, bwd, &s);
}

struct DecodeCase {
  molora_kv_cache c;
  int n_seq, Hq, width;
};
static void test_decode(int n_seq, int Hq, int Hkv, int D, int page, int width, int dtype) {
  DecodeCase t{{fake(0x1000), fake(0x2000), (uint8_t*)fake(0x3000), (uint8_t*)fake(0x4000), 8, Hkv, page, D, dtype},
               n_seq, Hq, width};
  size_t need = 0;
  CHECK(molora_attn_decode_workspace(&t.c, n_seq, Hq, width, &need) == MOLORA_OK, "decode workspace");
  auto go = [](void* ws, size_t n, void* c) {
    const DecodeCase* t = static_cast<DecodeCase*>(c);
    const molora_rows q = rows(t->Hq, t->c.head_dim);
    return molora_attn_decode(&t->c, &q, &q, nullptr, t->n_seq, t->Hq, (int32_t*)fake(0x5000), t->width,
                              (int32_t*)fake(0x6000), 0, 0, 0.1f, ws, n, nullptr);
  };
  if (n_seq > 0) with_workspace(need, "attn_decode", 1, go, &t);
}

struct ServeCase {
  int d, f, L, n_seq, N, width, k;
  std::vector<molora_xf_layer> layers;
  std::vector<molora_kv_cache> caches;
  bool single;
};
static void test_serve(int d, int f, int L, int n_seq, int N, int K, int r, int k, int width) {
  std::vector<HostHotset> hs(L);
  ServeCase t{d, f, L, n_seq, N, width, k, {}, {}, N == n_seq};
  for (int l = 0; l < L; ++l) {
    molora_xf_layer X{};
    X.norm1 = fake(0x1000);
    X.norm2 = fake(0x1100);
    for (int i = 0; i < 7; ++i) X.W[i] = fake(0x2000 + 0x100 * i);
    if (K > 0) {
      if (!make_hotset(hs[l], K, r, {{d, d}, {d, d}, {d, d}, {d, d}, {d, f}, {d, f}, {f, d}}, MOLORA_LAYOUT_DIRECT)) return;
      X.lora = hs[l].hs;
    }
    t.layers.push_back(X);
    t.caches.push_back({fake(0x1000), fake(0x2000), nullptr, nullptr, 8, d / 128, 16, 128, MOLORA_BF16});
  }
  auto go = [](void* ws, size_t n, void* c) {
    const ServeCase* t = static_cast<ServeCase*>(c);
    int32_t* p = (int32_t*)fake(0x8000);
    if (t->single)
      return molora_xf_decode(t->d, t->f, t->L, t->layers.data(), t->caches.data(), t->n_seq, p, t->width, p, 0, 0,
                              fake(0x3000), fake(0x4000), t->k, p, p, (float*)p, p, ws, n, nullptr);
    return molora_xf_prefill(t->d, t->f, t->L, t->layers.data(), t->caches.data(), t->n_seq, t->N, p, p, t->width, p, 0, 0,
                             fake(0x3000), fake(0x4000), t->k, p, p, (float*)p, p, ws, n, nullptr);
  };
  size_t need = 0;
  CHECK(molora_xf_serve_workspace(d, f, L, t.layers.data(), t.caches.data(), n_seq, N, width, k, &need) == MOLORA_OK, "serve");
  if (need <= kMaxBuf) {
    char* ws = static_cast<char*>(exact_alloc(need));
    g_ws_base = ws;
    g_ws_bytes = need;
    g_ranges.clear();
    const int l0 = g_launches;
    CHECK(go(ws, need, &t) == MOLORA_OK && g_launches == l0 + 1, "xf_serve");
    check_disjoint("xf_serve");
    CHECK(go(ws, 256, &t) == MOLORA_ENOSPC && g_launches == l0 + 1, "xf_serve: short workspace");
    g_ws_base = nullptr;
    free(ws);
  }
  if (K > 0 && L > 1) {  // adapters of two ranks
    HostHotset other;
    if (make_hotset(other, K, r + 16, {{d, d}, {d, d}, {d, d}, {d, d}, {d, f}, {d, f}, {f, d}}, MOLORA_LAYOUT_DIRECT)) {
      t.layers[1].lora = other.hs;
      CHECK(molora_xf_serve_workspace(d, f, L, t.layers.data(), t.caches.data(), n_seq, N, width, k, &need) == MOLORA_ENOTSUP,
            "two ranks accepted");
      molora_hotset_destroy(other.hs);
    }
  }
  for (auto& h : hs) molora_hotset_destroy(h.hs);
}

// The search key of a tile's slot: two sequences never meet, and every tile has a slot.
static void test_slots() {
  unsigned seed = 7;
  for (int trial = 0; trial < 200; ++trial) {
    int off = 0, end = 0, n_seq = 1 + trial % 40;
    for (int s = 0; s < n_seq; ++s) {
      seed = seed * 1664525u + 1013904223u;
      const int len = (seed >> 16) % (trial % 3 ? 300 : 5), first = (int)attn_slot0(off, s, kAttnQ);
      CHECK(first >= end, "slots meet");
      end = first + (len + kAttnQ - 1) / kAttnQ;
      off += len;
    }
    CHECK(end <= attn_slots(off, n_seq, kAttnQ), "slots past the grid");
  }
}

int main() {
  test_slots();
  for (int n_seq : {0, 1, 3, 40})
    for (int Tq : {0, 1, 63, 130, 1000})
      for (int Tkv : {0, 5, 1000, 6000})
        for (int window : {0, 64, 4000})
          for (int sinks : {0, 4, 300})
            for (int D : {64, 128}) test_attention(n_seq, 4, 2, D, Tq, Tkv, window, sinks);
  test_attention(1, 32, 8, 64, 8192, 8192, 1024, 16);
  test_attention(1, 1, 1, 64, 16000, 16000, 0, 0);
  test_attention(2000, 8, 8, 64, 5000, 5000, 100, 100);
  for (int dtype : {(int)MOLORA_BF16, (int)MOLORA_E4M3})
    for (int n_seq : {0, 1, 5, 300})
      for (int heads : {1, 16, 17, 40})
        for (int width : {0, 1, 40, 600})
          for (int D : {64, 128}) test_decode(n_seq, heads * 2, 2, D, 16, width, dtype);
  test_decode(1, 32, 8, 128, 256, 4000000, MOLORA_BF16);
  for (int K : {0, 4})
    for (int k : {1, 2})
      for (int N : {4, 100}) test_serve(256, 768, 2, 4, N, K, 16, k, 50);
  test_serve(512, 1408, 1, 40, 40, 3, 8, 1, 3);
  free(g_scratch);
  fprintf(stderr, "%d checks, %d failures\n", g_checks, g_fail);
  return g_fail == 0 ? 0 : 1;
}
