// What the C-ABI layers share: the hot-set descriptor, the error message of the calling thread
// and the checks of the decoder's model description.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <vector>

#include "molora.h"
#include "molora_launch.h"

struct molora_hotset {
  int K = 0, r = 0, r_pad = 0, layout = 0, n_targets = 0;
  float scale = 1.f;
  bool transposed = false;  // holds (B^T, A^T) of the given adapters (molora_hotset_init_transposed)
  std::vector<molora::TargetDev> tg;
  void* slab = nullptr;
  size_t slab_bytes = 0;
  // host copies of every adapter's slot addresses, [target][adapter] (both layouts)
  std::vector<std::vector<uint16_t*>> slotA, slotB;
};

namespace molora {

int fail(int code, const char* fmt, ...);         // sets the thread's message, returns code
int ok();                                         // clears it, returns MOLORA_OK
int hip_fail(hipError_t e, const char* what);     // MOLORA_EHIP with the runtime's message
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Shapes of the decoder's seven LoRA targets (q, k, v, o, gate, up, down).
void xf_dims(int d, int f, int* din, int* dout);
// Checks a decoder's layers for a batch of N tokens; on success *K is the adapters per target
// (0: no layer has LoRA), *lora_bytes the largest workspace of one layer's applies and paths
// (NULL or [4]) the resolved apply paths of q/k/v, o, gate/up and down.
int xf_check_layers(int d, int f, int n_layers, const molora_xf_layer* layers, long long N, int k, int* K,
                    size_t* lora_bytes, int* paths);
// The launchers' form of the layers.
void xf_layers_dev(int n_layers, const molora_xf_layer* layers, XfLayerDev* dev);

}  // namespace molora
