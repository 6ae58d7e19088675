// decode_window.cu -- the windowed kernels of decode attention over plain caches.
#include "decode_kernel.cuh"

namespace pda {

KernelFn pick_window_kernel(pda_dtype kv, int D, int G_u, int mode) {
  if (kv == PDA_F16) return pick_d<__half, __half, true>(D, G_u, mode);
  if (kv == PDA_BF16) return pick_d<__nv_bfloat16, __nv_bfloat16, true>(D, G_u, mode);
  return pick_d<float, float, true>(D, G_u, mode);
}

}  // namespace pda
