// decode_window_codes.cu -- the windowed kernels of decode attention over quantised caches.
#include "decode_kernel.cuh"

namespace pda {

KernelFn pick_window_codes_kernel(pda_dtype kv, int D, int G_u, int mode) {
  if (kv == PDA_NVFP4) return pick_d<nvfp4, __nv_bfloat16, true>(D, G_u, mode);
  return pick_d<fp8e4m3, __nv_bfloat16, true>(D, G_u, mode);
}

}  // namespace pda
