// Decode attention over a quantised cache of bf16 inputs.
#include "quant_decode.cuh"

namespace spd {

cudaError_t launch_quant_attend_bf16(const QuantAttendParams &p, int d, int bits, int G,
                                   cudaStream_t st) {
  const cudaError_t e = p.out_f32 ? launch_shape<__nv_bfloat16, true>(p, d, bits, G, st)
                                  : launch_shape<__nv_bfloat16, false>(p, d, bits, G, st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace spd
