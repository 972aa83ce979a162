// Decode attention over a quantised cache of fp16 inputs.
#include "quant_decode.cuh"

namespace spd {

cudaError_t launch_quant_attend_f16(const QuantAttendParams &p, int d, int bits, int G,
                                   cudaStream_t st) {
  const cudaError_t e = p.out_f32 ? launch_shape<__half, true>(p, d, bits, G, st)
                                  : launch_shape<__half, false>(p, d, bits, G, st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace spd
