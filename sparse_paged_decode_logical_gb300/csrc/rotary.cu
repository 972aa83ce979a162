// Rotary positions of q and k (sm_103a): spd_rotary, and the queries of long appends.
//
// Bound by memory: every value is read and written once, 4 bytes.  A CTA takes a few whole
// tokens: it makes their sines and cosines once in shared memory (as many as pairs, where q and
// k have heads times as many), then its threads walk the tokens' rows in units of two 16-byte
// vectors.  What counts is threads in flight: 20,011 tokens of 40 heads take 64.4 us (6.4 TB/s, 94%
// of the measured copy rate) with 32 to 36 registers a thread; 80 with two units of a thread under
// way in 54 registers, 87 with rows that come by asynchronous copies through shared memory, 16
// warps an SM.
#include "ptx.cuh"
#include "rotary.cuh"

namespace spd {
namespace {

constexpr int kThreads = 256;

// PLACES: a token's position is its place in its sequence.
template <typename T, bool PLACES>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryParams p,
                                                          const __grid_constant__ RotaryPlaces at) {
  __shared__ __align__(16) float2 cs[kRotaryTokens * sine_stride(128)];
  pdl_wait();
  pdl_launch_dependents();
  const int t0 = blockIdx.x * p.tokens_per_cta, nt = min(p.tokens_per_cta, p.n - t0);
  const RotaryShape s{p.table.head_dim, p.table.rotary_dim, p.table.neighbours};
  make_sines<kThreads>(p.table, nt, p.inverse, cs, [&](int axis, int t) {
    if constexpr (PLACES) {
      const int i = (t0 + t) / at.n_tokens;
      return at.first[i] + (t0 + t) - i * at.n_tokens;
    }
    return p.positions[(long long)axis * p.axis_stride + t0 + t];
  });
  __syncthreads();
  const int units = s.units(), heads = p.hq + p.hkv, row_units = heads * units;
  for (int i = threadIdx.x; i < nt * row_units; i += kThreads) {
    const int t = i / row_units, r = i - t * row_units, h = r / units, u = r - h * units;
    const long long tok = t0 + t;
    const T *src;
    T *dst;
    if (h < p.hq) {
      src = static_cast<const T *>(p.q) + tok * p.q_stride + h * s.d;
      dst = static_cast<T *>(p.q_out) + tok * p.q_out_stride + h * s.d;
    } else {
      src = static_cast<const T *>(p.k) + tok * p.k_stride + (h - p.hq) * s.d;
      dst = static_cast<T *>(p.k_out) + tok * p.k_out_stride + (h - p.hq) * s.d;
    }
    RotaryUnit<T> w;
    w.load(s, src, u);
    w.turn(s, cs + t * sine_stride(s.rot));
    w.store(dst);
  }
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams &p, const RotaryPlaces *places, int dtype,
                          cudaStream_t st) {
  const int grid = (p.n + p.tokens_per_cta - 1) / p.tokens_per_cta;
  static const RotaryPlaces none{};
  const RotaryPlaces &at = places ? *places : none;
  cudaError_t e;
  if (dtype == 0)
    e = launch_pdl(places ? rotary_kernel<__half, true> : rotary_kernel<__half, false>, grid, kThreads,
                   0, st, p, at);
  else
    e = launch_pdl(places ? rotary_kernel<__nv_bfloat16, true> : rotary_kernel<__nv_bfloat16, false>,
                   grid, kThreads, 0, st, p, at);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace spd
