// Rotary positions of q and k (sm_103a): spd_rotary.
//
// Bound by memory: every value is read and written once, 4 bytes.  A CTA takes a few whole
// tokens: it makes their sines and cosines once in shared memory (as many as pairs, where q
// and k have heads times as many), then its threads walk the tokens' rows in units of two
// 16-byte vectors.
#include "ptx.cuh"
#include "rotary.cuh"

namespace spd {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;  // per CTA

template <typename T>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
  __shared__ __align__(16) float2 cs[kMaxTokens * 64];
  pdl_wait();
  pdl_launch_dependents();
  const int t0 = blockIdx.x * p.tokens_per_cta, nt = min(p.tokens_per_cta, p.n - t0);
  const RotaryShape s{p.table.head_dim, p.table.rotary_dim, p.table.neighbours};
  const int pairs = s.rot >> 1;
  for (int i = threadIdx.x; i < nt * pairs; i += kThreads) {
    const int t = i / pairs, j = i - t * pairs;
    float2 e = turn_of(p.positions[(long long)p.table.axis[j] * p.n + t0 + t], p.table.turns[j]);
    if (p.inverse) e.y = -e.y;
    cs[i] = e;
  }
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
    w.turn(s, cs + t * pairs);
    w.store(dst);
  }
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams &p, int dtype, cudaStream_t st) {
  const int grid = (p.n + p.tokens_per_cta - 1) / p.tokens_per_cta;
  cudaError_t e = dtype == 0 ? launch_pdl(rotary_kernel<__half>, grid, kThreads, 0, st, p)
                             : launch_pdl(rotary_kernel<__nv_bfloat16>, grid, kThreads, 0, st, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace spd
