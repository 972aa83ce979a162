// Decode attention over a quantised cache (sm_103a): spd_quant_decode_attention.
//
// With value = lo + step code for keys and values alike,
//   q . k_t = sum over groups a of  lo_ta (sum of q in a) + step_ta (q . codes in a)
//   sum_t p_t v_t = sum_t p_t lo_ta + sum_t (p_t step_ta) codes_t
// so that the matrix products run over the codes themselves, which an fp16 operand holds
// exactly: an integer of 8 or 4 bits in the low bits of an fp16 number is that integer times
// 2^-24 (a subnormal, which the tensor cores take at full precision), 2^-20 four bits higher.
// A word of codes becomes operands by masks and shifts alone: 5 instructions for 8 codes of 4
// bits, 3 for 4 of 8.  (tcgen05 has no use here: it reads operands from shared or tensor
// memory, where the widened codes would first have to be written.)
//
// The products are transposed, S = K q and O = V p, so that a kv head's 1 to 8 query heads are
// the short side (n = 8) of m16n8k16; scores reach the second product by movmatrix.  Where at
// most four heads share the keys, the columns behind them hold copies: their lanes make the low
// halves of the weights, so that weights in two fp16 parts cost no product more.
//
// Bound by memory: the cache is read once.  Every warp walks a stretch of tiles through its own
// ring of bulk copies, without a barrier between warps; the launch's warps share all sequences'
// tiles evenly, a warp may end one unit (sequence, kv head) and start the next.  What a warp
// holds of a unit that others hold parts of, too, is joined in the CTA, then over CTAs by the
// last one to finish.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include <atomic>

#include "dense_math.cuh"
#include "ptx.cuh"
#include "rotary.cuh"
#include "spd_internal.h"

namespace spd {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr uint32_t kWaitPolls = 1u << 22;
constexpr int kThreads = kQuantWarps * 32;

// A weight enters the product as 2^(z - m' + 11) (mantissa of its step), z = score + exponent
// of the step, m' the largest z so far or at most 2^3 behind it: at most 2^15, and what fp16
// loses below its normal range is 2^-36 of the largest.
constexpr float kShift = 11.f, kLag = 3.f;

__device__ __forceinline__ void qd_set_err(int *err, int code, int a, int b, int c) {
  if (atomicCAS(err, 0, code) == 0) {
    err[1] = a;
    err[2] = b;
    err[3] = c;
  }
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_rz(float a, float b) {
  uint32_t r;
  asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ float pow2(int e) {  // -126 <= e <= 127
  return __uint_as_float((uint32_t)(e + 127) << 23);
}
// exponent of x >= 0: floor(log2 x), -127 for 0 and fp32's subnormal numbers
__device__ __forceinline__ int exponent(float x) { return (int)(__float_as_uint(x) >> 23) - 127; }

template <int D, int BITS, int G>
struct Shape {
  using Q = QuantTile<D, BITS>;
  static constexpr int kSlot = (G * D * 4 + G * 8 + 15) / 16 * 16;  // bytes of one partial
  static constexpr int kFirst = kQuantWarps * kSlot;
  // two CTAs of an SM share its 227 KB; the ring holds the partials at the end, too
  static constexpr int kRoom = 112 * 1024 - 1024 - kFirst;
  static constexpr int kFit = kRoom / (kQuantWarps * Q::kBytes);
  static constexpr int kStages = kFit < 2 ? 2 : kFit > 6 ? 6 : kFit;
  static constexpr int kRing = kQuantWarps * kStages * Q::kBytes;
  static constexpr int kLast = kQuantWarps * kSlot;
  static constexpr int kJoin = kQuantCtas * G * 4;  // weights of a unit's partials
  static constexpr int kRingOrJoin = kRing > kLast + kJoin ? kRing : kLast + kJoin;
  static constexpr int kBars = kQuantWarps * kStages * 8;
  static constexpr int kSmem = kRingOrJoin + kFirst + kBars;
};

// Where a warp is in the row of tiles.
struct Cursor {
  int at, end;            // places
  int i, h;               // sequence, kv head
  int tile, tiles;        // of the unit
  int left;               // tiles of the unit in this warp's stretch from here on

  // To the next place that holds a tile, from `at`; left = 0: none.
  __device__ __forceinline__ void seek(const QuantAttendParams &p) {
    left = 0;
    while (at < end) {
      while (i + 1 < p.n && p.seqs[i + 1].off <= at) ++i;
      const QuantAttendSeq &s = p.seqs[i];
      const int r = at - s.off;
      h = r / s.stride;
      if (h >= p.hkv) {  // (behind the last unit)
        at = end;
        return;
      }
      tile = r - h * s.stride;
      tiles = s.tiles;
      if (tile < tiles) {
        left = min(tiles - tile, end - at);
        return;
      }
      at += s.stride - tile;
    }
  }
  __device__ __forceinline__ void start(const QuantAttendParams &p, int from, int to) {
    at = from;
    end = to;
    int lo = 0, hi = p.n;
    i = 0;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (p.seqs[mid].off <= at) i = mid, lo = mid + 1;
      else hi = mid;
    }
    seek(p);
  }
  __device__ __forceinline__ void step(const QuantAttendParams &p) {
    ++at;
    ++tile;
    if (--left == 0) seek(p);
  }
};

template <typename T, int D, int BITS, int G, bool SPLIT>
struct Warp {
  using Q = QuantTile<D, BITS>;
  static constexpr int KS = D / 16;     // k-steps of S, m-tiles of O
  static constexpr int NG = Q::kGroups;
  static constexpr bool kTwo = SPLIT && G == 8;   // low halves need products of their own
  static constexpr bool kLanes = SPLIT && G < 8;  // low halves in the columns 4 .. 7

  uint32_t qb[KS][2];  // q as the second operand of S
  float qs[2][NG];     // sums of q over the groups, of the lane's two columns
  float fac[2];        // of the columns: 2^e of q (and 2^24 is applied before)
  float slope[2];
  float m[2], mz[2], l[2];
  float lo[2][NG];     // sum of p lo over the lane's tokens
  float o[KS][4];

  __device__ __forceinline__ void begin(const QuantAttendParams &p, int i, int h, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const T *row = static_cast<const T *>(p.q) + ((size_t)i * p.hkv * G + h * G + g % G) * D;
    float x[KS][4];
    float top = 0.f;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const uint2 v = *reinterpret_cast<const uint2 *>(row + 32 * (s >> 1) + 8 * t + 4 * (s & 1));
      const float2 a = unpack2<T>(v.x), b = unpack2<T>(v.y);
      x[s][0] = a.x, x[s][1] = a.y, x[s][2] = b.x, x[s][3] = b.y;
      top = fmaxf(top, fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(b.x), fabsf(b.y))));
    }
    top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
    top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
    // q in [2^14, 2^15) at its largest: fp16 keeps all of its bits down to 2^-28 of that
    const int e = max(exponent(top) - 14, -100);
    const float down = pow2(-e);
    float sum[NG];
#pragma unroll
    for (int a = 0; a < NG; ++a) sum[a] = 0.f;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        x[s][c] *= down;
        sum[s * NG / KS] += x[s][c];
      }
      // (codes of 4 bits: channels 2 and 3 come from high nibbles, 16 times as large)
      const float hi = BITS == 4 ? 0.0625f : 1.f;
      qb[s][0] = pack2<__half>(x[s][0], x[s][1]);
      qb[s][1] = pack2<__half>(x[s][2] * hi, x[s][3] * hi);
    }
    const float sl = p.rule.slopes ? p.rule.slopes[h * G + g % G] * 1.4426950408889634f : 0.f;
    const float up = pow2(e);
#pragma unroll
    for (int a = 0; a < NG; ++a) {
      sum[a] += __shfl_xor_sync(kFull, sum[a], 1);
      sum[a] += __shfl_xor_sync(kFull, sum[a], 2);
      sum[a] *= 0x1p-24f;
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int from = 4 * (2 * t + c);  // a lane of the column
      fac[c] = __shfl_sync(kFull, up, from);
      slope[c] = __shfl_sync(kFull, sl, from);
#pragma unroll
      for (int a = 0; a < NG; ++a) qs[c][a] = __shfl_sync(kFull, sum[a], from);
      m[c] = mz[c] = -CUDART_INF_F;
      l[c] = 0.f;
#pragma unroll
      for (int a = 0; a < NG; ++a) lo[c][a] = 0.f;
    }
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[s][k] = 0.f;
  }

  // The parameters of token r: lo and step of every group.
  static __device__ __forceinline__ void params(const char *half, int r, float (&lo)[NG],
                                                float (&st)[NG]) {
    const char *q = half + Q::kCodes + r * Q::kTokenParams;
    if constexpr (NG == 1) {
      const float2 e = unpack2<T>(*reinterpret_cast<const uint32_t *>(q));
      lo[0] = e.x, st[0] = e.y;
    } else if constexpr (NG == 2) {
      const uint2 v = *reinterpret_cast<const uint2 *>(q);
      const float2 a = unpack2<T>(v.x), b = unpack2<T>(v.y);
      lo[0] = a.x, lo[1] = a.y, st[0] = b.x, st[1] = b.y;
    } else {
      const uint4 v = *reinterpret_cast<const uint4 *>(q);
      const float2 a = unpack2<T>(v.x), b = unpack2<T>(v.y), c = unpack2<T>(v.z), d = unpack2<T>(v.w);
      lo[0] = a.x, lo[1] = a.y, lo[2] = b.x, lo[3] = b.y;
      st[0] = c.x, st[1] = c.y, st[2] = d.x, st[3] = d.y;
    }
  }

  // Operand registers of a k-step (K) or an m-tile (V) from its codes.
  static __device__ __forceinline__ void widen(const uint32_t *w, bool is_v, uint32_t (&a)[4]) {
    if constexpr (BITS == 4) {
      const uint32_t x = w[0], y = w[0] >> 8;
      // K: low nibbles k, high ones k + 8; V: low ones row g, high ones row g + 8
      a[0] = x & 0x000f000fu;
      a[is_v ? 1 : 2] = x & 0x00f000f0u;
      a[is_v ? 2 : 1] = y & 0x000f000fu;
      a[3] = y & 0x00f000f0u;
    } else {
      a[0] = w[0] & 0x00ff00ffu;
      a[1] = (w[0] >> 8) & 0x00ff00ffu;
      a[2] = w[1] & 0x00ff00ffu;
      a[3] = (w[1] >> 8) & 0x00ff00ffu;
    }
  }

  static __device__ __forceinline__ void product(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                                 uint32_t b1) {
    mma_16816<false>(d, a, b0, b1);
  }

  // One tile: tokens t0 .. t0 + 15, those in [first, L) attended.
  __device__ __forceinline__ void tile(const QuantAttendParams &p, const char *buf, int t0,
                                       int first, int L, int lane) {
    const int g = lane >> 2, t = lane & 3;
    float acc[NG][4];
#pragma unroll
    for (int a = 0; a < NG; ++a)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[a][k] = 0.f;
    constexpr int W = BITS / 4;  // words of a step
#pragma unroll
    for (int c = 0; c < Q::kWords / 4; ++c) {
      const uint4 v = reinterpret_cast<const uint4 *>(buf)[c * 32 + lane];
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4 / W; ++k) {
        const int s = c * (4 / W) + k;
        uint32_t a[4];
        widen(w + k * W, false, a);
        product(acc[s * NG / KS], a, qb[s][0], qb[s][1]);
      }
    }
    const bool edge = t0 < first || t0 + kQuantTile > L;
    float x[4];  // (token g, columns 2t, 2t + 1), (token g + 8, ...)
    {
      float kl[2][NG], ks[2][NG];
      params(buf, g, kl[0], ks[0]);
      params(buf, g + 8, kl[1], ks[1]);
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float s = 0.f;
#pragma unroll
          for (int a = 0; a < NG; ++a) {
            s = fmaf(kl[r][a], qs[c][a], s);
            s = fmaf(ks[r][a], acc[a][2 * r + c], s);
          }
          x[2 * r + c] = s * 0x1p24f * fac[c];
        }
    }
    if (p.rule.cap_out == 0.f) {
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] *= p.rule.scale_log2;
    } else if (p.precise_cap) {
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = cap_any(p.rule, x[k]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; k += 2) {
        const float2 y = cap_16bit(p.rule, make_float2(x[k], x[k + 1]));
        x[k] = y.x, x[k + 1] = y.y;
      }
    }
    if (p.rule.slopes) {
      const float far = (float)(L - 1 - t0 - g);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = fmaf(-slope[k & 1], far - (k >> 1) * 8.f, x[k]);
    }
    float vl[2][NG], vs[2][NG];
    params(buf + Q::kHalf, g, vl[0], vs[0]);
    params(buf + Q::kHalf, g + 8, vl[1], vs[1]);
    if (edge) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int at = t0 + g + 8 * r;
        if (at >= first && at < L) continue;
        x[2 * r] = x[2 * r + 1] = -CUDART_INF_F;
#pragma unroll
        for (int a = 0; a < NG; ++a) vl[r][a] = vs[r][a] = 0.f;  // (what lies there may be anything)
      }
    }
    float z[4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float top = vs[r][0];
#pragma unroll
      for (int a = 1; a < NG; ++a) top = fmaxf(top, vs[r][a]);
      const int e = exponent(top);
      const float down = pow2(-e);  // (e <= 125: a step is at most 2^128 / 15)
#pragma unroll
      for (int a = 0; a < NG; ++a) vs[r][a] *= down;
      z[2 * r] = x[2 * r] + (float)e;
      z[2 * r + 1] = x[2 * r + 1] + (float)e;
    }
    // A new reference only where a weight would leave its room: a vote in most tiles.
    bool up = false;
#pragma unroll
    for (int k = 0; k < 4; ++k) up = up || z[k] > mz[k & 1] + kLag || x[k] > m[k & 1] + 60.f;
    if (__any_sync(kFull, up)) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float a = fmaxf(m[c], fmaxf(x[c], x[2 + c])), b = fmaxf(mz[c], fmaxf(z[c], z[2 + c]));
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) {
          a = fmaxf(a, __shfl_xor_sync(kFull, a, k));
          b = fmaxf(b, __shfl_xor_sync(kFull, b, k));
        }
        const float fa = a == m[c] ? 1.f : ex2_approx(m[c] - a);
        const float fb = b == mz[c] ? 1.f : ex2_approx(mz[c] - b);
        m[c] = a;
        mz[c] = b;
        l[c] *= fa;
#pragma unroll
        for (int k = 0; k < NG; ++k) lo[c][k] *= fa;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          o[s][c] *= fb;
          o[s][2 + c] *= fb;
        }
      }
    }
    float w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float pr = ex2_approx(x[k] - m[k & 1]);
      w[k] = ex2_approx(z[k] - (mz[k & 1] - kShift));
      l[k & 1] += pr;
#pragma unroll
      for (int a = 0; a < NG; ++a) lo[k & 1][a] = fmaf(pr, vl[k >> 1][a], lo[k & 1][a]);
    }
    uint32_t b[NG][2], b2[NG][2];
#pragma unroll
    for (int a = 0; a < NG; ++a)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float y0 = w[2 * r] * vs[r][a], y1 = w[2 * r + 1] * vs[r][a];
        if constexpr (SPLIT) {
          // high part: the first 11 bits; low part: the next 11
          const float h0 = __uint_as_float(__float_as_uint(y0) & 0xffffe000u);
          const float h1 = __uint_as_float(__float_as_uint(y1) & 0xffffe000u);
          if constexpr (kTwo) {
            b[a][r] = transpose8(pack_rz(h0, h1));
            b2[a][r] = transpose8(pack_rz(y0 - h0, y1 - h1));
          } else {
            const float part = t >= 2 ? -1.f : 0.f;
            b[a][r] = transpose8(pack_rz(fmaf(h0, part, y0), fmaf(h1, part, y1)));
          }
        } else {
          b[a][r] = transpose8(pack2<__half>(y0, y1));
        }
      }
#pragma unroll
    for (int c = 0; c < Q::kWords / 4; ++c) {
      const uint4 v = reinterpret_cast<const uint4 *>(buf + Q::kHalf)[c * 32 + lane];
      const uint32_t wd[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4 / W; ++k) {
        const int s = c * (4 / W) + k, a0 = s * NG / KS;
        uint32_t a[4];
        widen(wd + k * W, true, a);
        product(o[s], a, b[a0][0], b[a0][1]);
        if constexpr (kTwo) product(o[s], a, b2[a0][0], b2[a0][1]);
      }
    }
  }

  // The sums of what the warp saw, relative to m: l whole, o with the lowest values' part.
  __device__ __forceinline__ void finish(int lane) {
    (void)lane;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int k = 4; k < 32; k <<= 1) {
        l[c] += __shfl_xor_sync(kFull, l[c], k);
#pragma unroll
        for (int a = 0; a < NG; ++a) lo[c][a] += __shfl_xor_sync(kFull, lo[c][a], k);
      }
      const float f = ex2_approx(mz[c] - m[c]);
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float &y = o[s][2 * r + c];
          if constexpr (kLanes) y += __shfl_xor_sync(kFull, y, 2);
          // 2^24 of the codes (a nibble higher 2^20), 2^-11 of the weights' shift
          y = fmaf(y * (BITS == 4 && r ? 0x1p9f : 0x1p13f), f, lo[c][s * NG / KS]);
        }
    }
  }

  // Column c of the lane's two as rows of channels: calls put(head, channel, float4).
  template <typename F>
  __device__ __forceinline__ void rows(int lane, F put) const {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int head = 2 * t + c;
      if (head >= G) continue;
#pragma unroll
      for (int b = 0; b < D / 32; ++b)
        put(head, c, 32 * b + 4 * g,
            make_float4(o[2 * b][c], o[2 * b][2 + c], o[2 * b + 1][c], o[2 * b + 1][2 + c]));
    }
  }
};

template <typename T>
__device__ __forceinline__ void store_out(void *out, bool f32, size_t at, float4 v) {
  if (f32) {
    *reinterpret_cast<float4 *>(static_cast<float *>(out) + at) = v;
  } else {
    *reinterpret_cast<uint2 *>(static_cast<T *>(out) + at) =
        make_uint2(pack2<T>(v.x, v.y), pack2<T>(v.z, v.w));
  }
}

template <typename T, int D, int BITS, int G, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 2)
    quant_attend_kernel(const __grid_constant__ QuantAttendParams p) {
  using S = Shape<D, BITS, G>;
  using Q = typename S::Q;
  using W = Warp<T, D, BITS, G, SPLIT>;
  extern __shared__ __align__(128) char smem[];
  char *const ring = smem;
  char *const firsts = smem + S::kRingOrJoin;
  uint64_t *const bars = reinterpret_cast<uint64_t *>(firsts + S::kFirst);
  __shared__ int unit_of[2 * kQuantWarps];  // of the warps' first and last partials, or -1
  __shared__ int last_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  char *const mine = ring + warp * S::kStages * Q::kBytes;
  uint64_t *const bar = bars + warp * S::kStages;
  if (lane == 0) {
    for (int k = 0; k < S::kStages; ++k) mbar_init(bar + k, 1);
    fence_mbar_init();
  }
  if (lane < 2) unit_of[2 * warp + lane] = -1;
  __syncwarp();
  pdl_wait();
  pdl_launch_dependents();

  const long long w0 = ((long long)blockIdx.x * kQuantWarps + warp) * p.per_warp;
  const int from = (int)min(w0, (long long)p.total);
  const int to = (int)min(w0 + p.per_warp, (long long)p.total);

  // Copies: lane k holds the physical page of the unit's page `base` + k.
  Cursor in;
  in.start(p, from, to);
  int page_unit = -1, base = 0, phys_lane = 0;
  const int per_page = p.P / kQuantTile;
  int page = 0, in_page = 0;
  auto enter = [&]() {  // the unit's (or the next 32) pages, from `page` on
    const QuantAttendSeq &s = p.seqs[in.i];
    base = page;
    const int blk = page + lane;
    phys_lane = 0;
    if (blk < p.max_pp && blk * (long long)p.P < s.L) {
      phys_lane = p.page_table[(size_t)s.slot * p.max_pp + blk];
      if (phys_lane < 0 || phys_lane >= p.num_phys) {
        qd_set_err(p.err, kDevBadPhys, s.slot, blk, phys_lane);
        phys_lane = 0;  // (read in its place: in the pool)
      }
    }
  };
  int issued = 0;
  auto issue = [&]() {  // the copy of the tile at the cursor, into the next stage
    if (in.left == 0) return;
    const int unit = in.i * p.hkv + in.h;
    if (unit != page_unit) {
      const int first = p.seqs[in.i].first / kQuantTile + in.tile;
      page_unit = unit;
      page = first / per_page;
      in_page = first - page * per_page;
      enter();
    } else if (page - base >= 32) {
      enter();
    }
    const int phys = __shfl_sync(kFull, phys_lane, page - base);
    const int k = issued % S::kStages;
    if (lane == 0) {
      const char *src = static_cast<const char *>(p.pool) +
                        (((size_t)phys * p.hkv + in.h) * per_page + in_page) * Q::kBytes;
      mbar_arrive_expect_tx(bar + k, Q::kBytes);
      bulk_load_1d(mine + k * Q::kBytes, src, Q::kBytes, bar + k);
    }
    ++issued;
    if (++in_page == per_page) in_page = 0, ++page;
    in.step(p);
  };
#pragma unroll 1
  for (int k = 0; k < S::kStages; ++k) issue();

  Cursor at;
  at.start(p, from, to);
  int done = 0;
  bool broken = false;
  W w;
  while (at.left > 0) {
    const int i = at.i, h = at.h, unit = i * p.hkv + h, n = at.left;
    const bool whole = at.tile == 0 && n == at.tiles;
    const int L = p.seqs[i].L, first = p.seqs[i].first;
    int t0 = (first / kQuantTile + at.tile) * kQuantTile;
    w.begin(p, i, h, lane);
#pragma unroll 1
    for (int k = 0; k < n; ++k, t0 += kQuantTile) {
      const int st = done % S::kStages;
      if (!broken && !mbar_wait(bar + st, (done / S::kStages) & 1, kWaitPolls)) {
        if (lane == 0) qd_set_err(p.err, kDevTimeout, p.seqs[i].slot, h, t0);
        broken = true;
      }
      broken = __any_sync(kFull, broken);
      if (broken) continue;  // (nothing is read or copied any more, units still end)
      w.tile(p, mine + st * Q::kBytes, t0, first, L, lane);
      ++done;
      __syncwarp();
      issue();
    }
    at.at += n;
    at.tile += n;
    at.left = 0;
    at.seek(p);
    w.finish(lane);
    if (whole) {
      const float inv[2] = {1.f / w.l[0], 1.f / w.l[1]};
      w.rows(lane, [&](int head, int c, int ch, float4 v) {
        const float f = inv[c];
        store_out<T>(p.out, p.out_f32, (((size_t)i * p.hkv + h) * G + head) * D + ch,
                     make_float4(v.x * f, v.y * f, v.z * f, v.w * f));
      });
    } else if (at.left > 0) {  // this warp's first unit, of which it holds the end
      if (lane == 0) unit_of[2 * warp] = unit;
      float *slot = reinterpret_cast<float *>(firsts + warp * S::kSlot);
      w.rows(lane, [&](int head, int c, int ch, float4 v) {
        *reinterpret_cast<float4 *>(slot + head * D + ch) = v;
        if (ch == 0) {
          slot[G * D + 2 * head] = w.m[c];
          slot[G * D + 2 * head + 1] = w.l[c];
        }
      });
    } else {
      if (lane == 0) unit_of[2 * warp + 1] = unit;
    }
  }
  // (after a wait that gave up: the copies still under way end before the ring is used again)
  for (; broken && done < issued; ++done)
    (void)mbar_wait(bar + done % S::kStages, (done / S::kStages) & 1, kWaitPolls);
  __syncthreads();
  if (unit_of[2 * warp + 1] >= 0) {
    float *slot = reinterpret_cast<float *>(ring + warp * S::kSlot);
    w.rows(lane, [&](int head, int c, int ch, float4 v) {
      *reinterpret_cast<float4 *>(slot + head * D + ch) = v;
      if (ch == 0) {
        slot[G * D + 2 * head] = w.m[c];
        slot[G * D + 2 * head + 1] = w.l[c];
      }
    });
  }
  __syncthreads();

  // Slots in order belong to units in order: runs of the same unit are joined.
  auto slot_of = [&](int k) {
    return reinterpret_cast<const float *>((k & 1 ? ring : firsts) + (k >> 1) * S::kSlot);
  };
  float *const join = reinterpret_cast<float *>(ring + S::kLast);
  const int per_cta = p.per_warp * kQuantWarps;
#pragma unroll 1
  for (int k0 = 0; k0 < 2 * kQuantWarps;) {
    const int unit = unit_of[k0];
    int k1 = k0 + 1;
    if (unit < 0) {
      k0 = k1;
      continue;
    }
    while (k1 < 2 * kQuantWarps && (unit_of[k1] == unit || unit_of[k1] < 0)) ++k1;
    const int i = unit / p.hkv, h = unit - i * p.hkv;
    const QuantAttendSeq &s = p.seqs[i];
    const int u0 = s.off + h * s.stride;
    const int c0 = u0 / per_cta, c1 = (u0 + s.tiles - 1) / per_cta;  // the unit's CTAs
    const bool alone = c0 == c1;
    // this CTA's two partials: of a unit that it starts with, of one that it ends with
    auto part = [&](int c) { return 2 * c + (c > c0 || u0 == c * per_cta ? 0 : 1); };
    const int to_slot = part(blockIdx.x);
#pragma unroll 1
    for (int e = threadIdx.x; e < G * D / 4; e += kThreads) {
      const int head = e / (D / 4), ch = 4 * (e - head * (D / 4));
      float m = -CUDART_INF_F, l = 0.f;
      for (int k = k0; k < k1; ++k)
        if (unit_of[k] >= 0) m = fmaxf(m, slot_of(k)[G * D + 2 * head]);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = k0; k < k1; ++k) {
        if (unit_of[k] < 0) continue;
        const float *q = slot_of(k);
        const float f = ex2_approx(q[G * D + 2 * head] - m);
        const float4 y = *reinterpret_cast<const float4 *>(q + head * D + ch);
        l = fmaf(f, q[G * D + 2 * head + 1], l);
        v.x = fmaf(f, y.x, v.x), v.y = fmaf(f, y.y, v.y);
        v.z = fmaf(f, y.z, v.z), v.w = fmaf(f, y.w, v.w);
      }
      if (alone) {
        const float f = 1.f / l;
        store_out<T>(p.out, p.out_f32, ((size_t)unit * G + head) * D + ch,
                     make_float4(v.x * f, v.y * f, v.z * f, v.w * f));
      } else {
        *reinterpret_cast<float4 *>(p.part_o + ((size_t)to_slot * G + head) * D + ch) = v;
        if (ch == 0) p.part_ml[(size_t)to_slot * G + head] = make_float2(m, l);
      }
    }
    if (!alone) {
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) {
        const int ticket = atom_add_acq_rel_gpu(p.tickets + unit, 1);
        last_flag = ticket == c1 - c0;
        if (last_flag) p.tickets[unit] = 0;  // (for the next launch)
      }
      __syncthreads();
      if (last_flag) {
        __threadfence();
        const int parts = c1 - c0 + 1;
        if (threadIdx.x < 32 * G) {  // a warp per head: the partials' weights
          const int head = warp;
          float m = -CUDART_INF_F, l = 0.f;
          for (int c = lane; c < parts; c += 32)
            m = fmaxf(m, __ldcg(&p.part_ml[(size_t)part(c0 + c) * G + head]).x);
#pragma unroll
          for (int k = 16; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, k));
          for (int c = lane; c < parts; c += 32) {
            const float2 ml = __ldcg(&p.part_ml[(size_t)part(c0 + c) * G + head]);
            const float f = ex2_approx(ml.x - m);
            join[c * G + head] = f;
            l = fmaf(f, ml.y, l);
          }
#pragma unroll
          for (int k = 16; k > 0; k >>= 1) l += __shfl_xor_sync(kFull, l, k);
          const float inv = 1.f / l;
          for (int c = lane; c < parts; c += 32) join[c * G + head] *= inv;
        }
        __syncthreads();
        for (int e = threadIdx.x; e < G * D; e += kThreads) {
          const int head = e / D, ch = e - head * D;
          float v = 0.f;
#pragma unroll 8
          for (int c = 0; c < parts; ++c)
            v = fmaf(join[c * G + head],
                     __ldcg(p.part_o + ((size_t)part(c0 + c) * G + head) * D + ch), v);
          const size_t to = ((size_t)unit * G + head) * D + ch;
          if (p.out_f32) static_cast<float *>(p.out)[to] = v;
          else static_cast<T *>(p.out)[to] = T(v);
        }
      }
      __syncthreads();  // (last_flag and the weights are used again)
    }
    k0 = k1;
  }
}

template <typename T, int D, int BITS, int G, bool SPLIT>
cudaError_t launch_one(const QuantAttendParams &p, cudaStream_t st) {
  using S = Shape<D, BITS, G>;
  static_assert(S::kSmem <= 113 * 1024, "two CTAs an SM");
  static std::atomic<uint64_t> ready{0};
  const auto kernel = quant_attend_kernel<T, D, BITS, G, SPLIT>;
  const cudaError_t e = allow_smem(kernel, S::kSmem, &ready);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, p.ctas, kThreads, S::kSmem, st, p);
}

template <typename T, int D, int BITS, bool SPLIT>
cudaError_t launch_heads(const QuantAttendParams &p, int G, cudaStream_t st) {
  switch (G) {
    case 1: return launch_one<T, D, BITS, 1, SPLIT>(p, st);
    case 2: return launch_one<T, D, BITS, 2, SPLIT>(p, st);
    case 4: return launch_one<T, D, BITS, 4, SPLIT>(p, st);
    default: return launch_one<T, D, BITS, 8, SPLIT>(p, st);
  }
}

// Outputs in bf16 (steps of 2^-8) do not show weights rounded to fp16's 11 bits; the others
// keep 22.
template <typename T, int D, int BITS>
cudaError_t launch_type(const QuantAttendParams &p, int G, cudaStream_t st) {
  if constexpr (sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value) {
    if (!p.out_f32) return launch_heads<T, D, BITS, false>(p, G, st);
  }
  return launch_heads<T, D, BITS, true>(p, G, st);
}

template <typename T>
cudaError_t launch_shape(const QuantAttendParams &p, int d, int bits, int G, cudaStream_t st) {
  if (d == 64) return bits == 8 ? launch_type<T, 64, 8>(p, G, st) : launch_type<T, 64, 4>(p, G, st);
  return bits == 8 ? launch_type<T, 128, 8>(p, G, st) : launch_type<T, 128, 4>(p, G, st);
}

}  // namespace

cudaError_t launch_quant_attend(const QuantAttendParams &p, int dtype, int d, int bits, int G,
                                cudaStream_t st) {
  const cudaError_t e = dtype == 0 ? launch_shape<__half>(p, d, bits, G, st)
                                   : launch_shape<__nv_bfloat16>(p, d, bits, G, st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace spd
