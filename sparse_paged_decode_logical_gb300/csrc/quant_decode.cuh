// Decode attention over a quantised cache (sm_103a): the kernel of spd_quant_decode_attention
// (instantiated in quant_decode_f16.cu and quant_decode_bf16.cu).
//
// With value = lo + step code for keys and values alike,
//   q . k_t = sum over groups a of  lo_ta (sum of q in a) + step_ta (q . codes in a)
//   sum_t p_t v_t = sum_t p_t lo_ta + sum_t (p_t step_ta) codes_t
// so that the matrix products run over the codes themselves, which an fp16 operand holds
// exactly: an integer of 8 or 4 bits in the low bits of an fp16 number is that integer times
// 2^-24, a subnormal, 2^-20 four bits higher.  A word of codes becomes operands by masks and
// shifts alone: 5 instructions for 8 codes of 4 bits, 3 for 4 of 8.  (tcgen05 has no use here: it
// reads operands from shared or tensor memory, where the widened codes would first have to be
// written.)
//
// The products are transposed, S = K q and O = V p, so that a kv head's 1 to 8 query heads are
// the short side (n = 8) of m16n8k16; scores reach the second product by movmatrix.  Where at
// most four heads share the keys, the columns behind them hold copies: their lanes make the low
// halves of the weights, so that weights in two fp16 parts cost no product more.
//
// Bound by memory, in 4 bits as nearly by instructions: the cache is read once.  131,072 tokens of
// 8 kv heads of 128 channels (32 query heads, bf16) take 49.3 us in 8 bits (83% of the measured
// copy rate) and 40.3 in 4 (62%), with 367 instructions a tile in all; about 6 us of that lie
// behind the loop, in five dependent rounds of joining.  Every warp walks a stretch of tiles
// through its own ring of bulk copies, without a barrier between warps; the launch's warps share
// all sequences' tiles evenly, a warp may end one unit (sequence, kv head) and start the next.
// What a warp holds of a unit that others hold parts of, too, is joined in the CTA, then over CTAs
// by the last one to finish.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include <atomic>
#include <type_traits>

#include "dense_math.cuh"
#include "ptx.cuh"
#include "rotary.cuh"
#include "spd_internal.h"

namespace spd {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr uint32_t kWaitPolls = 1u << 22;
constexpr int kThreads = kQuantWarps * 32;

// A weight enters the product as p 2^k step, p = 2^(score - m): 2^k moves the largest p step of
// a column to between 2^10 and 2^12, and a new k is taken where one would pass 2^15.  What fp16
// loses below its normal range is then 2^-35 of the largest.  k ends at 126, which a column of
// nothing but constant groups (step 0) is given, too: p 2^k beyond fp32's range, and 0 times that,
// take a new reference.  So does a p of 2^kHead (sums of p lo stay in range).
constexpr int kRoom = 11;
constexpr int kHead = 10;
// The reference before any score: finite, so that scores of -inf (a bias beyond fp32's range) are
// weights of 0 where a warp meets nothing else, too.
constexpr float kNoScore = -3.402823466e38f;

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
// D = A B + C in fp16 with fp32 sums; not volatile, so that what belongs to a step's tiles is
// scheduled into one another.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1, float c0, float c1, float c2, float c3) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
      " {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2),
        "f"(c3));
}
__device__ __forceinline__ void add4(float *y, const float (&x)[4]) {
  const float2 a = f2_add(make_float2(y[0], y[1]), make_float2(x[0], x[1]));
  const float2 b = f2_add(make_float2(y[2], y[3]), make_float2(x[2], x[3]));
  y[0] = a.x, y[1] = a.y, y[2] = b.x, y[3] = b.y;
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
  static constexpr int kSlot = quant_slot_bytes(D, G);  // one warp's partial
  static constexpr int kStage = quant_step_tiles(D) * Q::kBytes;
  // the CTAs of an SM share its 227 KB; the ring holds the partials at the end, too
  static constexpr int kMemory = (227 / kQuantPerSm - 2) * 1024;
  static constexpr int kFit = kMemory / (kQuantWarps * kStage);
  static constexpr int kStages = kFit > 4 ? 4 : kFit;
  static constexpr int kLast = kQuantWarps * kSlot;
  static constexpr int kRing = kQuantWarps * kStages * kStage;
  static constexpr int kJoin = kLast + kQuantWarps * 32 * 24;  // and a unit's partials' sums
  static constexpr int kBars = kRing > kJoin ? kRing : kJoin;
  static constexpr int kSmem = kBars + kQuantWarps * kStages * 8;
  static_assert(kStages >= 2 && kSmem <= kMemory + 1024, "the CTAs of an SM share its memory");
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
  __device__ __forceinline__ void advance(const QuantAttendParams &p, int n) {  // n <= left
    at += n;
    tile += n;
    left -= n;
    if (left == 0) seek(p);
  }
};

template <typename T, int D, int BITS, int G, bool FINE>
struct Warp {
  using Q = QuantTile<D, BITS>;
  static constexpr int KS = D / 16;     // k-steps of S, m-tiles of O
  static constexpr int NT = quant_step_tiles(D);
  static constexpr int NG = Q::kGroups;
  // FINE: outputs in fp32, sums to fp32's own error.  Weights have 22 bits whatever the output (with
  // 11, one bf16 output in five was not the rounding of the exact value; 131,072 tokens in 4 bits
  // 38.0 us, 40.0 with 22).
  static constexpr bool kTwo = G == 8;     // low halves need products of their own
  static constexpr bool kLanes = !kTwo;    // low halves in the columns 4 .. 7
  // Codes as fp16 numbers.  For 16-bit outputs: as they lie, a subnormal number, code 2^-24
  // (2^-20 in a high nibble).  The tensor cores cut a product's terms and its sum off, always
  // toward zero, so that sums of codes, never negative, lose in one direction.  V's tokens 8 to 15
  // of a tile therefore enter from their highest value down, hi - step (levels - code): the
  // complement of the codes, which the mask takes along, times a negative weight.  Both signs in
  // every product, a step's sums added to the walk's in fp32 outside: 5e-7 (8 bits) and 2e-6 (4) of
  // the output, from 3,000 tokens to walks of 1,024 tiles a warp.  (Codes of one sign: 1e-5 to 4e-4,
  // and in the accumulator over the whole walk 1e-3 at 64 tiles, 0.2 at 1,024.)  For fp32: ordinary
  // numbers around 0, code - 2^(b-1) (11 instructions a word of 4 bits instead of 5, 5 for 4 codes
  // of 8 bits instead of 3), and K's products over more than two operands are added in fp32 outside:
  // 2e-7 and 4e-7.  (131,072 tokens in 4 bits 51.5 us, 40.3 for 16-bit outputs.)
  static constexpr bool kNibbles = BITS == 4 && !FINE;  // high nibbles 2^4 as large
  static constexpr int kUnit = FINE ? 0 : 24;           // a code of 1 is 2^-kUnit
  static constexpr float kMid = FINE ? (BITS == 4 ? 8.f : 128.f) : 0.f;

  uint32_t qb[KS][2];  // q as the second operand of S
  float qs[2][NG];     // sums of q over the groups, of the lane's two columns
  float fac[2];        // of the columns: from sums to scores
  float slope[2];
  float m[2], l[2];    // reference of the weights, their sum
  float up[2];         // 2^k
  int k2[2];           // k
  float lo[2][NG];     // sum of p lo over the lane's tokens
  float o[KS][4];
  bool vast;           // a query beyond 2^100: its factor comes in two
  bool plain;          // neither vast nor capped nor biased

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
    // q in [2^14, 2^15) at its largest: fp16 keeps all of its bits down to 2^-28 of that (and the
    // products with keys of up to 2^104 stay in fp32's range)
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
      // (channels 2 and 3 come from high nibbles)
      const float hi = kNibbles ? 0.0625f : 1.f;
      qb[s][0] = pack2<__half>(x[s][0], x[s][1]);
      qb[s][1] = pack2<__half>(x[s][2] * hi, x[s][3] * hi);
    }
    const float sl = p.rule.slopes ? p.rule.slopes[h * G + g % G] * 1.4426950408889634f : 0.f;
    vast = __any_sync(kFull, e > 86);
    plain = !vast && p.rule.cap_out == 0.f && !p.rule.slopes;
    const float f = pow2(vast ? e : e + kUnit) * (p.rule.cap_out == 0.f ? p.rule.scale_log2 : 1.f);
#pragma unroll
    for (int a = 0; a < NG; ++a) {
      sum[a] += __shfl_xor_sync(kFull, sum[a], 1);
      sum[a] += __shfl_xor_sync(kFull, sum[a], 2);
      sum[a] *= pow2(-kUnit);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int from = 4 * (2 * t + c);  // a lane of the column
      fac[c] = __shfl_sync(kFull, f, from);
      slope[c] = __shfl_sync(kFull, sl, from);
#pragma unroll
      for (int a = 0; a < NG; ++a) qs[c][a] = __shfl_sync(kFull, sum[a], from);
      m[c] = kNoScore;
      up[c] = 1.f;
      k2[c] = 0;
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
  static __device__ __forceinline__ uint32_t centred(uint32_t x) {  // code in the low bits
    x |= 0x64006400u;                                               // 1024 + code
    const __half2 y = __hsub2(*reinterpret_cast<__half2 *>(&x), __float2half2_rn(1024.f + kMid));
    return *reinterpret_cast<const uint32_t *>(&y);
  }
  static __device__ __forceinline__ void widen(const uint32_t *w, bool is_v, uint32_t (&a)[4]) {
    // 4 bits.  K: low nibbles k, high ones k + 8; V: low ones row g, high ones row g + 8
    const int n1 = is_v ? 1 : 2, n2 = is_v ? 2 : 1;
    const uint32_t flip = is_v && !FINE ? ~0u : 0u;  // of V's tokens 8 and up: levels - code
    if constexpr (kNibbles) {
      const uint32_t x = w[0], y = w[0] >> 8;
      a[0] = x & 0x000f000fu;
      a[n1] = x & 0x00f000f0u;
      a[n2] = (y ^ flip) & 0x000f000fu;
      a[3] = (y ^ flip) & 0x00f000f0u;
    } else if constexpr (BITS == 4) {
      a[0] = centred(w[0] & 0x000f000fu);
      a[n1] = centred((w[0] >> 4) & 0x000f000fu);
      a[n2] = centred((w[0] >> 8) & 0x000f000fu);
      a[3] = centred((w[0] >> 12) & 0x000f000fu);
    } else {
      a[0] = w[0] & 0x00ff00ffu;
      a[1] = (w[0] >> 8) & 0x00ff00ffu;
      a[2] = (w[1] ^ flip) & 0x00ff00ffu;
      a[3] = ((w[1] >> 8) ^ flip) & 0x00ff00ffu;
      if constexpr (FINE) {
#pragma unroll
        for (int k = 0; k < 4; ++k) a[k] = centred(a[k]);
      }
    }
  }

  // The sums that a tile's scores are made of: x = (token g, columns 2t and 2t + 1),
  // (token g + 8, ...).
  __device__ __forceinline__ void sums(const char *buf, int lane, float (&x)[4]) const {
    const int g = lane >> 2;
    constexpr int W = BITS / 4;                                     // words of a step
    constexpr int CH = !FINE ? KS / NG : KS / NG > 2 ? 2 : KS / NG;  // products of one sum
    float acc[KS / CH][4];
#pragma unroll
    for (int c = 0; c < Q::kWords / 4; ++c) {
      const uint4 v = reinterpret_cast<const uint4 *>(buf)[c * 32 + lane];
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4 / W; ++k) {
        const int s = c * (4 / W) + k, n = s / CH;
        uint32_t a[4];
        widen(w + k * W, false, a);
        if (s % CH == 0)
          mma_f16(acc[n], a, qb[s][0], qb[s][1], 0.f, 0.f, 0.f, 0.f);
        else
          mma_f16(acc[n], a, qb[s][0], qb[s][1], acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
      }
    }
    constexpr int PER = KS / CH / NG;  // sums of a group
#pragma unroll
    for (int a = 0; a < NG; ++a)
#pragma unroll
      for (int n = 1; n < PER; ++n)
        add4(acc[a * PER], acc[a * PER + n]);
    float kl[2][NG], ks[2][NG];
    params(buf, g, kl[0], ks[0]);
    params(buf, g + 8, kl[1], ks[1]);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if constexpr (kMid != 0.f) {
#pragma unroll
        for (int a = 0; a < NG; ++a) kl[r][a] = fmaf(kMid, ks[r][a], kl[r][a]);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float s = kl[r][0] * qs[c][0];
#pragma unroll
        for (int a = 1; a < NG; ++a) s = fmaf(kl[r][a], qs[c][a], s);
#pragma unroll
        for (int a = 0; a < NG; ++a) s = fmaf(ks[r][a], acc[a * PER][2 * r + c], s);
        x[2 * r + c] = s * fac[c];
      }
    }
  }

  // Scores in base-2 units from what sums() left, where more than a factor makes them; far: the
  // tile's first token's distance.
  __device__ __forceinline__ void rule(const QuantAttendParams &p, float far, float (&x)[4]) const {
    if (vast) {
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] *= pow2(kUnit);
    }
    if (p.rule.cap_out != 0.f) {
      if (p.precise_cap) {
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = cap_any(p.rule, x[k]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
          const float2 y = cap_16bit(p.rule, make_float2(x[k], x[k + 1]));
          x[k] = y.x, x[k + 1] = y.y;
        }
      }
    }
    if (p.rule.slopes) {
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = fmaf(-slope[k & 1], far - (k >> 1) * 8.f, x[k]);
    }
  }

  // A step: the NT tiles from token t0 on, tokens in [first, end) attended (tiles behind the
  // first may hold none, and then anything).
  __device__ __forceinline__ void step(const QuantAttendParams &p, const char *buf, int t0,
                                       int first, int end, int L, int lane) {
    const int g = lane >> 2, t = lane & 3;
    float x[NT][4], vl[NT][2][NG], vs[NT][2][NG];
#pragma unroll
    for (int j = 0; j < NT; ++j) sums(buf + j * Q::kBytes, lane, x[j]);
    if (!plain) {
#pragma unroll
      for (int j = 0; j < NT; ++j) rule(p, (float)(L - 1 - t0 - g) - 16.f * j, x[j]);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int r = 0; r < 2; ++r)
        params(buf + j * Q::kBytes + Q::kHalf, g + 8 * r, vl[j][r], vs[j][r]);
    if (t0 < first || t0 + NT * kQuantTile > end) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int at = t0 + 16 * j + 8 * r + g;
          if (at >= first && at < end) continue;
          x[j][2 * r] = x[j][2 * r + 1] = -CUDART_INF_F;
#pragma unroll
          for (int a = 0; a < NG; ++a) vl[j][r][a] = vs[j][r][a] = 0.f;
        }
    }
    // p, and the largest it, with the largest step, could make a weight
    float pr[NT][4], most = 0.f, pm[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int k = 0; k < 4; ++k) pr[j][k] = ex2_approx(x[j][k] - m[k & 1]);
#pragma unroll
      for (int c = 0; c < 2; ++c) pm[c] = fmax3f(pm[c], pr[j][c], pr[j][2 + c]);
#pragma unroll
      for (int a = 0; a < NG; ++a) most = fmax3f(most, vs[j][0][a], vs[j][1][a]);
    }
    const float big = fmaxf(pm[0] * up[0], pm[1] * up[1]) * most;
    // A new reference only where a weight could leave its room (or the bound is not a number): a
    // vote in most steps.
    if (__any_sync(kFull, fmaxf(pm[0], pm[1]) > (float)(1 << kHead) || !(big <= 32768.f))) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float a = m[c];
#pragma unroll
        for (int j = 0; j < NT; ++j) a = fmax3f(a, x[j][c], x[j][2 + c]);
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) a = fmaxf(a, __shfl_xor_sync(kFull, a, k));
        // z: the largest p step so far, as a power of 2 (of differences of scores: a vast score
        // itself would round the exponent away)
        float z = (m[c] - a) + (float)(kRoom - k2[c]);
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float top = vs[j][r][0];
#pragma unroll
            for (int n = 1; n < NG; ++n) top = fmaxf(top, vs[j][r][n]);
            z = fmaxf(z, (x[j][2 * r + c] - a) + (float)exponent(top));
          }
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) z = fmaxf(z, __shfl_xor_sync(kFull, z, k));
        const int k = (int)fminf(fmaxf(floorf(-z), -120.f), 126.f - kRoom) + kRoom;
        const bool same = a == m[c];
        const float fa = same ? 1.f : ex2_approx(m[c] - a);
        const float fb = ex2_approx((same ? 0.f : m[c] - a) + (float)(k - k2[c]));
        m[c] = a;
        k2[c] = k;
        up[c] = pow2(k);
        l[c] *= fa;
#pragma unroll
        for (int n = 0; n < NG; ++n) lo[c][n] *= fa;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          o[s][c] *= fb;
          o[s][2 + c] *= fb;
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) pr[j][k] = ex2_approx(x[j][k] - m[k & 1]);
    }
    uint32_t b[NT][NG][2], b2[NT][kTwo ? NG : 1][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int a = 0; a < NG; ++a) {
          if (FINE || r) vl[j][r][a] = fmaf(FINE ? kMid : Q::kLevels, vs[j][r][a], vl[j][r][a]);
#pragma unroll
          for (int c = 0; c < 2; ++c) lo[c][a] = fmaf(pr[j][2 * r + c], vl[j][r][a], lo[c][a]);
        }
      float2 w[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        l[0] += pr[j][2 * r];
        l[1] += pr[j][2 * r + 1];
        const float sign = !FINE && r ? -1.f : 1.f;
        w[r] = f2_mul(make_float2(pr[j][2 * r], pr[j][2 * r + 1]), make_float2(sign * up[0], sign * up[1]));
      }
#pragma unroll
      for (int a = 0; a < NG; ++a)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float2 y = f2_mul(w[r], make_float2(vs[j][r][a], vs[j][r][a]));
          // high part: the first 11 bits; low part: the next 11
          const float2 h = make_float2(__uint_as_float(__float_as_uint(y.x) & 0xffffe000u),
                                       __uint_as_float(__float_as_uint(y.y) & 0xffffe000u));
          if constexpr (kTwo) {
            const float2 z = f2_sub(y, h);
            b[j][a][r] = transpose8(pack_rz(h.x, h.y));
            b2[j][a][r] = transpose8(pack_rz(z.x, z.y));
          } else {
            const float part = t >= 2 ? -1.f : 0.f;
            const float2 z = f2_fma(h, make_float2(part, part), y);
            b[j][a][r] = transpose8(pack_rz(z.x, z.y));
          }
        }
    }
    // O += V weights
    constexpr int W = BITS / 4;
#pragma unroll
    for (int c = 0; c < Q::kWords / 4; ++c) {
      uint32_t wd[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const uint4 v =
            reinterpret_cast<const uint4 *>(buf + j * Q::kBytes + Q::kHalf)[c * 32 + lane];
        wd[j][0] = v.x, wd[j][1] = v.y, wd[j][2] = v.z, wd[j][3] = v.w;
      }
#pragma unroll
      for (int k = 0; k < 4 / W; ++k) {
        const int s = c * (4 / W) + k, n = s * NG / KS;
        // (a step's sums are added to the walk's outside: in the accumulator every tile would be
        // cut off below what the walk has gathered)
        float d[4] = {0.f, 0.f, 0.f, 0.f}, e[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          uint32_t a[4];
          widen(wd[j] + k * W, true, a);
          mma_f16(d, a, b[j][n][0], b[j][n][1], d[0], d[1], d[2], d[3]);
          if constexpr (kTwo) {
            if constexpr (FINE)
              mma_f16(e, a, b2[j][n][0], b2[j][n][1], e[0], e[1], e[2], e[3]);
            else
              mma_f16(d, a, b2[j][n][0], b2[j][n][1], d[0], d[1], d[2], d[3]);
          }
        }
        add4(o[s], d);
        if constexpr (kTwo && FINE) add4(o[s], e);
      }
    }
  }

  // The sums of what the warp saw, relative to m: l whole, o with the lowest values' part.
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int k = 4; k < 32; k <<= 1) {
        l[c] += __shfl_xor_sync(kFull, l[c], k);
#pragma unroll
        for (int a = 0; a < NG; ++a) lo[c][a] += __shfl_xor_sync(kFull, lo[c][a], k);
      }
      const float f = pow2(-k2[c]);  // (|k| <= 126)
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float &y = o[s][2 * r + c];
          if constexpr (kLanes) y += __shfl_xor_sync(kFull, y, 2);
          y = fmaf(y * (kNibbles && r ? 0x1p20f : pow2(kUnit)), f, lo[c][s * NG / KS]);
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

template <typename T, int D, int BITS, int G, bool FINE>
__global__ void __launch_bounds__(kThreads, kQuantPerSm)
    quant_attend_kernel(const __grid_constant__ QuantAttendParams p) {
  using S = Shape<D, BITS, G>;
  using Q = typename S::Q;
  using W = Warp<T, D, BITS, G, FINE>;
  extern __shared__ __align__(128) char smem[];
  char *const ring = smem;
  char *const firsts = p.firsts + (size_t)blockIdx.x * S::kLast;
  uint64_t *const bars = reinterpret_cast<uint64_t *>(smem + S::kBars);
  __shared__ int unit_of[2 * kQuantWarps];  // of the warps' first and last partials, or -1
  __shared__ int last_flag[kQuantWarps];
  __shared__ int4 span_of[2 * kQuantWarps];     // their units' first and last CTA, second slot
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  char *const mine = ring + warp * S::kStages * S::kStage;
  uint64_t *const bar = bars + warp * S::kStages;
  if (lane == 0) {
    for (int k = 0; k < S::kStages; ++k) mbar_init(bar + k, 1);
    fence_mbar_init();
  }
  if (lane < 2) unit_of[2 * warp + lane] = -1;
  const long long w0 = ((long long)blockIdx.x * kQuantWarps + warp) * p.per_warp;
  const int from = (int)min(w0, (long long)p.total);
  const int to = (int)min(w0 + p.per_warp, (long long)p.total);
  Cursor at;
  at.start(p, from, to);
  Cursor in = at;
  __syncwarp();
  pdl_wait();
  pdl_launch_dependents();

  // Copies, a step's tiles into a stage.  Lane k holds the physical page of the unit's page
  // `base` + k.
  const int per_page = p.P / kQuantTile;
  int base = 0, phys_lane = 0, issued = 0;
  int todo = 0, tile_in = 0, head_in = 0;  // of the unit being copied: tiles behind the run, the next one
  int run = 0;                             // tiles that follow one another at src
  const char *src = nullptr;
  const QuantAttendSeq *seq_in = nullptr;
  bool fresh = true;  // the unit's pages are not known yet
  auto locate = [&]() {  // the next run of tiles on one page: src, run
    const int page = tile_in / per_page, in_page = tile_in - page * per_page;
    if (fresh || page - base >= 32) {
      fresh = false;
      base = page;
      const int blk = page + lane;
      phys_lane = 0;
      if (blk < p.max_pp && blk * (long long)p.P < seq_in->L) {
        phys_lane = p.page_table[(size_t)seq_in->slot * p.max_pp + blk];
        if (phys_lane < 0 || phys_lane >= p.num_phys) {
          qd_set_err(p.err, kDevBadPhys, seq_in->slot, blk, phys_lane);
          phys_lane = 0;  // (read in its place: in the pool)
        }
      }
    }
    const int phys = __shfl_sync(kFull, phys_lane, page - base);
    src = static_cast<const char *>(p.pool) +
          (((size_t)phys * p.hkv + head_in) * per_page + in_page) * Q::kBytes;
    run = min(todo, per_page - in_page);
    todo -= run;
    tile_in += run;
  };
  // The stage's next copies: a step's tiles, or what is left of the unit.
  auto issue_slow = [&](int stage) {
    if (run == 0 && todo == 0) {
      if (in.left == 0) return;
      todo = in.left;
      seq_in = p.seqs + in.i;
      head_in = in.h;
      tile_in = seq_in->first / kQuantTile + in.tile;
      fresh = true;
      // (the queries are asked for when the unit begins)
      if (lane < G)
        asm volatile("prefetch.global.L1 [%0];" ::"l"(static_cast<const T *>(p.q) +
                                                      ((size_t)(in.i * p.hkv + in.h) * G + lane) * D));
      in.advance(p, todo);
    }
    char *dst = mine + stage * S::kStage;
    int want = min(W::NT, run + todo);
    if (lane == 0) mbar_arrive_expect_tx(bar + stage, want * Q::kBytes);
#pragma unroll 1
    while (want > 0) {
      if (run == 0) locate();
      const int n = min(want, run);
      if (lane == 0) bulk_load_1d(dst, src, n * Q::kBytes, bar + stage);
      dst += n * Q::kBytes;
      src += n * Q::kBytes;
      run -= n;
      want -= n;
    }
    ++issued;
  };
  auto issue = [&](int stage) {
    if (run < W::NT) {
      issue_slow(stage);
      return;
    }
    if (lane == 0) {
      mbar_arrive_expect_tx(bar + stage, S::kStage);
      bulk_load_1d(mine + stage * S::kStage, src, S::kStage, bar + stage);
    }
    src += S::kStage;
    run -= W::NT;
    ++issued;
  };
#pragma unroll 1
  for (int k = 0; k < S::kStages; ++k) issue_slow(k);

  int done = 0, stage = 0;
  uint32_t parity = 0;
  bool broken = false, begun = false;
  W w;
  while (at.left > 0) {
    const int i = at.i, h = at.h, unit = i * p.hkv + h, n = at.left;
    const bool whole = at.tile == 0 && n == at.tiles;
    const int L = p.seqs[i].L, first = p.seqs[i].first;
    int t0 = (first / kQuantTile + at.tile) * kQuantTile;
    const int end = min(L, t0 + n * kQuantTile);
    if (lane == 0) {  // (while the first copies are under way)
      const int u0 = p.seqs[i].off + h * p.seqs[i].stride, per_cta = p.per_warp * kQuantWarps;
      const int c0 = u0 / per_cta;
      const int4 span = make_int4(c0, (u0 + at.tiles - 1) / per_cta, u0 != c0 * per_cta, 0);
      if (!begun) span_of[2 * warp] = span;  // (not by steps done: a wait that gave up leaves none)
      span_of[2 * warp + 1] = span;
    }
    begun = true;
    w.begin(p, i, h, lane);
#pragma unroll 1
    for (; t0 < end; t0 += W::NT * kQuantTile) {
      if (!__all_sync(kFull, mbar_try_wait(bar + stage, parity))) {
        bool there = false;
        for (uint32_t k = 0; k < kWaitPolls && !there && !broken; ++k)
          there = __all_sync(kFull, mbar_try_wait(bar + stage, parity));
        if (!there) {
          if (!broken && lane == 0) qd_set_err(p.err, kDevTimeout, p.seqs[i].slot, h, t0);
          broken = true;
          break;  // (nothing is read or copied any more, units still end)
        }
      }
      w.step(p, mine + stage * S::kStage, t0, first, end, L, lane);
      ++done;
      __syncwarp();
      issue(stage);
      if (++stage == S::kStages) stage = 0, parity ^= 1;
    }
    at.advance(p, n);
    w.finish();
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

  // Partials of the same unit are joined: by the whole CTA where all are of one, else side by
  // side by four warps or one each.  (Unit after unit by the CTA, 1,024 units of 1,024 tokens
  // took 52 us, 44 side by side.)
  constexpr int kSlots = 2 * kQuantWarps, kVectors = G * D / 4;
  static_assert(kSlots <= 32, "a lane per slot");
  static_assert(kThreads % 128 == 0, "teams of four warps: a barrier that 128 threads come to");
  const int slot_unit = lane < kSlots ? unit_of[lane] : -1;
  const unsigned taken = __ballot_sync(kFull, slot_unit >= 0);
  const unsigned before = taken & ((1u << lane) - 1u);
  const int last_unit = __shfl_sync(kFull, slot_unit, before ? 31 - __clz(before) : 0);
  // (a unit's slots follow one another: its first one stands for it)
  unsigned units = __ballot_sync(kFull, slot_unit >= 0 && (!before || last_unit != slot_unit));
  const int found = __popc(units);
  const int width = found == 1 ? kThreads : found <= kThreads / 128 ? 128 : 32;
  // (selected, not divided: that would take longer than the ballots)
  const bool fours = width == 128, single = width == 32;
  const int teams = single ? kQuantWarps : fours ? kThreads / 128 : 1;
  const int team = single ? warp : fours ? warp >> 2 : 0;
  const int tid = threadIdx.x - team * width;
  auto sync = [&]() {
    if (single) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(fours ? 1 + team : 0), "r"(width) : "memory");
  };
  const int sets = single ? (32 > kVectors ? 32 / kVectors : 1)
                   : fours ? (128 > kVectors ? 128 / kVectors : 1)
                           : (kThreads > kVectors ? kThreads / kVectors : 1);
  float4 *const sums = reinterpret_cast<float4 *>(ring + S::kLast) + team * width;
  float2 *const stats = reinterpret_cast<float2 *>(ring + S::kLast + kThreads * 16) + team * width;
  for (int k = 0; k < team; ++k) units &= units - 1;  // from this team's first unit on
#pragma unroll 1
  while (units) {
    const int slot0 = __ffs(units) - 1, unit = __shfl_sync(kFull, slot_unit, slot0);
    const unsigned members = __ballot_sync(kFull, slot_unit == unit);
    for (int k = 0; k < teams; ++k) units &= units - 1;
    const int c0 = span_of[slot0].x, c1 = span_of[slot0].y;  // the unit's CTAs
    const bool alone = c0 == c1;
    // this CTA's two partials: of a unit that it starts with, of one that it ends with
    const int second = span_of[slot0].z;  // (the unit begins inside its first CTA)
    char *const own = p.parts + (size_t)(2 * blockIdx.x + (blockIdx.x == c0 ? second : 0)) * S::kSlot;
    // The sources: last partials of neighbouring warps, then perhaps a first one; and once more
    // for the last CTA of the unit to come, every CTA's partial (in their order, whichever came
    // last).
    const unsigned odd = members & 0xaaaaaaaau, even = members & 0x55555555u;
    const char *base = ring + (odd ? (__ffs(odd) - 1) >> 1 : 0) * S::kSlot;
    int stride = S::kSlot, total = __popc(members), special = even ? total - 1 : -1;
    const char *there = firsts + (even ? (__ffs(even) - 1) >> 1 : 0) * S::kSlot;
    bool ends = alone;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
      // Threads in sets, each with every sets-th source, eight loads under way.
#pragma unroll 1
      for (int x = tid; x < sets * kVectors; x += width) {
        const int set = x / kVectors, e = x % kVectors, head = e / (D / 4);
        float m = -CUDART_INF_F, l = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int c = set; c < total; c += 8 * sets) {
          float2 ml[8];
          float4 y[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int at = c + k * sets;
            ml[k] = make_float2(-CUDART_INF_F, 0.f);
            y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (at < total) {
              const char *from = at == special ? there : base + (size_t)at * stride;
              ml[k] = reinterpret_cast<const float2 *>(from + G * D * 4)[head];
              y[k] = reinterpret_cast<const float4 *>(from)[e];
            }
          }
          float top = m;
#pragma unroll
          for (int k = 0; k < 8; ++k) top = fmaxf(top, ml[k].x);
          const float f0 = m == top ? 1.f : ex2_approx(m - top);
          m = top;
          l *= f0;
          v.x *= f0, v.y *= f0, v.z *= f0, v.w *= f0;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (c + k * sets >= total) continue;
            const float f = ex2_approx(ml[k].x - m);
            l = fmaf(f, ml[k].y, l);
            v.x = fmaf(f, y[k].x, v.x), v.y = fmaf(f, y[k].y, v.y);
            v.z = fmaf(f, y[k].z, v.z), v.w = fmaf(f, y[k].w, v.w);
          }
        }
        if (sets > 1) {
          sums[x] = v;
          stats[x] = make_float2(m, l);
          sync();
          if (set > 0) continue;
          for (int k = 1; k < sets && k < total; ++k) {
            const float2 ml = stats[k * kVectors + e];
            const float4 y = sums[k * kVectors + e];
            const float top = fmaxf(m, ml.x);
            const float f0 = m == top ? 1.f : ex2_approx(m - top), f = ex2_approx(ml.x - top);
            m = top;
            l = fmaf(f, ml.y, l * f0);
            v.x = fmaf(f, y.x, v.x * f0), v.y = fmaf(f, y.y, v.y * f0);
            v.z = fmaf(f, y.z, v.z * f0), v.w = fmaf(f, y.w, v.w * f0);
          }
        }
        if (ends) {
          const float f = 1.f / l;
          store_out<T>(p.out, p.out_f32, (size_t)unit * G * D + 4 * e,
                       make_float4(v.x * f, v.y * f, v.z * f, v.w * f));
        } else {
          reinterpret_cast<float4 *>(own)[e] = v;
          if (e % (D / 4) == 0) reinterpret_cast<float2 *>(own + G * D * 4)[head] = make_float2(m, l);
        }
      }
      if (ends) break;
      // (the barrier and the ticket's release publish this CTA's partial, its acquire and the
      // barrier behind show the others')
      sync();
      if (tid == 0) {
        const int last = atom_add_acq_rel_gpu(p.tickets + unit, 1) == c1 - c0;
        if (last) p.tickets[unit] = 0;  // (for the next launch)
        last_flag[team] = last;
      }
      sync();
      if (!last_flag[team]) break;
      ends = true;
      base = p.parts + (size_t)2 * c0 * S::kSlot;
      stride = 2 * S::kSlot;
      special = second ? 0 : -1;
      there = base + S::kSlot;
      total = c1 - c0 + 1;
    }
    sync();  // (the flag and the sums are used again)
  }
}

template <typename T, int D, int BITS, int G, bool FINE>
cudaError_t launch_one(const QuantAttendParams &p, cudaStream_t st) {
  using S = Shape<D, BITS, G>;
    static std::atomic<uint64_t> ready{0};
  const auto kernel = quant_attend_kernel<T, D, BITS, G, FINE>;
  const cudaError_t e = allow_smem(kernel, S::kSmem, &ready);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, p.ctas, kThreads, S::kSmem, st, p);
}

template <typename T, int D, int BITS, bool FINE>
cudaError_t launch_heads(const QuantAttendParams &p, int G, cudaStream_t st) {
  switch (G) {
    case 1: return launch_one<T, D, BITS, 1, FINE>(p, st);
    case 2: return launch_one<T, D, BITS, 2, FINE>(p, st);
    case 4: return launch_one<T, D, BITS, 4, FINE>(p, st);
    default: return launch_one<T, D, BITS, 8, FINE>(p, st);
  }
}

template <typename T, bool FINE>
cudaError_t launch_shape(const QuantAttendParams &p, int d, int bits, int G, cudaStream_t st) {
  if (d == 64)
    return bits == 8 ? launch_heads<T, 64, 8, FINE>(p, G, st) : launch_heads<T, 64, 4, FINE>(p, G, st);
  return bits == 8 ? launch_heads<T, 128, 8, FINE>(p, G, st) : launch_heads<T, 128, 4, FINE>(p, G, st);
}

}  // namespace
}  // namespace spd
