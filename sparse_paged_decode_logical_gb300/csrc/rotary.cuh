// Rotating rows of channels by positions, shared by the rotary kernel and the
// kernel that rotates keys on their way into a quantised cache.
//
// A pair (x, y) of channels becomes (x cos a - y sin a, x sin a + y cos a) with
// a = position * frequency.  Frequencies come as turns in units of 2^-64, so that
// position * frequency mod 2^64 is the angle's fraction of a turn: one integer product,
// exact whatever the position (an fp32 product is off by 0.06 at position 10^6), and the
// one sine and cosine of a (token, pair) serve all heads.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "quant.h"

namespace spd {

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t x);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t x) {
  return __half22float2(*reinterpret_cast<__half2 *>(&x));
}
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t x) {
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// (cos, sin) of one position and pair.  The angle is rounded to 24 bits of a half turn.
__device__ __forceinline__ float2 turn_of(int position, unsigned long long turns) {
  const unsigned long long phase = (unsigned long long)(long long)position * turns;
  const float half_turns = (float)(int)(phase >> 32) * 0x1p-31f;  // [-1, 1]
  float2 cs;
  sincospif(half_turns, &cs.y, &cs.x);
  return cs;
}

// A row falls into units of work of 8 or 16 channels: with halves rot / 16 units of 8 pairs
// (channels c and c + rot / 2), with neighbours rot / 8 of 4 pairs; then (d - rot) / 8 of
// channels that stay.
struct RotaryShape {
  int d, rot, neighbours;
  __device__ __forceinline__ int turned() const { return neighbours ? rot >> 3 : rot >> 4; }
  __device__ __forceinline__ int units() const { return turned() + ((d - rot) >> 3); }
};

// Where a pair's sines lie: what neighbouring units read together lies together.
__device__ __forceinline__ int sine_place(const RotaryShape &s, int pair) {
  const int n = s.turned();
  return s.neighbours ? (pair & 3) * n + (pair >> 2)
                      : 2 * (((pair & 7) >> 1) * n + (pair >> 3)) + (pair & 1);
}

template <typename T>
struct RotaryUnit {
  uint4 a, b;
  int c0, c1;  // channels; c1 < 0: one vector only

  __device__ __forceinline__ void load(const RotaryShape &s, const T *row, int u) {
    const int n = s.turned();
    c1 = -1;
    if (u >= n) {
      c0 = s.rot + 8 * (u - n);
    } else {
      c0 = 8 * u;
      if (!s.neighbours) c1 = c0 + (s.rot >> 1);
    }
    a = *reinterpret_cast<const uint4 *>(row + c0);
    if (c1 >= 0) b = *reinterpret_cast<const uint4 *>(row + c1);
  }
  // cs: the token's (cos, sin) of every pair, in the order of sine_place
  __device__ __forceinline__ void turn(const RotaryShape &s, const float2 *cs) {
    const int n = s.turned();
    if (c1 >= 0) {
      uint32_t *x = &a.x, *y = &b.x;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 e = reinterpret_cast<const float4 *>(cs)[i * n + (c0 >> 3)];  // two pairs
        const float2 p = unpack2<T>(x[i]), q = unpack2<T>(y[i]);
        x[i] = pack2<T>(p.x * e.x - q.x * e.y, p.y * e.z - q.y * e.w);
        y[i] = pack2<T>(q.x * e.x + p.x * e.y, q.y * e.z + p.y * e.w);
      }
    } else if (c0 < s.rot) {  // neighbours
      uint32_t *x = &a.x;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 e = cs[i * n + (c0 >> 3)], p = unpack2<T>(x[i]);
        x[i] = pack2<T>(p.x * e.x - p.y * e.y, p.y * e.x + p.x * e.y);
      }
    }
  }
  __device__ __forceinline__ void store(T *row) const {
    *reinterpret_cast<uint4 *>(row + c0) = a;
    if (c1 >= 0) *reinterpret_cast<uint4 *>(row + c1) = b;
  }
};

// Between the sines of two tokens (their 16-byte pieces begin at other banks).
__device__ __host__ constexpr int sine_stride(int rot) { return (rot >> 1) + 2; }

// The sines of n tokens' pairs, by a CTA's threads.  Neighbouring threads take the same pair of
// different tokens: the table lies in constant memory, which serves one address at a time (by
// pairs first, this took longer than the rows: 18 us of a 16,385-token append).
template <int THREADS, typename Position>
__device__ __forceinline__ void make_sines(const spd_rotary_table &table, int n, int inverse,
                                           float2 *cs, Position position) {
  const RotaryShape s{table.head_dim, table.rotary_dim, table.neighbours};
  const int pairs = s.rot >> 1;
  for (int e = threadIdx.x; e < n * pairs; e += THREADS) {
    const int j = e / n, t = e - j * n;
    float2 x = turn_of(position(table.axis[j], t), table.turns[j]);
    if (inverse) x.y = -x.y;
    cs[t * sine_stride(s.rot) + sine_place(s, j)] = x;
  }
}

}  // namespace spd
