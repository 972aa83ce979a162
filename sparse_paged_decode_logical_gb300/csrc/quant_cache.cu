// Writing keys and values into a quantised cache and reading them back (sm_103a).
//
// A group of channels of a token is held as value = lo + step * code: lo its lowest value,
// step the least number of the cache's type with levels * step >= highest - lowest, codes
// rounded to nearest, 0 .. levels.  A group that holds a value that is not finite (or whose
// span exceeds fp32) gets lo = NaN and step 0: it reads back as NaN throughout.
//
// Both directions are bound by memory: 2 bytes a value on one side, 1.03 or 0.63 on the other.
// One warp takes a whole tile of 16 tokens of K or of V of a head; its lanes read the
// channels whose codes fill the words that they store (layout in quant.h), so that a group's
// extremes are a few shuffles away and nothing passes through shared memory, except keys that
// are rotated first.  Tiles that are not filled at once go token by token, byte stores.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "ptx.cuh"
#include "rotary.cuh"
#include "spd_internal.h"

namespace spd {
namespace {

constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ void qc_set_err(int *err, int code, int a, int b, int c) {
  if (atomicCAS(err, 0, code) == 0) {
    err[1] = a;
    err[2] = b;
    err[3] = c;
  }
}

// min and max that keep NaN, of packed pairs
template <typename T>
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b);
template <>
__device__ __forceinline__ uint32_t min2_nan<__half>(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <>
__device__ __forceinline__ uint32_t min2_nan<__nv_bfloat16>(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Extremes as (lowest, -highest) in one register: joined by one packed minimum.
template <typename T, int N>
__device__ __forceinline__ uint32_t extremes(const uint32_t (&x)[N]) {
  uint32_t lo = x[0], hi = x[0] ^ 0x80008000u;
#pragma unroll
  for (int i = 1; i < N; ++i) {
    lo = min2_nan<T>(lo, x[i]);
    hi = min2_nan<T>(hi, x[i] ^ 0x80008000u);
  }
  return min2_nan<T>(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
}
template <typename T>
__device__ __forceinline__ uint32_t join(uint32_t e, int lane_mask) {
  return min2_nan<T>(e, __shfl_xor_sync(kFull, e, lane_mask));
}

// What a group's codes are made with.
template <typename T, int LEVELS>
struct Scale {
  uint32_t bits;  // lo, step: as stored
  float lo, step, inv;

  __device__ __forceinline__ explicit Scale(uint32_t e) {  // (lowest, -highest)
    const float2 x = unpack2<T>(e);
    const float span = -x.y - x.x;
    lo = x.x;
    if (!(span <= 3.402823466e38f)) {
      bits = 0x7fffu;  // NaN in either type, step 0
      lo = __uint_as_float(0x7fffffffu);
      step = inv = 0.f;
      return;
    }
    uint32_t h = pack2<T>(__fdiv_rn(span, (float)LEVELS), 0.f) & 0xffffu;
    step = unpack2<T>(h).x;
    if (step * (float)LEVELS < span) {  // (the product is exact: 11 + 8 bits)
      ++h;
      step = unpack2<T>(h).x;
    }
    bits = (e & 0xffffu) | h << 16;
    inv = step > 0.f ? __fdiv_rn(1.f, step) : 0.f;
  }
  // round((x - lo) / step).  The product with 1 / step is off by at most 3 2^-24 of a
  // quotient of at most 255; what lies within 1e-3 of the middle between two codes is
  // divided.  (bf16 steps below 2^-126 have no finite fp32 reciprocal: divided, too.)
  __device__ __forceinline__ uint32_t code(float x) const {
    const float d = x - lo, t = d * inv;
    float n = rintf(t);
    if (!(fabsf(t - n) < 0.499f) && step > 0.f) n = rintf(__fdiv_rn(d, step));
    return (uint32_t)__float2int_rn(n) & (uint32_t)LEVELS;
  }
};

// ---- whole tiles -------------------------------------------------------------------
// x[token][grp][..]: the lane's channels (quant.h) of its tokens.
template <typename T, int D, int BITS>
__device__ __forceinline__ void put_k(char *half, int lane, const uint4 (&x)[2][D / 32]) {
  using Q = QuantTile<D, BITS>;
  const int g = lane >> 2, t = lane & 3;
  uint32_t w[Q::kWords];
  uint32_t e[2][D / 32];
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int a = 0; a < D / 32; ++a) {
      const uint32_t v[4] = {x[r][a].x, x[r][a].y, x[r][a].z, x[r][a].w};
      e[r][a] = extremes<T>(v);
    }
#pragma unroll
  for (int i = 0; i < Q::kWords; ++i) w[i] = 0;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    if constexpr (BITS == 8) {
#pragma unroll
      for (int a = 1; a < D / 32; ++a) e[r][0] = min2_nan<T>(e[r][0], e[r][a]);
    }
    uint16_t *par = reinterpret_cast<uint16_t *>(half + Q::kCodes + (g + 8 * r) * Q::kTokenParams);
#pragma unroll
    for (int a = 0; a < Q::kGroups; ++a) {
      const Scale<T, Q::kLevels> s(join<T>(join<T>(e[r][a], 1), 2));
      if (t == 0) {
        par[a] = (uint16_t)s.bits;
        par[Q::kGroups + a] = (uint16_t)(s.bits >> 16);
      }
#pragma unroll
      for (int b = a * Q::kGroup / 32; b < (a + 1) * Q::kGroup / 32; ++b) {
        const uint32_t v[4] = {x[r][b].x, x[r][b].y, x[r][b].z, x[r][b].w};
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // k-step 2b + i: four channels
          const float2 p = unpack2<T>(v[2 * i]), q = unpack2<T>(v[2 * i + 1]);
          const uint32_t c0 = s.code(p.x), c1 = s.code(p.y), c2 = s.code(q.x), c3 = s.code(q.y);
          if constexpr (BITS == 4) {
            w[2 * b + i] |= (c0 | c2 << 4 | c1 << 16 | c3 << 20) << (8 * r);
          } else {
            w[2 * (2 * b + i)] |= (c0 | c1 << 16) << (8 * r);
            w[2 * (2 * b + i) + 1] |= (c2 | c3 << 16) << (8 * r);
          }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < Q::kWords / 4; ++i)
    reinterpret_cast<uint4 *>(half)[i * 32 + lane] =
        make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

// Tokens 2t, 2t + 1, 2t + 8, 2t + 9.
__device__ __forceinline__ int v_token(int t, int i) { return 2 * t + (i & 1) + 8 * (i >> 1); }

template <typename T, int D, int BITS>
__device__ __forceinline__ void put_v(char *half, int lane, const uint2 (&x)[4][D / 32]) {
  using Q = QuantTile<D, BITS>;
  const int g = lane >> 2, t = lane & 3;
  uint32_t w[Q::kWords];
#pragma unroll
  for (int i = 0; i < Q::kWords; ++i) w[i] = 0;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    uint32_t e[D / 32];
#pragma unroll
    for (int a = 0; a < D / 32; ++a) {
      const uint32_t v[2] = {x[r][a].x, x[r][a].y};
      e[a] = extremes<T>(v);
    }
    if constexpr (BITS == 8) {
#pragma unroll
      for (int a = 1; a < D / 32; ++a) e[0] = min2_nan<T>(e[0], e[a]);
    }
    uint16_t *par =
        reinterpret_cast<uint16_t *>(half + Q::kCodes + v_token(t, r) * Q::kTokenParams);
    const int at = ((r & 1) << 4) | ((r >> 1) << 3);  // 4 bits: bit of the token's byte
#pragma unroll
    for (int a = 0; a < Q::kGroups; ++a) {
      const Scale<T, Q::kLevels> s(join<T>(join<T>(join<T>(e[a], 4), 8), 16));
      if (g == 0) {
        par[a] = (uint16_t)s.bits;
        par[Q::kGroups + a] = (uint16_t)(s.bits >> 16);
      }
#pragma unroll
      for (int b = a * Q::kGroup / 32; b < (a + 1) * Q::kGroup / 32; ++b) {
        const uint32_t v[2] = {x[r][b].x, x[r][b].y};
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // m-tile 2b + i: two channels
          const float2 p = unpack2<T>(v[i]);
          const uint32_t c0 = s.code(p.x), c1 = s.code(p.y);
          if constexpr (BITS == 4)
            w[2 * b + i] |= (c0 | c1 << 4) << at;
          else
            w[2 * (2 * b + i) + (r >> 1)] |= (c0 | c1 << 8) << (16 * (r & 1));
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < Q::kWords / 4; ++i)
    reinterpret_cast<uint4 *>(half)[i * 32 + lane] =
        make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

// ---- single tokens -----------------------------------------------------------------
// Row r of a tile: lane i holds channels 4i .. 4i + 3 (lanes from D / 4 on hold copies of
// channels that are left out again).
template <typename T, int D, int BITS>
__device__ __forceinline__ void put_row(char *half, int lane, int r, bool is_v, const T *row) {
  using Q = QuantTile<D, BITS>;
  const int i = lane % (D / 4);
  const uint2 x = *reinterpret_cast<const uint2 *>(row + 4 * i);
  const uint32_t v[2] = {x.x, x.y};
  uint32_t e = extremes<T>(v);
#pragma unroll
  for (int m = 1; m < Q::kGroup / 4; m <<= 1) e = join<T>(e, m);
  const Scale<T, Q::kLevels> s(e);
  if (lane >= D / 4) return;
  uint16_t *par = reinterpret_cast<uint16_t *>(half + Q::kCodes + r * Q::kTokenParams);
  if (i % (Q::kGroup / 4) == 0) {
    const int a = i / (Q::kGroup / 4);
    par[a] = (uint16_t)s.bits;
    par[Q::kGroups + a] = (uint16_t)(s.bits >> 16);
  }
  const float2 p = unpack2<T>(x.x), q = unpack2<T>(x.y);
  const uint32_t c0 = s.code(p.x), c1 = s.code(p.y), c2 = s.code(q.x), c3 = s.code(q.y);
  auto word = [&](int w, int of) {  // byte address of word w of lane `of`
    return half + ((size_t)((w >> 2) * 32 + of) * 4 + (w & 3)) * 4;
  };
  if (!is_v) {
    // channels 4i ..: k-step s, lane t of the row's eight
    const int step = 2 * (i >> 3) + (i & 1), of = 4 * (r & 7) + ((i & 7) >> 1), b = r >> 3;
    if constexpr (BITS == 4) {
      char *w = word(step, of);
      w[b] = (char)(c0 | c2 << 4);
      w[b + 2] = (char)(c1 | c3 << 4);
    } else {
      char *w = word(2 * step, of), *w1 = word(2 * step + 1, of);
      w[b] = (char)c0;
      w[b + 2] = (char)c1;
      w1[b] = (char)c2;
      w1[b + 2] = (char)c3;
    }
  } else {
    const int j = 2 * (i >> 3), of = 4 * (i & 7) + ((r & 7) >> 1), odd = r & 1, up = r >> 3;
    if constexpr (BITS == 4) {
      word(j, of)[2 * odd + up] = (char)(c0 | c1 << 4);
      word(j + 1, of)[2 * odd + up] = (char)(c2 | c3 << 4);
    } else {
      char *w = word(2 * j + up, of), *w1 = word(2 * (j + 1) + up, of);
      w[2 * odd] = (char)c0;
      w[2 * odd + 1] = (char)c1;
      w1[2 * odd] = (char)c2;
      w1[2 * odd + 1] = (char)c3;
    }
  }
}

// The tile of a sequence's token t0 (a multiple of 16) and kv head, or null (with the error
// word set) where the page table points outside the pool.
template <int BYTES>
__device__ __forceinline__ char *tile_at(const void *pool, const int *page_table, int slot, int t0,
                                         int h, int hkv, int P, int max_pp, int num_phys, int *err) {
  const int blk = t0 / P;
  if (blk >= max_pp) {
    qc_set_err(err, kDevBadPage, slot, t0, blk);
    return nullptr;
  }
  const int phys = page_table[(size_t)slot * max_pp + blk];
  if (phys < 0 || phys >= num_phys) {
    qc_set_err(err, kDevBadPhys, slot, blk, phys);
    return nullptr;
  }
  const size_t tiles = P / kQuantTile;
  return static_cast<char *>(const_cast<void *>(pool)) +
         (((size_t)phys * hkv + h) * tiles + (t0 - blk * P) / kQuantTile) * BYTES;
}

// ---- write ---------------------------------------------------------------------------
// A CTA takes one tile's tokens and every parts-th of the heads: K and V of a head are a
// warp's work each, and so are a query head's rows when positions are applied.
constexpr int kWriteWarps = 8;
constexpr int kPad = 8;  // 16-bit elements behind a rotated row in shared memory

template <typename T, int D, int BITS, bool ROT>
__global__ void __launch_bounds__(kWriteWarps * 32)
    quant_append_kernel(const __grid_constant__ QuantAppendParams p) {
  using Q = QuantTile<D, BITS>;
  __shared__ __align__(16) float2 cs[ROT ? kQuantTile * D / 2 : 1];
  __shared__ __align__(16) T rows[ROT ? kWriteWarps : 1][ROT ? kQuantTile * (D + kPad) : 1];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int item = blockIdx.x / p.parts, part = blockIdx.x - item * p.parts;
  int i = 0;
  for (int lo = 0, hi = p.n_seqs; lo < hi;) {  // the last sequence with off <= item
    const int mid = (lo + hi) >> 1;
    if (p.seqs[mid].off <= item) i = mid, lo = mid + 1;
    else hi = mid;
  }
  const QuantSeq s = p.seqs[i];
  const int t0 = s.first / kQuantTile * kQuantTile + (item - s.off) * kQuantTile;
  const int a = max(t0, s.first), b = min(t0 + kQuantTile, s.first + p.n_tokens), n = b - a;
  const long long tok0 = (long long)(p.seq0 + i) * p.n_tokens + (a - s.first);  // of the call
  const RotaryShape shape{D, ROT ? p.table.rotary_dim : 0, ROT ? p.table.neighbours : 0};
  const int pairs = shape.rot >> 1;
  if constexpr (ROT) {
    for (int e = threadIdx.x; e < n * pairs; e += kWriteWarps * 32) {
      const int t = e / pairs, j = e - t * pairs;
      const int pos = p.positions
                          ? p.positions[(long long)p.table.axis[j] * p.total_seqs * p.n_tokens + tok0 + t]
                          : a + t;
      cs[e] = turn_of(pos, p.table.turns[j]);
    }
    __syncthreads();
  }
  const int units = shape.units();
  const int works = 2 * p.hkv + (ROT ? p.hq : 0);
  for (int w = part * kWriteWarps + warp; w < works; w += p.parts * kWriteWarps) {
    if (w >= 2 * p.hkv) {  // a query head's rows
      const int h = w - 2 * p.hkv;
      for (int u = lane; u < n * units; u += 32) {
        const int t = u / units;
        RotaryUnit<T> x;
        x.load(shape, static_cast<const T *>(p.q) + (tok0 + t) * p.q_stride + h * D, u - t * units);
        x.turn(shape, cs + t * pairs);
        x.store(static_cast<T *>(p.q_out) + ((tok0 + t) * p.hq + h) * D);
      }
      continue;
    }
    const bool is_v = w >= p.hkv;
    const int h = is_v ? w - p.hkv : w;
    char *tile = tile_at<Q::kBytes>(p.pool, p.page_table, s.slot, t0, h, p.hkv, p.P, p.max_pp,
                                    p.num_phys, p.err);
    if (!tile) continue;
    char *half = tile + (is_v ? Q::kHalf : 0);
    const T *src = is_v ? static_cast<const T *>(p.v) + tok0 * p.v_stride + h * D
                        : static_cast<const T *>(p.k) + tok0 * p.k_stride + h * D;
    long long stride = is_v ? p.v_stride : p.k_stride;
    if (ROT && !is_v) {
      T *mine = rows[ROT ? warp : 0];
      __syncwarp();  // (the tile before has been read)
      for (int u = lane; u < n * units; u += 32) {
        const int t = u / units;
        RotaryUnit<T> x;
        x.load(shape, src + t * stride, u - t * units);
        x.turn(shape, cs + t * pairs);
        x.store(mine + t * (D + kPad));
      }
      __syncwarp();
      src = mine;
      stride = D + kPad;
    }
    if (n == kQuantTile) {
      const int g = lane >> 2, t = lane & 3;
      if (is_v) {
        uint2 x[4][D / 32];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int c = 0; c < D / 32; ++c)
            x[r][c] = *reinterpret_cast<const uint2 *>(src + v_token(t, r) * stride + 32 * c + 4 * g);
        put_v<T, D, BITS>(half, lane, x);
      } else {
        uint4 x[2][D / 32];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int c = 0; c < D / 32; ++c)
            x[r][c] = *reinterpret_cast<const uint4 *>(src + (g + 8 * r) * stride + 32 * c + 8 * t);
        put_k<T, D, BITS>(half, lane, x);
      }
    } else {
      for (int t = 0; t < n; ++t)
        put_row<T, D, BITS>(half, lane, a - t0 + t, is_v, src + t * stride);
    }
  }
}

// ---- read ----------------------------------------------------------------------------
template <typename T, int D, int BITS>
__global__ void __launch_bounds__(kWriteWarps * 32)
    quant_read_kernel(const __grid_constant__ QuantReadParams p) {
  using Q = QuantTile<D, BITS>;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const long long job = (long long)blockIdx.x * kWriteWarps + (threadIdx.x >> 5);
  const int works = 2 * p.hkv;
  const int item = (int)(job / works), w = (int)(job - (long long)item * works);
  if (item >= p.tiles) return;
  int i = 0;
  for (int lo = 0, hi = p.n_seqs; lo < hi;) {
    const int mid = (lo + hi) >> 1;
    if (p.seqs[mid].off <= item) i = mid, lo = mid + 1;
    else hi = mid;
  }
  const QuantSeq s = p.seqs[i];
  const int t0 = s.first / kQuantTile * kQuantTile + (item - s.off) * kQuantTile;
  const int end = s.first + p.n_tokens;
  const bool is_v = w >= p.hkv;
  const int h = is_v ? w - p.hkv : w;
  const char *tile = tile_at<Q::kBytes>(p.pool, p.page_table, s.slot, t0, h, p.hkv, p.P, p.max_pp,
                                        p.num_phys, p.err);
  if (!tile) return;
  const char *half = tile + (is_v ? Q::kHalf : 0);
  uint32_t x[Q::kWords];
#pragma unroll
  for (int k = 0; k < Q::kWords / 4; ++k) {
    const uint4 v = reinterpret_cast<const uint4 *>(half)[k * 32 + lane];
    x[4 * k] = v.x, x[4 * k + 1] = v.y, x[4 * k + 2] = v.z, x[4 * k + 3] = v.w;
  }
  T *out = static_cast<T *>(is_v ? p.v : p.k) + (size_t)i * p.n_tokens * p.hkv * D + h * D;
  // (fp32 holds step * code exactly: value = lo + step * code is rounded once, then to T.  A
  // step reaches the highest value or a little further: not beyond T's largest number, either.)
  constexpr float kMost = std::is_same<T, __half>::value ? 65504.f : 0x1.fep127f;
  auto value = [&](float lo, float st, uint32_t code) {
    const float x = fmaf(st, (float)code, lo);
    return x > kMost ? kMost : x;
  };
  auto pair = [&](float2 lo, float2 st, uint32_t a, uint32_t b) {
    return pack2<T>(value(lo.x, st.x, a), value(lo.y, st.y, b));
  };
  auto param = [&](int r, int a) {  // of a token's group: lo, step
    const uint16_t *q = reinterpret_cast<const uint16_t *>(half + Q::kCodes + r * Q::kTokenParams);
    return unpack2<T>((uint32_t)q[a] | (uint32_t)q[Q::kGroups + a] << 16);
  };
  if (!is_v) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int at = t0 + g + 8 * r;
      if (at < s.first || at >= end) continue;
      T *row = out + (size_t)(at - s.first) * p.hkv * D;
#pragma unroll
      for (int b = 0; b < D / 32; ++b) {
        const float2 e = param(g + 8 * r, b * 32 / Q::kGroup);
        const float2 lo = make_float2(e.x, e.x), st = make_float2(e.y, e.y);
        uint32_t y[4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if constexpr (BITS == 4) {
            const uint32_t c = x[2 * b + k] >> (8 * r);
            y[2 * k] = pair(lo, st, c & 15u, c >> 16 & 15u);
            y[2 * k + 1] = pair(lo, st, c >> 4 & 15u, c >> 20 & 15u);
          } else {
            const uint32_t c = x[2 * (2 * b + k)] >> (8 * r), d = x[2 * (2 * b + k) + 1] >> (8 * r);
            y[2 * k] = pair(lo, st, c & 255u, c >> 16 & 255u);
            y[2 * k + 1] = pair(lo, st, d & 255u, d >> 16 & 255u);
          }
        }
        *reinterpret_cast<uint4 *>(row + 32 * b + 8 * t) = make_uint4(y[0], y[1], y[2], y[3]);
      }
    }
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int at = t0 + v_token(t, r);
      if (at < s.first || at >= end) continue;
      T *row = out + (size_t)(at - s.first) * p.hkv * D;
      const int bit = ((r & 1) << 4) | ((r >> 1) << 3);
#pragma unroll
      for (int b = 0; b < D / 32; ++b) {
        const float2 e = param(v_token(t, r), b * 32 / Q::kGroup);
        const float2 lo = make_float2(e.x, e.x), st = make_float2(e.y, e.y);
        uint32_t y[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if constexpr (BITS == 4) {
            const uint32_t c = x[2 * b + k] >> bit;
            y[k] = pair(lo, st, c & 15u, c >> 4 & 15u);
          } else {
            const uint32_t c = x[2 * (2 * b + k) + (r >> 1)] >> (16 * (r & 1));
            y[k] = pair(lo, st, c & 255u, c >> 8 & 255u);
          }
        }
        *reinterpret_cast<uint2 *>(row + 32 * b + 4 * g) = make_uint2(y[0], y[1]);
      }
    }
  }
}

template <typename T, int D, int BITS>
cudaError_t append_of(const QuantAppendParams &p, cudaStream_t st) {
  const int grid = p.tiles * p.parts;
  return p.rotate ? launch_pdl(quant_append_kernel<T, D, BITS, true>, grid, kWriteWarps * 32, 0, st, p)
                  : launch_pdl(quant_append_kernel<T, D, BITS, false>, grid, kWriteWarps * 32, 0, st, p);
}
template <typename T, int D, int BITS>
cudaError_t read_of(const QuantReadParams &p, cudaStream_t st) {
  const long long jobs = (long long)p.tiles * 2 * p.hkv;
  const int grid = (int)((jobs + kWriteWarps - 1) / kWriteWarps);
  return launch_pdl(quant_read_kernel<T, D, BITS>, grid, kWriteWarps * 32, 0, st, p);
}

}  // namespace

#define SPD_QUANT_PICK(FN)                                                                        \
  (dtype == 0 ? (d == 64 ? (bits == 8 ? FN<__half, 64, 8>(p, st) : FN<__half, 64, 4>(p, st))       \
                         : (bits == 8 ? FN<__half, 128, 8>(p, st) : FN<__half, 128, 4>(p, st)))    \
              : (d == 64 ? (bits == 8 ? FN<__nv_bfloat16, 64, 8>(p, st)                            \
                                      : FN<__nv_bfloat16, 64, 4>(p, st))                           \
                         : (bits == 8 ? FN<__nv_bfloat16, 128, 8>(p, st)                           \
                                      : FN<__nv_bfloat16, 128, 4>(p, st))))

cudaError_t launch_quant_append(const QuantAppendParams &p, int dtype, int d, int bits,
                                cudaStream_t st) {
  const cudaError_t e = SPD_QUANT_PICK(append_of);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_quant_read(const QuantReadParams &p, int dtype, int d, int bits,
                              cudaStream_t st) {
  const cudaError_t e = SPD_QUANT_PICK(read_of);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace spd
