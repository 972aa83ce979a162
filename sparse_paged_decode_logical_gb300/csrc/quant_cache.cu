// Writing keys and values into a quantised cache and reading them back (sm_103a).
//
// A group of channels of a token is held as value = lo + step * code: lo its lowest value,
// step the least number of the cache's type with levels * step >= highest - lowest, codes
// rounded to nearest, 0 .. levels; differences count exactly, also where fp32 rounds them.  A group that holds a value that is not finite (or whose
// span exceeds fp32) gets lo = NaN and step 0: it reads back as NaN throughout.
//
// A warp takes a head's tile of 16 tokens, K and V.  Their rows come to shared memory by
// asynchronous copies, keys are rotated there, and every lane reads the channels whose codes fill
// the words that it stores (layout in quant.h), so that a group's extremes are a few shuffles away.
// Tiles that are not filled at once go token by token, byte stores.
//
// 2 bytes a value on one side, 1.03 or 0.63 on the other.  Reading back is bound by memory (16,385
// tokens of 8 kv heads of 128 channels in 8 bits 15 us, its floor; 4 bits 14.7).  Writing keys and
// values is not: 43 us for a floor of 15, DRAM at 21% of its peak, ALU at 50%, 27% of the warps.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
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

constexpr float kMagic = 12582912.f;  // 1.5 2^23: added, it leaves a rounded number in the low bits

// The low bytes of four numbers.
__device__ __forceinline__ uint32_t low_bytes(float2 a, float2 b) {
  return __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                     __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
}
// What rounding left of a - b, the difference d: a - b = d + rest exactly.
__device__ __forceinline__ float rest_of(float a, float b, float d) {
  const float a1 = d + b, b1 = a1 - d;  // (Knuth's two-sum, of a and -b)
  return (a - a1) + (b1 - b);
}
// A code n (kMagic + n in y) for a distance x - lo, which may be one off: what n step leaves of it
// is compared with half a step, ties to even.  d, the rounded distance, and n step are numbers of
// a spacing that 2 |r| - step keeps, so that only the last sum is rounded, which keeps its sign.
__device__ __forceinline__ float exact_code(float y, float x, float lo, float step) {
  const float d = x - lo, r = fmaf(kMagic - y, step, d), rest = rest_of(x, lo, d);
  const float over = (fabsf(r) + fabsf(r) - step) + copysignf(2.f, r) * rest;
  const bool odd = __float_as_uint(y) & 1u;
  return over > 0.f || (over == 0.f && odd) ? y + copysignf(1.f, r) : y;
}
// Apart: 1 warp in 5 comes here in bf16, and copies in every place would fill the instruction
// cache.  (What rounding takes from a distance costs 16,385 tokens in 8 bits 2 of 103 us.)
__device__ __noinline__ uint32_t exact_codes(float2 ya, float2 yb, float2 a, float2 b, float lo,
                                             float step) {
  return low_bytes(make_float2(exact_code(ya.x, a.x, lo, step), exact_code(ya.y, a.y, lo, step)),
                   make_float2(exact_code(yb.x, b.x, lo, step), exact_code(yb.y, b.y, lo, step)));
}

// What a group's codes are made with.
template <typename T, int LEVELS>
struct Scale {
  uint32_t bits;  // lo, step: as stored
  float lo, step, inv;
  bool tiny;  // step below 2^-100: everything times 2^100

  __device__ __forceinline__ explicit Scale(uint32_t e) {  // (lowest, -highest)
    const float2 x = unpack2<T>(e);
    const float span = -x.y - x.x;  // highest - lowest, rounded
    lo = x.x;
    tiny = false;
    if (!(span <= 3.402823466e38f)) {
      bits = 0x7fffu;  // NaN in either type, step 0
      lo = __uint_as_float(0x7fffffffu);
      step = inv = 0.f;
      return;
    }
    // The least number of T that reaches: products with it are exact (11 + 8 bits).
    uint32_t h = pack2<T>(span * (1.f / LEVELS), 0.f) & 0xffffu;
    step = unpack2<T>(h).x;
    const float most = step * (float)LEVELS, less = h > 0 ? unpack2<T>(h - 1).x : -1.f;
    bool more = most < span, fewer = less * (float)LEVELS >= span;
    // (what rounding took from the span counts only here)
    if (most == span || less * (float)LEVELS == span) {
      const bool beyond = rest_of(-x.y, x.x, span) > 0.f;
      more |= beyond && most == span;
      fewer &= !beyond || less * (float)LEVELS > span;
    }
    if (more) step = unpack2<T>(++h).x;
    if (fewer) --h, step = less;
    bits = (e & 0xffffu) | h << 16;
    tiny = step < 0x1p-100f;
    if (tiny) {
      lo *= 0x1p100f;
      step *= 0x1p100f;
    }
    inv = step > 0.f ? rcp_near(step) : 0.f;
  }
  static __device__ __forceinline__ float rcp_near(float x) {  // within 2^-23
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
  }
  // round((x - lo) / step), ties to even, of the four channels of a pair of words: bytes.  The
  // product with 1 / step is off by less than 2^-21 of a quotient of at most LEVELS; where one
  // lies closer than that to the middle between two codes, exact_code decides.  (In bf16 that is
  // common, values and steps have 8 bits.)  Rounded by adding kMagic, whose low
  // bits then are the code: a conversion to an integer runs at a quarter of the rate.
  __device__ __forceinline__ uint32_t codes(uint32_t v0, uint32_t v1) const {
    constexpr float kNear = 0.5f - LEVELS * 0x1p-21f;
    const float2 l = make_float2(lo, lo), r = make_float2(inv, inv), m = make_float2(kMagic, kMagic);
    float2 a = unpack2<T>(v0), b = unpack2<T>(v1);
    if (tiny) {
      a = f2_mul(a, make_float2(0x1p100f, 0x1p100f));
      b = f2_mul(b, make_float2(0x1p100f, 0x1p100f));
    }
    const float2 ta = f2_mul(f2_sub(a, l), r), tb = f2_mul(f2_sub(b, l), r);
    const float2 ya = f2_add(ta, m), yb = f2_add(tb, m);
    const float2 ea = f2_sub(ta, f2_sub(ya, m)), eb = f2_sub(tb, f2_sub(yb, m));
    const float near = fmaxf(fmax3f(fabsf(ea.x), fabsf(ea.y), fabsf(eb.x)), fabsf(eb.y));
    return near >= kNear ? exact_codes(ya, yb, a, b, lo, step) : low_bytes(ya, yb);
  }
};

// ---- whole tiles -------------------------------------------------------------------
// From the rows of 16 tokens in shared memory.  The loops over groups stay loops: unrolled, the
// kernel waits for its instructions.
template <typename T, int D, int BITS>
__device__ __forceinline__ void put_param(char *half, int token, int group, uint32_t bits) {
  using Q = QuantTile<D, BITS>;
  uint16_t *par = reinterpret_cast<uint16_t *>(half + Q::kCodes + token * Q::kTokenParams) + group;
  par[0] = (uint16_t)bits;
  par[Q::kGroups] = (uint16_t)(bits >> 16);
}

template <typename T, int D, int BITS>
__device__ __forceinline__ void put_k(char *half, int lane, const T *rows, int stride) {
  using Q = QuantTile<D, BITS>;
  using S = Scale<T, Q::kLevels>;
  const int g = lane >> 2, t = lane & 3;
  rows += g * stride + 8 * t;
  auto piece = [&](int r, int b) {  // token g + 8r, the lane's 8 channels of 32
    return *reinterpret_cast<const uint4 *>(rows + 8 * r * stride + 32 * b);
  };
  auto span = [&](uint4 x) {
    const uint32_t v[4] = {x.x, x.y, x.z, x.w};
    return extremes<T>(v);
  };
  auto scale = [&](uint32_t e, int r, int group) {
    const S s(join<T>(join<T>(e, 1), 2));
    if (t == 0) put_param<T, D, BITS>(half, g + 8 * r, group, s.bits);
    return s;
  };
  if constexpr (BITS == 8) {
    uint32_t e0 = span(piece(0, 0)), e1 = span(piece(1, 0));
#pragma unroll
    for (int b = 1; b < D / 32; ++b) {
      e0 = min2_nan<T>(e0, span(piece(0, b)));
      e1 = min2_nan<T>(e1, span(piece(1, b)));
    }
    const S s0 = scale(e0, 0, 0), s1 = scale(e1, 1, 0);
#pragma unroll 1
    for (int b = 0; b < D / 32; ++b) {
      const uint4 x = piece(0, b), y = piece(1, b);
      const uint32_t x0 = s0.codes(x.x, x.y), x1 = s0.codes(x.z, x.w);
      const uint32_t y0 = s1.codes(y.x, y.y), y1 = s1.codes(y.z, y.w);
      reinterpret_cast<uint4 *>(half)[b * 32 + lane] =
          make_uint4(__byte_perm(x0, y0, 0x5140), __byte_perm(x0, y0, 0x7362),
                     __byte_perm(x1, y1, 0x5140), __byte_perm(x1, y1, 0x7362));
    }
  } else {
#pragma unroll 1
    for (int b = 0; b < D / 32; ++b) {
      const uint4 x = piece(0, b), y = piece(1, b);
      const S s0 = scale(span(x), 0, b), s1 = scale(span(y), 1, b);
      // (codes 0 and 2 in one byte, 1 and 3 in the next)
      auto nibbles = [](uint32_t c) { return c | c >> 12; };
      const uint32_t x0 = nibbles(s0.codes(x.x, x.y)), x1 = nibbles(s0.codes(x.z, x.w));
      const uint32_t y0 = nibbles(s1.codes(y.x, y.y)), y1 = nibbles(s1.codes(y.z, y.w));
      reinterpret_cast<uint2 *>(half)[((b >> 1) * 32 + lane) * 2 + (b & 1)] =
          make_uint2(__byte_perm(x0, y0, 0x5140), __byte_perm(x1, y1, 0x5140));
    }
  }
}

// Tokens 2t, 2t + 1, 2t + 8, 2t + 9.
__device__ __forceinline__ int v_token(int t, int i) { return 2 * t + (i & 1) + 8 * (i >> 1); }

template <typename T, int D, int BITS>
__device__ __forceinline__ void put_v(char *half, int lane, const T *rows, int stride) {
  using Q = QuantTile<D, BITS>;
  using S = Scale<T, Q::kLevels>;
  const int g = lane >> 2, t = lane & 3;
  rows += 2 * t * stride + 4 * g;
  auto piece = [&](int r, int b) {  // token v_token(t, r), the lane's 4 channels of 32
    return *reinterpret_cast<const uint2 *>(rows + ((r & 1) + 8 * (r >> 1)) * stride + 32 * b);
  };
  auto span = [&](uint2 x) {
    const uint32_t v[2] = {x.x, x.y};
    return extremes<T>(v);
  };
  auto scale = [&](uint32_t e, int r, int group) {
    const S s(join<T>(join<T>(join<T>(e, 4), 8), 16));
    if (g == 0) put_param<T, D, BITS>(half, v_token(t, r), group, s.bits);
    return s;
  };
  if constexpr (BITS == 8) {
    uint32_t e[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      e[r] = span(piece(r, 0));
#pragma unroll
      for (int b = 1; b < D / 32; ++b) e[r] = min2_nan<T>(e[r], span(piece(r, b)));
    }
    const S s0 = scale(e[0], 0, 0), s1 = scale(e[1], 1, 0), s2 = scale(e[2], 2, 0),
            s3 = scale(e[3], 3, 0);
#pragma unroll 1
    for (int b = 0; b < D / 32; ++b) {
      const uint2 x0 = piece(0, b), x1 = piece(1, b), x2 = piece(2, b), x3 = piece(3, b);
      const uint32_t c0 = s0.codes(x0.x, x0.y), c1 = s1.codes(x1.x, x1.y);
      const uint32_t c2 = s2.codes(x2.x, x2.y), c3 = s3.codes(x3.x, x3.y);
      reinterpret_cast<uint4 *>(half)[b * 32 + lane] =
          make_uint4(__byte_perm(c0, c1, 0x5410), __byte_perm(c2, c3, 0x5410),
                     __byte_perm(c0, c1, 0x7632), __byte_perm(c2, c3, 0x7632));
    }
  } else {
#pragma unroll 1
    for (int b = 0; b < D / 32; ++b) {
      uint32_t c[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint2 x = piece(r, b);
        c[r] = scale(span(x), r, b).codes(x.x, x.y);
        c[r] |= c[r] >> 4;  // (channels 0 and 1 in byte 0, 2 and 3 in byte 2)
      }
      const uint32_t a = __byte_perm(c[0], c[2], 0x6240), d = __byte_perm(c[1], c[3], 0x6240);
      reinterpret_cast<uint2 *>(half)[((b >> 1) * 32 + lane) * 2 + (b & 1)] =
          make_uint2(__byte_perm(a, d, 0x5410), __byte_perm(a, d, 0x7632));
    }
  }
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
  if (i % (Q::kGroup / 4) == 0) put_param<T, D, BITS>(half, r, i / (Q::kGroup / 4), s.bits);
  const uint32_t c = s.codes(x.x, x.y);
  auto word = [&](int w, int of) {  // byte address of word w of lane `of`
    return half + ((size_t)((w >> 2) * 32 + of) * 4 + (w & 3)) * 4;
  };
  if (!is_v) {
    // channels 4i ..: k-step, lane t of the row's eight
    const int step = 2 * (i >> 3) + (i & 1), of = 4 * (r & 7) + ((i & 7) >> 1), b = r >> 3;
    if constexpr (BITS == 4) {
      const uint32_t n = c | c >> 12;
      char *w = word(step, of);
      w[b] = (char)n;
      w[b + 2] = (char)(n >> 8);
    } else {
      char *w = word(2 * step, of), *w1 = word(2 * step + 1, of);
      w[b] = (char)c;
      w[b + 2] = (char)(c >> 8);
      w1[b] = (char)(c >> 16);
      w1[b + 2] = (char)(c >> 24);
    }
  } else {
    const int j = 2 * (i >> 3), of = 4 * (i & 7) + ((r & 7) >> 1), odd = r & 1, up = r >> 3;
    if constexpr (BITS == 4) {
      const uint32_t n = c | c >> 4;
      word(j, of)[2 * odd + up] = (char)n;
      word(j + 1, of)[2 * odd + up] = (char)(n >> 16);
    } else {
      char *w = word(2 * j + up, of), *w1 = word(2 * (j + 1) + up, of);
      w[2 * odd] = (char)c;
      w[2 * odd + 1] = (char)(c >> 8);
      w1[2 * odd] = (char)(c >> 16);
      w1[2 * odd + 1] = (char)(c >> 24);
    }
  }
}

// The physical page of a sequence's block, or -1 (with the error word set) where the page table
// has none in the pool.
__device__ __forceinline__ int page_of(const int *page_table, int slot, int blk, int max_pp,
                                       int num_phys, int *err) {
  if (blk >= max_pp) {
    qc_set_err(err, kDevBadPage, slot, 0, blk);
    return -1;
  }
  const int phys = page_table[(size_t)slot * max_pp + blk];
  if (phys < 0 || phys >= num_phys) {
    qc_set_err(err, kDevBadPhys, slot, blk, phys);
    return -1;
  }
  return phys;
}
// The tile of token t0 (a multiple of 16) and kv head h on a page.
template <int BYTES>
__device__ __forceinline__ char *tile_at(const void *pool, int phys, int t0, int h, int hkv, int P) {
  const size_t tiles = P / kQuantTile;
  return static_cast<char *>(const_cast<void *>(pool)) +
         (((size_t)phys * hkv + h) * tiles + t0 % P / kQuantTile) * BYTES;
}

// ---- write ---------------------------------------------------------------------------
constexpr int kWriteWarps = kQuantWriteWarps;
constexpr int kPad = 8;  // 16-bit elements behind a row in shared memory: rows start at other banks

// A head's rows of n tokens, rotated, a warp's.
template <typename T, typename Src, typename Dst>
__device__ __forceinline__ void rotate_rows(const RotaryShape &shape, int n, const float2 *cs,
                                            int lane, Src src, Dst dst) {
  const int units = shape.units(), all = n * units;
  const unsigned per = (65536u + units - 1) / units;  // u / units = u per / 2^16 for u <= 256
#pragma unroll 2
  for (int u = lane; u < all; u += 32) {
    const int t = (int)((unsigned)u * per >> 16);
    RotaryUnit<T> x;
    x.load(shape, src(t), u - t * units);
    x.turn(shape, cs + t * sine_stride(shape.rot));
    x.store(dst(t));
  }
}

// Rows of n tokens into a warp's buffer by asynchronous copies, which cost no registers while
// they are under way.
template <typename T, int D>
__device__ __forceinline__ void stage_rows(T *buf, const T *src, long long stride, int n, int lane) {
  constexpr int kChunks = D / 8;  // 16-byte pieces of a row
#pragma unroll
  for (int k = 0; k < kQuantTile * kChunks / 32; ++k) {
    const int i = lane + 32 * k, t = i / kChunks, c = i % kChunks;
    if (t < n)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(buf + t * (D + kPad) + 8 * c)),
                   "l"(src + t * stride + 8 * c)
                   : "memory");
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}

// A CTA takes one tile's tokens and every parts-th of the heads: K and V of a head are one
// warp's work, and so are a query head's rows when positions are applied.  Keys are on their way
// to shared memory, where they are rotated, while the sines are made and the values done.
// (80 registers where they suffice, for a sixth CTA on the SM: 6 x 1,111 tokens into 4 bits with
// reading back 9.4 us, 11.1 with 92.)
template <typename T, int D, int BITS, bool ROT>
__global__ void __launch_bounds__(kWriteWarps * 32, !ROT && (D == 64 || BITS == 4) ? 6 : 5)
    quant_append_kernel(const __grid_constant__ QuantAppendParams p) {
  using Q = QuantTile<D, BITS>;
  extern __shared__ __align__(16) char smem[];  // rows of K and V of every warp, the sines
  float2 *const cs = reinterpret_cast<float2 *>(smem + kWriteWarps * 2 * kQuantTile * (D + kPad) * 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int item = blockIdx.x / p.parts, part = blockIdx.x - item * p.parts;
  int i = 0;
  for (int lo = 0, hi = p.n_seqs; lo < hi;) {  // the last sequence with off <= item
    const int mid = (lo + hi) >> 1;
    if (p.seqs[mid].off <= item) i = mid, lo = mid + 1;
    else hi = mid;
  }
  const QuantAppendSeq s = p.seqs[i];
  const int t0 = s.first / kQuantTile * kQuantTile + (item - s.off) * kQuantTile;
  const int a = max(t0, s.first), b = min(t0 + kQuantTile, s.first + p.n_tokens), n = b - a;
  const long long tok0 = (long long)(p.seq0 + i) * p.n_tokens + (a - s.first);  // of the call
  const RotaryShape shape{D, ROT ? p.table.rotary_dim : 0, ROT ? p.table.neighbours : 0};
  T *const mine = reinterpret_cast<T *>(smem) + warp * 2 * kQuantTile * (D + kPad);
  pdl_wait();
  pdl_launch_dependents();
  T *const mine_v = mine + kQuantTile * (D + kPad);
  auto load = [&](int h) {
    stage_rows<T, D>(mine_v, static_cast<const T *>(p.v) + tok0 * p.v_stride + h * D, p.v_stride, n, lane);
    stage_rows<T, D>(mine, static_cast<const T *>(p.k) + tok0 * p.k_stride + h * D, p.k_stride, n, lane);
  };
  int h = part * kWriteWarps + warp;
  const int step = p.parts * kWriteWarps;
  if (h < p.hkv) load(h);
  if constexpr (ROT) {
    const long long axis_stride = (long long)p.total_seqs * p.n_tokens;
    make_sines<kWriteWarps * 32>(p.table, n, 0, cs, [&](int axis, int k) {
      return p.positions ? p.positions[axis * axis_stride + tok0 + k] : a + k;
    });
    __syncthreads();
  }
  // New pages come with the launch, which also writes them to the table: a decode step whose
  // sequences take pages is one launch.
  if (blockIdx.x == 0)
    for (int u = threadIdx.x; u < p.n_updates; u += kWriteWarps * 32)
      p.page_table[(size_t)p.updates[u].slot * p.max_pp + p.updates[u].index] = p.updates[u].phys;
  const int blk = t0 / p.P, fresh = blk - s.page;
  const int phys = fresh >= 0 && fresh < s.pages
                       ? p.updates[s.upd + fresh].phys
                       : page_of(p.page_table, s.slot, blk, p.max_pp, p.num_phys, p.err);
#pragma unroll 1
  for (; h < p.hkv; h += step) {
    char *tile = phys < 0 ? nullptr : tile_at<Q::kBytes>(p.pool, phys, t0, h, p.hkv, p.P);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncwarp();
    if (tile) {
      if (n == kQuantTile)
        put_v<T, D, BITS>(tile + Q::kHalf, lane, mine_v, D + kPad);
      else
        for (int k = 0; k < n; ++k)
          put_row<T, D, BITS>(tile + Q::kHalf, lane, a - t0 + k, true, mine_v + k * (D + kPad));
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
    if (ROT) {
      rotate_rows<T>(
          shape, n, cs, lane, [&](int k) { return mine + k * (D + kPad); },
          [&](int k) { return mine + k * (D + kPad); });
      __syncwarp();
    }
    if (tile) {
      if (n == kQuantTile)
        put_k<T, D, BITS>(tile, lane, mine, D + kPad);
      else
        for (int k = 0; k < n; ++k)
          put_row<T, D, BITS>(tile, lane, a - t0 + k, false, mine + k * (D + kPad));
    }
    __syncwarp();
    if (h + step < p.hkv) load(h + step);
  }
  if constexpr (ROT) {
    for (h -= p.hkv; h < p.hq; h += step)  // query heads
      rotate_rows<T>(
          shape, n, cs, lane,
          [&](int k) { return static_cast<const T *>(p.q) + (tok0 + k) * p.q_stride + h * D; },
          [&](int k) { return static_cast<T *>(p.q_out) + ((tok0 + k) * p.hq + h) * D; });
  }
}

// ---- read ----------------------------------------------------------------------------
constexpr int kReadWarps = 8;

template <typename T, int D, int BITS>
__global__ void __launch_bounds__(kReadWarps * 32)
    quant_read_kernel(const __grid_constant__ QuantReadParams p) {
  using Q = QuantTile<D, BITS>;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const long long job = (long long)blockIdx.x * kReadWarps + (threadIdx.x >> 5);
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
  const int phys = page_of(p.page_table, s.slot, t0 / p.P, p.max_pp, p.num_phys, p.err);
  if (phys < 0) return;
  const char *tile = tile_at<Q::kBytes>(p.pool, phys, t0, h, p.hkv, p.P);
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

template <typename T, int D, int BITS, bool ROT>
cudaError_t append_one(const QuantAppendParams &p, cudaStream_t st) {
  constexpr int smem = kWriteWarps * 2 * kQuantTile * (D + kPad) * 2 + (ROT ? kQuantTile * sine_stride(D) * 8 : 0);
  static std::atomic<uint64_t> ready{0};
  const auto kernel = quant_append_kernel<T, D, BITS, ROT>;
  const cudaError_t e = allow_smem(kernel, smem, &ready);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, p.tiles * p.parts, kWriteWarps * 32, smem, st, p);
}
template <typename T, int D, int BITS>
cudaError_t append_of(const QuantAppendParams &p, cudaStream_t st) {
  return p.rotate ? append_one<T, D, BITS, true>(p, st) : append_one<T, D, BITS, false>(p, st);
}
template <typename T, int D, int BITS>
cudaError_t read_of(const QuantReadParams &p, cudaStream_t st) {
  const long long jobs = (long long)p.tiles * 2 * p.hkv;
  const int grid = (int)((jobs + kReadWarps - 1) / kReadWarps);
  return launch_pdl(quant_read_kernel<T, D, BITS>, grid, kReadWarps * 32, 0, st, p);
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
