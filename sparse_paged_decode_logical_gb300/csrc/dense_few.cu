// Decode attention on the 5th-generation tensor cores for a prefix that 9 to 32
// (sequence, query head) rows of a kv head share, 128 channels.
//
// Few rows waste a product whose rows are queries, so keys take the rows:
//   S^T = K . Q^T      M 128 keys x N rows, K the A operand as it lies in the
//                      cache, fp32 in tensor memory; a thread holds one key's
//                      scores of every row;
//   softmax            against a reference per row that is moved (and O^T
//                      scaled) only when some score exceeds it by 2^8, so that a
//                      step needs one vote and no reduction over the keys; sums
//                      per thread, joined at the end;
//   O^T += V^T . P^T   M 128 channels x N rows: A is V read transposed, P^T goes
//                      through shared memory (16 bits, with kSplitP one or
//                      two more products for what the rounding left).
// A step of 128 keys moves 64 KB and takes 1,024 cycles of the tensor pipe (64
// bytes per cycle; an SM's share of HBM is 23), whatever the rows: memory is the
// bound.  K and V are single buffers, freed as soon as their product is done;
// two or three CTAs per SM overlap one another's waits.  5 sequences (20 rows)
// over 120,001 tokens with cap and bias: 98 us, 158 with mma.sync tiles of 16
// rows, 141 with the kernel whose rows are queries.  Up to 8 rows (a sequence's own
// tokens) the mma.sync kernel is as fast or faster: its warps start without the
// set-up of tensor memory and hand-overs between roles (64 sequences' own
// tokens 51 us against 54, one sequence's 6 against 11).
//
// Keys go from the newest to the oldest: a distance bias then finds its largest
// scores first.  Warps 0-3: softmax; 4: MMA issue; 5: TMA.  Every wait is
// bounded, and every waiter at most one completion behind its barrier; SF of a
// step also says that the step before's P . V is done.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <float.h>
#include <math_constants.h>

#include "dense.h"
#include "dense_math.cuh"
#include "ptx.cuh"
#include "spd_internal.h"

namespace spd {
namespace {

constexpr uint32_t kFewWait = 1u << 22;
constexpr int kFewD = 128, kFewThreads = 192;
constexpr float kFewNone = -FLT_MAX;  // the reference of a row that has met no key

// NR: rows of the products (a multiple of 16).
// kParts: 16-bit parts that a weight is kept in.
template <int NR, int kParts> struct FewSmem {
  static constexpr int kK = 0;                    // [2 x 64 channels][128 keys][128 B]
  static constexpr int kV = 32768;
  static constexpr int kQ = 65536;                // [2 x 64 channels][NR][128 B]
  static constexpr int kP = kQ + 2 * NR * 128;    // [part][2 x 64 keys][NR][128 B]
  static constexpr int kRow = kP + 2 * kParts * NR * 128;
  // per row: slope, tokens behind the keys; reference, factor; per warp and row:
  // max / sum
  static constexpr int kRef = kRow + NR * 8;
  static constexpr int kWarp = kRef + NR * 8;
  static constexpr int kBars = kWarp + 4 * NR * 4;
  static constexpr int kBytes = kBars + 80 + 1024;  // + alignment slack
};
// K full, V full, S done, P written, P . V done, Q written, the last P . V, drain
enum { kFewKF, kFewVF, kFewSF, kFewPF, kFewOD, kFewQF, kFewOF, kFewDR, kFewNumBars };

__device__ __forceinline__ void few_set_err(int *err, int code, int a, int b, int c) {
  if (atomicCAS(err, 0, code) == 0) {
    err[1] = a;
    err[2] = b;
    err[3] = c;
  }
}
__device__ __forceinline__ bool few_wait(uint64_t *bar, uint32_t parity, volatile int *fail) {
  for (uint32_t i = 0; i < kFewWait; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 255u) == 255u && *fail) return false;
  }
  *fail = 1;
  return false;
}
__device__ __forceinline__ void few_drain(uint64_t *bar, uint32_t parity) {
  for (uint32_t i = 0; i < kFewWait; ++i)
    if (mbar_try_wait(bar, parity)) return;
}
// The softmax warps' barrier, and whether any of them votes yes.
__device__ __forceinline__ void few_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool few_any(bool x) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, 1, 128, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}
// An integer that orders as the float does (NaN as -inf).
__device__ __forceinline__ int float_order(float x) {
  if (isnan(x)) x = -CUDART_INF_F;
  const int i = __float_as_int(x);
  return i >= 0 ? i : i ^ 0x7fffffff;
}
__device__ __forceinline__ float order_float(int i) {
  return __int_as_float(i >= 0 ? i : i ^ 0x7fffffff);
}

template <typename T> struct FewT;
template <> struct FewT<__nv_bfloat16> {
  static constexpr bool bf16 = true;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t x) {
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
  }
};
template <> struct FewT<__half> {
  static constexpr bool bf16 = false;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t x) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&x));
  }
};

// Outputs of 32 bits: 22 bits of a weight in two fp16 parts, 24 in three of bf16
// (two hold 16).
template <typename T, bool kSplitP>
constexpr int kFewParts = !kSplitP ? 1 : FewT<T>::bf16 ? 3 : 2;

// NR columns of the warp's 32 lanes.
template <int NR>
__device__ __forceinline__ void few_load(uint32_t taddr, float (&x)[NR]) {
  if constexpr (NR == 16) {
    uint32_t r[16];
    tmem_ld16(taddr, r);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      asm volatile("" : "+r"(r[i]));  // (not before the wait)
      x[i] = __uint_as_float(r[i]);
    }
  } else {
#pragma unroll
    for (int c = 0; c < NR; c += 32) {
      uint32_t r[32];
      tmem_ld32_sync(taddr + c, r);
#pragma unroll
      for (int i = 0; i < 32; ++i) x[c + i] = __uint_as_float(r[i]);
    }
  }
}

template <typename T, int NR, bool kSplitP>
__global__ void __launch_bounds__(kFewThreads, NR <= 16 ? 3 : 2)
    dense_few_kernel(const __grid_constant__ DenseDecodeParams p) {
  constexpr int kParts = kFewParts<T, kSplitP>;
  using Sm = FewSmem<NR, kParts>;
  extern __shared__ uint8_t few_smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(few_smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Sm::kBars);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Sm::kBars + 64);
  volatile int *fail = reinterpret_cast<volatile int *>(smem + Sm::kBars + 68);
  static_assert(kFewNumBars * 8 <= 64, "barriers");
  constexpr int kCols = 2 * NR < 32 ? 32 : 2 * NR;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // ---- the item: row tile, kv head, split, its tiles of 128 keys.  Row tiles of
  // the same keys lie next to one another: the second finds them in L2 ----
  const int row_tiles = (p.n * p.G + p.prefix_rows - 1) / p.prefix_rows;
  const int row_tile = blockIdx.x % row_tiles, rest = blockIdx.x / row_tiles;
  const int hk = rest / p.prefix_ns, split = rest % p.prefix_ns;
  const int row0 = row_tile * p.prefix_rows, rows = min(p.prefix_rows, p.n * p.G - row0);
  const int slot = p.prefix_slot, L = p.prefix_len;
  const int tile0 = split * p.prefix_tpi;
  const size_t at_row =
      ((size_t)(row_tile * p.Hkv + hk) * p.prefix_ns + split) * p.prefix_rows;
  float2 *ml_out = p.pre_ml + at_row;
  float *o_out = p.pre_o + at_row * kFewD;
  const int tile1 = min(tile0 + p.prefix_tpi, (L + kFewKeys - 1) / kFewKeys);
  const int nt = max(0, tile1 - tile0);
  auto key0_of = [&](int j) { return (tile1 - 1 - j) * kFewKeys; };

  if (warp == 4) tmem_alloc(tmem_slot, kCols);
  if (tid == 160) {
    for (int x = 0; x < kFewNumBars; ++x)
      mbar_init(&bars[x], x == kFewPF || x == kFewQF ? 4 : 1);  // (one arrival per softmax warp)
    *fail = 0;
    fence_mbar_init();
    prefetch_tmap(&p.tm_k);
    prefetch_tmap(&p.tm_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  // behind another kernel of this call nothing is waited for: that kernel started
  // its dependents after its own wait, so all that is read here is there, and
  // the two write to different places
  if (!p.follow) pdl_wait();
  pdl_launch_dependents();

  if (warp == 5) {
    // ---- TMA: boxes of box_rows rows, none of which crosses a page; only
    // those that hold a token ----
    if (lane == 0) {
      const int *table = p.page_table + (size_t)slot * p.max_pp;
      const int br = p.box_rows;
      int k_issued = 0, v_issued = 0;
      for (int j = 0; j < nt; ++j) {
        const int key0 = key0_of(j), nbox = (min(kFewKeys, L - key0) + br - 1) / br;
        int plane[8], y[8];
        bool ok = true;
        for (int b = 0; b < nbox; ++b) {
          const int t = key0 + b * br, blk = t / p.P;
          const int phys = blk < p.max_pp ? table[blk] : -1;
          if (phys < 0 || phys >= p.num_phys) {
            few_set_err(p.err, blk < p.max_pp ? kDevBadPhys : kDevBadPage, slot, blk, phys);
            *fail = 1;
            ok = false;
            break;
          }
          plane[b & 7] = phys * p.Hkv + hk;
          y[b & 7] = t - blk * p.P;
        }
        if (!ok) break;
        if (j > 0 && !few_wait(&bars[kFewSF], (j - 1) & 1, fail)) break;
        mbar_arrive_expect_tx(&bars[kFewKF], nbox * br * 256);
        for (int b = 0; b < nbox; ++b)
          for (int h = 0; h < 2; ++h)
            tma_load_4d(smem + Sm::kK + h * 16384 + b * br * 128, &p.tm_k, 0, y[b & 7], h,
                        plane[b & 7], &bars[kFewKF]);
        ++k_issued;
        if (j > 0 && !few_wait(&bars[kFewOD], (j - 1) & 1, fail)) break;
        mbar_arrive_expect_tx(&bars[kFewVF], nbox * br * 256);
        for (int b = 0; b < nbox; ++b)
          for (int h = 0; h < 2; ++h)
            tma_load_4d(smem + Sm::kV + h * 16384 + b * br * 128, &p.tm_v, 0, y[b & 7], h,
                        plane[b & 7], &bars[kFewVF]);
        ++v_issued;
      }
      // every copy lands before the CTA leaves
      if (k_issued) few_drain(&bars[kFewKF], (k_issued - 1) & 1);
      if (v_issued) few_drain(&bars[kFewVF], (v_issued - 1) & 1);
    }
  } else if (warp == 4) {
    // ---- MMA issue (the whole warp, one elected lane issuing) ----
    const bool bf = FewT<T>::bf16;
    const uint32_t idesc_s = umma_idesc_f16(bf, 128, NR, 0, 0);  // K . Q^T
    const uint32_t idesc_o = umma_idesc_f16(bf, 128, NR, 1, 0);  // V^T . P^T: V MN-major
    const uint64_t dk = umma_desc_sw128(smem_u32(smem + Sm::kK), 16, 1024);
    const uint64_t dq = umma_desc_sw128(smem_u32(smem + Sm::kQ), 16, 1024);
    // (V's 64-channel halves lie 16,384 bytes apart)
    const uint64_t dv = umma_desc_sw128(smem_u32(smem + Sm::kV), 16384, 1024);
    const uint64_t dp = umma_desc_sw128(smem_u32(smem + Sm::kP), 16, 1024);
    auto wwait = [&](int bar, uint32_t parity) {
      return __all_sync(0xffffffffu, few_wait(&bars[bar], parity, fail));
    };
    bool ok = nt > 0 && wwait(kFewQF, 0), any = false;
    for (int j = 0; j < nt && ok; ++j) {
      if (!(ok = wwait(kFewKF, j & 1))) break;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        umma_f16_warp(tmem, dk + (uint64_t)(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                      dq + (uint64_t)(((kk >> 2) * NR * 128 + (kk & 3) * 32) >> 4), idesc_s, kk > 0);
      umma_commit_warp(&bars[kFewSF]);
      any = true;
      if (!(ok = wwait(kFewVF, j & 1))) break;
      if (!(ok = wwait(kFewPF, j & 1))) break;
      tc_fence_after();
#pragma unroll
      for (int part = 0; part < kParts; ++part)
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          umma_f16_warp(tmem + NR, dv + (uint64_t)((kk * 2048) >> 4),
                        dp + (uint64_t)((part * 2 * NR * 128 + (kk >> 2) * NR * 128 + (kk & 3) * 32) >> 4),
                        idesc_o, j > 0 || part > 0 || kk > 0);
      umma_commit_warp(&bars[kFewOD]);
      if (j == nt - 1) umma_commit_warp(&bars[kFewOF]);
    }
    if (any) {  // every MMA done before the CTA frees its memory
      umma_commit_warp(&bars[kFewDR]);
      if (lane == 0) few_drain(&bars[kFewDR], 0);
    }
  } else {
    // ---- Q and the rows' constants ----
    const uint32_t lanes = tmem + ((uint32_t)(32 * warp) << 16);
    float2 *rowc = reinterpret_cast<float2 *>(smem + Sm::kRow);
    float *ref = reinterpret_cast<float *>(smem + Sm::kRef), *fac = ref + NR;
    float *wred = reinterpret_cast<float *>(smem + Sm::kWarp);  // [4][NR]
    for (int x = tid; x < NR * 16; x += 128) {
      const int r = x >> 4, ch = x & 15;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (r < rows) {
        const int sq = (row0 + r) / p.G, h = hk * p.G + (row0 + r) % p.G;
        v = *reinterpret_cast<const uint4 *>(static_cast<const T *>(p.q) +
                                             ((size_t)sq * p.Hq + h) * kFewD + ch * 8);
      }
      *reinterpret_cast<uint4 *>(smem + Sm::kQ + (ch >> 3) * NR * 128 + swz128(r, ch & 7)) = v;
    }
    for (int x = tid; x < 2 * kParts * NR * 8; x += 128)
      *reinterpret_cast<uint4 *>(smem + Sm::kP + x * 16) = make_uint4(0, 0, 0, 0);
    if (tid < NR) {
      const int sq = (row0 + tid) / p.G, h = hk * p.G + (row0 + tid) % p.G;
      const bool live = tid < rows;
      rowc[tid] = make_float2(
          live && p.rule.slopes ? p.rule.slopes[h] * 1.4426950408889634f : 0.f,
          live ? (float)p.seqs[sq].L : 0.f);  // the row's own tokens behind the prefix
      ref[tid] = kFewNone;
    }
    fence_proxy_async_smem();
    few_sync();
    if (lane == 0) mbar_arrive(&bars[kFewQF]);
    // where this thread's key lies in a row of P^T: 16-byte piece and place in it
    uint8_t *const prow = smem + Sm::kP + (tid >> 6) * (NR * 128) + (tid & 7) * 2;
    const uint32_t piece = ((tid >> 3) & 7) << 4;
    // sums, and what a weight's exponent counts from: the rows' references less
    // the shift
    float l[NR], rf[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      l[r] = 0.f;
      rf[r] = kFewNone;
    }
    bool ok = true;
    // (the four warps leave the loop together: a wait that gave up in one of them
    // shows in the next vote)
    for (int j = 0; j < nt; ++j) {
      const int key0 = key0_of(j), key = key0 + tid;
      const bool in = key < L;
      ok = __all_sync(0xffffffffu, ok && few_wait(&bars[kFewSF], j & 1, fail));
      tc_fence_after();
      float x[NR];
      few_load<NR>(lanes, x);
      if (p.rule.cap_out > 0.f) {
        if (p.precise) {
#pragma unroll
          for (int r = 0; r < NR; ++r) x[r] = cap_any(p.rule, x[r]);
        } else {
#pragma unroll
          for (int r = 0; r < NR; r += 2) {
            const float2 y = cap_16bit(p.rule, make_float2(x[r], x[r + 1]));
            x[r] = y.x;
            x[r + 1] = y.y;
          }
        }
      } else {
#pragma unroll
        for (int r = 0; r < NR; ++r) x[r] *= p.rule.scale_log2;
      }
      if (p.rule.slopes) {
        const float at = (float)(L - 1 - key);  // distance from the last key
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const float2 c = rowc[r];
          x[r] = fmaf(-c.x, c.y + at, x[r]);
        }
      }
      bool grow = false;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        if (!in) x[r] = -CUDART_INF_F;
        grow |= x[r] > rf[r] + (8.f + kWeightShift);
      }
      if (few_any(grow || !ok)) {
        if (few_any(!ok)) {
          ok = false;
          break;
        }
        // the rows whose scores outgrew their reference take the new largest one
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const int mx = __reduce_max_sync(0xffffffffu, float_order(x[r]));
          if (lane == (r & 31)) wred[warp * NR + r] = order_float(mx);
        }
        few_sync();
        if (tid < NR) {
          const float mx = fmaxf(fmaxf(wred[tid], wred[NR + tid]),
                                 fmaxf(wred[2 * NR + tid], wred[3 * NR + tid]));
          const float old = ref[tid];
          const bool up = mx > old + 8.f;
          fac[tid] = up ? exp2f(old - mx) : 1.f;
          if (up) ref[tid] = mx;
        }
        few_sync();
        float f[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          f[r] = fac[r];
          l[r] *= f[r];
          rf[r] = ref[r] - kWeightShift;
        }
        if (j > 0) {  // (SF of this step: the P . V before is done)
#pragma unroll
          for (int c = 0; c < NR; c += 16) {
            uint32_t o[16];
            tmem_ld16(lanes + NR + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              asm volatile("" : "+r"(o[e]));
              o[e] = __float_as_uint(__uint_as_float(o[e]) * f[c + e]);
            }
            tmem_st16(lanes + NR + c, o);
          }
          tmem_wait_st();
        }
      }
      // weights, their sums, and P^T
#pragma unroll
      for (int r = 0; r < NR; r += 2) {
        const float a = ex2_approx(x[r] - rf[r]), b = ex2_approx(x[r + 1] - rf[r + 1]);
        l[r] += a;
        l[r + 1] += b;
        const uint32_t h = FewT<T>::pack(a, b);
        uint8_t *const at0 = prow + r * 128 + (piece ^ ((r & 7) << 4)),
                      *const at1 = prow + (r + 1) * 128 + (piece ^ (((r + 1) & 7) << 4));
        *reinterpret_cast<uint16_t *>(at0) = (uint16_t)h;
        *reinterpret_cast<uint16_t *>(at1) = (uint16_t)(h >> 16);
        if constexpr (kSplitP) {
          const float2 g = FewT<T>::unpack(h);
          const uint32_t lo = FewT<T>::pack(a - g.x, b - g.y);
          *reinterpret_cast<uint16_t *>(at0 + 2 * NR * 128) = (uint16_t)lo;
          *reinterpret_cast<uint16_t *>(at1 + 2 * NR * 128) = (uint16_t)(lo >> 16);
          if constexpr (kParts == 3) {
            const float2 g2 = FewT<T>::unpack(lo);
            const uint32_t rest = FewT<T>::pack(a - g.x - g2.x, b - g.y - g2.y);
            *reinterpret_cast<uint16_t *>(at0 + 4 * NR * 128) = (uint16_t)rest;
            *reinterpret_cast<uint16_t *>(at1 + 4 * NR * 128) = (uint16_t)(rest >> 16);
          }
        }
      }
      if (L - key0 < kFewKeys) {
        // rows behind the sequence's end hold anything: their V becomes zero
        ok = __all_sync(0xffffffffu, few_wait(&bars[kFewVF], j & 1, fail));
        if (!in) {
#pragma unroll
          for (int c = 0; c < 16; ++c)
            *reinterpret_cast<uint4 *>(smem + Sm::kV + (c >> 3) * 16384 + tid * 128 + (c & 7) * 16) =
                make_uint4(0, 0, 0, 0);
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kFewPF]);
    }
    if (ok && nt > 0) {
      ok = few_wait(&bars[kFewOF], 0, fail);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
    }
    // ---- sums over the keys; O^T's lane is a channel, so a row leaves in lines ----
#pragma unroll
    for (int r = 0; r < NR; ++r) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
    }
    few_sync();  // (wred may still be read)
#pragma unroll
    for (int r = 0; r < NR; ++r)
      if (lane == (r & 31)) wred[warp * NR + r] = l[r];
    few_sync();
    if (tid < rows)
      ml_out[tid] = make_float2(
          ref[tid] - kWeightShift, (wred[tid] + wred[NR + tid]) + (wred[2 * NR + tid] + wred[3 * NR + tid]));
    float o[NR];
    __syncwarp();
    few_load<NR>(lanes + NR, o);
#pragma unroll
    for (int r = 0; r < NR; ++r)
      if (r < rows) o_out[(size_t)r * kFewD + tid] = nt > 0 ? o[r] : 0.f;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && *fail) few_set_err(p.err, kDevTimeout, slot, hk, tile0);  // (an earlier error stays)
  if (warp == 4) tmem_dealloc(tmem, kCols);
  if (p.follow) pdl_wait();  // (done only once that kernel is: the next one reads both)
}

template <typename T, int NR, bool kSplitP>
cudaError_t launch_few_t(const DenseDecodeParams &p, cudaStream_t st) {
  constexpr int kParts = kFewParts<T, kSplitP>;
  using Sm = FewSmem<NR, kParts>;
  auto k = dense_few_kernel<T, NR, kSplitP>;
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = allow_smem(k, Sm::kBytes, &ready);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, p.prefix_items, kFewThreads, (size_t)Sm::kBytes, st, p);
}

template <typename T, bool kSplitP>
cudaError_t launch_few_r(const DenseDecodeParams &p, cudaStream_t st) {
  return p.prefix_rows <= 16 ? launch_few_t<T, 16, kSplitP>(p, st)
                             : launch_few_t<T, 32, kSplitP>(p, st);
}

}  // namespace

cudaError_t launch_dense_few(const DenseDecodeParams &p, int dtype, cudaStream_t st) {
  const bool split = p.out_f32 != 0;
  if (dtype == 0) return split ? launch_few_r<__half, true>(p, st) : launch_few_r<__half, false>(p, st);
  return split ? launch_few_r<__nv_bfloat16, true>(p, st)
               : launch_few_r<__nv_bfloat16, false>(p, st);
}

}  // namespace spd
