// Decode attention of a batch over a shared prefix and over each sequence's
// own tokens in the paged cache: the split kernel for few query rows, and the
// kernel that joins all splits.
//
//   out_r = sum_t 2^(x_t - M) v_t / sum_t 2^(x_t - M),  t over prefix and own
//
// Split kernel: one CTA per work item, 16 query rows (a prefix's row group, or
// the G heads of one sequence padded) against a range of 16-key tiles.  Every
// warp takes every fourth tile through a TMA ring of its own (no CTA barrier
// in the loop), S = Q K^T and O += P V with mma.sync, online softmax in fp32.
// A decode step reads each own key once for G <= 8 rows, 2 G flops per byte:
// memory is the bound, and mma.sync's rate is far above it.  Weights are split
// into a 16-bit high part and the rounding of the rest (two products), so that
// the fp32 result keeps about 16 bits (bf16) or 22 (fp16) of each; fp32
// outputs of bf16 take a third part and keep 24.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include <type_traits>

#include "dense.h"
#include "dense_math.cuh"
#include "ptx.cuh"
#include "spd_internal.h"

namespace spd {
namespace {

constexpr uint32_t kDdWait = 1u << 22;
constexpr int kWarps = 4;

template <int D> struct DdSmem {
  static constexpr int kTileBytes = kDecodeTile * D * 2;  // K (or V) of a tile
  static constexpr int kStages = D == 128 ? 3 : 6;        // per warp: two CTAs fit an SM
  static constexpr int kRing = kWarps * kStages * 2 * kTileBytes;
  static constexpr int kMerge = kWarps * kDecodeRows * (D + 2) * 4;  // over the ring
  static constexpr int kBars = kRing;
  static constexpr int kBytes = kBars + kWarps * kStages * 8 + 1024;
  static_assert(kMerge <= kRing, "merge area");
};

__device__ __forceinline__ void dd_set_err(int *err, int code, int a, int b, int c) {
  if (atomicCAS(err, 0, code) == 0) {
    err[1] = a;
    err[2] = b;
    err[3] = c;
  }
}

template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
template <typename T> __device__ __forceinline__ float2 unpack2(uint32_t x);
template <> __device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t x) {
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
template <> __device__ __forceinline__ float2 unpack2<__half>(uint32_t x) {
  return __half22float2(*reinterpret_cast<const __half2 *>(&x));
}

// Where a row's splits lie: own partials first, then the prefix's.
struct RowSplits {
  const float2 *own_ml, *pre_ml;
  const float *own_o, *pre_o;
  size_t own_step, pre_step;  // rows between two splits
  int ns, nall;
};
__device__ __forceinline__ RowSplits row_splits(const DenseDecodeParams &p, int seq, int hk, int g,
                                                int D) {
  const DecodeSeq &s = p.seqs[seq];
  const int r = seq * p.G + g, tile = p.prefix_ns > 0 ? r / p.prefix_rows : 0;
  const size_t own = ((size_t)s.item_off + hk * s.ns) * p.G + g,
               pre = (size_t)(tile * p.Hkv + hk) * p.prefix_ns * p.prefix_rows +
                     (r - tile * p.prefix_rows);
  RowSplits x;
  x.own_ml = p.part_ml + own;
  x.own_o = p.part_o + own * D;
  x.pre_ml = p.pre_ml + pre;
  x.pre_o = p.pre_o + pre * D;
  x.own_step = p.G;
  x.pre_step = p.prefix_rows;
  x.ns = s.ns;
  x.nall = s.ns + p.prefix_ns;
  return x;
}
// One warp: the row's max (0 if nothing was met) and sum; factors to fac.
__device__ __forceinline__ float2 row_stats(const RowSplits &x, float *fac) {
  constexpr int kMax = kOwnMaxSplits + kDenseMaxSplits;
  const int lane = threadIdx.x & 31;
  float2 v[kMax / 32];
  float M = -CUDART_INF_F, L = 0.f;
#pragma unroll
  for (int j = 0; j < kMax / 32; ++j) {
    const int k = lane + 32 * j;
    v[j] = make_float2(-CUDART_INF_F, 0.f);
    if (32 * j < x.nall && k < x.nall)
      v[j] = __ldcg(k < x.ns ? x.own_ml + k * x.own_step : x.pre_ml + (k - x.ns) * x.pre_step);
    M = fmaxf(M, v[j].x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float base = M == -CUDART_INF_F ? 0.f : M;
#pragma unroll
  for (int j = 0; j < kMax / 32; ++j) {
    if (32 * j >= x.nall) break;
    const int k = lane + 32 * j;
    const float f = exp2f(v[j].x - base);
    if (fac && k < x.nall) fac[k] = f;
    L = fmaf(v[j].y, f, L);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  return make_float2(base, L);
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32, 2)
    dense_decode_kernel(const __grid_constant__ DenseDecodeParams p) {
  using Sm = DdSmem<D>;
  constexpr bool kBf = std::is_same<T, __nv_bfloat16>::value;
  constexpr int KB = D / 64, NT = D / 8;
  extern __shared__ uint8_t dd_smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(dd_smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g8 = lane >> 2, t4 = lane & 3;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Sm::kBars) + warp * Sm::kStages;
  uint8_t *ring = smem + warp * Sm::kStages * 2 * Sm::kTileBytes;

  // ---- the item: rows, the cache slot it reads, its tiles ----
  int item = blockIdx.x, hk, slot, L, tile0, tile1, row0, rows;
  int seq = 0;  // own items
  const bool pre = item < p.prefix_items;
  float2 *ml_out;
  float *o_out;
  if (pre) {
    const int unit = item / p.prefix_ns, split = item % p.prefix_ns;
    hk = unit % p.Hkv;
    row0 = (unit / p.Hkv) * kDecodeRows;
    rows = min(kDecodeRows, p.n * p.G - row0);
    slot = p.prefix_slot;
    L = p.prefix_len;
    tile0 = split * p.prefix_tpi;
    tile1 = tile0 + p.prefix_tpi;
    const size_t at = (size_t)item * kDecodeRows;
    ml_out = p.pre_ml + at;
    o_out = p.pre_o + at * D;
  } else {
    item -= p.prefix_items;
    int lo = 0, hi = p.n - 1;  // the last sequence whose items start at or before this one
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.seqs[mid].item_off <= item) lo = mid;
      else hi = mid - 1;
    }
    seq = lo;
    const DecodeSeq &s = p.seqs[seq];
    const int local = item - s.item_off;
    hk = local / s.ns;
    tile0 = (local % s.ns) * s.tpi;
    tile1 = tile0 + s.tpi;
    slot = s.slot;
    L = s.L;
    row0 = seq * p.G;
    rows = p.G;
    const size_t at = (size_t)item * p.G;
    ml_out = p.part_ml + at;
    o_out = p.part_o + at * D;
  }
  tile1 = min(tile1, (L + kDecodeTile - 1) / kDecodeTile);

  if (lane == 0) {
    for (int s = 0; s < Sm::kStages; ++s) mbar_init(&bars[s], 1);
    fence_mbar_init();
  }
  __syncwarp();
  // behind another kernel of this call nothing is waited for: that kernel started
  // its dependents after its own wait, so all that is read here is there, and
  // the two write to different places
  if (!p.follow) pdl_wait();
  pdl_launch_dependents();

  const int *table = p.page_table + (size_t)slot * p.max_pp;
  // tiles from the newest to the oldest (a distance bias then finds its largest
  // scores first, and the running max hardly moves): the warp's i-th is
  // first - 4 i
  const int first = tile1 - 1 - warp, ntile = first >= tile0 ? (first - tile0) / kWarps + 1 : 0;
  int issued = 0;
  bool ok = true;
  auto issue = [&](int i) {  // lane 0: the warp's i-th tile into its stage
    const int t = (first - i * kWarps) * kDecodeTile, blk = t / p.P;
    const int phys = blk < p.max_pp ? table[blk] : -1;
    if (phys < 0 || phys >= p.num_phys) {
      dd_set_err(p.err, blk < p.max_pp ? kDevBadPhys : kDevBadPage, slot, blk, phys);
      return false;
    }
    const int s = i % Sm::kStages;
    uint8_t *dst = ring + s * 2 * Sm::kTileBytes;
    mbar_arrive_expect_tx(&bars[s], 2 * Sm::kTileBytes);
    tma_load_4d(dst, &p.tm_k, 0, t % p.P, 0, phys * p.Hkv + hk, &bars[s]);
    tma_load_4d(dst + Sm::kTileBytes, &p.tm_v, 0, t % p.P, 0, phys * p.Hkv + hk, &bars[s]);
    return true;
  };
  for (; issued < min(ntile, Sm::kStages) && ok; ++issued)
    ok = __shfl_sync(0xffffffffu, lane == 0 ? (int)issue(issued) : 0, 0) != 0;
  if (!ok) --issued;  // (the tile that failed its check was not issued)

  // ---- Q fragments: rows g8 and g8 + 8 ----
  uint32_t qa[D / 16][4];
  float slope[2] = {0.f, 0.f};
  int pos[2] = {0, 0};
#pragma unroll
  for (int hrow = 0; hrow < 2; ++hrow) {
    const int r = g8 + 8 * hrow;
    const bool live = r < rows;
    const int gr = row0 + r, sq = gr / p.G, h = hk * p.G + gr % p.G;
    const uint32_t *q = reinterpret_cast<const uint32_t *>(static_cast<const T *>(p.q) +
                                                           ((size_t)sq * p.Hq + h) * D);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      qa[k][hrow] = live ? q[k * 8 + t4] : 0u;
      qa[k][2 + hrow] = live ? q[k * 8 + 4 + t4] : 0u;
    }
    if (live) {
      if (p.rule.slopes) slope[hrow] = p.rule.slopes[h] * 1.4426950408889634f;
      pos[hrow] = (pre ? L + p.seqs[sq].L : L) - 1;
    }
  }
  const bool upper = rows > 8;

  float o[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
  float m_run[2] = {-CUDART_INF_F, -CUDART_INF_F}, l_run[2] = {0.f, 0.f};
  const size_t l_stride = (size_t)(L + 3) & ~size_t(3);
  float *lg = !pre && p.logits
                  ? p.logits + (size_t)p.seqs[seq].l_off * p.Hkv * p.G + (size_t)hk * p.G * l_stride
                  : nullptr;

  for (int i = 0; i < ntile && ok; ++i) {
    const int s = i % Sm::kStages, t0 = (first - i * kWarps) * kDecodeTile;
    ok = __all_sync(0xffffffffu, mbar_wait(&bars[s], (i / Sm::kStages) & 1, kDdWait));
    if (!ok) {
      if (lane == 0) dd_set_err(p.err, kDevTimeout, slot, hk, t0);
      break;
    }
    uint8_t *kt = ring + s * 2 * Sm::kTileBytes, *vt = kt + Sm::kTileBytes;
    const int valid = L - t0;  // tokens of the tile
    if (valid < kDecodeTile) {
      // rows behind the sequence's end hold anything: their V becomes zero
      for (int c = lane; c < KB * kDecodeTile * 8; c += 32) {
        if (((c >> 3) & (kDecodeTile - 1)) >= valid)
          *reinterpret_cast<uint4 *>(vt + c * 16) = make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();  // (the stage is filled again later)
      __syncwarp();
    }
    // S = Q . K^T: 16 rows x 16 keys
    float sc[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[j][e] = 0.f;
    const uint32_t ka = smem_u32(kt), va = smem_u32(vt);
    const int krow = (lane & 7) + ((lane >> 4) & 1) * 8, kch = (lane >> 3) & 1;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      uint32_t b0, b1, b2, b3;
      const int ch = 2 * k + kch;
      ldmatrix_x4(ka + (ch >> 3) * 2048 + swz128(krow, ch & 7), b0, b1, b2, b3);
      mma_16816<kBf>(sc[0], qa[k], b0, b1);
      mma_16816<kBf>(sc[1], qa[k], b2, b3);
    }
    // scores in base 2, masked behind the end
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) {
      if (hr == 1 && !upper) break;
      if (p.rule.cap_out > 0.f) {
        if (p.precise) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            sc[j][2 * hr] = cap_any(p.rule, sc[j][2 * hr]);
            sc[j][2 * hr + 1] = cap_any(p.rule, sc[j][2 * hr + 1]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float2 x = cap_16bit(p.rule, make_float2(sc[j][2 * hr], sc[j][2 * hr + 1]));
            sc[j][2 * hr] = x.x;
            sc[j][2 * hr + 1] = x.y;
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          sc[j][2 * hr] *= p.rule.scale_log2;
          sc[j][2 * hr + 1] *= p.rule.scale_log2;
        }
      }
      if (p.rule.slopes) {
        const float far = (float)(pos[hr] - t0 - 2 * t4);  // distance of the lane's first key
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            sc[j][2 * hr + e] = fmaf(-slope[hr], far - (float)(8 * j + e), sc[j][2 * hr + e]);
      }
    }
    if (valid < kDecodeTile) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (8 * j + 2 * t4 + (e & 1) >= valid) sc[j][e] = -CUDART_INF_F;
    }
    if (lg) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int key = 8 * j + 2 * t4 + e;
          if (g8 < rows && key < valid) lg[(size_t)g8 * l_stride + t0 + key] = sc[j][e];
        }
    }
    // running max, moved only when it grows by more than 2^8
    bool grow = false;
    float mx[2];
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) {
      if (hr == 1 && !upper) break;
      float m = fmaxf(fmaxf(sc[0][2 * hr], sc[0][2 * hr + 1]),
                      fmaxf(sc[1][2 * hr], sc[1][2 * hr + 1]));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      mx[hr] = m;
      grow = grow || m > m_run[hr] + 8.f;
    }
    if (__any_sync(0xffffffffu, grow)) {
      float al[2] = {1.f, 1.f};
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
        if (hr == 1 && !upper) break;
        if (mx[hr] > m_run[hr] + 8.f) {
          al[hr] = m_run[hr] == -CUDART_INF_F ? 0.f : exp2f(m_run[hr] - mx[hr]);
          m_run[hr] = mx[hr];
          l_run[hr] *= al[hr];
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        o[n][0] *= al[0];
        o[n][1] *= al[0];
        o[n][2] *= al[1];
        o[n][3] *= al[1];
      }
    }
    uint32_t ph[4] = {0, 0, 0, 0}, pl[4] = {0, 0, 0, 0}, px[4] = {0, 0, 0, 0};
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) {
      if (hr == 1 && !upper) break;
      const float base = m_run[hr] == -CUDART_INF_F ? 0.f : m_run[hr] - kWeightShift;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float a = ex2_approx(sc[j][2 * hr] - base), b = ex2_approx(sc[j][2 * hr + 1] - base);
        l_run[hr] += a + b;
        const uint32_t h = pack2<T>(a, b);
        const float2 f = unpack2<T>(h);
        ph[2 * j + hr] = h;
        const uint32_t lo = pack2<T>(a - f.x, b - f.y);
        pl[2 * j + hr] = lo;
        if (kBf) {
          const float2 f2 = unpack2<T>(lo);
          px[2 * j + hr] = pack2<T>(a - f.x - f2.x, b - f.y - f2.y);
        }
      }
    }
    // O += P . V
    const int vrow = lane & 15, vch = lane >> 4;
#pragma unroll
    for (int n = 0; n < NT; n += 2) {
      uint32_t b0, b1, b2, b3;
      const int ch = n + vch;
      ldmatrix_x4_trans(va + (ch >> 3) * 2048 + swz128(vrow, ch & 7), b0, b1, b2, b3);
      mma_16816<kBf>(o[n], ph, b0, b1);
      mma_16816<kBf>(o[n], pl, b0, b1);
      mma_16816<kBf>(o[n + 1], ph, b2, b3);
      mma_16816<kBf>(o[n + 1], pl, b2, b3);
      if (kBf && p.out_f32) {
        mma_16816<kBf>(o[n], px, b0, b1);
        mma_16816<kBf>(o[n + 1], px, b2, b3);
      }
    }
    __syncwarp();
    if (issued < ntile) {
      ok = __shfl_sync(0xffffffffu, lane == 0 ? (int)issue(issued) : 0, 0) != 0;
      issued += ok;
    }
  }
  if (!ok) {  // copies in flight land before the shared memory is used again
    for (int i = max(0, issued - Sm::kStages); i < issued; ++i)
      mbar_wait(&bars[i % Sm::kStages], (i / Sm::kStages) & 1, kDdWait);
  }
  // ---- the four warps' sums over the same rows ----
#pragma unroll
  for (int hr = 0; hr < 2; ++hr) {
    l_run[hr] += __shfl_xor_sync(0xffffffffu, l_run[hr], 1);
    l_run[hr] += __shfl_xor_sync(0xffffffffu, l_run[hr], 2);
  }
  __syncthreads();
  float *mo = reinterpret_cast<float *>(smem);                  // [warp][16][D]
  float *mm = mo + kWarps * kDecodeRows * D;                    // [warp][16] max, then sums
  float *msum = mm + kWarps * kDecodeRows;
#pragma unroll
  for (int hr = 0; hr < 2; ++hr) {
    const int r = g8 + 8 * hr;
    float *dst = mo + (size_t)(warp * kDecodeRows + r) * D;
#pragma unroll
    for (int n = 0; n < NT; ++n)
      *reinterpret_cast<float2 *>(dst + 8 * n + 2 * t4) =
          make_float2(o[n][2 * hr], o[n][2 * hr + 1]);
    if (t4 == 0) {
      mm[warp * kDecodeRows + r] = m_run[hr];
      msum[warp * kDecodeRows + r] = l_run[hr];
    }
  }
  __syncthreads();
  for (int x = tid; x < rows * (D / 4); x += kWarps * 32) {
    const int r = x / (D / 4), c = (x % (D / 4)) * 4;
    float M = -CUDART_INF_F;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, mm[w * kDecodeRows + r]);
    const float base = M == -CUDART_INF_F ? 0.f : M;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = exp2f(mm[w * kDecodeRows + r] - base);
      const float4 v = *reinterpret_cast<const float4 *>(mo + (size_t)(w * kDecodeRows + r) * D + c);
      acc.x = fmaf(v.x, f, acc.x);
      acc.y = fmaf(v.y, f, acc.y);
      acc.z = fmaf(v.z, f, acc.z);
      acc.w = fmaf(v.w, f, acc.w);
      l = fmaf(msum[w * kDecodeRows + r], f, l);
    }
    *reinterpret_cast<float4 *>(o_out + (size_t)r * D + c) = acc;
    if (c == 0) ml_out[r] = make_float2(M - kWeightShift, l);
  }
  if (p.follow) pdl_wait();  // (done only once that kernel is: the next one reads both)
  if (!p.tickets) return;
  // ---- the last of a (sequence, kv head)'s items joins its splits: a warp per
  // query head ----
  __shared__ int mine[kDecodeRows];
  float *fac = reinterpret_cast<float *>(smem) + warp * (kOwnMaxSplits + kDenseMaxSplits);
  __threadfence();
  __syncthreads();  // (and the merge area has been read)
  const int first_seq = row0 / p.G, seqs = (rows + p.G - 1) / p.G;
  if (tid < seqs) {
    const int sq = first_seq + tid, need = p.seqs[sq].ns + p.prefix_ns;
    int *ticket = p.tickets + sq * p.Hkv + hk;
    const bool last = atom_add_acq_rel_gpu(ticket, 1) == need - 1;
    if (last) *ticket = 0;  // as it was found
    mine[tid] = last;
  }
  __syncthreads();
  for (int i = 0; i < seqs; ++i) {
    if (!mine[i]) continue;
    for (int g = warp; g < p.G; g += kWarps) {
      const RowSplits x = row_splits(p, first_seq + i, hk, g, D);
      __syncwarp();
      const float2 st = row_stats(x, fac);
      __syncwarp();
      constexpr int E = D / 32;
      float acc[E];
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = 0.f;
      auto add = [&](const float *src, float f) {
        if constexpr (E == 4) {
          const float4 v = __ldcg(reinterpret_cast<const float4 *>(src) + lane);
          acc[0] = fmaf(v.x, f, acc[0]);
          acc[1] = fmaf(v.y, f, acc[1]);
          acc[2] = fmaf(v.z, f, acc[2]);
          acc[3] = fmaf(v.w, f, acc[3]);
        } else {
          const float2 v = __ldcg(reinterpret_cast<const float2 *>(src) + lane);
          acc[0] = fmaf(v.x, f, acc[0]);
          acc[1] = fmaf(v.y, f, acc[1]);
        }
      };
#pragma unroll 8
      for (int k = 0; k < x.ns; ++k) add(x.own_o + k * x.own_step * D, fac[k]);
#pragma unroll 8
      for (int k = 0; k < x.nall - x.ns; ++k) add(x.pre_o + k * x.pre_step * D, fac[x.ns + k]);
      const float inv = 1.f / st.y;
      const size_t at = ((size_t)(first_seq + i) * p.Hq + hk * p.G + g) * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        if (p.out_f32)
          *reinterpret_cast<float2 *>(static_cast<float *>(p.out) + at + e) =
              make_float2(acc[e] * inv, acc[e + 1] * inv);
        else
          *reinterpret_cast<uint32_t *>(static_cast<T *>(p.out) + at + e) =
              pack2<T>(acc[e] * inv, acc[e + 1] * inv);
      }
    }
  }
}

// ---- joining prefix and own splits ------------------------------------------------
// CTAs [0, n Hq): the output of one (sequence, query head), its splits shared
// out over the CTA's groups of D / 4 threads.  The rest, when asked for: the
// weights of 1,024 own tokens of one (sequence, kv head),
// w_out = w_in + sum over the head's G queries of 2^(x - M) / L.
constexpr int kCombineThreads = 128, kWeightTokens = 1024;

template <typename T, int D>
__global__ void __launch_bounds__(kCombineThreads)
    dense_decode_combine_kernel(const __grid_constant__ DenseDecodeParams p) {
  constexpr int kCols = D / 4, kGroups = kCombineThreads / kCols;
  __shared__ float fac[kOwnMaxSplits + kDenseMaxSplits];
  __shared__ float2 stat[8];
  __shared__ float4 part[kGroups][kCols];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if ((int)blockIdx.x < p.n * p.Hq) {
    const int seq = blockIdx.x / p.Hq, h = blockIdx.x % p.Hq;
    const RowSplits x = row_splits(p, seq, h / p.G, h % p.G, D);
    if (warp == 0) {
      const float2 st = row_stats(x, fac);
      if (lane == 0) stat[0] = st;
    }
    __syncthreads();
    const int grp = tid / kCols, c = (tid % kCols) * 4;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float *src, float f) {
      const float4 v = __ldcs(reinterpret_cast<const float4 *>(src));
      acc.x = fmaf(v.x, f, acc.x);
      acc.y = fmaf(v.y, f, acc.y);
      acc.z = fmaf(v.z, f, acc.z);
      acc.w = fmaf(v.w, f, acc.w);
    };
    const float *own = x.own_o + c, *pre = x.pre_o + c;
#pragma unroll 4
    for (int k = grp; k < x.ns; k += kGroups) add(own + k * x.own_step * D, fac[k]);
#pragma unroll 8
    for (int k = grp; k < x.nall - x.ns; k += kGroups)
      add(pre + k * x.pre_step * D, fac[x.ns + k]);
    part[grp][tid % kCols] = acc;
    __syncthreads();
    if (grp == 0) {
#pragma unroll
      for (int j = 1; j < kGroups; ++j) {
        const float4 v = part[j][tid];
        acc.x += v.x;
        acc.y += v.y;
        acc.z += v.z;
        acc.w += v.w;
      }
      const float inv = 1.f / stat[0].y;
      const size_t at = ((size_t)seq * p.Hq + h) * D + c;
      if (p.out_f32)
        *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) =
            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
      else
        *reinterpret_cast<uint2 *>(static_cast<T *>(p.out) + at) =
            make_uint2(pack2<T>(acc.x * inv, acc.y * inv), pack2<T>(acc.z * inv, acc.w * inv));
    }
  } else {
    const int b = blockIdx.x - p.n * p.Hq, chunk = b % p.w_chunks, unit = b / p.w_chunks;
    const int seq = unit / p.Hkv, hk = unit % p.Hkv, L = p.seqs[seq].L;
    if (chunk * kWeightTokens >= L) return;
    for (int g = warp; g < p.G; g += kCombineThreads / 32) {
      const float2 st = row_stats(row_splits(p, seq, hk, g, D), nullptr);
      if (lane == 0) stat[g] = make_float2(st.x, 1.f / st.y);
    }
    __syncthreads();
    const size_t row = (size_t)unit;
    const size_t l_stride = (size_t)(L + 3) & ~size_t(3);
    const float *lg = p.logits + (size_t)p.seqs[seq].l_off * p.Hkv * p.G + (size_t)hk * p.G * l_stride;
    const int t1 = min(L, (chunk + 1) * kWeightTokens);
#pragma unroll 2
    for (int t = chunk * kWeightTokens + tid; t < t1; t += kCombineThreads) {
      float w = 0.f;
      for (int g = 0; g < p.G; ++g)
        w = fmaf(ex2_approx(lg[g * l_stride + t] - stat[g].x), stat[g].y, w);
      p.w_out[row * p.w_stride + t] = (p.w_in ? p.w_in[row * p.w_stride + t] : 0.f) + w;
    }
  }
}

template <typename T, int D>
cudaError_t launch_dd(const DenseDecodeParams &p, cudaStream_t st) {
  auto k = dense_decode_kernel<T, D>;
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = allow_smem(k, DdSmem<D>::kBytes, &ready);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, p.prefix_items + p.own_items, kWarps * 32, (size_t)DdSmem<D>::kBytes, st, p);
}

}  // namespace

cudaError_t launch_dense_decode(const DenseDecodeParams &p, int dtype, int d, cudaStream_t st) {
  if (dtype == 0) return d == 64 ? launch_dd<__half, 64>(p, st) : launch_dd<__half, 128>(p, st);
  return d == 64 ? launch_dd<__nv_bfloat16, 64>(p, st) : launch_dd<__nv_bfloat16, 128>(p, st);
}

cudaError_t launch_dense_decode_combine(const DenseDecodeParams &p, int dtype, int d,
                                        cudaStream_t st) {
  const int grid = p.n * (p.Hq + (p.w_out ? p.Hkv * p.w_chunks : 0));
  auto go = [&](auto kernel) { return launch_pdl(kernel, grid, kCombineThreads, 0, st, p); };
  if (dtype == 0)
    return d == 64 ? go(dense_decode_combine_kernel<__half, 64>)
                   : go(dense_decode_combine_kernel<__half, 128>);
  return d == 64 ? go(dense_decode_combine_kernel<__nv_bfloat16, 64>)
                 : go(dense_decode_combine_kernel<__nv_bfloat16, 128>);
}

}  // namespace spd
