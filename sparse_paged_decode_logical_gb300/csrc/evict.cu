// Eviction from the paged cache by accumulated attention weight: every kv head
// of a sequence keeps its newest tokens and the best of the others, compacted
// in order into another sequence together with their page metadata.
//
//   room = m - newest,  m = min(keep, L),  newest = min(recent, m)
//   kept = { t >= L - newest } + the `room` tokens t < L - newest of the
//          greatest weight, ties to the lower position
//
// Two kernels.  evict_select: one cluster per (sequence, kv head); each CTA
// holds its stretch of the weights in shared memory as order-preserving
// integers, and three rounds of an 11-, 11- and 10-bit radix histogram, summed
// over the cluster through distributed shared memory, give the exact value of
// the room-th greatest key; a prefix count then gives every kept token its
// place.  The weights are read once.  evict_copy: one CTA per 64 kept rows
// gathers K and V rows (memory is the bound: each kept row read and written
// once) and takes the metadata's min and max from the rows that it holds.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include "dense.h"
#include "ptx.cuh"
#include "spd_internal.h"

namespace spd {
namespace {

constexpr int kSelThreads = 512;
constexpr int kBins = 2048;
constexpr int kCacheKeys = 48 * 1024;  // keys a CTA holds; longer stretches are read again

__device__ __forceinline__ void ev_set_err(int *err, int code, int a, int b, int c) {
  if (atomicCAS(err, 0, code) == 0) {
    err[1] = a;
    err[2] = b;
    err[3] = c;
  }
}

// Order-preserving integer of a weight; NaN counts as the greatest, -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (isnan(w)) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ uint32_t ld_dsmem_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_dsmem_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Exclusive sums of the warps' two counts and their totals (one entry per warp
// in `tmp`, written by the callers' lane 0 before a barrier).
__device__ __forceinline__ void warp_prefix(const uint2 *tmp, uint2 *before, uint2 *all) {
  const int warp = threadIdx.x >> 5;
  uint2 b = make_uint2(0, 0), t = make_uint2(0, 0);
#pragma unroll
  for (int w = 0; w < kSelThreads / 32; ++w) {
    const uint2 x = tmp[w];
    if (w < warp) {
      b.x += x.x;
      b.y += x.y;
    }
    t.x += x.x;
    t.y += x.y;
  }
  *before = b;
  *all = t;
}

// One key into the histogram.  Many tokens share one weight (0 above all): keys
// that fall into the first active lane's bin are counted at once when they are
// more than a few.
__device__ __forceinline__ void count_bin(uint32_t *hist, bool in, uint32_t bin) {
  const uint32_t act = __ballot_sync(0xffffffffu, in);
  if (!act) return;
  const int lead = __ffs(act) - 1;
  const uint32_t lbin = __shfl_sync(0xffffffffu, bin, lead);
  const uint32_t same = __ballot_sync(0xffffffffu, in && bin == lbin);
  if (__popc(same) > 4) {
    if ((int)(threadIdx.x & 31) == lead) atomicAdd(&hist[lbin], __popc(same));
    in = in && bin != lbin;
  }
  if (in) atomicAdd(&hist[bin], 1u);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(
    const __grid_constant__ EvictParams p) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ uint32_t hist[kBins], tot[kBins];
  __shared__ uint2 tmp[kSelThreads / 32];
  __shared__ uint32_t counts[2];       // greater than, equal to the cut in this stretch
  __shared__ uint32_t found[2];        // the round's bin, keys above it
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cs = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
  const int unit = blockIdx.x / cs, seq = unit / p.Hkv;
  for (int b = tid; b < kBins; b += kSelThreads) hist[b] = 0;
  pdl_wait();
  pdl_launch_dependents();
  const EvictSeq s = p.seqs[seq];
  const int newest = min(p.recent, s.m), n_old = s.L - newest, room = s.m - newest;
  const float *w = p.weights + (size_t)unit * p.w_stride;
  int *kept = p.kept + (size_t)unit * p.keep;
  float *kw = p.kept_weights ? p.kept_weights + (size_t)unit * p.keep : nullptr;
  // the newest tokens and what lies behind the kept ones
  for (int i = room + rank * kSelThreads + tid; i < p.keep; i += cs * kSelThreads) {
    const int t = i < s.m ? n_old + (i - room) : -1;
    kept[i] = t;
    if (kw) kw[i] = t >= 0 ? w[t] : 0.f;
  }
  if (room >= n_old) {  // (the same for the whole cluster) everything is kept
    for (int i = rank * kSelThreads + tid; i < n_old; i += cs * kSelThreads) {
      kept[i] = i;
      if (kw) kw[i] = w[i];
    }
    return;
  }
  if (room == 0) return;
  const int seg = ((n_old + cs - 1) / cs + 3) & ~3;
  const int s0 = min(rank * seg, n_old), len = min(seg, n_old - s0);
  const float *ws = w + s0;
  auto key = [&](int i) { return i < kCacheKeys ? keys[i] : weight_key(ws[i]); };
  // four consecutive keys, i a multiple of 4 (behind the end: 0, which no key
  // is: the least, -inf, is 0x007fffff)
  auto keys4 = [&](int i, int end, uint32_t (&k)[4]) {
    if (i + 3 < min(end, kCacheKeys)) {
      const uint4 x = *reinterpret_cast<const uint4 *>(&keys[i]);
      k[0] = x.x;
      k[1] = x.y;
      k[2] = x.z;
      k[3] = x.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) k[j] = i + j < end ? key(i + j) : 0u;
    }
  };
  __syncthreads();
  // ---- the stretch into shared memory, counted by the leading 11 bits ----
  constexpr int kUnroll = 8;
  for (int i0 = 0; i0 < len; i0 += kSelThreads * kUnroll) {
    float x[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const int i = i0 + j * kSelThreads + tid;
      x[j] = i < len ? __ldg(ws + i) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const int i = i0 + j * kSelThreads + tid;
      if (i0 + j * kSelThreads >= len) break;  // (the same for the block)
      const uint32_t k = weight_key(x[j]);
      if (i < min(len, kCacheKeys)) keys[i] = k;
      count_bin(hist, i < len, k >> 21);
    }
  }

  uint32_t prefix = 0, need = (uint32_t)room;  // the cut's leading bits; its rank among them
  for (int round = 0; round < 3; ++round) {
    const int shift = round == 0 ? 21 : round == 1 ? 10 : 0, bits = round == 2 ? 10 : 11;
    if (round > 0) {
      for (int b = tid; b < kBins; b += kSelThreads) hist[b] = 0;
      __syncthreads();
#pragma unroll 2
      for (int i0 = 0; i0 < len; i0 += 4 * kSelThreads) {
        uint32_t k[4];
        keys4(i0 + 4 * tid, len, k);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // (0, behind the end, is of no key: it may only be counted where
          // the cut's leading bits are 0 themselves)
          const bool in = (k[j] >> (shift + bits)) == prefix && k[j] != 0;
          const uint32_t bin = (k[j] >> shift) & ((1u << bits) - 1);
          if (__popc(__ballot_sync(0xffffffffu, in)) > 8) count_bin(hist, in, bin);
          else if (in) atomicAdd(&hist[bin], 1u);
        }
      }
    }
    cluster_sync();  // every CTA's histogram is complete
    const int per = (kBins + cs - 1) / cs;
    for (int b = rank * per + tid; b < min(kBins, (rank + 1) * per); b += kSelThreads) {
      const uint32_t at = smem_u32(&hist[b]), to = smem_u32(&tot[b]);
      uint32_t sum = 0;
      for (int r = 0; r < cs; ++r) sum += ld_dsmem_u32(map_rank(at, r));
      for (int r = 0; r < cs; ++r) st_dsmem_u32(map_rank(to, r), sum);
    }
    cluster_sync();  // the sums are everywhere
    // the bin that holds the need-th greatest key: bins in descending order,
    // four per thread
    static_assert(kBins == kSelThreads * 4, "four bins per thread");
    uint32_t c[4], mine = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) mine += c[j] = tot[kBins - 1 - (tid * 4 + j)];
    uint32_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) tmp[warp] = make_uint2(inc, 0);
    __syncthreads();
    uint2 before, all;
    warp_prefix(tmp, &before, &all);
    inc += before.x;
    uint32_t above = inc - mine;
    if (above < need && need <= inc) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (above < need && need <= above + c[j]) {
          found[0] = kBins - 1 - (tid * 4 + j);
          found[1] = above;
          break;
        }
        above += c[j];
      }
    }
    __syncthreads();
    prefix = (prefix << bits) | found[0];
    need -= found[1];
  }
  // prefix is the cut itself: greater keys all stay, of the equal ones the
  // first `need`.  Every warp counts, then places, a stretch of its own.
  const int wlen = ((len + kSelThreads / 32 - 1) / (kSelThreads / 32) + 127) & ~127;
  const int w0 = min(warp * wlen, len), w1 = min(w0 + wlen, len);
  uint2 cnt = make_uint2(0, 0);
#pragma unroll 2
  for (int i = w0 + 4 * lane; i < w1; i += 128) {
    uint32_t k[4];
    keys4(i, w1, k);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      cnt.x += k[j] > prefix;
      cnt.y += k[j] == prefix;
    }
  }
  cnt.x = __reduce_add_sync(0xffffffffu, cnt.x);
  cnt.y = __reduce_add_sync(0xffffffffu, cnt.y);
  if (lane == 0) tmp[warp] = cnt;
  __syncthreads();
  uint2 before, total;
  warp_prefix(tmp, &before, &total);
  if (tid == 0) {
    counts[0] = total.x;
    counts[1] = total.y;
  }
  cluster_sync();
  uint32_t gt = before.x, eq = before.y;  // before this warp's stretch
  for (int r = 0; r < rank; ++r) {
    gt += ld_dsmem_u32(map_rank(smem_u32(&counts[0]), r));
    eq += ld_dsmem_u32(map_rank(smem_u32(&counts[1]), r));
  }
  cluster_arrive_release();  // the counts have been read: a CTA may leave
#pragma unroll 1
  for (int i0 = w0; i0 < w1; i0 += 128) {
    const int i = i0 + 4 * lane;
    uint32_t k[4], v = 0;  // (counts of up to 128: both in one word)
    keys4(i, w1, k);
#pragma unroll
    for (int j = 0; j < 4; ++j) v += (k[j] > prefix ? 1u : 0u) + (k[j] == prefix ? 0x10000u : 0u);
    if (!__any_sync(0xffffffffu, v != 0)) continue;
    uint32_t inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    uint32_t g = gt + ((inc - v) & 0xffffu), e = eq + ((inc - v) >> 16);
    float x[4];  // (all four on their way before the first is stored)
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = kw && k[j] >= prefix ? __ldg(ws + i + j) : 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool more = k[j] > prefix, tie = k[j] == prefix;
      if (more || (tie && e < need)) {
        const uint32_t at = g + min(e, need);
        kept[at] = s0 + i + j;
        if (kw) kw[at] = x[j];
      }
      g += more;
      e += tie;
    }
    const uint32_t all = __shfl_sync(0xffffffffu, inc, 31);
    gt += all & 0xffffu;
    eq += all >> 16;
  }
  __syncwarp();
  cluster_wait();
}

// ---- gather + metadata ---------------------------------------------------------
constexpr int kCopyRows = 64, kCopyThreads = 256;

// Order of two stored elements: fp8 codes by sign and magnitude.
struct F8 {
  uint8_t v;
};
template <typename T> __device__ __forceinline__ float elem_key(T x) { return (float)x; }
template <> __device__ __forceinline__ float elem_key<F8>(F8 x) { return (float)e4m3_key(x.v); }

// Two elements at once, and what no element is above or below.
template <typename T> struct Pair;
template <> struct Pair<__half> {
  using type = __half2;
  static __device__ __forceinline__ __half2 limit(bool low) {
    return __half2half2(__ushort_as_half(low ? 0xfc00 : 0x7c00));
  }
};
template <> struct Pair<__nv_bfloat16> {
  using type = __nv_bfloat162;
  static __device__ __forceinline__ __nv_bfloat162 limit(bool low) {
    return __bfloat162bfloat162(__ushort_as_bfloat16(low ? 0xff80 : 0x7f80));
  }
};
template <> struct Pair<F8> {
  using type = F8;
};

template <typename T, int D>
__global__ void __launch_bounds__(kCopyThreads, 5) evict_copy_kernel(
    const __grid_constant__ EvictParams p) {
  constexpr int kLanes = D * (int)sizeof(T) / 16;       // threads of one row
  constexpr int kStep = kCopyThreads / kLanes;          // rows at once
  constexpr int kIter = kCopyRows / kStep;
  __shared__ uint4 krows[kCopyRows * kLanes];
  __shared__ __align__(16) T ends[kCopyRows / 16][2][D];
  const int tid = threadIdx.x, groups = (p.keep + kCopyRows - 1) / kCopyRows;
  const int unit = blockIdx.x / groups, r0 = blockIdx.x % groups * kCopyRows;
  const int seq = unit / p.Hkv, hk = unit % p.Hkv;
  pdl_wait();
  pdl_launch_dependents();
  const EvictSeq s = p.seqs[seq];
  if (r0 >= s.m) return;
  const int n = min(kCopyRows, s.m - r0);
  const int *kept = p.kept + (size_t)unit * p.keep + r0;
  const int *src_pages = p.page_table + (size_t)s.src * p.max_pp;
  const int *dst_pages = p.page_table + (size_t)s.dst * p.max_pp;
  const uint4 *kp = static_cast<const uint4 *>(p.k_pool), *vp = static_cast<const uint4 *>(p.v_pool);
  uint4 *ko = static_cast<uint4 *>(p.k_pool), *vo = static_cast<uint4 *>(p.v_pool);
  const int lane = tid % kLanes, sub = tid / kLanes;
  // row t of a page list, or the largest value if the check fails
  constexpr uint32_t kNone = 0xffffffffu;
  auto row_at = [&](const int *pages, int t, int slot) -> uint32_t {
    const int blk = p.P_log2 >= 0 ? t >> p.P_log2 : t / p.P;
    const int phys = t >= 0 && blk < p.max_pp ? pages[blk] : -1;
    if (phys < 0 || phys >= p.num_phys) {
      ev_set_err(p.err, kDevBadPhys, slot, t, phys);
      return kNone;
    }
    return (uint32_t)(phys * p.Hkv + hk) * (uint32_t)p.P + (uint32_t)(t - blk * p.P);
  };
  uint32_t from[kIter], to[kIter];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int r = i * kStep + sub;
    from[i] = to[i] = kNone;
    if (r < n) {
      const int t = kept[r];
      from[i] = t < s.L ? row_at(src_pages, t, s.src) : kNone;
      to[i] = from[i] == kNone ? kNone : row_at(dst_pages, r0 + r, s.dst);
    }
  }
  uint4 kx[kIter], vx[kIter];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const bool in = to[i] != kNone;
    const size_t at = (size_t)from[i] * kLanes + lane;
    kx[i] = in ? __ldcs(kp + at) : make_uint4(0, 0, 0, 0);
    vx[i] = in ? __ldcs(vp + at) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    if (to[i] != kNone) {
      const size_t at = (size_t)to[i] * kLanes + lane;
      ko[at] = kx[i];
      vo[at] = vx[i];
    }
  }
  // metadata of the logical pages that begin in these rows (64 rows hold whole
  // ones): least and greatest of each channel per 16 rows, then per page
  T *meta = static_cast<T *>(p.meta);
  const int parts = (n + 15) / 16;
  if constexpr (sizeof(T) == 2) {
    // rows of a warp first, in registers, then the warps that share a part
    using T2 = typename Pair<T>::type;
    constexpr int kWarpRows = 32 / kLanes, kPerPart = 16 / kWarpRows;  // warps per 16 rows
    const T2 top = Pair<T>::limit(false), bottom = Pair<T>::limit(true);
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int r = i * kStep + sub;
      T2 lo[4], hi[4];
      const T2 *x = reinterpret_cast<const T2 *>(&kx[i]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        lo[e] = r < n ? x[e] : top;
        hi[e] = r < n ? x[e] : bottom;
#pragma unroll
        for (int o = kLanes; o < 32; o <<= 1) {
          lo[e] = __hmin2(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], o));
          hi[e] = __hmax2(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], o));
        }
      }
      if ((tid & 31) < kLanes) {
        uint4 *to = krows + ((i * (kCopyThreads / 32) + (tid >> 5)) * 2) * kLanes + lane;
        to[0] = *reinterpret_cast<const uint4 *>(lo);
        to[kLanes] = *reinterpret_cast<const uint4 *>(hi);
      }
    }
    __syncthreads();
    // entry w of krows: rows w kWarpRows ..; part j: entries j kPerPart ..
    for (int x = tid; x < parts * 2 * kLanes; x += kCopyThreads) {
      const int j = x / (2 * kLanes), which = x / kLanes & 1, ln = x % kLanes;
      uint4 v = krows[(j * kPerPart * 2 + which) * kLanes + ln];
      T2 *m = reinterpret_cast<T2 *>(&v);
#pragma unroll
      for (int w = 1; w < kPerPart; ++w) {
        const uint4 y = krows[((j * kPerPart + w) * 2 + which) * kLanes + ln];
        const T2 *ym = reinterpret_cast<const T2 *>(&y);
#pragma unroll
        for (int e = 0; e < 4; ++e) m[e] = which ? __hmax2(m[e], ym[e]) : __hmin2(m[e], ym[e]);
      }
      *reinterpret_cast<uint4 *>(&ends[j][which][ln * 8]) = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kIter; ++i) krows[(i * kStep + sub) * kLanes + lane] = kx[i];
    __syncthreads();
    const T *rows = reinterpret_cast<const T *>(krows);
    for (int x = tid; x < parts * D; x += kCopyThreads) {
      const int j = x / D, c = x % D, m = min(16, n - 16 * j);
      T lo = rows[16 * j * D + c], hi = lo;
      float flo = elem_key(lo), fhi = flo;
      for (int r = 1; r < m; ++r) {
        const T e = rows[(16 * j + r) * D + c];
        const float f = elem_key(e);
        if (f < flo) {
          flo = f;
          lo = e;
        }
        if (f > fhi) {
          fhi = f;
          hi = e;
        }
      }
      ends[j][0][c] = lo;
      ends[j][1][c] = hi;
    }
  }
  __syncthreads();
  const int pages = (n + p.ell - 1) / p.ell, ppg = p.ell / 16;
  for (int x = tid; x < pages * D; x += kCopyThreads) {
    const int j = x / D, c = x % D;
    T lo = ends[j * ppg][0][c], hi = ends[j * ppg][1][c];
    for (int r = j * ppg + 1; r < min((j + 1) * ppg, parts); ++r) {
      if (elem_key(ends[r][0][c]) < elem_key(lo)) lo = ends[r][0][c];
      if (elem_key(ends[r][1][c]) > elem_key(hi)) hi = ends[r][1][c];
    }
    const int t = r0 + j * p.ell, phys = dst_pages[t / p.P];
    if (phys < 0 || phys >= p.num_phys) continue;  // (reported above)
    T *m = meta + (((size_t)phys * p.Hkv + hk) * p.R + t % p.P / p.ell) * 2 * D + c;
    m[0] = lo;
    m[D] = hi;
  }
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, int dtype, int d, int cluster, cudaStream_t st) {
  int longest = 0;
  for (int i = 0; i < p.n; ++i) longest = longest > p.seqs[i].L ? longest : p.seqs[i].L;
  int seg = ((longest + cluster - 1) / cluster + 3) & ~3;
  const int smem = 4 * (seg < kCacheKeys ? seg : kCacheKeys);
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(evict_select_kernel, kCacheKeys * 4, &ready);
  if (e != cudaSuccess) return e;
  e = launch_pdl_cluster(evict_select_kernel, p.n * p.Hkv * cluster, kSelThreads, (size_t)smem,
                         cluster, st, p);
  if (e != cudaSuccess) return e;
  const int grid = p.n * p.Hkv * ((p.keep + kCopyRows - 1) / kCopyRows);
  auto go = [&](auto kernel) { return launch_pdl(kernel, grid, kCopyThreads, 0, st, p); };
  if (p.kv_fp8) return go(evict_copy_kernel<F8, 128>);
  if (dtype == 0) return d == 64 ? go(evict_copy_kernel<__half, 64>) : go(evict_copy_kernel<__half, 128>);
  return d == 64 ? go(evict_copy_kernel<__nv_bfloat16, 64>)
                 : go(evict_copy_kernel<__nv_bfloat16, 128>);
}

}  // namespace spd
