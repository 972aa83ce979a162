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
// integers; a histogram of their leading 11 bits, summed over the cluster
// through distributed shared memory, says where the room-th greatest key lies,
// and the keys that share its leading bits, when they are few, go to one CTA
// that finds its exact value (when they are many, ties above all, two more
// rounds over all keys do); a prefix count then gives every kept token its
// place.  The weights are read once.  evict_copy: CTAs
// take 64 kept rows at a time, gather K and V (memory is the bound: each kept
// row read and written once; the next rows' places are looked up while these
// arrive) and take the metadata's min and max from the rows that they hold.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include "dense.h"
#include "ptx.cuh"
#include "spd_internal.h"

namespace spd {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kBins = 2048;
constexpr int kCandidates = 4096;      // keys of the cut's first bin that one CTA finishes alone
constexpr int kCacheKeys = 40 * 1024;  // keys a CTA holds; longer stretches are read again

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

// The weight of a key; zeros and NaN, which keys do not tell apart, are read
// again.
__device__ __forceinline__ float key_weight(uint32_t k, const float *w) {
  if (k == 0x80000000u || k == 0xffffffffu) return __ldg(w);
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

__device__ __forceinline__ uint32_t ld_dsmem_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_dsmem_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Sum of the words at `addr` in the first n CTAs of the cluster (at most eight,
// all loads on their way before the first is used).
__device__ __forceinline__ uint32_t dsmem_sum(uint32_t addr, int n) {
  uint32_t v[8], sum = 0;
#pragma unroll
  for (int r = 0; r < 8; ++r) v[r] = r < n ? ld_dsmem_u32(map_rank(addr, r)) : 0u;
#pragma unroll
  for (int r = 0; r < 8; ++r) sum += v[r];
  return sum;
}

// Exclusive sums of the warps' two counts and their totals (one entry per warp
// in `tmp`, written by the callers' lane 0 before a barrier).
__device__ __forceinline__ void warp_prefix(const uint2 *tmp, uint2 *before, uint2 *all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint2 own = lane < kSelThreads / 32 ? tmp[lane] : make_uint2(0, 0);
  uint2 v = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, v.x, o), y = __shfl_up_sync(0xffffffffu, v.y, o);
    if (lane >= o) {
      v.x += x;
      v.y += y;
    }
  }
  before->x = __shfl_sync(0xffffffffu, v.x - own.x, warp);
  before->y = __shfl_sync(0xffffffffu, v.y - own.y, warp);
  all->x = __shfl_sync(0xffffffffu, v.x, 31);
  all->y = __shfl_sync(0xffffffffu, v.y, 31);
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

__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(
    const __grid_constant__ EvictParams p) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ uint32_t hist[kBins], tot[kBins];
  __shared__ uint2 tmp[kSelThreads / 32];
  __shared__ uint32_t counts[2];       // greater than, equal to the cut in this stretch
  __shared__ uint32_t found[2];        // a round's bin, keys above it
  __shared__ uint32_t result[2];       // the cut, how many equal to it stay
  __shared__ uint32_t cand[kCandidates];
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

  // the bin of `from` that holds the need-th greatest key, bins in descending
  // order, and the keys above it: into found[]
  constexpr int kPer = kBins / kSelThreads;
  auto find_bin = [&](const uint32_t *from, uint32_t need) {
    uint32_t c[kPer], mine = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) mine += c[j] = from[kBins - 1 - (tid * kPer + j)];
    uint32_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) tmp[warp] = make_uint2(inc, 0);
    __syncthreads();
    uint32_t below = lane < kSelThreads / 32 ? tmp[lane].x : 0u;  // warps' sums, summed up
    const uint32_t own = below;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, below, o);
      if (lane >= o) below += x;
    }
    inc += __shfl_sync(0xffffffffu, below - own, warp);
    uint32_t above = inc - mine;
    if (above < need && need <= inc) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        if (above < need && need <= above + c[j]) {
          found[0] = kBins - 1 - (tid * kPer + j);
          found[1] = above;
          break;
        }
        above += c[j];
      }
    }
    __syncthreads();
  };
  auto clear_hist = [&] {
    for (int b = tid; b < kBins; b += kSelThreads) hist[b] = 0;
    __syncthreads();
  };
  // the cluster's histograms summed into everyone's tot
  auto sum_hists = [&] {
    cluster_sync();  // every CTA's histogram is complete
    const int per = (kBins + cs - 1) / cs;
    for (int b = rank * per + tid; b < min(kBins, (rank + 1) * per); b += kSelThreads) {
      const uint32_t at = smem_u32(&hist[b]), to = smem_u32(&tot[b]);
      const uint32_t sum = dsmem_sum(at, cs);
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < cs) st_dsmem_u32(map_rank(to, r), sum);
    }
    cluster_sync();  // the sums are everywhere
  };

  // ---- the cut: 11, 11 and 10 bits ----
  uint32_t need = (uint32_t)room;
  sum_hists();
  find_bin(tot, need);
  uint32_t prefix = found[0];  // the cut's leading bits; need: its rank among them
  need -= found[1];
  if (tot[prefix] <= kCandidates) {
    // few keys share the leading bits: the cluster's first CTA takes them all
    if (tid == 0) counts[0] = dsmem_sum(smem_u32(&hist[prefix]), rank);
    __syncthreads();
#pragma unroll 2
    for (int i0 = 0; i0 < len; i0 += 4 * kSelThreads) {
      uint32_t k[4];
      keys4(i0 + 4 * tid, len, k);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if ((k[j] >> 21) == prefix && k[j] != 0)
          st_dsmem_u32(map_rank(smem_u32(&cand[atomicAdd(&counts[0], 1u)]), 0), k[j]);
    }
    cluster_sync();  // the candidates are there
    if (rank == 0) {
      const int m = (int)tot[prefix];
#pragma unroll 1
      for (int round = 1; round < 3; ++round) {
        const int shift = round == 1 ? 10 : 0, bits = round == 1 ? 11 : 10;
        clear_hist();
        for (int i = tid; i < m; i += kSelThreads) {
          const uint32_t k = cand[i];
          if ((k >> (shift + bits)) == prefix) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1u);
        }
        __syncthreads();
        find_bin(hist, need);
        prefix = (prefix << bits) | found[0];
        need -= found[1];
      }
      if (tid < cs) {
        st_dsmem_u32(map_rank(smem_u32(&result[0]), tid), prefix);
        st_dsmem_u32(map_rank(smem_u32(&result[1]), tid), need);
      }
    }
    cluster_sync();  // the cut is everywhere
    prefix = result[0];
    need = result[1];
  } else {
#pragma unroll 1
    for (int round = 1; round < 3; ++round) {
      const int shift = round == 1 ? 10 : 0, bits = round == 1 ? 11 : 10;
      clear_hist();
#pragma unroll 2
      for (int i0 = 0; i0 < len; i0 += 4 * kSelThreads) {
        uint32_t k[4];
        keys4(i0 + 4 * tid, len, k);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // (0, behind the end, is of no key)
          const bool in = (k[j] >> (shift + bits)) == prefix && k[j] != 0;
          const uint32_t bin = (k[j] >> shift) & ((1u << bits) - 1);
          if (__popc(__ballot_sync(0xffffffffu, in)) > 8) count_bin(hist, in, bin);
          else if (in) atomicAdd(&hist[bin], 1u);
        }
      }
      sum_hists();
      find_bin(tot, need);
      prefix = (prefix << bits) | found[0];
      need -= found[1];
    }
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
  uint32_t gt = before.x + dsmem_sum(smem_u32(&counts[0]), rank);  // before this warp's stretch
  uint32_t eq = before.y + dsmem_sum(smem_u32(&counts[1]), rank);
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
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool more = k[j] > prefix, tie = k[j] == prefix;
      if (more || (tie && e < need)) {
        const uint32_t at = g + min(e, need);
        kept[at] = s0 + i + j;
        if (kw) kw[at] = key_weight(k[j], ws + i + j);
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
constexpr int kCopyRows = 64, kCopyThreads = 256, kCopyCtas = 4;  // (CTAs per SM)

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
__global__ void __launch_bounds__(kCopyThreads, kCopyCtas) evict_copy_kernel(
    const __grid_constant__ EvictParams p) {
  constexpr int kLanes = D * (int)sizeof(T) / 16;       // threads of one row
  constexpr int kStep = kCopyThreads / kLanes;          // rows at once
  constexpr int kIter = kCopyRows / kStep;
  __shared__ uint4 krows[kCopyRows * kLanes];
  __shared__ __align__(16) T ends[kCopyRows / 16][2][D];
  const int tid = threadIdx.x, groups = (p.keep + kCopyRows - 1) / kCopyRows;
  const int total = p.n * p.Hkv * groups;
  pdl_wait();
  pdl_launch_dependents();
  const uint4 *kp = static_cast<const uint4 *>(p.k_pool), *vp = static_cast<const uint4 *>(p.v_pool);
  uint4 *ko = static_cast<uint4 *>(p.k_pool), *vo = static_cast<uint4 *>(p.v_pool);
  T *meta = static_cast<T *>(p.meta);
  const int lane = tid % kLanes, sub = tid / kLanes;
  constexpr uint32_t kNone = 0xffffffffu;
  // row t of a sequence's pages, or the largest value if the check fails
  auto row_at = [&](int slot, int hk, int t) -> uint32_t {
    const int blk = p.P_log2 >= 0 ? t >> p.P_log2 : t / p.P;
    const int phys = t >= 0 && blk < p.max_pp ? p.page_table[(size_t)slot * p.max_pp + blk] : -1;
    if (phys < 0 || phys >= p.num_phys) {
      ev_set_err(p.err, kDevBadPhys, slot, t, phys);
      return kNone;
    }
    return (uint32_t)(phys * p.Hkv + hk) * (uint32_t)p.P + (uint32_t)(t - blk * p.P);
  };
  // where the rows of group g lie
  auto look_up = [&](int g, uint32_t (&from)[kIter], uint32_t (&to)[kIter]) {
    const int unit = g / groups, r0 = g % groups * kCopyRows, hk = unit % p.Hkv;
    const EvictSeq &s = p.seqs[unit / p.Hkv];
    const int *kept = p.kept + (size_t)unit * p.keep + r0;
    int t[kIter];
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int r = i * kStep + sub;
      t[i] = r0 + r < s.m ? kept[r] : s.L;
    }
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      from[i] = t[i] < s.L ? row_at(s.src, hk, t[i]) : kNone;
      to[i] = from[i] == kNone ? kNone : row_at(s.dst, hk, r0 + i * kStep + sub);
    }
  };
  uint32_t from[kIter], to[kIter];
  if ((int)blockIdx.x < total) look_up(blockIdx.x, from, to);
  for (int g = blockIdx.x; g < total; g += gridDim.x) {
    uint4 kx[kIter], vx[kIter];
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const bool in = to[i] != kNone;
      const size_t at = (size_t)from[i] * kLanes + lane;
      kx[i] = in ? __ldcs(kp + at) : make_uint4(0, 0, 0, 0);
      vx[i] = in ? __ldcs(vp + at) : make_uint4(0, 0, 0, 0);
    }
    // the next group is looked up while this one's rows arrive
    uint32_t here[kIter];
#pragma unroll
    for (int i = 0; i < kIter; ++i) here[i] = to[i];
    if (g + (int)gridDim.x < total) look_up(g + gridDim.x, from, to);
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      if (here[i] != kNone) {
        const size_t at = (size_t)here[i] * kLanes + lane;
        ko[at] = kx[i];
        vo[at] = vx[i];
      }
    }
    // metadata of the logical pages that begin in these rows (64 rows hold whole
    // ones): least and greatest of each channel per 16 rows, then per page
    const int unit = g / groups, r0 = g % groups * kCopyRows, hk = unit % p.Hkv;
    const EvictSeq &s = p.seqs[unit / p.Hkv];
    const int n = min(kCopyRows, s.m - r0);
    if (n <= 0) continue;  // (the same for the block)
    const int parts = (n + 15) / 16;
    if constexpr (sizeof(T) == 2) {
      // rows of a warp first, in registers, then the warps that share a part
      using T2 = typename Pair<T>::type;
      constexpr int kPerPart = 16 * kLanes / 32;  // warps per 16 rows
      const T2 top = Pair<T>::limit(false), bottom = Pair<T>::limit(true);
#pragma unroll
      for (int i = 0; i < kIter; ++i) {
        const bool in = i * kStep + sub < n;
        T2 lo[4], hi[4];
        const T2 *x = reinterpret_cast<const T2 *>(&kx[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          lo[e] = in ? x[e] : top;
          hi[e] = in ? x[e] : bottom;
#pragma unroll
          for (int o = kLanes; o < 32; o <<= 1) {
            lo[e] = __hmin2(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], o));
            hi[e] = __hmax2(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], o));
          }
        }
        if ((tid & 31) < kLanes) {
          uint4 *at = krows + ((i * (kCopyThreads / 32) + (tid >> 5)) * 2) * kLanes + lane;
          at[0] = *reinterpret_cast<const uint4 *>(lo);
          at[kLanes] = *reinterpret_cast<const uint4 *>(hi);
        }
      }
      __syncthreads();
      // part j: krows' entries j kPerPart .. of the warps' (least, greatest)
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
        for (int r = 1; r < m; ++r) {
          const T e = rows[(16 * j + r) * D + c];
          if (elem_key(e) < elem_key(lo)) lo = e;
          if (elem_key(e) > elem_key(hi)) hi = e;
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
      const int t = r0 + j * p.ell, blk = t / p.P;
      const int phys = p.page_table[(size_t)s.dst * p.max_pp + blk];
      if (phys < 0 || phys >= p.num_phys) continue;  // (reported above)
      T *m = meta + (((size_t)phys * p.Hkv + hk) * p.R + (t - blk * p.P) / p.ell) * 2 * D + c;
      m[0] = lo;
      m[D] = hi;
    }
  }
}

}  // namespace

// Clusters of `cs` CTAs of evict_select that the current device runs at once.
static int active_clusters(int cs) {
  static std::atomic<int> known[64][9];
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) return 0;
  const bool keep = device < 64;
  int n = keep ? known[device][cs].load(std::memory_order_relaxed) : 0;
  if (n > 0) return n - 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)cs);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = kCacheKeys * 4;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cs;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, evict_select_kernel, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    n = 0;
  }
  if (keep) known[device][cs].store(n + 1, std::memory_order_relaxed);
  return n;
}

cudaError_t launch_evict(const EvictParams &p, int dtype, int d, int sms, cudaStream_t st) {
  int longest = 0;
  for (int i = 0; i < p.n; ++i) longest = longest > p.seqs[i].L ? longest : p.seqs[i].L;
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(evict_select_kernel, kCacheKeys * 4, &ready);
  if (e != cudaSuccess) return e;
  // CTAs per (sequence, kv head): as many as the GPU runs of such clusters at once
  // (a GPC holds whole clusters only), with at least 4,096 tokens each
  int cluster = 1;
  while (cluster < 8 && cluster * 4096 < longest && active_clusters(cluster + 1) >= p.n * p.Hkv)
    ++cluster;
  const int seg = ((longest + cluster - 1) / cluster + 3) & ~3;
  const int smem = 4 * (seg < kCacheKeys ? seg : kCacheKeys);
  e = launch_pdl_cluster(evict_select_kernel, p.n * p.Hkv * cluster, kSelThreads, (size_t)smem,
                         cluster, st, p);
  if (e != cudaSuccess) return e;
  const long long groups = (long long)p.n * p.Hkv * ((p.keep + kCopyRows - 1) / kCopyRows);
  const int grid = (int)(groups < (long long)sms * kCopyCtas ? groups : (long long)sms * kCopyCtas);
  auto go = [&](auto kernel) { return launch_pdl(kernel, grid, kCopyThreads, 0, st, p); };
  if (p.kv_fp8) return go(evict_copy_kernel<F8, 128>);
  if (dtype == 0) return d == 64 ? go(evict_copy_kernel<__half, 64>) : go(evict_copy_kernel<__half, 128>);
  return d == 64 ? go(evict_copy_kernel<__nv_bfloat16, 64>)
                 : go(evict_copy_kernel<__nv_bfloat16, 128>);
}

}  // namespace spd
