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

constexpr int kSelThreads = 512, kPerThread = 4;
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

// Inclusive sum over the block's threads in order (two 32-bit counts at once);
// `tmp` holds one entry per warp.
__device__ __forceinline__ uint2 block_scan(uint2 v, uint2 *tmp, uint2 *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, v.x, o), y = __shfl_up_sync(0xffffffffu, v.y, o);
    if (lane >= o) {
      v.x += x;
      v.y += y;
    }
  }
  __syncthreads();  // (tmp may still be read from the call before)
  if (lane == 31) tmp[warp] = v;
  __syncthreads();
  uint2 before = make_uint2(0, 0), all = make_uint2(0, 0);
#pragma unroll
  for (int w = 0; w < kSelThreads / 32; ++w) {
    const uint2 t = tmp[w];
    if (w < warp) {
      before.x += t.x;
      before.y += t.y;
    }
    all.x += t.x;
    all.y += t.y;
  }
  *total = all;
  return make_uint2(v.x + before.x, v.y + before.y);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(
    const __grid_constant__ EvictParams p) {
  extern __shared__ uint32_t keys[];
  __shared__ uint32_t hist[kBins], tot[kBins];
  __shared__ uint2 tmp[kSelThreads / 32];
  __shared__ uint32_t counts[2];       // greater than, equal to the cut in this stretch
  __shared__ uint32_t found[2];        // the round's bin, keys above it
  const int tid = threadIdx.x, lane = tid & 31;
  const int cs = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
  const int unit = blockIdx.x / cs, seq = unit / p.Hkv;
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
  for (int i = tid; i < min(len, kCacheKeys); i += kSelThreads) keys[i] = weight_key(w[s0 + i]);
  auto key = [&](int i) { return i < kCacheKeys ? keys[i] : weight_key(w[s0 + i]); };

  uint32_t prefix = 0, need = (uint32_t)room;  // the cut's leading bits; its rank among them
  for (int round = 0; round < 3; ++round) {
    const int shift = round == 0 ? 21 : round == 1 ? 10 : 0, bits = round == 2 ? 10 : 11;
    for (int b = tid; b < kBins; b += kSelThreads) hist[b] = 0;
    __syncthreads();
    for (int i0 = 0; i0 < len; i0 += kSelThreads) {
      const int i = i0 + tid;
      const uint32_t k = i < len ? key(i) : 0u;
      const bool in = i < len && (round == 0 || (k >> (shift + bits)) == prefix);
      const uint32_t bin = (k >> shift) & ((1u << bits) - 1);
      // many tokens share one weight (0 above all): the first lane's bin is
      // counted once for the warp
      const uint32_t act = __ballot_sync(0xffffffffu, in);
      if (!act) continue;
      const int lead = __ffs(act) - 1;
      const uint32_t lbin = __shfl_sync(0xffffffffu, bin, lead);
      const uint32_t same = __ballot_sync(0xffffffffu, in && bin == lbin);
      if (lane == lead) atomicAdd(&hist[lbin], __popc(same));
      if (in && bin != lbin) atomicAdd(&hist[bin], 1u);
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
    uint32_t c[4], mine = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) mine += c[j] = tot[kBins - 1 - (tid * 4 + j)];
    uint2 all;
    const uint2 inc = block_scan(make_uint2(mine, 0), tmp, &all);
    uint32_t above = inc.x - mine;
    if (above < need && need <= inc.x) {
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
  static_assert(kBins == kSelThreads * 4, "four bins per thread");
  // prefix is the cut itself: greater keys all stay, of the equal ones the
  // first `need`
  uint2 cnt = make_uint2(0, 0);
  for (int i = tid; i < len; i += kSelThreads) {
    const uint32_t k = key(i);
    cnt.x += k > prefix;
    cnt.y += k == prefix;
  }
  uint2 total;
  block_scan(cnt, tmp, &total);
  if (tid == 0) {
    counts[0] = total.x;
    counts[1] = total.y;
  }
  cluster_sync();
  uint32_t gt = 0, eq = 0;  // before this stretch
  for (int r = 0; r < rank; ++r) {
    gt += ld_dsmem_u32(map_rank(smem_u32(&counts[0]), r));
    eq += ld_dsmem_u32(map_rank(smem_u32(&counts[1]), r));
  }
  cluster_sync();  // the counts have been read: a CTA may leave
  for (int i0 = 0; i0 < len; i0 += kSelThreads * kPerThread) {
    const int i = i0 + tid * kPerThread;
    uint32_t k[kPerThread];
    uint2 v = make_uint2(0, 0);
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      k[j] = i + j < len ? key(i + j) : 0u;
      v.x += i + j < len && k[j] > prefix;
      v.y += i + j < len && k[j] == prefix;
    }
    const uint2 inc = block_scan(v, tmp, &total);
    uint32_t g = gt + inc.x - v.x, e = eq + inc.y - v.y;
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      if (i + j >= len) break;
      const bool more = k[j] > prefix, tie = k[j] == prefix;
      if (more || (tie && e < need)) {
        const uint32_t at = g + min(e, need);
        kept[at] = s0 + i + j;
        if (kw) kw[at] = w[s0 + i + j];
      }
      g += more;
      e += tie;
    }
    gt += total.x;
    eq += total.y;
  }
}

// ---- gather + metadata ---------------------------------------------------------
constexpr int kCopyRows = 64, kCopyThreads = 256;

// Order of two stored elements: fp8 codes by sign and magnitude.
struct F8 {
  uint8_t v;
};
template <typename T> __device__ __forceinline__ float elem_key(T x) { return (float)x; }
template <> __device__ __forceinline__ float elem_key<F8>(F8 x) { return (float)e4m3_key(x.v); }

template <typename T, int D>
__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(
    const __grid_constant__ EvictParams p) {
  constexpr int kLanes = D * (int)sizeof(T) / 16;       // threads of one row
  constexpr int kStep = kCopyThreads / kLanes;          // rows at once
  constexpr int kIter = kCopyRows / kStep;
  __shared__ uint4 krows[kCopyRows * kLanes];
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
  // row t of a page list, in units of 16 bytes; negative if the check fails
  auto row_at = [&](const int *pages, int t, int slot) -> long long {
    const int blk = t / p.P, phys = t >= 0 && blk < p.max_pp ? pages[blk] : -1;
    if (phys < 0 || phys >= p.num_phys) {
      ev_set_err(p.err, kDevBadPhys, slot, t, phys);
      return -1;
    }
    return (((long long)phys * p.Hkv + hk) * p.P + t % p.P) * kLanes + lane;
  };
  long long from[kIter], to[kIter];
  uint4 kx[kIter], vx[kIter];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int r = i * kStep + sub;
    from[i] = to[i] = -1;
    if (r < n) {
      const int t = kept[r];
      from[i] = t < s.L ? row_at(src_pages, t, s.src) : -1;
      to[i] = row_at(dst_pages, r0 + r, s.dst);
    }
  }
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const bool in = from[i] >= 0 && to[i] >= 0;
    kx[i] = in ? kp[from[i]] : make_uint4(0, 0, 0, 0);
    vx[i] = in ? vp[from[i]] : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    if (from[i] >= 0 && to[i] >= 0) {
      ko[to[i]] = kx[i];
      vo[to[i]] = vx[i];
    }
    krows[(i * kStep + sub) * kLanes + lane] = kx[i];
  }
  __syncthreads();
  // metadata of the logical pages that begin in these rows (64 rows hold whole ones)
  T *meta = static_cast<T *>(p.meta);
  const T *rows = reinterpret_cast<const T *>(krows);
  const int pages = (n + p.ell - 1) / p.ell;
  for (int x = tid; x < pages * D; x += kCopyThreads) {
    const int j = x / D, c = x % D;
    const int a = j * p.ell, b = min(a + p.ell, n);
    T lo = rows[a * D + c], hi = lo;
    float flo = elem_key(lo), fhi = flo;
    for (int r = a + 1; r < b; ++r) {
      const T e = rows[r * D + c];
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
    const int t = r0 + a, blk = t / p.P, phys = dst_pages[blk];
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
  cudaError_t e = cudaFuncSetAttribute(evict_select_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kCacheKeys * 4);
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
