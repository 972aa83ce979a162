// Dense attention with score rules on the 5th-generation tensor cores: prompts
// whose queries each attend an interval of keys, and the shared prefix of a
// decode batch.
//
//   x(r, t) = rule(q_r . k_t)  (ScoreRule, base 2), keys begin_r <= t < end_r
//   o_r = sum_t 2^(x - m_r) v_t / sum_t 2^(x - m_r)
//
// One CTA per (head group, kv head, tile, key split): two matrices of 128 query
// rows, a row being one (token, query head of the group) pair, so that the
// heads that share K and V share their tiles too.  Keys come in blocks of 64,
// two blocks (a pair) per stage of two-stage TMA rings of K and of V:
//   S_m = Q_m . K^T     tcgen05.mma M 128 x N 64, fp32 in tensor memory, the
//                       matrix's blocks in two buffers in turn;
//   softmax             one row per thread: score rule, mask, online max and
//                       sum in fp32, weights written back over S as 16 bits;
//   O_m += P_m . V      A = P from tensor memory, fp32 accumulation.
// An S of N 64 takes longer than half of one of N 128 (the read of Q's 128 rows
// bounds it), but two buffers let S of the block after next start as soon as
// P . V of this one is done: the hand-overs between the roles (about 300 cycles
// each) and the products of one buffer then pass while the softmax works on the
// other.  One product of N 128 per pair, with the next S behind the whole pair's
// P . V, took 1,319 us against 1,202 (2,048 queries over 49,152 keys), 461 against
// 420 (8,192 causal), 2,307 against 2,020 (8,192 over 16,384, 64 channels), 831
// against 623 (8,192 capped) and 67 against 55 (2,501 tokens with a bias and fp32
// output, 64 channels).
// Outputs of 32 bits keep P in kParts 16-bit parts, each the rounding of what the
// ones before left, a product each: two hold 22 bits of each weight with fp16 and
// 16 with bf16, which takes a third part (through shared memory: tensor memory is
// full): over a shared prefix always, in prompts where a CTA meets at most kThirdKeys
// keys (kParts 3).  Over longer stretches the tensor cores' own sums, which round
// towards 0 at every 16 keys, are off by as much where many keys count (two parts a
// relative 2e-6, the sums 2.9e-6 at 1,100 keys), and in prompts a third part
// everywhere costs 40% of the time (2,048 biased queries over 16,384 keys 650 and
// 929 us, 759 as it is; 64 sequences over 32,768 shared keys 86 and 97).  Outputs of
// 16 bits round P once, which is an error of the same size as the rounding of the
// output.
//
// A matrix leaves out the pairs before and behind its rows' keys.  With `dup` (at
// most 128 rows) both matrices hold the same rows, and matrix m takes block m of
// every pair; each then counts as a split of its own.  Splits leave unnormalised
// sums to a combining kernel.
//
// Blocks that some row attends only in part ("edge" blocks) are masked, and
// their V tile is scanned: a value that is not finite is replaced by zero in
// shared memory (0 x NaN would reach rows that do not attend the key) and added
// back, in the epilogue, to the rows that do.  Rows of a page behind the
// sequence's end are zeroed the same way.
//
// Warps: 0 .. 7 softmax (matrix warp / 4), 8 and 9 issue matrix 0's and 1's
// MMAs, 10 loads, 11 scans V.  Every wait is bounded.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <limits.h>
#include <math_constants.h>

#include "dense.h"
#include "dense_math.cuh"
#include "ptx.cuh"
#include "spd_internal.h"

namespace spd {
namespace {

constexpr uint32_t kDtWait = 1u << 22;  // bounded mbarrier polls
constexpr int kThirdKeys = 1024;        // a prompt CTA's keys up to which bf16 weights take three parts
constexpr float kDtRescaleAbove = 8.f;  // log2 growth of a row max that moves it

template <int D, bool kThird>
struct DtSmem {
  static constexpr int KB = D / 64;               // 64-column sub-tiles of a row
  static constexpr int kStages = 2;               // K / V ring, a pair of blocks per stage
  static constexpr int kStageBytes = KB * 16384;  // K (or V) of two 64-row blocks
  static constexpr int kQ = 0;                    // [2][KB][128 x 128 B]
  static constexpr int kK = 2 * KB * 16384;       // [stage][KB][block u][64 x 128 B]
  static constexpr int kV = kK + kStages * kStageBytes;  // [stage][block u][KB][64 x 128 B]
  static constexpr int kL = kV + kStages * kStageBytes;  // P's third part [2][128 x 128 B]
  static constexpr int kBars = kL + (kThird ? 2 * 16384 : 0);
  // mbarriers: Q; per stage K full, V full, V scanned, K empty, V empty; per
  // matrix and buffer S full, P full; per matrix O done (per block), O final,
  // drain.  Every waiter is at most one completion behind the barrier that it
  // polls by parity.
  static constexpr int kBarQ = 0;
  static constexpr int kBarKF = 1;
  static constexpr int kBarVF = kBarKF + kStages;
  static constexpr int kBarVC = kBarVF + kStages;
  static constexpr int kBarKE = kBarVC + kStages;
  static constexpr int kBarVE = kBarKE + kStages;
  static constexpr int kBarSF = kBarVE + kStages;
  static constexpr int kBarPF = kBarSF + 4;
  static constexpr int kBarOD = kBarPF + 4;
  static constexpr int kBarOF = kBarOD + 2;
  static constexpr int kBarDR = kBarOF + 2;
  static constexpr int kNumBars = kBarDR + 2;
  static constexpr int kMisc = kBars + 8 * kNumBars;  // ints, see below
  static constexpr int kBytes = kMisc + 64 + 1024;    // + alignment slack
  // tensor-memory columns: S / P of matrix m, block u at 128 m + 64 u; O_m at
  // 256 + D m
  static constexpr int kAlloc = 512;
  static constexpr int kMmaWarp = 8, kLoadWarp = 10, kScanWarp = 11;
  static constexpr int kThreads = 12 * 32;
  static_assert(kBytes <= 232448, "shared memory");
};
// kMisc: [0] tensor-memory base, [1] fail flag, [2] a V value was not finite,
// [3 + 4 m ..] of matrix m: least begin, greatest end, greatest begin, least end
constexpr int kMiscFail = 1, kMiscBad = 2, kMiscRange = 3;

__device__ __forceinline__ void dt_set_err(int *err, int code, int a, int b, int c) {
  if (atomicCAS(err, 0, code) == 0) {
    err[1] = a;
    err[2] = b;
    err[3] = c;
  }
}

// Bounded wait; gives up early once another role has raised the fail flag.
__device__ __forceinline__ bool dt_wait(uint64_t *bar, uint32_t parity, volatile int *fail) {
  for (uint32_t i = 0; i < kDtWait; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 255u) == 255u && *fail) return false;
  }
  *fail = 1;
  return false;
}
// Bounded wait that the fail flag does not cut short (work in flight).
__device__ __forceinline__ void dt_drain(uint64_t *bar, uint32_t parity) {
  for (uint32_t i = 0; i < kDtWait; ++i)
    if (mbar_try_wait(bar, parity)) return;
}

// Two weights rounded to 16 bits (element 0 in the low half); with the split,
// also the 16-bit rounding of what that left.
template <typename T> struct Weights;
template <> struct Weights<__nv_bfloat16> {
  static constexpr bool bf16 = true;
  static __device__ __forceinline__ uint32_t round(float2 p) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(p.x, p.y);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  static __device__ __forceinline__ void split(float2 p, uint32_t &hi, uint32_t &lo) {
    hi = round(p);
    lo = round(f2_sub(p, make_float2(__uint_as_float(hi << 16),
                                     __uint_as_float(hi & 0xffff0000u))));
  }
  static __device__ __forceinline__ uint32_t rest(float2 p, uint32_t hi, uint32_t lo) {
    const float2 r = f2_sub(p, make_float2(__uint_as_float(hi << 16),
                                           __uint_as_float(hi & 0xffff0000u)));
    return round(f2_sub(r, make_float2(__uint_as_float(lo << 16),
                                       __uint_as_float(lo & 0xffff0000u))));
  }
  static __device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
};
template <> struct Weights<__half> {
  static constexpr bool bf16 = false;
  static __device__ __forceinline__ uint32_t round(float2 p) {
    const __half2 h = __floats2half2_rn(p.x, p.y);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  static __device__ __forceinline__ void split(float2 p, uint32_t &hi, uint32_t &lo) {
    hi = round(p);
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    lo = round(f2_sub(p, f));
  }
  static __device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
};

// Bits 15 and 31: the low / high half is not finite (its exponent all ones;
// `exponent` in both halves, `step` one in the exponent's lowest bit: the sum
// carries into the half's sign bit exactly then).
__device__ __forceinline__ uint32_t nonfinite(uint32_t x, uint32_t exponent, uint32_t step) {
  return ((x & exponent) + step) & 0x80008000u;
}
__device__ __forceinline__ uint32_t without_nonfinite(uint32_t x, uint32_t exponent, uint32_t step) {
  const uint32_t f = nonfinite(x, exponent, step);
  return x & ~((f >> 15) * 0xffffu);  // (each flagged half's 16 bits)
}

// Where a prompt call's kernels record a failed check: one word (and details)
// per device that loads the library, zero until then, read and cleared by
// dense_error_word.
__device__ int g_dense_err[4];

// A rule's parts that an instance holds: nothing but the scale, a cap, a distance bias
// (and a cap if there is one).  Cap and bias apart: 8,192 tokens with a cap 572 -> 563
// us, 4,096 with both 231 -> 205.  (An instance with a bias still asks for the slopes
// where it adds it: as a constant, 2,048 queries over 16,384 keys with fp32 output took
// 796 us against 760.)
enum { kPlain, kCap, kBias };

template <typename T, int D, int kParts, int kRule>
__global__ void __launch_bounds__(DtSmem<D, false>::kThreads, 1)
    dense_tc_kernel(const __grid_constant__ DenseTcParams p) {
  constexpr bool kSplitP = kParts > 1, kThird = kParts == 3;
  using Sm = DtSmem<D, kThird>;
  constexpr int KB = Sm::KB, S = Sm::kStages;
  extern __shared__ uint8_t dt_smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(dt_smem_raw) + 1023) & ~uintptr_t(1023));
  int *const err = p.err ? p.err : g_dense_err;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Sm::kBars);
  int *misc = reinterpret_cast<int *>(smem + Sm::kMisc);
  volatile int *fail = misc + kMiscFail;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the last tiles (most keys when causal) first; heads fastest, so that the
  // CTAs that run together read the same K and V
  const int units_h = p.Hkv * p.HG;
  const int hg_hk = blockIdx.x % units_h, rest = blockIdx.x / units_h;
  const int hk = hg_hk / p.HG, hg = hg_hk % p.HG;
  const int split = rest % p.nsplit, tile = p.tiles - 1 - rest / p.nsplit;
  const int unit = tile * units_h + hg_hk;
  const int lhp = p.lhp, tpm = 128 >> lhp;           // tokens per matrix
  const int tok0 = tile * (p.dup ? tpm : 2 * tpm);   // the unit's first token
  const int h0 = hk * p.G + (hg << lhp);             // the group's first query head

  if (warp == Sm::kMmaWarp) tmem_alloc(reinterpret_cast<uint32_t *>(misc), Sm::kAlloc);
  if (tid == Sm::kLoadWarp * 32) {
    for (int x = 0; x < Sm::kNumBars; ++x)
      mbar_init(&bars[x], (x >= Sm::kBarPF && x < Sm::kBarOD)   ? 4  // P: one per softmax warp
                          : (x >= Sm::kBarKE && x < Sm::kBarSF) ? 2  // empty: one per MMA warp
                                                                : 1);
    *fail = 0;
    misc[kMiscBad] = 0;
    for (int m = 0; m < 2; ++m) {
      misc[kMiscRange + 4 * m] = INT_MAX;
      misc[kMiscRange + 4 * m + 1] = 0;
      misc[kMiscRange + 4 * m + 2] = 0;
      misc[kMiscRange + 4 * m + 3] = INT_MAX;
    }
    fence_mbar_init();
    prefetch_tmap(&p.tm_q);
    prefetch_tmap(&p.tm_k);
    prefetch_tmap(&p.tm_v);
    prefetch_tmap(&p.tm_out);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, (uint32_t)misc[0], 0);  // warp-uniform
  pdl_wait();
  pdl_launch_dependents();
  if (tid == Sm::kLoadWarp * 32) {  // Q is on its way while the intervals are read
    mbar_arrive_expect_tx(&bars[Sm::kBarQ], 2 * KB * 16384);
    for (int mm = 0; mm < 2; ++mm)
      for (int kb = 0; kb < KB; ++kb)
        tma_load_4d(smem + Sm::kQ + (mm * KB + kb) * 16384, &p.tm_q, 0, kb, h0,
                    tok0 + (p.dup ? 0 : mm * tpm), &bars[Sm::kBarQ]);
  }

  // ---- the interval of keys of every row, and of each matrix ----
  int rbeg = 0, rend = 0;  // of softmax thread tid's row (an empty one: 0, 0)
  const int m_row = (warp >> 2) & 1, row = tid & 127;
  const int tok = tok0 + (p.dup ? 0 : m_row * tpm) + (row >> lhp);
  const int h_row = h0 + (row & ((1 << lhp) - 1));
  if (warp < 8) {
    if (tok < p.Lq) {
      if (p.paged) {
        rend = p.Lk;
      } else if (p.key_begin) {
        rbeg = max(p.key_begin[tok], 0);
        rend = min(p.key_end[tok], p.Lk);
      } else {
        rend = min(p.pos0 + tok + 1, p.Lk);
      }
      if (rbeg >= rend) rbeg = rend = 0;
    }
    const bool some = rend > 0;
    const int b0 = __reduce_min_sync(0xffffffffu, some ? rbeg : INT_MAX);
    const int e1 = __reduce_max_sync(0xffffffffu, some ? rend : 0);
    const int b1 = __reduce_max_sync(0xffffffffu, some ? rbeg : 0);
    const int e0 = __reduce_min_sync(0xffffffffu, some ? rend : INT_MAX);
    if (lane == 0) {
      int *rg = misc + kMiscRange + 4 * m_row;
      atomicMin(rg, b0);
      atomicMax(rg + 1, e1);
      atomicMax(rg + 2, b1);
      atomicMin(rg + 3, e0);
    }
  }
  __syncthreads();
  const int *rg = misc + kMiscRange;
  // the split's blocks [kb0, kb0 + n) of the CTA's range, in pairs [0, pairs)
  const int all_beg = min(rg[0], rg[4]), all_end = max(rg[1], rg[5]);
  const int full_beg = max(rg[2], rg[6]), full_end = min(rg[3], rg[7]);
  int kb0 = 0, n = 0;
  if (all_beg < all_end) {
    const int first = all_beg / kDenseBlock, last = (all_end + kDenseBlock - 1) / kDenseBlock;
    const int per = ((last - first + p.nsplit - 1) / p.nsplit + 1) & ~1;  // whole pairs
    kb0 = first + split * per;
    n = max(0, min(last - kb0, per));
  }
  const int pairs = (n + 1) / 2;
  const bool third = kThird && p.out_f32 && (p.paged || n * kDenseBlock <= kThirdKeys);
  // Blocks in ascending order, so that the CTAs that run together read the same
  // K and V at the same time (descending, where each starts at its own newest
  // key, 1,227 us against 1,216 on 2,048 queries over 49,152 keys).  With a
  // distance bias in descending order: the largest scores come first and the
  // running max hardly moves (2,501 tokens 55 us against 66).  Block j of the
  // split begins at key0_of(j); pair pp holds blocks 2 pp and 2 pp + 1.
  constexpr bool desc = kRule == kBias;
  auto key0_of = [&](int j) { return (desc ? kb0 + n - 1 - j : kb0 + j) * kDenseBlock; };
  // the pairs [first, last) that matrix m computes (with dup its block m of each)
  auto pair_first = [&](int m) {
    const int past = desc ? kb0 + n - (rg[4 * m + 1] + kDenseBlock - 1) / kDenseBlock
                          : rg[4 * m] / kDenseBlock - kb0;  // blocks before its keys
    return p.dup ? 0 : min(pairs, max(0, past) / 2);
  };
  auto pair_last = [&](int m) {
    if (p.dup) return (n + 1 - m) / 2;
    if (rg[4 * m] >= rg[4 * m + 1]) return 0;
    const int blocks = desc ? kb0 + n - rg[4 * m] / kDenseBlock  // up to its last key's
                            : (rg[4 * m + 1] + kDenseBlock - 1) / kDenseBlock - kb0;
    const int last = min(pairs, max(0, blocks + 1) / 2);
    return last > pair_first(m) ? last : 0;  // (0: none of the split's keys)
  };
  // the pairs [0, np) that are loaded: up to the last one that a matrix computes.  (The
  // rows of one matrix may lie far from those of the other, with whole splits between
  // them.  A stage's K counts as read once both matrices say so, and only one that
  // computes the pair or a later one has waited for the copy.)
  const int np = max(pair_last(0), pair_last(1));
  auto is_edge = [&](int key0) {  // some row attends only a part of the block
    return key0 < full_beg || key0 + kDenseBlock > full_end;
  };

  if (warp == Sm::kLoadWarp) {
    // ---- TMA: K and V of every pair through the ring ----
    if (lane == 0) {
      int k_issued = 0, v_issued = 0;
      bool ok = true;
      for (int pp = 0; pp < np && ok; ++pp) {
        const int s = pp % S, nbk = min(2, n - 2 * pp);
        if (pp >= S && !(ok = dt_wait(&bars[Sm::kBarKE + s], ((pp / S) - 1) & 1, fail))) break;
        uint8_t *kt = smem + Sm::kK + s * Sm::kStageBytes, *vt = smem + Sm::kV + s * Sm::kStageBytes;
        auto v_free = [&] { return pp < S || dt_wait(&bars[Sm::kBarVE + s], ((pp / S) - 1) & 1, fail); };
        if (!p.paged) {
          mbar_arrive_expect_tx(&bars[Sm::kBarKF + s], nbk * KB * 8192);
          for (int u = 0; u < nbk; ++u)
            for (int kb = 0; kb < KB; ++kb)
              tma_load_4d(kt + kb * 16384 + u * 8192, &p.tm_k, 0, kb, hk, key0_of(2 * pp + u),
                          &bars[Sm::kBarKF + s]);
          ++k_issued;
          if (!(ok = v_free())) break;
          mbar_arrive_expect_tx(&bars[Sm::kBarVF + s], nbk * KB * 8192);
          for (int u = 0; u < nbk; ++u)
            for (int kb = 0; kb < KB; ++kb)
              tma_load_4d(vt + (u * KB + kb) * 8192, &p.tm_v, 0, kb, hk, key0_of(2 * pp + u),
                          &bars[Sm::kBarVF + s]);
        } else {
          // boxes of box_rows rows, none of which crosses a page; only those
          // that hold a token of the sequence
          const int br = p.box_rows;
          int planes[2][64 / 16], nbox[2] = {0, 0};
          for (int u = 0; u < nbk && ok; ++u) {
            const int key0 = key0_of(2 * pp + u);
            nbox[u] = (min(kDenseBlock, p.Lk - key0) + br - 1) / br;
            for (int b = 0; b < nbox[u]; ++b) {
              const int blk = (key0 + b * br) / p.P;
              const int phys = blk < p.max_pp ? p.page_row[blk] : -1;
              if (phys < 0 || phys >= p.num_phys) {
                dt_set_err(err, blk < p.max_pp ? kDevBadPhys : kDevBadPage, hk, blk, phys);
                *fail = 1;
                ok = false;
                break;
              }
              planes[u][b & 3] = phys * p.Hkv + hk;
            }
          }
          if (!ok) break;
          const int bytes = (nbox[0] + nbox[1]) * KB * br * 128;
          mbar_arrive_expect_tx(&bars[Sm::kBarKF + s], bytes);
          for (int u = 0; u < nbk; ++u)
            for (int b = 0; b < nbox[u]; ++b)
              for (int kb = 0; kb < KB; ++kb)
                tma_load_4d(kt + kb * 16384 + u * 8192 + b * br * 128, &p.tm_k, 0,
                            (key0_of(2 * pp + u) + b * br) % p.P, kb, planes[u][b & 3],
                            &bars[Sm::kBarKF + s]);
          ++k_issued;
          if (!(ok = v_free())) break;
          mbar_arrive_expect_tx(&bars[Sm::kBarVF + s], bytes);
          for (int u = 0; u < nbk; ++u)
            for (int b = 0; b < nbox[u]; ++b)
              for (int kb = 0; kb < KB; ++kb)
                tma_load_4d(vt + (u * KB + kb) * 8192 + b * br * 128, &p.tm_v, 0,
                            (key0_of(2 * pp + u) + b * br) % p.P, kb, planes[u][b & 3],
                            &bars[Sm::kBarVF + s]);
        }
        ++v_issued;
      }
      // every copy lands before the CTA leaves (other roles may have given up)
      dt_drain(&bars[Sm::kBarQ], 0);
      for (int pp = max(0, k_issued - S); pp < k_issued; ++pp)
        dt_drain(&bars[Sm::kBarKF + pp % S], (pp / S) & 1);
      for (int pp = max(0, v_issued - S); pp < v_issued; ++pp)
        dt_drain(&bars[Sm::kBarVF + pp % S], (pp / S) & 1);
    }
  } else if (warp == Sm::kScanWarp) {
    // ---- V of edge blocks: values that are not finite (and rows behind the
    // sequence's end, whatever they hold) become zero before the products ----
    constexpr uint32_t kExp = Weights<T>::bf16 ? 0x7f807f80u : 0x7c007c00u;
    constexpr uint32_t kStep = Weights<T>::bf16 ? 0x00800080u : 0x04000400u;
    bool ok = true;
    for (int pp = 0; pp < np && ok; ++pp) {
      const int s = pp % S, nbk = min(2, n - 2 * pp);
      ok = __all_sync(0xffffffffu, dt_wait(&bars[Sm::kBarVF + s], (pp / S) & 1, fail));
      if (!ok) break;
      bool touched = false, bad = false;
      for (int u = 0; u < nbk; ++u) {
        const int key0 = key0_of(2 * pp + u);
        if (!is_edge(key0)) continue;
        uint8_t *vt = smem + Sm::kV + s * Sm::kStageBytes + u * KB * 8192;
        uint4 *w = reinterpret_cast<uint4 *>(vt);
        if (!p.paged) {
          constexpr int kBatch = 8;
#pragma unroll 1
          for (int c = lane; c < KB * 512; c += 32 * kBatch) {
            uint4 x[kBatch];
            uint32_t any = 0;
#pragma unroll
            for (int e = 0; e < kBatch; ++e) x[e] = w[c + 32 * e];
#pragma unroll
            for (int e = 0; e < kBatch; ++e)
              any |= nonfinite(x[e].x, kExp, kStep) | nonfinite(x[e].y, kExp, kStep) |
                     nonfinite(x[e].z, kExp, kStep) | nonfinite(x[e].w, kExp, kStep);
            if (any) {
              touched = bad = true;
#pragma unroll
              for (int e = 0; e < kBatch; ++e)
                w[c + 32 * e] = make_uint4(without_nonfinite(x[e].x, kExp, kStep),
                                           without_nonfinite(x[e].y, kExp, kStep),
                                           without_nonfinite(x[e].z, kExp, kStep),
                                           without_nonfinite(x[e].w, kExp, kStep));
            }
          }
        } else {
          const int keep = p.Lk - key0;  // rows of the sequence
          for (int c = lane; c < KB * 512; c += 32)
            if (((c & 511) >> 3) >= keep) {
              w[c] = make_uint4(0, 0, 0, 0);
              touched = true;
            }
        }
      }
      if (bad) misc[kMiscBad] = 1;
      if (touched) fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bars[Sm::kBarVC + s]);
        // a matrix that has no more pairs frees the stages here (the other one has
        // this pair or a later one); the pairs before its first it frees itself
        for (int m = 0; m < 2; ++m)
          if (pp >= pair_last(m)) {
            mbar_arrive(&bars[Sm::kBarKE + s]);
            mbar_arrive(&bars[Sm::kBarVE + s]);
          }
      }
    }
  } else if (warp >= Sm::kMmaWarp) {
    // ---- MMA issue for matrix m (the whole warp, one elected lane issuing) ----
    const int m = warp - Sm::kMmaWarp;
    const bool bf = Weights<T>::bf16;
    const uint32_t idesc_s = umma_idesc_f16(bf, 128, 64, 0, 0);  // Q . K^T, a block
    const uint32_t idesc_o = umma_idesc_f16(bf, 128, D, 0, 1);   // P . V: V MN-major
    const uint64_t dq = umma_desc_sw128(smem_u32(smem + Sm::kQ + m * KB * 16384), 16, 1024);
    const uint64_t dk = umma_desc_sw128(smem_u32(smem + Sm::kK), 16, 1024);
    // (V's 64-channel halves lie 8,192 bytes apart: one product spans all channels)
    const uint64_t dv = umma_desc_sw128(smem_u32(smem + Sm::kV), 8192, 1024);
    const uint64_t dl = umma_desc_sw128(smem_u32(smem + Sm::kL + m * 16384), 16, 1024);
    const uint32_t t_o = tmem + 256 + D * m;
    const int begin = pair_first(m), end = pair_last(m), dup = p.dup;
    auto wwait = [&](uint64_t *bar, uint32_t parity) {
      return __all_sync(0xffffffffu, dt_wait(bar, parity, fail));
    };
    bool ok = begin < end && wwait(&bars[Sm::kBarQ], 0), any = false;
    for (int pp = 0; pp < begin && ok; ++pp) {  // (every phase is seen, in order)
      if (!(ok = wwait(&bars[Sm::kBarKF + pp % S], (pp / S) & 1))) break;
      if (lane == 0) mbar_arrive(&bars[Sm::kBarKE + pp % S]);
      if (!(ok = wwait(&bars[Sm::kBarVC + pp % S], (pp / S) & 1))) break;
      if (lane == 0) mbar_arrive(&bars[Sm::kBarVE + pp % S]);
    }
    // the S side runs two blocks ahead of the P . V side: block su of pair sp, the
    // matrix's block sb (buffer sb & 1)
    int sp = begin, su = dup ? m : 0, sb = 0;
    auto issue_s = [&]() {
      if (sp >= end) return;
      const int s = sp % S;
      if ((dup || su == 0) && !(ok = wwait(&bars[Sm::kBarKF + s], (sp / S) & 1))) return;
      tc_fence_after();
      any = true;
      const uint64_t kt = dk + (uint64_t)((s * Sm::kStageBytes + su * 8192) >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t off = (uint64_t)(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4);
        umma_f16_warp(tmem + 128 * m + 64 * (sb & 1), dq + off, kt + off, idesc_s, kk > 0);
      }
      umma_commit_warp(&bars[Sm::kBarSF + 2 * m + (sb & 1)]);
      ++sb;
      if (dup || su == 1 || 2 * sp + 1 == n) {
        umma_commit_warp(&bars[Sm::kBarKE + s]);
        ++sp;
        su = dup ? m : 0;
      } else {
        su = 1;
      }
    };
    if (ok) issue_s();
    if (ok) issue_s();
    int blocks = 0;  // of this matrix so far
    for (int pp = begin; pp < end && ok; ++pp) {
      const int s = pp % S, u0 = dup ? m : 0, u1 = dup ? m + 1 : min(2, n - 2 * pp);
      if (!(ok = wwait(&bars[Sm::kBarVC + s], (pp / S) & 1))) break;
      for (int u = u0; u < u1; ++u, ++blocks) {
        const int buf = blocks & 1;
        if (!(ok = wwait(&bars[Sm::kBarPF + 2 * m + buf], (blocks >> 1) & 1))) break;
        tc_fence_after();
        const uint64_t vt = dv + (uint64_t)((s * Sm::kStageBytes + u * KB * 8192) >> 4);
        const uint32_t pa = tmem + 128 * m + 64 * buf;
#pragma unroll
        for (int part = 0; part < (kSplitP ? 2 : 1); ++part)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_f16_ts_warp(t_o, pa + 32 * part + 8 * kk, vt + (uint64_t)((kk * 2048) >> 4),
                             idesc_o, blocks > 0 || part > 0 || kk > 0);
        if (third) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_f16_warp(t_o, dl + (uint64_t)((kk * 32) >> 4), vt + (uint64_t)((kk * 2048) >> 4),
                          idesc_o, true);
        }
        umma_commit_warp(&bars[Sm::kBarOD + m]);
        if (u == u1 - 1) {
          umma_commit_warp(&bars[Sm::kBarVE + s]);
          if (pp == end - 1) umma_commit_warp(&bars[Sm::kBarOF + m]);
        }
        if (sp < end) {  // the next S goes where this P was
          if (!(ok = wwait(&bars[Sm::kBarOD + m], blocks & 1))) break;
          issue_s();
          if (!ok) break;
        }
      }
    }
    if (any) {  // every MMA of this warp done before the CTA frees its memory
      umma_commit_warp(&bars[Sm::kBarDR + m]);
      if (lane == 0) dt_drain(&bars[Sm::kBarDR + m], 0);
    }
  } else {
    // ---- softmax: one query row per thread ----
    const int m = warp >> 2;
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t t_o = lanes + 256 + D * m;
    const int begin = pair_first(m), end = pair_last(m);
    const float slope = kRule == kBias && p.rule.slopes && tok < p.Lq
                            ? p.rule.slopes[h_row] * 1.4426950408889634f
                            : 0.f;
    // a prompt's distances count from the row's nearest key, wherever it stands: one
    // constant less in every score of the row, and the bias of the keys that matter
    // keeps its bits (|t - pos| less the nearest key's distance is |t - nearest| for
    // every attended t; integers, as fp32 holds distances up to 2^24 only).  The
    // nearest key of a decode row is its own newest token, at distance 0.
    const int pos = p.paged ? p.Lk + (tok < p.Lq ? p.lens[tok] : 0) - 1
                            : min(max(p.pos0 + tok, rbeg), rend - 1);
    const float sc = kRule != kPlain ? 1.f : p.rule.scale_log2;
    const bool idle = __all_sync(0xffffffffu, rend == 0);  // rows that attend nothing
    float m_run = -CUDART_INF_F, l_run = 0.f;
    bool ok = true;
    int blocks = 0;
    for (int pp = begin; pp < end && ok; ++pp) {
      const int u1 = p.dup ? m + 1 : min(2, n - 2 * pp);
#pragma unroll 1
      for (int u = p.dup ? m : 0; u < u1; ++u, ++blocks) {
        const int buf = blocks & 1;
        ok = dt_wait(&bars[Sm::kBarSF + 2 * m + buf], (blocks >> 1) & 1, fail);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;  // the tensor-memory accesses are warp-wide
        tc_fence_after();
        if (idle) {  // what the products make of these rows is never read
          if (lane == 0) mbar_arrive(&bars[Sm::kBarPF + 2 * m + buf]);
          continue;
        }
        const uint32_t t_s = lanes + 128 * m + 64 * buf;
        const int key0 = key0_of(2 * pp + u);
        uint32_t s[64];
        tmem_ld64_sync(t_s, s);
        const bool edge = is_edge(key0);
        auto row_max = [&] {
          float mq[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) mq[k] = __uint_as_float(s[k]);
#pragma unroll
          for (int c = 4; c < 60; c += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mq[k] = fmax3f(mq[k], __uint_as_float(s[c + 2 * k]), __uint_as_float(s[c + 2 * k + 1]));
#pragma unroll
          for (int k = 0; k < 4; ++k) mq[k] = fmaxf(mq[k], __uint_as_float(s[60 + k]));
          return fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
        };
        // a cap alone, 16-bit output, largest scores within the polynomial's range:
        // the cap is monotonic, so the row's max is taken first and the polynomial
        // goes into the exponent (rows that attend nothing have no say in it: what
        // they become is never read)
        bool quick = false;
        float top = 0.f;
        if constexpr (kRule == kCap && !kSplitP) {
          if (p.rule.quick > 0.f && !edge) {
            top = row_max();
            quick = __all_sync(0xffffffffu, rend == 0 || (top <= p.rule.quick &&
                                                          top >= p.rule.quick_floor));
          }
        }
        if (kRule != kPlain && !quick) {
          if (kRule == kCap || p.rule.cap_out > 0.f) {
            if constexpr (kSplitP) {
              // the short polynomial when it holds for the warp's 64 x 32 scores (not
              // in edge blocks, where keys that no row attends would have a say)
              float big = edge ? CUDART_INF_F : 0.f;
#pragma unroll
              for (int c = 0; c < 64; c += 2)
                big = fmaxf(fmaxf(big, fabsf(__uint_as_float(s[c]))),
                            fabsf(__uint_as_float(s[c + 1])));
              if (__all_sync(0xffffffffu, rend == 0 || big <= p.rule.small)) {
#pragma unroll
                for (int c = 0; c < 64; c += 2) {
                  const float2 x = cap_small(
                      p.rule, make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])));
                  s[c] = __float_as_uint(x.x);
                  s[c + 1] = __float_as_uint(x.y);
                }
              } else {
#pragma unroll
                for (int c = 0; c < 64; ++c)
                  s[c] = __float_as_uint(cap_any(p.rule, __uint_as_float(s[c])));
              }
            } else if (!p.rule.rough) {
#pragma unroll
              for (int c = 0; c < 64; ++c)
                s[c] = __float_as_uint(cap_any(p.rule, __uint_as_float(s[c])));
            } else {
#pragma unroll
              for (int c = 0; c < 64; c += 2) {
                const float2 x = cap_16bit(
                    p.rule, make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])));
                s[c] = __float_as_uint(x.x);
                s[c + 1] = __float_as_uint(x.y);
              }
            }
          }
          if (kRule == kBias && p.rule.slopes) {
            // keys at or before every row of the warp: the distance needs no
            // absolute value, and the bias is a line over the block
            const float d0 = (float)(pos - key0);
            const float2 sc2 = f2_dup(p.rule.cap_out > 0.f ? 1.f : p.rule.scale_log2);
            if (__all_sync(0xffffffffu, rend == 0 || d0 >= 63.f)) {
              const float2 up = f2_dup(slope), b0 = f2_dup(-slope * d0);
#pragma unroll
              for (int c = 0; c < 64; c += 2) {
                const float2 t = f2_fma(make_float2((float)c, (float)(c + 1)), up, b0);
                const float2 x = f2_fma(
                    make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sc2, t);
                s[c] = __float_as_uint(x.x);
                s[c + 1] = __float_as_uint(x.y);
              }
            } else {
#pragma unroll
              for (int c = 0; c < 64; ++c)
                s[c] = __float_as_uint(
                    fmaf(-slope, fabsf(d0 - (float)c), __uint_as_float(s[c]) * sc2.x));
            }
          }
        }
        if (edge) {
          const int c0 = rbeg - key0, c1 = rend - key0;
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c < c0 || c >= c1) s[c] = 0xff800000u;  // -inf
        }
        if (!quick) top = row_max();
        const float mx = quick ? cap_quick(p.rule, f2_dup(top), f2_dup(0.f)).x : top * sc;
        const bool need = mx > m_run + kDtRescaleAbove;
        if (__any_sync(0xffffffffu, need)) {
          const float m_new = need ? mx : m_run;
          const float alpha = need ? (m_run == -CUDART_INF_F ? 0.f : exp2f(m_run - m_new)) : 1.f;
          if (blocks > 0) {  // O_m follows the new max once the block before has landed
            ok = dt_wait(&bars[Sm::kBarOD + m], (blocks - 1) & 1, fail);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32_sync(t_o + 32 * c, o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32(t_o + 32 * c, o);
            }
            tmem_wait_st();
          }
          l_run *= alpha;
          m_run = m_new;
        }
        // weights 2^(x - m + kWeightShift); a row that has met no key yet keeps
        // 2^(-inf - 0) = 0
        const float base = m_run == -CUDART_INF_F ? 0.f : m_run - kWeightShift;
        uint32_t hi_w[32];
        uint32_t lo_w[kSplitP ? 32 : 1];
        const float2 sc2 = f2_dup(sc), nm2 = f2_dup(-base);
        float2 ls[2] = {f2_dup(0.f), f2_dup(0.f)};
        uint32_t rest[kThird ? 4 : 1];
        if (third && blocks > 0) {  // the block before has been read from there
          ok = dt_wait(&bars[Sm::kBarOD + m], (blocks - 1) & 1, fail);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
        }
        auto weights = [&](auto exponent) {
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float2 x = exponent(
                make_float2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])));
            const float2 w = make_float2(ex2_approx(x.x), ex2_approx(x.y));
            ls[c & 1] = f2_add(ls[c & 1], w);
            if constexpr (kSplitP) Weights<T>::split(w, hi_w[c], lo_w[c]);
            else hi_w[c] = Weights<T>::round(w);
            if constexpr (kThird) {
              if (third) {
                rest[c & 3] = Weights<T>::rest(w, hi_w[c], lo_w[c]);
                if ((c & 3) == 3)
                  *reinterpret_cast<uint4 *>(smem + Sm::kL + m * 16384 + swz128(row, c >> 2)) =
                      make_uint4(rest[0], rest[1], rest[2], rest[3]);
              }
            }
          }
        };
        if (kRule == kCap && !kSplitP && quick)
          weights([&](float2 x) { return cap_quick(p.rule, x, nm2); });
        else
          weights([&](float2 x) { return f2_fma(x, sc2, nm2); });
        l_run += (ls[0].x + ls[1].x) + (ls[0].y + ls[1].y);
        tmem_st32(t_s, hi_w);
        if constexpr (kSplitP) tmem_st32(t_s + 32, lo_w);
        tmem_wait_st();
        if (third) fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[Sm::kBarPF + 2 * m + buf]);
      }
    }
    if (ok) {  // (without products, Q's copy must have landed: its tile is written next)
      ok = dt_wait(blocks > 0 ? &bars[Sm::kBarOF + m] : &bars[Sm::kBarQ], 0, fail);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
    }
    if (ok) {
      // ---- the warp's 32 rows, 128 bytes of channels at a time, through the
      // matrix's Q tile (its products are done) and from there by TMA, which
      // leaves out the rows behind the last query ----
      const bool live = tok < p.Lq, empty = rend == 0;
      const bool fix = *reinterpret_cast<volatile int *>(misc + kMiscBad) && live && !empty;
      const size_t pr = ((size_t)unit * p.nsplit + split) * kDenseRows + m * 128 + row;
      if (p.partial && live) p.part_ml[pr] = make_float2(m_run - kWeightShift, empty ? 0.f : l_run);
      const float inv = empty ? 0.f : p.partial ? 1.f : 1.f / l_run;
      const bool f32 = p.partial || p.out_f32;
      // two buffers of [32][128 B], 16-byte pieces swizzled by the row
      uint8_t *stage = smem + Sm::kQ + m * KB * 16384 + (warp & 3) * (KB * 4096);
      const int at_h = p.partial ? 0 : h0, at_row = p.partial ? (int)(pr - lane) : tok - (lane >> lhp);
      int turn = 0;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t r[32];
        __syncwarp();
        if (blocks > 0) {
          tmem_ld32_sync(t_o + 32 * c, r);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) r[e] = 0u;
        }
        float f[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) f[e] = empty ? 0.f : __uint_as_float(r[e]) * inv;
        if (fix) {
          // the values that the scan took out, back into the rows that attend them
          const T *vg = static_cast<const T *>(p.v) + (size_t)hk * D + 32 * c;
          const int k1 = min(rend, (kb0 + n) * kDenseBlock);
          for (int t = max(rbeg, kb0 * kDenseBlock); t < k1; ++t) {
            if (!is_edge(t / kDenseBlock * kDenseBlock)) {
              t = (t / kDenseBlock + 1) * kDenseBlock - 1;
              continue;
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float x = Weights<T>::to_f(vg[(size_t)t * p.v_stride + e]);
              if (!isfinite(x)) f[e] += x;
            }
          }
        }
        uint8_t *buf;
        if (f32) {
          // (D 64 has one buffer of 4,096 bytes per warp)
          if (turn >= KB) {
            if (lane == 0) bulk_wait_read<KB - 1>();
            __syncwarp();
          }
          buf = stage + (turn % KB) * 4096;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<float4 *>(buf + swz128(lane, e)) =
                make_float4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]);
        } else {
          buf = stage + (c >> 1) * 4096;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<uint4 *>(buf + swz128(lane, 4 * (c & 1) + e)) =
                make_uint4(Weights<T>::round(make_float2(f[8 * e], f[8 * e + 1])),
                           Weights<T>::round(make_float2(f[8 * e + 2], f[8 * e + 3])),
                           Weights<T>::round(make_float2(f[8 * e + 4], f[8 * e + 5])),
                           Weights<T>::round(make_float2(f[8 * e + 6], f[8 * e + 7])));
          if (!(c & 1)) continue;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_4d(&p.tm_out, buf, 0, f32 ? c : c >> 1, at_h, at_row);
          bulk_commit();
        }
        ++turn;
      }
      if (lane == 0) bulk_wait<0>();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && *fail) dt_set_err(err, kDevTimeout, hk, tile, split);  // (an earlier error stays)
  if (warp == Sm::kMmaWarp) tmem_dealloc(tmem, Sm::kAlloc);
}

// ---- joining the splits of a prompt's rows --------------------------------------
// One warp per query row (token, head): M = max m_s, out = sum 2^(m_s - M) o_s
// / sum 2^(m_s - M) l_s.
template <typename T, int D>
__global__ void __launch_bounds__(256) dense_prompt_combine_kernel(
    const __grid_constant__ DenseTcParams p, void *out) {
  pdl_wait();
  pdl_launch_dependents();
  const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (w >= (long long)p.Lq * p.Hq) return;
  const int tok = (int)(w / p.Hq), h = (int)(w % p.Hq);
  const int hk = h / p.G, hg = (h % p.G) >> p.lhp;
  const int rt = p.dup ? 128 : kDenseRows, ns = p.nsplit * kDenseRows / rt;
  const int tpt = rt >> p.lhp, tile = tok / tpt;  // (heads per matrix: a power of two)
  const int r = ((tok % tpt) << p.lhp) + (h & ((1 << p.lhp) - 1));
  const size_t unit = (size_t)tile * p.Hkv * p.HG + hk * p.HG + hg;
  const float2 *ml = p.part_ml + unit * ns * rt + r;
  const float *po = p.part_o + (unit * ns * rt + r) * D;
  float M = -CUDART_INF_F;
  float2 mine[kDenseMaxSplits / 32];
#pragma unroll
  for (int k = 0; k < kDenseMaxSplits / 32; ++k) {
    const int s = lane + 32 * k;
    mine[k] = s < ns ? ml[(size_t)s * rt] : make_float2(-CUDART_INF_F, 0.f);
    M = fmaxf(M, mine[k].x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float base = M == -CUDART_INF_F ? 0.f : M;
  float L = 0.f, f[kDenseMaxSplits / 32];
#pragma unroll
  for (int k = 0; k < kDenseMaxSplits / 32; ++k) {
    f[k] = lane + 32 * k < ns ? exp2f(mine[k].x - base) : 0.f;
    L += mine[k].y * f[k];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  constexpr int E = D / 32;
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int s = 0; s < ns; ++s) {
    // a split that holds none of the row's keys left zeros (or nothing to weigh)
    const float fs = __shfl_sync(0xffffffffu, s < 32 ? f[0] : f[kDenseMaxSplits / 32 - 1], s & 31);
    const float *o = po + (size_t)s * rt * D + lane * E;
    float v[E];
    if constexpr (E == 4) *reinterpret_cast<float4 *>(v) = __ldcs(reinterpret_cast<const float4 *>(o));
    else *reinterpret_cast<float2 *>(v) = __ldcs(reinterpret_cast<const float2 *>(o));
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(v[e], fs, acc[e]);
  }
  bool empty;  // (a row whose interval holds no key is zero, one whose weights vanish is not)
  if (p.key_begin) {
    empty = max(p.key_begin[tok], 0) >= min(p.key_end[tok], p.Lk);
  } else {
    empty = min(p.pos0 + tok + 1, p.Lk) <= 0;
  }
  const float inv = empty ? 0.f : 1.f / L;
  const size_t at = ((size_t)tok * p.Hq + h) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] *= inv;
  if (p.out_f32) {
    float *o = static_cast<float *>(out) + at;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = acc[e];
  } else {
    uint32_t *o = reinterpret_cast<uint32_t *>(static_cast<T *>(out) + at);
#pragma unroll
    for (int e = 0; e < E; e += 2) o[e / 2] = Weights<T>::round(make_float2(acc[e], acc[e + 1]));
  }
}

// ---- intervals of packed documents ------------------------------------------------
// Token t of document i (offsets[i] <= t < offsets[i + 1]) attends from the
// document's start to the later of itself and the document's prefix; tokens
// outside every document attend nothing.
__global__ void __launch_bounds__(256) document_ranges_kernel(const int *offsets,
                                                              const int *prefix, int n_docs,
                                                              int total, int *kb, int *ke) {
  pdl_wait();
  pdl_launch_dependents();
  const int t = blockIdx.x * 256 + threadIdx.x;
  if (t >= total) return;
  int lo = 0, hi = n_docs;  // the last document that starts at or before t
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (offsets[mid] <= t) lo = mid + 1;
    else hi = mid;
  }
  const int i = lo - 1;
  int b = 0, e = 0;
  if (i >= 0 && t < offsets[i + 1]) {
    b = max(offsets[i], 0);
    const int seen = prefix ? max(prefix[i], 0) : 0;
    const int end = min(offsets[i + 1], total);
    e = max(t + 1, b + min(seen, end - b));
  }
  kb[t] = b;
  ke[t] = e;
}

template <typename T, int D, int kParts, int kRule>
cudaError_t launch_dt_r(const DenseTcParams &p, cudaStream_t st) {
  auto k = dense_tc_kernel<T, D, kParts, kRule>;
  static std::atomic<uint64_t> ready{0};
  using Sm = DtSmem<D, kParts == 3>;
  const cudaError_t e = allow_smem(k, Sm::kBytes, &ready);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, p.tiles * p.nsplit * p.Hkv * p.HG, Sm::kThreads, (size_t)Sm::kBytes, st, p);
}

template <typename T, int D, int kParts>
cudaError_t launch_dt(const DenseTcParams &p, cudaStream_t st) {
  if (p.rule.slopes) return launch_dt_r<T, D, kParts, kBias>(p, st);
  return p.rule.cap_out > 0.f ? launch_dt_r<T, D, kParts, kCap>(p, st)
                              : launch_dt_r<T, D, kParts, kPlain>(p, st);
}

template <typename T, int D>
cudaError_t launch_dt_p(const DenseTcParams &p, bool split_p, cudaStream_t st) {
  if (!split_p) return launch_dt<T, D, 1>(p, st);
  if constexpr (Weights<T>::bf16)
    return launch_dt<T, D, 3>(p, st);
  else
    return launch_dt<T, D, 2>(p, st);
}

template <typename T>
cudaError_t launch_dt_d(const DenseTcParams &p, int d, bool split_p, cudaStream_t st) {
  return d == 64 ? launch_dt_p<T, 64>(p, split_p, st) : launch_dt_p<T, 128>(p, split_p, st);
}

}  // namespace

cudaError_t launch_dense_tc(const DenseTcParams &p, int dtype, int d, bool split_p,
                            cudaStream_t st) {
  return dtype == 0 ? launch_dt_d<__half>(p, d, split_p, st)
                    : launch_dt_d<__nv_bfloat16>(p, d, split_p, st);
}

cudaError_t launch_dense_prompt_combine(const DenseTcParams &p, int dtype, int d, void *out,
                                        cudaStream_t st) {
  const int grid = (int)(((long long)p.Lq * p.Hq + 7) / 8);
  if (dtype == 0)
    return d == 64 ? launch_pdl(dense_prompt_combine_kernel<__half, 64>, grid, 256, 0, st, p, out)
                   : launch_pdl(dense_prompt_combine_kernel<__half, 128>, grid, 256, 0, st, p, out);
  return d == 64
             ? launch_pdl(dense_prompt_combine_kernel<__nv_bfloat16, 64>, grid, 256, 0, st, p, out)
             : launch_pdl(dense_prompt_combine_kernel<__nv_bfloat16, 128>, grid, 256, 0, st, p, out);
}

// The current device's error word, cleared.
cudaError_t dense_error_word(int (&w)[4]) {
  cudaError_t e = cudaMemcpyFromSymbol(w, g_dense_err, sizeof w);
  if (e != cudaSuccess || w[0] == 0) return e;
  const int zero[4] = {0, 0, 0, 0};
  return cudaMemcpyToSymbol(g_dense_err, zero, sizeof zero);
}

cudaError_t launch_document_ranges(const int *offsets, const int *prefix, int n_docs, int total,
                                   int *key_begin, int *key_end, cudaStream_t st) {
  return launch_pdl(document_ranges_kernel, (total + 255) / 256, 256, 0, st, offsets, prefix,
                    n_docs, total, key_begin, key_end);
}

}  // namespace spd
