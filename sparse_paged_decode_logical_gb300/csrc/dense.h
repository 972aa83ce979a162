// Internal interface of the dense attention kernels: prompt attention with
// score rules and key intervals (dense_tc.cu), decode attention of a batch
// over a shared prefix and each sequence's own tokens (dense_tc.cu for the
// prefix, dense_decode.cu for the rest), and eviction (evict.cu).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "spd.h"

namespace spd {

constexpr int kDenseBlock = 64;      // keys per block of the tensor-core kernel
constexpr int kDenseRows = 256;      // query rows of one of its CTAs (two matrices of 128)
constexpr int kDenseSeqs = 256;      // sequences described per parameter block
constexpr int kDecodeTile = 16;      // keys per tile of the decode kernel
constexpr int kDecodeRows = 16;      // query rows of one of its work items
constexpr int kFewKeys = 128;        // keys per step of dense_few
constexpr int kDenseMaxSplits = 64;  // key splits of one unit
constexpr int kOwnMaxSplits = 256;   // splits of one sequence's own tokens

// Weights are held as 2^(x - m + 7): a running max m may lag 2^8 behind a row's
// largest score, so that weights stay below fp16's 2^16, and what fp16 loses
// below its normal range is 2^-32 of the largest weight (without the shift
// 2^-25).  Sums carry the same factor, and partial sums come with m - 7.
constexpr float kWeightShift = 7.f;

// Allows a kernel its dynamic shared memory on the current device, once per
// device (`ready`: a bit for each of the first 64).
template <typename K>
inline cudaError_t allow_smem(K kernel, int bytes, std::atomic<uint64_t> *ready) {
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  const uint64_t bit = device < 64 ? 1ull << device : 0;
  if (ready->load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) ready->fetch_or(bit, std::memory_order_release);
  return e;
}

// The score of a query row and a key, in base-2 units ready for exp2:
//   s = scale q.k; softcap: s = cap tanh(s / cap); bias: s -= slope |distance|
struct ScoreRule {
  float scale_log2;      // scale * log2(e)
  float z_in;            // scale / cap
  float e_in;            // 2 log2(e) scale / cap
  float small;           // scores q.k up to this are within tanh's short polynomial
  float cap_out;         // cap * log2(e); 0: no cap
  int rough;             // 2^-22 of the cap does not show in 16-bit weights
  float poly[5];         // cap_out times tanh(z) / z as a polynomial in z^2, |z| <= 0.6
  float quick, quick_floor;  // a cap of 30 or more without slopes: rows whose largest q.k lies
                             // between these may take quick_poly; quick 0: none
  float quick_poly[5];   // the capped score over q.k as a polynomial in (q.k)^2
  const float *slopes;   // [Hq] or null
};

// Tensor-core kernel.  Row r of a unit (head group hg of kv head hk, tile): token (or sequence)
// tile * 256 / HP + r / HP, query head hk G + hg HP + r % HP.
struct DenseTcParams {
  CUtensorMap tm_q;        // {64, d / 64, Hq, tokens}, box {64, 1, HP, 128 / HP}
  CUtensorMap tm_k, tm_v;  // prompt: {64, d / 64, Hkv, Lk}, box {64, 1, 1, 64};
                           // paged: {64, P, d / 64, planes}, box {64, box_rows, 1, 1}
  CUtensorMap tm_out;      // final: {64 (fp32: 32), .., Hq, Lq}, box {.., 1, HP, 32 / HP};
                           // partials [unit][split][256][d]: {32, d / 32, 1, rows}, box {32, 1, 1, 32}
  int partial;             // splits: unnormalised sums to tm_out, statistics to part_ml
  const float *part_o;     // the partials (combining kernel)
  float2 *part_ml;         // [unit][split][256]  (row max in base-2 units, sum)
  const void *v;           // prompt: V itself (rows at v_stride elements), for non-finite values
  long long v_stride;
  const int *key_begin, *key_end;  // [Lq] or null: causal
  const int *page_row;     // paged: the sequence's row of the page table
  int *err;                // error word, or null: the library's own
  ScoreRule rule;
  int paged;
  int out_f32;             // type of out (paged: of what the splits become)
  int Lq, Lk, Hq, Hkv, G, lhp, HG;  // HP = 2^lhp heads per matrix, HG = G / HP head groups
  int tiles, nsplit;
  int dup;                 // both matrices hold the same 128 rows, each takes every second block
  int P, max_pp, num_phys, box_rows;
  int pos0;                // prompt: position of query 0 (Lk - Lq)
  int lens[kDenseSeqs];    // paged: tokens of each sequence after the prefix
};

cudaError_t launch_dense_tc(const DenseTcParams &p, int dtype, int d, bool split_p,
                            cudaStream_t st);
// Joins the splits of a prompt's units into out.
cudaError_t launch_dense_prompt_combine(const DenseTcParams &p, int dtype, int d, void *out,
                                        cudaStream_t st);
cudaError_t dense_error_word(int (&w)[4]);  // the current device's, cleared
cudaError_t launch_document_ranges(const int *offsets, const int *prefix, int n_docs, int total,
                                   int *key_begin, int *key_end, cudaStream_t st);

// Decode kernel: one CTA per work item.  Items [0, prefix_items) belong to the
// prefix (kv head, row group of 16, split), the rest to the sequences
// (sequence, kv head, split).
struct DecodeSeq {
  int slot, L;
  int item_off;  // first item, relative to the own items
  int ns;        // splits per kv head (0: no tokens)
  int tpi;       // tiles per split
  long long l_off;  // tokens (rounded up to 4) of the sequences before: its logits' place
};
struct DenseDecodeParams {
  CUtensorMap tm_k, tm_v;  // {64, P, d / 64, planes}, box {64, 16, d / 64, 1}
  const void *q;           // [n][Hq][d]
  void *out;               // [n][Hq][d], fp32 or T
  float *part_o;           // own items: [item][G][d]
  float2 *part_ml;         // [item][G]
  // prefix: [unit = row tile x kv head][split][prefix_rows][d], prefix_rows =
  // 256 or 128 (dense_tc), n G (dense_few) or 16 (decode kernel)
  float *pre_o;
  float2 *pre_ml;
  float *logits;           // per sequence [Hkv][G][own tokens rounded up to 4] from l_off Hkv G:
                           // base-2 scores of own tokens, or null
  const float *w_in;       // [n][Hkv][w_stride] or null
  float *w_out;
  const int *page_table;
  int *tickets;            // [n][Hkv], zero before and after: the last item of a (sequence,
                           // kv head) joins its splits; null: a combining kernel does
  int *err;
  ScoreRule rule;
  long long w_stride;
  int out_f32;
  int n, Hq, Hkv, G, P, max_pp, num_phys;
  int prefix_slot, prefix_len, prefix_items, prefix_ns, prefix_tpi, prefix_rows;
  int own_items;
  int precise;             // outputs that show 2^-22 of the cap (fp32, weights)
  int follow;              // the kernel before is another one of this call
  int w_chunks;            // weight CTAs per (sequence, kv head)
  int box_rows;            // dense_few: rows of a box
  DecodeSeq seqs[kDenseSeqs];
};
static_assert(sizeof(DenseDecodeParams) <= 32764, "parameter block too large");

cudaError_t launch_dense_decode(const DenseDecodeParams &p, int dtype, int d, cudaStream_t st);
// The prefix's items alone, for 9 to 32 rows (p.prefix_rows = n G of them, one
// unit per kv head) of 128 channels, on the tensor cores: tm_k, tm_v {64, P, 2,
// planes}, boxes {64, box_rows, 1, 1}, tiles of kFewKeys.
cudaError_t launch_dense_few(const DenseDecodeParams &p, int dtype, cudaStream_t st);
cudaError_t launch_dense_decode_combine(const DenseDecodeParams &p, int dtype, int d,
                                        cudaStream_t st);

struct EvictSeq {
  int src, dst;  // sequence slots
  int L, m;      // tokens before, tokens kept
};
struct EvictParams {
  void *k_pool, *v_pool, *meta;
  const int *page_table;
  const float *weights;   // [n][Hkv][w_stride]
  int *kept;              // [n][Hkv][keep]
  float *kept_weights;    // [n][Hkv][keep] or null
  int *err;
  long long w_stride;
  int n, Hkv, keep, recent, ell, P, R, max_pp, num_phys, kv_fp8;
  int P_log2;             // log2(P), -1 if P is no power of two
  EvictSeq seqs[kDenseSeqs];
};
cudaError_t launch_evict(const EvictParams &p, int dtype, int d, int sms, cudaStream_t st);

}  // namespace spd
