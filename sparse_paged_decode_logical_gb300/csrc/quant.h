// Internal interface of the rotary kernels, the cache in 8 or 4 bits and the
// decode attention over it (rotary.cu, quant_cache.cu, quant_decode.cuh).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "dense.h"
#include "spd.h"
#include "spd_internal.h"

namespace spd {

// ---- how a quantised cache is laid out ---------------------------------------------
// A (page, kv head) holds tiles of 16 tokens, keys and values of one tile side by side:
//   [K codes][K parameters][V codes][V parameters]
// Parameters: per token the lowest values of its groups, then their steps, in the cache's
// type.  Codes lie in the order in which a warp's m16n8k16 operands take them, so that a
// lane's whole operand is one 16-byte load and a few masks away; g = lane / 4, t = lane % 4:
//   K  word of k-step s holds tokens g and g + 8, channels 32 (s / 2) + 8 t + 4 (s % 2) +
//      {0, 1, 2, 3}
//   V  word of m-tile j holds tokens 2t, 2t + 1, 2t + 8, 2t + 9, channels 32 (j / 2) + 4 g +
//      2 (j % 2) + {0, 1}
// Every byte belongs to one token, so that single tokens are written with byte stores.
//   4 bits  K: bytes 0 and 2 are token g, 1 and 3 token g + 8; low nibbles channels 0 and
//           1, high ones 2 and 3.  V: bytes 0, 2, 1, 3 are the four tokens; low nibble
//           channel 0, high 1.
//   8 bits  two words.  K: bytes 0 and 2 are token g, 1 and 3 token g + 8; channels 0 and 1
//           in the first word, 2 and 3 in the second.  V: bytes 0 and 2 channel 0, 1 and 3
//           channel 1; tokens 2t and 2t + 1 in the first word, 2t + 8 and 2t + 9 in the second.
// Word w of a lane lies at ((w / 4) 32 + lane) 4 + w % 4.
constexpr int kQuantTile = 16;  // tokens

template <int D, int BITS>
struct QuantTile {
  static constexpr int kGroup = BITS == 8 ? D : 32;  // channels of a group
  static constexpr int kGroups = D / kGroup;
  static constexpr int kLevels = (1 << BITS) - 1;
  static constexpr int kWords = D / 16 * (BITS / 4);  // of a lane, for K or for V
  static constexpr int kCodes = kWords * 128;         // bytes
  static constexpr int kTokenParams = kGroups * 4;    // bytes
  static constexpr int kParams = kTokenParams * kQuantTile;
  static constexpr int kHalf = kCodes + kParams;  // K or V
  static constexpr int kBytes = 2 * kHalf;
};
inline size_t quant_tile_bytes(int d, int bits) {
  return bits == 8 ? 2 * ((size_t)d * 16 + 64) : 2 * ((size_t)d * 8 + (size_t)d / 32 * 64);
}

constexpr int kQuantSeqs = 256;  // sequences described per parameter block
constexpr int kQuantCtas = 256;  // most CTAs of an attention launch
constexpr int kQuantWarps = 12;  // per CTA
constexpr int kQuantWriteWarps = 4;  // of a writing CTA
constexpr int kQuantPerSm = 1;   // CTAs that an SM holds

// Tiles that a warp takes in one step: what a step costs besides is shared by them, and their
// chains of products fill one another's gaps (half as many: 131,072 tokens of 128 channels in 4 bits
// 44.0 instead of 40.3 us, 64 x 3,000 of 64 channels 35.5 instead of 34.4).
constexpr int quant_step_tiles(int d) { return d == 64 ? 4 : 2; }

// A share of a unit: [G][d] sums, [G] (reference, sum of weights).
constexpr int quant_slot_bytes(int d, int G) { return (G * d * 4 + G * 8 + 15) / 16 * 16; }

// ---- rotary ------------------------------------------------------------------------
struct RotaryParams {
  spd_rotary_table table;
  const void *q, *k;  // [n][heads][d] at strides, k may be null
  void *q_out, *k_out;
  long long q_stride, k_stride, q_out_stride, k_out_stride;  // elements between tokens
  const int *positions;  // [axes][axis_stride]
  long long axis_stride;
  int n, hq, hkv, inverse;
  int tokens_per_cta;  // at most kRotaryTokens
};
constexpr int kRotaryTokens = 4;
// Tokens n_tokens by n_tokens of sequences that begin at first[i].
struct RotaryPlaces {
  int n_tokens;
  int first[kQuantSeqs];
};
// places null: positions as p gives them
cudaError_t launch_rotary(const RotaryParams &p, const RotaryPlaces *places, int dtype,
                          cudaStream_t st);

// ---- writing and reading back --------------------------------------------------------
struct QuantSeq {
  int slot;
  int first;  // first token of this call's
  int off;    // writing and reading: the tiles of the sequences before
};
struct QuantAppendSeq {
  int slot, first, off;  // as QuantSeq
  int page, pages, upd;  // its pages [page, page + pages) are upd[upd], ...: not in the table yet
};
constexpr int kQuantUpdates = 128;
struct QuantAppendParams {
  spd_rotary_table table;  // (with rotate)
  const void *k, *v, *q;   // [n_seqs][n_tokens][heads][d], tokens at strides
  void *q_out;             // [n_seqs][n_tokens][hq][d]
  long long k_stride, v_stride, q_stride;
  const int *positions;  // [axes][n_seqs][n_tokens] or null: a token's place in its sequence
  void *pool;
  int *page_table;
  int *err;
  int n_seqs, n_tokens, hq, hkv, P, max_pp, num_phys;
  int n_updates;   // entries of the page table that this launch writes, any sequence's
  PtUpdate updates[kQuantUpdates];
  int total_seqs;  // sequences of the whole call (positions' axes are this far apart)
  int seq0;        // sequences before this launch's
  int rotate;      // keys, and hq heads of queries
  int tiles;       // of all sequences
  int parts;       // CTAs per tile, each with an equal share of the heads
  QuantAppendSeq seqs[kQuantSeqs];
};
cudaError_t launch_quant_append(const QuantAppendParams &p, int dtype, int d, int bits,
                                cudaStream_t st);

struct QuantReadParams {
  const void *pool;
  void *k, *v;  // [n_seqs][n_tokens][hkv][d]
  const int *page_table;
  int *err;
  int n_seqs, n_tokens, hkv, P, max_pp, num_phys;
  int tiles;
  QuantSeq seqs[kQuantSeqs];
};
cudaError_t launch_quant_read(const QuantReadParams &p, int dtype, int d, int bits,
                              cudaStream_t st);

// ---- attention ---------------------------------------------------------------------
// The tiles of all units (sequence, kv head) in a row, a unit's `stride` apart; warp w of the
// launch takes the tiles [w per_warp, (w + 1) per_warp).
struct QuantAttendSeq {
  int slot, L;
  int first;   // first attended token
  int tiles;   // that hold attended tokens
  int stride;  // >= tiles: places a unit takes in the row
  int off;     // place of the sequence's first unit
};
struct QuantAttendParams {
  const void *pool;
  const void *q;  // [n][hq][d]
  void *out;      // [n][hq][d], fp32 or the cache's type
  const int *page_table;
  char *parts;   // [2 x CTAs][quant_slot_bytes]: of units that several CTAs hold parts of
  char *firsts;  // [CTAs][warps][quant_slot_bytes]: of units that a warp ends before its last
  int *tickets;     // [n][hkv], zero before and after
  int *err;
  ScoreRule rule;
  int out_f32, precise_cap;
  int n, hkv, P, max_pp, num_phys;
  int per_warp, total;  // places
  int ctas;
  QuantAttendSeq seqs[kQuantSeqs];
};
cudaError_t launch_quant_attend_f16(const QuantAttendParams &p, int d, int bits, int G,
                                    cudaStream_t st);
cudaError_t launch_quant_attend_bf16(const QuantAttendParams &p, int d, int bits, int G,
                                     cudaStream_t st);

}  // namespace spd
