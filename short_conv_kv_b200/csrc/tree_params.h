// Arguments and launch constants of the drafted-tree kernels, shared by the
// kernels and the host code that launches them.
#pragma once
#include "common.cuh"

namespace sconv {

constexpr int kFlagTree = 16;
constexpr int kFlagContext = 32;
constexpr int kMaxDraft = 128;
constexpr int kMaskWords = kMaxDraft / 32;
constexpr int kMaxQueryHeads = 1 << 15;  // the host refuses more
// Query rows of a K/V head at most: a unit of this many is one a (sequence, head).
constexpr int kAllRows = kMaxDraft * kMaxQueryHeads;

struct PagedSeqs {
  const int32_t* cu;       // [num_seqs + 1]; nullptr: no drafted tokens
  const int32_t* parents;  // [num_tokens]
  const int32_t* lens;     // [num_seqs]
  const int32_t* table;    // [num_seqs, table_width], rows table_stride apart
  int64_t table_stride;
  int64_t capacity;  // table_width * page_size, at most 2^31 - 1
  int64_t num_tokens;
  int num_seqs;
  int max_draft;
  int num_pages;
  int page_size;
  uint32_t page_mul;  // p / page_size = (umulhi(p, mul) + p) >> shift, p < 2^31
  uint32_t page_shift;
  int64_t stride_page;  // elements
  int64_t stride_slot;
  int64_t stride_head;
  uint32_t page8;  // stride_page and stride_slot in units of 8 elements
  uint32_t slot8;
  int* err;
};

// Raw cache pointers: bf16 rows, or MXFP8 codes with their scales.
struct CacheParts {
  uint8_t* k;
  uint8_t* v;
  uint8_t* ks;
  uint8_t* vs;
  int ks_packed;      // a row's D/32 K scales can be loaded at once (aligned)
  int scales_packed;  // the same of V's as well
  int words;          // a head's scales begin at the same byte of a 4-byte word in every row
};

struct TreeStepParams {
  StepParams s;  // k, v, taps, gammas, state, slots, caches (cu_seqlens: drafted tokens)
  const int32_t* parents;
};

struct AcceptParams {
  PagedSeqs q;
  CacheParts c;
  int mx;
  int H;
  int D;
  const int32_t* leaves;
  int32_t* new_lens;
  float* weights;  // [S, H, ...] or nullptr
  int64_t w_seq;
  int64_t w_head;
  const uint16_t* k;  // raw rows
  const uint16_t* v;
  int64_t row_stride;
  int W;
  uint16_t* state;
  const int32_t* state_indices;
  int64_t pool;
  const int64_t* state_pos;
};

constexpr float kLog2e = 1.4426950408889634f;

// Attention: warps of attend_rows_kernel, and the keys they take a round.
constexpr int kRowsWarps = 4;
constexpr int kRowsTile = 16 * kRowsWarps;

struct AttendParams {
  PagedSeqs s;
  CacheParts c;
  const uint16_t* q;  // bf16, token stride q_tok, head stride q_head (elements)
  int64_t q_tok;
  int64_t q_head;
  uint16_t* out;
  int64_t o_tok;
  int64_t o_head;
  float* lse;  // [num_tokens, HQ], or nullptr
  int HQ;
  int H;
  int g;
  float scale_log2;  // scale * log2(e)
  // workspace: step prefix of the sequences [num_seqs + 2], then per CTA two
  // partial results of R rows: o (fp32 [R, D]) and (m, l)
  int64_t* prefix;
  float* part_o;
  float2* part_ml;
  int parts;  // CTAs that share the tiles
};

constexpr int kWeighWarps = 4;

struct WeighParams {
  AttendParams a;  // q, K cache, sequences, lse (read)
  float* weights;
  int64_t w_seq;
  int64_t w_head;
};

constexpr int kSelectThreads = 1024;
constexpr int kMoveThreads = 512;
constexpr int kMaxCluster = 8;

struct EvictParams {
  PagedSeqs q;
  CacheParts c;
  int mx;
  int H;
  int D;
  const float* weights;  // [S, H, ...]
  int64_t w_seq;
  int64_t w_head;
  float* weights_out;  // or nullptr
  int64_t o_seq;
  int64_t o_head;
  int keep;
  int sinks;
  int recent;
  int32_t* kept;  // [S, H, keep]
  int32_t* new_lens;
};

}  // namespace sconv
