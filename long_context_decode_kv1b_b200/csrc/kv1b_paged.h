// kv1b_paged.h -- internal interface of the paged-cache kernels: the block format, parameter blocks
// and launchers.
//
// A block holds 32 tokens of one kv-head in 3,200 contiguous bytes, so that one untiled bulk copy
// brings everything a warp needs for its tokens and a page, a power of two of tokens from 32 on, is a row of
// blocks.  Inside a block the planes are laid out for the attend's tensor-core fragments:
//   sign bits  row 8 i + 2 t + e is token 8 t + 2 i + e, so that the eight rows of score product i are
//              128 contiguous bytes (one ldmatrix) and lane t of a quad receives the logits of tokens
//              8 t .. 8 t + 7, the tokens of its code words;
//   codes      nibbles p and p + 4 of word w are tokens 8 w + 2 p and 8 w + 2 p + 1, so that one mask
//              of a word gives a pair of neighbouring tokens in the two halves of a register.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "kv1b.h"
#include "kv1b_launch.h"

namespace kv1b {

constexpr int kBlkTok = KV1B_PAGED_BLOCK_TOKENS;
constexpr int kBlkBytes = KV1B_PAGED_BLOCK_BYTES;
constexpr int kBlkOffNc = 512;      // f32 [32]  N / C
constexpr int kBlkOffScale = 640;   // f16 [4][32]
constexpr int kBlkOffMin = 896;     // f16 [4][32]
constexpr int kBlkOffCodes = 1152;  // u32 [128][4]
static_assert(kBlkTok == 32 && kBlkOffCodes + KV1B_HEAD_DIM * 16 == kBlkBytes && kBlkBytes % 16 == 0, "block layout");

struct PagedView {
  uint8_t* pages;
  const float* signs;
  int32_t* status;     // optional
  int32_t num_pages, Hkv;
  int32_t bpp_shift;   // log2 of the blocks per page
};

struct PagedAppendParams {
  PagedView c;
  const void* k;
  const void* v;
  int64_t k_st, k_sh, v_st, v_sh;  // element strides: token, head
  int32_t dtype;
  int32_t T, B;
  const int32_t* cu;       // [B + 1] first row of each sequence's new tokens
  const int32_t* start;    // [B] tokens each sequence holds already
  const int32_t* table;    // [B][table_stride]
  int64_t table_stride;
  int32_t max_pages;
  // rotary positions (cos_sin null: none)
  const float* cos_sin;    // [positions][rot]: cos of pair i at i, sin at rot / 2 + i
  int32_t cs_rows, rot, interleaved;
  int32_t sec0, sec01;     // pairs below sec0 take axis 0, below sec01 axis 1, the others axis 2
  const int32_t* pos;      // [axes][pos_stride]
  int64_t pos_stride;
  // queries to rotate (q null: none)
  const void* q;
  void* q_out;
  int64_t q_st, q_sh, qo_st, qo_sh;
  int32_t Hq;
  int32_t groups;          // bound of the 8-token groups of all sequences
  int32_t sms;
};

struct PagedAttendParams {
  PagedView c;
  const void* q;
  int32_t q_dtype;
  int32_t Hq, B;
  float scale;
  const int32_t* table;
  int64_t table_stride;
  int32_t max_pages;
  const int32_t* lengths;
  int32_t window, sinks;
  int32_t packed;          // first sequences of the plan that are the shared prefix, each for up to 8 rows of every
                           // kv-head's matrix (below); then the B sequences' own tokens
  const int32_t* prefix_pages;  // optional shared prefix: its pages and (device) token count
  const int32_t* prefix_len;
  int32_t max_prefix_pages;
  void* out;               // q_dtype [B][Hq][128]
  float* part;             // [ctas][2][G][2 + 128]
  float* first;            // [ctas][kAttendWarps][G][2 + 128]: ends of segments inside a warp's run
  float* rows;             // null, or [B][Hq][2 + 128] and, packed, [Hkv][B G][2 + 128]: whole segments leave
                           // (m, l, o) here, none is normalised
  int2* spread;            // [ctas] first output row and pieces of the segment a range boundary cuts, or with
                           // rows [packed + B][Hkv] first CTA and pieces of each segment; pieces 0: none
  int32_t ncta;
  int32_t min_units;       // blocks and what segments count besides (kSegUnits each) that a CTA takes at least
  int32_t beside;          // CTAs beside the matrix kernel's, if they end before it does (0: as min_units says)
  int32_t splits, tile_ns; // the prefix's token ranges, and the time of a tile there
};

constexpr int kMaxCtas = 192;     // of the attend's kernel: one an SM
constexpr int kMaxSplits = 148;   // token ranges of a shared prefix
constexpr int kAttendWarps = 12;  // of a CTA of the attend's kernel
constexpr int kSegUnits = 8;      // blocks that a segment counts for its start and end
// Times that the split of a shared call goes by: of the sequences' own tokens a CTA's start and end and a unit of
// its work; of the prefix a CTA's start and end and a 128-token tile for 256 rows and for 128.
constexpr int kCtaNs = 10000, kUnitNs = 120, kPrefixNs = 18000, kTile256Ns = 2150, kTile128Ns = 1100;

// The queries of a kv-head as the rows of one matrix: R = B G rows, row b G + g.
struct PagedSharedParams {
  int32_t R;
  int32_t two;             // a CTA's two lanes hold 256 rows, or 128 rows twice
  int32_t row_tiles;       // of 256 or 128 rows
  int32_t splits;          // token ranges
  uint8_t* codes;          // [Hkv][R][128] f8
  float2* factors;         // [Hkv][R]
  float* pieces;           // [Hkv][row_tiles][splits][2][128][2 + 128]
};

}  // namespace kv1b

cudaError_t kv1b_launch_paged_append(const kv1b::PagedAppendParams& p, cudaStream_t stream);
// The attend's kernel alone, and with the merge of what its ranges cut.
cudaError_t kv1b_launch_paged_pieces(const kv1b::PagedAttendParams& p, int32_t G, cudaStream_t stream);
cudaError_t kv1b_launch_paged_attend(const kv1b::PagedAttendParams& p, int32_t G, cudaStream_t stream);
cudaError_t kv1b_launch_paged_shared(const kv1b::PagedAttendParams& p, const kv1b::PagedSharedParams& s, int32_t G,
                                     cudaStream_t stream);
