// q4.h -- the paged 4-bit KV cache: record layout, device error and launcher
// interfaces shared by api.cu and the kernels of the serving step (page
// tables, q/k norm + rotation, cache write / read, decode).  Not part of the
// public ABI.
//
// The cache is uint8 [num_pages][Hkv][page_size / 16][18 d]: one record holds
// 16 consecutive tokens of one kv head, K and V, codes and scales, so that a
// record is one contiguous copy (2304 bytes at d 128) whatever the page.
// Channels are quantised in groups of 32: value = (code - 8) * scale, code - 8
// in -7..7, scale = max|x| / 7 cut (towards zero) to 5 significant bits, held
// in bf16.  3 bits times 5 bits: every stored value is exactly a bf16 number.
// The codes stand in the order in which the decode kernel's warp MMAs want
// them (G = d / 32 groups):
//   K codes   at 0     token r, t < 4, group w < G: the 32-bit word at
//                      r d/2 + t d/8 + 4 w holds channels 32 w + 8 t + e, e < 8,
//                      the code of e in the 4 bits at 16 (e & 1) + 4 (e >> 1),
//                      the word rotated left by 3: lane 4 g + t of a warp reads
//                      one 16-byte vector (d 128) per token, the A operand of
//                      its row, a pair of codes 16 bits apart;
//   V codes   at 8 d   the 32-bit word at hi 4 d + (4 g + t) d/8 + 4 j holds
//                      tokens 8 hi + 2 t (low half) and 8 hi + 2 t + 1 (high
//                      half), channels g d/8 + 4 j + i, i < 4, code at 4 i of
//                      the half: the value MMA contracts over tokens, so its
//                      operand pairs neighbouring tokens;
//   K scales  at 16 d  bf16 [16 tokens][G];
//   V scales  at 17 d  bf16 [G][16 tokens] (token pairs in one 32-bit word).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.cuh"

namespace flux {

// Device error word values of this part (continuing common.cuh's).
enum : int {
  DEV_ERR_PAGE = 5,        // page or slot outside the cache
};

constexpr int kQ4Rec = 16;                       // tokens per record
constexpr uint32_t kQ4LowBits = 27u << 23;       // 2^-100: a group below it is stored as zeros
constexpr uint32_t kQ4HighBits = 247u << 23;     // 2^120: a group above it is stored as NaN

template <int D>
struct Q4Layout {
  static constexpr int G = D / 32;               // scale groups per row
  static constexpr int VC = 8 * D;               // V codes
  static constexpr int KS = 16 * D;              // K scales
  static constexpr int VS = 17 * D;              // V scales
  static constexpr int BYTES = 18 * D;
};

struct PageTableLaunch {
  const int32_t* old_lens;
  const int32_t* new_lens;
  int B, page_size, sink_pages, window_pages;    // window_pages 0: no ring
  const int32_t* free_pages;
  int n_free;
  const int32_t* cursor;
  int32_t* cursor_out;
  int32_t* page_table;       // [B][max_pages]
  int max_pages;
  int64_t* slots;            // [n_slots]
  int32_t* positions;        // [n_slots]
  int n_slots;
  int32_t* cu_new;           // [B + 1] or null
  int* ticket;
  int* err;
};
constexpr int kPageTableMaxB = 8192;             // both prefix arrays live in shared memory
cudaError_t launch_page_table(const PageTableLaunch& p, int num_sms, cudaStream_t stream);

struct NormRopeLaunch {
  const uint16_t* q;
  const uint16_t* k;
  long long q_stride, k_stride;                  // elements between tokens
  uint16_t* q_out;
  uint16_t* k_out;
  long long q_out_stride, k_out_stride;
  const uint16_t* q_weight;                      // [d] or null
  const uint16_t* k_weight;
  float eps;
  const int32_t* positions;
  const float* inv_freq;                         // [rot / 2]
  int rot, interleaved;
  int N, Hq, Hkv, d;
};
cudaError_t launch_norm_rope(const NormRopeLaunch& p, int num_sms, cudaStream_t stream);

struct KvQ4Launch {
  const uint16_t* k;         // write: source; token stride below
  const uint16_t* v;
  long long k_stride, v_stride;
  uint16_t* k_out;           // read: destination, contiguous
  uint16_t* v_out;
  const int64_t* slots;
  int N, Hkv, d;
  uint8_t* pool;
  int num_pages, page_size;
  int* err;
};
cudaError_t launch_kv_write_q4(const KvQ4Launch& p, int num_sms, cudaStream_t stream);
cudaError_t launch_kv_read_q4(const KvQ4Launch& p, int num_sms, cudaStream_t stream);

struct DecodeQ4Launch {
  const uint16_t* q;
  const uint8_t* pool;
  int num_pages, page_size;
  const int32_t* page_table;
  int max_pages;
  const int32_t* seqlens;
  uint16_t* o;
  float* lse;
  int B, Hq, Hkv, d;
  const uint8_t* layer_mode;
  int layer;
  int sink_blocks, window_blocks, block;
  float scale;
  float* part;               // split partials (decode_q4_workspace_bytes)
  int* tickets;              // [B * Hkv], zero between calls
  DevStatus st;
};
size_t decode_q4_workspace_bytes(int d, int num_sms);
cudaError_t launch_decode_q4(const DecodeQ4Launch& p, int num_sms, cudaStream_t stream);

}  // namespace flux
