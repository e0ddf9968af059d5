// Declarations of the operators on a block-scaled cache: rotary positions, rows
// written into the cache and read back, and decode attention over it.
#pragma once

#include "kattn_internal.cuh"

namespace kattn {

// cos and sin of position * freq[i], i < half, as float pairs: table[position][i].
cudaError_t launch_rope_table(const double* freq, int n_positions, int half, float* table,
                              cudaStream_t stream);

struct RopeParams {
  const void* x;
  void* out;
  int64_t x_stride, out_stride;   // elements between rows
  const int32_t* positions;
  const float* table;             // [n_positions][half][2]
  int rows, heads, n_positions, half, interleaved;
};
cudaError_t launch_rope(const RopeParams& p, int x_type, int out_type, cudaStream_t stream);

// A paged cache whose rows share a scale per block of 2^block_shift rows and head.
struct BlockCache {
  uint8_t *k, *v;                 // codes [Hkv][cap_rows][128]
  float *k_scale, *v_scale;       // [Hkv][cap_rows >> block_shift]
  const int32_t* block_table;     // [B][max_pages]
  int Hkv, cap_rows, block_shift, page_shift, n_pages, max_pages;
};

// Ragged rows of B sequences: rows [cu[b], cu[b + 1]) are the keys start[b], ...
struct SpanParams {
  const int32_t* cu;
  const int32_t* start;
  int B, rows;                    // rows: an upper bound on cu[B]
  uint32_t* err;
};

struct AppendParams {
  BlockCache c;
  SpanParams s;
  const void *k_new, *v_new, *q;  // q may be null
  void* q_out;
  int64_t k_stride, v_stride, q_stride, q_out_stride;
  int Hq;
  const float* table;             // null: no rotation
  int n_positions, half, interleaved;
};
cudaError_t launch_append_blocks(const AppendParams& p, int x_type, int code_type, cudaStream_t stream);

struct ReadParams {
  BlockCache c;
  SpanParams s;
  void *out_k, *out_v;            // [rows][Hkv][128], either may be null
};
cudaError_t launch_read_blocks(const ReadParams& p, int code_type, int out_type, cudaStream_t stream);

struct BlockDecodeParams {
  BlockCache c;
  const void* q;
  void* out;
  int q_type;                     // a kattn_dtype, of q and out
  const int32_t* ctx_len;
  uint32_t* err_word;
  float* partials;
  int B, M, Hq, g, R;             // R = g * M rows per kv head
  int max_ctx, nwin_max, sms;
  float sm_scale;
};
int64_t block_decode_units(const BlockDecodeParams& p);
size_t block_decode_workspace_bytes(int B, int M, int Hq, int max_ctx);
void set_block_decode_workspace(BlockDecodeParams& p, void* workspace);
cudaError_t launch_decode_blocks(const BlockDecodeParams& p, int code_type, cudaStream_t stream);

}  // namespace kattn
