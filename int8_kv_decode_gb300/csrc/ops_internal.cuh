// Declarations of the operators beside the decode: differential attention,
// the norm with 8-bit output, and the page operations.
#pragma once

#include "kattn_internal.cuh"

namespace kattn {

// ------------------------------------------------ differential attention --
struct DiffParams {
  const float* q;
  const int8_t* k;
  const float* k_scale;
  const int8_t* v;
  const float* v_scale;
  const int64_t* row_start;     // contiguous layout (block_table == nullptr)
  const int32_t* ctx_len;
  const int32_t* block_table;   // paged layout, as DecodeParams
  int max_pages, page_shift, n_pages;
  const float* lam;
  int lam_per_row;              // lam is [B][M][H], else [H]
  float* out;
  uint32_t* err_word;
  float* partials;
  int B, M, Hq, Hkv, g, R;      // R = g * M rows of each map per plane pair
  int pairs;                    // Hkv / 2
  int cap_rows, max_ctx;
  int nwin_max;                 // windows of the longest sequence
  int sms;                      // multiprocessors of the device
  float sm_scale;
};
int64_t diff_units(const DiffParams& p);          // work units, at most
size_t diff_workspace_bytes(int B, int M, int Hq, int max_ctx);
void set_diff_workspace(DiffParams& p, void* workspace);
cudaError_t launch_decode_diff(const DiffParams& p, cudaStream_t stream);

// ------------------------------------------------- norm with 8-bit output --
struct NormParams {
  const void* x;
  const void* residual;
  const void* weight;
  void* residual_out;
  uint8_t* codes;
  float* scales;
  int64_t rows, x_stride, res_stride, res_out_stride;
  int d;
  int group;                    // channels per scale: d or 128
  float eps;
};
cudaError_t launch_rms_norm_quant(const NormParams& p, int x_type, int code_type,
                                  cudaStream_t stream);

// -------------------------------------------------------- page operations --
// Workspace, all of it zero before the first call:
//   [0, 256)     header: the error word
//   claim[S], mark[S]   slots named by a list; zero again after every call
//   flag[S]      per list entry
//   chunk[64]    counts per block of the cluster
//   list, list2, to     [n_pages] (list2: pairs)
struct PageWorkspace {
  uint32_t* err;
  int *claim, *mark, *flag, *chunk, *list, *to;
  int2* list2;
};
size_t page_workspace_bytes(int n_slots, int n_pages);

struct PageParams {
  int32_t* table;
  int n_slots, max_pages;
  int32_t* refs;
  int n_pages, page_shift;
  const int32_t *seqs, *parents, *lens;   // fork: seqs are the children
  int n;
  int32_t *src, *dst, *counts;
  int32_t *table_out, *ref_out;
  PageWorkspace ws;
};
void set_page_workspace(PageParams& p, void* workspace);
cudaError_t launch_reserve_pages(const PageParams& p, cudaStream_t stream);
cudaError_t launch_free_sequences(const PageParams& p, cudaStream_t stream);
cudaError_t launch_fork_sequences(const PageParams& p, cudaStream_t stream);
cudaError_t launch_compact_pages(const PageParams& p, cudaStream_t stream);

struct CopyParams {
  int8_t *k, *v;
  float *k_scale, *v_scale;
  int Hkv, cap_rows, page_rows, n_pages, n;
  const int32_t *src, *dst, *count;
  uint32_t* err;
};
cudaError_t launch_copy_pages(const CopyParams& p, cudaStream_t stream);

}  // namespace kattn
