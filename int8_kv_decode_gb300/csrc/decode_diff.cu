// Differential decode attention over the int8 cache:
//   out = softmax(s_0) V - lam softmax(s_1) V
// for a pair of query heads (2i, 2i + 1), the key planes 2p and 2p + 1 and the
// 256 value channels of both planes.
//
// One block per (sequence, draft column, differential head): thread t scores
// key t of a chunk of 256 keys against both maps, then sums value channel t
// over the chunk, with a running maximum and sum of each map.
#include "device_common.cuh"
#include "ops_internal.cuh"

namespace kattn {
namespace {

constexpr int kChunk = 256;

__device__ __forceinline__ bool diff_valid(const DiffParams& p, int b) {
  const int ctx = p.ctx_len[b];
  if (p.block_table == nullptr) return sequence_ok(p.row_start[b], ctx, p.M, p.cap_rows, p.max_ctx);
  if (ctx < 1 || ctx > p.max_ctx) return false;
  const int64_t keys = (int64_t)ctx + p.M - 1;
  return ((keys + (1 << p.page_shift) - 1) >> p.page_shift) <= (int64_t)p.max_pages;
}

__global__ void __launch_bounds__(kChunk) diff_row_kernel(const DiffParams p) {
  __shared__ uint32_t s_q[2][kD / 4];
  __shared__ float s_qs[2];
  __shared__ float s_p[2][kChunk];
  __shared__ int64_t s_row[kChunk];
  __shared__ float s_red[2][kChunk / 32];
  const int i = blockIdx.x, j = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int H = p.Hq / 2;
  float* out = p.out + (((int64_t)b * p.M + j) * H + i) * 2 * kD;
  if (!diff_valid(p, b)) {
    out[tid] = __int_as_float(0x7fc00000);
    if (tid == 0) atomicOr(p.err_word, KATTN_DEVERR_BAD_SEQUENCE);
    return;
  }
  if (warp < 2) {
    float qs;
    s_q[warp][lane] =
        warp_quantize_row(p.q + (((int64_t)b * p.M + j) * p.Hq + 2 * i + warp) * kD, &qs);
    if (lane == 0) s_qs[warp] = qs;
  }
  __syncthreads();
  const int pair = i / p.g, L = p.ctx_len[b] + j;
  const int64_t row0 = p.block_table ? 0 : p.row_start[b];
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f}, o[2] = {0.0f, 0.0f};
  for (int t0 = 0; t0 < L; t0 += kChunk) {
    const int t = t0 + tid, n = min(kChunk, L - t0);
    float s[2] = {-INFINITY, -INFINITY};
    if (t < L) {
      int64_t row = row0 + t;
      if (p.block_table) {
        int page = p.block_table[(int64_t)b * p.max_pages + (t >> p.page_shift)];
        if ((unsigned)page >= (unsigned)p.n_pages) {
          atomicOr(p.err_word, KATTN_DEVERR_BAD_PAGE);
          page = 0;
        }
        row = ((int64_t)page << p.page_shift) | (t & ((1 << p.page_shift) - 1));
      }
      s_row[tid] = row;
      for (int a = 0; a < 2; ++a) {
        const int64_t r = (int64_t)(2 * pair + a) * p.cap_rows + row;
        const int* kr = reinterpret_cast<const int*>(p.k + r * kD);
        int acc = 0;
        for (int w = 0; w < kD / 4; ++w) acc = __dp4a(kr[w], (int)s_q[a][w], acc);
        s[a] = __fmul_rn(__fmul_rn((float)acc, __fmul_rn(s_qs[a], p.k_scale[r])), p.sm_scale);
      }
    }
    for (int a = 0; a < 2; ++a) {
      const float w = warp_max(s[a]);
      if (lane == 0) s_red[a][warp] = w;
    }
    __syncthreads();
    float alpha[2];
    for (int a = 0; a < 2; ++a) {
      float mx = m[a];
      for (int w = 0; w < kChunk / 32; ++w) mx = fmaxf(mx, s_red[a][w]);
      alpha[a] = expf(m[a] - mx);
      m[a] = mx;
      s_p[a][tid] = t < L ? expf(s[a] - mx) : 0.0f;
    }
    __syncthreads();
    const int64_t plane = (int64_t)(2 * pair + (tid >> 7)) * p.cap_rows;
    float sum[2] = {0.0f, 0.0f}, acc[2] = {0.0f, 0.0f};
    for (int k = 0; k < n; ++k) {
      const int64_t r = plane + s_row[k];
      const float v = p.v_scale[r] * (float)p.v[r * kD + (tid & 127)];
      for (int a = 0; a < 2; ++a) {
        sum[a] += s_p[a][k];
        acc[a] = fmaf(s_p[a][k], v, acc[a]);
      }
    }
    for (int a = 0; a < 2; ++a) {
      l[a] = fmaf(l[a], alpha[a], sum[a]);
      o[a] = fmaf(o[a], alpha[a], acc[a]);
    }
    __syncthreads();
  }
  const float lam = p.lam[p.lam_per_row ? ((int64_t)b * p.M + j) * H + i : i];
  out[tid] = o[0] / l[0] - lam * (o[1] / l[1]);
}

}  // namespace

size_t diff_workspace_bytes(int B, int M, int Hq, int max_ctx) { return 256; }

void set_diff_workspace(DiffParams& p, void* workspace) {
  p.err_word = static_cast<uint32_t*>(workspace);
}

cudaError_t launch_decode_diff(const DiffParams& p, cudaStream_t stream) {
  diff_row_kernel<<<dim3((unsigned)(p.Hq / 2), (unsigned)p.M, (unsigned)p.B), kChunk, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace kattn
