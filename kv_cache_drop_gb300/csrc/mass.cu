// Attention mass: how much weight a chunk's rows put on each entry of their
// request's list,
//   out[b][j] = decay * in[b][j] + sum_{i sees j} sum_h exp(q_ih . k_j / 8 - lse_ih),
// the first term for entries older than the chunk (the chunk's own entries
// start at zero).  The weights are recomputed from the log-sum-exp that the
// chunk attention leaves, so neither the scores nor the values are stored or
// read.  A CTA owns 64 list entries of a request and walks every KV head and
// row of the chunk, so each sum is formed in one fixed order.
#include "chunk.cuh"

namespace akv {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

struct MassArgs {
  const float *lse;
  float decay;
  const float *in;
  float *out;
  int64_t stride;
};

struct MassSmem {
  float q[kD][kSimtPad], k[kD][kSimtPad];
  float lse[kSimt];
  float red[16][kSimt];
};

template <typename T>
__global__ void __launch_bounds__(kSimtThreads)
    mass_simt_kernel(const ChunkBatch a, const MassArgs ma) {
  __shared__ __align__(16) MassSmem sm;
  const int b = blockIdx.y, j0 = blockIdx.x * kSimt;
  const ChunkReq rq = chunk_req(a, b);
  if (j0 >= rq.n) return;
  const int grp = a.Hq / a.Hkv, rows = rq.m * grp;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  // first token that sees anything of this tile
  const int i0 = max(0, j0 - (rq.n - rq.m));
  float sum[4] = {};
  for (int g = 0; g < a.Hkv; ++g) {
    __syncthreads();
    simt_load_k<T>(sm.k, a, rq, g, j0, rq.n);
    for (int r0 = i0 * grp; r0 < rows; r0 += kSimt) {
      __syncthreads();
      simt_load_q<T>(sm.q, a, rq, g, r0);
      if (threadIdx.x < kSimt) {
        const int r = r0 + threadIdx.x;
        // +inf: a row that saw nothing, or no row, weighs 0
        float v = INFINITY;
        if (r < rows) {
          v = ma.lse[(int64_t)(rq.q0 + r / grp) * a.Hq + g * grp + r % grp];
          if (v == -INFINITY) v = INFINITY;
        }
        sm.lse[threadIdx.x] = v;
      }
      __syncthreads();
      float s[4][4] = {};
      simt_mma(sm.q, sm.k, ty, tx, s);
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int r = r0 + 4 * ty + p;
        const float v = sm.lse[4 * ty + p];
        const int lim = r < rows && v != INFINITY ? rq.limit(r / grp) : 0;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (j0 + 4 * tx + q < lim) sum[q] += exp2f(fmaf(s[p][q], 0.125f, -v) * kLog2e);
      }
    }
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) sm.red[ty][4 * tx + q] = sum[q];
  __syncthreads();
  const int j = j0 + threadIdx.x;
  if (threadIdx.x < kSimt && j < rq.n) {
    float x = 0.f;
    for (int y = 0; y < 16; ++y) x += sm.red[y][threadIdx.x];
    const int64_t at = (int64_t)b * ma.stride + j;
    if (ma.in && j < rq.n - rq.m) x = fmaf(ma.decay, ma.in[at], x);
    ma.out[at] = x;
  }
}

}  // namespace

size_t mass_workspace_bytes(int dtype, int B, int Hq, int Hkv, int n_rows, int max_q, int max_kv) {
  return 0;
}

cudaError_t launch_mass(int dtype, int B, int Hq, int Hkv, int n_rows, int S,
                        const int32_t *q_indptr, int max_q, const void *q, const void *k,
                        const int32_t *kv_indptr, const int32_t *kv_indices, int max_kv,
                        const float *lse, float decay, const float *in, float *out, int64_t stride,
                        void *ws, cudaStream_t s) {
  const ChunkBatch a{B, Hq, Hkv, n_rows, S, max_q, max_kv, q_indptr, kv_indptr, kv_indices, q, k,
                     nullptr};
  const MassArgs ma{lse, decay, in, out, stride};
  const dim3 grid((unsigned)((max_kv + kSimt - 1) / kSimt), B);
  if (dtype == AKV_BF16) mass_simt_kernel<__nv_bfloat16><<<grid, kSimtThreads, 0, s>>>(a, ma);
  else mass_simt_kernel<float><<<grid, kSimtThreads, 0, s>>>(a, ma);
  return cudaGetLastError();
}

}  // namespace akv
