// Attention of a chunk of new tokens over the active cache in a page-size-1
// pool (paper review page section 4 serving flow: a request whose history is
// cached appends its new message to the active cache; the system README:
// page size 1).  Row i of request b's m rows attends over the first
// n - m + i + 1 entries of its list, which ends with the chunk's own slots:
//   s_j = q . k_j / 8,  out = sum_j softmax(s)_j v_j,  lse = log sum_j exp(s_j).
#include "chunk.cuh"

#include <algorithm>

namespace akv {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Split-KV partials: [n_rows][Hq][ns], m in log2 units.
struct ChunkParts {
  float2 *ml;
  float *o;
  int ns, chunk;
};

template <typename T>
__device__ __forceinline__ void store4(T *dst, const float *x);
template <>
__device__ __forceinline__ void store4<float>(float *dst, const float *x) {
  *reinterpret_cast<float4 *>(dst) = make_float4(x[0], x[1], x[2], x[3]);
}
template <>
__device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16 *dst, const float *x) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
  *reinterpret_cast<uint2 *>(dst) = make_uint2(*reinterpret_cast<const uint32_t *>(&a),
                                               *reinterpret_cast<const uint32_t *>(&b));
}

struct SimtSmem {
  float q[kD][kSimtPad], k[kD][kSimtPad], v[kSimt][kSimtPad], p[kSimt][kSimtPad];
};

// CUDA-core form, every type and head count: CTA = 64 packed rows of one KV
// head x one key split, 64-key tiles, online softmax.
template <typename T>
__global__ void __launch_bounds__(kSimtThreads)
    chunk_simt_kernel(const ChunkBatch a, T *out, float *lse, const ChunkParts part) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SimtSmem &sm = *reinterpret_cast<SimtSmem *>(smem_raw);
  const int split = blockIdx.x % part.ns, rt = blockIdx.x / part.ns, g = blockIdx.y, b = blockIdx.z;
  const ChunkReq rq = chunk_req(a, b);
  const int grp = a.Hq / a.Hkv, rows = rq.m * grp, r0 = rt * kSimt;
  if (r0 >= rows) return;
  const int last = (min(rows, r0 + kSimt) - 1) / grp;  // the tile's last token
  const int c0 = split * part.chunk;
  const int c1 = min(rq.limit(last), c0 + part.chunk);
  if (part.ns > 1 && c0 >= c1) return;  // the merge reads only splits with visible entries
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  int lim[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int r = r0 + 4 * ty + p;
    lim[p] = r < rows ? rq.limit(r / grp) : 0;
  }
  simt_load_q<T>(sm.q, a, rq, g, r0);
  float o[4][4] = {}, m[4], l[4] = {};
#pragma unroll
  for (int p = 0; p < 4; ++p) m[p] = -INFINITY;
  for (int j0 = c0; j0 < c1; j0 += kSimt) {
    __syncthreads();  // the previous tile's readers are done
    simt_load_k<T>(sm.k, a, rq, g, j0, c1);
    for (int u = threadIdx.x; u < kSimt * (kD / Chunk<T>::kElems); u += kSimtThreads) {
      constexpr int E = Chunk<T>::kElems, C = kD / E;
      const int key = u / C, c = u % C;
      float f[E];
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = 0.f;
      if (j0 + key < c1)
        chunk_to_f32<T>(__ldg(reinterpret_cast<const uint4 *>(
                            (const T *)a.v + (chunk_slot(a, rq, j0 + key) * a.Hkv + g) * kD) + c), f);
#pragma unroll
      for (int e = 0; e < E; ++e) sm.v[key][c * E + e] = f[e];
    }
    __syncthreads();
    float s[4][4] = {};
    simt_mma(sm.q, sm.k, ty, tx, s);
    // A tile with a hidden entry keeps that entry's value out of the sum
    // whatever it holds (0 * NaN): such tiles skip hidden keys per row.
    const bool ragged = j0 + kSimt > rq.limit(r0 / grp);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      float mx = -INFINITY;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (j0 + 4 * tx + q >= min(lim[p], c1)) s[p][q] = -INFINITY;
        mx = fmaxf(mx, s[p][q]);
      }
#pragma unroll
      for (int x = 8; x; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
      const float mn = fmaxf(m[p], mx), ref = mn == -INFINITY ? 0.f : mn;
      const float alpha = exp2f((m[p] - ref) * (0.125f * kLog2e));
      m[p] = mn;
      l[p] *= alpha;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        o[p][q] *= alpha;
        // the difference is taken before the scale: its rounding is relative
        // to the distance from the maximum
        s[p][q] = exp2f((s[p][q] - ref) * (0.125f * kLog2e));
        l[p] += s[p][q];
        sm.p[4 * tx + q][4 * ty + p] = s[p][q];
      }
    }
    __syncthreads();
    if (!ragged) {
      simt_mma(sm.p, sm.v, ty, tx, o);
    } else {
      for (int d = 0; d < kSimt; ++d) {
#pragma unroll
        for (int p = 0; p < 4; ++p)
          if (j0 + d < lim[p])
#pragma unroll
            for (int q = 0; q < 4; ++q)
              o[p][q] = fmaf(sm.p[d][4 * ty + p], sm.v[d][4 * tx + q], o[p][q]);
      }
    }
  }
#pragma unroll
  for (int p = 0; p < 4; ++p) {
#pragma unroll
    for (int x = 8; x; x >>= 1) l[p] += __shfl_xor_sync(0xffffffffu, l[p], x);
    const int r = r0 + 4 * ty + p;
    if (r >= rows) continue;
    const int64_t row = (int64_t)(rq.q0 + r / grp) * a.Hq + g * grp + r % grp;
    if (part.ns == 1) {
      const bool none = lim[p] == 0;
      float y[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) y[q] = none ? 0.f : o[p][q] / l[p];
      store4<T>(out + row * kD + 4 * tx, y);
      if (lse && tx == 0) lse[row] = none ? -INFINITY : m[p] * 0.125f + logf(l[p]);
    } else {
      const int64_t pi = row * part.ns + split;
      store4<float>(part.o + pi * kD + 4 * tx, o[p]);
      if (tx == 0) part.ml[pi] = make_float2(m[p] * (0.125f * kLog2e), l[p]);
    }
  }
}

// Joins the splits of a row by their log-sum-exp: a warp per (row, head), two
// output columns per lane.
constexpr int kMergeWarps = 8;
template <typename T>
__global__ void __launch_bounds__(kMergeWarps * 32)
    chunk_merge_kernel(const ChunkBatch a, T *out, float *lse, const ChunkParts part) {
  const int64_t w = (int64_t)blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int t = (int)(w / a.Hq);
  if (t >= a.n_rows) return;
  int lo = 0, hi = a.B;  // the request that holds row t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.q_indptr[mid] <= t) lo = mid; else hi = mid;
  }
  const ChunkReq rq = chunk_req(a, lo);
  const int i = t - rq.q0;
  if (i < 0 || i >= rq.m) return;  // no request's row: left as it is
  const int used = (rq.limit(i) + part.chunk - 1) / part.chunk;
  const float2 *ml = part.ml + w * part.ns;
  float M = -INFINITY;
  for (int s = lane; s < used; s += 32) M = fmaxf(M, ml[s].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float ref = M == -INFINITY ? 0.f : M;
  float L = 0.f, x0 = 0.f, x1 = 0.f;
  for (int s0 = 0; s0 < used; s0 += 32) {
    float f = 0.f;
    if (s0 + lane < used) {
      const float2 v = ml[s0 + lane];
      f = exp2f(v.x - ref);
      L += v.y * f;
    }
    const int cnt = min(32, used - s0);
    for (int s = 0; s < cnt; ++s) {
      const float fs = __shfl_sync(0xffffffffu, f, s);
      const float2 v = reinterpret_cast<const float2 *>(part.o + (w * part.ns + s0 + s) * kD)[lane];
      x0 = fmaf(v.x, fs, x0);
      x1 = fmaf(v.y, fs, x1);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  const bool none = used == 0;
  const float y0 = none ? 0.f : x0 / L, y1 = none ? 0.f : x1 / L;
  if constexpr (sizeof(T) == 4)
    reinterpret_cast<float2 *>(out + w * kD)[lane] = make_float2(y0, y1);
  else
    reinterpret_cast<__nv_bfloat162 *>(out + w * kD)[lane] = __floats2bfloat162_rn(y0, y1);
  if (lse && lane == 0) lse[w] = none ? -INFINITY : M * kLn2 + logf(L);
}

int sm_count() {
  int dev = 0, sms = 152;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

// Splits of the key axis: a call whose row tiles alone give `waves` waves of
// CTAs is not split; otherwise the lists are cut into chunks of at least
// kMinSplit keys, as many as reach that.  The count depends on the host's
// bounds only, so that a captured call replays for any lengths within them.
constexpr int kMinSplit = 256;
constexpr int kMaxSplit = 1024;
int plan_splits(int64_t tiles, int max_kv, int64_t want, int *chunk) {
  int64_t ns = tiles >= want || tiles <= 0 ? 1 : (want + tiles - 1) / tiles;
  ns = std::min<int64_t>(std::min<int64_t>(ns, kMaxSplit), (max_kv + kMinSplit - 1) / kMinSplit);
  ns = std::max<int64_t>(ns, 1);
  *chunk = (int)(((int64_t)(max_kv + ns - 1) / ns + 127) / 128 * 128);
  if (*chunk < 128) *chunk = 128;
  return (int)std::max<int64_t>(1, ((int64_t)max_kv + *chunk - 1) / *chunk);
}

int64_t row_tiles(int Hq, int Hkv, int max_q, int tile) {
  return ((int64_t)max_q * (Hq / Hkv) + tile - 1) / tile;
}

struct ChunkPlan {
  int ns, chunk;
  int64_t tiles;  // row tiles of one (request, KV head)
};
ChunkPlan chunk_plan(int dtype, int B, int Hq, int Hkv, int max_q, int max_kv) {
  ChunkPlan p;
  p.tiles = row_tiles(Hq, Hkv, max_q, kSimt);
  p.ns = plan_splits(p.tiles * B * Hkv, max_kv, 4LL * sm_count(), &p.chunk);
  return p;
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

template <typename T>
cudaError_t launch_simt(const ChunkBatch &a, void *out, float *lse, const ChunkParts &part,
                        int64_t tiles, cudaStream_t s) {
  const int smem = (int)sizeof(SimtSmem);
  cudaError_t e = cudaFuncSetAttribute(chunk_simt_kernel<T>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  chunk_simt_kernel<T><<<dim3((unsigned)(tiles * part.ns), a.Hkv, a.B), kSimtThreads, smem, s>>>(
      a, (T *)out, lse, part);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_merge(const ChunkBatch &a, void *out, float *lse, const ChunkParts &part,
                         cudaStream_t s) {
  const int64_t warps = (int64_t)a.n_rows * a.Hq;
  chunk_merge_kernel<T><<<(unsigned)((warps + kMergeWarps - 1) / kMergeWarps), kMergeWarps * 32, 0,
                          s>>>(a, (T *)out, lse, part);
  return cudaGetLastError();
}

}  // namespace

int64_t chunk_grid_x(int dtype, int B, int Hq, int Hkv, int max_q, int max_kv) {
  const ChunkPlan p = chunk_plan(dtype, B, Hq, Hkv, max_q, max_kv);
  return p.tiles * p.ns;
}

size_t chunk_workspace_bytes(int dtype, int B, int Hq, int Hkv, int n_rows, int max_q, int max_kv) {
  const ChunkPlan p = chunk_plan(dtype, B, Hq, Hkv, max_q, max_kv);
  if (p.ns == 1) return 0;
  const size_t parts = (size_t)n_rows * Hq * p.ns;
  return up256(parts * sizeof(float2)) + up256(parts * kD * sizeof(float));
}

cudaError_t launch_chunk(int dtype, int B, int Hq, int Hkv, int n_rows, int S,
                         const int32_t *q_indptr, int max_q, const void *q, const void *k,
                         const void *v, const int32_t *kv_indptr, const int32_t *kv_indices,
                         int max_kv, void *out, float *lse, void *ws, cudaStream_t s) {
  const ChunkPlan p = chunk_plan(dtype, B, Hq, Hkv, max_q, max_kv);
  const ChunkBatch a{B, Hq, Hkv, n_rows, S, max_q, max_kv, q_indptr, kv_indptr, kv_indices, q, k, v};
  ChunkParts part{nullptr, nullptr, p.ns, p.chunk};
  if (p.ns > 1) {
    part.ml = (float2 *)ws;
    part.o = (float *)((char *)ws + up256((size_t)n_rows * Hq * p.ns * sizeof(float2)));
  }
  cudaError_t e = dtype == AKV_BF16 ? launch_simt<__nv_bfloat16>(a, out, lse, part, p.tiles, s)
                                    : launch_simt<float>(a, out, lse, part, p.tiles, s);
  if (e != cudaSuccess || p.ns == 1) return e;
  return dtype == AKV_BF16 ? launch_merge<__nv_bfloat16>(a, out, lse, part, s)
                           : launch_merge<float>(a, out, lse, part, s);
}

}  // namespace akv
