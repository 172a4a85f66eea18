// Attention of a chunk of new tokens over the active cache in a page-size-1
// pool (paper review page section 4 serving flow: a request whose history is
// cached appends its new message to the active cache; the system README:
// page size 1).  Row i of request b's m rows attends over the first
// n - m + i + 1 entries of its list, which ends with the chunk's own slots:
//   s_j = q . k_j / 8,  out = sum_j softmax(s)_j v_j,  lse = log sum_j exp(s_j).
#include "chunk.cuh"

#include <algorithm>
#include <type_traits>

namespace akv {
namespace {

constexpr float kLn2 = 0.6931471805599453f;

// Split-KV partials: [n_rows][Hq][ns], m in log2 units.  A row whose visible
// entries lie in one split is written out by that split; the merge passes it
// over.
struct ChunkParts {
  float2 *ml;
  float *o;
  int ns, chunk;
  __device__ __forceinline__ bool direct(int lim) const { return ns == 1 || lim <= chunk; }
};
constexpr int kMaxSplit = 1024;  // the merge keeps one weight per split in shared memory

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

// fp32, CUDA cores: CTA = 128 packed rows of one KV head x one key split, 64
// keys at a time, online softmax.  K of the next keys is copied while a step's
// weights are formed and multiplied with V, V while the next scores are.
// Tensor cores take no fp32 operands; this path is for single-precision
// parity, bound by the fp32 pipes and their shared-memory operands.  One CTA
// per SM: held to 128 registers for two, it spills and takes 257 us instead of
// 232 (3 chunks of 116-301 rows over 1,050-4,000 entries; 230 with the list
// entries of a step loaded before the step's scores).
struct F32Smem {
  float q[kFRows][kFPitch], p[kFRows][kFPitch], k[kFKeys][kFPitch], v[kFKeys][kFPitch];
};

__global__ void __launch_bounds__(kFThreads, 1)
    chunk_f32_kernel(const ChunkBatch a, float *out, float *lse, const ChunkParts part,
                     uint32_t *status) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  F32Smem &sm = *reinterpret_cast<F32Smem *>(smem_raw);
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  clear_status(status);
  const int split = blockIdx.x % part.ns, g = blockIdx.y, b = blockIdx.z;
  const int64_t r0 = (int64_t)(blockIdx.x / part.ns) * kFRows;
  const ChunkReq rq = chunk_req(a, b);
  const int grp = a.Hq / a.Hkv;
  const int64_t rows = (int64_t)rq.m * grp;
  if (r0 >= rows) return;
  const int64_t r1 = min(rows, r0 + kFRows);
  const int c0 = split * part.chunk;
  const int c1 = min(rq.limit((int)((r1 - 1) / grp)), c0 + part.chunk);
  if (split > 0 && c0 >= c1) return;  // the merge reads only splits with visible entries
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  const int first = rq.limit((int)(r0 / grp));  // every row sees the entries before it
  int lim[8];
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int r = (int)r0 + ty + 16 * p;
    lim[p] = r < r1 ? rq.limit(r / grp) : 0;
  }
  const auto commit = [] { asm volatile("cp.async.commit_group;\n" ::: "memory"); };
  int own[kFOwn];
  f32_rows(own, a, rq, c0, c1);
  f32_load_q(sm.q, a, rq, g, r0);
  f32_load_kv(sm.k, a.k, a, g, own);
  commit();
  f32_load_kv(sm.v, a.v, a, g, own);
  commit();
  float o[8][4], m[8], l[8];
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    o[p][0] = o[p][1] = o[p][2] = o[p][3] = l[p] = 0.f;
    m[p] = -INFINITY;
  }
  for (int j0 = c0; j0 < c1; j0 += kFKeys) {
    asm volatile("cp.async.wait_group 1;\n" ::: "memory");
    __syncthreads();  // K (and Q) landed
    f32_rows(own, a, rq, j0 + kFKeys, c1);
    float s[8][4];
    f32_scores(sm.q, sm.k, ty, tx, s);
    __syncthreads();  // K's readers are done
    f32_load_kv(sm.k, a.k, a, g, own);
    commit();
    const bool ragged = j0 + kFKeys > min(first, c1);
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      float mx = -INFINITY;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (ragged && j0 + tx + 16 * q >= min(lim[p], c1)) s[p][q] = -INFINITY;
        mx = fmaxf(mx, s[p][q]);
      }
#pragma unroll
      for (int x = 8; x; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
      const float mn = fmaxf(m[p], mx), ref = mn == -INFINITY ? 0.f : mn;
      const float alpha = ptx::ex2((m[p] - ref) * kScale);
      m[p] = mn;
      l[p] *= alpha;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        o[p][q] *= alpha;
        // the difference is taken before the scale: its rounding is relative
        // to the distance from the maximum
        const float w = ptx::ex2((s[p][q] - ref) * kScale);
        l[p] += w;
        sm.p[ty + 16 * p][tx + 16 * q] = w;
      }
    }
    asm volatile("cp.async.wait_group 1;\n" ::: "memory");
    __syncthreads();  // V landed, P written
    // o[p][q]: column 4 tx + q
    if (!ragged) {
#pragma unroll 4
      for (int j = 0; j < kFKeys; j += 4) {
        float4 w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = *reinterpret_cast<const float4 *>(&sm.v[j + e][4 * tx]);
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          const float4 u = *reinterpret_cast<const float4 *>(&sm.p[ty + 16 * p][j]);
          const float uu[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 d = make_float2(uu[e], uu[e]);
            float2 *oo = reinterpret_cast<float2 *>(o[p]);
            oo[0] = __ffma2_rn(d, make_float2(w[e].x, w[e].y), oo[0]);
            oo[1] = __ffma2_rn(d, make_float2(w[e].z, w[e].w), oo[1]);
          }
        }
      }
    } else {
      // a hidden entry's value stays out of the sum whatever it holds (0 * NaN)
#pragma unroll 1
      for (int j = 0; j < kFKeys; ++j) {
        const float4 w = *reinterpret_cast<const float4 *>(&sm.v[j][4 * tx]);
#pragma unroll
        for (int p = 0; p < 8; ++p)
          if (j0 + j < min(lim[p], c1)) {
            const float u = sm.p[ty + 16 * p][j];
            o[p][0] = fmaf(u, w.x, o[p][0]);
            o[p][1] = fmaf(u, w.y, o[p][1]);
            o[p][2] = fmaf(u, w.z, o[p][2]);
            o[p][3] = fmaf(u, w.w, o[p][3]);
          }
      }
    }
    __syncthreads();  // V's and P's readers are done
    f32_load_kv(sm.v, a.v, a, g, own);
    commit();
  }
  asm volatile("cp.async.wait_group 0;\n" ::: "memory");
#pragma unroll
  for (int p = 0; p < 8; ++p) {
#pragma unroll
    for (int x = 8; x; x >>= 1) l[p] += __shfl_xor_sync(0xffffffffu, l[p], x);
    const int64_t r = r0 + ty + 16 * p;
    if (r >= r1) continue;
    const int64_t row = (int64_t)(rq.q0 + (int)(r / grp)) * a.Hq + g * grp + (int)(r % grp);
    if (part.direct(lim[p])) {
      if (split > 0) continue;
      const bool none = lim[p] == 0;
      float y[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) y[q] = none ? 0.f : o[p][q] / l[p];
      store4<float>(out + row * kD + 4 * tx, y);
      if (lse && tx == 0) lse[row] = none ? -INFINITY : m[p] * 0.125f + logf(l[p]);
    } else {
      const int64_t pi = row * part.ns + split;
      store4<float>(part.o + pi * kD + 4 * tx, o[p]);
      if (tx == 0) part.ml[pi] = make_float2(m[p] * kScale, l[p]);
    }
  }
}

// The splits that hold row t's visible entries; 0 where there is nothing to
// merge (written by its one split, or no request's row).
__device__ __forceinline__ int merge_used(const ChunkBatch &a, const ChunkParts &part, int t) {
  int lo = 0, hi = a.B;  // the request that holds row t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(a.q_indptr + mid) <= t) lo = mid; else hi = mid;
  }
  const ChunkReq rq = chunk_req(a, lo);
  const int i = t - rq.q0;
  if (i < 0 || i >= rq.m) return 0;
  const int lim = rq.limit(i);
  return part.direct(lim) ? 0 : (lim + part.chunk - 1) / part.chunk;
}

// Joins the splits of a row by their log-sum-exp; launched as a programmatic
// dependent of the attention kernel.  Up to kWarpMerge splits: a warp per
// (row, head), two columns per lane, one split's weight per lane (a CTA per
// row and head took 120 us for 4,097 rows of 24 heads in two splits).
constexpr int kWarpMerge = 32;
constexpr int kMergeWarps = 8;
template <typename T>
__global__ void __launch_bounds__(kMergeWarps * 32)
    chunk_merge_warp_kernel(const ChunkBatch a, T *out, float *lse, const ChunkParts part) {
  const int64_t w = (int64_t)blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int t = (int)(w / a.Hq);
  const int used = t < a.n_rows ? merge_used(a, part, t) : 0;
  // every warp waits, so that this grid never ends before the one it follows
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  if (used == 0) return;
  const float2 ml = lane < used ? __ldcg(part.ml + w * part.ns + lane) : make_float2(-INFINITY, 0.f);
  float M = ml.x;
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float f = exp2f(ml.x - (M == -INFINITY ? 0.f : M));
  float L = ml.y * f;
#pragma unroll
  for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  float x0 = 0.f, x1 = 0.f;
  const float2 *po = reinterpret_cast<const float2 *>(part.o + w * part.ns * kD) + lane;
#pragma unroll 8
  for (int s = 0; s < used; ++s) {
    const float2 v = __ldcg(po + s * (kD / 2));
    const float fs = __shfl_sync(0xffffffffu, f, s);
    x0 = fmaf(v.x, fs, x0);
    x1 = fmaf(v.y, fs, x1);
  }
  x0 /= L;
  x1 /= L;
  if constexpr (sizeof(T) == 4) reinterpret_cast<float2 *>(out + w * kD)[lane] = make_float2(x0, x1);
  else reinterpret_cast<__nv_bfloat162 *>(out + w * kD)[lane] = __floats2bfloat162_rn(x0, x1);
  if (lse && lane == 0) lse[w] = M * kLn2 + logf(L);
}

// More splits (few rows): a CTA per (row, head), eight groups of 16 threads
// each summing every eighth split's output row, 16 bytes per load.
constexpr int kMergeThreads = 128;
template <typename T>
__global__ void __launch_bounds__(kMergeThreads)
    chunk_merge_kernel(const ChunkBatch a, T *out, float *lse, const ChunkParts part) {
  __shared__ float wgt[kMaxSplit];
  __shared__ float4 red[8][kD / 4];
  __shared__ float tot[kMergeThreads / 32], top[kMergeThreads / 32];
  const int64_t w = blockIdx.x;
  const int t = (int)(w / a.Hq);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int used = merge_used(a, part, t);
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  if (used == 0) return;
  const float2 *ml = part.ml + w * part.ns;
  float M = -INFINITY;
  for (int s = threadIdx.x; s < used; s += kMergeThreads) {
    const float m = __ldcg(&ml[s].x);
    wgt[s] = m;
    M = fmaxf(M, m);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) top[warp] = M;
  __syncthreads();
  M = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
  const float ref = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  for (int s = threadIdx.x; s < used; s += kMergeThreads) {
    const float f = exp2f(wgt[s] - ref);
    wgt[s] = f;
    L = fmaf(__ldcg(&ml[s].y), f, L);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  if (lane == 0) tot[warp] = L;
  __syncthreads();
  L = (tot[0] + tot[1]) + (tot[2] + tot[3]);
  const int cg = threadIdx.x & 15, sg = threadIdx.x >> 4;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = sg; s < used; s += 8) {
    const float4 v =
        __ldcg(reinterpret_cast<const float4 *>(part.o + (w * part.ns + s) * kD) + cg);
    const float f = wgt[s];
    acc.x = fmaf(v.x, f, acc.x);
    acc.y = fmaf(v.y, f, acc.y);
    acc.z = fmaf(v.z, f, acc.z);
    acc.w = fmaf(v.w, f, acc.w);
  }
  red[sg][cg] = acc;
  __syncthreads();
  if (threadIdx.x < kD / 4) {
    float y[4] = {};
    for (int g = 0; g < 8; ++g) {
      const float4 v = red[g][threadIdx.x];
      y[0] += v.x;
      y[1] += v.y;
      y[2] += v.z;
      y[3] += v.w;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] /= L;
    store4<T>(out + w * kD + 4 * threadIdx.x, y);
  }
  if (lse && threadIdx.x == 0) lse[w] = M * kLn2 + logf(L);
}

// ---------------------------------------------------------------------------
// bf16, few rows (decode steps, short verification chunks): up to 16
// packed rows per KV head.  CTA = key split x request, a warp per KV head (up
// to eight heads a CTA), so that a key's heads are read together.  Keys and
// values are gathered 16 rows at a time by 16-byte cp.async into an
// XOR-swizzled tile, several tiles in flight; the packed rows are the rows of
// m16n8k16 tiles: S = Q K^T with K as the B operand, P reused from the S
// registers for P V.  Bound by the gather from HBM (14 decode steps over 20,000
// to 90,000 entries, 64 / 8 heads: 235 us on the device, 0.94 of the floor, 239
// to 243 for the call); tcgen05 would
// spend a 128-row tile on 8 rows.
// ---------------------------------------------------------------------------
constexpr int kSSt = 3;  // K and V tiles per warp

__global__ void __launch_bounds__(kSHeads * 32, 2)
    chunk_small_kernel(const ChunkBatch a, __nv_bfloat16 *out, float *lse, const ChunkParts part,
                       uint32_t *status) {
  constexpr int kSt = kSSt;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  clear_status(status);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  const int split = blockIdx.x, b = blockIdx.y, g = blockIdx.z * kSHeads + warp;
  const ChunkReq rq = chunk_req(a, b);
  const int grp = a.Hq / a.Hkv, rows = rq.m * grp;
  if (rows == 0 || g >= a.Hkv) return;
  const int c0 = split * part.chunk, c1 = min(rq.limit(rq.m - 1), c0 + part.chunk);
  if (split > 0 && c0 >= c1) return;
  const int nk = max(0, c1 - c0), n_tiles = (nk + kSKeys - 1) / kSKeys;
  const uint32_t wsm = ptx::smem_addr(smem_raw) + warp * kSt * 2 * kSTile;
  int *const idx = reinterpret_cast<int *>(smem_raw + (blockDim.x >> 5) * kSt * 2 * kSTile) +
                   warp * 2 * kSt * kSKeys;
  uint8_t *const wsm_g = smem_raw + warp * kSt * 2 * kSTile;

  // List entries travel by cp.async too, a ring of stages before their rows: a
  // plain load returns only after all copies queued before it (251 -> 236 us).
  auto fetch = [&](int t) {
    const int k = t * kSKeys + lane;
    if (lane < kSKeys && k < nk)
      cp_async4(ptx::smem_addr(idx + t % (2 * kSt) * kSKeys + lane),
                a.kv_indices + (int64_t)rq.beg + c0 + k);
  };
  const __nv_bfloat16 *kp = (const __nv_bfloat16 *)a.k + g * kD;
  const __nv_bfloat16 *vp = (const __nv_bfloat16 *)a.v + g * kD;
  auto issue = [&](int t) {
    if (t < n_tiles) {
      const uint32_t at = wsm + (t % kSt) * 2 * kSTile;
      const int *entry = idx + t % (2 * kSt) * kSKeys;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = (lane >> 3) + 4 * i, ch = lane & 7;
        const bool valid = t * kSKeys + key < nk;
        const int sl = valid ? entry[key] : 0;
        const int64_t off = (int64_t)((unsigned)sl < (unsigned)a.S ? sl : 0) * a.Hkv * kD + ch * 8;
        cp_async16(at + tile_at(key, ch), kp + off, valid);
        cp_async16(at + kSTile + tile_at(key, ch), vp + off, valid);
      }
      fetch(t + kSt);
    }
    asm volatile("cp.async.commit_group;\n" ::: "memory");
  };
#pragma unroll
  for (int t = 0; t < kSt; ++t) fetch(t);

  // Q fragments and the rows' limits (relative to c0)
  uint32_t qa[4][4];
  int lim[2];
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    const int r = gid + 8 * hh;
    const bool ok = r < rows;
    const uint32_t *src = reinterpret_cast<const uint32_t *>(
        (const __nv_bfloat16 *)a.q +
        ((int64_t)(rq.q0 + (ok ? r / grp : 0)) * a.Hq + g * grp + (ok ? r % grp : 0)) * kD);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      qa[ks][hh] = ok ? __ldg(src + ks * 8 + tig) : 0u;
      qa[ks][2 + hh] = ok ? __ldg(src + ks * 8 + tig + 4) : 0u;
    }
    lim[hh] = (ok ? rq.limit(r / grp) : 0) - c0;
  }
  const int lim_min = rq.limit(0) - c0;  // the first token sees the least

  asm volatile("cp.async.wait_all;\n" ::: "memory");
  __syncwarp();
#pragma unroll
  for (int t = 0; t < kSt - 1; ++t) issue(t);

  float o[8][4], m[2], l[2];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  m[0] = m[1] = -INFINITY;
  l[0] = l[1] = 0.f;

  for (int it = 0; it < n_tiles; ++it) {
    issue(it + kSt - 1);
    asm volatile("cp.async.wait_group %0;\n" ::"n"(kSt - 1) : "memory");
    __syncwarp();
    const uint32_t kt = wsm + (it % kSt) * 2 * kSTile, vt = kt + kSTile;
    const int k0 = it * kSKeys;
    const bool ragged = k0 + kSKeys > min(lim_min, nk);
    float s[2][4];
#pragma unroll
    for (int nb = 0; nb < 2; ++nb) s[nb][0] = s[nb][1] = s[nb][2] = s[nb][3] = 0.f;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      uint32_t kb[4];
      const int mi = lane >> 3;
      ldsm4(kt + tile_at((mi >> 1) * 8 + (lane & 7), ks * 2 + (mi & 1)), kb);
      mma16816(s[0], qa[ks], kb[0], kb[1]);
      mma16816(s[1], qa[ks], kb[2], kb[3]);
    }
    if (ragged) {
#pragma unroll
      for (int nb = 0; nb < 2; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (k0 + nb * 8 + 2 * tig + (e & 1) >= min(lim[e >> 1], nk)) s[nb][e] = -INFINITY;
    }
    uint32_t pa[4];
    float alpha[2], ref[2];
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      float mx = fmaxf(fmaxf(s[0][2 * hh], s[0][2 * hh + 1]),
                       fmaxf(s[1][2 * hh], s[1][2 * hh + 1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float mn = fmaxf(m[hh], mx * kScale);
      ref[hh] = mn == -INFINITY ? 0.f : mn;
      alpha[hh] = ptx::ex2(m[hh] - ref[hh]);
      m[hh] = mn;
      l[hh] *= alpha[hh];
    }
#pragma unroll
    for (int nb = 0; nb < 2; ++nb)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[nb][e] = ptx::ex2(fmaf(s[nb][e], kScale, -ref[e >> 1]));
        l[e >> 1] += s[nb][e];
      }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      o[i][0] *= alpha[0];
      o[i][1] *= alpha[0];
      o[i][2] *= alpha[1];
      o[i][3] *= alpha[1];
    }
    // weights rounded to bf16 for the product; their sum l is not
    pa[0] = pack2(s[0][0], s[0][1]);
    pa[1] = pack2(s[0][2], s[0][3]);
    pa[2] = pack2(s[1][0], s[1][1]);
    pa[3] = pack2(s[1][2], s[1][3]);
    if (ragged) {
      // An infinity or NaN in a hidden entry's value would reach every row
      // of the tile as 0 * inf: such values are added to the rows that see
      // them and leave the tile.
      uint4 *vg = reinterpret_cast<uint4 *>(wsm_g + (it % kSt) * 2 * kSTile + kSTile);
      bool odd = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 x = vg[lane + 32 * i];
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) odd |= nonfinite_lo(w[e]) || nonfinite_hi(w[e]);
      }
      if (__any_sync(0xffffffffu, odd)) {
        for (int key = 0; key < kSKeys; ++key)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(
                reinterpret_cast<const uint8_t *>(vg) + tile_at(key, i) + 4 * tig);
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
              if (k0 + key < min(lim[hh], nk)) {
                if (nonfinite_lo(w)) o[i][2 * hh] += __uint_as_float(w << 16);
                if (nonfinite_hi(w)) o[i][2 * hh + 1] += __uint_as_float(w & 0xffff0000u);
              }
          }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 x = vg[lane + 32 * i];
          vg[lane + 32 * i] = make_uint4(finite_or_zero(x.x), finite_or_zero(x.y),
                                         finite_or_zero(x.z), finite_or_zero(x.w));
        }
        __syncwarp();
      }
    }
#pragma unroll
    for (int nb2 = 0; nb2 < 4; ++nb2) {
      const int mi = lane >> 3;
      uint32_t vb[4];
      ldsm4_t(vt + tile_at((mi & 1) * 8 + (lane & 7), nb2 * 2 + (mi >> 1)), vb);
      mma16816(o[2 * nb2], pa, vb[0], vb[1]);
      mma16816(o[2 * nb2 + 1], pa, vb[2], vb[3]);
    }
    __syncwarp();  // the tile's readers are done before it is refilled
  }
  asm volatile("cp.async.wait_group 0;\n" ::: "memory");

#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    float x = l[hh];
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    const int r = gid + 8 * hh;
    if (r >= rows) continue;
    const int64_t row = (int64_t)(rq.q0 + r / grp) * a.Hq + g * grp + r % grp;
    if (part.direct(lim[hh] + c0)) {
      if (split > 0) continue;
      const bool none = lim[hh] <= 0;
      const float inv = none ? 0.f : 1.f / x;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        reinterpret_cast<uint32_t *>(out + row * kD)[4 * i + tig] =
            none ? 0u : pack2(o[i][2 * hh] * inv, o[i][2 * hh + 1] * inv);
      if (lse && tig == 0) lse[row] = none ? -INFINITY : m[hh] * kLn2 + logf(x);
    } else {
      const int64_t pi = row * part.ns + split;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        reinterpret_cast<float2 *>(part.o + pi * kD)[4 * i + tig] =
            make_float2(o[i][2 * hh], o[i][2 * hh + 1]);
      if (tig == 0) part.ml[pi] = make_float2(m[hh], x);
    }
  }
}

// ---------------------------------------------------------------------------
// bf16, more rows: tcgen05.  CTA = kTiles tiles of 128 packed rows of one KV
// head (both read the same K/V windows) x one key split.
//   warps 4 i .. 4 i + 3  softmax of tile i (thread = packed row = TMEM lane)
//   then the producer warps: K and V windows of 96 keys through a ring of
//        stages, gathered by 16-byte cp.async into the 128-byte-swizzled layout
//        that the MMA reads.  (TMA gathers of four rows deliver one 128-byte
//        row per 24 clocks: 353 TFLOP/s at 1,024 rows over 16,384 entries.)
//   then the MMA warp: TMEM allocation, one thread issuing tcgen05.mma
// TMEM columns: three (one tile: one) score buffers of 96, then O_i (80 each),
// then Q_i (32 each).  Q_i (bf16 pairs) is the A operand of S_i = Q_i K^T; P_i
// overwrites the first 48 columns of its S_i as bf16 pairs and is the A operand
// of O_i += P_i V.  bf16 throughout, because A and B of one MMA have one type
// and the pool is bf16.  Two row sums: the softmax threads add the unrounded
// weights, so that the log-sum-exp is good to fp32, and V has 16 more columns of
// ones (a 2 KB tile that every window's last columns point at), so that the MMA
// adds the rounded ones.  The output is divided by that second sum: an average
// of V rows whose weights sum to 1, so that where few entries carry a row the
// rounding of their weights hardly shows (error against 64 bits 2.3e-3 ->
// 1.8e-3 on a mixed batch, of which the output's own rounding is 1.6e-3).
//
// With two tiles the MMA thread issues, per window, O_0 += P_0 V, S_1 of the
// next window, O_1 += P_1 V, S_0 of the window after that: the third score
// buffer lets a tile's scores be ready before its softmax asks for them, and 96
// is the window that three buffers, two O and two Q leave room for in 512
// columns (with 128 keys, two buffers and scores that wait for P V: 7.71
// instead of 7.52 ms at 2 x 4,096 rows over 50k-70k entries, a mixed batch 185
// instead of 170 us).  With copies, weights and most MMAs taken out in turn the
// kernel ran at 5.0 ms (copies alone), 6.4 ms (no copies) and 4.1 ms (barriers,
// TMEM loads and stores), from 7.5 to 6.9 ms in all: what bounds it, 6.5 to 6.6 ms
// now, is the softmax threads' chain of TMEM load, weights, TMEM store and
// barrier, lengthened by the copies.
//
// Hidden entries.  Windows from the first tile's limit on are masked per row.
// There a weight of 0 would still turn a hidden infinity or NaN of V into
// NaN, so the softmax threads look the V window over first, clear such values
// and remember; a row that sees one adds it at the end.
//
// Every wait is bounded: one that runs out marks the CTA (later waits return
// at the next poll) and the workspace's status word, and the CTA still frees
// its TMEM.  The named barriers are reached equally often whatever the waits
// return.
// ---------------------------------------------------------------------------
constexpr int kBarP = 3;         // hardware barriers kBarP + i (0 is __syncthreads)
constexpr int kBarAll = 2;       // all warps, after a pass
constexpr float kRescale = 8.f;       // log2 units by which a maximum may pass the reference
constexpr float kRaise = 65536.f;     // the row sum that raises it
constexpr float kHuge = 1.2089258e24f;  // 2^80: a window's sum that was computed too far above it
constexpr uint32_t kFar = 0x71800000u;  // 2^100: an output sum that says so too (its bits)

constexpr uint32_t kOnesBytes = 16 * kD * 2;
constexpr uint32_t kOCols = kD + 16;  // V's columns and the ones

constexpr int kWin = 96;                        // keys of a window
constexpr uint32_t kWinBytes = kWin * kD * 2;   // of K, and of V
constexpr int tc_stages(int tiles) { return tiles == 1 ? 4 : 6; }
constexpr int tc_bufs(int tiles) { return tiles == 1 ? 1 : 3; }  // of scores
// Warps: the softmax groups (a warpgroup each), then a warpgroup of three
// producers and the MMA warp.  A softmax thread holds a row of 96 scores, so
// registers move to these (setmaxnreg): with one tile 200 + 56 of 2 x 128
// launched, two CTAs per SM; with two tiles 2 x 224 + 56 of 3 x 168, one CTA.
// Three producers keep up, since they wait for no load (seven, and every
// barrier with more warps: 7.14 instead of 6.87 ms for 2 x 4,096 rows over
// 50k-70k entries, 360 instead of 351 us for 14 chunks of 32 over 50,000); the
// first windows are copied by all warps.
constexpr int kProducers = 3;
constexpr int tc_threads(int tiles) { return 128 * tiles + 128; }
constexpr int tc_launch_regs(int tiles) { return tiles == 1 ? 128 : 168; }
constexpr int tc_softmax_regs(int tiles) { return tiles == 1 ? 200 : 224; }
constexpr int kOtherRegs = 56;
static_assert(tc_softmax_regs(1) + kOtherRegs == 2 * tc_launch_regs(1) &&
                  2 * tc_softmax_regs(2) + kOtherRegs == 3 * tc_launch_regs(2),
              "the shares add up to the launch's");

template <int kTiles>
struct __align__(1024) TcSmem {
  uint8_t k[tc_stages(kTiles)][kWinBytes];
  uint8_t v[tc_stages(kTiles)][kWinBytes];
  uint8_t ones[kOnesBytes];  // 16 keys
  int idx[2 * tc_stages(kTiles)][kWin];  // list entries of windows to come
  uint64_t bar_s[kTiles][2], bar_o[kTiles], bar_done;
  uint32_t tmem_base;
  uint32_t gave_up;  // a wait of this CTA ran out
  uint32_t odd;      // V windows held an infinity or NaN beside hidden entries
  uint32_t again;    // weights were computed too far above their reference
};

template <int kTiles>
__global__ void __launch_bounds__(tc_threads(kTiles), kTiles == 1 ? 2 : 1)
    chunk_tc_kernel(const ChunkBatch a, __nv_bfloat16 *__restrict__ out, float *__restrict__ lse,
                    const ChunkParts part, uint32_t *status) {
  constexpr int kSt = tc_stages(kTiles), kFill = kTiles;
  constexpr int kProdWarp = 4 * kTiles, kMmaWarp = kProdWarp + kProducers;
  // a softmax group, the producers, the MMA warp
  constexpr int kBarPCount = 128 + 32 * kProducers + 32;
  constexpr uint32_t kCols = kTiles == 1 ? 256 : 512;
  constexpr int kBufs = tc_bufs(kTiles);
  constexpr uint32_t kColO = kWin * kBufs, kColQ = kColO + kOCols * kTiles;
  static_assert(kColQ + 32 * kTiles <= kCols, "TMEM columns");
  extern __shared__ uint8_t smem_raw[];
  TcSmem<kTiles> &sm = *reinterpret_cast<TcSmem<kTiles> *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  clear_status(status);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the last row tiles see the most: they come first
  const int split = blockIdx.x % part.ns, g = blockIdx.y, b = blockIdx.z;
  const int64_t r0 = (int64_t)(gridDim.x / part.ns - 1 - blockIdx.x / part.ns) * (kTiles * kTcRows);
  const ChunkReq rq = chunk_req(a, b);
  const int grp = a.Hq / a.Hkv;
  const int64_t rows = (int64_t)rq.m * grp;
  if (r0 >= rows) return;
  const int64_t r1 = min(rows, r0 + kTiles * kTcRows);
  const int c0 = split * part.chunk;
  const int c1 = min(rq.limit((int)((r1 - 1) / grp)), c0 + part.chunk);
  if (split > 0 && c0 >= c1) return;  // the merge reads only splits with visible entries
  const int n_win = c1 > c0 ? (c1 - c0 + kWin - 1) / kWin : 0;
  // first window with an entry hidden from a row of this CTA (or past c1)
  const int w_ragged = max(0, min(rq.limit((int)(r0 / grp)), c1) - c0) / kWin;

  // this thread's packed row
  const int i = warp >> 2;
  const int64_t r = r0 + threadIdx.x;
  const bool valid = warp < kProdWarp && r < r1;
  const int lim = valid ? rq.limit((int)(r / grp)) : 0;
  const int64_t row = valid ? (int64_t)(rq.q0 + (int)(r / grp)) * a.Hq + g * grp + (int)(r % grp) : 0;
  uint32_t qw[32];  // read before copies are queued
  if (warp < kProdWarp) {
    const uint4 *src = reinterpret_cast<const uint4 *>((const __nv_bfloat16 *)a.q + row * kD);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const uint4 x = valid ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
      qw[4 * c] = x.x;
      qw[4 * c + 1] = x.y;
      qw[4 * c + 2] = x.z;
      qw[4 * c + 3] = x.w;
    }
  }

  // Windows 0 .. kFill - 1, by all warps: a step is four entries, eight lanes
  // each.
  constexpr int kWarps = tc_threads(kTiles) / 32, kFillSteps = kWin / 4 * kFill / kWarps;
  static_assert(kFillSteps * kWarps * 4 == kWin * kFill, "whole steps");
  const uint32_t pitch = (uint32_t)a.Hkv * kD * 2;
  const int ch = lane & 7;
  // A step of the producers' copies is four entries; this one takes kSteps from
  // s0 on of every window (the other warps none).  It fetches their list entries
  // itself, a ring of stages before the rows, by cp.async too: a plain load
  // returns only after all copies queued before it, which held the copies to 2
  // bytes per clock and warp instead of 12 (8.2 -> 7.7 ms with loads two windows
  // ahead, 7.5 -> 7.2 ms without loads).
  constexpr int kSteps = kWin / 4 / kProducers, kRing = 2 * kSt;
  static_assert(4 * kSteps * kProducers == kWin && 4 * kSteps <= 32, "a lane fetches one entry");
  const int s0 = (warp - kProdWarp) * kSteps;
  auto fetch = [&](int n) {
    const int x = 4 * s0 + lane, j = c0 + n * kWin + x;
    if (lane < 4 * kSteps && n < n_win && j < c1)
      cp_async4(ptx::smem_addr(&sm.idx[n % kRing][x]), a.kv_indices + (int64_t)rq.beg + j);
  };
  const char *kg = (const char *)a.k + (g * kD + ch * 8) * 2;
  const char *vg = (const char *)a.v + (g * kD + ch * 8) * 2;
  {
    // the producers' entries of the other stages: loads too, as no copies are
    // queued yet
    const bool producer = warp >= kProdWarp && warp < kMmaWarp;
    const int own = 4 * s0 + lane;
    int stage[kSt - kFill];
    if (producer)
#pragma unroll
      for (int n = kFill; n < kSt; ++n) {
        const int j = c0 + n * kWin + own;
        stage[n - kFill] = lane < 4 * kSteps && n < n_win && j < c1 ? (int)chunk_slot(a, rq, j) : 0;
      }
    int fill[kFillSteps];
#pragma unroll
    for (int e = 0; e < kFillSteps; ++e) {
      const int j = c0 + 4 * (warp * kFillSteps + e) + (lane >> 3);
      fill[e] = j < c1 ? (int)chunk_slot(a, rq, j) : -1;
    }
#pragma unroll
    for (int e = 0; e < kFillSteps; ++e) {
      const int x = 4 * (warp * kFillSteps + e) + (lane >> 3);  // row of the windows, one after the other
      const uint32_t to = x * 128 + ((ch ^ (x & 7)) << 4);
      const uint64_t off = (uint64_t)max(fill[e], 0) * pitch;
      cp_async16(ptx::smem_addr(sm.k[0]) + to, kg + off, fill[e] >= 0);  // past the end: zeros
      cp_async16(ptx::smem_addr(sm.v[0]) + to, vg + off, fill[e] >= 0);
    }
    if (producer) {
#pragma unroll
      for (int n = kFill; n < kSt; ++n)
        if (lane < 4 * kSteps) sm.idx[n][own] = stage[n - kFill];
      for (int n = kSt; n < kRing; ++n) fetch(n);
    }
    asm volatile("cp.async.commit_group;\n" ::: "memory");
  }
  for (int c = threadIdx.x; c < (int)kOnesBytes / 4; c += tc_threads(kTiles))
    reinterpret_cast<uint32_t *>(sm.ones)[c] = 0x3f803f80u;
  // this warp's copies of those windows (and its ones), before its first barrier
  auto filled = [] {
    asm volatile("cp.async.wait_group 0;\n" ::: "memory");
    ptx::fence_proxy_async_smem();
    __syncwarp();
  };

  if (threadIdx.x == 0) {
    for (int x = 0; x < kTiles; ++x) {
      ptx::mbar_init(&sm.bar_s[x][0], 1);
      ptx::mbar_init(&sm.bar_s[x][1], 1);
      ptx::mbar_init(&sm.bar_o[x], 1);
    }
    ptx::mbar_init(&sm.bar_done, 1);
    sm.gave_up = sm.odd = sm.again = 0u;
    ptx::fence_barrier_init();
  }
  if (warp == kMmaWarp) ptx::tmem_alloc(&sm.tmem_base, kCols);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  const bool two = kTiles == 2 && r0 + kTcRows < r1;  // tile 1 has rows
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    if (!ptx::mbar_wait_grid(bar, parity, &sm.gave_up, 1u, kTcWaitBudget))
      atomicOr(status, kStatusWaitTimeout);
  };

  // Every warp, after a pass: whether there is another.  All copies and MMAs of
  // the pass are done when the barrier opens.
  auto run_again = [&](int pass) {
    ptx::named_bar_sync(kBarAll, tc_threads(kTiles));
    return pass == 0 && *(volatile uint32_t *)&sm.again != 0u;
  };

  if (warp >= kProdWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kOtherRegs));
    if (warp < kMmaWarp) {
      // A window is kWin rows of K and of V, 16 bytes per lane and copy, eight
      // lanes a row.  A stage is refilled without a wait: when tile 0's barrier of
      // window n opens, its softmax has seen S_0(n), whose commit tracks every MMA
      // issued before it.  With one tile that is P.V(n - 1), the last reader of
      // window n - 1, which is refilled; with two tiles S_0(n) was issued two
      // windows ahead, right behind P.V(n - 2) of both, so that only window
      // n - 2 may be (window n - 1 may still be read).  Each window is one group
      // of copies (empty past the end), with the list entries of the window kSt
      // further on, so that "window w has landed" is a count of groups still in
      // flight.
      const int key0 = 4 * s0 + (lane >> 3);
      const uint32_t kd = ptx::smem_addr(sm.k[0]) + key0 * 128;
      const uint32_t sw0 = (ch ^ (key0 & 7)) << 4, sw1 = (ch ^ ((key0 + 4) & 7)) << 4;
      // steps [from, to) of window n
      auto copy = [&](int n, int from, int to) {
        if (n >= n_win) return;
        const uint32_t at = (n % kSt) * kWinBytes, k0 = kd + at + sw0, k1 = kd + at + sw1;
        const int *entry = sm.idx[n % kRing] + key0;
        const int left = c1 - (c0 + n * kWin + key0);
        // whole windows without the tests of a last one, and rows at 32 x 32-bit
        // products: the producers' instructions compete with the softmax warps'
        // (7 % of the call for 2 x 4,096 rows over 50k-70k entries)
        auto steps = [&](auto whole) {
#pragma unroll
          for (int s = 0; s < kSteps; ++s) {
            if (s >= from && s < to) {
              const bool listed = decltype(whole)::value || 4 * s < left;
              const uint32_t slot = listed ? entry[4 * s] : 0;
              const uint64_t off = (uint64_t)(slot < (uint32_t)a.S ? slot : 0u) * pitch;
              const uint32_t dst = (s & 1 ? k1 : k0) + s * 512;
              cp_async16(dst, kg + off, listed);
              cp_async16(dst + kSt * kWinBytes, vg + off, listed);
            }
          }
        };
        if (c0 + (n + 1) * kWin <= c1) steps(std::true_type());
        else steps(std::false_type());
      };
      auto commit = [] { asm volatile("cp.async.commit_group;\n" ::: "memory"); };
      // every window but the newest `pending` has landed and is visible to the
      // tensor core
      auto landed = [&](auto pending) {
        asm volatile("cp.async.wait_group %0;\n" ::"n"(decltype(pending)::value) : "memory");
        ptx::fence_proxy_async_smem();
        __syncwarp();
      };
      // the first pass's other stages: two before the first barrier, the rest
      // behind it
      constexpr int kEarly = kFill + 2;
#pragma unroll 1
      for (int n = kFill; n < kEarly; ++n) {
        copy(n, 0, kSteps);
        commit();
      }
      for (int pass = 0;; ++pass) {
        landed(std::integral_constant<int, kEarly - kFill>());  // windows 0 .. kFill - 1
        ptx::named_bar_sync(kBarP, kBarPCount);
        if (kTiles == 2) ptx::named_bar_sync(kBarP + 1, kBarPCount);
#pragma unroll 1
        for (int n = kEarly; n < kSt; ++n) {
          copy(n, 0, kSteps);
          commit();
        }
        for (int n = 0; n < n_win; ++n) {
          if constexpr (kTiles == 1) {
            landed(std::integral_constant<int, kSt - 3>());  // window n + 1
            ptx::named_bar_sync(kBarP, kBarPCount);
            if (n >= 1) {
              copy(n - 1 + kSt, 0, kSteps);
              fetch(n - 1 + 2 * kSt);
              commit();
            }
          } else {
            // a window's copies are issued in two parts, so that neither tile's
            // barrier waits for all of them
            constexpr int kPart = (kSteps + 1) / 2;
            ptx::named_bar_sync(kBarP, kBarPCount);
            if (n >= 2) copy(n - 2 + kSt, 0, kPart);
            // window n + 2; the newest group is window max(kSt - 1, n - 3 + kSt)
            if (n == 0) landed(std::integral_constant<int, kSt - 3>());
            else if (n == 1) landed(std::integral_constant<int, kSt - 4>());
            else landed(std::integral_constant<int, kSt - 5>());
            ptx::named_bar_sync(kBarP + 1, kBarPCount);
            if (n >= 2) {
              copy(n - 2 + kSt, kPart, kSteps);
              fetch(n - 2 + 2 * kSt);
              commit();
            }
          }
        }
        if (!run_again(pass)) break;
        // the ring's first fill once more, by the producers alone
#pragma unroll 1
        for (int n = 0; n < kRing; ++n) fetch(n);
        asm volatile("cp.async.wait_all;\n" ::: "memory");
        __syncwarp();
#pragma unroll 1
        for (int n = 0; n < kEarly; ++n) {
          copy(n, 0, kSteps);
          if (n >= kFill - 1) commit();
        }
      }
      asm volatile("cp.async.wait_group 0;\n" ::: "memory");
    } else {
      constexpr uint32_t idS = ptx::idesc_bf16(128, kWin, false);
      constexpr uint32_t idO = ptx::idesc_bf16(128, kOCols, true);
      constexpr uint64_t kTileStep = kWinBytes >> 4;
      // B of P V: 16 keys of V, and its columns 64 .. 79 at an offset (LBO) that
      // leads to the ones from any window and key step: as the address grows,
      // the offset shrinks
      constexpr uint64_t kVUnit = 1 - ((uint64_t)1 << 16);
      const uint64_t dk = ptx::sdesc_sw128(ptx::smem_addr(sm.k[0]));
      const uint64_t dv =
          ptx::sdesc_sw128(ptx::smem_addr(sm.v[0]), ptx::smem_addr(sm.ones) - ptx::smem_addr(sm.v[0]));
      filled();
      auto buf = [&](int t, int n) { return tmem + kWin * ((kTiles * n + t) % kBufs); };
      auto issue_s = [&](int t, int n, int seq) {
        const uint32_t s = buf(t, n), st = n % kSt;
        if (!ptx::elect_one()) return;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          ptx::mma_f16_ts(s, tmem + kColQ + 32 * t + 8 * kk, dk + st * kTileStep + 2 * kk, idS, kk > 0);
        ptx::mma_commit(&sm.bar_s[t][seq & 1]);
      };
      auto issue_o = [&](int t, int n) {
        const uint32_t p = buf(t, n), st = n % kSt;
        if (!ptx::elect_one()) return;
#pragma unroll
        for (int kk = 0; kk < kWin / 16; ++kk)
          ptx::mma_f16_ts(tmem + kColO + kOCols * t, p + 8 * kk,
                          dv + (st * kTileStep + 128 * kk) * kVUnit, idO, (n > 0 || kk > 0) ? 1u : 0u);
        ptx::mma_commit(&sm.bar_o[t]);
      };
      for (int pass = 0;; ++pass) {
        const int seq = pass * n_win;  // of window 0
        ptx::named_bar_sync(kBarP, kBarPCount);  // Q_0 in TMEM, the first windows landed
        if (kTiles == 2) ptx::named_bar_sync(kBarP + 1, kBarPCount);
        ptx::tc_fence_after();
        if (n_win > 0) {
          issue_s(0, 0, seq);
          if (two) issue_s(kTiles - 1, 0, seq);
          if (kTiles == 2 && n_win > 1) issue_s(0, 1, seq + 1);
        }
        for (int n = 0; n < n_win; ++n) {
          ptx::named_bar_sync(kBarP, kBarPCount);  // P_0(n) in TMEM
          ptx::tc_fence_after();
          issue_o(0, n);
          if (kTiles == 1) {
            if (n + 1 < n_win) issue_s(0, n + 1, seq + n + 1);
          } else {
            if (two && n + 1 < n_win) issue_s(kTiles - 1, n + 1, seq + n + 1);
            ptx::named_bar_sync(kBarP + 1, kBarPCount);  // P_1(n) in TMEM, window n + 2 landed
            ptx::tc_fence_after();
            if (two) issue_o(kTiles - 1, n);
            if (n + 2 < n_win) issue_s(0, n + 2, seq + n + 2);
          }
        }
        if (ptx::elect_one()) ptx::mma_commit(&sm.bar_done);
        __syncwarp();
        wait(&sm.bar_done, pass & 1);
        if (!run_again(pass)) break;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(tc_softmax_regs(kTiles)));
    if (i == 1 && !two) {
      // no row in this tile: only the barriers
      filled();
      ptx::named_bar_sync(kBarP + 1, kBarPCount);
      for (int pass = 0;; ++pass) {
        for (int n = 0; n < n_win; ++n) ptx::named_bar_sync(kBarP + 1, kBarPCount);
        wait(&sm.bar_done, pass & 1);
        if (!run_again(pass)) break;
        ptx::named_bar_sync(kBarP + 1, kBarPCount);
      }
    } else {
      const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t tS0 = tmem + lane_base, tO = tmem + lane_base + kColO + kOCols * i;
      ptx::tmem_st32(tmem + lane_base + kColQ + 32 * i, qw);
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      filled();
      ptx::named_bar_sync(kBarP + i, kBarPCount);
      const float2 scale2 = make_float2(kScale, kScale);
      // Weights are 2^(score - m_run) with m_run any reference, not the running
      // maximum: the first window's maximum, raised by l's exponent whenever l
      // has passed 2^16.  fp32 and bf16 hold 2^(+-126), so a reference far
      // below the maximum costs no precision, and the windows after the first
      // need no maximum (9.2 -> 8.6 ms for 2 x 4,096 rows over 50k-70k entries).
      // If a window's weights sum to 2^80 or more (its scores jump by 55 over
      // all before it), or a row's output sums end at 2^100 or more, infinite
      // or NaN (a smaller jump, but large values: their product left fp32's
      // range, or would in the merge), the whole CTA runs once more with exact
      // maxima.  No weight is above 1 then, and no sum above 2^17 values.
      float m_run = -INFINITY, l = 0.f, neg = 0.f;  // neg: -m_run, 0 while there is none
      uint32_t o[64];  // output sums, after a pass
      for (int pass = 0;; ++pass) {
        const float slack = pass > 0 ? 0.f : kRescale;
        uint32_t s_col = kWin * i;
        bool huge = false, fresh = true;  // rows that have no reference yet
        for (int n = 0; n < n_win; ++n) {
          const int seq = pass * n_win + n;
          wait(&sm.bar_s[i][seq & 1], (seq >> 1) & 1);
          ptx::tc_fence_after();
          const uint32_t tS = tS0 + s_col;
          if (kBufs > 1) s_col = s_col == 0 ? 2 * kWin : s_col - kWin;  // buffer (2 n + i) % 3
          float alpha = 1.f;  // what the sums so far are scaled by
          bool scaled = false;
          if (__any_sync(0xffffffffu, l > kRaise)) {
            if (l > kRaise) {
              const int e = min(127, (int)(__float_as_uint(l) >> 23) - 127);
              m_run += (float)e;
              alpha = __uint_as_float((uint32_t)(127 - e) << 23);
            }
            neg = m_run == -INFINITY ? 0.f : -m_run;
            scaled = true;
          }
          uint32_t sr[kWin];
#pragma unroll
          for (int c = 0; c < kWin / 32; ++c) ptx::tmem_ld32(tS + 32 * c, sr + 32 * c);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < kWin / 32; ++c) ptx::reg_fence32(sr + 32 * c);
          if (fresh || n >= w_ragged) {
            if (n >= w_ragged) {
              const int seen = min(lim, c1) - (c0 + n * kWin);
#pragma unroll
              for (int c = 0; c < kWin; ++c)
                if (c >= seen) sr[c] = 0xff800000u;  // -inf
            }
            float mx8[8];
#pragma unroll
            for (int k8 = 0; k8 < 8; ++k8) mx8[k8] = -INFINITY;
#pragma unroll
            for (int c = 0; c < kWin; c += 16)
#pragma unroll
              for (int k8 = 0; k8 < 8; ++k8)
                mx8[k8] =
                    ptx::max3(mx8[k8], __uint_as_float(sr[c + k8]), __uint_as_float(sr[c + 8 + k8]));
            const float mx = fmaxf(ptx::max3(mx8[0], mx8[1], mx8[2]),
                                   fmaxf(ptx::max3(mx8[3], mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])));
            const float m_new = fmaxf(m_run, mx * kScale);
            if (m_new > m_run + slack) {
              alpha *= ptx::ex2(m_run - m_new);  // 0 on the first raise from -inf
              m_run = m_new;
            }
            fresh = pass > 0 || __any_sync(0xffffffffu, m_run == -INFINITY);
            neg = m_run == -INFINITY ? 0.f : -m_run;
            scaled |= __any_sync(0xffffffffu, alpha != 1.f) != 0;
          }
          const float2 neg2 = make_float2(neg, neg);
          // weights in fp32, summed as they are (in two chains, so that no
          // addition waits for the one before), rounded to bf16 pairs: word k
          // holds keys 2 k, 2 k + 1 and overwrites score column k, already read
          float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int qtr = 0; qtr < kWin / 32; ++qtr) {
            uint32_t pw[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const int c = 2 * (16 * qtr + k);
              const float2 x = __ffma2_rn(
                  make_float2(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), scale2, neg2);
              const float2 p = make_float2(ptx::ex2(x.x), ptx::ex2(x.y));
              l2[k & 1] = __fadd2_rn(l2[k & 1], p);
              pw[k] = pack2(p.x, p.y);
            }
            ptx::tmem_st16(tS + 16 * qtr, pw);
          }
          const float2 la = __fadd2_rn(l2[0], l2[1]);
          const float lw = la.x + la.y;
          huge |= !(lw < kHuge);
          l = fmaf(l, alpha, lw);
          if (n > 0 && scaled) {
            wait(&sm.bar_o[i], (seq - 1) & 1);  // P.V(n - 1)
            ptx::tc_fence_after();
#pragma unroll
            for (int hlf = 0; hlf < 2; ++hlf) {
              uint32_t o[32];
              ptx::tmem_ld32(tO + 32 * hlf, o);
              ptx::tmem_wait_ld();
              ptx::reg_fence32(o);
#pragma unroll
              for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
              ptx::tmem_st32(tO + 32 * hlf, o);
            }
            uint32_t sum[16];  // of the rounded weights, in each column
            ptx::tmem_ld16(tO + kD, sum);
            ptx::tmem_wait_ld();
            ptx::reg_fence16(sum);
#pragma unroll
            for (int c = 0; c < 16; ++c) sum[c] = __float_as_uint(__uint_as_float(sum[c]) * alpha);
            ptx::tmem_st16(tO + kD, sum);
          }
          if (n >= w_ragged) {
            uint4 *v4 = reinterpret_cast<uint4 *>(sm.v[n % kSt]);
            for (int c = threadIdx.x & 127; c < (int)(kWinBytes / 16); c += 128) {
              const uint4 x = v4[c];
              const uint4 y = make_uint4(finite_or_zero(x.x), finite_or_zero(x.y), finite_or_zero(x.z),
                                         finite_or_zero(x.w));
              if (x.x != y.x || x.y != y.y || x.z != y.z || x.w != y.w) {
                *(volatile uint32_t *)&sm.odd = 1u;
                __threadfence_block();
                v4[c] = y;
              }
            }
            ptx::fence_proxy_async_smem();  // before the tensor core reads the window
          }
          ptx::tmem_wait_st();
          ptx::tc_fence_before();
          ptx::named_bar_sync(kBarP + i, kBarPCount);
        }
        wait(&sm.bar_done, pass & 1);  // the last P.V
        ptx::tc_fence_after();
        if (n_win > 0) {
          ptx::tmem_ld32(tO, o);
          ptx::tmem_ld32(tO + 32, o + 32);
          ptx::tmem_wait_ld();
          ptx::reg_fence32(o);
          ptx::reg_fence32(o + 32);
          uint32_t top = 0u;
#pragma unroll
          for (int c = 0; c < 64; ++c) top = max(top, o[c] & 0x7fffffffu);
          huge |= top >= kFar;
        } else {
#pragma unroll
          for (int c = 0; c < 64; ++c) o[c] = 0u;
        }
        if (valid && huge && pass == 0) *(volatile uint32_t *)&sm.again = 1u;
        ptx::tc_fence_before();
        if (!run_again(pass)) break;
        m_run = -INFINITY;
        l = neg = 0.f;
        ptx::named_bar_sync(kBarP + i, kBarPCount);  // window 0 landed again
      }
      ptx::tc_fence_after();
      float l_rounded = 0.f;
      if (n_win > 0) {
        uint32_t sum[16];
        ptx::tmem_ld16(tO + kD, sum);
        ptx::tmem_wait_ld();
        ptx::reg_fence16(sum);
        l_rounded = __uint_as_float(sum[0]);
      }
      if (*(volatile uint32_t *)&sm.odd && valid) {
        for (int j = c0 + w_ragged * kWin; j < min(lim, c1); ++j) {
          const uint4 *src = reinterpret_cast<const uint4 *>(
              (const __nv_bfloat16 *)a.v + (chunk_slot(a, rq, j) * a.Hkv + g) * kD);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint4 x = __ldg(src + c);
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int d = 8 * c + 2 * e;
              if (nonfinite_lo(w[e]))
                o[d] = __float_as_uint(__uint_as_float(o[d]) + __uint_as_float(w[e] << 16));
              if (nonfinite_hi(w[e]))
                o[d + 1] = __float_as_uint(__uint_as_float(o[d + 1]) + __uint_as_float(w[e] & 0xffff0000u));
            }
          }
        }
      }
      const bool direct = part.direct(lim);
      if (valid && direct && split == 0) {
        const bool none = lim == 0;
        const float inv = none ? 0.f : 1.f / l_rounded;
        uint4 *dst = reinterpret_cast<uint4 *>(out + row * kD);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t w4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w4[e] = none ? 0u : pack2(__uint_as_float(o[8 * c + 2 * e]) * inv,
                                      __uint_as_float(o[8 * c + 2 * e + 1]) * inv);
          dst[c] = make_uint4(w4[0], w4[1], w4[2], w4[3]);
        }
        if (lse) lse[row] = none ? -INFINITY : m_run * kLn2 + logf(l);
      } else if (valid && !direct) {
        const int64_t pi = row * part.ns + split;
        float4 *dst = reinterpret_cast<float4 *>(part.o + pi * kD);
        const float to_l = l_rounded > 0.f ? l / l_rounded : 1.f;  // the merge divides by l
#pragma unroll
        for (int c = 0; c < 16; ++c)
          dst[c] = make_float4(__uint_as_float(o[4 * c]) * to_l, __uint_as_float(o[4 * c + 1]) * to_l,
                               __uint_as_float(o[4 * c + 2]) * to_l,
                               __uint_as_float(o[4 * c + 3]) * to_l);
        part.ml[pi] = make_float2(m_run, l);
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kCols);
  }
}

// Which kernel takes a call, and its cut of the work.  All of it follows from
// the host's bounds, so that a captured call replays for any lengths within
// them.
struct ChunkPlan {
  int kind;       // CUDA cores; mma.sync; tcgen05 with one or two (+ 1) 128-row tiles
  int ns, chunk;  // key splits and entries of each
  int64_t tiles;  // row tiles of one (request, KV head)
};
constexpr int kF32Kind = 0, kSmallKind = 1, kTcKind = 2;

// Key splits: none if `ctas` (the unsplit grid) reaches `want`; otherwise
// chunks of max_chunk entries halved until it does, but not below `least` --
// and below that, down to `least_idle`, only while SMs would stay idle.
void split_keys(ChunkPlan *p, int64_t ctas, int64_t want, int64_t resident, int max_kv,
                int max_chunk, int least, int least_idle) {
  const auto splits = [&](int c) { return std::max<int64_t>(1, ((int64_t)max_kv + c - 1) / c); };
  p->ns = 1;
  p->chunk = std::max(128, (int)(((int64_t)max_kv + 127) / 128 * 128));
  if (ctas >= want) return;
  int c = max_chunk;
  while (c > least && ctas * splits(c) < want) c /= 2;
  while (c > least_idle && ctas * splits(c) < resident) c /= 2;
  while (splits(c) > kMaxSplit) c *= 2;
  if (splits(c) == 1) return;
  p->chunk = c;
  p->ns = (int)splits(c);
}

// Key splits of the tcgen05 kernels, from what their CTAs measured: `window`
// us for 96 keys beside its neighbours, 8 us to start and end, and the partials
// written and read at 5 TB/s in a merge of 6 us.  The count that ends first when
// every list is max_kv long: the splits then fill whole waves of CTAs (448 CTAs
// of 196 windows instead of 896 of 128 and fewer: 1,078 -> 990 us for 14 chunks
// of 64 over 50,000 entries, at the time).
void split_windows(ChunkPlan *p, int64_t ctas, int64_t slots, double window, double row_bytes,
                   int max_kv) {
  const int windows = std::max(1, (max_kv + kWin - 1) / kWin);
  // at most eight waves, and four windows each
  const int most = (int)std::max<int64_t>(
      1, std::min<int64_t>(std::min(kMaxSplit, windows / 4), 8 * slots / std::max<int64_t>(1, ctas)));
  double best = 0;
  p->ns = 1;
  for (int ns = 1; ns <= most; ++ns) {
    const int per = (windows + ns - 1) / ns;
    if (ns > 1 && per * (ns - 1) >= windows) continue;  // a split would be empty
    const double t = (double)((ctas * ns + slots - 1) / slots) * (per * window + 8) +
                     (ns > 1 ? 6 + ns * row_bytes / 5e6 : 0);
    if (ns == 1 || t < best) {
      best = t;
      p->ns = ns;
    }
  }
  p->chunk = (windows + p->ns - 1) / p->ns * kWin;
}

ChunkPlan chunk_plan(int dtype, int B, int Hq, int Hkv, int n_rows, int max_q, int max_kv) {
  ChunkPlan p;
  const int sms = chunk_sms();
  const int64_t rows = (int64_t)max_q * (Hq / Hkv);
  if (dtype == AKV_BF16 && rows <= 16) {
    p.kind = kSmallKind;
    p.tiles = 1;
    const int warps = std::min(Hkv, kSHeads), per_sm = 16 / warps;
    const int64_t ctas = (int64_t)B * ((Hkv + kSHeads - 1) / kSHeads);
    split_keys(&p, ctas, 8LL * per_sm * sms, (int64_t)per_sm * sms, max_kv, 4096, 1024, 128);
  } else if (dtype == AKV_BF16) {
    p.kind = rows <= kTcRows ? kTcKind : kTcKind + 1;
    const int per_sm = p.kind == kTcKind ? 2 : 1, tile = p.kind == kTcKind ? kTcRows : 2 * kTcRows;
    p.tiles = (rows + tile - 1) / tile;
    split_windows(&p, p.tiles * B * Hkv, (int64_t)per_sm * sms, p.kind == kTcKind ? 1.4 : 0.8,
                  (double)n_rows * Hq * 528, max_kv);
  } else {
    p.kind = kF32Kind;
    p.tiles = (rows + kFRows - 1) / kFRows;
    split_keys(&p, p.tiles * B * Hkv, 4LL * 2 * sms, 2LL * sms, max_kv, 4096, 512, 128);
  }
  return p;
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

cudaError_t launch_f32(const ChunkBatch &a, void *out, float *lse, const ChunkParts &part,
                       int64_t tiles, uint32_t *status, cudaStream_t s) {
  const int smem = (int)sizeof(F32Smem);
  cudaError_t e =
      cudaFuncSetAttribute(chunk_f32_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  chunk_f32_kernel<<<dim3((unsigned)(tiles * part.ns), a.Hkv, a.B), kFThreads, smem, s>>>(
      a, (float *)out, lse, part, status);
  return cudaGetLastError();
}

cudaError_t launch_small(const ChunkBatch &a, void *out, float *lse, const ChunkParts &part,
                         uint32_t *status, cudaStream_t s) {
  const int warps = std::min(a.Hkv, kSHeads), smem = warps * kSSt * 2 * (kSTile + kSKeys * 4);
  cudaError_t e = cudaFuncSetAttribute(chunk_small_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  chunk_small_kernel<<<dim3(part.ns, a.B, (a.Hkv + kSHeads - 1) / kSHeads), warps * 32, smem, s>>>(
      a, (__nv_bfloat16 *)out, lse, part, status);
  return cudaGetLastError();
}

template <int kTiles>
cudaError_t launch_tc(const ChunkBatch &a, void *out, float *lse, const ChunkParts &part,
                      int64_t tiles, uint32_t *status, cudaStream_t s) {
  // the register shares hold for the launch's only: an inc beyond them would
  // wait forever
  static const bool regs_ok = [] {
    cudaFuncAttributes at;
    return cudaFuncGetAttributes(&at, chunk_tc_kernel<kTiles>) == cudaSuccess &&
           at.numRegs == tc_launch_regs(kTiles);
  }();
  if (!regs_ok) return cudaErrorInvalidConfiguration;
  const int smem = (int)sizeof(TcSmem<kTiles>) + 1024;
  cudaError_t e = cudaFuncSetAttribute(chunk_tc_kernel<kTiles>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  chunk_tc_kernel<kTiles><<<dim3((unsigned)(tiles * part.ns), a.Hkv, a.B), tc_threads(kTiles), smem, s>>>(
      a, (__nv_bfloat16 *)out, lse, part, status);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_merge(const ChunkBatch &a, void *out, float *lse, const ChunkParts &part,
                         cudaStream_t s) {
  const int64_t items = (int64_t)a.n_rows * a.Hq;
  const bool warps = part.ns <= kWarpMerge;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(warps ? (items + kMergeWarps - 1) / kMergeWarps : items));
  cfg.blockDim = dim3(warps ? kMergeWarps * 32 : kMergeThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, warps ? chunk_merge_warp_kernel<T> : chunk_merge_kernel<T>, a,
                            (T *)out, lse, part);
}

}  // namespace

int64_t chunk_grid_x(int dtype, int B, int Hq, int Hkv, int n_rows, int max_q, int max_kv) {
  const ChunkPlan p = chunk_plan(dtype, B, Hq, Hkv, n_rows, max_q, max_kv);
  return p.tiles * p.ns;
}

size_t chunk_workspace_bytes(int dtype, int B, int Hq, int Hkv, int n_rows, int max_q, int max_kv) {
  const ChunkPlan p = chunk_plan(dtype, B, Hq, Hkv, n_rows, max_q, max_kv);
  if (p.ns == 1) return kTcStatusBytes;
  const size_t parts = (size_t)n_rows * Hq * p.ns;
  return kTcStatusBytes + up256(parts * sizeof(float2)) + up256(parts * kD * sizeof(float));
}

cudaError_t launch_chunk(int dtype, int B, int Hq, int Hkv, int n_rows, int S,
                         const int32_t *q_indptr, int max_q, const void *q, const void *k,
                         const void *v, const int32_t *kv_indptr, const int32_t *kv_indices,
                         int max_kv, void *out, float *lse, void *ws, cudaStream_t s) {
  const ChunkPlan p = chunk_plan(dtype, B, Hq, Hkv, n_rows, max_q, max_kv);
  const ChunkBatch a{B, Hq, Hkv, n_rows, S, max_q, max_kv, q_indptr, kv_indptr, kv_indices, q, k, v};
  char *const w = (char *)ws + kTcStatusBytes;
  const ChunkParts part{(float2 *)w, (float *)(w + up256((size_t)n_rows * Hq * p.ns * sizeof(float2))),
                        p.ns, p.chunk};
  cudaError_t e;
  if (p.kind == kTcKind) e = launch_tc<1>(a, out, lse, part, p.tiles, (uint32_t *)ws, s);
  else if (p.kind == kTcKind + 1) e = launch_tc<2>(a, out, lse, part, p.tiles, (uint32_t *)ws, s);
  else if (p.kind == kSmallKind) e = launch_small(a, out, lse, part, (uint32_t *)ws, s);
  else e = launch_f32(a, out, lse, part, p.tiles, (uint32_t *)ws, s);
  if (e != cudaSuccess || p.ns == 1) return e;
  return dtype == AKV_BF16 ? launch_merge<__nv_bfloat16>(a, out, lse, part, s)
                           : launch_merge<float>(a, out, lse, part, s);
}

}  // namespace akv
