// Eviction of cache entries by the attention mass they have received, down to
// a budget per request (drop(P) of the paper review page section 3.3, P chosen
// by weight instead of by message).  Request b keeps the min(keep[b], n_b)
// entries of the largest mass, ties to the lowest list index; the first
// n_first and last n_recent entries rank above all others.
//
// A cluster of CTAs takes one request.  The k-th largest key is found by a
// radix select over the 32-bit order-preserving image of the mass, 8 bits a
// round, the CTAs' histograms summed through distributed shared memory; then
// every warp counts its own contiguous part of the list, the counts are
// scanned over warps and CTAs, and the warp streams its part again, writing
// kept and dropped entries in list order by ballot prefix.  No atomics on
// global memory: the result does not depend on timing.
#include "common.cuh"

#include <cooperative_groups.h>

namespace cg = cooperative_groups;

namespace akv {
namespace {

constexpr int kEvThreads = 512;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kCluster = 8;

struct EvictArgs {
  int B, max_kv;
  const int32_t *indptr, *indices, *pos;
  const float *mass;
  int64_t stride;
  const int32_t *keep;
  int n_first, n_recent;
  int32_t *out_indptr, *out_indices, *out_pos;
  float *out_mass;
  int64_t out_stride;
  int64_t out_cap, dropped_cap;  // entries that out_indices / out_pos and dropped hold
  int32_t *dropped_indptr, *dropped;
};

// order-preserving image of the mass; NaN ranks as -inf, -0 as +0
__device__ __forceinline__ uint32_t mass_key(float m) {
  if (!(m == m)) m = -INFINITY;
  const uint32_t u = __float_as_uint(m + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int req_len(const EvictArgs &a, int b) {
  return min(max(a.indptr[b + 1] - a.indptr[b], 0), a.max_kv);
}

__global__ void __launch_bounds__(kEvThreads) evict_kernel(const EvictArgs a) {
  cg::cluster_group cl = cg::this_cluster();
  __shared__ int hist[256];
  __shared__ int warp_n[2][kEvWarps];  // per warp: entries above / equal to the threshold
  __shared__ int cta_n[2];
  __shared__ int pick[2];              // chosen digit, entries still wanted in it
  __shared__ long long base_s[2];
  __shared__ long long red[2][kEvWarps];
  const int b = blockIdx.x / kCluster, rank = blockIdx.x % kCluster;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = req_len(a, b);
  const int kk = min(max(a.keep[b], 0), n);
  const float *mass = a.mass + (int64_t)b * a.stride;
  const int32_t beg = a.indptr[b];

  // where this request's kept and dropped entries start
  long long kept_before = 0, drop_before = 0;
  for (int o = threadIdx.x; o < b; o += kEvThreads) {
    const int no = req_len(a, o), ko = min(max(a.keep[o], 0), no);
    kept_before += ko;
    drop_before += no - ko;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    kept_before += __shfl_xor_sync(0xffffffffu, kept_before, o);
    drop_before += __shfl_xor_sync(0xffffffffu, drop_before, o);
  }
  if (lane == 0) {
    red[0][warp] = kept_before;
    red[1][warp] = drop_before;
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    long long s = 0;
    for (int w = 0; w < kEvWarps; ++w) s += red[threadIdx.x][w];
    base_s[threadIdx.x] = s;
    if (rank == 0) {
      int32_t *ptr = threadIdx.x ? a.dropped_indptr : a.out_indptr;
      if (b == 0) ptr[0] = 0;
      ptr[b + 1] = (int32_t)(s + (threadIdx.x ? n - kk : kk));
    }
  }
  __syncthreads();

  // this CTA's and warp's parts of the list
  const int per_warp = (n + kCluster * kEvWarps - 1) / (kCluster * kEvWarps);
  const int j0 = min(n, (rank * kEvWarps + warp) * per_warp), j1 = min(n, j0 + per_warp);
  auto key_at = [&](int j) -> uint32_t {
    return j < a.n_first || j >= n - a.n_recent ? mass_key(INFINITY) : mass_key(mass[j]);
  };

  // the kk-th largest key
  uint32_t prefix = 0;
  int want = kk;
  for (int shift = 24; kk > 0 && shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += kEvThreads) hist[i] = 0;
    __syncthreads();
    const uint32_t above = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
    for (int j = j0 + lane; j < j1; j += 32) {
      const uint32_t k = key_at(j);
      if ((k & above) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
    }
    cl.sync();
    if (warp == 0) {  // lane l: bins 255 - 8 l .. 248 - 8 l, highest first
      int c[8], sum = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        c[e] = 0;
        for (int o = 0; o < kCluster; ++o) c[e] += cl.map_shared_rank(hist, o)[255 - 8 * lane - e];
        sum += c[e];
      }
      int incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      int left = want - (incl - sum);
      if (left > 0 && left <= sum) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (left > 0 && left <= c[e]) {
            pick[0] = 255 - 8 * lane - e;
            pick[1] = left;
          }
          left -= c[e];
        }
      }
    }
    cl.sync();  // every CTA has read the histograms (and this one its pick)
    prefix |= (uint32_t)pick[0] << shift;
    want = pick[1];
    __syncthreads();
  }
  // kept: keys above `prefix`, and the first `want` equal ones
  int above_n = 0, equal_n = 0;
  if (kk > 0) {
    for (int j = j0 + lane; j < j1; j += 32) {
      const uint32_t k = key_at(j);
      above_n += k > prefix;
      equal_n += k == prefix;
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    above_n += __shfl_xor_sync(0xffffffffu, above_n, o);
    equal_n += __shfl_xor_sync(0xffffffffu, equal_n, o);
  }
  if (lane == 0) {
    warp_n[0][warp] = above_n;
    warp_n[1][warp] = equal_n;
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    int s = 0;
    for (int w = 0; w < kEvWarps; ++w) s += warp_n[threadIdx.x][w];
    cta_n[threadIdx.x] = s;
  }
  cl.sync();
  int above_before = 0, equal_before = 0;
  for (int o = 0; o < rank; ++o) {
    const int *c = cl.map_shared_rank(cta_n, o);
    above_before += c[0];
    equal_before += c[1];
  }
  for (int w = 0; w < warp; ++w) {
    above_before += warp_n[0][w];
    equal_before += warp_n[1][w];
  }
  int kept = above_before + min(equal_before, want);  // kept entries before the next one
  int equal = equal_before;
  const int64_t kept_base = base_s[0], drop_base = base_s[1];
  const uint32_t below = (1u << lane) - 1u;
  for (int j = j0; j < j1; j += 32) {
    const int e = j + lane;
    const bool there = e < j1;
    const uint32_t k = there && kk > 0 ? key_at(e) : 0u;
    const bool eq = there && kk > 0 && k == prefix;
    const uint32_t eqs = __ballot_sync(0xffffffffu, eq);
    const bool keep = there && kk > 0 &&
                      (k > prefix || (eq && equal + __popc(eqs & below) < want));
    const uint32_t keeps = __ballot_sync(0xffffffffu, keep);
    if (there) {
      const int32_t slot = a.indices[(int64_t)beg + e];
      const int kb = kept + __popc(keeps & below);
      if (keep) {
        const int64_t to = kept_base + kb;
        if (to < a.out_cap) {
          a.out_indices[to] = slot;
          if (a.out_pos) a.out_pos[to] = a.pos[(int64_t)beg + e];
        }
        if (kb < a.out_stride) a.out_mass[(int64_t)b * a.out_stride + kb] = mass[e];
      } else if (drop_base + (e - kb) < a.dropped_cap) {
        a.dropped[drop_base + (e - kb)] = slot;
      }
    }
    kept += __popc(keeps);
    equal += __popc(eqs);
  }
  cl.sync();  // a CTA's counts stay readable until every CTA has them
}

}  // namespace

cudaError_t launch_evict(int B, const int32_t *indptr, const int32_t *indices, const int32_t *pos,
                         int max_kv, const float *mass, int64_t stride, const int32_t *keep,
                         int n_first, int n_recent, int32_t *out_indptr, int32_t *out_indices,
                         int32_t *out_pos, float *out_mass, int64_t out_stride,
                         int64_t out_cap, int32_t *dropped_indptr, int32_t *dropped,
                         int64_t dropped_cap, cudaStream_t s) {
  EvictArgs a{B, max_kv, indptr, indices, pos, mass, stride, keep, n_first, n_recent, out_indptr,
              out_indices, out_pos, out_mass, out_stride, out_cap, dropped_cap, dropped_indptr,
              dropped};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)B * kCluster);
  cfg.blockDim = dim3(kEvThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_kernel, a);
}

}  // namespace akv
