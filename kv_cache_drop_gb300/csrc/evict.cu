// Eviction of cache entries by the attention mass they have received, down to
// a budget per request (drop(P) of the paper review page section 3.3, P chosen
// by weight instead of by message).  Request b keeps the min(keep[b], n_b)
// entries of the largest mass, ties to the lowest list index; the first
// n_first and last n_recent entries rank above all others.
//
// A cluster of CTAs takes one request.  The k-th largest key is found by a
// radix select over the 32-bit order-preserving image of the mass, in digits
// of 11, 11 and 10 bits (the first holds two mantissa bits, so that masses of
// one magnitude still spread over several counters), the CTAs' histograms
// summed through distributed shared memory; then every warp counts its own
// contiguous part of the list, the counts are scanned over warps and CTAs, and
// the warp goes over its part again, writing kept and dropped entries in list
// order by ballot prefix.  No atomics on global memory: the result does not
// depend on timing.  Keys of up to 16,384 entries per CTA stay in registers
// between the digits and the count; longer lists' masses are read again for
// each, from L2, eight loads in flight per thread.  The last pass reads masses,
// slots and positions from memory in either case.  14 lists of 20,000 to 90,000
// entries take 17.8 us on the device, one of 1.5 million 81, of which the last
// pass 34: bound by the latency of the passes and of five cluster barriers (short
// lists), and by what one cluster's SMs read and write (long ones).
#include "common.cuh"

#include <cooperative_groups.h>

#include <atomic>

namespace cg = cooperative_groups;

namespace akv {
namespace {

constexpr int kEvThreads = 1024;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kHold = 16;   // keys per thread that stay in registers
constexpr int kBatch = 8;   // loads in flight per thread otherwise
constexpr int kBins = 2048;
static_assert(kEvWarps == 32 && kBins == 64 * kEvWarps, "a lane per warp, 64 bins per warp");
constexpr int kMaxCluster = 16;  // above 8 is not portable: asked for only where it fits

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

// kInRegs: a thread's keys (entries j0 + 32 e + lane of its warp's part) are
// held in registers.
template <bool kInRegs>
__global__ void __launch_bounds__(kEvThreads) evict_kernel(const EvictArgs a) {
  cg::cluster_group cl = cg::this_cluster();
  __shared__ __align__(16) int hist[2][kBins];  // alternate digits, so that one barrier per digit does
  __shared__ int warp_n[2][kEvWarps];  // per warp: entries above / equal to the threshold
  __shared__ int cta_n[2];
  __shared__ int pick[2];              // chosen digit, entries still wanted in it
  __shared__ int coarse[2][kEvWarps];
  __shared__ long long base_s[2];
  __shared__ long long red[2][kEvWarps];
  const int size = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int b = blockIdx.x / size;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = req_len(a, b);
  const int kk = min(max(a.keep[b], 0), n);
  const float *mass = a.mass + (int64_t)b * a.stride;
  const int32_t beg = a.indptr[b];

  // this warp's part of the list
  const int per_warp = ((n + size * kEvWarps - 1) / (size * kEvWarps) + 31) / 32 * 32;
  const int j0 = (int)min((int64_t)n, (int64_t)(rank * kEvWarps + warp) * per_warp);
  const int j1 = min(n, j0 + per_warp);
  const int fixed_end = min(a.n_first, n), fixed_from = n - min(a.n_recent, n);
  auto key_of = [&](int j, float m) -> uint32_t {
    return mass_key(j < fixed_end || j >= fixed_from ? INFINITY : m);
  };
  // full batches of a part without protected entries skip those tests
  const bool plain = j0 >= fixed_end && j1 <= fixed_from;
  uint32_t held[kInRegs ? kHold : 1];
  if (kInRegs) {
#pragma unroll
    for (int e = 0; e < kHold; ++e) {
      const int j = j0 + 32 * e + lane;
      held[e] = j < j1 ? __float_as_uint(__ldg(mass + j)) : 0u;
    }
#pragma unroll
    for (int e = 0; e < kHold; ++e) held[e] = key_of(j0 + 32 * e + lane, __uint_as_float(held[e]));
  }
  // f(key) for every entry of this lane
  auto each = [&](auto f) {
    if constexpr (kInRegs) {
#pragma unroll
      for (int e = 0; e < kHold; ++e)
        if (j0 + 32 * e + lane < j1) f(held[e]);
    } else {
      int j = j0 + lane;
      if (plain) {
        const float *p = mass + j;
        for (int left = (j1 - j0) / (32 * kBatch); left > 0; --left, p += 32 * kBatch) {
          float m[kBatch];
#pragma unroll
          for (int e = 0; e < kBatch; ++e) m[e] = __ldg(p + 32 * e);
#pragma unroll
          for (int e = 0; e < kBatch; ++e) f(mass_key(m[e]));
        }
        j += (j1 - j0) / (32 * kBatch) * (32 * kBatch);
      }
#pragma unroll 4
      for (; j < j1; j += 32) f(key_of(j, __ldg(mass + j)));
    }
  };

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
  for (int i = threadIdx.x; i < 2 * kBins; i += kEvThreads) (&hist[0][0])[i] = 0;
  __syncthreads();
  if (warp < 2) {
    long long s = red[warp][lane];
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) {
      base_s[warp] = s;
      if (rank == 0) {
        int32_t *ptr = warp ? a.dropped_indptr : a.out_indptr;
        if (b == 0) ptr[0] = 0;
        ptr[b + 1] = (int32_t)(s + (warp ? n - kk : kk));
      }
    }
  }

  // the kk-th largest key, a digit at a time; every CTA comes to it by itself
  uint32_t prefix = 0;
  int want = kk;
  const bool some = kk > 0 && kk < n;  // else all or none are kept
  for (int d = 0; some && d < 3; ++d) {
    const int shift = d == 0 ? 21 : d == 1 ? 10 : 0;
    const uint32_t digit = d == 2 ? 0x3ffu : 0x7ffu;
    const uint32_t above = d == 0 ? 0u : d == 1 ? 0xffe00000u : 0xfffffc00u;
    int *h = hist[d & 1];
    each([&](uint32_t k) {
      if ((k & above) == prefix) atomicAdd(&h[(k >> shift) & digit], 1);
    });
    __syncthreads();
    // Coarse counts of 64 bins, one per warp, so that the cluster's counts are
    // found in two short steps: the coarse bin, then the bin in it.  (Every
    // CTA reading every bin of every other moved 64 KB: 4.2 us a digit.)
    {
      int x = h[64 * warp + lane] + h[64 * warp + 32 + lane];
#pragma unroll
      for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      if (lane == 0) coarse[d & 1][warp] = x;
    }
    cl.sync();
    if (warp == 0) {
      // lane l stands for the coarse bin 31 - l, then for two bins of the one
      // found, highest first
      const auto above_me = [&](int x) {  // sum over the lanes before this one
        int incl = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int t = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += t;
        }
        return incl - x;
      };
      int x = 0;
#pragma unroll 8
      for (int o = 0; o < size; ++o) x += cl.map_shared_rank(coarse[d & 1], o)[31 - lane];
      int left = want - above_me(x);
      const int at = __ffs(__ballot_sync(0xffffffffu, left > 0 && left <= x)) - 1;
      left = __shfl_sync(0xffffffffu, left, at);
      int hi = 0, lo = 0;
      const int bin = 64 * (31 - at) + 62 - 2 * lane;
#pragma unroll 8
      for (int o = 0; o < size; ++o) {
        const int2 v = *reinterpret_cast<const int2 *>(cl.map_shared_rank(h, o) + bin);
        lo += v.x;
        hi += v.y;
      }
      left -= above_me(hi + lo);
      if (left > 0 && left <= hi + lo) {
        pick[0] = left <= hi ? bin + 1 : bin;
        pick[1] = left <= hi ? left : left - hi;
      }
    }
    __syncthreads();
    prefix |= (uint32_t)pick[0] << shift;
    want = pick[1];
    // the other histogram's readers passed this digit's cluster barrier
    if (d == 1)
      for (int i = threadIdx.x; i < kBins; i += kEvThreads) hist[0][i] = 0;
    if (d == 1) __syncthreads();
  }
  // kept: keys above `prefix`, and the first `want` equal ones.  No key is 0
  // (-inf's image is 0x007fffff) and none 0xffffffff: all or none.
  if (!some) {
    prefix = kk > 0 ? 0u : 0xffffffffu;
    want = 0;
  }
  int above_n = 0, equal_n = 0;
  each([&](uint32_t k) {
    above_n += k > prefix;
    equal_n += k == prefix;
  });
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
  if (warp < 2) {  // the warps' counts become what lies before each
    const int x = warp_n[warp][lane];
    int incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    warp_n[warp][lane] = incl - x;
    if (lane == 31) cta_n[warp] = incl;
  }
  cl.sync();
  int above_before = 0, equal_before = 0;
  for (int o = 0; o < rank; ++o) {
    const int *c = cl.map_shared_rank(cta_n, o);
    above_before += c[0];
    equal_before += c[1];
  }
  above_before += warp_n[0][warp];
  equal_before += warp_n[1][warp];
  int kept = above_before + min(equal_before, want);  // kept entries before the next one
  int equal = equal_before;
  const int64_t kept_base = base_s[0], drop_base = base_s[1];
  const uint32_t below = (1u << lane) - 1u;
  // room from this request's first kept and dropped entry on
  const auto room = [](int64_t cap, int64_t base) {
    return (int)max((int64_t)0, min(cap - base, (int64_t)INT32_MAX));
  };
  const int kept_room = room(a.out_cap, kept_base), drop_room = room(a.dropped_cap, drop_base);
  const int mass_room = room(a.out_stride, 0);
  int32_t *const out_idx = a.out_indices + kept_base;
  int32_t *const out_pos = a.out_pos ? a.out_pos + kept_base : nullptr;
  float *const out_mass = a.out_mass + (int64_t)b * a.out_stride;
  int32_t *const out_drop = a.dropped + drop_base;
  // 32 entries: e = this lane's, its mass, slot and position at hand
  auto place = [&](int e, bool there, uint32_t k, float m, int32_t slot, int32_t pos) {
    bool keep = there && k > prefix;
    uint32_t eqs = __ballot_sync(0xffffffffu, there && k == prefix);
    if (eqs) {  // the first `want` of these
      keep |= (eqs >> lane & 1u) && equal + __popc(eqs & below) < want;
      equal += __popc(eqs);
    }
    const uint32_t keeps = __ballot_sync(0xffffffffu, keep);
    const int kb = kept + __popc(keeps & below);
    kept += __popc(keeps);
    if (keep) {
      if (kb < kept_room) {
        out_idx[kb] = slot;
        if (out_pos) out_pos[kb] = pos;
      }
      if (kb < mass_room) out_mass[kb] = m;
    } else if (there && e - kb < drop_room) {
      out_drop[e - kb] = slot;
    }
  };
  const int32_t *idx = a.indices + (int64_t)beg, *pos = a.pos ? a.pos + (int64_t)beg : idx;
  int j = j0;
  if (plain)
    for (; j + 32 * kBatch <= j1; j += 32 * kBatch) {
      float m[kBatch];
      int32_t s[kBatch], p[kBatch];
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        m[e] = __ldg(mass + j + lane + 32 * e);
        s[e] = __ldg(idx + j + lane + 32 * e);
        p[e] = __ldg(pos + j + lane + 32 * e);
      }
#pragma unroll
      for (int e = 0; e < kBatch; ++e)
        place(j + lane + 32 * e, true, mass_key(m[e]), m[e], s[e], p[e]);
    }
#pragma unroll 2
  for (; j < j1; j += 32) {
    const int e = j + lane;
    const bool there = e < j1;
    const float m = there ? __ldg(mass + e) : 0.f;
    place(e, there, key_of(e, m), m, there ? __ldg(idx + e) : 0, there ? __ldg(pos + e) : 0);
  }
  cl.sync();  // a CTA's counts stay readable until every CTA has them
}

// CTAs per request: enough for the lists to stay in registers, up to 8, or 16
// where the device takes such clusters and the requests leave SMs idle.
bool takes_16() {
  static std::atomic<int> known[64];  // per device: 0 not asked, 1 no, 2 yes
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  if (known[dev].load() == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kMaxCluster);
    cfg.blockDim = dim3(kEvThreads);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kMaxCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    const bool ok = cudaFuncSetAttribute(evict_kernel<false>, cudaFuncAttributeNonPortableClusterSizeAllowed,
                                         1) == cudaSuccess &&
                    cudaFuncSetAttribute(evict_kernel<true>, cudaFuncAttributeNonPortableClusterSizeAllowed,
                                         1) == cudaSuccess &&
                    cudaOccupancyMaxActiveClusters(&clusters, evict_kernel<false>, &cfg) == cudaSuccess &&
                    clusters > 0;
    if (!ok) (void)cudaGetLastError();
    known[dev].store(ok ? 2 : 1);
  }
  return known[dev].load() == 2;
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
  constexpr int kPerCta = kHold * kEvThreads;
  int size = 1;
  while (size < 8 && (int64_t)size * kPerCta < max_kv) size *= 2;
  if (size == 8 && max_kv > 8 * kPerCta && B <= 8 && takes_16()) size = kMaxCluster;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(B * size));
  cfg.blockDim = dim3(kEvThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)size;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, max_kv <= size * kPerCta ? evict_kernel<true> : evict_kernel<false>, a);
}

}  // namespace akv
