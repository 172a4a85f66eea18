// Decode over the active cache held in 8 bits (paper review page section 4
// serving flow: decode reads only the active cache; section 3.3: a key moves
// between positions by a rotation).  The pool keeps e4m3 keys before RoPE and
// values, with a power of two per head row (kv8.cuh); every list entry carries
// its position, and
//   s_j = R(q_pos) q . R(pos_j) k_j 2^ks_j / 8,  out = sum_j softmax(s)_j v_j 2^vs_j.
#include "kv8.cuh"

#include <algorithm>

namespace akv {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kScale = 0.125f * kLog2e;  // scores to log2 units

struct Decode8 {
  int B, Hq, Hkv, grp;
  const void *q;
  const int32_t *qpos;
  const void *k_new, *v_new;  // the step's rows, or NULL
  const int32_t *new_slot;
  Kv8Pool pool;
  const int32_t *indptr, *indices, *kvpos;
  int max_kv;
  // split-KV partials [B][Hq][ns]: (maximum in log2 units, sum), sums of weighted values
  float2 *ml;
  float *o;
  int ns, chunk;
};

// A request's entries, held to the bound the workspace was sized for.
__device__ __forceinline__ int list_of(const Decode8 &a, int b, int *beg) {
  *beg = a.indptr[b];
  return min(max(a.indptr[b + 1] - *beg, 0), a.max_kv);
}
// pool row of entry j; an index outside the pool reads its first row
__device__ __forceinline__ int64_t slot_of(const Decode8 &a, int beg, int j) {
  const int s = __ldg(a.indices + (int64_t)beg + j);
  return (unsigned)s < (unsigned)a.pool.S ? s : 0;
}

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 x) {
  return __bfloat162float(x);
}

// The step's row of head g in 8 bits, by one warp: two values a lane.  Called
// by the CTA that reads the request's last entry, before it reads.
template <typename T>
__device__ __forceinline__ void append_row(const Decode8 &a, int b, int g, bool value) {
  const int lane = threadIdx.x & 31, at = a.new_slot[b];
  if ((unsigned)at >= (unsigned)a.pool.S) return;
  const T *src = (const T *)(value ? a.v_new : a.k_new) + ((int64_t)b * a.Hkv + g) * kD + 2 * lane;
  float x[4] = {to_float<T>(src[0]), to_float<T>(src[1]), 0.f, 0.f};
  const uint32_t top = __reduce_max_sync(0xffffffffu, max(kv8_size(x[0]), kv8_size(x[1])));
  const uint32_t scale = kv8_scale(top);
  const int64_t to = (int64_t)at * a.Hkv + g;
  reinterpret_cast<uint16_t *>((value ? a.pool.v : a.pool.k) + to * kD)[lane] =
      (uint16_t)kv8_codes(x, kv8_inverse(scale));
  if (lane == 0) (value ? a.pool.v_scale : a.pool.k_scale)[to] = (uint8_t)scale;
}

// ---------------------------------------------------------------------------
// CUDA cores: CTA = key split x KV head (up to 16 of its query heads) x request,
// 128 entries at a time: a thread rotates one key in fp32 registers and takes
// its products with the query heads; a warp per head forms the weights; a thread
// per (dimension, every second head) sums the values from shared memory.
// ---------------------------------------------------------------------------
constexpr int kSThreads = 128, kSKeys = 128, kSHeads = 16;
struct SimtSmem {
  float q[kSHeads][kD];
  float p[kSHeads][kSKeys];
  float v[kSKeys][kD];
  float alpha[kSHeads];
  ThetaSmem ts;
};

template <typename T>
__global__ void __launch_bounds__(kSThreads)
    decode8_simt_kernel(const Decode8 a, const __grid_constant__ RopeTheta th) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SimtSmem &sm = *reinterpret_cast<SimtSmem *>(smem_raw);
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const int blocks = (a.grp + kSHeads - 1) / kSHeads;
  const int split = blockIdx.x, g = blockIdx.y / blocks, hb = blockIdx.y % blocks, b = blockIdx.z;
  const int h0 = g * a.grp + hb * kSHeads, heads = min(kSHeads, a.grp - hb * kSHeads);
  int beg;
  const int n = list_of(a, b, &beg);
  const int c0 = split * a.chunk, c1 = min(n, c0 + a.chunk);
  if (c0 >= n) return;  // the merge reads only splits that hold entries
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  stage_theta(th, sm.ts);
  // every head block writes the same bytes
  if (a.new_slot && c1 == n && warp < 2) append_row<T>(a, b, g, warp == 1);
  __syncthreads();
  for (int x = threadIdx.x; x < heads * (kD / 2); x += kSThreads) {
    const int h = x / (kD / 2), f = x % (kD / 2);
    float c, s;
    rope_cs(th, sm.ts, f, a.qpos[b], &c, &s);
    const T *row = (const T *)a.q + ((int64_t)b * a.Hq + h0 + h) * kD;
    const float x1 = to_float<T>(row[f]), x2 = to_float<T>(row[f + kD / 2]);
    sm.q[h][f] = x1 * c - x2 * s;
    sm.q[h][f + kD / 2] = x1 * s + x2 * c;
  }
  // each warp owns heads warp, warp + 4, ...; a thread dimension t % 64 of heads
  // t / 64, t / 64 + 2, ...
  float m[kSHeads / 4], l[kSHeads / 4], o[kSHeads / 2];
#pragma unroll
  for (int x = 0; x < kSHeads / 4; ++x) {
    m[x] = -INFINITY;
    l[x] = 0.f;
  }
#pragma unroll
  for (int x = 0; x < kSHeads / 2; ++x) o[x] = 0.f;
  const int d = threadIdx.x % kD, odd = threadIdx.x / kD;
  for (int j0 = c0; j0 < c1; j0 += kSKeys) {
    const int j = j0 + threadIdx.x;
    const bool have = j < c1;
    __syncthreads();  // the last step's readers are done
    if (have) {
      const int64_t row = slot_of(a, beg, j) * a.Hkv + g;
      const uint4 *kr = reinterpret_cast<const uint4 *>(a.pool.k + row * kD);
      const uint4 *vr = reinterpret_cast<const uint4 *>(a.pool.v + row * kD);
      const float kp = kv8_power(a.pool.k_scale[row]), vp = kv8_power(a.pool.v_scale[row]);
      const int pos = __ldg(a.kvpos + (int64_t)beg + j);
      float x[kD];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint4 w = kr[c];
        kv8_floats(w.x, kp, x + 16 * c);
        kv8_floats(w.y, kp, x + 16 * c + 4);
        kv8_floats(w.z, kp, x + 16 * c + 8);
        kv8_floats(w.w, kp, x + 16 * c + 12);
      }
#pragma unroll
      for (int f = 0; f < kD / 2; ++f) {
        float c, s;
        rope_cs(th, sm.ts, f, pos, &c, &s);
        const float x1 = x[f], x2 = x[f + kD / 2];
        x[f] = x1 * c - x2 * s;
        x[f + kD / 2] = x1 * s + x2 * c;
      }
      for (int h = 0; h < heads; ++h) {
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int e = 0; e < kD; e += 4) {
          const float4 u = *reinterpret_cast<const float4 *>(&sm.q[h][e]);
          s[0] = fmaf(u.x, x[e], s[0]);
          s[1] = fmaf(u.y, x[e + 1], s[1]);
          s[2] = fmaf(u.z, x[e + 2], s[2]);
          s[3] = fmaf(u.w, x[e + 3], s[3]);
        }
        sm.p[h][threadIdx.x] = (s[0] + s[1]) + (s[2] + s[3]);
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint4 w = vr[c];
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float y[4];
          kv8_floats(ww[e], vp, y);
          // 16-byte columns turned by the row, so that a warp's rows fall in
          // different banks
          *reinterpret_cast<float4 *>(&sm.v[threadIdx.x][((4 * c + e + threadIdx.x) % 16) * 4]) =
              make_float4(y[0], y[1], y[2], y[3]);
        }
      }
    } else {
      for (int h = 0; h < heads; ++h) sm.p[h][threadIdx.x] = -INFINITY;
#pragma unroll
      for (int e = 0; e < kD / 4; ++e)
        *reinterpret_cast<float4 *>(&sm.v[threadIdx.x][4 * e]) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kSHeads / 4; ++x) {
      const int h = warp + 4 * x;
      if (h >= heads) break;
      float s[4], mx = m[x];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[e] = sm.p[h][lane + 32 * e];
        mx = fmaxf(mx, s[e]);
      }
#pragma unroll
      for (int y = 16; y; y >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, y));
      const float ref = mx == -INFINITY ? 0.f : mx, alpha = exp2f((m[x] - ref) * kScale);
      m[x] = mx;
      l[x] *= alpha;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // the difference is taken before the scale: its rounding is relative to
        // the distance from the maximum
        const float w = exp2f((s[e] - ref) * kScale);
        l[x] += w;
        sm.p[h][lane + 32 * e] = w;
      }
      if (lane == 0) sm.alpha[h] = alpha;
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kSHeads / 2; ++x)
      if (odd + 2 * x < heads) o[x] *= sm.alpha[odd + 2 * x];
#pragma unroll 4
    for (int y = 0; y < kSKeys; ++y) {
      const float v = sm.v[y][((d / 4 + y) % 16) * 4 + d % 4];
#pragma unroll
      for (int x = 0; x < kSHeads / 2; ++x)
        if (odd + 2 * x < heads) o[x] = fmaf(sm.p[odd + 2 * x][y], v, o[x]);
    }
  }
#pragma unroll
  for (int x = 0; x < kSHeads / 2; ++x)
    if (odd + 2 * x < heads)
      a.o[(((int64_t)b * a.Hq + h0 + odd + 2 * x) * a.ns + split) * kD + d] = o[x];
#pragma unroll
  for (int x = 0; x < kSHeads / 4; ++x) {
    float s = l[x];
#pragma unroll
    for (int y = 16; y; y >>= 1) s += __shfl_xor_sync(0xffffffffu, s, y);
    if (lane == 0 && warp + 4 * x < heads)
      a.ml[((int64_t)b * a.Hq + h0 + warp + 4 * x) * a.ns + split] = make_float2(m[x] * kScale, s);
  }
}

// Joins the splits by their log-sum-exp: CTA = (query head, request), eight
// groups of 16 threads each summing every eighth split's row.  Launched as a
// programmatic dependent of the attention kernel.  A request without entries
// gets zeros.
constexpr int kMergeThreads = 128, kMaxSplit = 1024;
template <typename T>
__global__ void __launch_bounds__(kMergeThreads) decode8_merge_kernel(const Decode8 a, T *out) {
  __shared__ float wgt[kMaxSplit];
  __shared__ float4 red[8][kD / 4];
  __shared__ float tot[4], top[4];
  const int h = blockIdx.x, b = blockIdx.y;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int beg;
  const int n = list_of(a, b, &beg);
  const int used = (n + a.chunk - 1) / a.chunk;
  const int64_t w = (int64_t)b * a.Hq + h;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const float2 *ml = a.ml + w * a.ns;
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
    const float4 v = __ldcg(reinterpret_cast<const float4 *>(a.o + (w * a.ns + s) * kD) + cg);
    const float f = wgt[s];
    acc.x = fmaf(v.x, f, acc.x);
    acc.y = fmaf(v.y, f, acc.y);
    acc.z = fmaf(v.z, f, acc.z);
    acc.w = fmaf(v.w, f, acc.w);
  }
  red[sg][cg] = acc;
  __syncthreads();
  if (threadIdx.x < kD) {
    const int col = threadIdx.x;
    float x = 0.f;
#pragma unroll
    for (int y = 0; y < 8; ++y) x += reinterpret_cast<const float *>(&red[y][col >> 2])[col & 3];
    x = used > 0 ? x / L : 0.f;
    T *to = out + w * kD + col;
    if constexpr (sizeof(T) == 4) *to = x;
    else *to = __float2bfloat16_rn(x);
  }
}

int sm_count() {
  int dev = 0, sms = 152;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

// Key splits from the host's bounds alone, so that a captured call replays for
// any lengths within them.
struct Decode8Plan {
  int ns, chunk;
};
Decode8Plan plan_of(int B, int Hq, int Hkv, int max_kv) {
  const int grp = Hq / Hkv;
  const int64_t ctas = (int64_t)B * Hkv * ((grp + kSHeads - 1) / kSHeads);
  const int64_t want = 4LL * 4 * sm_count();
  int c = 4096;
  const auto splits = [&](int x) { return std::max<int64_t>(1, ((int64_t)max_kv + x - 1) / x); };
  while (c > kSKeys && ctas * splits(c) < want) c /= 2;
  while (splits(c) > kMaxSplit) c *= 2;
  return {(int)splits(c), c};
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

template <typename T>
cudaError_t launch(Decode8 &a, void *out, const RopeTheta &th, cudaStream_t s) {
  const int smem = (int)sizeof(SimtSmem);
  cudaError_t e = cudaFuncSetAttribute(decode8_simt_kernel<T>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int blocks = (a.grp + kSHeads - 1) / kSHeads;
  decode8_simt_kernel<T><<<dim3(a.ns, a.Hkv * blocks, a.B), kSThreads, smem, s>>>(a, th);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.Hq, a.B);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode8_merge_kernel<T>, a, (T *)out);
}

}  // namespace

size_t decode_q8_workspace_bytes(int dtype, int B, int Hq, int Hkv, int max_kv) {
  (void)dtype;
  const Decode8Plan p = plan_of(B, Hq, Hkv, max_kv);
  const size_t parts = (size_t)B * Hq * p.ns;
  return up256(parts * sizeof(float2)) + up256(parts * kD * sizeof(float));
}

cudaError_t launch_decode_q8(int dtype, int B, int Hq, int Hkv, const void *q, const int32_t *qpos,
                             const void *k_new, const void *v_new, const int32_t *new_slot,
                             const Kv8Pool &pool, const int32_t *indptr, const int32_t *indices,
                             const int32_t *kvpos, int max_kv, void *out, void *ws,
                             const RopeTheta &th, cudaStream_t s) {
  const Decode8Plan p = plan_of(B, Hq, Hkv, max_kv);
  Decode8 a{B,      Hq,      Hkv,   Hq / Hkv, q,      qpos, k_new, v_new, new_slot, pool,
            indptr, indices, kvpos, max_kv,   (float2 *)ws,
            (float *)((char *)ws + up256((size_t)B * Hq * p.ns * sizeof(float2))), p.ns, p.chunk};
  return dtype == AKV_BF16 ? launch<__nv_bfloat16>(a, out, th, s) : launch<float>(a, out, th, s);
}

}  // namespace akv
