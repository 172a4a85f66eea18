// Rows of a chunk of new tokens made ready for the pool in one pass: per-head
// RMSNorm of queries and keys, rotation at the token's position, and the
// append of key and value (paper review page section 3.3, append) --
//   y = x * rsqrt(mean(x^2) + eps) * w,   z = R(pos) y,
//   q_out = z_q,  k_pool[slot] = z_k,  v_pool[slot] = v,
// norm and rotation each optional for q and k.  All arithmetic is fp32 and
// every output is rounded once.  (Rows whose squares leave fp32's range could be
// scaled first; any test for them between the unrolled rows' sums cost every
// call 4 %: 60.3 -> 62.7 us for 16,384 tokens of 64 / 8 heads.)
//
// Bound by HBM: each row is read once and written once.  A head row of 64
// takes kLanes lanes, each holding the 16-byte chunks c and c + kLanes, which
// are the two halves of its rotation pairs, so the norm is log2(kLanes)
// shuffles and the rotation needs no exchange.  A warp walks head rows of one
// token, so lane f forms the angle of frequency f once per token and the
// lanes fetch theirs by shuffle; passes go two at a time, the next two's
// loads issued before a pair is computed.  Few tokens: a token's passes are spread over `parts`
// warps, which only repeat the one angle per lane.
#include "common.cuh"

#include <algorithm>

namespace akv {
namespace {

constexpr int kNormWarps = 8;
constexpr int kPair = 2;

template <typename T>
struct RowArgs {
  const T *q, *k, *v;
  int64_t qs, ks, vs;  // elements between tokens
  const float *qw, *kw;
  float eps;
  int flags;
  const int32_t *pos, *slot;
  int S;
  T *q_out, *kp, *vp;
  int n, Hq, Hkv;
  int parts;
};

template <typename T>
__global__ void __launch_bounds__(kNormWarps * 32, 3)
    qk_norm_append_kernel(const RowArgs<T> a, const __grid_constant__ RopeTheta th) {
  constexpr int E = Chunk<T>::kElems;
  constexpr int kLanes = (kD / 2) / E;  // lanes per head row: 4 (bf16), 8 (fp32)
  constexpr int kRows = 32 / kLanes;    // head rows per pass of a warp
  __shared__ ThetaSmem ts;
  __shared__ __align__(16) float wt[2][kD];
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * kNormWarps + (threadIdx.x >> 5);
  const int64_t i = w / a.parts;
  const int part = (int)(w % a.parts);
  stage_theta(th, ts);
  if (threadIdx.x < 2 * kD) {
    const float *src = threadIdx.x < kD ? a.qw : a.kw;
    wt[threadIdx.x / kD][threadIdx.x % kD] = src ? __ldg(src + threadIdx.x % kD) : 1.f;
  }
  const int slot = i < a.n ? a.slot[i] : -1;
  __syncthreads();
  if ((unsigned)slot >= (unsigned)a.S) return;  // padding: nothing read or written
  const int pos = (a.flags & (AKV_ROPE_Q | AKV_ROPE_K)) ? a.pos[i] : 0;
  const int c = lane % kLanes, r = lane / kLanes;
  // passes: the q rows, then the k rows, then the v rows of the token
  const int pq = (a.Hq + kRows - 1) / kRows, pk = (a.Hkv + kRows - 1) / kRows;
  const int total = pq + 2 * pk, per = (total + a.parts - 1) / a.parts;
  const int p0 = part * per, p1 = min(total, p0 + per);
  if (p0 >= p1) return;

  auto source = [&](int p) -> const uint4 * {  // this lane's row of pass p, or NULL
    if (p < pq) {
      const int h = p * kRows + r;
      return h < a.Hq ? reinterpret_cast<const uint4 *>(a.q + i * a.qs + (int64_t)h * kD) : nullptr;
    }
    const int h = (p - pq - (p < pq + pk ? 0 : pk)) * kRows + r;
    if (h >= a.Hkv) return nullptr;
    const T *b = p < pq + pk ? a.k + i * a.ks : a.v + i * a.vs;
    return reinterpret_cast<const uint4 *>(b + (int64_t)h * kD);
  };
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  uint4 x[kPair][2];
  auto fetch = [&](int p) {
#pragma unroll
    for (int u = 0; u < kPair; ++u) {
      x[u][0] = x[u][1] = zero;
      const uint4 *s = p + u < p1 ? source(p + u) : nullptr;
      if (s) {
        x[u][0] = s[c];
        x[u][1] = s[c + kLanes];
      }
    }
  };
  fetch(p0);
  // cos/sin of this lane's frequencies c * E .. c * E + E - 1
  float co[E], si[E];
  {
    float cf, sf;
    rope_cs(th, ts, lane, pos, &cf, &sf);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      co[e] = __shfl_sync(0xffffffffu, cf, c * E + e);
      si[e] = __shfl_sync(0xffffffffu, sf, c * E + e);
    }
  }
  for (int pp = p0; pp < p1; pp += kPair) {
    uint4 y[kPair][2];
#pragma unroll
    for (int u = 0; u < kPair; ++u) {
      y[u][0] = x[u][0];
      y[u][1] = x[u][1];
    }
    if (pp + kPair < p1) fetch(pp + kPair);
#pragma unroll
    for (int u = 0; u < kPair; ++u) {
      const int p = pp + u;
      if (p >= p1) break;
      const uint4 y0 = y[u][0], y1 = y[u][1];
      const int kind = p < pq ? 0 : p < pq + pk ? 1 : 2;
      const int h = (kind == 0 ? p : p - pq - (kind == 1 ? 0 : pk)) * kRows + r;
      uint4 z0 = y0, z1 = y1;
      if (kind < 2) {
        const bool norm = a.flags & (kind ? AKV_NORM_K : AKV_NORM_Q);
        const bool rope = a.flags & (kind ? AKV_ROPE_K : AKV_ROPE_Q);
        float f0[E], f1[E];
        chunk_to_f32<T>(y0, f0);
        chunk_to_f32<T>(y1, f1);
        if (norm) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < E; ++e) ss = fmaf(f0[e], f0[e], fmaf(f1[e], f1[e], ss));
#pragma unroll
          for (int o = kLanes / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float inv = rsqrtf(ss * (1.f / kD) + a.eps);
#pragma unroll
          for (int e = 0; e < E; ++e) {
            f0[e] = f0[e] * inv * wt[kind][c * E + e];
            f1[e] = f1[e] * inv * wt[kind][kD / 2 + c * E + e];
          }
        }
        if (rope) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float u = f0[e], v = f1[e];
            f0[e] = u * co[e] - v * si[e];
            f1[e] = u * si[e] + v * co[e];
          }
        }
        if (norm || rope) {
          z0 = f32_to_chunk<T>(f0);
          z1 = f32_to_chunk<T>(f1);
        }
      }
      if (h < (kind ? a.Hkv : a.Hq)) {
        T *dst = kind == 0   ? a.q_out + (i * a.Hq + h) * kD
                 : kind == 1 ? a.kp + ((int64_t)slot * a.Hkv + h) * kD
                             : a.vp + ((int64_t)slot * a.Hkv + h) * kD;
        reinterpret_cast<uint4 *>(dst)[c] = z0;
        reinterpret_cast<uint4 *>(dst)[c + kLanes] = z1;
      }
    }
  }
}

template <typename T>
cudaError_t launch(int Hq, int Hkv, int n, const void *q, int64_t qs, const void *k, int64_t ks,
                   const void *v, int64_t vs, const float *qw, const float *kw, float eps,
                   int flags, const int32_t *pos, const int32_t *slot, int S, void *q_out,
                   void *kp, void *vp, const RopeTheta &th, cudaStream_t s) {
  RowArgs<T> a{(const T *)q, (const T *)k, (const T *)v, qs, ks, vs, qw, kw, eps, flags,
               pos, slot, S, (T *)q_out, (T *)kp, (T *)vp, n, Hq, Hkv, 1};
  int dev = 0, sms = 152;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  // warps per token: about 16 warps per SM, at most one pass each
  constexpr int kRows = 32 / ((kD / 2) / Chunk<T>::kElems);
  const int total = (Hq + kRows - 1) / kRows + 2 * ((Hkv + kRows - 1) / kRows);
  a.parts = (int)std::min<int64_t>(total, std::max<int64_t>(1, (int64_t)sms * 16 / n));
  const int64_t warps = (int64_t)n * a.parts;
  qk_norm_append_kernel<T><<<(unsigned)((warps + kNormWarps - 1) / kNormWarps), kNormWarps * 32, 0,
                             s>>>(a, th);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_append(int dtype, int Hq, int Hkv, int n, const void *q, int64_t qs,
                                  const void *k, int64_t ks, const void *v, int64_t vs,
                                  const float *qw, const float *kw, float eps, int flags,
                                  const int32_t *pos, const int32_t *slot, int S, void *q_out,
                                  void *kp, void *vp, const RopeTheta &th, cudaStream_t s) {
  if (n == 0) return cudaSuccess;
  return dtype == AKV_BF16
             ? launch<__nv_bfloat16>(Hq, Hkv, n, q, qs, k, ks, v, vs, qw, kw, eps, flags, pos, slot,
                                     S, q_out, kp, vp, th, s)
             : launch<float>(Hq, Hkv, n, q, qs, k, ks, v, vs, qw, kw, eps, flags, pos, slot, S,
                             q_out, kp, vp, th, s);
}

}  // namespace akv
