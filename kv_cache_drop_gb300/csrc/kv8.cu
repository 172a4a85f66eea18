// Rows of an 8-bit cache written and read back (paper review page section 3.3:
// append stores a token's key and value; a repos turns a stored key to another
// position).  Keys are kept before RoPE, so that a repos only rewrites positions:
// a key that was stored rotated would be rounded to 8 bits again at every turn.
#include "kv8.cuh"

namespace akv {
namespace {

constexpr int kThreads = 256;
constexpr int kLanes = 4;             // lanes per head row
constexpr int kEach = kD / kLanes;    // values per lane

// Bound by HBM: a row is read once (128 or 256 bytes) and written once (64 and
// a byte).  Four lanes take a head row, 16 values each: the maximum is two
// shuffles and a lane's codes are one 16-byte store.  16,384 tokens of 8 heads,
// bf16: 11.2 us on the device, 4.5 TB/s, 14 to 20 for the call by the host; a few
// tokens: the host's call, 8.6.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    kv8_append_kernel(int rows, int Hkv, const T *__restrict__ k, int64_t ks,
                      const T *__restrict__ v, int64_t vs, const int32_t *__restrict__ slot,
                      const Kv8Pool pool) {
  constexpr int E = Chunk<T>::kElems;
  const uint32_t r = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;  // may pass 2^31 - 1
  const int c = threadIdx.x % kLanes;
  const bool value = blockIdx.y != 0;
  const int i = (int)(r / (uint32_t)Hkv), h = (int)(r - (uint32_t)i * (uint32_t)Hkv);
  const int at = r < (uint32_t)rows ? __ldg(slot + i) : -1;
  const bool real = (unsigned)at < (unsigned)pool.S;  // else padding: nothing read or written
  const uint4 *src = reinterpret_cast<const uint4 *>(
      (value ? v + (int64_t)i * vs : k + (int64_t)i * ks) + (int64_t)h * kD + c * kEach);
  float x[kEach];
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < kEach / E; ++j)
    chunk_to_f32<T>(real ? __ldg(src + j) : make_uint4(0u, 0u, 0u, 0u), x + j * E);
#pragma unroll
  for (int e = 0; e < kEach; ++e) top = max(top, kv8_size(x[e]));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  if (!real) return;
  const uint32_t scale = kv8_scale(top);
  const float inv = kv8_inverse(scale);
  const int64_t to = (int64_t)at * Hkv + h;
  reinterpret_cast<uint4 *>((value ? pool.v : pool.k) + to * kD)[c] =
      make_uint4(kv8_codes(x, inv), kv8_codes(x + 4, inv), kv8_codes(x + 8, inv),
                 kv8_codes(x + 12, inv));
  if (c == 0) (value ? pool.v_scale : pool.k_scale)[to] = (uint8_t)scale;
}

// A warp per entry: its 2 Hkv head rows, four at a time, kFlight such passes in
// flight (few registers, so that many warps are there too); lane f forms the angle of
// frequency f once and the lanes fetch theirs by shuffle.  Eight lanes take a head row:
// lane c holds values 4 c .. 4 c + 3 and the 32 + of these, the two sides of its
// rotation pairs.  26,081 entries of 8 heads to bf16, rotated: 22 us on the device, 3.7
// TB/s (26.6 us the call with one pass at a time and sincosf, 22.6 now).  24 or 40 warps
// per SM take the same time: the memory pipes are 65 % busy with 4-byte loads and
// 8-byte stores, 449 instructions an entry, and DRAM is not what bounds it.
constexpr int kReadLanes = 8, kReadRows = 32 / kReadLanes, kFlight = 4;
__device__ __forceinline__ void store4(float *to, const float *y) {
  *reinterpret_cast<float4 *>(to) = make_float4(y[0], y[1], y[2], y[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16 *to, const float *y) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(y[0], y[1]), b = __floats2bfloat162_rn(y[2], y[3]);
  *reinterpret_cast<uint2 *>(to) = make_uint2(*reinterpret_cast<const uint32_t *>(&a),
                                              *reinterpret_cast<const uint32_t *>(&b));
}
template <typename T>
__global__ void __launch_bounds__(kThreads, 5)
    kv8_read_kernel(int n, int Hkv, const int32_t *__restrict__ src,
                    const int32_t *__restrict__ pos, const int32_t *__restrict__ dst, int R,
                    const Kv8Pool pool, T *k_out, T *v_out, const __grid_constant__ Turns turns) {
  const int lane = threadIdx.x & 31, c = lane % kReadLanes, r = lane / kReadLanes;
  const int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (i >= n) return;
  const int from = __ldg(src + i), to = dst ? __ldg(dst + i) : (int)i;
  const int p = pos ? __ldg(pos + i) : 0;
  if ((unsigned)from >= (unsigned)pool.S || (unsigned)to >= (unsigned)R) return;
  const int64_t row0 = (int64_t)from * Hkv;
  T *const k_to = k_out + (int64_t)to * Hkv * kD, *const v_to = v_out + (int64_t)to * Hkv * kD;
  uint32_t w[kFlight][2], power[kFlight];
  auto fetch = [&](int x, int u) {
    if (x >= 2 * Hkv) return;
    const bool value = x >= Hkv;
    const int64_t at = row0 + (value ? x - Hkv : x);
    const uint32_t *row = reinterpret_cast<const uint32_t *>((value ? pool.v : pool.k) + at * kD);
    w[u][0] = __ldg(row + c);
    w[u][1] = __ldg(row + c + kReadLanes);
    power[u] = __ldg((value ? pool.v_scale : pool.k_scale) + at);
  };
#pragma unroll
  for (int u = 0; u < kFlight; ++u) fetch(r + u * kReadRows, u);
  float co[4], si[4];
  if (pos) {
    float cf, sf;
    turn_cs(turns.hi[lane], turns.lo[lane], p, &cf, &sf);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      co[e] = __shfl_sync(0xffffffffu, cf, 4 * c + e);
      si[e] = __shfl_sync(0xffffffffu, sf, 4 * c + e);
    }
  }
  for (int x0 = r; x0 < 2 * Hkv; x0 += kFlight * kReadRows) {
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int x = x0 + u * kReadRows;
      if (x >= 2 * Hkv) break;
      const bool value = x >= Hkv;
      const float f = kv8_power(power[u]);
      float y0[4], y1[4];
      kv8_floats(w[u][0], f, y0);
      kv8_floats(w[u][1], f, y1);
      fetch(x + kFlight * kReadRows, u);
      if (pos && !value) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float y = y0[e], z = y1[e];
          y0[e] = y * co[e] - z * si[e];
          y1[e] = y * si[e] + z * co[e];
        }
      }
      T *const out = (value ? v_to + (x - Hkv) * kD : k_to + x * kD) + 4 * c;
      store4(out, y0);
      store4(out + kD / 2, y1);
    }
  }
}

template <typename T>
cudaError_t append(int Hkv, int n, const void *k, int64_t ks, const void *v, int64_t vs,
                   const int32_t *slot, const Kv8Pool &pool, cudaStream_t s) {
  const int rows = n * Hkv, per = kThreads / kLanes;
  kv8_append_kernel<T><<<dim3((unsigned)(((int64_t)rows + per - 1) / per), 2), kThreads, 0, s>>>(
      rows, Hkv, (const T *)k, ks, (const T *)v, vs, slot, pool);
  return cudaGetLastError();
}

template <typename T>
cudaError_t read(int Hkv, int n, const int32_t *src, const int32_t *pos, const int32_t *dst, int R,
                 const Kv8Pool &pool, void *k_out, void *v_out, const RopeTheta &th,
                 cudaStream_t s) {
  const int per = kThreads / 32;
  kv8_read_kernel<T><<<(unsigned)(((int64_t)n + per - 1) / per), kThreads, 0, s>>>(
      n, Hkv, src, pos, dst, R, pool, (T *)k_out, (T *)v_out, turns_of(th));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append_q8(int dtype, int Hkv, int n, const void *k, int64_t ks, const void *v,
                             int64_t vs, const int32_t *slot, const Kv8Pool &pool, cudaStream_t s) {
  return dtype == AKV_BF16 ? append<__nv_bfloat16>(Hkv, n, k, ks, v, vs, slot, pool, s)
                           : append<float>(Hkv, n, k, ks, v, vs, slot, pool, s);
}

cudaError_t launch_read_q8(int dtype, int Hkv, int n, const int32_t *src, const int32_t *pos,
                           const int32_t *dst, int R, const Kv8Pool &pool, void *k_out, void *v_out,
                           const RopeTheta &th, cudaStream_t s) {
  return dtype == AKV_BF16
             ? read<__nv_bfloat16>(Hkv, n, src, pos, dst, R, pool, k_out, v_out, th, s)
             : read<float>(Hkv, n, src, pos, dst, R, pool, k_out, v_out, th, s);
}

}  // namespace akv
