// Shared by the kernels over a chunk of new tokens and a page-size-1 pool
// (chunk.cu, mass.cu): the batch, a request's view of it, and the 128 x 64
// score tile on the CUDA cores.
//
// Rows.  The query rows of KV head g are packed (token, head of the group):
// packed row r of request b is token i = r / grp of its chunk and query head
// g * grp + r % grp, so that one K/V tile serves every row that reads it.
// Row i of a chunk of m tokens sees the list entries j < n - m + i + 1.
#pragma once

#include "common.cuh"
#include "tc_ptx.cuh"

namespace akv {

struct ChunkBatch {
  int B, Hq, Hkv, n_rows, S, max_q, max_kv;
  const int32_t *q_indptr, *kv_indptr, *kv_indices;
  const void *q, *k, *v;
};

struct ChunkReq {
  int q0, m;    // first row of the chunk in q, its tokens
  int beg, n;   // first list entry, entries
  __device__ __forceinline__ int limit(int i) const {  // entries that token i sees
    return min(n, max(0, n - m + i + 1));
  }
};

// Rows and lengths are held to the bounds the call was given, so that no row
// of q, out or a workspace outside them is touched (kv_indptr itself is
// trusted, as by the decode calls).
__device__ __forceinline__ ChunkReq chunk_req(const ChunkBatch &a, int b) {
  ChunkReq r;
  r.q0 = max(0, a.q_indptr[b]);
  r.m = max(0, min(min(a.q_indptr[b + 1], a.n_rows) - r.q0, a.max_q));
  r.beg = a.kv_indptr[b];
  r.n = min(max(a.kv_indptr[b + 1] - r.beg, 0), a.max_kv);
  return r;
}

// pool row of list entry j; an index outside the pool reads its first row
__device__ __forceinline__ int64_t chunk_slot(const ChunkBatch &a, const ChunkReq &r, int j) {
  const int s = __ldg(a.kv_indices + (int64_t)r.beg + j);
  return (unsigned)s < (unsigned)a.S ? s : 0;
}

// The call's status word starts at 0: written by one thread of every kernel
// that opens a call (a wait that gives up sets its bit half a second later).
__device__ __forceinline__ void clear_status(uint32_t *status) {
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) *status = 0u;
}

// ---- tensor cores: 128 packed rows, key tiles of 128 (the mass; the attention has windows of its own) ----
constexpr int kTcRows = 128;
constexpr int kTcKeys = 128;
constexpr uint32_t kTcTileBytes = kTcKeys * kD * 2;      // one K or V window of a KV head
constexpr long long kTcWaitBudget = 1000000000LL;        // SM clocks (about 0.5 s)
constexpr size_t kTcStatusBytes = 256;                   // status word at the workspace's start

// ---- mma.sync: 16 keys at a time, a warp per KV head ----
constexpr int kSKeys = 16;
constexpr int kSTile = kSKeys * kD * 2;  // bytes of a K (or V) tile
constexpr int kSHeads = 8;               // warps (KV heads) per CTA at most
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kScale = 0.125f * kLog2e;  // scores to log2 units

inline int chunk_sms() {
  int dev = 0, sms = 152;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0));
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t *r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t *r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
// byte offset of (row, 16-byte chunk) in a [16][64] bf16 tile
__device__ __forceinline__ uint32_t tile_at(int row, int chunk) {
  return (uint32_t)(row * 128 + ((chunk ^ (row & 7)) << 4));
}

// A bf16 pair with an infinity or NaN in it.
__device__ __forceinline__ bool nonfinite_lo(uint32_t w) { return (w & 0x7f80u) == 0x7f80u; }
__device__ __forceinline__ bool nonfinite_hi(uint32_t w) {
  return (w & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t w) {
  return (nonfinite_lo(w) ? 0u : w & 0xffffu) | (nonfinite_hi(w) ? 0u : w & 0xffff0000u);
}

// ---- CUDA cores (fp32): 128 packed rows x 64 keys, 256 threads ----
// Thread (ty, tx) = (tid / 16, tid % 16) holds rows ty + 16 p (p < 8) and keys
// tx + 16 q (q < 4).  All tiles are row-major with rows of 272 bytes, so that
// they are copied as they lie in memory (cp.async) and every operand is a
// 16-byte shared load: a warp's two Q rows are broadcast, its 16 K rows fall in
// different banks.  12 loads feed 128 multiply-adds.
constexpr int kFRows = 128;
constexpr int kFKeys = 64;
constexpr int kFPitch = kD + 4;  // floats
constexpr int kFThreads = 256;

// packed rows r0.. of KV head g (rows past the chunk: zeros)
__device__ __forceinline__ void f32_load_q(float (*dst)[kFPitch], const ChunkBatch &a,
                                           const ChunkReq &rq, int g, int64_t r0) {
  const int grp = a.Hq / a.Hkv, c = threadIdx.x % 16;
  const int rows = rq.m * grp;  // 2^30 at most
  for (int x = threadIdx.x / 16; x < kFRows; x += kFThreads / 16) {
    const int r = (int)r0 + x;
    const bool ok = r < rows;
    const int i = ok ? r / grp : 0, h = ok ? r - i * grp : 0;
    cp_async16(ptx::smem_addr(&dst[x][4 * c]),
               (const float *)a.q + ((int64_t)(rq.q0 + i) * a.Hq + g * grp + h) * kD + 4 * c, ok);
  }
}
// Pool rows of this thread's entries from j0 on (-1 from `end` on).  Loaded well
// before the copies that use them: a load returns only after all copies that
// were queued before it.
constexpr int kFOwn = kFKeys / (kFThreads / 16);
__device__ __forceinline__ void f32_rows(int *row, const ChunkBatch &a, const ChunkReq &rq, int j0,
                                         int end) {
#pragma unroll
  for (int e = 0; e < kFOwn; ++e) {
    const int j = j0 + threadIdx.x / 16 + e * (kFThreads / 16);
    row[e] = j < end ? (int)chunk_slot(a, rq, j) : -1;
  }
}
// those rows of a pool, KV head g (zeros for -1)
__device__ __forceinline__ void f32_load_kv(float (*dst)[kFPitch], const void *pool,
                                            const ChunkBatch &a, int g, const int *row) {
  const int c = threadIdx.x % 16, x0 = threadIdx.x / 16;
#pragma unroll
  for (int e = 0; e < kFOwn; ++e)
    cp_async16(ptx::smem_addr(&dst[x0 + e * (kFThreads / 16)][4 * c]),
               (const float *)pool + ((int64_t)max(row[e], 0) * a.Hkv + g) * kD + 4 * c, row[e] >= 0);
}

// acc[p][q] = q row . k row, even and odd dimensions in packed pairs: half the
// instructions, which leaves the issue slots to the loads (mass f32 100 -> 94 us)
__device__ __forceinline__ void f32_scores(const float (*q)[kFPitch], const float (*k)[kFPitch],
                                           int ty, int tx, float (*acc)[4]) {
  float2 s[8][4];
#pragma unroll
  for (int p = 0; p < 8; ++p)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[p][e] = make_float2(0.f, 0.f);
#pragma unroll 2
  for (int d = 0; d < kD; d += 4) {
    float4 w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = *reinterpret_cast<const float4 *>(&k[tx + 16 * e][d]);
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const float4 u = *reinterpret_cast<const float4 *>(&q[ty + 16 * p][d]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[p][e] = __ffma2_rn(make_float2(u.x, u.y), make_float2(w[e].x, w[e].y), s[p][e]);
        s[p][e] = __ffma2_rn(make_float2(u.z, u.w), make_float2(w[e].z, w[e].w), s[p][e]);
      }
    }
  }
#pragma unroll
  for (int p = 0; p < 8; ++p)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[p][e] = s[p][e].x + s[p][e].y;
}

}  // namespace akv
