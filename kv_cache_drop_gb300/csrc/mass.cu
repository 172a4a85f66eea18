// Attention mass: how much weight a chunk's rows put on each entry of their
// request's list,
//   out[b][j] = decay * in[b][j] + sum_{i sees j} sum_h exp(q_ih . k_j / 8 - lse_ih),
// the first term for entries older than the chunk (the chunk's own entries
// start at zero).  The weights are recomputed from the log-sum-exp that the
// chunk attention leaves, so neither the scores nor the values are stored or
// read.  A CTA owns some list entries of a request and goes over KV heads and
// rows; every sum is formed in one fixed order, whatever the timing.
#include "chunk.cuh"

#include <algorithm>

namespace akv {
namespace {

struct MassArgs {
  const float *lse;
  float decay;
  const float *in;
  float *out;
  int64_t stride;
};

// Running sum of the items' sums.  One fp32 chain over a long chunk's rows and
// heads (some 10,000 terms) was off by 6e-6 of the mass; with the rounding of
// each addition carried over (Kahan) it is an item's own few roundings.
struct Total {
  float sum = 0.f, lost = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float y = __fadd_rn(x, -lost), t = __fadd_rn(sum, y);
    lost = __fadd_rn(__fadd_rn(t, -sum), -y);
    sum = t;
  }
};

// fp32, CUDA cores: CTA = 64 list entries x a share of the (KV head, 128-row
// tile) items; the next item's rows are copied while one is computed.  Each
// thread sums its four keys over its rows of every item, the 16 threads of a
// key are joined at the end.
struct MassF32Smem {
  float q[2][kFRows][kFPitch], k[kFKeys][kFPitch];
  float lse[2][kFRows];
  float red[16][kFKeys];
};

__global__ void __launch_bounds__(kFThreads, 2)
    mass_f32_kernel(const ChunkBatch a, const MassArgs ma, int parts, float *partial,
                    uint32_t *status) {
  clear_status(status);
  extern __shared__ __align__(16) uint8_t smem_raw[];
  MassF32Smem &sm = *reinterpret_cast<MassF32Smem *>(smem_raw);
  const int part = blockIdx.x % parts, b = blockIdx.y;
  const int j0 = (int)(blockIdx.x / parts) * kFKeys;
  const ChunkReq rq = chunk_req(a, b);
  if (j0 >= rq.n) return;
  const int grp = a.Hq / a.Hkv, rows = rq.m * grp;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  const int old = rq.n - rq.m;
  const int n_tiles = (rows + kFRows - 1) / kFRows;
  // first row tile that sees anything of this block
  const int t0 = min(n_tiles, (int)((int64_t)max(0, j0 - old) * grp / kFRows));
  const int per_head = n_tiles - t0;
  const int64_t items = (int64_t)per_head * a.Hkv;
  const int64_t it0 = items * part / parts;
  const int mine = (int)(items * (part + 1) / parts - it0);
  int g = mine ? (int)(it0 / per_head) : 0, t = mine ? t0 + (int)(it0 % per_head) : 0;
  auto load_rows = [&](int buf, int g, int t) {
    f32_load_q(sm.q[buf], a, rq, g, (int64_t)t * kFRows);
    if (threadIdx.x < kFRows) {
      const int r = t * kFRows + threadIdx.x, i = r / grp;
      if (r < rows)
        cp_async4(ptx::smem_addr(&sm.lse[buf][threadIdx.x]),
                  ma.lse + (int64_t)(rq.q0 + i) * a.Hq + g * grp + (r - i * grp));
    }
  };
  Total sum[4];
  if (mine) load_rows(0, g, t);
  for (int it = 0; it < mine; ++it) {
    const int r0 = t * kFRows, buf = it & 1;
    if (it == 0 || t == t0) {
      int own[kFOwn];
      f32_rows(own, a, rq, j0, rq.n);
      f32_load_kv(sm.k, a.k, a, g, own);
    }
    asm volatile("cp.async.commit_group;\n" ::: "memory");
    if (++t == n_tiles) {
      t = t0;
      ++g;
    }
    if (it + 1 < mine) load_rows(buf ^ 1, g, t);
    asm volatile("cp.async.commit_group;\n" ::: "memory");
    asm volatile("cp.async.wait_group 1;\n" ::: "memory");
    __syncthreads();
    float s[8][4];
    f32_scores(sm.q[buf], sm.k, ty, tx, s);
    const int last = min(rq.n, j0 + kFKeys) - 1;  // sees the fewest rows
    const bool plain = r0 >= (int64_t)max(0, last - old) * grp && r0 + kFRows <= rows;
    float x[4] = {};
    if (plain) {
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        const float v = sm.lse[buf][ty + 16 * p];
        if (v == -INFINITY) continue;  // counts nothing, whatever its scores
#pragma unroll
        for (int q = 0; q < 4; ++q) x[q] += ptx::ex2(fmaf(s[p][q], 0.125f, -v) * kLog2e);
      }
    } else {
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        const int r = r0 + ty + 16 * p;
        const float v = sm.lse[buf][ty + 16 * p];
        const int lim = r < rows && v != -INFINITY ? rq.limit(r / grp) : 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float w = ptx::ex2(fmaf(s[p][q], 0.125f, -v) * kLog2e);
          x[q] += j0 + tx + 16 * q < lim ? w : 0.f;
        }
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) sum[q].add(x[q]);
    __syncthreads();  // readers of this buffer and of K are done
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) sm.red[ty][tx + 16 * q] = sum[q].sum;
  __syncthreads();
  const int j = j0 + threadIdx.x;
  if (threadIdx.x < kFKeys && j < rq.n) {
    float x = 0.f;
#pragma unroll
    for (int y = 0; y < 16; ++y) x += sm.red[y][threadIdx.x];
    if (parts > 1) {
      partial[((int64_t)part * a.B + b) * a.max_kv + j] = x;
      return;
    }
    const int64_t at = (int64_t)b * ma.stride + j;
    if (ma.in && j < old) x = fmaf(ma.decay, ma.in[at], x);
    ma.out[at] = x;
  }
}

// -lse in log2 units, for mma.sync's scores; -inf for a row that counts nothing
__device__ __forceinline__ float log2_reference(float lse) {
  return isinf(lse) ? -INFINITY : -lse * kLog2e;
}

// ---------------------------------------------------------------------------
// bf16, few rows (decode steps): up to 16 kRT packed rows per KV head.  CTA =
// `chunk` list entries of a request and all KV heads, a warp per head (heads
// warp, warp + 8, ..), 16 keys at a time: S = Q K^T in m16n8k16 tiles, the
// weights summed over the rows in registers and shuffles, over the heads in
// shared memory.  Bound by the gather of K from HBM.
// ---------------------------------------------------------------------------
// Entries per CTA, K tiles per warp and CTAs per SM, measured for 14 requests
// of 40,000 entries, 64 / 8 heads: 256 / 3 / 4 102 us, 256 / 4 / 3 105,
// 512 / 3 / 3 114, 128 / 4 / 3 112, 512 / 6 / 2 135, 256 / 6 / 2 142.
constexpr int kMChunk = 256;
constexpr int mass_stages(int rt) { return rt == 1 ? 3 : rt == 2 ? 4 : 6; }
constexpr int mass_ctas(int rt) { return rt == 1 ? 4 : rt == 2 ? 3 : 2; }

template <int kRT>
__global__ void __launch_bounds__(kSHeads * 32, mass_ctas(kRT))
    mass_small_kernel(const ChunkBatch a, const MassArgs ma, int chunk, uint32_t *status) {
  clear_status(status);
  constexpr int kMSt = mass_stages(kRT);
  extern __shared__ __align__(128) uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int gid = lane >> 2, tig = lane & 3;
  const int b = blockIdx.y, c0 = blockIdx.x * chunk;
  const ChunkReq rq = chunk_req(a, b);
  if (c0 >= rq.n) return;
  const int grp = a.Hq / a.Hkv, rows = rq.m * grp;
  const int nk = min(rq.n - c0, chunk), n_tiles = (nk + kSKeys - 1) / kSKeys;
  const uint32_t wsm = ptx::smem_addr(smem_raw) + warp * kMSt * kSTile;
  float *const sums = reinterpret_cast<float *>(smem_raw + warps * kMSt * kSTile);  // [warps][chunk]
  float *const mine = sums + warp * chunk;

  for (int g = warp; g < a.Hkv; g += warps) {
    auto load_slot = [&](int t) {
      const int k = t * kSKeys + lane;
      return lane < kSKeys && k < nk ? (int)chunk_slot(a, rq, c0 + k) : 0;
    };
    const __nv_bfloat16 *kp = (const __nv_bfloat16 *)a.k + g * kD;
    auto issue = [&](int t, int slot) {
      if (t < n_tiles) {
        const uint32_t at = wsm + (t % kMSt) * kSTile;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = (lane >> 3) + 4 * i, ch = lane & 7;
          const int sl = __shfl_sync(0xffffffffu, slot, key);
          cp_async16(at + tile_at(key, ch), kp + (int64_t)sl * a.Hkv * kD + ch * 8,
                     t * kSKeys + key < nk);
        }
      }
      asm volatile("cp.async.commit_group;\n" ::: "memory");
    };
    int slot_nx = load_slot(0);
#pragma unroll
    for (int t = 0; t < kMSt - 1; ++t) {
      const int sl = slot_nx;
      slot_nx = load_slot(t + 1);
      issue(t, sl);
    }
    uint32_t qa[kRT][4][4];
    float nl[kRT][2];  // -lse in log2 units; -inf for a row that counts nothing
    int lim[kRT][2];
#pragma unroll
    for (int rt = 0; rt < kRT; ++rt)
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int r = rt * 16 + gid + 8 * hh;
        const bool ok = r < rows;
        const int64_t row = (int64_t)(rq.q0 + (ok ? r / grp : 0)) * a.Hq + g * grp + (ok ? r % grp : 0);
        const uint32_t *src = reinterpret_cast<const uint32_t *>((const __nv_bfloat16 *)a.q + row * kD);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          qa[rt][ks][hh] = ok ? __ldg(src + ks * 8 + tig) : 0u;
          qa[rt][ks][2 + hh] = ok ? __ldg(src + ks * 8 + tig + 4) : 0u;
        }
        const float v = ok ? __ldg(ma.lse + row) : -INFINITY;
        nl[rt][hh] = log2_reference(v);
        lim[rt][hh] = v == -INFINITY ? INT32_MIN : rq.limit(r / grp) - c0;
      }
    for (int it = 0; it < n_tiles; ++it) {
      const int sl = slot_nx;
      slot_nx = load_slot(it + kMSt);
      issue(it + kMSt - 1, sl);
      asm volatile("cp.async.wait_group %0;\n" ::"n"(kMSt - 1) : "memory");
      __syncwarp();
      const uint32_t kt = wsm + (it % kMSt) * kSTile;
      const int k0 = it * kSKeys;
      uint32_t kb[4][4];
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        const int mi = lane >> 3;
        ldsm4(kt + tile_at((mi >> 1) * 8 + (lane & 7), ks * 2 + (mi & 1)), kb[ks]);
      }
      // column sums: key 8 nb + 2 tig + e1
      float cs[2][2] = {};
#pragma unroll
      for (int rt = 0; rt < kRT; ++rt) {
        float s[2][4] = {};
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          mma16816(s[0], qa[rt][ks], kb[ks][0], kb[ks][1]);
          mma16816(s[1], qa[rt][ks], kb[ks][2], kb[ks][3]);
        }
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
          for (int e1 = 0; e1 < 2; ++e1)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const float p = ptx::ex2(fmaf(s[nb][2 * hh + e1], kScale, nl[rt][hh]));
              cs[nb][e1] += k0 + nb * 8 + 2 * tig + e1 < lim[rt][hh] ? p : 0.f;
            }
      }
#pragma unroll
      for (int nb = 0; nb < 2; ++nb)
#pragma unroll
        for (int e1 = 0; e1 < 2; ++e1)
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) cs[nb][e1] += __shfl_xor_sync(0xffffffffu, cs[nb][e1], o);
      if (gid < 2) {  // lanes of gid 0 and 1 write the two halves
        const int key = k0 + gid * 8 + 2 * tig;
        const float v0 = gid ? cs[1][0] : cs[0][0], v1 = gid ? cs[1][1] : cs[0][1];
        float2 *dst = reinterpret_cast<float2 *>(mine + key);
        if (g == warp) *dst = make_float2(v0, v1);
        else *dst = make_float2(dst->x + v0, dst->y + v1);
      }
      __syncwarp();
    }
    asm volatile("cp.async.wait_group 0;\n" ::: "memory");
    __syncwarp();
  }
  __syncthreads();
  for (int j = threadIdx.x; j < nk; j += blockDim.x) {
    float x = 0.f;
    for (int w = 0; w < min(warps, a.Hkv); ++w) x += sums[w * chunk + j];
    const int64_t at = (int64_t)b * ma.stride + c0 + j;
    if (ma.in && c0 + j < rq.n - rq.m) x = fmaf(ma.decay, ma.in[at], x);
    ma.out[at] = x;
  }
}

// ---------------------------------------------------------------------------
// bf16, more rows: tcgen05, the scores transposed.  CTA = 256 list entries
// (two tiles of 128 keys) x a share of the (KV head, 256-row tile) items:
//   warps 4 i .. 4 i + 3  every other 128-row half of the items: thread = TMEM
//        lane = one key of each key tile, so that the sums over rows stay in
//        the thread's registers
//   3 producer warps      K tiles (once per head), Q tiles and the rows' lse
//        through a ring, by cp.async into the 128-byte-swizzled layout
//   MMA warp              S^T = K Q^T - 8 lse, both operands from shared memory,
//        two 128 x 128 tiles per half, into the TMEM buffer of its warps
// The log-sum-exp is a fifth K step (keys: ones; rows: -8 lse in three bf16
// pieces) between the second and the third.  The tensor core truncates every
// step's sum.  Summed to the end, a score came out smaller by 4.4e-8 of itself,
// and with it the weights (error against 64 bits 8.1e-7 for 2 x 700-900 rows over
// 10k-14k entries); now the two sums before the step are cut towards one side,
// the two after it, of the other sign, towards the other, none is larger than
// half the score, and the last is near 0: 1.1e-7, as plain fp32 arithmetic.  The
// step's MMA costs less than the rows' references did in the weights' loop
// (1,629 -> 1,553 us for 2 x 1,100-1,500 rows over 40k-56k entries).
// Scores are taken 16 rows at a time, the next 16 being loaded while a step's
// weights are summed; the buffer is given back with the last load.  Each Q tile
// serves both key tiles: 32 KB from L2 per 65,536 weights.
// The items of an entry block may be shared by several CTAs (`parts`, when
// there are few blocks); their sums are added by mass_join_kernel in one
// fixed order.
// ---------------------------------------------------------------------------
constexpr int kQRows = 2 * kTcRows;
constexpr int kQSt = 4, kKBuf = 2;
constexpr int kMProducers = 3;
constexpr int kMThreads = 256 + 32 * kMProducers + 32;
constexpr int kKSteps = (kTcKeys / 4 + kMProducers - 1) / kMProducers;  // 4-row copy steps, per warp
constexpr int kQSteps = (kQRows / 4 + kMProducers - 1) / kMProducers;
constexpr int kMBlock = 2 * kTcKeys;
constexpr int kMaxParts = 64;
// Items whose copies are under way while the next is issued.  Measured with 2:
// 1,634 us where 1 takes 1,627 (mass of 2 x 1,100-1,500 rows over 40k-56k
// entries), 185 for 173 (14 x 256 rows over 20,000).
constexpr int kInFlight = 1;

struct __align__(1024) MassTcSmem {
  uint8_t k[kKBuf][2][kTcTileBytes];  // [buffer][key tile]
  uint8_t q[kQSt][2 * kTcTileBytes];
  // the K step of the log-sum-exp: the rows' columns 0 .. 7 (with Q's stage), the
  // keys', and columns 8 .. 15 of either
  uint4 lse[kQSt][kQRows], ones[kTcKeys], zeros[kTcKeys];
  uint64_t k_full[kKBuf], k_free[kKBuf], q_full[kQSt], q_free[kQSt];
  uint64_t s_full[2], s_free[2];  // per score buffer
  float join[kMBlock];            // sums of the odd halves
  uint32_t tmem_base;
  uint32_t gave_up;
};

// Columns 0 .. 7 of a row in the K step that takes its log-sum-exp off its scores:
// -8 lse (scores are not divided by 8 yet) as three bf16 values, which hold all 24
// bits.  A row that counts nothing gets -1e30, whose weight is 0.
__device__ __forceinline__ uint4 reference(float lse) {
  const float x = isinf(lse) ? -1e30f : -8.f * lse;
  const float hi = __bfloat162float(__float2bfloat16_rn(x));
  const float rest = isinf(hi) ? 0.f : x - hi;
  const float mid = __bfloat162float(__float2bfloat16_rn(rest));
  return make_uint4(pack2(hi, mid), pack2(rest - mid, 0.f), 0u, 0u);
}

// tokens that v packed rows from a token's first row on reach over; exact for
// v < 512 + grp
struct RowSplit {
  int grp;
  uint32_t inv;  // ceil(2^20 / grp)
  __device__ __forceinline__ explicit RowSplit(int g)
      : grp(g), inv(((1u << 20) + g - 1) / g) {}
  __device__ __forceinline__ int token(int v) const {
    return grp <= 128 ? (int)(((uint32_t)v * inv) >> 20) : (v >= grp) + (v >= 2 * grp);
  }
};

__global__ void __launch_bounds__(kMThreads, 1)
    mass_tc_kernel(const ChunkBatch a, const MassArgs ma, int parts, float *partial,
                   uint32_t *status) {
  extern __shared__ uint8_t smem_raw[];
  MassTcSmem &sm = *reinterpret_cast<MassTcSmem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                   ~uintptr_t(1023));
  clear_status(status);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = blockIdx.x % parts, b = blockIdx.y;
  const int j0 = (int)(blockIdx.x / parts) * kMBlock;
  const ChunkReq rq = chunk_req(a, b);
  if (j0 >= rq.n) return;
  const int grp = a.Hq / a.Hkv, rows = rq.m * grp;
  // row tiles from the first that sees an entry of this block on
  const int old = rq.n - rq.m;  // entries older than the chunk (negative: some rows see nothing)
  const int n_tiles = (rows + kQRows - 1) / kQRows;
  const int t0 = min(n_tiles, (int)((int64_t)max(0, j0 - old) * grp / kQRows));
  const int per_head = n_tiles - t0;
  const int64_t items = (int64_t)per_head * a.Hkv;
  const int64_t it0 = items * part / parts;
  const int mine = (int)(items * (part + 1) / parts - it0);
  const int g0 = mine ? (int)(it0 / per_head) : 0, tile0 = mine ? t0 + (int)(it0 % per_head) : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kKBuf; ++s) {
      ptx::mbar_init(&sm.k_full[s], kMProducers);
      ptx::mbar_init(&sm.k_free[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(&sm.s_full[s], 1);
      ptx::mbar_init(&sm.s_free[s], 4);
    }
    for (int s = 0; s < kQSt; ++s) {
      ptx::mbar_init(&sm.q_full[s], kMProducers);
      ptx::mbar_init(&sm.q_free[s], 1);
    }
    sm.gave_up = 0u;
    ptx::fence_barrier_init();
  }
  if (threadIdx.x < kTcKeys) {
    sm.ones[threadIdx.x] = make_uint4(0x3f803f80u, 0x3f80u, 0u, 0u);  // one per piece of lse
    sm.zeros[threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
    ptx::fence_proxy_async_smem();
  }
  if (warp == 8 + kMProducers) ptx::tmem_alloc(&sm.tmem_base, 512);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    if (!ptx::mbar_wait_grid(bar, parity, &sm.gave_up, 1u, kTcWaitBudget))
      atomicOr(status, kStatusWaitTimeout);
  };

  if (warp >= 8 && warp < 8 + kMProducers) {
    const int ch = lane & 7;
    const int ks0 = (warp - 8) * kKSteps, krow = 4 * ks0 + (lane >> 3);  // this lane's row of step 0
    const int qs0 = (warp - 8) * kQSteps, qrow = 4 * qs0 + (lane >> 3);
    const uint32_t kd = ptx::smem_addr(sm.k[0][0]) + krow * 128;
    const uint32_t qd = ptx::smem_addr(sm.q[0]) + qrow * 128;
    auto swizzle = [&](int row) { return (uint32_t)((ch ^ (row & 7)) << 4); };
    const uint32_t ksw0 = swizzle(krow), ksw1 = swizzle(krow + 4);
    const uint32_t qsw0 = swizzle(qrow), qsw1 = swizzle(qrow + 4);
    const int64_t pitch = (int64_t)a.Hkv * kD * 2;
    const RowSplit sp(grp);
    // Each item is one group of copies; its barrier is arrived on once the
    // group has landed, kInFlight items later.
    uint64_t *pend[kInFlight];
#pragma unroll
    for (int e = 0; e < kInFlight; ++e) pend[e] = nullptr;
    auto landed = [&](uint64_t *next) {  // the oldest pending item, then `next` joins the queue
      asm volatile("cp.async.commit_group;\n" ::: "memory");
      asm volatile("cp.async.wait_group %0;\n" ::"n"(kInFlight) : "memory");
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (pend[0] && lane == 0) ptx::mbar_arrive(pend[0]);
#pragma unroll
      for (int e = 0; e + 1 < kInFlight; ++e) pend[e] = pend[e + 1];
      pend[kInFlight - 1] = next;
    };
    // a buffer's release: before this warp waits for one it tells the MMA
    // warp of everything that has been copied, which it may be waiting for
    auto acquire = [&](uint64_t *bar, uint32_t parity) {
      if (__all_sync(0xffffffffu, ptx::mbar_test(bar, parity))) return;
      asm volatile("cp.async.wait_group 0;\n" ::: "memory");
      ptx::fence_proxy_async_smem();
      __syncwarp();
#pragma unroll
      for (int e = 0; e < kInFlight; ++e) {
        if (pend[e] && lane == 0) ptx::mbar_arrive(pend[e]);
        pend[e] = nullptr;
      }
      wait(bar, parity);
    };
    // pool rows of the block's entries, the same for every head
    int slot[2][kKSteps];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int s = 0; s < kKSteps; ++s) {
        const int j = j0 + i * kTcKeys + krow + 4 * s;
        slot[i][s] = ks0 + s < kTcKeys / 4 && j < rq.n ? (int)chunk_slot(a, rq, j) : -1;
      }
    // lse of rows x = 4 qs0 + lane + 32 u of a tile, loaded an item ahead
    constexpr int kLse = (4 * kQSteps + 31) / 32;
    float lse_nx[kLse];
    auto load_lse = [&](int g, int t) {
      const int r0 = t * kQRows, i0 = r0 / grp, h0 = r0 - i0 * grp;
#pragma unroll
      for (int u = 0; u < kLse; ++u) {
        const int x = 4 * qs0 + lane + 32 * u, v = h0 + x, i = sp.token(v);
        lse_nx[u] = INFINITY;  // no row: a weight of 0 too
        if (lane + 32 * u < 4 * kQSteps && x < kQRows && r0 + x < rows)
          lse_nx[u] = __ldg(ma.lse + (int64_t)(rq.q0 + i0 + i) * a.Hq + g * grp + (v - i * grp));
      }
    };
    // bytes from a tile's first token to this lane's row of each step: the
    // same for every tile that starts at the same head of its group
    int off[kQSteps], h_off = -1;
    int kn = 0, g = g0, t = tile0;
    if (mine) load_lse(g, t);
    for (int qn = 0; qn < mine; ++qn) {
      if (qn == 0 || t == t0) {  // the head's K tiles
        const int kb = kn % kKBuf;
        if (kn >= kKBuf) acquire(&sm.k_free[kb], (kn / kKBuf - 1) & 1);
        const char *kg = (const char *)a.k + (g * kD + ch * 8) * 2;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int s = 0; s < kKSteps; ++s)
            if (ks0 + s < kTcKeys / 4)
              cp_async16(kd + (kb * 2 + i) * kTcTileBytes + s * 512 + (s & 1 ? ksw1 : ksw0),
                         kg + max(slot[i][s], 0) * pitch, slot[i][s] >= 0);
        landed(&sm.k_full[kb]);
        ++kn;
      }
      const int st = qn % kQSt;
      if (qn >= kQSt) acquire(&sm.q_free[st], ((qn / kQSt) - 1) & 1);
      const int r0 = t * kQRows, i0 = r0 / grp, h0 = r0 - i0 * grp;
      if (h0 != h_off) {
        h_off = h0;
#pragma unroll
        for (int s = 0; s < kQSteps; ++s) {
          const int v = h0 + qrow + 4 * s, i = sp.token(v);
          off[s] = (i * a.Hq + (v - i * grp)) * (kD * 2);
        }
      }
      const char *qg = (const char *)a.q + ((int64_t)(rq.q0 + i0) * a.Hq + g * grp) * (kD * 2) + ch * 16;
      const uint32_t to = qd + st * 2 * kTcTileBytes;
      if (r0 + kQRows <= rows) {
#pragma unroll
        for (int s = 0; s < kQSteps; ++s)
          if (qs0 + s < kQRows / 4)
            cp_async16(to + s * 512 + (s & 1 ? qsw1 : qsw0), qg + off[s], true);
      } else {
#pragma unroll
        for (int s = 0; s < kQSteps; ++s)
          if (qs0 + s < kQRows / 4) {
            const bool ok = r0 + qrow + 4 * s < rows;
            cp_async16(to + s * 512 + (s & 1 ? qsw1 : qsw0), qg + (ok ? off[s] : 0), ok);
          }
      }
#pragma unroll
      for (int u = 0; u < kLse; ++u) {
        const int x = 4 * qs0 + lane + 32 * u;
        if (lane + 32 * u < 4 * kQSteps && x < kQRows)
          sm.lse[st][x] = reference(lse_nx[u]);
      }
      // A row that counts nothing may hold anything, and its reference makes a
      // weight of 0 of finite scores only: its copy becomes zeros.  (Telling the
      // warps that form the weights, 1.4 % of the call.)
      static_assert(kLse == 3, "rows per lane");
      const bool none = fminf(fminf(lse_nx[0], lse_nx[1]), lse_nx[2]) == -INFINITY;
      if (__any_sync(0xffffffffu, none)) {
        asm volatile("cp.async.wait_all;\n" ::: "memory");
        __syncwarp();
#pragma unroll 1
        for (int u = 0; u < kLse; ++u) {
          const float v = u == 0 ? lse_nx[0] : u == 1 ? lse_nx[1] : lse_nx[2];
          uint4 *row = reinterpret_cast<uint4 *>(sm.q[st]) + (4 * qs0 + lane + 32 * u) * (kD * 2 / 16);
          for (int c = 0; v == -INFINITY && c < kD * 2 / 16; ++c) row[c] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      landed(&sm.q_full[st]);
      if (++t == n_tiles) {
        t = t0;
        ++g;
      }
      if (qn + 1 < mine) load_lse(g, t);
    }
#pragma unroll
    for (int e = 0; e < kInFlight; ++e) landed(nullptr);
    asm volatile("cp.async.wait_group 0;\n" ::: "memory");
  } else if (warp == 8 + kMProducers) {
    constexpr uint32_t id = ptx::idesc_bf16(128, 128, false);
    constexpr uint64_t kTileStep = kTcTileBytes >> 4;
    const uint64_t dk = ptx::sdesc_sw128(ptx::smem_addr(sm.k[0][0]));
    const uint64_t dq = ptx::sdesc_sw128(ptx::smem_addr(sm.q[0]));
    const uint64_t d_ones =
        ptx::sdesc_plain(ptx::smem_addr(sm.ones), ptx::smem_addr(sm.zeros) - ptx::smem_addr(sm.ones), 128);
    int kn = 0, t = tile0, hseq = 0;
    for (int qn = 0; qn < mine; ++qn) {
      if (qn == 0 || t == t0) {  // the next head
        if (kn > 0 && ptx::elect_one()) ptx::mma_commit(&sm.k_free[(kn - 1) % kKBuf]);
        __syncwarp();
        wait(&sm.k_full[kn % kKBuf], (kn / kKBuf) & 1);
        ++kn;
      }
      const int halves = rows - t * kQRows > kTcRows ? 2 : 1;
      if (++t == n_tiles) t = t0;
      const int st = qn % kQSt;
      wait(&sm.q_full[st], (qn / kQSt) & 1);
      for (int hf = 0; hf < halves; ++hf, ++hseq) {
        const int buf = hseq & 1;
        if (hseq >= 2) wait(&sm.s_free[buf], ((hseq >> 1) - 1) & 1);
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
          const uint64_t ak = dk + ((kn - 1) % kKBuf) * 2 * kTileStep, bq = dq + (st * 2 + hf) * kTileStep;
          const uint32_t at = ptx::smem_addr(sm.lse[st] + hf * kTcRows);
          const uint64_t d_lse = ptx::sdesc_plain(at, ptx::smem_addr(sm.zeros) - at, 128);
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint32_t d = tmem + buf * 256 + i * 128;
              if (kk == 2) ptx::mma_f16_ss(d, d_ones, d_lse, id, 1u);
              ptx::mma_f16_ss(d, ak + i * kTileStep + 2 * kk, bq + 2 * kk, id, kk > 0);
            }
          ptx::mma_commit(&sm.s_full[buf]);
          if (hf + 1 == halves) ptx::mma_commit(&sm.q_free[st]);
        }
        __syncwarp();
      }
    }
  } else {
    const int buf = warp >> 2;
    const int key0 = j0 + (threadIdx.x & 127);  // and key0 + 128
    const uint32_t ts = tmem + ((uint32_t)((warp & 3) * 32) << 16) + buf * 256;
    // packed rows [r_min, rows) see a key (none past the list's end)
    const int64_t r_min0 = key0 < rq.n ? (int64_t)max(0, key0 - old) * grp : INT32_MAX;
    const int64_t r_min1 = key0 + 128 < rq.n ? (int64_t)max(0, key0 + 128 - old) * grp : INT32_MAX;
    // the last listed key of the block sees the fewest rows
    const int64_t all_see = (int64_t)max(0, min(rq.n, j0 + kMBlock) - 1 - old) * grp;
    const float2 scale2 = make_float2(kScale, kScale);
    Total total[2];
    constexpr int kStep = 16;
    int t = tile0, hseq = 0;
    for (int qn = 0; qn < mine; ++qn) {
      const int r_tile = t * kQRows, halves = rows - r_tile > kTcRows ? 2 : 1;
      if (++t == n_tiles) t = t0;
      const int hf = (hseq & 1) == buf ? 0 : 1;  // the half of this item in this buffer
      const int seq = hseq + hf;
      hseq += halves;
      if (hf >= halves) continue;
      const int r0 = r_tile + hf * kTcRows;
      float2 sum[2][2];  // of this half: [key][pair of rows]
#pragma unroll
      for (int e = 0; e < 2; ++e) sum[e][0] = sum[e][1] = make_float2(0.f, 0.f);
      wait(&sm.s_full[buf], (seq >> 1) & 1);
      ptx::tc_fence_after();
      auto give_back = [&] {  // all scores of the half are in registers
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sm.s_free[buf]);
      };
      if (r0 >= all_see && r0 + kTcRows <= rows) {
        uint32_t sr[2][2][kStep];  // [step parity][key]
        ptx::tmem_ld16(ts, sr[0][0]);
        ptx::tmem_ld16(ts + 128, sr[0][1]);
#pragma unroll
        for (int c = 0; c < kTcRows / kStep; ++c) {
          uint32_t(&s)[2][kStep] = sr[c & 1];
          ptx::tmem_wait_ld();
          ptx::reg_fence16(s[0]);
          ptx::reg_fence16(s[1]);
          if (c + 1 < kTcRows / kStep) {
            ptx::tmem_ld16(ts + (c + 1) * kStep, sr[(c + 1) & 1][0]);
            ptx::tmem_ld16(ts + 128 + (c + 1) * kStep, sr[(c + 1) & 1][1]);
          } else {
            give_back();
          }
#pragma unroll
          for (int q = 0; q < kStep / 4; ++q) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int w = 0; w < 2; ++w) {
                const int x = 4 * q + 2 * w;
                const float2 y = __fmul2_rn(
                    make_float2(__uint_as_float(s[e][x]), __uint_as_float(s[e][x + 1])), scale2);
                sum[e][w] = __fadd2_rn(sum[e][w], make_float2(ptx::ex2(y.x), ptx::ex2(y.y)));
              }
          }
        }
      } else {
        // rows [lo, hi) of the half see each key; a few halves per head
        const int lo0 = (int)min((int64_t)kTcRows, max((int64_t)0, r_min0 - r0));
        const int lo1 = (int)min((int64_t)kTcRows, max((int64_t)0, r_min1 - r0));
        const int hi = min(kTcRows, rows - r0);
#pragma unroll 1
        for (int c = 0; c < kTcRows; c += kStep) {
          uint32_t s[2][kStep];
          ptx::tmem_ld16(ts + c, s[0]);
          ptx::tmem_ld16(ts + 128 + c, s[1]);
          ptx::tmem_wait_ld();
          ptx::reg_fence16(s[0]);
          ptx::reg_fence16(s[1]);
          if (c + kStep == kTcRows) give_back();
#pragma unroll
          for (int x = 0; x < kStep; ++x) {
            const float p0 = ptx::ex2(__uint_as_float(s[0][x]) * kScale);
            const float p1 = ptx::ex2(__uint_as_float(s[1][x]) * kScale);
            if (c + x >= lo0 && c + x < hi) sum[0][0].x += p0;
            if (c + x >= lo1 && c + x < hi) sum[1][0].x += p1;
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 x = __fadd2_rn(sum[e][0], sum[e][1]);
        total[e].add(x.x + x.y);
      }
    }
    if (buf == 1) {
      sm.join[threadIdx.x & 127] = total[0].sum;
      sm.join[(threadIdx.x & 127) + 128] = total[1].sum;
    }
    ptx::named_bar_sync(1, 256);
    if (buf == 0) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int key = key0 + 128 * e;
        float x = total[e].sum + sm.join[key - j0];
        if (key >= rq.n) continue;
        if (parts > 1) {
          partial[((int64_t)part * a.B + b) * a.max_kv + key] = x;
        } else {
          const int64_t at = (int64_t)b * ma.stride + key;
          if (ma.in && key < old) x = fmaf(ma.decay, ma.in[at], x);
          ma.out[at] = x;
        }
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 8 + kMProducers) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// Sum of the parts of each entry, in part order, and what it had.
__global__ void __launch_bounds__(256)
    mass_join_kernel(const ChunkBatch a, const MassArgs ma, int parts, const float *partial) {
  const int b = blockIdx.y, j = blockIdx.x * 256 + threadIdx.x;
  const ChunkReq rq = chunk_req(a, b);
  if (j >= rq.n) return;
  float x = 0.f;
#pragma unroll 4
  for (int p = 0; p < parts; ++p) x += partial[((int64_t)p * a.B + b) * a.max_kv + j];
  const int64_t at = (int64_t)b * ma.stride + j;
  if (ma.in && j < rq.n - rq.m) x = fmaf(ma.decay, ma.in[at], x);
  ma.out[at] = x;
}

struct MassPlan {
  int kind;   // 0 CUDA cores; 1, 2, 4: mma.sync with that many 16-row tiles; 3: tcgen05
  int chunk;  // entries per CTA (kinds 1, 2, 4)
  int parts;  // CTAs per entry block (kinds 0, 3)
};

MassPlan mass_plan(int dtype, int B, int Hq, int Hkv, int max_q, int max_kv) {
  MassPlan p{0, 0, 1};
  const int64_t rows = (int64_t)max_q * (Hq / Hkv);
  const int sms = chunk_sms();
  if (dtype == AKV_BF16 && rows <= 64) {
    p.kind = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
    p.chunk = kMChunk;
    while (p.chunk > 64 && (int64_t)B * ((max_kv + p.chunk - 1) / p.chunk) < 2LL * sms) p.chunk /= 2;
    return p;
  }
  const bool tc = dtype == AKV_BF16;
  const int block = tc ? kMBlock : kFKeys, tile = tc ? kQRows : kFRows, resident = tc ? sms : 2 * sms;
  p.kind = tc ? 3 : 0;
  // about four waves of CTAs, the last of them as full as twice the parts can
  // make it; none with less than four items
  const int64_t blocks = std::max<int64_t>(1, (int64_t)B * ((max_kv + block - 1) / block));
  const int64_t items = (rows + tile - 1) / tile * Hkv;
  const int64_t most = std::max<int64_t>(1, std::min<int64_t>(kMaxParts, items / 4));
  const int64_t first = std::min<int64_t>(most, (4LL * resident + blocks - 1) / blocks);
  const auto idle = [&](int64_t n) {  // share of the launch's waves left empty
    const int64_t ctas = blocks * n, waves = (ctas + resident - 1) / resident;
    return (double)(waves * resident - ctas) / (double)(waves * resident);
  };
  p.parts = (int)first;
  for (int64_t n = first + 1; n <= std::min<int64_t>(most, 2 * first); ++n)
    if (idle(n) < idle(p.parts) - 0.02) p.parts = (int)n;
  return p;
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

template <int kRT>
cudaError_t launch_small(const ChunkBatch &a, const MassArgs &ma, int chunk, uint32_t *status,
                         cudaStream_t s) {
  const int warps = std::min(a.Hkv, kSHeads);
  const int smem = warps * (mass_stages(kRT) * kSTile + chunk * (int)sizeof(float));
  cudaError_t e = cudaFuncSetAttribute(mass_small_kernel<kRT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  mass_small_kernel<kRT><<<dim3((unsigned)((a.max_kv + chunk - 1) / chunk), a.B), warps * 32, smem, s>>>(
      a, ma, chunk, status);
  return cudaGetLastError();
}

}  // namespace

size_t mass_workspace_bytes(int dtype, int B, int Hq, int Hkv, int n_rows, int max_q, int max_kv) {
  const MassPlan p = mass_plan(dtype, B, Hq, Hkv, max_q, max_kv);
  return kTcStatusBytes + (p.parts > 1 ? up256((size_t)p.parts * B * max_kv * sizeof(float)) : 0);
}

cudaError_t launch_mass(int dtype, int B, int Hq, int Hkv, int n_rows, int S,
                        const int32_t *q_indptr, int max_q, const void *q, const void *k,
                        const int32_t *kv_indptr, const int32_t *kv_indices, int max_kv,
                        const float *lse, float decay, const float *in, float *out, int64_t stride,
                        void *ws, cudaStream_t s) {
  const ChunkBatch a{B, Hq, Hkv, n_rows, S, max_q, max_kv, q_indptr, kv_indptr, kv_indices, q, k,
                     nullptr};
  const MassArgs ma{lse, decay, in, out, stride};
  const MassPlan p = mass_plan(dtype, B, Hq, Hkv, max_q, max_kv);
  float *const partial = (float *)((char *)ws + kTcStatusBytes);
  cudaError_t e;
  if (p.kind == 1) return launch_small<1>(a, ma, p.chunk, (uint32_t *)ws, s);
  if (p.kind == 2) return launch_small<2>(a, ma, p.chunk, (uint32_t *)ws, s);
  if (p.kind == 4) return launch_small<4>(a, ma, p.chunk, (uint32_t *)ws, s);
  if (p.kind == 0) {
    const int smem = (int)sizeof(MassF32Smem);
    e = cudaFuncSetAttribute(mass_f32_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int64_t blocks = (max_kv + kFKeys - 1) / kFKeys;
    mass_f32_kernel<<<dim3((unsigned)(blocks * p.parts), B), kFThreads, smem, s>>>(a, ma, p.parts, partial,
                                                                                (uint32_t *)ws);
  } else {
    const int smem = (int)sizeof(MassTcSmem) + 1024;
    e = cudaFuncSetAttribute(mass_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int64_t blocks = (max_kv + kMBlock - 1) / kMBlock;
    mass_tc_kernel<<<dim3((unsigned)(blocks * p.parts), B), kMThreads, smem, s>>>(a, ma, p.parts, partial,
                                                                               (uint32_t *)ws);
  }
  e = cudaGetLastError();
  if (e != cudaSuccess || p.parts == 1) return e;
  mass_join_kernel<<<dim3((unsigned)((max_kv + 255) / 256), B), 256, 0, s>>>(a, ma, p.parts, partial);
  return cudaGetLastError();
}

}  // namespace akv
