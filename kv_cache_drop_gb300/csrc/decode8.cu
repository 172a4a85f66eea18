// Decode over the active cache held in 8 bits (paper review page section 4
// serving flow: decode reads only the active cache; section 3.3: a key moves
// between positions by a rotation).  The pool keeps e4m3 keys before RoPE and
// values, with a power of two per head row (kv8.cuh); every list entry carries
// its position, and
//   s_j = R(q_pos) q . R(pos_j) k_j 2^ks_j / 8,  out = sum_j softmax(s)_j v_j 2^vs_j.
#include "kv8.cuh"

#include <algorithm>
#include <type_traits>

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
  // partials: (maximum in log2 units, sum), sums of weighted values; fp32
  // [B][Hq][ctas], bf16 [range + request][sub][Hq]
  float2 *ml;
  float *o;
  int ctas;   // CTAs along a list (fp32), along all lists (bf16)
  int chunk;  // fp32: entries of each
  int sub;    // bf16: groups of warps that share out a CTA's entries
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
// per (dimension, every second head) sums the values from shared memory.  fp32 is
// the library's parity type, and the tensor cores take none.  3 requests of 500 to
// 4,000 entries, 16 / 4 heads: 17 us on the device, 20.5 for the call (37 with
// sincosf for the angles), bound by the chain within a CTA of one tile.
// ---------------------------------------------------------------------------
constexpr int kSThreads = 128, kSKeys = 128, kSHeads = 16;
struct SimtSmem {
  float q[kSHeads][kD];
  float p[kSHeads][kSKeys];
  float v[kSKeys][kD];
  float alpha[kSHeads];
  int turn_hi[kD / 2], turn_lo[kD / 2];
};

template <typename T>
__global__ void __launch_bounds__(kSThreads)
    decode8_simt_kernel(const Decode8 a, const __grid_constant__ Turns turns) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
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
  if (threadIdx.x < kD / 2) {
    sm.turn_hi[threadIdx.x] = turns.hi[threadIdx.x];
    sm.turn_lo[threadIdx.x] = turns.lo[threadIdx.x];
  }
  // every head block writes the same bytes
  if (a.new_slot && c1 == n && warp < 2) append_row<T>(a, b, g, warp == 1);
  __syncthreads();
  for (int x = threadIdx.x; x < heads * (kD / 2); x += kSThreads) {
    const int h = x / (kD / 2), f = x % (kD / 2);
    float c, s;
    turn_cs(sm.turn_hi[f], sm.turn_lo[f], a.qpos[b], &c, &s);
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
        turn_cs(turns.hi[f], turns.lo[f], pos, &c, &s);
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
      a.o[(((int64_t)b * a.Hq + h0 + odd + 2 * x) * a.ctas + split) * kD + d] = o[x];
#pragma unroll
  for (int x = 0; x < kSHeads / 4; ++x) {
    float s = l[x];
#pragma unroll
    for (int y = 16; y; y >>= 1) s += __shfl_xor_sync(0xffffffffu, s, y);
    if (lane == 0 && warp + 4 * x < heads)
      a.ml[((int64_t)b * a.Hq + h0 + warp + 4 * x) * a.ctas + split] = make_float2(m[x] * kScale, s);
  }
}

// ---------------------------------------------------------------------------
// bf16: mma.sync.  The entries of all lists, one list behind the other, are cut
// into equal ranges, one for each CTA that the GPU holds at a time, so that lists
// of any lengths leave no SM idle; a range may end inside a list and hold several
// lists, and leaves a partial for each list that it touches.  A CTA takes up to
// eight KV heads, a warp each, 32 entries at a time; with fewer heads kSub groups of
// warps take 32 entries each.
//   S = Q K^T      m16n8k16: rows 0 .. 7 are the query heads' high fp16 parts, rows
//                  8 .. 15 their low parts, so that a score is two accumulators
//                  and no row is padding; B is eight rotated keys.
//   O^T = V^T P^T  m16n8k16: 16 dimensions x eight heads, B is the weights as the
//                  scores' accumulators hold them.
// Codes become fp16 pairs by one conversion each, exactly.  Keys are rotated in
// fp16 (three roundings of 2^-11) from a table of cos and sin that all warps of the
// CTA fill for the next tile: half the instructions of fp32 and, for a key that
// has four significant bits, nothing lost.  Scales meet the scores, and the
// weights before their rounding to fp16, as fp32 powers of two.
//
// Weights are 2^(score - m) with m any reference near the maximum; times the
// value's scale and a power of two f they are rounded to fp16.  A tile in which
// a score passes m by 60 or a weight fp16's range, or which has a scale that times f
// might pass fp32's (a weight of 0 times infinity), raises m to the maximum and sets f
// so that the largest weight is near 2^8 and no scale of the tile times f passes 2^127.
//
// An entry's row of all the CTA's heads is copied by neighbouring lanes
// (cp.async), several tiles ahead, and so are list entries, scales and positions
// (a plain load returns only after the copies queued before it).
//
// 14 requests of 20,000 to 90,000 entries, 64 / 8 heads: 162.5 us the call, 4.7 TB/s
// (the floor is 111); decode_heads_kernel over bf16 keys before RoPE takes 292 for
// 766,000 entries, these are 720,000.  256 instructions per 16 entries and head; no
// pipe is full: with 16 warps per SM the latency of a step's chain and its barrier
// bound it.  With 16 entries a step, or splits of 512 entries instead of ranges, 219
// and 256 us.
// ---------------------------------------------------------------------------
constexpr int kMWarps = 8, kMThreads = 32 * kMWarps, kMKeys = 32;
// tiles of a warp, and of list entries and positions: what leaves room for two
// CTAs per SM (one with eight groups)
constexpr int stages_of(int sub) { return sub == 1 ? 3 : 2; }
constexpr int ring_of(int sub) { return sub == 1 ? 8 : 4; }
constexpr int kMTile = kMKeys * kD;       // bytes of a K (or V) tile of a head
constexpr int kMTable = kMKeys * kD * 2;  // cos and sin of a tile, fp16
constexpr int kMLeast = 2;                // tiles of a CTA, unless there are fewer
constexpr uint32_t kHighScale = (127u + 27) << 23;  // 2^27, which the largest f takes to 2^127
constexpr int kMScale = 16;               // bytes that hold a row's scales of eight heads from any byte on
template <int kSub>
struct __align__(16) MmaSmem {
  uint8_t kv[stages_of(kSub)][2][kMWarps][kMTile];
  uint8_t table[2][kSub][kMTable];
  uint8_t scale[stages_of(kSub)][2][kMKeys * kSub][kMScale];
  int idx[ring_of(kSub)][kMKeys * kSub], pos[ring_of(kSub)][kMKeys * kSub];
  float power[kMWarps][2][kMKeys];  // the current tile's scales of K and of V
  float cs[kD / 2], sn[kD / 2];  // of the query
};

__device__ __forceinline__ uint32_t smem_u32(const void *p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0));
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void load_matrices(uint32_t addr, uint32_t *r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void load_matrices_t(uint32_t addr, uint32_t *r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_f16(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_first(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float x, float y, float z) {
  float m;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(x), "f"(y), "f"(z));
  return m;
}
__device__ __forceinline__ __half2 half2_of(uint32_t x) { return *reinterpret_cast<__half2 *>(&x); }
__device__ __forceinline__ uint32_t bits_of(__half2 x) { return *reinterpret_cast<uint32_t *>(&x); }
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  return bits_of(__floats2half2_rn(lo, hi));
}
// byte offset of (key, 16-byte column) in a [32][64] tile of codes: eight keys at
// one column fall in different banks
__device__ __forceinline__ uint32_t code_at(int key, int col) {
  return (uint32_t)(key * kD + ((col ^ ((key >> 1) & 3)) << 4));
}

// The ranges of a call: `ctas` equal parts of its entries, but none of less than
// kMLeast tiles.
struct Ranges {
  int64_t base, total, parts;  // first entry, entries, ranges
  __device__ __forceinline__ Ranges(const Decode8 &a, int step) {
    base = a.indptr[0];
    total = max(0, a.indptr[a.B] - (int)base);
    parts = min((int64_t)a.ctas, max((int64_t)1, (total + step * kMLeast - 1) / (step * kMLeast)));
  }
  __device__ __forceinline__ int64_t first(int64_t i) const { return base + i * total / parts; }
  // the range that holds entry e
  __device__ __forceinline__ int range_of(int64_t e) const {
    return (int)(((e - base + 1) * parts - 1) / total);
  }
};

// kTiles: eight query heads each, one or two; kSub: groups of nh warps
template <int kTiles, int kSub>
__global__ void __launch_bounds__(kMThreads, kTiles == 1 && kSub < 8 ? 2 : 1)
    decode8_mma_kernel(const Decode8 a, const __grid_constant__ Turns turns, int nh) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  MmaSmem<kSub> &sm = *reinterpret_cast<MmaSmem<kSub> *>(smem_raw);
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  constexpr int kHeads = 8 * kTiles, kStep = kMKeys * kSub;
  constexpr int kMStages = stages_of(kSub), kMRing = ring_of(kSub);
  const int blocks = (a.grp + kHeads - 1) / kHeads;
  const int hb = blockIdx.y % blocks, g0 = blockIdx.y / blocks * nh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  const int part = warp / nh, hw = warp - part * nh, g = g0 + hw;
  const bool active = part < kSub && g < a.Hkv;
  const int h0 = g * a.grp + hb * kHeads, heads = min(kHeads, a.grp - hb * kHeads);
  const Ranges ranges(a, kStep);
  if (blockIdx.x >= ranges.parts) return;
  int64_t e0 = ranges.first(blockIdx.x);
  const int64_t e_end = ranges.first(blockIdx.x + 1);
  int b = 0;  // the last request whose list begins at e0 or before
  for (int hi = a.B; hi - b > 1;) {
    const int mid = (b + hi) >> 1;
    if (__ldg(a.indptr + mid) <= e0) b = mid; else hi = mid;
  }

  // This thread copies a 16-byte column of four rows of a step, a quarter of the
  // step apart, of K and of V.
  constexpr int kQuarter = kStep / 4;
  const int col = threadIdx.x % (4 * nh), row0 = threadIdx.x / (4 * nh);
  const bool copies = row0 < kQuarter && g0 + (col >> 2) < a.Hkv;
  const uint8_t *const k_col = a.pool.k + g0 * kD + col * 16, *const v_col = a.pool.v + g0 * kD + col * 16;
  const uint32_t col_at = smem_u32(sm.kv) + ((row0 / kMKeys) * nh + (col >> 2)) * kMTile +
                          code_at(row0 % kMKeys, col & 3);
  const uint32_t row_bytes = (uint32_t)a.Hkv * kD;
  const int64_t scales = (int64_t)a.pool.S * a.Hkv;
  const int odd = a.Hkv & 3;  // not 0: a row's scales may begin at any byte
  auto slot_in = [&](int slot) { return (unsigned)slot < (unsigned)a.pool.S ? (uint32_t)slot : 0u; };
  // this thread's frequencies of the table, f and f + 1
  const int tf = 2 * (threadIdx.x % 16), tkey = threadIdx.x / 16;
  const int t_hi[2] = {turns.hi[tf], turns.hi[tf + 1]}, t_lo[2] = {turns.lo[tf], turns.lo[tf + 1]};
  const uint32_t table_at = tkey * 128 +
                            ((((tf >> 4) * 4 + ((tf >> 2) & 3)) ^ ((tkey & 1) << 2)) << 4) +
                            ((tf >> 1) & 1) * 4;

  // this lane's part of the tiles: matrix rows of K and (columns 0, 16 of 64; ^ 32:
  // 32, 48) of V, cos and sin of dimensions 4 tig .. (^ 64: 16 + 4 tig ..)
  const uint32_t tile_at = smem_u32(sm.kv[0][0][warp]);
  const uint32_t k_at = code_at(lane & 7, lane >> 3);
  const uint32_t v_at = code_at((lane >> 3 & 1) * 8 + (lane & 7), lane >> 4);
  const uint32_t cs_at = gid * 128 + ((tig ^ ((gid & 1) << 2)) << 4);

  for (; e0 < e_end; ++b) {
    const int beg = __ldg(a.indptr + b), end = __ldg(a.indptr + b + 1);
    const int64_t e1 = min(e_end, (int64_t)end);
    const int c0 = (int)(e0 - beg), nk = min((int)(e1 - beg), a.max_kv) - c0;
    if (b + 1 >= a.B) e0 = e_end; else e0 = max(e0, e1);
    if (nk <= 0) continue;
    const int n = min(end - beg, a.max_kv);
    const int n_tiles = (nk + kStep - 1) / kStep;
    const int32_t *const list = a.indices + (int64_t)beg + c0, *const pos = a.kvpos + (int64_t)beg + c0;

    if (threadIdx.x < kD / 2) {
      const int f = threadIdx.x;
      turn_cs(turns.hi[f], turns.lo[f], a.qpos[b], &sm.cs[f], &sm.sn[f]);
    }
    for (int x = threadIdx.x; x < kMStages * kStep; x += kMThreads) {
      (&sm.idx[0][0])[x] = x < nk ? __ldg(list + x) : 0;
      (&sm.pos[0][0])[x] = x < nk ? __ldg(pos + x) : 0;
    }
    if (a.new_slot && c0 + nk == n && active && part == 0) {
      append_row<__nv_bfloat16>(a, b, g, false);
      append_row<__nv_bfloat16>(a, b, g, true);
    }

    // rows and scales of tile t, list entries and positions of tile t + kMStages
    auto issue = [&](int t) {
      const int left = nk - t * kStep;
      if (left > 0) {
        const int *entry = sm.idx[t % kMRing];
        const uint32_t stage = t % kMStages;
        if (copies) {
          const uint32_t to = col_at + stage * (2 * kMWarps * kMTile);
          auto rows = [&](auto whole) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int key = row0 + i * kQuarter;
              const bool listed = decltype(whole)::value || key < left;
              const uint64_t off = (uint64_t)(listed ? slot_in(entry[key]) : 0u) * row_bytes;
              const uint32_t at =
                  to + (i * kQuarter % kMKeys) * kD + (i * kQuarter / kMKeys) * nh * kMTile;
              copy16(at, k_col + off, listed);
              copy16(at + kMWarps * kMTile, v_col + off, listed);
            }
          };
          if (left >= kStep) rows(std::true_type());
          else rows(std::false_type());
        }
        // a warp's 32 threads have one of the four arrays
#pragma unroll
        for (int z = 0; z < 4 * kStep; z += kMThreads) {
          const int what = (z + threadIdx.x) / kStep, key = (z + threadIdx.x) % kStep;
          if (what < 2 && key < left) {
            const int64_t first = (int64_t)slot_in(entry[key]) * a.Hkv + g0;
            const uint8_t *const src = what ? a.pool.v_scale : a.pool.k_scale;
            const uint32_t to = smem_u32(sm.scale[stage][what][key]);
            if ((a.Hkv & 7) == 0) copy8(to, src + first);
            else if (a.Hkv == 4) copy4(to, src + first, 4);
            else {  // as many words as the CTA's heads lie in, up to the last row's end
              const int64_t word = first & ~(int64_t)3;
              for (int w = 0; w < (((int)(first & 3) + nh + 3) >> 2); ++w)
                if (word + 4 * w < scales)
                  copy4(to + 4 * w, src + word + 4 * w, (int)min(scales - word - 4 * w, (int64_t)4));
            }
          } else if (what >= 2 && what < 4) {
            const int x = (t + kMStages) * kStep + key;
            if (x < nk)
              copy4(smem_u32(&(what == 2 ? sm.idx : sm.pos)[(t + kMStages) % kMRing][key]),
                    (what == 2 ? list : pos) + x, 4);
          }
        }
      }
      asm volatile("cp.async.commit_group;\n" ::: "memory");
    };
    // cos and sin of tile t's positions for this thread's frequencies
    auto table = [&](int t) {
#pragma unroll
      for (int s = 0; s < 2 * kSub; ++s) {
        const int p = sm.pos[t % kMRing][s * 16 + tkey];
        float c[2], sn[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // the turn, half of one added, as a number in [1, 2): angles in +-pi
          const uint32_t u = turn_of(t_hi[e], t_lo[e], p) + 0x80000000u;
          const float x = fmaf(__uint_as_float(u >> 9 | 0x3f800000u), 6.2831853f, -9.4247780f);
          c[e] = __cosf(x);
          sn[e] = __sinf(x);
        }
        uint8_t *row = sm.table[t & 1][s >> 1] + (s & 1) * (kMTable / 2) + table_at;
        *reinterpret_cast<uint32_t *>(row) = pack_f16(c[0], c[1]);
        *reinterpret_cast<uint32_t *>(row + 8) = pack_f16(sn[0], sn[1]);
      }
    };
    __syncthreads();  // list entries, positions, the query's angles, the appended row
#pragma unroll
    for (int t = 0; t < kMStages - 1; ++t) issue(t);
    table(0);

    // Q: rotated, 1/sqrt(D) log2(e) folded in, scaled by a power of two to 16 .. 32,
    // split into fp16 parts.  k index 2 tig (+1) of step c is dimension 16 c + 4 tig
    // (+1), 2 tig + 8 (+1) the two after these, as a 4-byte piece of a row of codes
    // holds them.
    uint32_t qa[kTiles][4][4];
    float r[kTiles];  // the row's power of two
#pragma unroll
    for (int ht = 0; ht < kTiles; ++ht) {
      const bool ok = active && 8 * ht + gid < heads;
      const __nv_bfloat16 *src =
          (const __nv_bfloat16 *)a.q + ((int64_t)b * a.Hq + (ok ? h0 + 8 * ht + gid : 0)) * kD;
      float x[4][4];
      uint32_t top = 0;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint2 w = ok ? __ldg(reinterpret_cast<const uint2 *>(src + 16 * c + 4 * tig)) : make_uint2(0u, 0u);
        x[c][0] = __uint_as_float(w.x << 16) * kScale;
        x[c][1] = __uint_as_float(w.x & 0xffff0000u) * kScale;
        x[c][2] = __uint_as_float(w.y << 16) * kScale;
        x[c][3] = __uint_as_float(w.y & 0xffff0000u) * kScale;
      }
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int f = 16 * c + 4 * tig + e;
          const float u = x[c][e], w = x[c + 2][e];
          x[c][e] = u * sm.cs[f] - w * sm.sn[f];
          x[c + 2][e] = u * sm.sn[f] + w * sm.cs[f];
          top = max(top, max(__float_as_uint(x[c][e]) & 0x7fffffffu,
                             __float_as_uint(x[c + 2][e]) & 0x7fffffffu));
        }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // exponent of r: that of the largest component less 4, its inverse in range too
      const int e = min(max((int)(top >> 23) - 4, 4), 250);
      r[ht] = __uint_as_float((uint32_t)e << 23);
      const float inv = __uint_as_float((uint32_t)(254 - e) << 23);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float hi[4], lo[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const float y = x[c][d] * inv;
          hi[d] = __half2float(__float2half_rn(y));
          lo[d] = y - hi[d];
        }
        qa[ht][c][0] = pack_f16(hi[0], hi[1]);
        qa[ht][c][1] = pack_f16(lo[0], lo[1]);
        qa[ht][c][2] = pack_f16(hi[2], hi[3]);
        qa[ht][c][3] = pack_f16(lo[2], lo[3]);
      }
    }
    float o[kTiles][4][4], m[kTiles], l[kTiles], f[kTiles];
#pragma unroll
    for (int ht = 0; ht < kTiles; ++ht) {
#pragma unroll
      for (int c = 0; c < 4; ++c) o[ht][c][0] = o[ht][c][1] = o[ht][c][2] = o[ht][c][3] = 0.f;
      m[ht] = -INFINITY;
      l[ht] = 0.f;
      f[ht] = 1.f;
    }
    asm volatile("cp.async.wait_group %0;\n" ::"n"(kMStages - 2) : "memory");
    __syncthreads();  // tile 0 and its table

    for (int it = 0; it < n_tiles; ++it) {
      table(it + 1);  // past the end: of whatever the ring holds
      const int left = nk - it * kStep - kMKeys * part;
      if (!(active && left > 0)) {
        issue(it + kMStages - 1);
      } else {
        uint32_t value;  // bits of this lane's value scale, ordered as it is
        const uint32_t kt = tile_at + it % kMStages * (2 * kMWarps * kMTile), vt = kt + kMWarps * kMTile;
        {
          const int key = part * kMKeys + lane;
          const bool listed = lane < left;
          uint32_t off = hw;
          if (odd) off += (slot_in(listed ? sm.idx[it % kMRing][key] : 0) * a.Hkv + g0) & 3;
          const uint8_t(*scale)[kStep][kMScale] = sm.scale[it % kMStages];
          sm.power[warp][0][lane] = listed ? kv8_power(scale[0][key][off]) : 0.f;
          const float vp = listed ? kv8_power(scale[1][key][off]) : 0.f;
          sm.power[warp][1][lane] = vp;
          value = __float_as_uint(vp);
        }
        float s[kTiles][4][4];
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
          uint32_t kc[4], kb[4][2];
          load_matrices(kt + k_at + 8 * nb * kD, kc);
          const uint8_t *row = sm.table[it & 1][kSub == 1 ? 0 : part] + 8 * nb * 128;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint4 t4 = *reinterpret_cast<const uint4 *>(row + (c ? cs_at ^ 64 : cs_at));
            const uint32_t cs[2] = {t4.x, t4.y}, sn[2] = {t4.z, t4.w};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const __half2 x1 = half2_of(kv8_pair((uint16_t)(kc[c] >> (16 * e))));
              const __half2 x2 = half2_of(kv8_pair((uint16_t)(kc[c + 2] >> (16 * e))));
              const __half2 cc = half2_of(cs[e]), ss = half2_of(sn[e]);
              kb[c][e] = bits_of(__hfma2(x1, cc, __hneg2(__hmul2(x2, ss))));
              kb[c + 2][e] = bits_of(__hfma2(x1, ss, __hmul2(x2, cc)));
            }
          }
#pragma unroll
          for (int ht = 0; ht < kTiles; ++ht) {
            mma_f16_first(s[ht][nb], qa[ht][0], kb[0][0], kb[0][1]);
#pragma unroll
            for (int c = 1; c < 4; ++c) mma_f16(s[ht][nb], qa[ht][c], kb[c][0], kb[c][1]);
          }
        }
        __syncwarp();  // the powers
        uint32_t pb[kTiles][4];
#pragma unroll
        for (int ht = 0; ht < kTiles; ++ht) {
          float2 u[4], p[4], w[4];
          const float2 r2 = make_float2(r[ht], r[ht]), m2 = make_float2(-m[ht], -m[ht]);
          const float2 f2 = make_float2(f[ht], f[ht]);
          auto vp = [&](int nb) {
            return *reinterpret_cast<const float2 *>(&sm.power[warp][1][8 * nb + 2 * tig]);
          };
#pragma unroll
          for (int nb = 0; nb < 4; ++nb) {
            const float *x = s[ht][nb];
            const float2 kp = *reinterpret_cast<const float2 *>(&sm.power[warp][0][8 * nb + 2 * tig]);
            u[nb] = __fmul2_rn(__fadd2_rn(make_float2(x[0], x[1]), make_float2(x[2], x[3])),
                               __fmul2_rn(kp, r2));
          }
          if (left < kMKeys) {
#pragma unroll
            for (int nb = 0; nb < 4; ++nb) {
              if (8 * nb + 2 * tig >= left) u[nb].x = -INFINITY;
              if (8 * nb + 2 * tig + 1 >= left) u[nb].y = -INFINITY;
            }
          }
          float far = -INFINITY, most = 0.f;
#pragma unroll
          for (int nb = 0; nb < 4; ++nb) {
            const float2 x = __fadd2_rn(u[nb], m2);
            p[nb] = make_float2(ex2(x.x), ex2(x.y));
            w[nb] = __fmul2_rn(p[nb], __fmul2_rn(vp(nb), f2));
            far = max3(far, x.x, x.y);
            most = max3(most, w[nb].x, w[nb].y);
          }
          if (__any_sync(0xffffffffu, it == 0 || far > 60.f || most > 32768.f || value >= kHighScale)) {
            float mx = m[ht];
#pragma unroll
            for (int nb = 0; nb < 4; ++nb) mx = max3(mx, u[nb].x, u[nb].y);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float ref = mx == -INFINITY ? 0.f : mx, alpha = ex2(m[ht] - ref);
            m[ht] = mx;
            float big = 0.f;
#pragma unroll
            for (int nb = 0; nb < 4; ++nb) {
              p[nb] = make_float2(ex2(u[nb].x - ref), ex2(u[nb].y - ref));
              w[nb] = __fmul2_rn(p[nb], vp(nb));
              big = max3(big, w[nb].x, w[nb].y);
            }
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
            const uint32_t scale = __reduce_max_sync(0xffffffffu, value);
            // 2^8 over the largest weight's power of two, at most 2^100, 2^127 over
            // the largest scale and, once there are sums, 2^60 times what it was
            const int e8 = min(min(262 - (int)(__float_as_uint(big) >> 23), 227),
                               381 - (int)(scale >> 23));
            float f_new = __uint_as_float((uint32_t)e8 << 23);
            if (it > 0) f_new = fminf(f_new, f[ht] * 1.1529215e18f);
            const float ratio = it > 0 ? alpha * (f_new / f[ht]) : 0.f;
            f[ht] = f_new;
            l[ht] *= alpha;
            const float ra = __shfl_sync(0xffffffffu, ratio, 8 * tig);
            const float rb = __shfl_sync(0xffffffffu, ratio, 8 * tig + 4);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              o[ht][c][0] *= ra;
              o[ht][c][1] *= rb;
              o[ht][c][2] *= ra;
              o[ht][c][3] *= rb;
            }
#pragma unroll
            for (int nb = 0; nb < 4; ++nb)
              w[nb] = __fmul2_rn(p[nb], __fmul2_rn(vp(nb), make_float2(f_new, f_new)));
          }
          const float2 sum = __fadd2_rn(__fadd2_rn(p[0], p[1]), __fadd2_rn(p[2], p[3]));
          l[ht] += sum.x + sum.y;
#pragma unroll
          for (int nb = 0; nb < 4; ++nb) pb[ht][nb] = pack_f16(w[nb].x, w[nb].y);
        }
        issue(it + kMStages - 1);  // while the weights' products wait for nothing else
        // V: a transposed matrix's register holds dimensions d, d + 1 of two keys
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
            uint32_t vc[4];
            load_matrices_t(vt + (cc ? v_at ^ 32 : v_at) + 16 * kk * kD, vc);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const uint32_t x0 = __byte_perm(vc[2 * c], 0, 0x3120), x1 = __byte_perm(vc[2 * c + 1], 0, 0x3120);
              const uint32_t va[4] = {kv8_pair((uint16_t)x0), kv8_pair((uint16_t)(x0 >> 16)),
                                      kv8_pair((uint16_t)x1), kv8_pair((uint16_t)(x1 >> 16))};
#pragma unroll
              for (int ht = 0; ht < kTiles; ++ht)
                mma_f16(o[ht][2 * cc + c], va, pb[ht][2 * kk], pb[ht][2 * kk + 1]);
            }
          }
      }
      asm volatile("cp.async.wait_group %0;\n" ::"n"(kMStages - 2) : "memory");
      __syncthreads();  // the next tile and its table; this one's readers are done
    }
    asm volatile("cp.async.wait_group 0;\n" ::: "memory");
    if (active) {
#pragma unroll
      for (int ht = 0; ht < kTiles; ++ht) {
        l[ht] += __shfl_xor_sync(0xffffffffu, l[ht], 1);
        l[ht] += __shfl_xor_sync(0xffffffffu, l[ht], 2);
        const float inv = 1.f / f[ht];
        // range + request never repeats: along the entries one of the two grows
        const int64_t base = ((int64_t)(blockIdx.x + b) * kSub + part) * a.Hq + h0 + 8 * ht;
        if (tig == 0 && 8 * ht + gid < heads) a.ml[base + gid] = make_float2(m[ht], l[ht]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float y = __shfl_sync(0xffffffffu, inv, 8 * tig + 4 * e);
          if (8 * ht + 2 * tig + e >= heads) continue;
          float *to = a.o + (base + 2 * tig + e) * kD + 2 * gid;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            *reinterpret_cast<float2 *>(to + 16 * c) = make_float2(o[ht][c][e] * y, o[ht][c][2 + e] * y);
        }
      }
    }
  }
}

// Joins a row's partials by their log-sum-exp: CTA = (query head, request), 16
// groups of 16 threads each summing every 16th partial's row, eight loads in
// flight (one request may have 304 partials).  Launched as a
// programmatic dependent of the attention kernel.  A request without entries
// gets zeros.
constexpr int kMergeThreads = 256, kMergeGroups = kMergeThreads / 16, kMaxParts = 2560;
template <typename T>
__global__ void __launch_bounds__(kMergeThreads) decode8_merge_kernel(const Decode8 a, T *out) {
  __shared__ float2 part[kMaxParts];  // (maximum, then weight; sum)
  __shared__ float4 red[kMergeGroups][kD / 4];
  __shared__ float tot[kMergeThreads / 32], top[kMergeThreads / 32];
  const int h = blockIdx.x, b = blockIdx.y;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int beg;
  const int n = list_of(a, b, &beg);
  // partials of this row: the first, how many, how far apart
  int64_t at, apart;
  int used = 0;
  if constexpr (sizeof(T) == 4) {
    used = (n + a.chunk - 1) / a.chunk;
    at = ((int64_t)b * a.Hq + h) * a.ctas;
    apart = 1;
  } else {
    const Ranges ranges(a, kMKeys * a.sub);
    int first = 0;
    if (n > 0) {
      first = ranges.range_of(beg);
      used = (ranges.range_of((int64_t)beg + n - 1) - first + 1) * a.sub;
    }
    at = (int64_t)(first + b) * a.sub * a.Hq + h;
    apart = a.Hq;
  }
  const int64_t w = (int64_t)b * a.Hq + h;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const float2 *ml = a.ml + at;
  float M = -INFINITY;
  for (int s = threadIdx.x; s < used; s += kMergeThreads) {
    part[s] = __ldcg(ml + s * apart);
    M = fmaxf(M, part[s].x);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) top[warp] = M;
  __syncthreads();
#pragma unroll
  for (int x = 0; x < kMergeThreads / 32; ++x) M = fmaxf(M, top[x]);
  const float ref = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  for (int s = threadIdx.x; s < used; s += kMergeThreads) {
    const float f = exp2f(part[s].x - ref);
    part[s].x = f;
    L = fmaf(part[s].y, f, L);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  if (lane == 0) tot[warp] = L;
  __syncthreads();
  L = 0.f;
#pragma unroll
  for (int x = 0; x < kMergeThreads / 32; ++x) L += tot[x];
  const int cg = threadIdx.x & 15, sg = threadIdx.x >> 4;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int s = sg; s < used; s += kMergeGroups) {
    const float4 v = __ldcg(reinterpret_cast<const float4 *>(a.o + (at + s * apart) * kD) + cg);
    const float f = part[s].x;
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
    for (int y = 0; y < kMergeGroups; ++y)
      x += reinterpret_cast<const float *>(&red[y][col >> 2])[col & 3];
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

// The cut of the work, from the host's bounds alone, so that a captured call
// replays for any lengths within them.
struct Decode8Plan {
  int ctas, chunk, sub;
  int nh, blocks;  // KV heads per CTA (bf16), query head blocks of a KV head
  size_t parts;    // partials of a query head, over the batch
  size_t most;     // the most of any call with no larger B and max_kv
};
Decode8Plan plan_of(int dtype, int B, int Hq, int Hkv, int max_kv) {
  Decode8Plan p;
  const int grp = Hq / Hkv, sms = sm_count();
  if (dtype == AKV_BF16) {
    const int tiles = grp <= 8 ? 1 : 2;
    p.blocks = (grp + 8 * tiles - 1) / (8 * tiles);
    p.nh = std::min(Hkv, kMWarps);
    p.sub = kMWarps / p.nh >= 8 ? 8 : kMWarps / p.nh >= 4 ? 4 : kMWarps / p.nh >= 2 ? 2 : 1;
    p.chunk = 0;
    // as many as the SMs hold at a time; no more than the merge's table has room for
    const int ny = (Hkv + p.nh - 1) / p.nh * p.blocks, per_sm = tiles == 1 && p.sub < 8 ? 2 : 1;
    p.ctas = std::min(std::max(1, per_sm * sms / ny), kMaxParts / p.sub);
    p.parts = p.most = ((size_t)p.ctas + B) * p.sub;
  } else {
    p.blocks = (grp + kSHeads - 1) / kSHeads;
    p.nh = p.sub = 1;
    const auto splits = [&](int x) { return std::max<int64_t>(1, ((int64_t)max_kv + x - 1) / x); };
    const int64_t rows = (int64_t)B * Hkv * p.blocks;
    int c = 4096;
    const int64_t want = 4LL * 4 * sms;
    while (c > kSKeys && rows * splits(c) < want) c /= 2;
    while (splits(c) > kMaxParts) c *= 2;
    p.ctas = (int)splits(c);
    p.chunk = c;
    p.parts = (size_t)p.ctas * B;
    // A smaller batch or shorter lists may be cut finer.  Splits below the longest
    // were chosen because twice their length left rows * splits below `want`, so
    // that rows * splits is below 2 * want; none is shorter than kSKeys.
    const int64_t fine = std::min(B * splits(kSKeys), (2 * want - 1) / (Hkv * p.blocks));
    p.most = (size_t)std::max(fine, B * std::min<int64_t>(splits(4096), kMaxParts));
  }
  return p;
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

template <typename T>
cudaError_t launch_merge(const Decode8 &a, void *out, cudaStream_t s) {
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

cudaError_t launch_simt(const Decode8 &a, const Decode8Plan &p, const RopeTheta &th, cudaStream_t s) {
  const int smem = (int)sizeof(SimtSmem);
  const cudaError_t e = cudaFuncSetAttribute(decode8_simt_kernel<float>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  decode8_simt_kernel<float><<<dim3(p.ctas, a.Hkv * p.blocks, a.B), kSThreads, smem, s>>>(a, turns_of(th));
  return cudaGetLastError();
}

template <int kTiles, int kSub>
cudaError_t launch_mma(const Decode8 &a, const Decode8Plan &p, const Turns &turns, cudaStream_t s) {
  const int smem = (int)sizeof(MmaSmem<kSub>);
  const cudaError_t e = cudaFuncSetAttribute(decode8_mma_kernel<kTiles, kSub>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  decode8_mma_kernel<kTiles, kSub>
      <<<dim3(p.ctas, (a.Hkv + p.nh - 1) / p.nh * p.blocks), kMThreads, smem, s>>>(a, turns, p.nh);
  return cudaGetLastError();
}
template <int kTiles>
cudaError_t launch_mma(const Decode8 &a, const Decode8Plan &p, const RopeTheta &th, cudaStream_t s) {
  const Turns turns = turns_of(th);
  return p.sub == 8   ? launch_mma<kTiles, 8>(a, p, turns, s)
         : p.sub == 4 ? launch_mma<kTiles, 4>(a, p, turns, s)
         : p.sub == 2 ? launch_mma<kTiles, 2>(a, p, turns, s)
                      : launch_mma<kTiles, 1>(a, p, turns, s);
}

}  // namespace

size_t decode_q8_workspace_bytes(int dtype, int B, int Hq, int Hkv, int max_kv) {
  const size_t parts = plan_of(dtype, B, Hq, Hkv, max_kv).most * Hq;
  return up256(parts * sizeof(float2)) + up256(parts * kD * sizeof(float));
}

cudaError_t launch_decode_q8(int dtype, int B, int Hq, int Hkv, const void *q, const int32_t *qpos,
                             const void *k_new, const void *v_new, const int32_t *new_slot,
                             const Kv8Pool &pool, const int32_t *indptr, const int32_t *indices,
                             const int32_t *kvpos, int max_kv, void *out, void *ws,
                             const RopeTheta &th, cudaStream_t s) {
  const Decode8Plan p = plan_of(dtype, B, Hq, Hkv, max_kv);
  const Decode8 a{B, Hq, Hkv, Hq / Hkv, q, qpos, k_new, v_new, new_slot, pool, indptr, indices, kvpos,
                  max_kv, (float2 *)ws, (float *)((char *)ws + up256(p.parts * Hq * sizeof(float2))),
                  p.ctas, p.chunk, p.sub};
  const cudaError_t e = dtype != AKV_BF16 ? launch_simt(a, p, th, s)
                        : a.grp <= 8      ? launch_mma<1>(a, p, th, s)
                                          : launch_mma<2>(a, p, th, s);
  if (e != cudaSuccess) return e;
  return dtype == AKV_BF16 ? launch_merge<__nv_bfloat16>(a, out, s) : launch_merge<float>(a, out, s);
}

}  // namespace akv
