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
  int ns, chunk, per;  // partials, entries of a split, partials of a split
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

// ---------------------------------------------------------------------------
// bf16: mma.sync, a warp per (KV head, 16 entries at a time).  CTA = key split x up
// to eight KV heads x request; with fewer heads the warps share out the tiles
// (`sub` of them at a time), each with a partial of its own.
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
// a score passes m by 60 or a weight fp16's range raises m to the maximum and
// sets f so that the largest weight is near 2^8.
//
// Rows travel by cp.async, several tiles ahead, and so do list entries, scales
// and positions (a plain load returns only after the copies queued before it).
// ---------------------------------------------------------------------------
constexpr int kMWarps = 8, kMThreads = 32 * kMWarps, kMKeys = 16, kMStages = 4;
constexpr int kMTile = kMKeys * kD;      // bytes of a K (or V) tile
constexpr int kMRing = 2 * kMStages;     // of list entries and positions
constexpr int kMTable = kMKeys * kD * 2; // cos and sin of a tile, fp16
struct __align__(16) MmaSmem {
  uint8_t kv[kMWarps][kMStages][2][kMTile];
  uint32_t scale[kMWarps][kMStages][32];  // the words that hold 16 K and 16 V scales
  float power[kMWarps][32];               // these scales of the current tile
  int idx[kMWarps][kMRing][kMKeys];
  float cs[kD / 2], sn[kD / 2];           // of the query
  ThetaSmem ts;
  double thd[kD / 2];
  // then pos [kMRing][16 sub], the tables [2][sub][kMTable]
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
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ __half2 half2_of(uint32_t x) { return *reinterpret_cast<__half2 *>(&x); }
__device__ __forceinline__ uint32_t bits_of(__half2 x) { return *reinterpret_cast<uint32_t *>(&x); }
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  return bits_of(__floats2half2_rn(lo, hi));
}
// byte offset of (key, 16-byte column) in a [16][64] tile of codes: eight keys at
// one column fall in different banks
__device__ __forceinline__ uint32_t code_at(int key, int col) {
  return (uint32_t)(key * kD + ((col ^ ((key >> 1) & 3)) << 4));
}
// cos/sin of positions past 2^18; rare, so out of line
__device__ __noinline__ float2 cs_wide(double theta, int pos) {
  float2 r;
  rope_cs(theta, (double)pos, &r.x, &r.y);
  return r;
}

// kTiles: eight query heads each, one or two
template <int kTiles>
__global__ void __launch_bounds__(kMThreads, kTiles == 1 ? 2 : 1)
    decode8_mma_kernel(const Decode8 a, const __grid_constant__ RopeTheta th, int nh, int sub) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  MmaSmem &sm = *reinterpret_cast<MmaSmem *>(smem_raw);
  int *const pos_ring = reinterpret_cast<int *>(smem_raw + sizeof(MmaSmem));
  uint8_t *const tables = smem_raw + sizeof(MmaSmem) + kMRing * kMKeys * sub * 4;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  constexpr int kHeads = 8 * kTiles;
  const int blocks = (a.grp + kHeads - 1) / kHeads;
  const int split = blockIdx.x, hb = blockIdx.y % blocks, b = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  const int part = warp / nh, g = (blockIdx.y / blocks) * nh + warp % nh;
  const bool active = part < sub && g < a.Hkv;
  const int h0 = g * a.grp + hb * kHeads, heads = min(kHeads, a.grp - hb * kHeads);
  int beg;
  const int n = list_of(a, b, &beg);
  const int c0 = split * a.chunk;
  if (c0 >= n) return;  // the merge reads only splits that hold entries
  const int nk = min(n - c0, a.chunk);
  const int step = kMKeys * sub, n_tiles = (nk + step - 1) / step;
  const int32_t *const list = a.indices + (int64_t)beg + c0, *const pos = a.kvpos + (int64_t)beg + c0;

  stage_theta(th, sm.ts);
  if (threadIdx.x < kD / 2) {
    sm.thd[threadIdx.x] = th.th[threadIdx.x];
    rope_cs_lane(th, threadIdx.x, a.qpos[b], &sm.cs[threadIdx.x], &sm.sn[threadIdx.x]);
  }
  for (int x = threadIdx.x; x < 2 * step; x += kMThreads) pos_ring[x] = x < nk ? __ldg(pos + x) : 0;
  if (a.new_slot && c0 + nk == n && active && part == 0) {
    append_row<__nv_bfloat16>(a, b, g, false);
    append_row<__nv_bfloat16>(a, b, g, true);
  }

  // first entry of this warp's tile t is 16 (t sub + part)
  const uint32_t kv = smem_u32(sm.kv[warp]);
  const int own = active ? nk - kMKeys * part : 0;  // entries from its first on
  auto fetch = [&](int t) {
    const int x = t * step + lane;
    if (lane < kMKeys && x < own)
      copy4(smem_u32(&sm.idx[warp][t % kMRing][lane]), list + kMKeys * part + x, 4);
  };
  const int64_t scales = (int64_t)a.pool.S * a.Hkv;
  auto row_of = [&](int slot) { return (int64_t)((unsigned)slot < (unsigned)a.pool.S ? slot : 0) * a.Hkv + g; };
  auto issue = [&](int t) {
    const int left = own - t * step;
    if (left > 0) {
      const int *entry = sm.idx[warp][t % kMRing];
      const uint32_t at = kv + t % kMStages * 2 * kMTile;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int key = (lane >> 2) + 8 * i, col = lane & 3;
        const bool valid = key < left;
        const int64_t off = row_of(valid ? entry[key] : 0) * kD + col * 16;
        copy16(at + code_at(key, col), a.pool.k + off, valid);
        copy16(at + kMTile + code_at(key, col), a.pool.v + off, valid);
      }
      const int key = lane & 15;
      const int64_t word = row_of(key < left ? entry[key] : 0) & ~(int64_t)3;
      copy4(smem_u32(&sm.scale[warp][t % kMStages][lane]),
            (lane < 16 ? a.pool.k_scale : a.pool.v_scale) + word,
            (int)min(scales - word, (int64_t)4));
      fetch(t + kMStages);
    }
    const int u = t + 2;  // the positions of the table to come
    for (int x = threadIdx.x; x < step; x += kMThreads)
      if (u * step + x < nk) copy4(smem_u32(pos_ring + u % kMRing * step + x), pos + u * step + x, 4);
    asm volatile("cp.async.commit_group;\n" ::: "memory");
  };
  // cos and sin of tile t's positions for this thread's frequencies f, f + 1
  const int tf = 2 * (threadIdx.x % 16);
  const uint32_t table_col = (tf >> 4) * 4 + ((tf >> 2) & 3), table_word = ((tf >> 1) & 1) * 4;
  auto table = [&](int t, int s) {
    const int key = threadIdx.x / 16, p = pos_ring[t % kMRing * step + s * kMKeys + key];
    float c0f, s0f, c1f, s1f;
    if (p < -262144 || p > 262144) {
      const float2 u = cs_wide(sm.thd[tf], p), w = cs_wide(sm.thd[tf + 1], p);
      c0f = u.x, s0f = u.y, c1f = w.x, s1f = w.y;
    } else {
      __sincosf(rope_angle(sm.ts.hi[tf], sm.ts.lo[tf], p), &s0f, &c0f);
      __sincosf(rope_angle(sm.ts.hi[tf + 1], sm.ts.lo[tf + 1], p), &s1f, &c1f);
    }
    uint8_t *row = tables + ((t & 1) * sub + s) * kMTable + key * 128 +
                   ((table_col ^ ((key & 1) << 2)) << 4) + table_word;
    *reinterpret_cast<uint32_t *>(row) = pack_f16(c0f, c1f);
    *reinterpret_cast<uint32_t *>(row + 8) = pack_f16(s0f, s1f);
  };
#pragma unroll
  for (int t = 0; t < kMStages; ++t) fetch(t);
  asm volatile("cp.async.wait_all;\n" ::: "memory");
  __syncthreads();  // frequencies, positions, the appended row
#pragma unroll
  for (int t = 0; t < kMStages - 1; ++t) issue(t);
  for (int s = 0; s < sub; ++s) table(0, s);

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
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        x[c][e] = ok ? __bfloat162float(src[16 * c + 4 * tig + e]) * kScale : 0.f;
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
      for (int e2 = 0; e2 < 4; ++e2) {
        const float y = x[c][e2] * inv;
        hi[e2] = __half2float(__float2half_rn(y));
        lo[e2] = y - hi[e2];
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
  __syncthreads();  // table 0

  for (int it = 0; it < n_tiles; ++it) {
    issue(it + kMStages - 1);
    if (it + 1 < n_tiles)
      for (int s = 0; s < sub; ++s) table(it + 1, s);
    asm volatile("cp.async.wait_group %0;\n" ::"n"(kMStages - 1) : "memory");
    __syncwarp();
    const int left = own - it * step;
    if (left > 0) {
      const uint32_t kt = kv + it % kMStages * 2 * kMTile, vt = kt + kMTile;
      {
        const int slot = sm.idx[warp][it % kMRing][lane & 15];
        const uint32_t shift = ((uint32_t)row_of((lane & 15) < left ? slot : 0) & 3) * 8;
        sm.power[warp][lane] = kv8_power((sm.scale[warp][it % kMStages][lane] >> shift) & 255u);
      }
      float s[kTiles][2][4];
#pragma unroll
      for (int nb = 0; nb < 2; ++nb) {
        uint32_t kc[4], kb[4][2];
        load_matrices(kt + code_at(8 * nb + (lane & 7), lane >> 3), kc);
        const int key = 8 * nb + gid;
        const uint8_t *row = tables + ((it & 1) * sub + part) * kMTable + key * 128;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint4 t4 =
              *reinterpret_cast<const uint4 *>(row + (((c * 4 + tig) ^ ((key & 1) << 2)) << 4));
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
          s[ht][nb][0] = s[ht][nb][1] = s[ht][nb][2] = s[ht][nb][3] = 0.f;
#pragma unroll
          for (int c = 0; c < 4; ++c) mma_f16(s[ht][nb], qa[ht][c], kb[c][0], kb[c][1]);
        }
      }
      __syncwarp();  // the powers
      float2 kp[2], vp[2];
#pragma unroll
      for (int nb = 0; nb < 2; ++nb) {
        kp[nb] = *reinterpret_cast<const float2 *>(&sm.power[warp][8 * nb + 2 * tig]);
        vp[nb] = *reinterpret_cast<const float2 *>(&sm.power[warp][16 + 8 * nb + 2 * tig]);
      }
      uint32_t pb[kTiles][2];
#pragma unroll
      for (int ht = 0; ht < kTiles; ++ht) {
        float u[4], w[4];
#pragma unroll
        for (int nb = 0; nb < 2; ++nb) {
          u[2 * nb] = (s[ht][nb][0] + s[ht][nb][2]) * (kp[nb].x * r[ht]);
          u[2 * nb + 1] = (s[ht][nb][1] + s[ht][nb][3]) * (kp[nb].y * r[ht]);
        }
        if (left < kMKeys) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if ((e >> 1) * 8 + 2 * tig + (e & 1) >= left) u[e] = -INFINITY;
        }
        const float v[4] = {vp[0].x, vp[0].y, vp[1].x, vp[1].y};
        float p[4], most = 0.f, far = -INFINITY;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = u[e] - m[ht];
          p[e] = ex2(x);
          w[e] = p[e] * (v[e] * f[ht]);
          far = fmaxf(far, x);
          most = fmaxf(most, w[e]);
        }
        if (__any_sync(0xffffffffu, it == 0 || far > 60.f || most > 32768.f)) {
          float mx = fmaxf(fmaxf(u[0], u[1]), fmaxf(u[2], u[3]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          mx = fmaxf(mx, m[ht]);
          const float ref = mx == -INFINITY ? 0.f : mx, alpha = ex2(m[ht] - ref);
          m[ht] = mx;
          most = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[e] = ex2(u[e] - ref);
            most = fmaxf(most, p[e] * v[e]);
          }
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
          // 2^8 over the largest weight's power of two, at most 2^100 and, once
          // there are sums, 2^60 times what it was
          const int e8 = min(262 - (int)(__float_as_uint(most) >> 23), 227);
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
          for (int e = 0; e < 4; ++e) w[e] = p[e] * (v[e] * f_new);
        }
        l[ht] += (p[0] + p[1]) + (p[2] + p[3]);
        pb[ht][0] = pack_f16(w[0], w[1]);
        pb[ht][1] = pack_f16(w[2], w[3]);
      }
      // V: a transposed matrix's register holds dimensions d, d + 1 of two keys
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        uint32_t vc[4];
        load_matrices_t(vt + code_at((lane >> 3 & 1) * 8 + (lane & 7), 2 * cc + (lane >> 4)), vc);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t x0 = __byte_perm(vc[2 * c], 0, 0x3120), x1 = __byte_perm(vc[2 * c + 1], 0, 0x3120);
          const uint32_t va[4] = {kv8_pair((uint16_t)x0), kv8_pair((uint16_t)(x0 >> 16)),
                                  kv8_pair((uint16_t)x1), kv8_pair((uint16_t)(x1 >> 16))};
#pragma unroll
          for (int ht = 0; ht < kTiles; ++ht) mma_f16(o[ht][2 * cc + c], va, pb[ht][0], pb[ht][1]);
        }
      }
    }
    __syncthreads();  // the next table; this one's and the tiles' readers are done
  }
  asm volatile("cp.async.wait_group 0;\n" ::: "memory");
  if (!active) return;
#pragma unroll
  for (int ht = 0; ht < kTiles; ++ht) {
    l[ht] += __shfl_xor_sync(0xffffffffu, l[ht], 1);
    l[ht] += __shfl_xor_sync(0xffffffffu, l[ht], 2);
    const float inv = 1.f / f[ht];
    const int64_t base = ((int64_t)b * a.Hq + h0 + 8 * ht) * a.ns + split * sub + part;
    if (tig == 0 && 8 * ht + gid < heads) a.ml[base + (int64_t)gid * a.ns] = make_float2(m[ht], l[ht]);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float y = __shfl_sync(0xffffffffu, inv, 8 * tig + 4 * e);
      if (8 * ht + 2 * tig + e >= heads) continue;
      float *to = a.o + (base + (int64_t)(2 * tig + e) * a.ns) * kD + 2 * gid;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        *reinterpret_cast<float2 *>(to + 16 * c) = make_float2(o[ht][c][e] * y, o[ht][c][2 + e] * y);
    }
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
  const int used = (n + a.chunk - 1) / a.chunk * a.per;
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
  int splits, chunk, per;  // CTAs along a list, entries of each, partials of each
  int nh, blocks;          // KV heads per CTA (mma.sync), query head blocks of a KV head
};
Decode8Plan plan_of(int dtype, int B, int Hq, int Hkv, int max_kv) {
  Decode8Plan p;
  const int grp = Hq / Hkv;
  int64_t ctas, want;
  int c, least;
  if (dtype == AKV_BF16) {
    const int tiles = grp <= 8 ? 1 : 2;
    p.blocks = (grp + 8 * tiles - 1) / (8 * tiles);
    p.nh = std::min(Hkv, kMWarps);
    p.per = kMWarps / p.nh;
    ctas = (int64_t)B * ((Hkv + p.nh - 1) / p.nh) * p.blocks;
    want = 4LL * 2 * sm_count();
    c = 2048 * p.per;
    least = kMKeys * p.per * 8;
  } else {
    p.blocks = (grp + kSHeads - 1) / kSHeads;
    p.nh = p.per = 1;
    ctas = (int64_t)B * Hkv * p.blocks;
    want = 4LL * 4 * sm_count();
    c = 4096;
    least = kSKeys;
  }
  const auto splits = [&](int x) { return std::max<int64_t>(1, ((int64_t)max_kv + x - 1) / x); };
  while (c / 2 >= least && ctas * splits(c) < want) c /= 2;
  while (splits(c) * p.per > kMaxSplit) c *= 2;
  p.splits = (int)splits(c);
  p.chunk = c;
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
  decode8_simt_kernel<float><<<dim3(p.splits, a.Hkv * p.blocks, a.B), kSThreads, smem, s>>>(a, th);
  return cudaGetLastError();
}

template <int kTiles>
cudaError_t launch_mma(const Decode8 &a, const Decode8Plan &p, const RopeTheta &th, cudaStream_t s) {
  const int smem = (int)sizeof(MmaSmem) + p.per * (kMRing * kMKeys * 4 + 2 * kMTable);
  const cudaError_t e = cudaFuncSetAttribute(decode8_mma_kernel<kTiles>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  decode8_mma_kernel<kTiles><<<dim3(p.splits, (a.Hkv + p.nh - 1) / p.nh * p.blocks, a.B), kMThreads, smem,
                               s>>>(a, th, p.nh, p.per);
  return cudaGetLastError();
}

}  // namespace

size_t decode_q8_workspace_bytes(int dtype, int B, int Hq, int Hkv, int max_kv) {
  const Decode8Plan p = plan_of(dtype, B, Hq, Hkv, max_kv);
  const size_t parts = (size_t)B * Hq * p.splits * p.per;
  return up256(parts * sizeof(float2)) + up256(parts * kD * sizeof(float));
}

cudaError_t launch_decode_q8(int dtype, int B, int Hq, int Hkv, const void *q, const int32_t *qpos,
                             const void *k_new, const void *v_new, const int32_t *new_slot,
                             const Kv8Pool &pool, const int32_t *indptr, const int32_t *indices,
                             const int32_t *kvpos, int max_kv, void *out, void *ws,
                             const RopeTheta &th, cudaStream_t s) {
  const Decode8Plan p = plan_of(dtype, B, Hq, Hkv, max_kv);
  const int ns = p.splits * p.per;
  const Decode8 a{B, Hq, Hkv, Hq / Hkv, q, qpos, k_new, v_new, new_slot, pool, indptr, indices, kvpos,
                  max_kv, (float2 *)ws,
                  (float *)((char *)ws + up256((size_t)B * Hq * ns * sizeof(float2))), ns, p.chunk, p.per};
  const cudaError_t e = dtype != AKV_BF16 ? launch_simt(a, p, th, s)
                        : a.grp <= 8      ? launch_mma<1>(a, p, th, s)
                                          : launch_mma<2>(a, p, th, s);
  if (e != cudaSuccess) return e;
  return dtype == AKV_BF16 ? launch_merge<__nv_bfloat16>(a, out, s) : launch_merge<float>(a, out, s);
}

}  // namespace akv
