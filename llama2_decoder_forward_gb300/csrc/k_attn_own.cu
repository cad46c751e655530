// Decode attention with capped or biased scores: the keys a sequence owns
// (from the shared prefix's end to its position), bf16, head_dim 128, and the
// merge with the prefix's partial results (k_attn_forms_tc.cu).
//
//   x = scale q.k;  s = (cap tanh(x / cap) or x) - slope (i - j);  softmax;  sum p v
//
// Bound by the K/V bytes: each key is read once, for all query heads of its
// group. One CTA per (key split, K/V head, sequence): a producer warp streams
// 64-key tiles (128-byte swizzled TMA boxes, L2 evict-first) into a 2-stage
// ring (with three CTAs per SM as many bytes in flight as 3 stages with two,
// and more warps to hide the consumers' latencies: 32 sequences of up to 1100
// keys, 32 heads, 36.4 -> 32.7 us); four consumer warps take 16 keys each and
// run S and P V on mma.sync, with an fp32 online softmax; the warps' (max, sum,
// O) merge in shared memory. Groups of up to 8 heads put the keys on the MMA's
// rows (S^T = K Q^T, O^T = V^T P^T), larger ones the heads. P is a bf16 pair
// (high part and remainder), free while memory bounds the kernel.
//
// More CTAs than are resident take the longest sequences first (128 sequences of
// 1 to 3500 keys over 16384 shared ones: 180 -> 168 us). Up to 8 key splits of a
// (K/V head, sequence) form a thread-block cluster and merge through distributed
// shared memory; more (few sequences with very long contexts) leave partials for
// a joining kernel. The splits share the keys that a sequence has, not those that
// the cache has room for (8 sequences of up to 4000 keys, 8 K/V heads: 18.7 ->
// 16.1 us). How many there are, and whether the longest start first, is chosen on
// the host, which knows the room and not the keys. One sequence, 466 keys, 32 K/V
// heads: 8.7 us unsplit, 5.9 us as clusters of 8, which it gets with room for up to
// 1024 keys; with room for 4096 and 32768 it is 7.6 and 7.7 us (8 K/V heads: 4.8,
// 6.7 and 7.0), and 256 sequences of 250 keys take 43.5, 62.5 and 62.9 us.
//
// Beside a prefix: the launch follows the prefix kernel's and starts on the SMs
// that it leaves free. That kernel lets it start only after its own wait, so
// whatever ran before the prefix kernel is complete; what is read here comes
// from L2 (TMA, .cg). After a long prefix every CTA leaves partials and goes, so
// that the next one can start (waiting for the prefix in each early CTA kept its
// SM idle); one CTA's producer waits for the prefix kernel, so that the joining
// kernel, which waits for this one, finds both kinds of partials. A short prefix
// is over before most CTAs are: they wait and merge, which saves the third launch
// (32 sequences over 500 shared keys: 32 us, with the joining kernel 36). 128
// sequences over 16384 shared keys: 154 us, 6.1 TB/s of keys and values.
#include <algorithm>
#include <climits>

#include "attn_score.cuh"
#include "internal.h"

namespace llgb {

namespace {

constexpr int HD = 128;
constexpr int SUB = 16;                         // keys of a warp's step
constexpr int TILE_K = 64;                      // keys of a stage
constexpr int STAGES = 2;
constexpr int OWN_THREADS = 160;                // 4 consumer warps + the producer
constexpr uint32_t SUB_HALF = SUB * 128;        // 16 keys x 64 dims
constexpr uint32_t HALF = TILE_K * 128;         // 64 keys x 64 dims: 8 KB
constexpr uint32_t STAGE = 4 * HALF;            // K and V, two dim halves each
constexpr int SORT_MAX = 256;                   // sequences that a CTA sorts
constexpr uint32_t OFF_SORT = STAGES * STAGE + 256;
constexpr size_t OWN_SMEM = OFF_SORT + (2 * SORT_MAX + 4) * 4 + 1024;
static_assert((4 * 16 * HD + 128) * 4 <= STAGES * STAGE, "the merge area aliases the ring");

struct OwnParams {
  const bf16* q;
  bf16* out;
  const int32_t *positions, *page_table;
  uint32_t* status;
  int n_q, n_kv, G, layer;
  int page_size, capacity, n_pages, max_pages, box_rows;
  int key_limit, first;        // keys from `first` on; position limit
  int base;                    // first rounded down to a tile
  int splits, min_share, cluster;  // a split has at least min_share keys
  int sorted;                  // sequences (B) to take longest first; 0: in order
  int prefix_parts;            // partials per row of the prefix kernel, at most
  const int* used;             // how many it wrote
  int join;                    // leave partials for the joining kernel
  float *part_o, *part_ml;     // [B n_q][prefix_parts][...]
  float *own_o, *own_ml;       // [B n_q][splits][...] (with a prefix, or splits > 1 without cluster)
  size_t rows, own_room;       // B n_q; partials behind the prefix's
  float scale, cap;
  const float* slopes;
};

__device__ __forceinline__ void consumers_bar() { asm volatile("bar.sync 2, 128;" ::: "memory"); }

// Keys of a split, a multiple of 64: the n - base that there are, shared evenly.
__device__ __forceinline__ int own_share(const OwnParams& p, int n) {
  if (p.splits == 1) return INT_MAX - p.base;
  const int keys = max(n - p.base, 1);
  return max(p.min_share, ((keys + p.splits - 1) / p.splits + 63) & ~63);
}
// Page id of key k0 of sequence b (-1: past its table), and the cache row there.
__device__ __forceinline__ int own_page(const OwnParams& p, int b, int k0) {
  const int pi = p.page_size == 0 ? 0 : k0 / p.page_size;
  return p.page_size != 0 && pi < p.max_pages ? __ldcg(p.page_table + (size_t)b * p.max_pages + pi) : -1;
}
__device__ __forceinline__ int own_kv_row(const OwnParams& p, int b, int g, int k0, int page) {
  if (p.page_size == 0) return (b * p.n_kv + g) * p.capacity + k0;
  const int pi = k0 / p.page_size;
  if (page < 0 || page >= p.n_pages) {
    flag(p.status, LLAMA_FLAG_PAGE_RANGE);
    return -64;
  }
  return (page * p.n_kv + g) * p.page_size + (k0 - pi * p.page_size);
}

// Scores in log2 units: cl tanh(y), cl = cap log2e, y = x yk with yk = scale / cap,
// or x c without a cap; the distance bias is subtracted later. Up to |y| = 1 tanh
// is the polynomial that the prefix kernel takes, beyond it 1 - 2 / (1 + e^2y):
// that difference has an error relative to the cap, which for caps far above the
// scores would swallow them (weights off by 4 % at a cap of 1e6).
struct ScoreConst {
  float c, cl, yk;
  bool cap;
  __device__ __forceinline__ ScoreConst(float scale, float cap_)
      : c(scale * 1.4426950408889634f), cl(cap_ * 1.4426950408889634f),
        yk(cap_ > 0.f ? scale / cap_ : 0.f), cap(cap_ > 0.f) {}
};
__device__ __forceinline__ float score(const ScoreConst& k, float x) {
  if (!k.cap) return x * k.c;
  constexpr float kTanh6[6] = {kTanh[7], kTanh[8], kTanh[9], kTanh[10], kTanh[11], kTanh[12]};
  const float y = x * k.yk, w = y * y;
  float q = kTanh6[5];
#pragma unroll
  for (int i = 4; i >= 0; --i) q = fmaf(q, w, kTanh6[i]);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2(y * 2.885390081777927f)));
  return k.cl * (fabsf(y) <= 1.f ? y * q : fmaf(-2.f, r, 1.f));
}

// Rows of a 16-key step outside [lead, valid) may hold anything: zero their V.
__device__ __forceinline__ void clean_v(uint8_t* v, int lead, int valid, int lane) {
  if (lead == 0 && valid == SUB) return;
  for (int i = lane; i < SUB * 16; i += 32) {
    const int row = i >> 4, half = (i >> 3) & 1, chunk = i & 7;
    if (row < lead || row >= valid)
      *reinterpret_cast<uint4*>(v + half * HALF + row * 128 + chunk * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// Groups of up to 8 heads: keys on the MMA rows. Lane l tracks heads 2(l%4)
// and 2(l%4) + 1. Leaves (max, sum, O) of this warp in shared memory.
__device__ __forceinline__ void consume_keys(const OwnParams& p, uint8_t* smem, uint64_t* full,
                                             uint64_t* empty, volatile uint32_t* stop, int b, int g,
                                             int kbeg, int kend, int pos, int warp, int lane) {
  const int G = p.G, hq = lane >> 2, hc = 2 * (lane & 3);
  uint32_t qf[8][2];  // Q^T fragments: head lane/4
  const bf16* qb = p.q + ((size_t)b * p.n_q + (size_t)g * G + hq) * HD;
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    const int col = kk * 16 + 2 * (lane & 3);
    qf[kk][0] = hq < G ? __ldcg(reinterpret_cast<const unsigned*>(qb + col)) : 0u;
    qf[kk][1] = hq < G ? __ldcg(reinterpret_cast<const unsigned*>(qb + col + 8)) : 0u;
  }
  constexpr float kLog2e = 1.4426950408889634f;
  const ScoreConst sc(p.scale, p.cap);
  float sl[2] = {0.f, 0.f};
  if (p.slopes) {
#pragma unroll
    for (int j = 0; j < 2; ++j) sl[j] = hc + j < G ? __ldcg(p.slopes + g * G + hc + j) * kLog2e : 0.f;
  }
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  const int mi = lane >> 3, rr = lane & 7;
  const int n_tiles = (kend - kbeg + TILE_K - 1) / TILE_K;
  int s = 0;
  uint32_t ph = 0;
  for (int t = 0; t < n_tiles; ++t) {
    if (*stop) break;
    if (!mbar_wait(&full[s], ph, p.status)) {
      *stop = 1;
      break;
    }
    const int k0 = kbeg + t * TILE_K + warp * SUB;
    const int lead = max(0, p.first - k0), valid = min(SUB, kend - k0);
    if (lead < valid) {
      uint8_t* st = smem + s * STAGE;
      const uint32_t kbase = smem_u32(st + warp * SUB_HALF);
      uint8_t* vptr = st + 2 * HALF + warp * SUB_HALF;
      clean_v(vptr, lead, valid, lane);
      const uint32_t vbase = smem_u32(vptr);
      float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {  // even and odd steps in separate chains
        const int row = ((mi & 1) << 3) + rr, chunk = (kk & 3) * 2 + (mi >> 1);
        uint32_t a[4];
        ldsm_x4(kbase + (kk >> 2) * HALF + swz128(row, chunk), a[0], a[1], a[2], a[3]);
        mma_bf16_16816((kk & 1) ? s1 : s0, a, qf[kk][0], qf[kk][1]);
      }
      float sv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = (lane >> 2) + (i >= 2 ? 8 : 0);
        float x = score(sc, s0[i] + s1[i]);
        if (p.slopes) x = fmaf(-sl[i & 1], (float)(pos - k0 - key), x);
        sv[i] = key >= lead && key < valid ? x : -INFINITY;
      }
      float corr[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float mx = fmaxf(sv[j], sv[j + 2]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        const float mn = fmaxf(m[j], mx);
        corr[j] = mn == m[j] ? 1.f : ex2(m[j] - mn);
        m[j] = mn;
      }
      float pv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) pv[i] = ex2(sv[i] - (m[i & 1] == -INFINITY ? 0.f : m[i & 1]));
      l[0] = l[0] * corr[0] + pv[0] + pv[2];
      l[1] = l[1] * corr[1] + pv[1] + pv[3];
      if (__any_sync(0xffffffffu, corr[0] != 1.f || corr[1] != 1.f)) {
#pragma unroll
        for (int d = 0; d < 8; ++d) {
          o[d][0] *= corr[0];
          o[d][1] *= corr[1];
          o[d][2] *= corr[0];
          o[d][3] *= corr[1];
        }
      }
      uint32_t p0h, p0l, p1h, p1l;
      split_pack(pv[0], pv[1], p0h, p0l);
      split_pack(pv[2], pv[3], p1h, p1l);
      const uint32_t bh0 = movmatrix_t(p0h), bh1 = movmatrix_t(p1h);
      const uint32_t bl0 = movmatrix_t(p0l), bl1 = movmatrix_t(p1l);
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        const int c16 = d * 2 + (mi & 1), row = ((mi >> 1) << 3) + rr;
        uint32_t a[4];
        ldsm_x4_t(vbase + (c16 >> 3) * HALF + swz128(row, c16 & 7), a[0], a[1], a[2], a[3]);
        mma_bf16_16816(o[d], a, bh0, bh1);
        mma_bf16_16816(o[d], a, bl0, bl1);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s]);
    if (++s == STAGES) {
      s = 0;
      ph ^= 1;
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    l[j] += __shfl_xor_sync(0xffffffffu, l[j], 4);
    l[j] += __shfl_xor_sync(0xffffffffu, l[j], 8);
    l[j] += __shfl_xor_sync(0xffffffffu, l[j], 16);
  }
  float* so = reinterpret_cast<float*>(smem);  // [4][16][128], then max [4][16], sum [4][16]
  float* sm = so + 4 * 16 * HD;
  consumers_bar();  // every consumer is done with the ring
#pragma unroll
  for (int d = 0; d < 8; ++d)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (hc + (i & 1) < G)
        so[(warp * 16 + hc + (i & 1)) * HD + d * 16 + (lane >> 2) + (i >= 2 ? 8 : 0)] = o[d][i];
  if (lane < 4) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (hc + j < G) {
        sm[warp * 16 + hc + j] = merge_max(m[j], l[j]);
        sm[64 + warp * 16 + hc + j] = l[j];
      }
  }
}

// Groups of 9 to 16 heads: heads on the MMA rows (zero-padded to 16).
__device__ __forceinline__ void consume_heads(const OwnParams& p, uint8_t* smem, uint64_t* full,
                                              uint64_t* empty, volatile uint32_t* stop, int b, int g,
                                              int kbeg, int kend, int pos, int warp, int lane) {
  const int G = p.G, r0 = lane >> 2;
  uint32_t qa[8][4];
  const bf16* qb = p.q + ((size_t)b * p.n_q + (size_t)g * G) * HD;
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = r0 + 8 * (i & 1), col = kk * 16 + 2 * (lane & 3) + 8 * (i >> 1);
      qa[kk][i] = row < G ? __ldcg(reinterpret_cast<const unsigned*>(qb + row * HD + col)) : 0u;
    }
  constexpr float kLog2e = 1.4426950408889634f;
  const ScoreConst sc(p.scale, p.cap);
  float sl[2] = {0.f, 0.f};
  if (p.slopes) {
#pragma unroll
    for (int j = 0; j < 2; ++j) sl[j] = r0 + 8 * j < G ? __ldcg(p.slopes + g * G + r0 + 8 * j) * kLog2e : 0.f;
  }
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[16][4];
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  const int mi = lane >> 3, rr = lane & 7;
  const int n_tiles = (kend - kbeg + TILE_K - 1) / TILE_K;
  int s = 0;
  uint32_t ph = 0;
  for (int t = 0; t < n_tiles; ++t) {
    if (*stop) break;
    if (!mbar_wait(&full[s], ph, p.status)) {
      *stop = 1;
      break;
    }
    const int k0 = kbeg + t * TILE_K + warp * SUB;
    const int lead = max(0, p.first - k0), valid = min(SUB, kend - k0);
    if (lead < valid) {
      uint8_t* st = smem + s * STAGE;
      const uint32_t kbase = smem_u32(st + warp * SUB_HALF);
      uint8_t* vptr = st + 2 * HALF + warp * SUB_HALF;
      clean_v(vptr, lead, valid, lane);
      const uint32_t vbase = smem_u32(vptr);
      float sv[2][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) sv[0][i] = sv[1][i] = 0.f;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const int chunk = (kk & 3) * 2 + (mi & 1), row = ((mi >> 1) << 3) + rr;
        uint32_t b0, b1, b2, b3;
        ldsm_x4(kbase + (kk >> 2) * HALF + swz128(row, chunk), b0, b1, b2, b3);
        mma_bf16_16816(sv[0], qa[kk], b0, b1);
        mma_bf16_16816(sv[1], qa[kk], b2, b3);
      }
      float mx[2] = {-INFINITY, -INFINITY}, corr[2], ps[2] = {0.f, 0.f};
#pragma unroll
      for (int nb = 0; nb < 2; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = nb * 8 + 2 * (lane & 3) + (i & 1);
          float x = score(sc, sv[nb][i]);
          if (p.slopes) x = fmaf(-sl[i >> 1], (float)(pos - k0 - key), x);
          sv[nb][i] = key >= lead && key < valid ? x : -INFINITY;
          mx[i >> 1] = fmaxf(mx[i >> 1], sv[nb][i]);
        }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
        const float mn = fmaxf(m[h], mx[h]);
        corr[h] = mn == m[h] ? 1.f : ex2(m[h] - mn);
        m[h] = mn;
      }
#pragma unroll
      for (int nb = 0; nb < 2; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = ex2(sv[nb][i] - (m[i >> 1] == -INFINITY ? 0.f : m[i >> 1]));
          sv[nb][i] = e;
          ps[i >> 1] += e;
        }
      l[0] = l[0] * corr[0] + ps[0];
      l[1] = l[1] * corr[1] + ps[1];
#pragma unroll
      for (int d = 0; d < 16; ++d) {
        o[d][0] *= corr[0];
        o[d][1] *= corr[0];
        o[d][2] *= corr[1];
        o[d][3] *= corr[1];
      }
      uint32_t pa[4], pl[4];
      split_pack(sv[0][0], sv[0][1], pa[0], pl[0]);
      split_pack(sv[0][2], sv[0][3], pa[1], pl[1]);
      split_pack(sv[1][0], sv[1][1], pa[2], pl[2]);
      split_pack(sv[1][2], sv[1][3], pa[3], pl[3]);
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        const int c16 = d * 2 + (mi >> 1), row = ((mi & 1) << 3) + rr;
        uint32_t b0, b1, b2, b3;
        ldsm_x4_t(vbase + (c16 >> 3) * HALF + swz128(row, c16 & 7), b0, b1, b2, b3);
        mma_bf16_16816(o[2 * d], pa, b0, b1);
        mma_bf16_16816(o[2 * d + 1], pa, b2, b3);
        mma_bf16_16816(o[2 * d], pl, b0, b1);
        mma_bf16_16816(o[2 * d + 1], pl, b2, b3);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s]);
    if (++s == STAGES) {
      s = 0;
      ph ^= 1;
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
  }
  float* so = reinterpret_cast<float*>(smem);
  float* sm = so + 4 * 16 * HD;
  consumers_bar();
#pragma unroll
  for (int d = 0; d < 16; ++d)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      so[(warp * 16 + r0 + (i >= 2 ? 8 : 0)) * HD + d * 8 + 2 * (lane & 3) + (i & 1)] = o[d][i];
  if ((lane & 3) == 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      sm[warp * 16 + r0 + 8 * h] = merge_max(m[h], l[h]);
      sm[64 + warp * 16 + r0 + 8 * h] = l[h];
    }
  }
}

// A row's running merge in one warp: maximum and sum (the same in every lane)
// and the output's dims 4 lane .. 4 lane + 3, unnormalised.
struct RowSum {
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  __device__ __forceinline__ void add(float f, const float4& v) {
    o.x = fmaf(v.x, f, o.x);
    o.y = fmaf(v.y, f, o.y);
    o.z = fmaf(v.z, f, o.z);
    o.w = fmaf(v.w, f, o.w);
  }
  __device__ __forceinline__ void scale_to(float mx) {
    const float f = m == -INFINITY ? 0.f : exp2f(m - mx);
    l *= f;
    o.x *= f;
    o.y *= f;
    o.z *= f;
    o.w *= f;
    m = mx;
  }
};

// The partials of a row: lane s holds part s's maximum and sum, so they take
// one load for 32 parts, and the first outputs are loaded beside them, before it
// is known how many of the `cap` parts there is room for are there.
template <int AHEAD>
struct Parts {
  const float4* o;
  const float2* ml;
  int cap;
  float2 x;
  float4 v[AHEAD];
  __device__ __forceinline__ void outputs(int s, int n, int lane) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (s + i < n) v[i] = __ldcg(o + (size_t)(s + i) * (HD / 4) + lane);
  }
  __device__ __forceinline__ void load(const float* po, const float* pml, size_t at, int room, int lane) {
    o = reinterpret_cast<const float4*>(po + at * HD);
    ml = reinterpret_cast<const float2*>(pml) + at;
    cap = room;
    x = make_float2(-INFINITY, 0.f);
    if (lane < cap) x = __ldcg(ml + lane);
    outputs(0, cap, lane);
  }
  // adds the first `parts` of them to r, in their order
  __device__ __forceinline__ void fold(int parts, int lane, RowSum& r) {
    for (int s0 = 0; s0 < parts; s0 += 32) {
      const int k = min(32, parts - s0);
      if (s0 > 0) {
        if (lane < k) x = __ldcg(ml + s0 + lane);
        outputs(s0, s0 + k, lane);
      }
      if (lane >= k) x = make_float2(-INFINITY, 0.f);
      float mx = x.x;
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      mx = fmaxf(mx, r.m);
      if (mx == -INFINITY) continue;
      r.scale_to(mx);
      const float f = x.x == -INFINITY ? 0.f : exp2f(x.x - mx);
      float ls = f == 0.f ? 0.f : x.y * f;
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, w);
      r.l += ls;
      for (int s = 0; s < k; s += AHEAD) {
        if (s > 0) outputs(s0 + s, s0 + k, lane);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
          const float fs = __shfl_sync(0xffffffffu, f, (s + i) & 31);
          // a part without keys may hold anything: its O was not written
          if (s + i < k && fs != 0.f) r.add(fs, v[i]);
        }
      }
    }
  }
};

__device__ __forceinline__ void store_row(bf16* dst, int lane, const RowSum& r) {
  const float i = r.l > 0.f || r.l != r.l ? 1.f / r.l : 0.f;
  reinterpret_cast<uint2*>(dst)[lane] =
      make_uint2(pack_bf16(r.o.x * i, r.o.y * i), pack_bf16(r.o.z * i, r.o.w * i));
}

template <bool KEYS>
__global__ void __launch_bounds__(OWN_THREADS, KEYS ? 3 : 2)
    attn_own_kernel(const __grid_constant__ CUtensorMap mapK,
                    const __grid_constant__ CUtensorMap mapV,
                    const __grid_constant__ CUtensorMap mapK16,
                    const __grid_constant__ CUtensorMap mapV16, OwnParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * STAGE);
  uint64_t* empty = full + STAGES;
  volatile uint32_t* stop = reinterpret_cast<volatile uint32_t*>(empty + STAGES);
  const int split = blockIdx.x, g = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // With a prefix kernel before this one, what this one reads is complete: that
  // kernel waited for it. One CTA's producer waits for the prefix kernel itself,
  // so that whoever waits for this kernel has waited for both.
  const bool prefix = p.prefix_parts != 0;
  const bool waits = prefix && split == p.splits - 1 && g == p.n_kv - 1 && blockIdx.z == gridDim.z - 1;
  if (!prefix) grid_dep_wait();
  grid_dep_launch();
  if (!bc_smem(smem, (uint32_t)(OWN_SMEM - 1024), 1024, threadIdx.x == 0 ? p.status : nullptr)) {
    if (waits) grid_dep_wait();
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 4);
    }
    *stop = 0;
    fence_mbar_init();
  }
  if (warp == 4 && lane == 0) {
    tma_prefetch_desc(&mapK);
    tma_prefetch_desc(&mapV);
    tma_prefetch_desc(&mapK16);
    tma_prefetch_desc(&mapV16);
  }
  int b = blockIdx.z, pos;
  if (p.sorted) {
    // the blockIdx.z-th longest sequence, so that the longest start first: one key
    // of 32 bits per sequence, its length and (ties) its number
    int* key = reinterpret_cast<int*>(smem + OFF_SORT);
    int* at = key + SORT_MAX;
    for (int i = threadIdx.x; i < SORT_MAX; i += OWN_THREADS) {
      const int x = i < p.sorted ? __ldcg(p.positions + i) : -1;
      at[i] = x;
      key[i] = i < p.sorted ? (key_position(x, p.key_limit) + 1) * SORT_MAX + SORT_MAX - 1 - i : -1;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.sorted; i += OWN_THREADS) {
      const int mine = key[i];
      int rank = 0;
#pragma unroll 4
      for (int j = 0; j < p.sorted; j += 4) {
        const int4 x = *reinterpret_cast<const int4*>(key + j);
        rank += (x.x > mine) + (x.y > mine) + (x.z > mine) + (x.w > mine);
      }
      if (rank == b) at[SORT_MAX] = i;
    }
    __syncthreads();
    b = at[SORT_MAX];
    pos = at[b];
  } else {
    pos = __ldcg(p.positions + b);
  }
  // the producer's first page ids, without splits loaded beside the position
  int page = warp == 4 && p.splits == 1 ? own_page(p, b, p.base + lane * SUB) : 0;
  if (!p.sorted) __syncthreads();
  if ((pos < 0 || pos >= p.key_limit) && split == 0 && threadIdx.x == 0) flag(p.status, LLAMA_FLAG_POS_RANGE);
  pos = key_position(pos, p.key_limit);
  const int n = pos + 1;
  const int share = own_share(p, n), kbeg = p.base + split * share;
  const int kend = min(n, kbeg + share);
  const bool any = kend > max(kbeg, p.first);
  if (any) {
    const int n_tiles = (kend - kbeg + TILE_K - 1) / TILE_K;
    if (warp == 4) {  // ------------------------------------------------ producer
      // The whole warp: lane i looks up the cache row of 16-key step i of the
      // next 32 (one load for their page ids), and lanes 0-15 issue a tile's
      // sixteen small boxes together.
      const uint64_t pol = l2_policy_evict_first();  // own keys are streamed once
      const int n_steps = (kend - kbeg + SUB - 1) / SUB, first_step = max(0, p.first - kbeg) / SUB;
      int s = 0, issued = 0, rows = 0;
      uint32_t ph = 1;
      for (int t = 0; t < n_tiles; ++t) {
        if ((t & 7) == 0) {
          const int step = 4 * t + lane;
          if ((t > 0 || p.splits > 1) && step < n_steps) page = own_page(p, b, kbeg + step * SUB);
          rows = step >= first_step && step < n_steps ? own_kv_row(p, b, g, kbeg + step * SUB, page) : 0;
        }
        const bool go = !*stop && mbar_wait(&empty[s], ph, p.status);
        if (!__all_sync(0xffffffffu, go)) {
          *stop = 1;
          break;
        }
        const int j0 = max(0, first_step - 4 * t), j1 = min(TILE_K / SUB, n_steps - 4 * t);
        uint8_t* st = smem + s * STAGE;
        const bool whole = p.box_rows == TILE_K && j0 == 0 && j1 == TILE_K / SUB;
        if (lane == 0)
          mbar_arrive_expect_tx(&full[s], whole ? STAGE : (uint32_t)(j1 - j0) * 4 * SUB_HALF);
        // lane = 4 * step + (K low dims, K high, V low, V high)
        const int j = lane >> 2, part = lane & 3;
        const int row = __shfl_sync(0xffffffffu, rows, (4 * (t & 7) + j) & 31);
        uint8_t* d = st + part * HALF + j * SUB_HALF;
        if (whole ? j == 0 : j >= j0 && j < j1) {
          const CUtensorMap* m = whole ? (part < 2 ? &mapK : &mapV) : (part < 2 ? &mapK16 : &mapV16);
          tma_load_3d_hint(d, m, &full[s], 64 * (part & 1), row, p.layer, pol);
        }
        ++issued;
        if (++s == STAGES) {
          s = 0;
          ph ^= 1;
        }
      }
      // no copy in flight when the CTA exits, whoever gave up
      for (int t = max(0, issued - STAGES); t < issued; ++t)
        mbar_wait(&full[t % STAGES], (t / STAGES) & 1, p.status);
      if (waits) grid_dep_wait();
      return;
    }
    if (KEYS)
      consume_keys(p, smem, full, empty, stop, b, g, kbeg, kend, pos, warp, lane);
    else
      consume_heads(p, smem, full, empty, stop, b, g, kbeg, kend, pos, warp, lane);
    consumers_bar();
    if (*stop && !p.cluster) return;
  } else if (warp == 4) {  // (a cluster's barriers do not count threads that left)
    if (waits) grid_dep_wait();
    return;
  }
  if (!any && p.join) return;  // the joining kernel skips this split
  int parts = 0;
  if (prefix && !p.join) {
    grid_dep_wait();
    parts = __ldcg(p.used);
    if (!bc_ok(parts <= p.prefix_parts, p.status)) parts = 0;
  }
  const float* so = reinterpret_cast<const float*>(smem);
  const float* sm = so + 4 * 16 * HD;
  // a cluster's rows: [16][128] outputs, then maximum and sum [16][2]
  float* mine = reinterpret_cast<float*>(smem) + 4 * 16 * HD + 128;
  static_assert((4 * 16 * HD + 128 + 16 * (HD + 2)) * 4 <= STAGES * STAGE, "the cluster's rows fit the ring");
  for (int r = warp; r < p.G; r += 4) {  // a warp per row
    RowSum x;
    if (any && !*stop) {
      float mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < 4; ++w) mx = fmaxf(mx, sm[w * 16 + r]);
      if (mx != -INFINITY) {
        x.m = mx;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float mw = sm[w * 16 + r];
          const float f = mw == -INFINITY ? 0.f : exp2f(mw - mx);
          x.l = fmaf(sm[64 + w * 16 + r], f, x.l);
          x.add(f, reinterpret_cast<const float4*>(so + (w * 16 + r) * HD)[lane]);
        }
      }
    }
    const size_t bh = (size_t)b * p.n_q + (size_t)g * p.G + r;
    if (!bc_ok(bh < p.rows && (!p.join || bh * p.splits + split < p.own_room), p.status)) continue;
    if (p.cluster) {
      reinterpret_cast<float4*>(mine + r * HD)[lane] = x.o;
      if (lane == 0) *reinterpret_cast<float2*>(mine + 16 * HD + 2 * r) = make_float2(x.m, x.l);
    } else if (!p.join) {
      Parts<8> pre;
      pre.load(p.part_o, p.part_ml, bh * p.prefix_parts, parts, lane);
      pre.fold(parts, lane, x);
      store_row(p.out + bh * HD, lane, x);
    } else {
      const size_t at = bh * p.splits + split;
      reinterpret_cast<float4*>(p.own_o + at * HD)[lane] = x.o;
      if (lane == 0) *reinterpret_cast<float2*>(p.own_ml + 2 * at) = make_float2(x.m, x.l);
    }
  }
  if (!p.cluster) return;
  cluster_sync_all();
  // row r is folded by CTA r % splits of the cluster, in the order of the splits
  for (int i = warp; i * p.splits + split < p.G; i += 4) {
    const int r = i * p.splits + split;
    const uint32_t ro = smem_u32(mine + r * HD) + 16 * lane, rm = smem_u32(mine + 16 * HD + 2 * r);
    float2 ml = make_float2(-INFINITY, 0.f);
    if (lane < p.splits) ml = dsmem_ld2(dsmem_addr(rm, lane));
    float mx = ml.x;
#pragma unroll
    for (int w = 4; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
    mx = __shfl_sync(0xffffffffu, mx, 0);
    RowSum x;
    if (mx != -INFINITY) {
      x.m = mx;
      const float f = ml.x == -INFINITY ? 0.f : exp2f(ml.x - mx);
#pragma unroll 8
      for (int q = 0; q < p.splits; ++q) {
        const float fq = __shfl_sync(0xffffffffu, f, q);
        x.l = fmaf(__shfl_sync(0xffffffffu, ml.y, q), fq, x.l);
        x.add(fq, dsmem_ld4(dsmem_addr(ro, q)));
      }
    }
    const size_t bh = (size_t)b * p.n_q + (size_t)g * p.G + r;
    Parts<8> pre;
    pre.load(p.part_o, p.part_ml, bh * p.prefix_parts, parts, lane);
    pre.fold(parts, lane, x);
    store_row(p.out + bh * HD, lane, x);
  }
  cluster_sync_all();  // nobody leaves while its rows are read
}

// Joins a row's prefix partials and own splits, one warp per (sequence, head).
__global__ void __launch_bounds__(128, 7) attn_own_join_kernel(OwnParams p, int rows) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, bh = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (bh >= rows) return;
  Parts<8> pre;
  Parts<2> own;
  pre.load(p.part_o, p.part_ml, (size_t)bh * p.prefix_parts, p.prefix_parts, lane);
  own.load(p.own_o, p.own_ml, (size_t)bh * p.splits, p.splits, lane);
  int parts = p.prefix_parts ? __ldcg(p.used) : 0;
  if (!bc_ok(parts <= p.prefix_parts && (size_t)rows * p.splits <= p.own_room, p.status)) return;
  const int n = key_position(__ldcg(p.positions + bh / p.n_q), p.key_limit) + 1;
  int used = n > p.first;  // own splits that have keys
  if (used && p.splits > 1) {
    const int share = own_share(p, n);
    used = (n - p.base + share - 1) / share;
    if (!bc_ok(used <= p.splits, p.status)) return;
  }
  RowSum x;
  pre.fold(parts, lane, x);
  own.fold(used, lane, x);
  store_row(p.out + (size_t)bh * HD, lane, x);
}

}  // namespace

cudaError_t attn_own_prepare() {
  cudaError_t e = cudaFuncSetAttribute(attn_own_kernel<true>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)OWN_SMEM);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(attn_own_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)OWN_SMEM);
  return e;
}

SharedPlan shared_plan(int B, int n_q, int n_kv, int key_limit, int shared_len, int sm_count) {
  SharedPlan s{};
  const int G = n_q / n_kv;
  // prefix: one CTA per SM, each with its share of the key tiles
  s.rows_seq = 128 / G;
  s.alternate = B <= s.rows_seq;
  s.row_blocks = s.alternate ? 1 : (B + 2 * s.rows_seq - 1) / (2 * s.rows_seq);
  const int tiles = (shared_len + 127) / 128;
  if (tiles > 0) {
    const int want = std::max(1, sm_count / (n_kv * s.row_blocks));
    s.tiles_per_split = (tiles + want - 1) / want;
    s.prefix_splits = (tiles + s.tiles_per_split - 1) / s.tiles_per_split;
    s.prefix_parts = s.prefix_splits * (s.alternate ? 2 : 1);
  }
  // own keys: split while two CTAs per SM are not reached and a split keeps 64
  // keys (one tile); where a cluster's 8 CTAs do not reach them, as many as are
  // resident, with 256 keys (their partials are read again)
  s.base = shared_len / 64 * 64;
  const int keys = std::max(1, key_limit - s.base), pairs = B * n_kv;
  int k = 1;
  while (pairs * k < 2 * sm_count && k < 8 && keys / (2 * k) >= 64) k *= 2;
  if (k == 8 && pairs * k < 2 * sm_count) k = std::max(k, std::min({128, 3 * sm_count / pairs, keys / 256}));
  s.keys = keys;
  s.own_splits = k;
  s.min_share = k > 8 ? 256 : 64;
  // A long prefix: own CTAs that started beside it leave partials for a joining
  // kernel, so that others can follow on their SMs. A short one (4 turns): they
  // wait for it and merge.
  const int turns = s.alternate ? (s.tiles_per_split + 1) / 2 : s.tiles_per_split;
  s.join = k > 8 || turns > 4;
  s.cluster = k > 1 && !s.join;
  const size_t rows = (size_t)B * n_q;
  s.partials = rows * s.prefix_parts + (s.join ? rows * s.own_splits : 0);
  return s;
}

size_t shared_partial_bytes(int max_batch, int n_q, int n_kv, int max_seq, int sm_count) {
  // shared_plan's partials over every batch up to max_batch and every prefix:
  // prefix parts are at most 256 rows a CTA at one CTA per SM, or two per row;
  // own splits stay below 4 CTAs per SM
  const size_t rows = (size_t)max_batch * n_q, G = n_q / n_kv;
  const size_t tiles = (size_t)(max_seq + 127) / 128;
  const size_t prefix = std::max(2 * rows, std::min<size_t>(256 * (size_t)sm_count, rows * 2 * tiles));
  const size_t own = std::max(rows, std::min<size_t>(4 * (size_t)sm_count * G, rows * 128));
  return (prefix + own) * (HD + 2) * sizeof(float) + 16;
}

cudaError_t launch_shared_own(const SharedArgs& a, const SharedPlan& s, cudaStream_t st) {
  OwnParams p{};
  p.q = (const bf16*)a.q;
  p.out = (bf16*)a.out;
  p.positions = a.positions;
  p.page_table = a.page_table;
  p.status = a.status;
  p.n_q = a.n_q;
  p.n_kv = a.n_kv;
  p.G = a.n_q / a.n_kv;
  p.layer = a.layer;
  p.page_size = a.page_size;
  p.capacity = a.capacity;
  p.n_pages = a.n_pages;
  p.max_pages = a.max_pages;
  p.box_rows = a.box_rows;
  p.key_limit = a.key_limit;
  p.first = a.shared_len;
  p.base = s.base;
  p.splits = s.own_splits;
  p.min_share = s.min_share;
  p.prefix_parts = s.prefix_parts;
  p.cluster = s.cluster;
  p.join = s.join;
  p.used = reinterpret_cast<const int*>(a.partial + s.partials * (HD + 2));
  // Longest first where there are more CTAs than resident ones, unless they are too
  // short for it: each CTA looks at all positions. Sorted and in order, 8 K/V heads:
  // 128 sequences of up to 512 keys 21.5 and 19.5 us, 256 of up to 1024 73 and 54 us,
  // 200 of up to 2000 78 and 82 us; 128 of up to 3500 (and a prefix) 168 and 180 us.
  const bool waves = s.own_splits * a.n_kv * a.B > 3 * a.sm_count;
  p.sorted = waves && a.B > 1 && a.B <= SORT_MAX && s.keys / s.own_splits > 7 * a.B &&
                     a.key_limit < INT_MAX / SORT_MAX
                 ? a.B
                 : 0;
  const size_t rows = (size_t)a.B * a.n_q;
  p.part_o = a.partial;
  p.part_ml = p.part_o + s.partials * HD;
  p.rows = rows;
  p.own_room = s.partials - rows * s.prefix_parts;
  p.own_o = p.part_o + rows * s.prefix_parts * HD;
  p.own_ml = p.part_ml + rows * s.prefix_parts * 2;
  p.scale = a.sc.scale;
  p.cap = a.sc.cap;
  p.slopes = a.sc.slopes;
  const dim3 grid(s.own_splits, a.n_kv, a.B), block(OWN_THREADS);
  const dim3 cluster(s.cluster ? s.own_splits : 0, 1, 1);
  const cudaError_t e =
      p.G <= 8 ? launch_kc(attn_own_kernel<true>, grid, block, OWN_SMEM, st, cluster, *a.map_k,
                           *a.map_v, *a.map_k16, *a.map_v16, p)
               : launch_kc(attn_own_kernel<false>, grid, block, OWN_SMEM, st, cluster, *a.map_k,
                           *a.map_v, *a.map_k16, *a.map_v16, p);
  if (e != cudaSuccess || !s.join) return e;
  return launch_k(attn_own_join_kernel, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, st, 0, p,
                  (int)rows);
}

}  // namespace llgb
