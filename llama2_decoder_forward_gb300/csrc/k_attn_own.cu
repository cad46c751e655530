// Decode attention with capped or biased scores: the keys a sequence owns
// (from the shared prefix's end to its position), bf16, head_dim 128, and the
// merge with the prefix's partial results (k_attn_forms_tc.cu). The same kernel adds up
// how much each key weighs, and takes trees of few rows.
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
constexpr int TREE_COUNTED = 128;               // sequences whose blocks of tree rows a CTA counts
constexpr uint32_t OFF_SORT = STAGES * STAGE + 256;
constexpr uint32_t OFF_KEEP = OFF_SORT + (2 * SORT_MAX + 4) * 4;  // key weights: scores, in the kernel that adds them up
constexpr size_t OWN_SMEM = OFF_KEEP + 1024;
constexpr size_t OWN_SMEM_MOST = kOwnSmemMost;
static_assert(OWN_SMEM == kOwnSmem && HD == kPlanHeadDim, "what the plans count on");
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
  // key weights: every score (log2 units), [B][n_q][ld], for the joining kernel
  float* scores;
  float* weights;              // [B][n_kv][ld]
  int64_t ld;
  int keep;                    // room for so many of a row's scores in shared memory, the weights added here; 0: above
  // small trees: a sequence's rows in blocks of 2^tree_shift
  const int32_t *cu_rows, *start_pos, *row_pos;
  TreeMask tree;
  int n_rows, n_seq, tree_shift, slices, per;  // a group's heads in slices of `per`
};

// What a launch works on: a decode row per sequence; the same with its scores kept; the
// rows of small trees.
enum { ODecode, OWeigh, OTree };

// The rows of a CTA: the query heads of one K/V head, of one decode row or of several
// tree rows (row r: head r % per of the slice, of tree row i0 + r / per).
struct OwnRows {
  int b, g, count;             // sequence, K/V head, rows
  int pos;                     // decode: the row's position
  int lo, i0, start, there;    // trees: the sequence's first row, the block's, cached keys, tree rows in the cache
  int head;                    // and the first query head
};
// Where the scores are kept: row r's of key k at at[r ld + k - first].
struct OwnKeep {
  float* at;
  int64_t ld;
  int first;
};
// Which (row, query head) of q and the output row r is.
template <int MODE>
__device__ __forceinline__ size_t row_head(const OwnParams& p, const OwnRows& R, int r) {
  if (MODE != OTree) return (size_t)R.b * p.n_q + (size_t)R.g * p.G + r;
  const int i = r / p.per;
  return (size_t)(R.lo + R.i0 + i) * p.n_q + R.head + (r - i * p.per);
}
template <int MODE>
__device__ __forceinline__ float row_slope(const OwnParams& p, const OwnRows& R, int r) {
  return r < R.count ? __ldcg(p.slopes + (MODE == OTree ? R.head + r % p.per : R.g * p.G + r)) * 1.4426950408889634f : 0.f;
}
// Trees: the position of row r, of key k (n keys in all), and the visible ones of 32 keys from k on.
__device__ __forceinline__ int tree_pos(const OwnParams& p, const OwnRows& R, int x) {
  return p.row_pos ? min(max(__ldcg(p.row_pos + R.lo + x), 0), kMaxPos) : R.start + x;
}
__device__ __forceinline__ int tree_key_pos(const OwnParams& p, const OwnRows& R, int k) {
  return k < R.start || k - R.start >= R.there ? k : tree_pos(p, R, k - R.start);
}
__device__ __forceinline__ uint32_t row_sees(const OwnParams& p, const OwnRows& R, int r, int k) {
  const int i = R.i0 + r / p.per;
  return r < R.count ? tree_bits(p.tree, (size_t)R.lo + i, i, R.there, k - R.start) : 0u;
}

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

// Up to 8 rows: keys on the MMA rows. Lane l tracks rows 2(l%4) and 2(l%4) + 1. Leaves
// (max, sum, O) of this warp in shared memory.
template <int MODE>
__device__ __forceinline__ void consume_keys(const OwnParams& p, uint8_t* smem, uint64_t* full,
                                             uint64_t* empty, volatile uint32_t* stop, const OwnRows& R, const OwnKeep& keep,
                                             int kbeg, int kend, int warp, int lane) {
  const int G = R.count, hq = lane >> 2, hc = 2 * (lane & 3);
  uint32_t qf[8][2];  // Q^T fragments: head lane/4
  const bf16* qb = p.q + row_head<MODE>(p, R, hq) * HD;
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    const int col = kk * 16 + 2 * (lane & 3);
    qf[kk][0] = hq < G ? __ldcg(reinterpret_cast<const unsigned*>(qb + col)) : 0u;
    qf[kk][1] = hq < G ? __ldcg(reinterpret_cast<const unsigned*>(qb + col + 8)) : 0u;
  }
  const ScoreConst sc(p.scale, p.cap);
  float sl[2] = {0.f, 0.f};
  if (p.slopes) {
#pragma unroll
    for (int j = 0; j < 2; ++j) sl[j] = row_slope<MODE>(p, R, hc + j);
  }
  int pos[2] = {0, 0};  // trees: the two rows' positions, for the bias
  if (MODE == OTree && p.slopes) {
#pragma unroll
    for (int j = 0; j < 2; ++j) pos[j] = hc + j < G ? tree_pos(p, R, R.i0 + (hc + j) / p.per) : 0;
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
      uint32_t sees[2] = {~0u, ~0u};  // trees: the keys that the two rows see
      if (MODE == OTree && k0 + SUB > R.start) {
        sees[0] = row_sees(p, R, hc, k0);
        sees[1] = row_sees(p, R, hc + 1, k0);
      }
      float sv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = (lane >> 2) + (i >= 2 ? 8 : 0);
        float x = score(sc, s0[i] + s1[i]);
        if (p.slopes)
          x = fmaf(-sl[i & 1], MODE == OTree ? fabsf((float)(pos[i & 1] - tree_key_pos(p, R, k0 + key)))
                                             : (float)(R.pos - k0 - key), x);
        sv[i] = key >= lead && key < valid && (MODE != OTree || (sees[i & 1] >> key & 1u)) ? x : -INFINITY;
        if (MODE == OWeigh && key < valid && hc + (i & 1) < G)
          keep.at[(hc + (i & 1)) * keep.ld + (k0 + key - keep.first)] = x;
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
template <int MODE>
__device__ __forceinline__ void consume_heads(const OwnParams& p, uint8_t* smem, uint64_t* full,
                                              uint64_t* empty, volatile uint32_t* stop, const OwnRows& R, const OwnKeep& keep,
                                              int kbeg, int kend, int warp, int lane) {
  const int G = R.count, r0 = lane >> 2;
  uint32_t qa[8][4];
  const bf16* qb = p.q + row_head<MODE>(p, R, 0) * HD;
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = r0 + 8 * (i & 1), col = kk * 16 + 2 * (lane & 3) + 8 * (i >> 1);
      qa[kk][i] = row < G ? __ldcg(reinterpret_cast<const unsigned*>(qb + row * HD + col)) : 0u;
    }
  const ScoreConst sc(p.scale, p.cap);
  float sl[2] = {0.f, 0.f};
  if (p.slopes) {
#pragma unroll
    for (int j = 0; j < 2; ++j) sl[j] = row_slope<MODE>(p, R, r0 + 8 * j);
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
          if (p.slopes) x = fmaf(-sl[i >> 1], (float)(R.pos - k0 - key), x);
          sv[nb][i] = key >= lead && key < valid ? x : -INFINITY;
          if (MODE == OWeigh && key < valid && r0 + 8 * (i >> 1) < G)
            keep.at[(r0 + 8 * (i >> 1)) * keep.ld + (k0 + key - keep.first)] = x;
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

// Small trees: which block of 2^tree_shift rows CTA z has, for a whole warp; false: none. Few
// sequences' blocks are counted, so that CTAs to spare come last (64 sequences of 13 rows, 32
// heads, 1000 keys 141 us, searched 148). Among many sequence b's begin with CTA
// cu_rows[b] / 2^tree_shift + b, which leaves room for each and one CTA or none to spare, and
// a lookup goes 32 ways (256 sequences of a row, 32 heads, 512 keys: counted 192 us, searched 179;
// 512 sequences, 64 / 8 heads, 256 keys 145 and 92).
__device__ __forceinline__ bool tree_block(const OwnParams& p, int z, int lane, int& b, int& i0, int& lo, int& n) {
  if (p.n_seq > TREE_COUNTED) {
    auto begin = [&](int i) { return (min(max(p.cu_rows[i], 0), p.n_rows) >> p.tree_shift) + i; };
    b = 0;
    for (int len = p.n_seq; len > 1;) {
      const int step = (len + 31) / 32, i = lane * step;
      const uint32_t m = __ballot_sync(0xffffffffu, i < len && begin(b + i) <= z);
      const int w = m ? 31 - __clz(m) : 0;
      b += w * step;
      len = min(step, len - w * step);
    }
    doc_rows(p.cu_rows, b, p.n_rows, nullptr, lo, n);
    i0 = (z - begin(b)) << p.tree_shift;
    return i0 >= 0 && i0 < n;
  }
  for (int b0 = 0; b0 < p.n_seq; b0 += 32) {
    int my_lo = 0, my_n = 0;
    if (b0 + lane < p.n_seq) doc_rows(p.cu_rows, b0 + lane, p.n_rows, nullptr, my_lo, my_n);
    const int blocks = (my_n + (1 << p.tree_shift) - 1) >> p.tree_shift;
    int upto = blocks;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    const uint32_t m = __ballot_sync(0xffffffffu, z < upto);
    if (m) {
      const int w = __ffs(m) - 1;
      b = b0 + w;
      i0 = (z - __shfl_sync(0xffffffffu, upto - blocks, w)) << p.tree_shift;
      lo = __shfl_sync(0xffffffffu, my_lo, w);
      n = __shfl_sync(0xffffffffu, my_n, w);
      return true;
    }
    z -= __shfl_sync(0xffffffffu, upto, 31);
  }
  return false;
}

// The sequence of a packed row, for a whole warp, or -1.
__device__ __forceinline__ int tree_sequence(const OwnParams& p, int row, int lane) {
  for (int b0 = 0; b0 < p.n_seq; b0 += 32) {
    int lo = 0, n = 0;
    if (b0 + lane < p.n_seq) doc_rows(p.cu_rows, b0 + lane, p.n_rows, nullptr, lo, n);
    const uint32_t m = __ballot_sync(0xffffffffu, row >= lo && row < lo + n);
    if (m) return b0 + __ffs(m) - 1;
  }
  return -1;
}
// Keys of sequence b, and what its rows need of them.
__device__ __forceinline__ int tree_keys(const OwnParams& p, int b, OwnRows& R) {
  int lo, n;
  doc_rows(p.cu_rows, b, p.n_rows, nullptr, lo, n);
  const int start = p.start_pos[b];
  const long long end = (long long)start + n;
  const int keys = start < 0 ? 0 : (int)(end < p.key_limit ? end : p.key_limit);
  R.start = start < 0 ? 0 : min(start, keys);
  R.there = keys - R.start;
  return keys;
}

template <bool KEYS, int MODE>
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
  const int split = blockIdx.x, g = MODE == OTree ? blockIdx.y / p.slices : blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  OwnRows R{};
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
  if (MODE == OTree) {
    int n;
    if ((blockIdx.x | blockIdx.y | blockIdx.z) == 0 && warp == 0)  // bad bounds are flagged once
      for (int i = lane, x, y; i < p.n_seq; i += 32) doc_rows(p.cu_rows, i, p.n_rows, p.status, x, y);
    if (!tree_block(p, blockIdx.z, lane, b, R.i0, R.lo, n)) return;  // a cluster's CTAs all do
    pos = tree_keys(p, b, R) - 1;  // the last key
    if ((p.start_pos[b] < 0 || R.there < n) && split == 0 && threadIdx.x == 0) flag(p.status, LLAMA_FLAG_POS_RANGE);
    const int h = (blockIdx.y - g * p.slices) * p.per;
    R.head = g * p.G + h;
    R.count = min(1 << p.tree_shift, n - R.i0) * min(p.per, p.G - h);
  } else if (p.sorted) {
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
  if (MODE != OTree) {
    if ((pos < 0 || pos >= p.key_limit) && split == 0 && threadIdx.x == 0) flag(p.status, LLAMA_FLAG_POS_RANGE);
    pos = key_position(pos, p.key_limit);
    R.count = p.G;
  }
  R.b = b;
  R.g = g;
  R.pos = pos;
  const int n = pos + 1;
  const int share = own_share(p, n), kbeg = p.base + split * share;
  const int kend = min(n, kbeg + share);
  const bool any = kend > max(kbeg, p.first);
  OwnKeep keep{};
  if (MODE == OWeigh) {
    if (p.keep)
      keep = OwnKeep{reinterpret_cast<float*>(smem + OFF_KEEP), p.keep, kbeg};
    else
      keep = OwnKeep{p.scores + row_head<MODE>(p, R, 0) * p.ld, p.ld, 0};
    if (!bc_ok(!any || kend - keep.first <= keep.ld, p.status)) return;
  }
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
      consume_keys<MODE>(p, smem, full, empty, stop, R, keep, kbeg, kend, warp, lane);
    else
      consume_heads<MODE>(p, smem, full, empty, stop, R, keep, kbeg, kend, warp, lane);
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
  // key weights added here: the rows' maxima and reciprocal sums, and the first keys' old weights
  float2* stat = reinterpret_cast<float2*>(smem + OFF_SORT);
  constexpr int OLD = 4;
  float old[OLD];
  float* w = MODE == OWeigh ? p.weights + ((size_t)b * p.n_kv + g) * p.ld : nullptr;
  if (MODE == OWeigh && p.keep) {
#pragma unroll
    for (int q = 0; q < OLD; ++q)
      if (kbeg + (int)threadIdx.x + 128 * q < kend) old[q] = w[kbeg + threadIdx.x + 128 * q];
  }
  for (int r = warp; r < R.count; r += 4) {  // a warp per row
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
    const size_t bh = row_head<MODE>(p, R, r);
    if (!bc_ok(bh < p.rows && (!p.join || bh * p.splits + split < p.own_room), p.status)) continue;
    if (MODE == OWeigh && p.keep && lane == 0)
      stat[r] = make_float2(x.m == -INFINITY ? 0.f : x.m, x.l > 0.f || x.l != x.l ? 1.f / x.l : 0.f);
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
  if (MODE == OWeigh && p.keep) {
    consumers_bar();  // `stat`
    if (*stop) return;
    for (int q = 0; kbeg + (int)threadIdx.x + 128 * q < kend; ++q) {
      const int i = kbeg + threadIdx.x + 128 * q;
      float sum = 0.f;
      for (int r = 0; r < R.count; ++r) sum = fmaf(ex2(keep.at[r * keep.ld + (i - kbeg)] - stat[r].x), stat[r].y, sum);
      w[i] = (q == 0 ? old[0] : q == 1 ? old[1] : q == 2 ? old[2] : q == 3 ? old[3] : w[i]) + sum;
    }
  }
  if (!p.cluster) return;
  cluster_sync_all();
  // row r is folded by CTA r % splits of the cluster, in the order of the splits
  for (int i = warp; i * p.splits + split < R.count; i += 4) {
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
    const size_t bh = row_head<MODE>(p, R, r);
    Parts<8> pre;
    pre.load(p.part_o, p.part_ml, bh * p.prefix_parts, parts, lane);
    pre.fold(parts, lane, x);
    store_row(p.out + bh * HD, lane, x);
  }
  cluster_sync_all();  // nobody leaves while its rows are read
}

// Joins a row's prefix partials and own splits, one warp per (sequence, head).
template <int MODE>
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
  int n;  // keys of the row
  if (MODE == OTree) {
    const int b = tree_sequence(p, bh / p.n_q, lane);
    if (b < 0) return;  // a row of no sequence
    OwnRows R{};
    n = tree_keys(p, b, R);
  } else {
    n = key_position(__ldcg(p.positions + bh / p.n_q), p.key_limit) + 1;
  }
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

// Key weights: joins a row's splits, and adds to the weight of every key of a
// (sequence, K/V head) what the group's heads gave it,
//   weights[key] += sum over heads of 2^(score - max) / sum,
// each key by one thread and its heads in order. NAT: scores in natural units,
// one part per row, whose output is there already (fp32 models). A thread takes 4
// keys at a time, a block's width apart (rows of any stride are read whole lines at a
// time), and 4 heads; the first ones are loaded before the maxima and sums. Bound by
// latency and the scores' bytes, in L2 while they fit: 64 sequences of up to 16384 keys, 32 / 8
// heads, 91 MB, 25 us beside 328 of the kernel that leaves them (2.29 GB, 6.96 TB/s).
constexpr int WEIGH_THREADS = 256, WEIGH_KEYS = 4, WEIGH_HEADS = 4;
template <bool NAT>
__global__ void __launch_bounds__(WEIGH_THREADS, 4) attn_weights_kernel(OwnParams p) {
  grid_dep_wait();
  grid_dep_launch();
  extern __shared__ float2 stat[];  // maximum and reciprocal sum of the group's G heads
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = p.G;
  const int g = blockIdx.y, b = blockIdx.z;
  const int n = key_position(p.positions[b], p.key_limit) + 1;
  int used = n > 0;  // splits that have keys
  if (used && p.splits > 1) {
    const int share = own_share(p, n);
    used = (n + share - 1) / share;
  }
  if (!bc_ok(used <= p.splits && n <= p.ld, p.status)) return;
  const size_t row0 = (size_t)b * p.n_q + (size_t)g * G;
  float* w = p.weights + ((size_t)b * p.n_kv + g) * p.ld;
  const float* sc = p.scores + row0 * p.ld;
  const int key_blocks = NAT ? gridDim.x : gridDim.x - 1;
  if (!NAT && blockIdx.x == key_blocks) {  // one block joins the output rows
    for (int r = warp; r < G; r += WEIGH_THREADS / 32) {
      Parts<8> own;
      RowSum row;
      own.load(p.own_o, p.own_ml, (row0 + r) * p.splits, p.splits, lane);
      own.fold(used, lane, row);
      store_row(p.out + (row0 + r) * HD, lane, row);
    }
    return;
  }
  if (blockIdx.x * (WEIGH_THREADS * WEIGH_KEYS) >= n) return;
  int i = blockIdx.x * (WEIGH_THREADS * WEIGH_KEYS) + threadIdx.x;
  float old[WEIGH_KEYS], x[WEIGH_HEADS][WEIGH_KEYS];
  auto load = [&](int r0) {
#pragma unroll
    for (int k = 0; k < WEIGH_HEADS; ++k)
#pragma unroll
      for (int q = 0; q < WEIGH_KEYS; ++q)
        if (r0 + k < G && i + q * WEIGH_THREADS < n) x[k][q] = sc[(size_t)(r0 + k) * p.ld + i + q * WEIGH_THREADS];
  };
  auto load_old = [&] {
#pragma unroll
    for (int q = 0; q < WEIGH_KEYS; ++q)
      if (i + q * WEIGH_THREADS < n) old[q] = w[i + q * WEIGH_THREADS];
  };
  load_old();
  load(0);
  for (int r = warp; r < G; r += WEIGH_THREADS / 32) {
    const float2* ml = reinterpret_cast<const float2*>(p.own_ml) + (row0 + r) * p.splits;
    float m = -INFINITY, l = 0.f;
    for (int s = lane; s < used; s += 32) m = fmaxf(m, ml[s].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    for (int s = lane; s < used; s += 32) {
      const float2 y = ml[s];
      if (y.x != -INFINITY) l = fmaf(y.y, NAT ? expf(y.x - m) : exp2f(y.x - m), l);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) stat[r] = make_float2(m == -INFINITY ? 0.f : m, l > 0.f || l != l ? 1.f / l : 0.f);
  }
  __syncthreads();
  for (bool first = true; i < n; i += key_blocks * (WEIGH_THREADS * WEIGH_KEYS), first = false) {
    if (!first) {
      load_old();
      load(0);
    }
    float sum[WEIGH_KEYS] = {};
    for (int r0 = 0; r0 < G; r0 += WEIGH_HEADS) {
      if (r0 > 0) load(r0);
#pragma unroll
      for (int k = 0; k < WEIGH_HEADS; ++k) {
        if (r0 + k >= G) break;
        const float2 st = stat[r0 + k];
#pragma unroll
        for (int q = 0; q < WEIGH_KEYS; ++q) {
          const float y = x[k][q] - st.x;
          sum[q] = fmaf(NAT ? expf(y) : ex2(y), st.y, sum[q]);
        }
      }
    }
#pragma unroll
    for (int q = 0; q < WEIGH_KEYS; ++q)
      if (i + q * WEIGH_THREADS < n) w[i + q * WEIGH_THREADS] = old[q] + sum[q];
  }
}

}  // namespace

cudaError_t attn_own_prepare() {
  const void* const all[] = {(const void*)attn_own_kernel<true, ODecode>, (const void*)attn_own_kernel<false, ODecode>,
                             (const void*)attn_own_kernel<true, OWeigh>, (const void*)attn_own_kernel<false, OWeigh>,
                             (const void*)attn_own_kernel<true, OTree>};
  for (const void* f : all) {
    const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)OWN_SMEM_MOST);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

static OwnParams own_params(const SharedArgs& a, const SharedPlan& s) {
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
  return p;
}

cudaError_t launch_shared_own(const SharedArgs& a, const SharedPlan& s, cudaStream_t st) {
  const OwnParams p = own_params(a, s);
  const size_t rows = p.rows;
  const dim3 grid(s.own_splits, a.n_kv, a.B), block(OWN_THREADS);
  const dim3 cluster(s.cluster ? s.own_splits : 0, 1, 1);
  const cudaError_t e =
      p.G <= 8 ? launch_kc(attn_own_kernel<true, ODecode>, grid, block, OWN_SMEM, st, cluster, *a.map_k,
                           *a.map_v, *a.map_k16, *a.map_v16, p)
               : launch_kc(attn_own_kernel<false, ODecode>, grid, block, OWN_SMEM, st, cluster, *a.map_k,
                           *a.map_v, *a.map_k16, *a.map_v16, p);
  if (e != cudaSuccess || !s.join) return e;
  return launch_k(attn_own_join_kernel<ODecode>, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, st, 0, p,
                  (int)rows);
}

// 16 CTAs per SM share the keys of all (sequence, K/V head) pairs, a pass of the threads each at
// least (64 sequences of up to 16384 keys 367 us, eight 371; short ones the same).
template <bool NAT>
static cudaError_t launch_weights(const OwnParams& p, const SharedArgs& a, cudaStream_t st) {
  const int per = WEIGH_THREADS * WEIGH_KEYS;
  const int chunks = std::max(1, std::min((a.key_limit + per - 1) / per, 16 * a.sm_count / (a.B * a.n_kv)));
  return launch_k(attn_weights_kernel<NAT>, dim3(chunks + !NAT, a.n_kv, a.B), dim3(WEIGH_THREADS),
                  p.G * sizeof(float2), st, 0, p);
}

cudaError_t launch_decode_weights(const SharedArgs& a, const SharedPlan& s, const WeightsArgs& w, cudaStream_t st) {
  OwnParams p = own_params(a, s);
  p.scores = w.scores;
  p.weights = w.weights;
  p.ld = w.ld;
  p.keep = s.keep;
  const dim3 grid(s.own_splits, a.n_kv, a.B), block(OWN_THREADS);
  const size_t sm = OWN_SMEM + (size_t)4 * p.G * s.keep;
  const cudaError_t e =
      p.G <= 8 ? launch_k(attn_own_kernel<true, OWeigh>, grid, block, sm, st, 0, *a.map_k, *a.map_v,
                          *a.map_k16, *a.map_v16, p)
               : launch_k(attn_own_kernel<false, OWeigh>, grid, block, sm, st, 0, *a.map_k, *a.map_v,
                           *a.map_k16, *a.map_v16, p);
  if (e != cudaSuccess || s.keep) return e;
  return launch_weights<false>(p, a, st);
}

cudaError_t launch_add_weights_f32(const SharedArgs& a, const WeightsArgs& w, cudaStream_t st) {
  OwnParams p{};
  p.positions = a.positions;
  p.status = a.status;
  p.n_q = a.n_q;
  p.n_kv = a.n_kv;
  p.G = a.n_q / a.n_kv;
  p.key_limit = a.key_limit;
  p.splits = 1;
  p.own_ml = w.stats;
  p.scores = w.scores;
  p.weights = w.weights;
  p.ld = w.ld;
  return launch_weights<true>(p, a, st);
}

// Trees of few rows: blocks of 8 (row, head) pairs of a K/V head on this kernel, or 128
// and 256 on the tensor-core kernel. In a cache with room for 4096 positions, this kernel and
// that one: 16 sequences of 8 rows, 32 heads 104 and 122 us, 64 of one row, 32 / 8 heads
// 104 and 112; two blocks (a second pass over the keys, mostly from L2) 8 sequences of 13
// rows, 40 heads, up to 500 keys 19 and 32, up to 8000 138 and 108, up to 2000 capped 48
// and 73 (the softmax of the other kernel works on all 128 rows); three 91 and 60. Where 8
// CTAs for each (sequence, K/V head) are few and the context may be long, the other
// kernel's equal shares count: one row, 8 K/V heads, 30000 keys 34 (57 CTAs each) and 30 us.
// Several blocks of few short sequences: all of their CTAs are resident, and the other
// kernel takes 10 us and more whatever they hold (one sequence, 64 / 8 heads, 750 and 1500
// keys: 4 rows 9.9 and 11.0 us, the other 13.0 and 14.7; 26 rows 14.1 and 20.2, the other 15.4 and
// 16.2; 4 sequences of 8 rows, 300 and 750 keys 12.1 and 17.8, the other 13.7 and 14.4). And where
// the other kernel has several items per SM, of a tile or so (6 sequences of 17 rows, 32 heads,
// 20 and 120 keys 11.5 and 13.8, the other 22.3 and 15.9; 40 of 30 rows, 8 heads, 130 keys 22.6, 20.5).
// Groups of more than 8 heads: in slices, each with a pass over the keys (one sequence of 4 rows, 16 / 1
// heads, 300 and 1100 keys 8.6 and 8.8 us, the other kernel 11.5 and 14.0).
static void tree_slices(int G, int* slices, int* per) {
  *slices = (G + 7) / 8;
  *per = (G + *slices - 1) / *slices;
}
static long long tree_pairs(const TreeArgs& a) {  // CTAs without splits, by the mean rows
  const int rows = (a.n_rows + a.B - 1) / a.B;
  int shift = 0, slices, per;
  tree_slices(a.n_q / a.n_kv, &slices, &per);
  while (2 * per << shift <= 8) ++shift;
  return (long long)a.B * a.n_kv * slices * ((rows + (1 << shift) - 1) >> shift);
}
bool tree_own_applies(const TreeArgs& a) {
  const int G = a.n_q / a.n_kv;
  if (a.head_dim != HD || (long long)a.B + a.n_rows > 65535 || a.n_kv > 32767) return false;  // the launch's grid
  const long long heads = (long long)a.B * a.n_kv, pairs = tree_pairs(a), rows = (a.n_rows + a.B - 1) / a.B;
  if (8 * heads < 2 * a.sm_count && a.key_limit > 8192) return false;
  if (pairs == heads || (pairs == 2 * heads && (a.sc.cap > 0.f || a.sc.slopes || a.key_limit <= 2048))) return true;
  const long long items = heads * ((rows * G + 127) / 128);  // about, the other kernel's
  return (pairs <= 3 * a.sm_count && pairs * a.key_limit <= 1100ll * a.sm_count) ||
         (items > a.sm_count && pairs <= 4 * items && pairs * a.key_limit <= 450ll * a.sm_count);
}

cudaError_t launch_tree_own(const TreeArgs& a, const TreePlan& t, cudaStream_t st, int64_t* launches) {
  OwnParams p{};
  p.q = (const bf16*)a.q;
  p.out = (bf16*)a.out;
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
  p.rows = (size_t)a.n_rows * a.n_q;
  p.scale = a.sc.scale;
  p.cap = a.sc.cap;
  p.slopes = a.sc.slopes;
  p.cu_rows = a.cu_rows;
  p.start_pos = a.start_pos;
  p.row_pos = a.row_pos;
  p.tree = TreeMask{a.mask, a.mask_words};
  p.n_rows = a.n_rows;
  p.n_seq = a.B;
  p.tree_shift = t.shift;
  p.slices = t.slices;
  p.per = t.per;
  p.splits = t.splits;
  p.min_share = t.min_share;
  p.cluster = t.cluster;
  p.join = t.join;
  const int blocks = (a.n_rows >> t.shift) + a.B, k = t.splits;
  *launches += p.join ? 2 : 1;
  p.own_room = p.rows * k;
  p.own_o = a.partial;
  p.own_ml = a.partial + p.own_room * HD;
  p.part_o = p.own_o;  // no prefix: no parts of it
  p.part_ml = p.own_ml;
  const cudaError_t e = launch_kc(attn_own_kernel<true, OTree>, dim3(k, a.n_kv * p.slices, blocks),
                                  dim3(OWN_THREADS), OWN_SMEM, st, dim3(p.cluster ? k : 0, 1, 1), *a.map_k,
                                  *a.map_v, *a.map_k16, *a.map_v16, p);
  if (e != cudaSuccess || !p.join) return e;
  return launch_k(attn_own_join_kernel<OTree>, dim3((unsigned)((p.rows + 3) / 4)), dim3(128), 0, st, 0, p,
                  (int)p.rows);
}

}  // namespace llgb
