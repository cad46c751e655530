// Attention with capped or biased scores on the CUDA cores, for fp32 models
// with any head_dim up to 256: packed documents (two-way prefix, causal rest),
// decode over a cache with a shared prefix (if asked, its scores and each row's maximum
// and sum are kept for the key weights), and drafted trees, whose rows are taken as a
// document's and whose keys come from the cache.
//
//   x = scale q.k;  s = (cap tanh(x / cap) or x) - slope |i - j|;  softmax;  sum p v
//
// One CTA of 256 threads per (8 RW query rows, K/V source): documents take 32
// rows of one head (RW 4), decode up to 16 query heads of one K/V head and
// sequence (RW 2). K and V tiles of 64 keys come through shared memory with
// asynchronous copies; several CTAs per SM hide each other's waits. A warp owns
// RW rows: for the scores a lane has keys lane and lane + 32, for the output
// head_dim / 32 dims, so K and V are read once per warp without conflicts, and
// Q and P as broadcasts. Row maxima are folded with butterflies (the running
// maximum and sum of an online softmax, in fp32), and P goes through shared
// memory within the warp. fp32 arithmetic throughout (exp and tanh of the CUDA
// math library). Where there are few items, up to 8 CTAs (a cluster) take an
// item's key tiles in turn and merge through distributed shared memory.
//
// Bound by shared memory before arithmetic: per four dims a warp reads two K vectors
// (4 wavefronts each) and a broadcast per row, 12 wavefronts for documents against
// the 8 cycles that its 32 multiply-adds take of the SM, and P V the same; in
// decode the row slots beyond a K/V head's query heads compute rows that are not
// stored. On top comes latency: with 4 warps per scheduler (two CTAs per SM) half of
// the cycles issue nothing, for waits on shared memory and on barriers between tiles;
// hence the small single stage (four CTAs at 64 dims). Measured, against 16
// lanes per row with two rows each: documents of 700 rows in all, 8 heads, 64
// dims 49 -> 44 us; one document of 4000 rows 558 -> 549 us, with 128 dims 980 ->
// 1040 us, 2000 rows with 256 dims 389 -> 305 us; decode of 32 sequences of 1000
// keys, 8 heads of 128 dims 208 -> 136 us. Two stages of K and V instead of more
// CTAs: 48 instead of 44 us; 64 rows per CTA: 46 (4000 rows 570 instead of 549).
#include <algorithm>

#include "attn_score.cuh"
#include "internal.h"

namespace llgb {

namespace {

constexpr int SK = 64;        // keys per tile
constexpr int S_THREADS = 256;

struct SimtParams {
  const float *q, *k, *v;
  float* out;
  int n_q, n_kv, G, d;
  ScoreArgs sc;
  uint32_t* status;
  // documents
  const int32_t *cu_rows, *prefix_len;
  int n_rows, n_docs;
  // decode
  const int32_t *positions, *page_table;
  int layer, page_size, capacity, batch_cap, n_pages, max_pages, key_limit, shared_len, shared_seq;
  int n_seq;
  int row_chunks;  // chunks of 16 heads per K/V head
  int splits;      // CTAs (a cluster) that share an item's key tiles
  // key weights: the scores [n_seq][n_q][ld] and every row's maximum and sum, or null
  float *scores, *stats;
  int64_t ld;
  // trees: out, cu_rows, n_rows, n_docs as documents, the cache as in decode
  const int32_t *start_pos, *row_pos;
  const uint32_t* mask;
  int mask_words;
};

// What a launch works on: decode rows, documents, trees of drafted rows over a cache.
enum { SDecode, SDocs, STree };

// Work item -> (document, tile of `rows` query rows, first row, row count), for a
// whole warp: 32 documents per step, their tile counts summed by a warp scan.
// Tiles of a document come last first (the longest rows of a causal mask).
// False when the item is past the last document's tiles.
__device__ __forceinline__ bool find_tile(const int32_t* cu, int n_docs, int n_rows, int rows,
                                          int item, uint32_t* status, int& b, int& tile, int& lo,
                                          int& n) {
  const int lane = threadIdx.x & 31;
  for (int b0 = 0; b0 < n_docs; b0 += 32) {
    int my_lo = 0, my_n = 0;
    if (b0 + lane < n_docs) doc_rows(cu, b0 + lane, n_rows, status, my_lo, my_n);
    int upto = (my_n + rows - 1) / rows;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    const uint32_t m = __ballot_sync(0xffffffffu, item < upto);
    if (m) {
      const int w = __ffs(m) - 1;
      b = b0 + w;
      tile = __shfl_sync(0xffffffffu, upto, w) - 1 - item;
      lo = __shfl_sync(0xffffffffu, my_lo, w);
      n = __shfl_sync(0xffffffffu, my_n, w);
      return true;
    }
    item -= __shfl_sync(0xffffffffu, upto, 31);
  }
  return false;
}

// Element offset of key j of sequence b, K/V head g in the cache; -1 (flagged)
// for a page outside the pool.
__device__ __forceinline__ long long key_offset(const SimtParams& p, int b, int g, int j) {
  if (j < p.shared_len) b = p.shared_seq;
  if (!bc_ok(p.page_size == 0 ? b < p.batch_cap && j < p.capacity : j / p.page_size < p.max_pages, p.status))
    return -1;
  if (p.page_size == 0)
    return ((((long long)p.layer * p.batch_cap + b) * p.n_kv + g) * p.capacity + j) * p.d;
  const int pi = j / p.page_size;
  const int page = p.page_table[(size_t)b * p.max_pages + pi];
  if (page < 0 || page >= p.n_pages) {
    flag(p.status, LLAMA_FLAG_PAGE_RANGE);
    return -1;
  }
  return ((((long long)p.layer * p.n_pages + page) * p.n_kv + g) * p.page_size + j - pi * p.page_size) *
         p.d;
}

// 16 bytes global -> shared, or zeros
__device__ __forceinline__ void copy16(float* dst, const float* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

template <int RW, int DM>
struct SimtTile {  // RW: query rows of a warp; DM: head_dim rounded up to 64, 128 or 256
  static constexpr int RT = RW * S_THREADS / 32, LD = DM + 4;
  static constexpr size_t bytes = (size_t)(RT * DM + 2 * SK * LD + RT * SK) * sizeof(float);
};

// A lane's DL consecutive values of a row, DL 2 or 4 (or two fours, 128 apart)
template <int DL>
__device__ __forceinline__ void load_dims(const float* row, int lane, float* v) {
  if (DL == 2) {
    const float2 x = *reinterpret_cast<const float2*>(row + 2 * lane);
    v[0] = x.x;
    v[1] = x.y;
  } else {
#pragma unroll
    for (int i = 0; i < DL; i += 4) {
      const float4 x = *reinterpret_cast<const float4*>(row + 4 * lane + 32 * i);
      v[i] = x.x;
      v[i + 1] = x.y;
      v[i + 2] = x.z;
      v[i + 3] = x.w;
    }
  }
}
template <int DL>
__device__ __forceinline__ void store_dims(float* row, int lane, int d, const float* v) {
  if (DL == 2) {
    if (2 * lane < d) *reinterpret_cast<float2*>(row + 2 * lane) = make_float2(v[0], v[1]);
  } else {
#pragma unroll
    for (int i = 0; i < DL; i += 4)
      if (4 * lane + 32 * i < d)
        *reinterpret_cast<float4*>(row + 4 * lane + 32 * i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  }
}

template <int RW, int DM, int MODE>
__global__ void __launch_bounds__(S_THREADS) attn_simt_kernel(SimtParams p) {
  constexpr bool TREE = MODE == STree, DOCS = MODE == SDocs || TREE;  // DOCS: packed rows of one head
  grid_dep_wait();
  grid_dep_launch();
  using Tile = SimtTile<RW, DM>;
  constexpr int RT = Tile::RT, LD = Tile::LD, DL = DM / 32;
  extern __shared__ __align__(16) float sm[];
  float* sq = sm;                     // [RT][DM]
  float* sk = sq + RT * DM;           // [SK][LD], and V behind it
  float* sv = sk + SK * LD;
  float* sp = sv + SK * LD;           // [RT][SK]
  if (!bc_smem(sm, (uint32_t)Tile::bytes, 16, threadIdx.x == 0 ? p.status : nullptr)) return;
  const int lane = threadIdx.x & 31, r0 = threadIdx.x / 32 * RW;  // the warp's rows r0 .. r0 + RW - 1
  const int d = p.d;
  const int item = blockIdx.x / p.splits, part = blockIdx.x - item * p.splits;
  // which rows
  int b, g, h0, lo = 0, n = 0, q0 = 0, rows, n_keys, pre = 0, pos = 0, start = 0;
  if (DOCS) {
    const int h = item % p.n_q;
    int tile;
    if (!find_tile(p.cu_rows, p.n_docs, p.n_rows, RT, item / p.n_q, p.status, b, tile, lo, n))
      return;
    h0 = h;
    g = h / p.G;
    q0 = tile * RT;
    rows = min(RT, n - q0);
    if (!bc_ok(lo + q0 + rows <= p.n_rows && h0 < p.n_q, p.status)) return;
    if (TREE) {
      start = p.start_pos[b];
      const long long end = (long long)start + n;
      if ((start < 0 || end > p.key_limit) && q0 == 0 && part == 0 && threadIdx.x == 0)
        flag(p.status, LLAMA_FLAG_POS_RANGE);
      n_keys = start < 0 ? 0 : (int)(end < p.key_limit ? end : p.key_limit);
      // rows past the cache lie behind all keys, as far as the bias's softmax can tell, and start + row stays an int
      start = min(max(start, 0), n_keys);
    } else {
      pre = p.prefix_len ? min(max(p.prefix_len[b], 0), n) : 0;
      n_keys = max(q0 + rows, pre);
    }
  } else {
    const int c = item % p.row_chunks;
    g = (item / p.row_chunks) % p.n_kv;
    b = item / (p.row_chunks * p.n_kv);
    h0 = g * p.G + c * RT;
    rows = min(RT, p.G - c * RT);
    if (!bc_ok(b < p.n_seq && h0 + rows <= p.n_q, p.status)) return;
    pos = p.positions[b];
    if ((pos < 0 || pos >= p.key_limit) && part == 0 && threadIdx.x == 0)
      flag(p.status, LLAMA_FLAG_POS_RANGE);
    pos = key_position(pos, p.key_limit);
    n_keys = pos + 1;
  }
  // element offset of row r (documents: packed row, one head; decode: one row, head h0 + r)
  auto row_off = [&](int r) -> size_t {
    return DOCS ? ((size_t)(lo + q0 + r) * p.n_q + h0) * d : ((size_t)b * p.n_q + h0 + r) * d;
  };
  // K and V of the tile at k0; keys past n_keys and dims past d are zeros
  auto load_tile = [&](int k0) {
    for (int i = threadIdx.x; i < SK * (DM / 4); i += S_THREADS) {
      const int j = i / (DM / 4), x = 4 * (i % (DM / 4));
      long long off = -1;
      if (k0 + j < n_keys && x < d)
        off = MODE == SDocs ? ((long long)(lo + k0 + j) * p.n_kv + g) * d : key_offset(p, b, g, k0 + j);
      copy16(sk + j * LD + x, off < 0 ? p.k : p.k + off + x, off >= 0);
      copy16(sv + j * LD + x, off < 0 ? p.v : p.v + off + x, off >= 0);
    }
  };
  const int first = part * SK, step = p.splits * SK;  // this CTA's key tiles
  if (first < n_keys) load_tile(first);
  for (int i = threadIdx.x; i < RT * (DM / 4); i += S_THREADS) {
    const int r = i / (DM / 4), x = 4 * (i % (DM / 4));
    *reinterpret_cast<float4*>(sq + r * DM + x) =
        r < rows && x < d ? *reinterpret_cast<const float4*>(p.q + row_off(r) + x)
                          : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float slope[RW];
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    const int r = r0 + i;
    slope[i] = p.sc.slopes && r < rows ? p.sc.slopes[DOCS ? h0 : h0 + r] : 0.f;
  }
  float m[RW], l[RW], o[RW][DL];
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int x = 0; x < DL; ++x) o[i][x] = 0.f;
  }
  const float icap = p.sc.cap > 0.f ? 1.f / p.sc.cap : 0.f;
  for (int k0 = first; k0 < n_keys; k0 += step) {
    copies_wait();
    __syncthreads();
    float s[RW][2];
#pragma unroll
    for (int i = 0; i < RW; ++i) s[i][0] = s[i][1] = 0.f;
#pragma unroll 4
    for (int x = 0; x < DM; x += 4) {
      const float4 ka = *reinterpret_cast<const float4*>(sk + lane * LD + x);
      const float4 kb = *reinterpret_cast<const float4*>(sk + (lane + 32) * LD + x);
#pragma unroll
      for (int i = 0; i < RW; ++i) {
        const float4 qv = *reinterpret_cast<const float4*>(sq + (r0 + i) * DM + x);
        s[i][0] = fmaf(qv.x, ka.x, fmaf(qv.y, ka.y, fmaf(qv.z, ka.z, fmaf(qv.w, ka.w, s[i][0]))));
        s[i][1] = fmaf(qv.x, kb.x, fmaf(qv.y, kb.y, fmaf(qv.z, kb.z, fmaf(qv.w, kb.w, s[i][1]))));
      }
    }
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      // the row's index, and (trees: for the bias alone) its position
      const int ri = q0 + r0 + i;
      int qi = DOCS ? ri : pos;
      if (TREE && p.sc.slopes && r0 + i < rows)
        qi = p.row_pos ? min(max(p.row_pos[lo + ri], 0), kMaxPos) : start + ri;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int key = k0 + lane + 32 * j;
        float v = s[i][j] * p.sc.scale;
        if (p.sc.cap > 0.f) v = p.sc.cap * tanhf(v * icap);
        const int x = key - start;  // trees: the key's row
        if (p.sc.slopes) {
          int at = key;
          if (TREE && p.row_pos && x >= 0 && key < n_keys) at = min(max(p.row_pos[lo + x], 0), kMaxPos);
          v -= slope[i] * fabsf((float)(qi - at));
        }
        bool keep = key < n_keys;
        if (MODE == SDocs) keep = keep && (key <= qi || key < pre);
        if (TREE && keep && x >= 0)
          keep = r0 + i < rows && (p.mask ? x < 32 * p.mask_words &&
                                                (p.mask[(size_t)(lo + ri) * p.mask_words + (x >> 5)] >> (x & 31) & 1u)
                                          : x <= ri);
        if (!DOCS && p.scores && keep && r0 + i < rows)
          p.scores[((size_t)b * p.n_q + h0 + r0 + i) * p.ld + key] = v;
        s[i][j] = keep ? v : -INFINITY;
      }
      float mx = fmaxf(s[i][0], s[i][1]);
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float mn = fmaxf(m[i], mx);
      const float mu = mn == -INFINITY ? 0.f : mn;  // no finite score yet: weights 0 (of NaN: NaN)
      const float f = expf(m[i] - mu);
      m[i] = mn;
      const float ea = expf(s[i][0] - mu), eb = expf(s[i][1] - mu);
      sp[(r0 + i) * SK + lane] = ea;
      sp[(r0 + i) * SK + lane + 32] = eb;
      l[i] = l[i] * f + (ea + eb);  // this lane's share of the row's sum
#pragma unroll
      for (int x = 0; x < DL; ++x) o[i][x] *= f;
    }
    __syncwarp();  // a row's P is written and read by one warp
    const int nk = min(SK, n_keys - k0);
    // V rows past the last key are zeros, and so are their weights: whole fours
    for (int j = 0; j < nk; j += 4) {
      float vv[4][DL];
#pragma unroll
      for (int q = 0; q < 4; ++q) load_dims<DL>(sv + (j + q) * LD, lane, vv[q]);
#pragma unroll
      for (int i = 0; i < RW; ++i) {
        const float4 pr = *reinterpret_cast<const float4*>(sp + (r0 + i) * SK + j);
#pragma unroll
        for (int x = 0; x < DL; ++x)
          o[i][x] = fmaf(pr.w, vv[3][x], fmaf(pr.z, vv[2][x], fmaf(pr.y, vv[1][x], fmaf(pr.x, vv[0][x], o[i][x]))));
      }
    }
    __syncthreads();  // the tiles may be overwritten
    if (k0 + step < n_keys) load_tile(k0 + step);
  }
#pragma unroll
  for (int i = 0; i < RW; ++i)
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
  if (p.splits > 1) {
    // The cluster's CTAs leave (O, maximum, sum) in their shared memory; row r is
    // merged by CTA r % splits, in the order of the parts.
    float* so = sk;             // [RT][DM], over the tiles
    float* sml = so + RT * DM;  // [RT][2]
    static_assert(RT * (DM + 2) <= 2 * SK * LD, "the rows fit over the tiles");
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      store_dims<DL>(so + (r0 + i) * DM, lane, DM, o[i]);
      if (lane == 0) *reinterpret_cast<float2*>(sml + 2 * (r0 + i)) = make_float2(m[i], l[i]);
    }
    cluster_sync_all();
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      if ((r0 + i) % p.splits != part) continue;
      const uint32_t am = smem_u32(sml + 2 * (r0 + i)), ao = smem_u32(so + (r0 + i) * DM);
      float M = -INFINITY, L = 0.f;
      for (int c = 0; c < p.splits; ++c) M = fmaxf(M, dsmem_ld2(dsmem_addr(am, c)).x);
#pragma unroll
      for (int x = 0; x < DL; ++x) o[i][x] = 0.f;
      for (int c = 0; c < p.splits; ++c) {
        const float2 ml = dsmem_ld2(dsmem_addr(am, c));
        const float f = ml.x == -INFINITY ? 0.f : expf(ml.x - M);
        L = fmaf(ml.y, f, L);
        const uint32_t src = dsmem_addr(ao, c);
        if (DL == 2) {
          const float2 v = dsmem_ld2(src + 8 * lane);
          o[i][0] = fmaf(v.x, f, o[i][0]);
          o[i][1] = fmaf(v.y, f, o[i][1]);
        } else {
#pragma unroll
          for (int x = 0; x < DL; x += 4) {
            const float4 v = dsmem_ld4(src + 16 * lane + 128 * x);
            o[i][x] = fmaf(v.x, f, o[i][x]);
            o[i][x + 1] = fmaf(v.y, f, o[i][x + 1]);
            o[i][x + 2] = fmaf(v.z, f, o[i][x + 2]);
            o[i][x + 3] = fmaf(v.w, f, o[i][x + 3]);
          }
        }
      }
      m[i] = M;
      l[i] = L;
    }
    cluster_sync_all();  // nobody leaves while its rows are read
  }
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    const int r = r0 + i;
    if (r >= rows || (p.splits > 1 && r % p.splits != part)) continue;
    float w[DL];
#pragma unroll
    for (int x = 0; x < DL; ++x) w[x] = n_keys > 0 && (!TREE || l[i] != 0.f) ? o[i][x] / l[i] : 0.f;
    store_dims<DL>(p.out + row_off(r), lane, d, w);
    if (!DOCS && p.stats && lane == 0)
      *reinterpret_cast<float2*>(p.stats + 2 * ((size_t)b * p.n_q + h0 + r)) = make_float2(merge_max(m[i], l[i]), l[i]);
  }
}

template <int RW, int DM, int MODE>
cudaError_t prep() {
  return cudaFuncSetAttribute(attn_simt_kernel<RW, DM, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)SimtTile<RW, DM>::bytes);
}

template <int RW, int MODE>
cudaError_t run(const SimtParams& p, long long items, cudaStream_t st) {
  const dim3 grid((unsigned)(items * p.splits)), cluster(p.splits > 1 ? p.splits : 0, 1, 1);
  if (p.d <= 64)
    return launch_kc(attn_simt_kernel<RW, 64, MODE>, grid, dim3(S_THREADS), SimtTile<RW, 64>::bytes,
                     st, cluster, p);
  if (p.d <= 128)
    return launch_kc(attn_simt_kernel<RW, 128, MODE>, grid, dim3(S_THREADS), SimtTile<RW, 128>::bytes,
                     st, cluster, p);
  return launch_kc(attn_simt_kernel<RW, 256, MODE>, grid, dim3(S_THREADS), SimtTile<RW, 256>::bytes,
                   st, cluster, p);
}

// CTAs that share an item's keys: doubled up to a cluster's 8 while there are
// fewer than three CTAs per SM and each keeps a tile of the longest (700 rows:
// three and four per SM 44 us, six 51).
int simt_splits(long long items, int keys, int sm_count) {
  int s = 1;
  while (s < 8 && items * s < 3 * sm_count && keys >= 2 * s * SK) s *= 2;
  return s;
}

}  // namespace

cudaError_t attn_simt_prepare() {
  cudaError_t (*const all[])() = {prep<4, 64, SDocs>,   prep<4, 128, SDocs>,   prep<4, 256, SDocs>,
                                  prep<2, 64, SDecode>, prep<2, 128, SDecode>, prep<2, 256, SDecode>,
                                  prep<4, 64, STree>,   prep<4, 128, STree>,   prep<4, 256, STree>};
  for (auto f : all) {
    const cudaError_t e = f();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_docs_simt(const DocsArgs& a, cudaStream_t st) {
  SimtParams p{};
  p.q = (const float*)a.q;
  p.k = (const float*)a.k;
  p.v = (const float*)a.v;
  p.out = (float*)a.out;
  p.n_q = a.n_q;
  p.n_kv = a.n_kv;
  p.G = a.n_q / a.n_kv;
  p.d = a.head_dim;
  p.sc = a.sc;
  p.status = a.status;
  p.cu_rows = a.cu_rows;
  p.prefix_len = a.prefix_len;
  p.n_rows = a.n_rows;
  p.n_docs = a.n_docs;
  const long long tiles = a.n_rows / 32 + std::min(a.n_docs, a.n_rows);  // an upper bound
  p.splits = simt_splits(tiles * a.n_q, a.n_rows, a.sm_count);
  return run<4, SDocs>(p, tiles * a.n_q, st);
}

cudaError_t launch_shared_simt(const SharedArgs& a, cudaStream_t st, const WeightsArgs* w) {
  SimtParams p{};
  if (w) {
    p.scores = w->scores;
    p.stats = w->stats;
    p.ld = w->ld;
  }
  p.q = (const float*)a.q;
  p.k = (const float*)a.k_cache;
  p.v = (const float*)a.v_cache;
  p.out = (float*)a.out;
  p.n_q = a.n_q;
  p.n_kv = a.n_kv;
  p.G = a.n_q / a.n_kv;
  p.d = a.head_dim;
  p.sc = a.sc;
  p.status = a.status;
  p.positions = a.positions;
  p.page_table = a.page_table;
  p.layer = a.layer;
  p.page_size = a.page_size;
  p.capacity = a.capacity;
  p.batch_cap = a.batch_cap;
  p.n_pages = a.n_pages;
  p.max_pages = a.max_pages;
  p.key_limit = a.key_limit;
  p.shared_len = a.shared_len;
  p.shared_seq = a.shared_seq;
  p.n_seq = a.B;
  p.row_chunks = (p.G + 15) / 16;
  const long long items = (long long)a.B * a.n_kv * p.row_chunks;
  p.splits = simt_splits(items, a.key_limit, a.sm_count);
  return run<2, SDecode>(p, items, st);
}

cudaError_t launch_tree_simt(const TreeArgs& a, cudaStream_t st) {
  SimtParams p{};
  p.q = (const float*)a.q;
  p.k = (const float*)a.k_cache;
  p.v = (const float*)a.v_cache;
  p.out = (float*)a.out;
  p.n_q = a.n_q;
  p.n_kv = a.n_kv;
  p.G = a.n_q / a.n_kv;
  p.d = a.head_dim;
  p.sc = a.sc;
  p.status = a.status;
  p.cu_rows = a.cu_rows;
  p.n_rows = a.n_rows;
  p.n_docs = a.B;
  p.start_pos = a.start_pos;
  p.row_pos = a.row_pos;
  p.mask = a.mask;
  p.mask_words = a.mask_words;
  p.page_table = a.page_table;
  p.layer = a.layer;
  p.page_size = a.page_size;
  p.capacity = a.capacity;
  p.batch_cap = a.batch_cap;
  p.n_pages = a.n_pages;
  p.max_pages = a.max_pages;
  p.key_limit = a.key_limit;
  const long long tiles = a.n_rows / 32 + std::min(a.B, a.n_rows);  // an upper bound
  p.splits = simt_splits(tiles * a.n_q, a.key_limit, a.sm_count);
  return run<4, STree>(p, tiles * a.n_q, st);
}

}  // namespace llgb
