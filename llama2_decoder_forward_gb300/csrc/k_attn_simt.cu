// Attention with capped or biased scores on the CUDA cores, for fp32 models
// with any head_dim up to 256: packed documents (two-way prefix, causal rest)
// and decode over a cache with a shared prefix.
//
//   x = scale q.k;  s = (cap tanh(x / cap) or x) - slope |i - j|;  softmax;  sum p v
//
// One CTA of 256 threads per (16 RI query rows, K/V source): documents take rows
// of one head, decode the query heads of one K/V head and sequence. K and V
// tiles of 64 keys come through shared memory with asynchronous copies, the
// next tile's while the current one is used (two stages up to 128 dims).
// Thread (ty, tx) computes the scores of rows ty + 16 i and keys tx + 16 j; the 16
// threads of a row sit in one half-warp and fold its maximum and sum with
// butterflies (the running maximum and sum of an online softmax, in fp32);
// P goes through shared memory within the warp, and the same thread
// accumulates its rows' dims 4 tx + 64 m. fp32 arithmetic throughout (exp and
// tanh of the CUDA math library). Where there are few items, up to 8 CTAs (a
// cluster) take an item's key tiles in turn and merge through distributed shared
// memory. Bound by the fp32 FMA pipe and, with 32-row tiles, the shared-memory
// reads that feed it (documents of 700 rows in all, 8 heads, 64 dims: 68 us
// unsplit, 50 us with splits).
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
  int row_chunks;  // chunks of 16 RI heads per K/V head
  int splits;      // CTAs (a cluster) that share an item's key tiles
};

// Element offset of key j of sequence b, K/V head g in the cache; -1 (flagged)
// for a page outside the pool.
__device__ __forceinline__ long long key_offset(const SimtParams& p, int b, int g, int j) {
  if (j < p.shared_len) b = p.shared_seq;
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
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int RI, int DM>
struct SimtTile {  // DM: head_dim rounded up to 64, 128 or 256
  static constexpr int RT = 16 * RI, LD = DM + 4, STAGES = DM <= 128 ? 2 : 1;
  static constexpr size_t bytes =
      (size_t)(RT * LD + STAGES * 2 * SK * LD + RT * (SK + 4)) * sizeof(float);
};

template <int RI, int DM, bool DOCS>
__global__ void __launch_bounds__(S_THREADS) attn_simt_kernel(SimtParams p) {
  grid_dep_wait();
  grid_dep_launch();
  using Tile = SimtTile<RI, DM>;
  constexpr int RT = Tile::RT, LD = Tile::LD, ST = Tile::STAGES;
  extern __shared__ __align__(16) float sm[];
  float* sq = sm;                     // [RT][LD]
  float* skv = sq + RT * LD;          // [ST][K, V][SK][LD]
  float* sp = skv + ST * 2 * SK * LD; // [RT][SK + 4]
  if (!bc_smem(sm, (uint32_t)Tile::bytes, 16, threadIdx.x == 0 ? p.status : nullptr)) return;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int d = p.d;
  const int item = blockIdx.x / p.splits, part = blockIdx.x - item * p.splits;
  // which rows
  int b, g, h0, lo = 0, n = 0, q0 = 0, rows, n_keys, pre = 0, pos = 0;
  if (DOCS) {
    const int h = item % p.n_q;
    int tile;
    if (!find_tile(p.cu_rows, p.n_docs, p.n_rows, RT, item / p.n_q, p.status, b, tile, lo, n))
      return;
    h0 = h;
    g = h / p.G;
    q0 = tile * RT;
    rows = min(RT, n - q0);
    pre = p.prefix_len ? min(max(p.prefix_len[b], 0), n) : 0;
    n_keys = max(q0 + rows, pre);
  } else {
    const int c = item % p.row_chunks;
    g = (item / p.row_chunks) % p.n_kv;
    b = item / (p.row_chunks * p.n_kv);
    h0 = g * p.G + c * RT;
    rows = min(RT, p.G - c * RT);
    pos = p.positions[b];
    n_keys = pos + 1;
    if (pos < 0 || pos >= p.key_limit) {
      if (part == 0 && threadIdx.x == 0) flag(p.status, LLAMA_FLAG_POS_RANGE);
      n_keys = pos < 0 ? 0 : p.key_limit;
    }
  }
  // element offset of row r (documents: packed row, one head; decode: one row, head h0 + r)
  auto row_off = [&](int r) -> size_t {
    return DOCS ? ((size_t)(lo + q0 + r) * p.n_q + h0) * d : ((size_t)b * p.n_q + h0 + r) * d;
  };
  // K and V of the tile at k0; keys past n_keys and dims past d are zeros
  auto load_tile = [&](int k0, int stage) {
    float* dk = skv + stage * 2 * SK * LD;
    for (int i = threadIdx.x; i < SK * (DM / 4); i += S_THREADS) {
      const int j = i / (DM / 4), x = 4 * (i % (DM / 4));
      long long off = -1;
      if (k0 + j < n_keys && x < d)
        off = DOCS ? ((long long)(lo + k0 + j) * p.n_kv + g) * d : key_offset(p, b, g, k0 + j);
      copy16(dk + j * LD + x, off < 0 ? p.k : p.k + off + x, off >= 0);
      copy16(dk + (SK + j) * LD + x, off < 0 ? p.v : p.v + off + x, off >= 0);
    }
    copies_commit();
  };
  const int first = part * SK, step = p.splits * SK;  // this CTA's key tiles
  if (first < n_keys) load_tile(first, 0);
  for (int i = threadIdx.x; i < RT * (DM / 4); i += S_THREADS) {
    const int r = i / (DM / 4), x = 4 * (i % (DM / 4));
    *reinterpret_cast<float4*>(sq + r * LD + x) =
        r < rows && x < d ? *reinterpret_cast<const float4*>(p.q + row_off(r) + x)
                          : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float slope[RI];
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    const int r = ty + 16 * i;
    slope[i] = p.sc.slopes && r < rows ? p.sc.slopes[DOCS ? h0 : h0 + r] : 0.f;
  }
  float m[RI], l[RI], o[RI][DM / 16];
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int x = 0; x < DM / 16; ++x) o[i][x] = 0.f;
  }
  int stage = 0;
  for (int k0 = first; k0 < n_keys; k0 += step) {
    if (ST == 2 && k0 + step < n_keys) {
      load_tile(k0 + step, stage ^ 1);
      copies_wait<1>();
    } else {
      copies_wait<0>();
    }
    __syncthreads();
    const float* sk = skv + stage * 2 * SK * LD;
    const float* sv = sk + SK * LD;
    float s[RI][4];
#pragma unroll
    for (int i = 0; i < RI; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll 4
    for (int x = 0; x < DM; x += 4) {
      float4 kv[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4*>(sk + (tx + 16 * j) * LD + x);
#pragma unroll
      for (int i = 0; i < RI; ++i) {
        const float4 qv = *reinterpret_cast<const float4*>(sq + (ty + 16 * i) * LD + x);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s[i][j] = fmaf(qv.x, kv[j].x, fmaf(qv.y, kv[j].y, fmaf(qv.z, kv[j].z, fmaf(qv.w, kv[j].w, s[i][j]))));
      }
    }
#pragma unroll
    for (int i = 0; i < RI; ++i) {
      const int qi = DOCS ? q0 + ty + 16 * i : pos;
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = k0 + tx + 16 * j;
        float v = s[i][j] * p.sc.scale;
        if (p.sc.cap > 0.f) v = p.sc.cap * tanhf(v / p.sc.cap);
        if (p.sc.slopes) v -= slope[i] * fabsf((float)(qi - key));
        const bool keep = key < n_keys && (!DOCS || key <= qi || key < pre);
        s[i][j] = keep ? v : -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float mn = fmaxf(m[i], mx);
      const float mu = mn == -INFINITY ? 0.f : mn;  // no finite score yet: weights 0 (of NaN: NaN)
      const float f = expf(m[i] - mu);
      m[i] = mn;
      float ls = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float e = expf(s[i][j] - mu);
        ls += e;
        sp[(ty + 16 * i) * (SK + 4) + tx + 16 * j] = e;
      }
      l[i] = l[i] * f + ls;  // this thread's share of the row's sum
#pragma unroll
      for (int x = 0; x < DM / 16; ++x) o[i][x] *= f;
    }
    __syncwarp();  // a row's P is written and read by one half-warp
    const int nk = min(SK, n_keys - k0);
    // V rows past the last key are zeros, and so are their weights: whole fours
    for (int j = 0; j < nk; j += 4) {
      float4 pr[RI];
#pragma unroll
      for (int i = 0; i < RI; ++i) pr[i] = *reinterpret_cast<const float4*>(sp + (ty + 16 * i) * (SK + 4) + j);
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int x = 0; x < DM / 64; ++x) {
          const float4 vv = *reinterpret_cast<const float4*>(sv + (j + q) * LD + 4 * tx + 64 * x);
#pragma unroll
          for (int i = 0; i < RI; ++i) {
            const float w = q == 0 ? pr[i].x : q == 1 ? pr[i].y : q == 2 ? pr[i].z : pr[i].w;
            o[i][4 * x] = fmaf(w, vv.x, o[i][4 * x]);
            o[i][4 * x + 1] = fmaf(w, vv.y, o[i][4 * x + 1]);
            o[i][4 * x + 2] = fmaf(w, vv.z, o[i][4 * x + 2]);
            o[i][4 * x + 3] = fmaf(w, vv.w, o[i][4 * x + 3]);
          }
        }
    }
    __syncthreads();  // the stage may be overwritten
    if (ST == 2)
      stage ^= 1;
    else if (k0 + step < n_keys)
      load_tile(k0 + step, 0);
  }
#pragma unroll
  for (int i = 0; i < RI; ++i)
#pragma unroll
    for (int w = 8; w > 0; w >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
  if (p.splits > 1) {
    // The cluster's CTAs leave (O, maximum, sum) in their shared memory; row r is
    // merged by CTA r % splits, in the order of the parts.
    float* so = skv;            // [RT][DM], over the tiles
    float* sml = so + RT * DM;  // [RT][2]
    static_assert(RT * (DM + 2) <= ST * 2 * SK * LD, "the rows fit over the tiles");
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RI; ++i) {
      const int r = ty + 16 * i;
#pragma unroll
      for (int x = 0; x < DM / 64; ++x)
        *reinterpret_cast<float4*>(so + r * DM + 64 * x + 4 * tx) =
            make_float4(o[i][4 * x], o[i][4 * x + 1], o[i][4 * x + 2], o[i][4 * x + 3]);
      if (tx == 0) *reinterpret_cast<float2*>(sml + 2 * r) = make_float2(m[i], l[i]);
    }
    cluster_sync_all();
    if (ty % p.splits == part) {  // 16 is a multiple of the cluster's size
#pragma unroll
      for (int i = 0; i < RI; ++i) {
        const int r = ty + 16 * i;
        const uint32_t am = smem_u32(sml + 2 * r), ao = smem_u32(so + r * DM + 4 * tx);
        float M = -INFINITY, L = 0.f;
        for (int c = 0; c < p.splits; ++c) M = fmaxf(M, dsmem_ld2(dsmem_addr(am, c)).x);
#pragma unroll
        for (int x = 0; x < DM / 16; ++x) o[i][x] = 0.f;
        for (int c = 0; c < p.splits; ++c) {
          const float2 ml = dsmem_ld2(dsmem_addr(am, c));
          const float f = ml.x == -INFINITY ? 0.f : expf(ml.x - M);
          L = fmaf(ml.y, f, L);
#pragma unroll
          for (int x = 0; x < DM / 64; ++x) {
            const float4 v = dsmem_ld4(dsmem_addr(ao + 256 * x, c));
            o[i][4 * x] = fmaf(v.x, f, o[i][4 * x]);
            o[i][4 * x + 1] = fmaf(v.y, f, o[i][4 * x + 1]);
            o[i][4 * x + 2] = fmaf(v.z, f, o[i][4 * x + 2]);
            o[i][4 * x + 3] = fmaf(v.w, f, o[i][4 * x + 3]);
          }
        }
        l[i] = L;
      }
    }
    cluster_sync_all();  // nobody leaves while its rows are read
    if (ty % p.splits != part) return;
  }
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    const int r = ty + 16 * i;
    if (r >= rows) continue;
    float* dst = p.out + row_off(r);
#pragma unroll
    for (int x = 0; x < DM / 64; ++x) {
      const int dim = 64 * x + 4 * tx;
      if (dim >= d) continue;
      float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
      if (n_keys > 0)
        w = make_float4(o[i][4 * x] / l[i], o[i][4 * x + 1] / l[i], o[i][4 * x + 2] / l[i],
                        o[i][4 * x + 3] / l[i]);
      *reinterpret_cast<float4*>(dst + dim) = w;
    }
  }
}

template <int RI, int DM, bool DOCS>
cudaError_t prep() {
  return cudaFuncSetAttribute(attn_simt_kernel<RI, DM, DOCS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)SimtTile<RI, DM>::bytes);
}

template <int RI, bool DOCS>
cudaError_t run(const SimtParams& p, long long items, cudaStream_t st) {
  const dim3 grid((unsigned)(items * p.splits)), cluster(p.splits > 1 ? p.splits : 0, 1, 1);
  if (p.d <= 64)
    return launch_kc(attn_simt_kernel<RI, 64, DOCS>, grid, dim3(S_THREADS), SimtTile<RI, 64>::bytes,
                     st, cluster, p);
  if (p.d <= 128)
    return launch_kc(attn_simt_kernel<RI, 128, DOCS>, grid, dim3(S_THREADS), SimtTile<RI, 128>::bytes,
                     st, cluster, p);
  return launch_kc(attn_simt_kernel<RI, 256, DOCS>, grid, dim3(S_THREADS), SimtTile<RI, 256>::bytes,
                   st, cluster, p);
}

// CTAs that share an item's keys: doubled up to a cluster's 8 while there are
// fewer than three CTAs per SM and each keeps a tile of the longest (three per SM
// 50 us, two 61, six 68).
int simt_splits(long long items, int keys, int sm_count) {
  int s = 1;
  while (s < 8 && items * s < 3 * sm_count && keys >= 2 * s * SK) s *= 2;
  return s;
}

}  // namespace

cudaError_t attn_simt_prepare() {
  cudaError_t (*const all[])() = {prep<4, 64, true>,  prep<4, 128, true>,  prep<4, 256, true>,
                                  prep<2, 64, true>,  prep<2, 128, true>,  prep<2, 256, true>,
                                  prep<1, 64, false>, prep<1, 128, false>, prep<1, 256, false>};
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
  // 64-row tiles feed the FMA pipe best; where they leave SMs without work (fewer
  // than two per SM), 32 rows (700 rows, 8 heads, keys split: 57 us with 64, 50
  // with 32)
  const long long docs = std::min(a.n_docs, a.n_rows);
  auto tiles = [&](int rows) { return (a.n_rows / rows + docs) * a.n_q; };  // an upper bound
  const bool big = tiles(64) >= 2 * a.sm_count;
  p.splits = simt_splits(tiles(big ? 64 : 32), a.n_rows, a.sm_count);
  return big ? run<4, true>(p, tiles(64), st) : run<2, true>(p, tiles(32), st);
}

cudaError_t launch_shared_simt(const SharedArgs& a, cudaStream_t st) {
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
  p.row_chunks = (p.G + 15) / 16;
  const long long items = (long long)a.B * a.n_kv * p.row_chunks;
  p.splits = simt_splits(items, a.key_limit, a.sm_count);
  return run<1, false>(p, items, st);
}

}  // namespace llgb
