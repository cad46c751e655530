// Attention with capped or biased scores on the CUDA cores, for fp32 models
// and any head_dim up to 256: packed documents (two-way prefix, causal rest)
// and decode over a cache with a shared prefix.
//
//   x = scale q.k;  s = (cap tanh(x / cap) or x) - slope |i - j|;  softmax;  sum p v
//
// One CTA of 256 threads per (RT query rows, K/V source): documents take RT
// rows of one head, decode the query heads of one K/V head and sequence.
// Tiles of 64 keys pass through shared memory once; thread (ty, tx) computes
// the scores of rows ty + 16 i and keys tx + 16 j, the row maxima and sums
// are folded over the 16 threads of a row with butterflies (the running
// maximum and sum of an online softmax, in fp32), P goes through shared
// memory, and the same thread accumulates its rows' dims tx*4 + 64 m. Exact
// fp32 arithmetic throughout (exp and tanh of the CUDA math library).
// Bound by the fp32 FMA pipe and the shared-memory reads that feed it.
#include <algorithm>

#include "attn_score.cuh"
#include "internal.h"

namespace llgb {

namespace {

constexpr int SK = 64;        // keys per tile
constexpr int S_THREADS = 256;

template <typename T>
struct SimtParams {
  const T *q, *k, *v;
  T* out;
  int n_q, n_kv, G, d;
  ScoreArgs sc;
  uint32_t* status;
  // documents
  const int32_t *cu_rows, *prefix_len;
  int n_rows, n_docs;
  // decode
  const int32_t *positions, *page_table;
  int layer, page_size, capacity, batch_cap, n_pages, max_pages, key_limit, shared_len, shared_seq;
  int row_chunks;  // chunks of RT heads per K/V head
};

// Element offset of key j of sequence b, K/V head g in the cache; -1 (flagged)
// for a page outside the pool.
template <typename T>
__device__ __forceinline__ long long key_offset(const SimtParams<T>& p, int b, int g, int j) {
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

// RT: query rows of a CTA (16 RI); DM: head_dim rounded up to 64, 128 or 256.
template <typename T, int RI, int DM, bool DOCS>
__global__ void __launch_bounds__(S_THREADS) attn_simt_kernel(SimtParams<T> p) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int RT = 16 * RI, LD = DM + 4;
  extern __shared__ __align__(16) float sm[];
  float* sq = sm;                // [RT][LD]
  float* sk = sq + RT * LD;      // [SK][LD], K then V of a tile
  float* sp = sk + SK * LD;      // [RT][SK + 4]
  if (!bc_smem(sm, (uint32_t)((RT + SK) * LD + RT * (SK + 4)) * 4, 16,
               threadIdx.x == 0 ? p.status : nullptr))
    return;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int d = p.d;
  // which rows
  int b, g, h0, lo = 0, n = 0, q0 = 0, rows, n_keys, pre = 0, pos = 0;
  if (DOCS) {
    const int h = blockIdx.x % p.n_q;
    int tile;
    DocCursor cursor;
    if (!find_tile(p.cu_rows, p.n_docs, p.n_rows, RT, blockIdx.x / p.n_q, p.status, cursor, b, tile,
                   lo, n))
      return;
    h0 = h;
    g = h / p.G;
    q0 = tile * RT;
    rows = min(RT, n - q0);
    pre = p.prefix_len ? min(max(p.prefix_len[b], 0), n) : 0;
    n_keys = max(q0 + rows, pre);
  } else {
    const int c = blockIdx.x % p.row_chunks;
    g = (blockIdx.x / p.row_chunks) % p.n_kv;
    b = blockIdx.x / (p.row_chunks * p.n_kv);
    h0 = g * p.G + c * RT;
    rows = min(RT, p.G - c * RT);
    pos = p.positions[b];
    n_keys = pos + 1;
    if (pos < 0 || pos >= p.key_limit) {
      if (threadIdx.x == 0) flag(p.status, LLAMA_FLAG_POS_RANGE);
      n_keys = pos < 0 ? 0 : p.key_limit;
    }
  }
  // element offset of row r (documents: packed row, one head; decode: one row, head h0 + r)
  auto row_off = [&](int r) -> size_t {
    return DOCS ? ((size_t)(lo + q0 + r) * p.n_q + h0) * d : ((size_t)b * p.n_q + h0 + r) * d;
  };
  for (int i = threadIdx.x; i < RT * DM; i += S_THREADS) {
    const int r = i / DM, x = i % DM;
    sq[r * LD + x] = r < rows && x < d ? to_f32(p.q[row_off(r) + x]) : 0.f;
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
  auto load_tile = [&](const T* src, int k0) {  // keys past n_keys are zeros
    for (int i = threadIdx.x; i < SK * (DM / 4); i += S_THREADS) {
      const int j = i / (DM / 4), x = 4 * (i % (DM / 4));
      float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k0 + j < n_keys && x < d) {
        const long long off = DOCS ? ((long long)(lo + k0 + j) * p.n_kv + g) * d
                                   : key_offset(p, b, g, k0 + j);
        if (off >= 0) {
          const T* s = src + off + x;
          w = make_float4(to_f32(s[0]), to_f32(s[1]), to_f32(s[2]), to_f32(s[3]));
        }
      }
      *reinterpret_cast<float4*>(sk + j * LD + x) = w;
    }
  };
  for (int k0 = 0; k0 < n_keys; k0 += SK) {
    __syncthreads();
    load_tile(p.k, k0);
    __syncthreads();
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
      const float f = mn == -INFINITY ? 1.f : expf(m[i] - mn);
      m[i] = mn;
      float ls = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float e = mn == -INFINITY ? 0.f : expf(s[i][j] - mn);
        ls += e;
        sp[(ty + 16 * i) * (SK + 4) + tx + 16 * j] = e;
      }
      l[i] = l[i] * f + ls;  // this thread's share of the row's sum
#pragma unroll
      for (int x = 0; x < DM / 16; ++x) o[i][x] *= f;
    }
    __syncthreads();
    load_tile(p.v, k0);
    __syncthreads();
    const int nk = min(SK, n_keys - k0);
    for (int j = 0; j < nk; ++j) {
      float pr[RI];
#pragma unroll
      for (int i = 0; i < RI; ++i) pr[i] = sp[(ty + 16 * i) * (SK + 4) + j];
#pragma unroll
      for (int x = 0; x < DM / 64; ++x) {
        const float4 vv = *reinterpret_cast<const float4*>(sk + j * LD + 4 * tx + 64 * x);
#pragma unroll
        for (int i = 0; i < RI; ++i) {
          o[i][4 * x] = fmaf(pr[i], vv.x, o[i][4 * x]);
          o[i][4 * x + 1] = fmaf(pr[i], vv.y, o[i][4 * x + 1]);
          o[i][4 * x + 2] = fmaf(pr[i], vv.z, o[i][4 * x + 2]);
          o[i][4 * x + 3] = fmaf(pr[i], vv.w, o[i][4 * x + 3]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    float lt = l[i];
#pragma unroll
    for (int w = 8; w > 0; w >>= 1) lt += __shfl_xor_sync(0xffffffffu, lt, w);
    const int r = ty + 16 * i;
    if (r >= rows) continue;
    T* dst = p.out + row_off(r);
#pragma unroll
    for (int x = 0; x < DM / 64; ++x)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int dim = 64 * x + 4 * tx + c;
        if (dim < d) dst[dim] = from_f32<T>(n_keys > 0 ? o[i][4 * x + c] / lt : 0.f);
      }
  }
}

template <int RI, int DM>
constexpr size_t simt_smem() {
  return (size_t)((16 * RI + SK) * (DM + 4) + 16 * RI * (SK + 4)) * sizeof(float);
}

template <typename T, int RI, bool DOCS>
cudaError_t prep() {
  cudaError_t e = cudaFuncSetAttribute(attn_simt_kernel<T, RI, 64, DOCS>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)simt_smem<RI, 64>());
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(attn_simt_kernel<T, RI, 128, DOCS>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)simt_smem<RI, 128>());
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(attn_simt_kernel<T, RI, 256, DOCS>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)simt_smem<RI, 256>());
  return e;
}

template <typename T, int RI, bool DOCS>
cudaError_t run(const SimtParams<T>& p, unsigned grid, cudaStream_t st) {
  if (p.d <= 64)
    return launch_k(attn_simt_kernel<T, RI, 64, DOCS>, dim3(grid), dim3(S_THREADS),
                    simt_smem<RI, 64>(), st, 0, p);
  if (p.d <= 128)
    return launch_k(attn_simt_kernel<T, RI, 128, DOCS>, dim3(grid), dim3(S_THREADS),
                    simt_smem<RI, 128>(), st, 0, p);
  return launch_k(attn_simt_kernel<T, RI, 256, DOCS>, dim3(grid), dim3(S_THREADS),
                  simt_smem<RI, 256>(), st, 0, p);
}

template <typename T>
cudaError_t docs_simt(const DocsArgs& a, cudaStream_t st) {
  SimtParams<T> p{};
  p.q = (const T*)a.q;
  p.k = (const T*)a.k;
  p.v = (const T*)a.v;
  p.out = (T*)a.out;
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
  const long long tiles = a.n_rows / 64 + (long long)std::min(a.n_docs, a.n_rows);  // an upper bound
  return run<T, 4, true>(p, (unsigned)(tiles * a.n_q), st);
}

template <typename T>
cudaError_t shared_simt(const SharedArgs& a, cudaStream_t st) {
  SimtParams<T> p{};
  p.q = (const T*)a.q;
  p.k = (const T*)a.k_cache;
  p.v = (const T*)a.v_cache;
  p.out = (T*)a.out;
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
  return run<T, 1, false>(p, (unsigned)((long long)a.B * a.n_kv * p.row_chunks), st);
}

}  // namespace

cudaError_t attn_simt_prepare() {
  cudaError_t e = prep<float, 4, true>();
  if (e == cudaSuccess) e = prep<float, 1, false>();
  if (e == cudaSuccess) e = prep<bf16, 4, true>();
  if (e == cudaSuccess) e = prep<bf16, 1, false>();
  return e;
}

cudaError_t launch_docs_simt(int dtype, const DocsArgs& a, cudaStream_t st) {
  return dtype == LLAMA_F32 ? docs_simt<float>(a, st) : docs_simt<bf16>(a, st);
}
cudaError_t launch_shared_simt(int dtype, const SharedArgs& a, cudaStream_t st) {
  return dtype == LLAMA_F32 ? shared_simt<float>(a, st) : shared_simt<bf16>(a, st);
}

}  // namespace llgb
