// Rows of a KV cache moved together: the accepted rows of a drafted tree
// (commit), and the keys that an eviction by accumulated attention weight keeps
// ("Llama2架构与推理全解析" §2.4: the cache that decode appends to).
//
//   commit: slot start + i  <-  slot start + path[i],   path ascending
//   evict : slot i          <-  slot kept[i], kept the ascending list of the first, the
//           recent and the heaviest of the other slots (equal weights: the lower slot)
//
// Both lists ascend, so list[i] >= i, and a cache is compacted in place without a
// second one: chunk c of the list writes slots that only chunks 0 .. c read, so a
// CTA that has loaded a chunk may store it (after a barrier), and the next chunk's
// loads need not wait for those stores. CTAs share nothing: each owns a slice of
// the columns of K or of V of one (layer, sequence, K/V head), down to 32 bytes (a
// sector) where there are few heads.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace llgb {

namespace {

constexpr int UNITS = 8;            // 16-byte units that a thread has in flight
constexpr int MAX_ROWS = 1024;      // rows of a chunk (256 threads x 8 units, slices of 2 units)

// Row of a slot within its layer; -1 (flagged) for a page outside the pool.
__device__ __forceinline__ int move_row(const CacheMoveArgs& a, int b, int g, int slot) {
  if (a.page_size == 0) return (b * a.n_kv + g) * a.capacity + slot;
  const int pi = slot / a.page_size;
  const int page = pi < a.max_pages ? a.page_table[(size_t)b * a.max_pages + pi] : -1;
  if (page < 0 || page >= a.n_pages) {
    flag(a.status, LLAMA_FLAG_PAGE_RANGE);
    return -1;
  }
  return (page * a.n_kv + g) * a.page_size + (slot - pi * a.page_size);
}

// Grid: slices, then K / V, K/V head, sequence, layer.
__global__ void cache_move_kernel(CacheMoveArgs a, int slices, int rows_chunk) {
  grid_dep_wait();
  grid_dep_launch();
  // (from, to) rows of a chunk, from < 0: no move; [3][rows_chunk], because beside a
  // thread that still stores a chunk another one may look up the chunk after the next
  extern __shared__ int2 moves[];
  const int T = blockDim.x;
  long long item = blockIdx.x;
  const int slice = (int)(item % slices);
  item /= slices;
  const int is_v = (int)(item & 1);
  item >>= 1;
  const int g = (int)(item % a.n_kv);
  item /= a.n_kv;
  const int b = (int)(item % a.B), l = (int)(item / a.B);
  const int upr = a.row_bytes / 16 / slices;  // units of a row of the slice
  // the list, and how much of it there is
  const int32_t* list;
  int n, base = 0, first = 0;
  if (a.path) {
    list = a.path + (size_t)b * a.list_ld;
    base = a.start[b];
    n = a.count[b];
    const bool ok = base >= 0 && n >= 0 && n <= a.list_ld;
    if (!ok && threadIdx.x == 0) flag(a.status, LLAMA_FLAG_POS_RANGE);
    n = base < 0 ? 0 : min(max(n, 0), a.list_ld);
  } else {
    list = a.kept + (((size_t)l * a.B + b) * a.n_kv + g) * a.list_ld;
    const int len = min(max(a.lens[b], 0), a.limit);
    n = len <= a.list_ld ? 0 : a.list_ld;  // nothing was dropped: nothing moves
    // the first slot that moves: list[i] == i up to there
    for (int step = (n + T - 1) / T, end = n; end > first && step > 0;) {
      const int i = first + threadIdx.x * step;
      const int same = __syncthreads_count(i < end && list[i] == i);
      if (same == 0) break;
      if (step == 1) {
        first += same;
        break;
      }
      first += (same - 1) * step;
      end = min(end, first + step);
      step = (end - first + T - 1) / T;
    }
  }
  // rows of the chunk at i0, into its half of `moves`
  auto look_up = [&](int i0, int2* to) {
    for (int r = threadIdx.x; r < rows_chunk; r += T) {
      const int i = i0 + r;
      int2 m = make_int2(-1, -1);
      if (i < n) {
        const int s = list[i];
        if (a.path && (s < i || (i > 0 && s <= list[i - 1]) || s >= a.limit - base)) {
          if (is_v == 0 && slice == 0) flag(a.status, LLAMA_FLAG_POS_RANGE);
        } else if (s != i && bc_ok(s > i && base + s < a.limit, a.status)) {
          m = make_int2(move_row(a, b, g, base + s), move_row(a, b, g, base + i));
          if (m.y < 0) m.x = -1;
        }
      }
      to[r] = m;
    }
  };
  uint4* cache = reinterpret_cast<uint4*>(is_v ? a.v : a.k) +
                 (size_t)(a.layer + l) * a.layer_rows * (a.row_bytes / 16) + (size_t)slice * upr;
  const int ld = a.row_bytes / 16;
  look_up(first, moves);
  __syncthreads();
  int part = 0;
  for (int i0 = first; i0 < n; i0 += rows_chunk) {
    const int2* mv = moves + part * rows_chunk;
    part = part == 2 ? 0 : part + 1;
    uint4 x[UNITS];
#pragma unroll
    for (int k = 0; k < UNITS; ++k) {
      const int u = threadIdx.x + k * T, r = u / upr;
      if (r < rows_chunk && mv[r].x >= 0) x[k] = cache[(size_t)mv[r].x * ld + (u - r * upr)];
    }
    if (i0 + rows_chunk < n) look_up(i0 + rows_chunk, moves + part * rows_chunk);
    __syncthreads();  // the chunk is read: its slots may be written
#pragma unroll
    for (int k = 0; k < UNITS; ++k) {
      const int u = threadIdx.x + k * T, r = u / upr;
      if (r < rows_chunk && mv[r].x >= 0) cache[(size_t)mv[r].y * ld + (u - r * upr)] = x[k];
    }
  }
}

// ---------------------------------------------------------------- which keys stay
constexpr int SEL_THREADS = 512, SEL_WARPS = SEL_THREADS / 32;
constexpr int BINS = 2048;

// Weights in ascending order as unsigned numbers: -0 as 0, NaN below everything.
__device__ __forceinline__ uint32_t order_of(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);
  return w != w ? 0u : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// One CTA per (layer, sequence, K/V head): the m-th largest of the weights between
// the first and the recent slots by three counting passes of 11, 11 and 10 bits,
// then one ordered pass that lists what stays and moves its weights.
__global__ void __launch_bounds__(SEL_THREADS) evict_select_kernel(EvictArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ uint32_t bins[BINS];
  __shared__ int part[2][SEL_WARPS];
  __shared__ uint32_t found[2];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int b = (int)(blockIdx.x / a.n_kv % a.B);
  const float* w = a.weights + (size_t)blockIdx.x * a.ld;
  float* out = a.weights_out + (size_t)blockIdx.x * a.ld;
  int32_t* kept = a.kept + (size_t)blockIdx.x * a.keep;
  const int len = a.lens[b], n = min(max(len, 0), a.limit);
  if (len != n && t == 0 && blockIdx.x % a.n_kv == 0) flag(a.status, LLAMA_FLAG_POS_RANGE);
  const bool all = n <= a.keep;
  const int lo = a.first, hi = n - a.recent;  // candidates
  uint32_t least = 0, ties = 0;               // the smallest weight that stays, and how many equal to it
  int want = a.keep - a.first - a.recent;
  if (!all && want > 0) {
    int shift = 21;
    uint32_t prefix = 0, mask = 0;
    for (int pass = 0; pass < 3; ++pass) {
      const int width = pass == 2 ? 10 : 11;
      for (int i = t; i < BINS; i += SEL_THREADS) bins[i] = 0;
      __syncthreads();
      for (int i = lo + t; i < hi; i += SEL_THREADS) {
        const uint32_t u = order_of(w[i]);
        if ((u & mask) == prefix) atomicAdd(&bins[(u >> shift) & ((1u << width) - 1u)], 1u);
      }
      __syncthreads();
      // suffix sums from the largest bin on: thread t has bins BINS - 1 - 4 t and the three below
      const int top = BINS - 1 - 4 * t;
      uint32_t c[4], sum = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) sum += c[k] = bins[top - k];
      uint32_t upto = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      if (lane == 31) part[0][warp] = (int)upto;
      __syncthreads();
      uint32_t before = upto - sum;
      for (int k = 0; k < warp; ++k) before += (uint32_t)part[0][k];
      if (before < (uint32_t)want && before + sum >= (uint32_t)want) {
        int k = 0;
        while (before + c[k] < (uint32_t)want) before += c[k++];
        found[0] = (uint32_t)(top - k);
        found[1] = before;
      }
      __syncthreads();
      prefix |= found[0] << shift;
      mask |= ((1u << width) - 1u) << shift;
      want -= (int)found[1];
      shift = pass == 0 ? 10 : 0;
      __syncthreads();
    }
    least = prefix;
    ties = (uint32_t)want;
  }
  // what stays, in order; a slot's weight moves to a slot that was read before or with it
  const bool none = a.keep - a.first - a.recent == 0;
  int done = 0, tied = 0;  // listed so far, equal to `least` so far
  for (int i0 = 0; i0 < n; i0 += SEL_THREADS) {
    const int i = i0 + t;
    const float x = i < n ? w[i] : 0.f;
    bool stays = i < n && (all || i < lo || i >= hi), tie = false;
    if (i < n && !stays && !none) {
      const uint32_t u = order_of(x);
      stays = u > least;
      tie = u == least;
    }
    const uint32_t mt = __ballot_sync(0xffffffffu, tie);
    if (lane == 0) part[0][warp] = __popc(mt);
    __syncthreads();  // (also: every weight of these slots is read)
    int rank = tied + __popc(mt & ((1u << lane) - 1u));
    for (int k = 0; k < SEL_WARPS; ++k) {
      if (k < warp) rank += part[0][k];
      tied += part[0][k];
    }
    stays |= tie && rank < (int)ties;
    const uint32_t ms = __ballot_sync(0xffffffffu, stays);
    if (lane == 0) part[1][warp] = __popc(ms);
    __syncthreads();
    int at = done + __popc(ms & ((1u << lane) - 1u));
    for (int k = 0; k < SEL_WARPS; ++k) {
      if (k < warp) at += part[1][k];
      done += part[1][k];
    }
    if (stays && bc_ok(at < a.keep && at <= i, a.status)) {
      kept[at] = i;
      out[at] = x;
    }
  }
  __syncthreads();
  for (int i = done + t; i < a.keep; i += SEL_THREADS) kept[i] = -1;
  for (long long i = done + t; i < a.ld; i += SEL_THREADS) out[i] = 0.f;
}

}  // namespace

cudaError_t launch_cache_move(const CacheMoveArgs& a, cudaStream_t st) {
  const int upr = a.row_bytes / 16;
  const long long items = (long long)a.layers * a.B * a.n_kv * 2;
  int slices = 1, T = 256;
  if (a.path) {
    // a few rows: as many threads as the longest path needs
    while (T > 32 && (long long)T / 2 * UNITS >= (long long)a.list_ld * upr) T /= 2;
  } else {
    while (upr / slices % 2 == 0 && upr / slices > 2 && items * slices < 4 * a.sm_count) slices *= 2;
  }
  const int rows = std::min(MAX_ROWS, std::max(1, T * UNITS / (upr / slices)));
  return launch_k(cache_move_kernel, dim3((unsigned)(items * slices)), dim3(T), 3 * rows * sizeof(int2), st, 0, a,
                  slices, rows);
}

cudaError_t launch_evict_select(const EvictArgs& a, cudaStream_t st) {
  return launch_k(evict_select_kernel, dim3((unsigned)((long long)a.layers * a.B * a.n_kv)), dim3(SEL_THREADS), 0, st,
                  0, a);
}

}  // namespace llgb
