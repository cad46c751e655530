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
// loads need not wait for those stores. CTAs share no row they move.
//
// Bound by the bytes of the rows, read and written once each.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace llgb {

namespace {

constexpr int MOVE_THREADS = 256;

// Row, within its layer, of a slot's K/V head 0 (the heads are slot_step rows apart); -1
// (flagged) for a page outside the pool.
__device__ __forceinline__ int move_row(const CacheMoveArgs& a, int b, int slot) {
  if (a.page_size == 0) return b * a.n_kv * a.capacity + slot;
  const int pi = slot / a.page_size;
  const int page = pi < a.max_pages ? a.page_table[(size_t)b * a.max_pages + pi] : -1;
  if (page < 0 || page >= a.n_pages) {
    flag(a.status, LLAMA_FLAG_PAGE_RANGE);
    return -1;
  }
  return page * a.n_kv * a.page_size + (slot - pi * a.page_size);
}

// Commit. Grid: groups of `heads` K/V heads, sequences, runs of layers. A sequence's path
// and pages are the same for all layers and heads, K and V, so a block looks them up once
// for as many heads as fill its threads and walks its layers: while it waits for
// one layer's rows to store them, the next one's are on their way. A path is mostly one
// chunk. Bound by the latency of look-ups and rows, so by how many blocks are resident: 64
// sequences, 32 layers of 32 E4M3 heads (66 MB read and written), 8 blocks per SM with 2 units a
// thread 28.1 us, 4 with 4 32.1, 3 with 4 35.7, 8 with 1 38.
constexpr int COMMIT_UNITS = 2;
__global__ void __launch_bounds__(MOVE_THREADS, 8) cache_commit_kernel(CacheMoveArgs a, int heads, int rows_chunk,
                                                                       int run) {
  grid_dep_wait();
  grid_dep_launch();
  extern __shared__ int2 moves[];  // [rows_chunk] (from, to) rows of K/V head 0; from < 0: no move
  const int b = blockIdx.y, l0 = blockIdx.z * run, l1 = min(a.layers, l0 + run);
  const int g0 = blockIdx.x * heads, n_heads = min(heads, a.n_kv - g0);
  const int upr = a.row_bytes / 16, step = a.page_size == 0 ? a.capacity : a.page_size;
  const bool report = blockIdx.x == 0 && l0 == 0;
  const int base = a.start[b], len = a.count[b];
  if ((base < 0 || len < 0 || len > a.list_ld) && report && threadIdx.x == 0) flag(a.status, LLAMA_FLAG_POS_RANGE);
  const int n = base < 0 ? 0 : min(max(len, 0), a.list_ld);
  const int32_t* path = a.path + (size_t)b * a.list_ld;
  const size_t layer_units = a.layer_rows * upr;
  for (int i0 = 0; i0 < n; i0 += rows_chunk) {
    const int rows = min(rows_chunk, n - i0), per_head = rows * upr;
    if (i0 > 0) __syncthreads();
    for (int r = threadIdx.x; r < rows; r += MOVE_THREADS) {
      const int i = i0 + r, s = path[i], before = i > 0 ? path[i - 1] : -1;
      int2 m = make_int2(-1, -1);
      if (s < i || s <= before || s >= a.limit - base) {
        if (report) flag(a.status, LLAMA_FLAG_POS_RANGE);
      } else if (s != i) {
        m = make_int2(move_row(a, b, base + s), move_row(a, b, base + i));
        if (m.y < 0) m.x = -1;
      }
      moves[r] = m;
    }
    __syncthreads();
    // Unit u = (K / V, head, row, 16 bytes): a thread's units are MOVE_THREADS apart, so one
    // division finds the first and additions the others. Its places in the first layer:
    const int step_hk = MOVE_THREADS / per_head, step_r = (MOVE_THREADS - step_hk * per_head) / upr,
              step_c = MOVE_THREADS - step_hk * per_head - step_r * upr;
    int hk = threadIdx.x / per_head, r = (threadIdx.x - hk * per_head) / upr;
    int c = threadIdx.x - hk * per_head - r * upr;
    const uint4* from[COMMIT_UNITS];
    int to[COMMIT_UNITS];  // rows further down; 0: no move
#pragma unroll
    for (int k = 0; k < COMMIT_UNITS; ++k) {
      from[k] = nullptr;
      to[k] = 0;
      if (hk < 2 * n_heads && moves[r].x >= 0) {
        const int2 m = moves[r];
        const int v = hk >= n_heads, g = g0 + hk - (v ? n_heads : 0);
        const size_t row = (size_t)m.x + (size_t)g * step;
        if (bc_ok(row < a.layer_rows && (size_t)m.y + (size_t)g * step < a.layer_rows, a.status)) {
          from[k] = reinterpret_cast<const uint4*>(v ? a.v : a.k) + (a.layer + l0) * layer_units + row * upr + c;
          to[k] = m.y - m.x;
        }
      }
      c += step_c;
      r += step_r;
      hk += step_hk;
      if (c >= upr) {
        c -= upr;
        ++r;
      }
      if (r >= rows) {
        r -= rows;
        ++hk;
      }
    }
    uint4 x[2][COMMIT_UNITS];
    auto load = [&](int l, uint4* y) {
#pragma unroll
      for (int k = 0; k < COMMIT_UNITS; ++k)
        if (from[k]) y[k] = from[k][(l - l0) * layer_units];
    };
    auto store = [&](int l, const uint4* y) {
      __syncthreads();  // every thread has read its rows of this layer: they may be written
#pragma unroll
      for (int k = 0; k < COMMIT_UNITS; ++k)
        if (from[k]) const_cast<uint4*>(from[k])[(l - l0) * layer_units + (long long)to[k] * upr] = y[k];
    };
    load(l0, x[0]);
    for (int l = l0; l < l1; l += 2) {
      if (l + 1 < l1) load(l + 1, x[1]);
      store(l, x[0]);
      if (l + 1 == l1) break;
      if (l + 2 < l1) load(l + 2, x[0]);
      store(l + 1, x[1]);
    }
  }
}

// Evict: the kept rows of one K/V head, moved by a CTA of T threads, U units each at a
// time: of each row `cols` units from unit col0 on, of K's row and, behind it, V's. Slots
// look up their rows a chunk ahead, and the list is read two chunks ahead, so that a
// chunk waits for one latency. moves: [3][rows_chunk], because beside a thread that still
// stores a chunk another one may look up the chunk after the next.
template <int T, int U>
__device__ __forceinline__ void move_kept(const CacheMoveArgs& a, int2* moves, const int32_t* list, int l, int b, int g,
                                          int col0, int cols) {
  const int rows_chunk = T / cols * U;
  constexpr int MINE = (T / 2 * U + T - 1) / T;  // rows of a chunk that a thread looks up, with 2 columns
  const int n = a.list_ld, ld = a.row_bytes / 16;
  // the first slot that moves: list[i] == i up to there (two loads in a row; a few
  // chunks in which nothing moves are done sooner)
  int first = 0;
  if (n > 4 * rows_chunk) for (int step = (n + T - 1) / T, end = n; end > first;) {
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
  const int head = g * (a.page_size == 0 ? a.capacity : a.page_size);
  int slot[MINE];
  auto read_list = [&](int i0) {
#pragma unroll
    for (int k = 0; k < MINE; ++k) {
      const int r = threadIdx.x + k * T;
      slot[k] = r < rows_chunk && i0 + r < n ? list[i0 + r] : -1;
    }
  };
  // (from, to) rows of the chunk at i0, whose slots were read, into its part of `moves`; from < 0: no move
  auto look_up = [&](int i0, int2* to) {
#pragma unroll
    for (int k = 0; k < MINE; ++k) {
      const int r = threadIdx.x + k * T, i = i0 + r, s = slot[k];
      if (r >= rows_chunk) break;
      int2 m = make_int2(-1, -1);
      if (s > i && bc_ok(s < a.limit, a.status)) {
        m = make_int2(move_row(a, b, s), move_row(a, b, i));
        m = m.x < 0 || m.y < 0 ? make_int2(-1, -1) : make_int2(m.x + head, m.y + head);
        if (!bc_ok((size_t)max(m.x, m.y) < a.layer_rows || m.x < 0, a.status)) m.x = -1;
      }
      to[r] = m;
    }
  };
  // a thread's units: one column of the rows r0, r0 + step_r, ..
  const int step_r = T / cols, r0 = threadIdx.x / cols, col = col0 + (int)threadIdx.x - r0 * cols;
  uint4* at = reinterpret_cast<uint4*>(col < ld ? a.k : a.v) + (size_t)(a.layer + l) * a.layer_rows * ld +
              (col < ld ? col : col - ld);
  read_list(first);
  look_up(first, moves);
  read_list(first + rows_chunk);
  __syncthreads();
  int part = 0;
  for (int i0 = first; i0 < n; i0 += rows_chunk) {
    const int2* mv = moves + part * rows_chunk;
    part = part == 2 ? 0 : part + 1;
    int2 m[U];
    uint4 x[U];
#pragma unroll
    for (int k = 0; k < U; ++k) m[k] = r0 < step_r ? mv[r0 + k * step_r] : make_int2(-1, -1);
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (m[k].x >= 0) x[k] = at[(size_t)m[k].x * ld];
    look_up(i0 + rows_chunk, moves + part * rows_chunk);
    read_list(i0 + 2 * rows_chunk);
    __syncthreads();  // the chunk is read: its slots may be written
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (m[k].x >= 0) at[(size_t)m[k].y * ld] = x[k];
  }
}

// ---------------------------------------------------------------- which keys stay
constexpr int SPAN = 8192;                    // weights that a CTA holds
constexpr int BINS = 2048;

// Weights in ascending order as unsigned numbers: -0 as 0, NaN below everything.
__device__ __forceinline__ uint32_t order_of(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);
  return w != w ? 0u : u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}

// What stays of one (layer, sequence, K/V head), by a CTA of T threads: the m-th largest of the weights
// between the first and the recent slots, by counting how many have each value of
// their upper 11 bits; those that share the found ones, if few, are compared with each
// other, else counted by the next 11 and the last 10 bits; then one ordered pass that
// lists what stays and moves its weights. A
// warp owns consecutive slots, 32 at a time, so ranks within it are bit counts and
// the warps exchange one pair of counts. Up to 8192 weights are read once and stay in
// shared memory; longer lists are read again for every pass, 8192 at a time. Bound by
// the instructions per weight and, where there are few heads, by the barriers.
constexpr int LISTED = 256;
template <int T>
__device__ __forceinline__ void select_kept(const EvictArgs& a, float* held, int item) {
  constexpr int WARPS = T / 32, PER = BINS / T;
  static_assert((SPAN + BINS + BINS / 8 + LISTED + 2 * WARPS + 4) * 4 <= 48 * 1024, "without an opt-in");
  static_assert(SPAN / T <= 32, "a thread's slots of a span are the bits of a word");
  __shared__ uint32_t bins[BINS + BINS / 8];  // bin i at i + i / 8: a thread's bins lie in a row, and conflict-free
  auto bin = [&](uint32_t i) -> uint32_t& { return bins[i + (i >> 3)]; };
  __shared__ uint32_t listed[LISTED];
  __shared__ int2 part[WARPS];
  __shared__ uint32_t found[2], n_listed;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const uint32_t below = (1u << lane) - 1u;
  const int b = item / a.n_kv % a.B;
  const float* w = a.weights + (size_t)item * a.ld;
  float* out = a.weights_out + (size_t)item * a.ld;
  int32_t* kept = a.kept + (size_t)item * a.keep;
  const int len = a.lens[b], n = min(max(len, 0), a.limit);
  if (len != n && t == 0 && item % a.n_kv == 0) flag(a.status, LLAMA_FLAG_POS_RANGE);
  const bool all = n <= a.keep;
  const int lo = a.first, hi = n - a.recent;  // candidates
  auto load = [&](int s0) {
#pragma unroll 8
    for (int i = t; i < min(SPAN, n - s0); i += T) held[i] = w[s0 + i];
    __syncthreads();
  };
  // f for every candidate's order, a span at a time
  auto candidates = [&](bool again, auto&& f) {
#pragma unroll 1
    for (int s0 = 0; s0 < n; s0 += SPAN) {
      if (n > SPAN && (s0 > 0 || again)) {
        __syncthreads();
        load(s0);
      }
      const int to = min(SPAN, hi - s0);
#pragma unroll 4
      for (int i = max(0, lo - s0) + t; i < to; i += T) f(order_of(held[i]));
    }
  };
  // sums over the warps in front of this one, and over all
  auto across = [&](int2 mine, int2& all) {
    if (lane == 0) part[warp] = mine;
    __syncthreads();
    const int2 c = lane < WARPS ? part[lane] : make_int2(0, 0);
    int2 up = c;
#pragma unroll
    for (int o = 1; o < WARPS; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, up.x, o), y = __shfl_up_sync(0xffffffffu, up.y, o);
      if (lane >= o) {
        up.x += x;
        up.y += y;
      }
    }
    all = make_int2(__shfl_sync(0xffffffffu, up.x, WARPS - 1), __shfl_sync(0xffffffffu, up.y, WARPS - 1));
    return make_int2(__shfl_sync(0xffffffffu, up.x - c.x, warp), __shfl_sync(0xffffffffu, up.y - c.y, warp));
  };
  int want = a.keep - a.first - a.recent;
  // the bin that the want-th largest is in; want becomes its rank there; the bins are 0 again
  auto find = [&] {
    __syncthreads();
    // suffix sums from the largest bin on: thread t has the PER bins below BINS - PER t
    const int top = BINS - 1 - PER * t;
    uint32_t c[PER], sum = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      sum += c[k] = bin(top - k);
      bin(top - k) = 0;
    }
    uint32_t upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    int2 total;
    const int2 mine = make_int2((int)__shfl_sync(0xffffffffu, upto, 31), 0);
    uint32_t before = upto - sum + (uint32_t)across(mine, total).x;
    if (before < (uint32_t)want && before + sum >= (uint32_t)want) {
      int k = 0;
      while (before + c[k] < (uint32_t)want) before += c[k++];
      found[0] = (uint32_t)(top - k);
      found[1] = before;
    }
    __syncthreads();
    want -= (int)found[1];
    return found[0];
  };
  for (int i = t; i < BINS + BINS / 8; i += T) bins[i] = 0;
  if (t == 0) n_listed = 0;
  load(0);
  uint32_t least = 0, ties = 0;  // the smallest weight that stays, and how many equal to it
  if (!all && want > 0) {
    candidates(false, [&](uint32_t u) { atomicAdd(&bin(u >> 21), 1u); });
    const uint32_t upper = find();
    candidates(true, [&](uint32_t u) {
      if (u >> 21 != upper) return;
      const uint32_t at = atomicAdd(&n_listed, 1u);
      if (at < LISTED) listed[at] = u;
    });
    __syncthreads();
    if (n_listed <= LISTED) {  // each against all: whose rank is want?
      const int m = (int)n_listed;
      if (t < m) {
        const uint32_t u = listed[t];
        int above = 0, equal = 0;
        for (int i = 0; i < m; ++i) {
          above += listed[i] > u;
          equal += listed[i] == u;
        }
        if (above < want && want <= above + equal) {  // the same from every thread that has this weight
          found[0] = u;
          found[1] = (uint32_t)above;
        }
      }
      __syncthreads();
      least = found[0];
      want -= (int)found[1];
    } else {
      candidates(true, [&](uint32_t u) {
        if (u >> 21 == upper) atomicAdd(&bin((u >> 10) & 2047u), 1u);
      });
      const uint32_t middle = upper << 11 | find();
      candidates(true, [&](uint32_t u) {
        if (u >> 10 == middle) atomicAdd(&bin(u & 1023u), 1u);
      });
      least = middle << 10 | find();
    }
    ties = (uint32_t)want;
  }
  // What stays, in order: the spans one after the other, the warps of a span in parallel.
  // A weight moves to a slot that its span or an earlier one holds, and those were read.
  const bool none = a.keep - a.first - a.recent == 0;
  int done = 0, tied = 0;  // listed so far, equal to `least` so far
#pragma unroll 1
  for (int s0 = 0; s0 < n; s0 += SPAN) {
    if (n > SPAN) {
      __syncthreads();
      load(s0);
    }
    const int m = min(SPAN, n - s0), own = (m + T - 1) / T;  // 32-slot steps of a warp
    const int at0 = warp * 32 * own + lane;
    uint32_t sure = 0, tie = 0;  // bit k: slot at0 + 32 k stays whatever the ties, is one
#pragma unroll 4
    for (int k = 0; k < own; ++k) {
      const int i = at0 + 32 * k;
      if (i >= m) break;
      const bool always = all || s0 + i < lo || s0 + i >= hi;
      const uint32_t u = order_of(held[i]);
      sure |= (uint32_t)(always || (!none && u > least)) << k;
      tie |= (uint32_t)(!always && !none && u == least) << k;
    }
    int2 sums;
    const int2 front = across(make_int2(__reduce_add_sync(0xffffffffu, __popc(sure)),
                                        __reduce_add_sync(0xffffffffu, __popc(tie))), sums);
    // the ties that stay are the first ones: `ties` of them in all
    int rank = tied + front.y, at = done + front.x + max(0, min(front.y, (int)ties - tied));
#pragma unroll 4
    for (int k = 0; k < own; ++k) {
      bool s = sure >> k & 1u;
      const uint32_t me = __ballot_sync(0xffffffffu, tie >> k & 1u);
      if (me) {
        s = s || ((tie >> k & 1u) && rank + __popc(me & below) < (int)ties);
        rank += __popc(me);
      }
      const uint32_t ms = __ballot_sync(0xffffffffu, s);
      const int i = at0 + 32 * k, to = at + __popc(ms & below);
      if (s && bc_ok(to < a.keep && to <= s0 + i, a.status)) {
        kept[to] = s0 + i;
        out[to] = held[i];
      }
      at += __popc(ms);
    }
    done += sums.x + max(0, min(sums.y, (int)ties - tied));
    tied += sums.y;
    __syncthreads();  // `part` and `held` have been read
  }
  for (long long i = done + t; i < a.keep; i += T) kept[i] = -1;
  for (long long i = done + t; i < a.ld; i += T) out[i] = 0.f;
}

// A head's keys selected and moved by a CTA, so that one CTA's counting and the others'
// moves share an SM; or, where heads are few, by a cluster of `ctas`: its first CTA selects,
// and each moves a slice of the columns, down to 32 bytes (a sector).
template <int T, int U>
__global__ void __launch_bounds__(T, 1024 / T) evict_kernel(EvictArgs e, CacheMoveArgs a, int ctas) {
  grid_dep_wait();
  grid_dep_launch();
  extern __shared__ __align__(16) float held[];  // [min(SPAN, most slots)]; then the moves, int2 [3][rows of a chunk]
  const int item = blockIdx.x / ctas, rank = blockIdx.x - item * ctas, b = item / a.n_kv % a.B;
  const int cols = a.row_bytes / 8 / ctas;
  if (!bc_smem(held, max(min(SPAN, e.limit) * 4, 3 * (T / cols * U) * 8), 16, threadIdx.x == 0 ? a.status : nullptr))
    return;  // a cluster's CTAs all do
  if (rank == 0) select_kept<T>(e, held, item);
  if (ctas > 1)
    cluster_sync_all();  // the list is written
  else
    __syncthreads();     // and `held` free
  if (min(max(a.lens[b], 0), a.limit) <= a.list_ld) return;  // nothing was dropped: nothing moves
  move_kept<T, U>(a, reinterpret_cast<int2*>(held), a.kept + (size_t)item * a.list_ld, item / a.n_kv / a.B, b,
                  item % a.n_kv, rank * cols, cols);
}

}  // namespace

cudaError_t launch_cache_commit(const CacheMoveArgs& a, cudaStream_t st) {
  const int upr = a.row_bytes / 16, room = MOVE_THREADS * COMMIT_UNITS / (2 * upr);  // rows of one head's K and V
  const int heads = std::max(1, std::min(room / a.list_ld, a.n_kv)), rows = std::min(a.list_ld, room / heads);
  const int groups = (a.n_kv + heads - 1) / heads;
  // runs of layers that give every SM twice its 8 blocks (once 30.1 instead of 28.1 us in the
  // same case; four times 28.7, but 11.8 instead of 10.0 with 8 heads)
  const long long pairs = (long long)groups * a.B;
  const int runs = (int)std::min<long long>(a.layers, (16 * a.sm_count + pairs - 1) / pairs);
  const int run = (a.layers + runs - 1) / runs;
  return launch_k(cache_commit_kernel, dim3(groups, a.B, (a.layers + run - 1) / run), dim3(MOVE_THREADS),
                  rows * sizeof(int2), st, 0, a, heads, rows, run);
}

template <int T, int U>
static cudaError_t run_evict(const EvictArgs& e, const CacheMoveArgs& a, int items, int ctas, cudaStream_t st) {
  const int rows = T / (a.row_bytes / 8 / ctas) * U;
  const size_t sm = std::max(std::min(SPAN, e.limit) * sizeof(float), 3 * rows * sizeof(int2));
  return launch_kc(evict_kernel<T, U>, dim3((unsigned)(items * ctas)), dim3(T), sm, st,
                   ctas > 1 ? dim3(ctas, 1, 1) : dim3(0, 0, 0), e, a, ctas);
}

cudaError_t launch_evict(const EvictArgs& e, const CacheMoveArgs& a, cudaStream_t st) {
  const int items = a.layers * a.B * a.n_kv;
  // 1024 heads of 4096 slots, 1500 kept: 272 us with four CTAs per SM and 5 units a thread,
  // 299 with three and 8, 319 with four and 4; select and move as two kernels 290
  if (items > 2 * a.sm_count) return run_evict<256, 5>(e, a, items, 1, st);
  // more heads than SMs: two CTAs of half the size each (160 heads of 1088 slots 44.7 us, one of
  // 512 threads 51.9; but of 200 slots 10.1 and 9.4)
  if (items > a.sm_count && e.limit >= 512) return run_evict<256, 5>(e, a, items, 2, st);
  // up to two CTAs per SM, which are resident at once (48 heads of 62 slots 7.7 us, twice as many
  // CTAs 13.6; 144 of 4000, 1500 kept, 56 and 70)
  int ctas = 1;
  while (ctas < 8 && items * ctas <= a.sm_count && a.row_bytes / 8 / (2 * ctas) >= 2 &&
         a.row_bytes / 8 % (2 * ctas) == 0)
    ctas *= 2;
  return run_evict<512, 4>(e, a, items, ctas, st);
}

}  // namespace llgb
