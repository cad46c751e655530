// Attention with capped or biased scores on the 5th-generation tensor cores
// (tcgen05), head_dim 128, bf16: packed documents (causal, with a two-way
// prefix), and the shared prefix of a decode batch.
//
//   x = scale q.k;  s = (cap tanh(x / cap) or x) - slope |i - j|;  p = softmax(s);  o = sum p v
//
// One pass over the keys with the running maximum and sum of each row: the
// scores never leave the SM. One CTA per SM works on two tiles of 128 query rows
// (MMA M, one tensor-memory lane per row) against key tiles of 128:
//   warps 0-7, 8-15  softmax of row tile 0 and 1: two threads per row, one for
//                    keys 0-63 of a tile and output dims 0-63, one for the rest;
//   warp 16, 17      TMA producers of Q + K and of V (rings of 32 KB tiles);
//   warp 18, 19      issue the MMAs of row tile 0 and 1.
// A turn of an issuer is O += P_j V_j, then S_{j+1} = Q K^T_{j+1}; the turns
// alternate between the row tiles, so while one tile's softmax runs on the CUDA
// cores the tensor cores work for the other. (Without that order the tensor pipe
// interleaves the two tiles' MMAs, both softmaxes then run at the same time, and
// the pipe idles meanwhile; with one issuer for both, its waits between turns
// leave the pipe idle.) tcgen05 operations of one thread execute in order: P_j
// (bf16, written over the scores it came from) is read before S_{j+1} replaces
// it, and the arrival of S_{j+1} also says that O += P_j V_j is done. Tensor
// memory: per row tile 128 columns of S / P and 128 of O, all 512.
// The two row tiles are
//   documents, n_q / n_kv even : two query heads of one K/V head, same rows;
//   documents, else            : rows q0 .. q0+127 and q0+128 .. q0+255;
//   prefix, over 128 rows      : two blocks of (sequence, head of the group) rows;
//   prefix, up to 128 rows     : the same rows; tile t takes every second key tile
//                                (two key splits; each K/V tile has one reader).
// so K and V are loaded once for both. Every mask here is "keys below a row's
// limit": max(position + 1, prefix) for documents, the sequence's keys for the
// prefix. O is rescaled lazily, when a row's maximum grows by more than 2^8.
//
// Documents run as one CTA per SM that takes its share of the work items: the
// producers load the next item's Q, K and V while the softmax and the store of
// the last one go on, and barriers and tensor memory are set up once (17 packed
// documents of 8192 rows, 64 heads: 246 us with a CTA per item, 216 us so, and
// 162 us with the items dealt out longest first and published by one warp, and
// whole sectors stored; back to back, 169 us among other work).
//
// P is rounded once to bf16 (V's type, which the MMA shares), and the sum that
// normalises it is that of the rounded weights, in fp32: what the dominant keys
// of a row lose by rounding cancels (error against 64 bits, relative to the
// outputs' root mean square, packed biased documents: 0.0019 instead of 0.0022;
// prefixes 0.0020, capped scores 0.0021-0.0022; rounding the output alone is
// 0.0016-0.0017). The add takes a bf16 operand, so it costs nothing beside the sum of
// the unrounded weights but its latency (1 %; unpacked first, 6 %).
//
// What bounds it: plain scores, the tensor pipe and the hand-overs between it
// and the softmax (2640 cycles per pair of turns, 2048 of them MMAs); capped and
// biased ones the issue slots of the softmax (3200 and more).
#include <algorithm>
#include <climits>

#include "attn_score.cuh"
#include "internal.h"

namespace llgb {

namespace {

constexpr int TM = 128;                     // rows of a tile
constexpr int TN = 128;                     // keys of a tile
constexpr uint32_t HALF = 128 * 128;        // 128 rows x 64 dims bf16, 128-byte swizzled: 16 KB
constexpr uint32_t TILE = 2 * HALF;         // 128 rows x 128 dims
constexpr int SLOTS = 7;                    // Q 0, (Q 1), then the K ring and the V ring
constexpr uint32_t OFF_BAR = SLOTS * TILE;
// what the two threads of a row exchange: fp32 [2 row tiles][2 halves][128], the
// tile's maxima, at the end the sums. One buffer is enough: a tile's maxima are
// read before its P is announced, and the next tile's scores come after that.
constexpr uint32_t OFF_WORK = OFF_BAR + 256;  // documents: two published work items, 32 bytes each
constexpr uint32_t OFF_X = OFF_WORK + 64;
constexpr size_t FORMS_SMEM = OFF_X + 2 * 2 * 128 * 4;
constexpr int FORMS_THREADS = 640;
constexpr int MAXK = 4, MAXV = 2;           // ring sizes at most
constexpr uint32_t O_COL = 256;             // S tiles at columns 0 and 128, O tiles at 256 and 384
constexpr float kLazy = 8.f;
static_assert(FORMS_SMEM <= 232448, "227 KB of shared memory per CTA");

struct FormsParams {
  int n_q, n_kv, G;
  float scale, cap;
  const float* slopes;
  uint32_t* status;
  // documents
  bf16* out;
  const int32_t *cu_rows, *prefix_len;
  int n_rows, n_docs, head_pairs;
  int out32;                                // out is 32-byte aligned
  // prefix of a decode batch
  const int32_t *positions, *page_table;
  int B, rows_seq;                          // sequences of a row tile (128 / G)
  int alternate;                            // both row tiles hold the same rows
  int layer, page_size, capacity, n_pages, max_pages, box_rows;
  int key_limit, shared_len, shared_seq;
  float *part_o, *part_ml;                  // [B n_q][splits][128], [B n_q][splits][2] (max log2, sum)
  int splits;                               // partials a row has room for
  size_t partials;                          // partials in all
  int *used;                                // how many of them are written
  int sm_count;
  int waiting;                              // the own keys' CTAs wait for this kernel
  float own_items;                          // how many those are
  float poly[13];                           // KCapFixed: kTanh times powers of scale / cap
};

// What the scores need. A cap bounds them, so up to kFixedCap (log2 units) the
// weights are 2^s with no maximum subtracted: 2^+-72 times a sum stays inside fp32
// (and bf16's exponent) for |V| below 2^55 / keys, and the row maxima, their
// exchange and every rescale fall away.
enum { KPlain, KBias, KCapFixed, KCap };
constexpr float kFixedCap = 72.5f;  // caps up to 50

// Bounded wait without a call (setmaxnreg leaves no registers for one); the
// clock and the abort flag are read once every 64 tries. False, and the flag
// set for everyone, when the time is up.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile uint32_t* stop,
                                         uint32_t* status) {
  uint64_t since = 0;
#pragma unroll 1
  for (uint32_t i = 1; !mbar_try_wait(bar, parity); ++i) {
    if ((i & 63) == 0) {
      const uint64_t now = globaltimer_ns();
      if (since == 0) since = now;
      if (*stop) return false;
      if (now - since > kWaitLimitNs) {
        *stop = 1;
        flag(status, LLAMA_FLAG_WAIT_TIMEOUT);
        return false;
      }
    }
  }
  return true;
}
// The same for the other issuer's turns to reach n. (An order for speed's sake:
// what the MMAs read and write is guarded by the barriers.)
__device__ __forceinline__ bool wait_turn(volatile uint32_t* turns, uint32_t n, volatile uint32_t* stop,
                                          uint32_t* status) {
  uint64_t since = 0;
#pragma unroll 1
  for (uint32_t i = 1; (int32_t)(*turns - n) < 0; ++i) {
    __nanosleep(20);  // polling steals issue slots from the softmax
    if ((i & 63) == 0) {
      const uint64_t now = globaltimer_ns();
      if (since == 0) since = now;
      if (*stop) return false;
      if (now - since > kWaitLimitNs) {
        *stop = 1;
        flag(status, LLAMA_FLAG_WAIT_TIMEOUT);
        return false;
      }
    }
  }
  return true;
}

// Ring position: slot and phase parity of the n-th use.
struct Ring {
  int n, slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ explicit Ring(int size) : n(size) {}
  __device__ __forceinline__ void step(int k = 1) {
    slot += k;
    if (slot >= n) {
      slot -= n;
      phase ^= 1;
    }
  }
};

// Cache row of the keys starting at k0 of sequence b, K/V head g; a page
// outside the pool is flagged and mapped to rows that TMA fills with zeros.
__device__ __forceinline__ int forms_kv_row(const FormsParams& p, int b, int g, int k0) {
  if (p.page_size == 0) return (b * p.n_kv + g) * p.capacity + k0;
  const int pi = k0 / p.page_size;
  const int page = pi < p.max_pages ? p.page_table[(size_t)b * p.max_pages + pi] : -1;
  if (page < 0 || page >= p.n_pages) {
    flag(p.status, LLAMA_FLAG_PAGE_RANGE);
    return -64;
  }
  return (page * p.n_kv + g) * p.page_size + (k0 - pi * p.page_size);
}

// Cache rows of a prefix's next four key tiles, one 16-key step per lane (tile
// j + lane / 8, step lane % 8): looked up once per four tiles and ahead of the
// wait for a free slot (a lookup per box in front of its copy held every tile
// back by some 2000 cycles).
__device__ __forceinline__ int tile_rows(const FormsParams& p, int g, int tile, int kmax, int lane) {
  const int k0 = (tile + (lane >> 3)) * TN + (lane & 7) * 16;
  return k0 < kmax ? forms_kv_row(p, p.shared_seq, g, k0) : 0;
}

// K or V tile of keys k0 .. k0 + nvalid - 1 by a whole warp, completing on bar.
// Prefix: per 64 keys one box per dim half where the view has 64-row boxes and
// the keys are all there, else 16-key boxes; rows as from tile_rows, j the tile.
template <bool DOCS>
__device__ __forceinline__ void load_tile(const FormsParams& p, const CUtensorMap* big,
                                          const CUtensorMap* m16, uint8_t* dst, uint64_t* bar, int g,
                                          int rowbase, int k0, int nvalid, int rows, int j, int lane) {
  if (DOCS) {
    if (lane == 0) {
      mbar_arrive_expect_tx(bar, TILE);
      tma_load_3d(dst, big, bar, 0, g, rowbase + k0);
      tma_load_3d(dst + HALF, big, bar, 64, g, rowbase + k0);
    }
    return;
  }
  if (lane == 0) mbar_arrive_expect_tx(bar, 2 * ((nvalid + 15) / 16) * 16 * 128);
  __syncwarp();
  const int step = lane >> 1, half = lane & 1;  // lanes 0-15
  const int row = __shfl_sync(0xffffffffu, rows, 8 * (j & 3) + (step & 7));
  const bool whole = p.box_rows == 64 && nvalid - (step >> 2) * 64 >= 64;
  if (step < 8 && step * 16 < nvalid && (!whole || (step & 3) == 0))
    tma_load_3d(dst + half * HALF + step * 16 * 128, whole ? big : m16, bar, 64 * half, row, p.layer);
}

// Of the fits of tanh (kTanh) a warp takes the shortest that covers its scores: caps
// are seldom approached. On the special-function unit a cap would cost an
// exponential and a reciprocal per score beside the softmax's own exponential.
// Eight x times the polynomial with N coefficients c[0..] in w = x^2 (UNIT: of y =
// x yk), step by step over all eight: written element by element the compiler
// keeps that order, and the chain of dependent multiply-adds took 1287 cycles
// per 64 scores and warp instead of 656 (measured alone; 1507 and 1172 for two
// warps per scheduler). Scalar, because a pair instruction, fma.rn.f32x2,
// occupies the FMA pipe for 4.4 cycles a warp, a scalar one for 1.2.
template <int N, bool UNIT>
__device__ __forceinline__ void odd_poly8(float* x, const float* c, float yk) {
  float w[8], q[8];
  if (UNIT) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= yk;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = x[i] * x[i];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = fmaf(c[N - 1], w[i], c[N - 2]);
#pragma unroll
  for (int d = N - 3; d >= 0; --d)
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = fmaf(q[i], w[i], c[d]);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] *= q[i];
}

// Which fit covers a warp's scores x (in units of 1 / yk): 0, 1, 2, or 3 for none.
template <int N>
__device__ __forceinline__ int cap_level(const float* x, float yk) {
  float big = 0.f;
#pragma unroll
  for (int i = 0; i < N; i += 2) big = max3(big, fabsf(x[i]), fabsf(x[i + 1]));
  big *= yk;
  return __reduce_max_sync(0xffffffffu, (big > 0.25f) + (big > 0.5f) + (big > 1.f));
}

// cap tanh(x / cap) in log2 units for any x (in units of 1 / zc): cl (1 - 2 / (1 + e^2y))
__device__ __forceinline__ float cap_any(float x, float zc, float cl) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2(x * zc)));
  return fmaf(-2.f * cl, r, cl);
}

// Scores of keys from `left` on replaced.
template <int N>
__device__ __forceinline__ void hide(float* x, int left, float with) {
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = i < left ? x[i] : with;
}

// a = a c + m, b likewise, as one pair instruction: half the issue slots, which
// bound plain scores more than the FMA pipe (per 64 scores and four warps per
// scheduler 1335 cycles with two scalar ones, 1112 with the pair)
__device__ __forceinline__ void fma_pair(float& a, float& b, float c, float m) {
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tmov.b64 z, {%3, %3};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(c), "f"(m));
}

// a += low half of the bf16 pair x, b += its high half
__device__ __forceinline__ void add_pair(float& a, float& b, uint32_t x) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "add.rn.f32.bf16 %0, l, %0;\n\tadd.rn.f32.bf16 %1, h, %1;\n\t}"
      : "+f"(a), "+f"(b)
      : "r"(x));
}

// 32 aligned bytes: a thread owns a row, so a smaller store would write half a sector
__device__ __forceinline__ void store_sector(void* dst, const uint32_t* x) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(x[0]), "r"(x[1]),
               "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}

__device__ __forceinline__ void half_bar(int id) {  // the two warps that share 32 rows
  asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory");
}

// The documents' work items in descending order of their key tiles, asked for in
// ascending order by a whole warp. With C the key tiles of a causal item and P
// those of the document's prefix, an item has max(C, P). Per count k and 32
// documents, a lane knows how many items of its document have exactly k: with
// tiles of 128 rows C = 1, 2, ..; with 256 rows C = 2, 4, .. and last the
// document's own tile count. Longest first, dealt out in alternating order:
// 17 packed documents end 1 % above the mean load (in the documents' order 13 %),
// three with prefixes 13 % (61 %).
// (Beyond 32 documents, 32 at a time: every count over all documents would be
// documents / 32 loads per count.)
struct DocCursor {
  int k = -1, b0 = 0, before = 0;  // key tiles (-1: a new step) and first document of the step, items before
  int lo = 0, n = 0, P = 0;        // the lane's document of the step
};
__device__ __forceinline__ bool find_item(const FormsParams& p, int item, int per, DocCursor& c, int& b,
                                          int& tile, int& lo, int& n, int& head) {
  const int lane = threadIdx.x & 31;
  for (; c.b0 < p.n_docs; c.b0 += 32, c.k = -1) {
    if (c.k < 0) {
      c.lo = c.n = c.P = 0;
      if (c.b0 + lane < p.n_docs) {
        doc_rows(p.cu_rows, c.b0 + lane, p.n_rows, p.status, c.lo, c.n);
        const int pre = p.prefix_len ? min(max(p.prefix_len[c.b0 + lane], 0), c.n) : 0;
        c.P = (pre + TN - 1) / TN;
      }
      c.k = __reduce_max_sync(0xffffffffu, (c.n + TN - 1) / TN);
    }
    for (; c.k > 0; --c.k) {
      const int N = (c.n + TN - 1) / TN;  // key tiles of the whole document
      int have = 0, first = 0;            // items with k key tiles, the first of them
      if (c.k == c.P) {
        have = p.head_pairs ? c.P : c.P >= N ? (N + 1) / 2 : c.P / 2;  // C up to P
      } else if (c.k > c.P && c.k <= N) {
        have = p.head_pairs || (c.k & 1) == 0 || c.k == N;
        first = p.head_pairs ? c.k - 1 : (c.k + 1) / 2 - 1;
      }
      int upto = have;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      const int total = __shfl_sync(0xffffffffu, upto, 31);
      if (item - c.before < total * per) {
        const int i = (item - c.before) / per;
        head = item - c.before - i * per;
        const int w = __ffs(__ballot_sync(0xffffffffu, i < upto)) - 1;
        b = c.b0 + w;
        tile = __shfl_sync(0xffffffffu, first + i - (upto - have), w);
        lo = __shfl_sync(0xffffffffu, c.lo, w);
        n = __shfl_sync(0xffffffffu, c.n, w);
        return true;
      }
      c.before += total * per;
    }
  }
  return false;
}

// One work item: its two row tiles and the key tiles that they visit.
struct FormsWork {
  int lo, n, q0, pre;   // documents: the document's rows [lo, lo + n), first query row, prefix
  int g, h0;            // K/V head, query head of row tile 0
  int t0, n_tiles;      // first key tile and how many
  int kmax;             // keys below this exist for some row
  int nt0, nt1;         // key tiles that row tile 0 / 1 visits
  int split, seq0;      // prefix: key split, first sequence
  int last_rows;        // keys of the last tile; over TN: all
};
// Documents: what follows from an item's document, first row and head.
__device__ __forceinline__ void doc_work(const FormsParams& p, int lo, int n, int q0, int pre, int h0, int g,
                                         FormsWork& w) {
  w.lo = lo;
  w.n = n;
  w.q0 = q0;
  w.pre = pre;
  w.h0 = h0;
  w.g = g;
  const int last0 = max(min(q0 + TM, n), pre);
  const int last1 = p.head_pairs ? last0 : q0 + TM < n ? max(min(q0 + 2 * TM, n), pre) : 0;
  w.nt0 = (last0 + TN - 1) / TN;
  w.nt1 = (last1 + TN - 1) / TN;
  w.kmax = max(last0, last1);
  w.n_tiles = max(w.nt0, w.nt1);
  w.t0 = w.split = w.seq0 = 0;
  w.last_rows = w.kmax - (w.n_tiles - 1) * TN;
}
// The CTA's it-th document item; false: no more.
__device__ __forceinline__ bool next_doc(const FormsParams& p, int it, DocCursor& cursor, FormsWork& w) {
  const int per = p.head_pairs ? p.n_q / 2 : p.n_q, rows = p.head_pairs ? TM : 2 * TM;
  // every other round backwards: whoever had the longest item of one round
  // gets the shortest of the next
  const long long item = (long long)it * gridDim.x + ((it & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
  if (item >= 0x7fffffffll) return false;
  int b, tile, hx, lo, n;
  if (!find_item(p, (int)item, per, cursor, b, tile, lo, n, hx)) return false;
  const int h0 = p.head_pairs ? 2 * hx : hx;
  doc_work(p, lo, n, tile * rows, p.prefix_len ? min(max(p.prefix_len[b], 0), n) : 0, h0, h0 / p.G, w);
  return true;
}
// The CTA's prefix item; false: the splits end before this one. share: key tiles of a split.
__device__ __forceinline__ bool prefix_work(const FormsParams& p, int share, FormsWork& w) {
  w.lo = w.n = w.q0 = w.pre = w.h0 = 0;
  w.split = blockIdx.x;
  w.g = blockIdx.z;
  w.seq0 = blockIdx.y * p.rows_seq * (p.alternate ? 1 : 2);
  w.t0 = w.split * share;
  w.n_tiles = min(share, (p.shared_len + TN - 1) / TN - w.t0);
  if (w.n_tiles <= 0) return false;
  w.kmax = p.shared_len;
  w.nt0 = p.alternate ? (w.n_tiles + 1) / 2 : w.n_tiles;
  w.nt1 = p.alternate ? w.n_tiles / 2 : w.seq0 + p.rows_seq < p.B ? w.n_tiles : 0;
  w.last_rows = w.kmax - (w.t0 + w.n_tiles - 1) * TN;
  return true;
}

// Key tiles per prefix split, for a whole warp; the same in every CTA. A smaller
// prefix grid leaves SMs to the own keys' kernel, which starts beside it and is
// bound by bytes; a larger one ends sooner. Of all grids, the one with the
// smallest estimate of both: 6 us and 1.3 - 2.1 us per turn here; an own CTA
// 3.5 us and its bytes at 29 GB/s, three per free SM, 6.3 TB/s together at most,
// and 6 us more for what is left when the prefix ends.
template <int KIND>
__device__ __forceinline__ int prefix_share(const FormsParams& p, int lane) {
  float own = 0.f;
  for (int i = lane; i < p.B; i += 32)
    own += (float)max(0, key_position(p.positions[i], p.key_limit) + 1 - p.shared_len);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) own += __shfl_xor_sync(0xffffffffu, own, o);
  own *= 512.f * gridDim.z;  // K and V
  const float item = own / p.own_items;
  const float sm_rate = 3.f * item / (3.5f + item / 0.029e6f);
  constexpr float turn = KIND == KPlain ? 1.3f : KIND == KBias ? 1.6f : KIND == KCapFixed ? 1.95f : 2.1f;
  const int tiles = (p.shared_len + TN - 1) / TN, unit = gridDim.y * gridDim.z;
  float best = INFINITY;
  int share = tiles;
  for (int s = lane + 1; s <= gridDim.x; s += 32) {
    const int n = (tiles + s - 1) / s, turns = p.alternate ? (n + 1) / 2 : n;
    const float t = 6.f + turn * turns;
    const float sms = (float)max(0, p.sm_count - (tiles + n - 1) / n * unit);
    float done = fminf(6.3e6f, sm_rate * sms) * t;
    if (p.waiting) done = fminf(done, 3.f * sms * item);  // one item per resident CTA
    const float total = t + (own > done ? 6.f + (own - done) / 6.3e6f : 0.f);
    if (total < best) {
      best = total;
      share = n;
    }
  }
  const uint32_t top = __reduce_min_sync(0xffffffffu, __float_as_uint(best));
  return __reduce_min_sync(0xffffffffu, __float_as_uint(best) == top ? share : INT_MAX);
}

template <bool DOCS, int KIND>
__global__ void __launch_bounds__(FORMS_THREADS, 1)
    attn_forms_kernel(const __grid_constant__ CUtensorMap mapQ,
                      const __grid_constant__ CUtensorMap mapK,
                      const __grid_constant__ CUtensorMap mapV,
                      const __grid_constant__ CUtensorMap mapK16,
                      const __grid_constant__ CUtensorMap mapV16, FormsParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* qfull = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  uint64_t* qempty = qfull + 1;
  uint64_t* kfull = qempty + 1;
  uint64_t* kempty = kfull + MAXK;
  uint64_t* vfull = kempty + MAXK;
  uint64_t* vempty = vfull + MAXV;
  uint64_t* vland = vempty + MAXV;  // a ragged last V tile is there; vfull follows when it is cleaned
  uint64_t* sfull = vland + 1;      // [2] S_j of row tile t is in tensor memory
  uint64_t* pready = sfull + 2;     // [2][2] each part of P_j is, and O is rescaled
  uint64_t* fin = pready + 4;       // [2] the row tile's last O += P V is done
  uint64_t* drained = fin + 2;      // [2] every MMA of the issuer is done
  uint64_t* wfull = drained + 2;    // [2] a work item is published, [2] every other warp has read it
  uint64_t* wempty = wfull + 2;
  // tensor memory, abort, and the turns at the tensor pipe that each issuer has
  // had (counts, because a phase bit could be lapped); a prefix split's key tiles
  volatile uint32_t* ctl = reinterpret_cast<volatile uint32_t*>(wempty + 2);
  volatile uint32_t* stop = ctl + 1;
  static_assert((2 + 2 * MAXK + 2 * MAXV + 1 + 10 + 4) * 8 + 20 <= 256, "barrier block");
  volatile int4* box = reinterpret_cast<volatile int4*>(smem + OFF_WORK);
  grid_dep_wait();
  grid_dep_launch();
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if ((smem_u32(smem) & 1023u) != 0 ||  // the swizzled tiles need 1024-byte alignment
      !bc_smem(smem, FORMS_SMEM, 1024, threadIdx.x == 0 ? p.status : nullptr)) {
    if (threadIdx.x == 0) flag(p.status, LLAMA_FLAG_INDEX);
    return;
  }
  const bool alt = !DOCS && p.alternate;
  const int KR = alt ? 4 : 3, VR = 2;  // even rings when each slot has one reader
  uint8_t* kslots = smem + (alt ? 1 : 2) * TILE;
  uint8_t* vslots = kslots + KR * TILE;

  if (threadIdx.x == 0) {
    const uint32_t readers = alt ? 1 : 2;
    mbar_init(qfull, 1);
    mbar_init(qempty, 2);
    for (int s = 0; s < MAXK; ++s) {
      mbar_init(&kfull[s], 1);
      mbar_init(&kempty[s], readers);
    }
    for (int s = 0; s < MAXV; ++s) {
      mbar_init(&vfull[s], 1);
      mbar_init(&vempty[s], readers);
    }
    mbar_init(vland, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sfull[t], 1);
      mbar_init(&pready[2 * t], 8);
      mbar_init(&pready[2 * t + 1], 8);
      mbar_init(&fin[t], 1);
      mbar_init(&drained[t], 1);
      mbar_init(&wfull[t], 1);
      mbar_init(&wempty[t], FORMS_THREADS / 32 - 1);
    }
    ctl[1] = ctl[2] = ctl[3] = 0;
    fence_mbar_init();
  }
  if (warp == 18) tmem_alloc(const_cast<uint32_t*>(ctl), 512);
  if (!DOCS && warp == 17) {
    const int n = prefix_share<KIND>(p, lane);
    if (lane == 0) {
      ctl[4] = n;
      const int used = ((p.shared_len + TN - 1) / TN + n - 1) / n * (p.alternate ? 2 : 1);
      if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && bc_ok(used <= p.splits, p.status))
        *p.used = used;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl[0], 0);
  const int share = DOCS ? 0 : __shfl_sync(0xffffffffu, ctl[4], 0);

  // launched with 640 x 96 registers: 512 x 104 + 128 x 64
  // The it-th work item, as the Q and K producer published it: the walk to it
  // costs some 3000 cycles, which in every warp delayed each item's start.
  auto work = [&](int it, FormsWork& w) -> bool {
    if (!DOCS) return it == 0 && prefix_work(p, share, w);
    const int s = it & 1;
    const bool ok = __all_sync(0xffffffffu, wait_bar(&wfull[s], (it >> 1) & 1, stop, p.status));
    const int lo = box[2 * s].x, n = box[2 * s].y, q0 = box[2 * s].z, pre = box[2 * s].w;
    const int h0 = box[2 * s + 1].x, g = box[2 * s + 1].y;
    __syncwarp();
    if (lane == 0) mbar_arrive(&wempty[s]);
    if (!ok || n == 0) return false;
    doc_work(p, lo, n, q0, pre, h0, g, w);
    return true;
  };
  if (warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    FormsWork w{};
    if (warp == 16) {  // ------------------------------------------- Q and K producer
      if (lane == 0) {
        tma_prefetch_desc(&mapQ);
        tma_prefetch_desc(&mapK);
      }
      Ring r(KR);
      int issued = 0, loaded_q = 0, rows = 0;
      bool ok = true;
      DocCursor cursor;
      for (int it = 0; ok; ++it) {
        if (DOCS) {
          const bool more = next_doc(p, it, cursor, w);
          ok = __all_sync(0xffffffffu, wait_bar(&wempty[it & 1], ((it >> 1) & 1) ^ 1, stop, p.status));
          if (!ok) break;
          if (lane == 0) {
            volatile int4* to = box + 2 * (it & 1);
            to->x = w.lo;
            to->y = more ? w.n : 0;  // an item's document is never empty
            to->z = w.q0;
            to->w = w.pre;
            to[1].x = w.h0;
            to[1].y = w.g;
            mbar_arrive(&wfull[it & 1]);
          }
          __syncwarp();
          if (!more) break;
        } else {
          if (it > 0 || !prefix_work(p, share, w)) break;
          rows = tile_rows(p, w.g, w.t0, w.kmax, lane);
        }
        ok = __all_sync(0xffffffffu, wait_bar(qempty, (it & 1) ^ 1, stop, p.status));
        if (!ok) break;
        ++loaded_q;
        if (lane == 0) {
          const int q_tiles = alt || w.nt1 == 0 ? 1 : 2;
          const uint32_t qbytes = DOCS ? TILE : (uint32_t)(p.rows_seq * p.G) * 256;
          mbar_arrive_expect_tx(qfull, q_tiles * qbytes);
          for (int t = 0; t < q_tiles; ++t)
            for (int half = 0; half < 2; ++half) {
              uint8_t* d = smem + t * TILE + half * HALF;
              if (DOCS)
                tma_load_3d(d, &mapQ, qfull, 64 * half, p.head_pairs ? w.h0 + t : w.h0,
                            w.lo + w.q0 + (p.head_pairs ? 0 : t * TM));
              else
                tma_load_3d(d, &mapQ, qfull, 64 * half, w.g * p.G, w.seq0 + t * p.rows_seq);
            }
        }
        for (int j = 0; j < w.n_tiles; ++j) {
          if (!DOCS && j > 0 && (j & 3) == 0) rows = tile_rows(p, w.g, w.t0 + j, w.kmax, lane);
          ok = __all_sync(0xffffffffu, wait_bar(&kempty[r.slot], r.phase ^ 1, stop, p.status));
          if (!ok) break;
          load_tile<DOCS>(p, &mapK, &mapK16, kslots + r.slot * TILE, &kfull[r.slot], w.g, w.lo,
                          (w.t0 + j) * TN, min(TN, w.kmax - (w.t0 + j) * TN), rows, j, lane);
          ++issued;
          r.step();
        }
      }
      // no copy in flight when the CTA exits
      if (loaded_q) mbar_wait(qfull, (loaded_q - 1) & 1, p.status);
      for (int j = max(0, issued - KR); j < issued; ++j)
        mbar_wait(&kfull[j % KR], (j / KR) & 1, p.status);
    } else if (warp == 17) {  // ------------------------------------ V producer
      if (lane == 0) tma_prefetch_desc(&mapV);
      Ring r(VR);
      int issued = 0;
      uint32_t ph_land = 0;
      int rows = 0;
      bool ok = true;
      for (int it = 0; ok && work(it, w); ++it) {
        for (int j = 0; ok && j < w.n_tiles; ++j) {
          if (!DOCS && (j & 3) == 0) rows = tile_rows(p, w.g, w.t0 + j, w.kmax, lane);
          ok = __all_sync(0xffffffffu, wait_bar(&vempty[r.slot], r.phase ^ 1, stop, p.status));
          if (!ok) break;
          const bool ragged = j + 1 == w.n_tiles && w.last_rows < TN;
          load_tile<DOCS>(p, &mapV, &mapV16, vslots + r.slot * TILE, ragged ? vland : &vfull[r.slot],
                          w.g, w.lo, (w.t0 + j) * TN, min(TN, w.kmax - (w.t0 + j) * TN), rows, j, lane);
          if (ragged) {
            // V rows past the last key may hold anything, and 0 * NaN is not 0
            __syncwarp();
            ok = __all_sync(0xffffffffu, wait_bar(vland, ph_land, stop, p.status));
            ph_land ^= 1;
            uint8_t* vt = vslots + r.slot * TILE;
            const int nz = (TN - w.last_rows) * 16;
            for (int i = lane; ok && i < nz; i += 32) {
              const int row = w.last_rows + (i >> 4), half = (i >> 3) & 1, chunk = i & 7;
              *reinterpret_cast<uint4*>(vt + half * HALF + row * 128 + chunk * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();  // the MMA reads V through the async proxy
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(&vfull[r.slot]);
          }
          if (ok) ++issued;
          r.step();
        }
      }
      for (int j = max(0, issued - VR); j < issued; ++j)
        mbar_wait(&vfull[j % VR], (j / VR) & 1, p.status);
    } else {  // ---------------------------------------------------- MMA issuers
      // The whole warp walks the tiles and one elected lane issues, so slots,
      // descriptors and addresses stay in uniform registers: from a branch that
      // one lane takes alone, moving them there made an MMA's issue take some
      // 100 cycles against the 64 of its work.
      const int t = warp - 18;
      const uint32_t id_s = idesc_bf16_f32(TM, TN);
      const uint32_t id_o = idesc_bf16_f32(TM, 128) | (1u << 16);  // B (V) MN-major
      const uint64_t qd = smem_desc_sw128(smem_u32(smem)) + (uint64_t)(alt ? 0 : t * (TILE >> 4));
      const uint64_t kd0 = smem_desc_sw128(smem_u32(kslots));
      const uint64_t vd0 = smem_desc_sw128_mn(smem_u32(vslots), HALF);
      const uint32_t sc = tmem + (uint32_t)t * TN, oc = tmem + O_COL + (uint32_t)t * 128;
      // When a turn ends: plain scores, with its last MMA issued (the tensor pipe
      // bounds them, and the hand-over passes while it executes); biased and
      // capped ones, with S complete: their softmax is the longer part, and the
      // further the row tiles are out of step the less the two share the CUDA
      // cores. Measured, turn at issue and at completion: 2500 plain rows 47.6 and
      // 52.7 us, 128 sequences over a prefix 180 and 184 us; packed biased
      // documents 220 and 215 us, a capped prompt of 8192 rows 945 and 926 us.
      constexpr bool LATE_TURN = KIND != KPlain;
      const int stride = alt ? 2 : 1;
      Ring kr(KR), vr(VR);
      if (alt) {
        kr.step(t);
        vr.step(t);
      }
      uint32_t ph_p = 0, ph_s = 0;  // phases of pready, sfull
      uint32_t mine = 0, theirs = 0;  // turns taken, and the other row tile's before this item
      // No wait's outcome is looked at here (nor by the softmax): after an abort
      // every wait returns at once, the rest runs on whatever is there, and
      // nothing is stored. Checks and votes between the waits and the MMAs
      // measured 5-15 % on all cases.
      for (int it = 0; work(it, w); ++it) {
        const int count = t ? w.nt1 : w.nt0, others = t ? w.nt0 : w.nt1;
        auto score = [&](int slot, bool last) {  // S of a key tile
          const uint64_t kd = kd0 + (uint64_t)(slot * (TILE >> 4));
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)  // 16 dims per MMA: 32 bytes of Q and K rows
            tc_mma_f16(sc, qd + ((kk >> 2) * HALF + (kk & 3) * 32) / 16,
                       kd + ((kk >> 2) * HALF + (kk & 3) * 32) / 16, id_s, kk > 0 ? 1u : 0u);
          tc_commit(&sfull[t]);
          tc_commit(&kempty[slot]);
          if (last) tc_commit(qempty);
        };
        wait_bar(qfull, it & 1, stop, p.status);
        if (count > 0) {
          const int slot = __shfl_sync(0xffffffffu, kr.slot, 0);
          wait_bar(&kfull[slot], kr.phase, stop, p.status);
          tc_fence_after();
          if (elect_one()) score(slot, count == 1);
          ph_s ^= 1;
          kr.step(stride);
        } else if (lane == 0) {
          mbar_arrive(qempty);
        }
        for (int j = 0; j < count; ++j) {
          // The issuer shares its scheduler with four softmax warps, so what it
          // executes between a P and the MMAs is kept short: all other waits
          // (V, the next K) come before P's.
          const int slot = __shfl_sync(0xffffffffu, vr.slot, 0), next = __shfl_sync(0xffffffffu, kr.slot, 0);
          const bool more = j + 1 < count;
          const uint64_t vd = vd0 + (uint64_t)(slot * (TILE >> 4));
          ++mine;
          // 16 keys per MMA: 8 P columns, two 8-key V groups. P: keys 64 h .. at
          // columns 64 h ..; the first part is keys 0-31 of both halves
          auto add_pv = [&](int part, uint32_t acc) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int kk = 4 * (i >> 1) + 2 * part + (i & 1);
              tc_mma_f16_ts(oc, sc + 64u * (kk >> 2) + 8u * (kk & 3), vd + kk * (2048 / 16), id_o,
                            acc | (uint32_t)(i > 0));
            }
          };
          wait_bar(&vfull[slot], vr.phase, stop, p.status);
          if (more) wait_bar(&kfull[next], kr.phase, stop, p.status);
          wait_bar(&pready[2 * t], ph_p, stop, p.status);
          // the turn: after the other row tile's j-th, or (j - 1)-th for tile 0
          // (last, when it has mostly come: this wait polls)
          wait_turn(ctl + 2 + (t ^ 1), theirs + min(t ? j + 1 : j, others), stop, p.status);
          tc_fence_after();
          // the first part of P while the softmax works on the second
          if (elect_one()) add_pv(0, j > 0);
          wait_bar(&pready[2 * t + 1], ph_p, stop, p.status);
          tc_fence_after();
          if (elect_one()) {
            add_pv(1, 1u);
            tc_commit(&vempty[slot]);
            if (more)
              score(next, j + 2 == count);
            else
              tc_commit(&fin[t]);
            if (!LATE_TURN || !more) ctl[2 + t] = mine;
          }
          __syncwarp();
          if (more) {
            if (LATE_TURN) {
              wait_bar(&sfull[t], ph_s, stop, p.status);
              if (lane == 0) ctl[2 + t] = mine;
            }
            ph_s ^= 1;
          }
          ph_p ^= 1;
          vr.step(stride);
          if (more) kr.step(stride);
        }
        if (!alt)  // slots that only the other row tile reads
          for (int j = count; j < w.n_tiles; ++j) {
            wait_bar(&kfull[kr.slot], kr.phase, stop, p.status);
            wait_bar(&vfull[vr.slot], vr.phase, stop, p.status);
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&kempty[kr.slot]);
              mbar_arrive(&vempty[vr.slot]);
            }
            kr.step();
            vr.step();
          }
        theirs += others;
      }
      if (elect_one()) tc_commit(&drained[t]);
      __syncwarp();
      mbar_wait(&drained[t], 0, p.status);  // retired before the tensor memory is freed
    }
  } else {  // ----------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    const float kTanh3[3] = {kTanh[0], kTanh[1], kTanh[2]},
                kTanh6[6] = {kTanh[7], kTanh[8], kTanh[9], kTanh[10], kTanh[11], kTanh[12]};
    constexpr bool CAP = KIND == KCapFixed || KIND == KCap, BIAS = KIND == KBias || KIND == KCap;
    constexpr int NK = TN / 2;  // keys of a thread
    const int t = warp >> 3, grp = (warp >> 2) & 1, quad = warp & 3;
    const int r = quad * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)(quad * 32) << 16);
    // this thread's scores (then P at the same columns) and O dims
    const uint32_t sc = tl + (uint32_t)(t * TN + NK * grp), oc = tl + O_COL + (uint32_t)(t * 128 + 64 * grp);
    float* xch = reinterpret_cast<float*>(smem + OFF_X) + t * 256 + r;
    const int bar_id = 1 + t * 4 + quad;
    constexpr float kLog2e = 1.4426950408889634f;
    const float c = p.scale * kLog2e;
    const float cl = p.cap * kLog2e, yk = CAP ? p.scale / p.cap : 0.f;
    const float ct = KIND == KCap ? cl : c;  // log2 units of a raw score (of tanh)
    FormsWork w{};
    uint32_t ph_s = 0, ph_fin = 0;  // phases of sfull, fin
#pragma unroll 1
    for (int it = 0; work(it, w); ++it) {
    const int count = t ? w.nt1 : w.nt0;
    if (DOCS && count == 0) continue;
    // this row: its position, its visible keys, where it goes
    bool row_ok;
    int pos, lim, head;
    size_t row;  // documents: packed row; prefix: sequence
    const int pre = w.pre;
    if (DOCS) {
      const int i = w.q0 + (p.head_pairs ? 0 : t * TM) + r;
      row_ok = i < w.n;
      pos = i;
      lim = min(max(i + 1, pre), w.n);
      head = p.head_pairs ? w.h0 + t : w.h0;
      row = (size_t)w.lo + i;
    } else {
      const int s = w.seq0 + (p.alternate ? 0 : t * p.rows_seq) + r / p.G;
      row_ok = r < p.rows_seq * p.G && s < p.B;
      pos = row_ok ? key_position(p.positions[s], p.key_limit) : -1;
      lim = min(pos + 1, p.shared_len);
      head = w.g * p.G + r % p.G;
      row = s;
    }
    const float sl = BIAS && p.slopes && row_ok ? p.slopes[head] * kLog2e : 0.f;
    float m = KIND == KCapFixed ? 0.f : -INFINITY, l = 0.f;
    for (int j = 0; j < count; ++j) {
      wait_bar(&sfull[t], ph_s, stop, p.status);
      ph_s ^= 1;
      tc_fence_after();
      const int k0 = (w.t0 + (alt ? 2 * j + t : j)) * TN + NK * grp;  // this thread's first key
      const int left = lim - k0;                                    // visible keys (over NK: all)
      const bool part = !__all_sync(0xffffffffu, left >= NK);
      // a warp that sees none of the tile's keys (above the diagonal): its weights are 0
      const bool none = !__any_sync(0xffffffffu, left > 0);
      float x[KIND == KCapFixed ? 1 : NK];
      if (KIND != KCapFixed) {
        tmem_ld32(sc, reinterpret_cast<uint32_t*>(x));
        tmem_ld32(sc + 32, reinterpret_cast<uint32_t*>(x + 32));
        tmem_ld_wait();
      }
      if (KIND == KCap && !none) {
        // hidden keys and rows must not choose the path: they may hold anything,
        // and the paths differ in the last bits
        if (part) hide<NK>(x, left, 0.f);
        const int level = cap_level<NK>(x, row_ok ? yk : 0.f);  // tanh; times cl with the bias below
        if (level == 0) {
#pragma unroll
          for (int i = 0; i < NK; i += 8) odd_poly8<3, true>(x + i, kTanh3, yk);
        } else if (level <= 2) {
#pragma unroll
          for (int i = 0; i < NK; i += 8) odd_poly8<6, true>(x + i, kTanh6, yk);
        } else {
          const float zc = 2.f * c / p.cap;
#pragma unroll
          for (int i = 0; i < NK; ++i) x[i] = cap_any(x[i], zc, 1.f);
        }
      }
      // The bias, -slope (pos - key) log2e = base + sb i, joins a score in the exponent.
      // The reference of the weights need not be the row's maximum, only near and
      // not below it: each 8 keys count with their largest score and their
      // largest bias. Not so where 8 keys' biases are far apart (steep slopes) or
      // keys ahead of a row are visible (a prefix, |pos - key|): there the scores
      // are biased here, and factor 1, base 0, step 0 remain.
      float cb = ct, sb = sl, base = BIAS ? sl * (float)(k0 - pos) : 0.f;
      if (BIAS && !none) {
        const int d0 = k0 - pos;
        const bool ahead = DOCS && __any_sync(0xffffffffu, pre > pos && d0 + NK - 1 > 0);
        if (ahead || __any_sync(0xffffffffu, fabsf(sl) > 2.f)) {
#pragma unroll
          for (int i = 0; i < NK; ++i) {
            const float dist = (float)(d0 + i);
            x[i] = fmaf(sl, ahead ? -fabsf(dist) : dist, x[i] * ct);
          }
          cb = 1.f;
          sb = base = 0.f;
        }
      }
      float mu = 0.f;
      if (KIND != KCapFixed) {
        if (part && !none) hide<NK>(x, left, -INFINITY);
        // ---- the row's maximum, and O rescaled when it grew
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if (none) {
        } else if (BIAS) {
          const float top = base + fmaxf(0.f, 7.f * sb);
#pragma unroll
          for (int i = 0; i < NK; i += 8) {
            const float a = max3(max3(x[i], x[i + 1], x[i + 2]), x[i + 3], x[i + 4]);
            const float m8 = max3(a, fmaxf(x[i + 5], x[i + 6]), x[i + 7]);
            mx[(i >> 3) & 3] = fmaxf(mx[(i >> 3) & 3], fmaf(m8, cb, fmaf(sb, (float)i, top)));
          }
        } else {
#pragma unroll
          for (int i = 0; i < NK; i += 2) mx[(i >> 1) & 3] = max3(mx[(i >> 1) & 3], x[i], x[i + 1]);
        }
        const float mh = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
        xch[128 * grp] = mh;
        half_bar(bar_id);
        const float mt = fmaxf(mh, xch[128 * (grp ^ 1)]) * (KIND == KPlain ? c : 1.f);
        const float m_new = fmaxf(m, mt);
        const bool need = m_new > m + kLazy;  // also the first finite maximum
        if (__any_sync(0xffffffffu, need && j > 0)) {
          const float f = !need ? 1.f : m == -INFINITY ? 0.f : ex2(m - m_new);
#pragma unroll 1
          for (int q = 0; q < 64; q += 16) {
            uint32_t u[16];
            tmem_ld16(oc + q, u);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) * f);
            tmem_st16(oc + q, u);
          }
          l *= f;
        }
        if (need) m = m_new;
        mu = m == -INFINITY ? 0.f : -m;
      }
      // ---- weights, their sum, P over the scores
      float ls[4] = {0.f, 0.f, 0.f, 0.f};
      auto weigh = [&](float* y, int q) {  // y: the scores of keys q .. q + 31
        uint32_t w[16];
        const float bmu = base + mu;
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          float e0 = y[i], e1 = y[i + 1];
          if (KIND == KPlain) {
            fma_pair(e0, e1, c, mu);
          } else if (BIAS) {
            e0 = fmaf(e0, cb, fmaf(sb, (float)(q + i), bmu));
            e1 = fmaf(e1, cb, fmaf(sb, (float)(q + i + 1), bmu));
          }
          e0 = ex2(e0);  // hidden: -inf -> 0
          e1 = ex2(e1);
          w[i / 2] = pack_bf16(e0, e1);
          add_pair(ls[i & 2], ls[(i & 2) + 1], w[i / 2]);
        }
        tmem_st16(sc + q / 2, w);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pready[2 * t + q / 32]);
      };
      if (none) {
        const uint32_t zero[16] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
        tmem_st16(sc, zero);
        tmem_st16(sc + 16, zero);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&pready[2 * t]);
          mbar_arrive(&pready[2 * t + 1]);
        }
      } else if (KIND == KCapFixed) {
        // scores straight from tensor memory, 32 at a time in a rolled loop
#pragma unroll 1
        for (int q = 0; q < NK; q += 32) {
          float y[32];
          tmem_ld32(sc + q, reinterpret_cast<uint32_t*>(y));
          tmem_ld_wait();
          // hidden keys and rows must not choose the path: they may hold
          // anything, and the paths differ in the last bits
          if (part) hide<32>(y, left - q, 0.f);
          const int level = cap_level<32>(y, row_ok ? yk : 0.f);
          if (level == 0) {  // the coefficients hold scale, cap and log2e
#pragma unroll
            for (int i = 0; i < 32; i += 8) odd_poly8<3, false>(y + i, p.poly, 0.f);
          } else if (level == 1) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) odd_poly8<4, false>(y + i, p.poly + 3, 0.f);
          } else if (level == 2) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) odd_poly8<6, false>(y + i, p.poly + 7, 0.f);
          } else {
            const float zc = 2.f * c / p.cap;
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] = cap_any(y[i], zc, cl);
          }
          if (part) hide<32>(y, left - q, -INFINITY);
          weigh(y, q);
        }
      } else {
#pragma unroll
        for (int q = 0; q < NK; q += 32) weigh(x + q, q);
      }
      l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
    }
    // ---- epilogue: this thread's 64 dims; l of both halves
    if (count > 0) {
      wait_bar(&fin[t], ph_fin, stop, p.status);
      ph_fin ^= 1;
    }
    xch[128 * grp] = l;
    half_bar(bar_id);
    l = xch[0] + xch[128];
    half_bar(bar_id);  // both have read: the next item may write
    if (!__any_sync(0xffffffffu, *stop)) {
      tc_fence_after();
      if (DOCS) {
        if (count > 0) {
          const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
          bf16* dst = p.out + (row * p.n_q + head) * 128 + 64 * grp;
#pragma unroll 1
          for (int q = 0; q < 64; q += 32) {
            float u[32];
            tmem_ld32(oc + q, reinterpret_cast<uint32_t*>(u));
            tmem_ld_wait();
            if (row_ok && bc_ok(row < (size_t)p.n_rows, p.status)) {
#pragma unroll
              for (int i = 0; i < 32; i += 16) {
                uint32_t x[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = pack_bf16(u[i + 2 * k] * inv, u[i + 2 * k + 1] * inv);
                if (p.out32) {
                  store_sector(dst + q + i, x);
                } else {
                  *reinterpret_cast<uint4*>(dst + q + i) = make_uint4(x[0], x[1], x[2], x[3]);
                  *reinterpret_cast<uint4*>(dst + q + i + 8) = make_uint4(x[4], x[5], x[6], x[7]);
                }
              }
            }
          }
        }
      } else {
        const int mine = p.alternate ? 2 * w.split + t : w.split;
        const size_t at = (row * p.n_q + head) * p.splits + mine;
        const bool store = row_ok && bc_ok(mine < p.splits && at < p.partials, p.status);
        if (count > 0) {
#pragma unroll 1
          for (int q = 0; q < 64; q += 32) {
            float u[32];
            tmem_ld32(oc + q, reinterpret_cast<uint32_t*>(u));
            tmem_ld_wait();
            if (store) {
#pragma unroll
              for (int i = 0; i < 32; i += 8)
                store_sector(p.part_o + at * 128 + 64 * grp + q + i, reinterpret_cast<const uint32_t*>(u + i));
            }
          }
        }
        if (store && grp == 0 && (p.alternate || count > 0)) {  // no visible key: no mass
          p.part_ml[2 * at] = l == 0.f ? -INFINITY : merge_max(m, l);
          p.part_ml[2 * at + 1] = l;
        }
      }
    }
    }  // items
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 18) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

using FormsKernel = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap,
                             const CUtensorMap, const CUtensorMap, FormsParams);

template <bool DOCS>
FormsKernel forms_kernel(int kind) {
  switch (kind) {
    case KPlain: return attn_forms_kernel<DOCS, KPlain>;
    case KBias: return attn_forms_kernel<DOCS, KBias>;
    case KCapFixed: return attn_forms_kernel<DOCS, KCapFixed>;
    default: return attn_forms_kernel<DOCS, KCap>;
  }
}

// The kernel for these scores, and what it needs of them. KCapFixed scales the
// polynomial's coefficients by powers of scale / cap up to the 11th, which
// have to stay normal fp32 numbers, as have the powers of x up to cap / scale.
int score_kind(const ScoreArgs& s, FormsParams* p) {
  p->scale = s.scale;
  p->cap = s.cap;
  p->slopes = s.slopes;
  if (!(s.cap > 0.f)) return s.slopes ? KBias : KPlain;
  const double cl = (double)s.cap * 1.4426950408889634, k = (double)s.scale / s.cap;
  if (s.slopes || cl > kFixedCap || k < 1.0 / 512 || k > 8.0) return KCap;
  for (int at = 0, n = 3; at < 13; at += n, n = n == 3 ? 4 : 6) {
    double f = cl * k;
    for (int i = 0; i < n; ++i, f *= k * k) p->poly[at + i] = (float)(f * kTanh[at + i]);
  }
  return KCapFixed;
}

template <bool DOCS>
cudaError_t prep() {
  for (int i = 0; i < 4; ++i) {
    const cudaError_t e = cudaFuncSetAttribute(
        forms_kernel<DOCS>(i), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)FORMS_SMEM);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t attn_forms_prepare() {
  const cudaError_t e = prep<true>();
  return e == cudaSuccess ? prep<false>() : e;
}

cudaError_t launch_docs_tc(const DocsArgs& a, cudaStream_t st) {
  if (a.head_dim != 128) return cudaErrorInvalidValue;
  FormsParams p{};
  p.n_q = a.n_q;
  p.n_kv = a.n_kv;
  p.G = a.n_q / a.n_kv;
  const int kind = score_kind(a.sc, &p);
  p.status = a.status;
  p.out = (bf16*)a.out;
  p.out32 = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
  p.cu_rows = a.cu_rows;
  p.prefix_len = a.prefix_len;
  p.n_rows = a.n_rows;
  p.n_docs = a.n_docs;
  p.head_pairs = p.G % 2 == 0;
  const int rows = p.head_pairs ? TM : 2 * TM, per = p.head_pairs ? a.n_q / 2 : a.n_q;
  const long long tiles = a.n_rows / rows + (long long)std::min(a.n_docs, a.n_rows);  // an upper bound
  const unsigned grid = (unsigned)std::min<long long>(tiles * per, a.sm_count);
  return launch_k(forms_kernel<true>(kind), dim3(grid), dim3(FORMS_THREADS), FORMS_SMEM, st, 0,
                  *a.map_q, *a.map_k, *a.map_v, *a.map_k, *a.map_v, p);
}

cudaError_t launch_shared_prefix(const SharedArgs& a, const SharedPlan& s, cudaStream_t st) {
  if (a.head_dim != 128) return cudaErrorInvalidValue;
  FormsParams p{};
  p.n_q = a.n_q;
  p.n_kv = a.n_kv;
  p.G = a.n_q / a.n_kv;
  const int kind = score_kind(a.sc, &p);
  p.status = a.status;
  p.positions = a.positions;
  p.page_table = a.page_table;
  p.B = a.B;
  p.rows_seq = s.rows_seq;
  p.alternate = s.alternate;
  p.layer = a.layer;
  p.page_size = a.page_size;
  p.capacity = a.capacity;
  p.n_pages = a.n_pages;
  p.max_pages = a.max_pages;
  p.box_rows = a.box_rows;
  p.key_limit = a.key_limit;
  p.shared_len = a.shared_len;
  p.shared_seq = a.shared_seq;
  p.part_o = a.partial;
  p.part_ml = a.partial + s.partials * 128;
  p.splits = s.prefix_parts;
  p.partials = s.partials;
  p.used = reinterpret_cast<int*>(a.partial + s.partials * 130);
  p.sm_count = a.sm_count;
  p.waiting = !s.join;
  p.own_items = (float)((double)a.B * a.n_kv * s.own_splits);
  return launch_k(forms_kernel<false>(kind), dim3(s.prefix_splits, s.row_blocks, a.n_kv),
                  dim3(FORMS_THREADS), FORMS_SMEM, st, 0, *a.map_q, *a.map_k, *a.map_v, *a.map_k16,
                  *a.map_v16, p);
}

}  // namespace llgb
