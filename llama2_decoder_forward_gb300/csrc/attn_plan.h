// How decode attention over a shared prefix, key weights and drafted trees are cut into
// CTAs, and the room that their partial results take: host arithmetic on the sizes of a
// call (rows, heads, the cache's room, SMs), apart from the launches so that it can be
// checked over many sizes without a GPU. Times are of GB300, 152 SMs.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace llgb {

constexpr int kPlanHeadDim = 128;                             // the bf16 kernels' only one
constexpr size_t kPartial = (kPlanHeadDim + 2) * sizeof(float);  // a row's partial result: O, maximum, sum
// shared memory of the own keys' kernel: without kept scores, and with two CTAs per SM
constexpr size_t kOwnSmem = 2 * 32768 + 256 + (2 * 256 + 4) * 4 + 1024, kOwnSmemMost = 113 * 1024;

// A decode batch over a shared prefix: the prefix kernel's grid (prefix_splits,
// row_blocks, n_kv) and the own keys' splits.
struct SharedPlan {
  int rows_seq;         // sequences of a 128-row tile
  int alternate;        // one row tile: the two halves of a CTA share its keys
  int row_blocks, tiles_per_split, prefix_splits;
  int prefix_parts;     // partials per row of the prefix kernel (0: no prefix)
  int base, keys;       // own keys start in the tile at base, and are `keys` at most
  int own_splits, min_share;  // key splits, and the keys that a split has at least
  int cluster;          // the own splits of a row form a thread-block cluster
  int join;             // own splits leave partials, which a joining kernel merges
  size_t partials;      // partial rows in all
  int keep;             // key weights: scores of a row that a CTA keeps (0: they go to the joining kernel)
};

inline SharedPlan shared_plan(int B, int n_q, int n_kv, int key_limit, int shared_len, int sm_count) {
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

// Scores of a row that the kernel itself can keep, so that it adds up the weights and the
// joining kernel falls away: where one CTA has all keys of a row, and shared memory for
// them costs no CTA that would be resident otherwise. 0: none. (64 sequences of up to 60
// keys, 8 K/V heads 9.5 us, with the joining kernel 12.0, 32 of up to 200, 32 heads 19.6 and 22.2; the
// splits of a cluster likewise measured slower, 4 sequences of up to 1000 keys 18.7 and 13.4.)
inline int weights_keep(const SharedPlan& s, int B, int n_q, int n_kv, int sm_count) {
  const int G = n_q / n_kv, most = G <= 8 ? 3 : 2;
  const long long bytes = (long long)kOwnSmem + 4ll * G * s.keys;
  if (s.own_splits > 1 || bytes > (long long)kOwnSmemMost) return 0;
  const long long resident = std::min<long long>(most, 227 * 1024 / (bytes + 1024));
  return resident == most || resident * sm_count >= (long long)B * n_kv ? s.keys : 0;
}

inline SharedPlan weights_plan(int B, int n_q, int n_kv, int key_limit, int sm_count) {
  SharedPlan s = shared_plan(B, n_q, n_kv, key_limit, 0, sm_count);
  s.keep = weights_keep(s, B, n_q, n_kv, sm_count);
  if (s.keep) return s;
  // The splits are joined by the second kernel in any case, so that more of them, of long
  // rows, cost little and leave SMs less idle at the end: 5 CTAs per SM with 1024 keys (64
  // sequences of up to 16384 keys, 8 K/V heads, one CTA each 412 us, two 371; 32 of up to 4096,
  // two 64.2, three 62.5, four 65.5; 64 of up to 1500 keys, one 52.5, two 56.2).
  const int pairs = B * n_kv, once = s.own_splits;
  while (pairs * s.own_splits < 5 * sm_count && s.own_splits < 8 && s.keys / (s.own_splits + 1) >= 1024) ++s.own_splits;
  if (once == 1 && s.own_splits > 1) s.min_share = 512;
  s.cluster = 0;  // the weights need a row's maximum and sum over all splits first
  s.join = 1;
  s.partials = (size_t)B * n_q * s.own_splits;
  return s;
}

// Room for the partial results of every batch up to max_batch: own splits, which stay
// below 4 CTAs per SM (G rows each), or are up to 128 and below 3 CTAs per SM.
inline size_t own_partials(int max_batch, int n_q, int n_kv, int sm_count) {
  const size_t rows = (size_t)max_batch * n_q, G = n_q / n_kv;
  return std::max(rows, std::min<size_t>(4 * (size_t)sm_count * G, rows * 128));
}
inline size_t shared_partial_bytes(int max_batch, int n_q, int n_kv, int max_seq, int sm_count) {
  // shared_plan's over every prefix: prefix parts are at most 256 rows a CTA at one CTA per
  // SM, or two per row
  const size_t rows = (size_t)max_batch * n_q, tiles = (size_t)(max_seq + 127) / 128;
  const size_t prefix = std::max(2 * rows, std::min<size_t>(256 * (size_t)sm_count, rows * 2 * tiles));
  return (prefix + own_partials(max_batch, n_q, n_kv, sm_count)) * kPartial + 16;
}
inline size_t weights_partial_bytes(int max_batch, int n_q, int n_kv, int max_seq, int sm_count) {
  // weights_plan's: shared_plan's own splits, or of long rows up to 8 of 1024 keys and up to the
  // first number that reaches 5 CTAs per SM
  const size_t rows = (size_t)max_batch * n_q, G = n_q / n_kv;
  const size_t few = std::min(std::min<size_t>(8, max_seq / 1024) * rows, 5 * (size_t)sm_count * G + rows);
  return std::max(own_partials(max_batch, n_q, n_kv, sm_count), few) * kPartial + 16;
}

// Trees of few rows: blocks of 8 (row, head) pairs of a K/V head on the own keys' kernel, or
// 128 and 256 on the tensor-core kernel. In a cache with room for 4096 positions, the former and
// the latter: 16 sequences of 8 rows, 32 heads 104 and 122 us, 64 of one row, 32 / 8 heads
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
struct TreePlan {
  int own;                 // on the own keys' kernel, else on the tensor cores (and nothing else here counts)
  int shift, slices, per;  // blocks of 2^shift rows; a group's heads in slices of `per`
  int splits, min_share, cluster, join;  // as in SharedPlan
};
// room: bytes for partial results; scored: capped or biased scores
inline TreePlan tree_plan(int n_rows, int B, int n_q, int n_kv, int key_limit, bool scored, int sm_count, size_t room) {
  TreePlan t{};
  const int G = n_q / n_kv;
  t.slices = (G + 7) / 8;
  t.per = (G + t.slices - 1) / t.slices;
  while (2 * t.per << t.shift <= 8) ++t.shift;
  if ((long long)B + n_rows > 65535 || n_kv > 32767) return t;  // the launch's grid
  const int rows = (n_rows + B - 1) / B;  // the mean, all that the host knows of a sequence's rows
  // CTAs without splits, and about as many items of the other kernel's
  const long long heads = (long long)B * n_kv, pairs = heads * t.slices * ((rows + (1 << t.shift) - 1) >> t.shift),
                  items = heads * (((long long)rows * G + 127) / 128);
  if (8 * heads < 2 * sm_count && key_limit > 8192) return t;
  t.own = pairs == heads || (pairs == 2 * heads && (scored || key_limit <= 2048)) ||
          (pairs <= 3 * sm_count && pairs * key_limit <= 1100ll * sm_count) ||
          (items > sm_count && pairs <= 4 * items && pairs * key_limit <= 450ll * sm_count);
  if (!t.own) return t;
  // As many splits as are resident at once, three CTAs per SM, in clusters; of the odd sizes
  // that of 3 pays (128 pairs of up to 1500 keys 16.0 us, clusters of 2 19.7, more than are resident
  // with a joining kernel 23.8; 64 pairs of 750 in clusters of 4 11.1, of 7 18.3). Long sequences
  // take the joining kernel (64 pairs of up to 6700 keys, 4 splits 44.7, 8 with it 40.0).
  int k = 1;
  for (const int x : {8, 4, 3, 2})
    if (k == 1 && pairs * x <= (x == 8 && key_limit > 4096 ? 4 : 3) * sm_count && key_limit / x >= 64) k = x;
  t.min_share = 64;
  // enough CTAs, but one each: a long sequence among short ones is cut in two (5 sequences of 13
  // rows, 40 heads, 2000 keys the longest 36.8 -> 33.7 us, 8 of 8 rows 37.9 -> 33.4; shares
  // of 64 keys and more, and four of them, up to 3 us more; twice as many pairs 43 -> 46 so)
  if (k == 1 && pairs < 4 * sm_count && key_limit >= 1024) {
    k = 2;
    t.min_share = 512;
  }
  while (k > 1 && (size_t)n_rows * n_q * k * kPartial > room) k /= 2;
  t.splits = k;
  t.cluster = k > 1 && pairs * k <= 3 * sm_count;
  t.join = k > 1 && !t.cluster;
  return t;
}

}  // namespace llgb
