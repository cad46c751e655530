// Head norms, rotation and KV-cache append of new rows in one pass, and the
// table of scaled rotation angles ("Llama2架构与推理全解析" §1.2 RMSNorm, here
// over each Q / K head; §1.4 RoPE; §2.4 append).
//
//   u = x / sqrt(mean(x^2) + eps) * gain           (Q and K heads, optional)
//   (y0, y1) = (u0 c - u1 s, u0 s + u1 c)          for the rotating pairs
//
// Bound by the bytes of the rows: each source value is read once and each
// output written once. A thread owns 8 values of one head as two groups of 4
// at e0 and e1: for the half layout e0 = 4u and e1 = rotary/2 + 4u, so both
// values of a pair sit in one thread and nothing is exchanged; else 8
// consecutive values. The lanes of a head (16 at 128 values) add up its
// squares with butterflies. Measured: 8192 rows of 32 + 2 x 32 heads of 128, fp32
// source, norms and side outputs: 122 us, 6.07 TB/s (90 % of the copy rate; the
// scheduler issues in 80 % of the cycles); one row 2.6 us, a launch; 200 and 600 rows
// 6.8 and 10.0 us (2.7 and 8.0 us of bytes). 4000 rows to an E4M3 cache: 67 us from
// fp32 and 80 us from bf16 rows (48 and 34 us of bytes); why was not profiled.
#include "common.cuh"
#include "internal.h"

namespace llgb {

namespace {

__device__ __forceinline__ void load4(const float* p, float* v) {
  const float4 x = *reinterpret_cast<const float4*>(p);
  v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
}
__device__ __forceinline__ void load4(const bf16* p, float* v) {
  const uint2 x = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(x.x << 16);
  v[1] = __uint_as_float(x.x & 0xffff0000u);
  v[2] = __uint_as_float(x.y << 16);
  v[3] = __uint_as_float(x.y & 0xffff0000u);
}
__device__ __forceinline__ void store4(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(bf16* p, const float* v) {  // nearest even, the cache's type
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
}
__device__ __forceinline__ uint32_t e4m3x4(const float* v, float scale) {
  return (uint32_t)f32_to_e4m3(v[0] / scale) | (uint32_t)f32_to_e4m3(v[1] / scale) << 8 |
         (uint32_t)f32_to_e4m3(v[2] / scale) << 16 | (uint32_t)f32_to_e4m3(v[3] / scale) << 24;
}

// The sequence of packed row r: the largest b with cu[b] <= r, or -1 when no
// sequence owns the row. A whole warp searches 32 ways per step, one load
// each, so 1024 sequences cost two dependent loads.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int n_seq, int r, int lane) {
  int lo = 0, n = n_seq;
  while (n > 1) {
    const int step = (n + 31) / 32, i = lane * step;
    const uint32_t m = __ballot_sync(0xffffffffu, i < n && cu[lo + i] <= r);
    const int k = max(0, __popc(m) - 1);
    lo += k * step;
    n = max(1, min(step, n - k * step));
  }
  return cu[lo] <= r && r < cu[lo + 1] ? lo : -1;
}

constexpr int RN_THREADS = 256;

// One block: `per_block` chunks of RN_THREADS / lanes heads of one row; grid:
// blocks of a row, rows, flattened. What depends on the row alone (its sequence,
// position, page) is a chain of dependent loads, so it is looked up once per
// block, beside the first chunk's values, and the next chunk's values are
// loaded before the current ones are used.
template <typename S, typename T>
__global__ void __launch_bounds__(RN_THREADS) rope_norm_append_kernel(RopeNormArgs a, int lanes,
                                                                      int chunks, int per_block) {
  grid_dep_wait();
  grid_dep_launch();
  const int d = a.head_dim, heads = a.n_q + 2 * a.n_kv;
  const int blocks = (chunks + per_block - 1) / per_block;
  const int r = blockIdx.x / blocks, chunk0 = (blockIdx.x - r * blocks) * per_block;
  const int step = RN_THREADS / lanes;  // heads of a chunk
  const int u = threadIdx.x & (lanes - 1);
  const int head0 = chunk0 * step + threadIdx.x / lanes;
  const int head_end = min(heads, (chunk0 + per_block) * step);
  const bool unit = u < d / 8;
  int e0 = 8 * u, e1 = 8 * u + 4;
  if (a.half && u < a.rotary / 8) {
    e0 = 4 * u;
    e1 = a.rotary / 2 + 4 * u;
  }
  const S* src = reinterpret_cast<const S*>(a.qkv) + (size_t)r * a.ld;
  float nx[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (unit && head0 < head_end) {
    load4(src + (size_t)head0 * d + e0, nx);
    load4(src + (size_t)head0 * d + e1, nx + 4);
  }
  // the row's sequence and position
  int b = r, pos;
  if (a.cu_rows) {
    b = sequence_of(a.cu_rows, a.n_seq, r, threadIdx.x & 31);
    if (b < 0) return;  // a row of no sequence
    pos = a.start_pos[b] + (r - a.cu_rows[b]);
  } else {
    pos = a.start_pos[b];
  }
  const bool pos_ok = pos >= 0 && (a.rotary == 0 || pos < a.n_pos);
  if (!pos_ok && chunk0 == 0 && threadIdx.x == 0) flag(a.status, LLAMA_FLAG_POS_RANGE);
  // its cache slot, of K/V head 0 (the heads lie slot_step slots apart); -1: not cached
  long long slot0 = -1;
  const long long slot_step = a.page_size == 0 ? a.capacity : a.page_size;
  if (pos_ok && head_end > a.n_q) {
    uint32_t bad = 0;
    if (a.page_size == 0) {
      if (pos < a.capacity && b < a.batch_cap)
        slot0 = ((long long)a.layer * a.batch_cap + b) * a.n_kv * a.capacity + pos;
      else
        bad = LLAMA_FLAG_POS_RANGE;
    } else {
      const int pi = pos / a.page_size;
      if (pi < a.max_pages) {
        const int page = a.page_table[(size_t)b * a.max_pages + pi];
        if (page >= 0 && page < a.n_pages)
          slot0 = ((long long)a.layer * a.n_pages + page) * a.n_kv * a.page_size + (pos - pi * a.page_size);
        else
          bad = LLAMA_FLAG_PAGE_RANGE;
      } else {
        bad = LLAMA_FLAG_POS_RANGE;
      }
    }
    if (bad && threadIdx.x == 0) flag(a.status, bad);
  }
  // (the checked build: the layer's slots end there)
  const long long slots = (long long)(a.layer + 1) * (a.page_size == 0 ? a.batch_cap : a.n_pages) * a.n_kv * slot_step;
  if (slot0 >= 0 && !bc_ok(slot0 + (a.n_kv - 1) * slot_step < slots, a.status)) slot0 = -1;
  if (!bc_ok(r < a.n_rows && (!a.cu_rows || (r >= a.cu_rows[b] && r < a.cu_rows[b + 1])), a.status)) return;
  // this thread's four angles: the same ones for every head
  float c[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
  const bool turns = u < a.rotary / 8;
  if (turns && pos_ok) {
    const float4* cs4 = reinterpret_cast<const float4*>(a.table + (size_t)pos * (a.rotary / 2) + 4 * u);
    const float4 c01 = cs4[0], c23 = cs4[1];
    c[0] = c01.x; c[1] = c01.z; c[2] = c23.x; c[3] = c23.z;
    sn[0] = c01.y; sn[1] = c01.w; sn[2] = c23.y; sn[3] = c23.w;
  }
  const float rd = 1.f / (float)d;
  const bool norms = a.q_gain || a.k_gain;
#pragma unroll 1
  for (int head = head0; head - head0 + chunk0 * step < head_end; head += step) {  // a block's trips are equal
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = nx[i];
    const bool on = unit && head < head_end;
    if (unit && head + step < head_end) {
      load4(src + (size_t)(head + step) * d + e0, nx);
      load4(src + (size_t)(head + step) * d + e1, nx + 4);
    }
    const bool is_v = head >= a.n_q + a.n_kv;
    if (norms) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
      if (!unit) ss = 0.f;
      for (int o = lanes >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const T* gain = reinterpret_cast<const T*>(is_v ? nullptr : head < a.n_q ? a.q_gain : a.k_gain);
      if (on && gain) {
        // bf16 outputs keep nothing of the last bits of 1 / sqrt
        const float inv = sizeof(T) == 2 ? rsqrtf(fmaf(ss, rd, a.eps)) : 1.0f / sqrtf(ss / (float)d + a.eps);
        float g[8];
        load4(gain + e0, g);
        load4(gain + e1, g + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] * inv * g[i];
      }
    }
    if (!on) continue;
    if (!pos_ok) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
    } else if (turns && !is_v) {
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int i0 = a.half ? p : 2 * p, i1 = a.half ? 4 + p : 2 * p + 1;
        const float x0 = v[i0], x1 = v[i1];
        v[i0] = x0 * c[p] - x1 * sn[p];
        v[i1] = x0 * sn[p] + x1 * c[p];
      }
    }
    if (head < a.n_q) {
      T* dst = reinterpret_cast<T*>(a.q_out) + ((size_t)r * a.n_q + head) * d;
      store4(dst + e0, v);
      store4(dst + e1, v + 4);
      continue;
    }
    const int g = is_v ? head - a.n_q - a.n_kv : head - a.n_q;
    if (void* side = is_v ? a.v_out : a.k_out) {
      T* dst = reinterpret_cast<T*>(side) + ((size_t)r * a.n_kv + g) * d;
      store4(dst + e0, v);
      store4(dst + e1, v + 4);
    }
    if (slot0 < 0) continue;
    const size_t slot = (size_t)(slot0 + g * slot_step);
    void* cache = is_v ? a.v_cache : a.k_cache;
    if (a.kv_fp8) {
      uint8_t* dst = reinterpret_cast<uint8_t*>(cache) + slot * d;
      const float sc = is_v ? a.v_scale : a.k_scale;
      *reinterpret_cast<uint32_t*>(dst + e0) = e4m3x4(v, sc);
      *reinterpret_cast<uint32_t*>(dst + e1) = e4m3x4(v + 4, sc);
    } else {
      T* dst = reinterpret_cast<T*>(cache) + slot * d;
      store4(dst + e0, v);
      store4(dst + e1, v + 4);
    }
  }
}

// table[m * n + j] = magnitude * (cos, sin)(m * f_j), n = rotary_dim / 2; the
// angles in fp64 (a far position's angle has no fp32 digits left), rounded once.
__global__ void rope_scaled_table_kernel(llama_rope_scaling s, int n, int n_pos, float2* table) {
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= (long long)n_pos * n) return;
  const int m = (int)(i / n), j = (int)(i - (long long)m * n);
  double f = pow((double)s.theta, -(double)j / (double)n);
  if (s.kind == LLAMA_ROPE_LINEAR) {
    f /= (double)s.factor;
  } else if (s.kind == LLAMA_ROPE_BANDS) {
    const double turns = (double)s.original_len * f / 6.283185307179586476925;
    const double lo = (double)s.low_turns, hi = (double)s.high_turns;
    const double g = fmin(1.0, fmax(0.0, (turns - lo) / (hi - lo)));
    f *= g + (1.0 - g) / (double)s.factor;
  }
  double sn, cs;
  sincos((double)m * f, &sn, &cs);
  table[i] = make_float2((float)(cs * (double)s.magnitude), (float)(sn * (double)s.magnitude));
}

template <typename S, typename T>
cudaError_t launch_rn(const RopeNormArgs& a, cudaStream_t st) {
  int lanes = 1;
  while (lanes * 8 < a.head_dim) lanes <<= 1;
  const int per = RN_THREADS / lanes, chunks = (a.n_q + 2 * a.n_kv + per - 1) / per;
  // few rows: a block per chunk (latency); many (a wave of 8 blocks per SM and
  // more): a block per row. The rule was measured at 1 and at 8192 rows; 96 heads take
  // the second form from 203 rows on
  const int per_block = (long long)chunks * a.n_rows <= 8 * a.sm_count ? 1 : chunks;
  const long long blocks = (long long)(chunks + per_block - 1) / per_block * a.n_rows;
  return launch_k(rope_norm_append_kernel<S, T>, dim3((unsigned)blocks), dim3(RN_THREADS), 0, st, 0,
                  a, lanes, chunks, per_block);
}

}  // namespace

cudaError_t launch_rope_norm_append(int dtype, int src_dtype, const RopeNormArgs& a,
                                    cudaStream_t st) {
  if (dtype == LLAMA_F32) return launch_rn<float, float>(a, st);
  return src_dtype == LLAMA_F32 ? launch_rn<float, bf16>(a, st) : launch_rn<bf16, bf16>(a, st);
}

cudaError_t launch_rope_scaled_table(const llama_rope_scaling& s, int rotary_dim, int n_pos,
                                     float2* table, cudaStream_t st) {
  const long long n = (long long)n_pos * (rotary_dim / 2);
  rope_scaled_table_kernel<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(s, rotary_dim / 2, n_pos,
                                                                        table);
  return cudaGetLastError();
}

}  // namespace llgb
