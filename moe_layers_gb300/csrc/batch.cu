// A step's tables from the requests' lengths, and rotary positions with the
// write of k and v into the paged cache.
#include <algorithm>
#include <climits>
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace dec {

// ---------------------------------------------------------------- tables
constexpr int kTableThreads = 1024;

// Exclusive sum over the block's threads (one value each); *total gets the sum.
__device__ __forceinline__ int block_exclusive_sum(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    int w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  const int before = warp > 0 ? warp_sums[warp - 1] : 0;
  *total = warp_sums[31];
  __syncthreads();
  return before + inc - v;
}

// Last index i in [0, n) with first[i] <= x (first[0] <= x).
__device__ __forceinline__ int last_at_most(const int* first, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// One CTA, thread b for request b: two running sums (rows and new blocks)
// place every row and every new block; then the threads take the new blocks
// and the rows one by one, finding each one's request by bisection in shared
// memory. Nothing is written before every length has been read.
__global__ void __launch_bounds__(kTableThreads) tables_kernel(const int32_t* ctx_len, const int32_t* new_len, int n,
                                                               const int32_t* free_blocks, const int32_t* free_count,
                                                               int32_t* table, int max_blocks, int shift, int offset,
                                                               int rows, dec_step_tables out) {
  __shared__ int s_row[kTableThreads + 1], s_base[kTableThreads + 1], s_ctx[kTableThreads], s_held[kTableThreads];
  __shared__ int s_warp[32];
  __shared__ int s_missing;
  const int b = threadIdx.x, size = 1 << shift;
  pdl_trigger();
  pdl_wait();
  if (b == 0) s_missing = 0;
  const int c = b < n ? max(ld_act_s32(ctx_len + b), 0) : 0;
  const int want = b < n ? min(max(ld_act_s32(new_len + b), 0), rows) : 0;  // clamped: the sum stays below 2^30
  const int have = max(ld_act_s32(free_count), 0);
  int total;
  const int start = block_exclusive_sum(want, s_warp, &total);
  const int r0 = min(start, rows), r1 = min(start + want, rows);
  const int used = min(total, rows);
  const int held = (int)min(((long long)c + size - 1) >> shift, (long long)max_blocks);
  const int need = (int)min(((long long)c + (r1 - r0) + size - 1) >> shift, (long long)max_blocks) - held;
  int fresh;
  const int base = block_exclusive_sum(need, s_warp, &fresh);
  s_row[b] = r0;
  s_base[b] = base;
  s_ctx[b] = c;
  s_held[b] = held;
  __syncthreads();
  if (b < n) {
    out.row_start[b] = r0;
    out.own_len[b] = (int)min((long long)c + (r1 - r0), (long long)INT_MAX);
  }
  if (b == 0) {
    out.row_start[n] = used;
    out.left[0] = max(have - fresh, 0);
  }
  auto fresh_block = [&](int i) { return i < have ? ld_act_s32(free_blocks + (have - 1 - i)) : -1; };
  for (int i = threadIdx.x; i < fresh; i += blockDim.x) {
    const int q = last_at_most(s_base, n, i);
    table[(long long)q * max_blocks + s_held[q] + (i - s_base[q])] = fresh_block(i);
  }
  int missing = 0;
  for (int t = threadIdx.x; t < rows; t += blockDim.x) {
    int slot = -1, position = 0;
    if (t < used) {
      const int q = last_at_most(s_row, n, t);
      const long long j = (long long)s_ctx[q] + (t - s_row[q]);
      const long long blk = j >> shift;
      int id = -1;
      if (blk < s_held[q])
        id = ld_act_s32(table + (long long)q * max_blocks + blk);
      else if (blk < max_blocks)
        id = fresh_block(s_base[q] + (int)(blk - s_held[q]));
      const long long sl = (long long)id * size + (j & (size - 1));
      slot = id >= 0 && sl <= INT_MAX ? (int)sl : -1;
      missing += slot < 0;
      position = (int)min((long long)offset + j, (long long)INT_MAX);
    }
    out.positions[t] = position;
    out.slots[t] = slot;
  }
  if (missing) atomicAdd(&s_missing, missing);
  __syncthreads();
  if (b == 0) out.left[1] = s_missing;
}

cudaError_t launch_tables(dec_handle* h, const int32_t* ctx_len, const int32_t* new_len, int n,
                          const int32_t* free_blocks, const int32_t* free_count, int32_t* table, int max_blocks,
                          int block_size, int offset, int rows, const dec_step_tables& out, cudaStream_t s) {
  int shift = 0;
  while ((1 << shift) < block_size) ++shift;
  return launch_k(h, tables_kernel, dim3(1), dim3(kTableThreads), 0, s, ctx_len, new_len, n, free_blocks, free_count,
                  table, max_blocks, shift, offset, rows, out);
}

// ---------------------------------------------------------------- rotary positions
// Phase step of pair i in 2^-64 turns (64-bit floating point).
__global__ void __launch_bounds__(64) rope_phases_kernel(uint64_t* phases, int r, double base, int scaling,
                                                         double factor, double length, double low, double high) {
  const int i = threadIdx.x;
  pdl_trigger();
  pdl_wait();
  if (i >= r / 2) return;
  constexpr double kTwoPi = 6.283185307179586476925;
  const double b = scaling == DEC_ROPE_NTK ? base * pow(factor, (double)r / (r - 2)) : base;
  const double f = pow(b, -2.0 * i / r);
  double g = f;
  if (scaling == DEC_ROPE_LINEAR) g = f / factor;
  if (scaling == DEC_ROPE_BANDS) {
    const double k = fmin(fmax((length * f / kTwoPi - low) / (high - low), 0.0), 1.0);
    g = k * f + (1.0 - k) * f / factor;
  }
  if (scaling == DEC_ROPE_YARN) {
    const double lb = 2.0 * log(base);
    const double lo = fmax(floor(r * log(length / (high * kTwoPi)) / lb), 0.0);
    const double hi = fmin(ceil(r * log(length / (low * kTwoPi)) / lb), (double)(r - 1));
    const double k = 1.0 - fmin(fmax((i - lo) / fmax(hi - lo, 0.001), 0.0), 1.0);
    g = k * f + (1.0 - k) * f / factor;
  }
  // f <= 1 radian: below a sixth of a turn, so the product stays below 2^62
  phases[i] = (uint64_t)__double2ull_rn(g / kTwoPi * 18446744073709551616.0);
}

cudaError_t launch_rope_phases(dec_handle* h, uint64_t* phases, int r, double base, int scaling, double factor,
                               double length, double low, double high, cudaStream_t s) {
  return launch_k(h, rope_phases_kernel, dim3(1), dim3(64), 0, s, phases, r, base, scaling, factor, length, low,
                  high);
}

// cos and sin of `position` steps of `phase` (2^-64 turns): the product wraps
// at whole turns, its top 32 bits are the angle in [-1/2, 1/2) turns to 2^-32.
__device__ __forceinline__ void rope_angle(uint64_t phase, int position, float magnitude, float* c, float* s) {
  const uint64_t turns = phase * (uint64_t)(int64_t)position;
  const float half_turns = (float)(int32_t)(turns >> 32) * 4.656612873077393e-10f;  // 2^-31
  sincospif(half_turns, s, c);
  *c *= magnitude;
  *s *= magnitude;
}

struct RopeParams {
  const uint16_t *q, *k, *v;
  long long ldq, ldk, ldv, ldqo;
  uint16_t *qo, *ck, *cv;
  long long block_stride;
  const int32_t *positions, *slots;
  const uint64_t* phases;
  float magnitude;
  int q_heads, kv_heads, dim, rot, interleaved, shift, slots_n;
};

__device__ __forceinline__ uint32_t pack_bf(float a, float b) { return (uint32_t)f2bf(a) | ((uint32_t)f2bf(b) << 16); }

// One CTA per row. The row's cosines and sines are computed once into shared
// memory; a work item is 8 elements of a head (16 with the half layout's
// partners), read, turned and written by one thread, so q may be turned in
// place.
__global__ void __launch_bounds__(256) rope_kernel(const RopeParams P) {
  __shared__ float s_cos[64], s_sin[64];
  const int t = blockIdx.x;
  pdl_trigger();
  pdl_wait();
  const int pos = ld_act_s32(P.positions + t), slot = ld_act_s32(P.slots + t);
  if (threadIdx.x < P.rot / 2) {
    float c, s;
    rope_angle(P.phases[threadIdx.x], pos, P.magnitude, &c, &s);
    s_cos[threadIdx.x] = c;
    s_sin[threadIdx.x] = s;
  }
  __syncthreads();
  const int d8 = P.dim / 8, turn8 = P.interleaved ? P.rot / 8 : P.rot / 16;  // items that turn
  const int per_head = P.interleaved ? d8 : d8 - P.rot / 16;
  const bool write = slot >= 0 && slot < P.slots_n;
  const long long dst = write ? (long long)(slot >> P.shift) * P.block_stride +
                                    (long long)(slot & ((1 << P.shift) - 1)) * P.dim
                              : 0;
  const long long head_step = (long long)P.dim << P.shift;
  const int nq = P.q_heads * per_head, nk = write ? P.kv_heads * per_head : 0, nv = write ? P.kv_heads * d8 : 0;
  for (int it = threadIdx.x; it < nq + nk + nv; it += blockDim.x) {
    if (it >= nq + nk) {
      const int head = (it - nq - nk) / d8, i = (it - nq - nk) % d8;
      *reinterpret_cast<uint4*>(P.cv + dst + head * head_step + i * 8) =
          ld_act16(P.v + t * P.ldv + (long long)head * P.dim + i * 8);
      continue;
    }
    const int at = it < nq ? it : it - nq;
    const int head = at / per_head, i = at % per_head;
    const uint16_t* src = it < nq ? P.q + t * P.ldq + (long long)head * P.dim
                                  : P.k + t * P.ldk + (long long)head * P.dim;
    uint16_t* to = it < nq ? P.qo + t * P.ldqo + (long long)head * P.dim : P.ck + dst + head * head_step;
    if (i >= turn8) {  // an element behind the rotary part
      const int e = (P.interleaved ? i : i + P.rot / 16) * 8;
      *reinterpret_cast<uint4*>(to + e) = ld_act16(src + e);
    } else if (P.interleaved) {
      const uint4 x = ld_act16(src + i * 8);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
      uint32_t o[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float a = bf_lo(w[p]), b = bf_hi(w[p]), c = s_cos[i * 4 + p], s = s_sin[i * 4 + p];
        o[p] = pack_bf(a * c - b * s, b * c + a * s);
      }
      *reinterpret_cast<uint4*>(to + i * 8) = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
      const int half = P.rot / 2;
      const uint4 xa = ld_act16(src + i * 8), xb = ld_act16(src + half + i * 8);
      const uint32_t wa[4] = {xa.x, xa.y, xa.z, xa.w}, wb[4] = {xb.x, xb.y, xb.z, xb.w};
      uint32_t oa[4], ob[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float c0 = s_cos[i * 8 + 2 * p], s0 = s_sin[i * 8 + 2 * p];
        const float c1 = s_cos[i * 8 + 2 * p + 1], s1 = s_sin[i * 8 + 2 * p + 1];
        const float a0 = bf_lo(wa[p]), a1 = bf_hi(wa[p]), b0 = bf_lo(wb[p]), b1 = bf_hi(wb[p]);
        oa[p] = pack_bf(a0 * c0 - b0 * s0, a1 * c1 - b1 * s1);
        ob[p] = pack_bf(b0 * c0 + a0 * s0, b1 * c1 + a1 * s1);
      }
      *reinterpret_cast<uint4*>(to + i * 8) = make_uint4(oa[0], oa[1], oa[2], oa[3]);
      *reinterpret_cast<uint4*>(to + half + i * 8) = make_uint4(ob[0], ob[1], ob[2], ob[3]);
    }
  }
}

cudaError_t launch_rope_append(dec_handle* h, const dec_rope& rope, const uint16_t* q, long long ldq,
                               const uint16_t* k, long long ldk, const uint16_t* v, long long ldv, uint16_t* qo,
                               long long ldqo, int rows, int q_heads, const int32_t* positions, const int32_t* slots,
                               const dec_kv_cache& cache, cudaStream_t s) {
  RopeParams P;
  P.q = q;
  P.k = k;
  P.v = v;
  P.ldq = ldq;
  P.ldk = ldk;
  P.ldv = ldv;
  P.ldqo = ldqo;
  P.qo = qo;
  P.ck = cache.k;
  P.cv = cache.v;
  P.block_stride = cache.block_stride;
  P.positions = positions;
  P.slots = slots;
  P.phases = rope.phases;
  P.magnitude = rope.magnitude;
  P.q_heads = q_heads;
  P.kv_heads = cache.kv_heads;
  P.dim = cache.head_dim;
  P.rot = rope.rotary_dim;
  P.interleaved = rope.interleaved;
  P.shift = 0;
  while ((1 << P.shift) < cache.block_size) ++P.shift;
  P.slots_n = cache.blocks << P.shift;
  return launch_k(h, rope_kernel, dim3(rows), dim3(256), 0, s, P);
}

}  // namespace dec
