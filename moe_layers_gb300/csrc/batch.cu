// A step's tables from the requests' lengths, and rotary positions with the
// write of k and v into the paged cache.
#include <algorithm>
#include <climits>
#include <cmath>

#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"

namespace dec {

// ---------------------------------------------------------------- tables
constexpr int kTableThreads = 1024;

// Exclusive sum over the block's threads (one value each); *total gets the sum.
__device__ __forceinline__ int block_exclusive_sum(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  // every warp adds up the sums itself
  int w = lane < warps ? warp_sums[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += u;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  __syncthreads();
  return (warp > 0 ? before : 0) + inc - v;
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

// Thread b for request b: two running sums (rows and new blocks) place every
// row and every new block; then the threads take the new blocks and the rows,
// four rows at a time, finding a row's request by bisection in shared memory.
// A few hundred rows are one CTA, bound by the latency of a launch and three
// dependent reads (2.4 us for 64 requests). Prompts take a cluster of 8 CTAs that
// each repeat the sums and share the rows: no output may be written before
// every CTA has read the lengths, as own_len and left may lie over inputs, and a
// cluster can wait for that without a workspace. 69,000 rows of 24 prompts take
// 8.9 us, 2.8 of them without the rows (4 CTAs 13 us; 16, past the portable
// cluster, 7.4; reads for several fours of rows under way at once, the same).
template <bool CLUSTER>
__global__ void __launch_bounds__(kTableThreads) tables_kernel(const int32_t* ctx_len, const int32_t* new_len, int n,
                                                               const int32_t* free_blocks, const int32_t* free_count,
                                                               int32_t* table, int max_blocks, int shift, int offset,
                                                               int rows, dec_step_tables out) {
  namespace cg = cooperative_groups;
  __shared__ int s_row[kTableThreads + 1], s_base[kTableThreads], s_ctx[kTableThreads], s_held[kTableThreads];
  __shared__ int s_warp[32];
  __shared__ int s_missing;
  const int b = threadIdx.x, size = 1 << shift;
  const int first = blockIdx.x * blockDim.x + b, step = gridDim.x * blockDim.x;
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
  if (b == n - 1) s_row[n] = r1;
  __syncthreads();
  if (CLUSTER) cg::this_cluster().sync();  // every CTA has read the lengths and the count
  if (blockIdx.x == 0) {
    if (b < n) {
      out.row_start[b] = r0;
      out.own_len[b] = (int)min((long long)c + (r1 - r0), (long long)INT_MAX);
    }
    if (b == 0) {
      out.row_start[n] = used;
      out.left[0] = max(have - fresh, 0);
    }
  }
  for (int i = first; i < fresh; i += step) {
    const int q = last_at_most(s_base, n, i);
    table[(long long)q * max_blocks + s_held[q] + (i - s_base[q])] =
        i < have ? ld_act_s32(free_blocks + (have - 1 - i)) : -1;
  }
  int missing = 0;
  // cache id of block blk of request q
  auto block_of = [&](int q, uint32_t blk) {
    const int32_t* p = nullptr;
    if (blk < (uint32_t)s_held[q]) {
      p = table + (long long)q * max_blocks + blk;
    } else if (blk < (uint32_t)max_blocks) {
      const int i = have - 1 - s_base[q] - (int)(blk - s_held[q]);
      if (i >= 0) p = free_blocks + i;
    }
    return p ? ld_act_s32(p) : -1;
  };
  // own token that is row t of request q (below 2^31 + 2^20)
  auto token = [&](int q, int t) { return (uint32_t)s_ctx[q] + (uint32_t)(t - s_row[q]); };
  // position and slot of a request's token j in the block with cache id `id`
  auto place = [&](uint32_t j, int id, int& position, int& slot) {
    slot = id >= 0 && id <= INT_MAX >> shift ? (id << shift) + (int)(j & (size - 1)) : -1;
    missing += slot < 0;
    position = (int)min((uint32_t)offset + min(j, (uint32_t)INT_MAX), (uint32_t)INT_MAX);
  };
  const bool wide = ((reinterpret_cast<uintptr_t>(out.positions) | reinterpret_cast<uintptr_t>(out.slots)) & 15) == 0;
  if (CLUSTER && wide) {
    for (int t0 = 4 * first; t0 < rows; t0 += 4 * step) {
      int slot[4] = {-1, -1, -1, -1}, position[4] = {0, 0, 0, 0};
      int q = t0 < used ? last_at_most(s_row, n, t0) : 0, at = -1, id = -1;
      uint32_t blk = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (t0 + k < used) {
          while (s_row[q + 1] <= t0 + k) ++q;
          const uint32_t j = token(q, t0 + k);
          if (at != q || blk != j >> shift) {  // one read for rows in the same block
            at = q;
            blk = j >> shift;
            id = block_of(q, blk);
          }
          place(j, id, position[k], slot[k]);
        }
      if (t0 + 4 <= rows) {
        *reinterpret_cast<int4*>(out.positions + t0) = make_int4(position[0], position[1], position[2], position[3]);
        *reinterpret_cast<int4*>(out.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      } else {
#pragma unroll
        for (int k = 0; k < 3; ++k)
          if (t0 + k < rows) out.positions[t0 + k] = position[k], out.slots[t0 + k] = slot[k];
      }
    }
  } else {
    for (int t = first; t < rows; t += step) {
      int slot = -1, position = 0;
      if (t < used) {
        const int q = last_at_most(s_row, n, t);
        const uint32_t j = token(q, t);
        place(j, block_of(q, j >> shift), position, slot);
      }
      out.positions[t] = position;
      out.slots[t] = slot;
    }
  }
  if (CLUSTER) {
    cg::cluster_group cluster = cg::this_cluster();
    if (missing) atomicAdd(cluster.map_shared_rank(&s_missing, 0), missing);
    cluster.sync();
  } else {
    if (missing) atomicAdd(&s_missing, missing);
    __syncthreads();
  }
  if (first == 0) out.left[1] = s_missing;
}

cudaError_t launch_tables(dec_handle* h, const int32_t* ctx_len, const int32_t* new_len, int n,
                          const int32_t* free_blocks, const int32_t* free_count, int32_t* table, int max_blocks,
                          int block_size, int offset, int rows, const dec_step_tables& out, cudaStream_t s) {
  int shift = 0;
  while ((1 << shift) < block_size) ++shift;
  cudaLaunchConfig_t cfg = {};
  // The cluster from 4096 rows on, where one CTA's rows take longer than the two
  // cluster barriers (16 requests, one CTA against 8: 3000 rows 4.4 and 4.8 us,
  // 4096 rows 5.4 and 4.6). Below, a thread for each request and row, up to 1024
  // (512 rows 2.6 us; by 128 threads 4.4, by 1024 3.0; 64 rows 2.0, by 1024 2.6).
  const int ctas = rows >= 4096 ? 8 : 1;
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(ctas > 1 ? kTableThreads : std::min(kTableThreads, (std::max(n, rows) + 127) & ~127));
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = h->pdl ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, ctas > 1 ? tables_kernel<true> : tables_kernel<false>, ctx_len, new_len, n,
                            free_blocks, free_count, table, max_blocks, shift, offset, rows, out);
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
  int rows, q_heads, kv_heads, dim, rot, interleaved, shift, slots_n;
};

// A row's heads are cut into items of 8 elements (with the half layout, of 8
// and their 8 partners); a thread reads, turns and writes whole items, so q may
// be turned in place. Bound by the copy. A CTA has 128 NI of a row's items for
// one row after another: where an item lies within its row is worked out once,
// the reads of a row are all issued before any is used, and its cosines and
// sines are computed under them. NI = 2 for many rows; few rows take NI = 1, so
// that a row is spread over several CTAs, as the latency of one CTA's reads is
// then all there is.
constexpr int kRopeThreads = 128;

template <int NI, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams P) {
  __shared__ alignas(16) float s_cos[2][64], s_sin[2][64];
  const int d8 = P.dim / 8, turn8 = INTER ? P.rot / 8 : P.rot / 16;  // items of a head that turn
  const int per_head = INTER ? d8 : d8 - P.rot / 16;
  const int half = P.rot / 2;
  const int nq = P.q_heads * per_head, nk = P.kv_heads * per_head, n = nq + nk + P.kv_heads * d8;
  int src[NI], dst[NI], kind[NI], turn[NI];  // kind: 0 q, 1 k, 2 v, -1 none; turn: first pair, -1 for a copy
#pragma unroll
  for (int k = 0; k < NI; ++k) {
    const int it = (blockIdx.x * NI + k) * kRopeThreads + threadIdx.x;
    kind[k] = it >= n ? -1 : it >= nq + nk ? 2 : it >= nq ? 1 : 0;
    const int at = it - (kind[k] == 2 ? nq + nk : kind[k] == 1 ? nq : 0), each = kind[k] == 2 ? d8 : per_head;
    const int head = at / each, i = at - head * each;
    const bool turns = kind[k] < 2 && i < turn8;
    const int e = (INTER || kind[k] == 2 || turns ? i : i + P.rot / 16) * 8;
    src[k] = head * P.dim + e;
    dst[k] = kind[k] == 0 ? src[k] : head * (P.dim << P.shift) + e;
    turn[k] = turns ? i * (INTER ? 4 : 8) : -1;
  }
  pdl_trigger();
  pdl_wait();
  const uint64_t phase = threadIdx.x < half ? P.phases[threadIdx.x] : 0;
  int t = blockIdx.y, pos = ld_act_s32(P.positions + t), slot = ld_act_s32(P.slots + t);
  for (int buf = 0; t < P.rows; buf ^= 1) {
    uint4 xa[NI], xb[NI];
#pragma unroll
    for (int k = 0; k < NI; ++k) {
      if (kind[k] < 0) continue;
      const uint16_t* from = (kind[k] == 0 ? P.q + t * P.ldq : kind[k] == 1 ? P.k + t * P.ldk : P.v + t * P.ldv) + src[k];
      xa[k] = ld_act16(from);
      if (!INTER && turn[k] >= 0) xb[k] = ld_act16(from + half);
    }
    const int next = t + gridDim.y;
    int next_pos = 0, next_slot = 0;
    if (next < P.rows) next_pos = ld_act_s32(P.positions + next), next_slot = ld_act_s32(P.slots + next);
    if (threadIdx.x < half) rope_angle(phase, pos, P.magnitude, &s_cos[buf][threadIdx.x], &s_sin[buf][threadIdx.x]);
    __syncthreads();  // one a row: the other buffer is written only behind the next one
    const bool write = slot >= 0 && slot < P.slots_n;
    const long long at = (long long)(slot >> P.shift) * P.block_stride + (slot & ((1 << P.shift) - 1)) * P.dim;
#pragma unroll
    for (int k = 0; k < NI; ++k) {
      if (kind[k] < 0 || (kind[k] > 0 && !write)) continue;
      uint16_t* to = (kind[k] == 0 ? P.qo + t * P.ldqo : (kind[k] == 1 ? P.ck : P.cv) + at) + dst[k];
      if (turn[k] < 0) {
        *reinterpret_cast<uint4*>(to) = xa[k];
        continue;
      }
      const float* cs = s_cos[buf] + turn[k];
      const float* sn = s_sin[buf] + turn[k];
      if (INTER) {
        const uint32_t w[4] = {xa[k].x, xa[k].y, xa[k].z, xa[k].w};
        const float4 c4 = *reinterpret_cast<const float4*>(cs), s4 = *reinterpret_cast<const float4*>(sn);
        const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
        uint32_t o[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const float a = bf_lo(w[p]), b = bf_hi(w[p]);
          o[p] = pack_bf16x2(a * c[p] - b * s[p], b * c[p] + a * s[p]);
        }
        *reinterpret_cast<uint4*>(to) = make_uint4(o[0], o[1], o[2], o[3]);
      } else {
        const uint32_t wa[4] = {xa[k].x, xa[k].y, xa[k].z, xa[k].w}, wb[4] = {xb[k].x, xb[k].y, xb[k].z, xb[k].w};
        uint32_t oa[4], ob[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 c4 = *reinterpret_cast<const float4*>(cs + 4 * h), s4 = *reinterpret_cast<const float4*>(sn + 4 * h);
          const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const uint32_t va = wa[2 * h + p], vb = wb[2 * h + p];
            const float a0 = bf_lo(va), a1 = bf_hi(va), b0 = bf_lo(vb), b1 = bf_hi(vb);
            oa[2 * h + p] = pack_bf16x2(a0 * c[2 * p] - b0 * s[2 * p], a1 * c[2 * p + 1] - b1 * s[2 * p + 1]);
            ob[2 * h + p] = pack_bf16x2(b0 * c[2 * p] + a0 * s[2 * p], b1 * c[2 * p + 1] + a1 * s[2 * p + 1]);
          }
        }
        *reinterpret_cast<uint4*>(to) = make_uint4(oa[0], oa[1], oa[2], oa[3]);
        *reinterpret_cast<uint4*>(to + half) = make_uint4(ob[0], ob[1], ob[2], ob[3]);
      }
    }
    t = next;
    pos = next_pos;
    slot = next_slot;
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
  P.rows = rows;
  const int d8 = P.dim / 8, per_head = P.interleaved ? d8 : d8 - P.rot / 16;
  const int items = (P.q_heads + P.kv_heads) * per_head + P.kv_heads * d8;
  // One item a thread up to 2048 threads an SM (10 to 12 CTAs are resident, at 37
  // to 44 registers, the rest follow). Above, two a thread and up to 60 CTAs an SM:
  // more than the 9 or 10 that are resident (56 and 46 registers), so that those
  // that begin overlap those that end, and few enough to take several rows each
  // (8192 rows of 64 + 16 + 16 heads of 128: 60.6 us; with one wave of CTAs 73, a
  // CTA for every row 63, four items a thread 65, one 66).
  const bool few = (long long)rows * items <= 2048LL * h->sms;
  const int ni = few ? 1 : 2;
  const int chunks = (items + kRopeThreads * ni - 1) / (kRopeThreads * ni);
  const int wave = (few ? 16 : 60) * h->sms;
  const dim3 grid(chunks, std::max(1, std::min(rows, wave / chunks)));
  if (P.interleaved)
    return few ? launch_k(h, rope_kernel<1, true>, grid, dim3(kRopeThreads), 0, s, P)
               : launch_k(h, rope_kernel<2, true>, grid, dim3(kRopeThreads), 0, s, P);
  return few ? launch_k(h, rope_kernel<1, false>, grid, dim3(kRopeThreads), 0, s, P)
             : launch_k(h, rope_kernel<2, false>, grid, dim3(kRopeThreads), 0, s, P);
}

}  // namespace dec
