// Attention of a decode step over the paged cache.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace dec {

// One CTA per (row, key / value head), a warp per quarter of the keys, four
// query heads at a time: lane l holds elements [l D/32, (l + 1) D/32) of the
// query, key and value rows. Running maximum and sum per head; the warps'
// parts are joined through shared memory.
template <int D>
__global__ void __launch_bounds__(128) attention_kernel(const AttentionParams P) {
  constexpr int V = D / 32, G = 4, W = 4;
  __shared__ float s_acc[W][G][D], s_m[W][G], s_l[W][G];
  const int t = blockIdx.x, kvh = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  pdl_wait();
  // the row's request: the last one whose first row is at or before t
  int b = -1, first = 0, n = 0;
  for (int r = 0; r < P.requests; ++r) {
    const int r0 = ld_act_s32(P.row_start + r), r1 = ld_act_s32(P.row_start + r + 1);
    if (t >= r0 && t < r1) b = r, first = r0, n = r1 - r0;
  }
  if (b < 0) return;
  const long long sees = (long long)ld_act_s32(P.own_len + b) - n + (t - first) + 1;
  const int own = (int)min(max(sees, 0LL), (long long)P.max_blocks << P.shift);
  const int group = P.q_heads / P.kv_heads, mask = (1 << P.shift) - 1;
  for (int g0 = 0; g0 < group; g0 += G) {
    float q[G][V], acc[G][V], m[G], l[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      m[g] = -INFINITY;
      l[g] = 0.f;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        acc[g][e] = 0.f;
        q[g][e] = g0 + g < group ? bf2f(ld_act_u16(P.q + t * P.ldq + ((long long)kvh * group + g0 + g) * D + lane * V + e))
                                 : 0.f;
      }
    }
    for (int j = warp; j < P.prefix_len + own; j += W) {
      const bool pre = j < P.prefix_len;
      const int jj = pre ? j : j - P.prefix_len;
      const int id = pre ? ld_act_s32(P.prefix_table + (jj >> P.shift))
                         : ld_act_s32(P.block_table + (long long)b * P.max_blocks + (jj >> P.shift));
      if (id < 0 || id >= P.blocks) continue;
      const long long at =
          (long long)id * P.block_stride + (((long long)kvh << P.shift) + (jj & mask)) * D + lane * V;
      float kk[V], vv[V];
#pragma unroll
      for (int e = 0; e < V; ++e) kk[e] = bf2f(ld_act_u16(P.k + at + e)), vv[e] = bf2f(ld_act_u16(P.v + at + e));
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) s = fmaf(q[g][e], kk[e], s);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        s *= P.scale;
        const float mn = fmaxf(m[g], s);
        const float ref = mn == -INFINITY ? 0.f : mn;
        const float c = expf(m[g] - ref), p = expf(s - ref);
        m[g] = mn;
        l[g] = l[g] * c + p;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[g][e] = acc[g][e] * c + p * vv[e];
      }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
#pragma unroll
      for (int e = 0; e < V; ++e) s_acc[warp][g][lane * V + e] = acc[g][e];
      if (lane == 0) s_m[warp][g] = m[g], s_l[warp][g] = l[g];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < G * D; i += blockDim.x) {
      const int g = i / D, e = i % D;
      if (g0 + g >= group) break;
      float top = -INFINITY, sum = 0.f, x = 0.f;
      for (int w = 0; w < W; ++w) top = fmaxf(top, s_m[w][g]);
      const float ref = top == -INFINITY ? 0.f : top;
      for (int w = 0; w < W; ++w) {
        const float c = expf(s_m[w][g] - ref);
        sum += s_l[w][g] * c;
        x += s_acc[w][g][e] * c;
      }
      P.out[t * P.ldo + ((long long)kvh * group + g0 + g) * D + e] = f2bf(sum > 0.f ? x / sum : (sum == 0.f ? 0.f : sum));
    }
    __syncthreads();
  }
}

size_t attention_ws_bytes(const dec_handle*, int, int, const dec_kv_cache&, const dec_batch&) { return 0; }

cudaError_t launch_attention(dec_handle* h, const AttentionParams& P, int M, cudaStream_t s) {
  const dim3 grid(M, P.kv_heads);
  if (P.dim == 64) return launch_k(h, attention_kernel<64>, grid, dim3(128), 0, s, P);
  return launch_k(h, attention_kernel<128>, grid, dim3(128), 0, s, P);
}

}  // namespace dec
