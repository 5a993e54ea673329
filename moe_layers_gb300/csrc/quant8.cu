// 8-bit numbers with scales: the norm that writes them, and the quantisation
// of weights.
//
// An e4m3 number has 3 bits of mantissa and a largest value of 448; a group of
// values shares a 32-bit scale that maps its largest absolute value to 448.
// Rows (activations) have a scale for each 128 values, weights one for each
// block of 128 x 128.
#include <algorithm>

#include "common.cuh"
#include "fp8.cuh"
#include "internal.h"

namespace dec {

// One row in a CTA of 256 threads, held in registers between its only read and
// its only write:
//   a = bf16(x + r); y = a / sqrt(mean(a^2) + eps) * gamma (fp32);
//   each 128 values of y by their largest: scale = max / 448, q = e4m3(y 448 / max)
// The vectors, their order in the sum of squares and the norm's products are
// those of the RMSNorm kernel, so y has the same bits as there. Thread t holds the
// 8-value vectors t, t + 256, ...; 16 threads of a half warp hold a group, so its
// maximum takes four shuffles. The maximum is taken over bit patterns, which puts
// NaN above every number: a group with a NaN or an infinity gets it as its scale.
//
// Bound by memory: 2 bytes in (4 with the residual), 1 + 4/128 out (3 with the
// sum kept, 5 with y as well).
template <int VPT>
__global__ void __launch_bounds__(256) norm_quant_kernel(const QuantRows P) {
  const int tid = threadIdx.x;
  const long long row = blockIdx.x;
  __shared__ float red[8];
  pdl_trigger();
  pdl_wait();
  const int H8 = P.H >> 3;
  uint4 xv[VPT];
  const uint16_t* xr = P.x + row * P.ldx;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = tid + 256 * j;
    xv[j] = v < H8 ? ld_act16(xr + (size_t)v * 8) : make_uint4(0, 0, 0, 0);
  }
  if (P.res != nullptr) {
    uint4 rv[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = tid + 256 * j;
      rv[j] = v < H8 ? ld_act16(P.res + row * P.ldr + (size_t)v * 8) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = tid + 256 * j;
      xv[j] = make_uint4(add_bf16x2(xv[j].x, rv[j].x), add_bf16x2(xv[j].y, rv[j].y), add_bf16x2(xv[j].z, rv[j].z),
                         add_bf16x2(xv[j].w, rv[j].w));
      if (P.sum != nullptr && v < H8) *reinterpret_cast<uint4*>(P.sum + row * P.lds + (size_t)v * 8) = xv[j];
    }
  }
  float rho = 1.f;
  if (P.gamma != nullptr) rho = block_rms_scale<8>(thread_sumsq<VPT, 256>(xv, H8), P.H, P.eps, red);
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = tid + 256 * j;
    if (256 * j >= H8) break;  // the whole CTA leaves together: the shuffles below take full warps
    float y[8];
    {
      const uint32_t w[4] = {xv[j].x, xv[j].y, xv[j].z, xv[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) y[2 * i] = bf_lo(w[i]), y[2 * i + 1] = bf_hi(w[i]);
      if (P.gamma != nullptr) {
        const uint4 g4 = v < H8 ? *reinterpret_cast<const uint4*>(P.gamma + (size_t)v * 8) : make_uint4(0, 0, 0, 0);
        const uint32_t g[4] = {g4.x, g4.y, g4.z, g4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y[2 * i] = y[2 * i] * rho * bf_lo(g[i]);
          y[2 * i + 1] = y[2 * i + 1] * rho * bf_hi(g[i]);
        }
      }
      if (P.y != nullptr && v < H8) {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(y[2 * i], y[2 * i + 1]);
        *reinterpret_cast<uint4*>(P.y + row * P.ldy + (size_t)v * 8) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint(y[i]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
    const Scale8 s = scale_e4m3(__uint_as_float(most));
    if (v < H8) {
      uint2 o;
      o.x = pack_e4m3x4(y[0] * s.up, y[1] * s.up, y[2] * s.up, y[3] * s.up);
      o.y = pack_e4m3x4(y[4] * s.up, y[5] * s.up, y[6] * s.up, y[7] * s.up);
      *reinterpret_cast<uint2*>(P.q + row * P.ldq + (size_t)v * 8) = o;
      if ((tid & 15) == 0) P.scales[row * P.ldsc + (v >> 4)] = s.scale;
    }
  }
}

// A block of 128 x 128 weights in a CTA of 256 threads: 8-value vector c = t % 16
// of the rows t / 16, t / 16 + 16, ... Read once at load time, so it is kept plain.
__global__ void __launch_bounds__(256) weight_quant_kernel(const uint16_t* W, long long N, int K, uint8_t* q,
                                                           float* scales) {
  const int t = threadIdx.x, c = t & 15;
  const long long n0 = (long long)blockIdx.x * 128 + (t >> 4);
  const int k = blockIdx.y * 128 + c * 8;
  __shared__ uint32_t s_most;
  if (t == 0) s_most = 0;
  pdl_wait();
  __syncthreads();
  uint4 v[8];
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = n0 + 16 * i < N && k < K ? ld_act16(W + (n0 + 16 * i) * K + k) : make_uint4(0, 0, 0, 0);
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) most = max(most, max(w[j] << 16 & 0x7FFF0000u, w[j] & 0x7FFF0000u));
  }
  atomicMax(&s_most, most);
  __syncthreads();
  const Scale8 s = scale_e4m3(__uint_as_float(s_most));
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (n0 + 16 * i < N && k < K) {
      uint2 o;
      o.x = pack_e4m3x4(bf_lo(v[i].x) * s.up, bf_hi(v[i].x) * s.up, bf_lo(v[i].y) * s.up, bf_hi(v[i].y) * s.up);
      o.y = pack_e4m3x4(bf_lo(v[i].z) * s.up, bf_hi(v[i].z) * s.up, bf_lo(v[i].w) * s.up, bf_hi(v[i].w) * s.up);
      *reinterpret_cast<uint2*>(q + (n0 + 16 * i) * K + k) = o;
    }
  if (t == 0) scales[(long long)blockIdx.x * gridDim.y + blockIdx.y] = s.scale;
}

cudaError_t launch_norm_quant(dec_handle* h, const QuantRows& P, int M, cudaStream_t s) {
  const int n = (P.H / 8 + 255) / 256;
  const dim3 g(M), b(256);
  if (n <= 1) return launch_k(h, norm_quant_kernel<1>, g, b, 0, s, P);
  if (n <= 2) return launch_k(h, norm_quant_kernel<2>, g, b, 0, s, P);
  if (n <= 4) return launch_k(h, norm_quant_kernel<4>, g, b, 0, s, P);
  if (n <= 8) return launch_k(h, norm_quant_kernel<8>, g, b, 0, s, P);
  if (n <= 16) return launch_k(h, norm_quant_kernel<16>, g, b, 0, s, P);
  return launch_k(h, norm_quant_kernel<32>, g, b, 0, s, P);
}

cudaError_t launch_weight_quant(dec_handle* h, const uint16_t* W, long long N, int K, uint8_t* q, float* scales,
                                cudaStream_t s) {
  return launch_k(h, weight_quant_kernel, dim3((unsigned)((N + 127) / 128), (K + 127) / 128), dim3(256), 0, s, W, N, K,
                  q, scales);
}

}  // namespace dec
