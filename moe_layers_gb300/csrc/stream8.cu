// Products of 8-bit weights with a few 8-bit rows: projections of up to 16 rows
// and the experts.
//
//   y[t][n] = sum_b sx[t][b] sw[n / 128][b] sum_{k in b} xq[t][k] wq[n][k]
//
// over blocks b of 128 values. Every weight byte is used for a few rows only, so
// the kernel is a stream of weights past the tensor cores. The products are
// mma.sync's (16 weight rows x 8 activation rows x 32 values; measured 1.3 clocks
// a warp instruction and SM, 30 times what the stream needs at 8 rows), because
// their operands come straight from registers: a lane's 16-byte load of a weight
// row holds the words that it feeds for two products if both operands take the
// row's 64 bytes in the same permuted order, and a sum does not mind its order.
// So weights pass from memory to the products with no shared memory between, as
// deep in flight as registers allow (tcgen05's operands would have to be staged,
// and its accumulators fetched again for each block of 128, which has a scale of
// its own). The fp32 sum of a block is scaled and added to the total right away.
//
// Work: a problem is R weight rows for up to 8 NT activation rows; problems' rows
// form one sequence, cut into one equal range per CTA (one CTA per SM), so that
// every SM streams the same bytes. Inside a CTA a segment (the rows of its range
// that belong to one problem) is a sequence of units of 16 rows x 128 bytes, cut
// once more into one equal range per warp; a warp that holds all blocks of 16
// rows writes them out, the pieces of rows that several warps share are added in
// block order after the segment's one barrier. No atomics: the results follow
// from the inputs and the shape alone.
#include <algorithm>

#include "common.cuh"
#include "fp8.cuh"
#include "internal.h"

namespace dec {

namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxSmem = 232448;

}  // namespace

struct Stream8Params {
  const uint8_t* x;  // activation rows
  long long ldx;
  const float* xs;   // their scales
  long long ldxs;
  Stream8Bank bank, shared;  // the routed (or only) weights, and the shared expert's
  const int* table;          // problems (grouped), see Experts8Table
  int slots, P_max;
  bool by_token;  // activation rows by the slot's token, else by the slot
  int R, K, KB, rows;
  const uint16_t* res;
  long long ldr;
  void* out;
  long long ldo;
};

// Weights in flight ahead of the products, in units a warp.
template <bool PAIR>
constexpr int kDepth = PAIR ? 2 : 4;

__host__ __device__ constexpr int row_pitch(int K) { return (K + 127) / 128 * 128 + 64; }  // 16-byte reads of 2 rows x 64 bytes: no bank twice

template <int NT, bool PAIR>
static size_t smem_bytes(int K) {
  const size_t KB = (K + 127) / 128;
  return 8 * NT * (size_t)row_pitch(K) + KB * 8 * NT * 4 + (size_t)2 * kWarps * (PAIR ? 2 : 1) * 4 * NT * 32 * 4;
}

template <bool PAIR>
struct Unit {
  uint4 a[PAIR ? 2 : 1][2][2];  // [matrix][row g, g + 8][64-byte half]
  float s[PAIR ? 2 : 1][2];     // weight scale of the row's block
};

template <int NT, bool PAIR, bool GROUPED>
__global__ void __launch_bounds__(kThreads, 1) stream8_kernel(const Stream8Params P) {
  constexpr int NA = PAIR ? 2 : 1;
  constexpr int D = kDepth<PAIR>;
  constexpr int COLS = 8 * NT;
  extern __shared__ __align__(16) uint8_t sm[];
  const int KB = P.KB, pitch = row_pitch(P.K);
  uint8_t* xq = sm;                                                              // [COLS][pitch]
  float* xsc = reinterpret_cast<float*>(sm + (size_t)COLS * pitch);              // [KB][COLS]
  float* red = xsc + (size_t)KB * COLS;                                          // [2 kWarps][NA * 4 * NT][32]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint64_t pol = policy_evict_first();
  pdl_trigger();

  long long problems = 1;
  if (GROUPED) {
    pdl_wait();
    problems = ld_act_s32(P.table);
  }
  const long long total = problems * P.R, G = gridDim.x, c = blockIdx.x;
  const long long q0 = c * total / G, q1 = (c + 1) * total / G;
  bool waited = GROUPED;

  for (long long q = q0; q < q1;) {
    const int p = (int)(q / P.R), ra = (int)(q % P.R), rb = (int)min((long long)P.R, ra + (q1 - q));
    q += rb - ra;
    Stream8Bank B = P.bank;
    int cnt = P.rows;
    long long slot0 = 0;
    if (GROUPED) {
      const int e = ld_act_s32(P.table + 1 + 3 * p);
      slot0 = ld_act_s32(P.table + 2 + 3 * p);
      cnt = ld_act_s32(P.table + 3 + 3 * p);
      if (e < 0) {
        B = P.shared;
      } else {
        const size_t w = (size_t)e * P.R * P.K, s = (size_t)e * ((P.R + 127) / 128) * KB;
        for (int a = 0; a < NA; ++a) B.W[a] += w, B.scales[a] += s;
      }
    }
    const int groups = (rb - ra + 15) >> 4, U = groups * KB;
    const int u0 = (int)((long long)warp * U / kWarps), u1 = (int)((long long)(warp + 1) * U / kWarps);

    // The next unit to load: group lg, block lk.
    int lg = u0 / KB, lk = u0 % KB;
    Unit<PAIR> w[D];
    auto load = [&](Unit<PAIR>& v) {
      const int k = lk * 128 + t * 16;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = ra + lg * 16 + g + 8 * i;
#pragma unroll
        for (int a = 0; a < NA; ++a) {
          const uint8_t* src = B.W[a] + (size_t)r * P.K + k;
#pragma unroll
          for (int half = 0; half < 2; ++half)
            v.a[a][i][half] = r < rb && k + 64 * half < P.K ? ld_stream(src + 64 * half, pol) : make_uint4(0, 0, 0, 0);
          v.s[a][i] = r < rb ? __ldg(B.scales[a] + (size_t)(r >> 7) * KB + lk) : 0.f;
        }
      }
      if (++lk == KB) lk = 0, ++lg;
    };
#pragma unroll
    for (int d = 0; d < D; ++d)
      if (u0 + d < u1) load(w[d]);

    // This problem's activation rows: values zero up to a whole block.
    if (!waited) pdl_wait();
    waited = true;
    __syncthreads();  // the previous segment is done with them
    const int chunks = (pitch - 64) >> 4;
    for (int i = threadIdx.x; i < cnt * chunks; i += kThreads) {
      const int j = i / chunks, k = (i - j * chunks) * 16;
      long long row = slot0 + j;
      if (GROUPED && P.by_token) row = ld_act_s32(P.table + 1 + 3 * P.P_max + slot0 + j);
      *reinterpret_cast<uint4*>(xq + (size_t)j * pitch + k) =
          k < P.K ? ld_act16(P.x + row * P.ldx + k) : make_uint4(0, 0, 0, 0);
    }
    for (int i = threadIdx.x; i < KB * COLS; i += kThreads) {
      const int b = i / COLS, j = i % COLS;
      float v = 0.f;
      if (j < cnt) {
        long long row = slot0 + j;
        if (GROUPED && P.by_token) row = ld_act_s32(P.table + 1 + 3 * P.P_max + slot0 + j);
        v = ld_act_f32(P.xs + row * P.ldxs + b);
      }
      xsc[i] = v;
    }
    __syncthreads();

    float tot[NA][NT][4];
    auto clear = [&]() {
#pragma unroll
      for (int a = 0; a < NA; ++a)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) tot[a][nt][i] = 0.f;
    };
    clear();

    // Sixteen finished rows: this lane's rows g and g + 8, columns 2 t and 2 t + 1 of each eight.
    auto emit = [&](int gi) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = ra + gi * 16 + g + 8 * (i >> 1), j = nt * 8 + 2 * t + (i & 1);
          if (r >= rb || j >= cnt) continue;
          if (PAIR) {
            const float z = tot[0][nt][i];
            static_cast<float*>(P.out)[(slot0 + j) * P.ldo + r] = z / (1.0f + expf(-z)) * tot[NA - 1][nt][i];
          } else if (GROUPED) {
            static_cast<float*>(P.out)[(slot0 + j) * P.ldo + r] = tot[0][nt][i];
          } else {
            float v = tot[0][nt][i];
            if (P.res != nullptr) v += bf2f(ld_act_u16(P.res + j * P.ldr + r));
            static_cast<uint16_t*>(P.out)[j * P.ldo + r] = f2bf(v);
          }
        }
    };

    int gi = u0 / KB, kb = u0 % KB;
    const int first = gi;
    auto compute = [&](const Unit<PAIR>& v, int u) {
      const uint8_t* xk = xq + (size_t)g * pitch + kb * 128 + t * 16;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint4 b0 = *reinterpret_cast<const uint4*>(xk + (size_t)nt * 8 * pitch);
        const uint4 b1 = *reinterpret_cast<const uint4*>(xk + (size_t)nt * 8 * pitch + 64);
        const float2 sx = *reinterpret_cast<const float2*>(xsc + (size_t)kb * COLS + nt * 8 + 2 * t);
#pragma unroll
        for (int a = 0; a < NA; ++a) {
          float acc[4] = {0.f, 0.f, 0.f, 0.f};
          const uint4 l0 = v.a[a][0][0], l1 = v.a[a][0][1], h0 = v.a[a][1][0], h1 = v.a[a][1][1];
          mma_e4m3(acc, l0.x, h0.x, l0.y, h0.y, b0.x, b0.y);
          mma_e4m3(acc, l0.z, h0.z, l0.w, h0.w, b0.z, b0.w);
          mma_e4m3(acc, l1.x, h1.x, l1.y, h1.y, b1.x, b1.y);
          mma_e4m3(acc, l1.z, h1.z, l1.w, h1.w, b1.z, b1.w);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            tot[a][nt][i] = fmaf(acc[i], v.s[a][i >> 1] * ((i & 1) ? sx.y : sx.x), tot[a][nt][i]);
        }
      }
      if (++kb == KB || u + 1 == u1) {
        if (gi * KB >= u0 && (gi + 1) * KB <= u1) {
          emit(gi);
        } else {
          float* slot = red + (size_t)(2 * warp + (gi == first ? 0 : 1)) * (NA * 4 * NT) * 32 + lane;
#pragma unroll
          for (int a = 0; a < NA; ++a)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) slot[((a * NT + nt) * 4 + i) * 32] = tot[a][nt][i];
        }
        clear();
        kb = 0;
        ++gi;
      }
    };
    for (int u = u0; u < u1; u += D) {
#pragma unroll
      for (int d = 0; d < D; ++d)
        if (u + d < u1) {
          compute(w[d], u + d);
          if (u + d + D < u1) load(w[d]);
        }
    }
    __syncthreads();
    // Rows whose blocks several warps hold: a warp adds their pieces in block order.
    for (int s = warp; s < groups; s += kWarps) {
      const int wa = (int)((((long long)s * KB + 1) * kWarps - 1) / U);
      const int wb = (int)((((long long)(s + 1) * KB) * kWarps - 1) / U);
      if (wa == wb) continue;
      clear();
      for (int v = wa; v <= wb; ++v) {
        const int a0 = (int)((long long)v * U / kWarps), a1 = (int)((long long)(v + 1) * U / kWarps);
        if (a0 == a1) continue;
        const float* slot = red + (size_t)(2 * v + (a0 / KB == s ? 0 : 1)) * (NA * 4 * NT) * 32 + lane;
#pragma unroll
        for (int a = 0; a < NA; ++a)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) tot[a][nt][i] += slot[((a * NT + nt) * 4 + i) * 32];
      }
      emit(s);
    }
  }
}

// ---------------------------------------------------------------- experts: problems and their sums
// The problems of a batch's experts, by one CTA of 1024 threads: entries (token t,
// choice j) are counted by expert, an expert's entries get consecutive slots, and
// its problems are runs of up to `most` of them; the shared expert's slots, one a
// token, follow. An entry whose id is outside [0, E) gets no slot. The place of an
// entry among its expert's follows the order of atomics; a slot's values do not
// depend on its place.
//   table: [0] problems; 3 words each: expert (-1: shared), first slot, rows;
//   at 1 + 3 P_max the slots' tokens; then the entries' slots.
__global__ void __launch_bounds__(1024) experts8_table_kernel(const int32_t* idx, int M, int k, int E, bool shared,
                                                              int most, int P_max, int* table) {
  __shared__ int count[1024], slot[1024], prob[1024], part[2][32];
  const int i = threadIdx.x, lane = i & 31, warp = i >> 5, n = M * k;
  count[i] = 0;
  pdl_trigger();
  pdl_wait();
  __syncthreads();
  const int e = i < n ? ld_act_s32(idx + i) : -1;
  const bool in = e >= 0 && e < E;
  const int rank = in ? atomicAdd(&count[e], 1) : 0;
  __syncthreads();
  // running sums over the experts of slots and problems
  const int mine = count[i], probs = (mine + most - 1) / most;
  int a = mine, b = probs;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int ua = __shfl_up_sync(0xffffffffu, a, o), ub = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) a += ua, b += ub;
  }
  if (lane == 31) part[0][warp] = a, part[1][warp] = b;
  __syncthreads();
  int sa = 0, sb = 0, ta = 0, tb = 0;
  for (int w = 0; w < 32; ++w) {
    if (w == warp) sa = ta, sb = tb;
    ta += part[0][w];
    tb += part[1][w];
  }
  slot[i] = sa + a - mine;
  prob[i] = sb + b - probs;
  for (int j = 0; j < probs; ++j) {
    int* q = table + 1 + 3 * (prob[i] + j);
    q[0] = i;
    q[1] = slot[i] + j * most;
    q[2] = min(most, mine - j * most);
  }
  __syncthreads();
  int* token = table + 1 + 3 * P_max;
  int* entry = token + n + M;
  if (i < n) {
    entry[i] = in ? slot[e] + rank : -1;
    if (in) token[slot[e] + rank] = i / k;
  }
  const int more = shared ? (M + most - 1) / most : 0;
  if (i < more) {
    int* q = table + 1 + 3 * (tb + i);
    q[0] = -1;
    q[1] = n + i * most;
    q[2] = min(most, M - i * most);
  }
  if (i < M) token[n + i] = i;
  if (i == 0) table[0] = tb + more;
}

// out[t] = bf16(sum_j w[t][j] y[slot(t, j)] (+ y[shared slot of t]) (+ res[t])), fp32 sums in that order.
__global__ void __launch_bounds__(256) experts8_combine_kernel(const float* y, const int* entry, const float* w, int M,
                                                               int k, bool shared, const uint16_t* res, uint16_t* out,
                                                               int H) {
  const int t = blockIdx.y, c = (blockIdx.x * 256 + threadIdx.x) * 4;
  pdl_trigger();
  pdl_wait();
  if (c >= H) return;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j = 0; j < k; ++j) {
    const int slot = ld_act_s32(entry + t * k + j);
    if (slot < 0) continue;
    const float wj = ld_act_f32(w + t * k + j);
    const float4 v = ld_act_f4(y + (size_t)slot * H + c);
    a.x = fmaf(wj, v.x, a.x), a.y = fmaf(wj, v.y, a.y), a.z = fmaf(wj, v.z, a.z), a.w = fmaf(wj, v.w, a.w);
  }
  if (shared) {
    const float4 v = ld_act_f4(y + (size_t)(M * k + t) * H + c);
    a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
  }
  if (res != nullptr) {
    const uint2 r = ld_act8(res + (size_t)t * H + c);
    a.x += bf_lo(r.x), a.y += bf_hi(r.x), a.z += bf_lo(r.y), a.w += bf_hi(r.y);
  }
  *reinterpret_cast<uint2*>(out + (size_t)t * H + c) = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
}

// ---------------------------------------------------------------- host side
template <int NT, bool PAIR, bool GROUPED>
static cudaError_t launch_one(dec_handle* h, const Stream8Params& P, int grid, cudaStream_t s) {
  const size_t smem = smem_bytes<NT, PAIR>(P.K);
  static bool attr_set = false;  // per process; every device gets the same attribute
  if (!attr_set) {
    const cudaError_t e = cudaFuncSetAttribute(stream8_kernel<NT, PAIR, GROUPED>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e != cudaSuccess) return e;
    attr_set = true;
  }
  return launch_k(h, stream8_kernel<NT, PAIR, GROUPED>, dim3(grid), dim3(kThreads), smem, s, P);
}

int stream8_rows(int K, bool pair) {
  if (pair) return smem_bytes<2, true>(K) <= kMaxSmem ? 16 : smem_bytes<1, true>(K) <= kMaxSmem ? 8 : 0;
  return smem_bytes<2, false>(K) <= kMaxSmem ? 16 : smem_bytes<1, false>(K) <= kMaxSmem ? 8 : 0;
}

cudaError_t launch_stream8_linear(dec_handle* h, const Linear8& L, cudaStream_t s) {
  Stream8Params P = {};
  P.x = L.x;
  P.ldx = L.ldx;
  P.xs = L.xs;
  P.ldxs = L.ldxs;
  P.bank.W[0] = L.W;
  P.bank.scales[0] = L.ws;
  P.R = L.N;
  P.K = L.K;
  P.KB = (L.K + 127) / 128;
  P.rows = L.M;
  P.res = L.res;
  P.ldr = L.ldr;
  P.out = L.y;
  P.ldo = L.ldy;
  const int grid = std::min(h->sms, L.N);
  return L.M <= 8 ? launch_one<1, false, false>(h, P, grid, s) : launch_one<2, false, false>(h, P, grid, s);
}

Experts8Plan experts8_plan(int M, int k, int E, int H, int I, bool shared) {
  Experts8Plan p;
  p.most = std::min(std::min(stream8_rows(H, true), stream8_rows(I, false)), M * k <= 8 ? 8 : 16);
  p.slots = M * k + M;
  const int most = std::max(p.most, 1);
  p.P_max = std::min(M * k, E + M * k / most) + (shared ? (M + most - 1) / most : 0);
  p.words = 1 + 3 * p.P_max + p.slots + M * k;
  return p;
}

cudaError_t launch_experts8(dec_handle* h, const Experts8& X, const Experts8Plan& plan, int* table, float* inner,
                            uint8_t* hq, float* hs, float* y, cudaStream_t s) {
  const int M = X.M, k = X.k, H = X.H, I = X.I;
  const bool shared = X.sgate.W[0] != nullptr;
  cudaError_t e;
  {
    LaunchScope scope(h, "experts8_table", s);
    e = launch_k(h, experts8_table_kernel, dim3(1), dim3(1024), 0, s, X.idx, M, k, X.E, shared, plan.most, plan.P_max,
                 table);
    if (e != cudaSuccess) return e;
  }
  Stream8Params P = {};
  P.x = X.x;
  P.ldx = X.ldx;
  P.xs = X.xs;
  P.ldxs = X.ldxs;
  P.bank = X.gate;
  P.shared = X.sgate;
  P.table = table;
  P.slots = plan.slots;
  P.P_max = plan.P_max;
  P.by_token = true;
  P.R = I;
  P.K = H;
  P.KB = H / 128;
  P.out = inner;
  P.ldo = I;
  {
    LaunchScope scope(h, "experts8_gate_up", s);
    e = plan.most <= 8 ? launch_one<1, true, true>(h, P, h->sms, s) : launch_one<2, true, true>(h, P, h->sms, s);
    if (e != cudaSuccess) return e;
  }
  {
    QuantRows Q = {};
    Q.x = inner;
    Q.ldx = I;
    Q.q = hq;
    Q.ldq = I;
    Q.scales = hs;
    Q.ldsc = I / 128;
    Q.H = I;
    LaunchScope scope(h, "experts8_quant", s);
    e = launch_norm_quant(h, Q, shared ? plan.slots : M * k, true, s);
    if (e != cudaSuccess) return e;
  }
  P.x = hq;
  P.ldx = I;
  P.xs = hs;
  P.ldxs = I / 128;
  P.bank = X.down;
  P.shared = X.sdown;
  P.by_token = false;
  P.R = H;
  P.K = I;
  P.KB = I / 128;
  P.out = y;
  P.ldo = H;
  {
    LaunchScope scope(h, "experts8_down", s);
    e = plan.most <= 8 ? launch_one<1, false, true>(h, P, h->sms, s) : launch_one<2, false, true>(h, P, h->sms, s);
    if (e != cudaSuccess) return e;
  }
  LaunchScope scope(h, "experts8_combine", s);
  return launch_k(h, experts8_combine_kernel, dim3((H / 4 + 255) / 256, M), dim3(256), 0, s, (const float*)y,
                  (const int*)(table + 1 + 3 * plan.P_max + plan.slots), X.w, M, k, shared, X.res, X.out, H);
}

}  // namespace dec
