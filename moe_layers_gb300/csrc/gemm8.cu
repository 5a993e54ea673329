// Products of 8-bit weights with many 8-bit rows, on tcgen05: decode batches above
// what the streaming kernel takes, and prompts.
//
//   y[t][n] = [r[t][n] +] sum_b sx[t][b] sw[n / 128][b] sum_{k in b} xq[t][k] wq[n][k]
//
// A tile is 128 rows x BN weights. Its k-blocks of 128 values have scales of their own,
// so the tensor cores' sum of a block is not kept: each block goes to a tensor-memory
// buffer of its own, is fetched by eight warps, scaled and added to totals in registers,
// while the next blocks are multiplied. Rows are the product's M side, so a thread owns
// one row and BN / 2 columns of one block of weights: its scale is one number a k-block,
// and a fetched value costs half a packed fused multiply-add.
//
// One CTA per SM. Whole tiles go round the CTAs as long as there is one for each, in panels
// of 16 tiles of rows, so that the tiles in work at a time share rows and weights in L2. A
// tile that is left over (any, for a decode batch) may be shared by two to four CTAs, a run of
// k-blocks each. Without whole rounds they are a cluster, and each finishes its part of the
// columns from the pieces that the others put into its shared memory; else the one that
// publishes its piece last adds all of them. Either way in k order, without atomics on values:
// the results follow from the inputs and the shape alone.
//
// Measured, in a replayed graph: 12288 x 7168 at 4096 rows 392 us (1.84 PFLOP/s), 64 rows 22.2
// us (0.61 of the copy rate), 64 x 4096 x 4096 9.7 us. Bound, at many rows, by the adding warps: a
// k-block of 128 x 256 is multiplied in some 540 clocks (the same without them) and takes 1170; at
// few rows by the 600 clocks a k-block that pass between product, fetch and next product.
//
// Per CTA: warp 0 issues the TMA loads of a k-block's rows and weights (128-byte
// swizzle) into a ring in shared memory, warp 1 the tcgen05.mma (128 x BN x 32, kind
// f8f6f4), warps 4-11 fetch, scale and add.
#include <algorithm>

#include "common.cuh"
#include "fp8.cuh"
#include "internal.h"

namespace dec {

namespace {

constexpr int kRows = 128;
constexpr int kBlock = 128;  // k values of a block, one row of the swizzle
constexpr int kAdders = 256;
constexpr int kThreads = 128 + kAdders;
constexpr int kTmem = 512;

template <int BN>
struct Plan {
  static constexpr int kABytes = kRows * kBlock;
  static constexpr int kStageBytes = kABytes + BN * kBlock;
  static constexpr int kStages = 221184 / kStageBytes;
  static constexpr int kBuffers = kTmem / BN < 8 ? kTmem / BN : 8;
  static constexpr int kCols = BN / 2;                            // a thread's
  static constexpr int kFetch = kCols % 32 == 0 ? 32 : 16;        // columns of one instruction
  // Columns fetched before any is added. (More at once would take registers that are not there:
  // 64 of 128 columns spill, and 4096 rows take 506 us instead of 398.)
  static constexpr int kAtOnce = kCols <= 48 ? kCols : 32;
  static_assert(kCols % kAtOnce == 0 && kAtOnce % kFetch == 0, "whole instructions");
  static constexpr bool kStraddle = 128 % kCols != 0;             // they may lie in two blocks of weights
  static constexpr int kBarOff = kStages * kStageBytes;
  static constexpr int kScaleOff = kBarOff + (8 * (2 * kStages + 2 * kBuffers + 1) + 16 + 63) / 64 * 64;
  static constexpr int kBytes = kScaleOff + 2 * 8 * kRows * 4 + 1024;
  static_assert(kBytes <= 232448, "shared memory above the opt-in maximum");
};

struct Gemm8Params {
  int M, N, K, KB, mtiles, ntiles;
  int split;     // CTAs that share a tile of those left after whole rounds
  int cluster;   // they are a cluster (no whole rounds then): pieces go through its shared memory
  int box_rows;  // rows of a copy: a tile's, or the whole batch's up to eight
  const float* xs;
  long long ldxs;
  const float* ws;
  const uint16_t* res;
  long long ldr;
  uint16_t* y;
  long long ldy;
  float* pieces;
  int piece_rows;  // rows of a published piece: the tile's, or the batch's up to a warp's
  int* counters;   // one for each shared tile: pieces published
  int* err;
  unsigned long long wait_ns;
  int give_up;  // a test's: CTAs of a multiple of this index give up at once
};

constexpr int kPanel = 16;  // tiles of rows

// Instruction descriptor, kind::f8f6f4: D fp32, A and B e4m3, both K-major, 128 x N.
constexpr uint32_t idesc_e4m3(int N) { return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24); }

__device__ __forceinline__ void umma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Consecutive fp32 columns of this thread's tensor-memory lane, there after tmem_wait
// and, so that no use of them is moved before it, tmem_here.
__device__ __forceinline__ void tmem_fetch(uint32_t at, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void tmem_fetch(uint32_t at, uint32_t (&r)[32]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_here(uint32_t (&r)[16]) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}
__device__ __forceinline__ void tmem_here(uint32_t (&r)[32]) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}

// Another CTA's shared memory of the cluster, and the barrier of all its threads.
__device__ __forceinline__ uint32_t peer_at(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void peer_store(uint32_t at, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// Moves registers between the warps that copy and multiply, which need few, and those that add.
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

// acc + v * f for two values, fp32.
__device__ __forceinline__ uint64_t fma2(uint32_t lo, uint32_t hi, uint64_t f, uint64_t acc) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(v), "l"(f));
  return acc;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  uint32_t lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
  return make_float2(__uint_as_float(lo), __uint_as_float(hi));
}
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(__float_as_uint(lo)), "r"(__float_as_uint(hi)));
  return v;
}

}  // namespace

// The work of a CTA: `rounds` whole tiles, then, of what is left, a part of a tile.
struct Work {
  int KB, mtiles, ntiles, split, rounds, left;
  int r = 0;
  int tile, kb0, kb1;  // the current part: k-blocks [kb0, kb1) of a tile
  __device__ Work(const Gemm8Params& P) : KB(P.KB), mtiles(P.mtiles), ntiles(P.ntiles), split(P.split) {
    const int tiles = P.mtiles * P.ntiles;
    rounds = tiles / (int)gridDim.x;
    left = tiles - rounds * (int)gridDim.x;
  }
  __device__ bool next() {
    const int c = blockIdx.x;
    if (r < rounds) {
      tile = r++ * (int)gridDim.x + c;
      kb0 = 0;
      kb1 = KB;
      return true;
    }
    if (r++ > rounds || c >= left * split) return false;
    const int t = c / split, part = c - t * split;
    tile = rounds * (int)gridDim.x + t;
    kb0 = part * KB / split;
    kb1 = (part + 1) * KB / split;
    return true;
  }
  __device__ void place(int& mt, int& nt) const {
    const int whole = kPanel * ntiles, panel = tile / whole, in = tile - panel * whole;
    const int height = min(kPanel, mtiles - panel * kPanel);
    nt = in / height;
    mt = panel * kPanel + in - nt * height;
  }
};

template <int BN>
__global__ void __launch_bounds__(kThreads, 1)
    gemm8_kernel(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap tw, const Gemm8Params P) {
  using L = Plan<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint64_t* empty = full + L::kStages;
  uint64_t* tfull = empty + L::kStages;
  uint64_t* tempty = tfull + L::kBuffers;
  uint64_t* done = tempty + L::kBuffers;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* s_last = abort_flag + 1;
  float* s_scales = reinterpret_cast<float*>(smem + L::kScaleOff);  // [2][8][kRows]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < L::kBuffers; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], kAdders / 32);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tmap_prefetch(&tx);
    tmap_prefetch(&tw);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot), smem_at = smem_u32(smem);
  const WaitCtl wc{abort_flag, P.err, P.wait_ns}, drain{nullptr, P.err, P.wait_ns};

  // 384 threads start with 168 registers each; 256 x 208 + 128 x 80 are fewer.
  if (warp < 4) regs_down<80>();
  if (warp == 0) {
    // ------------------------------------------------------------ copies
    const uint64_t pol_w = P.mtiles == 1 ? policy_evict_first() : policy_evict_last();  // read once, or again
    const uint64_t pol_x = policy_evict_last();
    const uint32_t tx_bytes = (uint32_t)((P.box_rows + BN) * kBlock);
    // Static weights of the first ring's worth before the dependency wait.
    int pre = 0, mt, nt;
    for (Work work(P); pre < L::kStages && work.next();) {
      work.place(mt, nt);
      for (int kb = work.kb0; kb < work.kb1 && pre < L::kStages; ++kb, ++pre) {
        const int su = uniform(pre), k = uniform(kb * kBlock), row = uniform(nt * BN);
        if (elect_one()) {
          mbar_arrive_expect_tx(&full[su], tx_bytes);
          tma_load_2d(smem + su * L::kStageBytes + L::kABytes, &tw, &full[su], k, row, pol_w);
        }
      }
    }
    pdl_wait();
    int s = 0, issued = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (Work work(P); ok && work.next();) {
      work.place(mt, nt);
      const int row_w = uniform(nt * BN), row_x = uniform(mt * kRows);
      for (int kb = work.kb0; kb < work.kb1; ++kb) {
        const int su = uniform(s), k = uniform(kb * kBlock);
        if (pre > 0) {
          --pre;
        } else {
          if (!__all_sync(0xffffffffu, mbar_wait_soon(&empty[su], ph ^ 1u, wc))) {
            ok = false;
            break;
          }
          if (elect_one()) {
            mbar_arrive_expect_tx(&full[su], tx_bytes);
            tma_load_2d(smem + su * L::kStageBytes + L::kABytes, &tw, &full[su], k, row_w, pol_w);
          }
        }
        if (elect_one()) tma_load_2d(smem + su * L::kStageBytes, &tx, &full[su], k, row_x, pol_x);
        __syncwarp();
        if (++s == L::kStages) s = 0, ph ^= 1u;
        issued = min(issued + 1, L::kStages);
      }
    }
    // No copy may still be in flight when the CTA exits.
    for (; issued > 0; --issued) {
      if (--s < 0) s = L::kStages - 1, ph ^= 1u;
      mbar_wait_soon(&full[s], ph, drain);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    pdl_wait();  // the time of the kernel ahead is not a wait's
    int s = 0, b = 0;
    uint32_t ph = 0, tph = 0;
    bool ok = true;
    for (Work work(P); ok && work.next();)
      for (int kb = work.kb0; kb < work.kb1; ++kb) {
        const int su = uniform(s), bu = uniform(b);
        if (!__all_sync(0xffffffffu, mbar_wait_soon(&tempty[bu], tph ^ 1u, wc) && mbar_wait_soon(&full[su], ph, wc))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(bu * BN);
        const uint64_t a = sw128_desc(smem_at + su * L::kStageBytes), w = sw128_desc(smem_at + su * L::kStageBytes + L::kABytes);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kBlock / 32; ++k) umma_e4m3(d, a + 2 * k, w + 2 * k, idesc_e4m3(BN), k > 0);
          umma_commit(&tfull[bu]);
          umma_commit(&empty[su]);
        }
        __syncwarp();
        if (++s == L::kStages) s = 0, ph ^= 1u;
        if (++b == L::kBuffers) b = 0, tph ^= 1u;
      }
    // Every product issued above must complete before tensor memory is released.
    if (elect_one()) umma_commit(done);
    __syncwarp();
    mbar_wait_soon(done, 0, drain);
  } else if (warp >= 4) {
    // ------------------------------------------------------------ sums
    regs_up<208>();
    int syncs = P.cluster ? 2 : 0;  // barriers of the cluster that are still to come
    const int q = warp & 3, row = q * 32 + lane;  // tensor-memory lanes 32 q ..
    const int half = (warp - 4) >> 2, col0 = half * L::kCols;
    const int et = threadIdx.x - 128;
    const bool out_vec = (reinterpret_cast<uintptr_t>(P.y) & 15) == 0 && (P.ldy & 7) == 0;
    const bool res_vec = (reinterpret_cast<uintptr_t>(P.res) & 15) == 0 && (P.ldr & 7) == 0;
    pdl_wait();
    int b = 0, turn = 0;
    uint32_t tph = 0;
    bool ok = P.give_up == 0 || (int)blockIdx.x % P.give_up != 0;
    if (!ok && et == 0) {
      *abort_flag = 1;
      atomicOr(P.err, DEV_ERR_TIMEOUT);
    }
    const int KB = P.KB;
    for (Work work(P); work.next();) {
      const int kb0 = work.kb0, kb1 = work.kb1;
      int mt, nt;
      work.place(mt, nt);
      const int m0 = mt * kRows, n0 = nt * BN;
      const bool rows_here = m0 + q * 32 < P.M;  // this warp's rows hold some of the batch's
      const float* xs = P.xs + (long long)min(m0 + row, P.M - 1) * P.ldxs;
      const int block0 = (n0 + col0) >> 7;                      // the columns' first block of weights
      const int edge = ((block0 + 1) << 7) - (n0 + col0);       // columns in it
      const float* ws = P.ws + (long long)min(block0 + (L::kStraddle ? (lane >> 3) & 1 : 0), (P.N - 1) >> 7) * KB;
      uint64_t acc[L::kCols / 2];
#pragma unroll
      for (int i = 0; i < L::kCols / 2; ++i) acc[i] = 0;
      // Scales of eight blocks at a time, the next eight's loads in flight. The rows' lie far
      // apart, so each of the two warps that share rows loads four blocks' and leaves them
      // for both; the weights' (of the warp's columns) are spread over lanes 0-7, those of
      // a second block over 8-15.
      // (No load is conditional: the branch around it would wait for it.)
      float nx[4], sw, nw;
      auto load_scales = [&](int kb) {
#pragma unroll
        for (int i = 0; i < 4; ++i) nx[i] = ld_act_f32(xs + min(kb + 4 * half + i, KB - 1));
        nw = ld_act_f32(ws + min(kb + (lane & 7), KB - 1));
      };
      if (rows_here) load_scales(kb0);
      // a warp that gave up a wait goes on without waiting, through the same barriers as the others
      for (int kb = kb0; kb < kb1; kb += 8) {
        float* sx = s_scales + ((turn++ & 1) * 8) * kRows + row;
        if (rows_here) {
#pragma unroll
          for (int i = 0; i < 4; ++i) sx[(4 * half + i) * kRows] = nx[i];
          sw = nw;
          load_scales(kb + 8);
          named_bar_sync(2 + q, 64);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (kb + i >= kb1) break;
          uint64_t f0, f1;
          if (rows_here) {
            const float x = sx[i * kRows];
            const float a = x * __shfl_sync(0xffffffffu, sw, i);
            const float c = L::kStraddle ? x * __shfl_sync(0xffffffffu, sw, 8 + i) : a;
            f0 = pack2(a, a);
            f1 = pack2(c, c);
          }
          ok = ok && __all_sync(0xffffffffu, mbar_wait_soon(&tfull[b], tph, wc));
          if (!ok) break;
          const int here = min(1, kb1 - kb - i);  // 1
          if (rows_here) {
            tc_fence_after();
            const uint32_t at = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * BN + col0);
#pragma unroll
            for (int ch = 0; ch < L::kCols; ch += L::kAtOnce) {
              uint32_t v[L::kAtOnce / L::kFetch][L::kFetch];
#pragma unroll
              for (int p = 0; p < L::kAtOnce / L::kFetch; ++p) tmem_fetch(at + ch + p * L::kFetch, v[p]);
              tmem_wait();
#pragma unroll
              for (int p = 0; p < L::kAtOnce / L::kFetch; ++p) tmem_here(v[p]);
              if (ch + L::kAtOnce == L::kCols) {
                // all fetched: the buffer is free
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&tempty[b]);
              }
              // Always so: behind a branch the additions stay together, before the next fetch. Mixed with
              // it they spill registers, and 4096 rows take 475 us instead of 398.
              if (here > 0) {
#pragma unroll
                for (int p = 0; p < L::kAtOnce / L::kFetch; ++p)
#pragma unroll
                  for (int e = 0; e < L::kFetch / 2; ++e) {
                    const int pair = (ch + p * L::kFetch) / 2 + e;
                    acc[pair] = fma2(v[p][2 * e], v[p][2 * e + 1], L::kStraddle && pair / 4 * 8 >= edge ? f1 : f0, acc[pair]);
                  }
              }
            }
          } else if (lane == 0) {
            mbar_arrive(&tempty[b]);
          }
          if (++b == L::kBuffers) b = 0, tph ^= 1u;
        }
      }
      if (!named_bar_and(1, kAdders, ok)) {  // leave together if a warp gave up
        // This call's result is lost, and the error word says so. The CTA takes its turn at its shared tile's counter
        // all the same (a piece is its last work): the counters are zero after every call.
        if (!P.cluster && P.split > 1 && et == 0 && (int)blockIdx.x < work.left * P.split) {
          int* counter = P.counters + (int)blockIdx.x / P.split;
          if (atom_add_acq_rel_gpu(counter, 1) == P.split - 1) *counter = 0;
        }
        break;
      }

      int from = 0, to = L::kCols;  // this thread's columns that this CTA finishes
      if (P.cluster) {
        // Each CTA finishes an equal part of the columns: a thread's half of them, or (of four) a half of that. Its
        // ring, empty once all have multiplied their last block, receives a piece of it from every CTA.
        const int rank = (int)blockIdx.x % P.split, width = P.split == 2 ? L::kCols : L::kCols / 2;
        cluster_sync();
        --syncs;
        if (rows_here) {
#pragma unroll
          for (int i = 0; i < L::kCols / 4; ++i) {
            const int part = P.split == 4 && 4 * i >= L::kCols / 2 ? 1 : 0;
            const int owner = P.split == 2 ? half : 2 * half + part, in = 4 * i - part * width;
            const float2 lo = unpack2(acc[2 * i]), hi = unpack2(acc[2 * i + 1]);
            peer_store(peer_at(smem_at + (uint32_t)(((rank * width + in) / 4 * kRows + row) * 16), owner),
                       make_float4(lo.x, lo.y, hi.x, hi.y));
          }
        }
        cluster_sync();
        --syncs;
        if (rank * 2 / P.split != half) continue;  // the other half of the columns
        from = P.split == 2 ? 0 : (rank & 1) * width;
        to = from + width;
#pragma unroll
        for (int i = 0; i < L::kCols / 2; ++i) acc[i] = 0;
        if (rows_here)
          for (int r = 0; r < P.split; ++r) {  // in k order
            const float4* src = reinterpret_cast<const float4*>(smem) + (r * width - from) / 4 * kRows + row;
#pragma unroll
            for (int i = 0; i < L::kCols / 4; ++i)
              if (4 * i >= from && 4 * i < to) {
                const float4 v = src[i * kRows];
                const float2 lo = unpack2(acc[2 * i]), hi = unpack2(acc[2 * i + 1]);
                acc[2 * i] = pack2(lo.x + v.x, lo.y + v.y);
                acc[2 * i + 1] = pack2(hi.x + v.z, hi.y + v.w);
              }
          }
      } else if (kb1 - kb0 < KB) {
        // A piece: published, four columns of a row at a time; whoever publishes the last adds them all in k order.
        const int p_rows = P.piece_rows, shared = (int)blockIdx.x / P.split;
        auto piece = [&](int cc) {
          return reinterpret_cast<float4*>(P.pieces) + (size_t)cc * (BN / 4) * p_rows + (size_t)(col0 / 4) * p_rows + row;
        };
        if (rows_here) {
          float4* dst = piece((int)blockIdx.x);
#pragma unroll
          for (int i = 0; i < L::kCols / 4; ++i) {
            const float2 lo = unpack2(acc[2 * i]), hi = unpack2(acc[2 * i + 1]);
            __stcg(dst + (size_t)i * p_rows, make_float4(lo.x, lo.y, hi.x, hi.y));
          }
        }
        __threadfence();
        named_bar_sync(1, kAdders);
        if (et == 0) *s_last = atom_add_acq_rel_gpu(P.counters + shared, 1) == P.split - 1 ? 1 : 0;
        named_bar_sync(1, kAdders);
        const bool last = *s_last != 0;
        named_bar_sync(1, kAdders);  // read by all before the next piece
        if (!last) continue;
        __threadfence();
        if (et == 0) P.counters[shared] = 0;  // leave the workspace reusable
        if (rows_here) {
#pragma unroll
          for (int i = 0; i < L::kCols / 2; ++i) acc[i] = 0;
          for (int cc = shared * P.split; cc < (shared + 1) * P.split; ++cc) {
            const float4* src = piece(cc);
#pragma unroll
            for (int i = 0; i < L::kCols / 4; ++i) {
              const float4 v = __ldcg(src + (size_t)i * p_rows);
              const float2 lo = unpack2(acc[2 * i]), hi = unpack2(acc[2 * i + 1]);
              acc[2 * i] = pack2(lo.x + v.x, lo.y + v.y);
              acc[2 * i + 1] = pack2(hi.x + v.z, hi.y + v.w);
            }
          }
        }
      }
      // This thread's columns of its row.
      if (m0 + row < P.M) {
        const int n = n0 + col0;
        uint16_t* out = P.y + (long long)(m0 + row) * P.ldy + n;
        const uint16_t* res = P.res != nullptr ? P.res + (long long)(m0 + row) * P.ldr + n : nullptr;
#pragma unroll
        for (int i = 0; i < L::kCols / 8; ++i) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 d = unpack2(acc[4 * i + e]);
            v[2 * e] = d.x, v[2 * e + 1] = d.y;
          }
          const int left = P.N - n - 8 * i;  // columns from here on
          if (left <= 0) break;
          if (8 * i < from || 8 * i >= to) continue;
          if (res != nullptr) {
            if (res_vec && left >= 8) {
              const uint4 r = ld_act16(res + 8 * i);
              const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) v[2 * e] += bf_lo(w[e]), v[2 * e + 1] += bf_hi(w[e]);
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (e < left) v[e] += bf2f(ld_act_u16(res + 8 * i + e));
            }
          }
          if (out_vec && left >= 8) {
            *reinterpret_cast<uint4*>(out + 8 * i) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                                pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (e < left) out[8 * i + e] = f2bf(v[e]);
          }
        }
      }
    }
    for (; syncs > 0; --syncs) cluster_sync();
  }
  if (P.cluster && warp < 4) {
    cluster_sync();
    cluster_sync();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmem);
  }
}

// ---------------------------------------------------------------- host side
// How many clusters of 2 or 4 CTAs, one CTA to an SM, this device holds at a time: the parts of the chip have
// different numbers of SMs, and not the same ones on every chip. (None if the runtime does not say.)
static int clusters_held(const dec_handle* h, int size) {
  static std::atomic<int> held[16][5];  // by device; 0: not asked yet, -1: none
  if (h->device < 0 || h->device >= 16) return 0;
  int n = held[h->device][size].load();
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(size);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Plan<256>::kBytes;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    DeviceGuard dev(h->device);
    int got = 0;
    const bool ok = dev.ok &&
                    cudaFuncSetAttribute(gemm8_kernel<256>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Plan<256>::kBytes) == cudaSuccess &&
                    cudaOccupancyMaxActiveClusters(&got, gemm8_kernel<256>, &cfg) == cudaSuccess;
    if (!ok) cudaGetLastError();  // the answer is no; nothing else failed
    n = ok && got > 0 ? got : -1;
    held[h->device][size].store(n);
  }
  return std::max(n, 0);
}

struct Choice {
  int bn, grid, split;
  bool cluster;
};
// Weights a tile, and CTAs to a left-over tile: by the time of the longest CTA, in clocks. A
// k-block of a tile takes 520 + 2.5 BN (measured at 4096 x 12288 x 7168, BN 32 to 256: 609, 636,
// 757, 750, 1030, 1170), a tile's output some 1500; the weights' bytes pass at 23 a clock and SM at
// most. The exchange of a shared tile's pieces counts 16000 to 22000 through L2 and 5600 or 7200 in a
// cluster: not measured by itself, but set from whole launches (64 x 4096 x 4096: 13.1 us through L2,
// 9.6 in clusters).
static Choice choose(const dec_handle* h, int M, int N, int K) {
  const long long mt = (M + kRows - 1) / kRows, KB = (K + kBlock - 1) / kBlock;
  Choice best = {256, 1, 1, false};
  double least = 1e300;
  for (int bn : {32, 64, 96, 128, 192, 256}) {
    const long long tiles = mt * ((N + bn - 1) / bn);
    const double block = 520 + 2.5 * bn;
    const double memory = (double)N * K / (h->sms * 23.0);
    for (int split = 1; split <= 4; ++split) {
      const long long rounds = tiles / h->sms, left = tiles - rounds * h->sms;
      if (split > 1 && (left * split > h->sms || KB / split < 4)) continue;
      if (rounds == 0 && split > 1 && (split == 3 || left > clusters_held(h, split))) continue;
      const double blocks = (double)(rounds * KB) + (left ? (double)((KB + split - 1) / split) : 0.0);
      const double exchange = left == 0 || split == 1 ? 0 : rounds == 0 ? 4000 + 800.0 * split : 10000 + 3000.0 * split;
      const double t = std::max(blocks * block + (rounds + (left > 0)) * 1500.0, memory) + exchange;
      if (t < least) least = t, best = {bn, (int)(rounds ? h->sms : left * split), split, rounds == 0 && split > 1};
    }
  }
  return best;
}

static int piece_rows(int M) { return std::min(kRows, (M + 31) / 32 * 32); }
static size_t counter_bytes(const dec_handle* h) { return ((size_t)h->sms * 4 + 255) & ~size_t(255); }

size_t gemm8_ws_bytes(const dec_handle* h, int M, int N, int K) {
  const Choice c = choose(h, M, N, K);
  return counter_bytes(h) + (c.split > 1 && !c.cluster ? (size_t)c.grid * c.bn * piece_rows(M) * 4 : 0);
}

static bool encode_tile(const dec_handle* h, CUtensorMap* m, const uint8_t* p, int K, int rows, long long ld, int box_rows) {
  cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)ld};
  cuuint32_t box[2] = {kBlock, (cuuint32_t)box_rows};
  cuuint32_t es[2] = {1, 1};
  return h->encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p), dims, strides, box, es,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN>
static cudaError_t launch_bn(dec_handle* h, const Linear8& A, const Choice& c, void* ws, cudaStream_t s) {
  using L = Plan<BN>;
  const int box_rows = std::min(kRows, (A.M + 7) / 8 * 8);
  CUtensorMap tx, tw;
  if (!encode_tile(h, &tx, A.x, A.K, A.M, A.ldx, box_rows) || !encode_tile(h, &tw, A.W, A.K, A.N, A.K, BN))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = allow_smem(h, ready, (const void*)gemm8_kernel<BN>, L::kBytes);
  if (e != cudaSuccess) return e;
  Gemm8Params P = {};
  P.M = A.M;
  P.N = A.N;
  P.K = A.K;
  P.KB = (A.K + kBlock - 1) / kBlock;
  P.mtiles = (A.M + kRows - 1) / kRows;
  P.ntiles = (A.N + BN - 1) / BN;
  P.box_rows = box_rows;
  P.split = c.split;
  P.cluster = c.cluster ? 1 : 0;
  P.xs = A.xs;
  P.ldxs = A.ldxs;
  P.ws = A.ws;
  P.res = A.res;
  P.ldr = A.ldr;
  P.y = A.y;
  P.ldy = A.ldy;
  P.counters = static_cast<int*>(ws);
  P.pieces = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + counter_bytes(h));
  P.piece_rows = piece_rows(A.M);
  P.err = h->d_err;
  P.wait_ns = h->wait_ns;
  P.give_up = h->gemm8_give_up;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(c.grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = L::kBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = h->pdl ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = c.cluster ? c.split : 1;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, gemm8_kernel<BN>, tx, tw, P);
}

cudaError_t launch_gemm8(dec_handle* h, const Linear8& A, void* ws, cudaStream_t s) {
  const Choice c = choose(h, A.M, A.N, A.K);
  switch (c.bn) {
    case 32: return launch_bn<32>(h, A, c, ws, s);
    case 64: return launch_bn<64>(h, A, c, ws, s);
    case 96: return launch_bn<96>(h, A, c, ws, s);
    case 128: return launch_bn<128>(h, A, c, ws, s);
    case 192: return launch_bn<192>(h, A, c, ws, s);
    default: return launch_bn<256>(h, A, c, ws, s);
  }
}

}  // namespace dec
