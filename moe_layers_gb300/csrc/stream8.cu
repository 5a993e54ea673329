// Products of 8-bit weights with a few 8-bit rows: projections of up to 16 rows
// and the experts.
//
//   y[t][n] = sum_b sx[t][b] sw[n / 128][b] sum_{k in b} xq[t][k] wq[n][k]
//
// over blocks b of 128 values. Every weight byte is used for a few rows only, so
// the kernel is a stream of weights. The products are mma.sync's (16 weight rows x
// 8 activation rows x 32 values; measured 1.2 clocks an instruction and SM, a
// seventeenth of the stream's time at 8 rows): a block's fp32 sum lies in
// registers, where it is scaled and added to the total, while tcgen05's would have
// to be fetched from tensor memory for every block of 128.
//
// One thread copies weights by TMA into a ring in shared memory, a stage with one copy
// (of each matrix): groups of h <= 16 rows x blocks of 128 bytes, of
// which each of eight warps multiplies one (two of a single matrix). Large copies: with eight
// of 2 KB to a stage the weights streamed at 0.25 of the copy rate, and loads from global memory
// straight into the products' registers, which touch 64 bytes of 8 rows an instruction, at 0.6.
// A lane reads 16 bytes of a
// row for two products, both operands in the same permuted order, which a sum does not
// mind. The boxes have the 128-byte swizzle; product row g is group row g / 2 + 4 (g % 2),
// so that the two rows that are read at once lie in different halves of the banks.
// Warps that share rows leave their sums in shared memory and take turns at adding
// them, in block order. No atomics: the results follow from the inputs and the shape
// alone.
//
// Work: a problem is R weight rows for up to 8 NT activation rows, cut into groups of h
// rows; all problems' groups form one sequence, cut into one equal range per CTA. h is
// chosen so that the largest range holds few rows beyond the mean. Two CTAs to an SM where
// their rings fit (one or two rows of 7168): the next launch's then fill their rings beside
// the last of this one's. The groups of a CTA's range that belong to one problem are a
// segment. The ring runs on from one segment into the next, while the activation rows change.
//
// Measured, in a replayed graph, of the copy rate of 6.7 TB/s: 12288 x 7168 at one row 15.8 us
// (0.83), at eight 18.2 (0.72: one CTA to an SM); 64 tokens of 384 experts of 7168 x 256 259 us
// (0.91), 8 tokens of 32 experts of 7168 x 2048 222 (0.88). Bound by memory, and by 3 us a launch
// of ramp and last sums.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "fp8.cuh"
#include "internal.h"

namespace dec {

namespace {

constexpr int kWarps = 8;                   // that multiply
constexpr int kThreads = (kWarps + 1) * 32;  // and one that copies
constexpr int kSums = 2;                    // groups whose sums may wait for their turn
constexpr int kMaxStages = 12;
constexpr int kMaxSmem = 232448;
constexpr int kHalfSmem = 115712;           // with two CTAs to an SM
constexpr int kBarBytes = 8 * (2 * kMaxStages + 2 * kWarps * kSums) + 16;

// 4-byte asynchronous copy from global to shared memory.
__device__ __forceinline__ void copy4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// Shared memory by its 32-bit address: volatile, so that reads stay behind the waits.
__device__ __forceinline__ uint4 lds16(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p));
  return v;
}
__device__ __forceinline__ float2 lds8(uint32_t p) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(p));
  return v;
}

// The whole warp leaves a wait together.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitCtl& wc) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, wc));
}

}  // namespace

struct Stream8Params {
  const uint8_t* x;  // activation rows
  long long ldx;
  const float* xs;   // their scales
  long long ldxs;
  Stream8Bank bank, shared;  // the routed (or only) weights, and the shared expert's
  const float* inner;        // or fp32 rows [slots][K], quantised as they are read (x and xs unused)
  const int* table;          // problems (grouped), see experts8_table_kernel
  int P_max;
  const int32_t* idx;        // or, for one token: its k choices are the problems, and the shared expert
  int k, E;
  bool first;     // of the experts' two products (gate and up)
  bool by_token;  // activation rows by the slot's token, else by the slot
  int R, K, KB, rows;
  int height;      // rows of a group
  int WK;          // warps that share 16 rows, a block of 128 each: 1, 2, 4 or 8
  int stages, xrows;
  const uint16_t* res;
  long long ldr;
  void* out;
  long long ldo;
  int* err;
  unsigned long long wait_ns;
};

// Distance of activation rows in shared memory: 16-byte reads of 2 rows x 64 bytes then meet no bank twice.
__host__ __device__ constexpr int pitch_of(int bytes) { return (bytes + 127) / 128 * 128 + 64; }
// WK warps take the blocks along a group's rows, UW each, WG = kWarps / WK groups a
// stage. A stage of the ring holds [WK UW][WG h][128] bytes of each matrix, then, if the
// last block of a row is short, [WG h][128] of such blocks. (A stage costs its readers
// some 500 clocks of waiting and reading beside the products, so it is large: 32 KB.)
__host__ __device__ constexpr int blocks_each(int na) { return na == 2 ? 1 : 2; }
__host__ __device__ constexpr int up1024(int n) { return (n + 1023) & ~1023; }
__host__ __device__ constexpr int main_bytes(int na, int h) { return up1024(kWarps * blocks_each(na) * h * 128); }
__host__ __device__ constexpr int warps_along(int KB, int na) {
  return KB >= 8 * blocks_each(na) ? 8 : KB >= 4 * blocks_each(na) ? 4 : KB >= 2 * blocks_each(na) ? 2 : 1;
}
__host__ __device__ constexpr int stage_bytes(int na, int h, int K) {
  return na * main_bytes(na, h) + (K % 128 ? up1024(kWarps / warps_along((K + 127) / 128, na) * h * 128) : 0);
}

// The groups [ga, gb) of problem p, the part of a CTA's range [.., q1) that begins at q.
struct Segment {
  int p, ga, gb;
  __device__ Segment(long long q, long long q1, int per_problem) {
    p = (int)(q / per_problem);
    ga = (int)(q - (long long)p * per_problem);
    gb = (int)min((long long)per_problem, ga + (q1 - q));
  }
};

template <int NT, bool PAIR, bool GROUPED>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1)
    stream8_kernel(const __grid_constant__ CUtensorMap tm0, const __grid_constant__ CUtensorMap tm1,
                   const __grid_constant__ CUtensorMap ts0, const __grid_constant__ CUtensorMap ts1,
                   const Stream8Params P) {
  constexpr int NA = PAIR ? 2 : 1;
  constexpr int COLS = 8 * NT;
  constexpr int VALUES = NA * NT * 4;  // totals a lane
  constexpr int UW = blocks_each(NA);
  constexpr int BATCH = 8 / UW;        // stages for which a warp's scales are loaded at once
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int KB = P.KB, WK = P.WK, WG = kWarps / WK, xpitch = pitch_of(P.K), h = P.height;
  const int stage = stage_bytes(NA, h, P.K);
  const int chunks = (KB + WK * UW - 1) / (WK * UW), per_problem = (P.R + h - 1) / h;
  uint8_t* xq = ring + (size_t)P.stages * stage;                         // [xrows][xpitch]
  float* xsc = reinterpret_cast<float*>(xq + (size_t)P.xrows * xpitch);  // [KB][COLS]
  float* sums = xsc + (size_t)KB * COLS;                                 // [kSums][kWarps][VALUES][32]
  uint64_t* full = reinterpret_cast<uint64_t*>(sums + kSums * kWarps * VALUES * 32);
  uint64_t* empty = full + kMaxStages;
  uint64_t* sfull = empty + kMaxStages;  // [kSums][WG]
  uint64_t* sempty = sfull + kSums * kWarps;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sempty + kSums * kWarps);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // The experts' first product lets its dependent start only after its own dependency wait: when the
  // second one starts, the routing is complete, and it reads that and streams weights before it waits
  // (past L1, which may hold what lay at the same addresses for an earlier call).
  if (!P.first) pdl_trigger();
  if (threadIdx.x == 0) {
    for (int i = 0; i < P.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kWarps);
    }
    for (int i = 0; i < kSums * WG; ++i) {
      mbar_init(&sfull[i], WK);
      mbar_init(&sempty[i], 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  const WaitCtl wc{abort_flag, P.err, P.wait_ns};

  int problems = 1;
  if (GROUPED) {
    if (P.first) {
      pdl_wait();
      pdl_trigger();
    }
    if (P.idx == nullptr) problems = ld_cg_s32(P.table);
  }
  // One token: its choices with an id in [0, E) are the problems, in order, and the shared expert. Lane j holds choice j,
  // -1 for one that is left out.
  int choice = -1;
  if (GROUPED && P.idx != nullptr) {
    if (lane < P.k) choice = ld_cg_s32(P.idx + lane);
    if (choice < 0 || choice >= P.E) choice = -1;
    problems = __popc(__ballot_sync(0xffffffffu, choice >= 0)) + (P.shared.W[0] != nullptr ? 1 : 0);
  }
  // Problem p: expert (-1: the shared one), first slot and rows. Taken by whole warps.
  struct Problem {
    int e = 0, slot0 = 0, cnt = 0;
  };
  auto problem = [&](int p) {
    Problem r;
    if (!GROUPED) {
      r.cnt = P.rows;
    } else if (P.idx != nullptr) {
      const uint32_t in = __ballot_sync(0xffffffffu, choice >= 0);
      const uint32_t at = __ballot_sync(0xffffffffu, choice >= 0 && __popc(in & ((1u << lane) - 1)) == p);
      r.slot0 = at != 0 ? __ffs(at) - 1 : P.k;
      r.e = __shfl_sync(0xffffffffu, choice, at != 0 ? r.slot0 : 31);  // lane 31 holds no choice
      r.cnt = 1;
    } else {
      r.e = ld_cg_s32(P.table + 1 + 3 * p);
      r.slot0 = ld_cg_s32(P.table + 2 + 3 * p);
      r.cnt = ld_cg_s32(P.table + 3 + 3 * p);
    }
    return r;
  };
  // At most 1088 problems of 2048 groups, or one of 2^17: 32 bits hold them times the CTAs. (Divisions of 64 bits, behind
  // the load of the routing: one token, 384 experts of 7168 x 256 20.2 us instead of 19.4.)
  const uint32_t total = (uint32_t)problems * per_problem, G = gridDim.x, c = blockIdx.x;
  const long long q0 = c * total / G, q1 = (c + 1) * total / G;
  const int* tokens = P.table + 1 + 3 * P.P_max;

  if (warp == kWarps) {
    // ------------------------------------------------------------ copies
    const uint64_t pol = policy_evict_first();
    int s = 0;        // the next stage of the ring
    uint32_t ph = 0;  // and how often the ring has gone round, mod 2
    int issued = 0;   // stages, up to the ring's
    bool ok = true;
    for (long long q = q0; q < q1 && ok;) {
      const Segment S(q, q1, per_problem);
      q += S.gb - S.ga;
      const int e = problem(S.p).e;
      const CUtensorMap* m0 = e < 0 ? &ts0 : &tm0;
      const CUtensorMap* m1 = e < 0 ? &ts1 : &tm1;
      const int row = (e < 0 ? 0 : e) * P.R;  // at most 2^31 rows in a bank
      for (int j = S.ga; j < S.gb && ok; j += WG)
        for (int ch = 0; ch < chunks; ++ch) {
          if (!warp_wait(&empty[s], ph ^ 1u, wc)) {
            ok = false;
            break;
          }
          const int su = uniform(s), kb0 = uniform(ch * WK * UW), from = uniform(row + j * h);
          const bool tail = !PAIR && kb0 + WK * UW > P.K / 128 && P.K % 128 != 0;  // the stage holds the short block
          if (elect_one()) {
            mbar_arrive_expect_tx(&full[su], (uint32_t)((NA * kWarps * UW + (tail ? WG : 0)) * h * 128));
            uint8_t* dst = ring + (size_t)su * stage;
            tma_load_3d(dst, m0, &full[su], 0, from, kb0, pol);
            if (PAIR) tma_load_3d(dst + main_bytes(NA, h), m1, &full[su], 0, from, kb0, pol);
            if (tail) tma_load_2d(dst + main_bytes(NA, h), &tm1, &full[su], (KB - 1) * 128, from, pol);
          }
          __syncwarp();
          issued = min(issued + 1, P.stages);
          if (++s == P.stages) {
            // From here on stages have to come back: not before the kernel ahead has ended, whose time is not a wait's.
            if (ph == 0) pdl_wait();
            s = 0, ph ^= 1u;
          }
        }
    }
    // No copy may still be in flight when the CTA exits: the ring's last stages, newest first.
    for (; issued > 0; --issued) {
      if (--s < 0) s = P.stages - 1, ph ^= 1u;
      mbar_wait_drain(&full[s], ph, P.err, P.wait_ns);
    }
    return;
  }

  // -------------------------------------------------------------- products
  const int g = lane >> 2, t = lane & 3;
  const int rg = (g >> 1) + 4 * (g & 1);         // this lane's group rows: rg, rg + 8
  const int sub = warp / WK, along = warp % WK;  // group of a stage, block of its width
  // this lane's first 16 bytes of row rg in a stage (the second: 64 bytes on, swizzled), and in a stage's short blocks
  const int line = along * UW * WG * h + sub * h + rg, short_line = sub * h + rg;
  const int short_at = NA * main_bytes(NA, h) + short_line * 128 + ((t ^ (short_line & 7)) << 4);
  const int short_kb = P.K % 128 != 0 ? KB - 1 : -1;
  int at[UW];
#pragma unroll
  for (int u = 0; u < UW; ++u) at[u] = (line + u * WG * h) * 128 + ((t ^ ((line + u * WG * h) & 7)) << 4);
  const uint32_t ring_at = smem_u32(ring), up_at = main_bytes(NA, h);
  // its 16 bytes of an activation row and two columns' scales; columns behind the rows repeat the last one, and nothing
  // reads their sums
  uint32_t x_at[NT], xsc_at[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    x_at[nt] = smem_u32(xq) + (uint32_t)min(nt * 8 + g, P.xrows - 1) * xpitch + t * 16;
    xsc_at[nt] = smem_u32(xsc) + (nt * 8 + 2 * t) * 4;
  }
  if (!GROUPED || !P.first) pdl_wait();
  int s = 0;           // the ring's next stage
  uint32_t sph = 0;    // and how often the ring has gone round, mod 2
  uint32_t turns = 0;  // groups whose sums this warp's group has left so far
  bool ok = true;
  for (long long q = q0; q < q1;) {
    const Segment S(q, q1, per_problem);
    q += S.gb - S.ga;
    const Problem pr = problem(S.p);
    const int slot0 = pr.slot0, cnt = pr.cnt, e = pr.e;

    // Weight scales of a warp's blocks in the BATCH stages from `ch` on of the group j: lane = matrix,
    // block of rows (16 rows lie in two at most), block.
    const float* sbase;
    {
      const Stream8Bank& B = e < 0 ? P.shared : P.bank;
      sbase = B.scales[PAIR ? lane >> 4 : 0] + (e < 0 ? 0 : (size_t)e * ((P.R + 127) / 128) * KB);
    }
    auto load_scales = [&](int j, int ch) {
      const int i = lane & 7, kb = min(((ch + i / UW) * WK + along) * UW + i % UW, KB - 1);
      const int block = min(((j + sub) * h >> 7) + ((lane >> 3) & 1), (P.R - 1) >> 7);
      return ld_act_f32(sbase + (size_t)block * KB + kb);  // not conditional: a branch around it would wait for it
    };
    float sc = load_scales(S.ga, 0);

    // This problem's activation rows, zeros up to a whole block: all copies in flight at once.
    if (!named_bar_and(1, kWarps * 32, ok)) return;  // the previous segment is done with them
    if (GROUPED && P.inner != nullptr) {
      // a warp's lanes take four values each of a group of 128: its largest, its scale, 8 bits
      for (int n = warp; n < cnt * KB; n += kWarps) {
        const int j = n / KB, b = n - j * KB;
        const float4 v = ld_act_f4(P.inner + (size_t)(slot0 + j) * P.K + b * 128 + lane * 4);
        uint32_t most = 0;
        for (float f : {v.x, v.y, v.z, v.w}) most = max(most, __float_as_uint(f) & 0x7FFFFFFFu);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
        const Scale8 sc = scale_e4m3(__uint_as_float(most));
        *reinterpret_cast<uint32_t*>(xq + (size_t)j * xpitch + b * 128 + lane * 4) =
            pack_e4m3x4(v.x * sc.up, v.y * sc.up, v.z * sc.up, v.w * sc.up);
        if (lane == 0) xsc[b * COLS + j] = sc.scale;
      }
    } else {
      for (int j = warp; j < COLS; j += kWarps) {
        const bool in = j < cnt;
        const long long row =
            in && GROUPED && P.by_token && P.idx == nullptr ? ld_act_s32(tokens + slot0 + j) : slot0 + j;
        if (in) {
          const uint8_t* src = P.x + (GROUPED && P.idx != nullptr ? 0 : row) * P.ldx;
          uint8_t* dst = xq + (size_t)j * xpitch;
          for (int k = lane * 16; k < xpitch - 64; k += 512) {
            if (k < P.K)
              cp_async16(dst + k, src + k);
            else
              *reinterpret_cast<uint4*>(dst + k) = make_uint4(0, 0, 0, 0);
          }
        }
        for (int b = lane; b < KB; b += 32) {
          if (in)
            copy4(xsc + b * COLS + j, P.xs + (GROUPED && P.idx != nullptr ? 0 : row) * P.ldxs + b);
          else
            xsc[b * COLS + j] = 0.f;
        }
      }
    }
    cp_async_wait_all();
    named_bar_sync(1, kWarps * 32);

    for (int j = S.ga; j < S.gb && ok; j += WG) {
      const bool mine = j + sub < S.gb;
      const int r0 = (j + sub) * h + rg;  // this lane's weight rows: r0, r0 + 8
      // lanes that hold the scales of their blocks (the group's first or second block of rows)
      const int from[2] = {((min(r0, P.R - 1) >> 7) - ((j + sub) * h >> 7)) << 3,
                           min((min(r0 + 8, P.R - 1) >> 7) - ((j + sub) * h >> 7), 1) << 3};
      float tot[NA][NT][4];
#pragma unroll
      for (int a = 0; a < NA; ++a)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) tot[a][nt][e] = 0.f;

      for (int ch = 0; ch < chunks && ok; ch += BATCH) {
        const float next = ch + BATCH < chunks ? load_scales(j, ch + BATCH) : load_scales(j + WG, 0);
#pragma unroll
        for (int n = 0; n < BATCH; ++n) {
          if (ch + n >= chunks) break;
          if (!warp_wait(&full[s], sph, wc)) {
            ok = false;
            break;
          }
          const int kb0 = ((ch + n) * WK + along) * UW;
          uint4 w[UW][NA][2][2];
          const uint32_t base = ring_at + (uint32_t)(s * stage);
#pragma unroll
          for (int u = 0; u < UW; ++u) {
            const uint32_t off = !PAIR && kb0 + u == short_kb ? short_at : at[u];
#pragma unroll
            for (int a = 0; a < NA; ++a)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                w[u][a][e][0] = lds16(base + off + a * up_at + e * 1024);
                w[u][a][e][1] = lds16(base + (off ^ 64) + a * up_at + e * 1024);
              }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty[s]);
          if (++s == P.stages) s = 0, sph ^= 1u;
          if (!mine) continue;
#pragma unroll
          for (int u = 0; u < UW; ++u) {
            // blocks behind the last are zeros of the copies
            const int kb = min(kb0 + u, KB - 1);
            float ws[NA][2];
#pragma unroll
            for (int a = 0; a < NA; ++a)
#pragma unroll
              for (int e = 0; e < 2; ++e) ws[a][e] = __shfl_sync(0xffffffffu, sc, a * 16 + from[e] + n * UW + u);
            auto column = [&](int nt) {
              const uint4 b0 = lds16(x_at[nt] + kb * 128), b1 = lds16(x_at[nt] + kb * 128 + 64);
              const float2 sx = lds8(xsc_at[nt] + kb * (COLS * 4));
#pragma unroll
              for (int a = 0; a < NA; ++a) {
                float acc[4] = {0.f, 0.f, 0.f, 0.f};
                const uint4 l0 = w[u][a][0][0], l1 = w[u][a][0][1], h0 = w[u][a][1][0], h1 = w[u][a][1][1];
                mma_e4m3(acc, l0.x, h0.x, l0.y, h0.y, b0.x, b0.y);
                mma_e4m3(acc, l0.z, h0.z, l0.w, h0.w, b0.z, b0.w);
                mma_e4m3(acc, l1.x, h1.x, l1.y, h1.y, b1.x, b1.y);
                mma_e4m3(acc, l1.z, h1.z, l1.w, h1.w, b1.z, b1.w);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  tot[a][nt][e] = fmaf(acc[e], ws[a][e >> 1] * ((e & 1) ? sx.y : sx.x), tot[a][nt][e]);
              }
            };
            column(0);
            if (NT == 2 && (!GROUPED || cnt > 8)) column(NT - 1);
          }
        }
        sc = next;
      }
      if (!ok) break;
      if (!mine) continue;

      if (WK > 1) {
        // Every warp of the group leaves its sums; one of them, in turn, adds them up.
        const int n = (int)(turns % kSums), b = n * WG + sub;
        const uint32_t ph = (turns / kSums) & 1u;
        const int reducer = (int)(turns % WK);
        ++turns;
        if (!warp_wait(&sempty[b], ph ^ 1u, wc)) {
          ok = false;
          break;
        }
        float* slot = sums + (size_t)(n * kWarps + warp) * VALUES * 32 + lane;
#pragma unroll
        for (int a = 0; a < NA; ++a)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) slot[((a * NT + nt) * 4 + e) * 32] = tot[a][nt][e];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sfull[b]);
        if (along != reducer) continue;
        if (!warp_wait(&sfull[b], ph, wc)) {
          ok = false;
          break;
        }
        const float* piece = sums + (size_t)(n * kWarps + sub * WK) * VALUES * 32 + lane;
#pragma unroll
        for (int a = 0; a < NA; ++a)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float* v = piece + ((a * NT + nt) * 4 + e) * 32;
              float sum = v[0];
#pragma unroll
              for (int w = 1; w < kWarps; ++w)
                if (w < WK) sum += v[w * VALUES * 32];
              tot[a][nt][e] = sum;
            }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sempty[b]);
      }
      // Finished rows: this lane's two, columns 2 t and 2 t + 1 of each eight.
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = r0 + 8 * (e >> 1), col = nt * 8 + 2 * t + (e & 1);
          if (rg + 8 * (e >> 1) >= h || r >= P.R || col >= cnt) continue;
          const float v = tot[0][nt][e];
          if (PAIR) {
            static_cast<float*>(P.out)[(long long)(slot0 + col) * P.ldo + r] = v / (1.0f + expf(-v)) * tot[NA - 1][nt][e];
          } else if (GROUPED) {
            static_cast<float*>(P.out)[(long long)(slot0 + col) * P.ldo + r] = v;
          } else {
            const float a = P.res != nullptr ? bf2f(ld_act_u16(P.res + col * P.ldr + r)) : 0.f;
            static_cast<uint16_t*>(P.out)[col * P.ldo + r] = f2bf(v + a);
          }
        }
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
__global__ void __launch_bounds__(128) experts8_combine_kernel(const float* y, const int* entry, const int32_t* idx,
                                                               int E, const float* w, int M, int k, bool shared,
                                                               const uint16_t* res, uint16_t* out, int H) {
  const int t = blockIdx.y, c = (blockIdx.x * 128 + threadIdx.x) * 4;
  pdl_trigger();
  pdl_wait();
  if (c >= H) return;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  // Eight choices at a time: their slots and weights, then their values, all loads in flight before any is used.
  for (int j0 = 0; j0 < k; j0 += 8) {
    int slot[8];
    float wj[8];
    float4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int j = min(j0 + u, k - 1);
      slot[u] = ld_act_s32(entry != nullptr ? entry + t * k + j : idx + j);
      wj[u] = ld_act_f32(w + t * k + j);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int j = min(j0 + u, k - 1);
      // one token: choice j's slot is j, if its id is one
      if (entry == nullptr) slot[u] = slot[u] >= 0 && slot[u] < E ? j : -1;
      v[u] = ld_act_f4(y + (size_t)max(slot[u], 0) * H + c);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (j0 + u < k && slot[u] >= 0) {
        a.x = fmaf(wj[u], v[u].x, a.x), a.y = fmaf(wj[u], v[u].y, a.y);
        a.z = fmaf(wj[u], v[u].z, a.z), a.w = fmaf(wj[u], v[u].w, a.w);
      }
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
// Shared memory besides the ring.
static size_t fixed_bytes(int xrows, int nt, int K, bool pair) {
  const size_t KB = (K + 127) / 128;
  return 1024 + (size_t)xrows * pitch_of(K) + KB * 8 * nt * 4 + (size_t)kSums * kWarps * (pair ? 2 : 1) * nt * 4 * 32 * 4 +
         kBarBytes;
}
static size_t one_stage(int K, bool pair, int h) { return stage_bytes(pair ? 2 : 1, h, K); }
// Ring stages that fit beside it.
static int stages_for(int xrows, int nt, int K, bool pair, int h, int smem = kMaxSmem) {
  const size_t fixed = fixed_bytes(xrows, nt, K, pair);
  if (fixed >= (size_t)smem) return 0;
  return std::min<int>(kMaxStages, (int)((smem - fixed) / one_stage(K, pair, h)));
}

// Rows of a group: the largest range of a CTA in rows, with two rows' time for each group.
static int group_height(int R, double problems, int grid) {
  int best = 16;
  double least = 1e30;
  for (int h = 16; h >= 8; --h) {
    const double groups = std::ceil(problems * ((R + h - 1) / h) / grid);
    const double cost = groups * (h + 2);
    if (cost < least) least = cost, best = h;
  }
  return best;
}

// Weights [rows][K]: whole blocks of 128 as [K / 128][rows][128], boxes of `blocks` x `height` rows; or, for
// the short block at a row's end, as they are (what is beyond K reads as zeros).
static bool encode_blocks(const dec_handle* h, CUtensorMap* m, const uint8_t* W, int K, long long rows, int height,
                          int blocks) {
  const int whole = std::max(1, K / 128);
  cuuint64_t dims[3] = {(cuuint64_t)std::min(128, K), (cuuint64_t)rows, (cuuint64_t)whole};
  cuuint64_t strides[2] = {(cuuint64_t)K, 128};
  cuuint32_t box[3] = {128, (cuuint32_t)height, (cuuint32_t)blocks};
  cuuint32_t es[3] = {1, 1, 1};
  return h->encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(W), dims, strides, box, es,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
static bool encode_short(const dec_handle* h, CUtensorMap* m, const uint8_t* W, int K, long long rows, int height) {
  cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)K};
  cuuint32_t box[2] = {128, (cuuint32_t)height};
  cuuint32_t es[2] = {1, 1};
  return h->encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(W), dims, strides, box, es,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// `problems`: how many there will be, about; E: experts in the bank (1 for one matrix).
template <int NT, bool PAIR, bool GROUPED>
static cudaError_t launch_one(dec_handle* h, Stream8Params P, int xrows, double problems, int E, cudaStream_t s) {
  P.KB = (P.K + 127) / 128;
  P.WK = warps_along(P.KB, PAIR ? 2 : 1);
  // The experts' second product has rows enough for several groups a stage: fewer warps along a group, so
  // that its sums are joined every four stages at most (8 tokens of 32 experts of 7168 x 2048: 244 -> 221 us).
  if (GROUPED && !PAIR)
    while (P.WK > 1 && P.KB < 4 * P.WK * blocks_each(1)) P.WK /= 2;
  P.xrows = xrows;
  // Two CTAs to an SM where each has a ring of three stages: the next launch's CTAs then start, and
  // fill their rings, beside the last of this one's.
  int ctas = 2;
  P.height = group_height(P.R, problems, h->sms * ctas);
  P.stages = stages_for(xrows, NT, P.K, PAIR, P.height, kHalfSmem);
  if (NT > 1 || P.stages < 3) {
    ctas = 1;
    P.height = group_height(P.R, problems, h->sms);
    P.stages = stages_for(xrows, NT, P.K, PAIR, P.height);
  }
  P.err = h->d_err;
  P.wait_ns = h->wait_ns;
  if (P.stages < 2) return cudaErrorInvalidConfiguration;
  const int box = kWarps / P.WK * P.height, across = P.WK * blocks_each(PAIR ? 2 : 1);
  const long long rows = (long long)E * P.R;
  const Stream8Bank& S = P.shared.W[0] != nullptr ? P.shared : P.bank;
  const long long srows = P.shared.W[0] != nullptr ? P.R : rows;
  CUtensorMap m[4];
  if (!encode_blocks(h, &m[0], P.bank.W[0], P.K, rows, box, across) ||
      !encode_blocks(h, &m[2], S.W[0], P.K, srows, box, across))
    return cudaErrorInvalidValue;
  m[1] = m[0];
  m[3] = m[2];
  if (PAIR && (!encode_blocks(h, &m[1], P.bank.W[1], P.K, rows, box, across) ||
               !encode_blocks(h, &m[3], S.W[1], P.K, srows, box, across)))
    return cudaErrorInvalidValue;
  if (!PAIR && P.K % 128 != 0 && !encode_short(h, &m[1], P.bank.W[0], P.K, rows, box)) return cudaErrorInvalidValue;
  const size_t smem = fixed_bytes(xrows, NT, P.K, PAIR) + (size_t)P.stages * one_stage(P.K, PAIR, P.height);
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = allow_smem(h, ready, (const void*)stream8_kernel<NT, PAIR, GROUPED>, kMaxSmem);
  if (e != cudaSuccess) return e;
  return launch_k(h, stream8_kernel<NT, PAIR, GROUPED>, dim3(h->sms * ctas), dim3(kThreads), smem, s, m[0], m[1], m[2],
                  m[3], P);
}

int stream8_rows(int K, bool pair) {
  for (int rows = 16; rows > 0; --rows)
    if (stages_for(rows, rows > 8 ? 2 : 1, K, pair, 16) >= 2) return rows;
  return 0;
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
  P.rows = L.M;
  P.res = L.res;
  P.ldr = L.ldr;
  P.out = L.y;
  P.ldo = L.ldy;
  return L.M <= 8 ? launch_one<1, false, false>(h, P, L.M, 1, 1, s) : launch_one<2, false, false>(h, P, L.M, 1, 1, s);
}

Experts8Plan experts8_plan(int M, int k, int E, int H, int I, bool shared) {
  Experts8Plan p;
  // Problems of up to 16 rows where the experts have four tokens and more in the mean, else of 8,
  // whose rows leave twice the room for weights in flight (64 tokens, 384 experts of 7168 x 256: 260 us,
  // with 16 rows 350; 64 tokens that all choose the same 8 experts of 7168 x 2048 read each expert four
  // times with 16: 395 us).
  const int want = M * k >= 4 * E ? 16 : 8;
  p.most = std::min(std::min(stream8_rows(H, true), stream8_rows(I, false)), want);
  p.slots = M * k + M;
  const int most = std::max(p.most, 1);
  p.P_max = std::min(M * k, E + M * k / most) + (shared ? (M + most - 1) / most : 0);
  p.words = 1 + 3 * p.P_max + p.slots + M * k;
  return p;
}

cudaError_t launch_experts8(dec_handle* h, const Experts8& X, const Experts8Plan& plan, int* table, float* inner, float* y,
                            cudaStream_t s) {
  const int M = X.M, k = X.k, H = X.H, I = X.I;
  const bool shared = X.sgate.W[0] != nullptr;
  // experts that at least one of M k even choices falls on
  const double problems = X.E * (1.0 - std::pow(1.0 - 1.0 / X.E, M * k)) + (shared ? (M + plan.most - 1) / plan.most : 0);
  const int xrows = std::min(plan.most, M * k);
  cudaError_t e;
  Stream8Params P = {};
  if (M == 1) {
    P.idx = X.idx;
    P.k = k;
    P.E = X.E;
  } else {
    P.table = table;
    P.P_max = plan.P_max;
    LaunchScope scope(h, "experts8_table", s);
    e = launch_k(h, experts8_table_kernel, dim3(1), dim3(1024), 0, s, X.idx, M, k, X.E, shared, plan.most, plan.P_max,
                 table);
    if (e != cudaSuccess) return e;
  }
  P.x = X.x;
  P.ldx = X.ldx;
  P.xs = X.xs;
  P.ldxs = X.ldxs;
  P.bank = X.gate;
  P.shared = X.sgate;
  P.by_token = true;
  P.first = true;
  P.R = I;
  P.K = H;
  P.out = inner;
  P.ldo = I;
  {
    LaunchScope scope(h, "experts8_gate_up", s);
    e = plan.most <= 8 ? launch_one<1, true, true>(h, P, xrows, problems, X.E, s)
                       : launch_one<2, true, true>(h, P, xrows, problems, X.E, s);
    if (e != cudaSuccess) return e;
  }
  P.inner = inner;
  P.bank = X.down;
  P.shared = X.sdown;
  P.by_token = false;
  P.first = false;
  P.R = H;
  P.K = I;
  P.out = y;
  P.ldo = H;
  {
    LaunchScope scope(h, "experts8_down", s);
    e = plan.most <= 8 ? launch_one<1, false, true>(h, P, xrows, problems, X.E, s)
                       : launch_one<2, false, true>(h, P, xrows, problems, X.E, s);
    if (e != cudaSuccess) return e;
  }
  LaunchScope scope(h, "experts8_combine", s);
  return launch_k(h, experts8_combine_kernel, dim3((H / 4 + 127) / 128, M), dim3(128), 0, s, (const float*)y,
                  M == 1 ? (const int*)nullptr : (const int*)(table + 1 + 3 * plan.P_max + plan.slots), X.idx, X.E, X.w, M, k,
                  shared, X.res, X.out, H);
}

}  // namespace dec
