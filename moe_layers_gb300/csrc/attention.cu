// Attention of a decode step over the paged cache.
//
// One pass over the keys with a running maximum and sum per row: for a tile of
// 64 keys, S = Q K^T, m' = max(m, max S), O = O 2^(m - m') + P V with
// P = 2^(S - m'), l = l 2^(m - m') + sum P, the scale and log2 e folded into
// one factor on S. What bounds it is the read of the cache: 4 query rows to a
// key row make 4 flops a byte. The cache therefore streams through a ring of
// TMA copies (one box per block and 64 elements, 128-byte swizzle) that two
// warps keep full, one with K and one with V, while four warps multiply with
// mma.sync m16n8k16, whose fragments come from the ring by ldmatrix without bank
// conflicts; up to 32 rows the multiplications are no limit. Each CTA streams one
// equal share of all tiles (attention.cuh); rows that several CTAs took are
// joined by a second kernel. Measured (64 heads on 16, head dim 128, calls back to
// back): one request of 131000 tokens 157 us, 6.8 TB/s, the copy rate; 61 requests
// of 1..4096 tokens 49 us, 5.6 TB/s; 8 requests of 8 drafts on 2000..16000 tokens
// 82 us, 5.9 TB/s.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "attention.cuh"

namespace dec {

constexpr int kTileKeys = 64;
constexpr int kAttnThreads = 192;  // 4 multiplying warps, one copying K, one copying V
// Two CTAs an SM: one warp per scheduler leaves the products' latency exposed
// (870 cycles a tile against the 1370 that an SM's share of the memory rate
// takes for one), and a CTA between two pieces does not stop the SM's stream.
constexpr int kAttnCtasPerSm = 2;
constexpr int kAttnSmem = 115712;
// Tiles that beginning and ending a (head, chunk) costs as much as: 0.5 us
// against 0.78 a tile (61 ragged requests of 1..4096 tokens: 60.9 us with 0, 44.6
// with 1, 44.8 with 2; without ragged lengths no difference).
constexpr int kPieceLead = 1;
// The same of the tcgen05 kernel, in its 128-key tiles (64 requests on 32768
// shared tokens: 104 us with 3, 101 with 5 and 6; 4 requests of 16 drafts at 1000
// tokens: 19.2, 19.9 and 20.4).
constexpr int kPieceLeadTc = 5;

// How the four warps share a chunk: WK of them split a tile's keys, 4 / WK
// groups of 16 rows split its rows. HALF: chunks of 8 rows (the lower half of
// each 16-row product is not used).
template <int WK_, bool HALF_>
struct Rows {
  static constexpr int WK = WK_, WM = 4 / WK_;
  static constexpr bool HALF = HALF_;
  static constexpr int kRows = HALF ? 8 : 16 * WM;
  static constexpr int kKeys = kTileKeys / WK;  // keys of one warp
  static_assert(!HALF || WK == 4, "a chunk of 8 rows has one group of warps");
};
using Rows8 = Rows<4, true>;
using Rows16 = Rows<4, false>;
using Rows32 = Rows<2, false>;

// Shared memory of the kernel with chunks RP for the prefix and RO for own tokens.
template <int D, class RP, class RO>
struct AttnShape {
  static constexpr int kHalf = kTileKeys * D * 2;  // K or V bytes of a stage
  static constexpr int kStage = 2 * kHalf;
  // sums of the warps that join another at the end of a piece, 8 rows at a time
  static constexpr int kMerge = std::max((RP::WK - 1) * RP::WM, (RO::WK - 1) * RO::WM) * 8 * D * 4;
  static constexpr int kQ = RO::HALF ? 8 * D * 2 : 0;  // query rows of 8-row chunks
  static constexpr int kFixed = 1024 + 2048;  // alignment, barriers and tables
  static constexpr int kStages = std::min(12, (kAttnSmem - kFixed - kMerge - kQ) / kStage);
  static constexpr int kTotal = kStages * kStage + kMerge + kQ + kFixed;
  static_assert(kStages >= 3 && kTotal <= kAttnSmem, "shared memory");
};

struct AttnShared {
  uint64_t full[12], empty[12], qfull;
  PartTable parts;
  float2 ml[4][8];
  uint8_t valid[12];  // per stage: which 16-key quarters lie in blocks of the cache
  int abort;
};
static_assert(sizeof(AttnShared) <= 2048, "attention tables");

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Byte offset of 16-byte vector c (of a row of 64 elements) of row r in a
// sub-tile of 128-byte rows with the 128-byte swizzle.
__device__ __forceinline__ uint32_t swz(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

template <int D, class RP, class RO>
__global__ void __launch_bounds__(kAttnThreads, kAttnCtasPerSm)
    attention_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                     const __grid_constant__ AttentionLaunch L) {
  using S = AttnShape<D, RP, RO>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float2* s_merge = reinterpret_cast<float2*>(smem + S::kStages * S::kStage);  // [warp][D / 8][lane]
  uint8_t* s_q = smem + S::kStages * S::kStage + S::kMerge;  // [D / 64][8 rows][128 bytes], swizzled
  AttnShared& sh = *reinterpret_cast<AttnShared*>(s_q + S::kQ);
  const AttentionParams& a = L.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = a.group;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&sh.full[i], 2);
      mbar_init(&sh.empty[i], 4);
    }
    mbar_init(&sh.qfull, 128);
    sh.abort = 0;
    fence_mbar_init();
    tmap_prefetch(&tk);
    tmap_prefetch(&tv);
  }
  warm_l2(a);
  // Dependents start only behind this wait, when every earlier launch of the
  // stream is complete: the joining kernel reads the lengths before its own
  // wait, and the own tokens' launch behind a prefix launch (late_wait) does not
  // need that one's results: it waits at its end, so that its completion is both.
  if (!L.late_wait) pdl_wait();
  pdl_trigger();
  if (warp == 0) build_parts(sh.parts, a, L.plan);
  __syncthreads();
  const long long W = sh.parts.first[a.requests + 1], G = plan_ctas(W, L.plan.ctas), c = blockIdx.x;
  const long long u0 = c < G ? unit_start(c, W, G) : 0, u1 = c < G ? unit_start(c + 1, W, G) : 0;
  const WaitCtl wc{&sh.abort, L.err, L.wait_ns};
  Piece q;
  if (u0 < u1) q.begin(sh.parts, a, L.plan, u0, u1);

  if (warp >= 4) {
    // ------------------------------------------------------------ copies
    const bool keys = warp == 4;  // this warp copies K, the other V
    const int box = min(1 << a.shift, kTileKeys);  // keys of one box
    const int per = kTileKeys / box;               // boxes (blocks) of a tile
    constexpr int kSub = D / 64;
    const uint64_t first = policy_evict_first(), normal = policy_evict_normal();
    uint32_t issued = 0;
    int s = 0;
    uint32_t phase = 1;
    for (long long u = u0; u < u1 && !q.empty();) {
      {
        // The queries of the next piece into L2 (this warp is a few tiles ahead of
        // the products): read from DRAM under load they took 2.5 us of each piece.
        Piece n = q;
        if (keys && u + q.units < u1) {
          n.next(sh.parts, a, L.plan, u + q.units, u1);
          const int each = n.part == 0 ? RP::kRows : RO::kRows;
          const int rows = n.empty() ? 0 : min(each, sh.parts.rows[n.part] * group - n.chunk * each);
          for (int i = lane; i < rows * kSub; i += 32) {
            const int rr = n.chunk * each + i / kSub, row = div_group(rr, L.group_mul);
            const uint16_t* src = a.q + (long long)(sh.parts.row0[n.part] + row) * a.ldq +
                                  (long long)(n.kvh * group + rr - row * group) * D + (i % kSub) * 64;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(src));
          }
        }
      }
      const int len = sh.parts.len[q.part];
      const int32_t* table = q.part == 0 ? a.prefix_table : a.block_table + (long long)(q.part - 1) * a.max_blocks;
      const uint64_t policy = q.chunks == 1 ? first : normal;
      BlockIds ids(table, (int)(((long long)len + (1 << a.shift) - 1) >> a.shift));
      bool ok = true;
      for (int t = q.tile0; t < q.tile1; ++t) {
        const int key0 = t * kTileKeys;
        const int boxes = min(per, (len - key0 + box - 1) / box);  // boxes with keys of the part
        ids.advance(key0 >> a.shift);
        // lane b < per: the cache block of box b, a.blocks if it is not there
        const int id = ids.get((key0 >> a.shift) + min(lane, per - 1));
        const bool there = lane < boxes && id >= 0 && id < a.blocks;
        const uint32_t mask = __ballot_sync(0xffffffffu, there);
        const int from = there ? id : a.blocks;  // past the end of the cache: reads zeros
        ok = warp_wait(&sh.empty[s], phase, wc);
        if (!ok) break;
        const int su = uniform(s);
        uint8_t* dst = smem + su * S::kStage + (keys ? 0 : S::kHalf);
        const int row = uniform((q.kvh << a.shift) + (key0 & ((1 << a.shift) - 1)));
        if (elect_one()) {
          if (keys) {
            int quarters = 0;  // 16-key quarters in blocks of the cache
            for (int i = 0; i < 4; ++i) quarters |= ((mask >> (i * 16 / box)) & 1) << i;
            sh.valid[su] = (uint8_t)quarters;
          }
          mbar_arrive_expect_tx(&sh.full[su], (uint32_t)(boxes * box * D * 2));
        }
        for (int b = 0; b < boxes; ++b) {
          const int block = __shfl_sync(0xffffffffu, from, b);
          if (elect_one()) {
#pragma unroll
            for (int half = 0; half < kSub; ++half)
              tma_load_3d(dst + half * (kTileKeys * 128) + b * box * 128, keys ? &tk : &tv, &sh.full[su], half * 64, row,
                          block, policy);
          }
        }
        __syncwarp();
        ++issued;
        if (++s == S::kStages) s = 0, phase ^= 1u;
      }
      if (!ok) break;
      u += q.units;
      if (u < u1) q.next(sh.parts, a, L.plan, u, u1);
    }
    // No copy may be in flight when the CTA exits.
    if (lane == 0)
      for (uint32_t i = issued > (uint32_t)S::kStages ? issued - S::kStages : 0; i < issued; ++i)
        mbar_wait_drain(&sh.full[i % S::kStages], (i / S::kStages) & 1, L.err, L.wait_ns);
  } else {
    // ------------------------------------------------------------ products
    const int g = lane >> 2, t4 = lane & 3;
    int s = 0;
    uint32_t phase = 0;
    long long u = u0;
    // Every piece from u on in chunks of `shape`: all that are left, or those of the
    // prefix (which come first); false if a wait gave up.
    auto run = [&](auto shape, auto prefix_only) -> bool {
    using R = decltype(shape);
    constexpr bool kPrefixOnly = decltype(prefix_only)::value;
    auto mine = [&]() { return u < u1 && !q.empty() && (!kPrefixOnly || q.part == 0); };
    constexpr int WK = R::WK;
    constexpr int NK = R::kKeys / 8;       // 8-key columns of S
    constexpr int NE = R::HALF ? 1 : 2;    // this thread's rows
    const int wk = warp % WK, wm = warp / WK;  // which keys of a tile, which 16 rows of a chunk
    // Barriers of the warps that join their sums, apart for the two groupings: a
    // warp may be in its first own piece while others end their last prefix piece.
    // (Pieces of the prefix come first, so the sums' memory changes hands only
    // behind the barrier of all four warps that ends an own piece.)
    const int bar_end = WK == 4 ? 1 : 3 + wm, bar_sums = WK == 4 ? 2 : 5 + wm;
    uint32_t qf[D / 16][4];
    int sees[NE];
    // the keys that this thread's rows (g and g + 8 of the warp's 16) see
    auto look = [&]() {
      const int len = sh.parts.len[q.part], rows = sh.parts.rows[q.part] * group;
#pragma unroll
      for (int e = 0; e < NE; ++e) {
        const int r = q.chunk * R::kRows + wm * 16 + g + 8 * e;
        sees[e] = r >= rows ? 0 : min(len, q.part == 0 ? len : sh.parts.last[q.part] + div_group(r, L.group_mul));
      }
    };
    auto q_row = [&](int r) {  // row r of the part
      const int row = div_group(r, L.group_mul);
      return a.q + (long long)(sh.parts.row0[q.part] + row) * a.ldq + (long long)(q.kvh * group + r - row * group) * D;
    };
    // A piece's queries on their way: to fragments in registers (4 bytes a read),
    // or for 8 rows by one asynchronous 16-byte copy a thread to shared memory,
    // which all four warps read as fragments (fetch_q): 32 reads a thread fewer
    // in every piece.
    auto load_q = [&]() {
      const int rows = sh.parts.rows[q.part] * group;
      if constexpr (R::HALF) {
        if (threadIdx.x < D) {
          const int i = threadIdx.x / (D / 8), v = threadIdx.x % (D / 8), r = q.chunk * 8 + i;
          const bool in = r < rows;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                           smem_u32(s_q + (v >> 3) * 1024) + swz(i, v & 7)),
                       "l"(q_row(in ? r : 0) + v * 8), "r"(in ? 16 : 0)
                       : "memory");
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&sh.qfull)) : "memory");
      } else {
        look();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = q.chunk * R::kRows + wm * 16 + g + 8 * e;
          const bool in = r < rows;
          const uint16_t* src = q_row(in ? r : 0) + 2 * t4;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            qf[i][e] = in ? (uint32_t)ld_act_s32(src + i * 16) : 0u;
            qf[i][e + 2] = in ? (uint32_t)ld_act_s32(src + i * 16 + 8) : 0u;
          }
        }
      }
    };
    uint32_t qphase = 0;
    auto fetch_q = [&]() -> bool {
      if constexpr (R::HALF) {
        look();
        if (!warp_wait(&sh.qfull, qphase, wc)) return false;
        qphase ^= 1u;
#pragma unroll
        for (int i = 0; i < D / 16; i += 2) {
          uint32_t b[4];  // elements 0-7 and 8-15 of steps i and i + 1
          const int cv = 2 * i + (lane >> 3);
          ldsm4(b, smem_u32(s_q + (cv >> 3) * 1024) + swz(lane & 7, cv & 7));
          qf[i][0] = b[0], qf[i][2] = b[1], qf[i][1] = qf[i][3] = 0u;
          qf[i + 1][0] = b[2], qf[i + 1][2] = b[3], qf[i + 1][1] = qf[i + 1][3] = 0u;
        }
      }
      return true;
    };
    if (mine()) load_q();
    while (mine()) {
      const int len = sh.parts.len[q.part], rows = sh.parts.rows[q.part] * group;
      float o[D / 8][4], m[NE], l[NE];
#pragma unroll
      for (int e = 0; e < NE; ++e) m[e] = -INFINITY, l[e] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
      // the fewest keys that any row of the chunk sees
      const int fewest =
          q.part == 0 ? len : min(len, sh.parts.last[q.part] + div_group(q.chunk * R::kRows, L.group_mul));

      const int in_chunk = min(R::kRows, rows - q.chunk * R::kRows);
      bool ok = fetch_q();
      for (int t = q.tile0; ok && t < q.tile1; ++t) {
        ok = warp_wait(&sh.full[s], phase, wc);
        if (!ok) break;
        const uint32_t kb = smem_u32(smem + s * S::kStage), vb = kb + S::kHalf;
        const int valid = sh.valid[s];
        const int key0 = t * kTileKeys + wk * R::kKeys;  // the warp's first key
        const bool edge = key0 + R::kKeys > fewest || valid != 15;
        float p[NK][4];
#pragma unroll
        for (int j = 0; j < NK; ++j) p[j][0] = p[j][1] = p[j][2] = p[j][3] = 0.f;
        if (NK == 2) {
          // few independent sums: even and odd steps apart, half the chain
          float p2[NK][4];
#pragma unroll
          for (int j = 0; j < NK; ++j) p2[j][0] = p2[j][1] = p2[j][2] = p2[j][3] = 0.f;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            uint32_t b[4];
            const int kr = wk * R::kKeys + ((lane >> 4) << 3) + (lane & 7);
            const int cv = i * 2 + ((lane >> 3) & 1);
            ldsm4(b, kb + (cv >> 3) * (kTileKeys * 128) + swz(kr, cv & 7));
            mma16816(i & 1 ? p2[0] : p[0], qf[i], b[0], b[1]);
            mma16816(i & 1 ? p2[NK - 1] : p[NK - 1], qf[i], b[2], b[3]);
          }
#pragma unroll
          for (int j = 0; j < NK; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) p[j][e] += p2[j][e];
        } else {
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int j = 0; j < NK / 2; ++j) {
              // matrices: keys 0-7 and 8-15 by elements 0-7 and 8-15 of step i
              uint32_t b[4];
              const int kr = wk * R::kKeys + j * 16 + ((lane >> 4) << 3) + (lane & 7);
              const int cv = i * 2 + ((lane >> 3) & 1);
              ldsm4(b, kb + (cv >> 3) * (kTileKeys * 128) + swz(kr, cv & 7));
              mma16816(p[2 * j], qf[i], b[0], b[1]);
              mma16816(p[2 * j + 1], qf[i], b[2], b[3]);
            }
        }
        if (edge) {
#pragma unroll
          for (int j = 0; j < NK; ++j)
#pragma unroll
            for (int e = 0; e < 2 * NE; ++e) {
              const int kk = wk * R::kKeys + j * 8 + 2 * t4 + (e & 1);  // key within the tile
              const bool see = t * kTileKeys + kk < sees[e >> 1] && ((valid >> (kk >> 4)) & 1);
              p[j][e] = see ? p[j][e] : -INFINITY;
            }
        }
        // running maximum, shared by the four threads of a row
        float ref[NE], up[NE];
        bool grew = false;
#pragma unroll
        for (int e = 0; e < NE; ++e) {
          float x = -INFINITY;
#pragma unroll
          for (int j = 0; j < NK; ++j) x = fmaxf(x, fmaxf(p[j][2 * e], p[j][2 * e + 1]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
          const float mn = fmaxf(m[e], x);
          grew = grew || mn > m[e];
          ref[e] = mn == -INFINITY ? 0.f : mn;
          up[e] = ex2_from(m[e], ref[e], L.scale_log2);
          m[e] = mn;
        }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int e = 0; e < NE; ++e) {
            l[e] *= up[e];
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
              o[i][2 * e] *= up[e];
              o[i][2 * e + 1] *= up[e];
            }
          }
        }
        uint32_t pf[NK / 2][4];
#pragma unroll
        for (int j = 0; j < NK; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (e >= NE) {
              pf[j >> 1][(j & 1) * 2 + e] = 0u;
              continue;
            }
            const float w0 = ex2((p[j][2 * e] - ref[e % NE]) * L.scale_log2);
            const float w1 = ex2((p[j][2 * e + 1] - ref[e % NE]) * L.scale_log2);
            l[e % NE] += w0 + w1;
            // P is rounded to bf16 for the product with V (fp32 sums; l keeps the unrounded weights)
            pf[j >> 1][(j & 1) * 2 + e] = pack_bf16x2(w0, w1);
          }
        int stop = len;
        if (edge && fewest < len) {
          // Keys that some rows see and others do not. Where one of their V is an
          // infinity or NaN, the product would carry it to the others as 0 * V: these
          // keys are then added row by row.
          const int lo = max(fewest, key0), hi = min(len, key0 + R::kKeys), kr0 = lo - t * kTileKeys;
          bool bad = false;
          for (int i = lane; i < (hi - lo) * (D / 8); i += 32) {
            const int cv = i % (D / 8);
            const uint4 x = *reinterpret_cast<const uint4*>(smem + s * S::kStage + S::kHalf + (cv >> 3) * (kTileKeys * 128) +
                                                            swz(kr0 + i / (D / 8), cv & 7));
            bad = bad || not_finite(x.x) || not_finite(x.y) || not_finite(x.z) || not_finite(x.w);
          }
          if (__any_sync(0xffffffffu, bad)) {
            stop = lo;
#pragma unroll
            for (int j = 0; j < NK; ++j)
#pragma unroll 1
              for (int k = 0; k < 8; ++k) {
                float w[NE];
#pragma unroll
                for (int e = 0; e < NE; ++e) {
                  const uint32_t pair = __shfl_sync(0xffffffffu, pf[j >> 1][(j & 1) * 2 + e], (lane & ~3) | (k >> 1));
                  w[e] = k & 1 ? bf_hi(pair) : bf_lo(pair);
                }
                const int kk = key0 + j * 8 + k;
                if (kk < lo || kk >= hi) continue;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                  const uint32_t x = *reinterpret_cast<const uint32_t*>(
                      smem + s * S::kStage + S::kHalf + (i >> 3) * (kTileKeys * 128) + swz(kk - t * kTileKeys, i & 7) + 4 * t4);
#pragma unroll
                  for (int e = 0; e < NE; ++e)
                    if (kk < sees[e]) {
                      o[i][2 * e] = fmaf(w[e], bf_lo(x), o[i][2 * e]);
                      o[i][2 * e + 1] = fmaf(w[e], bf_hi(x), o[i][2 * e + 1]);
                    }
                }
              }
          }
        }
#pragma unroll
        for (int j = 0; j < NK / 2; ++j) {
          // Keys behind the part's last one hold anything (NaN too): their V is
          // taken as zero, as 0 * NaN would not be.
          uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
          if (edge) {
            const int kk = key0 + j * 16 + 2 * t4;
            keep0 = (kk < stop ? 0xffffu : 0u) | (kk + 1 < stop ? 0xffff0000u : 0u);
            keep1 = (kk + 8 < stop ? 0xffffu : 0u) | (kk + 9 < stop ? 0xffff0000u : 0u);
          }
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            // matrices (transposed): keys 0-7 and 8-15 by elements 0-7 and 8-15 of pair i
            uint32_t b[4];
            const int kr = wk * R::kKeys + j * 16 + (lane & 15);
            const int cv = i * 2 + (lane >> 4);
            ldsm4_t(b, vb + (cv >> 3) * (kTileKeys * 128) + swz(kr, cv & 7));
            if (edge) {
              b[0] &= keep0;
              b[1] &= keep1;
              b[2] &= keep0;
              b[3] &= keep1;
            }
            mma16816(o[2 * i], pf[j], b[0], b[1]);
            mma16816(o[2 * i + 1], pf[j], b[2], b[3]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[s]);
        if (++s == S::kStages) s = 0, phase ^= 1u;
      }
      // The warps that join their sums leave together if a wait gave up; this
      // barrier also ends the reads of the previous piece's sums.
      if (!named_bar_and(bar_end, WK * 32, ok)) return false;

      // ---------------------------------------------------------- the piece's rows
      const Piece done = q;
      u += q.units;
      if (u < u1) {  // the next piece's queries are on their way during what follows
        q.next(sh.parts, a, L.plan, u, u1);
        if (mine()) load_q();
      }
      const bool begins = done.tile0 == 0;
      const bool direct = begins && done.tile1 == done.tiles && a.prefix_len == 0;
      const Pieces& keep = begins ? L.start[done.part > 0] : L.plan.rest;
#pragma unroll
      for (int e = 0; e < NE; ++e) {
        if (wm * 16 + 8 * e >= in_chunk) break;
        const int r = wm * 16 + 8 * e + g;
        float mt = m[e], lt = l[e];
        lt += __shfl_xor_sync(0xffffffffu, lt, 1);
        lt += __shfl_xor_sync(0xffffffffu, lt, 2);
        // warps 1.. of the group hand their sums to warp 0, fragment by fragment
        float2* mine = s_merge + (wm * (WK - 1) + wk - 1) * (D / 8) * 32 + lane;
        if (e > 0) named_bar_sync(bar_end, WK * 32);  // the first half has been read
        if (wk > 0) {
#pragma unroll
          for (int i = 0; i < D / 8; ++i) mine[i * 32] = make_float2(o[i][2 * e], o[i][2 * e + 1]);
          if (t4 == 0) sh.ml[warp][g] = make_float2(mt, lt);
          named_bar_arrive(bar_sums, WK * 32);
          continue;
        }
        named_bar_sync(bar_sums, WK * 32);
        float f[WK], top = mt;
#pragma unroll
        for (int w = 1; w < WK; ++w) top = fmaxf(top, sh.ml[warp + w][g].x);
        f[0] = ex2_from(mt, top, L.scale_log2);
        lt *= f[0];
#pragma unroll
        for (int w = 1; w < WK; ++w) {
          const float2 ml = sh.ml[warp + w][g];
          f[w] = ex2_from(ml.x, top, L.scale_log2);
          lt = fmaf(ml.y, f[w], lt);
        }
        mt = top;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][2 * e] *= f[0];
          o[i][2 * e + 1] *= f[0];
#pragma unroll
          for (int w = 1; w < WK; ++w) {
            const float2 y = s_merge[((wm * (WK - 1) + w - 1) * (D / 8) + i) * 32 + lane];
            o[i][2 * e] = fmaf(y.x, f[w], o[i][2 * e]);
            o[i][2 * e + 1] = fmaf(y.y, f[w], o[i][2 * e + 1]);
          }
        }
        if (r >= in_chunk) continue;
        const int rr = done.chunk * R::kRows + r, row = div_group(rr, L.group_mul);
        const long long t = sh.parts.row0[done.part] + row;
        const int head = done.kvh * group + rr - row * group;
        if (direct) {
          const float inv = lt == 0.f ? 0.f : 1.f / lt;
          uint16_t* to = a.out + t * a.ldo + (long long)head * D + 2 * t4;
#pragma unroll
          for (int i = 0; i < D / 8; ++i)
            *reinterpret_cast<uint32_t*>(to + 8 * i) = pack_bf16x2(o[i][2 * e] * inv, o[i][2 * e + 1] * inv);
        } else {
          const long long at = begins ? t * a.q_heads + head : c * L.plan.rest_rows + r;
          float* to = keep.o + at * D + 2 * t4;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) *reinterpret_cast<float2*>(to + 8 * i) = make_float2(o[i][2 * e], o[i][2 * e + 1]);
          if (t4 == 0) keep.ml[at] = make_float2(mt, lt);
        }
      }
    }
    return true;
    };
    if constexpr (std::is_same<RP, RO>::value) {
      run(RO(), std::false_type());
    } else {
      if (run(RP(), std::true_type())) run(RO(), std::false_type());
    }
    cp_async_wait_all();  // none in flight at exit
  }
  if (L.late_wait) pdl_wait();
}

// Joins the pieces of the rows that more than one CTA, or the prefix and the
// own tokens, gave: out = sum O_i 2^(m_i - m) / sum l_i 2^(m_i - m). A CTA
// takes R rows (of M q_heads), 8 / R warps each, which share a row's pieces:
// what bounds it is the latency of their reads from L2, so few rows take many
// warps each. A row with no piece at all gets zeros. The pieces are summed in
// a fixed order.
template <int D, int R>
__global__ void __launch_bounds__(256, 4) join_attention_kernel(const __grid_constant__ AttentionLaunch P,
                                                             const __grid_constant__ AttentionLaunch O) {
  constexpr int NW = 8 / R, V = D / 32;
  __shared__ PartTable tp, to;
  __shared__ float s_o[8][D];
  __shared__ float2 s_ml[8];
  const AttentionParams& a = O.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = a.group;
  // The launch before this one starts its dependents after its own wait, so
  // the lengths are final here; its pieces are not until pdl_wait().
  if (warp == 0) build_parts(to, O.a, O.plan);
  if (warp == 1) build_parts(tp, P.a, P.plan);
  __syncthreads();
  pdl_trigger();
  const int item = blockIdx.x * R + warp / NW, w = warp % NW;
  const int t = item / a.q_heads, head = item - t * a.q_heads, kvh = div_group(head, O.group_mul);
  int part = 0;
  if (t < a.M) {
    // the request that has row t
    const int n = a.requests;
#pragma unroll
    for (int k = 0; k < (kMaxParts + 31) / 32; ++k) {
      const int i = 1 + k * 32 + lane;
      const bool has = i <= n && t >= to.row0[i] && t < to.row0[i] + to.rows[i];
      const uint32_t hit = __ballot_sync(0xffffffffu, has);
      if (hit) part = 1 + k * 32 + __ffs(hit) - 1;
    }
  }
  // pieces of one part: the starting one, then one for each further CTA
  struct Span {
    long long at;      // row of `start`
    int c0, count, r;  // first CTA, pieces, row within the chunk
  };
  auto span_of = [&](const PartTable& T, const AttentionLaunch& L, int i) {
    Span s{(long long)t * a.q_heads + head, 0, 0, 0};
    const long long W = T.first[a.requests + 1], G = plan_ctas(W, L.plan.ctas);
    const long long tiles = ((long long)T.len[i] + (1 << L.plan.tile_shift) - 1) >> L.plan.tile_shift;
    if (T.first[i + 1] == T.first[i]) return s;
    const int shift = L.plan.row_shift[i > 0];
    const int rr = (t - T.row0[i]) * group + head - kvh * group;
    const int chunk = rr >> shift;
    const long long u = T.first[i] + ((long long)kvh * T.chunks[i] + chunk) * (tiles + L.plan.lead) + L.plan.lead;
    s.r = rr - (chunk << shift);
    s.c0 = cta_of_unit(u, W, G);
    s.count = cta_of_unit(u + tiles - 1, W, G) - s.c0 + 1;
    return s;
  };
  Span sp{0, 0, 0, 0}, so{0, 0, 0, 0};
  int n = part == 0 && t < a.M && a.zero_idle ? 0 : -1;  // pieces; -1: nothing to write
  if (part > 0) {
    if (a.prefix_len > 0) sp = span_of(tp, P, 0);
    so = span_of(to, O, part);
    // a row that one CTA had whole has been written by it
    if (sp.count > 0 || so.count != 1) n = sp.count + so.count;
  }
  pdl_wait();
  float x[V], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) x[e] = 0.f;
  constexpr int B = 6;  // pieces in flight per warp
  for (int i0 = w; i0 < n; i0 += NW * B) {
    float y[B][V];
    float2 ml[B];
#pragma unroll
    for (int k = 0; k < B; ++k) {
      const int i = i0 + NW * k;
      ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int e = 0; e < V; ++e) y[k][e] = 0.f;
      if (i < n) {
        const bool pre = i < sp.count;
        const int j = pre ? i : i - sp.count;
        const Span& s = pre ? sp : so;
        const Pieces& from = j == 0 ? O.start[pre ? 0 : 1] : (pre ? P.plan.rest : O.plan.rest);
        const long long at = j == 0 ? s.at : (long long)(s.c0 + j) * (pre ? P.plan.rest_rows : O.plan.rest_rows) + s.r;
        const uint2 raw = ld_act8(from.ml + at);
        ml[k] = make_float2(__uint_as_float(raw.x), __uint_as_float(raw.y));
        if (V == 4) {
          const float4 f = ld_act_f4(from.o + at * D + lane * 4);
          y[k][0] = f.x, y[k][1 % V] = f.y, y[k][2 % V] = f.z, y[k][3 % V] = f.w;
        } else {
          const uint2 f = ld_act8(from.o + at * D + lane * 2);
          y[k][0] = __uint_as_float(f.x), y[k][1] = __uint_as_float(f.y);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < B; ++k) {
      const float top = fmaxf(m, ml[k].x);
      const float f0 = ex2_from(m, top, O.scale_log2), f1 = ex2_from(ml[k].x, top, O.scale_log2);
      m = top;
      l = l * f0 + ml[k].y * f1;
#pragma unroll
      for (int e = 0; e < V; ++e) x[e] = x[e] * f0 + y[k][e] * f1;
    }
  }
  if (NW > 1) {
#pragma unroll
    for (int e = 0; e < V; ++e) s_o[warp][lane * V + e] = x[e];
    if (lane == 0) s_ml[warp] = make_float2(m, l);
    __syncthreads();
    if (w == 0) {
#pragma unroll
      for (int v = 1; v < NW; ++v) {
        const float2 ml = s_ml[warp + v];
        const float top = fmaxf(m, ml.x);
        const float f0 = ex2_from(m, top, O.scale_log2), f1 = ex2_from(ml.x, top, O.scale_log2);
        m = top;
        l = l * f0 + ml.y * f1;
#pragma unroll
        for (int e = 0; e < V; ++e) x[e] = x[e] * f0 + s_o[warp + v][lane * V + e] * f1;
      }
    }
  }
  if (n < 0 || w > 0) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint32_t* out = reinterpret_cast<uint32_t*>(a.out + (long long)t * a.ldo + (long long)head * D + lane * V);
#pragma unroll
  for (int e = 0; e < V / 2; ++e) out[e] = pack_bf16x2(x[2 * e] * inv, x[2 * e + 1] * inv);
}

// ---------------------------------------------------------------------------- host side
namespace {

int chunk_shift(int rows) { return rows <= 8 ? 3 : rows <= 16 ? 4 : 5; }

struct AttnWs {
  Pieces start[2], rest[2];
  size_t bytes = 0;
};

// Workspace: the starting pieces of the prefix and the own tokens by row and
// head, and one piece per CTA of either launch. Nothing in it needs a value
// before a call.
AttnWs carve(const dec_handle* h, void* base, int M, int q_heads, int dim, int prefix_len) {
  AttnWs w;
  size_t used = 0;
  auto take = [&](size_t bytes) {
    char* p = base ? static_cast<char*>(base) + used : nullptr;
    used += (bytes + 255) & ~size_t(255);
    return p;
  };
  auto pieces = [&](size_t rows) {
    Pieces p;
    p.o = reinterpret_cast<float*>(take(rows * dim * sizeof(float)));
    p.ml = reinterpret_cast<float2*>(take(rows * sizeof(float2)));
    return p;
  };
  for (int i = prefix_len > 0 ? 0 : 1; i < 2; ++i) {
    w.start[i] = pieces((size_t)M * q_heads);
    w.rest[i] = pieces((size_t)h->sms * std::max(kAttnCtasPerSm * Rows32::kRows, 256));
  }
  w.bytes = used;
  return w;
}

bool encode_cache(const dec_handle* h, CUtensorMap* m, const uint16_t* base, const AttentionParams& a) {
  const uint32_t size = 1u << a.shift;
  cuuint64_t dims[3] = {(cuuint64_t)a.dim, (cuuint64_t)a.kv_heads * size, (cuuint64_t)a.blocks};
  cuuint64_t strides[2] = {(cuuint64_t)a.dim * 2, (cuuint64_t)a.block_stride * 2};
  cuuint32_t box[3] = {64, std::min<cuuint32_t>(size, kTileKeys), 1};
  cuuint32_t es[3] = {1, 1, 1};
  return h->encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(base), dims, strides, box, es,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, class RP, class RO>
cudaError_t launch_shape(dec_handle* h, const CUtensorMap& tk, const CUtensorMap& tv, const AttentionLaunch& L,
                         cudaStream_t s) {
  using S = AttnShape<D, RP, RO>;
  static std::atomic<uint64_t> ready{0};  // devices whose function attribute is set
  const uint64_t bit = 1ull << (h->device & 63);
  if (!(ready.load() & bit)) {
    const cudaError_t e =
        cudaFuncSetAttribute(attention_kernel<D, RP, RO>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kTotal);
    if (e != cudaSuccess) return e;
    if (h->device < 64) ready.fetch_or(bit);
  }
  return launch_k(h, attention_kernel<D, RP, RO>, dim3(L.plan.ctas), dim3(kAttnThreads), (size_t)S::kTotal, s, tk, tv, L);
}

// Own chunks RO; the prefix in the same chunks or in those that hold more rows.
template <int D, class RO>
cudaError_t launch_own(dec_handle* h, const CUtensorMap& tk, const CUtensorMap& tv, const AttentionLaunch& L,
                       cudaStream_t s) {
  const int pre = L.plan.prefix ? 1 << L.plan.row_shift[0] : RO::kRows;
  if constexpr (RO::kRows < 16)
    if (pre == 16) return launch_shape<D, Rows16, RO>(h, tk, tv, L, s);
  if constexpr (RO::kRows < 32)
    if (pre == 32) return launch_shape<D, Rows32, RO>(h, tk, tv, L, s);
  return launch_shape<D, RO, RO>(h, tk, tv, L, s);
}

template <int D>
cudaError_t launch_mma(dec_handle* h, const CUtensorMap& tk, const CUtensorMap& tv, const AttentionLaunch& L,
                       cudaStream_t s) {
  switch (1 << L.plan.row_shift[1]) {
    case 8: return launch_own<D, Rows8>(h, tk, tv, L, s);
    case 16: return launch_own<D, Rows16>(h, tk, tv, L, s);
    default: return launch_own<D, Rows32>(h, tk, tv, L, s);
  }
}

cudaError_t launch_chunks(dec_handle* h, const CUtensorMap& tk, const CUtensorMap& tv, const AttentionLaunch& L,
                          cudaStream_t s) {
  if (L.plan.tile_shift == 7) return launch_attention_tc(h, tk, tv, L, s);
  return L.a.dim == 64 ? launch_mma<64>(h, tk, tv, L, s) : launch_mma<128>(h, tk, tv, L, s);
}

// Rows of a joining CTA: 8 (a warp each) from 2432 rows on, where one wave of
// CTAs holds them all, fewer rows and more warps to each below.
template <int D>
cudaError_t launch_join(dec_handle* h, const AttentionLaunch& pre, const AttentionLaunch& own, cudaStream_t s) {
  const int rows = own.a.M * own.a.q_heads, wave = 4 * h->sms;
  if (rows <= wave) return launch_k(h, join_attention_kernel<D, 1>, dim3(rows), dim3(256), 0, s, pre, own);
  if (rows <= 2 * wave) return launch_k(h, join_attention_kernel<D, 2>, dim3((rows + 1) / 2), dim3(256), 0, s, pre, own);
  if (rows <= 4 * wave) return launch_k(h, join_attention_kernel<D, 4>, dim3((rows + 3) / 4), dim3(256), 0, s, pre, own);
  return launch_k(h, join_attention_kernel<D, 8>, dim3((rows + 7) / 8), dim3(256), 0, s, pre, own);
}

}  // namespace

size_t attention_ws_bytes(const dec_handle* h, int M, int q_heads, const dec_kv_cache& cache, const dec_batch& batch) {
  return carve(h, nullptr, M, q_heads, cache.head_dim, batch.prefix_len).bytes;
}

cudaError_t launch_attention(dec_handle* h, const AttentionParams& P, void* ws, cudaStream_t s) {
  const AttnWs w = carve(h, ws, P.M, P.q_heads, P.dim, P.prefix_len);
  CUtensorMap tk, tv;
  if (!encode_cache(h, &tk, P.k, P) || !encode_cache(h, &tv, P.v, P)) return cudaErrorInvalidValue;
  const int group = P.q_heads / P.kv_heads;
  AttentionLaunch own;
  own.a = P;
  own.start[0] = w.start[0];
  own.start[1] = w.start[1];
  own.late_wait = false;
  own.scale_log2 = P.scale * 1.4426950408889634f;
  own.group_mul = (uint32_t)(((1 << 20) + group - 1) / group);
  own.err = h->d_err;
  own.wait_ns = h->wait_ns;
  // Query rows of a key head: of all requests on the prefix, and of one request.
  const int rows_p = P.M * group, rows_o = std::min(P.max_new, P.M) * group;
  const long long prefix_tiles = (long long)P.kv_heads * (((long long)P.prefix_len + 63) / 64);
  // tcgen05 for requests of more than 32 query rows to a key head (4 requests of 16
  // drafts by 4 heads, 16000 tokens each: 96 us, in chunks of 32 rows 162 us; 1000
  // tokens each: 19.3 and 18.3 us), and for a prefix of more than 32 rows and 40
  // 64-key tiles of 32 rows an SM (64 heads on 16, own tokens 500 each, tcgen05
  // against chunks of 32 in one launch with the own tokens: 16 requests, 8192
  // tokens 41 and 36 us, 32768 tokens 72 and 97; 32 requests, 2048 tokens 46 and
  // 39, 8192 tokens 56 and 60; 64 requests, 2048 tokens 72 and 68, 8192 82 and 109).
  const bool tc_own = rows_o > 32;
  const bool tc_prefix =
      P.prefix_len > 0 && rows_p > 32 && (tc_own || prefix_tiles * ((rows_p + 31) / 32) >= 40LL * h->sms);
  auto mma_plan = [&](bool prefix, bool own, const Pieces& rest) {
    Plan p{prefix, own, {chunk_shift(std::max(rows_o, rows_p)), chunk_shift(rows_o)}, 0, kPieceLead, 6,
           h->sms * kAttnCtasPerSm, rest};
    p.rest_rows = 1 << p.row_shift[!prefix];
    return p;
  };
  auto tc_plan = [&](bool prefix, bool own, const Pieces& rest) {
    const int shift = (prefix ? rows_p : rows_o) <= 128 ? 7 : 8;
    return Plan{prefix, own, {shift, shift}, 1 << shift, kPieceLeadTc, 7, h->sms, rest};
  };
  AttentionLaunch pre = own;
  cudaError_t e = cudaSuccess;
  const bool apart = tc_prefix && !tc_own;  // a launch for the prefix, one for the own tokens
  own.plan = tc_own ? tc_plan(P.prefix_len > 0, true, w.rest[1]) : mma_plan(P.prefix_len > 0 && !apart, true, w.rest[1]);
  pre.plan = own.plan;
  if (apart) {
    pre.plan = tc_plan(true, false, w.rest[0]);
    LaunchScope scope(h, "attention_prefix", s);
    e = launch_chunks(h, tk, tv, pre, s);
    if (e != cudaSuccess) return e;
    own.late_wait = true;
  }
  {
    LaunchScope scope(h, "attention", s);
    e = launch_chunks(h, tk, tv, own, s);
    if (e != cudaSuccess) return e;
  }
  LaunchScope scope(h, "attention_join", s);
  return P.dim == 64 ? launch_join<64>(h, pre, own, s) : launch_join<128>(h, pre, own, s);
}

}  // namespace dec
