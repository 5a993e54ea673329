// Attention for many query rows to a key head (a batch on a shared prefix, long
// runs of new tokens): the products on tcgen05.
//
// 64 rows of 4 heads on one prefix are 256 flops to a byte of the cache, near
// the ridge of the tensor cores (280), where mma.sync stops at a third of
// their rate. A CTA holds 128 or 256 query rows and streams 128-key tiles;
// each 128 rows are one stream of
//   S = Q K^T (128 x 128, fp32 in TMEM)           tcgen05.mma, Q and K in shared memory
//   P = 2^(S - m), bf16, over S in TMEM            a thread per row: no shuffles
//   O += P V (128 x D, fp32 in TMEM)               tcgen05.mma, P from TMEM, V in shared memory
// One warp issues the products. With two streams (all of TMEM) it takes them in
// turn, so that one's products run under the other one's exponentials; with a
// warp per stream the two fell into step and took turns as a pair (64 requests
// on 32768 shared tokens: 147 and 124 us). One stream has two buffers of S, and
// the next tile's scores are there when a softmax ends. (64-key tiles with two
// buffers for both streams: 113 us where this takes 93; a product of 64 columns
// reads as much of Q as one of 128.) The running maximum is raised only when a
// row's scores pass it by more than 2^8 (P <= 256 then, exact in fp32 sums), so O
// is read and rescaled a few times, not every tile. K is a K-major operand as it
// lies in the cache, V an MN-major one: both come by TMA with the 128-byte
// swizzle, in separate rings that two warps fill. With two streams of head dim 128
// a tile costs 1.71 us (32768 more tokens of the prefix: 46 us more) where its
// read takes 1.47; the softmax is most of the difference (without one, 0.2 us a
// tile less), and the rings' three K and two V tiles are enough (two and two: the
// same times). What remains of a call's 96 us with 64 rows of 64 heads on 32768
// shared tokens is the ramp and the way out, the own tokens' launch and the join.
#include <atomic>

#include "attention.cuh"

namespace dec {

namespace {

constexpr int kTcTile = 128;
constexpr int kTcThreads = 384;  // warps 0-7 softmax (4 a stream), 8 copies K, 9 copies V, 10 issues products
constexpr int kTcSmem = 232448;
constexpr float kRaise = 8.f;    // log2 of the growth of the weights that is left in P

template <int D, int NT>
struct TcShape {
  static constexpr int kTileBytes = kTcTile * D * 2;       // K or V of a tile; also 128 query rows
  static constexpr int kQ = NT * kTileBytes;
  static constexpr int kFixed = 1024 + 2048;
  static constexpr int kSlots = (kTcSmem - kFixed - kQ) / kTileBytes;
  static constexpr int kK = kSlots >= 12 ? 6 : (kSlots + 1) / 2, kV = kSlots >= 12 ? 6 : kSlots / 2;
  static constexpr int kTotal = (kK + kV) * kTileBytes + kQ + kFixed;
  static_assert(kK >= 2 && kV >= 2 && kTotal <= kTcSmem, "shared memory");
  // TMEM columns: S (P over it) in kBuf buffers and O of each stream
  static constexpr uint32_t kBuf = NT == 1 ? 2 : 1;
  static constexpr uint32_t kO = 256;
  static constexpr uint32_t kCols = 512;
  __device__ static constexpr uint32_t s_col(uint32_t j, uint32_t b) { return (j * kBuf + b) * 128; }
  // buffer of the c-th tile, and the parity of its barriers' phase
  __device__ static constexpr uint32_t buf(uint32_t c) { return kBuf == 2 ? c & 1 : 0; }
  __device__ static constexpr uint32_t phase(uint32_t c) { return kBuf == 2 ? (c >> 1) & 1 : c & 1; }
};

struct TcShared {
  uint64_t kfull[6], kempty[6], vfull[6], vempty[6];
  uint64_t sfull[2][2], pfull[2][2], pvdone[2], qfull, done;  // [stream][buffer], [stream]
  PartTable parts;
  uint8_t valid[16];  // per tile (modulo 16): which 16-key eighths lie in blocks of the cache
  uint32_t tmem;
  uint32_t bad;  // 1 + the first tile (of all of the CTA's) of the last piece with a V to be added at its end
  int abort;
};
static_assert(sizeof(TcShared) <= 2048, "attention tables");

// Descriptor of an MN-major operand with the 128-byte swizzle: rows (one k
// each) of 64 contiguous elements, 8-row groups 1024 bytes apart (SBO), the
// next 64 elements lbo bytes on.
__device__ __forceinline__ uint64_t sw128_mn_desc(uint32_t smem_addr, uint32_t lbo) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(lbo >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// D[tmem] (+)= A[tmem] * B[smem], issued by one thread.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

#define DEC_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), \
                     "=r"(r[i + 6]), "=r"(r[i + 7])
#define DEC_W8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), \
                     "r"(r[i + 6]), "r"(r[i + 7])

// 32 consecutive columns of this thread's TMEM lane. The values may be used
// behind tmem_wait_ld(), which takes them so that no use moves above it.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : DEC_R8(r, 0), DEC_R8(r, 8), DEC_R8(r, 16), DEC_R8(r, 24)
      : "r"(taddr)
      : "memory");
}
#define DEC_RW8(r, i) "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]), \
                      "+r"(r[i + 6]), "+r"(r[i + 7])
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&x)[32], uint32_t (&y)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  asm volatile("" : DEC_RW8(x, 0), DEC_RW8(x, 8), DEC_RW8(x, 16), DEC_RW8(x, 24));
  asm volatile("" : DEC_RW8(y, 0), DEC_RW8(y, 8), DEC_RW8(y, 16), DEC_RW8(y, 24));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::DEC_W8(
          r, 0),
      DEC_W8(r, 8), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two fp32 values in one 64-bit register, and operations on both at once.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}

template <int D, int NT>
__global__ void __launch_bounds__(kTcThreads, 1)
    attention_tc_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                        const __grid_constant__ AttentionLaunch L) {
  using S = TcShape<D, NT>;
  constexpr int kRows = NT * 128, kSub = D / 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_q = smem;                                  // [NT][kSub][128 rows][128 bytes], swizzled
  uint8_t* s_k = smem + S::kQ;                          // [kK][kSub][128 keys][128 bytes]
  uint8_t* s_v = s_k + S::kK * S::kTileBytes;           // [kV][the same]
  TcShared& sh = *reinterpret_cast<TcShared*>(s_v + S::kV * S::kTileBytes);
  const AttentionParams& a = L.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = a.group;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 6; ++i) {
      mbar_init(&sh.kfull[i], 1);
      mbar_init(&sh.vfull[i], 1);
      mbar_init(&sh.kempty[i], 1);
      mbar_init(&sh.vempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(&sh.sfull[i][b], 1);
        mbar_init(&sh.pfull[i][b], 128);
      }
      mbar_init(&sh.pvdone[i], 1);
    }
    mbar_init(&sh.done, 1);
    mbar_init(&sh.qfull, kRows);
    sh.abort = 0;
    sh.bad = 0;
    fence_mbar_init();
    tmap_prefetch(&tk);
    tmap_prefetch(&tv);
  }
  if (warp == 11) {
    tmem_alloc(&sh.tmem, S::kCols);
    tmem_relinquish();
  }
  warm_l2(a);
  pdl_wait();
  pdl_trigger();  // after the wait: see the joining kernel and the launch of the own tokens
  if (warp == 0) build_parts(sh.parts, a, L.plan);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)sh.tmem);
  const long long W = sh.parts.first[a.requests + 1], G = plan_ctas(W, L.plan.ctas), c = blockIdx.x;
  const long long u0 = c < G ? unit_start(c, W, G) : 0, u1 = c < G ? unit_start(c + 1, W, G) : 0;
  const WaitCtl wc{&sh.abort, L.err, L.wait_ns};
  Piece q;
  if (u0 < u1) q.begin(sh.parts, a, L.plan, u0, u1);

  if (warp == 8 || warp == 9) {
    // ------------------------------------------------------------ copies
    const bool keys = warp == 8;
    uint64_t* full = keys ? sh.kfull : sh.vfull;
    uint64_t* empty = keys ? sh.kempty : sh.vempty;
    uint8_t* ring = keys ? s_k : s_v;
    const int slots = keys ? S::kK : S::kV;
    const int box = min(1 << a.shift, 64);  // keys of one box
    const int per = kTcTile / box;
    const uint64_t first = policy_evict_first(), normal = policy_evict_normal();
    uint32_t issued = 0;
    int s = 0;
    uint32_t phase = 1;
    for (long long u = u0; u < u1 && !q.empty();) {
      const int len = sh.parts.len[q.part];
      const int32_t* table = q.part == 0 ? a.prefix_table : a.block_table + (long long)(q.part - 1) * a.max_blocks;
      const uint64_t policy = q.chunks == 1 ? first : normal;
      BlockIds ids(table, (int)(((long long)len + (1 << a.shift) - 1) >> a.shift));
      bool ok = true;
      for (int t = q.tile0; t < q.tile1; ++t) {
        const int key0 = t * kTcTile;
        const int boxes = min(per, (len - key0 + box - 1) / box);
        ids.advance(key0 >> a.shift);
        // lane b < per: the cache block of box b, a.blocks if it is not there
        const int id = ids.get((key0 + min(lane, per - 1) * box) >> a.shift);
        const bool there = lane < boxes && id >= 0 && id < a.blocks;
        const uint32_t mask = __ballot_sync(0xffffffffu, there);
        const int from = there ? id : a.blocks;  // past the end of the cache: reads zeros
        ok = warp_wait(&empty[s], phase, wc);
        if (!ok) break;
        const int su = uniform(s);
        uint8_t* dst = ring + su * S::kTileBytes;
        const int row = uniform((q.kvh << a.shift) + (key0 & ((1 << a.shift) - 1)));
        if (elect_one()) {
          if (keys) {
            int eighths = 0;
            for (int i = 0; i < 8; ++i) eighths |= ((mask >> (i * 16 / box)) & 1) << i;
            sh.valid[issued & 15] = (uint8_t)eighths;
          }
          mbar_arrive_expect_tx(&full[su], (uint32_t)(boxes * box * D * 2));
        }
        for (int b = 0; b < boxes; ++b) {
          const int block = __shfl_sync(0xffffffffu, from, b);
          // a 128-token block is two boxes
          const int at = a.shift == 7 ? row + b * 64 : row;
          if (elect_one()) {
#pragma unroll
            for (int half = 0; half < kSub; ++half)
              tma_load_3d(dst + half * (kTcTile * 128) + b * box * 128, keys ? &tk : &tv, &full[su], half * 64, at, block,
                          policy);
          }
        }
        __syncwarp();
        ++issued;
        if (++s == slots) s = 0, phase ^= 1u;
      }
      if (!ok) break;
      u += q.units;
      if (u < u1) q.next(sh.parts, a, L.plan, u, u1);
    }
    if (lane == 0)
      for (uint32_t i = issued > (uint32_t)slots ? issued - slots : 0; i < issued; ++i)
        mbar_wait_drain(&full[i % slots], (i / slots) & 1, L.err, L.wait_ns);
  } else if (warp >= 8) {
    // ------------------------------------------------------------ products
    if (warp == 10) {
      int ks = 0, vs = 0;
      uint32_t kph = 0, vph = 0, qph = 0;
      uint32_t n = 0;  // tiles so far
      constexpr uint32_t idesc_s = umma_idesc_bf16(128, kTcTile);
      constexpr uint32_t idesc_o = umma_idesc_bf16(128, D) | (1u << 16);  // B is MN-major
      auto issue_s = [&](int j, int slot, uint32_t tile) {
        const int su = uniform(slot), b = uniform((int)S::buf(tile));
        const uint64_t qd = sw128_desc(smem_u32(s_q) + j * S::kTileBytes);
        const uint64_t kd = sw128_desc(smem_u32(s_k) + su * S::kTileBytes);
        const uint32_t ts = tmem + S::s_col(j, b);
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const uint64_t off = ((i >> 2) * (kTcTile * 128) + (i & 3) * 32) >> 4;  // the descriptors' address unit
            umma_bf16(ts, qd + off, kd + off, idesc_s, i > 0);
          }
          umma_commit(&sh.sfull[j][b]);
          if (j == NT - 1) umma_commit(&sh.kempty[su]);
        }
        __syncwarp();
      };
      bool ok = true;
      for (long long u = u0; ok && u < u1 && !q.empty();) {
        // the queries are there, and O has been read; the first tile's scores
        ok = warp_wait(&sh.qfull, qph, wc) && warp_wait(&sh.kfull[ks], kph, wc);
        if (!ok) break;
        qph ^= 1u;
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < NT; ++j) issue_s(j, ks, n);
        if (++ks == S::kK) ks = 0, kph ^= 1u;
        for (int t = q.tile0; ok && t < q.tile1; ++t, ++n) {
          const bool more = t + 1 < q.tile1;
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            if (!ok) break;
            // The next tile's scores go where P of kBuf - 1 tiles ago is: only once it
            // has been multiplied (before a piece's first tile, all have been).
            auto next_scores = [&](bool wait, uint32_t after) {
              ok = (j > 0 || warp_wait(&sh.kfull[ks], kph, wc)) && (!wait || warp_wait(&sh.pvdone[j], after & 1, wc));
              if (!ok) return;
              tc_fence_after();
              issue_s(j, ks, n + 1);
            };
            if (S::kBuf == 2 && more) next_scores(t > q.tile0, n - 1);
            ok = ok && warp_wait(&sh.pfull[j][S::buf(n)], S::phase(n), wc) && (j > 0 || warp_wait(&sh.vfull[vs], vph, wc));
            if (!ok) break;
            tc_fence_after();
            const int su = uniform(vs);
            const uint64_t vd = sw128_mn_desc(smem_u32(s_v) + su * S::kTileBytes, kTcTile * 128);
            const uint32_t ts = tmem + S::s_col(j, uniform((int)S::buf(n))), to = tmem + S::kO + j * D;
            const uint32_t first = uniform(t > q.tile0);
            if (elect_one()) {
#pragma unroll
              for (int i = 0; i < kTcTile / 16; ++i)
                umma_bf16_ts(to, ts + i * 8, vd + i * (2048 >> 4), idesc_o, i > 0 ? 1u : first);
              umma_commit(&sh.pvdone[j]);
              if (j == NT - 1) umma_commit(&sh.vempty[su]);
            }
            __syncwarp();
            if (S::kBuf == 1 && more) next_scores(true, n);
          }
          if (more && ++ks == S::kK) ks = 0, kph ^= 1u;
          if (++vs == S::kV) vs = 0, vph ^= 1u;
        }
        u += q.units;
        if (u < u1) q.next(sh.parts, a, L.plan, u, u1);
      }
      // every product issued must be complete before TMEM is released
      __syncwarp();
      if (elect_one()) {
        umma_commit(&sh.done);
        mbar_wait_drain(&sh.done, 0, L.err, L.wait_ns);
      }
      __syncwarp();
    }
  } else if (warp / 4 < NT) {
    // ------------------------------------------------------------ softmax of stream j, one thread a row
    const int j = warp >> 2, r = threadIdx.x;  // row of the chunk
    const int rj = r & 127;
    const uint32_t quarter = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t to = tmem + S::kO + j * D + quarter;
    uint32_t n = 0;  // tiles so far
    int vs = 0;
    uint32_t vph = 0;
    int sees = 0;
    const float room = kRaise / L.scale_log2;  // above the maximum, in scores
    // The stream's 128 query rows into shared memory (16 bytes a thread, rows
    // contiguous over lanes, every load before any store), and the keys that
    // this thread's row sees.
    auto load_q = [&]() {
      const int rows = sh.parts.rows[q.part] * group, len = sh.parts.len[q.part], r0 = q.chunk * kRows;
      const int mine = r0 + r;
      sees = mine < rows ? min(len, q.part == 0 ? len : sh.parts.last[q.part] + div_group(mine, L.group_mul)) : 0;
      constexpr int kVec = D / 8;  // 16-byte vectors of a row; 128 / kVec rows a step
#pragma unroll
      for (int h = 0; h < kVec; h += 8) {
        uint4 x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int at = (h + k) * 128 + rj, rr = r0 + j * 128 + at / kVec;
          const bool in = rr < rows;
          const int row = in ? div_group(rr, L.group_mul) : 0;
          x[k] = make_uint4(0u, 0u, 0u, 0u);
          if (in)
            x[k] = ld_act16(a.q + (long long)(sh.parts.row0[q.part] + row) * a.ldq +
                            (long long)(q.kvh * group + rr - row * group) * D + (at % kVec) * 8);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int at = (h + k) * 128 + rj, qr = at / kVec, v = at % kVec;
          *reinterpret_cast<uint4*>(s_q + j * S::kTileBytes + (v >> 3) * (128 * 128) + qr * 128 +
                                    (((v & 7) ^ (qr & 7)) << 4)) = x[k];
        }
      }
      fence_async_smem();
      tc_fence_before();
      mbar_arrive(&sh.qfull);
    };
    if (u0 < u1 && !q.empty()) load_q();
    bool ok = true;
    for (long long u = u0; ok && u < u1 && !q.empty();) {
      const int len = sh.parts.len[q.part], rows = sh.parts.rows[q.part] * group;
      // the fewest keys that any row of the chunk sees
      const int fewest =
          q.part == 0 ? len : min(len, sh.parts.last[q.part] + div_group(q.chunk * kRows, L.group_mul));
      float m = -INFINITY, l = 0.f;
      const uint32_t id = n + 1;  // of the piece
      for (int t = q.tile0; t < q.tile1; ++t, ++n) {
        const uint32_t ts = tmem + S::s_col(j, S::buf(n)) + quarter;
        ok = warp_wait(&sh.sfull[j][S::buf(n)], S::phase(n), wc);
        if (!ok) break;
        tc_fence_after();
        const int key0 = t * kTcTile;
        const int valid = sh.valid[n & 15];
        const bool edge = key0 + kTcTile > fewest || valid != 255;
        const int see = sees - key0;  // columns of the tile that the row sees
        if (edge) {
          // Scores that the row does not see become -inf in TMEM (one pass apart, so
          // that the code of all other tiles stays short).
#pragma unroll 1
          for (int h = 0; h < 8; ++h) {
            float x[16];
            uint32_t y[16];
            tmem_ld16(ts + h * 16, x);
            const bool there = (valid >> h) & 1;
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = there && h * 16 + i < see ? __float_as_uint(x[i]) : 0xff800000u;
            tmem_st16(ts + h * 16, y);
          }
          tmem_wait_st();
        }
        // Columns 64.. first, then 0..63, which stay in registers; 64.. are read
        // again while those are worked on (128 scores and their weights would not
        // fit the registers). P lies over the columns already used.
        auto largest = [&](const uint32_t (&x)[32]) {
          float t0 = __uint_as_float(x[0]), t1 = __uint_as_float(x[1]);
#pragma unroll
          for (int i = 2; i < 32; i += 2) {
            t0 = fmaxf(t0, __uint_as_float(x[i]));
            t1 = fmaxf(t1, __uint_as_float(x[i + 1]));
          }
          return fmaxf(t0, t1);
        };
        uint32_t x0[32], x1[32], x2[32];
        tmem_ld32_async(ts + 64, x0);
        tmem_ld32_async(ts + 96, x1);
        tmem_wait_ld(x0, x1);
        float top = fmaxf(largest(x0), largest(x1));
        tmem_ld32_async(ts, x0);
        tmem_ld32_async(ts + 32, x1);
        tmem_wait_ld(x0, x1);
        top = fmaxf(top, fmaxf(largest(x0), largest(x1)));
        const bool raise = top > m + room || (m == -INFINITY && top > -INFINITY);
        if (__any_sync(0xffffffffu, raise)) {
          const float f = raise ? ex2_from(m, top, L.scale_log2) : 1.f;
          if (raise) m = top;
          l *= f;
          if (t > q.tile0) {
            // O is still until this tile's P is there, once the tile before is added
            // (the one before that is: these scores were issued behind it)
            ok = warp_wait(&sh.pvdone[j], (n - 1) & 1, wc);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int h = 0; h < D / 16; ++h) {
              float o[16];
              tmem_ld16(to + h * 16, o);
              uint32_t y[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(o[i] * f);
              tmem_st16(to + h * 16, y);
            }
          }
        }
        const float ref = m == -INFINITY ? 0.f : m;
        const uint64_t less = pair(-ref, -ref), scale = pair(L.scale_log2, L.scale_log2);
        uint64_t sum = 0;  // of even and odd columns
        auto weigh = [&](const uint32_t (&x)[32], int h) {
          uint32_t p[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint64_t s2 = pair(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
            const float2 e = unpair(mul2(add2(s2, less), scale));
            // P is rounded to bf16 for the product with V; l sums the rounded weights too:
            // with the maximum left behind by up to 2^8, the weight of a key that dominates
            // is no power of two, and its rounding cancels only so
            p[i] = pack_bf16x2(ex2(e.x), ex2(e.y));
            sum = add2(sum, pair(bf_lo(p[i]), bf_hi(p[i])));
          }
          tmem_st16(ts + h * 16, p);
        };
        tmem_ld32_async(ts + 64, x2);
        weigh(x0, 0);
        tmem_wait_ld(x2, x1);
        tmem_ld32_async(ts + 96, x0);
        weigh(x1, 1);
        weigh(x2, 2);
        tmem_wait_ld(x0, x1);
        weigh(x0, 3);
        const float2 both = unpair(sum);
        l += both.x + both.y;
        if (key0 + kTcTile > fewest) {
          // Keys behind the part's last one hold anything (NaN too): their V is
          // made zero, as 0 * NaN would not be. Keys that some rows see and others
          // do not carry an infinity or NaN to the others the same way: those
          // elements are made zero too, and added at the end of the piece. (Both
          // streams do this to the same tile, the one behind may find it done.)
          ok = warp_wait(&sh.vfull[vs], vph, wc);
          if (!ok) break;
          const int from = max(fewest - key0, 0);
          for (int i = rj; i < (kTcTile - from) * kSub * 8; i += 128) {
            const int key = from + i / (kSub * 8), h = (i >> 3) % kSub, v = i & 7;
            uint4* at = reinterpret_cast<uint4*>(s_v + vs * S::kTileBytes + h * (kTcTile * 128) + key * 128 + v * 16);
            if (key0 + key >= len) {
              *at = make_uint4(0u, 0u, 0u, 0u);
              continue;
            }
            const uint4 x = *at;
            if (not_finite(x.x) || not_finite(x.y) || not_finite(x.z) || not_finite(x.w)) {
              *const_cast<volatile uint32_t*>(&sh.bad) = id;
              __threadfence_block();
              *at = make_uint4(finite_of(x.x), finite_of(x.y), finite_of(x.z), finite_of(x.w));
            }
          }
          fence_async_smem();
        }
        if (++vs == S::kV) vs = 0, vph ^= 1u;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&sh.pfull[j][S::buf(n)]);
      }
      // The last product of the piece. With two buffers the one before it may still
      // be under way, and a wait for a phase's parity passes while the phase before
      // is open: that one first. The stream's warps leave together if a wait gave up.
      if (ok && S::kBuf == 2 && q.tile1 - q.tile0 > 1) ok = warp_wait(&sh.pvdone[j], n & 1, wc);
      if (ok) ok = warp_wait(&sh.pvdone[j], (n - 1) & 1, wc);
      ok = named_bar_and(1 + j, 128, ok);
      if (!ok) break;
      tc_fence_after();
      if (*const_cast<volatile uint32_t*>(&sh.bad) == id) {
        // The infinities and NaN that were left out, from the cache, to the rows that
        // see them (their weight would not change them).
        const int32_t* table = a.block_table + (long long)(q.part - 1) * a.max_blocks;  // the prefix has no such keys
        for (int key = max(fewest, q.tile0 * kTcTile); key < min(len, q.tile1 * kTcTile); ++key) {
          const int block = ld_act_s32(table + (key >> a.shift));
          if (block < 0 || block >= a.blocks) continue;
          const uint16_t* v = a.v + block * a.block_stride +
                              (long long)((q.kvh << a.shift) + (key & ((1 << a.shift) - 1))) * D;
#pragma unroll 1
          for (int h = 0; h < D / 16; ++h) {
            float o[16];
            tmem_ld16(to + h * 16, o);
            uint32_t y[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint32_t x = (uint32_t)v[h * 16 + i];
              const float f = not_finite(x) && key < sees ? __uint_as_float(x << 16) : 0.f;
              y[i] = __float_as_uint(o[i] + f);
            }
            tmem_st16(to + h * 16, y);
          }
          tmem_wait_st();
        }
      }
      const Piece done = q;
      const bool begins = done.tile0 == 0;
      const bool direct = begins && done.tile1 == done.tiles && a.prefix_len == 0;
      const Pieces& keep = begins ? L.start[done.part > 0] : L.plan.rest;
      // O leaves through the stream's query rows (every product that read them is
      // complete), 64 columns at a time, so that a row's 256 bytes are written by 16
      // neighbouring threads: from the threads that hold the rows, each store
      // touched 32 rows and the piece took 4 us. 16-byte vector v of row i lies at
      // v ^ (i & 15).
      uint8_t* stage = s_q + j * S::kTileBytes;
      constexpr int kPass = D == 64 ? 32 : 64;  // columns that fit 128 rows of fp32
      const float inv = direct ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
      constexpr int kV = kPass / 4;
      const int r0 = done.chunk * kRows + j * 128;
#pragma unroll 1
      for (int h = 0; h < D / kPass; ++h) {
#pragma unroll
        for (int w = 0; w < kPass / 16; ++w) {
          float x[16];
          tmem_ld16(to + h * kPass + w * 16, x);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float4*>(stage + rj * (kPass * 4) + (((w * 4 + i) ^ (rj & (kV - 1))) << 4)) =
                make_float4(x[4 * i] * inv, x[4 * i + 1] * inv, x[4 * i + 2] * inv, x[4 * i + 3] * inv);
        }
        named_bar_sync(1 + j, 128);
#pragma unroll 4
        for (int k = 0; k < kV; ++k) {
          const int at = k * 128 + rj, i = at / kV, v = at % kV, rr = r0 + i;
          if (rr < rows) {
            const float4 x = *reinterpret_cast<const float4*>(stage + i * (kPass * 4) + ((v ^ (i & (kV - 1))) << 4));
            const int row = div_group(rr, L.group_mul);
            const long long t = sh.parts.row0[done.part] + row;
            const int head = done.kvh * group + rr - row * group;
            if (direct)
              *reinterpret_cast<uint2*>(a.out + t * a.ldo + (long long)head * D + h * kPass + v * 4) =
                  make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
            else
              *reinterpret_cast<float4*>(keep.o + (begins ? t * a.q_heads + head : c * kRows + j * 128 + i) * D +
                                         h * kPass + v * 4) = x;
          }
        }
        named_bar_sync(1 + j, 128);
      }
      const int rr = done.chunk * kRows + r;
      if (rr < rows && !direct) {
        const int row = div_group(rr, L.group_mul);
        const long long at = begins ? (long long)(sh.parts.row0[done.part] + row) * a.q_heads + done.kvh * group + rr - row * group
                                    : c * kRows + r;
        keep.ml[at] = make_float2(m, l);
      }
      u += q.units;
      if (u < u1) {
        q.next(sh.parts, a, L.plan, u, u1);
        if (!q.empty()) load_q();
      }
    }
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 11) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kCols);
  }
}

template <int D, int NT>
cudaError_t launch_shape(dec_handle* h, const CUtensorMap& tk, const CUtensorMap& tv, const AttentionLaunch& L,
                         cudaStream_t s) {
  using S = TcShape<D, NT>;
  static std::atomic<uint64_t> ready{0};  // devices whose function attribute is set
  const uint64_t bit = 1ull << (h->device & 63);
  if (!(ready.load() & bit)) {
    const cudaError_t e =
        cudaFuncSetAttribute(attention_tc_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kTotal);
    if (e != cudaSuccess) return e;
    if (h->device < 64) ready.fetch_or(bit);
  }
  return launch_k(h, attention_tc_kernel<D, NT>, dim3(L.plan.ctas), dim3(kTcThreads), (size_t)S::kTotal, s, tk, tv, L);
}

}  // namespace

cudaError_t launch_attention_tc(dec_handle* h, const CUtensorMap& tk, const CUtensorMap& tv, const AttentionLaunch& L,
                                cudaStream_t s) {
  const bool two = L.plan.rest_rows > 128;
  if (L.a.dim == 64) return two ? launch_shape<64, 2>(h, tk, tv, L, s) : launch_shape<64, 1>(h, tk, tv, L, s);
  return two ? launch_shape<128, 2>(h, tk, tv, L, s) : launch_shape<128, 1>(h, tk, tv, L, s);
}

}  // namespace dec
