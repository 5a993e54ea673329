// Attention of a decode step over the paged cache.
//
// One pass over the keys with a running maximum and sum per row: for a tile of
// 64 keys, S = Q K^T, m' = max(m, max S), O = O 2^(m - m') + P V with
// P = 2^(S - m'), l = l 2^(m - m') + sum P, the scale and log2 e folded into
// one factor on S. What bounds it is the read of the cache: 4 query rows to a
// key row make 4 flops a byte. The cache therefore streams through a ring of
// TMA copies (one box per block and 64 elements, 128-byte swizzle) that one
// warp keeps full, while four warps multiply with mma.sync m16n8k16, whose
// fragments come from the ring by ldmatrix without bank conflicts. Each CTA
// streams one equal share of all tiles (attention.cuh); rows that several CTAs
// took are joined by the combine kernel.
#include <algorithm>
#include <atomic>

#include "attention.cuh"

namespace dec {

constexpr int kAttnThreads = 160;  // 4 multiplying warps, 1 copying warp
constexpr int kAttnSmem = 232448;

// WK warps share a tile's keys, 4 / WK groups of 16 rows share its rows.
template <int D, int WK>
struct AttnShape {
  static constexpr int kWM = 4 / WK;
  static constexpr int kRows = 16 * kWM;
  static constexpr int kKeys = kTileKeys / WK;             // keys of one warp
  static constexpr int kHalf = kTileKeys * D * 2;          // K or V bytes of a stage
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kMerge = WK > 1 ? 4 * 16 * D * 4 : 0;  // the warps' sums, joined at the end of a piece
  static constexpr int kFixed = 1024 + 2048;               // alignment, barriers and tables
  static constexpr int kStages = std::min(12, (kAttnSmem - kFixed - kMerge) / kStage);
  static constexpr int kTotal = kStages * kStage + kMerge + kFixed;
  static_assert(kStages >= 3 && kTotal <= kAttnSmem, "shared memory");
};

struct AttnShared {
  uint64_t full[12], empty[12];
  PartTable parts;
  float2 ml[4][16];
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

template <int D, int WK>
__global__ void __launch_bounds__(kAttnThreads, 1)
    attention_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                     const AttentionLaunch L) {
  using S = AttnShape<D, WK>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* s_merge = reinterpret_cast<float*>(smem + S::kStages * S::kStage);  // [4][16][D], column ^ 8 (row % 8)
  AttnShared& sh = *reinterpret_cast<AttnShared*>(smem + S::kStages * S::kStage + S::kMerge);
  const AttentionParams& a = L.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = a.q_heads / a.kv_heads;

  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 4);
    }
    sh.abort = 0;
    fence_mbar_init();
    tmap_prefetch(&tk);
    tmap_prefetch(&tv);
  }
  pdl_wait();
  if (warp == 0) build_parts(sh.parts, a, L.plan);
  __syncthreads();
  const long long W = sh.parts.first[a.requests + 1], G = plan_ctas(W, L.plan.ctas), c = blockIdx.x;
  const long long u0 = c < G ? unit_start(c, W, G) : 0, u1 = c < G ? unit_start(c + 1, W, G) : 0;
  const WaitCtl wc{&sh.abort, L.err, L.wait_ns};

  if (warp == 4) {
    // ------------------------------------------------------------ copies
    const int box = min(1 << a.shift, kTileKeys);  // keys of one box
    const int per = kTileKeys / box;               // boxes (blocks) of a tile
    constexpr int kSub = D / 64;
    long long issued = 0;
    int part = 0;
    bool ok = true;
    for (long long u = u0; ok && u < u1;) {
      const Piece q = piece_at(sh.parts, a, L.plan, u, u1, part);
      u += q.tile1 - q.tile0;
      const int len = sh.parts.len[part];
      const int32_t* table = part == 0 ? a.prefix_table : a.block_table + (long long)(part - 1) * a.max_blocks;
      BlockIds ids(table, (int)(((long long)len + (1 << a.shift) - 1) >> a.shift));
      for (int t = q.tile0; t < q.tile1; ++t, ++issued) {
        const int s = (int)(issued % S::kStages);
        ok = __all_sync(0xffffffffu, mbar_wait(&sh.empty[s], (uint32_t)((issued / S::kStages) & 1) ^ 1u, wc));
        if (!ok) break;
        const int key0 = t * kTileKeys;
        const int boxes = min(per, (len - key0 + box - 1) / box);  // boxes with keys of the part
        ids.advance(key0 >> a.shift);
        // lane: box (lane / (2 kSub)), 64-element half, k or v
        const int b = lane / (2 * kSub), half = (lane >> 1) % kSub;
        const int key = key0 + b * box;
        const int id = ids.get(key >> a.shift);
        const bool load = b < boxes;
        const bool there = load && id >= 0 && id < a.blocks;
        const uint32_t mask = __ballot_sync(0xffffffffu, there && lane % (2 * kSub) == 0);
        if (lane == 0) {
          int quarters = 0;  // 16-key quarters in blocks of the cache
          for (int i = 0; i < 4; ++i) quarters |= ((mask >> ((i * 16 / box) * 2 * kSub)) & 1) << i;
          sh.valid[s] = (uint8_t)quarters;
          mbar_arrive_expect_tx(&sh.full[s], (uint32_t)(boxes * box * D * 4));
        }
        __syncwarp();
        if (load) {
          uint8_t* dst = smem + s * S::kStage + (lane & 1) * S::kHalf + half * (kTileKeys * 128) + b * box * 128;
          // a block that is not there reads zeros from past the end of the cache
          tma_load_3d(dst, (lane & 1) ? &tv : &tk, &sh.full[s], half * 64, (q.kvh << a.shift) + (key & ((1 << a.shift) - 1)),
                      there ? id : a.blocks);
        }
      }
    }
    // No copy may be in flight when the CTA exits.
    if (lane == 0)
      for (long long i = max(0LL, issued - S::kStages); i < issued; ++i)
        mbar_wait_drain(&sh.full[i % S::kStages], (uint32_t)((i / S::kStages) & 1), L.err, L.wait_ns);
  } else {
    // ------------------------------------------------------------ products
    const int wk = warp % WK, wm = warp / WK;  // which keys of a tile, which 16 rows of a chunk
    const int g = lane >> 2, t4 = lane & 3;
    constexpr int NK = S::kKeys / 8;           // 8-key columns of S
    long long seen = 0;
    int part = 0;
    for (long long u = u0; u < u1;) {
      const Piece q = piece_at(sh.parts, a, L.plan, u, u1, part);
      u += q.tile1 - q.tile0;
      const int len = sh.parts.len[part], rows = sh.parts.rows[part] * group;
      const int r0 = q.chunk * S::kRows + wm * 16;
      // this thread's two rows: g and g + 8 of the warp's 16
      uint32_t qf[D / 16][4];
      int sees[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = r0 + g + 8 * e;
        const bool in = r < rows;
        const int row = in ? r / group : 0;
        sees[e] = in ? min(len, part == 0 ? len : sh.parts.last[part] + row) : 0;
        const uint16_t* src = a.q + (long long)(sh.parts.row0[part] + row) * a.ldq +
                              (long long)(q.kvh * group + (in ? r % group : 0)) * D + 2 * t4;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          qf[i][e] = in ? (uint32_t)ld_act_s32(src + i * 16) : 0u;
          qf[i][e + 2] = in ? (uint32_t)ld_act_s32(src + i * 16 + 8) : 0u;
        }
      }
      float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
      // the fewest keys that any row of the chunk sees
      const int fewest = part == 0 ? len : min(len, sh.parts.last[part] + (q.chunk * S::kRows) / group);

      bool ok = true;
      for (int t = q.tile0; t < q.tile1; ++t, ++seen) {
        const int s = (int)(seen % S::kStages);
        ok = __all_sync(0xffffffffu, mbar_wait(&sh.full[s], (uint32_t)((seen / S::kStages) & 1), wc));
        if (!ok) break;
        const uint32_t kb = smem_u32(smem + s * S::kStage), vb = kb + S::kHalf;
        const int valid = sh.valid[s];
        const int key0 = t * kTileKeys + wk * S::kKeys;  // the warp's first key
        const bool edge = key0 + S::kKeys > fewest || valid != 15;
        float p[NK][4];
#pragma unroll
        for (int j = 0; j < NK; ++j) p[j][0] = p[j][1] = p[j][2] = p[j][3] = 0.f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int j = 0; j < NK / 2; ++j) {
            // matrices: keys 0-7 and 8-15 by elements 0-7 and 8-15 of step i
            uint32_t b[4];
            const int kr = wk * S::kKeys + j * 16 + ((lane >> 4) << 3) + (lane & 7);
            const int cv = i * 2 + ((lane >> 3) & 1);
            ldsm4(b, kb + (cv >> 3) * (kTileKeys * 128) + swz(kr, cv & 7));
            mma16816(p[2 * j], qf[i], b[0], b[1]);
            mma16816(p[2 * j + 1], qf[i], b[2], b[3]);
          }
        if (edge) {
#pragma unroll
          for (int j = 0; j < NK; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int kk = wk * S::kKeys + j * 8 + 2 * t4 + (e & 1);  // key within the tile
              const bool see = t * kTileKeys + kk < sees[e >> 1] && ((valid >> (kk >> 4)) & 1);
              p[j][e] = see ? p[j][e] : -INFINITY;
            }
        }
        // running maximum (log2 units), shared by the four threads of a row
        float ref[2], up[2];
        bool grew = false;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = -INFINITY;
#pragma unroll
          for (int j = 0; j < NK; ++j) x = fmaxf(x, fmaxf(p[j][2 * e], p[j][2 * e + 1]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
          const float mn = fmaxf(m[e], x * L.scale_log2);
          grew = grew || mn > m[e];
          ref[e] = mn == -INFINITY ? 0.f : mn;
          up[e] = ex2_from(m[e], ref[e]);
          m[e] = mn;
        }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int e = 0; e < 2; ++e) l[e] *= up[e];
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            o[i][0] *= up[0];
            o[i][1] *= up[0];
            o[i][2] *= up[1];
            o[i][3] *= up[1];
          }
        }
        uint32_t pf[NK / 2][4];
#pragma unroll
        for (int j = 0; j < NK; ++j) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = ex2(fmaf(p[j][e], L.scale_log2, -ref[e >> 1]));
          l[0] += w[0] + w[1];
          l[1] += w[2] + w[3];
          // P is rounded to bf16 for the product with V (fp32 sums; l keeps the unrounded weights)
          pf[j >> 1][(j & 1) * 2] = pack_bf16x2(w[0], w[1]);
          pf[j >> 1][(j & 1) * 2 + 1] = pack_bf16x2(w[2], w[3]);
        }
#pragma unroll
        for (int j = 0; j < NK / 2; ++j) {
          // Keys behind the part's last one hold anything (NaN too): their V is
          // taken as zero, as 0 * NaN would not be.
          uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
          if (edge) {
            const int kk = key0 + j * 16 + 2 * t4;
            keep0 = (kk < len ? 0xffffu : 0u) | (kk + 1 < len ? 0xffff0000u : 0u);
            keep1 = (kk + 8 < len ? 0xffffu : 0u) | (kk + 9 < len ? 0xffff0000u : 0u);
          }
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            // matrices (transposed): keys 0-7 and 8-15 by elements 0-7 and 8-15 of pair i
            uint32_t b[4];
            const int kr = wk * S::kKeys + j * 16 + (lane & 15);
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
      }
      // the warps that join their sums leave together; this barrier also ends the
      // reads of the previous piece's sums
      if (WK > 1 ? !named_bar_and(1, 128, ok) : !ok) break;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
      }

      // ---------------------------------------------------------- the piece's rows
      const bool whole = q.tile0 == 0 && q.tile1 == q.tiles;
      const bool direct = whole && part > 0 && a.prefix_len == 0;
      const bool begins = q.tile0 == 0;
      const int in_chunk = min(S::kRows, rows - q.chunk * S::kRows);
      // where row r of the chunk goes: 8 or 4 consecutive elements at column col
      auto out_row = [&](int r) {
        const int rr = q.chunk * S::kRows + r;
        return (long long)(sh.parts.row0[part] + rr / group) * a.ldo + (long long)(q.kvh * group + rr % group) * D;
      };
      auto keep_at = [&](int r) {
        const int rr = q.chunk * S::kRows + r;
        return begins ? (long long)(sh.parts.row0[part] + rr / group) * a.q_heads + q.kvh * group + rr % group
                      : c * S::kRows + r;
      };
      const Pieces& keep = begins ? L.start[part > 0] : L.plan.rest;
      if (WK == 1) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = wm * 16 + g + 8 * e;
          if (r >= in_chunk) continue;
          if (direct) {
            const float inv = l[e] == 0.f ? 0.f : 1.f / l[e];
            uint16_t* to = a.out + out_row(r) + 2 * t4;
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
              *reinterpret_cast<uint32_t*>(to + 8 * i) = pack_bf16x2(o[i][2 * e] * inv, o[i][2 * e + 1] * inv);
          } else {
            const long long at = keep_at(r);
            float* to = keep.o + at * D + 2 * t4;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) *reinterpret_cast<float2*>(to + 8 * i) = make_float2(o[i][2 * e], o[i][2 * e + 1]);
            if (t4 == 0) keep.ml[at] = make_float2(m[e], l[e]);
          }
        }
      } else {
        // join the WK warps that hold the same rows
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = g + 8 * e;
          if (wm * 16 + r >= in_chunk) continue;
          float* to = s_merge + (warp * 16 + r) * D;
#pragma unroll
          for (int i = 0; i < D / 8; ++i)
            *reinterpret_cast<float2*>(to + ((8 * i + 2 * t4) ^ ((r & 7) << 3))) = make_float2(o[i][2 * e], o[i][2 * e + 1]);
          if (t4 == 0) sh.ml[warp][r] = make_float2(m[e], l[e]);
        }
        named_bar_sync(1, 128);
        for (int it = threadIdx.x; it < in_chunk * (D / 4); it += 128) {
          const int r = it / (D / 4), col = (it % (D / 4)) * 4;
          const int w0 = (r >> 4) * WK, rr = r & 15;
          float top = -INFINITY, sum = 0.f;
#pragma unroll
          for (int w = 0; w < WK; ++w) top = fmaxf(top, sh.ml[w0 + w][rr].x);
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < WK; ++w) {
            const float2 ml = sh.ml[w0 + w][rr];
            const float f = ex2_from(ml.x, top);
            const float4 y = *reinterpret_cast<const float4*>(s_merge + ((w0 + w) * 16 + rr) * D + (col ^ ((rr & 7) << 3)));
            sum = fmaf(ml.y, f, sum);
            x.x = fmaf(y.x, f, x.x);
            x.y = fmaf(y.y, f, x.y);
            x.z = fmaf(y.z, f, x.z);
            x.w = fmaf(y.w, f, x.w);
          }
          if (direct) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            *reinterpret_cast<uint2*>(a.out + out_row(r) + col) =
                make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv));
          } else {
            const long long at = keep_at(r);
            *reinterpret_cast<float4*>(keep.o + at * D + col) = x;
            if (col == 0) keep.ml[at] = make_float2(top, sum);
          }
        }
      }
    }
  }
}

// Joins the pieces of the rows that more than one CTA, or the prefix and the
// own tokens, gave: out = sum O_i 2^(m_i - m) / sum l_i 2^(m_i - m). One CTA per
// (row, head), the pieces spread over its 8 warps: what bounds it is the
// latency of their reads from L2. A row with no piece at all gets zeros.
template <int D>
__global__ void __launch_bounds__(256) combine_attention_kernel(const AttentionLaunch P, const AttentionLaunch O) {
  __shared__ PartTable tp, to;
  __shared__ float s_o[8][D];
  __shared__ float2 s_ml[8];
  const AttentionParams& a = O.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x, head = blockIdx.y;
  const int group = a.q_heads / a.kv_heads, kvh = head / group;
  pdl_trigger();
  pdl_wait();
  if (warp == 0) build_parts(to, O.a, O.plan);
  if (warp == 1) build_parts(tp, P.a, P.plan);
  __syncthreads();
  int part = 0;
  for (int i = 1; i <= a.requests; ++i)
    if (t >= to.row0[i] && t < to.row0[i] + to.rows[i]) part = i;
  if (part == 0) return;  // a row of no request

  // pieces of one part: the starting one, then one for each further CTA
  struct Span {
    long long at;        // row of `start`
    int c0, count, r;    // first CTA, pieces, row within the chunk
  };
  auto span_of = [&](const PartTable& T, const AttentionLaunch& L, int i) {
    Span s{(long long)t * a.q_heads + head, 0, 0, 0};
    const long long W = T.first[a.requests + 1];
    const long long tiles = ((long long)T.len[i] + kTileKeys - 1) / kTileKeys;
    if (T.first[i + 1] == T.first[i]) return s;
    const long long G = plan_ctas(W, L.plan.ctas);
    const int chunks = (T.rows[i] * group + L.plan.rows - 1) / L.plan.rows;
    const int rr = (t - T.row0[i]) * group + head % group;
    const long long u = T.first[i] + ((long long)kvh * chunks + rr / L.plan.rows) * tiles;
    s.r = rr % L.plan.rows;
    s.c0 = (int)cta_of_unit(u, W, G);
    s.count = (int)cta_of_unit(u + tiles - 1, W, G) - s.c0 + 1;
    return s;
  };
  const Span sp = span_of(tp, P, 0), so = span_of(to, O, part);
  if (sp.count == 0 && so.count == 1) return;  // written by the one CTA that had it
  const int n = sp.count + so.count;
  constexpr int V = D / 32;
  float x[V], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) x[e] = 0.f;
  constexpr int B = 4;  // pieces in flight per warp
  for (int i0 = warp; i0 < n; i0 += 8 * B) {
    float y[B][V];
    float2 ml[B];
#pragma unroll
    for (int k = 0; k < B; ++k) {
      const int i = i0 + 8 * k;
      ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int e = 0; e < V; ++e) y[k][e] = 0.f;
      if (i < n) {
        const bool pre = i < sp.count;
        const int j = pre ? i : i - sp.count;
        const Pieces& from = j == 0 ? O.start[pre ? 0 : 1] : (pre ? P.plan.rest : O.plan.rest);
        const Span& s = pre ? sp : so;
        const long long at = j == 0 ? s.at : (long long)(s.c0 + j) * (pre ? P.plan.rows : O.plan.rows) + s.r;
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
      const float f0 = ex2_from(m, top), f1 = ex2_from(ml[k].x, top);
      m = top;
      l = l * f0 + ml[k].y * f1;
#pragma unroll
      for (int e = 0; e < V; ++e) x[e] = x[e] * f0 + y[k][e] * f1;
    }
  }
#pragma unroll
  for (int e = 0; e < V; ++e) s_o[warp][lane * V + e] = x[e];
  if (lane == 0) s_ml[warp] = make_float2(m, l);
  __syncthreads();
  if (threadIdx.x < D / 2) {
    float top = -INFINITY, sum = 0.f, v0 = 0.f, v1 = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) top = fmaxf(top, s_ml[w].x);
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const float f = ex2_from(s_ml[w].x, top);
      sum = fmaf(s_ml[w].y, f, sum);
      v0 = fmaf(s_o[w][2 * threadIdx.x], f, v0);
      v1 = fmaf(s_o[w][2 * threadIdx.x + 1], f, v1);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    *reinterpret_cast<uint32_t*>(a.out + (long long)t * a.ldo + (long long)head * D + 2 * threadIdx.x) =
        pack_bf16x2(v0 * inv, v1 * inv);
  }
}

// ---------------------------------------------------------------------------- host side
namespace {

// Rows of the smallest chunk kernel that holds `rows` query rows.
int chunk_rows(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

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
    w.rest[i] = pieces((size_t)h->sms * 64);
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

template <int D, int WK>
cudaError_t launch_shape(dec_handle* h, const CUtensorMap& tk, const CUtensorMap& tv, const AttentionLaunch& L,
                         cudaStream_t s) {
  using S = AttnShape<D, WK>;
  static std::atomic<uint64_t> ready{0};  // devices whose function attribute is set
  const uint64_t bit = 1ull << (h->device & 63);
  if (!(ready.load() & bit)) {
    const cudaError_t e =
        cudaFuncSetAttribute(attention_kernel<D, WK>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kTotal);
    if (e != cudaSuccess) return e;
    if (h->device < 64) ready.fetch_or(bit);
  }
  return launch_k(h, attention_kernel<D, WK>, dim3(L.plan.ctas), dim3(kAttnThreads), (size_t)S::kTotal, s, tk, tv, L);
}

cudaError_t launch_chunks(dec_handle* h, const CUtensorMap& tk, const CUtensorMap& tv, const AttentionLaunch& L,
                          cudaStream_t s) {
  const bool d64 = L.a.dim == 64;
  switch (L.plan.rows) {
    case 16: return d64 ? launch_shape<64, 4>(h, tk, tv, L, s) : launch_shape<128, 4>(h, tk, tv, L, s);
    case 32: return d64 ? launch_shape<64, 2>(h, tk, tv, L, s) : launch_shape<128, 2>(h, tk, tv, L, s);
    default: return d64 ? launch_shape<64, 1>(h, tk, tv, L, s) : launch_shape<128, 1>(h, tk, tv, L, s);
  }
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
  own.scale_log2 = P.scale * 1.4426950408889634f;
  own.err = h->d_err;
  own.wait_ns = h->wait_ns;
  own.plan = Plan{0, 1, chunk_rows(std::min(P.max_new, P.M) * group), h->sms, w.rest[1]};
  AttentionLaunch pre = own;
  pre.plan = Plan{P.prefix_len > 0 ? 1 : 0, 0, chunk_rows(P.M * group), h->sms, w.rest[0]};
  cudaError_t e = cudaSuccess;
  if (P.prefix_len > 0) {
    if (pre.plan.rows == own.plan.rows) {
      // the same kernel: one launch takes both
      own.plan.prefix = 1;
      pre.plan = own.plan;
    } else {
      LaunchScope scope(h, "attention_prefix", s);
      e = launch_chunks(h, tk, tv, pre, s);
      if (e != cudaSuccess) return e;
    }
  }
  {
    LaunchScope scope(h, "attention", s);
    e = launch_chunks(h, tk, tv, own, s);
    if (e != cudaSuccess) return e;
  }
  LaunchScope scope(h, "attention_join", s);
  const dim3 grid(P.M, P.q_heads);
  if (P.dim == 64) return launch_k(h, combine_attention_kernel<64>, grid, dim3(256), 0, s, pre, own);
  return launch_k(h, combine_attention_kernel<128>, grid, dim3(256), 0, s, pre, own);
}

}  // namespace dec
