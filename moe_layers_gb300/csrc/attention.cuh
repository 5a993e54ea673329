// What the attention kernels share: how a step's work is cut into tiles and
// divided among CTAs, and where the parts of a row that several CTAs computed
// are kept until they are joined.
//
// A step has parts: part 0 is the shared prefix (its rows: every row of the
// batch), part b + 1 the own tokens of request b. For one part and one key /
// value head the query rows are (row of the part, head of the group), in
// chunks of as many as the kernel holds, and the keys are in tiles of 64 or 128. A
// (head, chunk) is as many units as it has tiles, behind `lead` units that
// stand for the cost of beginning and ending it; the units of a part are
// ordered (head, chunk, tile), the parts follow each other, and CTA c of G (at
// most W) takes units [c W / G, (c + 1) W / G) of all W: every CTA has the same
// work, however ragged the lengths are. The tiles of one (head, chunk) that
// one CTA takes are a piece. A piece that holds the first tile is kept by its
// rows (`start`); any other is the first piece of its CTA and is kept by the
// CTA (`rest`). The whole plan follows from the lengths in device memory, so
// nothing of it depends on the host.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace dec {

constexpr int kMaxParts = 65;

// Unnormalised sums [rows][dim] with their (maximum, sum) pairs, maxima of q . k
// as it is, without the scale.
struct Pieces {
  float* o = nullptr;
  float2* ml = nullptr;
};

// One launch's share of the plan.
struct Plan {
  bool prefix, own;  // which parts the launch takes
  int row_shift[2]; // a chunk is 1 << row_shift query rows: prefix, own
  int rest_rows;    // rows of a piece in `rest`
  int lead;         // units a (head, chunk) counts for besides its tiles
  int tile_shift;   // a tile is 1 << tile_shift keys
  int ctas;
  Pieces rest;      // [ctas][rest_rows]
};

struct AttentionLaunch {
  AttentionParams a;
  Plan plan;
  Pieces start[2];  // prefix, own: [M][q_heads]
  float scale_log2;    // the scale times log2 e
  bool late_wait;      // the launch before it on the stream is the same call's prefix launch
  uint32_t group_mul;  // ceil(2^20 / group)
  int* err;
  unsigned long long wait_ns;
};

struct PartTable {
  long long first[kMaxParts + 1];  // first unit; first[n] = all units
  short row0[kMaxParts], rows[kMaxParts], chunks[kMaxParts];
  int len[kMaxParts];
  int last[kMaxParts];  // keys that the part's first row sees; each further row sees one more (own parts)
};

// CTAs that take part: none without a unit, so that the pieces of a (head,
// chunk) lie in consecutive CTAs.
__device__ __forceinline__ long long plan_ctas(long long W, int ctas) { return W < 1 ? 1 : W < ctas ? W : ctas; }
// c W / G, rounded down (an approximate quotient and exact products).
__device__ __forceinline__ long long unit_start(long long c, long long W, long long G) {
  const long long x = c * W;
  if (x >> 40) return x / G;
  long long q = (long long)((float)x / (float)G);  // off by at most x / G 2^-22 + 1
  const long long e = x - q * G;
  if (e < 0 || e >= G) q += e >= 0 ? (int)((uint32_t)e / (uint32_t)G) : -(int)((uint32_t)(G - 1 - e) / (uint32_t)G);
  return q;
}
// The c with unit_start(c) <= u < unit_start(c + 1), that is c W < (u + 1) G <= (c + 1) W.
__device__ __forceinline__ int cta_of_unit(long long u, long long W, long long G) {
  const long long x = (u + 1) * G;
  int c = (int)((float)x / (float)W);
  while (c * W >= x) --c;
  while ((c + 1) * W < x) ++c;
  return c;
}

// r / group for 0 <= r < 64 group, group <= 128, by a product: mul = ceil(2^20 / group).
__device__ __forceinline__ int div_group(int r, uint32_t mul) { return (int)(((uint32_t)r * mul) >> 20); }

// Fills the table with one warp (all 32 lanes). Lengths are brought into
// range: rows into [0, M] and not decreasing, the requests' within part 0's (the
// joining kernel looks each of them up in both), keys to at most max_blocks blocks.
__device__ __forceinline__ void build_parts(PartTable& t, const AttentionParams& a, const Plan& p) {
  constexpr int kRounds = (kMaxParts + 31) / 32;
  const int lane = threadIdx.x & 31, n = a.requests + 1;
  int r0[kRounds], r1[kRounds], own[kRounds];
#pragma unroll
  for (int k = 0; k < kRounds; ++k) {  // every load before any use
    const int i = k * 32 + lane;
    r0[k] = r1[k] = own[k] = 0;
    if (i < n) {
      r0[k] = ld_act_s32(a.row_start + (i == 0 ? 0 : i - 1));
      r1[k] = ld_act_s32(a.row_start + (i == 0 ? a.requests : i));
      if (i > 0) own[k] = ld_act_s32(a.own_len + i - 1);
    }
  }
  const int begin = min(max(__shfl_sync(0xffffffffu, r0[0], 0), 0), a.M);
  const int end = min(max(__shfl_sync(0xffffffffu, r1[0], 0), begin), a.M);
  long long carry = 0;
#pragma unroll
  for (int k = 0; k < kRounds; ++k) {
    if (k * 32 >= n) break;
    const int i = k * 32 + lane;
    long long units = 0;
    if (i < n) {
      const int first = min(max(r0[k], begin), end), rows = min(max(r1[k], first), end) - first;
      int len = a.prefix_len, last = a.prefix_len;
      if (i > 0) {
        len = max(0, (int)min((long long)own[k], (long long)a.max_blocks << a.shift));
        last = (int)min(max((long long)own[k] - rows + 1, -1000LL), 0x7fffff00LL);  // room for the rows on top
      }
      t.row0[i] = (short)first;
      t.rows[i] = (short)rows;
      t.len[i] = len;
      t.last[i] = last;
      if (i == 0 ? p.prefix : p.own) {
        const int shift = p.row_shift[i > 0], chunks = (rows * a.group + (1 << shift) - 1) >> shift;
        t.chunks[i] = (short)chunks;
        const long long tiles = ((long long)len + (1 << p.tile_shift) - 1) >> p.tile_shift;
        units = tiles > 0 ? (long long)a.kv_heads * chunks * (tiles + p.lead) : 0;
      }
    }
    long long inc = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (i < n) t.first[i] = carry + inc - units;
    carry += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (lane == 0) t.first[n] = carry;
}

// Walks the pieces of units [u, u_end). A piece without tiles (its units are
// leading ones) can only be the last.
struct Piece {
  int part = 0, kvh = 0, chunk = 0, chunks = 1, tiles = 0, tile0 = 0, tile1 = 0, units = 0;
  __device__ __forceinline__ bool empty() const { return tile1 <= tile0; }
  __device__ __forceinline__ void enter(const PartTable& t, const Plan& p) {
    chunks = t.chunks[part];
    tiles = (int)(((long long)t.len[part] + (1 << p.tile_shift) - 1) >> p.tile_shift);
  }
  __device__ __forceinline__ void cut(const Plan& p, int x0, long long room) {
    units = (int)min((long long)(tiles + p.lead - x0), room);
    tile0 = max(0, x0 - p.lead);
    tile1 = max(0, x0 + units - p.lead);
  }
  __device__ __forceinline__ void begin(const PartTable& t, const AttentionParams& a, const Plan& p, long long u,
                                        long long u_end) {
    // the part that holds unit u (all lanes of a warp, the same u)
#pragma unroll
    for (int k = 0; k < (kMaxParts + 31) / 32; ++k) {
      const int i = k * 32 + (threadIdx.x & 31);
      const uint32_t hit = __ballot_sync(0xffffffffu, i <= a.requests && t.first[i] <= u && u < t.first[i + 1]);
      if (hit) part = k * 32 + __ffs(hit) - 1;
    }
    enter(t, p);
    const long long at = u - t.first[part];
    const int each = tiles + p.lead;
    const int hc = (at >> 32) == 0 ? (int)((uint32_t)at / (uint32_t)each) : (int)(at / each);
    kvh = chunks == 1 ? hc : hc / chunks;
    chunk = hc - kvh * chunks;
    cut(p, (int)(at - (long long)hc * each), u_end - u);
  }
  // the next piece, which starts at unit u
  __device__ __forceinline__ void next(const PartTable& t, const AttentionParams& a, const Plan& p, long long u,
                                       long long u_end) {
    if (++chunk == chunks) {
      chunk = 0;
      if (++kvh == a.kv_heads) {
        kvh = 0;
        do ++part;
        while (t.first[part + 1] <= u);
        enter(t, p);
      }
    }
    cut(p, 0, u_end - u);
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^(scale (m - top)), 0 for a part that saw nothing (m = -inf, whatever top is).
// The difference comes before the scale, here and for the weights: the largest
// score's weight is then 1 whatever its size. (With fma(score, scale, -maximum),
// an instruction less, the rounding of the maximum remains, and from scores of
// 2^31 on it alone passes the range of an exponential.)
__device__ __forceinline__ float ex2_from(float m, float top, float scale) {
  return m == -INFINITY ? 0.f : ex2((m - top) * scale);
}

// Whether one of two bf16 values is an infinity or NaN (its exponent is all ones).
__device__ __forceinline__ bool not_finite(uint32_t pair) {
  return (((pair & 0x7f807f80u) + 0x00800080u) & 0x80008000u) != 0;
}
// The pair with zeros in place of infinities and NaN.
__device__ __forceinline__ uint32_t finite_of(uint32_t pair) {
  const uint32_t top = ((pair & 0x7f807f80u) + 0x00800080u) & 0x80008000u;  // the top bit of each such half
  return pair & ~(top | (top - (top >> 15)));
}

// A warp's bounded wait: true in every lane, or false in every lane.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitCtl& wc) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, wc));
}

// Requests the lengths, tables and query rows into L2 while the launch before
// drains (a hint: nothing is read). Each CTA takes a share of the lines.
__device__ __forceinline__ void warm_l2(const AttentionParams& a) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x, n = gridDim.x * blockDim.x;
  auto want = [](const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); };
  const int row_lines = (a.q_heads * a.dim * 2 + 127) / 128;
  for (int k = i; k < a.M * row_lines; k += n) {
    const int t = k / row_lines;
    want(a.q + t * a.ldq + (k - t * row_lines) * 64);
  }
  for (int k = i; k * 32 <= a.requests; k += n) {
    want(a.row_start + k * 32);
    if (k * 32 < a.requests) want(a.own_len + k * 32);
  }
  const int blocks = (int)(((long long)a.prefix_len + (1 << a.shift) - 1) >> a.shift);
  for (int k = i; k * 32 < blocks; k += n) want(a.prefix_table + k * 32);
}

// One lane of a converged warp. Copies and products are issued behind it from
// values that are the same in every lane: the instructions take their operands
// from uniform registers, and a lane that diverges to issue them moves each
// operand there first (100 cycles a copy or product instead of about 25).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

__device__ __forceinline__ void named_bar_arrive(int id, int count) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
}

// The cache is read once, and leaves L2 first, so that lengths, tables, queries
// and pieces stay there; the keys of several chunks of rows are read again soon.
__device__ __forceinline__ uint64_t policy_evict_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* m, uint64_t* bar, int c0, int c1, int c2,
                                            uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "l"(pol)
      : "memory");
}

// Cache ids of a part's blocks, read 32 at a time by a whole warp, the next 32 ahead.
struct BlockIds {
  const int32_t* table;
  int count;  // entries that may be read
  int base = -64, cur = -1, next = -1;
  __device__ __forceinline__ BlockIds(const int32_t* t, int n) : table(t), count(n) {}
  __device__ __forceinline__ int load(int i) const { return i < count ? ld_act_s32(table + i) : -1; }
  // Makes the 32 entries around i present (the same i in every lane; a tile's
  // entries lie in one aligned group of 32, and i never falls).
  __device__ __forceinline__ void advance(int i) {
    const int want = i & ~31;
    if (want == base) return;
    cur = want == base + 32 ? next : load(want + (threadIdx.x & 31));
    base = want;
    next = load(want + 32 + (threadIdx.x & 31));
  }
  __device__ __forceinline__ int get(int i) const { return __shfl_sync(0xffffffffu, cur, i & 31); }
};

// The tcgen05 kernel (attention_tc.cu), for chunks of 128 or 256 rows.
cudaError_t launch_attention_tc(dec_handle* h, const CUtensorMap& tk, const CUtensorMap& tv, const AttentionLaunch& L,
                                cudaStream_t s);

}  // namespace dec
