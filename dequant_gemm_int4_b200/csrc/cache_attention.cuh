// Attention over the 4-bit cache for few query rows (decoding, and chunks of
// queries): the tensor-core kernel and the kernel that joins its pieces.
//
// Mathematics.  For the RT query rows that share one key/value head (the
// query heads of the group times the sequence's query tokens), per tile of
// tokens:
//   S^T = K Q^T          mma.m16n8k16, tokens x query rows
//   P   = 2^(S - max)    running maximum and sum per row, in fp32
//   O^T += V^T P^T       mma.m16n8k16, head elements x query rows
// The codes enter the products as they are: a nibble n (offset to 0..15) in
// the low bits of a half is the fp16 subnormal n 2^-24, which the tensor core
// takes as it is, so expanding 8 codes takes a shift and four bitwise
// operations and no arithmetic.  The second nibble of a byte stays four bits
// up and counts 16-fold; the query's element (or the output row) is divided
// by 16 instead, exactly.  With z the zero point (8 in the symmetric scheme,
// whose codes are turned to 0..15 by flipping the sign bit)
//   sum_d q_d (n_d - z) s = s (sum_d q_d n_d - z sum_d q_d), per group, and
//   sum_t p_t s_t (n_t - z_t) = sum_t w_t n_t - sum_t w_t z_t, w_t = p_t s_t,
// the second sum by one more matrix product whose A operand holds the z_t.
//
// Precision.  q enters in fp16 after a power-of-two scaling by the row's
// largest element: exact for bf16 and fp16 but for elements 2^-24 times
// smaller than that one, whose error stays below 2^-38 of it.  S, the
// softmax's maximum and sum and O are fp32.  w_t is rounded to fp16 twice
// (each by at most 2^-11 of itself): p_t, taken by a power of two that follows
// the largest value scale so far (of tokens that some row sees), and its product
// with s_t.  A product with that scale lies below 2^15, so weights keep their
// full precision down to 2^-20 of the largest and in half the fp16 range below
// it some of it.  With fp32 products the second rounding would go, and a
// conversion and two multiplications for each weight would come.
// The tensor core aligns the terms of a step by their operands' exponents, where
// a subnormal counts as 2^-14, and cuts them off about 25 bits below the
// largest: the sums over n and over z keep 15 bits or more of sum_t p_t s_t z_t
// (an output whose values cancel came out 3.5e-5 of that off; 2.6e-4 is what
// the weights' roundings leave of an output's norm), S about 20 of its terms'
// (lse: 3e-6 to 7e-6 at scores near 10).  All codes moved up to bit 6 (three
// shifts more for each word of values) brought the first below 9e-6 and cost 3
// to 5 % of the decoding cases: not taken, the weights' roundings being larger.
//
// Layout.  One warp takes 64 tokens at a time (32, for 16 or 32 rows and for
// heads of 256: the scores fill the registers): their key and value rows are
// copied to shared memory by 16-byte asynchronous copies, several tiles
// ahead, each warp on its own.  ldmatrix then gives each lane whole words of
// a token's codes (keys), and its transposed form gives halfwords of two
// neighbouring tokens (values), which are the A operands after the bitwise
// expansion: the contraction order inside a block of 32 elements is permuted
// and Q is stored in the same order.
//
// Work split.  The tokens of all (sequence, head, row tile) items are counted
// in steps of a tile for each of four warps and shared evenly among one wave of blocks, whatever the
// lengths; a block's share may begin or end inside an item, and the pieces of
// a split item are joined by a second kernel in a fixed order.  Every block
// finds its share from the lengths on the device, so a captured graph can be
// replayed with other lengths.  Where the table has room for a few steps an
// item only, an item is given to the blocks of one cluster instead: they join
// through each other's shared memory, and the second kernel is saved (one
// sequence of 2048 tokens, 32 query heads on 8: 8.9 us with it, 7.2 without).
//
// What bounds it (times in a captured graph).  64 sequences of up to 8192 tokens,
// 64 query heads of 128 on 8: 75 us for 313 MB, 4.2 TB/s; the slope between two
// lengths is 6.2 TB/s, and 16 us of set-up, merges and join come on top.  One
// sequence of 131071 tokens in groups of 32: 42 us for 151 MB, four scales and
// products to a head beside the codes.  One sequence of 2048 tokens, 7.2 us: the
// latency of the set-up (2), the first tile (2), merge and cluster join (2).  More
// rows to a tile (8 queries of 4 heads, 32 sequences of up to 4096 tokens, 53 us):
// latency of the products and the softmax at three warps a scheduler (issue slots
// 49 % taken, tensor pipe 31 %).
#pragma once

#include <atomic>
#include <type_traits>

#include "cache.cuh"
#include "internal.h"
#include "sm100_ptx.cuh"

namespace int4lib {

constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = 32 * kAttnWarps;
// Tokens of a warp's tile and of a block's step, by the row tile: 64 while the
// scores of 8 rows fit beside the accumulators, else 32.
__host__ __device__ constexpr int attention_tokens(int head_dim, int rt) { return rt == 8 && head_dim <= 128 ? 64 : 32; }
__host__ __device__ constexpr int attention_step(int head_dim, int rt) { return kAttnWarps * attention_tokens(head_dim, rt); }

// Where the pieces of split items go, in the caller's workspace.
inline size_t attention_prefix_bytes(int64_t batch) {
  return (static_cast<size_t>(batch + 1) * 4 + 255) / 256 * 256;
}
struct AttentionSpace {
  int32_t* prefix;  // [batch + 1]: units of the sequences before each
  float* o;         // [2 * blocks][RT][D]: sums relative to the piece's maximum
  float* ml;        // [2 * blocks][RT][2]: maximum (log2) and sum
  int blocks;
  int cluster;  // 0: shares of all units; else blocks to an item, joined inside their cluster
};

// Row tile `rt` (rows [rt RT, (rt + 1) RT) of a sequence's query tokens x
// ratio): the tokens that its rows see, from first to hi, those that it needs,
// from lo (first rounded down to a multiple of a warp's tile) on, and its steps.
struct RowTile {
  int lo, first, hi, steps;
  __device__ __forceinline__ void set(const AttentionArgs& a, int len, int count, int rt, int RT) {
    const int step = attention_step(a.cache.head_dim, RT);
    const int r0 = rt * RT, rows = count * a.ratio;
    const int r1 = min(r0 + RT, rows) - 1;
    const int i0 = a.token_of(r0), i1 = a.token_of(r1);  // the tile's first and last query token
    int lo0, hi0, lo1, hi1;
    a.visible(len - count + i0, len, lo0, hi0);
    a.visible(len - count + i1, len, lo1, hi1);
    first = lo0;
    lo = lo0 & -(step / kAttnWarps);
    hi = hi1;
    steps = hi > lo ? (hi - lo + step - 1) / step : 0;
  }
};

__device__ __forceinline__ int row_tiles(const AttentionArgs& a, int count, int RT) {
  return (count * a.ratio + RT - 1) / RT;
}

// Steps of one head of sequence b, over all its row tiles.
__device__ __forceinline__ int head_units(const AttentionArgs& a, int b, int RT) {
  int first, count;
  a.queries(b, first, count);
  const int len = a.kv_len(b);
  const int n = row_tiles(a, count, RT);
  int u = 0;
  for (int rt = 0; rt < n; ++rt) {
    RowTile r;
    r.set(a, len, count, rt, RT);
    u += r.steps;
  }
  return u;
}

// The units (steps, over all heads) of all sequences, counted in their order
// by each warp for itself: lane l holds the sequences [l per, (l + 1) per).
struct Plan {
  int units;       // of all sequences
  int per;
  int mine, upto;  // of this lane's sequences; of those and all before

  __device__ __forceinline__ Plan(const AttentionArgs& a, int RT) {
    const int lane = threadIdx.x & 31;
    per = (a.batch + 31) / 32;
    mine = 0;
    for (int i = 0; i < per; ++i) {
      const int b = lane * per + i;
      if (b < a.batch) mine += head_units(a, b, RT) * a.cache.heads;
    }
    upto = scan(mine);
    units = __shfl_sync(0xffffffffu, upto, 31);
  }
  __device__ __forceinline__ static int scan(int v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += x;
    }
    return v;
  }
  // The sequence that holds unit u (0 <= u < units), and u's place in it.
  __device__ __forceinline__ void find(const AttentionArgs& a, int RT, int u, int& b, int& off) const {
    const int lane = threadIdx.x & 31;
    const int owner = __ffs(__ballot_sync(0xffffffffu, upto > u)) - 1;
    int before = __shfl_sync(0xffffffffu, upto - mine, owner);
    b = owner * per;
    off = u - before;
    if (per == 1) return;
    if (per <= 8) {  // one after the other, the same in every lane
      for (;; ++b) {
        const int v = head_units(a, b, RT) * a.cache.heads;
        if (off < v) return;
        off -= v;
      }
    }
    for (int i0 = 0; i0 < per; i0 += 32) {
      const int x = b + i0 + lane;
      const int v = i0 + lane < per && x < a.batch ? head_units(a, x, RT) * a.cache.heads : 0;
      const int sum = scan(v);
      const uint32_t past = __ballot_sync(0xffffffffu, before + sum > u);
      if (past != 0u) {
        const int at = __ffs(past) - 1;
        b += i0 + at;
        off = u - before - __shfl_sync(0xffffffffu, sum - v, at);
        return;
      }
      before += __shfl_sync(0xffffffffu, sum, 31);
    }
  }
  // Writes prefix[b + 1], the units up to and with sequence b, for the joins.
  __device__ __forceinline__ void store(const AttentionArgs& a, int RT, int32_t* prefix) const {
    const int lane = threadIdx.x & 31;
    if (lane == 0) prefix[0] = 0;
    int sum = upto - mine;
    for (int i = 0; i < per; ++i) {
      const int b = lane * per + i;
      if (b >= a.batch) break;
      sum += per == 1 ? mine : head_units(a, b, RT) * a.cache.heads;
      prefix[b + 1] = sum;
    }
  }
};

// How `units` steps are shared: the first `more` blocks take `each` + 1, the
// other active ones `each`.
struct Shares {
  int units, active, each, more;
  __device__ __forceinline__ Shares(int units_, int blocks) : units(units_), active(min(units_, blocks)) {
    each = active > 0 ? units / active : 0;
    more = units - each * active;
  }
  __device__ __forceinline__ int begin(int c) const { return c * each + min(c, more); }
  // The block whose share holds unit u.
  __device__ __forceinline__ int block_of(int u) const {
    const int in_larger = more * (each + 1);
    return u < in_larger ? u / (each + 1) : more + (u - in_larger) / each;
  }
};

template <int D_, int GROUP_, int NT_, bool ASYM_>
struct AttnCfg {
  static constexpr int D = D_, GROUP = GROUP_, NT = NT_;
  static constexpr bool ASYM = ASYM_;
  static constexpr int RT = 8 * NT;            // query rows of a tile
  static constexpr int DB = D / 32;            // blocks of 32 elements
  static constexpr int NG = D / GROUP;         // groups of a row
  static constexpr int BPG = GROUP / 32;       // blocks of a group
  static constexpr int RB = D / 2;             // bytes of a row
  static constexpr int RC = RB / 16;           // 16-byte chunks of a row
  // Blocks on an SM, by the registers of the accumulators (D / 4 NT a lane).
  static constexpr int kBlocks = D * NT <= 64 ? 4 : (D * NT <= 256 ? 3 : 2);
  // One warp's tile: keys, values, their scales, their zero points.
  static constexpr int TOK = attention_tokens(D, RT);
  static constexpr int MB = TOK / 16;          // blocks of 16 tokens
  static constexpr int kCodes = TOK * RB;
  static constexpr int kScales = TOK * NG * 2;
  static constexpr int kZeros = ASYM ? TOK * NG : 0;
  static constexpr int kScaleAt = 2 * kCodes;
  static constexpr int kZeroAt = kScaleAt + 2 * kScales;
  static constexpr int kStage = (kZeroAt + 2 * kZeros + 127) / 128 * 128;
  static constexpr int kQ = D * RT * 2;                                // Q in fragment order
  static constexpr int kSmall = RT * (NG + 3 + 2 * kAttnWarps) * 4 + 128;
  static constexpr int kBudget = 227 * 1024 / kBlocks - 1024 - kQ - kSmall;
  static constexpr int kFit = kBudget / (kAttnWarps * kStage);
  static constexpr int kStages = kFit < 2 ? 2 : (kFit > 4 ? 4 : kFit);
  static constexpr int kMergePitch = D + 4;                            // floats of a row
  static constexpr int kMerge = kAttnWarps * 8 * kMergePitch * 4;
  static constexpr int kRing = kAttnWarps * kStages * kStage;
  static constexpr int kRingBytes = kRing > kMerge ? kRing : kMerge;
  static constexpr int kSmem = kRingBytes + kQ + kSmall;
  static constexpr bool kQInRegs = D * NT <= 256;
};

namespace attn {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with the sum begun at {c0, c1} in both halves of the rows.
__device__ __forceinline__ void mma_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1, float c0, float c1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%10,%11};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_half2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// (w ^ flip) & mask in one operation.
template <bool ASYM>
__device__ __forceinline__ uint32_t pick(uint32_t w, uint32_t mask) {
  if (ASYM) return w & mask;
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0x28;" : "=r"(r) : "r"(w), "r"(0x88888888u), "r"(mask));
  return r;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts_u16(uint32_t a, uint32_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(a), "h"(static_cast<uint16_t>(v)) : "memory");
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float2 lds_f2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}

// All threads of a cluster's blocks (of the block, outside a cluster).
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Loads from the same place in the shared memory of block `rank` of the cluster.
__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr, uint32_t rank) {
  float2 v;
  asm volatile("{\n .reg .u32 r;\n mapa.shared::cluster.u32 r, %2, %3;\n ld.shared::cluster.v2.f32 {%0,%1}, [r];\n}"
               : "=f"(v.x), "=f"(v.y) : "r"(addr), "r"(rank) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr, uint32_t rank) {
  float4 v;
  asm volatile("{\n .reg .u32 r;\n mapa.shared::cluster.u32 r, %4, %5;\n ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [r];\n}"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr), "r"(rank) : "memory");
  return v;
}

// Four 16-bit elements, as one load where they are 8-byte aligned.
__device__ __forceinline__ uint2 load_four(const uint16_t* p, bool aligned) {
  if (aligned) return __ldg(reinterpret_cast<const uint2*>(p));
  return make_uint2(__ldg(p) | (static_cast<uint32_t>(__ldg(p + 1)) << 16),
                    __ldg(p + 2) | (static_cast<uint32_t>(__ldg(p + 3)) << 16));
}

// 16-byte chunk c of token row r in a tile: permuted so that the 8 rows of
// an ldmatrix fall into different banks.
template <int RB>
__device__ __forceinline__ int chunk_of(int r, int c) {
  if (RB == 128) return c ^ (r & 7);
  if (RB == 64) return c ^ ((r >> 1) & 3);
  if (RB == 32) return c ^ ((r >> 2) & 1);
  return c;  // rows of 48 bytes: 8 of them fall into different banks as they are
}

}  // namespace attn

template <typename T, class C>
__global__ void __launch_bounds__(kAttnThreads, C::kBlocks)
    attention_mma_kernel(const __grid_constant__ AttentionArgs a, const AttentionSpace ws, const int page_shift) {
  using namespace attn;
  constexpr int D = C::D, NT = C::NT, RT = C::RT, DB = C::DB, NG = C::NG, RB = C::RB, RC = C::RC, MB = C::MB, TOK = C::TOK;
  constexpr int kStep = kAttnWarps * TOK;
  constexpr bool ASYM = C::ASYM;
  constexpr float kNegInf = -__builtin_huge_valf();

  extern __shared__ __align__(128) uint8_t smem[];
  const CacheView& cache = a.cache;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* const sq = smem + C::kRingBytes;
  float* const s_qsum = reinterpret_cast<float*>(sq + C::kQ);  // [NG][RT]
  float* const s_f = s_qsum + RT * NG;                          // [RT]
  int* const s_lo = reinterpret_cast<int*>(s_f + RT);           // [RT]
  int* const s_hi = s_lo + RT;                                  // [RT]
  float* const s_m = reinterpret_cast<float*>(s_hi + RT);       // [warps][RT]
  float* const s_l = s_m + kAttnWarps * RT;                     // [warps][RT]
  // A block's piece of its cluster's item, behind the warps' own: [RT][D], [RT][2].
  float* const s_part = reinterpret_cast<float*>(smem + C::kMerge);
  static_assert(C::kMerge + RT * (D + 2) * 4 <= C::kRingBytes || NT > 1, "the piece lies in the ring");

  int b, h, rt = 0, s0, left, first, count, len, n_rt;
  RowTile tile;
  if (ws.cluster > 0) {
    // ---- This block's steps of its cluster's item (one row tile a sequence).
    const int item = blockIdx.x / ws.cluster, rank = blockIdx.x - item * ws.cluster;
    b = item / cache.heads;
    h = item - b * cache.heads;
    a.queries(b, first, count);
    len = a.kv_len(b);
    n_rt = 1;
    tile.set(a, len, count, 0, RT);
    s0 = rank * tile.steps / ws.cluster;
    left = (rank + 1) * tile.steps / ws.cluster - s0;
  } else {
    // ---- This block's share: units [u0, u0 + left) of all.
    const Plan plan(a, RT);
    if (blockIdx.x == 0 && warp == 0) plan.store(a, RT, ws.prefix);
    // The join may be set up now; it waits for this grid's end before it reads.
    ptx::launch_dependents();
    const Shares shares(plan.units, ws.blocks);
    if (static_cast<int>(blockIdx.x) >= shares.active) return;
    const int u0 = shares.begin(blockIdx.x);
    left = shares.begin(blockIdx.x + 1) - u0;

    // ---- The item in which the share begins.
    int off;
    plan.find(a, RT, u0, b, off);
    a.queries(b, first, count);
    len = a.kv_len(b);
    n_rt = row_tiles(a, count, RT);
    const int per_head = head_units(a, b, RT);
    h = off / per_head;
    off -= h * per_head;
    tile.set(a, len, count, 0, RT);
    while (off >= tile.steps) {
      off -= tile.steps;
      tile.set(a, len, count, ++rt, RT);
    }
    s0 = off;
  }

  // q takes the sign of sm_scale.
  const float sign = a.sm_scale > 0.0f ? 1.0f : (a.sm_scale < 0.0f ? -1.0f : 0.0f);
  const bool q_vec = (reinterpret_cast<uintptr_t>(a.q) & 7) == 0 && a.q_token_stride % 4 == 0 && a.q_head_stride % 4 == 0;
  const int split = max(0, (TOK == 64 ? 6 : 5) - page_shift);
  const uint32_t ring = ptx::smem_u32(smem) + warp * C::kStages * C::kStage;

  while (left > 0) {
    const int n = min(left, tile.steps - s0);
    const int r0 = rt * RT;
    const int rows = min(count * a.ratio - r0, RT);

    // ---- Copies.  A lane keeps the page of a tile, or where pages are smaller
    // than tiles of one of its 2^split parts.
    const int tile_base = tile.lo + s0 * kStep + warp * TOK;
    const int64_t page_rows = static_cast<int64_t>(2 * cache.heads) << page_shift;
    const int64_t head_row = static_cast<int64_t>(h) << page_shift;
    const int64_t to_values = static_cast<int64_t>(cache.heads) << page_shift;
    int page_ids = -1;
    uint32_t live_blocks = 0u;  // MB bits a stage: which blocks of 16 tokens are there
    auto issue = [&](int k, int stage) {
      if (k < n) {
        const int in_ids = k & ((32 >> split) - 1);
        if (in_ids == 0) {
          const int tok = tile_base + (k + (lane >> split)) * kStep + ((lane & ((1 << split) - 1)) << page_shift);
          page_ids = -1;
          if (tok < tile.hi) {
            const int id = __ldg(a.page_table + b * a.table_stride + (tok >> page_shift));
            page_ids = id >= 0 && id < cache.pages ? id : -1;
          }
        }
        const uint32_t dst = ring + stage * C::kStage;
        const int tok0 = tile_base + k * kStep;
        uint32_t live = 0u;
        // Rows of one page are contiguous, keys and values apart: `blocks`
        // blocks of 16 tokens from row `row` on, at block `at` of the tile.
        auto copy = [&](auto blocks, int64_t row, int at) {
          constexpr int B = decltype(blocks)::value;
          const uint8_t* const k_src = cache.packed + (head_row + row) * RB + lane * 16;
          const uint8_t* const v_src = k_src + to_values * RB;
#pragma unroll
          for (int i = 0; i < B * 16 * RC; i += 32) {
            if ((B * 16 * RC) % 32 == 0 || i + lane < B * 16 * RC) {
              const int r = (i + lane) / RC, c = (i + lane) % RC;
              const uint32_t to = dst + at * 16 * RB + r * RB + chunk_of<RB>(r, c) * 16;
              cp16(to, k_src + i * 16);
              cp16(to + C::kCodes, v_src + i * 16);
            }
          }
          constexpr int kSc = B * 2 * NG, kZe = B * NG;  // chunks of the scales, of the zero points
#pragma unroll
          for (int i0 = 0; i0 < 2 * kSc; i0 += 32) {
            const int i = i0 + lane, kv = i / kSc, c = i % kSc;
            if (i < 2 * kSc)
              cp16(dst + C::kScaleAt + kv * C::kScales + at * 32 * NG + c * 16,
                   cache.scales + (head_row + row + kv * to_values) * NG + c * 8);
          }
          if (ASYM) {
#pragma unroll
            for (int i0 = 0; i0 < 2 * kZe; i0 += 32) {
              const int i = i0 + lane, kv = i / kZe, c = i % kZe;
              if (i < 2 * kZe)
                cp16(dst + C::kZeroAt + kv * C::kZeros + at * 16 * NG + c * 16,
                     cache.zeros + (head_row + row + kv * to_values) * NG + c * 16);
            }
          }
        };
        if (split == 0) {
          const int id = __shfl_sync(0xffffffffu, page_ids, in_ids);
          if (id >= 0) {
            live = (1u << MB) - 1;
            copy(std::integral_constant<int, MB>{}, id * page_rows + (tok0 & (cache.page_size - 1)), 0);
          }
        } else {
#pragma unroll 1
          for (int i = 0; i < MB; ++i) {
            const int id = __shfl_sync(0xffffffffu, page_ids, (in_ids << split) + ((i * 16) >> page_shift));
            if (id >= 0) {
              live |= 1u << i;
              copy(std::integral_constant<int, 1>{}, id * page_rows + ((tok0 + i * 16) & (cache.page_size - 1)), i);
            }
          }
        }
        live_blocks = (live_blocks & ~(((1u << MB) - 1) << (MB * stage))) | (live << (MB * stage));
      }
      cp_commit();
    };
    int all_lo = 0, all_hi = 0;  // tokens that every row of the tile sees
    uint2 qf[C::kQInRegs ? DB * 2 * NT : 1];
    float2 f[NT], qs1[NT];
    float o[DB][2][NT][4], zo[NG][NT][4];
    // Per row: the maximum of S / f, the same negated (0 before the first
    // token), and this lane's part of the sum.
    float m[NT][2];
    float2 nm[NT], l[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int c = 0; c < DB; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k) o[c][k >> 2][nt][k & 3] = 0.0f;
#pragma unroll
      for (int gi = 0; gi < NG; ++gi)
#pragma unroll
        for (int k = 0; k < 4; ++k) zo[gi][nt][k] = 0.0f;
      m[nt][0] = m[nt][1] = kNegInf;
      nm[nt] = l[nt] = make_float2(0.0f, 0.0f);
    }
    int x_run = 15;  // weights are held 2^x_run fold
    uint32_t bad_rows = 0u;  // rows (two bits an nt) that see a value scale that is not finite: so is their output

    int stage = 0, fill = 0;  // the tile in use, the one to be filled
#pragma unroll 1
    for (int k = 1 - C::kStages; k < n; ++k) {
      if (k == 0) {  // the first tiles are on their way: the queries now
        // ---- Queries of the tile: fp16 in fragment order, group sums, bounds.
        // Eight lanes a row, lane j of them with elements 4 j .. 4 j + 3 of each
        // block of 32.
#pragma unroll
        for (int rr = 0; rr < RT; rr += 4 * kAttnWarps) {
          if (rr + warp * 4 >= RT) break;
          const int r = rr + warp * 4 + (lane >> 3), j = lane & 7;
          const bool live = r < rows;
          const int i = live ? a.token_of(r0 + r) : 0;
          const int hq = h * a.ratio + (live ? r0 + r - i * a.ratio : 0);
          const T* qp = static_cast<const T*>(a.q) + (first + i) * a.q_token_stride + hq * a.q_head_stride + 4 * j;
          uint2 raw[DB];
#pragma unroll
          for (int c = 0; c < DB; ++c) {
            raw[c] = make_uint2(0u, 0u);
            if (live) raw[c] = load_four(reinterpret_cast<const uint16_t*>(qp + 32 * c), q_vec);
          }
          auto lo_of = [](uint32_t x) {
            return std::is_same<T, __half>::value ? f16_bits_to_float(x & 0xFFFFu) : __uint_as_float(x << 16);
          };
          auto hi_of = [](uint32_t x) {
            return std::is_same<T, __half>::value ? f16_bits_to_float(x >> 16) : __uint_as_float(x & 0xFFFF0000u);
          };
          float top = 0.0f;
#pragma unroll
          for (int c = 0; c < DB; ++c)
            top = fmaxf(top, fmaxf(fmaxf(fabsf(lo_of(raw[c].x)), fabsf(hi_of(raw[c].x))),
                                   fmaxf(fabsf(lo_of(raw[c].y)), fabsf(hi_of(raw[c].y)))));
#pragma unroll
          for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          // top in [2^e, 2^(e+1)); elements are scaled by 2^(14 - e).
          int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
          e = e < -100 ? -100 : e;
          const float scale = sign * __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
          // Elements 8 t + 2 s + k and 8 t + 2 s + k + 4 of a block are the two
          // halves of B register k of step s and lane t of the row's quad: lanes
          // 2 t and 2 t + 1 here hold the two, and store a step each.  k = 1
          // divided by 16.
          const int nt = r >> 3, gr = r & 7, odd = j & 1;
          float sum = 0.0f;
#pragma unroll
          for (int c = 0; c < DB; ++c) {
            const uint32_t x01 = pack_half2(lo_of(raw[c].x) * scale, hi_of(raw[c].x) * scale);
            const uint32_t x23 = pack_half2(lo_of(raw[c].y) * scale, hi_of(raw[c].y) * scale);
            sum += (f16_bits_to_float(x01 & 0xFFFFu) + f16_bits_to_float(x01 >> 16)) +
                   (f16_bits_to_float(x23 & 0xFFFFu) + f16_bits_to_float(x23 >> 16));
            const uint32_t y01 = mul_half2(x01, 0x2C003C00u), y23 = mul_half2(x23, 0x2C003C00u);
            const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? y01 : y23, 1);
            const uint32_t low = odd ? got : y01, high = odd ? y23 : got;
            reinterpret_cast<uint2*>(sq)[((c * 2 + odd) * NT + nt) * 32 + gr * 4 + (j >> 1)] =
                make_uint2(__byte_perm(low, high, 0x5410), __byte_perm(low, high, 0x7632));
            if (c % C::BPG == C::BPG - 1) {
#pragma unroll
              for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
              if (j == 0) s_qsum[(c / C::BPG) * RT + r] = -sum * (ASYM ? 0x1p-24f : 0x1p-21f);
              sum = 0.0f;
            }
          }
          if (j == 0) {
            int lo = 0, hi = 0;
            if (live) a.visible(len - count + i, len, lo, hi);
            s_lo[r] = lo;
            s_hi[r] = hi;
            // Positive, so that it may be applied after the maximum.
            const float f1 = __uint_as_float(static_cast<uint32_t>(127 + e - 14) << 23) * (fabsf(a.sm_scale) * 1.4426950408889634f);
            s_f[r] = sign == 0.0f ? 1.0f : fminf(fmaxf(f1, 0x1p-126f), 0x1p127f);
          }
        }
        __syncthreads();
        all_lo = s_lo[rows - 1];
        all_hi = s_hi[0];
        if (C::kQInRegs) {
#pragma unroll
          for (int i = 0; i < DB * 2 * NT; ++i) qf[i] = reinterpret_cast<const uint2*>(sq)[i * 32 + lane];
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          f[nt] = *reinterpret_cast<const float2*>(s_f + nt * 8 + 2 * t);
          qs1[nt] = *reinterpret_cast<const float2*>(s_qsum + nt * 8 + 2 * t);
        }
      }
      if (k >= 0) {
        cp_wait<C::kStages - 2>();
        __syncwarp();
      }
      issue(k + C::kStages - 1, fill);
      fill = fill == C::kStages - 1 ? 0 : fill + 1;
      if (k < 0) continue;
      const uint32_t st = ring + stage * C::kStage;
      const uint32_t live = (live_blocks >> (MB * stage)) & ((1u << MB) - 1);
      stage = stage == C::kStages - 1 ? 0 : stage + 1;
      const int base = tile_base + k * kStep;
      if (live == 0u) continue;  // past the end, or no page: the warp has no tokens here

      // ---- S^T / f = K Q^T by blocks of 16 tokens; s[mb][nt][half] holds
      // token mb * 16 + half * 8 + g and rows nt * 8 + 2 t, + 1.
      float2 s[MB][NT][2];
      {
        float acc[MB][NT][4];
#pragma unroll
        for (int c = 0; c < DB; ++c) {
          const int gi = c / C::BPG;
          uint32_t kr[2 * MB];
#pragma unroll
          for (int i = 0; i < MB; i += 2)
            ldsm4(st + (i * 16 + lane) * RB + chunk_of<RB>(lane, c) * 16, kr + 2 * i);
#pragma unroll
          for (int step = 0; step < 2; ++step) {
            uint32_t lo[2 * MB], hi[2 * MB];
#pragma unroll
            for (int i = 0; i < 2 * MB; ++i) {
              lo[i] = pick<ASYM>(kr[i], 0x000F000Fu);
              hi[i] = pick<ASYM>(kr[i], 0x00F000F0u);
              kr[i] >>= 8;
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const int at = (c * 2 + step) * NT + nt;
              const uint2 q2 = C::kQInRegs ? qf[C::kQInRegs ? at : 0]
                                           : ptx::lds64(ptx::smem_u32(sq) + (at * 32 + lane) * 8);
              if (c % C::BPG == 0 && step == 0) {
                float2 init = make_float2(0.0f, 0.0f);
                if (!ASYM) init = NG == 1 ? qs1[nt] : lds_f2(ptx::smem_u32(s_qsum + gi * RT + nt * 8 + 2 * t));
#pragma unroll
                for (int mb = 0; mb < MB; ++mb)
                  mma_from(acc[mb][nt], lo[2 * mb], lo[2 * mb + 1], hi[2 * mb], hi[2 * mb + 1], q2.x, q2.y, init.x, init.y);
              } else {
#pragma unroll
                for (int mb = 0; mb < MB; ++mb)
                  mma(acc[mb][nt], lo[2 * mb], lo[2 * mb + 1], hi[2 * mb], hi[2 * mb + 1], q2.x, q2.y);
              }
            }
          }
          if (c % C::BPG == C::BPG - 1) {
            float2 qz[NT];
            if (ASYM) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                qz[nt] = NG == 1 ? qs1[nt] : lds_f2(ptx::smem_u32(s_qsum + gi * RT + nt * 8 + 2 * t));
            }
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                const int tok = mb * 16 + half * 8 + g;
                const float k1 = f16_bits_to_float(lds_u16(st + C::kScaleAt + (tok * NG + gi) * 2));
                const float ks = fmaf(k1, 0x1p24f, k1 * 0.0f);  // an infinite scale gives NaN, as its values do
                const float2 ks2 = make_float2(ks, ks);
                float2 kz2 = make_float2(0.0f, 0.0f);
                if (ASYM) kz2.x = kz2.y = static_cast<float>(lds_u8(st + C::kZeroAt + tok * NG + gi));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  float2 x = make_float2(acc[mb][nt][2 * half], acc[mb][nt][2 * half + 1]);
                  if (ASYM) x = __ffma2_rn(kz2, qz[nt], x);
                  s[mb][nt][half] = gi == 0 ? __fmul2_rn(ks2, x) : __ffma2_rn(ks2, x, s[mb][nt][half]);
                }
              }
          }
        }
      }
      if (base < tile.first || base + TOK > tile.hi || live != (1u << MB) - 1) {
        // x_run follows the largest value scale of the tile, and W its products:
        // 0 for the tokens that no row sees, and in the place of a block that is
        // not there, which holds anything.
#pragma unroll
        for (int i = 0; i < TOK; i += 32) {
          const int tok = base + i + lane;
          if (((live >> ((i + lane) >> 4)) & 1u) != 0u && tok >= tile.first && tok < tile.hi) continue;
#pragma unroll
          for (int c = 0; c < NG; ++c) sts_u16(st + C::kScaleAt + C::kScales + ((i + lane) * NG + c) * 2, 0u);
        }
        __syncwarp();
      }
      // ---- Value scales of tokens 2t, 2t + 1 of each group of 8: NG words
      // hold the two tokens' scales; x_new follows the largest one's exponent.
      uint32_t vs[MB][2][NG];
      uint32_t vtop = 0u;
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t va = st + C::kScaleAt + C::kScales + (mb * 16 + half * 8 + 2 * t) * NG * 2;
          if constexpr (NG % 4 == 0) {
#pragma unroll
            for (int i = 0; i < NG / 4; ++i) {
              const uint4 w = ptx::lds128(va + 16 * i);
              vs[mb][half][4 * i] = w.x;
              vs[mb][half][4 * i + 1] = w.y;
              vs[mb][half][4 * i + 2] = w.z;
              vs[mb][half][4 * i + 3] = w.w;
            }
          } else if constexpr (NG == 2) {
            const uint2 w = ptx::lds64(va);
            vs[mb][half][0] = w.x;
            vs[mb][half][1] = w.y;
          } else {
#pragma unroll
            for (int i = 0; i < NG; ++i) vs[mb][half][i] = ptx::lds32(va + 4 * i);
          }
        }
      // ---- Mask, where some row does not see every token of the tile.
      const bool edge = base < all_lo || base + TOK > all_hi || live != (1u << MB) - 1;
      if (edge) {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int tok = base + mb * 16 + half * 8 + g;
            const bool here = ((live >> mb) & 1u) != 0u;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const int r = nt * 8 + 2 * t;
              if (!here || tok < s_lo[r] || tok >= s_hi[r]) s[mb][nt][half].x = kNegInf;
              if (!here || tok < s_lo[r + 1] || tok >= s_hi[r + 1]) s[mb][nt][half].y = kNegInf;
            }
            // A value scale that is not finite counts as 0, so that hidden
            // tokens add nothing; a row that sees one is remembered.
#pragma unroll
            for (int i = 0; i < NG; ++i) {
              const uint32_t w = vs[mb][half][i];
              vs[mb][half][i] = ((w & 0x7C00u) != 0x7C00u ? w & 0xFFFFu : 0u) |
                                ((w & 0x7C000000u) != 0x7C000000u ? w & 0xFFFF0000u : 0u);
              vtop = attn::max_half2(vtop, vs[mb][half][i]);
              const uint32_t own = lds_u16(st + C::kScaleAt + C::kScales + ((mb * 16 + half * 8 + g) * NG + i) * 2);
              if ((own & 0x7C00u) == 0x7C00u) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  if (s[mb][nt][half].x != kNegInf) bad_rows |= 1u << (2 * nt);
                  if (s[mb][nt][half].y != kNegInf) bad_rows |= 2u << (2 * nt);
                }
              }
            }
          }
      } else {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int i = 0; i < NG; ++i) vtop = attn::max_half2(vtop, vs[mb][half][i]);
      }
      const int e_tile = static_cast<int>(__reduce_max_sync(0xffffffffu, max(vtop & 0xFFFFu, vtop >> 16)) >> 10);
      const int x_new = min(x_run, 29 - e_tile);
      // ---- Running maxima.
      float mx[NT][2];
      bool grew = x_new != x_run;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float x = kNegInf;
#pragma unroll
          for (int mb = 0; mb < MB; ++mb)
            x = fmaxf(x, j == 0 ? fmaxf(s[mb][nt][0].x, s[mb][nt][1].x) : fmaxf(s[mb][nt][0].y, s[mb][nt][1].y));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          mx[nt][j] = fmaxf(m[nt][j], x);
          grew = grew || mx[nt][j] != m[nt][j];
        }
      if (__any_sync(0xffffffffu, grew)) {
        const float shrink = __uint_as_float(static_cast<uint32_t>(127 + x_new - x_run) << 23);
        x_run = x_new;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float2 al;
          al.x = m[nt][0] == mx[nt][0] ? 1.0f : ex2((m[nt][0] - mx[nt][0]) * f[nt].x);
          al.y = m[nt][1] == mx[nt][1] ? 1.0f : ex2((m[nt][1] - mx[nt][1]) * f[nt].y);
          l[nt] = __fmul2_rn(l[nt], al);
          m[nt][0] = mx[nt][0];
          m[nt][1] = mx[nt][1];
          nm[nt].x = m[nt][0] == kNegInf ? 0.0f : -m[nt][0];
          nm[nt].y = m[nt][1] == kNegInf ? 0.0f : -m[nt][1];
          al.x *= shrink;
          al.y *= shrink;
#pragma unroll
          for (int c = 0; c < DB; ++c)
#pragma unroll
            for (int k2 = 0; k2 < 8; ++k2) o[c][k2 >> 2][nt][k2 & 3] *= (k2 & 1) ? al.y : al.x;
#pragma unroll
          for (int gi = 0; gi < NG; ++gi)
#pragma unroll
            for (int k2 = 0; k2 < 4; ++k2) zo[gi][nt][k2] *= (k2 & 1) ? al.y : al.x;
        }
      }
      // ---- P, its sum, and P 2^x_run in fp16 as the B operand of tokens x rows.
      // The maximum is taken off before the product with f, so that its own
      // weight is 1 whatever its size: S f - (m f) in one FMA is off by the
      // rounding of m f, which passes 1 from |m f| = 2^24 on (and W fp16's range).
      const float xf = __uint_as_float(static_cast<uint32_t>(127 + x_run) << 23);
      const float2 xf2 = make_float2(xf, xf);
      uint32_t pt[MB][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            float2 p = __fmul2_rn(__fadd2_rn(s[mb][nt][half], nm[nt]), f[nt]);
            p.x = ex2(p.x);
            p.y = ex2(p.y);
            l[nt] = __fadd2_rn(l[nt], p);
            p = __fmul2_rn(p, xf2);
            pt[mb][nt][half] = transpose8x8(pack_half2(p.x, p.y));
          }
      // ---- O^T += V^T W^T with W = P times the value scales, group by group.
      uint32_t pb[MB][NT][2];
#pragma unroll
      for (int c = 0; c < DB; ++c) {
        const int gi = c / C::BPG;
        if (c % C::BPG == 0) {
#pragma unroll
          for (int mb = 0; mb < MB; ++mb) {
            uint32_t z[2] = {0x00080008u, 0x00080008u};
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              // Scales gi and NG + gi of the words' 2 NG: the two tokens'.
              constexpr uint32_t kPick[4] = {0x5410u, 0x7610u, 0x5432u, 0x7632u};
              const uint32_t w = __byte_perm(vs[mb][half][gi / 2], vs[mb][half][(NG + gi) / 2],
                                             kPick[(gi & 1) * 2 + ((NG + gi) & 1)]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) pb[mb][nt][half] = mul_half2(pt[mb][nt][half], w);
              if (ASYM) {
                const uint32_t za = st + C::kZeroAt + C::kZeros + (mb * 16 + half * 8 + 2 * t) * NG + gi;
                z[half] = lds_u8(za) | (lds_u8(za + NG) << 16);
              }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma(zo[gi][nt], z[0], z[0], z[1], z[1], pb[mb][nt][0], pb[mb][nt][1]);
          }
        }
        uint32_t vr[2 * MB];
#pragma unroll
        for (int i = 0; i < MB; i += 2)
          ldsm4t(st + C::kCodes + (i * 16 + lane) * RB + chunk_of<RB>(lane, c) * 16, vr + 2 * i);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t lo[2 * MB], hi[2 * MB];
#pragma unroll
          for (int i = 0; i < 2 * MB; ++i) {
            lo[i] = pick<ASYM>(vr[i], 0x000F000Fu);
            hi[i] = pick<ASYM>(vr[i], 0x00F000F0u);
            vr[i] >>= 8;
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
              mma(o[c][half][nt], lo[2 * mb], hi[2 * mb], lo[2 * mb + 1], hi[2 * mb + 1], pb[mb][nt][0], pb[mb][nt][1]);
        }
      }
    }
    cp_wait<0>();

    // ---- Join the warps, then store the item's result or the piece's sums.
    if (__any_sync(0xffffffffu, bad_rows != 0u)) {
#pragma unroll
      for (int o2 = 4; o2 < 32; o2 <<= 1) bad_rows |= __shfl_xor_sync(0xffffffffu, bad_rows, o2);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float sum = j == 0 ? l[nt].x : l[nt].y;
#pragma unroll
        for (int o2 = 4; o2 < 32; o2 <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o2);
        if (g == 0) {  // from here on the maxima are S's own
          s_m[warp * RT + nt * 8 + 2 * t + j] = m[nt][j] * (j == 0 ? f[nt].x : f[nt].y);
          s_l[warp * RT + nt * 8 + 2 * t + j] = sum;
        }
      }
    const bool whole = ws.cluster == 0 && n == tile.steps;
    const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (s0 == 0 ? 1 : 0);
    float* const piece_o = ws.cluster > 0 ? s_part : ws.o + slot * RT * D;
    float* const piece_ml = ws.cluster > 0 ? s_part + RT * D : ws.ml + slot * RT * 2;
    float* const buf = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      __syncthreads();  // tiles read (first time), or the last rows' sums read
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = nt * 8 + 2 * t + j;
        const float mine = s_m[warp * RT + r];
        float top = s_m[r];
#pragma unroll
        for (int w = 1; w < kAttnWarps; ++w) top = fmaxf(top, s_m[w * RT + r]);
        // Codes are 2^-24 times themselves, weights 2^x_run.
        float scale =
            (mine == top ? 1.0f : ex2(mine - top)) * __uint_as_float(static_cast<uint32_t>(127 + 24 - x_run) << 23);
        if ((bad_rows >> (2 * nt + j)) & 1u) scale = __int_as_float(0x7FC00000);
        float* dst = buf + (warp * 8 + 2 * t + j) * C::kMergePitch + 4 * g;
#pragma unroll
        for (int c = 0; c < DB; ++c) {
          const float z = zo[c / C::BPG][nt][j];
          float4 v;
          v.x = (o[c][0][nt][j] - z) * scale;
          v.y = (o[c][0][nt][2 + j] * 0.0625f - z) * scale;
          v.z = (o[c][1][nt][j] - z) * scale;
          v.w = (o[c][1][nt][2 + j] * 0.0625f - z) * scale;
          *reinterpret_cast<float4*>(dst + 32 * c) = v;
        }
      }
      __syncthreads();
#pragma unroll 1
      for (int k = tid; k < 8 * (D / 4); k += kAttnThreads) {
        const int rr = k / (D / 4), d = (k % (D / 4)) * 4;
        const int r = nt * 8 + rr;
        if (r >= rows) continue;
        float4 v = *reinterpret_cast<const float4*>(buf + rr * C::kMergePitch + d);
        float top = s_m[r];
#pragma unroll
        for (int w = 1; w < kAttnWarps; ++w) {
          const float4 x = *reinterpret_cast<const float4*>(buf + (w * 8 + rr) * C::kMergePitch + d);
          v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
          top = fmaxf(top, s_m[w * RT + r]);
        }
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w) {
          const float mw = s_m[w * RT + r];
          sum += s_l[w * RT + r] * (mw == top ? 1.0f : ex2(mw - top));
        }
        if (whole) {
          const int i = a.token_of(r0 + r);
          const int at = (first + i) * a.q_heads + h * a.ratio + (r0 + r - i * a.ratio);
          const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
          T* out = static_cast<T*>(a.out) + static_cast<int64_t>(at) * D + d;
          alignas(8) T four[4];
          store_as(four, v.x * inv);
          store_as(four + 1, v.y * inv);
          store_as(four + 2, v.z * inv);
          store_as(four + 3, v.w * inv);
          *reinterpret_cast<uint2*>(out) = *reinterpret_cast<const uint2*>(four);
          if (d == 0 && a.lse != nullptr)
            a.lse[at] = sum == 0.0f ? kNegInf : (top + log2f(sum)) * 0.6931471805599453f;
        } else {
          *reinterpret_cast<float4*>(piece_o + r * D + d) = v;
          if (d == 0) *reinterpret_cast<float2*>(piece_ml + r * 2) = make_float2(top, sum);
        }
      }
    }
    __syncthreads();

    // ---- The next item.
    left -= n;
    if (left == 0) break;
    s0 = 0;
    do {
      if (++rt == n_rt) {
        rt = 0;
        if (++h == cache.heads) {
          h = 0;
          do {
            ++b;
            a.queries(b, first, count);
            len = a.kv_len(b);
            n_rt = row_tiles(a, count, RT);
          } while (n_rt == 0);
        }
      }
      tile.set(a, len, count, rt, RT);
    } while (tile.steps == 0);
  }

  if constexpr (NT == 1) {
    if (ws.cluster > 0) {
      // ---- The cluster's pieces together, a row of the item to a warp.
      const int rank = blockIdx.x % ws.cluster;
      const int rows = min(count * a.ratio, RT);
      if (rank * tile.steps / ws.cluster == (rank + 1) * tile.steps / ws.cluster) {  // no step was this block's
        for (int k = tid; k < RT * D; k += kAttnThreads) s_part[k] = 0.0f;
        if (tid < RT) *reinterpret_cast<float2*>(s_part + RT * D + 2 * tid) = make_float2(kNegInf, 0.0f);
      }
      cluster_sync();
      for (int r = warp * ws.cluster + rank; r < rows; r += kAttnWarps * ws.cluster) {
        const uint32_t at = ptx::smem_u32(s_part);
        float2 ml = make_float2(kNegInf, 0.0f);
        if (lane < ws.cluster) ml = ld_cluster_f2(at + (RT * D + 2 * r) * 4, lane);
        float top = ml.x;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        top = __shfl_sync(0xffffffffu, top, 0);
        const float w = ml.x == top ? 1.0f : ex2(ml.x - top);
        float sum = ml.y * w;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        sum = __shfl_sync(0xffffffffu, sum, 0);
        const int i = a.token_of(r);
        const int out_row = (first + i) * a.q_heads + h * a.ratio + r - i * a.ratio;
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        for (int d0 = 0; d0 < D; d0 += 128) {
          const int d = d0 + lane * 4;
          float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          for (int p = 0; p < ws.cluster; ++p) {
            const float wp = __shfl_sync(0xffffffffu, w, p);
            if (d < D) {
              const float4 x = ld_cluster_f4(at + (r * D + d) * 4, p);
              v.x = fmaf(wp, x.x, v.x);
              v.y = fmaf(wp, x.y, v.y);
              v.z = fmaf(wp, x.z, v.z);
              v.w = fmaf(wp, x.w, v.w);
            }
          }
          if (d < D) {
            alignas(8) T four[4];
            store_as(four, v.x * inv);
            store_as(four + 1, v.y * inv);
            store_as(four + 2, v.z * inv);
            store_as(four + 3, v.w * inv);
            *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + static_cast<int64_t>(out_row) * D + d) =
                *reinterpret_cast<const uint2*>(four);
          }
        }
        if (lane == 0 && a.lse != nullptr)
          a.lse[out_row] = sum == 0.0f ? kNegInf : (top + log2f(sum)) * 0.6931471805599453f;
      }
      cluster_sync();  // no block leaves while another reads its shared memory
    }
  }
}

// Joins the pieces of split items and writes the rows that see nothing, where
// sequences have few row tiles: every row's warp walks those before its own.  A
// query row of one head is given to `wpr` of the block's warps (1 when there
// are rows enough to fill the GPU, else all of them), a share of the pieces
// to each.
template <typename T>
__global__ void __launch_bounds__(256)
    attention_join_kernel(const __grid_constant__ AttentionArgs a, const AttentionSpace ws, const int RT, const int wpr) {
  constexpr float kNegInf = -__builtin_huge_valf();
  __shared__ float part[8][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int D = a.cache.head_dim;
  const int index = blockIdx.x * (8 / wpr) + warp / wpr;
  const int tok = index / a.q_heads;
  const int hq = index - tok * a.q_heads;
  int b = -1;
  if (tok < a.rows) b = a.sequence_of(tok);
  int r = 0, before = 0, per_head = 0, p_end = 0, p0 = 0, steps = 0, rt = 0;
  if (b >= 0) {
    int first, count;
    a.queries(b, first, count);
    const int len = a.kv_len(b);
    r = (tok - first) * a.ratio + hq % a.ratio;
    rt = r / RT;
    const int n = row_tiles(a, count, RT);
    for (int i = 0; i < n; ++i) {
      RowTile tile;
      tile.set(a, len, count, i, RT);
      if (i < rt) before += tile.steps;
      if (i == rt) steps = tile.steps;
      per_head += tile.steps;
    }
  }
  ptx::grid_dependency_wait();
  if (steps > 0) {
    const Shares shares(ws.prefix[a.batch], ws.blocks);
    const int begin = ws.prefix[b] + (hq / a.ratio) * per_head + before;
    p0 = shares.block_of(begin);
    p_end = shares.block_of(begin + steps - 1) + 1;
  }
  const bool join = p_end - p0 > 1;
  const bool empty = b >= 0 && steps == 0;
  const int rr = r - rt * RT;
  // The first piece ends its block's share, every other one begins its own.
  auto slot = [&](int p) { return static_cast<int64_t>(2 * p + (p == p0 ? 1 : 0)) * RT + rr; };
  float4 v[2] = {make_float4(0.0f, 0.0f, 0.0f, 0.0f), make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
  float top = kNegInf, sum = 0.0f;
  if (join) {
    const int pieces = p_end - p0;
    for (int base = 0; base < pieces; base += 32) {
      // A lane's piece of these 32, and the first four of the warp's own.
      const int here = min(pieces - base, 32);
      float2 ml = make_float2(kNegInf, 0.0f);
      if (lane < here) ml = *reinterpret_cast<const float2*>(ws.ml + slot(p0 + base + lane) * 2);
      float4 x[4][2];
      auto load = [&](int k0) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int d = i * 128 + lane * 4, q = k0 + k * wpr;
            x[k][i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (q < here && d < D) x[k][i] = *reinterpret_cast<const float4*>(ws.o + slot(p0 + base + q) * D + d);
          }
      };
      load(warp % wpr);
      float m = ml.x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      m = fmaxf(m, top);
      const float old = top == m ? 1.0f : attn::ex2(top - m);
      const float w = ml.x == m ? 1.0f : attn::ex2(ml.x - m);
      float l = ml.y * w;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      top = m;
      sum = fmaf(sum, old, l);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        v[i].x *= old; v[i].y *= old; v[i].z *= old; v[i].w *= old;
      }
      for (int k0 = warp % wpr; k0 < here; k0 += 4 * wpr) {
        if (k0 >= 4 * wpr) load(k0);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float wk = __shfl_sync(0xffffffffu, w, (k0 + k * wpr) & 31);
#pragma unroll
          for (int i = 0; i < 2; ++i) {  // what is not there is 0
            v[i].x = fmaf(wk, x[k][i].x, v[i].x);
            v[i].y = fmaf(wk, x[k][i].y, v[i].y);
            v[i].z = fmaf(wk, x[k][i].z, v[i].z);
            v[i].w = fmaf(wk, x[k][i].w, v[i].w);
          }
        }
      }
    }
  }
  if (wpr > 1) {  // one row a block: join is the same for all its threads
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int d = i * 128 + lane * 4;
      *reinterpret_cast<float4*>(&part[warp][d]) = v[i];
    }
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int d = i * 128 + lane * 4;
      for (int w = 1; w < 8; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(&part[w][d]);
        v[i].x += x.x; v[i].y += x.y; v[i].z += x.z; v[i].w += x.w;
      }
    }
  }
  if (!join && !empty) return;
  const int64_t at = index;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int d = i * 128 + lane * 4;
    if (d < D) {
      alignas(8) T four[4];
      store_as(four, v[i].x * inv);
      store_as(four + 1, v[i].y * inv);
      store_as(four + 2, v[i].z * inv);
      store_as(four + 3, v[i].w * inv);
      *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + at * D + d) = *reinterpret_cast<const uint2*>(four);
    }
  }
  if (lane == 0 && a.lse != nullptr)
    a.lse[at] = sum == 0.0f ? kNegInf : (top + log2f(sum)) * 0.6931471805599453f;
}

// The join by items, where a sequence has several row tiles (and for the large
// ones of the tcgen05 kernel): block (c, i) joins rows [8 i, 8 i + 8) of the item
// that begins in share c and goes on in the next ones, if there is one; blocks
// (ws.blocks + b, i) write the rows of sequence b's tiles that see nothing.
template <typename T>
__global__ void __launch_bounds__(256)
    attention_join_items_kernel(const __grid_constant__ AttentionArgs a, const AttentionSpace ws, const int RT) {
  constexpr float kNegInf = -__builtin_huge_valf();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int D = a.cache.head_dim;
  const int rr = blockIdx.y * 8 + warp;  // row of the tile
  auto store = [&](int at, int d, float4 v) {
    alignas(8) T four[4];
    store_as(four, v.x);
    store_as(four + 1, v.y);
    store_as(four + 2, v.z);
    store_as(four + 3, v.w);
    *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + static_cast<int64_t>(at) * D + d) =
        *reinterpret_cast<const uint2*>(four);
  };
  if (static_cast<int>(blockIdx.x) >= ws.blocks) {
    const int b = blockIdx.x - ws.blocks;
    int first, count;
    a.queries(b, first, count);
    const int len = a.kv_len(b), n = row_tiles(a, count, RT);
    ptx::grid_dependency_wait();
    for (int rt = 0; rt < n; ++rt) {
      RowTile tile;
      tile.set(a, len, count, rt, RT);
      const int r = rt * RT + rr;
      if (tile.steps > 0 || r >= count * a.ratio) continue;
      const int i = a.token_of(r);
      for (int h = 0; h < a.cache.heads; ++h) {
        const int at = (first + i) * a.q_heads + h * a.ratio + r - i * a.ratio;
        for (int d = lane * 4; d < D; d += 128) store(at, d, make_float4(0.0f, 0.0f, 0.0f, 0.0f));
        if (lane == 0 && a.lse != nullptr) a.lse[at] = kNegInf;
      }
    }
    return;
  }
  ptx::grid_dependency_wait();
  const Shares shares(ws.prefix[a.batch], ws.blocks);
  const int c = blockIdx.x;
  if (c + 1 >= shares.active) return;
  const int begin = shares.begin(c), last = shares.begin(c + 1) - 1;
  int b = 0, hi_b = a.batch;  // the sequence of unit `last`
  while (hi_b - b > 1) {
    const int mid = (b + hi_b) >> 1;
    if (ws.prefix[mid] <= last) b = mid; else hi_b = mid;
  }
  const int in_seq = last - ws.prefix[b];
  int first, count;
  a.queries(b, first, count);
  const int len = a.kv_len(b), n = row_tiles(a, count, RT);
  // Its head and row tile, a lane to each of 32 tiles at a time.
  int per_head = 0;
  for (int i = lane; i < n; i += 32) {
    RowTile tile;
    tile.set(a, len, count, i, RT);
    per_head += tile.steps;
  }
  per_head = __reduce_add_sync(0xffffffffu, per_head);
  const int h = in_seq / per_head, off = in_seq - h * per_head;
  int rt = 0, before = 0, steps = 0;
  for (int i0 = 0, sum = 0; i0 < n; i0 += 32) {
    RowTile tile;
    tile.steps = 0;
    if (i0 + lane < n) tile.set(a, len, count, i0 + lane, RT);
    int upto = tile.steps;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, sum + upto > off);
    if (past != 0u) {
      const int at = __ffs(past) - 1;
      rt = i0 + at;
      steps = __shfl_sync(0xffffffffu, tile.steps, at);
      before = sum + __shfl_sync(0xffffffffu, upto, at) - steps;
      break;
    }
    sum += __shfl_sync(0xffffffffu, upto, 31);
  }
  const int item = last - off + before;
  if (item < begin || item + steps <= last + 1) return;  // begun earlier, or ends here
  const int p_end = shares.block_of(item + steps - 1) + 1;
  const int r = rt * RT + rr;
  if (r >= count * a.ratio) return;
  auto slot = [&](int p) { return static_cast<int64_t>(2 * p + (p == c ? 1 : 0)) * RT + rr; };
  float top = kNegInf, sum = 0.0f;
  for (int p = c; p < p_end; ++p) top = fmaxf(top, ws.ml[slot(p) * 2]);
  float4 v[2] = {make_float4(0.0f, 0.0f, 0.0f, 0.0f), make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
  for (int p = c; p < p_end; ++p) {
    const int64_t s = slot(p);
    const float mp = ws.ml[s * 2];
    const float w = mp == top ? 1.0f : attn::ex2(mp - top);
    sum = fmaf(w, ws.ml[s * 2 + 1], sum);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int d = i * 128 + lane * 4;
      if (d < D) {
        const float4 x = *reinterpret_cast<const float4*>(ws.o + s * D + d);
        v[i].x = fmaf(w, x.x, v[i].x);
        v[i].y = fmaf(w, x.y, v[i].y);
        v[i].z = fmaf(w, x.z, v[i].z);
        v[i].w = fmaf(w, x.w, v[i].w);
      }
    }
  }
  const int i = a.token_of(r);
  const int at = (first + i) * a.q_heads + h * a.ratio + r - i * a.ratio;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int d = k * 128 + lane * 4;
    if (d < D) store(at, d, make_float4(v[k].x * inv, v[k].y * inv, v[k].z * inv, v[k].w * inv));
  }
  if (lane == 0 && a.lse != nullptr)
    a.lse[at] = sum == 0.0f ? kNegInf : (top + log2f(sum)) * 0.6931471805599453f;
}

// ---- Host side ------------------------------------------------------------

// Query rows of a tile, by the rows of an average sequence (query tokens times
// ratio): 8 for up to 8; else 32 where an even number of tiles of 16 holds them
// and 16 where an odd one does.  16 for 256 elements, where the accumulators of
// 32 rows do not fit in registers, and for groups of 32 of 64 or 128 elements,
// where they spill (up to 800 bytes a thread).  32 sequences of 4096 tokens, 8
// heads, in us as tiles of 32 / of 16 rows:
//   rows                  32          48          64          96
//   128, one group      98 / 105   169 / 144   173 / 185   244 / 266
//   128, groups of 64  112 / 124   199 / 176   201 / 226   289 / 335
//   96, one group       83 / 90    141 / 122   145 / 157   205 / 225
//   64, one group       74 / 73    131 / 98    133 / 126   180 / 180
//   96, groups of 32   102 / 108   182 / 147   185 / 190   264 / 273
//   128, groups of 32  196 / 153   362 / 223   369 / 288   538 / 426
//   64, groups of 32   106 / 79    182 / 108   187 / 138   262 / 197
__host__ __device__ constexpr bool attention_has_tile_32(int head_dim, int group) {
  return head_dim <= 128 && (group != 32 || head_dim == 96);
}
inline int attention_row_tile(int head_dim, int group, int64_t rows, int64_t batch, int ratio) {
  const int64_t r = (rows * ratio + batch - 1) / batch;
  if (r <= 8) return 8;
  return !attention_has_tile_32(head_dim, group) || (r + 15) / 16 % 2 == 1 ? 16 : 32;
}

// Sets a kernel's dynamic shared memory once on each device.
template <auto kKernel>
cudaError_t allow_shared(int bytes) {
  static std::atomic<bool> done[64];  // one array for each kernel
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev].store(true, std::memory_order_release);
  return e;
}

// The parts of a workspace.
inline AttentionSpace attention_space(void* workspace, int batch, int blocks, int rt, int head_dim) {
  AttentionSpace ws;
  uint8_t* p = static_cast<uint8_t*>(workspace);
  ws.blocks = blocks;
  ws.cluster = 0;
  ws.prefix = reinterpret_cast<int32_t*>(p);
  ws.o = reinterpret_cast<float*>(p + attention_prefix_bytes(batch));
  ws.ml = ws.o + 2LL * blocks * rt * head_dim;
  return ws;
}
inline size_t attention_space_bytes(int64_t batch, int64_t blocks, int rt, int head_dim) {
  return attention_prefix_bytes(batch) + (2 * blocks * rt * (head_dim + 2) * sizeof(float) + 255) / 256 * 256;
}

// The joins, launched early where the kernel before lets them (they wait for
// its end before they read).
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
template <typename T>
cudaError_t launch_attention_join(const AttentionArgs& a, const AttentionSpace& ws, int rt, cudaStream_t stream) {
  const int rows = a.rows * a.q_heads;
  const int wpr = rows <= 2048 ? 8 : 1;
  return launch_dependent(attention_join_kernel<T>, dim3(wpr == 8 ? rows : (rows + 7) / 8), stream, a, ws, rt, wpr);
}
template <typename T>
cudaError_t launch_attention_join_items(const AttentionArgs& a, const AttentionSpace& ws, int rt, cudaStream_t stream) {
  return launch_dependent(attention_join_items_kernel<T>, dim3(ws.blocks + a.batch, rt / 8), stream, a, ws, rt);
}

// Blocks of a cluster for each item, or 0 for shares of all units: sequences of
// equally many queries, one row tile of 8 each, and room in the table for at
// most four steps a block, all items' blocks at once on the GPU (or items enough
// for one block each).
inline int attention_cluster(const AttentionArgs& a, int rt, int blocks) {
  if (rt != 8 || a.q_starts != nullptr || (a.rows / a.batch) * a.ratio > rt) return 0;
  const int64_t items = static_cast<int64_t>(a.batch) * a.cache.heads;
  const int step = attention_step(a.cache.head_dim, rt);
  const int64_t steps = (static_cast<int64_t>(a.max_pages) * a.cache.page_size + step - 1) / step;
  int c = 8;
  while (c > 1 && (items * c > blocks || c >= 2 * steps)) c /= 2;
  return steps <= 4 * c && items <= (1 << 24) ? c : 0;
}

template <class C>
int attention_blocks() {
  return num_sms() * C::kBlocks;
}

template <typename T, class C>
cudaError_t launch_attention_cfg(const AttentionArgs& a, void* workspace, cudaStream_t stream) {
  AttentionSpace ws = attention_space(workspace, a.batch, attention_blocks<C>(), C::RT, C::D);
  constexpr auto kernel = attention_mma_kernel<T, C>;
  cudaError_t e = allow_shared<kernel>(C::kSmem);
  if (e != cudaSuccess) return e;
  int shift = 0;
  while ((1 << shift) < a.cache.page_size) ++shift;
  ws.cluster = attention_cluster(a, C::RT, ws.blocks);
  if (ws.cluster > 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.batch) * a.cache.heads * ws.cluster);
    cfg.blockDim = dim3(kAttnThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ws.cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, ws, shift);
  }
  kernel<<<ws.blocks, kAttnThreads, C::kSmem, stream>>>(a, ws, shift);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // Rows walk the row tiles of their sequence in the join by rows (and blocks
  // the pieces of an item in the one by items): 4096 rows of 64 heads of 256 on
  // 4096 tokens 41.9 ms by rows, 4.3 ms by items; 4 rows of 64 heads of 128 on
  // 131071 tokens, one row tile, 92 and 104 us.
  const int64_t rows = static_cast<int64_t>(a.rows) * a.ratio;
  const bool by_items = rows > static_cast<int64_t>(C::RT) * a.batch || rows > 64 * C::RT;
  return by_items ? launch_attention_join_items<T>(a, ws, C::RT, stream)
                  : launch_attention_join<T>(a, ws, C::RT, stream);
}

// Calls f with the configuration for a cache and row tile; false if none.
template <int D, int GROUP, class F>
bool with_attention_cfg(bool asym, int rt, F&& f) {
  if (rt == 8) {
    if (asym) f(AttnCfg<D, GROUP, 1, true>{}); else f(AttnCfg<D, GROUP, 1, false>{});
    return true;
  }
  if (rt == 16) {
    if (asym) f(AttnCfg<D, GROUP, 2, true>{}); else f(AttnCfg<D, GROUP, 2, false>{});
    return true;
  }
  if constexpr (attention_has_tile_32(D, GROUP)) {
    if (rt == 32) {
      if (asym) f(AttnCfg<D, GROUP, 4, true>{}); else f(AttnCfg<D, GROUP, 4, false>{});
      return true;
    }
  }
  return false;
}

}  // namespace int4lib
