// Attention over the 4-bit cache for many query rows (prompts in chunks), on
// the tcgen05 tensor cores (sm_100a).
//
// Same operator and split over the lengths as the kernel for few rows
// (cache_attention.cuh); here a block's item is 256 query rows of one key/value
// head, two MMA tiles of 128 rows that share every tile of 128 tokens, taken in
// two halves:
//   S_m = Q_m K^T         128 x 64 x D, both operands in shared memory
//   O_m += W_m V          128 x D x 64, W from tensor memory
// Tensor memory holds two buffers of S for each m (fp32, 64 columns; W_m, fp16,
// overlays the first half of its S once that has been read) and O_0, O_1 (D
// columns each).  So S of the next half tile is ready before the softmax of
// this one has ended: with one buffer of 128 columns, S waited for W V of the
// same columns, and the chain S, softmax, W V took 2.2 times as long.
//
// Roles of the block's 16 warps:
//   warps 0-3    warp 0 issues the MMAs; the others only lend their registers
//   warps 4-7    expand codes: thread t owns token t of the tile, its key row
//                and its value row
//   warps 8-15   softmax: thread r of group m owns query row r of tile m
//
// q enters in fp16 after a power-of-two scaling of its row (see
// cache_attention.cuh).  With one group a head, keys and values are the integers
// n - z, exactly: the token's key scale multiplies its column of S in fp32, its
// value scale the weight, W = 2^x P s rounded to fp16 once (x: a power of two
// that keeps it in range).  With several groups, the power of two u of the
// token's largest scale takes the scale's place there, and the elements are
// (n - z) s / u: the sum of two fp16 numbers, a product each, which hold all of
// their at most 16 bits (to 2^-20 u, where the scales of a token's groups differ
// by more than 2^9); the second takes the place of the second stage in shared
// memory.  Values for bf16 outputs are rounded to one fp16 number, 2^-11 beside
// the output's 2^-8; for fp16 outputs that would add half the error that they
// have (3.0e-4 of the output's norm, 2.4e-4 in two parts; 2048 rows in groups of
// 32 on 16384 tokens: 327 us and 401 us).  S, the maximum and
// the sum are fp32; O is fp32 in tensor memory.  Weights are taken relative to a
// reference that follows the row's maximum only when that has passed it by
// more than a factor 2^8: a half tile's weights are computed at once under the
// old reference, and only where that turns out too far behind, or some row
// does not see all tokens, with the maximum first.
//
// What bounds it.  1789 queries of two prompts on 8192 and 6757 tokens, 64 heads
// of 128 on 8: 580 us, of 256 us at the tensor pipe's measured rate (the pipe is
// active in 37 % of the cycles).  Copies of the kernel that leave parts out took
// 250 us with the MMAs alone and 440 us with the hand-overs between S, softmax and
// W V and a trivial softmax: each change between the two products drains the pipe
// for about 300 cycles, and tensor memory has no room for longer products.
// With groups it is the second products, half as many MMAs again: 8 heads of 128,
// 2048 rows of one sequence of 16384 tokens take 265 us in one group, 327 us in
// groups of 32 (401 us with the values in two parts), alike in groups of 64.
//
// Inside blocks of 8 elements, keys and queries are stored in the order 0, 4,
// 1, 5, 2, 6, 3, 7 in which a code word expands pair by pair; O's columns come
// out in that order and are put right when they are stored.
#pragma once

#include <type_traits>

#include "cache.cuh"
#include "cache_attention.cuh"
#include "internal.h"
#include "sm100_ptx.cuh"

namespace int4lib {

namespace {

constexpr int kRows = kPrefillRowTile;  // query rows of an item
constexpr int kTok = 128;      // tokens of a tile
constexpr int kThreadsP = 512;
constexpr int kScaleRing = 4;  // tiles of column scales held
constexpr float kGrow = 8.0f;  // log2 of how far a weight may pass the maximum it is relative to
// log2 of exponentials up to which the reference is taken off in the same FMA,
// rounded: by at most 2^-4, for which fp16's range has room beside kGrow.
constexpr float kNear = 0x1p20f;
constexpr uint64_t kWaitNs = 250000000ull;  // far above any legitimate wait

struct Bars {
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t sc_full[kScaleRing];
  uint64_t s_full[2][2], w_full[2][2];  // per row tile and buffer: S computed; W stored
  uint64_t o_done[2];                   // per row tile: W V added
  uint64_t q_full, o_full;        // per item
  uint64_t drain;
};

template <int D>
struct Smem {
  static constexpr int kSub = 128 * 128;         // 128 rows of 128 bytes: 64 elements, 128-byte swizzle
  static constexpr int kTile = (D + 63) / 64 * kSub;  // 128 rows of D elements
  static constexpr int offQ = 0;                 // two row tiles
  static constexpr int offK = offQ + 2 * kTile;  // two stages
  static constexpr int offV = offK + 2 * kTile;  // two stages
  static constexpr int offScale = offV + 2 * kTile;             // [ring][key, value][128] fp32
  static constexpr int offBits = offScale + kScaleRing * 2 * kTok * 4;  // [ring][3][4]: see Bits
  static constexpr int offBar = offBits + kScaleRing * 12 * 4;
  static constexpr int offMisc = offBar + static_cast<int>(sizeof(Bars));
  static constexpr int kAlloc = offMisc + 64 + 1024;  // slack to align the base to 1024
};

// Shared-memory descriptors of operands with the 128-byte swizzle, built from
// a low word, in which tiles differ by their address alone (an addition of
// bytes / 16), and a constant high word.  K along the rows' 128 bytes: as
// ptx::sw128_kmajor_desc.  N along them (the value tile): 8 rows of an atom
// along K, atoms 1024 bytes apart (stride offset); atoms of 64 elements along N
// `atom_bytes` apart (leading offset).
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t atom_bytes) {
  return ((addr & 0x3FFFFu) >> 4) | ((atom_bytes >> 4) << 16);
}
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint64_t desc_at(uint32_t lo, uint32_t bytes) {
  return (static_cast<uint64_t>(kDescHi) << 32) | (lo + (bytes >> 4));
}

// D[tmem] (+)= A * B[smem desc], kind::f16, one CTA, A from shared or tensor
// memory; issued by the lane whose `lead` is 1.  Predicated rather than inside
// a branch of one lane: the code around stays uniform, and the operands in
// uniform registers.
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
// Arrive once on `bar` when all MMAs that this lane has issued are complete.
__device__ __forceinline__ void commit(uint32_t lead, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(bar), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_32x32b_x8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// fp16 operands, fp32 result, M = 128; n_major: B contiguous along N.
__device__ __forceinline__ constexpr uint32_t instr_desc(int n, bool n_major) {
  return (1u << 4) | (n_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}

// What the expanders say of a tile besides its scales: word i is that of tokens
// [32 i, 32 i + 32).
struct Bits {
  uint32_t live[4];  // tokens that are there
  uint32_t bad[4];   // of those, the ones whose value scale is not finite
  uint32_t top[4];   // the largest finite value scale, as fp16 bits
};

struct Wait {
  volatile uint32_t* abort;
  uint32_t* status;
};
// Bounded wait for a barrier's phase: false when the block is giving up.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, const Wait& w) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer();
  for (uint32_t i = 1; i != 0; ++i) {
    if (ptx::mbar_try_wait_sleep(bar, parity, 20000u)) return true;
    if ((i & 15u) == 0u) {
      if (*w.abort) return false;
      if (ptx::globaltimer() - t0 > kWaitNs) break;
    }
  }
  *w.abort = 1u;
  report_status(w.status, kStatusTimeout);
  return false;
}
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, const Wait& w) {
  return __all_sync(0xffffffffu, wait_for(bar, parity, w));
}

// A code word as 8 fp16 integers n - z in the order 0 4 1 5 2 6 3 7: with
// n in a half's low bits under the exponent of 1024 it is 1024 + n, four bits
// up 1024 + 16 n.  b1 = -(1024 + z) and b16 = -(64 + z) in both halves.
template <bool ASYM>
__device__ __forceinline__ uint4 expand(uint32_t w, uint32_t b1, uint32_t b16) {
  // (w & mask) | 0x64006400, with the sign bit of two's-complement codes
  // flipped (n - 8): 0x6a = (a & b) ^ c.
  constexpr uint32_t k1 = ASYM ? 0x64006400u : 0x64086408u, k16 = ASYM ? 0x64006400u : 0x64806480u;
  uint32_t x[4], o[4];
  asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(x[0]) : "r"(w), "r"(0x000F000Fu), "r"(k1));
  asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(x[1]) : "r"(w), "r"(0x00F000F0u), "r"(k16));
  w >>= 8;
  asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(x[2]) : "r"(w), "r"(0x000F000Fu), "r"(k1));
  asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(x[3]) : "r"(w), "r"(0x00F000F0u), "r"(k16));
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(o[i]) : "r"(x[i]), "r"(b1));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(o[i + 1]) : "r"(x[i + 1]), "r"(0x2C002C00u), "r"(b16));
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

template <typename T, int D, bool ASYM, bool GROUPED>
__global__ void __launch_bounds__(kThreadsP, 1)
    attention_prefill_kernel(const __grid_constant__ AttentionArgs a, const AttentionSpace ws, const int page_shift,
                             uint32_t* status) {
  using L = Smem<D>;
  constexpr int kStagesK = GROUPED ? 1 : 2;
  constexpr bool kExactV = GROUPED && std::is_same<T, __half>::value;  // values in two parts
  constexpr int kStagesV = kExactV ? 1 : 2;
  constexpr float kNegInf = -__builtin_huge_valf();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                   ~static_cast<uintptr_t>(1023));
  const CacheView& cache = a.cache;
  Bars* const bars = reinterpret_cast<Bars*>(smem + L::offBar);
  uint32_t* const misc = reinterpret_cast<uint32_t*>(smem + L::offMisc);  // TMEM address, abort flag, s_steps
  volatile uint32_t* const abort_flag = misc + 1;
  volatile int* const s_steps = reinterpret_cast<volatile int*>(misc + 2);  // [2]: tiles of an item, 0 after the last
  float* const s_scale = reinterpret_cast<float*>(smem + L::offScale);
  Bits* const s_bits = reinterpret_cast<Bits*>(smem + L::offBits);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto bar = [&](uint64_t& b) { return ptx::smem_u32(&b); };
  const Wait wc{abort_flag, status};

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bar(bars->k_full[i]), 4);
      ptx::mbar_init(bar(bars->k_empty[i]), 1);
      ptx::mbar_init(bar(bars->v_full[i]), 4);
      ptx::mbar_init(bar(bars->v_empty[i]), 1);
      for (int k = 0; k < 2; ++k) {
        ptx::mbar_init(bar(bars->s_full[i][k]), 1);
        ptx::mbar_init(bar(bars->w_full[i][k]), 4);
      }
      ptx::mbar_init(bar(bars->o_done[i]), 1);
    }
    for (int i = 0; i < kScaleRing; ++i) ptx::mbar_init(bar(bars->sc_full[i]), 4);
    ptx::mbar_init(bar(bars->q_full), 8);
    ptx::mbar_init(bar(bars->o_full), 1);
    ptx::mbar_init(bar(bars->drain), 1);
    *abort_flag = 0u;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(misc), 512);
    ptx::tmem_relinquish();
  }

  // ---- This block's share (each warp finds it).
  const Plan plan(a, kRows);
  if (blockIdx.x == 0 && warp == 2) plan.store(a, kRows, ws.prefix);
  const Shares shares(plan.units, ws.blocks);
  const bool working = static_cast<int>(blockIdx.x) < shares.active;
  const int u0 = working ? shares.begin(blockIdx.x) : 0;
  const int my_units = working ? shares.begin(blockIdx.x + 1) - u0 : 0;
  int b_start = 0, off_start = 0;
  if (working) plan.find(a, kRows, u0, b_start, off_start);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = misc[0];

  // ---- The walk over the share's items, the same in every role.
  struct Walk {
    int b, h, rt, n_rt, first, count, len, s0, left;
    RowTile tile;
    __device__ __forceinline__ void start(const AttentionArgs& a, int b_, int off, int units_) {
      b = b_;
      left = units_;
      if (left == 0) return;
      a.queries(b, first, count);
      len = a.kv_len(b);
      n_rt = row_tiles(a, count, kRows);
      const int per_head = head_units(a, b, kRows);
      h = off / per_head;
      off -= h * per_head;
      rt = 0;
      tile.set(a, len, count, 0, kRows);
      while (off >= tile.steps) {
        off -= tile.steps;
        tile.set(a, len, count, ++rt, kRows);
      }
      s0 = off;
    }
    __device__ __forceinline__ int steps() const { return min(left, tile.steps - s0); }
    __device__ __forceinline__ void next(const AttentionArgs& a) {
      left -= steps();
      if (left == 0) return;
      s0 = 0;
      do {
        if (++rt == n_rt) {
          rt = 0;
          if (++h == a.cache.heads) {
            h = 0;
            do {
              ++b;
              a.queries(b, first, count);
              len = a.kv_len(b);
              n_rt = row_tiles(a, count, kRows);
            } while (n_rt == 0);
          }
        }
        tile.set(a, len, count, rt, kRows);
      } while (tile.steps == 0);
    }
  };
  // Each warp of a role keeps its place in shared memory (all its lanes agree).
  __shared__ Walk s_walk[16];
  Walk& w = s_walk[warp];
  auto walk_start = [&]() {
    Walk x;
    x.start(a, b_start, off_start, my_units);
    if (lane == 0) w = x;
    __syncwarp();
  };
  auto walk_next = [&]() {
    Walk x = w;
    x.next(a);
    __syncwarp();
    if (lane == 0) w = x;
    __syncwarp();
  };

  // Registers a thread: 40 for the MMA warps, 88 for the expanders, 192 for
  // the softmax; 128 * 40 + 128 * 88 + 256 * 192 = 65536 = 512 * 128, what the
  // block is launched with.
  if (warp < 4) {
    ptx::regs_dec<40>();
    if (warp == 0) {
      // ---------------- MMA issuer ----------------
      const uint32_t lead = ptx::elect_one() ? 1u : 0u;
      constexpr uint32_t id_s = instr_desc(64, false), id_o = instr_desc(D, true);
      // The leading offset of K-major operands is not used (1, as elsewhere).
      const uint32_t q_lo = desc_lo(ptx::smem_u32(smem + L::offQ), 16), k_lo0 = desc_lo(ptx::smem_u32(smem + L::offK), 16),
                     v_lo0 = desc_lo(ptx::smem_u32(smem + L::offV), L::kSub);
      // Half `h` of a stage's tokens lies 64 rows of 128 bytes on.
      auto s_mma = [&](int m, int stage, int h) {
        const uint32_t k_lo = k_lo0 + stage * (L::kTile >> 4);
#pragma unroll
        for (int part = 0; part < (GROUPED ? 2 : 1); ++part) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = (k / 4) * L::kSub + (k % 4) * 32;
            mma_ss(lead, tmem + m * kTok + h * 64, desc_at(q_lo, m * L::kTile + off),
                   desc_at(k_lo, part * L::kTile + h * 8192 + off), id_s, part == 0 && k == 0 ? 0u : 1u);
          }
        }
        commit(lead, bar(bars->s_full[m][h]));
      };
      auto o_mma = [&](int m, int stage, int h, bool first) {
        const uint32_t v_lo = v_lo0 + stage * (L::kTile >> 4);
#pragma unroll
        for (int part = 0; part < (kExactV ? 2 : 1); ++part) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ts(lead, tmem + 2 * kTok + m * D, tmem + m * kTok + h * 64 + 8 * k,
                   desc_at(v_lo, part * L::kTile + h * 8192 + k * 2048), id_o, first && part == 0 && k == 0 ? 0u : 1u);
        }
        commit(lead, bar(bars->o_done[m]));
      };
      int t = 0;  // tiles before this one
      uint32_t item = 0;
      bool ok = true;
      while (true) {
        if (!(ok = wait_all(bar(bars->q_full), item & 1u, wc))) break;
        const int n = s_steps[item & 1u];
        if (n == 0) break;
        if (!(ok = wait_all(bar(bars->k_full[t % kStagesK]), (t / kStagesK) & 1u, wc))) break;
        ptx::tc_fence_after();
#pragma unroll
        for (int i = 0; i < 4; ++i) s_mma(i & 1, t % kStagesK, i >> 1);
        commit(lead, bar(bars->k_empty[t % kStagesK]));
        for (int j = 0; ok && j < n; ++j, ++t) {
          ok = wait_all(bar(bars->v_full[t % kStagesV]), (t / kStagesV) & 1u, wc);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int m = i & 1, h = i >> 1;
            ok = ok && wait_all(bar(bars->w_full[m][h]), t & 1u, wc);
            if (!ok) break;
            ptx::tc_fence_after();
            o_mma(m, t % kStagesV, h, j == 0 && h == 0);
            // Then S into the buffer that the W V before this one has read, one
            // step behind, so that it does not wait for it.
            if (i == 0) {
              if (j > 0) {
                s_mma(1, t % kStagesK, 1);
                commit(lead, bar(bars->k_empty[t % kStagesK]));
              }
            } else if (j + 1 < n) {
              if (i == 1) {
                ok = wait_all(bar(bars->k_full[(t + 1) % kStagesK]), ((t + 1) / kStagesK) & 1u, wc);
                if (!ok) break;
                ptx::tc_fence_after();
              }
              s_mma((i - 1) & 1, (t + 1) % kStagesK, (i - 1) >> 1);
            }
          }
          if (!ok) break;
          commit(lead, bar(bars->v_empty[t % kStagesV]));
          if (j + 1 == n) commit(lead, bar(bars->o_full));
        }
        if (!ok) break;
        ++item;
      }
      if (*abort_flag) {  // nothing may be in flight when tensor memory is freed
        commit(lead, bar(bars->drain));
        const uint64_t t0 = ptx::globaltimer();
        for (uint32_t i = 0; i != 0xFFFFFFFFu; ++i) {
          if (ptx::mbar_try_wait(bar(bars->drain), 0)) break;
          if ((i & 127u) == 0u && ptx::globaltimer() - t0 > kWaitNs) break;
        }
      }
    }
  } else if (warp < 8) {
    ptx::regs_dec<88>();
    // ---------------- expanders: thread = token of the tile ----------------
    walk_start();
    const int r = tid - 128;
    const int sw = r & 7;
    const int64_t page_rows = static_cast<int64_t>(2 * cache.heads) << page_shift;
    const int64_t to_values = static_cast<int64_t>(cache.heads) << page_shift;
    constexpr int kVec = D / 32;  // 16-byte vectors of a row
    // The row of this thread's token in the tile at `tok`, -1 if there is none
    // or no row sees it.
    auto find = [&](int tok) -> int64_t {
      if (tok < w.tile.first || tok >= w.tile.hi) return -1;
      const int id = __ldg(a.page_table + w.b * a.table_stride + (tok >> page_shift));
      if (id < 0 || id >= cache.pages) return -1;
      return id * page_rows + (static_cast<int64_t>(w.h) << page_shift) + (tok & (cache.page_size - 1));
    };
    // Scales (and zero points) of a row: one, or one for each 32 elements.
    constexpr int kScales = GROUPED ? kVec : 1;
    const int per_scale = cache.group >> 6;  // 0 or 1: log2 of the 32-element blocks of a group
    struct Row {
      uint4 v[kVec];
      uint32_t s[kScales], z[kScales];
      // Bits of the largest finite scale, and whether all are finite.
      __device__ __forceinline__ uint32_t top(bool& finite) const {
        uint32_t m = 0u;
        finite = true;
#pragma unroll
        for (int i = 0; i < kScales; ++i) {
          if ((s[i] & 0x7C00u) == 0x7C00u)
            finite = false;
          else
            m = max(m, s[i] & 0x7FFFu);
        }
        return m;
      }
    };
    auto load = [&](int64_t row, Row& x) {
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        x.v[i] = row < 0 ? make_uint4(0u, 0u, 0u, 0u)
                         : __ldg(reinterpret_cast<const uint4*>(cache.packed + row * (D / 2)) + i);
#pragma unroll
      for (int i = 0; i < kScales; ++i) {
        const int64_t at = GROUPED ? row * cache.groups + (i >> per_scale) : row;
        x.s[i] = row < 0 ? 0u : __ldg(cache.scales + at);
        x.z[i] = ASYM && row >= 0 ? __ldg(cache.zeros + at) : 0u;
      }
    };
    // What multiplies the token's column in fp32: its scale, or the power of two
    // of its largest one.
    auto column = [&](const Row& x, uint32_t top) {
      return GROUPED ? __uint_as_float((127u - 15u + max(top >> 10, 1u)) << 23) : f16_bits_to_float(x.s[0]);
    };
    auto store = [&](const Row& x, uint32_t at, uint32_t top, bool two_parts) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const uint32_t z = ASYM ? x.z[GROUPED ? i : 0] : 8u;
        // -(1024 + z) and -(64 + z), exact.
        const uint32_t b1 = (0xE400u + z) * 0x00010001u;
        const uint32_t b16 = __half_as_ushort(__int2half_rn(-64 - static_cast<int>(z))) * 0x00010001u;
        // The scale over u, in [0, 2); 0 for one that is not finite.
        uint32_t ratio = 0u;
        if (GROUPED && (x.s[GROUPED ? i : 0] & 0x7C00u) != 0x7C00u) {
          const float u_inv = __uint_as_float((127u + 15u - max(top >> 10, 1u)) << 23);
          ratio = __half_as_ushort(__float2half_rn(f16_bits_to_float(x.s[GROUPED ? i : 0]) * u_inv)) * 0x00010001u;
        }
        const uint32_t words[4] = {x.v[i].x, x.v[i].y, x.v[i].z, x.v[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int c = 4 * i + k;
          const uint32_t to = at + (c >> 3) * L::kSub + r * 128 + (((c & 7) ^ sw) << 4);
          const uint4 q = expand<ASYM>(words[k], b1, b16);
          if (!GROUPED) {
            ptx::sts128(to, q);
            continue;
          }
          const uint32_t n[4] = {q.x, q.y, q.z, q.w};
          uint32_t y[4], rest[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y[e] = attn::mul_half2(n[e], ratio);
            // (n - z) s / u less what was kept of it: exact.
            if (two_parts)
              asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(rest[e]) : "r"(n[e]), "r"(ratio), "r"(y[e] ^ 0x80008000u));
          }
          ptx::sts128(to, make_uint4(y[0], y[1], y[2], y[3]));
          if (two_parts) ptx::sts128(to + L::kTile, make_uint4(rest[0], rest[1], rest[2], rest[3]));
        }
      }
    };
    int t = 0;
    bool ok = true;
    while (ok && w.left > 0) {
      const int n = w.steps();
      const int base = w.tile.lo + w.s0 * kTok + r;
      int64_t row = find(base);
      int64_t row_next = n > 1 ? find(base + kTok) : -1;
      Row kx, vx;
      load(row, kx);
      load(row < 0 ? row : row + to_values, vx);
      for (int j = 0; j < n; ++j, ++t) {
        const int64_t row_after = j + 2 < n ? find(base + (j + 2) * kTok) : -1;
        bool k_finite, v_finite;
        const uint32_t k_top = kx.top(k_finite), v_top = vx.top(v_finite);
        const uint32_t live = __ballot_sync(0xffffffffu, row >= 0);
        const uint32_t bad = __ballot_sync(0xffffffffu, !v_finite);
        const uint32_t top = __reduce_max_sync(0xffffffffu, v_top);  // orders as the scales do
        // A key scale that is not finite gives NaN, as its values do.
        const float ks = k_finite ? column(kx, k_top) : __int_as_float(0x7FC00000);
        const float vs = v_finite ? column(vx, v_top) : 0.0f;
        // Keys.  The stage's last reader finished (first use: at once); the
        // scales' entry was last used four tiles ago, by a softmax that has
        // since handed on a later tile.
        if (!(ok = wait_all(bar(bars->k_empty[t % kStagesK]), ((t / kStagesK) & 1u) ^ 1u, wc))) break;
        const int ring = t & (kScaleRing - 1);
        s_scale[(ring * 2) * kTok + r] = ks;
        s_scale[(ring * 2 + 1) * kTok + r] = vs;
        if (lane == 0) {
          s_bits[ring].live[warp - 4] = live;
          s_bits[ring].bad[warp - 4] = bad;
          s_bits[ring].top[warp - 4] = top;
        }
        store(kx, ptx::smem_u32(smem + L::offK + (t % kStagesK) * L::kTile), k_top, GROUPED);
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(bar(bars->sc_full[ring]));
          ptx::mbar_arrive(bar(bars->k_full[t % kStagesK]));
        }
        if (j + 1 < n) load(row_next, kx);
        if (!(ok = wait_all(bar(bars->v_empty[t % kStagesV]), ((t / kStagesV) & 1u) ^ 1u, wc))) break;
        store(vx, ptx::smem_u32(smem + L::offV + (t % kStagesV) * L::kTile), v_top, kExactV);
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(bars->v_full[t % kStagesV]));
        if (j + 1 < n) load(row_next < 0 ? row_next : row_next + to_values, vx);
        row = row_next;
        row_next = row_after;
      }
      if (!ok) break;
      walk_next();
    }
  } else {
    ptx::regs_inc<192>();
    // ---------------- softmax: thread = query row ----------------
    walk_start();
    const int m = (warp - 8) >> 2;           // row tile
    const int q4 = warp & 3;                 // lanes of tensor memory this warp reads
    const int in_tile = q4 * 32 + lane, r = m * 128 + in_tile;  // row of the item
    const uint32_t lane_at = tmem + (static_cast<uint32_t>(32 * q4) << 16);
    const uint32_t o_at = lane_at + 2 * kTok + m * D;
    const float sign = a.sm_scale > 0.0f ? 1.0f : (a.sm_scale < 0.0f ? -1.0f : 0.0f);
    const bool q_vec = (reinterpret_cast<uintptr_t>(a.q) & 15) == 0 && a.q_token_stride % 8 == 0 && a.q_head_stride % 8 == 0;
    int t = 0;
    uint32_t item = 0;
    bool ok = true;
    while (ok && w.left > 0) {
      const int n = w.steps();
      const int base0 = w.tile.lo + w.s0 * kTok;
      const int r0 = w.rt * kRows;
      const int rows = min(w.count * a.ratio - r0, kRows);
      const bool live_row = r < rows;
      // ---- This row of Q.
      float f;
      int lo = 0, hi = 0;
      {
        const int i_tok = a.token_of(r0 + (live_row ? r : 0));
        const int hq = w.h * a.ratio + (r0 + (live_row ? r : 0)) - i_tok * a.ratio;
        uint32_t raw[D / 2];
        const T* qp = static_cast<const T*>(a.q) + (w.first + i_tok) * a.q_token_stride + hq * a.q_head_stride;
        if (q_vec) {
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            const uint4 x = __ldg(reinterpret_cast<const uint4*>(qp) + c);
            raw[4 * c] = x.x; raw[4 * c + 1] = x.y; raw[4 * c + 2] = x.z; raw[4 * c + 3] = x.w;
          }
        } else {
          const unsigned short* p = reinterpret_cast<const unsigned short*>(qp);
#pragma unroll
          for (int c = 0; c < D / 2; ++c)
            raw[c] = __ldg(p + 2 * c) | (static_cast<uint32_t>(__ldg(p + 2 * c + 1)) << 16);
        }
        auto lo_of = [](uint32_t x) {
          return std::is_same<T, __half>::value ? f16_bits_to_float(x & 0xFFFFu) : __uint_as_float(x << 16);
        };
        auto hi_of = [](uint32_t x) {
          return std::is_same<T, __half>::value ? f16_bits_to_float(x >> 16) : __uint_as_float(x & 0xFFFF0000u);
        };
        float top = 0.0f;
#pragma unroll
        for (int c = 0; c < D / 2; ++c) {
          if (!live_row) raw[c] = 0u;
          top = fmaxf(top, fmaxf(fabsf(lo_of(raw[c])), fabsf(hi_of(raw[c]))));
        }
        int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
        e = e < -100 ? -100 : e;
        // An infinite element makes the whole row NaN: its products alone could
        // give -infinity for every score, as if the row saw nothing.
        const float scale = e == 128 ? __int_as_float(0x7FC00000) : sign * __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
        const uint32_t at = ptx::smem_u32(smem + L::offQ + m * L::kTile) + in_tile * 128;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          // Elements 0 4, 1 5, 2 6, 3 7 of the block.
          const uint32_t* x = raw + 4 * c;
          const uint4 y = make_uint4(attn::pack_half2(lo_of(x[0]) * scale, lo_of(x[2]) * scale),
                                     attn::pack_half2(hi_of(x[0]) * scale, hi_of(x[2]) * scale),
                                     attn::pack_half2(lo_of(x[1]) * scale, lo_of(x[3]) * scale),
                                     attn::pack_half2(hi_of(x[1]) * scale, hi_of(x[3]) * scale));
          ptx::sts128(at + (c >> 3) * L::kSub + (((c & 7) ^ (in_tile & 7)) << 4), y);
        }
        const float f1 = __uint_as_float(static_cast<uint32_t>(127 + e - 14) << 23) * (fabsf(a.sm_scale) * 1.4426950408889634f);
        f = sign == 0.0f ? 1.0f : fminf(fmaxf(f1, 0x1p-126f), 0x1p127f);
        if (live_row) a.visible(w.len - w.count + i_tok, w.len, lo, hi);
      }
      ptx::fence_proxy_async_smem();
      ptx::tc_fence_before();  // O of the item before has been read
      if (warp == 8) s_steps[item & 1u] = n;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(bars->q_full));
      // Tokens that all live rows of this warp see.
      const int all_lo = __reduce_max_sync(0xffffffffu, live_row ? lo : 0);
      const int all_hi = __reduce_min_sync(0xffffffffu, live_row ? hi : 0x7FFFFFFF);

      float ref = kNegInf, nmf = 15.0f;  // the reference of S / f; x_run - ref * f
      float2 l = make_float2(0.0f, 0.0f);
      int x_run = 15;
      bool bad_row = false;  // sees a value scale that is not finite: so is its output
      const float2 f2 = make_float2(f, f);
      for (int u = 0; u < 2 * n; ++u) {  // half tiles
        const int h = u & 1, ring = t & (kScaleRing - 1);
        ok = (h == 1 || wait_all(bar(bars->sc_full[ring]), (t / kScaleRing) & 1u, wc)) &&
             wait_all(bar(bars->s_full[m][h]), t & 1u, wc);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t s_at = lane_at + m * kTok + h * 64;
        const float* const kc = s_scale + ring * 2 * kTok + h * 64;
        const float* const vc = kc + kTok;
        const int base = base0 + u * 64;
        const uint2 live = *reinterpret_cast<const uint2*>(s_bits[ring].live + 2 * h);
        const uint2 bad = *reinterpret_cast<const uint2*>(s_bits[ring].bad + 2 * h);
        const uint2 top2u = *reinterpret_cast<const uint2*>(s_bits[ring].top + 2 * h);
        const int x_new = min(x_run, 21 - static_cast<int>(max(top2u.x, top2u.y) >> 10));
        // Scores of the 16 columns from c on: S / f.
        auto scores = [&](int c, const uint32_t (&x)[16], float2 (&s)[8]) {
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const float4 k4 = *reinterpret_cast<const float4*>(kc + c + i);
            s[i / 2] = __fmul2_rn(make_float2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), make_float2(k4.x, k4.y));
            s[i / 2 + 1] = __fmul2_rn(make_float2(__uint_as_float(x[i + 2]), __uint_as_float(x[i + 3])), make_float2(k4.z, k4.w));
          }
        };
        // Their weights W = 2^x P s, and the weights' sum without s.  log2_p: of
        // a pair of scores, log2 (2^x P).
        auto weights = [&](int c, const float2 (&s)[8], auto log2_p, float2& sum, uint32_t (&pw)[8]) {
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float4 v4 = *reinterpret_cast<const float4*>(vc + c + 2 * i);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float2 p = log2_p(s[i + k]);
              p.x = attn::ex2(p.x);
              p.y = attn::ex2(p.y);
              sum = __fadd2_rn(sum, p);
              const float2 y = __fmul2_rn(p, k == 0 ? make_float2(v4.x, v4.y) : make_float2(v4.z, v4.w));
              pw[i + k] = attn::pack_half2(y.x, y.y);
            }
          }
        };
        float2 sum = make_float2(0.0f, 0.0f);
        const bool edge = base < all_lo || base + 64 > all_hi || (live.x & live.y) != 0xffffffffu;
        bool slow = edge || x_new != x_run || (bad.x | bad.y) != 0u || __any_sync(0xffffffffu, fabsf(nmf) > kNear);
        if (!slow) {
          // ---- All rows see all tokens: the weights under the reference so
          // far, in registers until it has proved near enough.  One piece of
          // straight code, so that its 64 columns overlap.
          float2 top2[2] = {make_float2(kNegInf, kNegInf), make_float2(kNegInf, kNegInf)};
          const float2 nmf2 = make_float2(nmf, nmf);
          uint32_t x[4][16], pw[4][8];
#pragma unroll
          for (int c = 0; c < 4; ++c) ptx::tmem_ld_32x32b_x16(s_at + 16 * c, x[c]);
          ptx::tmem_ld_wait();
          float2 part[2] = {sum, sum};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float2 s[8];
            scores(16 * c, x[c], s);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              top2[i & 1].x = fmaxf(top2[i & 1].x, s[i].x);
              top2[i & 1].y = fmaxf(top2[i & 1].y, s[i].y);
            }
            weights(16 * c, s, [&](float2 y) { return __ffma2_rn(y, f2, nmf2); }, part[c & 1], pw[c]);
          }
          sum = __fadd2_rn(part[0], part[1]);
          const float top = fmaxf(fmaxf(top2[0].x, top2[0].y), fmaxf(top2[1].x, top2[1].y));
          slow = __any_sync(0xffffffffu, top > ref && (ref == kNegInf || (top - ref) * f > kGrow));
          if (!slow) {
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_st_32x32b_x8(s_at + 8 * c, pw[c]);
          }
        }
        if (slow) {
          // ---- Otherwise the maximum first, of the tokens that the row sees.
          uint32_t seen[2] = {0xffffffffu, 0xffffffffu};
          if (edge) {
            const uint32_t here[2] = {live.x, live.y};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int from = min(max(lo - (base + 32 * i), 0), 32), to = min(max(hi - (base + 32 * i), 0), 32);
              const uint32_t below = to == 32 ? 0xffffffffu : (1u << to) - 1u;
              seen[i] = from == 32 ? 0u : here[i] & below & (0xffffffffu << from);
            }
          }
          if ((bad.x | bad.y) != 0u) bad_row = bad_row || ((bad.x & seen[0]) | (bad.y & seen[1])) != 0u;
          auto load = [&](int c, float2 (&s)[8]) {
            uint32_t x[16];
            ptx::tmem_ld_32x32b_x16(s_at + c, x);
            ptx::tmem_ld_wait();
            scores(c, x, s);
            const uint32_t visible = (c < 32 ? seen[0] : seen[1]) >> (c & 16);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if (((visible >> (2 * i)) & 1u) == 0u) s[i].x = kNegInf;
              if (((visible >> (2 * i + 1)) & 1u) == 0u) s[i].y = kNegInf;
            }
          };
          float top = kNegInf;
#pragma unroll 1
          for (int c = 0; c < 64; c += 16) {
            float2 s[8];
            load(c, s);
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, fmaxf(s[i].x, s[i].y));
          }
          const bool behind = top > ref && (ref == kNegInf || (top - ref) * f > kGrow);
          if (__any_sync(0xffffffffu, behind) || x_new != x_run) {
            const float new_ref = fmaxf(ref, top);
            float al = new_ref == ref ? 1.0f : attn::ex2((ref - new_ref) * f);
            al *= __uint_as_float(static_cast<uint32_t>(127 + x_new - x_run) << 23);
            ref = new_ref;
            x_run = x_new;
            nmf = static_cast<float>(x_run) - (ref == kNegInf ? 0.0f : ref * f);
            l = __fmul2_rn(l, make_float2(al, al));
            if (u > 0) {
              // The products of the half tile before are still being added, or
              // their turn has not come.
              if (!(ok = wait_all(bar(bars->o_done[m]), (2 * t + h - 1) & 1u, wc))) break;
              ptx::tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D; c += 16) {
                uint32_t y[16];
                ptx::tmem_ld_32x32b_x16(o_at + c, y);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) * al);
                tmem_st_32x32b_x16(o_at + c, y);
              }
            }
          }
          // W follows over the columns of S that have been read.  The reference
          // is taken off before the product with f: see cache_attention.cuh.
          const float nr = ref == kNegInf ? 0.0f : -ref;
          const float2 nr2 = make_float2(nr, nr), x2 = make_float2(static_cast<float>(x_run), static_cast<float>(x_run));
          sum = make_float2(0.0f, 0.0f);
#pragma unroll 1
          for (int c = 0; c < 64; c += 16) {
            float2 s[8];
            uint32_t y[8];
            load(c, s);
            weights(c, s, [&](float2 z) { return __ffma2_rn(__fadd2_rn(z, nr2), f2, x2); }, sum, y);
            tmem_st_32x32b_x8(s_at + c / 2, y);
          }
        }
        l = __fadd2_rn(l, sum);
        tmem_st_wait();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(bars->w_full[m][h]));
        t += h;
      }
      if (!ok) break;
      // ---- O.
      if (!(ok = wait_all(bar(bars->o_full), item & 1u, wc))) break;
      ptx::tc_fence_after();
      const bool whole = n == w.tile.steps;
      const float sum = l.x + l.y;
      const int i_tok = a.token_of(r0 + (live_row ? r : 0));
      const int at = (w.first + i_tok) * a.q_heads + w.h * a.ratio + (r0 + (live_row ? r : 0)) - i_tok * a.ratio;
      const int64_t slot = (2 * static_cast<int64_t>(blockIdx.x) + (w.s0 == 0 ? 1 : 0)) * kRows + r;
      const float back = __uint_as_float(static_cast<uint32_t>(127 - x_run) << 23);
      float inv = whole ? (sum == 0.0f ? 0.0f : 1.0f / sum) : back;
      if (bad_row) inv = __int_as_float(0x7FC00000);
#pragma unroll
      for (int c = 0; c < D; c += 16) {
        uint32_t x[16];
        ptx::tmem_ld_32x32b_x16(o_at + c, x);
        ptx::tmem_ld_wait();
        if (live_row) {
#pragma unroll
          for (int i = 0; i < 16; i += 8) {
            float v[8];  // columns 0 .. 7 of a block are its elements 0 4 1 5 2 6 3 7
#pragma unroll
            for (int k = 0; k < 8; ++k) v[(k >> 1) + 4 * (k & 1)] = __uint_as_float(x[i + k]) * inv;
            if (whole) {
              alignas(16) T y[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) store_as(y + k, v[k]);
              *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + static_cast<int64_t>(at) * D + c + i) =
                  *reinterpret_cast<const uint4*>(y);
            } else {
              float4* const dst = reinterpret_cast<float4*>(ws.o + slot * D + c + i);
              dst[0] = make_float4(v[0], v[1], v[2], v[3]);
              dst[1] = make_float4(v[4], v[5], v[6], v[7]);
            }
          }
        }
      }
      if (live_row) {
        const float top = ref * f;
        if (!whole) {
          ws.ml[slot * 2] = top;
          ws.ml[slot * 2 + 1] = sum * back;
        } else if (a.lse != nullptr) {
          a.lse[at] = sum == 0.0f ? kNegInf
                                  : (top + log2f(sum) - static_cast<float>(x_run)) * 0.6931471805599453f;
        }
      }
      ++item;
      walk_next();
    }
    if (ok) {  // no more items
      if (warp == 8) s_steps[item & 1u] = 0;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(bars->q_full));
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

template <typename T, int D, bool ASYM, bool GROUPED>
cudaError_t launch_prefill_typed(const AttentionArgs& a, void* workspace, cudaStream_t stream) {
  uint32_t* status = status_word();
  if (status == nullptr) return cudaErrorInvalidSymbol;
  const AttentionSpace ws = attention_space(workspace, a.batch, num_sms(), kRows, D);
  constexpr auto kernel = attention_prefill_kernel<T, D, ASYM, GROUPED>;
  constexpr int bytes = Smem<D>::kAlloc;
  static_assert(bytes <= 227 * 1024, "one block's shared memory");
  cudaError_t e = allow_shared<kernel>(bytes);
  if (e != cudaSuccess) return e;
  int shift = 0;
  while ((1 << shift) < a.cache.page_size) ++shift;
  kernel<<<ws.blocks, kThreadsP, bytes, stream>>>(a, ws, shift, status);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_attention_join_items<T>(a, ws, kRows, stream);
}

template <typename T, int D>
cudaError_t launch_prefill_scheme(const AttentionArgs& a, void* workspace, cudaStream_t stream) {
  const bool asym = a.cache.zeros != nullptr;
  if (a.cache.group == D)
    return asym ? launch_prefill_typed<T, D, true, false>(a, workspace, stream)
                : launch_prefill_typed<T, D, false, false>(a, workspace, stream);
  return asym ? launch_prefill_typed<T, D, true, true>(a, workspace, stream)
              : launch_prefill_typed<T, D, false, true>(a, workspace, stream);
}

template <int D>
cudaError_t launch_prefill(const AttentionArgs& a, DType t, void* workspace, cudaStream_t stream) {
  return t == DType::BF16 ? launch_prefill_scheme<__nv_bfloat16, D>(a, workspace, stream)
                          : launch_prefill_scheme<__half, D>(a, workspace, stream);
}

}  // namespace

}  // namespace int4lib
