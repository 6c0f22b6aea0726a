// The 4-bit key/value cache: its layout, shared by the kernels that write
// it, read it back and attend over it (sm_100a).
//
//   packed [P, 2, H, S, ceil(D / 2)] uint8   keys at index 0, values at 1
//   scales [P, 2, H, S, G] fp16              G = ceil(D / group)
//   zeros  [P, 2, H, S, G] uint8             affine scheme only
//
// P pages of S tokens each, H heads of D elements.  A token's row of one head
// is coded exactly as a row of int4_quantize (or int4_quantize_affine), with
// K = D: element 2j in the low nibble of byte j, groups along D.  The S rows
// of one (page, keys or values, head) are contiguous, so a tile of tokens of
// one head is one contiguous run of bytes inside its page.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace int4lib {

struct CacheView {
  uint8_t* packed;
  uint16_t* scales;
  uint8_t* zeros;  // nullptr: symmetric scheme
  int64_t pages;
  int32_t page_size;
  int32_t heads;
  int32_t head_dim;
  int32_t group;
  int32_t row_bytes;  // ceil(head_dim / 2)
  int32_t groups;     // ceil(head_dim / group)

  // Row of token `offset` of a page, counted over [P, 2, H, S].
  __device__ __forceinline__ int64_t row(int64_t page, int kv, int head, int64_t offset) const {
    return ((page * 2 + kv) * heads + head) * page_size + offset;
  }
};

// Stores of dequantized or attended values: one rounding, to nearest even.
__device__ __forceinline__ void store_as(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_as(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store_as(__half* p, float v) { *p = __float2half_rn(v); }

// The integer of a nibble: two's complement, or unsigned less the group's
// zero point.
template <bool ASYM>
__device__ __forceinline__ float code_value(uint32_t nib, int zp) {
  if (ASYM) return static_cast<float>(static_cast<int>(nib & 0xFu) - zp);
  return static_cast<float>(static_cast<int32_t>(nib << 28) >> 28);
}

// What an attention call reads besides the cache.  All strides in elements.
struct AttentionArgs {
  CacheView cache;
  const void* q;  // [rows, q_heads, D]
  int64_t q_token_stride, q_head_stride;
  void* out;   // [rows, q_heads, D], dense
  float* lse;  // [rows, q_heads], dense, or nullptr
  const int32_t* page_table;  // [batch, max_pages]
  int64_t table_stride;
  const int32_t* kv_lens;   // [batch]
  const int32_t* q_starts;  // [batch + 1], or nullptr: rows / batch queries each
  int32_t rows;  // rows * q_heads is below 2^31: so are all row indexes
  int32_t batch;
  int32_t max_pages;
  int32_t q_heads;
  int32_t ratio;  // q_heads / heads
  uint32_t ratio_m, ratio_s;  // r / ratio = (r * ratio_m >> 32) >> ratio_s for 0 <= r < 2^31, ratio > 1
  int32_t causal;
  int32_t window;  // 0: none
  float sm_scale;

  // Row r of a sequence's (query token, query head of a group) rows: its token.
  __device__ __forceinline__ int token_of(int r) const {
    return ratio == 1 ? r : static_cast<int>(__umulhi(static_cast<uint32_t>(r), ratio_m) >> ratio_s);
  }
  // Cached tokens of sequence b, never more than its row of the table holds.
  __device__ __forceinline__ int kv_len(int b) const {
    const int64_t cap = static_cast<int64_t>(max_pages) * cache.page_size;
    const int n = max(__ldg(kv_lens + b), 0);
    return n < cap ? n : static_cast<int>(cap);
  }
  // First query row of sequence b and their number, inside [0, rows).
  __device__ __forceinline__ void queries(int b, int& first, int& count) const {
    if (q_starts == nullptr) {
      count = rows / batch;
      first = count * b;
      return;
    }
    first = min(max(__ldg(q_starts + b), 0), rows);
    count = max(min(__ldg(q_starts + b + 1), rows) - first, 0);
  }
  // Keys [lo, hi) that the query at position `pos` of a sequence of `len`
  // tokens sees (none where hi <= lo).
  __device__ __forceinline__ void visible(int pos, int len, int& lo, int& hi) const {
    hi = causal != 0 ? max(min(pos + 1, len), 0) : len;
    lo = window > 0 && pos >= window ? pos - window + 1 : 0;
  }
  // The sequence that holds query row t, or -1.
  __device__ __forceinline__ int sequence_of(int t) const {
    if (q_starts == nullptr) return t / (rows / batch);
    int lo = 0, hi = batch;  // last b with q_starts[b] <= t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(q_starts + mid) <= t) lo = mid; else hi = mid;
    }
    return __ldg(q_starts + lo) <= t && t < __ldg(q_starts + lo + 1) ? lo : -1;
  }
};

}  // namespace int4lib
