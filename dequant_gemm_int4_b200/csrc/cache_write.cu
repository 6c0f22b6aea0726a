// Writing the 4-bit key/value cache and reading it back (sm_100a).
//
// A new token's key and value rows are coded in the library's two schemes,
// bit for bit as int4_quantize and int4_quantize_affine code a weight row:
//   symmetric  s = fp16(fp32(absmax / 7)), q = clamp(rint(fp32(x / s)), -8, 7)
//   affine     s = fp16(fp32((max - min) / 15)),
//              z = clamp(rint(fp32(-min / s)), 0, 15),
//              q = clamp(rint(fp32(fp32(x / s) + z)), 0, 15)
// with q = 0 (and z = 0) where s is 0 or infinite, and stored at the token's
// slot.  Reading a slot gives q s or (q - z) s, rounded once.
//
// A decoding step's few tokens cost a launch.  65536 tokens of 8 heads of 128 in
// bf16 are read in 67 us, bound by HBM (5.0 TB/s of codes and values), and
// written in 87 us (affine groups of 64: 102 us), bound by instruction issue: 279
// instructions (affine 325) for 16 elements of a warp's 32 lanes, in 79 % of the
// issue slots (widening, extremes, correctly rounded quotients, packing).  Shapes
// and strides that the fast kernels do not take are not tuned: 65536 tokens of 8
// heads of 80 in groups of 48 are written in 915 us.
#include <type_traits>

#include "cache.cuh"
#include "internal.h"

namespace int4lib {

namespace {

// fp32(v / s), correctly rounded, from r = RN(1 / s): q = RN(v r) is within
// an ulp of the quotient, the residual v - q s is exact by FMA, and
// RN(q + residual r) is the correctly rounded quotient (Markstein).  Holds
// where |v r| stays far below overflow and the quotient is 1/4 or more; a
// smaller quotient rounds to the same code either way.
__device__ __forceinline__ float quotient(float v, float s, float r) {
  const float q = __fmul_rn(v, r);
  return __fmaf_rn(__fmaf_rn(-q, s, v), r, q);
}

// fp32(v / N), correctly rounded, for finite v >= 0: one residual correction
// with c = RN(1 / N) (Markstein, as above); where the residual could round (v
// subnormal) the scale is 0 either way.  An infinite v stays infinite.
template <int N>
__device__ __forceinline__ float over(float v) {
  constexpr float c = N == 7 ? 0.142857149f : 0.0666666701f;
  static_assert(N == 7 || N == 15, "the schemes' divisors");
  const float q = __fmul_rn(v, c);
  const float r = __fmaf_rn(__fmaf_rn(-static_cast<float>(N), q, v), c, q);
  return v < 0x1p127f ? r : __fdiv_rn(v, static_cast<float>(N));
}

// Scale and zero point of a group, and the codes of its elements.
struct Coder {
  float s;         // the scale as stored
  float r;         // RN(1 / s)
  float z;         // the zero point
  bool live;       // s neither 0 nor infinite: elsewhere every code is 0
  bool divide;     // quotients may be too large for quotient()
  uint16_t bits = 0;

  // lo, hi: the group's extremes (affine), or 0 and its absmax (symmetric).
  template <bool ASYM>
  __device__ __forceinline__ void set(float lo, float hi) {
    const float d = ASYM ? over<15>(__fsub_rn(hi, lo)) : over<7>(hi);
    bits = __half_as_ushort(__float2half_rn(d));
    s = f16_bits_to_float(bits);
    live = s > 0.0f && bits != 0x7C00u;
    r = live ? __frcp_rn(s) : 0.0f;
    z = 0.0f;
    // In the symmetric scheme |x / s| <= 14 (a scale rounded to the smallest
    // fp16 subnormal halves at most).
    divide = ASYM && !(__fmul_rn(fmaxf(fabsf(lo), fabsf(hi)), r) < 0x1p99f);
    if (ASYM && live) z = fminf(fmaxf(rintf(div(-lo)), 0.0f), 15.0f);
  }
  __device__ __forceinline__ float div(float v) const {
    return divide ? __fdiv_rn(v, s) : quotient(v, s, r);
  }
  // Clamped before rounding (the bounds are integers), then rounded to an
  // integer, ties to even, by adding 1.5 * 2^23.
  template <bool ASYM>
  __device__ __forceinline__ uint32_t code(float v) const {
    float u = div(v);
    if (ASYM) u = __fadd_rn(u, z);
    u = fminf(fmaxf(u, ASYM ? 0.0f : -8.0f), ASYM ? 15.0f : 7.0f);
    return live ? __float_as_uint(__fadd_rn(u, 12582912.0f)) & 0xFu : 0u;
  }
  // Eight codes, the first in the lowest nibble; two elements an instruction
  // (each rounded as by code()) where no quotient is too large.
  template <bool ASYM>
  __device__ __forceinline__ void codes8(const float* v, uint32_t& word) const {
    word = 0u;
    if (!live) return;
    if (divide) {
#pragma unroll
      for (int k = 0; k < 8; ++k) word |= code<ASYM>(v[k]) << (4 * k);
      return;
    }
    const float2 r2 = make_float2(r, r), ns2 = make_float2(-s, -s), z2 = make_float2(z, z);
    const float2 magic = make_float2(12582912.0f, 12582912.0f);
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      const float2 x = make_float2(v[k], v[k + 1]);
      const float2 q = __fmul2_rn(x, r2);
      float2 u = __ffma2_rn(__ffma2_rn(q, ns2, x), r2, q);
      if (ASYM) u = __fadd2_rn(u, z2);
      u.x = fminf(fmaxf(u.x, ASYM ? 0.0f : -8.0f), ASYM ? 15.0f : 7.0f);
      u.y = fminf(fmaxf(u.y, ASYM ? 0.0f : -8.0f), ASYM ? 15.0f : 7.0f);
      const float2 t = __fadd2_rn(u, magic);
      word |= ((__float_as_uint(t.x) & 0xFu) | ((__float_as_uint(t.y) & 0xFu) << 4)) << (4 * k);
    }
  }
};

struct WriteArgs {
  CacheView cache;
  const void* src[2];  // k, v
  int64_t token_stride[2], head_stride[2];
  const int64_t* slots;
  int64_t tokens;
};

struct ReadArgs {
  CacheView cache;
  void* dst[2];
  const int64_t* slots;
  int64_t tokens;
};

// A block of the fast kernels takes 2^tokens_log whole tokens, whose 2 H rows
// are cut into pieces of 16 elements, `per_row` of them.  Piece i of the block
// belongs to row r = i / per_row, the token r % 2^tokens_log and the key or value
// head r >> tokens_log: neighbouring rows of a warp are neighbouring tokens of
// one head, whose codes and scales are neighbours in the cache (with the heads
// of one token side by side instead, reading 65536 tokens of 8 heads of 128 took
// 78 us, not 67).  The division is a
// multiplication with m = ceil(2^32 / per_row), exact for the products below
// 2^32 that occur (i < 2^16, divisors from 2 to 2^16).
struct Pieces {
  uint32_t per_row, per_row_m;
  uint32_t rows;  // 2 H
  uint32_t tokens_log;
};
constexpr int kMaxBlockTokens = 64;

// The cache rows of a block's tokens: that of head 0's key, or -1 where the
// slot is outside the cache.
__device__ __forceinline__ void find_rows(const CacheView& c, const int64_t* slots, int64_t token0,
                                          int64_t tokens, int per_block, int64_t (&rows)[kMaxBlockTokens]) {
  for (int i = threadIdx.x; i < per_block; i += blockDim.x) {
    const int64_t slot = token0 + i < tokens ? __ldg(slots + token0 + i) : -1;
    int64_t row = -1;
    if (slot >= 0 && slot < c.pages * c.page_size) {
      // A slot below 2^32 is divided in 32 bits.
      const int64_t page = slot < (1LL << 32) ? static_cast<uint32_t>(slot) / static_cast<uint32_t>(c.page_size)
                                              : slot / c.page_size;
      row = c.row(page, 0, 0, slot - page * c.page_size);
    }
    rows[i] = row;
  }
  __syncthreads();
}

// 16 elements as they are stored, and widened (exactly).
template <typename T>
struct Raw16 {
  static constexpr int kVecs = sizeof(T) == 4 ? 4 : 2;
  uint4 x[kVecs];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) x[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) x[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void widen(float (&v)[16]) const {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (sizeof(T) == 4) {
          v[4 * i + k] = __uint_as_float(w[k]);
        } else if (std::is_same<T, __half>::value) {
          v[8 * i + 2 * k] = f16_bits_to_float(w[k] & 0xFFFFu);
          v[8 * i + 2 * k + 1] = f16_bits_to_float(w[k] >> 16);
        } else {
          v[8 * i + 2 * k] = __uint_as_float(w[k] << 16);
          v[8 * i + 2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
        }
      }
    }
  }
};

// group a multiple of 16 up to 512 that divides D, every source row 16-byte
// aligned, packed 8-byte aligned.  A thread codes 16 consecutive elements of
// one row (two 16-byte loads of 16-bit elements, one 8-byte store); a group has
// `lpg` lanes, the next power of two from group / 16 on, which lie in one warp
// and find its extremes with shuffles (the lanes past group / 16 only take
// part in those).  The next piece is loaded while this one is coded.
template <typename T, bool ASYM>
__global__ void __launch_bounds__(256) cache_write_kernel(const __grid_constant__ WriteArgs a,
                                                          const Pieces p, const int lpg_log) {
  const CacheView& c = a.cache;
  __shared__ int64_t s_rows[kMaxBlockTokens];
  const int64_t token0 = static_cast<int64_t>(blockIdx.x) << p.tokens_log;
  find_rows(c, a.slots, token0, a.tokens, 1 << p.tokens_log, s_rows);
  const uint32_t total = (p.rows << p.tokens_log) * p.per_row;
  const int lpg = 1 << lpg_log;
  struct Piece {
    Raw16<T> raw;
    int64_t at;  // its row in the cache, -1: none
    int group, d;
  };
  auto load = [&](uint32_t base, Piece& x) {
    const uint32_t i = base + threadIdx.x;
    const uint32_t r = __umulhi(i, p.per_row_m), in_row = i - r * p.per_row;
    const uint32_t row = r >> p.tokens_log, tok = r - (row << p.tokens_log);
    x.group = in_row >> lpg_log;
    const int in_group = (in_row & (lpg - 1)) * 16;
    x.d = x.group * c.group + in_group;
    x.at = i < total && in_group < c.group ? s_rows[tok] : -1;
    x.raw.clear();
    if (x.at < 0) return;
    x.at += static_cast<int64_t>(row) * c.page_size;  // values follow the keys of all heads
    const int kv = row >= static_cast<uint32_t>(c.heads) ? 1 : 0;
    const T* src = static_cast<const T*>(kv ? a.src[1] : a.src[0]) +
                   (token0 + tok) * (kv ? a.token_stride[1] : a.token_stride[0]) +
                   static_cast<int>(row - kv * c.heads) * (kv ? a.head_stride[1] : a.head_stride[0]) + x.d;
    x.raw.load(src);
  };
  // Whole warps take part in every step, so that the shuffles are uniform.
  Piece x;
  load(0, x);
  for (uint32_t base = 0; base < total; base += blockDim.x) {
    Piece next;
    next.at = -1;
    if (base + blockDim.x < total) load(base + blockDim.x, next);
    float v[16];
    x.raw.widen(v);
    float lo = ASYM ? v[0] : 0.0f, hi = ASYM ? v[0] : fabsf(v[0]);
#pragma unroll
    for (int k = 1; k < 16; ++k) {
      if (ASYM) lo = fminf(lo, v[k]);
      hi = fmaxf(hi, ASYM ? v[k] : fabsf(v[k]));
    }
    if (ASYM && x.at < 0) {  // nothing of the group: neutral
      lo = __int_as_float(0x7F800000);
      hi = __int_as_float(0xFF800000);
    }
    for (int off = 1; off < lpg; off <<= 1) {
      if (ASYM) lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
    }
    if (x.at >= 0) {
      Coder q;
      q.set<ASYM>(lo, hi);
      uint2 word = make_uint2(0u, 0u);
      q.codes8<ASYM>(v, word.x);
      q.codes8<ASYM>(v + 8, word.y);
      *reinterpret_cast<uint2*>(c.packed + x.at * c.row_bytes + (x.d >> 1)) = word;
      if ((threadIdx.x & (lpg - 1)) == 0) {
        const int64_t g = x.at * c.groups + x.group;
        c.scales[g] = q.bits;
        if (ASYM) c.zeros[g] = static_cast<uint8_t>(q.z);
      }
    }
    x = next;
  }
}

// Any D, group, stride and alignment: a warp codes one row.
template <typename T, bool ASYM>
__global__ void __launch_bounds__(256) cache_write_any_kernel(const __grid_constant__ WriteArgs a) {
  const CacheView& c = a.cache;
  const int lane = threadIdx.x & 31;
  const int64_t rows = 2LL * c.heads;
  const int64_t total = a.tokens * rows;
  const int64_t step = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
  for (int64_t w = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; w < total; w += step) {
    const int64_t t = w / rows;
    const uint32_t row = static_cast<uint32_t>(w - t * rows);  // below 2^32: heads are below 2^31
    const int kv = row >= static_cast<uint32_t>(c.heads) ? 1 : 0;
    const int h = static_cast<int>(row - kv * static_cast<uint32_t>(c.heads));
    const int64_t slot = __ldg(a.slots + t);
    if (slot < 0 || slot >= c.pages * c.page_size) continue;
    const T* x = static_cast<const T*>(a.src[kv]) + t * a.token_stride[kv] + h * a.head_stride[kv];
    const int64_t at = c.row(slot / c.page_size, kv, h, slot % c.page_size);
    // The byte at an odd group's edge belongs to two groups: nibbles are
    // collected lane by lane over whole bytes, each under its own group.
    for (int b0 = 0; b0 < c.row_bytes; b0 += 32) {
      const int b = b0 + lane;
      uint32_t byte = 0u;
      const int d_first = 2 * b0, d_last = min(2 * (b0 + 32), c.head_dim) - 1;
      for (int g = d_first / c.group; g <= d_last / c.group; ++g) {
        const int64_t g_begin = static_cast<int64_t>(g) * c.group;
        const int64_t g_end64 = g_begin + c.group;
        const int g0 = static_cast<int>(g_begin);
        const int g1 = g_end64 < c.head_dim ? static_cast<int>(g_end64) : c.head_dim;
        float lo = ASYM ? __int_as_float(0x7F800000) : 0.0f;
        float hi = ASYM ? __int_as_float(0xFF800000) : 0.0f;
        for (int d = g0 + lane; d < g1; d += 32) {
          const float v = Elem<T>::load(x + d);
          if (ASYM) lo = fminf(lo, v);
          hi = fmaxf(hi, ASYM ? v : fabsf(v));
        }
        for (int off = 1; off < 32; off <<= 1) {
          if (ASYM) lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
          hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
        }
        Coder q;
        q.set<ASYM>(lo, hi);
        if (b < c.row_bytes) {
          if (2 * b >= g0 && 2 * b < g1) byte |= q.code<ASYM>(Elem<T>::load(x + 2 * b));
          if (2 * b + 1 >= g0 && 2 * b + 1 < g1) byte |= q.code<ASYM>(Elem<T>::load(x + 2 * b + 1)) << 4;
        }
        if (lane == 0 && g0 >= d_first) {  // the window in which the group begins stores its scale
          c.scales[at * c.groups + g] = q.bits;
          if (ASYM) c.zeros[at * c.groups + g] = static_cast<uint8_t>(q.z);
        }
      }
      if (b < c.row_bytes) c.packed[at * c.row_bytes + b] = static_cast<uint8_t>(byte);
    }
  }
}

template <typename TO>
__device__ __forceinline__ void store8(TO* p, const float (&v)[8]);
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
}
template <>
__device__ __forceinline__ void store8<__half>(__half* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// D and group multiples of 16, packed 8-byte and outputs 16-byte aligned: a
// thread gives 16 consecutive elements of one row (one 8-byte load, two
// 16-byte stores of 16-bit elements).
template <typename TO, bool ASYM>
__global__ void __launch_bounds__(256) cache_read_kernel(const __grid_constant__ ReadArgs a, const Pieces p) {
  const CacheView& c = a.cache;
  __shared__ int64_t s_rows[kMaxBlockTokens];
  const int64_t token0 = static_cast<int64_t>(blockIdx.x) << p.tokens_log;
  find_rows(c, a.slots, token0, a.tokens, 1 << p.tokens_log, s_rows);
  const uint32_t total = (p.rows << p.tokens_log) * p.per_row;
#pragma unroll 4
  for (uint32_t i = threadIdx.x; i < total; i += blockDim.x) {
    const uint32_t r = __umulhi(i, p.per_row_m), d = (i - r * p.per_row) * 16;
    const uint32_t row = r >> p.tokens_log, tok = r - (row << p.tokens_log);
    if (token0 + tok >= a.tokens) continue;
    const int64_t at0 = s_rows[tok];
    const int kv = row >= static_cast<uint32_t>(c.heads) ? 1 : 0;
    const int h = row - kv * c.heads;
    const int64_t at = at0 + static_cast<int64_t>(row) * c.page_size;
    uint2 w = make_uint2(0u, 0u);
    float s = 0.0f;
    int zp = 0;
    if (at0 >= 0) {
      w = __ldg(reinterpret_cast<const uint2*>(c.packed + at * c.row_bytes + (d >> 1)));
      const int64_t g = at * c.groups + d / c.group;
      s = f16_bits_to_float(__ldg(c.scales + g));
      if (ASYM) zp = static_cast<int>(__ldg(c.zeros + g));
    }
    TO* out = static_cast<TO*>(kv ? a.dst[1] : a.dst[0]) + ((token0 + tok) * c.heads + h) * c.head_dim + d;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = code_value<ASYM>(((half ? w.y : w.x) >> (4 * k)) & 0xFu, zp) * s;
      if (at0 < 0) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = 0.0f;
      }
      store8<TO>(out + 8 * half, v);
    }
  }
}

// Any D, group and alignment: a thread gives the two elements of one byte.
template <typename TO, bool ASYM>
__global__ void __launch_bounds__(256) cache_read_any_kernel(const __grid_constant__ ReadArgs a) {
  const CacheView& c = a.cache;
  const int64_t per_token = 2LL * c.heads * c.row_bytes;
  const int64_t total = a.tokens * per_token;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total; i += step) {
    const int64_t t = i / per_token;
    const int64_t in_token = i - t * per_token;
    const uint32_t row = static_cast<uint32_t>(in_token / c.row_bytes);  // as above
    const int b = static_cast<int>(in_token - static_cast<int64_t>(row) * c.row_bytes);
    const int kv = row >= static_cast<uint32_t>(c.heads) ? 1 : 0;
    const int h = static_cast<int>(row - kv * static_cast<uint32_t>(c.heads));
    const int64_t slot = __ldg(a.slots + t);
    const bool live = slot >= 0 && slot < c.pages * c.page_size;
    const int64_t at = live ? c.row(slot / c.page_size, kv, h, slot % c.page_size) : 0;
    const uint32_t byte = live ? __ldg(c.packed + at * c.row_bytes + b) : 0u;
    TO* out = static_cast<TO*>(a.dst[kv]) + (t * c.heads + h) * c.head_dim;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int d = 2 * b + k;
      if (d >= c.head_dim) break;
      float v = 0.0f;
      if (live) {
        const int64_t g = at * c.groups + d / c.group;
        const int zp = ASYM ? static_cast<int>(__ldg(c.zeros + g)) : 0;
        v = code_value<ASYM>((byte >> (4 * k)) & 0xFu, zp) * f16_bits_to_float(__ldg(c.scales + g));
      }
      store_as(out + d, v);
    }
  }
}

bool multiple_of(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// The blocks of a fast kernel: about four pieces a thread, fewer where that
// would leave SMs without a block.  False where the sizes are out of its range.
bool cut(const CacheView& c, int64_t tokens, int64_t per_row, Pieces* p, int64_t* grid) {
  const int64_t rows = 2LL * c.heads;
  if (c.head_dim % 16 != 0 || c.group % 16 != 0 || per_row < 2 || rows * per_row > 8192) return false;
  const int64_t spread = (tokens + 4 * num_sms() - 1) / (4 * num_sms());
  uint32_t log = 0;
  while ((2 << log) <= kMaxBlockTokens && (2 << log) * rows * per_row <= 1024 && (2 << log) <= spread) ++log;
  *p = {static_cast<uint32_t>(per_row), static_cast<uint32_t>(((1LL << 32) + per_row - 1) / per_row),
        static_cast<uint32_t>(rows), log};
  *grid = (tokens + (1LL << log) - 1) >> log;
  return *grid <= 0x7FFFFFFF;
}

template <typename T, bool ASYM>
cudaError_t write_typed(const WriteArgs& a, cudaStream_t stream) {
  const CacheView& c = a.cache;
  int lpg_log = 0;
  while ((16 << lpg_log) < c.group) ++lpg_log;
  Pieces p;
  int64_t grid;
  bool fast = c.head_dim % c.group == 0 && lpg_log <= 5 && multiple_of(c.packed, 8) &&
              cut(c, a.tokens, static_cast<int64_t>(c.groups) << lpg_log, &p, &grid);
  for (int kv = 0; kv < 2; ++kv)
    fast = fast && multiple_of(a.src[kv], 16) && (a.token_stride[kv] * sizeof(T)) % 16 == 0 &&
           (a.head_stride[kv] * sizeof(T)) % 16 == 0;
  if (fast) {
    cache_write_kernel<T, ASYM><<<static_cast<unsigned>(grid), 256, 0, stream>>>(a, p, lpg_log);
    return cudaGetLastError();
  }
  const int64_t warps = a.tokens * 2 * c.heads;
  cache_write_any_kernel<T, ASYM><<<resident_grid(cache_write_any_kernel<T, ASYM>, (warps + 7) / 8), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

template <typename TO, bool ASYM>
cudaError_t read_typed(const ReadArgs& a, cudaStream_t stream) {
  const CacheView& c = a.cache;
  Pieces p;
  int64_t grid;
  if (cut(c, a.tokens, c.head_dim / 16, &p, &grid) && multiple_of(c.packed, 8) && multiple_of(a.dst[0], 16) && multiple_of(a.dst[1], 16)) {
    cache_read_kernel<TO, ASYM><<<static_cast<unsigned>(grid), 256, 0, stream>>>(a, p);
    return cudaGetLastError();
  }
  const int64_t bytes = a.tokens * 2 * c.heads * c.row_bytes;
  cache_read_any_kernel<TO, ASYM><<<resident_grid(cache_read_any_kernel<TO, ASYM>, (bytes + 255) / 256), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t write_any_scheme(const WriteArgs& a, cudaStream_t s) {
  return a.cache.zeros != nullptr ? write_typed<T, true>(a, s) : write_typed<T, false>(a, s);
}
template <typename T>
cudaError_t read_any_scheme(const ReadArgs& a, cudaStream_t s) {
  return a.cache.zeros != nullptr ? read_typed<T, true>(a, s) : read_typed<T, false>(a, s);
}

}  // namespace

cudaError_t launch_cache_write(const CacheView& cache, const void* k, const void* v, DType t,
                               int64_t tokens, const int64_t (&token_stride)[2],
                               const int64_t (&head_stride)[2], const int64_t* slots,
                               cudaStream_t stream) {
  const WriteArgs a = {cache, {k, v}, {token_stride[0], token_stride[1]},
                       {head_stride[0], head_stride[1]}, slots, tokens};
  switch (t) {
    case DType::F32: return write_any_scheme<float>(a, stream);
    case DType::BF16: return write_any_scheme<__nv_bfloat16>(a, stream);
    default: return write_any_scheme<__half>(a, stream);
  }
}

cudaError_t launch_cache_read(const CacheView& cache, const int64_t* slots, int64_t tokens, void* k,
                              void* v, DType t, cudaStream_t stream) {
  const ReadArgs a = {cache, {k, v}, slots, tokens};
  switch (t) {
    case DType::F32: return read_any_scheme<float>(a, stream);
    case DType::BF16: return read_any_scheme<__nv_bfloat16>(a, stream);
    default: return read_any_scheme<__half>(a, stream);
  }
}

}  // namespace int4lib
