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
// Both are bound by HBM for long runs of tokens and by launch latency for a
// decoding step's few tokens.
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
    const float d = ASYM ? __fdiv_rn(__fsub_rn(hi, lo), 15.0f) : __fdiv_rn(hi, 7.0f);
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

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
template <>
__device__ __forceinline__ void load8<__half>(const __half* p, float (&v)[8]) {
  const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = f16_bits_to_float(w[i] & 0xFFFFu);
    v[2 * i + 1] = f16_bits_to_float(w[i] >> 16);
  }
}

// D a multiple of 8, group = 8 LPG dividing D with LPG a power of two <= 32,
// every source row 16-byte aligned, packed 4-byte aligned.  A thread codes 8
// consecutive elements of one row (one 16-byte load of 16-bit elements, one
// 4-byte store); the LPG lanes of a group find its extremes with shuffles.
// A block takes `per_block` whole tokens; `chunks` = 2 H D / 8 of a token.
template <typename T, bool ASYM>
__global__ void __launch_bounds__(256) cache_write_kernel(const __grid_constant__ WriteArgs a,
                                                          int chunks, int per_block, int lpg) {
  const CacheView& c = a.cache;
  const int per_row = c.head_dim >> 3;
  const int64_t token0 = static_cast<int64_t>(blockIdx.x) * per_block;
  const int total = per_block * chunks;
  // Whole warps take part in every step, so that the shuffles are uniform.
  for (int base = 0; base < total; base += blockDim.x) {
    const int i = base + threadIdx.x;
    const int64_t t = token0 + i / chunks;
    bool live = i < total && t < a.tokens;
    int64_t slot = live ? __ldg(a.slots + t) : -1;
    live = slot >= 0 && slot < c.pages * c.page_size;
    const int chunk = i % chunks;
    const int row = chunk / per_row;  // kv * H + h
    const int d = (chunk - row * per_row) * 8;
    const int kv = row >= c.heads ? 1 : 0;
    const int h = row - kv * c.heads;
    float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (live)
      load8<T>(static_cast<const T*>(a.src[kv]) + t * a.token_stride[kv] + h * a.head_stride[kv] + d, v);
    float lo = ASYM ? v[0] : 0.0f, hi = ASYM ? v[0] : fabsf(v[0]);
#pragma unroll
    for (int k = 1; k < 8; ++k) {
      if (ASYM) lo = fminf(lo, v[k]);
      hi = fmaxf(hi, ASYM ? v[k] : fabsf(v[k]));
    }
    for (int off = 1; off < lpg; off <<= 1) {
      if (ASYM) lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
    }
    if (!live) continue;
    Coder q;
    q.set<ASYM>(lo, hi);
    uint32_t word = 0u;
#pragma unroll
    for (int k = 0; k < 8; ++k) word |= q.code<ASYM>(v[k]) << (4 * k);
    const int64_t at = c.row(slot / c.page_size, kv, h, slot % c.page_size);
    *reinterpret_cast<uint32_t*>(c.packed + at * c.row_bytes + (d >> 1)) = word;
    if ((threadIdx.x & (lpg - 1)) == 0) {
      const int64_t g = at * c.groups + d / c.group;
      c.scales[g] = q.bits;
      if (ASYM) c.zeros[g] = static_cast<uint8_t>(q.z);
    }
  }
}

// Any D, group, stride and alignment: a warp codes one row.
template <typename T, bool ASYM>
__global__ void __launch_bounds__(256) cache_write_any_kernel(const __grid_constant__ WriteArgs a) {
  const CacheView& c = a.cache;
  const int lane = threadIdx.x & 31;
  const int rows = 2 * c.heads;
  const int64_t total = a.tokens * rows;
  const int64_t step = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
  for (int64_t w = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; w < total; w += step) {
    const int64_t t = w / rows;
    const int row = static_cast<int>(w - t * rows);
    const int kv = row >= c.heads ? 1 : 0;
    const int h = row - kv * c.heads;
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
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
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

// D and group multiples of 8, packed 4-byte and outputs 16-byte aligned: a
// thread gives 8 consecutive elements of one row.
template <typename TO, bool ASYM>
__global__ void __launch_bounds__(256) cache_read_kernel(const __grid_constant__ ReadArgs a, int chunks,
                                                         int per_block) {
  const CacheView& c = a.cache;
  const int per_row = c.head_dim >> 3;
  const int64_t token0 = static_cast<int64_t>(blockIdx.x) * per_block;
  const int total = per_block * chunks;
  for (int i = threadIdx.x; i < total; i += blockDim.x) {
    const int64_t t = token0 + i / chunks;
    if (t >= a.tokens) return;
    const int64_t slot = __ldg(a.slots + t);
    const int chunk = i % chunks;
    const int row = chunk / per_row;
    const int d = (chunk - row * per_row) * 8;
    const int kv = row >= c.heads ? 1 : 0;
    const int h = row - kv * c.heads;
    float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (slot >= 0 && slot < c.pages * c.page_size) {
      const int64_t at = c.row(slot / c.page_size, kv, h, slot % c.page_size);
      const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(c.packed + at * c.row_bytes + (d >> 1)));
      const int64_t g = at * c.groups + d / c.group;
      const float s = f16_bits_to_float(__ldg(c.scales + g));
      const int zp = ASYM ? static_cast<int>(__ldg(c.zeros + g)) : 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = code_value<ASYM>((w >> (4 * k)) & 0xFu, zp) * s;
    }
    TO* out = static_cast<TO*>(a.dst[kv]) + (t * c.heads + h) * c.head_dim + d;
    store8<TO>(out, v);
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
    const int row = static_cast<int>(in_token / c.row_bytes);
    const int b = static_cast<int>(in_token - static_cast<int64_t>(row) * c.row_bytes);
    const int kv = row >= c.heads ? 1 : 0;
    const int h = row - kv * c.heads;
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

template <typename T, bool ASYM>
cudaError_t write_typed(const WriteArgs& a, cudaStream_t stream) {
  const CacheView& c = a.cache;
  const int lpg = c.group / 8;
  const int64_t chunks = 2LL * c.heads * (c.head_dim / 8);
  bool fast = c.head_dim % 8 == 0 && c.group % 8 == 0 && lpg <= 32 && (lpg & (lpg - 1)) == 0 &&
              c.head_dim % c.group == 0 && multiple_of(c.packed, 4) && chunks <= (1 << 20);
  for (int kv = 0; kv < 2; ++kv)
    fast = fast && multiple_of(a.src[kv], 16) && (a.token_stride[kv] * sizeof(T)) % 16 == 0 &&
           (a.head_stride[kv] * sizeof(T)) % 16 == 0;
  if (fast) {
    const int per_block = chunks >= 256 ? 1 : static_cast<int>(256 / chunks);
    const int64_t grid = (a.tokens + per_block - 1) / per_block;
    if (grid <= 0x7FFFFFFF) {
      cache_write_kernel<T, ASYM><<<static_cast<unsigned>(grid), 256, 0, stream>>>(
          a, static_cast<int>(chunks), per_block, lpg);
      return cudaGetLastError();
    }
  }
  const int64_t warps = a.tokens * 2 * c.heads;
  const int grid = resident_grid(cache_write_any_kernel<T, ASYM>, (warps + 7) / 8);
  cache_write_any_kernel<T, ASYM><<<grid, 256, 0, stream>>>(a);
  return cudaGetLastError();
}

template <typename TO, bool ASYM>
cudaError_t read_typed(const ReadArgs& a, cudaStream_t stream) {
  const CacheView& c = a.cache;
  const int64_t chunks = 2LL * c.heads * (c.head_dim / 8);
  const bool fast = c.head_dim % 8 == 0 && c.group % 8 == 0 && multiple_of(c.packed, 4) &&
                    multiple_of(a.dst[0], 16) && multiple_of(a.dst[1], 16) && chunks <= (1 << 20);
  if (fast) {
    const int per_block = chunks >= 256 ? 1 : static_cast<int>(256 / chunks);
    const int64_t grid = (a.tokens + per_block - 1) / per_block;
    if (grid <= 0x7FFFFFFF) {
      cache_read_kernel<TO, ASYM><<<static_cast<unsigned>(grid), 256, 0, stream>>>(
          a, static_cast<int>(chunks), per_block);
      return cudaGetLastError();
    }
  }
  const int64_t bytes = a.tokens * 2 * c.heads * c.row_bytes;
  const int grid = resident_grid(cache_read_any_kernel<TO, ASYM>, (bytes + 255) / 256);
  cache_read_any_kernel<TO, ASYM><<<grid, 256, 0, stream>>>(a);
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
