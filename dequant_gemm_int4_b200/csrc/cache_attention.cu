// Attention over the 4-bit key/value cache (sm_100a): the general kernel, and
// the choice between it and the tensor-core kernel.
//
// A query row q at position p of its sequence (the last query sits on the
// last cached token) sees the tokens j with 0 <= j < len, j <= p if causal
// and j > p - window if there is a window, and gets
//   S_j = sm_scale * sum_d q_d K_hat[j, d],   lse = log sum_j exp(S_j),
//   out = sum_j exp(S_j - lse) V_hat[j];      no visible token: 0 and -inf,
// with K_hat, V_hat the values that int4_cache_read gives in fp32.
#include "cache.cuh"
#include "cache_attention.cuh"
#include "internal.h"

namespace int4lib {

namespace {

constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Any head dimension up to 512, any group, page size, type and alignment:
// a block computes one query row of one head.  Its warps take tokens in
// turn; a lane holds the elements of bytes lane, lane + 32, ... of a row, so
// each row is one coalesced load.  fp32 throughout, each warp with its own
// running maximum and sum, joined at the end in warp order.
template <typename T, bool ASYM, int BYTES>  // BYTES: bytes of a row per lane
__global__ void __launch_bounds__(32 * kWarps) attention_any_kernel(
    const __grid_constant__ AttentionArgs a) {
  const CacheView& c = a.cache;
  const int t = blockIdx.x / a.q_heads;
  const int hq = blockIdx.x - t * a.q_heads;
  const int b = a.sequence_of(t);
  if (b < 0) return;  // a row of no sequence stays as it is
  const int h = hq / a.ratio;
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  int first, count, lo, hi;
  a.queries(b, first, count);
  const int len = a.kv_len(b);
  a.visible(len - count + (t - first), len, lo, hi);

  float q[2 * BYTES], o[2 * BYTES];
  const T* qp = static_cast<const T*>(a.q) + t * a.q_token_stride + hq * a.q_head_stride;
#pragma unroll
  for (int i = 0; i < BYTES; ++i) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int d = 2 * (lane + 32 * i) + k;
      const float x = d < c.head_dim ? Elem<T>::load(qp + d) : 0.0f;
      // Infinity counts as NaN: its products alone could give -infinity for
      // every score, as if the row saw nothing.
      q[2 * i + k] = fmaf(x, 0.0f, x);
      o[2 * i + k] = 0.0f;
    }
  }
  float m = __int_as_float(0xFF800000), l = 0.0f;  // in units of log2
  const float to_log2 = a.sm_scale * kLog2e;
  // Unsigned: hi may be 2^31 - 1, and the last step goes past it.
  const uint32_t page_size = c.page_size;
  for (uint32_t j = lo + warp; j < static_cast<uint32_t>(hi); j += kWarps) {
    const int64_t page = __ldg(a.page_table + b * a.table_stride + j / page_size);
    if (page < 0 || page >= c.pages) continue;  // no such page: its tokens are not there
    const int64_t kr = c.row(page, 0, h, j % page_size);
    const int64_t vr = c.row(page, 1, h, j % page_size);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < BYTES; ++i) {
      const int at = lane + 32 * i;
      if (at < c.row_bytes) {
        const uint32_t byte = __ldg(c.packed + kr * c.row_bytes + at);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int d = 2 * at + k;
          if (d < c.head_dim) {
            const int64_t g = kr * c.groups + d / c.group;
            const int zp = ASYM ? static_cast<int>(__ldg(c.zeros + g)) : 0;
            s = fmaf(q[2 * i + k],
                     code_value<ASYM>((byte >> (4 * k)) & 0xFu, zp) * f16_bits_to_float(__ldg(c.scales + g)), s);
          }
        }
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    s *= to_log2;
    const float m_new = fmaxf(m, s);
    const float base = m_new == __int_as_float(0xFF800000) ? 0.0f : m_new;
    const float old = exp2f(m - base), p = exp2f(s - base);
    m = m_new;
    l = fmaf(l, old, p);
#pragma unroll
    for (int i = 0; i < BYTES; ++i) {
      const int at = lane + 32 * i;
      const uint32_t byte = at < c.row_bytes ? __ldg(c.packed + vr * c.row_bytes + at) : 0u;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int d = 2 * at + k;
        if (d < c.head_dim) {
          const int64_t g = vr * c.groups + d / c.group;
          const int zp = ASYM ? static_cast<int>(__ldg(c.zeros + g)) : 0;
          const float v = code_value<ASYM>((byte >> (4 * k)) & 0xFu, zp) * f16_bits_to_float(__ldg(c.scales + g));
          o[2 * i + k] = fmaf(p, v, o[2 * i + k] * old);
        }
      }
    }
  }

  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][64 * BYTES];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < 2 * BYTES; ++i) so[warp][2 * (lane + 32 * (i >> 1)) + (i & 1)] = o[i];
  __syncthreads();
  float top = sm[0];
  for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sm[w]);
  const float base = top == __int_as_float(0xFF800000) ? 0.0f : top;
  float total = 0.0f;
  for (int w = 0; w < kWarps; ++w) total = fmaf(sl[w], exp2f(sm[w] - base), total);
  const int64_t at = static_cast<int64_t>(t) * a.q_heads + hq;
  for (int d = threadIdx.x; d < c.head_dim; d += blockDim.x) {
    float v = 0.0f;
    for (int w = 0; w < kWarps; ++w) v = fmaf(so[w][d], exp2f(sm[w] - base), v);
    // total == 0: nothing visible (a visible token at the maximum adds 1).
    store_as(static_cast<T*>(a.out) + at * c.head_dim + d, total == 0.0f ? 0.0f : v / total);
  }
  if (threadIdx.x == 0 && a.lse != nullptr)
    a.lse[at] = total == 0.0f ? __int_as_float(0xFF800000) : (base + log2f(total)) * kLn2;
}

template <typename T, bool ASYM>
cudaError_t launch_any_typed(const AttentionArgs& a, cudaStream_t stream) {
  const unsigned n = static_cast<unsigned>(a.rows) * a.q_heads;
  const int bytes = (a.cache.row_bytes + 31) / 32;
  if (bytes <= 2)
    attention_any_kernel<T, ASYM, 2><<<n, 32 * kWarps, 0, stream>>>(a);
  else if (bytes <= 4)
    attention_any_kernel<T, ASYM, 4><<<n, 32 * kWarps, 0, stream>>>(a);
  else
    attention_any_kernel<T, ASYM, 8><<<n, 32 * kWarps, 0, stream>>>(a);
  return cudaGetLastError();
}

bool multiple_of(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace

cudaError_t launch_cache_attention_any(const AttentionArgs& a, DType t, cudaStream_t stream) {
  const bool asym = a.cache.zeros != nullptr;
  switch (t) {
    case DType::F32:
      return asym ? launch_any_typed<float, true>(a, stream) : launch_any_typed<float, false>(a, stream);
    case DType::BF16:
      return asym ? launch_any_typed<__nv_bfloat16, true>(a, stream)
                  : launch_any_typed<__nv_bfloat16, false>(a, stream);
    default:
      return asym ? launch_any_typed<__half, true>(a, stream) : launch_any_typed<__half, false>(a, stream);
  }
}

namespace {

// The tensor-core kernels take 16-bit queries, heads of 64, 96, 128 or 256
// elements in groups of 32, 64, 128 or the whole head, and pages of a power
// of two of tokens, at least 16 (a block of 16 tokens then lies in one page).
// Token positions are 32-bit there, with room for a look-ahead of 16 steps.
// So are all counts of steps, of 128 tokens or more for each `row_tile` rows
// of a head.
bool mma_supported(const CacheView& c, DType t, const void* out, int64_t rows, int64_t batch, int ratio,
                   int64_t max_pages, int row_tile) {
  const int d = c.head_dim, g = c.group;
  const bool shape = (d == 64 || d == 96 || d == 128 || d == 256) && d % g == 0 &&
                     (g == 32 || g == d || (d != 96 && (g == 64 || g == 128)));
  const bool pages = c.page_size >= 16 && (c.page_size & (c.page_size - 1)) == 0 &&
                     max_pages * c.page_size <= (1LL << 30) &&
                     static_cast<double>(c.heads) * (static_cast<double>(rows) * ratio / row_tile + batch) *
                             (static_cast<double>(max_pages) * c.page_size / 128 + 1) < 0x7FFF0000;
  return t != DType::F32 && shape && pages && multiple_of(c.packed, 16) && multiple_of(c.scales, 16) &&
         multiple_of(c.zeros, 16) && multiple_of(out, 8);
}

}  // namespace

bool cache_attention_mma_supported(const CacheView& c, DType t, const void* out, int64_t rows, int64_t batch,
                                   int ratio, int64_t max_pages) {
  const int rt = batch > 0 ? attention_row_tile(c.head_dim, c.group, rows, batch, ratio) : 8;
  return mma_supported(c, t, out, rows, batch, ratio, max_pages, rt);
}

// The tcgen05 kernel takes heads of 64, 96 or 128 elements in one group or in
// groups of 32 or 64, and outputs aligned to 16 bytes.
bool cache_prefill_supported(const CacheView& c, DType t, const void* out, int64_t rows, int64_t batch, int ratio,
                             int64_t max_pages) {
  return (c.head_dim == 64 || c.head_dim == 96 || c.head_dim == 128) && multiple_of(out, 16) &&
         mma_supported(c, t, out, rows, batch, ratio, max_pages, kPrefillRowTile);
}

// By head, groups and type, as the two kernels were measured: 32 sequences of
// 4096 tokens, 8 heads, random codes, us with the kernels for few rows / with the
// tcgen05 kernel:
//   rows                         80          96         112         128         144
//   128, one group          223 / 244   244 / 252   303 / 255   317 / 259   384 / 263
//   128, groups of 64       274 / 342   287 / 345   373 / 348   374 / 349   471 / 352
//   128, groups of 64, fp16 274 / 414   288 / 417   373 / 418   373 / 420   471 / 423
//   128, groups of 32       344 / 343   425 / 344   466 / 347   557 / 348   596 / 350
//   128, groups of 32, fp16 344 / 415   425 / 415   466 / 418   555 / 420   594 / 424
//   96, one group           190 / 236   204 / 237   256 / 242   263 / 246   325 / 249
//   96, groups of 32        230 / 257   264 / 260   313 / 263   343 / 269   398 / 268
//   96, groups of 32, fp16  230 / 313   264 / 315   313 / 317   343 / 320   398 / 322
//   64, one group           151 / 214   180 / 221   205 / 225   231 / 228   260 / 237
//   64, groups of 32        166 / 235   196 / 238   225 / 243   254 / 244   284 / 250
//   64, groups of 32, fp16  165 / 244   196 / 246   225 / 250   254 / 253   285 / 257
// (types that are not named are alike).  One sequence alone, of 16384 tokens, would
// be better off with the kernels for few rows up to 160 rows or so (heads of 128 in
// one group: 128 rows 61 / 69, 160 69 / 74, 256 94 / 88).
int cache_few_rows(const CacheView& c, DType t) {
  const bool fp16 = t == DType::F16;
  if (c.head_dim == 64) return 112;
  if (c.head_dim == 128 && c.group == 64) return fp16 ? 128 : 96;
  if (c.head_dim == 128 && c.group == 32) return fp16 ? 80 : 64;
  return 96;
}

size_t cache_prefill_workspace(const CacheView& c, int64_t batch) {
  return attention_space_bytes(batch, num_sms(), kPrefillRowTile, c.head_dim);
}

size_t cache_attention_mma_workspace(const CacheView& c, int64_t rows, int64_t batch, int ratio) {
  const int rt = attention_row_tile(c.head_dim, c.group, rows, batch, ratio);
  const bool asym = c.zeros != nullptr;
  int blocks = 0;
  switch (c.head_dim) {
    case 64: blocks = cache_attention_blocks_64(c.group, asym, rt); break;
    case 96: blocks = cache_attention_blocks_96(c.group, asym, rt); break;
    case 128: blocks = cache_attention_blocks_128(c.group, asym, rt); break;
    default: blocks = cache_attention_blocks_256(c.group, asym, rt); break;
  }
  return attention_space_bytes(batch, blocks, rt, c.head_dim);
}

cudaError_t launch_cache_prefill(const AttentionArgs& a, DType t, void* workspace, cudaStream_t stream) {
  switch (a.cache.head_dim) {
    case 64: return launch_cache_prefill_64(a, t, workspace, stream);
    case 96: return launch_cache_prefill_96(a, t, workspace, stream);
    default: return launch_cache_prefill_128(a, t, workspace, stream);
  }
}

cudaError_t launch_cache_attention_mma(const AttentionArgs& a, DType t, void* workspace, cudaStream_t stream) {
  const int rt = attention_row_tile(a.cache.head_dim, a.cache.group, a.rows, a.batch, a.ratio);
  switch (a.cache.head_dim) {
    case 64: return launch_cache_attention_64(a, t, rt, workspace, stream);
    case 96: return launch_cache_attention_96(a, t, rt, workspace, stream);
    case 128: return launch_cache_attention_128(a, t, rt, workspace, stream);
    default: return launch_cache_attention_256(a, t, rt, workspace, stream);
  }
}

}  // namespace int4lib
