// iamap_cache_write / iamap_cache_read: quantising new keys or values into their pages, and reading
// ranges of sequences back as packed bf16 rows (format: quant_cache.cuh).
//
//   m = max |x| of a group of 32,  s = fp16(min(m / Q, 65504)),  c = clamp(rint(x / s), -Q, Q)
//
// Both are bound by HBM: 2 + bits / 8 + 1 / 16 bytes an element.
#include "internal.h"
#include "quant_cache.cuh"

namespace iamap {
namespace {

constexpr int kThreads = 256;

struct CacheIoParams {
  const __nv_bfloat16* x;   // write: rows to quantise, x_stride elements apart
  __nv_bfloat16* out;       // read: rows to fill, packed
  int64_t x_stride;
  int64_t n;                // rows of x / out
  const int32_t* cu;        // [num_seqs + 1] rows of each sequence
  const int32_t* starts;    // [num_seqs] position of each sequence's first row
  int num_seqs;
  int d;
  QuantPages pages;
  uint8_t* codes;           // write: pages.codes, pages.scales
  __half* scales;
  unsigned int* status;
};

// Cache row of packed row i and head h: -1 if the row belongs to no sequence (a padded batch),
// -2 if its position or page is out of range.
__device__ __forceinline__ int64_t place_of(const CacheIoParams& p, int64_t i, int h) {
  if (i < p.cu[0] || i >= p.cu[p.num_seqs]) return -1;
  int lo = 0, hi = p.num_seqs;          // cu[lo] <= i < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.cu[mid] <= i) lo = mid; else hi = mid;
  }
  const int64_t pos = (int64_t)p.starts[lo] + (i - p.cu[lo]);
  if (pos < 0 || pos >= (int64_t)p.pages.max_pages * p.pages.page_size || pos > 0x7fffffff)
    return -2;
  const int64_t row = quant_row(p.pages, lo, h, (int)pos);
  return row < 0 ? -2 : row;
}

// Four lanes a group: each holds eight elements (two runs of four).
template <int BITS>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(CacheIoParams p) {
  constexpr int Q = BITS == 4 ? 7 : 127;
  const int lanes = p.d / 8;                               // lanes a row
  const int64_t unit = (int64_t)blockIdx.x * (kThreads / lanes) + threadIdx.x / lanes;
  const int l = threadIdx.x % lanes, g = l >> 2, t = l & 3;
  const int64_t i = unit / p.pages.H;
  const int h = (int)(unit - i * p.pages.H);
  const int64_t row = i < p.n ? place_of(p, i, h) : -1;
  uint4 raw = make_uint4(0, 0, 0, 0);
  if (row >= 0)
    raw = __ldcs(reinterpret_cast<const uint4*>(p.x + i * p.x_stride + (int64_t)h * p.d + 8 * l));
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  // largest magnitude by the bits: infinities and NaN compare above every finite value
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) m = max(m, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  if (row == -2) raise_status(p.status, IAMAP_DEV_BAD_INDEX);
  if (row < 0) return;
  __half s = __float2half_rn(fminf(__fdiv_rn(__uint_as_float(m << 16), (float)Q), 65504.f));
  if (m >= 0x7f80u) s = __ushort_as_half(0x7e00);          // a group with an infinity or NaN
  const float sf = __half2float(s);
  uint32_t u[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = __uint_as_float(e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
    const float c = sf > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(x, sf)), (float)-Q), (float)Q) : 0.f;
    u[e] = (uint32_t)((int)c + (BITS == 4 ? 8 : 128));
  }
  const int ng = p.d / kQuantGroup;
  if (t == 0) p.scales[row * ng + g] = s;
  if (BITS == 4) {
    uint16_t* dst = reinterpret_cast<uint16_t*>(p.codes + row * (p.d / 2));
    dst[(2 * t) * ng + g] = (uint16_t)(u[0] | u[1] << 4 | u[2] << 8 | u[3] << 12);
    dst[(2 * t + 1) * ng + g] = (uint16_t)(u[4] | u[5] << 4 | u[6] << 8 | u[7] << 12);
  } else {
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.codes + row * p.d);
    dst[(2 * t) * ng + g] = u[0] | u[1] << 8 | u[2] << 16 | u[3] << 24;
    dst[(2 * t + 1) * ng + g] = u[4] | u[5] << 8 | u[6] << 16 | u[7] << 24;
  }
}

template <int BITS>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(CacheIoParams p) {
  const int lanes = p.d / 8;
  const int64_t unit = (int64_t)blockIdx.x * (kThreads / lanes) + threadIdx.x / lanes;
  const int l = threadIdx.x % lanes, g = l >> 2, t = l & 3;
  const int64_t i = unit / p.pages.H;
  const int h = (int)(unit - i * p.pages.H);
  if (i >= p.n) return;
  const int64_t row = place_of(p, i, h);
  if (row == -1) return;                                   // rows behind the last sequence
  uint4 o = make_uint4(0, 0, 0, 0);
  if (row >= 0) {
    const int ng = p.d / kQuantGroup;
    const float s = __half2float(p.pages.scales[row * ng + g]);
    float v[8];
    if (BITS == 4) {
      const uint16_t* src = reinterpret_cast<const uint16_t*>(p.pages.codes + row * (p.d / 2));
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t c = src[(2 * t + r) * ng + g];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * r + e] = (float)((int)((c >> (4 * e)) & 15u) - 8) * s;
      }
    } else {
      const uint32_t* src = reinterpret_cast<const uint32_t*>(p.pages.codes + row * p.d);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t c = src[(2 * t + r) * ng + g];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * r + e] = (float)((int)((c >> (8 * e)) & 255u) - 128) * s;
      }
    }
    o = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                   pack_bf16(v[6], v[7]));
  } else {
    raise_status(p.status, IAMAP_DEV_BAD_INDEX);
  }
  *reinterpret_cast<uint4*>(p.out + (i * p.pages.H + h) * p.d + 8 * l) = o;
}

int cache_io_check(const void* rows, const int32_t* cu, const int32_t* starts, int num_seqs,
                   int64_t n) {
  if (!rows || !cu || !starts) return set_error(IAMAP_ERR_INVALID_ARG, "null pointer");
  if (num_seqs < 1 || n < 0 || n > 0x7fffffff)
    return set_error(IAMAP_ERR_INVALID_ARG, "need num_seqs >= 1 and 0 <= n < 2^31");
  if ((reinterpret_cast<uintptr_t>(rows) & 15u) != 0)
    return set_error(IAMAP_ERR_INVALID_ARG, "the bf16 rows must be 16-byte aligned");
  return IAMAP_OK;
}

int cache_io_grid(int64_t n, int H, int d, unsigned int* blocks) {
  const int64_t per = kThreads / (d / 8);
  const int64_t b = (n * H + per - 1) / per;
  if (b > 0x7fffffff) return set_error(IAMAP_ERR_UNSUPPORTED, "too many rows for one call");
  *blocks = (unsigned int)b;
  return IAMAP_OK;
}

}  // namespace

int check_quant_pages(const void* codes, const void* scales, int64_t num_pages,
                      const int32_t* page_table, int max_pages, int page_size, int H, int d,
                      int bits) {
  if (bits != 4 && bits != 8)
    return set_error(IAMAP_ERR_UNSUPPORTED, "a cache holds 4 or 8 bits an element, not %d", bits);
  if (d != 64 && d != 128) return set_error(IAMAP_ERR_UNSUPPORTED, "head dim must be 64 or 128");
  if (!codes || !scales || !page_table) return set_error(IAMAP_ERR_INVALID_ARG, "null pointer");
  if (num_pages < 0 || max_pages < 0 || page_size < 1 || H < 1)
    return set_error(IAMAP_ERR_INVALID_ARG, "bad sizes of the cache");
  if (((reinterpret_cast<uintptr_t>(codes) | reinterpret_cast<uintptr_t>(scales)) & 15u) != 0)
    return set_error(IAMAP_ERR_INVALID_ARG, "codes and scales must be 16-byte aligned");
  // the kernels number the (page, head, slot) rows in 32 bits
  if (num_pages > 0 && (int64_t)H * page_size > 0xffffffffll / num_pages)
    return set_error(IAMAP_ERR_UNSUPPORTED, "num_pages * H * page_size must be below 2^32");
  return IAMAP_OK;
}

int check_quant_batch(const int32_t* ctx_lens, int max_ctx, int batch, int max_pages,
                      int page_size) {
  if (!ctx_lens) return set_error(IAMAP_ERR_INVALID_ARG, "null pointer");
  if (batch < 1 || max_ctx < 0) return set_error(IAMAP_ERR_INVALID_ARG, "bad sizes");
  if ((int64_t)max_ctx > (int64_t)max_pages * page_size)
    return set_error(IAMAP_ERR_INVALID_ARG, "max_ctx=%d exceeds the page table", max_ctx);
  if (max_ctx > 1 << 30) return set_error(IAMAP_ERR_UNSUPPORTED, "max_ctx must be at most 2^30");
  return IAMAP_OK;
}

}  // namespace iamap

using namespace iamap;

extern "C" int iamap_cache_write(const void* x, int64_t x_stride, int64_t n, const int32_t* cu,
                                 const int32_t* starts, int num_seqs, const int32_t* page_table,
                                 int max_pages, int page_size, int64_t num_pages, int H, int d,
                                 int bits, void* codes, void* scales, void* stream) {
  clear_error();
  int rc = check_quant_pages(codes, scales, num_pages, page_table, max_pages, page_size, H, d, bits);
  if (rc) return rc;
  rc = cache_io_check(x, cu, starts, num_seqs, n);
  if (rc) return rc;
  if (x_stride < (int64_t)H * d || x_stride % 8 != 0)
    return set_error(IAMAP_ERR_INVALID_ARG, "x_stride must be a multiple of 8, at least H * d");
  unsigned int blocks = 0;
  rc = cache_io_grid(n, H, d, &blocks);
  if (rc) return rc;
  if (blocks == 0) return IAMAP_OK;
  DeviceContext* ctx = device_context();
  if (!ctx) return IAMAP_ERR_CUDA;
  CacheIoParams p{};
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.x_stride = x_stride;
  p.n = n;
  p.cu = cu;
  p.starts = starts;
  p.num_seqs = num_seqs;
  p.d = d;
  p.codes = static_cast<uint8_t*>(codes);
  p.scales = static_cast<__half*>(scales);
  p.pages = QuantPages{p.codes, p.scales, num_pages, page_table, max_pages, page_size, H};
  p.status = ctx->status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (bits == 4)
    cache_write_kernel<4><<<blocks, kThreads, 0, st>>>(p);
  else
    cache_write_kernel<8><<<blocks, kThreads, 0, st>>>(p);
  IAMAP_LAUNCH_CHECK("cache_write_kernel");
  return IAMAP_OK;
}

extern "C" int iamap_cache_read(const void* codes, const void* scales, int64_t num_pages,
                                const int32_t* page_table, int max_pages, int page_size,
                                const int32_t* cu, const int32_t* starts, int num_seqs, int64_t n,
                                int H, int d, int bits, void* out, void* stream) {
  clear_error();
  int rc = check_quant_pages(codes, scales, num_pages, page_table, max_pages, page_size, H, d, bits);
  if (rc) return rc;
  rc = cache_io_check(out, cu, starts, num_seqs, n);
  if (rc) return rc;
  unsigned int blocks = 0;
  rc = cache_io_grid(n, H, d, &blocks);
  if (rc) return rc;
  if (blocks == 0) return IAMAP_OK;
  DeviceContext* ctx = device_context();
  if (!ctx) return IAMAP_ERR_CUDA;
  CacheIoParams p{};
  p.out = static_cast<__nv_bfloat16*>(out);
  p.n = n;
  p.cu = cu;
  p.starts = starts;
  p.num_seqs = num_seqs;
  p.d = d;
  p.pages = QuantPages{static_cast<const uint8_t*>(codes), static_cast<const __half*>(scales),
                       num_pages, page_table, max_pages, page_size, H};
  p.status = ctx->status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (bits == 4)
    cache_read_kernel<4><<<blocks, kThreads, 0, st>>>(p);
  else
    cache_read_kernel<8><<<blocks, kThreads, 0, st>>>(p);
  IAMAP_LAUNCH_CHECK("cache_read_kernel");
  return IAMAP_OK;
}
