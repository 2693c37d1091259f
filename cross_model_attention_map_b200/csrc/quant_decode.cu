// Decode over a quantised paged cache (format: quant_cache.cuh):
//
//   iamap_sender_rows_quant      p[b, h, j] = softmax over j < ctx[b] of q[b, h] . k^[b, j] / sqrt(d)
//   iamap_mapped_av_paged_quant  out[b, r] = sum_j (sum_s W[r, s] p[b, s, j]) v^[b, j]
//   iamap_attention_paged_quant  out[b, h] = sum_j softmax(...)_j v^[b, j], and the log-sum-exp
//
// with query (receiver) head h reading key (value) head h / group. First form: one CTA a head and
// sequence walks the context 128 tokens at a time, one token a thread for scores and weights, one
// element a thread for the products.
#include <algorithm>

#include "internal.h"
#include "quant_cache.cuh"

namespace iamap {
namespace {

constexpr int kTile = 128;     // tokens at a time = threads a CTA

struct QuantDecodeParams {
  const __nv_bfloat16* q;      // [batch, Hq, d]
  QuantPages k, v;
  int k_bits, v_bits;
  const int32_t* ctx_lens;
  int max_ctx;
  int Hq, d;
  float scale_log2;            // log2(e) / sqrt(d)
  float* rows;                 // rows out (softmax rows) or mapped in, [batch, *, stride]
  int stride;
  const float* W;              // [Hq, H_s]
  int H_s;
  float* out_f32;
  __nv_bfloat16* out_bf16;
  float* lse;
  unsigned int* status;
};

// Code of stored place `at` of a row.
__device__ __forceinline__ float quant_code(const uint8_t* row, int at, int bits) {
  if (bits == 8) return (float)((int)row[at] - 128);
  return (float)((int)((row[at >> 1] >> ((at & 1) * 4)) & 15) - 8);
}

__device__ float quant_dot(const QuantPages& k, int bits, int64_t row, int d, const float* q_s) {
  const uint8_t* c = k.codes + row * (d * bits / 8);
  const int ng = d / kQuantGroup;
  float x = 0.f;
  for (int g = 0; g < ng; ++g) {
    float a = 0.f;
    for (int e = 0; e < kQuantGroup; ++e)
      a = fmaf(quant_code(c, (e >> 2) * (d / 8) + 4 * g + (e & 3), bits), q_s[g * 32 + e], a);
    x = fmaf(a, __half2float(k.scales[row * ng + g]), x);
  }
  return x;
}

__device__ __forceinline__ float quant_value(const QuantPages& v, int bits, int64_t row, int d,
                                             int e) {
  const uint8_t* c = v.codes + row * (d * bits / 8);
  const int g = e / kQuantGroup, r = (e % kQuantGroup) >> 2;
  return quant_code(c, r * (d / 8) + 4 * g + (e & 3), bits) *
         __half2float(v.scales[row * (d / kQuantGroup) + g]);
}

__device__ float block_max(float x, float* red) {
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  return fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
}
__device__ float block_sum(float x, float* red) {
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

// Softmax rows and attention: the online softmax of one query head.
template <bool ROWS>
__global__ void __launch_bounds__(kTile) quant_softmax_kernel(QuantDecodeParams p) {
  __shared__ float q_s[128], p_s[kTile], red[4];
  __shared__ int64_t row_s[kTile];
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const int ctx = quant_ctx(p.ctx_lens, b, p.max_ctx, p.status);
  const int kh = h / (p.Hq / p.k.H);
  if (tid < p.d) q_s[tid] = __bfloat162float(p.q[((int64_t)b * p.Hq + h) * p.d + tid]);
  __syncthreads();
  float* prow = ROWS ? p.rows + ((int64_t)b * p.Hq + h) * p.stride : nullptr;
  float m = -INFINITY, z = 0.f, o = 0.f;
  for (int j0 = 0; j0 < ctx; j0 += kTile) {
    const int j = j0 + tid;
    float x = -INFINITY;
    int64_t vrow = -1;
    if (j < ctx) {
      const int64_t row = quant_row(p.k, b, kh, j);
      if (row >= 0)
        x = quant_dot(p.k, p.k_bits, row, p.d, q_s) * p.scale_log2;
      else
        raise_status(p.status, IAMAP_DEV_BAD_INDEX);
      if (!ROWS) vrow = quant_row(p.v, b, kh, j);
      if (!ROWS && vrow < 0) x = -INFINITY;      // a bad page: probability 0
      if (ROWS) prow[j] = x;
    }
    const float mn = fmaxf(m, block_max(x, red));
    const float e = mn == -INFINITY ? 0.f : exp2f(x - mn);
    const float f = mn == -INFINITY ? 1.f : exp2f(m - mn);
    z = z * f + block_sum(e, red);
    m = mn;
    if (!ROWS) {
      p_s[tid] = e;
      row_s[tid] = vrow;
      __syncthreads();
      o *= f;
      if (tid < p.d)
        for (int t = 0; t < min(kTile, ctx - j0); ++t)
          if (row_s[t] >= 0) o = fmaf(p_s[t], quant_value(p.v, p.v_bits, row_s[t], p.d, tid), o);
    }
  }
  if (ROWS) {
    const float lse = m + log2f(z);
    for (int j = tid; j < p.stride; j += kTile)
      prow[j] = j < ctx && m != -INFINITY ? exp2f(prow[j] - lse) : 0.f;
  } else {
    const int64_t at = (int64_t)b * p.Hq + h;
    if (tid < p.d) p.out_bf16[at * p.d + tid] = __float2bfloat16(z == 0.f ? 0.f : o / z);
    if (tid == 0 && p.lse) p.lse[at] = (m + log2f(z)) * kLn2;
  }
}

__global__ void __launch_bounds__(kTile) quant_mapped_kernel(QuantDecodeParams p) {
  __shared__ float p_s[kTile];
  __shared__ int64_t row_s[kTile];
  const int r = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const int ctx = quant_ctx(p.ctx_lens, b, p.max_ctx, p.status);
  const int vh = r / (p.Hq / p.v.H);
  float o = 0.f;
  for (int j0 = 0; j0 < ctx; j0 += kTile) {
    const int j = j0 + tid;
    float w = 0.f;
    int64_t row = -1;
    if (j < ctx) {
      for (int s = 0; s < p.H_s; ++s)
        w = fmaf(p.W[r * p.H_s + s], p.rows[((int64_t)b * p.H_s + s) * p.stride + j], w);
      row = quant_row(p.v, b, vh, j);
      if (row < 0) raise_status(p.status, IAMAP_DEV_BAD_INDEX);
    }
    __syncthreads();
    p_s[tid] = w;
    row_s[tid] = row;
    __syncthreads();
    if (tid < p.d)
      for (int t = 0; t < min(kTile, ctx - j0); ++t)
        if (row_s[t] >= 0) o = fmaf(p_s[t], quant_value(p.v, p.v_bits, row_s[t], p.d, tid), o);
  }
  if (tid < p.d) p.out_f32[((int64_t)b * p.Hq + r) * p.d + tid] = o;
}

QuantPages pages_of(const void* codes, const void* scales, int64_t num_pages, const int32_t* table,
                    int max_pages, int page_size, int H) {
  return QuantPages{static_cast<const uint8_t*>(codes), static_cast<const __half*>(scales),
                    num_pages, table, max_pages, page_size, H};
}

}  // namespace
}  // namespace iamap

using namespace iamap;

extern "C" size_t iamap_sender_rows_quant_workspace_bytes(int batch, int H_s, int max_ctx) {
  if (batch < 1 || H_s < 1 || max_ctx < 0) return 0;
  return 256;
}

extern "C" int iamap_sender_rows_quant(const void* q, const void* k_codes, const void* k_scales,
                                       int64_t num_pages, const int32_t* page_table, int max_pages,
                                       int page_size, const int32_t* ctx_lens, int max_ctx,
                                       int batch, int H_s, int H_k, int d, int bits, float* p_rows,
                                       int ctx_stride, void* ws, size_t ws_bytes, void* stream) {
  clear_error();
  int rc = check_quant_pages(k_codes, k_scales, num_pages, page_table, max_pages, page_size, H_k, d,
                             bits);
  if (rc) return rc;
  rc = check_quant_batch(ctx_lens, max_ctx, batch, max_pages, page_size);
  if (rc) return rc;
  if (H_s < 1 || H_s % H_k != 0)
    return set_error(IAMAP_ERR_INVALID_ARG, "H_k=%d must divide H_s=%d", H_k, H_s);
  if (!q || !p_rows) return set_error(IAMAP_ERR_INVALID_ARG, "null pointer");
  if ((reinterpret_cast<uintptr_t>(q) & 15u) != 0)
    return set_error(IAMAP_ERR_INVALID_ARG, "q must be 16-byte aligned");
  if (ctx_stride < 1 || ctx_stride < max_ctx)
    return set_error(IAMAP_ERR_INVALID_ARG, "ctx_stride=%d is below max_ctx=%d", ctx_stride, max_ctx);
  const size_t need = iamap_sender_rows_quant_workspace_bytes(batch, H_s, max_ctx);
  if (!ws || ws_bytes < need)
    return set_error(IAMAP_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws_bytes);
  DeviceContext* ctx = device_context();
  if (!ctx) return IAMAP_ERR_CUDA;
  QuantDecodeParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = pages_of(k_codes, k_scales, num_pages, page_table, max_pages, page_size, H_k);
  p.k_bits = bits;
  p.ctx_lens = ctx_lens;
  p.max_ctx = max_ctx;
  p.Hq = H_s;
  p.d = d;
  p.scale_log2 = kLog2e / sqrtf((float)d);
  p.rows = p_rows;
  p.stride = ctx_stride;
  p.status = ctx->status;
  quant_softmax_kernel<true><<<dim3(H_s, batch), kTile, 0, static_cast<cudaStream_t>(stream)>>>(p);
  IAMAP_LAUNCH_CHECK("quant_softmax_kernel");
  return IAMAP_OK;
}
