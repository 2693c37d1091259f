// iamap_sender_rows_quant: the small model's attention rows over a quantised key cache.
//
//   p[b, h, j] = 2^(x_j - ref) / z,  x_j = q[b, h] . k^[b, j, h / group] log2(e) / sqrt(d),  j < ctx[b]
//
// Bound by the key bytes (36 a token and head of 64 in 4 bits) and the rows written (4 bytes a token
// and query head). The first kernel streams the keys as quant_attention.cu does, writes x in place of p
// and the (reference, sum) of each range of tokens; the second joins a row's ranges in their order and
// normalises its tokens, which are still in L2. Where max_ctx fits one range the first kernel does it all.
// Four sequences of 8704 tokens, 14 heads of 64 in 4 bits: 14.4 us a pass; sixteen of up to 32768, 14 heads
// on 2 key heads in 8 bits: 20.5 us. Both are mostly latency: the lengths, the page table, the codes and the join
// are read one after the other.
#include <algorithm>

#include "internal.h"
#include "quant_tile.cuh"

namespace iamap {
namespace {

using namespace qt;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kHeads = 8;            // query heads a CTA
constexpr float kNoRef = -3e38f;

struct RowsParams {
  const __nv_bfloat16* q;
  QuantPages k;
  const int32_t* ctx_lens;
  int max_ctx, batch, Hq, group, htiles;
  int chunk, splits;
  bool single;                       // the first kernel normalises its rows: one range, a short stride
  float scale_log2;
  float* rows;                       // [batch, Hq, stride]
  int stride;
  float2* ml;                        // [batch * Hq][splits]: (reference, sum of 2^(x - reference))
  unsigned int* status;
};

template <int D, int BITS, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, 5) quant_rows_kernel(const RowsParams p) {
  // 64 tokens a step where a warp's two stages of them take at most 9 KB
  constexpr int NG = D / 32, SB = NG * 2, R = D * BITS / 8, TI = R <= 64 ? 4 : 2, TK = TI * kTok;
  constexpr int K = TK * R, kStage = K + TK * SB, ST = 2;
  __shared__ __align__(128) uint8_t smem[kWarps * ST * kStage];
  __shared__ StreamShared<TI, ST> shared[kWarps];
  __shared__ float2 ml_s[kWarps][kHeads];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, tid = lane & 3;
  let_next_start();
  const int hk = blockIdx.x / p.htiles, ht = blockIdx.x - hk * p.htiles, b = blockIdx.y, split = blockIdx.z;
  const int ctx = quant_ctx(p.ctx_lens, b, p.max_ctx, p.status);
  const int j0 = split * p.chunk, j1 = min(ctx, j0 + p.chunk);
  if (j0 >= j1 && !p.single) return;
  const int h0 = hk * p.group + ht * kHeads;
  const int nh = min(kHeads, p.group - ht * kHeads);
  Stream<ALIGNED, TI, 2, ST> in;
  in.init(&p.k, b, hk, j0 + warp * TK, kWarps * TK, j1, p.status,
          smem_u32(smem) + warp * ST * kStage, &shared[warp]);
  in.template add<0>(p.k.codes, D * BITS / 8);
  in.template add<1>(p.k.scales, SB);
#pragma unroll
  for (int i = 0; i < ST - 1; ++i) in.fill(i);
  uint32_t qf[NG][4];
  float fq[2];
  load_query<D, BITS>(p.q + ((int64_t)b * p.Hq + h0) * D, nh, p.scale_log2, qf, fq);
  // a reference near the maximum, moved when a score exceeds it by more than 64 (sums stay in fp32)
  float ref[2] = {kNoRef, kNoRef}, l[2] = {0.f, 0.f};
  const int t0 = (gid >> 1) + 4 * (gid & 1);
  const int jw = j0 + warp * TK + t0;
  float* row0 = p.rows + ((int64_t)b * p.Hq + h0 + 2 * tid) * p.stride + jw;

  for (int i = 0; i < in.nsteps; ++i) {
    in.fill(i + ST - 1);
    uint32_t st;
    const uint32_t* masks;
    if (!in.take(&st, &masks)) break;
#pragma unroll
    for (int h = 0; h < TI / 2; ++h) {
      const uint32_t mask = masks[h];
      float x[2][4];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        tile_scores<D, BITS>(st + (2 * h + t) * (kTok * R), st + K + (2 * h + t) * (kTok * SB), qf, x[t]);
#pragma unroll
        for (int c = 0; c < 4; ++c) x[t][c] *= fq[c & 1];
      }
      if (mask != 0xffffffffu) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!((mask >> (16 * t + t0)) & 1)) x[t][0] = x[t][1] = -INFINITY;
          if (!((mask >> (16 * t + t0 + 8)) & 1)) x[t][2] = x[t][3] = -INFINITY;
        }
      }
      const float m0 = fmaxf(fmaxf(x[0][0], x[0][2]), fmaxf(x[1][0], x[1][2]));
      const float m1 = fmaxf(fmaxf(x[0][1], x[0][3]), fmaxf(x[1][1], x[1][3]));
      if (__any_sync(0xffffffffu, m0 > ref[0] + 64.f || m1 > ref[1] + 64.f)) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float m = c ? m1 : m0;
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
          if (m > ref[c] + 64.f) {
            l[c] *= ex2(ref[c] - m);
            ref[c] = m;
          }
          __syncwarp();
        }
      }
      const int at = i * kWarps * TK + h * kPair;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          l[c] += ex2(x[t][c] - ref[c]) + ex2(x[t][c + 2] - ref[c]);
          if (2 * tid + c < nh) {
            float* dst = row0 + (int64_t)c * p.stride + at + 16 * t;
            if (jw + at + 16 * t < j1) dst[0] = x[t][c];
            if (jw + at + 16 * t + 8 < j1) dst[8] = x[t][c + 2];
          }
        }
    }
    __syncwarp();
  }
  if (!ALIGNED) cp_async_wait<0>();
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    l[c] += __shfl_xor_sync(0xffffffffu, l[c], 4);
    l[c] += __shfl_xor_sync(0xffffffffu, l[c], 8);
    l[c] += __shfl_xor_sync(0xffffffffu, l[c], 16);
    if (gid == 0) ml_s[warp][2 * tid + c] = make_float2(ref[c], l[c]);
  }
  __syncthreads();
  if (threadIdx.x < nh) {
    float m = kNoRef, z = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, ml_s[w][threadIdx.x].x);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) z += ml_s[w][threadIdx.x].y * ex2(ml_s[w][threadIdx.x].x - m);
    if (!p.single)
      p.ml[((int64_t)b * p.Hq + h0 + threadIdx.x) * p.splits + split] = make_float2(m, z);
    else
      ml_s[0][threadIdx.x] = make_float2(m, z == 0.f ? 0.f : 1.f / z);
  }
  if (!p.single) return;
  __syncthreads();                                           // this CTA wrote all of its rows' scores
  for (int h = warp; h < nh; h += kWarps) {
    float* row = p.rows + ((int64_t)b * p.Hq + h0 + h) * p.stride;
    const float2 mi = ml_s[0][h];
    for (int j = lane; j < p.stride; j += 32)
      row[j] = j < ctx && mi.y != 0.f ? ex2(row[j] - mi.x) * mi.y : 0.f;
  }
}

// The second kernel: a CTA normalises 4096 tokens of a row. Its logits are under way before the ranges'
// (reference, sum) pairs are joined, which every warp does by itself (read after the join, one at a time,
// they made this kernel as long as the first).
constexpr int kNormTokens = 4096, kNormThreads = 256;
__global__ void __launch_bounds__(kNormThreads) quant_rows_norm_kernel(RowsParams p, int parts) {
  constexpr int N = kNormTokens / kNormThreads;
  const int part = blockIdx.x % parts;
  const int64_t r = blockIdx.x / parts;                    // row b * Hq + h
  const int ctx = min(max(p.ctx_lens[r / p.Hq], 0), p.max_ctx);
  const int n = (ctx + p.chunk - 1) / p.chunk;
  const int lane = threadIdx.x & 31, j0 = part * kNormTokens + threadIdx.x;
  float* row = p.rows + r * p.stride;
  after_previous();
  float x[N];
#pragma unroll
  for (int k = 0; k < N; ++k) x[k] = j0 + k * kNormThreads < ctx ? row[j0 + k * kNormThreads] : 0.f;
  float top = 0.f, inv = 0.f;
  if (part * kNormTokens < ctx) {
    const float2* ml = p.ml + r * p.splits;
    float m = kNoRef, z = 0.f;
    for (int s = lane; s < n; s += 32) {
      const float2 v = ml[s];
      const float t = fmaxf(m, v.x);
      z = z * ex2(m - t) + v.y * ex2(v.x - t);
      m = t;
    }
    top = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    z *= ex2(m - top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    if (z != 0.f) inv = 1.f / z;
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int j = j0 + k * kNormThreads;
    if (j < p.stride) row[j] = j < ctx && inv != 0.f ? ex2(x[k] - top) * inv : 0.f;
  }
}

// Ranges: twice as many CTAs as the SMs hold at five each (sixteen ragged sequences: 20.5 us, 22.6 with
// half as many, while four equal ones take the same), 256 to 2048 tokens; one range up to 512 tokens, which
// saves the second kernel.
void rows_split(int units, int max_ctx, int* chunk, int* splits) {
  const int64_t total = (int64_t)units * max_ctx;
  int64_t c = (total + kSms * 10 - 1) / (kSms * 10);
  c = (c + 255) / 256 * 256;
  *chunk = max_ctx <= 512 ? 512 : (int)std::min<int64_t>(2048, std::max<int64_t>(256, c));
  while ((max_ctx - 1) / *chunk >= 65535) *chunk *= 2;      // the grid's third dimension
  *splits = std::max(1, (max_ctx + *chunk - 1) / *chunk);
}

template <int D>
int launch_d(const RowsParams& p, int bits, cudaStream_t st) {
  const bool al = p.k.page_size % kTok == 0;
  const dim3 grid(p.k.H * p.htiles, p.batch, p.splits);
  if (bits == 4) {
    if (al) quant_rows_kernel<D, 4, true><<<grid, kThreads, 0, st>>>(p);
    else quant_rows_kernel<D, 4, false><<<grid, kThreads, 0, st>>>(p);
  } else {
    if (al) quant_rows_kernel<D, 8, true><<<grid, kThreads, 0, st>>>(p);
    else quant_rows_kernel<D, 8, false><<<grid, kThreads, 0, st>>>(p);
  }
  IAMAP_LAUNCH_CHECK("quant_rows_kernel");
  if (p.single) return IAMAP_OK;
  const int parts = (p.stride + kNormTokens - 1) / kNormTokens;
  return launch_next("quant_rows_norm_kernel", quant_rows_norm_kernel,
                     dim3((unsigned int)((int64_t)p.batch * p.Hq * parts)), kNormThreads, 0, st, p, parts);
}

}  // namespace
}  // namespace iamap

using namespace iamap;

extern "C" size_t iamap_sender_rows_quant_workspace_bytes(int batch, int H_s, int max_ctx) {
  if (batch < 1 || H_s < 1 || max_ctx < 0) return 0;
  if (batch > 65535 || (int64_t)batch * H_s > 0x7fffff || max_ctx > kMaxCtx) return 0;   // refused by the call
  // the most that any grouping of the H_s heads needs
  size_t most = 256;
  for (int group = 1; group <= H_s; ++group) {
    if (H_s % group != 0) continue;
    int chunk, splits;
    rows_split(batch * (H_s / group) * ((group + kHeads - 1) / kHeads), max_ctx, &chunk, &splits);
    most = std::max(most, sizeof(float2) * (size_t)batch * H_s * splits);
  }
  return most;
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
  RowsParams p{};
  p.group = H_s / H_k;
  p.htiles = (p.group + kHeads - 1) / kHeads;
  const int64_t units = (int64_t)batch * H_k * p.htiles;
  if (batch > 65535 || (int64_t)batch * H_s > 0x7fffff ||
      (int64_t)batch * H_s * ((ctx_stride + (int64_t)kNormTokens - 1) / kNormTokens) > 0x7fffffff)
    return set_error(IAMAP_ERR_UNSUPPORTED, "batch above 65535, or batch times heads times ctx_stride too large");
  rows_split((int)units, max_ctx, &p.chunk, &p.splits);
  p.single = p.splits == 1 && ctx_stride <= kNormTokens;
  const size_t need = sizeof(float2) * (size_t)batch * H_s * p.splits;
  if (!ws || ws_bytes < need)
    return set_error(IAMAP_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws_bytes);
  if ((reinterpret_cast<uintptr_t>(ws) & 15u) != 0)
    return set_error(IAMAP_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  DeviceContext* ctx = device_context();
  if (!ctx) return IAMAP_ERR_CUDA;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = QuantPages{static_cast<const uint8_t*>(k_codes), static_cast<const __half*>(k_scales),
                   num_pages, page_table, max_pages, page_size, H_k};
  p.ctx_lens = ctx_lens;
  p.max_ctx = max_ctx;
  p.batch = batch;
  p.Hq = H_s;
  p.scale_log2 = kLog2e / sqrtf((float)d);
  p.rows = p_rows;
  p.stride = ctx_stride;
  p.ml = static_cast<float2*>(ws);
  p.status = ctx->status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return d == 64 ? launch_d<64>(p, bits, st) : launch_d<128>(p, bits, st);
}
