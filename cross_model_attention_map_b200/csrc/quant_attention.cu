// iamap_attention_paged_quant: decode attention over a quantised paged cache.
//
//   out[b, h] = sum_j p_j v^[b, j],  p = softmax_j(q[b, h] . k^[b, j] / sqrt(d)),  j < ctx[b]
//
// Bound by the cache bytes (72 + 72 a token and head of 128 in 4 bits). One CTA takes a range of tokens
// of one (sequence, key head) and up to eight of the query heads that share it; each of its four warps
// streams every fourth 16-token tile through a ring of asynchronous copies of its own, so no barrier
// stands in the loop, and keeps scores, softmax and output in registers:
//
//   S^T = K^ q^T (codes; group scales in fp32), x = S / sqrt(d) in base 2, p = 2^(x - ref),
//   O^T += V^T (p s) with s the token's scale of the group.
//
// ref is a reference near the running maximum, not the maximum itself: it moves only when a score
// exceeds it by more than 15 (then to 8 below the new maximum), which is rare after the first tiles,
// so most tiles need no reduction across lanes and no rescaling. p and p s are fp16 (11 bits; the
// output has 8): between 2^-24 and 2^15, with at least one p of the warp's tokens near 2^8 or above.
// A product p s beyond 2^15 (scales above 2^7 or so) raises ref by 16. l = sum p is fp32.
//
// Ranges of one sequence are joined by a second kernel; a sequence that fits in one range is written by
// the first.
#include <algorithm>

#include "internal.h"
#include "quant_tile.cuh"

namespace iamap {
namespace {

using namespace qt;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 4;
constexpr int kHeads = 8;            // query heads a CTA
constexpr float kNoRef = -3e38f;

struct AttnParams {
  const __nv_bfloat16* q;
  QuantPages k;                      // pages, table and sizes are those of the values too
  const uint8_t* v_codes;
  const __half* v_scales;
  const int32_t* ctx_lens;
  int max_ctx, batch, Hq, group, htiles;
  int hpu;                           // partial rows a unit: min(group, kHeads)
  int chunk;                         // tokens a range
  int splits;                        // ranges of max_ctx tokens
  float scale_log2;
  __nv_bfloat16* out;
  float* lse;
  float* acc;                        // [unit][splits][hpu][D]
  float2* ml;                        // [unit][splits][hpu]: (ref, l)
  unsigned int* status;
};

template <int D, int KB, int VB>
struct Ring {
  static constexpr int K = kTok * D * KB / 8, V = kTok * D * VB / 8, S = kTok * (D / 32) * 2;
  static constexpr int kStage = K + V + 2 * S;
  static constexpr int kWarp = kStages * kStage;
  static constexpr int kMerge = kWarps * kHeads * D * 4;
  static constexpr int kBytes = kWarps * kWarp > kMerge ? kWarps * kWarp : kMerge;
};

template <int D, int KB, int VB, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, 4) quant_attention_kernel(const AttnParams p) {
  using RB = Ring<D, KB, VB>;
  constexpr int NG = D / 32;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t masks[kWarps][kStages];
  __shared__ float2 ml_s[kWarps][kHeads];

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, tid = lane & 3;
  int u = blockIdx.x;
  const int ht = u % p.htiles;
  u /= p.htiles;
  const int hk = u % p.k.H;
  u /= p.k.H;
  const int b = u % p.batch, split = u / p.batch;
  const int ctx = quant_ctx(p.ctx_lens, b, p.max_ctx, p.status);
  const int nsplit = max(1, (ctx + p.chunk - 1) / p.chunk);
  if (split >= nsplit) return;
  const int j0 = split * p.chunk, j1 = min(ctx, j0 + p.chunk);
  const int h0 = hk * p.group + ht * kHeads;               // first query head of the CTA
  const int nh = min(kHeads, p.group - ht * kHeads);

  // this warp's tiles: tokens j0 + 16 (warp + 4 i)
  const int ntiles = max(0, (j1 - j0 + kTok - 1) / kTok - warp + kWarps - 1) / kWarps;
  const uint32_t ring = smem_u32(smem) + warp * RB::kWarp;
  TileRows<ALIGNED> src;
  src.init(&p.k, b, hk, j0 + warp * kTok, kWarps * kTok, j1, p.status);
  const uint8_t* kc = codes_base<D, KB, ALIGNED>(p.k.codes);
  const uint8_t* vc = codes_base<D, VB, ALIGNED>(p.v_codes);
  const __half* sc_pool = lane < 16 ? p.k.scales : p.v_scales;   // lanes 0..15 the keys' scales
  const uint32_t sc_dst = lane < 16 ? RB::K : RB::K + RB::S + RB::V;
  auto issue = [&](int i) {
    if (i < ntiles) {
      const int s = i % kStages;
      const uint32_t dst = ring + s * RB::kStage;
      const Tile tl = src.tile(i);
      load_codes<D, KB, ALIGNED>(dst, kc, tl);
      load_codes<D, VB, ALIGNED>(dst + RB::K + RB::S, vc, tl);
      load_scales<D, ALIGNED>(dst + sc_dst, sc_pool, tl, lane & 15);
      if (lane == 0) masks[warp][s] = tl.mask;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i);

  uint32_t qf[NG][4];
  float fq[2];
  load_query<D, KB>(p.q + ((int64_t)b * p.Hq + h0) * D, nh, p.scale_log2, qf, fq);

  float o[2 * NG][4];
#pragma unroll
  for (int i = 0; i < 2 * NG; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) o[i][c] = 0.f;
  float ref[2] = {kNoRef, kNoRef}, l[2] = {0.f, 0.f};
  const int t0 = (gid >> 1) + 4 * (gid & 1);               // tokens of this lane's score rows: t0, t0 + 8

  for (int i = 0; i < ntiles; ++i) {
    cp_async_wait<kStages - 2>();
    __syncwarp();
    const uint32_t st = ring + (i % kStages) * RB::kStage;
    const uint32_t mask = masks[warp][i % kStages];
    float x[4];
    tile_scores<D, KB>(st, st + RB::K, qf, x);
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] *= fq[c & 1];
    if (mask != 0xffffu) {
      if (!((mask >> t0) & 1)) x[0] = x[1] = -INFINITY;
      if (!((mask >> (t0 + 8)) & 1)) x[2] = x[3] = -INFINITY;
    }
    if (__any_sync(0xffffffffu, fmaxf(x[0], x[2]) > ref[0] + 15.f || fmaxf(x[1], x[3]) > ref[1] + 15.f)) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float m = fmaxf(x[c], x[c + 2]);
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
        if (m > ref[c] + 15.f) {
          const float f = ex2(ref[c] - (m - 8.f));
          ref[c] = m - 8.f;
          l[c] *= f;
#pragma unroll
          for (int k = 0; k < 2 * NG; ++k) o[k][c] *= f, o[k][c + 2] *= f;
        }
      }
    }
    float e[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) e[c] = ex2(x[c] - ref[c & 1]);

    // value operands and the weights p s
    const uint32_t vs = st + RB::K + RB::S;
    ValueTile<D, VB> vt;
    vt.load(vs);
    uint2 sc[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) sc[k] = lds_scales<NG>(vs + RB::V + (tid + 4 * k) * (2 * NG));
    uint32_t pb[NG][2];
    auto weights = [&]() {
      const uint32_t b0 = movmatrix_trans(pack_f16(e[0], e[1]));
      const uint32_t b1 = movmatrix_trans(pack_f16(e[2], e[3]));
      __half2 most = __float2half2_rn(0.f);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        pb[g][0] = hmul2(b0, scale_pair(sc, g));
        pb[g][1] = hmul2(b1, scale_pair(sc + 2, g));
        most = __hmax2(most, __hmax2(*reinterpret_cast<__half2*>(&pb[g][0]),
                                     *reinterpret_cast<__half2*>(&pb[g][1])));
      }
      return __hmax(__low2half(most), __high2half(most));
    };
    if (__any_sync(0xffffffffu, __hgt(weights(), __float2half(32768.f)))) {
      constexpr float kDown = 1.f / 65536.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) e[c] *= kDown;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        ref[c] += ref[c] > kNoRef ? 16.f : 0.f;
        l[c] *= kDown;
      }
#pragma unroll
      for (int k = 0; k < 2 * NG; ++k)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[k][c] *= kDown;
      weights();
    }
    l[0] += e[0] + e[2];
    l[1] += e[1] + e[3];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      uint32_t r[4], t[4];
      vt.group(g, r, t);
      mma_f16(o[2 * g], r[0], r[1], t[0], t[1], pb[g][0], pb[g][1]);
      mma_f16(o[2 * g + 1], r[2], r[3], t[2], t[3], pb[g][0], pb[g][1]);
    }
    __syncwarp();
    issue(i + kStages - 1);
  }
  cp_async_wait<0>();

  // join the four warps
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    l[c] += __shfl_xor_sync(0xffffffffu, l[c], 4);
    l[c] += __shfl_xor_sync(0xffffffffu, l[c], 8);
    l[c] += __shfl_xor_sync(0xffffffffu, l[c], 16);
    if (gid == 0) ml_s[warp][2 * tid + c] = make_float2(ref[c], l[c]);
  }
  __syncthreads();
  float* o_s = reinterpret_cast<float*>(smem);             // [warp][head][D]
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int h = 2 * tid + c;
    float m = kNoRef;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, ml_s[w][h].x);
    const float f = ex2(ref[c] - m);
    float* dst = o_s + (warp * kHeads + h) * D + 4 * gid;
#pragma unroll
    for (int g = 0; g < NG; ++g)
      *reinterpret_cast<float4*>(dst + 32 * g) =
          make_float4(o[2 * g][c] * f, o[2 * g][c + 2] * f, o[2 * g + 1][c] * f, o[2 * g + 1][c + 2] * f);
  }
  __syncthreads();
  const int64_t unit = ((int64_t)b * p.k.H + hk) * p.htiles + ht;
  for (int at = threadIdx.x * 4; at < nh * D; at += kThreads * 4) {
    const int h = at / D;
    float m = kNoRef, z = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, ml_s[w][h].x);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) z += ml_s[w][h].y * ex2(ml_s[w][h].x - m);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 t = *reinterpret_cast<const float4*>(o_s + w * kHeads * D + at);
      a.x += t.x, a.y += t.y, a.z += t.z, a.w += t.w;
    }
    if (nsplit == 1) {
      const float inv = z == 0.f ? 0.f : 1.f / z;
      const int64_t row = (int64_t)b * p.Hq + h0 + h;
      *reinterpret_cast<uint2*>(p.out + row * D + (at - h * D)) =
          make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
      if (p.lse && at == h * D) p.lse[row] = z == 0.f ? -INFINITY : (m + log2f(z)) * kLn2;
    } else {
      const int64_t part = (unit * p.splits + split) * p.hpu + h;
      *reinterpret_cast<float4*>(p.acc + part * D + (at - h * D)) = a;
      if (at == h * D) p.ml[part] = make_float2(m, z);
    }
  }
}

// Joins the ranges of one query head, in their order.
template <int D>
__global__ void __launch_bounds__(D) quant_attention_join_kernel(const AttnParams p) {
  const int h = blockIdx.x % p.Hq, b = blockIdx.x / p.Hq;
  const int ctx = min(max(p.ctx_lens[b], 0), p.max_ctx);
  const int nsplit = (ctx + p.chunk - 1) / p.chunk;
  if (nsplit <= 1) return;
  const int hk = h / p.group, hg = h - hk * p.group;
  const int64_t unit = ((int64_t)b * p.k.H + hk) * p.htiles + hg / kHeads;
  const int64_t first = unit * p.splits * p.hpu + hg % kHeads;
  __shared__ float red[D / 32];
  float m = kNoRef;
  for (int s = threadIdx.x; s < nsplit; s += D) m = fmaxf(m, p.ml[first + (int64_t)s * p.hpu].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < D / 32; ++w) m = fmaxf(m, red[w]);
  float z = 0.f, a = 0.f;
#pragma unroll 4
  for (int s = 0; s < nsplit; ++s) {
    const int64_t part = first + (int64_t)s * p.hpu;
    const float2 ml = p.ml[part];
    const float f = ex2(ml.x - m);
    z = fmaf(ml.y, f, z);
    a = fmaf(p.acc[part * D + threadIdx.x], f, a);
  }
  const int64_t row = (int64_t)b * p.Hq + h;
  p.out[row * D + threadIdx.x] = __float2bfloat16(z == 0.f ? 0.f : a / z);
  if (p.lse && threadIdx.x == 0) p.lse[row] = z == 0.f ? -INFINITY : (m + log2f(z)) * kLn2;
}

// Ranges: enough CTAs to fill the device's 148 SMs four times over, at least 64 tokens (a tile a warp)
// and at most 2048 each, so that one long sequence in a ragged batch is still spread.
void attention_split(int batch, int units, int max_ctx, int* chunk, int* splits) {
  const int64_t total = (int64_t)units * max_ctx;
  int64_t c = (total + 148 * 4 - 1) / (148 * 4);
  c = (c + 63) / 64 * 64;
  *chunk = (int)std::min<int64_t>(2048, std::max<int64_t>(64, c));
  *splits = std::max(1, (max_ctx + *chunk - 1) / *chunk);
}

size_t attention_bytes(int64_t units, int splits, int hpu, int D, size_t* ml_at) {
  const size_t a = sizeof(float) * (size_t)units * splits * hpu * D;
  if (ml_at) *ml_at = a;
  return a + sizeof(float2) * (size_t)units * splits * hpu;
}

template <int D, int KB, int VB, bool ALIGNED>
int launch(const AttnParams& p, unsigned int blocks, cudaStream_t st) {
  constexpr int bytes = Ring<D, KB, VB>::kBytes;
  if (bytes > 48 * 1024)
    IAMAP_CUDA_CHECK(cudaFuncSetAttribute(quant_attention_kernel<D, KB, VB, ALIGNED>,
                                          cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
  quant_attention_kernel<D, KB, VB, ALIGNED><<<blocks, kThreads, bytes, st>>>(p);
  IAMAP_LAUNCH_CHECK("quant_attention_kernel");
  if (p.splits > 1) {
    quant_attention_join_kernel<D><<<p.batch * p.Hq, D, 0, st>>>(p);
    IAMAP_LAUNCH_CHECK("quant_attention_join_kernel");
  }
  return IAMAP_OK;
}
template <int D, int KB, int VB>
int launch_a(const AttnParams& p, unsigned int blocks, cudaStream_t st) {
  return p.k.page_size % kTok == 0 ? launch<D, KB, VB, true>(p, blocks, st)
                                   : launch<D, KB, VB, false>(p, blocks, st);
}
template <int D>
int launch_d(const AttnParams& p, int kb, int vb, unsigned int blocks, cudaStream_t st) {
  if (kb == 4) return vb == 4 ? launch_a<D, 4, 4>(p, blocks, st) : launch_a<D, 4, 8>(p, blocks, st);
  return vb == 4 ? launch_a<D, 8, 4>(p, blocks, st) : launch_a<D, 8, 8>(p, blocks, st);
}

}  // namespace
}  // namespace iamap

using namespace iamap;

extern "C" size_t iamap_attention_paged_quant_workspace_bytes(int batch, int H_q, int d,
                                                              int max_ctx) {
  if (batch < 1 || H_q < 1 || d < 1 || max_ctx < 0) return 0;
  // the most that any grouping of the H_q heads needs: a unit is up to eight of them
  size_t most = 256;
  for (int group = 1; group <= H_q; ++group) {
    if (H_q % group != 0) continue;
    int chunk, splits;
    const int units = batch * (H_q / group) * ((group + kHeads - 1) / kHeads);
    attention_split(batch, units, max_ctx, &chunk, &splits);
    if (splits > 1) most = std::max(most, attention_bytes(units, splits, std::min(group, kHeads), d, nullptr));
  }
  return most;
}

extern "C" int iamap_attention_paged_quant(const void* q, const void* k_codes, const void* k_scales,
                                           int k_bits, const void* v_codes, const void* v_scales,
                                           int v_bits, int64_t num_pages, const int32_t* page_table,
                                           int max_pages, int page_size, const int32_t* ctx_lens,
                                           int max_ctx, int batch, int H_q, int H_kv, int d,
                                           void* out, float* lse, void* ws, size_t ws_bytes,
                                           void* stream) {
  clear_error();
  int rc = check_quant_pages(k_codes, k_scales, num_pages, page_table, max_pages, page_size, H_kv, d,
                             k_bits);
  if (rc) return rc;
  rc = check_quant_pages(v_codes, v_scales, num_pages, page_table, max_pages, page_size, H_kv, d,
                         v_bits);
  if (rc) return rc;
  rc = check_quant_batch(ctx_lens, max_ctx, batch, max_pages, page_size);
  if (rc) return rc;
  if (H_q < 1 || H_q % H_kv != 0)
    return set_error(IAMAP_ERR_INVALID_ARG, "H_kv=%d must divide H_q=%d", H_kv, H_q);
  if (!q || !out) return set_error(IAMAP_ERR_INVALID_ARG, "null pointer");
  if (((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15u) != 0)
    return set_error(IAMAP_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
  AttnParams p{};
  p.group = H_q / H_kv;
  p.htiles = (p.group + kHeads - 1) / kHeads;
  p.hpu = std::min(p.group, kHeads);
  const int64_t units = (int64_t)batch * H_kv * p.htiles;
  if (units > 0x7fffff || (int64_t)batch * H_q > 0x7fffffff)
    return set_error(IAMAP_ERR_UNSUPPORTED, "batch times heads is too large");
  attention_split(batch, (int)units, max_ctx, &p.chunk, &p.splits);
  if (units * p.splits > 0x7fffffff)
    return set_error(IAMAP_ERR_UNSUPPORTED, "batch times heads times max_ctx is too large");
  size_t ml_at = 0;
  const size_t need = p.splits > 1 ? attention_bytes(units, p.splits, p.hpu, d, &ml_at) : 1;
  if (!ws || ws_bytes < need)
    return set_error(IAMAP_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws_bytes);
  if ((reinterpret_cast<uintptr_t>(ws) & 15u) != 0)
    return set_error(IAMAP_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  DeviceContext* ctx = device_context();
  if (!ctx) return IAMAP_ERR_CUDA;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = QuantPages{static_cast<const uint8_t*>(k_codes), static_cast<const __half*>(k_scales),
                   num_pages, page_table, max_pages, page_size, H_kv};
  p.v_codes = static_cast<const uint8_t*>(v_codes);
  p.v_scales = static_cast<const __half*>(v_scales);
  p.ctx_lens = ctx_lens;
  p.max_ctx = max_ctx;
  p.batch = batch;
  p.Hq = H_q;
  p.scale_log2 = kLog2e / sqrtf((float)d);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.acc = static_cast<float*>(ws);
  p.ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + ml_at);
  p.status = ctx->status;
  const unsigned int blocks = (unsigned int)(units * p.splits);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return d == 64 ? launch_d<64>(p, k_bits, v_bits, blocks, st)
                 : launch_d<128>(p, k_bits, v_bits, blocks, st);
}
