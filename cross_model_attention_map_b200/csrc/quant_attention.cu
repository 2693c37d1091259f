// iamap_attention_paged_quant: decode attention over a quantised paged cache.
//
//   out[b, h] = sum_j p_j v^[b, j],  p = softmax_j(q[b, h] . k^[b, j] / sqrt(d)),  j < ctx[b]
//
// Bound by the cache bytes (72 + 72 a token and head of 128 in 4 bits). One CTA takes a range of tokens
// of one (sequence, key head) and up to eight of the query heads that share it; each of its four warps
// streams every fourth step of 32 tokens through a ring of copies of its own and keeps scores, softmax
// and output in registers:
//
//   S^T = K^ q^T (codes; group scales in fp32), x = S / sqrt(d) in base 2, p = 2^(x - ref),
//   O^T += V^T (p s) with s the token's scale of the group.
//
// p and p s are fp16 (11 bits; the output has 8, and l = sum p is fp32), so their smallest step, 2^-24, has to be
// small beside the probabilities that count. ref is an integer near the maximum of the step at hand: it moves
// to 10 below that maximum, and only when the largest p leaves [2^2, 2^14], which is rare after the first
// step, so most steps need no rescaling. It falls too: behind a token that takes almost all of the
// weight, with values near zero, the others make up the output, and with a ref that only rises they are
// rounded away (19 % off beside 0.9999; 164 us where this takes 165).
// A group's scales are taken times a power of two where they are 2 and more or small (ScalePowers), so p s
// stays under 2^15.
//
// Ranges of one sequence are joined by a second kernel; a sequence that fits in one range is written by
// the first. 48 sequences of 4587 to 16384 tokens, 64 heads on 8 of 128, all in 4 bits: 165 us a pass, 3.5
// TB/s of the cache; one of 131071, keys in 8 bits and values in 4: 51 us, 4.3 TB/s. What bounds it is turning
// codes into fp16 operands: 63 % of the issue slots while an SM works and 58 % of the integer pipe, which the
// matrix instructions' issue takes from as well, with four warps a scheduler.
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
// Base-2 logarithms of the largest p of a step: where a move of ref puts it, and the limits that bring one on.
constexpr float kSet = 10.f, kMost = 14.f, kLeast = 2.f;
constexpr float kFall = 48.f;        // ref stays this near its highest, so that rescaled sums fit fp32

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
  // 32 tokens a step and two stages a warp fit four CTAs an SM (three where both are 8 bits of 128). With
  // three CTAs and 64 tokens the batch of 48 took as long, and one sequence of 131071 tokens 59 us, not 49.
  static constexpr int kTiles = 2, kTokens = kTiles * kTok, kStages = 2;
  static constexpr int K = kTokens * D * KB / 8, V = kTokens * D * VB / 8, S = kTokens * (D / 32) * 2;
  static constexpr int kStage = K + S + V + S;           // keys' codes and scales, values'
  static constexpr int kWarp = kStages * kStage;
  static constexpr int kMerge = kWarps * kHeads * D * 4;
  static constexpr int kBytes = kWarps * kWarp > kMerge ? kWarps * kWarp : kMerge;
};

template <int D, int KB, int VB, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, 4) quant_attention_kernel(const AttnParams p) {
  using RB = Ring<D, KB, VB>;
  constexpr int NG = D / 32, ST = RB::kStages, SB = NG * 2, TK = RB::kTokens;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ StreamShared<RB::kTiles, ST> shared[kWarps];
  __shared__ float2 ml_s[kWarps][kHeads];

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, tid = lane & 3;
  let_next_start();
  const int hk = blockIdx.x / p.htiles, ht = blockIdx.x - hk * p.htiles, b = blockIdx.y, split = blockIdx.z;
  const int ctx = quant_ctx(p.ctx_lens, b, p.max_ctx, p.status);
  const int j0 = split * p.chunk, j1 = min(ctx, j0 + p.chunk);
  if (j0 >= j1 && split > 0) return;
  const int h0 = hk * p.group + ht * kHeads;               // first query head of the CTA
  const int nh = min(kHeads, p.group - ht * kHeads);
  const bool single = ctx <= p.chunk;                      // the only range of its sequence

  Stream<ALIGNED, RB::kTiles, 4, ST> in;
  in.init(&p.k, b, hk, j0 + warp * TK, kWarps * TK, j1, p.status,
          smem_u32(smem) + warp * RB::kWarp, &shared[warp]);
  in.template add<0>(p.k.codes, D * KB / 8);
  in.template add<1>(p.k.scales, SB);
  in.template add<2>(p.v_codes, D * VB / 8);
  in.template add<3>(p.v_scales, SB);
#pragma unroll
  for (int i = 0; i < ST - 1; ++i) in.fill(i);

  uint32_t qf[NG][4];
  float fq[2];
  load_query<D, KB>(p.q + ((int64_t)b * p.Hq + h0) * D, nh, p.scale_log2, qf, fq);

  float o[2 * NG][4];
#pragma unroll
  for (int i = 0; i < 2 * NG; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) o[i][c] = 0.f;
  float ref[2] = {kNoRef, kNoRef}, highest[2] = {kNoRef, kNoRef}, l[2] = {0.f, 0.f};
  ScalePowers<NG, false> pw;
  pw.init();
  const int t0 = (gid >> 1) + 4 * (gid & 1);               // tokens of a tile in this lane's score rows: t0, t0 + 8

  for (int i = 0; i < in.nsteps; ++i) {
    in.fill(i + ST - 1);
    uint32_t st;
    const uint32_t* masks;
    if (!in.take(&st, &masks)) break;
    const uint32_t vs = st + RB::K + RB::S;
    const uint32_t mask = masks[0];
    // a scale among the step's values that its group's power does not serve
    const uint4 all = lds128(vs + RB::V + lane * 16 % RB::S);
    const uint32_t served = pw.served(all.x, 0) & pw.served(all.y, 1) & pw.served(all.z, 0) & pw.served(all.w, 1);
    if (__any_sync(0xffffffffu, (served & 0x80008000u) != 0x80008000u)) {
      uint32_t m[NG / 2] = {};
      const uint32_t q[4] = {all.x, all.y, all.z, all.w};
#pragma unroll
      for (int w = 0; w < 4; ++w)
        if (mask >> (lane * 16 % RB::S + 4 * w) / SB & 1) m[w % (NG / 2)] = pw.larger(m[w % (NG / 2)], q[w]);
      float f[NG];
      pw.raise(m, f);
#pragma unroll
      for (int k = 0; k < 2 * NG; ++k)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[k][c] *= f[k / 2];
    }
    // scores of two tiles, to be multiplied by fq: x[t][c], c = 0, 1 row gid, 2, 3 row gid + 8
    float x[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
      tile_scores<D, KB>(st + t * (kTok * D * KB / 8), st + RB::K + t * (kTok * SB), qf, x[t]);
    uint2 sc[2][4];                                      // the values' scales of tokens tid + 4 k
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        sc[t][k] = lds_scales<NG>(vs + RB::V + (16 * t + tid + 4 * k) * SB);
    if (mask != 0xffffffffu) {
      // tokens that do not exist: no probability, and no scale (memory behind them may hold anything)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (!((mask >> (16 * t + t0)) & 1)) x[t][0] = x[t][1] = -INFINITY;
        if (!((mask >> (16 * t + t0 + 8)) & 1)) x[t][2] = x[t][3] = -INFINITY;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (!((mask >> (16 * t + tid + 4 * k)) & 1)) sc[t][k] = make_uint2(0, 0);
      }
    }
    if (pw.any()) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          sc[t][k].x = hmul2(sc[t][k].x, pw.half(0) | pw.half(1) << 16);
          if (NG == 4) sc[t][k].y = hmul2(sc[t][k].y, pw.half(NG - 2) | pw.half(NG - 1) << 16);
        }
    }
    const float m0 = fmaxf(fmaxf(x[0][0], x[0][2]), fmaxf(x[1][0], x[1][2]));
    const float m1 = fmaxf(fmaxf(x[0][1], x[0][3]), fmaxf(x[1][1], x[1][3]));
    // a lane's own four tokens decide most steps: their largest p lies between the limits in every lane
    const float y0 = fmaf(m0, fq[0], -ref[0]), y1 = fmaf(m1, fq[1], -ref[1]);
    if (!__all_sync(0xffffffffu, y0 >= kLeast && y0 <= kMost && y1 >= kLeast && y1 <= kMost)) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float m = c ? m1 : m0;
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
        const float y = fmaf(m, fq[c], -ref[c]);
        if (m > -INFINITY && !(y >= kLeast && y <= kMost)) {
          const float r = fmaxf(floorf(m * fq[c]) - kSet, highest[c] - kFall), f = ex2(ref[c] - r);
          ref[c] = r;
          highest[c] = fmaxf(highest[c], r);
          l[c] *= f;
#pragma unroll
          for (int k = 0; k < 2 * NG; ++k) o[k][c] *= f, o[k][c + 2] *= f;
        }
        __syncwarp();
      }
    }
    // probabilities as the operand of the second product: pb[t][0] tokens (tid, tid + 4), [1] + 8
    uint32_t pb[2][2];
    float e[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int c = 0; c < 4; ++c) e[t][c] = ex2(fmaf(x[t][c], fq[c & 1], -ref[c & 1]));
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      pb[t][0] = movmatrix_trans(pack_f16(e[t][0], e[t][1]));
      pb[t][1] = movmatrix_trans(pack_f16(e[t][2], e[t][3]));
    }
    l[0] += (e[0][0] + e[0][2]) + (e[1][0] + e[1][2]);
    l[1] += (e[0][1] + e[0][3]) + (e[1][1] + e[1][3]);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      ValueTile<D, VB> vt;
      vt.load(vs + t * (kTok * D * VB / 8));
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const uint32_t w0 = hmul2(pb[t][0], scale_pair(sc[t], g));
        const uint32_t w1 = hmul2(pb[t][1], scale_pair(sc[t] + 2, g));
        uint32_t r[4], q[4];
        vt.group(g, r, q);
        mma_f16(o[2 * g], r[0], r[1], q[0], q[1], w0, w1);
        mma_f16(o[2 * g + 1], r[2], r[3], q[2], q[3], w0, w1);
      }
    }
    __syncwarp();
  }
  if (!ALIGNED) cp_async_wait<0>();

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
    for (int g = 0; g < NG; ++g) {
      const float fg = f * pow2i(pw.e(g));
      *reinterpret_cast<float4*>(dst + 32 * g) =
          make_float4(o[2 * g][c] * fg, o[2 * g][c + 2] * fg, o[2 * g + 1][c] * fg, o[2 * g + 1][c + 2] * fg);
    }
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
    if (single) {
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

// Joins the ranges of one query head: a warp (half of one for D = 64) takes a range in turn and keeps its own
// running reference, sum and output, then these are added in a fixed order. T = 256 threads, or 1024 where
// there are more than 32 ranges. (One thread an element over all ranges took 21 us for one sequence of
// 131071 tokens, mostly latency; the largest reference looked up first, and 256 threads for its 74 ranges, 9.)
template <int D, int T>
__global__ void __launch_bounds__(T) quant_attention_join_kernel(AttnParams p) {
  constexpr int L = D / 4, G = T / L;                        // lanes a range, ranges at a time
  const int h = blockIdx.x % p.Hq, b = blockIdx.x / p.Hq;
  const int ctx = min(max(p.ctx_lens[b], 0), p.max_ctx);
  const int nsplit = (ctx + p.chunk - 1) / p.chunk;
  const int hk = h / p.group, hg = h - hk * p.group;
  const int64_t unit = ((int64_t)b * p.k.H + hk) * p.htiles + hg / kHeads;
  const int64_t first = unit * p.splits * p.hpu + hg % kHeads;
  __shared__ float2 mz_s[G];
  __shared__ __align__(16) float a_s[G][D];
  after_previous();
  if (nsplit <= 1) return;
  const int g = threadIdx.x / L, e = threadIdx.x % L * 4;
  float m = kNoRef, z = 0.f;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = g; s < nsplit; s += G) {
    const int64_t part = first + (int64_t)s * p.hpu;
    const float2 ml = p.ml[part];
    const float4 x = *reinterpret_cast<const float4*>(p.acc + part * D + e);
    const float top = fmaxf(m, ml.x), old = ex2(m - top), f = ex2(ml.x - top);
    m = top;
    z = fmaf(ml.y, f, z * old);
    a.x = fmaf(x.x, f, a.x * old), a.y = fmaf(x.y, f, a.y * old);
    a.z = fmaf(x.z, f, a.z * old), a.w = fmaf(x.w, f, a.w * old);
  }
  *reinterpret_cast<float4*>(&a_s[g][e]) = a;
  if (e == 0) mz_s[g] = make_float2(m, z);
  __syncthreads();
  if (threadIdx.x >= D) return;
  m = kNoRef;
#pragma unroll 8
  for (int k = 0; k < G; ++k) m = fmaxf(m, mz_s[k].x);
  float sum = 0.f;
  z = 0.f;
#pragma unroll 8
  for (int k = 0; k < G; ++k) {
    const float f = ex2(mz_s[k].x - m);
    sum = fmaf(a_s[k][threadIdx.x], f, sum), z = fmaf(mz_s[k].y, f, z);
  }
  const int64_t row = (int64_t)b * p.Hq + h;
  p.out[row * D + threadIdx.x] = __float2bfloat16(z == 0.f ? 0.f : sum / z);
  if (p.lse && threadIdx.x == 0) p.lse[row] = z == 0.f ? -INFINITY : (m + log2f(z)) * kLn2;
}

// Ranges: enough CTAs to fill the device's SMs four times over, at least 256 tokens and at most 2048
// each, so that one long sequence in a ragged batch is still spread; one range up to 512 tokens, which
// saves the second kernel.
void attention_split(int batch, int units, int max_ctx, int* chunk, int* splits) {
  const int64_t total = (int64_t)units * max_ctx;
  int64_t c = (total + kSms * 4 - 1) / (kSms * 4);
  c = (c + 255) / 256 * 256;
  *chunk = max_ctx <= 512 ? 512 : (int)std::min<int64_t>(2048, std::max<int64_t>(256, c));
  while ((max_ctx - 1) / *chunk >= 65535) *chunk *= 2;      // the grid's third dimension
  *splits = std::max(1, (max_ctx + *chunk - 1) / *chunk);
}

size_t attention_bytes(int64_t units, int splits, int hpu, int D, size_t* ml_at) {
  const size_t a = sizeof(float) * (size_t)units * splits * hpu * D;
  if (ml_at) *ml_at = a;
  return a + sizeof(float2) * (size_t)units * splits * hpu;
}

template <int D, int KB, int VB, bool ALIGNED>
int launch(const AttnParams& p, cudaStream_t st) {
  constexpr int bytes = Ring<D, KB, VB>::kBytes;
  if (bytes > 48 * 1024)
    IAMAP_CUDA_CHECK(cudaFuncSetAttribute(quant_attention_kernel<D, KB, VB, ALIGNED>,
                                          cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
  const dim3 grid(p.k.H * p.htiles, p.batch, p.splits);
  quant_attention_kernel<D, KB, VB, ALIGNED><<<grid, kThreads, bytes, st>>>(p);
  IAMAP_LAUNCH_CHECK("quant_attention_kernel");
  if (p.splits == 1) return IAMAP_OK;
  const dim3 rows(p.batch * p.Hq);
  return p.splits > 32
             ? launch_next("quant_attention_join_kernel", quant_attention_join_kernel<D, 1024>, rows, 1024, 0, st, p)
             : launch_next("quant_attention_join_kernel", quant_attention_join_kernel<D, 256>, rows, 256, 0, st, p);
}
template <int D, int KB, int VB>
int launch_a(const AttnParams& p, cudaStream_t st) {
  return p.k.page_size % kTok == 0 ? launch<D, KB, VB, true>(p, st)
                                   : launch<D, KB, VB, false>(p, st);
}
template <int D>
int launch_d(const AttnParams& p, int kb, int vb, cudaStream_t st) {
  if (kb == 4) return vb == 4 ? launch_a<D, 4, 4>(p, st) : launch_a<D, 4, 8>(p, st);
  return vb == 4 ? launch_a<D, 8, 4>(p, st) : launch_a<D, 8, 8>(p, st);
}

}  // namespace
}  // namespace iamap

using namespace iamap;

extern "C" size_t iamap_attention_paged_quant_workspace_bytes(int batch, int H_q, int d,
                                                              int max_ctx) {
  if (batch < 1 || H_q < 1 || d < 1 || max_ctx < 0) return 0;
  if (batch > 65535 || (int64_t)batch * H_q > 0x7fffff || max_ctx > kMaxCtx) return 0;   // refused by the call
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
  if (batch > 65535 || (int64_t)batch * H_q > 0x7fffff)
    return set_error(IAMAP_ERR_UNSUPPORTED, "batch above 65535, or batch times heads too large");
  attention_split(batch, (int)units, max_ctx, &p.chunk, &p.splits);
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
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return d == 64 ? launch_d<64>(p, k_bits, v_bits, st)
                 : launch_d<128>(p, k_bits, v_bits, st);
}
