// iamap_mapped_av_paged_quant: the mapped decode step over a quantised value cache.
//
//   out[b, r] = sum_{j < ctx[b]} w[r, j] v^[b, j, r / group],  w[r, j] = sum_s W[r, s] p[b, s, j]
//
// Bound by the value bytes (72 a token and head of 128 in 4 bits). A CTA takes a range of tokens of one
// sequence and up to eight units, a unit being a value head with up to eight of the receiver heads that
// read it. First the CTA forms w of its receivers and tokens in shared memory (fp32); then each warp
// streams the tokens of one unit through a ring of copies, 32 at a time.
//
// The product runs on matrix instructions with the codes as one operand (quant_tile.cuh). Its other
// operand, the weight times the token's scale of the group, has to keep fp32's precision in fp16, so it
// is held as two parts, hi + lo, in two columns of the same instruction:
//
//   w 2^k = h + l,  P1 = rn(h s),  P2 = rn(l s + (h s - P1))    (h s - P1 is exact in one fma)
//
// which leaves an error of 2^-22 relative, or 2^-25 absolute: k brings the largest |w| of the unit's
// tokens near 2^15, and scales outside [2^-8, 1) are brought under 1 by a power of two of the unit, so
// nothing overflows and the absolute part is far below the largest products.
// With one receiver a value head (group 1), the eight columns are the (group of 32, part) pairs, and
// one operand serves all groups; otherwise they are (receiver, part) and the operand is formed a group.
//
// Partial sums of the ranges go to the workspace; a second kernel adds them in a fixed order.
#include <algorithm>

#include "internal.h"
#include "quant_tile.cuh"

namespace iamap {
namespace {

using namespace qt;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kChunk = 512;          // tokens a CTA, two a thread
constexpr int kMaxRecv = 16;         // receivers a CTA
constexpr int kPad = 4;              // floats between the receivers' weight rows

struct MappedParams {
  const float* rows;                 // [batch, H_s, stride]
  int stride;
  const float* W;                    // [H_r, H_s]
  QuantPages v;
  const int32_t* ctx_lens;
  int max_ctx, batch, H_s, H_r, group;
  int rj;                            // receivers a unit
  int rtiles;                        // units a value head
  int units;                         // of a sequence: value heads * rtiles
  int hs, parts;                     // units a CTA; warps that share a unit's tokens
  int slices;                        // CTAs a range
  int chunks;                        // ranges of max_ctx tokens
  float* out;                        // [batch, H_r, d]
  float* partial;                    // [batch][chunks][H_r][d]
  unsigned int* status;
};

// Exponent k that brings the largest |w| (bits of a non-negative float) into [2^14, 2^15).
__device__ __forceinline__ int boost_exp(uint32_t wmax) {
  return wmax == 0 || wmax >= 0x7f800000u ? 0 : 14 - ((int)(wmax >> 23) - 127);
}
__device__ __forceinline__ float pow2i(int k) {
  // k in [-126, 127] after clamping; larger shifts are made in two steps by the caller
  return __uint_as_float((uint32_t)(min(max(k, -126), 127) + 127) << 23);
}

template <int D, int BITS>
struct Ring {
  static constexpr int kStage = kPair * D * BITS / 8;
  static constexpr int kStages = kStage <= 2048 ? 3 : 2;
  static constexpr int kWarp = kChunk * (D / 32) * 2 + kStages * kStage;   // scales and stages
};

// GM 0: group 1; GM 1, 2: up to four, eight receivers a unit.
template <int D, int BITS, bool ALIGNED, int GM>
__global__ void __launch_bounds__(kThreads, 2) quant_mapped_kernel(const MappedParams p) {
  constexpr int NG = D / 32, R = D * BITS / 8, SB = NG * 2, CT = GM == 2 ? 2 : 1;
  using RB = Ring<D, BITS>;
  constexpr int ST = RB::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ StreamShared<2, ST> shared[kWarps];
  __shared__ int up_s[kMaxRecv];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, tid = lane & 3;

  int u = blockIdx.x;
  const int slice = u % p.slices;
  u /= p.slices;
  const int b = u % p.batch, chunk = u / p.batch;
  const int ctx = quant_ctx(p.ctx_lens, b, p.max_ctx, p.status);
  const int nchunk = max(1, (ctx + kChunk - 1) / kChunk);
  if (chunk >= nchunk) return;
  const int j0 = chunk * kChunk, ntok = min(ctx - j0, kChunk);

  // this warp's unit and tokens: steps of 32 at j0 + 32 (part + parts i)
  const int unit = slice * p.hs + warp % p.hs, part = warp / p.hs;
  const bool live = unit < p.units;
  const int hk = live ? unit / p.rtiles : 0, rt = unit % p.rtiles;
  float* w_s = reinterpret_cast<float*>(smem + kWarps * RB::kWarp);
  const uint32_t scales = smem_u32(smem) + warp * RB::kWarp;   // the unit's scales, step after step
  Stream<ALIGNED, 2, 1, ST> in;
  in.init(&p.v, b, hk, j0 + part * kPair, p.parts * kPair, live ? j0 + ntok : 0, p.status,
          scales + kChunk * SB, &shared[warp]);
  in.template add<0>(p.v.codes, R);
  // all scales of the unit's tokens first (a few KB): their largest sets the operand's scale
  for (int i = 0; i < in.nsteps; ++i) {
    const uint32_t row = in.rows.at(j0 + (part + p.parts * i) * kPair + lane, p.status);
    cp_async<SB>(scales + (i * kPair + lane) * SB,
                 reinterpret_cast<const uint8_t*>(p.v.scales) + (row == kNoRow ? 0 : (uint64_t)row * SB),
                 row != kNoRow);
  }
  cp_async_commit();
#pragma unroll
  for (int i = 0; i < ST - 1; ++i) in.fill(i);

  // the weights of the CTA's receivers: two tokens a thread, eight receivers at a time
  const int recv = p.hs * p.rj;
  float* W_s = w_s + recv * (kChunk + kPad);               // [H_s][wcols], wcols a multiple of 8
  const int wcols = (recv + 7) & ~7;
  for (int e = threadIdx.x; e < p.H_s * wcols; e += kThreads) {
    const int s = e / wcols, r = e - s * wcols, un = slice * p.hs + r / p.rj;
    const int in = (un % p.rtiles) * p.rj + r % p.rj;        // receiver within its value head
    const bool ok = r < recv && un < p.units && in < p.group;
    W_s[e] = ok ? __ldg(p.W + ((int64_t)(un / p.rtiles) * p.group + in) * p.H_s + s) : 0.f;
  }
  __syncthreads();
  {
    const int t = threadIdx.x;
    const float* row = p.rows + (int64_t)b * p.H_s * p.stride + j0 + t;
    const bool ok0 = t < ntok, ok1 = t + kThreads < ntok;
    for (int r0 = 0; r0 < recv; r0 += 8) {
      float a[8], c[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) a[k] = c[k] = 0.f;
#pragma unroll 4
      for (int s = 0; s < p.H_s; ++s) {
        const float x = ok0 ? __ldg(row + (int64_t)s * p.stride) : 0.f;
        const float y = ok1 ? __ldg(row + (int64_t)s * p.stride + kThreads) : 0.f;
        const float4 u0 = *reinterpret_cast<const float4*>(W_s + s * wcols + r0);
        const float4 u1 = *reinterpret_cast<const float4*>(W_s + s * wcols + r0 + 4);
        const float wk[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) a[k] = fmaf(wk[k], x, a[k]), c[k] = fmaf(wk[k], y, c[k]);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (r0 + k < recv) {
          w_s[(r0 + k) * (kChunk + kPad) + t] = ok0 ? a[k] : 0.f;
          w_s[(r0 + k) * (kChunk + kPad) + t + kThreads] = ok1 ? c[k] : 0.f;
        }
    }
  }
  __syncthreads();
  // each receiver's weights, times the power of two that brings the largest near 2^15, as two fp16 parts
  // (high part in the low half) in place
  for (int r = warp; r < recv; r += kWarps) {
    float* w = w_s + r * (kChunk + kPad);
    uint32_t m = 0;
    float v[kChunk / 32];
#pragma unroll
    for (int k = 0; k < kChunk / 32; ++k) {
      v[k] = w[lane + 32 * k];
      m = max(m, __float_as_uint(v[k]) & 0x7fffffffu);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    const int up = boost_exp(m);
    const float up0 = pow2i(up / 2), up1 = pow2i(up - up / 2);
#pragma unroll
    for (int k = 0; k < kChunk / 32; ++k) {
      const float x = v[k] * up0 * up1, h = __half2float(__float2half_rn(x));
      reinterpret_cast<uint32_t*>(w)[lane + 32 * k] = pack_f16(h, x - h);
    }
    if (lane == 0) up_s[r] = up;
  }
  __syncthreads();

  // largest scale of the unit's tokens
  cp_async_wait<ALIGNED ? 0 : ST - 1>();                     // the scales, started before the ring's copies
  __syncwarp();
  const int nrj = min(p.rj, p.group - rt * p.rj);            // receivers of this unit
  uint32_t smax = 0;
  for (int e = lane * 4; e < in.nsteps * kPair * SB; e += 128) {
    const uint32_t v = lds32(scales + e) & 0x7fff7fffu;
    smax = __vmaxu2(smax, v & ~__vcmpgtu2(v, 0x7bff7bffu));   // infinities and NaN set no scale
  }
  smax = max(smax & 0xffffu, smax >> 16);
  smax = __reduce_max_sync(0xffffffffu, smax);
  int sdown = 0;
  if (smax != 0) {
    const int es = (int)(__float_as_uint(__half2float(__ushort_as_half((unsigned short)smax))) >> 23) - 127;
    if (es >= 0 || es < -8) {                                // unusual sizes: scales brought under 1
      sdown = es + 1;
      // 2^-sdown in two factors that fp16 has (sdown is in [-23, 16])
      const uint32_t f0 = pack_f16(pow2i(-(sdown / 2)), pow2i(-(sdown / 2)));
      const uint32_t f1 = pack_f16(pow2i(-(sdown - sdown / 2)), pow2i(-(sdown - sdown / 2)));
      for (int e = lane * 4; e < in.nsteps * kPair * SB; e += 128)
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(scales + e),
                     "r"(hmul2(hmul2(lds32(scales + e), f0), f1))
                     : "memory");
      __syncwarp();
    }
  }
  // this column's receiver (0 stands in for one that the unit lacks)
  uint32_t wr[CT];
  int kexp[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    int r = GM == 0 ? 0 : 4 * c + (gid >> 1);
    r = (warp % p.hs) * p.rj + (r < nrj ? r : 0);
    wr[c] = smem_u32(w_s + r * (kChunk + kPad) + part * kPair + tid);
    kexp[c] = up_s[r] - sdown;
  }

  float o[CT][2 * NG][4];
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int i = 0; i < 2 * NG; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[c][i][e] = 0.f;
  const bool lo = gid & 1;

  for (int i = 0; i < in.nsteps; ++i) {
    in.fill(i + ST - 1);
    uint32_t st;
    const uint32_t* masks;
    if (!in.take(&st, &masks)) break;
    const uint32_t mask = masks[0];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      ValueTile<D, BITS> vt;
      vt.load(st + q * kTok * R);
      const uint32_t sp = scales + (i * kPair + q * kTok + tid) * SB;   // tokens tid + 4 k
      uint2 sc[4];
      if (GM != 0) {
#pragma unroll
        for (int k = 0; k < 4; ++k) sc[k] = lds_scales<NG>(sp + 4 * k * SB);
      }
      uint32_t hp[CT][2], lp[CT][2];                          // weight pairs, high and low parts
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t at = wr[c] + (i * p.parts * kPair + q * kTok) * 4 + 32 * h;
          const uint32_t a = lds32(at), d = lds32(at + 16);
          hp[c][h] = __byte_perm(a, d, 0x5410);
          lp[c][h] = __byte_perm(a, d, 0x7632);
        }
      if (mask != 0xffffffffu) {
        // tokens that do not exist: no weight (their scales are 0, their codes may be anything)
        const uint32_t m = mask >> (q * kTok + tid);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t keep = ((m >> (8 * h)) & 1 ? 0xffffu : 0u) | ((m >> (8 * h + 4)) & 1 ? 0xffff0000u : 0u);
#pragma unroll
          for (int c = 0; c < CT; ++c) hp[c][h] &= keep, lp[c][h] &= keep;
        }
      }
      auto weight = [&](int c, int h, uint32_t s) {
        const uint32_t p1 = hmul2(hp[c][h], s);
        const uint32_t p2 = hfma2(lp[c][h], s, hfma2(hp[c][h], s, p1 ^ 0x80008000u));
        return lo ? p2 : p1;
      };
      uint32_t pb[CT][2];
      if (GM == 0) {
        const uint32_t sg = sp + 2 * ((gid >> 1) % NG);       // this column's group
#pragma unroll
        for (int h = 0; h < 2; ++h)
          pb[0][h] = weight(0, h, __byte_perm(lds16(sg + 8 * h * SB), lds16(sg + (8 * h + 4) * SB), 0x5410));
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if (GM != 0) {
#pragma unroll
          for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h) pb[c][h] = weight(c, h, scale_pair(sc + 2 * h, g));
        }
        uint32_t r[4], t[4];
        vt.group(g, r, t);
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          mma_f16(o[c][2 * g], r[0], r[1], t[0], t[1], pb[c][0], pb[c][1]);
          mma_f16(o[c][2 * g + 1], r[2], r[3], t[2], t[3], pb[c][0], pb[c][1]);
        }
      }
    }
    __syncwarp();
  }
  if (!ALIGNED) cp_async_wait<0>();

  // columns 2 tid, 2 tid + 1 are the two parts of receiver tid (GM 0: of group tid)
  const bool direct = nchunk == 1;
  float* o_s = reinterpret_cast<float*>(smem);               // [part][unit of the CTA][rj][D]
  if (p.parts > 1) __syncthreads();                          // the rings are free
  auto row_of = [&](int un, int r) {                         // where a receiver's sums go
    const int64_t row = (int64_t)(un / p.rtiles) * p.group + (un % p.rtiles) * p.rj + r;
    return direct ? p.out + ((int64_t)b * p.H_r + row) * D
                  : p.partial + (((int64_t)b * p.chunks + chunk) * p.H_r + row) * D;
  };
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    const int r = GM == 0 ? 0 : 4 * c + tid;
    const int k = __shfl_sync(0xffffffffu, kexp[c], GM == 0 ? 0 : 8 * tid);
    const float dn0 = pow2i(-(k / 2)), dn1 = pow2i(-(k - k / 2));
    if (r >= nrj || !live) continue;
    float* dst = (p.parts > 1 ? o_s + ((part * p.hs + warp % p.hs) * p.rj + r) * D : row_of(unit, r)) +
                 4 * gid;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      if (GM == 0 && tid != g) continue;
      const float* a = o[c][2 * g];
      const float* d = o[c][2 * g + 1];
      *reinterpret_cast<float4*>(dst + 32 * g) =
          make_float4((a[0] + a[1]) * dn0 * dn1, (a[2] + a[3]) * dn0 * dn1, (d[0] + d[1]) * dn0 * dn1,
                      (d[2] + d[3]) * dn0 * dn1);
    }
  }
  if (p.parts == 1) return;
  __syncthreads();
  const int span = p.hs * p.rj * D;                          // floats of one part
  for (int at = threadIdx.x * 4; at < span; at += kThreads * 4) {
    const int e = at / D, un = slice * p.hs + e / p.rj, r = e % p.rj;
    if (un >= p.units || (un % p.rtiles) * p.rj + r >= p.group) continue;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int q = 0; q < p.parts; ++q) {
      const float4 x = *reinterpret_cast<const float4*>(o_s + q * span + at);
      a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w;
    }
    *reinterpret_cast<float4*>(row_of(un, r) + (at - e * D)) = a;
  }
}

__global__ void __launch_bounds__(256) quant_mapped_join_kernel(const MappedParams p, int d) {
  const int E = p.H_r * d;
  const int b = blockIdx.y, e = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (e >= E) return;
  const int ctx = min(max(p.ctx_lens[b], 0), p.max_ctx);
  const int n = (ctx + kChunk - 1) / kChunk;
  if (n <= 1) return;
  const float* src = p.partial + (int64_t)b * p.chunks * E + e;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int c = 0; c < n; ++c) {
    const float4 x = *reinterpret_cast<const float4*>(src + (int64_t)c * E);
    a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w;
  }
  *reinterpret_cast<float4*>(p.out + (int64_t)b * E + e) = a;
}

// Units and their place in a CTA for `group` receivers a value head.
void mapped_shape(int H_kv, int group, int max_ctx, MappedParams* p) {
  p->group = group;
  p->rj = std::min(group, 8);
  p->rtiles = (group + p->rj - 1) / p->rj;
  p->units = H_kv * p->rtiles;
  // at most kMaxRecv receivers a CTA keep their weights in 33 KB, so that two CTAs fit an SM
  p->hs = 1;
  while (p->hs * 2 <= std::min(p->units, kWarps) && p->hs * 2 * p->rj <= kMaxRecv) p->hs *= 2;
  p->parts = kWarps / p->hs;
  p->slices = (p->units + p->hs - 1) / p->hs;
  p->chunks = std::max(1, (max_ctx + kChunk - 1) / kChunk);
}

template <int D, int BITS, bool ALIGNED, int GM>
int launch(const MappedParams& p, unsigned int blocks, cudaStream_t st) {
  const int bytes = kWarps * Ring<D, BITS>::kWarp +
                    p.hs * p.rj * (kChunk + kPad) * 4 + p.H_s * ((p.hs * p.rj + 7) & ~7) * 4;
  IAMAP_CUDA_CHECK(cudaFuncSetAttribute(quant_mapped_kernel<D, BITS, ALIGNED, GM>,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
  quant_mapped_kernel<D, BITS, ALIGNED, GM><<<blocks, kThreads, bytes, st>>>(p);
  IAMAP_LAUNCH_CHECK("quant_mapped_kernel");
  if (p.chunks > 1) {
    quant_mapped_join_kernel<<<dim3((p.H_r * D / 4 + 255) / 256, p.batch), 256, 0, st>>>(p, D);
    IAMAP_LAUNCH_CHECK("quant_mapped_join_kernel");
  }
  return IAMAP_OK;
}
template <int D, int BITS>
int launch_d(const MappedParams& p, unsigned int blocks, cudaStream_t st) {
  const bool al = p.v.page_size % kTok == 0;
  if (p.group == 1)
    return al ? launch<D, BITS, true, 0>(p, blocks, st) : launch<D, BITS, false, 0>(p, blocks, st);
  if (p.rj <= 4)
    return al ? launch<D, BITS, true, 1>(p, blocks, st) : launch<D, BITS, false, 1>(p, blocks, st);
  return al ? launch<D, BITS, true, 2>(p, blocks, st) : launch<D, BITS, false, 2>(p, blocks, st);
}

}  // namespace
}  // namespace iamap

using namespace iamap;

extern "C" size_t iamap_mapped_av_paged_quant_workspace_bytes(int batch, int H_r, int d_v,
                                                              int max_ctx) {
  if (batch < 1 || H_r < 1 || d_v < 1 || max_ctx < 0) return 0;
  const size_t chunks = std::max(1, (max_ctx + kChunk - 1) / kChunk);
  return chunks > 1 ? sizeof(float) * batch * chunks * H_r * d_v : 256;
}

extern "C" int iamap_mapped_av_paged_quant(const float* p_rows, int ctx_stride, const float* W,
                                           const void* v_codes, const void* v_scales,
                                           int64_t num_pages, const int32_t* page_table,
                                           int max_pages, int page_size, const int32_t* ctx_lens,
                                           int max_ctx, int batch, int H_s, int H_r, int H_kv,
                                           int d_v, int bits, float* out, void* ws,
                                           size_t ws_bytes, void* stream) {
  clear_error();
  int rc = check_quant_pages(v_codes, v_scales, num_pages, page_table, max_pages, page_size, H_kv,
                             d_v, bits);
  if (rc) return rc;
  rc = check_quant_batch(ctx_lens, max_ctx, batch, max_pages, page_size);
  if (rc) return rc;
  if (H_r < 1 || H_r % H_kv != 0)
    return set_error(IAMAP_ERR_INVALID_ARG, "H_kv=%d must divide H_r=%d", H_kv, H_r);
  if (!p_rows || !W || !out) return set_error(IAMAP_ERR_INVALID_ARG, "null pointer");
  if (H_s < 1 || H_s > 128 || H_r > 128)
    return set_error(IAMAP_ERR_UNSUPPORTED, "H_s and H_r must be in [1, 128]");
  if (batch > 65535) return set_error(IAMAP_ERR_UNSUPPORTED, "batch must be at most 65535");
  if ((reinterpret_cast<uintptr_t>(out) & 15u) != 0)
    return set_error(IAMAP_ERR_INVALID_ARG, "out must be 16-byte aligned");
  if (ctx_stride < 1 || ctx_stride < max_ctx)
    return set_error(IAMAP_ERR_INVALID_ARG, "ctx_stride=%d is below max_ctx=%d", ctx_stride, max_ctx);
  MappedParams p{};
  mapped_shape(H_kv, H_r / H_kv, max_ctx, &p);
  const size_t need = p.chunks > 1 ? sizeof(float) * batch * p.chunks * H_r * d_v : 1;
  if (!ws || ws_bytes < need)
    return set_error(IAMAP_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws_bytes);
  if ((reinterpret_cast<uintptr_t>(ws) & 15u) != 0)
    return set_error(IAMAP_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  const int64_t blocks = (int64_t)p.chunks * batch * p.slices;
  if (blocks > 0x7fffffff)
    return set_error(IAMAP_ERR_UNSUPPORTED, "batch times heads times max_ctx is too large");
  DeviceContext* ctx = device_context();
  if (!ctx) return IAMAP_ERR_CUDA;
  p.rows = p_rows;
  p.stride = ctx_stride;
  p.W = W;
  p.v = QuantPages{static_cast<const uint8_t*>(v_codes), static_cast<const __half*>(v_scales),
                   num_pages, page_table, max_pages, page_size, H_kv};
  p.ctx_lens = ctx_lens;
  p.max_ctx = max_ctx;
  p.batch = batch;
  p.H_s = H_s;
  p.H_r = H_r;
  p.out = out;
  p.partial = static_cast<float*>(ws);
  p.status = ctx->status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (d_v == 64)
    return bits == 4 ? launch_d<64, 4>(p, (unsigned int)blocks, st)
                     : launch_d<64, 8>(p, (unsigned int)blocks, st);
  return bits == 4 ? launch_d<128, 4>(p, (unsigned int)blocks, st)
                   : launch_d<128, 8>(p, (unsigned int)blocks, st);
}
