// iamap_mapped_av_paged_quant: the mapped decode step over a quantised value cache.
//
//   out[b, r] = sum_{j < ctx[b]} w[r, j] v^[b, j, r / group],  w[r, j] = sum_s W[r, s] p[b, s, j]
//
// Bound by the value bytes (72 a token and head of 128 in 4 bits). A first kernel forms the weights w and
// leaves them in the workspace; then a CTA takes a range of tokens of one sequence and up to eight units, a
// unit being a value head with up to eight of the receiver heads that read it, and each warp streams the
// tokens of one unit with their weights through a ring of copies, 64 (or 32) at a time. No barrier stands
// in the loop. Twelve ragged sequences of up to 32768 tokens, 14 rows to 64 heads over 8 value heads of 128
// in 8 bits: 64 us, the weights 18 of them (weights formed by the CTA for its whole range, between barriers:
// 104; by every warp for each step: 125). Four of 8704 tokens, 64 value heads in 4 bits: 57 us (62 with
// 32 tokens a step and three CTAs an SM).
//
// The product runs on matrix instructions with the codes as one operand (quant_tile.cuh). Its other
// operand, the weight times the token's scale of the group, has to keep fp32's precision in fp16, so the
// product t is formed in fp32 and held as two parts, high and low, in two columns of their own sums:
//
//   t = w 2^k (s 2^-e),  t = high + 2^-12 low,  error at most 2^-22 |t| or 2^-37
//
// The first kernel brings the largest |w| of each receiver and 512 tokens, which is what a range holds, into
// [2^13, 2^14), and ScalePowers a group's largest s into [1/2, 1): the absolute part is 2^-49 of the product
// of the two, so a token that takes almost all of the weight, with values near zero, leaves the others their
// bits. (Parts formed in fp16, from weights held in two, keep 2^-39 of it; 57 and 62 us where this takes 57
// and 64.) With one receiver a value head (group 1), the eight columns are the (group of 32, part) pairs, and
// one operand serves all groups; otherwise the operand is formed a group: up to four receivers with their
// parts side by side, or eight with their parts in two tiles.
//
// Partial sums of the ranges go to the workspace; a third kernel adds them in a fixed order.
#include <algorithm>

#include "internal.h"
#include "quant_tile.cuh"

namespace iamap {
namespace {

using namespace qt;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kBlock = 32;           // tokens of one record of weights, RJ receivers'
// Tokens of a range. Four equal sequences of 8704 and twelve ragged ones of up to 32768, before products were
// formed in fp32: 56 and 62 us; with ranges of 256 59 and 65, with 1024 55 and 98 (a ragged batch then has
// fewer ranges than the device CTAs).
constexpr int kChunk = 512;

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
  uint8_t* records;                  // [batch][units][blocks] records of weights
  int* powers;                       // [batch][units][chunks][RJ]: the powers of two of a range's weights
  float* partial;                    // [batch][chunks][H_r][d]
  unsigned int* status;
};

// x = b[0] + b[1] + b[2] in bf16, each part the rounding of what the ones before it leave, for a pair of values
__device__ __forceinline__ void split3(float x, float y, uint32_t (&b)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(b[i]) : "f"(y), "f"(x));
    x -= __uint_as_float(b[i] << 16);
    y -= __uint_as_float(b[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
               "{%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Weights of 32 tokens and one unit: of the tokens t and t + 4 a pair in fp32,
// [4 groups of 8 tokens][RJ / 4][t = 0..3][receiver] for four and eight receivers, [4][t] for one: the order in
// which a warp's lanes want them.
//
// The weights: a CTA a range of tokens for sixteen receivers, a warp 64 of the tokens. The products run on
// matrix instructions with both factors in three bf16 parts, of 2^-8 and 2^-17 of the first at most; the six
// products of the larger parts leave out 1.5 x 2^-24 of a product, fp32's own rounding. (fp32 arithmetic,
// eight receivers a CTA: 28 us where this takes 19, 118 thousand tokens, 14 rows to 64 heads; a CTA for
// every range up to max_ctx, most of them behind a sequence's end: 24.)
constexpr int kWeightSlots = 16, kWeightTokens = 64, kWeightThreads = kChunk / kWeightTokens * 32;
template <int RJ>
__global__ void __launch_bounds__(kWeightThreads, 2) quant_weights_kernel(const MappedParams p, int slices) {
  constexpr int UN = kWeightSlots / RJ, NT = kWeightSlots / 8, MT = kWeightTokens / 16;
  __shared__ uint32_t max_s[3][kWeightSlots];                // of this item, the next, and the last
  let_next_start();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, tid = lane & 3;
  if (threadIdx.x < 3 * kWeightSlots) max_s[0][threadIdx.x] = 0;
  __syncthreads();
  // Items are counted over the ranges that the sequences have, so that short ones beside a long one leave
  // no CTAs that only find nothing to do: `ranges` of the 32 sequences from b0 on, `before` up to there.
  int b0 = 0, before = 0, len = 0, ranges = 0, upto = 0;
  auto lengths = [&] {
    len = b0 + lane < p.batch ? quant_ctx(p.ctx_lens, b0 + lane, p.max_ctx, p.status) : 0;
    upto = (len + kChunk - 1) / kChunk;
#pragma unroll
    for (int x = 1; x < 32; x *= 2) {
      const int y = __shfl_up_sync(0xffffffffu, upto, x);
      if (lane >= x) upto += y;
    }
    ranges = __shfl_sync(0xffffffffu, upto, 31);
  };
  lengths();
  int now = 0;
  for (int item = blockIdx.x;; item += gridDim.x, now = now == 2 ? 0 : now + 1) {
    const int u0 = item % slices * UN, range = item / slices;
    while (range - before >= ranges && b0 + 32 < p.batch) before += ranges, b0 += 32, lengths();
    if (range - before >= ranges) return;
    const int which = __ffs(__ballot_sync(0xffffffffu, range - before < upto)) - 1, b = b0 + which;
    const int ctx = __shfl_sync(0xffffffffu, len, which);
    const int chunk = range - before - (__shfl_sync(0xffffffffu, upto, which) - (ctx + kChunk - 1) / kChunk);
    // rows gid and gid + 8 of a matrix tile are the tokens j and j + 4
    const int j0 = chunk * kChunk + warp * kWeightTokens, j = j0 + (gid & 3) + 8 * (gid >> 2);
    const bool live = j0 < ctx;
    float w[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) w[m][i][e] = 0.f;
    if (live) {
      const float* W[NT];                                    // column gid's row of W
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int k = 8 * i + gid, un = u0 + k / RJ, of = un % p.rtiles * p.rj + k % RJ;
        const bool ok = un < p.units && k % RJ < p.rj && of < p.group;
        W[i] = ok ? p.W + ((int64_t)(un / p.rtiles) * p.group + of) * p.H_s : nullptr;
      }
      int at[2 * MT];                                        // tokens that do not exist read the last one's row
#pragma unroll
      for (int m = 0; m < 2 * MT; ++m) at[m] = min(j + 16 * (m >> 1) + 4 * (m & 1), ctx - 1);
      for (int s0 = 0; s0 < p.H_s; s0 += 16) {
        const float* row[4];
        bool ok[4];
        uint32_t wb[NT][2][3];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int s = s0 + 2 * tid + (e & 1) + 8 * (e >> 1);
          ok[e] = s < p.H_s;
          row[e] = p.rows + ((int64_t)b * p.H_s + s) * p.stride;
        }
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float* f = W[i] + s0 + 2 * tid + 8 * e;
            split3(W[i] && ok[2 * e] ? __ldg(f) : 0.f, W[i] && ok[2 * e + 1] ? __ldg(f + 1) : 0.f, wb[i][e]);
          }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          uint32_t a[4][3];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int h = 2 * (e >> 1), t = at[2 * m + (e & 1)];
            split3(ok[h] ? __ldg(row[h] + t) : 0.f, ok[h + 1] ? __ldg(row[h + 1] + t) : 0.f, a[e]);
          }
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            constexpr int part[6][2] = {{2, 0}, {1, 1}, {0, 2}, {1, 0}, {0, 1}, {0, 0}};
#pragma unroll
            for (int e = 0; e < 6; ++e) {
              const int x = part[e][0], y = part[e][1];
              mma_bf16(w[m][i], a[0][x], a[1][x], a[2][x], a[3][x], wb[i][0][y], wb[i][1][y]);
            }
          }
        }
      }
      if (j0 + kWeightTokens > ctx) {
        // a weight of a token that does not exist is 0, whatever W holds
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (j + 16 * m + 4 * (e >> 1) >= ctx) {
#pragma unroll
              for (int i = 0; i < NT; ++i) w[m][i][e] = 0.f;
            }
      }
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {                          // column 2 tid + e
          uint32_t m = 0;
#pragma unroll
          for (int k = 0; k < MT; ++k)
            m = max(m, max(__float_as_uint(w[k][i][e]) & 0x7fffffffu,
                         __float_as_uint(w[k][i][e + 2]) & 0x7fffffffu));
#pragma unroll
          for (int x = 4; x < 32; x *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, x));
          if (gid == 0) atomicMax(&max_s[now][8 * i + 2 * tid + e], m);
        }
    }
    if (threadIdx.x < kWeightSlots) max_s[now == 2 ? 0 : now + 1][threadIdx.x] = 0;
    __syncthreads();
    if (!live) continue;
    // infinities and NaN stay what they are
    auto power = [&](int k) {
      const uint32_t m = max_s[now][k];
      return m == 0 || m >= 0x7f800000u ? 0 : min(13 - ((int)(m >> 23) - 127), 126);
    };
    if (threadIdx.x < kWeightSlots && u0 + threadIdx.x / RJ < p.units)
      p.powers[(((int64_t)b * p.units + u0 + threadIdx.x / RJ) * p.chunks + chunk) * RJ + threadIdx.x % RJ] =
          power(threadIdx.x);
    const int n = p.chunks * (kChunk / kBlock), block = j0 / kBlock;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const float f0 = pow2i(power(8 * i + 2 * tid)), f1 = pow2i(power(8 * i + 2 * tid + 1));
      const int un = u0 + (8 * i + 2 * tid) / RJ;
      if (un >= p.units) continue;
      float* rec = reinterpret_cast<float*>(p.records) +
                      (((int64_t)b * p.units + un) * n + block) * (RJ * kBlock) +
                      (RJ == 8 ? (tid >> 1) * 32 : 0) + (gid & 3) * (RJ == 1 ? 2 : 8) + (RJ == 1 ? 0 : (tid & 1) * 4);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const float* c = w[m][i];
        const float4 v = make_float4(c[0] * f0, c[2] * f0, c[1] * f1, c[3] * f1);   // two receivers
        float* to = rec + (m >> 1) * (RJ * kBlock) + ((m & 1) * 2 + (gid >> 2)) * (RJ * 8);
        if (RJ == 1) {
          *reinterpret_cast<float2*>(to) = make_float2(v.x, v.y);
          if (un + 1 < p.units) *reinterpret_cast<float2*>(to + (int64_t)n * kBlock) = make_float2(v.z, v.w);
        } else {
          *reinterpret_cast<float4*>(to) = v;
        }
      }
    }
  }
}

template <int D, int BITS, int RJ>
struct Ring {
  static constexpr int kRow = D * BITS / 8 + (D / 32) * 2;
  // Tiles a step: as many as leave two CTAs an SM two stages a warp.
  static constexpr int kTiles = kRow <= 72 ? 4 : 2, kTokens = kTiles * kTok, kStages = 2;
  static constexpr int kExtra = kTokens * RJ * 4;          // weights a step
  static constexpr int kWarp = kStages * (kTokens * kRow + kExtra);
};

// GM 0: group 1; GM 1, 2: up to four, eight receivers a unit.
template <int D, int BITS, bool ALIGNED, int GM>
__global__ void __launch_bounds__(kThreads, 2) quant_mapped_kernel(MappedParams p) {
  constexpr int NG = D / 32, R = D * BITS / 8, SB = NG * 2, CT = GM == 2 ? 2 : 1;
  constexpr int RJ = GM == 0 ? 1 : 4 * GM;
  using RB = Ring<D, BITS, RJ>;
  constexpr int ST = RB::kStages, TK = RB::kTokens, REC = kBlock * RJ * 4;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ StreamShared<RB::kTiles, ST> shared[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, tid = lane & 3;

  let_next_start();
  int u = blockIdx.x;
  const int slice = u % p.slices;
  u /= p.slices;
  const int b = u % p.batch, chunk = u / p.batch;
  const int ctx = quant_ctx(p.ctx_lens, b, p.max_ctx, p.status);
  const int j0 = chunk * kChunk, j1 = min(ctx, j0 + kChunk);
  if (j0 >= j1 && chunk > 0) return;

  // this warp's unit and tokens: steps of TK at j0 + TK (part + parts i)
  const int unit = slice * p.hs + warp % p.hs, part = warp / p.hs;
  const bool live = unit < p.units;
  const int hk = live ? unit / p.rtiles : 0, rt = unit % p.rtiles;
  const int nrj = min(p.rj, p.group - rt * p.rj);            // receivers of this unit
  Stream<ALIGNED, RB::kTiles, 2, ST> in;
  in.init(&p.v, b, hk, j0 + part * TK, p.parts * TK, live ? j1 : 0, p.status,
          smem_u32(smem) + warp * RB::kWarp, &shared[warp]);
  in.template add<0>(p.v.codes, R);
  in.template add<1>(p.v.scales, SB);
  in.add_extra(p.records + (((int64_t)b * p.units + (live ? unit : 0)) * p.chunks * kChunk + in.first) * (RJ * 4),
               RB::kExtra, in.step * (RJ * 4));
  after_previous();                                          // the weights
#pragma unroll
  for (int i = 0; i < ST - 1; ++i) in.fill(i);

  float o[CT][2 * NG][4];
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int i = 0; i < 2 * NG; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[c][i][e] = 0.f;
  const bool low = gid & 1;                                  // GM 0, 1: this column holds low parts
  ScalePowers<NG, true> pw;
  pw.init();
  uint32_t down[NG / 2];                                     // the groups' 2^-e; GM 0: all of this column's group
#pragma unroll
  for (int k = 0; k < NG / 2; ++k) down[k] = 0x3c003c00u;

  for (int i = 0; i < in.nsteps; ++i) {
    in.fill(i + ST - 1);
    uint32_t st;
    const uint32_t* masks;
    if (!in.take(&st, &masks)) break;
    const uint32_t scales = st + TK * R;
    const uint32_t weights = scales + TK * SB +
                             (GM == 0 ? tid * 8 : tid * 32 + (GM == 1 ? gid >> 1 : (gid >> 2) * 16 + (gid & 3)) * 8);
    // a scale in the step that its group's power does not serve
    const uint2 all = lds64(scales + lane * 8 % (TK * SB));
    const uint2 all2 = TK * SB > 256 ? lds64(scales + 256 + lane * 8) : all;
    const uint32_t served = pw.served(all.x, 0) & pw.served(all.y, 1) & pw.served(all2.x, 0) & pw.served(all2.y, 1);
    if (__any_sync(0xffffffffu, (served & 0x80008000u) != 0x80008000u)) {
      uint32_t m[NG / 2] = {};
      const uint32_t q[4] = {all.x, all.y, all2.x, all2.y};
#pragma unroll
      for (int e = 0; e < (TK * SB > 256 ? 4 : 2); ++e) {
        const int t = (lane * 8 % (TK * SB) + 256 * (e >> 1) + 4 * (e & 1)) / SB;        // the word's token
        if ((masks[t >> 5] >> (t & 31)) & 1) m[e % (NG / 2)] = pw.larger(m[e % (NG / 2)], q[e]);
      }
      float f[NG];
      pw.raise(m, f);
      if (GM == 0) {                                         // this lane's columns are group tid's
#pragma unroll
        for (int g = 1; g < NG; ++g) f[0] = tid == g ? f[g] : f[0];
      }
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int k = 0; k < 2 * NG; ++k)
#pragma unroll
          for (int z = 0; z < 4; ++z) o[c][k][z] *= f[GM == 0 ? 0 : k / 2];
#pragma unroll
      for (int k = 0; k < NG / 2; ++k) {
        down[k] = pw.half(2 * k) | pw.half(2 * k + 1) << 16;
        if (GM == 0)
#pragma unroll
          for (int g = 0; g < NG; ++g)
            if ((gid >> 1) % NG == g) down[k] = pw.half(g) * 0x10001u;
      }
    }
#pragma unroll 1
    for (int h = 0; h < RB::kTiles / 2; ++h) {
      const uint32_t mask = masks[h];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int tile = 2 * h + q;
        ValueTile<D, BITS> vt;
        vt.load(st + tile * kTok * R);
        const uint32_t sp = scales + (tile * kTok + tid) * SB;           // tokens tid + 4 k
        uint2 sc[4];                                         // GM 0: this column's group's scale alone
#pragma unroll
        for (int k = 0; k < 4; ++k)
          sc[k] = GM != 0 ? lds_scales<NG>(sp + 4 * k * SB)
                          : make_uint2(lds16(sp + 4 * k * SB + 2 * ((gid >> 1) % NG)), 0u);
        float2 w[2];                                         // weights of tokens (tid, tid + 4), + 8
#pragma unroll
        for (int k = 0; k < 2; ++k)
          w[k] = lds<float2>(weights + h * REC + (2 * q + k) * (RJ * 32));
        if (mask != 0xffffffffu) {
          // tokens that do not exist: no weight and no scale (memory behind them may hold anything)
          const uint32_t m = mask >> (q * kTok + tid);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if (!((m >> (8 * k)) & 1)) w[k].x = 0.f, sc[2 * k] = make_uint2(0, 0);
            if (!((m >> (8 * k + 4)) & 1)) w[k].y = 0.f, sc[2 * k + 1] = make_uint2(0, 0);
          }
        }
        // operands of group g: tokens (tid, tid + 4) and + 8; c = 1 the low parts (GM 2)
        uint32_t pb[CT][2];
        auto operands = [&](int g) {
          const uint16_t f = (uint16_t)(down[(g >> 1) % (NG / 2)] >> 16 * (g & 1));
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t s0 = g < 2 ? sc[2 * k].x : sc[2 * k].y, s1 = g < 2 ? sc[2 * k + 1].x : sc[2 * k + 1].y;
            const uint64_t s = pair_f32(fma_f16((uint16_t)(s0 >> 16 * (g & 1)), f, 0.f),
                                        fma_f16((uint16_t)(s1 >> 16 * (g & 1)), f, 0.f));
            uint32_t hi, lo;
            split_f16(mul2(pair_f32(w[k].x, w[k].y), s), hi, lo);
            pb[0][k] = GM != 2 && low ? lo : hi;
            if (GM == 2) pb[CT - 1][k] = lo;
          }
        };
        if (GM == 0) operands(0);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          if (GM != 0) operands(g);
          uint32_t r[4], t[4];
          vt.group(g, r, t);
#pragma unroll
          for (int c = 0; c < CT; ++c) {
            mma_f16(o[c][2 * g], r[0], r[1], t[0], t[1], pb[c][0], pb[c][1]);
            mma_f16(o[c][2 * g + 1], r[2], r[3], t[2], t[3], pb[c][0], pb[c][1]);
          }
        }
      }
    }
    __syncwarp();
  }
  if (!ALIGNED) cp_async_wait<0>();

  // columns 2 tid, 2 tid + 1 are the two parts of receiver tid (GM 0: of group tid), or of GM 2's two tiles the
  // receivers 2 tid and 2 tid + 1
  const bool direct = ctx <= kChunk;
  float* o_s = reinterpret_cast<float*>(smem);               // [part][unit of the CTA][rj][D]
  if (p.parts > 1) __syncthreads();                          // the rings are free
  auto row_of = [&](int un, int r) {                         // where a receiver's sums go
    const int64_t row = (int64_t)(un / p.rtiles) * p.group + (un % p.rtiles) * p.rj + r;
    return direct ? p.out + ((int64_t)b * p.H_r + row) * D
                  : p.partial + (((int64_t)b * p.chunks + chunk) * p.H_r + row) * D;
  };
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    const int r = GM == 0 ? 0 : GM == 1 ? tid : 2 * tid + c;
    if (r >= nrj || !live) continue;
    const int power = j0 < j1 ? p.powers[(((int64_t)b * p.units + unit) * p.chunks + chunk) * RJ + r] : 0;
    float* dst = (p.parts > 1 ? o_s + ((part * p.hs + warp % p.hs) * p.rj + r) * D : row_of(unit, r)) +
                 4 * gid;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      if (GM == 0 && tid != g) continue;
      const int k = power - pw.e(g);
      const float dn0 = pow2i(-(k / 2)), dn1 = pow2i(-(k - k / 2));
      auto sum = [&](int i, int z) {                         // row z / 2 of the pair, both parts
        return fmaf(GM == 2 ? o[CT - 1][i][z + c] : o[0][i][z + 1], kLow, o[0][i][GM == 2 ? z + c : z]) * dn0 * dn1;
      };
      *reinterpret_cast<float4*>(dst + 32 * g) =
          make_float4(sum(2 * g, 0), sum(2 * g, 2), sum(2 * g + 1, 0), sum(2 * g + 1, 2));
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

// Adds the ranges of 128 output elements: eight warps take a range each in turn.
__global__ void __launch_bounds__(256) quant_mapped_join_kernel(MappedParams p, int d) {
  const int E = p.H_r * d;
  const int b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e = blockIdx.x * 128 + lane * 4;
  const int ctx = min(max(p.ctx_lens[b], 0), p.max_ctx);
  after_previous();
  const int n = (ctx + kChunk - 1) / kChunk;
  if (n <= 1) return;
  __shared__ __align__(16) float a_s[8][128];
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (e < E) {
    const float* src = p.partial + (int64_t)b * p.chunks * E + e;
#pragma unroll 4
    for (int c = warp; c < n; c += 8) {
      const float4 x = *reinterpret_cast<const float4*>(src + (int64_t)c * E);
      a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w;
    }
  }
  *reinterpret_cast<float4*>(&a_s[warp][lane * 4]) = a;
  __syncthreads();
  const int t = threadIdx.x;
  if (t >= 128 || blockIdx.x * 128 + t >= E) return;
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) sum += a_s[k][t];
  p.out[(int64_t)b * E + blockIdx.x * 128 + t] = sum;
}

// Units and their place in a CTA for `group` receivers a value head, and the workspace: records, powers
// from *powers_at, partial sums from *partial_at.
size_t mapped_shape(int batch, int H_kv, int group, int d, int max_ctx, MappedParams* p,
                    size_t* powers_at, size_t* partial_at) {
  p->group = group;
  p->rj = std::min(group, 8);
  p->rtiles = (group + p->rj - 1) / p->rj;
  p->units = H_kv * p->rtiles;
  p->hs = 1;
  while (p->hs * 2 <= std::min(p->units, kWarps)) p->hs *= 2;
  p->parts = kWarps / p->hs;
  p->slices = (p->units + p->hs - 1) / p->hs;
  p->chunks = std::max(1, (max_ctx + kChunk - 1) / kChunk);
  const size_t rj = p->rj == 1 ? 1 : p->rj <= 4 ? 4 : 8, ranges = (size_t)batch * p->units * p->chunks;
  *powers_at = ranges * kChunk * rj * 4;
  *partial_at = *powers_at + (ranges * rj * 4 + 255) / 256 * 256;
  return *partial_at +
         (p->chunks > 1 ? sizeof(float) * batch * p->chunks * H_kv * group * (size_t)d : 0);
}

template <int RJ>
int launch_weights(const MappedParams& p, cudaStream_t st) {
  constexpr int UN = kWeightSlots / RJ;
  const int slices = (p.units + UN - 1) / UN;
  const int64_t items = (int64_t)slices * p.batch * p.chunks;
  quant_weights_kernel<RJ><<<(unsigned int)std::min<int64_t>(items, kSms * 2), kWeightThreads, 0, st>>>(p, slices);
  IAMAP_LAUNCH_CHECK("quant_weights_kernel");
  return IAMAP_OK;
}

template <int D, int BITS, bool ALIGNED, int GM>
int launch(const MappedParams& p, unsigned int blocks, cudaStream_t st) {
  constexpr int RJ = GM == 0 ? 1 : 4 * GM;
  int rc = launch_weights<RJ>(p, st);
  if (rc) return rc;
  const int bytes = std::max(kWarps * Ring<D, BITS, RJ>::kWarp, p.parts > 1 ? kWarps * p.rj * D * 4 : 0);
  IAMAP_CUDA_CHECK(cudaFuncSetAttribute(quant_mapped_kernel<D, BITS, ALIGNED, GM>,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
  rc = launch_next("quant_mapped_kernel", quant_mapped_kernel<D, BITS, ALIGNED, GM>, dim3(blocks), kThreads,
                   bytes, st, p);
  if (rc || p.chunks == 1) return rc;
  return launch_next("quant_mapped_join_kernel", quant_mapped_join_kernel,
                     dim3((p.H_r * D + 127) / 128, p.batch), 256, 0, st, p, D);
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
  if (batch > 65535 || H_r > 128 || max_ctx > kMaxCtx) return 0;     // refused by the call
  // the most that any grouping of the H_r heads needs
  size_t most = 256;
  for (int group = 1; group <= H_r; ++group) {
    if (H_r % group != 0) continue;
    MappedParams p{};
    size_t a, b;
    most = std::max(most, mapped_shape(batch, H_r / group, group, d_v, max_ctx, &p, &a, &b));
  }
  return most;
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
  size_t powers_at = 0, partial_at = 0;
  const size_t need = mapped_shape(batch, H_kv, H_r / H_kv, d_v, max_ctx, &p, &powers_at, &partial_at);
  const int64_t blocks = (int64_t)p.chunks * batch * p.slices;
  if (blocks > 0x7fffffff)
    return set_error(IAMAP_ERR_UNSUPPORTED, "batch times heads times max_ctx is too large");
  if (!ws || ws_bytes < need)
    return set_error(IAMAP_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws_bytes);
  if ((reinterpret_cast<uintptr_t>(ws) & 15u) != 0)
    return set_error(IAMAP_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
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
  p.records = static_cast<uint8_t*>(ws);
  p.powers = reinterpret_cast<int*>(static_cast<uint8_t*>(ws) + powers_at);
  p.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + partial_at);
  p.status = ctx->status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (d_v == 64)
    return bits == 4 ? launch_d<64, 4>(p, (unsigned int)blocks, st)
                     : launch_d<64, 8>(p, (unsigned int)blocks, st);
  return bits == 4 ? launch_d<128, 4>(p, (unsigned int)blocks, st)
                   : launch_d<128, 8>(p, (unsigned int)blocks, st);
}
