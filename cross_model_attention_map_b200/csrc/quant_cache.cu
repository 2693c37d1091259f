// iamap_cache_write / iamap_cache_read: quantising new keys or values into their pages, and reading
// ranges of sequences back as packed bf16 rows (format: quant_cache.cuh).
//
//   m = max |x| of a group of 32,  s = fp16(min(m / Q, 65504)),  c = clamp(rint(x / s), -Q, Q)
//
// Both are bound by HBM: 2 + bits / 8 + 1 / 16 bytes an element. At that rate an SM has some 100
// instructions for every 8 elements of 32 lanes, so: a lane holds half a group (the scale, its reciprocal
// and the addresses serve 16 elements), a quotient is half of a paired fused multiply-add and addition, and
// a CTA looks its tokens' places up once, while its loads are in flight. 40960 tokens of 40 heads of 128 in
// 4 bits, written and read back, a pass launched from Python: 207 us for 1.07 GB, 5.2 TB/s. Alone and cold the
// write takes 103 us, with 3 in 4 issue slots taken, and the read 88 (rows not loaded ahead and single additions
// made the pass 9 % longer; 8 elements a lane with IEEE divisions and a lookup a lane 3.5 times as long).
#include <algorithm>

#include "internal.h"
#include "quant_cache.cuh"

namespace iamap {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 2;         // half-groups in flight a thread that writes
constexpr int kReadUnroll = 3;     // one that reads
constexpr int kMaxTokens = 128;    // tokens a CTA

// A row's place: the pool row of its head 0 (head h: h * page_size rows further), or
constexpr int64_t kNoToken = -1;   // the row belongs to no sequence (a padded batch)
constexpr int64_t kBadPlace = -2;  // its position or page is out of range

struct CacheIoParams {
  const __nv_bfloat16* x;   // write: rows to quantise, x_stride elements apart
  __nv_bfloat16* out;       // read: rows to fill, packed
  int64_t x_stride;
  int64_t n;                // rows of x / out
  const int32_t* cu;        // [num_seqs + 1] rows of each sequence
  const int32_t* starts;    // [num_seqs] position of each sequence's first row
  int num_seqs;
  int tokens;               // rows a CTA
  int per;                  // half-groups a row: H * d / 16
  uint32_t per_inv;         // ceil(2^32 / per)
  QuantPages pages;
  uint8_t* codes;           // write: pages.codes, pages.scales
  __half* scales;
  unsigned int* status;
};

__device__ __forceinline__ int64_t place_of(const CacheIoParams& p, int64_t i) {
  if (i >= p.n || i < p.cu[0] || i >= p.cu[p.num_seqs]) return kNoToken;
  int lo = 0, hi = p.num_seqs;          // cu[lo] <= i < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.cu[mid] <= i) lo = mid; else hi = mid;
  }
  const int64_t pos = (int64_t)p.starts[lo] + (i - p.cu[lo]);
  if (pos < 0 || pos >= (int64_t)p.pages.max_pages * p.pages.page_size || pos > 0x7fffffff)
    return kBadPlace;
  const int64_t row = quant_row(p.pages, lo, 0, (int)pos);
  return row < 0 ? kBadPlace : row;
}

// The places of the CTA's tokens; bad ones are reported.
__device__ __forceinline__ void find_places(const CacheIoParams& p, int64_t i0, int64_t* place) {
  for (int t = threadIdx.x; t < p.tokens; t += kThreads) {
    place[t] = place_of(p, i0 + t);
    if (place[t] == kBadPlace) raise_status(p.status, IAMAP_DEV_BAD_INDEX);
  }
}

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
  return d;
}

// Levels of eight elements w (bf16 pairs) under the scale whose reciprocal is r (within 1 ulp): x / s
// rounded to even, exactly, plus the offset, in the low byte of each u. x r + 1536 is rounded to
// multiples of 2^-13 and |x / s| < 128, so it is within 2^-13 of x / s + 1536. x has 8 significant bits and s at
// most 11: x / s is a tie k + 1/2, which is then met exactly (the error before that rounding is below
// 2^-15), or at least 2^-12 away from one, and stays on its side. The addition of 2^23 + 2^22 + offset -
// 1536 rounds to an integer, ties to even (the offset is even).
template <int BITS>
__device__ __forceinline__ void levels(const uint32_t* w, float r, uint32_t* u) {
  constexpr float kOff = 12582912.f + (BITS == 4 ? 8.f : 128.f) - 1536.f;
  const uint64_t rr = pair(r, r), add = pair(1536.f, 1536.f), off = pair(kOff, kOff);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint64_t t;
    asm("{ .reg .b64 t; fma.rn.f32x2 t, %1, %2, %3; add.rn.f32x2 %0, t, %4; }"
        : "=l"(t) : "l"(pair(bf16_lo(w[e]), bf16_hi(w[e]))), "l"(rr), "l"(add), "l"(off));
    asm("mov.b64 {%0, %1}, %2;" : "=r"(u[2 * e]), "=r"(u[2 * e + 1]) : "l"(t));
  }
}
// The same where x / s may exceed Q: s is subnormal, saturated or 0.
template <int BITS>
__device__ __forceinline__ void levels_clamped(const uint32_t* w, float s, uint32_t* u) {
  constexpr float Q = BITS == 4 ? 7.f : 127.f;
  const float r = s > 0.f ? rcp(s) : 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = e & 1 ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]);
    const float t = s > 0.f ? fminf(fmaxf(__fmul_rn(x, r), -Q), Q) : 0.f;
    u[e] = __float_as_uint(__fadd_rn(__fadd_rn(t, 1536.f), 12582912.f + (BITS == 4 ? 8.f : 128.f) - 1536.f));
  }
}
// Low bytes of four words.
__device__ __forceinline__ uint32_t low_bytes(const uint32_t* u) {
  return __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
}

// Lane 2 g + h of a row holds elements 8 h .. 8 h + 7 and 16 + 8 h .. of group g (so that the two lanes of
// a group load whole sectors): its runs 2 h, 2 h + 1, 4 + 2 h and 5 + 2 h.
template <int D, int BITS>
__global__ void __launch_bounds__(kThreads, 4) cache_write_kernel(const CacheIoParams p) {
  constexpr int L = D / 16, NG = D / kQuantGroup;
  constexpr float Q = BITS == 4 ? 7.f : 127.f;
  constexpr int RW = D * BITS / 32;                          // words of a row's codes
  __shared__ int64_t place[kMaxTokens];
  __shared__ __align__(16) uint32_t stage[kThreads / 32][32 / L][RW + 4];   // a warp's rows, with their scales
  const int64_t i0 = (int64_t)blockIdx.x * p.tokens;
  const int units = p.tokens * p.per;
  const int lane = threadIdx.x & 31, l = threadIdx.x % L, g = l >> 1, h = l & 1;
  const __nv_bfloat16* x0 = p.x + i0 * p.x_stride;
  const int live = (int)min((int64_t)p.tokens, p.n - i0);    // tokens that there are
  auto half = [&](int c, int* tok, int* rest) {
    *tok = p.tokens == 1 ? 0 : (int)__umulhi((uint32_t)c, p.per_inv);
    *rest = c - *tok * p.per;
  };
  uint32_t next[kUnroll][8];
  auto load = [&](int base) {
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int c = base + threadIdx.x + k * kThreads;
      if (c - lane >= units) break;                          // the whole warp
      int tok, rest;
      half(c < units ? c : h, &tok, &rest);
      // a lane past the CTA's rows reads its first one, past the last row that one; neither is stored
      const uint4* src =
          reinterpret_cast<const uint4*>(x0 + min(tok, live - 1) * p.x_stride + 16 * rest - 8 * h);
      const uint4 a = __ldcs(src), b = __ldcs(src + 2);
      next[k][0] = a.x, next[k][1] = a.y, next[k][2] = a.z, next[k][3] = a.w;
      next[k][4] = b.x, next[k][5] = b.y, next[k][6] = b.z, next[k][7] = b.w;
    }
  };
  load(0);
  find_places(p, i0, place);
  __syncthreads();
  for (int base = 0; base < units; base += kThreads * kUnroll) {
    uint32_t w[kUnroll][8];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) w[k][e] = next[k][e];
    load(base + kThreads * kUnroll);
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int c = base + threadIdx.x + k * kThreads;
      if (c - lane >= units) break;                          // the whole warp
      int tok, rest;
      half(c, &tok, &rest);
      const int64_t at = c < units ? place[tok] : kNoToken;
      // largest magnitude by the bits: infinities and NaN compare above every finite value
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = __vmaxu2(m, w[k][e] & 0x7fff7fffu);
      m = max(m & 0xffffu, m >> 16);
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      // A normal fp16 quotient m / Q lies no nearer than 2^-15 of itself to a border of fp16's rounding unless
      // it is a number of fp16, so the product with fl(1 / Q) rounds as the quotient does. A subnormal one can
      // be halfway between two (91 x 2^-25 / 7): there the quotient itself is rounded, which fp32 holds exactly
      // at such a border and on its side beside one (all finite m were compared).
      const float top = __uint_as_float(m << 16) * (1.f / Q);
      __half s = __float2half_rn(top);
      const float sf = __half2float(s);
      uint32_t u[16];
      if (sf >= 6.103515625e-05f && top <= 65504.f) {
        const float r = rcp(sf);
        levels<BITS>(w[k], r, u);
        levels<BITS>(w[k] + 4, r, u + 8);
      } else {
        const bool odd = m >= 0x7f80u;                       // a group with an infinity or NaN
        s = odd ? __ushort_as_half(0x7e00)
                : __float2half_rn(fminf(__fdiv_rn(__uint_as_float(m << 16), Q), 65504.f));
        const float cs = odd ? 0.f : __half2float(s);
        levels_clamped<BITS>(w[k], cs, u);
        levels_clamped<BITS>(w[k] + 4, cs, u + 8);
      }
      // the row's bytes meet in shared memory and leave in order, 8 or 16 a lane (stored from where they
      // are made, in pieces of 4 and 2, they took 2.2 times as long)
      uint32_t* mine = stage[threadIdx.x / 32][lane / L];
      if (BITS == 8) {
#pragma unroll
        for (int r = 0; r < 4; ++r) mine[(2 * h + r + (r & 2)) * NG + g] = low_bytes(u + 4 * r);
      } else {
        // two runs a word: nibbles e of bytes [u0 u2 u4 u6] and [u1 u3 u5 u7]
        uint32_t v[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t a = low_bytes(u + 8 * r), b = low_bytes(u + 8 * r + 4);
          v[r] = __byte_perm(a, b, 0x6420) + (__byte_perm(a, b, 0x7531) << 4);
        }
        // a stored word holds one run of an even group and of the next: the lanes of the two (two
        // apart) exchange two runs, and the even one has runs 2h, 2h + 1, the odd one 4 + 2h, 5 + 2h
        const bool odd_g = g & 1;
        const uint32_t other = __shfl_xor_sync(0xffffffffu, odd_g ? v[0] : v[1], 2);
        const uint32_t lo = odd_g ? other : v[0], hi = odd_g ? v[1] : other;
        uint32_t* to = mine + (2 * h + (odd_g ? 4 : 0)) * (NG / 2) + g / 2;
        to[0] = __byte_perm(lo, hi, 0x5410);
        to[NG / 2] = __byte_perm(lo, hi, 0x7632);
      }
      if (h == 0) reinterpret_cast<__half*>(mine + RW)[g] = s;
      __syncwarp();
      if (at >= 0) {
        // pool row: at + head * page_size
        const int64_t row = at + (uint32_t)(rest / L) * (uint64_t)p.pages.page_size;
        uint8_t* to = p.codes + row * (RW * 4);
        if (BITS == 4)
          reinterpret_cast<uint2*>(to)[l] = reinterpret_cast<const uint2*>(mine)[l];
        else
          reinterpret_cast<uint4*>(to)[l] = reinterpret_cast<const uint4*>(mine)[l];
        if (l < NG / 2) reinterpret_cast<uint32_t*>(p.scales + row * NG)[l] = mine[RW + l];
      }
      __syncwarp();
    }
  }
}

// Byte e of w as c s = (32768 + offset + c) s - (32768 + offset) s: the fp32 number 0x47000000 | u << 8 is
// 32768 + u, the second product is exact (24 bits), so the sum is c s exactly.
__device__ __forceinline__ float level_value(uint32_t w, int e, float s, float minus) {
  return __fmaf_rn(__uint_as_float(__byte_perm(w, 0x47000000u, 0x7604 | e << 4)), s, minus);
}

template <int D, int BITS>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const CacheIoParams p) {
  constexpr int L = D / 16, NG = D / kQuantGroup, W = BITS / 2;      // words of codes a lane
  __shared__ int64_t place[kMaxTokens];
  const int64_t i0 = (int64_t)blockIdx.x * p.tokens;
  const int units = p.tokens * p.per;
  const int lane = threadIdx.x & 31, l = threadIdx.x % L, g = l >> 1, h = l & 1;
  const bool odd_g = g & 1;
  find_places(p, i0, place);
  __syncthreads();
  __nv_bfloat16* out0 = p.out + i0 * (int64_t)p.per * 16;
  for (int base = 0; base < units; base += kThreads * kReadUnroll) {
    uint32_t w[kReadUnroll][W];
    uint16_t sb[kReadUnroll];
    int64_t at[kReadUnroll];
#pragma unroll
    for (int k = 0; k < kReadUnroll; ++k) {
      const int c = base + threadIdx.x + k * kThreads;
      const int tok = p.tokens == 1 ? 0 : (int)__umulhi((uint32_t)c, p.per_inv);
      at[k] = c < units ? place[tok] : kNoToken;
      const int64_t row = at[k] + (uint32_t)((c - tok * p.per) / L) * (uint64_t)p.pages.page_size;
#pragma unroll
      for (int r = 0; r < W; ++r) w[k][r] = 0;
      sb[k] = 0;
      if (at[k] >= 0) {
        // 4 bits: the words of runs 2h, 2h + 1 (even group) or 4 + 2h, 5 + 2h; 8 bits: all four
        const uint32_t* src = reinterpret_cast<const uint32_t*>(p.pages.codes + row * (D * BITS / 8)) +
                              (BITS == 4 ? (2 * h + (odd_g ? 4 : 0)) * (NG / 2) + g / 2 : 2 * h * NG + g);
#pragma unroll
        for (int r = 0; r < W; ++r) w[k][r] = __ldg(src + (BITS == 4 ? r * (NG / 2) : (r + (r & 2)) * NG));
        sb[k] = __ldg(reinterpret_cast<const uint16_t*>(p.pages.scales) + row * NG + g);
      }
    }
#pragma unroll
    for (int k = 0; k < kReadUnroll; ++k) {
      const int c = base + threadIdx.x + k * kThreads;
      if (c - lane >= units) break;                          // the whole warp
      const float s = __half2float(__ushort_as_half(sb[k]));
      const float minus = -(BITS == 4 ? 32776.f : 32896.f) * s;
      uint32_t o[8];
      if (BITS == 4) {
        const uint32_t mine = __byte_perm(w[k][0], w[k][1], odd_g ? 0x7632 : 0x5410);
        const uint32_t give = __byte_perm(w[k][0], w[k][1], odd_g ? 0x5410 : 0x7632);
        const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 2);
        const uint32_t runs[2] = {odd_g ? got : mine, odd_g ? mine : got};
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t a = runs[r] & 0x0f0f0f0fu, b = (runs[r] >> 4) & 0x0f0f0f0fu;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            o[4 * r + e] = pack_bf16(level_value(a, e, s, minus), level_value(b, e, s, minus));
        }
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            o[2 * r + e] = pack_bf16(level_value(w[k][r % W], 2 * e, s, minus),
                                     level_value(w[k][r % W], 2 * e + 1, s, minus));
      }
      if (at[k] != kNoToken) {                               // rows behind the last sequence stay
        uint4* dst = reinterpret_cast<uint4*>(out0 + 16 * (int64_t)c - 8 * h);
        const bool ok = at[k] >= 0;
        __stcs(dst, ok ? make_uint4(o[0], o[1], o[2], o[3]) : make_uint4(0, 0, 0, 0));
        __stcs(dst + 2, ok ? make_uint4(o[4], o[5], o[6], o[7]) : make_uint4(0, 0, 0, 0));
      }
    }
  }
}

int cache_io_check(const void* rows, const int32_t* cu, const int32_t* starts, int num_seqs,
                   int64_t n) {
  if ((n != 0 && !rows) || !cu || !starts) return set_error(IAMAP_ERR_INVALID_ARG, "null pointer");
  if (num_seqs < 1 || n < 0 || n > 0x7fffffff)
    return set_error(IAMAP_ERR_INVALID_ARG, "need num_seqs >= 1 and 0 <= n < 2^31");
  if ((reinterpret_cast<uintptr_t>(rows) & 15u) != 0)
    return set_error(IAMAP_ERR_INVALID_ARG, "the bf16 rows must be 16-byte aligned");
  return IAMAP_OK;
}

// Rows a CTA: up to eight rounds of its threads, so that the places' latency is met once for many rows,
// but no more than leave six CTAs an SM.
int cache_io_shape(int64_t n, int H, int d, CacheIoParams* p, unsigned int* blocks) {
  const int64_t per = (int64_t)H * (d / 16);
  if (per > 0x7fffffff / 2) return set_error(IAMAP_ERR_UNSUPPORTED, "too many heads");
  p->per = (int)per;
  const int64_t most = std::min<int64_t>(kMaxTokens, 4096 / per), spread = (n + kSms * 6 - 1) / (kSms * 6);
  p->tokens = (int)std::max<int64_t>(1, std::min(most, spread));
  p->per_inv = (uint32_t)(((1ull << 32) + per - 1) / per);   // exact: used for numbers below 2^13 only
  *blocks = (unsigned int)((n + p->tokens - 1) / p->tokens);
  return IAMAP_OK;
}

}  // namespace

int check_quant_pages(const void* codes, const void* scales, int64_t num_pages,
                      const int32_t* page_table, int max_pages, int page_size, int H, int d,
                      int bits) {
  if (bits != 4 && bits != 8)
    return set_error(IAMAP_ERR_UNSUPPORTED, "a cache holds 4 or 8 bits an element, not %d", bits);
  if (d != 64 && d != 128) return set_error(IAMAP_ERR_UNSUPPORTED, "head dim must be 64 or 128");
  // an empty page table has no address
  if (!codes || !scales || (!page_table && max_pages != 0)) return set_error(IAMAP_ERR_INVALID_ARG, "null pointer");
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
  if (max_ctx > kMaxCtx) return set_error(IAMAP_ERR_UNSUPPORTED, "max_ctx must be at most 2^30");
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
  CacheIoParams p{};
  unsigned int blocks = 0;
  rc = cache_io_shape(n, H, d, &p, &blocks);
  if (rc) return rc;
  if (blocks == 0) return IAMAP_OK;
  DeviceContext* ctx = device_context();
  if (!ctx) return IAMAP_ERR_CUDA;
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.x_stride = x_stride;
  p.n = n;
  p.cu = cu;
  p.starts = starts;
  p.num_seqs = num_seqs;
  p.codes = static_cast<uint8_t*>(codes);
  p.scales = static_cast<__half*>(scales);
  p.pages = QuantPages{p.codes, p.scales, num_pages, page_table, max_pages, page_size, H};
  p.status = ctx->status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (d == 64) {
    if (bits == 4) cache_write_kernel<64, 4><<<blocks, kThreads, 0, st>>>(p);
    else cache_write_kernel<64, 8><<<blocks, kThreads, 0, st>>>(p);
  } else {
    if (bits == 4) cache_write_kernel<128, 4><<<blocks, kThreads, 0, st>>>(p);
    else cache_write_kernel<128, 8><<<blocks, kThreads, 0, st>>>(p);
  }
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
  CacheIoParams p{};
  unsigned int blocks = 0;
  rc = cache_io_shape(n, H, d, &p, &blocks);
  if (rc) return rc;
  if (blocks == 0) return IAMAP_OK;
  DeviceContext* ctx = device_context();
  if (!ctx) return IAMAP_ERR_CUDA;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.n = n;
  p.cu = cu;
  p.starts = starts;
  p.num_seqs = num_seqs;
  p.pages = QuantPages{static_cast<const uint8_t*>(codes), static_cast<const __half*>(scales),
                       num_pages, page_table, max_pages, page_size, H};
  p.status = ctx->status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (d == 64) {
    if (bits == 4) cache_read_kernel<64, 4><<<blocks, kThreads, 0, st>>>(p);
    else cache_read_kernel<64, 8><<<blocks, kThreads, 0, st>>>(p);
  } else {
    if (bits == 4) cache_read_kernel<128, 4><<<blocks, kThreads, 0, st>>>(p);
    else cache_read_kernel<128, 8><<<blocks, kThreads, 0, st>>>(p);
  }
  IAMAP_LAUNCH_CHECK("cache_read_kernel");
  return IAMAP_OK;
}
