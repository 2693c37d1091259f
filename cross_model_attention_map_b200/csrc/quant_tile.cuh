// Tiles of a quantised paged cache as matrix-instruction operands.
//
// Decode over a 4- or 8-bit cache moves few bytes an element, so what a warp may spend on one is
// small: at the HBM rate an SM receives some 40 four-bit elements a clock, and its four schedulers
// issue 128 lane instructions. The tiles are therefore laid out so that codes go from shared memory to
// the operands of mma.sync.m16n8k16 with about 1.2 instructions an element and no shuffles:
//
//   keys    S^T [16 tokens x 8 heads] = K^ [tokens x d] . q^T. Lane (gid = lane / 4, tid = lane % 4)
//           holds rows gid and gid + 8; the order of d inside a product is free, so the lane takes
//           runs 2 tid and 2 tid + 1 of every group, one contiguous load, and q's operand is gathered
//           in the same order once. A group's two k-steps accumulate the codes' products alone; its
//           scale multiplies the fp32 sums.
//   values  O^T [d x 8 columns] += V^T [d x 16 tokens] . P. The lane owns run gid of every group (four
//           elements) of four tokens; a byte permutation pairs two tokens, and the columns P carry the
//           weight times the scale.
//
// Codes become fp16 exactly by the widely published conversion that writes a small integer into the
// mantissa of a number whose last bit counts 1: 1024 + u is the fp16 number 0x6400 | u, from which
// 1024 + offset is taken (for nibbles in the upper half of a byte 1024 + 16 u, one fused multiply-add).
//
// Row r of a 16-token tile is token (r & 8) + ((r & 7) >> 1) + 4 (r & 1): the two tokens of a pair of
// columns 2 tid, 2 tid + 1 of P are then tokens tid and tid + 4 (+ 8), so that the lanes of one load of
// values read neighbouring rows. A tile lies in shared memory as in the pool, token after token, so one
// bulk copy brings it where pages are multiples of 16 tokens; its loads have at worst two- (4 bits) or
// four-way (values of 8 bits) bank conflicts, less than placing 16-byte pieces by address costs in
// instructions.
#pragma once

#include "quant_cache.cuh"
#include "tc_utils.cuh"

namespace iamap {
namespace qt {

constexpr uint32_t kNoRow = 0xffffffffu;
constexpr int kTok = 16;                       // tokens a tile

constexpr int kPair = 2 * kTok;                // tokens of one mask

// Loads from shared addresses. Plain loads, not asm: the compiler may move them among the matrix
// instructions, but not across the waits.
template <typename T>
__device__ __forceinline__ T lds(uint32_t a) {
  return *static_cast<const T*>(__cvta_shared_to_generic(a));
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) { return lds<uint16_t>(a); }
__device__ __forceinline__ uint32_t lds32(uint32_t a) { return lds<uint32_t>(a); }
__device__ __forceinline__ uint2 lds64(uint32_t a) { return lds<uint2>(a); }
__device__ __forceinline__ uint4 lds128(uint32_t a) { return lds<uint4>(a); }

// cp.async of N (4, 8 or 16) bytes; zeros where !valid.
template <int N>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? N : 0;
  if (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(n));
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;\n" ::"r"(dst), "l"(src), "n"(N),
                 "r"(n));
}

__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// (a & mask) | 0x64006400
template <uint32_t MASK>
__device__ __forceinline__ uint32_t magic(uint32_t a) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(a), "n"(MASK), "r"(0x64006400u));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t h) {
  const __half2 v = *reinterpret_cast<const __half2*>(&h);
  return __half22float2(v);
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// D = A (16 x 16 fp16, row) . B (16 x 8 fp16, col) + D in fp32. Volatile, as every instruction here that
// takes the whole warp: the compiler may otherwise copy it into branches that only some lanes take.
__device__ __forceinline__ void mma_f16(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// D = A . B
__device__ __forceinline__ void mma_f16_first(float* d, uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// The eight codes of a word of nibbles as fp16 pairs: r[i] = (nibble i, nibble 4 + i) - 8.
__device__ __forceinline__ void nibbles(uint32_t w, uint32_t* r) {
  constexpr uint32_t kSixteenth = 0x2c002c00u, kMinus72 = 0xd480d480u, k1032 = 0x64086408u;
  r[0] = hsub2(magic<0x000f000fu>(w), k1032);
  r[1] = hfma2(magic<0x00f000f0u>(w), kSixteenth, kMinus72);
  w >>= 8;
  r[2] = hsub2(magic<0x000f000fu>(w), k1032);
  r[3] = hfma2(magic<0x00f000f0u>(w), kSixteenth, kMinus72);
}
// Bytes (i, j) of a word as an fp16 pair, - 128. SEL is 0x4j4i.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t byte_pair(uint32_t w) {
  return hsub2(__byte_perm(w, 0x64646464u, SEL), 0x64806480u);
}

// The four groups' (two for d = 64) scales of a token, unpaired.
template <int NG>
__device__ __forceinline__ uint2 lds_scales(uint32_t a) {
  if (NG == 4) return lds64(a);
  return make_uint2(lds32(a), 0u);
}

// A query head's operand order: element of pair p (0..3), half e of lane tid's eight elements of a group.
template <int BITS>
__device__ __forceinline__ int q_elem(int p, int e) {
  return BITS == 4 ? p + 4 * e : 2 * p + e;
}

// The query operand of up to eight heads q[h * D], h < nh (the other columns are zero): head gid,
// elements 8 tid .. 8 tid + 7 of every group. A head's largest element is brought to [2^14, 2^15) by a
// power of two, so that bf16 values of any size are exact in fp16 down to 2^-31 of it (less is rounded, by
// at most 2^-39 of it); fq[c] takes the scores of columns 2 tid + c back, times `scale`.
template <int D, int BITS>
__device__ __forceinline__ void load_query(const __nv_bfloat16* q, int nh, float scale,
                                           uint32_t (*qf)[4], float* fq) {
  constexpr int NG = D / 32;
  const int lane = threadIdx.x & 31, gid = lane >> 2, tid = lane & 3;
  const bool live = gid < nh;
  uint4 raw[NG];
  uint32_t m = 0;
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    raw[g] = live ? *reinterpret_cast<const uint4*>(q + gid * D + 32 * g + 8 * tid)
                  : make_uint4(0, 0, 0, 0);
    const uint32_t w[4] = {raw[g].x, raw[g].y, raw[g].z, raw[g].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) m = max(m, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
  }
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const int down = min(253, max(1, 268 - (int)(m >> 7)));          // exponent field of the power of two
  const float f = __uint_as_float((uint32_t)down << 23);
  const float back = __uint_as_float((uint32_t)(254 - down) << 23) * scale;
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const uint32_t w[4] = {raw[g].x, raw[g].y, raw[g].z, raw[g].w};
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[e] = __uint_as_float(e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16) * f;
#pragma unroll
    for (int i = 0; i < 4; ++i) qf[g][i] = pack_f16(v[q_elem<BITS>(i, 0)], v[q_elem<BITS>(i, 1)]);
  }
  fq[0] = __shfl_sync(0xffffffffu, back, 8 * tid);
  fq[1] = __shfl_sync(0xffffffffu, back, 8 * tid + 4);
}

// Scores of a tile: s[0..1] = row gid, s[2..3] = row gid + 8, columns 2 tid and 2 tid + 1, in the
// units of the fp16 query operand qf[group][4]. `codes` and `scales` are the tile's addresses.
template <int D, int BITS>
__device__ __forceinline__ void tile_scores(uint32_t codes, uint32_t scales, const uint32_t (*qf)[4],
                                            float* s) {
  constexpr int NG = D / 32, R = D * BITS / 8;
  const int lane = threadIdx.x & 31, gid = lane >> 2, tid = lane & 3;
  const int t0 = (gid >> 1) + 4 * (gid & 1);
  uint32_t w[2][R / 16];                       // row gid, gid + 8: runs 2 tid and 2 tid + 1
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int t = t0 + 8 * h;
    const uint32_t at = codes + t * R + tid * (R / 4);
    if (R == 128) {
      const uint4 a = lds128(at), b = lds128(at + 16);
      w[h][0] = a.x, w[h][1] = a.y, w[h][2 % (R / 16)] = a.z, w[h][3 % (R / 16)] = a.w;
      w[h][4 % (R / 16)] = b.x, w[h][5 % (R / 16)] = b.y, w[h][6 % (R / 16)] = b.z,
      w[h][7 % (R / 16)] = b.w;
    } else if (R == 64) {
      const uint4 a = lds128(at);
      w[h][0] = a.x, w[h][1] = a.y, w[h][2 % (R / 16)] = a.z, w[h][3 % (R / 16)] = a.w;
    } else {
      const uint2 a = lds64(at);
      w[h][0] = a.x, w[h][1] = a.y;
    }
  }
  const uint2 sc0 = lds_scales<NG>(scales + t0 * (2 * NG));
  const uint2 sc1 = lds_scales<NG>(scales + (t0 + 8) * (2 * NG));
  s[0] = s[1] = s[2] = s[3] = 0.f;
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    uint32_t a[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (BITS == 4) {
        nibbles(__byte_perm(w[h][g >> 1], w[h][NG / 2 + (g >> 1)], g & 1 ? 0x7632 : 0x5410), a[h]);
      } else {
        a[h][0] = byte_pair<0x4140>(w[h][g]);
        a[h][1] = byte_pair<0x4342>(w[h][g]);
        a[h][2] = byte_pair<0x4140>(w[h][(NG + g) % (R / 16)]);
        a[h][3] = byte_pair<0x4342>(w[h][(NG + g) % (R / 16)]);
      }
    }
    float c[4];
    mma_f16_first(c, a[0][0], a[1][0], a[0][1], a[1][1], qf[g][0], qf[g][1]);
    mma_f16(c, a[0][2], a[1][2], a[0][3], a[1][3], qf[g][2], qf[g][3]);
    const float2 f0 = unpack_f16(g < 2 ? sc0.x : sc0.y), f1 = unpack_f16(g < 2 ? sc1.x : sc1.y);
    const float s0 = g & 1 ? f0.y : f0.x, s1 = g & 1 ? f1.y : f1.x;
    s[0] = fmaf(c[0], s0, s[0]);
    s[1] = fmaf(c[1], s0, s[1]);
    s[2] = fmaf(c[2], s1, s[2]);
    s[3] = fmaf(c[3], s1, s[3]);
  }
}

// The lane's part of a tile of values: run gid of every group, tokens tid, tid + 4, tid + 8, tid + 12.
template <int D, int BITS>
struct ValueTile {
  static constexpr int NG = D / 32, R = D * BITS / 8, N = R / 32;
  uint32_t w[4][N];
  __device__ __forceinline__ void load(uint32_t codes) {
    const int lane = threadIdx.x & 31, gid = lane >> 2, tid = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t at = codes + (tid + 4 * i) * R + gid * (R / 8);
      if (R == 128) {
        const uint4 a = lds128(at);
        w[i][0] = a.x, w[i][1 % N] = a.y, w[i][2 % N] = a.z, w[i][3 % N] = a.w;
      } else if (R == 64) {
        const uint2 a = lds64(at);
        w[i][0] = a.x, w[i][1 % N] = a.y;
      } else {
        w[i][0] = lds32(at);
      }
    }
  }
  // Operands of group g: r[i] = element i of the run, tokens (tid, tid + 4); t[i]: (tid + 8, tid + 12).
  __device__ __forceinline__ void group(int g, uint32_t* r, uint32_t* t) const {
    if (BITS == 4) {
      const uint32_t sel = g & 1 ? 0x7632 : 0x5410;
      nibbles(__byte_perm(w[0][(g >> 1) % N], w[1][(g >> 1) % N], sel), r);
      nibbles(__byte_perm(w[2][(g >> 1) % N], w[3][(g >> 1) % N], sel), t);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t* o = h ? t : r;
        const uint32_t lo = __byte_perm(w[2 * h][g % N], w[2 * h + 1][g % N], 0x5140);
        const uint32_t hi = __byte_perm(w[2 * h][g % N], w[2 * h + 1][g % N], 0x7362);
        o[0] = byte_pair<0x4140>(lo);
        o[1] = byte_pair<0x4342>(lo);
        o[2] = byte_pair<0x4140>(hi);
        o[3] = byte_pair<0x4342>(hi);
      }
    }
  }
};

// Scales of group g for the token pairs of a P column: (tid, tid + 4) from sc[0], sc[1], and
// (tid + 8, tid + 12) from sc[2], sc[3].
__device__ __forceinline__ uint32_t scale_pair(const uint2* sc, int g) {
  const uint32_t sel = g & 1 ? 0x7632 : 0x5410;
  return g < 2 ? __byte_perm(sc[0].x, sc[1].x, sel) : __byte_perm(sc[0].y, sc[1].y, sel);
}

// Two fp32 numbers in a register pair, and their products.
__device__ __forceinline__ uint64_t pair_f32(float x, float y) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
  return d;
}
__device__ __forceinline__ float2 unpair_f32(uint64_t a) {
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(a));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// a * b + c of fp16 numbers a and b, in fp32.
__device__ __forceinline__ float fma_f16(uint16_t a, uint16_t b, float c) {
  float d;
  asm("fma.rn.f32.f16 %0, %1, %2, %3;" : "=f"(d) : "h"(a), "h"(b), "f"(c));
  return d;
}
// A pair t of fp32 numbers as fp16 pairs: t = high + low 2^-12. A |t| under 2^15 leaves at most 2^3 to the low
// part, and what is below fp16's range in the high one is not lost: the error is at most 2^-22 |t|, or 2^-37.
constexpr float kLow = 1.f / 4096.f;
__device__ __forceinline__ void split_f16(uint64_t t, uint32_t& high, uint32_t& low) {
  const float2 x = unpair_f32(t), y = unpair_f32(mul2(t, pair_f32(4096.f, 4096.f)));
  high = pack_f16(x.x, x.y);
  low = pack_f16(fma_f16((uint16_t)high, 0xec00, y.x), fma_f16((uint16_t)(high >> 16), 0xec00, y.y));
}

// Exact 2^k for k in [-126, 127], clamped to it; larger shifts are made in two steps by the caller.
__device__ __forceinline__ float pow2i(int k) {
  return __uint_as_float((uint32_t)(min(max(k, -126), 127) + 127) << 23);
}

// A power of two for each group of a warp's value scales. The groups are elements that share nothing but
// their tokens, so a large group may not cost a small one its bits: group g's scales are taken times 2^-e[g],
// under 2. e serves the largest scale S so far and only rises, so a group's sums are rescaled a few times at
// most. CLOSE: e brings S to [1/2, 1), beyond 2^15 and under 2^-16 as near as fp16 has the power, and serves
// scales up to 4 S. Otherwise the same below 2^-8, 0 for S in [2^-8, 2), where nothing needs to be multiplied, and
// above it S is brought to [1, 2).
template <int NG, bool CLOSE>
struct ScalePowers {
  uint32_t held;                   // e[g] in byte g
  uint32_t limit[NG / 2];          // pairs of 0x8000 | the largest scale that e serves (0 before the first)
  __device__ __forceinline__ void init() {
    held = 0;
#pragma unroll
    for (int i = 0; i < NG / 2; ++i) limit[i] = 0x80008000u;
  }
  __device__ __forceinline__ int e(int g) const { return (int)(held << (24 - 8 * g)) >> 24; }
  __device__ __forceinline__ bool any() const { return held != 0; }
  // 2^-e of group g in fp16, exact: e is in [-15, 15].
  __device__ __forceinline__ uint32_t half(int g) const { return e(g) == 15 ? 0x200u : (uint32_t)(15 - e(g)) << 10; }
  // Bits 15 and 31 are set where word w of a token's scales (word i: groups 2 i and 2 i + 1) is served. Words of
  // tokens that do not exist hold anything: they may ask for a look at the scales, which skips them.
  __device__ __forceinline__ uint32_t served(uint32_t w, int i) const { return limit[i % (NG / 2)] - w; }
  // Larger of m and the word's finite scales: infinities and NaN set no power.
  static __device__ __forceinline__ uint32_t larger(uint32_t m, uint32_t w) {
    const uint32_t v = w & 0x7fff7fffu;
    return __vmaxu2(m, v & ~__vcmpgtu2(v, 0x7bff7bffu));
  }
  // Takes the lanes' maxima m into the powers (the whole warp); f[g] is what group g's sums are to be
  // multiplied by.
  __device__ __forceinline__ void raise(uint32_t* m, float* f) {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const int up = 16 * (g & 1), top = (int)__reduce_max_sync(0xffffffffu, m[g >> 1] >> up & 0xffffu);
      f[g] = 1.f;
      if (top <= (int)(limit[g >> 1] >> up & 0x7fffu)) continue;
      const int k = top >= 0x400 ? (top >> 10) - 15 : 7 - __clz(top);      // floor(log2)
      const int to = CLOSE || k < -8 ? min(max(k + 1, -15), 15) : max(k, 0);
      const int most = to < 15 ? ((to + 16) << 10) - 1 : 0x7bff;
      f[g] = pow2i(e(g) - to);
      held = (held & ~(0xffu << 8 * g)) | ((uint32_t)to & 0xffu) << 8 * g;
      limit[g >> 1] = (limit[g >> 1] & (0xffff0000u >> up)) | (0x8000u | most) << up;
    }
  }
};

// ------------------------------------------------------------------------------------------------
// A warp's stream of tokens
// ------------------------------------------------------------------------------------------------

// Row of the pools that holds a token of one (sequence, head), or kNoRow: past `end`, or on a bad page
// (which is reported).
struct QuantRow {
  const QuantPages* p;
  const int32_t* table;            // of the sequence
  int head, end;
  __device__ __forceinline__ uint32_t at(int pos, unsigned int* status) const {
    if (pos >= end) return kNoRow;
    const int pi = pos / p->page_size;
    const int page = __ldg(table + pi);
    if (page < 0 || page >= p->num_pages) {
      raise_status(status, IAMAP_DEV_BAD_INDEX);
      return kNoRow;
    }
    return (uint32_t)(((int64_t)page * p->H + head) * p->page_size + (pos - pi * p->page_size));
  }
};

// The barriers and masks of one warp's ring, and its abort flag.
template <int TILES, int STAGES>
struct StreamShared {
  uint64_t full[STAGES];
  uint32_t mask[STAGES][TILES / 2];      // which of 32 tokens exist
  int abort_flag;
};

// Brings the tokens of one (sequence, head), TILES tiles at a time, into a ring of stages in shared
// memory that belongs to one warp, so that warps run apart (a ring shared by the CTA's warps, filled in
// turns, was slower: 198 against 165 us in attention at 48 sequences of up to 16384). Up to ARRAYS pools
// with the same rows are brought together (keys' codes, their scales, ...), one after the other in a
// stage. More tiles a step spread its bookkeeping.
//
// ALIGNED (page_size a multiple of 16): a tile of 16 tokens is one run of memory in each pool, and lane
// a + ARRAYS * tile starts one bulk copy; completion is counted on the stage's mbarrier. Tokens past the
// end of the range come with their tile and hold anything: what uses them masks them. Otherwise every
// row is copied by itself in pieces of 16 (codes) or 4 or 8 (scales) bytes, and tokens that do not exist
// are zeros.
//
// A further array without pages may come with them: `extra_bytes` a step from one run of memory, after the
// others in the stage.
//
// Page indices: ALIGNED, lane l looks up tile l of the next 32; otherwise lane l looks up token l of
// each 32 of a step.
template <bool ALIGNED, int TILES, int ARRAYS, int STAGES>
struct Stream {
  static_assert(TILES * ARRAYS < 32 && TILES % 2 == 0 && 32 % TILES == 0, "one bulk copy a lane");
  static constexpr int kTokens = TILES * kTok;
  QuantRow rows;
  unsigned int* status;
  StreamShared<TILES, STAGES>* sh;
  int first, step, nsteps;
  uint32_t held, good;             // row of a tile, and which of the 32 tiles have one
  uint32_t ring, stage_bytes, tile_bytes;
  int s_in, s_out;                 // next stage to fill and to use
  uint32_t parity;
  // this lane's copy (ALIGNED): lanes below TILES * ARRAYS
  const uint8_t* src;
  uint32_t mul, dst;
  // all arrays (otherwise)
  const uint8_t* pool[ARRAYS];
  uint32_t row_bytes[ARRAYS];
  const uint8_t* extra;            // step i's: extra + i * extra_step
  uint32_t extra_bytes, extra_step;

  // Step i is tokens first + i * step .. + kTokens of the sequence, below `end`.
  __device__ __forceinline__ void init(const QuantPages* pages, int seq, int head, int first_,
                                       int step_, int end, unsigned int* st, uint32_t ring_,
                                       StreamShared<TILES, STAGES>* shared) {
    rows = QuantRow{pages, pages->table + (int64_t)seq * pages->max_pages, head, end};
    first = first_, step = step_, status = st, sh = shared, ring = ring_;
    nsteps = end > first ? (end - first + step - 1) / step : 0;
    s_in = s_out = 0, parity = 0, stage_bytes = tile_bytes = 0, good = held = 0;
    src = extra = nullptr, mul = dst = extra_bytes = extra_step = 0;
    const int lane = threadIdx.x & 31;
    if (ALIGNED) {
      if (lane < STAGES) tc::mbar_init(smem_u32(&sh->full[lane]), 1);
      if (lane == 0) sh->abort_flag = 0;
      tc::fence_barrier_init();
    }
    __syncwarp();
  }
  // Array A: its pool and the bytes of one row. Arrays are added in order 0, 1, ...
  template <int A>
  __device__ __forceinline__ void add(const void* base, uint32_t bytes) {
    const int lane = threadIdx.x & 31;
    if (ALIGNED) {
      if (lane % ARRAYS == A) {
        src = static_cast<const uint8_t*>(base);
        mul = bytes;
        dst = stage_bytes + lane / ARRAYS * kTok * bytes;
      }
    } else {
      pool[A] = static_cast<const uint8_t*>(base);
      row_bytes[A] = bytes;
    }
    stage_bytes += kTokens * bytes;
    tile_bytes += kTok * bytes;
  }

  // The array without pages, after the others (16-byte aligned, multiples of 16 bytes).
  __device__ __forceinline__ void add_extra(const void* base, uint32_t bytes, uint32_t step_bytes) {
    extra = static_cast<const uint8_t*>(base);
    extra_bytes = bytes, extra_step = step_bytes;
    if ((threadIdx.x & 31) == TILES * ARRAYS) dst = stage_bytes;
    stage_bytes += bytes;
  }

  // Starts step i (called for i = 0, 1, ... by the whole warp; nothing past the last step). Steps
  // 0 .. STAGES - 2 are started first; then step i + STAGES - 1 is started before step i is taken, into
  // the stage that step i - 1 left (the warp has met since its last read).
  __device__ __forceinline__ void fill(int i) {
    const int lane = threadIdx.x & 31;
    if (i < nsteps) {
      const uint32_t stage = ring + s_in * stage_bytes;
      if constexpr (ALIGNED) {
        constexpr int kHeld = 32 / TILES;          // steps a lookup serves
        const int k = i % kHeld * TILES;
        if (k == 0) {
          held = rows.at(first + (i + lane / TILES) * step + lane % TILES * kTok, status);
          good = __ballot_sync(0xffffffffu, held != kNoRow);
        }
        const uint32_t row = __shfl_sync(0xffffffffu, held, k + lane / ARRAYS % TILES);
        const uint32_t bar = smem_u32(&sh->full[s_in]);
        const bool linear = lane == TILES * ARRAYS && extra_bytes != 0;
        if ((lane < TILES * ARRAYS && row != kNoRow) || linear)
          asm volatile(
              "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                  stage + dst),
              "l"(linear ? extra + (uint64_t)i * extra_step : src + (uint64_t)row * mul),
              "r"(linear ? extra_bytes : mul * kTok), "r"(bar)
              : "memory");
        const uint32_t g = good >> k & ((1u << TILES) - 1u);
        const int left = rows.end - (first + i * step);
        uint32_t bytes = tile_bytes * TILES;
        if (g != (1u << TILES) - 1u || left < kTokens) {
          bytes = tile_bytes * __popc(g);
          if (lane < TILES / 2) {
            uint32_t m = (g >> (2 * lane) & 1 ? 0xffffu : 0u) | (g >> (2 * lane) & 2 ? 0xffff0000u : 0u);
            const int here = left - lane * kPair;
            if (here < kPair) m &= here <= 0 ? 0u : (1u << here) - 1u;
            sh->mask[s_in][lane] = m;
          }
          __syncwarp();
        } else if (lane < TILES / 2) {
          sh->mask[s_in][lane] = 0xffffffffu;
        }
        // the arrival completes the phase once these bytes have come, before or after it
        if (lane == 0) tc::mbar_expect_tx(bar, bytes + extra_bytes);
        __syncwarp();
      } else {
#pragma unroll 1
        for (int h = 0; h < TILES / 2; ++h) {
          const uint32_t row = rows.at(first + i * step + h * kPair + lane, status);
          uint32_t at = stage;
#pragma unroll
          for (int a = 0; a < ARRAYS; ++a) {
            const uint32_t rb = row_bytes[a], to = at + h * kPair * rb;
            if (rb >= 32) {
              for (uint32_t id = lane; id < 2 * rb; id += 32) {       // kPair * rb / 16 pieces
                const uint32_t t = id * 16 / rb, c = id * 16 - t * rb;
                const uint32_t r = __shfl_sync(0xffffffffu, row, t);
                cp_async<16>(to + id * 16, pool[a] + (r == kNoRow ? 0 : (uint64_t)r * rb + c),
                             r != kNoRow);
              }
            } else if (rb == 8) {
              cp_async<8>(to + lane * 8, pool[a] + (row == kNoRow ? 0 : (uint64_t)row * 8), row != kNoRow);
            } else {
              cp_async<4>(to + lane * 4, pool[a] + (row == kNoRow ? 0 : (uint64_t)row * 4), row != kNoRow);
            }
            at += kTokens * rb;
          }
          const uint32_t m = __ballot_sync(0xffffffffu, row != kNoRow);
          if (lane == 0) sh->mask[s_in][h] = m;
        }
        for (uint32_t at = lane * 16; at < extra_bytes; at += 512)
          cp_async<16>(stage + stage_bytes - extra_bytes + at, extra + (uint64_t)i * extra_step + at, true);
        __syncwarp();
      }
      s_in = s_in + 1 == STAGES ? 0 : s_in + 1;
    }
    if (!ALIGNED) cp_async_commit();
  }

  // Waits for the next step: its stage's address, and where its masks are. False if the wait gave up
  // (IAMAP_DEV_TIMEOUT is set): the stream is over, and its copies in flight have landed or been waited
  // for.
  __device__ __forceinline__ bool take(uint32_t* stage, const uint32_t** mask) {
    if constexpr (ALIGNED) {
      const uint32_t bar = smem_u32(&sh->full[s_out]);
      bool ok = tc::mbar_try_wait(bar, parity);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = ok || tc::wait_bar(bar, parity, &sh->abort_flag, status);
        if (!__all_sync(0xffffffffu, ok)) {
          for (int k = 0; k < STAGES; ++k) {
            tc::drain_bar(smem_u32(&sh->full[s_out]), parity);
            s_out = s_out + 1 == STAGES ? 0 : s_out + 1;
            if (s_out == 0) parity ^= 1;
            if (s_out == s_in) break;
          }
          return false;
        }
      }
    } else {
      cp_async_wait<STAGES - 1>();
      __syncwarp();
    }
    *stage = ring + s_out * stage_bytes;
    *mask = sh->mask[s_out];
    s_out = s_out + 1 == STAGES ? 0 : s_out + 1;
    if (s_out == 0) parity ^= 1;
    return true;
  }
};

}  // namespace qt
}  // namespace iamap
