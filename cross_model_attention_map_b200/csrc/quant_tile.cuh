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
// Codes become fp16 exactly: 1024 + u is the fp16 number 0x6400 | u, from which 1024 + offset is taken
// (for nibbles in the upper half of a byte 1024 + 16 u, one fused multiply-add).
//
// Row r of a 16-token tile is token (r & 8) + ((r & 7) >> 1) + 4 (r & 1): the two tokens of a pair of
// columns 2 tid, 2 tid + 1 of P are then tokens tid and tid + 4 (+ 8), so that lanes of one load read
// neighbouring rows. tile_off() places rows and 16-byte pieces so that both the keys' and the values'
// loads are free of bank conflicts.
#pragma once

#include "quant_cache.cuh"

namespace iamap {
namespace qt {

constexpr uint32_t kNoRow = 0xffffffffu;
constexpr int kTok = 16;                       // tokens a tile

// Byte offset of 16-byte piece c of token t in a tile of R-byte rows.
template <int R>
__device__ __forceinline__ int tile_off(int t, int c) {
  if (R == 128) return t * 128 + ((c ^ (((t & 3) << 1) | ((t >> 2) & 1))) << 4);
  if (R == 64)
    return (t >> 1) * 128 + (((t ^ (t >> 2)) & 1) << 6) + ((c ^ (((t >> 1) & 1) << 1)) << 4);
  return (t ^ (((t >> 2) & 1) << 1)) * 32 + (c << 4);
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}

// Asynchronous copy of N (4, 8 or 16) bytes; zeros where !valid.
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
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// D = A (16 x 16 fp16, row) . B (16 x 8 fp16, col) + D in fp32.
__device__ __forceinline__ void mma_f16(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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
// elements 8 tid .. 8 tid + 7 of every group. A head is brought near 2^7 by a power of two, so that bf16
// values of any size are exact in fp16 (what is 2^-21 of the largest or less is rounded); fq[c] takes the
// scores of columns 2 tid + c back, times `scale`.
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
  const int down = min(253, max(1, 261 - (int)(m >> 7)));          // exponent field of the power of two
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
    if (R == 128) {
      const uint4 a = lds128(codes + tile_off<R>(t, 2 * tid));
      const uint4 b = lds128(codes + tile_off<R>(t, 2 * tid + 1));
      w[h][0] = a.x, w[h][1] = a.y, w[h][2] = a.z, w[h][3] = a.w;
      w[h][4 % (R / 16)] = b.x, w[h][5 % (R / 16)] = b.y, w[h][6 % (R / 16)] = b.z,
      w[h][7 % (R / 16)] = b.w;
    } else if (R == 64) {
      const uint4 a = lds128(codes + tile_off<R>(t, tid));
      w[h][0] = a.x, w[h][1] = a.y, w[h][2 % (R / 16)] = a.z, w[h][3 % (R / 16)] = a.w;
    } else {
      const uint2 a = lds64(codes + tile_off<R>(t, tid >> 1) + 8 * (tid & 1));
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
    float c[4] = {0.f, 0.f, 0.f, 0.f};
    mma_f16(c, a[0][0], a[1][0], a[0][1], a[1][1], qf[g][0], qf[g][1]);
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
      const int t = tid + 4 * i;
      if (R == 128) {
        const uint4 a = lds128(codes + tile_off<R>(t, gid));
        w[i][0] = a.x, w[i][1 % N] = a.y, w[i][2 % N] = a.z, w[i][3 % N] = a.w;
      } else if (R == 64) {
        const uint2 a = lds64(codes + tile_off<R>(t, gid >> 1) + 8 * (gid & 1));
        w[i][0] = a.x, w[i][1 % N] = a.y;
      } else {
        w[i][0] = lds32(codes + tile_off<R>(t, gid >> 2) + 4 * (gid & 3));
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

// ------------------------------------------------------------------------------------------------
// Where a tile's rows lie, and their copies
// ------------------------------------------------------------------------------------------------

// A 16-token tile's rows in the pools: ALIGNED (page_size a multiple of 16), the first of 16
// consecutive rows, the same in every lane; otherwise the row of token lane % 16. Bit t of mask says
// that token t exists: below the end of the range, on a good page.
struct Tile {
  uint32_t row, mask;
};

// The tiles of one (sequence, head), tokens first + i * step .. of the warp's i-th tile. ALIGNED: lane l
// looks up the page of tile (base + l), 32 tiles at a time; otherwise every token is looked up, one
// tile ahead of its use.
template <bool ALIGNED>
struct TileRows {
  const QuantPages* p;
  const int32_t* table;
  int head, first, step, end;
  uint32_t held;
  int held_at;
  unsigned int* status;

  __device__ __forceinline__ uint32_t look(int pos) const {
    if (pos >= end) return kNoRow;
    const int pi = pos / p->page_size;
    const int page = __ldg(table + pi);
    if (page < 0 || page >= p->num_pages) {
      raise_status(status, IAMAP_DEV_BAD_INDEX);
      return kNoRow;
    }
    return (uint32_t)(((int64_t)page * p->H + head) * p->page_size + (pos - pi * p->page_size));
  }
  __device__ __forceinline__ void init(const QuantPages* pages, int seq, int head_, int first_,
                                       int step_, int end_, unsigned int* st) {
    p = pages;
    table = pages->table + (int64_t)seq * pages->max_pages;
    head = head_, first = first_, step = step_, end = end_, status = st;
    held_at = 0;
    const int lane = threadIdx.x & 31;
    held = ALIGNED ? look(first + lane * step) : look(first + (lane & 15));
  }
  // Must be called with i = 0, 1, 2, ... by the whole warp.
  __device__ __forceinline__ Tile tile(int i) {
    const int lane = threadIdx.x & 31;
    Tile t;
    if (ALIGNED) {
      if (i - held_at == 32) {
        held_at = i;
        held = look(first + (i + lane) * step);
      }
      t.row = __shfl_sync(0xffffffffu, held, i - held_at);
      const int left = end - (first + i * step);
      t.mask = t.row == kNoRow ? 0u : left >= kTok ? 0xffffu : (1u << left) - 1u;
    } else {
      t.row = held;
      t.mask = __ballot_sync(0xffffffffu, held != kNoRow) & 0xffffu;
      held = look(first + (i + 1) * step + (lane & 15));
    }
    return t;
  }
};

// Starts the copy of a tile's codes. `base` is the pool's codes plus 16 * lane where ALIGNED: a tile is
// then one contiguous run, and 16-byte pieces lane, lane + 32, .. of it go to their places.
template <int D, int BITS, bool ALIGNED>
__device__ __forceinline__ const uint8_t* codes_base(const uint8_t* codes) {
  return ALIGNED ? codes + 16 * (threadIdx.x & 31) : codes;
}
template <int D, int BITS, bool ALIGNED>
__device__ __forceinline__ void load_codes(uint32_t dst, const uint8_t* base, Tile tl) {
  constexpr int R = D * BITS / 8, PER = R / 16, N = PER * kTok / 32;     // pieces a row, a lane
  const int lane = threadIdx.x & 31;
  if constexpr (ALIGNED) {
    const uint8_t* src = base + (uint64_t)tl.row * R;
    if (tl.mask == 0xffffu) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int id = i * 32 + lane;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(
                         dst + tile_off<R>(id / PER, id % PER)),
                     "l"(src + 512 * i));
      }
      return;
    }
    if (tl.mask == 0) src = base;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int id = i * 32 + lane;
      cp_async<16>(dst + tile_off<R>(id / PER, id % PER), src + 512 * i, (tl.mask >> (id / PER)) & 1);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int id = i * 32 + lane, t = id / PER, c = id % PER;
      const uint32_t r = __shfl_sync(0xffffffffu, tl.row, t);
      cp_async<16>(dst + tile_off<R>(t, c), base + (r == kNoRow ? 0 : (uint64_t)r * R + c * 16),
                   r != kNoRow);
    }
  }
}

// Starts the copy of a tile's scales by lanes first .. first + 15 (`lane16` is the lane's place among
// them; the other lanes pass a place of 16 or more).
template <int D, bool ALIGNED>
__device__ __forceinline__ void load_scales(uint32_t dst, const __half* scales, Tile tl, int lane16) {
  constexpr int B = D / 32 * 2;
  const uint8_t* src = reinterpret_cast<const uint8_t*>(scales);
  if (ALIGNED && tl.mask == 0xffffu) {
    if (lane16 < B)                            // 16 rows of B bytes are B pieces of 16
      cp_async<16>(dst + lane16 * 16, src + (uint64_t)tl.row * B + lane16 * 16, true);
    return;
  }
  if (lane16 < kTok) {
    const bool ok = (tl.mask >> lane16) & 1;
    const uint32_t row = ALIGNED ? tl.row + lane16 : tl.row;
    cp_async<B>(dst + lane16 * B, src + (ok ? (uint64_t)row * B : 0), ok);
  }
}

}  // namespace qt
}  // namespace iamap
