// The quantised paged cache: its format, device helpers and the argument checks shared by the entry
// points that write and read it.
//
// A (token, head) row of d elements is d / 32 groups. A group is stored as integer codes c in
// [-Q, Q] (Q = 7 in 4 bits, 127 in 8) and one fp16 scale s, and stands for c * s. Integers with one
// scale keep the products exact: c is exact in fp16, so a matrix instruction multiplies the codes
// themselves and the scale enters in fp32.
//
// Order of a row: element 32 g + 4 r + i (group g, run r < 8, place i < 4) is stored at place
// r * (d / 8) + 4 g + i. The eight runs then are eight equal pieces of the row, each holding four
// elements of EVERY group: the lane of a matrix fragment that owns run r of the values reads one
// contiguous piece and finds one 4-element part per group in it, and a lane that owns runs 2t and
// 2t + 1 of the keys reads eight elements of every group with one load.
//
// Pages are head-major, [num_pages, H, page_size, row]: the rows of one head in one page are
// contiguous, so a CTA that works on one head reads whole lines (with [page_size, H, row] a 64-byte
// row and its 8-byte scales would each be a separate piece of a line).
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace iamap {

constexpr int kQuantGroup = 32;
constexpr int kMaxCtx = 1 << 30;     // longest max_ctx of the decode calls
// SMs that ranges are made for: a constant, because the workspace queries split without a device and the calls
// have to split alike.
constexpr int kSms = 148;

// The pages of one quantised cache and the page table that a call reads them through.
struct QuantPages {
  const uint8_t* codes;     // [num_pages, H, page_size, d * bits / 8]
  const __half* scales;     // [num_pages, H, page_size, d / 32]
  int64_t num_pages;
  const int32_t* table;     // [sequences, max_pages]
  int max_pages;
  int page_size;
  int H;
};

// Row of (page, head, slot) in the pools, or -1 for a page outside them.
__device__ __forceinline__ int64_t quant_row(const QuantPages& p, int seq, int head, int pos) {
  const int pi = pos / p.page_size;
  const int page = p.table[(int64_t)seq * p.max_pages + pi];
  if (page < 0 || page >= p.num_pages) return -1;
  return ((int64_t)page * p.H + head) * p.page_size + (pos - pi * p.page_size);
}

// A sequence's context length as the device holds it, inside [0, max_ctx]; a value outside is
// clamped and reported.
__device__ __forceinline__ int quant_ctx(const int32_t* ctx_lens, int seq, int max_ctx,
                                         unsigned int* status) {
  const int c = ctx_lens[seq];
  if (c < 0 || c > max_ctx) {
    if (threadIdx.x == 0) raise_status(status, IAMAP_DEV_BAD_INDEX);
    return c < 0 ? 0 : max_ctx;
  }
  return c;
}

// A kernel that follows another of the same call starts while that one drains: what it does before
// after_previous() may not touch what the earlier kernel writes. The first kernel of a call is launched as
// usual, so everything before the call is complete when any of its kernels starts.
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;"); }
template <typename P, typename... A>
int launch_next(const char* what, void (*kernel)(P, A...), dim3 grid, unsigned int threads, size_t smem,
                cudaStream_t st, P p, A... a) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p, a...);
  if (e != cudaSuccess)
    return set_error(IAMAP_ERR_CUDA, "launch of %s failed: %s", what, cudaGetErrorString(e));
  return IAMAP_OK;
}

// Host checks of a quantised cache and its page table; IAMAP_OK or an error code.
int check_quant_pages(const void* codes, const void* scales, int64_t num_pages,
                      const int32_t* page_table, int max_pages, int page_size, int H, int d,
                      int bits);
// Host check of a decode batch over such a cache.
int check_quant_batch(const int32_t* ctx_lens, int max_ctx, int batch, int max_pages,
                      int page_size);

}  // namespace iamap
