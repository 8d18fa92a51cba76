// Launch parameters of the paged-cache operators (mk_paged_*.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <utility>

#include "../../include/mk.h"

namespace mk {

struct PagedTablesParams {
  const int32_t *ctx, *add, *free_pages, *n_free;
  int32_t *table, *cu, *kv, *pos, *slot, *n_left, *status;
  int n, max_blocks, max_tokens, free_cap, page_shift;
};

struct PagedAppendParams {
  const uint16_t *q, *k, *v, *q_gain, *k_gain;
  uint16_t *q_out, *kc, *vc;
  const int32_t *pos, *slot;
  int32_t* status;
  int64_t q_stride, k_stride, v_stride, qo_stride, pos_stride;
  int64_t page_stride, head_stride, token_stride;
  int hq, hkv, n_tokens, n_slots, page_shift;
  float eps;
  mk_rope rope;  // rotary_dim 0: no rotation
};

struct PagedAttnParams {
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  const int32_t *table, *cu, *kv;
  int32_t* status;
  int64_t q_stride, o_stride;
  int n, max_blocks, rows, max_new, n_pages, page_shift;
  int hkv, rep, window;  // window 0x7fffffff: none
  int device;
  int few_rows;  // requests of at most this many rows (new tokens x rep) go to the few-row kernel
  int rep_inv;  // ceil(2^16 / rep)
  int join_shares;  // log2 of the warps that join one row of the few-row kernel
  float scale;
#ifdef __CUDACC__
  // token of a tile's row (row < 256, rep <= 64: the error, row / 2^16, stays
  // below 1 / rep)
  __device__ __forceinline__ int token_of(int row) const { return (row * rep_inv) >> 16; }
#endif
};

// The cache as the tensor maps see it.
struct PagedKv {
  const void *k, *v;
  int64_t page_stride, head_stride, token_stride;
  int n_pages, hkv, page;
};

// A pair's (or tile's) rows whose keys were divided among CTAs: `parts` of them
// from CTA desc index on; 0: none.
struct alignas(16) PartDesc {
  int row0, rows, head, parts;
};
// Workspace of one kernel's divided rows: part 2 c (+ 1) is CTA c's first (second)
// unfinished run of keys: o, rt rows x head_dim unnormalised, ml [part][rt]
// maximum (base 2) and sum.
struct PagedParts {
  PartDesc* desc;
  float2* ml;
  float* o;
  int rt, ctas;
};

// Opt a kernel into `smem` bytes of shared memory, once per device (the limit
// is set to the largest a call can ask for).  `regs`: what the kernel has to be
// compiled to, 0: any.  `done` is the kernel's own word, a bit per device.
cudaError_t paged_prepare(const void* kernel, int smem, int regs, int device, std::atomic<uint64_t>* done);

// Launch, as a programmatic dependent of what precedes in the stream or not.
template <class... P, class... A>
inline cudaError_t paged_launch_if(bool dependent, void (*kernel)(P...), int grid, int threads, int smem,
                                   cudaStream_t st, A&&... args) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &at;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}
template <class... P, class... A>
inline cudaError_t paged_launch(void (*kernel)(P...), int grid, int threads, int smem, cudaStream_t st, A&&... args) {
  return paged_launch_if(true, kernel, grid, threads, smem, st, std::forward<A>(args)...);
}

cudaError_t paged_few_launch(const PagedAttnParams& p, const PagedKv& kv, const PagedParts& w, int d,
                             bool bf, cudaStream_t st);
cudaError_t paged_chunk_launch(const PagedAttnParams& p, const PagedKv& kv, const PagedParts& w, int d,
                               bool bf, cudaStream_t st);
cudaError_t paged_join_launch(const PagedAttnParams& p, const PagedParts& a, const PagedParts& b, int d,
                              bool bf, cudaStream_t st);

}  // namespace mk
