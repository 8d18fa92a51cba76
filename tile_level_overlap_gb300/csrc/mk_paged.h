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
  // trees: bit j of a row's mask: it sees the request's new token j; requests of more than
  // 32 mask_words new tokens are causal.  NULL: all are.
  const uint32_t* masks;
  int mask_words;
  int cluster, cluster_tiles;  // CTAs of a tile's cluster (0: no clusters), tiles
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

// Argument checks of the entry points (MK_OK or the code to return); the code of a
// call whose launches said `e`; log2 of a page size, -1 where it is none.
int paged_check_cache(const mk_paged_cache* c);
int paged_check_batch(const mk_paged_batch* b);
int paged_done(cudaError_t e);
int paged_log2(int page);
inline bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
inline bool al4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

// Words [at, at + words) of a call's arrays.
struct PagedWords {
  const void* at;
  int64_t words;
};
// Whether one of the first `written` arrays shares a word with another.
bool paged_overlap(const PagedWords* a, int n, int written);

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

// Launch in clusters of `cluster` CTAs, as a programmatic dependent.
template <class... P, class... A>
inline cudaError_t paged_launch_clusters(void (*kernel)(P...), int grid, int cluster, int threads, int smem,
                                         cudaStream_t st, A&&... args) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[2]{};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

// Clusters of `ctas` (<= 16) CTAs of a kernel that the device holds at once; asked once
// for each size, `known` keeps one more than the number.
inline int paged_clusters_at_once(const void* kernel, int threads, int smem, int device, int ctas, std::atomic<int> (&known)[64][17]) {
  std::atomic<int>* mine = device < 64 ? &known[device][ctas] : nullptr;
  int n = mine ? mine->load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = ctas;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    if ((smem > 0 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) ||
        (ctas > 8 && cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();
      return 0;  // no answer: the next call asks again
    }
    ++n;
    if (mine) mine->store(n, std::memory_order_relaxed);
  }
  return n - 1;
}

cudaError_t paged_few_launch(const PagedAttnParams& p, const PagedKv& kv, const PagedParts& w, int d,
                             bool bf, cudaStream_t st);
cudaError_t paged_chunk_launch(const PagedAttnParams& p, const PagedKv& kv, const PagedParts& w, int d,
                               bool bf, cudaStream_t st);
void paged_chunk_clusters(PagedAttnParams* p, int d, bool bf);
cudaError_t paged_join_tiles_launch(const PagedAttnParams& p, const PagedParts& b, int d, bool bf, cudaStream_t st);
cudaError_t paged_join_launch(const PagedAttnParams& p, const PagedParts& a, const PagedParts& b, int d,
                              bool bf, cudaStream_t st);

}  // namespace mk
