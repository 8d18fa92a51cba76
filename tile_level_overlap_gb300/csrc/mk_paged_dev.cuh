// Device helpers of the paged-cache kernels: conversions, the requests' scan,
// bounded mbarrier waits, page loads.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mk_device.cuh"
#include "mk_paged.h"

namespace mk {

__device__ __forceinline__ void latch(int32_t* status, int code) {
  if (status) atomicCAS(status, MK_OK, code);
}

// Largest r in [0, n) with a[r] <= x (a non-decreasing, a[0] <= x).
__device__ __forceinline__ int find_le(const int* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// ---------------------------------------------------------------- 16-bit pairs
template <bool BF>
__device__ __forceinline__ float2 up2(uint32_t w) {
  if constexpr (BF) return make_float2(bf_lo(w), bf_hi(w));
  const __half2 h = *reinterpret_cast<const __half2*>(&w);
  return __half22float2(h);
}
template <bool BF>
__device__ __forceinline__ uint32_t down2(float a, float b) {
  if constexpr (BF) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
__device__ __forceinline__ u64 mul_f32x2(u64 a, u64 b) {
  u64 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A row's factor and log-sum-exp from its maximum (base 2) and sum: 0 and -inf
// where it saw no key; a NaN among its scores stays one.
__device__ __forceinline__ float inv_of(float l) { return l != 0.f ? 1.f / l : 0.f; }
__device__ __forceinline__ float lse_of(float m, float l) {
  return l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// ---------------------------------------------------------------- dependent launches
// Every kernel here is launched as a programmatic dependent of what precedes it
// in the stream: it may be set up while that one's last blocks run, and uses
// global memory only after grid_wait_prior() has seen it complete.  (The join reads
// the workspace once before, to fetch its own code, and drops what it read.)  A
// kernel that starts early has what earlier kernels wrote from its own wait alone,
// so every one waits before its first read, also where its predecessor has.
__device__ __forceinline__ void grid_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void grid_wait_prior() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ---------------------------------------------------------------- clusters
// (A barrier of the cluster waits for the threads that have not exited, and every
// kernel here passes its barriers whatever its inputs hold.)
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of the same shared variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ u64 ld_cluster64(uint32_t a) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_cluster32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster64(uint32_t a, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ void st_cluster128(uint32_t a, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
__device__ __forceinline__ void st_cluster32(uint32_t a, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// ---------------------------------------------------------------- bounded waits
// Wait for the phase.  After WAIT_TRIES tries (each suspends the thread for a
// while; tens of milliseconds at the very least, and no wait here depends on
// another CTA) give up: `*dead` is raised, the status latched, and every later
// wait of the CTA returns soon.  Tries are counted, not time: reading a timer
// between two tries costs as much as the waits themselves.
constexpr uint32_t WAIT_TRIES = 1u << 23;
__device__ __forceinline__ void wait_phase(uint64_t* bar, uint32_t parity, volatile int* dead,
                                           int32_t* status) {
  uint32_t tries = 0;
  while (!mbar_try_wait(bar, parity)) {
    if ((++tries & 1023u) == 0) {
      if (*dead) return;
      if (tries >= WAIT_TRIES) {
        *dead = 1;
        latch(status, MK_ERR_TIMEOUT);
        return;
      }
    }
  }
}

// ---------------------------------------------------------------- loads
// Untiled copy into shared memory (addresses and size: multiples of 16 bytes).
__device__ __forceinline__ void bulk_in(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
// Box of 64 elements x tokens x parts of one head and page, from part `part` on
// (the map's dimensions: element, token, part, head, page).  A page outside the
// map reads as zeros.
__device__ __forceinline__ void tma_page(void* dst, const void* tmap, int token, int part, int head,
                                         int page, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
      "l"(tmap), "r"(0), "r"(token), "r"(part), "r"(head), "r"(page), "r"(smem_u32(bar))
      : "memory");
}

// The same, with an L2 policy.
__device__ __forceinline__ void tma_page(void* dst, const void* tmap, int token, int part, int head,
                                         int page, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(smem_u32(dst)),
      "l"(tmap), "r"(0), "r"(token), "r"(part), "r"(head), "r"(page), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// ---------------------------------------------------------------- the requests
// What a request asks of attention, from the device arrays; `bad` where the
// status is to be latched.  Keys [lo, hi) are what any of its rows may see;
// its first row stands at pos0.
struct Request {
  int row0, add, pos0, lo, hi;
  bool bad, falls;
};
__device__ __forceinline__ Request make_request(const PagedAttnParams& P, int c0, int c1, int kv) {
  Request q;
  const int room = P.max_blocks << P.page_shift;
  const int kvp = max(kv, 0);
  q.bad = kv < 0 || kvp > room;
  q.row0 = c0;
  q.add = 0;
  q.falls = c1 < c0;
  if (c0 < 0 || c1 < c0 || c1 > P.rows || c1 - c0 > P.max_new) q.bad = true;
  else q.add = c1 - c0;
  q.pos0 = kvp - q.add;
  q.hi = min(kvp, room);
  // the first row's window begins at pos0 - window + 1
  q.lo = q.pos0 >= P.window ? min(q.pos0 - P.window + 1, q.hi) : 0;
  return q;
}

// Whether a request that begins at cu[r] does so below an earlier offset (its rows may
// be another's); the block's threads together.
__device__ __forceinline__ bool begins_below(const int32_t* cu, int r, int c0) {
  bool low = false;
  for (int i = threadIdx.x; i < r; i += blockDim.x) low |= cu[i] > c0;
  return __syncthreads_or(low);
}

// The scan's results in shared memory: pre [n + 1], a request's first unit, and
// for n up to REQ_KEPT also what read_request read, so that the walk over the
// units does not wait for it again.
constexpr int REQ_KEPT = 1024;
struct Kept {
  int *pre, *c0, *c1, *kv;
  __host__ __device__ static constexpr int bytes(int n) { return 4 * (n + 1) + (n <= REQ_KEPT ? 12 * n : 0); }
  __device__ __forceinline__ Kept(void* base, int n) : pre((int*)base), c0(pre + n + 1), c1(c0 + n), kv(c1 + n) {}
  __device__ __forceinline__ Request read(const PagedAttnParams& P, int r) const {
    const int a = P.cu[r], b = P.cu[r + 1], k = P.kv[r];
    if (P.n <= REQ_KEPT) { c0[r] = a; c1[r] = b; kv[r] = k; }
    return make_request(P, a, b, k);
  }
  __device__ __forceinline__ Request again(const PagedAttnParams& P, int r) const {
    if (P.n <= REQ_KEPT) return make_request(P, c0[r], c1[r], kv[r]);
    return make_request(P, P.cu[r], P.cu[r + 1], P.kv[r]);
  }
};
constexpr int KEPT_MOST = Kept::bytes(REQ_KEPT) > Kept::bytes(MK_PAGED_MAX_REQUESTS)
                              ? Kept::bytes(REQ_KEPT)
                              : Kept::bytes(MK_PAGED_MAX_REQUESTS);

// T units in G runs of equal length (the first T % G one longer).
struct Runs {
  int len, more;
  __device__ __forceinline__ Runs(int T, int G) : len(T / G), more(T - len * G) {}
  __device__ __forceinline__ int start(int c) const { return c * len + min(c, more); }
  __device__ __forceinline__ int of(int u) const {  // run of unit u
    const int split = more * (len + 1);
    return u < split ? u / (len + 1) : more + (u - split) / len;
  }
};

// Exclusive prefix sums of one value per thread of a block of W warps; whether
// any thread says `flag`.  (Unsigned: the sums wrap where the flag discards them.)
template <int W>
__device__ __forceinline__ uint32_t block_scan(uint32_t v, bool flag, int* tmp, int* total, bool* any) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += u;
  }
  if (lane == 31) tmp[warp] = (int)x;
  *any = __syncthreads_or(flag);
  uint32_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const uint32_t t = (uint32_t)tmp[w];
    before += w < warp ? t : 0;
    all += t;
  }
  *total = (int)all;
  return before + x - v;
}

// Where cu falls: requests that begin below an earlier offset have no units
// (each thread's `per` consecutive requests; returns what is left of them).  Out
// of line, so that the kernels' code is as without it.
template <int W>
__device__ __noinline__ uint32_t refuse_below(const int32_t* cu, int n, int* pre, int per, int* tmp) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r0 = min(tid * per, n), r1 = min(r0 + per, n);
  int before = -0x7fffffff - 1;  // the largest offset of the requests before
  for (int r = r0; r < r1; ++r) before = max(before, max(cu[r], cu[r + 1]));
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before = max(before, u);
  }
  __syncthreads();  // tmp has been read
  if (lane == 31) tmp[warp] = before;
  before = __shfl_up_sync(0xffffffffu, before, 1);
  if (lane == 0) before = -0x7fffffff - 1;
  __syncthreads();
  for (int w = 0; w < warp; ++w) before = max(before, tmp[w]);
  __syncthreads();
  uint32_t left = 0;
  for (int r = r0; r < r1; ++r) {
    if (cu[r] < before) pre[r] = 0;
    left += (uint32_t)pre[r];
    before = max(before, max(cu[r], cu[r + 1]));
  }
  return left;
}

// The units of the requests, pre[r] (each thread's `per` consecutive ones, `mine`
// of them together), to a request's first unit; returns their number.  `falls`:
// cu falls at one of the thread's requests.  Rows below an earlier offset may be
// another request's, and the units of overlapping requests have no bound (the
// launch's check counts every row of the step once).
template <int W>
__device__ __forceinline__ int place_units(const PagedAttnParams& P, int* pre, int per, uint32_t mine, bool falls, int* tmp) {
  const int tid = threadIdx.x, r0 = min(tid * per, P.n), r1 = min(r0 + per, P.n);
  int T;
  bool any;
  uint32_t at = block_scan<W>(mine, falls, tmp, &T, &any);
  if (any) at = block_scan<W>(refuse_below<W>(P.cu, P.n, pre, per, tmp), false, tmp, &T, &any);
  for (int r = r0; r < r1; ++r) {
    const int u = pre[r];
    pre[r] = (int)at;
    at += (uint32_t)u;
  }
  if (tid == 0) pre[P.n] = T;
  return T;
}

}  // namespace mk
