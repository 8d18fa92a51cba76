// Attention over a paged KV cache.
#include "mk_paged_dev.cuh"

namespace mk {
namespace {

template <bool BF>
__device__ __forceinline__ float up1(uint16_t w) {
  if constexpr (BF) return __uint_as_float((uint32_t)w << 16);
  return __half2float(__ushort_as_half(w));
}
template <bool BF>
__device__ __forceinline__ uint16_t down1(float x) {
  if constexpr (BF) return __bfloat16_as_ushort(__float2bfloat16_rn(x));
  return __half_as_ushort(__float2half_rn(x));
}

// One warp per (row, query head): the keys one after another, the running
// maximum and sum of the softmax, lane l holding elements l, l + 32, ...
template <int HD, bool BF>
__global__ void __launch_bounds__(256) paged_attn_kernel(const PagedAttnParams P) {
  const int lane = threadIdx.x & 31;
  const int hq = P.hkv * P.rep;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (w >= (int64_t)P.rows * hq) return;
  const int row = (int)(w / hq), h = (int)(w % hq);
  int r = -1;
  for (int i = 0; i < P.n; ++i)
    if (P.cu[i] <= row && row < P.cu[i + 1]) {
      r = i;
      break;
    }
  if (r < 0) return;
  if ((int64_t)(P.cu[r + 1] - P.cu[r]) * P.rep <= P.few_rows) return;
  const int first = P.cu[r], add = P.cu[r + 1] - first, room = P.max_blocks << P.page_shift;
  const int kv_raw = P.kv[r], kv = min(max(kv_raw, 0), room);
  if (kv != kv_raw && P.status && lane == 0) atomicCAS(P.status, MK_OK, MK_ERR_BOUNDS);
  if (first < 0 || P.cu[r + 1] > P.rows || add > P.max_new) {
    if (P.status && lane == 0) atomicCAS(P.status, MK_OK, MK_ERR_BOUNDS);
    return;
  }
  const int pos = kv_raw - add + (row - first);
  const int lo = max(0, P.window == 0x7fffffff ? 0 : pos - P.window + 1), hi = min(pos, kv - 1);
  constexpr int E = HD / 32;
  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = up1<BF>(P.q[row * P.q_stride + h * HD + lane + 32 * e]) * P.scale;
    o[e] = 0.f;
  }
  for (int j = lo; j <= hi; ++j) {
    const int page = P.table[(int64_t)r * P.max_blocks + (j >> P.page_shift)];
    const bool ok = page >= 0 && page < P.n_pages;
    if (!ok && P.status && lane == 0) atomicCAS(P.status, MK_OK, MK_ERR_BOUNDS);
    const int64_t at = page * P.page_stride + (h / P.rep) * P.head_stride +
                       (j & ((1 << P.page_shift) - 1)) * P.token_stride;
    float s = 0.f, v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      s += ok ? q[e] * up1<BF>(P.kc[at + lane + 32 * e]) : 0.f;
      v[e] = ok ? up1<BF>(P.vc[at + lane + 32 * e]) : 0.f;
    }
    s = warp_sum(s);
    const float mn = fmaxf(m, s), a = expf(m - mn), p = expf(s - mn);
    l = l * a + p;
    m = mn;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * a + p * v[e];
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) P.out[row * P.o_stride + h * HD + lane + 32 * e] = down1<BF>(o[e] * inv);
  if (P.lse && lane == 0) P.lse[(int64_t)row * hq + h] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

cudaError_t paged_attention_launch(const PagedAttnParams& p0, const PagedKv& kv, int d, int dtype,
                                   void* workspace, cudaStream_t st) {
  PagedAttnParams p = p0;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const bool bf = dtype == MK_BF16;
  // rows of the few-row kernel: those of the longest request where it takes
  // them all, else those of single tokens
  const int64_t most = (int64_t)p.max_new * p.rep;
  const bool all_few = most <= 32;
  const int want = all_few ? (int)most : p.rep;
  p.few_rows = want <= 8 ? 8 : want <= 16 ? 16 : want <= 32 ? 32 : 0;
  uint8_t* w = (uint8_t*)workspace;
  PagedParts few{};
  few.rt = p.few_rows;
  few.ctas = sms;
  few.desc = (PartDesc*)w;
  few.ml = (float2*)(w + 16384);
  few.o = (float*)(w + 16384 + 2 * 8 * 32 * (size_t)sms);
  e = paged_few_launch(p, kv, few, d, bf, st);
  if (e != cudaSuccess) return e;
  e = paged_join_launch(p, few, PagedParts{}, d, bf, st);
  if (e != cudaSuccess || all_few) return e;
  const int64_t warps = (int64_t)p.rows * p.hkv * p.rep;
  const unsigned grid = (unsigned)((warps + 7) / 8);
  if (d == 128 && dtype == MK_BF16) paged_attn_kernel<128, true><<<grid, 256, 0, st>>>(p);
  else if (d == 128) paged_attn_kernel<128, false><<<grid, 256, 0, st>>>(p);
  else if (dtype == MK_BF16) paged_attn_kernel<64, true><<<grid, 256, 0, st>>>(p);
  else paged_attn_kernel<64, false><<<grid, 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace mk
