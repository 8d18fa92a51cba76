// Paged KV cache: a step's tables from the requests' lengths, the new tokens'
// norm, rotary positions and write to their pages, and the C entry points of
// the paged operators (include/mk.h).
#include <algorithm>
#include <cmath>
#include <cstring>

#include "mk_paged_dev.cuh"

namespace mk {
namespace {

// ---------------------------------------------------------------- tables
// Every CTA scans all requests (n <= 4096: a few KB, from L2) into shared
// memory, so that no CTA waits on another, and then fills its share of the
// taken pages and of the rows by a search in the scanned offsets.  Latency
// bound: one launch, one scan, one search.
constexpr int PT_THREADS = 512;
constexpr int PT_PER_THREAD = MK_PAGED_MAX_REQUESTS / PT_THREADS;

struct PtSmem {
  long long wrow[PT_THREADS / 32];
  int wpage[PT_THREADS / 32];
  int taken, pad;
  // then cu [n + 1]: first row of each request (clamped to max_tokens); upto
  // [n + 1]: pages needed by the requests before; ctx [n]: cached tokens, -1: refused
  static size_t bytes(int n) { return sizeof(PtSmem) + 4 * (3 * (size_t)n + 2); }
};

__global__ void __launch_bounds__(PT_THREADS) paged_tables_kernel(const PagedTablesParams P) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  PtSmem& S = *reinterpret_cast<PtSmem*>(smem_raw);
  int* s_cu = reinterpret_cast<int*>(&S + 1);
  int* s_upto = s_cu + P.n + 1;
  int* s_ctx = s_upto + P.n + 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int page_mask = (1 << P.page_shift) - 1;
  grid_launch_dependents();
  grid_wait_prior();
  const int free_raw = *P.n_free;
  const int n_free = min(max(free_raw, 0), P.free_cap);
  const long long room = (long long)P.max_blocks << P.page_shift;
  bool bad = free_raw != n_free;

  // per-thread run of consecutive requests, then a scan over the threads
  const int per = (P.n + PT_THREADS - 1) / PT_THREADS;
  int ctx[PT_PER_THREAD], add[PT_PER_THREAD], need[PT_PER_THREAD];
  long long rows = 0;
  int pages = 0;
#pragma unroll
  for (int i = 0; i < PT_PER_THREAD; ++i) {
    const int r = tid * per + i;
    ctx[i] = add[i] = need[i] = 0;
    if (i < per && r < P.n) {
      const int c = P.ctx[r], a = P.add[r];
      if (c < 0 || a < 0 || (long long)c + a > room) {
        ctx[i] = -1;  // refused: no rows, no pages
        bad = true;
      } else {
        ctx[i] = c;
        add[i] = a;
        need[i] = (int)(((long long)c + a + page_mask) >> P.page_shift) -
                  (int)(((long long)c + page_mask) >> P.page_shift);
      }
      rows += add[i];
      pages += need[i];
    }
  }
  long long xr = rows;
  int xp = pages;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long ur = __shfl_up_sync(0xffffffffu, xr, o);
    const int up = __shfl_up_sync(0xffffffffu, xp, o);
    if (lane >= o) {
      xr += ur;
      xp += up;
    }
  }
  if (lane == 31) {
    S.wrow[warp] = xr;
    S.wpage[warp] = xp;
  }
  if (tid == 0) S.taken = 0;
  __syncthreads();
  for (int w = 0; w < warp; ++w) {
    xr += S.wrow[w];
    xp += S.wpage[w];
  }
  long long row0 = xr - rows;
  int page0 = xp - pages, served_upto = 0;
#pragma unroll
  for (int i = 0; i < PT_PER_THREAD; ++i) {
    const int r = tid * per + i;
    if (i < per && r < P.n) {
      const long long row1 = row0 + add[i];
      const int page1 = page0 + need[i];
      bool served = ctx[i] >= 0;
      if (served && (row1 > P.max_tokens || (need[i] > 0 && page1 > n_free))) {
        served = false;
        bad = true;
      }
      s_cu[r] = (int)min(row0, (long long)P.max_tokens);
      s_upto[r] = page0;
      s_ctx[r] = served ? ctx[i] : -1;
      if (served && need[i] > 0) served_upto = max(served_upto, page1);
      if (r == P.n - 1) {
        s_cu[P.n] = (int)min(row1, (long long)P.max_tokens);
        s_upto[P.n] = page1;
      }
      if (blockIdx.x == 0) {
        P.cu[r + 1] = (int)min(row1, (long long)P.max_tokens);
        P.kv[r] = served ? ctx[i] + add[i] : 0;
      }
      row0 = row1;
      page0 = page1;
    }
  }
  if (served_upto > 0) atomicMax(&S.taken, served_upto);
  if (bad && blockIdx.x == 0) latch(P.status, MK_ERR_BOUNDS);
  __syncthreads();
  const int taken = S.taken;
  if (blockIdx.x == 0 && tid == 0) {
    P.cu[0] = 0;
    *P.n_left = n_free - taken;
  }
  const int gtid = blockIdx.x * PT_THREADS + tid, gsize = gridDim.x * PT_THREADS;
  for (int p = gtid; p < taken; p += gsize) {
    const int r = find_le(s_upto, P.n, p);
    if (s_ctx[r] < 0) continue;  // before the last served one every request that needs pages is served
    const int held = (int)(((long long)s_ctx[r] + page_mask) >> P.page_shift);
    P.table[(int64_t)r * P.max_blocks + held + (p - s_upto[r])] = P.free_pages[n_free - 1 - p];
  }
  const int total = s_cu[P.n];
  for (int t = gtid; t < P.max_tokens; t += gsize) {
    int pos = 0, slot = -1;
    if (t < total) {
      const int r = find_le(s_cu, P.n, t);
      const int c = s_ctx[r];
      if (c >= 0) {
        pos = c + (t - s_cu[r]);
        const int blk = pos >> P.page_shift;
        const int held = (int)(((long long)c + page_mask) >> P.page_shift);
        const int page = blk < held ? P.table[(int64_t)r * P.max_blocks + blk]
                                    : P.free_pages[n_free - 1 - (s_upto[r] + blk - held)];
        // a page that no cache has gives the slot that append refuses
        const long long at = ((long long)page << P.page_shift) | (pos & page_mask);
        slot = at >= 0 && at < 0x7fffffffll ? (int)at : 0x7fffffff;
      }
    }
    P.pos[t] = pos;
    P.slot[t] = slot;
  }
}

// ---------------------------------------------------------------- append
// One pass: every head row is read once, normed and turned in registers and
// written once (HBM bound).  Lane j of a group of HD/16 lanes holds the two
// 16-byte chunks j and j + rotary/16 of a head, whose elements are each
// other's pairs, so the rotation needs no exchange.
constexpr int PA_THREADS = 256;

template <int HD, bool BF>
__global__ void __launch_bounds__(PA_THREADS) paged_append_kernel(const __grid_constant__ PagedAppendParams P) {
  __shared__ float2 cs[HD / 2];  // cos, sin of the token's pairs
  const int t = blockIdx.x, tid = threadIdx.x;
  grid_launch_dependents();
  grid_wait_prior();
  const int slot = P.slot[t];
  if (slot < 0) return;
  if (slot >= P.n_slots) {
    if (tid == 0) latch(P.status, MK_ERR_BOUNDS);
    return;
  }
  const int half = P.rope.rotary_dim / 2;
  if (tid < half) {
    const int pos = P.pos[P.rope.axis[tid] * P.pos_stride + t];
    // whole turns drop out of the low 64 bits; the top 32 of those, signed, are
    // the angle in [-1/2, 1/2) turns to 2^-33
    const int32_t frac = (int32_t)(((uint64_t)(int64_t)pos * P.rope.turn[tid]) >> 32);
    float s, c;
    sincospif((float)frac * 4.656612873077393e-10f, &s, &c);  // 2 * frac / 2^32 half turns
    cs[tid] = make_float2(c, s);
  }
  __syncthreads();
  constexpr int G = HD / 16;  // lanes of a head
  const int j = tid % G, hc = half / 8;
  const bool turn = j < hc;
  // chunks of this lane: a pair of the rotated part, or two of the rest
  const int ca = turn ? j : 2 * hc + 2 * (j - hc), cb = turn ? j + hc : ca + 1;
  const int heads = P.hq + 2 * P.hkv;
  const int page = slot >> P.page_shift, off = slot & ((1 << P.page_shift) - 1);
  const int64_t crow = (int64_t)page * P.page_stride + (int64_t)off * P.token_stride;
  for (int h0 = 0; h0 < heads; h0 += PA_THREADS / G) {
    const int h = h0 + tid / G;
    const bool live = h < heads;
    const bool is_q = h < P.hq, is_k = !is_q && h < P.hq + P.hkv;
    const uint16_t* src = is_q ? P.q + t * P.q_stride + (int64_t)h * HD
                         : is_k ? P.k + t * P.k_stride + (int64_t)(h - P.hq) * HD
                                : P.v + t * P.v_stride + (int64_t)(h - P.hq - P.hkv) * HD;
    uint16_t* dst = is_q ? P.q_out + t * P.qo_stride + (int64_t)h * HD
                   : is_k ? P.kc + crow + (int64_t)(h - P.hq) * P.head_stride
                          : P.vc + crow + (int64_t)(h - P.hq - P.hkv) * P.head_stride;
    uint4 wa = make_uint4(0, 0, 0, 0), wb = wa;
    if (live) {
      wa = reinterpret_cast<const uint4*>(src)[ca];
      wb = reinterpret_cast<const uint4*>(src)[cb];
    }
    const uint16_t* gain = is_q ? P.q_gain : is_k ? P.k_gain : nullptr;
    float a[8], b[8];
    up8<BF>(wa, a);
    up8<BF>(wb, b);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += a[i] * a[i] + b[i] * b[i];
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (gain) {
      const float inv = rsqrtf(ss / HD + P.eps);
      float ga[8], gb[8];
      up8<BF>(reinterpret_cast<const uint4*>(gain)[ca], ga);
      up8<BF>(reinterpret_cast<const uint4*>(gain)[cb], gb);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] *= inv * ga[i];
        b[i] *= inv * gb[i];
      }
    }
    if (turn && (is_q || is_k)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 w = cs[8 * j + i];
        const float x = a[i], y = b[i];
        a[i] = x * w.x - y * w.y;
        b[i] = y * w.x + x * w.y;
      }
    }
    if (live) {
      reinterpret_cast<uint4*>(dst)[ca] = down8<BF>(a);
      reinterpret_cast<uint4*>(dst)[cb] = down8<BF>(b);
    }
  }
}

template <int HD>
cudaError_t append_launch(const PagedAppendParams& p, int dtype, cudaStream_t st) {
  return dtype == MK_BF16 ? paged_launch(paged_append_kernel<HD, true>, p.n_tokens, PA_THREADS, 0, st, p)
                          : paged_launch(paged_append_kernel<HD, false>, p.n_tokens, PA_THREADS, 0, st, p);
}

// ---------------------------------------------------------------- attention
// Which kernel takes which request is a rule on its rows (new tokens x query
// heads per kv head); both walk the same device arrays and leave the other's
// requests out, so that a step may mix them.
cudaError_t attention_launch(PagedAttnParams& p, const PagedKv& kv, int d, bool bf, void* workspace,
                             cudaStream_t st) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  p.device = dev;
  p.rep_inv = (65536 + p.rep - 1) / p.rep;
  // The few-row kernel has the rows of the longest request where it takes them
  // all, else those of a single token (its products cost by the row).
  const int64_t most = (int64_t)p.max_new * p.rep;
  const bool all_few = most <= 32;
  const int want = all_few ? (int)most : p.rep;
  p.few_rows = want <= 8 ? 8 : want <= 16 ? 16 : want <= 32 ? 32 : 0;
  // rows a pair has at most: a warp each in the join, or several for one
  p.join_shares = !all_few || want > 4 ? 0 : want > 2 ? 1 : want > 1 ? 2 : 3;
  // workspace: descriptions, maxima and sums, outputs of the two kernels' parts
  const int ctas = std::min(sms, 224);
  uint8_t* w = (uint8_t*)workspace;
  PagedParts few{}, chunk{};
  few.rt = 32;
  chunk.rt = 256;
  few.ctas = ctas;
  chunk.ctas = all_few ? 0 : ctas;
  few.desc = (PartDesc*)w;
  chunk.desc = few.desc + ctas;
  few.ml = (float2*)(chunk.desc + ctas);
  chunk.ml = few.ml + (size_t)2 * ctas * few.rt;
  few.o = (float*)(chunk.ml + (size_t)2 * ctas * chunk.rt);
  chunk.o = few.o + (size_t)2 * ctas * few.rt * d;
  static_assert(224 * (2 * 16 + 2 * (32 + 256) * (8 + 128 * 4)) <= MK_PAGED_WORKSPACE_BYTES, "workspace");
  e = paged_few_launch(p, kv, few, d, bf, st);
  if (e == cudaSuccess && !all_few) e = paged_chunk_launch(p, kv, chunk, d, bf, st);
  if (e == cudaSuccess) e = paged_join_launch(p, few, chunk, d, bf, st);
  return e;
}

// ---------------------------------------------------------------- argument checks
bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool al4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

int log2_page(int page) {
  for (int s = 4; s <= 8; ++s)
    if (page == 1 << s) return s;
  return -1;
}

int check_cache(const mk_paged_cache* c) {
  if (!c || !c->k || !c->v || !al16(c->k) || !al16(c->v) || !al4(c->status)) return MK_ERR_INVALID_ARG;
  if (c->n_q_heads < 1 || c->n_kv_heads < 1 || c->n_pages < 1) return MK_ERR_INVALID_ARG;
  if (c->dtype != MK_BF16 && c->dtype != MK_FP16) return MK_ERR_INVALID_ARG;
  // a stride from token to token, head to head, page to page; one that joins
  // nothing (one head, one page) is not used
  const int64_t strides[] = {c->token_stride, c->n_kv_heads > 1 ? c->head_stride : c->token_stride,
                             c->n_pages > 1 ? c->page_stride : c->token_stride};
  for (int64_t s : strides)
    if ((s & 7) || s < c->head_dim || s >= (1ll << 38)) return MK_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return MK_ERR_UNSUPPORTED;
  if (log2_page(c->page_size) < 0) return MK_ERR_UNSUPPORTED;
  if ((int64_t)c->n_pages * c->page_size > 0x7fffffffll) return MK_ERR_UNSUPPORTED;
  return MK_OK;
}

// The code of a call whose launches said `e` (a failed one leaves nothing behind
// for the next CUDA call to report).
int done(cudaError_t e) {
  if (e == cudaSuccess) return MK_OK;
  cudaGetLastError();
  return MK_ERR_CUDA;
}

int check_batch(const mk_paged_batch* b) {
  if (!b || !b->block_table || !b->cu_new || !b->kv_lens) return MK_ERR_INVALID_ARG;
  if (!al4(b->block_table) || !al4(b->cu_new) || !al4(b->kv_lens)) return MK_ERR_INVALID_ARG;
  if (b->n < 1 || b->max_blocks < 1 || b->max_tokens < 0) return MK_ERR_INVALID_ARG;
  if (b->n > MK_PAGED_MAX_REQUESTS || log2_page(b->page_size) < 0) return MK_ERR_UNSUPPORTED;
  if ((int64_t)b->n * b->max_blocks > 0x7fffffffll ||
      (int64_t)b->max_blocks * b->page_size > 0x7fffffffll)
    return MK_ERR_UNSUPPORTED;
  return MK_OK;
}

}  // namespace

cudaError_t paged_prepare(const void* kernel, int smem, int regs, int device, std::atomic<uint64_t>* done) {
  const uint64_t bit = 1ull << (device & 63);
  if (device < 64 && (done->load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  cudaFuncAttributes fa;
  cudaError_t e = cudaFuncGetAttributes(&fa, kernel);
  if (e == cudaSuccess && regs && fa.numRegs != regs) e = cudaErrorInvalidKernelImage;
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_relaxed);
  return e;
}

}  // namespace mk

using namespace mk;

extern "C" int mk_paged_tables(const mk_paged_batch* b, const int32_t* ctx_lens,
                               const int32_t* new_lens, const int32_t* free_pages,
                               int free_capacity, const int32_t* n_free, int32_t* n_left,
                               int32_t* status, void* stream) {
  const int rc = check_batch(b);
  if (rc != MK_OK) return rc;
  if (!ctx_lens || !new_lens || !n_free || !n_left || n_left == n_free || free_capacity < 0 ||
      (free_capacity > 0 && !free_pages) || (b->max_tokens > 0 && (!b->positions || !b->slots)))
    return MK_ERR_INVALID_ARG;
  const void* ptrs[] = {ctx_lens, new_lens, free_pages, n_free, n_left, status, b->positions, b->slots};
  for (const void* p : ptrs)
    if (!al4(p)) return MK_ERR_INVALID_ARG;
  PagedTablesParams p{};
  p.ctx = ctx_lens; p.add = new_lens; p.free_pages = free_pages; p.n_free = n_free;
  p.table = b->block_table; p.cu = b->cu_new; p.kv = b->kv_lens; p.pos = b->positions;
  p.slot = b->slots; p.n_left = n_left; p.status = status;
  p.n = b->n; p.max_blocks = b->max_blocks; p.max_tokens = b->max_tokens;
  p.free_cap = free_capacity; p.page_shift = log2_page(b->page_size);
  const size_t smem = PtSmem::bytes(b->n);
  if (smem > 49152 && cudaFuncSetAttribute(paged_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           (int)smem) != cudaSuccess) {
    cudaGetLastError();
    return MK_ERR_CUDA;
  }
  const int grid = min(152, max(1, (b->max_tokens + 2 * PT_THREADS - 1) / (2 * PT_THREADS)));
  return done(paged_launch(paged_tables_kernel, grid, PT_THREADS, (int)smem, (cudaStream_t)stream, p));
}

extern "C" int mk_rope_init(mk_rope* rope, int rotary_dim, double theta, const double* inv_freq,
                            int n_axes, const uint8_t* axis_of_pair) {
  if (!rope || rotary_dim < 16 || rotary_dim > 128 || rotary_dim % 16 || n_axes < 1 || n_axes > 4 ||
      (!inv_freq && !(theta > 0.0 && std::isfinite(theta))) || (n_axes > 1 && !axis_of_pair))
    return MK_ERR_INVALID_ARG;
  mk_rope r;
  std::memset(&r, 0, sizeof(r));
  r.rotary_dim = rotary_dim;
  r.n_axes = n_axes;
  for (int i = 0; i < rotary_dim / 2; ++i) {
    const double w = inv_freq ? inv_freq[i] : std::pow(theta, -2.0 * i / rotary_dim);
    if (!std::isfinite(w) || (axis_of_pair && axis_of_pair[i] >= n_axes)) return MK_ERR_INVALID_ARG;
    const double turns = w / 6.283185307179586476925;
    const double frac = turns - std::floor(turns);  // [0, 1]; 1 where a tiny negative rounds up
    r.turn[i] = frac < 1.0 ? (uint64_t)std::ldexp(frac, 64) : 0;
    r.axis[i] = axis_of_pair ? axis_of_pair[i] : 0;
  }
  *rope = r;
  return MK_OK;
}

extern "C" int mk_paged_append(const mk_paged_cache* c, const void* q, int64_t q_stride, const void* k,
                               int64_t k_stride, const void* v, int64_t v_stride, void* q_out,
                               int64_t q_out_stride, const void* q_norm, const void* k_norm, float eps,
                               const mk_rope* rope, const int32_t* positions, int64_t pos_stride,
                               const int32_t* slots, int n_tokens, void* stream) {
  const int rc = check_cache(c);
  if (rc != MK_OK) return rc;
  if (n_tokens < 0 || !q || !k || !v || !q_out || !slots || !al4(slots)) return MK_ERR_INVALID_ARG;
  const void* ptrs[] = {q, k, v, q_out, q_norm, k_norm};
  for (const void* p : ptrs)
    if (!al16(p)) return MK_ERR_INVALID_ARG;
  const int64_t qw = (int64_t)c->n_q_heads * c->head_dim, kw = (int64_t)c->n_kv_heads * c->head_dim;
  if (((q_stride | k_stride | v_stride | q_out_stride) & 7) || q_stride < qw || q_out_stride < qw ||
      k_stride < kw || v_stride < kw || !(eps >= 0.f))
    return MK_ERR_INVALID_ARG;
  if (q == q_out && q_stride != q_out_stride) return MK_ERR_INVALID_ARG;
  if (rope) {
    if (!positions || !al4(positions) || pos_stride < 0 || rope->rotary_dim < 16 ||
        rope->rotary_dim % 16 || rope->rotary_dim > c->head_dim || rope->n_axes < 1 || rope->n_axes > 4)
      return MK_ERR_INVALID_ARG;
    for (int i = 0; i < rope->rotary_dim / 2; ++i)
      if (rope->axis[i] >= rope->n_axes) return MK_ERR_INVALID_ARG;
  }
  if (n_tokens == 0) return MK_OK;
  PagedAppendParams p{};
  p.q = (const uint16_t*)q; p.k = (const uint16_t*)k; p.v = (const uint16_t*)v;
  p.q_gain = (const uint16_t*)q_norm; p.k_gain = (const uint16_t*)k_norm;
  p.q_out = (uint16_t*)q_out; p.kc = (uint16_t*)c->k; p.vc = (uint16_t*)c->v;
  p.pos = positions; p.slot = slots; p.status = c->status;
  p.q_stride = q_stride; p.k_stride = k_stride; p.v_stride = v_stride; p.qo_stride = q_out_stride;
  p.pos_stride = pos_stride; p.page_stride = c->page_stride; p.head_stride = c->head_stride;
  p.token_stride = c->token_stride;
  p.hq = c->n_q_heads; p.hkv = c->n_kv_heads; p.n_tokens = n_tokens;
  p.n_slots = c->n_pages * c->page_size; p.page_shift = log2_page(c->page_size);
  p.eps = eps;
  if (rope) p.rope = *rope;
  const cudaError_t e = c->head_dim == 128 ? append_launch<128>(p, c->dtype, (cudaStream_t)stream)
                                           : append_launch<64>(p, c->dtype, (cudaStream_t)stream);
  return done(e);
}

extern "C" int mk_paged_attention(const mk_paged_cache* c, const mk_paged_batch* b, const void* q,
                                  int64_t q_stride, void* out, int64_t out_stride, float* lse,
                                  float scale, int window, void* stream) {
  int rc = check_cache(c);
  if (rc != MK_OK) return rc;
  rc = check_batch(b);
  if (rc != MK_OK) return rc;
  if (!q || !out || q == out || !al16(q) || !al16(out) || !al4(lse) || !c->workspace ||
      !al16(c->workspace))
    return MK_ERR_INVALID_ARG;
  const int64_t qw = (int64_t)c->n_q_heads * c->head_dim;
  if (((q_stride | out_stride) & 7) || q_stride < qw || out_stride < qw || window < 0 ||
      !std::isfinite(scale) || b->page_size != c->page_size || b->max_new < 1)
    return MK_ERR_INVALID_ARG;
  if (c->n_q_heads % c->n_kv_heads) return MK_ERR_INVALID_ARG;
  if (c->n_q_heads / c->n_kv_heads > 64) return MK_ERR_UNSUPPORTED;
  if (b->max_tokens == 0) return MK_OK;
  PagedAttnParams p{};
  p.q = (const uint16_t*)q; p.out = (uint16_t*)out; p.lse = lse;
  p.table = b->block_table; p.cu = b->cu_new; p.kv = b->kv_lens; p.status = c->status;
  p.q_stride = q_stride; p.o_stride = out_stride;
  p.n = b->n; p.max_blocks = b->max_blocks; p.rows = b->max_tokens; p.max_new = b->max_new;
  p.n_pages = c->n_pages; p.page_shift = log2_page(c->page_size);
  p.hkv = c->n_kv_heads; p.rep = c->n_q_heads / c->n_kv_heads;
  p.window = window ? window : 0x7fffffff;
  p.scale = scale != 0.f ? scale : 1.0f / sqrtf((float)c->head_dim);
  // units of work are counted in 32 bits (64 keys x (128 rows or a request))
  const int64_t tiles = (int64_t)b->max_tokens * p.rep / 64 + b->n;
  if (tiles * c->n_kv_heads * ((int64_t)b->max_blocks * b->page_size / 64 + 1) > 0x7fffffffll)
    return MK_ERR_UNSUPPORTED;
  const PagedKv kv = {c->k, c->v, c->page_stride, c->head_stride, c->token_stride,
                      c->n_pages, c->n_kv_heads, c->page_size};
  const cudaError_t e = attention_launch(p, kv, c->head_dim, c->dtype == MK_BF16, c->workspace, (cudaStream_t)stream);
  return done(e);
}
