// Paged KV cache: a step's tables from the requests' lengths, the new tokens'
// norm, rotary positions and write to their pages, and the C entry points of
// the paged operators (include/mk.h).
#include <algorithm>
#include <cmath>
#include <cstring>

#include "mk_paged_dev.cuh"

namespace mk {
namespace {

cudaError_t device_sms(int* device, int* sms) {
  const cudaError_t e = cudaGetDevice(device);
  return e != cudaSuccess ? e : cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *device);
}

// ---------------------------------------------------------------- tables
// Every CTA scans all requests (n <= 4096: a few KB, from L2) into shared
// memory, so that no CTA waits on another, and then fills its share of the
// taken pages and of the rows by a search in the scanned offsets.  Latency
// bound: one launch, one scan, one search (32 decoding requests 2.7 us, 64 prompts
// of 141K tokens in all 4.4 us).
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
// 16-byte chunks j and j + rotary/16 of a head, whose elements are each other's
// pairs, so the rotation needs no exchange; a warp takes 32 / (HD/16) heads at a
// time, and a lane's cosines, sines and gains are the same for all of them.
constexpr int PA_THREADS = 256, PA_WARPS = PA_THREADS / 32;

// cos and sin of a pair's angle.  Whole turns drop out of the low 64 bits of the
// product; the top 32 of those, signed, are the angle in [-1/2, 1/2) turns to
// 2^-33.
__device__ __forceinline__ float2 pair_turn(int pos, uint64_t turn) {
  const int32_t frac = (int32_t)(((uint64_t)(int64_t)pos * turn) >> 32);
  float s, c;
  sincospif((float)frac * 4.656612873077393e-10f, &s, &c);  // 2 * frac / 2^32 half turns
  return make_float2(c, s);
}

// A lane's share of a head: two chunks, the angles of their pairs where they
// turn, and the gains.  Packed pairs of floats, two IEEE operations an
// instruction.
template <int HD, bool BF>
struct HeadLane {
  static constexpr int G = HD / 16;
  int ca, cb;
  bool turn;
  u64 c[4], s[4];  // cos, sin of the eight pairs
  uint4 gq[2], gk[2];
  static __device__ __forceinline__ u64 widen(uint32_t w) {
    const float2 f = up2<BF>(w);
    return pack_f32x2(f.x, f.y);
  }
  static __device__ __forceinline__ uint32_t narrow(u64 x) {
    return down2<BF>(__uint_as_float((uint32_t)x), __uint_as_float((uint32_t)(x >> 32)));
  }
  __device__ __forceinline__ HeadLane(const PagedAppendParams& P, int lane) {
    const int j = lane % G, hc = P.rope.rotary_dim / 16;
    turn = j < hc;
    ca = turn ? j : 2 * hc + 2 * (j - hc);
    cb = turn ? j + hc : ca + 1;
    gq[0] = gq[1] = gk[0] = gk[1] = make_uint4(0, 0, 0, 0);
    if (P.q_gain) {
      gq[0] = reinterpret_cast<const uint4*>(P.q_gain)[ca];
      gq[1] = reinterpret_cast<const uint4*>(P.q_gain)[cb];
    }
    if (P.k_gain) {
      gk[0] = reinterpret_cast<const uint4*>(P.k_gain)[ca];
      gk[1] = reinterpret_cast<const uint4*>(P.k_gain)[cb];
    }
  }
  // cs holds pair p at (p % 8) * G + p / 8: a lane's eight are G apart, the
  // lanes of a head end to end
  static __device__ __forceinline__ int place(int pair) { return (pair & 7) * G + (pair >> 3); }
  __device__ __forceinline__ void angles(const float2* cs, int lane) {
    if (!turn) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = cs[2 * i * G + lane % G], y = cs[(2 * i + 1) * G + lane % G];
      c[i] = pack_f32x2(x.x, y.x);
      s[i] = pack_f32x2(x.y, y.y);
    }
  }
  // Norm and turn a head's chunks in place (whole warp; is_q: a query head).
  // Chunks that do not turn pass through no rotation (0 times an infinity is a
  // NaN); without a gain either they stay bit for bit.
  __device__ __forceinline__ void apply(const PagedAppendParams& P, uint4& wa, uint4& wb, bool is_q) {
    const uint32_t ua[4] = {wa.x, wa.y, wa.z, wa.w}, ub[4] = {wb.x, wb.y, wb.z, wb.w};
    u64 a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = widen(ua[i]);
      b[i] = widen(ub[i]);
    }
    const bool gain = is_q ? P.q_gain != nullptr : P.k_gain != nullptr;
    if (P.q_gain || P.k_gain) {
      u64 acc = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc = fma_f32x2(a[i], a[i], fma_f32x2(b[i], b[i], acc));
      float ss = pair_sum(acc);
#pragma unroll
      for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (gain) {
        const float inv = rsqrtf(ss * (1.f / HD) + P.eps);
        const u64 inv2 = pack_f32x2(inv, inv);
        const uint4 x = is_q ? gq[0] : gk[0], y = is_q ? gq[1] : gk[1];
        const uint32_t ga[4] = {x.x, x.y, x.z, x.w}, gb[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = mul_f32x2(mul_f32x2(a[i], inv2), widen(ga[i]));
          b[i] = mul_f32x2(mul_f32x2(b[i], inv2), widen(gb[i]));
        }
      }
    }
    uint32_t oa[4], ob[4];
    if (!turn) {
      if (!gain) return;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        oa[i] = narrow(a[i]);
        ob[i] = narrow(b[i]);
      }
      wa = make_uint4(oa[0], oa[1], oa[2], oa[3]);
      wb = make_uint4(ob[0], ob[1], ob[2], ob[3]);
      return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u64 minus = s[i] ^ 0x8000000080000000ull;
      oa[i] = narrow(fma_f32x2(b[i], minus, mul_f32x2(a[i], c[i])));
      ob[i] = narrow(fma_f32x2(a[i], s[i], mul_f32x2(b[i], c[i])));
    }
    wa = make_uint4(oa[0], oa[1], oa[2], oa[3]);
    wb = make_uint4(ob[0], ob[1], ob[2], ob[3]);
  }
};

// Where the heads of a token go.
template <int HD>
struct TokenOut {
  uint16_t *q, *k, *v;
  __device__ __forceinline__ TokenOut(const PagedAppendParams& P, int t, int slot) {
    const int64_t at = (int64_t)(slot >> P.page_shift) * P.page_stride +
                       (int64_t)(slot & ((1 << P.page_shift) - 1)) * P.token_stride;
    q = P.q_out + t * P.qo_stride;
    k = P.kc + at - P.hq * P.head_stride;
    v = P.vc + at - (P.hq + P.hkv) * P.head_stride;
  }
  __device__ __forceinline__ uint4* head(const PagedAppendParams& P, int h) const {
    return reinterpret_cast<uint4*>(h < P.hq ? q + h * HD : (h < P.hq + P.hkv ? k : v) + h * P.head_stride);
  }
};

// Few tokens: a block each.  Latency bound (3.5 us for 32 tokens of 32 + 16
// heads of 128): every warp works the angles out for itself, while its first
// rows are on their way, so that no barrier stands between.
template <int HD, bool BF>
__global__ void __launch_bounds__(PA_THREADS) paged_append_kernel(const __grid_constant__ PagedAppendParams P) {
  using Lane = HeadLane<HD, BF>;
  constexpr int HPW = 32 / Lane::G, BATCH = 2;
  __shared__ float2 cs[PA_WARPS][HD / 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = blockIdx.x, half = P.rope.rotary_dim / 2;
  grid_launch_dependents();
  grid_wait_prior();
  const int heads = P.hq + 2 * P.hkv, slot = P.slot[t];
  const uint16_t *q = P.q + t * P.q_stride, *k = P.k + t * P.k_stride, *v = P.v + t * P.v_stride;
  Lane L(P, lane);
  for (int h0 = warp * HPW; h0 < heads; h0 += PA_WARPS * HPW * BATCH) {
    uint4 wa[BATCH], wb[BATCH];
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const int h = h0 + u * PA_WARPS * HPW + lane / Lane::G;
      wa[u] = wb[u] = make_uint4(0, 0, 0, 0);
      if (h < heads) {
        const uint4* src = reinterpret_cast<const uint4*>(
            h < P.hq ? q + h * HD : h < P.hq + P.hkv ? k + (h - P.hq) * HD : v + (h - P.hq - P.hkv) * HD);
        wa[u] = src[L.ca];
        wb[u] = src[L.cb];
      }
    }
    if (h0 == warp * HPW) {
      for (int i = lane; i < half; i += 32)
        cs[warp][Lane::place(i)] = pair_turn(P.pos[P.rope.axis[i] * P.pos_stride + t], P.rope.turn[i]);
      __syncwarp();
      L.angles(cs[warp], lane);
      if (slot < 0) return;  // left out
      if (slot >= P.n_slots) {
        if (lane == 0) latch(P.status, MK_ERR_BOUNDS);
        return;
      }
    }
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const int hb = h0 + u * PA_WARPS * HPW, h = hb + lane / Lane::G;  // the step's first head, this lane's
      if (hb >= heads) break;
      uint4 a = wa[u], b = wb[u];
      if (hb < P.hq + P.hkv) L.apply(P, a, b, h < P.hq);
      if (h < heads) {
        const bool value = h >= P.hq + P.hkv;  // values stay as they are
        uint4* dst = TokenOut<HD>(P, t, slot).head(P, h);
        dst[L.ca] = value ? wa[u] : a;
        dst[L.cb] = value ? wb[u] : b;
      }
    }
  }
}

// Many tokens: persistent blocks, one per SM.  Four warps load whole tokens into a
// ring in shared memory (bulk copies: what is in flight costs no registers and
// is there however the other warps are placed), teams of two warps take the
// tokens in turn.  8190 tokens of 32 + 16 heads of 128: 36 us (5.6 TB/s; rows
// loaded to registers, three 16-byte pairs a lane in flight: 46-49 us; one loading
// warp, whose turn takes a quarter of a microsecond and more: 38 us, and with heads
// of 64 29 against 20 us).
constexpr int PR_WARPS = 2, PR_LOADERS = 4;  // warps of a team; loading warps
constexpr int PR_TEAMS = 16 / PR_WARPS, PR_TEAM = 32 * PR_WARPS;
constexpr int PR_THREADS = PR_TEAMS * PR_TEAM + 32 * PR_LOADERS, PR_MOST = 32;

struct PrSmem {
  uint64_t full[PR_MOST], empty[PR_MOST];
  int slot[PR_MOST];
  int dead, pad[3];
  float2 cs[PR_TEAMS][2][64];
};
// Depth of the ring for rows of `row` bytes: a multiple of the teams and of the
// loading warps, so that a slot always has the same ones.  (One that came to a
// slot only every other round would not see all phases of its barriers, and
// could take the last but one for the one it waits for.)  0: the other kernel.
static_assert(PR_TEAMS % PR_LOADERS == 0 && PR_MOST % PR_TEAMS == 0, "ring");
inline int ring_depth(int row) {
  return std::min(PR_MOST, (int)((232448 - sizeof(PrSmem)) / row) / PR_TEAMS * PR_TEAMS);
}

template <int HD, bool BF>
__global__ void __launch_bounds__(PR_THREADS, 1)
    paged_append_ring_kernel(const __grid_constant__ PagedAppendParams P, int depth) {
  using Lane = HeadLane<HD, BF>;
  constexpr int HPW = 32 / Lane::G;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  PrSmem& S = *reinterpret_cast<PrSmem*>(smem_raw);
  uint8_t* ring = smem_raw + sizeof(PrSmem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, half = P.rope.rotary_dim / 2;
  const int heads = P.hq + 2 * P.hkv, row = heads * HD * 2;
  volatile int* dead = &S.dead;
  if (tid == 0) {
    for (int s = 0; s < depth; ++s) {
      mbar_init(&S.full[s], 1);
      mbar_init(&S.empty[s], PR_WARPS);
    }
    S.dead = 0;
    fence_mbar_init();
  }
  grid_launch_dependents();
  grid_wait_prior();
  __syncthreads();
  // tokens blockIdx.x + i gridDim.x, i = 0, 1, ...
  const int mine = (P.n_tokens - blockIdx.x + gridDim.x - 1) / gridDim.x;
  if (warp >= PR_TEAMS * PR_WARPS) {
    // Each loading warp takes every PR_LOADERS-th token (a turn of the loop
    // costs it a quarter of a microsecond or more); it reads 32 of its tokens'
    // slots at once, and lanes 0, 1, 2 copy q, k, v.
    const int first = warp - PR_TEAMS * PR_WARPS;
    auto slot_of = [&](int n) {  // of this warp's n-th token
      const int i = first + n * PR_LOADERS;
      return i < mine ? P.slot[blockIdx.x + i * gridDim.x] : -1;
    };
    int s = first, slots = -1, ahead = slot_of(lane);
    uint32_t phase = 1;
    const uint16_t* src = lane == 0 ? P.q : lane == 1 ? P.k : P.v;
    const int64_t stride = lane == 0 ? P.q_stride : lane == 1 ? P.k_stride : P.v_stride;
    const int bytes = (lane == 0 ? P.hq : P.hkv) * HD * 2;
    const int dst = (lane == 0 ? 0 : lane == 1 ? P.hq : P.hq + P.hkv) * HD * 2;
    for (int i = first, n = 0; i < mine; i += PR_LOADERS, ++n) {
      if ((n & 31) == 0) {
        slots = ahead;
        ahead = slot_of(n + 32 + lane);
      }
      const int t = blockIdx.x + i * gridDim.x, slot = __shfl_sync(0xffffffffu, slots, n & 31);
      wait_phase(&S.empty[s], phase, dead, P.status);
      if (*dead) break;
      const bool use = slot >= 0 && slot < P.n_slots;
      if (lane == 0) {
        if (slot >= P.n_slots) latch(P.status, MK_ERR_BOUNDS);
        S.slot[s] = use ? slot : -1;
        if (use) mbar_arrive_expect_tx(&S.full[s], row);
        else mbar_arrive(&S.full[s]);
      }
      __syncwarp();
      if (use && lane < 3) bulk_in(ring + (size_t)s * row + dst, src + t * stride, bytes, &S.full[s]);
      s += PR_LOADERS;
      if (s >= depth) {
        s -= depth;
        phase ^= 1;
      }
    }
    if (*dead) {
      const uint64_t t0 = globaltimer();
      while (globaltimer() - t0 < 1000000ull) {  // the copies in flight land
      }
    }
    return;
  }
  const int team = warp / PR_WARPS, sub = warp % PR_WARPS, tt = tid % PR_TEAM;
  Lane L(P, lane);
  // this thread's pair (read once: the words lie in the constant bank, which
  // gives a warp's 32 different words one after another)
  const bool turns = tt < half;
  const uint64_t turn = turns ? P.rope.turn[tt] : 0;
  const int32_t* pos_row = P.pos + (turns ? P.rope.axis[tt] * P.pos_stride : 0) + blockIdx.x;
  auto position = [&](int i) { return turns && i < mine ? pos_row[i * gridDim.x] : 0; };
  int pos = position(team), buf = 0;
  for (int i = team; i < mine; i += PR_TEAMS, buf ^= 1) {
    const int t = blockIdx.x + i * gridDim.x, s = i % depth;
    if (turns) S.cs[team][buf][Lane::place(tt)] = pair_turn(pos, turn);
    pos = position(i + PR_TEAMS);
    named_bar(1 + team, PR_TEAM);
    L.angles(S.cs[team][buf], lane);
    wait_phase(&S.full[s], (i / depth) & 1, dead, P.status);
    const int slot = S.slot[s];
    if (slot >= 0 && !*dead) {
      const uint8_t* src = ring + (size_t)s * row;
      const TokenOut<HD> out(P, t, slot);
#pragma unroll 1
      for (int hb = sub * HPW; hb < heads; hb += PR_WARPS * HPW) {
        const int h = hb + lane / Lane::G;
        const uint4* w = reinterpret_cast<const uint4*>(src + min(h, heads - 1) * HD * 2);
        const uint4 wa = w[L.ca], wb = w[L.cb];
        uint4 a = wa, b = wb;
        if (hb < P.hq + P.hkv) L.apply(P, a, b, h < P.hq);
        if (h < heads) {
          const bool value = h >= P.hq + P.hkv;
          uint4* dst = out.head(P, h);
          dst[L.ca] = value ? wa : a;
          dst[L.cb] = value ? wb : b;
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.empty[s]);
  }
}

// The ring from two tokens an SM on (400 tokens of 32 + 16 heads of 128: 5.6 us
// against 7.2 us; 304: 5.3 against 4.8), for rows of which it holds eight.
template <int HD, bool BF>
cudaError_t append_launch(const PagedAppendParams& p, int device, int sms, cudaStream_t st) {
  const int row = (p.hq + 2 * p.hkv) * HD * 2, depth = ring_depth(row);
  if (p.n_tokens <= 2 * sms || depth == 0)
    return paged_launch(paged_append_kernel<HD, BF>, p.n_tokens, PA_THREADS, 0, st, p);
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = paged_prepare((const void*)paged_append_ring_kernel<HD, BF>, 232448, 0, device, &ready);
  if (e != cudaSuccess) return e;
  return paged_launch(paged_append_ring_kernel<HD, BF>, sms, PR_THREADS, (int)sizeof(PrSmem) + depth * row, st, p, depth);
}

// ---------------------------------------------------------------- attention
// Which kernel takes which request is a rule on its rows (new tokens x query
// heads per kv head); both walk the same device arrays and leave the other's
// requests out, so that a step may mix them.
cudaError_t attention_launch(PagedAttnParams& p, const PagedKv& kv, int d, bool bf, void* workspace,
                             cudaStream_t st) {
  int dev = 0, sms = 0;
  cudaError_t e = device_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  p.device = dev;
  p.rep_inv = (65536 + p.rep - 1) / p.rep;
  // The few-row kernel has the rows of the longest request where it takes them
  // all, else those of a single token (its products cost by the row: with 32 rows
  // 16 requests of 8 drafted tokens over 3-8K keys took it 105 us, the tile kernel
  // 67; with 9 to 16 rows it is ahead, 16 query heads on a kv head at 4096 keys 19
  // against 27 us).
  const int64_t most = (int64_t)p.max_new * p.rep;
  const bool all_few = most <= 16;
  const int want = all_few ? (int)most : p.rep;
  p.few_rows = want <= 8 ? 8 : want <= 16 ? 16 : 0;
  // rows a pair has at most: a warp each in the join, or several for one
  p.join_shares = !all_few || want > 4 ? 0 : want > 2 ? 1 : want > 1 ? 2 : 3;
  // workspace: descriptions, maxima and sums, outputs of the two kernels' parts
  const int ctas = std::min(sms, 224);
  uint8_t* w = (uint8_t*)workspace;
  PagedParts few{}, chunk{};
  few.rt = 16;
  chunk.rt = 256;
  few.ctas = p.few_rows ? ctas : 0;
  chunk.ctas = all_few ? 0 : ctas;
  few.desc = (PartDesc*)w;
  chunk.desc = few.desc + ctas;
  few.ml = (float2*)(chunk.desc + ctas);
  chunk.ml = few.ml + (size_t)2 * ctas * few.rt;
  few.o = (float*)(chunk.ml + (size_t)2 * ctas * chunk.rt);
  chunk.o = few.o + (size_t)2 * ctas * few.rt * d;
  static_assert(224 * (2 * 16 + 2 * (16 + 256) * (8 + 128 * 4)) <= MK_PAGED_WORKSPACE_BYTES, "workspace");
  if (few.ctas) e = paged_few_launch(p, kv, few, d, bf, st);
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
  // a token's heads are counted in bytes in 32 bits
  if (c->n_q_heads > MK_PAGED_MAX_HEADS || c->n_kv_heads > MK_PAGED_MAX_HEADS) return MK_ERR_UNSUPPORTED;
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
  if ((int64_t)b->n * b->max_blocks > 0x7fffffffll || (int64_t)b->max_blocks * b->page_size > (1ll << 30))
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
  if (!ctx_lens || !new_lens || !n_free || !n_left || free_capacity < 0 ||
      (free_capacity > 0 && !free_pages) || (b->max_tokens > 0 && (!b->positions || !b->slots)))
    return MK_ERR_INVALID_ARG;
  const void* ptrs[] = {ctx_lens, new_lens, free_pages, n_free, n_left, status, b->positions, b->slots};
  for (const void* p : ptrs)
    if (!al4(p)) return MK_ERR_INVALID_ARG;
  // A block may still read the lengths when another has written its part: what
  // is written shares no word with anything else of the call.
  const struct { const int32_t* at; int64_t words; } arrays[] = {
      {b->block_table, (int64_t)b->n * b->max_blocks}, {b->cu_new, b->n + 1}, {b->kv_lens, b->n},
      {b->positions, b->max_tokens}, {b->slots, b->max_tokens}, {n_left, 1}, {status, status ? 1 : 0},
      {ctx_lens, b->n}, {new_lens, b->n}, {free_pages, free_capacity}, {n_free, 1}};
  constexpr int n_arrays = sizeof(arrays) / sizeof(arrays[0]), n_written = 7;
  for (int i = 0; i < n_written; ++i)
    for (int j = i + 1; j < n_arrays; ++j)
      if (arrays[i].words > 0 && arrays[j].words > 0 &&
          (uintptr_t)arrays[i].at < (uintptr_t)arrays[j].at + 4 * arrays[j].words &&
          (uintptr_t)arrays[j].at < (uintptr_t)arrays[i].at + 4 * arrays[i].words)
        return MK_ERR_INVALID_ARG;
  PagedTablesParams p{};
  p.ctx = ctx_lens; p.add = new_lens; p.free_pages = free_pages; p.n_free = n_free;
  p.table = b->block_table; p.cu = b->cu_new; p.kv = b->kv_lens; p.pos = b->positions;
  p.slot = b->slots; p.n_left = n_left; p.status = status;
  p.n = b->n; p.max_blocks = b->max_blocks; p.max_tokens = b->max_tokens;
  p.free_cap = free_capacity; p.page_shift = log2_page(b->page_size);
  const size_t smem = PtSmem::bytes(b->n);
  if (smem > 49152) {  // the limit is the process's: set once, to the most a call takes
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
      e = paged_prepare((const void*)paged_tables_kernel, (int)PtSmem::bytes(MK_PAGED_MAX_REQUESTS), 0, dev, &ready);
    if (e != cudaSuccess) return done(e);
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
  cudaStream_t st = (cudaStream_t)stream;
  int dev = 0, sms = 0;
  cudaError_t e = device_sms(&dev, &sms);
  if (e == cudaSuccess) {
    if (c->dtype == MK_BF16)
      e = c->head_dim == 128 ? append_launch<128, true>(p, dev, sms, st) : append_launch<64, true>(p, dev, sms, st);
    else
      e = c->head_dim == 128 ? append_launch<128, false>(p, dev, sms, st) : append_launch<64, false>(p, dev, sms, st);
  }
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
  if (((q_stride | out_stride) & 7) || q_stride < qw || out_stride < qw || q_stride >= (1ll << 38) || window < 0 ||
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
  // units of work (key blocks and overheads of tiles or requests) are counted in 32
  // bits; their bound itself may pass 64
  const double tiles = (double)((int64_t)b->max_tokens * p.rep / 64 + b->n);
  if (tiles * c->n_kv_heads * (double)((int64_t)b->max_blocks * b->page_size / 64 + 4) > 2147483647.0)
    return MK_ERR_UNSUPPORTED;
  const PagedKv kv = {c->k, c->v, c->page_stride, c->head_stride, c->token_stride,
                      c->n_pages, c->n_kv_heads, c->page_size};
  const cudaError_t e = attention_launch(p, kv, c->head_dim, c->dtype == MK_BF16, c->workspace, (cudaStream_t)stream);
  return done(e);
}
