// Trees of drafted tokens: masks and positions of their rows, and which of them
// stand against the target's probabilities (include/mk.h).
#include <algorithm>

#include "mk_paged_dev.cuh"

namespace mk {
namespace {

// ---------------------------------------------------------------- masks, positions
// A CTA per request (and some for the rows behind the last one): its parents go to
// shared memory, a thread takes a row and a word of its mask and walks up.  Parents
// precede their children, so a walk ends below its word.  Latency bound for shallow
// trees (32 of 16 tokens 2.0 us, 256 of up to 128 with four words a row 4.4 us, one of
// 512 at random 38).  A path is walked once for each word of its row, a step a read of
// shared memory: chains take words x nodes^2 steps, 128 with four words 10.3 us, with
// 16 31.6, 256 with eight 60, 512 with 16 437, 1024 with 32 3.4 ms.
constexpr int TT_THREADS = 128;

struct TreeParams {
  const int32_t *cu, *kv, *parents;
  uint32_t* masks;
  int32_t *pos, *status;
  int n, rows, words;
};

__global__ void __launch_bounds__(TT_THREADS) paged_tree_kernel(const TreeParams P) {
  __shared__ int up[MK_TREE_MAX_NODES];
  const int tid = threadIdx.x, r = blockIdx.x;
  grid_launch_dependents();
  grid_wait_prior();
  if (r >= P.n) {  // rows of no request: behind every offset
    __shared__ int behind;
    if (tid == 0) behind = 0;
    __syncthreads();
    int most = 0;
    for (int i = tid; i <= P.n; i += TT_THREADS) most = max(most, P.cu[i]);
    atomicMax(&behind, most);
    __syncthreads();
    const int end = min(behind, P.rows);
    for (int t = end + (r - P.n) * TT_THREADS + tid; t < P.rows; t += (gridDim.x - P.n) * TT_THREADS) P.pos[t] = 0;
    return;
  }
  const int c0 = P.cu[r], c1 = P.cu[r + 1], kv = P.kv[r], k = c1 - c0;
  const bool below = begins_below(P.cu, r, c0);
  if (below || c0 < 0 || c1 < c0 || c1 > P.rows) {
    if (tid == 0) latch(P.status, MK_ERR_BOUNDS);
    return;
  }
  const bool here = kv >= k;
  const int ctx = kv - k;
  if (k > 32 * P.words) {
    for (int i = tid; i < k; i += TT_THREADS) P.pos[c0 + i] = here ? ctx + i : 0;
    return;
  }
  for (int i = tid; i < k; i += TT_THREADS) {
    const int u = P.parents[c0 + i];
    const bool ok = u >= -1 && u < i;
    if (!ok) latch(P.status, MK_ERR_BOUNDS);
    up[i] = ok ? u : -1;
  }
  __syncthreads();
  for (int x = tid; x < k * P.words; x += TT_THREADS) {
    const int i = x / P.words, w = x - i * P.words;
    uint32_t bits = 0;
    int depth = 0;
    for (int a = i; a >= 32 * w; a = up[a]) {
      if (a < 32 * w + 32) bits |= 1u << (a & 31);
      ++depth;
    }
    P.masks[(int64_t)c0 * P.words + x] = bits;
    if (w == 0) P.pos[c0 + i] = here ? ctx + depth - 1 : 0;
  }
}

// ---------------------------------------------------------------- verification
// A cluster of CTAs per request.  Its first CTA reads the probabilities of all
// drafted tokens (two of each, at once), walks the tree and says which row's rest
// is to be summed; all of them sum their share of the vocabulary.  A chain (and a chunk
// of a prompt, where nothing is walked) needs one such pass, to draw its last token; a tree one more for every refused child that has
// siblings behind it.  For q >= 0 the rest after several refusals is
// max(p - S q, 0) with S the sum of the Z so far (max(max(a, 0) - b, 0) =
// max(a - b, 0)), so that a pass reads the two rows and keeps nothing.
//
// Probabilities are summed as whole numbers in units of 2^-43, each rounded once: the
// order of a sum does not matter, so the token is the same whatever the cluster, and a
// sum of 150000 is off by 2^-36 (32-bit floats would be off by 2^-24 at each of the
// places between two tokens).  x = hi 2^-22 + lo comes from adding 3: the bits of x + 3
// are hi, the rest is exact and gets its bits in the same way; six instructions, of
// which none is 64 bits wide.  p - S q has its parts subtracted, with the product's
// rounding error from a second multiply-add.  (64-bit whole numbers, 40 instructions a
// pair of values, took 32 trees 68 us instead of 39.)  Bound by latency for few requests
// (one of five rows of 128256 7.6 us), by HBM (the rows that are drawn from) and these
// instructions for many: 64 chains without draft probabilities 12.6 us, 32 trees of 17
// to 32 tokens of 151936, in up to five passes, 38.3 us.  256 threads with four
// vectors of each row in flight, two CTAs an SM: 512 with two 51 us, with eight in
// flight 39.2.
constexpr int TV_THREADS = 256, TV_WARPS = TV_THREADS / 32;
constexpr int TV_U = 4, TV_BATCH = 64 * TV_U;  // vectors in flight a lane and row (of one row twice as many)

struct VerifyParams {
  const int32_t *cu, *kv, *parents, *tokens;
  const float *p, *q, *u, *u_last;
  int32_t *path, *emitted, *kept, *lens, *status;
  int64_t p_stride, q_stride;
  int n, rows, vocab;
  int words;  // requests of more than 32 words new tokens are chunks of prompts; 0: none is
};

__device__ __forceinline__ float probability(float x) { return __saturatef(x); }  // NaN: 0

// x in [0, 1) as a fraction of 2^64, rounded down.
__device__ __forceinline__ u64 fraction(float x) {
  const uint32_t b = __float_as_uint(x);
  const int sh = (int)(b >> 23) - 86;
  const u64 m = (b & 0x7fffffu) | 0x800000u;
  return sh >= 0 ? m << sh : sh > -24 ? m >> -sh : 0;
}

// S, what the draft's row is multiplied by: none (0), 1, or hi + lo.
struct Refusals {
  float hi, lo;
  __device__ __forceinline__ Refusals(double s) : hi((float)s), lo((float)(s - (double)(float)s)) {}
};
// Sum of whole numbers: hi in units of 2^-22, lo of 2^-43 (some 250 values of up to
// 1 before it has to be taken out).
constexpr float HI_AT = 3.f, LO_AT = 0x1.8p-20f;
struct Units {
  int hi = 0, lo = 0;
  __device__ __forceinline__ void add(float x) {  // x in [0, 1]
    const float t = x + HI_AT, y = (x - (t - HI_AT)) + LO_AT;
    hi += __float_as_int(t) - __float_as_int(HI_AT);
    lo += __float_as_int(y) - __float_as_int(LO_AT);
  }
  // max(p - S q, 0)
  template <bool ONE>
  __device__ __forceinline__ void add(float p, float q, const Refusals& S) {
    float x = q, err = 0.f;
    if constexpr (!ONE) {
      x = S.hi * q;
      err = fmaf(S.lo, q, fmaf(S.hi, q, -x));
      x = fminf(x, 2.f);  // over any p all the same
    }
    const float tp = p + HI_AT, tx = x + HI_AT;
    const float lo_part = (p - (tp - HI_AT)) - (x - (tx - HI_AT)) - err;
    if ((tp - tx) + lo_part > 0.f) {
      hi += __float_as_int(tp) - __float_as_int(tx);
      lo += __float_as_int(lo_part + LO_AT) - __float_as_int(LO_AT);
    }
  }
  __device__ __forceinline__ u64 value() const { return (u64)(((int64_t)hi << 21) + lo); }
};
__device__ __forceinline__ u64 units(float x) {
  Units a;
  a.add(x);
  return a.value();
}
__device__ __forceinline__ u64 rest_units(float p, float q, double S) {
  Units a;
  if (S == 0.0) a.add(probability(p));
  else if (S == 1.0) a.add<true>(probability(p), probability(q), Refusals(S));
  else a.add<false>(probability(p), probability(q), Refusals(S));
  return a.value();
}

struct VerifyCtl {  // what the first CTA asks of the others
  int row, last, refused;  // last: 1 the pass that draws the last token, 2 nothing to draw
  int emitted;             // row that receives it
  double S;
};

struct VerifySmem {
  int up[MK_TREE_MAX_NODES], tok[MK_TREE_MAX_NODES], path[MK_TREE_MAX_NODES];
  float p[MK_TREE_MAX_NODES], q[MK_TREE_MAX_NODES], u[MK_TREE_MAX_NODES];
  uint32_t first[MK_TREE_MAX_NODES / 32];  // tokens that stand if none of their siblings has been refused
  int gone[MK_TREE_MAX_NODES];      // tokens found that were refused at this node, and their units
  u64 gone_units[MK_TREE_MAX_NODES];
  u64 warp_sum[TV_WARPS], total, scan[TV_WARPS];
  u64 piece[TV_WARPS][32];          // of a warp's share, 32 consecutive pieces' sums
  VerifyCtl ctl;
};

// Next child of `cur` from row `from` on; k where there is none (a warp together).
__device__ __forceinline__ int next_child(const int* up, int k, int cur, int from, int lane) {
  for (int b = from & ~31; b < k; b += 32) {
    const int i = b + lane;
    const uint32_t m = __ballot_sync(0xffffffffu, i >= from && i < k && up[i] == cur);
    if (m) return b + __ffs(m) - 1;
  }
  return k;
}

// Elements 4 v .. 4 v + 3 of a row, zeros past its end.  `wide`: the row is 16-byte
// aligned.
__device__ __forceinline__ float4 load4(const float* row, int v, int vocab, bool wide) {
  const int e = 4 * v;
  if (wide && e + 4 <= vocab) return __ldcg(reinterpret_cast<const float4*>(row + e));
  float4 x;
  x.x = e < vocab ? row[e] : 0.f;
  x.y = e + 1 < vocab ? row[e + 1] : 0.f;
  x.z = e + 2 < vocab ? row[e + 2] : 0.f;
  x.w = e + 3 < vocab ? row[e + 3] : 0.f;
  return x;
}

// A warp's sums of the rest over the vectors [v, v1): lane i gets the sum of the i-th
// piece of `piece` vectors (a multiple of 32 U; 32 of them cover all).  Lanes side by
// side, U vectors of each row in flight a lane.
enum { REST_P, REST_ONE, REST_S };
template <int U, int KIND>
__device__ __forceinline__ u64 sum_rest(const float* rp, const float* rq, double s, int v, int v1, int piece, int vocab, bool wide) {
  const Refusals S(s);
  const int lane = threadIdx.x & 31;
  u64 sum = 0, mine = 0;
  int left = piece, at = 0;
  for (v += lane; v - lane < v1; v += 32 * U) {
    float4 a[U], b[U];
    if (wide && v - lane + 32 * U <= min(v1, vocab / 4)) {
      // (without a branch between the loads)
#pragma unroll
      for (int i = 0; i < U; ++i) {
        a[i] = __ldcg(reinterpret_cast<const float4*>(rp) + v + 32 * i);
        b[i] = KIND != REST_P ? __ldcg(reinterpret_cast<const float4*>(rq) + v + 32 * i) : a[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        a[i] = b[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (v + 32 * i < v1) {
          a[i] = load4(rp, v + 32 * i, vocab, wide);
          if (KIND != REST_P) b[i] = load4(rq, v + 32 * i, vocab, wide);
        }
      }
    }
    Units x;
    auto one = [&](float p, float q) {
      if constexpr (KIND == REST_P) x.add(probability(p));
      else x.template add<KIND == REST_ONE>(probability(p), probability(q), S);
    };
#pragma unroll
    for (int i = 0; i < U; ++i) {
      one(a[i].x, b[i].x);
      one(a[i].y, b[i].y);
      one(a[i].z, b[i].z);
      one(a[i].w, b[i].w);
    }
    sum += x.value();
    left -= 32 * U;
    if (left == 0 || v - lane + 32 * U >= v1) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == at) mine = sum;
      sum = 0;
      left = piece;
      ++at;
    }
  }
  return mine;
}

// Of n <= 32 sums in the lanes, the first whose running sum passes *want; *want becomes
// what is left of it there, *all their sum.
__device__ __forceinline__ int find_sum(u64 mine, int n, int lane, u64* want) {
  u64 upto = lane < n ? mine : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  const uint32_t m = __ballot_sync(0xffffffffu, lane < n && upto > *want);
  const int at = m ? __ffs(m) - 1 : n - 1;
  const u64 before = __shfl_sync(0xffffffffu, upto - mine, at);
  *want -= before;
  return at;
}

__global__ void __launch_bounds__(TV_THREADS, 2) tree_verify_kernel(const VerifyParams P) {
  __shared__ VerifySmem S;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = cluster_rank(), ctas = cluster_size(), r = blockIdx.x / ctas;
  grid_launch_dependents();
  grid_wait_prior();
  float ul = P.u_last[r];
  ul = ul >= 1.f ? 0x1.fffffep-1f : fmaxf(ul, 0.f);
  // state of the walk, in the first CTA's first warp
  int k = 0, c0 = 0, kv = 0, cur = 0, depth = 0, at = 0, n_gone = 0;
  double sum_z = 0.0, z = 1.0;
  bool none = false;  // nothing to draw from: this request gets no token
  bool chunk = false;  // of a prompt: all of it stands, its last row says what follows
  if (rank == 0) {
    c0 = P.cu[r];
    const int c1 = P.cu[r + 1];
    kv = P.kv[r];
    k = c1 - c0;
    chunk = P.words > 0 && k > 32 * P.words;
    const bool below = begins_below(P.cu, r, c0), bad = below || c0 < 0 || c1 < c0 || c1 > P.rows || (k > MK_TREE_MAX_NODES && !chunk);
    none = bad || k == 0 || kv < k;
    if (none) {
      if (!bad)
        for (int i = tid; i < k; i += TV_THREADS) P.path[c0 + i] = P.emitted[c0 + i] = -1;
      if (tid == 0) {
        if (bad) latch(P.status, MK_ERR_BOUNDS);
        P.kept[r] = 0;
        P.lens[r] = kv;
      }
      k = 0;
      chunk = false;
    }
    for (int i = tid; i < (chunk ? 0 : (k + 31) & ~31); i += TV_THREADS) {
      int up = -1, x = -1;
      float p = 0.f, q = 0.f, u = 0.f;
      if (i > 0 && i < k) {
        up = P.parents[c0 + i];
        x = P.tokens[c0 + i];
        u = P.u[c0 + i];
        if (up < -1 || up >= i || x < 0 || x >= P.vocab) latch(P.status, MK_ERR_BOUNDS);
        if (up < 0 || up >= i) up = -1;
        if (x < 0 || x >= P.vocab) x = -1;
        if (up >= 0 && x >= 0) {
          p = probability(P.p[(c0 + up) * P.p_stride + x]);
          if (P.q) q = probability(P.q[(c0 + up) * P.q_stride + x]);
        }
      }
      u = u >= 1.f ? 0x1.fffffep-1f : fmaxf(u, 0.f);
      S.up[i] = up; S.tok[i] = x; S.p[i] = p; S.q[i] = q;
      S.u[i] = u;
      const uint32_t m = __ballot_sync(0xffffffffu, (double)u * (P.q ? (double)q : 1.0) < (double)p);
      if (lane == 0) S.first[i / 32] = m;
    }
    __syncthreads();
    if (chunk) {
      cur = depth = k - 1;
      at = k;
    } else if (warp == 0 && k > 0) {
      at = next_child(S.up, k, 0, 1, lane);
    }
  }

  const int vecs = (P.vocab + 3) / 4, per_cta = (vecs + ctas - 1) / ctas, per_warp = (per_cta + TV_WARPS - 1) / TV_WARPS;
  const int piece = ((per_warp + TV_BATCH - 1) / TV_BATCH + 31) / 32 * TV_BATCH;  // a multiple of what is in flight
  const int v_end = min(vecs, (rank + 1) * per_cta);
  auto warp_first = [&](int w) { return min(v_end, rank * per_cta + w * per_warp); };
  const uint32_t ctl0 = cluster_addr(&S.ctl, 0);
  for (;;) {
    if (rank == 0 && warp == 0) {
      while (at < k) {
        const int i = at, x = S.tok[i];
        bool again = false, stands;
        if (P.q ? sum_z == 0.0 : n_gone == 0) {
          stands = S.first[i / 32] >> (i & 31) & 1u;
        } else if (P.q) {
          const double left = fmax((double)S.p[i] - sum_z * (double)S.q[i], 0.0);
          stands = (double)S.u[i] * (double)S.q[i] * z < left;
        } else {
          for (int b = 0; b < n_gone; b += 32)
            again |= __any_sync(0xffffffffu, b + lane < n_gone && S.gone[min(b + lane, n_gone - 1)] == x);
          stands = (double)S.u[i] * z < (again ? 0.0 : (double)S.p[i]);
        }
        if (stands) {
          cur = i;
          ++depth;
          if (lane == 0) S.path[depth] = i;
          at = next_child(S.up, k, cur, i + 1, lane);
          sum_z = 0.0;
          z = 1.0;
          n_gone = 0;
          continue;
        }
        at = next_child(S.up, k, cur, i + 1, lane);
        if (P.q) {
          sum_z += z;
          if (at < k) break;  // its siblings are asked against the rest's sum
        } else if (!again && x >= 0) {
          if (lane == 0) {
            S.gone[n_gone] = x;
            S.gone_units[n_gone] = units(S.p[i]);
          }
          ++n_gone;
          z = fmax(z - (double)S.p[i], 0.0);
          __syncwarp();
        }
      }
      if (lane == 0) S.ctl = {c0 + cur, none ? 2 : at >= k, n_gone, c0 + depth, sum_z};
    }
    cluster_sync();
    VerifyCtl c;
    c.row = ld_cluster32(ctl0);
    c.last = ld_cluster32(ctl0 + 4);
    c.refused = ld_cluster32(ctl0 + 8);
    c.emitted = ld_cluster32(ctl0 + 12);
    c.S = __longlong_as_double((long long)ld_cluster64(ctl0 + 16));
    if (c.last == 2) break;
    const float* rp = P.p + c.row * P.p_stride;
    const float* rq = P.q ? P.q + c.row * P.q_stride : rp;
    const bool wide = ((uintptr_t)rp & 15) == 0 && ((uintptr_t)rq & 15) == 0;

    // sum of the rest over this CTA's share (a second time without refusals where
    // nothing of it is left)
    u64 total = 0, cta_total = 0;
    for (int pass = 0; pass < 2; ++pass) {
      const int v0 = warp_first(warp), v1 = warp_first(warp + 1);
      u64 sum = c.S == 0.0   ? sum_rest<2 * TV_U, REST_P>(rp, rq, 0.0, v0, v1, piece, P.vocab, wide)
                : c.S == 1.0 ? sum_rest<TV_U, REST_ONE>(rp, rq, 1.0, v0, v1, piece, P.vocab, wide)
                             : sum_rest<TV_U, REST_S>(rp, rq, c.S, v0, v1, piece, P.vocab, wide);
      if (c.last) S.piece[warp][lane] = sum;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) S.warp_sum[warp] = sum;
      __syncthreads();
      if (c.refused > 0) {  // without what was refused
        for (int g = tid; g < c.refused; g += TV_THREADS) {
          const int v = (int)ld_cluster32(cluster_addr(&S.gone[g], 0)) / 4;
          if (v / per_cta == rank) {
            const int w = (v - rank * per_cta) / per_warp;
            const u64 less = 0ull - ld_cluster64(cluster_addr(&S.gone_units[g], 0));
            atomicAdd(&S.warp_sum[w], less);
            if (c.last) atomicAdd(&S.piece[w][(v - warp_first(w)) / piece], less);
          }
        }
        __syncthreads();
      }
      if (warp == 0) {
        u64 t = lane < TV_WARPS ? S.warp_sum[lane] : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        if (lane == 0) S.total = t;
      }
      if (pass == 0 && c.last && rank == 0) {  // meanwhile, what the walk has found
        for (int j = tid; j < k; j += TV_THREADS) {
          const int d = c.emitted - c0;
          P.path[c0 + j] = j == 0 ? 0 : chunk ? j : j <= d ? S.path[j] : -1;
          if (j != d) P.emitted[c0 + j] = j < d && !chunk ? S.tok[S.path[j + 1]] : -1;
        }
        if (tid == 0) {
          P.kept[r] = c.emitted - c0 + 1;
          P.lens[r] = kv - k + c.emitted - c0 + 1;
        }
      }
      cluster_sync();
      cta_total = lane < ctas ? ld_cluster64(cluster_addr(&S.total, lane)) : 0;
      total = cta_total;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
      if (!c.last || total != 0 || pass == 1) break;
      c.S = 0.0;
      c.refused = 0;
      cluster_sync();  // the totals have been read
    }
    if (!c.last) {
      z = (double)total * 0x1p-43;
      continue;
    }
    // the last token: the element where the running sum passes u total
    u64 want = __umul64hi(total, fraction(ul));
    const int owner = find_sum(cta_total, ctas, lane, &want);
    int32_t* last = P.emitted + c.emitted;
    if (total == 0) {
      if (rank == 0 && tid == 0) {
        if (!chunk) latch(P.status, MK_ERR_BOUNDS);
        *last = chunk ? -1 : 0;
      }
    } else if (owner == rank) {
      const int w = find_sum(lane < TV_WARPS ? S.warp_sum[lane] : 0, TV_WARPS, lane, &want);
      const int part = find_sum(S.piece[w][lane], 32, lane, &want);
      const int v0 = min(warp_first(w) + part * piece, warp_first(w + 1)), v1 = min(v0 + piece, warp_first(w + 1));
      bool found = false;
      for (int b = v0; b < v1 && !found; b += TV_THREADS) {
        const int v = b + tid;
        u64 x[4] = {0, 0, 0, 0};
        if (v < v1) {
          const float4 a = load4(rp, v, P.vocab, wide), q = c.S != 0.0 ? load4(rq, v, P.vocab, wide) : a;
          x[0] = rest_units(a.x, q.x, c.S); x[1] = rest_units(a.y, q.y, c.S); x[2] = rest_units(a.z, q.z, c.S); x[3] = rest_units(a.w, q.w, c.S);
          for (int g = 0; g < c.refused; ++g) {
            const int t = (int)ld_cluster32(cluster_addr(&S.gone[g], 0));
            if (t / 4 == v) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if ((t & 3) == e) x[e] = 0;
            }
          }
        }
        const u64 mine = x[0] + x[1] + x[2] + x[3];
        u64 upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const u64 y = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += y;
        }
        if (lane == 31) S.scan[warp] = upto;
        __syncthreads();
        u64 all = 0;
        for (int y = 0; y < TV_WARPS; ++y) {
          if (y < warp) upto += S.scan[y];
          all += S.scan[y];
        }
        u64 before = upto - mine;
        const bool here = before <= want && want < upto;
        if (here) {
          int e = 0;
          while (e < 3 && want >= before + x[e]) before += x[e++];
          *last = 4 * v + e;
        }
        found = __syncthreads_or(here);
        want -= all;
      }
      // (sums that pass 2^64, of rows that are no probabilities, may miss it)
      if (!found && tid == 0) *last = min(max(4 * v1 - 1, 0), P.vocab - 1);
    }
    break;
  }
  cluster_sync();  // no CTA's shared memory is read any more
}

// CTAs of a request: as many as all requests' fit the GPU at once (two an SM), not
// powers of two alone (40 trees of 17 to 24 tokens of 128256 34.7 against 40.3 us, 80
// chains of 5 rows 22.6 against 27.4).
cudaError_t verify_launch(const VerifyParams& p, cudaStream_t st) {
  static std::atomic<int> known[64][17];
  int dev = 0, cluster = 16;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  while (cluster > 1 && p.n > paged_clusters_at_once((const void*)tree_verify_kernel, TV_THREADS, 0, dev, cluster, known)) --cluster;
  return paged_launch_clusters(tree_verify_kernel, p.n * cluster, cluster, TV_THREADS, 0, st, p);
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" int mk_paged_tree(const mk_paged_batch* b, const int32_t* parents, uint32_t* masks, int mask_words,
                             int32_t* positions, int32_t* status, void* stream) {
  const int rc = paged_check_batch(b);
  if (rc != MK_OK) return rc;
  if (!parents || !masks || !positions || mask_words < 1) return MK_ERR_INVALID_ARG;
  if (mask_words > MK_TREE_MAX_NODES / 32) return MK_ERR_UNSUPPORTED;
  const void* ptrs[] = {parents, masks, positions, status};
  for (const void* p : ptrs)
    if (!al4(p)) return MK_ERR_INVALID_ARG;
  const PagedWords arrays[] = {{masks, (int64_t)b->max_tokens * mask_words}, {positions, b->max_tokens},
                               {status, status ? 1 : 0}, {parents, b->max_tokens}, {b->cu_new, b->n + 1}, {b->kv_lens, b->n}};
  if (paged_overlap(arrays, 6, 3)) return MK_ERR_INVALID_ARG;
  if (b->max_tokens == 0) return MK_OK;
  TreeParams p{};
  p.cu = b->cu_new; p.kv = b->kv_lens; p.parents = parents; p.masks = masks; p.pos = positions; p.status = status;
  p.n = b->n; p.rows = b->max_tokens; p.words = mask_words;
  const int behind = min(64, (p.rows + 4 * TT_THREADS - 1) / (4 * TT_THREADS));
  return paged_done(paged_launch(paged_tree_kernel, p.n + behind, TT_THREADS, 0, (cudaStream_t)stream, p));
}

static int verify(const mk_paged_batch* b, int mask_words, const int32_t* parents, const int32_t* tokens,
                  const float* target_probs, int64_t target_stride, const float* draft_probs, int64_t draft_stride,
                  int vocab, const float* uniforms, const float* last_uniforms, int32_t* path, int32_t* emitted,
                  int32_t* kept, int32_t* lens, int32_t* status, void* stream) {
  const int rc = paged_check_batch(b);
  if (rc != MK_OK) return rc;
  if (!parents || !tokens || !target_probs || !uniforms || !last_uniforms || !path || !emitted || !kept || !lens || vocab < 1 ||
      target_stride < vocab || (draft_probs && draft_stride < vocab))
    return MK_ERR_INVALID_ARG;
  if (vocab > 1 << 24 || target_stride >= (1ll << 38) || (draft_probs && draft_stride >= (1ll << 38))) return MK_ERR_UNSUPPORTED;
  // the rows' extent in bytes is counted in 64 bits
  const int64_t most = (1ll << 60) / std::max(b->max_tokens, 1);
  if (target_stride > most || (draft_probs && draft_stride > most)) return MK_ERR_UNSUPPORTED;
  const void* ptrs[] = {parents, tokens, target_probs, draft_probs, uniforms, last_uniforms, path, emitted, kept, lens, status};
  for (const void* p : ptrs)
    if (!al4(p)) return MK_ERR_INVALID_ARG;
  const int64_t rows = b->max_tokens;
  const PagedWords arrays[] = {{path, rows}, {emitted, rows}, {kept, b->n}, {lens, b->n}, {status, status ? 1 : 0},
                               {parents, rows}, {tokens, rows}, {uniforms, rows}, {last_uniforms, b->n},
                               {target_probs, rows ? (rows - 1) * target_stride + vocab : 0},
                               {draft_probs, rows && draft_probs ? (rows - 1) * draft_stride + vocab : 0},
                               {b->cu_new, b->n + 1}, {b->kv_lens, b->n}};
  if (paged_overlap(arrays, 13, 5)) return MK_ERR_INVALID_ARG;
  VerifyParams p{};
  p.cu = b->cu_new; p.kv = b->kv_lens; p.parents = parents; p.tokens = tokens;
  p.p = target_probs; p.q = draft_probs; p.u = uniforms; p.u_last = last_uniforms;
  p.path = path; p.emitted = emitted; p.kept = kept; p.lens = lens; p.status = status;
  p.p_stride = target_stride; p.q_stride = draft_stride;
  p.n = b->n; p.rows = b->max_tokens; p.vocab = vocab; p.words = mask_words;
  return paged_done(verify_launch(p, (cudaStream_t)stream));
}

extern "C" int mk_tree_verify(const mk_paged_batch* b, const int32_t* parents, const int32_t* tokens,
                              const float* target_probs, int64_t target_stride, const float* draft_probs,
                              int64_t draft_stride, int vocab, const float* uniforms, const float* last_uniforms,
                              int32_t* path, int32_t* emitted, int32_t* kept, int32_t* lens, int32_t* status,
                              void* stream) {
  return verify(b, 0, parents, tokens, target_probs, target_stride, draft_probs, draft_stride, vocab, uniforms,
                last_uniforms, path, emitted, kept, lens, status, stream);
}

extern "C" int mk_tree_verify_mixed(const mk_paged_batch* b, int mask_words, const int32_t* parents, const int32_t* tokens,
                                    const float* target_probs, int64_t target_stride, const float* draft_probs,
                                    int64_t draft_stride, int vocab, const float* uniforms, const float* last_uniforms,
                                    int32_t* path, int32_t* emitted, int32_t* kept, int32_t* lens, int32_t* status,
                                    void* stream) {
  if (mask_words < 1) return MK_ERR_INVALID_ARG;
  if (mask_words > MK_TREE_MAX_NODES / 32) return MK_ERR_UNSUPPORTED;
  return verify(b, mask_words, parents, tokens, target_probs, target_stride, draft_probs, draft_stride, vocab, uniforms,
                last_uniforms, path, emitted, kept, lens, status, stream);
}
