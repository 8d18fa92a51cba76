// Pages of caches: who holds them, copies of them, and tokens that move within a
// request's pages (include/mk.h).
#include <algorithm>

#include "mk_paged_dev.cuh"

namespace mk {
namespace {

// ---------------------------------------------------------------- holders, free list
// One cluster.  Every CTA scans the requests into shared memory (as the step's
// tables do), so that the entries whose holders change are a flat list; the changes
// are added to shared[] atomically, which ends with the same counts in any order.
// A page that nobody holds then stands below zero.  Its place among the freed ones
// is that of the first entry that let it go, found by a minimum over the entries'
// numbers in the same word; entries that won are counted in order, and write their
// pages behind the free ones.  Latency bound: five barriers of the cluster, between
// them one or two round trips to L2 (16 beams of 63 pages 9.6 us, 256 requests that
// let 1100 entries go 9.7 us).  It is the same cluster for long contexts, whose entries
// are found again in every pass: 64 requests from 16 of 2048 pages 41 us, from 64 110.
constexpr int FK_THREADS = 512, FK_WARPS = FK_THREADS / 32, FK_CLUSTER = 8, FK_SLOTS = 2 * FK_THREADS;

struct ForkParams {
  const int32_t *table, *lens, *keep, *parents, *n_free;
  int32_t *next, *next_lens, *copies, *shared, *free_pages, *n_left, *status;
  int n, m, max_blocks, page_shift, n_pages, free_cap;
};

struct ForkSmem {
  int wa[FK_WARPS], wb[FK_WARPS];
  uint32_t freed[FK_CLUSTER];
  int key[FK_SLOTS], count[FK_SLOTS], least[FK_SLOTS];  // pages let go, how often, the first entry
  // then by request: whole [n] blocks that stay whole, and flags; held [n]; children
  // [n]; first [n] child; act [n + 1] entries whose holders may change before;
  // by new request: up [m]; need [m + 1] fresh pages before; pre [m + 1] entries of
  // next_table before
  static size_t bytes(int n, int m) { return sizeof(ForkSmem) + 4 * (5 * (size_t)n + 1 + 3 * (size_t)m + 2); }
};
constexpr int FK_PART = 1 << 27, FK_OWN = 1 << 28, FK_WHOLE = FK_PART - 1;

// Exclusive prefix sums of a[0 .. n) in place, a[n] their sum (a thread has
// consecutive ones).
__device__ __forceinline__ int scan_inplace(int* a, int n, int* tmp) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (n + FK_THREADS - 1) / FK_THREADS, i0 = min(tid * per, n), i1 = min(i0 + per, n);
  int sum = 0;
  for (int i = i0; i < i1; ++i) sum += a[i];
  int x = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) tmp[warp] = x;
  __syncthreads();
  int before = x - sum, all = 0;
  for (int w = 0; w < FK_WARPS; ++w) {
    if (w < warp) before += tmp[w];
    all += tmp[w];
  }
  for (int i = i0; i < i1; ++i) {
    const int v = a[i];
    a[i] = before;
    before += v;
  }
  if (tid == 0) a[n] = all;
  __syncthreads();
  return all;
}

__global__ void __launch_bounds__(FK_THREADS) paged_fork_kernel(const ForkParams P) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  ForkSmem& S = *reinterpret_cast<ForkSmem*>(smem_raw);
  int* whole = reinterpret_cast<int*>(&S + 1);
  int* held = whole + P.n;
  int* children = held + P.n;
  int* first = children + P.n;
  int* act = first + P.n;
  int* up = act + P.n + 1;
  int* need = up + P.m;
  int* pre = need + P.m + 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = cluster_rank(), ctas = cluster_size();
  const int page_mask = (1 << P.page_shift) - 1;
  const bool moving = P.parents != nullptr;
  grid_launch_dependents();
  grid_wait_prior();
  const int free_raw = *P.n_free, n_free = min(max(free_raw, 0), P.free_cap);
  bool bad = free_raw != n_free;

  for (int s = tid; s < P.n; s += FK_THREADS) {
    children[s] = 0;
    first[s] = P.m;
  }
  __syncthreads();
  for (int i = tid; i < P.m; i += FK_THREADS) {
    int u = moving ? P.parents[i] : i;
    if (u < -1 || u >= P.n) {
      bad = true;
      u = -1;
    }
    up[i] = u;
    if (u >= 0) {
      atomicAdd(&children[u], 1);
      atomicMin(&first[u], i);
    }
  }
  __syncthreads();
  auto entry = [&](int s, int b) { return P.table[(int64_t)s * P.max_blocks + b]; };
  auto is_page = [&](int p) { return p >= 0 && p < P.n_pages; };
  // tokens of request s, and what stays of them
  auto cut = [&](int s, int* len, bool* wrong) {
    const int l = P.lens[s], most = min((int64_t)P.max_blocks << P.page_shift, (int64_t)0x7fffffff);
    *len = min(max(l, 0), most);
    const int k = P.keep ? P.keep[s] : *len, kk = min(max(k, 0), *len);
    *wrong = *len != l || kk != k;
    return kk;
  };
  for (int s = tid; s < P.n; s += FK_THREADS) {
    int len;
    bool wrong;
    const int keep = cut(s, &len, &wrong), f = keep >> P.page_shift, c = children[s];
    bad |= wrong;
    const bool part = keep & page_mask;
    bool own = false;
    if (part && c > 0) {
      const int p = entry(s, f);
      own = !is_page(p) || __ldcg(P.shared + p) == 0;
    }
    held[s] = (int)(((int64_t)len + page_mask) >> P.page_shift);
    whole[s] = f | (part ? FK_PART : 0) | (own ? FK_OWN : 0);
    act[s] = c == 1 ? held[s] - f - own : held[s];
  }
  __syncthreads();
  const int E = scan_inplace(act, P.n, S.wa);
  for (int i = tid; i < P.m; i += FK_THREADS) {
    const int u = up[i];
    need[i] = u >= 0 && (whole[u] & FK_PART) && !((whole[u] & FK_OWN) && first[u] == i);
  }
  __syncthreads();
  const int wanted = scan_inplace(need, P.m, S.wb), taken = min(wanted, P.copies ? n_free : 0);
  bad |= taken < wanted;
  if (moving) {
    for (int i = tid; i < P.m; i += FK_THREADS) {
      const int u = up[i];
      pre[i] = u < 0 ? 0 : (whole[u] & FK_WHOLE) + ((whole[u] & FK_PART) && !(need[i + 1] > need[i] && need[i] >= taken));
    }
    __syncthreads();
  }
  const int rows = moving ? scan_inplace(pre, P.m, S.wa) : 0;
  cluster_sync();  // the counts that decide have been read
  // the holders' changes; an entry's own is -1, 0 or children - 1
  struct Entry {
    int s, b, page, change;
  };
  auto at = [&](int e) {
    Entry x;
    x.s = find_le(act, P.n, e);
    const int w = whole[x.s], f = w & FK_WHOLE, c = children[x.s];
    x.b = e - act[x.s] + (c == 1 ? f + ((w & FK_OWN) != 0) : 0);
    x.page = entry(x.s, x.b);
    x.change = x.b < f ? c - 1 : x.b == f && (w & FK_OWN) ? 0 : -1;
    if (!is_page(x.page)) {
      x.page = -1;
      x.change = 0;
    }
    return x;
  };
  // Few changes in place (a step's rejected tokens): one CTA makes them, a thread an
  // entry.  What lets go of the same page is counted in shared memory, so that each page
  // is one atomic (32 requests: the steps below, for any number, 9.4 us, this 5.8).
  if (!moving && E <= FK_THREADS) {
    if (rank > 0) return;
    for (int i = tid; i < FK_SLOTS; i += FK_THREADS) {
      S.key[i] = -1;
      S.count[i] = 0;
      S.least[i] = FK_THREADS;
    }
    Entry x{0, 0, -1, 0};
    int fresh = -1;
    if (tid < E) {
      x = at(tid);
      bad |= x.page < 0;
      if (x.b == (whole[x.s] & FK_WHOLE) && need[x.s + 1] > need[x.s] && need[x.s] < taken) fresh = P.free_pages[n_free - 1 - need[x.s]];
    }
    for (int i = tid; i < P.m; i += FK_THREADS) {
      bool wrong;
      int len, from = -1, to = -1, copied = 0, tokens = cut(i, &len, &wrong);
      if (need[i + 1] > need[i]) {
        if (need[i] < taken) {
          from = entry(i, whole[i] & FK_WHOLE);
          to = P.free_pages[n_free - 1 - need[i]];
          copied = tokens & page_mask;
        } else {
          tokens &= ~page_mask;
        }
      }
      P.next_lens[i] = tokens;
      if (P.copies) {
        P.copies[i] = from;
        P.copies[P.m + i] = to;
        P.copies[2 * P.m + i] = copied;
      }
    }
    __syncthreads();  // the table and the free list's end have been read
    int at_slot = -1;
    if (x.change < 0) {
      for (uint32_t h = (uint32_t)x.page * 2654435761u;; ++h) {  // (no more pages than half of the slots)
        at_slot = (int)(h % FK_SLOTS);
        const int was = atomicCAS(&S.key[at_slot], -1, x.page);
        if (was == -1 || was == x.page) break;
      }
      atomicAdd(&S.count[at_slot], 1);
      atomicMin(&S.least[at_slot], tid);
    }
    if (fresh >= 0) P.next[(int64_t)x.s * P.max_blocks + x.b] = fresh;
    __syncthreads();
    bool won = false;
    if (at_slot >= 0 && S.least[at_slot] == tid) {
      const int left = atomicAdd(P.shared + x.page, -S.count[at_slot]) - S.count[at_slot];
      won = left < 0;
      bad |= left < -1;
      if (won) P.shared[x.page] = 0;
    }
    const uint32_t m = __ballot_sync(0xffffffffu, won);
    if (lane == 0) S.wb[warp] = __popc(m);
    __syncthreads();
    int to = n_free - taken + __popc(m & ((1u << lane) - 1)), all = n_free - taken;
    for (int w = 0; w < FK_WARPS; ++w) {
      if (w < warp) to += S.wb[w];
      all += S.wb[w];
    }
    if (won && to < P.free_cap) P.free_pages[to] = x.page;
    if (tid == 0) {
      *P.n_left = min(all, P.free_cap);
      bad |= all > P.free_cap;
    }
    if (bad) latch(P.status, MK_ERR_BOUNDS);
    return;
  }
  const int gtid = rank * FK_THREADS + tid, gsize = ctas * FK_THREADS;

  // a warp's entries are consecutive; where they are at most 32 they stay in registers
  const int G = ctas * FK_WARPS, len = ((E + G - 1) / G + 31) & ~31, w0 = rank * FK_WARPS + warp;
  const int e0 = (int)min((int64_t)w0 * len, (int64_t)E), e1 = (int)min((int64_t)e0 + len, (int64_t)E);
  Entry kept{0, 0, -1, 0};
  if (len == 32 && e0 + lane < e1) kept = at(e0 + lane);
  auto get = [&](int e) { return len == 32 ? kept : at(e); };
  for (int e = e0 + lane; e < e1; e += 32) {
    const Entry x = get(e);
    if (x.page < 0) bad = true;
    else if (x.change != 0 && atomicAdd(P.shared + x.page, x.change) + x.change < -1) bad = true;
  }
  for (int j = gtid; j < rows; j += gsize) {
    const int i = find_le(pre, P.m, j), b = j - pre[i], u = up[i];
    const bool fresh = need[i + 1] > need[i] && b == (whole[u] & FK_WHOLE);
    P.next[(int64_t)i * P.max_blocks + b] = fresh ? P.free_pages[n_free - 1 - need[i]] : entry(u, b);
  }
  for (int i = gtid; i < P.m; i += gsize) {
    const int u = up[i];
    int tokens = 0, from = -1, to = -1, copied = 0;
    if (u >= 0) {
      bool wrong;
      tokens = cut(u, &from, &wrong);
      from = -1;
      if (need[i + 1] > need[i]) {
        if (need[i] < taken) {
          from = entry(u, whole[u] & FK_WHOLE);
          to = P.free_pages[n_free - 1 - need[i]];
          copied = tokens & page_mask;
        } else {
          tokens &= ~page_mask;
        }
      }
    }
    P.next_lens[i] = tokens;
    if (P.copies) {
      P.copies[i] = from;
      P.copies[P.m + i] = to;
      P.copies[2 * P.m + i] = copied;
    }
  }
  cluster_sync();  // all changes are in
  for (int e = e0 + lane; e < e1; e += 32) {
    const Entry x = get(e);
    if (x.change < 0 && __ldcg(P.shared + x.page) < 0) atomicMin(P.shared + x.page, -2 - (E - 1 - e));
  }
  cluster_sync();  // the first entry of each page is known
  auto won = [&](const Entry& x, int e) { return x.change < 0 && __ldcg(P.shared + x.page) == -2 - (E - 1 - e); };
  int mine = 0;
  uint32_t kept_won = 0;
  for (int b = e0; b < e1; b += 32) {
    const int e = b + lane;
    kept_won = __ballot_sync(0xffffffffu, e < e1 && won(get(e), e));
    mine += __popc(kept_won);
  }
  if (lane == 0) S.wb[warp] = mine;
  __syncthreads();
  if (tid < ctas) {
    int t = 0;
    for (int w = 0; w < FK_WARPS; ++w) t += S.wb[w];
    st_cluster32(cluster_addr(&S.freed[rank], tid), (uint32_t)t);
  }
  cluster_sync();  // every CTA knows all counts
  int pos = n_free - taken, all = pos;
  for (int x = 0; x < ctas; ++x) {
    if (x < rank) pos += (int)S.freed[x];
    all += (int)S.freed[x];
  }
  for (int w = 0; w < warp; ++w) pos += S.wb[w];
  for (int b = e0; b < e1; b += 32) {
    const int e = b + lane;
    Entry x{0, 0, -1, 0};
    if (e < e1) {
      x = get(e);
      // in place: a page of its own for one filled in part that others hold (named
      // in copies: the free list's end may have been written by now)
      const int f = whole[x.s] & FK_WHOLE;
      if (!moving && x.b == f && need[x.s + 1] > need[x.s] && need[x.s] < taken)
        P.next[(int64_t)x.s * P.max_blocks + f] = __ldcg(P.copies + P.m + x.s);
    }
    const uint32_t m = len == 32 ? kept_won : __ballot_sync(0xffffffffu, e < e1 && won(x, e));
    if (m >> lane & 1u) {
      P.shared[x.page] = 0;
      const int to = pos + __popc(m & ((1u << lane) - 1));
      if (to < P.free_cap) P.free_pages[to] = x.page;
    }
    pos += __popc(m);
  }
  if (rank == 0 && tid == 0) {
    *P.n_left = min(all, P.free_cap);
    bad |= all > P.free_cap;
  }
  if (bad) latch(P.status, MK_ERR_BOUNDS);
}

// ---------------------------------------------------------------- layers
struct Layers {
  uint16_t* kv[2 * MK_PAGED_MAX_LAYERS];  // keys, values of each layer in turn
  int64_t page_stride, head_stride, token_stride;
  int32_t* status;
  int hkv, n_pages, page_shift, lanes, lane_shift;  // lanes: 16-byte pieces of a head, log2 of it
};

// ---------------------------------------------------------------- copies of pages
// Bound by HBM.  Where the tokens of a head lie end to end (or a token's heads and the
// tokens) what is copied of a page is a few spans: a warp copies up to 64 KB of them
// through shared memory with bulk copies, three warps an SM in turn.  (16 bytes a thread
// and load, as below, spends 70% of the issue slots on addresses: 56 pages of 64
// tokens in 32 layers 68 us, 55 with spans.)
constexpr int PC_SPANS = 65536;  // bytes of a CTA

__global__ void __launch_bounds__(32) paged_copy_spans_kernel(const __grid_constant__ Layers L, const int32_t* copies, int n, int groups, int per, int span,
                                                              bool tokens_first) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ uint64_t bar;
  __shared__ volatile int dead;
  const int lane = threadIdx.x;
  if (lane == 0) {
    mbar_init(&bar, 1);
    dead = 0;
    fence_mbar_init();
  }
  grid_launch_dependents();
  grid_wait_prior();
  __syncwarp();
  const int i = blockIdx.x / groups, s = (blockIdx.x - i * groups) * per + lane, page = 1 << L.page_shift;
  const int from = copies[i], to = copies[n + i];
  if (from == -1) return;
  int tokens = copies[2 * n + i];
  const bool bad = from < 0 || from >= L.n_pages || to < 0 || to >= L.n_pages;
  if ((bad || tokens < 0 || tokens > page) && lane == 0) latch(L.status, MK_ERR_BOUNDS);
  if (bad) return;
  tokens = min(max(tokens, 0), page);
  // this lane's span: a head's tokens, or `span` bytes of the tokens
  const int64_t row = (int64_t)L.lanes * 16;
  int64_t at, len;
  if (tokens_first) {
    at = (int64_t)s * span;
    len = min((int64_t)span, tokens * row * L.hkv - at);
  } else {
    at = s * L.head_stride * 2;
    len = s < L.hkv ? tokens * row : 0;
  }
  if (lane >= per || len < 0) len = 0;
  const uint32_t mine = (uint32_t)len;
  uint32_t all = mine;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
  if (all == 0) return;
  uint8_t* base = reinterpret_cast<uint8_t*>(L.kv[blockIdx.y]);
  uint8_t* buf = smem_raw + (int64_t)lane * span;
  if (lane == 0) mbar_arrive_expect_tx(&bar, all);
  __syncwarp();
  if (mine) bulk_in(buf, base + from * L.page_stride * 2 + at, mine, &bar);
  wait_phase(&bar, 0, &dead, L.status);
  if (dead) {  // leave after the loads, none of which takes a millisecond, have landed
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 1000000ull) {
    }
    return;
  }
  if (mine) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(base + to * L.page_stride * 2 + at), "r"(smem_u32(buf)), "r"(mine) : "memory");
    asm volatile("cp.async.bulk.commit_group;\ncp.async.bulk.wait_group.read 0;" ::: "memory");
  }
}

// Any layout: a row is one head of one token, and each thread has all its loads in
// flight at once.
constexpr int PC_COPY_THREADS = 256, PC_UNROLL = 4;

__global__ void __launch_bounds__(PC_COPY_THREADS) paged_copy_kernel(const __grid_constant__ Layers L, const int32_t* copies, int n, int parts) {
  grid_launch_dependents();
  grid_wait_prior();
  const int i = blockIdx.x / parts, part = blockIdx.x - i * parts;
  const int from = copies[i], to = copies[n + i];
  if (from == -1) return;
  int tokens = copies[2 * n + i];
  const int page = 1 << L.page_shift;
  const bool bad = from < 0 || from >= L.n_pages || to < 0 || to >= L.n_pages;
  if ((bad || tokens < 0 || tokens > page) && threadIdx.x == 0) latch(L.status, MK_ERR_BOUNDS);
  if (bad) return;
  tokens = min(max(tokens, 0), page);
  uint16_t* base = L.kv[blockIdx.y];
  const uint16_t* src = base + from * L.page_stride;
  uint16_t* dst = base + to * L.page_stride;
  if (tokens == 0) return;
  // row / tokens by its reciprocal: the error, row 2^-32 at most, is below 1 / tokens (rows
  // are below 2^24, tokens at most 2^8, and an exact quotient's error is none of below)
  const uint32_t inv = 0xffffffffu / (uint32_t)tokens + 1;
  const int total = L.hkv * tokens * L.lanes, step = parts * PC_COPY_THREADS;
  for (int x0 = part * PC_COPY_THREADS + threadIdx.x; x0 < total; x0 += PC_UNROLL * step) {
    uint4 v[PC_UNROLL];
    int64_t at[PC_UNROLL];
#pragma unroll
    for (int k = 0; k < PC_UNROLL; ++k) {
      const int x = x0 + k * step;
      if (x < total) {
        const int row = x >> L.lane_shift, c = x & (L.lanes - 1), h = tokens == 1 ? row : (int)__umulhi((uint32_t)row, inv), t = row - h * tokens;
        at[k] = h * L.head_stride + t * L.token_stride + c * 8;
        v[k] = __ldcs(reinterpret_cast<const uint4*>(src + at[k]));
      }
    }
#pragma unroll
    for (int k = 0; k < PC_UNROLL; ++k)
      if (x0 + k * step < total) __stcs(reinterpret_cast<uint4*>(dst + at[k]), v[k]);
  }
}

// ---------------------------------------------------------------- tokens that stay
// A CTA takes one request and a share of the columns (a 16-byte piece of a head, keys
// or values of one layer): the path's moves are worked out once, in shared memory, and
// a thread makes them all for its columns, four loads in flight.  Paths increase, so
// that no token is read after another has been moved to its place.  (A CTA for each
// request and layer, which works the path out for itself: 256 requests in 16 layers
// 24.5 us instead of 13.9.)
constexpr int PK_THREADS = 256, PK_AHEAD = 4, PK_MOVES = 256;

__global__ void __launch_bounds__(PK_THREADS, 6) paged_keep_kernel(const __grid_constant__ Layers L, const int32_t* cu, const int32_t* slots, const int32_t* path, int rows, int columns) {
  __shared__ int64_t from_at[PK_MOVES], to_at[PK_MOVES];
  __shared__ int n_moves, stop;
  const int tid = threadIdx.x, lane = tid & 31;
  grid_launch_dependents();
  grid_wait_prior();
  const int r = blockIdx.x, c0 = cu[r], c1 = cu[r + 1];
  const bool below = begins_below(cu, r, c0);
  if (below || c0 < 0 || c1 < c0 || c1 > rows) {
    if (tid == 0) latch(L.status, MK_ERR_BOUNDS);
    return;
  }
  const int k = c1 - c0, page_mask = (1 << L.page_shift) - 1, pieces = L.hkv * L.lanes;
  const int64_t n_slots = (int64_t)L.n_pages << L.page_shift;
  auto place = [&](int slot) { return (slot >> L.page_shift) * L.page_stride + (slot & page_mask) * L.token_stride; };
  if (tid == 0) stop = k;
  for (int j0 = 0; j0 < k; j0 += PK_MOVES) {
    if (tid == 0) n_moves = 0;
    __syncthreads();
    // the first entry that ends the path
    const int j = j0 + tid;
    int from = -1, before = -1;
    if (j < k) {
      from = path[c0 + j];
      if (j > 0) before = path[c0 + j - 1];
      if (from <= before || from < 0 || from >= k) atomicMin(&stop, j);
    }
    __syncthreads();
    if (j == stop && j < k && from != -1) latch(L.status, MK_ERR_BOUNDS);
    bool move = j < stop && from != j;
    int s = 0, d = 0;
    if (move) {
      s = slots[c0 + from];
      d = slots[c0 + j];
      if (s >= n_slots || d >= n_slots) latch(L.status, MK_ERR_BOUNDS);
      move = s >= 0 && d >= 0 && s < n_slots && d < n_slots;
    }
    // in the order of the path: a warp's moves behind those of the warps before
    const uint32_t m = __ballot_sync(0xffffffffu, move);
    for (int w = 0; w < PK_THREADS / 32; ++w) {
      if (tid >> 5 == w) {
        const int at = n_moves;
        __syncwarp();
        if (move) {
          from_at[at + __popc(m & ((1u << lane) - 1))] = place(s);
          to_at[at + __popc(m & ((1u << lane) - 1))] = place(d);
        }
        if (lane == 0) n_moves = at + __popc(m);
      }
      __syncthreads();
      if (j0 + 32 * (w + 1) >= min(stop, k)) break;
    }
    const int n = n_moves;
    for (int x = blockIdx.y * PK_THREADS + tid; x < columns && n > 0; x += gridDim.y * PK_THREADS) {
      const int layer = x / pieces, y = x - layer * pieces, h = y / L.lanes;
      uint16_t* base = L.kv[layer] + h * L.head_stride + (y - h * L.lanes) * 8;
      for (int i0 = 0; i0 < n; i0 += PK_AHEAD) {
        uint4 v[PK_AHEAD];
#pragma unroll
        for (int i = 0; i < PK_AHEAD; ++i)
          if (i0 + i < n) v[i] = *reinterpret_cast<const uint4*>(base + from_at[i0 + i]);
#pragma unroll
        for (int i = 0; i < PK_AHEAD; ++i)
          if (i0 + i < n) *reinterpret_cast<uint4*>(base + to_at[i0 + i]) = v[i];
      }
    }
    if (stop < j0 + PK_MOVES) break;
    __syncthreads();
  }
}

int fill_layers(const mk_paged_cache* c, void* const* ks, void* const* vs, int n, Layers* L) {
  int rc = paged_check_cache(c);
  if (rc != MK_OK) return rc;
  if (!ks || !vs || n < 1) return MK_ERR_INVALID_ARG;
  if (n > MK_PAGED_MAX_LAYERS) return MK_ERR_UNSUPPORTED;
  for (int l = 0; l < n; ++l) {
    if (!ks[l] || !vs[l] || !al16(ks[l]) || !al16(vs[l])) return MK_ERR_INVALID_ARG;
    L->kv[2 * l] = (uint16_t*)ks[l];
    L->kv[2 * l + 1] = (uint16_t*)vs[l];
  }
  L->page_stride = c->page_stride; L->head_stride = c->head_stride; L->token_stride = c->token_stride;
  L->status = c->status;
  L->hkv = c->n_kv_heads; L->n_pages = c->n_pages; L->page_shift = paged_log2(c->page_size); L->lanes = c->head_dim / 8;
  L->lane_shift = c->head_dim == 128 ? 4 : 3;
  return MK_OK;
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" int mk_paged_fork(const int32_t* table, int n, const int32_t* lens, const int32_t* keep, const int32_t* parents,
                             int32_t* next_table, int32_t* next_lens, int m, int max_blocks, int page_size,
                             int32_t* copies, int32_t* shared, int n_pages, int32_t* free_pages, int free_capacity,
                             const int32_t* n_free, int32_t* n_left, int32_t* status, void* stream) {
  if (!table || !lens || !next_table || !next_lens || !shared || !n_free || !n_left || n < 1 || m < 1 || max_blocks < 1 ||
      n_pages < 1 || free_capacity < 0 || (free_capacity > 0 && !free_pages))
    return MK_ERR_INVALID_ARG;
  if (!parents && (m != n || next_table != table)) return MK_ERR_INVALID_ARG;
  const int shift = paged_log2(page_size);
  if (n > MK_PAGED_MAX_REQUESTS || m > MK_PAGED_MAX_REQUESTS || shift < 0 || (int64_t)std::max(n, m) * max_blocks > 0x7fffffffll ||
      (int64_t)max_blocks * page_size > (1ll << 30))
    return MK_ERR_UNSUPPORTED;
  const void* ptrs[] = {table, lens, keep, parents, next_table, next_lens, copies, shared, free_pages, n_free, n_left, status};
  for (const void* p : ptrs)
    if (!al4(p)) return MK_ERR_INVALID_ARG;
  const bool same = n_left == n_free;
  const PagedWords arrays[] = {{next_table, (int64_t)m * max_blocks}, {next_lens, m}, {copies, copies ? 3 * (int64_t)m : 0}, {shared, n_pages},
                               {free_pages, free_capacity}, {n_left, 1}, {status, status ? 1 : 0},
                               {table, parents ? (int64_t)n * max_blocks : 0}, {lens, n}, {keep, keep ? n : 0}, {parents, parents ? m : 0},
                               {n_free, same ? 0 : 1}};
  if (paged_overlap(arrays, 12, 7)) return MK_ERR_INVALID_ARG;
  ForkParams p{};
  p.table = table; p.lens = lens; p.keep = keep; p.parents = parents; p.n_free = n_free;
  p.next = next_table; p.next_lens = next_lens; p.copies = copies; p.shared = shared; p.free_pages = free_pages;
  p.n_left = n_left; p.status = status;
  p.n = n; p.m = m; p.max_blocks = max_blocks; p.page_shift = shift; p.n_pages = n_pages; p.free_cap = free_capacity;
  const size_t smem = ForkSmem::bytes(n, m);
  if (smem > 49152) {  // the limit is the process's: set once, to the most a call takes
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
      e = paged_prepare((const void*)paged_fork_kernel, (int)ForkSmem::bytes(MK_PAGED_MAX_REQUESTS, MK_PAGED_MAX_REQUESTS), 0, dev, &ready);
    if (e != cudaSuccess) return paged_done(e);
  }
  return paged_done(paged_launch_clusters(paged_fork_kernel, FK_CLUSTER, FK_CLUSTER, FK_THREADS, (int)smem, (cudaStream_t)stream, p));
}

extern "C" int mk_paged_copy(const mk_paged_cache* c, void* const* ks, void* const* vs, int n_layers,
                             const int32_t* copies, int n_copies, void* stream) {
  Layers L{};
  const int rc = fill_layers(c, ks, vs, n_layers, &L);
  if (rc != MK_OK) return rc;
  if (!copies || !al4(copies) || n_copies < 0) return MK_ERR_INVALID_ARG;
  if (n_copies > MK_PAGED_MAX_REQUESTS) return MK_ERR_UNSUPPORTED;
  if (n_copies == 0) return MK_OK;
  const int row = L.lanes * 16;
  // spans: the heads' tokens, or the tokens' heads, end to end
  const bool heads_first = c->token_stride == c->head_dim, tokens_first = !heads_first && c->head_stride == c->head_dim && c->token_stride == (int64_t)c->n_kv_heads * c->head_dim;
  if (heads_first || tokens_first) {
    const int64_t bytes = (int64_t)c->page_size * c->n_kv_heads * row;
    const int span = heads_first ? c->page_size * row : (int)std::min<int64_t>(16384, bytes);
    const int64_t spans = heads_first ? c->n_kv_heads : (bytes + span - 1) / span;
    const int per = (int)std::min<int64_t>({32, PC_SPANS / span, spans});
    const int64_t groups = (spans + per - 1) / per;
    if (groups * n_copies <= 0x7fffffff) {
      static std::atomic<uint64_t> ready{0};
      int dev = 0;
      cudaError_t e = cudaGetDevice(&dev);
      if (e == cudaSuccess) e = paged_prepare((const void*)paged_copy_spans_kernel, PC_SPANS, 0, dev, &ready);
      if (e != cudaSuccess) return paged_done(e);
      cudaLaunchConfig_t cfg{};
      cudaLaunchAttribute at{};
      at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
      at.val.programmaticStreamSerializationAllowed = 1;
      cfg.gridDim = dim3((int)(groups * n_copies), 2 * n_layers);
      cfg.blockDim = dim3(32);
      cfg.dynamicSmemBytes = per * span;
      cfg.stream = (cudaStream_t)stream;
      cfg.attrs = &at;
      cfg.numAttrs = 1;
      return paged_done(cudaLaunchKernelEx(&cfg, paged_copy_spans_kernel, L, copies, n_copies, (int)groups, per, span, tokens_first));
    }
  }
  const int64_t pieces = (int64_t)c->n_kv_heads * c->page_size * L.lanes;
  const int parts = (int)std::min<int64_t>(64, (pieces + PC_COPY_THREADS * PC_UNROLL - 1) / (PC_COPY_THREADS * PC_UNROLL));
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(n_copies * parts, 2 * n_layers);
  cfg.blockDim = dim3(PC_COPY_THREADS);
  cfg.stream = (cudaStream_t)stream;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return paged_done(cudaLaunchKernelEx(&cfg, paged_copy_kernel, L, copies, n_copies, parts));
}

extern "C" int mk_paged_keep(const mk_paged_cache* c, void* const* ks, void* const* vs, int n_layers,
                             const mk_paged_batch* b, const int32_t* path, void* stream) {
  Layers L{};
  int rc = fill_layers(c, ks, vs, n_layers, &L);
  if (rc == MK_OK) rc = paged_check_batch(b);
  if (rc != MK_OK) return rc;
  if (!path || !al4(path) || b->page_size != c->page_size || (b->max_tokens > 0 && (!b->slots || !al4(b->slots)))) return MK_ERR_INVALID_ARG;
  if (b->max_tokens == 0) return MK_OK;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  // some sixteen CTAs an SM, with work for each thread
  const int64_t columns = (int64_t)2 * n_layers * c->n_kv_heads * L.lanes;
  const int shares = (int)std::min<int64_t>((columns + PK_THREADS - 1) / PK_THREADS, std::max(1, 16 * 152 / b->n));
  cfg.gridDim = dim3(b->n, shares);
  cfg.blockDim = dim3(PK_THREADS);
  cfg.stream = (cudaStream_t)stream;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return paged_done(cudaLaunchKernelEx(&cfg, paged_keep_kernel, L, (const int32_t*)b->cu_new, (const int32_t*)b->slots, path, (int)b->max_tokens, (int)columns));
}
