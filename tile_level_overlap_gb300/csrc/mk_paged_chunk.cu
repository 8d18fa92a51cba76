// Attention over a paged cache for requests with many rows: chunks of prompts.
//
// Bound by the tensor cores: 4 head_dim flops per (row, key).  A tile is up to
// 256 rows of one (request, kv head), as two halves of 128: whole tokens, each
// with all query heads of the kv head, so that one load of a key block serves
// them all.  The work is the list of key blocks (128 keys) of all tiles, end
// to end, after the causal bound and the window; each persistent CTA (one per
// SM) takes an equal run of it, and rows whose keys lie in several runs are
// joined as in the few-row kernel.  Measured with 32 query heads on 8 kv heads of
// 128: a prompt of 8192 tokens 363 us (1514 TFLOP/s; 385 us, 1428, without a pause,
// when the power limit holds the clock at 1.94 GHz), of 16384 1390 us (1580), 2 x 512
// tokens over 4-12K cached keys 104 us; a block of keys takes 3050 cycles, 2048 of
// them products.
//
// Warps of a CTA: two load (TMA: queries, K and V blocks page by page, 128-byte
// swizzle), one for each half issues tcgen05.mma, two groups of four own
// a half each (thread = row).  Per half and block: S = Q K^T into 128 TMEM columns; its
// group reads the row, masks it where the block crosses a bound, exponentiates
// relative to a running maximum and writes P over S in the cache's type (one
// rounding a weight: a second product for what it drops would cost half of the
// tensor time); O += P V with P read from TMEM.  The two halves alternate on the tensor cores: while
// one's softmax runs the other's products do.  The maximum that P is relative
// to is only moved when it has grown by more than 2^8 (the known lazy form of the
// online softmax: P stays inside the 16-bit range and sums are fp32), so O, which
// lives in TMEM, is seldom rescaled.
// No wait on O is needed for that: S of block j is issued behind P V of block
// j - 1, so when S is complete O is at rest.
//
// The kernel's other forms take trees of drafted tokens, whose rows see the cached keys
// and the new ones that their masks name: the masks change the blocks that hold new
// tokens, as four words of bits a row.  Bound by HBM where tiles have one half
// (2 x 16 tokens over 128K keys 166 us, 6.5 TB/s), else by the softmax as above (1.8 us
// a block, HBM 1.5).  Forms, their rules and figures stand at the kernel, is_pair,
// paged_chunk_clusters and the join.
#include "mk_paged_dev.cuh"
#include "mk_paged_tc.cuh"
#include "mk_tmap.h"

namespace mk {
namespace {

constexpr int PC_THREADS = 384;
constexpr int PC_LOAD = 8, PC_MMA = 9, PC_LOAD_V = 11;  // warps (9, 10: products); 0-3 and 4-7 own the halves
constexpr int PC_SPLIT_V = 5;                // log2 of the page size from which one warp loads K and V
constexpr int PC_REGS = 168, PC_REGS_SOFT = 216, PC_REGS_REST = 72;
static_assert(2 * PC_REGS_SOFT + PC_REGS_REST == 3 * PC_REGS, "registers of the three warpgroups");
// What a tile costs beside its blocks (filling the pipeline, writing the rows),
// in blocks: without it the SMs with the short tiles of a prompt's start ended
// a quarter later than the others.  Of trees 1, their blocks take longer (1.7 us, a tile
// 2: with 2 blocks a mixed step 40.6 us, with 1 39.4, with none 42.5; 32 requests over
// 500 to 2000 keys 63.5, 62.9, 65.6).
constexpr int PC_OVER = 2, PC_OVER_TREE = 1;
// P is relative to a maximum that may lag by 2^PC_LAG.  In fp16 it is scaled by
// 2^PC_TOP_FP16 besides (together 2^15): weights lose bits only 2^21 or more below
// the row's largest, and are lost 2^32 or more below it, instead of 2^14 and 2^25.
constexpr float PC_LAG = 8.f, PC_TOP_FP16 = 7.f;

template <int HD>
struct ChunkCfg {
  static constexpr int TILE = 128 * HD * 2;                // 128 rows or keys
  static constexpr int STAGES = HD == 128 ? 4 : 8;         // K and V blocks in turn
  static constexpr int SLOTS = 2;
  static constexpr int o_kv = 2 * TILE;                    // after the queries' halves
  static constexpr int o_meta = o_kv + STAGES * TILE;
  static constexpr int o_bar = o_meta + SLOTS * 64;
  static constexpr int o_pre = o_bar + 320;
  static constexpr int total(int n) { return o_pre + Kept::bytes(n); }
  static constexpr int most = o_pre + KEPT_MOST;
};
static_assert(ChunkCfg<128>::most <= 232448 && ChunkCfg<64>::most <= 232448, "shared memory of a CTA");

constexpr int PART_PAIR = 1 << 30;  // in a PartDesc's head: rows of two heads, the second's from 128 on

struct Tile {
  int key0, nblk;          // first key of the run; 0 blocks: the end
  int row0, ntok, head;    // first token (row of q), tokens of the tile
  int pos0;                // position of the first token
  int lo, hi;              // keys the request's rows may see
  int part;                // workspace part, -1: all of the tile's blocks
  int req;                 // its request
  int ctx;                 // of a tree: its cached tokens; else -2^31
  int pair;                // the halves are two heads' rows, from `head` on
  int pad[4];
};
static_assert(sizeof(Tile) == 64, "meta slot");

// Whether a request's rows have masks.
template <bool TREE>
__device__ __forceinline__ bool is_tree(const PagedAttnParams& P, const Request& q) {
  return TREE && q.add <= 32 * P.mask_words;
}

// Trees of at most 128 rows go in pairs of kv heads, where heads are 64 wide and of even
// number: a tile's halves are the rows of two heads, whose blocks take turns in the
// ring.  Alone a half's softmax takes more than the 0.73 us that HBM needs of a block
// (32 requests of 13 tokens over 2048 keys 43.2 us alone, with the halves' S in turn,
// 37.4 in pairs).  Of 128-wide heads HBM needs 1.47: pairs only make the parts larger
// (32 of 32 over 1280 48.4 alone, without turns, 54.8 in pairs).
template <bool PAIRS>
__device__ __forceinline__ bool is_pair(const PagedAttnParams& P, const Request& q, int TS) {
  return PAIRS && (P.hkv & 1) == 0 && q.add <= TS;
}

// First block and number of blocks of tile t of a request (TT tokens a tile).  Any
// row of a tree may stand where its root does.
template <bool TREE>
__device__ __forceinline__ int tile_blocks(const PagedAttnParams& P, const Request& q, int t, int TT, int* first) {
  const int p0 = q.pos0 + (is_tree<TREE>(P, q) ? 0 : t * TT), p1 = q.pos0 + min(q.add, (t + 1) * TT);
  const int hi = min(max(p1, 0), q.hi);
  const int lo = p0 >= P.window ? min(p0 - P.window + 1, hi) : 0;
  *first = lo / 128;
  return max(1, (hi + 127) / 128 - lo / 128);
}

// First of n blocks that CTA k of a cluster takes (the first ones have one more: the
// last blocks, with masks, take longer).
__device__ __forceinline__ int share_of(int n, int k, int ctas) { return (n * k + ctas - 1) / ctas; }

__device__ __forceinline__ void let_land() {
  const uint64_t t0 = globaltimer();
  while (globaltimer() - t0 < 1000000ull) {
  }
}

// Lanes l and l ^ D exchange: the lower one's b for the upper one's a.
template <int D>
__device__ __forceinline__ void quad_swap(uint32_t (&a)[4], uint32_t (&b)[4], int lane) {
  const bool up = lane & D;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? a[i] : b[i], D);
    if (up) a[i] = got;
    else b[i] = got;
  }
}

// TREE: rows of requests with masks see the cached keys and the new ones that their
// masks name.  FORM: runs of all tiles' blocks, the same where no tile has two halves, or
// a cluster for each tile.  In the last two a tile of one half has the S of both in turn:
// the next block's product is there when a block's softmax ends, which else takes a
// chain of 1.4 us a block of 128-wide heads (32 x 32 tokens over 8192 keys 186.4 -> 182.7
// us, over 1280 48.9 -> 47.2, one of 32 over 4096 14.0 -> 13.2; 20 heads on 5 of 64, 32 x
// 13 over 2048 35.6 -> 31.6).  A block's P may then be written before that of the one
// before has been seen, so P has barriers in turn too; a rescaled O waits for the last
// P V.  Where tiles of both kinds meet, the second half's S would have to change hands
// (32 requests of 1 to 64 tokens 63.2 -> 64.8 us).
enum { RUNS, RUNS_OF_HALVES, CLUSTERS };
template <int HD, bool BF, bool TREE, int FORM>
__global__ void __launch_bounds__(PC_THREADS, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv, const __grid_constant__ PagedAttnParams P,
                       const __grid_constant__ PagedParts W) {
  using C = ChunkCfg<HD>;
  constexpr int ST = C::STAGES;
  constexpr bool PAIRS = TREE && FORM == RUNS && HD == 64, TURNS = FORM != RUNS;
  constexpr int OVER = TREE ? PC_OVER_TREE : PC_OVER;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::o_bar);
  uint64_t* empty = full + ST;
  uint64_t* qfull = empty + ST;
  uint64_t* qempty = qfull + 1;
  uint64_t* mfull = qempty + 1;
  uint64_t* mempty = mfull + C::SLOTS;
  uint64_t* sfull = mempty + C::SLOTS;   // S of half h complete
  uint64_t* pfull = sfull + 2;           // P of half h written
  uint64_t* ofull = pfull + 2;           // O of half h complete
  volatile int* dead = reinterpret_cast<volatile int*>(ofull + 2);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(const_cast<int*>(dead) + 1);
  int* joined = reinterpret_cast<int*>(tslot + 1);  // [4] a cluster's tile: rows, first token, blocks, head
  uint64_t* pdone = reinterpret_cast<uint64_t*>(joined + 4);  // both halves have seen the loads of a pair
  uint64_t* sturn = pdone + 1;  // blocks in turns: S of turn b complete
  uint64_t* oturn = sturn + 2;  // P V of turn b complete
  uint64_t* pturn = oturn + 2;  // P of turn b written
  static_assert((2 * ST + 2 + 2 * C::SLOTS + 6) * 8 + 8 + 16 + 8 + 48 <= C::o_pre - C::o_bar, "barriers");
  Tile* meta = reinterpret_cast<Tile*>(smem + C::o_meta);
  const Kept kept(smem + C::o_pre, P.n);
  int* pre = kept.pre;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int TS = 128 / P.rep, TT = 2 * TS;  // tokens of a half, of a tile
  const bool split_v = P.page_shift < PC_SPLIT_V;

  grid_launch_dependents();
  if (TREE && tid >= 32 && tid < 35)  // (their first use would wait for them)
    asm volatile("prefetch.tensormap [%0];" ::"l"(tid == 32 ? &tk : tid == 33 ? &tv : &tq) : "memory");
  if (tid == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 2);
    }
    mbar_init(qfull, 1);
    mbar_init(qempty, 2);
    for (int s = 0; s < C::SLOTS; ++s) {
      mbar_init(&mfull[s], 1);
      mbar_init(&mempty[s], split_v ? 11 : 10);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(&sfull[h], 1);
      mbar_init(&pfull[h], 4);
      mbar_init(&ofull[h], 1);
    }
    if (PAIRS) mbar_init(pdone, 2);
    if (TURNS)
      for (int b = 0; b < 2; ++b) {
        mbar_init(&sturn[b], 1);
        mbar_init(&oturn[b], 1);
        mbar_init(&pturn[b], 4);
      }
    *dead = 0;
    fence_mbar_init();
  }
  // query rows that no token fills (128 % rep) stay zero
  for (int i = tid; i < 2 * C::TILE / 16; i += PC_THREADS)
    reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (warp == PC_MMA) tmem_alloc(tslot, 512);
  // (Behind the few-row kernel this waits for all of it.  What is read here was
  // written before that one's own wait, but a grid is promised to see it only by
  // waiting itself: mixed step of 27 requests 46.8 us, with the wait at the end 44.5.)
  grid_wait_prior();
  constexpr bool clustered = FORM == CLUSTERS;
  if (tid == 0 && !clustered) W.desc[blockIdx.x].parts = 0;

  // In clusters: this one's tile, of which the CTA takes blocks [cb0, cb1).
  Request cq;
  int cr = 0, ch = 0, ct = 0, cnb = 0, cb0 = 0, cb1 = 0, rank = 0;
  if constexpr (clustered) {
    const int tiles = (P.max_new + TT - 1) / TT, id = blockIdx.x / P.cluster;
    rank = (int)cluster_rank();
    cr = id / (P.hkv * tiles);
    ch = id / tiles - cr * P.hkv;
    ct = id % tiles;
    const int first = P.cu[cr];
    cq = make_request(P, first, P.cu[cr + 1], P.kv[cr]);
    if (begins_below(P.cu, cr, first)) cq.add = 0;
    int f;
    if ((int64_t)ct * TT < cq.add) cnb = tile_blocks<TREE>(P, cq, ct, TT, &f);
    cb0 = share_of(cnb, rank, P.cluster);
    cb1 = share_of(cnb, rank + 1, P.cluster);
    if (cq.bad && tid == 0) latch(P.status, MK_ERR_BOUNDS);
    if (tid == 0) {  // for the join
      joined[0] = cnb > 0 ? min(TT, cq.add - ct * TT) * P.rep : 0;
      joined[1] = cq.row0 + ct * TT;
      joined[2] = cnb;
      joined[3] = ch;
    }
  }

  // units: the tiles' blocks and overheads.  A thread counts its requests'
  // tiles; a warp together those of a request with many.
  const int per = clustered ? 0 : (P.n + PC_THREADS - 1) / PC_THREADS;
  uint32_t mine = 0;
  bool bad = false, falls = false;
  for (int i = 0; i < per; ++i) {
    const int r = tid * per + i;
    int u = 0, ntile = 0, b0;
    Request q{};
    if (r < P.n) {
      q = kept.read(P, r);
      bad |= q.bad;
      falls |= q.falls;
      if ((int64_t)q.add * P.rep > P.few_rows) ntile = (q.add + TT - 1) / TT;
    }
    if (ntile <= 8)
      for (int t = 0; t < ntile; ++t) u += tile_blocks<TREE>(P, q, t, TT, &b0);
    for (uint32_t many = __ballot_sync(0xffffffffu, ntile > 8); many; many &= many - 1) {
      const int from = __ffs(many) - 1;
      Request x{};
      x.add = __shfl_sync(0xffffffffu, q.add, from);
      x.pos0 = __shfl_sync(0xffffffffu, q.pos0, from);
      x.hi = __shfl_sync(0xffffffffu, q.hi, from);
      const int nt = __shfl_sync(0xffffffffu, ntile, from);
      int v = 0;
      for (int t = lane; t < nt; t += 32) v += tile_blocks<TREE>(P, x, t, TT, &b0);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == from) u = v;
    }
    u = (u + OVER * ntile) * (is_pair<PAIRS>(P, q, TS) ? P.hkv / 2 : P.hkv);
    if (r < P.n) pre[r] = u;
    mine += u;
  }
  int* scan_tmp = reinterpret_cast<int*>(smem + C::o_kv);  // not loaded to yet
  const int T = clustered ? 0 : place_units<PC_THREADS / 32>(P, pre, per, mine, falls, scan_tmp);
  if (bad && blockIdx.x == 0) latch(P.status, MK_ERR_BOUNDS);
  fence_proxy_async_smem();  // the scan's words, before a load takes their place
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // every column is this CTA's: the allocation starts at column 0
  constexpr uint32_t T_S = 0, T_O = 256;

  const int G = min((int)gridDim.x, T), c = blockIdx.x;
  const Runs runs(T, max(G, 1));
  const int u0 = c < G ? runs.start(c) : 0, u1 = clustered ? (cb0 < cb1 ? 1 : 0) : c < G ? runs.start(c + 1) : 0;

  // Values are loaded by a warp of their own where pages are of 16 tokens: a
  // block's keys and values are then 32 boxes of 2 KB, which one warp does not
  // issue in the block's time (2 x 512 tokens over 4-12K: 102 against 120 us;
  // 8192-token prompt: 366 against 448).  With larger boxes one warp is enough,
  // and the keys' and values' loads in turn disturb the products' reads of shared
  // memory less (prompt, pages of 32: 371 against 381 us, of 64: 374 against 411).
  if (warp >= PC_LOAD) {
    setmaxnreg_dec<PC_REGS_REST>();
    const int boxt = min(128, 1 << P.page_shift), nbox = 128 / boxt;
    // page of this lane's box of a block; -1 where no row of the request sees any of it
    auto seen = [&](int b, int lo, int hi) {
      const int key = b * 128 + lane * boxt;
      return lane < nbox && key < hi && key + boxt > lo;
    };
    auto entry_of = [&](const int32_t* tab, int b) { return tab[(b * 128 + lane * boxt) >> P.page_shift]; };
    auto page_in = [&](int p) {
      if (p >= 0 && p < P.n_pages) return p;
      latch(P.status, MK_ERR_BOUNDS);
      return -1;
    };
    auto page_of = [&](const int32_t* tab, int b, int lo, int hi) {
      const int key = b * 128 + lane * boxt;
      if (lane >= nbox || key >= hi || key + boxt <= lo) return -1;
      const int p = tab[key >> P.page_shift];
      if (p >= 0 && p < P.n_pages) return p;
      latch(P.status, MK_ERR_BOUNDS);
      return -1;
    };
    // Keys and values that only one tile reads leave L2 before the parts do, which the
    // join reads (32 x 32 tokens over 1280 keys 46.4 -> 44.1 us, over 8192 180 -> 174.7,
    // 16 x 32 over 4000 58.5 -> 53.8).  It is no loss beside a chunk of a prompt, whose tiles
    // read them again (16 x 16 with a chunk of 600 over 2000 keys 64.6 -> 62.3, over 8000 177
    // -> 173), it is one for trees of several tiles (4 x 160, 8 heads a kv head, 146.4 -> 148)
    // and where requests share pages in tiles of two halves (32 x 64 over the same 8192
    // tokens 222.9 -> 229.6; 32 x 32 144.6 -> 141).
    const uint64_t once = TREE ? policy_evict_first() : 0;
    // a block's keys or values into a stage
    auto load = [&](const CUtensorMap* tm, int stage, uint32_t phase, int b, int head, int page) {
      wait_phase(&empty[stage], phase, dead, P.status);
      if (*dead) return false;
      if (lane == 0) mbar_arrive_expect_tx(&full[stage], C::TILE);
      __syncwarp();
      if (lane < nbox) {
        uint8_t* dst = smem + C::o_kv + stage * C::TILE + lane * boxt * 128;
        const int tok = (b * 128 + lane * boxt) & ((1 << P.page_shift) - 1);
#pragma unroll
        for (int x = 0; x < HD / 64; ++x) {
          if constexpr (TREE) tma_page(dst + x * 16384, tm, tok, x, head, page, &full[stage], once);
          else tma_page(dst + x * 16384, tm, tok, x, head, page, &full[stage]);
        }
      }
      return true;
    };
    if (warp == PC_LOAD_V && split_v) {
      // ---------------------------------------------------------- loads of V
      int stage = 1, slot = 0;
      uint32_t sphase = 1, mphase = 0;
      for (;;) {
        wait_phase(&mfull[slot], mphase, dead, P.status);
        if (*dead) break;
        const Tile m = meta[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(&mempty[slot]);
        if (m.nblk == 0) break;
        if (++slot == C::SLOTS) { slot = 0; mphase ^= 1; }
        const int32_t* tab = P.table + (int64_t)m.req * P.max_blocks;
        const int b0 = m.key0 / 128;
        int page = page_of(tab, b0, m.lo, m.hi);
        bool up = true;
        for (int i = 0; i < m.nblk && up; ++i) {
          const int next = i + 1 < m.nblk ? page_of(tab, b0 + i + 1, m.lo, m.hi) : -1;
          for (int h = 0; h <= (PAIRS ? m.pair : 0) && up; ++h) {
            up = load(&tv, stage, sphase, b0 + i, m.head + h, page);
            stage += 2;
            if (stage > ST) { stage = 1; sphase ^= 1; }
          }
          page = next;
        }
        if (!up) break;
      }
      if (*dead) let_land();
    } else if (warp == PC_LOAD) {
      // ---------------------------------------------------------- tiles, loads of Q and K
      int stage = 0, slot = 0;
      uint32_t sphase = 1, mphase = 1, qphase = 1;
      const int step = split_v ? 2 : 1;
      int r = clustered ? cr : u0 < u1 ? find_le(pre, P.n, u0) : 0, t = clustered ? ct : -1, head = clustered ? ch : 0;
      bool up = true;
      for (int u = u0; u < u1 && up;) {
        while (!clustered && pre[r + 1] <= u) {
          ++r;
          t = -1;
        }
        Request q;
        if constexpr (clustered) q = cq;
        else q = kept.again(P, r);
        const bool pair = is_pair<PAIRS>(P, q, TS);
        const int per_head = clustered ? 1 : (pre[r + 1] - pre[r]) / (pair ? P.hkv / 2 : P.hkv), ntile = (q.add + TT - 1) / TT;
        int x0 = 0, b0;  // first unit of the tile in this run
        if (t < 0) {  // find the tile of unit u
          const int local = u - pre[r];
          head = local / per_head;
          int rem = local - head * per_head;
          for (int base = 0;; base += 32) {
            int f, k = 0;
            if (base + lane < ntile) k = tile_blocks<TREE>(P, q, base + lane, TT, &f) + OVER;
            int x = k;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const int y = __shfl_up_sync(0xffffffffu, x, o);
              if (lane >= o) x += y;
            }
            const uint32_t over = __ballot_sync(0xffffffffu, x > rem);
            if (over || base + 32 >= ntile) {
              const int l = over ? __ffs(over) - 1 : 31;
              t = base + l;
              x0 = rem - __shfl_sync(0xffffffffu, x - k, l);
              break;
            }
            rem -= __shfl_sync(0xffffffffu, x, 31);
          }
        }
        // units [x0, x1) of the tile: blocks [blk, blk + nblk)
        const int nb = tile_blocks<TREE>(P, q, t, TT, &b0), x1 = min(nb + OVER, x0 + u1 - u);
        const int blk = clustered ? cb0 : max(0, x0 - OVER), nblk = clustered ? cb1 - cb0 : max(0, x1 - OVER) - blk;
        const int ntok = min(TT, q.add - t * TT), end = u - x0 + nb + OVER;
        if (nblk == 0) break;  // the run ends with the tile's overhead: the next CTA has it all
        const int first_head = pair ? 2 * head : head;
        const bool whole = blk == 0 && nblk == nb;
        if (blk == 0 && !whole && lane == 0 && !clustered) {
          const int last = runs.of(end - 1);  // CTA of the tile's last unit
          PartDesc d;
          d.row0 = q.row0 + t * TT; d.rows = ntok * P.rep; d.head = first_head | (pair ? PART_PAIR : 0); d.parts = last - c + 1;
          W.desc[c] = d;
        }
        // (The queries' loads are written out at both places, and what only trees need is
        // left out at compile time: the compiler's order of the causal form's code depends
        // on it.  8192-token prompt 361 us so and before there were trees, 364 with a
        // lambda, with a function 2 more than that.)
        const int halves = pair || ntok > TS ? 2 : 1;
        const int q_head = first_head * P.rep, q_tok = q.row0 + t * TT, next_head = pair ? P.rep : 0, next_tok = pair ? 0 : TS;
        const int32_t* tab;
        int page;
        bool has_page;
        if constexpr (TURNS) {
          tab = P.table + (int64_t)r * P.max_blocks;
          page = -1;
          // The first tile's queries while its pages are read, before all SMs' first
          // blocks are on their way (32 x 32 tokens over 1280 keys 47.2 -> 46.3 us; runs with
          // tiles of two halves gain nothing, 1 to 64 tokens 63.2, 63.5).
          has_page = seen(b0 + blk, q.lo, q.hi);
          if (has_page) page = entry_of(tab, b0 + blk);
          if (u == u0) {
            qphase ^= 1;  // (nothing has to be waited for)
            if (lane == 0) {
              mbar_arrive_expect_tx(qfull, halves * (HD / 64) * TS * P.rep * 128);
              for (int y = 0; y < halves; ++y)
                for (int x = 0; x < HD / 64; ++x)
                  tma_rows(smem + y * C::TILE + x * 16384, &tq, 64 * x, q_head + y * next_head, q_tok + y * next_tok, qfull);
            }
            __syncwarp();
          }
        }
        wait_phase(&mempty[slot], mphase, dead, P.status);
        if (*dead) break;
        if (lane == 0) {
          Tile m;
          m.key0 = (b0 + blk) * 128; m.nblk = nblk; m.row0 = q.row0 + t * TT; m.ntok = ntok; m.head = first_head;
          if constexpr (TREE) m.pair = pair;
          m.pos0 = q.pos0 + t * TT; m.lo = q.lo; m.hi = q.hi;
          if constexpr (clustered) m.part = P.cluster > 1 ? -2 : -1;
          else m.part = whole ? -1 : 2 * c + (blk == 0 ? 1 : 0);
          m.req = r;
          if constexpr (TREE) m.ctx = is_tree<TREE>(P, q) ? q.pos0 : -0x7fffffff - 1;
          meta[slot] = m;
          mbar_arrive(&mfull[slot]);
        }
        if (++slot == C::SLOTS) { slot = 0; mphase ^= 1; }
        if constexpr (TURNS) {
          if (has_page) page = page_in(page);
        } else {
          tab = P.table + (int64_t)r * P.max_blocks;
          page = page_of(tab, b0 + blk, q.lo, q.hi);
        }
        for (int i = 0; i < nblk && up; ++i) {
          const int b = b0 + blk + i;
          const int next = i + 1 < nblk ? page_of(tab, b + 1, q.lo, q.hi) : -1;
          int h = 0;
          do {
            up = load(&tk, stage, sphase, b, first_head + h, page);
            stage += step;
            if (up && i == 0 && h == 0 && !(TURNS && u == u0)) {
              wait_phase(qempty, qphase, dead, P.status);
              qphase ^= 1;
              if (*dead) { up = false; break; }
              if (lane == 0) {
                mbar_arrive_expect_tx(qfull, halves * (HD / 64) * TS * P.rep * 128);
                for (int y = 0; y < halves; ++y)
                  for (int x = 0; x < HD / 64; ++x)
                    tma_rows(smem + y * C::TILE + x * 16384, &tq, 64 * x, q_head + y * next_head, q_tok + y * next_tok, qfull);
              }
              __syncwarp();
            }
            if (up && !split_v) {
              up = load(&tv, stage, sphase, b, first_head + h, page);
              ++stage;
            }
            if (stage >= ST) { stage = 0; sphase ^= 1; }
          } while (PAIRS && pair && up && ++h < 2);
          page = next;
        }
        u += x1 - x0;
        if (++t == ntile) {
          t = 0;
          ++head;
        }
      }
      if (!*dead) wait_phase(&mempty[slot], mphase, dead, P.status);
      if (*dead) {
        let_land();
      } else if (lane == 0) {
        meta[slot].nblk = 0;
        mbar_arrive(&mfull[slot]);
      }
    } else if (warp >= PC_MMA && warp < PC_MMA + 2) {
      // ---------------------------------------------------------- products
      // A warp for each half: to issue a half's 16 products and their commits
      // takes one thread most of the time that the products of both take.  The
      // whole warp walks the run (addresses and descriptors stay in uniform
      // registers); one elected thread issues.
      const int h = warp - PC_MMA;
      constexpr uint32_t id_s = idesc_f16(128, 128, BF), id_o = idesc_f16(128, HD, BF, true);
      const uint64_t dq = sdesc_sw128(smem_u32(smem + h * C::TILE)), dk = sdesc_sw128(smem_u32(smem + C::o_kv));
      const uint64_t dv = sdesc_sw128_mn(smem_u32(smem + C::o_kv), 16384u);
      const uint32_t t_s = T_S + 128u * h, t_o = T_O + 128u * h;
      uint32_t blkn = 0, pn = 0, qn = 0;  // blocks loaded, P's and tiles seen
      uint32_t pairs = 0, pairs_seen = 0;
      int slot = 0;
      uint32_t mphase = 0;
      auto kst = [](uint32_t b) { return (2 * b) % ST; };
      auto kph = [](uint32_t b) { return ((2 * b) / ST) & 1; };
      // S from the K block in stage st
      uint32_t turn = 0;
      auto s_product_to = [&](uint32_t t, uint32_t st) {
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk) {
          const uint32_t off = ((uint32_t)(kk >> 2) * 16384u + (uint32_t)(kk & 3) * 32u) >> 4;
          tc_mma(t, dq + off, dk + (st * (C::TILE / 16) + off), id_s, kk != 0);
        }
      };
      auto s_product = [&](uint32_t st) {
        s_product_to(t_s, st);
        tc_commit(&sfull[h]);
      };
      for (;;) {
        wait_phase(&mfull[slot], mphase, dead, P.status);
        if (*dead) break;
        const int nblk = meta[slot].nblk;
        const bool mine = h == 0 || meta[slot].ntok > TS, pair = PAIRS && meta[slot].pair;
        const bool in_turn = TURNS && meta[slot].ntok <= TS;
        __syncwarp();
        if (lane == 0) mbar_arrive(&mempty[slot]);
        if (nblk == 0) break;
        if (++slot == C::SLOTS) { slot = 0; mphase ^= 1; }
        wait_phase(qfull, qn & 1, dead, P.status);
        ++qn;
        if (PAIRS && pair) {
          // A half's products are those of its own head's blocks, every other one; a
          // stage is released twice by the one that used it.  A pair's blocks are even
          // in number, and so are the stages: while tiles are pairs a half always has
          // the same stages and sees all their phases.
          const uint32_t end = blkn + 2 * nblk;
          uint32_t b = blkn + h;
          blkn = end;
          auto s_of = [&](uint32_t st) {
            s_product(st);
            tc_commit(&empty[st]);
            tc_commit(&empty[st]);
          };
          wait_phase(&full[kst(b)], kph(b), dead, P.status);
          if (*dead) break;
          tc_fence_after();
          if (elect_one()) {
            s_of(kst(b));
            if (nblk == 1) tc_commit(qempty);
          }
          for (bool first = true; b < end; b += 2, first = false) {
            const uint32_t vst = kst(b) + 1;
            const bool more = b + 2 < end;
            wait_phase(&full[vst], kph(b), dead, P.status);
            if (more) wait_phase(&full[kst(b + 2)], kph(b + 2), dead, P.status);
            wait_phase(&pfull[h], pn & 1, dead, P.status);
            ++pn;
            if (*dead) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                tc_mma_ta(t_o, t_s + 8u * kk, dv + (vst * (C::TILE / 16) + 128u * kk), id_o, !first || kk != 0);
              if (more) {
                s_of(kst(b + 2));
                if (b + 4 >= end) tc_commit(qempty);
              } else {
                tc_commit(&ofull[h]);
              }
              tc_commit(&empty[vst]);
              tc_commit(&empty[vst]);
            }
          }
          if (*dead) break;
          if (lane == 0) mbar_arrive(pdone);
          ++pairs;
          continue;
        }
        // Behind a pair a half may come to a stage that the other one had: not before
        // that one has seen its loads land, or a wait for this phase could be met by
        // the one before.  (The other is at most a tile behind: its queries' room was
        // needed for this one's.)
        if (PAIRS && pairs != pairs_seen) {
          wait_phase(pdone, (pairs - 1) & 1, dead, P.status);
          pairs_seen = pairs;
          if (*dead) break;
        }
        if (!mine) {  // a tile of one half: see every phase, use nothing
          if (lane == 0) mbar_arrive(qempty);
          for (int j = 0; j < 2 * nblk; ++j) {
            const uint32_t st = kst(blkn) + (j & 1);
            wait_phase(&full[st], kph(blkn), dead, P.status);
            if (lane == 0) mbar_arrive(&empty[st]);
            blkn += j & 1;
          }
          if (*dead) break;
          continue;
        }
        if (TURNS && in_turn) {
          auto s_turn = [&](int j) {
            const uint32_t st = kst(blkn + j);
            wait_phase(&full[st], kph(blkn + j), dead, P.status);
            if (*dead) return;
            tc_fence_after();
            if (elect_one()) {
              const uint32_t b = (turn + j) & 1;
              s_product_to(T_S + 128u * (j & 1), st);
              tc_commit(&sturn[b]);
              tc_commit(&empty[st]);
              if (j + 1 == nblk) tc_commit(qempty);
            }
            __syncwarp();
          };
          s_turn(0);
          if (nblk > 1 && !*dead) s_turn(1);
          for (int j = 0; j < nblk; ++j) {
            const uint32_t vst = kst(blkn + j) + 1, b = (turn + j) & 1;
            wait_phase(&full[vst], kph(blkn + j), dead, P.status);
            wait_phase(&pturn[b], ((turn + j) >> 1) & 1, dead, P.status);
            if (*dead) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                tc_mma_ta(t_o, T_S + 128u * (j & 1) + 8u * kk, dv + (vst * (C::TILE / 16) + 128u * kk), id_o, (j | kk) != 0);
              tc_commit(&oturn[b]);
              tc_commit(&empty[vst]);
              if (j + 1 == nblk) tc_commit(&ofull[h]);
            }
            __syncwarp();
            if (j + 2 < nblk) s_turn(j + 2);
          }
          if (*dead) break;
          blkn += nblk;
          turn += nblk;
          continue;
        }
        wait_phase(&full[kst(blkn)], kph(blkn), dead, P.status);
        tc_fence_after();
        if (elect_one()) {
          s_product(kst(blkn));
          tc_commit(&empty[kst(blkn)]);
          if (nblk == 1) tc_commit(qempty);
        }
        for (int j = 0; j < nblk; ++j, ++blkn) {
          const uint32_t vst = kst(blkn) + 1, nst = kst(blkn + 1);
          const bool more = j + 1 < nblk;
          // (a wait that is met already costs 150 cycles: not behind P's)
          wait_phase(&full[vst], kph(blkn), dead, P.status);
          if (more) wait_phase(&full[nst], kph(blkn + 1), dead, P.status);
          wait_phase(&pfull[h], pn & 1, dead, P.status);
          ++pn;
          if (*dead) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              tc_mma_ta(t_o, t_s + 8u * kk, dv + (vst * (C::TILE / 16) + 128u * kk), id_o, (j | kk) != 0);
            if (more) {
              s_product(nst);
              tc_commit(&empty[vst]);
              tc_commit(&empty[nst]);
              if (j + 2 == nblk) tc_commit(qempty);
            } else {
              tc_commit(&ofull[h]);
              tc_commit(&empty[vst]);
            }
          }
        }
        if (*dead) break;
      }
      if (*dead) let_land();
      __syncwarp();
    }
    if constexpr (clustered) if (P.cluster > 1) {
      cluster_sync();
      cluster_sync();
    }
  } else {
    // ------------------------------------------------------------ softmax
    setmaxnreg_inc<PC_REGS_SOFT>();
    const int half = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_t0 = T_S + 128u * half + lanes;
    const uint32_t o_t = T_O + 128u * half + lanes;
    const int tok_in = P.token_of(row), hq_in = row - tok_in * P.rep;
    const float cs = fabsf(P.scale) * 1.4426950408889634f;
    const bool neg = P.scale < 0.f;
    constexpr float top = BF ? 0.f : PC_TOP_FP16;
    uint32_t blkn = 0, sn = 0, on = 0, turn = 0;
    int slot = 0;
    uint32_t mphase = 0;
    int held = -1;  // in a cluster: this thread's row of the tile, its maximum and sum
    float held_m = 0.f, held_l = 0.f;
    for (;;) {
      wait_phase(&mfull[slot], mphase, dead, P.status);
      if (*dead) break;
      const Tile m = meta[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&mempty[slot]);
      if (m.nblk == 0) break;
      if (++slot == C::SLOTS) { slot = 0; mphase ^= 1; }
      const bool pair = PAIRS && m.pair;
      const int tok0 = pair ? 0 : half * TS;  // this half's first token of the tile
      if (tok0 >= m.ntok) {
        blkn += m.nblk;
        continue;
      }
      const int ntok = min(TS, m.ntok - tok0);
      const int pos0 = m.pos0 + tok0, pos = pos0 + min(tok_in, ntok - 1), end = pos0 + ntok - 1;
      int last = min(pos, m.hi - 1), first = pos >= P.window ? pos - P.window + 1 : 0;
      // every row of the half sees the keys [all_lo, all_hi)
      const int all_lo = end >= P.window ? end - P.window + 1 : 0;
      int all_hi = min(pos0 + 1, m.hi);
      // a tree's row: the cached keys [first, last], and of the new ones those of its
      // mask from bit `least` to itself
      const bool tree = TREE && m.ctx != -0x7fffffff - 1;
      const uint32_t* mask = nullptr;
      int node = 0, least = 0;
      if constexpr (TREE) {
        if (tree) {
          node = pos - m.ctx;
          mask = P.masks + (int64_t)(m.row0 + tok0 + min(tok_in, ntok - 1)) * P.mask_words;
          last = min(m.ctx, m.hi) - 1;
          all_hi = min(m.ctx, m.hi);
          if (P.window != 0x7fffffff) {
            int have = 0;  // set bits so far, from the row itself down
            bool some = false;
            for (int w = node >> 5; w >= 0; --w) {
              uint32_t x = mask[w];
              if (w == node >> 5) x &= (2u << (node & 31)) - 1;
              const int n = __popc(x);
              if (!some && have + n >= P.window) {  // the window's last bit is in this word
                for (int k = have + n; k > P.window; --k) x &= x - 1;
                least = 32 * w + __ffs(x) - 1;
                some = true;
              }
              have += n;
            }
            const int p = m.ctx + max(have, 1) - 1;
            first = p >= P.window ? p - P.window + 1 : 0;
          }
        }
      }
      float mx = -INFINITY, l = 0.f;
      const uint32_t blk_step = pair ? 2 : 1;
      if (pair) blkn += half;
      // in turns: a buffer and barriers of every other block
      const uint32_t two = TURNS && m.ntok <= TS ? 1 : 0;
      uint64_t *s_bar = two ? sturn : &sfull[half], *p_bar = two ? pturn : &pfull[half];
      uint32_t count = two ? turn : sn;
      for (int j = 0; j < m.nblk; ++j, blkn += blk_step) {
        const int key0 = m.key0 + 128 * j;
        uint32_t named[4] = {0, 0, 0, 0};  // columns of the block that the row's mask names
        if constexpr (TREE) {
          if (tree && key0 + 128 > all_hi) {
            const int d = key0 - m.ctx;  // new token of column 0
            const int top = min(node, m.hi - 1 - m.ctx);
            uint32_t w[5];
#pragma unroll
            for (int i = 0; i < 5; ++i) {
              const int at = (d >> 5) + i, b = 32 * at;  // bits of new tokens b .. b + 31
              w[i] = at >= 0 && b <= top ? mask[at] : 0u;
              if (b + 31 > top && b <= top) w[i] &= (2u << (top - b)) - 1;
              if (least > b) w[i] = least > b + 31 ? 0u : w[i] & (0xffffffffu << (least - b));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) named[i] = __funnelshift_r(w[i], w[i + 1], d & 31);
          }
        }
        uint32_t s_t = s_t0;
        if constexpr (TURNS) {
          s_t = s_t0 + ((j & two) << 7);
          wait_phase(&s_bar[count & two], (count >> two) & 1, dead, P.status);
        } else {
          wait_phase(&sfull[half], sn & 1, dead, P.status);
          ++sn;
        }
        tc_fence_after();
        float s[128];
        tmem_ld128(s_t, s);
        if (neg) {
#pragma unroll
          for (int i = 0; i < 128; ++i) s[i] = -s[i];
        }
        if (key0 < all_lo || key0 + 128 > all_hi) {
          const int c0 = first - key0, width = last + 1 - first;  // visible columns [c0, c0 + width)
          const uint32_t w = width > 0 ? (uint32_t)width : 0u;
          if constexpr (TREE) {
            const int c1 = width > 0 ? c0 + width : c0;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              // bits [c0 - 32 q, c1 - 32 q) of a word, and the named ones
              const int b0 = min(max(c0 - 32 * q, 0), 32), b1 = min(max(c1 - 32 * q, 0), 32);
              const uint32_t keep = ((uint32_t)((1ull << b1) - 1) & ~(uint32_t)((1ull << b0) - 1)) | named[q];
              if (__any_sync(0xffffffffu, keep != 0xffffffffu)) {
#pragma unroll
                for (int i = 0; i < 32; ++i) s[32 * q + i] = keep >> i & 1u ? s[32 * q + i] : -INFINITY;
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < 128; ++i)
              if ((uint32_t)(i - c0) >= w) s[i] = -INFINITY;
          }
        }
        float t0 = s[0], t1 = s[1], t2 = s[2], t3 = s[3];
#pragma unroll
        for (int i = 4; i < 124; i += 8) {
          t0 = max3(t0, s[i], s[i + 1]);
          t1 = max3(t1, s[i + 2], s[i + 3]);
          t2 = max3(t2, s[i + 4], s[i + 5]);
          t3 = max3(t3, s[i + 6], s[i + 7]);
        }
        t0 = max3(t0, s[124], s[125]);
        t1 = max3(t1, s[126], s[127]);
        const float bm = max3(t0, t1, fmaxf(t2, t3));
        const float mn = fmaxf(mx, bm);
        if (__any_sync(0xffffffffu, (mn - mx) * cs > PC_LAG)) {
          const float a = mx == -INFINITY ? 0.f : ex2((mx - mn) * cs);
          l *= a;
          mx = mn;
          if (j > 0) {
            if (TURNS && two) {  // (S of this block was issued before P V of the last)
              wait_phase(&oturn[(count - 1) & 1], ((count - 1) >> 1) & 1, dead, P.status);
              tc_fence_after();
            }
#pragma unroll 1
            for (int x = 0; x < HD; x += 32) {
              float o[32];
              tmem_ld32(o_t + x, o);
              uint32_t w[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(o[i] * a);
              tmem_st32(o_t + x, w);
            }
          }
        }
        const float ref = (mx == -INFINITY ? 0.f : mx * cs) - top;
        const u64 cs2 = pack_f32x2(cs, cs), ref2 = pack_f32x2(-ref, -ref);
        u64 sum0 = 0, sum1 = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t pk[32 / 2];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const u64 x = fma_f32x2(pack_f32x2(s[32 * q + 2 * i], s[32 * q + 2 * i + 1]), cs2, ref2);
            const float p0 = ex2(__uint_as_float((uint32_t)x)), p1 = ex2(__uint_as_float((uint32_t)(x >> 32)));
            if (i & 1) sum1 = add_f32x2(sum1, pack_f32x2(p0, p1));
            else sum0 = add_f32x2(sum0, pack_f32x2(p0, p1));
            pk[i] = down2<BF>(p0, p1);
          }
          tmem_st16(s_t + 16 * q, pk);
        }
        l += pair_sum(add_f32x2(sum0, sum1));
        // values of keys that no row sees may be anything: each half's group
        // makes them zero before its product with V (both write the same)
        if (key0 < m.lo || key0 + 128 > m.hi) {
          const uint32_t vst = (2 * blkn) % ST + 1;
          wait_phase(&full[vst], ((2 * blkn) / ST) & 1, dead, P.status);
          uint8_t* v = smem + C::o_kv + vst * C::TILE;
          if constexpr (TREE) {
            // (pages that no row sees have arrived as zeros: what is hidden of those
            // that a row sees, 16 bytes after 16)
            const int boxt = min(128, 1 << P.page_shift);
            const int h0 = max(0, (m.lo & ~(boxt - 1)) - key0), h1 = m.lo - key0;              // before the first seen key
            const int t0 = m.hi - key0, t1 = min(128, ((m.hi + boxt - 1) & ~(boxt - 1)) - key0);  // behind the last
            auto clear = [&](int a, int b) {
              for (int i = a * 8 + row; i < b * 8; i += 128)
#pragma unroll
                for (int x = 0; x < HD / 64; ++x) *reinterpret_cast<uint4*>(v + x * 16384 + 16 * i) = make_uint4(0, 0, 0, 0);
            };
            clear(h0, min(h1, 128));
            clear(max(t0, 0), t1);
          } else {
            const int key = key0 + row;  // rows of 128 threads
            if (key < m.lo || key >= m.hi) {
              uint8_t* r = v + row * 128;
#pragma unroll
              for (int x = 0; x < HD / 64; ++x)
#pragma unroll
                for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(r + x * 16384 + 16 * i) = make_uint4(0, 0, 0, 0);
            }
          }
          fence_proxy_async_smem();
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if constexpr (TURNS) {
          if (lane == 0) mbar_arrive(&p_bar[count & two]);
          ++count;
        } else {
          if (lane == 0) mbar_arrive(&pfull[half]);
        }
      }
      if (TURNS && two) turn = count;
      else if (TURNS) sn = count;
      if (pair) blkn -= half;  // the tile's end
      wait_phase(&ofull[half], on & 1, dead, P.status);
      ++on;
      tc_fence_after();
      const bool live = tok_in < ntok;
      const int prow = (pair ? 128 * half : tok0 * P.rep) + row, head = m.head + (pair ? half : 0);
      if constexpr (clustered) {
        if (m.part == -2) {  // (the one tile)
          if (live) held = prow;
          held_m = mx * cs - top;
          held_l = l;
          continue;
        }
      }
      if (m.part < 0) {
        // Four lanes exchange 16-byte pieces so that a store writes 64
        // contiguous bytes of a row: lane 4 a + b then has piece b of the rows
        // 4 a + i (16 scattered bytes a lane took three times as long).
        const float inv = inv_of(l);
        uint16_t* dst[4];
        bool put[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rw = (row & ~3) + i, tk = P.token_of(rw);
          put[i] = tk < ntok;
          dst[i] = P.out + (int64_t)(m.row0 + tok0 + tk) * P.o_stride +
                   (int64_t)(head * P.rep + rw - tk * P.rep) * HD + (lane & 3) * 8;
        }
#pragma unroll 1
        for (int x = 0; x < HD; x += 32) {
          float o[32];
          tmem_ld32(o_t + x, o);
          uint32_t c[4][4];
#pragma unroll
          for (int i = 0; i < 16; ++i) c[i >> 2][i & 3] = down2<BF>(o[2 * i] * inv, o[2 * i + 1] * inv);
          quad_swap<1>(c[0], c[1], lane);
          quad_swap<1>(c[2], c[3], lane);
          quad_swap<2>(c[0], c[2], lane);
          quad_swap<2>(c[1], c[3], lane);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (put[i]) *reinterpret_cast<uint4*>(dst[i] + x) = make_uint4(c[i][0], c[i][1], c[i][2], c[i][3]);
        }
        if (live && P.lse)
          P.lse[(int64_t)(m.row0 + tok0 + tok_in) * (P.hkv * P.rep) + head * P.rep + hq_in] =
              lse_of(mx * cs - top, l);
      } else {
        // a part: [4 columns][row], a warp's lanes end to end
        float* dst = W.o + (int64_t)m.part * W.rt * HD + prow * 4;
#pragma unroll 1
        for (int x = 0; x < HD; x += 32) {
          float o[32];
          tmem_ld32(o_t + x, o);
          if (live) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<float4*>(dst + (x + i) * W.rt) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          }
        }
        if (live) W.ml[(int64_t)m.part * W.rt + prow] = make_float2(mx * cs - top, l);
      }
      tc_fence_before();  // the next tile's first P V is issued behind this group's next P
    }
    if constexpr (clustered) if (P.cluster > 1) {
      // A cluster's CTAs have the tile's rows, each over its share of the keys: CTA k
      // joins rows [k per, (k + 1) per), which all of them write to its shared memory
      // ([CTA][4 columns][row]), where the keys and values were and before them (rows
      // of up to 15 more than the tile has), maxima and sums at its start.
      constexpr int o_parts = C::o_kv - 16384;
      static_assert((256 + 15) * HD * 4 <= C::o_meta - o_parts && (256 + 15) * 8 <= 8192 && 8192 + (256 + 15) * 4 <= o_parts, "room for the parts");
      const int cl = P.cluster, rows = joined[0], nb = joined[2], per_cta = max(1, (rows + cl - 1) / cl), rk = (int)cluster_rank();
      const uint32_t has = __ballot_sync(0xffffffffu, lane < cl && share_of(nb, lane, cl) < share_of(nb, lane + 1, cl));  // CTAs that had keys
      cluster_sync();  // nothing of the cluster's products and loads is on its way
      if (__any_sync(0xffffffffu, held >= 0)) {
        const int owner = max(held, 0) / per_cta, at = max(held, 0) - owner * per_cta;
        const uint32_t o_to = cluster_addr(smem + o_parts, owner) + (uint32_t)((rk * per_cta * HD + at * 4) * 4);
        const uint32_t ml_to = cluster_addr(smem, owner) + (uint32_t)((rk * per_cta + at) * 8);
        if (held >= 0) st_cluster64(ml_to, pack_f32x2(held_m, held_l));
#pragma unroll 1
        for (int x = 0; x < HD; x += 32) {
          float o[32];
          tmem_ld32(o_t + x, o);
          if (held >= 0) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              st_cluster128(o_to + (uint32_t)((x + i) * per_cta * 4), make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]));
          }
        }
        tc_fence_before();
      }
      cluster_sync();
      // the CTAs' factors of a row (16 lanes a row, one a CTA), then the rows
      const float2* ml = reinterpret_cast<const float2*>(smem);
      float* factor = reinterpret_cast<float*>(smem + 8192);
      const float4* part = reinterpret_cast<const float4*>(smem + o_parts);
      if (!*dead) {
        for (int rw0 = warp * 2; rw0 < per_cta; rw0 += 16) {
          const int rw = rw0 + (lane >> 4), c = lane & 15;
          const bool in = rw < per_cta && (has >> c & 1u);
          const float2 y = in ? ml[c * per_cta + rw] : make_float2(-INFINITY, 0.f);
          float mm = y.x;
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
          const float f = ex2(y.x - (mm == -INFINITY ? 0.f : mm));
          float ll = in ? y.y * f : 0.f;
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) ll += __shfl_xor_sync(0xffffffffu, ll, o);
          if (c < cl && rw < per_cta) factor[c * per_cta + rw] = f * inv_of(ll);
          const int prow = rk * per_cta + rw;
          if (c == 0 && P.lse && rw < per_cta && prow < rows) {
            const int tk = P.token_of(prow);
            P.lse[(int64_t)(joined[1] + tk) * (P.hkv * P.rep) + joined[3] * P.rep + prow - tk * P.rep] = lse_of(mm, ll);
          }
        }
      }
      named_bar(1, 256);
      for (int i = tid; i < per_cta * (HD / 4) && !*dead; i += 256) {
        const int d4 = i / per_cta, rw = i - d4 * per_cta, prow = rk * per_cta + rw;
        if (prow >= rows) continue;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c0 = 0; c0 < cl; c0 += 4) {
          float f[4];
          float4 v[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {  // (of a CTA without keys: factor 0 and whatever was there)
            const int k = min(c0 + c, cl - 1);
            f[c] = factor[k * per_cta + rw];
            v[c] = part[(k * (HD / 4) + d4) * per_cta + rw];
            if (c0 + c >= cl || f[c] == 0.f) v[c] = make_float4(0.f, 0.f, 0.f, 0.f);
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            acc.x += v[c].x * f[c]; acc.y += v[c].y * f[c]; acc.z += v[c].z * f[c]; acc.w += v[c].w * f[c];
          }
        }
        const int tk = P.token_of(prow);
        *reinterpret_cast<uint2*>(P.out + (int64_t)(joined[1] + tk) * P.o_stride + (int64_t)(joined[3] * P.rep + prow - tk * P.rep) * HD + d4 * 4) =
            make_uint2(down2<BF>(acc.x, acc.y), down2<BF>(acc.z, acc.w));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == PC_MMA) {
    tc_fence_after();
    tmem_dealloc(*tslot, 512);
  }
}

// ---------------------------------------------------------------- join
// The tile kernel's parts of trees, where no few-row kernel precedes it: 32 rows of
// a tile at a time, lanes on the rows, warps on the dimensions; the items of all
// tiles end to end.  Latency bound: what counts is that all loads of an item are in
// flight at once and that the items go round few times.  With few of them (a lone
// request: 8 tiles of 19 parts) an item is 32 dimensions of which the block's two
// teams take every other part (a lone request of 32 tokens over 4096 keys 30.7 -> 17.3
// us by this and the spared launch); with many (two parts each, mostly) each warp takes
// 8 dimensions of an item for itself and writes 16 bytes a row (32 requests over 500 to
// 2000 keys 59.6 us; by teams, through shared memory 61.4; 16 dimensions a warp 60.7,
// 4 63.3).
constexpr int JT_THREADS = 512;

// A team's warp `quad` joins parts first, first + step, .. of 32 rows (one a lane), Q
// groups of four dimensions, AHEAD parts in flight.
template <int HD, int Q, int AHEAD>
__device__ __forceinline__ void join_parts(const PagedParts& B, int c, int parts, int row, int quad, int first, int step,
                                           float* m_out, float* l_out, float4 (&o)[Q]) {
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int q = 0; q < Q; ++q) o[q] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = first; k0 < parts; k0 += step * AHEAD) {
    float2 ml[AHEAD];
    float4 v[AHEAD][Q];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int k = k0 + step * i;
      ml[i] = make_float2(-INFINITY, 0.f);
      if (k < parts) {
        const int64_t part = k == 0 ? 2 * c + 1 : 2 * (c + k);
        ml[i] = __ldcg(B.ml + part * B.rt + row);
#pragma unroll
        for (int q = 0; q < Q; ++q)
          v[i][q] = __ldcg(reinterpret_cast<const float4*>(B.o + part * B.rt * HD + ((int64_t)(quad + q) * B.rt + row) * 4));
      }
    }
    float mn = m;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) mn = fmaxf(mn, ml[i].x);
    const float ref = mn == -INFINITY ? 0.f : mn, a = ex2(m - ref);
    l *= a;
#pragma unroll
    for (int q = 0; q < Q; ++q) { o[q].x *= a; o[q].y *= a; o[q].z *= a; o[q].w *= a; }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (k0 + step * i < parts) {
        const float f = ex2(ml[i].x - ref);
        l += ml[i].y * f;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          o[q].x += v[i][q].x * f; o[q].y += v[i][q].y * f; o[q].z += v[i][q].z * f; o[q].w += v[i][q].w * f;
        }
      }
    }
    m = mn;
  }
  *m_out = m;
  *l_out = l;
}

template <int HD, bool BF>
__global__ void __launch_bounds__(JT_THREADS, 2) paged_join_tiles_kernel(const __grid_constant__ PagedAttnParams P, const __grid_constant__ PagedParts B) {
  constexpr int DG = HD / 32;
  __shared__ int upto[225], tmp[JT_THREADS / 32];
  __shared__ PartDesc desc[224];
  __shared__ float other[8][4][33];
  __shared__ float2 other_ml[32];
  __shared__ uint2 rows_out[32][9];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, team = warp >> 3, quad = warp & 7;
  grid_launch_dependents();
  grid_wait_prior();
  PartDesc d{};
  if (tid < B.ctas) desc[tid] = d = B.desc[tid];
  int total;  // items of all dimensions
  bool any;
  // items of a tile: its rows by 32, of a pair those of each head
  const uint32_t at = block_scan<JT_THREADS / 32>(d.parts ? (uint32_t)((d.rows + 31) / 32 << (d.head >= PART_PAIR ? 1 : 0)) : 0u, false, tmp, &total, &any);
  if (tid <= B.ctas) upto[tid] = (int)at;
  __syncthreads();
  // item x of a tile: the tile as of one head, the item's first row, its first row in the parts
  auto item_of = [&](PartDesc& t, int x, int* row0) {
    const int per = (t.rows + 31) / 32, half = t.head >= PART_PAIR && x >= per ? 1 : 0;
    t.head = (t.head & ~PART_PAIR) + half;
    *row0 = (x - half * per) * 32;
    return *row0 + 128 * half;
  };
  auto put_lse = [&](const PartDesc& t, int row, float m, float l) {
    if (!P.lse || row >= t.rows) return;
    const int tk = P.token_of(row);
    P.lse[(int64_t)(t.row0 + tk) * (P.hkv * P.rep) + t.head * P.rep + row - tk * P.rep] = lse_of(m, l);
  };
  if (total * DG > 2 * (int)gridDim.x) {
    constexpr int WARPS = HD / 8, Q = 2;
    for (int x = JT_THREADS / 32 * blockIdx.x + warp; x < WARPS * total; x += JT_THREADS / 32 * gridDim.x) {
      const int item = x / WARPS, d0 = x % WARPS * 8, c = find_le(upto, B.ctas, item);
      PartDesc t = desc[c];
      int row0;
      const int in_part = item_of(t, item - upto[c], &row0), row = row0 + lane;
      float m, l;
      float4 o[Q];
      join_parts<HD, Q, 2>(B, c, t.parts, in_part + lane, d0 / 4, 0, 1, &m, &l, o);
      if (d0 == 0) put_lse(t, row, m, l);
      if (row >= t.rows) continue;
      const float inv = inv_of(l);
      const int tk = P.token_of(row);
      uint4* dst = reinterpret_cast<uint4*>(P.out + (int64_t)(t.row0 + tk) * P.o_stride + (int64_t)(t.head * P.rep + row - tk * P.rep) * HD + d0);
#pragma unroll
      for (int q = 0; q < Q; q += 2)
        dst[q / 2] = make_uint4(down2<BF>(o[q].x * inv, o[q].y * inv), down2<BF>(o[q].z * inv, o[q].w * inv),
                                down2<BF>(o[q + 1].x * inv, o[q + 1].y * inv), down2<BF>(o[q + 1].z * inv, o[q + 1].w * inv));
    }
    return;
  }
  for (int item = blockIdx.x; item < total * DG; item += gridDim.x) {
    const int c = find_le(upto, B.ctas, item / DG), d0 = item % DG * 32;
    PartDesc t = desc[c];
    int row0;
    const int in_part = item_of(t, item / DG - upto[c], &row0);
    float m, l;
    float4 o[1];
    join_parts<HD, 1, 5>(B, c, t.parts, in_part + lane, d0 / 4 + quad, team, 2, &m, &l, o);
    if (team) {
      other[quad][0][lane] = o[0].x; other[quad][1][lane] = o[0].y; other[quad][2][lane] = o[0].z; other[quad][3][lane] = o[0].w;
      if (quad == 0) other_ml[lane] = make_float2(m, l);
    }
    __syncthreads();
    if (!team) {
      const float2 y = other_ml[lane];
      const float mn = fmaxf(m, y.x), ref = mn == -INFINITY ? 0.f : mn, a = ex2(m - ref), f = ex2(y.x - ref);
      l = l * a + y.y * f;
      const float inv = inv_of(l);
      rows_out[lane][quad] = make_uint2(down2<BF>((o[0].x * a + other[quad][0][lane] * f) * inv, (o[0].y * a + other[quad][1][lane] * f) * inv),
                                        down2<BF>((o[0].z * a + other[quad][2][lane] * f) * inv, (o[0].w * a + other[quad][3][lane] * f) * inv));
      if (quad == 0 && d0 == 0) put_lse(t, row0 + lane, mn, l);
    }
    __syncthreads();
    if (!team) {  // 64 bytes a row
      const int rw = row0 + tid / 8, q = tid % 8, tk = P.token_of(rw);
      if (rw < t.rows)
        *reinterpret_cast<uint2*>(P.out + (int64_t)(t.row0 + tk) * P.o_stride + (int64_t)(t.head * P.rep + rw - tk * P.rep) * HD + d0 + q * 4) = rows_out[tid / 8][q];
    }
  }
}

template <int HD, bool BF>
int clusters_at_once(int device, int ctas) {
  static std::atomic<int> known[64][17];
  return paged_clusters_at_once((const void*)paged_chunk_kernel<HD, BF, true, CLUSTERS>, PC_THREADS, ChunkCfg<HD>::most, device, ctas, known);
}

template <int HD, bool BF, bool TREE, int FORM>
cudaError_t launch(const PagedAttnParams& p, const PagedKv& kv, const PagedParts& w, cudaStream_t st) {
  CUtensorMap tq, tk, tv;
  if (!make_page_tmap(&tk, kv.k, kv, HD, 128, 1, BF) || !make_page_tmap(&tv, kv.v, kv, HD, 128, 1, BF) ||
      !make_rows_tmap(&tq, p.q, p.rows, p.hkv * p.rep, HD, p.q_stride, p.rep, 128 / p.rep, BF))
    return cudaErrorInvalidValue;
  // the register split needs the block to be launched with what it counts on
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = paged_prepare((const void*)paged_chunk_kernel<HD, BF, TREE, FORM>,
                                      ChunkCfg<HD>::most, PC_REGS, p.device, &ready);
  if (e != cudaSuccess) return e;
  if constexpr (FORM == CLUSTERS)
    return paged_launch_clusters(paged_chunk_kernel<HD, BF, TREE, FORM>, p.cluster_tiles * p.cluster, p.cluster, PC_THREADS,
                                 ChunkCfg<HD>::total(p.n), st, tq, tk, tv, p, w);
  // behind the few-row kernel it is set up while that one ends; alone it is launched
  // behind the whole of what precedes (8192-token prompt 363 against 368 us)
  return paged_launch_if(TREE || p.few_rows > 0, paged_chunk_kernel<HD, BF, TREE, FORM>, w.ctas, PC_THREADS, ChunkCfg<HD>::total(p.n), st,
                         tq, tk, tv, p, w);
}

template <bool TREE, int FORM>
cudaError_t launch_type(const PagedAttnParams& p, const PagedKv& kv, const PagedParts& w, int d, bool bf, cudaStream_t st) {
  if (d == 128) return bf ? launch<128, true, TREE, FORM>(p, kv, w, st) : launch<128, false, TREE, FORM>(p, kv, w, st);
  return bf ? launch<64, true, TREE, FORM>(p, kv, w, st) : launch<64, false, TREE, FORM>(p, kv, w, st);
}

}  // namespace

cudaError_t paged_chunk_launch(const PagedAttnParams& p, const PagedKv& kv, const PagedParts& w, int d,
                               bool bf, cudaStream_t st) {
  if (p.masks) {
    if (p.cluster) return launch_type<true, CLUSTERS>(p, kv, w, d, bf, st);
    // (heads of 64 of even number go in pairs)
    if (p.max_new <= 128 / p.rep && (d == 128 || (p.hkv & 1))) return launch_type<true, RUNS_OF_HALVES>(p, kv, w, d, bf, st);
    return launch_type<true, RUNS>(p, kv, w, d, bf, st);
  }
  return launch_type<false, RUNS>(p, kv, w, d, bf, st);
}

// Few tiles over few keys: a cluster for each, of as many CTAs as the device holds at
// once for all, joined in their shared memory (a lone request of 32 tokens over 4096
// keys, 8 kv heads of 128, 12.9 against 16.9 us of runs over all SMs, parts in memory
// and the join's launch; 16 of them over 512 keys, a CTA a tile, 13.0 against 23.2; 4 over
// 2000 15.4, 20.3).  The host does not know the lengths: what a tile may have is bounded
// by the table's width, so that with tables of 32768 tokens these calls take the second
// figures.  Past 8 blocks a
// CTA the SMs that no cluster fills, and requests that are shorter than the longest,
// cost what the join does (2 requests of 32 tokens over 9168 keys, 8 CTAs of 9 blocks, 25.2
// against 23.9 us; 8 over 50 to 2000 keys, 2 CTAs of 8, 20.6 both, to 3000 25.0, 21.9);
// with 3 to 6 CTAs, whose exchange is short, past 12 (4 requests over 6000 keys 25.8,
// 29.7; over 50 to 6000 24.0, 25.1).  Tiles of two halves exchange twice as much: up to
// 6 CTAs of 4 blocks (4 requests of 64 tokens over 2000 keys 22.8, 24.0; 5 over 1456 24.6,
// 26.4; 3 over 2992 25.2, 24.8; of 16 CTAs, a lone one over 2000 16.6, 15.9, over 4016
// 19.0, 19.8).  A CTA a tile has nothing to exchange (10 requests of 32 tokens over 2000
// keys 24.9, 28.4).
void paged_chunk_clusters(PagedAttnParams* p, int d, bool bf) {
  const int tt = 2 * (128 / p->rep);
  const int64_t tiles = (int64_t)p->n * p->hkv * (((int64_t)p->max_new + tt - 1) / tt);
  const int64_t blocks = (((int64_t)p->max_blocks << p->page_shift) + 127) / 128;
  p->cluster = p->cluster_tiles = 0;
  if (tiles > 256) return;
  for (int c = 16; c >= 1; --c) {
    const int most = d == 128 ? (bf ? clusters_at_once<128, true>(p->device, c) : clusters_at_once<128, false>(p->device, c))
                              : (bf ? clusters_at_once<64, true>(p->device, c) : clusters_at_once<64, false>(p->device, c));
    if (tiles > most) continue;
    const int each = (int64_t)p->max_new * p->rep > 128 ? (c <= 6 ? 4 : 0) : c >= 3 && c <= 6 ? 12 : 8;
    const int64_t most_blocks = c == 1 ? 16 : c * each;
    if (blocks <= most_blocks) {
      p->cluster = c;
      p->cluster_tiles = (int)tiles;
    }
    return;
  }
}

cudaError_t paged_join_tiles_launch(const PagedAttnParams& p, const PagedParts& b, int d, bool bf, cudaStream_t st) {
  const int grid = 2 * b.ctas;
  if (d == 128)
    return bf ? paged_launch(paged_join_tiles_kernel<128, true>, grid, JT_THREADS, 0, st, p, b)
              : paged_launch(paged_join_tiles_kernel<128, false>, grid, JT_THREADS, 0, st, p, b);
  return bf ? paged_launch(paged_join_tiles_kernel<64, true>, grid, JT_THREADS, 0, st, p, b)
            : paged_launch(paged_join_tiles_kernel<64, false>, grid, JT_THREADS, 0, st, p, b);
}

}  // namespace mk
