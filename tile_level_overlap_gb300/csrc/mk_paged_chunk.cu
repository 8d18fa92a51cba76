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
// a quarter later than the others.
constexpr int PC_OVER = 2;
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
  static constexpr int o_pre = o_bar + 256;
  static constexpr int total(int n) { return o_pre + Kept::bytes(n); }
  static constexpr int most = o_pre + KEPT_MOST;
};
static_assert(ChunkCfg<128>::most <= 232448 && ChunkCfg<64>::most <= 232448, "shared memory of a CTA");

struct Tile {
  int key0, nblk;          // first key of the run; 0 blocks: the end
  int row0, ntok, head;    // first token (row of q), tokens of the tile
  int pos0;                // position of the first token
  int lo, hi;              // keys the request's rows may see
  int part;                // workspace part, -1: all of the tile's blocks
  int req;                 // its request
  int pad[6];
};
static_assert(sizeof(Tile) == 64, "meta slot");

// First block and number of blocks of tile t of a request (TT tokens a tile).
__device__ __forceinline__ int tile_blocks(const PagedAttnParams& P, const Request& q, int t, int TT, int* first) {
  const int p0 = q.pos0 + t * TT, p1 = q.pos0 + min(q.add, (t + 1) * TT);
  const int hi = min(max(p1, 0), q.hi);
  const int lo = p0 >= P.window ? min(p0 - P.window + 1, hi) : 0;
  *first = lo / 128;
  return max(1, (hi + 127) / 128 - lo / 128);
}

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

template <int HD, bool BF>
__global__ void __launch_bounds__(PC_THREADS, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv, const __grid_constant__ PagedAttnParams P,
                       const __grid_constant__ PagedParts W) {
  using C = ChunkCfg<HD>;
  constexpr int ST = C::STAGES;
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
  Tile* meta = reinterpret_cast<Tile*>(smem + C::o_meta);
  const Kept kept(smem + C::o_pre, P.n);
  int* pre = kept.pre;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int TS = 128 / P.rep, TT = 2 * TS;  // tokens of a half, of a tile
  const bool split_v = P.page_shift < PC_SPLIT_V;

  grid_launch_dependents();
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
  if (tid == 0) W.desc[blockIdx.x].parts = 0;

  // units: the tiles' blocks and overheads.  A thread counts its requests'
  // tiles; a warp together those of a request with many.
  const int per = (P.n + PC_THREADS - 1) / PC_THREADS;
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
      for (int t = 0; t < ntile; ++t) u += tile_blocks(P, q, t, TT, &b0);
    for (uint32_t many = __ballot_sync(0xffffffffu, ntile > 8); many; many &= many - 1) {
      const int from = __ffs(many) - 1;
      Request x{};
      x.add = __shfl_sync(0xffffffffu, q.add, from);
      x.pos0 = __shfl_sync(0xffffffffu, q.pos0, from);
      x.hi = __shfl_sync(0xffffffffu, q.hi, from);
      const int nt = __shfl_sync(0xffffffffu, ntile, from);
      int v = 0;
      for (int t = lane; t < nt; t += 32) v += tile_blocks(P, x, t, TT, &b0);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == from) u = v;
    }
    u = (u + PC_OVER * ntile) * P.hkv;
    if (r < P.n) pre[r] = u;
    mine += u;
  }
  int* scan_tmp = reinterpret_cast<int*>(smem + C::o_kv);  // not loaded to yet
  const int T = place_units<PC_THREADS / 32>(P, pre, per, mine, falls, scan_tmp);
  if (bad && blockIdx.x == 0) latch(P.status, MK_ERR_BOUNDS);
  fence_proxy_async_smem();  // the scan's words, before a load takes their place
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // every column is this CTA's: the allocation starts at column 0
  constexpr uint32_t T_S = 0, T_O = 256;

  const int G = min((int)gridDim.x, T), c = blockIdx.x;
  const Runs runs(T, max(G, 1));
  const int u0 = c < G ? runs.start(c) : 0, u1 = c < G ? runs.start(c + 1) : 0;

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
    auto page_of = [&](const int32_t* tab, int b, int lo, int hi) {
      const int key = b * 128 + lane * boxt;
      if (lane >= nbox || key >= hi || key + boxt <= lo) return -1;
      const int p = tab[key >> P.page_shift];
      if (p >= 0 && p < P.n_pages) return p;
      latch(P.status, MK_ERR_BOUNDS);
      return -1;
    };
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
        for (int x = 0; x < HD / 64; ++x) tma_page(dst + x * 16384, tm, tok, x, head, page, &full[stage]);
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
          up = load(&tv, stage, sphase, b0 + i, m.head, page);
          stage += 2;
          if (stage > ST) { stage = 1; sphase ^= 1; }
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
      int r = u0 < u1 ? find_le(pre, P.n, u0) : 0, t = -1, head = 0;
      bool up = true;
      for (int u = u0; u < u1 && up;) {
        while (pre[r + 1] <= u) {
          ++r;
          t = -1;
        }
        const Request q = kept.again(P, r);
        const int per_head = (pre[r + 1] - pre[r]) / P.hkv, ntile = (q.add + TT - 1) / TT;
        int x0 = 0, b0;  // first unit of the tile in this run
        if (t < 0) {  // find the tile of unit u
          const int local = u - pre[r];
          head = local / per_head;
          int rem = local - head * per_head;
          for (int base = 0;; base += 32) {
            int f, k = 0;
            if (base + lane < ntile) k = tile_blocks(P, q, base + lane, TT, &f) + PC_OVER;
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
        const int nb = tile_blocks(P, q, t, TT, &b0), x1 = min(nb + PC_OVER, x0 + u1 - u);
        const int blk = max(0, x0 - PC_OVER), nblk = max(0, x1 - PC_OVER) - blk;
        const int ntok = min(TT, q.add - t * TT), end = u - x0 + nb + PC_OVER;
        if (nblk == 0) break;  // the run ends with the tile's overhead: the next CTA has it all
        const bool whole = blk == 0 && nblk == nb;
        if (blk == 0 && !whole && lane == 0) {
          const int last = runs.of(end - 1);  // CTA of the tile's last unit
          PartDesc d;
          d.row0 = q.row0 + t * TT; d.rows = ntok * P.rep; d.head = head; d.parts = last - c + 1;
          W.desc[c] = d;
        }
        wait_phase(&mempty[slot], mphase, dead, P.status);
        if (*dead) break;
        if (lane == 0) {
          Tile m;
          m.key0 = (b0 + blk) * 128; m.nblk = nblk; m.row0 = q.row0 + t * TT; m.ntok = ntok; m.head = head;
          m.pos0 = q.pos0 + t * TT; m.lo = q.lo; m.hi = q.hi;
          m.part = whole ? -1 : 2 * c + (blk == 0 ? 1 : 0);
          m.req = r;
          meta[slot] = m;
          mbar_arrive(&mfull[slot]);
        }
        if (++slot == C::SLOTS) { slot = 0; mphase ^= 1; }
        const int32_t* tab = P.table + (int64_t)r * P.max_blocks;
        int page = page_of(tab, b0 + blk, q.lo, q.hi);
        for (int i = 0; i < nblk && up; ++i) {
          const int b = b0 + blk + i;
          const int next = i + 1 < nblk ? page_of(tab, b + 1, q.lo, q.hi) : -1;
          up = load(&tk, stage, sphase, b, head, page);
          stage += step;
          if (up && i == 0) {
            wait_phase(qempty, qphase, dead, P.status);
            qphase ^= 1;
            if (*dead) { up = false; break; }
            const int halves = ntok > TS ? 2 : 1;
            if (lane == 0) {
              mbar_arrive_expect_tx(qfull, halves * (HD / 64) * TS * P.rep * 128);
              for (int h = 0; h < halves; ++h)
                for (int x = 0; x < HD / 64; ++x)
                  tma_rows(smem + h * C::TILE + x * 16384, &tq, 64 * x, head * P.rep,
                           q.row0 + t * TT + h * TS, qfull);
            }
            __syncwarp();
          }
          if (up && !split_v) {
            up = load(&tv, stage, sphase, b, head, page);
            ++stage;
          }
          if (stage >= ST) { stage = 0; sphase ^= 1; }
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
      int slot = 0;
      uint32_t mphase = 0;
      auto kst = [](uint32_t b) { return (2 * b) % ST; };
      auto kph = [](uint32_t b) { return ((2 * b) / ST) & 1; };
      // S from the K block in stage st
      auto s_product = [&](uint32_t st) {
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk) {
          const uint32_t off = ((uint32_t)(kk >> 2) * 16384u + (uint32_t)(kk & 3) * 32u) >> 4;
          tc_mma(t_s, dq + off, dk + (st * (C::TILE / 16) + off), id_s, kk != 0);
        }
        tc_commit(&sfull[h]);
      };
      for (;;) {
        wait_phase(&mfull[slot], mphase, dead, P.status);
        if (*dead) break;
        const int nblk = meta[slot].nblk;
        const bool mine = h == 0 || meta[slot].ntok > TS;
        __syncwarp();
        if (lane == 0) mbar_arrive(&mempty[slot]);
        if (nblk == 0) break;
        if (++slot == C::SLOTS) { slot = 0; mphase ^= 1; }
        wait_phase(qfull, qn & 1, dead, P.status);
        ++qn;
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
  } else {
    // ------------------------------------------------------------ softmax
    setmaxnreg_inc<PC_REGS_SOFT>();
    const int half = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_t = T_S + 128u * half + lanes, o_t = T_O + 128u * half + lanes;
    const int tok_in = P.token_of(row), hq_in = row - tok_in * P.rep;
    const float cs = fabsf(P.scale) * 1.4426950408889634f;
    const bool neg = P.scale < 0.f;
    constexpr float top = BF ? 0.f : PC_TOP_FP16;
    uint32_t blkn = 0, sn = 0, on = 0;
    int slot = 0;
    uint32_t mphase = 0;
    for (;;) {
      wait_phase(&mfull[slot], mphase, dead, P.status);
      if (*dead) break;
      const Tile m = meta[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&mempty[slot]);
      if (m.nblk == 0) break;
      if (++slot == C::SLOTS) { slot = 0; mphase ^= 1; }
      const int tok0 = half * TS;             // this half's first token of the tile
      if (tok0 >= m.ntok) {
        blkn += m.nblk;
        continue;
      }
      const int ntok = min(TS, m.ntok - tok0);
      const int pos0 = m.pos0 + tok0, pos = pos0 + min(tok_in, ntok - 1), end = pos0 + ntok - 1;
      const int last = min(pos, m.hi - 1), first = pos >= P.window ? pos - P.window + 1 : 0;
      // every row of the half sees the keys [all_lo, all_hi)
      const int all_lo = end >= P.window ? end - P.window + 1 : 0, all_hi = min(pos0 + 1, m.hi);
      float mx = -INFINITY, l = 0.f;
      for (int j = 0; j < m.nblk; ++j, ++blkn) {
        const int key0 = m.key0 + 128 * j;
        wait_phase(&sfull[half], sn & 1, dead, P.status);
        ++sn;
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
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if ((uint32_t)(i - c0) >= w) s[i] = -INFINITY;
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
          const int key = key0 + row;  // rows of 128 threads
          if (key < m.lo || key >= m.hi) {
            uint8_t* v = smem + C::o_kv + vst * C::TILE + row * 128;
#pragma unroll
            for (int x = 0; x < HD / 64; ++x)
#pragma unroll
              for (int i = 0; i < 8; ++i)
                *reinterpret_cast<uint4*>(v + x * 16384 + 16 * i) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[half]);
      }
      wait_phase(&ofull[half], on & 1, dead, P.status);
      ++on;
      tc_fence_after();
      const bool live = tok_in < ntok;
      const int prow = tok0 * P.rep + row;
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
                   (int64_t)(m.head * P.rep + rw - tk * P.rep) * HD + (lane & 3) * 8;
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
          P.lse[(int64_t)(m.row0 + tok0 + tok_in) * (P.hkv * P.rep) + m.head * P.rep + hq_in] =
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
  }
  tc_fence_before();
  __syncthreads();
  if (warp == PC_MMA) {
    tc_fence_after();
    tmem_dealloc(*tslot, 512);
  }
}

template <int HD, bool BF>
cudaError_t launch(const PagedAttnParams& p, const PagedKv& kv, const PagedParts& w, cudaStream_t st) {
  CUtensorMap tq, tk, tv;
  if (!make_page_tmap(&tk, kv.k, kv, HD, 128, 1, BF) || !make_page_tmap(&tv, kv.v, kv, HD, 128, 1, BF) ||
      !make_rows_tmap(&tq, p.q, p.rows, p.hkv * p.rep, HD, p.q_stride, p.rep, 128 / p.rep, BF))
    return cudaErrorInvalidValue;
  // the register split needs the block to be launched with what it counts on
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = paged_prepare((const void*)paged_chunk_kernel<HD, BF>,
                                      ChunkCfg<HD>::most, PC_REGS, p.device, &ready);
  if (e != cudaSuccess) return e;
  // behind the few-row kernel it is set up while that one ends; alone it is launched
  // behind the whole of what precedes (8192-token prompt 363 against 368 us)
  return paged_launch_if(p.few_rows > 0, paged_chunk_kernel<HD, BF>, w.ctas, PC_THREADS, ChunkCfg<HD>::total(p.n), st,
                         tq, tk, tv, p, w);
}

}  // namespace

cudaError_t paged_chunk_launch(const PagedAttnParams& p, const PagedKv& kv, const PagedParts& w, int d,
                               bool bf, cudaStream_t st) {
  if (d == 128) return bf ? launch<128, true>(p, kv, w, st) : launch<128, false>(p, kv, w, st);
  return bf ? launch<64, true>(p, kv, w, st) : launch<64, false>(p, kv, w, st);
}

}  // namespace mk
