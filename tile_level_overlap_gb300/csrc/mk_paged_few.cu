// Attention over a paged cache for requests with few rows (new tokens x query
// heads per kv head <= 16): decode steps and drafted tokens.
//
// Bound by HBM: every key and value of a (request, kv head) is read once, 4
// head_dim bytes, for 4 head_dim flops per row.  The work is the list of key
// blocks of all (request, kv head) pairs, end to end; each of the persistent
// CTAs (one per SM) takes an equal run of it, whatever the lengths, so a run
// may begin and end inside a pair's keys.  Such a part leaves its running
// maximum, sum and unnormalised output in the workspace, and a second launch
// joins the parts of each pair in the order of their keys.  Measured with 32 query
// heads on 8 kv heads of 128: 64 rows over 4096 keys in pages of 16 169 us (6.4
// TB/s), over 16384 627 us (6.9 TB/s); 2 x 4 drafted tokens over 128K keys in pages
// of 64 165 us (6.45 TB/s); one row over 4096 keys 9.5 us, join included.
//
// A warp walks the run: it posts each pair's description and query rows (bulk
// copies) to a small ring and loads the key blocks (32 KB of keys and values: 64
// keys at head_dim 128, 128 at 64) page by page through a ring with TMA, 128-byte
// swizzle; another loads the values (one warp for both took longer to issue the
// small pages' boxes than HBM takes for them: 64 x 4096 keys in pages of 16 174
// against 169 us, 32 ragged rows of heads of 64 23.8 against 20.7).  Eight
// consumer warps in two groups take the blocks in turn, 16 (32) keys each warp,
// with a softmax state of their own: S^T = K Q^T and O^T += V^T P^T by warp-level
// products, keys and dimensions on the 16-row side and the query rows on the
// 8-column side, so that 8 rows fill a product that would be half empty the other
// way round, and the softmax of a row stays in the lanes that rescale its output.
// The weights are rounded once to the cache's type for the product with V, as in
// the tile kernel (half a step of the softmax-weighted mean of |v|, about the
// output's own rounding; their sum keeps 32 bits).
// The legacy tensor path is ample here (a block costs its four warps 16 products
// each).  At the end of a pair the eight states are joined in shared memory.
#include "mk_paged_dev.cuh"
#include "mk_tmap.h"

namespace mk {
namespace {

constexpr int PF_WARPS = 8;             // consumers
constexpr int PF_THREADS = 32 * (PF_WARPS + 2);  // and two that load
constexpr int PF_STAGE = 32768;         // one block's keys, then its values
constexpr int PF_OVER = 1;              // what a pair costs beside its blocks, in blocks
// log2 of a row's largest weight in the product with V (its maximum is exact):
// weights lose bits only 2^28 below it, and are lost 2^39 below it, where fp16
// from 1 on has 2^14 and 2^25.
constexpr float PF_TOP_FP16 = 14.f;

template <int HD, int NT>
struct FewCfg {
  static constexpr int KS = HD == 128 ? 64 : 128;  // keys of a block
  static constexpr int RT = 8 * NT;                // rows of an item
  static constexpr int QROW = HD * 2 + 16;         // padded: conflict-free row reads
  static constexpr int QSLOTS = NT == 1 ? 4 : 3;
  static constexpr int OROW = HD + 4;              // floats; conflict-free column pairs
  static constexpr int STAGES = 5;
  static constexpr int o_q = STAGES * PF_STAGE;
  static constexpr int o_merge = o_q + QSLOTS * RT * QROW;
  static constexpr int o_ml = o_merge + PF_WARPS * 8 * OROW * 4;
  static constexpr int o_meta = o_ml + PF_WARPS * RT * 8;
  static constexpr int o_mask = o_meta + QSLOTS * 48;  // of trees
  static constexpr int o_bar = o_mask + QSLOTS * RT * 4;
  static constexpr int o_pre = o_bar + 8 * (2 * STAGES + 3 * QSLOTS) + 64;
  static constexpr int total(int n) { return o_pre + Kept::bytes(n); }
  static constexpr int most = o_pre + KEPT_MOST;
};
static_assert(FewCfg<128, 1>::most <= 232448 && FewCfg<128, 2>::most <= 232448, "shared memory of a CTA");

// One part of a (request, kv head): blocks [blk, blk + nblk) of its `of`.
struct Segment {
  int key0, nblk;            // first key; 0 blocks: the end of the run
  int row0, rows, head;
  int pos0, lo, hi;          // Request's
  int part;                  // workspace part, -1: all of the pair's blocks
  int req;                   // its request
  int pad[2];
};
static_assert(sizeof(Segment) == 48, "meta slot");
// A slot's rows have their masks behind the descriptions (the rows of a tree that
// comes here are at most 16 tokens: the first word).

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t movm(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
template <bool BF>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF) {
    mma_bf16_16816(c, a[0], a[1], a[2], a[3], b0, b1);
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}

// Whether any of the barrier's threads says so.
__device__ __forceinline__ bool any_of(int id, int n, bool x) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %3, 0;\n barrier.cta.red.or.pred q, %1, %2, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(id), "r"(n), "r"((uint32_t)x)
      : "memory");
  return r != 0;
}

// A CTA that gives up leaves only after its loads in flight, none of which
// takes a millisecond, have landed.
__device__ __noinline__ void let_copies_land() {
  const uint64_t t0 = globaltimer();
  while (globaltimer() - t0 < 1000000ull) {
  }
}

// (The bound for few rows keeps the kernel to 128 registers, so that the blocks
// of the join fit beside it and are set up before it ends.)
// TREE: rows see the cached keys and the new ones that their masks name (at most 16
// tokens come here: a word a row, which the loading warp fetches beside the page table;
// 32 requests of 4 tokens over 1280 keys take 42.4 us with masks and without, 1.7 times
// what HBM needs; 64 over 500 to 2000 76.5, one over 4096 16.1).
template <int HD, bool BF, int NT, bool TREE>
__global__ void __launch_bounds__(NT == 1 ? 512 : PF_THREADS, 1)
    paged_few_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                     const __grid_constant__ PagedAttnParams P, const __grid_constant__ PagedParts W) {
  using C = FewCfg<HD, NT>;
  constexpr int KS = C::KS, RT = C::RT, MT = KS / 64;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::o_bar);
  uint64_t* empty = full + C::STAGES;
  uint64_t* qfull = empty + C::STAGES;
  uint64_t* qempty = qfull + C::QSLOTS;
  uint64_t* mfull = qempty + C::QSLOTS;  // the description alone, for the warp that loads values
  volatile int* dead = reinterpret_cast<volatile int*>(mfull + C::QSLOTS);
  int* scan_tmp = const_cast<int*>(dead) + 1;
  const Kept kept(smem + C::o_pre, P.n);
  int* pre = kept.pre;
  Segment* meta = reinterpret_cast<Segment*>(smem + C::o_meta);
  uint32_t* mask_of = reinterpret_cast<uint32_t*>(smem + C::o_mask);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 2);
      mbar_init(&empty[s], PF_WARPS);
    }
    for (int s = 0; s < C::QSLOTS; ++s) {
      mbar_init(&qfull[s], 1);
      mbar_init(&mfull[s], 1);
      mbar_init(&qempty[s], PF_WARPS + 1);
    }
    *dead = 0;
    fence_mbar_init();
  }
  for (int i = tid; i < C::QSLOTS * RT * C::QROW / 16; i += PF_THREADS)
    reinterpret_cast<uint4*>(smem + C::o_q)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();

  grid_wait_prior();
  grid_launch_dependents();
  if (tid == 0) W.desc[blockIdx.x].parts = 0;

  // units: key blocks of all (request, kv head) pairs, pairs of a request end to end
  const int per = (P.n + PF_THREADS - 1) / PF_THREADS;
  uint32_t mine = 0;
  bool bad = false, falls = false;
  for (int i = 0; i < per; ++i) {
    const int r = tid * per + i;
    if (r >= P.n) break;
    const Request q = kept.read(P, r);
    bad |= q.bad;
    falls |= q.falls;
    int u = 0;
    if (q.add > 0 && (int64_t)q.add * P.rep <= P.few_rows)
      u = P.hkv * (max(1, (q.hi + KS - 1) / KS - q.lo / KS) + PF_OVER);
    pre[r] = u;
    mine += u;
  }
  const int T = place_units<PF_THREADS / 32>(P, pre, per, mine, falls, scan_tmp);
  if (bad && blockIdx.x == 0) latch(P.status, MK_ERR_BOUNDS);
  __syncthreads();

  // this CTA's run of units, of the G CTAs in use
  const int G = min((int)gridDim.x, T), c = blockIdx.x;
  if (c >= G) return;
  const Runs runs(T, G);
  const int u0 = runs.start(c), u1 = runs.start(c + 1);

  if (warp >= PF_WARPS) {
    // ------------------------------------------------------------- loads
    const int boxt = min(KS, 1 << P.page_shift), nbox = KS / boxt;
    const int mask = (1 << P.page_shift) - 1, my_tok = P.token_of(lane);
    // page of this lane's box of a block; -1 where no row sees any of it
    auto page_of = [&](const int32_t* tab, int b, int lo, int hi) {
      const int key = b * KS + lane * boxt;
      if (lane >= nbox || key >= hi || key + boxt <= lo) return -1;
      const int p = tab[key >> P.page_shift];
      if (p >= 0 && p < P.n_pages) return p;
      latch(P.status, MK_ERR_BOUNDS);
      return -1;
    };
    int stage = 0, slot = 0;
    uint32_t sphase = 1;
    // blocks [b0, b0 + nblk) of a head: their keys (at 0 of a stage) or values
    const CUtensorMap* tm = warp == PF_WARPS ? &tk : &tv;
    uint8_t* ring = smem + (warp == PF_WARPS ? 0 : PF_STAGE / 2);
    auto load = [&](const int32_t* tab, int b0, int nblk, int head, int lo, int hi, int page) {
      for (int i = 0; i < nblk; ++i) {
        const int next = i + 1 < nblk ? page_of(tab, b0 + i + 1, lo, hi) : -1;
        wait_phase(&empty[stage], sphase, dead, P.status);
        if (*dead) return false;
        if (lane == 0) mbar_arrive_expect_tx(&full[stage], PF_STAGE / 2);
        __syncwarp();
        if (lane < nbox)
          tma_page(ring + stage * PF_STAGE + lane * boxt * (2 * HD), tm, ((b0 + i) * KS + lane * boxt) & mask, 0, head,
                   page, &full[stage]);
        if (++stage == C::STAGES) { stage = 0; sphase ^= 1; }
        page = next;
      }
      return true;
    };
    if (warp > PF_WARPS) {  // values
      uint32_t mphase = 0;
      for (;;) {
        wait_phase(&mfull[slot], mphase, dead, P.status);
        if (*dead) return let_copies_land();
        const Segment s = meta[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(&qempty[slot]);
        if (s.nblk == 0) return;
        if (++slot == C::QSLOTS) { slot = 0; mphase ^= 1; }
        const int32_t* tab = P.table + (int64_t)s.req * P.max_blocks;
        const int b0 = s.key0 / KS;
        if (!load(tab, b0, s.nblk, s.head, s.lo, s.hi, page_of(tab, b0, s.lo, s.hi))) return let_copies_land();
      }
    }
    int r = find_le(pre, P.n, u0);
    uint32_t qphase = 1;  // parity of the "empty" waits
    for (int u = u0; u < u1;) {
      while (pre[r + 1] <= u) ++r;
      const Request q = kept.again(P, r);
      // units [x0, x1) of the pair: blocks [blk, blk + nblk)
      const int units = (pre[r + 1] - pre[r]) / P.hkv, local = u - pre[r], nb = units - PF_OVER;
      const int head = local / units, x0 = local - head * units, x1 = min(units, x0 + u1 - u);
      const int blk = max(0, x0 - PF_OVER), nblk = max(0, x1 - PF_OVER) - blk;
      if (nblk == 0) break;  // the run ends with the pair's overhead: the next CTA has it all
      const int b0 = q.lo / KS + blk, rows = q.add * P.rep;
      const int32_t* tab = P.table + (int64_t)r * P.max_blocks;
      const int page = page_of(tab, b0, q.lo, q.hi);
      uint32_t seen = 0;  // this lane's row, up to itself
      if constexpr (TREE)
        if (lane < rows) seen = P.masks[(int64_t)(q.row0 + my_tok) * P.mask_words] & ((2u << my_tok) - 1);
      const bool whole = blk == 0 && nblk == nb;
      if (blk == 0 && !whole) {  // joined by this CTA's block of the second launch
        const int last = runs.of(u - x0 + units - 1);  // CTA of the pair's last unit
        if (lane == 0) {
          PartDesc d;
          d.row0 = q.row0; d.rows = rows; d.head = head; d.parts = last - c + 1;
          W.desc[c] = d;
        }
      }
      wait_phase(&qempty[slot], qphase, dead, P.status);
      if (*dead) return let_copies_land();
      if constexpr (TREE) {
        if (lane < RT) mask_of[slot * RT + lane] = seen;
        __syncwarp();  // before lane 0's arrival
      }
      if (lane == 0) {
        Segment s;
        s.key0 = b0 * KS; s.nblk = nblk; s.row0 = q.row0; s.rows = rows; s.head = head;
        s.pos0 = q.pos0; s.lo = q.lo; s.hi = q.hi;
        s.part = whole ? -1 : 2 * c + (blk == 0 ? 1 : 0);
        s.req = r;
        meta[slot] = s;
        mbar_arrive(&mfull[slot]);
        mbar_arrive_expect_tx(&qfull[slot], (uint32_t)rows * HD * 2);
      }
      __syncwarp();
      if (lane < rows)
        bulk_in(smem + C::o_q + (slot * RT + lane) * C::QROW,
                 P.q + (int64_t)(q.row0 + my_tok) * P.q_stride + (int64_t)(head * P.rep + lane - my_tok * P.rep) * HD,
                 HD * 2, &qfull[slot]);
      if (++slot == C::QSLOTS) { slot = 0; qphase ^= 1; }
      if (!load(tab, b0, nblk, head, q.lo, q.hi, page)) return let_copies_land();
      u += x1 - x0;
    }
    // the end of the run
    wait_phase(&qempty[slot], qphase, dead, P.status);
    if (*dead) return let_copies_land();
    if (lane == 0) {
      meta[slot].nblk = 0;
      mbar_arrive(&mfull[slot]);
      mbar_arrive(&qfull[slot]);
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  const int grp = warp >> 2, kw = warp & 3, g = lane >> 2, t = lane & 3;
  const float cs = P.scale * 1.4426950408889634f;
  constexpr float top = BF ? 0.f : PF_TOP_FP16;
  float* merge = reinterpret_cast<float*>(smem + C::o_merge);
  float2* mls = reinterpret_cast<float2*>(smem + C::o_ml);
  // row and 16-byte chunk that this lane addresses in a 16 x 16 matrix load
  const int lr = (lane & 7) + ((lane >> 3) & 1) * 8, lc = lane >> 4;     // keys on rows
  const int vr = (lane & 7) + (lane >> 4) * 8, vc = (lane >> 3) & 1;     // transposed
  // A box holds the first 64 elements of its tokens, then the next 64: byte
  // offsets of this lane's rows in a block, and of a box's second half.
  const int bsh = min(P.page_shift, HD == 128 ? 6 : 7);
  const uint32_t part = HD == 128 ? 128u << bsh : 0u;
  auto row_at = [&](int key) -> uint32_t {
    return ((uint32_t)(key >> bsh) * (2u * HD) << bsh) + (uint32_t)(key & ((1 << bsh) - 1)) * 128u;
  };
  uint32_t k_at[MT], v_at[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    k_at[mt] = row_at((kw * MT + mt) * 16 + lr);
    v_at[mt] = row_at((kw * MT + mt) * 16 + vr);
  }
  int stage = 0, slot = 0, turn = 0;
  uint32_t sphase = 0, qphase = 0;
  for (;;) {
    wait_phase(&qfull[slot], qphase, dead, P.status);
    if (any_of(2, 32 * PF_WARPS, *dead)) break;  // all warps agree, also on giving up
    const Segment s = meta[slot];
    if (s.nblk == 0) break;
    const uint32_t qs = smem_u32(smem + C::o_q + slot * RT * C::QROW);
    uint32_t qf[NT][HD / 16][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k2 = 0; k2 < HD / 32; ++k2) {
        uint32_t r4[4];
        ldsm4(r4, qs + (nt * 8 + (lane & 7)) * C::QROW + k2 * 64 + (lane >> 3) * 16);
        qf[nt][2 * k2][0] = r4[0]; qf[nt][2 * k2][1] = r4[1];
        qf[nt][2 * k2 + 1][0] = r4[2]; qf[nt][2 * k2 + 1][1] = r4[3];
      }
    // keys [first, last] are what this lane's rows see (in a tree, of the cached ones;
    // of the new ones those in `named`)
    int first[NT][2], last[NT][2];
    uint32_t named[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = nt * 8 + 2 * t + e;
        int pos = s.pos0 + (row < s.rows ? P.token_of(row) : 0);
        if constexpr (TREE) {
          uint32_t m = mask_of[slot * RT + row];
          const int have = __popc(m);
          pos = s.pos0 + max(have, 1) - 1;
          for (int x = have; x > P.window; --x) m &= m - 1;
          named[nt][e] = m;
          last[nt][e] = min(s.pos0, s.hi) - 1;
        } else {
          last[nt][e] = min(pos, s.hi - 1);
        }
        first[nt][e] = pos >= P.window ? pos - P.window + 1 : 0;
      }
    __syncwarp();
    if (lane == 0) mbar_arrive(&qempty[slot]);
    if (++slot == C::QSLOTS) { slot = 0; qphase ^= 1; }
    float m[NT][2], l[NT][2], o[HD / 16][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < HD / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][nt][e] = 0.f;
    }
    // every row sees the keys [all_lo, all_hi)
    const int end = s.pos0 + P.token_of(s.rows - 1);
    const int all_lo = end >= P.window ? end - P.window + 1 : 0, all_hi = min(s.pos0 + (TREE ? 0 : 1), s.hi);
    for (int i = 0; i < s.nblk; ++i) {
      // both groups see every block's phase, also of those they leave to the
      // other one (a warp that skipped one could take the next for it)
      wait_phase(&full[stage], sphase, dead, P.status);
      if (turn == grp) {
        const uint32_t kb = smem_u32(smem + stage * PF_STAGE), vb = kb + PF_STAGE / 2;
        const int key0 = s.key0 + i * KS;
        const bool partial = key0 < all_lo || key0 + KS > all_hi;
        float sc[MT][NT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[mt][nt][e] = 0.f;
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            uint32_t a[4];
            const int ch = 2 * ks + lc;
            ldsm4(a, kb + k_at[mt] + (ks >= 4 ? part : 0u) + (((ch & 7) ^ (lr & 7)) << 4));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16<BF>(sc[mt][nt], a, qf[nt][ks][0], qf[nt][ks][1]);
          }
        }
        // softmax of the block's columns: this lane has keys g, g + 8 of each
        // 16, rows 2t and 2t + 1 of each 8
        float al[NT][2];
        bool move = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = -INFINITY;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float x = sc[mt][nt][2 * h + e] * cs;
                if (partial) {
                  const int key = key0 + (kw * MT + mt) * 16 + g + 8 * h;
                  bool out = key > last[nt][e] || key < first[nt][e];
                  if constexpr (TREE) {
                    const uint32_t j = (uint32_t)(key - s.pos0);  // (a cached key's is past 31)
                    if (j < 32u && (named[nt][e] >> j & 1u)) out = key >= s.hi;
                  }
                  if (out) x = -INFINITY;
                }
                sc[mt][nt][2 * h + e] = x;
                mx = fmaxf(mx, x);
              }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float mn = fmaxf(m[nt][e], mx), ref = mn == -INFINITY ? 0.f : mn;
            al[nt][e] = ex2(m[nt][e] - ref);
            move |= mn != m[nt][e];
            m[nt][e] = mn;
            float sum = 0.f;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float p = ex2(sc[mt][nt][2 * h + e] - (ref - top));
                sc[mt][nt][2 * h + e] = p;
                sum += p;
              }
            l[nt][e] = l[nt][e] * al[nt][e] + sum;
          }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
          for (int x = 0; x < HD / 16; ++x)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[x][nt][e] *= al[nt][e & 1];
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          uint32_t b[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            b[nt][0] = movm(down2<BF>(sc[mt][nt][0], sc[mt][nt][1]));
            b[nt][1] = movm(down2<BF>(sc[mt][nt][2], sc[mt][nt][3]));
          }
          // values of keys that no row sees may be anything: made zero
          uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
          if (partial) {
            const int key = key0 + (kw * MT + mt) * 16 + 2 * t;
            auto seen = [&](int k) { return k >= s.lo && k < s.hi; };
            keep0 = (seen(key) ? 0xffffu : 0u) | (seen(key + 1) ? 0xffff0000u : 0u);
            keep1 = (seen(key + 8) ? 0xffffu : 0u) | (seen(key + 9) ? 0xffff0000u : 0u);
          }
#pragma unroll
          for (int x = 0; x < HD / 16; ++x) {
            uint32_t a[4];
            const int ch = 2 * x + vc;
            ldsm4t(a, vb + v_at[mt] + (x >= 4 ? part : 0u) + (((ch & 7) ^ (vr & 7)) << 4));
            a[0] &= keep0; a[1] &= keep0; a[2] &= keep1; a[3] &= keep1;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16<BF>(o[x][nt], a, b[nt][0], b[nt][1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stage]);
      turn ^= 1;
      if (++stage == C::STAGES) { stage = 0; sphase ^= 1; }
    }

    // join the eight warps' states, eight rows at a time
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (nt * 8 >= s.rows) break;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[nt][e];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        l[nt][e] = x;
      }
      named_bar(1, 32 * PF_WARPS);  // the previous rows have been read
      if (g == 0) {
        mls[warp * RT + nt * 8 + 2 * t] = make_float2(m[nt][0] - top, l[nt][0]);
        mls[warp * RT + nt * 8 + 2 * t + 1] = make_float2(m[nt][1] - top, l[nt][1]);
      }
      float* mine_o = merge + warp * 8 * C::OROW;
#pragma unroll
      for (int x = 0; x < HD / 16; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mine_o[(2 * t + (e & 1)) * C::OROW + 16 * x + g + 8 * (e >> 1)] = o[x][nt][e];
      named_bar(1, 32 * PF_WARPS);
      constexpr int LPR = HD / 4;  // threads of a row
      const int row = tid / LPR, d4 = (tid % LPR) * 4, irow = nt * 8 + row;
      if (row < 8 && irow < s.rows) {
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < PF_WARPS; ++w) mm = fmaxf(mm, mls[w * RT + irow].x);
        const float ref = mm == -INFINITY ? 0.f : mm;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float ll = 0.f;
#pragma unroll
        for (int w = 0; w < PF_WARPS; ++w) {
          const float2 ml = mls[w * RT + irow];
          const float f = ex2(ml.x - ref);
          const float4 v = *reinterpret_cast<const float4*>(merge + (w * 8 + row) * C::OROW + d4);
          ll += ml.y * f;
          acc.x += v.x * f; acc.y += v.y * f; acc.z += v.z * f; acc.w += v.w * f;
        }
        if (s.part < 0) {
          const int ti = P.token_of(irow), tok = s.row0 + ti, hq = s.head * P.rep + irow - ti * P.rep;
          const float inv = inv_of(ll);
          *reinterpret_cast<uint2*>(P.out + (int64_t)tok * P.o_stride + (int64_t)hq * HD + d4) =
              make_uint2(down2<BF>(acc.x * inv, acc.y * inv), down2<BF>(acc.z * inv, acc.w * inv));
          if (P.lse && d4 == 0)
            P.lse[(int64_t)tok * (P.hkv * P.rep) + hq] = lse_of(mm, ll);
        } else {
          *reinterpret_cast<float4*>(W.o + ((int64_t)s.part * W.rt + irow) * HD + d4) = acc;
          if (d4 == 0) W.ml[(int64_t)s.part * W.rt + irow] = make_float2(mm, ll);
        }
      }
    }
  }
}

// ---------------------------------------------------------------- join
// The parts of the pair (tile) that CTA c of a kernel left open, in the order
// of their keys: its own second part and the first parts of the CTAs after it.
// Latency bound: few bytes, read right after the launch that wrote them.
constexpr int JOIN_ROWS = 32;  // of a tile, a block
constexpr int JOIN_THREADS = 256;

template <int HD, bool BF>
__global__ void __launch_bounds__(JOIN_THREADS, 4) paged_join_kernel(const __grid_constant__ PagedAttnParams P,
                                                                  const __grid_constant__ PagedParts A,
                                                                  const __grid_constant__ PagedParts B) {
  constexpr int LPR = HD / 4, WARPS = JOIN_THREADS / 32, E = HD / 32;
  __shared__ uint2 rows_out[JOIN_ROWS][LPR + 1];
  __shared__ float shared_o[WARPS][HD];
  __shared__ float2 shared_ml[WARPS];
  grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, hqs = P.hkv * P.rep;
  if ((int)blockIdx.x < A.ctas) {
    // few-row kernel, parts [row][dimension]: a warp joins a row, lanes on the
    // dimensions; where the rows are fewer than the warps, 2^sh warps take
    // every 2^sh-th part.  A round trip to L2 takes most of a microsecond: the
    // first N parts are read with the description, before it says how many
    // there are (any part's place can be read).
    // While the launch before still runs, the block goes through the same code
    // once with what the workspace happens to hold and stores nothing: its
    // instructions, which the last kernels have pushed out of the SM's caches,
    // are fetched then (all reads here bypass L1).
    constexpr int N = 5;
    const int c = blockIdx.x, sh = P.join_shares, share = warp >> (3 - sh), step = WARPS >> sh;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
      if (pass) grid_wait_prior();
      PartDesc d;
      *reinterpret_cast<int4*>(&d) = __ldcg(reinterpret_cast<const int4*>(A.desc + c));
      if (!pass) {
        d.rows = step;
        d.parts = N;
      }
      for (int row0 = 0, rows = step; row0 < rows; row0 += step) {
        const int row = row0 + (warp & (step - 1));
        auto at = [&](int k) {
          const int part = k == 0 ? 2 * c + 1 : 2 * min(c + k, A.ctas - 1);
          return (int64_t)part * A.rt + row;
        };
        float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = 0.f;
        for (int i0 = 0, n = N; i0 < n; i0 += N) {
          float2 ml[N];
          float v[N][E];
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int64_t x = at(share + ((i0 + i) << sh));
            ml[i] = __ldcg(A.ml + x);
            const float* src = A.o + x * HD + lane * E;
            if constexpr (E == 4) *reinterpret_cast<float4*>(v[i]) = __ldcg(reinterpret_cast<const float4*>(src));
            else *reinterpret_cast<float2*>(v[i]) = __ldcg(reinterpret_cast<const float2*>(src));
          }
          n = (d.parts - share + (1 << sh) - 1) >> sh;  // parts of this share
          float mn = m;
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (i0 + i < n) mn = fmaxf(mn, ml[i].x);
          const float ref = mn == -INFINITY ? 0.f : mn, f0 = ex2(m - ref);
          l *= f0;
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] *= f0;
#pragma unroll
          for (int i = 0; i < N; ++i) {
            if (i0 + i < n) {
              const float f = ex2(ml[i].x - ref);
              l += ml[i].y * f;
#pragma unroll
              for (int e = 0; e < E; ++e) o[e] += v[i][e] * f;
            }
          }
          m = mn;
        }
        if (d.parts == 0) return;
        rows = d.rows;
        if (sh > 0) {  // (one pass over the rows)
#pragma unroll
          for (int e = 0; e < E; ++e) shared_o[warp][lane * E + e] = o[e];
          if (lane == 0) shared_ml[warp] = make_float2(m, l);
          __syncthreads();
          float mm = -INFINITY;
          for (int s = 0; s < 1 << sh; ++s) mm = fmaxf(mm, shared_ml[(warp & (step - 1)) + s * step].x);
          const float ref = mm == -INFINITY ? 0.f : mm;
          l = 0.f;
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] = 0.f;
          for (int s = 0; s < 1 << sh; ++s) {
            const int w = (warp & (step - 1)) + s * step;
            const float f = ex2(shared_ml[w].x - ref);
            l += shared_ml[w].y * f;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] += shared_o[w][lane * E + e] * f;
          }
          m = mm;
          __syncthreads();
        }
        if (pass && row < d.rows && share == 0) {
          const int t = P.token_of(row), hq = d.head * P.rep + row - t * P.rep;
          const float inv = inv_of(l);
          uint32_t* dst = reinterpret_cast<uint32_t*>(P.out + (int64_t)(d.row0 + t) * P.o_stride + (int64_t)hq * HD) + lane * (E / 2);
#pragma unroll
          for (int e = 0; e < E; e += 2) dst[e / 2] = down2<BF>(o[e] * inv, o[e + 1] * inv);
          if (P.lse && lane == 0) P.lse[(int64_t)(d.row0 + t) * hqs + hq] = lse_of(m, l);
        }
      }
    }
    return;
  }
  grid_wait_prior();
  // tile kernel, parts [4 dimensions][row]: a block joins 32 rows, lanes on the
  // rows, each warp Q groups of four dimensions at once
  constexpr int Q = LPR / WARPS;
  const int per = B.rt / JOIN_ROWS, b = blockIdx.x - A.ctas, c = b / per, row0 = (b - c * per) * JOIN_ROWS;
  const int row = row0 + lane;
  const PartDesc d = B.desc[c];
  if (d.parts == 0 || row0 >= d.rows) return;
  float m = -INFINITY, l = 0.f;
  float4 o[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) o[q] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int k = 0; k < d.parts; ++k) {
    const int64_t part = k == 0 ? 2 * c + 1 : 2 * (c + k);
    const float2 ml = B.ml[part * B.rt + row];
    float4 v[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q)
      v[q] = *reinterpret_cast<const float4*>(B.o + part * B.rt * HD + ((warp * Q + q) * B.rt + row) * 4);
    const float mn = fmaxf(m, ml.x), ref = mn == -INFINITY ? 0.f : mn;
    const float x = ex2(m - ref), f = ex2(ml.x - ref);
    l = l * x + ml.y * f;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      o[q].x = o[q].x * x + v[q].x * f; o[q].y = o[q].y * x + v[q].y * f;
      o[q].z = o[q].z * x + v[q].z * f; o[q].w = o[q].w * x + v[q].w * f;
    }
    m = mn;
  }
  const float inv = inv_of(l);
#pragma unroll
  for (int q = 0; q < Q; ++q)
    rows_out[lane][warp * Q + q] = make_uint2(down2<BF>(o[q].x * inv, o[q].y * inv), down2<BF>(o[q].z * inv, o[q].w * inv));
  if (warp == 0 && P.lse && row < d.rows) {
    const int t = P.token_of(row);
    P.lse[(int64_t)(d.row0 + t) * hqs + d.head * P.rep + row - t * P.rep] = lse_of(m, l);
  }
  __syncthreads();
  for (int i = tid; i < JOIN_ROWS * LPR; i += JOIN_THREADS) {
    const int rw = row0 + i / LPR, q = i % LPR;
    if (rw >= d.rows) break;
    const int t = P.token_of(rw);
    *reinterpret_cast<uint2*>(P.out + (int64_t)(d.row0 + t) * P.o_stride +
                              (int64_t)(d.head * P.rep + rw - t * P.rep) * HD + q * 4) = rows_out[i / LPR][q];
  }
}

template <int HD, bool BF, int NT, bool TREE>
cudaError_t launch(const PagedAttnParams& p, const PagedKv& kv, const PagedParts& w, cudaStream_t st) {
  CUtensorMap tk, tv;
  if (!make_page_tmap(&tk, kv.k, kv, HD, FewCfg<HD, NT>::KS, HD / 64, BF) ||
      !make_page_tmap(&tv, kv.v, kv, HD, FewCfg<HD, NT>::KS, HD / 64, BF))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = paged_prepare((const void*)paged_few_kernel<HD, BF, NT, TREE>,
                                      FewCfg<HD, NT>::most, 0, p.device, &ready);
  if (e != cudaSuccess) return e;
  return paged_launch(paged_few_kernel<HD, BF, NT, TREE>, w.ctas, PF_THREADS, FewCfg<HD, NT>::total(p.n), st, tk, tv, p, w);
}

template <int HD, bool BF>
cudaError_t launch_rows(const PagedAttnParams& p, const PagedKv& kv, const PagedParts& w, cudaStream_t st) {
  if (p.masks) return p.few_rows <= 8 ? launch<HD, BF, 1, true>(p, kv, w, st) : launch<HD, BF, 2, true>(p, kv, w, st);
  return p.few_rows <= 8 ? launch<HD, BF, 1, false>(p, kv, w, st) : launch<HD, BF, 2, false>(p, kv, w, st);
}

}  // namespace

cudaError_t paged_few_launch(const PagedAttnParams& p, const PagedKv& kv, const PagedParts& w, int d,
                             bool bf, cudaStream_t st) {
  if (d == 128) return bf ? launch_rows<128, true>(p, kv, w, st) : launch_rows<128, false>(p, kv, w, st);
  return bf ? launch_rows<64, true>(p, kv, w, st) : launch_rows<64, false>(p, kv, w, st);
}

cudaError_t paged_join_launch(const PagedAttnParams& p, const PagedParts& a, const PagedParts& b, int d,
                              bool bf, cudaStream_t st) {
  const int grid = a.ctas + b.ctas * (b.rt / JOIN_ROWS);
  if (d == 128)
    return bf ? paged_launch(paged_join_kernel<128, true>, grid, JOIN_THREADS, 0, st, p, a, b)
              : paged_launch(paged_join_kernel<128, false>, grid, JOIN_THREADS, 0, st, p, a, b);
  return bf ? paged_launch(paged_join_kernel<64, true>, grid, JOIN_THREADS, 0, st, p, a, b)
            : paged_launch(paged_join_kernel<64, false>, grid, JOIN_THREADS, 0, st, p, a, b);
}

}  // namespace mk
