// Attention of chunks of new tokens over a paged cache on the 5th-generation
// tensor cores (tcgen05 + TMEM + TMA), bf16, head_dim D = 128 or 64.
//
// For a row at position p with keys u <= p:  z_u = scale <q, k_u>,
//   m = running base, l = sum 2^(z - m), o = sum 2^(z - m) v_u / l
// (z in units of log2(e)).  A CTA works through its share of the line of key
// tiles (paged.cuh); an item is 256 rows (new token, query head of the group)
// of one kv head, as two 128-row tiles Q0 / Q1 that share every K/V tile of 128
// keys.  Roles:
//   warps 0-3  softmax for Q0        warps 4-7  softmax for Q1
//   warp 8     TMA producer (and TMEM allocation)
//   warp 9     tcgen05.mma issuer    warp 10    cleans V tiles at the mask
//   warp 11    works out the CTA's parts, up to four ahead of the other roles
// Per tile: S_w = Q_w K^T (SS MMA, fp32 in TMEM), the softmax warps turn it into
// bf16 probabilities in place, O_w += P_w V (TS MMA).  The issue order PV0_i,
// S0_{i+1}, PV1_i, S1_{i+1} keeps the tensor cores on one row tile while the
// other's softmax runs.  The K/V pipeline runs on across the items of a CTA.
//
// A tile's pages are fetched as boxes of min(page, 128) slots by a 4-D map of
// the pool; pages that are missing are fetched from behind the pool, which reads
// as zeros and counts its bytes.  Slots behind a sequence's length may hold
// anything, and a later token's value may be an infinity or NaN: 0 times it would
// reach rows that do not see it.  Warp 10 therefore clears, in the tiles that
// some row does not see whole, the slots behind the end and the non-finite
// elements, and notes the keys that had some; the epilogue adds those elements
// to the rows that see them.
//
// Bound: the exponentials (16 a clock and SM) and the MMAs of a tile take 2048
// clocks each at D = 128 and overlap only in part, since S(i+1) cannot be issued
// before P(i), which lies in its place, is read.  Measured back to back, under the
// power cap (32 / 8 heads of 128): 4096 tokens at 131072 in 8.2 ms, 1055 TFLOP/s (0.76
// of the library product's sustained rate), 2048 at 65536 in 2.15 ms (1006); a prompt
// of 8192 tokens 590 us (931), of 2048 75 us (458), where setting up (6 us), queries,
// mask and epilogue of each item (some 5 us) and the joining of cut items (8 us)
// count.  At D = 64 the MMAs take half, the exponentials the same: 690 TFLOP/s for
// 4096 tokens at 16384, 510 for ragged chunks.
//
// TMEM: S0 [0,128) S1 [128,256) O0 [256,256+D) O1 [384,384+D) columns.
// SMEM: Q0 Q1, K and V double buffered, 128 rows x D each, 128-byte swizzled in
// 64-column halves.  Every wait is bounded (2 s); on expiry the CTA drains what
// it issued, frees TMEM and reports MOBA_ERR_TIMEOUT through the status word.
#include <cudaTypedefs.h>

#include <atomic>

#include "paged.cuh"
#include "sm100.cuh"

namespace moba {

namespace {

using namespace sm100;

constexpr int kQT = 128, kBK = 128, kBR = 256;
constexpr int kThreads = 384;
constexpr int kWorkers = 148;            // one CTA an SM
constexpr int kMinTiles = 2;
// What an item costs beside its tiles (2.1 us each): its queries' load, the
// cleaning at the mask and the epilogue take some 5 us.  With no cost counted,
// the workers of a short prompt's first items ended after 92 us and those of its
// last after 50.  1, 2, 3, 4, 5 tiles, one run: 79, 78, 75, 75, 75 us for 2048 tokens,
// 588, 558, 544, 547, 553 for 8192 (590 back to back under the power cap).
constexpr int kItemCost = 3;
constexpr int kReaders = 11;             // warps 0-10 read the planner's parts
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 216, kServiceRegs = 64;
static_assert(2 * 128 * kSoftmaxRegs + 128 * kServiceRegs <= kThreads * kLaunchRegs,
              "register split exceeds the launch allocation");
constexpr uint32_t kHalf = 16384;
// O is rescaled only when a row's max passes its base by 2^15; a tile whose
// probabilities sum to at most 2^15 cannot have done so, and is accepted
// without computing its max.  The two rules agree, so that a row's arithmetic
// does not depend on the other rows of its warp.
constexpr float kRescale = 15.f, kFastSumLimit = 32768.f;

template <int D>
struct Geo {
  static constexpr uint32_t kTile = kBK * D * 2;
  static constexpr int kHalves = D / 64;
  static constexpr uint32_t kOffQ = 0, kOffK = 2 * kTile, kOffV = 4 * kTile;
  // output rows on their way out, 32 channels of a warp's 32 rows
  static constexpr uint32_t kOffOut = 6 * kTile, kOutWarp = 32 * 64;
  static constexpr uint32_t kSmem = kOffOut + 8 * kOutWarp + 1024;
  static constexpr int kChunks = D / 8, kRowsPerOp = 32 / kChunks;
};

using Rounds = PagedRounds<kThreads, kWorkers>;

// a CTA's part of an item
struct Part {
  int b, h, first, len;   // sequence, kv head, row of its first new token, keys
  int t0, t1, tiles;      // key tiles of the part, and of the item
  int row0, rows, nq;     // nq = 0: the CTA's work is done
  int old;                // position of the sequence's first new token
  int all, fix0;          // keys that every row sees; the first tile that has others
  int parts;              // workers of the item, where this part begins it and does not end it
};

// Where the planner is in its CTA's work: whole items, then its part of the line's rest.
struct PagedWalk {
  PagedItem it;
  int64_t pos;
  int round;
};

struct Ctl {
  uint64_t q_full[2], k_full[2], v_full[2], v_fix[2], k_free[2], v_free[2], s_full[2], p_full[2], o_full[2];
  uint64_t f_full[4];
  uint64_t drain;
  uint32_t bad[4][4][4];   // [segment & 3][tile at the mask][32 keys each]: keys with non-finite values
  uint64_t part_full[4], part_empty[4];
  Part part[4];            // [segment & 3]
  uint32_t tmem_base;
  int abort;
};

MOBA_DEV uint32_t bar(const uint64_t* b) { return smem_u32(b); }

// 16-byte chunk c of row rr in the output staging (64-byte rows): a quarter-warp's
// rows, and a row's chunks, lie in different banks
MOBA_DEV uint32_t stage_off(int rr, int c) { return (uint32_t)(rr * 64 + ((c ^ ((rr >> 1) & 3)) << 4)); }
MOBA_DEV void st_shared_v4(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
MOBA_DEV uint4 ld_shared_v4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
MOBA_DEV void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// the non-finite halves of a packed pair cleared
MOBA_DEV void clear_nonfinite(uint32_t& w) {
  if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
  if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
}

// The planner's view of the line of tiles (whole warp).
struct Line {
  const PagedPlan<kThreads>& plan;
  const Rounds& rounds;
  const PagedArgs& a;
  const PagedDims& dm;
  int E, me;

  MOBA_DEV int64_t stop() const { return rounds.start[me + 1]; }
  MOBA_DEV bool more(const PagedWalk& k) const { return k.round < rounds.rounds || k.pos < stop(); }
  MOBA_DEV void find(PagedWalk& k) const {
    if (k.round < rounds.rounds)
      k.it = paged_locate_item<kBR, kBK, kItemCost>(rounds, (int64_t)k.round * E + me, a.cu, a.kv_len, dm);
    else if (k.pos < stop())
      k.it = paged_locate<kBR, kBK, kItemCost, kThreads>(plan, k.pos, a.cu, a.kv_len, dm);
  }
  MOBA_DEV PagedWalk first() const {
    PagedWalk k;
    k.round = 0;
    k.pos = rounds.start[me];
    find(k);
    return k;
  }
  MOBA_DEV Part part(const PagedWalk& k) const {
    const bool whole = k.round < rounds.rounds;
    Part p;
    p.b = k.it.b;
    p.h = k.it.h;
    p.first = k.it.s.first;
    p.len = k.it.s.len;
    p.tiles = k.it.tiles - kItemCost;
    p.t0 = whole ? 0 : max(k.it.tile - kItemCost, 0);
    p.t1 = whole ? p.tiles : (int)min((int64_t)k.it.tiles, k.it.tile + (stop() - k.pos)) - kItemCost;
    p.row0 = k.it.rt * kBR;
    p.rows = (int)min((uint32_t)kBR, (uint32_t)k.it.s.n * dm.G - p.row0);
    p.nq = p.rows > kQT ? 2 : 1;
    p.old = k.it.s.len - k.it.s.n;
    p.all = p.old + p.row0 / dm.G + 1;
    p.fix0 = max(p.all, 0) / kBK;
    p.parts = 0;
    if (p.t0 == 0 && p.t1 < p.tiles) {   // the workers whose parts of the rest begin before the item's end
      const int64_t end = k.pos - k.it.tile + k.it.tiles;
      int v = me + 1;
      while (v < E && rounds.start[v] < end) ++v;
      p.parts = v - me;
    }
    return p;
  }
  MOBA_DEV void next(PagedWalk& k) const {
    if (k.round < rounds.rounds) {
      ++k.round;
      find(k);
    } else {
      k.pos += k.it.tiles - k.it.tile;
      if (k.pos < stop()) paged_next<kBR, kBK, kItemCost>(k.it, a.cu, a.kv_len, dm);
    }
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
paged_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, PagedArgs a, PagedDims dm,
                int box, PagedHeader* __restrict__ hdr, float* __restrict__ part_o, float* __restrict__ part_ml) {
  using Gm = Geo<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Ctl ctl;
  __shared__ PagedPlan<kThreads> plan;
  __shared__ Rounds rounds;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  after_previous();
  const int64_t W = paged_plan<kBR, kBK, kItemCost, kThreads>(plan, a.cu, a.kv_len, dm, rounds.items, &rounds.largest);
  const int E = (int)min((int64_t)kWorkers, (W + kMinTiles - 1) / kMinTiles), me = blockIdx.x;
  if (tid == 0) hdr[me].parts = 0;
  if (blockIdx.x == 0 && a.status != nullptr)
    for (int b = tid; b < dm.batch; b += kThreads)
      if (a.kv_len[b] > ((int64_t)dm.max_pages << dm.page_shift)) atomicExch(a.status, (int)MOBA_ERR_INTERNAL);
  if (me >= E) return;

  if (tid == 0) {
    for (int w = 0; w < 2; ++w) {
      mbar_init(bar(&ctl.q_full[w]), kQT);
      mbar_init(bar(&ctl.p_full[w]), kQT);
      mbar_init(bar(&ctl.k_full[w]), 1);
      mbar_init(bar(&ctl.v_full[w]), 1);
      mbar_init(bar(&ctl.v_fix[w]), 32);
      mbar_init(bar(&ctl.k_free[w]), 1);
      mbar_init(bar(&ctl.v_free[w]), 2);   // the MMAs that read it, and warp 10
      mbar_init(bar(&ctl.s_full[w]), 1);
      mbar_init(bar(&ctl.o_full[w]), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(&ctl.f_full[i]), 32);
      mbar_init(bar(&ctl.part_full[i]), 1);
      mbar_init(bar(&ctl.part_empty[i]), kReaders);
    }
    mbar_init(bar(&ctl.drain), 1);
    ctl.abort = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(&ctl.tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  paged_rounds<kBR, kBK, kItemCost>(rounds, plan, W, E, a.cu, a.kv_len, dm);   // ends with a block barrier
  const Line line{plan, rounds, a, dm, E, me};
  tc_fence_after();
  const uint32_t tb = ctl.tmem_base;
  volatile int* abort_flag = &ctl.abort;
  // the CTA's parts one after another: the planner's next one is waited for and given back by each reading warp
  int seg = 0;
  auto await_part = [&]() { return mbar_wait(bar(&ctl.part_full[seg & 3]), (seg >> 2) & 1, abort_flag); };
  auto done_part = [&]() { mbar_arrive(bar(&ctl.part_empty[seg & 3])); };

  if (warp < 8)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftmaxRegs));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kServiceRegs));

  if (warp < 8) {
    // ------------------------------------------------------------ softmax
    const int w = warp >> 2, rho = tid & 127;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tb + (w ? 128u : 0u) + lane_off;
    const uint32_t tO = tb + (w ? 384u : 256u) + lane_off;
    const uint32_t qs = base + Gm::kOffQ + w * Gm::kTile;
    const float sl2 = dm.scale_log2;
    int tiles = 0, mine = 0;   // tiles and items this row tile took part in
    bool ok = true;
    // the thread's row of the part: its token, head and the end of its keys; rows behind the last take part as if
    // they saw all keys (their queries are zero)
    struct Row {
      bool valid;
      int tok, head, lim;
    };
    auto row_of = [&](const Part& p) {
      Row r;
      r.valid = w * kQT + rho < p.rows;
      const int row = p.row0 + w * kQT + rho;
      r.tok = r.valid ? row / dm.G : 0;
      r.head = p.h * dm.G + (r.valid ? row % dm.G : 0);
      r.lim = r.valid ? p.old + r.tok + 1 : 0x7fffffff;
      return r;
    };
    // the warp's 32 query rows of a part, whole rows a copy instruction
    auto load_q = [&](const Part& p) {
      const Row r = row_of(p);
      const int64_t qrow = (int64_t)(p.first + r.tok) * dm.q_stride + (int64_t)r.head * D;
      const int wrow0 = (warp & 3) * 32, cc = lane % Gm::kChunks;
#pragma unroll
      for (int k2 = 0; k2 < 32 / Gm::kRowsPerOp; ++k2) {
        const int rl = Gm::kRowsPerOp * k2 + lane / Gm::kChunks;
        const int64_t rs = __shfl_sync(0xffffffffu, (long long)qrow, rl);
        const bool vs = __shfl_sync(0xffffffffu, r.valid, rl);
        cp_async16(qs + (cc >> 3) * kHalf + sw128_off(wrow0 + rl, cc & 7), (const __nv_bfloat16*)a.q + (vs ? rs : 0) + cc * 8, vs);
      }
      cp_async_commit();
      cp_async_wait<0>();
      fence_proxy_async_smem();
      mbar_arrive(bar(&ctl.q_full[w]));
    };
    bool loaded = false;   // this part's queries, while the last part ended
    for (;; ++seg) {
      ok = __all_sync(0xffffffffu, await_part());
      if (!ok) break;
      const Part& p = ctl.part[seg & 3];
      if (p.nq == 0) break;
      const int t0 = p.t0, t1 = p.t1, lim = row_of(p).lim;
      if (w < p.nq) {
        if (!loaded) load_q(p);
        loaded = false;
        float m_used = -INFINITY, l = 0.f;
        auto load_s = [&](uint32_t (&sr)[128], int t) {
          tmem_ld32(tS + 0, sr);
          tmem_ld32(tS + 32, sr + 32);
          tmem_ld32(tS + 64, sr + 64);
          tmem_ld32(tS + 96, sr + 96);
          tmem_wait_ld();
          const int see = lim - t * kBK;
          if (see < kBK) {
#pragma unroll
            for (int c = 0; c < 128; ++c)
              if (c >= see) sr[c] = __float_as_uint(-INFINITY);
          }
        };
        // 2^(s scale log2(e) - mb) as bf16 pairs; returns their fp32 sum before the rounding (which moves each
        // by 2^-9 of itself at most, below the result's own rounding)
        auto exp_tile = [&](const uint32_t (&sr)[128], float mb, uint32_t (&pk)[64]) -> float {
          const uint64_t sl2x2 = f2_pack(sl2, sl2), nmbx2 = f2_pack(-mb, -mb);
          uint64_t rs4[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
          for (int c = 0; c < 64; ++c) {
            const uint64_t x2 =
                f2_fma(f2_pack(__uint_as_float(sr[2 * c]), __uint_as_float(sr[2 * c + 1])), sl2x2, nmbx2);
            float x0, x1;
            f2_unpack(x2, x0, x1);
            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
            rs4[c & 3] = f2_add(rs4[c & 3], f2_pack(p0, p1));
            pk[c] = pack_bf16x2(p0, p1);
          }
          float a0, a1;
          f2_unpack(f2_add(f2_add(rs4[0], rs4[1]), f2_add(rs4[2], rs4[3])), a0, a1);
          return a0 + a1;
        };
        for (int t = t0; t < t1 && ok; ++t, ++tiles) {
          ok = __all_sync(0xffffffffu, mbar_wait(bar(&ctl.s_full[w]), tiles & 1, abort_flag));
          if (!ok) break;
          tc_fence_after();
          uint32_t sr[128], pk[64];
          float ts = 0.f;
          load_s(sr, t);
          bool slow = __any_sync(0xffffffffu, m_used == -INFINITY);
          if (!slow) {
            ts = exp_tile(sr, m_used, pk);
            slow = __any_sync(0xffffffffu, !(ts <= kFastSumLimit));
            if (slow) load_s(sr, t);
          }
          if (slow) {
            float mx4[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) mx4[u] = fmaxf(__uint_as_float(sr[2 * u]), __uint_as_float(sr[2 * u + 1]));
#pragma unroll
            for (int c = 8; c < 128; c += 8)
#pragma unroll
              for (int u = 0; u < 4; ++u)
                mx4[u] = max3(mx4[u], __uint_as_float(sr[c + 2 * u]), __uint_as_float(sr[c + 2 * u + 1]));
            const float mxs = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * sl2;
            const bool need = mxs > m_used + kRescale;
            if (t > t0 && __any_sync(0xffffffffu, need)) {
              // S complete implies that the PV before it is (MMA issue order), so O is final here
              const float f = need ? exp2f(m_used - mxs) : 1.f;
#pragma unroll
              for (int cc = 0; cc < D / 32; ++cc) {
                uint32_t o[32];
                tmem_ld32(tO + cc * 32, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st32(tO + cc * 32, o);
              }
              tmem_wait_st();
            }
            if (need) {
              l *= exp2f(m_used - mxs);
              m_used = mxs;
            }
            ts = exp_tile(sr, m_used == -INFINITY ? 0.f : m_used, pk);
          }
          l += ts;
          tmem_st32(tS + 0, pk);
          tmem_st32(tS + 32, pk + 32);
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(bar(&ctl.p_full[w]));
        }
        if (ok) {
          // the last S is complete: the next part's queries take their place while PV runs
          ++seg;
          ok = __all_sync(0xffffffffu, await_part());
          loaded = ok && w < ctl.part[seg & 3].nq;
          if (loaded) load_q(ctl.part[seg & 3]);
          --seg;
        }
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(&ctl.o_full[w]), mine & 1, abort_flag) &&
                                                 mbar_wait(bar(&ctl.f_full[seg & 3]), (seg >> 2) & 1, abort_flag));
        if (ok) {
          tc_fence_after();
          const Row r = row_of(p);
          const bool valid = r.valid;
          const int tok = r.tok, head = r.head;
          const bool begins = p.t0 == 0, ends = p.t1 == p.tiles;
          const uint32_t(*bad)[4] = ctl.bad[seg & 3];
          uint32_t some = 0;
#pragma unroll
          for (int i = 0; i < 16; ++i) some |= bad[i >> 2][i & 3];
          // the non-finite values that the row sees, added to channels [32 cc, +32)
          auto add_bad = [&](uint32_t (&o)[32], int cc) {
            for (int i = 0; i < 16; ++i) {
              for (uint32_t bits = bad[i >> 2][i & 3]; bits != 0; bits &= bits - 1) {
                const int u = (p.fix0 + (i >> 2)) * kBK + (i & 3) * 32 + __ffs(bits) - 1;
                if (!valid || u >= lim) continue;
                const int64_t page = a.table[(int64_t)p.b * dm.max_pages + (u >> dm.page_shift)];
                if (page < 0 || page >= dm.num_pages) continue;
                const __nv_bfloat16* v = (const __nv_bfloat16*)a.v_pool + page * dm.v_page_stride +
                                         (((int64_t)p.h << dm.page_shift) + (u & ((1 << dm.page_shift) - 1))) * D + cc * 32;
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                  const float x = to_f32(v[e]);
                  if (!isfinite(x)) o[e] = __float_as_uint(__uint_as_float(o[e]) + x);
                }
              }
            }
          };
          if (begins && ends) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const uint32_t stg = base + Gm::kOffOut + (uint32_t)warp * Gm::kOutWarp;
            const int64_t orow = (int64_t)(p.first + tok) * dm.hq + head;
#pragma unroll
            for (int cc = 0; cc < D / 32; ++cc) {
              uint32_t o[32];
              tmem_ld32(tO + cc * 32, o);
              tmem_wait_ld();
              if (some) add_bad(o, cc);
#pragma unroll
              for (int e8 = 0; e8 < 4; ++e8)
                st_shared_v4(stg + stage_off(lane, e8),
                             pack_bf16x2(__uint_as_float(o[8 * e8 + 0]) * inv, __uint_as_float(o[8 * e8 + 1]) * inv),
                             pack_bf16x2(__uint_as_float(o[8 * e8 + 2]) * inv, __uint_as_float(o[8 * e8 + 3]) * inv),
                             pack_bf16x2(__uint_as_float(o[8 * e8 + 4]) * inv, __uint_as_float(o[8 * e8 + 5]) * inv),
                             pack_bf16x2(__uint_as_float(o[8 * e8 + 6]) * inv, __uint_as_float(o[8 * e8 + 7]) * inv));
              __syncwarp();
#pragma unroll
              for (int k2 = 0; k2 < 4; ++k2) {
                const int rl = 8 * k2 + (lane >> 2);
                const int64_t rd = __shfl_sync(0xffffffffu, (long long)orow, rl);
                const bool vd = __shfl_sync(0xffffffffu, valid, rl);
                const uint4 x = ld_shared_v4(stg + stage_off(rl, lane & 3));
                if (vd) *reinterpret_cast<uint4*>((__nv_bfloat16*)a.out + rd * D + cc * 32 + (lane & 3) * 8) = x;
              }
              __syncwarp();
            }
            if (valid && a.lse != nullptr)
              a.lse[(size_t)head * dm.tokens + p.first + tok] = l == 0.f ? -INFINITY : (m_used + log2f(l)) * kLn2;
          } else {
            const size_t slot = (size_t)(begins ? 2 * me + 1 : 2 * me) * kBR + w * kQT + rho;
            const uint32_t stg = base + Gm::kOffOut + (uint32_t)warp * Gm::kOutWarp;
#pragma unroll
            for (int cc = 0; cc < D / 32; ++cc) {
              uint32_t o[32];
              tmem_ld32(tO + cc * 32, o);
              tmem_wait_ld();
              if (some) add_bad(o, cc);
              // 16 channels of the warp's 32 rows at a time, so that a store writes 64 bytes of 8 rows
#pragma unroll
              for (int hh = 0; hh < 2; ++hh) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  st_shared_v4(stg + stage_off(lane, e), o[16 * hh + 4 * e], o[16 * hh + 4 * e + 1], o[16 * hh + 4 * e + 2],
                               o[16 * hh + 4 * e + 3]);
                __syncwarp();
#pragma unroll
                for (int k2 = 0; k2 < 4; ++k2) {
                  const int rl = 8 * k2 + (lane >> 2);
                  const uint4 x = ld_shared_v4(stg + stage_off(rl, lane & 3));
                  if (w * kQT + (warp & 3) * 32 + rl < p.rows)
                    *reinterpret_cast<uint4*>(part_o + (slot - lane + rl) * D + cc * 32 + hh * 16 + (lane & 3) * 4) = x;
                }
                __syncwarp();
              }
            }
            if (valid) *reinterpret_cast<float2*>(part_ml + 2 * slot) = make_float2(m_used, l);
            if (begins && tid == 0) {
              PagedHeader h;
              h.parts = p.parts;
              h.first = p.first;
              h.h = p.h;
              h.row0 = p.row0;
              h.rows = p.rows;
              h.pad[0] = h.pad[1] = h.pad[2] = 0;
              hdr[me] = h;
            }
          }
          tc_fence_before();   // O is read: the next P this warp hands over orders it before the next PV
        }
        ++mine;
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) done_part();
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmV);
    }
    int gt = 0, issued_k = 0, issued_v = 0;
    bool ok = true;
    for (;; ++seg) {
      ok = __all_sync(0xffffffffu, await_part());
      if (!ok) break;
      const Part p = ctl.part[seg & 3];
      if (p.nq == 0) break;
      const int32_t* row = a.table + (int64_t)p.b * dm.max_pages;
      const int have = (p.len + (1 << dm.page_shift) - 1) >> dm.page_shift;   // pages with keys
      // lanes hold 32 table entries, the next 32 on their way
      auto entries = [&](int first) {
        const int i = first + lane;
        int e = dm.num_pages;
        if (i < have) {
          e = row[i];
          if (e < 0 || e >= dm.num_pages) {
            e = dm.num_pages;   // behind the pool: reads as zeros
            if (a.status != nullptr) atomicExch(a.status, (int)MOBA_ERR_INTERNAL);
          }
        }
        return e;
      };
      int first = ((p.t0 * kBK) >> dm.page_shift) & ~31;
      int cur = entries(first), nxt = entries(first + 32);
      for (int t = p.t0; t < p.t1 && ok; ++t, ++gt) {
        const int s = gt & 1;
        const uint32_t ks = base + Gm::kOffK + s * Gm::kTile, vs = base + Gm::kOffV + s * Gm::kTile;
        const int u0 = t * kBK, p0 = u0 >> dm.page_shift;
        if (p0 >= first + 32) {
          first += 32;
          cur = nxt;
          nxt = entries(first + 32);
        }
        // a tile's pages (at most 8, aligned with their number) lie in one group of 32
        if (gt >= 2) ok = __all_sync(0xffffffffu, mbar_wait(bar(&ctl.k_free[s]), ((gt >> 1) - 1) & 1, abort_flag));
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(bar(&ctl.k_full[s]), Gm::kTile);
        __syncwarp();
        for (int r = 0; r < kBK; r += box) {
          const int page = __shfl_sync(0xffffffffu, cur, ((u0 + r) >> dm.page_shift) - first);
          const int y = (u0 + r) & ((1 << dm.page_shift) - 1);
          if (lane < Gm::kHalves)
            tma_load_4d(ks + lane * kHalf + r * 128, &tmK, 64 * lane, y, p.h, page, bar(&ctl.k_full[s]));
        }
        issued_k = gt + 1;
        if (gt >= 2) ok = __all_sync(0xffffffffu, mbar_wait(bar(&ctl.v_free[s]), ((gt >> 1) - 1) & 1, abort_flag));
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(bar(&ctl.v_full[s]), Gm::kTile);
        __syncwarp();
        for (int r = 0; r < kBK; r += box) {
          const int page = __shfl_sync(0xffffffffu, cur, ((u0 + r) >> dm.page_shift) - first);
          const int y = (u0 + r) & ((1 << dm.page_shift) - 1);
          if (lane < Gm::kHalves)
            tma_load_4d(vs + lane * kHalf + r * 128, &tmV, 64 * lane, y, p.h, page, bar(&ctl.v_full[s]));
        }
        issued_v = gt + 1;
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) done_part();
    }
    if (*abort_flag) {
      // let the copies this warp issued land before the CTA exits
      int never = 0;
      for (int i = (issued_k > 2 ? issued_k - 2 : 0); i < issued_k; ++i)
        mbar_wait(bar(&ctl.k_full[i & 1]), (i >> 1) & 1, &never);
      for (int i = (issued_v > 2 ? issued_v - 2 : 0); i < issued_v; ++i)
        mbar_wait(bar(&ctl.v_full[i & 1]), (i >> 1) & 1, &never);
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint32_t idS = idesc_bf16(128, kBK, false);
      const uint32_t idO = idesc_bf16(128, D, true);
      const uint32_t hi = sdesc_hi(1024);
      const uint32_t loQ = sdesc_lo(base + Gm::kOffQ, 16), loK = sdesc_lo(base + Gm::kOffK, 16),
                     loV = sdesc_lo(base + Gm::kOffV, kHalf);
      auto issue_s = [&](int w, int s) {
        const uint32_t qa = loQ + (w ? (Gm::kTile >> 4) : 0u), ka = loK + (s ? (Gm::kTile >> 4) : 0u);
        const uint32_t d = tb + (w ? 128u : 0u);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
          mma_ss(d, sdesc_join(qa + off, hi), sdesc_join(ka + off, hi), idS, kk > 0);
        }
        mma_commit(bar(&ctl.s_full[w]));
      };
      auto issue_pv = [&](int w, int s, bool acc) {
        const uint32_t va = loV + (s ? (Gm::kTile >> 4) : 0u);
        const uint32_t d = tb + (w ? 384u : 256u), pa = tb + (w ? 128u : 0u);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts(d, pa + kk * 8, sdesc_join(va + ((kk * 2048) >> 4), hi), idO, (acc || kk > 0) ? 1u : 0u);
      };
      int gt = 0, mine[2] = {0, 0}, tiles[2] = {0, 0}, fixed[2] = {0, 0};
      bool ok = true;
      for (;; ++seg) {
        ok = await_part();
        if (!ok) break;
        const struct { int t0, nq, fix0; } p = {ctl.part[seg & 3].t0, ctl.part[seg & 3].nq, ctl.part[seg & 3].fix0};
        if (p.nq == 0) break;
        const int n = ctl.part[seg & 3].t1 - p.t0;
        ok = mbar_wait(bar(&ctl.k_full[gt & 1]), (gt >> 1) & 1, abort_flag) &&
             mbar_wait(bar(&ctl.q_full[0]), mine[0] & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        issue_s(0, gt & 1);
        if (p.nq == 2) {
          ok = mbar_wait(bar(&ctl.q_full[1]), mine[1] & 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
          issue_s(1, gt & 1);
        }
        mma_commit(bar(&ctl.k_free[gt & 1]));
        for (int i = 0; i < n && ok; ++i, ++gt) {
          const int s = gt & 1, s1 = s ^ 1;
          const bool more = i + 1 < n;
          ok = mbar_wait(bar(&ctl.v_full[s]), (gt >> 1) & 1, abort_flag) &&
               (p.t0 + i < p.fix0 || mbar_wait(bar(&ctl.v_fix[s]), fixed[s]++ & 1, abort_flag)) &&
               (!more || mbar_wait(bar(&ctl.k_full[s1]), ((gt + 1) >> 1) & 1, abort_flag)) &&
               mbar_wait(bar(&ctl.p_full[0]), tiles[0]++ & 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
          issue_pv(0, s, i > 0);
          if (more) issue_s(0, s1); else mma_commit(bar(&ctl.o_full[0]));
          if (p.nq == 2) {
            if (!(ok = mbar_wait(bar(&ctl.p_full[1]), tiles[1]++ & 1, abort_flag))) break;
            tc_fence_after();
            issue_pv(1, s, i > 0);
            if (more) issue_s(1, s1); else mma_commit(bar(&ctl.o_full[1]));
          }
          mma_commit(bar(&ctl.v_free[s]));
          if (more) mma_commit(bar(&ctl.k_free[s1]));
        }
        ++mine[0];
        if (p.nq == 2) ++mine[1];
        if (!ok) break;
        done_part();
      }
      // every MMA this thread issued is complete before TMEM is released
      int never = 0;
      mma_commit(bar(&ctl.drain));
      mbar_wait(bar(&ctl.drain), 0, &never);
    }
  } else if (warp == 10) {
    // ------------------------------------------------------------ V tiles at the mask
    int gt = 0;
    bool ok = true;
    for (;; ++seg) {
      ok = __all_sync(0xffffffffu, await_part());
      if (!ok) break;
      const int t0 = ctl.part[seg & 3].t0, t1 = ctl.part[seg & 3].t1, fix0 = ctl.part[seg & 3].fix0,
                len = ctl.part[seg & 3].len, all = ctl.part[seg & 3].all;
      if (ctl.part[seg & 3].nq == 0) break;
      uint32_t* bad = &ctl.bad[seg & 3][0][0];
      if (lane < 16) bad[lane] = 0;
      __syncwarp();
      for (int t = t0; t < t1; ++t, ++gt) {
        // every tile is waited for and released here, whether it needs cleaning or not: a role that skipped tiles
        // would lose count of the barrier's phases
        const int s = gt & 1;
        ok = __all_sync(0xffffffffu, mbar_wait(bar(&ctl.v_full[s]), (gt >> 1) & 1, abort_flag));
        if (!ok) break;
        if (t >= fix0) {
          const uint32_t vs = base + Gm::kOffV + s * Gm::kTile;
          // keys from `all` on are not seen by every row; the ones before need no cleaning
#pragma unroll 1
          for (int r0 = max(all - t * kBK, 0) & ~31; r0 < kBK; r0 += 32) {
            const int r = r0 + lane;
            const bool behind = t * kBK + r >= len;
            // the largest exponent field decides (as magnitudes, 16-bit integers order like the values)
            uint32_t m = 0;
            if (behind) {
#pragma unroll
              for (int c = 0; c < Gm::kChunks; ++c) st_shared_v4(vs + (c >> 3) * kHalf + sw128_off(r, c & 7), 0, 0, 0, 0);
            } else {
#pragma unroll
              for (int c = 0; c < Gm::kChunks; ++c) {
                const uint4 x = ld_shared_v4(vs + (c >> 3) * kHalf + sw128_off(r, c & 7));
                m = __vmaxu2(m, __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                         __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
              }
            }
            const bool odd = (m & 0xffffu) >= 0x7f80u || (m >> 16) >= 0x7f80u;
            const uint32_t word = __ballot_sync(0xffffffffu, odd);
            if (word != 0) {
              if (odd) {
#pragma unroll 1
                for (int c = 0; c < Gm::kChunks; ++c) {
                  const uint32_t at = vs + (c >> 3) * kHalf + sw128_off(r, c & 7);
                  uint4 x = ld_shared_v4(at);
                  clear_nonfinite(x.x); clear_nonfinite(x.y); clear_nonfinite(x.z); clear_nonfinite(x.w);
                  st_shared_v4(at, x.x, x.y, x.z, x.w);
                }
              }
              if (lane == 0) bad[(t - fix0) * 4 + (r0 >> 5)] = word;
            }
          }
          fence_proxy_async_smem();
          mbar_arrive(bar(&ctl.v_fix[s]));
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(bar(&ctl.v_free[s]));
      }
      if (!ok) break;
      __syncwarp();
      mbar_arrive(bar(&ctl.f_full[seg & 3]));
      if (lane == 0) done_part();
    }
  } else {
    // ------------------------------------------------------------ planner
    PagedWalk walk = line.first();
    for (;; ++seg) {
      // the readers may be at work on the four parts before for longer than the other waits last (2 s are some 10^8
      // keys): up to 32 times that, unless one of them gave up
      bool ok = seg < 4;
      for (int i = 0; i < 32 && !ok && !*abort_flag; ++i) {
        int late = 0;
        ok = __all_sync(0xffffffffu, mbar_wait(bar(&ctl.part_empty[seg & 3]), ((seg >> 2) - 1) & 1, &late));
      }
      if (!__all_sync(0xffffffffu, ok)) break;
      Part p = {};
      if (line.more(walk)) p = line.part(walk);
      // a part that ends within an item's fixed cost has no keys: the next worker begins the item
      const bool more = p.nq != 0 && p.t1 > p.t0;
      if (!more) p.nq = 0;
      if (lane == 0) {
        ctl.part[seg & 3] = p;
        mbar_arrive(bar(&ctl.part_full[seg & 3]));
      }
      if (!more) break;
      line.next(walk);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tb, 512);
  if (tid == 0 && ctl.abort && a.status != nullptr) atomicExch(a.status, (int)MOBA_ERR_TIMEOUT);
}

template <int D>
cudaError_t launch(const PagedDims& dm, const PagedArgs& a, const PagedWs& l, cudaStream_t stream) {
  const int box = (1 << dm.page_shift) < kBK ? 1 << dm.page_shift : kBK;
  CUtensorMap mk, mv;
  if (!make_pool_map(&mk, a.k_pool, dm, D, dm.k_page_stride, box) ||
      !make_pool_map(&mv, a.v_pool, dm, D, dm.v_page_stride, box))
    return cudaErrorInvalidValue;
  // the setmaxnreg split is only safe if the kernel launches with kLaunchRegs
  static std::atomic<int> regs{-1};   // calls may come from several threads
  if (regs < 0) {
    cudaFuncAttributes fa;
    cudaError_t e = cudaFuncGetAttributes(&fa, paged_tc_kernel<D>);
    if (e != cudaSuccess) return e;
    regs = fa.numRegs;
  }
  if (regs < kLaunchRegs) return cudaErrorInvalidConfiguration;
  cudaError_t e = cudaFuncSetAttribute(paged_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_early(paged_tc_kernel<D>, kWorkers, kThreads, Geo<D>::kSmem, stream, mk, mv, a, dm, box, l.hdr, l.part_o,
                      l.part_ml);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> fn{nullptr};
  if (fn == nullptr) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult qr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &qr) == cudaSuccess &&
        qr == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  return fn;
}

}  // namespace

// map of a pool: [pages][heads][slots][D], boxes of `box` slots x 64 channels
bool make_pool_map(CUtensorMap* map, const void* pool, const PagedDims& dm, int D, int64_t page_stride, int box) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t page = 1ull << dm.page_shift;
  cuuint64_t dims[4] = {(cuuint64_t)D, page, (cuuint64_t)dm.hkv, (cuuint64_t)dm.num_pages};
  cuuint64_t strides[3] = {(cuuint64_t)D * 2, page * D * 2, (cuuint64_t)page_stride * 2};
  cuuint32_t boxes[4] = {64, (cuuint32_t)box, 1, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(pool), dims, strides, boxes, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t paged_tc_ws(int d) { return paged_ws_bytes(kWorkers, kBR, d); }

cudaError_t launch_paged_tc(const PagedDims& dm, int d, const PagedArgs& a, void* ws, cudaStream_t stream, int* launches) {
  const PagedWs l = paged_ws_layout(ws, kWorkers, kBR);
  cudaError_t e = d == 128 ? launch<128>(dm, a, l, stream) : launch<64>(dm, a, l, stream);
  if (e != cudaSuccess) return e;
  ++*launches;
  return launch_paged_combine(MOBA_BF16, d, l, kWorkers, kBR, a, dm, stream, launches);
}

}  // namespace moba
