// Attention of few new tokens a sequence over a paged cache (decode steps and
// short drafts), bf16, head_dim D = 128 or 64.
//
// For a row at position p with keys u <= p:  z_u = scale <q, k_u>,
//   m = running base, l = sum 2^(z - m), o = sum 2^(z - m) v_u / l
// (z in units of log2(e)), one pass over the keys.  Bound: reading the cache.
// The rows of a kv head's group are few, so a tensor-core tile of 128 rows would
// be mostly empty; one warp keeps 16 rows (new token, head of the group) as the
// fragments of m16n8k16 products, and needs no other warp until the end:
//   - a worker is a consumer warp with a producer warp of its own; it walks its
//     share of the line of 32-key tiles (paged.cuh) across items, its K/V tiles
//     arriving by TMA in a private ring of 3 stages, so that a block's four
//     workers keep 128 KB (D = 128) in flight and never meet;
//   - S = Q K^T and O += P V from swizzled shared memory (ldmatrix), the base
//     moved only when a row's max passes it by 2^8, probabilities rounded to bf16
//     for the product (2^-9 of each, the sum l unrounded);
//   - items cut by a worker's border are joined by the combine kernel.
// Measured (32 / 8 heads of 128): 64 sequences of up to 16K keys, 2.6 GB, in 408 us
// (6.4 TB/s, 0.98 of the copy benchmark's rate); 131072 keys of one sequence, 0.54 GB, in 86
// us and 8 more for joining the 74 parts of each head; the smallest call 11 us,
// some eight memory latencies one after another in the two kernels.
// In tiles that some row does not see whole, slots behind the sequence's end and
// non-finite values are cleared first and the latter added at the end to the
// rows that see them (0 times an infinity is not 0).
#include "paged.cuh"
#include "sm100.cuh"

namespace moba {

namespace {

using namespace sm100;

constexpr int kBR = 16, kBK = 32, kStages = 3, kPairs = 4;
constexpr int kThreads = 64 * kPairs;
constexpr int kMinTiles = 2;
constexpr float kRescale = 8.f;
// blocks an SM: the rings of one block with D = 128, of two with D = 64
constexpr int blocks_per_sm(int D) { return D == 128 ? 1 : 2; }
constexpr int workers(int D) { return 148 * blocks_per_sm(D) * kPairs; }

template <int D>
struct Geo {
  static constexpr uint32_t kHalf = kBK * 128;                 // 64 channels of a tile
  static constexpr uint32_t kTile = kBK * D * 2;               // K or V
  static constexpr uint32_t kStage = 2 * kTile, kRing = kStages * kStage;
  static constexpr uint32_t kSmem = kPairs * kRing + 1024;
};

MOBA_DEV void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
MOBA_DEV void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
MOBA_DEV void ldsm4_t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
MOBA_DEV void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
MOBA_DEV bool clear_nonfinite(uint32_t& w) {
  const bool lo = (w & 0x7f80u) == 0x7f80u, hi = (w & 0x7f800000u) == 0x7f800000u;
  if (lo) w &= 0xffff0000u;
  if (hi) w &= 0x0000ffffu;
  return lo || hi;
}

template <int D>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(D))
paged_decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, PagedArgs a, PagedDims dm,
                    int box, PagedHeader* __restrict__ hdr, float* __restrict__ part_o, float* __restrict__ part_ml) {
  using Gm = Geo<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ PagedPlan<kThreads> plan;
  __shared__ uint64_t full[kPairs][kStages], empty[kPairs][kStages];
  __shared__ int abort_word;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, pair = warp & (kPairs - 1);
  after_previous();
  if (tid < kPairs * kStages) {
    mbar_init(smem_u32(&full[tid / kStages][tid % kStages]), 1);
    mbar_init(smem_u32(&empty[tid / kStages][tid % kStages]), 1);
    fence_mbar_init();
  }
  if (tid == 0) abort_word = 0;
  const int64_t W = paged_plan<kBR, kBK, 0, kThreads>(plan, a.cu, a.kv_len, dm);   // two block barriers
  const int64_t E = min((int64_t)workers(D), (W + kMinTiles - 1) / kMinTiles);
  const int64_t me = (int64_t)blockIdx.x * kPairs + pair;
  volatile int* abort_flag = &abort_word;
  if (warp < kPairs && lane == 0) hdr[me].parts = 0;
  if (blockIdx.x == 0 && a.status != nullptr)
    for (int b = tid; b < dm.batch; b += kThreads)
      if (a.kv_len[b] > ((int64_t)dm.max_pages << dm.page_shift)) atomicExch(a.status, (int)MOBA_ERR_INTERNAL);
  if (me >= E) return;
  const int64_t stop = (me + 1) * W / E;
  int64_t pos = me * W / E;
  PagedItem it = paged_locate<kBR, kBK, 0, kThreads>(plan, pos, a.cu, a.kv_len, dm);
  const uint32_t ring = ((smem_u32(smem_raw) + 1023u) & ~1023u) + pair * Gm::kRing;

  if (warp >= kPairs) {
    // ------------------------------------------------------------ producer
    int n = 0;   // tiles issued
    bool ok = true;
    while (pos < stop && ok) {
      const int t1 = (int)min((int64_t)it.tiles, it.tile + (stop - pos));
      const int32_t* row = a.table + (int64_t)it.b * dm.max_pages;
      const int have = (it.s.len + (1 << dm.page_shift) - 1) >> dm.page_shift;   // pages with keys
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
      int first = ((it.tile * kBK) >> dm.page_shift) & ~31;
      int cur = entries(first), nxt = entries(first + 32);
      for (int t = it.tile; t < t1; ++t, ++n) {
        const int s = n % kStages, u0 = t * kBK;
        if ((u0 >> dm.page_shift) >= first + 32) {
          first += 32;
          cur = nxt;
          nxt = entries(first + 32);
        }
        if (n >= kStages)
          ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&empty[pair][s]), (n / kStages - 1) & 1, abort_flag));
        if (!ok) break;
        const uint32_t fb = smem_u32(&full[pair][s]), dst = ring + s * Gm::kStage;
        if (lane == 0) mbar_arrive_expect_tx(fb, Gm::kStage);
        __syncwarp();
        for (int r = 0; r < kBK; r += box) {
          const int page = __shfl_sync(0xffffffffu, cur, ((u0 + r) >> dm.page_shift) - first);
          const int y = (u0 + r) & ((1 << dm.page_shift) - 1);
          // one lane a box: halves of K, then of V
          if (lane < 2 * (D / 64)) {
            const int half = lane % (D / 64), v = lane / (D / 64);
            tma_load_4d(dst + v * Gm::kTile + half * Gm::kHalf + r * 128, v ? &tmV : &tmK, 64 * half, y, it.h, page, fb);
          }
        }
      }
      pos += t1 - it.tile;
      if (pos < stop) paged_next<kBR, kBK, 0>(it, a.cu, a.kv_len, dm);
    }
    // the copies outlive neither the consumer nor this warp
    for (int i = n > kStages ? n - kStages : 0; i < n && ok; ++i)
      ok = mbar_wait(smem_u32(&empty[pair][i % kStages]), (i / kStages) & 1, abort_flag);
    if (!ok) {
      int never = 0;
      for (int i = n > kStages ? n - kStages : 0; i < n; ++i)
        mbar_wait(smem_u32(&full[pair][i % kStages]), (i / kStages) & 1, &never);
      if (lane == 0 && a.status != nullptr) atomicExch(a.status, (int)MOBA_ERR_TIMEOUT);
    }
    return;
  }

  // -------------------------------------------------------------- consumer
  const int r0 = lane >> 2, c0 = (lane & 3) * 2;   // fragment rows r0, r0 + 8; columns c0, c0 + 1 of each 8
  int n = 0;
  bool ok = true;
  while (pos < stop && ok) {
    const int t0 = it.tile, t1 = (int)min((int64_t)it.tiles, it.tile + (stop - pos));
    const int row0 = it.rt * kBR, rows = (int)min((int64_t)kBR, (int64_t)it.s.n * dm.G - row0);
    const int old = it.s.len - it.s.n;
    const int all = old + row0 / dm.G + 1;          // keys that every row sees
    const int fix0 = max(all, 0) / kBK;             // first tile that some row does not see whole
    int lim[2];
    uint32_t qf[D / 16][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = r0 + 8 * i;
      const bool valid = r < rows;
      const int tok = valid ? (row0 + r) / dm.G : 0, head = it.h * dm.G + (valid ? (row0 + r) % dm.G : 0);
      lim[i] = valid ? old + tok + 1 : 0x7fffffff;   // rows behind the last: zero queries that see all
      const __nv_bfloat16* q = (const __nv_bfloat16*)a.q + (int64_t)(it.s.first + tok) * dm.q_stride + (int64_t)head * D + c0;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        qf[kk][i] = valid ? *reinterpret_cast<const uint32_t*>(q + 16 * kk) : 0u;
        qf[kk][i + 2] = valid ? *reinterpret_cast<const uint32_t*>(q + 16 * kk + 8) : 0u;
      }
    }
    float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    uint32_t bad[2] = {0u, 0u};   // keys of tiles fix0, fix0 + 1 with non-finite values

    for (int t = t0; t < t1; ++t, ++n) {
      const int s = n % kStages;
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&full[pair][s]), (n / kStages) & 1, abort_flag));
      if (!ok) break;
      const uint32_t kt = ring + s * Gm::kStage, vt = kt + Gm::kTile;
      if (t >= fix0) {
        const bool behind = t * kBK + lane >= it.s.len;
        bool odd = false;
        for (int c = 0; c < D / 8; ++c) {
          const uint32_t at = vt + (c >> 3) * Gm::kHalf + sw128_off(lane, c & 7);
          uint32_t x[4];
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n"
                       : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at) : "memory");
          bool any = behind;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool b = clear_nonfinite(x[e]);
            if (behind) x[e] = 0u;
            odd |= b && !behind;
            any |= b;
          }
          if (any)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(at), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3])
                         : "memory");
        }
        const uint32_t word = __ballot_sync(0xffffffffu, odd);
        if (t == fix0) bad[0] = word; else bad[1] = word;
        fence_proxy_async_smem();   // the stage is written by TMA next
        __syncwarp();
      }
      // S: 16 rows x 32 keys
      float z[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) z[i][0] = z[i][1] = z[i][2] = z[i][3] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const int key = 16 * p + ((lane >> 4) << 3) + (lane & 7), c = 2 * kk + ((lane >> 3) & 1);
          uint32_t b[4];
          ldsm4(b, kt + (c >> 3) * Gm::kHalf + sw128_off(key, c & 7));
          mma16816(z[2 * p], qf[kk], b[0], b[1]);
          mma16816(z[2 * p + 1], qf[kk], b[2], b[3]);
        }
      }
      const bool masked = t >= fix0;
      float base[2];
      bool move[2];
      float mx[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mx[i] = -INFINITY;
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float& x = z[nt][2 * i + e];
            x *= dm.scale_log2;
            if (masked && t * kBK + nt * 8 + c0 + e >= lim[i]) x = -INFINITY;
            mx[i] = fmaxf(mx[i], x);
          }
        }
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
        move[i] = mx[i] > m[i] + kRescale;
      }
      if (__any_sync(0xffffffffu, move[0] || move[1])) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float f = move[i] ? exp2f(m[i] - mx[i]) : 1.f;
          if (move[i]) m[i] = mx[i];
          l[i] *= f;
#pragma unroll
          for (int nt = 0; nt < D / 8; ++nt) {
            o[nt][2 * i] *= f;
            o[nt][2 * i + 1] *= f;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        base[i] = m[i] == -INFINITY ? 0.f : m[i];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            z[nt][2 * i + e] = ex2_approx(z[nt][2 * i + e] - base[i]);
            l[i] += z[nt][2 * i + e];
          }
        }
      }
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        const uint32_t pf[4] = {pack_bf16x2(z[2 * kk][0], z[2 * kk][1]), pack_bf16x2(z[2 * kk][2], z[2 * kk][3]),
                                pack_bf16x2(z[2 * kk + 1][0], z[2 * kk + 1][1]), pack_bf16x2(z[2 * kk + 1][2], z[2 * kk + 1][3])};
#pragma unroll
        for (int dp = 0; dp < D / 16; ++dp) {
          const int key = 16 * kk + (((lane >> 3) & 1) << 3) + (lane & 7), c = 2 * dp + (lane >> 4);
          uint32_t b[4];
          ldsm4_t(b, vt + (c >> 3) * Gm::kHalf + sw128_off(key, c & 7));
          mma16816(o[2 * dp], pf, b[0], b[1]);
          mma16816(o[2 * dp + 1], pf, b[2], b[3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&empty[pair][s]));
    }
    if (!ok) break;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    }
    if (bad[0] | bad[1]) {
      // the non-finite values that a row sees
      for (int f = 0; f < 2; ++f) {
        for (uint32_t bits = bad[f]; bits != 0; bits &= bits - 1) {
          const int u = (fix0 + f) * kBK + __ffs(bits) - 1;
          const int64_t page = a.table[(int64_t)it.b * dm.max_pages + (u >> dm.page_shift)];
          if (page < 0 || page >= dm.num_pages) continue;
          const __nv_bfloat16* v = (const __nv_bfloat16*)a.v_pool + page * dm.v_page_stride +
                                   (((int64_t)it.h << dm.page_shift) + (u & ((1 << dm.page_shift) - 1))) * D + c0;
#pragma unroll
          for (int nt = 0; nt < D / 8; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float x = to_f32(v[8 * nt + e]);
              if (!isfinite(x)) {
                if (u < lim[0]) o[nt][e] += x;
                if (u < lim[1]) o[nt][2 + e] += x;
              }
            }
          }
        }
      }
    }
    const bool begins = t0 == 0, ends = t1 == it.tiles;
    if (begins && !ends && lane == 0) {
      PagedHeader h;
      h.parts = paged_parts(pos + it.tiles, W, E, me);
      h.first = it.s.first;
      h.h = it.h;
      h.row0 = row0;
      h.rows = rows;
      h.pad[0] = h.pad[1] = h.pad[2] = 0;
      hdr[me] = h;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = r0 + 8 * i;
      if (r >= rows) continue;
      if (begins && ends) {
        const int tok = it.s.first + (row0 + r) / dm.G, head = it.h * dm.G + (row0 + r) % dm.G;
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
        __nv_bfloat16* dst = (__nv_bfloat16*)a.out + ((size_t)tok * dm.hq + head) * D + c0;
#pragma unroll
        for (int nt = 0; nt < D / 8; ++nt)
          *reinterpret_cast<uint32_t*>(dst + 8 * nt) = pack_bf16x2(o[nt][2 * i] * inv, o[nt][2 * i + 1] * inv);
        if (c0 == 0 && a.lse != nullptr)
          a.lse[(size_t)head * dm.tokens + tok] = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
      } else {
        const size_t slot = (size_t)(begins ? 2 * me + 1 : 2 * me) * kBR + r;
#pragma unroll
        for (int nt = 0; nt < D / 8; ++nt)
          *reinterpret_cast<float2*>(part_o + slot * D + 8 * nt + c0) = make_float2(o[nt][2 * i], o[nt][2 * i + 1]);
        if (c0 == 0) *reinterpret_cast<float2*>(part_ml + 2 * slot) = make_float2(m[i], l[i]);
      }
    }
    pos += t1 - t0;
    if (pos < stop) paged_next<kBR, kBK, 0>(it, a.cu, a.kv_len, dm);
  }
}

template <int D>
cudaError_t launch(const PagedDims& dm, const PagedArgs& a, const PagedWs& l, cudaStream_t stream) {
  const int box = (1 << dm.page_shift) < kBK ? 1 << dm.page_shift : kBK;
  CUtensorMap mk, mv;
  if (!make_pool_map(&mk, a.k_pool, dm, D, dm.k_page_stride, box) ||
      !make_pool_map(&mv, a.v_pool, dm, D, dm.v_page_stride, box))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(paged_decode_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_early(paged_decode_kernel<D>, workers(D) / kPairs, kThreads, Geo<D>::kSmem, stream, mk, mv, a, dm, box, l.hdr,
                      l.part_o, l.part_ml);
}

}  // namespace

size_t paged_decode_ws(int d) { return paged_ws_bytes(workers(d), kBR, d); }

cudaError_t launch_paged_decode(const PagedDims& dm, int d, const PagedArgs& a, void* ws, cudaStream_t stream, int* launches) {
  const PagedWs l = paged_ws_layout(ws, workers(d), kBR);
  cudaError_t e = d == 128 ? launch<128>(dm, a, l, stream) : launch<64>(dm, a, l, stream);
  if (e != cudaSuccess) return e;
  ++*launches;
  return launch_paged_combine(MOBA_BF16, d, l, workers(d), kBR, a, dm, stream, launches);
}

}  // namespace moba
