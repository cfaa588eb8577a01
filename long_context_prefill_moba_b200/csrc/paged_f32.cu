// Attention of chunks of new tokens over a paged cache in fp32, on CUDA cores.
//
// For a row at position p with keys u <= p:  z_u = scale <q, k_u>,
//   m = running max, l = sum 2^(z - m), o = sum 2^(z - m) v_u / l
// (z in units of log2(e)).  fp32 results are held to fp32 accuracy, so the
// products run as packed fp32 FMAs, which bound the kernel (128 a clock and SM).
// A worker is a block of 128 threads, two to an SM: 64 rows (new token, head of
// the group) against BK keys a step, both products as register tiles: a thread
// has 4 rows x BK/8 keys of the scores and 4 rows x D/8 channels of o, so that
// 64 FMAs use 8 to 12 shared-memory reads of 16 bytes, broadcast or free of
// conflicts by rows padded to D + 4.  The 8 threads of 4 rows are neighbours in a
// warp: their max, and the probabilities they hand over, need no block barrier.
// Keys and values arrive by cp.async, one tile ahead; slots behind the
// sequence's end are filled with zeros, and in tiles that some row does not see
// whole a value meets only the rows that see it (0 times an infinity is not 0).
//
// Measured: 300 tokens at 8300 keys, 32 / 8 heads of 128, 1.05 ms (38 TFLOP/s;
// the FMA pipes are busy 57% of the time, shared memory 73%), three chunks of up to
// 257 tokens with 16 heads of 64 120 us, where a fifth of the row tiles is padding.
#include <type_traits>

#include "paged.cuh"
#include "sm100.cuh"

namespace moba {

namespace {

using sm100::f2_fma;
using sm100::f2_pack;
using sm100::f2_unpack;

constexpr int kBR = 64, kThreads = 128, kWorkers = 148 * 2, kMinTiles = 2;
// an item's queries, first tiles and epilogue, in tiles
constexpr int kItemCost = 1;

template <int D>
struct Geo {
  static constexpr int kBK = D == 64 ? 64 : 32;
  static constexpr int kRow = D + 4, kPRow = kBK + 4;
  static constexpr int kQ = kBR * kRow, kKV = kBK * kRow, kP = kBR * kPRow;
  static constexpr int kSmem = (kQ + 4 * kKV + kP) * (int)sizeof(float);
};

template <int D>
__global__ void __launch_bounds__(kThreads, 2) paged_f32_kernel(PagedArgs a, PagedDims dm, PagedHeader* __restrict__ hdr,
                                                               float* __restrict__ part_o, float* __restrict__ part_ml) {
  using Gm = Geo<D>;
  constexpr int BK = Gm::kBK, KPT = BK / 8, C4 = D / 32;   // keys, and groups of 4 channels, of a thread
  extern __shared__ __align__(16) float smem[];
  __shared__ PagedPlan<kThreads> plan;
  float* sq = smem;
  float* sk = sq + Gm::kQ;                // [2][BK][D + 4]
  float* sv = sk + 2 * Gm::kKV;
  float* sp = sv + 2 * Gm::kKV;           // [64][BK + 4]
  const int tid = threadIdx.x, tx = tid & 7, ty = tid >> 3;
  after_previous();
  const int64_t W = paged_plan<kBR, BK, kItemCost, kThreads>(plan, a.cu, a.kv_len, dm);
  const int64_t E = min((int64_t)kWorkers, (W + kMinTiles - 1) / kMinTiles), me = blockIdx.x;
  if (tid == 0) hdr[me].parts = 0;
  if (blockIdx.x == 0 && a.status != nullptr)
    for (int b = tid; b < dm.batch; b += kThreads)
      if (a.kv_len[b] > ((int64_t)dm.max_pages << dm.page_shift)) atomicExch(a.status, (int)MOBA_ERR_INTERNAL);
  if (me >= E) return;
  int64_t pos = me * W / E;
  const int64_t stop = (me + 1) * W / E;
  PagedItem it = paged_locate<kBR, BK, kItemCost, kThreads>(plan, pos, a.cu, a.kv_len, dm);

  for (; pos < stop;) {
    const int tiles = it.tiles - kItemCost, t0 = max(it.tile - kItemCost, 0),
              t1 = (int)min((int64_t)it.tiles, it.tile + (stop - pos)) - kItemCost;
    if (t1 <= t0) break;   // within the item's fixed cost: the next worker begins the item
    const int row0 = it.rt * kBR, rows = min(kBR, it.s.n * dm.G - row0);
    const int old = it.s.len - it.s.n, all = old + row0 / dm.G + 1;   // `all`: keys that every row sees
    const int32_t* table = a.table + (int64_t)it.b * dm.max_pages;

    auto load_tile = [&](int t, int buf) {
      constexpr int kChunks = D / 4;
#pragma unroll 4
      for (int i = tid; i < BK * kChunks; i += kThreads) {
        const int r = i / kChunks, c = i % kChunks, u = t * BK + r;
        int page = -1;
        if (u < it.s.len) {
          page = __ldg(table + (u >> dm.page_shift));
          if (page < 0 || page >= dm.num_pages) {
            page = -1;   // keys of a page that the pool does not have read as zeros
            if (c == 0 && a.status != nullptr) atomicExch(a.status, (int)MOBA_ERR_INTERNAL);
          }
        }
        const int64_t at = (((int64_t)it.h << dm.page_shift) + (u & ((1 << dm.page_shift) - 1))) * D + 4 * c;
        const bool live = page >= 0;
        cp_async16(smem_u32(sk + buf * Gm::kKV + r * Gm::kRow + 4 * c),
                   (const float*)a.k_pool + (live ? page * dm.k_page_stride + at : 0), live);
        cp_async16(smem_u32(sv + buf * Gm::kKV + r * Gm::kRow + 4 * c),
                   (const float*)a.v_pool + (live ? page * dm.v_page_stride + at : 0), live);
      }
      cp_async_commit();
    };
    for (int i = tid; i < kBR * (D / 4); i += kThreads) {
      const int r = i / (D / 4), c = i % (D / 4);
      const bool live = r < rows;
      const int tok = live ? (row0 + r) / dm.G : 0, head = it.h * dm.G + (live ? (row0 + r) % dm.G : 0);
      cp_async16(smem_u32(sq + r * Gm::kRow + 4 * c),
                 (const float*)a.q + (int64_t)(it.s.first + tok) * dm.q_stride + (int64_t)head * D + 4 * c, live);
    }
    load_tile(t0, t0 & 1);

    uint64_t o[4][2 * C4];
    float m[4], l[4];
    int lim[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
      const int row = 4 * ty + r;
      lim[r] = row < rows ? old + (row0 + row) / dm.G + 1 : 0;
#pragma unroll
      for (int c = 0; c < 2 * C4; ++c) o[r][c] = 0;
    }
    for (int t = t0; t < t1; ++t) {
      if (t + 1 < t1) {
        load_tile(t + 1, (t + 1) & 1);
        cp_async_wait<1>();
      } else {
        cp_async_wait<0>();
      }
      __syncthreads();
      const float* kt = sk + (t & 1) * Gm::kKV;
      const float* vt = sv + (t & 1) * Gm::kKV;
      // scores: keys tx + 8 i; even and odd channels summed apart in the halves of a pair
      uint64_t s[4][KPT];
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int i = 0; i < KPT; ++i) s[r][i] = 0;
#pragma unroll 16
      for (int c = 0; c < D; c += 4) {
        ulonglong2 q[4], k[KPT];
#pragma unroll
        for (int r = 0; r < 4; ++r) q[r] = *reinterpret_cast<const ulonglong2*>(sq + (4 * ty + r) * Gm::kRow + c);
#pragma unroll
        for (int i = 0; i < KPT; ++i) k[i] = *reinterpret_cast<const ulonglong2*>(kt + (tx + 8 * i) * Gm::kRow + c);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int i = 0; i < KPT; ++i) s[r][i] = f2_fma(q[r].y, k[i].y, f2_fma(q[r].x, k[i].x, s[r][i]));
      }
      const bool masked = (t + 1) * BK > all;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float z[KPT], top = -INFINITY;
#pragma unroll
        for (int i = 0; i < KPT; ++i) {
          float x, y;
          f2_unpack(s[r][i], x, y);
          z[i] = (x + y) * dm.scale_log2;
          if (masked && t * BK + tx + 8 * i >= lim[r]) z[i] = -INFINITY;
          top = fmaxf(top, z[i]);
        }
#pragma unroll
        for (int x = 4; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        const float mn = fmaxf(m[r], top), base = mn == -INFINITY ? 0.f : mn;
        if (mn != m[r]) {
          const float f = exp2f(m[r] - base);
          const uint64_t f2 = f2_pack(f, f);
          l[r] *= f;
          m[r] = mn;
#pragma unroll
          for (int c = 0; c < 2 * C4; ++c) o[r][c] = f2_fma(o[r][c], f2, 0ull);
        }
#pragma unroll
        for (int i = 0; i < KPT; ++i) {
          const float p = exp2f(z[i] - base);
          l[r] += p;
          sp[(4 * ty + r) * Gm::kPRow + tx + 8 * i] = p;
        }
      }
      __syncwarp();
      // o += P V; in tiles that some row does not see whole, key by key as the rows see them
      auto add_pv = [&](auto whole) {
#pragma unroll 4
        for (int u = 0; u < BK; u += 4) {
          float4 p[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) p[r] = *reinterpret_cast<const float4*>(sp + (4 * ty + r) * Gm::kPRow + u);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            ulonglong2 v[C4];
#pragma unroll
            for (int c = 0; c < C4; ++c) v[c] = *reinterpret_cast<const ulonglong2*>(vt + (u + e) * Gm::kRow + 4 * tx + 32 * c);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float x = e == 0 ? p[r].x : e == 1 ? p[r].y : e == 2 ? p[r].z : p[r].w;
              if (!decltype(whole)::value && t * BK + u + e >= lim[r]) continue;
              const uint64_t x2 = f2_pack(x, x);
#pragma unroll
              for (int c = 0; c < C4; ++c) {
                o[r][2 * c] = f2_fma(x2, v[c].x, o[r][2 * c]);
                o[r][2 * c + 1] = f2_fma(x2, v[c].y, o[r][2 * c + 1]);
              }
            }
          }
        }
      };
      if (masked) add_pv(std::false_type()); else add_pv(std::true_type());
      __syncthreads();   // the tile, and with the last one the queries, may be overwritten
    }

    const bool begins = t0 == 0, ends = t1 == tiles;
    if (begins && !ends && tid == 0) {
      PagedHeader h;
      h.parts = paged_parts(pos - it.tile + it.tiles, W, E, me);
      h.first = it.s.first;
      h.h = it.h;
      h.row0 = row0;
      h.rows = rows;
      h.pad[0] = h.pad[1] = h.pad[2] = 0;
      hdr[me] = h;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
#pragma unroll
      for (int x = 4; x > 0; x >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], x);
      const int row = 4 * ty + r;
      if (row >= rows) continue;
      const bool done = begins && ends;
      const int tok = it.s.first + (row0 + row) / dm.G, head = it.h * dm.G + (row0 + row) % dm.G;
      const size_t slot = (size_t)(begins ? 2 * me + 1 : 2 * me) * kBR + row;
      float* dst = done ? (float*)a.out + ((size_t)tok * dm.hq + head) * D : part_o + slot * D;
      const float f = !done ? 1.f : l[r] == 0.f ? 0.f : 1.f / l[r];
#pragma unroll
      for (int c = 0; c < C4; ++c) {
        float4 x;
        f2_unpack(o[r][2 * c], x.x, x.y);
        f2_unpack(o[r][2 * c + 1], x.z, x.w);
        *reinterpret_cast<float4*>(dst + 4 * tx + 32 * c) = make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
      }
      if (tx == 0) {
        if (!done)
          *reinterpret_cast<float2*>(part_ml + 2 * slot) = make_float2(m[r], l[r]);
        else if (a.lse != nullptr)
          a.lse[(size_t)head * dm.tokens + tok] = l[r] == 0.f ? -INFINITY : (m[r] + log2f(l[r])) * kLn2;
      }
    }
    pos += it.tiles - it.tile;
    if (pos < stop) paged_next<kBR, BK, kItemCost>(it, a.cu, a.kv_len, dm);
  }
}

template <int D>
cudaError_t launch(const PagedDims& dm, const PagedArgs& a, const PagedWs& l, cudaStream_t stream) {
  cudaError_t e = cudaFuncSetAttribute(paged_f32_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_early(paged_f32_kernel<D>, kWorkers, kThreads, Geo<D>::kSmem, stream, a, dm, l.hdr, l.part_o, l.part_ml);
}

}  // namespace

size_t paged_f32_ws(int d) { return paged_ws_bytes(kWorkers, kBR, d); }

cudaError_t launch_paged_f32(const PagedDims& dm, int d, const PagedArgs& a, void* ws, cudaStream_t stream, int* launches) {
  const PagedWs l = paged_ws_layout(ws, kWorkers, kBR);
  cudaError_t e = d == 128 ? launch<128>(dm, a, l, stream) : launch<64>(dm, a, l, stream);
  if (e != cudaSuccess) return e;
  ++*launches;
  return launch_paged_combine(MOBA_F32, d, l, kWorkers, kBR, a, dm, stream, launches);
}

}  // namespace moba
