// Attention of new tokens over a paged cache: the choice of the kernel, the fp32
// kernel on CUDA cores, and the combine kernel that joins the parts of an item
// (paged.cuh).
//
// For a row at position p with keys u <= p:  z_u = scale <q, k_u>,
//   m = max z, l = sum 2^(z - m), o = sum 2^(z - m) v_u / l, lse = m + log l
// in one pass over the keys with a running (m, l, o); z in units of log2(e).
// A row that sees no key gives o = 0, lse = -inf.
#include <type_traits>

#include "paged.cuh"

namespace moba {

// ---- combine ---------------------------------------------------------------
// Joins the cut items: weights 2^(m_i - m) of their parts' sums.  A unit is the
// item that worker w begins and kRows of its rows.  Short row tiles may be in
// hundreds of parts: kShare warps a row divide them.  Units of one worker go to blocks apart, and a block looks
// at the headers of all its units at once: most are empty.  (One block an item,
// its rows in turn, took 75 us to join 8 items of 74 parts and 80 us for items of
// 256 rows.)
// a prime number of blocks: the units of a worker, E apart, meet in none
constexpr int kCombineGrid = 1181, kCombineThreads = 256;

template <typename T, int D>
__global__ void __launch_bounds__(kCombineThreads) paged_combine_kernel(const PagedHeader* __restrict__ hdr, int E, int BR,
                                                                        const float* __restrict__ part_o,
                                                                        const float* __restrict__ part_ml,
                                                                        T* __restrict__ out, float* __restrict__ lse,
                                                                        PagedDims dm) {
  constexpr int C = D / 32, kWarps = kCombineThreads / 32, kShare = 4, kRows = kWarps / kShare;
  __shared__ float sm_o[kWarps][D];
  __shared__ float sm_l[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  after_previous();
  const int units = E * ((BR + kRows - 1) / kRows);
  for (int u0 = blockIdx.x; u0 < units; u0 += 32 * gridDim.x) {
    const int mine = u0 + lane * gridDim.x;
    const int parts = mine < units ? hdr[mine % E].parts : 0;
    for (uint32_t live = __ballot_sync(0xffffffffu, parts > 0); live != 0; live &= live - 1) {
      const int u = u0 + (__ffs(live) - 1) * gridDim.x, w = u % E;
      const PagedHeader h = hdr[w];
      const int r = u / E * kRows + warp / kShare;
      const bool on = r < h.rows;
      if (u / E * kRows >= h.rows) continue;   // for the whole block
      // part 0 is slot 2w + 1, part i > 0 is slot 2(w + i)
      auto slot = [&](int i) { return (size_t)(i == 0 ? 2 * w + 1 : 2 * (w + i)) * BR + r; };
      float m = -INFINITY, l = 0.f, o[C];
#pragma unroll
      for (int c = 0; c < C; ++c) o[c] = 0.f;
      if (on) {
        for (int i = lane; i < h.parts; i += 32) m = fmaxf(m, part_ml[2 * slot(i)]);
        m = warp_max(m);
        const float mb = m == -INFINITY ? 0.f : m;
#pragma unroll 8
        for (int i = warp % kShare; i < h.parts; i += kShare) {
          const size_t sl = slot(i);
          const float2 ml = *reinterpret_cast<const float2*>(part_ml + 2 * sl);
          const float wt = exp2f(ml.x - mb);
          l = fmaf(ml.y, wt, l);
          const float* src = part_o + sl * D + lane * C;
          if constexpr (C == 4) {
            const float4 x = *reinterpret_cast<const float4*>(src);
            o[0] = fmaf(x.x, wt, o[0]); o[1] = fmaf(x.y, wt, o[1]); o[2] = fmaf(x.z, wt, o[2]); o[3] = fmaf(x.w, wt, o[3]);
          } else {
            const float2 x = *reinterpret_cast<const float2*>(src);
            o[0] = fmaf(x.x, wt, o[0]); o[1] = fmaf(x.y, wt, o[1]);
          }
        }
      }
      if (lane == 0) sm_l[warp] = l;
#pragma unroll
      for (int c = 0; c < C; ++c) sm_o[warp][lane * C + c] = o[c];
      __syncthreads();
      if (warp % kShare == 0) {
#pragma unroll
        for (int i = 1; i < kShare; ++i) {
          l += sm_l[warp + i];
#pragma unroll
          for (int c = 0; c < C; ++c) o[c] += sm_o[warp + i][lane * C + c];
        }
      }
      __syncthreads();
      if (on && warp % kShare == 0) {
        const int row = h.row0 + r, tok = row / dm.G, head = h.h * dm.G + row % dm.G;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        T* dst = out + ((size_t)(h.first + tok) * dm.hq + head) * D + lane * C;
#pragma unroll
        for (int c = 0; c < C; ++c) o[c] *= inv;
        if constexpr (sizeof(T) == 4) {
          if constexpr (C == 4) *reinterpret_cast<float4*>(dst) = make_float4(o[0], o[1], o[2], o[3]);
          else *reinterpret_cast<float2*>(dst) = make_float2(o[0], o[1]);
        } else {
#pragma unroll
          for (int c = 0; c < C; c += 2) *reinterpret_cast<uint32_t*>(dst + c) = pack_bf16x2(o[c], o[c + 1]);
        }
        if (lane == 0 && lse != nullptr)
          lse[(size_t)head * dm.tokens + h.first + tok] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      }
    }
  }
}

// The same for long row tiles (in few parts): 8 lanes a row, 4 rows a warp.  (A
// warp a row spent 20 us on its own instructions for 148 items of 256 rows.)
template <typename T, int D>
__global__ void __launch_bounds__(kCombineThreads) paged_combine_rows_kernel(const PagedHeader* __restrict__ hdr, int E,
                                                                             int BR, const float* __restrict__ part_o,
                                                                             const float* __restrict__ part_ml,
                                                                             T* __restrict__ out, float* __restrict__ lse,
                                                                             PagedDims dm) {
  constexpr int V = D / 32, kRows = kCombineThreads / 8;   // groups of 4 channels a lane, rows a unit
  const int lane = threadIdx.x & 31, sub = threadIdx.x & 7;
  after_previous();
  const int units = E * (BR / kRows);
  for (int u0 = blockIdx.x; u0 < units; u0 += 32 * gridDim.x) {
    const int mine = u0 + lane * gridDim.x;
    const int parts = mine < units ? hdr[mine % E].parts : 0;
    for (uint32_t live = __ballot_sync(0xffffffffu, parts > 0); live != 0; live &= live - 1) {
      const int u = u0 + (__ffs(live) - 1) * gridDim.x, w = u % E;
      const PagedHeader h = hdr[w];
      if (u / E * kRows >= h.rows) continue;
      const int r = u / E * kRows + (threadIdx.x >> 3);
      const bool on = r < h.rows;
      // part 0 is slot 2w + 1, part i > 0 is slot 2(w + i)
      const size_t at0 = (size_t)(2 * w + 1) * BR + (on ? r : 0), step = (size_t)2 * BR;
      auto slot = [&](int i) { return i == 0 ? at0 : at0 - BR + i * step; };
      float m = -INFINITY, l = 0.f;
      for (int i = sub; i < h.parts; i += 8) m = fmaxf(m, part_ml[2 * slot(i)]);
#pragma unroll
      for (int x = 4; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
      const float mb = m == -INFINITY ? 0.f : m;
      float4 o[V];
#pragma unroll
      for (int v = 0; v < V; ++v) o[v] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int i = 0; i < h.parts; ++i) {
        const size_t sl = slot(i);
        const float2 ml = *reinterpret_cast<const float2*>(part_ml + 2 * sl);
        const float wt = exp2f(ml.x - mb);
        l = fmaf(ml.y, wt, l);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float4 x = *reinterpret_cast<const float4*>(part_o + sl * D + 32 * v + 4 * sub);
          o[v] = make_float4(fmaf(x.x, wt, o[v].x), fmaf(x.y, wt, o[v].y), fmaf(x.z, wt, o[v].z), fmaf(x.w, wt, o[v].w));
        }
      }
      if (!on) continue;
      const int row = h.row0 + r, tok = row / dm.G, head = h.h * dm.G + row - tok * dm.G;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      T* dst = out + ((size_t)(h.first + tok) * dm.hq + head) * D + 4 * sub;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if constexpr (sizeof(T) == 4)
          *reinterpret_cast<float4*>(dst + 32 * v) = make_float4(o[v].x * inv, o[v].y * inv, o[v].z * inv, o[v].w * inv);
        else
          *reinterpret_cast<uint2*>(dst + 32 * v) =
              make_uint2(pack_bf16x2(o[v].x * inv, o[v].y * inv), pack_bf16x2(o[v].z * inv, o[v].w * inv));
      }
      if (sub == 0 && lse != nullptr)
        lse[(size_t)head * dm.tokens + h.first + tok] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
  }
}

namespace {

// ---- CUDA-core kernel ----------------------------------------------------------
// A worker is a warp: R rows of a group, its lanes the channels (D / 32 each),
// 8 keys at a time straight from the pages into registers, one coalesced row a
// load.  The 8 R dot products are summed over the lanes by halving: each step
// sends half of the values, so that 62 shuffles do the work of 320 for R = 8.
// Bound: memory for one token of a few heads (32 sequences of 2.5K keys, 8 kv heads
// of 128: 0.65 GB in 123 us, 5.3 TB/s), beyond some 8 rows the FMAs and shuffles.
constexpr int kVecThreads = 256, kVecWarps = 8;
constexpr int kVecBK = 16;                        // keys a tile: the smallest page
// blocks an SM: 4 rows fit 128 registers a thread, 8 rows do not
constexpr int vec_blocks(int R) { return R == 4 ? 2 : 1; }
constexpr int vec_workers(int R) { return 148 * vec_blocks(R) * kVecWarps; }
constexpr int kVecMinTiles = 4;                   // a worker takes 64 keys at least

template <typename T, int C> struct LaneVec;      // C channels as loaded
template <> struct LaneVec<float, 4> {
  float4 v;
  MOBA_DEV void load(const float* p) { v = __ldg(reinterpret_cast<const float4*>(p)); }
  MOBA_DEV void zero() { v = make_float4(0.f, 0.f, 0.f, 0.f); }
  MOBA_DEV void widen(float* f) const { f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w; }
};
template <> struct LaneVec<float, 2> {
  float2 v;
  MOBA_DEV void load(const float* p) { v = __ldg(reinterpret_cast<const float2*>(p)); }
  MOBA_DEV void zero() { v = make_float2(0.f, 0.f); }
  MOBA_DEV void widen(float* f) const { f[0] = v.x; f[1] = v.y; }
};
// values v[0 .. N) of every lane summed over the 32 lanes: lane i ends with the
// sums of values i N / 32 .. (i + 1) N / 32 - 1, in v[0 .. N / 32)
template <int N>
MOBA_DEV void halving_sum(float* v, int lane) {
  int n = N;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    n >>= 1;
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      if (i < n) {
        const float keep = up ? v[i + n] : v[i], give = up ? v[i] : v[i + n];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
      }
    }
  }
}

template <typename T, int D, int R>
__global__ void __launch_bounds__(kVecThreads, vec_blocks(R)) paged_vec_kernel(PagedArgs a, PagedDims dm, PagedHeader* __restrict__ hdr,
                                                                   float* __restrict__ part_o,
                                                                   float* __restrict__ part_ml) {
  constexpr int C = D / 32, N = 8 * R, V = N / 32, LPR = 32 / R;   // values a lane, lanes a row
  __shared__ PagedPlan<kVecThreads> plan;
  __shared__ __align__(16) float sp[kVecWarps][N];
  __shared__ float sa[kVecWarps][R];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  after_previous();
  const int64_t W = paged_plan<R, kVecBK, 0, kVecThreads>(plan, a.cu, a.kv_len, dm);
  const int64_t E = min((int64_t)vec_workers(R), (W + kVecMinTiles - 1) / kVecMinTiles);
  const int64_t w = (int64_t)blockIdx.x * kVecWarps + warp;
  if (lane == 0) hdr[w].parts = 0;
  if (blockIdx.x == 0 && a.status != nullptr)
    for (int b = threadIdx.x; b < dm.batch; b += kVecThreads)
      if (a.kv_len[b] > ((int64_t)dm.max_pages << dm.page_shift)) atomicExch(a.status, (int)MOBA_ERR_INTERNAL);
  if (w >= E) return;
  const T* kp = (const T*)a.k_pool;
  const T* vp = (const T*)a.v_pool;
  const int myrow = lane / LPR;
  int64_t pos = w * W / E;
  const int64_t stop = (w + 1) * W / E;
  PagedItem it = paged_locate<R, kVecBK, 0, kVecThreads>(plan, pos, a.cu, a.kv_len, dm);

  while (pos < stop) {
    const int t0 = it.tile, t1 = (int)min((int64_t)it.tiles, it.tile + (stop - pos));
    const int row0 = it.rt * R, rows = min(R, it.s.n * dm.G - row0);
    const int old = it.s.len - it.s.n;
    float q[R][C], o[R][C];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      LaneVec<T, C> x;
      x.zero();
      if (r < rows) {
        const int tok = (row0 + r) / dm.G, g = (row0 + r) % dm.G;
        x.load((const T*)a.q + (int64_t)(it.s.first + tok) * dm.q_stride + (it.h * dm.G + g) * D + lane * C);
      }
      x.widen(q[r]);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        q[r][c] *= dm.scale_log2;
        o[r][c] = 0.f;
      }
    }
    // keys that the lane's row sees, and that every row of the tile sees
    const int lim = myrow < rows ? old + (row0 + myrow) / dm.G + 1 : 0;
    const int all = old + row0 / dm.G + 1;
    float m = -INFINITY, l = 0.f;

    for (int t = t0; t < t1; ++t) {
      const int u0 = t * kVecBK;
      const int pi = u0 >> dm.page_shift;
      int page = -1;
      if (u0 < it.s.len) {
        page = a.table[(int64_t)it.b * dm.max_pages + pi];
        if (page < 0 || page >= dm.num_pages) {
          // keys of a page that the pool does not have read as zeros
          page = -1;
          if (lane == 0 && a.status != nullptr) atomicExch(a.status, (int)MOBA_ERR_INTERNAL);
        }
      }
      const int64_t in_page = ((int64_t)it.h << dm.page_shift) + (u0 & ((1 << dm.page_shift) - 1));
      const T* kt = kp + page * dm.k_page_stride + in_page * D + lane * C;
      const T* vt = vp + page * dm.v_page_stride + in_page * D + lane * C;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int u = u0 + 8 * half;
        if (u >= it.s.len && u > u0) break;
        LaneVec<T, C> kr[8], vr[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          kr[i].zero();
          vr[i].zero();
          if (page >= 0 && u + i < it.s.len) {
            kr[i].load(kt + (8 * half + i) * D);
            vr[i].load(vt + (8 * half + i) * D);
          }
        }
        float z[N];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float k[C];
          kr[i].widen(k);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            float d = q[r][0] * k[0];
#pragma unroll
            for (int c = 1; c < C; ++c) d = fmaf(q[r][c], k[c], d);
            z[r * 8 + i] = d;
          }
        }
        halving_sum<N>(z, lane);
        // the lane's V values: row myrow, keys (lane % LPR) V ..
        float top = -INFINITY;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (u + (lane % LPR) * V + v >= lim) z[v] = -INFINITY;
          top = fmaxf(top, z[v]);
        }
#pragma unroll
        for (int x = LPR / 2; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        const float mn = fmaxf(m, top), base = mn == -INFINITY ? 0.f : mn;
        const float f = exp2f(m - base);
        l *= f;
        m = mn;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float p = exp2f(z[v] - base);
          l += p;
          sp[warp][lane * V + v] = p;
        }
        const bool moved = __any_sync(0xffffffffu, f != 1.f);
        if (lane % LPR == 0) sa[warp][myrow] = f;
        __syncwarp();
        if (moved) {
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float fr = sa[warp][r];
#pragma unroll
            for (int c = 0; c < C; ++c) o[r][c] *= fr;
          }
        }
        float v[8][C];
#pragma unroll
        for (int i = 0; i < 8; ++i) vr[i].widen(v[i]);
        if (u + 8 <= all) {
#pragma unroll
          for (int r = 0; r < R; ++r) {
            float p[8];
            *reinterpret_cast<float4*>(p) = *reinterpret_cast<const float4*>(&sp[warp][r * 8]);
            *reinterpret_cast<float4*>(p + 4) = *reinterpret_cast<const float4*>(&sp[warp][r * 8 + 4]);
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
              for (int c = 0; c < C; ++c) o[r][c] = fmaf(p[i], v[i][c], o[r][c]);
          }
        } else {
          // some row does not see all of these keys: an infinity or NaN there
          // must not meet its zero probability
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const int lr = r < rows ? old + (row0 + r) / dm.G + 1 : 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float p = sp[warp][r * 8 + i];
              if (u + i < lr) {
#pragma unroll
                for (int c = 0; c < C; ++c) o[r][c] = fmaf(p, v[i][c], o[r][c]);
              }
            }
          }
        }
        __syncwarp();
      }
    }
#pragma unroll
    for (int x = LPR / 2; x > 0; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);

    const bool begins = t0 == 0, ends = t1 == it.tiles;
    const size_t slot = (size_t)(begins ? 2 * w + 1 : 2 * w) * R;
    if (!(begins && ends) && begins && lane == 0) {
      PagedHeader h;
      h.parts = paged_parts(pos + it.tiles, W, E, w);
      h.first = it.s.first;
      h.h = it.h;
      h.row0 = row0;
      h.rows = rows;
      h.pad[0] = h.pad[1] = h.pad[2] = 0;
      hdr[w] = h;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float lr = __shfl_sync(0xffffffffu, l, r * LPR), mr = __shfl_sync(0xffffffffu, m, r * LPR);
      if (r >= rows) continue;
      if (begins && ends) {
        const int tok = it.s.first + (row0 + r) / dm.G, head = it.h * dm.G + (row0 + r) % dm.G;
        const float inv = lr == 0.f ? 0.f : 1.f / lr;
        T* dst = (T*)a.out + ((size_t)tok * dm.hq + head) * D + lane * C;
#pragma unroll
        for (int c = 0; c < C; ++c) dst[c] = from_f32<T>(o[r][c] * inv);
        if (lane == 0 && a.lse != nullptr)
          a.lse[(size_t)head * dm.tokens + tok] = lr == 0.f ? -INFINITY : (mr + log2f(lr)) * kLn2;
      } else {
#pragma unroll
        for (int c = 0; c < C; ++c) part_o[(slot + r) * D + lane * C + c] = o[r][c];
        if (lane == 0) {
          part_ml[2 * (slot + r)] = mr;
          part_ml[2 * (slot + r) + 1] = lr;
        }
      }
    }
    pos += t1 - t0;
    if (pos < stop) paged_next<R, kVecBK, 0>(it, a.cu, a.kv_len, dm);
  }
}

template <typename T, int D, int R>
cudaError_t launch_vec(const PagedDims& dm, const PagedArgs& a, void* ws, cudaStream_t stream, int* launches) {
  constexpr int kE = vec_workers(R);
  const PagedWs l = paged_ws_layout(ws, kE, R);
  cudaError_t e = launch_early(paged_vec_kernel<T, D, R>, kE / kVecWarps, kVecThreads, 0, stream, a, dm, l.hdr, l.part_o,
                               l.part_ml);
  if (e != cudaSuccess) return e;
  ++*launches;
  return launch_paged_combine(sizeof(T) == 2 ? MOBA_BF16 : MOBA_F32, D, l, kE, R, a, dm, stream, launches);
}

// 4 rows a warp leave room for twice the warps, 8 read a key for twice the rows.
// head_dim 128, 32K keys: 1 row of 16 heads takes 105 us with 4 rows a warp and
// 128 with 8, 4 rows of 8 heads 75 and 80; 32 sequences of 2.5K keys with 8 rows
// 166 and 157, with 32 rows 449 and 369.  head_dim 64 with 8 rows: 99 and 123.
template <typename T, int D>
cudaError_t launch_vec_rows(const PagedDims& dm, const PagedArgs& a, void* ws, cudaStream_t stream, int* launches) {
  if constexpr (D == 128)
    if ((int64_t)dm.tokens * dm.G > 4 * (int64_t)dm.batch) return launch_vec<T, D, 8>(dm, a, ws, stream, launches);
  return launch_vec<T, D, 4>(dm, a, ws, stream, launches);
}

}  // namespace

cudaError_t launch_paged_combine(int dtype, int d, const PagedWs& l, int E, int BR, const PagedArgs& a, const PagedDims& dm,
                                 cudaStream_t stream, int* launches) {
  auto go = [&](auto* out, auto dim) {
    using T = typename std::remove_pointer<decltype(out)>::type;
    auto* kernel = BR > 16 ? paged_combine_rows_kernel<T, decltype(dim)::value> : paged_combine_kernel<T, decltype(dim)::value>;
    return launch_early(kernel, kCombineGrid, kCombineThreads, 0, stream, (const PagedHeader*)l.hdr, E, BR,
                        (const float*)l.part_o, (const float*)l.part_ml, out, a.lse, dm);
  };
  cudaError_t e;
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  if (dtype == MOBA_BF16) {
    e = d == 128 ? go((__nv_bfloat16*)a.out, D128()) : go((__nv_bfloat16*)a.out, D64());
  } else {
    e = d == 128 ? go((float*)a.out, D128()) : go((float*)a.out, D64());
  }
  if (e == cudaSuccess) ++*launches;
  return e;
}

size_t paged_decode_ws(int d);
cudaError_t launch_paged_decode(const PagedDims& dm, int d, const PagedArgs& a, void* ws, cudaStream_t stream, int* launches);
size_t paged_tc_ws(int d);
size_t paged_f32_ws(int d);
cudaError_t launch_paged_f32(const PagedDims& dm, int d, const PagedArgs& a, void* ws, cudaStream_t stream, int* launches);
cudaError_t launch_paged_tc(const PagedDims& dm, int d, const PagedArgs& a, void* ws, cudaStream_t stream, int* launches);

size_t paged_attn_ws(int dtype, int d) {
  if (dtype == MOBA_BF16) {
    const size_t a = paged_tc_ws(d), b = paged_decode_ws(d);
    return a > b ? a : b;
  }
  size_t most = paged_f32_ws(d);
  for (int R : {4, 8}) {
    const size_t b = paged_ws_bytes(vec_workers(R), R, d);
    most = most > b ? most : b;
  }
  return most;
}

cudaError_t launch_paged_attn(const PagedDims& dm, int dtype, int d, const PagedArgs& a, void* ws, cudaStream_t stream,
                              int* launches) {
  if (dm.tokens == 0) return cudaSuccess;
  // Rows of a kv head's group a sequence, on average: with few, reading the cache
  // bounds the call, with many the products.  32 / 8 heads of 128, one sequence of
  // 32K keys / 32 of 2.5K on average, bf16: 32 rows take 39 / 94 us on the decode
  // kernel and 53 / 99 on tcgen05, 64 rows 59 / 141 and 57 / 102.  fp32: 32 rows
  // 209 / 369 us by warps and 243 / 559 by tiles, 64 rows 387 / 650 and 246 / 566.
  // Both sides are sequences alike.  The average also takes in sequences without new
  // tokens and rows of padding, and one kernel gets a mixed step whole: 63 tokens at 8K
  // keys beside a chunk of 400 at 32K take 1199 us, as two calls 332 and 262; beside one
  // at 8K 431, 324 and 84; 512 tokens at 2K beside 3500 at 4K 1043, 652 and 177.
  const bool few = (int64_t)dm.tokens * dm.G <= 32 * (int64_t)dm.batch;
  if (dtype == MOBA_BF16)
    return few ? launch_paged_decode(dm, d, a, ws, stream, launches) : launch_paged_tc(dm, d, a, ws, stream, launches);
  if (!few) return launch_paged_f32(dm, d, a, ws, stream, launches);
  return d == 128 ? launch_vec_rows<float, 128>(dm, a, ws, stream, launches)
                  : launch_vec_rows<float, 64>(dm, a, ws, stream, launches);
}

}  // namespace moba
