// Per-head norm of queries and keys with the position rotation in one pass
// (forward and backward), and the same pass writing keys and values into a
// paged cache.
//
//   y = x r w,  r = (mean(x^2) + eps)^(-1/2)          one head x of d numbers
//   (a, b) -> (a c - b s, b c + a s)                  pair i of the rotated part,
//   c, s = cos, sin of position * f_i; (a, b) = (y[i], y[i + rot/2]), or
//   (y[2i], y[2i + 1]) where pairs are interleaved
// Backward, with z the gradient turned back (the transposed rotation), g = z w:
//   dx = r g - x r^3 <x, g> / d,     dw = sum over tokens and heads of z x r
//
// Bound: memory.  Every element is read once and written once, so a head stays
// in the registers of d/16 lanes (16 elements a lane, two 8-element vectors
// that hold both halves of the lane's 8 pairs), a warp takes 512/d heads at a
// time, and the one reduction is a few shuffles.  The angle is position * f_i
// in 64 bits, reduced to a turn before it is rounded: at position 10^7 a 32-bit
// product is off by half a radian.  A warp computes its token's rot/2 sines and
// cosines once, in shared memory, for all of the token's heads.
// Sums are fp32; results are rounded once, on the store.
//
// Measured (bf16, 32768 tokens, 32 / 8 heads of 128; the copy benchmark moves 6.56
// TB/s): forward 0.67 GB in 112 to 114 us (5.9 TB/s), backward 1.01 GB in 178 us (5.65),
// weight gradients' rows 6 us more.  fp32, 12000 tokens of the same heads: forward
// 90 us (5.5 TB/s), backward with the rows 129 (5.7).  The forward waits for loads
// and issues at 70% of its slots; the backward's 128 registers hold it to 16 warps an
// SM, and less registers spill.  Append of 16K tokens with the norm: 0.40 GB in 75 us (5.3 TB/s).
#include "launch.h"
#include "sm100.cuh"

namespace moba {

namespace {

using sm100::f2_add;
using sm100::f2_fma;
using sm100::f2_pack;
using sm100::f2_sub;
using sm100::f2_unpack;
MOBA_DEV uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
MOBA_DEV float f2_sum(uint64_t a) {
  float x, y;
  f2_unpack(a, x, y);
  return x + y;
}

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kSms = 148;

// 8 consecutive elements as loaded; widened to 4 packed fp32 pairs (the arithmetic
// below runs on pairs: half the instructions, which bound these kernels before the
// memory did)
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
  uint4 u;
  MOBA_DEV void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  MOBA_DEV void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = u; }
  MOBA_DEV void zero() { u = make_uint4(0, 0, 0, 0); }
  MOBA_DEV void widen(uint64_t* f) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  MOBA_DEV void round(const uint64_t* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x, y;
      f2_unpack(f[i], x, y);
      w[i] = pack_bf16x2(x, y);
    }
    u = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Raw8<float> {
  float4 a, b;
  MOBA_DEV void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  MOBA_DEV void store(float* p) const {
    *reinterpret_cast<float4*>(p) = a;
    *reinterpret_cast<float4*>(p + 4) = b;
  }
  MOBA_DEV void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  MOBA_DEV void widen(uint64_t* f) const {
    f[0] = f2_pack(a.x, a.y); f[1] = f2_pack(a.z, a.w);
    f[2] = f2_pack(b.x, b.y); f[3] = f2_pack(b.z, b.w);
  }
  MOBA_DEV void round(const uint64_t* f) {
    f2_unpack(f[0], a.x, a.y); f2_unpack(f[1], a.z, a.w);
    f2_unpack(f[2], b.x, b.y); f2_unpack(f[3], b.z, b.w);
  }
};

// Lane j of a head holds the vectors (va, vb): rotated lanes (j < rot/16) the
// two halves of pairs 8j .. 8j+7, the others two vectors of the rest.
template <int D>
MOBA_DEV void lane_vectors(int j, int rot, bool interleaved, int& va, int& vb) {
  if (interleaved) {
    va = 2 * j;
    vb = va + 1;
  } else if (j < rot / 16) {
    va = j;
    vb = j + rot / 16;
  } else {
    va = rot / 8 + 2 * (j - rot / 16);
    vb = va + 1;
  }
}

// cos and sin of the warp's token, for pair 8 j + e of lane j at
// [e / 4][cos, sin][j][e % 4]: a lane's reads are 16 bytes, without bank conflicts
// (as (cos, sin) pair after pair they took 70% of the shared memory's time)
template <int LPH> struct Angles { float4 v[2][2][LPH]; };
template <int LPH>
MOBA_DEV void warp_angles(Angles<LPH>& cs, int pos, const double (&freq)[LPH / 4], int half, int lane) {
  constexpr double kInv2Pi = 0.15915494309189533576888;
  float* f = reinterpret_cast<float*>(&cs);
  __syncwarp();   // the last token's angles are read
#pragma unroll
  for (int n = 0; n < LPH / 4; ++n) {
    const int i = lane + 32 * n;
    if (i >= half) continue;
    double turns = (double)pos * freq[n] * kInv2Pi;
    turns -= rint(turns);
    float s, c;
    sincospif((float)(2.0 * turns), &s, &c);
    const int at = ((((i >> 2) & 1) * 2 * LPH + (i >> 3)) << 2) + (i & 3);
    f[at] = c;
    f[at + 4 * LPH] = s;
  }
  __syncwarp();
}

// turn the lane's 8 packed pairs of elements (vectors a = y[0..4), b = y[4..8))
// by its angles, or back
template <int LPH, bool kBack>
MOBA_DEV void turn(uint64_t* y, const Angles<LPH>& cs, int j, bool interleaved) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float4 c = cs.v[h][0][j], s = cs.v[h][1][j];
    if (interleaved) {
      // (a, b) of pair 4 h + i is the packed y[4 h + i]
      const float cv[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float a, b;
        f2_unpack(y[4 * h + i], a, b);
        const float t = kBack ? -sv[i] : sv[i];
        y[4 * h + i] = f2_pack(a * cv[i] - b * t, b * cv[i] + a * t);
      }
    } else {
      const uint64_t c2[2] = {f2_pack(c.x, c.y), f2_pack(c.z, c.w)}, s2[2] = {f2_pack(s.x, s.y), f2_pack(s.z, s.w)};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint64_t a = y[2 * h + i], b = y[4 + 2 * h + i];
        if (kBack) {
          y[2 * h + i] = f2_fma(b, s2[i], f2_mul(a, c2[i]));
          y[4 + 2 * h + i] = f2_sub(f2_mul(b, c2[i]), f2_mul(a, s2[i]));
        } else {
          y[2 * h + i] = f2_sub(f2_mul(a, c2[i]), f2_mul(b, s2[i]));
          y[4 + 2 * h + i] = f2_fma(a, s2[i], f2_mul(b, c2[i]));
        }
      }
    }
  }
}

// the lane's frequencies: of pairs lane and lane + 32
template <int N>
MOBA_DEV void load_freq(double (&f)[N], const double* __restrict__ inv_freq, int half, int lane) {
#pragma unroll
  for (int n = 0; n < N; ++n) f[n] = lane + 32 * n < half ? inv_freq[lane + 32 * n] : 0.0;
}

template <int LPH>
MOBA_DEV float head_sum(float v) {
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// 16 weights of the lane's two vectors, in packed fp32
MOBA_DEV void load_weights(uint64_t* w, const void* p, int wf32, int va, int vb) {
  if (wf32) {
    Raw8<float> r;
    r.load((const float*)p + 8 * va); r.widen(w);
    r.load((const float*)p + 8 * vb); r.widen(w + 4);
  } else {
    Raw8<__nv_bfloat16> r;
    r.load((const __nv_bfloat16*)p + 8 * va); r.widen(w);
    r.load((const __nv_bfloat16*)p + 8 * vb); r.widen(w + 4);
  }
}

// sequence of new token t: the first b with cu[b + 1] > t, found 32 ways at a time
MOBA_DEV int seq_of_token(const int32_t* __restrict__ cu, int batch, int t, int lane) {
  int lo = 0, n = batch;
  while (n > 32) {
    const int step = (n + 31) >> 5;
    const int at = (lane + 1) * step;
    const int c = __popc(__ballot_sync(0xffffffffu, at <= n && cu[lo + (at <= n ? at : n)] <= t));
    lo += c * step;
    n = min(step, n - c * step);
  }
  const int c = __popc(__ballot_sync(0xffffffffu, lane < n && cu[lo + (lane < n ? lane : 0) + 1] <= t));
  return min(lo + c, batch - 1);
}

// Blocks an SM: the registers of a thread against the warps that hide each
// other's waits.  bf16, 32768 tokens: 4 blocks of 64 registers, one head group
// loaded ahead of the one in work, take 112 us; 3 blocks of 80 with one ahead
// 119, with two 125, with three 121; 2 blocks with two to four ahead 140 to 149.
template <typename T> constexpr int kFwdBlocks = sizeof(T) == 2 ? 4 : 3;

// A warp takes tokens in a stride (or every split-th head group of them, where
// there are few tokens) as one run of head groups, loads running ahead across
// tokens.
template <typename T, int D, bool kAppend>
__global__ void __launch_bounds__(kThreads, kFwdBlocks<T>) norm_rope_kernel(RopeArgs a) {
  constexpr int LPH = D / 16, HPW = 32 / LPH, kRing = 2;   // a head group in work, one on its way
  __shared__ Angles<LPH> cs_all[kWarps];
  __shared__ ulonglong2 sm_w[2][4][LPH];   // weights of queries and keys as lane j reads them
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gw = blockIdx.x * kWarps + warp;
  const int s = gw % a.split, t0 = gw / a.split, step = gridDim.x * kWarps / a.split;
  // rows behind the last sequence are left as they were
  const int tokens = kAppend ? min(a.tokens, a.cu[a.batch]) : a.tokens;
  const int j = lane % LPH, hl = lane / LPH;
  int va, vb;
  lane_vectors<D>(j, a.rot, a.interleaved != 0, va, vb);
  const int gq = a.q == nullptr ? 0 : (a.hq + HPW - 1) / HPW, gk = (a.hkv + HPW - 1) / HPW;
  const int groups = gq + (kAppend ? 2 : 1) * gk;

  auto locate = [&](int g, int& kind, int& head) {
    kind = g < gq ? 0 : g < gq + gk ? 1 : 2;
    head = (kind == 0 ? g : kind == 1 ? g - gq : g - gq - gk) * HPW + hl;
    return head < (kind == 0 ? a.hq : a.hkv);
  };
  int lt = t0, lg = s;   // the next group to load
  Raw8<T> ring[kRing][2];
  auto load = [&](Raw8<T> (&x)[2]) {
    int kind, head;
    x[0].zero();
    x[1].zero();
    if (lt < tokens && locate(lg, kind, head)) {
      const T* p = kind == 0 ? (const T*)a.q + lt * a.q_stride
                             : kind == 1 ? (const T*)a.k + lt * a.k_stride : (const T*)a.v + lt * a.v_stride;
      x[0].load(p + head * D + 8 * va);
      x[1].load(p + head * D + 8 * vb);
    }
    lg += a.split;
    if (lg >= groups) {
      lg = s;
      lt = step < tokens - lt ? lt + step : tokens;
    }
  };
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) load(ring[i]);

  if (warp < 2 && lane < LPH) {
    const void* wp = warp == 0 ? a.q_weight : a.k_weight;
    if (wp != nullptr) {
      uint64_t w[8];
      load_weights(w, wp, a.weight_f32, va, vb);
#pragma unroll
      for (int e = 0; e < 4; ++e) sm_w[warp][e][j] = make_ulonglong2(w[2 * e], w[2 * e + 1]);
    }
  }
  __syncthreads();
  if (t0 >= tokens) return;
  double freq[LPH / 4];
  load_freq(freq, a.inv_freq, a.rot / 2, lane);
  const bool rotated = j < a.rot / 16;
  const Angles<LPH>& cs = cs_all[warp];
  int slot = 0;
  int64_t page = -1;
  int next_pos = !kAppend && a.rot > 0 ? a.positions[t0] : 0;
  // position, page and angles of a token
  auto begin = [&](int t) {
    int pos;
    if (kAppend) {
      const int b = seq_of_token(a.cu, a.batch, t, lane);
      pos = a.kv_len[b] - (a.cu[b + 1] - t);
      const int pi = pos >> a.page_shift;
      slot = pos & ((1 << a.page_shift) - 1);
      page = -1;
      if (pos >= 0 && pi < a.max_pages) page = a.table[(int64_t)b * a.max_pages + pi];
      if (page < 0 || page >= a.num_pages) {
        // no page for this token: nothing is written, the status word says so
        page = -1;
        if (lane == 0 && a.status != nullptr) atomicExch(a.status, (int)MOBA_ERR_INTERNAL);
      }
    } else {
      pos = next_pos;
      if (a.rot > 0 && step < tokens - t) next_pos = a.positions[t + step];
    }
    if (a.rot > 0) warp_angles<LPH>(cs_all[warp], pos, freq, a.rot / 2, lane);
  };

  int t = t0, g = s;
  while (t < tokens) {
#pragma unroll
    for (int i = 0; i < kRing; ++i) {
      if (t >= tokens) break;
      load(ring[(i + kRing - 1) % kRing]);
      Raw8<T>&x0 = ring[i][0], &x1 = ring[i][1];
      if (g == s) begin(t);
      int kind, head;
      const bool live = locate(g, kind, head);
      T* dst;
      if (kind == 0) {
        dst = (T*)a.q_out + ((int64_t)t * a.hq + head) * D;
      } else if (!kAppend) {
        dst = (T*)a.k_out + ((int64_t)t * a.hkv + head) * D;
      } else {
        dst = (kind == 1 ? (T*)a.k_out + page * a.k_page_stride : (T*)a.v_out + page * a.v_page_stride) +
              (((int64_t)head << a.page_shift) + slot) * D;
      }
      const bool put = live && (kind == 0 || !kAppend || page >= 0);
      if (!kAppend || kind < 2) {
        uint64_t y[8];
        x0.widen(y);
        x1.widen(y + 4);
        if ((kind == 0 ? a.q_weight : a.k_weight) != nullptr) {
          uint64_t s0 = f2_mul(y[0], y[0]), s1 = f2_mul(y[1], y[1]);
#pragma unroll
          for (int e = 2; e < 8; e += 2) {
            s0 = f2_fma(y[e], y[e], s0);
            s1 = f2_fma(y[e + 1], y[e + 1], s1);
          }
          const float r = rsqrtf(head_sum<LPH>(f2_sum(f2_add(s0, s1))) * (1.f / D) + a.eps);
          const uint64_t r2 = f2_pack(r, r);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const ulonglong2 w = sm_w[kind][e][j];
            y[2 * e] = f2_mul(y[2 * e], f2_mul(r2, w.x));
            y[2 * e + 1] = f2_mul(y[2 * e + 1], f2_mul(r2, w.y));
          }
        }
        if (rotated) turn<LPH, false>(y, cs, j, a.interleaved != 0);
        x0.round(y);
        x1.round(y + 4);
      }
      if (put) {
        x0.store(dst + 8 * va);
        x1.store(dst + 8 * vb);
      }
      g += a.split;
      if (g >= groups) {
        g = s;
        t = step < tokens - t ? t + step : tokens;
      }
    }
  }
}

template <typename T> constexpr int kBwdPerSm = sizeof(T) == 2 ? 2 : 1;   // blocks an SM, for 128 and 255 registers

// Backward.  Blocks [0, nbq) take the queries, the rest the keys, so that a
// lane has one weight gradient (16 channels) to sum; a block's sums go to its
// row of `part`, in a fixed order, and the reduction kernel adds the rows.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, kBwdPerSm<T>) norm_rope_bwd_kernel(RopeArgs a, const void* dq_out, const void* dk_out,
                                                                 float* part, int nbq) {
  constexpr int LPH = D / 16, HPW = 32 / LPH;
  __shared__ Angles<LPH> cs_all[kWarps];
  __shared__ float sums[kWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;\n" ::);   // the reduction kernel may be launched
  const bool isq = (int)blockIdx.x < nbq;
  const int nb = isq ? nbq : gridDim.x - nbq, bi = isq ? blockIdx.x : blockIdx.x - nbq;
  const int heads = isq ? a.hq : a.hkv, groups = (heads + HPW - 1) / HPW;
  const T* x = (const T*)(isq ? a.q : a.k);
  const int64_t xs = isq ? a.q_stride : a.k_stride;
  const T* dy = (const T*)(isq ? dq_out : dk_out);
  T* dx = (T*)(isq ? a.q_out : a.k_out);
  const int j = lane % LPH, hl = lane / LPH;
  int va, vb;
  lane_vectors<D>(j, a.rot, a.interleaved != 0, va, vb);
  const bool rotated = j < a.rot / 16;
  const Angles<LPH>& cs = cs_all[warp];
  uint64_t w[8], dw[8];
  load_weights(w, isq ? a.q_weight : a.k_weight, a.weight_f32, va, vb);
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[e] = 0;

  double freq[LPH / 4];
  load_freq(freq, a.inv_freq, a.rot / 2, lane);
  const int step = nb * kWarps;
  int lt = bi * kWarps + warp, lg = 0;   // the next group to load: one ahead, across tokens
  int t = lt, g = 0;
  auto load = [&](Raw8<T>& p0, Raw8<T>& p1, Raw8<T>& r0, Raw8<T>& r1) {
    const int head = lg * HPW + hl;
    if (lt < a.tokens && head < heads) {
      const T* p = x + lt * xs + head * D;
      const T* r = dy + ((int64_t)lt * heads + head) * D;
      p0.load(p + 8 * va); p1.load(p + 8 * vb);
      r0.load(r + 8 * va); r1.load(r + 8 * vb);
    } else {
      p0.zero(); p1.zero(); r0.zero(); r1.zero();
    }
    if (++lg >= groups) {
      lg = 0;
      lt = lt < a.tokens && step < a.tokens - lt ? lt + step : a.tokens;
    }
  };
  // registers of a group in work and of the next in turn: a copy between them would wait for the loads
  Raw8<T> ring[2][4];
  load(ring[0][0], ring[0][1], ring[0][2], ring[0][3]);
  int next_pos = t < a.tokens && a.rot > 0 ? a.positions[t] : 0;
  while (t < a.tokens) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (t >= a.tokens) break;
      load(ring[1 - i][0], ring[1 - i][1], ring[1 - i][2], ring[1 - i][3]);
      Raw8<T>&x0 = ring[i][0], &x1 = ring[i][1], &d0 = ring[i][2], &d1 = ring[i][3];
      if (g == 0 && a.rot > 0) {
        const int pos = next_pos;
        if (step < a.tokens - t) next_pos = a.positions[t + step];
        warp_angles<LPH>(cs_all[warp], pos, freq, a.rot / 2, lane);
      }
      uint64_t xv[8], z[8];
      x0.widen(xv); x1.widen(xv + 4);
      d0.widen(z); d1.widen(z + 4);
      if (rotated) turn<LPH, true>(z, cs, j, a.interleaved != 0);
      uint64_t s0 = 0, s1 = 0, u0 = 0, u1 = 0;
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        s0 = f2_fma(xv[e], xv[e], s0);
        s1 = f2_fma(xv[e + 1], xv[e + 1], s1);
        u0 = f2_fma(xv[e], f2_mul(z[e], w[e]), u0);
        u1 = f2_fma(xv[e + 1], f2_mul(z[e + 1], w[e + 1]), u1);
      }
      const float ss = head_sum<LPH>(f2_sum(f2_add(s0, s1))), dot = head_sum<LPH>(f2_sum(f2_add(u0, u1)));
      // lanes without a head hold zeros, whose r would be infinite for eps = 0 and reach dw as 0 times an infinity
      const int head = g * HPW + hl;
      const float r = head < heads ? rsqrtf(ss * (1.f / D) + a.eps) : 0.f;
      const float c = -(r * dot * (1.f / D)) * r * r;   // r^3 alone leaves fp32 outside 3e-13 .. 6e12
      const uint64_t r2 = f2_pack(r, r), c2 = f2_pack(c, c);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint64_t rz = f2_mul(r2, z[e]);
        dw[e] = f2_fma(rz, xv[e], dw[e]);
        z[e] = f2_fma(c2, xv[e], f2_mul(rz, w[e]));
      }
      if (head < heads) {
        T* p = dx + ((int64_t)t * heads + head) * D;
        d0.round(z); d1.round(z + 4);
        d0.store(p + 8 * va); d1.store(p + 8 * vb);
      }
      if (++g >= groups) {
        g = 0;
        t = step < a.tokens - t ? t + step : a.tokens;
      }
    }
  }
  // heads of the warp, then the warps, in order
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float x, y;
    f2_unpack(dw[e], x, y);
#pragma unroll
    for (int o = LPH; o < 32; o <<= 1) {
      x += __shfl_xor_sync(0xffffffffu, x, o);
      y += __shfl_xor_sync(0xffffffffu, y, o);
    }
    if (hl == 0) {
      const int at = 8 * (e < 4 ? va : vb) + 2 * (e & 3);
      sums[warp][at] = x;
      sums[warp][at + 1] = y;
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < D; c += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) v += sums[i][c];
    part[(int64_t)blockIdx.x * D + c] = v;
  }
}

// dw of the queries (the first D / 32 blocks) and of the keys: 32 channels a block,
// whose 32 warps add the rows of `part`, in a fixed order.  (One block for all
// channels took 10 us for 592 rows.)
template <int D>
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const float* __restrict__ part, int nbq, int nbk,
                                                            void* dqw, void* dkw, int weight_f32) {
  __shared__ float sums[32][33];
  const int lane = threadIdx.x & 31, p = threadIdx.x >> 5, slab = blockIdx.x % (D / 32), c = slab * 32 + lane;
  const bool isq = blockIdx.x < D / 32;
  after_previous();
  const int lo = isq ? 0 : nbq, hi = isq ? nbq : nbq + nbk;
  float v = 0.f;
#pragma unroll 8
  for (int i = lo + p; i < hi; i += 32) v += part[(int64_t)i * D + c];
  sums[p][lane] = v;
  __syncthreads();
  v = warp_sum(sums[lane][p]);   // channel p of the block
  if (lane == 0) {
    void* dst = isq ? dqw : dkw;
    const int at = slab * 32 + p;
    if (weight_f32) ((float*)dst)[at] = v; else ((__nv_bfloat16*)dst)[at] = __float2bfloat16_rn(v);
  }
}

template <typename T, int D>
cudaError_t launch_fwd(RopeArgs a, bool append, cudaStream_t stream, int* launches) {
  constexpr int HPW = 512 / D;
  const int groups = (a.q == nullptr ? 0 : (a.hq + HPW - 1) / HPW) + (append ? 2 : 1) * ((a.hkv + HPW - 1) / HPW);
  // a token's groups over several warps until two rounds of them fill the card: 6000 tokens of 32 / 8 heads take 28.0,
  // 25.2, 26.8, 33.3 us with units up to 32, 64, 128, 192 an SM, 2000 tokens 10.5 to 11.1, 20000 all 70.5
  a.split = 1;
  while (a.split * 2 <= groups && (int64_t)a.tokens * a.split < 64 * kSms && a.split < kWarps) a.split *= 2;
  const int64_t need = ((int64_t)a.tokens * a.split + kWarps - 1) / kWarps;
  const int64_t blocks = need < kFwdBlocks<T> * kSms ? need : kFwdBlocks<T> * kSms;
  if (blocks == 0) return cudaSuccess;
  // (launched early like the attention's kernels it gained nothing: 75 us for chunks became 78)
  if (append)
    norm_rope_kernel<T, D, true><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
  else
    norm_rope_kernel<T, D, false><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
  ++*launches;
  return cudaGetLastError();
}

// Blocks of the backward: at most kBwdBlocks, shared between queries and keys by
// their time: a token's angles cost about as much as 3/4 of a head group.
constexpr int kBwdBlocks = 2 * kSms;
template <typename T, int D>
void bwd_blocks(int tokens, int hq, int hkv, int& nbq, int& nbk) {
  constexpr int HPW = 512 / D;
  const int all = kBwdPerSm<T> * kSms, cq = 4 * ((hq + HPW - 1) / HPW) + 3, ck = 4 * ((hkv + HPW - 1) / HPW) + 3;
  const int most = (tokens + kWarps - 1) / kWarps;
  nbk = (all * ck + (cq + ck) / 2) / (cq + ck);
  nbk = nbk < 1 ? 1 : nbk;
  nbq = all - nbk;
  nbq = nbq < most ? nbq : most;
  nbk = nbk < most ? nbk : most;
}

template <typename T, int D>
cudaError_t launch_bwd(const RopeArgs& a, const void* dq_out, const void* dk_out, void* dqw, void* dkw, float* part,
                       cudaStream_t stream, int* launches) {
  int nbq, nbk;
  bwd_blocks<T, D>(a.tokens, a.hq, a.hkv, nbq, nbk);
  if (nbq + nbk > 0) {
    norm_rope_bwd_kernel<T, D><<<nbq + nbk, kThreads, 0, stream>>>(a, dq_out, dk_out, part, nbq);
    ++*launches;
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  // D / 32 blocks for the queries and as many for the keys
  const cudaError_t e = launch_early(norm_rope_dw_kernel<D>, 2 * (D / 32), 1024, 0, stream, part, nbq, nbk, dqw, dkw, a.weight_f32);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace

cudaError_t launch_norm_rope(const RopeArgs& a, int dtype, int d, bool append, cudaStream_t stream, int* launches) {
  if (dtype == MOBA_BF16)
    return d == 128 ? launch_fwd<__nv_bfloat16, 128>(a, append, stream, launches)
                    : launch_fwd<__nv_bfloat16, 64>(a, append, stream, launches);
  return d == 128 ? launch_fwd<float, 128>(a, append, stream, launches)
                  : launch_fwd<float, 64>(a, append, stream, launches);
}

size_t norm_rope_bwd_ws(int d) { return (size_t)kBwdBlocks * d * sizeof(float); }

cudaError_t launch_norm_rope_bwd(const RopeArgs& a, int dtype, int d, const void* dq_out, const void* dk_out, void* dqw,
                                 void* dkw, float* part, cudaStream_t stream, int* launches) {
  if (dtype == MOBA_BF16)
    return d == 128 ? launch_bwd<__nv_bfloat16, 128>(a, dq_out, dk_out, dqw, dkw, part, stream, launches)
                    : launch_bwd<__nv_bfloat16, 64>(a, dq_out, dk_out, dqw, dkw, part, stream, launches);
  return d == 128 ? launch_bwd<float, 128>(a, dq_out, dk_out, dqw, dkw, part, stream, launches)
                  : launch_bwd<float, 64>(a, dq_out, dk_out, dqw, dkw, part, stream, launches);
}

}  // namespace moba
