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
#include "launch.h"

namespace moba {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kSms = 148;

// 8 consecutive elements as loaded
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
  uint4 u;
  MOBA_DEV void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  MOBA_DEV void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = u; }
  MOBA_DEV void zero() { u = make_uint4(0, 0, 0, 0); }
  MOBA_DEV void widen(float* f) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  MOBA_DEV void round(const float* f) {
    u = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                   pack_bf16x2(f[6], f[7]));
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
  MOBA_DEV void widen(float* f) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  MOBA_DEV void round(const float* f) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
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

// cos and sin of the warp's token into cs[rot/2]
MOBA_DEV void warp_angles(float2* cs, int pos, const double* __restrict__ inv_freq, int half, int lane) {
  constexpr double kInv2Pi = 0.15915494309189533576888;
  for (int i = lane; i < half; i += 32) {
    double turns = (double)pos * inv_freq[i] * kInv2Pi;
    turns -= rint(turns);
    float s, c;
    sincospif((float)(2.0 * turns), &s, &c);
    cs[i] = make_float2(c, s);
  }
  __syncwarp();
}

// rotate the lane's 16 elements y = (a[8], b[8]) by its 8 pairs' angles (way =
// 1), or back (way = -1)
MOBA_DEV void turn(float* y, const float2* cs, bool interleaved, float way) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float2 t = cs[e];
    const float s = way * t.y;
    const int ia = interleaved ? 2 * e : e, ib = interleaved ? 2 * e + 1 : 8 + e;
    const float a = y[ia], b = y[ib];
    y[ia] = a * t.x - b * s;
    y[ib] = b * t.x + a * s;
  }
}
MOBA_DEV void turn_lane(float* y, const float2* cs, bool interleaved, float way) {
  if (interleaved) turn(y, cs, true, way); else turn(y, cs, false, way);
}

template <int LPH>
MOBA_DEV float head_sum(float v) {
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// 16 weights of the lane's two vectors, in fp32
template <typename T>
MOBA_DEV void load_weights(float* w, const void* p, int wf32, int va, int vb) {
  if (wf32) {
    Raw8<float> r;
    r.load((const float*)p + 8 * va); r.widen(w);
    r.load((const float*)p + 8 * vb); r.widen(w + 8);
  } else {
    Raw8<__nv_bfloat16> r;
    r.load((const __nv_bfloat16*)p + 8 * va); r.widen(w);
    r.load((const __nv_bfloat16*)p + 8 * vb); r.widen(w + 8);
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

// One warp = one token (or every split-th head group of it, where there are
// few tokens).
template <typename T, int D, bool kAppend>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(RopeArgs a) {
  constexpr int LPH = D / 16, HPW = 32 / LPH;
  __shared__ float2 cs_all[kWarps][D / 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t gw = (int64_t)blockIdx.x * kWarps + warp;
  const int t = (int)(gw / a.split), s = (int)(gw % a.split);
  if (t >= a.tokens) return;
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
  auto load = [&](int g, Raw8<T>& x0, Raw8<T>& x1) {
    int kind, head;
    x0.zero();
    x1.zero();
    if (g >= groups || !locate(g, kind, head)) return;
    const T* p = kind == 0 ? (const T*)a.q + t * a.q_stride
                           : kind == 1 ? (const T*)a.k + t * a.k_stride : (const T*)a.v + t * a.v_stride;
    x0.load(p + head * D + 8 * va);
    x1.load(p + head * D + 8 * vb);
  };
  Raw8<T> x0, x1;
  load(s, x0, x1);

  int pos, slot = 0;
  int64_t page = -1;
  if (kAppend) {
    // a row behind the last sequence is left as it was
    if (t >= a.cu[a.batch]) return;
    const int b = seq_of_token(a.cu, a.batch, t, lane);
    pos = a.kv_len[b] - (a.cu[b + 1] - t);
    const int pi = pos >> a.page_shift;
    slot = pos & ((1 << a.page_shift) - 1);
    if (pos >= 0 && pi < a.max_pages) page = a.table[(int64_t)b * a.max_pages + pi];
    if (page < 0 || page >= a.num_pages) {
      // no page for this token: nothing is written, the status word says so
      page = -1;
      if (lane == 0 && a.status != nullptr) atomicExch(a.status, (int)MOBA_ERR_INTERNAL);
    }
  } else {
    pos = a.positions != nullptr ? a.positions[t] : 0;
  }
  const bool rotated = j < a.rot / 16;
  const float2* cs = cs_all[warp] + 8 * j;
  if (a.rot > 0) warp_angles(cs_all[warp], pos, a.inv_freq, a.rot / 2, lane);

  float w[16];
  int have = -1;
  for (int g = s; g < groups; g += a.split) {
    Raw8<T> n0, n1;
    load(g + a.split, n0, n1);
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
      const void* wp = kind == 0 ? a.q_weight : a.k_weight;
      float y[16];
      x0.widen(y);
      x1.widen(y + 8);
      if (wp != nullptr) {
        if (have != kind) {
          load_weights<T>(w, wp, a.weight_f32, va, vb);
          have = kind;
        }
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) ss = fmaf(y[e], y[e], ss);
        const float r = rsqrtf(head_sum<LPH>(ss) * (1.f / D) + a.eps);
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] *= r * w[e];
      }
      if (rotated) turn_lane(y, cs, a.interleaved != 0, 1.f);
      x0.round(y);
      x1.round(y + 8);
    }
    if (put) {
      x0.store(dst + 8 * va);
      x1.store(dst + 8 * vb);
    }
    x0 = n0;
    x1 = n1;
  }
}

// Backward.  Blocks [0, nbq) take the queries, the rest the keys, so that a
// lane has one weight gradient (16 channels) to sum; a block's sums go to its
// row of `part`, in a fixed order, and the reduction kernel adds the rows.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) norm_rope_bwd_kernel(RopeArgs a, const void* dq_out, const void* dk_out,
                                                                 float* part, int nbq) {
  constexpr int LPH = D / 16, HPW = 32 / LPH;
  __shared__ float2 cs_all[kWarps][D / 2];
  __shared__ float sums[kWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
  const float2* cs = cs_all[warp] + 8 * j;
  float w[16], dw[16];
  load_weights<T>(w, isq ? a.q_weight : a.k_weight, a.weight_f32, va, vb);
#pragma unroll
  for (int e = 0; e < 16; ++e) dw[e] = 0.f;

  for (int t = bi * kWarps + warp; t < a.tokens; t += nb * kWarps) {
    Raw8<T> x0, x1, d0, d1;
    auto load = [&](int g, Raw8<T>& p0, Raw8<T>& p1, Raw8<T>& r0, Raw8<T>& r1) {
      const int head = g * HPW + hl;
      if (head < heads) {
        const T* p = x + t * xs + head * D;
        const T* r = dy + ((int64_t)t * heads + head) * D;
        p0.load(p + 8 * va); p1.load(p + 8 * vb);
        r0.load(r + 8 * va); r1.load(r + 8 * vb);
      } else {
        p0.zero(); p1.zero(); r0.zero(); r1.zero();
      }
    };
    load(0, x0, x1, d0, d1);
    __syncwarp();
    if (a.rot > 0) warp_angles(cs_all[warp], a.positions[t], a.inv_freq, a.rot / 2, lane);
    for (int g = 0; g < groups; ++g) {
      Raw8<T> n0, n1, m0, m1;
      load(g + 1, n0, n1, m0, m1);
      float xv[16], z[16];
      x0.widen(xv); x1.widen(xv + 8);
      d0.widen(z); d1.widen(z + 8);
      if (rotated) turn_lane(z, cs, a.interleaved != 0, -1.f);
      float ss = 0.f, dot = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        ss = fmaf(xv[e], xv[e], ss);
        dot = fmaf(xv[e], z[e] * w[e], dot);
      }
      ss = head_sum<LPH>(ss);
      dot = head_sum<LPH>(dot);
      const float r = rsqrtf(ss * (1.f / D) + a.eps);
      const float c = r * r * r * dot * (1.f / D);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float rz = r * z[e];
        dw[e] = fmaf(rz, xv[e], dw[e]);
        z[e] = rz * w[e] - c * xv[e];
      }
      const int head = g * HPW + hl;
      if (head < heads) {
        T* p = dx + ((int64_t)t * heads + head) * D;
        d0.round(z); d1.round(z + 8);
        d0.store(p + 8 * va); d1.store(p + 8 * vb);
      }
      x0 = n0; x1 = n1; d0 = m0; d1 = m1;
    }
  }
  // heads of the warp, then the warps, in order
#pragma unroll
  for (int e = 0; e < 16; ++e) {
#pragma unroll
    for (int o = LPH; o < 32; o <<= 1) dw[e] += __shfl_xor_sync(0xffffffffu, dw[e], o);
  }
  if (hl == 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      sums[warp][8 * va + e] = dw[e];
      sums[warp][8 * vb + e] = dw[8 + e];
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

// dw of the queries (block 0) and of the keys (block 1): the blocks' rows of
// `part` added by 1024 / D threads a channel, in a fixed order
template <int D>
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const float* __restrict__ part, int nbq, int nbk,
                                                            void* dqw, void* dkw, int weight_f32) {
  constexpr int kParts = 1024 / D;
  __shared__ float sums[kParts][D];
  const int c = threadIdx.x % D, p = threadIdx.x / D;
  const int lo = blockIdx.x == 0 ? 0 : nbq, hi = blockIdx.x == 0 ? nbq : nbq + nbk;
  float v = 0.f;
#pragma unroll 8
  for (int i = lo + p; i < hi; i += kParts) v += part[(int64_t)i * D + c];
  sums[p][c] = v;
  __syncthreads();
  if (p == 0) {
#pragma unroll
    for (int i = 1; i < kParts; ++i) v += sums[i][c];
    void* dst = blockIdx.x == 0 ? dqw : dkw;
    if (weight_f32) ((float*)dst)[c] = v; else ((__nv_bfloat16*)dst)[c] = __float2bfloat16_rn(v);
  }
}

template <typename T, int D>
cudaError_t launch_fwd(RopeArgs a, bool append, cudaStream_t stream, int* launches) {
  constexpr int HPW = 512 / D;
  const int groups = (a.q == nullptr ? 0 : (a.hq + HPW - 1) / HPW) + (append ? 2 : 1) * ((a.hkv + HPW - 1) / HPW);
  a.split = 1;
  while (a.split * 2 <= groups && (int64_t)a.tokens * a.split < 32 * kSms) a.split *= 2;
  const int64_t blocks = ((int64_t)a.tokens * a.split + kWarps - 1) / kWarps;
  if (blocks == 0) return cudaSuccess;
  if (append)
    norm_rope_kernel<T, D, true><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
  else
    norm_rope_kernel<T, D, false><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
  ++*launches;
  return cudaGetLastError();
}

// Blocks of the backward: at most kBwdBlocks, shared between queries and keys
// by their heads.
constexpr int kBwdBlocks = 4 * kSms;
void bwd_blocks(int tokens, int hq, int hkv, int& nbq, int& nbk) {
  const int most = (tokens + kWarps - 1) / kWarps;
  nbk = kBwdBlocks * hkv / (hq + hkv);
  nbk = nbk < 1 ? 1 : nbk;
  nbq = kBwdBlocks - nbk;
  nbq = nbq < most ? nbq : most;
  nbk = nbk < most ? nbk : most;
}

template <typename T, int D>
cudaError_t launch_bwd(const RopeArgs& a, const void* dq_out, const void* dk_out, void* dqw, void* dkw, float* part,
                       cudaStream_t stream, int* launches) {
  int nbq, nbk;
  bwd_blocks(a.tokens, a.hq, a.hkv, nbq, nbk);
  if (nbq + nbk > 0) {
    norm_rope_bwd_kernel<T, D><<<nbq + nbk, kThreads, 0, stream>>>(a, dq_out, dk_out, part, nbq);
    ++*launches;
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  norm_rope_dw_kernel<D><<<2, 1024, 0, stream>>>(part, nbq, nbk, dqw, dkw, a.weight_f32);
  ++*launches;
  return cudaGetLastError();
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
