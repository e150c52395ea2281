// ssm_qk.cu -- normalisation of queries and keys over each head and their rotation by position, in one
// pass, and the gradients of that.
//
//   s = 1 / sqrt(mean(v^2) + eps), n = v s w           (n = v without the norm)
//   (n_p, n_q) -> scale (n_p cos - n_q sin, n_q cos + n_p sin), angle = position * inv_freq[j], for the
//   rot / 2 pairs (j, j + rot/2), or (2 j, 2 j + 1) interleaved; the other elements pass.
// Backward, with e the gradient turned back by the same angle:
//   dw = sum e v s,  dv = s (e w - v s^2 mean(e w v))   (dv = e without the norm)
//
// Both are streams: every element read once and written once, all sums within a row in fp32.
//
// Head elements innermost (state_last): a row is cut into units of 16 elements (two 16-byte runs) such
// that both members of a pair are in one unit -- elements [8u, 8u+8) and [rot/2 + 8u, ...) of the
// half layout, 16 consecutive ones of the interleaved layout and of the unrotated rest -- so the rotation needs
// no exchange between lanes. G lanes hold a row (G = units rounded up to a power of two) and add
// its squares by shuffles. A group of lanes takes several heads of one token, queries and keys alike, and
// computes the token's cosines and sines once for them. Head sizes or alignments that do not fit
// take the same kernel with units of one pair and a warp per row.
//
// Time innermost (time_last): a thread owns consecutive steps (8 where rows are whole 16-byte runs, else 1)
// of a few pairs; the squares meet in shared memory, and with more than one pair a thread the elements are
// read a second time, from L1.
//
// Angles. In 32 bits position * inv_freq loses the angle of a far position (at 10^6 the spacing is 1/16 of
// a radian), so the product and its reduction to a fraction of a turn are in 64 bits; what is left
// goes through the hardware sine (absolute error 2^-21) for bf16, sincospif for fp32 inputs.
#include "ssm_internal.h"
#include "ssm_vec.cuh"

namespace ssm {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThr = 256;                 // threads per CTA
constexpr int kBwdCtas = 148 * 3;         // CTAs of a backward that keeps sums (three per SM)
constexpr double kInvTwoPi = 0.15915494309189533577;

__device__ __forceinline__ float ld1(const void *p, int bf16, int64_t i) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]) : static_cast<const float *>(p)[i];
}
__device__ __forceinline__ void st1(void *p, int bf16, int64_t i, float v) {
  if (bf16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<float *>(p)[i] = v;
}
__device__ __forceinline__ void ld8any(const void *p, int bf16, int64_t i, float *v) {
  if (bf16) {
    Raw8<__nv_bfloat16> r;
    ld8(static_cast<const __nv_bfloat16 *>(p) + i, r);
    unpack8(r, v);
  } else {
    Raw8<float> r;
    ld8(static_cast<const float *>(p) + i, r);
    unpack8(r, v);
  }
}
__device__ __forceinline__ void st8any(void *p, int bf16, int64_t i, const float *v) {
  if (bf16) st8(static_cast<__nv_bfloat16 *>(p) + i, v);
  else st8(static_cast<float *>(p) + i, v);
}

__device__ __forceinline__ double position(const QkParams &p, int64_t b, int64_t t) {
  if (!p.pos) return (double)(p.pos0 + t);
  return p.pos_i64 ? (double)static_cast<const int64_t *>(p.pos)[b * p.L + t]
                   : (double)static_cast<const int32_t *>(p.pos)[b * p.L + t];
}
__device__ __forceinline__ double frequency(const QkParams &p, int j) {
  return p.freq_f64 ? static_cast<const double *>(p.inv_freq)[j] : (double)static_cast<const float *>(p.inv_freq)[j];
}
// Cosine and sine of pos * f, times the scale.
template <bool PRECISE>
__device__ __forceinline__ void turn(double pos, double f, float scale, float &c, float &s) {
  const double t = pos * f * kInvTwoPi;
  const float frac = (float)(t - rint(t));  // a fraction of a turn in [-1/2, 1/2]
  if (PRECISE) {
    sincospif(2.f * frac, &s, &c);
  } else {
    const float x = frac * 6.283185307179586f;
    c = __cosf(x);
    s = __sinf(x);
  }
  c *= scale;
  s *= scale;
}
template <bool PRECISE> __device__ __forceinline__ float inv_rms(const QkParams &p, float sum) {
  const float ms = fmaf(sum, p.inv_D, p.eps);
  return PRECISE ? 1.f / sqrtf(ms) : rsqrtf(ms);
}

// Unit u of a row, V elements at o1 and V at o2, in pairs when it is one of the `ur` rotated units:
// (o1 + e, o2 + e) of the half layout; (2 e, 2 e + 1) of the 2 V at o1 of the interleaved one.
template <int V> struct Unit {
  int o1, o2;
  bool on, rot;
};
template <int V> __device__ __forceinline__ Unit<V> unit_of(const QkParams &p, int u) {
  const int ur = p.rot / (2 * V), n = (p.D - p.rot + 2 * V - 1) / (2 * V);
  Unit<V> r;
  r.rot = u < ur;
  r.on = u < ur + n;
  const bool half = r.rot && !p.interleaved;
  r.o1 = half ? u * V : 2 * V * u;  // the rest follows the rotated units at 2 V u too
  r.o2 = half ? p.rot / 2 + u * V : r.o1 + V;
  return r;
}

// Turn the 2 V elements of a rotated unit by its V angles (sign -1: back).
template <int V>
__device__ __forceinline__ void turn_unit(const QkParams &p, float *v, const float *c, const float *s, float sign) {
  if (p.interleaved) {
#pragma unroll
    for (int e = 0; e < V; e++) {
      const float a = v[2 * e], b = v[2 * e + 1], sn = sign * s[e];
      v[2 * e] = a * c[e] - b * sn;
      v[2 * e + 1] = b * c[e] + a * sn;
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; e++) {
      const float a = v[e], b = v[V + e], sn = sign * s[e];
      v[e] = a * c[e] - b * sn;
      v[V + e] = b * c[e] + a * sn;
    }
  }
}

template <int V>
__device__ __forceinline__ void load_unit(const void *p, int bf16, int64_t at, const Unit<V> &u, int D, float *v) {
  if constexpr (V == 8) {
    if (u.on) {
      ld8any(p, bf16, at + u.o1, v);
      ld8any(p, bf16, at + u.o2, v + 8);
    } else {
#pragma unroll
      for (int e = 0; e < 16; e++) v[e] = 0.f;
    }
  } else {
    v[0] = u.on ? ld1(p, bf16, at + u.o1) : 0.f;
    v[1] = u.on && u.o2 < D ? ld1(p, bf16, at + u.o2) : 0.f;
  }
}
template <int V>
__device__ __forceinline__ void store_unit(void *p, int bf16, int64_t at, const Unit<V> &u, int D, const float *v) {
  if (!u.on) return;
  if constexpr (V == 8) {
    st8any(p, bf16, at + u.o1, v);
    st8any(p, bf16, at + u.o2, v + 8);
  } else {
    st1(p, bf16, at + u.o1, v[0]);
    if (u.o2 < D) st1(p, bf16, at + u.o2, v[1]);
  }
}
// The weights of a unit (1 without weights).
template <int V>
__device__ __forceinline__ void load_weights(const float *w, const Unit<V> &u, int D, float *v) {
#pragma unroll
  for (int e = 0; e < 2 * V; e++) v[e] = 1.f;
  if (!w || !u.on) return;
  if constexpr (V == 8) {
    Raw8<float> r;
    ld8(w + u.o1, r);
    unpack8(r, v);
    ld8(w + u.o2, r);
    unpack8(r, v + 8);
  } else {
    v[0] = w[u.o1];
    if (u.o2 < D) v[1] = w[u.o2];
  }
}

// n / d and the remainder, in 32 bits where both fit.
__device__ __forceinline__ void divide(int64_t n, int64_t d, int64_t &q, int64_t &r) {
  if ((n | d) <= 0x7fffffffLL) {
    q = (uint32_t)n / (uint32_t)d;
    r = (uint32_t)n % (uint32_t)d;
  } else {
    q = n / d;
    r = n % d;
  }
}

}  // namespace

// ---- head elements innermost -------------------------------------------------------------------

// A group of G lanes takes HP rows (heads; queries first, then keys) of one token. NU units a lane.
template <typename T, int V, int NU, int HP>
__global__ void __launch_bounds__(kThr) qk_fwd_kernel(const __grid_constant__ QkParams p, int G, int64_t chunks) {
  constexpr bool PRECISE = sizeof(T) == 4;
  const int lane = threadIdx.x & 31, sub = lane % G;
  const int64_t item = ((int64_t)blockIdx.x * kThr + threadIdx.x) / G;
  int64_t token, chunk, b, t;
  divide(item, chunks, token, chunk);
  divide(token, p.L, b, t);
  const bool live = b < p.Bt;  // dead groups follow along for the shuffles
  Unit<V> u[NU];
#pragma unroll
  for (int n = 0; n < NU; n++) {
    u[n] = unit_of<V>(p, sub + n * G);
    u[n].on = u[n].on && live;
  }
  const int h0 = (int)chunk * HP;
  float v[HP][NU][2 * V];
#pragma unroll
  for (int k = 0; k < HP; k++) {
    const int h = h0 + k, side = h >= p.H[0];
    const bool on = h < p.H[0] + p.H[1];
    const QkTensor &in = p.in[side];
    const int64_t at = b * in.sb + t * in.sr + (h - (side ? p.H[0] : 0)) * in.sh;
#pragma unroll
    for (int n = 0; n < NU; n++) {
      Unit<V> un = u[n];
      un.on = un.on && on;
      load_unit<V>(in.p, PRECISE ? 0 : 1, at, un, p.D, v[k][n]);
    }
  }
  float c[NU][V], s[NU][V];
  const double pos = live && p.rot ? position(p, b, t) : 0.0;
#pragma unroll
  for (int n = 0; n < NU; n++)
    if (u[n].on && u[n].rot) {
#pragma unroll
      for (int e = 0; e < V; e++) turn<PRECISE>(pos, frequency(p, (sub + n * G) * V + e), p.rot_scale, c[n][e], s[n][e]);
    }
#pragma unroll
  for (int k = 0; k < HP; k++) {
    const int h = h0 + k, side = h >= p.H[0];
    const bool on = h < p.H[0] + p.H[1];
    if (p.norm) {
      float sum = 0.f;
#pragma unroll
      for (int n = 0; n < NU; n++)
#pragma unroll
        for (int e = 0; e < 2 * V; e++) sum = fmaf(v[k][n][e], v[k][n][e], sum);
      for (int off = G / 2; off >= 1; off >>= 1) sum += __shfl_xor_sync(kFull, sum, off);
      const float sc = inv_rms<PRECISE>(p, sum);
#pragma unroll
      for (int n = 0; n < NU; n++) {
        float w[2 * V];
        load_weights<V>(p.w[side], u[n], p.D, w);
#pragma unroll
        for (int e = 0; e < 2 * V; e++) v[k][n][e] *= sc * w[e];
      }
    }
    const QkTensor &out = p.out[side];
    const int64_t at = b * out.sb + t * out.sr + (h - (side ? p.H[0] : 0)) * out.sh;
#pragma unroll
    for (int n = 0; n < NU; n++) {
      if (u[n].rot) turn_unit<V>(p, v[k][n], c[n], s[n], 1.f);
      Unit<V> un = u[n];
      un.on = un.on && on;
      store_unit<V>(out.p, out.bf16, at, un, p.D, v[k][n]);
    }
  }
}

// Groups of lanes walk the rows of one side (blocks [0, nb0) the queries, the others the keys) with a stride
// of the side's groups, HP heads of a token at a time, and keep their share of dw in registers.
template <typename T, int V, int NU, int HP>
__global__ void __launch_bounds__(kThr) qk_bwd_kernel(const __grid_constant__ QkParams p, int G, int nb0) {
  constexpr bool PRECISE = sizeof(T) == 4;
  extern __shared__ float sdw[];  // (groups, D) with dw
  const int side = (int)blockIdx.x >= nb0;
  const int64_t block = side ? blockIdx.x - nb0 : blockIdx.x, blocks = side ? gridDim.x - nb0 : nb0;
  const int lane = threadIdx.x & 31, sub = lane % G, per_cta = kThr / G;
  const int64_t chunks = (p.H[side] + HP - 1) / HP, items = p.Bt * p.L * chunks;
  const QkTensor in = p.in[side], dout = p.dout[side], out = p.out[side];
  Unit<V> u[NU];
  float w[NU][2 * V], dw[NU][2 * V];
#pragma unroll
  for (int n = 0; n < NU; n++) {
    u[n] = unit_of<V>(p, sub + n * G);
    if (p.norm) load_weights<V>(p.w[side], u[n], p.D, w[n]);
#pragma unroll
    for (int e = 0; e < 2 * V; e++) dw[n][e] = 0.f;
  }
  const int64_t stride = blocks * per_cta;
  // the trip count is the block's, so that every lane of a warp is there for the shuffles
  for (int64_t i0 = block * per_cta; i0 < items; i0 += stride) {
    const int64_t item = i0 + threadIdx.x / G;
    const bool live = item < items;
    int64_t token, chunk, b, t;
    divide(live ? item : 0, chunks, token, chunk);
    divide(token, p.L, b, t);
    float v[HP][NU][2 * V], g[HP][NU][2 * V];
#pragma unroll
    for (int k = 0; k < HP; k++) {
      const int64_t h = chunk * HP + k;
#pragma unroll
      for (int n = 0; n < NU; n++) {
        Unit<V> un = u[n];
        un.on = un.on && live && h < p.H[side];
        load_unit<V>(dout.p, dout.bf16, b * dout.sb + t * dout.sr + h * dout.sh, un, p.D, g[k][n]);
        if (p.norm) load_unit<V>(in.p, PRECISE ? 0 : 1, b * in.sb + t * in.sr + h * in.sh, un, p.D, v[k][n]);
      }
    }
    const double pos = p.rot ? position(p, b, t) : 0.0;
#pragma unroll
    for (int n = 0; n < NU; n++)
      if (u[n].on && u[n].rot) {
        float c[V], s[V];
#pragma unroll
        for (int e = 0; e < V; e++) turn<PRECISE>(pos, frequency(p, (sub + n * G) * V + e), p.rot_scale, c[e], s[e]);
#pragma unroll
        for (int k = 0; k < HP; k++) turn_unit<V>(p, g[k][n], c, s, -1.f);
      }
#pragma unroll
    for (int k = 0; k < HP; k++) {
      const int64_t h = chunk * HP + k;
      if (p.norm) {
        float sum = 0.f, dot = 0.f;
#pragma unroll
        for (int n = 0; n < NU; n++)
#pragma unroll
          for (int e = 0; e < 2 * V; e++) {
            sum = fmaf(v[k][n][e], v[k][n][e], sum);
            dot = fmaf(g[k][n][e] * w[n][e], v[k][n][e], dot);
          }
        for (int off = G / 2; off >= 1; off >>= 1) {
          sum += __shfl_xor_sync(kFull, sum, off);
          dot += __shfl_xor_sync(kFull, dot, off);
        }
        const float sc = inv_rms<PRECISE>(p, sum);
        const float back = sc * sc * dot * p.inv_D;
#pragma unroll
        for (int n = 0; n < NU; n++)
#pragma unroll
          for (int e = 0; e < 2 * V; e++) {
            dw[n][e] = fmaf(g[k][n][e] * sc, v[k][n][e], dw[n][e]);
            g[k][n][e] = sc * (g[k][n][e] * w[n][e] - v[k][n][e] * back);
          }
      }
      if (out.p) {
#pragma unroll
        for (int n = 0; n < NU; n++) {
          Unit<V> un = u[n];
          un.on = un.on && live && h < p.H[side];
          store_unit<V>(out.p, out.bf16, b * out.sb + t * out.sr + h * out.sh, un, p.D, g[k][n]);
        }
      }
    }
  }
  if (!p.dw[side]) return;
  // the block's share of dw: the groups' in their order
#pragma unroll
  for (int n = 0; n < NU; n++)
    if (u[n].on) {
      float *row = sdw + (threadIdx.x / G) * p.D;
#pragma unroll
      for (int e = 0; e < V; e++) {
        row[u[n].o1 + e] = dw[n][e];
        if (V == 8 || u[n].o2 < p.D) row[u[n].o2 + e] = dw[n][V + e];
      }
    }
  __syncthreads();
  for (int j = threadIdx.x; j < p.D; j += kThr) {
    float s = 0.f;
    for (int r = 0; r < per_cta; r++) s += sdw[r * p.D + j];
    p.part[(int64_t)blockIdx.x * p.D + j] = s;
  }
}

// ---- time innermost ----------------------------------------------------------------------------

// TX threads over time, TV steps each, TY = kThr / TX over the pairs of a head, NS pairs a thread.
// A pair unit is unit_of<1>: elements o1 and o2 (or o1 alone at an odd end).
template <typename T, int TV> struct TimeLoad {
  static __device__ __forceinline__ void get(const void *p, int bf16, int64_t i, int n, float *v) {
    if constexpr (TV == 8) {
      if (n == 8) {
        ld8any(p, bf16, i, v);
        return;
      }
    }
#pragma unroll
    for (int e = 0; e < TV; e++) v[e] = e < n ? ld1(p, bf16, i + e) : 0.f;
  }
  static __device__ __forceinline__ void put(void *p, int bf16, int64_t i, int n, const float *v) {
    if constexpr (TV == 8) {
      if (n == 8) {
        st8any(p, bf16, i, v);
        return;
      }
    }
#pragma unroll
    for (int e = 0; e < TV; e++)
      if (e < n) st1(p, bf16, i + e, v[e]);
  }
};

// A tile: (batch, head, kThr / TY * TV steps). Forward: one per CTA. Backward: the CTAs of a side walk
// its tiles and keep dw in registers.
template <typename T, int TV, int NS, bool BWD>
__global__ void __launch_bounds__(kThr) qk_time_kernel(const __grid_constant__ QkParams p, int TX, int nb0, int64_t tiles0, int64_t tiles1) {
  constexpr bool PRECISE = sizeof(T) == 4;
  using M = TimeLoad<T, TV>;
  extern __shared__ float sh[];  // sums over the pairs: (TY, TX * TV), twice for the backward
  const int TY = kThr / TX, tx = threadIdx.x % TX, ty = threadIdx.x / TX;
  const int side = BWD ? (int)blockIdx.x >= nb0 : 0;
  const int64_t span = (int64_t)TX * TV, per_row = (p.L + span - 1) / span;
  const int64_t tiles = BWD ? (side ? tiles1 : tiles0) : tiles0 + tiles1;
  const int64_t first = BWD && side ? blockIdx.x - nb0 : blockIdx.x;
  const int64_t stride = !BWD ? gridDim.x : side ? gridDim.x - nb0 : nb0;
  const int n_units = p.rot / 2 + (p.D - p.rot + 1) / 2;
  float dwa[NS], dwb[NS];
#pragma unroll
  for (int n = 0; n < NS; n++) dwa[n] = dwb[n] = 0.f;
  for (int64_t tile = first; tile < tiles; tile += stride) {
    const int sd = BWD ? side : tile >= tiles0;
    const QkTensor &in = p.in[sd], &out = p.out[sd];
    int64_t bh, tt, b, h;
    divide(!BWD && sd ? tile - tiles0 : tile, per_row, bh, tt);
    divide(bh, p.H[sd], b, h);
    const int64_t t0 = tt * span + (int64_t)tx * TV;
    const int m = (int)(p.L - t0 < 0 ? 0 : p.L - t0 < TV ? p.L - t0 : TV);  // live steps of this thread
    const int64_t at = b * in.sb + h * in.sh + t0;
    const int64_t dat = BWD ? b * p.dout[sd].sb + h * p.dout[sd].sh + t0 : 0;
    const int64_t oat = b * out.sb + h * out.sh + t0;
    float a[TV], c[TV], ga[TV], gc[TV];  // the elements of a pair, and their gradients
    float sum[TV], dot[TV];
#pragma unroll
    for (int e = 0; e < TV; e++) sum[e] = dot[e] = 0.f;
    // the elements of pair unit u, its gradients turned back
    auto fetch = [&](const Unit<1> &u, int unit) {
      const bool two = u.o2 < p.D;
      if (!BWD || p.norm) {
        M::get(in.p, PRECISE ? 0 : 1, at + u.o1 * in.sr, m, a);
        M::get(in.p, PRECISE ? 0 : 1, at + u.o2 * in.sr, two ? m : 0, c);
      }
      if (BWD) {
        const QkTensor &dt = p.dout[sd];
        M::get(dt.p, dt.bf16, dat + u.o1 * dt.sr, m, ga);
        M::get(dt.p, dt.bf16, dat + u.o2 * dt.sr, two ? m : 0, gc);
        if (u.rot) {
          const double f = frequency(p, unit);
#pragma unroll
          for (int e = 0; e < TV; e++)
            if (e < m) {
              float cs, sn;
              turn<PRECISE>(position(p, b, t0 + e), f, p.rot_scale, cs, sn);
              const float x = ga[e], y = gc[e];
              ga[e] = x * cs + y * sn;
              gc[e] = y * cs - x * sn;
            }
        }
      }
    };
    auto weight = [&](int o) { return p.w[sd] ? p.w[sd][o] : 1.f; };
    if (p.norm) {
#pragma unroll
      for (int n = 0; n < NS; n++) {
        const int unit = ty + n * TY;
        if (unit < n_units) {
          const Unit<1> u = unit_of<1>(p, unit);
          fetch(u, unit);
          const float wa = BWD ? weight(u.o1) : 0.f, wc = BWD && u.o2 < p.D ? weight(u.o2) : 0.f;
#pragma unroll
          for (int e = 0; e < TV; e++) {
            sum[e] = fmaf(a[e], a[e], fmaf(c[e], c[e], sum[e]));
            if (BWD) dot[e] = fmaf(ga[e] * wa, a[e], fmaf(gc[e] * wc, c[e], dot[e]));
          }
        }
      }
      // over the threads that share a step, in their order
      __syncthreads();  // the tile before has been read
#pragma unroll
      for (int e = 0; e < TV; e++) {
        sh[(ty * TX + tx) * TV + e] = sum[e];
        if (BWD) sh[kThr * TV + (ty * TX + tx) * TV + e] = dot[e];
      }
      __syncthreads();
#pragma unroll
      for (int e = 0; e < TV; e++) {
        float s = 0.f, q = 0.f;
        for (int y = 0; y < TY; y++) {
          s += sh[(y * TX + tx) * TV + e];
          if (BWD) q += sh[kThr * TV + (y * TX + tx) * TV + e];
        }
        sum[e] = inv_rms<PRECISE>(p, s);
        dot[e] = sum[e] * sum[e] * q * p.inv_D;
      }
    }
#pragma unroll
    for (int n = 0; n < NS; n++) {
      const int unit = ty + n * TY;
      if (unit < n_units) {
        const Unit<1> u = unit_of<1>(p, unit);
        const bool two = u.o2 < p.D;
        if (NS > 1 || !p.norm) fetch(u, unit);  // with one pair it is still here
        const float wa = p.norm ? weight(u.o1) : 1.f, wc = p.norm && two ? weight(u.o2) : 1.f;
        if (BWD) {
          if (p.norm) {
#pragma unroll
            for (int e = 0; e < TV; e++) {
              dwa[n] = fmaf(ga[e] * sum[e], a[e], dwa[n]);
              dwb[n] = fmaf(gc[e] * sum[e], c[e], dwb[n]);
              ga[e] = sum[e] * (ga[e] * wa - a[e] * dot[e]);
              gc[e] = sum[e] * (gc[e] * wc - c[e] * dot[e]);
            }
          }
          if (out.p) {
            M::put(out.p, out.bf16, oat + u.o1 * out.sr, m, ga);
            if (two) M::put(out.p, out.bf16, oat + u.o2 * out.sr, m, gc);
          }
        } else {
          const double f = u.rot ? frequency(p, unit) : 0.0;
#pragma unroll
          for (int e = 0; e < TV; e++) {
            if (p.norm) a[e] *= sum[e] * wa, c[e] *= sum[e] * wc;
            if (u.rot && e < m) {
              float cs, sn;
              turn<PRECISE>(position(p, b, t0 + e), f, p.rot_scale, cs, sn);
              const float x = a[e], y = c[e];
              a[e] = x * cs - y * sn;
              c[e] = y * cs + x * sn;
            }
          }
          M::put(out.p, out.bf16, oat + u.o1 * out.sr, m, a);
          if (two) M::put(out.p, out.bf16, oat + u.o2 * out.sr, m, c);
        }
      }
    }
  }
  if (!BWD || !p.dw[side]) return;
  // the block's share of dw: over the TX threads that share a pair, in their order
#pragma unroll
  for (int n = 0; n < NS; n++) {
    __syncthreads();
    sh[2 * threadIdx.x] = dwa[n];
    sh[2 * threadIdx.x + 1] = dwb[n];
    __syncthreads();
    const int unit = ty + n * TY;
    if (tx == 0 && unit < n_units) {
      const Unit<1> u = unit_of<1>(p, unit);
      float x = 0.f, y = 0.f;
      for (int k = 0; k < TX; k++) {
        x += sh[2 * (ty * TX + k)];
        y += sh[2 * (ty * TX + k) + 1];
      }
      p.part[(int64_t)blockIdx.x * p.D + u.o1] = x;
      if (u.o2 < p.D) p.part[(int64_t)blockIdx.x * p.D + u.o2] = y;
    }
  }
}

// dw of both sides from the blocks' shares, in a fixed order: a CTA takes 32 elements of one side,
// its 8 rows every eighth share each.
__global__ void __launch_bounds__(256) qk_dw_kernel(const __grid_constant__ QkParams p, int nb0, int nb) {
  __shared__ float red[8][32];
  const int side = blockIdx.y, x = threadIdx.x & 31, y = threadIdx.x >> 5;
  if (!p.dw[side]) return;
  const int j = blockIdx.x * 32 + x, lo = side ? nb0 : 0, hi = side ? nb : nb0;
  float s = 0.f;
  if (j < p.D)
    for (int k = lo + y; k < hi; k += 8) s += p.part[(int64_t)k * p.D + j];
  red[y][x] = s;
  __syncthreads();
  if (y || j >= p.D) return;
  for (int k = 1; k < 8; k++) s += red[k][x];
  p.dw[side][j] = s;
}

// ---- launchers ---------------------------------------------------------------------------------

namespace {

int pow2_at_least(int n) {
  int g = 1;
  while (g < n) g *= 2;
  return g;
}

// Lanes that hold a row with units of 2 V elements, at most a warp.
int lanes_per_row(const QkParams &p, int V) {
  const int units = p.rot / (2 * V) + (p.D - p.rot + 2 * V - 1) / (2 * V);
  const int g = pow2_at_least(units);
  return g < 32 ? g : 32;
}

// Threads over time of a time_last tile: as few pairs a thread as possible, 8 threads over time at least.
int time_lanes(const QkParams &p) {
  const int units = p.rot / 2 + (p.D - p.rot + 1) / 2;
  const int ty = pow2_at_least(units);
  return kThr / (ty < 32 ? ty : 32);
}

struct TimePlan {
  int TX;
  int64_t tiles[2];
};
TimePlan time_plan(const QkParams &p) {
  TimePlan t;
  t.TX = time_lanes(p);
  const int64_t span = (int64_t)t.TX * (p.vec ? 8 : 1);
  for (int s = 0; s < 2; s++) t.tiles[s] = p.Bt * p.H[s] * ((p.L + span - 1) / span);
  return t;
}

// CTAs of the backward: in proportion to the rows of a side, at least one where it has any.
void bwd_blocks(const QkParams &p, const int64_t *work, int *nb0, int *nb1) {
  const int64_t all = work[0] + work[1], most = all < kBwdCtas ? all : kBwdCtas;
  int64_t n[2];
  for (int s = 0; s < 2; s++) {
    n[s] = all ? work[s] * most / all : 0;
    if (work[s] && !n[s]) n[s] = 1;
  }
  *nb0 = (int)n[0];
  *nb1 = (int)n[1];
}

// Heads per step of a backward's group: two where a side has two.
int bwd_heads(const QkParams &p) { return p.H[0] > 1 && p.H[1] != 1 ? 2 : 1; }

void bwd_plan(const QkParams &p, int *nb0, int *nb1, int *G, TimePlan *tp) {
  int64_t work[2];
  if (p.time_last) {
    *tp = time_plan(p);
    work[0] = tp->tiles[0];
    work[1] = tp->tiles[1];
  } else {
    *G = lanes_per_row(p, p.vec ? 8 : 1);
    const int per_cta = kThr / *G, hp = p.vec ? bwd_heads(p) : 1;
    for (int s = 0; s < 2; s++) work[s] = (p.Bt * p.L * ((p.H[s] + hp - 1) / hp) + per_cta - 1) / per_cta;
  }
  bwd_blocks(p, work, nb0, nb1);
}

template <typename T, int V, int NU, int HP>
cudaError_t fwd_launch(const QkParams &p, cudaStream_t s) {
  const int G = lanes_per_row(p, V);
  const int64_t chunks = (p.H[0] + p.H[1] + HP - 1) / HP, groups = p.Bt * p.L * chunks;
  const int64_t blocks = (groups * G + kThr - 1) / kThr;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  qk_fwd_kernel<T, V, NU, HP><<<(unsigned)blocks, kThr, 0, s>>>(p, G, chunks);
  return cudaGetLastError();
}

template <typename T, int TV, int NS>
cudaError_t fwd_time(const QkParams &p, cudaStream_t s) {
  const TimePlan t = time_plan(p);
  const int64_t tiles = t.tiles[0] + t.tiles[1];
  if (tiles > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const size_t smem = sizeof(float) * kThr * TV;
  qk_time_kernel<T, TV, NS, false><<<(unsigned)tiles, kThr, smem, s>>>(p, t.TX, 0, t.tiles[0], t.tiles[1]);
  return cudaGetLastError();
}

template <typename T> cudaError_t fwd_t(const QkParams &p, cudaStream_t s) {
  if (p.time_last) {
    const bool one = p.rot / 2 + (p.D - p.rot + 1) / 2 <= 32;
    if (p.vec) return one ? fwd_time<T, 8, 1>(p, s) : fwd_time<T, 8, 8>(p, s);
    return one ? fwd_time<T, 1, 1>(p, s) : fwd_time<T, 1, 8>(p, s);
  }
  if (!p.vec) {
    const bool few = p.rot / 2 + (p.D - p.rot + 1) / 2 <= 64;
    return few ? fwd_launch<T, 1, 2, 1>(p, s) : fwd_launch<T, 1, 8, 1>(p, s);
  }
  // several heads a group share its angles; one where the rows are too few to fill the GPU's warps
  const int heads = p.H[0] + p.H[1];
  const int64_t warps = p.Bt * p.L * heads * lanes_per_row(p, 8) / 32;
  if (heads >= 4 && warps >= 148 * 64) return fwd_launch<T, 8, 1, 4>(p, s);
  if (heads >= 2 && warps >= 148 * 32) return fwd_launch<T, 8, 1, 2>(p, s);
  return fwd_launch<T, 8, 1, 1>(p, s);
}

template <typename T, int V, int NU, int HP>
cudaError_t bwd_launch(const QkParams &p, int G, int nb0, int nb, cudaStream_t s) {
  const size_t smem = p.dw[0] || p.dw[1] ? sizeof(float) * (size_t)(kThr / G) * p.D : 0;
  qk_bwd_kernel<T, V, NU, HP><<<nb, kThr, smem, s>>>(p, G, nb0);
  return cudaGetLastError();
}

template <typename T, int TV, int NS>
cudaError_t bwd_time(const QkParams &p, const TimePlan &t, int nb0, int nb, cudaStream_t s) {
  const size_t smem = sizeof(float) * kThr * (TV == 1 ? 2 : 2 * TV);
  qk_time_kernel<T, TV, NS, true><<<nb, kThr, smem, s>>>(p, t.TX, nb0, t.tiles[0], t.tiles[1]);
  return cudaGetLastError();
}

template <typename T> cudaError_t bwd_t(const QkParams &p, cudaStream_t s) {
  int nb0 = 0, nb1 = 0, G = 1;
  TimePlan tp;
  bwd_plan(p, &nb0, &nb1, &G, &tp);
  const int nb = nb0 + nb1;
  cudaError_t e;
  if (p.time_last) {
    const bool one = p.rot / 2 + (p.D - p.rot + 1) / 2 <= 32;
    if (p.vec) e = one ? bwd_time<T, 8, 1>(p, tp, nb0, nb, s) : bwd_time<T, 8, 8>(p, tp, nb0, nb, s);
    else e = one ? bwd_time<T, 1, 1>(p, tp, nb0, nb, s) : bwd_time<T, 1, 8>(p, tp, nb0, nb, s);
  } else if (!p.vec) {
    const bool few = p.rot / 2 + (p.D - p.rot + 1) / 2 <= 64;
    e = few ? bwd_launch<T, 1, 2, 1>(p, G, nb0, nb, s) : bwd_launch<T, 1, 8, 1>(p, G, nb0, nb, s);
  } else {
    e = bwd_heads(p) == 2 ? bwd_launch<T, 8, 1, 2>(p, G, nb0, nb, s) : bwd_launch<T, 8, 1, 1>(p, G, nb0, nb, s);
  }
  if (e != cudaSuccess || (!p.dw[0] && !p.dw[1])) return e;
  qk_dw_kernel<<<dim3((unsigned)((p.D + 31) / 32), 2), 256, 0, s>>>(p, nb0, nb);
  return cudaGetLastError();
}

}  // namespace

// Whatever the plan: at most kBwdCtas shares, one more where a side rounds up from none.
size_t qk_bwd_workspace_bytes(const QkParams &p) {
  return p.dw[0] || p.dw[1] ? sizeof(float) * (size_t)(kBwdCtas + 2) * (size_t)p.D : 0;
}

cudaError_t launch_qk_fwd(const QkParams &p, int in_bf16, cudaStream_t s) {
  return in_bf16 ? fwd_t<__nv_bfloat16>(p, s) : fwd_t<float>(p, s);
}
cudaError_t launch_qk_bwd(const QkParams &p, int in_bf16, cudaStream_t s) {
  return in_bf16 ? bwd_t<__nv_bfloat16>(p, s) : bwd_t<float>(p, s);
}

}  // namespace ssm
