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
// its squares by shuffles. Head sizes, strides or alignments that do not fit take units of one pair.
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
constexpr int kBwdCtas = 148 * 3;         // most CTAs of a backward (each keeps a share of dw)
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

// Rows asked for ahead, and in use, per group of lanes: 16 KB of slots a CTA in bf16.
template <typename T, typename Td, bool BWD> constexpr int kRowStages = BWD ? (sizeof(T) + sizeof(Td) <= 4 ? 4 : 3) : (sizeof(T) == 2 ? 4 : 3);

// Of token b L + t.
__device__ __forceinline__ double position(const QkParams &p, int64_t token, int64_t t) {
  if (!p.pos) return (double)(p.pos0 + t);
  return p.pos_i64 ? (double)static_cast<const int64_t *>(p.pos)[token]
                   : (double)static_cast<const int32_t *>(p.pos)[token];
}
// Turns per position of pair j.
__device__ __forceinline__ double frequency(const QkParams &p, int j) {
  return kInvTwoPi *
         (p.freq_f64 ? static_cast<const double *>(p.inv_freq)[j] : (double)static_cast<const float *>(p.inv_freq)[j]);
}
// Cosine and sine of pos * f turns, times the scale.
template <bool PRECISE>
__device__ __forceinline__ void turn(double pos, double f, float scale, float &c, float &s) {
  const double t = pos * f;
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
__device__ __forceinline__ float inv_rms(const QkParams &p, float sum) {
  float r;  // 2^-23 of the result at most
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(sum, p.inv_D, p.eps)));
  return r;
}

// Pair unit u of a row: elements o1 and o2, turned as a pair where rot; o2 == D at an odd end.
struct Unit {
  int o1, o2;
  bool on, rot;
};
__device__ __forceinline__ Unit unit_of(const QkParams &p, int u) {
  const int ur = p.rot / 2, n = (p.D - p.rot + 1) / 2;
  Unit r;
  r.rot = u < ur;
  r.on = u < ur + n;
  const bool half = r.rot && !p.interleaved;
  r.o1 = half ? u : 2 * u;  // the rest follows the rotated pairs at 2 u too
  r.o2 = half ? ur + u : r.o1 + 1;
  return r;
}
__device__ __forceinline__ void load_unit(const void *p, int bf16, int64_t at, const Unit &u, bool on, int D, float *v) {
  v[0] = u.on && on ? ld1(p, bf16, at + u.o1) : 0.f;
  v[1] = u.on && on && u.o2 < D ? ld1(p, bf16, at + u.o2) : 0.f;
}
__device__ __forceinline__ void store_unit(void *p, int bf16, int64_t at, const Unit &u, bool on, int D, const float *v) {
  if (!u.on || !on) return;
  st1(p, bf16, at + u.o1, v[0]);
  if (u.o2 < D) st1(p, bf16, at + u.o2, v[1]);
}
__device__ __forceinline__ void load_weights(const float *w, const Unit &u, int D, float *v) {
  v[0] = w && u.on ? w[u.o1] : 1.f;
  v[1] = w && u.on && u.o2 < D ? w[u.o2] : 1.f;
}

__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 neg2(float2 a) { return make_float2(-a.x, -a.y); }

// The 16 elements of a unit as two runs of 8, first and second members of its pairs: the two groups of the
// half layout, the even and the odd elements of the interleaved one.
template <bool INTER, typename T> __device__ __forceinline__ void runs(const Raw8<T> &a, const Raw8<T> &b, float2 *f, float2 *s) {
  float v[16];
  unpack8(a, v);
  unpack8(b, v + 8);
#pragma unroll
  for (int j = 0; j < 4; j++) {
    f[j] = INTER ? make_float2(v[4 * j], v[4 * j + 2]) : make_float2(v[2 * j], v[2 * j + 1]);
    s[j] = INTER ? make_float2(v[4 * j + 1], v[4 * j + 3]) : make_float2(v[8 + 2 * j], v[8 + 2 * j + 1]);
  }
}
template <bool INTER>
__device__ __forceinline__ void store_runs(void *p, int bf16, int64_t o1, int64_t o2, const float2 *f, const float2 *s) {
  float v[16];
#pragma unroll
  for (int j = 0; j < 4; j++) {
    v[INTER ? 4 * j : 2 * j] = f[j].x;
    v[INTER ? 4 * j + 2 : 2 * j + 1] = f[j].y;
    v[INTER ? 4 * j + 1 : 8 + 2 * j] = s[j].x;
    v[INTER ? 4 * j + 3 : 8 + 2 * j + 1] = s[j].y;
  }
  st8any(p, bf16, o1, v);
  st8any(p, bf16, o2, v + 8);
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

// Rows (b, t, h) of one side, heads fastest, walked in steps of dt tokens and dh heads.
struct Walk {
  int64_t token;  // b L + t
  int t, h;
  __device__ __forceinline__ void start(int64_t row, int64_t H, int64_t L, int64_t &b) {
    int64_t hh, tt;
    divide(row, H, token, hh);
    divide(token, L, b, tt);
    t = (int)tt;
    h = (int)hh;
  }
};
// A lane's place in one tensor along a walk, moved by additions alone: a step, a step that passes the last head of a
// token, a step past the last token of a batch element.
struct Place {
  int64_t at, step, wrap, turn;
  __device__ __forceinline__ Place(const QkTensor &x, const Walk &w, int64_t b, int dt, int dh, int H, int L, int o) {
    at = b * x.sb + w.t * x.sr + w.h * x.sh + o;
    step = dt * x.sr + dh * x.sh;
    wrap = x.sr - H * x.sh;
    turn = x.sb - L * x.sr;
  }
};
// One step; true where the token changed.
template <typename... P>
__device__ __forceinline__ bool advance(Walk &w, int dt, int dh, int H, int L, P &...places) {
  w.h += dh;
  const bool more = w.h >= H;
  const int moved = dt + (more ? 1 : 0);
  w.t += moved;
  w.token += moved;
  ((places.at += places.step), ...);
  if (more) {
    w.h -= H;
    ((places.at += places.wrap), ...);
  }
  while (w.t >= L) {
    w.t -= L;
    ((places.at += places.turn), ...);
  }
  return moved != 0;
}
// Sums over the G lanes of a row.
template <typename... F> __device__ __forceinline__ void sum_lanes(int G, F &...v) {
  if (G == 8) {  // heads of 128
#pragma unroll
    for (int off = 4; off >= 1; off >>= 1) ((v += __shfl_xor_sync(kFull, v, off)), ...);
  } else {
    for (int off = G / 2; off >= 1; off >>= 1) ((v += __shfl_xor_sync(kFull, v, off)), ...);
  }
}

// Rows in 16-byte runs. CTAs [0, nb0) take the queries, the others the keys; a warp takes `per` consecutive rows
// of its side, 32 / G at a time (G lanes a row, a unit of 16 elements each), and the rows ahead travel in a ring of
// cp.async slots that every lane fills and reads alone. Cosines and sines are recomputed where the token
// changes; a unit that is not rotated keeps 1 and 0. The backward adds its share of dw over all its rows.
template <typename T, typename Td, bool BWD, bool INTER>
__global__ void __launch_bounds__(kThr, BWD ? 2 : 3)
qk_rows_kernel(const __grid_constant__ QkParams p, int G, int nb0, int64_t per0, int64_t per1) {
  constexpr bool PRECISE = sizeof(T) == 4;
  constexpr int kSlotsV = sizeof(T), kSlotsG = BWD ? sizeof(Td) : 0;  // 16-byte slots of 16 elements
  constexpr int kSlots = kSlotsV + kSlotsG;
  constexpr int S = kRowStages<T, Td, BWD>;
  extern __shared__ __align__(16) char smem[];  // the ring; afterwards (groups, D) sums of dw
  const int side = (int)blockIdx.x >= nb0;
  const int block = side ? blockIdx.x - nb0 : blockIdx.x;
  const int lane = threadIdx.x & 31, sub = lane & (G - 1), grp = lane / G, step = 32 / G;
  const int64_t per = side ? per1 : per0;
  const int H = p.H[side], L = (int)p.L;
  const QkTensor in = p.in[side], dout = p.dout[side], out = p.out[side];
  const int64_t first = ((int64_t)block * (kThr / 32) + (threadIdx.x >> 5)) * per;
  const int64_t total = p.Bt * p.L * H;
  const int n_rows = (int)(first >= total ? 0 : total - first < per ? total - first : per);  // of this warp
  const int dt = step / H, dh = step % H;
  // the lane's unit
  const int ur = p.rot / 16;
  const bool on = sub < p.D / 16, rot = sub < ur;
  const bool half = rot && !INTER;
  const int o1 = half ? 8 * sub : 16 * sub, o2 = half ? p.rot / 2 + 8 * sub : o1 + 8;
  // in shared memory, by unit: the weights of its two runs, and its pairs' turns per position
  __shared__ float4 sw[4][32];
  __shared__ double sf[8][32];
  if (threadIdx.x < p.D / 16) {
    float2 w[8];
#pragma unroll
    for (int j = 0; j < 8; j++) w[j] = splat(1.f);
    if (p.norm && p.w[side]) {
      const int u = threadIdx.x;
      const bool h = u < ur && !INTER;
      Raw8<float> a, b;
      ld8(p.w[side] + (h ? 8 * u : 16 * u), a);
      ld8(p.w[side] + (h ? p.rot / 2 + 8 * u : 16 * u + 8), b);
      runs<INTER>(a, b, w, w + 4);
    }
#pragma unroll
    for (int j = 0; j < 4; j++) sw[j][threadIdx.x] = make_float4(w[2 * j].x, w[2 * j].y, w[2 * j + 1].x, w[2 * j + 1].y);
  }
  for (int j = threadIdx.x; j < p.rot / 2; j += kThr) sf[j & 7][j >> 3] = frequency(p, j);
  float2 d1[4], d2[4], c[4], s[4];
#pragma unroll
  for (int j = 0; j < 4; j++) {
    d1[j] = d2[j] = s[j] = splat(0.f);
    c[j] = splat(1.f);
  }
  char *const mine = smem + threadIdx.x * 16;
  auto slot = [&](int stage, int k) { return mine + (stage * kSlots + k) * (kThr * 16); };
  auto clear = [&](int stage) {
#pragma unroll
    for (int k = 0; k < kSlots; k++) *reinterpret_cast<uint4 *>(slot(stage, k)) = make_uint4(0, 0, 0, 0);
  };
  if (!on) {  // lanes without a unit hold zeros throughout
#pragma unroll
    for (int j = 0; j < S; j++) clear(j);
  }
  const bool reads_v = !BWD || p.norm;
  const int gap = o2 - o1;
  Walk ahead, now;
  int64_t b0;
  ahead.start(first + grp, H, L, b0);
  now = ahead;
  Place from(in, ahead, b0, dt, dh, H, L, o1), dfrom(dout, ahead, b0, dt, dh, H, L, o1), to(out, now, b0, dt, dh, H, L, o1);
  int left = n_rows - grp;  // rows of this group still to be asked for, times step
  auto fetch = [&](int stage) {
    if (left > 0) {
      if (on) {
        if (reads_v) {
          const T *a = static_cast<const T *>(in.p) + from.at, *b = a + gap;
#pragma unroll
          for (int k = 0; k < kSlotsV / 2; k++) {
            cp_async16(slot(stage, k), reinterpret_cast<const char *>(a) + 16 * k);
            cp_async16(slot(stage, kSlotsV / 2 + k), reinterpret_cast<const char *>(b) + 16 * k);
          }
        }
        if (BWD) {
          const Td *a = static_cast<const Td *>(dout.p) + dfrom.at, *b = a + gap;
#pragma unroll
          for (int k = 0; k < kSlotsG / 2; k++) {
            cp_async16(slot(stage, kSlotsV + k), reinterpret_cast<const char *>(a) + 16 * k);
            cp_async16(slot(stage, kSlotsV + kSlotsG / 2 + k), reinterpret_cast<const char *>(b) + 16 * k);
          }
        }
      }
      left -= step;
      if (BWD) advance(ahead, dt, dh, H, L, from, dfrom);
      else advance(ahead, dt, dh, H, L, from);
    } else {
      clear(stage);  // behind the group's last row: zeros, which add nothing to dw
    }
    cp_async_commit();
  };
  auto take = [&](int stage, int k, auto &a, auto &b) {
    constexpr int n = sizeof(a) / 16;
#pragma unroll
    for (int j = 0; j < n; j++) {
      reinterpret_cast<uint4 *>(&a)[j] = *reinterpret_cast<const uint4 *>(slot(stage, k + j));
      reinterpret_cast<uint4 *>(&b)[j] = *reinterpret_cast<const uint4 *>(slot(stage, k + n + j));
    }
  };
#pragma unroll
  for (int j = 0; j < S - 1; j++) fetch(j);
  // the weights of run 1 (pairs 0 .. 3) or 2 (4 .. 7)
  auto weights = [&](int run, float2 *w) {
    const float4 a = sw[2 * run][sub], b = sw[2 * run + 1][sub];
    w[0] = make_float2(a.x, a.y);
    w[1] = make_float2(a.z, a.w);
    w[2] = make_float2(b.x, b.y);
    w[3] = make_float2(b.z, b.w);
  };
  __syncthreads();
  int stage = 0;
  bool fresh = true;
  for (int i = 0; i < n_rows; i += step) {
    const bool live = i + grp < n_rows;
    fetch(stage == 0 ? S - 1 : stage - 1);
    if (fresh && rot && live) {
      const double pos = position(p, now.token, now.t);
#pragma unroll
      for (int j = 0; j < 4; j++) {
        turn<PRECISE>(pos, sf[2 * j][sub], p.rot_scale, c[j].x, s[j].x);
        turn<PRECISE>(pos, sf[2 * j + 1][sub], p.rot_scale, c[j].y, s[j].y);
      }
    }
    cp_async_wait<S - 1>();
    float2 v1[4], v2[4];
    if (reads_v) {
      Raw8<T> a, b;
      take(stage, 0, a, b);
      runs<INTER>(a, b, v1, v2);
    }
    if constexpr (BWD) {
      float2 g1[4], g2[4];
      {
        Raw8<Td> a, b;
        take(stage, kSlotsV, a, b);
        runs<INTER>(a, b, g1, g2);
      }
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const float2 x = g1[j], y = g2[j];
        g1[j] = fma2(y, s[j], mul2(x, c[j]));
        g2[j] = fma2(x, neg2(s[j]), mul2(y, c[j]));
      }
      if (p.norm) {
        float2 s2 = splat(0.f), t2 = splat(0.f), gw1[4], gw2[4];
        weights(0, gw1);
        weights(1, gw2);
#pragma unroll
        for (int j = 0; j < 4; j++) {
          gw1[j] = mul2(g1[j], gw1[j]);
          gw2[j] = mul2(g2[j], gw2[j]);
          s2 = fma2(v1[j], v1[j], s2);
          s2 = fma2(v2[j], v2[j], s2);
          t2 = fma2(gw1[j], v1[j], t2);
          t2 = fma2(gw2[j], v2[j], t2);
        }
        float sum = s2.x + s2.y, dot = t2.x + t2.y;
        sum_lanes(G, sum, dot);
        const float sc = live ? inv_rms(p, sum) : 0.f;  // with an eps of 0, 1 / sqrt(0) of a row that is none
        const float2 k2 = splat(-sc * sc * sc * dot * p.inv_D), sc2 = splat(sc);
#pragma unroll
        for (int j = 0; j < 4; j++) {
          d1[j] = fma2(mul2(g1[j], sc2), v1[j], d1[j]);
          d2[j] = fma2(mul2(g2[j], sc2), v2[j], d2[j]);
          g1[j] = fma2(v1[j], k2, mul2(gw1[j], sc2));
          g2[j] = fma2(v2[j], k2, mul2(gw2[j], sc2));
        }
      }
      if (out.p && on && live) store_runs<INTER>(out.p, out.bf16, to.at, to.at + gap, g1, g2);
    } else {
      if (p.norm) {
        float2 s2 = splat(0.f);
#pragma unroll
        for (int j = 0; j < 4; j++) {
          s2 = fma2(v1[j], v1[j], s2);
          s2 = fma2(v2[j], v2[j], s2);
        }
        float sum = s2.x + s2.y;
        sum_lanes(G, sum);
        const float2 sc2 = splat(inv_rms(p, sum));
        float2 w[4];
        weights(0, w);
#pragma unroll
        for (int j = 0; j < 4; j++) v1[j] = mul2(v1[j], mul2(w[j], sc2));
        weights(1, w);
#pragma unroll
        for (int j = 0; j < 4; j++) v2[j] = mul2(v2[j], mul2(w[j], sc2));
      }
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const float2 x = v1[j], y = v2[j];
        v1[j] = fma2(y, neg2(s[j]), mul2(x, c[j]));
        v2[j] = fma2(x, s[j], mul2(y, c[j]));
      }
      if (on && live) store_runs<INTER>(out.p, out.bf16, to.at, to.at + gap, v1, v2);
    }
    stage = stage == S - 1 ? 0 : stage + 1;
    fresh = advance(now, dt, dh, H, L, to);
  }
  if (!BWD || !p.dw[side]) return;
  // the block's share of dw: the groups' in their order
  cp_async_wait<0>();
  __syncthreads();
  float *const sums = reinterpret_cast<float *>(smem);
  if (on) {
    float *row = sums + (threadIdx.x / G) * p.D;
#pragma unroll
    for (int j = 0; j < 4; j++) {
      row[INTER ? o1 + 4 * j : o1 + 2 * j] = d1[j].x;
      row[INTER ? o1 + 4 * j + 2 : o1 + 2 * j + 1] = d1[j].y;
      row[INTER ? o1 + 4 * j + 1 : o2 + 2 * j] = d2[j].x;
      row[INTER ? o1 + 4 * j + 3 : o2 + 2 * j + 1] = d2[j].y;
    }
  }
  __syncthreads();
  for (int j = threadIdx.x; j < p.D; j += kThr) {
    float t = 0.f;
    for (int r = 0; r < kThr / G; r++) t += sums[r * p.D + j];
    p.part[(int64_t)blockIdx.x * p.D + j] = t;
  }
}

// Any head size, stride and alignment: units of one pair, NU a lane. G lanes take a row at a time.
template <typename T, int NU>
__global__ void __launch_bounds__(kThr) qk_pairs_fwd_kernel(const __grid_constant__ QkParams p, int G) {
  constexpr bool PRECISE = sizeof(T) == 4;
  const int lane = threadIdx.x & 31, sub = lane & (G - 1);
  const int64_t heads = p.H[0] + p.H[1], item = ((int64_t)blockIdx.x * kThr + threadIdx.x) / G;
  int64_t token, h, b, t;
  divide(item, heads, token, h);
  divide(token, p.L, b, t);
  const bool live = b < p.Bt;  // dead groups follow along for the shuffles
  const int side = h >= p.H[0];
  if (side) h -= p.H[0];
  const QkTensor &in = p.in[side], &out = p.out[side];
  const int64_t at = b * in.sb + t * in.sr + h * in.sh, to = b * out.sb + t * out.sr + h * out.sh;
  float v[NU][2], sum = 0.f;
#pragma unroll
  for (int n = 0; n < NU; n++) {
    load_unit(in.p, PRECISE ? 0 : 1, at, unit_of(p, sub + n * G), live, p.D, v[n]);
    sum = fmaf(v[n][0], v[n][0], fmaf(v[n][1], v[n][1], sum));
  }
  const double pos = live && p.rot ? position(p, token, t) : 0.0;
  if (p.norm) {
    sum_lanes(G, sum);
    sum = inv_rms(p, sum);
  }
#pragma unroll
  for (int n = 0; n < NU; n++) {
    const Unit u = unit_of(p, sub + n * G);
    if (p.norm) {
      float w[2];
      load_weights(p.w[side], u, p.D, w);
      v[n][0] *= sum * w[0];
      v[n][1] *= sum * w[1];
    }
    if (u.rot) {
      float c, s;
      turn<PRECISE>(pos, frequency(p, sub + n * G), p.rot_scale, c, s);
      const float x = v[n][0], y = v[n][1];
      v[n][0] = x * c - y * s;
      v[n][1] = y * c + x * s;
    }
    store_unit(out.p, out.bf16, to, u, live, p.D, v[n]);
  }
}

// Groups of lanes walk the rows of one side (blocks [0, nb0) the queries, the others the keys) with a stride
// of the side's groups and keep their share of dw in registers.
template <typename T, int NU>
__global__ void __launch_bounds__(kThr) qk_pairs_bwd_kernel(const __grid_constant__ QkParams p, int G, int nb0) {
  constexpr bool PRECISE = sizeof(T) == 4;
  extern __shared__ float sdw[];  // (groups, D) with dw
  const int side = (int)blockIdx.x >= nb0;
  const int64_t block = side ? blockIdx.x - nb0 : blockIdx.x, blocks = side ? gridDim.x - nb0 : nb0;
  const int lane = threadIdx.x & 31, sub = lane & (G - 1), per_cta = kThr / G;
  const int64_t items = p.Bt * p.L * p.H[side];
  const QkTensor in = p.in[side], dout = p.dout[side], out = p.out[side];
  float w[NU][2], dw[NU][2];
#pragma unroll
  for (int n = 0; n < NU; n++) {
    if (p.norm) load_weights(p.w[side], unit_of(p, sub + n * G), p.D, w[n]);
    dw[n][0] = dw[n][1] = 0.f;
  }
  // the trip count is the block's, so that every lane of a warp is there for the shuffles
  for (int64_t i0 = block * per_cta; i0 < items; i0 += blocks * per_cta) {
    const int64_t item = i0 + threadIdx.x / G;
    const bool live = item < items;
    int64_t token, h, b, t;
    divide(live ? item : 0, p.H[side], token, h);
    divide(token, p.L, b, t);
    float v[NU][2], g[NU][2], sum = 0.f, dot = 0.f;
    const int64_t gat = b * dout.sb + t * dout.sr + h * dout.sh, at = b * in.sb + t * in.sr + h * in.sh;
#pragma unroll
    for (int n = 0; n < NU; n++) {
      const Unit u = unit_of(p, sub + n * G);
      load_unit(dout.p, dout.bf16, gat, u, live, p.D, g[n]);
      if (p.norm) load_unit(in.p, PRECISE ? 0 : 1, at, u, live, p.D, v[n]);
    }
    const double pos = p.rot ? position(p, token, t) : 0.0;
#pragma unroll
    for (int n = 0; n < NU; n++) {
      if (unit_of(p, sub + n * G).rot) {
        float c, s;
        turn<PRECISE>(pos, frequency(p, sub + n * G), p.rot_scale, c, s);
        const float x = g[n][0], y = g[n][1];
        g[n][0] = x * c + y * s;
        g[n][1] = y * c - x * s;
      }
      if (p.norm) {
        sum = fmaf(v[n][0], v[n][0], fmaf(v[n][1], v[n][1], sum));
        dot = fmaf(g[n][0] * w[n][0], v[n][0], fmaf(g[n][1] * w[n][1], v[n][1], dot));
      }
    }
    if (p.norm) {
      sum_lanes(G, sum, dot);
      const float sc = inv_rms(p, sum), back = sc * sc * dot * p.inv_D;
#pragma unroll
      for (int n = 0; n < NU; n++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
          dw[n][e] = fmaf(g[n][e] * sc, v[n][e], dw[n][e]);
          g[n][e] = sc * (g[n][e] * w[n][e] - v[n][e] * back);
        }
    }
    if (out.p) {
      const int64_t to = b * out.sb + t * out.sr + h * out.sh;
#pragma unroll
      for (int n = 0; n < NU; n++) store_unit(out.p, out.bf16, to, unit_of(p, sub + n * G), live, p.D, g[n]);
    }
  }
  if (!p.dw[side]) return;
  // the block's share of dw: the groups' in their order
#pragma unroll
  for (int n = 0; n < NU; n++) {
    const Unit u = unit_of(p, sub + n * G);
    if (!u.on) continue;
    float *row = sdw + (threadIdx.x / G) * p.D;
    row[u.o1] = dw[n][0];
    if (u.o2 < p.D) row[u.o2] = dw[n][1];
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
// A pair unit is unit_of: elements o1 and o2 (or o1 alone at an odd end).
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
    auto fetch = [&](const Unit &u, int unit) {
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
              turn<PRECISE>(position(p, b * p.L + t0 + e, t0 + e), f, p.rot_scale, cs, sn);
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
          const Unit u = unit_of(p, unit);
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
        sum[e] = inv_rms(p, s);
        dot[e] = sum[e] * sum[e] * q * p.inv_D;
      }
    }
#pragma unroll
    for (int n = 0; n < NS; n++) {
      const int unit = ty + n * TY;
      if (unit < n_units) {
        const Unit u = unit_of(p, unit);
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
              turn<PRECISE>(position(p, b * p.L + t0 + e, t0 + e), f, p.rot_scale, cs, sn);
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
      const Unit u = unit_of(p, unit);
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

// dw of both sides from the blocks' shares, in a fixed order: a CTA takes 32 elements of one side, each of
// its 32 rows every 32nd share, up to 14 loads in flight.
__global__ void __launch_bounds__(1024) qk_dw_kernel(const __grid_constant__ QkParams p, int nb0, int nb) {
  __shared__ float red[32][33];
  const int side = blockIdx.y, x = threadIdx.x & 31, y = threadIdx.x >> 5;
  if (!p.dw[side]) return;
  const int j = blockIdx.x * 32 + x, lo = side ? nb0 : 0, hi = side ? nb : nb0;
  float v[kBwdCtas / 32 + 1], s = 0.f;
#pragma unroll
  for (int k = 0; k < kBwdCtas / 32 + 1; k++) {
    const int at = lo + y + 32 * k;
    v[k] = j < p.D && at < hi ? p.part[(int64_t)at * p.D + j] : 0.f;
  }
#pragma unroll
  for (int k = 0; k < kBwdCtas / 32 + 1; k++) s += v[k];
  red[y][x] = s;
  __syncthreads();
  s = red[x][y];  // element y's shares
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(kFull, s, off);
  const int e = blockIdx.x * 32 + y;
  if (x == 0 && e < p.D) p.dw[side][e] = s;
}

// ---- launchers ---------------------------------------------------------------------------------

namespace {

int pow2_at_least(int n) {
  int g = 1;
  while (g < n) g *= 2;
  return g;
}

// Lanes that hold a row: a unit of 16 elements each (vec); at least a fourth of the pairs otherwise, at most a warp.
int lanes_per_row(const QkParams &p) {
  if (p.vec) return pow2_at_least(p.D / 16);
  const int pairs = p.rot / 2 + (p.D - p.rot + 1) / 2, g = pow2_at_least((pairs + 3) / 4);
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

// At most `most` CTAs over both sides, in proportion to their work (in CTAs), at least one where a side has any.
void split_blocks(const int64_t *work, int64_t most, int *nb0, int *nb1) {
  const int64_t all = work[0] + work[1];
  if (all < most) most = all;
  int64_t n[2];
  for (int s = 0; s < 2; s++) {
    n[s] = all ? work[s] * most / all : 0;
    if (work[s] && !n[s]) n[s] = 1;
  }
  *nb0 = (int)n[0];
  *nb1 = (int)n[1];
}

template <typename T, typename Td, bool BWD, bool INTER>
cudaError_t rows_launch(const QkParams &p, int *nb0, int *nb, cudaStream_t s) {
  constexpr int kWarps = kThr / 32;
  const int G = lanes_per_row(p), step = 32 / G;
  int64_t rows[2], work[2], per[2] = {1, 1};
  for (int j = 0; j < 2; j++) {
    rows[j] = p.Bt * p.L * p.H[j];
    work[j] = (rows[j] + kWarps * step - 1) / (kWarps * step);
  }
  int n[2];
  split_blocks(work, 148 * (BWD ? 2 : 3), &n[0], &n[1]);
  for (int j = 0; j < 2; j++) {  // rows per warp, whole steps
    if (!n[j]) continue;
    per[j] = (rows[j] + (int64_t)n[j] * kWarps - 1) / ((int64_t)n[j] * kWarps);
    per[j] = (per[j] + step - 1) / step * step;
    if (per[j] > 0x7fffff00) return cudaErrorInvalidConfiguration;
  }
  *nb0 = n[0];
  *nb = n[0] + n[1];
  constexpr int kSlots = sizeof(T) + (BWD ? sizeof(Td) : 0);
  const int ring = kThr * 16 * kSlots * kRowStages<T, Td, BWD>, sums = (int)sizeof(float) * (kThr / G) * p.D;
  const int smem = BWD && sums > ring ? sums : ring;
  const auto kernel = qk_rows_kernel<T, Td, BWD, INTER>;
  if (smem > 47 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  kernel<<<*nb, kThr, smem, s>>>(p, G, n[0], per[0], per[1]);
  return cudaGetLastError();
}

template <typename T, int NU> cudaError_t pairs_fwd(const QkParams &p, cudaStream_t s) {
  const int G = lanes_per_row(p);
  const int64_t blocks = (p.Bt * p.L * (p.H[0] + p.H[1]) * G + kThr - 1) / kThr;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  qk_pairs_fwd_kernel<T, NU><<<(unsigned)blocks, kThr, 0, s>>>(p, G);
  return cudaGetLastError();
}

template <typename T, int NU> cudaError_t pairs_bwd(const QkParams &p, int *nb0, int *nb, cudaStream_t s) {
  const int G = lanes_per_row(p), per_cta = kThr / G;
  int64_t work[2];
  for (int j = 0; j < 2; j++) work[j] = (p.Bt * p.L * p.H[j] + per_cta - 1) / per_cta;
  int nb1;
  split_blocks(work, kBwdCtas, nb0, &nb1);
  *nb = *nb0 + nb1;
  const size_t smem = p.dw[0] || p.dw[1] ? sizeof(float) * (size_t)per_cta * p.D : 0;
  qk_pairs_bwd_kernel<T, NU><<<*nb, kThr, smem, s>>>(p, G, *nb0);
  return cudaGetLastError();
}

template <typename T, int TV, int NS>
cudaError_t time_fwd(const QkParams &p, cudaStream_t s) {
  const TimePlan t = time_plan(p);
  const int64_t tiles = t.tiles[0] + t.tiles[1];
  if (tiles > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const size_t smem = sizeof(float) * kThr * TV;
  qk_time_kernel<T, TV, NS, false><<<(unsigned)tiles, kThr, smem, s>>>(p, t.TX, 0, t.tiles[0], t.tiles[1]);
  return cudaGetLastError();
}

template <typename T, int TV, int NS>
cudaError_t time_bwd(const QkParams &p, int *nb0, int *nb, cudaStream_t s) {
  const TimePlan t = time_plan(p);
  int nb1;
  split_blocks(t.tiles, kBwdCtas, nb0, &nb1);
  *nb = *nb0 + nb1;
  const size_t smem = sizeof(float) * kThr * 2 * TV;
  qk_time_kernel<T, TV, NS, true><<<*nb, kThr, smem, s>>>(p, t.TX, *nb0, t.tiles[0], t.tiles[1]);
  return cudaGetLastError();
}

template <typename T> cudaError_t fwd_t(const QkParams &p, cudaStream_t s) {
  const int pairs = p.rot / 2 + (p.D - p.rot + 1) / 2;
  if (p.time_last) {
    if (p.vec) return pairs <= 32 ? time_fwd<T, 8, 1>(p, s) : time_fwd<T, 8, 8>(p, s);
    return pairs <= 32 ? time_fwd<T, 1, 1>(p, s) : time_fwd<T, 1, 8>(p, s);
  }
  if (!p.vec) return pairs <= 128 ? pairs_fwd<T, 4>(p, s) : pairs_fwd<T, 8>(p, s);
  int nb0, nb;
  return p.interleaved ? rows_launch<T, T, false, true>(p, &nb0, &nb, s) : rows_launch<T, T, false, false>(p, &nb0, &nb, s);
}

template <typename T, typename Td> cudaError_t bwd_rows(const QkParams &p, int *nb0, int *nb, cudaStream_t s) {
  return p.interleaved ? rows_launch<T, Td, true, true>(p, nb0, nb, s) : rows_launch<T, Td, true, false>(p, nb0, nb, s);
}

template <typename T> cudaError_t bwd_t(const QkParams &p, cudaStream_t s) {
  const int pairs = p.rot / 2 + (p.D - p.rot + 1) / 2;
  int nb0 = 0, nb = 0;
  cudaError_t e;
  if (p.time_last) {
    if (p.vec) e = pairs <= 32 ? time_bwd<T, 8, 1>(p, &nb0, &nb, s) : time_bwd<T, 8, 8>(p, &nb0, &nb, s);
    else e = pairs <= 32 ? time_bwd<T, 1, 1>(p, &nb0, &nb, s) : time_bwd<T, 1, 8>(p, &nb0, &nb, s);
  } else if (!p.vec) {
    e = pairs <= 128 ? pairs_bwd<T, 4>(p, &nb0, &nb, s) : pairs_bwd<T, 8>(p, &nb0, &nb, s);
  } else {
    e = p.dout[p.H[0] == 0].bf16 ? bwd_rows<T, __nv_bfloat16>(p, &nb0, &nb, s) : bwd_rows<T, float>(p, &nb0, &nb, s);
  }
  if (e != cudaSuccess || (!p.dw[0] && !p.dw[1])) return e;
  qk_dw_kernel<<<dim3((unsigned)((p.D + 31) / 32), 2), 1024, 0, s>>>(p, nb0, nb);
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
