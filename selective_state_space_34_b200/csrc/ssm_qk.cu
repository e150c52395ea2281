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
// Time innermost (time_last): a thread owns consecutive steps of a pair and walks the heads with one set of cosines and
// sines; the squares of a step meet in shared memory.
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
  // the lane's unit; the interleaved layout may turn some of a unit's pairs
  const int ur = INTER ? (p.rot + 15) / 16 : p.rot / 16, turned = p.rot / 2 - 8 * sub;
  const bool on = sub < p.D / 16, rot = sub < ur;
  const bool half = rot && !INTER;
  const int o1 = half ? 8 * sub : 16 * sub, o2 = half ? p.rot / 2 + 8 * sub : o1 + 8;
  // in shared memory, by unit: the weights of its two runs, and its pairs' turns per position
  __shared__ float4 sw[4][32];
  __shared__ double sf[8][32];
  if (threadIdx.x < 32) {  // lanes without a unit read weights too: 1, which their zeros stay 0 with
    float2 w[8];
#pragma unroll
    for (int j = 0; j < 8; j++) w[j] = splat(1.f);
    if ((int)threadIdx.x < p.D / 16 && p.norm && p.w[side]) {
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
        if (!INTER || 2 * j < turned) turn<PRECISE>(pos, sf[2 * j][sub], p.rot_scale, c[j].x, s[j].x);
        if (!INTER || 2 * j + 1 < turned) turn<PRECISE>(pos, sf[2 * j + 1][sub], p.rot_scale, c[j].y, s[j].y);
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

// Any head size, stride and alignment: units of one pair, NU a lane, over the same walk; the next row's elements are
// loaded into registers while a row is worked on.
template <typename T, typename Td, bool BWD, int NU>
__global__ void __launch_bounds__(kThr)
qk_pairs_kernel(const __grid_constant__ QkParams p, int G, int nb0, int64_t per0, int64_t per1) {
  constexpr bool PRECISE = sizeof(T) == 4;
  extern __shared__ float sdw[];  // (groups, D) sums of dw
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
  const bool reads_v = !BWD || p.norm;
  // the lane's units: first element, distance to the second (0: none), weights, sums of dw
  int o[NU], gap[NU];
  bool on[NU], rot[NU];
  float w[NU][2], dw[NU][2], c[NU], s[NU];
#pragma unroll
  for (int n = 0; n < NU; n++) {
    const Unit u = unit_of(p, sub + n * G);
    on[n] = u.on;
    rot[n] = u.on && u.rot;
    o[n] = u.o1;
    gap[n] = u.o2 < p.D ? u.o2 - u.o1 : 0;
    w[n][0] = w[n][1] = c[n] = 1.f;
    dw[n][0] = dw[n][1] = s[n] = 0.f;
    if (p.norm && p.w[side] && u.on) {
      w[n][0] = p.w[side][u.o1];
      if (gap[n]) w[n][1] = p.w[side][u.o2];
    }
  }
  Walk ahead, now;
  int64_t b0;
  ahead.start(first + grp, H, L, b0);
  now = ahead;
  Place from(in, ahead, b0, dt, dh, H, L, 0), dfrom(dout, ahead, b0, dt, dh, H, L, 0), to(out, now, b0, dt, dh, H, L, 0);
  T nv[NU][2];
  Td ng[NU][2];
  int left = n_rows - grp;
  auto fetch = [&]() {
    const T *a = static_cast<const T *>(in.p) + from.at;
    const Td *g = static_cast<const Td *>(dout.p) + dfrom.at;
#pragma unroll
    for (int n = 0; n < NU; n++) {
      nv[n][0] = nv[n][1] = from_f32<T>(0.f);
      ng[n][0] = ng[n][1] = from_f32<Td>(0.f);
      if (left > 0 && on[n]) {
        if (reads_v) {
          nv[n][0] = a[o[n]];
          if (gap[n]) nv[n][1] = a[o[n] + gap[n]];
        }
        if (BWD) {
          ng[n][0] = g[o[n]];
          if (gap[n]) ng[n][1] = g[o[n] + gap[n]];
        }
      }
    }
    left -= step;
    if (BWD) advance(ahead, dt, dh, H, L, from, dfrom);
    else advance(ahead, dt, dh, H, L, from);
  };
  fetch();
  bool fresh = true;
  for (int i = 0; i < n_rows; i += step) {
    const bool live = i + grp < n_rows;
    float v[NU][2], g[NU][2];
#pragma unroll
    for (int n = 0; n < NU; n++)
#pragma unroll
      for (int e = 0; e < 2; e++) {
        v[n][e] = to_f32(nv[n][e]);
        if (BWD) g[n][e] = to_f32(ng[n][e]);
      }
    fetch();
    if (fresh && live && p.rot) {
      const double pos = position(p, now.token, now.t);
#pragma unroll
      for (int n = 0; n < NU; n++)
        if (rot[n]) turn<PRECISE>(pos, frequency(p, sub + n * G), p.rot_scale, c[n], s[n]);
    }
    float sum = 0.f, dot = 0.f;
#pragma unroll
    for (int n = 0; n < NU; n++) {
      if (BWD) {
        const float x = g[n][0], y = g[n][1];
        g[n][0] = x * c[n] + y * s[n];
        g[n][1] = y * c[n] - x * s[n];
        dot = fmaf(g[n][0] * w[n][0], v[n][0], fmaf(g[n][1] * w[n][1], v[n][1], dot));
      }
      sum = fmaf(v[n][0], v[n][0], fmaf(v[n][1], v[n][1], sum));
    }
    float sc = 1.f, back = 0.f;
    if (p.norm) {
      sum_lanes(G, sum, dot);
      sc = live ? inv_rms(p, sum) : 0.f;  // with an eps of 0, 1 / sqrt(0) of a row that is none
      back = sc * sc * dot * p.inv_D;
    }
#pragma unroll
    for (int n = 0; n < NU; n++) {
      float x, y;
      if (BWD) {
        if (p.norm) {
          dw[n][0] = fmaf(g[n][0] * sc, v[n][0], dw[n][0]);
          dw[n][1] = fmaf(g[n][1] * sc, v[n][1], dw[n][1]);
        }
        x = p.norm ? sc * (g[n][0] * w[n][0] - v[n][0] * back) : g[n][0];
        y = p.norm ? sc * (g[n][1] * w[n][1] - v[n][1] * back) : g[n][1];
      } else {
        const float a = v[n][0] * (sc * w[n][0]), b = v[n][1] * (sc * w[n][1]);
        x = a * c[n] - b * s[n];
        y = b * c[n] + a * s[n];
      }
      if (out.p && live && on[n]) {
        st1(out.p, out.bf16, to.at + o[n], x);
        if (gap[n]) st1(out.p, out.bf16, to.at + o[n] + gap[n], y);
      }
    }
    fresh = advance(now, dt, dh, H, L, to);
  }
  if (!BWD || !p.dw[side]) return;
  // the block's share of dw: the groups' in their order
#pragma unroll
  for (int n = 0; n < NU; n++)
    if (on[n]) {
      float *row = sdw + (threadIdx.x / G) * p.D + o[n];
      row[0] = dw[n][0];
      if (gap[n]) row[gap[n]] = dw[n][1];
    }
  __syncthreads();
  for (int j = threadIdx.x; j < p.D; j += kThr) {
    float t = 0.f;
    for (int r = 0; r < kThr / G; r++) t += sdw[r * p.D + j];
    p.part[(int64_t)blockIdx.x * p.D + j] = t;
  }
}

// ---- time innermost ----------------------------------------------------------------------------

// m of the TV consecutive elements at i.
template <int TV> __device__ __forceinline__ void get_run(const void *p, int bf16, int64_t i, int m, float *v) {
  if constexpr (TV == 8) {
    if (m == 8) {
      ld8any(p, bf16, i, v);
      return;
    }
  }
#pragma unroll
  for (int e = 0; e < TV; e++) v[e] = e < m ? ld1(p, bf16, i + e) : 0.f;
}
template <int TV> __device__ __forceinline__ void put_run(void *p, int bf16, int64_t i, int m, const float *v) {
  if constexpr (TV == 8) {
    if (m == 8) {
      st8any(p, bf16, i, v);
      return;
    }
  }
#pragma unroll
  for (int e = 0; e < TV; e++)
    if (e < m) st1(p, bf16, i + e, v[e]);
}

// A tile is TX * TV steps of one batch element and a chunk of its heads (queries, then keys). A thread owns TV
// consecutive steps (8 where rows are whole 16-byte runs, else 1) of NS pairs, every TY-th, TY = kThr / TX; a
// pair unit is elements o1 and o2 (or o1 alone at an odd end). The squares of a step meet in shared memory. With one
// pair a thread the elements stay in registers and its cosines and sines serve every head of the chunk; with more
// the elements are read a second time, from L1.
template <typename T, int TV, int NS, bool BWD>
__global__ void __launch_bounds__(kThr)
qk_time_kernel(const __grid_constant__ QkParams p, int TX, int heads, int64_t chunks, int64_t tiles) {
  constexpr bool PRECISE = sizeof(T) == 4;
  extern __shared__ __align__(16) float sh[];
  const int TY = kThr / TX, tx = threadIdx.x % TX, ty = threadIdx.x / TX;
  const int span = TX * TV, per_row = (int)((p.L + span - 1) / span);
  // R threads add the squares of one step; rows of sh are padded so that they hit different banks
  const int R = span < kThr ? kThr / span : 1, pitch = span + 32 / R;
  float *const sums = sh, *const dots = sh + TY * pitch, *const res = sh + (BWD ? 2 : 1) * TY * pitch, *const res2 = res + span;
  const int n_units = p.rot / 2 + (p.D - p.rot + 1) / 2, all = p.H[0] + p.H[1];
  float dw[2][NS][2];
#pragma unroll
  for (int n = 0; n < NS; n++) dw[0][n][0] = dw[0][n][1] = dw[1][n][0] = dw[1][n][1] = 0.f;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    int64_t bc, tt, b, chunk;
    divide(tile, per_row, bc, tt);
    divide(bc, chunks, b, chunk);
    const int64_t t0 = tt * span + (int64_t)tx * TV;
    const int m = (int)(p.L - t0 < 0 ? 0 : p.L - t0 < TV ? p.L - t0 : TV);  // live steps of this thread
    float cs[TV], sn[TV];
    auto angles = [&](const Unit &u, int unit) {
      const double f = u.rot ? frequency(p, unit) : 0.0;
#pragma unroll
      for (int e = 0; e < TV; e++) {
        cs[e] = 1.f;
        sn[e] = 0.f;
        if (u.rot && e < m) turn<PRECISE>(position(p, b * p.L + t0 + e, t0 + e), f, p.rot_scale, cs[e], sn[e]);
      }
    };
    if (NS == 1) angles(unit_of(p, ty), ty);
    const int h_end = min(all, (int)(chunk + 1) * heads);
    for (int hh = (int)chunk * heads; hh < h_end; hh++) {
      const int sd = hh >= p.H[0], h = sd ? hh - p.H[0] : hh;
      const QkTensor &in = p.in[sd], &out = p.out[sd], &dout = p.dout[sd];
      const int64_t at = b * in.sb + h * in.sh + t0, dat = BWD ? b * dout.sb + h * dout.sh + t0 : 0;
      const int64_t oat = b * out.sb + h * out.sh + t0;
      float a[TV], c[TV], ga[TV], gc[TV];  // the elements of a pair, and their gradients turned back
      auto fetch = [&](const Unit &u, int unit) {
        const int m2 = u.o2 < p.D ? m : 0;
        if (!BWD || p.norm) {
          get_run<TV>(in.p, PRECISE ? 0 : 1, at + u.o1 * in.sr, m, a);
          get_run<TV>(in.p, PRECISE ? 0 : 1, at + u.o2 * in.sr, m2, c);
        }
        if (BWD) {
          get_run<TV>(dout.p, dout.bf16, dat + u.o1 * dout.sr, m, ga);
          get_run<TV>(dout.p, dout.bf16, dat + u.o2 * dout.sr, m2, gc);
          if (NS > 1) angles(u, unit);
#pragma unroll
          for (int e = 0; e < TV; e++) {
            const float x = ga[e], y = gc[e];
            ga[e] = x * cs[e] + y * sn[e];
            gc[e] = y * cs[e] - x * sn[e];
          }
        }
      };
      const float *w = p.w[sd];
      float sc[TV], back[TV];
#pragma unroll
      for (int e = 0; e < TV; e++) sc[e] = back[e] = 0.f;
      if (p.norm) {
#pragma unroll
        for (int n = 0; n < NS; n++) {
          const int unit = ty + n * TY;
          if (unit < n_units) {
            const Unit u = unit_of(p, unit);
            fetch(u, unit);
            const float wa = BWD ? (w ? w[u.o1] : 1.f) : 0.f, wc = BWD && u.o2 < p.D ? (w ? w[u.o2] : 1.f) : 0.f;
#pragma unroll
            for (int e = 0; e < TV; e++) {
              sc[e] = fmaf(a[e], a[e], fmaf(c[e], c[e], sc[e]));
              if (BWD) back[e] = fmaf(ga[e] * wa, a[e], fmaf(gc[e] * wc, c[e], back[e]));
            }
          }
        }
        // every thread's partial sums, then a step's over its TY threads in a fixed order
        if constexpr (TV == 8) {
#pragma unroll
          for (int e = 0; e < 8; e += 4) {
            *reinterpret_cast<float4 *>(sums + ty * pitch + tx * 8 + e) = make_float4(sc[e], sc[e + 1], sc[e + 2], sc[e + 3]);
            if (BWD)
              *reinterpret_cast<float4 *>(dots + ty * pitch + tx * 8 + e) = make_float4(back[e], back[e + 1], back[e + 2], back[e + 3]);
          }
        } else {
          sums[ty * pitch + tx] = sc[0];
          if (BWD) dots[ty * pitch + tx] = back[0];
        }
        __syncthreads();
        for (int k = threadIdx.x / R; k < span; k += kThr / R) {
          float s = 0.f, d = 0.f;
          for (int y = threadIdx.x % R; y < TY; y += R) {
            s += sums[y * pitch + k];
            if (BWD) d += dots[y * pitch + k];
          }
          for (int off = R / 2; off >= 1; off >>= 1) {
            s += __shfl_xor_sync(kFull, s, off);
            if (BWD) d += __shfl_xor_sync(kFull, d, off);
          }
          if (threadIdx.x % R == 0) {
            const float r = inv_rms(p, s);
            res[k] = r;
            if (BWD) res2[k] = r * r * d * p.inv_D;
          }
        }
        __syncthreads();  // the sums are read; the next head's go in after the next barrier of this kind
#pragma unroll
        for (int e = 0; e < TV; e++) {
          sc[e] = res[tx * TV + e];
          if (BWD) back[e] = res2[tx * TV + e];
        }
      }
#pragma unroll
      for (int n = 0; n < NS; n++) {
        const int unit = ty + n * TY;
        if (unit < n_units) {
          const Unit u = unit_of(p, unit);
          const bool two = u.o2 < p.D;
          if (NS > 1 || !p.norm) fetch(u, unit);  // with one pair it is still here
          const float wa = w ? w[u.o1] : 1.f, wc = w && two ? w[u.o2] : 1.f;
          if (BWD) {
            if (p.norm) {
              float x = 0.f, y = 0.f;
#pragma unroll
              for (int e = 0; e < TV; e++) {
                if (e < m) {  // a step that is none has no 1 / sqrt(0) either
                  x = fmaf(ga[e] * sc[e], a[e], x);
                  y = fmaf(gc[e] * sc[e], c[e], y);
                }
                ga[e] = sc[e] * (ga[e] * wa - a[e] * back[e]);
                gc[e] = sc[e] * (gc[e] * wc - c[e] * back[e]);
              }
              dw[0][n][0] += sd ? 0.f : x;
              dw[0][n][1] += sd ? 0.f : y;
              dw[1][n][0] += sd ? x : 0.f;
              dw[1][n][1] += sd ? y : 0.f;
            }
            if (out.p) {
              put_run<TV>(out.p, out.bf16, oat + u.o1 * out.sr, m, ga);
              if (two) put_run<TV>(out.p, out.bf16, oat + u.o2 * out.sr, m, gc);
            }
          } else {
            if (NS > 1) angles(u, unit);
#pragma unroll
            for (int e = 0; e < TV; e++) {
              const float x = p.norm ? a[e] * (sc[e] * wa) : a[e], y = p.norm ? c[e] * (sc[e] * wc) : c[e];
              a[e] = x * cs[e] - y * sn[e];
              c[e] = y * cs[e] + x * sn[e];
            }
            put_run<TV>(out.p, out.bf16, oat + u.o1 * out.sr, m, a);
            if (two) put_run<TV>(out.p, out.bf16, oat + u.o2 * out.sr, m, c);
          }
        }
      }
    }
  }
  if (!BWD || (!p.dw[0] && !p.dw[1])) return;
  // the block's shares of dw, rows 2 block + side: over the TX threads of a pair
  const int lanes = TX < 32 ? TX : 32;
#pragma unroll
  for (int sd = 0; sd < 2; sd++) {
    if (!p.dw[sd]) continue;
#pragma unroll
    for (int n = 0; n < NS; n++) {
      float x = dw[sd][n][0], y = dw[sd][n][1];
      for (int off = lanes / 2; off >= 1; off >>= 1) {
        x += __shfl_xor_sync(kFull, x, off);
        y += __shfl_xor_sync(kFull, y, off);
      }
      if (TX > 32) {
        __syncthreads();
        if (threadIdx.x % 32 == 0) {
          sh[threadIdx.x / 16] = x;
          sh[threadIdx.x / 16 + 1] = y;
        }
        __syncthreads();
        x = y = 0.f;
        for (int k = 0; k < TX / 32; k++) {
          x += sh[2 * (ty * (TX / 32) + k)];
          y += sh[2 * (ty * (TX / 32) + k) + 1];
        }
      }
      const int unit = ty + n * TY;
      if (tx == 0 && unit < n_units) {
        const Unit u = unit_of(p, unit);
        float *row = p.part + (2 * (int64_t)blockIdx.x + sd) * p.D;
        row[u.o1] = x;
        if (u.o2 < p.D) row[u.o2] = y;
      }
    }
  }
}

// dw of both sides from the blocks' shares, in a fixed order: side 0's are every stride-th of the first nb0 rows, side
// 1's every stride-th of the others from lo1. A CTA takes 32 elements of one side, each of its 32 rows every 32nd share, all
// loads in flight.
__global__ void __launch_bounds__(1024) qk_dw_kernel(const __grid_constant__ QkParams p, int n0, int lo1, int n1, int stride) {
  __shared__ float red[32][33];
  const int side = blockIdx.y, x = threadIdx.x & 31, y = threadIdx.x >> 5;
  if (!p.dw[side]) return;
  const int j = blockIdx.x * 32 + x, n = side ? n1 : n0;
  const float *part = p.part + (side ? (int64_t)lo1 * p.D : 0);
  float v[kBwdCtas / 32 + 1], s = 0.f;
#pragma unroll
  for (int k = 0; k < kBwdCtas / 32 + 1; k++) {
    const int at = y + 32 * k;
    v[k] = j < p.D && at < n ? part[(int64_t)at * stride * p.D + j] : 0.f;
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

// Pair units of a row.
int pairs_of(const QkParams &p) { return p.rot / 2 + (p.D - p.rot + 1) / 2; }

// Lanes that hold a row: a unit of 16 elements each (vec); at least a fourth of the pairs otherwise, at most a warp.
int lanes_per_row(const QkParams &p) {
  if (p.vec) return pow2_at_least(p.D / 16);
  const int g = pow2_at_least((pairs_of(p) + 3) / 4);
  return g < 32 ? g : 32;
}

// Time innermost: threads over time, heads per tile, tiles, shared memory. As few pairs a thread as possible with 8
// threads (of 8 steps) or 32 (of one step) over time at least, so that a row's accesses are 64 bytes and more; all heads of
// a batch element in one tile, for their common angles, where that leaves two tiles per SM.
struct TimePlan {
  int TX, heads;
  int64_t chunks, tiles;
  int smem;
};
TimePlan time_plan(const QkParams &p, bool bwd) {
  TimePlan t;
  const int TV = p.vec ? 8 : 1, ty = pow2_at_least(pairs_of(p)), most = p.vec ? 32 : 8;
  t.TX = kThr / (ty < most ? ty : most);
  const int span = t.TX * TV, R = span < kThr ? kThr / span : 1;
  const int64_t slices = p.Bt * ((p.L + span - 1) / span);
  const int all = p.H[0] + p.H[1];
  t.heads = slices >= 2 * 148 ? all : 1;
  t.chunks = (all + t.heads - 1) / t.heads;
  t.tiles = slices * t.chunks;
  t.smem = (int)sizeof(float) * ((bwd ? 2 : 1) * (kThr / t.TX) * (span + 32 / R) + 2 * span);
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

// How the rows of both sides are cut: CTAs of the queries and of both, rows per warp (whole steps of 32 / G rows).
struct RowPlan {
  int G, nb0, nb;
  int64_t per[2];
};
bool plan_rows(const QkParams &p, int64_t most, RowPlan *r) {
  constexpr int kWarps = kThr / 32;
  r->G = lanes_per_row(p);
  const int step = 32 / r->G;
  int64_t rows[2], work[2];
  int n[2];
  for (int j = 0; j < 2; j++) {
    rows[j] = p.Bt * p.L * p.H[j];
    work[j] = (rows[j] + kWarps * step - 1) / (kWarps * step);
  }
  split_blocks(work, most, &n[0], &n[1]);
  for (int j = 0; j < 2; j++) {
    r->per[j] = step;
    if (!n[j]) continue;
    const int64_t warps = (int64_t)n[j] * kWarps, per = (rows[j] + warps - 1) / warps;
    r->per[j] = (per + step - 1) / step * step;
    if (r->per[j] > 0x7fffff00) return false;
  }
  r->nb0 = n[0];
  r->nb = n[0] + n[1];
  return true;
}

template <typename K> cudaError_t launch_rows(K kernel, const QkParams &p, const RowPlan &r, int smem, cudaStream_t s) {
  if (smem > 40 * 1024) {  // with the kernels' own 4 KB more than the default 48 KB
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  kernel<<<r.nb, kThr, smem, s>>>(p, r.G, r.nb0, r.per[0], r.per[1]);
  return cudaGetLastError();
}

// Head elements innermost, forward (Td = T) or backward. CTAs: what fits the SMs at once, at most kBwdCtas of a backward.
template <typename T, typename Td, bool BWD> cudaError_t rows_run(const QkParams &p, RowPlan *r, cudaStream_t s) {
  if (!plan_rows(p, BWD ? (p.vec ? 148 * 2 : kBwdCtas) : 148 * (p.vec ? 3 : 6), r)) return cudaErrorInvalidConfiguration;
  const int sums = BWD && (p.dw[0] || p.dw[1]) ? (int)sizeof(float) * (kThr / r->G) * p.D : 0;
  if (p.vec) {
    constexpr int kSlots = sizeof(T) + (BWD ? sizeof(Td) : 0);
    const int ring = kThr * 16 * kSlots * kRowStages<T, Td, BWD>;
    return launch_rows(p.interleaved ? qk_rows_kernel<T, Td, BWD, true> : qk_rows_kernel<T, Td, BWD, false>, p, *r,
                       sums > ring ? sums : ring, s);
  }
  return launch_rows(pairs_of(p) <= 4 * r->G ? qk_pairs_kernel<T, Td, BWD, 4> : qk_pairs_kernel<T, Td, BWD, 8>, p, *r, sums, s);
}

// CTAs of a time_last launch: four per SM forwards, the backward's two (each keeps a share of dw of both sides).
template <typename T, bool BWD> cudaError_t time_run(const QkParams &p, int *nb, cudaStream_t s) {
  const TimePlan t = time_plan(p, BWD);
  const int64_t most = BWD ? 2 * 148 : 4 * 148;
  *nb = (int)(t.tiles < most ? t.tiles : most);
  const int pairs = pairs_of(p), TY = kThr / t.TX;
  const auto kernel = p.vec ? (pairs <= TY ? qk_time_kernel<T, 8, 1, BWD> : qk_time_kernel<T, 8, 8, BWD>)
                            : (pairs <= TY       ? qk_time_kernel<T, 1, 1, BWD>
                               : pairs <= 4 * TY ? qk_time_kernel<T, 1, 4, BWD>
                                                 : qk_time_kernel<T, 1, 32, BWD>);
  kernel<<<*nb, kThr, t.smem, s>>>(p, t.TX, t.heads, t.chunks, t.tiles);
  return cudaGetLastError();
}

template <typename T> cudaError_t fwd_t(const QkParams &p, cudaStream_t s) {
  int nb;
  if (p.time_last) return time_run<T, false>(p, &nb, s);
  RowPlan r;
  return rows_run<T, T, false>(p, &r, s);
}

template <typename T> cudaError_t bwd_t(const QkParams &p, cudaStream_t s) {
  const bool sums = p.dw[0] || p.dw[1];
  const dim3 grid((unsigned)((p.D + 31) / 32), 2);
  if (p.time_last) {
    int nb;
    const cudaError_t e = time_run<T, true>(p, &nb, s);
    if (e != cudaSuccess || !sums) return e;
    qk_dw_kernel<<<grid, 1024, 0, s>>>(p, nb, 1, nb, 2);
  } else {
    RowPlan r;
    const cudaError_t e = p.dout[p.H[0] == 0].bf16 ? rows_run<T, __nv_bfloat16, true>(p, &r, s) : rows_run<T, float, true>(p, &r, s);
    if (e != cudaSuccess || !sums) return e;
    qk_dw_kernel<<<grid, 1024, 0, s>>>(p, r.nb0, r.nb0, r.nb - r.nb0, 1);
  }
  return cudaGetLastError();
}

}  // namespace

// Whatever the plan: at most kBwdCtas shares, one more where a side rounds up from none; two from each of 2 * 148 CTAs with
// time innermost.
size_t qk_bwd_workspace_bytes(const QkParams &p) {
  return p.dw[0] || p.dw[1] ? sizeof(float) * (size_t)(4 * 148) * (size_t)p.D : 0;
}
static_assert(kBwdCtas + 2 <= 4 * 148 && 2 * 148 <= kBwdCtas, "the workspace and the reduction hold every plan's shares");

cudaError_t launch_qk_fwd(const QkParams &p, int in_bf16, cudaStream_t s) {
  return in_bf16 ? fwd_t<__nv_bfloat16>(p, s) : fwd_t<float>(p, s);
}
cudaError_t launch_qk_bwd(const QkParams &p, int in_bf16, cudaStream_t s) {
  return in_bf16 ? bwd_t<__nv_bfloat16>(p, s) : bwd_t<float>(p, s);
}

}  // namespace ssm
