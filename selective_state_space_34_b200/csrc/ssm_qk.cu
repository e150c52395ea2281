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
// its squares by shuffles. Where runs start at multiples of 4 or 2 elements only, they travel in 8- or 4-byte pieces of the same
// units; odd head sizes take units of one pair. A group of lanes walks the heads of a token, for their common angles.
//
// Time innermost (time_last): a warp owns 32 consecutive steps of 8 or 16 pairs and walks the heads on one set of cosines and
// sines; a step's squares meet by shuffles, and across the warps of a larger head through shared memory.
//
// Angles. In 32 bits position * inv_freq loses the angle of a far position (at 10^6 the spacing is 1/16 of
// a radian). A frequency is kept as turns per position in units of 2^-64, so that the product with the position modulo 2^64 is
// the reduced angle, exact but for the frequency's roundings in 64 bits (an angle of x radians is off by x 2^-52 at most); the upper 32
// bits of that (rounded down: 1.5e-9 radians), in fp32, go through the hardware sine (absolute error 2^-21) for bf16, sincospif for fp32
// inputs.
//
// What bounds it. HBM by its bytes; in fact issue and the latency of a row's chain together (60% and 56% of the slots, 13 a element
// forwards and 23 backwards, of which the angles are 1 to 6 by the number of heads that share them). 2 x 4096 tokens x 40 heads x 128,
// bf16: forward and backward 88 us (4.8 TB/s for both calls' bytes), with direct loads of four rows a step 176 us. Time innermost,
// 8 x 65536 steps x 16 components, queries and keys, bf16 gradients, forward and backward: 62 us (fp32 gradients 71, without the ring, from L1,
// 116); 4 x 8192 steps x 3 heads of 128: 55 us (59, and by one warp for all pairs, in two passes from L1, 126).
#include <type_traits>

#include "ssm_internal.h"
#include "ssm_vec.cuh"

namespace ssm {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThr = 256;                 // threads per CTA
constexpr int kCtas = 148 * 2;            // most CTAs of a backward (each keeps a share of dw) and of a rows forward
constexpr double kInvTwoPi = 0.15915494309189533577;

__device__ __forceinline__ void st1(void *p, int bf16, int64_t i, float v) {
  if (bf16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<float *>(p)[i] = v;
}
// Rows in use and asked for ahead, per group of lanes (2 to 4 measured within 3% of each other).
template <typename T, typename Td, bool BWD> constexpr int kRowStages = BWD ? (sizeof(T) + sizeof(Td) <= 4 ? 4 : 3) : (sizeof(T) == 2 ? 4 : 3);

// Of token b L + t.
__device__ __forceinline__ int64_t position(const QkParams &p, int64_t token, int64_t t) {
  if (!p.pos) return p.pos0 + t;
  return p.pos_i64 ? static_cast<const int64_t *>(p.pos)[token] : (int64_t)static_cast<const int32_t *>(p.pos)[token];
}
// Turns per position of a pair, in units of 2^-64 turns modulo 1, and the factor on its cosine and sine: the call's, or NaN where the
// frequency is NaN or infinite, which the integer cannot say.
struct alignas(16) Rate {
  uint64_t turns;
  float scale;
};
__device__ __forceinline__ Rate rate_of(const QkParams &p, int j) {
  const double f = kInvTwoPi *
                   (p.freq_f64 ? static_cast<const double *>(p.inv_freq)[j] : (double)static_cast<const float *>(p.inv_freq)[j]);
  if (!isfinite(f)) return {0, __int_as_float(0x7fffffff)};
  return {(uint64_t)((f - floor(f)) * 18446744073709551616.0), p.rot_scale};
}
// Cosine and sine of pos turns of a pair, times the factor. The product modulo 2^64 is the angle's fraction of a turn, whatever the
// position and its sign.
template <bool PRECISE> __device__ __forceinline__ void turn(int64_t pos, const Rate &r, float &c, float &s) {
  const float frac = (float)(int32_t)(((uint64_t)pos * r.turns) >> 32);  // in 2^-32 turns, from -1/2 to 1/2
  if (PRECISE) {
    sincospif(frac * 0x1p-31f, &s, &c);
  } else {
    const float x = frac * (6.283185307179586f * 0x1p-32f);
    c = __cosf(x);
    s = __sinf(x);
  }
  c *= r.scale;
  s *= r.scale;
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
// Back to the order of memory: the first run, then the second.
template <bool INTER> __device__ __forceinline__ void in_order(const float2 *f, const float2 *s, float *v) {
#pragma unroll
  for (int j = 0; j < 4; j++) {
    v[INTER ? 4 * j : 2 * j] = f[j].x;
    v[INTER ? 4 * j + 2 : 2 * j + 1] = f[j].y;
    v[INTER ? 4 * j + 1 : 8 + 2 * j] = s[j].x;
    v[INTER ? 4 * j + 3 : 8 + 2 * j + 1] = s[j].y;
  }
}
// The first n of 8 elements in pieces of V.
template <typename T, int V> __device__ __forceinline__ void store_pieces(T *p, const float *v, int n) {
  if constexpr (V == 8) {
    if (n == 8) st8(p, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; e += V) {
      if (e >= n) break;
      if constexpr (V == 1) {
        p[e] = from_f32<T>(v[e]);
      } else if constexpr (sizeof(T) == 2) {
        uint32_t w[V / 2];
#pragma unroll
        for (int j = 0; j < V / 2; j++) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(v[e + 2 * j], v[e + 2 * j + 1]);
          w[j] = *reinterpret_cast<const uint32_t *>(&h);
        }
        if constexpr (V == 4) *reinterpret_cast<uint2 *>(p + e) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t *>(p + e) = w[0];
      } else {
        if constexpr (V == 4) *reinterpret_cast<float4 *>(p + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        else *reinterpret_cast<float2 *>(p + e) = make_float2(v[e], v[e + 1]);
      }
    }
  }
}
// N bytes on their way to shared memory.
// The first n (2 or 4) bytes of a 4-byte word, 0 in the others.
__device__ __forceinline__ void cp_async_part(void *dst, const void *src, int n) {
  const uint32_t s = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(s), "l"(src), "r"(n) : "memory");
}
template <int N> __device__ __forceinline__ void cp_async_piece(void *dst, const void *src) {
  if constexpr (N == 16) {
    cp_async16(dst, src);
  } else {
    const uint32_t s = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(s), "l"(src), "n"(N) : "memory");
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

// Rows (b, t, h) of one side, heads fastest, walked one by one.
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
// A lane's place in one tensor along a walk, moved by additions alone: to the next head, past the last head of a token, past
// the last token of a batch element.
struct Place {
  int64_t at, step, wrap, turn;
  __device__ __forceinline__ Place(const QkTensor &x, const Walk &w, int64_t b, int H, int L, int o) {
    at = b * x.sb + w.t * x.sr + w.h * x.sh + o;
    step = x.sh;
    wrap = x.sr - H * x.sh;
    turn = x.sb - L * x.sr;
  }
};
// One row on; true where the token changed.
template <typename... P> __device__ __forceinline__ bool advance(Walk &w, int H, int L, P &...places) {
  ((places.at += places.step), ...);
  if (++w.h < H) return false;
  w.h = 0;
  w.token++;
  ((places.at += places.wrap), ...);
  if (++w.t == L) {
    w.t = 0;
    ((places.at += places.turn), ...);
  }
  return true;
}
// Sums over the G lanes of a row.
template <typename... F> __device__ __forceinline__ void sum_lanes(int G, F &...v) {
  if (G == 8) {  // heads of 65 to 128 elements, mostly
#pragma unroll
    for (int off = 4; off >= 1; off >>= 1) ((v += __shfl_xor_sync(kFull, v, off)), ...);
  } else {
    for (int off = G / 2; off >= 1; off >>= 1) ((v += __shfl_xor_sync(kFull, v, off)), ...);
  }
}

// Rows in runs that start at multiples of V elements. CTAs [0, nb0) take the queries, the others the keys; G lanes take `per`
// consecutive rows of their side, one at a time, a unit of up to 16 elements each, and the rows ahead
// travel in a ring of cp.async slots that every lane fills, in pieces of V elements, and reads alone. Cosines and sines are
// recomputed where the token changes; pairs that are not rotated keep 1 and 0. The backward adds its share of dw over all its
// rows.
template <typename T, typename Td, bool BWD, bool INTER, int V>
__global__ void __launch_bounds__(kThr, 2)
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
  const int64_t total = p.Bt * p.L * H, first = ((int64_t)block * (kThr / 32) + (threadIdx.x >> 5)) * step * per;
  auto rows_from = [&](int64_t row) { return (int)(row >= total ? 0 : total - row < per ? total - row : per); };
  const int n_steps = rows_from(first), n_rows = rows_from(first + grp * per);  // of the warp, of this group
  // unit u: two runs, of n1 elements at o1 and n2 at o2. Half layout: the first and the second members of 8 pairs (fewer in the
  // last such unit), then 16 elements a unit behind the rotated part; interleaved: 16 elements a unit.
  const int ur = (p.rot / 2 + 7) / 8, half_rot = p.rot / 2;
  auto unit = [&](int u, int &o1, int &o2, int &n1, int &n2) {
    if (!INTER && u < ur) {
      o1 = 8 * u;
      o2 = half_rot + o1;
      n1 = n2 = min(8, half_rot - o1);
    } else {
      o1 = INTER ? 16 * u : p.rot + 16 * (u - ur);
      o2 = o1 + 8;
      n1 = max(0, min(8, p.D - o1));
      n2 = max(0, min(8, p.D - o2));
    }
  };
  int o1, o2, n1, n2;
  unit(sub, o1, o2, n1, n2);
  const bool on = n1 > 0, rot = sub < ur;
  const int turned = half_rot - 8 * sub;  // rotated pairs of the unit
  constexpr bool kAll = !INTER && V == 8;  // all 8 of a rotated unit (the half layout's run starts are then multiples of 8)
  // in shared memory, by unit: the weights of its pairs' members, and its pairs' turns per position
  __shared__ float4 sw[4][32];
  __shared__ Rate sf[8][32];
  for (int j = threadIdx.x; j < 16 * G; j += kThr) {  // lanes without a unit read weights too: 1, which their zeros stay 0 with
    const int u = j >> 4, e = j & 15;
    int a1, a2, m1, m2;
    unit(u, a1, a2, m1, m2);
    const int at = e < 8 ? a1 + e : a2 + e - 8;
    const bool has = p.norm && p.w[side] && (e < 8 ? e < m1 : e - 8 < m2);
    const int k = INTER ? (e & 1) * 8 + e / 2 : e;  // first members of the 8 pairs, then second ones
    reinterpret_cast<float *>(&sw[k >> 2][u])[k & 3] = has ? p.w[side][at] : 1.f;
  }
  for (int j = threadIdx.x; j < p.rot / 2; j += kThr) sf[j & 7][j >> 3] = rate_of(p, j);
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
  if (n1 < 8 || n2 < 8) {  // what a unit lacks is 0 throughout
#pragma unroll
    for (int j = 0; j < S; j++) clear(j);
  }
  const bool reads_v = !BWD || p.norm;
  const int gap = o2 - o1;
  // n elements at src into the slots from k on
  auto copy = [&](int stage, int k, const auto *src, int n) {
    constexpr int es = sizeof(*src), bytes = V * es < 16 ? V * es : 16;
#pragma unroll
    for (int j = 0; j < 8 * es / bytes; j++)
      if (V == 8 ? n == 8 : j * (bytes / es) < n)
        cp_async_piece<bytes>(slot(stage, k + j * bytes / 16) + j * bytes % 16, reinterpret_cast<const char *>(src) + j * bytes);
  };
  Walk ahead, now;
  int64_t b0;
  ahead.start(first + grp * per, H, L, b0);
  now = ahead;
  Place from(in, ahead, b0, H, L, o1), dfrom(dout, ahead, b0, H, L, o1), to(out, now, b0, H, L, o1);
  int left = n_rows;  // rows still to be asked for
  auto fetch = [&](int stage) {
    if (left > 0) {
      if (reads_v) {
        const T *a = static_cast<const T *>(in.p) + from.at;
        copy(stage, 0, a, n1);
        copy(stage, kSlotsV / 2, a + gap, n2);
      }
      if (BWD) {
        const Td *a = static_cast<const Td *>(dout.p) + dfrom.at;
        copy(stage, kSlotsV, a, n1);
        copy(stage, kSlotsV + kSlotsG / 2, a + gap, n2);
      }
      left--;
      if (BWD) advance(ahead, H, L, from, dfrom);
      else advance(ahead, H, L, from);
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
  auto store = [&](const float2 *f, const float2 *s) {
    float v[16];
    in_order<INTER>(f, s, v);
    if (out.bf16) {
      __nv_bfloat16 *q = static_cast<__nv_bfloat16 *>(out.p) + to.at;
      store_pieces<__nv_bfloat16, V>(q, v, n1);
      store_pieces<__nv_bfloat16, V>(q + gap, v + 8, n2);
    } else {
      float *q = static_cast<float *>(out.p) + to.at;
      store_pieces<float, V>(q, v, n1);
      store_pieces<float, V>(q + gap, v + 8, n2);
    }
  };
  // given positions: the next token's is loaded when a token begins
  const bool known = p.pos && rot;
  int64_t coming = known && n_rows ? position(p, now.token, now.t) : 0;
  __syncthreads();
  int stage = 0;
  bool fresh = true;
  for (int i = 0; i < n_steps; i++) {
    const bool live = i < n_rows;
    fetch(stage == 0 ? S - 1 : stage - 1);
    if (fresh && rot && live) {
      const int64_t pos = known ? coming : position(p, now.token, now.t);
      if (known) {
        const int64_t token = min(now.token + 1, p.Bt * p.L - 1);
        coming = position(p, token, 0);
      }
#pragma unroll
      for (int j = 0; j < 4; j++) {
        if (kAll || 2 * j < turned) turn<PRECISE>(pos, sf[2 * j][sub], c[j].x, s[j].x);
        if (kAll || 2 * j + 1 < turned) turn<PRECISE>(pos, sf[2 * j + 1][sub], c[j].y, s[j].y);
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
        const float2 k2 = splat(-(sc * sc * dot * p.inv_D) * sc), sc2 = splat(sc);
#pragma unroll
        for (int j = 0; j < 4; j++) {
          d1[j] = fma2(mul2(g1[j], sc2), v1[j], d1[j]);
          d2[j] = fma2(mul2(g2[j], sc2), v2[j], d2[j]);
          g1[j] = fma2(v1[j], k2, mul2(gw1[j], sc2));
          g2[j] = fma2(v2[j], k2, mul2(gw2[j], sc2));
        }
      }
      if (out.p && on && live) store(g1, g2);
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
      if (on && live) store(v1, v2);
    }
    stage = stage == S - 1 ? 0 : stage + 1;
    fresh = advance(now, H, L, to);
  }
  if constexpr (!BWD) return;
  if (!p.dw[side]) return;
  // the block's share of dw: the groups' in their order
  cp_async_wait<0>();
  __syncthreads();
  float *const sums = reinterpret_cast<float *>(smem);
  float v[16];
  in_order<INTER>(d1, d2, v);
  float *row = sums + (threadIdx.x / G) * p.D;
#pragma unroll
  for (int e = 0; e < 8; e++) {
    if (e < n1) row[o1 + e] = v[e];
    if (e < n2) row[o2 + e] = v[8 + e];
  }
  __syncthreads();
  for (int j = threadIdx.x; j < p.D; j += kThr) {
    float t = 0.f;
    for (int r = 0; r < kThr / G; r++) t += sums[r * p.D + j];
    p.part[(int64_t)blockIdx.x * p.D + j] = t;
  }
}

// What is left (odd head sizes, bf16 tensors off the 4-byte boundary, more units than lanes), over the same walk: units of one
// pair, NU a lane, the next row's loaded into registers while a row is worked on.
template <typename T, typename Td, bool BWD, int NU>
__global__ void __launch_bounds__(kThr, NU == 8 ? 1 : BWD ? 2 : 3)
qk_pairs_kernel(const __grid_constant__ QkParams p, int G, int nb0, int64_t per0, int64_t per1) {
  constexpr bool PRECISE = sizeof(T) == 4;
  extern __shared__ float sdw[];  // (groups, D) sums of dw
  const int side = (int)blockIdx.x >= nb0;
  const int block = side ? blockIdx.x - nb0 : blockIdx.x;
  const int lane = threadIdx.x & 31, sub = lane & (G - 1), grp = lane / G, step = 32 / G;
  const int64_t per = side ? per1 : per0;
  const int H = p.H[side], L = (int)p.L;
  const QkTensor in = p.in[side], dout = p.dout[side], out = p.out[side];
  const int64_t total = p.Bt * p.L * H, first = ((int64_t)block * (kThr / 32) + (threadIdx.x >> 5)) * step * per;
  auto rows_from = [&](int64_t row) { return (int)(row >= total ? 0 : total - row < per ? total - row : per); };
  const int n_steps = rows_from(first), n_rows = rows_from(first + grp * per);  // of the warp, of this group
  const bool reads_v = !BWD || p.norm;
  // the lane's units: first run, distance to the second (0: none, at an odd end), weights, sums of dw
  int o[NU], gap[NU];
  bool on[NU], rot[NU];
  float w[NU][2], dw[NU][2], c[NU], s[NU];
#pragma unroll
  for (int n = 0; n < NU; n++) {
    const Unit u = unit_of(p, sub + n * G);
    on[n] = u.on;
    rot[n] = u.rot;
    o[n] = u.o1;
    gap[n] = u.o2 < p.D ? u.o2 - u.o1 : 0;
    w[n][0] = w[n][1] = c[n] = 1.f;
    dw[n][0] = dw[n][1] = s[n] = 0.f;
    if (p.norm && p.w[side] && on[n]) {
      w[n][0] = p.w[side][u.o1];
      if (gap[n]) w[n][1] = p.w[side][u.o2];
    }
  }
  Walk ahead, now;
  int64_t b0;
  ahead.start(first + grp * per, H, L, b0);
  now = ahead;
  Place from(in, ahead, b0, H, L, 0), dfrom(dout, ahead, b0, H, L, 0), to(out, now, b0, H, L, 0);
  T nv[NU][2];
  Td ng[NU][2];
  int left = n_rows;  // rows still to be asked for
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
    left--;
    if (BWD) advance(ahead, H, L, from, dfrom);
    else advance(ahead, H, L, from);
  };
  fetch();
  bool fresh = true;
  for (int i = 0; i < n_steps; i++) {
    const bool live = i < n_rows;
    float v[NU][2], g[NU][2];
#pragma unroll
    for (int n = 0; n < NU; n++)
#pragma unroll
      for (int r = 0; r < 2; r++) {
        v[n][r] = to_f32(nv[n][r]);
        if (BWD) g[n][r] = to_f32(ng[n][r]);
      }
    fetch();
    if (fresh && live && p.rot) {
      const int64_t pos = position(p, now.token, now.t);
#pragma unroll
      for (int n = 0; n < NU; n++)
        if (rot[n]) turn<PRECISE>(pos, rate_of(p, sub + n * G), c[n], s[n]);
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
    fresh = advance(now, H, L, to);
  }
  if constexpr (BWD) {
    if (!p.dw[side]) return;
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
}

// ---- time innermost ----------------------------------------------------------------------------

// The first m of 8 elements at i (m a multiple of V), in pieces of V elements.
__device__ __forceinline__ void put_run(void *p, int bf16, int64_t i, int m, int V, const float *v) {
  auto put = [&](auto *q) {
    using E = std::remove_reference_t<decltype(*q)>;
    if (V == 8 && m == 8) st8(q, v);
    else if (V >= 4) store_pieces<E, 4>(q, v, m);
    else if (V == 2) store_pieces<E, 2>(q, v, m);
    else store_pieces<E, 1>(q, v, m);
  };
  if (bf16) put(static_cast<__nv_bfloat16 *>(p) + i);
  else put(static_cast<float *>(p) + i);
}
// Sums of 8 values over the 8 lanes of a warp that share bits 0 and 1 of their number, every lane ending with the sum of one
// value (7 exchanges in place of 24).
__device__ __forceinline__ float scatter_sum(int lane, const float2 *f) {
  const float v[8] = {f[0].x, f[0].y, f[1].x, f[1].y, f[2].x, f[2].y, f[3].x, f[3].y};
  float a[4], b[2];
  const bool h4 = lane & 16, h2 = lane & 8, h1 = lane & 4;
#pragma unroll
  for (int e = 0; e < 4; e++) a[e] = (h4 ? v[e + 4] : v[e]) + __shfl_xor_sync(kFull, h4 ? v[e] : v[e + 4], 16);
#pragma unroll
  for (int e = 0; e < 2; e++) b[e] = (h2 ? a[e + 2] : a[e]) + __shfl_xor_sync(kFull, h2 ? a[e] : a[e + 2], 8);
  return (h1 ? b[1] : b[0]) + __shfl_xor_sync(kFull, h1 ? b[0] : b[1], 4);
}
// W warps take 32 steps of one batch element for a chunk of its heads (queries, then keys), each warp 8 NP of the pairs, 4 lanes
// of 8 consecutive steps by 8 lanes of NP pairs. A pair unit is elements o1 and o2 (or o1 alone at an odd end). The
// runs of the heads ahead travel in a ring of cp.async slots that every lane fills (in pieces of as many elements as the rows'
// starts are multiples of) and reads alone. A lane keeps its pairs' cosines and sines for all heads of its steps; a step's squares
// meet by shuffles, and those of W > 1 warps through shared memory, with one barrier of theirs a head.
// Single bf16 elements have no copy of their own: a run off the 4-byte boundary travels as the five words around it, of which the
// first and last are copied only as far as the row goes; the fifth words have slots of their own.
template <typename T, typename Td, bool BWD, int NP, bool FULL> struct TimeRing {
  static constexpr int kV = sizeof(T) / 2, kG = BWD ? sizeof(Td) / 2 : 0;  // 16-byte slots of a run of 8
  static constexpr int kRuns = 2 * NP * (kV + kG), kFifth = FULL ? 0 : 2 * NP * ((kV == 1) + (kG == 1));
  static constexpr int kSlots = kRuns + (kFifth + 3) / 4, kStageBytes = kSlots * 512;  // of a lane; of a warp
  static constexpr int S = kStageBytes <= 3 << 10 ? 4 : kStageBytes <= 4 << 10 ? 3 : kStageBytes <= 6 << 10 ? 2 : 1;
  static constexpr int kWarpBytes = S * kStageBytes;  // 12 KB at most
  static constexpr int kMost = NP == 2 ? kThr / 16 : kThr / 32;  // most warps of a CTA
  // The most dynamic shared memory of a launch: rings and sums of dw. W warps hold D <= 16 NP W elements, so that the kMost / W groups'
  // 8 D bytes each are 128 NP a warp at most.
  static constexpr int kMostBytes = kMost * (kWarpBytes + 128 * NP);
  static constexpr int kStatic = kMost * 32 * (BWD ? 2 : 1) * 3 * 4 + kMost * (32 + 16 * NP) * 8;  // the kernel's own arrays
  static_assert(kMostBytes + kStatic <= 227 << 10, "more shared memory than an SM gives a CTA");
};
// How the steps are cut: warps a slice of 32, its heads at a time, their chunks, slices of a batch element; and the batch
// elements, chunks and slices from one item of a group of warps to its next.
struct TimePlan {
  int W, heads, chunks, per_row, dchunk, dtt;
  int64_t db;
};
template <typename T, typename Td, bool BWD, int NP, bool FULL>
__global__ void __launch_bounds__(NP == 2 ? 2 * kThr : kThr, NP == 2 ? 1 : BWD || !FULL ? 2 : 3)
qk_time_ring_kernel(const __grid_constant__ QkParams p, const __grid_constant__ TimePlan plan) {
  const int W = plan.W;
  constexpr bool PRECISE = sizeof(T) == 4;
  using Ring = TimeRing<T, Td, BWD, NP, FULL>;
  constexpr int S = Ring::S, kV = Ring::kV, kG = Ring::kG, kMost = Ring::kMost;
  extern __shared__ __align__(16) char smem[];  // the ring, then (groups, 2, D) sums of dw
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tl = lane & 3, pl = lane >> 2;
  const int all = p.H[0] + p.H[1];
  const bool sums = BWD && p.norm && (p.dw[0] || p.dw[1]), reads_v = !BWD || p.norm;
  const int groups = blockDim.x / 32 / W, group = warp / W, first = group * W;  // warps left over have no group
  float *const sdw = reinterpret_cast<float *>(smem + blockDim.x / 32 * Ring::kWarpBytes);
  float acc[2][NP][2];  // this lane's share of dw, by side
#pragma unroll
  for (int n = 0; n < NP; n++) acc[0][n][0] = acc[0][n][1] = acc[1][n][0] = acc[1][n][1] = 0.f;
  __shared__ float shares[2][kMost][BWD ? 2 : 1][32];  // the warps' sums of each step, for this head and the one before
  __shared__ int64_t positions[kMost][32];
  __shared__ __align__(16) float factors[kMost][BWD ? 2 : 1][32];
  char *const base = smem + warp * Ring::kWarpBytes + lane * 16;
  auto slot = [&](int stage, int k) { return base + (stage * Ring::kSlots + k) * 512; };
  Unit u[NP];
#pragma unroll
  for (int n = 0; n < NP; n++) u[n] = unit_of(p, pl + 8 * (warp - first + n * W));
#pragma unroll
  for (int k = 0; k < S * Ring::kSlots; k++) *reinterpret_cast<uint4 *>(slot(0, k)) = make_uint4(0, 0, 0, 0);
  const int own = 8 * tl + (lane >> 4 & 1) * 4 + (lane >> 3 & 1) * 2 + (lane >> 2 & 1);  // the step whose sum this lane ends with
  // one head of one item at a time; items are numbered batch element, chunk of heads, slice of 32 steps, the last fastest
  struct Job {
    int64_t b, t0;  // t0: of the warps
    int tt, chunk, h, h_end;
    bool on;
  };
  auto open = [&](Job &j) {
    j.on = j.b < p.Bt;
    j.t0 = (int64_t)j.tt * 32;
    j.h = j.chunk * plan.heads;
    j.h_end = min(all, j.h + plan.heads);
  };
  auto next_item = [&](Job &j) {
    j.tt += plan.dtt;
    j.chunk += plan.dchunk;
    j.b += plan.db;
    if (j.tt >= plan.per_row) {
      j.tt -= plan.per_row;
      j.chunk++;
    }
    if (j.chunk >= plan.chunks) {
      j.chunk -= plan.chunks;
      j.b++;
    }
    open(j);
  };
  auto next = [&](Job &j) {
    if (++j.h < j.h_end) return false;
    next_item(j);
    return true;
  };
  Job ahead;
  int64_t bc, left;
  divide((int64_t)blockIdx.x * groups + group, plan.per_row, bc, left);
  ahead.tt = (int)left;
  divide(bc, plan.chunks, ahead.b, left);
  ahead.chunk = (int)left;
  if (group >= groups) ahead.b = p.Bt;
  open(ahead);
  Job now = ahead;
  const int V = p.vec;
  constexpr int kFifthG = kV == 1 ? 2 * NP : 0;  // the gradients' first
  auto fifth = [&](int stage, int run) { return reinterpret_cast<uint32_t *>(slot(stage, Ring::kRuns + run / 4) + run % 4 * 4); };
  // the m live ones (a multiple of V) of 8 steps of one row into the slots from k on, in pieces of V elements, 0 behind them;
  // run: its fifth word; begin: of the row
  auto copy = [&](int stage, int k, int run, const auto *src, int m, bool begin) {
    using E = std::remove_cv_t<std::remove_reference_t<decltype(*src)>>;
    constexpr int es = sizeof(E);
    const char *from = reinterpret_cast<const char *>(src);
    auto piece = [&](auto n, int at) {  // n bytes at byte `at` of the run
      cp_async_piece<decltype(n)::value>(slot(stage, k + at / 16) + at % 16, from + at);
    };
    if constexpr (FULL) {
#pragma unroll
      for (int j = 0; j < 8 * es; j += 16) {
        if (m) cp_async_piece<16>(slot(stage, k + j / 16), from + j);
        else *reinterpret_cast<uint4 *>(slot(stage, k + j / 16)) = make_uint4(0, 0, 0, 0);
      }
      return;
    }
    if (es == 2 && V == 1) {
      const int odd = (int)(reinterpret_cast<uintptr_t>(src) >> 1 & 1);
#pragma unroll
      for (int j = 0; j < 5; j++) {  // elements 2 j - odd and the one behind it
        uint32_t *const to = j < 4 ? reinterpret_cast<uint32_t *>(slot(stage, k)) + j : fifth(stage, run);
        const int n = m ? min(2, m - 2 * j + odd) : 0;
        if (j == 0 && odd && begin) *to = m ? (uint32_t)*reinterpret_cast<const uint16_t *>(src) << 16 : 0;
        else if (n > 0) cp_async_part(to, from + 4 * j - 2 * odd, 2 * n);
        else *to = 0;
      }
      return;
    }
    if (V == 8 && m == 8) {
#pragma unroll
      for (int j = 0; j < 8 * es; j += 16) piece(std::integral_constant<int, 16>(), j);
      return;
    }
    if (m < 8) {  // the pieces behind the live ones; a piece is written here or by a copy, not by both
#pragma unroll
      for (int j = 0; j < 8; j++)
        if (j >= m) *reinterpret_cast<E *>(slot(stage, k + j * es / 16) + j * es % 16) = from_f32<E>(0.f);
    }
    if (V >= 4) {
#pragma unroll
      for (int j = 0; j < 8; j += 4)
        if (j < m) piece(std::integral_constant<int, 4 * es>(), j * es);
    } else if (V == 2) {
#pragma unroll
      for (int j = 0; j < 8; j += 2)
        if (j < m) piece(std::integral_constant<int, 2 * es>(), j * es);
    } else if (es == 4) {
#pragma unroll
      for (int j = 0; j < 8; j++)
        if (j < m) piece(std::integral_constant<int, 4>(), j * es);
    }
  };
  auto live = [&](const Job &j) {
    const int64_t left = p.L - j.t0 - 8 * tl;
    return (int)(left < 0 ? 0 : left < 8 ? left : 8);
  };
  auto fetch = [&](int stage) {
    if (ahead.on) {
      const int m = live(ahead), sd = ahead.h >= p.H[0], h = ahead.h - (sd ? p.H[0] : 0);
      const int64_t t = ahead.t0 + 8 * tl;
#pragma unroll
      for (int n = 0; n < NP; n++) {
        if (!u[n].on) continue;
        const bool two = u[n].o2 < p.D;
        if (reads_v) {
          const QkTensor &x = p.in[sd];
          const T *a = static_cast<const T *>(x.p) + ahead.b * x.sb + h * x.sh + t;
          copy(stage, 2 * n * kV, 2 * n, a + u[n].o1 * x.sr, m, t == 0);
          if (two) copy(stage, (2 * n + 1) * kV, 2 * n + 1, a + u[n].o2 * x.sr, m, t == 0);
        }
        if (BWD) {
          const QkTensor &x = p.dout[sd];
          const Td *a = static_cast<const Td *>(x.p) + ahead.b * x.sb + h * x.sh + t;
          copy(stage, 2 * NP * kV + 2 * n * kG, kFifthG + 2 * n, a + u[n].o1 * x.sr, m, t == 0);
          if (two) copy(stage, 2 * NP * kV + (2 * n + 1) * kG, kFifthG + 2 * n + 1, a + u[n].o2 * x.sr, m, t == 0);
        }
      }
      next(ahead);
    }
    cp_async_commit();
  };
  // a run of row o of x
  auto take = [&](int stage, int k, int run, auto tag, const QkTensor &x, int64_t head, int o, float2 *f) {
    Raw8<decltype(tag)> r;
    float v[8];
#pragma unroll
    for (int j = 0; j < (int)sizeof(tag) / 2; j++) reinterpret_cast<uint4 *>(&r)[j] = *reinterpret_cast<const uint4 *>(slot(stage, k + j));
    if constexpr (!FULL && sizeof(tag) == 2) {
      const uint32_t at = (uint32_t)(reinterpret_cast<uintptr_t>(x.p) >> 1) + (uint32_t)head + (uint32_t)o * (uint32_t)x.sr;
      if (V == 1) {
        const uint32_t by = at & 1 ? 0x5432 : 0x3210, w[5] = {r.a.x, r.a.y, r.a.z, r.a.w, *fifth(stage, run)};
        r.a = make_uint4(__byte_perm(w[0], w[1], by), __byte_perm(w[1], w[2], by), __byte_perm(w[2], w[3], by), __byte_perm(w[3], w[4], by));
      }
    }
    unpack8(r, v);
#pragma unroll
    for (int e = 0; e < 4; e++) f[e] = make_float2(v[2 * e], v[2 * e + 1]);
  };
#pragma unroll
  for (int j = 0; j < S - 1; j++) fetch(j);
  __shared__ Rate freq[kMost][NP][8];  // by pair
  float2 cs[NP][4], sn[NP][4];
#pragma unroll
  for (int n = 0; n < NP; n++) {
    if (tl == 0 && u[n].on && u[n].rot) freq[warp][n][pl] = rate_of(p, pl + 8 * (warp - first + n * W));
#pragma unroll
    for (int e = 0; e < 4; e++) {
      cs[n][e] = splat(1.f);
      sn[n][e] = splat(0.f);
    }
  }
  // the m live ones of 8 results of one row at i
  auto put = [&](const QkTensor &x, int64_t i, int m, const float2 *f) {
    const float v[8] = {f[0].x, f[0].y, f[1].x, f[1].y, f[2].x, f[2].y, f[3].x, f[3].y};
    if constexpr (FULL) {
      if (!m) return;
      if (x.bf16) st8(static_cast<__nv_bfloat16 *>(x.p) + i, v);
      else st8(static_cast<float *>(x.p) + i, v);
    } else if (V == 1 && m == 8 && x.bf16) {  // three whole words, then another or the elements at both ends
      char *const to = static_cast<char *>(x.p) + 2 * i;
      const int odd = (int)(reinterpret_cast<uintptr_t>(to) >> 1 & 1);
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
        w[e] = *reinterpret_cast<const uint32_t *>(&b);
      }
#pragma unroll
      for (int e = 0; e < 3; e++) *reinterpret_cast<uint32_t *>(to + 4 * e + 2 * odd) = odd ? __byte_perm(w[e], w[e + 1], 0x5432) : w[e];
      if (odd) {
        *reinterpret_cast<uint16_t *>(to) = (uint16_t)w[0];
        *reinterpret_cast<uint16_t *>(to + 14) = (uint16_t)(w[3] >> 16);
      } else {
        *reinterpret_cast<uint32_t *>(to + 12) = w[3];
      }
    } else {
      put_run(x.p, x.bf16, i, m, V, v);
    }
  };
  // the position of this lane's step, an item ahead
  auto step_position = [&](const Job &j) {
    const int64_t t = j.t0 + lane;
    return p.rot && j.on && t < p.L ? position(p, j.b * p.L + t, t) : 0;
  };
  int64_t coming = step_position(now);
  int stage = 0, half = 0;
  bool fresh = true;
  while (now.on) {
    fetch(stage == 0 ? S - 1 : stage - 1);
    const int m = live(now), sd = now.h >= p.H[0], h = now.h - (sd ? p.H[0] : 0);
    if (fresh) {
      __syncwarp();  // the item before is done with the positions
      positions[warp][lane] = coming;
      __syncwarp();
      Job after = now;
      next_item(after);
      coming = step_position(after);
#pragma unroll
      for (int n = 0; n < NP; n++)
        if (u[n].on && u[n].rot) {
          const Rate f = freq[warp][n][pl];
#pragma unroll
          for (int e = 0; e < 4; e++) {
            turn<PRECISE>(positions[warp][8 * tl + 2 * e], f, cs[n][e].x, sn[n][e].x);
            turn<PRECISE>(positions[warp][8 * tl + 2 * e + 1], f, cs[n][e].y, sn[n][e].y);
          }
        }
    }
    cp_async_wait<S - 1>();
    const float *w = p.w[sd];
    const QkTensor &in = p.in[sd], &dout = p.dout[sd];
    const int64_t at = now.b * in.sb + h * in.sh, dat = now.b * dout.sb + h * dout.sh;
    // one pair's elements, and backwards its gradients turned back
    float2 a[4], c[4], ga[4], gc[4];
    float wa, wc;
    auto pair = [&](int n) {
      wa = w && u[n].on ? w[u[n].o1] : 1.f;
      wc = w && u[n].on && u[n].o2 < p.D ? w[u[n].o2] : 1.f;
      if (reads_v) {
        take(stage, 2 * n * kV, 2 * n, T(), in, at, u[n].o1, a);
        take(stage, (2 * n + 1) * kV, 2 * n + 1, T(), in, at, u[n].o2, c);
      }
      if constexpr (BWD) {
        take(stage, 2 * NP * kV + 2 * n * kG, kFifthG + 2 * n, Td(), dout, dat, u[n].o1, ga);
        take(stage, 2 * NP * kV + (2 * n + 1) * kG, kFifthG + 2 * n + 1, Td(), dout, dat, u[n].o2, gc);
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const float2 x = ga[e], y = gc[e];
          ga[e] = fma2(y, sn[n][e], mul2(x, cs[n][e]));
          gc[e] = fma2(x, neg2(sn[n][e]), mul2(y, cs[n][e]));
        }
      }
    };
    float2 sc[4], back[4];
#pragma unroll
    for (int e = 0; e < 4; e++) sc[e] = back[e] = splat(0.f);
    if (p.norm) {
#pragma unroll
      for (int n = 0; n < NP; n++) {
        pair(n);
#pragma unroll
        for (int e = 0; e < 4; e++) {
          sc[e] = fma2(a[e], a[e], fma2(c[e], c[e], sc[e]));
          if (BWD) back[e] = fma2(mul2(ga[e], splat(wa)), a[e], fma2(mul2(gc[e], splat(wc)), c[e], back[e]));
        }
      }
      float sum = scatter_sum(lane, sc), dot = BWD ? scatter_sum(lane, back) : 0.f;
      int step = own;  // of the 32, whose sums these are
      if (W > 1) {
        shares[half][warp][0][own] = sum;
        if (BWD) shares[half][warp][BWD ? 1 : 0][own] = dot;
        asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * W) : "memory");
        step = lane;
        sum = dot = 0.f;
#pragma unroll 4
        for (int j = first; j < first + W; j++) {
          sum += shares[half][j][0][lane];
          if (BWD) dot += shares[half][j][BWD ? 1 : 0][lane];
        }
        half ^= 1;  // written again two heads on: everyone has passed the barrier between
      }
      const float r = now.t0 + step < p.L ? inv_rms(p, sum) : 0.f;  // with an eps of 0, 1 / sqrt(0) of a step that is none
      __syncwarp();  // the head before is done with the factors
      factors[warp][0][step] = r;
      if (BWD) factors[warp][BWD ? 1 : 0][step] = -(r * r * dot * p.inv_D) * r;
      __syncwarp();
#pragma unroll
      for (int e = 0; e < 4; e++) {
        sc[e] = *reinterpret_cast<const float2 *>(&factors[warp][0][8 * tl + 2 * e]);
        if (BWD) back[e] = *reinterpret_cast<const float2 *>(&factors[warp][BWD ? 1 : 0][8 * tl + 2 * e]);
      }
    }
    const QkTensor &out = p.out[sd];
    const int64_t to = now.b * out.sb + h * out.sh + now.t0 + 8 * tl;
#pragma unroll
    for (int n = 0; n < NP; n++) {
      if (NP > 1 || !p.norm) pair(n);  // one pair is still here
      if constexpr (BWD) {
        if (p.norm) {
          float2 dx = splat(0.f), dy = splat(0.f);
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const float2 x = mul2(ga[e], sc[e]), y = mul2(gc[e], sc[e]);
            dx = fma2(x, a[e], dx);
            dy = fma2(y, c[e], dy);
            a[e] = fma2(a[e], back[e], mul2(x, splat(wa)));
            c[e] = fma2(c[e], back[e], mul2(y, splat(wc)));
          }
          acc[0][n][0] += sd ? 0.f : dx.x + dx.y;
          acc[0][n][1] += sd ? 0.f : dy.x + dy.y;
          acc[1][n][0] += sd ? dx.x + dx.y : 0.f;
          acc[1][n][1] += sd ? dy.x + dy.y : 0.f;
        } else {
#pragma unroll
          for (int e = 0; e < 4; e++) {
            a[e] = ga[e];
            c[e] = gc[e];
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const float2 x = p.norm ? mul2(a[e], mul2(sc[e], splat(wa))) : a[e], y = p.norm ? mul2(c[e], mul2(sc[e], splat(wc))) : c[e];
          a[e] = fma2(y, neg2(sn[n][e]), mul2(x, cs[n][e]));
          c[e] = fma2(x, sn[n][e], mul2(y, cs[n][e]));
        }
      }
      if (out.p && u[n].on) {
        put(out, to + u[n].o1 * out.sr, m, a);
        if (u[n].o2 < p.D) put(out, to + u[n].o2 * out.sr, m, c);
      }
    }
    stage = stage == S - 1 ? 0 : stage + 1;
    fresh = next(now);
  }
  if constexpr (BWD) {
    if (!sums) return;
    // the block's shares, rows 2 block + side: a pair's over its 4 lanes, then the groups' in their order
#pragma unroll
    for (int n = 0; n < NP; n++)
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const int sd = j >> 1, at = sd * p.D + (j & 1 ? u[n].o2 : u[n].o1);
        float v = acc[sd][n][j & 1];
        v += __shfl_xor_sync(kFull, v, 1);
        v += __shfl_xor_sync(kFull, v, 2);
        if (tl == 0 && group < groups && u[n].on && (!(j & 1) || u[n].o2 < p.D)) sdw[group * 2 * p.D + at] = v;
      }
    __syncthreads();
    for (int j = threadIdx.x; j < 2 * p.D; j += blockDim.x) {
      float t = 0.f;
      for (int g = 0; g < groups; g++) t += sdw[g * 2 * p.D + j];
      p.part[2 * (int64_t)blockIdx.x * p.D + j] = t;
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
  float v[kCtas / 32 + 1], s = 0.f;
#pragma unroll
  for (int k = 0; k < kCtas / 32 + 1; k++) {
    const int at = y + 32 * k;
    v[k] = j < p.D && at < n ? part[(int64_t)at * stride * p.D + j] : 0.f;
  }
#pragma unroll
  for (int k = 0; k < kCtas / 32 + 1; k++) s += v[k];
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

// The most elements (8, 4, 2; 1 of fp32) that every run of a row starts at multiples of, and the addresses and strides of both
// sides are (those of axes that are stepped along: one of length 1 may have any); 0 where a row does not make such runs or more units
// than a warp has lanes.
int run_of(const QkParams &p) {
  const int units = p.interleaved ? (p.D + 15) / 16 : (p.rot / 2 + 7) / 8 + (p.D - p.rot + 15) / 16;
  if (units > 32) return 0;
  bool wide = true;  // fp32 throughout: single elements travel as 4 bytes
  for (int s = 0; s < 2; s++)
    if (p.H[s])
      for (const QkTensor *t : {&p.in[s], &p.dout[s]})
        if (t->bf16) wide = false;  // (of a tensor that is not read too: the kernel's type goes by it)
  for (int V = 8; V >= (wide ? 1 : 2); V /= 2) {
    bool fits = p.D % V == 0 && (p.interleaved || (p.rot / 2 % V == 0 && p.rot % V == 0));
    for (int s = 0; s < 2 && fits; s++) {
      if (p.H[s] == 0) continue;
      for (const QkTensor *t : {&p.in[s], &p.out[s], &p.dout[s]}) {
        const int bytes = V * (t->bf16 ? 2 : 4) < 16 ? V * (t->bf16 ? 2 : 4) : 16;
        if (t->p && (reinterpret_cast<uintptr_t>(t->p) % bytes || (p.Bt > 1 && t->sb % V) || (p.H[s] > 1 && t->sh % V) ||
                     (p.L > 1 && t->sr % V)))
          fits = false;
      }
    }
    if (fits) return V;
  }
  return 0;
}
// Lanes that hold a row: a unit each, or four pairs (eight of the largest heads).
int lanes_per_row(const QkParams &p, int V) {
  const int pairs = pairs_of(p), per = pairs <= 128 ? 4 : 8;
  if (!V) return pow2_at_least((pairs + per - 1) / per);
  return pow2_at_least(p.interleaved ? (p.D + 15) / 16 : (p.rot / 2 + 7) / 8 + (p.D - p.rot + 15) / 16);
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

// How the rows of both sides are cut: CTAs of the queries and of both, rows per group of G lanes: whole tokens where
// that adds a quarter at most, so that the groups of a warp need their angles at the same steps (2 x 4096 tokens x 40 heads of 128,
// forward and backward: 88 us so, 95 without); not where rows are copied element by element (fp32, 24 x 197 x 7 heads of 192
// with 126 turned: 36 us so, 29 without).
struct RowPlan {
  int V, G, nb0, nb;
  int64_t per[2];
};
bool plan_rows(const QkParams &p, bool bwd, RowPlan *r) {
  constexpr int kWarps = kThr / 32;
  r->V = run_of(p);
  r->G = lanes_per_row(p, r->V);
  const int64_t most = bwd || r->V ? kCtas : 3 * 148;
  const int step = 32 / r->G;
  int64_t rows[2], work[2];
  int n[2];
  for (int j = 0; j < 2; j++) {
    rows[j] = p.Bt * p.L * p.H[j];
    work[j] = (rows[j] + kWarps * step - 1) / (kWarps * step);
  }
  split_blocks(work, most, &n[0], &n[1]);
  for (int j = 0; j < 2; j++) {
    r->per[j] = 1;
    if (!n[j]) continue;
    const int64_t groups = (int64_t)n[j] * kWarps * step, per = (rows[j] + groups - 1) / groups;
    const int64_t whole = (per + p.H[j] - 1) / p.H[j] * p.H[j];
    r->per[j] = r->V != 1 && (whole - per) * 4 <= per ? whole : per;
    if (r->per[j] > 0x7fffff00) return false;
    n[j] = (int)((rows[j] + r->per[j] * kWarps * step - 1) / (r->per[j] * kWarps * step));
  }
  r->nb0 = n[0];
  r->nb = n[0] + n[1];
  return true;
}

// smem: the same for every call of a kernel of runs, for the limit is the kernel's and other host threads may be between setting it and
// their launch; below what needs asking for where rows go by pairs.
template <typename K> cudaError_t launch_rows(K kernel, const QkParams &p, const RowPlan &r, int smem, cudaStream_t s) {
  if (smem > 40 * 1024) {  // with the kernels' own 6 KB more than the default 48 KB
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  kernel<<<r.nb, kThr, smem, s>>>(p, r.G, r.nb0, r.per[0], r.per[1]);
  return cudaGetLastError();
}

// Head elements innermost, forward (Td = T) or backward. CTAs: what fits the SMs at once, two each, three where a
// forward goes by pairs. (Three forward CTAs of runs an SM, which leaves 80 registers and a few spills: 4 x 4096 tokens x
// one query and one key of 128, 8.5 us against 7.7; 2 x 4096 x 40 of 128 alike.)
template <typename T, typename Td, bool BWD> cudaError_t rows_run(const QkParams &p, RowPlan *r, cudaStream_t s) {
  if (!plan_rows(p, BWD, r)) return cudaErrorInvalidConfiguration;
  const int sums = BWD && (p.dw[0] || p.dw[1]) ? (int)sizeof(float) * (kThr / r->G) * p.D : 0;
  constexpr int kSlots = sizeof(T) + (BWD ? sizeof(Td) : 0);
  constexpr int smem = kThr * 16 * kSlots * kRowStages<T, Td, BWD>;
  static_assert(smem >= kThr * 16 * 4, "G lanes hold D <= 16 G elements: the groups' sums are no more than this");
  const bool inter = p.interleaved;
  switch (r->V) {
    case 8: return launch_rows(inter ? qk_rows_kernel<T, Td, BWD, true, 8> : qk_rows_kernel<T, Td, BWD, false, 8>, p, *r, smem, s);
    case 4: return launch_rows(inter ? qk_rows_kernel<T, Td, BWD, true, 4> : qk_rows_kernel<T, Td, BWD, false, 4>, p, *r, smem, s);
    case 2: return launch_rows(inter ? qk_rows_kernel<T, Td, BWD, true, 2> : qk_rows_kernel<T, Td, BWD, false, 2>, p, *r, smem, s);
    case 1:
      if constexpr (sizeof(T) == 4 && sizeof(Td) == 4)
        return launch_rows(inter ? qk_rows_kernel<T, Td, BWD, true, 1> : qk_rows_kernel<T, Td, BWD, false, 1>, p, *r, smem, s);
  }
  return launch_rows(pairs_of(p) <= 128 ? qk_pairs_kernel<T, Td, BWD, 4> : qk_pairs_kernel<T, Td, BWD, 8>, p, *r, sums, s);
}

// Time innermost. All heads of a batch element go to one group of warps, for their common angles, where that leaves 16 warps
// per SM. CTAs: what fits the SMs at once (the backward's each keep a share of dw of both sides).
template <typename T, typename Td, bool BWD, int NP>
cudaError_t time_ring(const QkParams &p, const TimePlan &plan, int nb, int warps, int sums, cudaStream_t s) {
  const bool full = p.vec == 8 && p.L % 8 == 0;
  using Full = TimeRing<T, Td, BWD, NP, true>;
  using Part = TimeRing<T, Td, BWD, NP, false>;
  const auto kernel = full ? qk_time_ring_kernel<T, Td, BWD, NP, true> : qk_time_ring_kernel<T, Td, BWD, NP, false>;
  const int smem = warps * (full ? Full::kWarpBytes : Part::kWarpBytes) + sums;
  // The limit belongs to the kernel, not to this launch: always the same one, so that another host thread's call cannot lower it
  // between here and the launch.
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, full ? Full::kMostBytes : Part::kMostBytes);
  if (e != cudaSuccess) return e;
  kernel<<<nb, 32 * warps, smem, s>>>(p, plan);
  return cudaGetLastError();
}

template <typename T, typename Td, bool BWD> cudaError_t time_run(const QkParams &p, int *nb, cudaStream_t s) {
  const int all = p.H[0] + p.H[1], pairs = pairs_of(p);
  // one pair a lane where eight warps hold them all (4 x 8192 steps x 3 heads of 128, forward and backward: 72 us so, 108 us with two
  // pairs in half the warps), else two, in up to sixteen warps
  const int NP = pairs <= kThr / 4 ? 1 : 2, warps = pairs <= kThr / 2 ? kThr / 32 : kThr / 16;
  TimePlan t;
  t.W = (pairs + 8 * NP - 1) / (8 * NP);
  t.per_row = (int)((p.L + 31) / 32);
  const int64_t slices = p.Bt * t.per_row;
  t.heads = slices * t.W >= 16 * 148 ? all : slices * t.W * 2 >= 16 * 148 && all > 2 ? 2 : 1;
  t.chunks = (all + t.heads - 1) / t.heads;
  const int groups = warps / t.W;
  const int64_t ctas = (slices * t.chunks + groups - 1) / groups, most = BWD ? kCtas : 3 * 148;
  *nb = (int)(ctas < most ? ctas : most);
  const int64_t stride = (int64_t)*nb * groups;
  t.dtt = (int)(stride % t.per_row);
  t.dchunk = (int)(stride / t.per_row % t.chunks);
  t.db = stride / t.per_row / t.chunks;
  const int sums = BWD && (p.dw[0] || p.dw[1]) ? (int)sizeof(float) * groups * 2 * p.D : 0;
  return NP == 1 ? time_ring<T, Td, BWD, 1>(p, t, *nb, warps, sums, s) : time_ring<T, Td, BWD, 2>(p, t, *nb, warps, sums, s);
}

template <typename T> cudaError_t fwd_t(const QkParams &p, cudaStream_t s) {
  int nb;
  if (p.time_last) return time_run<T, T, false>(p, &nb, s);
  RowPlan r;
  return rows_run<T, T, false>(p, &r, s);
}

template <typename T> cudaError_t bwd_t(const QkParams &p, cudaStream_t s) {
  const bool sums = p.dw[0] || p.dw[1];
  const dim3 grid((unsigned)((p.D + 31) / 32), 2);
  if (p.time_last) {
    int nb;
    const cudaError_t e = p.dout[p.H[0] == 0].bf16 ? time_run<T, __nv_bfloat16, true>(p, &nb, s) : time_run<T, float, true>(p, &nb, s);
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

// Whatever the plan: at most kCtas shares, one more where a side rounds up from none; two from each of kCtas CTAs with
// time innermost. (qk_dw_kernel reads up to kCtas + 32 - kCtas % 32 of a side.)
size_t qk_bwd_workspace_bytes(const QkParams &p) {
  return p.dw[0] || p.dw[1] ? sizeof(float) * (size_t)(2 * kCtas + 2) * (size_t)p.D : 0;
}

cudaError_t launch_qk_fwd(const QkParams &p, int in_bf16, cudaStream_t s) {
  return in_bf16 ? fwd_t<__nv_bfloat16>(p, s) : fwd_t<float>(p, s);
}
cudaError_t launch_qk_bwd(const QkParams &p, int in_bf16, cudaStream_t s) {
  return in_bf16 ? bwd_t<__nv_bfloat16>(p, s) : bwd_t<float>(p, s);
}

}  // namespace ssm
