// ssm_lru.cu -- the gated linear recurrence: forward, backward and one-token step.
//
//   r = sigmoid(r~ + r_bias), g = sigmoid(i~ + i_bias), la = -c softplus(lam) r  (log of the decay)
//   a = e^la, m = sqrt(1 - a^2), b = m g x,  h_t = a_t h_{t-1} + b_t              (out = h)
//
// Forward. Time is innermost, so a warp takes 256 consecutive steps of one (batch, channel) row, 8 a
// lane (one 16-byte access per bf16 tensor). A lane composes its steps into one affine map
// h -> P h + H, the warp composes the 32 maps with five levels of shuffles, and the state that
// enters a lane then gives its 8 states in order. Row and state never leave the SM; every input
// is read once and every output written once. W warps share a row where rows alone do not fill the
// GPU (each takes every W-th chunk of 256, the chunks' maps meet in shared memory once per round).
//
// Alignment. Lanes work on groups of 8 elements whose flat index (row L + t) is a multiple of 8, so
// rows of any length move in 16-byte accesses: a row that starts inside a group treats the elements
// before it as identity maps (a = 1, b = 0), and so are those behind its end. Chunk k of a row
// therefore covers t in [256 k - f, 256 (k + 1) - f) with f = (row L) mod 8, whatever the
// pointers are (tensors off the 16-byte boundary take element accesses over the same groups).
//
// Backward. lambda_t = dout_t + a_{t+1} lambda_{t+1} runs from the end over the same chunks with
// mu_t = a_t (dout_t + mu_{t+1}), an affine map of what arrives from behind; the states come from the
// state that entered each chunk (saved by the forward) and a second composition. With
// rho = la / m^2 the gradient of la times la is q = lambda (la h - rho b): the a^2 / m of
// d sqrt(1 - a^2) is folded into b / m^2, which stays finite as a -> 1 (rho -> -1/2).
//   dx = lambda m g, di~ = lambda b (1 - g), dr~ = q (1 - r), dlam = sum q sigmoid(lam)/softplus(lam)
//
// Precision. The decay goes through em = e^la - 1 (a polynomial for small |la|): 1 - a^2 =
// -em (2 + em) keeps its relative precision where a is near 1, which a itself in 32 bits does not.
#include <type_traits>

#include "ssm_internal.h"
#include "ssm_vec.cuh"

namespace ssm {

namespace {

constexpr int kChunk = 256;  // steps per warp and round: 32 lanes x 8
constexpr unsigned kFull = 0xffffffffu;
constexpr int kMaxWarps = 16;

// Clamp that keeps NaN (fminf would drop it).
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float rsqrt_approx(float x) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// sigmoid(u) and sigmoid(v). Fast: both from one reciprocal, 1/((1+eu)(1+ev)); the exponents are
// held at 2^60 so that the product stays finite (a gate below 2^-60 reads 2^-60).
template <bool PRECISE>
__device__ __forceinline__ void sigmoid2(float u, float v, float &su, float &sv) {
  if (PRECISE) {
    su = sigmoid<true>(u);
    sv = sigmoid<true>(v);
  } else {
    const float pu = 1.f + ex2_approx(min_nan(-u * kLog2e, 60.f));
    const float pv = 1.f + ex2_approx(min_nan(-v * kLog2e, 60.f));
    const float inv = rcp_approx(pu * pv);
    su = pv * inv;
    sv = pu * inv;
  }
}

// a = e^y and em = e^y - 1 for y <= 0, both with relative precision: em by the Taylor polynomial of degree
// 6 where |y| < 1/4 (the next term is below y^6/5040 < 5e-8 of the sum), a by ex2 beyond (its 2^-22 of 1
// is 5e-7 of em >= 0.22 at most).
template <bool PRECISE> __device__ __forceinline__ void decay(float y, float &a, float &em) {
  if (PRECISE) {
    em = expm1f(y);
    a = y > -0.25f ? 1.f + em : expf(y);
  } else {
    const float far = ex2_approx(y * kLog2e);
    float p = fmaf(y, 1.f / 720.f, 1.f / 120.f);
    p = fmaf(y, p, 1.f / 24.f);
    p = fmaf(y, p, 1.f / 6.f);
    p = fmaf(y, p, 0.5f);
    p = y * fmaf(y, p, 1.f);
    const bool near = y > -0.25f;
    em = near ? p : far - 1.f;
    a = near ? 1.f + p : far;
  }
}

// 1 / sqrt(s) of s = 1 - a^2, and 0 where s is 0 (m and b are then 0 too).
template <bool PRECISE> __device__ __forceinline__ float inv_sqrt(float s) {
  const float r = PRECISE ? 1.0f / sqrtf(s) : rsqrt_approx(s);
  return s < 1e-36f ? 0.f : r;
}

// rate = c softplus(lam) of a row, and its gradient over itself, sigmoid(lam) / softplus(lam) (1 as lam -> -inf).
__device__ __forceinline__ float decay_rate(float c, float lam) { return c * softplus<true>(lam); }

struct Row {
  int64_t flat;  // flat index of the row's first element
  int f;         // elements of its first group that belong to the row before
  int64_t len;   // live steps
};

__device__ __forceinline__ Row row_of(const LruParams &p, int64_t row, int64_t b) {
  Row r;
  r.flat = row * p.L;
  r.f = (int)(r.flat & 7);
  r.len = p.lengths ? imin64(p.L, p.lengths[b] > 0 ? (int64_t)p.lengths[b] : 0) : p.L;
  return r;
}

// The 8 elements at steps t0 .. t0 + 7 of a row: one vector access where the group lies inside the
// tensor, element by element otherwise; elements outside [0, len) read as 0 or as a neighbour's.
template <typename T>
__device__ __forceinline__ void load_group(const T *base, const Row &r, int64_t t0, int64_t total, int vec,
                                           Raw8<T> &out) {
  const int64_t at = r.flat + t0;
  if (t0 + 8 > 0 && t0 < r.len && vec && at >= 0 && at + 8 <= total) {
    ld8(base + at, out);
    return;
  }
  zero8(out);
  if (t0 + 8 > 0 && t0 < r.len) {
#pragma unroll
    for (int e = 0; e < 8; e++)
      if (t0 + e >= 0 && t0 + e < r.len) put8(out, e, base[at + e]);
  }
}

// Store the elements of the group that lie in [0, L).
template <typename T>
__device__ __forceinline__ void store_group(T *base, const Row &r, int64_t t0, int64_t L, int vec, const float *v) {
  if (vec && t0 >= 0 && t0 + 8 <= L) {
    st8(base + r.flat + t0, v);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; e++)
    if (t0 + e >= 0 && t0 + e < L) base[r.flat + t0 + e] = from_f32<T>(v[e]);
}

// Bit e: step t0 + e starts a new sequence.
__device__ __forceinline__ unsigned load_resets(const uint8_t *reset, int64_t base, int64_t t0, int64_t len) {
  unsigned m = 0;
#pragma unroll
  for (int e = 0; e < 8; e++)
    if (t0 + e >= 0 && t0 + e < len && reset[base + t0 + e]) m |= 1u << e;
  return m;
}

// x -> P x + H after x -> Q x + G, where a P of 0 cuts off whatever came before (a reset: NaN and
// infinity of an earlier sequence must not reach this one through 0 * NaN).
template <bool RESET> __device__ __forceinline__ float after(float P, float x, float H) {
  return RESET && P == 0.f ? H : fmaf(P, x, H);
}
// The factor of the same composition, with the same cut.
template <bool RESET> __device__ __forceinline__ float times(float P, float Q) {
  return RESET && P == 0.f ? 0.f : P * Q;
}

}  // namespace

// ---- forward -----------------------------------------------------------------------------------

// W warps per row; with W = 1 the CTA's four warps take four rows.
template <typename T, typename Tout, int W, bool RESET>
__global__ void __launch_bounds__(W == 1 ? 128 : 32 * W) lru_fwd_kernel(const LruParams p) {
  constexpr bool PRECISE = sizeof(T) == 4;
  __shared__ float sP[2][W], sH[2][W];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = W == 1 ? (int64_t)blockIdx.x * 4 + warp : (int64_t)blockIdx.x;
  if (row >= p.Bt * p.Dn) return;  // whole warps, and with W > 1 never (one CTA per row)
  const int64_t b = row / p.Dn, d = row - b * p.Dn;
  const Row R = row_of(p, row, b);
  const int64_t total = p.Bt * p.Dn * p.L;
  const T *x = static_cast<const T *>(p.x), *rg = static_cast<const T *>(p.r), *ig = static_cast<const T *>(p.i);
  const float rb = p.r_bias ? p.r_bias[d] : 0.f, ib = p.i_bias ? p.i_bias[d] : 0.f;
  const float rate = decay_rate(p.c, p.lam[d]);
  float carry = p.h0 ? p.h0[row] : 0.f;  // the state that enters the round
  const int64_t n_ck = (p.L + R.f + kChunk - 1) / kChunk;
  const int w = W == 1 ? 0 : warp;
  Raw8<T> nx, nr, ni;
  {
    const int64_t t0 = (int64_t)w * kChunk + 8 * lane - R.f;
    load_group(x, R, t0, total, p.vec, nx);
    load_group(rg, R, t0, total, p.vec, nr);
    load_group(ig, R, t0, total, p.vec, ni);
  }
  int buf = 0;
  for (int64_t k0 = 0; k0 < n_ck; k0 += W, buf ^= 1) {
    const int64_t k = k0 + w;
    const int64_t t0 = k * kChunk + 8 * lane - R.f;
    float xv[8], a[8], bb[8], tmp[8];
    unpack8(nx, xv);
    unpack8(nr, a);
    unpack8(ni, tmp);
    {  // the next round's inputs
      const int64_t tn = t0 + (int64_t)W * kChunk;
      load_group(x, R, tn, total, p.vec, nx);
      load_group(rg, R, tn, total, p.vec, nr);
      load_group(ig, R, tn, total, p.vec, ni);
    }
    const unsigned cut = RESET ? load_resets(p.reset, b * p.L, t0, R.len) : 0u;
    const bool whole = t0 >= 0 && t0 + 8 <= R.len;
#pragma unroll
    for (int e = 0; e < 8; e++) {
      float r, g;
      sigmoid2<PRECISE>(a[e] + rb, tmp[e] + ib, r, g);
      float em;
      decay<PRECISE>(-rate * r, a[e], em);
      const float s = -em * (em + 2.f);
      const float m = s * inv_sqrt<PRECISE>(s);
      if (RESET && (cut >> e & 1)) a[e] = 0.f;
      bb[e] = m * g * xv[e];
    }
    if (!whole) {
#pragma unroll
      for (int e = 0; e < 8; e++)
        if (t0 + e < 0 || t0 + e >= R.len) a[e] = 1.f, bb[e] = 0.f;
    }
    float P = a[0], H = bb[0];
#pragma unroll
    for (int e = 1; e < 8; e++) {
      H = after<RESET>(a[e], H, bb[e]);
      P = times<RESET>(a[e], P);
    }
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const float Q = __shfl_up_sync(kFull, P, off), G = __shfl_up_sync(kFull, H, off);
      if (lane >= off) {
        H = after<RESET>(P, G, H);
        P = times<RESET>(P, Q);
      }
    }
    float in = carry;  // the state that enters this warp's chunk
    if (W > 1) {
      if (lane == 31) {
        sP[buf][w] = P;
        sH[buf][w] = H;
      }
      __syncthreads();  // two buffers: a warp can be one round ahead of the slowest reader, not two
      float c = carry;
#pragma unroll
      for (int v = 0; v < W; v++) {
        if (v == w) in = c;
        c = after<RESET>(sP[buf][v], c, sH[buf][v]);
      }
      carry = c;
    }
    // the state that enters the lane
    const float Pe = __shfl_up_sync(kFull, P, 1), He = __shfl_up_sync(kFull, H, 1);
    float h = lane == 0 ? in : after<RESET>(Pe, in, He);
    if (W == 1) carry = after<RESET>(__shfl_sync(kFull, P, 31), carry, __shfl_sync(kFull, H, 31));
    if (k < n_ck) {
      if (p.states && lane == 0) p.states[row * p.n_states + k] = in;
      if (p.out) {
#pragma unroll
        for (int e = 0; e < 8; e++) bb[e] = h = after<RESET>(a[e], h, bb[e]);
        if (!whole) {
#pragma unroll
          for (int e = 0; e < 8; e++)
            if (t0 + e >= R.len) bb[e] = 0.f;
        }
        store_group(static_cast<Tout *>(p.out), R, t0, p.L, p.vec_out, bb);
      }
    }
  }
  if (p.h_last && threadIdx.x % (32 * W) == 0) p.h_last[row] = carry;
}

// ---- backward ----------------------------------------------------------------------------------

template <typename T, typename Tg, int W, bool RESET>
__global__ void __launch_bounds__(W == 1 ? 128 : 32 * W) lru_bwd_kernel(const LruBwdParams q) {
  constexpr bool PRECISE = sizeof(T) == 4;
  const LruParams &p = q.f;
  __shared__ float sP[2][W], sM[2][W];
  __shared__ float sS[3][W];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = W == 1 ? (int64_t)blockIdx.x * 4 + warp : (int64_t)blockIdx.x;
  if (row >= p.Bt * p.Dn) return;  // whole warps, and with W > 1 never
  const int64_t b = row / p.Dn, d = row - b * p.Dn;
  const Row R = row_of(p, row, b);
  const int64_t total = p.Bt * p.Dn * p.L;
  const T *x = static_cast<const T *>(p.x), *rg = static_cast<const T *>(p.r), *ig = static_cast<const T *>(p.i);
  const T *dout = static_cast<const T *>(q.dout);
  const float rb = p.r_bias ? p.r_bias[d] : 0.f, ib = p.i_bias ? p.i_bias[d] : 0.f;
  const float lam = p.lam[d];
  const float rate = decay_rate(p.c, lam);
  float carry = q.dh_last ? q.dh_last[row] : 0.f;  // mu arriving at the round's last step from behind
  const int64_t n_ck = (p.L + R.f + kChunk - 1) / kChunk;
  const int64_t rounds = (n_ck + W - 1) / W;
  const int w = W == 1 ? 0 : warp;
  float sum_q = 0.f, sum_r = 0.f, sum_i = 0.f;
  Raw8<T> nx, nr, ni, nd;
  float nh = 0.f;
  {
    const int64_t k = (rounds - 1) * W + w;
    const int64_t t0 = k * kChunk + 8 * lane - R.f;
    load_group(x, R, t0, total, p.vec, nx);
    load_group(rg, R, t0, total, p.vec, nr);
    load_group(ig, R, t0, total, p.vec, ni);
    load_group(dout, R, t0, total, p.vec, nd);
    if (k < n_ck) nh = p.states[row * p.n_states + k];
  }
  int buf = 0;
  for (int64_t it = rounds - 1; it >= 0; it--, buf ^= 1) {
    const int64_t k = it * W + w;
    const int64_t t0 = k * kChunk + 8 * lane - R.f;
    float a[8], la[8], u[8], v[8], z[8], bb[8], dv[8];
    unpack8(nx, bb);
    unpack8(nr, a);
    unpack8(ni, v);
    unpack8(nd, dv);
    const float hin = nh;
    if (it > 0) {  // the next round's inputs
      const int64_t tn = t0 - (int64_t)W * kChunk;
      load_group(x, R, tn, total, p.vec, nx);
      load_group(rg, R, tn, total, p.vec, nr);
      load_group(ig, R, tn, total, p.vec, ni);
      load_group(dout, R, tn, total, p.vec, nd);
      nh = p.states[row * p.n_states + k - W];
    }
    const unsigned cut = RESET ? load_resets(p.reset, b * p.L, t0, R.len) : 0u;
    const bool whole = t0 >= 0 && t0 + 8 <= R.len;
#pragma unroll
    for (int e = 0; e < 8; e++) {
      float r, g;
      sigmoid2<PRECISE>(a[e] + rb, v[e] + ib, r, g);
      la[e] = -rate * r;
      float em;
      decay<PRECISE>(la[e], a[e], em);
      const float s = -em * (em + 2.f);
      const float is = inv_sqrt<PRECISE>(s);
      if (RESET && (cut >> e & 1)) a[e] = 0.f;
      u[e] = s * is * g;             // m g
      bb[e] *= u[e];                 // m g x
      v[e] = bb[e] * (1.f - g);
      z[e] = la[e] * is * is * bb[e];  // rho b
    }
    if (!whole) {
#pragma unroll
      for (int e = 0; e < 8; e++)
        if (t0 + e < 0 || t0 + e >= R.len) a[e] = 1.f, bb[e] = la[e] = u[e] = v[e] = z[e] = dv[e] = 0.f;
    }
    // the states, from the state that entered the chunk
    float P = a[0], H = bb[0];
#pragma unroll
    for (int e = 1; e < 8; e++) {
      H = after<RESET>(a[e], H, bb[e]);
      P = times<RESET>(a[e], P);
    }
    // and what leaves the lane's first step backwards: mu -> P mu + M
    float S = RESET && cut ? 0.f : P, M = 0.f;
#pragma unroll
    for (int e = 7; e >= 0; e--) M = after<RESET>(a[e], dv[e] + M, 0.f);
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const float Q = __shfl_up_sync(kFull, P, off), G = __shfl_up_sync(kFull, H, off);
      const float Z = __shfl_down_sync(kFull, S, off), N = __shfl_down_sync(kFull, M, off);
      if (lane >= off) {
        H = after<RESET>(P, G, H);
        P = times<RESET>(P, Q);
      }
      if (lane + off < 32) {
        M = after<RESET>(S, N, M);
        S = times<RESET>(S, Z);
      }
    }
    float in = carry;  // mu arriving behind this warp's chunk
    if (W > 1) {
      if (lane == 0) {
        sP[buf][w] = S;
        sM[buf][w] = M;
      }
      __syncthreads();
      float c = carry;
#pragma unroll
      for (int o = W - 1; o >= 0; o--) {
        if (o == w) in = c;
        c = after<RESET>(sP[buf][o], c, sM[buf][o]);
      }
      carry = c;
    }
    const float Pe = __shfl_up_sync(kFull, P, 1), He = __shfl_up_sync(kFull, H, 1);
    float h = lane == 0 ? hin : after<RESET>(Pe, hin, He);
    const float Se = __shfl_down_sync(kFull, S, 1), Me = __shfl_down_sync(kFull, M, 1);
    float mu = lane == 31 ? in : after<RESET>(Se, in, Me);
    if (W == 1) carry = after<RESET>(__shfl_sync(kFull, S, 0), carry, __shfl_sync(kFull, M, 0));
    if (k >= n_ck) continue;
#pragma unroll
    for (int e = 0; e < 8; e++) {
      h = after<RESET>(a[e], h, bb[e]);
      z[e] = fmaf(la[e], h, -z[e]);  // la h - rho b
    }
    const float inv_rate = rate > 0.f ? 1.f / rate : 0.f;
#pragma unroll
    for (int e = 7; e >= 0; e--) {
      const float lm = dv[e] + mu;
      mu = after<RESET>(a[e], lm, 0.f);
      u[e] *= lm;
      v[e] *= lm;
      const float g = lm * z[e];
      z[e] = g * fmaf(la[e], inv_rate, 1.f);  // 1 - r = 1 + la / rate
      bb[e] = g;
    }
    if (!whole) {  // steps outside the row hold 0 (0 times an infinite lambda would not be)
#pragma unroll
      for (int e = 0; e < 8; e++)
        if (t0 + e < 0 || t0 + e >= R.len) u[e] = v[e] = z[e] = bb[e] = 0.f;
    }
    if (q.dx) store_group(static_cast<Tg *>(q.dx), R, t0, p.L, q.vec_grad, u);
    if (q.di) store_group(static_cast<Tg *>(q.di), R, t0, p.L, q.vec_grad, v);
    if (q.dr) store_group(static_cast<Tg *>(q.dr), R, t0, p.L, q.vec_grad, z);
#pragma unroll
    for (int e = 0; e < 8; e++) sum_q += bb[e], sum_r += z[e], sum_i += v[e];
  }
  if (q.dh0 && threadIdx.x % (32 * W) == 0) q.dh0[row] = carry;
  if (!q.p_dlam && !q.p_dr && !q.p_di) return;
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) {
    sum_q += __shfl_xor_sync(kFull, sum_q, off);
    sum_r += __shfl_xor_sync(kFull, sum_r, off);
    sum_i += __shfl_xor_sync(kFull, sum_i, off);
  }
  if (W > 1) {
    if (lane == 0) sS[0][w] = sum_q, sS[1][w] = sum_r, sS[2][w] = sum_i;
    __syncthreads();
    if (threadIdx.x != 0) return;
    sum_q = sum_r = sum_i = 0.f;
    for (int o = 0; o < W; o++) sum_q += sS[0][o], sum_r += sS[1][o], sum_i += sS[2][o];
  } else if (lane != 0) {
    return;
  }
  // sigmoid / softplus: 1 as lam -> -inf, where softplus reaches 0
  const float sp = softplus<true>(lam);
  if (q.p_dlam) q.p_dlam[row] = sum_q * (sp > 0.f ? sigmoid<true>(lam) / sp : 1.f);
  if (q.p_dr) q.p_dr[row] = sum_r;
  if (q.p_di) q.p_di[row] = sum_i;
}

// Per-row sums over the batch in a fixed order.
__global__ void __launch_bounds__(128) lru_param_sum_kernel(const LruBwdParams q) {
  const int64_t d = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (d >= q.f.Dn) return;
  const float *src[3] = {q.p_dlam, q.p_dr, q.p_di};
  float *dst[3] = {q.dlam, q.dr_bias, q.di_bias};
#pragma unroll
  for (int j = 0; j < 3; j++) {
    if (!dst[j]) continue;
    float s = 0.f;
    for (int64_t b = 0; b < q.f.Bt; b++) s += src[j][b * q.f.Dn + d];
    dst[j][d] = s;
  }
}

// ---- one-token step ----------------------------------------------------------------------------

// V consecutive channels a thread (V = 4: Dn a multiple of 4 and every pointer on a vector boundary).
template <typename T, typename Tout, int V>
__global__ void __launch_bounds__(128) lru_step_kernel(const LruStepParams p) {
  constexpr bool PRECISE = sizeof(T) == 4;
  const int64_t i0 = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * V;
  if (i0 >= p.Bt * p.Dn) return;
  const int64_t d = i0 % p.Dn;
  alignas(16) T x[V], r[V], g[V];
  alignas(16) float h[V], lam[V], rb[V], ib[V];
  alignas(16) Tout o[V];
  if constexpr (V == 4) {
    using V4 = typename std::conditional<PRECISE, float4, uint2>::type;
    *reinterpret_cast<V4 *>(x) = *reinterpret_cast<const V4 *>(static_cast<const T *>(p.x) + i0);
    *reinterpret_cast<V4 *>(r) = *reinterpret_cast<const V4 *>(static_cast<const T *>(p.r) + i0);
    *reinterpret_cast<V4 *>(g) = *reinterpret_cast<const V4 *>(static_cast<const T *>(p.i) + i0);
    *reinterpret_cast<float4 *>(h) = *reinterpret_cast<const float4 *>(p.h + i0);
    *reinterpret_cast<float4 *>(lam) = *reinterpret_cast<const float4 *>(p.lam + d);
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    *reinterpret_cast<float4 *>(rb) = p.r_bias ? *reinterpret_cast<const float4 *>(p.r_bias + d) : zero;
    *reinterpret_cast<float4 *>(ib) = p.i_bias ? *reinterpret_cast<const float4 *>(p.i_bias + d) : zero;
  } else {
    x[0] = static_cast<const T *>(p.x)[i0];
    r[0] = static_cast<const T *>(p.r)[i0];
    g[0] = static_cast<const T *>(p.i)[i0];
    h[0] = p.h[i0];
    lam[0] = p.lam[d];
    rb[0] = p.r_bias ? p.r_bias[d] : 0.f;
    ib[0] = p.i_bias ? p.i_bias[d] : 0.f;
  }
#pragma unroll
  for (int e = 0; e < V; e++) {
    float rr, gg;
    sigmoid2<PRECISE>(to_f32(r[e]) + rb[e], to_f32(g[e]) + ib[e], rr, gg);
    float a, em;
    decay<PRECISE>(-decay_rate(p.c, lam[e]) * rr, a, em);
    const float s = -em * (em + 2.f);
    h[e] = fmaf(a, h[e], s * inv_sqrt<PRECISE>(s) * gg * to_f32(x[e]));
    o[e] = from_f32<Tout>(h[e]);
  }
  if constexpr (V == 4) {
    using O4 = typename std::conditional<sizeof(Tout) == 4, float4, uint2>::type;
    *reinterpret_cast<float4 *>(p.h + i0) = *reinterpret_cast<const float4 *>(h);
    *reinterpret_cast<O4 *>(static_cast<Tout *>(p.out) + i0) = *reinterpret_cast<const O4 *>(o);
  } else {
    p.h[i0] = h[0];
    static_cast<Tout *>(p.out)[i0] = o[0];
  }
}

// ---- launchers ---------------------------------------------------------------------------------

namespace {

// Warps per row: one where the rows alone give every SM enough warps to hide the memory latency
// (kWantWarps in flight on the whole GPU), else the fewest of 4, 8, 16 that do, and never many more
// than the row has chunks.
constexpr int64_t kWantWarps = 148 * 24;

int warps_per_row(int64_t rows, int64_t L) {
  const int64_t chunks = (L + 7 + kChunk - 1) / kChunk;
  if (chunks <= 2) return 1;
  int w = 1;
  while (w < kMaxWarps && rows * w < kWantWarps && w < chunks) w = w == 1 ? 4 : 2 * w;
  return w;
}

template <typename T, typename Tout, int W>
cudaError_t fwd_w(const LruParams &p, cudaStream_t s) {
  const int64_t rows = p.Bt * p.Dn, blocks = W == 1 ? (rows + 3) / 4 : rows;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const int threads = W == 1 ? 128 : 32 * W;
  if (p.reset)
    lru_fwd_kernel<T, Tout, W, true><<<(unsigned)blocks, threads, 0, s>>>(p);
  else
    lru_fwd_kernel<T, Tout, W, false><<<(unsigned)blocks, threads, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T, typename Tout> cudaError_t fwd_t(const LruParams &p, cudaStream_t s) {
  switch (warps_per_row(p.Bt * p.Dn, p.L)) {
    case 1: return fwd_w<T, Tout, 1>(p, s);
    case 4: return fwd_w<T, Tout, 4>(p, s);
    case 8: return fwd_w<T, Tout, 8>(p, s);
    default: return fwd_w<T, Tout, 16>(p, s);
  }
}

template <typename T, typename Tg, int W>
cudaError_t bwd_w(const LruBwdParams &q, cudaStream_t s) {
  const int64_t rows = q.f.Bt * q.f.Dn, blocks = W == 1 ? (rows + 3) / 4 : rows;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const int threads = W == 1 ? 128 : 32 * W;
  if (q.f.reset)
    lru_bwd_kernel<T, Tg, W, true><<<(unsigned)blocks, threads, 0, s>>>(q);
  else
    lru_bwd_kernel<T, Tg, W, false><<<(unsigned)blocks, threads, 0, s>>>(q);
  return cudaGetLastError();
}

template <typename T, typename Tg> cudaError_t bwd_t(const LruBwdParams &q, cudaStream_t s) {
  switch (warps_per_row(q.f.Bt * q.f.Dn, q.f.L)) {
    case 1: return bwd_w<T, Tg, 1>(q, s);
    case 4: return bwd_w<T, Tg, 4>(q, s);
    case 8: return bwd_w<T, Tg, 8>(q, s);
    default: return bwd_w<T, Tg, 16>(q, s);
  }
}

template <typename T, typename Tout> cudaError_t step_t(const LruStepParams &p, cudaStream_t s) {
  const int64_t n = p.Bt * p.Dn;
  const int64_t blocks = p.vec ? (n / 4 + 127) / 128 : (n + 127) / 128;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (p.vec)
    lru_step_kernel<T, Tout, 4><<<(unsigned)blocks, 128, 0, s>>>(p);
  else
    lru_step_kernel<T, Tout, 1><<<(unsigned)blocks, 128, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_lru_fwd(const LruParams &p, int in_bf16, int out_bf16, cudaStream_t s) {
  if (in_bf16) return out_bf16 ? fwd_t<__nv_bfloat16, __nv_bfloat16>(p, s) : fwd_t<__nv_bfloat16, float>(p, s);
  return out_bf16 ? fwd_t<float, __nv_bfloat16>(p, s) : fwd_t<float, float>(p, s);
}

cudaError_t launch_lru_bwd(const LruBwdParams &q, int in_bf16, int grad_bf16, cudaStream_t s) {
  cudaError_t e;
  if (in_bf16)
    e = grad_bf16 ? bwd_t<__nv_bfloat16, __nv_bfloat16>(q, s) : bwd_t<__nv_bfloat16, float>(q, s);
  else
    e = grad_bf16 ? bwd_t<float, __nv_bfloat16>(q, s) : bwd_t<float, float>(q, s);
  if (e != cudaSuccess || q.f.Bt == 1 || (!q.dlam && !q.dr_bias && !q.di_bias)) return e;
  lru_param_sum_kernel<<<(unsigned)((q.f.Dn + 127) / 128), 128, 0, s>>>(q);
  return cudaGetLastError();
}

cudaError_t launch_lru_step(const LruStepParams &p, int in_bf16, int out_bf16, cudaStream_t s) {
  if (in_bf16) return out_bf16 ? step_t<__nv_bfloat16, __nv_bfloat16>(p, s) : step_t<__nv_bfloat16, float>(p, s);
  return out_bf16 ? step_t<float, __nv_bfloat16>(p, s) : step_t<float, float>(p, s);
}

}  // namespace ssm
