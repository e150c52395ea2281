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
// state that entered each chunk (saved by the forward) and a second composition. With y = -la, w = y a and
// s = 1 - a^2 the gradient of y times y is q = -lambda w (h_{t-1} - a b / s): y / s stays finite as a -> 1 (it
// tends to 1/2), and neither term holds what the other cancels as a -> 0 (y (h_t - b / s), one instruction a pair shorter, left
// the rounding of y b in results of the size of y a).
//   dx = lambda m g, di~ = lambda b (1 - g), dr~ = q (1 - r), dlam = sum q sigmoid(lam)/softplus(lam)
// 1 - r comes from the gate's own exponential: y over the rate would lose it at a gate held open, and be infinite where
// softplus(lam) is a denormal.
//
// Precision. The decay goes through n = 1 - a (a polynomial for small |la|): 1 - a^2 = n + n a keeps its relative
// precision where a is near 1, which a itself in 32 bits does not. States, sums and gradients are fp32 up to their one
// rounding into the output's type; sigmoid, exp2 and the root are the hardware's (1 to 4 units of 2^-24), for
// fp32 inputs too: against float64 the fp32 outputs and gradients of 3 x 1001 x 2047 are off by 3e-7 together.
//
// What bounds it. HBM, at 82% of the measured copy rate on long rows in a burst (bf16, 1 x 5120 x 65536 forward: 498 us, 5.4 TB/s; 534 to
// 568 us call after call, when the chip is warm; 4 x 4096 x 4096 forward and backward 270 us of 225): 38 issue slots per element
// forwards and 58 backwards are 72% and 65% of the SMs' issue, the four MUFU operations per element 60% of theirs forwards.
#include <type_traits>

#include "ssm_internal.h"
#include "ssm_vec.cuh"

namespace ssm {

namespace {

constexpr int kChunk = 256;  // steps per warp and round: 32 lanes x 8
constexpr unsigned kFull = 0xffffffffu;
constexpr int kMaxWarps = 16;
__device__ __forceinline__ float rsqrt_approx(float x) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// min and max that keep NaN (fminf would drop it).
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }

// A lane's 8 elements as 4 pairs (j, j + 4): two half runs of 4 steps in the two halves of the packed fp32
// instructions, so that the recurrence itself is packed too.
__device__ __forceinline__ void pairs(const Raw8<__nv_bfloat16> &r, float2 *v) {
  v[0] = make_float2(__uint_as_float(r.a.x << 16), __uint_as_float(r.a.z << 16));
  v[1] = make_float2(__uint_as_float(r.a.x & 0xffff0000u), __uint_as_float(r.a.z & 0xffff0000u));
  v[2] = make_float2(__uint_as_float(r.a.y << 16), __uint_as_float(r.a.w << 16));
  v[3] = make_float2(__uint_as_float(r.a.y & 0xffff0000u), __uint_as_float(r.a.w & 0xffff0000u));
}
__device__ __forceinline__ void pairs(const Raw8<float> &r, float2 *v) {
  v[0] = make_float2(r.a.x, r.b.x);
  v[1] = make_float2(r.a.y, r.b.y);
  v[2] = make_float2(r.a.z, r.b.z);
  v[3] = make_float2(r.a.w, r.b.w);
}
__device__ __forceinline__ void in_order(const float2 *v, float *o) {
#pragma unroll
  for (int j = 0; j < 4; j++) o[j] = v[j].x, o[4 + j] = v[j].y;
}

// What a row's gates need of its parameters. A gate's argument is kept above -44 (its sigmoid above 2^-63), so
// that the product of two denominators 1 + e^-v stays finite; NaN passes. bf16 inputs are clamped as they are, two
// at a time, to `low`, which rounding to bf16 moves by 2 at most while the bias is within 960 (`low` then within 1024); a row
// with a larger one (a gate held shut or open) clamps the arguments themselves, at -41.6, as fp32 inputs do.
struct Gate {
  float shift;         // -bias log2 e
  __nv_bfloat162 low;  // -41.5 - bias
  bool wide;
};
__device__ __forceinline__ Gate gate_of(float bias) {
  return {-bias * kLog2e, __float2bfloat162_rn(-41.5f - bias), !(fabsf(bias) <= 960.f)};
}
__device__ __forceinline__ void clamp(float2 *t) {
#pragma unroll
  for (int j = 0; j < 4; j++) t[j] = make_float2(min_nan(t[j].x, 60.f), min_nan(t[j].y, 60.f));
}
__device__ __forceinline__ void arguments(const Raw8<__nv_bfloat16> &raw, const Gate &g, float2 *t) {
  Raw8<__nv_bfloat16> c = raw;
  if (!g.wide) {
    __nv_bfloat162 *w = reinterpret_cast<__nv_bfloat162 *>(&c.a);
#pragma unroll
    for (int j = 0; j < 4; j++) w[j] = __hmax2_nan(w[j], g.low);
  }
  pairs(c, t);
#pragma unroll
  for (int j = 0; j < 4; j++) t[j] = fma2(t[j], splat(-kLog2e), splat(g.shift));
  if (g.wide) clamp(t);
}
__device__ __forceinline__ void arguments(const Raw8<float> &raw, const Gate &g, float2 *t) {
  pairs(raw, t);
#pragma unroll
  for (int j = 0; j < 4; j++) t[j] = fma2(t[j], splat(-kLog2e), splat(g.shift));
  clamp(t);
}
// Both sigmoids from -v log2 e, with one reciprocal: 1/((1+eu)(1+ev)); eu and ev are e^-u and e^-v, with which
// 1 - sigmoid(v) = ev sigmoid(v) keeps its relative precision at a gate held open.
__device__ __forceinline__ void sigmoid2(float2 tu, float2 tv, float2 &su, float2 &sv, float2 &eu, float2 &ev) {
  eu = make_float2(ex2_approx(tu.x), ex2_approx(tu.y));
  ev = make_float2(ex2_approx(tv.x), ex2_approx(tv.y));
  const float2 pu = add2(eu, splat(1.f)), pv = add2(ev, splat(1.f));
  const float2 d = mul2(pu, pv);
  const float2 inv = make_float2(rcp_approx(d.x), rcp_approx(d.y));
  su = mul2(pv, inv);
  sv = mul2(pu, inv);
}

// From y = -la >= 0: n = 1 - a and a = e^-y, both with relative precision, s = 1 - a^2 = n + n a, and 1 / sqrt(s).
// n is y times a polynomial of degree 4 (a minimax fit on [0, 1/2], relative error 8e-8, 2e-7 with the
// roundings) where y < 1/2, and 1 - ex2 beyond, where a comes from ex2 (2^-22 of it, 3e-7 of n >= 0.39 at most).
// NEAR: the whole row is in the first case, y <= rate < 1/2. Callers add kTiny to y, so that s is above 0 and
// the root finite where the decay is 1; m = s / sqrt(s) is then below 2e-18.
constexpr float kNear = 0.5f, kTiny = 1e-36f;
template <bool NEAR> __device__ __forceinline__ void decay(float2 y, float2 &a, float2 &s, float2 &is) {
  float2 p = fma2(y, splat(0x1.bbbf2ap-8f), splat(-0x1.4fe1eap-5f));
  p = fma2(y, p, splat(0x1.551732p-3f));
  p = fma2(y, p, splat(-0x1.fffe08p-2f));
  p = fma2(y, p, splat(0x1.fffffep-1f));
  float2 n = mul2(y, p);
  a = fma2(n, splat(-1.f), splat(1.f));
  if (!NEAR) {
    const float2 t = mul2(y, splat(-kLog2e));
    const float2 far = make_float2(ex2_approx(t.x), ex2_approx(t.y)), fn = fma2(far, splat(-1.f), splat(1.f));
    if (!(y.x < kNear)) a.x = far.x, n.x = fn.x;
    if (!(y.y < kNear)) a.y = far.y, n.y = fn.y;
  }
  s = fma2(n, a, n);
  is = make_float2(rsqrt_approx(s.x), rsqrt_approx(s.y));
}

// rate = c softplus(lam), the log decay of an open gate.
__device__ __forceinline__ float decay_rate(float c, float lam) { return c * softplus<true>(lam); }

struct Row {
  int64_t flat;  // flat index of the row's first element
  int f;         // elements of its first group that belong to the row before
  int len;       // live steps (L is below 2^31 - 2^15, so steps and chunks count in 32 bits)
  int k_lo, k_hi;  // the chunks inside the live steps
  int n_live;      // chunks that hold live steps
};

__device__ __forceinline__ Row row_of(const LruParams &p, int64_t row, int64_t b) {
  Row r;
  r.flat = row * p.L;
  r.f = (int)(r.flat & 7);
  r.len = p.lengths ? min((int)p.L, max(p.lengths[b], 0)) : (int)p.L;
  r.k_lo = r.f ? 1 : 0;
  r.k_hi = (r.len + r.f) / kChunk;
  r.n_live = r.len > 0 ? (r.len + r.f + kChunk - 1) / kChunk : 0;
  return r;
}

// Chunk k of a row lies inside its live steps: no element of a lane is masked.
__device__ __forceinline__ bool inside(const Row &r, int k) { return k >= r.k_lo && k < r.k_hi; }

// The 8 elements at steps t0 .. t0 + 7 of a row that may reach over its ends: one vector access where the group lies
// inside the tensor, element by element otherwise; elements outside [0, len) read as 0 or as a neighbour's.
template <typename T>
__device__ __forceinline__ void load_edge(const T *base, const Row &r, int t0, int64_t total, int vec, Raw8<T> &out) {
  const int64_t at = r.flat + t0;
  if (vec && t0 < r.len && at >= 0 && at + 8 <= total) {
    ld8(base + at, out);
    return;
  }
  zero8(out);
  if (t0 < r.len) {
#pragma unroll
    for (int e = 0; e < 8; e++)
      if (t0 + e >= 0 && t0 + e < r.len) put8(out, e, base[at + e]);
  }
}

// A lane's groups of NT tensors on their way, S rounds of them, in shared memory: each lane copies (cp.async) and
// reads only its own 16-byte slots, so nothing but its own copies is waited for, and no register holds
// what is in flight.
template <typename T, int NT, int S> struct Ring {
  static constexpr int kHalves = sizeof(T) * 8 / 16;                // 16-byte slots per group
  static constexpr int kWarpBytes = S * NT * kHalves * 32 * 16;
  char *base;                                                       // the lane's first slot
  __device__ __forceinline__ Ring(char *smem, int warp, int lane) : base(smem + warp * kWarpBytes + lane * 16) {}
  __device__ __forceinline__ char *slot(int stage, int tensor, int half) const {
    return base + ((stage * NT + tensor) * kHalves + half) * 512;
  }
  __device__ __forceinline__ void copy(int stage, int tensor, const T *src) const {
#pragma unroll
    for (int h = 0; h < kHalves; h++) cp_async16(slot(stage, tensor, h), reinterpret_cast<const char *>(src) + 16 * h);
  }
  __device__ __forceinline__ void put(int stage, int tensor, const Raw8<T> &v) const {
#pragma unroll
    for (int h = 0; h < kHalves; h++)
      *reinterpret_cast<uint4 *>(slot(stage, tensor, h)) = reinterpret_cast<const uint4 *>(&v)[h];
  }
  __device__ __forceinline__ void get(int stage, int tensor, Raw8<T> &v) const {
#pragma unroll
    for (int h = 0; h < kHalves; h++)
      reinterpret_cast<uint4 *>(&v)[h] = *reinterpret_cast<const uint4 *>(slot(stage, tensor, h));
  }
};
// Rounds in use and in flight: three of bf16, two of fp32 (twice the bytes each) or of 16 warps. (One-warp rows
// of bf16: 2 to 5 measured within 5% of each other on every shape.)
template <typename T, int W> constexpr int kStages = sizeof(T) == 4 || W == 16 ? 2 : 3;

// Store the elements of the group that lie in [0, L).
template <typename T>
__device__ __forceinline__ void store_group(T *base, const Row &r, bool in, int t0, int L, int vec, const float2 *pv) {
  float v[8];
  in_order(pv, v);
  T *at = base + (r.flat + t0);
  if (vec && (in || (t0 >= 0 && t0 + 8 <= L))) {
    st8(at, v);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; e++)
    if (t0 + e >= 0 && t0 + e < L) at[e] = from_f32<T>(v[e]);
}

// The reset bytes of steps t0 .. t0 + 7 (0 outside [0, len)): two aligned words and a shift where both lie inside the
// mask, byte by byte at its ends.
__device__ __forceinline__ uint64_t load_resets(const LruParams &p, int64_t b, const Row &r, int t0) {
  if (t0 >= r.len) return 0;
  const uint8_t *at = p.reset + b * p.L + t0;
  const int shift = (int)(reinterpret_cast<uintptr_t>(at) & 7);
  const uint8_t *word = at - shift;
  if (t0 >= 0 && t0 + 8 <= r.len && word >= p.reset && word + 16 <= p.reset + p.Bt * p.L) {
    const uint64_t lo = reinterpret_cast<const uint64_t *>(word)[0], hi = reinterpret_cast<const uint64_t *>(word)[1];
    return shift ? lo >> (8 * shift) | hi << (64 - 8 * shift) : lo;
  }
  uint64_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; e++)
    if (t0 + e >= 0 && t0 + e < r.len && at[e]) m |= UINT64_C(1) << (8 * e);
  return m;
}

// A lane's cuts (its steps that start a sequence) as bits, and the lanes of its row that hold any. What is composed asks these where a cut
// lies, not a factor of 0: NaN and infinity of an earlier sequence must not reach a later one through 0 * NaN, and a factor that
// underflows must not hide a NaN of its own sequence.
struct Cuts {
  uint32_t bits = 0, lanes = 0;
  __device__ __forceinline__ bool at(int e) const { return bits >> e & 1; }
  __device__ __forceinline__ bool first() const { return bits & 0xf; }  // in the lane's first half run
  __device__ __forceinline__ bool second() const { return bits >> 4; }
  __device__ __forceinline__ bool before(int lane) const { return lanes & ((1u << lane) - 1); }
  __device__ __forceinline__ bool behind(int lane) const { return lanes >> lane >> 1; }
};
// Bits of the non-zero bytes of a word.
__device__ __forceinline__ uint32_t byte_bits(uint32_t v) {
  const uint32_t high = (((v & 0x7f7f7f7fu) + 0x7f7f7f7fu) | v) & 0x80808080u;
  return (high >> 7) * 0x10204080u >> 28;  // bits 0, 8, 16, 24 to 28 .. 31, every other product elsewhere
}
__device__ __forceinline__ uint32_t cut_bits(uint64_t bytes) {
  return byte_bits((uint32_t)bytes) | byte_bits((uint32_t)(bytes >> 32)) << 4;
}

// x -> P x + H, or H alone behind a cut.
__device__ __forceinline__ float after(bool cut, float P, float x, float H) { return cut ? H : fmaf(P, x, H); }
// Of step j of both half runs.
template <bool CUT> __device__ __forceinline__ float2 after2(const Cuts &c, int j, float2 P, float2 x, float2 H) {
  const float2 r = fma2(P, x, H);
  if (CUT) return make_float2(c.at(j) ? H.x : r.x, c.at(j + 4) ? H.y : r.y);
  return r;
}

// The maps of a lane's two half runs, and of the lanes up to and including this one (the factors only where no cut lies).
template <bool CUT>
__device__ __forceinline__ void compose(const Cuts &c, const float2 *a, const float2 *b, float2 &P2, float2 &H2) {
  P2 = a[0];
  H2 = b[0];
#pragma unroll
  for (int j = 1; j < 4; j++) {
    H2 = after2<CUT>(c, j, a[j], H2, b[j]);
    P2 = mul2(a[j], P2);
  }
}
template <bool CUT> __device__ __forceinline__ void scan_up_step(int lane, int off, int last, float &P, float &H) {
  const float Q = __shfl_up_sync(kFull, P, off), G = __shfl_up_sync(kFull, H, off);
  if (lane >= off) {
    H = after(CUT && last < off, P, G, H);
    P *= Q;
  }
}
// Lanes back to the last one with a cut, this one's 0 (lane + 1 with none).
__device__ __forceinline__ int last_cut(const Cuts &c, int lane) { return lane - 31 + __clz(c.lanes & ((2u << lane) - 1)); }
template <bool CUT> __device__ __forceinline__ void scan_up(int lane, const Cuts &c, float &P, float &H) {
  const int last = CUT ? last_cut(c, lane) : 0;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) scan_up_step<CUT>(lane, off, last, P, H);
}
template <bool CUT> __device__ __forceinline__ void scan_down_step(int lane, int off, int G, unsigned next, float &S, float &M) {
  const float Z = __shfl_down_sync(kFull, S, off), N = __shfl_down_sync(kFull, M, off);
  if (lane + off < G) {
    M = after(CUT && next < off, S, N, M);
    S *= Z;
  }
}
// Lanes on to the next one with a cut (a large number with none).
__device__ __forceinline__ unsigned next_cut(const Cuts &c, int lane) { return (unsigned)__ffs(c.lanes >> lane) - 1u; }
template <bool CUT> __device__ __forceinline__ void scan_down(int lane, const Cuts &c, float &S, float &M) {
  const unsigned next = CUT ? next_cut(c, lane) : 0;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) scan_down_step<CUT>(lane, off, 32, next, S, M);
}
// A chunk's factor for the other warps: 0 says that a cut lies in it, and nothing else does.
__device__ __forceinline__ float factor_of(const Cuts &c, float P) { return c.lanes ? 0.f : max_nan(P, 1.17549435e-38f); }

// Element e of a pair array.
__device__ __forceinline__ float &elem(float2 *v, int e) { return e < 4 ? v[e].x : v[e - 4].y; }

}  // namespace

// ---- forward -----------------------------------------------------------------------------------

// A CTA of W warps per row. One-warp CTAs for the common case: as many rows as an SM has warps, no barriers, and a
// tail of single rows (4 x 4096 x 4096 bf16 forward + backward 267 us, with four rows per CTA 283 us).
template <typename T, typename Tout, int W, bool RESET>
__global__ void __launch_bounds__(32 * W, W <= 4 ? 28 / W : 1) lru_fwd_kernel(const __grid_constant__ LruParams p) {
  extern __shared__ __align__(16) char ring_smem[];
  constexpr int S = kStages<T, W>;
  __shared__ float sP[2][W], sH[2][W];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t row = blockIdx.x;
  const int64_t b = row / p.Dn, d = row - b * p.Dn;
  const Row R = row_of(p, row, b);
  const int64_t total = p.Bt * p.Dn * p.L;
  const T *x = static_cast<const T *>(p.x), *rg = static_cast<const T *>(p.r), *ig = static_cast<const T *>(p.i);
  const int L = (int)p.L, n_ck = (L + R.f + kChunk - 1) / kChunk;
  const Ring<T, 3, S> ring(ring_smem, w, lane);
  uint64_t ncut = 0;
  auto fetch = [&](int k, int stage) {
    const int t0 = k * kChunk + 8 * lane - R.f;
    if (p.vec && inside(R, k)) {
      const int64_t at = R.flat + t0;
      ring.copy(stage, 0, x + at);
      ring.copy(stage, 1, rg + at);
      ring.copy(stage, 2, ig + at);
    } else {
      Raw8<T> v;
      load_edge(x, R, t0, total, p.vec, v);
      ring.put(stage, 0, v);
      load_edge(rg, R, t0, total, p.vec, v);
      ring.put(stage, 1, v);
      load_edge(ig, R, t0, total, p.vec, v);
      ring.put(stage, 2, v);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int j = 0; j < S - 1; j++) fetch(w + j * W, j);
  if (RESET) ncut = load_resets(p, b, R, w * kChunk + 8 * lane - R.f);
  const Gate gr = gate_of(p.r_bias ? p.r_bias[d] : 0.f), gi = gate_of(p.i_bias ? p.i_bias[d] : 0.f);
  const float rate = decay_rate(p.c, p.lam[d]);
  float carry = p.h0 ? p.h0[row] : 0.f;  // the state that enters the round
  int buf = 0, stage = 0;
  const int rounds = (R.n_live + W - 1) / W;
  for (int it = 0; it < rounds; it++, buf ^= 1) {
    const int k = it * W + w;
    const bool in = inside(R, k);
    const int t0 = k * kChunk + 8 * lane - R.f;
    float2 a[4], bb[4], r[4], g[4];
    fetch(k + (S - 1) * W, stage == 0 ? S - 1 : stage - 1);  // into the slots of the round before
    cp_async_wait<S - 1>();
    {
      Raw8<T> v;
      ring.get(stage, 1, v);
      arguments(v, gr, r);
      ring.get(stage, 2, v);
      arguments(v, gi, g);
      ring.get(stage, 0, v);
      pairs(v, bb);
    }
    stage = stage == S - 1 ? 0 : stage + 1;
    const uint64_t cut = ncut;
    if (RESET) ncut = load_resets(p, b, R, t0 + W * kChunk);
    auto coefficients = [&](auto near) {
#pragma unroll
      for (int j = 0; j < 4; j++) {
        float2 eu, ev, sq, is;
        sigmoid2(r[j], g[j], r[j], g[j], eu, ev);
        decay<decltype(near)::value>(fma2(r[j], splat(rate), splat(kTiny)), a[j], sq, is);
        bb[j] = mul2(mul2(mul2(sq, is), g[j]), bb[j]);
      }
    };
    if (rate < kNear) coefficients(std::true_type());
    else coefficients(std::false_type());
    if (!in) {
#pragma unroll
      for (int e = 0; e < 8; e++)
        if (t0 + e < 0 || t0 + e >= R.len) elem(a, e) = 1.f, elem(bb, e) = 0.f;
    }
    float2 P2, H2;
    float P, H;
    Cuts c;
    if (RESET) c.lanes = __ballot_sync(kFull, cut != 0);
    const bool cuts = RESET && c.lanes;
    if (cuts) {
      c.bits = cut_bits(cut);
      compose<true>(c, a, bb, P2, H2);
      P = P2.y * P2.x;
      H = after(c.second(), P2.y, H2.x, H2.y);
      scan_up<true>(lane, c, P, H);
    } else {
      compose<false>(c, a, bb, P2, H2);
      P = P2.y * P2.x;
      H = fmaf(P2.y, H2.x, H2.y);
      scan_up<false>(lane, c, P, H);
    }
    float into = carry;  // the state that enters this warp's chunk
    if (W > 1) {
      if (lane == 31) {
        sP[buf][w] = RESET ? factor_of(c, P) : P;
        sH[buf][w] = H;
      }
      __syncthreads();  // two buffers: a warp can be one round ahead of the slowest reader, not two
      float x = carry;
#pragma unroll
      for (int v = 0; v < W; v++) {
        if (v == w) into = x;
        x = after(RESET && sP[buf][v] == 0.f, sP[buf][v], x, sH[buf][v]);
      }
      carry = x;
    }
    // the states of the two half runs, from the state that enters each
    const float Pe = __shfl_up_sync(kFull, P, 1), He = __shfl_up_sync(kFull, H, 1);
    float2 h;
    h.x = lane == 0 ? into : after(RESET && c.before(lane), Pe, into, He);
    h.y = after(RESET && c.first(), P2.x, h.x, H2.x);
    if (p.states && lane == 0 && k < n_ck) p.states[row * p.n_states + k] = into;
    if (cuts) {
#pragma unroll
      for (int j = 0; j < 4; j++) bb[j] = h = after2<true>(c, j, a[j], h, bb[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; j++) bb[j] = h = fma2(a[j], h, bb[j]);
    }
    if (W == 1) carry = __shfl_sync(kFull, h.y, 31);
    if (p.out && k < n_ck) {
      if (!in) {
#pragma unroll
        for (int e = 0; e < 8; e++)
          if (t0 + e >= R.len) elem(bb, e) = 0.f;
      }
      store_group(static_cast<Tout *>(p.out), R, in, t0, L, p.vec_out, bb);
    }
  }
  for (int k = rounds * W + w; k < n_ck; k += W) {  // behind the last live step
    const float2 none[4] = {};
    if (p.states && lane == 0) p.states[row * p.n_states + k] = carry;
    if (p.out) store_group(static_cast<Tout *>(p.out), R, false, k * kChunk + 8 * lane - R.f, L, p.vec_out, none);
  }
  if (p.h_last && threadIdx.x == 0) p.h_last[row] = carry;
}

// ---- backward ----------------------------------------------------------------------------------

// 16 warps an SM by their registers, of one to sixteen a row. (Eight a row with 138 registers and one CTA an SM: 1 x 256 x 65536
// forward and backward 123 us, with 128 and two 102 us.)
template <typename T, typename Tg, int W, bool RESET>
__global__ void __launch_bounds__(32 * W, W <= 8 ? 16 / W : 1) lru_bwd_kernel(const __grid_constant__ LruBwdParams q) {
  const LruParams &p = q.f;
  extern __shared__ __align__(16) char ring_smem[];
  constexpr int S = kStages<T, W>;
  __shared__ float sP[2][W], sM[2][W];
  __shared__ float sS[3][W];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t row = blockIdx.x;
  const int64_t b = row / p.Dn, d = row - b * p.Dn;
  const Row R = row_of(p, row, b);
  const int64_t total = p.Bt * p.Dn * p.L;
  const T *x = static_cast<const T *>(p.x), *rg = static_cast<const T *>(p.r), *ig = static_cast<const T *>(p.i);
  const T *dout = static_cast<const T *>(q.dout);
  const int L = (int)p.L, n_ck = (L + R.f + kChunk - 1) / kChunk, rounds = (R.n_live + W - 1) / W;
  float2 sum_q = splat(0.f), sum_r = splat(0.f), sum_i = splat(0.f);
  const Ring<T, 4, S> ring(ring_smem, w, lane);
  auto fetch = [&](int k, int stage) {
    const int t0 = k * kChunk + 8 * lane - R.f;
    if (k < 0) {
    } else if (p.vec && inside(R, k)) {
      const int64_t at = R.flat + t0;
      ring.copy(stage, 0, x + at);
      ring.copy(stage, 1, rg + at);
      ring.copy(stage, 2, ig + at);
      ring.copy(stage, 3, dout + at);
    } else {
      Raw8<T> v;
      load_edge(x, R, t0, total, p.vec, v);
      ring.put(stage, 0, v);
      load_edge(rg, R, t0, total, p.vec, v);
      ring.put(stage, 1, v);
      load_edge(ig, R, t0, total, p.vec, v);
      ring.put(stage, 2, v);
      load_edge(dout, R, t0, total, p.vec, v);
      ring.put(stage, 3, v);
    }
    cp_async_commit();
  };
  uint64_t ncut = 0;
  float nh = 0.f;
  auto fetch_small = [&](int k) {
    if (RESET) ncut = load_resets(p, b, R, k * kChunk + 8 * lane - R.f);
    if (k >= 0 && k < n_ck) nh = p.states[row * p.n_states + k];
  };
#pragma unroll
  for (int j = 0; j < S - 1; j++) fetch((rounds - 1 - j) * W + w, j);
  fetch_small((rounds - 1) * W + w);
  const Gate gr = gate_of(p.r_bias ? p.r_bias[d] : 0.f), gi = gate_of(p.i_bias ? p.i_bias[d] : 0.f);
  const float lam = p.lam[d];
  const float rate = decay_rate(p.c, lam);
  float carry = q.dh_last ? q.dh_last[row] : 0.f;  // mu arriving at the round's last step from behind
  int buf = 0, stage = 0;
  for (int it = rounds - 1; it >= 0; it--, buf ^= 1) {
    const int k = it * W + w;
    const bool in = inside(R, k);
    const int t0 = k * kChunk + 8 * lane - R.f;
    float2 a[4], ya[4], o[4], u[4], v[4], z[4], bb[4], dv[4];
    fetch(k - (S - 1) * W, stage == 0 ? S - 1 : stage - 1);  // into the slots of the round before
    cp_async_wait<S - 1>();
    {
      Raw8<T> raw;
      ring.get(stage, 1, raw);
      arguments(raw, gr, ya);
      ring.get(stage, 2, raw);
      arguments(raw, gi, v);
      ring.get(stage, 0, raw);
      pairs(raw, bb);
      ring.get(stage, 3, raw);
      pairs(raw, dv);
    }
    stage = stage == S - 1 ? 0 : stage + 1;
    const float hin = nh;
    const uint64_t cut = ncut;
    if (it > 0) fetch_small(k - W);
    auto coefficients = [&](auto near) {
#pragma unroll
      for (int j = 0; j < 4; j++) {
        float2 r, g, eu, ev, sq, is;
        sigmoid2(ya[j], v[j], r, g, eu, ev);
        o[j] = mul2(eu, r);                               // 1 - r
        const float2 y = fma2(r, splat(rate), splat(kTiny));
        decay<decltype(near)::value>(y, a[j], sq, is);
        ya[j] = mul2(y, a[j]);
        u[j] = mul2(mul2(sq, is), g);                     // m g
        bb[j] = mul2(bb[j], u[j]);                        // m g x
        v[j] = mul2(bb[j], mul2(ev, g));                  // b (1 - g)
        z[j] = mul2(mul2(mul2(mul2(ya[j], is), is), a[j]), bb[j]);  // y a^2 b / s
      }
    };
    if (rate < kNear) coefficients(std::true_type());
    else coefficients(std::false_type());
    if (!in) {
#pragma unroll
      for (int e = 0; e < 8; e++)
        if (t0 + e < 0 || t0 + e >= R.len) {
          elem(a, e) = 1.f;
          elem(bb, e) = elem(ya, e) = elem(o, e) = elem(u, e) = elem(v, e) = elem(z, e) = elem(dv, e) = 0.f;
        }
    }
    // the states' maps forwards, and mu -> S mu + M of what leaves the lane's first step backwards
    float2 P2, H2, M2 = splat(0.f);
    float P, H, S, M;
    Cuts c;
    if (RESET) c.lanes = __ballot_sync(kFull, cut != 0);
    const bool cuts = RESET && c.lanes;
    if (cuts) {
      c.bits = cut_bits(cut);
      compose<true>(c, a, bb, P2, H2);
#pragma unroll
      for (int j = 3; j >= 0; j--) M2 = after2<true>(c, j, a[j], add2(dv[j], M2), splat(0.f));
      P = S = P2.y * P2.x;
      H = after(c.second(), P2.y, H2.x, H2.y);
      M = after(c.first(), P2.x, M2.y, M2.x);
      scan_up<true>(lane, c, P, H);
      scan_down<true>(lane, c, S, M);
    } else {
      compose<false>(c, a, bb, P2, H2);
#pragma unroll
      for (int j = 3; j >= 0; j--) M2 = mul2(a[j], add2(dv[j], M2));
      P = S = P2.y * P2.x;
      H = fmaf(P2.y, H2.x, H2.y);
      M = fmaf(P2.x, M2.y, M2.x);
      scan_up<false>(lane, c, P, H);
      scan_down<false>(lane, c, S, M);
    }
    float into = carry;  // mu arriving behind this warp's chunk
    if (W > 1) {
      if (lane == 0) {
        sP[buf][w] = RESET ? factor_of(c, S) : S;
        sM[buf][w] = M;
      }
      __syncthreads();
      float x = carry;
#pragma unroll
      for (int o = W - 1; o >= 0; o--) {
        if (o == w) into = x;
        x = after(RESET && sP[buf][o] == 0.f, sP[buf][o], x, sM[buf][o]);
      }
      carry = x;
    }
    const float Pe = __shfl_up_sync(kFull, P, 1), He = __shfl_up_sync(kFull, H, 1);
    const float Se = __shfl_down_sync(kFull, S, 1), Me = __shfl_down_sync(kFull, M, 1);
    float2 h, mu;
    h.x = lane == 0 ? hin : after(RESET && c.before(lane), Pe, hin, He);
    h.y = after(RESET && c.first(), P2.x, h.x, H2.x);
    mu.y = lane == 31 ? into : after(RESET && c.behind(lane), Se, into, Me);
    mu.x = after(RESET && c.second(), P2.y, mu.y, M2.y);
#pragma unroll
    for (int j = 0; j < 4; j++) {  // -y (a h_{t-1} - a^2 b / s)
      z[j] = fma2(cuts ? after2<true>(c, j, ya[j], h, splat(0.f)) : mul2(ya[j], h), splat(-1.f), z[j]);
      h = cuts ? after2<true>(c, j, a[j], h, bb[j]) : fma2(a[j], h, bb[j]);
    }
#pragma unroll
    for (int j = 3; j >= 0; j--) {
      const float2 lm = add2(dv[j], mu);
      mu = cuts ? after2<true>(c, j, a[j], lm, splat(0.f)) : mul2(a[j], lm);
      u[j] = mul2(u[j], lm);
      v[j] = mul2(v[j], lm);
      bb[j] = mul2(z[j], lm);
      z[j] = mul2(bb[j], o[j]);
    }
    if (W == 1) carry = __shfl_sync(kFull, mu.x, 0);
    if (k >= n_ck) continue;
    if (!in) {  // steps outside the row hold 0 (0 times an infinite lambda would not be)
#pragma unroll
      for (int e = 0; e < 8; e++)
        if (t0 + e < 0 || t0 + e >= R.len) elem(u, e) = elem(v, e) = elem(z, e) = elem(bb, e) = 0.f;
    }
    if (q.dx) store_group(static_cast<Tg *>(q.dx), R, in, t0, L, q.vec_grad, u);
    if (q.di) store_group(static_cast<Tg *>(q.di), R, in, t0, L, q.vec_grad, v);
    if (q.dr) store_group(static_cast<Tg *>(q.dr), R, in, t0, L, q.vec_grad, z);
#pragma unroll
    for (int j = 0; j < 4; j++) {
      sum_q = add2(sum_q, bb[j]);
      sum_r = add2(sum_r, z[j]);
      sum_i = add2(sum_i, v[j]);
    }
  }
  for (int k = rounds * W + w; k < n_ck; k += W) {  // behind the last live step
    const float2 none[4] = {};
    const int t0 = k * kChunk + 8 * lane - R.f;
    if (q.dx) store_group(static_cast<Tg *>(q.dx), R, false, t0, L, q.vec_grad, none);
    if (q.di) store_group(static_cast<Tg *>(q.di), R, false, t0, L, q.vec_grad, none);
    if (q.dr) store_group(static_cast<Tg *>(q.dr), R, false, t0, L, q.vec_grad, none);
  }
  if (q.dh0 && threadIdx.x == 0) q.dh0[row] = carry;
  if (!q.p_dlam && !q.p_dr && !q.p_di) return;
  float sq = sum_q.x + sum_q.y, sr = sum_r.x + sum_r.y, si = sum_i.x + sum_i.y;
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) {
    sq += __shfl_xor_sync(kFull, sq, off);
    sr += __shfl_xor_sync(kFull, sr, off);
    si += __shfl_xor_sync(kFull, si, off);
  }
  if (W > 1) {
    if (lane == 0) sS[0][w] = sq, sS[1][w] = sr, sS[2][w] = si;
    __syncthreads();
    if (threadIdx.x != 0) return;
    sq = sr = si = 0.f;
    for (int o = 0; o < W; o++) sq += sS[0][o], sr += sS[1][o], si += sS[2][o];
  } else if (lane != 0) {
    return;
  }
  // sigmoid / softplus: 1 as lam -> -inf, where softplus reaches 0
  const float sp = softplus<true>(lam);
  if (q.p_dlam) q.p_dlam[row] = sq * (sp > 0.f ? sigmoid<true>(lam) / sp : 1.f);
  if (q.p_dr) q.p_dr[row] = sr;
  if (q.p_di) q.p_di[row] = si;
}

// ---- rows of up to 128 places ------------------------------------------------------------------

// G lanes a row (G a power of two, G * 8 places and more of them), 32 / G rows a warp, one group of 8 steps a lane:
// the same composition over G lanes instead of 32, without rounds. (A warp per row would leave lanes idle and be bound by the rate at
// which CTAs start: 8 x 5000 rows of 8 or 100 steps took 33 us forwards whatever their length.)
template <bool CUT> __device__ __forceinline__ void scan_up_group(int gl, int G, const Cuts &c, float &P, float &H) {
  const int last = CUT ? last_cut(c, gl) : 0;
  for (int off = 1; off < G; off <<= 1) scan_up_step<CUT>(gl, off, last, P, H);
}
template <bool CUT> __device__ __forceinline__ void scan_down_group(int gl, int G, const Cuts &c, float &S, float &M) {
  const unsigned next = CUT ? next_cut(c, gl) : 0;
  for (int off = 1; off < G; off <<= 1) scan_down_step<CUT>(gl, off, G, next, S, M);
}
// The cuts of a lane and of its group of G <= 16 lanes.
__device__ __forceinline__ Cuts group_cuts(uint64_t bytes, int gl, int G) {
  Cuts c;
  c.bits = cut_bits(bytes);
  c.lanes = __ballot_sync(kFull, c.bits != 0) >> ((threadIdx.x & 31) - gl) & ((1u << G) - 1);
  return c;
}

__device__ __forceinline__ int64_t batch_of(int64_t row, int64_t Dn) {
  return (row | Dn) >> 32 ? row / Dn : (int64_t)((uint32_t)row / (uint32_t)Dn);
}

template <typename T, typename Tout, bool RESET>
__global__ void __launch_bounds__(128) lru_fwd_short_kernel(const __grid_constant__ LruParams p, int lg) {
  const int G = 1 << lg, gl = threadIdx.x & (G - 1);
  const int64_t rows = p.Bt * p.Dn, id = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> lg;
  const bool live = id < rows;
  const int64_t row = live ? id : rows - 1;  // groups behind the last row follow along on it and store nothing
  const int64_t b = batch_of(row, p.Dn), d = row - b * p.Dn;
  const Row R = row_of(p, row, b);
  const int64_t total = rows * p.L;
  const int t0 = 8 * gl - R.f, L = (int)p.L;
  Raw8<T> rx, rr, ri;
  load_edge(static_cast<const T *>(p.x), R, t0, total, p.vec, rx);
  load_edge(static_cast<const T *>(p.r), R, t0, total, p.vec, rr);
  load_edge(static_cast<const T *>(p.i), R, t0, total, p.vec, ri);
  const uint64_t cut = RESET ? load_resets(p, b, R, t0) : 0;
  const Gate gr = gate_of(p.r_bias ? p.r_bias[d] : 0.f), gi = gate_of(p.i_bias ? p.i_bias[d] : 0.f);
  const float rate = decay_rate(p.c, p.lam[d]), h0 = p.h0 ? p.h0[row] : 0.f;
  float2 a[4], bb[4], r[4], g[4];
  arguments(rr, gr, r);
  arguments(ri, gi, g);
  pairs(rx, bb);
#pragma unroll
  for (int j = 0; j < 4; j++) {
    float2 eu, ev, sq, is;
    sigmoid2(r[j], g[j], r[j], g[j], eu, ev);
    decay<false>(fma2(r[j], splat(rate), splat(kTiny)), a[j], sq, is);
    bb[j] = mul2(mul2(mul2(sq, is), g[j]), bb[j]);
  }
  const bool in = t0 >= 0 && t0 + 8 <= R.len;
  if (!in) {
#pragma unroll
    for (int e = 0; e < 8; e++)
      if (t0 + e < 0 || t0 + e >= R.len) elem(a, e) = 1.f, elem(bb, e) = 0.f;
  }
  Cuts c;
  if (RESET) c = group_cuts(cut, gl, G);
  float2 P2, H2;
  compose<RESET>(c, a, bb, P2, H2);
  float P = P2.y * P2.x, H = after(RESET && c.second(), P2.y, H2.x, H2.y);
  scan_up_group<RESET>(gl, G, c, P, H);
  const float Pe = __shfl_up_sync(kFull, P, 1), He = __shfl_up_sync(kFull, H, 1);
  float2 h;
  h.x = gl == 0 ? h0 : after(RESET && c.before(gl), Pe, h0, He);
  h.y = after(RESET && c.first(), P2.x, h.x, H2.x);
#pragma unroll
  for (int j = 0; j < 4; j++) bb[j] = h = after2<RESET>(c, j, a[j], h, bb[j]);
  if (!live) return;
  if (p.states && gl == 0) p.states[row * p.n_states] = h0;
  if (p.h_last && gl == G - 1) p.h_last[row] = h.y;
  if (p.out) {
    if (!in) {
#pragma unroll
      for (int e = 0; e < 8; e++)
        if (t0 + e >= R.len) elem(bb, e) = 0.f;
    }
    store_group(static_cast<Tout *>(p.out), R, in, t0, L, p.vec_out, bb);
  }
}

// Five CTAs an SM: 8 x 5000 packed fp32 rows of 100, forward and backward 65.5 us; with the 108 registers that resets would take, and four, 69.5 us.
template <typename T, typename Tg, bool RESET>
__global__ void __launch_bounds__(128, 5) lru_bwd_short_kernel(const __grid_constant__ LruBwdParams q, int lg) {
  const LruParams &p = q.f;
  const int G = 1 << lg, gl = threadIdx.x & (G - 1);
  const int64_t rows = p.Bt * p.Dn, id = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> lg;
  const bool live = id < rows;
  const int64_t row = live ? id : rows - 1;
  const int64_t b = batch_of(row, p.Dn), d = row - b * p.Dn;
  const Row R = row_of(p, row, b);
  const int64_t total = rows * p.L;
  const int t0 = 8 * gl - R.f, L = (int)p.L;
  Raw8<T> rx, rr, ri, rd;
  load_edge(static_cast<const T *>(p.x), R, t0, total, p.vec, rx);
  load_edge(static_cast<const T *>(p.r), R, t0, total, p.vec, rr);
  load_edge(static_cast<const T *>(p.i), R, t0, total, p.vec, ri);
  load_edge(static_cast<const T *>(q.dout), R, t0, total, p.vec, rd);
  const uint64_t cut = RESET ? load_resets(p, b, R, t0) : 0;
  const Gate gr = gate_of(p.r_bias ? p.r_bias[d] : 0.f), gi = gate_of(p.i_bias ? p.i_bias[d] : 0.f);
  const float lam = p.lam[d];
  const float rate = decay_rate(p.c, lam);
  const float hin = p.states[row * p.n_states], behind = q.dh_last ? q.dh_last[row] : 0.f;
  float2 a[4], ya[4], o[4], u[4], v[4], z[4], bb[4], dv[4];
  arguments(rr, gr, ya);
  arguments(ri, gi, v);
  pairs(rx, bb);
  pairs(rd, dv);
#pragma unroll
  for (int j = 0; j < 4; j++) {
    float2 rg, g, eu, ev, sq, is;
    sigmoid2(ya[j], v[j], rg, g, eu, ev);
    o[j] = mul2(eu, rg);
    const float2 y = fma2(rg, splat(rate), splat(kTiny));
    decay<false>(y, a[j], sq, is);
    ya[j] = mul2(y, a[j]);
    u[j] = mul2(mul2(sq, is), g);
    bb[j] = mul2(bb[j], u[j]);
    v[j] = mul2(bb[j], mul2(ev, g));
    z[j] = mul2(mul2(mul2(mul2(ya[j], is), is), a[j]), bb[j]);
  }
  const bool in = t0 >= 0 && t0 + 8 <= R.len;
  if (!in) {
#pragma unroll
    for (int e = 0; e < 8; e++)
      if (t0 + e < 0 || t0 + e >= R.len) {
        elem(a, e) = 1.f;
        elem(bb, e) = elem(ya, e) = elem(o, e) = elem(u, e) = elem(v, e) = elem(z, e) = elem(dv, e) = 0.f;
      }
  }
  Cuts c;
  if (RESET) c = group_cuts(cut, gl, G);
  float2 P2, H2, M2 = splat(0.f);
  compose<RESET>(c, a, bb, P2, H2);
#pragma unroll
  for (int j = 3; j >= 0; j--) M2 = after2<RESET>(c, j, a[j], add2(dv[j], M2), splat(0.f));
  float P = P2.y * P2.x, S = P, H = after(RESET && c.second(), P2.y, H2.x, H2.y), M = after(RESET && c.first(), P2.x, M2.y, M2.x);
  scan_up_group<RESET>(gl, G, c, P, H);
  scan_down_group<RESET>(gl, G, c, S, M);
  const float Pe = __shfl_up_sync(kFull, P, 1), He = __shfl_up_sync(kFull, H, 1);
  const float Se = __shfl_down_sync(kFull, S, 1), Me = __shfl_down_sync(kFull, M, 1);
  float2 h, mu;
  h.x = gl == 0 ? hin : after(RESET && c.before(gl), Pe, hin, He);
  h.y = after(RESET && c.first(), P2.x, h.x, H2.x);
  mu.y = gl == G - 1 ? behind : after(RESET && c.behind(gl), Se, behind, Me);
  mu.x = after(RESET && c.second(), P2.y, mu.y, M2.y);
#pragma unroll
  for (int j = 0; j < 4; j++) {
    z[j] = fma2(after2<RESET>(c, j, ya[j], h, splat(0.f)), splat(-1.f), z[j]);  // -y (a h_{t-1} - a^2 b / s)
    h = after2<RESET>(c, j, a[j], h, bb[j]);
  }
#pragma unroll
  for (int j = 3; j >= 0; j--) {
    const float2 lm = add2(dv[j], mu);
    mu = after2<RESET>(c, j, a[j], lm, splat(0.f));
    u[j] = mul2(u[j], lm);
    v[j] = mul2(v[j], lm);
    bb[j] = mul2(z[j], lm);
    z[j] = mul2(bb[j], o[j]);
  }
  if (!in) {  // steps outside the row hold 0 (0 times an infinite lambda would not be)
#pragma unroll
    for (int e = 0; e < 8; e++)
      if (t0 + e < 0 || t0 + e >= R.len) elem(u, e) = elem(v, e) = elem(z, e) = elem(bb, e) = 0.f;
  }
  float2 sq2 = splat(0.f), sr2 = splat(0.f), si2 = splat(0.f);
#pragma unroll
  for (int j = 0; j < 4; j++) {
    sq2 = add2(sq2, bb[j]);
    sr2 = add2(sr2, z[j]);
    si2 = add2(si2, v[j]);
  }
  float sq = sq2.x + sq2.y, sr = sr2.x + sr2.y, si = si2.x + si2.y;
  for (int off = G / 2; off >= 1; off >>= 1) {
    sq += __shfl_xor_sync(kFull, sq, off);
    sr += __shfl_xor_sync(kFull, sr, off);
    si += __shfl_xor_sync(kFull, si, off);
  }
  if (!live) return;
  if (q.dx) store_group(static_cast<Tg *>(q.dx), R, in, t0, L, q.vec_grad, u);
  if (q.di) store_group(static_cast<Tg *>(q.di), R, in, t0, L, q.vec_grad, v);
  if (q.dr) store_group(static_cast<Tg *>(q.dr), R, in, t0, L, q.vec_grad, z);
  if (gl) return;
  if (q.dh0) q.dh0[row] = mu.x;
  const float sp = softplus<true>(lam);
  if (q.p_dlam) q.p_dlam[row] = sq * (sp > 0.f ? sigmoid<true>(lam) / sp : 1.f);
  if (q.p_dr) q.p_dr[row] = sr;
  if (q.p_di) q.p_di[row] = si;
}

// Per-row sums over the batch in a fixed order, eight loads in flight. blockIdx.y: dlam, dr_bias or di_bias.
__global__ void __launch_bounds__(128) lru_param_sum_kernel(const __grid_constant__ LruBwdParams q) {
  const int64_t d = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const float *src = blockIdx.y == 0 ? q.p_dlam : blockIdx.y == 1 ? q.p_dr : q.p_di;
  float *dst = blockIdx.y == 0 ? q.dlam : blockIdx.y == 1 ? q.dr_bias : q.di_bias;
  if (d >= q.f.Dn || !dst) return;
  float s = 0.f;
  for (int64_t b0 = 0; b0 < q.f.Bt; b0 += 8) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] = b0 + j < q.f.Bt ? src[(b0 + j) * q.f.Dn + d] : 0.f;
#pragma unroll
    for (int j = 0; j < 8; j++) s += v[j];
  }
  dst[d] = s;
}

// ---- one-token step ----------------------------------------------------------------------------

// V consecutive channels a thread (V = 4: Dn a multiple of 4 and every pointer on a vector boundary).
template <typename T, typename Tout, int V>
__global__ void __launch_bounds__(128) lru_step_kernel(const __grid_constant__ LruStepParams p) {
  const int64_t i0 = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * V;
  if (i0 >= p.Bt * p.Dn) return;
  const int64_t d = i0 % p.Dn;
  alignas(16) T x[V], r[V], g[V];
  alignas(16) float h[V], lam[V], rb[V], ib[V];
  alignas(16) Tout o[V];
  if constexpr (V == 4) {
    using V4 = typename std::conditional<sizeof(T) == 4, float4, uint2>::type;
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
  for (int e = 0; e < V; e += 2) {  // two channels a packed instruction (V = 1: the same one twice)
    const int f = V == 1 ? e : e + 1;
    float2 t = fma2(make_float2(to_f32(r[e]), to_f32(r[f])), splat(-kLog2e), mul2(make_float2(rb[e], rb[f]), splat(-kLog2e)));
    float2 n = fma2(make_float2(to_f32(g[e]), to_f32(g[f])), splat(-kLog2e), mul2(make_float2(ib[e], ib[f]), splat(-kLog2e)));
    float2 rr, gg, eu, ev, a, s, is;
    sigmoid2(make_float2(min_nan(t.x, 60.f), min_nan(t.y, 60.f)), make_float2(min_nan(n.x, 60.f), min_nan(n.y, 60.f)), rr, gg, eu, ev);
    decay<false>(fma2(make_float2(decay_rate(p.c, lam[e]), decay_rate(p.c, lam[f])), rr, splat(kTiny)), a, s, is);
    const float2 in = mul2(mul2(mul2(s, is), gg), make_float2(to_f32(x[e]), to_f32(x[f])));
    const float2 hn = fma2(a, make_float2(h[e], h[f]), in);
    h[e] = hn.x;
    h[f] = hn.y;
    o[e] = from_f32<Tout>(hn.x);
    o[f] = from_f32<Tout>(hn.y);
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

// Warps per row: one where the rows alone give every SM eight warps, else the fewest of 4, 8, 16 that do, and never many
// more than the row has chunks. (2 x 1536 x 2048: 15 us with one, 17.5 us with four; 1 x 256 x 65536: 42 us with eight, 49 us
// with sixteen.)
constexpr int64_t kWantWarps = 148 * 8;

int warps_per_row(int64_t rows, int64_t L) {
  const int64_t chunks = (L + 7 + kChunk - 1) / kChunk;
  if (chunks <= 2) return 1;
  int w = 1;
  while (w < kMaxWarps && rows * w < kWantWarps && w < chunks) w = w == 1 ? 4 : 2 * w;
  return w;
}

// Shared memory beyond the default 48 KB is asked for on the current device, at every launch.
template <typename K> cudaError_t allow_smem(K kernel, int bytes) {
  if (bytes <= 47 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

// Lanes per row of the short-row kernels, as a power of two; -1 for longer rows.
int short_lanes(int64_t L) {
  const int64_t groups = (L + (L % 8 ? 7 : 0) + 7) / 8;  // rows of whole groups start on one
  if (groups > 16) return -1;
  int lg = 0;
  while (1 << lg < groups) lg++;
  return lg;
}

template <typename T, typename Tout, int W>
cudaError_t fwd_w(const LruParams &p, cudaStream_t s) {
  const int64_t blocks = p.Bt * p.Dn;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const int smem = W * Ring<T, 3, kStages<T, W>>::kWarpBytes;
  const auto kernel = p.reset ? lru_fwd_kernel<T, Tout, W, true> : lru_fwd_kernel<T, Tout, W, false>;
  if (cudaError_t e = allow_smem(kernel, smem)) return e;
  kernel<<<(unsigned)blocks, 32 * W, smem, s>>>(p);
  return cudaGetLastError();
}

template <typename T, typename Tout> cudaError_t fwd_t(const LruParams &p, cudaStream_t s) {
  if (const int lg = short_lanes(p.L); lg >= 0) {
    const int64_t blocks = (((p.Bt * p.Dn) << lg) + 127) / 128;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const auto kernel = p.reset ? lru_fwd_short_kernel<T, Tout, true> : lru_fwd_short_kernel<T, Tout, false>;
    kernel<<<(unsigned)blocks, 128, 0, s>>>(p, lg);
    return cudaGetLastError();
  }
  switch (warps_per_row(p.Bt * p.Dn, p.L)) {
    case 1: return fwd_w<T, Tout, 1>(p, s);
    case 4: return fwd_w<T, Tout, 4>(p, s);
    case 8: return fwd_w<T, Tout, 8>(p, s);
    default: return fwd_w<T, Tout, 16>(p, s);
  }
}

template <typename T, typename Tg, int W>
cudaError_t bwd_w(const LruBwdParams &q, cudaStream_t s) {
  const int64_t blocks = q.f.Bt * q.f.Dn;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const int smem = W * Ring<T, 4, kStages<T, W>>::kWarpBytes;
  const auto kernel = q.f.reset ? lru_bwd_kernel<T, Tg, W, true> : lru_bwd_kernel<T, Tg, W, false>;
  if (cudaError_t e = allow_smem(kernel, smem)) return e;
  kernel<<<(unsigned)blocks, 32 * W, smem, s>>>(q);
  return cudaGetLastError();
}

template <typename T, typename Tg> cudaError_t bwd_t(const LruBwdParams &q, cudaStream_t s) {
  if (const int lg = short_lanes(q.f.L); lg >= 0) {
    const int64_t blocks = (((q.f.Bt * q.f.Dn) << lg) + 127) / 128;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const auto kernel = q.f.reset ? lru_bwd_short_kernel<T, Tg, true> : lru_bwd_short_kernel<T, Tg, false>;
    kernel<<<(unsigned)blocks, 128, 0, s>>>(q, lg);
    return cudaGetLastError();
  }
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
  lru_param_sum_kernel<<<dim3((unsigned)((q.f.Dn + 127) / 128), 3), 128, 0, s>>>(q);
  return cudaGetLastError();
}

cudaError_t launch_lru_step(const LruStepParams &p, int in_bf16, int out_bf16, cudaStream_t s) {
  if (in_bf16) return out_bf16 ? step_t<__nv_bfloat16, __nv_bfloat16>(p, s) : step_t<__nv_bfloat16, float>(p, s);
  return out_bf16 ? step_t<float, __nv_bfloat16>(p, s) : step_t<float, float>(p, s);
}

}  // namespace ssm
