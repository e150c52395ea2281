// ssm_api_ops.cu -- extern "C" entry points of the gated linear recurrence, of the normalisation and
// rotation of queries and keys, and of the state-space-dual step: host-side validation (synchronous,
// before any launch), workspace carving, dispatch. No exception crosses the ABI, no device memory
// is allocated.
#include <float.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "../../include/ssm_scan.h"
#include "ssm_api_util.h"
#include "ssm_internal.h"

namespace {

constexpr int64_t kMaxElems = INT64_C(1) << 50;
constexpr int64_t kMaxSteps = (INT64_C(1) << 31) - (1 << 15);  // the recurrence counts a row's steps in 32 bits

ssm_status cuda_status(cudaError_t e) { return (ssm_status)ssm::record_cuda_error_code(e); }

size_t rnd256(size_t x) { return (x + 255) & ~size_t(255); }

template <size_t n> bool all_aligned(const void *const (&ptrs)[n], size_t a) {
  for (const void *p : ptrs)
    if (p && !aligned(p, a)) return false;
  return true;
}

// ---- gated linear recurrence -------------------------------------------------------------------

ssm_status check_lru(const ssm_lru_args *a, bool need_out, bool *empty) {
  if (!a) return SSM_ERR_NULL;
  if (!dtype_ok(a->in_dtype) || (need_out && !dtype_ok(a->out_dtype))) return SSM_ERR_DTYPE;
  if (a->Bt < 0 || a->Dn <= 0 || a->L < 0) return SSM_ERR_SHAPE;
  if (!(a->c > 0.f) || !isfinite(a->c) || a->L >= kMaxSteps) return SSM_ERR_UNSUPPORTED;
  int64_t rows, elems;
  if (!mul_ok(a->Bt, a->Dn, &rows) || !mul_ok(rows, a->L, &elems) || elems > kMaxElems || rows > kMaxElems)
    return SSM_ERR_SHAPE;
  const void *const f32[6] = {a->lam, a->r_bias, a->i_bias, a->h0, a->chunk_states, a->h_last};
  if (!all_aligned(f32, 4) || !aligned(a->lengths, 4)) return SSM_ERR_ALIGN;
  *empty = a->Bt == 0 || a->L == 0;
  if (*empty) return SSM_OK;
  if (!a->x || !a->r || !a->i || !a->lam || (need_out && !a->out)) return SSM_ERR_NULL;
  const void *const in[3] = {a->x, a->r, a->i};
  if (!all_aligned(in, dtype_size(a->in_dtype))) return SSM_ERR_ALIGN;
  if (need_out && !aligned(a->out, dtype_size(a->out_dtype))) return SSM_ERR_ALIGN;
  return SSM_OK;
}

ssm::LruParams lru_params(const ssm_lru_args *a) {
  ssm::LruParams p;
  memset(&p, 0, sizeof(p));
  p.x = a->x;
  p.r = a->r;
  p.i = a->i;
  p.lam = a->lam;
  p.r_bias = a->r_bias;
  p.i_bias = a->i_bias;
  p.h0 = a->h0;
  p.reset = a->reset;
  p.lengths = a->lengths;
  p.Bt = a->Bt;
  p.Dn = a->Dn;
  p.L = a->L;
  p.n_states = ssm_lru_num_states(a->L);
  p.c = a->c;
  p.vec = aligned(a->x, 16) && aligned(a->r, 16) && aligned(a->i, 16);
  return p;
}

// dst = src or 0, n floats.
cudaError_t copy_or_zero(float *dst, const float *src, size_t n, cudaStream_t s) {
  if (!dst || dst == src || n == 0) return cudaSuccess;
  return src ? cudaMemcpyAsync(dst, src, n * sizeof(float), cudaMemcpyDeviceToDevice, s)
             : cudaMemsetAsync(dst, 0, n * sizeof(float), s);
}

ssm_status check_lru_bwd(const ssm_lru_bwd_args *a, bool *empty) {
  if (!a) return SSM_ERR_NULL;
  const ssm_status st = check_lru(&a->fwd, false, empty);
  if (st != SSM_OK) return st;
  if (!dtype_ok(a->grad_dtype)) return SSM_ERR_DTYPE;
  const void *const f32[5] = {a->dh_last, a->dlam, a->dr_bias, a->di_bias, a->dh0};
  if (!all_aligned(f32, 4)) return SSM_ERR_ALIGN;
  const void *const g[3] = {a->dx, a->dr, a->di};
  if (!all_aligned(g, dtype_size(a->grad_dtype))) return SSM_ERR_ALIGN;
  if (*empty) return SSM_OK;
  if (!a->dout) return SSM_ERR_NULL;
  if (!aligned(a->dout, dtype_size(a->fwd.in_dtype))) return SSM_ERR_ALIGN;
  return SSM_OK;
}

size_t lru_sums_bytes(const ssm_lru_bwd_args *a) {  // one (Bt, Dn) array per wanted parameter gradient
  return a->fwd.Bt > 1 ? rnd256(sizeof(float) * (size_t)(a->fwd.Bt * a->fwd.Dn)) : 0;
}
size_t lru_states_bytes(const ssm_lru_bwd_args *a) {
  return a->fwd.chunk_states
             ? 0
             : rnd256(sizeof(float) * (size_t)(a->fwd.Bt * a->fwd.Dn * ssm_lru_num_states(a->fwd.L)));
}
size_t lru_bwd_bytes(const ssm_lru_bwd_args *a) {
  const int wanted = (a->dlam != nullptr) + (a->dr_bias != nullptr) + (a->di_bias != nullptr);
  return lru_states_bytes(a) + wanted * lru_sums_bytes(a);
}

// ---- queries and keys --------------------------------------------------------------------------

struct Axis {
  int64_t n, stride;
};

// Whether no two elements of a tensor with these axes share a place, found by nesting the axes in the order of their strides.
bool disjoint(Axis (&ax)[4]) {
  for (int i = 0; i < 4; i++)
    for (int j = i + 1; j < 4; j++)
      if (ax[j].stride < ax[i].stride) {
        const Axis t = ax[i];
        ax[i] = ax[j];
        ax[j] = t;
      }
  int64_t reach = 1;  // places that the axes so far cover
  for (const Axis &x : ax) {
    if (x.n <= 1) continue;
    if (x.stride < reach) return false;
    int64_t more;
    if (!mul_ok(x.stride, x.n - 1, &more) || more > kMaxElems) return false;
    reach += more;
  }
  return true;
}

bool qk_disjoint(const ssm_qk_args *a, int64_t H, int64_t sb, int64_t sh, int64_t sr) {
  const bool time = a->layout == SSM_QK_TIME_LAST;
  Axis ax[4] = {{a->Bt, sb}, {H, sh}, {time ? a->D : a->L, sr}, {time ? a->L : a->D, 1}};
  return disjoint(ax);
}

ssm_status check_qk(const ssm_qk_args *a, bool bwd, bool *empty) {
  if (!a) return SSM_ERR_NULL;
  if (!dtype_ok(a->in_dtype) || (!bwd && !dtype_ok(a->out_dtype))) return SSM_ERR_DTYPE;
  if (a->Bt < 0 || a->L < 0 || a->Hq < 0 || a->Hk < 0 || a->D <= 0) return SSM_ERR_SHAPE;
  if (a->rot < 0 || a->rot > a->D || a->rot % 2 != 0) return SSM_ERR_SHAPE;
  if (a->D > ssm::kQkMaxDim) return SSM_ERR_UNSUPPORTED;
  if (a->layout != SSM_QK_STATE_LAST && a->layout != SSM_QK_TIME_LAST) return SSM_ERR_UNSUPPORTED;
  if (!(a->eps >= 0.f) || (!a->norm && (a->q_weight || a->k_weight))) return SSM_ERR_UNSUPPORTED;
  int64_t tokens, heads, elems;
  if (a->Hq > (1 << 24) || a->Hk > (1 << 24) || a->Bt > 0x7fffffff || a->L > 0x7fffff00 || !mul_ok(a->Bt, a->L, &tokens) ||
      !mul_ok(tokens, a->Hq + a->Hk, &heads) || !mul_ok(heads, a->D, &elems) || elems > kMaxElems || tokens > kMaxElems)
    return SSM_ERR_SHAPE;
  if (!aligned(a->q_weight, 4) || !aligned(a->k_weight, 4) || !aligned(a->inv_freq, a->freq_f64 ? 8 : 4) ||
      !aligned(a->positions, a->pos_i64 ? 8 : 4))
    return SSM_ERR_ALIGN;
  *empty = a->Bt == 0 || a->L == 0 || a->Hq + a->Hk == 0;
  if (*empty) return SSM_OK;
  if (a->rot > 0 && !a->inv_freq) return SSM_ERR_NULL;
  const size_t ei = dtype_size(a->in_dtype), eo = bwd ? 1 : dtype_size(a->out_dtype);
  if (a->Hq > 0) {
    if ((!a->q && (!bwd || a->norm)) || (!bwd && !a->q_out)) return SSM_ERR_NULL;
    if (!aligned(a->q, ei) || (!bwd && !aligned(a->q_out, eo))) return SSM_ERR_ALIGN;
    if (!bwd && !qk_disjoint(a, a->Hq, a->q_out_sb, a->q_out_sh, a->q_out_sr)) return SSM_ERR_SHAPE;
  }
  if (a->Hk > 0) {
    if ((!a->k && (!bwd || a->norm)) || (!bwd && !a->k_out)) return SSM_ERR_NULL;
    if (!aligned(a->k, ei) || (!bwd && !aligned(a->k_out, eo))) return SSM_ERR_ALIGN;
    if (!bwd && !qk_disjoint(a, a->Hk, a->k_out_sb, a->k_out_sh, a->k_out_sr)) return SSM_ERR_SHAPE;
  }
  return SSM_OK;
}

ssm::QkTensor tensor(const void *p, int64_t sb, int64_t sh, int64_t sr, int32_t dtype) {
  return {const_cast<void *>(p), sb, sh, sr, dtype == SSM_BF16};
}

ssm::QkParams qk_params(const ssm_qk_args *a) {
  ssm::QkParams p;
  memset(&p, 0, sizeof(p));
  p.in[0] = tensor(a->q, a->q_sb, a->q_sh, a->q_sr, a->in_dtype);
  p.in[1] = tensor(a->k, a->k_sb, a->k_sh, a->k_sr, a->in_dtype);
  p.w[0] = a->q_weight;
  p.w[1] = a->k_weight;
  p.inv_freq = a->inv_freq;
  p.pos = a->positions;
  p.pos0 = a->pos0;
  p.Bt = a->Bt;
  p.L = a->L;
  p.H[0] = (int)a->Hq;
  p.H[1] = (int)a->Hk;
  p.D = (int)a->D;
  p.rot = (int)a->rot;
  p.freq_f64 = a->freq_f64 != 0;
  p.pos_i64 = a->pos_i64 != 0;
  p.interleaved = a->interleaved != 0;
  p.norm = a->norm != 0;
  p.time_last = a->layout == SSM_QK_TIME_LAST;
  // a reciprocal root of 2^63 at most: its square is finite in fp32, and a subnormal mean square never stands alone under a root that flushes it
  p.eps = a->eps > FLT_MIN ? a->eps : FLT_MIN;
  p.rot_scale = a->rot_scale;
  p.inv_D = 1.f / (float)a->D;
  return p;
}

// Time innermost: the most elements (8, 4, 2 or 1) that the strides and the addresses of both sides are multiples of, and L of 4 at
// least with 8, of as many otherwise: a row's last run is then whole pieces of 4, 2 or 1.
int qk_time_run(const ssm::QkParams &p) {
  for (int V = 8; V > 1; V /= 2) {
    bool fits = p.L % (V < 4 ? V : 4) == 0;
    for (int s = 0; s < 2 && fits; s++) {
      if (p.H[s] == 0) continue;
      for (const ssm::QkTensor *t : {&p.in[s], &p.out[s], &p.dout[s]}) {
        const size_t bytes = (size_t)V * (t->bf16 ? 2 : 4);
        if (t->p && (!aligned(t->p, bytes < 16 ? bytes : 16) || (p.Bt > 1 && t->sb % V) || (p.H[s] > 1 && t->sh % V) ||
                     (p.D > 1 && t->sr % V)))
          fits = false;
      }
    }
    if (fits) return V;
  }
  return 1;
}

ssm_status check_qk_bwd(const ssm_qk_bwd_args *a, bool *empty) {
  if (!a) return SSM_ERR_NULL;
  const ssm_qk_args *f = &a->fwd;
  const ssm_status st = check_qk(f, true, empty);
  if (st != SSM_OK) return st;
  if (!dtype_ok(a->dout_dtype) || !dtype_ok(a->grad_dtype)) return SSM_ERR_DTYPE;
  if (!f->norm && (a->dq_weight || a->dk_weight)) return SSM_ERR_UNSUPPORTED;
  if (!aligned(a->dq_weight, 4) || !aligned(a->dk_weight, 4)) return SSM_ERR_ALIGN;
  if (*empty) return SSM_OK;
  const size_t ed = dtype_size(a->dout_dtype), eg = dtype_size(a->grad_dtype);
  if (f->Hq > 0) {
    if (!a->dq_out) return SSM_ERR_NULL;
    if (!aligned(a->dq_out, ed) || !aligned(a->dq, eg)) return SSM_ERR_ALIGN;
    if (a->dq && !qk_disjoint(f, f->Hq, a->dq_sb, a->dq_sh, a->dq_sr)) return SSM_ERR_SHAPE;
  }
  if (f->Hk > 0) {
    if (!a->dk_out) return SSM_ERR_NULL;
    if (!aligned(a->dk_out, ed) || !aligned(a->dk, eg)) return SSM_ERR_ALIGN;
    if (a->dk && !qk_disjoint(f, f->Hk, a->dk_sb, a->dk_sh, a->dk_sr)) return SSM_ERR_SHAPE;
  }
  return SSM_OK;
}

ssm::QkParams qk_bwd_params(const ssm_qk_bwd_args *a) {
  const ssm_qk_args *f = &a->fwd;
  ssm::QkParams p = qk_params(f);
  if (!p.norm) p.in[0].p = p.in[1].p = nullptr;  // not read
  p.dout[0] = tensor(a->dq_out, f->q_out_sb, f->q_out_sh, f->q_out_sr, a->dout_dtype);
  p.dout[1] = tensor(a->dk_out, f->k_out_sb, f->k_out_sh, f->k_out_sr, a->dout_dtype);
  p.out[0] = tensor(a->dq, a->dq_sb, a->dq_sh, a->dq_sr, a->grad_dtype);
  p.out[1] = tensor(a->dk, a->dk_sb, a->dk_sh, a->dk_sr, a->grad_dtype);
  p.dw[0] = f->Hq > 0 ? a->dq_weight : nullptr;
  p.dw[1] = f->Hk > 0 ? a->dk_weight : nullptr;
  p.vec = p.time_last ? qk_time_run(p) : 0;
  return p;
}

// ---- state-space-dual step ---------------------------------------------------------------------

ssm_status check_ssd_step(const ssm_ssd_step_args *a, bool *empty) {
  if (!a) return SSM_ERR_NULL;
  if (!dtype_ok(a->in_dtype) || !dtype_ok(a->out_dtype)) return SSM_ERR_DTYPE;
  if (a->discretization != SSM_ZOH && a->discretization != SSM_EULER) return SSM_ERR_UNSUPPORTED;
  if (a->Bt < 0 || a->H <= 0 || a->P <= 0 || a->N <= 0) return SSM_ERR_SHAPE;
  if (a->P > 256 || a->N > 256) return SSM_ERR_UNSUPPORTED;
  int64_t heads;
  if (!mul_ok(a->Bt, a->H, &heads) || heads > (INT64_C(1) << 40)) return SSM_ERR_SHAPE;
  *empty = a->Bt == 0;
  if (*empty) return SSM_OK;
  if (!a->x || !a->dt || !a->A_log || !a->B || !a->C || !a->h || !a->out) return SSM_ERR_NULL;
  const void *const in[4] = {a->x, a->dt, a->B, a->C};
  const void *const f32[4] = {a->dt_bias, a->A_log, a->D, a->h};
  if (!all_aligned(in, dtype_size(a->in_dtype)) || !all_aligned(f32, 4) || !aligned(a->out, dtype_size(a->out_dtype)))
    return SSM_ERR_ALIGN;
  return SSM_OK;
}

}  // namespace

extern "C" {

// 256 steps a state; a row that starts inside a group of 8 elements covers up to 7 more places.
int64_t ssm_lru_num_states(int64_t L) { return L <= 0 ? 0 : (L + 7 + 255) / 256; }

ssm_status ssm_lru_fwd(const ssm_lru_args *args, void *stream) {
  SSM_RANGE("ssm_lru_fwd");
  bool empty = false;
  const ssm_status st = check_lru(args, true, &empty);
  if (st != SSM_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (empty) return cuda_status(copy_or_zero(args->h_last, args->h0, (size_t)(args->Bt * args->Dn), s));
  ssm::LruParams p = lru_params(args);
  p.out = args->out;
  p.states = args->chunk_states;
  p.h_last = args->h_last;
  p.vec_out = aligned(args->out, 16);
  return cuda_status(ssm::launch_lru_fwd(p, args->in_dtype == SSM_BF16, args->out_dtype == SSM_BF16, s));
}

size_t ssm_lru_bwd_workspace_size(const ssm_lru_bwd_args *args) {
  bool empty = false;
  if (check_lru_bwd(args, &empty) != SSM_OK || empty) return 0;
  return lru_bwd_bytes(args);
}

ssm_status ssm_lru_bwd(const ssm_lru_bwd_args *args, void *stream) {
  SSM_RANGE("ssm_lru_bwd");
  bool empty = false;
  const ssm_status st = check_lru_bwd(args, &empty);
  if (st != SSM_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const ssm_lru_args *a = &args->fwd;
  if (empty) {
    cudaError_t e = copy_or_zero(args->dh0, args->dh_last, (size_t)(a->Bt * a->Dn), s);
    float *const sums[3] = {args->dlam, args->dr_bias, args->di_bias};
    for (float *g : sums)
      if (e == cudaSuccess) e = copy_or_zero(g, nullptr, (size_t)a->Dn, s);
    return cuda_status(e);
  }
  const size_t need = lru_bwd_bytes(args);
  if (need && (!args->workspace || args->workspace_bytes < need || !aligned(args->workspace, 256)))
    return SSM_ERR_WORKSPACE;
  char *ws = static_cast<char *>(args->workspace);
  ssm::LruBwdParams q;
  memset(&q, 0, sizeof(q));
  q.f = lru_params(a);
  if (a->chunk_states) {
    q.f.states = a->chunk_states;
  } else {  // the forward without its outputs
    q.f.states = reinterpret_cast<float *>(ws);
    ws += lru_states_bytes(args);
    const cudaError_t e = ssm::launch_lru_fwd(q.f, a->in_dtype == SSM_BF16, 0, s);
    if (e != cudaSuccess) return cuda_status(e);
  }
  q.f.vec = q.f.vec && aligned(args->dout, 16);
  q.dout = args->dout;
  q.dx = args->dx;
  q.dr = args->dr;
  q.di = args->di;
  q.vec_grad = aligned(args->dx, 16) && aligned(args->dr, 16) && aligned(args->di, 16);
  q.dh_last = args->dh_last;
  q.dh0 = args->dh0;
  q.dlam = args->dlam;
  q.dr_bias = args->dr_bias;
  q.di_bias = args->di_bias;
  float *const sums[3] = {args->dlam, args->dr_bias, args->di_bias};
  float **const parts[3] = {&q.p_dlam, &q.p_dr, &q.p_di};
  for (int j = 0; j < 3; j++) {
    if (!sums[j]) continue;
    *parts[j] = a->Bt > 1 ? reinterpret_cast<float *>(ws) : sums[j];
    ws += lru_sums_bytes(args);
  }
  return cuda_status(ssm::launch_lru_bwd(q, a->in_dtype == SSM_BF16, args->grad_dtype == SSM_BF16, s));
}

ssm_status ssm_lru_step(const ssm_lru_step_args *a, void *stream) {
  SSM_RANGE("ssm_lru_step");
  if (!a) return SSM_ERR_NULL;
  if (!dtype_ok(a->in_dtype) || !dtype_ok(a->out_dtype)) return SSM_ERR_DTYPE;
  if (a->Bt < 0 || a->Dn <= 0) return SSM_ERR_SHAPE;
  if (!(a->c > 0.f) || !isfinite(a->c)) return SSM_ERR_UNSUPPORTED;
  int64_t rows;
  if (!mul_ok(a->Bt, a->Dn, &rows) || rows > (INT64_C(1) << 38)) return SSM_ERR_SHAPE;
  if (a->Bt == 0) return SSM_OK;
  if (!a->x || !a->r || !a->i || !a->lam || !a->h || !a->out) return SSM_ERR_NULL;
  const size_t ei = dtype_size(a->in_dtype), eo = dtype_size(a->out_dtype);
  const void *const in[3] = {a->x, a->r, a->i};
  const void *const f32[4] = {a->lam, a->r_bias, a->i_bias, a->h};
  if (!all_aligned(in, ei) || !all_aligned(f32, 4) || !aligned(a->out, eo)) return SSM_ERR_ALIGN;
  ssm::LruStepParams p;
  memset(&p, 0, sizeof(p));
  p.x = a->x;
  p.r = a->r;
  p.i = a->i;
  p.lam = a->lam;
  p.r_bias = a->r_bias;
  p.i_bias = a->i_bias;
  p.h = a->h;
  p.out = a->out;
  p.Bt = a->Bt;
  p.Dn = a->Dn;
  p.c = a->c;
  p.vec = a->Dn % 4 == 0 && all_aligned(in, 4 * ei) && all_aligned(f32, 16) && aligned(a->out, 4 * eo);
  return cuda_status(ssm::launch_lru_step(p, a->in_dtype == SSM_BF16, a->out_dtype == SSM_BF16,
                                          static_cast<cudaStream_t>(stream)));
}

ssm_status ssm_qk_norm_rope_fwd(const ssm_qk_args *args, void *stream) {
  SSM_RANGE("ssm_qk_norm_rope_fwd");
  bool empty = false;
  const ssm_status st = check_qk(args, false, &empty);
  if (st != SSM_OK || empty) return st;
  ssm::QkParams p = qk_params(args);
  p.out[0] = tensor(args->q_out, args->q_out_sb, args->q_out_sh, args->q_out_sr, args->out_dtype);
  p.out[1] = tensor(args->k_out, args->k_out_sb, args->k_out_sh, args->k_out_sr, args->out_dtype);
  p.vec = p.time_last ? qk_time_run(p) : 0;
  return cuda_status(ssm::launch_qk_fwd(p, args->in_dtype == SSM_BF16, static_cast<cudaStream_t>(stream)));
}

size_t ssm_qk_norm_rope_bwd_workspace_size(const ssm_qk_bwd_args *args) {
  bool empty = false;
  if (check_qk_bwd(args, &empty) != SSM_OK || empty) return 0;
  return ssm::qk_bwd_workspace_bytes(qk_bwd_params(args));
}

ssm_status ssm_qk_norm_rope_bwd(const ssm_qk_bwd_args *args, void *stream) {
  SSM_RANGE("ssm_qk_norm_rope_bwd");
  bool empty = false;
  const ssm_status st = check_qk_bwd(args, &empty);
  if (st != SSM_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  float *const dw[2] = {args->dq_weight, args->dk_weight};
  const int64_t H[2] = {args->fwd.Hq, args->fwd.Hk};
  ssm::QkParams p = qk_bwd_params(args);
  if (!empty) {
    const size_t need = ssm::qk_bwd_workspace_bytes(p);
    if (need && (!args->workspace || args->workspace_bytes < need || !aligned(args->workspace, 256)))
      return SSM_ERR_WORKSPACE;
  }
  for (int j = 0; j < 2; j++)  // a side without rows
    if (empty || H[j] == 0) {
      const cudaError_t e = copy_or_zero(dw[j], nullptr, (size_t)args->fwd.D, s);
      if (e != cudaSuccess) return cuda_status(e);
    }
  if (empty) return SSM_OK;
  p.part = static_cast<float *>(args->workspace);
  return cuda_status(ssm::launch_qk_bwd(p, args->fwd.in_dtype == SSM_BF16, s));
}

ssm_status ssm_ssd_step(const ssm_ssd_step_args *args, void *stream) {
  SSM_RANGE("ssm_ssd_step");
  bool empty = false;
  const ssm_status st = check_ssd_step(args, &empty);
  if (st != SSM_OK || empty) return st;
  ssm::SsdStepParams p;
  memset(&p, 0, sizeof(p));
  p.x = args->x;
  p.dt = args->dt;
  p.dt_bias = args->dt_bias;
  p.A_log = args->A_log;
  p.B = args->B;
  p.C = args->C;
  p.D = args->D;
  p.h = args->h;
  p.out = args->out;
  p.Bt = args->Bt;
  p.H = args->H;
  p.P = args->P;
  p.N = args->N;
  p.delta_softplus = args->delta_softplus != 0;
  p.euler = args->discretization == SSM_EULER;
  p.vec = args->P % 4 == 0 && aligned(args->h, 16);
  return cuda_status(ssm::launch_ssd_step(p, args->in_dtype == SSM_BF16, args->out_dtype == SSM_BF16,
                                          static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
