// kda_api_block.cu -- the extern "C" entry points of what stands around the recurrent core:
// selective scan (prompts and step), draft verification, block norm (see include/kda.h).
// As in kda_api.cu every argument is validated before anything is enqueued.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdio>

#include "../../include/kda.h"
#include "kda_internal.h"

namespace {

kda_status fail(kda_status s, const char *who, const char *what) {
  char buf[256];
  std::snprintf(buf, sizeof buf, "%s: %s", who, what);
  kda::set_last_error(buf);
  return s;
}
kda_status done(cudaError_t e, const char *who) {
  if (e != cudaSuccess) return fail(KDA_ERR_CUDA, who, cudaGetErrorString(e));
  kda::set_last_error("");
  return KDA_OK;
}
bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool have(const void *p, size_t a) { return p && aligned(p, a); }   // required
bool fine(const void *p, size_t a) { return !p || aligned(p, a); }  // optional
bool io_ok(int io) { return io == KDA_BF16 || io == KDA_F32; }

// Head geometry shared by the scan's two calls.
kda_status check_heads(int heads, int groups, int head_dim, int d_state, int io, const char *who) {
  if (!io_ok(io)) return fail(KDA_ERR_UNSUPPORTED, who, "io_dtype must be KDA_BF16 or KDA_F32");
  if ((head_dim != 64 && head_dim != 128) || d_state != kda::SSM_N)
    return fail(KDA_ERR_UNSUPPORTED, who, "head_dim must be 64 or 128 and d_state 128");
  if (heads < 1 || heads > 65536 || groups < 1 || heads % groups != 0)
    return fail(KDA_ERR_INVALID_ARG, who, "need 1 <= heads <= 65536 and groups a divisor of heads");
  return KDA_OK;
}

kda_status check_ssm(const kda_ssm_args *a, const char *who) {
  if (!a) return fail(KDA_ERR_INVALID_ARG, who, "args is NULL");
  const kda_status st = check_heads(a->heads, a->groups, a->head_dim, a->d_state, a->io_dtype, who);
  if (st != KDA_OK) return st;
  if (a->n_seqs < 0 || a->n_seqs > 65535 || a->total_tokens < 0 || a->total_tokens > 0x7fffffffLL)
    return fail(KDA_ERR_INVALID_ARG, who, "need 0 <= n_seqs <= 65535 and 0 <= total_tokens < 2^31");
  if (a->n_seqs == 0 && a->total_tokens > 0) return fail(KDA_ERR_INVALID_ARG, who, "tokens without sequences");
  if ((int64_t)a->n_seqs * a->heads * (a->head_dim / kda::SSM_COLS) >= (a->io_dtype == KDA_F32 ? 1LL << 31 : kda::SSM_TC_ITEMS))
    return fail(KDA_ERR_UNSUPPORTED, who, "n_seqs * heads * head_dim / 64 must be below 2^30 (fp32 I/O: 2^31)");
  if (!a->cu_seqlens && a->n_seqs > 0 && a->total_tokens % a->n_seqs != 0)
    return fail(KDA_ERR_INVALID_ARG, who, "without cu_seqlens total_tokens must divide into n_seqs equal sequences");
  if (!fine(a->cu_seqlens, 4) || !fine(a->dev_status, 4)) return fail(KDA_ERR_INVALID_ARG, who, "an int32 array is misaligned");
  const int64_t wx = (int64_t)a->heads * a->head_dim, wb = (int64_t)a->groups * a->d_state;
  if (a->ldx < wx || a->ldb < wb || a->ldc < wb || a->ldx % 8 || a->ldb % 8 || a->ldc % 8)
    return fail(KDA_ERR_INVALID_ARG, who, "row strides must be multiples of 8 and cover a row");
  if (a->ldx > (1LL << 31) || a->ldb > (1LL << 31) || a->ldc > (1LL << 31))
    return fail(KDA_ERR_INVALID_ARG, who, "row strides must be at most 2^31");
  if (a->total_tokens > 0 && (!have(a->x, 16) || !have(a->b, 16) || !have(a->c, 16) || !have(a->y, 16) || !have(a->dt, 4)))
    return fail(KDA_ERR_INVALID_ARG, who, "x, b, c, dt and y are required and aligned");
  if (a->n_seqs > 0 && !have(a->a, 4)) return fail(KDA_ERR_INVALID_ARG, who, "a is NULL or misaligned");
  if (!fine(a->dt_bias, 4) || !fine(a->d_skip, 4) || !fine(a->h0, 16) || !fine(a->hT, 16))
    return fail(KDA_ERR_INVALID_ARG, who, "dt_bias, d_skip, h0 or hT is misaligned");
  return KDA_OK;
}

kda::SsmParams ssm_params(const kda_ssm_args *a) {
  kda::SsmParams p{};
  p.n_seqs = a->n_seqs;
  p.H = a->heads;
  p.G = a->groups;
  p.P = a->head_dim;
  p.T = a->total_tokens;
  p.softplus = a->dt_softplus != 0;
  p.cu = a->cu_seqlens;
  p.x = a->x, p.b = a->b, p.c = a->c;
  p.ldx = a->ldx, p.ldb = a->ldb, p.ldc = a->ldc;
  p.dt = a->dt, p.a = a->a, p.dt_bias = a->dt_bias, p.d_skip = a->d_skip, p.h0 = a->h0;
  p.y = a->y;
  p.hT = a->hT;
  p.status = a->dev_status;
  return p;
}

size_t ssm_step_channels(const kda_ssm_step_args *a) {
  return (size_t)a->heads * a->head_dim + (size_t)2 * a->groups * a->d_state;
}

kda_status check_norm(const kda_block_norm_args *a, const char *who) {
  if (!a) return fail(KDA_ERR_INVALID_ARG, who, "args is NULL");
  if (!io_ok(a->io_dtype)) return fail(KDA_ERR_UNSUPPORTED, who, "io_dtype must be KDA_BF16 or KDA_F32");
  if (a->dim < 8 || a->dim > 16384 || a->dim % 8) return fail(KDA_ERR_UNSUPPORTED, who, "dim must be a multiple of 8 in 8..16384");
  if (a->rows < 0 || a->rows > 0x7fffffffLL) return fail(KDA_ERR_INVALID_ARG, who, "need 0 <= rows < 2^31");
  if (!(a->eps > 0.f)) return fail(KDA_ERR_INVALID_ARG, who, "eps must be positive");
  if (a->gate && a->gate_act != KDA_GATE_SIGMOID && a->gate_act != KDA_GATE_SILU)
    return fail(KDA_ERR_INVALID_ARG, who, "gate_act must be KDA_GATE_SIGMOID or KDA_GATE_SILU");
  if (!fine(a->w_post, 16) || !fine(a->scale, 16) || !fine(a->w_pre, 16))
    return fail(KDA_ERR_INVALID_ARG, who, "w_post, scale or w_pre is misaligned");
  if (a->rows > 0 && (!have(a->u, 16) || !fine(a->gate, 16) || !fine(a->residual, 16)))
    return fail(KDA_ERR_INVALID_ARG, who, "u is required; u, gate and residual are 16-byte aligned");
  if (a->rows > 0 && ((a->w_post && !have(a->rstd_post, 4)) || (a->w_pre && !have(a->rstd_pre, 4))))
    return fail(KDA_ERR_INVALID_ARG, who, "rstd_post goes with w_post and rstd_pre with w_pre");
  return KDA_OK;
}

kda::BlockNormParams norm_params(const kda_block_norm_args *a) {
  kda::BlockNormParams p{};
  p.rows = a->rows;
  p.dim = a->dim;
  p.silu = a->gate_act == KDA_GATE_SILU;
  p.eps = a->eps;
  p.inv_dim = 1.f / (float)a->dim;
  p.u = a->u, p.gate = a->gate, p.residual = a->residual;
  p.w_post = a->w_post, p.scale = a->scale, p.w_pre = a->w_pre;
  p.out = a->out, p.normed = a->normed;
  p.rstd_post = a->rstd_post, p.rstd_pre = a->rstd_pre;
  return p;
}
}  // namespace

extern "C" {

size_t kda_ssm_fwd_workspace_size(const kda_ssm_args *a) {
  if (check_ssm(a, "kda_ssm_fwd_workspace_size") != KDA_OK) return 0;
  if (a->io_dtype == KDA_F32) return kda::ssm_rec_plan(a->n_seqs, a->total_tokens, a->heads, a->head_dim).bytes;
  const int units = a->heads * (a->head_dim / kda::SSM_COLS);
  return kda::ssm_segment_bytes(a->n_seqs, units, kda::ssm_segments(a->n_seqs, a->total_tokens, units));
}

kda_status kda_ssm_fwd(const kda_ssm_args *a, cudaStream_t stream) {
  const char *who = "kda_ssm_fwd";
  const kda_status st = check_ssm(a, who);
  if (st != KDA_OK) return st;
  if (a->n_seqs == 0) return done(cudaSuccess, who);
  const bool f32 = a->io_dtype == KDA_F32;
  const kda::SsmRecPlan rec = kda::ssm_rec_plan(a->n_seqs, a->total_tokens, a->heads, a->head_dim);
  const int units = a->heads * (a->head_dim / kda::SSM_COLS), nseg = kda::ssm_segments(a->n_seqs, a->total_tokens, units);
  const size_t need = f32 ? rec.bytes : kda::ssm_segment_bytes(a->n_seqs, units, nseg);
  if (need > 0 && (!have(a->workspace, 16) || a->workspace_bytes < need))
    return fail(KDA_ERR_INVALID_ARG, who, "workspace missing, misaligned or smaller than kda_ssm_fwd_workspace_size()");
  if (f32) return done(kda::launch_ssm_fwd_f32(ssm_params(a), rec, a->workspace, stream), who);
  return done(kda::launch_ssm_fwd_tc(ssm_params(a), nseg, a->workspace, stream), who);
}

size_t kda_ssm_step_workspace_size(const kda_ssm_step_args *a) {
  if (!a || a->n_seqs < 0 || a->steps < 1 || a->steps > 8 || a->heads < 1 || a->groups < 1 || a->head_dim < 1 || a->d_state < 1) return 0;
  return (size_t)a->n_seqs * a->steps * ssm_step_channels(a) * sizeof(float);
}

kda_status kda_ssm_step(const kda_ssm_step_args *a, cudaStream_t stream) {
  const char *who = "kda_ssm_step";
  if (!a) return fail(KDA_ERR_INVALID_ARG, who, "args is NULL");
  const kda_status st = check_heads(a->heads, a->groups, a->head_dim, a->d_state, a->io_dtype, who);
  if (st != KDA_OK) return st;
  if (a->width < 1 || a->width > KDA_CONV_MAX_WIDTH) return fail(KDA_ERR_UNSUPPORTED, who, "width must be 1..4");
  if (a->activation != KDA_ACT_NONE && a->activation != KDA_ACT_SILU)
    return fail(KDA_ERR_INVALID_ARG, who, "activation must be KDA_ACT_NONE or KDA_ACT_SILU");
  if (a->n_seqs < 0 || a->n_seqs > 65535 || a->steps < 1 || a->steps > 8)
    return fail(KDA_ERR_INVALID_ARG, who, "need 0 <= n_seqs <= 65535 and 1 <= steps <= 8");
  if (ssm_step_channels(a) > (size_t)1 << 24) return fail(KDA_ERR_UNSUPPORTED, who, "more than 2^24 channels");
  if (a->n_seqs == 0) return done(cudaSuccess, who);
  if (a->state_indices && a->n_slots < 1) return fail(KDA_ERR_INVALID_ARG, who, "n_slots must be >= 1 with state_indices");
  if (!have(a->xbc, 16) || !have(a->y, 16) || !have(a->state, 16) || (a->width > 1 && !have(a->conv_state, 16)))
    return fail(KDA_ERR_INVALID_ARG, who, "xbc, y and the states are required and 16-byte aligned");
  if (!have(a->conv_weight, 4) || !have(a->dt, 4) || !have(a->a, 4) || !fine(a->conv_bias, 4) || !fine(a->dt_bias, 4) || !fine(a->d_skip, 4))
    return fail(KDA_ERR_INVALID_ARG, who, "conv_weight, dt and a are required; an fp32 array is misaligned");
  if (!fine(a->state_indices, 4) || !fine(a->accept_len, 4) || !fine(a->first_slot, 4) || !fine(a->dev_status, 4))
    return fail(KDA_ERR_INVALID_ARG, who, "an int32 array is misaligned");
  if (!have(a->workspace, 16) || a->workspace_bytes < kda_ssm_step_workspace_size(a))
    return fail(KDA_ERR_INVALID_ARG, who, "workspace missing, misaligned or smaller than kda_ssm_step_workspace_size()");
  kda::SsmParams p{};
  p.n_seqs = a->n_seqs;
  p.H = a->heads;
  p.G = a->groups;
  p.P = a->head_dim;
  p.softplus = a->dt_softplus != 0;
  p.dt = a->dt, p.a = a->a, p.dt_bias = a->dt_bias, p.d_skip = a->d_skip;
  p.y = a->y;
  p.status = a->dev_status;
  p.L = a->steps;
  p.n_slots = a->state_indices ? a->n_slots : a->n_seqs;
  p.W = a->width;
  p.act = a->activation == KDA_ACT_SILU;
  p.xbc = a->xbc;
  p.cw = a->conv_weight, p.cbias = a->conv_bias;
  p.conv_state = a->conv_state;
  p.conv = static_cast<float *>(a->workspace);
  p.state = a->state;
  p.idx = a->state_indices, p.acc = a->accept_len, p.first = a->first_slot;
  return done(kda::launch_ssm_step(p, a->io_dtype == KDA_F32, stream), who);
}

kda_status kda_draft_verify(const kda_draft_verify_args *a, cudaStream_t stream) {
  const char *who = "kda_draft_verify";
  if (!a) return fail(KDA_ERR_INVALID_ARG, who, "args is NULL");
  if (!io_ok(a->io_dtype)) return fail(KDA_ERR_UNSUPPORTED, who, "io_dtype must be KDA_BF16 or KDA_F32");
  if (a->n_seqs < 0 || a->n_seqs > 65535 || a->drafts < 1 || a->drafts > 8 || a->vocab < 1 || a->vocab > 1 << 30)
    return fail(KDA_ERR_INVALID_ARG, who, "need 0 <= n_seqs <= 65535, 1 <= drafts <= 8 and 1 <= vocab <= 2^30");
  if (a->n_seqs == 0) return done(cudaSuccess, who);
  if (!have(a->p, 16) || !fine(a->q, 16) || !have(a->noise, 16)) return fail(KDA_ERR_INVALID_ARG, who, "p and noise are required; p, q and noise are 16-byte aligned");
  if (!have(a->draft, 4) || !have(a->u, 4) || !fine(a->draft_len, 4)) return fail(KDA_ERR_INVALID_ARG, who, "draft and u are required; an array is misaligned");
  if (!have(a->accept_len, 4) || !have(a->tokens, 4) || !fine(a->first_slot, 4))
    return fail(KDA_ERR_INVALID_ARG, who, "accept_len and tokens are required; an output is misaligned");
  kda::VerifyParams p{};
  p.n_seqs = a->n_seqs;
  p.L = a->drafts;
  p.V = a->vocab;
  p.p = a->p, p.q = a->q;
  p.draft = a->draft, p.draft_len = a->draft_len;
  p.u = a->u, p.noise = a->noise;
  p.accept = a->accept_len, p.first = a->first_slot, p.tokens = a->tokens;
  return done(kda::launch_draft_verify(p, a->io_dtype == KDA_F32, stream), who);
}

kda_status kda_block_norm_fwd(const kda_block_norm_args *a, cudaStream_t stream) {
  const char *who = "kda_block_norm_fwd";
  const kda_status st = check_norm(a, who);
  if (st != KDA_OK) return st;
  if (a->rows > 0 && (!have(a->out, 16) || (a->w_pre && !have(a->normed, 16))))
    return fail(KDA_ERR_INVALID_ARG, who, "out (and normed with w_pre) is NULL or misaligned");
  return done(kda::launch_block_norm_fwd(norm_params(a), a->io_dtype == KDA_F32, stream), who);
}

size_t kda_block_norm_bwd_workspace_size(const kda_block_norm_bwd_args *a) {
  if (!a || !io_ok(a->fwd.io_dtype) || a->fwd.dim < 8 || a->fwd.dim > 16384 || a->fwd.dim % 8 || a->fwd.rows < 0) return 0;
  return (size_t)kda::block_norm_bwd_ctas(a->fwd.rows, a->fwd.dim, a->fwd.io_dtype == KDA_F32) * 2 * a->fwd.dim * sizeof(float);
}

kda_status kda_block_norm_bwd(const kda_block_norm_bwd_args *a, cudaStream_t stream) {
  const char *who = "kda_block_norm_bwd";
  if (!a) return fail(KDA_ERR_INVALID_ARG, who, "args is NULL");
  const kda_block_norm_args &f = a->fwd;
  const kda_status st = check_norm(&f, who);
  if (st != KDA_OK) return st;
  if (f.rows > 0 && (!fine(a->d_out, 16) || !fine(a->d_normed, 16) || !have(a->du, 16) || (f.gate && !have(a->d_gate, 16)) ||
                     (f.residual && !have(a->d_residual, 16))))
    return fail(KDA_ERR_INVALID_ARG, who, "du (d_gate with gate, d_residual with residual) is NULL, or a gradient is misaligned");
  if ((f.w_post && !have(a->dw_post, 4)) || (f.scale && !have(a->dscale, 4)) || (f.w_pre && !have(a->dw_pre, 4)))
    return fail(KDA_ERR_INVALID_ARG, who, "dw_post, dscale and dw_pre go with w_post, scale and w_pre");
  if (!have(a->workspace, 16) || a->workspace_bytes < kda_block_norm_bwd_workspace_size(a))
    return fail(KDA_ERR_INVALID_ARG, who, "workspace missing, misaligned or smaller than kda_block_norm_bwd_workspace_size()");
  kda::BlockNormParams p = norm_params(&f);
  p.d_out = a->d_out, p.d_normed = f.w_pre ? a->d_normed : nullptr;
  p.du = a->du, p.d_gate = a->d_gate, p.d_residual = a->d_residual;
  p.dw_post = f.w_post ? a->dw_post : nullptr;
  p.dscale = f.scale ? a->dscale : nullptr;
  p.dw_pre = f.w_pre ? a->dw_pre : nullptr;
  p.partial = static_cast<float *>(a->workspace);
  p.status = a->dev_status;
  return done(kda::launch_block_norm_bwd(p, f.io_dtype == KDA_F32, stream), who);
}

}  // extern "C"
