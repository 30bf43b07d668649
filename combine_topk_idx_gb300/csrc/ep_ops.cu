// Host side of the operators around dispatch and combine: argument checks,
// workspaces, launches.
#include <algorithm>
#include <cmath>

#include "ep_clip.cuh"
#include "ep_ffn.cuh"
#include "ep_host.cuh"

namespace ep {
namespace {

// A required array, and an optional one.
bool have(const void *p, uintptr_t a) { return p != nullptr && aligned(p, a); }
bool maybe(const void *p, uintptr_t a) { return aligned(p, a); }  // NULL is aligned

SfLayout sf_layout(const ep_handle *h, int64_t n) {
  const ep_config &c = h->cfg;
  const int64_t nb = n / kFp8Block;
  const int64_t per = c.fixed_capacity ? h->lp.fixed_cap : h->rows_alloc;
  SfLayout l{};
  if (c.use_tma_aligned_col_major_sf) {
    l.ts = 1;
    l.hs = align_up(per, 4);
    l.numel = nb * l.hs;
  } else {
    l.ts = nb;
    l.hs = 1;
    l.numel = nb * per;
  }
  if (c.fixed_capacity) {
    l.cap = h->lp.fixed_cap;
    l.es = l.numel;
    l.numel *= c.num_experts;
  }
  return l;
}

// The rows an operator on a layout's rows works on (h may be NULL: all).
RowsParams rows_params(const ep_handle *h, int64_t rows) {
  RowsParams r{};
  r.rows = rows;
  if (h == nullptr) return r;
  const ep_config &c = h->cfg;
  r.num_rows = h->lp.ctrl + (c.do_expand ? kCtrlNumExpanded : kCtrlNumRecv);
  r.meta = h->lp.meta;
  r.psum_e = h->lp.psum_e;
  r.cnt_e = h->lp.cnt_e;
  r.E = c.num_experts;
  r.fixed_cap = h->lp.fixed_cap;
  r.zero_padding = c.do_expand && c.do_zero_padding;
  return r;
}

ep_status check_rows(const ep_handle *h, int64_t rows, int32_t ffn, bool fp8) {
  if (rows < 0 || ffn < 1) return EP_ERR_INVALID_ARG;
  if (ffn % (fp8 ? kFp8Block : 8) != 0) return EP_ERR_INVALID_ARG;
  if (ffn > EP_MAX_HIDDEN || rows > 0x7fffffffLL) return EP_ERR_UNSUPPORTED;
  if (h != nullptr && rows != h->rows_alloc) return EP_ERR_INVALID_ARG;
  return EP_OK;
}

SfLayout rows_sf(const ep_handle *h, int64_t n) {
  if (h != nullptr) return sf_layout(h, n);
  SfLayout l{};
  l.ts = n / kFp8Block;
  l.hs = 1;
  return l;
}

ep_status check_norm(int32_t num_tokens, int32_t hidden) {
  if (num_tokens < 0 || hidden < 8 || hidden % 8 != 0) return EP_ERR_INVALID_ARG;
  return hidden > EP_MAX_HIDDEN ? EP_ERR_UNSUPPORTED : EP_OK;
}

// A dimension of a matrix that the tensor cores take.
bool gemm_size(int64_t n) { return n >= 8 && n % 8 == 0; }

// Checks what the calls of the feed-forward block share: the rows (h may be NULL:
// `rows` rows, one matrix), the sizes of the matrix.
ep_status check_ffn(const ep_handle *h, int64_t rows, int64_t n, int64_t k, int64_t most_n) {
  if (rows < 0 || !gemm_size(n) || !gemm_size(k)) return EP_ERR_INVALID_ARG;
  if (n > most_n || k > EP_MAX_GEMM || rows > 0x7fffffffLL) return EP_ERR_UNSUPPORTED;
  if (h == nullptr) return EP_OK;
  if (!h->cfg.do_expand) return EP_ERR_UNSUPPORTED;
  if (rows != h->rows_alloc) return EP_ERR_INVALID_ARG;
  return check_device(h);
}

bool row_stride(int64_t stride, int64_t n) { return stride >= n && stride % 8 == 0; }

FfnParams ffn_params(const ep_handle *h, int64_t rows) {
  FfnParams p{};
  p.s.E = 1;
  p.s.rows = rows;
  p.max_segments = 1;
  if (h == nullptr) return p;
  const ep_config &c = h->cfg;
  p.s.psum_e = h->lp.psum_e;
  p.s.cnt_e = h->lp.cnt_e;
  p.s.E = c.num_experts;
  p.s.fixed_cap = h->lp.fixed_cap;
  p.s.zero_padding = c.do_zero_padding;
  p.max_segments = (int64_t)c.num_tokens * c.num_topk;
  p.err = reinterpret_cast<unsigned *>(h->lp.ctrl + kCtrlError);
  return p;
}

ep_status run_ffn(int mode, FfnParams &p, const ep_handle *h, ep_stream_t stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const size_t bytes = ffn_workspace(mode, &p, nullptr);
  void *ws = nullptr;
  if (bytes > 0) {
    const cudaError_t e = workspace_alloc(bytes, s, &ws);
    if (e != cudaSuccess) return cuda_status(e);
    ffn_workspace(mode, &p, ws);
  }
  cudaError_t e = launch_ffn(mode, p, h != nullptr ? h->cfg.num_sms : 0, s);
  if (ws != nullptr) {
    const cudaError_t f = workspace_free(ws, s);
    if (e == cudaSuccess) e = f;
  }
  return cuda_status(e);
}

}  // namespace
}  // namespace ep

using ep::have;
using ep::maybe;

extern "C" {

ep_status ep_sf_layout(const ep_handle *h, int32_t n, int64_t *numel, int64_t *token_stride,
                       int64_t *hidden_stride, int64_t *expert_stride) {
  if (h == nullptr || n < ep::kFp8Block || n % ep::kFp8Block != 0 || numel == nullptr ||
      token_stride == nullptr || hidden_stride == nullptr || expert_stride == nullptr)
    return EP_ERR_INVALID_ARG;
  const ep::SfLayout l = ep::sf_layout(h, n);
  *numel = l.numel;
  *token_stride = l.ts;
  *hidden_stride = l.hs;
  *expert_stride = l.es;
  return EP_OK;
}

ep_status ep_rmsnorm(int32_t num_tokens, int32_t hidden, const void *x, int64_t x_stride,
                     const void *residual, int64_t residual_stride, const void *gamma,
                     int32_t gamma_is_fp32, float eps, void *residual_out, void *y, void *y_fp8,
                     float *y_sf, int64_t y_sf_token_stride, int64_t y_sf_hidden_stride,
                     float *rstd, ep_stream_t stream) {
  if (const ep_status st = ep::check_norm(num_tokens, hidden); st != EP_OK) return st;
  if (!(eps >= 0.f) || !std::isfinite(eps) || gamma_is_fp32 < 0 || gamma_is_fp32 > 1)
    return EP_ERR_INVALID_ARG;
  if (residual_out == nullptr && y == nullptr && y_fp8 == nullptr && rstd == nullptr &&
      num_tokens > 0)
    return EP_ERR_INVALID_ARG;
  if (x_stride < hidden || x_stride % 8 != 0) return EP_ERR_INVALID_ARG;
  if (residual != nullptr && (residual_stride < hidden || residual_stride % 8 != 0))
    return EP_ERR_INVALID_ARG;
  if (num_tokens == 0) return EP_OK;
  if (!have(x, 16) || !maybe(residual, 16) || !have(gamma, 16) || !maybe(residual_out, 16) ||
      !maybe(y, 16) || !maybe(y_fp8, 16) || !maybe(y_sf, 4) || !maybe(rstd, 4))
    return EP_ERR_INVALID_ARG;
  // written over the residual only row by row in place
  if (residual_out != nullptr && residual_out == residual && residual_stride != hidden)
    return EP_ERR_INVALID_ARG;
  if ((y_fp8 == nullptr) != (y_sf == nullptr)) return EP_ERR_INVALID_ARG;
  if (y_fp8 != nullptr &&
      (hidden % ep::kFp8Block != 0 || y_sf_token_stride < 1 || y_sf_hidden_stride < 1))
    return EP_ERR_INVALID_ARG;
  ep::NormParams p{};
  p.x = static_cast<const uint16_t *>(x);
  p.residual = static_cast<const uint16_t *>(residual);
  p.x_stride = x_stride;
  p.res_stride = residual_stride;
  p.gamma = gamma;
  p.gamma_f32 = gamma_is_fp32;
  p.eps = eps;
  p.T = num_tokens;
  p.H = hidden;
  p.res_out = static_cast<uint16_t *>(residual_out);
  p.y = static_cast<uint16_t *>(y);
  p.q = static_cast<uint8_t *>(y_fp8);
  p.sf = y_sf;
  p.sf_ts = y_sf_token_stride;
  p.sf_hs = y_sf_hidden_stride;
  p.rstd = rstd;
  return ep::cuda_status(ep::launch_norm(p, reinterpret_cast<cudaStream_t>(stream)));
}

ep_status ep_rmsnorm_backward(int32_t num_tokens, int32_t hidden, const void *grad_y,
                              const void *normed, const void *gamma, int32_t gamma_is_fp32,
                              const float *rstd, const void *grad_residual, void *grad_x,
                              float *grad_gamma, ep_stream_t stream) {
  if (const ep_status st = ep::check_norm(num_tokens, hidden); st != EP_OK) return st;
  if (gamma_is_fp32 < 0 || gamma_is_fp32 > 1 || !maybe(grad_gamma, 16)) return EP_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (num_tokens == 0) {
    if (grad_gamma == nullptr) return EP_OK;
    return ep::cuda_status(cudaMemsetAsync(grad_gamma, 0, sizeof(float) * hidden, s));
  }
  if (!have(grad_y, 16) || !have(normed, 16) || !have(gamma, 16) || !have(rstd, 4) ||
      !maybe(grad_residual, 16) || !have(grad_x, 16))
    return EP_ERR_INVALID_ARG;
  ep::NormBackwardParams p{};
  p.gy = static_cast<const uint16_t *>(grad_y);
  p.r = static_cast<const uint16_t *>(normed);
  p.gres = static_cast<const uint16_t *>(grad_residual);
  p.gamma = gamma;
  p.gamma_f32 = gamma_is_fp32;
  p.rstd = rstd;
  p.T = num_tokens;
  p.H = hidden;
  p.gx = static_cast<uint16_t *>(grad_x);
  p.ggamma = grad_gamma;
  void *ws = nullptr;
  cudaError_t e = ep::norm_backward_parts(p, &p.parts);
  if (e != cudaSuccess) return ep::cuda_status(e);
  if (grad_gamma != nullptr) {
    e = ep::workspace_alloc(sizeof(float) * (size_t)p.parts * hidden, s, &ws);
    if (e != cudaSuccess) return ep::cuda_status(e);
    p.part = static_cast<float *>(ws);
  }
  e = ep::launch_norm_backward(p, s);
  if (ws != nullptr) {
    const cudaError_t f = ep::workspace_free(ws, s);
    if (e == cudaSuccess) e = f;
  }
  return ep::cuda_status(e);
}

ep_status ep_swiglu(const ep_handle *h, int64_t rows, int32_t ffn, const void *gate_up,
                    const float *row_weights, void *act, void *act_fp8, float *act_sf,
                    void *ckpt_fp8, float *ckpt_sf, ep_stream_t stream) {
  const bool fp8 = act_fp8 != nullptr || ckpt_fp8 != nullptr;
  if (const ep_status st = ep::check_rows(h, rows, ffn, fp8); st != EP_OK) return st;
  if (h != nullptr)
    if (const ep_status st = ep::check_device(h); st != EP_OK) return st;
  if (rows == 0) return EP_OK;
  if (act == nullptr && !fp8) return EP_ERR_INVALID_ARG;
  if ((act_fp8 == nullptr) != (act_sf == nullptr) || (ckpt_fp8 == nullptr) != (ckpt_sf == nullptr))
    return EP_ERR_INVALID_ARG;
  if (!have(gate_up, 16) || !maybe(row_weights, 4) || !maybe(act, 16) || !maybe(act_fp8, 16) ||
      !maybe(act_sf, 4) || !maybe(ckpt_fp8, 16) || !maybe(ckpt_sf, 4))
    return EP_ERR_INVALID_ARG;
  ep::SwigluParams p{};
  p.r = ep::rows_params(h, rows);
  p.h = static_cast<const uint16_t *>(gate_up);
  p.row_w = row_weights;
  p.F = ffn;
  p.act = static_cast<uint16_t *>(act);
  p.q = static_cast<uint8_t *>(act_fp8);
  p.sf = act_sf;
  p.sfl = ep::rows_sf(h, ffn);
  p.ckpt = static_cast<uint8_t *>(ckpt_fp8);
  p.ckpt_sf = ckpt_sf;
  return ep::cuda_status(ep::launch_swiglu(p, h != nullptr ? h->cfg.num_sms : 0,
                                           reinterpret_cast<cudaStream_t>(stream)));
}

ep_status ep_swiglu_backward(const ep_handle *h, int64_t rows, int32_t ffn, const void *grad_act,
                             const void *ckpt_fp8, const float *ckpt_sf, const float *row_weights,
                             void *grad_gate_up, void *grad_fp8, float *grad_sf,
                             float *grad_row_weights, ep_stream_t stream) {
  if (const ep_status st = ep::check_rows(h, rows, ffn, true); st != EP_OK) return st;
  if (h != nullptr)
    if (const ep_status st = ep::check_device(h); st != EP_OK) return st;
  if (rows == 0) return EP_OK;
  if (grad_gate_up == nullptr && grad_fp8 == nullptr && grad_row_weights == nullptr)
    return EP_ERR_INVALID_ARG;
  if ((grad_fp8 == nullptr) != (grad_sf == nullptr)) return EP_ERR_INVALID_ARG;
  if (!have(grad_act, 16) || !have(ckpt_fp8, 16) || !have(ckpt_sf, 4) || !maybe(row_weights, 4) ||
      !maybe(grad_gate_up, 16) || !maybe(grad_fp8, 16) || !maybe(grad_sf, 4) ||
      !maybe(grad_row_weights, 4))
    return EP_ERR_INVALID_ARG;
  ep::SwigluBackwardParams p{};
  p.r = ep::rows_params(h, rows);
  p.ga = static_cast<const uint16_t *>(grad_act);
  p.ckpt = static_cast<const uint8_t *>(ckpt_fp8);
  p.ckpt_sf = ckpt_sf;
  p.row_w = row_weights;
  p.F = ffn;
  p.gh = static_cast<uint16_t *>(grad_gate_up);
  p.q = static_cast<uint8_t *>(grad_fp8);
  p.sf = grad_sf;
  p.sfl = ep::rows_sf(h, 2 * (int64_t)ffn);
  p.gw = grad_row_weights;
  return ep::cuda_status(ep::launch_swiglu_backward(p, h != nullptr ? h->cfg.num_sms : 0,
                                                    reinterpret_cast<cudaStream_t>(stream)));
}

ep_status ep_combine_weighted_backward(const ep_handle *h, const void *grad_out, const void *y,
                                       const float *topk_weights, const void *expert_bias,
                                       void *grad_y, void *grad_y_fp8, float *grad_y_sf,
                                       float *grad_topk_weights, float *grad_expert_bias,
                                       ep_stream_t stream) {
  if (h == nullptr) return EP_ERR_INVALID_ARG;
  const ep_config &c = h->cfg;
  const int T = c.num_tokens;
  if (grad_y == nullptr && grad_y_fp8 == nullptr && grad_topk_weights == nullptr &&
      grad_expert_bias == nullptr && T > 0 && h->rows_alloc > 0)
    return EP_ERR_INVALID_ARG;
  if (T > 0 && (!have(grad_out, 16) || !have(topk_weights, 4))) return EP_ERR_INVALID_ARG;
  if (!maybe(y, 16) || (T > 0 && h->rows_alloc > 0 && grad_topk_weights != nullptr && y == nullptr))
    return EP_ERR_INVALID_ARG;
  if (h->rows_alloc > 0) {
    if ((grad_y_fp8 == nullptr) != (grad_y_sf == nullptr)) return EP_ERR_INVALID_ARG;
    if (grad_y_fp8 != nullptr && c.hidden % ep::kFp8Block != 0) return EP_ERR_INVALID_ARG;
  }
  if (!maybe(expert_bias, 16) || !maybe(grad_y, 16) || !maybe(grad_y_fp8, 16) ||
      !maybe(grad_y_sf, 4) || !maybe(grad_topk_weights, 4) || !maybe(grad_expert_bias, 16))
    return EP_ERR_INVALID_ARG;
  if (const ep_status st = ep::check_device(h); st != EP_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  ep::CombineGradParams p{};
  p.g = static_cast<const uint16_t *>(grad_out);
  p.y = static_cast<const uint16_t *>(y);
  p.topk_w = topk_weights;
  p.topk32 = h->lp.topk32;
  p.dst = h->lp.dst;
  p.ebias = static_cast<const uint16_t *>(expert_bias);
  p.psum_e = h->lp.psum_e;
  p.cnt_e = h->lp.cnt_e;
  p.psum_pad = h->lp.psum_pad;
  p.T = T;
  p.K = c.num_topk;
  p.E = c.num_experts;
  p.H = c.hidden;
  p.do_expand = c.do_expand;
  p.zero_padding = c.do_expand && c.do_zero_padding;
  p.rows_alloc = h->rows_alloc;
  if (h->rows_alloc > 0) {
    p.gy = static_cast<uint16_t *>(grad_y);
    p.q = static_cast<uint8_t *>(grad_y_fp8);
    p.sf = grad_y_sf;
    if (p.q != nullptr) p.sfl = ep::sf_layout(h, c.hidden);
  }
  p.gw = grad_topk_weights;
  p.gbias = grad_expert_bias;
  void *ws = nullptr;
  cudaError_t e = cudaSuccess;
  if (p.gbias != nullptr) {
    size_t bytes = 0;
    e = ep::combine_grad_workspace(&p, &bytes, nullptr);
    if (e == cudaSuccess) e = ep::workspace_alloc(bytes, s, &ws);
    if (e == cudaSuccess) e = ep::combine_grad_workspace(&p, &bytes, ws);
    if (e != cudaSuccess) {
      if (ws != nullptr) ep::workspace_free(ws, s);
      return ep::cuda_status(e);
    }
  }
  e = ep::launch_combine_grad(p, c.num_sms, s);
  if (ws != nullptr) {
    const cudaError_t f = ep::workspace_free(ws, s);
    if (e == cudaSuccess) e = f;
  }
  return ep::cuda_status(e);
}

ep_status ep_expert_gemm(const ep_handle *h, int32_t n, int32_t k, const void *a_fp8,
                         const float *a_sf, const void *w_fp8, const float *w_sf, void *out,
                         ep_stream_t stream) {
  if (h == nullptr) return EP_ERR_INVALID_ARG;
  const ep_config &c = h->cfg;
  if (n < 8 || n % 8 != 0 || k < ep::kFp8Block || k % ep::kFp8Block != 0)
    return EP_ERR_INVALID_ARG;
  if (!c.do_expand || n > EP_MAX_GEMM || k > EP_MAX_GEMM ||
      (int64_t)c.num_experts * n > 0x7fffffffLL)
    return EP_ERR_UNSUPPORTED;
  if (!have(w_fp8, 16) || !have(w_sf, 4)) return EP_ERR_INVALID_ARG;
  if (const ep_status st = ep::check_device(h); st != EP_OK) return st;
  if (h->rows_alloc == 0) return EP_OK;
  if (!have(a_fp8, 16) || !have(a_sf, 4) || !have(out, 16)) return EP_ERR_INVALID_ARG;
  ep::ExpertGemmParams p{};
  p.a = static_cast<const uint8_t *>(a_fp8);
  p.sf = a_sf;
  p.sfl = ep::sf_layout(h, k);
  p.w = static_cast<const uint8_t *>(w_fp8);
  p.w_sf = w_sf;
  p.out = static_cast<uint16_t *>(out);
  p.out32 = ep::aligned(out, 32) && n % 16 == 0;
  p.psum_e = h->lp.psum_e;
  p.cnt_e = h->lp.cnt_e;
  p.E = c.num_experts;
  p.N = n;
  p.K = k;
  p.fixed_cap = h->lp.fixed_cap;
  p.zero_padding = c.do_zero_padding;
  p.rows_alloc = h->rows_alloc;
  p.max_slots = (int64_t)c.num_tokens * c.num_topk;
  p.err = reinterpret_cast<unsigned *>(h->lp.ctrl + ep::kCtrlError);
  return ep::cuda_status(
      ep::launch_expert_gemm(p, c.num_sms, reinterpret_cast<cudaStream_t>(stream)));
}

ep_status ep_ffn_gated(const ep_handle *h, int64_t rows, int32_t ffn, int32_t k, const void *x,
                       int64_t x_stride, const void *w, void *act, void *gate_up,
                       ep_stream_t stream) {
  if (const ep_status st = ep::check_ffn(h, rows, ffn, k, EP_MAX_GEMM / 2); st != EP_OK) return st;
  if (act == nullptr && gate_up == nullptr && rows > 0) return EP_ERR_INVALID_ARG;
  if (!ep::row_stride(x_stride, k)) return EP_ERR_INVALID_ARG;
  if (rows == 0) return EP_OK;
  if (!have(x, 16) || !have(w, 16) || !maybe(act, 16) || !maybe(gate_up, 16))
    return EP_ERR_INVALID_ARG;
  ep::FfnParams p = ep::ffn_params(h, rows);
  p.a = static_cast<const uint16_t *>(x);
  p.a_stride = x_stride;
  p.b = static_cast<const uint16_t *>(w);
  p.N = ffn;
  p.K = k;
  p.out = static_cast<uint16_t *>(act);
  p.out2 = static_cast<uint16_t *>(gate_up);
  return ep::run_ffn(ep::kFfnGated, p, h, stream);
}

ep_status ep_ffn_gated_backward(const ep_handle *h, int64_t rows, int32_t ffn, int32_t n,
                                const void *grad_out, int64_t grad_out_stride, const void *w,
                                const void *gate_up, void *grad_gate_up, void *act,
                                ep_stream_t stream) {
  if (const ep_status st = ep::check_ffn(h, rows, ffn, n, EP_MAX_GEMM / 2); st != EP_OK) return st;
  if (!ep::row_stride(grad_out_stride, n)) return EP_ERR_INVALID_ARG;
  if (rows == 0) return EP_OK;
  if (!have(grad_out, 16) || !have(w, 16) || !have(gate_up, 16) || !have(grad_gate_up, 16) ||
      !maybe(act, 16))
    return EP_ERR_INVALID_ARG;
  ep::FfnParams p = ep::ffn_params(h, rows);
  p.a = static_cast<const uint16_t *>(grad_out);
  p.a_stride = grad_out_stride;
  p.b = static_cast<const uint16_t *>(w);
  p.N = ffn;
  p.K = n;
  p.kept = static_cast<const uint16_t *>(gate_up);
  p.out = static_cast<uint16_t *>(grad_gate_up);
  p.out2 = static_cast<uint16_t *>(act);
  return ep::run_ffn(ep::kFfnGatedGrad, p, h, stream);
}

ep_status ep_ffn_product(const ep_handle *h, int64_t rows, int32_t n, int32_t k, const void *a,
                         int64_t a_stride, const void *w, int32_t transposed, void *out,
                         ep_stream_t stream) {
  if (const ep_status st = ep::check_ffn(h, rows, n, k, EP_MAX_GEMM); st != EP_OK) return st;
  if (!ep::row_stride(a_stride, k) || transposed < 0 || transposed > 1) return EP_ERR_INVALID_ARG;
  if (rows == 0) return EP_OK;
  if (!have(a, 16) || !have(w, 16) || !have(out, 16)) return EP_ERR_INVALID_ARG;
  ep::FfnParams p = ep::ffn_params(h, rows);
  p.a = static_cast<const uint16_t *>(a);
  p.a_stride = a_stride;
  p.b = static_cast<const uint16_t *>(w);
  p.N = n;
  p.K = k;
  p.out = static_cast<uint16_t *>(out);
  return ep::run_ffn(transposed ? ep::kFfnProductT : ep::kFfnProduct, p, h, stream);
}

ep_status ep_ffn_weight_grad(const ep_handle *h, int64_t rows, int32_t n, int32_t k,
                             const void *grad, int64_t grad_stride, const void *a,
                             int64_t a_stride, void *grad_w, int32_t grad_w_is_fp32,
                             int32_t accumulate, ep_stream_t stream) {
  if (const ep_status st = ep::check_ffn(h, rows, n, k, EP_MAX_GEMM); st != EP_OK) return st;
  if (!ep::row_stride(grad_stride, n) || !ep::row_stride(a_stride, k) || grad_w_is_fp32 < 0 ||
      grad_w_is_fp32 > 1 || accumulate < 0 || accumulate > 1)
    return EP_ERR_INVALID_ARG;
  if (!have(grad_w, 16)) return EP_ERR_INVALID_ARG;
  ep::FfnParams p = ep::ffn_params(h, rows);
  if (rows == 0) {
    if (accumulate) return EP_OK;
    const size_t bytes = (size_t)p.s.E * n * k * (grad_w_is_fp32 ? 4 : 2);
    return ep::cuda_status(
        cudaMemsetAsync(grad_w, 0, bytes, reinterpret_cast<cudaStream_t>(stream)));
  }
  if (!have(grad, 16) || !have(a, 16)) return EP_ERR_INVALID_ARG;
  p.a = static_cast<const uint16_t *>(grad);
  p.a_stride = grad_stride;
  p.b = static_cast<const uint16_t *>(a);
  p.b_stride = a_stride;
  p.M = n;
  p.N = k;
  p.out = static_cast<uint16_t *>(grad_w);
  p.accumulate = accumulate;
  return ep::run_ffn(grad_w_is_fp32 ? ep::kFfnWeightGrad32 : ep::kFfnWeightGrad, p, h, stream);
}

ep_status ep_clip_grads(int32_t count, const void *const *grads, void *const *outs,
                        const int64_t *numels, const uint8_t *is_fp32, float max_norm, float *norm,
                        ep_stream_t stream) {
  if (count < 0 || !(max_norm >= 0.f) || !maybe(norm, 4)) return EP_ERR_INVALID_ARG;
  if (outs == nullptr && norm == nullptr) return EP_ERR_INVALID_ARG;
  if (count > 0 && (grads == nullptr || numels == nullptr || is_fp32 == nullptr))
    return EP_ERR_INVALID_ARG;
  for (int32_t i = 0; i < count; ++i) {
    if (numels[i] < 0 || is_fp32[i] > 1) return EP_ERR_INVALID_ARG;
    if (numels[i] > (1LL << 40)) return EP_ERR_UNSUPPORTED;
    if (numels[i] == 0) continue;
    const uintptr_t size = is_fp32[i] ? 4 : 2;
    if (!have(grads[i], size) || (outs != nullptr && !have(outs[i], size)))
      return EP_ERR_INVALID_ARG;
  }
  int dev = 0;
  if (const cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return ep::cuda_status(e);
  const ep::GradList l{count, grads, outs, numels, is_fp32};
  const int sms = ep::device_sm_count(dev);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  void *ws = nullptr;
  cudaError_t e = cudaSuccess;
  if (const size_t bytes = ep::clip_workspace(l, sms); bytes > 0) {
    e = ep::workspace_alloc(bytes, s, &ws);
    if (e != cudaSuccess) return ep::cuda_status(e);
  }
  e = ep::launch_clip(l, max_norm, norm, ws, sms, s);
  if (ws != nullptr) {
    const cudaError_t f = ep::workspace_free(ws, s);
    if (e == cudaSuccess) e = f;
  }
  return ep::cuda_status(e);
}

}  // extern "C"
