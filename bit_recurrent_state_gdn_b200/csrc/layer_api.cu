// C ABI of the operators around the recurrence: argument checks and dispatch to the kernels. See
// include/gdnq_layer.h for the contract of every entry point.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "layer_args.h"
#include "overlap.h"
#include "status.h"

using gdnq::clear_error;
using gdnq::cuda_fail;
using gdnq::fail;
using gdnq::need_ptr;

namespace {

struct Shape {
  int64_t B, L, H, D;
  bool empty() const { return B == 0 || H == 0; }
  size_t heads() const { return (size_t)B * (size_t)H * (size_t)D; }  // elements of [B][H][D]
};

gdn_status check_shape(int64_t B, int64_t L, int64_t H, int64_t D, int act_dtype) {
  if (B < 0 || H < 0) return fail(GDN_ERR_INVALID_ARG, "B=%lld, H=%lld must be >= 0", (long long)B, (long long)H);
  if (L < 0) return fail(GDN_ERR_INVALID_ARG, "L=%lld must be >= 0", (long long)L);
  if (L > (int64_t)1 << 30) return fail(GDN_ERR_INVALID_ARG, "L=%lld exceeds 2^30", (long long)L);
  if (D < 1) return fail(GDN_ERR_INVALID_ARG, "D=%lld must be >= 1", (long long)D);
  if (H * D > (int64_t)1 << 30) return fail(GDN_ERR_INVALID_ARG, "H*D exceeds 2^30");
  if (B * H > INT32_MAX) return fail(GDN_ERR_INVALID_ARG, "B*H exceeds 2^31-1");
  if (B * H > ((int64_t)1 << 36) / D) return fail(GDN_ERR_INVALID_ARG, "B*H*D exceeds 2^36");
  if (act_dtype != GDN_DTYPE_F32 && act_dtype != GDN_DTYPE_BF16)
    return fail(GDN_ERR_INVALID_ARG, "act_dtype=%d is not a gdn_dtype", act_dtype);
  return GDN_OK;
}

unsigned act_bytes(int act_dtype) { return act_dtype == GDN_DTYPE_F32 ? 4u : 2u; }

// The array's pointer and strides; of an output also that no two elements share a place, which
// holds when each stride steps over all that the smaller ones span.
gdn_status check_tokens(const gdn_tokens* t, const char* name, const Shape& s, unsigned elem,
                        bool output) {
  if (!t) return fail(GDN_ERR_INVALID_ARG, "%s is null", name);
  if (s.L == 0) return GDN_OK;
  gdn_status st = need_ptr(t->ptr, name, elem);
  if (st != GDN_OK) return st;
  struct Dim {
    int64_t stride, size;
  } dims[3] = {{t->sb, s.B}, {t->sl, s.L}, {t->sh, s.H}};
  double span = (double)s.D;
  for (const Dim& d : dims) {
    if (d.stride < 0) return fail(GDN_ERR_INVALID_ARG, "%s has a negative stride", name);
    span += (double)(d.size - 1) * (double)d.stride;
  }
  if (s.L > 1 && t->sl > (int64_t)1 << 27)
    return fail(GDN_ERR_UNSUPPORTED, "%s: tokens further than 2^27 elements apart are not built", name);
  if (span * elem > 4e18) return fail(GDN_ERR_INVALID_ARG, "%s spans too many bytes", name);
  if (!output) return GDN_OK;
  std::sort(dims, dims + 3, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
  int64_t extent = s.D;
  for (const Dim& d : dims) {
    if (d.size == 1) continue;
    if (d.stride < extent)
      return fail(GDN_ERR_INVALID_ARG, "%s is written: its elements may not share memory", name);
    extent += (d.size - 1) * d.stride;
  }
  return GDN_OK;
}

gdn_status check_opt(const void* p, const char* name, unsigned align) {
  return p ? need_ptr(p, name, align) : GDN_OK;
}

gdn_status check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return GDN_OK;
  gdn_status st = need_ptr(ws, "workspace");
  if (st != GDN_OK) return st;
  if (have < need)
    return fail(GDN_ERR_INVALID_ARG, "workspace holds %zu bytes, the call needs %zu", have, need);
  return GDN_OK;
}

void add(gdnq::Arrays& all, const gdn_tokens* t, const char* name, const Shape& s, unsigned elem,
         bool output) {
  all.tokens(t, name, s.B, s.L, s.H, s.D, elem, output);
}

int64_t chunks(int64_t L) { return (L + GDN_SCAN_CHUNK - 1) / GDN_SCAN_CHUNK; }

size_t norm_params(const gdn_norm_config* c) {
  return (size_t)c->D * (c->weight == GDN_WEIGHT_CHANNEL ? (size_t)c->H : 1);
}

gdnq::Tok tok(const gdn_tokens* t) {
  return t ? gdnq::Tok{t->ptr, t->sb, t->sl, t->sh} : gdnq::Tok{nullptr, 0, 0, 0};
}

gdn_status check_scan(const gdn_scan_config* c, int32_t L, Shape* s) {
  if (!c) return fail(GDN_ERR_INVALID_ARG, "cfg is null");
  const gdn_status st = check_shape(c->B, L, c->H, c->D, c->act_dtype);
  if (st != GDN_OK) return st;
  if (c->scale < GDN_SCALE_NONE || c->scale > GDN_SCALE_SQRT)
    return fail(GDN_ERR_INVALID_ARG, "scale=%d is not a gdn_input_scale", c->scale);
  *s = Shape{c->B, L, c->H, c->D};
  return GDN_OK;
}

cudaError_t launch_scan(const gdnq::ScanArgs& a, const gdn_scan_config* c, bool backward,
                        gdn_stream_t stream) {
  return c->act_dtype == GDN_DTYPE_F32
             ? gdnq::launch_scan_f32(a, c->scale, backward, (cudaStream_t)stream)
             : gdnq::launch_scan_bf16(a, c->scale, backward, (cudaStream_t)stream);
}

gdn_status check_norm(const gdn_norm_config* c, int32_t L, Shape* s) {
  if (!c) return fail(GDN_ERR_INVALID_ARG, "cfg is null");
  const gdn_status st = check_shape(c->B, L, c->H, c->D, c->act_dtype);
  if (st != GDN_OK) return st;
  if (c->activation < GDN_ACT_NONE || c->activation > GDN_ACT_SIGMOID)
    return fail(GDN_ERR_INVALID_ARG, "activation=%d is not a gdn_activation", c->activation);
  if (c->weight != GDN_WEIGHT_HEAD && c->weight != GDN_WEIGHT_CHANNEL)
    return fail(GDN_ERR_INVALID_ARG, "weight=%d is not a gdn_weight_kind", c->weight);
  if (c->center != 0 && c->center != 1)
    return fail(GDN_ERR_INVALID_ARG, "center=%d must be 0 or 1", c->center);
  if (!(c->eps > 0.f) || !std::isfinite(c->eps))
    return fail(GDN_ERR_INVALID_ARG, "eps=%g must be positive", (double)c->eps);
  if (c->D > GDN_NORM_MAX_D)
    return fail(GDN_ERR_UNSUPPORTED, "D=%d exceeds %d", c->D, GDN_NORM_MAX_D);
  *s = Shape{c->B, L, c->H, c->D};
  return GDN_OK;
}

gdn_status check_conv(const gdn_conv_config* c, int32_t L, Shape* s) {
  if (!c) return fail(GDN_ERR_INVALID_ARG, "cfg is null");
  const gdn_status st = check_shape(c->B, L, c->H, c->D, c->act_dtype);
  if (st != GDN_OK) return st;
  if (c->activation != GDN_ACT_NONE && c->activation != GDN_ACT_SILU)
    return fail(GDN_ERR_INVALID_ARG, "activation=%d must be GDN_ACT_NONE or GDN_ACT_SILU",
                c->activation);
  if (c->K < 1) return fail(GDN_ERR_INVALID_ARG, "K=%d must be >= 2", c->K);
  if (c->K < 2 || c->K > GDN_CONV_MAX_K)
    return fail(GDN_ERR_UNSUPPORTED, "K=%d is not built (2..%d)", c->K, GDN_CONV_MAX_K);
  *s = Shape{c->B, L, c->H, c->D};
  return GDN_OK;
}

gdnq::NormArgs norm_args(const gdn_norm_config* c, int32_t L) {
  gdnq::NormArgs a{};
  a.eps = c->eps;
  a.inv_d = 1.0f / (float)c->D;
  a.B = c->B, a.L = L, a.H = c->H, a.D = c->D;
  a.center = c->center;
  a.activation = c->activation;
  a.per_channel = c->weight == GDN_WEIGHT_CHANNEL;
  return a;
}

cudaError_t launch_norm(const gdnq::NormArgs& a, const gdn_norm_config* c, bool backward,
                        gdn_stream_t stream) {
  const cudaStream_t st = (cudaStream_t)stream;
  if (c->act_dtype == GDN_DTYPE_F32)
    return backward ? gdnq::launch_norm_f32_backward(a, st) : gdnq::launch_norm_f32_forward(a, st);
  return backward ? gdnq::launch_norm_bf16_backward(a, st) : gdnq::launch_norm_bf16_forward(a, st);
}

cudaError_t launch_conv(const gdnq::ConvArgs& a, const gdn_conv_config* c, bool backward,
                        gdn_stream_t stream) {
  return c->act_dtype == GDN_DTYPE_F32 ? gdnq::launch_conv_f32(a, backward, (cudaStream_t)stream)
                                       : gdnq::launch_conv_bf16(a, backward, (cudaStream_t)stream);
}

// Gradients of parameters that no token reaches.
gdn_status zero(float* p, size_t n, gdn_stream_t stream, const char* where) {
  if (!p || n == 0) return GDN_OK;
  const cudaError_t e = cudaMemsetAsync(p, 0, n * sizeof(float), (cudaStream_t)stream);
  return e == cudaSuccess ? GDN_OK : cuda_fail(e, where);
}

}  // namespace

#define GDNQ_TRY(call)                                   \
  do {                                                   \
    const gdn_status status_of_call = (call);            \
    if (status_of_call != GDN_OK) return status_of_call; \
  } while (0)

extern "C" {

size_t gdn_gated_scan_workspace_bytes(const gdn_scan_config* cfg, int32_t L) {
  clear_error();
  Shape s;
  if (check_scan(cfg, L, &s) != GDN_OK || s.empty()) return 0;
  gdnq::ScanArgs a{};
  a.B = cfg->B, a.L = L, a.C = cfg->H * cfg->D;
  return gdnq::scan_spans(a);
}

gdn_status gdn_gated_scan(const gdn_scan_config* cfg, int32_t L, const gdn_tokens* x,
                          const gdn_tokens* g, const gdn_tokens* o, const float* h0, float* hT,
                          float* hist, const int32_t* lens, void* workspace,
                          size_t workspace_bytes, gdn_stream_t stream) {
  clear_error();
  Shape s;
  GDNQ_TRY(check_scan(cfg, L, &s));
  if (s.empty()) return GDN_OK;
  const unsigned e = act_bytes(cfg->act_dtype);
  GDNQ_TRY(check_tokens(x, "x", s, e, false));
  GDNQ_TRY(check_tokens(g, "g", s, 4, false));
  GDNQ_TRY(check_tokens(o, "o", s, e, true));
  GDNQ_TRY(check_opt(h0, "h0", 4));
  GDNQ_TRY(check_opt(hT, "hT", 4));
  GDNQ_TRY(check_opt(hist, "hist", 4));
  GDNQ_TRY(check_opt(lens, "lens", 4));
  gdnq::ScanArgs a{};
  a.x = tok(x), a.g = tok(g), a.o = tok(o);
  a.h0 = h0, a.hT = hT, a.hist = hist, a.lens = lens;
  a.B = cfg->B, a.L = L, a.H = cfg->H, a.D = cfg->D, a.C = cfg->H * cfg->D;
  const size_t need = gdnq::scan_spans(a);
  GDNQ_TRY(check_workspace(workspace, workspace_bytes, need));
  gdnq::Arrays all;
  add(all, x, "x", s, e, false), add(all, g, "g", s, 4, false), add(all, o, "o", s, e, true);
  const size_t state = 4 * s.heads();
  all.dense(h0, "h0", state, false), all.dense(hT, "hT", state, true);
  all.dense(hist, "hist", state * (size_t)chunks(L), true);
  all.dense(lens, "lens", 4 * (size_t)s.B, false), all.dense(workspace, "workspace", need, true);
  GDNQ_TRY(all.check(hT, h0));
  a.spans = need > 0 ? workspace : nullptr;
  const cudaError_t err = launch_scan(a, cfg, false, stream);
  return err == cudaSuccess ? GDN_OK : cuda_fail(err, "gdn_gated_scan");
}

gdn_status gdn_gated_scan_backward(const gdn_scan_config* cfg, int32_t L, const gdn_tokens* x,
                                   const gdn_tokens* g, const float* hist,
                                   const gdn_tokens* grad_o, const float* grad_hT,
                                   const gdn_tokens* grad_x, const gdn_tokens* grad_g,
                                   float* grad_h0, const int32_t* lens, void* workspace,
                                   size_t workspace_bytes, gdn_stream_t stream) {
  clear_error();
  Shape s;
  GDNQ_TRY(check_scan(cfg, L, &s));
  if (s.empty()) return GDN_OK;
  const unsigned e = act_bytes(cfg->act_dtype);
  GDNQ_TRY(check_tokens(x, "x", s, e, false));
  GDNQ_TRY(check_tokens(g, "g", s, 4, false));
  GDNQ_TRY(check_tokens(grad_o, "grad_o", s, e, false));
  GDNQ_TRY(check_tokens(grad_x, "grad_x", s, e, true));
  GDNQ_TRY(check_tokens(grad_g, "grad_g", s, 4, true));
  if (L > 0) GDNQ_TRY(need_ptr(hist, "hist", 4));
  GDNQ_TRY(check_opt(grad_hT, "grad_hT", 4));
  GDNQ_TRY(check_opt(grad_h0, "grad_h0", 4));
  GDNQ_TRY(check_opt(lens, "lens", 4));
  gdnq::ScanArgs a{};
  a.x = tok(x), a.g = tok(g);
  a.grad_o = tok(grad_o), a.grad_x = tok(grad_x), a.grad_g = tok(grad_g);
  a.h0 = grad_hT, a.hT = grad_h0, a.hist = const_cast<float*>(hist), a.lens = lens;
  a.B = cfg->B, a.L = L, a.H = cfg->H, a.D = cfg->D, a.C = cfg->H * cfg->D;
  const size_t need = gdnq::scan_spans(a);
  GDNQ_TRY(check_workspace(workspace, workspace_bytes, need));
  gdnq::Arrays all;
  add(all, x, "x", s, e, false), add(all, g, "g", s, 4, false), add(all, grad_o, "grad_o", s, e, false);
  add(all, grad_x, "grad_x", s, e, true), add(all, grad_g, "grad_g", s, 4, true);
  const size_t state = 4 * s.heads();
  all.dense(grad_hT, "grad_hT", state, false), all.dense(grad_h0, "grad_h0", state, true);
  all.dense(hist, "hist", state * (size_t)chunks(L), false);
  all.dense(lens, "lens", 4 * (size_t)s.B, false), all.dense(workspace, "workspace", need, true);
  GDNQ_TRY(all.check(grad_h0, grad_hT));
  a.spans = need > 0 ? workspace : nullptr;
  const cudaError_t err = launch_scan(a, cfg, true, stream);
  return err == cudaSuccess ? GDN_OK : cuda_fail(err, "gdn_gated_scan_backward");
}

gdn_status gdn_group_norm(const gdn_norm_config* cfg, int32_t L, const gdn_tokens* x,
                          const float* w, const float* bias, const gdn_tokens* z,
                          const gdn_tokens* y, const int32_t* lens, gdn_stream_t stream) {
  clear_error();
  Shape s;
  GDNQ_TRY(check_norm(cfg, L, &s));
  if (s.empty()) return GDN_OK;
  const unsigned e = act_bytes(cfg->act_dtype);
  GDNQ_TRY(check_tokens(x, "x", s, e, false));
  if (z) GDNQ_TRY(check_tokens(z, "z", s, e, false));
  GDNQ_TRY(check_tokens(y, "y", s, e, true));
  if (L == 0) return GDN_OK;
  GDNQ_TRY(need_ptr(w, "w", 4));
  GDNQ_TRY(check_opt(bias, "bias", 4));
  GDNQ_TRY(check_opt(lens, "lens", 4));
  gdnq::Arrays all;
  add(all, x, "x", s, e, false), add(all, z, "z", s, e, false), add(all, y, "y", s, e, true);
  const size_t params = 4 * norm_params(cfg);
  all.dense(w, "w", params, false), all.dense(bias, "bias", params, false);
  all.dense(lens, "lens", 4 * (size_t)s.B, false);
  GDNQ_TRY(all.check());
  gdnq::NormArgs a = norm_args(cfg, L);
  a.x = tok(x), a.z = tok(z), a.y = tok(y);
  a.w = w, a.bias = bias, a.lens = lens;
  const cudaError_t err = launch_norm(a, cfg, false, stream);
  return err == cudaSuccess ? GDN_OK : cuda_fail(err, "gdn_group_norm");
}

size_t gdn_group_norm_backward_workspace_bytes(const gdn_norm_config* cfg, int32_t L) {
  clear_error();
  Shape s;
  if (check_norm(cfg, L, &s) != GDN_OK || s.empty() || L == 0) return 0;
  return gdnq::norm_backward_workspace(*cfg, L);
}

gdn_status gdn_group_norm_backward(const gdn_norm_config* cfg, int32_t L, const gdn_tokens* x,
                                   const float* w, const float* bias, const gdn_tokens* z,
                                   const gdn_tokens* grad_y, const gdn_tokens* grad_x,
                                   const gdn_tokens* grad_z, float* grad_w, float* grad_bias,
                                   const int32_t* lens, void* workspace, size_t workspace_bytes,
                                   gdn_stream_t stream) {
  clear_error();
  Shape s;
  GDNQ_TRY(check_norm(cfg, L, &s));
  if (s.H == 0 && cfg->weight == GDN_WEIGHT_CHANNEL) return GDN_OK;  // nothing is written
  if ((z == nullptr) != (grad_z == nullptr))
    return fail(GDN_ERR_INVALID_ARG, "grad_z goes with z");
  if ((bias == nullptr) != (grad_bias == nullptr))
    return fail(GDN_ERR_INVALID_ARG, "grad_bias goes with bias");
  GDNQ_TRY(need_ptr(grad_w, "grad_w", 4));
  GDNQ_TRY(check_opt(grad_bias, "grad_bias", 4));
  if (s.empty() || L == 0) {
    const size_t n = norm_params(cfg);
    GDNQ_TRY(zero(grad_w, n, stream, "gdn_group_norm_backward"));
    return zero(grad_bias, n, stream, "gdn_group_norm_backward");
  }
  const unsigned e = act_bytes(cfg->act_dtype);
  GDNQ_TRY(check_tokens(x, "x", s, e, false));
  if (z) GDNQ_TRY(check_tokens(z, "z", s, e, false));
  GDNQ_TRY(check_tokens(grad_y, "grad_y", s, e, false));
  GDNQ_TRY(check_tokens(grad_x, "grad_x", s, e, true));
  if (z) GDNQ_TRY(check_tokens(grad_z, "grad_z", s, e, true));
  GDNQ_TRY(need_ptr(w, "w", 4));
  GDNQ_TRY(check_opt(bias, "bias", 4));
  GDNQ_TRY(check_opt(lens, "lens", 4));
  const size_t need = gdnq::norm_backward_workspace(*cfg, L), params = 4 * norm_params(cfg);
  GDNQ_TRY(check_workspace(workspace, workspace_bytes, need));
  gdnq::Arrays all;
  add(all, x, "x", s, e, false), add(all, z, "z", s, e, false), add(all, grad_y, "grad_y", s, e, false);
  add(all, grad_x, "grad_x", s, e, true), add(all, grad_z, "grad_z", s, e, true);
  all.dense(w, "w", params, false), all.dense(bias, "bias", params, false);
  all.dense(grad_w, "grad_w", params, true), all.dense(grad_bias, "grad_bias", params, true);
  all.dense(lens, "lens", 4 * (size_t)s.B, false), all.dense(workspace, "workspace", need, true);
  GDNQ_TRY(all.check());
  gdnq::NormArgs a = norm_args(cfg, L);
  a.x = tok(x), a.z = tok(z);
  a.grad_y = tok(grad_y), a.grad_x = tok(grad_x), a.grad_z = tok(grad_z);
  a.w = w, a.bias = bias, a.grad_w = grad_w, a.grad_bias = grad_bias, a.lens = lens;
  a.partials = static_cast<float*>(workspace);
  const cudaError_t err = launch_norm(a, cfg, true, stream);
  return err == cudaSuccess ? GDN_OK : cuda_fail(err, "gdn_group_norm_backward");
}

gdn_status gdn_short_conv(const gdn_conv_config* cfg, int32_t L, const gdn_tokens* x,
                          const float* w, const float* bias, const void* state_in,
                          const gdn_tokens* y, void* state_out, const int32_t* lens,
                          gdn_stream_t stream) {
  clear_error();
  Shape s;
  GDNQ_TRY(check_conv(cfg, L, &s));
  if (s.empty()) return GDN_OK;
  const unsigned e = act_bytes(cfg->act_dtype);
  GDNQ_TRY(check_tokens(x, "x", s, e, false));
  GDNQ_TRY(check_tokens(y, "y", s, e, true));
  GDNQ_TRY(need_ptr(w, "w", 4));
  GDNQ_TRY(check_opt(bias, "bias", 4));
  GDNQ_TRY(check_opt(state_in, "state_in", e));
  GDNQ_TRY(check_opt(state_out, "state_out", e));
  GDNQ_TRY(check_opt(lens, "lens", 4));
  gdnq::Arrays all;
  add(all, x, "x", s, e, false), add(all, y, "y", s, e, true);
  const size_t C = (size_t)(s.H * s.D), state = (size_t)e * s.heads() * (size_t)(cfg->K - 1);
  all.dense(w, "w", 4 * C * (size_t)cfg->K, false), all.dense(bias, "bias", 4 * C, false);
  all.dense(state_in, "state_in", state, false), all.dense(state_out, "state_out", state, true);
  all.dense(lens, "lens", 4 * (size_t)s.B, false);
  GDNQ_TRY(all.check(state_out, state_in));
  gdnq::ConvArgs a{};
  a.x = tok(x), a.y = tok(y);
  a.w = w, a.bias = bias, a.state_in = state_in, a.state_out = state_out, a.lens = lens;
  a.B = cfg->B, a.L = L, a.H = cfg->H, a.D = cfg->D, a.C = cfg->H * cfg->D, a.K = cfg->K;
  a.activation = cfg->activation;
  const cudaError_t err = launch_conv(a, cfg, false, stream);
  return err == cudaSuccess ? GDN_OK : cuda_fail(err, "gdn_short_conv");
}

size_t gdn_short_conv_backward_workspace_bytes(const gdn_conv_config* cfg, int32_t L) {
  clear_error();
  Shape s;
  if (check_conv(cfg, L, &s) != GDN_OK || s.empty()) return 0;
  return gdnq::conv_backward_workspace(*cfg, L);
}

gdn_status gdn_short_conv_backward(const gdn_conv_config* cfg, int32_t L, const gdn_tokens* x,
                                   const float* w, const float* bias, const void* state_in,
                                   const gdn_tokens* grad_y, const void* grad_state_out,
                                   const gdn_tokens* grad_x, float* grad_w, float* grad_bias,
                                   void* grad_state_in, const int32_t* lens, void* workspace,
                                   size_t workspace_bytes, gdn_stream_t stream) {
  clear_error();
  Shape s;
  GDNQ_TRY(check_conv(cfg, L, &s));
  if (s.H == 0) return GDN_OK;
  if ((bias == nullptr) != (grad_bias == nullptr))
    return fail(GDN_ERR_INVALID_ARG, "grad_bias goes with bias");
  GDNQ_TRY(need_ptr(grad_w, "grad_w", 4));
  GDNQ_TRY(check_opt(grad_bias, "grad_bias", 4));
  if (s.B == 0) {
    const size_t n = (size_t)s.H * (size_t)s.D;
    GDNQ_TRY(zero(grad_w, n * (size_t)cfg->K, stream, "gdn_short_conv_backward"));
    return zero(grad_bias, n, stream, "gdn_short_conv_backward");
  }
  const unsigned e = act_bytes(cfg->act_dtype);
  GDNQ_TRY(check_tokens(x, "x", s, e, false));
  GDNQ_TRY(check_tokens(grad_y, "grad_y", s, e, false));
  GDNQ_TRY(check_tokens(grad_x, "grad_x", s, e, true));
  GDNQ_TRY(need_ptr(w, "w", 4));
  GDNQ_TRY(check_opt(bias, "bias", 4));
  GDNQ_TRY(check_opt(state_in, "state_in", e));
  GDNQ_TRY(check_opt(grad_state_out, "grad_state_out", e));
  GDNQ_TRY(check_opt(grad_state_in, "grad_state_in", e));
  GDNQ_TRY(check_opt(lens, "lens", 4));
  const size_t need = gdnq::conv_backward_workspace(*cfg, L);
  GDNQ_TRY(check_workspace(workspace, workspace_bytes, need));
  gdnq::Arrays all;
  add(all, x, "x", s, e, false), add(all, grad_y, "grad_y", s, e, false), add(all, grad_x, "grad_x", s, e, true);
  const size_t C = (size_t)(s.H * s.D), state = (size_t)e * s.heads() * (size_t)(cfg->K - 1);
  all.dense(w, "w", 4 * C * (size_t)cfg->K, false), all.dense(bias, "bias", 4 * C, false);
  all.dense(grad_w, "grad_w", 4 * C * (size_t)cfg->K, true), all.dense(grad_bias, "grad_bias", 4 * C, true);
  all.dense(state_in, "state_in", state, false);
  all.dense(grad_state_out, "grad_state_out", state, false);
  all.dense(grad_state_in, "grad_state_in", state, true);
  all.dense(lens, "lens", 4 * (size_t)s.B, false), all.dense(workspace, "workspace", need, true);
  GDNQ_TRY(all.check());
  gdnq::ConvArgs a{};
  a.x = tok(x), a.grad_y = tok(grad_y), a.grad_x = tok(grad_x);
  a.w = w, a.bias = bias, a.state_in = state_in, a.grad_state_out = grad_state_out;
  a.grad_w = grad_w, a.grad_bias = grad_bias, a.grad_state_in = grad_state_in, a.lens = lens;
  a.partials = static_cast<float*>(workspace);
  a.B = cfg->B, a.L = L, a.H = cfg->H, a.D = cfg->D, a.C = cfg->H * cfg->D, a.K = cfg->K;
  a.activation = cfg->activation;
  const cudaError_t err = launch_conv(a, cfg, true, stream);
  return err == cudaSuccess ? GDN_OK : cuda_fail(err, "gdn_short_conv_backward");
}

}  // extern "C"
