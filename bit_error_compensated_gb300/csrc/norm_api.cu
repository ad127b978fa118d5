// norm_api.cu -- host side of the residual join: plans, argument checks,
// launches (contract in include/echo.h).
#include <cmath>
#include <cstring>
#include <new>

#include "norm_common.h"

struct echo_norm_plan_s {
  int width = 0, dtype = 0, param_dtype = 0, kind = 0, post = 0, device = 0, sms = 0;
  float eps = 0.f, scale = 1.f;
  float* workspace = nullptr;        // [6][workers][width]: four sums and two gate slots
  int64_t workers = 0;
};

namespace {
using namespace echo;

bool aligned(const void* p, uintptr_t a) { return p == nullptr || on_boundary(p, a); }

// One tensor of a call: absent, or checked for its row distance and element
// alignment; `vec` is cleared where 16-byte accesses are not possible.
int check_rows(const void* p, int64_t ld, int64_t rows, int width, int size, bool* vec) {
  if (p == nullptr) return ECHO_OK;
  if (rows > 1 && (ld < width || ld > ((int64_t)1 << 40))) return ECHO_ERR_SHAPE;
  if (!on_boundary(p, size)) return ECHO_ERR_ALIGN;
  if (!on_boundary(p, 16) || (rows > 1 && ld * size % 16 != 0)) *vec = false;
  return ECHO_OK;
}

int check_params(const echo_norm_plan_s* plan, const echo_norm_params* p, bool* vec) {
  if (p == nullptr) return ECHO_OK;
  const int size = elem_size(plan->param_dtype);
  if (!plan->post && (p->w_post || p->b_post)) return ECHO_ERR_ARG;
  if (plan->kind == ECHO_NORM_RMS && (p->b_post || p->b_pre)) return ECHO_ERR_ARG;
  const void* all[4] = {p->w_post, p->b_post, p->w_pre, p->b_pre};
  for (const void* v : all) {
    if (!aligned(v, size)) return ECHO_ERR_ALIGN;
    if (!aligned(v, 16)) *vec = false;
  }
  return ECHO_OK;
}

// A gate of gate_rows x gate_cols: how many rows share one of its rows.
int check_gate(const echo_norm_plan_s* plan, const void* gate, int64_t gate_rows, int64_t gate_cols,
               int64_t rows, const void* y, int64_t* span, bool* vec) {
  *span = 1;
  if (gate == nullptr) return ECHO_OK;
  if (y == nullptr && rows > 0) return ECHO_ERR_ARG;
  if (gate_cols != plan->width && gate_cols != 1) return ECHO_ERR_SHAPE;
  if (gate_rows < 1 || rows % gate_rows != 0) return ECHO_ERR_SHAPE;
  const int size = elem_size(plan->param_dtype);
  if (!on_boundary(gate, size)) return ECHO_ERR_ALIGN;
  if (gate_cols == plan->width && !on_boundary(gate, 16)) *vec = false;
  *span = rows / gate_rows > 0 ? rows / gate_rows : 1;
  return ECHO_OK;
}

int check_device(const echo_norm_plan_s* plan) {
  int dev = -1;
  ECHO_OPS_CUDA(cudaGetDevice(&dev));
  return dev == plan->device ? ECHO_OK : ECHO_ERR_ARG;
}

#define ECHO_TRY(call)                  \
  do {                                  \
    const int rc_ = (call);             \
    if (rc_ != ECHO_OK) return rc_;     \
  } while (0)

Region vector_region(const void* p, int64_t n, int size) { return region(p, 1, n, n, size); }

}  // namespace

extern "C" {

int echo_norm_plan(int64_t width, int dtype, int param_dtype, int kind, int post, float eps,
                   float scale, echo_norm_plan_t* out) {
  if (out == nullptr) return ECHO_ERR_ARG;
  *out = nullptr;
  if (kind != ECHO_NORM_RMS && kind != ECHO_NORM_LAYER) return ECHO_ERR_ARG;
  if (post != 0 && post != 1) return ECHO_ERR_ARG;
  if (!std::isfinite(eps) || eps < 0.f || !std::isfinite(scale)) return ECHO_ERR_ARG;
  if (!known_dtype(dtype) || !known_dtype(param_dtype)) return ECHO_ERR_UNSUPPORTED;
  if (param_dtype != dtype && param_dtype != ECHO_F32) return ECHO_ERR_UNSUPPORTED;
  if (width < 1) return ECHO_ERR_SHAPE;
  if (width > ECHO_NORM_MAX_WIDTH) return ECHO_ERR_UNSUPPORTED;

  echo_norm_plan_s* p = new (std::nothrow) echo_norm_plan_s();
  if (p == nullptr) return ECHO_ERR_ARG;
  p->width = (int)width;
  p->dtype = dtype;
  p->param_dtype = param_dtype;
  p->kind = kind;
  p->post = post;
  p->eps = eps;
  p->scale = scale;
  cudaError_t e = cudaGetDevice(&p->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&p->sms, cudaDevAttrMultiProcessorCount, p->device);
  if (e == cudaSuccess) {
    p->workers = norm_grad_max_workers(p->width, p->sms);
    e = cudaMalloc((void**)&p->workspace, (size_t)(6 * p->workers * width) * sizeof(float));
  }
  if (e != cudaSuccess) {
    echo_norm_plan_destroy(p);
    cudaGetLastError();                // the caller's next check is not this call's
    return note_cuda_error(e);
  }
  *out = p;
  return ECHO_OK;
}

void echo_norm_plan_destroy(echo_norm_plan_t plan) {
  if (plan == nullptr) return;
  if (plan->workspace) cudaFree(plan->workspace);
  delete plan;
}

int echo_norm(echo_norm_plan_t plan, const echo_norm_params* params, const echo_norm_io* io,
              void* stream) {
  if (plan == nullptr || io == nullptr) return ECHO_ERR_ARG;
  static const echo_norm_params none = {nullptr, nullptr, nullptr, nullptr};
  const echo_norm_params& p = params ? *params : none;
  const int64_t T = io->rows;
  const int W = plan->width, size = elem_size(plan->dtype);
  if (T < 0) return ECHO_ERR_SHAPE;
  if (io->x == nullptr && T > 0) return ECHO_ERR_ARG;
  if ((io->codes == nullptr) != (io->scales == nullptr)) return ECHO_ERR_ARG;
  const int code_vec = 16 / size;
  bool vec = W * size % 16 == 0;
  ECHO_TRY(check_rows(io->x, io->ld_x, T, W, size, &vec));
  ECHO_TRY(check_rows(io->y, io->ld_y, T, W, size, &vec));
  ECHO_TRY(check_rows(io->r, io->ld_r, T, W, size, &vec));
  ECHO_TRY(check_rows(io->h, io->ld_h, T, W, size, &vec));
  if (io->codes) {
    if (T > 1 && (io->ld_codes < W || io->ld_codes > ((int64_t)1 << 40))) return ECHO_ERR_SHAPE;
    if (!on_boundary(io->codes, code_vec) || (T > 1 && io->ld_codes % code_vec != 0)) vec = false;
    if (!on_boundary(io->scales, 4)) return ECHO_ERR_ALIGN;
  }
  if (!aligned(io->stats, 16)) return ECHO_ERR_ALIGN;
  ECHO_TRY(check_params(plan, &p, &vec));
  int64_t span = 1;
  ECHO_TRY(check_gate(plan, io->gate, io->gate_rows, io->gate_cols, T, io->y, &span, &vec));

  const int psize = elem_size(plan->param_dtype);
  const Region x = region(io->x, T, W, io->ld_x, size), y = region(io->y, T, W, io->ld_y, size);
  const Region r = region(io->r, T, W, io->ld_r, size), h = region(io->h, T, W, io->ld_h, size);
  const Region out[5] = {r, h, region(io->codes, T, W, io->ld_codes, 1),
                         vector_region(io->scales, T, 4), vector_region(io->stats, 4 * T, 4)};
  const Region in[7] = {x, y, vector_region(io->gate, io->gate ? io->gate_rows * io->gate_cols : 0, psize),
                        vector_region(p.w_post, W, psize), vector_region(p.b_post, W, psize),
                        vector_region(p.w_pre, W, psize), vector_region(p.b_pre, W, psize)};
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < 7; ++j) {
      if ((i == 0 && j == 0) || (i == 1 && j == 1)) {
        if (out[i].rows && same(out[i], in[j])) continue;       // r in place of x, h of y
      }
      if (overlaps(out[i], in[j])) return ECHO_ERR_ARG;
    }
    for (int j = i + 1; j < 5; ++j)
      if (overlaps(out[i], out[j])) return ECHO_ERR_ARG;
  }
  ECHO_TRY(check_device(plan));
  if (T == 0 || !(io->r || io->h || io->codes || io->stats)) return ECHO_OK;

  NormArgs a;
  std::memset(&a, 0, sizeof(a));
  a.rows = T;
  a.width = W;
  a.x = io->x; a.ld_x = io->ld_x;
  a.y = io->y; a.ld_y = io->ld_y;
  a.gate = io->gate;
  a.gate_span = span;
  a.gate_scalar = io->gate && io->gate_cols == 1 && W != 1;
  a.w_post = p.w_post; a.b_post = p.b_post; a.w_pre = p.w_pre; a.b_pre = p.b_pre;
  a.r = io->r; a.ld_r = io->ld_r;
  a.h = io->h; a.ld_h = io->ld_h;
  a.codes = io->codes; a.ld_codes = io->ld_codes;
  a.scales = io->scales;
  a.stats = io->stats;
  a.eps = plan->eps;
  a.scale = plan->scale;
  a.post = plan->post && io->y;
  a.params_f32 = plan->param_dtype == ECHO_F32;
  const int layer = plan->kind == ECHO_NORM_LAYER;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  ECHO_OPS_CUDA(plan->dtype == ECHO_F32    ? launch_norm<float>(a, layer, vec, plan->sms, s)
                : plan->dtype == ECHO_BF16 ? launch_norm<__nv_bfloat16>(a, layer, vec, plan->sms, s)
                                           : launch_norm<__half>(a, layer, vec, plan->sms, s));
  return ECHO_OK;
}

int echo_norm_backward(echo_norm_plan_t plan, const echo_norm_params* params,
                       const echo_norm_grad_io* io, const echo_norm_params* grads, void* stream) {
  if (plan == nullptr || io == nullptr) return ECHO_ERR_ARG;
  static const echo_norm_params none = {nullptr, nullptr, nullptr, nullptr};
  const echo_norm_params& p = params ? *params : none;
  const echo_norm_params& g = grads ? *grads : none;
  const int64_t T = io->rows;
  const int W = plan->width, size = elem_size(plan->dtype), psize = elem_size(plan->param_dtype);
  if (T < 0) return ECHO_ERR_SHAPE;
  if (io->x == nullptr && T > 0) return ECHO_ERR_ARG;
  if (io->y == nullptr && io->dy != nullptr) return ECHO_ERR_ARG;
  if (io->gate == nullptr && io->dgate != nullptr) return ECHO_ERR_ARG;
  bool vec = W * size % 16 == 0;
  ECHO_TRY(check_rows(io->x, io->ld_x, T, W, size, &vec));
  ECHO_TRY(check_rows(io->y, io->ld_y, T, W, size, &vec));
  ECHO_TRY(check_rows(io->dr, io->ld_dr, T, W, size, &vec));
  ECHO_TRY(check_rows(io->dh, io->ld_dh, T, W, size, &vec));
  ECHO_TRY(check_rows(io->dx, io->ld_dx, T, W, size, &vec));
  ECHO_TRY(check_rows(io->dy, io->ld_dy, T, W, size, &vec));
  if (!aligned(io->stats, 16)) return ECHO_ERR_ALIGN;
  ECHO_TRY(check_params(plan, &p, &vec));
  ECHO_TRY(check_params(plan, &g, &vec));
  int64_t span = 1;
  ECHO_TRY(check_gate(plan, io->gate, io->gate_rows, io->gate_cols, T, io->y, &span, &vec));
  int64_t dgate_span = 1;            // the same, or 1 without dgate
  ECHO_TRY(check_gate(plan, io->dgate, io->gate_rows, io->gate_cols, T, io->y, &dgate_span, &vec));
  const bool post = plan->post && io->y;
  if (T > 0 && io->stats == nullptr && (post || io->dh)) return ECHO_ERR_ARG;

  const int64_t gate_n = io->gate ? io->gate_rows * io->gate_cols : 0;
  const Region out[7] = {region(io->dx, T, W, io->ld_dx, size), region(io->dy, T, W, io->ld_dy, size),
                         vector_region(io->dgate, gate_n, psize),
                         vector_region(g.w_post, W, psize), vector_region(g.b_post, W, psize),
                         vector_region(g.w_pre, W, psize), vector_region(g.b_pre, W, psize)};
  const Region in[10] = {region(io->dr, T, W, io->ld_dr, size), region(io->dh, T, W, io->ld_dh, size),
                         region(io->y, T, W, io->ld_y, size), region(io->x, T, W, io->ld_x, size),
                         vector_region(io->stats, 4 * T, 4), vector_region(io->gate, gate_n, psize),
                         vector_region(p.w_post, W, psize), vector_region(p.b_post, W, psize),
                         vector_region(p.w_pre, W, psize), vector_region(p.b_pre, W, psize)};
  for (int i = 0; i < 7; ++i) {
    for (int j = 0; j < 10; ++j) {
      // dx in place of dr or dh, dy of dr, dh or y: each element is read by
      // the thread that writes it, before it does.
      const bool in_place = (i == 0 && j < 2) || (i == 1 && j < 3);
      if (in_place && out[i].rows && same(out[i], in[j])) continue;
      if (overlaps(out[i], in[j])) return ECHO_ERR_ARG;
    }
    for (int j = i + 1; j < 7; ++j)
      if (overlaps(out[i], out[j])) return ECHO_ERR_ARG;
  }
  ECHO_TRY(check_device(plan));

  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  void* const dparam[4] = {g.w_post, g.b_post, g.w_pre, g.b_pre};
  if (T == 0) {                      // sums over no rows
    for (void* d : dparam)
      if (d) ECHO_OPS_CUDA(cudaMemsetAsync(d, 0, (size_t)W * psize, s));
    if (io->dgate) ECHO_OPS_CUDA(cudaMemsetAsync(io->dgate, 0, (size_t)(gate_n * psize), s));
    return ECHO_OK;
  }
  NormGradArgs a;
  std::memset(&a, 0, sizeof(a));
  a.rows = T;
  a.width = W;
  a.x = io->x; a.ld_x = io->ld_x;
  a.y = io->y; a.ld_y = io->ld_y;
  a.gate = io->gate;
  a.gate_span = span;
  a.gate_scalar = io->gate && io->gate_cols == 1 && W != 1;
  a.w_post = p.w_post; a.b_post = p.b_post; a.w_pre = p.w_pre;
  a.stats = io->stats;
  a.dr = io->dr; a.ld_dr = io->ld_dr;
  a.dh = io->dh; a.ld_dh = io->ld_dh;
  a.dx = io->dx; a.ld_dx = io->ld_dx;
  a.dy = io->dy; a.ld_dy = io->ld_dy;
  a.dgate = io->dgate;
  const int64_t stride = plan->workers * W;
  for (int k = 0; k < 4; ++k) {
    a.dparam[k] = dparam[k];
    // the first two are dgate's too
    a.partial[k] = dparam[k] || (k < 2 && io->dgate) ? plan->workspace + k * stride : nullptr;
  }
  a.gate_partial = plan->workspace + 4 * stride;
  a.scale = plan->scale;
  a.post = post;
  a.params_f32 = plan->param_dtype == ECHO_F32;
  const int layer = plan->kind == ECHO_NORM_LAYER;
  ECHO_OPS_CUDA(plan->dtype == ECHO_F32    ? launch_norm_grad<float>(a, layer, vec, plan->sms, s)
                : plan->dtype == ECHO_BF16 ? launch_norm_grad<__nv_bfloat16>(a, layer, vec, plan->sms, s)
                                           : launch_norm_grad<__half>(a, layer, vec, plan->sms, s));
  return ECHO_OK;
}

}  // extern "C"
