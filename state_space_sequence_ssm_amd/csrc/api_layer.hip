// C ABI of the layer operators (causal convolution, selective scan, gated and
// residual norms): host-side validation and dispatch.  Every check runs on the
// host before any HIP call.
#include <initializer_list>

#include "layer_internal.hpp"

namespace {

constexpr double kMaxElems = 34359738368.0;  // 2^35 elements of one tensor
constexpr double kMaxInt = 2147483647.0;
constexpr int kMaxWidth = 1 << 28;   // L and D: an index a block's width past them stays in 32 bits
constexpr int kMaxGroups = 1 << 20;  // of a norm's row

bool ok_dtype(int t) { return t == M3_F32 || t == M3_BF16; }
size_t elem(int t) { return t == M3_BF16 ? 2 : 4; }
bool flag(int v) { return v == 0 || v == 1; }
bool at(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool all_at(std::initializer_list<const void*> ps, size_t a) {
  for (const void* p : ps)
    if (!at(p, a)) return false;
  return true;
}
bool all_set(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (p == nullptr) return false;
  return true;
}
// Whether any output is one of the inputs or another output.
bool clash(std::initializer_list<const void*> outs, std::initializer_list<const void*> ins) {
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    if (*o == nullptr) continue;
    for (const void* i : ins)
      if (*o == i) return true;
    for (auto q = outs.begin(); q != o; ++q)
      if (*q == *o) return true;
  }
  return false;
}
// Distance between rows of `width` elements: 0 = dense.
bool set_ld(int64_t& ld, int64_t width) {
  if (ld == 0) ld = width;
  return ld >= width && ld < (int64_t(1) << 31);
}
// The scan's tiles address their rows with 32 bits.
bool scan_ld(int64_t& ld, int64_t width) { return set_ld(ld, width) && ld < (int64_t(1) << 24); }
bool ok_eps(float e) { return e >= 0.f && e <= 3.0e38f; }
int hip_status(hipError_t e) { return e == hipSuccess ? M3_OK : M3_ERR_HIP; }
hipStream_t str(void* s) { return static_cast<hipStream_t>(s); }

int check_rows(int64_t Bt, int64_t L, int64_t D) {
  if (Bt < 1 || L < 1 || D < 1) return M3_ERR_INVALID_ARG;
  if (double(Bt) * D > kMaxInt || double(Bt) * L * D > kMaxElems || L > kMaxWidth || D > kMaxWidth) return M3_ERR_UNSUPPORTED;
  return M3_OK;
}

int check_conv_shape(int64_t Bt, int64_t L, int64_t D, int W, int dtype, int silu) {
  const int rc = check_rows(Bt, L, D);
  if (rc != M3_OK) return rc;
  if (!ok_dtype(dtype) || W < 2 || W > 4) return M3_ERR_UNSUPPORTED;
  return flag(silu) ? M3_OK : M3_ERR_INVALID_ARG;
}

int check_scan_shape(int64_t Bt, int64_t L, int64_t D, int N, int G, int dtype, int softplus) {
  const int rc = check_rows(Bt, L, D);
  if (rc != M3_OK) return rc;
  if (N < 1 || G < 1 || D % G != 0 || !flag(softplus)) return M3_ERR_INVALID_ARG;
  // 64 states and 128 values of B and C per row are what the blocks' tiles hold
  if (!ok_dtype(dtype) || N > 64 || double(Bt) * L * G * 128 > 256.0 * kMaxInt) return M3_ERR_UNSUPPORTED;
  return M3_OK;
}

// Inputs shared by the scan and its backward; fills the row distances.
int check_scan_inputs(m3_scan_args& f) {
  const int rc = check_scan_shape(f.Bt, f.L, f.D, f.N, f.G, f.in_dtype, f.dt_softplus);
  if (rc != M3_OK) return rc;
  if (!all_set({f.x, f.dt, f.A, f.B, f.C}) || (f.dt_bias != nullptr && !f.dt_softplus)) return M3_ERR_INVALID_ARG;
  const int64_t GN = int64_t(f.G) * f.N;
  if (!scan_ld(f.x_ld, f.D) || !scan_ld(f.dt_ld, f.D) || !scan_ld(f.z_ld, f.D) || !scan_ld(f.B_ld, GN) || !scan_ld(f.C_ld, GN))
    return M3_ERR_INVALID_ARG;
  if (!all_at({f.x, f.dt, f.B, f.C, f.z}, elem(f.in_dtype)) || !all_at({f.A, f.D_skip, f.dt_bias, f.h0, f.lengths}, 4))
    return M3_ERR_INVALID_ARG;
  return M3_OK;
}

bool ok_scan_size(const m3_scan_args* a) {
  return a != nullptr && check_scan_shape(a->Bt, a->L, a->D, a->N, a->G, a->in_dtype, 0) == M3_OK;
}

int check_gated(m3_gated_norm_args& f) {
  if (f.M < 1 || f.D < 1 || f.G < 1 || f.D % f.G != 0 || !flag(f.gate_first) || !ok_eps(f.eps)) return M3_ERR_INVALID_ARG;
  if (!ok_dtype(f.in_dtype) || f.G > kMaxGroups || f.D > kMaxWidth || double(f.M) * f.G > kMaxInt || double(f.M) * f.D > kMaxElems)
    return M3_ERR_UNSUPPORTED;
  if (f.x == nullptr || !set_ld(f.x_ld, f.D) || !set_ld(f.z_ld, f.D)) return M3_ERR_INVALID_ARG;
  return all_at({f.x, f.z}, elem(f.in_dtype)) && at(f.w, 4) ? M3_OK : M3_ERR_INVALID_ARG;
}
bool ok_gated_size(const m3_gated_norm_args& f) {
  return f.M >= 1 && f.D >= 1 && f.G >= 1 && f.D % f.G == 0 && f.G <= kMaxGroups && f.D <= kMaxWidth && ok_dtype(f.in_dtype) &&
         double(f.M) * f.G <= kMaxInt && double(f.M) * f.D <= kMaxElems;
}

int check_residual_shape(int64_t M, int64_t D, int in_dtype, int res_dtype, float eps) {
  if (M < 1 || D < 1 || !ok_eps(eps)) return M3_ERR_INVALID_ARG;
  if (!ok_dtype(in_dtype) || (res_dtype != in_dtype && res_dtype != M3_F32)) return M3_ERR_UNSUPPORTED;
  if (D > kMaxWidth || double(M) > kMaxInt || double(M) * D > kMaxElems) return M3_ERR_UNSUPPORTED;
  return M3_OK;
}

}  // namespace

extern "C" {

int m3_causal_conv(const m3_conv_args* args, void* stream) {
  if (args == nullptr) return M3_ERR_INVALID_ARG;
  m3_conv_args a = *args;
  const int rc = check_conv_shape(a.Bt, a.L, a.D, a.W, a.in_dtype, a.silu);
  if (rc != M3_OK) return rc;
  if (!all_set({a.x, a.w, a.y}) || !set_ld(a.x_ld, a.D)) return M3_ERR_INVALID_ARG;
  if (!all_at({a.x, a.state, a.y, a.state_out}, elem(a.in_dtype)) || !all_at({a.w, a.bias, a.lengths}, 4)) return M3_ERR_INVALID_ARG;
  if (clash({a.y, a.state_out}, {a.x, a.w, a.bias, a.lengths}) || a.y == a.state) return M3_ERR_INVALID_ARG;
  return hip_status(m3::launch_conv(a, str(stream)));
}

int m3_causal_conv_step(const m3_conv_step_args* args, void* stream) {
  if (args == nullptr) return M3_ERR_INVALID_ARG;
  m3_conv_step_args a = *args;
  const int rc = check_conv_shape(a.Bt, 1, a.D, a.W, a.in_dtype, a.silu);
  if (rc != M3_OK) return rc;
  if (!all_set({a.x, a.w, a.y, a.state}) || !set_ld(a.x_ld, a.D)) return M3_ERR_INVALID_ARG;
  if (a.state_out == nullptr) a.state_out = a.state;
  if (!all_at({a.x, a.state, a.y, a.state_out}, elem(a.in_dtype)) || !all_at({a.w, a.bias}, 4)) return M3_ERR_INVALID_ARG;
  if (clash({a.y, a.state_out}, {a.x, a.w, a.bias}) || a.y == a.state) return M3_ERR_INVALID_ARG;
  return hip_status(m3::launch_conv_step(a, str(stream)));
}

size_t m3_causal_conv_backward_workspace_size(const m3_conv_backward_args* a) {
  if (a == nullptr || check_conv_shape(a->Bt, a->L, a->D, a->W, a->in_dtype, 0) != M3_OK) return 0;
  return m3::conv_backward_workspace(*a);
}

int m3_causal_conv_backward(const m3_conv_backward_args* args, void* stream) {
  if (args == nullptr) return M3_ERR_INVALID_ARG;
  m3_conv_backward_args a = *args;
  const int rc = check_conv_shape(a.Bt, a.L, a.D, a.W, a.in_dtype, a.silu);
  if (rc != M3_OK) return rc;
  const size_t need = m3::conv_backward_workspace(a);
  if (need == 0) return M3_ERR_UNSUPPORTED;
  if (!all_set({a.x, a.w, a.dy, a.dx, a.dw, a.workspace}) || !set_ld(a.x_ld, a.D)) return M3_ERR_INVALID_ARG;
  if (!all_at({a.x, a.state, a.dy, a.dx, a.dstate}, elem(a.in_dtype)) || !all_at({a.w, a.bias, a.lengths, a.dw, a.dbias}, 4))
    return M3_ERR_INVALID_ARG;
  if (clash({a.dx, a.dw, a.dbias, a.dstate, a.workspace}, {a.x, a.w, a.bias, a.lengths, a.state, a.dy})) return M3_ERR_INVALID_ARG;
  if (!at(a.workspace, 256) || a.workspace_bytes < need) return M3_ERR_INVALID_ARG;
  return hip_status(m3::launch_conv_backward(a, str(stream)));
}

size_t m3_selective_scan_workspace_size(const m3_scan_args* a) {
  return ok_scan_size(a) && m3::scan_fits(*a) ? m3::scan_workspace(*a) : 0;
}

int m3_selective_scan(const m3_scan_args* args, void* stream) {
  if (args == nullptr) return M3_ERR_INVALID_ARG;
  m3_scan_args a = *args;
  const int rc = check_scan_inputs(a);
  if (rc != M3_OK) return rc;
  if (!m3::scan_fits(a)) return M3_ERR_UNSUPPORTED;
  if (a.y == nullptr || !at(a.y, elem(a.in_dtype)) || !at(a.h_final, 4)) return M3_ERR_INVALID_ARG;
  if (clash({a.y, a.h_final, a.workspace}, {a.x, a.dt, a.z, a.B, a.C, a.A, a.D_skip, a.dt_bias, a.h0, a.lengths}))
    return M3_ERR_INVALID_ARG;
  if (a.workspace != nullptr && (!at(a.workspace, 256) || a.workspace_bytes < m3::scan_workspace(a))) return M3_ERR_INVALID_ARG;
  return hip_status(m3::launch_scan(a, str(stream)));
}

int m3_selective_scan_step(const m3_scan_step_args* args, void* stream) {
  if (args == nullptr) return M3_ERR_INVALID_ARG;
  m3_scan_step_args a = *args;
  const int rc = check_scan_shape(a.Bt, 1, a.D, a.N, a.G, a.in_dtype, a.dt_softplus);
  if (rc != M3_OK) return rc;
  if (!m3::scan_step_fits(a)) return M3_ERR_UNSUPPORTED;
  if (!all_set({a.x, a.dt, a.A, a.B, a.C, a.h, a.y}) || (a.dt_bias != nullptr && !a.dt_softplus)) return M3_ERR_INVALID_ARG;
  const int64_t GN = int64_t(a.G) * a.N;
  if (!scan_ld(a.x_ld, a.D) || !scan_ld(a.dt_ld, a.D) || !scan_ld(a.z_ld, a.D) || !scan_ld(a.B_ld, GN) || !scan_ld(a.C_ld, GN))
    return M3_ERR_INVALID_ARG;
  if (a.h_out == nullptr) a.h_out = a.h;
  if (!all_at({a.x, a.dt, a.B, a.C, a.z, a.y}, elem(a.in_dtype)) || !all_at({a.A, a.D_skip, a.dt_bias, a.h, a.h_out}, 4))
    return M3_ERR_INVALID_ARG;
  if (clash({a.y, a.h_out}, {a.x, a.dt, a.z, a.B, a.C, a.A, a.D_skip, a.dt_bias}) || a.y == a.h) return M3_ERR_INVALID_ARG;
  return hip_status(m3::launch_scan_step(a, str(stream)));
}

size_t m3_selective_scan_backward_workspace_size(const m3_scan_backward_args* a) {
  return a != nullptr && ok_scan_size(&a->fwd) ? m3::scan_backward_workspace(*a) : 0;
}

int m3_selective_scan_backward(const m3_scan_backward_args* args, void* stream) {
  if (args == nullptr) return M3_ERR_INVALID_ARG;
  m3_scan_backward_args a = *args;
  const int rc = check_scan_inputs(a.fwd);
  if (rc != M3_OK) return rc;
  const size_t need = m3::scan_backward_workspace(a);
  if (need == 0) return M3_ERR_UNSUPPORTED;
  const m3_scan_args& f = a.fwd;
  if (!all_set({a.dy, a.dx, a.ddt, a.dA, a.dB, a.dC, a.workspace})) return M3_ERR_INVALID_ARG;
  if ((f.D_skip == nullptr) != (a.dD == nullptr) || (f.z == nullptr) != (a.dz == nullptr) ||
      (f.dt_bias == nullptr) != (a.ddt_bias == nullptr))
    return M3_ERR_INVALID_ARG;
  if (!all_at({a.dy, a.dx, a.ddt, a.dB, a.dC, a.dz}, elem(f.in_dtype)) || !all_at({a.dh_final, a.dA, a.dD, a.ddt_bias, a.dh0}, 4))
    return M3_ERR_INVALID_ARG;
  if (clash({a.dx, a.ddt, a.dA, a.dB, a.dC, a.dD, a.dz, a.ddt_bias, a.dh0, a.workspace},
            {f.x, f.dt, f.z, f.B, f.C, f.A, f.D_skip, f.dt_bias, f.h0, f.lengths, a.dy, a.dh_final}))
    return M3_ERR_INVALID_ARG;
  if (!at(a.workspace, 256) || a.workspace_bytes < need) return M3_ERR_INVALID_ARG;
  return hip_status(m3::launch_scan_backward(a, str(stream)));
}

int m3_gated_norm(const m3_gated_norm_args* args, void* stream) {
  if (args == nullptr) return M3_ERR_INVALID_ARG;
  m3_gated_norm_args a = *args;
  const int rc = check_gated(a);
  if (rc != M3_OK) return rc;
  if (a.y == nullptr || !at(a.y, elem(a.in_dtype)) || a.y == a.w) return M3_ERR_INVALID_ARG;
  // in place only over rows that lie as y's do
  if ((a.y == a.x && a.x_ld != a.D) || (a.y == a.z && a.z_ld != a.D)) return M3_ERR_INVALID_ARG;
  return hip_status(m3::launch_gated_norm(a, str(stream)));
}

size_t m3_gated_norm_backward_workspace_size(const m3_gated_norm_backward_args* a) {
  return a != nullptr && ok_gated_size(a->fwd) && m3::gated_norm_backward_fits(*a) ? m3::gated_norm_backward_workspace(*a) : 0;
}

int m3_gated_norm_backward(const m3_gated_norm_backward_args* args, void* stream) {
  if (args == nullptr) return M3_ERR_INVALID_ARG;
  m3_gated_norm_backward_args a = *args;
  const int rc = check_gated(a.fwd);
  if (rc != M3_OK) return rc;
  if (!m3::gated_norm_backward_fits(a)) return M3_ERR_UNSUPPORTED;
  const m3_gated_norm_args& f = a.fwd;
  if (!all_set({a.dy, a.dx}) || (f.z == nullptr) != (a.dz == nullptr) || (f.w == nullptr) != (a.dw == nullptr))
    return M3_ERR_INVALID_ARG;
  if (!all_at({a.dy, a.dx, a.dz}, elem(f.in_dtype)) || !at(a.dw, 4)) return M3_ERR_INVALID_ARG;
  if (clash({a.dx, a.dz, a.dw, a.workspace}, {f.x, f.z, f.w, a.dy})) return M3_ERR_INVALID_ARG;
  const size_t need = m3::gated_norm_backward_workspace(a);
  if (need > 0 && (a.workspace == nullptr || !at(a.workspace, 256) || a.workspace_bytes < need)) return M3_ERR_INVALID_ARG;
  return hip_status(m3::launch_gated_norm_backward(a, str(stream)));
}

int m3_residual_norm(const m3_residual_norm_args* args, void* stream) {
  if (args == nullptr) return M3_ERR_INVALID_ARG;
  m3_residual_norm_args a = *args;
  const int rc = check_residual_shape(a.M, a.D, a.in_dtype, a.res_dtype, a.eps);
  if (rc != M3_OK) return rc;
  if (!all_set({a.x, a.y}) || !set_ld(a.x_ld, a.D)) return M3_ERR_INVALID_ARG;
  if (!all_at({a.x, a.y}, elem(a.in_dtype)) || !all_at({a.residual, a.residual_out}, elem(a.res_dtype)) || !all_at({a.scale, a.w}, 4))
    return M3_ERR_INVALID_ARG;
  if (clash({a.y, a.residual_out}, {a.x, a.scale, a.w}) || a.y == a.residual) return M3_ERR_INVALID_ARG;
  return hip_status(m3::launch_residual_norm(a, str(stream)));
}

size_t m3_residual_norm_backward_workspace_size(const m3_residual_norm_backward_args* a) {
  if (a == nullptr || check_residual_shape(a->M, a->D, a->in_dtype, a->res_dtype, 0.f) != M3_OK) return 0;
  return m3::residual_norm_backward_fits(*a) ? m3::residual_norm_backward_workspace(*a) : 0;
}

int m3_residual_norm_backward(const m3_residual_norm_backward_args* args, void* stream) {
  if (args == nullptr) return M3_ERR_INVALID_ARG;
  m3_residual_norm_backward_args a = *args;
  const int rc = check_residual_shape(a.M, a.D, a.in_dtype, a.res_dtype, a.eps);
  if (rc != M3_OK) return rc;
  if (!m3::residual_norm_backward_fits(a)) return M3_ERR_UNSUPPORTED;
  if (!all_set({a.h, a.dy}) || !set_ld(a.x_ld, a.D)) return M3_ERR_INVALID_ARG;
  if ((a.w == nullptr) != (a.dw == nullptr) || (a.scale == nullptr) != (a.dscale == nullptr)) return M3_ERR_INVALID_ARG;
  if (a.scale != nullptr && a.x == nullptr) return M3_ERR_INVALID_ARG;
  if (!all_at({a.x, a.dy, a.dx}, elem(a.in_dtype)) || !all_at({a.h, a.dresidual_out, a.dresidual}, elem(a.res_dtype)) ||
      !all_at({a.scale, a.w, a.dw, a.dscale}, 4))
    return M3_ERR_INVALID_ARG;
  if (clash({a.dx, a.dresidual, a.dw, a.dscale, a.workspace}, {a.h, a.x, a.scale, a.w, a.dy}) ||
      (a.dresidual_out != nullptr && (a.dx == a.dresidual_out || a.workspace == a.dresidual_out)))
    return M3_ERR_INVALID_ARG;
  const size_t need = m3::residual_norm_backward_workspace(a);
  if (need > 0 && (a.workspace == nullptr || !at(a.workspace, 256) || a.workspace_bytes < need)) return M3_ERR_INVALID_ARG;
  return hip_status(m3::launch_residual_norm_backward(a, str(stream)));
}

}  // extern "C"
