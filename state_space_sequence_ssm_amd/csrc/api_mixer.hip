// C ABI of linear attention and of the norm and rotation of its queries and keys:
// host-side validation and dispatch.  Every check runs on the host before any HIP call.
#include <initializer_list>

#include "mixer_internal.hpp"

namespace {

constexpr double kMaxElems = 34359738368.0;  // 2^35 elements of one tensor
constexpr double kMaxInt = 2147483647.0;
constexpr int kMaxLength = 1 << 28;
constexpr int kMaxRow = 1 << 24;     // elements from one token to the next: 64 of them are addressed in 32 bits
constexpr int kMaxHeadDim = 256;   // K and V: what a block's state and tiles hold
constexpr int kMaxRopeDim = 1024;  // D of the rotated heads: what a wave's angles hold

bool ok_dtype(int t) { return t == M3_F32 || t == M3_BF16; }
size_t elem(int t) { return t == M3_BF16 ? 2 : 4; }
bool flag(int v) { return v == 0 || v == 1; }
bool all_at(std::initializer_list<const void*> ps, size_t a) {
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) % a != 0) return false;
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
// Distance between rows of `width` elements: 0 = dense.  Tokens' rows are addressed 64 at a
// time in 32 bits; the rows of single tokens lie as far apart as a batch of long sequences.
bool set_ld(int64_t& ld, int64_t width, int bits) {
  if (ld == 0) ld = width;
  return ld >= width && ld < (int64_t(1) << bits);
}
int hip_status(hipError_t e) { return e == hipSuccess ? M3_OK : M3_ERR_HIP; }
hipStream_t str(void* s) { return static_cast<hipStream_t>(s); }
bool workspace_ok(const void* p, size_t have, size_t need) {
  return need == 0 || (p != nullptr && reinterpret_cast<uintptr_t>(p) % 256 == 0 && have >= need);
}

int check_attention_shape(int64_t Bt, int64_t L, int64_t H, int64_t Hk, int64_t K, int64_t V, int dtype) {
  if (Bt < 1 || L < 1 || H < 1 || Hk < 1 || K < 1 || V < 1 || H % Hk != 0) return M3_ERR_INVALID_ARG;
  if (!ok_dtype(dtype) || K > kMaxHeadDim || V > kMaxHeadDim || L > kMaxLength) return M3_ERR_UNSUPPORTED;
  const double wide = double(H) * (K > V ? K : V);
  if (double(Bt) * wide > kMaxInt || double(Bt) * L * wide > kMaxElems || double(Bt) * H * K * V > kMaxElems) return M3_ERR_UNSUPPORTED;
  return M3_OK;
}
int check_attention_inputs(m3_linear_attention_args& f) {
  const int rc = check_attention_shape(f.Bt, f.L, f.H, f.Hk, f.K, f.V, f.in_dtype);
  if (rc != M3_OK) return rc;
  if (!all_set({f.q, f.k, f.v, f.log_decay})) return M3_ERR_INVALID_ARG;
  if (!set_ld(f.q_ld, int64_t(f.H) * f.K, 24) || !set_ld(f.k_ld, int64_t(f.Hk) * f.K, 24) || !set_ld(f.v_ld, int64_t(f.Hk) * f.V, 24))
    return M3_ERR_INVALID_ARG;
  return all_at({f.q, f.k, f.v}, elem(f.in_dtype)) && all_at({f.log_decay, f.h0, f.lengths}, 4) ? M3_OK : M3_ERR_INVALID_ARG;
}
bool ok_attention_size(const m3_linear_attention_args* a) {
  return a != nullptr && check_attention_shape(a->Bt, a->L, a->H, a->Hk, a->K, a->V, a->in_dtype) == M3_OK;
}

int check_rope_shape(const m3_qk_norm_rope_args& f) {
  if (f.Bt < 1 || f.L < 1 || f.H < 1 || f.Hk < 0 || f.D < 1 || f.R < 0 || f.R % 2 != 0 || f.R > f.D) return M3_ERR_INVALID_ARG;
  if (!flag(f.norm) || !flag(f.adjacent)) return M3_ERR_INVALID_ARG;
  if (!ok_dtype(f.in_dtype) || f.D > kMaxRopeDim || f.L > kMaxLength) return M3_ERR_UNSUPPORTED;
  const double wide = (double(f.H) + f.Hk) * f.D;
  if (wide > kMaxInt || double(f.Bt) * f.L > kMaxInt || double(f.Bt) * f.L * wide > kMaxElems) return M3_ERR_UNSUPPORTED;
  return M3_OK;
}
int check_rope(m3_qk_norm_rope_args& f) {
  const int rc = check_rope_shape(f);
  if (rc != M3_OK) return rc;
  if (!(f.eps >= 0.f && f.eps <= 3.0e38f)) return M3_ERR_INVALID_ARG;
  if (f.q == nullptr || (f.k == nullptr) != (f.Hk == 0) || (f.k == nullptr && f.k_w != nullptr)) return M3_ERR_INVALID_ARG;
  if ((f.freqs == nullptr) != (f.R == 0) || (!f.norm && (f.q_w != nullptr || f.k_w != nullptr))) return M3_ERR_INVALID_ARG;
  const int bits = f.L == 1 ? 40 : 24;  // single tokens
  if (!set_ld(f.q_ld, int64_t(f.H) * f.D, bits)) return M3_ERR_INVALID_ARG;
  if (f.k != nullptr && !set_ld(f.k_ld, int64_t(f.Hk) * f.D, bits)) return M3_ERR_INVALID_ARG;
  return all_at({f.q, f.k}, elem(f.in_dtype)) && all_at({f.q_w, f.k_w, f.freqs, f.positions, f.lengths}, 4) ? M3_OK : M3_ERR_INVALID_ARG;
}

}  // namespace

extern "C" {

size_t m3_linear_attention_workspace_size(const m3_linear_attention_args* a) {
  return ok_attention_size(a) && m3::attention_fits(*a) ? m3::attention_workspace(*a) : 0;
}

int m3_linear_attention(const m3_linear_attention_args* args, void* stream) {
  if (args == nullptr) return M3_ERR_INVALID_ARG;
  m3_linear_attention_args a = *args;
  const int rc = check_attention_inputs(a);
  if (rc != M3_OK) return rc;
  if (!m3::attention_fits(a) || int64_t(a.H) * a.V >= kMaxRow) return M3_ERR_UNSUPPORTED;
  if (a.y == nullptr || !all_at({a.y}, elem(a.in_dtype)) || !all_at({a.h_final}, 4)) return M3_ERR_INVALID_ARG;
  if (clash({a.y, a.h_final, a.workspace}, {a.q, a.k, a.v, a.log_decay, a.lengths}) || a.y == a.h0 ||
      (a.workspace != nullptr && a.workspace == a.h0))
    return M3_ERR_INVALID_ARG;
  if (!all_at({a.workspace}, 256) || (a.workspace != nullptr && a.workspace_bytes < m3::attention_workspace(a))) return M3_ERR_INVALID_ARG;
  return hip_status(m3::launch_attention(a, str(stream)));
}

int m3_linear_attention_step(const m3_linear_attention_step_args* args, void* stream) {
  if (args == nullptr) return M3_ERR_INVALID_ARG;
  m3_linear_attention_step_args a = *args;
  const int rc = check_attention_shape(a.Bt, 1, a.H, a.Hk, a.K, a.V, a.in_dtype);
  if (rc != M3_OK) return rc;
  if (!all_set({a.q, a.k, a.v, a.log_decay, a.h, a.y})) return M3_ERR_INVALID_ARG;
  if (!set_ld(a.q_ld, int64_t(a.H) * a.K, 40) || !set_ld(a.k_ld, int64_t(a.Hk) * a.K, 40) || !set_ld(a.v_ld, int64_t(a.Hk) * a.V, 40))
    return M3_ERR_INVALID_ARG;
  if (a.h_out == nullptr) a.h_out = a.h;
  if (!all_at({a.q, a.k, a.v, a.y}, elem(a.in_dtype)) || !all_at({a.log_decay, a.h, a.h_out}, 4)) return M3_ERR_INVALID_ARG;
  if (clash({a.y, a.h_out}, {a.q, a.k, a.v, a.log_decay}) || a.y == a.h) return M3_ERR_INVALID_ARG;
  if (!m3::attention_step_fits(a)) return M3_ERR_UNSUPPORTED;
  return hip_status(m3::launch_attention_step(a, str(stream)));
}

size_t m3_linear_attention_backward_workspace_size(const m3_linear_attention_backward_args* a) {
  return a != nullptr && ok_attention_size(&a->fwd) && m3::attention_backward_fits(*a) ? m3::attention_backward_workspace(*a) : 0;
}

int m3_linear_attention_backward(const m3_linear_attention_backward_args* args, void* stream) {
  if (args == nullptr) return M3_ERR_INVALID_ARG;
  m3_linear_attention_backward_args a = *args;
  const int rc = check_attention_inputs(a.fwd);
  if (rc != M3_OK) return rc;
  if (!m3::attention_backward_fits(a) || int64_t(a.fwd.H) * a.fwd.V >= kMaxRow) return M3_ERR_UNSUPPORTED;
  const m3_linear_attention_args& f = a.fwd;
  if (!all_set({a.dy, a.dq, a.dk, a.dv})) return M3_ERR_INVALID_ARG;
  if (!all_at({a.dy, a.dq, a.dk, a.dv}, elem(f.in_dtype)) || !all_at({a.dh_final, a.dh0}, 4)) return M3_ERR_INVALID_ARG;
  const size_t need = m3::attention_backward_workspace(a);
  if (!workspace_ok(a.workspace, a.workspace_bytes, need)) return M3_ERR_INVALID_ARG;
  if (clash({a.dq, a.dk, a.dv, a.dh0, need == 0 ? nullptr : a.workspace},
            {f.q, f.k, f.v, f.log_decay, f.h0, f.lengths, a.dy, a.dh_final}))
    return M3_ERR_INVALID_ARG;
  return hip_status(m3::launch_attention_backward(a, str(stream)));
}

int m3_qk_norm_rope(const m3_qk_norm_rope_args* args, void* stream) {
  if (args == nullptr) return M3_ERR_INVALID_ARG;
  m3_qk_norm_rope_args a = *args;
  const int rc = check_rope(a);
  if (rc != M3_OK) return rc;
  if (a.q_out == nullptr || (a.k == nullptr) != (a.k_out == nullptr) || !all_at({a.q_out, a.k_out}, elem(a.in_dtype)))
    return M3_ERR_INVALID_ARG;
  // in place only over rows that lie as the output's do
  if ((a.q_out == a.q && a.q_ld != int64_t(a.H) * a.D) || (a.k != nullptr && a.k_out == a.k && a.k_ld != int64_t(a.Hk) * a.D))
    return M3_ERR_INVALID_ARG;
  if (clash({a.q_out, a.k_out}, {a.q_w, a.k_w, a.freqs, a.positions, a.lengths}) || a.q_out == a.k ||
      (a.k_out != nullptr && a.k_out == a.q))
    return M3_ERR_INVALID_ARG;
  return hip_status(m3::launch_rope(a, str(stream)));
}

size_t m3_qk_norm_rope_backward_workspace_size(const m3_qk_norm_rope_backward_args* a) {
  return a != nullptr && check_rope_shape(a->fwd) == M3_OK ? m3::rope_backward_workspace(*a) : 0;
}

int m3_qk_norm_rope_backward(const m3_qk_norm_rope_backward_args* args, void* stream) {
  if (args == nullptr) return M3_ERR_INVALID_ARG;
  m3_qk_norm_rope_backward_args a = *args;
  const int rc = check_rope(a.fwd);
  if (rc != M3_OK) return rc;
  const m3_qk_norm_rope_args& f = a.fwd;
  if (!all_set({a.dq_out, a.dq}) || (f.k == nullptr) != (a.dk_out == nullptr) || (f.k == nullptr) != (a.dk == nullptr))
    return M3_ERR_INVALID_ARG;
  if ((f.q_w == nullptr) != (a.dq_w == nullptr) || (f.k_w == nullptr) != (a.dk_w == nullptr)) return M3_ERR_INVALID_ARG;
  if (!all_at({a.dq_out, a.dk_out, a.dq, a.dk}, elem(f.in_dtype)) || !all_at({a.dq_w, a.dk_w}, 4)) return M3_ERR_INVALID_ARG;
  const size_t need = m3::rope_backward_workspace(a);
  if (!workspace_ok(a.workspace, a.workspace_bytes, need)) return M3_ERR_INVALID_ARG;
  if (clash({a.dq, a.dk, a.dq_w, a.dk_w, need == 0 ? nullptr : a.workspace}, {f.q, f.k, f.q_w, f.k_w, f.freqs, f.positions, f.lengths}) ||
      a.dq == a.dk_out || (a.dk != nullptr && a.dk == a.dq_out))
    return M3_ERR_INVALID_ARG;
  for (const void* d : {a.dq_out, a.dk_out})
    if (d != nullptr && (d == a.dq_w || d == a.dk_w || (need > 0 && d == a.workspace))) return M3_ERR_INVALID_ARG;
  return hip_status(m3::launch_rope_backward(a, str(stream)));
}

}  // extern "C"
