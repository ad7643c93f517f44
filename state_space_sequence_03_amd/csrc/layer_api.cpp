// layer_api.cpp -- host side of the operators around the scan (ssd_layer.h):
// argument checks in the documented order, workspace sizes, launches.  Nothing
// is enqueued before every check has passed, and no exception leaves this file.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "../../include/ssd_layer.h"
#include "layer_host.hpp"

namespace ssd {
ssd_status report(ssd_status st, const char* msg);   // ssd_api.cpp: the thread's last error
}

namespace {

ssd_status fail(ssd_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
ssd_status fail(ssd_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return ssd::report(st, buf);
}
ssd_status ok() { return ssd::report(SSD_OK, ""); }
ssd_status launched(hipError_t e, const char* what) {
  return e == hipSuccess ? ok() : fail(SSD_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

template <typename F>
ssd_status guarded(F f) {
  try {
    return f();
  } catch (...) {
    return ssd::report(SSD_ERR_INTERNAL, "unexpected exception");
  }
}

// Whether the product of the sizes, in elements of 8 bytes, fits int64.
template <typename... I>
bool fits(I... sizes) {
  int64_t room = INT64_MAX / 8;
  for (int64_t s : {(int64_t)sizes...}) {
    if (s < 1) return false;
    room /= s;
  }
  return room > 0;
}

bool is_aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
template <typename... P>
bool aligned16(P... ps) {
  for (const void* p : {static_cast<const void*>(ps)...})
    if (!is_aligned(p, 16)) return false;
  return true;
}

// A strided operand's strides (contiguous ones for NULL).
void strides_of(const ssd_strides* s, int64_t L, int64_t width, int64_t out[2]) {
  out[0] = s ? s->batch : L * width;
  out[1] = s ? s->token : width;
}
ssd_status check_strides(const char* name, const int64_t s[2], int64_t batch, int64_t L,
                         int64_t width, bool output) {
  if (s[0] < 0 || s[1] < 0) return fail(SSD_ERR_BAD_VALUE, "%s: strides must not be negative", name);
  // the offset of the last element, in bytes, has to fit int64
  const __int128 last = (__int128)(batch - 1) * s[0] + (__int128)(L - 1) * s[1] + width;
  if (last > INT64_MAX / 8) return fail(SSD_ERR_BAD_SHAPE, "%s: strides overflow int64", name);
  if (output) {
    const bool rows = L == 1 || s[1] >= width;
    const bool outer = batch == 1 || (L == 1 ? s[0] >= width : s[0] >= (L - 1) * s[1] + width);
    const bool inner = batch == 1 || (s[0] >= width && (L == 1 || s[1] >= (batch - 1) * s[0] + width));
    if (!rows || !(outer || inner))
      return fail(SSD_ERR_BAD_VALUE, "%s: the rows of an output must not overlap", name);
  }
  return SSD_OK;
}
// Accesses of `per` elements of `size` bytes to every row of a strided operand.
bool row_vectors(const void* p, const int64_t s[2], int per, size_t size) {
  return is_aligned(p, per * size) && s[0] % per == 0 && s[1] % per == 0;
}
// Whether two buffers of `bytes` share memory (neither does where one is absent).
bool overlap(const void* a, const void* b, int64_t bytes) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
  return p && q && (p < q ? q - p : p - q) < (uintptr_t)bytes;
}

ssd_status check_io(int32_t io_dtype, int64_t reserved) {
  if (io_dtype != SSD_BF16 && io_dtype != SSD_F32)
    return fail(SSD_ERR_BAD_DTYPE, "io_dtype must be SSD_BF16 or SSD_F32 (got %d)", io_dtype);
  if (reserved != 0) return fail(SSD_ERR_BAD_DTYPE, "reserved field must be 0");
  return SSD_OK;
}
size_t element(int32_t io_dtype) { return io_dtype == SSD_BF16 ? 2 : 4; }

// ---- convolution ----

ssd_status conv_shape(const ssd_conv_problem& p) {
  if (p.batch <= 0 || p.seqlen <= 0 || p.channels <= 0 || p.width <= 0)
    return fail(SSD_ERR_BAD_SHAPE, "every size must be positive");
  if (p.nsplit < 1 || p.nsplit > 3) return fail(SSD_ERR_BAD_SHAPE, "nsplit must be 1, 2 or 3");
  int64_t left = p.channels;
  for (int64_t i = 0; i < p.nsplit; ++i) {
    if (p.split[i] <= 0 || p.split[i] > left)
      return fail(SSD_ERR_BAD_SHAPE, "the split must be positive and add up to channels");
    left -= p.split[i];
  }
  if (left != 0) return fail(SSD_ERR_BAD_SHAPE, "the split must add up to channels");
  if (!fits(p.batch, p.seqlen, p.channels) || !fits(p.batch, p.width, p.channels))
    return fail(SSD_ERR_BAD_SHAPE, "tensor size overflows int64");
  ssd_status st = check_io(p.io_dtype, p.reserved);
  if (st != SSD_OK) return st;
  if (p.activation != 0 && p.activation != 1)
    return fail(SSD_ERR_BAD_VALUE, "activation must be 0 or 1 (got %d)", p.activation);
  return SSD_OK;
}
ssd_status conv_supported(const ssd_conv_problem& p) {
  if (p.width < 2 || p.width > 4)
    return fail(SSD_ERR_UNSUPPORTED, "width must be 2, 3 or 4 (got %lld)", (long long)p.width);
  if (!ssd::conv_grid_ok(p.batch, p.seqlen, p.channels))
    return fail(SSD_ERR_UNSUPPORTED, "grid too large for this build");
  return SSD_OK;
}
void conv_args(const ssd_conv_problem& p, const int64_t xs[2], const void* x, const float* w,
               const float* bias, ssd::ConvArgs* a) {
  a->batch = p.batch;
  a->L = p.seqlen;
  a->C = p.channels;
  a->W = (int)p.width;
  a->bf16 = p.io_dtype == SSD_BF16;
  a->silu = p.activation;
  a->x = x;
  a->xs[0] = xs[0];
  a->xs[1] = xs[1];
  a->w = w;
  a->bias = bias;
  int64_t end = 0;
  for (int i = 0; i < 3; ++i) {
    if (i < p.nsplit) end += p.split[i];
    a->end[i] = end;
  }
}
// Accesses of four channels: x (and dx) by rows, outputs or gradients by their sizes.
constexpr int kConvVector = 4;
bool conv_vectors(const ssd_conv_problem& p) {
  for (int64_t i = 0; i < p.nsplit; ++i)
    if (p.split[i] % kConvVector != 0) return false;
  return true;
}

ssd_status conv_run(const ssd_conv_problem* prob, const void* x, const ssd_strides* xst,
                    const float* weight, const float* bias, const void* init, void* const* y,
                    void* fin, int in_place, void* stream) {
  const ssd_conv_problem& p = *prob;
  ssd_status st = conv_shape(p);
  if (st != SSD_OK) return st;
  for (int64_t i = 0; i < p.nsplit; ++i)
    if (!y[i]) return fail(SSD_ERR_NULL_POINTER, "y[%lld] must not be NULL", (long long)i);
  int64_t xs[2];
  strides_of(xst, p.seqlen, p.channels, xs);
  st = check_strides("x", xs, p.batch, p.seqlen, p.channels, false);
  if (st != SSD_OK) return st;
  if (!in_place && overlap(init, fin, p.batch * (p.width - 1) * p.channels * (int64_t)element(p.io_dtype)))
    return fail(SSD_ERR_BAD_VALUE, "final_state must not overlap init_state");
  if (!is_aligned(x, element(p.io_dtype)))
    return fail(SSD_ERR_MISALIGNED, "x must have the alignment of its element");
  bool fine = aligned16(weight, bias, init, fin);
  for (int64_t i = 0; i < p.nsplit; ++i) fine = fine && is_aligned(y[i], 16);
  if (!fine) return fail(SSD_ERR_MISALIGNED, "every other tensor pointer must be 16-byte aligned");
  st = conv_supported(p);
  if (st != SSD_OK) return st;
  ssd::ConvArgs a{};
  conv_args(p, xs, x, weight, bias, &a);
  a.init = init;
  a.fin = fin;
  a.one_run = in_place;
  for (int64_t i = 0; i < p.nsplit; ++i) a.y[i] = y[i];
  a.vec = conv_vectors(p) && row_vectors(x, xs, kConvVector, element(p.io_dtype));
  return launched(ssd::launch_conv_fwd(a, static_cast<hipStream_t>(stream)), "convolution launch");
}

// ---- selective scan ----

ssd_status scan_shape(const ssd_selscan_problem& p) {
  if (p.batch <= 0 || p.seqlen <= 0 || p.channels <= 0 || p.dstate <= 0 || p.ngroups <= 0)
    return fail(SSD_ERR_BAD_SHAPE, "every size must be positive");
  if (p.channels % p.ngroups != 0)
    return fail(SSD_ERR_BAD_SHAPE, "channels (%lld) must be a multiple of ngroups (%lld)",
                (long long)p.channels, (long long)p.ngroups);
  if (!fits(p.batch, p.seqlen, p.channels) || !fits(p.batch, p.seqlen, p.ngroups, p.dstate) ||
      !fits(p.batch, p.channels, p.dstate))
    return fail(SSD_ERR_BAD_SHAPE, "tensor size overflows int64");
  return check_io(p.io_dtype, p.reserved);
}
ssd_status scan_supported(const ssd_selscan_problem& p) {
  if (p.dstate > 64)
    return fail(SSD_ERR_UNSUPPORTED, "dstate must be at most 64 (got %lld)", (long long)p.dstate);
  if (p.channels > (1 << 24) || !ssd::selscan_grid_ok(p.batch, p.seqlen, p.channels, p.dstate, p.ngroups))
    return fail(SSD_ERR_UNSUPPORTED, "grid too large for this build");
  return SSD_OK;
}
// The kernels reach eight rows of z and dz by 32-bit byte offsets, and drop what they
// store past the last token by its place behind that row's end.  With one token the
// caller's stride says neither how far rows are apart nor that they are, so a row's
// width takes its place.
void one_token_rows(const ssd_selscan_problem& p, int64_t s[2]) {
  if (p.seqlen == 1) s[1] = p.channels;
}
ssd_status scan_rows(const ssd_selscan_problem& p, const ssd::ScanArgs& a) {
  const int64_t most = ((int64_t(1) << 28) - 1) / (int64_t)element(p.io_dtype);
  if ((a.z && a.zs[1] > most) || (a.dz && a.dzs[1] > most))
    return fail(SSD_ERR_UNSUPPORTED, "tokens of z and dz must be less than 2^28 bytes apart");
  return SSD_OK;
}
ssd_status scan_transform(const ssd_dt_transform* dtx, ssd::DtXform* xf) {
  if (!dtx) return SSD_OK;
  if (dtx->softplus != 0 && dtx->softplus != 1)
    return fail(SSD_ERR_BAD_VALUE, "dt transform: softplus must be 0 or 1 (got %d)", dtx->softplus);
  if (dtx->reserved != 0) return fail(SSD_ERR_BAD_VALUE, "dt transform: reserved field must be 0");
  if (!(dtx->dt_min <= dtx->dt_max))
    return fail(SSD_ERR_BAD_VALUE, "dt transform: dt_min and dt_max must be numbers, dt_min <= dt_max");
  xf->bias = dtx->dt_bias;
  xf->softplus = dtx->softplus;
  xf->lo = dtx->dt_min;
  xf->hi = dtx->dt_max;
  return SSD_OK;
}
// What the three entry points check alike after their NULL checks; fills the
// arguments that they share.
ssd_status scan_common(const ssd_selscan_problem& p, const ssd_dt_transform* dtx, const void* x,
                       const void* dt, const float* A, const void* B, const ssd_strides* bst,
                       const void* C, const ssd_strides* cst, const float* D, const void* z,
                       const ssd_strides* zst, ssd::DtXform* xf, ssd::ScanArgs* a) {
  ssd_status st = scan_shape(p);
  if (st != SSD_OK) return st;
  st = scan_transform(dtx, xf);
  if (st != SSD_OK) return st;
  a->batch = p.batch; a->L = p.seqlen; a->D = p.channels; a->N = p.dstate; a->G = p.ngroups;
  a->bf16 = p.io_dtype == SSD_BF16;
  a->xf = dtx ? xf : nullptr;
  a->x = x; a->dt = dt; a->A = A; a->B = B; a->C = C; a->Dv = D; a->z = z;
  strides_of(bst, p.seqlen, p.ngroups * p.dstate, a->bs);
  strides_of(cst, p.seqlen, p.ngroups * p.dstate, a->cs);
  strides_of(zst, p.seqlen, p.channels, a->zs);
  st = check_strides("B", a->bs, p.batch, p.seqlen, p.ngroups * p.dstate, false);
  if (st != SSD_OK) return st;
  st = check_strides("C", a->cs, p.batch, p.seqlen, p.ngroups * p.dstate, false);
  if (st != SSD_OK) return st;
  if (z) {
    st = check_strides("z", a->zs, p.batch, p.seqlen, p.channels, false);
    if (st != SSD_OK) return st;
    one_token_rows(p, a->zs);
  }
  return SSD_OK;
}
ssd_status scan_alignment(const ssd_selscan_problem& p, const ssd::ScanArgs& a,
                          const ssd_dt_transform* dtx) {
  const size_t e = element(p.io_dtype);
  if (!is_aligned(a.B, e) || !is_aligned(a.C, e) || !is_aligned(a.z, e) || !is_aligned(a.dz, e))
    return fail(SSD_ERR_MISALIGNED, "strided operands must have the alignment of their element");
  if (!aligned16(a.x, a.dt, a.A, a.Dv, a.init, a.y, a.fin, a.state, a.dy, a.dfin, a.dx, a.ddt, a.dA,
                 a.dB, a.dC, a.dD, a.dinit, a.dbias, a.workspace, dtx ? dtx->dt_bias : nullptr))
    return fail(SSD_ERR_MISALIGNED, "every other tensor pointer must be 16-byte aligned");
  return SSD_OK;
}

// ---- gated norm ----

ssd_status norm_shape(const ssd_gated_norm_problem& p) {
  if (p.batch <= 0 || p.seqlen <= 0 || p.channels <= 0 || p.ngroups <= 0)
    return fail(SSD_ERR_BAD_SHAPE, "every size must be positive");
  if (p.channels % p.ngroups != 0)
    return fail(SSD_ERR_BAD_SHAPE, "channels (%lld) must be a multiple of ngroups (%lld)",
                (long long)p.channels, (long long)p.ngroups);
  if (!fits(p.batch, p.seqlen, p.channels))
    return fail(SSD_ERR_BAD_SHAPE, "tensor size overflows int64");
  ssd_status st = check_io(p.io_dtype, p.reserved);
  if (st != SSD_OK) return st;
  if (!(p.eps >= 0.0f) || std::isinf(p.eps)) return fail(SSD_ERR_BAD_VALUE, "eps must be finite and >= 0");
  if (p.norm_before_gate != 0 && p.norm_before_gate != 1)
    return fail(SSD_ERR_BAD_VALUE, "norm_before_gate must be 0 or 1 (got %d)", p.norm_before_gate);
  return SSD_OK;
}
ssd_status norm_supported(const ssd_gated_norm_problem& p) {
  if (p.channels / p.ngroups > ssd::norm_group_limit())
    return fail(SSD_ERR_UNSUPPORTED, "at most %lld channels per group (got %lld)",
                (long long)ssd::norm_group_limit(), (long long)(p.channels / p.ngroups));
  if (!ssd::norm_grid_ok(p.batch, p.seqlen, p.channels, p.ngroups))
    return fail(SSD_ERR_UNSUPPORTED, "grid too large for this build");
  return SSD_OK;
}
void norm_args(const ssd_gated_norm_problem& p, const void* x, const void* z, const float* w,
               ssd::NormArgs* a) {
  a->batch = p.batch;
  a->L = p.seqlen;
  a->D = p.channels;
  a->G = p.ngroups;
  a->eps = p.eps;
  a->before = p.norm_before_gate;
  a->bf16 = p.io_dtype == SSD_BF16;
  a->x = x;
  a->z = z;
  a->w = w;
}

}  // namespace

extern "C" {

int ssd_layer_abi_version(void) { return SSD_LAYER_ABI_VERSION; }

ssd_status ssd_conv_fwd(const ssd_conv_problem* prob, const void* x, const ssd_strides* x_strides,
                        const float* weight, const float* bias, const void* init_state,
                        void* const* y, void* final_state, void* stream) {
  return guarded([&] {
    if (!prob || !x || !weight || !y)
      return fail(SSD_ERR_NULL_POINTER, "prob, x, weight and y must not be NULL");
    return conv_run(prob, x, x_strides, weight, bias, init_state, y, final_state, 0, stream);
  });
}

ssd_status ssd_conv_step(const ssd_conv_problem* prob, void* state, const void* x,
                         const ssd_strides* x_strides, const float* weight, const float* bias,
                         void* const* y, void* stream) {
  return guarded([&] {
    if (!prob || !state || !x || !weight || !y)
      return fail(SSD_ERR_NULL_POINTER, "prob, state, x, weight and y must not be NULL");
    return conv_run(prob, x, x_strides, weight, bias, state, y, state, 1, stream);
  });
}

ssd_status ssd_conv_bwd_workspace_size(const ssd_conv_problem* prob, size_t* bytes) {
  return guarded([&] {
    if (!prob || !bytes) return fail(SSD_ERR_NULL_POINTER, "prob and bytes must not be NULL");
    ssd_status st = conv_shape(*prob);
    if (st == SSD_OK) st = conv_supported(*prob);
    if (st != SSD_OK) return st;
    *bytes = ssd::conv_bwd_workspace(prob->batch, prob->seqlen, prob->channels, (int)prob->width);
    return ok();
  });
}

ssd_status ssd_conv_bwd(const ssd_conv_problem* prob, const void* x, const ssd_strides* x_strides,
                        const float* weight, const float* bias, const void* init_state,
                        const void* const* dy, const void* dfinal, void* dx,
                        const ssd_strides* dx_strides, float* dweight, float* dbias, void* dinit,
                        void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&] {
    if (!prob || !x || !weight || !dy || !dx || !dweight || !workspace)
      return fail(SSD_ERR_NULL_POINTER,
                  "prob, x, weight, dy, dx, dweight and workspace must not be NULL");
    const ssd_conv_problem& p = *prob;
    ssd_status st = conv_shape(p);
    if (st != SSD_OK) return st;
    for (int64_t i = 0; i < p.nsplit; ++i)
      if (!dy[i]) return fail(SSD_ERR_NULL_POINTER, "dy[%lld] must not be NULL", (long long)i);
    int64_t xs[2], dxs[2];
    strides_of(x_strides, p.seqlen, p.channels, xs);
    strides_of(dx_strides, p.seqlen, p.channels, dxs);
    st = check_strides("x", xs, p.batch, p.seqlen, p.channels, false);
    if (st != SSD_OK) return st;
    st = check_strides("dx", dxs, p.batch, p.seqlen, p.channels, true);
    if (st != SSD_OK) return st;
    const size_t e = element(p.io_dtype);
    if (!is_aligned(x, e) || !is_aligned(dx, e))
      return fail(SSD_ERR_MISALIGNED, "x and dx must have the alignment of their element");
    bool fine = aligned16(weight, bias, init_state, dfinal, dweight, dbias, dinit, workspace);
    for (int64_t i = 0; i < p.nsplit; ++i) fine = fine && is_aligned(dy[i], 16);
    if (!fine) return fail(SSD_ERR_MISALIGNED, "every other tensor pointer must be 16-byte aligned");
    st = conv_supported(p);
    if (st != SSD_OK) return st;
    ssd::ConvArgs a{};
    conv_args(p, xs, x, weight, bias, &a);
    const size_t need = ssd::conv_bwd_workspace(p.batch, p.seqlen, p.channels, a.W);
    if (workspace_bytes < need)
      return fail(SSD_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
    a.init = init_state;
    for (int64_t i = 0; i < p.nsplit; ++i) a.y[i] = const_cast<void*>(dy[i]);
    a.dfin = dfinal;
    a.dx = dx;
    a.dxs[0] = dxs[0];
    a.dxs[1] = dxs[1];
    a.dw = dweight;
    a.db = dbias;
    a.dinit = dinit;
    a.workspace = workspace;
    a.vec = conv_vectors(p) && row_vectors(x, xs, kConvVector, e) && row_vectors(dx, dxs, kConvVector, e);
    return launched(ssd::launch_conv_bwd(a, static_cast<hipStream_t>(stream)),
                    "convolution backward launch");
  });
}

ssd_status ssd_selscan_fwd_workspace_size(const ssd_selscan_problem* prob, size_t* bytes) {
  return guarded([&] {
    if (!prob || !bytes) return fail(SSD_ERR_NULL_POINTER, "prob and bytes must not be NULL");
    ssd_status st = scan_shape(*prob);
    if (st == SSD_OK) st = scan_supported(*prob);
    if (st != SSD_OK) return st;
    *bytes = ssd::selscan_fwd_workspace(prob->batch, prob->seqlen, prob->channels, prob->dstate,
                                        prob->ngroups);
    return ok();
  });
}

ssd_status ssd_selscan_fwd(const ssd_selscan_problem* prob, const ssd_dt_transform* dtx,
                           const void* x, const void* dt, const float* A, const void* B,
                           const ssd_strides* b_strides, const void* C,
                           const ssd_strides* c_strides, const float* D, const void* z,
                           const ssd_strides* z_strides, const float* init_state, void* y,
                           float* final_state, void* workspace, size_t workspace_bytes,
                           void* stream) {
  return guarded([&] {
    if (!prob || !x || !dt || !A || !B || !C || !y)
      return fail(SSD_ERR_NULL_POINTER, "prob, x, dt, A, B, C and y must not be NULL");
    ssd::ScanArgs a{};
    ssd::DtXform xf{};
    ssd_status st = scan_common(*prob, dtx, x, dt, A, B, b_strides, C, c_strides, D, z, z_strides, &xf, &a);
    if (st != SSD_OK) return st;
    if (overlap(init_state, final_state, a.batch * a.D * a.N * (int64_t)sizeof(float)))
      return fail(SSD_ERR_BAD_VALUE, "final_state must not overlap init_state");
    a.init = init_state;
    a.y = y;
    a.fin = final_state;
    a.workspace = workspace;
    st = scan_alignment(*prob, a, dtx);
    if (st != SSD_OK) return st;
    st = scan_supported(*prob);
    if (st == SSD_OK) st = scan_rows(*prob, a);
    if (st != SSD_OK) return st;
    const size_t need = ssd::selscan_fwd_workspace(a.batch, a.L, a.D, a.N, a.G);
    if (need > 0 && (!workspace || workspace_bytes < need))
      return fail(SSD_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu",
                  workspace ? workspace_bytes : size_t(0), need);
    return launched(ssd::launch_selscan_fwd(a, static_cast<hipStream_t>(stream)), "selective scan launch");
  });
}

ssd_status ssd_selscan_step(const ssd_selscan_problem* prob, const ssd_dt_transform* dtx,
                            float* state, const void* x, const void* dt, const float* A,
                            const void* B, const ssd_strides* b_strides, const void* C,
                            const ssd_strides* c_strides, const float* D, const void* z,
                            const ssd_strides* z_strides, void* y, void* stream) {
  return guarded([&] {
    if (!prob || !state || !x || !dt || !A || !B || !C || !y)
      return fail(SSD_ERR_NULL_POINTER, "prob, state, x, dt, A, B, C and y must not be NULL");
    ssd::ScanArgs a{};
    ssd::DtXform xf{};
    ssd_status st = scan_common(*prob, dtx, x, dt, A, B, b_strides, C, c_strides, D, z, z_strides, &xf, &a);
    if (st != SSD_OK) return st;
    a.state = state;
    a.y = y;
    st = scan_alignment(*prob, a, dtx);
    if (st != SSD_OK) return st;
    st = scan_supported(*prob);
    if (st != SSD_OK) return st;
    const size_t four = 4 * element(prob->io_dtype);
    a.vec = a.N % 4 == 0 && is_aligned(B, four) && is_aligned(C, four) && a.bs[0] % 4 == 0 &&
            a.bs[1] % 4 == 0 && a.cs[0] % 4 == 0 && a.cs[1] % 4 == 0;
    return launched(ssd::launch_selscan_step(a, static_cast<hipStream_t>(stream)),
                    "selective scan step launch");
  });
}

ssd_status ssd_selscan_bwd_workspace_size(const ssd_selscan_problem* prob, size_t* bytes) {
  return guarded([&] {
    if (!prob || !bytes) return fail(SSD_ERR_NULL_POINTER, "prob and bytes must not be NULL");
    ssd_status st = scan_shape(*prob);
    if (st == SSD_OK) st = scan_supported(*prob);
    if (st != SSD_OK) return st;
    *bytes = ssd::selscan_bwd_workspace(prob->batch, prob->seqlen, prob->channels, prob->dstate,
                                        prob->ngroups);
    return ok();
  });
}

ssd_status ssd_selscan_bwd(const ssd_selscan_problem* prob, const ssd_dt_transform* dtx,
                           const void* x, const void* dt, const float* A, const void* B,
                           const ssd_strides* b_strides, const void* C,
                           const ssd_strides* c_strides, const float* D, const void* z,
                           const ssd_strides* z_strides, const float* init_state, const void* dy,
                           const float* dfinal, void* dx, void* ddt, float* dA, void* dB, void* dC,
                           float* dD, void* dz, const ssd_strides* dz_strides, float* dinit,
                           float* ddt_bias, void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&] {
    if (!prob || !x || !dt || !A || !B || !C || !dy || !dx || !ddt || !dA || !dB || !dC ||
        !workspace || (z && !dz))
      return fail(SSD_ERR_NULL_POINTER,
                  "prob, x, dt, A, B, C, dy, dx, ddt, dA, dB, dC, workspace and, with z, dz must not be NULL");
    ssd::ScanArgs a{};
    ssd::DtXform xf{};
    ssd_status st = scan_common(*prob, dtx, x, dt, A, B, b_strides, C, c_strides, D, z, z_strides, &xf, &a);
    if (st != SSD_OK) return st;
    strides_of(dz_strides, a.L, a.D, a.dzs);
    if (z) {
      st = check_strides("dz", a.dzs, a.batch, a.L, a.D, true);
      if (st != SSD_OK) return st;
      one_token_rows(*prob, a.dzs);
    }
    a.init = init_state;
    a.dy = dy;
    a.dfin = dfinal;
    a.dx = dx;
    a.ddt = ddt;
    a.dA = dA;
    a.dB = dB;
    a.dC = dC;
    a.dD = dD;
    a.dz = z ? dz : nullptr;
    a.dinit = dinit;
    a.dbias = ddt_bias;
    a.workspace = workspace;
    st = scan_alignment(*prob, a, dtx);
    if (st != SSD_OK) return st;
    st = scan_supported(*prob);
    if (st == SSD_OK) st = scan_rows(*prob, a);
    if (st != SSD_OK) return st;
    const size_t need = ssd::selscan_bwd_workspace(a.batch, a.L, a.D, a.N, a.G);
    if (workspace_bytes < need)
      return fail(SSD_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
    return launched(ssd::launch_selscan_bwd(a, static_cast<hipStream_t>(stream)),
                    "selective scan backward launch");
  });
}

ssd_status ssd_gated_norm_fwd(const ssd_gated_norm_problem* prob, const void* x, const void* z,
                              const ssd_strides* z_strides, const float* weight, void* y,
                              void* stream) {
  return guarded([&] {
    if (!prob || !x || !weight || !y)
      return fail(SSD_ERR_NULL_POINTER, "prob, x, weight and y must not be NULL");
    const ssd_gated_norm_problem& p = *prob;
    ssd_status st = norm_shape(p);
    if (st != SSD_OK) return st;
    ssd::NormArgs a{};
    norm_args(p, x, z, weight, &a);
    strides_of(z_strides, a.L, a.D, a.zs);
    if (z) {
      st = check_strides("z", a.zs, a.batch, a.L, a.D, false);
      if (st != SSD_OK) return st;
    }
    if (!is_aligned(z, element(p.io_dtype)))
      return fail(SSD_ERR_MISALIGNED, "z must have the alignment of its element");
    if (!aligned16(x, weight, y))
      return fail(SSD_ERR_MISALIGNED, "every other tensor pointer must be 16-byte aligned");
    st = norm_supported(p);
    if (st != SSD_OK) return st;
    a.y = y;
    const int per = a.bf16 ? 8 : 4;
    a.vec = (a.D / a.G) % per == 0 && (!z || row_vectors(z, a.zs, per, element(p.io_dtype)));
    return launched(ssd::launch_norm_fwd(a, static_cast<hipStream_t>(stream)), "gated norm launch");
  });
}

ssd_status ssd_gated_norm_bwd_workspace_size(const ssd_gated_norm_problem* prob, size_t* bytes) {
  return guarded([&] {
    if (!prob || !bytes) return fail(SSD_ERR_NULL_POINTER, "prob and bytes must not be NULL");
    ssd_status st = norm_shape(*prob);
    if (st == SSD_OK) st = norm_supported(*prob);
    if (st != SSD_OK) return st;
    *bytes = ssd::norm_bwd_workspace(prob->batch, prob->seqlen, prob->channels, prob->ngroups,
                                     prob->io_dtype == SSD_BF16);
    return ok();
  });
}

ssd_status ssd_gated_norm_bwd(const ssd_gated_norm_problem* prob, const void* x, const void* z,
                              const ssd_strides* z_strides, const float* weight, const void* dy,
                              void* dx, void* dz, const ssd_strides* dz_strides, float* dweight,
                              void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&] {
    if (!prob || !x || !weight || !dy || !dx || !dweight || !workspace || (z && !dz))
      return fail(SSD_ERR_NULL_POINTER,
                  "prob, x, weight, dy, dx, dweight, workspace and, with z, dz must not be NULL");
    const ssd_gated_norm_problem& p = *prob;
    ssd_status st = norm_shape(p);
    if (st != SSD_OK) return st;
    ssd::NormArgs a{};
    norm_args(p, x, z, weight, &a);
    strides_of(z_strides, a.L, a.D, a.zs);
    strides_of(dz_strides, a.L, a.D, a.dzs);
    if (z) {
      st = check_strides("z", a.zs, a.batch, a.L, a.D, false);
      if (st != SSD_OK) return st;
      st = check_strides("dz", a.dzs, a.batch, a.L, a.D, true);
      if (st != SSD_OK) return st;
      if (!is_aligned(z, element(p.io_dtype)) || !is_aligned(dz, element(p.io_dtype)))
        return fail(SSD_ERR_MISALIGNED, "z and dz must have the alignment of their element");
    }
    if (!aligned16(x, weight, dy, dx, dweight, workspace))
      return fail(SSD_ERR_MISALIGNED, "every other tensor pointer must be 16-byte aligned");
    st = norm_supported(p);
    if (st != SSD_OK) return st;
    const size_t need = ssd::norm_bwd_workspace(a.batch, a.L, a.D, a.G, a.bf16);
    if (workspace_bytes < need)
      return fail(SSD_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
    a.dy = dy;
    a.dx = dx;
    a.dz = z ? dz : nullptr;
    a.dw = dweight;
    a.workspace = workspace;
    const int per = a.bf16 ? 8 : 4;
    a.vec = (a.D / a.G) % per == 0 && (!z || (row_vectors(z, a.zs, per, element(p.io_dtype)) &&
                                         row_vectors(dz, a.dzs, per, element(p.io_dtype))));
    return launched(ssd::launch_norm_bwd(a, static_cast<hipStream_t>(stream)), "gated norm backward launch");
  });
}

}  // extern "C"
