// block_api.cpp -- host side of the operators of a residual block and of its training step
// (ssd_block.h): argument checks in the documented order, workspace sizes, launches.
#include <algorithm>
#include <vector>

#include "block_host.hpp"
#include "layer_checks.hpp"

namespace {

using namespace ssd;

constexpr int64_t kMostRows = INT32_MAX;

// A strided operand whose batches follow each other like its tokens is one long batch.
void join_batches(int64_t* batch, int64_t* L, int64_t s[2]) {
  if (*batch > 1 && *L > 1 && s[0] == *L * s[1]) {
    *L *= *batch;
    *batch = 1;
  } else if (*L == 1 && *batch > 1) {
    *L = *batch;
    *batch = 1;
    s[1] = s[0];
  }
}

// ---- residual and norm ----

ssd_status add_norm_shape(const ssd_add_norm_problem& p) {
  if (p.batch <= 0 || p.seqlen <= 0 || p.channels <= 0)
    return fail(SSD_ERR_BAD_SHAPE, "every size must be positive");
  if (!fits(p.batch, p.seqlen, p.channels)) return fail(SSD_ERR_BAD_SHAPE, "tensor size overflows int64");
  ssd_status st = check_io(p.io_dtype, p.reserved);
  if (st != SSD_OK) return st;
  if (p.residual_dtype != SSD_F32 && !(p.residual_dtype == SSD_BF16 && p.io_dtype == SSD_BF16))
    return fail(SSD_ERR_BAD_DTYPE, "residual_dtype must be SSD_F32, or SSD_BF16 with io_dtype SSD_BF16 (got %d)",
                p.residual_dtype);
  if (!(p.eps >= 0.0f) || std::isinf(p.eps)) return fail(SSD_ERR_BAD_VALUE, "eps must be finite and >= 0");
  return SSD_OK;
}
// `launch`: of the forward pass, whose workgroups grow with the tokens (those of the gradients do not).
ssd_status add_norm_supported(const ssd_add_norm_problem& p, bool launch) {
  if (p.channels > block_norm_limit())
    return fail(SSD_ERR_UNSUPPORTED, "at most %lld channels (got %lld)", (long long)block_norm_limit(),
                (long long)p.channels);
  if (p.batch > kMostRows / p.seqlen) return fail(SSD_ERR_UNSUPPORTED, "at most 2^31 - 1 tokens");
  if (launch && !block_norm_grid_ok(p.batch, p.seqlen, p.channels, 1, 0))
    return fail(SSD_ERR_UNSUPPORTED, "grid too large for this build");
  return SSD_OK;
}

// ---- quantising ----

ssd_status quant_shape(const ssd_quant8_problem& p) {
  if (p.batch <= 0 || p.seqlen <= 0 || p.channels <= 0)
    return fail(SSD_ERR_BAD_SHAPE, "every size must be positive");
  // whole blocks of 128 x 128 have to fit too
  if (p.batch > INT64_MAX / 1024 || p.seqlen > INT64_MAX / 1024 || p.channels > INT64_MAX / 1024 ||
      !fits(p.batch, p.seqlen, p.channels + 127) || !fits(p.batch + 127, p.seqlen + 127, p.channels))
    return fail(SSD_ERR_BAD_SHAPE, "tensor size overflows int64");
  ssd_status st = check_io(p.io_dtype, p.reserved);
  if (st != SSD_OK) return st;
  if (p.tile != 0 && p.tile != 1) return fail(SSD_ERR_BAD_VALUE, "tile must be 0 or 1 (got %d)", p.tile);
  return SSD_OK;
}

// ---- matrix product ----

ssd_status matmul_shape(const ssd_matmul8_problem& p) {
  if (p.rows <= 0 || p.cols <= 0 || p.depth <= 0) return fail(SSD_ERR_BAD_SHAPE, "every size must be positive");
  if (p.depth % 128 != 0)
    return fail(SSD_ERR_BAD_SHAPE, "depth must be a multiple of 128 (got %lld)", (long long)p.depth);
  if (!fits(p.rows, p.cols) || !fits(p.rows, p.depth) || !fits(p.cols, p.depth))
    return fail(SSD_ERR_BAD_SHAPE, "tensor size overflows int64");
  ssd_status st = check_io(p.out_dtype, p.reserved);
  if (st != SSD_OK) return st;
  if (p.w_tile != 0 && p.w_tile != 1) return fail(SSD_ERR_BAD_VALUE, "w_tile must be 0 or 1 (got %d)", p.w_tile);
  return SSD_OK;
}
ssd_status matmul_supported(const ssd_matmul8_problem& p) {
  // 256 rows of a tile are reached by 32-bit offsets
  if (p.rows > kMostRows || p.cols > kMostRows || p.depth > (1 << 23))
    return fail(SSD_ERR_UNSUPPORTED, "at most 2^31 - 1 rows and columns, and a depth of 2^23");
  if (!matmul8_grid_ok(p.rows, p.cols, p.depth, p.out_dtype == SSD_BF16))
    return fail(SSD_ERR_UNSUPPORTED, "grid too large for this build");
  return SSD_OK;
}

// ---- clipping ----

struct Span {
  uintptr_t begin, end;
  bool written;
};

ssd_status clip_list(const ssd_grad* grads, int64_t n) {
  if (n <= 0) return fail(SSD_ERR_BAD_SHAPE, "there must be at least one tensor");
  if (n > (1 << 20)) return fail(SSD_ERR_UNSUPPORTED, "at most 2^20 tensors");
  int64_t total = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (grads[i].elements < 0) return fail(SSD_ERR_BAD_SHAPE, "grads[%lld]: negative size", (long long)i);
    if (grads[i].elements > (int64_t(1) << 40)) return fail(SSD_ERR_UNSUPPORTED, "at most 2^40 elements");
    total += grads[i].elements;
  }
  if (total > (int64_t(1) << 40)) return fail(SSD_ERR_UNSUPPORTED, "at most 2^40 elements");
  return SSD_OK;
}

ssd_status clip_overlaps(const ssd_grad* grads, int64_t n, const float* norm) {
  std::vector<Span> spans;
  spans.reserve(2 * n + 1);
  const uintptr_t at = reinterpret_cast<uintptr_t>(norm);
  spans.push_back({at, at + sizeof(float), true});
  for (int64_t i = 0; i < n; ++i) {
    const ssd_grad& g = grads[i];
    if (g.elements == 0) continue;
    const uintptr_t in = reinterpret_cast<uintptr_t>(g.grad), out = reinterpret_cast<uintptr_t>(g.out);
    if (in != out || g.dtype != g.out_dtype) spans.push_back({in, in + g.elements * element(g.dtype), false});
    spans.push_back({out, out + g.elements * element(g.out_dtype), true});
  }
  std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.begin < b.begin; });
  uintptr_t any = 0, written = 0;   // the furthest ends so far
  for (const Span& s : spans) {
    if (s.begin < (s.written ? any : written))
      return fail(SSD_ERR_BAD_VALUE, "an output overlaps another tensor");
    any = std::max(any, s.end);
    if (s.written) written = std::max(written, s.end);
  }
  return SSD_OK;
}

}  // namespace

extern "C" {

int ssd_block_abi_version(void) { return SSD_BLOCK_ABI_VERSION; }

ssd_status ssd_add_norm_fwd(const ssd_add_norm_problem* prob, const void* x,
                            const ssd_strides* x_strides, const void* residual,
                            const float* weight, void* h, void* y, void* q, float* scale,
                            void* stream) {
  return guarded([&] {
    if (!prob || !x || !weight || (!y && !q) || !q != !scale)
      return fail(SSD_ERR_NULL_POINTER,
                  "prob, x, weight and y or q must not be NULL, and q and scale go together");
    const ssd_add_norm_problem& p = *prob;
    ssd_status st = add_norm_shape(p);
    if (st != SSD_OK) return st;
    BlockNormArgs a{};
    strides_of(x_strides, p.seqlen, p.channels, a.xs);
    st = check_strides("x", a.xs, p.batch, p.seqlen, p.channels, false);
    if (st != SSD_OK) return st;
    if (!is_aligned(x, element(p.io_dtype)))
      return fail(SSD_ERR_MISALIGNED, "x must have the alignment of its element");
    if (!aligned16(residual, weight, h, y, q, scale))
      return fail(SSD_ERR_MISALIGNED, "every other tensor pointer must be 16-byte aligned");
    st = add_norm_supported(p, true);
    if (st != SSD_OK) return st;
    a.batch = p.batch;
    a.L = p.seqlen;
    join_batches(&a.batch, &a.L, a.xs);
    a.C = p.channels;
    a.G = 1;
    a.eps = p.eps;
    a.bf16 = p.io_dtype == SSD_BF16;
    a.res_bf16 = p.residual_dtype == SSD_BF16;
    a.x = x;
    a.r = residual;
    a.w = weight;
    a.h = h;
    a.y = y;
    a.q = static_cast<unsigned char*>(q);
    a.scale = scale;
    return launched(launch_block_norm(a, static_cast<hipStream_t>(stream)), "residual norm launch");
  });
}

ssd_status ssd_add_norm_bwd_workspace_size(const ssd_add_norm_problem* prob, size_t* bytes) {
  return guarded([&] {
    if (!prob || !bytes) return fail(SSD_ERR_NULL_POINTER, "prob and bytes must not be NULL");
    ssd_status st = add_norm_shape(*prob);
    if (st == SSD_OK) st = add_norm_supported(*prob, false);
    if (st != SSD_OK) return st;
    *bytes = add_norm_bwd_workspace(prob->batch * prob->seqlen, prob->channels, prob->io_dtype == SSD_BF16,
                                    prob->residual_dtype == SSD_BF16);
    return ok();
  });
}

ssd_status ssd_add_norm_bwd(const ssd_add_norm_problem* prob, const void* h, const float* weight,
                            const void* dy, const void* dh, void* dx, void* dresidual,
                            float* dweight, void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&] {
    if (!prob || !h || !weight || !dy || (!dx && !dresidual) || !dweight || !workspace)
      return fail(SSD_ERR_NULL_POINTER,
                  "prob, h, weight, dy, dx or dresidual, dweight and workspace must not be NULL");
    const ssd_add_norm_problem& p = *prob;
    ssd_status st = add_norm_shape(p);
    if (st != SSD_OK) return st;
    if (!aligned16(h, weight, dy, dh, dx, dresidual, dweight, workspace))
      return fail(SSD_ERR_MISALIGNED, "every tensor pointer must be 16-byte aligned");
    st = add_norm_supported(p, false);
    if (st != SSD_OK) return st;
    AddNormBwdArgs a{};
    a.rows = p.batch * p.seqlen;
    a.C = p.channels;
    const size_t need = add_norm_bwd_workspace(a.rows, a.C, p.io_dtype == SSD_BF16, p.residual_dtype == SSD_BF16);
    if (workspace_bytes < need)
      return fail(SSD_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
    a.eps = p.eps;
    a.bf16 = p.io_dtype == SSD_BF16;
    a.res_bf16 = p.residual_dtype == SSD_BF16;
    a.h = h;
    a.w = weight;
    a.dy = dy;
    a.dh = dh;
    a.dx = dx;
    a.dres = dresidual;
    a.dw = dweight;
    a.workspace = workspace;
    return launched(launch_add_norm_bwd(a, static_cast<hipStream_t>(stream)), "residual norm backward launch");
  });
}

ssd_status ssd_gated_norm_fwd_8bit(const ssd_gated_norm_problem* prob, const void* x,
                                   const void* z, const ssd_strides* z_strides,
                                   const float* weight, void* q, float* scale, void* stream) {
  return guarded([&] {
    if (!prob || !x || !weight || !q || !scale)
      return fail(SSD_ERR_NULL_POINTER, "prob, x, weight, q and scale must not be NULL");
    const ssd_gated_norm_problem& p = *prob;
    ssd_status st = norm_shape(p);
    if (st != SSD_OK) return st;
    BlockNormArgs a{};
    strides_of(nullptr, p.seqlen, p.channels, a.xs);
    strides_of(z_strides, p.seqlen, p.channels, a.zs);
    if (z) {
      st = check_strides("z", a.zs, p.batch, p.seqlen, p.channels, false);
      if (st != SSD_OK) return st;
    }
    if (!is_aligned(z, element(p.io_dtype)))
      return fail(SSD_ERR_MISALIGNED, "z must have the alignment of its element");
    if (!aligned16(x, weight, q, scale))
      return fail(SSD_ERR_MISALIGNED, "every other tensor pointer must be 16-byte aligned");
    st = norm_supported(p);
    if (st != SSD_OK) return st;
    if (p.ngroups > 1 && p.channels / p.ngroups % 128 != 0)
      return fail(SSD_ERR_UNSUPPORTED, "the channels of several groups must be whole blocks of 128 (got %lld)",
                  (long long)(p.channels / p.ngroups));
    if (!block_norm_grid_ok(p.batch, p.seqlen, p.channels, p.ngroups, z != nullptr))
      return fail(SSD_ERR_UNSUPPORTED, "grid too large for this build");
    a.batch = p.batch;
    a.L = p.seqlen;
    a.C = p.channels;
    a.G = p.ngroups;
    a.eps = p.eps;
    a.bf16 = p.io_dtype == SSD_BF16;
    a.gate = z ? 1 + p.norm_before_gate : 0;
    a.res_bf16 = a.bf16;
    a.x = x;
    a.r = z;
    a.w = weight;
    a.q = static_cast<unsigned char*>(q);
    a.scale = scale;
    return launched(launch_block_norm(a, static_cast<hipStream_t>(stream)), "8-bit gated norm launch");
  });
}

ssd_status ssd_quant8(const ssd_quant8_problem* prob, const void* x, const ssd_strides* x_strides,
                      void* q, float* scale, void* qt, float* scale_t, void* stream) {
  return guarded([&] {
    if (!prob || !x || (!q && !qt) || !q != !scale || !qt != !scale_t)
      return fail(SSD_ERR_NULL_POINTER,
                  "prob, x and q or qt must not be NULL, and q and scale, qt and scale_t go together");
    const ssd_quant8_problem& p = *prob;
    ssd_status st = quant_shape(p);
    if (st != SSD_OK) return st;
    Quant8Args a{};
    strides_of(x_strides, p.seqlen, p.channels, a.xs);
    st = check_strides("x", a.xs, p.batch, p.seqlen, p.channels, false);
    if (st != SSD_OK) return st;
    if (!is_aligned(x, element(p.io_dtype)))
      return fail(SSD_ERR_MISALIGNED, "x must have the alignment of its element");
    if (!aligned16(q, scale, qt, scale_t))
      return fail(SSD_ERR_MISALIGNED, "every other tensor pointer must be 16-byte aligned");
    if ((__int128)p.batch * p.seqlen > kMostRows || p.channels > kMostRows)
      return fail(SSD_ERR_UNSUPPORTED, "at most 2^31 - 1 rows and columns");
    if (!quant8_grid_ok(p.batch * p.seqlen, p.channels, p.tile, qt != nullptr))
      return fail(SSD_ERR_UNSUPPORTED, "grid too large for this build");
    a.batch = p.batch;
    a.L = p.seqlen;
    join_batches(&a.batch, &a.L, a.xs);
    a.C = p.channels;
    a.bf16 = p.io_dtype == SSD_BF16;
    a.tile = p.tile;
    a.x = x;
    a.q = static_cast<unsigned char*>(q);
    a.scale = scale;
    a.qt = static_cast<unsigned char*>(qt);
    a.scale_t = scale_t;
    return launched(launch_quant8(a, static_cast<hipStream_t>(stream)), "quantising launch");
  });
}

ssd_status ssd_matmul8_workspace_size(const ssd_matmul8_problem* prob, size_t* bytes) {
  return guarded([&] {
    if (!prob || !bytes) return fail(SSD_ERR_NULL_POINTER, "prob and bytes must not be NULL");
    ssd_status st = matmul_shape(*prob);
    if (st == SSD_OK) st = matmul_supported(*prob);
    if (st != SSD_OK) return st;
    *bytes = matmul8_workspace(prob->rows, prob->cols, prob->depth, prob->out_dtype == SSD_BF16);
    return ok();
  });
}

ssd_status ssd_matmul8(const ssd_matmul8_problem* prob, const void* x, const float* xs,
                       const void* w, const float* ws, void* y, void* workspace,
                       size_t workspace_bytes, void* stream) {
  return guarded([&] {
    if (!prob || !x || !xs || !w || !ws || !y)
      return fail(SSD_ERR_NULL_POINTER, "prob, x, xs, w, ws and y must not be NULL");
    const ssd_matmul8_problem& p = *prob;
    ssd_status st = matmul_shape(p);
    if (st != SSD_OK) return st;
    if (!aligned16(x, xs, w, ws, y, workspace))
      return fail(SSD_ERR_MISALIGNED, "every tensor pointer must be 16-byte aligned");
    st = matmul_supported(p);
    if (st != SSD_OK) return st;
    const size_t need = matmul8_workspace(p.rows, p.cols, p.depth, p.out_dtype == SSD_BF16);
    if (need > 0 && (!workspace || workspace_bytes < need))
      return fail(SSD_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace ? workspace_bytes : size_t(0),
                  need);
    Matmul8Args a{};
    a.M = p.rows;
    a.N = p.cols;
    a.K = p.depth;
    a.tile = p.w_tile;
    a.out_bf16 = p.out_dtype == SSD_BF16;
    a.x = static_cast<const unsigned char*>(x);
    a.xs = xs;
    a.w = static_cast<const unsigned char*>(w);
    a.ws = ws;
    a.y = y;
    a.workspace = workspace;
    return launched(launch_matmul8(a, static_cast<hipStream_t>(stream)), "8-bit product launch");
  });
}

ssd_status ssd_clip_grads_workspace_size(const ssd_grad* grads, int64_t n, size_t* bytes) {
  return guarded([&] {
    if (!grads || !bytes) return fail(SSD_ERR_NULL_POINTER, "grads and bytes must not be NULL");
    ssd_status st = clip_list(grads, n);
    if (st != SSD_OK) return st;
    *bytes = clip_workspace(grads, n);
    return ok();
  });
}

ssd_status ssd_clip_grads(const ssd_grad* grads, int64_t n, const ssd_clip_options* options,
                          float* norm, void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&] {
    if (!grads || !options || !norm || !workspace)
      return fail(SSD_ERR_NULL_POINTER, "grads, options, norm and workspace must not be NULL");
    for (int64_t i = 0; i < n; ++i)
      if (grads[i].elements > 0 && (!grads[i].grad || !grads[i].out))
        return fail(SSD_ERR_NULL_POINTER, "grads[%lld]: grad and out must not be NULL", (long long)i);
    if (n <= 0) return fail(SSD_ERR_BAD_SHAPE, "there must be at least one tensor");
    for (int64_t i = 0; i < n; ++i)
      if (grads[i].elements < 0) return fail(SSD_ERR_BAD_SHAPE, "grads[%lld]: negative size", (long long)i);
    for (int64_t i = 0; i < n; ++i)
      for (int32_t d : {grads[i].dtype, grads[i].out_dtype})
        if (d != SSD_BF16 && d != SSD_F32)
          return fail(SSD_ERR_BAD_DTYPE, "grads[%lld]: dtypes must be SSD_BF16 or SSD_F32 (got %d)", (long long)i, d);
    const ssd_clip_options& o = *options;
    if (o.reserved != 0) return fail(SSD_ERR_BAD_DTYPE, "reserved field must be 0");
    if (!(o.max_norm > 0.0)) return fail(SSD_ERR_BAD_VALUE, "max_norm must be > 0");
    if (!(o.eps >= 0.0) || std::isinf(o.eps)) return fail(SSD_ERR_BAD_VALUE, "eps must be finite and >= 0");
    if (!(o.grad_scale > 0.0) || std::isinf(o.grad_scale))
      return fail(SSD_ERR_BAD_VALUE, "grad_scale must be finite and > 0");
    ssd_status st = clip_list(grads, n);   // sizes that overflow nothing, before they are added up
    if (st != SSD_OK) return st;
    st = clip_overlaps(grads, n, norm);
    if (st != SSD_OK) return st;
    for (int64_t i = 0; i < n; ++i)
      if (grads[i].elements > 0 &&
          (!is_aligned(grads[i].grad, element(grads[i].dtype)) || !is_aligned(grads[i].out, element(grads[i].out_dtype))))
        return fail(SSD_ERR_MISALIGNED, "grads[%lld]: must have the alignment of its element", (long long)i);
    if (!is_aligned(norm, 4) || !is_aligned(workspace, 16))
      return fail(SSD_ERR_MISALIGNED, "norm must be 4-byte and workspace 16-byte aligned");
    const size_t need = clip_workspace(grads, n);
    if (workspace_bytes < need)
      return fail(SSD_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
    return launched(launch_clip(grads, n, o, norm, workspace, static_cast<hipStream_t>(stream)), "clipping launch");
  });
}

}  // extern "C"
