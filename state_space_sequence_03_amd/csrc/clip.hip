// clip.hip -- the global norm over many gradients, and clipping by it.
//
//     norm = s sqrt(sum g^2),  out = g s min(1, most / (norm + eps))   (s alone where the
//     norm, rounded to fp32, is not finite)
//
// Bound by HBM: every gradient is read twice, since no factor is known before the last
// one has been read, and written once: 241 M bf16 gradients into fp32 410 us, 1.93 GB at
// 4.7 TB/s (a large copy: 5.07).  A launch takes the pointers of up to kTensors
// tensors in its arguments, so a call needs no copy to the device and can be captured;
// longer lists take more launches.  Sums of squares are 64-bit from the first addition
// (two double operations per element, far below the memory's rate), part sums lie in the
// workspace and are added in a fixed order.
#include "block_device.hpp"
#include "block_host.hpp"

namespace ssd {

constexpr int kTensors = 128;       // 29 bytes each
constexpr int64_t kLeastChunk = 8192;
constexpr int64_t kMostParts = 1024;   // part sums that every workgroup of the second pass adds by itself

struct Tensors {
  const void* grad[kTensors];
  void* out[kTensors];
  int64_t n[kTensors];
  int32_t first[kTensors + 1];   // its first workgroup
  uint8_t kind[kTensors];        // 1: grad is bf16, 2: out is bf16
  int32_t count;
  int32_t chunk8;                // chunk / 8
};
// with the other arguments of clip_scale_kernel
static_assert(sizeof(Tensors) + 5 * 8 + 8 + 8 <= 4096, "a launch's arguments have 4 KB");

// The tensor of workgroup b.
__device__ __forceinline__ int tensor_of(const Tensors& t, int b) {
  int lo = 0, hi = t.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (t.first[mid] <= b) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ double block_sum(double v) {
  __shared__ double waves[4];
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, kWave);
  __syncthreads();
  if (threadIdx.x % kWave == 0) waves[threadIdx.x / kWave] = v;
  __syncthreads();
  return (waves[0] + waves[1]) + (waves[2] + waves[3]);
}

// f(position, raw values, how many of them count) for every eighth element of a thread's share of n,
// with kAhead loads on their way at a time.
constexpr int kAhead = 4;
template <typename T, typename F>
__device__ __forceinline__ void each_piece(const T* g, int64_t n, F f) {
  constexpr int64_t kStep = 8 * 256;
  int64_t i = 8 * (int64_t)threadIdx.x;
  for (; i + (kAhead - 1) * kStep + 8 <= n; i += kAhead * kStep) {
    Raw8<T> v[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) v[k] = raw8(g + i + k * kStep, 8);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) f(i + k * kStep, v[k], 8);
  }
  for (; i < n; i += kStep) {
    const int m = (int)(n - i < 8 ? n - i : 8);
    f(i, raw8(g + i, m), m);
  }
}

template <typename T>
__device__ __forceinline__ double squares(const T* g, int64_t n) {
  double s[2] = {0.0, 0.0};
  each_piece(g, n, [&](int64_t, const Raw8<T>& v, int) {
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e % 2] = fma((double)v[e], (double)v[e], s[e % 2]);
  });
  return s[0] + s[1];
}

__global__ void __launch_bounds__(256)
clip_squares_kernel(const Tensors t, double* __restrict__ part) {
  const int k = tensor_of(t, blockIdx.x);
  const int64_t chunk = 8 * (int64_t)t.chunk8, at = (blockIdx.x - t.first[k]) * chunk;
  const int64_t n = t.n[k] - at < chunk ? t.n[k] - at : chunk;
  const double s = t.kind[k] & 1 ? squares(static_cast<const bf16*>(t.grad[k]) + at, n)
                                 : squares(static_cast<const float*>(t.grad[k]) + at, n);
  const double sum = block_sum(s);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// The sum of n part sums, in every thread of a workgroup.
__device__ __forceinline__ double parts_sum(const double* part, int64_t n) {
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += 256) s += part[i];
  return block_sum(s);
}

// Many part sums into one.
__global__ void __launch_bounds__(256) clip_parts_kernel(const double* part, int64_t n, double* sum) {
  const double s = parts_sum(part, n);
  if (threadIdx.x == 0) *sum = s;
}

template <typename T, typename O>
__device__ __forceinline__ void scale_chunk(const T* g, O* out, int64_t n, float by) {
  each_piece(g, n, [&](int64_t i, const Raw8<T>& r, int m) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = r[e] * by;
    store8(out + i, m, v);
  });
}

__global__ void __launch_bounds__(256)
clip_scale_kernel(const Tensors t, const double* __restrict__ part, int64_t parts, double most,
                  double eps, double scale, float* __restrict__ norm_out, int first_launch) {
  const double norm = scale * sqrt(parts_sum(part, parts));
  if (first_launch && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
  double c = scale;
  if ((float)norm < INFINITY) c *= fmin(1.0, most / (norm + eps));   // finite as it is reported; false for NaN
  const float by = (float)c;
  const int b = gridDim.x - 1 - blockIdx.x;   // the last chunks first: they may still be in a cache
  const int k = tensor_of(t, b);
  const int64_t chunk = 8 * (int64_t)t.chunk8, at = (b - t.first[k]) * chunk;
  const int64_t n = t.n[k] - at < chunk ? t.n[k] - at : chunk;
  if (by == 1.0f && t.out[k] == t.grad[k]) return;
  const bf16* gb = static_cast<const bf16*>(t.grad[k]) + at;
  const float* gf = static_cast<const float*>(t.grad[k]) + at;
  bf16* ob = static_cast<bf16*>(t.out[k]) + at;
  float* of = static_cast<float*>(t.out[k]) + at;
  switch (t.kind[k]) {
    case 0: scale_chunk(gf, of, n, by); break;
    case 1: scale_chunk(gb, of, n, by); break;
    case 2: scale_chunk(gf, ob, n, by); break;
    default: scale_chunk(gb, ob, n, by); break;
  }
}

// Nothing but empty tensors.
__global__ void clip_none_kernel(float* norm_out) { *norm_out = 0.0f; }

// ---- host ----

namespace {

struct ClipPlan {
  int64_t chunk, parts;
};
// Chunks so that a large list takes about 4096 workgroups (241 M gradients 410 us; 8192: 418, 2048: 430), a small one at least
// kLeastChunk elements each.
ClipPlan clip_plan(const ssd_grad* g, int64_t n) {
  int64_t total = 0;
  for (int64_t i = 0; i < n; ++i) total += g[i].elements;
  ClipPlan p;
  p.chunk = total / 4096 / 8 * 8;
  if (p.chunk < kLeastChunk) p.chunk = kLeastChunk;
  p.parts = 0;
  for (int64_t i = 0; i < n; ++i) p.parts += (g[i].elements + p.chunk - 1) / p.chunk;
  return p;
}

}  // namespace

size_t clip_workspace(const ssd_grad* grads, int64_t n) {
  const ClipPlan p = clip_plan(grads, n);
  return size_t(p.parts + 1) * sizeof(double);
}

hipError_t launch_clip(const ssd_grad* grads, int64_t n, const ssd_clip_options& opt, float* norm,
                       void* workspace, hipStream_t stream) {
  const ClipPlan p = clip_plan(grads, n);
  double* part = static_cast<double*>(workspace);
  double* sum = part + p.parts;
  if (p.parts == 0) {
    hipLaunchKernelGGL(clip_none_kernel, dim3(1), dim3(1), 0, stream, norm);
    return hipGetLastError();
  }
  const bool many = p.parts > kMostParts;
  auto pass = [&](bool second) -> hipError_t {
    Tensors t;
    t.chunk8 = (int32_t)(p.chunk / 8);
    int64_t done = 0;
    for (int64_t i = 0; i < n;) {
      t.count = 0;
      t.first[0] = 0;
      for (; i < n && t.count < kTensors; ++i) {
        if (grads[i].elements == 0) continue;
        const int k = t.count++;
        t.grad[k] = grads[i].grad;
        t.out[k] = grads[i].out;
        t.n[k] = grads[i].elements;
        t.kind[k] = (uint8_t)((grads[i].dtype == SSD_BF16 ? 1 : 0) | (grads[i].out_dtype == SSD_BF16 ? 2 : 0));
        t.first[k + 1] = t.first[k] + (int32_t)((grads[i].elements + p.chunk - 1) / p.chunk);
      }
      if (t.count == 0) break;
      const dim3 grid((unsigned)t.first[t.count]);
      if (second)
        hipLaunchKernelGGL(clip_scale_kernel, grid, dim3(256), 0, stream, t, many ? sum : part,
                           many ? int64_t(1) : p.parts, opt.max_norm, opt.eps, opt.grad_scale, norm,
                           done == 0 ? 1 : 0);
      else
        hipLaunchKernelGGL(clip_squares_kernel, grid, dim3(256), 0, stream, t, part + done);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      done += t.first[t.count];
    }
    return hipSuccess;
  };
  hipError_t e = pass(false);
  if (e != hipSuccess) return e;
  if (many) {
    hipLaunchKernelGGL(clip_parts_kernel, dim3(1), dim3(256), 0, stream, part, p.parts, sum);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return pass(true);
}

}  // namespace ssd
