// layer_host.hpp -- between layer_api.cpp (argument checks) and the kernels'
// launchers: one plain struct of checked arguments per operator.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "ssd_device.hpp"

namespace ssd {

struct ConvArgs {
  int64_t batch, L, C;
  int W, bf16, silu;
  int vec;        // every pointer, stride and split allows accesses of four channels
  int one_run;    // forward with fin == init: one thread takes all tokens of its channels
  const void* x;
  int64_t xs[2];
  const float *w, *bias;
  const void* init;
  void* y[3];     // outputs, or the upstream gradients of the backward pass
  int64_t end[3]; // running channel counts of the outputs
  void* fin;
  const void* dfin;
  void* dx;
  int64_t dxs[2];
  float *dw, *db;
  void* dinit;
  void* workspace;
};
hipError_t launch_conv_fwd(const ConvArgs& a, hipStream_t stream);
hipError_t launch_conv_bwd(const ConvArgs& a, hipStream_t stream);
size_t conv_bwd_workspace(int64_t batch, int64_t L, int64_t C, int W);
int conv_grid_ok(int64_t batch, int64_t L, int64_t C);

struct NormArgs {
  int64_t batch, L, D;
  int64_t G;
  float eps;
  int before, bf16;
  int vec;        // every pointer, stride and group allows 16-byte accesses
  const void *x, *z;
  int64_t zs[2];
  const float* w;
  void* y;
  const void* dy;
  void *dx, *dz;
  int64_t dzs[2];
  float* dw;
  void* workspace;
};
hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t stream);
hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t stream);
size_t norm_bwd_workspace(int64_t batch, int64_t L, int64_t D, int64_t G, int io_bf16);
int64_t norm_group_limit();
int norm_grid_ok(int64_t batch, int64_t L, int64_t D, int64_t G);

struct ScanArgs {
  int64_t batch, L, D, N, G;
  int bf16;
  int vec;           // the step: B and C allow accesses of 4 elements, dstate is a multiple of 4
  const DtXform* xf;
  const void *x, *dt;
  const float* A;
  const void* B;
  int64_t bs[2];
  const void* C;
  int64_t cs[2];
  const float* Dv;
  const void* z;
  int64_t zs[2];
  const float* init;
  void* y;
  float* fin;
  float* state;      // the step: read and written
  const void* dy;
  const float* dfin;
  void *dx, *ddt;
  float* dA;
  void *dB, *dC;
  float* dD;
  void* dz;
  int64_t dzs[2];
  float *dinit, *dbias;
  void* workspace;
};
hipError_t launch_selscan_fwd(const ScanArgs& a, hipStream_t stream);
hipError_t launch_selscan_step(const ScanArgs& a, hipStream_t stream);
hipError_t launch_selscan_bwd(const ScanArgs& a, hipStream_t stream);
size_t selscan_fwd_workspace(int64_t batch, int64_t L, int64_t D, int64_t N, int64_t G);
size_t selscan_bwd_workspace(int64_t batch, int64_t L, int64_t D, int64_t N, int64_t G);
int selscan_grid_ok(int64_t batch, int64_t L, int64_t D, int64_t N, int64_t G);

}  // namespace ssd
