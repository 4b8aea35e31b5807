// Internal launch interface of the layer operators (kda_conv.cu, kda_ssm.cu,
// kda_ssm_bwd.cu, kda_norm.cu), called by the C-ABI layer (kda_layer_api.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

namespace kda {

enum Act { kActNone = 0, kActSilu = 1, kActSigmoid = 2 };

// From kda_api.cu: stream-ordered workspace (see there) and the last CUDA
// error of the calling thread.
cudaError_t api_take_workspace(size_t bytes, cudaStream_t stream, void** ws);
void api_record_cuda_error(cudaError_t e);

// SM count of the current device (looked up once per device).
inline int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  n = known[dev].load(std::memory_order_relaxed);
  if (n > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
    return 148;
  known[dev].store(n, std::memory_order_relaxed);
  return n;
}

inline bool aligned_to(const void* p, size_t bytes) {
  return ((uintptr_t)p % bytes) == 0;
}

struct ConvArgs {
  const void* x;
  const float* weight;
  const float* bias;      // or null
  const void* past;       // initial state [n_seqs, W-1, D], or null
  const int32_t* cu;      // or null (dense)
  void* out;
  void* final_state;      // or null
  const void* d_out;      // backward
  const void* d_final;    // or null
  void* dx;
  float* dw;
  float* db;              // or null
  void* d_past;           // or null
  int n_seqs, T, D, W, act;
  int64_t tokens, x_stride;
  bool bf16;
};
cudaError_t launch_conv_fwd(const ConvArgs& a, cudaStream_t stream);
size_t conv_bwd_workspace_bytes(const ConvArgs& a);
cudaError_t launch_conv_bwd(const ConvArgs& a, void* workspace, cudaStream_t stream);
// a.past is read and overwritten through a.final_state (the same memory)
cudaError_t launch_conv_step(const ConvArgs& a, cudaStream_t stream);

struct SsmArgs {
  const void *u, *delta, *B, *C, *z;  // z may be null
  const float *A, *skip, *bias, *h0;  // skip, bias, h0 may be null
  const int32_t* cu;
  void* out;
  float* h_out;  // final state or null
  int n_seqs, T, D, S, G;
  int64_t tokens, u_stride, delta_stride, z_stride, b_stride, b_group, c_stride, c_group;
  bool bf16, softplus;
};
// The scan of long sequences with few CTAs runs split (sms: the device's SMs).
size_t ssm_fwd_workspace_bytes(const SsmArgs& a, int sms);
cudaError_t launch_ssm_fwd(const SsmArgs& a, void* workspace, int sms, cudaStream_t stream);
cudaError_t launch_ssm_step(const SsmArgs& a, cudaStream_t stream);
struct SsmBwdArgs {
  SsmArgs f;
  const void* d_out;
  const float* d_final;  // or null
  void *du, *ddelta, *dB, *dC, *dz;
  float *dA, *dskip, *dbias, *dh0;
};
size_t ssm_bwd_workspace_bytes(const SsmBwdArgs& a, int sms);
int ssm_bwd_kernel_count(const SsmBwdArgs& a, int sms);
cudaError_t launch_ssm_bwd(const SsmBwdArgs& a, void* workspace, int sms, cudaStream_t stream);

struct NormArgs {
  const void *x, *gate, *residual;               // gate, residual may be null
  const float *post_weight, *scale, *pre_weight;  // each may be null
  void *out, *normed;
  const void *d_out, *d_normed;  // each may be null (zero)
  void *dx, *dgate, *dres;
  float *dpost, *dscale, *dpre;
  int64_t tokens, x_stride, gate_stride;
  int heads, width, act;
  bool bf16, res_bf16, gate_first;
  float eps;
};
cudaError_t launch_norm_fwd(const NormArgs& a, cudaStream_t stream);
size_t norm_bwd_workspace_bytes(const NormArgs& a, int sms);
cudaError_t launch_norm_bwd(const NormArgs& a, void* workspace, int sms, cudaStream_t stream);

}  // namespace kda
