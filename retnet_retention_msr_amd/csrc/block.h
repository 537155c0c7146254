// Host-side launchers of the block operators (gated recurrence, gated norm,
// residual norm). Arguments were validated by the C ABI (block_api.cpp); each
// launcher returns the HIP status of its launches. Plain host C++, so that the
// validation code builds with a host compiler alone.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

namespace ret {

// A [B, H, N, d] tensor with a contiguous last dimension; strides in elements,
// 0 for dimensions of size 1.
struct View {
  char* data;
  int64_t sb, sh, sn;
};

// The sequences of a recurrence call: [S] rows of N tokens, or, with cu, S
// pieces of one row of N tokens, each at most max_len long.
struct Sequences {
  int S, H, N, d, max_len;
  const int* cu;  // device [S + 1] or nullptr
};

// Planning of a recurrence call: a pure function of the sizes.
struct ScanPlan {
  int64_t blocks;  // workgroups of the launch
  size_t bytes;    // workspace
};
inline ScanPlan plan_scan(int S, int H, int /*max_len*/, int d) {
  ScanPlan p{};
  p.blocks = static_cast<int64_t>(S) * H * ((d + 63) / 64);
  p.bytes = 0;
  return p;
}
hipError_t launch_gated_recurrence(int form, int dtype, const View& x, const View& gate, const View& h,
                                   const Sequences& q, const float* state_in, float* state_out, void* workspace,
                                   hipStream_t stream);
// x.data is nullptr when not given (log form).
hipError_t launch_gated_recurrence_backward(int form, int dtype, const View& grad_h, const View& x, const View& gate,
                                            const View& h, const View& grad_x, const View& grad_gate,
                                            const Sequences& q, const float* state_in, const float* grad_state_out,
                                            float* grad_state_in, void* workspace, hipStream_t stream);
hipError_t launch_gated_recurrence_step(int form, int dtype, const View& x, const View& gate, const View& h, int B,
                                        int H, int d, float* states, int nstates, const int* slots,
                                        hipStream_t stream);

struct NormArgs {
  float eps;
  int rms;
  const float* weight;
  const float* bias;
};

// gate.data is nullptr without a gate.
hipError_t launch_gated_norm(int dtype, const View& o, const View& gate, const View& y, int B, int H, int N, int d,
                             const NormArgs& norm, hipStream_t stream);
// Partial sums of the parameter gradients of `heads` heads of `rows` rows of d
// values: `parts` workgroups per head leave `sums` rows of d floats each.
struct ParamPlan {
  int parts;
  size_t bytes;
};
inline ParamPlan plan_params(int heads, int64_t rows, int d, int sums) {
  ParamPlan p{};
  p.parts = static_cast<int>(rows < 64 ? rows : 64);
  p.bytes = static_cast<size_t>(heads) * p.parts * sums * d * sizeof(float);
  return p;
}
constexpr int kGatedNormSums = 2;     // weight, bias
constexpr int kResidualNormSums = 3;  // scale, weight, bias
hipError_t launch_gated_norm_backward(int dtype, const View& grad_y, const View& o, const View& gate,
                                      const View& grad_o, const View& grad_gate, int B, int H, int N, int d,
                                      const NormArgs& norm, float* grad_weight, float* grad_bias, void* workspace,
                                      hipStream_t stream);
hipError_t launch_residual_norm(int dtype, int stream_dtype, const View& x, const View& residual, const View& y,
                                const View& r, int B, int N, int D, const NormArgs& norm, const float* scale,
                                float alpha, hipStream_t stream);
// grad_r.data, x.data and grad_x.data may be nullptr.
hipError_t launch_residual_norm_backward(int dtype, int stream_dtype, const View& grad_y, const View& grad_r,
                                         const View& r, const View& x, const View& grad_x, const View& grad_residual,
                                         int B, int N, int D, const NormArgs& norm, const float* scale, float alpha,
                                         float* grad_scale, float* grad_weight, float* grad_bias, void* workspace,
                                         hipStream_t stream);

}  // namespace ret
