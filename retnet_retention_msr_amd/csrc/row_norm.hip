// Norms of a block and their gradients, a row at a time.
//
//   gated norm (per head): z = xhat w + b, y = z sw(g), sw(g) = g sigmoid(g)
//     dz = dy sw(g), dg = dy z sw'(g), sw'(g) = s (1 + g (1 - s)), s = sigmoid(g)
//   residual norm: r = alpha residual + scale x, y = xhat(r) w + b
// with xhat = (v - mean) rstd (layer form) or v rstd (rms form), and
//   dv = rstd (q - mean(q) - xhat mean(q xhat)), q the gradient of xhat
// (without mean(q) in the rms form). Parameter gradients are sums over rows.
//
// One workgroup of 256 threads takes a row at a time and reads it again for
// each pass over it.
#include "block.h"
#include "gate.h"

namespace ret {

namespace {

constexpr int kThreads = 256;

// Mean and 1 / deviation of a row given by load(c), c < d.
template <typename F>
__device__ __forceinline__ void row_stats(F load, int d, const NormArgs& n, float* red, float& mean, float& rstd) {
  mean = 0.0f;
  if (!n.rms) {
    float s = 0.0f;
    for (int c = threadIdx.x; c < d; c += kThreads) s += load(c);
    mean = block_sum_256(s, red) / d;
  }
  float s = 0.0f;
  for (int c = threadIdx.x; c < d; c += kThreads) {
    const float e = load(c) - mean;
    s += e * e;
  }
  rstd = 1.0f / sqrtf(block_sum_256(s, red) / d + n.eps);
}

__device__ __forceinline__ float param(const float* p, int64_t i, float none) { return p ? p[i] : none; }

template <typename T>
__global__ void __launch_bounds__(kThreads) gated_norm_kernel(View o, View gate, View y, int H, int N, int d, NormArgs n) {
  __shared__ float red[4];
  const int64_t row = blockIdx.x;
  const int t = static_cast<int>(row % N), h = static_cast<int>(row / N % H), b = static_cast<int>(row / N / H);
  const T* op = reinterpret_cast<const T*>(o.data) + b * o.sb + h * o.sh + t * o.sn;
  const T* gp = reinterpret_cast<const T*>(gate.data) + b * gate.sb + h * gate.sh + t * gate.sn;
  T* yp = reinterpret_cast<T*>(y.data) + b * y.sb + h * y.sh + t * y.sn;
  float mean, rstd;
  row_stats([&](int c) { return Elem<T>::load(op, c); }, d, n, red, mean, rstd);
  for (int c = threadIdx.x; c < d; c += kThreads) {
    const int64_t i = static_cast<int64_t>(h) * d + c;
    float z = fmaf((Elem<T>::load(op, c) - mean) * rstd, param(n.weight, i, 1.0f), param(n.bias, i, 0.0f));
    if (gate.data) {
      float s, less;
      const float g = Elem<T>::load(gp, c);
      sigmoid_pair(g, s, less);
      z *= g * s;
    }
    Elem<T>::store(yp, c, z);
  }
}

// Grid (parts, H): a workgroup takes every parts-th row of its head and adds
// what its threads' columns contribute to its own rows of the partial sums.
template <typename T>
__global__ void __launch_bounds__(kThreads)
gated_norm_backward_kernel(View dy, View o, View gate, View d_o, View d_gate, int B, int H, int N, int d, NormArgs n,
                           float* partial) {
  __shared__ float red[4];
  const int h = blockIdx.y, parts = gridDim.x;
  float* sums = partial ? partial + (static_cast<int64_t>(h) * parts + blockIdx.x) * kGatedNormSums * d : nullptr;
  if (sums)
    for (int c = threadIdx.x; c < d; c += kThreads) sums[c] = sums[d + c] = 0.0f;
  for (int64_t row = blockIdx.x; row < static_cast<int64_t>(B) * N; row += parts) {
    const int t = static_cast<int>(row % N), b = static_cast<int>(row / N);
    const T* dyp = reinterpret_cast<const T*>(dy.data) + b * dy.sb + h * dy.sh + t * dy.sn;
    const T* op = reinterpret_cast<const T*>(o.data) + b * o.sb + h * o.sh + t * o.sn;
    const T* gp = reinterpret_cast<const T*>(gate.data) + b * gate.sb + h * gate.sh + t * gate.sn;
    T* dop = reinterpret_cast<T*>(d_o.data) + b * d_o.sb + h * d_o.sh + t * d_o.sn;
    T* dgp = reinterpret_cast<T*>(d_gate.data) + b * d_gate.sb + h * d_gate.sh + t * d_gate.sn;
    float mean, rstd;
    row_stats([&](int c) { return Elem<T>::load(op, c); }, d, n, red, mean, rstd);
    auto dz_of = [&](int c) {
      float v = Elem<T>::load(dyp, c);
      if (gate.data) {
        float s, less;
        const float g = Elem<T>::load(gp, c);
        sigmoid_pair(g, s, less);
        v *= g * s;
      }
      return v;
    };
    float s1 = 0.0f, s2 = 0.0f;
    for (int c = threadIdx.x; c < d; c += kThreads) {
      const int64_t i = static_cast<int64_t>(h) * d + c;
      const float xhat = (Elem<T>::load(op, c) - mean) * rstd;
      const float dz = dz_of(c);
      if (gate.data) {
        float s, less;
        const float g = Elem<T>::load(gp, c);
        sigmoid_pair(g, s, less);
        const float z = fmaf(xhat, param(n.weight, i, 1.0f), param(n.bias, i, 0.0f));
        Elem<T>::store(dgp, c, Elem<T>::load(dyp, c) * z * (s * fmaf(g, less, 1.0f)));
      }
      if (sums) {
        sums[c] += dz * xhat;
        sums[d + c] += dz;
      }
      const float q = dz * param(n.weight, i, 1.0f);
      s1 += q;
      s2 += q * xhat;
    }
    s1 = n.rms ? 0.0f : block_sum_256(s1, red) / d;
    s2 = block_sum_256(s2, red) / d;
    for (int c = threadIdx.x; c < d; c += kThreads) {
      const int64_t i = static_cast<int64_t>(h) * d + c;
      const float xhat = (Elem<T>::load(op, c) - mean) * rstd;
      Elem<T>::store(dop, c, rstd * (dz_of(c) * param(n.weight, i, 1.0f) - s1 - xhat * s2));
    }
  }
}

// out[k][head * d + c] = sum over parts of partial[head][part][k][c].
__global__ void __launch_bounds__(kThreads)
param_sum_kernel(const float* partial, int heads, int parts, int sums, int d, float* out0, float* out1, float* out2) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int k = blockIdx.y;
  float* out = k == 0 ? out0 : k == 1 ? out1 : out2;
  if (!out || i >= static_cast<int64_t>(heads) * d) return;
  const int64_t head = i / d;
  const int c = static_cast<int>(i - head * d);
  float s = 0.0f;
  for (int p = 0; p < parts; ++p) s += partial[((head * parts + p) * sums + k) * d + c];
  out[i] = s;
}

hipError_t sum_params(const float* partial, int heads, int parts, int sums, int d, float* out0, float* out1,
                      float* out2, hipStream_t stream) {
  const int64_t n = static_cast<int64_t>(heads) * d;
  param_sum_kernel<<<dim3(static_cast<unsigned>((n + kThreads - 1) / kThreads), sums), kThreads, 0, stream>>>(
      partial, heads, parts, sums, d, out0, out1, out2);
  return hipGetLastError();
}

template <typename T, typename TR>
__global__ void __launch_bounds__(kThreads)
residual_norm_kernel(View x, View residual, View y, View r, int N, int D, NormArgs n, const float* scale, float alpha) {
  __shared__ float red[4];
  const int t = blockIdx.x % N, b = blockIdx.x / N;
  const T* xp = reinterpret_cast<const T*>(x.data) + b * x.sb + t * x.sn;
  const TR* sp = reinterpret_cast<const TR*>(residual.data) + b * residual.sb + t * residual.sn;
  T* yp = reinterpret_cast<T*>(y.data) + b * y.sb + t * y.sn;
  TR* rp = reinterpret_cast<TR*>(r.data) + b * r.sb + t * r.sn;
  auto value = [&](int c) {
    return fmaf(alpha, Elem<TR>::load(sp, c), param(scale, c, 1.0f) * Elem<T>::load(xp, c));
  };
  float mean, rstd;
  row_stats(value, D, n, red, mean, rstd);
  for (int c = threadIdx.x; c < D; c += kThreads) {
    const float v = value(c);
    Elem<TR>::store(rp, c, v);
    Elem<T>::store(yp, c, fmaf((v - mean) * rstd, param(n.weight, c, 1.0f), param(n.bias, c, 0.0f)));
  }
}

template <typename T, typename TR>
__global__ void __launch_bounds__(kThreads)
residual_norm_backward_kernel(View dy, View dr, View r, View x, View dx, View dres, int64_t rows, int N, int D,
                              NormArgs n, const float* scale, float alpha, float* partial) {
  __shared__ float red[4];
  float* sums = partial ? partial + static_cast<int64_t>(blockIdx.x) * kResidualNormSums * D : nullptr;
  if (sums)
    for (int c = threadIdx.x; c < kResidualNormSums * D; c += kThreads) sums[c] = 0.0f;
  __syncthreads();
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int t = static_cast<int>(row % N), b = static_cast<int>(row / N);
    const T* dyp = reinterpret_cast<const T*>(dy.data) + b * dy.sb + t * dy.sn;
    const TR* drp = dr.data ? reinterpret_cast<const TR*>(dr.data) + b * dr.sb + t * dr.sn : nullptr;
    const TR* rp = reinterpret_cast<const TR*>(r.data) + b * r.sb + t * r.sn;
    const T* xp = x.data ? reinterpret_cast<const T*>(x.data) + b * x.sb + t * x.sn : nullptr;
    T* dxp = dx.data ? reinterpret_cast<T*>(dx.data) + b * dx.sb + t * dx.sn : nullptr;
    TR* dsp = reinterpret_cast<TR*>(dres.data) + b * dres.sb + t * dres.sn;
    float mean, rstd;
    row_stats([&](int c) { return Elem<TR>::load(rp, c); }, D, n, red, mean, rstd);
    float s1 = 0.0f, s2 = 0.0f;
    for (int c = threadIdx.x; c < D; c += kThreads) {
      const float q = Elem<T>::load(dyp, c) * param(n.weight, c, 1.0f);
      s1 += q;
      s2 += q * ((Elem<TR>::load(rp, c) - mean) * rstd);
    }
    s1 = n.rms ? 0.0f : block_sum_256(s1, red) / D;
    s2 = block_sum_256(s2, red) / D;
    for (int c = threadIdx.x; c < D; c += kThreads) {
      const float g = Elem<T>::load(dyp, c);
      const float xhat = (Elem<TR>::load(rp, c) - mean) * rstd;
      const float v = (drp ? Elem<TR>::load(drp, c) : 0.0f) +
                      rstd * (g * param(n.weight, c, 1.0f) - s1 - xhat * s2);
      if (sums) {
        if (xp) sums[c] += v * Elem<T>::load(xp, c);
        sums[D + c] += g * xhat;
        sums[2 * D + c] += g;
      }
      Elem<TR>::store(dsp, c, alpha * v);
      if (dxp) Elem<T>::store(dxp, c, param(scale, c, 1.0f) * v);
    }
  }
}

}  // namespace

hipError_t launch_gated_norm(int dtype, const View& o, const View& gate, const View& y, int B, int H, int N, int d,
                             const NormArgs& norm, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(B) * H * N));
  if (dtype == 0) gated_norm_kernel<float><<<grid, kThreads, 0, stream>>>(o, gate, y, H, N, d, norm);
  else gated_norm_kernel<uint16_t><<<grid, kThreads, 0, stream>>>(o, gate, y, H, N, d, norm);
  return hipGetLastError();
}

hipError_t launch_gated_norm_backward(int dtype, const View& grad_y, const View& o, const View& gate,
                                      const View& grad_o, const View& grad_gate, int B, int H, int N, int d,
                                      const NormArgs& norm, float* grad_weight, float* grad_bias, void* workspace,
                                      hipStream_t stream) {
  const ParamPlan p = plan_params(H, static_cast<int64_t>(B) * N, d, kGatedNormSums);
  float* partial = grad_weight || grad_bias ? static_cast<float*>(workspace) : nullptr;
  const dim3 grid(p.parts, H);
  if (dtype == 0)
    gated_norm_backward_kernel<float><<<grid, kThreads, 0, stream>>>(grad_y, o, gate, grad_o, grad_gate, B, H, N, d,
                                                                     norm, partial);
  else
    gated_norm_backward_kernel<uint16_t><<<grid, kThreads, 0, stream>>>(grad_y, o, gate, grad_o, grad_gate, B, H, N,
                                                                        d, norm, partial);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !partial) return e;
  return sum_params(partial, H, p.parts, kGatedNormSums, d, grad_weight, grad_bias, nullptr, stream);
}

hipError_t launch_residual_norm(int dtype, int stream_dtype, const View& x, const View& residual, const View& y,
                                const View& r, int B, int N, int D, const NormArgs& norm, const float* scale,
                                float alpha, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(B) * N));
  if (dtype == 0)
    residual_norm_kernel<float, float><<<grid, kThreads, 0, stream>>>(x, residual, y, r, N, D, norm, scale, alpha);
  else if (stream_dtype == 0)
    residual_norm_kernel<uint16_t, float><<<grid, kThreads, 0, stream>>>(x, residual, y, r, N, D, norm, scale, alpha);
  else
    residual_norm_kernel<uint16_t, uint16_t><<<grid, kThreads, 0, stream>>>(x, residual, y, r, N, D, norm, scale,
                                                                            alpha);
  return hipGetLastError();
}

hipError_t launch_residual_norm_backward(int dtype, int stream_dtype, const View& grad_y, const View& grad_r,
                                         const View& r, const View& x, const View& grad_x, const View& grad_residual,
                                         int B, int N, int D, const NormArgs& norm, const float* scale, float alpha,
                                         float* grad_scale, float* grad_weight, float* grad_bias, void* workspace,
                                         hipStream_t stream) {
  const int64_t rows = static_cast<int64_t>(B) * N;
  const ParamPlan p = plan_params(1, rows, D, kResidualNormSums);
  float* partial = grad_scale || grad_weight || grad_bias ? static_cast<float*>(workspace) : nullptr;
  View xs = x;
  if (!grad_scale) xs.data = nullptr;
  const dim3 grid(p.parts);
  if (dtype == 0)
    residual_norm_backward_kernel<float, float><<<grid, kThreads, 0, stream>>>(
        grad_y, grad_r, r, xs, grad_x, grad_residual, rows, N, D, norm, scale, alpha, partial);
  else if (stream_dtype == 0)
    residual_norm_backward_kernel<uint16_t, float><<<grid, kThreads, 0, stream>>>(
        grad_y, grad_r, r, xs, grad_x, grad_residual, rows, N, D, norm, scale, alpha, partial);
  else
    residual_norm_backward_kernel<uint16_t, uint16_t><<<grid, kThreads, 0, stream>>>(
        grad_y, grad_r, r, xs, grad_x, grad_residual, rows, N, D, norm, scale, alpha, partial);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !partial) return e;
  return sum_params(partial, 1, p.parts, kResidualNormSums, D, grad_scale, grad_weight, grad_bias, stream);
}

}  // namespace ret
