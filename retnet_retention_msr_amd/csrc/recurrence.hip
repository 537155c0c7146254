// Gated linear recurrence per channel, its backward and its single token.
//
//   sigmoid form: a = 1 / (1 + e^-g), h_t = a_t h_{t-1} + (1 - a_t) x_t
//   log form:     a = e^g,            h_t = a_t h_{t-1} + x_t
// Backward, from the last token: w_t = a_t (dh_t + w_{t+1}) carries what
// h_{t-1} receives, u_t = dh_t + w_{t+1} is the whole gradient of h_t;
//   sigmoid form: dx = (1 - a) u, dg = a (1 - a) (h_{t-1} - x_t) u
//   log form:     dx = u,         dg = a h_{t-1} u
//
// One thread walks the tokens of one channel.
#include "block.h"
#include "gate.h"

namespace ret {

namespace {

constexpr int kThreads = 64;

template <int FORM>
__device__ __forceinline__ void gate_of(float g, float& a, float& c) {
  if (FORM == 0) {
    sigmoid_pair(g, a, c);
  } else {
    a = __builtin_amdgcn_exp2f(kLog2e * g);
    c = 1.0f;
  }
}

struct Piece {
  int64_t first;  // its first token in the row
  int len;
  int b;  // row of the batch
};
__device__ __forceinline__ Piece piece_of(const Sequences& q, int s) {
  if (!q.cu) return {0, q.N, s};
  int lo = q.cu[s], hi = q.cu[s + 1];
  lo = lo < 0 ? 0 : lo > q.N ? q.N : lo;
  hi = hi < lo ? lo : hi > q.N ? q.N : hi;
  return {lo, hi - lo > q.max_len ? q.max_len : hi - lo, 0};
}

template <typename T>
__device__ __forceinline__ T* row_of(const View& v, int b, int h) {
  return reinterpret_cast<T*>(v.data) + b * v.sb + h * v.sh;
}

template <typename T, int FORM>
__global__ void __launch_bounds__(kThreads)
recurrence_kernel(View x, View gate, View out, Sequences q, const float* state_in, float* state_out) {
  const int slabs = (q.d + kThreads - 1) / kThreads;
  const int64_t sh = blockIdx.x / slabs;
  const int c = (blockIdx.x % slabs) * kThreads + threadIdx.x;
  const int s = static_cast<int>(sh / q.H), h = static_cast<int>(sh % q.H);
  if (c >= q.d) return;
  const Piece p = piece_of(q, s);
  const T* xr = row_of<T>(x, p.b, h) + p.first * x.sn + c;
  const T* gr = row_of<T>(gate, p.b, h) + p.first * gate.sn + c;
  T* hr = row_of<T>(out, p.b, h) + p.first * out.sn + c;
  float now = state_in ? state_in[sh * q.d + c] : 0.0f;
  for (int t = 0; t < p.len; ++t) {
    float a, w;
    gate_of<FORM>(Elem<T>::load(gr, t * gate.sn), a, w);
    now = fmaf(a, now, w * Elem<T>::load(xr, t * x.sn));
    Elem<T>::store(hr, t * out.sn, now);
  }
  if (state_out) state_out[sh * q.d + c] = now;
}

template <typename T, int FORM>
__global__ void __launch_bounds__(kThreads)
recurrence_backward_kernel(View grad_h, View x, View gate, View hv, View grad_x, View grad_gate, Sequences q,
                           const float* state_in, const float* grad_state_out, float* grad_state_in) {
  const int slabs = (q.d + kThreads - 1) / kThreads;
  const int64_t sh = blockIdx.x / slabs;
  const int c = (blockIdx.x % slabs) * kThreads + threadIdx.x;
  const int s = static_cast<int>(sh / q.H), h = static_cast<int>(sh % q.H);
  if (c >= q.d) return;
  const Piece p = piece_of(q, s);
  const T* dr = row_of<T>(grad_h, p.b, h) + p.first * grad_h.sn + c;
  const T* xr = FORM == 0 ? row_of<T>(x, p.b, h) + p.first * x.sn + c : nullptr;
  const T* gr = row_of<T>(gate, p.b, h) + p.first * gate.sn + c;
  const T* hr = row_of<T>(hv, p.b, h) + p.first * hv.sn + c;
  T* dxr = row_of<T>(grad_x, p.b, h) + p.first * grad_x.sn + c;
  T* dgr = row_of<T>(grad_gate, p.b, h) + p.first * grad_gate.sn + c;
  const float start = state_in ? state_in[sh * q.d + c] : 0.0f;
  float w = grad_state_out ? grad_state_out[sh * q.d + c] : 0.0f;
  for (int t = p.len - 1; t >= 0; --t) {
    float a, keep;
    gate_of<FORM>(Elem<T>::load(gr, t * gate.sn), a, keep);
    const float u = Elem<T>::load(dr, t * grad_h.sn) + w;
    const float before = t > 0 ? Elem<T>::load(hr, (t - 1) * hv.sn) : start;
    if (FORM == 0) {
      Elem<T>::store(dxr, t * grad_x.sn, keep * u);
      Elem<T>::store(dgr, t * grad_gate.sn, a * keep * (before - Elem<T>::load(xr, t * x.sn)) * u);
    } else {
      Elem<T>::store(dxr, t * grad_x.sn, u);
      Elem<T>::store(dgr, t * grad_gate.sn, a * before * u);
    }
    w = a * u;
  }
  if (grad_state_in) grad_state_in[sh * q.d + c] = w;
}

// Grid: x over the channels of a row (H * d), y-strided over the B rows. A
// block takes row b unless an earlier row names the same slot; then it goes on
// with the later rows of that slot.
template <typename T, int FORM>
__global__ void __launch_bounds__(kThreads)
step_kernel(View x, View gate, View out, int B, int H, int d, float* states, int nstates, const int* slots) {
  const int channels = H * d;
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= channels) return;
  const int h = c / d, j = c - h * d;
  for (int b = blockIdx.y; b < B; b += gridDim.y) {
    int slot = b;
    if (slots) {
      slot = slots[b];
      if (slot < 0 || slot >= nstates) continue;
      bool later = false;
      for (int i = 0; i < b; ++i) later |= slots[i] == slot;
      if (later) continue;
    }
    float* at = states + static_cast<int64_t>(slot) * channels + c;
    float now = *at;
    for (int i = b; i < B; ++i) {
      if (i > b && (!slots || slots[i] != slot)) continue;
      float a, w;
      gate_of<FORM>(Elem<T>::load(row_of<T>(gate, i, h), j), a, w);
      now = fmaf(a, now, w * Elem<T>::load(row_of<T>(x, i, h), j));
      Elem<T>::store(row_of<T>(out, i, h), j, now);
    }
    *at = now;
  }
}

}  // namespace

#define RET_BY_FORM_AND_TYPE(kernel, ...)                                              \
  do {                                                                                 \
    if (dtype == 0) {                                                                  \
      if (form == 0) kernel<float, 0><<<grid, kThreads, 0, stream>>>(__VA_ARGS__);     \
      else kernel<float, 1><<<grid, kThreads, 0, stream>>>(__VA_ARGS__);               \
    } else {                                                                           \
      if (form == 0) kernel<uint16_t, 0><<<grid, kThreads, 0, stream>>>(__VA_ARGS__);  \
      else kernel<uint16_t, 1><<<grid, kThreads, 0, stream>>>(__VA_ARGS__);            \
    }                                                                                  \
  } while (0)

hipError_t launch_gated_recurrence(int form, int dtype, const View& x, const View& gate, const View& h,
                                   const Sequences& q, const float* state_in, float* state_out, void*,
                                   hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(plan_scan(q.S, q.H, q.max_len, q.d).blocks));
  RET_BY_FORM_AND_TYPE(recurrence_kernel, x, gate, h, q, state_in, state_out);
  return hipGetLastError();
}

hipError_t launch_gated_recurrence_backward(int form, int dtype, const View& grad_h, const View& x, const View& gate,
                                            const View& h, const View& grad_x, const View& grad_gate,
                                            const Sequences& q, const float* state_in, const float* grad_state_out,
                                            float* grad_state_in, void*, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(plan_scan(q.S, q.H, q.max_len, q.d).blocks));
  RET_BY_FORM_AND_TYPE(recurrence_backward_kernel, grad_h, x, gate, h, grad_x, grad_gate, q, state_in, grad_state_out,
                       grad_state_in);
  return hipGetLastError();
}

hipError_t launch_gated_recurrence_step(int form, int dtype, const View& x, const View& gate, const View& h, int B,
                                        int H, int d, float* states, int nstates, const int* slots,
                                        hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>((H * d + kThreads - 1) / kThreads), B < 65535 ? B : 65535);
  RET_BY_FORM_AND_TYPE(step_kernel, x, gate, h, B, H, d, states, nstates, slots);
  return hipGetLastError();
}

}  // namespace ret
