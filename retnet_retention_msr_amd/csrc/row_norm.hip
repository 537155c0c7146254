// Norms of a block and their gradients, a row at a time.
//
//   gated norm (per head): z = xhat w + b, y = z sw(g), sw(g) = g sigmoid(g)
//     dz = dy sw(g), dg = dy z sw'(g), sw'(g) = s (1 + g (1 - s)), s = sigmoid(g)
//   residual norm: r = alpha residual + scale x, y = xhat(r) w + b
// with xhat = (v - mean) rstd (layer form) or v rstd (rms form), and
//   dv = rstd (q - mean(q) - xhat mean(q xhat)), q the gradient of xhat
// (without mean(q) in the rms form). Parameter gradients are sums over rows.
//
// Every operator here reads its tensors once and writes its results once and
// is bound by HBM. A row is held in the registers of L lanes, at most 16
// values each: part of a wave for narrow heads (several rows to a wave), a
// wave up to 1024 values, a workgroup beyond. Its statistics are sums over
// registers, then lane exchanges, then, across waves, one exchange through
// LDS; the backward forms them again from the row it has to read anyway, so
// nothing but the forward's input is kept. Threads stay with their channels
// and go over the rows, holding the weights, and the parameters' sums in the
// backward, in registers; each workgroup leaves one row of partial sums, which
// a second kernel adds in a fixed order.
#include "block.h"
#include "gate.h"
#include "pack.h"

namespace ret {

namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------------------
// Sums over the L lanes of a row

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}

// The sum over each aligned group of L <= 64 lanes, in every lane: neighbours,
// pairs, fours (mirrored within 8), eights (mirrored within 16), then the
// 16-lane rows and the two halves exchanged.
template <int L>
__device__ __forceinline__ float lanes_sum(float x) {
  if constexpr (L >= 2) x += dpp<0xB1>(x);
  if constexpr (L >= 4) x += dpp<0x4E>(x);
  if constexpr (L >= 8) x += dpp<0x141>(x);
  if constexpr (L >= 16) x += dpp<0x140>(x);
  if constexpr (L >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (L >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return x;
}

// ---------------------------------------------------------------------------
// A thread's part of a row

// K chunks of V neighbouring channels, L threads side by side. With MASK the
// row may end anywhere: a chunk that crosses its end is moved back to end with
// it, its first lo[k] channels belonging to the neighbour (V of them, all, for
// a chunk past the end).
template <int L, int V, int K, bool MASK>
struct Part {
  static constexpr int E = V * K;
  int start[K], lo[K];
  __device__ __forceinline__ explicit Part(int lane, int d) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * L + lane) * V;
      start[k] = MASK && c > d - V ? d - V : c;
      lo[k] = !MASK ? 0 : c < d ? c - start[k] : V;
    }
  }
  __device__ __forceinline__ bool own(int k, int j) const { return !MASK || j >= lo[k]; }

  // Values of the row at p (0 for channels that are not the thread's own).
  template <typename T>
  struct Raw {
    typename Pack<T, V>::raw w[K];
  };
  template <typename T>
  __device__ __forceinline__ Raw<T> load(const T* p) const {
    Raw<T> r;
#pragma unroll
    for (int k = 0; k < K; ++k) r.w[k] = Pack<T, V>::load(p + start[k]);
    return r;
  }
  template <typename T>
  __device__ __forceinline__ void values(const Raw<T>& r, float (&x)[E]) const {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float v[V];
      Pack<T, V>::unpack(r.w[k], v);
#pragma unroll
      for (int j = 0; j < V; ++j) x[k * V + j] = own(k, j) ? v[j] : 0.0f;
    }
  }
  // Parameters at p, or `none`.
  __device__ __forceinline__ void params(const float* p, float none, float (&x)[E]) const {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float v[V];
      if (p) Pack<float, V>::unpack(Pack<float, V>::load(p + start[k]), v);
#pragma unroll
      for (int j = 0; j < V; ++j) x[k * V + j] = p ? v[j] : none;
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(T* p, const float (&x)[E]) const {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float v[V];
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = x[k * V + j];
      if (!MASK || lo[k] == 0) {
        Pack<T, V>::store(p + start[k], v);
      } else {
#pragma unroll
        for (int j = 1; j < V; ++j)
          if (j >= lo[k]) Elem<T>::store(p + start[k], j, v[j]);
      }
    }
  }
  // Puts what is the thread's own into the float row at p.
  __device__ __forceinline__ void put(float* p, const float (&x)[E]) const {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (own(k, j)) p[start[k] + j] = x[k * V + j];
  }
  // How many channels of the row wave `w` holds.
  static __device__ __forceinline__ int count(int w, int d) {
    int n = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int left = d - (k * L + w * 64) * V;
      n += left < 0 ? 0 : left < 64 * V ? left : 64 * V;
    }
    return n;
  }
};

// What the waves of a row exchange, in two sets used in turn: a fast wave
// writes a row's set while a slow one may still read the last row's.
template <int L>
struct RowShared {
  float4 part[2][L / 64 > 0 ? L / 64 : 1];
};

// Mean and 1 / deviation of the row v; with BACK also s1 = the mean of q and
// s2 = the mean of q xhat. Each wave takes its sums about its own mean:
//   M2 = sum M2_w + n_w (mean_w - mean)^2
//   sum q (v - mean) = sum over waves of C_w + Q_w (mean_w - mean)
// with Q_w the wave's sum of q and C_w that of q (v - mean_w), so that one
// exchange joins them, with nothing lost to a mean far from 0. q is 0 for
// channels that are not the thread's own.
template <bool BACK, int L, int V, int K, bool MASK>
__device__ __forceinline__ void row_stats(const float (&v)[V * K], const float (&q)[V * K],
                                          const Part<L, V, K, MASK>& part, int d, const NormArgs& n,
                                          RowShared<L>& shared, int turn, float& mean, float& rstd, float& s1,
                                          float& s2) {
  constexpr int E = V * K, W = L / 64, LW = L < 64 ? L : 64;
  const float inv = 1.0f / d;
  const int lane = threadIdx.x & 63, wave = L > 64 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
  float sum = 0.0f, m2 = 0.0f, Q = 0.0f, C = 0.0f;
  mean = 0.0f;
  if (!n.rms) {
#pragma unroll
    for (int e = 0; e < E; ++e) sum += v[e];
    sum = lanes_sum<LW>(sum);
    if constexpr (L > 64) {
      const int own = Part<L, V, K, MASK>::count(wave, d);
      mean = own > 0 ? sum / own : 0.0f;
    } else {
      mean = sum * inv;
    }
  }
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float e = part.own(k, j) ? v[k * V + j] - mean : 0.0f;
      m2 = fmaf(e, e, m2);
      if (BACK) {
        Q += q[k * V + j];
        C = fmaf(q[k * V + j], e, C);
      }
    }
  m2 = lanes_sum<LW>(m2);
  if (BACK) {
    Q = lanes_sum<LW>(Q);
    C = lanes_sum<LW>(C);
  }
  if constexpr (L > 64) {
    if (lane == 0) shared.part[turn][wave] = make_float4(sum, m2, Q, C);
    lds_only_barrier();
    const int w = lane % W;
    const float4 p = shared.part[turn][w];
    m2 = p.y;
    Q = p.z;
    C = p.w;
    if (!n.rms) {
      const int own = Part<L, V, K, MASK>::count(w, d);
      mean = lanes_sum<W>(p.x) * inv;
      const float off = own > 0 ? p.x / own - mean : 0.0f;
      m2 = fmaf(own * off, off, m2);
      C = fmaf(Q, off, C);
    }
    m2 = lanes_sum<W>(m2);
    if (BACK) {
      Q = lanes_sum<W>(Q);
      C = lanes_sum<W>(C);
    }
  }
  rstd = 1.0f / sqrtf(fmaf(m2, inv, n.eps));
  if (BACK) {
    s1 = n.rms ? 0.0f : Q * inv;
    s2 = C * rstd * inv;
  }
}

// The rows of a thread: row `first` of the batch's B * N, then every step-th.
struct RowWalk {
  int b, n, db, dn, N;
  __device__ __forceinline__ RowWalk(int first, int step, int N) : N(N) {
    b = first / N;
    n = first - b * N;
    db = step / N;
    dn = step - db * N;
  }
  __device__ __forceinline__ void next() {
    b += db;
    n += dn;
    if (n >= N) {
      n -= N;
      ++b;
    }
  }
};

template <typename T>
__device__ __forceinline__ T* at(const View& v, int b, int h, int n) {
  return reinterpret_cast<T*>(v.data) + b * v.sb + h * v.sh + n * v.sn;
}

// ---------------------------------------------------------------------------
// Gated norm

// Grid (parts, H), 256 / L rows of a head at a time. Bound by HBM: bf16,
// 8 x 16 x 8192 x 512 in 575-612 us over GPUs (5.3-5.6 TB/s).
template <typename T, int L, int V, int K, bool MASK>
__global__ void __launch_bounds__(kThreads)
gated_norm_kernel(View o, View gate, View y, int rows, int N, int d, NormArgs n) {
  constexpr int E = V * K, G = kThreads / L;
  __shared__ RowShared<L> shared;
  const int h = blockIdx.y, g = threadIdx.x / L;
  const Part<L, V, K, MASK> part(threadIdx.x % L, d);
  float w[E], b[E];
  part.params(n.weight ? n.weight + static_cast<int64_t>(h) * d : nullptr, 1.0f, w);
  part.params(n.bias ? n.bias + static_cast<int64_t>(h) * d : nullptr, 0.0f, b);
  const int step = gridDim.x * G;
  RowWalk row(blockIdx.x * G + g, step, N);
  for (int64_t base = blockIdx.x * G; base < rows; base += step, row.next()) {
    const bool live = base + g < rows;  // a group past the rows goes along on row 0
    const int rb = live ? row.b : 0, rn = live ? row.n : 0;
    const auto ow = part.load(at<const T>(o, rb, h, rn));
    auto gw = ow;
    if (gate.data) gw = part.load(at<const T>(gate, rb, h, rn));
    float x[E], gv[E], mean, rstd, s1, s2;
    part.values(ow, x);
    row_stats<false>(x, x, part, d, n, shared, 0, mean, rstd, s1, s2);
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = fmaf((x[e] - mean) * rstd, w[e], b[e]);
    if (gate.data) {
      part.values(gw, gv);
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] *= swish(gv[e]);
    }
    if (live) part.store(at<T>(y, rb, h, rn), x);
  }
}

// The workgroup's sums of SUMS parameters, from its G groups' registers, to
// its row of the partial sums; those whose bit is set in `wanted`.
template <int SUMS, int G, typename P>
__device__ __forceinline__ void leave_sums(const P& part, const float (&sums)[SUMS][P::E], float* to, int d,
                                           uint32_t wanted) {
  if constexpr (G == 1) {
#pragma unroll
    for (int s = 0; s < SUMS; ++s)
      if (wanted >> s & 1) part.put(to + static_cast<int64_t>(s) * d, sums[s]);
  } else {
    // One parameter at a time, to keep the LDS at 16 KiB.
    constexpr int width = kThreads * P::E / G;
    __shared__ float all[G][width];
#pragma unroll
    for (int s = 0; s < SUMS; ++s) {
      if (!(wanted >> s & 1)) continue;
      __syncthreads();
      part.put(all[threadIdx.x / (kThreads / G)], sums[s]);
      __syncthreads();
      for (int c = threadIdx.x; c < d; c += kThreads) {
        float v = 0.0f;
#pragma unroll
        for (int g = 0; g < G; ++g) v += all[g][c];
        to[static_cast<int64_t>(s) * d + c] = v;
      }
    }
  }
}

// Bound by HBM: bf16, 8 x 16 x 8192 x 512 in 934-1060 us over GPUs (5.1-5.7
// TB/s), the sums of the parameters (4 us) with it; 2 x 8 x 2048 x 512 in 33 us.
// The next row's loads are on their way while a row is worked on.
template <typename T, int L, int V, int K, bool MASK>
__global__ void __launch_bounds__(kThreads)
gated_norm_backward_kernel(View dy, View o, View gate, View d_o, View d_gate, int rows, int N, int d, NormArgs n,
                           float* partial, uint32_t wanted) {
  constexpr int E = V * K, G = kThreads / L;
  typedef Part<L, V, K, MASK> P;
  __shared__ RowShared<L> shared;
  const int h = blockIdx.y, g = threadIdx.x / L;
  const P part(threadIdx.x % L, d);
  float w[E], b[E], sums[kGatedNormSums][E];
  part.params(n.weight ? n.weight + static_cast<int64_t>(h) * d : nullptr, 1.0f, w);
  part.params(n.bias ? n.bias + static_cast<int64_t>(h) * d : nullptr, 0.0f, b);
#pragma unroll
  for (int e = 0; e < E; ++e) sums[0][e] = sums[1][e] = 0.0f;
  const int step = gridDim.x * G;
  RowWalk row(blockIdx.x * G + g, step, N);
  typename P::template Raw<T> ow, dw, gw;
  auto load = [&](bool live) {
    const int rb = live ? row.b : 0, rn = live ? row.n : 0;
    ow = part.load(at<const T>(o, rb, h, rn));
    dw = part.load(at<const T>(dy, rb, h, rn));
    if (gate.data) gw = part.load(at<const T>(gate, rb, h, rn));
  };
  load(blockIdx.x * G + g < rows);
  for (int64_t base = blockIdx.x * G; base < rows; base += step) {
    const bool live = base + g < rows;
    const int rb = live ? row.b : 0, rn = live ? row.n : 0;
    float x[E], dyv[E], q[E], gv[E], mean, rstd, s1, s2;
    part.values(ow, x);
    part.values(dw, dyv);
    if (gate.data) part.values(gw, gv);
    row.next();
    if (base + step < rows) load(base + step + g < rows);  // the next row comes while this one is worked on
    if (!live) {
#pragma unroll
      for (int e = 0; e < E; ++e) dyv[e] = 0.0f;
    }
    float slope[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {  // dyv is 0 for channels that are not the thread's own
      q[e] = dyv[e];
      if (gate.data) {
        float s, less;
        sigmoid_pair(gv[e], s, less);
        slope[e] = s * fmaf(gv[e], less, 1.0f);
        q[e] *= gv[e] * s;
      }
      sums[1][e] += q[e];
    }
    float qw[E];
#pragma unroll
    for (int e = 0; e < E; ++e) qw[e] = q[e] * w[e];
    row_stats<true>(x, qw, part, d, n, shared, 0, mean, rstd, s1, s2);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      x[e] = (x[e] - mean) * rstd;
      sums[0][e] = fmaf(q[e], x[e], sums[0][e]);
      if (gate.data) gv[e] = dyv[e] * fmaf(x[e], w[e], b[e]) * slope[e];
      q[e] = rstd * (qw[e] - s1 - x[e] * s2);
    }
    if (gate.data && live) part.store(at<T>(d_gate, rb, h, rn), gv);
    if (live) part.store(at<T>(d_o, rb, h, rn), q);
  }
  if (partial)
    leave_sums<kGatedNormSums, G, P>(
        part, sums, partial + (static_cast<int64_t>(h) * gridDim.x + blockIdx.x) * kGatedNormSums * d, d, wanted);
}

// out[k][head * d + c] = sum over parts of partial[head][part][k][c]: 32
// columns (a cache line) of a head to a workgroup, 8 threads a column, joined
// in a fixed order. Grid (columns / 32, sums, heads). 4 us for the 4.2 MB of
// 1024 parts over 8 heads of 512, 6 us for 25 MB of 512 parts of 4096: the parts
// are mostly in the caches still, the launch and two trips to memory remain.
__global__ void __launch_bounds__(kThreads)
param_sum_kernel(const float* partial, int parts, int sums, int d, float* out0, float* out1, float* out2) {
  constexpr int kCols = 32, kLots = kThreads / kCols;
  __shared__ float all[kLots][kCols];
  const int k = blockIdx.y, head = blockIdx.z;
  float* out = k == 0 ? out0 : k == 1 ? out1 : out2;
  if (!out) return;
  const int col = threadIdx.x % kCols, lot = threadIdx.x / kCols;
  const int c = blockIdx.x * kCols + col;
  float s = 0.0f;
  if (c < d) {
    const int64_t stride = static_cast<int64_t>(sums) * d;
    const float* p = partial + (static_cast<int64_t>(head) * parts * sums + k) * d + c;
#pragma unroll 16
    for (int q = lot; q < parts; q += kLots) s += p[q * stride];
  }
  all[lot][col] = s;
  __syncthreads();
  if (lot == 0 && c < d) {
    s = 0.0f;
#pragma unroll
    for (int q = 0; q < kLots; ++q) s += all[q][col];
    out[static_cast<int64_t>(head) * d + c] = s;
  }
}

hipError_t sum_params(const float* partial, int heads, int parts, int sums, int d, float* out0, float* out1,
                      float* out2, hipStream_t stream) {
  param_sum_kernel<<<dim3((d + 31) / 32, sums, heads), kThreads, 0, stream>>>(partial, parts, sums, d, out0, out1,
                                                                              out2);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Residual norm: a workgroup of max(256, L) threads, 256 / L rows at a time.

constexpr int threads_of(int L) { return L > kThreads ? L : kThreads; }

// A thread's parameters at p (null: never asked for): in registers while its
// values are few, else read again for each row (from the caches).
template <typename P>
struct Held {
  static constexpr bool kHold = P::E <= 8;
  const P& part;
  const float* p;
  float v[kHold ? P::E : 1];
  __device__ __forceinline__ Held(const P& part, const float* p) : part(part), p(p) {
    if constexpr (kHold) part.params(p, 0.0f, v);
  }
  __device__ __forceinline__ void get(float (&x)[P::E]) const {
    if constexpr (kHold) {
#pragma unroll
      for (int e = 0; e < P::E; ++e) x[e] = v[e];
    } else {
      part.params(p, 0.0f, x);
    }
  }
};

// Bound by HBM: bf16 with an fp32 stream and scale, 16384 x 4096 in 148 us (5.4
// TB/s).
template <typename T, typename TR, int L, int V, int K, bool MASK>
__global__ void __launch_bounds__(threads_of(L))
residual_norm_kernel(View x, View residual, View y, View r, int rows, int N, int D, NormArgs n, const float* scale,
                     float alpha) {
  constexpr int E = V * K, G = threads_of(L) / L;
  __shared__ RowShared<L> shared;
  const int g = threadIdx.x / L;
  typedef Part<L, V, K, MASK> P;
  const P part(threadIdx.x % L, D);
  const Held<P> scales(part, scale), weights(part, n.weight), biases(part, n.bias);
  const int step = gridDim.x * G;
  RowWalk row(blockIdx.x * G + g, step, N);
  int turn = 0;
  for (int64_t base = blockIdx.x * G; base < rows; base += step, row.next(), turn ^= 1) {
    const bool live = base + g < rows;
    const int rb = live ? row.b : 0, rn = live ? row.n : 0;
    const auto rw = part.load(at<const TR>(residual, rb, 0, rn));
    const auto xw = part.load(at<const T>(x, rb, 0, rn));
    float v[E], p[E], mean, rstd, s1, s2;
    part.values(xw, v);
    if (scale) {
      scales.get(p);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] *= p[e];
    }
    part.values(rw, p);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = fmaf(alpha, p[e], v[e]);
    if (live) part.store(at<TR>(r, rb, 0, rn), v);
    row_stats<false>(v, v, part, D, n, shared, turn, mean, rstd, s1, s2);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = (v[e] - mean) * rstd;
    if (n.weight) {
      weights.get(p);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] *= p[e];
    }
    if (n.bias) {
      biases.get(p);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] += p[e];
    }
    if (live) part.store(at<T>(y, rb, 0, rn), v);
  }
}

// A thread's running sums, in registers or, where those of a row's three
// tensors leave no room for them, in LDS of its own (4096 x 16384, whole
// backward: bf16 159 us against 197, fp32 343 against 525).
template <int E, bool LDS>
struct RunningSums {
  float v[E];
  __device__ __forceinline__ explicit RunningSums(float4*) {
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = 0.0f;
  }
  template <typename F>
  __device__ __forceinline__ void add(F term) {
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = term(e, v[e]);
  }
  __device__ __forceinline__ void get(float (&x)[E]) const {
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = v[e];
  }
};
template <int E>
struct RunningSums<E, true> {
  float4* at;  // E / 4 words of four, a workgroup's threads side by side
  __device__ __forceinline__ explicit RunningSums(float4* all) : at(all + threadIdx.x) {
#pragma unroll
    for (int k = 0; k < E / 4; ++k) at[k * blockDim.x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  template <typename F>
  __device__ __forceinline__ void add(F term) {
#pragma unroll
    for (int k = 0; k < E / 4; ++k) {
      float4 w = at[k * blockDim.x];
      w.x = term(4 * k, w.x);
      w.y = term(4 * k + 1, w.y);
      w.z = term(4 * k + 2, w.z);
      w.w = term(4 * k + 3, w.w);
      at[k * blockDim.x] = w;
    }
  }
  __device__ __forceinline__ void get(float (&x)[E]) const {
#pragma unroll
    for (int k = 0; k < E / 4; ++k) {
      const float4 w = at[k * blockDim.x];
      x[4 * k] = w.x;
      x[4 * k + 1] = w.y;
      x[4 * k + 2] = w.z;
      x[4 * k + 3] = w.w;
    }
  }
};

// The row is r or, with `residual`, formed again from it and x. Bound by HBM up
// to 8192 values a row: the case above 235 us with the parameters' sums (5.1
// TB/s), 8192 x 8192 222 us (5.4 TB/s). Wider rows take 16 values a thread in
// 1024 threads, two of their three sums in LDS; a CU then has one row at a time
// and the next one's loads wait for it, and 17 to 66 of its registers spill:
// 4096 x 16384 bf16 159 us (3.4 TB/s), fp32 343 us (4.7 TB/s). With a bf16 x and
// an fp32 stream 2 or 3 spill up to 4096 values a row (8 where the width is
// ragged).
template <typename T, typename TR, int L, int V, int K, bool MASK>
__global__ void __launch_bounds__(threads_of(L), (sizeof(T) == 2 && V * K <= 8) || L == 1024 ? 4 : 2)
residual_norm_backward_kernel(View dy, View dr, View r, View x, View residual, View dx, View dres, int rows, int N,
                              int D, NormArgs n, const float* scale, float alpha, float* partial, uint32_t wanted) {
  constexpr int E = V * K, G = threads_of(L) / L;
  constexpr bool kEarly = L <= 512;
  typedef Part<L, V, K, MASK> P;
  __shared__ RowShared<L> shared;
  const int g = threadIdx.x / L;
  const P part(threadIdx.x % L, D);
  const Held<P> scales(part, scale), weights(part, n.weight);
  constexpr bool kLds = L == 1024 && E > 8;
  __shared__ float4 held[2][kLds ? L * E / 4 : 1];
  RunningSums<E, kLds> sum0(held[0]), sum1(held[1]);
  RunningSums<E, false> sum2(nullptr);
  const int step = gridDim.x * G;
  RowWalk row(blockIdx.x * G + g, step, N);
  const View& from = residual.data ? residual : r;
  typename P::template Raw<TR> vw, sw;
  typename P::template Raw<T> gw, xw;
  auto load = [&](bool live) {
    const int rb = live ? row.b : 0, rn = live ? row.n : 0;
    vw = part.load(at<const TR>(from, rb, 0, rn));
    if (x.data) xw = part.load(at<const T>(x, rb, 0, rn));
    gw = part.load(at<const T>(dy, rb, 0, rn));
    if (dr.data) sw = part.load(at<const TR>(dr, rb, 0, rn));
  };
  load(blockIdx.x * G + g < rows);
  int turn = 0;
  for (int64_t base = blockIdx.x * G; base < rows; base += step, turn ^= 1) {
    const bool live = base + g < rows;
    const int rb = live ? row.b : 0, rn = live ? row.n : 0;
    float v[E], q[E], p[E], mean, rstd, s1, s2;
    part.values(vw, v);
    part.values(gw, q);
    const auto sw_now = sw;
    const auto xw_now = xw;
    row.next();
    // The next row comes while this one is worked on, where registers allow.
    if (kEarly && base + step < rows) load(base + step + g < rows);
    if (residual.data) {
      float b[E];
      part.values(xw_now, b);
      if (scale) {
        scales.get(p);
#pragma unroll
        for (int e = 0; e < E; ++e) b[e] *= p[e];
      }
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = fmaf(alpha, v[e], b[e]);
    }
    if (!live) {
#pragma unroll
      for (int e = 0; e < E; ++e) q[e] = 0.0f;
    }
    float qw[E];
#pragma unroll
    for (int e = 0; e < E; ++e) qw[e] = q[e];
    if (n.weight) {
      weights.get(p);
#pragma unroll
      for (int e = 0; e < E; ++e) qw[e] *= p[e];
    }
    row_stats<true>(v, qw, part, D, n, shared, turn, mean, rstd, s1, s2);
#pragma unroll
    for (int e = 0; e < E; ++e) {  // q is 0 for channels that are not the thread's own
      v[e] = (v[e] - mean) * rstd;
      sum2.v[e] += q[e];
    }
    if (!kLds || partial) sum1.add([&](int e, float s) { return fmaf(q[e], v[e], s); });
#pragma unroll
    for (int e = 0; e < E; ++e) q[e] = rstd * (qw[e] - s1 - v[e] * s2);
    if (dr.data) {
      part.values(sw_now, p);
#pragma unroll
      for (int e = 0; e < E; ++e) q[e] += p[e];
    }
    if (x.data) {
      part.values(xw_now, p);  // 0 for channels that are not the thread's own
      if (!kLds || partial) sum0.add([&](int e, float s) { return live ? fmaf(q[e], p[e], s) : s; });
    }
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = alpha * q[e];
    if (live) part.store(at<TR>(dres, rb, 0, rn), v);
    if (dx.data) {
      if (scale) {
        scales.get(p);
#pragma unroll
        for (int e = 0; e < E; ++e) q[e] *= p[e];
      }
      if (live) part.store(at<T>(dx, rb, 0, rn), q);
    }
    if (!kEarly && base + step < rows) load(base + step + g < rows);
  }
  if (partial) {
    float sums[kResidualNormSums][E];
    sum0.get(sums[0]);
    sum1.get(sums[1]);
    sum2.get(sums[2]);
    leave_sums<kResidualNormSums, G, P>(part, sums,
                                        partial + static_cast<int64_t>(blockIdx.x) * kResidualNormSums * D, D,
                                        wanted);
  }
}

// ---------------------------------------------------------------------------
// Which instance takes a width: the fewest lanes that hold it at 8 values each
// (one access of bf16, two of fp32; four for narrow fp32 heads, 16 where 8
// would need more than a wave for a row up to 1024 or more than a workgroup),
// one value a lane for rows shorter than an access. Rows of 4096 at 16 values in
// 256 threads against 8 in 512, forward with an fp32 stream: 162 and 152 us at
// 16384 rows.

#define RET_ROW(kernel, L, V, K, ...)                                                \
  do {                                                                               \
    if (d == L * V * K) kernel(L, V, K, false, __VA_ARGS__);                         \
    else kernel(L, V, K, true, __VA_ARGS__);                                         \
    return hipGetLastError();                                                        \
  } while (0)

#define RET_HEAD_ROWS(kernel, V, ...)                                                \
  do {                                                                               \
    if (d < V) RET_ROW(kernel, 8, 1, 1, __VA_ARGS__);                                \
    if (d <= 8 * V) RET_ROW(kernel, 8, V, 1, __VA_ARGS__);                           \
    if (d <= 16 * V) RET_ROW(kernel, 16, V, 1, __VA_ARGS__);                         \
    if (d <= 32 * V) RET_ROW(kernel, 32, V, 1, __VA_ARGS__);                         \
    if (d <= 64 * V) RET_ROW(kernel, 64, V, 1, __VA_ARGS__);                         \
    if (V < 8 && d <= 128 * V) RET_ROW(kernel, 64, V, (V < 8 ? 2 : 1), __VA_ARGS__); \
    RET_ROW(kernel, 64, V, 16 / V, __VA_ARGS__);                                     \
  } while (0)

#define RET_MODEL_ROWS(kernel, V, ...)                                               \
  do {                                                                               \
    if (d < V) RET_ROW(kernel, 64, 1, 1, __VA_ARGS__);                               \
    if (d <= 64 * V) RET_ROW(kernel, 64, V, 1, __VA_ARGS__);                         \
    if (d <= 1024) RET_ROW(kernel, 64, V, 16 / V, __VA_ARGS__);                      \
    if (d <= 2048) RET_ROW(kernel, 256, V, 8 / V, __VA_ARGS__);                      \
    if (d <= 4096) RET_ROW(kernel, 512, V, 8 / V, __VA_ARGS__);                      \
    if (d <= 8192) RET_ROW(kernel, 1024, V, 8 / V, __VA_ARGS__);                     \
    RET_ROW(kernel, 1024, V, 16 / V, __VA_ARGS__);                                   \
  } while (0)

// Rows that a workgroup of a launch over rows of d values takes at a time.
int rows_at_once(int d, int dtype, bool heads) {
  const int V = dtype == 0 ? 4 : 8;
  int L = 64;
  if (heads) {
    L = d < V ? 8 : d <= 8 * V ? 8 : d <= 16 * V ? 16 : d <= 32 * V ? 32 : 64;
  } else if (d > 1024) {
    return 1;
  }
  return kThreads / L;
}

}  // namespace

hipError_t launch_gated_norm(int dtype, const View& o, const View& gate, const View& y, int B, int H, int N, int d,
                             const NormArgs& norm, hipStream_t stream) {
  const int rows = B * N;
  const dim3 grid(norm_parts(H, rows, rows_at_once(d, dtype, true), kForwardGroups), H);
#define RET_LAUNCH(L, V, K, MASK, T) \
  gated_norm_kernel<T, L, V, K, MASK><<<grid, kThreads, 0, stream>>>(o, gate, y, rows, N, d, norm)
  if (dtype == 0) RET_HEAD_ROWS(RET_LAUNCH, 4, float);
  RET_HEAD_ROWS(RET_LAUNCH, 8, uint16_t);
#undef RET_LAUNCH
}

namespace {

hipError_t gated_norm_backward(int dtype, const View& dy, const View& o, const View& gate, const View& d_o,
                               const View& d_gate, int parts, int H, int rows, int N, int d, const NormArgs& norm,
                               float* partial, uint32_t wanted, hipStream_t stream) {
  const dim3 grid(parts, H);
#define RET_LAUNCH(L, V, K, MASK, T)                                                                             \
  gated_norm_backward_kernel<T, L, V, K, MASK><<<grid, kThreads, 0, stream>>>(dy, o, gate, d_o, d_gate, rows, N, \
                                                                              d, norm, partial, wanted)
  if (dtype == 0) RET_HEAD_ROWS(RET_LAUNCH, 4, float);
  RET_HEAD_ROWS(RET_LAUNCH, 8, uint16_t);
#undef RET_LAUNCH
}

hipError_t residual_norm_backward(int dtype, int stream_dtype, const View& dy, const View& dr, const View& r,
                                  const View& x, const View& residual, const View& dx, const View& dres, int parts,
                                  int rows, int N, int d, const NormArgs& norm, const float* scale, float alpha,
                                  float* partial, uint32_t wanted, hipStream_t stream) {
#define RET_LAUNCH(L, V, K, MASK, T, TR)                                                              \
  residual_norm_backward_kernel<T, TR, L, V, K, MASK><<<parts, threads_of(L), 0, stream>>>(           \
      dy, dr, r, x, residual, dx, dres, rows, N, d, norm, scale, alpha, partial, wanted)
  if (dtype == 0) RET_MODEL_ROWS(RET_LAUNCH, 4, float, float);
  if (stream_dtype == 0) RET_MODEL_ROWS(RET_LAUNCH, 8, uint16_t, float);
  RET_MODEL_ROWS(RET_LAUNCH, 8, uint16_t, uint16_t);
#undef RET_LAUNCH
}

}  // namespace

hipError_t launch_gated_norm_backward(int dtype, const View& grad_y, const View& o, const View& gate,
                                      const View& grad_o, const View& grad_gate, int B, int H, int N, int d,
                                      const NormArgs& norm, float* grad_weight, float* grad_bias, void* workspace,
                                      hipStream_t stream) {
  const int rows = B * N, at_once = rows_at_once(d, dtype, true);
  const int parts = norm_parts(H, rows, at_once, gated_back_groups(H, rows, at_once));
  float* partial = grad_weight || grad_bias ? static_cast<float*>(workspace) : nullptr;
  const hipError_t e =
      gated_norm_backward(dtype, grad_y, o, gate, grad_o, grad_gate, parts, H, rows, N, d, norm, partial,
                          (grad_weight ? 1u : 0u) | (grad_bias ? 2u : 0u), stream);
  if (e != hipSuccess || !partial) return e;
  return sum_params(partial, H, parts, kGatedNormSums, d, grad_weight, grad_bias, nullptr, stream);
}

hipError_t launch_residual_norm(int dtype, int stream_dtype, const View& x, const View& residual, const View& y,
                                const View& r, int B, int N, int d, const NormArgs& norm, const float* scale,
                                float alpha, hipStream_t stream) {
  const int rows = B * N, parts = norm_parts(1, rows, rows_at_once(d, dtype, false), kForwardGroups);
#define RET_LAUNCH(L, V, K, MASK, T, TR)                                                                          \
  residual_norm_kernel<T, TR, L, V, K, MASK><<<parts, threads_of(L), 0, stream>>>(x, residual, y, r, rows, N, d, \
                                                                                  norm, scale, alpha)
  if (dtype == 0) RET_MODEL_ROWS(RET_LAUNCH, 4, float, float);
  if (stream_dtype == 0) RET_MODEL_ROWS(RET_LAUNCH, 8, uint16_t, float);
  RET_MODEL_ROWS(RET_LAUNCH, 8, uint16_t, uint16_t);
#undef RET_LAUNCH
}

hipError_t launch_residual_norm_backward(int dtype, int stream_dtype, const View& grad_y, const View& grad_r,
                                         const View& r, const View& x, const View& residual, const View& grad_x,
                                         const View& grad_residual, int B, int N, int d, const NormArgs& norm,
                                         const float* scale, float alpha, float* grad_scale, float* grad_weight,
                                         float* grad_bias, void* workspace, hipStream_t stream) {
  const int rows = B * N, parts = norm_parts(1, rows, rows_at_once(d, dtype, false), residual_back_groups(d));
  float* partial = grad_scale || grad_weight || grad_bias ? static_cast<float*>(workspace) : nullptr;
  View xs = x;
  if (!grad_scale && !residual.data) xs.data = nullptr;
  const uint32_t wanted = (grad_scale ? 1u : 0u) | (grad_weight ? 2u : 0u) | (grad_bias ? 4u : 0u);
  const hipError_t e = residual_norm_backward(dtype, stream_dtype, grad_y, grad_r, r, xs, residual, grad_x,
                                              grad_residual, parts, rows, N, d, norm, scale, alpha, partial, wanted,
                                              stream);
  if (e != hipSuccess || !partial) return e;
  return sum_params(partial, 1, parts, kResidualNormSums, d, grad_scale, grad_weight, grad_bias, stream);
}

}  // namespace ret
