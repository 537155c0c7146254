// C ABI of the block operators (include/retention_block.h): argument
// validation and launches. Validation runs on the host, before any HIP call,
// and looks at pointers, sizes and strides only.
#include <cmath>
#include <cstdint>

#include "block.h"
#include "retention_block.h"

namespace {

using ret::NormArgs;
using ret::Sequences;
using ret::View;

constexpr int64_t kMaxSpan = int64_t{1} << 46;  // elements a view may span
constexpr int kMaxChannels = 1 << 20;           // d of the recurrence
constexpr int64_t kMaxTokenStride = int64_t{1} << 24;  // elements; offsets within a wave's tokens are 32-bit
constexpr int64_t kMaxThreads = int64_t{1} << 32;  // below which a launch's stay
constexpr int64_t kMaxStepChannels = int64_t{1} << 30;
constexpr int kMaxSequences = 1 << 20;

static_assert(RETENTION_H_F32 == ret::kWideH, "the launchers' flag is the ABI's");
int h_type(int dtype) { return dtype & RETENTION_H_F32 ? static_cast<int>(RET_F32) : dtype; }
int base_type(int dtype) { return dtype & ~RETENTION_H_F32; }

int status_of(hipError_t e) { return e == hipSuccess ? RET_OK : RET_ERR_HIP; }
bool valid_dtype(int dtype) { return dtype == RET_F32 || dtype == RET_BF16; }
int64_t elem_size(int dtype) { return dtype == RET_F32 ? 4 : 2; }
bool misaligned(const void* p, int64_t to) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(to) != 0; }

// The bytes [lo, hi) that a tensor spans. With a pitch it holds `width` bytes
// at lo and at multiples of the pitch from there, and none between.
struct Range {
  uintptr_t lo = 0, hi = 0;
  uintptr_t pitch = 0, width = 0;
};
Range range_of(const void* p, int64_t bytes) {
  Range r;
  if (p) {
    r.lo = reinterpret_cast<uintptr_t>(p);
    r.hi = r.lo + static_cast<uintptr_t>(bytes);
  }
  return r;
}
// Whether two tensors may share a byte: their ranges meet, and they are not
// columns of one larger tensor that lie side by side.
bool meet(const Range& a, const Range& b) {
  if (a.lo >= b.hi || b.lo >= a.hi) return false;
  if (a.pitch == 0 || a.pitch != b.pitch) return true;
  const uintptr_t ahead = b.lo >= a.lo ? (b.lo - a.lo) % a.pitch : (a.pitch - (a.lo - b.lo) % a.pitch) % a.pitch;
  return ahead < a.width || ahead + b.width > a.pitch;
}

// The byte ranges of a call's tensors; a null tensor's is empty and meets none.
struct Ranges {
  Range in[12], out[8];
  int nin = 0, nout = 0;
  void input(const Range& r) { in[nin++] = r; }
  void output(const Range& r) { out[nout++] = r; }
  bool clash() const {
    for (int i = 0; i < nout; ++i) {
      for (int j = 0; j < nin; ++j)
        if (meet(out[i], in[j])) return true;
      for (int j = 0; j < i; ++j)
        if (meet(out[i], out[j])) return true;
    }
    return false;
  }
};

int check_dims(int B, int H, int N, int d, int dtype) {
  if (B <= 0 || H <= 0 || N <= 0 || d <= 0 || !valid_dtype(dtype)) return RET_ERR_INVALID_ARG;
  if (static_cast<int64_t>(B) * H >= (int64_t{1} << 31) / N) return RET_ERR_UNSUPPORTED;
  return RET_OK;
}

// Checks a view of [B, H, N, d] elements of `dtype`, and that an output's
// elements lie apart; *out gets its strides (0 for sizes of 1), *range the
// bytes it spans. A null view is an error only where `required`.
int check_view(const retention_view_t* v, int B, int H, int N, int d, int dtype, bool required, bool is_output,
               View* out, Range* range) {
  *out = View{nullptr, 0, 0, 0};
  *range = Range{};
  if (!v || !v->data) return required ? RET_ERR_INVALID_ARG : RET_OK;
  const int64_t es = elem_size(dtype);
  if (misaligned(v->data, es)) return RET_ERR_INVALID_ARG;
  const int64_t size[3] = {B, H, N};
  const int64_t given[3] = {v->stride_b, v->stride_h, v->stride_n};
  int64_t stride[3], last = 0;
  for (int i = 0; i < 3; ++i) {
    stride[i] = size[i] > 1 ? given[i] : 0;
    if (stride[i] < 0) return RET_ERR_INVALID_ARG;
    if (stride[i] > kMaxSpan / size[i]) return RET_ERR_UNSUPPORTED;
    last += (size[i] - 1) * stride[i];
  }
  // Dimensions from the smallest stride up.
  int order[3] = {0, 1, 2};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (stride[order[j]] > stride[order[j + 1]]) {
        const int t = order[j];
        order[j] = order[j + 1];
        order[j + 1] = t;
      }
  if (is_output) {  // each stride must step over all that the smaller ones span
    int64_t span = d;
    for (int i : order) {
      if (size[i] == 1) continue;
      if (stride[i] < span) return RET_ERR_INVALID_ARG;
      span += (size[i] - 1) * stride[i];
    }
  }
  *out = View{static_cast<char*>(v->data), stride[0], stride[1], stride[2]};
  *range = range_of(v->data, (last + d) * es);
  // Dimensions that go on where the smaller ones end (heads of a token) widen
  // the columns; the pitch is the next stride, if it divides the others and
  // holds the columns.
  int64_t width = d, pitch = 0;
  for (int i : order) {
    if (stride[i] == 0) continue;  // adds no place
    if (pitch == 0 && stride[i] == width) width *= size[i];
    else if (pitch == 0) pitch = stride[i];
    else if (stride[i] % pitch != 0) return RET_OK;
  }
  if (pitch >= width) {
    range->pitch = static_cast<uintptr_t>(pitch * es);
    range->width = static_cast<uintptr_t>(width * es);
  }
  return RET_OK;
}

int check_norm(const retention_norm_t* norm, int64_t params, NormArgs* out, Ranges* ranges) {
  if (!norm || !std::isfinite(norm->eps) || norm->eps < 0.0f) return RET_ERR_INVALID_ARG;
  if (misaligned(norm->weight, 4) || misaligned(norm->bias, 4)) return RET_ERR_INVALID_ARG;
  *out = NormArgs{norm->eps, norm->rms != 0, norm->weight, norm->bias};
  ranges->input(range_of(norm->weight, params * 4));
  ranges->input(range_of(norm->bias, params * 4));
  return RET_OK;
}

int check_float_array(const float* p, int64_t n, Range* r) {
  if (misaligned(p, 4)) return RET_ERR_INVALID_ARG;
  *r = range_of(p, n * 4);
  return RET_OK;
}

// The largest of what the recurrence and its backward need in either form: one
// workspace serves them all. 0 blocks where a launch would be out of range.
ret::ScanPlan plan_any(int sequences, int H, int N, int max_len, bool packed, int d, int dtype) {
  ret::ScanPlan most{};
  for (int i = 0; i < 4; ++i) {
    const ret::ScanPlan p = ret::plan_scan(sequences, H, N, max_len, packed, d, dtype, i & 1, i >> 1);
    if (p.blocks >= kMaxThreads / 64 / p.waves) return ret::ScanPlan{};
    most.blocks = most.blocks > p.blocks ? most.blocks : p.blocks;
    most.bytes = most.bytes > p.bytes ? most.bytes : p.bytes;
  }
  return most;
}

// The checks the recurrence and its backward share.
int check_sequences(int B, int H, int N, int d, int form, int dtype, const int* cu, int sequences, int max_len,
                    void* workspace, size_t workspace_bytes, Sequences* q, Ranges* ranges) {
  const int st = check_dims(B, H, N, d, dtype);
  if (st != RET_OK) return st;
  if (form != RET_GATE_SIGMOID && form != RET_GATE_LOG) return RET_ERR_INVALID_ARG;
  if (sequences <= 0 || max_len <= 0) return RET_ERR_INVALID_ARG;
  if (cu ? B != 1 : (sequences != B || max_len != N)) return RET_ERR_INVALID_ARG;
  if (misaligned(cu, 4)) return RET_ERR_INVALID_ARG;
  if (d > kMaxChannels || (cu && sequences > kMaxSequences)) return RET_ERR_UNSUPPORTED;
  if (max_len > N) max_len = N;
  const ret::ScanPlan plan = plan_any(sequences, H, N, max_len, cu != nullptr, d, dtype);
  if (plan.blocks <= 0) return RET_ERR_UNSUPPORTED;
  if (plan.bytes > 0 && (!workspace || workspace_bytes < plan.bytes || misaligned(workspace, 8)))
    return RET_ERR_INVALID_ARG;
  *q = Sequences{sequences, H, N, d, max_len, cu};
  ranges->input(range_of(cu, (static_cast<int64_t>(sequences) + 1) * 4));
  ranges->output(plan.bytes > 0 ? range_of(workspace, static_cast<int64_t>(plan.bytes)) : Range{});
  return RET_OK;
}

bool far_tokens(const View& v) { return v.sn >= kMaxTokenStride; }

// Adds a state pair to the ranges: `to` may be `from` itself, not part of it.
int check_states(const float* from, const float* to, int64_t n, Ranges* ranges) {
  Range a, b;
  int st = check_float_array(from, n, &a);
  if (st == RET_OK) st = check_float_array(to, n, &b);
  if (st != RET_OK) return st;
  if (from != to) ranges->input(a);
  ranges->output(b);
  return RET_OK;
}

}  // namespace

extern "C" {

size_t retention_gated_recurrence_workspace_bytes(int sequences, int H, int N, int max_len, int packed, int d,
                                                  int dtype) {
  dtype = base_type(dtype);
  if (sequences <= 0 || max_len <= 0 || d > kMaxChannels || (packed && sequences > kMaxSequences)) return 0;
  if (!packed && max_len != N) return 0;
  if (check_dims(packed ? 1 : sequences, H, N, d, dtype) != RET_OK) return 0;
  const ret::ScanPlan plan = plan_any(sequences, H, N, max_len < N ? max_len : N, packed != 0, d, dtype);
  return plan.blocks > 0 ? plan.bytes : 0;
}

int retention_gated_recurrence(const retention_view_t* x, const retention_view_t* gate, const retention_view_t* h,
                               int B, int H, int N, int d, int form, int dtype, const float* state_in,
                               float* state_out, const int* cu_seqlens, int sequences, int max_len, void* workspace,
                               size_t workspace_bytes, void* stream) {
  Ranges ranges;
  Sequences q;
  const int given = dtype, h_dtype = h_type(dtype);
  dtype = base_type(dtype);
  int st = check_sequences(B, H, N, d, form, dtype, cu_seqlens, sequences, max_len, workspace, workspace_bytes, &q,
                           &ranges);
  if (st != RET_OK) return st;
  View vx, vg, vh;
  Range r;
  if ((st = check_view(x, B, H, N, d, dtype, true, false, &vx, &r)) != RET_OK) return st;
  ranges.input(r);
  if ((st = check_view(gate, B, H, N, d, dtype, true, false, &vg, &r)) != RET_OK) return st;
  ranges.input(r);
  if ((st = check_view(h, B, H, N, d, h_dtype, true, true, &vh, &r)) != RET_OK) return st;
  ranges.output(r);
  if (far_tokens(vx) || far_tokens(vg) || far_tokens(vh)) return RET_ERR_UNSUPPORTED;
  st = check_states(state_in, state_out, static_cast<int64_t>(sequences) * H * d, &ranges);
  if (st != RET_OK) return st;
  if (ranges.clash()) return RET_ERR_INVALID_ARG;
  return status_of(ret::launch_gated_recurrence(form, given, vx, vg, vh, q, state_in, state_out, workspace,
                                                static_cast<hipStream_t>(stream)));
}

int retention_gated_recurrence_backward(const retention_view_t* grad_h, const retention_view_t* x,
                                        const retention_view_t* gate, const retention_view_t* h,
                                        const retention_view_t* grad_x, const retention_view_t* grad_gate, int B,
                                        int H, int N, int d, int form, int dtype, const float* state_in,
                                        const float* grad_state_out, float* grad_state_in, const int* cu_seqlens,
                                        int sequences, int max_len, void* workspace, size_t workspace_bytes,
                                        void* stream) {
  Ranges ranges;
  Sequences q;
  const int given = dtype, h_dtype = h_type(dtype);
  dtype = base_type(dtype);
  int st = check_sequences(B, H, N, d, form, dtype, cu_seqlens, sequences, max_len, workspace, workspace_bytes, &q,
                           &ranges);
  if (st != RET_OK) return st;
  View in[4], out[2];
  const retention_view_t* given_in[4] = {grad_h, x, gate, h};
  const retention_view_t* given_out[2] = {grad_x, grad_gate};
  Range r;
  for (int i = 0; i < 4; ++i) {
    const bool required = i != 1 || form == RET_GATE_SIGMOID;
    st = check_view(given_in[i], B, H, N, d, i == 3 ? h_dtype : dtype, required, false, &in[i], &r);
    if (st != RET_OK) return st;
    ranges.input(r);
  }
  for (int i = 0; i < 2; ++i) {
    if ((st = check_view(given_out[i], B, H, N, d, dtype, true, true, &out[i], &r)) != RET_OK) return st;
    ranges.output(r);
  }
  for (const View& v : in)
    if (far_tokens(v)) return RET_ERR_UNSUPPORTED;
  if (far_tokens(out[0]) || far_tokens(out[1])) return RET_ERR_UNSUPPORTED;
  const int64_t states = static_cast<int64_t>(sequences) * H * d;
  if ((st = check_float_array(state_in, states, &r)) != RET_OK) return st;
  ranges.input(r);
  if ((st = check_states(grad_state_out, grad_state_in, states, &ranges)) != RET_OK) return st;
  if (ranges.clash()) return RET_ERR_INVALID_ARG;
  return status_of(ret::launch_gated_recurrence_backward(form, given, in[0], in[1], in[2], in[3], out[0], out[1], q,
                                                         state_in, grad_state_out, grad_state_in, workspace,
                                                         static_cast<hipStream_t>(stream)));
}

int retention_gated_recurrence_step(const retention_view_t* x, const retention_view_t* gate,
                                    const retention_view_t* h, int B, int H, int d, int form, int dtype,
                                    float* states, int nstates, const int* slots, void* stream) {
  int st = check_dims(B, H, 1, d, dtype);
  if (st != RET_OK) return st;
  if (form != RET_GATE_SIGMOID && form != RET_GATE_LOG) return RET_ERR_INVALID_ARG;
  if (!states || nstates <= 0 || (!slots && nstates < B) || misaligned(slots, 4)) return RET_ERR_INVALID_ARG;
  if (d > kMaxChannels || static_cast<int64_t>(H) * d > kMaxStepChannels) return RET_ERR_UNSUPPORTED;
  Ranges ranges;
  View vx, vg, vh;
  Range r;
  if ((st = check_view(x, B, H, 1, d, dtype, true, false, &vx, &r)) != RET_OK) return st;
  ranges.input(r);
  if ((st = check_view(gate, B, H, 1, d, dtype, true, false, &vg, &r)) != RET_OK) return st;
  ranges.input(r);
  if ((st = check_view(h, B, H, 1, d, dtype, true, true, &vh, &r)) != RET_OK) return st;
  ranges.output(r);
  if ((st = check_float_array(states, static_cast<int64_t>(nstates) * H * d, &r)) != RET_OK) return st;
  ranges.output(r);
  ranges.input(range_of(slots, static_cast<int64_t>(B) * 4));
  if (ranges.clash()) return RET_ERR_INVALID_ARG;
  return status_of(ret::launch_gated_recurrence_step(form, dtype, vx, vg, vh, B, H, d, states, nstates, slots,
                                                     static_cast<hipStream_t>(stream)));
}

int retention_gated_norm(const retention_view_t* o, const retention_view_t* gate, const retention_view_t* y, int B,
                         int H, int N, int d, int dtype, const retention_norm_t* norm, void* stream) {
  int st = check_dims(B, H, N, d, dtype);
  if (st != RET_OK) return st;
  if (d > RETENTION_MAX_DV || H > RETENTION_MAX_HEADS) return RET_ERR_UNSUPPORTED;
  Ranges ranges;
  NormArgs n;
  if ((st = check_norm(norm, static_cast<int64_t>(H) * d, &n, &ranges)) != RET_OK) return st;
  View vo, vg, vy;
  Range r;
  if ((st = check_view(o, B, H, N, d, dtype, true, false, &vo, &r)) != RET_OK) return st;
  ranges.input(r);
  if ((st = check_view(gate, B, H, N, d, dtype, false, false, &vg, &r)) != RET_OK) return st;
  ranges.input(r);
  if ((st = check_view(y, B, H, N, d, dtype, true, true, &vy, &r)) != RET_OK) return st;
  ranges.output(r);
  if (ranges.clash()) return RET_ERR_INVALID_ARG;
  return status_of(ret::launch_gated_norm(dtype, vo, vg, vy, B, H, N, d, n, static_cast<hipStream_t>(stream)));
}

size_t retention_gated_norm_backward_workspace_bytes(int B, int H, int N, int d, int dtype, int with_params) {
  if (check_dims(B, H, N, d, dtype) != RET_OK || d > RETENTION_MAX_DV || H > RETENTION_MAX_HEADS || !with_params)
    return 0;
  return ret::param_bytes(H, B * N, d, ret::kGatedNormSums, ret::kGatedBackGroups);
}

int retention_gated_norm_backward(const retention_view_t* grad_y, const retention_view_t* o,
                                  const retention_view_t* gate, const retention_view_t* grad_o,
                                  const retention_view_t* grad_gate, int B, int H, int N, int d, int dtype,
                                  const retention_norm_t* norm, float* grad_weight, float* grad_bias,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_dims(B, H, N, d, dtype);
  if (st != RET_OK) return st;
  if (d > RETENTION_MAX_DV || H > RETENTION_MAX_HEADS) return RET_ERR_UNSUPPORTED;
  Ranges ranges;
  NormArgs n;
  const int64_t params = static_cast<int64_t>(H) * d;
  if ((st = check_norm(norm, params, &n, &ranges)) != RET_OK) return st;
  View vdy, vo, vg, vdo, vdg;
  Range r;
  if ((st = check_view(grad_y, B, H, N, d, dtype, true, false, &vdy, &r)) != RET_OK) return st;
  ranges.input(r);
  if ((st = check_view(o, B, H, N, d, dtype, true, false, &vo, &r)) != RET_OK) return st;
  ranges.input(r);
  if ((st = check_view(gate, B, H, N, d, dtype, false, false, &vg, &r)) != RET_OK) return st;
  ranges.input(r);
  if ((st = check_view(grad_o, B, H, N, d, dtype, true, true, &vdo, &r)) != RET_OK) return st;
  ranges.output(r);
  if ((st = check_view(grad_gate, B, H, N, d, dtype, vg.data != nullptr, true, &vdg, &r)) != RET_OK) return st;
  if (vdg.data && !vg.data) return RET_ERR_INVALID_ARG;
  ranges.output(r);
  for (float* p : {grad_weight, grad_bias}) {
    if ((st = check_float_array(p, params, &r)) != RET_OK) return st;
    ranges.output(r);
  }
  if (grad_weight || grad_bias) {
    const size_t need = ret::param_bytes(H, B * N, d, ret::kGatedNormSums, ret::kGatedBackGroups);
    if (!workspace || workspace_bytes < need || misaligned(workspace, 4)) return RET_ERR_INVALID_ARG;
    ranges.output(range_of(workspace, static_cast<int64_t>(need)));
  }
  if (ranges.clash()) return RET_ERR_INVALID_ARG;
  return status_of(ret::launch_gated_norm_backward(dtype, vdy, vo, vg, vdo, vdg, B, H, N, d, n, grad_weight, grad_bias,
                                                   workspace, static_cast<hipStream_t>(stream)));
}

int retention_residual_norm(const retention_view_t* x, const retention_view_t* residual, const retention_view_t* y,
                            const retention_view_t* r, int B, int N, int D, int dtype, int stream_dtype,
                            const retention_norm_t* norm, const float* scale, float alpha, void* stream) {
  int st = check_dims(B, 1, N, D, dtype);
  if (st != RET_OK) return st;
  if (stream_dtype != dtype && stream_dtype != RET_F32) return RET_ERR_INVALID_ARG;
  if (!std::isfinite(alpha)) return RET_ERR_INVALID_ARG;
  if (D > RETENTION_MAX_MODEL_DIM) return RET_ERR_UNSUPPORTED;
  Ranges ranges;
  NormArgs n;
  if ((st = check_norm(norm, D, &n, &ranges)) != RET_OK) return st;
  View vx, vres, vy, vr;
  Range g, res;
  if ((st = check_view(x, B, 1, N, D, dtype, true, false, &vx, &g)) != RET_OK) return st;
  ranges.input(g);
  if ((st = check_view(residual, B, 1, N, D, stream_dtype, true, false, &vres, &res)) != RET_OK) return st;
  if ((st = check_view(y, B, 1, N, D, dtype, true, true, &vy, &g)) != RET_OK) return st;
  ranges.output(g);
  if ((st = check_view(r, B, 1, N, D, stream_dtype, true, true, &vr, &g)) != RET_OK) return st;
  ranges.output(g);
  // r may be the residual itself: a thread reads its values of a row before it
  // writes them, and no other takes them for its own.
  if (vr.data != vres.data || vr.sb != vres.sb || vr.sn != vres.sn) ranges.input(res);
  if ((st = check_float_array(scale, D, &g)) != RET_OK) return st;
  ranges.input(g);
  if (ranges.clash()) return RET_ERR_INVALID_ARG;
  return status_of(ret::launch_residual_norm(dtype, stream_dtype, vx, vres, vy, vr, B, N, D, n, scale, alpha,
                                             static_cast<hipStream_t>(stream)));
}

size_t retention_residual_norm_backward_workspace_bytes(int B, int N, int D, int dtype, int with_params) {
  if (check_dims(B, 1, N, D, dtype) != RET_OK || D > RETENTION_MAX_MODEL_DIM || !with_params) return 0;
  return ret::param_bytes(1, B * N, D, ret::kResidualNormSums, ret::residual_back_groups(D));
}

int retention_residual_norm_backward(const retention_view_t* grad_y, const retention_view_t* grad_r,
                                     const retention_view_t* r, const retention_view_t* x,
                                     const retention_view_t* residual, const retention_view_t* grad_x,
                                     const retention_view_t* grad_residual, int B,
                                     int N, int D, int dtype, int stream_dtype, const retention_norm_t* norm,
                                     const float* scale, float alpha, float* grad_scale, float* grad_weight,
                                     float* grad_bias, void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_dims(B, 1, N, D, dtype);
  if (st != RET_OK) return st;
  if (stream_dtype != dtype && stream_dtype != RET_F32) return RET_ERR_INVALID_ARG;
  if (!std::isfinite(alpha)) return RET_ERR_INVALID_ARG;
  if (D > RETENTION_MAX_MODEL_DIM) return RET_ERR_UNSUPPORTED;
  Ranges ranges;
  NormArgs n;
  if ((st = check_norm(norm, D, &n, &ranges)) != RET_OK) return st;
  View vdy, vdr, vr, vx, vres, vdx, vdres;
  Range g;
  if ((st = check_view(grad_y, B, 1, N, D, dtype, true, false, &vdy, &g)) != RET_OK) return st;
  ranges.input(g);
  if ((st = check_view(grad_r, B, 1, N, D, stream_dtype, false, false, &vdr, &g)) != RET_OK) return st;
  ranges.input(g);
  if ((st = check_view(residual, B, 1, N, D, stream_dtype, false, false, &vres, &g)) != RET_OK) return st;
  ranges.input(g);
  if ((st = check_view(r, B, 1, N, D, stream_dtype, !vres.data, false, &vr, &g)) != RET_OK) return st;
  ranges.input(g);
  if ((st = check_view(x, B, 1, N, D, dtype, grad_scale || vres.data, false, &vx, &g)) != RET_OK) return st;
  ranges.input(g);
  if ((st = check_view(grad_x, B, 1, N, D, dtype, false, true, &vdx, &g)) != RET_OK) return st;
  ranges.output(g);
  if ((st = check_view(grad_residual, B, 1, N, D, stream_dtype, true, true, &vdres, &g)) != RET_OK) return st;
  ranges.output(g);
  if ((st = check_float_array(scale, D, &g)) != RET_OK) return st;
  ranges.input(g);
  for (float* p : {grad_scale, grad_weight, grad_bias}) {
    if ((st = check_float_array(p, D, &g)) != RET_OK) return st;
    ranges.output(g);
  }
  if (grad_scale || grad_weight || grad_bias) {
    const size_t need = ret::param_bytes(1, B * N, D, ret::kResidualNormSums, ret::residual_back_groups(D));
    if (!workspace || workspace_bytes < need || misaligned(workspace, 4)) return RET_ERR_INVALID_ARG;
    ranges.output(range_of(workspace, static_cast<int64_t>(need)));
  }
  if (ranges.clash()) return RET_ERR_INVALID_ARG;
  return status_of(ret::launch_residual_norm_backward(dtype, stream_dtype, vdy, vdr, vr, vx, vres, vdx, vdres, B, N, D,
                                                      n, scale, alpha, grad_scale, grad_weight, grad_bias, workspace,
                                                      static_cast<hipStream_t>(stream)));
}

}  // extern "C"
