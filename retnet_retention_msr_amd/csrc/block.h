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

// Planning of a recurrence call: a pure function of the sizes. A unit is a
// sequence's (or head's) slab of kScanChannels channels; it is cut into tiles
// of `rows` tokens, one workgroup of `waves` waves of `wave_rows` tokens each.
// With more than one tile the workspace holds a status word and, per unit, a
// ticket and, per tile and channel, what the tile passes on (recurrence.hip). Lanes take `vec`
// channels, or one where the whole row is shorter: four of them, 16 bytes of
// fp32 and 8 of bf16, and in bf16's backward eight. A lane then holds fewer
// tokens, and more lanes' folds have to be joined (24 exchanges of three words
// against 8): forward, bf16, us at four and at eight: 8 x 8192 x 4096 301 and
// 305, 16 heads x 65536 x 128 179 and 185, 2 x 2048 x 2048 15.3 and 17.1. The
// backward's six tensors in pieces of 8 bytes cost more than that: 655 at four
// and 619 at eight (8 x 8192 x 4096, sigmoid form).
constexpr int kScanChannels = 64;
constexpr uint32_t kXcds = 8, kXcdUnits = 9;
constexpr int kScanMaxWaves = 8;
constexpr size_t kScanStatusBytes = 256;  // of the workspace: the status word, then nothing
// Tokens of a wave: forward 32 against 16, bf16, 302 us against 320 at 8 x 8192 x
// 4096, 157 against 187 at 4 x 8192 x 4096 in the log form. The sigmoid form's
// backward reads four tensors; waves of 16 tokens let it hold them in 128
// registers, four waves to a SIMD: 620 us at 8 x 8192 x 4096 against 987 with
// 32, of which 49 registers spill. 8 where a lane has one channel, so that a
// short row's tile stays in registers.
constexpr int kScanRows = 32;
constexpr int kScanSigmoidBackRows = 16;
constexpr int kScanNarrowRows = 8;
struct ScanPlan {
  int vec, waves, wave_rows, rows;
  int64_t units, tiles;  // tiles of the longest sequence
  int64_t slots;         // tiles of a slab over all sequences: the workspace's places
  bool folds;            // whether tiles pass on their folds too, or their states alone
  int64_t blocks;        // workgroups of the launch
  size_t bytes;          // workspace
};
// The tiles of S packed sequences in N tokens have the slots floor(first token
// / rows) + s + tile: no two share one, and there are at most N / rows + S,
// however long the longest may be.
// Workgroups of four waves where there are many units, of eight where there
// are few. With many, most of the tiles in flight belong to different units
// and wait for none of the others, and the smaller workgroups keep loads and
// stores of different ones side by side; with few, the tiles of a unit wait
// for one another, and half as many of them, twice as long, wait less. Forward,
// bf16, us at four and at eight: 512 units (8 x 8192 x 4096) 302 and 338, 256
// units (4 x 8192 x 4096) 154 and 148, 32 units (65536 x 2048) 194 and 184, 4
// units (32768 x 256) 34 and 24. Backward, log form: 240 units (15 x 4096 x
// 1024) 130 and 132, 128 units 77 and 78, 32 units (65536 x 2048) 300 and 291,
// 16 units (8192 x 1024) 32 and 26. The tiles of a sequence are
// equally long: 130 tokens as two of three waves, not of four and one, 95 us
// against 116 at 240 x 130 x 2048.
// With many units a tile waits for its predecessor's state alone: it is mostly
// there, and the folds' words would have to be filled, written and read (8 x
// 8192 x 4096: 302 us against 320). Packed sequences always publish folds: they may be one long
// sequence and many empty ones.
constexpr int64_t kScanManyUnits = 256;
// Workgroups that start for n units of one tile: rounded up where they are
// shared out among the XCDs in runs.
#ifdef __HIPCC__
__host__ __device__
#endif
inline uint32_t scan_round(uint32_t n) {
  return n % kXcds && n < kXcdUnits ? n : (n + kXcds - 1) / kXcds * kXcds;
}
inline ScanPlan plan_scan(int S, int H, int N, int max_len, bool packed, int d, int dtype, bool backward, int form) {
  ScanPlan p{};
  p.waves = 1;
  p.vec = dtype != 0 && backward ? 8 : 4;
  if (d < p.vec) p.vec = 1;
  const int64_t columns = static_cast<int64_t>(H) * ((d + kScanChannels - 1) / kScanChannels);
  if (columns > (int64_t{1} << 30)) {
    p.blocks = columns;  // beyond any launch, and the products below
    return p;
  }
  p.units = S * columns;
  p.wave_rows = p.vec == 1 ? kScanNarrowRows : backward && form == 0 ? kScanSigmoidBackRows : kScanRows;
  const int64_t most = p.units >= kScanManyUnits ? kScanMaxWaves / 2 : kScanMaxWaves;
  const int64_t waves = (static_cast<int64_t>(max_len) + p.wave_rows - 1) / p.wave_rows;
  const int64_t cut = (waves + most - 1) / most;
  p.waves = static_cast<int>((waves + cut - 1) / cut);
  p.rows = p.waves * p.wave_rows;
  p.tiles = (static_cast<int64_t>(max_len) + p.rows - 1) / p.rows;
  p.slots = packed && p.tiles > 1 ? N / p.rows + S : p.tiles * S;
  const int64_t together = packed && p.tiles > 1 ? columns : p.units;
  if (together > (int64_t{1} << 30)) {
    p.blocks = together;
    return p;
  }
  p.blocks = int64_t{scan_round(static_cast<uint32_t>(together))} * (columns * p.slots / together);
  p.folds = packed || p.units < kScanManyUnits;
  if (p.tiles > 1)
    p.bytes = kScanStatusBytes + (static_cast<size_t>(p.units) * 4 + 255) / 256 * 256 +
              static_cast<size_t>(columns) * p.slots * kScanChannels * (p.folds ? 12 : 4);
  return p;
}
// In the dtype of the launches over sequences: h is fp32, the rest of dtype.
constexpr int kWideH = 0x100;
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
// Workgroups of a norm's launch, per head: as many as the rows give at
// `at_once` rows each, at most `groups` over all heads.
constexpr int kForwardGroups = 4096;
inline int norm_parts(int heads, int rows, int at_once, int groups) {
  const int want = (rows - 1) / at_once + 1, most = (groups + heads - 1) / heads;
  return want < most ? want : most;
}
// A workgroup of the backward should go over enough rows that its partial sums
// do not count: 8 turns at least, and 512 workgroups at least. Up to 4096
// where there are rows enough: the workgroups at work then lie in fewer heads.
constexpr int kGatedBackGroups = 4096;
inline int gated_back_groups(int heads, int rows, int at_once) {
  const int64_t turns = static_cast<int64_t>(heads) * ((rows - 1) / at_once + 1) / 8;
  return turns < 512 ? 512 : turns < kGatedBackGroups ? static_cast<int>(turns) : kGatedBackGroups;
}
// As many workgroups as are at work at once: four of 256 threads to a CU, two
// of 512, one of 1024 (8192 x 8192 with an fp32 stream 222 us, with twice as
// many 236: each leaves a row of partial sums).
constexpr int kResidualBackGroups = 1024;
inline int residual_back_groups(int d) {
  return d <= 2048 ? kResidualBackGroups : d <= 4096 ? kResidualBackGroups / 2 : kResidualBackGroups / 4;
}
// Bytes of the backward's partial sums: a row of `sums` times d floats for
// each of its workgroups (whatever the rows a workgroup takes at a time).
inline size_t param_bytes(int heads, int rows, int d, int sums, int groups) {
  return static_cast<size_t>(heads) * norm_parts(heads, rows, 1, groups) * sums * d * sizeof(float);
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
// grad_r.data, x.data and grad_x.data may be nullptr; with residual.data the
// row is formed from residual and x and r.data may be nullptr.
hipError_t launch_residual_norm_backward(int dtype, int stream_dtype, const View& grad_y, const View& grad_r,
                                         const View& r, const View& x, const View& residual, const View& grad_x,
                                         const View& grad_residual, int B, int N, int D, const NormArgs& norm,
                                         const float* scale, float alpha, float* grad_scale, float* grad_weight,
                                         float* grad_bias, void* workspace, hipStream_t stream);

}  // namespace ret
