// Gated linear recurrence per channel, its backward and its single token.
//
//   sigmoid form: a = 1 / (1 + e^-g), h_t = a_t h_{t-1} + (1 - a_t) x_t
//   log form:     a = e^g,            h_t = a_t h_{t-1} + x_t
// Backward, from the last token: w_t = a_t (dh_t + w_{t+1}) carries what
// h_{t-1} receives, u_t = dh_t + w_{t+1} is the whole gradient of h_t;
//   sigmoid form: dx = (1 - a) u, dg = a (1 - a) (h_{t-1} - x_t) u
//   log form:     dx = u,         dg = a h_{t-1} u
//
// Both directions are the linear recurrence y_t = a_t y_{t-1} + b_t (backward:
// y = w, b = a dh, tokens taken from the last), bound by HBM: 3 values per
// token and channel forward, 5 or 6 backward, about 10 flops each. A workgroup
// takes a tile of tokens of 64 channels, reads it once into registers and
// writes its outputs once; what the tokens before it contribute reaches it
// through a few words per tile:
//   - a lane holds V neighbouring channels (one access, whatever its alignment;
//     where d is no multiple of V the last lane's is moved back to end with the
//     row) of R = E / V consecutive tokens, and folds them into
//     (A, Y): y_out = A y_in + Y; pairs of folds join by
//     (A1, Y1) then (A2, Y2) = (A1 A2, A2 Y1 + Y2). Beside A goes M = A - 1,
//     formed from the tokens' 1 - a without A's rounding, M = M1 + M2 A1:
//     where A is near 1 the carry into the next tile is y_in + (M y_in + Y).
//     With A itself, rounded in steps of 2^-24, a channel with a memory of L
//     tokens would be off by up to L 2^-25 (1.7e-3 of h at 65536 tokens of
//     constant gates, 2e-6 so). Within a tile the steps of A y_in + Y are few:
//     a lane's A near 1 is taken from its M;
//   - the V groups of lanes that hold the same channels at consecutive tokens
//     join theirs through lane exchanges, the waves of the workgroup theirs
//     through LDS;
//   - the carry into the tile is the finished state of the tile before it or,
//     with few units, where the tiles in flight are of the same sequences, the
//     nearest finished state run through the folds published since; then the
//     tile's own finished state is published. Tiles of a unit are handed out by
//     a ticket, in order, so every tile that is waited for is already running,
//     and tile 0 waits for none;
//   - each lane then runs its tokens again from its carry, which is in order
//     and in fp32, and rounds its outputs once.
// A gate of -inf (a reset) forgets the state before it whatever it holds, and
// one of +inf in the sigmoid form passes over whatever x holds, where the
// formulas' products have 0 times infinity or NaN. A wave in which a lane may
// hold a reset (sigmoid form: a decay that is 0, log form: gates whose sum is
// -inf), or in the sigmoid form a token that is passed over (forward: a Y that is
// not finite, backward: a 1 - a of 0), takes its tokens a second time, looking at
// each (`special`); the others are spared that: without either kind of token the
// products do what they should. A fold with a reset in it is marked by M = NaN
// with A = 0; a decay that is 0 in fp32 alone is no reset, and an infinite state
// stays infinite or becomes NaN.
// Published words hold their own "not there yet" value (all ones, written by
// scan_fill_kernel before each launch, 1 to 6 us), so one relaxed access is
// enough.
#include "block.h"
#include "gate.h"
#include "pack.h"

#include <type_traits>

namespace ret {

namespace {

constexpr int64_t kScanCacheBytes = int64_t{200} << 20;  // of the 256 MiB Infinity Cache

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

// The gate that gives a decay of 1.
template <int FORM>
constexpr float kKeepGate = FORM == 0 ? __builtin_inff() : 0.0f;

// The decay of a gate value, and 1 less it.
template <int FORM>
__device__ __forceinline__ void gate_of(float g, float& a, float& c) {
  if (FORM == 0) sigmoid_pair(g, a, c);
  else exp_pair(g, a, c);
}

// A token's decay a, in the sigmoid form with 1 - a in c.
template <int FORM>
__device__ __forceinline__ void token_decay(float g, float& a, float& c) {
  if (FORM == 0) sigmoid_pair(g, a, c);
  else a = __builtin_amdgcn_exp2f(kLog2e * g);
}
// In a special wave: 0 is kept for resets.
__device__ __forceinline__ float mark_token(float g, float a) {
  return a == 0.0f && g != -__builtin_inff() ? __uint_as_float(1u) : a;
}
// A lane's A and M with its token i. In the log form A is the sum of the gates
// until lane_decays(): one exponential and one series a lane, not one a token.
template <int FORM>
__device__ __forceinline__ void lane_decay(int i, float g, float a, float c, float& A, float& M) {
  if (FORM == 0) {
    M = i ? fmaf(-c, A, M) : -c;
    A = i ? A * a : a;
  } else {
    A = i ? A + g : g;
  }
}
// Returns whether the lane may hold a reset (in the sigmoid form also where a
// product of decays above 0 has become 0).
template <int FORM, int V>
__device__ __forceinline__ bool lane_decays(float (&A)[V], float (&M)[V]) {
  bool odd = false;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    odd |= !(A[j] > (FORM == 0 ? 0.0f : -__builtin_inff()));
    if (FORM == 1) {
      exp_pair(A[j], A[j], M[j]);
      M[j] = -M[j];
    }
    A[j] = M[j] >= -0.5f ? 1.0f + M[j] : A[j];  // one rounding, not one a token
  }
  return odd;
}
// Whether one of a lane's decays is 0 (and not -0, which stands for 1 where it
// is held as its distance from 1).
template <int R, int V>
__device__ __forceinline__ bool any_zero(const float (&a)[R][V]) {
  bool zero = false;
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) zero |= __float_as_uint(a[i][j]) == 0;
  return zero;
}
// Marks the channels whose bit is set in `resets`.
template <int V>
__device__ __forceinline__ void mark_resets(uint32_t resets, float (&A)[V], float (&M)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (!(resets >> j & 1)) continue;
    A[j] = 0.0f;
    M[j] = __builtin_nanf("");
  }
}
__device__ __forceinline__ bool resets(float A, float M) { return A == 0.0f && M != M; }
__device__ __forceinline__ bool finite(float x) { return __builtin_fabsf(x) < __builtin_inff(); }

// The workspace of a launch with more than one tile. A column is a head's slab;
// the tiles of its sequences have the slots s * tiles + tile, or, packed,
// floor(first token / rows) + s + tile, which no two of them share.
struct ScanWords {
  uint32_t* status;  // 0 where a wait was given up
  uint32_t* ticket;  // [units], from all ones up
  uint32_t* state;   // [columns][slots][64]: the state after the tile
  uint64_t* fold;    // [columns][slots][64]: Y, decay_word(A, M); null: states alone
  int64_t slots;
};

__global__ void __launch_bounds__(256) scan_fill_kernel(uint64_t* words, int64_t n) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += step) words[i] = ~uint64_t{0};
}

__device__ __forceinline__ void publish(uint32_t* at, float v) {
  const uint32_t w = __float_as_uint(v);
  __hip_atomic_store(at, w == ~0u ? 0x7fc00000u : w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void publish(uint64_t* at, float m, float Y) {
  uint64_t w = static_cast<uint64_t>(__float_as_uint(Y)) << 32 | __float_as_uint(m);
  if (w == ~uint64_t{0}) w = uint64_t{0x7fc00000u} << 32 | 0x7fc00000u;
  __hip_atomic_store(at, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// A fold's A and M in one word: M, its sign bit set, for A from 1/2 to 1, and
// else A, which has no sign: 0 for a reset, and where a product of decays above
// 0 has become 0 the least number above it, so that an infinite state stays
// infinite.
__device__ __forceinline__ float decay_word(float A, float M) {
  const float far = A == 0.0f && !resets(A, M) ? __uint_as_float(1u) : A;
  // A distance that no y has the digits for is none: with an infinite one it would give NaN.
  return M >= -0.5f && M <= 0.0f ? (M < -0x1p-64f ? M : -0.0f) : far;
}
// A y + Y for such a word: near 1 the sum is rounded once, to y's steps.
__device__ __forceinline__ float fold_on(float m, float Y, float y) {
  return (__float_as_int(m) < 0 ? y : 0.0f) + fmaf(m, m == 0.0f ? 0.0f : y, Y);
}

// The states of 64 channels (a lane each) before `tile` > 0, from the words of
// the tiles before it: the nearest finished state among the last kDepth, run
// forward through the folds of the tiles since. Whichever state it starts
// from, the arithmetic is that of going through the tiles one by one, so the
// result does not depend on timing. Looks at the nearest tile first, then
// kAhead at a time, the folds of the nearer ones put aside in `stash` (with
// many units the nearest state is mostly there, and reading further tiles'
// words for it costs 2%; four at a time cost registers: 4% of the log backward). `fold`
// and `state` are the words of the unit's tile 0, 64 words a tile. Polls at
// most kPolls times (about a second), then gives NaN and says so in the status
// word: a wave reaches the end whatever the workspace holds.
constexpr int kAhead = 2;
constexpr int kDepth = 32;
constexpr int kPolls = 1 << 20;
__device__ __forceinline__ float fold_on(uint64_t f, float y) {
  return fold_on(__uint_as_float(static_cast<uint32_t>(f)), __uint_as_float(static_cast<uint32_t>(f >> 32)), y);
}
typedef uint64_t Stash[kDepth][kScanChannels];

// Looks at K tiles from `tile` - 1 - depth back. True with the state before
// `tile` in y; else depth grows by K where all K folds were there.
template <int K>
__device__ __forceinline__ bool look(const uint64_t* fold, const uint32_t* state, int tile, Stash& stash, int lane,
                                     int& depth, float& y) {
  uint32_t s[K];
  uint64_t f[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int from = tile - 1 - depth - k;
    const int64_t i = static_cast<int64_t>(from > 0 ? from : 0) * kScanChannels;
    s[k] = __hip_atomic_load(state + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    f[k] = __hip_atomic_load(fold + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  bool folds = true;  // of the tiles nearer than k, all there
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (folds && __all(s[k] != ~0u)) {
      y = __uint_as_float(s[k]);
#pragma unroll
      for (int j = K - 1; j >= 0; --j)
        if (j < k) y = fold_on(f[j], y);
      for (int j = depth - 1; j >= 0; --j) y = fold_on(stash[j][lane], y);
      return true;
    }
    folds = folds && __all(f[k] != ~uint64_t{0});  // never tile 0's, which publishes its state alone
  }
  if (folds && depth + K <= kDepth) {
#pragma unroll
    for (int k = 0; k < K; ++k) stash[depth + k][lane] = f[k];
    depth += K;
  } else {
    __builtin_amdgcn_s_sleep(1);
  }
  return false;
}

__device__ __forceinline__ float give_up(uint32_t* status) {
  __hip_atomic_store(status, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return __uint_as_float(0x7fc00000u);
}
__device__ __forceinline__ float look_back(uint32_t* status, const uint64_t* fold, const uint32_t* state, int tile,
                                           Stash& stash, int lane) {
  int depth = 0;
  float y;
  for (int poll = 0; poll < kPolls; ++poll) {
    if (depth == 0 ? look<1>(fold, state, tile, stash, lane, depth, y)
                   : look<kAhead>(fold, state, tile, stash, lane, depth, y))
      return y;
  }
  return give_up(status);
}

// The same from the last tile's state alone.
__device__ __forceinline__ float last_state(uint32_t* status, const uint32_t* state, int tile) {
  for (int poll = 0; poll < kPolls; ++poll) {
    const uint32_t s = __hip_atomic_load(state + static_cast<int64_t>(tile - 1) * kScanChannels, __ATOMIC_RELAXED,
                                         __HIP_MEMORY_SCOPE_AGENT);
    if (__all(s != ~0u)) return __uint_as_float(s);
    __builtin_amdgcn_s_sleep(1);
  }
  return give_up(status);
}

// What a workgroup shares. Channel i of the slab is fold[wave][kPad + i]; the
// last lanes of a row whose width is no multiple of V use the places before 0.
constexpr int kPad = 8;
struct ScanShared {
  float4 fold[kScanMaxWaves][kPad + kScanChannels];  // the waves' folds A, Y, M, then in x the carry into each wave
  float after[kPad + kScanChannels];                 // the state after the sequence's last tile
  Stash stash;
  int tile;
};

// A lane's place: V channels from `start` of the row, tokens sub * R on of its
// wave's. The last lane of a row moves `shift` channels back to end with it;
// the channels it shares with its neighbour are computed by both and stored by
// the neighbour. A lane past the row (`in` false) reads the row's last channels.
template <int V>
struct ScanLane {
  int wave, sub, start, shift;
  int word;  // of the lane's first channel in ScanShared::fold[]
  bool in;
  __device__ __forceinline__ ScanLane(int slab, int d) {
    constexpr int CG = kScanChannels / V;
    const int lane = threadIdx.x & 63, cg = lane % CG;
    const int c = slab * kScanChannels + cg * V;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    sub = lane / CG;
    in = c < d;
    start = c < d - V ? c : d - V;
    shift = in ? c - start : 0;
    word = kPad + cg * V - shift;
  }
};

// The unit of this workgroup and the tile its number stands for. Workgroups go
// round the eight XCDs. Each XCD takes a run of neighbouring slabs, so that the
// pieces of a row meet in one L2 (10 to 12% faster at 8 x 8192 x 4096), and
// keeps them, so that the words between a unit's tiles stay near (runs that
// moved on with the tiles: 27 us against 21 at 32768 x 256). Of n units the
// runs are floor or ceil(n / 8) long, and a workgroup past the end of its run
// has nothing to do; below kXcdUnits, where the longest run would hold up the
// rest, the units go round one by one instead.
struct ScanPlace {
  int64_t unit, sh, slot0;  // slot0: of the unit's tile 0, over all columns
  int h, slab, tile;
  Piece piece;
};
__device__ __forceinline__ bool side_by_side(uint32_t n, uint32_t& i, int& tile) {
  const uint32_t round = scan_round(n);
  tile = blockIdx.x / round;
  i = blockIdx.x % round;
  if (n % kXcds && n < kXcdUnits) return true;
  const uint32_t run = i % kXcds;
  auto begin = [&](uint32_t r) { return n / kXcds * r + n % kXcds * r / kXcds; };  // floor(r n / 8)
  i = begin(run) + i / kXcds;
  return i < begin(run + 1);
}
// First slot of packed sequence s; it grows with s, by at least the sequence's
// tiles and at least 1.
__device__ __forceinline__ int first_slot(const Sequences& q, int s, int rows) {
  const int c = q.cu[s];
  return (c < 0 ? 0 : c > q.N ? q.N : c) / rows + s;
}
__device__ __forceinline__ ScanPlace scan_place(const Sequences& q, uint32_t units, int tiles, int rows,
                                                const ScanWords& w) {
  ScanPlace p{};
  const uint32_t slabs = (q.d + kScanChannels - 1) / kScanChannels, columns = q.H * slabs;
  int s;
  uint32_t column;
  if (q.cu && tiles > 1) {
    // Tile after tile along the packed row, the columns of each together. The
    // last sequence whose first slot is not past this one, 64 lanes looking at
    // a time.
    int slot;
    if (!side_by_side(columns, column, slot)) {
      p.tile = -1;
      return p;
    }
    const int lane = threadIdx.x & 63;
    s = 0;
    int left = q.S;  // sequences s .. s + left - 1 are in question
    while (left > 1) {
      const int step = (left + 63) / 64, mine = lane * step;
      const bool before = mine < left && first_slot(q, s + mine, rows) <= slot;
      const int n = __popcll(__ballot(before));
      const int skip = (n > 0 ? n - 1 : 0) * step;
      s += skip;
      left = left - skip < step ? left - skip : step;
    }
    s = __builtin_amdgcn_readfirstlane(s);
    const int first = first_slot(q, s, rows);
    p.tile = __builtin_amdgcn_readfirstlane(slot - first);
    p.slot0 = column * w.slots + first;
  } else {
    // The units of one tile of tokens together, so that most tiles at work
    // belong to different ones.
    uint32_t unit;
    if (!side_by_side(units, unit, p.tile)) {
      p.tile = -1;
      return p;
    }
    s = unit / columns;
    column = unit - s * columns;
    p.slot0 = column * w.slots + static_cast<int64_t>(s) * tiles;
  }
  p.h = column / slabs;
  p.slab = column - p.h * slabs;
  p.sh = static_cast<int64_t>(s) * q.H + p.h;
  p.unit = static_cast<int64_t>(s) * columns + column;
  p.piece = piece_of(q, s);
  return p;
}

// The next tile of the unit.
__device__ __forceinline__ int take_ticket(const ScanWords& w, int64_t unit, int& at) {
  if (threadIdx.x == 0)
    at = static_cast<int>(
        __hip_atomic_fetch_add(w.ticket + unit, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1u);
  lds_only_barrier();
  return __builtin_amdgcn_readfirstlane(at);
}

// Joins the lanes' folds (A, M, Y) of the workgroup, gets the tile's carry and
// leaves in y the state before each lane's first token. `first` and `last` are
// the states before the sequence (may be null) and after it (null: not
// wanted), at this unit's channel 0; `left` how many channels there are.
template <int V, int K>
__device__ __forceinline__ void scan_carry(float (&A)[V], float (&M)[V], float (&Y)[V], float (&y)[V], bool special,
                                           const ScanWords& w, const ScanPlace& p, bool end, const float* first,
                                           float* last, int left, const ScanLane<V>& at, ScanShared& shared) {
  constexpr int CG = kScanChannels / V;  // lanes side by side
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  // Inclusive over the V groups of lanes, K channels at a time: the words on
  // their way are registers (all of V at once spills).
  auto join = [&](auto careful) {
#pragma unroll
    for (int off = 1; off < V; off *= 2) {
#pragma unroll
      for (int j0 = 0; j0 < V; j0 += K) {
        float A1[K], M1[K], Y1[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
          A1[k] = __shfl_up(A[j0 + k], off * CG, 64);
          M1[k] = __shfl_up(M[j0 + k], off * CG, 64);
          Y1[k] = __shfl_up(Y[j0 + k], off * CG, 64);
        }
        if (at.sub >= off) {
#pragma unroll
          for (int k = 0; k < K; ++k) {
            const int j = j0 + k;
            if (careful && resets(A[j], M[j])) continue;
            Y[j] = fmaf(A[j], Y1[k], Y[j]);
            M[j] = fmaf(M[j], A1[k], M1[k]);
            A[j] *= A1[k];
          }
        }
      }
    }
  };
  if (special) join(std::true_type());
  else join(std::false_type());
  if (at.sub == V - 1) {
#pragma unroll
    for (int j = 0; j < V; ++j) shared.fold[at.wave][at.word + j] = make_float4(A[j], Y[j], M[j], 0.0f);
  }
  if (special) {  // M is not passed on: a reset is -0 from here
#pragma unroll
    for (int j = 0; j < V; ++j) A[j] = resets(A[j], M[j]) ? -0.0f : A[j];
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const float A1 = __shfl_up(A[j], CG, 64), Y1 = __shfl_up(Y[j], CG, 64);
    A[j] = at.sub ? A1 : 1.0f;
    Y[j] = at.sub ? Y1 : 0.0f;
  }
  lds_only_barrier();
  if (at.wave == 0) {  // a lane per channel
    float TA = 1.0f, TM = 0.0f, TY = 0.0f;
#pragma unroll 2  // more in flight spill where the backward holds four tensors
    for (int k = 0; k < waves; ++k) {
      const float4 g = shared.fold[k][kPad + lane];
      TY = fmaf(g.x, TY, g.y);
      TM = fmaf(g.z, TA, TM);
      TA *= g.x;
    }
    const bool tile_special = __any(TM != TM);  // a reset, or a gate that is NaN
    if (tile_special) {
      TA = 1.0f;
      TY = 0.0f;
#pragma unroll 1
      for (int k = 0; k < waves; ++k) {
        const float4 g = shared.fold[k][kPad + lane];
        TY = resets(g.x, g.z) ? g.y : fmaf(g.x, TY, g.y);
        TA = resets(g.x, g.z) ? 0.0f : TA * g.x;
      }
    }
    const float m = decay_word(TA, TM);
    const int64_t word = p.slot0 * kScanChannels + lane;
    const int64_t here = word + static_cast<int64_t>(p.tile) * kScanChannels;
    float carry;
    if (p.tile == 0) {
      carry = first && lane < left ? first[lane] : 0.0f;
    } else {
      if (w.fold) {
        if (!end) publish(w.fold + here, m, TY);
        carry = look_back(w.status, w.fold + word, w.state + word, p.tile, shared.stash, lane);
      } else {
        carry = last_state(w.status, w.state + word, p.tile);
      }
    }
    const float after = fold_on(m, TY, carry);
    if (end) {
      shared.after[kPad + lane] = after;
      if (last && lane < left) last[lane] = after;
    } else {
      publish(w.state + here, after);
    }
    if (tile_special) {
#pragma unroll 1
      for (int k = 0; k < waves; ++k) {
        const float4 g = shared.fold[k][kPad + lane];
        shared.fold[k][kPad + lane].x = carry;
        carry = resets(g.x, g.z) ? g.y : fmaf(g.x, carry, g.y);
      }
    } else {
#pragma unroll 2
      for (int k = 0; k < waves; ++k) {
        const float4 g = shared.fold[k][kPad + lane];
        shared.fold[k][kPad + lane].x = carry;
        carry = fmaf(g.x, carry, g.y);
      }
    }
  }
  lds_only_barrier();
#pragma unroll
  for (int j = 0; j < V; ++j) y[j] = fmaf(A[j], shared.fold[at.wave][at.word + j].x, Y[j]);
  if (special) {
#pragma unroll
    for (int j = 0; j < V; ++j) y[j] = __float_as_uint(A[j]) == 1u << 31 ? Y[j] : y[j];
  }
}

// Stores a lane's channels: all V, or the last V - shift of them. CACHED: not
// past the caches, for rows whose pieces share cache lines (a template: the
// compiler would make one ordinary store of the two sides of a branch).
template <bool CACHED, typename T, int V>
__device__ __forceinline__ void store_channels(T* p, const float (&x)[V], const ScanLane<V>& at) {
  if (!at.in) return;
  if (at.shift == 0) {
    if constexpr (CACHED) Pack<T, V>::keep(p, x);
    else Pack<T, V>::store(p, x);
  } else {
#pragma unroll
    for (int j = 1; j < V; ++j)
      if (j >= at.shift) Elem<T>::store(p, j, x[j]);
  }
}

// bf16, with the fill: 8 x 8192 x 4096 301 us (5.4 TB/s, a device copy of 1 GiB
// 5.1), 4 x 8192 x 4096 152 us. With few units a tile waits for the slowest of
// those before it: 65536 x 2048 (32 units) 185 us (4.4 TB/s), 32768 x 256 (4)
// 24 us (2.1 TB/s). Rows that are no multiple of a cache line move up to a
// quarter more bytes than theirs: 4 x 7501 x 1001 fp32 87 us (4.1 TB/s).
// TH is h's type: T, or fp32 for a backward that takes h without T's rounding.
template <typename T, typename TH, int FORM, int V, int E, bool CACHED>
__global__ void __launch_bounds__(64 * kScanMaxWaves, 4)
recurrence_kernel(View x, View gate, View out, Sequences q, const float* state_in, float* state_out, ScanWords w,
                  uint32_t units, int tiles) {
  __shared__ ScanShared shared;
  constexpr int R = E / V;
  typedef Pack<T, V> P;
  const int rows = static_cast<int>(blockDim.x >> 6) * E;
  ScanPlace p = scan_place(q, units, tiles, rows, w);
  if (p.tile < 0) return;
  const ScanLane<V> at(p.slab, q.d);
  const int len = p.piece.len;
  const T* xr = row_of<T>(x, p.piece.b, p.h) + p.piece.first * x.sn;
  const T* gr = row_of<T>(gate, p.piece.b, p.h) + p.piece.first * gate.sn;

  typename P::raw xw[R], gw[R];
  auto load = [&](int tile) {
    const int64_t row = static_cast<int64_t>(tile) * rows;  // below len
    if (row + rows <= len) {
      const T* xb = xr + (row + at.wave * E) * x.sn;
      const T* gb = gr + (row + at.wave * E) * gate.sn;
      const uint32_t xo = at.sub * R * static_cast<uint32_t>(x.sn) + at.start;
      const uint32_t go = at.sub * R * static_cast<uint32_t>(gate.sn) + at.start;
#pragma unroll
      for (int i = 0; i < R; ++i) gw[i] = P::load(gb + i * gate.sn + go);
      __builtin_amdgcn_sched_barrier(0);  // gates first: 299 us at 8 x 8192 x 4096 against 301
#pragma unroll
      for (int i = 0; i < R; ++i) xw[i] = P::load(xb + i * x.sn + xo);
    } else {  // tokens past the end read the last one
#pragma unroll
      for (int i = 0; i < R; ++i) {
        int64_t t = row + at.wave * E + at.sub * R + i;
        t = t < len ? t : len - 1;
        gw[i] = P::load(gr + t * gate.sn + at.start);
        xw[i] = P::load(xr + t * x.sn + at.start);
      }
    }
  };
  // A workgroup whose number stands for a tile past the end takes no ticket: as
  // many are left as the sequence has tiles. An empty sequence's tile 0 passes
  // its state on. With many units the loads start for the tile of the
  // workgroup's number while the ticket is on its way (the backward at 8 x 8192
  // x 4096 takes a seventh longer without); with few, where tickets of
  // neighbouring tiles cross and such loads are lost, they wait for it (backward
  // of 4 x 7501 x 1001 fp32: 167 us against 190).
  if (p.tile > 0 && static_cast<int64_t>(p.tile) * rows >= len) return;
  if (len > 0 && !w.fold) load(p.tile);
  if (tiles > 1) {
    const int tile = take_ticket(w, p.unit, shared.tile);
    if (tile > 0 && static_cast<int64_t>(tile) * rows >= len) return;
    if (w.fold ? len > 0 : tile != p.tile) load(tile);
    p.tile = tile;
  }
  const int64_t row0 = static_cast<int64_t>(p.tile) * rows;
  const int64_t t0 = row0 + at.wave * E + at.sub * R;
  const bool full = row0 + rows <= len;

  float a[R][V], b[R][V], A[V], M[V], Y[V], y[V];
  float lowest = 1.0f;  // of the lane's decays
  auto fold = [&](auto careful) {
    if (!full) {  // tokens past the end: a = 1, x = 0
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (t0 + i < len) continue;
        gw[i] = P::all(kKeepGate<FORM>);
        xw[i] = P::all(0.0f);
      }
    }
    uint32_t zero = 0;  // channels with a reset
#pragma unroll
    for (int i = 0; i < R; ++i) {
      P::unpack(gw[i], a[i]);
      P::unpack(xw[i], b[i]);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float g = a[i][j];
        float c;
        token_decay<FORM>(g, a[i][j], c);
        if (FORM == 0) lowest = fminf(lowest, a[i][j]);
        if (FORM == 0) b[i][j] = careful && c == 0.0f ? 0.0f : b[i][j] * c;
        lane_decay<FORM>(i, g, a[i][j], c, A[j], M[j]);
        if (careful) a[i][j] = mark_token(g, a[i][j]);
        const bool reset = careful && a[i][j] == 0.0f;
        if (reset) zero |= 1u << j;
        Y[j] = i && !reset ? fmaf(a[i][j], Y[j], b[i][j]) : b[i][j];
      }
    }
    bool odd = lane_decays<FORM>(A, M);
    if (careful) {
      mark_resets(zero, A, M);
      return true;
    }
    if (FORM == 0) odd = lowest == 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) odd |= FORM == 0 && !finite(Y[j]);
    return odd;
  };
  const bool special = __any(fold(std::false_type()));
  if (special) {
    load(p.tile);
    fold(std::true_type());
  }
  const int64_t unit_state = p.sh * q.d + p.slab * kScanChannels;
  const bool end = row0 + rows >= len;
  scan_carry<V, 4>(A, M, Y, y, special, w, p, end, state_in ? state_in + unit_state : nullptr,
                state_out ? state_out + unit_state : nullptr, q.d - p.slab * kScanChannels, at, shared);
  TH* hr = row_of<TH>(out, p.piece.b, p.h) + p.piece.first * out.sn;
  if (full && !special) {
    TH* hb = hr + (row0 + at.wave * E) * out.sn;
    const uint32_t ho = at.sub * R * static_cast<uint32_t>(out.sn) + at.start;
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int j = 0; j < V; ++j) y[j] = fmaf(a[i][j], y[j], b[i][j]);
      store_channels<CACHED, TH, V>(hb + i * out.sn + ho, y, at);
    }
  } else {
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int j = 0; j < V; ++j) y[j] = a[i][j] == 0.0f ? b[i][j] : fmaf(a[i][j], y[j], b[i][j]);
      if (t0 + i < len) store_channels<CACHED, TH, V>(hr + (t0 + i) * out.sn + at.start, y, at);
    }
  }
  if (end && t0 < len && len <= t0 + R) {  // the last h is the final state, to the bit
#pragma unroll
    for (int j = 0; j < V; ++j) y[j] = shared.after[at.word + j];
    store_channels<CACHED, TH, V>(hr + (len - 1) * out.sn + at.start, y, at);
  }
}

// The same from the last token on: token t of the recurrence is row
// len - 1 - t of the sequence. grad_h and the gate are loaded first; h and x
// are needed after the carry only and stay in flight until then. bf16, with the
// fill: sigmoid form 8 x 8192 x 4096 620 us (5.2 TB/s; 601 without M and the
// look for special waves), log form 4 x 8192 x 4096 262 us (5.1 TB/s), 65536 x
// 2048 285 us (4.7 TB/s). Bounds of four waves to a SIMD where the registers
// suffice, or nearly (the log form in bf16 spills 4): its three tensors of 32
// tokens in fp32, or with an fp32 h, do not fit.
template <typename T, typename TH, int FORM, int V, int E, bool CACHED>
__global__ void __launch_bounds__(64 * kScanMaxWaves, FORM == 0 || sizeof(TH) == 2 ? 4 : 2)
recurrence_backward_kernel(View grad_h, View x, View gate, View hv, View grad_x, View grad_gate, Sequences q,
                           const float* state_in, const float* grad_state_out, float* grad_state_in, ScanWords w,
                           uint32_t units, int tiles) {
  __shared__ ScanShared shared;
  constexpr int R = E / V;
  typedef Pack<T, V> P;
  const int rows = static_cast<int>(blockDim.x >> 6) * E;
  ScanPlace p = scan_place(q, units, tiles, rows, w);
  if (p.tile < 0) return;
  const ScanLane<V> at(p.slab, q.d);
  const int len = p.piece.len;
  typedef Pack<TH, V> PH;
  auto row = [&](const View& v) { return row_of<T>(v, p.piece.b, p.h) + p.piece.first * v.sn; };
  const T *dr = row(grad_h), *gr = row(gate), *xr = FORM == 0 ? row(x) : nullptr;
  const TH* hr = row_of<TH>(hv, p.piece.b, p.h) + p.piece.first * hv.sn;

  typename P::raw xw[R], gw[R], dw[R];
  typename PH::raw hw[R];
  // A tile's tokens and the one before them all exist where row + rows < len.
  auto load = [&](int tile) {
    const int64_t t = static_cast<int64_t>(tile) * rows;  // below len
    if (t + rows < len) {
      const int64_t low = len - (t + at.wave * E + E);  // the wave's first row in memory
      const uint32_t lane_row = (V - 1 - at.sub) * R;
      auto get = [&](const auto* from, int64_t sn, auto (&to)[R], int64_t back) {
        const auto* base = from + (low - back) * sn;
        const uint32_t o = lane_row * static_cast<uint32_t>(sn) + at.start;
#pragma unroll
        for (int i = 0; i < R; ++i)
          to[i] = Pack<std::remove_const_t<std::remove_pointer_t<decltype(from)>>, V>::load(base + (R - 1 - i) * sn + o);
      };
      get(gr, gate.sn, gw, 0);
      // In the order they are needed in: 610 us at 8 x 8192 x 4096 in the sigmoid
      // form, 619 in the compiler's own.
      __builtin_amdgcn_sched_barrier(0);
      get(dr, grad_h.sn, dw, 0);
      __builtin_amdgcn_sched_barrier(0);
      get(hr, hv.sn, hw, 1);
      if (FORM == 0) get(xr, x.sn, xw, 0);
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        int64_t r = len - 1 - (t + at.wave * E + at.sub * R + i);
        r = r > 0 ? r : 0;
        gw[i] = P::load(gr + r * gate.sn + at.start);
        dw[i] = P::load(dr + r * grad_h.sn + at.start);
        hw[i] = PH::load(hr + (r > 0 ? r - 1 : 0) * hv.sn + at.start);
        if (FORM == 0) xw[i] = P::load(xr + r * x.sn + at.start);
      }
    }
  };
  if (p.tile > 0 && static_cast<int64_t>(p.tile) * rows >= len) return;
  if (len > 0 && !w.fold) load(p.tile);
  if (tiles > 1) {
    const int tile = take_ticket(w, p.unit, shared.tile);
    if (tile > 0 && static_cast<int64_t>(tile) * rows >= len) return;
    if (w.fold ? len > 0 : tile != p.tile) load(tile);
    p.tile = tile;
  }
  const int64_t row0 = static_cast<int64_t>(p.tile) * rows;
  const int64_t t0 = row0 + at.wave * E + at.sub * R;
  const bool full = row0 + rows < len;

  // In the sigmoid form a decay near 1 is held as its negated distance from 1,
  // which has more digits, and any other as it is.
  auto decay = [](float v) { return FORM == 0 && __float_as_int(v) < 0 ? 1.0f + v : v; };
  auto rest = [](float v) { return __float_as_int(v) < 0 ? -v : 1.0f - v; };
  float a[R][V], A[V], M[V], Y[V], y[V];
  float least = 1.0f;  // 1 - a of the lane's tokens: 0 where one is passed over
  auto fold = [&](auto careful) {
    if (!full) {  // tokens past the end: a = 1, dh = 0
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (t0 + i < len) continue;
        // Not +inf: a 1 - a of 0 makes the wave special (240 x 317 x 2048 191 us, so 186).
        gw[i] = P::all(FORM == 0 ? 80.0f : 0.0f);
        dw[i] = P::all(0.0f);
      }
    }
    uint32_t zero = 0;  // channels with a reset
    float last[V];      // the decay of the token before; Y is the gradient of its h until the end
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float dh[V];
      P::unpack(gw[i], a[i]);
      P::unpack(dw[i], dh);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float g = a[i][j];
        float d, c;
        token_decay<FORM>(g, d, c);
        lane_decay<FORM>(i, g, d, c, A[j], M[j]);
        if (FORM == 0) least = fminf(least, c);
        if (careful) d = mark_token(g, d);
        a[i][j] = FORM == 0 && d > 0.5f ? -c : d;
        if (careful && d == 0.0f) zero |= 1u << j;
        Y[j] = i && !(careful && last[j] == 0.0f) ? fmaf(last[j], Y[j], dh[j]) : dh[j];
        last[j] = d;
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) Y[j] = careful && last[j] == 0.0f ? 0.0f : last[j] * Y[j];
    bool odd = lane_decays<FORM>(A, M);
    if (careful) {
      mark_resets(zero, A, M);
      return true;
    }
    if (FORM == 0 && __any(odd)) odd = any_zero(a);
    return odd || (FORM == 0 && least == 0.0f);
  };
  const bool special = __any(fold(std::false_type()));
  if (special) {
    load(p.tile);
    fold(std::true_type());
  }
  const int64_t unit_state = p.sh * q.d + p.slab * kScanChannels;
  scan_carry<V, 1>(A, M, Y, y, special, w, p, row0 + rows >= len, grad_state_out ? grad_state_out + unit_state : nullptr,
                grad_state_in ? grad_state_in + unit_state : nullptr, q.d - p.slab * kScanChannels, at, shared);
  T *dxr = row(grad_x), *dgr = row(grad_gate);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t r = len - 1 - (t0 + i);
    float before[V], v[V], dh[V], dx[V], dg[V];
    // Unpacked again: the compiler would hold both, and spill.
    if constexpr (sizeof(T) == 2 && V > 1) asm volatile("" : "+v"(dw[i]));
    P::unpack(dw[i], dh);
    PH::unpack(hw[i], before);
    if (FORM == 0) P::unpack(xw[i], v);
    if (!full && r == 0) {
#pragma unroll
      for (int j = 0; j < V; ++j) before[j] = state_in ? state_in[p.sh * q.d + at.start + j] : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float d = decay(a[i][j]), u = dh[j] + y[j];
      y[j] = d * u;
      if (FORM == 0) {
        dx[j] = rest(a[i][j]) * u;
        dg[j] = d * (before[j] - v[j]) * dx[j];
      } else {
        dx[j] = u;
        dg[j] = before[j] * y[j];
      }
    }
    // Resets, and tokens that are passed over: the products above may be 0 times
    // what is not finite, be it h of the token before, x or u.
    if (special) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const bool forgets = decay(a[i][j]) == 0.0f, keeps = FORM == 0 && rest(a[i][j]) == 0.0f;
        y[j] = forgets ? 0.0f : y[j];
        dx[j] = keeps ? 0.0f : dx[j];
        dg[j] = forgets || keeps ? 0.0f : dg[j];
      }
    }
    if (full || r >= 0) {
      store_channels<CACHED, T, V>(dxr + r * grad_x.sn + at.start, dx, at);
      store_channels<CACHED, T, V>(dgr + r * grad_gate.sn + at.start, dg, at);
    }
  }
}

// ---------------------------------------------------------------------------
// One token

constexpr int kStepThreads = 256;

// Grid: x over the pieces of V channels of a row's H heads, y over the B rows
// (strided). A thread takes V channels of a head; the last piece of a head is
// moved back to end with it, its first `shift` channels left to the neighbour.
// With slots a block first looks through them, its loads already on their
// way: a row whose slot an earlier row names is left to that row's block,
// which goes on with the later rows of its slot in order. Bound by HBM for
// large batches (three elements and an fp32 state read and written per
// channel): 512 rows of 8192 channels in bf16 11 us, 5.3 TB/s; below a few
// megabytes by the call, 9 us from Python.
template <typename T, int FORM, int V>
__global__ void __launch_bounds__(kStepThreads)
step_kernel(View x, View gate, View out, int B, int H, int d, float* states, int nstates, const int* slots) {
  __shared__ int named[kStepThreads / 64];
  typedef Pack<T, V> P;
  const int pieces = (d + V - 1) / V;
  const int piece = blockIdx.x * kStepThreads + threadIdx.x;
  const bool in = piece < pieces * H;
  const int h = in ? piece / pieces : 0;
  const int c = in ? (piece - h * pieces) * V : 0;
  const int start = c < d - V ? c : d - V, shift = c - start;
  for (int b = blockIdx.y; b < B; b += gridDim.y) {
    const int slot = slots ? slots[b] : b;
    if (slot < 0 || slot >= nstates) continue;
    float* state = states + (static_cast<int64_t>(slot) * H + h) * d + start;
    float now[V];
    Pack<float, V>::unpack(Pack<float, V>::load(state), now);
    auto gw = P::load(row_of<T>(gate, b, h) + start);
    auto xw = P::load(row_of<T>(x, b, h) + start);
    bool later = false;
    if (slots) {
      bool earlier = false;
      for (int i = threadIdx.x; i < B; i += kStepThreads) {
        const bool same = slots[i] == slot;
        earlier |= same && i < b;
        later |= same && i > b;
      }
      const int found = (__any(earlier) ? 1 : 0) | (__any(later) ? 2 : 0);
      __syncthreads();  // the last row's words have been read
      if ((threadIdx.x & 63) == 0) named[threadIdx.x >> 6] = found;
      __syncthreads();
      int all = 0;
#pragma unroll
      for (int w = 0; w < kStepThreads / 64; ++w) all |= named[w];
      if (all & 1) continue;
      later = all & 2;
    }
    for (int i = b;;) {
      float g[V], v[V];
      P::unpack(gw, g);
      P::unpack(xw, v);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float a, c;
        gate_of<FORM>(g[j], a, c);
        if (FORM == 0) v[j] = c == 0.0f ? 0.0f : v[j] * c;
        // As fold_on(): over many steps a's own rounding would add up.
        const bool near = c <= 0.5f && (FORM == 0 || c >= 0.0f);
        const float old = g[j] == -__builtin_inff() ? 0.0f : now[j];  // a reset forgets whatever it is
        now[j] = fmaf(near ? -c : a, old, v[j]) + (near ? old : 0.0f);
      }
      if (in) {
        T* o = row_of<T>(out, i, h) + start;
        if (shift == 0) {
          P::keep(o, now);
        } else {
#pragma unroll
          for (int j = 1; j < V; ++j)
            if (j >= shift) Elem<T>::store(o, j, now[j]);
        }
      }
      if (!later) break;
      do ++i;
      while (i < B && slots[i] != slot);
      if (i >= B) break;
      gw = P::load(row_of<T>(gate, i, h) + start);
      xw = P::load(row_of<T>(x, i, h) + start);
    }
    if (in) {
      if (shift == 0) {
        Pack<float, V>::keep(state, now);
      } else {
#pragma unroll
        for (int j = 1; j < V; ++j)
          if (j >= shift) state[j] = now[j];
      }
    }
  }
}

}  // namespace

namespace {

// Fills the words of a launch with several tiles; *words points into them.
hipError_t scan_words(const ScanPlan& p, void* workspace, ScanWords* words, hipStream_t stream) {
  *words = ScanWords{};
  if (p.tiles <= 1) return hipSuccess;
  char* base = static_cast<char*>(workspace);
  words->status = reinterpret_cast<uint32_t*>(base);
  base += kScanStatusBytes;
  words->ticket = reinterpret_cast<uint32_t*>(base);
  base += (static_cast<size_t>(p.units) * 4 + 255) / 256 * 256;
  words->state = reinterpret_cast<uint32_t*>(base);
  const size_t states = (p.bytes - static_cast<size_t>(base - static_cast<char*>(workspace))) / (p.folds ? 3 : 1);
  if (p.folds) words->fold = reinterpret_cast<uint64_t*>(base + states);
  words->slots = p.slots;
  const int64_t n = static_cast<int64_t>(p.bytes / sizeof(uint64_t));
  const int64_t blocks = (n + 255) / 256;
  scan_fill_kernel<<<static_cast<unsigned>(blocks < 2048 ? blocks : 2048), 256, 0, stream>>>(
      reinterpret_cast<uint64_t*>(workspace), n);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gated_recurrence(int form, int dtype, const View& x, const View& gate, const View& h,
                                   const Sequences& q, const float* state_in, float* state_out, void* workspace,
                                   hipStream_t stream) {
  const bool wide_h = dtype & kWideH;
  dtype &= ~kWideH;
  const ScanPlan p = plan_scan(q.S, q.H, q.N, q.max_len, q.cu != nullptr, q.d, dtype, false, form);
  ScanWords words;
  const hipError_t e = scan_words(p, workspace, &words, stream);
  if (e != hipSuccess) return e;
  const dim3 grid(static_cast<unsigned>(p.blocks)), block(64 * p.waves);
  // Rows that do not all begin on a cache line: the pieces that two workgroups
  // write meet within lines and go through the caches (8 x 4096 x 4104 bf16 179
  // us against 239 past them, 64 x 1024 x 1032 98 against 125, 64 x 640 x 1001
  // fp32 104 against 121). Where x, gate and h are small enough for the inputs
  // to be in the Infinity Cache still, results past it leave them there (176 MB,
  // 10749 x 2728 bf16: 54 against 46; 240 MB, 2 x 20000 x 1001 bf16: 74 and 76).
  const int64_t size = dtype == 0 ? 4 : 2;
  const int64_t h_size = wide_h ? 4 : size;
  const int64_t rows = int64_t{q.cu ? 1 : q.S} * q.H * q.N;
  const bool cached = h.sn * h_size % 128 != 0 && rows * q.d * (2 * size + h_size) > kScanCacheBytes;
#define RET_SCAN(T, TH, FORM, V, E, CACHED)                                                                \
  recurrence_kernel<T, TH, FORM, V, E, CACHED><<<grid, block, 0, stream>>>(x, gate, h, q, state_in,        \
                                                                           state_out, words,               \
                                                                           static_cast<uint32_t>(p.units), \
                                                                           static_cast<int>(p.tiles))
#define RET_SCAN_VEC(T, TH, FORM, V)                                     \
  do {                                                                   \
    if (p.vec == V && cached) RET_SCAN(T, TH, FORM, V, kScanRows, true); \
    else if (p.vec == V) RET_SCAN(T, TH, FORM, V, kScanRows, false);     \
    else RET_SCAN(T, TH, FORM, 1, kScanNarrowRows, true);                \
  } while (0)
  if (dtype == 0) {
    if (form == 0) RET_SCAN_VEC(float, float, 0, 4);
    else RET_SCAN_VEC(float, float, 1, 4);
  } else if (wide_h) {
    if (form == 0) RET_SCAN_VEC(uint16_t, float, 0, 4);
    else RET_SCAN_VEC(uint16_t, float, 1, 4);
  } else {
    if (form == 0) RET_SCAN_VEC(uint16_t, uint16_t, 0, 4);
    else RET_SCAN_VEC(uint16_t, uint16_t, 1, 4);
  }
#undef RET_SCAN_VEC
#undef RET_SCAN
  return hipGetLastError();
}

hipError_t launch_gated_recurrence_backward(int form, int dtype, const View& grad_h, const View& x, const View& gate,
                                            const View& h, const View& grad_x, const View& grad_gate,
                                            const Sequences& q, const float* state_in, const float* grad_state_out,
                                            float* grad_state_in, void* workspace, hipStream_t stream) {
  const bool wide_h = dtype & kWideH;
  dtype &= ~kWideH;
  const ScanPlan p = plan_scan(q.S, q.H, q.N, q.max_len, q.cu != nullptr, q.d, dtype, true, form);
  ScanWords words;
  const hipError_t e = scan_words(p, workspace, &words, stream);
  if (e != hipSuccess) return e;
  const dim3 grid(static_cast<unsigned>(p.blocks)), block(64 * p.waves);
  // Rows that do not all begin on a cache line: the pieces that two workgroups
  // write meet within lines, and two results of them fare better through the
  // caches (bf16: 4 x 7501 x 1001 111 us against 128, 55 x 193 x 3824 108
  // against 130, 10749 x 2728 110 against 113; fp32: 4 x 7501 x 1001 167
  // against 193, 4 x 19454 x 696 289 against 302).
  const int64_t size = dtype == 0 ? 4 : 2;
  const bool cached = grad_x.sn * size % 128 != 0 || grad_gate.sn * size % 128 != 0;
#define RET_SCAN(T, TH, FORM, V, E, CACHED)                                                                \
  recurrence_backward_kernel<T, TH, FORM, V, E, CACHED><<<grid, block, 0, stream>>>(                       \
      grad_h, x, gate, h, grad_x, grad_gate, q, state_in, grad_state_out, grad_state_in, words,            \
      static_cast<uint32_t>(p.units), static_cast<int>(p.tiles))
#define RET_SCAN_VEC(T, TH, FORM, V, E)                                \
  do {                                                                 \
    if (p.vec == V && cached) RET_SCAN(T, TH, FORM, V, E, true);       \
    else if (p.vec == V) RET_SCAN(T, TH, FORM, V, E, false);           \
    else RET_SCAN(T, TH, FORM, 1, kScanNarrowRows, true);              \
  } while (0)
  if (dtype == 0) {
    if (form == 0) RET_SCAN_VEC(float, float, 0, 4, kScanSigmoidBackRows);
    else RET_SCAN_VEC(float, float, 1, 4, kScanRows);
  } else if (wide_h) {
    if (form == 0) RET_SCAN_VEC(uint16_t, float, 0, 8, kScanSigmoidBackRows);
    else RET_SCAN_VEC(uint16_t, float, 1, 8, kScanRows);
  } else {
    if (form == 0) RET_SCAN_VEC(uint16_t, uint16_t, 0, 8, kScanSigmoidBackRows);
    else RET_SCAN_VEC(uint16_t, uint16_t, 1, 8, kScanRows);
  }
#undef RET_SCAN_VEC
#undef RET_SCAN
  return hipGetLastError();
}

hipError_t launch_gated_recurrence_step(int form, int dtype, const View& x, const View& gate, const View& h, int B,
                                        int H, int d, float* states, int nstates, const int* slots,
                                        hipStream_t stream) {
  // Heads that lie one behind the other are one long head.
  if (x.sh == (H > 1 ? d : 0) && gate.sh == x.sh && h.sh == x.sh) {
    d *= H;
    H = 1;
  }
  const int vec = d < (dtype == 0 ? 4 : 8) ? 1 : dtype == 0 ? 4 : 8;
  const int64_t pieces = static_cast<int64_t>((d + vec - 1) / vec) * H;
  const dim3 grid(static_cast<unsigned>((pieces + kStepThreads - 1) / kStepThreads), B < 65535 ? B : 65535);
#define RET_STEP(T, FORM, V) \
  step_kernel<T, FORM, V><<<grid, kStepThreads, 0, stream>>>(x, gate, h, B, H, d, states, nstates, slots)
#define RET_STEP_VEC(T, FORM, V)              \
  do {                                        \
    if (vec == V) RET_STEP(T, FORM, V);       \
    else RET_STEP(T, FORM, 1);                \
  } while (0)
  if (dtype == 0) {
    if (form == 0) RET_STEP_VEC(float, 0, 4);
    else RET_STEP_VEC(float, 1, 4);
  } else {
    if (form == 0) RET_STEP_VEC(uint16_t, 0, 8);
    else RET_STEP_VEC(uint16_t, 1, 8);
  }
#undef RET_STEP_VEC
#undef RET_STEP
  return hipGetLastError();
}

}  // namespace ret
