// The selective scan: a recurrence with its own decay for every channel c and
// state n, d_t[c] the step:
//   h_t[c][n] = exp(d_t[c] A[c][n]) h_{t-1}[c][n] + d_t[c] u_t[c] B_t[n]
//   y_t[c] = (sum_n h_t[c][n] C_t[n] + D[c] u_t[c]) silu(z_t[c]).
//
// Work and split.  Per token and state one exponential and three multiply-adds:
// at 16 states latency bounds it, not memory and no unit (2 x 2048 x 5120 bf16:
// issue slots 54 %, shared memory 63 %, special-function unit 31 %): the
// registers leave each scheduler one warp of the recurrence.  A block of 16 channels (32 for up to 8 states) walks
// down the tokens in tiles of 32, and has two sides that meet once a tile:
//  - the recurrence: a lane keeps four states of two channels in registers (so
//    a token's B and C are read once for both), T lanes share a channel,
//    multiply-adds go two at a time (f32x2).  Four tokens' sums are joined over
//    a channel's lanes together: with four lanes three shuffles for four tokens,
//    and every lane ends with one token's sum;
//  - the memory side (two warps): 16-byte loads one tile ahead, the steps put
//    through softplus once and kept with d u in shared memory, and the outputs
//    of the tile before (skip term, gate, 16-byte stores).
// With both sides' work in one warp a block's latency, not its work, set the
// pace (2 x 2048 x 5120, 16 states, bf16: 304 us); with one warp for the memory
// side 194, with two 165.  Four blocks on a multiprocessor take about 31 cycles
// a token each, and issue in 54 % of them; their recurrence warps lie on its four
// schedulers then.  With a fifth two share one (whole sequences of 2 x 2048
// tokens, 16 states, bf16, 1, 2, 3, 4 and 5 blocks of 16 channels a
// multiprocessor: 88, 101, 115, 124 and 166 us), and a grid that starts while the
// one in front still runs is spread as unevenly as that.  So it starts alone, and
// numbers of blocks that do not divide evenly are cut in runs that do
// (scan_slots_kernel; 2 x 2048 x 5120: 166 -> 142 us).
//
// Segments.  With few channels a sequence is cut into segments that run side by
// side: a first launch computes every segment's state from zero and its sum of
// steps, the second starts each segment from what those give,
//   h = exp(A sum d) h + h_segment,  segment by segment,
// and computes the outputs.  The exponentials are paid twice, so segments are
// cut only where the blocks would not fill the GPU otherwise (segment_count).
#include "layer.cuh"

namespace ssd {
namespace {

constexpr int kNS = 4;    // states a lane keeps of each of its two channels
constexpr int kTile = 32;  // tokens a tile

struct ScanParams {
  int64_t L;
  int D, N, G, per, tiles, softplus;  // per: channels of a group; tiles: blocks of a group
  const void *u, *delta, *z, *Bm, *Cm;
  int64_t ub, ut, db, dt, zb, zt, Bb, Bt, Cb, Ct;
  const float *A, *skip, *delta_bias, *init;
  float* final_state;
  void* y;
  const int32_t* lengths;
  int segments;
  int64_t segment;   // tokens a segment, a multiple of kTile
  float* seg_state;  // [batch][segments][D][N]: init_state, then each segment's state from zero
  float* seg_sum;    // [batch][segments][D]: each segment's sum of steps
  int64_t quota;     // slots: tiles of tokens a block takes, no fewer than a sequence has
  uint64_t* handed;  // slots: states at a cut, [batch][G * tiles][states of a lane, two each][lane]
  int* ready;        // slots: [batch][G * tiles], `at_first`, then kReady or kTaken
  int at_first, polls;  // slots: 0, and how often a block looks for a state before it gives up
};

// 16 bytes of consecutive values as they lie in memory.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  static constexpr int kE = 8;
  uint4 v;
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void set(int i, __nv_bfloat16 x) {
    const uint32_t bits = __bfloat16_as_ushort(x);
    uint32_t* w = &v.x;
    w[i / 2] = i % 2 ? (w[i / 2] & 0xFFFFu) | (bits << 16) : (w[i / 2] & 0xFFFF0000u) | bits;
  }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t w = (&v.x)[i / 2];
    return __uint_as_float(i % 2 ? w & 0xFFFF0000u : w << 16);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 two = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&two);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Raw<float> {
  static constexpr int kE = 4;
  float4 v;
  __device__ __forceinline__ void zero() { v = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void set(int i, float x) { (&v.x)[i] = x; }
  __device__ __forceinline__ float get(int i) const { return (&v.x)[i]; }
  static __device__ __forceinline__ void store(float* p, const float (&f)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  }
};

// A vector from p, its first n values there (0 for the rest).  kVec: all or none, 16-byte aligned.
template <typename T, bool kVec>
__device__ __forceinline__ void load16(Raw<T>& r, const T* p, int n) {
  r.zero();
  if constexpr (kVec) {
    if (n > 0) r.load(p);
  } else {
#pragma unroll
    for (int i = 0; i < Raw<T>::kE; ++i)
      if (i < n) r.set(i, p[i]);
  }
}

// The decay 2^(d a).  The special-function unit's results for arguments in (-1, 0) were measured 2e-8
// too small on average (6e-9 above -0.003), which over the hundreds of tokens that a state remembers adds
// up to more than all roundings do.  The exponent gets kNudge back, in a multiply-add that takes the
// multiplication's place: the states' error fell from 3.5e-7 to 2.1e-7 of their norm (1500 tokens, fp32),
// from 1.1e-6 to 5.7e-7 (53 tokens).  2^kNudge is 1: a step of 0 keeps the state's bits.
constexpr float kNudge = 1.8e-8f;

// softplus of two numbers, its polynomial two at a time.
__device__ __forceinline__ void softplus2(float& v0, float& v1) {
  const float e0 = expf(-fabsf(v0)), e1 = expf(-fabsf(v1));
  const uint64_t s = pack2(e0 * rcp_fast(2.f + e0), e1 * rcp_fast(2.f + e1));
  const uint64_t q = mul2(s, s);
  auto both = [](float c) { return pack2(c, c); };
  uint64_t r = fma2(q, both(kAtanh4), both(kAtanh3));
  r = fma2(q, r, both(kAtanh2));
  r = fma2(q, r, both(kAtanh1));
  r = fma2(q, r, both(kAtanh0));
  r = fma2(mul2(q, s), r, s);
  float r0, r1;
  unpack2(r, r0, r1);
  v0 = fmaf(2.f, r0, fmaxf(v0, 0.f));
  v1 = fmaf(2.f, r1, fmaxf(v1, 0.f));
}

// Sizes that follow from T, the lanes of a channel (T * kNS states), and the type of the inputs.
template <typename V, int T>
struct Shape {
  static constexpr int kE = Raw<V>::kE;
  static constexpr int kN = T * kNS;
  static constexpr int kChannels = T == 2 ? 32 : 16;       // of a block
  static constexpr int kThreads = kChannels / 2 * T;       // of the recurrence
  static constexpr int kHelp = T == 16 ? 128 : 64;         // of the memory side
  // blocks that a multiprocessor's registers have to hold: of the outputs' launch, of the states'
  static constexpr int kBlocks[2] = {T == 2 ? (kE == 4 ? 2 : 4) : T == 4 ? (kE == 4 ? 4 : 5) : T == 8 ? (kE == 4 ? 3 : 4) : 2,
                                     T == 2 ? 7 : T == 4 ? 8 : T == 8 ? 6 : 3};
  static constexpr int kCols = kChannels / kE;             // vectors in a row of channels
  static constexpr int kIO = kTile * kCols;                // and in a tile
  static constexpr int kIOEach = (kIO + kHelp - 1) / kHelp;
  static constexpr int kBC = kTile * kN / kE;              // vectors in a tile of B (or C)
  static constexpr int kBCEach = (2 * kBC + kHelp - 1) / kHelp;
  // rows in floats, padded so that neighbouring rows fall into different banks
  static constexpr int kStepRow = 2 * kChannels + 4, kYRow = kChannels + 8;
};

// What a block walks along: tokens [begin, stop) of a sequence.
struct Walk {
  int64_t begin, stop;
  int seg;               // the segment, 0 of 1 elsewhere
  bool last;             // the sequence's last tokens: the state is the final one
  const uint64_t* from;  // a state left by another block to start from, or null
  uint64_t* to;          // where the state is left for another block, or null
};

// kState: only the segment's state from zero and its sum of steps (the first of two launches).
template <typename V, int T, bool kVec, bool kState>
__device__ __forceinline__ void walk(const ScanParams& p, int block, int64_t b, const Walk& w) {
  using S = Shape<V, T>;
  constexpr int kE = S::kE;
  __shared__ __align__(16) float s_step[2][kTile][S::kStepRow];  // (d, d u) of each channel
  __shared__ __align__(16) float s_B[2][kTile][S::kN], s_C[2][kTile][S::kN];
  __shared__ __align__(16) float s_y[2][kTile][S::kYRow];
  const int group = block / p.tiles;
  const int in_group = (block % p.tiles) * S::kChannels;
  const int c0 = group * p.per + in_group;
  const int nc = p.per - in_group < S::kChannels ? p.per - in_group : S::kChannels;
  const int seg = w.seg;
  int64_t len = p.L;
  if (p.lengths) len = p.lengths[b] < 0 ? 0 : p.lengths[b] < p.L ? p.lengths[b] : p.L;
  const int64_t begin = w.begin, stop = w.stop;  // of the outputs
  const int64_t end = len < stop ? len : stop;   // of the recurrence
  const int tiles = end > begin ? static_cast<int>((end - begin + kTile - 1) / kTile) : 0;

  if (threadIdx.x >= S::kThreads) {
    // ---- memory side: loads, steps, and the outputs of the tile before ----
    const int tid = threadIdx.x - S::kThreads;
    const V* u = static_cast<const V*>(p.u) + b * p.ub + c0;
    const V* delta = static_cast<const V*>(p.delta) + b * p.db + c0;
    const V* z = static_cast<const V*>(p.z) + b * p.zb + c0;
    const V* Bm = static_cast<const V*>(p.Bm) + b * p.Bb + static_cast<int64_t>(group) * p.N;
    const V* Cm = static_cast<const V*>(p.Cm) + b * p.Cb + static_cast<int64_t>(group) * p.N;
    // a thread's vectors all lie in the same channels (kHelp is a multiple of kCols)
    const int col0 = tid % S::kCols * kE;
    float bias[kE], skip[kE];
#pragma unroll
    for (int i = 0; i < kE; ++i) {
      bias[i] = p.delta_bias && col0 + i < nc ? p.delta_bias[c0 + col0 + i] : 0.f;
      skip[i] = !kState && p.skip && col0 + i < nc ? p.skip[c0 + col0 + i] : 0.f;
    }
    struct Tile {
      Raw<V> u[S::kIOEach], d[S::kIOEach], z[S::kIOEach], bc[S::kBCEach];
    } r;                                                                    // the tile on its way
    Raw<V> u1[S::kIOEach], z1[S::kIOEach], u2[S::kIOEach], z2[S::kIOEach];  // the two staged last
    auto fetch = [&](int64_t t0) {
#pragma unroll
      for (int i = 0; i < S::kIOEach; ++i) {
        const int v = tid + i * S::kHelp;
        const int64_t t = t0 + v / S::kCols;
        const int n = v < S::kIO && t < end ? nc - col0 : 0;
        load16<V, kVec>(r.u[i], u + t * p.ut + col0, n);
        load16<V, kVec>(r.d[i], delta + t * p.dt + col0, n);
        if constexpr (!kState) {
          if (p.z) load16<V, kVec>(r.z[i], z + t * p.zt + col0, n);
        }
      }
#pragma unroll
      for (int i = 0; i < S::kBCEach; ++i) {
        const int v = tid + i * S::kHelp;
        const bool is_c = v >= S::kBC;
        const int at = is_c ? v - S::kBC : v;
        const int64_t t = t0 + at / (S::kN / kE);
        const int n = at % (S::kN / kE) * kE;
        if (v < (kState ? S::kBC : 2 * S::kBC))
          load16<V, kVec>(r.bc[i], (is_c ? Cm + t * p.Ct : Bm + t * p.Bt) + n, t < end ? p.N - n : 0);
      }
    };
    auto stage = [&](int64_t t0, int buf) {  // the tile's steps and rows of B and C
#pragma unroll
      for (int j = 0; j < S::kIOEach; ++j) {
        const int v = tid + j * S::kHelp;
        const int row = v / S::kCols;
        if (v < S::kIO) {
          const bool there = t0 + row < end;
          float4* dst = reinterpret_cast<float4*>(&s_step[buf][row][2 * col0]);
#pragma unroll
          for (int i = 0; i < kE; i += 2) {
            float d0 = r.d[j].get(i) + bias[i], d1 = r.d[j].get(i + 1) + bias[i + 1];
            if (p.softplus) softplus2(d0, d1);
            if (!there) d0 = d1 = 0.f;  // past the end the state stays
            dst[i / 2] = make_float4(d0, d0 * r.u[j].get(i), d1, d1 * r.u[j].get(i + 1));
          }
        }
      }
#pragma unroll
      for (int i = 0; i < S::kBCEach; ++i) {
        const int v = tid + i * S::kHelp;
        const bool is_c = v >= S::kBC;
        const int at = is_c ? v - S::kBC : v;
        if (v < (kState ? S::kBC : 2 * S::kBC)) {
          float* dst = (is_c ? s_C : s_B)[buf][at / (S::kN / kE)] + at % (S::kN / kE) * kE;
#pragma unroll
          for (int e = 0; e < kE; e += 4)
            *reinterpret_cast<float4*>(dst + e) =
                make_float4(r.bc[i].get(e), r.bc[i].get(e + 1), r.bc[i].get(e + 2), r.bc[i].get(e + 3));
        }
      }
    };
    auto put = [&](int64_t t0, int buf) {  // the outputs, with the inputs of two tiles ago
#pragma unroll
      for (int j = 0; j < S::kIOEach; ++j) {
        const int v = tid + j * S::kHelp;
        const int row = v / S::kCols;
        if (v >= S::kIO || t0 + row >= end || col0 >= nc) continue;
        V* y = static_cast<V*>(p.y) + (b * p.L + t0 + row) * p.D + c0 + col0;
        float out[kE];
#pragma unroll
        for (int i = 0; i < kE; i += 4) {
          const float4 sum = *reinterpret_cast<const float4*>(&s_y[buf][row][col0 + i]);
          out[i] = sum.x, out[i + 1] = sum.y, out[i + 2] = sum.z, out[i + 3] = sum.w;
        }
#pragma unroll
        for (int i = 0; i < kE; ++i) {
          out[i] = fmaf(skip[i], u2[j].get(i), out[i]);
          if (p.z) out[i] *= silu(z2[j].get(i));
        }
        if constexpr (kVec) {
          Raw<V>::store(y, out);
        } else {
#pragma unroll
          for (int i = 0; i < kE; ++i)
            if (col0 + i < nc) y[i] = from_f32<V>(out[i]);
        }
      }
    };
    fetch(begin);
    for (int i = 0; i <= tiles; ++i) {  // stage tile i, put tile i - 2, load tile i + 1
      const int64_t t0 = begin + static_cast<int64_t>(i) * kTile;
      if (i < tiles) stage(t0, i & 1);
      if constexpr (!kState) {
        if (i >= 2) put(t0 - 2 * kTile, i & 1);
#pragma unroll
        for (int j = 0; j < S::kIOEach; ++j) u2[j] = u1[j], z2[j] = z1[j], u1[j] = r.u[j], z1[j] = r.z[j];
      }
      fetch(t0 + kTile);  // (past the end: no loads)
      __syncthreads();
    }
    if constexpr (!kState) {
      if (tiles > 0) put(begin + static_cast<int64_t>(tiles - 1) * kTile, (tiles - 1) & 1);
      for (int64_t t = (end > begin ? end : begin) + tid / S::kCols; t < stop; t += S::kHelp / S::kCols) {
        V* y = static_cast<V*>(p.y) + (b * p.L + t) * p.D + c0 + col0;  // after the sequence's end
#pragma unroll
        for (int i = 0; i < kE; ++i)
          if (col0 + i < nc) y[i] = from_f32<V>(0.f);
      }
    }
    return;  // (of this walk)
  }

  // ---- the recurrence: two channels a lane, a share of their states ----
  const int tid = threadIdx.x;
  const int ch = tid / T * 2, part = tid % T;
  const int n0 = part * kNS;
  uint64_t a2[2][kNS / 2], h2[2][kNS / 2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int64_t state_row = (b * p.D + c0 + ch + k) * p.N;
#pragma unroll
    for (int i = 0; i < kNS / 2; ++i) {
      float a[2], h[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int n = n0 + 2 * i + e;
        const bool in = ch + k < nc && n < p.N;
        a[e] = in ? p.A[static_cast<int64_t>(c0 + ch + k) * p.N + n] * kLog2e : 0.f;
        h[e] = in && p.init && p.segments == 1 && !w.from ? p.init[state_row + n] : 0.f;
        // final_state may be init_state, and the last segment's block may end before another reads
        // its state: in segments all read a copy
        if (kState && seg == 0 && in)
          p.seg_state[(b * p.segments * p.D + c0 + ch + k) * p.N + n] = p.init ? p.init[state_row + n] : 0.f;
      }
      a2[k][i] = pack2(a[0], a[1]);
      h2[k][i] = w.from ? load_l2(w.from + (k * kNS / 2 + i) * S::kThreads + tid) : pack2(h[0], h[1]);
    }
  }
  if (!kState && p.segments > 1) {
#pragma unroll 2
    for (int j = 0; j <= seg; ++j) {  // the state entering this segment
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const bool live = ch + k < nc;
        const int64_t at = (b * p.segments + j) * p.D + c0 + ch + k;
        const float sum = live && j > 0 ? p.seg_sum[at - p.D] : 0.f;
        const uint64_t sum2 = pack2(sum, sum);
#pragma unroll
        for (int i = 0; i < kNS / 2; ++i) {
          const int n = n0 + 2 * i;
          const float lo = live && n < p.N ? p.seg_state[at * p.N + n] : 0.f;
          const float hi = live && n + 1 < p.N ? p.seg_state[at * p.N + n + 1] : 0.f;
          float x, y;
          unpack2(mul2(sum2, a2[k][i]), x, y);
          h2[k][i] = fma2(pack2(exp2_fast(x), exp2_fast(y)), h2[k][i], pack2(lo, hi));
        }
      }
    }
  }
  const uint64_t nudge2 = pack2(kNudge, kNudge);
  float total[2] = {0.f, 0.f};
  __syncthreads();
  for (int i = 0; i < tiles; ++i) {
    const int buf = i & 1;
    // all tokens of a tile, whatever the tile holds (steps past the end are 0): one straight run, in which the
    // joining of four tokens' sums overlaps the next four
#pragma unroll 2
    for (int t = 0; t < kTile; t += 4) {
      float acc[2][4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 st = *reinterpret_cast<const float4*>(&s_step[buf][t + q][2 * ch]);
        const ulonglong2 B4 = *reinterpret_cast<const ulonglong2*>(&s_B[buf][t + q][n0]);
        ulonglong2 C4;
        if constexpr (!kState) C4 = *reinterpret_cast<const ulonglong2*>(&s_C[buf][t + q][n0]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float d = k ? st.z : st.x, du = k ? st.w : st.y;
          const uint64_t d2 = pack2(d, d), du2 = pack2(du, du);
          if (kState) total[k] += d;
          uint64_t sum2 = 0;
#pragma unroll
          for (int j = 0; j < kNS / 2; ++j) {
            float x, y;
            unpack2(fma2(d2, a2[k][j], nudge2), x, y);
            h2[k][j] = fma2(pack2(exp2_fast(x), exp2_fast(y)), h2[k][j], mul2(du2, j ? B4.y : B4.x));
            if constexpr (!kState) sum2 = j ? fma2(h2[k][j], C4.y, sum2) : mul2(h2[k][j], C4.x);
          }
          if constexpr (!kState) {
            float lo, hi;
            unpack2(sum2, lo, hi);
            acc[k][q] = lo + hi;
          }
        }
      }
      if constexpr (!kState) {
        // lanes with bit 0 keep tokens 1 and 3, then those with bit 1 the later of the two left; over
        // higher bits the sums are added
        const bool b0 = part & 1, b1 = part & 2;
        float one[2], two[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          one[k] = (b0 ? acc[k][1] : acc[k][0]) + __shfl_xor_sync(0xffffffffu, b0 ? acc[k][0] : acc[k][1], 1);
          two[k] = (b0 ? acc[k][3] : acc[k][2]) + __shfl_xor_sync(0xffffffffu, b0 ? acc[k][2] : acc[k][3], 1);
        }
        if constexpr (T == 2) {
          *reinterpret_cast<float2*>(&s_y[buf][t + part][ch]) = make_float2(one[0], one[1]);
          *reinterpret_cast<float2*>(&s_y[buf][t + 2 + part][ch]) = make_float2(two[0], two[1]);
        } else {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            one[k] = (b1 ? two[k] : one[k]) + __shfl_xor_sync(0xffffffffu, b1 ? one[k] : two[k], 2);
#pragma unroll
            for (int o = 4; o < T; o *= 2) one[k] += __shfl_xor_sync(0xffffffffu, one[k], o);
          }
          if (part < 4) *reinterpret_cast<float2*>(&s_y[buf][t + part][ch]) = make_float2(one[0], one[1]);
        }
      }
    }
    __syncthreads();
  }
  if constexpr (kState) {
    grid_dep_launch();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (ch + k >= nc) continue;
      const int64_t at = (b * p.segments + seg + 1) * p.D + c0 + ch + k;
      if (part == 0) p.seg_sum[at - p.D] = total[k];
#pragma unroll
      for (int i = 0; i < kNS / 2; ++i) {
        float lo, hi;
        unpack2(h2[k][i], lo, hi);
        if (n0 + 2 * i < p.N) p.seg_state[at * p.N + n0 + 2 * i] = lo;
        if (n0 + 2 * i + 1 < p.N) p.seg_state[at * p.N + n0 + 2 * i + 1] = hi;
      }
    }
  } else if (w.to) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < kNS / 2; ++i) w.to[(k * kNS / 2 + i) * S::kThreads + tid] = h2[k][i];
  } else if (p.final_state && w.last) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (ch + k >= nc) continue;
      const int64_t state_row = (b * p.D + c0 + ch + k) * p.N;
#pragma unroll
      for (int i = 0; i < kNS / 2; ++i) {
        float lo, hi;
        unpack2(h2[k][i], lo, hi);
        if (n0 + 2 * i < p.N) p.final_state[state_row + n0 + 2 * i] = lo;
        if (n0 + 2 * i + 1 < p.N) p.final_state[state_row + n0 + 2 * i + 1] = hi;
      }
    }
  }
}

// A grid of (blocks, segments, batch): every block takes a segment, the whole sequence if there is one.
template <typename V, int T, bool kVec, bool kState>
__global__ void __launch_bounds__(Shape<V, T>::kThreads + Shape<V, T>::kHelp, Shape<V, T>::kBlocks[kState]) scan_kernel(ScanParams p) {
  grid_dep_wait();
  if constexpr (!kState) grid_dep_launch();  // (the first of two launches: at its end)
  const int seg = blockIdx.y;
  const int64_t begin = seg * p.segment;
  const bool last = seg + 1 == p.segments;
  const int64_t stop = !last && begin + p.segment < p.L ? begin + p.segment : p.L;
  walk<V, T, kVec, kState>(p, blockIdx.x, blockIdx.z, {begin, stop, seg, last, nullptr, nullptr});
}

// Slots.  All sequences' tiles of tokens, one (sequence, block of channels) after the other, are cut into
// equal runs, one a block of the grid, and all blocks are resident at once.  A run is as long as a sequence or
// longer, below two, so a sequence is cut at most once.  A block walks its run's last part first: the earlier
// tokens of a cut sequence are a block's first work and the later ones the next block's last, and by the time
// that these begin the state at the cut has been there for (quota - tiles of a sequence) tiles.
// 2 x 2048 tokens, 16 states, bf16, 5120, 5504, 6080 and 7296 channels: 142, 154, 169 and 206 us, whole sequences
// 166, 166, 166 and 219.  The loop over walks costs some 8 % of the rate (one walk alone 124 us, in the loop 134: the
// memory side waits for loads it holds across it); the walks written out one after the other cost more where the
// blocks of a multiprocessor are in different ones (5504: 182).
constexpr int kSlots = 4;  // blocks on a multiprocessor
constexpr int kReady = 1, kTaken = 2, kLost = 3, kPolls = 1 << 20;  // (kLost: never ready, for tests)

// The states a block of channels starts from, as one block hands them to another.
template <typename V, int T>
__device__ __forceinline__ void copy_init(const ScanParams& p, int block, int64_t b, uint64_t* to) {
  using S = Shape<V, T>;
  const int tid = threadIdx.x;
  if (tid >= S::kThreads) return;
  const int in_group = block % p.tiles * S::kChannels + tid / T * 2;
  for (int k = 0; k < 2; ++k) {
    const int64_t row = (b * p.D + block / p.tiles * p.per + in_group + k) * p.N;
    for (int i = 0; i < kNS / 2; ++i) {
      const int n = tid % T * kNS + 2 * i;
      const bool in = in_group + k < p.per;
      to[(k * kNS / 2 + i) * S::kThreads + tid] =
          pack2(in && n < p.N ? p.init[row + n] : 0.f, in && n + 1 < p.N ? p.init[row + n + 1] : 0.f);
    }
  }
}

template <typename V, int T, bool kVec>
__global__ void __launch_bounds__(Shape<V, T>::kThreads + Shape<V, T>::kHelp, kSlots)
scan_slots_kernel(ScanParams p, int64_t batch) {
  constexpr int kStates = kNS * Shape<V, T>::kThreads;
  __shared__ int s_flag;
  begin_kernel();
  const int64_t length = (p.L + kTile - 1) / kTile, blocks = static_cast<int64_t>(p.G) * p.tiles;
  const int64_t lo = blockIdx.x * p.quota, total = batch * blocks * length;
  const int64_t hi = lo + p.quota < total ? lo + p.quota : total;
  for (int64_t top = hi; top > lo;) {
    const int64_t q = (top - 1) / length;  // the sequence and block of channels
    int64_t begin = lo > q * length ? (lo - q * length) * kTile : 0;
    const bool last = top == (q + 1) * length;
    const int64_t stop = last ? p.L : (top - q * length) * kTile;
    uint64_t* state = p.handed + q * kStates;
    top = lo > q * length ? lo : q * length;
    bool mine = true, copied = false;
    if (begin > 0) {
      // The state comes from the block before.  Should it not come (the hardware starts blocks in their order, but
      // does not promise it), this block takes the sequence over from its first token.
      if (threadIdx.x == 0) {
        int flag = 0;
        for (int i = 0; i < p.polls && flag != kReady; ++i) {
          asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(flag) : "l"(p.ready + q) : "memory");
          if (flag != kReady) __nanosleep(200);
        }
        s_flag = flag == kReady ? flag : atomicCAS(p.ready + q, 0, kTaken);
        __threadfence();  // what the block writes comes after its claim
      }
      __syncthreads();
      if (s_flag != kReady) begin = 0;
    } else if (!last && p.init && p.init == p.final_state) {
      // In place, a block that took the sequence over may have overwritten the state to start from, or do so at any
      // time: this one starts from a copy, which is whole if the sequence was not yet taken over after it was made.
      copy_init<V, T>(p, static_cast<int>(q % blocks), q / blocks, state);
      copied = true;
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) s_flag = atomicAdd(p.ready + q, 0);
      __syncthreads();
      mine = s_flag != kTaken;
    }
    if (mine)
      walk<V, T, kVec, false>(p, static_cast<int>(q % blocks), q / blocks,
                              {begin, stop, 0, last, begin > 0 || copied ? state : nullptr, last ? nullptr : state});
    __syncthreads();
    if (!last && mine && threadIdx.x == 0) {
      __threadfence();
      atomicCAS(p.ready + q, 0, kReady);
    }
  }
}

// In front of it; it starts when this has ended, on a GPU that holds nothing else, so that the hardware
// gives every multiprocessor the same number of blocks.
__global__ void __launch_bounds__(256) clear_kernel(int* ready, int64_t n, int at_first) {
  grid_dep_wait();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i < n) ready[i] = at_first;
}

// One token: every state is read and written once and there is nothing to walk along, so memory
// bounds it.  A thread takes eight states of a channel of one sequence, T neighbouring lanes share the
// channel (its step is formed by each of them).  64 x 5120, 16 states, bf16, with four states a thread
// 13.2 us, with eight 9.4, with sixteen 11.3; two sequences a thread 10.8 (fewer warps on the SM).
constexpr int kTokenThreads = 128, kTokenNS = 8;

template <typename V, int T, bool kVec>
__global__ void __launch_bounds__(kTokenThreads, 8) scan_token_kernel(ScanParams p) {
  begin_kernel();
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kTokenThreads + threadIdx.x;
  const int part = static_cast<int>(id % T), n0 = kTokenNS * part;
  const bool live = id / T < p.D;
  const int c = live ? static_cast<int>(id / T) : p.D - 1;  // lanes past the end repeat the last channel
  const int g = c / p.per;
  const int64_t b = blockIdx.y;

  auto load_f = [&](const float* t, float (&v)[kTokenNS]) {  // states from t, 0 past N
#pragma unroll
    for (int q = 0; q < kTokenNS; q += 4) {
      if constexpr (kVec) {
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (n0 + q < p.N) f = *reinterpret_cast<const float4*>(t + q);
        v[q] = f.x, v[q + 1] = f.y, v[q + 2] = f.z, v[q + 3] = f.w;
      } else {
#pragma unroll
        for (int e = q; e < q + 4; ++e) v[e] = n0 + e < p.N ? t[e] : 0.f;
      }
    }
  };
  auto load_v = [&](const V* t, float (&v)[kTokenNS]) {
    if constexpr (kVec && sizeof(V) == 2) {
#pragma unroll
      for (int q = 0; q < kTokenNS; q += 4) {
        uint2 w = make_uint2(0, 0);
        if (n0 + q < p.N) w = *reinterpret_cast<const uint2*>(t + q);
        v[q] = __uint_as_float(w.x << 16), v[q + 1] = __uint_as_float(w.x & 0xFFFF0000u);
        v[q + 2] = __uint_as_float(w.y << 16), v[q + 3] = __uint_as_float(w.y & 0xFFFF0000u);
      }
    } else if constexpr (kVec) {
      load_f(reinterpret_cast<const float*>(t), v);
    } else {
#pragma unroll
      for (int e = 0; e < kTokenNS; ++e) v[e] = n0 + e < p.N ? to_f32(t[e]) : 0.f;
    }
  };

  const bool on = !p.lengths || p.lengths[b] > 0;
  float a[kTokenNS], h[kTokenNS] = {}, Bv[kTokenNS] = {}, Cv[kTokenNS] = {}, u = 0.f, step = 0.f, z = 0.f;
  const int64_t state = (b * p.D + c) * p.N + n0;
  if (p.init) load_f(p.init + state, h);
  if (on) {  // a sequence without a token keeps its state, and its inputs are not looked at
    u = to_f32(static_cast<const V*>(p.u)[b * p.ub + c]);
    step = to_f32(static_cast<const V*>(p.delta)[b * p.db + c]);
    if (p.z) z = to_f32(static_cast<const V*>(p.z)[b * p.zb + c]);
    load_v(static_cast<const V*>(p.Bm) + b * p.Bb + static_cast<int64_t>(g) * p.N + n0, Bv);
    load_v(static_cast<const V*>(p.Cm) + b * p.Cb + static_cast<int64_t>(g) * p.N + n0, Cv);
  }
  load_f(p.A + static_cast<int64_t>(c) * p.N + n0, a);
  const float skip = p.skip ? p.skip[c] : 0.f;
  if (p.delta_bias) step += p.delta_bias[c];
  if (p.softplus) step = softplus(step);
  if (!on) step = 0.f;
  const float du = step * u;
  float sum = 0.f;
#pragma unroll
  for (int e = 0; e < kTokenNS; ++e) {
    h[e] = fmaf(exp2_fast(fmaf(step, a[e] * kLog2e, kNudge)), h[e], du * Bv[e]);
    sum = fmaf(h[e], Cv[e], sum);
  }
#pragma unroll
  for (int o = 1; o < T; o *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (!live) return;
  if (part == 0) {
    float y = fmaf(skip, u, sum);
    if (p.z) y *= silu(z);
    static_cast<V*>(p.y)[b * p.D + c] = from_f32<V>(on ? y : 0.f);
  }
  if (!p.final_state) return;
  float* out = p.final_state + state;
#pragma unroll
  for (int q = 0; q < kTokenNS; q += 4) {
    if constexpr (kVec) {
      if (n0 + q < p.N) *reinterpret_cast<float4*>(out + q) = make_float4(h[q], h[q + 1], h[q + 2], h[q + 3]);
    } else {
#pragma unroll
      for (int e = q; e < q + 4; ++e)
        if (n0 + e < p.N) out[e] = h[e];
    }
  }
}

// Segments a sequence is cut into: enough recurrence warps for kFill on every multiprocessor, but no
// segment below kLeast tokens and no more than kMost (a segment joins all states before it).  Measured:
// 16384 x 2048 fp32 in 9, 11, 14, 16, 19 and 23 segments 339, 394, 332, 369, 331 and 349 us (19 taken);
// 2048 x 2048 bf16 in 4 and 16: 84 and 57 us.  Fewer than five pay more for the first launch than they
// gain: 513 x 5120 fp32 in four and whole 39 and 36 us, 2 x 2048 x 5120 bf16 in three and whole 205 and
// 165 us.  Nor does it pay where whole sequences fill the multiprocessors nearly as well: 2 x 2048 x 3648 in five and
// whole 143 and 118 us, 2 x 2048 x 2432 in eight and whole 104 and 101; so seven at least by the first rule (kWorth).
constexpr int64_t kFill = 16, kLeast = 128, kMost = 64, kWorth = 7;

int segment_count(int64_t batch, int64_t L, int64_t blocks, int warps) {
  const int64_t all = batch * blocks * warps;
  int64_t s = kFill * layer_sm_count() / all;
  if (s < kWorth) return 1;
  s = s < L / kLeast ? s : L / kLeast;
  s = s < kMost ? s : kMost;
  return s < 5 ? 1 : static_cast<int>(s);
}

template <typename V, int T>
cudaError_t launch_token(const ScanParams& p, int64_t batch, cudaStream_t stream) {
  const int64_t es = sizeof(V);
  // four states at a time where they start on 16 bytes (B and C: on four elements) everywhere
  const bool vec = p.N % 4 == 0 && aligned_to(p.A, 16) && aligned_to(p.init, 16) && aligned_to(p.final_state, 16) &&
                   aligned_to(p.Bm, 4 * es) && aligned_to(p.Cm, 4 * es) &&
                   (batch == 1 || (p.Bb % 4 == 0 && p.Cb % 4 == 0));
  const dim3 grid(static_cast<unsigned>(ceil_div(static_cast<int64_t>(p.D) * T, kTokenThreads)),
                  static_cast<unsigned>(batch));
  return launch_k(vec ? scan_token_kernel<V, T, true> : scan_token_kernel<V, T, false>, grid, dim3(kTokenThreads), 0,
                  stream, true, p);
}

template <typename V, int T, bool kVec>
cudaError_t launch_lanes(ScanParams p, int64_t batch, cudaStream_t stream) {
  constexpr int kThreads = Shape<V, T>::kThreads + Shape<V, T>::kHelp;
  const unsigned blocks = static_cast<unsigned>(p.G * p.tiles);
  const int64_t all = batch * blocks;
  if constexpr (T == 4) {
    if (p.quota > 0) {
      const cudaError_t e = launch_k(clear_kernel, dim3(static_cast<unsigned>(ceil_div(all, 256))), dim3(256), 0,
                                     stream, true, p.ready, all, p.at_first);
      if (e != cudaSuccess) return e;
      return launch_k(scan_slots_kernel<V, T, kVec>,
                      dim3(static_cast<unsigned>(ceil_div(all * ceil_div(p.L, kTile), p.quota))), dim3(kThreads), 0,
                      stream, true, p, batch);
    }
  }
  if (p.segments > 1) {
    const cudaError_t e = launch_k(scan_kernel<V, T, kVec, true>,
                                   dim3(blocks, static_cast<unsigned>(p.segments - 1), static_cast<unsigned>(batch)),
                                   dim3(kThreads), 0, stream, true, p);
    if (e != cudaSuccess) return e;
  }
  // Blocks that start while the kernel in front still holds multiprocessors are spread unevenly, and where a
  // multiprocessor gets several, the one with most sets the time (2 x 2048 x 4864, 16 states, bf16: 160 us, started
  // after that kernel's end 123; 3 x 501 x 2056: 40 and 32).
  const bool overlap = p.segments > 1 || all <= layer_sm_count();
  return launch_k(scan_kernel<V, T, kVec, false>,
                  dim3(blocks, static_cast<unsigned>(p.segments), static_cast<unsigned>(batch)), dim3(kThreads),
                  0, stream, overlap, p);
}

// Lanes a channel's states are spread over.
int lanes_of(int N) { return N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }

template <typename V, bool kVec>
cudaError_t launch_vec(const ScanParams& p, int64_t batch, cudaStream_t stream) {
  switch (lanes_of(p.N)) {
    case 2: return launch_lanes<V, 2, kVec>(p, batch, stream);
    case 4: return launch_lanes<V, 4, kVec>(p, batch, stream);
    case 8: return launch_lanes<V, 8, kVec>(p, batch, stream);
    default: return launch_lanes<V, 16, kVec>(p, batch, stream);
  }
}

template <typename T>
cudaError_t launch(const ScanParams& p, int64_t batch, cudaStream_t stream) {
  if (p.L == 1) {
    if (p.N <= kTokenNS) return launch_token<T, 1>(p, batch, stream);
    if (p.N <= 2 * kTokenNS) return launch_token<T, 2>(p, batch, stream);
    return p.N <= 4 * kTokenNS ? launch_token<T, 4>(p, batch, stream) : launch_token<T, 8>(p, batch, stream);
  }
  // 16-byte loads where every vector of channels (of states) starts on 16 bytes and is whole
  const int64_t es = sizeof(T);
  auto row16 = [&](const void* t, int64_t s0, int64_t s1) {
    return aligned_to(t, 16) && (batch == 1 || s0 * es % 16 == 0) && s1 * es % 16 == 0;
  };
  const bool vec = p.per % Raw<T>::kE == 0 && p.N % Raw<T>::kE == 0 && row16(p.u, p.ub, p.ut) && row16(p.delta, p.db, p.dt) &&
                   row16(p.z, p.zb, p.zt) && row16(p.Bm, p.Bb, p.Bt) && row16(p.Cm, p.Cb, p.Ct) && aligned_to(p.y, 16);
  return vec ? launch_vec<T, true>(p, batch, stream) : launch_vec<T, false>(p, batch, stream);
}

ssd_status check_sizes(const ssd_selective_scan_args* a) {
  if (!a || a->size != static_cast<int64_t>(sizeof(*a))) return SSD_ERR_INVALID_ARG;
  if (a->batch < 0 || a->seqlen < 0 || a->channels <= 0 || a->dstate <= 0 || a->ngroups <= 0) return SSD_ERR_INVALID_ARG;
  if (a->dstate > 64 || a->channels % a->ngroups != 0 || a->batch > 65535) return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

int channels_of_block(int N) { return lanes_of(N) == 2 ? Shape<float, 2>::kChannels : Shape<float, 4>::kChannels; }

int64_t blocks_of(const ssd_selective_scan_args* a) {
  return ceil_div(a->channels / a->ngroups, channels_of_block(a->dstate)) * a->ngroups;
}

int segments_of(const ssd_selective_scan_args* a) {
  const int64_t blocks = blocks_of(a);
  return segment_count(a->batch, a->seqlen, blocks, lanes_of(a->dstate) < 4 ? 1 : lanes_of(a->dstate) / 4);
}

// Slots are taken where whole sequences would leave some multiprocessors with a block more than others, and no more
// than seven on each: with more, blocks that end early make room for others (eight: 256 us in slots, 245 whole).
int64_t quota_of(const ssd_selective_scan_args* a) {
  if (segments_of(a) > 1 || a->seqlen <= kTile || lanes_of(a->dstate) != 4) return 0;
  const int64_t all = a->batch * blocks_of(a), sm = layer_sm_count();
  if (all <= kSlots * sm || all > 7 * sm) return 0;
  const int64_t length = ceil_div(a->seqlen, kTile), quota = ceil_div(all * length, kSlots * sm);
  return quota < 2 * length ? quota : 0;
}

// Bytes of the states at the cuts; the flags follow.
size_t handed_bytes(const ssd_selective_scan_args* a) {
  const int lanes = channels_of_block(a->dstate) / 2 * lanes_of(a->dstate);
  return static_cast<size_t>(a->batch) * blocks_of(a) * kNS * lanes * sizeof(uint64_t);
}

}  // namespace
}  // namespace ssd

extern "C" size_t ssd_selective_scan_workspace_size(const ssd_selective_scan_args* a) {
  using namespace ssd;
  if (check_sizes(a) != SSD_OK || a->batch == 0) return 0;
  if (quota_of(a) > 0) return handed_bytes(a) + static_cast<size_t>(a->batch) * blocks_of(a) * sizeof(int);
  const int s = segments_of(a);
  return s == 1 ? 0 : static_cast<size_t>(s) * a->batch * a->channels * (a->dstate + 1) * sizeof(float);
}

// at_first, polls: ScanParams.
static ssd_status scan(const ssd_selective_scan_args* a, int at_first, int polls, ssd_stream_t stream) {
  using namespace ssd;
  ssd_status st = check_sizes(a);
  if (st != SSD_OK) return st;
  if (!known_dtype(a->dtype)) return SSD_ERR_UNSUPPORTED;
  if (a->batch == 0) return SSD_OK;
  const size_t es = elem_size(a->dtype);
  if (!a->A) return SSD_ERR_INVALID_ARG;
  for (const void* f : {(const void*)a->A, (const void*)a->D, (const void*)a->delta_bias, (const void*)a->init_state,
                        (const void*)a->final_state, (const void*)a->lengths})
    if (!aligned_to(f, 4)) return SSD_ERR_INVALID_ARG;
  if (a->seqlen > 0) {
    for (const void* t : {a->u, a->delta, a->Bm, a->Cm, (const void*)a->y})
      if (!t || !aligned_to(t, es)) return SSD_ERR_INVALID_ARG;
    if (!aligned_to(a->z, es)) return SSD_ERR_INVALID_ARG;
  } else if (!a->final_state) {
    return SSD_OK;
  }
  ScanParams p{};
  p.segments = segments_of(a);
  p.quota = quota_of(a);
  if (p.segments > 1 || p.quota > 0) {
    if (!a->workspace || !aligned_to(a->workspace, 16)) return SSD_ERR_INVALID_ARG;
    if (a->workspace_bytes < ssd_selective_scan_workspace_size(a)) return SSD_ERR_WORKSPACE;
  }
  p.segment = ceil_div(ceil_div(a->seqlen, p.segments), kTile) * kTile;
  p.seg_state = static_cast<float*>(a->workspace);
  if (p.segments > 1) p.seg_sum = p.seg_state + static_cast<int64_t>(p.segments) * a->batch * a->channels * a->dstate;
  if (p.quota > 0) {
    p.handed = static_cast<uint64_t*>(a->workspace);
    p.ready = reinterpret_cast<int*>(static_cast<char*>(a->workspace) + handed_bytes(a));
  }
  p.at_first = at_first, p.polls = polls;
  p.L = a->seqlen;
  p.D = a->channels;
  p.N = a->dstate;
  p.G = a->ngroups;
  p.per = a->channels / a->ngroups;
  p.tiles = static_cast<int>(ceil_div(p.per, channels_of_block(p.N)));
  p.softplus = a->softplus != 0;
  p.u = a->u, p.delta = a->delta, p.z = a->z, p.Bm = a->Bm, p.Cm = a->Cm;
  p.ub = a->u_batch, p.ut = a->u_token, p.db = a->delta_batch, p.dt = a->delta_token;
  p.zb = a->z_batch, p.zt = a->z_token, p.Bb = a->B_batch, p.Bt = a->B_token, p.Cb = a->C_batch, p.Ct = a->C_token;
  p.A = a->A, p.skip = a->D, p.delta_bias = a->delta_bias, p.init = a->init_state;
  p.final_state = a->final_state;
  p.y = a->y;
  p.lengths = a->lengths;
  return launched(a->dtype == SSD_BF16 ? launch<__nv_bfloat16>(p, a->batch, stream)
                                       : launch<float>(p, a->batch, stream));
}

extern "C" ssd_status ssd_selective_scan(const ssd_selective_scan_args* a, ssd_stream_t stream) {
  return scan(a, 0, ssd::kPolls, stream);
}

extern "C" ssd_status ssd_debug_scan_handover(const ssd_selective_scan_args* a, int32_t taken, ssd_stream_t stream) {
  return scan(a, taken ? ssd::kTaken : ssd::kLost, 1000, stream);
}
