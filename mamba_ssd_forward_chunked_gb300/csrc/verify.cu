// Verification of drafted tokens: p and q the target's and the draft's
// probabilities (softmax of scale * logits), draft d_i is accepted while
// u_i q_i(d_i) < p_i(d_i); at the first that is not, a token is drawn from
// max(p - q, 0), or from p where all were accepted, by the inverse of its
// cumulative sums at the last random number.
//
// The first launch reads all logits once: the maximum and the sum of
// exponentials of every piece of a row.  In the second a cluster of blocks joins
// them, finds the first draft that is not accepted, and draws.
//
// Which token a random number hits goes by sums over the whole vocabulary: an
// error e of the sums moves it, for some 2 e vocab of all numbers, and 32-bit
// exponentials alone would do that for one number in a thousand.  So the drawing
// row's exponentials are formed in two 32-bit parts, to 2^-40 (reduction by a
// table, as Tang's of 1989), and summed as whole numbers of 2^-44: sums do not
// depend on their order, and the drawn token is the one that 64-bit arithmetic
// finds.  Whether a draft is accepted is a question of one ratio and goes by
// 32-bit sums: a random number within 2^-20 of it may fall either way.
//
// 32 requests of 7 drafts, 131072 bf16 logits with the draft's: 54 us, 126 MB at
// 6.8 TB/s would be 18.6.  The first launch takes 27 on cold caches (60 % of the
// DRAM's rate), the second 28: its two rows' weights fill the issue slots for
// 12, the rest is latency (joining, three barriers of the cluster's, the search).
// Every run's sums of p, of q and of both where p is larger are formed in one
// pass (a pass for the normalisers and one for the differences: 137 us).
#include <cooperative_groups.h>

#include <climits>

#include "layer.cuh"

namespace ssd {
namespace {

namespace cg = cooperative_groups;

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

constexpr int kThreads = 256;
constexpr int kMaxDrafts = 64;
constexpr int kMaxCluster = 8;
constexpr int kDrawThreads = 512;
constexpr int kDrawWarps = kDrawThreads / 32;
constexpr int kMaxVocab = 1 << 19;  // sums of weights are 2^63 at most, that of as many equal logits
constexpr float kLog2eLow = 1.925963e-8f;  // log2(e) - kLog2e

struct VerifyParams {
  int64_t logits_batch, logits_row, draft_batch, draft_row;
  int T, V, rows, pieces, piece;
  const void *logits, *draft_logits;
  const int32_t *draft, *lengths;
  const float *uniforms, *scale;
  float2* sums;  // [batch][rows][pieces]; rows: the target's T + 1, then the draft's T
  int32_t *tokens, *accepted;
  float* logprobs;
};

__device__ __forceinline__ float scale_of(const VerifyParams& p, int64_t b) { return p.scale ? p.scale[b] : 1.f; }
__device__ __forceinline__ bool usable(float scale) { return scale > 0.f && scale <= 1e37f; }
__device__ __forceinline__ int count_of(const VerifyParams& p, int64_t b) {
  const int n = p.lengths ? p.lengths[b] : p.T;
  return n < 0 ? 0 : n > p.T ? p.T : n;
}
// A NaN counts as -infinity, +infinity as the largest number.
__device__ __forceinline__ float plain_logit(float v) { return fminf(fmaxf(v, -INFINITY), 3.402823466e38f); }

template <typename T>
__device__ __forceinline__ void load_vector(const T* from, float (&v)[16 / sizeof(T)]) {
  const uint4 raw = *reinterpret_cast<const uint4*>(from);
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2)
      v[2 * i] = bf16_lo(w[i]), v[2 * i + 1] = bf16_hi(w[i]);
    else
      v[i] = __uint_as_float(w[i]);
  }
}

// The maximum and the sum of exponentials over a warp's parts.
__device__ __forceinline__ float2 join_sums(float2 v, float f) {
  float top = v.x;
#pragma unroll
  for (int o = 16; o; o /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float sum = v.x > -INFINITY ? v.y * exp2_fast((v.x - top) * f) : 0.f;
#pragma unroll
  for (int o = 16; o; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return make_float2(top, sum);
}

// 16 bytes of logits as they are: their largest (a NaN is no number), and the sum of exp2(f (v - top)).
template <typename T>
__device__ __forceinline__ float largest(const uint4& raw, float top);
template <>
__device__ __forceinline__ float largest<float>(const uint4& raw, float top) {
  return fmaxf(fmaxf(fmaxf(__uint_as_float(raw.x), __uint_as_float(raw.y)), fmaxf(__uint_as_float(raw.z), __uint_as_float(raw.w))), top);
}
template <>
__device__ __forceinline__ float largest<__nv_bfloat16>(const uint4& raw, float top) {
  const __nv_bfloat162* v = reinterpret_cast<const __nv_bfloat162*>(&raw);
  const __nv_bfloat162 m = __hmax2(__hmax2(v[0], v[1]), __hmax2(v[2], v[3]));
  return fmaxf(fmaxf(__low2float(m), __high2float(m)), top);
}
__device__ __forceinline__ uint64_t exp_pair(uint64_t v, uint64_t minus_top, uint64_t f, uint64_t sum) {
  float lo, hi;
  unpack2(mul2(add2(v, minus_top), f), lo, hi);
  return add2(sum, pack2(exp2_fast(lo), exp2_fast(hi)));
}
template <typename T>
__device__ __forceinline__ uint64_t exp_sum(const uint4& raw, uint64_t minus_top, uint64_t f, uint64_t sum) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; i += sizeof(T) / 2) {
    const uint64_t v = sizeof(T) == 2 ? pack2(bf16_lo(w[i]), bf16_hi(w[i])) : pack2(__uint_as_float(w[i]), __uint_as_float(w[(i + 1) & 3]));
    sum = exp_pair(v, minus_top, f, sum);
  }
  return sum;
}

// The maximum and the sum of exponentials (of the scaled differences from it) of one piece of a row.
// Pieces are counted from the 16-byte boundary at or before the row, so that all loads but those at the
// row's ends are vectors whatever its alignment.  A thread keeps a maximum of its own, so the block's
// threads meet once a piece, and has the next vectors on their way while it takes the present ones.  NaN
// and +infinity make its sum no number: then it goes over its logits once more, with their replacements.
template <typename T, int kVecs>
__global__ void __launch_bounds__(kThreads) verify_sums_kernel(VerifyParams p) {
  constexpr int kE = 16 / sizeof(T), kStep = kVecs * kThreads * kE;
  __shared__ float2 s_part[kThreads / 32];
  begin_kernel();
  const int64_t b = blockIdx.z;
  const int row = blockIdx.y, tid = threadIdx.x;
  const float scale = scale_of(p, b);
  const int count = count_of(p, b);
  if (!usable(scale) || (row <= p.T ? row > count : row - p.T - 1 >= count)) return;
  const T* base = row <= p.T ? static_cast<const T*>(p.logits) + b * p.logits_batch + row * p.logits_row
                             : static_cast<const T*>(p.draft_logits) + b * p.draft_batch + (row - p.T - 1) * p.draft_row;
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(base) & 15) / sizeof(T));
  base -= off;
  const int last = off + p.V;
  const int begin = blockIdx.x * p.piece, end = begin + p.piece < last ? begin + p.piece : last;
  const float f = scale * kLog2e;
  const uint32_t none = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;  // -infinity
  uint4 next[kVecs];
  auto load = [&](int at0) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int at = at0 + (i * kThreads + tid) * kE;
      if (at >= off && at + kE <= last) {
        next[i] = *reinterpret_cast<const uint4*>(base + at);
      } else {
        next[i] = make_uint4(none, none, none, none);
        if (at < last)  // at an end of the row
#pragma unroll
          for (int e = 0; e < kE; ++e)
            if (at + e >= off && at + e < last) reinterpret_cast<T*>(&next[i])[e] = base[at + e];
      }
    }
  };
  const uint64_t f2 = pack2(f, f);
  float top = -INFINITY;
  uint64_t sum2 = 0;
  load(begin);
  for (int at0 = begin; at0 < end; at0 += kStep) {
    uint4 now[kVecs];
    float high = top;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) now[i] = next[i], high = largest<T>(now[i], high);
    if (at0 + kStep < end) load(at0 + kStep);
    if (high > top) {
      const float less = exp2_fast((top - high) * f);
      sum2 = mul2(sum2, pack2(less, less)), top = high;
    }
    if (top > -INFINITY) {
      const uint64_t minus_top = pack2(-top, -top);
#pragma unroll
      for (int i = 0; i < kVecs; ++i) sum2 = exp_sum<T>(now[i], minus_top, f2, sum2);
    }
  }
  float lo, hi;
  unpack2(sum2, lo, hi);
  float sum = lo + hi;
  if (!(sum < INFINITY)) {
    top = -INFINITY, sum = 0.f;
    for (int pass = 0; pass < 2; ++pass)
      for (int at0 = begin; at0 < end; at0 += kStep)
        for (int i = 0; i < kVecs; ++i)
          for (int e = 0; e < kE; ++e) {
            const int at = at0 + (i * kThreads + tid) * kE + e;
            if (at < off || at >= last) continue;
            const float v = plain_logit(to_f32(base[at]));
            if (pass == 0)
              top = fmaxf(top, v);
            else if (v > -INFINITY)
              sum += exp2_fast((v - top) * f);
          }
  }
  const float2 all = join_sums(make_float2(top, sum), f);
  if ((tid & 31) == 0) s_part[tid >> 5] = all;
  __syncthreads();
  if (tid < 32) {
    const float2 piece = join_sums(tid < kThreads / 32 ? s_part[tid] : make_float2(-INFINITY, 0.f), f);
    if (tid == 0) p.sums[(b * p.rows + row) * p.pieces + blockIdx.x] = piece;
  }
}

// ------------------------------------------------------------------ exact weights

constexpr int kPowerBits = 8;
constexpr int kPowers = 1 << kPowerBits;

// 2^(i/16) and 2^(i/256) in two parts.
__device__ const float2 kCoarse[16] = {
    {0x1.000000p+0f, 0x0.0p+0f}, {0x1.0b5586p+0f, 0x1.9f3122p-25f}, {0x1.172b84p+0f, -0x1.c15742p-27f}, {0x1.2387a6p+0f, 0x1.ceac48p-25f},
    {0x1.306fe0p+0f, 0x1.4636e2p-25f}, {0x1.3dea64p+0f, 0x1.824684p-25f}, {0x1.4bfdaep+0f, -0x1.593abcp-25f}, {0x1.5ab07ep+0f, -0x1.5bd5ecp-27f},
    {0x1.6a09e6p+0f, 0x1.9fcef4p-26f}, {0x1.7a1148p+0f, -0x1.829fd0p-25f}, {0x1.8ace54p+0f, 0x1.15506ep-27f}, {0x1.9c4918p+0f, 0x1.51f848p-27f},
    {0x1.ae89fap+0f, -0x1.a94b14p-26f}, {0x1.c199bep+0f, -0x1.3d56b2p-27f}, {0x1.d5818ep+0f, -0x1.822dbcp-27f}, {0x1.ea4afap+0f, 0x1.52486cp-27f},
};
__device__ const float2 kFine[16] = {
    {0x1.000000p+0f, 0x0.0p+0f}, {0x1.00b1b0p+0f, -0x1.6950d0p-26f}, {0x1.0163dap+0f, 0x1.3f6666p-25f}, {0x1.021682p+0f, -0x1.789fb0p-25f},
    {0x1.02c9a4p+0f, -0x1.887fa0p-28f}, {0x1.037d42p+0f, 0x1.c2377ap-25f}, {0x1.04315ep+0f, 0x1.0dcff0p-25f}, {0x1.04e5f8p+0f, -0x1.a1356ap-25f},
    {0x1.059b0ep+0f, -0x1.9d4f52p-25f}, {0x1.0650a0p+0f, 0x1.c783f2p-25f}, {0x1.0706b2p+0f, 0x1.3bbedcp-25f}, {0x1.07bd42p+0f, 0x1.6e5506p-25f},
    {0x1.087452p+0f, -0x1.e2990ep-26f}, {0x1.092be0p+0f, -0x1.333f04p-25f}, {0x1.09e3ecp+0f, 0x1.58de70p-25f}, {0x1.0a9c7ap+0f, -0x1.3831bap-26f},
};

// What the exponentials of a row take: its maximum, and scale * log2(e) in two parts.
struct Row {
  float top, fh, fl;
};

// exp(scale * (x - top)): in two 32-bit parts to 2^-38 of it, and as the whole number (high 2^22 + low)
// of units, still as the bits of 3 + high 2^-22 and 3 2^-22 + low 2^-44 (whose last places those are, so
// that adding up bits adds up the numbers).  With z = scale * log2(e) * (x - top) in two parts and k the
// nearest whole number to 256 z it is 2^(k/256) exp(y), y = (z - k/256) ln 2, |y| < 0.0014, by the
// series of exp; 2^(k/256) in two parts from a table.  z is cut off at -64, where no unit is left.
// Both passes have to form the same number, so no sum here may be contracted in one and not in the other.
struct Weight {
  float value;
  int high, low;
};
constexpr float kHigh = 3.f, kLow = 0x1.8p-21f;
__device__ __forceinline__ Weight weight_of(float v, const Row& r, const float2* powers) {
  const float x = fminf(fmaxf(v, -INFINITY), r.top);  // (a NaN is -infinity, +infinity the maximum)
  const float dh = x - r.top;
  const float zh = fmaxf(__fmul_rn(dh, r.fh), -64.f);
  const float back = dh - x;
  const float dl = (x - (dh - back)) + (-r.top - back);  // what the difference lost (Knuth's sum)
  float zl = fmaf(dl, r.fh, fmaf(dh, r.fl, fmaf(dh, r.fh, -zh)));
  if (!(zh > -64.f)) zl = 0.f;
  const float shifted = fmaf(zh, kPowers, 12582912.f);  // 1.5 * 2^23: the nearest whole number in the low bits
  const int k = __float_as_int(shifted);                // of which the high bits fall out of both uses
  const float near = fmaf(shifted - 12582912.f, -1.f / kPowers, zh);
  const float rest = near + zl;  // (zl can be 2^-19, too much for the series to leave out its products)
  const float restl = zl - (rest - near);
  constexpr float kLn2h = 0x1.62e43p-1f, kLn2l = -0x1.05c61p-29f;
  const float yh = __fmul_rn(rest, kLn2h);
  const float yl = fmaf(restl, kLn2h, fmaf(rest, kLn2l, fmaf(rest, kLn2h, -yh)));
  const float q = fmaf(__fmul_rn(yh, yh), fmaf(yh, 1.f / 6, 0.5f), yl);  // exp(y) - 1 = yh + q
  const float2 power = powers[k & (kPowers - 1)];
  const float eh = fmaf(power.x, yh + q, power.x);
  const float el = fmaf(power.y, yh, fmaf(power.x, q, fmaf(power.x, yh, power.x - eh))) + power.y;  // what that lost
  const float f = __int_as_float(((k >> kPowerBits) << 23) + 0x3F800000);  // 2^(k / 256), at least 2^-64
  Weight w;
  w.value = __fmul_rn(eh, f);
  const float high = w.value + kHigh;
  w.high = __float_as_int(high);
  w.low = __float_as_int(fmaf(el, f, w.value - (high - kHigh)) + kLow);
  return w;
}

// A sum of weights: bits are added up for a few, then taken into 64 bits.
struct Sum {
  uint64_t all = 0;
  uint32_t high = 0, low = 0;
  __device__ __forceinline__ void add(const Weight& w) { high += w.high, low += w.low; }
  __device__ __forceinline__ void take(uint32_t count) {  // of the weights added, 256 at most
    all += (static_cast<int64_t>(static_cast<int32_t>(high - count * 0x40400000u)) << 22) +
           static_cast<int32_t>(low - count * static_cast<uint32_t>(0x35400000));
    high = low = 0;
  }
};
__device__ __forceinline__ uint64_t units_of(const Weight& w) {
  return (static_cast<int64_t>(w.high - 0x40400000) << 22) + (w.low - 0x35400000);
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int o = 16; o; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ uint64_t warp_scan(uint64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const uint64_t other = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += other;
  }
  return v;
}

// A probability in units of 2^-61: weights over the sum of all (Z), multiplied by 2^125 / (Z 2^shift),
// where Z 2^shift is at least 2^62 and at most 2^63.
struct Share {
  uint64_t inv;
  int shift;
  __device__ __forceinline__ uint64_t operator()(uint64_t sum) const { return __umul64hi(sum << shift, inv); }
};
__device__ __forceinline__ Share share_of(uint64_t all) {
  Share s{0, 0};
  if (all == 0) return s;
  s.shift = max(__clzll(static_cast<long long>(all)) - 1, 0);
  s.inv = static_cast<uint64_t>(0x1p125 / static_cast<double>(all << s.shift));
  return s;
}

// floor(r * total) for r in [0, 1), and total - 1 at most.
__device__ __forceinline__ uint64_t goal_of(float r, uint64_t total) {
  if (!(r > 0.f)) return 0;
  int e;
  const float m = frexpf(fminf(r, 0.99999994f), &e);  // r = m 2^e, m a multiple of 2^-24
  if (-e >= 64) return 0;
  return __umul64hi(static_cast<uint64_t>(m * 16777216.f) << 40, total) >> -e;
}

// The row that is drawn from: max(p - q, 0).  Which of the two is larger goes by their 32-bit values and
// sums: it is uncertain only where they are equal to 2^-20, and then it matters as little, unless all tokens'
// differences add up to no more than that: a draft is refused there for one number in 2^20 only, as many as may
// fall either way.  (A second pass with the exact sums for such rows: 32 x 7 x 131072 54 -> 55.6 us.)
struct Draw {
  Row target, draft;
  float ratio;  // sum of the target's exponentials over the draft's
  int minus;    // 0: p itself; 1: less the draft row; 2: less one token
  int token;    // that token
};

// Eight neighbouring logits, as they are until they are used; those behind the row are -infinity.
template <typename T>
struct Eight {
  uint4 raw[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* row, int v, int n, bool vec) {
    if (vec && n >= 8) {
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) raw[i] = reinterpret_cast<const uint4*>(row + v)[i];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) reinterpret_cast<T*>(raw)[e] = e < n ? row[v + e] : from_f32<T>(-INFINITY);
    }
  }
  __device__ __forceinline__ float operator[](int e) const { return to_f32(reinterpret_cast<const T*>(raw)[e]); }
};

// A run's sums: all of p and of q, and both where p is the larger.
enum { kAllP, kAllQ, kMoreP, kMoreQ, kSums };
__device__ __forceinline__ uint64_t rest_of(const uint64_t (&run)[kSums], bool plain, const Share& p, const Share& q) {
  if (plain) return p(run[kAllP]);
  const uint64_t more = p(run[kMoreP]), less = q(run[kMoreQ]);
  return more > less ? more - less : 0;
}

template <typename T>
__global__ void __launch_bounds__(kDrawThreads, 2) verify_draw_kernel(VerifyParams p) {
  constexpr int kMaxRuns = kMaxCluster * kDrawWarps;
  __shared__ float2 s_row[2 * kMaxDrafts + 1];  // maximum and sum of every row
  __shared__ float2 s_powers[kPowers];
  __shared__ uint64_t s_mine[kDrawWarps][kSums];  // of the block's runs
  __shared__ uint64_t s_run[kMaxRuns][kSums];     // of all
  __shared__ Share s_share[2];
  __shared__ uint64_t s_upto[2][kDrawWarps];
  __shared__ uint32_t s_taken[kMaxDrafts / 32];
  __shared__ uint64_t s_below;
  __shared__ int s_which, s_plain, s_found;
  begin_kernel();
  cg::cluster_group cluster = cg::this_cluster();
  const int64_t b = blockIdx.y;
  const int part = blockIdx.x, runs = gridDim.x * kDrawWarps;  // a cluster is a row of the grid
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float scale = scale_of(p, b);
  int32_t* tokens = p.tokens + b * (p.T + 1);
  float* logprobs = p.logprobs + b * (p.T + 1);
  if (!usable(scale)) {  // (the whole cluster alike)
    if (part == 0) {
      for (int i = tid; i <= p.T; i += kDrawThreads) tokens[i] = -1, logprobs[i] = 0.f;
      if (tid == 0) p.accepted[b] = 0;
    }
    return;
  }
  const int count = count_of(p, b);
  const bool probs = p.draft_logits != nullptr;
  const T* target = static_cast<const T*>(p.logits) + b * p.logits_batch;
  const T* drafts = static_cast<const T*>(p.draft_logits) + b * p.draft_batch;
  const int32_t* draft = p.draft + b * p.T;
  const float* u = p.uniforms + b * (p.T + 1);
  if (tid < kPowers) {  // 2^(tid / 256), a product of two parts each
    const float2 a = kCoarse[tid >> 4], c = kFine[tid & 15];
    const float h = a.x * c.x, l = fmaf(a.x, c.x, -h) + fmaf(a.x, c.y, a.y * c.x);
    s_powers[tid] = make_float2(h + l, l - ((h + l) - h));
  }

  // the drafts, one a thread: what they take is on its way while the rows' sums are joined
  int d = -1;
  float number = 0.f, logit = 0.f, logit_q = 0.f;
  if (tid < count) {
    d = draft[tid], number = u[tid];
    if (d >= 0 && d < p.V) {
      logit = to_f32(target[tid * p.logits_row + d]);
      if (probs) logit_q = to_f32(drafts[tid * p.draft_row + d]);
    }
  }
  // the rows' sums
  const float f = scale * kLog2e;
  for (int j = warp; j < p.rows; j += kDrawWarps) {
    if (j <= p.T ? j > count : j - p.T - 1 >= count) continue;
    const float2* from = p.sums + (b * p.rows + j) * p.pieces;
    float2 v = make_float2(-INFINITY, 0.f);
    for (int i = lane; i < p.pieces; i += 32) {
      const float2 w = from[i];
      if (w.x > v.x)
        v = make_float2(w.x, fmaf(v.y, exp2_fast((v.x - w.x) * f), w.y));
      else if (w.x > -INFINITY)
        v.y = fmaf(w.y, exp2_fast((w.x - v.x) * f), v.y);
    }
    v = join_sums(v, f);
    if (lane == 0) s_row[j] = v;
  }
  __syncthreads();
  float logp = 0.f;
  if (tid < kMaxDrafts) {
    bool taken = false;
    if (tid < count) {
      const float2 t = s_row[tid];
      if (d >= 0 && d < p.V && t.y > 0.f) {
        const float z = scale * (plain_logit(logit) - t.x);
        logp = z - logf(t.y);
        float zq = 0.f, sum_q = 1.f;
        if (probs) {
          const float2 r = s_row[p.T + 1 + tid];
          zq = -INFINITY;
          if (r.y > 0.f) zq = scale * (plain_logit(logit_q) - r.x), sum_q = r.y;
        }
        // from the larger of the two, so that neither is lost where both are small; and p itself is above 0 where its
        // exponential is not
        const float top = fmaxf(z, zq);
        if (top > -INFINITY) taken = number * expf(zq - top) * t.y < expf(z - top) * sum_q;
        if (number == 0.f) taken = z > -INFINITY;
      }
    }
    const uint32_t mask = __ballot_sync(0xffffffffu, taken);
    if (lane == 0) s_taken[warp] = mask;
  }
  __syncthreads();
  int n = __ffs(~s_taken[0]) - 1;
  if (n < 0) n = 32 + (~s_taken[1] ? __ffs(~s_taken[1]) - 1 : 32);
  if (part == 0) {
    if (tid < n) tokens[tid] = d, logprobs[tid] = logp;
    for (int i = n + 1 + tid; i <= p.T; i += kDrawThreads) tokens[i] = -1, logprobs[i] = 0.f;
    if (tid == 0) p.accepted[b] = n;
  }
  const float2 t = s_row[n];
  if (!(t.y > 0.f)) {  // the target allows no token (the whole cluster alike)
    if (part == 0 && tid == 0) tokens[n] = -1, logprobs[n] = 0.f;
    return;
  }

  // what is drawn from
  Draw rest{};
  rest.target.top = t.x;
  rest.target.fh = rest.draft.fh = f;
  rest.target.fl = rest.draft.fl = fmaf(scale, kLog2e, -f) + scale * kLog2eLow;
  rest.token = -1;
  if (n < count) {
    const float2 r = s_row[probs ? p.T + 1 + n : n];
    if (!probs) {
      rest.minus = 2, rest.token = draft[n];
    } else if (r.y > 0.f) {
      rest.minus = 1, rest.ratio = t.y / r.y;
      rest.draft.top = r.x;
    }
  }
  const T* row = target + n * p.logits_row;
  const T* row_q = rest.minus == 1 ? drafts + n * p.draft_row : row;
  const bool vec = (reinterpret_cast<uintptr_t>(row) & 15) == 0, vec_q = (reinterpret_cast<uintptr_t>(row_q) & 15) == 0;

  // the sums of every warp's run of the vocabulary
  const int run = (p.V + runs * 256 - 1) / (runs * 256) * 256;
  {
    const int first = (part * kDrawWarps + warp) * run;  // (below 2^20)
    const int end = first >= p.V ? first : p.V - first < run ? p.V : first + run;
    Sum sums[kSums];
    Eight<T> next, next_q;
    const int at = first + 8 * lane;
    if (at < end) {
      next.load(row, at, p.V - at, vec);
      if (rest.minus == 1) next_q.load(row_q, at, p.V - at, vec_q);
    }
    for (int v = at; v < end; v += 256) {
      const Eight<T> x = next, xq = next_q;
      if (v + 256 < end) {
        next.load(row, v + 256, p.V - v - 256, vec);
        if (rest.minus == 1) next_q.load(row_q, v + 256, p.V - v - 256, vec_q);
      }
      uint32_t more = 0;
      if (rest.minus == 1) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const Weight w = weight_of(x[e], rest.target, s_powers), q = weight_of(xq[e], rest.draft, s_powers);
          sums[kAllP].add(w), sums[kAllQ].add(q);
          if (w.value > q.value * rest.ratio) sums[kMoreP].add(w), sums[kMoreQ].add(q), ++more;
        }
        sums[kAllQ].take(8), sums[kMoreQ].take(more);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const Weight w = weight_of(x[e], rest.target, s_powers);
          sums[kAllP].add(w);
          if (v + e != rest.token) sums[kMoreP].add(w), ++more;
        }
      }
      sums[kAllP].take(8), sums[kMoreP].take(more);
    }
#pragma unroll
    for (int i = 0; i < kSums; ++i) {
      const uint64_t s = warp_sum(sums[i].all);
      if (lane == 0) s_mine[warp][i] = s;
    }
  }
  cluster_arrive(), cluster_wait();
  for (int i = tid; i < runs * kSums; i += kDrawThreads)
    (&s_run[0][0])[i] = cluster.map_shared_rank(&s_mine[0][0], i / (kDrawWarps * kSums))[i % (kDrawWarps * kSums)];
  cluster_arrive();  // (waited for at the end: nobody leaves while the others read its sums)
  __syncthreads();

  // the run that the random number hits
  if (warp == 0) {
    uint64_t sum[kSums];
    for (int i = 0; i < kSums; ++i) {
      sum[i] = 0;
      for (int r = lane; r < runs; r += 32) sum[i] += s_run[r][i];
      sum[i] = warp_sum(sum[i]);
    }
    const Share share = share_of(lane == 0 ? sum[kAllP] : sum[kAllQ]);
    if (lane < 2) s_share[lane] = share;
    // (the maximum alone weighs 2^44, so the sum is above 0 and one lane finds its run below; the search stays in
    // bounds without that)
    if (lane == 0) s_which = 0, s_below = 0, s_plain = true;
    __syncwarp();
    const Share share_p = s_share[0], share_q = s_share[1];
    // p itself where (next to) nothing is left of p - q: 2^-49, which the runs' roundings cannot use up
    const bool plain = rest.minus == 0 || share_p(sum[kMoreP]) <= share_q(sum[kMoreQ]) + 4096;
    const int each = (runs + 31) / 32, first = lane * each;  // a lane's runs
    uint64_t part_sum = 0;
    for (int r = first; r < first + each && r < runs; ++r) part_sum += rest_of(s_run[r], plain, share_p, share_q);
    const uint64_t upto = warp_scan(part_sum, lane);
    const uint64_t total = __shfl_sync(0xffffffffu, upto, 31);
    const uint64_t goal = goal_of(u[p.T], total);
    uint64_t below = upto - part_sum;
    if (goal >= below && goal < upto) {  // one lane's
      int r = first;
      for (; r + 1 < first + each; ++r) {
        const uint64_t more = rest_of(s_run[r], plain, share_p, share_q);
        if (goal - below < more) break;
        below += more;
      }
      s_which = r, s_below = goal - below, s_plain = plain;
    }
  }
  if (tid == 0) s_found = INT_MAX;
  __syncthreads();

  // and in it, the token
  if (s_which / kDrawWarps == part) {
    const int start = s_which * run;
    const int stop = p.V - start < run ? p.V : start + run;
    const bool plain = s_plain;
    const uint64_t goal = s_below;
    const Share share_p = s_share[0], share_q = s_share[1];
    uint64_t sum = 0, sum_q = 0;
    for (int v0 = start; v0 < stop; v0 += kDrawThreads) {
      const int v = v0 + tid;
      uint64_t w = 0, q = 0;
      if (v < stop) {
        const Weight wp = weight_of(to_f32(row[v]), rest.target, s_powers);
        if (plain || rest.minus == 0) {
          w = units_of(wp);
        } else if (rest.minus == 1) {
          const Weight wq = weight_of(to_f32(row_q[v]), rest.draft, s_powers);
          if (wp.value > wq.value * rest.ratio) w = units_of(wp), q = units_of(wq);
        } else if (v != rest.token) {
          w = units_of(wp);
        }
      }
      const uint64_t upto = warp_scan(w, lane), upto_q = warp_scan(q, lane);
      if (lane == 31) s_upto[0][warp] = upto, s_upto[1][warp] = upto_q;
      __syncthreads();
      uint64_t all = sum + upto, all_q = sum_q + upto_q;
      for (int i = 0; i < kDrawWarps; ++i) {
        if (i < warp) all += s_upto[0][i], all_q += s_upto[1][i];
        sum += s_upto[0][i], sum_q += s_upto[1][i];
      }
      if (v < stop && w > 0 && share_p(all) > goal + share_q(all_q)) atomicMin(&s_found, v);
      __syncthreads();
      if (s_found != INT_MAX) break;
    }
    if (tid == 0) {
      const int v = s_found != INT_MAX ? s_found : stop - 1;  // (the run's weights are above the goal)
      tokens[n] = v;
      logprobs[n] = scale * (plain_logit(to_f32(row[v])) - t.x) - logf(t.y);
    }
  }
  cluster_wait();
}

// Values of a piece: 4 vectors a thread four times over, or less as long as that leaves every
// multiprocessor fewer than eight blocks.
int piece_of(int64_t batch, int rows, int V, int dtype) {
  const int per = static_cast<int>(16 / elem_size(dtype)) * kThreads;
  int vecs = 16;
  while (vecs > 1 && batch * rows * ceil_div(V, static_cast<int64_t>(per) * vecs) < 8 * layer_sm_count()) vecs /= 2;
  return per * vecs;
}

template <typename T, int kVecs>
cudaError_t launch_sums(const VerifyParams& p, int64_t batch, cudaStream_t stream) {
  return launch_k(verify_sums_kernel<T, kVecs>, dim3(p.pieces, p.rows, static_cast<unsigned>(batch)), dim3(kThreads), 0, stream, true, p);
}

template <typename T>
cudaError_t launch_verify(const VerifyParams& p, int64_t batch, cudaStream_t stream) {
  const int vecs = p.piece * static_cast<int>(sizeof(T)) / (16 * kThreads);
  const cudaError_t e = vecs >= 4 ? launch_sums<T, 4>(p, batch, stream) : vecs == 2 ? launch_sums<T, 2>(p, batch, stream)
                                                                                    : launch_sums<T, 1>(p, batch, stream);
  if (e != cudaSuccess) return e;
  // as large a cluster a sequence as leaves all of them resident at once, two blocks a multiprocessor
  // (64 sequences of 50001 tokens: 8 blocks each 30 us, 4 26)
  int cluster = kMaxCluster;
  while (cluster > 1 && cluster * batch > 2 * layer_sm_count()) cluster /= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(cluster), static_cast<unsigned>(batch));
  cfg.blockDim = dim3(kDrawThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster), attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_draw_kernel<T>, p);
}

ssd_status check_verify(const ssd_draft_verify_args* a) {
  if (!a || a->size != static_cast<int64_t>(sizeof(*a))) return SSD_ERR_INVALID_ARG;
  if (a->batch < 0 || a->drafts < 0 || a->vocab <= 0) return SSD_ERR_INVALID_ARG;
  if (!known_dtype(a->dtype)) return SSD_ERR_UNSUPPORTED;
  if (a->batch > 65535 || a->drafts > kMaxDrafts || a->vocab > kMaxVocab) return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

int rows_of(const ssd_draft_verify_args* a) { return a->drafts + 1 + (a->draft_logits ? a->drafts : 0); }
int pieces_of(const ssd_draft_verify_args* a, int piece) {
  // (a row begins up to one vector after its 16-byte boundary)
  return static_cast<int>(ceil_div(a->vocab + static_cast<int64_t>(16 / elem_size(a->dtype)) - 1, piece));
}

}  // namespace
}  // namespace ssd

extern "C" size_t ssd_draft_verify_workspace_size(const ssd_draft_verify_args* a) {
  using namespace ssd;
  if (check_verify(a) != SSD_OK) return 0;
  return static_cast<size_t>(a->batch) * rows_of(a) * pieces_of(a, piece_of(a->batch, rows_of(a), a->vocab, a->dtype)) * sizeof(float2);
}

extern "C" ssd_status ssd_draft_verify(const ssd_draft_verify_args* a, ssd_stream_t stream) {
  using namespace ssd;
  const ssd_status st = check_verify(a);
  if (st != SSD_OK) return st;
  if (a->batch == 0) return SSD_OK;
  const size_t es = elem_size(a->dtype);
  if (!a->logits || !aligned_to(a->logits, es) || !aligned_to(a->draft_logits, es)) return SSD_ERR_INVALID_ARG;
  for (const void* t : {(const void*)a->uniforms, (const void*)a->tokens, (const void*)a->accepted, (const void*)a->logprobs})
    if (!t || !aligned_to(t, 4)) return SSD_ERR_INVALID_ARG;
  if ((a->drafts > 0 && !a->draft) || !aligned_to(a->draft, 4) || !aligned_to(a->scale, 4) || !aligned_to(a->lengths, 4))
    return SSD_ERR_INVALID_ARG;
  if (!a->workspace || !aligned_to(a->workspace, 16)) return SSD_ERR_INVALID_ARG;
  if (a->workspace_bytes < ssd_draft_verify_workspace_size(a)) return SSD_ERR_WORKSPACE;
  VerifyParams p{};
  p.logits_batch = a->logits_batch, p.logits_row = a->logits_row;
  p.draft_batch = a->draft_logits_batch, p.draft_row = a->draft_logits_row;
  p.T = a->drafts, p.V = a->vocab, p.rows = rows_of(a);
  p.piece = piece_of(a->batch, p.rows, p.V, a->dtype), p.pieces = pieces_of(a, p.piece);
  p.logits = a->logits, p.draft_logits = a->draft_logits;
  p.draft = a->draft, p.lengths = a->lengths, p.uniforms = a->uniforms, p.scale = a->scale;
  p.sums = static_cast<float2*>(a->workspace);
  p.tokens = a->tokens, p.accepted = a->accepted, p.logprobs = a->logprobs;
  return launched(a->dtype == SSD_BF16 ? launch_verify<__nv_bfloat16>(p, a->batch, stream)
                                       : launch_verify<float>(p, a->batch, stream));
}
