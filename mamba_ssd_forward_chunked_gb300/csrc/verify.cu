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
// row's exponentials are formed in two 32-bit parts, to 2^-38, and summed as
// whole numbers: sums do not depend on their order, and the token is the one
// that 64-bit arithmetic finds.
#include <cooperative_groups.h>

#include "layer.cuh"

namespace ssd {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kMaxDrafts = 64;
constexpr int kCluster = 8;
constexpr int kDrawThreads = 512;
constexpr int kDrawWarps = kDrawThreads / 32;

struct VerifyParams {
  int64_t logits_batch, logits_row, draft_batch, draft_row;
  int T, V, rows, pieces, piece, bits;  // bits: of a sum's unit, 2^-bits
  const void *logits, *draft_logits;
  const int32_t *draft, *lengths;
  const float *uniforms, *scale;
  float2* sums;  // [batch][rows][pieces]; rows: the target's T + 1, then the draft's T
  int32_t *tokens, *accepted;
  float* logprobs;
};

__device__ __forceinline__ float scale_of(const VerifyParams& p, int64_t b) { return p.scale ? p.scale[b] : 1.f; }
__device__ __forceinline__ bool usable(float scale) { return scale > 0.f && scale < INFINITY; }
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

// The maximum and the sum of exponentials (of the scaled differences from it) of one piece of a row.
// Pieces are counted from the 16-byte boundary at or before the row, so that all loads but those at the
// row's ends are vectors whatever its alignment.
template <typename T, int kVecs>
__global__ void __launch_bounds__(kThreads) verify_sums_kernel(VerifyParams p) {
  constexpr int kE = 16 / sizeof(T);
  __shared__ float s_part[kThreads / 32], s_max;
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
  float v[kVecs][kE];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int64_t at = static_cast<int64_t>(blockIdx.x) * p.piece + (i * kThreads + tid) * kE;
    if (at >= off && at + kE <= off + p.V) {
      load_vector(base + at, v[i]);
    } else {
#pragma unroll
      for (int e = 0; e < kE; ++e) v[i][e] = at + e >= off && at + e < off + p.V ? to_f32(base[at + e]) : -INFINITY;
    }
  }
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
#pragma unroll
    for (int e = 0; e < kE; ++e) v[i][e] = plain_logit(v[i][e]), top = fmaxf(top, v[i][e]);
#pragma unroll
  for (int o = 16; o; o /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((tid & 31) == 0) s_part[tid >> 5] = top;
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < kThreads / 32; ++i) top = fmaxf(top, s_part[i]);
    s_max = top;
  }
  __syncthreads();
  top = s_max;
  float sum = 0.f;
  if (top > -INFINITY) {
    const float f = scale * kLog2e;
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
      for (int e = 0; e < kE; ++e) sum += exp2_fast((v[i][e] - top) * f);
  }
#pragma unroll
  for (int o = 16; o; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((tid & 31) == 0) s_part[tid >> 5] = sum;
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < kThreads / 32; ++i) sum += s_part[i];
    p.sums[(b * p.rows + row) * p.pieces + blockIdx.x] = make_float2(top, sum);
  }
}

// ------------------------------------------------------------------ exact weights

// 2^(i/32) in two parts.
__device__ __constant__ float2 kPowers[32] = {
    {0x1.000000p+0f, 0x0.0p+0f}, {0x1.059b0ep+0f, -0x1.9d4f52p-25f}, {0x1.0b5586p+0f, 0x1.9f3122p-25f}, {0x1.11301ep+0f, -0x1.fdb496p-25f},
    {0x1.172b84p+0f, -0x1.c15742p-27f}, {0x1.1d4874p+0f, -0x1.d2e8cap-25f}, {0x1.2387a6p+0f, 0x1.ceac48p-25f}, {0x1.29e9e0p+0f, -0x1.5c0424p-25f},
    {0x1.306fe0p+0f, 0x1.4636e2p-25f}, {0x1.371a74p+0f, -0x1.18aac6p-25f}, {0x1.3dea64p+0f, 0x1.824684p-25f}, {0x1.44e086p+0f, 0x1.8624b4p-30f},
    {0x1.4bfdaep+0f, -0x1.593abcp-25f}, {0x1.5342b6p+0f, -0x1.2c5610p-25f}, {0x1.5ab07ep+0f, -0x1.5bd5ecp-27f}, {0x1.6247ecp+0f, -0x1.f8b550p-25f},
    {0x1.6a09e6p+0f, 0x1.9fcef4p-26f}, {0x1.71f75ep+0f, 0x1.1d8beep-25f}, {0x1.7a1148p+0f, -0x1.829fd0p-25f}, {0x1.82589ap+0f, -0x1.accc7cp-26f},
    {0x1.8ace54p+0f, 0x1.15506ep-27f}, {0x1.93737cp+0f, -0x1.e64744p-25f}, {0x1.9c4918p+0f, 0x1.51f848p-27f}, {0x1.a5503cp+0f, -0x1.b83b54p-25f},
    {0x1.ae89fap+0f, -0x1.a94b14p-26f}, {0x1.b7f770p+0f, -0x1.a09438p-25f}, {0x1.c199bep+0f, -0x1.3d56b2p-27f}, {0x1.cb720ep+0f, -0x1.8837ccp-27f},
    {0x1.d5818ep+0f, -0x1.822dbcp-27f}, {0x1.dfc974p+0f, -0x1.908c94p-25f}, {0x1.ea4afap+0f, 0x1.52486cp-27f}, {0x1.f50766p+0f, -0x1.246eb0p-26f},
};

// What the exponentials of a row take: its maximum, scale * log2(e) in two parts, and the exponent
// below which a weight is less than half a unit.
struct Row {
  float top, fh, fl, low;
};

// exp(scale * (x - top)) * 2^bits as a whole number, off by 2^-38 of it and one unit.  With
// z = scale * log2(e) * (x - top) in two parts and k the nearest whole number to 32 z, it is
// 2^(k/32) exp(y), y = (z - k/32) ln 2, |y| < 0.011, by the series of exp.
__device__ __forceinline__ uint64_t weight(float x, const Row& r, const float2* powers, int bits) {
  const float dh = x - r.top;  // the difference in two parts (Knuth)
  const float back = dh - x;
  const float dl = (x - (dh - back)) + (-r.top - back);
  const float zh = dh * r.fh;
  if (!(zh > r.low)) return 0;  // (and where x is -infinity)
  const float zl = fmaf(dl, r.fh, fmaf(dh, r.fl, fmaf(dh, r.fh, -zh)));
  const float shifted = fmaf(zh, 32.f, 12582912.f);  // 1.5 * 2^23: the nearest whole number in the low bits
  const int k = __float_as_int(shifted) - 0x4B400000;
  const float rest = fmaf(shifted - 12582912.f, -0.03125f, zh);
  constexpr float kLn2h = 0x1.62e43p-1f, kLn2l = -0x1.05c61p-29f;
  const float yh = rest * kLn2h;
  const float yl = fmaf(zl, kLn2h, fmaf(rest, kLn2l, fmaf(rest, kLn2h, -yh)));
  const float c = fmaf(yh, fmaf(yh, fmaf(yh, 1.f / 120, 1.f / 24), 1.f / 6), 0.5f);
  const float q = fmaf(yh * yh, c, yl);  // exp(y) - 1 = yh + q
  const float2 power = powers[k & 31];
  const float ph = power.x * yh;
  const float pl = fmaf(power.y, yh, fmaf(power.x, q, fmaf(power.x, yh, -ph))) + power.y;
  const float eh = power.x + ph;
  const float el = (ph - (eh - power.x)) + pl;
  const int64_t whole = (static_cast<int64_t>(__float2int_rn(eh * 16777216.f)) << 24) + __float2int_rn(el * 0x1p48f);
  const int shift = 48 - bits - (k >> 5);  // 2 to 50
  return (static_cast<uint64_t>(whole) + (uint64_t(1) << (shift - 1))) >> shift;
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int o = 16; o; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The row that is drawn from: the target's weights, less the draft's.
struct Draw {
  Row target, draft;
  uint64_t inv_target, inv_draft;  // 2^(63 + bits) / sum of weights: a probability is weight * inv / 2^63
  int minus;                       // 0: p itself; 1: less the draft row; 2: less one token
  int token;                       // that token
};
// max(p - q, 0) of token v in units of 2^-62.
__device__ __forceinline__ uint64_t rest_of(const Draw& d, int v, float x, float xq, const float2* powers, int bits) {
  const uint64_t pw = __umul64hi(weight(x, d.target, powers, bits) << (63 - bits), d.inv_target);
  if (d.minus == 2) return v == d.token ? 0 : pw;
  if (d.minus == 0) return pw;
  const uint64_t qw = __umul64hi(weight(xq, d.draft, powers, bits) << (63 - bits), d.inv_draft);
  return pw > qw ? pw - qw : 0;
}

template <typename T>
__device__ __forceinline__ void load_run(const T* row, int v, int n, bool vec, float (&out)[8]) {
  if (vec && n >= 8) {
    if constexpr (sizeof(T) == 2) {
      load_vector(row + v, out);
    } else {
      float a[4], c[4];
      load_vector(row + v, a), load_vector(row + v + 4, c);
#pragma unroll
      for (int e = 0; e < 4; ++e) out[e] = a[e], out[4 + e] = c[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = e < n ? to_f32(row[v + e]) : -INFINITY;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) out[e] = plain_logit(out[e]);
}

template <typename T>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kDrawThreads) verify_draw_kernel(VerifyParams p) {
  __shared__ float2 s_row[2 * kMaxDrafts + 1];  // maximum and sum of every row
  __shared__ float2 s_powers[32];
  __shared__ uint64_t s_warp[2][kDrawWarps];
  __shared__ uint64_t s_sum[2], s_rest, s_before, s_total;
  __shared__ int s_taken[kMaxDrafts];
  __shared__ uint64_t s_scan[kDrawWarps];
  begin_kernel();
  cg::cluster_group cluster = cg::this_cluster();
  const int64_t b = blockIdx.y;
  const int part = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
  if (tid < 32) s_powers[tid] = kPowers[tid];

  // the rows' sums
  const float f = scale * kLog2e;
  for (int j = warp; j < p.rows; j += kDrawWarps) {
    if (j <= p.T ? j > count : j - p.T - 1 >= count) continue;
    const float2* from = p.sums + (b * p.rows + j) * p.pieces;
    float top = -INFINITY, sum = 0.f;
    for (int i = lane; i < p.pieces; i += 32) top = fmaxf(top, from[i].x);
#pragma unroll
    for (int o = 16; o; o /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (top > -INFINITY)
      for (int i = lane; i < p.pieces; i += 32) {
        const float2 v = from[i];
        sum = fmaf(v.y, exp2_fast((v.x - top) * f), sum);
      }
#pragma unroll
    for (int o = 16; o; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s_row[j] = make_float2(top, sum);
  }
  __syncthreads();
  // the drafts, one a thread
  float logp = 0.f;
  if (tid < count) {
    const int d = draft[tid];
    const float2 t = s_row[tid];
    float ep = 0.f, eq = 0.f, zq = 1.f;
    if (d >= 0 && d < p.V) {
      if (t.y > 0.f) {
        const float z = scale * (plain_logit(to_f32(target[tid * p.logits_row + d])) - t.x);
        ep = expf(z), logp = z - logf(t.y);
      }
      eq = 1.f;
      if (probs) {
        const float2 r = s_row[p.T + 1 + tid];
        eq = 0.f;
        if (r.y > 0.f) eq = expf(scale * (plain_logit(to_f32(drafts[tid * p.draft_row + d])) - r.x)), zq = r.y;
      }
    }
    s_taken[tid] = u[tid] * eq * t.y < ep * zq;
  }
  __syncthreads();
  int n = 0;
  while (n < count && s_taken[n]) ++n;
  if (part == 0) {
    if (tid < n) tokens[tid] = draft[tid], logprobs[tid] = logp;
    for (int i = n + 1 + tid; i <= p.T; i += kDrawThreads) tokens[i] = -1, logprobs[i] = 0.f;
    if (tid == 0) p.accepted[b] = n;
  }
  const float2 t = s_row[n];
  if (!(t.y > 0.f)) {  // the target allows no token (the whole cluster alike)
    if (part == 0 && tid == 0) tokens[n] = -1, logprobs[n] = 0.f;
    return;
  }

  // the sums of the drawing rows' weights
  Draw d{};
  const double factor = static_cast<double>(scale) * 1.4426950408889634;
  d.target.fh = d.draft.fh = static_cast<float>(factor);
  d.target.fl = d.draft.fl = static_cast<float>(factor - d.target.fh);
  d.target.low = d.draft.low = -static_cast<float>(p.bits + 1);
  d.target.top = t.x;
  d.token = -1;
  if (n < count) {
    if (!probs) {
      d.minus = 2, d.token = draft[n];
    } else if (s_row[p.T + 1 + n].y > 0.f) {
      d.minus = 1, d.draft.top = s_row[p.T + 1 + n].x;
    }
  }
  const T* row = target + n * p.logits_row;
  const T* row_q = d.minus == 1 ? drafts + n * p.draft_row : row;
  const bool vec = (reinterpret_cast<uintptr_t>(row) & 15) == 0, vec_q = (reinterpret_cast<uintptr_t>(row_q) & 15) == 0;
  // a block has a run of the vocabulary, a warp a run of the block's
  const int run = static_cast<int>((static_cast<int64_t>(p.V) + kCluster * kDrawWarps * 256 - 1) / (kCluster * kDrawWarps * 256)) * 256;
  const int first = (part * kDrawWarps + warp) * run;
  const int end = first >= p.V ? first : p.V - first < run ? p.V : first + run;
  uint64_t sum = 0, sum_q = 0;
  for (int v = first + 8 * lane; v < end; v += 256) {
    float x[8];
    load_run(row, v, p.V - v, vec, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += weight(x[e], d.target, s_powers, p.bits);
    if (d.minus == 1) {
      load_run(row_q, v, p.V - v, vec_q, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum_q += weight(x[e], d.draft, s_powers, p.bits);
    }
  }
  sum = warp_sum(sum), sum_q = warp_sum(sum_q);
  if (lane == 0) s_warp[0][warp] = sum, s_warp[1][warp] = sum_q;
  __syncthreads();
  if (tid < 2) {
    uint64_t s = 0;
    for (int i = 0; i < kDrawWarps; ++i) s += s_warp[tid][i];
    s_sum[tid] = s;
  }
  cluster.sync();
  uint64_t all[2] = {0, 0};
  for (int r = 0; r < kCluster; ++r) {
    const uint64_t* theirs = cluster.map_shared_rank(s_sum, r);
    all[0] += theirs[0], all[1] += theirs[1];
  }
  d.inv_target = static_cast<uint64_t>(exp2(63.0 + p.bits) / static_cast<double>(all[0]));
  d.inv_draft = all[1] ? static_cast<uint64_t>(exp2(63.0 + p.bits) / static_cast<double>(all[1])) : 0;

  // what is drawn from: p - q, or p where nothing of that is left
  for (;;) {
    uint64_t rest = 0;
    for (int v = first + 8 * lane; v < end; v += 256) {
      float x[8], xq[8] = {};
      load_run(row, v, p.V - v, vec, x);
      if (d.minus == 1) load_run(row_q, v, p.V - v, vec_q, xq);
#pragma unroll
      for (int e = 0; e < 8; ++e) rest += rest_of(d, v + e, x[e], xq[e], s_powers, p.bits);
    }
    rest = warp_sum(rest);
    if (lane == 0) s_scan[warp] = rest;
    __syncthreads();
    if (tid == 0) {
      uint64_t s = 0;
      for (int i = 0; i < kDrawWarps; ++i) s += s_scan[i];
      s_rest = s;
    }
    cluster.sync();
    if (tid == 0) {
      uint64_t before = 0, total = 0;
      for (int r = 0; r < kCluster; ++r) {
        const uint64_t theirs = *cluster.map_shared_rank(&s_rest, r);
        if (r < part) before += theirs;
        total += theirs;
      }
      s_before = before, s_total = total;
    }
    cluster.sync();  // (nobody leaves, or writes its sum again, while the others read it)
    if (s_total > 0 || d.minus == 0) break;
    d.minus = 0;
  }
  const uint64_t total = s_total;
  if (total == 0) {  // cannot be: p has weights
    if (part == 0 && tid == 0) tokens[n] = -1, logprobs[n] = 0.f;
    return;
  }
  // the first token whose sum is above floor(r * total)
  const float r = u[p.T];
  uint64_t goal = 0;
  if (r > 0.f) {
    int e;
    const float m = frexpf(fminf(r, 0.99999994f), &e);  // r = m 2^e, m a multiple of 2^-24
    const uint64_t whole = static_cast<uint64_t>(m * 16777216.f) << 40;  // m 2^64
    goal = -e < 64 ? __umul64hi(whole, total) >> -e : 0;
  }
  if (goal >= total) goal = total - 1;
  uint64_t below = s_before;
  int mine = -1;  // the warp's run with the token
  for (int i = 0; i < kDrawWarps; ++i) {
    if (goal >= below && goal - below < s_scan[i]) {
      mine = i;
      break;
    }
    below += s_scan[i];
  }
  if (mine < 0) return;  // another block's (all of the block alike)
  __syncthreads();       // s_scan is written again
  const int start = (part * kDrawWarps + mine) * run;
  const int stop = p.V - start < run ? p.V : start + run;
  for (int v0 = start; v0 < stop; v0 += kDrawThreads) {
    const int v = v0 + tid;
    uint64_t w = 0;
    float x = -INFINITY;
    if (v < stop) {
      x = plain_logit(to_f32(row[v]));
      w = rest_of(d, v, x, plain_logit(to_f32(row_q[v])), s_powers, p.bits);
    }
    uint64_t upto = w;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const uint64_t other = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += other;
    }
    if (lane == 31) s_scan[warp] = upto;
    __syncthreads();
    uint64_t before = below;
    for (int i = 0; i < warp; ++i) before += s_scan[i];
    const uint64_t after = before + upto;
    if (after > goal && after - w <= goal) {
      tokens[n] = v;
      logprobs[n] = scale * (x - t.x) - logf(t.y);
    }
    for (int i = 0; i < kDrawWarps; ++i) below += s_scan[i];
    if (below > goal) break;
    __syncthreads();
  }
}

int piece_vecs(int64_t batch, int rows, int V, int dtype) {
  // vectors a thread: as many as leave every multiprocessor four blocks, one to four
  const int per = static_cast<int>(16 / elem_size(dtype)) * kThreads;
  int vecs = 4;
  while (vecs > 1 && batch * rows * ceil_div(V, static_cast<int64_t>(per) * vecs) < 4 * layer_sm_count()) vecs /= 2;
  return vecs;
}

template <typename T, int kVecs>
cudaError_t launch_sums(const VerifyParams& p, int64_t batch, cudaStream_t stream) {
  return launch_k(verify_sums_kernel<T, kVecs>, dim3(p.pieces, p.rows, static_cast<unsigned>(batch)), dim3(kThreads), 0, stream, true, p);
}

template <typename T>
cudaError_t launch_verify(const VerifyParams& p, int vecs, int64_t batch, cudaStream_t stream) {
  const cudaError_t e = vecs == 4 ? launch_sums<T, 4>(p, batch, stream) : vecs == 2 ? launch_sums<T, 2>(p, batch, stream)
                                                                                    : launch_sums<T, 1>(p, batch, stream);
  if (e != cudaSuccess) return e;
  return launch_k(verify_draw_kernel<T>, dim3(kCluster, static_cast<unsigned>(batch)), dim3(kDrawThreads), 0, stream, true, p);
}

ssd_status check_verify(const ssd_draft_verify_args* a) {
  if (!a || a->size != static_cast<int64_t>(sizeof(*a))) return SSD_ERR_INVALID_ARG;
  if (a->batch < 0 || a->drafts < 0 || a->vocab <= 0) return SSD_ERR_INVALID_ARG;
  if (!known_dtype(a->dtype)) return SSD_ERR_UNSUPPORTED;
  if (a->batch > 65535 || a->drafts > kMaxDrafts || a->vocab > 1 << 24) return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

int rows_of(const ssd_draft_verify_args* a) { return a->drafts + 1 + (a->draft_logits ? a->drafts : 0); }
int pieces_of(const ssd_draft_verify_args* a, int vecs) {
  // (a row begins up to one vector after its 16-byte boundary)
  const int per = static_cast<int>(16 / elem_size(a->dtype));
  return static_cast<int>(ceil_div(a->vocab + per - 1, per * kThreads * vecs));
}

}  // namespace
}  // namespace ssd

extern "C" size_t ssd_draft_verify_workspace_size(const ssd_draft_verify_args* a) {
  using namespace ssd;
  if (check_verify(a) != SSD_OK) return 0;
  return static_cast<size_t>(a->batch) * rows_of(a) * pieces_of(a, piece_vecs(a->batch, rows_of(a), a->vocab, a->dtype)) * sizeof(float2);
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
  const int vecs = piece_vecs(a->batch, rows_of(a), a->vocab, a->dtype);
  p.logits_batch = a->logits_batch, p.logits_row = a->logits_row;
  p.draft_batch = a->draft_logits_batch, p.draft_row = a->draft_logits_row;
  p.T = a->drafts, p.V = a->vocab, p.rows = rows_of(a), p.pieces = pieces_of(a, vecs);
  p.piece = static_cast<int>(16 / es) * kThreads * vecs;
  p.bits = 46;
  while ((int64_t(1) << (62 - p.bits)) < a->vocab) --p.bits;  // sums of a row stay below 2^62
  p.logits = a->logits, p.draft_logits = a->draft_logits;
  p.draft = a->draft, p.lengths = a->lengths, p.uniforms = a->uniforms, p.scale = a->scale;
  p.sums = static_cast<float2*>(a->workspace);
  p.tokens = a->tokens, p.accepted = a->accepted, p.logprobs = a->logprobs;
  return launched(a->dtype == SSD_BF16 ? launch_verify<__nv_bfloat16>(p, vecs, a->batch, stream)
                                       : launch_verify<float>(p, vecs, a->batch, stream));
}
