// The gated delta rule for whole prompts, in chunks of 64 tokens on the tensor cores.
//
// With G the sum of dt A from the chunk's start to a token (that one included), k and q the normalised
// rows and h the state that enters the chunk, the values that the rule writes, v_i, solve
//     v_i + sum_{j<i} beta_i e^{G_i-G_j} (k_i.k_j) v_j = r_i,     r_i = beta_i (x_i - e^{G_i} h k_i),
// so with A that strictly lower triangular matrix, T = (I + A)^-1 and P the products of q and k
//     v = T r,   y_i = scale (e^{G_i} h q_i + sum_{j<=i} e^{G_i-G_j} (q_i.k_j) v_j) = .. + (P T r)_i,
//     h <- e^{G_64} h + sum_j e^{G_64-G_j} v_j k_j^T = .. + (W r)^T,   W = sum_i e^{G_64-G_i} k_i T_i.
// W, P T and the tokens' factors need no state: a first launch forms them for all chunks at once.  The
// second has a block for some columns of a head's state and walks the chunks: r from [K; Q] h, then the new
// state from W r (and y from P T r beside it), with tokens or state rows in the 128 lanes of tensor memory.
// Nobody forms v: that would be a third product in the chain, and its way through the threads.
//
// The state stays in registers, in 32 bits, and enters its product as two fp16 parts, as r does: 11 bits
// each, and with a power of two that brings a tile's largest value to 2^14 the second part's last place is
// at most 2^-22 of a value or 2^-38 of the largest.  (Three bf16 parts need no scale, but half as much again
// of shared memory, stores and products.)  A row of bf16 K or Q times a power of two is fp16; 32-bit ones have
// two parts as well, and so has P T then.  Parts lie side by side along the product's columns, and the threads
// add up what comes out.  Keys enter with lengths near 1 whatever they are (their own powers of two go into beta and x),
// a row of P T and eight columns of T with powers of two of their own.
//
// What it takes, of 128 x 128 states in bf16: 4 x 4096 tokens of 32 heads 570 us (61 for the bytes alone), the first
// launch 261 and the walk 329 (each alone, cold); 16384 tokens of 16 heads 440 (40), a walk's chunk 1.19.  The first
// launch is bound by shared memory and its barriers (58 % of the wavefronts, 51 % of the issue slots, 29 % of the
// DRAM), the walk by its chain: one block an SM, 16 columns, passes a chunk in 2,250 cycles, two products of 570 each,
// r and the state 550 each on their way through the threads and their barriers.  So nothing else is in the chain: x and
// the factors of the next chunk are read while W r runs, the largest values are agreed on while y is written, and y is
// written while the next product runs.  Chunks of 64 tokens: W and P T are one operand of a product each, and 128
// tokens would need twice the columns of tensor memory and four times the first launch's work per chunk, for half the
// chain.
#include <cuda_fp16.h>

#include "delta_chunk.cuh"

namespace ssd {
namespace {

constexpr int kC = 64;  // tokens of a chunk
// Fewer tokens go one by one.  (31 tokens of 16 heads 21 us so, 16 in a chunk; of 128 heads 27 and 31, of 1024
// heads 131 and 116, in 32 bits 139 and 187.)
constexpr int64_t kMinTokens = 32;

// What the first launch leaves, as shared memory holds it (rows of 128 bytes in the 128-byte swizzle).  Of a
// chunk of a head: two parts of W (N rows), P T (64 rows; for bf16 one part, as it goes into y alone, which has
// 8 bits), and the tokens' factors.  Of a chunk of a group, for every part and 64 of N: 64 rows of K, then of Q.
constexpr uint32_t kSlab = 8192;  // 64 rows of 128 bytes
enum { kBeta, kFromState, kOutState, kOutRest, kScalars, kFactors };
constexpr uint32_t kFactorBytes = 4 * kC * 4 + 16;  // with the four scalars
enum { kDecay, kUpdate, kReach, kSpread };  // the scalars: e^{G_64}; what undoes W's scale; see the bounds of delta_walk_kernel
template <typename T>
constexpr int kParts = sizeof(T) == 2 ? 1 : 2;  // of K, Q and P T
__host__ __device__ constexpr uint32_t tile_bytes(int N, int parts) { return (2 * (N / 64) + parts) * kSlab; }
__host__ __device__ constexpr uint32_t record_bytes(int N, int parts) { return tile_bytes(N, parts) + kFactors * kC * 4; }
__host__ __device__ constexpr uint32_t rows_bytes(int N, int parts) { return N / 64 * 2 * kSlab * parts; }

// The power of two that brings numbers up to `largest` (its bits) below 2^15, and its inverse.
struct Scale {
  float up, down;
};
__device__ __forceinline__ Scale scale_for(uint32_t largest) {
  const uint32_t e = max(largest >> 23 & 0xFF, 15u);
  return {__uint_as_float((268 - e) << 23), __uint_as_float((e - 14) << 23)};
}

// Two neighbouring values as two fp16 parts.  (The first rounded: cut off, the second has half as many bits of
// use, 1.1e-6 of 32-bit outputs instead of 0.8e-6, for 1% of the time.)
__device__ __forceinline__ void split(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(a - f.x, b - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h), lo = *reinterpret_cast<const uint32_t*>(&l);
}

// ------------------------------------------------------------------ first launch

constexpr int kPrepThreads = 256;
constexpr int kStride = 68;  // (floats) of A and T: what a fragment's load takes lies in 32 banks

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void stmatrix4(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// cp.async.bulk: bytes from shared to global memory, of the thread's bulk group.
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(__cvta_generic_to_global(dst)), "r"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A product in TF32, each factor as two parts (2^-22 of it is left out).  A thread gives rows g and g + 8 of the
// first factor in columns 2 c and 2 c + 1 (a[0], a[1] and a[2], a[3]; g = lane / 4, c = lane % 4), as an earlier
// product leaves them, where the instruction wants c and c + 4: so it gives those rows of the second factor, at
// column g.
__device__ __forceinline__ void mma_tf32_parts(float (&o)[4], const float (&a)[4], float b0, float b1) {
  uint32_t ah[4], al[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) ah[e] = __float_as_uint(a[e]) & 0xFFFFE000u, al[e] = __float_as_uint(a[e] - __uint_as_float(ah[e]));
  const uint32_t h0 = __float_as_uint(b0) & 0xFFFFE000u, h1 = __float_as_uint(b1) & 0xFFFFE000u;
  mma_tf32(o, al, h0, h1);
  mma_tf32(o, ah, __float_as_uint(b0 - __uint_as_float(h0)), __float_as_uint(b1 - __uint_as_float(h1)));
  mma_tf32(o, ah, h0, h1);
}

template <typename T, int N>
struct PrepSmem {
  static constexpr uint32_t kRow = N * 2 + 16;  // bytes of a row of K or Q, eight rows in different banks
  // K; Q, whose place A takes; T; second parts of K and Q
  static constexpr uint32_t kA = kC * kRow, kSize = kRow > kStride * 4 ? kRow : kStride * 4, kT = kA + kC * kSize;
  static constexpr uint32_t kLow = kT + kC * kStride * 4;
  static constexpr uint32_t kVec = kLow + (kParts<T> == 2 ? 2 * kC * kRow : 0);
  static constexpr uint32_t kTotal = kVec + 9 * kC * 4 + 64;
};

template <typename T, int N>
__global__ void __launch_bounds__(kPrepThreads, kParts<T> == 1 ? 4 : 2) delta_prepare_kernel(DeltaParams p, DeltaChunks s) {
  using M = PrepSmem<T, N>;
  constexpr int kP = kParts<T>;
  extern __shared__ __align__(16) uint8_t smem[];
  float* s_A = reinterpret_cast<float*>(smem + M::kA);
  float* s_T = reinterpret_cast<float*>(smem + M::kT);
  float* s_hi = reinterpret_cast<float*>(smem + M::kVec);
  float *s_lo = s_hi + kC, *s_beta = s_lo + kC, *s_kn = s_beta + kC, *s_qn = s_kn + kC, *s_to = s_qn + kC, *s_len = s_to + kC,
        *s_bx = s_len + kC, *s_down = s_bx + kC;
  int64_t* s_half = reinterpret_cast<int64_t*>(s_down + kC);
  uint32_t* s_largest = reinterpret_cast<uint32_t*>(s_half + 1);  // of every warp
  float *s_most = reinterpret_cast<float*>(s_largest + 8), *s_reach = s_most + 1;
  float2* s_squares = reinterpret_cast<float2*>(smem + M::kT);  // of a row, and what undoes its scale (T comes later)
  // A pair of launches before this one may still walk its chunks, from the other buffer: only the end of this
  // launch waits for it, in one block, so that the next walk finds both complete (see launch_delta_chunks).
  if (!s.follows)
    begin_kernel();
  else
    grid_dep_launch();
  const bool holds_on = s.follows && blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1 && blockIdx.z == gridDim.z - 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t b = blockIdx.z;
  const int h = blockIdx.y, chunk = s.first + blockIdx.x;
  const DeltaSeq seq = delta_sequence(p, b);
  const int64_t t0 = static_cast<int64_t>(chunk) * kC;
  if (seq.row < 0 || t0 >= seq.length) {
    if (holds_on) grid_dep_wait();
    return;
  }
  const int n = seq.length - t0 < kC ? static_cast<int>(seq.length - t0) : kC;
  const int per = p.H / p.G, g = h / per;

  // rows of K (four warps, 16 each), of Q (four more); rows behind the sequence are 0
  constexpr int kRowLanes = N / 8, kPer = 32 / kRowLanes, kLoads = 16 / kPer;  // a lane has 8 of a row
  const bool is_q = warp >= 4;
  const int row0 = 16 * warp + lane / kRowLanes, token0 = row0 & 63, col = lane % kRowLanes;
  struct Eight {
    uint4 raw[kP];
  };
  Eight eight[kLoads];
  {
    const int64_t step = is_q ? p.C_token : p.B_token;
    const T* from = static_cast<const T*>(is_q ? p.Cm : p.Bm) + b * (is_q ? p.C_batch : p.B_batch) + (t0 + token0) * step +
                    static_cast<int64_t>(g) * N + col * 8;
#pragma unroll
    for (int i = 0; i < kLoads; ++i, from += kPer * step) {
#pragma unroll
      for (int e = 0; e < kP; ++e) eight[i].raw[e] = make_uint4(0, 0, 0, 0);
      if (token0 + i * kPer >= n) continue;
      if (s.vectors) {
#pragma unroll
        for (int e = 0; e < kP; ++e) eight[i].raw[e] = reinterpret_cast<const uint4*>(from)[e];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) reinterpret_cast<T*>(eight[i].raw)[e] = from[e];
      }
    }
  }
  // G in whole numbers of 2^-32 (base 2; a token's decay is 2^-1000 at least, which is 0), kept as two
  // 32-bit numbers, the first of few enough bits that differences of it are exact
  if (tid < kC) {
    float d = 0.f, beta = 0.f;
    if (tid < n) d = delta_log_decay<T>(p, b, t0 + tid, h) * kLog2e, beta = delta_beta<T>(p, b, t0 + tid, h);
    if (!(d == d)) beta = d;  // a NaN goes on through beta
    int64_t G = __float2ll_rn(fminf(fmaxf(d, -1000.f), 1000.f) * 4294967296.f);
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int64_t other = __shfl_up_sync(0xffffffffu, G, o);
      if (lane >= o) G += other;
    }
    if (tid == 31) *s_half = G;
    named_bar_sync(1, kC);
    if (warp == 1) G += *s_half;
    s_hi[tid] = static_cast<float>(static_cast<int>(G >> 24)) * 0x1p-8f;
    s_lo[tid] = static_cast<float>(static_cast<int>(G & 0xFFFFFF)) * 0x1p-32f;
    s_beta[tid] = beta;
  }
  // in fp16, times a power of two
  uint8_t* rows_out = h == g * per ? s.rows + ((b * p.G + g) * s.count + blockIdx.x) * static_cast<int64_t>(rows_bytes(N, kP)) +
                                         (col >> 3) * 2 * kSlab + row0 * 128
                                   : nullptr;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = row0 + i * kPer;
    float v[8], squares = 0.f, largest = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t w = (&eight[i].raw[0].x)[kP == 1 ? e / 2 : e];
      v[e] = kP == 2 ? __uint_as_float(w) : e & 1 ? bf16_hi(w) : bf16_lo(w);
      squares = fmaf(v[e], v[e], squares), largest = fmaxf(largest, fabsf(v[e]));
    }
#pragma unroll
    for (int o = kRowLanes / 2; o; o /= 2) {
      squares += __shfl_xor_sync(0xffffffffu, squares, o);
      largest = fmaxf(largest, __shfl_xor_sync(0xffffffffu, largest, o));
    }
    const Scale scale = scale_for(__float_as_uint(largest));
    uint4 half[kP];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float lo = v[2 * e] * scale.up, hi = v[2 * e + 1] * scale.up;
      if constexpr (kP == 1) {
        const __half2 pair = __floats2half2_rn(lo, hi);
        (&half[0].x)[e] = *reinterpret_cast<const uint32_t*>(&pair);
      } else {
        split(lo, hi, (&half[0].x)[e], (&half[kP - 1].x)[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < kP; ++e) {
      *reinterpret_cast<uint4*>(smem + (e ? M::kLow : 0) + r * M::kRow + col * 16) = half[e];
      if (rows_out) *reinterpret_cast<uint4*>(rows_out + e * rows_bytes(N, 1) + i * kPer * 128 + (((col & 7) ^ (r & 7)) << 4)) = half[e];
    }
    if (col == 0) s_squares[r] = make_float2(squares, scale.down);
  }
  __syncthreads();

  // K K^T (four warps, 16 rows each) and Q K^T (four more)
  const int mt = is_q ? 7 - warp : warp;  // (beside a warp of few columns one of many)
  const uint32_t rows = smem_u32(smem);
  float acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
  {
    const uint32_t at = rows + ((is_q ? kC : 0) + 16 * mt + (lane & 15)) * M::kRow + (lane >> 4) * 16;
    const uint32_t bt = rows + ((lane & 7) + (lane >> 4) * 8) * M::kRow + ((lane >> 3) & 1) * 16;
#pragma unroll
    for (int k = 0; k < N / 16; ++k) {
      uint32_t a[4], al[4];
      ldmatrix4(a, at + k * 32);
      if (kP == 2) ldmatrix4(al, at + M::kLow + k * 32);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j > mt) break;
        uint32_t v[4];
        ldmatrix4(v, bt + j * 16 * M::kRow + k * 32);
        if constexpr (kP == 2) {
          uint32_t l[4];
          ldmatrix4(l, bt + M::kLow + j * 16 * M::kRow + k * 32);
          mma_f16(acc[2 * j], al, v[0], v[1]), mma_f16(acc[2 * j + 1], al, v[2], v[3]);
          mma_f16(acc[2 * j], a, l[0], l[1]), mma_f16(acc[2 * j + 1], a, l[2], l[3]);
        }
        mma_f16(acc[2 * j], a, v[0], v[1]);
        mma_f16(acc[2 * j + 1], a, v[2], v[3]);
      }
    }
  }
  // What makes of a row, times its power of two, the row that counts: of K by the first two warps, of Q by the last, who
  // had the fewest columns.
  if (tid < kC || tid >= 3 * kC) {
    const int at = tid < kC ? tid : tid - 2 * kC, token = tid & 63;
    const float2 v = s_squares[at];
    const float up = __int_as_float(0x7F000000 - __float_as_int(v.y));
    float norm = v.y, squares = v.x * up * up;  // (of the row times its power of two: below 2^38)
    if (!(v.x > 0x1p-80f && v.x < 0x1p120f) && token < n) {  // squares that 32 bits may not have held
      squares = 0.f;
#pragma unroll 1
      for (int i = 0; i < N; ++i) {
        const __half* from = reinterpret_cast<const __half*>(smem + at * M::kRow);
        float e = __half2float(from[i]);
        if (kP == 2) e += __half2float(from[M::kLow / 2 + i]);
        squares = fmaf(e, e, squares);
      }
    }
    if (p.norm_eps >= 0.f) {
      const float e = p.norm_eps * up * up;
      norm = e < 0x1p80f ? rsqrtf(squares + e) : v.y * rsqrtf(p.norm_eps);
    }
    if (squares == 0.f || token >= n) norm = 0.f;
    if (tid >= kC) {
      s_qn[token] = norm;
    } else {
      // A key times 2^-e, x times 2^-e and beta times 2^2e are the same rule: with lengths between 0.7 and 1.4 the keys'
      // own sizes set none of the scales below, whether they are normalised or as they are.
      const float length = norm * sqrtf(squares);
      const int e = min(max((__float_as_int(length * 1.41421356f) >> 23 & 0xFF) - 127, -126), 126);
      const float longer = __int_as_float((127 + e) << 23), shorter = __int_as_float((127 - e) << 23);
      const float bx = s_beta[token] * longer;
      s_kn[token] = norm * shorter, s_len[token] = length * shorter, s_bx[token] = bx, s_beta[token] = bx * longer;
    }
  }
  __syncthreads();  // Q's rows have been read
  // A; P, whose rows' norms, powers of two and scale wait for the end, stays in registers
  {
    const int row = 16 * mt + (lane >> 2);
    const float hi0 = s_hi[row], hi8 = s_hi[row + 8], lo0 = s_lo[row], lo8 = s_lo[row + 8];
    const float f0 = is_q ? 0x1p-14f : s_kn[row] * s_beta[row], f8 = is_q ? 0x1p-14f : s_kn[row + 8] * s_beta[row + 8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j > 2 * mt + 1) break;
      const int col = 8 * j + (lane & 3) * 2;
      const float2 hi = *reinterpret_cast<const float2*>(&s_hi[col]), lo = *reinterpret_cast<const float2*>(&s_lo[col]),
                   kn = *reinterpret_cast<const float2*>(&s_kn[col]);
      float(&v)[4] = acc[j];
      v[0] *= exp2_fast((hi0 - hi.x) + (lo0 - lo.x)) * (kn.x * f0);
      v[1] *= exp2_fast((hi0 - hi.y) + (lo0 - lo.y)) * (kn.y * f0);
      v[2] *= exp2_fast((hi8 - hi.x) + (lo8 - lo.x)) * (kn.x * f8);
      v[3] *= exp2_fast((hi8 - hi.y) + (lo8 - lo.y)) * (kn.y * f8);
      // below the diagonal (P: and on it); a factor above it may be infinite
      const int below = col - (is_q ? 1 : 0);
      v[0] = below < row ? v[0] : 0.f, v[1] = below + 1 < row ? v[1] : 0.f;
      v[2] = below < row + 8 ? v[2] : 0.f, v[3] = below + 1 < row + 8 ? v[3] : 0.f;
      if (!is_q) {
        *reinterpret_cast<float2*>(&s_A[row * kStride + col]) = make_float2(v[0], v[1]);
        *reinterpret_cast<float2*>(&s_A[(row + 8) * kStride + col]) = make_float2(v[2], v[3]);
      }
    }
  }
  __syncthreads();

  // the factors of T's rows in W, e^{G_64-G_i} k's norm, over the largest of them
  if (warp == 3) {
    float v[2], reach = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = lane + 32 * e;
      const float own = fabsf(s_beta[i]) * exp2f(s_hi[i] + s_lo[i]) * s_len[i];
      reach = fmaxf(reach, own < INFINITY ? own : 0.f);
      v[e] = i < n ? s_kn[i] * exp2f((s_hi[kC - 1] - s_hi[i]) + (s_lo[kC - 1] - s_lo[i])) : 0.f;
    }
    const float most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(v[0], v[1]))));
    // (keys of zeros, or keys that the chunk's end has forgotten to 2^-120: nothing is written into the state)
    const float f = most > 0x1p-120f ? 1.f / most : 0.f;
    s_to[lane] = v[0] * f, s_to[lane + 32] = v[1] * f;
    reach = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(reach)));
    if (lane == 0) *s_most = most, *s_reach = reach;
  }

  // T: the diagonal blocks of 16 by substitution, the others below from those above them,
  // T_ij = -T_ii sum_{j <= k < i} A_ik T_kj
  if (tid < kC) {
    const int d0 = tid & ~15, c = tid & 15;
    float v[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      float sum = r == c ? 1.f : 0.f;
#pragma unroll
      for (int k4 = 0; k4 < r; k4 += 4) {
        const float4 a = *reinterpret_cast<const float4*>(&s_A[(d0 + r) * kStride + d0 + k4]);
        sum = fmaf(-a.x, v[k4], sum);
        if (k4 + 1 < r) sum = fmaf(-a.y, v[k4 + 1], sum);
        if (k4 + 2 < r) sum = fmaf(-a.z, v[k4 + 2], sum);
        if (k4 + 3 < r) sum = fmaf(-a.w, v[k4 + 3], sum);
      }
      v[r] = sum;
      s_T[(d0 + r) * kStride + d0 + c] = sum;
    }
  }
  __syncthreads();
  // (two warps a row of blocks, 8 columns each; the products T_ii A_ik need nothing but the diagonal)
  {
    const int i = 1 + (warp >> 1), half = warp & 1;
    const int gr = lane >> 2, gc = (lane & 3) * 2;
    float f[3][2][4];
    if (i < 4) {
      float t[2][4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float* at = &s_T[(16 * i + gr) * kStride + 16 * i + 8 * k + gc];
        const float2 a = *reinterpret_cast<const float2*>(at), b8 = *reinterpret_cast<const float2*>(at + 8 * kStride);
        t[k][0] = a.x, t[k][1] = b8.x, t[k][2] = a.y, t[k][3] = b8.y;
      }
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        if (k >= i) break;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float* at = &s_A[(16 * i + 8 * e + gc) * kStride + 16 * k + 8 * u + gr];
            mma_tf32_parts(o, t[e], at[0], at[kStride]);
          }
          f[k][u][0] = o[0], f[k][u][1] = o[2], f[k][u][2] = o[1], f[k][u][3] = o[3];
        }
      }
    }
#pragma unroll
    for (int d = 1; d < 4; ++d) {
      const int j = i - d;
      if (i < 4 && j >= 0) {
        float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          if (k < j || k >= i) continue;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float* at = &s_T[(16 * k + 8 * u + gc) * kStride + 16 * j + 8 * half + gr];
            mma_tf32_parts(o, f[k][u], at[0], at[kStride]);
          }
        }
        float* to = &s_T[(16 * i + gr) * kStride + 16 * j + 8 * half + gc];
        *reinterpret_cast<float2*>(to) = make_float2(-o[0], -o[1]);
        *reinterpret_cast<float2*>(to + 8 * kStride) = make_float2(-o[2], -o[3]);
      }
      __syncthreads();
    }
  }

  // P T, whose rows a warp has in registers as the products of above have theirs
  if (is_q) {
    float o[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
    const float* t = s_T + (lane & 3) * 2 * kStride + (lane >> 2);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (k > 2 * mt + 1) break;
      const float a[4] = {acc[k][0], acc[k][2], acc[k][1], acc[k][3]};
#pragma unroll
      for (int j = 0; j <= k; ++j) mma_tf32_parts(o[j], a, t[8 * k * kStride + 8 * j], t[(8 * k + 1) * kStride + 8 * j]);
    }
    // as the second launch reads it, where A was; blocks above the diagonal are 0.  A row has a power of two of its own,
    // which its factor undoes: rows behind strong decays keep their digits.
    float top = 0.f, top8 = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      top = fmaxf(fmaxf(top, fabsf(o[j][0])), fabsf(o[j][1]));
      top8 = fmaxf(fmaxf(top8, fabsf(o[j][2])), fabsf(o[j][3]));
    }
#pragma unroll
    for (int e = 1; e < 4; e *= 2) {
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, e));
      top8 = fmaxf(top8, __shfl_xor_sync(0xffffffffu, top8, e));
    }
    const Scale of = scale_for(__float_as_uint(top)), of8 = scale_for(__float_as_uint(top8));
    if ((lane & 3) == 0) s_down[16 * mt + (lane >> 2)] = of.down, s_down[16 * mt + (lane >> 2) + 8] = of8.down;
    const int at_row = 16 * mt + (lane >> 3 & 1) * 8 + (lane & 7);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      uint32_t v[4], l[4] = {};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float* from_o = &o[j + (e >> 1)][e & 1 ? 2 : 0];
        const float up = e & 1 ? of8.up : of.up;
        if constexpr (kP == 1) {
          const __half2 pair = __floats2half2_rn(from_o[0] * up, from_o[1] * up);
          v[e] = *reinterpret_cast<const uint32_t*>(&pair);
        } else {
          split(from_o[0] * up, from_o[1] * up, v[e], l[e]);
        }
      }
      const uint32_t to = rows + at_row * 128 + (((j + (lane >> 4)) ^ (at_row & 7)) << 4);
      stmatrix4(to + M::kA, v[0], v[1], v[2], v[3]);
      if (kP == 2) stmatrix4(to + M::kLow + kC * M::kRow, l[0], l[1], l[2], l[3]);  // (where Q's second part was)
    }
  }

  // W = K^T T', T's rows times their factors in two fp16 parts (K is one): 8 columns a warp, with a power of two
  constexpr int kTiles = N / 16;
  float w[kTiles][4];
  uint32_t bh[4][2], bl[4][2];
  float factored[4][2][2], top = 0.f;
#pragma unroll
  for (int m = 0; m < kTiles; ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e) w[m][e] = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (k < warp >> 1) continue;  // above the diagonal
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 16 * k + 8 * e + (lane & 3) * 2;
      const float* t = &s_T[i * kStride + 8 * warp + (lane >> 2)];
      factored[k][e][0] = t[0] * s_to[i], factored[k][e][1] = t[kStride] * s_to[i + 1];
      top = fmaxf(fmaxf(top, fabsf(factored[k][e][0])), fabsf(factored[k][e][1]));
    }
  }
  const Scale own = scale_for(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (k < warp >> 1) continue;
#pragma unroll
    for (int e = 0; e < 2; ++e) split(factored[k][e][0] * own.up, factored[k][e][1] * own.up, bh[k][e], bl[k][e]);
  }
  const uint32_t kt = rows + ((lane & 7) + (lane >> 4) * 8) * M::kRow + ((lane >> 3) & 1) * 16;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (k < warp >> 1) continue;
#pragma unroll
    for (int m = 0; m < kTiles; ++m) {
      uint32_t a[4];
      ldmatrix4_t(a, kt + k * 16 * M::kRow + m * 32);
      if constexpr (kP == 2) {
        uint32_t al[4];
        ldmatrix4_t(al, kt + M::kLow + k * 16 * M::kRow + m * 32);
        mma_f16(w[m], al, bh[k][0], bh[k][1]);
      }
      mma_f16(w[m], a, bl[k][0], bl[k][1]);
      mma_f16(w[m], a, bh[k][0], bh[k][1]);
    }
  }
  top = 0.f;
#pragma unroll
  for (int m = 0; m < kTiles; ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e) w[m][e] *= own.down, top = fmaxf(top, fabsf(w[m][e]));
  const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
  if (lane == 0) s_largest[warp] = bits;
  __syncthreads();
  uint32_t most_bits = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) most_bits = max(most_bits, s_largest[i]);
  const Scale scale = scale_for(most_bits);
  // the parts where K and T were, and all into global memory
#pragma unroll
  for (int m = 0; m < kTiles; ++m) {
    const int at_row = 16 * m + (lane >> 3 & 1) * 8 + (lane & 7);
    uint32_t hi[2], lo[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) split(w[m][2 * e] * scale.up, w[m][2 * e + 1] * scale.up, hi[e], lo[e]);
    stmatrix4(rows + (lane < 16 ? 0 : M::kT) + at_row * 128 + ((warp ^ (at_row & 7)) << 4), hi[0], hi[1], lo[0], lo[1]);
  }
  fence_proxy_async_smem();
  __syncthreads();
  uint8_t* out = s.records + ((b * p.H + h) * s.count + blockIdx.x) * static_cast<int64_t>(record_bytes(N, kP));
  if (tid < kC) {
    float* factors = reinterpret_cast<float*>(out + tile_bytes(N, kP));
    const float since = exp2f(s_hi[tid] + s_lo[tid]), qn = p.scale * s_qn[tid];
    factors[kBeta * kC + tid] = s_bx[tid];
    factors[kFromState * kC + tid] = s_beta[tid] * s_kn[tid] * since;
    factors[kOutState * kC + tid] = qn * since;
    factors[kOutRest * kC + tid] = qn * 0x1p14f * s_down[tid];
    if (tid == kC - 1) {
      float* scalars = factors + kScalars * kC;
      scalars[kDecay] = since, scalars[kUpdate] = scale.down * *s_most;
      scalars[kReach] = *s_reach * (N == 64 ? 8.f : 11.5f);  // (a row's sum of magnitudes is sqrt(N) of its length at most)
      scalars[kSpread] = kC * 32768.f * scalars[kUpdate];    // (W's largest is below 2^15 of its unit)
    }
  }
  if (tid == kC) {
    bulk_store(out, rows, N * 128);
    bulk_store(out + N * 128, rows + M::kT, N * 128);
    bulk_store(out + 2 * N * 128, rows + M::kA, kSlab);
    if (kP == 2) bulk_store(out + 2 * N * 128 + kSlab, rows + M::kLow + kC * M::kRow, kSlab);
    tma_store_commit();
    tma_store_wait_all();
  }
  if (holds_on) grid_dep_wait();
}

// ------------------------------------------------------------------ second launch

enum {
  kRowsFull, kRowsFull1, kRowsEmpty, kRowsEmpty1,  // K and Q
  kSideFull, kSideFull1, kSideEmpty, kSideEmpty1,  // the factors and x
  kTileFull, kTileFull1, kTileEmpty, kTileEmpty1,  // W and P T
  kStateReady, kFromStateDone, kRestReady, kUpdateDone, kRestDone,  // the chain
  kLargestReady, kDrained, kBarriers
};

// kPT: columns of the state (values of a head) that a block has; kGroups: warpgroups that share them;
// kStages: buffers of rows and of [T; P T].
template <typename T, int N, int kPT, int kGroups, int kStages>
struct Walk {
  static constexpr int kP = kParts<T>;
  static constexpr int kWorkers = 4 * kGroups;             // warps with the state
  static constexpr int kThreads = 32 * (kWorkers + 2);     // and one that loads, one that issues the products
  static constexpr int kCols = kPT / kGroups;              // of a thread
  static constexpr int kSlabs = (2 * kPT + 63) / 64;       // 64 columns each of the two parts side by side
  static constexpr uint32_t kSlabS = N * 128;
  static constexpr uint32_t kRows = 0, kTile = kRows + kStages * rows_bytes(N, kP), kS = kTile + kStages * tile_bytes(N, kP);
  static constexpr uint32_t kR = kS + kSlabs * kSlabS;
  static constexpr uint32_t kEnd = kR + kSlabs * kSlab;
  static constexpr uint32_t kLargest = kEnd + (kBarriers * 8 + 2 * 4 + 15) / 16 * 16, kSeen = kLargest + 4 * kWorkers * 4;
  static constexpr uint32_t kF = kSeen + kWorkers * 4;
  static constexpr uint32_t kX = kF + 2 * kFactorBytes;            // x, a token's row after the other
  static constexpr uint32_t kXRow = kPT * sizeof(T) + 16;          // (so that eight rows lie in different banks)
  static constexpr uint32_t kTotal = kX + 2 * kC * kXRow;
  static constexpr uint32_t kTmem = 4 * kPT;               // columns of tensor memory
};

// cp.async.bulk: bytes from global to shared memory, counted by the barrier.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
               "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ void tmem_ld8(uint32_t at, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(at));
}

// One thread of a warp that is together, always the same one.  What the others compute beside it is known to be the
// same in all, so that descriptors stay in uniform registers: a product is issued every 41 cycles (M 128, N 32), under
// a plain test of the lane every 60.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

template <typename T, int N, int kPT, int kGroups, int kStages, int kBlocks>
__global__ void __launch_bounds__(Walk<T, N, kPT, kGroups, kStages>::kThreads, kBlocks) delta_walk_kernel(DeltaParams p, DeltaChunks s) {
  using M = Walk<T, N, kPT, kGroups, kStages>;
  constexpr int kP = M::kP, kCols = M::kCols, kWorkers = M::kWorkers, kVecs = kCols * static_cast<int>(sizeof(T)) / 16;
  constexpr uint32_t kColD1 = 0, kColD3 = 2 * kPT;  // W r goes where [K; Q] h was
  extern __shared__ __align__(1024) uint8_t walk_smem[];
  uint8_t* smem = walk_smem;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + M::kEnd);
  uint32_t* holder = reinterpret_cast<uint32_t*>(bars + kBarriers);
  volatile int* failed = reinterpret_cast<volatile int*>(holder + 1);
  uint32_t* s_largest = reinterpret_cast<uint32_t*>(smem + M::kLargest);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t b = blockIdx.z;
  const int h = blockIdx.y, p0 = blockIdx.x * kPT;
  if (tid == 0) {
    for (int i = 0; i < kBarriers; ++i)
      mbar_init(&bars[i], i == kStateReady || i == kLargestReady || i == kRestReady || i == kSideEmpty || i == kSideEmpty1 ? kWorkers : i == kSideFull || i == kSideFull1 ? 33 : 1);
    fence_mbar_init();
    *failed = 0;
    for (int i = 0; i < 4 * kWorkers; ++i) s_largest[i] = 0;
  }
  if (warp == kWorkers) {
    tmem_alloc(holder, M::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *holder;
  begin_kernel();

  const DeltaSeq seq = delta_sequence(p, b);
  const int64_t begin = static_cast<int64_t>(s.first) * kC;  // this call's tokens
  const int64_t end = begin + static_cast<int64_t>(s.count) * kC < p.seqlen ? begin + static_cast<int64_t>(s.count) * kC : p.seqlen;
  const int64_t length = seq.row < 0 || seq.length < begin ? begin : seq.length < end ? seq.length : end;
  const int chunks = static_cast<int>((length - begin + kC - 1) / kC);
  const int g = h / (p.H / p.G);
  const uint8_t* records = s.records + (b * p.H + h) * s.count * static_cast<int64_t>(record_bytes(N, kP));
  const uint8_t* rows = s.rows + (b * p.G + g) * s.count * static_cast<int64_t>(rows_bytes(N, kP));
  auto wait = [&](int bar, int phase) {
    if (mbar_try_wait_short(&bars[bar], phase & 1)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
      if (mbar_try_wait_short(&bars[bar], phase & 1)) return true;
      if (*failed) return false;
      if (globaltimer_ns() - t0 > s.limit_ns) {
        *failed = 1;
        return false;
      }
    }
  };
  // The same without suspending the thread between tests: the products' thread is in the chain.
  auto spin = [&](int bar, int phase) {
    for (int i = 0; i < 4096; ++i)
      if (mbar_test_wait(&bars[bar], phase & 1)) return true;
    return wait(bar, phase);
  };

  if (warp == kWorkers) {
    // loads
    bool ok = true;
    const uint32_t x_bytes = (p.P - p0 < kPT ? p.P - p0 : kPT) * static_cast<uint32_t>(sizeof(T));
    const T* x = static_cast<const T*>(p.x) + b * p.x_batch + static_cast<int64_t>(h) * p.P + p0;
    // what the threads read themselves, the factors and x (of that, by all lanes, neighbours on a row)
    auto load_side = [&](int c) {
      const int st = c & 1, turn = c >> 1;
      if (!__all_sync(0xffffffffu, turn == 0 || wait(kSideEmpty + st, turn - 1))) return false;
      const int64_t t0 = begin + static_cast<int64_t>(c) * kC;
      const uint32_t tokens = !s.vectors ? 0 : length - t0 < kC ? static_cast<uint32_t>(length - t0) : kC;
      uint64_t* full = &bars[kSideFull + st];
      if (lane == 0) {
        mbar_arrive_expect_tx(full, kFactorBytes);
        bulk_load(smem + M::kF + st * kFactorBytes, records + c * static_cast<int64_t>(record_bytes(N, kP)) + tile_bytes(N, kP), kFactorBytes, full);
      }
      constexpr uint32_t kPer = kPT * sizeof(T) / 16;
#pragma unroll
      for (uint32_t i = lane; i < kC * kPer; i += 32) {
        const uint32_t token = i / kPer, at = i % kPer * 16;
        if (token >= tokens || at >= x_bytes) continue;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem + M::kX + (st * kC + token) * M::kXRow + at)),
                     "l"(__cvta_generic_to_global(reinterpret_cast<const uint8_t*>(x + (t0 + token) * p.x_token) + at))
                     : "memory");
      }
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(full)) : "memory");
      return true;
    };
    int sides = 0, c = 0, t = 0;  // chunks whose factors, rows and tiles are on their way
    if (chunks > 0) load_side(sides++);
    while (t < chunks) {
      const int st = t % kStages, turn = t / kStages;
      if (sides < chunks) {
        ok = load_side(sides);
        if (!ok) break;
        ++sides;
      }
      ok = __all_sync(0xffffffffu, turn == 0 || wait(kRowsEmpty + st, turn - 1));
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars[kRowsFull + st], rows_bytes(N, kP));
        bulk_load(smem + M::kRows + st * rows_bytes(N, kP), rows + c * static_cast<int64_t>(rows_bytes(N, kP)), rows_bytes(N, kP), &bars[kRowsFull + st]);
      }
      ++c;
      ok = __all_sync(0xffffffffu, turn == 0 || wait(kTileEmpty + st, turn - 1));
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars[kTileFull + st], tile_bytes(N, kP));
        bulk_load(smem + M::kTile + st * tile_bytes(N, kP), records + t * static_cast<int64_t>(record_bytes(N, kP)), tile_bytes(N, kP), &bars[kTileFull + st]);
      }
      ++t;
    }
    // nothing is in flight when the block ends, whoever has given up
    for (int i = sides > 2 ? sides - 2 : 0; i < sides; ++i) mbar_wait(&bars[kSideFull + (i & 1)], (i >> 1) & 1, s.limit_ns);
    for (int i = c > kStages ? c - kStages : 0; i < c; ++i) mbar_wait(&bars[kRowsFull + i % kStages], (i / kStages) & 1, s.limit_ns);
    for (int i = t > kStages ? t - kStages : 0; i < t; ++i) mbar_wait(&bars[kTileFull + i % kStages], (i / kStages) & 1, s.limit_ns);
  } else if (warp == kWorkers + 1) {
    // products: the warp stays together and one thread issues (see elect_one)
    constexpr uint32_t id_two = idesc_f32acc(0, 128, 2 * kPT, 0, 1), id_one = idesc_f32acc(0, 128, kPT, 0, 1);
    const uint32_t base = smem_u32(smem);
    const uint64_t dS = sdesc_sw128(base + M::kS, M::kSlabS, 1024), dR = sdesc_sw128(base + M::kR, kSlab, 1024);
    for (int c = 0; c < chunks; ++c) {
      const int st = c % kStages, turn = c / kStages;
      const uint32_t kq = base + M::kRows + st * rows_bytes(N, kP);
      if (!__all_sync(0xffffffffu, wait(kRowsFull + st, turn) && spin(kStateReady, c))) break;
      tc_fence_after();
      const uint64_t kq_rows = sdesc_sw128(kq, 16, 1024);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < N / 16; ++k)
          mma_ss<false>(tmem + kColD1, kq_rows + (((k >> 2) * 2 * kSlab + (k & 3) * 32) >> 4), dS + (k * 2048 >> 4), id_two, k != 0);
        if constexpr (kP == 2) {
#pragma unroll
          for (int k = 0; k < N / 16; ++k)
            mma_ss<false>(tmem + kColD1, kq_rows + ((rows_bytes(N, 1) + (k >> 2) * 2 * kSlab + (k & 3) * 32) >> 4), dS + (k * 2048 >> 4), id_one, 1);
        }
        mma_commit(&bars[kFromStateDone]);
        mma_commit(&bars[kRowsEmpty + st]);
      }
      __syncwarp();
      if (!__all_sync(0xffffffffu, wait(kTileFull + st, turn) && spin(kRestReady, c))) break;
      tc_fence_after();
      const uint32_t tile = base + M::kTile + st * tile_bytes(N, kP);
      const uint64_t w = sdesc_sw128(tile, 16, 1024);
      // P T's 64 rows go to the lanes of Q: they are the second half of 128 that begin in what lies before them
      const uint64_t pt = sdesc_sw128(tile + (2 * (N / 64) - 1) * kSlab, 16, 1024);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kC / 16; ++k) {  // both first parts, and the second of either with the first of the other
          mma_ss<false>(tmem + kColD1, w + (k * 32 >> 4), dR + (k * 2048 >> 4), id_two, k != 0);
          mma_ss<false>(tmem + kColD1, w + ((N / 64 * kSlab + k * 32) >> 4), dR + (k * 2048 >> 4), id_one, 1);
        }  // (N 64: the upper lanes' product is nobody's)
        mma_commit(&bars[kUpdateDone]);
#pragma unroll
        for (int k = 0; k < kC / 16; ++k) {
          mma_ss<false>(tmem + kColD3, pt + (k * 32 >> 4), dR + (k * 2048 >> 4), id_two, k != 0);
          if constexpr (kP == 2) mma_ss<false>(tmem + kColD3, pt + ((kSlab + k * 32) >> 4), dR + (k * 2048 >> 4), id_one, 1);
        }
        mma_commit(&bars[kRestDone]);
        mma_commit(&bars[kTileEmpty + st]);
      }
      __syncwarp();
    }
    if (elect_one()) {
      mma_commit(&bars[kDrained]);
      mbar_wait(&bars[kDrained], 0, s.limit_ns);
    }
  } else {
    // the state, and everything between the products
    const int group = warp >> 2, quarter = warp & 3;
    const int row = 32 * quarter + lane;  // of tensor memory: token (and 64 more: its output) or state row
    const bool has_state = quarter < N / 32, is_token = quarter < 2;
    const int token = row & 63;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * quarter) << 16) + group * kCols;
    const int col0 = p0 + group * kCols;  // the thread's values of the head
    const int64_t y_token = static_cast<int64_t>(p.H) * p.P;
    T* y = static_cast<T*>(p.y) + b * p.seqlen * y_token + static_cast<int64_t>(h) * p.P + col0;
    const T* x = static_cast<const T*>(p.x) + b * p.x_batch + static_cast<int64_t>(h) * p.P + col0;

    // kCols values of a row, scaled, as two parts side by side: rows of 128 bytes in slabs of 64 columns
    auto put = [&](uint32_t tile, uint32_t slab, int at_row, const float (&v)[kCols], float up) {
#pragma unroll
      for (int i = 0; i < kCols / 8; ++i) {
        uint4 hi, lo;
#pragma unroll
        for (int e = 0; e < 4; ++e) split(v[8 * i + 2 * e] * up, v[8 * i + 2 * e + 1] * up, (&hi.x)[e], (&lo.x)[e]);
        const int c0 = group * kCols + 8 * i, c1 = kPT + c0;
        uint8_t* to = smem + tile + at_row * 128;
        *reinterpret_cast<uint4*>(to + (c0 >> 6) * slab + ((((c0 & 63) >> 3) ^ (at_row & 7)) << 4)) = hi;
        *reinterpret_cast<uint4*>(to + (c1 >> 6) * slab + ((((c1 & 63) >> 3) ^ (at_row & 7)) << 4)) = lo;
      }
      fence_proxy_async_smem();
    };
    // the two parts' sums of kCols columns
    auto take = [&](uint32_t at, float (&v)[kCols]) {
      if constexpr (kCols == 8) {
        uint32_t a[8], c[8];
        tmem_ld8(lanes + at, a);
        tmem_ld8(lanes + at + kPT, c);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(a[i]) + __uint_as_float(c[i]);
      } else {
#pragma unroll
        for (int j = 0; j < kCols; j += 16) {
          uint32_t a[16], c[16];
          tmem_ld16(lanes + at + j, a);
          tmem_ld16(lanes + at + kPT + j, c);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) v[j + i] = __uint_as_float(a[i]) + __uint_as_float(c[i]);
        }
      }
    };
    auto arrive = [&](int bar) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[bar]);
    };
    auto all_wait = [&](int bar, int phase) { return __all_sync(0xffffffffu, wait(bar, phase)) != 0; };
    // Largest finite magnitudes that the warps have left, [state, beta x][chunk mod 2][warp].  Columns are independent of
    // each other, so an infinity, which is NaN in its parts whatever the scale, must not set that of its neighbours:
    // twice the bits plus 2^24 wraps around to less than 2^24, that of 0, for infinities and NaN.
    auto leave = [&](int which, int c, const float (&v)[kCols], int place) {
      constexpr uint32_t kZero = 0x01000000u;
      uint32_t top = kZero;
#pragma unroll
      for (int i = 0; i < kCols; ++i) top = max(top, 2 * __float_as_uint(v[i]) + kZero);
      top = __reduce_max_sync(0xffffffffu, top);
      if (lane == 0) s_largest[(2 * which + (c & 1)) * kWorkers + place] = (top - kZero) >> 1;
    };
    auto largest_of = [&](int which, int c, int warps) {
      const uint4* at = reinterpret_cast<const uint4*>(s_largest + (2 * which + (c & 1)) * kWorkers);
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < kWorkers / 4; ++i) {
        if (4 * i >= warps) break;
        const uint4 v = at[i];
        top = max(max(top, max(v.x, v.y)), max(v.z, v.w));
      }
      return __uint_as_float(top);
    };

    float S[kCols];
    {
      const float* from = s.first == 0 ? seq.row >= 0 && seq.resumed ? p.init_state + seq.row * p.H * p.P * N : nullptr
                                       : s.carry + b * p.H * p.P * N;
#pragma unroll
      for (int i = 0; i < kCols; ++i)
        S[i] = from && has_state && col0 + i < p.P ? from[(static_cast<int64_t>(h) * p.P + col0 + i) * N + row] : 0.f;
    }
    // Scales go by bounds that are known while the products run, not by what comes out of them, so that nobody
    // waits for the others in the chain: with s the largest of the state
    //     |r| <= max |beta x| + s max_j beta e^{G_j} |k_j|_1,    |state after| <= e^{G_64} s + 64 max |W| max |r|.
    // They can be a thousand times too large (the sums' signs); two parts have 2^17 to spare.  One past 32 bits is
    // infinite, which scale_for takes for 2^128.
    Scale state{1.f, 1.f};
    bool ok = true;
    float bx[kCols], fa, fb;  // beta x of tokens, and then the state's part of y of the others; the row's factors
    float4 scalars;
    auto ahead = [&](int c) {
      if (!all_wait(kSideFull + (c & 1), c >> 1)) return false;
      const float* factors = reinterpret_cast<const float*>(smem + M::kF + (c & 1) * kFactorBytes);
      scalars = *reinterpret_cast<const float4*>(factors + kScalars * kC);
      fa = factors[(is_token ? kBeta : kOutState) * kC + token], fb = factors[(is_token ? kFromState : kOutRest) * kC + token];
      if (is_token) {
        const uint8_t* s_x = smem + M::kX + ((c & 1) * kC + token) * M::kXRow + group * kCols * sizeof(T);
        const int64_t t = begin + static_cast<int64_t>(c) * kC + token;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
          constexpr int kE = 16 / sizeof(T);
          uint4 xs = make_uint4(0, 0, 0, 0);
          if (t < length && col0 + kE * i < p.P) {
            if (s.vectors) {
              xs = *reinterpret_cast<const uint4*>(s_x + 16 * i);
            } else {
#pragma unroll
              for (int e = 0; e < kE; ++e) reinterpret_cast<T*>(&xs)[e] = x[t * p.x_token + kE * i + e];
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t w = (&xs.x)[e];
            if constexpr (kP == 1)
              bx[8 * i + 2 * e] = fa * bf16_lo(w), bx[8 * i + 2 * e + 1] = fa * bf16_hi(w);
            else
              bx[4 * i + e] = fa * __uint_as_float(w);
          }
        }
        leave(1, c, bx, 2 * group + quarter);
      }
      // The loads have to be over before the buffer is given back, and a load that is only under way does not hold up an
      // arrival (it may wait for hundreds of cycles while copies fill the shared memory): what all lanes have read goes
      // into a word that nobody wants, whose store lies before the arrival.
      const uint32_t seen = __reduce_or_sync(0xffffffffu, __float_as_uint(fa) | __float_as_uint(fb) | __float_as_uint(scalars.x) |
                                                              __float_as_uint(scalars.y) | __float_as_uint(scalars.z) | __float_as_uint(scalars.w));
      if (lane == 0) {
        asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(smem_u32(smem + M::kSeen + 4 * warp)), "r"(seen) : "memory");
        mbar_arrive(&bars[kSideEmpty + (c & 1)]);
      }
      return true;
    };
    auto leave_state = [&](int c) {
      leave(0, c, S, warp);
      if (lane == 0) mbar_arrive(&bars[kLargestReady]);
    };
    if (chunks > 0) {
      ok = ahead(0);
      leave(0, 1, S, warp);
      named_bar_sync(1, 32 * kWorkers);
      state = scale_for(__float_as_uint(largest_of(0, 1, kWorkers)));
      if (has_state) put(M::kS, M::kSlabS, row, S, state.up);
      if (ok) arrive(kStateReady);
      leave_state(0);
    }
    for (int c = 0; c < chunks; ++c) {
      const int64_t t = begin + static_cast<int64_t>(c) * kC + token;
      const bool live = t < length;
      ok = ok && all_wait(kLargestReady, c);
      if (!ok) break;
      const float largest = largest_of(0, c, kWorkers);
      const float decay = scalars.x, update = scalars.y;
      const float rest_bound = largest_of(1, c, kWorkers / 2) + scalars.z * largest;
      const Scale rest = scale_for(__float_as_uint(rest_bound));
      const Scale next = scale_for(__float_as_uint(fmaf(decay, largest, scalars.w * rest_bound)));
      float v[kCols];
      ok = all_wait(kFromStateDone, c);
      tc_fence_after();
      if (ok) take(kColD1, v);
      if (is_token) {
        // r = beta x - beta e^G h k
        const float from_state = fb * state.down;
#pragma unroll
        for (int i = 0; i < kCols; ++i) v[i] = live ? fmaf(-from_state, v[i], bx[i]) : 0.f;
        if (ok) put(M::kR, kSlab, token, v, rest.up);
      } else {
        const float from_state = fa * state.down;
#pragma unroll
        for (int i = 0; i < kCols; ++i) bx[i] = from_state * v[i];  // the state's part of y
      }
      if (ok) arrive(kRestReady);
      const float out_rest = fb * rest.down;
      if (c + 1 < chunks) ok = ok && ahead(c + 1);  // while the products run
      // the state
      ok = ok && all_wait(kUpdateDone, c);
      tc_fence_after();
      if (ok) take(kColD1, v);
      if (has_state) {
        const float back = update * rest.down;
#pragma unroll
        for (int i = 0; i < kCols; ++i) S[i] = fmaf(decay, S[i], back * v[i]);
      }
      state = next;
      const bool more = c + 1 < chunks;
      if (more && has_state && ok) put(M::kS, M::kSlabS, row, S, state.up);
      if (more && ok) arrive(kStateReady), leave_state(c + 1);
      // (the next P T r waits for these warps' next arrival, which comes after this)
      if (!is_token) ok = ok && all_wait(kRestDone, c);
      tc_fence_after();
      if (!is_token && ok) take(kColD3, v);
      if (!is_token && live && ok) {
        // y: the state's part, and P T r
#pragma unroll
        for (int i = 0; i < kCols; ++i) v[i] = fmaf(out_rest, v[i], bx[i]);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
          constexpr int kE = 16 / sizeof(T);
          if (col0 + kE * i >= p.P) break;
          uint4 w;
#pragma unroll
          for (int e = 0; e < 4; ++e) (&w.x)[e] = kP == 1 ? pack_bf16x2(v[kE * i + 2 * e % kE], v[kE * i + 2 * e % kE + 1]) : __float_as_uint(v[kE * i + e]);
          if (s.vectors) {
            *reinterpret_cast<uint4*>(y + t * y_token + kE * i) = w;
          } else {
#pragma unroll
            for (int e = 0; e < kE; ++e) y[t * y_token + kE * i + e] = reinterpret_cast<const T*>(&w)[e];
          }
        }
      }
    }
    if (!ok) {
#pragma unroll
      for (int i = 0; i < kCols; ++i) S[i] = __int_as_float(0x7FC00000);
    }
    float* to = s.last ? (p.final_state && seq.row >= 0 ? p.final_state + seq.row * p.H * p.P * N : nullptr) : s.carry + b * p.H * p.P * N;
    if (to && has_state) {
#pragma unroll
      for (int i = 0; i < kCols; ++i)
        if (col0 + i < p.P) to[(static_cast<int64_t>(h) * p.P + col0 + i) * N + row] = S[i];
    }
    // rows of y behind the sequence are 0; a wait that ran out leaves NaN
    const uint32_t rest = ok ? 0u : 0x7FC07FC0u;  // (a NaN in both types)
    for (int64_t t = (ok ? length : begin) + row; t < end; t += 128)
      for (int i = 0; i < kCols && col0 + i < p.P; i += 8) {
        if (s.vectors) {
#pragma unroll
          for (int e = 0; e < kP; ++e) reinterpret_cast<uint4*>(y + t * y_token + i)[e] = make_uint4(rest, rest, rest, rest);
        } else {
          for (int e = 0; e < 8; ++e) {
            if constexpr (kP == 1)
              y[t * y_token + i + e] = __ushort_as_bfloat16(static_cast<unsigned short>(rest));
            else
              y[t * y_token + i + e] = __uint_as_float(rest);
          }
        }
      }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWorkers) {
    tc_fence_after();
    tmem_dealloc(tmem, M::kTmem);
  }
}

template <typename T, int N, int kPT, int kGroups, int kStages, int kBlocks>
cudaError_t launch_walk(const DeltaParams& p, const DeltaChunks& s, cudaStream_t stream) {
  using M = Walk<T, N, kPT, kGroups, kStages>;
  constexpr int bytes = static_cast<int>(M::kTotal);
  static_assert(kBlocks * (bytes + 1024) <= 228 * 1024 && kBlocks * M::kTmem <= 512, "shared or tensor memory");
  auto kernel = delta_walk_kernel<T, N, kPT, kGroups, kStages, kBlocks>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  return launch_k(kernel, dim3(static_cast<unsigned>(ceil_div(p.P, kPT)), static_cast<unsigned>(p.H), static_cast<unsigned>(p.batch)),
                  dim3(M::kThreads), bytes, stream, true, p, s);
}

template <typename T, int N>
cudaError_t launch_chunks(const DeltaParams& p, const DeltaChunks& s, cudaStream_t stream) {
  constexpr int bytes = static_cast<int>(PrepSmem<T, N>::kTotal);
  cudaError_t e = cudaFuncSetAttribute(delta_prepare_kernel<T, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess)
    e = launch_k(delta_prepare_kernel<T, N>, dim3(static_cast<unsigned>(s.count), static_cast<unsigned>(p.H), static_cast<unsigned>(p.batch)),
                 dim3(kPrepThreads), bytes, stream, true, p, s);
  if (e != cudaSuccess) return e;
  // Columns of a block: as few as leave every block a multiprocessor of its own (the chain is the shorter, and what is
  // loaded for it the same), 32 where there are more, two blocks on each.  16 heads of 128 x 128, 16384 tokens:
  // 16 columns 379 us, 32 482; 128 heads, 4096 tokens: 32 columns 479 and, two blocks each, 360, 16 491 (all of an
  // earlier form; now 307 and 329 for the first and the last choice).
  const int64_t heads = p.batch * p.H, sms = layer_sm_count();
  // (64 columns, one block an SM: the walk of the last 385 us, when 32 had 355.)
  // 32-bit rows take twice the shared memory: one buffer, and one block on each.
  if constexpr (sizeof(T) == 4)
    return heads * ceil_div(p.P, 16) <= sms ? launch_walk<T, N, 16, 2, 1, 1>(p, s, stream) : launch_walk<T, N, 32, 2, 1, 1>(p, s, stream);
  else
    return heads * ceil_div(p.P, 16) <= sms ? launch_walk<T, N, 16, 2, 2, 1>(p, s, stream)
           : heads * ceil_div(p.P, 32) <= sms ? launch_walk<T, N, 32, 2, 2, 1>(p, s, stream)
                                              : launch_walk<T, N, 32, 2, 1, 2>(p, s, stream);
}

// Chunks of a pair of launches.  Pairs overlap, the first launch of one with the walk of the one before, but every
// walk begins and ends once more.  Where the walk leaves no room (more blocks than multiprocessors) pairs only limit
// the workspace.  16 heads, 16384 tokens: 48 MB 465 us, 64 MB 442, 128 MB 436, one pair 443; 128 heads, 4096 tokens:
// one pair 651, 48 MB 675 (both before the walk was as fast as now).
constexpr int64_t kPairBytes = int64_t(128) << 20, kPairBytesFull = int64_t(512) << 20;
// Sequences that would leave a pair fewer chunks than 16 are taken in parts, one after the other, so that a call's
// workspace is twice kPairBytesFull and a part's states at most (two chunks of all heads of one sequence, where that is
// more).  32 heads, 2048 tokens: 256 sequences at once 16.96 ms with 15.9 GB; in pairs of 8 chunks 18.1 with 8.2, of
// one 28.2 with 1.5; in parts of 16 sequences 17.1 with 1.0.
constexpr int64_t kPairChunks = 16;

int64_t bytes_of_chunk(const DeltaParams& p) { return p.batch * (int64_t(record_bytes(p.N, p.parts)) * p.H + int64_t(rows_bytes(p.N, p.parts)) * p.G); }
int64_t chunks_of(const DeltaParams& p) { return ceil_div(p.seqlen, kC); }
// Blocks of 16 columns leave multiprocessors without one: pairs that overlap pay.
bool few_blocks(const DeltaParams& p) { return p.batch * p.H * ceil_div(p.P, 16) <= layer_sm_count(); }
// All at once, in the place of two pairs.
bool one_pair(const DeltaParams& p) { return !few_blocks(p) && chunks_of(p) <= 2 * kPairBytesFull / bytes_of_chunk(p); }
// Sequences of a part, as even as they come.
int64_t sequences_at_once(const DeltaParams& p) {
  const int64_t chunks = chunks_of(p) < kPairChunks ? chunks_of(p) : kPairChunks, fit = kPairBytesFull / (chunks * (bytes_of_chunk(p) / p.batch));
  return one_pair(p) || fit >= p.batch ? p.batch : fit < 1 ? 1 : ceil_div(p.batch, ceil_div(p.batch, fit));
}
// Chunks of a pair, p.batch being a part's sequences.
int64_t chunks_at_once(const DeltaParams& p) {
  if (one_pair(p)) return chunks_of(p);
  const int64_t fit = (few_blocks(p) ? kPairBytes : kPairBytesFull) / bytes_of_chunk(p);
  return ceil_div(chunks_of(p), ceil_div(chunks_of(p), fit < 1 ? 1 : fit));
}
// A part of the sequences as a call of its own.
DeltaParams part_of(const DeltaParams& p, int64_t first, int64_t count) {
  DeltaParams q = p;
  const int64_t es = p.parts == 1 ? 2 : 4, gs = p.gate_f32 ? 4 : 2;
  auto on = [](const void* at, int64_t bytes) { return static_cast<const void*>(static_cast<const uint8_t*>(at) + bytes); };
  q.batch = count;
  q.x = on(p.x, first * p.x_batch * es), q.Bm = on(p.Bm, first * p.B_batch * es), q.Cm = on(p.Cm, first * p.C_batch * es);
  q.dt = on(p.dt, first * p.dt_batch * gs), q.beta = on(p.beta, first * p.beta_batch * gs);
  q.y = static_cast<uint8_t*>(p.y) + first * p.seqlen * p.H * p.P * es;
  if (p.slots) {
    q.slots = p.slots + first;
  } else {  // row b is sequence b's
    const int64_t state = first * p.H * p.P * p.N;
    q.nslots = p.nslots - first;
    if (p.init_state) q.init_state = p.init_state + state;
    if (p.final_state) q.final_state = p.final_state + state;
  }
  if (p.positions) q.positions = p.positions + first;
  if (p.lengths) q.lengths = p.lengths + first;
  return q;
}

}  // namespace

bool delta_chunked(int dtype, int64_t seqlen, int dstate) {
  (void)dtype;
  return (dstate == 64 || dstate == 128) && seqlen >= kMinTokens;
}

size_t delta_chunks_workspace(const DeltaParams& call) {
  DeltaParams p = call;
  p.batch = sequences_at_once(call);
  const int64_t count = chunks_at_once(p);
  const size_t pair = static_cast<size_t>(count * bytes_of_chunk(p));
  return count * kC >= p.seqlen ? pair : 2 * pair + static_cast<size_t>(p.batch) * p.H * p.P * p.N * sizeof(float);
}

ssd_status launch_delta_chunks(const DeltaParams& call, void* workspace, cudaStream_t stream) {
  DeltaChunks s{};
  s.limit_ns = spin_limit_ns();
  s.vectors = 1;
  for (const void* t : {call.x, call.Bm, call.Cm, (const void*)call.y}) s.vectors &= aligned_to(t, 16);
  for (int64_t stride : {call.x_batch, call.x_token, call.B_batch, call.B_token, call.C_batch, call.C_token}) s.vectors &= stride * (call.parts == 1 ? 2 : 4) % 16 == 0;
  const int64_t at_once = sequences_at_once(call);
  int64_t pair = 0;
  for (int64_t b = 0; b < call.batch; b += at_once) {
    DeltaParams p = part_of(call, b, at_once);  // (a full part's sizes give the buffers)
    const int64_t all = chunks_of(p), most = chunks_at_once(p), bytes = most * bytes_of_chunk(p);
    uint8_t* pairs = static_cast<uint8_t*>(workspace);  // two, used in turn
    s.carry = reinterpret_cast<float*>(pairs + 2 * bytes);
    if (call.batch - b < at_once) p.batch = call.batch - b;
    // Each launch is a dependent of the one before it in the stream and may begin beside it.  A walk waits for the
    // first launch of its pair, which ends after the walk before; a first launch writes a buffer whose last walk
    // ended before the present one began.
    for (int64_t first = 0; first < all; first += most, ++pair) {
      s.follows = pair > 0 && most < all;
      s.records = pairs + (most < all ? (pair & 1) * bytes : 0);
      s.rows = s.records + p.batch * p.H * most * record_bytes(p.N, p.parts);
      s.first = static_cast<int>(first), s.count = static_cast<int>(all - first < most ? all - first : most);
      s.last = first + most >= all;
      const cudaError_t e = p.parts == 1 ? (p.N == 64 ? launch_chunks<__nv_bfloat16, 64>(p, s, stream) : launch_chunks<__nv_bfloat16, 128>(p, s, stream))
                                         : (p.N == 64 ? launch_chunks<float, 64>(p, s, stream) : launch_chunks<float, 128>(p, s, stream));
      if (e != cudaSuccess) return SSD_ERR_CUDA;
    }
  }
  return SSD_OK;
}

}  // namespace ssd
