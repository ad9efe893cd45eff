// The gated delta rule for whole bf16 prompts, in chunks of 64 tokens on the tensor cores.
//
// With G the sum of dt A from the chunk's start to a token (that one included), k and q the normalised
// rows and h the state that enters the chunk, the values that the rule writes, v_i, solve
//     v_i + sum_{j<i} beta_i e^{G_i-G_j} (k_i.k_j) v_j = r_i,     r_i = beta_i (x_i - e^{G_i} h k_i),
// so with A that strictly lower triangular matrix and T = (I + A)^-1
//     v = T r,   y_i = scale (e^{G_i} h q_i + sum_{j<=i} e^{G_i-G_j} (q_i.k_j) v_j) = .. + (P T r)_i,
//     h <- e^{G_64} h + sum_j e^{G_64-G_j} v_j k_j^T.
// T, P T and the tokens' factors need no state: a first launch forms them for all chunks at once.  The
// second has a block for some columns of a head's state and walks the chunks: three products each, [K; Q] h,
// [T; P T] r and K^T v, with tokens or state rows in the 128 lanes of tensor memory.
//
// The state stays in registers, in 32 bits.  bf16 keeps 8 bits of a number, so r, v, h and T enter the
// products as three bf16 parts each (K and Q are bf16 as they come, P T goes into y alone and has two): parts
// lie side by side along the product's columns, and the threads add up what comes out.  Two parts would leave
// 2^-17 of every value, more than 32-bit sums lose.
#include "delta_chunk.cuh"

namespace ssd {
namespace {

constexpr int kC = 64;  // tokens of a chunk
constexpr int64_t kMinTokens = 64;
constexpr int64_t kRecordBytes = int64_t(1) << 40;

// What the first launch leaves of a chunk of a head: the parts of [T; P T] as shared memory holds them
// (rows of 128 bytes in the 128-byte swizzle; the third part has T alone), and the tokens' factors.
constexpr uint32_t kPartBytes = 16384, kTileBytes = 2 * kPartBytes + 8192;
enum { kBeta, kFromState, kToState, kFromStateOut, kDecay, kFactors };  // (of kDecay one number)
constexpr uint32_t kRecord = kTileBytes + kFactors * kC * 4;

// Four bytes of part `part` (0, 1, 2) of two neighbouring values.
__device__ __forceinline__ void split3(float a, float b, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  hi = pack_bf16x2(a, b);
  a -= bf16_lo(hi), b -= bf16_hi(hi);
  mid = pack_bf16x2(a, b);
  a -= bf16_lo(mid), b -= bf16_hi(mid);
  lo = pack_bf16x2(a, b);
}

// ------------------------------------------------------------------ first launch

constexpr int kPrepThreads = 128;
constexpr int kStrideA = 68, kStrideT = 72;  // (floats) rows that the fragments' and vectors' loads find in different banks

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int N>
struct PrepSmem {
  static constexpr uint32_t kRow = N * 2 + 16;  // bytes of a row of K or Q, eight rows in different banks
  static constexpr uint32_t kRows = 128 * kRow, kMats = 2 * kC * kStrideA * 4;
  static constexpr uint32_t kT = kRows > kMats ? kRows : kMats;  // A and P take the rows' place
  static constexpr uint32_t kVec = kT + kC * kStrideT * 4;
  static constexpr uint32_t kTotal = kVec + 5 * kC * 4 + 16;
};

template <int N>
__global__ void __launch_bounds__(kPrepThreads, 4) delta_prepare_kernel(DeltaParams p, DeltaChunks s) {
  using M = PrepSmem<N>;
  extern __shared__ __align__(16) uint8_t smem[];
  float* s_A = reinterpret_cast<float*>(smem);
  float* s_P = s_A + kC * kStrideA;
  float* s_T = reinterpret_cast<float*>(smem + M::kT);
  float* s_hi = reinterpret_cast<float*>(smem + M::kVec);
  float *s_lo = s_hi + kC, *s_beta = s_lo + kC, *s_kn = s_beta + kC, *s_qn = s_kn + kC;
  int64_t* s_half = reinterpret_cast<int64_t*>(s_qn + kC);
  begin_kernel();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t b = blockIdx.z;
  const int h = blockIdx.y, chunk = s.first + blockIdx.x;
  const DeltaSeq seq = delta_sequence(p, b);
  const int64_t t0 = static_cast<int64_t>(chunk) * kC;
  if (seq.row < 0 || t0 >= seq.length) return;
  const int n = seq.length - t0 < kC ? static_cast<int>(seq.length - t0) : kC;
  const int g = h / (p.H / p.G);

  // rows of K, then of Q, with the sums of their squares; rows behind the sequence are 0
  constexpr int kRowLanes = N / 8, kPer = 32 / kRowLanes, kLoads = 32 / kPer;
  const __nv_bfloat16* from[2] = {static_cast<const __nv_bfloat16*>(p.Bm) + b * p.B_batch + t0 * p.B_token + static_cast<int64_t>(g) * N,
                                  static_cast<const __nv_bfloat16*>(p.Cm) + b * p.C_batch + t0 * p.C_token + static_cast<int64_t>(g) * N};
  uint4 raw[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = warp * 32 + i * kPer + lane / kRowLanes, t = r & 63;
    raw[i] = make_uint4(0, 0, 0, 0);
    if (t < n) raw[i] = *reinterpret_cast<const uint4*>((r < kC ? from[0] + t * p.B_token : from[1] + t * p.C_token) + lane % kRowLanes * 8);
  }
  // G in whole numbers of 2^-32 (base 2; a token's decay is 2^-1000 at least, which is 0), kept as two
  // 32-bit numbers, the first of few enough bits that differences of it are exact
  if (tid < kC) {
    float d = 0.f, beta = 0.f;
    if (tid < n) d = delta_log_decay<__nv_bfloat16>(p, b, t0 + tid, h) * kLog2e, beta = delta_beta<__nv_bfloat16>(p, b, t0 + tid, h);
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
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = warp * 32 + i * kPer + lane / kRowLanes;
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
    float squares = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) squares = fmaf(bf16_lo(w[e]), bf16_lo(w[e]), fmaf(bf16_hi(w[e]), bf16_hi(w[e]), squares));
#pragma unroll
    for (int o = kRowLanes / 2; o; o /= 2) squares += __shfl_xor_sync(0xffffffffu, squares, o);
    *reinterpret_cast<uint4*>(smem + r * M::kRow + lane % kRowLanes * 16) = raw[i];
    if (lane % kRowLanes == 0) (r < kC ? s_kn : s_qn)[r & 63] = delta_norm(p, squares);
  }
  __syncthreads();

  // K K^T and Q K^T, 16 rows a warp of each (those with fewest columns beside those with most)
  float acc[2][8][4];
  const int mt[2] = {warp, 3 - warp};
  const uint32_t rows = smem_u32(smem);
#pragma unroll
  for (int m = 0; m < 2; ++m) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[m][i][e] = 0.f;
    const uint32_t at = rows + (64 * m + 16 * mt[m] + (lane & 15)) * M::kRow + (lane >> 4) * 16;
    const uint32_t bt = rows + ((lane & 7) + (lane >> 4) * 8) * M::kRow + ((lane >> 3) & 1) * 16;
#pragma unroll
    for (int k = 0; k < N / 16; ++k) {
      uint32_t a[4];
      ldmatrix4(a, at + k * 32);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j > mt[m]) break;
        uint32_t v[4];
        ldmatrix4(v, bt + j * 16 * M::kRow + k * 32);
        mma_bf16(acc[m][2 * j], a, v[0], v[1]);
        mma_bf16(acc[m][2 * j + 1], a, v[2], v[3]);
      }
    }
  }
  __syncthreads();  // the rows have been read
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j > 2 * mt[m] + 1) break;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = 16 * mt[m] + (lane >> 2) + (e >> 1) * 8, col = 8 * j + (lane & 3) * 2 + (e & 1);
        const float decay = exp2f((s_hi[row] - s_hi[col]) + (s_lo[row] - s_lo[col])) * s_kn[col] * acc[m][j][e];
        if (m == 0)
          s_A[row * kStrideA + col] = col < row && row < n ? decay * s_kn[row] * s_beta[row] : 0.f;
        else
          s_P[row * kStrideA + col] = col <= row && row < n ? decay * s_qn[row] * p.scale : 0.f;
      }
    }
  __syncthreads();

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
        const float4 a = *reinterpret_cast<const float4*>(&s_A[(d0 + r) * kStrideA + d0 + k4]);
        sum = fmaf(-a.x, v[k4], sum);
        if (k4 + 1 < r) sum = fmaf(-a.y, v[k4 + 1], sum);
        if (k4 + 2 < r) sum = fmaf(-a.z, v[k4 + 2], sum);
        if (k4 + 3 < r) sum = fmaf(-a.w, v[k4 + 3], sum);
      }
      v[r] = sum;
      s_T[(d0 + r) * kStrideT + d0 + c] = sum;
    }
  }
  __syncthreads();
  const int c = tid & 15, r = tid >> 4 << 1;  // a thread's column and two rows of every block
#pragma unroll
  for (int d = 1; d < 4; ++d) {
    float w[3][2];
#pragma unroll
    for (int j = 0; j + d < 4; ++j) {
      const int i = j + d;
      float s0 = 0.f, s1 = 0.f;
#pragma unroll 4
      for (int k = 16 * j; k < 16 * i; k += 4) {
        const float4 a0 = *reinterpret_cast<const float4*>(&s_A[(16 * i + r) * kStrideA + k]);
        const float4 a1 = *reinterpret_cast<const float4*>(&s_A[(16 * i + r + 1) * kStrideA + k]);
        const float* t = &s_T[k * kStrideT + 16 * j + c];
        s0 = fmaf(a0.x, t[0], s0), s1 = fmaf(a1.x, t[0], s1);
        s0 = fmaf(a0.y, t[kStrideT], s0), s1 = fmaf(a1.y, t[kStrideT], s1);
        s0 = fmaf(a0.z, t[2 * kStrideT], s0), s1 = fmaf(a1.z, t[2 * kStrideT], s1);
        s0 = fmaf(a0.w, t[3 * kStrideT], s0), s1 = fmaf(a1.w, t[3 * kStrideT], s1);
      }
      s_T[(16 * i + r) * kStrideT + 16 * j + c] = s0;
      s_T[(16 * i + r + 1) * kStrideT + 16 * j + c] = s1;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j + d < 4; ++j) {
      const int i = j + d;
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int k = 0; k < 16; k += 4) {
        const float4 a0 = *reinterpret_cast<const float4*>(&s_T[(16 * i + r) * kStrideT + 16 * i + k]);
        const float4 a1 = *reinterpret_cast<const float4*>(&s_T[(16 * i + r + 1) * kStrideT + 16 * i + k]);
        const float* t = &s_T[(16 * i + k) * kStrideT + 16 * j + c];
        // (above the diagonal T has not been written)
        s0 = fmaf(k <= r ? a0.x : 0.f, t[0], s0), s1 = fmaf(k <= r + 1 ? a1.x : 0.f, t[0], s1);
        s0 = fmaf(k + 1 <= r ? a0.y : 0.f, t[kStrideT], s0), s1 = fmaf(k + 1 <= r + 1 ? a1.y : 0.f, t[kStrideT], s1);
        s0 = fmaf(k + 2 <= r ? a0.z : 0.f, t[2 * kStrideT], s0), s1 = fmaf(k + 2 <= r + 1 ? a1.z : 0.f, t[2 * kStrideT], s1);
        s0 = fmaf(k + 3 <= r ? a0.w : 0.f, t[3 * kStrideT], s0), s1 = fmaf(k + 3 <= r + 1 ? a1.w : 0.f, t[3 * kStrideT], s1);
      }
      w[j][0] = -s0, w[j][1] = -s1;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j + d < 4; ++j) {
      s_T[(16 * (j + d) + r) * kStrideT + 16 * j + c] = w[j][0];
      s_T[(16 * (j + d) + r + 1) * kStrideT + 16 * j + c] = w[j][1];
    }
    __syncthreads();
  }

  // P T in place of A: TF32 products, each factor as two parts (2^-22 of it is left out)
  {
    const int m = warp, gr = lane >> 2, gc = lane & 3;
    const float* prow = &s_P[(16 * m + gr) * kStrideA + gc];
    for (int j = 0; j <= 2 * m + 1; ++j) {
      float o[4] = {0.f, 0.f, 0.f, 0.f};
      for (int k = j; k <= 2 * m + 1; ++k) {
        const float a[4] = {prow[8 * k], prow[8 * kStrideA + 8 * k], prow[8 * k + 4], prow[8 * kStrideA + 8 * k + 4]};
        // T above the diagonal is 0 (and has not been written)
        const int k0 = 8 * k + gc, col = 8 * j + gr;
        const float t[2] = {col <= k0 ? s_T[k0 * kStrideT + col] : 0.f, col <= k0 + 4 ? s_T[(k0 + 4) * kStrideT + col] : 0.f};
        uint32_t ah[4], al[4], th[2], tl[2];
#pragma unroll
        for (int e = 0; e < 4; ++e) ah[e] = __float_as_uint(round_tf32(a[e])), al[e] = __float_as_uint(a[e] - __uint_as_float(ah[e]));
#pragma unroll
        for (int e = 0; e < 2; ++e) th[e] = __float_as_uint(round_tf32(t[e])), tl[e] = __float_as_uint(t[e] - __uint_as_float(th[e]));
        mma_tf32(o, al, th[0], th[1]);
        mma_tf32(o, ah, tl[0], tl[1]);
        mma_tf32(o, ah, th[0], th[1]);
      }
      float* to = &s_A[(16 * m + gr) * kStrideA + 8 * j + 2 * gc];
      to[0] = o[0], to[1] = o[1], to[8 * kStrideA] = o[2], to[8 * kStrideA + 1] = o[3];
    }
  }
  __syncthreads();

  uint8_t* out = s.records + ((b * p.H + h) * s.count + blockIdx.x) * static_cast<int64_t>(kRecord);
#pragma unroll 2
  for (int i = 0; i < 8; ++i) {
    const int item = tid + kPrepThreads * i, row = item >> 3, q = item & 7, t = row & 63;
    const float* src = row < kC ? &s_T[t * kStrideT + 8 * q] : &s_A[t * kStrideA + 8 * q];
    uint4 hi, mid, lo;
    uint32_t *ph = &hi.x, *pm = &mid.x, *pl = &lo.x;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int col = 8 * q + 2 * e;
      const float2 v = *reinterpret_cast<const float2*>(src + 2 * e);
      split3(col <= t ? v.x : 0.f, col + 1 <= t ? v.y : 0.f, ph[e], pm[e], pl[e]);
    }
    uint8_t* to = out + row * 128 + ((q ^ (row & 7)) << 4);
    *reinterpret_cast<uint4*>(to) = hi;
    *reinterpret_cast<uint4*>(to + kPartBytes) = mid;
    if (row < kC) *reinterpret_cast<uint4*>(to + 2 * kPartBytes) = lo;
  }
  if (tid < kC) {
    float* factors = reinterpret_cast<float*>(out + kTileBytes);
    const float since = exp2f(s_hi[tid] + s_lo[tid]);
    const float until = exp2f((s_hi[kC - 1] - s_hi[tid]) + (s_lo[kC - 1] - s_lo[tid]));
    factors[kBeta * kC + tid] = s_beta[tid];
    factors[kFromState * kC + tid] = s_beta[tid] * s_kn[tid] * since;
    factors[kToState * kC + tid] = s_kn[tid] * until;
    factors[kFromStateOut * kC + tid] = p.scale * s_qn[tid] * since;
    if (tid == kC - 1) factors[kDecay * kC] = since;
  }
}

// ------------------------------------------------------------------ second launch

constexpr int kGroups = 4;                      // warpgroups that share a tile's columns
constexpr int kWorkers = 16;                    // their warps
constexpr int kThreads = 32 * (kWorkers + 2);   // and one that loads, one that issues the products

struct WalkMaps {
  CUtensorMap k, q;  // Bm, Cm [B][L][G][N], box {64 n, 1, 64 tokens, 1}
};

// kPT: columns of the state (values of a head) that a block has.
template <int N, int kPT>
struct WalkSmem {
  static constexpr uint32_t kStage = N / 64 * 16384;          // per 64 n: 64 rows of K, then of Q
  static constexpr int kTiles = kPT == 32 ? 2 : 1;            // buffers of [T; P T]
  static constexpr uint32_t kTile = 3 * kPartBytes;           // the third part's lower half stays 0
  static constexpr int kSlabs = (3 * kPT + 63) / 64;          // 64 columns each of the parts side by side
  static constexpr uint32_t kSlabS = N * 128, kSlabR = kC * 128;
  static constexpr uint32_t kKQ = 0, kA = kKQ + 2 * kStage, kS = kA + kTiles * kTile, kR = kS + kSlabs * kSlabS;
  static constexpr uint32_t kBars = kR + kSlabs * kSlabR, kTotal = kBars + 16 * 8 + 16 + 1024;
};

enum { kKQFull, kKQFull1, kKQEmpty, kKQEmpty1, kTFull, kTFull1, kTEmpty, kTEmpty1, kStateReady, kFromStateDone, kRestReady,
       kValuesDone, kValuesReady, kUpdateDone, kDrained, kBarriers };

// cp.async.bulk: bytes from global to shared memory, counted by the barrier.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
               "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

template <int kCols>
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&r)[kCols]) {
  if constexpr (kCols == 16) {
    tmem_ld16(at, r);
  } else {
    static_assert(kCols == 8);
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(at));
  }
}

template <int N, int kPT>
__global__ void __launch_bounds__(kThreads, 1) delta_walk_kernel(DeltaParams p, DeltaChunks s, const __grid_constant__ WalkMaps maps) {
  using M = WalkSmem<N, kPT>;
  constexpr int kCols = kPT / kGroups;  // of a thread
  constexpr uint32_t kColD1 = 0, kColD3 = 256;  // K^T v goes where [K; Q] h was
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + M::kBars);
  uint32_t* holder = reinterpret_cast<uint32_t*>(bars + kBarriers);
  volatile int* failed = reinterpret_cast<volatile int*>(holder + 1);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t b = blockIdx.z;
  const int h = blockIdx.y, p0 = blockIdx.x * kPT;
  if (tid == 0) {
    for (int i = 0; i < kBarriers; ++i) mbar_init(&bars[i], i == kStateReady || i == kRestReady || i == kValuesReady ? kWorkers : 1);
    fence_mbar_init();
    *failed = 0;
  }
  if (warp == kWorkers) {
    tmem_alloc(holder, 512);
    tmem_relinquish();
  }
  // rows 64 to 127 of the third part
  for (int i = tid; i < M::kTiles * 512; i += kThreads)
    *reinterpret_cast<uint4*>(smem + M::kA + (i >> 9) * M::kTile + 2 * kPartBytes + 8192 + (i & 511) * 16) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
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
  const uint8_t* records = s.records + (b * p.H + h) * s.count * static_cast<int64_t>(kRecord);
  const int g = h / (p.H / p.G);
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

  if (warp == kWorkers) {
    // loads
    if (lane == 0) {
      int c = 0, t = 0;  // chunks whose rows, and whose tiles, are on their way
      bool ok = true;
      for (; c < chunks && ok; ++c) {
        const int st = c & 1, ts = c % M::kTiles;
        ok = c < 2 || wait(kKQEmpty + st, (c >> 1) - 1);
        if (!ok) break;
        mbar_arrive_expect_tx(&bars[kKQFull + st], M::kStage);
        for (int a = 0; a < N / 64; ++a) {
          uint8_t* to = smem + M::kKQ + st * M::kStage + a * 16384;
          tma_load_4d(to, &maps.k, &bars[kKQFull + st], a * 64, g, static_cast<int>(begin) + c * kC, static_cast<int>(b));
          tma_load_4d(to + 8192, &maps.q, &bars[kKQFull + st], a * 64, g, static_cast<int>(begin) + c * kC, static_cast<int>(b));
        }
        ok = c < M::kTiles || wait(kTEmpty + ts, c / M::kTiles - 1);
        if (!ok) {
          ++c;
          break;
        }
        mbar_arrive_expect_tx(&bars[kTFull + ts], kTileBytes);
        bulk_load(smem + M::kA + ts * M::kTile, records + c * static_cast<int64_t>(kRecord), kTileBytes, &bars[kTFull + ts]);
        t = c + 1;
      }
      if (!ok || *failed) {  // nothing is in flight when the block ends
        for (int i = c > 2 ? c - 2 : 0; i < c; ++i) mbar_wait(&bars[kKQFull + (i & 1)], (i >> 1) & 1, s.limit_ns);
        for (int i = t > M::kTiles ? t - M::kTiles : 0; i < t; ++i)
          mbar_wait(&bars[kTFull + i % M::kTiles], (i / M::kTiles) & 1, s.limit_ns);
      }
    }
  } else if (warp == kWorkers + 1) {
    // products
    if (lane == 0) {
      constexpr uint32_t id_state = idesc_f32acc(1, 128, 3 * kPT, 0, 1), id_two = idesc_f32acc(1, 128, 2 * kPT, 0, 1),
                         id_one = idesc_f32acc(1, 128, kPT, 0, 1), id_update = idesc_f32acc(1, 128, 3 * kPT, 1, 1);
      const uint32_t base = smem_u32(smem);
      const uint64_t dS = sdesc_sw128(base + M::kS, M::kSlabS, 1024), dR = sdesc_sw128(base + M::kR, M::kSlabR, 1024);
      bool ok = true;
      int c = 0;
      for (; c < chunks && ok; ++c) {
        const int st = c & 1, ts = c % M::kTiles;
        const uint32_t kq = base + M::kKQ + st * M::kStage, tile = base + M::kA + ts * M::kTile;
        ok = wait(kKQFull + st, c >> 1) && wait(kStateReady, c);
        if (!ok) break;
        tc_fence_after();
        const uint64_t rows = sdesc_sw128(kq, 16, 1024);
#pragma unroll
        for (int k = 0; k < N / 16; ++k)
          mma_ss<false>(tmem + kColD1, rows + ((k >> 2) * 16384 + (k & 3) * 32 >> 4), dS + (k * 2048 >> 4), id_state, k != 0);
        mma_commit(&bars[kFromStateDone]);
        ok = wait(kTFull + ts, c / M::kTiles) && wait(kRestReady, c);
        if (!ok) break;
        tc_fence_after();
        const uint64_t t0 = sdesc_sw128(tile, 16, 1024);
#pragma unroll
        for (int k = 0; k < kC / 16; ++k) {  // all parts that matter: their indexes add up to two at most
          mma_ss<false>(tmem + kColD3, t0 + (k * 32 >> 4), dR + (k * 2048 >> 4), id_state, k != 0);
          mma_ss<false>(tmem + kColD3, t0 + (kPartBytes + k * 32 >> 4), dR + (k * 2048 >> 4), id_two, 1);
          mma_ss<false>(tmem + kColD3, t0 + (2 * kPartBytes + k * 32 >> 4), dR + (k * 2048 >> 4), id_one, 1);
        }
        mma_commit(&bars[kValuesDone]);
        mma_commit(&bars[kTEmpty + ts]);
        ok = wait(kValuesReady, c);
        if (!ok) break;
        tc_fence_after();
        const uint64_t kt = sdesc_sw128(kq, 16384, 1024);
#pragma unroll
        for (int k = 0; k < kC / 16; ++k)
          mma_ss<false>(tmem + kColD1, kt + (k * 2048 >> 4), dR + (k * 2048 >> 4), id_update, k != 0);
        mma_commit(&bars[kUpdateDone]);
        mma_commit(&bars[kKQEmpty + st]);
      }
      mma_commit(&bars[kDrained]);
      mbar_wait(&bars[kDrained], 0, s.limit_ns);
    }
  } else {
    // the state, and everything between the products
    const int group = warp >> 2, quarter = warp & 3;
    const int row = 32 * quarter + lane;  // of tensor memory: token (and 64 more: its output) or state row
    const bool has_state = row < N, is_token = quarter < 2;
    const int token = row & 63;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * quarter) << 16) + group * kCols;
    const int col0 = p0 + group * kCols;  // the thread's values of the head
    const int64_t y_token = static_cast<int64_t>(p.H) * p.P;
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y) + b * p.seqlen * y_token + static_cast<int64_t>(h) * p.P + col0;
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x) + b * p.x_batch + static_cast<int64_t>(h) * p.P + col0;

    // kCols values of a row as parts side by side: row * 128 bytes in slabs of 64 columns
    auto put = [&](uint32_t tile, uint32_t slab, int at_row, const float (&v)[kCols]) {
      uint32_t part[3][kCols / 2];
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) split3(v[2 * i], v[2 * i + 1], part[0][i], part[1][i], part[2][i]);
#pragma unroll
      for (int r = 0; r < 3; ++r)
#pragma unroll
        for (int i = 0; i < kCols / 8; ++i) {
          const int col = r * kPT + group * kCols + 8 * i;
          *reinterpret_cast<uint4*>(smem + tile + (col >> 6) * slab + at_row * 128 + ((((col & 63) >> 3) ^ (at_row & 7)) << 4)) =
              make_uint4(part[r][4 * i], part[r][4 * i + 1], part[r][4 * i + 2], part[r][4 * i + 3]);
        }
    };
    // the three parts' sums of kCols columns
    auto take = [&](uint32_t at, float (&v)[kCols]) {
      uint32_t a[kCols], c[kCols], d[kCols];
      tmem_load<kCols>(lanes + at + 2 * kPT, d);
      tmem_load<kCols>(lanes + at + kPT, c);
      tmem_load<kCols>(lanes + at, a);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < kCols; ++i) v[i] = __uint_as_float(a[i]) + (__uint_as_float(c[i]) + __uint_as_float(d[i]));
    };
    auto all_wait = [&](int bar, int phase) { return __all_sync(0xffffffffu, wait(bar, phase)) != 0; };
    auto arrive = [&](int bar) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[bar]);
    };

    float S[kCols];
    {
      const float* from = s.first == 0 ? seq.row >= 0 && seq.resumed ? p.init_state + seq.row * p.H * p.P * N : nullptr
                                       : s.carry + b * p.H * p.P * N;
#pragma unroll
      for (int i = 0; i < kCols; ++i)
        S[i] = from && has_state && col0 + i < p.P ? from[(static_cast<int64_t>(h) * p.P + col0 + i) * N + row] : 0.f;
    }
    // what comes from global memory is asked for a chunk ahead
    uint4 next_x[kCols / 8];
    float next_a = 0.f, next_b = 0.f, next_c = 0.f, next_decay = 0.f;
    auto ask = [&](int c) {
      if (c >= chunks) return;
      const float* f = reinterpret_cast<const float*>(records + c * static_cast<int64_t>(kRecord) + kTileBytes);
      const int64_t t = begin + static_cast<int64_t>(c) * kC + token;
      next_decay = f[kDecay * kC];
      if (is_token) {
        next_a = f[kBeta * kC + token], next_b = f[kFromState * kC + token], next_c = f[kToState * kC + token];
#pragma unroll
        for (int i = 0; i < kCols / 8; ++i) {
          next_x[i] = make_uint4(0, 0, 0, 0);
          if (t < length && col0 + 8 * i < p.P) next_x[i] = *reinterpret_cast<const uint4*>(x + t * p.x_token + 8 * i);
        }
      } else {
        next_a = f[kFromStateOut * kC + token];
      }
    };
    ask(0);
    if (chunks > 0) {
      if (has_state) put(M::kS, M::kSlabS, row, S), fence_proxy_async_smem();
      arrive(kStateReady);
    }
    bool ok = true;
    for (int c = 0; c < chunks; ++c) {
      const int64_t t = begin + static_cast<int64_t>(c) * kC + token;
      const bool live = t < length;
      const float fa = next_a, fb = next_b, fc = next_c, decay = next_decay;
      uint4 xs[kCols / 8];
#pragma unroll
      for (int i = 0; i < kCols / 8; ++i) xs[i] = next_x[i];
      ask(c + 1);
      float v[kCols], out[kCols];
      // r = beta x - beta e^G h k, and the state's part of y
      if (!(ok = all_wait(kFromStateDone, c))) break;
      tc_fence_after();
      take(kColD1, v);
      if (is_token) {
#pragma unroll
        for (int i = 0; i < kCols; ++i) {
          const uint32_t w = (&xs[i / 8].x)[i / 2 % 4];
          v[i] = live ? fmaf(fa, i & 1 ? bf16_hi(w) : bf16_lo(w), -fb * v[i]) : 0.f;
        }
        put(M::kR, M::kSlabR, token, v);
        if (!live) {  // K's rows behind the sequence, which the state's product multiplies by 0
          for (int a = 0; a < N / 64; ++a)
            for (int i = 2 * group; i < 2 * group + 2; ++i)
              *reinterpret_cast<uint4*>(smem + M::kKQ + (c & 1) * M::kStage + a * 16384 + token * 128 + i * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      } else {
#pragma unroll
        for (int i = 0; i < kCols; ++i) out[i] = fa * v[i];
      }
      arrive(kRestReady);
      // v = T r, as the state takes it
      if (!(ok = all_wait(kValuesDone, c))) break;
      tc_fence_after();
      take(kColD3, v);
      if (is_token) {
#pragma unroll
        for (int i = 0; i < kCols; ++i) v[i] = live ? fc * v[i] : 0.f;
        put(M::kR, M::kSlabR, token, v);
        fence_proxy_async_smem();
      }
      arrive(kValuesReady);
      if (!is_token && live) {
#pragma unroll
        for (int i = 0; i < kCols / 8; ++i) {
          if (col0 + 8 * i >= p.P) break;
          uint4 w;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            (&w.x)[e] = pack_bf16x2(out[8 * i + 2 * e] + v[8 * i + 2 * e], out[8 * i + 2 * e + 1] + v[8 * i + 2 * e + 1]);
          *reinterpret_cast<uint4*>(y + t * y_token + 8 * i) = w;
        }
      }
      // the state
      if (!(ok = all_wait(kUpdateDone, c))) break;
      tc_fence_after();
      take(kColD1, v);
      if (has_state) {
#pragma unroll
        for (int i = 0; i < kCols; ++i) S[i] = fmaf(decay, S[i], v[i]);
        if (c + 1 < chunks) put(M::kS, M::kSlabS, row, S), fence_proxy_async_smem();
      }
      if (c + 1 < chunks) arrive(kStateReady);
    }
    const float poison = __int_as_float(0x7FC00000);
    if (!ok) {
#pragma unroll
      for (int i = 0; i < kCols; ++i) S[i] = poison;
    }
    float* to = s.last ? (p.final_state && seq.row >= 0 ? p.final_state + seq.row * p.H * p.P * N : nullptr) : s.carry + b * p.H * p.P * N;
    if (to && has_state) {
#pragma unroll
      for (int i = 0; i < kCols; ++i)
        if (col0 + i < p.P) to[(static_cast<int64_t>(h) * p.P + col0 + i) * N + row] = S[i];
    }
    // rows of y behind the sequence are 0; a wait that ran out leaves NaN
    const uint32_t rest = ok ? 0u : 0x7FC07FC0u;
    for (int64_t t = (ok ? length : begin) + row; t < end; t += 128)
      for (int i = 0; i < kCols; i += 8)
        if (col0 + i < p.P) *reinterpret_cast<uint4*>(y + t * y_token + i) = make_uint4(rest, rest, rest, rest);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWorkers) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int N, int kPT>
cudaError_t launch_walk(const DeltaParams& p, const DeltaChunks& s, const WalkMaps& maps, cudaStream_t stream) {
  constexpr int bytes = static_cast<int>(WalkSmem<N, kPT>::kTotal);
  static_assert(bytes <= 227 * 1024, "shared memory");
  const cudaError_t e = cudaFuncSetAttribute(delta_walk_kernel<N, kPT>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  return launch_k(delta_walk_kernel<N, kPT>, dim3(static_cast<unsigned>(ceil_div(p.P, kPT)), static_cast<unsigned>(p.H), static_cast<unsigned>(p.batch)),
                  dim3(kThreads), bytes, stream, true, p, s, maps);
}

template <int N>
cudaError_t launch_chunks(const DeltaParams& p, const DeltaChunks& s, const WalkMaps& maps, cudaStream_t stream) {
  constexpr int bytes = static_cast<int>(PrepSmem<N>::kTotal);
  cudaError_t e = cudaFuncSetAttribute(delta_prepare_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess)
    e = launch_k(delta_prepare_kernel<N>, dim3(static_cast<unsigned>(s.count), static_cast<unsigned>(p.H), static_cast<unsigned>(p.batch)),
                 dim3(kPrepThreads), bytes, stream, true, p, s);
  if (e != cudaSuccess) return e;
  const bool narrow = p.batch * p.H * ceil_div(p.P, 32) <= layer_sm_count();
  return narrow ? launch_walk<N, 32>(p, s, maps, stream) : launch_walk<N, 64>(p, s, maps, stream);
}

}  // namespace

bool delta_chunked(int dtype, int64_t seqlen, int dstate) {
  return dtype == SSD_BF16 && (dstate == 64 || dstate == 128) && seqlen >= kMinTokens;
}

// Chunks of a pair of launches: as many as keep their records within half the L2.
static int64_t chunks_at_once(const DeltaParams& p) {
  const int64_t all = ceil_div(p.seqlen, kC), fit = kRecordBytes / (kRecord * p.batch * p.H);
  return fit < 8 ? (all < 8 ? all : 8) : fit < all ? fit : all;
}

size_t delta_chunks_workspace(const DeltaParams& p) {
  const int64_t heads = p.batch * p.H, count = chunks_at_once(p);
  return static_cast<size_t>(heads * count * kRecord) +
         (count * kC < p.seqlen ? static_cast<size_t>(heads) * p.P * p.N * sizeof(float) : 0);
}

bool delta_chunks_aligned(const DeltaParams& p) {
  for (const void* t : {p.x, p.Bm, p.Cm, (const void*)p.y})
    if (!aligned_to(t, 16)) return false;
  // (8 values are 16 bytes; a dimension of one element may have any stride, but the map wants a valid one)
  for (int64_t stride : {p.x_batch, p.x_token, p.B_batch, p.B_token, p.C_batch, p.C_token})
    if (stride < 8 || stride % 8 != 0 || stride >= int64_t(1) << 38) return false;
  return true;
}

ssd_status launch_delta_chunks(const DeltaParams& p, void* workspace, cudaStream_t stream) {
  WalkMaps maps;
  for (int i = 0; i < 2; ++i) {
    const uint64_t dims[4] = {static_cast<uint64_t>(p.N), static_cast<uint64_t>(p.G), static_cast<uint64_t>(p.seqlen), static_cast<uint64_t>(p.batch)};
    const uint64_t strides[3] = {static_cast<uint64_t>(p.N) * 2, static_cast<uint64_t>(i ? p.C_token : p.B_token) * 2,
                                 static_cast<uint64_t>(i ? p.C_batch : p.B_batch) * 2};
    const uint32_t box[4] = {64, 1, kC, 1};
    if (!encode_bf16_map(i ? &maps.q : &maps.k, 4, i ? p.Cm : p.Bm, dims, strides, box)) return SSD_ERR_CUDA;
  }
  const int64_t all = ceil_div(p.seqlen, kC), most = chunks_at_once(p);
  DeltaChunks s{};
  s.records = static_cast<uint8_t*>(workspace);
  s.carry = reinterpret_cast<float*>(s.records + p.batch * p.H * most * kRecord);
  s.limit_ns = spin_limit_ns();
  for (int64_t first = 0; first < all; first += most) {
    s.first = static_cast<int>(first), s.count = static_cast<int>(all - first < most ? all - first : most);
    s.last = first + most >= all;
    const cudaError_t e = p.N == 64 ? launch_chunks<64>(p, s, maps, stream) : launch_chunks<128>(p, s, maps, stream);
    if (e != cudaSuccess) return SSD_ERR_CUDA;
  }
  return SSD_OK;
}

}  // namespace ssd
