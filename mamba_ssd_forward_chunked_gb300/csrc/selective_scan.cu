// The selective scan: a recurrence with its own decay for every channel c and
// state n, d_t[c] the step:
//   h_t[c][n] = exp(d_t[c] A[c][n]) h_{t-1}[c][n] + d_t[c] u_t[c] B_t[n]
//   y_t[c] = (sum_n h_t[c][n] C_t[n] + D[c] u_t[c]) silu(z_t[c]).
//
// Work and split.  Per token and state one exponential and three multiply-adds:
// at 16 states the special-function unit and the issue slots bound it, not
// memory.  A block takes 32 channels, four lanes a channel, each lane a quarter
// of the states, and walks down the tokens in tiles of 32: the tile's u, delta,
// z, B and C come by 16-byte loads one tile ahead (in registers while the tile
// before is computed), the steps are put through softplus once and kept with
// d u in shared memory, the states stay in registers, multiply-adds go two at a
// time (f32x2).  Four tokens' sums are joined over the four lanes together:
// three shuffles for four tokens, and every lane ends with one token's sum.
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

constexpr int kThreads = 128;
constexpr int kLanes = 4;      // lanes a channel
constexpr int kChannels = kThreads / kLanes;
constexpr int kTile = 32;      // tokens a tile
constexpr int kYRow = 40;      // floats a row of sums: four rows of 8 channels fall into different banks
constexpr float kLog2e = 1.4426950408889634f;

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
};

// Eight consecutive values as they lie in memory.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void set(int i, __nv_bfloat16 x) {
    const uint32_t bits = __bfloat16_as_ushort(x);
    uint32_t* w = &v.x;
    w[i / 2] = i % 2 ? (w[i / 2] & 0xFFFFu) | (bits << 16) : (w[i / 2] & 0xFFFF0000u) | bits;
  }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t w = (&v.x)[i / 2];
    return __uint_as_float(i % 2 ? w & 0xFFFF0000u : w << 16);
  }
};
template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void set(int i, float x) { (i < 4 ? &a.x : &b.x)[i % 4] = x; }
  __device__ __forceinline__ float get(int i) const { return (i < 4 ? &a.x : &b.x)[i % 4]; }
};

// Eight values from p, the first n of them there (0 for the rest).  kVec: all or none, 16-byte aligned.
template <typename T, bool kVec>
__device__ __forceinline__ void load8(Raw<T>& r, const T* p, int n) {
  r.zero();
  if constexpr (kVec) {
    if (n > 0) r.load(p);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) r.set(i, p[i]);
  }
}

// log(1 + exp(v)) = max(v, 0) + log(1 + e), e = exp(-|v|), and with s = e / (2 + e) <= 1/3
// log(1 + e) = 2 atanh(s) = 2 (s + s^3/3 + s^5/5 + ...): no digits are lost for small e, as they
// are in log(1 + e) itself.  Seven terms leave 2 s^15/15 < 2^-26 s.
__device__ __forceinline__ float softplus_exact(float v) {
  const float e = expf(-fabsf(v));
  const float s = __fdividef(e, 2.f + e);
  const float q = s * s;
  float r = fmaf(q, 1.f / 13.f, 1.f / 11.f);
  r = fmaf(q, r, 1.f / 9.f);
  r = fmaf(q, r, 1.f / 7.f);
  r = fmaf(q, r, 1.f / 5.f);
  r = fmaf(q, r, 1.f / 3.f);
  r = fmaf(q * s, r, s);
  return fmaxf(v, 0.f) + 2.f * r;
}

__device__ __forceinline__ float exp2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Two 32-bit numbers in one 64-bit register, for the packed multiply-adds.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// kState: only the segment's state from zero and its sum of steps (the first of two launches).
template <typename T, int NS, bool kVec, bool kState>
__global__ void __launch_bounds__(kThreads) scan_kernel(ScanParams p) {
  constexpr int kN = kLanes * NS;  // states, padded
  constexpr int kBC = kTile * kN / 8;             // vectors of eight in a tile of B (or C)
  constexpr int kBCEach = (2 * kBC + kThreads - 1) / kThreads;
  __shared__ __align__(16) float2 s_step[kTile][kChannels];  // (d, d u)
  __shared__ __align__(16) float s_B[kTile][kN], s_C[kTile][kN];
  __shared__ __align__(16) float s_y[kTile][kYRow];

  const int group = blockIdx.x / p.tiles;
  const int in_group = (blockIdx.x % p.tiles) * kChannels;
  const int c0 = group * p.per + in_group;
  const int nc = p.per - in_group < kChannels ? p.per - in_group : kChannels;
  const int64_t b = blockIdx.z;
  const int seg = blockIdx.y;
  int64_t len = p.L;
  if (p.lengths) len = p.lengths[b] < 0 ? 0 : p.lengths[b] < p.L ? p.lengths[b] : p.L;
  const int64_t begin = seg * p.segment;
  const int64_t stop = seg + 1 < p.segments && begin + p.segment < p.L ? begin + p.segment : p.L;  // of the outputs
  const int64_t end = len < stop ? len : stop;                                 // of the recurrence

  const int tid = threadIdx.x;
  const int row = tid / 4, col = (tid % 4) * 8;  // loads and stores: a token, eight channels
  const int valid = nc - col;
  const int ch = tid / kLanes, part = tid % kLanes;  // recurrence: a channel, a quarter of its states
  const bool live = ch < nc;

  const T* u = static_cast<const T*>(p.u) + b * p.ub + c0 + col;
  const T* delta = static_cast<const T*>(p.delta) + b * p.db + c0 + col;
  const T* z = static_cast<const T*>(p.z) + b * p.zb + c0 + col;
  const T* Bm = static_cast<const T*>(p.Bm) + b * p.Bb + static_cast<int64_t>(group) * p.N;
  const T* Cm = static_cast<const T*>(p.Cm) + b * p.Cb + static_cast<int64_t>(group) * p.N;

  Raw<T> ru, rd, rz, rbc[kBCEach];
  auto fetch = [&](int64_t t0) {
    const int64_t t = t0 + row;
    const int n = t < end ? valid : 0;
    load8<T, kVec>(ru, u + t * p.ut, n);
    load8<T, kVec>(rd, delta + t * p.dt, n);
    if constexpr (!kState) {
      if (p.z) load8<T, kVec>(rz, z + t * p.zt, n);
    }
#pragma unroll
    for (int i = 0; i < kBCEach; ++i) {
      const int v = tid + i * kThreads;
      const bool is_c = v >= kBC;
      const int at = is_c ? v - kBC : v;
      const int64_t tt = t0 + at / (kN / 8);
      const int n0 = at % (kN / 8) * 8;
      if (v < (kState ? kBC : 2 * kBC))
        load8<T, kVec>(rbc[i], (is_c ? Cm + tt * p.Ct : Bm + tt * p.Bt) + n0, tt < end ? p.N - n0 : 0);
    }
  };
  fetch(begin);

  uint64_t a2[NS / 2], h2[NS / 2];
  const int64_t state_row = (b * p.D + c0 + ch) * p.N;
  const int n0 = part * NS;
#pragma unroll
  for (int i = 0; i < NS / 2; ++i) {
    float a[2], h[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int n = n0 + 2 * i + e;
      const bool in = live && n < p.N;
      a[e] = in ? p.A[static_cast<int64_t>(c0 + ch) * p.N + n] * kLog2e : 0.f;
      h[e] = in && p.init && p.segments == 1 ? p.init[state_row + n] : 0.f;
      // final_state may be init_state, and the last segment's block may end before another reads
      // its state: in segments all read a copy
      if (kState && seg == 0 && in)
        p.seg_state[((b * p.segments) * p.D + c0 + ch) * p.N + n] = p.init ? p.init[state_row + n] : 0.f;
    }
    a2[i] = pack2(a[0], a[1]);
    h2[i] = pack2(h[0], h[1]);
  }
  if (!kState && p.segments > 1) {
    grid_dep_wait();
#pragma unroll 4
    for (int j = 0; j <= seg; ++j) {  // the state entering this segment
      const int64_t at = (b * p.segments + j) * p.D + c0 + ch;
      const float sum = live && j > 0 ? p.seg_sum[at - p.D] : 0.f;
      const uint64_t sum2 = pack2(sum, sum);
#pragma unroll
      for (int i = 0; i < NS / 2; ++i) {
        const int n = n0 + 2 * i;
        const float lo = live && n < p.N ? p.seg_state[at * p.N + n] : 0.f;
        const float hi = live && n + 1 < p.N ? p.seg_state[at * p.N + n + 1] : 0.f;
        float x, y;
        unpack2(mul2(sum2, a2[i]), x, y);
        h2[i] = fma2(pack2(exp2_fast(x), exp2_fast(y)), h2[i], pack2(lo, hi));
      }
    }
  }
  float bias[8], skip[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    bias[i] = p.delta_bias && i < valid ? p.delta_bias[c0 + col + i] : 0.f;
    skip[i] = !kState && p.skip && i < valid ? p.skip[c0 + col + i] : 0.f;
  }

  float total = 0.f;
  for (int64_t t0 = begin; t0 < end; t0 += kTile) {
    // the tile's steps and rows of B and C
    const bool there = t0 + row < end;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float d = rd.get(i) + bias[i];
      if (p.softplus) d = softplus_exact(d);
      if (!there) d = 0.f;  // past the end the state stays
      s_step[row][col + i] = make_float2(d, d * ru.get(i));
    }
#pragma unroll
    for (int i = 0; i < kBCEach; ++i) {
      const int v = tid + i * kThreads;
      const bool is_c = v >= kBC;
      const int at = is_c ? v - kBC : v;
      if (v < (kState ? kBC : 2 * kBC)) {
        float* dst = (is_c ? s_C : s_B)[at / (kN / 8)] + at % (kN / 8) * 8;
#pragma unroll
        for (int e = 0; e < 8; e += 4)
          *reinterpret_cast<float4*>(dst + e) =
              make_float4(rbc[i].get(e), rbc[i].get(e + 1), rbc[i].get(e + 2), rbc[i].get(e + 3));
      }
    }
    const Raw<T> cu = ru, cz = rz;
    __syncthreads();
    if (t0 + kTile < end) fetch(t0 + kTile);

    const int nt = end - t0 < kTile ? static_cast<int>(end - t0) : kTile;
    for (int t = 0; t < nt; t += 4) {
      float acc[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 st = s_step[t + k][ch];
        const uint64_t d2 = pack2(st.x, st.x), du2 = pack2(st.y, st.y);
        if (kState) total += st.x;
        uint64_t sum2 = 0;
        const uint64_t* B2 = reinterpret_cast<const uint64_t*>(&s_B[t + k][n0]);
        const uint64_t* C2 = reinterpret_cast<const uint64_t*>(&s_C[t + k][n0]);
#pragma unroll
        for (int i = 0; i < NS / 2; ++i) {
          float x, y;
          unpack2(mul2(d2, a2[i]), x, y);
          h2[i] = fma2(pack2(exp2_fast(x), exp2_fast(y)), h2[i], mul2(du2, B2[i]));
          if constexpr (!kState) sum2 = fma2(h2[i], C2[i], sum2);
        }
        if constexpr (!kState) {
          float lo, hi;
          unpack2(sum2, lo, hi);
          acc[k] = lo + hi;
        }
      }
      if constexpr (!kState) {
        // lanes with bit 0 keep tokens 1 and 3, then those with bit 1 the later of the two left
        const bool b0 = part & 1, b1 = part & 2;
        float k0 = b0 ? acc[1] : acc[0], k1 = b0 ? acc[3] : acc[2];
        k0 += __shfl_xor_sync(0xffffffffu, b0 ? acc[0] : acc[1], 1);
        k1 += __shfl_xor_sync(0xffffffffu, b0 ? acc[2] : acc[3], 1);
        const float sum = (b1 ? k1 : k0) + __shfl_xor_sync(0xffffffffu, b1 ? k0 : k1, 2);
        s_y[t + (part & 1) + (part & 2)][ch] = sum;
      }
    }
    __syncthreads();
    if constexpr (!kState) {
      if (there && valid > 0) {
        T* y = static_cast<T*>(p.y) + (b * p.L + t0 + row) * p.D + c0 + col;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = fmaf(skip[i], cu.get(i), s_y[row][col + i]);
          if (p.z) v[i] *= silu(cz.get(i));
        }
        if constexpr (kVec) {
          Raw<T> out;
#pragma unroll
          for (int i = 0; i < 8; ++i) out.set(i, from_f32<T>(v[i]));
          if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<uint4*>(y) = out.v;
          } else {
            reinterpret_cast<float4*>(y)[0] = out.a;
            reinterpret_cast<float4*>(y)[1] = out.b;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i < valid) y[i] = from_f32<T>(v[i]);
        }
      }
    }
  }
  if constexpr (kState) {
    grid_dep_launch();
    const int64_t at = (b * p.segments + seg + 1) * p.D + c0 + ch;
    if (live) {
      if (part == 0) p.seg_sum[at - p.D] = total;
#pragma unroll
      for (int i = 0; i < NS / 2; ++i) {
        float lo, hi;
        unpack2(h2[i], lo, hi);
        if (n0 + 2 * i < p.N) p.seg_state[at * p.N + n0 + 2 * i] = lo;
        if (n0 + 2 * i + 1 < p.N) p.seg_state[at * p.N + n0 + 2 * i + 1] = hi;
      }
    }
  } else {
    for (int64_t t = (end > begin ? end : begin) + row; t < stop; t += kThreads / 4) {  // after the sequence's end
      T* y = static_cast<T*>(p.y) + (b * p.L + t) * p.D + c0 + col;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < valid) y[i] = from_f32<T>(0.f);
    }
    if (p.final_state && seg + 1 == p.segments && live) {
#pragma unroll
      for (int i = 0; i < NS / 2; ++i) {
        float lo, hi;
        unpack2(h2[i], lo, hi);
        if (n0 + 2 * i < p.N) p.final_state[state_row + n0 + 2 * i] = lo;
        if (n0 + 2 * i + 1 < p.N) p.final_state[state_row + n0 + 2 * i + 1] = hi;
      }
    }
  }
}

// Segments a sequence is cut into: enough blocks for `kFill` on every multiprocessor, but no
// segment below kLeast tokens.
constexpr int64_t kFill = 6, kLeast = 128;

int segment_count(int64_t batch, int64_t L, int blocks) {
  const int64_t all = batch * blocks;
  const int64_t want = kFill * layer_sm_count();
  if (2 * all > want) return 1;
  int64_t s = want / all;
  const int64_t most = L / kLeast;
  if (s > most) s = most;
  return s < 3 ? 1 : static_cast<int>(s);  // two segments pay for one in the first launch and gain nothing
}

template <typename T, int NS, bool kVec>
cudaError_t launch_ns(const ScanParams& p, int64_t batch, cudaStream_t stream) {
  const unsigned blocks = static_cast<unsigned>(p.G * p.tiles);
  if (p.segments > 1) {
    const cudaError_t e = launch_k(scan_kernel<T, NS, kVec, true>,
                                   dim3(blocks, static_cast<unsigned>(p.segments - 1), static_cast<unsigned>(batch)),
                                   dim3(kThreads), 0, stream, false, p);
    if (e != cudaSuccess) return e;
  }
  return launch_k(scan_kernel<T, NS, kVec, false>,
                  dim3(blocks, static_cast<unsigned>(p.segments), static_cast<unsigned>(batch)), dim3(kThreads), 0,
                  stream, p.segments > 1, p);
}

template <typename T, bool kVec>
cudaError_t launch_vec(const ScanParams& p, int64_t batch, cudaStream_t stream) {
  if (p.N <= 8) return launch_ns<T, 2, kVec>(p, batch, stream);
  if (p.N <= 16) return launch_ns<T, 4, kVec>(p, batch, stream);
  if (p.N <= 32) return launch_ns<T, 8, kVec>(p, batch, stream);
  return launch_ns<T, 16, kVec>(p, batch, stream);
}

template <typename T>
cudaError_t launch(const ScanParams& p, int64_t batch, cudaStream_t stream) {
  // 16-byte loads where every row of eight channels (of eight states) starts on 16 bytes and is whole
  const int64_t es = sizeof(T);
  auto row16 = [&](const void* t, int64_t s0, int64_t s1) {
    return aligned_to(t, 16) && (batch == 1 || s0 * es % 16 == 0) && (p.L <= 1 || s1 * es % 16 == 0);
  };
  const bool vec = p.per % 8 == 0 && p.N % 8 == 0 && row16(p.u, p.ub, p.ut) && row16(p.delta, p.db, p.dt) &&
                   row16(p.z, p.zb, p.zt) && row16(p.Bm, p.Bb, p.Bt) && row16(p.Cm, p.Cb, p.Ct) && aligned_to(p.y, 16);
  return vec ? launch_vec<T, true>(p, batch, stream) : launch_vec<T, false>(p, batch, stream);
}

ssd_status check_sizes(const ssd_selective_scan_args* a) {
  if (!a || a->size != static_cast<int64_t>(sizeof(*a))) return SSD_ERR_INVALID_ARG;
  if (a->batch < 0 || a->seqlen < 0 || a->channels <= 0 || a->dstate <= 0 || a->ngroups <= 0) return SSD_ERR_INVALID_ARG;
  if (a->dstate > 64 || a->channels % a->ngroups != 0 || a->batch > 65535) return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

int blocks_of(const ssd_selective_scan_args* a) {
  return a->ngroups * static_cast<int>(ceil_div(a->channels / a->ngroups, kChannels));
}

}  // namespace
}  // namespace ssd

extern "C" size_t ssd_selective_scan_workspace_size(const ssd_selective_scan_args* a) {
  using namespace ssd;
  if (check_sizes(a) != SSD_OK || a->batch == 0) return 0;
  const int s = segment_count(a->batch, a->seqlen, blocks_of(a));
  return s == 1 ? 0 : static_cast<size_t>(s) * a->batch * a->channels * (a->dstate + 1) * sizeof(float);
}

extern "C" ssd_status ssd_selective_scan(const ssd_selective_scan_args* a, ssd_stream_t stream) {
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
  p.segments = segment_count(a->batch, a->seqlen, blocks_of(a));
  if (p.segments > 1) {
    if (!a->workspace || !aligned_to(a->workspace, 16)) return SSD_ERR_INVALID_ARG;
    if (a->workspace_bytes < ssd_selective_scan_workspace_size(a)) return SSD_ERR_WORKSPACE;
  }
  p.segment = ceil_div(ceil_div(a->seqlen, p.segments), kTile) * kTile;
  p.seg_state = static_cast<float*>(a->workspace);
  if (p.segments > 1) p.seg_sum = p.seg_state + static_cast<int64_t>(p.segments) * a->batch * a->channels * a->dstate;
  p.L = a->seqlen;
  p.D = a->channels;
  p.N = a->dstate;
  p.G = a->ngroups;
  p.per = a->channels / a->ngroups;
  p.tiles = static_cast<int>(ceil_div(p.per, kChannels));
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
