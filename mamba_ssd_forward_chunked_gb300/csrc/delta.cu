// The gated delta rule, token by token:
//   h' = exp(dt A) h,   h = h' + beta (x - h' k) k^T,   y = scale h q
// with k and q the group's rows of Bm and Cm.
//
// Every row of a head's state is a recurrence of its own.  N/16 lanes share a
// row, 16 values each in registers, and a lane has R rows; the sums over a row
// are joined by shuffles.  Tokens are laid out in shared memory, a tile at a
// time: k and q with their norms, x, the gates.
//
// The state's bytes bound it: it is read and written once, 64 KB of a head of 128 x 128 for each token or handful
// of tokens.  256 single tokens of 32 heads 170 us, 94 % of a copy's rate; 32 times 5 drafted tokens 28 us (floor
// 20: a block loads, computes and stores one after the other); one token 4.1 us, a launch's latency.  16 values a
// lane, so that a row's sum takes two or three shuffles; four rows a lane share them (join_rows), two where there
// are too few blocks.
#include "delta.cuh"
#include "delta_chunk.cuh"

namespace ssd {
namespace {

constexpr int kTokens = 16;  // of a tile

// Sums s[0..R) over kLanes neighbouring lanes, joined together: over the first lane bits a lane keeps
// half of the sums it holds.  Returns the sum that the lane ends with, of row held_row().
template <int R, int kLanes>
__device__ __forceinline__ float join_rows(float (&s)[R], int lane) {
  int bit = 1;
#pragma unroll
  for (int n = R; n > 1; n /= 2, bit *= 2) {
    const bool upper = lane & bit;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float give = upper ? s[i] : s[i + n / 2];
      s[i] = (upper ? s[i + n / 2] : s[i]) + __shfl_xor_sync(0xffffffffu, give, bit);
    }
  }
#pragma unroll
  for (; bit < kLanes; bit *= 2) s[0] += __shfl_xor_sync(0xffffffffu, s[0], bit);
  return s[0];
}
template <int R>
__device__ __forceinline__ int held_row(int lane) {
  return R == 4 ? (lane & 1) * 2 + (lane >> 1 & 1) : R == 2 ? lane & 1 : 0;
}
// The lane (of its row's lanes) that ends with row i.
template <int R>
__device__ __forceinline__ constexpr int lane_of_row(int i) {
  return R == 4 ? (i >> 1) | (i & 1) << 1 : i;
}

// For a row whose squares may not have stayed in 32 bits: a power of two, and the factor of the row times that (1 and
// what it was given where the row is 0 or not finite).  A call of its own, so that it costs the others nothing.
template <typename T, int N>
__device__ __noinline__ float2 norm_by_power(float eps, const T* row, float factor) {
  const int lane = threadIdx.x & 31;
  float largest = 0.f, squares = 0.f;
  for (int i = lane; i < N; i += 32) largest = fmaxf(largest, fabsf(to_f32(row[i])));
  largest = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(largest)));
  if (!(largest > 0.f && largest < INFINITY)) return make_float2(1.f, factor);
  const float up = exp2f(static_cast<float>(-max(ilogbf(largest), -126)));
  for (int i = lane; i < N; i += 32) {
    const float v = to_f32(row[i]) * up;
    squares = fmaf(v, v, squares);
  }
  for (int o = 16; o; o /= 2) squares += __shfl_xor_sync(0xffffffffu, squares, o);
  const float e = eps * up * up;
  return make_float2(up, e < 0x1p80f ? 1.f / sqrtf(squares + e) : 1.f / (sqrtf(eps) * up));
}

template <typename T, int N, int R, int kWarps>
__global__ void __launch_bounds__(32 * kWarps) delta_scan_kernel(DeltaParams p, int tiles) {
  constexpr int kLanes = N / 16;
  constexpr int kPer = 32 / kLanes;              // rows of a warp in one pass
  constexpr int kRows = kWarps * kPer * R;       // of a block
  __shared__ __align__(16) float s_k[kTokens][N], s_q[kTokens][N];
  __shared__ float s_x[kTokens][kRows], s_decay[kTokens], s_beta[kTokens];
  begin_kernel();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x / tiles, row0 = blockIdx.x % tiles * kRows;
  const int64_t b = blockIdx.y;
  const int g = h / (p.H / p.G);
  const DeltaSeq seq = delta_sequence(p, b);
  T* y = static_cast<T*>(p.y) + (b * p.seqlen * p.H + h) * p.P;
  const int64_t y_token = static_cast<int64_t>(p.H) * p.P;
  const int in = lane % kLanes;                                    // the lane's place in its row
  const int local0 = warp * kPer * R + lane / kLanes;              // its first row, of the block
  const int64_t head = (seq.row * p.H + h) * p.P;

  // the states: pairs of values n, n + 1 of each row
  uint64_t S[R][8];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int row = row0 + local0 + i * kPer;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (seq.row >= 0 && seq.resumed && row < p.P) v = load_once(p.init_state + (head + row) * N + 4 * (in + kLanes * j));
      S[i][2 * j] = pack2(v.x, v.y), S[i][2 * j + 1] = pack2(v.z, v.w);
    }
  }
  const int length = seq.row < 0 ? 0 : seq.length;
  const T* x = static_cast<const T*>(p.x) + b * p.x_batch + static_cast<int64_t>(h) * p.P + row0;
  const T* Bm = static_cast<const T*>(p.Bm) + b * p.B_batch + static_cast<int64_t>(g) * N;
  const T* Cm = static_cast<const T*>(p.Cm) + b * p.C_batch + static_cast<int64_t>(g) * N;
  const int left = p.P - row0 < kRows ? p.P - row0 : kRows;

  for (int t0 = 0; t0 < length; t0 += kTokens) {
    const int n = length - t0 < kTokens ? length - t0 : kTokens;
    __syncthreads();
    for (int j = warp; j < 2 * n; j += kWarps) {  // a warp lays out a row of k or q
      const int64_t t = t0 + (j >> 1);
      const T* from = j & 1 ? Cm + t * p.C_token : Bm + t * p.B_token;
      float v[N / 32], squares = 0.f;
#pragma unroll
      for (int i = 0; i < N / 32; ++i) v[i] = to_f32(from[lane + 32 * i]), squares = fmaf(v[i], v[i], squares);
#pragma unroll
      for (int o = 16; o; o /= 2) squares += __shfl_xor_sync(0xffffffffu, squares, o);
      float f = delta_norm(p, squares);
      if (p.norm_eps >= 0.f && !(squares > 0x1p-80f && squares < 0x1p120f)) {  // squares that 32 bits may not have held
        const float2 scaled = norm_by_power<T, N>(p.norm_eps, from, f);
        f = scaled.y;
#pragma unroll
        for (int i = 0; i < N / 32; ++i) v[i] *= scaled.x;
      }
      f *= j & 1 ? p.scale : 1.f;
      float* to = j & 1 ? s_q[j >> 1] : s_k[j >> 1];
#pragma unroll
      for (int i = 0; i < N / 32; ++i) to[lane + 32 * i] = v[i] * f;
    }
    for (int i = tid; i < n * left; i += 32 * kWarps) {
      const int t = i / left;
      s_x[t][i - t * left] = to_f32(x[(t0 + t) * p.x_token + (i - t * left)]);
    }
    if (tid < n) s_decay[tid] = expf(delta_log_decay<T>(p, b, t0 + tid, h)), s_beta[tid] = delta_beta<T>(p, b, t0 + tid, h);
    __syncthreads();

    for (int t = 0; t < n; ++t) {
      uint64_t k[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 v = *reinterpret_cast<const float4*>(&s_k[t][4 * (in + kLanes * j)]);
        k[2 * j] = pack2(v.x, v.y), k[2 * j + 1] = pack2(v.z, v.w);
      }
      const float decay = s_decay[t];
      float sum[R];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        uint64_t a = mul2(S[i][0], k[0]), c = mul2(S[i][1], k[1]);
#pragma unroll
        for (int j = 2; j < 8; j += 2) a = fma2(S[i][j], k[j], a), c = fma2(S[i][j + 1], k[j + 1], c);
        float lo, hi;
        unpack2(add2(a, c), lo, hi);
        sum[i] = lo + hi;
      }
      const float dot = join_rows<R, kLanes>(sum, in);
      const float u = s_beta[t] * fmaf(-decay, dot, s_x[t][local0 + held_row<R>(in) * kPer]);
      const uint64_t decay2 = pack2(decay, decay);
      uint64_t q[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 v = *reinterpret_cast<const float4*>(&s_q[t][4 * (in + kLanes * j)]);
        q[2 * j] = pack2(v.x, v.y), q[2 * j + 1] = pack2(v.z, v.w);
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float w = __shfl_sync(0xffffffffu, u, (lane - in) + lane_of_row<R>(i));
        const uint64_t w2 = pack2(w, w);
        uint64_t a = 0, c = 0;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          S[i][j] = fma2(w2, k[j], mul2(decay2, S[i][j]));
          S[i][j + 1] = fma2(w2, k[j + 1], mul2(decay2, S[i][j + 1]));
          a = j ? fma2(S[i][j], q[j], a) : mul2(S[i][j], q[j]);
          c = j ? fma2(S[i][j + 1], q[j + 1], c) : mul2(S[i][j + 1], q[j + 1]);
        }
        float lo, hi;
        unpack2(add2(a, c), lo, hi);
        sum[i] = lo + hi;
      }
      const float out = join_rows<R, kLanes>(sum, in);
      const int row = row0 + local0 + held_row<R>(in) * kPer;
      if (in < R && row < p.P) y[(t0 + t) * y_token + row] = from_f32<T>(out);
    }
  }

  for (int64_t i = tid; i < (p.seqlen - length) * left; i += 32 * kWarps)
    y[(length + i / left) * y_token + row0 + i % left] = from_f32<T>(0.f);
  if (!p.final_state || seq.row < 0) return;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int row = row0 + local0 + i * kPer;
    if (row >= p.P) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float4 v;
      unpack2(S[i][2 * j], v.x, v.y), unpack2(S[i][2 * j + 1], v.z, v.w);
      __stcs(reinterpret_cast<float4*>(p.final_state + (head + row) * N + 4 * (in + kLanes * j)), v);
    }
  }
}

template <typename T, int N, int R, int kWarps>
cudaError_t launch_scan(const DeltaParams& p, cudaStream_t stream) {
  const int tiles = static_cast<int>(ceil_div(p.P, kWarps * (512 / N) * R));
  return launch_k(delta_scan_kernel<T, N, R, kWarps>, dim3(static_cast<unsigned>(p.H * tiles), static_cast<unsigned>(p.batch)),
                  dim3(32 * kWarps), 0, stream, true, p, tiles);
}

template <typename T, int N>
cudaError_t launch_rows(const DeltaParams& p, cudaStream_t stream) {
  // rows a lane: four, whose sums are joined together, or two while four leave multiprocessors without a block
  // (31 tokens of 16 heads 18.5 us with two, 21.4 with four, one and more warps 16.7; single tokens 5 us with any)
  const bool few = p.batch * p.H * ceil_div(p.P, 4 * 2048 / N) < 2 * static_cast<int64_t>(layer_sm_count());
  return few ? launch_scan<T, N, 2, 4>(p, stream) : launch_scan<T, N, 4, 4>(p, stream);
}

template <typename T>
cudaError_t launch_delta(const DeltaParams& p, cudaStream_t stream) {
  return p.N == 64 ? launch_rows<T, 64>(p, stream) : p.N == 128 ? launch_rows<T, 128>(p, stream) : launch_rows<T, 256>(p, stream);
}

ssd_status check_delta(const ssd_delta_args* a) {
  if (!a || a->size != static_cast<int64_t>(sizeof(*a))) return SSD_ERR_INVALID_ARG;
  if (a->batch < 0 || a->seqlen < 0 || a->nslots < 0 || a->nheads <= 0 || a->headdim <= 0 || a->ngroups <= 0 || a->dstate <= 0)
    return SSD_ERR_INVALID_ARG;
  if (!known_dtype(a->dtype) || (a->gate_dtype != a->dtype && a->gate_dtype != SSD_F32)) return SSD_ERR_UNSUPPORTED;
  if (a->headdim % 16 != 0 || a->headdim > 1024 || (a->dstate != 64 && a->dstate != 128 && a->dstate != 256)) return SSD_ERR_UNSUPPORTED;
  if (a->nheads % a->ngroups != 0 || a->nheads > 65535 || a->batch > 65535 || a->seqlen > int64_t(1) << 30) return SSD_ERR_UNSUPPORTED;
  // (written so that NaN is refused)
  if (!(a->scale >= -3.4e38f && a->scale <= 3.4e38f) || !(a->norm_eps >= -3.4e38f && a->norm_eps <= 3.4e38f)) return SSD_ERR_INVALID_ARG;
  return SSD_OK;
}

DeltaParams params_of(const ssd_delta_args* a) {
  DeltaParams p{};
  p.batch = a->batch, p.seqlen = a->seqlen, p.nslots = a->nslots;
  p.x_batch = a->x_batch, p.x_token = a->x_token;
  p.B_batch = a->B_batch, p.B_token = a->B_token, p.C_batch = a->C_batch, p.C_token = a->C_token;
  p.dt_batch = a->dt_batch, p.dt_token = a->dt_token, p.beta_batch = a->beta_batch, p.beta_token = a->beta_token;
  p.H = a->nheads, p.G = a->ngroups, p.P = a->headdim, p.N = a->dstate;
  p.parts = a->dtype == SSD_BF16 ? 1 : 2;
  p.gate_f32 = a->gate_dtype == SSD_F32, p.softplus = a->dt_softplus != 0, p.sigmoid = a->beta_sigmoid != 0;
  p.scale = a->scale, p.norm_eps = a->norm_eps;
  p.x = a->x, p.Bm = a->Bm, p.Cm = a->Cm, p.dt = a->dt, p.beta = a->beta;
  p.A = a->A, p.dt_bias = a->dt_bias;
  p.init_state = a->init_state, p.final_state = a->final_state;
  p.slots = a->slots, p.positions = a->positions, p.lengths = a->lengths;
  p.y = a->y;
  return p;
}

}  // namespace
}  // namespace ssd

extern "C" size_t ssd_delta_workspace_size(const ssd_delta_args* a) {
  using namespace ssd;
  if (check_delta(a) != SSD_OK || a->batch == 0 || !delta_chunked(a->dtype, a->seqlen, a->dstate)) return 0;
  return delta_chunks_workspace(params_of(a));
}

extern "C" ssd_status ssd_delta_fwd(const ssd_delta_args* a, ssd_stream_t stream) {
  using namespace ssd;
  const ssd_status st = check_delta(a);
  if (st != SSD_OK) return st;
  if (a->batch == 0) return SSD_OK;
  const size_t es = elem_size(a->dtype), gs = elem_size(a->gate_dtype);
  if (a->seqlen > 0) {
    for (const void* t : {a->x, a->Bm, a->Cm, (const void*)a->y})
      if (!t || !aligned_to(t, es)) return SSD_ERR_INVALID_ARG;
    for (const void* t : {a->dt, a->beta})
      if (!t || !aligned_to(t, gs)) return SSD_ERR_INVALID_ARG;
    if (!a->A) return SSD_ERR_INVALID_ARG;
  }
  for (const void* t : {(const void*)a->A, (const void*)a->dt_bias, (const void*)a->slots, (const void*)a->positions, (const void*)a->lengths})
    if (!aligned_to(t, 4)) return SSD_ERR_INVALID_ARG;
  if (!aligned_to(a->init_state, 16) || !aligned_to(a->final_state, 16)) return SSD_ERR_INVALID_ARG;
  if (!a->slots && a->nslots < a->batch) return SSD_ERR_INVALID_ARG;
  const DeltaParams p = params_of(a);
  if (const size_t need = ssd_delta_workspace_size(a)) {
    if (!a->workspace || !aligned_to(a->workspace, 16)) return SSD_ERR_INVALID_ARG;
    if (a->workspace_bytes < need) return SSD_ERR_WORKSPACE;
    return launch_delta_chunks(p, a->workspace, stream);
  }
  return launched(a->dtype == SSD_BF16 ? launch_delta<__nv_bfloat16>(p, stream) : launch_delta<float>(p, stream));
}
