// One token of a Mamba-2 layer for a batch of sequences: the convolution of
// the token's x, B, C channels with its ring, then per head
//   h = exp(d A) h + d x b^T,   y = (h c + D x) silu(z).
//
// Every state is read and written once, so HBM bounds it (one sequence: the
// latency of one launch).  A block takes a head of a sequence, or a quarter of
// its rows where there are few heads in the batch.  The convolution's inputs and
// then the block's states (16 bytes a load, up to 16 loads a thread) are all on
// their way before it forms the head's x and its group's B and C by itself, so
// that the whole layer step is one launch: B and C are formed again by every
// head of a group, a few hundred multiplications against the head's 2 x 32 KB of
// state.  The ring has one slot more than the taps reach back, so the slot that
// takes the new token is read by nobody in this launch, and B's and C's are
// written by one block of the group alone.  80 heads of 64 x 128 states: 256
// sequences 202 us, 6.7 TB/s (states asked for before the convolution's inputs:
// 292 us); one sequence 3.3 us.
#include "layer.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 256;
constexpr int kP = 64;  // headdim

struct StepParams {
  int64_t nslots, u_batch, z_batch, dt_batch;
  int H, G, N, W, dt_f32, softplus, weight16;
  const void *u, *z, *dt;
  const float *weight, *bias, *A, *D, *dt_bias;
  void* ring;
  const float* state;
  float* new_state;
  const int32_t *positions, *slots;
  void* y;
};

// kRows: rows of the head's 64 that a block takes.
template <typename T, int N, int kRows, int W>
__global__ void __launch_bounds__(kThreads) step_kernel(StepParams p) {
  constexpr int kLanes = N >= 128 ? 32 : 16;           // lanes that share a row
  constexpr int kVecs = N / (4 * kLanes);              // float4 a lane has of a row
  constexpr int kPerPass = kThreads / kLanes;          // rows the block takes in one pass
  constexpr int kPasses = kRows / kPerPass;
  constexpr int kChannels = kRows + 2 * N;             // x, B, C channels the block forms
  constexpr int kEach = (kChannels + kThreads - 1) / kThreads;
  __shared__ __align__(16) float s_x[kRows], s_B[N], s_C[N];
  __shared__ float s_y[kRows];
  begin_kernel();
  const int row0 = blockIdx.x % (kP / kRows) * kRows;
  const int h = blockIdx.x / (kP / kRows);
  const int64_t b = blockIdx.y;
  const int g = h / (p.H / p.G);
  const bool writes_group = h % (p.H / p.G) == 0 && row0 == 0;  // keeps the group's B and C in the ring
  const int64_t slot = p.slots ? p.slots[b] : b;
  const int position = p.positions[b];
  const int tid = threadIdx.x;
  T* y = static_cast<T*>(p.y) + (b * p.H + h) * kP + row0;
  if (slot < 0 || slot >= p.nslots) {
    if (tid < kRows) y[tid] = from_f32<T>(0.f);
    return;
  }

  // the convolution's inputs
  const int pos = position > 0 ? position : 0;
  const int newest = pos % W;
  const int inner = p.H * kP;
  const int C = inner + 2 * p.G * N;
  const T* u = static_cast<const T*>(p.u) + b * p.u_batch;
  T* ring = static_cast<T*>(p.ring) + slot * W * C;
  T now[kEach], past[kEach][W - 1];
  float w[kEach][W], acc[kEach];
  int chan[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = tid + e * kThreads;
    if (i >= kChannels) break;
    const int c = i < kRows ? h * kP + row0 + i
                            : inner + (i < kRows + N ? g * N + (i - kRows) : (p.G + g) * N + (i - kRows - N));
    chan[e] = c;
    now[e] = u[c];
#pragma unroll
    for (int j = 1; j < W; ++j)  // the token j before this one; before the first there is none
      if (j <= pos) past[e][j - 1] = ring[(newest >= j ? newest - j : newest - j + W) * C + c];
    const float* taps = p.weight + static_cast<int64_t>(c) * W;
    if (W == 4 && p.weight16) {
      const float4 f = *reinterpret_cast<const float4*>(taps);
      w[e][0] = f.x, w[e][1] = f.y, w[e][W - 2] = f.z, w[e][W - 1] = f.w;
    } else {
#pragma unroll
      for (int j = 0; j < W; ++j) w[e][j] = taps[j];
    }
    acc[e] = p.bias ? p.bias[c] : 0.f;
  }
  float d = p.dt_f32 ? static_cast<const float*>(p.dt)[b * p.dt_batch + h]
                     : to_f32(static_cast<const T*>(p.dt)[b * p.dt_batch + h]);
  if (p.dt_bias) d += p.dt_bias[h];
  const float rate = p.A[h], skip = p.D[h];
  float z = 0.f;
  if (p.z && tid < kRows) z = to_f32(static_cast<const T*>(p.z)[b * p.z_batch + h * kP + row0 + tid]);

  // the states
  const int lane = tid % kLanes, row_in = tid / kLanes;
  const int64_t base = ((slot * p.H + h) * kP + row0 + row_in) * N + 4 * lane;
  const float* from = p.state + base;
  float4 st[kPasses][kVecs];
#pragma unroll
  for (int i = 0; i < kPasses; ++i)
#pragma unroll
    for (int v = 0; v < kVecs; ++v)
      st[i][v] = load_once(from + i * kPerPass * N + v * 4 * kLanes);

#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = tid + e * kThreads;
    if (i >= kChannels) break;
    float sum = fmaf(w[e][W - 1], to_f32(now[e]), acc[e]);
#pragma unroll
    for (int j = 1; j < W; ++j)
      if (j <= pos) sum = fmaf(w[e][W - 1 - j], to_f32(past[e][j - 1]), sum);
    if (i < kRows || writes_group) ring[newest * C + chan[e]] = now[e];
    (i < kRows ? s_x[i] : i < kRows + N ? s_B[i - kRows] : s_C[i - kRows - N]) = silu(sum);
  }
  __syncthreads();
  if (p.softplus) d = softplus(d);
  const float decay = expf(d * rate);
  float* out = (p.new_state ? p.new_state : const_cast<float*>(p.state)) + base;
  float sums[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) sums[i] = 0.f;
#pragma unroll
  for (int v = 0; v < kVecs; ++v) {
    const float4 B4 = *reinterpret_cast<const float4*>(&s_B[4 * lane + v * 4 * kLanes]);
    const float4 C4 = *reinterpret_cast<const float4*>(&s_C[4 * lane + v * 4 * kLanes]);
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const float dx = d * s_x[row_in + i * kPerPass];
      float4 s = st[i][v];
      s.x = fmaf(decay, s.x, dx * B4.x);
      s.y = fmaf(decay, s.y, dx * B4.y);
      s.z = fmaf(decay, s.z, dx * B4.z);
      s.w = fmaf(decay, s.w, dx * B4.w);
      sums[i] = fmaf(s.x, C4.x, fmaf(s.y, C4.y, fmaf(s.z, C4.z, fmaf(s.w, C4.w, sums[i]))));
      __stcs(reinterpret_cast<float4*>(out + i * kPerPass * N + v * 4 * kLanes), s);
    }
  }
  // The passes' sums are joined together: over the first lane bits a lane keeps half of the sums it
  // holds, until it holds one, and over the other bits that one is added up.
  int held = 0;  // the pass whose sum the lane ends with
  int bit = 1;
#pragma unroll
  for (int n = kPasses; n > 1; n /= 2, bit *= 2) {
    const bool upper = lane & bit;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float give = upper ? sums[i] : sums[i + n / 2];
      sums[i] = (upper ? sums[i + n / 2] : sums[i]) + __shfl_xor_sync(0xffffffffu, give, bit);
    }
    if (upper) held += n / 2;
  }
#pragma unroll
  for (; bit < kLanes; bit *= 2) sums[0] += __shfl_xor_sync(0xffffffffu, sums[0], bit);
  if (lane < kPasses) s_y[row_in + held * kPerPass] = sums[0];
  __syncthreads();
  if (tid < kRows) {
    float v = fmaf(skip, s_x[tid], s_y[tid]);
    if (p.z) v *= silu(z);
    y[tid] = from_f32<T>(v);
  }
}

template <typename T, int N, int W>
cudaError_t launch(const StepParams& p, int64_t batch, cudaStream_t stream) {
  // a head a block, or quarters of heads while those leave the GPU room
  const bool few = batch * p.H < 2 * static_cast<int64_t>(layer_sm_count());
  const dim3 grid(static_cast<unsigned>(p.H * (few ? 4 : 1)), static_cast<unsigned>(batch));
  return launch_k(few ? step_kernel<T, N, 16, W> : step_kernel<T, N, 64, W>, grid, dim3(kThreads), 0, stream, true, p);
}

template <typename T, int N>
cudaError_t launch_w(const StepParams& p, int64_t batch, cudaStream_t stream) {
  return p.W == 2 ? launch<T, N, 2>(p, batch, stream) : p.W == 3 ? launch<T, N, 3>(p, batch, stream)
                                                                 : launch<T, N, 4>(p, batch, stream);
}

template <typename T>
cudaError_t launch_n(const StepParams& p, int64_t batch, cudaStream_t stream) {
  return p.N == 64 ? launch_w<T, 64>(p, batch, stream) : p.N == 128 ? launch_w<T, 128>(p, batch, stream)
                                                                    : launch_w<T, 256>(p, batch, stream);
}

}  // namespace
}  // namespace ssd

extern "C" ssd_status ssd_step(const ssd_step_args* a, ssd_stream_t stream) {
  using namespace ssd;
  if (!a || a->size != static_cast<int64_t>(sizeof(*a))) return SSD_ERR_INVALID_ARG;
  if (a->batch < 0 || a->nslots < 0 || a->nheads <= 0 || a->headdim <= 0 || a->ngroups <= 0 || a->dstate <= 0)
    return SSD_ERR_INVALID_ARG;
  if (!known_dtype(a->dtype) || (a->dt_dtype != a->dtype && a->dt_dtype != SSD_F32)) return SSD_ERR_UNSUPPORTED;
  if (a->headdim != kP || (a->dstate != 64 && a->dstate != 128 && a->dstate != 256)) return SSD_ERR_UNSUPPORTED;
  if (a->nheads % a->ngroups != 0 || a->width < 2 || a->width > 4 || a->batch > 65535) return SSD_ERR_UNSUPPORTED;
  // offsets within a row of the ring are 32 bits
  const int64_t channels = int64_t(a->nheads) * a->headdim + 2 * int64_t(a->ngroups) * a->dstate;
  if (channels * a->width >= int64_t(1) << 31) return SSD_ERR_UNSUPPORTED;
  if (a->batch == 0) return SSD_OK;
  const size_t es = elem_size(a->dtype);
  for (const void* t : {a->u, (const void*)a->ring, (const void*)a->y})
    if (!t || !aligned_to(t, es)) return SSD_ERR_INVALID_ARG;
  if (!aligned_to(a->z, es) || !a->dt || !aligned_to(a->dt, elem_size(a->dt_dtype))) return SSD_ERR_INVALID_ARG;
  for (const void* t : {(const void*)a->weight, (const void*)a->A, (const void*)a->D, (const void*)a->positions})
    if (!t || !aligned_to(t, 4)) return SSD_ERR_INVALID_ARG;
  if (!aligned_to(a->bias, 4) || !aligned_to(a->dt_bias, 4) || !aligned_to(a->slots, 4)) return SSD_ERR_INVALID_ARG;
  if (!a->state || !aligned_to(a->state, 16) || !aligned_to(a->new_state, 16)) return SSD_ERR_INVALID_ARG;
  if (!a->slots && a->nslots < a->batch) return SSD_ERR_INVALID_ARG;
  StepParams p{};
  p.nslots = a->nslots;
  p.u_batch = a->u_batch, p.z_batch = a->z_batch, p.dt_batch = a->dt_batch;
  p.H = a->nheads, p.G = a->ngroups, p.N = a->dstate, p.W = a->width;
  p.dt_f32 = a->dt_dtype == SSD_F32, p.softplus = a->softplus != 0;
  p.u = a->u, p.z = a->z, p.dt = a->dt;
  p.weight = a->weight, p.bias = a->bias, p.A = a->A, p.D = a->D, p.dt_bias = a->dt_bias;
  p.ring = a->ring, p.state = a->state, p.new_state = a->new_state;
  p.positions = a->positions, p.slots = a->slots;
  p.y = a->y;
  p.weight16 = aligned_to(a->weight, 16);
  return launched(a->dtype == SSD_BF16 ? launch_n<__nv_bfloat16>(p, a->batch, stream)
                                       : launch_n<float>(p, a->batch, stream));
}
