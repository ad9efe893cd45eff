// One token of a Mamba-2 layer for a batch of sequences: the convolution of
// the token's x, B, C channels with its ring, then per head
//   h = exp(d A) h + d x b^T,   y = (h c + D x) silu(z).
//
// Every state is read and written once, so HBM bounds it (one sequence: the
// latency of one launch).  A block takes a head of a sequence, or a quarter of
// its rows where there are few heads in the batch.  Its states are on their way,
// 16 bytes a load and up to 16 loads a thread, before it forms the head's x and
// its group's B and C by itself, so that the whole layer step is one launch: B
// and C are formed again by every head of a group, a few hundred multiplications
// against the head's 2 x 32 KB of state.  The ring has one slot more than the
// taps reach back, so the slot that takes the new token is read by nobody in
// this launch, and B's and C's are written by one block of the group alone.
#include "layer.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 256;
constexpr int kP = 64;  // headdim

struct StepParams {
  int64_t nslots, u_batch, z_batch, dt_batch;
  int H, G, N, W, dt_f32, softplus;
  const void *u, *z, *dt;
  const float *weight, *bias, *A, *D, *dt_bias;
  void* ring;
  const float* state;
  float* new_state;
  const int32_t *positions, *slots;
  void* y;
};

// kRows: rows of the head's 64 that a block takes.
template <typename T, int N, int kRows>
__global__ void __launch_bounds__(kThreads) step_kernel(StepParams p) {
  constexpr int kLanes = N >= 128 ? 32 : 16;           // lanes that share a row
  constexpr int kVecs = N / (4 * kLanes);              // float4 a lane has of a row
  constexpr int kPerPass = kThreads / kLanes;          // rows the block takes in one pass
  constexpr int kPasses = kRows / kPerPass;
  __shared__ __align__(16) float s_x[kRows], s_B[N], s_C[N];
  __shared__ float s_y[kRows];
  const int row0 = blockIdx.x % (kP / kRows) * kRows;
  const int h = blockIdx.x / (kP / kRows);
  const int64_t b = blockIdx.y;
  const int g = h / (p.H / p.G);
  const bool writes_group = h % (p.H / p.G) == 0 && row0 == 0;  // keeps the group's B and C in the ring
  const int64_t slot = p.slots ? p.slots[b] : b;
  const int tid = threadIdx.x;
  T* y = static_cast<T*>(p.y) + (b * p.H + h) * kP + row0;
  if (slot < 0 || slot >= p.nslots) {
    if (tid < kRows) y[tid] = from_f32<T>(0.f);
    return;
  }

  const int lane = tid % kLanes, row_in = tid / kLanes;
  const int64_t base = ((slot * p.H + h) * kP + row0 + row_in) * N + 4 * lane;
  float4 st[kPasses][kVecs];
#pragma unroll
  for (int i = 0; i < kPasses; ++i)
#pragma unroll
    for (int v = 0; v < kVecs; ++v)
      st[i][v] = __ldcs(reinterpret_cast<const float4*>(p.state + base + i * kPerPass * N + v * 4 * kLanes));

  float d = p.dt_f32 ? static_cast<const float*>(p.dt)[b * p.dt_batch + h]
                     : to_f32(static_cast<const T*>(p.dt)[b * p.dt_batch + h]);
  if (p.dt_bias) d += p.dt_bias[h];
  const float rate = p.A[h], skip = p.D[h];
  float z = 0.f;
  if (p.z && tid < kRows) z = to_f32(static_cast<const T*>(p.z)[b * p.z_batch + h * kP + row0 + tid]);

  const int64_t pos = p.positions[b] > 0 ? p.positions[b] : 0;
  const int inner = p.H * kP;
  const int64_t C = inner + 2 * p.G * N;
  const T* u = static_cast<const T*>(p.u) + b * p.u_batch;
  T* ring = static_cast<T*>(p.ring) + slot * p.W * C;
  const int newest = static_cast<int>(pos % p.W);
#pragma unroll
  for (int i = tid; i < kRows + 2 * N; i += kThreads) {
    const int c = i < kRows ? h * kP + row0 + i
                            : inner + (i < kRows + N ? g * N + (i - kRows) : (p.G + g) * N + (i - kRows - N));
    const float* w = p.weight + static_cast<int64_t>(c) * p.W;
    const T now = u[c];
    float acc = p.bias ? p.bias[c] : 0.f;
    acc = fmaf(w[p.W - 1], to_f32(now), acc);
#pragma unroll
    for (int j = 1; j < 4; ++j) {  // the token j before this one
      if (j >= p.W || j > pos) break;
      const int q = newest >= j ? newest - j : newest - j + p.W;
      acc = fmaf(w[p.W - 1 - j], to_f32(ring[q * C + c]), acc);
    }
    if (i < kRows || writes_group) ring[newest * C + c] = now;
    (i < kRows ? s_x[i] : i < kRows + N ? s_B[i - kRows] : s_C[i - kRows - N]) = silu(acc);
  }
  __syncthreads();
  if (p.softplus) d = softplus(d);
  const float decay = expf(d * rate);
  float* out = (p.new_state ? p.new_state : const_cast<float*>(p.state)) + base;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const float dx = d * s_x[row_in + i * kPerPass];
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const float4 B4 = *reinterpret_cast<const float4*>(&s_B[4 * lane + v * 4 * kLanes]);
      const float4 C4 = *reinterpret_cast<const float4*>(&s_C[4 * lane + v * 4 * kLanes]);
      float4 s = st[i][v];
      s.x = fmaf(decay, s.x, dx * B4.x);
      s.y = fmaf(decay, s.y, dx * B4.y);
      s.z = fmaf(decay, s.z, dx * B4.z);
      s.w = fmaf(decay, s.w, dx * B4.w);
      sum = fmaf(s.x, C4.x, fmaf(s.y, C4.y, fmaf(s.z, C4.z, fmaf(s.w, C4.w, sum))));
      __stcs(reinterpret_cast<float4*>(out + i * kPerPass * N + v * 4 * kLanes), s);
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s_y[row_in + i * kPerPass] = sum;
  }
  __syncthreads();
  if (tid < kRows) {
    float v = fmaf(skip, s_x[tid], s_y[tid]);
    if (p.z) v *= silu(z);
    y[tid] = from_f32<T>(v);
  }
}

template <typename T, int N>
cudaError_t launch(const StepParams& p, int64_t batch, cudaStream_t stream) {
  // a head a block, or quarters of heads while those leave the GPU room
  const bool few = batch * p.H < 2 * static_cast<int64_t>(layer_sm_count());
  const dim3 grid(static_cast<unsigned>(p.H * (few ? 4 : 1)), static_cast<unsigned>(batch));
  return launch_k(few ? step_kernel<T, N, 16> : step_kernel<T, N, 64>, grid, dim3(kThreads), 0, stream, false, p);
}

template <typename T>
cudaError_t launch_n(const StepParams& p, int64_t batch, cudaStream_t stream) {
  return p.N == 64 ? launch<T, 64>(p, batch, stream) : p.N == 128 ? launch<T, 128>(p, batch, stream)
                                                                  : launch<T, 256>(p, batch, stream);
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
  return launched(a->dtype == SSD_BF16 ? launch_n<__nv_bfloat16>(p, a->batch, stream)
                                       : launch_n<float>(p, a->batch, stream));
}
