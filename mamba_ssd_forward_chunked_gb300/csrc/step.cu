// One token of a Mamba-2 layer for a batch of sequences: the convolution of
// the token's x, B, C channels with its ring, then per head
//   h = exp(d A) h + d x b^T,   y = (h c + D x) silu(z).
//
// One block per (sequence, head).  It forms the head's x and its group's B and
// C itself, so the whole layer step is one launch: B and C are formed again by
// every head of a group, a few hundred multiplications against the head's
// 2 x 32 KB of state.  The ring has one slot more than the taps reach back, so
// the slot that takes the new token is read by nobody in this launch.
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

template <typename T>
__global__ void __launch_bounds__(kThreads) step_kernel(StepParams p) {
  __shared__ float xbc[kP + 2 * 256];
  const int h = blockIdx.x;
  const int64_t b = blockIdx.y;
  const int g = h / (p.H / p.G);
  const bool writes_group = h % (p.H / p.G) == 0;  // the group's first head keeps its B and C in the ring
  const int64_t slot = p.slots ? p.slots[b] : b;
  T* y = static_cast<T*>(p.y) + (b * p.H + h) * kP;
  if (slot < 0 || slot >= p.nslots) {
    if (threadIdx.x < kP) y[threadIdx.x] = from_f32<T>(0.f);
    return;
  }
  const int64_t pos = p.positions[b] > 0 ? p.positions[b] : 0;
  const int inner = p.H * kP;
  const int64_t C = inner + 2 * p.G * p.N;
  const T* u = static_cast<const T*>(p.u) + b * p.u_batch;
  T* ring = static_cast<T*>(p.ring) + slot * p.W * C;
  for (int i = threadIdx.x; i < kP + 2 * p.N; i += kThreads) {
    const int c = i < kP ? h * kP + i
                         : inner + (i < kP + p.N ? g * p.N + (i - kP) : p.G * p.N + g * p.N + (i - kP - p.N));
    const float* w = p.weight + static_cast<int64_t>(c) * p.W;
    float acc = p.bias ? p.bias[c] : 0.f;
    for (int j = 0; j < p.W - 1; ++j) {
      const int64_t t = pos - (p.W - 1) + j;
      if (t >= 0) acc = fmaf(w[j], to_f32(ring[(t % p.W) * C + c]), acc);
    }
    acc = fmaf(w[p.W - 1], to_f32(u[c]), acc);
    xbc[i] = silu(acc);
    if (i < kP || writes_group) ring[(pos % p.W) * C + c] = u[c];
  }
  __syncthreads();
  float d = p.dt_f32 ? static_cast<const float*>(p.dt)[b * p.dt_batch + h]
                     : to_f32(static_cast<const T*>(p.dt)[b * p.dt_batch + h]);
  if (p.dt_bias) d += p.dt_bias[h];
  if (p.softplus) d = softplus(d);
  const float decay = expf(d * p.A[h]);
  const float skip = p.D[h];
  const int64_t base = (slot * p.H + h) * kP * p.N;
  float* out = p.new_state ? p.new_state : const_cast<float*>(p.state);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (int r = warp; r < kP; r += kThreads / 32) {
    const float dx = d * xbc[r];
    float acc = 0.f;
    for (int n = lane; n < p.N; n += 32) {
      const int64_t i = base + r * p.N + n;
      const float v = fmaf(decay, p.state[i], dx * xbc[kP + n]);
      out[i] = v;
      acc = fmaf(v, xbc[kP + p.N + n], acc);
    }
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (lane == 0) {
      acc = fmaf(skip, xbc[r], acc);
      if (p.z) acc *= silu(to_f32(static_cast<const T*>(p.z)[b * p.z_batch + h * kP + r]));
      y[r] = from_f32<T>(acc);
    }
  }
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
  const dim3 grid(static_cast<unsigned>(p.H), static_cast<unsigned>(a->batch));
  return launched(a->dtype == SSD_BF16
                      ? launch_k(step_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, stream, false, p)
                      : launch_k(step_kernel<float>, grid, dim3(kThreads), 0, stream, false, p));
}
