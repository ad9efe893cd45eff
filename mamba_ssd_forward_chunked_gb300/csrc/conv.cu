// The short causal convolution of a Mamba layer, for prompts and single tokens:
//   y[t][c] = act(bias[c] + sum_{j<W} w[c][j] u[t - W + 1 + j][c]).
//
// Each input element is used by W outputs of its own channel only, so the work
// is one pass over memory: a thread walks down a run of tokens of its channel
// with the last W - 1 inputs in registers.
//
// The ring may be read and updated in place: the thread that owns a channel's
// first run is the only one that reads the ring, and it writes it too, after
// that read.
#include "layer.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 128;
constexpr int kRun = 32;  // tokens per block

struct ConvParams {
  int64_t L, u_batch, u_token, nslots;
  int C, silu;
  const void* u;
  const float *weight, *bias;
  const void* ring;
  void* new_ring;
  const int32_t *positions, *lengths, *slots;
  void* out[3];
  int begin[4];  // first channel of each output; begin[nout] = C
};

template <typename T, int W>
__global__ void __launch_bounds__(kThreads) conv_kernel(ConvParams p) {
  const int c = blockIdx.x * kThreads + threadIdx.x;
  const int b = blockIdx.z;
  if (c >= p.C) return;
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * kRun;
  const int64_t t1 = t0 + kRun < p.L ? t0 + kRun : p.L;
  const int64_t slot = p.slots ? p.slots[b] : b;
  const bool idle = slot < 0 || slot >= p.nslots;
  int64_t len = p.L;
  if (p.lengths) len = p.lengths[b] < 0 ? 0 : p.lengths[b] < p.L ? p.lengths[b] : p.L;
  if (idle && p.ring) len = 0;
  const int64_t pos = p.positions && p.positions[b] > 0 ? p.positions[b] : 0;
  const T* u = static_cast<const T*>(p.u) + b * p.u_batch + c;
  const T* ring = static_cast<const T*>(p.ring);
  if (ring && !idle) ring += slot * W * p.C + c;

  float w[W], win[W];  // win[j]: input of token t - W + 1 + j
#pragma unroll
  for (int j = 0; j < W; ++j) w[j] = p.weight[static_cast<int64_t>(c) * W + j];
  const float bias = p.bias ? p.bias[c] : 0.f;
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    const int64_t t = t0 - (W - 1) + j;
    win[j + 1] = 0.f;
    if (t >= 0) {
      if (t < len) win[j + 1] = to_f32(u[t * p.u_token]);
    } else if (ring && !idle && pos + t >= 0) {
      win[j + 1] = to_f32(ring[((pos + t) % W) * p.C]);
    }
  }
  if (t0 == 0 && ring && !idle) {
    T* nr = p.new_ring ? static_cast<T*>(p.new_ring) + slot * W * p.C + c : const_cast<T*>(ring);
    if (p.new_ring && len < W) {
#pragma unroll
      for (int q = 0; q < W; ++q) nr[q * p.C] = ring[q * p.C];
    }
    for (int64_t t = len > W ? len - W : 0; t < len; ++t) nr[((pos + t) % W) * p.C] = u[t * p.u_token];
  }
  int part = 0;
  while (c >= p.begin[part + 1]) ++part;
  const int64_t width = p.begin[part + 1] - p.begin[part];
  T* out = static_cast<T*>(p.out[part]) + static_cast<int64_t>(b) * p.L * width + (c - p.begin[part]);
  for (int64_t t = t0; t < t1; ++t) {
    if (t >= len) {
      out[t * width] = from_f32<T>(0.f);
      continue;
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) win[j] = win[j + 1];
    win[W - 1] = to_f32(u[t * p.u_token]);
    float acc = bias;
#pragma unroll
    for (int j = 0; j < W; ++j) acc = fmaf(w[j], win[j], acc);
    out[t * width] = from_f32<T>(p.silu ? silu(acc) : acc);
  }
}

template <typename T>
cudaError_t launch(const ConvParams& p, int width, int64_t batch, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(ceil_div(p.C, kThreads)),
                  static_cast<unsigned>(p.L > 0 ? ceil_div(p.L, kRun) : 1), static_cast<unsigned>(batch));
  auto k = width == 2 ? conv_kernel<T, 2> : width == 3 ? conv_kernel<T, 3> : conv_kernel<T, 4>;
  return launch_k(k, grid, dim3(kThreads), 0, stream, false, p);
}

}  // namespace

int layer_sm_count() {
  static int cache[64] = {0};
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
  if (cache[dev] == 0 && cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) cache[dev] = n;
  return cache[dev] > 0 ? cache[dev] : 152;
}

}  // namespace ssd

extern "C" ssd_status ssd_conv_fwd(const ssd_conv_args* a, ssd_stream_t stream) {
  using namespace ssd;
  if (!a || a->size != static_cast<int64_t>(sizeof(*a))) return SSD_ERR_INVALID_ARG;
  if (a->batch < 0 || a->seqlen < 0 || a->channels <= 0 || a->nslots < 0) return SSD_ERR_INVALID_ARG;
  if (!known_dtype(a->dtype) || a->width < 2 || a->width > 4) return SSD_ERR_UNSUPPORTED;
  if (a->activation != SSD_ACT_NONE && a->activation != SSD_ACT_SILU) return SSD_ERR_UNSUPPORTED;
  if (a->batch > 65535 || ceil_div(a->seqlen, kRun) > 65535) return SSD_ERR_UNSUPPORTED;
  if (a->nout < 1 || a->nout > 3) return SSD_ERR_INVALID_ARG;
  const size_t es = elem_size(a->dtype);
  ConvParams p{};
  int64_t sum = 0;
  for (int i = 0; i < a->nout; ++i) {
    if (a->out_channels[i] <= 0) return SSD_ERR_INVALID_ARG;
    p.begin[i] = static_cast<int>(sum);
    sum += a->out_channels[i];
    if (sum > a->channels) return SSD_ERR_INVALID_ARG;
    p.out[i] = a->out[i];
  }
  if (sum != a->channels) return SSD_ERR_INVALID_ARG;
  for (int i = a->nout; i < 4; ++i) p.begin[i] = a->channels;
  if (a->batch == 0) return SSD_OK;
  if (!a->weight) return SSD_ERR_INVALID_ARG;
  for (const void* t : {(const void*)a->weight, (const void*)a->bias, (const void*)a->positions,
                        (const void*)a->lengths, (const void*)a->slots})
    if (!aligned_to(t, 4)) return SSD_ERR_INVALID_ARG;
  if (a->seqlen > 0) {
    if (!a->u || !aligned_to(a->u, es)) return SSD_ERR_INVALID_ARG;
    for (int i = 0; i < a->nout; ++i)
      if (!a->out[i] || !aligned_to(a->out[i], es)) return SSD_ERR_INVALID_ARG;
  }
  if (a->ring) {
    if (!aligned_to(a->ring, es) || !aligned_to(a->new_ring, es)) return SSD_ERR_INVALID_ARG;
    if (!a->slots && a->nslots < a->batch) return SSD_ERR_INVALID_ARG;
  } else {
    if (a->new_ring || a->slots) return SSD_ERR_INVALID_ARG;
    if (a->seqlen == 0) return SSD_OK;
  }
  p.L = a->seqlen;
  p.u_batch = a->u_batch;
  p.u_token = a->u_token;
  p.nslots = a->nslots;
  p.C = a->channels;
  p.silu = a->activation == SSD_ACT_SILU;
  p.u = a->u;
  p.weight = a->weight;
  p.bias = a->bias;
  p.ring = a->ring;
  p.new_ring = a->new_ring == a->ring ? nullptr : a->new_ring;
  p.positions = a->positions;
  p.lengths = a->lengths;
  p.slots = a->slots;
  return launched(a->dtype == SSD_BF16 ? launch<__nv_bfloat16>(p, a->width, a->batch, stream)
                                       : launch<float>(p, a->width, a->batch, stream));
}
