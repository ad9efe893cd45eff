// The short causal convolution of a Mamba layer, for prompts and single tokens:
//   y[t][c] = act(bias[c] + sum_{j<W} w[c][j] u[t - W + 1 + j][c]).
//
// Each input element is used by W outputs of its own channel only, so the work
// is one pass over memory, and HBM bounds it.  A thread takes four channels (8 or
// 16 bytes) and walks down a run of tokens with the last W - 1 inputs in
// registers; the next eight tokens are on their way while eight are computed.
// A run reads the W - 1 tokens before it again (from L2, mostly).  4 x 4096 x 5376
// bf16, out of rows of 10576: 59 us, 6.0 TB/s (a contiguous copy of as many bytes
// 55 us); 3 x 1021 x 2304 fp32 10 us.
//
// The ring may be read and updated in place: the thread that owns a channel's
// first run is the only one that reads the ring, and it writes it too, after
// that read.
#include "layer.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 128;
constexpr int kStep = 8;  // tokens loaded together

struct ConvParams {
  int64_t L, u_batch, u_token, nslots;
  int C, silu, run;  // run: tokens a thread walks down, a multiple of kStep
  const void* u;
  const float *weight, *bias;
  const void* ring;
  void* new_ring;
  const int32_t *positions, *lengths, *slots;
  void* out[3];
  int begin[4];  // first channel of each output; begin[nout] = C
};

// kC consecutive channels of one token, as they lie in memory.
template <typename T, int kC>
struct Chans;
template <typename T>
struct Chans<T, 1> {
  T v;
  __device__ __forceinline__ void load(const T* p) { v = *p; }
  __device__ __forceinline__ void store(T* p) const { *p = v; }
  __device__ __forceinline__ float get(int) const { return to_f32(v); }
  __device__ __forceinline__ void set(const float (&f)[1]) { v = from_f32<T>(f[0]); }
};
template <>
struct Chans<float, 4> {
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = v; }
  __device__ __forceinline__ float get(int i) const { return (&v.x)[i]; }
  __device__ __forceinline__ void set(const float (&f)[4]) { v = make_float4(f[0], f[1], f[2], f[3]); }
};
template <>
struct Chans<__nv_bfloat16, 4> {
  uint2 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint2*>(p) = v; }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t w = i < 2 ? v.x : v.y;
    return __uint_as_float(i % 2 ? w & 0xFFFF0000u : w << 16);
  }
  __device__ __forceinline__ void set(const float (&f)[4]) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(f[0], f[1]), hi = __floats2bfloat162_rn(f[2], f[3]);
    v = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
};

template <typename T, int W, int kC>
__global__ void __launch_bounds__(kThreads) conv_kernel(ConvParams p) {
  using Ch = Chans<T, kC>;
  begin_kernel();
  const int groups = p.C / kC;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t t0 = id / groups * p.run;
  const int c = static_cast<int>(id % groups) * kC;
  const int b = blockIdx.y;
  if (t0 >= p.L && t0 > 0) return;
  const int64_t t1 = t0 + p.run < p.L ? t0 + p.run : p.L;
  const int64_t slot = p.slots ? p.slots[b] : b;
  const bool idle = p.ring && (slot < 0 || slot >= p.nslots);
  int64_t len = p.L;
  if (p.lengths) len = p.lengths[b] < 0 ? 0 : p.lengths[b] < p.L ? p.lengths[b] : p.L;
  if (idle) len = 0;
  const int64_t end = len < t1 ? len : t1;
  const int64_t pos = p.positions && p.positions[b] > 0 ? p.positions[b] : 0;
  const T* u = static_cast<const T*>(p.u) + b * p.u_batch + c;
  const T* ring = p.ring && !idle ? static_cast<const T*>(p.ring) + slot * W * p.C + c : nullptr;

  // token t0 + n of the run lies at u + n * step (a run is short: 32-bit offsets)
  const int n1 = static_cast<int>(t1 - t0), nend = end > t0 ? static_cast<int>(end - t0) : 0;
  const T* in = u + t0 * p.u_token;
  Ch next[kStep];
  auto fetch = [&](int n) {
    const T* from = in + n * p.u_token;
    if (n + kStep <= nend) {
#pragma unroll
      for (int k = 0; k < kStep; ++k, from += p.u_token) next[k].load(from);
    } else {
#pragma unroll
      for (int k = 0; k < kStep; ++k, from += p.u_token)
        if (n + k < nend) next[k].load(from);
    }
  };
  fetch(0);

  float w[W][kC], win[W][kC], bias[kC];  // win[j]: input of token t - W + 1 + j
  if constexpr (W == 4) {
    static_assert(sizeof(float4) == W * sizeof(float), "a channel's taps are one vector");
    const bool vec = (reinterpret_cast<uintptr_t>(p.weight) & 15) == 0;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const float* row = p.weight + static_cast<int64_t>(c + i) * W;
      float4 f;
      if (vec) f = *reinterpret_cast<const float4*>(row);
      else f = make_float4(row[0], row[1], row[2], row[3]);
      w[0][i] = f.x, w[1][i] = f.y, w[2][i] = f.z, w[3][i] = f.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kC; ++i)
#pragma unroll
      for (int j = 0; j < W; ++j) w[j][i] = p.weight[static_cast<int64_t>(c + i) * W + j];
  }
#pragma unroll
  for (int i = 0; i < kC; ++i) bias[i] = p.bias ? p.bias[c + i] : 0.f;
#pragma unroll
  for (int j = 1; j < W; ++j) {
    const int64_t t = t0 - W + j;
    Ch before;
    const bool in_call = t >= 0 && t < len, in_ring = t < 0 && ring && pos + t >= 0;
    if (in_call) before.load(u + t * p.u_token);
    else if (in_ring) before.load(ring + (pos + t) % W * p.C);
#pragma unroll
    for (int i = 0; i < kC; ++i) win[j][i] = in_call || in_ring ? before.get(i) : 0.f;
  }
  if (t0 == 0 && ring) {
    T* keep = p.new_ring ? static_cast<T*>(p.new_ring) + slot * W * p.C + c : const_cast<T*>(ring);
    Ch v;
    if (p.new_ring && len < W) {  // slots that no token of this call takes
#pragma unroll
      for (int q = 0; q < W; ++q) {
        v.load(ring + static_cast<int64_t>(q) * p.C);
        v.store(keep + static_cast<int64_t>(q) * p.C);
      }
    }
    for (int64_t t = len > W ? len - W : 0; t < len; ++t) {
      v.load(u + t * p.u_token);
      v.store(keep + (pos + t) % W * p.C);
    }
  }
  int part = 0;
  while (c >= p.begin[part + 1]) ++part;
  const int64_t width = p.begin[part + 1] - p.begin[part];
  T* out = static_cast<T*>(p.out[part]) + static_cast<int64_t>(b) * p.L * width + (c - p.begin[part]);
  out += t0 * width;
  for (int n = 0; n < n1; n += kStep) {
    Ch now[kStep];
#pragma unroll
    for (int k = 0; k < kStep; ++k) now[k] = next[k];
    fetch(n + kStep);
    auto put = [&](int k, bool live) {
      float acc[kC];
#pragma unroll
      for (int i = 0; i < kC; ++i) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) win[j][i] = win[j + 1][i];
        win[W - 1][i] = now[k].get(i);
        acc[i] = bias[i];
#pragma unroll
        for (int j = 0; j < W; ++j) acc[i] = fmaf(w[j][i], win[j][i], acc[i]);
        if (p.silu) acc[i] = silu(acc[i]);
        if (!live) acc[i] = 0.f;
      }
      Ch y;
      y.set(acc);
      y.store(out);
      out += width;
    };
    if (n + kStep <= nend) {
#pragma unroll
      for (int k = 0; k < kStep; ++k) put(k, true);
    } else {
#pragma unroll
      for (int k = 0; k < kStep; ++k)
        if (n + k < n1) put(k, n + k < nend);
    }
  }
}

template <typename T>
cudaError_t launch(ConvParams p, int width, int64_t batch, cudaStream_t stream) {
  // four channels at a time where they start on a whole vector in every row
  const size_t bytes = 4 * sizeof(T);
  bool vec = p.C % 4 == 0 && aligned_to(p.u, bytes) && p.u_token % 4 == 0 && p.u_batch % 4 == 0 &&
             aligned_to(p.ring, bytes) && aligned_to(p.new_ring, bytes);
  for (int i = 0; i < 3; ++i) vec = vec && p.begin[i] % 4 == 0 && aligned_to(p.out[i], bytes);
  const int64_t groups = vec ? p.C / 4 : p.C;
  // The shortest runs whose blocks are all resident at once (five a multiprocessor in bf16, four in
  // fp32, by their registers): every thread starts at once and none waits for a second wave.  Up to
  // kMost tokens; above that blocks come in waves.  Runs of 8, 16, 24 and 32 for 3 x 1021 x 2304 fp32
  // (24 fit): 12.2, 11.4, 9.6 and 10.9 us; 4 x 4096 x 5376 bf16 with runs of 64, 128 and 240 (which fit):
  // 65, 63 and 59 us; 2 x 8191 x 4352 fp32 with 128 and 472: 87 and 92 us.
  constexpr bool kHalf = sizeof(T) == 2;
  constexpr int kMost = kHalf ? 1024 : 128;
  const int64_t resident = (kHalf ? 5 : 4) * static_cast<int64_t>(layer_sm_count());
  p.run = kStep;
  while (p.run < kMost && ceil_div(groups * ceil_div(p.L, p.run), kThreads) * batch > resident) p.run += kStep;
  const int64_t runs = p.L > 0 ? ceil_div(p.L, p.run) : 1;
  const dim3 grid(static_cast<unsigned>(ceil_div(groups * runs, kThreads)), static_cast<unsigned>(batch));
  auto k = vec ? (width == 2 ? conv_kernel<T, 2, 4> : width == 3 ? conv_kernel<T, 3, 4> : conv_kernel<T, 4, 4>)
               : (width == 2 ? conv_kernel<T, 2, 1> : width == 3 ? conv_kernel<T, 3, 1> : conv_kernel<T, 4, 1>);
  return launch_k(k, grid, dim3(kThreads), 0, stream, true, p);
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
  if (a->batch > 65535 || a->seqlen > (int64_t(1) << 30)) return SSD_ERR_UNSUPPORTED;
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
