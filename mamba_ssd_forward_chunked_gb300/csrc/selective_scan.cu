// The selective scan: a recurrence with its own decay for every channel c and
// state n, d_t[c] the step:
//   h_t[c][n] = exp(d_t[c] A[c][n]) h_{t-1}[c][n] + d_t[c] u_t[c] B_t[n]
//   y_t[c] = (sum_n h_t[c][n] C_t[n] + D[c] u_t[c]) silu(z_t[c]).
//
// One thread per channel walks down the tokens with the channel's states in
// registers.  The decay is 2^(d A log2 e), log2 e folded into A once.
#include "layer.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 64;
constexpr float kLog2e = 1.4426950408889634f;

struct ScanParams {
  int64_t L;
  int D, N, G, softplus;
  const void *u, *delta, *z, *Bm, *Cm;
  int64_t ub, ut, db, dt, zb, zt, Bb, Bt, Cb, Ct;
  const float *A, *skip, *delta_bias, *init;
  float* final_state;
  void* y;
  const int32_t* lengths;
};

template <typename T, int NS>
__global__ void __launch_bounds__(kThreads) scan_kernel(ScanParams p) {
  const int c = blockIdx.x * kThreads + threadIdx.x;
  const int64_t b = blockIdx.y;
  if (c >= p.D) return;
  int64_t len = p.L;
  if (p.lengths) len = p.lengths[b] < 0 ? 0 : p.lengths[b] < p.L ? p.lengths[b] : p.L;
  const int g = c / (p.D / p.G);
  const int64_t row = (b * p.D + c) * p.N;
  float h[NS], a[NS];
#pragma unroll
  for (int n = 0; n < NS; ++n) {
    a[n] = n < p.N ? p.A[static_cast<int64_t>(c) * p.N + n] * kLog2e : 0.f;
    h[n] = n < p.N && p.init ? p.init[row + n] : 0.f;
  }
  const float skip = p.skip ? p.skip[c] : 0.f, bias = p.delta_bias ? p.delta_bias[c] : 0.f;
  const T* u = static_cast<const T*>(p.u) + b * p.ub + c;
  const T* delta = static_cast<const T*>(p.delta) + b * p.db + c;
  const T* z = p.z ? static_cast<const T*>(p.z) + b * p.zb + c : nullptr;
  const T* Bm = static_cast<const T*>(p.Bm) + b * p.Bb + static_cast<int64_t>(g) * p.N;
  const T* Cm = static_cast<const T*>(p.Cm) + b * p.Cb + static_cast<int64_t>(g) * p.N;
  T* y = static_cast<T*>(p.y) + b * p.L * p.D + c;
  for (int64_t t = 0; t < len; ++t) {
    float d = to_f32(delta[t * p.dt]) + bias;
    if (p.softplus) d = softplus(d);
    const float ut = to_f32(u[t * p.ut]);
    const float du = d * ut;
    float acc = skip * ut;
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      if (n < p.N) {
        h[n] = fmaf(exp2f(d * a[n]), h[n], du * to_f32(Bm[t * p.Bt + n]));
        acc = fmaf(h[n], to_f32(Cm[t * p.Ct + n]), acc);
      }
    }
    if (z) acc *= silu(to_f32(z[t * p.zt]));
    y[t * p.D] = from_f32<T>(acc);
  }
  for (int64_t t = len; t < p.L; ++t) y[t * p.D] = from_f32<T>(0.f);
  if (p.final_state) {
#pragma unroll
    for (int n = 0; n < NS; ++n)
      if (n < p.N) p.final_state[row + n] = h[n];
  }
}

template <typename T>
cudaError_t launch(const ScanParams& p, int64_t batch, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(ceil_div(p.D, kThreads)), static_cast<unsigned>(batch));
  auto k = p.N <= 16 ? scan_kernel<T, 16> : p.N <= 32 ? scan_kernel<T, 32> : scan_kernel<T, 64>;
  return launch_k(k, grid, dim3(kThreads), 0, stream, false, p);
}

ssd_status check_sizes(const ssd_selective_scan_args* a) {
  if (!a || a->size != static_cast<int64_t>(sizeof(*a))) return SSD_ERR_INVALID_ARG;
  if (a->batch < 0 || a->seqlen < 0 || a->channels <= 0 || a->dstate <= 0 || a->ngroups <= 0) return SSD_ERR_INVALID_ARG;
  if (a->dstate > 64 || a->channels % a->ngroups != 0 || a->batch > 65535) return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

}  // namespace
}  // namespace ssd

extern "C" size_t ssd_selective_scan_workspace_size(const ssd_selective_scan_args* a) {
  if (ssd::check_sizes(a) != SSD_OK) return 0;
  return 0;
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
  p.L = a->seqlen;
  p.D = a->channels;
  p.N = a->dstate;
  p.G = a->ngroups;
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
