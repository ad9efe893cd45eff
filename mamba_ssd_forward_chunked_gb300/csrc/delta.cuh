// The gated delta rule's launches and what they share: parameters and the gates.
#pragma once
#include "layer.cuh"

namespace ssd {

struct DeltaParams {
  int64_t batch, seqlen, nslots;
  int64_t x_batch, x_token, B_batch, B_token, C_batch, C_token, dt_batch, dt_token, beta_batch, beta_token;
  int H, G, P, N;
  int parts;  // 16-bit numbers a value of x, Bm, Cm and y takes: 1 or 2
  int gate_f32, softplus, sigmoid;
  float scale, norm_eps;  // norm_eps below 0: rows as they are
  const void *x, *Bm, *Cm, *dt, *beta;
  const float *A, *dt_bias;
  const float* init_state;
  float* final_state;
  const int32_t *slots, *positions, *lengths;
  void* y;
};

// A sequence's row of the cache (-1: idle), whether it has a state, and its tokens.
struct DeltaSeq {
  int64_t row;
  bool resumed;
  int length;
};
__device__ __forceinline__ DeltaSeq delta_sequence(const DeltaParams& p, int64_t b) {
  DeltaSeq s;
  s.row = p.slots ? p.slots[b] : b;
  if (s.row < 0 || s.row >= p.nslots) s.row = -1;
  s.resumed = p.init_state && (!p.positions || p.positions[b] > 0);
  const int64_t n = p.lengths ? p.lengths[b] : p.seqlen;
  s.length = static_cast<int>(n < 0 ? 0 : n > p.seqlen ? p.seqlen : n);
  return s;
}

template <typename T>
__device__ __forceinline__ float delta_gate(const DeltaParams& p, const void* base, int64_t at) {
  return p.gate_f32 ? static_cast<const float*>(base)[at] : to_f32(static_cast<const T*>(base)[at]);
}
// dt * A, the logarithm of a token's decay, and beta.
template <typename T>
__device__ __forceinline__ float delta_log_decay(const DeltaParams& p, int64_t b, int64_t t, int h) {
  float d = delta_gate<T>(p, p.dt, b * p.dt_batch + t * p.dt_token + h);
  if (p.dt_bias) d += p.dt_bias[h];
  if (p.softplus) d = softplus(d);
  return d * p.A[h];
}
template <typename T>
__device__ __forceinline__ float delta_beta(const DeltaParams& p, int64_t b, int64_t t, int h) {
  const float v = delta_gate<T>(p, p.beta, b * p.beta_batch + t * p.beta_token + h);
  return p.sigmoid ? 1.f / (1.f + expf(-v)) : v;
}
// What a row with this sum of squares is multiplied by.
__device__ __forceinline__ float delta_norm(const DeltaParams& p, float squares) {
  if (p.norm_eps < 0.f) return 1.f;
  const float s = squares + p.norm_eps;
  return s > 0.f ? 1.f / sqrtf(s) : 0.f;
}

}  // namespace ssd
