// Beam search: the k best of beams x vocab candidates, and the reordering of
// the states that the choice decides.
//
// Selection in two launches: each beam's log-sum-exp, then per request k rounds
// over all candidates, each taking the largest key below the last one taken.  A
// key holds a score in the order of unsigned integers and the complement of the
// candidate's index, so keys differ and equal scores fall by rising index.
//
// Reordering moves bytes: a thread owns a few bytes' position in all rows of a
// request, reads them all, then writes, so that it may work in place.
#include <cfloat>

#include "layer.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxBeams = 64;

struct SelectParams {
  int64_t logits_batch, logits_beam;
  int beams, vocab, k, eos;
  const void* logits;
  const float* scores;
  const uint8_t* finished;
  float* out_scores;
  int32_t *parents, *tokens;
  float* lse;  // [batch][beams]
};

// Scores in the order of unsigned integers; -0 and +0 are one score.
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}

// A candidate's score; a NaN counts as -infinity.
__device__ __forceinline__ float score_of(float beam, float x, float lse) {
  const float s = beam + (x - lse);
  return s == s ? s : -INFINITY;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) lse_kernel(SelectParams p) {
  __shared__ float red[kThreads];
  const int64_t b = blockIdx.y;
  const int w = blockIdx.x;
  const T* x = static_cast<const T*>(p.logits) + b * p.logits_batch + w * p.logits_beam;
  float top = -INFINITY;
  bool nan = false;
  for (int v = threadIdx.x; v < p.vocab; v += kThreads) {
    const float f = to_f32(x[v]);
    nan |= f != f;
    top = fmaxf(top, f);
  }
  nan = __syncthreads_or(nan);
  red[threadIdx.x] = top;
  __syncthreads();
  for (int o = kThreads / 2; o > 0; o >>= 1) {
    if (threadIdx.x < o) red[threadIdx.x] = fmaxf(red[threadIdx.x], red[threadIdx.x + o]);
    __syncthreads();
  }
  top = red[0];
  __syncthreads();
  float sum = 0.f;
  for (int v = threadIdx.x; v < p.vocab; v += kThreads) sum += expf(to_f32(x[v]) - top);
  red[threadIdx.x] = sum;
  __syncthreads();
  for (int o = kThreads / 2; o > 0; o >>= 1) {
    if (threadIdx.x < o) red[threadIdx.x] += red[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) p.lse[b * p.beams + w] = nan ? NAN : top + logf(red[0]);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) select_kernel(SelectParams p) {
  __shared__ unsigned long long red[kThreads];
  const int64_t b = blockIdx.x;
  unsigned long long last = ~0ull;
  for (int i = 0; i < p.k; ++i) {
    unsigned long long best = 0;
    for (int w = 0; w < p.beams; ++w) {
      const T* x = static_cast<const T*>(p.logits) + b * p.logits_batch + w * p.logits_beam;
      const float s = p.scores[b * p.beams + w], lse = p.lse[b * p.beams + w];
      const bool done = p.finished && p.finished[b * p.beams + w];
      for (int v = threadIdx.x; v < p.vocab; v += kThreads) {
        float f = done ? (v == p.eos ? s : -INFINITY) : score_of(s, to_f32(x[v]), lse);
        if (f != f) f = -INFINITY;
        const uint32_t flat = static_cast<uint32_t>(w) * p.vocab + v;
        const unsigned long long key = (static_cast<unsigned long long>(order_of(f)) << 32) | (~flat);
        if (key < last && key > best) best = key;
      }
    }
    red[threadIdx.x] = best;
    __syncthreads();
    for (int o = kThreads / 2; o > 0; o >>= 1) {
      if (threadIdx.x < o && red[threadIdx.x + o] > red[threadIdx.x]) red[threadIdx.x] = red[threadIdx.x + o];
      __syncthreads();
    }
    last = red[0];
    __syncthreads();
    if (threadIdx.x == 0) {
      const uint32_t flat = ~static_cast<uint32_t>(last);
      p.out_scores[b * p.k + i] = value_of(static_cast<uint32_t>(last >> 32));
      p.parents[b * p.k + i] = static_cast<int32_t>(flat / p.vocab);
      p.tokens[b * p.k + i] = static_cast<int32_t>(flat % p.vocab);
    }
  }
}

struct ReorderParams {
  int beams, k, count;
  const int32_t* parents;
  const void* src[SSD_REORDER_MAX];
  void* dst[SSD_REORDER_MAX];
  int64_t row_bytes[SSD_REORDER_MAX];
};

template <typename V>
__global__ void __launch_bounds__(kThreads) reorder_kernel(ReorderParams p, int j) {
  const int64_t units = p.row_bytes[j] / static_cast<int64_t>(sizeof(V));
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t b = blockIdx.y;
  if (at >= units) return;
  const V* src = static_cast<const V*>(p.src[j]) + b * p.beams * units + at;
  V* dst = static_cast<V*>(p.dst[j]) + b * p.k * units + at;
  const bool in_place = p.src[j] == p.dst[j];
  V v[kMaxBeams];
  for (int i = 0; i < p.k; ++i) {
    const int from = p.parents[b * p.k + i];
    if (from >= 0 && from < p.beams && !(in_place && from == i)) v[i] = src[from * units];
  }
  for (int i = 0; i < p.k; ++i) {
    const int from = p.parents[b * p.k + i];
    if (from >= 0 && from < p.beams && !(in_place && from == i)) dst[i * units] = v[i];
  }
}

template <typename V>
cudaError_t launch_reorder(const ReorderParams& p, int j, int64_t batch, cudaStream_t stream) {
  const int64_t units = p.row_bytes[j] / static_cast<int64_t>(sizeof(V));
  const dim3 grid(static_cast<unsigned>(ceil_div(units, kThreads)), static_cast<unsigned>(batch));
  return launch_k(reorder_kernel<V>, grid, dim3(kThreads), 0, stream, false, p, j);
}

ssd_status check_select(const ssd_beam_select_args* a) {
  if (!a || a->size != static_cast<int64_t>(sizeof(*a))) return SSD_ERR_INVALID_ARG;
  if (a->batch < 0 || a->beams <= 0 || a->vocab <= 0 || a->k <= 0) return SSD_ERR_INVALID_ARG;
  const int64_t all = static_cast<int64_t>(a->beams) * a->vocab;
  if (a->batch > 65535 || a->beams > kMaxBeams || a->k > kMaxBeams || all >= (int64_t(1) << 31))
    return SSD_ERR_UNSUPPORTED;
  if (a->k > all) return SSD_ERR_INVALID_ARG;
  return SSD_OK;
}

}  // namespace
}  // namespace ssd

extern "C" size_t ssd_beam_select_workspace_size(const ssd_beam_select_args* a) {
  if (ssd::check_select(a) != SSD_OK) return 0;
  return static_cast<size_t>(a->batch) * a->beams * sizeof(float);
}

extern "C" ssd_status ssd_beam_select(const ssd_beam_select_args* a, ssd_stream_t stream) {
  using namespace ssd;
  ssd_status st = check_select(a);
  if (st != SSD_OK) return st;
  if (!known_dtype(a->dtype)) return SSD_ERR_UNSUPPORTED;
  if (a->finished && (a->eos < 0 || a->eos >= a->vocab)) return SSD_ERR_INVALID_ARG;
  if (a->batch == 0) return SSD_OK;
  if (!a->logits || !aligned_to(a->logits, elem_size(a->dtype))) return SSD_ERR_INVALID_ARG;
  for (const void* t : {(const void*)a->scores, (const void*)a->out_scores, (const void*)a->parents, (const void*)a->tokens})
    if (!t || !aligned_to(t, 4)) return SSD_ERR_INVALID_ARG;
  if (!a->workspace || !aligned_to(a->workspace, 16)) return SSD_ERR_INVALID_ARG;
  if (a->workspace_bytes < ssd_beam_select_workspace_size(a)) return SSD_ERR_WORKSPACE;
  SelectParams p{};
  p.logits_batch = a->logits_batch, p.logits_beam = a->logits_beam;
  p.beams = a->beams, p.vocab = a->vocab, p.k = a->k, p.eos = a->eos;
  p.logits = a->logits, p.scores = a->scores, p.finished = a->finished;
  p.out_scores = a->out_scores, p.parents = a->parents, p.tokens = a->tokens;
  p.lse = static_cast<float*>(a->workspace);
  const unsigned batch = static_cast<unsigned>(a->batch);
  const dim3 rows(static_cast<unsigned>(p.beams), batch);
  const bool bf16 = a->dtype == SSD_BF16;
  cudaError_t e = bf16 ? launch_k(lse_kernel<__nv_bfloat16>, rows, dim3(kThreads), 0, stream, false, p)
                       : launch_k(lse_kernel<float>, rows, dim3(kThreads), 0, stream, false, p);
  if (e != cudaSuccess) return SSD_ERR_CUDA;
  e = bf16 ? launch_k(select_kernel<__nv_bfloat16>, dim3(batch), dim3(kThreads), 0, stream, false, p)
           : launch_k(select_kernel<float>, dim3(batch), dim3(kThreads), 0, stream, false, p);
  return launched(e);
}

extern "C" ssd_status ssd_beam_reorder(const ssd_beam_reorder_args* a, ssd_stream_t stream) {
  using namespace ssd;
  if (!a || a->size != static_cast<int64_t>(sizeof(*a))) return SSD_ERR_INVALID_ARG;
  if (a->batch < 0 || a->beams <= 0 || a->k <= 0 || a->count < 0 || a->count > SSD_REORDER_MAX) return SSD_ERR_INVALID_ARG;
  if (a->batch > 65535 || a->beams > kMaxBeams || a->k > kMaxBeams) return SSD_ERR_UNSUPPORTED;
  ReorderParams p{};
  p.beams = a->beams, p.k = a->k, p.count = a->count, p.parents = a->parents;
  for (int j = 0; j < a->count; ++j) {
    if (a->row_bytes[j] < 0) return SSD_ERR_INVALID_ARG;
    if (a->row_bytes[j] > 0 && a->batch > 0 && (!a->src[j] || !a->dst[j])) return SSD_ERR_INVALID_ARG;
    if (a->src[j] == a->dst[j] && a->k != a->beams) return SSD_ERR_INVALID_ARG;
    p.src[j] = a->src[j], p.dst[j] = a->dst[j], p.row_bytes[j] = a->row_bytes[j];
  }
  if (a->batch == 0 || a->count == 0) return SSD_OK;
  if (!a->parents || !aligned_to(a->parents, 4)) return SSD_ERR_INVALID_ARG;
  for (int j = 0; j < a->count; ++j) {
    if (p.row_bytes[j] == 0) continue;
    const uintptr_t bits = reinterpret_cast<uintptr_t>(p.src[j]) | reinterpret_cast<uintptr_t>(p.dst[j]) |
                           static_cast<uintptr_t>(p.row_bytes[j]);
    const cudaError_t e = (bits & 15) == 0 ? launch_reorder<uint4>(p, j, a->batch, stream)
                          : (bits & 3) == 0 ? launch_reorder<uint32_t>(p, j, a->batch, stream)
                                            : launch_reorder<uint8_t>(p, j, a->batch, stream);
    if (e != cudaSuccess) return SSD_ERR_CUDA;
  }
  return SSD_OK;
}
