// Products of a few tokens with 4-bit weights in groups of columns:
//   y[m][n] = sum_k x[m][k] (q[n][k] - 8) s[n][k / group]  (+ add[m][n]).
//
// One warp per (row n, token m): its lanes walk along the row's codes, sum each
// in 32 bits, and join at the end.
#include "layer.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 256;

struct W4Params {
  int64_t M, x_token, add_token;
  int n, k, group, ktiles, ngroups;
  const void* x;
  const uint32_t* packed;
  const float* scales;
  const void* add;
  void* y;
};

template <typename T>
__global__ void __launch_bounds__(kThreads) w4_kernel(W4Params p) {
  const int row = blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  const int64_t m = blockIdx.y;
  if (row >= p.n) return;
  const int lane = threadIdx.x % 32;
  const T* x = static_cast<const T*>(p.x) + m * p.x_token;
  const int a = (row >> 3) & 1, r = row & 7;
  float acc = 0.f;
  for (int k = lane; k < p.k; k += 32) {
    const int in = k & 63;
    const int h = in >> 5, c = (in >> 3) & 3, i = (in >> 2) & 1, e = (in >> 1) & 1, q = in & 1;
    const int64_t tile = static_cast<int64_t>(row >> 4) * p.ktiles + (k >> 6);
    const uint32_t word = p.packed[tile * 128 + (4 * r + c) * 4 + 2 * h + i];
    const int code = (word >> (4 * (a + 2 * e) + 16 * q)) & 15;
    acc = fmaf(to_f32(x[k]), (code - 8) * p.scales[static_cast<int64_t>(row) * p.ngroups + k / p.group], acc);
  }
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if (lane == 0) {
    if (p.add) acc += to_f32(static_cast<const T*>(p.add)[m * p.add_token + row]);
    static_cast<T*>(p.y)[m * p.n + row] = from_f32<T>(acc);
  }
}

}  // namespace
}  // namespace ssd

extern "C" ssd_status ssd_w4_matvec(const ssd_w4_matvec_args* a, ssd_stream_t stream) {
  using namespace ssd;
  if (!a || a->size != static_cast<int64_t>(sizeof(*a))) return SSD_ERR_INVALID_ARG;
  if (a->tokens < 0 || a->n <= 0 || a->k <= 0) return SSD_ERR_INVALID_ARG;
  if (!known_dtype(a->dtype) || (a->group != 32 && a->group != 64 && a->group != 128) || a->tokens > 65535)
    return SSD_ERR_UNSUPPORTED;
  if (a->tokens == 0) return SSD_OK;
  const size_t es = elem_size(a->dtype);
  if (!a->x || !aligned_to(a->x, es) || !a->y || !aligned_to(a->y, es) || !aligned_to(a->add, es) || !a->packed ||
      !aligned_to(a->packed, 16) || !a->scales || !aligned_to(a->scales, 4))
    return SSD_ERR_INVALID_ARG;
  W4Params p{};
  p.M = a->tokens, p.x_token = a->x_token, p.add_token = a->add_token;
  p.n = a->n, p.k = a->k, p.group = a->group;
  p.ktiles = static_cast<int>(ceil_div(a->k, 64)), p.ngroups = static_cast<int>(ceil_div(a->k, a->group));
  p.x = a->x, p.packed = static_cast<const uint32_t*>(a->packed), p.scales = a->scales, p.add = a->add, p.y = a->y;
  const dim3 grid(static_cast<unsigned>(ceil_div(p.n, kThreads / 32)), static_cast<unsigned>(p.M));
  return launched(a->dtype == SSD_BF16
                      ? launch_k(w4_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, stream, false, p)
                      : launch_k(w4_kernel<float>, grid, dim3(kThreads), 0, stream, false, p));
}
