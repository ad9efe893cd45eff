// Products of a few tokens with 4-bit weights in groups of columns:
//   y[m][n] = sum_k x[m][k] (q[n][k] - 8) s[n][k / group]  (+ add[m][n]).
//
// The codes are read once, half a byte each, and set the floor (HBM, or L2 for a
// layer's weights that stay there); what comes next is turning codes into
// operands.  The tensor core multiplies 16 rows by 16 columns by 8 tokens
// (mma.sync m16n8k16; the accumulator of a tcgen05 product has 128 rows of
// weights, which would be written to shared memory as bf16 first, four times the
// codes' bytes): a code becomes an exact bf16 by a mask into the low bits of 128
// (0x4300 | q = 128 + q) and a subtraction of 136, eight codes in 3 shifts, 4
// masks and 4 subtractions, and one token costs no less than eight.  The codes
// lie in the order of the product's fragments, so a lane's 16-byte load is its
// share of four products.
//
// x enters exactly: bf16 as it is, a 32-bit x as three bf16 parts
// x = hi + mid + lo in three columns of the product, added in 32 bits at the
// end.  A group's sum is scaled in 32 bits when its columns are done.
//
// A block takes 16 rows; its warps take column tiles in turn and their sums are
// joined in shared memory in a fixed order.
#include "layer.cuh"

namespace ssd {
namespace {

constexpr int kMaxWarps = 16;  // of a block

struct W4Params {
  int64_t x_token, add_token;
  int M, n, k, ktiles, ngroups;
  const void* x;
  const uint4* packed;
  const float* scales;
  const void* add;
  void* y;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Codes j of both halves of a word (bits 4 j and 16 + 4 j) minus 8, as two bf16.
template <int j>
__device__ __forceinline__ uint32_t codes(uint32_t w) {
  const uint32_t v = ((w >> (4 * j)) & 0x000F000Fu) | 0x43004300u;  // 128 + q
  __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), __nv_bfloat162(136.f, 136.f));
  return *reinterpret_cast<uint32_t*>(&r);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// A lane's eight columns (k0 ..) of its token, as the four operand words of two products.
template <bool kVec>
__device__ __forceinline__ void load_x(const __nv_bfloat16* x, int, int left, uint32_t (&w)[4]) {
  w[0] = w[1] = w[2] = w[3] = 0;
  if constexpr (kVec) {
    if (left > 0) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(x));
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) w[i / 2] |= static_cast<uint32_t>(__bfloat16_as_ushort(x[i])) << (16 * (i % 2));
  }
}
template <bool kVec>
__device__ __forceinline__ void load_x(const float* x, int part, int left, uint32_t (&w)[4]) {
  float f[8];
  if constexpr (kVec) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    if (left > 0) a = __ldg(reinterpret_cast<const float4*>(x)), b = __ldg(reinterpret_cast<const float4*>(x) + 1);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < left ? x[i] : 0.f;
  }
  // the part'th eight bits of x (cut, not rounded, so that no part overflows): 3 x 8 = 24 bits are all
  // of it.  An infinity or NaN is its own first part.
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    auto cut = [](float v) { return __uint_as_float(__float_as_uint(v) & 0xFFFF0000u); };
    if (fabsf(f[i]) < INFINITY) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (j < part) f[i] -= cut(f[i]);
      f[i] = cut(f[i]);
    } else if (part > 0) {
      f[i] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
}

// kCols: products' token columns in blocks of 8.  kGroup: columns a scale holds for.  kVec: k is a
// multiple of 8 and x's rows are 16-byte aligned.
template <typename T, int kCols, int kGroup, bool kVec>
__global__ void __launch_bounds__(kMaxWarps * 32) w4_kernel(W4Params p) {
  constexpr int kParts = sizeof(T) == 4 ? 3 : 1;        // columns of a token
  constexpr int kTokens = kCols * 8 / kParts;           // tokens of a block (fp32: 2 in 8 columns)
  extern __shared__ float red[];                        // [warps][kCols][4][32]
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int r = lane / 4, c = lane % 4;
  const int m0 = blockIdx.y * kTokens;
  const int row = blockIdx.x * 16 + r;

  const T* x[kCols];
  int part[kCols];
#pragma unroll
  for (int t = 0; t < kCols; ++t) {
    const int col = t * 8 + r;
    const int m = m0 + col / kParts;
    part[t] = col % kParts;
    x[t] = col / kParts < kTokens && m < p.M ? static_cast<const T*>(p.x) + m * p.x_token : nullptr;
  }
  // rows past the matrix hold codes of 8 and any scale will do
  const float* s0 = p.scales + static_cast<int64_t>(row < p.n ? row : p.n - 1) * p.ngroups;
  const float* s1 = p.scales + static_cast<int64_t>(row + 8 < p.n ? row + 8 : p.n - 1) * p.ngroups;
  const uint4* packed = p.packed + static_cast<int64_t>(blockIdx.x) * p.ktiles * 32 + lane;

  float total[kCols][4] = {};
  // a warp's unit: two tiles, 128 columns; its next kAhead units' codes are on their way together
  constexpr int kAhead = kCols * kParts == 1 ? 4 : 2;
  const int units = (p.ktiles + 1) / 2;
  for (int base = warp; base < units; base += kAhead * warps) {
    uint4 q[kAhead][2];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int kt = 2 * (base + u * warps) + h;
        q[u][h] = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);  // zeros past the end
        if (kt < p.ktiles) q[u][h] = __ldg(packed + static_cast<int64_t>(kt) * 32);
      }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int unit = base + u * warps;
      if (unit >= units) break;
      float sum[kCols][4] = {};
#pragma unroll
      for (int part4 = 0; part4 < 4; ++part4) {  // 32 columns: two products
        const int k0 = unit * 128 + part4 * 32 + c * 8;
        uint32_t xw[kCols][4];
#pragma unroll
        for (int t = 0; t < kCols; ++t) load_x<kVec>(x[t] + k0, part[t], x[t] ? p.k - k0 : 0, xw[t]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4& v = q[u][part4 / 2];
          const uint32_t w = part4 % 2 ? (i ? v.w : v.z) : (i ? v.y : v.x);
          const uint32_t a[4] = {codes<0>(w), codes<1>(w), codes<2>(w), codes<3>(w)};
#pragma unroll
          for (int t = 0; t < kCols; ++t) mma_bf16(sum[t], a, xw[t][2 * i], xw[t][2 * i + 1]);
        }
        constexpr int kParts32 = kGroup / 32;  // 32-column parts a scale holds for
        if (part4 % kParts32 == kParts32 - 1) {
          const int g = unit * (4 / kParts32) + part4 / kParts32;
          const float f0 = g < p.ngroups ? __ldg(s0 + g) : 0.f, f1 = g < p.ngroups ? __ldg(s1 + g) : 0.f;
#pragma unroll
          for (int t = 0; t < kCols; ++t) {
            total[t][0] = fmaf(f0, sum[t][0], total[t][0]);
            total[t][1] = fmaf(f0, sum[t][1], total[t][1]);
            total[t][2] = fmaf(f1, sum[t][2], total[t][2]);
            total[t][3] = fmaf(f1, sum[t][3], total[t][3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[t][e] = 0.f;
          }
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < kCols; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) red[((warp * kCols + t) * 4 + e) * 32 + lane] = total[t][e];
  __syncthreads();
  // (row i, token j) of the block: entry e = 2 (i / 8) + col % 2 of lane 4 (i % 8) + col % 8 / 2
  for (int at = threadIdx.x; at < 16 * kTokens; at += blockDim.x) {
    const int i = at % 16, j = at / 16;
    const int n = blockIdx.x * 16 + i, m = m0 + j;
    if (n >= p.n || m >= p.M) continue;
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < kParts; ++q) {
      const int col = j * kParts + q;
      const int e = 2 * (i / 8) + col % 2, from = 4 * (i % 8) + col % 8 / 2;
      float part_sum = 0.f;
      for (int w = 0; w < warps; ++w) part_sum += red[((w * kCols + col / 8) * 4 + e) * 32 + from];
      v += part_sum;
    }
    if (p.add) v += to_f32(static_cast<const T*>(p.add)[m * p.add_token + n]);
    static_cast<T*>(p.y)[static_cast<int64_t>(m) * p.n + n] = from_f32<T>(v);
  }
}

template <typename T, int kCols, int kGroup>
cudaError_t launch_cols(const W4Params& p, cudaStream_t stream) {
  constexpr int kTokens = kCols * 8 / (sizeof(T) == 4 ? 3 : 1);
  const bool vec = p.k % 8 == 0 && aligned_to(p.x, 16) && p.x_token * static_cast<int64_t>(sizeof(T)) % 16 == 0;
  const int64_t units = ceil_div(p.ktiles, 2);
  const dim3 grid(static_cast<unsigned>(ceil_div(p.n, 16)), static_cast<unsigned>(ceil_div(p.M, kTokens)));
  // as many warps as give every multiprocessor kWarps, at least 4, and no more than there are units
  // (2560 -> 10576, one token, with 16, 24, 32, 48 and 64: 6.3, 6.3, 6.0, 6.9 and 7.5 us)
  constexpr int64_t kWarps = 32;
  int64_t warps = ceil_div(kWarps * layer_sm_count(), static_cast<int64_t>(grid.x) * grid.y);
  warps = warps < 4 ? 4 : warps > kMaxWarps ? kMaxWarps : warps;
  if (warps > units) warps = units;
  const size_t smem = static_cast<size_t>(warps) * kCols * 4 * 32 * sizeof(float);
  return launch_k(vec ? w4_kernel<T, kCols, kGroup, true> : w4_kernel<T, kCols, kGroup, false>, grid,
                  dim3(static_cast<unsigned>(warps) * 32),
                  smem, stream, false, p);
}

template <typename T, int kGroup>
cudaError_t launch(const W4Params& p, cudaStream_t stream) {
  // one block of eight columns where all tokens fit, else two (twice the tokens for the codes' price)
  constexpr int kOne = 8 / (sizeof(T) == 4 ? 3 : 1);
  return p.M <= kOne ? launch_cols<T, 1, kGroup>(p, stream) : launch_cols<T, 2, kGroup>(p, stream);
}

template <typename T>
cudaError_t launch_group(const W4Params& p, int group, cudaStream_t stream) {
  return group == 32 ? launch<T, 32>(p, stream) : group == 64 ? launch<T, 64>(p, stream) : launch<T, 128>(p, stream);
}

}  // namespace
}  // namespace ssd

extern "C" ssd_status ssd_w4_matvec(const ssd_w4_matvec_args* a, ssd_stream_t stream) {
  using namespace ssd;
  if (!a || a->size != static_cast<int64_t>(sizeof(*a))) return SSD_ERR_INVALID_ARG;
  if (a->tokens < 0 || a->n <= 0 || a->k <= 0) return SSD_ERR_INVALID_ARG;
  if (!known_dtype(a->dtype) || (a->group != 32 && a->group != 64 && a->group != 128) || a->tokens > 65535)
    return SSD_ERR_UNSUPPORTED;
  if (a->k > (1 << 30)) return SSD_ERR_UNSUPPORTED;
  if (a->tokens == 0) return SSD_OK;
  const size_t es = elem_size(a->dtype);
  if (!a->x || !aligned_to(a->x, es) || !a->y || !aligned_to(a->y, es) || !aligned_to(a->add, es) || !a->packed ||
      !aligned_to(a->packed, 16) || !a->scales || !aligned_to(a->scales, 4))
    return SSD_ERR_INVALID_ARG;
  W4Params p{};
  p.M = static_cast<int>(a->tokens), p.x_token = a->x_token, p.add_token = a->add_token;
  p.n = a->n, p.k = a->k;
  p.ktiles = static_cast<int>(ceil_div(a->k, 64)), p.ngroups = static_cast<int>(ceil_div(a->k, a->group));
  p.x = a->x, p.packed = static_cast<const uint4*>(a->packed), p.scales = a->scales, p.add = a->add, p.y = a->y;
  return launched(a->dtype == SSD_BF16 ? launch_group<__nv_bfloat16>(p, a->group, stream)
                                       : launch_group<float>(p, a->group, stream));
}
