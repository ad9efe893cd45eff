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
// end.  The parts (and bf16 rows that are not 16-byte vectors) are laid out by a
// small launch in front, in the workspace; the product's launch overlaps it and
// has its first codes on their way before it waits for it.  A group's sum is
// scaled in 32 bits when its columns are done.
//
// A block takes 16 or 32 rows; its warps take pairs of column tiles in turn and
// their sums are joined in shared memory in a fixed order.  2560 -> 10576, one
// bf16 token: 6.2 us (2.3 TB/s; codes, then x and scales, then a join: latency, in
// 661 blocks of which 608 are resident); 5120 -> 2560, eight: 5.7 us; 8001 ->
// 16001, 16 fp32 tokens: 96 us.
#include "layer.cuh"

namespace ssd {
namespace {

// Warps of a block at most: two row tiles' sums take up to 255 registers a thread.
constexpr int max_warps(int tiles) { return tiles == 1 ? 16 : 8; }

struct W4Params {
  int64_t x_token, add_token;  // x_token: of the columns
  int M, n, k, ktiles, ngroups;
  const __nv_bfloat16* x;  // the product's columns: [tokens * parts][..], 16-byte rows
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

// The top 16 bits of a 32-bit number as a number; cut, not rounded, so that no part overflows.
__device__ __forceinline__ float cut(float v) { return __uint_as_float(__float_as_uint(v) & 0xFFFF0000u); }

// The product's columns of x [tokens][k]: zeros from k to the row's end; of a 32-bit x its three parts
// of 8 bits (24 in all).  An infinity or NaN is its own first part.
constexpr int kColumnThreads = 256;
__global__ void __launch_bounds__(kColumnThreads) columns_kernel(const __nv_bfloat16* x, int64_t x_token, int k, int row,
                                                                 __nv_bfloat16* out) {
  begin_kernel();  // (the product's launch reads weights before it waits, when all work before this is done)
  const int at = blockIdx.x * kColumnThreads + threadIdx.x;
  const int64_t m = blockIdx.y;
  if (at < row) out[m * row + at] = at < k ? x[m * x_token + at] : __float2bfloat16_rn(0.f);
}
__global__ void __launch_bounds__(kColumnThreads) columns_kernel(const float* x, int64_t x_token, int k, int row,
                                                                 __nv_bfloat16* out) {
  begin_kernel();  // (the product's launch reads weights before it waits, when all work before this is done)
  const int at = blockIdx.x * kColumnThreads + threadIdx.x;
  const int64_t m = blockIdx.y;
  if (at >= row) return;
  const float v = at < k ? x[m * x_token + at] : 0.f;
  const bool finite = fabsf(v) < INFINITY;
  const float hi = finite ? cut(v) : v, mid = finite ? cut(v - hi) : 0.f, lo = finite ? v - hi - mid : 0.f;
  out += 3 * m * row + at;
  out[0] = __float2bfloat16_rn(hi);
  out[row] = __float2bfloat16_rn(mid);
  out[2 * row] = __float2bfloat16_rn(lo);
}

// kCols: products' columns in blocks of 8.  kGroup: columns of weights a scale holds for.  kTiles: row tiles of a
// block, which share what is read of x.  kDirect: the columns are x itself; the launch in front may be writing x, the
// codes or the scales while this one is set up, so all is read after the wait.  Else that launch is columns_kernel,
// which lets this one start only when it has waited for all work before it: the codes may be read before the wait.
// Ordinary loads everywhere (the read-only path is not for what may be written meanwhile, and gains nothing: 6.2 and
// 5.7 us for the layer's two projections, 6.3 and 5.6 through it).
template <typename T, int kCols, int kTiles, int kGroup, bool kDirect>
__global__ void __launch_bounds__(max_warps(kTiles) * 32, kCols == 1 ? 2 : 1) w4_kernel(W4Params p) {
  constexpr int kParts = sizeof(T) == 4 ? 3 : 1;        // columns of a token
  constexpr int kTokens = kCols * 8 / kParts;           // tokens of a block (fp32: 2 in 8 columns)
  extern __shared__ float red[];                        // [warps][kTiles][kCols][4][32]
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int r = lane / 4, c = lane % 4;
  const int m0 = blockIdx.y * kTokens;
  if (kDirect) grid_dep_wait();
  grid_dep_launch();

  const __nv_bfloat16* x[kCols];
#pragma unroll
  for (int t = 0; t < kCols; ++t) {
    const int col = t * 8 + r;
    const bool in = col / kParts < kTokens && m0 + col / kParts < p.M;
    x[t] = in ? p.x + (static_cast<int64_t>(m0) * kParts + col) * p.x_token : nullptr;
  }
  const float *s0[kTiles], *s1[kTiles];
  const uint4* packed[kTiles];
#pragma unroll
  for (int j = 0; j < kTiles; ++j) {
    // rows past the matrix hold codes of 8 and any scale will do; tiles past it repeat the last
    const int tiles = (p.n + 15) / 16, tile = blockIdx.x * kTiles + j < tiles ? blockIdx.x * kTiles + j : tiles - 1;
    const int row = tile * 16 + r;
    s0[j] = p.scales + static_cast<int64_t>(row < p.n ? row : p.n - 1) * p.ngroups;
    s1[j] = p.scales + static_cast<int64_t>(row + 8 < p.n ? row + 8 : p.n - 1) * p.ngroups;
    packed[j] = p.packed + static_cast<int64_t>(tile) * p.ktiles * 32 + lane;
  }

  float total[kTiles][kCols][4] = {};
  // a warp's unit: two column tiles, 128 columns; its next kAhead units' codes are on their way together
  constexpr int kAhead = kCols == 1 ? 4 : 2;
  const int units = (p.ktiles + 1) / 2;
  bool waited = false;
  for (int base = warp; base < units; base += kAhead * warps) {
    uint4 q[kAhead][kTiles][2];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int j = 0; j < kTiles; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int kt = 2 * (base + u * warps) + h;
          q[u][j][h] = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);  // zeros past the end
          if (kt < p.ktiles) q[u][j][h] = packed[j][static_cast<int64_t>(kt) * 32];
        }
    if (!kDirect && !waited) grid_dep_wait();  // for the launch in front
    waited = true;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int unit = base + u * warps;
      if (unit >= units) break;
      float sum[kTiles][kCols][4] = {};
#pragma unroll
      for (int part4 = 0; part4 < 4; ++part4) {  // 32 columns: two products
        const int k0 = unit * 128 + part4 * 32 + c * 8;
        uint4 xw[kCols];
#pragma unroll
        for (int t = 0; t < kCols; ++t) {
          xw[t] = make_uint4(0, 0, 0, 0);
          if (x[t] && k0 < p.k) xw[t] = *reinterpret_cast<const uint4*>(x[t] + k0);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < kTiles; ++j) {
            const uint4& v = q[u][j][part4 / 2];
            const uint32_t w = part4 % 2 ? (i ? v.w : v.z) : (i ? v.y : v.x);
            const uint32_t a[4] = {codes<0>(w), codes<1>(w), codes<2>(w), codes<3>(w)};
#pragma unroll
            for (int t = 0; t < kCols; ++t) mma_bf16(sum[j][t], a, i ? xw[t].z : xw[t].x, i ? xw[t].w : xw[t].y);
          }
        constexpr int kParts32 = kGroup / 32;  // 32-column parts a scale holds for
        if (part4 % kParts32 == kParts32 - 1) {
          const int g = unit * (4 / kParts32) + part4 / kParts32;
#pragma unroll
          for (int j = 0; j < kTiles; ++j) {
            const float f0 = g < p.ngroups ? s0[j][g] : 0.f, f1 = g < p.ngroups ? s1[j][g] : 0.f;
#pragma unroll
            for (int t = 0; t < kCols; ++t) {
              total[j][t][0] = fmaf(f0, sum[j][t][0], total[j][t][0]);
              total[j][t][1] = fmaf(f0, sum[j][t][1], total[j][t][1]);
              total[j][t][2] = fmaf(f1, sum[j][t][2], total[j][t][2]);
              total[j][t][3] = fmaf(f1, sum[j][t][3], total[j][t][3]);
#pragma unroll
              for (int e = 0; e < 4; ++e) sum[j][t][e] = 0.f;
            }
          }
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kTiles; ++j)
#pragma unroll
    for (int t = 0; t < kCols; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[(((warp * kTiles + j) * kCols + t) * 4 + e) * 32 + lane] = total[j][t][e];
  __syncthreads();
  // (row i, token m) of the block: entry e = 2 (i % 16 / 8) + col % 2 of lane 4 (i % 8) + col % 8 / 2
  for (int at = threadIdx.x; at < 16 * kTiles * kTokens; at += blockDim.x) {
    const int i = at % (16 * kTiles), token = at / (16 * kTiles);
    const int n = blockIdx.x * 16 * kTiles + i, m = m0 + token;
    if (n >= p.n || m >= p.M) continue;
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < kParts; ++q) {
      const int col = token * kParts + q;
      const int e = 2 * (i % 16 / 8) + col % 2, from = 4 * (i % 8) + col % 8 / 2;
      float part_sum = 0.f;
      for (int w = 0; w < warps; ++w) part_sum += red[(((w * kTiles + i / 16) * kCols + col / 8) * 4 + e) * 32 + from];
      v += part_sum;
    }
    if (p.add) v += to_f32(static_cast<const T*>(p.add)[m * p.add_token + n]);
    static_cast<T*>(p.y)[static_cast<int64_t>(m) * p.n + n] = from_f32<T>(v);
  }
}

template <typename T, int kCols, int kTiles, int kGroup, bool kDirect>
cudaError_t launch_tiles(const W4Params& p, cudaStream_t stream) {
  constexpr int kTokens = kCols * 8 / (sizeof(T) == 4 ? 3 : 1);
  const int64_t units = ceil_div(p.ktiles, 2);
  const dim3 grid(static_cast<unsigned>(ceil_div(p.n, 16 * kTiles)), static_cast<unsigned>(ceil_div(p.M, kTokens)));
  // as many warps as give every multiprocessor kWarps, at least 4, and no more than there are units
  // (2560 -> 10576, one token, with 16, 24, 32, 48 and 64: 6.3, 6.3, 6.0, 6.9 and 7.5 us)
  constexpr int64_t kWarps = 32;
  int64_t warps = ceil_div(kWarps * layer_sm_count(), static_cast<int64_t>(grid.x) * grid.y);
  warps = warps < 4 ? 4 : warps > max_warps(kTiles) ? max_warps(kTiles) : warps;
  if (warps > units) warps = units;
  const size_t smem = static_cast<size_t>(warps) * kTiles * kCols * 4 * 32 * sizeof(float);  // at most 48 KB
  return launch_k(w4_kernel<T, kCols, kTiles, kGroup, kDirect>, grid, dim3(static_cast<unsigned>(warps) * 32), smem, stream,
                  true, p);
}

// From two blocks of columns on, x is more bytes than the codes for every row tile: two tiles share it
// where there are rows enough to fill the GPU all the same (8001 -> 16001, 16 fp32 tokens 156 -> 96 us,
// 16 bf16 tokens 47 -> 44).
template <typename T, int kCols, int kGroup, bool kDirect>
cudaError_t launch_cols(const W4Params& p, cudaStream_t stream) {
  if constexpr (kCols > 1) {
    if (ceil_div(p.n, 32) >= 2 * static_cast<int64_t>(layer_sm_count()))
      return launch_tiles<T, kCols, 2, kGroup, kDirect>(p, stream);
  }
  return launch_tiles<T, kCols, 1, kGroup, kDirect>(p, stream);
}

template <typename T, int kGroup, bool kDirect>
cudaError_t launch(const W4Params& p, cudaStream_t stream) {
  // the fewest blocks of eight columns that hold all tokens, up to 16 (fp32) or 32 (bf16): the codes are
  // then read once
  const int64_t columns = static_cast<int64_t>(p.M) * (sizeof(T) == 4 ? 3 : 1);
  if (columns <= 8) return launch_cols<T, 1, kGroup, kDirect>(p, stream);
  if (columns <= 16) return launch_cols<T, 2, kGroup, kDirect>(p, stream);
  if constexpr (sizeof(T) == 4) {
    if (columns > 32) return launch_cols<T, 6, kGroup, kDirect>(p, stream);
  }
  return launch_cols<T, 4, kGroup, kDirect>(p, stream);
}

template <typename T, bool kDirect>
cudaError_t launch_group(const W4Params& p, int group, cudaStream_t stream) {
  return group == 32   ? launch<T, 32, kDirect>(p, stream)
         : group == 64 ? launch<T, 64, kDirect>(p, stream)
                       : launch<T, 128, kDirect>(p, stream);
}

// x laid out as columns in the workspace, then the product.
template <typename T>
cudaError_t launch_columns(W4Params p, const ssd_w4_matvec_args* a, cudaStream_t stream) {
  const int row = p.ktiles * 64;
  const dim3 grid(static_cast<unsigned>(ceil_div(row, kColumnThreads)), static_cast<unsigned>(p.M));
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a->workspace);
  void (*k)(const T*, int64_t, int, int, __nv_bfloat16*) = columns_kernel;
  const cudaError_t e =
      launch_k(k, grid, dim3(kColumnThreads), 0, stream, true, static_cast<const T*>(a->x), a->x_token, p.k, row, out);
  if (e != cudaSuccess) return e;
  p.x = out, p.x_token = row, p.k = row;
  return launch_group<T, false>(p, a->group, stream);
}

ssd_status check_sizes(const ssd_w4_matvec_args* a) {
  if (!a || a->size != static_cast<int64_t>(sizeof(*a))) return SSD_ERR_INVALID_ARG;
  if (a->tokens < 0 || a->n <= 0 || a->k <= 0) return SSD_ERR_INVALID_ARG;
  if (!known_dtype(a->dtype) || (a->group != 32 && a->group != 64 && a->group != 128) || a->tokens > 65535)
    return SSD_ERR_UNSUPPORTED;
  return a->k > (1 << 30) || a->n > (1 << 30) ? SSD_ERR_UNSUPPORTED : SSD_OK;
}

// Whether x has to be laid out as columns first: 32-bit values, or rows that are not 16-byte vectors.
bool needs_columns(const ssd_w4_matvec_args* a) {
  return a->dtype == SSD_F32 || a->k % 8 != 0 || !aligned_to(a->x, 16) || a->x_token % 8 != 0;
}

}  // namespace
}  // namespace ssd

extern "C" size_t ssd_w4_matvec_workspace_size(const ssd_w4_matvec_args* a) {
  using namespace ssd;
  if (check_sizes(a) != SSD_OK || !needs_columns(a)) return 0;
  return static_cast<size_t>(a->tokens) * (a->dtype == SSD_F32 ? 3 : 1) * ceil_div(a->k, 64) * 64 * 2;
}

extern "C" ssd_status ssd_w4_matvec(const ssd_w4_matvec_args* a, ssd_stream_t stream) {
  using namespace ssd;
  const ssd_status st = check_sizes(a);
  if (st != SSD_OK) return st;
  if (a->tokens == 0) return SSD_OK;
  const size_t es = elem_size(a->dtype);
  if (!a->x || !aligned_to(a->x, es) || !a->y || !aligned_to(a->y, es) || !aligned_to(a->add, es) || !a->packed ||
      !aligned_to(a->packed, 16) || !a->scales || !aligned_to(a->scales, 4))
    return SSD_ERR_INVALID_ARG;
  const bool columns = needs_columns(a);
  if (columns) {
    if (!a->workspace || !aligned_to(a->workspace, 16)) return SSD_ERR_INVALID_ARG;
    if (a->workspace_bytes < ssd_w4_matvec_workspace_size(a)) return SSD_ERR_WORKSPACE;
  }
  W4Params p{};
  p.M = static_cast<int>(a->tokens), p.add_token = a->add_token;
  p.n = a->n, p.k = a->k;
  p.ktiles = static_cast<int>(ceil_div(a->k, 64)), p.ngroups = static_cast<int>(ceil_div(a->k, a->group));
  p.packed = static_cast<const uint4*>(a->packed), p.scales = a->scales, p.add = a->add, p.y = a->y;
  if (a->dtype == SSD_F32) return launched(launch_columns<float>(p, a, stream));
  if (columns) return launched(launch_columns<__nv_bfloat16>(p, a, stream));
  p.x = static_cast<const __nv_bfloat16*>(a->x), p.x_token = a->x_token;
  return launched(launch_group<__nv_bfloat16, true>(p, a->group, stream));
}
