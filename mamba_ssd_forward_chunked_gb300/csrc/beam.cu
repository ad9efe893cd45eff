// Beam search: the k best of beams x vocab candidates, and the reordering of
// the states that the choice decides.
//
// Selection reads the logits once.  Within a beam the score s + (x - lse) never
// falls as the logit x rises, so a block that reads a piece of a row can name its
// best by logit before the row's log-sum-exp is known: it writes the k + 1 best
// and the piece's maximum and sum of exponentials.  A second launch joins the
// sums in a fixed order and picks the k best scores of a request among its
// pieces' candidates.  32 x 8 x 131072 bf16: the pieces 33 us (HBM 10; the
// ranking's instructions and barriers fill the issue slots), the join 8 (one
// block a request: latency); 4 x 32768 fp32, both 6 us.
//
// A key holds a value in the order of unsigned integers and the complement of
// the candidate's index, so keys differ and equal values fall by rising index.
// The n best of a block: every group of four (or two) threads has a largest key;
// no key below the n-th largest of those can be among the n best, few keys reach
// it, and those are ranked by counting.
//
// Rounding can give different logits of a beam one score, and then the lower
// index goes first although its logit is smaller.  Such a candidate may be
// missing from its piece's list, but only if the piece's (k + 1)-th still has
// the k-th best score (or, where that is -infinity, lists finite logits with
// this score); then the second launch looks through the pieces that reach this
// score once more, in the order of indexes.
//
// Reordering moves bytes: a thread owns 16 bytes' position in all rows of a
// request, reads them all, then writes, so that it may work in place.  256 rows
// of 268 KB: 14 us.
#include "layer.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxBeams = 64;
constexpr int kMaxGroups = 128;
constexpr int kMergeKeys = 1024;  // candidates the second launch ranks at once
using Key = unsigned long long;

struct SelectParams {
  int64_t logits_batch, logits_beam;
  int beams, vocab, k, eos, pieces, keep;  // keep: keys of a piece, k + 1
  const void* logits;
  const float* scores;
  const uint8_t* finished;
  float* out_scores;
  int32_t *parents, *tokens;
  Key* keys;      // [batch][beams][pieces][keep]: best logits of a piece, 0 where it has fewer
  float2* sums;   // [batch][beams][pieces]: (maximum, sum of exp(x - maximum))
};

// Values in the order of unsigned integers; -0 and +0 are one value, and a NaN counts as -infinity.
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t b = __float_as_uint(v == v ? v + 0.f : -INFINITY);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ Key key_of(float v, uint32_t index) {
  return (static_cast<Key>(order_of(v)) << 32) | static_cast<uint32_t>(~index);
}
__device__ __forceinline__ float key_value(Key k) { return value_of(static_cast<uint32_t>(k >> 32)); }
__device__ __forceinline__ uint32_t key_index(Key k) { return ~static_cast<uint32_t>(k); }

// A candidate's score; a NaN counts as -infinity.
__device__ __forceinline__ float score_of(float beam, float x, float lse) {
  const float s = beam + (x - lse);
  return s == s ? s : -INFINITY;
}

// Threads that share a group where the n best are wanted: at least n groups.
__host__ __device__ constexpr int share_of(int n) { return 4 * n <= kThreads ? 4 : 2; }

// The n-th largest of the block's groups' largest keys: no smaller key is among the n best.  0 where
// fewer than n groups have any.
__device__ __forceinline__ Key bound_of(Key mine, int n, Key (&s_group)[kMaxGroups], Key& s_bound) {
  const int share = share_of(n), groups = kThreads / share;
  for (int o = 1; o < share; o *= 2) {
    const Key other = __shfl_xor_sync(0xffffffffu, mine, o);
    mine = other > mine ? other : mine;
  }
  if (threadIdx.x % share == 0) s_group[threadIdx.x / share] = mine;
  if (threadIdx.x == 0) s_bound = 0;
  __syncthreads();
  {  // each thread counts a share of the groups that are above its own
    const int part = threadIdx.x % share;
    int rank = 0;
#pragma unroll 8
    for (int i = part; i < groups; i += share) rank += s_group[i] > mine;
    for (int o = 1; o < share; o *= 2) rank += __shfl_xor_sync(0xffffffffu, rank, o);
    if (part == 0 && rank == n - 1 && mine) s_bound = mine;  // keys differ: one group at most
  }
  __syncthreads();
  return s_bound;
}

// Writes the k largest of the n different keys in order (0 where there are fewer).
__device__ __forceinline__ void rank_keys(const Key* keys, int n, int k, Key* out) {
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const Key key = keys[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += keys[j] > key;
    if (rank < k) out[rank] = key;
  }
  for (int i = n + threadIdx.x; i < k; i += kThreads) out[i] = 0;
}

// Eight consecutive logits (16 or 32 bytes) as they lie in memory.
template <typename T>
struct Eight;
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p), b = *(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ float get(int i) const { return (i < 4 ? &a.x : &b.x)[i % 4]; }
};
template <>
struct Eight<__nv_bfloat16> {
  uint4 q;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { q = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t w = (&q.x)[i / 2];
    return __uint_as_float(i % 2 ? w & 0xFFFF0000u : w << 16);
  }
};

// One piece of a row: kEights times eight logits a thread.  They are read once; of each eight a
// thread keeps the maximum, and the few eights that reach the bound are read again, from cache.
// kVec: rows are 16-byte aligned.
template <typename T, int kEights, bool kVec>
__global__ void __launch_bounds__(kThreads) piece_kernel(SelectParams p) {
  extern __shared__ __align__(16) unsigned char raw[];
  Key* s_keys = reinterpret_cast<Key*>(raw);
  __shared__ Key s_group[kMaxGroups], s_bound;
  __shared__ float s_red[2][kThreads / 32];
  __shared__ int s_count;
  begin_kernel();
  const int piece = blockIdx.x, w = blockIdx.y, tid = threadIdx.x;
  const int64_t b = blockIdx.z, row = b * p.beams + w;
  const int v0 = piece * kThreads * 8 * kEights;
  if (tid == 0) s_count = 0;

  // element i of the thread's eight g: its index rises with g and i
  auto at = [&](int g, int i) { return v0 + g * (8 * kThreads) + (kVec ? 8 * tid + i : kThreads * i + tid); };
  const T* src = static_cast<const T*>(p.logits) + b * p.logits_batch + w * p.logits_beam;
  const bool done = p.finished && p.finished[row];
  const bool whole = kVec && p.vocab - v0 >= kThreads * 8 * kEights, plain = whole && !done;
  auto read = [&](int g, float (&v)[8]) {
    if (plain) {
      Eight<T> x;
      x.load(src + at(g, 0));
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = x.get(i);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = -INFINITY;  // past the row's end; adds nothing
        // a finished beam's one candidate, at the beam's score: logits of 0 and -infinity, whose
        // log-sum-exp is 0
        if (done) v[i] = at(g, i) == p.eos ? 0.f : -INFINITY;
        else if (at(g, i) < p.vocab) v[i] = to_f32(src[at(g, i)]);
      }
    }
  };

  // maximum and sum of exponentials, the sum for the thread's maximum so far
  float top8[kEights], top = -INFINITY, sum = 0.f;
  auto add = [&](int g, const float (&v)[8]) {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) m = fmaxf(m, v[i]);
    top8[g] = m;
    const float before = top;
    top = fmaxf(top, m);
    const float shift = top > -INFINITY ? top : 0.f;  // nothing but -infinity sums to 0
    const uint64_t minus2 = pack2(-shift, -shift), scale2 = pack2(kLog2e, kLog2e);
    uint64_t sum2 = pack2(sum * exp2_fast((before - shift) * kLog2e), 0.f);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      float lo, hi;
      unpack2(mul2(add2(pack2(v[i], v[i + 1]), minus2), scale2), lo, hi);
      sum2 = add2(sum2, pack2(exp2_fast(lo), exp2_fast(hi)));
    }
    float hi;
    unpack2(sum2, sum, hi);
    sum += hi;
  };
  Eight<T> x[kEights];
  if (whole) {  // (a finished beam's logits too: whether it is finished is not known yet)
#pragma unroll
    for (int g = 0; g < kEights; ++g) x[g].load(src + at(g, 0));
  }
  if (plain) {
#pragma unroll
    for (int g = 0; g < kEights; ++g) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = x[g].get(i);
      add(g, v);
    }
  } else {
#pragma unroll
    for (int g = 0; g < kEights; ++g) {
      float v[8];
      read(g, v);
      add(g, v);
    }
  }

  // The thread's largest key or a little less: the index is that of the last of the eight that hold
  // the first of its largest logits, so `keep` keys reach the bound all the same (more, with ties).
  int best = kEights - 1;  // the first eight that hold the largest logit
#pragma unroll
  for (int g = kEights - 1; g >= 0; --g) best = top8[g] == top ? g : best;
  Key mine = 0;
  if (at(0, 0) < p.vocab) mine = key_of(top, static_cast<uint32_t>(at(best, 7)));
  float piece_top = top;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) piece_top = fmaxf(piece_top, __shfl_xor_sync(0xffffffffu, piece_top, o));
  if (tid % 32 == 0) s_red[0][tid / 32] = piece_top;

  // The keys from the bound up.  Where the groups' keys are exact they lie in `keep` groups at most,
  // for which there is room; with ties the first round may overrun it, and a second takes exact keys.
  const int room = p.keep * share_of(p.keep) * 8 * kEights;
#pragma unroll 1
  for (int round = 0;; ++round) {
    const Key bound = bound_of(mine, p.keep, s_group, s_bound);
    const float least = key_value(bound);
    unsigned hits = 0;
#pragma unroll
    for (int g = 0; g < kEights; ++g)
      if (!bound || !(top8[g] < least)) hits |= 1u << g;  // (NaN go on, as -infinity)
    for (; hits; hits &= hits - 1) {
      if (*static_cast<volatile int*>(&s_count) > room) break;
      const int g = __ffs(static_cast<int>(hits)) - 1;
      float v[8];
      read(g, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if ((bound && v[i] < least) || at(g, i) >= p.vocab) continue;
        const Key key = key_of(v[i], static_cast<uint32_t>(at(g, i)));
        if (key < bound) continue;
        const int n = atomicAdd(&s_count, 1);
        if (n < room) s_keys[n] = key;
      }
    }
    __syncthreads();
    if (s_count <= room || round == 1) break;
    // (a NaN counts as -infinity and is in no maximum, so a thread without more starts at its first)
    mine = 0;
    for (int g = top > -INFINITY ? best : 0; g < kEights; ++g) {
      float v[8];
      read(g, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const Key key = at(g, i) < p.vocab ? key_of(v[i], static_cast<uint32_t>(at(g, i))) : 0;
        mine = key > mine ? key : mine;
      }
      if (mine) break;
    }
    __syncthreads();
    if (tid == 0) s_count = 0;
  }

#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) piece_top = fmaxf(piece_top, s_red[0][i]);
  if (top > -INFINITY) sum *= exp2_fast((top - piece_top) * kLog2e);  // (else it is 0, or lost)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (tid % 32 == 0) s_red[1][tid / 32] = sum;
  __syncthreads();
  rank_keys(s_keys, s_count < room ? s_count : room, p.keep, p.keys + (row * p.pieces + piece) * p.keep);
  if (tid == 0) {
    sum = 0.f;
    for (int i = 0; i < kThreads / 32; ++i) sum += s_red[1][i];
    p.sums[row * p.pieces + piece] = make_float2(piece_top, sum);
  }
}

// The k best of a request's candidates.
template <typename T>
__global__ void __launch_bounds__(kThreads) merge_kernel(SelectParams p, int piece_size) {
  __shared__ Key s_keys[kMergeKeys], s_best[kMaxBeams], s_group[kMaxGroups], s_bound;
  __shared__ float s_lse[kMaxBeams], s_score[kMaxBeams];
  __shared__ int s_count;
  begin_kernel();
  const int64_t b = blockIdx.x;
  const int tid = threadIdx.x, lane = tid % 32;
  const float2* sums = p.sums + b * p.beams * p.pieces;
  const int per = p.pieces * p.keep, all = p.beams * per;
  const Key* keys = p.keys + b * all;
  // As a rule a thread's candidates fit registers: they are on their way before the sums are joined,
  // and read once.
  constexpr int kOwn = 4;
  const bool few = all <= kOwn * kThreads;
  Key own[kOwn];
#pragma unroll
  for (int q = 0; q < kOwn; ++q) own[q] = few && tid + q * kThreads < all ? keys[tid + q * kThreads] : 0;
  for (int w = tid / 32; w < p.beams; w += kThreads / 32) {  // a warp a beam
    float top = -INFINITY, sum = 0.f;
    for (int i = lane; i < p.pieces; i += 32) top = fmaxf(top, sums[w * p.pieces + i].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    for (int i = lane; i < p.pieces; i += 32) {
      const float2 v = sums[w * p.pieces + i];
      sum += v.x > -INFINITY || v.y != v.y ? v.y * expf(v.x - top) : 0.f;  // a NaN in the sum stays
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
      s_lse[w] = top + logf(sum);
      s_score[w] = p.scores[b * p.beams + w];
    }
  }
  if (tid == 0) s_count = 0;
  __syncthreads();

  // of a piece's key (logit, index in the row): the candidate's (score, index in the request)
  auto candidate = [&](int i, Key key) -> Key {
    if (!key) return 0;
    const int w = i / per;
    return key_of(score_of(s_score[w], key_value(key), s_lse[w]), static_cast<uint32_t>(w) * p.vocab + key_index(key));
  };
  Key mine = 0, scored[kOwn];
#pragma unroll
  for (int q = 0; q < kOwn; ++q) {
    scored[q] = candidate(tid + q * kThreads, own[q]);
    mine = scored[q] > mine ? scored[q] : mine;
  }
  for (int i = tid; !few && i < all; i += kThreads) {
    const Key key = candidate(i, keys[i]);
    mine = key > mine ? key : mine;
  }
  const Key bound = bound_of(mine, p.k, s_group, s_bound);
  auto collect = [&](Key key) {
    if (key && key >= bound) {
      const int n = atomicAdd(&s_count, 1);
      if (n < kMergeKeys) s_keys[n] = key;
    }
  };
#pragma unroll
  for (int q = 0; q < kOwn; ++q) collect(scored[q]);
  for (int i = tid; !few && i < all; i += kThreads) collect(candidate(i, keys[i]));
  __syncthreads();
  if (s_count <= kMergeKeys) {
    rank_keys(s_keys, s_count, p.k, s_best);
    __syncthreads();
  } else {
    // too many reach the bound (as with rows of equal logits and a large k): k rounds over them
    Key last = ~0ull;
    for (int i = 0; i < p.k; ++i) {
      mine = 0;
      for (int j = tid; j < all; j += kThreads) {
        const Key key = candidate(j, keys[j]);
        if (key < last && key > mine) mine = key;
      }
      last = bound_of(mine, 1, s_group, s_bound);
      if (tid == 0) s_best[i] = last;
      __syncthreads();
    }
  }

  // equal scores below a piece's list
  const uint32_t worst = static_cast<uint32_t>(s_best[p.k - 1] >> 32);
  bool hidden = false;
  auto at_worst = [&](int w, Key key) { return order_of(score_of(s_score[w], key_value(key), s_lse[w])) == worst; };
  auto hides = [&](int i, int w, Key key) {  // a piece's last key, the i-th of all: whether candidates at the k-th
    if (!key || !at_worst(w, key)) return false;  // score, at lower indexes than some of the piece's, lie behind it
    if (key_value(key) > -INFINITY) return true;
    // Behind a last key of -infinity there are logits of -infinity alone, at higher indexes than the listed ones.
    // The lowest logit above -infinity that is listed may lie higher still: in a lost beam its score is the same.
    for (int j = 1; j <= p.k; ++j)
      if (key_value(keys[i - j]) > -INFINITY) return at_worst(w, keys[i - j]);
    return false;
  };
#pragma unroll
  for (int q = 0; q < kOwn; ++q) {
    const int i = tid + q * kThreads;
    if (own[q] && i % p.keep == p.k && hides(i, i / per, own[q])) hidden = true;
  }
  for (int i = p.k + tid * p.keep; !few && i < all; i += kThreads * p.keep)
    if (hides(i, i / per, keys[i])) hidden = true;
  if (__syncthreads_or(hidden)) {
    int found = 0;  // the candidates above the k-th score stay; those at it are gathered by rising index
    while (static_cast<uint32_t>(s_best[found] >> 32) != worst) ++found;
    for (int i = 0; i < p.beams * p.pieces && found < p.k; ++i) {
      const int w = i / p.pieces, piece = i % p.pieces;
      const bool done = p.finished && p.finished[b * p.beams + w];
      if (order_of(score_of(s_score[w], sums[i].x, s_lse[w])) < worst) continue;  // (a NaN is in no maximum)
      const T* src = static_cast<const T*>(p.logits) + b * p.logits_batch + w * p.logits_beam;
      const int stop = p.vocab - piece * piece_size < piece_size ? p.vocab : (piece + 1) * piece_size;
      for (int v0 = piece * piece_size; v0 < stop && found < p.k; v0 += kThreads) {
        const int v = v0 + tid;
        bool hit = false;
        if (v < stop) {
          const float x = done ? (v == p.eos ? 0.f : -INFINITY) : to_f32(src[v]);
          hit = order_of(score_of(s_score[w], x, s_lse[w])) == worst;
        }
        const unsigned votes = __ballot_sync(0xffffffffu, hit);
        if (lane == 0) s_group[tid / 32] = __popc(votes);
        __syncthreads();
        int before = found, total = 0;
        for (int j = 0; j < kThreads / 32; ++j) {
          if (j < tid / 32) before += static_cast<int>(s_group[j]);
          total += static_cast<int>(s_group[j]);
        }
        before += __popc(votes & ((1u << lane) - 1u));
        if (hit && before < p.k)
          s_best[before] = (static_cast<Key>(worst) << 32) |
                           static_cast<uint32_t>(~(static_cast<uint32_t>(w) * p.vocab + v));
        found += total;
        __syncthreads();
      }
    }
    __syncthreads();
  }
  if (tid < p.k) {
    const Key key = s_best[tid];
    p.out_scores[b * p.k + tid] = key_value(key);
    p.parents[b * p.k + tid] = static_cast<int32_t>(key_index(key) / p.vocab);
    p.tokens[b * p.k + tid] = static_cast<int32_t>(key_index(key) % p.vocab);
  }
}

// Times eight logits that a thread reads: eight, or one where that would leave fewer than four pieces a
// multiprocessor.
int eights_of(int64_t batch, int beams, int vocab) {
  return batch * beams * ceil_div(vocab, 64 * kThreads) >= 4 * static_cast<int64_t>(layer_sm_count()) ? 8 : 1;
}

// Bytes of a piece's list of keys.
constexpr size_t list_bytes(int keep, int eights) {
  return static_cast<size_t>(keep) * share_of(keep) * 8 * eights * sizeof(Key);
}
// The most that any k takes: four threads share a group up to the largest `keep` but one.
constexpr size_t most_list_bytes(int eights) {
  static_assert(share_of(kMaxBeams) == 4 && share_of(kMaxBeams + 1) == 2, "keep is at most kMaxBeams + 1");
  return list_bytes(kMaxBeams, eights);
}

template <typename T, int kEights>
cudaError_t launch_pieces(const SelectParams& p, bool vec, int64_t batch, cudaStream_t stream) {
  const size_t smem = list_bytes(p.keep, kEights);
  auto k = vec ? piece_kernel<T, kEights, true> : piece_kernel<T, kEights, false>;
  if (smem > 40 * 1024) {
    // one limit whatever k is: it belongs to the kernel, and other threads' launches go by it too
    const cudaError_t e =
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most_list_bytes(kEights)));
    if (e != cudaSuccess) return e;
  }
  const dim3 grid(static_cast<unsigned>(p.pieces), static_cast<unsigned>(p.beams), static_cast<unsigned>(batch));
  return launch_k(k, grid, dim3(kThreads), smem, stream, true, p);
}

template <typename T>
cudaError_t launch_select(const SelectParams& p, int64_t batch, cudaStream_t stream) {
  const int64_t es = sizeof(T);
  const bool vec = aligned_to(p.logits, 16) && p.logits_beam * es % 16 == 0 && p.logits_batch * es % 16 == 0;
  const int eights = eights_of(batch, p.beams, p.vocab);
  const cudaError_t e = eights == 8 ? launch_pieces<T, 8>(p, vec, batch, stream) : launch_pieces<T, 1>(p, vec, batch, stream);
  if (e != cudaSuccess) return e;
  return launch_k(merge_kernel<T>, dim3(static_cast<unsigned>(batch)), dim3(kThreads), 0, stream, true, p,
                  eights * 8 * kThreads);
}

struct ReorderParams {
  int beams, k, count;
  const int32_t* parents;
  const void* src[SSD_REORDER_MAX];
  void* dst[SSD_REORDER_MAX];
  int64_t row_bytes[SSD_REORDER_MAX];
};

// kK: an upper limit of the rows of a request.
template <typename V, int kK>
__global__ void __launch_bounds__(kThreads) reorder_kernel(ReorderParams p) {
  __shared__ int s_parent[kK];
  begin_kernel();
  const int j = blockIdx.z;
  const int64_t b = blockIdx.y;
  const int64_t units = p.row_bytes[j] / static_cast<int64_t>(sizeof(V));
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const bool in_place = p.src[j] == p.dst[j];
  if (threadIdx.x < p.k) {
    const int from = p.parents[b * p.k + threadIdx.x];
    s_parent[threadIdx.x] = from < 0 || from >= p.beams || (in_place && from == static_cast<int>(threadIdx.x)) ? -1 : from;
  }
  __syncthreads();
  if (at >= units) return;
  const V* src = static_cast<const V*>(p.src[j]) + b * p.beams * units + at;
  V* dst = static_cast<V*>(p.dst[j]) + b * p.k * units + at;
  V v[kK];
#pragma unroll
  for (int i = 0; i < kK; ++i)
    if (i < p.k && s_parent[i] >= 0) v[i] = src[s_parent[i] * units];
#pragma unroll
  for (int i = 0; i < kK; ++i)
    if (i < p.k && s_parent[i] >= 0) dst[i * units] = v[i];
}

// One launch for all tensors that move in units of V.
template <typename V>
cudaError_t launch_reorder(const ReorderParams& all, int unit, int64_t batch, cudaStream_t stream) {
  ReorderParams p = all;
  int64_t most = 0;
  p.count = 0;
  for (int j = 0; j < all.count; ++j) {
    const uintptr_t bits = reinterpret_cast<uintptr_t>(all.src[j]) | reinterpret_cast<uintptr_t>(all.dst[j]) |
                           static_cast<uintptr_t>(all.row_bytes[j]);
    if (all.row_bytes[j] == 0 || ((bits & 15) == 0 ? 16 : (bits & 3) == 0 ? 4 : 1) != unit) continue;
    p.src[p.count] = all.src[j], p.dst[p.count] = all.dst[j], p.row_bytes[p.count] = all.row_bytes[j];
    ++p.count;
    if (all.row_bytes[j] / unit > most) most = all.row_bytes[j] / unit;
  }
  if (p.count == 0) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>(ceil_div(most, kThreads)), static_cast<unsigned>(batch),
                  static_cast<unsigned>(p.count));
  auto k = p.k <= 4 ? reorder_kernel<V, 4> : p.k <= 8 ? reorder_kernel<V, 8> : p.k <= 16 ? reorder_kernel<V, 16>
                                                                                         : reorder_kernel<V, 64>;
  return launch_k(k, grid, dim3(kThreads), 0, stream, true, p);
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
  using namespace ssd;
  if (check_select(a) != SSD_OK) return 0;
  const size_t pieces = ceil_div(a->vocab, eights_of(a->batch, a->beams, a->vocab) * 8 * kThreads);
  return static_cast<size_t>(a->batch) * a->beams * pieces * ((a->k + 1) * sizeof(Key) + sizeof(float2));
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
  p.pieces = static_cast<int>(ceil_div(p.vocab, eights_of(a->batch, p.beams, p.vocab) * 8 * kThreads));
  p.keep = p.k + 1;
  p.keys = static_cast<Key*>(a->workspace);
  p.sums = reinterpret_cast<float2*>(p.keys + a->batch * p.beams * p.pieces * p.keep);
  return launched(a->dtype == SSD_BF16 ? launch_select<__nv_bfloat16>(p, a->batch, stream)
                                       : launch_select<float>(p, a->batch, stream));
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
  cudaError_t e = launch_reorder<uint4>(p, 16, a->batch, stream);
  if (e == cudaSuccess) e = launch_reorder<uint32_t>(p, 4, a->batch, stream);
  if (e == cudaSuccess) e = launch_reorder<uint8_t>(p, 1, a->batch, stream);
  return launched(e);
}
