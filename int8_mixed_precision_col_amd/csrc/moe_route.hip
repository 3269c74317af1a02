// Routing of any number of tokens, and the way back from the experts' rows to tokens.
//
// Routing: for token t the top_k experts of the largest logits (ties to the lowest index, -inf is
// off) with their softmax weights, as in moe.hip, and the T k (token, place) pairs ordered by
// expert and then token: row p of that order is token rows[p]; expert e has the rows offsets[e]
// up to offsets[e + 1]; the pair (t, j) is row slots[t, j]. A token chooses an expert at most once,
// so a pair's row is offsets[e] + the number of earlier tokens that chose e: counts of the
// tokens before its workgroup's (kept by the first launch), of those before its 64, and the
// bits below its own in the mask of those 64. No atomics decide an order.
#include "group_launch.hpp"
#include "moe_keys.hpp"
#include "mx4.hpp"

namespace i8mm {

constexpr int kRouteWaves = 16, kRouteThreads = 64 * kRouteWaves;
constexpr int kRouteChunk = 64;      // tokens of a workgroup at a time: the bits of a mask
constexpr int kRouteMaxBlocks = 256;
constexpr int kRouteTokens = kRouteChunk / kRouteWaves;  // of a wave at a time

// Chunks of 64 tokens per workgroup, and workgroups.
static void route_geometry(int64_t T, int* chunks, int* blocks) {
  const int64_t all = (T + kRouteChunk - 1) / kRouteChunk;
  *chunks = static_cast<int>((all + kRouteMaxBlocks - 1) / kRouteMaxBlocks);
  *blocks = static_cast<int>((all + *chunks - 1) / *chunks);
}

// The wave's tokens of a chunk, side by side (a token's rounds are one chain of dependent steps).
// Lane l holds experts V l .. V l + V - 1, so that the lowest lane and then the lowest of its
// experts is the lowest index. Lane j leaves with place j's expert (-1: none).
template <int V>
__device__ __forceinline__ void route_tokens(const RouteArgs& a, int t0, int lane, int (&id)[kRouteTokens]) {
  unsigned key[kRouteTokens][V], first[kRouteTokens], mine[kRouteTokens];
  float all[kRouteTokens];
#pragma unroll
  for (int p = 0; p < kRouteTokens; ++p) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = V * lane + i;
      key[p][i] = t0 + p < a.T && e < a.E
                      ? moe_key(moe_logit(a.logits, a.logits_type, static_cast<int64_t>(t0 + p) * a.E + e))
                      : 0u;
    }
  }
#pragma unroll
  for (int p = 0; p < kRouteTokens; ++p) {
    unsigned best = key[p][0];
#pragma unroll
    for (int i = 1; i < V; ++i) best = max(best, key[p][i]);
    first[p] = wave_max_u32(best);
    mine[p] = 0;
    id[p] = -1;
    all[p] = 0.0f;
    if (!a.renormalize) {
      const float most = moe_unkey(first[p]);
#pragma unroll
      for (int i = 0; i < V; ++i) all[p] += key[p][i] ? expf(moe_unkey(key[p][i]) - most) : 0.0f;
    }
  }
  for (int j = 0; j < a.k; ++j) {
#pragma unroll
    for (int p = 0; p < kRouteTokens; ++p) {
      unsigned best = key[p][0];
      int at = 0;
#pragma unroll
      for (int i = 1; i < V; ++i)
        if (key[p][i] > best) {
          best = key[p][i];
          at = i;
        }
      const unsigned top = wave_max_u32(best);  // 0: no expert left
      const int who = __builtin_ctzll(__ballot(best == top));
      const int e = V * who + (V > 1 ? __builtin_amdgcn_readlane(at, who) : 0);
      if (lane == j && top) {
        mine[p] = top;
        id[p] = e;
      }
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (V * lane + i == e) key[p][i] = 0u;
    }
  }
#pragma unroll
  for (int p = 0; p < kRouteTokens; ++p) {
    const float w = mine[p] ? expf(moe_unkey(mine[p]) - moe_unkey(first[p])) : 0.0f;
    float sum = a.renormalize ? w : all[p];
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
    if (lane < a.k && t0 + p < a.T) {
      const int64_t o = static_cast<int64_t>(t0 + p) * a.k + lane;
      a.ids[o] = id[p];
      a.weights[o] = id[p] < 0 ? 0.0f : __fdiv_rn(w, sum);
    }
  }
}

// Exclusive prefix sum of n <= kMoeMaxExperts + 1 counts in LDS, in place of thread i's count;
// returns it, with the sum of all in `total`. All threads of the workgroup take part.
__device__ __forceinline__ int block_exclusive(int v, int tid, int* wave_sums, int& total) {
  int upto = wave_prefix_sum(v);
  if ((tid & 63) == 63) wave_sums[tid >> 6] = upto;
  __syncthreads();
  total = 0;
  for (int w = 0; w < kRouteWaves; ++w) {
    if (w < tid >> 6) upto += wave_sums[w];
    total += wave_sums[w];
  }
  return upto - v;
}

// The rows of a chunk's pairs: `base` [E] is the next row of each expert; on return it is past
// the chunk's. ids: this wave's tokens of the chunk, place `lane` of each.
struct RouteMasks {
  unsigned bits[kMoeMaxExperts][2];
  int base[kMoeMaxExperts];
};
__device__ __forceinline__ void place_chunk(const RouteArgs& a, int chunk0, const int (&id)[kRouteTokens], RouteMasks& m,
                                            int tid, int lane, int wave) {
  for (int e = tid; e < a.E; e += kRouteThreads) m.bits[e][0] = m.bits[e][1] = 0u;
  __syncthreads();
  const int in0 = wave * kRouteTokens;
#pragma unroll
  for (int p = 0; p < kRouteTokens; ++p)
    if (id[p] >= 0) atomicOr(&m.bits[id[p]][(in0 + p) >> 5], 1u << ((in0 + p) & 31));
  __syncthreads();
#pragma unroll
  for (int p = 0; p < kRouteTokens; ++p) {
    const int t = chunk0 + in0 + p;
    if (lane >= a.k || t >= a.T) continue;
    int row = -1;
    if (id[p] >= 0) {
      const int b = in0 + p;
      const unsigned lo = m.bits[id[p]][0], hi = m.bits[id[p]][1];
      const unsigned below = (1u << (b & 31)) - 1u;
      row = m.base[id[p]] + (b < 32 ? __builtin_popcount(lo & below) : __builtin_popcount(lo) + __builtin_popcount(hi & below));
      a.rows[row] = t;
    }
    a.slots[static_cast<int64_t>(t) * a.k + lane] = row;
  }
  __syncthreads();
  for (int e = tid; e < a.E; e += kRouteThreads)
    m.base[e] += __builtin_popcount(m.bits[e][0]) + __builtin_popcount(m.bits[e][1]);
}

// First launch: the chosen experts of every token, and how many tokens of the workgroup chose each
// expert. With one workgroup of one chunk (ONE) the rows too.
template <int V, bool ONE>
__global__ __launch_bounds__(kRouteThreads) void k_route(RouteArgs a, int chunks) {
  __shared__ int count[kMoeMaxExperts];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  for (int e = tid; e < a.E; e += kRouteThreads) count[e] = 0;
  __syncthreads();
  int id[kRouteTokens];
  for (int c = 0; c < (ONE ? 1 : chunks); ++c) {
    const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * chunks + c) * kRouteChunk + wave * kRouteTokens;
    if (t0 >= a.T) {
#pragma unroll
      for (int p = 0; p < kRouteTokens; ++p) id[p] = -1;
      break;
    }
    route_tokens<V>(a, static_cast<int>(t0), lane, id);
#pragma unroll
    for (int p = 0; p < kRouteTokens; ++p)
      if (id[p] >= 0) atomicAdd(&count[id[p]], 1);
  }
  __syncthreads();
  if constexpr (ONE) {
    __shared__ RouteMasks masks;
    __shared__ int wave_sums[kRouteWaves];
    int total;
    const int before = block_exclusive(tid < a.E ? count[tid] : 0, tid, wave_sums, total);
    if (tid < a.E) masks.base[tid] = before;
    if (tid <= a.E) a.offsets[tid] = before;
    for (int p = total + tid; p < a.T * a.k; p += kRouteThreads) a.rows[p] = -1;
    place_chunk(a, 0, id, masks, tid, lane, wave);
  } else {
    for (int e = tid; e < a.E; e += kRouteThreads) a.counts[blockIdx.x * a.E + e] = count[e];
  }
}

// Second launch: every workgroup works out its experts' first rows from all counts, and places
// its tokens. 2^LOG_E >= E threads per row of counts.
template <int LOG_E>
__global__ __launch_bounds__(kRouteThreads) void k_route_place(RouteArgs a, int chunks) {
  constexpr int EP = 1 << LOG_E, SETS = kRouteThreads / EP, UNROLL = 8;
  __shared__ RouteMasks masks;
  __shared__ int sums[2][SETS][EP];
  __shared__ int wave_sums[kRouteWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int e = tid & (EP - 1), set = tid >> LOG_E, blocks = gridDim.x;
  int all = 0, mine = 0;  // tokens that chose e: of every workgroup, of those before this one
  for (int b0 = set; b0 < blocks; b0 += SETS * UNROLL) {
    int v[UNROLL];
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
      const int b = b0 + i * SETS;
      v[i] = b < blocks && e < a.E ? a.counts[b * a.E + e] : 0;
    }
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
      all += v[i];
      mine += b0 + i * SETS < static_cast<int>(blockIdx.x) ? v[i] : 0;
    }
  }
  sums[0][set][e] = all;
  sums[1][set][e] = mine;
  __syncthreads();
  all = mine = 0;
  if (tid < EP)
    for (int i = 0; i < SETS; ++i) {
      all += sums[0][i][tid];
      mine += sums[1][i][tid];
    }
  int total;
  const int before = block_exclusive(all, tid, wave_sums, total);
  if (tid < a.E) masks.base[tid] = before + mine;
  if (blockIdx.x == 0 && tid <= a.E) a.offsets[tid] = before;
  for (int p = total + blockIdx.x * kRouteThreads + tid; p < a.T * a.k; p += gridDim.x * kRouteThreads) a.rows[p] = -1;
  for (int c = 0; c < chunks; ++c) {
    const int64_t chunk0 = (static_cast<int64_t>(blockIdx.x) * chunks + c) * kRouteChunk;
    if (chunk0 >= a.T) break;
    int id[kRouteTokens];
#pragma unroll
    for (int p = 0; p < kRouteTokens; ++p) {
      const int64_t t = chunk0 + wave * kRouteTokens + p;
      id[p] = t < a.T && lane < a.k ? a.ids[t * a.k + lane] : -1;
    }
    place_chunk(a, static_cast<int>(chunk0), id, masks, tid, lane, wave);
    __syncthreads();
  }
}

size_t route_scratch_bytes(int64_t T, int64_t E) {
  int chunks, blocks;
  route_geometry(T, &chunks, &blocks);
  return blocks == 1 && chunks == 1 ? 0 : static_cast<size_t>(blocks) * E * 4;
}

template <int V>
static hipError_t route(const RouteArgs& a, hipStream_t s) {
  int chunks, blocks;
  route_geometry(a.T, &chunks, &blocks);
  if (blocks == 1 && chunks == 1) {
    hipLaunchKernelGGL((k_route<V, true>), dim3(1), dim3(kRouteThreads), 0, s, a, 1);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((k_route<V, false>), dim3(blocks), dim3(kRouteThreads), 0, s, a, chunks);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  constexpr int LOG_E = V == 1 ? 6 : V == 2 ? 7 : V == 4 ? 8 : 9;
  hipLaunchKernelGGL(k_route_place<LOG_E>, dim3(blocks), dim3(kRouteThreads), 0, s, a, chunks);
  return hipGetLastError();
}

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
  if (a.E <= 64) return route<1>(a, s);
  if (a.E <= 128) return route<2>(a, s);
  if (a.E <= 256) return route<4>(a, s);
  return route<8>(a, s);
}

// Y[t] = sum over places j of weights[t, j] P[slots[t, j]], in fp32, j ascending, one rounding; a
// slot outside P adds nothing. A thread has 8 features of a token; every row's 16 bytes are
// asked for before the first is used (a row that is not there through an empty buffer).
template <class T, int K>
__global__ __launch_bounds__(256) void k_combine(CombineArgs a) {
  typedef typename T::elem v8e __attribute__((ext_vector_type(8)));
  const int per = a.D / 8;
  const int64_t t = blockIdx.x;
  const int c = blockIdx.y * 256 + threadIdx.x;
  if (c >= per) return;
  float sum[8] = {};
  for (int j0 = 0; j0 < a.k; j0 += K) {
    v4u x[K];
    float w[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const int slot = j0 + j < a.k ? a.slots[t * a.k + j0 + j] : -1;
      const bool on = slot >= 0 && slot < a.rows;
      w[j] = on ? a.weights[t * a.k + j0 + j] : 0.0f;
      const char* row = static_cast<const char*>(a.P) + static_cast<size_t>(on ? slot : 0) * a.D * 2;
      x[j] = buf_load16(make_rsrc(row, on ? a.D * 2u : 0u), c * 16u);
    }
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const v8e v = __builtin_bit_cast(v8e, x[j]);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] = __builtin_fmaf(w[j], static_cast<float>(v[e]), sum[e]);
    }
  }
  v8e out;
#pragma unroll
  for (int e = 0; e < 8; ++e) out[e] = T::round(sum[e]);
  *reinterpret_cast<v8e*>(static_cast<uint16_t*>(a.Y) + t * a.D + 8 * c) = out;
}

template <class T>
static hipError_t combine(const CombineArgs& a, hipStream_t s) {
  const dim3 grid(a.T, (a.D / 8 + 255) / 256);
  if (a.k <= 1) hipLaunchKernelGGL((k_combine<T, 1>), grid, dim3(256), 0, s, a);
  else if (a.k <= 2) hipLaunchKernelGGL((k_combine<T, 2>), grid, dim3(256), 0, s, a);
  else if (a.k <= 4) hipLaunchKernelGGL((k_combine<T, 4>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_combine<T, 8>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_combine(const CombineArgs& a, int type, hipStream_t s) {
  return type == kMxF16 ? combine<F16>(a, s) : combine<B16>(a, s);
}

}  // namespace i8mm
