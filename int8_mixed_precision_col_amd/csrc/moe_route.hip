// Routing of any number of tokens, and the way back from the experts' rows to tokens.
//
// Routing: for token t the top_k experts of the largest logits (ties to the lowest index, -inf is
// off) with their softmax weights, as in moe.hip, and the T k (token, place) pairs ordered by
// expert and then token: row p of that order is token rows[p]; expert e has the rows offsets[e]
// up to offsets[e + 1]; the pair (t, j) is row slots[t, j]. A token chooses an expert at most once,
// so a pair's row is offsets[e] + the number of earlier tokens that chose e: counts of the
// tokens before its workgroup's (kept by the first launch), of those before its 32, and the
// bits below its own in the mask of those 32. No atomics decide an order.
//
// Bound by the chain of instructions per token and by launches, not by bytes (4.2 MB in, 1.3 MB out
// for 8192 tokens, 8 of 256 experts: 1 us). 16 lanes to a token: four tokens advance by the same
// instructions and a maximum takes four steps instead of six (a wave per token, four of them
// interleaved: 18.3 us for the first launch of that case, now 8.5, of 256 workgroups; the second
// 6.8 with 16-bit counts, 8.4 with 32-bit ones). 1 token, 8 of 64: 3.3 us, an empty launch 1.8.
#include "group_launch.hpp"
#include "moe_keys.hpp"
#include "mx4.hpp"

namespace i8mm {

constexpr int kRouteWaves = 8, kRouteThreads = 64 * kRouteWaves;
constexpr int kRouteTokens = 4;                           // of a wave at a time, 16 lanes each
constexpr int kRouteChunk = kRouteWaves * kRouteTokens;   // of a workgroup: the bits of a mask
constexpr int kRouteMaxBlocks = 260;                      // 2^24 tokens are less than 2^16 for each
constexpr int kRouteOneChunks = 2;                        // of one workgroup that needs no second launch

// Chunks per workgroup, and workgroups.
static void route_geometry(int64_t T, int* chunks, int* blocks) {
  const int64_t all = (T + kRouteChunk - 1) / kRouteChunk;
  *chunks = static_cast<int>(all <= kRouteOneChunks ? all : (all + kRouteMaxBlocks - 1) / kRouteMaxBlocks);
  *blocks = static_cast<int>((all + *chunks - 1) / *chunks);
}

// Reductions over the 16 lanes of a token, the result in all of them.
template <class F>
__device__ __forceinline__ unsigned over_token(unsigned v, F f) {
  v = f(v, static_cast<unsigned>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x128, 0xF, 0xF, true)));  // row_ror:8
  v = f(v, static_cast<unsigned>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x124, 0xF, 0xF, true)));
  v = f(v, static_cast<unsigned>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x122, 0xF, 0xF, true)));
  return f(v, static_cast<unsigned>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x121, 0xF, 0xF, true)));
}
__device__ __forceinline__ unsigned token_max(unsigned v) {
  return over_token(v, [](unsigned x, unsigned y) { return max(x, y); });
}
__device__ __forceinline__ float token_sum(float v) {
  return __builtin_bit_cast(float, over_token(__builtin_bit_cast(unsigned, v), [](unsigned x, unsigned y) {
    return __builtin_bit_cast(unsigned, __builtin_bit_cast(float, x) + __builtin_bit_cast(float, y));
  }));
}

// Keys of logits, greater for what is chosen first, 0 for an expert that is off: of fp32 logits the
// ordered bits (moe_keys.hpp), of 16-bit ones the ordered bits above 0xffff - expert, so that the
// greatest key tells the expert and no two are equal.
template <bool NARROW>
struct RouteKey {
  static __device__ __forceinline__ unsigned make(unsigned bits, int type, int e) {
    if constexpr (!NARROW) return moe_key(__builtin_bit_cast(float, bits));
    const unsigned inf = type == kMxF16 ? 0x7c00u : 0x7f80u, mag = bits & 0x7fffu, neg = bits >> 15;
    if (mag == inf && neg) return 0u;
    const unsigned key = mag > inf ? 0xffffu : mag == 0u ? 0x8000u : neg ? bits ^ 0xffffu : bits ^ 0x8000u;
    return key << 16 | (0xffffu - static_cast<unsigned>(e));
  }
  static __device__ __forceinline__ float value(unsigned key, int type) {
    if constexpr (!NARROW) return moe_unkey(key);
    const unsigned k = key >> 16;
    if (k == 0xffffu) return __builtin_nanf("");
    const unsigned short bits = static_cast<unsigned short>(k & 0x8000u ? k ^ 0x8000u : k ^ 0xffffu);
    return type == kMxF16 ? static_cast<float>(__builtin_bit_cast(_Float16, bits))
                          : __builtin_bit_cast(float, static_cast<unsigned>(bits) << 16);
  }
};

// The wave's four tokens t0 .. t0 + 3, 16 lanes each, all by the same instructions: lane l of a token
// has the experts 2 l + 32 i and 2 l + 32 i + 1, i < V / 2. Lane j leaves with place j's expert (-1:
// none) and stores it with its weight.
template <int V, bool NARROW>
__device__ __forceinline__ int route_tokens(const RouteArgs& a, int64_t t0, int lane) {
  typedef RouteKey<NARROW> Key;
  const int l = lane & 15;
  const int64_t t = t0 + (lane >> 4);
  const bool on = t < a.T;
  const int64_t row = (on ? t : a.T - 1) * a.E;
  unsigned key[V];
  if (a.E % 2 == 0) {
    unsigned raw[NARROW ? V / 2 : V];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const int64_t at = row + min(2 * l + 32 * i, a.E - 2);
      if constexpr (NARROW) {
        raw[i] = *reinterpret_cast<const unsigned*>(static_cast<const uint16_t*>(a.logits) + at);
      } else {
        const v2u two = *reinterpret_cast<const v2u*>(static_cast<const float*>(a.logits) + at);
        raw[2 * i] = two[0];
        raw[2 * i + 1] = two[1];
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = 2 * l + 32 * (i / 2) + (i & 1);
      unsigned bits;
      if constexpr (NARROW) bits = i & 1 ? raw[i / 2] >> 16 : raw[i / 2] & 0xffffu;
      else bits = raw[i];
      key[i] = on && e < a.E ? Key::make(bits, a.logits_type, e) : 0u;
    }
  } else {
    unsigned raw[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int64_t at = row + min(2 * l + 32 * (i / 2) + (i & 1), a.E - 1);
      if constexpr (NARROW) raw[i] = static_cast<const uint16_t*>(a.logits)[at];
      else raw[i] = static_cast<const unsigned*>(a.logits)[at];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = 2 * l + 32 * (i / 2) + (i & 1);
      key[i] = on && e < a.E ? Key::make(raw[i], a.logits_type, e) : 0u;
    }
  }
  unsigned best = key[0];
#pragma unroll
  for (int i = 1; i < V; ++i) best = max(best, key[i]);
  unsigned top = token_max(best);  // 0: no expert is on
  const float most = Key::value(top, a.logits_type);
  float all = 0.0f;
  if (!a.renormalize)
#pragma unroll
    for (int i = 0; i < V; ++i) all += key[i] ? expf(Key::value(key[i], a.logits_type) - most) : 0.0f;
  unsigned mine = 0;
  int id = -1;
  for (int j = 0; j < a.k; ++j) {
    int e;
    if constexpr (NARROW) {
      e = static_cast<int>(0xffffu - (top & 0xffffu));
    } else {
      unsigned at = 0xffffffffu;  // the lowest expert with this logit
#pragma unroll
      for (int i = V - 1; i >= 0; --i) at = key[i] == top ? 2 * l + 32 * (i / 2) + (i & 1) : at;
      e = static_cast<int>(over_token(at, [](unsigned x, unsigned y) { return min(x, y); }));
    }
    if (l == j && top) {
      mine = top;
      id = e;
    }
    best = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (NARROW) key[i] = key[i] == top ? 0u : key[i];
      else key[i] = 2 * l + 32 * (i / 2) + (i & 1) == e ? 0u : key[i];
      best = max(best, key[i]);
    }
    top = token_max(best);
  }
  const float w = mine ? expf(Key::value(mine, a.logits_type) - most) : 0.0f;
  const float sum = token_sum(a.renormalize ? w : all);
  if (l < a.k && on) {
    a.ids[t * a.k + l] = id;
    a.weights[t * a.k + l] = id < 0 ? 0.0f : __fdiv_rn(w, sum);
  }
  return id;
}

// Exclusive prefix sum of the threads' counts v, with the sum of all in `total`. All threads of the
// workgroup take part.
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
// the chunk's. id: place l of token 4 wave + lane / 16 of the chunk.
struct RouteMasks {
  unsigned bits[kMoeMaxExperts];  // of the chunk's tokens
  int base[kMoeMaxExperts];
};
__device__ __forceinline__ void place_chunk(const RouteArgs& a, int64_t chunk0, int id, RouteMasks& m, int tid) {
  static_assert(kRouteChunk == 32, "a mask's bits");
  const int l = tid & 15, in = tid >> 4;  // 16 lanes to a token
  const int64_t t = chunk0 + in;
  for (int e = tid; e < a.E; e += kRouteThreads) m.bits[e] = 0u;
  __syncthreads();
  if (id >= 0) atomicOr(&m.bits[id], 1u << in);
  __syncthreads();
  if (l < a.k && t < a.T) {
    const int row = id < 0 ? -1 : m.base[id] + __builtin_popcount(m.bits[id] & ((1u << in) - 1u));
    if (row >= 0) a.rows[row] = static_cast<int>(t);
    a.slots[t * a.k + l] = row;
  }
  __syncthreads();
  for (int e = tid; e < a.E; e += kRouteThreads) m.base[e] += __builtin_popcount(m.bits[e]);
  __syncthreads();
}

// First launch: the chosen experts of every token, and how many tokens of the workgroup chose each
// expert. With one workgroup (ONE) the rows too.
template <int V, bool NARROW, bool ONE>
__global__ __launch_bounds__(kRouteThreads) void k_route(RouteArgs a, int chunks) {
  __shared__ int count[kMoeMaxExperts];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  for (int e = tid; e < a.E; e += kRouteThreads) count[e] = 0;
  __syncthreads();
  int id[ONE ? kRouteOneChunks : 1];
  if constexpr (ONE) {
#pragma unroll
    for (int c = 0; c < kRouteOneChunks; ++c) {
      id[c] = -1;
      const int t0 = c * kRouteChunk + wave * kRouteTokens;
      if (t0 < a.T) id[c] = route_tokens<V, NARROW>(a, t0, lane);
      if (id[c] >= 0) atomicAdd(&count[id[c]], 1);
    }
  } else {
    for (int c = 0; c < chunks; ++c) {
      const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * chunks + c) * kRouteChunk + wave * kRouteTokens;
      if (t0 >= a.T) break;
      id[0] = route_tokens<V, NARROW>(a, t0, lane);
      if (id[0] >= 0) atomicAdd(&count[id[0]], 1);
    }
  }
  __syncthreads();
  if constexpr (ONE) {
    __shared__ RouteMasks masks;
    __shared__ int wave_sums[kRouteWaves];
    int total;
    const int before = block_exclusive(tid < a.E ? count[tid] : 0, tid, wave_sums, total);
    if (tid < a.E) {
      masks.base[tid] = before;
      a.offsets[tid] = before;
    }
    if (tid == 0) a.offsets[a.E] = total;
    for (int p = total + tid; p < a.T * a.k; p += kRouteThreads) a.rows[p] = -1;
    place_chunk(a, 0, id[0], masks, tid);
    if (a.T > kRouteChunk) place_chunk(a, kRouteChunk, id[1], masks, tid);
  } else {
    const int words = (a.E + 1) / 2;  // two experts to a word
    for (int i = tid; i < words; i += kRouteThreads)
      a.counts[blockIdx.x * words + i] = count[2 * i] | (2 * i + 1 < a.E ? count[2 * i + 1] << 16 : 0);
  }
}

// Second launch: every workgroup works out its experts' first rows from all counts, and places
// its tokens. 2^LOG_E >= E / 2 threads per row of counts, two experts each.
template <int LOG_E>
__global__ __launch_bounds__(kRouteThreads) void k_route_place(RouteArgs a, int chunks) {
  constexpr int WP = 1 << LOG_E, SETS = kRouteThreads / WP, UNROLL = 16;
  __shared__ RouteMasks masks;
  __shared__ int sums[2][SETS][2 * WP];
  __shared__ int wave_sums[kRouteWaves];
  const int tid = threadIdx.x, l = tid & 15, words = (a.E + 1) / 2;
  const int w = tid & (WP - 1), set = tid >> LOG_E, blocks = gridDim.x;
  auto place = [&](int c) -> int64_t { return (static_cast<int64_t>(blockIdx.x) * chunks + c) * kRouteChunk + (tid >> 4); };
  auto id_of = [&](int c) { return l < a.k && place(c) < a.T ? a.ids[place(c) * a.k + l] : -1; };
  int id = id_of(0);
  int all0 = 0, all1 = 0, mine0 = 0, mine1 = 0;  // tokens of every workgroup, of those before this one
  for (int b0 = set; b0 < blocks; b0 += SETS * UNROLL) {
    unsigned v[UNROLL];
#pragma unroll
    for (int i = 0; i < UNROLL; ++i)
      v[i] = static_cast<unsigned>(a.counts[min(b0 + i * SETS, blocks - 1) * words + min(w, words - 1)]);
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
      const int b = b0 + i * SETS;
      const int lo = b < blocks ? v[i] & 0xffffu : 0, hi = b < blocks ? v[i] >> 16 : 0;
      all0 += lo;
      all1 += hi;
      mine0 += b < static_cast<int>(blockIdx.x) ? lo : 0;
      mine1 += b < static_cast<int>(blockIdx.x) ? hi : 0;
    }
  }
  sums[0][set][2 * w] = all0;
  sums[0][set][2 * w + 1] = all1;
  sums[1][set][2 * w] = mine0;
  sums[1][set][2 * w + 1] = mine1;
  __syncthreads();
  int all = 0, mine = 0;
  if (tid < a.E)
    for (int i = 0; i < SETS; ++i) {
      all += sums[0][i][tid];
      mine += sums[1][i][tid];
    }
  int total;
  const int before = block_exclusive(all, tid, wave_sums, total);
  if (tid < a.E) {
    masks.base[tid] = before + mine;
    if (blockIdx.x == 0) a.offsets[tid] = before;
  }
  if (blockIdx.x == 0 && tid == 0) a.offsets[a.E] = total;
  for (int p = total + blockIdx.x * kRouteThreads + tid; p < a.T * a.k; p += gridDim.x * kRouteThreads) a.rows[p] = -1;
  for (int c = 0; c < chunks; ++c) {
    const int64_t chunk0 = (static_cast<int64_t>(blockIdx.x) * chunks + c) * kRouteChunk;
    if (chunk0 >= a.T) break;
    if (c > 0) id = id_of(c);
    place_chunk(a, chunk0, id, masks, tid);
  }
}

size_t route_scratch_bytes(int64_t T, int64_t E) {
  int chunks, blocks;
  route_geometry(T, &chunks, &blocks);
  return blocks == 1 ? 0 : static_cast<size_t>(blocks) * ((E + 1) / 2) * 4;
}

template <int V, bool NARROW>
static hipError_t route(const RouteArgs& a, hipStream_t s) {
  int chunks, blocks;
  route_geometry(a.T, &chunks, &blocks);
  if (blocks == 1) {
    hipLaunchKernelGGL((k_route<V, NARROW, true>), dim3(1), dim3(kRouteThreads), 0, s, a, chunks);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((k_route<V, NARROW, false>), dim3(blocks), dim3(kRouteThreads), 0, s, a, chunks);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  constexpr int LOG_E = V == 4 ? 5 : V == 8 ? 6 : V == 16 ? 7 : 8;
  hipLaunchKernelGGL(k_route_place<LOG_E>, dim3(blocks), dim3(kRouteThreads), 0, s, a, chunks);
  return hipGetLastError();
}

template <bool NARROW>
static hipError_t route(const RouteArgs& a, hipStream_t s) {
  if (a.E <= 64) return route<4, NARROW>(a, s);
  if (a.E <= 128) return route<8, NARROW>(a, s);
  if (a.E <= 256) return route<16, NARROW>(a, s);
  return route<32, NARROW>(a, s);
}

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
  return a.logits_type == kMxF32 ? route<false>(a, s) : route<true>(a, s);
}

// Y[t] = sum over places j of weights[t, j] P[slots[t, j]], in fp32, j ascending, one rounding; a
// slot outside P adds nothing. A thread has 8 features of a token; every row's 16 bytes are
// asked for before the first is used (a row that is not there through an empty buffer). Bound by
// HBM: 4096 tokens, 8 rows each of 4096 features, 302 MB, 53.5 us, 5.6 TB/s (58 through the caches; a
// large copy moves 5.1, a launch that only reads 6.3).
template <class T, int K>
__global__ __launch_bounds__(256) void k_combine(CombineArgs a) {
  typedef typename T::elem v8e __attribute__((ext_vector_type(8)));
  const int per = a.D / 8;
  const int64_t t = blockIdx.x + static_cast<int64_t>(gridDim.x) * blockIdx.z;
  const int c = blockIdx.y * 256 + threadIdx.x;
  if (c >= per || t >= a.T) return;
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
      // past the caches (2): each row is read once
      x[j] = __builtin_amdgcn_raw_buffer_load_b128(make_rsrc(row, on ? a.D * 2u : 0u), c * 16, 0, 2);
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
  // a launch has less than 2^32 threads in x: more tokens than that lie side by side in z
  const unsigned sides = a.T < 1 << 24 ? 1 : 2;
  const dim3 grid((a.T + sides - 1) / sides, (a.D / 8 + 255) / 256, sides);
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
