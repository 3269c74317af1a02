// Low-rank adapters of many requests beside a shared projection: row m with adapter a = ids[m],
//   out[m] = Y[m] + scale_a B_a (A_a X[m]),   A_a [r_a, K], B_a [N, r_a],
// and out[m] = Y[m] where ids[m] is no adapter. fp32 sums, one rounding of out.
//
// Two products with a weight per group of rows, both far below what the matrix cores could do:
// what bounds them is reading X, Y and the adapters and writing out. k_lora_shrink: V = A X over
// a part of K for a tile of up to 64 rows of one adapter, fp32 sums to scratch (parts of K as
// few as fill the chip). k_lora_expand: the tile's V, summed over the parts, against a range of
// features. V enters the matrix instructions as two parts, its rounding to the type and what that left
// (bf16 16 bits together, fp16 22 under a power of two per row that keeps both in range); the
// output's own rounding is to 8 and 11 bits.
//
// Rows in order: up to 64 rows every workgroup orders for itself by comparing the ids (no launch);
// beyond, one workgroup sorts them first (k_lora_order).
#include "group.hpp"
#include "group_launch.hpp"
#include "mx4.hpp"
#include "mx4_launch.hpp"

namespace i8mm {

constexpr int kLoraFew = 64;  // rows that each workgroup orders by itself
constexpr int kLoraWaves = 4;

// ---- rows by adapter ----

// Counting sort of ids into S adapters and, last, the rows without one; stable. 16 waves each take
// a stretch of the rows and count it, then place it, 64 rows at a time; then the table of tiles.
constexpr int kOrderWaves = 16, kOrderThreads = 64 * kOrderWaves;
__global__ __launch_bounds__(kOrderThreads) void k_lora_order(LoraArgs a, int most) {
  extern __shared__ int lds[];
  const int G = a.S + 1, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int* next = lds;                  // [wave][G]: rows, then the next place
  int* first = lds + kOrderWaves * G;  // [G + 1]
  __shared__ int wave_sums[kOrderWaves];
  const int chunks = (a.M + 63) / 64, per = (chunks + kOrderWaves - 1) / kOrderWaves;
  const int m0 = min(wave * per * 64, a.M), m1 = min(m0 + per * 64, a.M);
  for (int i = tid; i < kOrderWaves * G; i += kOrderThreads) next[i] = 0;
  __syncthreads();
  auto group_of = [&](int m) {
    const int id = a.ids[m];
    return id >= 0 && id < a.S ? id : a.S;
  };
  for (int m = m0 + lane; m < m1; m += 64) atomicAdd(&next[wave * G + group_of(m)], 1);
  __syncthreads();
  // exclusive sums: over the groups (a thread has one or two, G <= 1025), within one over the waves
  int run = 0;
  for (int g0 = 0; g0 < G; g0 += kOrderThreads) {
    const int g = g0 + tid;
    int n = 0;
    if (g < G)
      for (int w = 0; w < kOrderWaves; ++w) n += next[w * G + g];
    int upto = wave_prefix_sum(n);
    if (lane == 63) wave_sums[wave] = upto;
    __syncthreads();
    int total = 0;
    for (int w = 0; w < kOrderWaves; ++w) {
      if (w < wave) upto += wave_sums[w];
      total += wave_sums[w];
    }
    if (g < G) {
      int at = run + upto - n;
      first[g] = at;
      for (int w = 0; w < kOrderWaves; ++w) {
        const int c = next[w * G + g];
        next[w * G + g] = at;
        at += c;
      }
    }
    run += total;
    __syncthreads();
  }
  if (tid == 0) first[G] = a.M;
  __syncthreads();
  for (int c0 = m0; c0 < m1; c0 += 64) {
    const int m = c0 + lane;
    const bool on = m < m1;
    const int g = on ? group_of(m) : -1;
    // the lanes of equal group: rank among them, and the last one moves the group's next place on
    unsigned long long left = __ballot(on);
    while (left) {
      const int who = __builtin_ctzll(left);
      const int lead = __builtin_amdgcn_readlane(g, who);
      const unsigned long long same = __ballot(g == lead);
      if (g == lead) {
        const int rank = __builtin_popcountll(same & ((1ull << lane) - 1ull));
        a.order[next[wave * G + lead] + rank] = m;
      }
      wave_lds_fence();
      if (lane == who) next[wave * G + lead] += __builtin_popcountll(same);
      wave_lds_fence();
      left &= ~same;
    }
  }
  __syncthreads();
  // the rows without an adapter are the table's group -1
  make_group_tiles<kOrderThreads>(first, a.S, a.M, kLoraRows, most, a.table);
}

// The tile of workgroup column b: its adapter (-1: none) and its rows, in LDS. false: no such tile.
struct LoraTile {
  int adapter, rows;
};
__device__ __forceinline__ bool lora_tile(const LoraArgs& a, int b, int* row_of, LoraTile& t) {
  const int tid = threadIdx.x, lane = tid & 63;
  if (a.M <= kLoraFew) {
    // every wave finds the rows whose id no earlier row has: the b-th of them leads tile b
    const int id0 = lane < a.M ? a.ids[lane] : -2;
    const int id = lane >= a.M ? -2 : id0 >= 0 && id0 < a.S ? id0 : -1;
    unsigned long long mine = 0, leaders = 0;
    for (int m = 0; m < a.M; ++m) {
      const unsigned long long same = __ballot(id == __builtin_amdgcn_readlane(id, m));
      if (__builtin_ctzll(same) == m) {
        if (__builtin_popcountll(leaders) == b) {
          mine = same;
          t.adapter = __builtin_amdgcn_readlane(id, m);
        }
        leaders |= 1ull << m;
      }
    }
    if (mine == 0) return false;
    t.rows = __builtin_popcountll(mine);
    if (tid < 64 && (mine >> lane & 1)) row_of[__builtin_popcountll(mine & ((1ull << lane) - 1ull))] = lane;
  } else {
    if (b >= a.table[0].x) return false;
    const int4 e = a.table[1 + b];
    t.adapter = e.x;
    t.rows = e.z;
    if (tid < e.z) row_of[tid] = a.order[e.y + tid];
  }
  __syncthreads();
  return true;
}

__device__ __forceinline__ int lora_rank(const LoraArgs& a, int adapter) {
  return a.ranks ? min(max(a.ranks[adapter], 0), a.R) : a.R;
}

// ---- V = A X over a part of K ----

// RB: blocks of 16 ranks. The waves share the part's K in steps of 32; each lane loads 16 bytes of
// a row, in the order of the matrix instruction's operand: rows l % 16, elements 8 (l / 16) .. + 7.
template <class T, int RB>
__global__ __launch_bounds__(64 * kLoraWaves) void k_lora_shrink(LoraArgs a) {
  __shared__ int row_of[kLoraRows];
  __shared__ __attribute__((aligned(16))) float red[kLoraWaves][kLoraRows][20];
  LoraTile tile;
  if (!lora_tile(a, blockIdx.x, row_of, tile) || tile.adapter < 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, lq = lane >> 4;
  const int steps = (a.K + 31) / 32, split = blockIdx.y, splits = gridDim.y;
  const int s0 = static_cast<int>(static_cast<int64_t>(steps) * split / splits);
  const int s1 = static_cast<int>(static_cast<int64_t>(steps) * (split + 1) / splits);
  const int rank = lora_rank(a, tile.adapter);
  const uint16_t *x[4], *w[RB];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    x[j] = static_cast<const uint16_t*>(a.X) + static_cast<int64_t>(row_of[min(16 * j + l16, tile.rows - 1)]) * a.ldx + 8 * lq;
#pragma unroll
  for (int i = 0; i < RB; ++i)
    w[i] = static_cast<const uint16_t*>(a.A) +
           (static_cast<int64_t>(tile.adapter) * a.R + min(16 * i + l16, max(rank - 1, 0))) * a.K + 8 * lq;
  v4f acc[RB][4];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = v4f{};
  const int blocks = (tile.rows + 15) / 16;
  for (int s = s0 + wave; s < s1; s += kLoraWaves) {
    const int k = 32 * s;
    const bool in = k + 8 * lq < a.K;
    v4u xv[4], wv[RB];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      xv[j] = v4u{};
      if (j < blocks && in) xv[j] = *reinterpret_cast<const v4u*>(x[j] + k);
    }
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      wv[i] = v4u{};
      if (in) wv[i] = *reinterpret_cast<const v4u*>(w[i] + k);
    }
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < blocks) acc[i][j] = T::mfma(wv[i], xv[j], acc[i][j]);
  }
  // lane l holds row 16 j + l % 16, ranks 16 i + 4 (l / 16) .. + 3: the waves' sums through LDS
  const int R16 = 16 * RB;
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    if (i > 0) __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < blocks) *reinterpret_cast<v4f*>(&red[wave][16 * j + l16][4 * lq]) = acc[i][j];
    __syncthreads();
    const int r = tid >> 2, c = 4 * (tid & 3);
    if (r < tile.rows) {
      v4f sum = *reinterpret_cast<const v4f*>(&red[0][r][c]);
#pragma unroll
      for (int v = 1; v < kLoraWaves; ++v) sum += *reinterpret_cast<const v4f*>(&red[v][r][c]);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] = 16 * i + c + e < rank ? sum[e] : 0.0f;
      *reinterpret_cast<v4f*>(a.part + (static_cast<int64_t>(split) * a.M + row_of[r]) * R16 + 16 * i + c) = sum;
    }
  }
}

// ---- out = Y + scale B V ----

// A workgroup takes a tile's rows and `span` features, its waves 32 of them at a time: two
// blocks of 16 of B's rows, taken so that a lane ends with 8 consecutive features of a row.
// KS: steps of 32 ranks.
template <class T, int KS>
__global__ __launch_bounds__(64 * kLoraWaves) void k_lora_expand(LoraArgs a, int span) {
  typedef typename T::elem elem;
  typedef elem v8e __attribute__((ext_vector_type(8)));
  typedef elem v4e __attribute__((ext_vector_type(4)));
  constexpr int LR = 32 * KS + 8;  // padded row of V in LDS
  __shared__ int row_of[kLoraRows];
  __shared__ __attribute__((aligned(16))) elem v[2][kLoraRows][LR];
  __shared__ float row_scale[kLoraRows];
  LoraTile tile;
  if (!lora_tile(a, blockIdx.x, row_of, tile)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, lq = lane >> 4;
  const int n0 = blockIdx.y * span, n1 = min(n0 + span, a.N);
  const uint16_t* Y = static_cast<const uint16_t*>(a.Y);
  uint16_t* out = static_cast<uint16_t*>(a.out);
  const int rank = tile.adapter < 0 ? 0 : lora_rank(a, tile.adapter);
  if (rank == 0) {
    if (Y == out) return;
    const int per = (n1 - n0) / 8;
    for (int t = tid; t < tile.rows * per; t += 64 * kLoraWaves) {
      const int64_t m = row_of[t / per];
      const int n = n0 + t % per * 8;
      *reinterpret_cast<v4u*>(out + m * a.ldo + n) = *reinterpret_cast<const v4u*>(Y + m * a.ldy + n);
    }
    return;
  }
  const int R16 = (a.R + 15) & ~15;
  // V: four threads to a row, each 4 ranks of every 16
  {
    const int r = tid >> 2, c = 4 * (tid & 3);
    v4f sum[2 * KS];
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < 2 * KS; ++i) {
      sum[i] = v4f{};
      if (r < tile.rows && 16 * i < R16) {
        const float* p = a.part + static_cast<int64_t>(row_of[r]) * R16 + 16 * i + c;
        for (int s = 0; s < a.splits; ++s) sum[i] += *reinterpret_cast<const v4f*>(p + static_cast<int64_t>(s) * a.M * R16);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) most = fmaxf(most, fabsf(sum[i][e]));
    }
    float up = 1.0f, down = 1.0f;
    if constexpr (!T::bf) {
      most = fmaxf(most, __shfl_xor(most, 1, 64));
      most = fmaxf(most, __shfl_xor(most, 2, 64));
      // the row's largest to [2^14, 2^15)
      const int e = most > 0.0f && most < __builtin_inff() ? 14 - ilogbf(most) : 0;
      up = ldexpf(1.0f, min(max(e, -126), 126));
      down = ldexpf(1.0f, -min(max(e, -126), 126));
    }
#pragma unroll
    for (int i = 0; i < 2 * KS; ++i) {
      v4e hi, lo;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float f = sum[i][e] * up;
        hi[e] = T::round(f);
        lo[e] = T::round(f - static_cast<float>(hi[e]));
      }
      *reinterpret_cast<v4e*>(&v[0][r][16 * i + c]) = hi;
      *reinterpret_cast<v4e*>(&v[1][r][16 * i + c]) = lo;
    }
    if ((tid & 3) == 0) row_scale[r] = down * (a.scales ? a.scales[tile.adapter] : 1.0f);
  }
  __syncthreads();
  const int blocks = (tile.rows + 15) / 16;
  const uint16_t* B = static_cast<const uint16_t*>(a.B) + static_cast<int64_t>(tile.adapter) * a.N * a.R;
  for (int n = n0 + 32 * wave; n < n1; n += 32 * kLoraWaves) {
    const int at = n + 8 * lq;  // this lane's output features
    v4u y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      y[j] = v4u{};
      if (16 * j + l16 < tile.rows && at < n1)
        y[j] = *reinterpret_cast<const v4u*>(Y + static_cast<int64_t>(row_of[16 * j + l16]) * a.ldy + at);
    }
    // row l % 16 of block h is feature 8 (l % 16 / 4) + 4 h + l % 4
    v4u b[2][KS];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int f = min(n + 8 * (l16 >> 2) + 4 * h + (l16 & 3), a.N - 1);
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int k = 32 * s + 8 * lq;
        b[h][s] = v4u{};
        if (k < rank) b[h][s] = *reinterpret_cast<const v4u*>(B + static_cast<int64_t>(f) * a.R + k);
        // ranks past this adapter's may hold anything
        if (k < rank && k + 8 > rank) {
#pragma unroll
          for (int d = 0; d < 4; ++d)
            b[h][s][d] &= (k + 2 * d < rank ? 0xffffu : 0u) | (k + 2 * d + 1 < rank ? 0xffff0000u : 0u);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j >= blocks) break;
      v4f acc[2] = {v4f{}, v4f{}};
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const v4u x = *reinterpret_cast<const v4u*>(&v[p][16 * j + l16][32 * s + 8 * lq]);
          acc[0] = T::mfma(b[0][s], x, acc[0]);
          acc[1] = T::mfma(b[1][s], x, acc[1]);
        }
      if (16 * j + l16 < tile.rows && at < n1) {
        const float sc = row_scale[16 * j + l16];
        const v8e old = __builtin_bit_cast(v8e, y[j]);
        v8e o;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = T::round(__builtin_fmaf(sc, acc[e >> 2][e & 3], static_cast<float>(old[e])));
        *reinterpret_cast<v8e*>(out + static_cast<int64_t>(row_of[16 * j + l16]) * a.ldo + at) = o;
      }
    }
  }
}

// Tiles of the rows, as many as there may be.
static int64_t lora_tiles(int64_t M, int64_t S) {
  if (M <= kLoraFew) return S + 1 < M ? S + 1 : M;
  return group_tiles_most(M, S, kLoraRows);
}

int lora_splits(int64_t M, int64_t K, int64_t S) {
  const int64_t by_tiles = 1024 / lora_tiles(M, S), by_k = K / 256;
  const int64_t n = by_tiles < by_k ? by_tiles : by_k;
  return static_cast<int>(n < 1 ? 1 : n > 64 ? 64 : n);
}

template <class T>
static hipError_t lora(const LoraArgs& a, hipStream_t s) {
  const unsigned tiles = static_cast<unsigned>(lora_tiles(a.M, a.S));
  if (a.M > kLoraFew) {
    const size_t lds = (static_cast<size_t>(kOrderWaves + 1) * (a.S + 1) + 1) * 4;
    hipLaunchKernelGGL(k_lora_order, dim3(1), dim3(kOrderThreads), lds, s, a, static_cast<int>(tiles));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const dim3 threads(64 * kLoraWaves), shrink(tiles, a.splits);
  switch ((a.R + 15) / 16) {
    case 1: hipLaunchKernelGGL((k_lora_shrink<T, 1>), shrink, threads, 0, s, a); break;
    case 2: hipLaunchKernelGGL((k_lora_shrink<T, 2>), shrink, threads, 0, s, a); break;
    case 3: hipLaunchKernelGGL((k_lora_shrink<T, 3>), shrink, threads, 0, s, a); break;
    case 4: hipLaunchKernelGGL((k_lora_shrink<T, 4>), shrink, threads, 0, s, a); break;
    case 5: hipLaunchKernelGGL((k_lora_shrink<T, 5>), shrink, threads, 0, s, a); break;
    case 6: hipLaunchKernelGGL((k_lora_shrink<T, 6>), shrink, threads, 0, s, a); break;
    case 7: hipLaunchKernelGGL((k_lora_shrink<T, 7>), shrink, threads, 0, s, a); break;
    default: hipLaunchKernelGGL((k_lora_shrink<T, 8>), shrink, threads, 0, s, a); break;
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // features per workgroup: whole rounds of its waves, about four workgroups per CU
  constexpr int round = 32 * kLoraWaves;
  const int64_t want = (static_cast<int64_t>(a.N) * tiles + 1023) / 1024;
  const int span = static_cast<int>((want + round - 1) / round * round);
  const dim3 expand(tiles, (a.N + span - 1) / span);
  switch ((a.R + 31) / 32) {
    case 1: hipLaunchKernelGGL((k_lora_expand<T, 1>), expand, threads, 0, s, a, span); break;
    case 2: hipLaunchKernelGGL((k_lora_expand<T, 2>), expand, threads, 0, s, a, span); break;
    case 3: hipLaunchKernelGGL((k_lora_expand<T, 3>), expand, threads, 0, s, a, span); break;
    default: hipLaunchKernelGGL((k_lora_expand<T, 4>), expand, threads, 0, s, a, span); break;
  }
  return hipGetLastError();
}

hipError_t launch_lora(const LoraArgs& a, int type, hipStream_t s) {
  return type == kMxF16 ? lora<F16>(a, s) : lora<B16>(a, s);
}

}  // namespace i8mm
