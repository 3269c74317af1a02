// Low-rank adapters of many requests beside a shared projection: row m with adapter a = ids[m],
//   out[m] = Y[m] + scale_a B_a (A_a X[m]),   A_a [r_a, K], B_a [N, r_a],
// and out[m] = Y[m] where ids[m] is no adapter. fp32 sums, one rounding of out.
//
// Two products with a weight per group of rows, both far below what the matrix cores could do:
// what bounds them is reading X, Y and the adapters and writing out. k_lora_shrink: V = A X over
// a part of K for a tile of up to 64 rows of one adapter, fp32 sums to scratch (parts of K as
// few as fill the chip). k_lora_expand: the tile's V, summed over the parts, against a range of
// features. V enters the matrix instructions as parts of the type, each of what those before it
// left: in bf16 three, all 24 bits of an fp32 sum; in fp16 two, within 2^-23 of a value, or
// 2^-39 of its row's largest where that is more (a power of two per row brings the largest to
// 2^14 .. 2^15, and fp16 ends at 2^-24). Where an adapter nearly cancels its projection those bits are
// what is left. The third part's cost, us in a graph: up to rank 64 less than 2% (4096 x 8192 x 8192 of
// rank 32 65.5 -> 65.6, 256 x 4096 x 4096 of 16 16.1 -> 16.4), at 96 and 128 up to 3% (2048 x 4096 x
// 14336 59.0 -> 60.9, 3000 x 8192 x 10240 83.9 -> 85.6).
//
// Rows in order: up to 64 rows every workgroup orders for itself by comparing the ids (no launch);
// beyond, one workgroup sorts them first (k_lora_order).
#include "gemm_kernel.hpp"
#include "group.hpp"
#include "group_launch.hpp"
#include "mx4.hpp"
#include "mx4_launch.hpp"

namespace i8mm {

constexpr int kLoraFew = 64;  // rows that each workgroup orders by itself
constexpr int kLoraWaves = 8;
constexpr int kLoraSplits = 8;  // parts of K at most
template <class T>
constexpr int kLoraParts = T::bf ? 3 : 2;  // of V's values

// ---- rows by adapter ----

// Counting sort of ids into S adapters and, last, the rows without one; stable. 16 waves each take
// a stretch of the rows, 64 at a time: lanes of equal group find each other by a ballot per bit of
// the group's number, so no order depends on atomics. Counts, their sums, places; then the table of
// tiles. Up to 4096 rows a wave's groups stay in registers from the counts to
// the places (3333 x 4096 x 11008 60.9 -> 59.5 us in all, 256 x 4096 x 4096 16.5 -> 16.1).
constexpr int kOrderWaves = 16, kOrderThreads = 64 * kOrderWaves;
constexpr int kOrderBatch = 4;  // chunks of 64 rows whose ids are asked for together
__global__ __launch_bounds__(kOrderThreads) void k_lora_order(LoraArgs a, int most) {
  extern __shared__ int lds[];
  const int G = a.S + 1, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int* next = lds + wave * G;          // this wave's rows of each group, then their next place
  int* first = lds + kOrderWaves * G;  // [G + 1]
  __shared__ int wave_sums[kOrderWaves];
  const int per = ((a.M + 63) / 64 + kOrderWaves - 1) / kOrderWaves;
  const int m0 = min(wave * per * 64, a.M), m1 = min(m0 + per * 64, a.M);
  const int bits = 32 - __builtin_clz(a.S);
  for (int g = lane; g < G; g += 64) next[g] = 0;
  wave_lds_fence();
  int group[kOrderBatch];
  unsigned long long same[kOrderBatch];  // the lanes of a chunk whose row is in this one's group
  auto find = [&](int c0) {
    int id[kOrderBatch];
#pragma unroll
    for (int i = 0; i < kOrderBatch; ++i) id[i] = a.ids[min(c0 + 64 * i + lane, a.M - 1)];
#pragma unroll
    for (int i = 0; i < kOrderBatch; ++i) {
      if (c0 + 64 * i >= m1) break;
      const int g = id[i] >= 0 && id[i] < a.S ? id[i] : a.S;
      group[i] = g;
      same[i] = __ballot(c0 + 64 * i + lane < m1);
      for (int b = 0; b < bits; ++b) {
        const unsigned long long set = __ballot(g >> b & 1);
        same[i] &= g >> b & 1 ? set : ~set;
      }
    }
  };
  auto rank = [&](int i) { return __builtin_popcountll(same[i] & ((1ull << lane) - 1ull)); };
  for (int c0 = m0; c0 < m1; c0 += 64 * kOrderBatch) {
    find(c0);
#pragma unroll
    for (int i = 0; i < kOrderBatch; ++i) {
      if (c0 + 64 * i >= m1) break;
      if (c0 + 64 * i + lane < m1 && rank(i) == 0) next[group[i]] += __builtin_popcountll(same[i]);
      wave_lds_fence();
    }
  }
  __syncthreads();
  // exclusive sums: over the groups (a thread has one or two, G <= 1025), within one over the waves
  int run = 0;
  for (int g0 = 0; g0 < G; g0 += kOrderThreads) {
    const int g = g0 + tid;
    int n = 0;
    if (g < G)
      for (int w = 0; w < kOrderWaves; ++w) n += lds[w * G + g];
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
        const int c = lds[w * G + g];
        lds[w * G + g] = at;
        at += c;
      }
    }
    run += total;
    __syncthreads();
  }
  if (tid == 0) first[G] = a.M;
  for (int c0 = m0; c0 < m1; c0 += 64 * kOrderBatch) {
    if (per > kOrderBatch) find(c0);  // one batch is still known
#pragma unroll
    for (int i = 0; i < kOrderBatch; ++i) {
      const int m = c0 + 64 * i + lane;
      if (m - lane >= m1) break;
      if (m < m1) {
        const int at = next[group[i]];
        a.order[at + rank(i)] = m;
        if (rank(i) == 0) next[group[i]] = at + __builtin_popcountll(same[i]);
      }
      wave_lds_fence();
    }
  }
  __syncthreads();
  // the rows without an adapter are the table's group -1
  make_group_tiles<kOrderThreads>(first, a.S, a.M, kLoraRows, most, a.table);
}

// A workgroup's tile, of a grid of as many tiles as there may be times parts: the tile's adapter (-1: none)
// and its rows, in LDS, and the part. false: none. RUNS, beyond kLoraFew rows: each XCD (workgroup
// number mod 8) takes a contiguous run of the tiles with all their parts, so that its L2 holds few
// adapters and a tile's V comes from memory once. The run's bounds cost a load of the table's head
// before the tile's: the staged expand gains by it (3333 x 4096 x 11008 of rank 64, 64.7 -> 61.0 us in
// all), the shrink loses (61.5).
struct LoraTile {
  int adapter, rows, part;
};
template <bool RUNS = false>
__device__ __forceinline__ bool lora_tile(const LoraArgs& a, int* row_of, LoraTile& t) {
  const int tid = threadIdx.x, lane = tid & 63;
  int b = blockIdx.x;
  t.part = blockIdx.y;
  if (!RUNS && a.M <= kLoraFew) {
    // every wave finds each row's rows of equal id, by a ballot per bit of its number; the b-th row
    // that no such row is in front of leads tile b
    const int id = a.ids[min(lane, a.M - 1)], g = id >= 0 && id < a.S ? id : a.S;
    unsigned long long same = __ballot(lane < a.M);
    for (int bit = 0; bit < 32 - __builtin_clz(a.S); ++bit) {
      const unsigned long long set = __ballot(g >> bit & 1);
      same &= g >> bit & 1 ? set : ~set;
    }
    const unsigned long long leaders = __ballot(lane < a.M && __builtin_ctzll(same) == lane);
    if (b >= __builtin_popcountll(leaders)) return false;
    const int who = __builtin_ctzll(__ballot((leaders >> lane & 1) && __builtin_popcountll(leaders & ((1ull << lane) - 1ull)) == b));
    const unsigned long long mine = static_cast<unsigned long long>(static_cast<unsigned>(__builtin_amdgcn_readlane(static_cast<int>(same), who))) |
                                    static_cast<unsigned long long>(static_cast<unsigned>(__builtin_amdgcn_readlane(static_cast<int>(same >> 32), who))) << 32;
    const int adapter = __builtin_amdgcn_readlane(g, who);
    t.adapter = adapter < a.S ? adapter : -1;
    t.rows = __builtin_popcountll(mine);
    if (tid < 64 && (mine >> lane & 1)) row_of[__builtin_popcountll(mine & ((1ull << lane) - 1ull))] = lane;
  } else {
    int4 head = a.table[0], e;
    if constexpr (RUNS) {
      const int workgroups = head.x * gridDim.y, number = blockIdx.x + gridDim.x * blockIdx.y;
      if (number >= workgroups) return false;
      const int at = group_order(number, workgroups);
      b = at / static_cast<int>(gridDim.y);
      t.part = at - b * gridDim.y;
      e = a.table[1 + b];
    } else {
      e = a.table[1 + b];  // with the head on its way too
      if (b >= head.x) return false;
    }
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

// RB: blocks of 16 ranks. The waves share the part's K in steps of 64, so that the row pieces
// they ask for are whole 128-byte lines: lane l has row l % 16, elements 16 (l / 16) .. + 15 of the
// step, the first 8 for one matrix instruction and the others for the next (both operands take K
// in this order, so it does not matter which element is where). No load
// is under a condition (the compiler waits for one at once): rows behind the tile's last are the
// last one, and what lies behind K is the row's last 8 elements against zeros in A.
template <class T, int RB, int J>
__device__ __forceinline__ void lora_shrink(const LoraArgs& a, const LoraTile& tile, int rank, const int* row_of,
                                            float (&red)[kLoraWaves][kLoraRows][36]) {
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, lq = lane >> 4;
  const int steps = (a.K + 63) / 64, split = tile.part, splits = gridDim.y;
  const int s0 = static_cast<int>(static_cast<int64_t>(steps) * split / splits);
  const int s1 = static_cast<int>(static_cast<int64_t>(steps) * (split + 1) / splits);
  const uint16_t *x[J], *w[RB];
#pragma unroll
  for (int j = 0; j < J; ++j)
    x[j] = static_cast<const uint16_t*>(a.X) + static_cast<int64_t>(row_of[min(16 * j + l16, tile.rows - 1)]) * a.ldx;
#pragma unroll
  for (int i = 0; i < RB; ++i)
    w[i] = static_cast<const uint16_t*>(a.A) +
           (static_cast<int64_t>(tile.adapter) * a.R + min(16 * i + l16, max(rank - 1, 0))) * a.K;
  v4f acc[RB][J];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < J; ++j) acc[i][j] = v4f{};
  typedef v4u Pieces[2][J];
  auto load_x = [&](Pieces& xv, int s) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < J; ++j) xv[h][j] = *reinterpret_cast<const v4u*>(x[j] + min(64 * s + 16 * lq + 8 * h, a.K - 8));
  };
  // a step of the loaded X against A; meanwhile() asks for more of X behind A
  auto multiply = [&](const Pieces& xv, int s, auto meanwhile) {
    v4u wv[2][RB];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < RB; ++i) wv[h][i] = *reinterpret_cast<const v4u*>(w[i] + min(64 * s + 16 * lq + 8 * h, a.K - 8));
    meanwhile();
    if (64 * s + 64 > a.K) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const unsigned keep = 64 * s + 16 * lq + 8 * h < a.K ? ~0u : 0u;
#pragma unroll
        for (int i = 0; i < RB; ++i) wv[h][i] &= keep;
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < J; ++j) acc[i][j] = T::mfma(wv[h][i], xv[h][j], acc[i][j]);
  };
  int s = s0 + wave;
  // X, from memory, a step ahead, as far as there are registers (4096 x 8192 x 8192 of rank 32 75.5 -> 66.0
  // us in all; two steps per wave, 4096 x 4096 x 4096 of rank 16, 36.3 -> 35.8)
  if constexpr (RB <= 6) {
    if (s < s1) {
      Pieces now, next;
      load_x(now, s);
      for (; s + kLoraWaves < s1; s += kLoraWaves) {
        multiply(now, s, [&] { load_x(next, s + kLoraWaves); });
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < J; ++j) now[h][j] = next[h][j];
      }
      multiply(now, s, [] {});
    }
  } else {
    for (; s < s1; s += kLoraWaves) {
      Pieces now;
      load_x(now, s);
      multiply(now, s, [] {});
    }
  }
  // lane l holds row 16 j + l % 16, ranks 16 i + 4 (l / 16) .. + 3: the waves' sums through LDS, 32
  // ranks at a time
  const int R16 = 16 * RB;
#pragma unroll
  for (int i0 = 0; i0 < RB; i0 += 2) {
    if (i0 > 0) __syncthreads();
#pragma unroll
    for (int i = i0; i < i0 + 2 && i < RB; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j) *reinterpret_cast<v4f*>(&red[wave][16 * j + l16][16 * (i - i0) + 4 * lq]) = acc[i][j];
    __syncthreads();
    const int r = tid >> 3, c = 4 * (tid & 7), at = 16 * i0 + c;
    if (r < tile.rows && at < R16) {
      v4f sum = *reinterpret_cast<const v4f*>(&red[0][r][c]);
#pragma unroll
      for (int v = 1; v < kLoraWaves; ++v) sum += *reinterpret_cast<const v4f*>(&red[v][r][c]);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] = at + e < rank ? sum[e] : 0.0f;
      *reinterpret_cast<v4f*>(a.part + (static_cast<int64_t>(split) * a.M + row_of[r]) * R16 + at) = sum;
    }
  }
}

template <class T, int RB>
__global__ __launch_bounds__(64 * kLoraWaves) void k_lora_shrink(LoraArgs a) {
  __shared__ int row_of[kLoraRows];
  __shared__ __attribute__((aligned(16))) float red[kLoraWaves][kLoraRows][36];
  LoraTile tile;
  if (!lora_tile(a, row_of, tile) || tile.adapter < 0) return;
  const int rank = lora_rank(a, tile.adapter);
  if (tile.rows <= 16) lora_shrink<T, RB, 1>(a, tile, rank, row_of, red);
  else if (tile.rows <= 32) lora_shrink<T, RB, 2>(a, tile, rank, row_of, red);
  else lora_shrink<T, RB, 4>(a, tile, rank, row_of, red);
}

// ---- out = Y + scale B V ----

// For up to kLoraFew rows. Features n0 .. n1 of a tile's rows, 32 at a time for each wave: two blocks
// of 16 of B's rows, straight from memory, taken so that a lane ends with 8 consecutive features of a
// row. The next 32 features' Y and B are on their way while these are multiplied and stored, and the
// first ones' while V is put together. No load or store is under a condition, or the compiler would
// wait for all of them where it needs one: rows behind the tile's last are the last one and
// features behind n1 the last 8, and such lanes compute and store the same values again. KS: steps
// of 32 ranks, J: blocks of 16 rows.
template <class T, int KS, int J>
struct LoraExpand {
  typedef typename T::elem v8e __attribute__((ext_vector_type(8)));
  const LoraArgs& a;
  const uint16_t* B;
  int last_row, n1, rank, l16, lq;
  const uint16_t* y_row[J];
  uint16_t* o_row[J];
  struct Operands {
    v4u y[J], b[2][KS];
  };

  __device__ __forceinline__ LoraExpand(const LoraArgs& a_, const LoraTile& tile, int rank_, const int* row_of, int n1_)
      : a(a_), last_row(tile.rows - 1), n1(n1_), rank(rank_) {
    const int lane = threadIdx.x & 63;
    l16 = lane & 15;
    lq = lane >> 4;
    B = static_cast<const uint16_t*>(a.B) + static_cast<int64_t>(tile.adapter) * a.N * a.R;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int64_t m = row_of[min(16 * j + l16, last_row)];
      y_row[j] = static_cast<const uint16_t*>(a.Y) + m * a.ldy;
      o_row[j] = static_cast<uint16_t*>(a.out) + m * a.ldo;
    }
  }
  // first of the 8 features of lane group g
  __device__ __forceinline__ int feature(int n, int g) const { return min(n + 8 * g, n1 - 8); }
  __device__ __forceinline__ void load(Operands& o, int n) const {
#pragma unroll
    for (int j = 0; j < J; ++j) o.y[j] = *reinterpret_cast<const v4u*>(y_row[j] + feature(n, lq));
    // row l % 16 of block h is feature 4 h + l % 4 of lane group l % 16 / 4
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int s = 0; s < KS; ++s)
        o.b[h][s] = *reinterpret_cast<const v4u*>(B + static_cast<int64_t>(feature(n, l16 >> 2) + 4 * h + (l16 & 3)) * a.R +
                                                  min(32 * s + 8 * lq, a.R - 8));
  }
  template <int LR>
  __device__ __forceinline__ void multiply(Operands& o, int n, const typename T::elem (&v)[kLoraParts<T>][kLoraRows][LR],
                                           const float* row_scale) const {
    if (rank < 32 * KS) {  // ranks past this adapter's may hold anything
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const int k = 32 * s + 8 * lq + 2 * d;
          const unsigned keep = (k < rank ? 0xffffu : 0u) | (k + 1 < rank ? 0xffff0000u : 0u);
          o.b[0][s][d] &= keep;
          o.b[1][s][d] &= keep;
        }
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int r = min(16 * j + l16, last_row);
      __builtin_amdgcn_sched_barrier(0);  // V is read for 16 rows at a time: all of it does not fit the registers
      v4f acc[2] = {v4f{}, v4f{}};
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int p = 0; p < kLoraParts<T>; ++p) {
          const v4u x = *reinterpret_cast<const v4u*>(&v[p][r][32 * s + 8 * lq]);
          acc[0] = T::mfma(o.b[0][s], x, acc[0]);
          acc[1] = T::mfma(o.b[1][s], x, acc[1]);
        }
      const float sc = row_scale[r];
      const v8e old = __builtin_bit_cast(v8e, o.y[j]);
      v8e out;
#pragma unroll
      for (int e = 0; e < 8; ++e) out[e] = T::round(__builtin_fmaf(sc, acc[e >> 2][e & 3], static_cast<float>(old[e])));
      *reinterpret_cast<v8e*>(o_row[j] + feature(n, lq)) = out;
    }
  }
};

// f as a sum of kLoraParts<T> values of the type. bf16: 8 bits at a time, cut off rather than rounded, so
// that the largest fp32 values do not become infinite.
template <class T>
__device__ __forceinline__ void lora_parts(float f, typename T::elem (&part)[kLoraParts<T>]) {
#pragma unroll
  for (int p = 0; p < kLoraParts<T>; ++p) {
    if constexpr (T::bf)
      part[p] = __builtin_bit_cast(typename T::elem, static_cast<unsigned short>(__builtin_bit_cast(unsigned, f) >> 16));
    else
      part[p] = T::round(f);
    f -= static_cast<float>(part[p]);
  }
}

// V of the tile's rows: LPR lanes to a row, 4 ranks each; the parts of K, up to SPLITS, together. put(r,
// c, f): ranks c .. c + 3 of row r of the tile.
template <class T, int KS, int THREADS, int SPLITS, class F>
__device__ __forceinline__ void lora_gather_v(const LoraArgs& a, const LoraTile& tile, const int* row_of, float* row_scale,
                                              F put) {
  constexpr int LPR = KS == 1 ? 8 : KS == 2 ? 16 : 32, RPP = THREADS / LPR;
  const int c = 4 * (threadIdx.x % LPR), R16 = (a.R + 15) & ~15;
  for (int r = threadIdx.x / LPR; r < tile.rows; r += RPP) {
    const float* p = a.part + static_cast<int64_t>(row_of[r]) * R16 + min(c, R16 - 4);
    v4f part[SPLITS], sum = v4f{};
#pragma unroll
    for (int i = 0; i < SPLITS; ++i)
      part[i] = *reinterpret_cast<const v4f*>(p + static_cast<int64_t>(min(i, a.splits - 1)) * a.M * R16);
#pragma unroll
    for (int i = 0; i < SPLITS; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] += i < a.splits && c < R16 ? part[i][e] : 0.0f;
    float up = 1.0f, down = 1.0f;
    if constexpr (!T::bf) {
      float most = fmaxf(fmaxf(fabsf(sum[0]), fabsf(sum[1])), fmaxf(fabsf(sum[2]), fabsf(sum[3])));
#pragma unroll
      for (int o = 1; o < LPR; o <<= 1) most = fmaxf(most, __shfl_xor(most, o, 64));
      // the row's largest to [2^14, 2^15)
      const int e = most > 0.0f && most < __builtin_inff() ? 14 - ilogbf(most) : 0;
      up = ldexpf(1.0f, min(max(e, -126), 126));
      down = ldexpf(1.0f, -min(max(e, -126), 126));
    }
    if (c < 32 * KS) put(r, c, sum * up);
    if (c == 0) row_scale[r] = down * (a.scales ? a.scales[tile.adapter] : 1.0f);
  }
}

// Rows without an adapter: out is Y.
template <int THREADS>
__device__ __forceinline__ void lora_copy_rows(const LoraArgs& a, const LoraTile& tile, const int* row_of, int n0, int n1) {
  if (a.Y == a.out) return;
  const int per = (n1 - n0) / 8;
  for (int t = threadIdx.x; t < tile.rows * per; t += THREADS) {
    const int64_t m = row_of[t / per];
    const int n = n0 + t % per * 8;
    *reinterpret_cast<v4u*>(static_cast<uint16_t*>(a.out) + m * a.ldo + n) =
        *reinterpret_cast<const v4u*>(static_cast<const uint16_t*>(a.Y) + m * a.ldy + n);
  }
}

// A workgroup takes a tile's rows and `span` features.
template <class T, int KS, int J, int LR>
__device__ __forceinline__ void lora_expand(const LoraArgs& a, const LoraTile& tile, int rank, const int* row_of,
                                            typename T::elem (&v)[kLoraParts<T>][kLoraRows][LR], float* row_scale, int n0,
                                            int n1) {
  typedef typename T::elem v4e __attribute__((ext_vector_type(4)));
  constexpr int step = 32 * kLoraWaves;
  const LoraExpand<T, KS, J> e(a, tile, rank, row_of, n1);
  int n = n0 + 32 * __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  typename LoraExpand<T, KS, J>::Operands x, y;
  e.load(x, n);
  lora_gather_v<T, KS, 64 * kLoraWaves, kLoraSplits>(a, tile, row_of, row_scale, [&](int r, int c, v4f f) {
    v4e part[kLoraParts<T>];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      typename T::elem of[kLoraParts<T>];
      lora_parts<T>(f[e], of);
#pragma unroll
      for (int p = 0; p < kLoraParts<T>; ++p) part[p][e] = of[p];
    }
#pragma unroll
    for (int p = 0; p < kLoraParts<T>; ++p) *reinterpret_cast<v4e*>(&v[p][r][c]) = part[p];
  });
  lds_barrier();
  for (; n < n1; n += 2 * step) {
    e.load(y, n + step);
    e.multiply(x, n, v, row_scale);
    if (n + step >= n1) break;
    e.load(x, n + 2 * step);
    e.multiply(y, n + step, v, row_scale);
  }
}

template <class T, int KS>
__global__ __launch_bounds__(64 * kLoraWaves) void k_lora_expand(LoraArgs a, int span) {
  constexpr int LR = 32 * KS + 8;  // padded row of a part of V in LDS
  __shared__ int row_of[kLoraRows];
  __shared__ __attribute__((aligned(16))) typename T::elem v[kLoraParts<T>][kLoraRows][LR];
  __shared__ float row_scale[kLoraRows];
  LoraTile tile;
  if (!lora_tile(a, row_of, tile)) return;
  const int n0 = tile.part * span, n1 = min(n0 + span, a.N);
  const int rank = tile.adapter < 0 ? 0 : lora_rank(a, tile.adapter);
  if (rank == 0) {
    lora_copy_rows<64 * kLoraWaves>(a, tile, row_of, n0, n1);
    return;
  }
  if (tile.rows <= 16) lora_expand<T, KS, 1>(a, tile, rank, row_of, v, row_scale, n0, n1);
  else if (tile.rows <= 32) lora_expand<T, KS, 2>(a, tile, rank, row_of, v, row_scale, n0, n1);
  else lora_expand<T, KS, 4>(a, tile, rank, row_of, v, row_scale, n0, n1);
}

// For more than kLoraFew rows. A tile's rows share B: each of four waves has 16 of the rows,
// with their V's parts in registers (V itself comes through LDS in fp32: the parts of rank 128 would leave
// room for one workgroup per CU), and B comes 128 features at a time through LDS (two buffers, filled by
// DMA), read by all four. Of eight blocks of 16 of its rows, block h has the features 8 c + h, so that
// a lane has 8 consecutive features of four rows and 16 lanes together 256 contiguous bytes of a row.
// Y is asked for two steps ahead, and nothing is under a condition, as above.
constexpr int kStagedWaves = 4;
template <class T, int KS>
struct LoraStaged {
  typedef typename T::elem v8e __attribute__((ext_vector_type(8)));
  static constexpr int CPR = 4 * KS, ROWS = 128, BYTES = ROWS * CPR * 16;  // 16-byte pieces of a staged row
  static constexpr int DMAS = BYTES / 1024 / kStagedWaves;
  const LoraArgs& a;
  const uint16_t* B;
  int n1, rank, wave, lane, l16, lq;

  // Row 16 h + c of the buffer is feature 8 c + h, its piece p at p ^ swizzle(c): the 16 rows of a
  // fragment read then lie in different banks.
  static __device__ __forceinline__ int swizzle(int c) { return KS == 4 ? c : KS == 2 ? (c >> 1) & 7 : (c >> 2) & 3; }
  // first of the 8 features of column c (the last 8 behind n1)
  __device__ __forceinline__ int feature(int n, int c) const { return min(n + 8 * c, n1 - 8); }

  // this wave's share of B's rows for features n .. n + 127; pieces past the adapter's rank are zeros
  __device__ __forceinline__ void bring(char* buf, int n) const {
#pragma unroll
    for (int i = 0; i < DMAS; ++i) {
      const int at = (i * kStagedWaves + wave) * 64 + lane, r = at / CPR, c = r & 15, p = (at % CPR) ^ swizzle(c);
      const void* src = 8 * p < rank ? static_cast<const void*>(B + static_cast<int64_t>(feature(n, c) + (r >> 4)) * a.R + 8 * p)
                                     : static_cast<const void*>(kZero16);
      dma16<0>(src, (__attribute__((address_space(3))) void*)(buf + (i * kStagedWaves + wave) * 1024));
    }
  }
  __device__ __forceinline__ v4u piece(const char* buf, int h, int s) const {
    v4u b = *reinterpret_cast<const v4u*>(buf + ((16 * h + l16) * CPR + ((4 * s + lq) ^ swizzle(l16))) * 16);
    if (rank & 7) {  // the adapter's last piece: ranks past its own may hold anything
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const int k = 32 * s + 8 * lq + 2 * d;
        b[d] &= (k < rank ? 0xffffu : 0u) | (k + 1 < rank ? 0xffff0000u : 0u);
      }
    }
    return b;
  }
};

// SPLITS: parts of K at most. The bound on registers, three workgroups per CU up to rank 64, then two, also
// keeps the accumulators out of the other register file, which costs moves (rank 64 in bf16 took 201 of
// 168 without it).
template <class T, int KS, int SPLITS>
__global__ __launch_bounds__(64 * kStagedWaves, KS <= 2 ? 3 : 2) void k_lora_expand_staged(LoraArgs a, int span) {
  typedef LoraStaged<T, KS> Staged;
  typedef typename Staged::v8e v8e;
  typedef float V[kLoraRows][32 * KS + 4];  // padded rows
  __shared__ int row_of[kLoraRows];
  __shared__ float row_scale[kLoraRows];
  __shared__ __attribute__((aligned(1024))) char buf0[Staged::BYTES];
  __shared__ __attribute__((aligned(1024))) char buf1[sizeof(V) > Staged::BYTES ? sizeof(V) : Staged::BYTES];
  V& v = *reinterpret_cast<V*>(buf1);  // until it is in registers
  LoraTile tile;
  if (!lora_tile<true>(a, row_of, tile)) return;
  const int n0 = tile.part * span, n1 = min(n0 + span, a.N);
  const int rank = tile.adapter < 0 ? 0 : lora_rank(a, tile.adapter);
  if (rank == 0) {
    lora_copy_rows<64 * kStagedWaves>(a, tile, row_of, n0, n1);
    return;
  }
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Staged st{a, static_cast<const uint16_t*>(a.B) + static_cast<int64_t>(tile.adapter) * a.N * a.R, n1, rank,
                  wave, lane, lane & 15, lane >> 4};
  st.bring(buf0, n0);
  const uint16_t* y_row[4];
  uint16_t* o_row[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int64_t m = row_of[min(16 * wave + 4 * st.lq + e, tile.rows - 1)];
    y_row[e] = static_cast<const uint16_t*>(a.Y) + m * a.ldy;
    o_row[e] = static_cast<uint16_t*>(a.out) + m * a.ldo;
  }
  auto load_y = [&](v4u (&y)[4], int n) {
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = *reinterpret_cast<const v4u*>(y_row[e] + st.feature(n, st.l16));
  };
  v4u y0[4], y1[4];
  load_y(y0, n0);
  load_y(y1, n0 + 128);
  lora_gather_v<T, KS, 64 * kStagedWaves, SPLITS>(a, tile, row_of, row_scale,
                                                  [&](int r, int c, v4f f) { *reinterpret_cast<v4f*>(&v[r][c]) = f; });
  wait_and_barrier<0>();
  if (16 * wave >= tile.rows) {  // no rows: only its share of B
    lds_barrier();
    for (int n = n0; n < n1; n += 256) {
      if (n > n0) wait_and_barrier<0>();
      st.bring(buf1, n + 128);
      if (n + 128 >= n1) break;
      wait_and_barrier<0>();
      st.bring(buf0, n + 256);
    }
    __builtin_amdgcn_s_waitcnt(0);
    return;
  }
  v4u x[kLoraParts<T>][KS];
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    const float* f = &v[min(16 * wave + st.l16, tile.rows - 1)][32 * s + 8 * st.lq];
    const v4f half[2] = {*reinterpret_cast<const v4f*>(f), *reinterpret_cast<const v4f*>(f + 4)};
    v8e part[kLoraParts<T>];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      typename T::elem of[kLoraParts<T>];
      lora_parts<T>(half[e >> 2][e & 3], of);
#pragma unroll
      for (int p = 0; p < kLoraParts<T>; ++p) part[p][e] = of[p];
    }
#pragma unroll
    for (int p = 0; p < kLoraParts<T>; ++p) x[p][s] = __builtin_bit_cast(v4u, part[p]);
  }
  float sc[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) sc[e] = row_scale[min(16 * wave + 4 * st.lq + e, tile.rows - 1)];
  lds_barrier();  // every wave has its V: the second buffer is free
  auto step = [&](const char* buf, char* other, v4u (&y)[4], int n) {
    st.bring(other, n + 128);
    asm volatile("" ::: "memory");  // what is asked for from here on comes after B's share: the next wait counts on it
    v4f acc[8];
#pragma unroll
    for (int h = 0; h < 8; ++h) acc[h] = v4f{};
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        const v4u b = st.piece(buf, h, s);
#pragma unroll
        for (int p = 0; p < kLoraParts<T>; ++p) acc[h] = T::mfma(x[p][s], b, acc[h]);
      }
    v8e out[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const v8e old = __builtin_bit_cast(v8e, y[e]);
#pragma unroll
      for (int h = 0; h < 8; ++h) out[e][h] = T::round(__builtin_fmaf(sc[e], acc[h][e], static_cast<float>(old[h])));
    }
    load_y(y, n + 256);
#pragma unroll
    for (int e = 0; e < 4; ++e) *reinterpret_cast<v8e*>(o_row[e] + st.feature(n, st.l16)) = out[e];
  };
  for (int n = n0; n < n1; n += 256) {
    // B's share of this step was asked for before the last step's 4 loads and 4 stores
    if (n > n0) wait_and_barrier<8>();
    step(buf0, buf1, y0, n);
    if (n + 128 >= n1) break;
    wait_and_barrier<8>();
    step(buf1, buf0, y1, n + 128);
  }
  __builtin_amdgcn_s_waitcnt(0);  // no DMA may still be writing this workgroup's LDS
}

// Tiles of the rows, as many as there may be.
static int64_t lora_tiles(int64_t M, int64_t S) {
  if (M <= kLoraFew) return S + 1 < M ? S + 1 : M;
  return group_tiles_most(M, S, kLoraRows);
}

// Parts of K: a workgroup of the first product per CU, two of few rows; every workgroup of the second
// reads each part. us in all with 3 / 4 / 6 of them: 3333 x 4096 x 11008, rank 64, 59 tiles 62.2 / 60.2 /
// 62.7; 4096 x 4096 x 4096, rank 16, 72 tiles 33.1 / 35.8 / 34.1; 2048, rank 128, 36 tiles 47.3 / 43.6 / 41.4.
int lora_splits(int64_t M, int64_t K, int64_t S) {
  const int64_t by_tiles = (M <= kLoraFew ? 512 : 264) / lora_tiles(M, S), by_k = K / (64 * kLoraWaves);
  const int64_t n = by_tiles < by_k ? by_tiles : by_k;
  return static_cast<int>(n < 1 ? 1 : n > kLoraSplits ? kLoraSplits : n);
}

template <class T, int SPLITS>
static void expand_staged(const LoraArgs& a, dim3 expand, int span, hipStream_t s) {
  switch ((a.R + 31) / 32) {
    case 1: hipLaunchKernelGGL((k_lora_expand_staged<T, 1, SPLITS>), expand, dim3(64 * kStagedWaves), 0, s, a, span); break;
    case 2: hipLaunchKernelGGL((k_lora_expand_staged<T, 2, SPLITS>), expand, dim3(64 * kStagedWaves), 0, s, a, span); break;
    case 3: hipLaunchKernelGGL((k_lora_expand_staged<T, 3, SPLITS>), expand, dim3(64 * kStagedWaves), 0, s, a, span); break;
    default: hipLaunchKernelGGL((k_lora_expand_staged<T, 4, SPLITS>), expand, dim3(64 * kStagedWaves), 0, s, a, span); break;
  }
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
  // features per workgroup: as many workgroups as the GPU holds, of the staged expand three per CU up to
  // rank 64, then two (3000 x 8192 x 10240, rank 128: 768 workgroups 98.2 us, 512 87.8)
  const bool few = a.M <= kLoraFew;
  const int round = few ? 32 * kLoraWaves : 128;
  const int64_t room = few || a.R > 64 ? 512 : 768, per = room / tiles < 1 ? 1 : room / tiles;
  const int span = static_cast<int>(((a.N + per - 1) / per + round - 1) / round * round);
  const dim3 expand(tiles, (a.N + span - 1) / span);
  if (!few) {
    if (a.splits <= kLoraSplits / 2) expand_staged<T, kLoraSplits / 2>(a, expand, span, s);
    else expand_staged<T, kLoraSplits>(a, expand, span, s);
    return hipGetLastError();
  }
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
