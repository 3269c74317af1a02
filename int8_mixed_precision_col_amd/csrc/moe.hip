// A mixture-of-experts layer for at most 16 tokens, in two launches.
//
// For token t with router logits l [E]: the top_k experts of the largest logits (ties to the
// lowest index; an expert at -inf is off), weights p_e = exp(l_e - max l) over the sum of
// the chosen ones (renormalize) or of all experts, and
//   y_t = sum_e p_e Down_e (silu(Gate_e x_t) * (Up_e x_t)),  silu(g) = g / (1 + exp(-g)),
// with int8 or MX4 expert weights and 16-bit activations, fp32 accumulation and one rounding
// of y. It is the weights of the chosen experts that bound it: each is read once.
//
// k_moe_gate_up: every workgroup works out the routing for itself (T x E logits, a few KB
// from L2, one wave per token) rather than wait for a launch of its own: 1.4 us for up to 8
// tokens, 2.8 for 16. The gate and up rows of all chosen experts, 16 + 16 features at a time,
// are one list of steps that 256 workgroups, one per CU, share evenly, whatever the number of
// experts turns out to be; a workgroup goes over its part with the next step's weights in
// flight while it multiplies, adds up its waves and writes the hidden values of the tokens
// that chose the expert.
// k_moe_down: a workgroup per 16 output features goes over all chosen experts, its waves
// sharing the (pass, K quad) items in order (a pass: up to four tokens of one expert), so
// that the weighted sum over experts needs no third launch and is the same on every run. With
// few features several workgroups share 16 of them, and the last one there adds up their sums.
//
// The hidden values stay fp32 between the launches, and enter the matrix instructions as three
// bf16 parts of 8 significant bits, 24 together. The parts cost no matrix instructions: a pass
// has four tokens, so rows 0-3, 4-7 and 8-11 of the 16-row operand hold their first, second
// and third parts, and the three sums are added in the end.
//
// Measured (us per layer in graphs over rotated weights; bytes of the chosen experts over that
// time): 16 tokens, 8 of 64 experts of 4096 x 1280, int8 165 us, 5.4 TB/s, MX4 102 us, 4.6 TB/s;
// of 2048 x 768 65 and 49.5 us; 1 token of these 17.9 and 15.0 us, of which 7.5 and 4.0 us are the
// bytes at 5 TB/s and the rest two chains of launch, routing or tables, first loads and join.
#include "moe_keys.hpp"
#include "mx4_launch.hpp"
#include "weight_stream.hpp"

namespace i8mm {

constexpr int kMoeMaxLists = kMoeMaxTokens * kMoeMaxTopK;
constexpr int kMoeExpertWords = kMoeMaxExperts / 32;

// The chosen experts of all tokens, in LDS: a bit per expert that some token chose, and per
// expert the mask of its tokens and its place in each one's list. The experts are used in
// ascending order; `slot` is a place there.
struct MoeTable {
  unsigned on[kMoeExpertWords], tokens[kMoeMaxExperts];
  uint8_t place[kMoeMaxExperts * kMoeMaxTokens];

  __device__ __forceinline__ void clear(int tid, int threads) {
    if (tid < kMoeExpertWords) on[tid] = 0u;
    for (int i = tid; i < kMoeMaxExperts; i += threads) tokens[i] = 0u;
  }
  __device__ __forceinline__ void add(int expert, int t, int j) {
    atomicOr(&on[expert >> 5], 1u << (expert & 31));
    atomicOr(&tokens[expert], 1u << t);
    place[expert * kMoeMaxTokens + t] = static_cast<uint8_t>(j);
  }
};

// A wave's view of MoeTable::on: word i and the number of experts up to its end in lane i.
struct MoeOrder {
  int word, upto;
  __device__ __forceinline__ MoeOrder(const MoeTable& t, int lane) {
    word = lane < kMoeExpertWords ? static_cast<int>(t.on[lane]) : 0;
    upto = wave_prefix_sum(__builtin_popcount(static_cast<unsigned>(word)));
  }
  __device__ __forceinline__ int count() const { return __builtin_amdgcn_readlane(upto, 63); }
  __device__ __forceinline__ int expert(int slot) const {  // slot < count()
    const int at = __builtin_ctzll(__ballot(upto > slot));
    unsigned bits = static_cast<unsigned>(__builtin_amdgcn_readlane(word, at));
    int before = slot - (__builtin_amdgcn_readlane(upto, at) - __builtin_popcount(bits));
    while (before-- > 0) bits &= bits - 1;
    return 32 * at + __builtin_ctz(bits);
  }
};

// One wave routes NT tokens, two of them side by side (a token's rounds are one chain of
// dependent steps). Lane l holds experts V l .. V l + V - 1, so that the lowest lane and then
// the lowest of its experts is the lowest index.
template <int V, int NT>
struct MoeRouter {
  int token[NT];
  unsigned key[NT][V];

  // tokens t, t + stride (past T: every expert is off)
  __device__ __forceinline__ MoeRouter(const MoeArgs& a, int t, int stride, int lane) {
#pragma unroll
    for (int p = 0; p < NT; ++p) {
      token[p] = t + p * stride;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = V * lane + i;
        key[p][i] = token[p] < a.T && e < a.E
                        ? moe_key(moe_logit(a.logits, a.logits_type, static_cast<int64_t>(token[p]) * a.E + e))
                        : 0u;
      }
    }
  }

  // enters the chosen experts into the table; writes the lists where ids is given (id -1 and
  // weight 0 past the last expert that is on)
  __device__ __forceinline__ void route(const MoeArgs& a, int lane, MoeTable& table, int* ids, float* weights) {
    unsigned kept[NT][V], first[NT], mine[NT];  // the keys; the largest; lane j: that of place j
    int mine_id[NT];
#pragma unroll
    for (int p = 0; p < NT; ++p) {
      first[p] = mine[p] = 0;
      mine_id[p] = -1;
#pragma unroll
      for (int i = 0; i < V; ++i) kept[p][i] = key[p][i];
    }
    for (int j = 0; j < a.k; ++j) {
#pragma unroll
      for (int p = 0; p < NT; ++p) {
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
        const int id = V * who + (V > 1 ? __builtin_amdgcn_readlane(at, who) : 0);
        if (j == 0) first[p] = top;
        if (lane == j && top) {
          mine[p] = top;
          mine_id[p] = id;
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (V * lane + i == id) key[p][i] = 0u;
      }
    }
#pragma unroll
    for (int p = 0; p < NT; ++p)
      if (mine_id[p] >= 0) table.add(mine_id[p], token[p], lane);
    if (!ids) return;
#pragma unroll
    for (int p = 0; p < NT; ++p) {
      const float most = moe_unkey(first[p]);
      const float w = mine[p] ? expf(moe_unkey(mine[p]) - most) : 0.0f;
      float sum = w;
      if (!a.renormalize) {
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) sum += kept[p][i] ? expf(moe_unkey(kept[p][i]) - most) : 0.0f;
      }
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
      if (lane < a.k && token[p] < a.T) {
        const float share = mine_id[p] < 0 ? 0.0f : __fdiv_rn(w, sum);
        const int o = token[p] * a.k + lane;
        ids[o] = mine_id[p];
        weights[o] = share;
        if (a.ids) a.ids[o] = mine_id[p];
        if (a.weights) a.weights[o] = share;
      }
    }
  }
};

constexpr int kUpWaves = 8;
// LDS for the activations of k_moe_gate_up: with all of X in it (T x D up to 64 K elements) X
// is read once per workgroup, while the routing is worked out; otherwise each wave reads the
// quad it multiplies, of the tokens that chose the expert.
constexpr int kUpResident = 132 << 10;
template <bool MX>
__host__ __device__ __forceinline__ bool up_resident(int T, int quads) {
  return quads * act_bytes<MX>(T) <= kUpResident;
}

// Workgroups of k_moe_gate_up: one per CU. Two for each (they fit with int8 weights and X in LDS, in
// 126 registers) gain nothing that a rule could go by: of 8 of 64 experts with I = 768 / 1280, one
// against two, 2 tokens of D = 2048 24.8 / 25.8, 39.5 / 40.3 us, 3328 33.6 / 33.4, 47.8 / 48.5, 4096
// 36.0 / 35.4, 53.9 / 50.3, 5120 49.0 / 49.8, 73.1 / 76.6, 7168 56.4 / 56.5, 88.0 / 83.1; 4 tokens of
// 4096 53.3 / 49.9, 84.3 / 80.8, 5120 74.3 / 78.1, 108.8 / 107.6.
constexpr int kMoeBlocks = 256;

// What k_moe_gate_up leaves for k_moe_down (with the hidden values), and what its workgroups
// leave for each other.
struct MoeLists {
  int* ids;        // [kMoeMaxLists]
  float* weights;  // [kMoeMaxLists]
  int* arrived;    // [kMoeBlocks] zeros
  float* sums;     // [kMoeBlocks][256]
};

// Waves that share the quads of a group: a workgroup's steps each cost a turn per quad of a wave
// and about as much again for the sums' exchange and the hidden values, so the fewest of
// steps x (1 + turns). Few sharers exchange little and give each wave loads to have in flight
// over a step's end; many leave fewer features to the last step. Measured, us per layer at 8 /
// 4 / 2 sharers: 16 tokens, 8 of 64 experts of 4096 x 1280, MX4 116 / 104 / 106, int8 171 / 171 /
// 171 (chosen by cost 167); of 2048 x 768, int8 70 / 65.5 / 64.6, 4 tokens 39.7 / 37.6 / 38.7, 1 token
// 19.8 / 18.6 / 21.4; 1 token of 4096 x 1280, MX4 26.1 / 25.7 / 24.1. (One, with the hidden values in two
// parts: 102 and 179 for the first two, where two sharers took 97 and 167.)
template <bool MX>
__device__ __forceinline__ int up_share(int experts, int groups, int quads) {
  const int most = quads >= 5 ? 8 : quads >= 3 ? 4 : MX ? quads : 2;  // int8: at most four groups at once
  int best = most, least = 0x7fffffff;
  for (int share = most; share >= 2 || share == most; share >>= 1) {
    const int par = kUpWaves / share, steps = experts * ((groups + par - 1) / par);
    const int cost = (steps + kMoeBlocks - 1) / kMoeBlocks * (1 + (quads + share - 1) / share);
    if (cost < least) {
      least = cost;
      best = share;
    }
  }
  return best;
}

// V experts per lane and NT tokens per wave in the routing; RES: all of X in LDS. Kernels of their
// own rather than branches of one: a launch runs a few KB of code, once, and finds it faster in
// 8 KB than in 37 (1 token, 8 of 64 experts of 2048 x 768, int8 20.9 -> 19.2 us; 8 tokens of 4096 x
// 1280, MX4, 79 -> 73 us).
template <class T, bool MX, int V, int NT, bool RES>
__global__ __launch_bounds__(64 * kUpWaves, 2) void k_moe_gate_up(MoeArgs a, MoeLists lists) {
  extern __shared__ __attribute__((aligned(16))) char s_x[];  // [quads or waves][act_bytes(T)]
  __shared__ MoeTable table;
  __shared__ float red[kUpWaves][2][16][17];
  __shared__ float s_col[128];  // int8: gate and up constants of the step's groups, over 127
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  constexpr int UK = WeightFmt<MX>::UK;
  const int ks = (a.D + UK - 1) / UK, quads = (ks + 3) >> 2, groups = a.I / 16;
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.X, static_cast<unsigned>(((a.T - 1) * a.ldx + a.D) * 2));
  // the logits first, then X: both are on their way while the table is cleared and the wave
  // routes its tokens
  static_assert(2 * kUpWaves >= kMoeMaxTokens, "two tokens per wave");
  auto row_of = [&](int t) { return static_cast<unsigned>(t * a.ldx) * 2u; };
  ActQuad<MX, 8 * NT> x;
  MoeRouter<V, NT> router(a, wave, kUpWaves, lane);
  if (RES && wave < quads) x.load(xr, wave, a.D, a.T, lane, row_of);
  table.clear(tid, 64 * kUpWaves);
  lds_barrier();
  // One workgroup writes what the second launch goes by, all of it from its own view of the
  // logits, so that it is consistent whatever else happens to them meanwhile.
  router.route(a, lane, table, blockIdx.x == 0 ? lists.ids : nullptr, lists.weights);
  if (!MX && blockIdx.x == 0 && tid < kMoeBlocks) lists.arrived[tid] = 0;
  lds_barrier();
  const MoeOrder order(table, lane);

  // A step is `par` neighbouring 16-feature groups of one expert, `share` waves on the quads
  // of each.
  const int share = up_share<MX>(order.count(), groups, quads);
  const int par = kUpWaves / share;
  const int steps = (groups + par - 1) / par;
  // steps [first, last) of the list are this workgroup's
  const unsigned all = static_cast<unsigned>(order.count() * steps), some = all / gridDim.x, more = all % gridDim.x;
  const unsigned first = blockIdx.x * some + min(blockIdx.x, more);
  const int n_steps = static_cast<int>(some + (blockIdx.x < more ? 1u : 0u));
  if (n_steps == 0) return;
  int slot = static_cast<int>(first / steps), in = static_cast<int>(first % steps);  // its place in the expert
  const int sub = wave / share, kk = wave - sub * share;

  WeightQuad<MX> next[2];
  auto prefetch = [&](int e, int at, int q) {
    const int group = min(at * par + sub, groups - 1);
    const size_t gate = static_cast<size_t>(e) * 2 * groups + group;
    next[0].load(a.w13, static_cast<const uint32_t*>(a.s13), gate, ks, quads, q, lane);
    next[1].load(a.w13, static_cast<const uint32_t*>(a.s13), gate + groups, ks, quads, q, lane);
  };
  // unconditional (a wave without a quad repeats the last), so that the wait for X below counts
  // these loads and does not wait for them
  int expert = order.expert(slot);
  prefetch(expert, in, min(kk, quads - 1));
  if constexpr (RES) {
    if (wave < quads) x.store(s_x + wave * act_bytes<MX>(a.T), a.T, a.T, lane);
    for (int q = wave + kUpWaves; q < quads; q += kUpWaves) {
      x.load(xr, q, a.D, a.T, lane, row_of);
      x.store(s_x + q * act_bytes<MX>(a.T), a.T, a.T, lane);
    }
  }
  lds_barrier();
  const int row = min(lane & 15, a.T - 1);  // rows past T repeat the last (discarded)
  for (int step = 0; step < n_steps; ++step) {
    const unsigned tokens = __builtin_amdgcn_readfirstlane(table.tokens[expert]);
    const int next_in = in + 1 < steps ? in + 1 : 0;
    const int next_expert = next_in == 0 && step + 1 < n_steps ? order.expert(slot + 1) : expert;
    // int8: the step's column constants, one per thread. Asked for here, in front of the next
    // step's weights: loads return in order, so that a wait for them behind those waits for both
    // (with the down product's: 16 tokens, 8 of 64 experts of 4096 x 1280, 158 -> 152 us).
    float col = 0.0f;
    if (!MX && tid < 128) {
      const int group = min(in * par + ((tid >> 4) & 3), groups - 1);
      col = static_cast<const float*>(a.s13)[(static_cast<size_t>(expert) * 2 * groups + group) * 16 + (tid & 15) +
                                             (tid < 64 ? 0 : a.I)];
    }
    v4f acc[2] = {};
    for (int q = kk; q < quads; q += share) {
      const char* buf = s_x + (RES ? q : wave) * act_bytes<MX>(a.T);
      if constexpr (!RES) {
        x.load(xr, q, a.D, a.T, lane, [&](int t) { return (tokens >> t) & 1u ? row_of(t) : kOOB; });
        wave_lds_fence();
        x.store(s_x + wave * act_bytes<MX>(a.T), a.T, a.T, lane);
        wave_lds_fence();
      }
      WeightQuad<MX> w[2] = {next[0], next[1]};
      if (q + share < quads) prefetch(expert, in, q + share);
      else if (step + 1 < n_steps) prefetch(next_expert, next_in, kk);
      mma_quad<T, MX, 2>(w, acc, [&](int j, int v) { return act_operand<MX>(buf, a.T, row, j, v, lane); });
    }
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[wave][p][4 * (lane >> 4) + e][lane & 15] = acc[p][e];
    if (!MX && tid < 128) s_col[tid] = __fdiv_rn(col, 127.0f);
    lds_barrier();
    for (int o = tid; o < 256 * par; o += 64 * kUpWaves) {
      const int n = o & 15, t = (o >> 4) & 15, s = o >> 8;
      const int group = in * par + s;
      if (group >= groups || !((tokens >> t) & 1u)) continue;
      float g = 0.0f, u = 0.0f;
      for (int w = 0; w < share; ++w) {
        g += red[s * share + w][0][t][n];
        u += red[s * share + w][1][t][n];
      }
      if constexpr (!MX) {
        g *= s_col[16 * s + n];
        u *= s_col[64 + 16 * s + n];
      }
      const float h = __fdiv_rn(g, 1.0f + expf(-g)) * u;
      const int list = t * a.k + table.place[expert * kMoeMaxTokens + t];
      a.h[static_cast<size_t>(list) * a.I + group * 16 + n] = h;
    }
    lds_barrier();  // red is read
    slot += next_in == 0;
    in = next_in;
    expert = next_expert;
  }
}

// A pass over an expert's quads serves TOK of its tokens (kMoeParts TOK rows); further ones read
// its weights again, from a cache. Eight tokens per pass (measured with two parts each) leave
// LDS for 8 waves instead of 16: 132 for 114 us (16 tokens, 8 of 64 experts of 2048 x 1280,
// int8), 112.6 for 111.2 (8 of 32 of 4096 x 1280), 51.8 for 51.0 (4 of 8), 24.3 for 21.9 (one
// expert), and at best 39.9 for 41.5 (8 tokens, 4 of 8). A load of the next item's h ahead of the
// products, as the weights', leaves 8 waves too for MX4 (111 for 97 us, 16 tokens of 4096 x
// 1280) and gave nothing where 16 fit (int8).
constexpr int kDownWaves = 16, kDownTokens = 4;
constexpr int kMoeParts = 3;  // bf16 parts of a hidden value
constexpr float kMoeMost = 0x1p127f;

// The hidden values of one quad for a pass of m tokens, a token's piece (1 KB) per load, split into
// bf16 parts on the way to the wave's LDS buffer: part p of token c is its row kDownTokens p + c. The
// parts are cut off (a value's leading 8 significant bits are its upper half), not rounded, and
// both remainders are exact. Split here, a hidden value is 4 bytes of what a CU takes in; as three bf16
// planes from the first launch it was 6 (16 tokens, 8 of 64 experts of 4096 x 1280, MX4, 111 against 101
// us; of 2048 x 768 53.5 against 49).
template <bool MX>
struct HiddenQuad {
  static constexpr int P = ActQuad<MX, 2>::P;
  v4u raw[P][kDownTokens];

  // off[c]: byte offset of token c's row
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, int q, int I, int m, int lane,
                                       const unsigned (&off)[kDownTokens]) {
#pragma unroll
    for (int v = 0; v < P; ++v) {
      const int k = (P * q + v) * kActPiece + 4 * lane;
#pragma unroll
      for (int c = 0; c < kDownTokens; ++c)
        if (c < m) raw[v][c] = buf_load16(r, k < I ? 4u * k : kOOB, off[c]);
    }
  }
  __device__ __forceinline__ void store_piece(int v, char* buf, int m, int lane) const {
#pragma unroll
    for (int c = 0; c < kDownTokens; ++c)
      if (c < m) {
        v2u part[kMoeParts];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          unsigned f[2] = {raw[v][c][2 * e], raw[v][c][2 * e + 1]};
#pragma unroll
          for (int p = 0; p < kMoeParts; ++p) {
            part[p][e] = __builtin_amdgcn_perm(f[1], f[0], 0x07060302u);
#pragma unroll
            for (int d = 0; d < 2; ++d) {
              float rest = __builtin_bit_cast(float, f[d]) - __builtin_bit_cast(float, f[d] & 0xffff0000u);
              // an infinity is all in its first part; the median of NaN and these is finite
              if (p == 0) rest = __builtin_amdgcn_fmed3f(rest, -kMoeMost, kMoeMost);
              f[d] = __builtin_bit_cast(unsigned, rest);
            }
          }
        }
#pragma unroll
        for (int p = 0; p < kMoeParts; ++p)
          *reinterpret_cast<v2u*>(buf + (kDownTokens * p + c) * kActStride + 8 * lane) = part[p];
      }
  }
};

// SPLIT: gridDim.y workgroups share the items of 16 features. Each writes its sums, [T][16], and
// counts itself in; the last adds them up in order, so the result does not depend on which that
// is. Nobody waits for another workgroup.
template <class T, bool MX, bool SPLIT>
__global__ __launch_bounds__(64 * kDownWaves) void k_moe_down(MoeArgs a, MoeLists lists) {
  constexpr int WAVES = kDownWaves, TOK = kDownTokens, ROWS = kMoeParts * TOK;
  __shared__ __attribute__((aligned(16))) char s_x[WAVES * ROWS * kActStride];
  __shared__ unsigned s_tokens[kMoeMaxExperts];
  __shared__ uint8_t s_place[kMoeMaxExperts * kMoeMaxTokens];
  __shared__ uint64_t s_first[kMoeMaxLists / 64];
  __shared__ float s_w[kMoeMaxLists];
  // passes: expert, number of tokens, and by token (bytes) the list entry and the token
  __shared__ __attribute__((aligned(16))) v4i s_pass[kMoeMaxLists];
  __shared__ __attribute__((aligned(16))) v4f s_share[kMoeMaxLists];  // by token its weight
  __shared__ float total[WAVES][kMoeMaxTokens][17];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n_lists = a.T * a.k;
  char* buf = s_x + wave * ROWS * kActStride;
  int id = -1;
  float weight = 0.0f;
  if (tid < n_lists) {
    id = lists.ids[tid];
    weight = lists.weights[tid];
  }
  for (int i = tid; i < a.E; i += 64 * WAVES) s_tokens[i] = 0u;
  for (int i = lane; i < kMoeMaxTokens * 17; i += 64) (&total[wave][0][0])[i] = 0.0f;
  lds_barrier();
  // Addresses come out of the ids: checked here too, so that a workspace that another call
  // wrote to meanwhile, which the interface forbids, gives wrong values at worst.
  const int t_of = tid / a.k;
  if (id >= a.E) id = -1;
  if (id >= 0) {
    atomicOr(&s_tokens[id], 1u << t_of);
    s_place[id * kMoeMaxTokens + t_of] = static_cast<uint8_t>(tid - t_of * a.k);
  }
  if (tid < n_lists) s_w[tid] = weight;
  lds_barrier();
  // Passes: TOK tokens of one expert, each written by the list entry of its first token and kept
  // in that order. A pass is a wave's unit whatever its expert, so that an expert with many
  // tokens does not hold up one wave.
  const int before = id < 0 ? 0 : __builtin_popcount(s_tokens[id] & ((1u << (t_of & 31)) - 1));
  const uint64_t starts = __ballot(id >= 0 && before % TOK == 0);
  if (lane == 0 && wave < kMoeMaxLists / 64) s_first[wave] = starts;
  lds_barrier();
  int passes = 0, mine = 0;
#pragma unroll
  for (int i = 0; i < kMoeMaxLists / 64; ++i) {
    if (i == wave) mine = passes;
    passes += __builtin_popcountll(s_first[i]);
  }
  if (id >= 0 && before % TOK == 0) {
    static_assert(TOK == 4, "four bytes, four weights");
    unsigned left = s_tokens[id] & ~((1u << t_of) - 1), entries = 0, tokens = 0;
    v4f w = {};
    const int m = min(__builtin_popcount(left), TOK);
#pragma unroll
    for (int c = 0; c < TOK; ++c)
      if (c < m) {
        const int t = __builtin_ctz(left), entry = t * a.k + s_place[id * kMoeMaxTokens + t];
        left &= left - 1;
        entries |= static_cast<unsigned>(entry) << (8 * c);
        tokens |= static_cast<unsigned>(t) << (8 * c);
        w[c] = s_w[entry];
      }
    const int pass = mine + __builtin_popcountll(starts & ((uint64_t(1) << lane) - 1));
    s_pass[pass] = v4i{id, m, static_cast<int>(entries), static_cast<int>(tokens)};
    s_share[pass] = w;
  }
  lds_barrier();
  passes = __builtin_amdgcn_readfirstlane(passes);

  constexpr int UK = WeightFmt<MX>::UK;
  const int ks = (a.I + UK - 1) / UK, quads = (ks + 3) >> 2;
  const int parts = SPLIT ? gridDim.y : 1, waves = WAVES * parts, at = SPLIT ? blockIdx.y * WAVES + wave : wave;
  const int items = passes * quads, per = (items + waves - 1) / waves;
  int begin = min(items, per * at), end = min(items, begin + per);
  // With waves for every pass no wave's share crosses into a second pass, whose rows it would
  // have to wait for again; neighbouring waves, on different SIMDs, take different passes (1
  // token, 8 of 64 experts of 2048 x 768, int8 19.4 -> 18.6 us, of 4096 x 1280 36.4 -> 35.6; with
  // neighbours on the same pass, so on two SIMDs, 4 of 32 of 1024 x 512 11.9 -> 13.3).
  if (passes > 0 && passes <= waves) {
    const int share = waves / passes, n = (quads + share - 1) / share, s = at / passes, p = at - s * passes;
    if (n <= per) {
      begin = p * quads + min(quads, s * n);
      end = p * quads + min(quads, (s + 1) * n);
      if (s >= share) begin = end = 0;
    }
  }
  const unsigned plane = static_cast<unsigned>(n_lists) * a.I * 4u;  // bytes
  const __amdgpu_buffer_rsrc_t hr = make_rsrc(a.h, plane);
  const int r = lane & 15, g = lane >> 4;
  WeightQuad<MX> next;
  float col = 1.0f, col_next = 1.0f;  // int8: the feature's column constant
  auto prefetch = [&](int expert, int q) {
    next.load(a.w2, static_cast<const uint32_t*>(a.s2), static_cast<size_t>(expert) * (a.D / 16) + blockIdx.x, ks, quads,
              q, lane);
  };
  // the first quad of a wave's share of a pass, in front of it the constant (loads return in order)
  auto enter = [&](int pass, int q) {
    const int expert = __builtin_amdgcn_readfirstlane(s_pass[pass][0]);
    if constexpr (!MX) col_next = static_cast<const float*>(a.s2)[static_cast<size_t>(expert) * a.D + blockIdx.x * 16 + r];
    prefetch(expert, q);
  };
  int pass = begin / quads;
  if (begin < end) enter(pass, begin - pass * quads);
  for (int i = begin; i < end; ++pass) {
    // items [i, stop) are quads of one pass, the wave's share of it
    const int q0 = i - pass * quads, stop = min(end, (pass + 1) * quads), q1 = stop - pass * quads;
    i = stop;
    const v4i p = s_pass[pass];
    const int expert = __builtin_amdgcn_readfirstlane(p[0]), m = __builtin_amdgcn_readfirstlane(p[1]);
    const unsigned entries = __builtin_amdgcn_readfirstlane(p[2]), tokens = __builtin_amdgcn_readfirstlane(p[3]);
    col = col_next;
    unsigned off[TOK];
#pragma unroll
    for (int c = 0; c < TOK; ++c) off[c] = ((entries >> (8 * c)) & 255u) * (a.I * 4u);
    // operand rows TOK p .. are part p of the tokens, those past m and past the parts repeat one
    const int row = TOK * min(r / TOK, kMoeParts - 1) + min(r % TOK, m - 1);
    v4f acc[1] = {};
    for (int q = q0; q < q1; ++q) {
      WeightQuad<MX> w[1] = {next};
      HiddenQuad<MX> x;
      x.load(hr, q, a.I, m, lane, off);
      // The hidden values are here before the next weights are asked for: behind them, with the
      // number of loads in flight known at run time alone, a wait for them would be one for all
      // (1 token, 8 of 64 experts of 2048 x 768, int8 18.6 -> 17.9 us; 16 tokens 66.8 -> 65.4).
      wave_load_fence();
      if (q + 1 < q1) prefetch(expert, q + 1);
      else if (i < end) enter(pass + 1, 0);
      wave_lds_fence();
      x.store_piece(0, buf, m, lane);
      wave_lds_fence();
      constexpr int HALF = MX ? 2 : 4;
      mma_quad<B16, MX, 1, 0, HALF>(w, acc, [&](int j, int v) { return act_operand<MX>(buf, 0, row, j, v, lane); });
      if constexpr (MX) {
        wave_lds_fence();
        x.store_piece(1, buf, m, lane);
        wave_lds_fence();
        mma_quad<B16, MX, 1, 2, 4>(w, acc, [&](int j, int v) { return act_operand<MX>(buf, 0, row, j, v, lane); });
      }
    }
    // weigh the sums into the tokens': lane r of group p holds the sums of the tokens' part p
    static_assert(TOK == 4 && kMoeParts == 3, "a lane group's four rows are one part");
    const v4f weights = s_share[pass];
    const float scale = MX ? 1.0f : __fdiv_rn(col, 127.0f);
#pragma unroll
    for (int c = 0; c < TOK; ++c) {
      const float y = acc[0][c] + (__shfl_xor(acc[0][c], 16, 64) + __shfl_xor(acc[0][c], 32, 64));
      if (g == 0 && c < m) total[wave][(tokens >> (8 * c)) & 255u][r] += y * scale * weights[c];
    }
  }
  lds_barrier();
  const int t = tid >> 4, f = tid & 15;
  float y = 0.0f;
  if (t < a.T) {
#pragma unroll
    for (int w = 0; w < WAVES; ++w) y += total[w][t][f];
  }
  if constexpr (SPLIT) {
    // The sums pass through memory that every XCD sees: written and read as device-scope atomics,
    // ordered by the count, one release and acquire per workgroup (a fence in every wave took
    // 30 us).
    __shared__ bool s_last;
    float* sums = lists.sums + (static_cast<size_t>(blockIdx.x) * parts) * 256 + tid;
    if (t < a.T) __hip_atomic_store(sums + blockIdx.y * 256, y, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (tid == 0)
      s_last = __hip_atomic_fetch_add(lists.arrived + blockIdx.x, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == parts - 1;
    __syncthreads();
    if (!s_last) return;
    y = 0.0f;
    if (t < a.T)
      for (int p = 0; p < parts; ++p) y += __hip_atomic_load(sums + p * 256, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (t < a.T)
    static_cast<typename T::elem*>(a.Y)[static_cast<size_t>(t) * a.D + blockIdx.x * 16 + f] = T::round(y);
}

template <class T, bool MX, int V, int NT, bool RES>
static hipError_t run_up(const MoeArgs& a, const MoeLists& lists, hipStream_t s) {
  const int n_slots = a.E < a.T * a.k ? a.E : a.T * a.k;
  constexpr int UK = WeightFmt<MX>::UK;
  const int quads = ((a.D + UK - 1) / UK + 3) / 4;
  const size_t lds = static_cast<size_t>(RES ? quads : kUpWaves) * act_bytes<MX>(a.T);
  constexpr size_t kStatic = sizeof(MoeTable) + sizeof(float) * (kUpWaves * 2 * 16 * 17 + 128);
  static_assert(kUpResident + kStatic <= kMaxLds && kUpWaves * act_bytes<MX>(kMoeMaxTokens) + kStatic <= kMaxLds,
                "k_moe_gate_up's LDS");
  const int64_t steps = static_cast<int64_t>(n_slots) * (a.I / 16);
  const unsigned blocks = static_cast<unsigned>(steps < kMoeBlocks ? steps : kMoeBlocks);
  hipLaunchKernelGGL((k_moe_gate_up<T, MX, V, NT, RES>), dim3(blocks), dim3(64 * kUpWaves), lds, s, a, lists);
  return hipGetLastError();
}

// Workgroups that share 16 features of Y: few features leave CUs idle, the more items of a wave
// the longer; the exchange costs 1 us and about another per 64 workgroups. int8, at least three items per
// wave saved (by the most passes that the lists can have). One workgroup against the split taken: 8 of 64
// experts of 2048 x 768, 4 / 8 / 16 tokens 37.7 / 37.3, 51.8 / 48.0, 68.3 / 63.4 us; 4 of 60 of 2048 x 1408, 16
// tokens 89.5 / 78.5; 2 of 16 of 512 x 2048, four workgroups, 4 / 16 tokens 19.3 / 17.2, 34.0 / 24.4, but 8 tokens
// of 1024 x 1024 19.9 / 22.1; with fewer saved, 2 tokens of 2048 x 768 24.8 / 26.8. Over 125 layers of 256 to
// 2048 features the choice is 0.7% from the best of one, two and four. An MX4 item is half as long (with hidden
// values in two parts): 16 tokens 48.0 / 46.2, 49.4 / 50.8, 8 tokens 38.3 / 37.2, 38.6 / 41.6: not worth it.
static int down_parts(const MoeArgs& a, int quads) {
  const int parts = a.D <= 16 * kMoeBlocks / 4 ? 4 : a.D <= 16 * kMoeBlocks / 2 ? 2 : 1;
  const int n = a.T * a.k, most = a.E + n / kDownTokens, passes = n < most ? n : most;
  const int per = (passes * quads + kDownWaves - 1) / kDownWaves, split = (per + parts - 1) / parts;
  return per - split >= 3 ? parts : 1;
}

template <class T, bool MX>
static hipError_t run(const MoeArgs& a, const MoeLists& lists, hipStream_t s) {
  constexpr int UK = WeightFmt<MX>::UK, V = kMoeMaxExperts / 64;
  const bool few = a.T <= kUpWaves, small = a.E <= 64;
  hipError_t e;
  if (!up_resident<MX>(a.T, ((a.D + UK - 1) / UK + 3) / 4)) e = run_up<T, MX, V, 2, false>(a, lists, s);
  else if (few) e = small ? run_up<T, MX, 1, 1, true>(a, lists, s) : run_up<T, MX, V, 1, true>(a, lists, s);
  else e = small ? run_up<T, MX, 1, 2, true>(a, lists, s) : run_up<T, MX, V, 2, true>(a, lists, s);
  if (e != hipSuccess) return e;
  if constexpr (!MX) {
    const int parts = down_parts(a, ((a.I + UK - 1) / UK + 3) / 4);
    if (parts > 1) {
      hipLaunchKernelGGL((k_moe_down<T, MX, true>), dim3(a.D / 16, parts), dim3(64 * kDownWaves), 0, s, a, lists);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((k_moe_down<T, MX, false>), dim3(a.D / 16), dim3(64 * kDownWaves), 0, s, a, lists);
  return hipGetLastError();
}

// Workspace: the lists, the down product's counts and sums, then the hidden values.
constexpr size_t kMoeListBytes = kMoeMaxLists * (sizeof(int) + sizeof(float)) + kMoeBlocks * (sizeof(int) + 256 * sizeof(float));
size_t moe_workspace(int T, int I, int k) { return kMoeListBytes + static_cast<size_t>(T) * k * I * 4; }

hipError_t launch_moe(MoeArgs a, void* workspace, int type, bool mx4, hipStream_t s) {
  MoeLists l;
  l.ids = static_cast<int*>(workspace);
  l.weights = reinterpret_cast<float*>(l.ids + kMoeMaxLists);
  l.arrived = reinterpret_cast<int*>(l.weights + kMoeMaxLists);
  l.sums = reinterpret_cast<float*>(l.arrived + kMoeBlocks);
  a.h = reinterpret_cast<float*>(static_cast<char*>(workspace) + kMoeListBytes);
  if (type == kMxF16) return mx4 ? run<F16, true>(a, l, s) : run<F16, false>(a, l, s);
  return mx4 ? run<B16, true>(a, l, s) : run<B16, false>(a, l, s);
}

}  // namespace i8mm
