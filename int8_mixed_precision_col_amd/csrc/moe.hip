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
// from L2, one wave per token) rather than wait for a launch of its own; workgroup (i, s)
// then takes rows 16 i .. of the gate and of the up part of the s-th chosen expert, against
// the tokens that chose it, and writes their hidden values.
// k_moe_down: a workgroup per 16 output features goes over all chosen experts, its waves
// sharing the (expert, K quad) items in order, so that the weighted sum over experts needs
// neither atomics nor a third launch and is the same on every run.
//
// The hidden values stay near fp32: they are kept as a bf16 pair, high part and remainder
// (16 significant bits, the full exponent range, so that no |h| > 65504 turns into an
// infinity), and the pair costs nothing in the down product: an expert has few tokens, so
// rows 0-7 of the 16-row operand hold the high parts of eight of them and rows 8-15 the
// remainders, and their two sums are added in the end.
#include "mx4_launch.hpp"
#include "weight_stream.hpp"

namespace i8mm {

constexpr int kMoeWaves = 8;
constexpr int kMoeMaxSlots = kMoeMaxTokens * kMoeMaxTopK;
constexpr int kMoeExpertWords = kMoeMaxExperts / 32;

// What k_moe_gate_up leaves for k_moe_down: per chosen expert its index and its tokens in
// ascending order, each a byte 16 t + (the expert's place in token t's list).
struct MoeSlot {
  uint32_t expert, count;
  uint8_t token[kMoeMaxTokens];
};

__device__ __forceinline__ float moe_logit(const void* p, int type, int64_t i) {
  if (type == kMxF32) return static_cast<const float*>(p)[i];
  if (type == kMxF16) return static_cast<float>(static_cast<const _Float16*>(p)[i]);
  return static_cast<float>(static_cast<const __bf16*>(p)[i]);
}

// Order-preserving map of fp32 to unsigned: -inf to 0 (an expert that is off), any NaN to
// the greatest.
__device__ __forceinline__ unsigned moe_key(float v) {
  const unsigned b = __builtin_bit_cast(unsigned, v);
  if (v != v) return 0xffffffffu;
  if (b == 0xff800000u) return 0u;
  const unsigned z = b == 0x80000000u ? 0u : b;  // -0 ties with +0
  return z ^ (z >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float moe_unkey(unsigned k) {
  if (k == 0xffffffffu) return __builtin_nanf("");
  return __builtin_bit_cast(float, k ^ (k >> 31 ? 0x80000000u : 0xffffffffu));
}

// One wave: the list of token t into ids [k] and weights [k] (id -1 and weight 0 past the
// last expert that is on).
__device__ __forceinline__ void moe_route(const MoeArgs& a, int t, int lane, int* ids, float* weights) {
  constexpr int V = kMoeMaxExperts / 64;
  const int per = (a.E + 63) / 64;  // lane's experts: per * lane ..
  unsigned key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = per * lane + i;
    key[i] = i < per && e < a.E ? moe_key(moe_logit(a.logits, a.logits_type, static_cast<int64_t>(t) * a.E + e)) : 0u;
  }
  unsigned first = 0;   // the largest key
  float all = 0.0f;     // sum over every expert
  float mine = 0.0f;    // lane j: weight of place j, unnormalized
  int mine_id = -1;
  float chosen = 0.0f;
  for (int j = 0; j < a.k; ++j) {
    unsigned best = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i;
      }
    const unsigned top = wave_max_u32(best);
    if (j == 0) {
      first = top;
      if (!a.renormalize) {
#pragma unroll
        for (int i = 0; i < V; ++i) all += key[i] ? expf(moe_unkey(key[i]) - moe_unkey(top)) : 0.0f;
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) all += __shfl_xor(all, o, 64);
      }
    }
    if (top == 0u) break;  // no expert left
    const int who = __builtin_ctzll(__ballot(best == top));
    const int id = per * who + __builtin_amdgcn_readlane(at, who);
    const float w = expf(moe_unkey(top) - moe_unkey(first));
    chosen += w;
    if (lane == j) {
      mine = w;
      mine_id = id;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane == who && i == at) key[i] = 0u;
  }
  if (lane < a.k) {
    ids[lane] = mine_id;
    weights[lane] = mine_id < 0 ? 0.0f : __fdiv_rn(mine, a.renormalize ? chosen : all);
  }
}

template <class T, bool MX>
__global__ __launch_bounds__(64 * kMoeWaves) void k_moe_gate_up(MoeArgs a, MoeSlot* slots, float* weights) {
  extern __shared__ __attribute__((aligned(16))) char s_x[];  // [waves][T][kActStride]
  __shared__ int s_ids[kMoeMaxSlots];
  __shared__ float s_w[kMoeMaxSlots];
  __shared__ unsigned s_on[kMoeExpertWords], s_tokens, s_mask[kMoeMaxSlots];
  __shared__ uint8_t s_token[kMoeMaxTokens];
  __shared__ float red[kMoeWaves][2][16][17];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  if (tid < kMoeExpertWords) s_on[tid] = 0u;
  if (tid == kMoeExpertWords) s_tokens = 0u;
  if (tid < kMoeMaxSlots) s_mask[tid] = 0u;
  for (int t = wave; t < a.T; t += kMoeWaves) moe_route(a, t, lane, s_ids + t * a.k, s_w + t * a.k);
  lds_barrier();
  const int n_lists = a.T * a.k;
  const int my_id = tid < n_lists ? s_ids[tid] : -1;
  if (my_id >= 0) atomicOr(&s_on[my_id >> 5], 1u << (my_id & 31));
  lds_barrier();
  // One workgroup writes what the second launch goes by, all of it from its own view of the
  // logits, so that it is consistent whatever else happens to them meanwhile.
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    const int t = tid / a.k;
    int rank = 0;
    if (my_id >= 0) {
      for (int i = 0; i < my_id >> 5; ++i) rank += __builtin_popcount(s_on[i]);
      rank += __builtin_popcount(s_on[my_id >> 5] & ((1u << (my_id & 31)) - 1));
      atomicOr(&s_mask[rank], 1u << t);
    }
    lds_barrier();
    if (tid < n_lists) {
      weights[tid] = s_w[tid];
      if (a.ids) a.ids[tid] = my_id;
      if (a.weights) a.weights[tid] = s_w[tid];
    }
    if (my_id >= 0) {
      const unsigned mask = s_mask[rank];
      const int c = __builtin_popcount(mask & ((1u << t) - 1));
      slots[rank].token[c] = static_cast<uint8_t>(16 * t + (tid - t * a.k));
      if (c == 0) {
        slots[rank].expert = static_cast<uint32_t>(my_id);
        slots[rank].count = static_cast<uint32_t>(__builtin_popcount(mask));
      }
    }
    if (tid < gridDim.y && s_mask[tid] == 0u) slots[tid].count = 0u;
  }
  // this workgroup's expert: the blockIdx.y-th that is on
  const int word = lane < kMoeExpertWords ? static_cast<int>(s_on[lane]) : 0;
  const int upto = wave_prefix_sum(__builtin_popcount(static_cast<unsigned>(word)));
  const int slot = blockIdx.y;
  const uint64_t past = __ballot(upto > slot);
  if (past == 0) return;  // fewer experts are on
  const int at = __builtin_ctzll(past);
  unsigned bits = static_cast<unsigned>(__builtin_amdgcn_readlane(word, at));
  int before = slot - (__builtin_amdgcn_readlane(upto, at) - __builtin_popcount(bits));
  while (before-- > 0) bits &= bits - 1;
  const int expert = 32 * at + __builtin_ctz(bits);
  if (my_id == expert) atomicOr(&s_tokens, 1u << (tid / a.k));
  lds_barrier();
  const unsigned tokens = s_tokens;
  const int count = __builtin_popcount(tokens);
  if (my_id == expert) {
    const int t = tid / a.k, c = __builtin_popcount(tokens & ((1u << t) - 1));
    s_token[c] = static_cast<uint8_t>(16 * t + (tid - t * a.k));
  }
  lds_barrier();

  constexpr int UK = WeightFmt<MX>::UK;
  const int ks = (a.D + UK - 1) / UK, quads = (ks + 3) >> 2;
  const size_t gate = static_cast<size_t>(expert) * 2 * (a.I / 16) + blockIdx.x, up = gate + a.I / 16;
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.X, static_cast<unsigned>(((a.T - 1) * a.ldx + a.D) * 2));
  char* buf = s_x + wave * a.T * kActStride;
  const int row = min(lane & 15, count - 1);  // rows past the last token repeat it (discarded)
  v4f acc[2] = {};
  for (int q = wave; q < quads; q += kMoeWaves) {
    WeightQuad<MX> w[2];
    ActQuad<MX> x;
    x.load(xr, q, a.D, count, lane, [&](int i) {
      return i < count ? static_cast<unsigned>((s_token[i] >> 4) * a.ldx) * 2u : kOOB; });
    w[0].load(a.w13, static_cast<const uint32_t*>(a.s13), gate, ks, quads, q, lane);
    w[1].load(a.w13, static_cast<const uint32_t*>(a.s13), up, ks, quads, q, lane);
    mma_quad<T, MX, 2>(
        w, acc,
        [&](int p) {
          wave_lds_fence();
          x.stage(p, buf, count, lane, [](int i) { return i; });
          wave_lds_fence();
        },
        [&](int, int j, int v) { return act_operand<MX>(buf, row, j, v, lane); });
  }
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int e = 0; e < 4; ++e) red[wave][p][4 * (lane >> 4) + e][lane & 15] = acc[p][e];
  lds_barrier();
  const int c = tid >> 4, n = tid & 15;
  if (c < count) {
    float g = 0.0f, u = 0.0f;
#pragma unroll
    for (int w = 0; w < kMoeWaves; ++w) {
      g += red[w][0][c][n];
      u += red[w][1][c][n];
    }
    if constexpr (!MX) {
      const float* aw = static_cast<const float*>(a.s13);
      g *= __fdiv_rn(aw[gate * 16 + n], 127.0f);
      u *= __fdiv_rn(aw[up * 16 + n], 127.0f);
    }
    const float h = __fdiv_rn(g, 1.0f + expf(-g)) * u;
    const __bf16 hi = static_cast<__bf16>(h);
    const float rest = h - static_cast<float>(hi);
    const __bf16 lo = static_cast<__bf16>(fabsf(rest) < __builtin_inff() ? rest : 0.0f);
    const int list = (s_token[c] >> 4) * a.k + (s_token[c] & 15);
    const size_t o = static_cast<size_t>(list) * a.I + blockIdx.x * 16 + n;
    a.h[o] = __builtin_bit_cast(uint16_t, hi);
    a.h[static_cast<size_t>(n_lists) * a.I + o] = __builtin_bit_cast(uint16_t, lo);
  }
}

// Rows that a pass of k_moe_down stages: the high parts and the remainders of 8 tokens.
__host__ __device__ __forceinline__ int moe_down_rows(int T) { return 2 * (T < 8 ? T : 8); }

template <class T, bool MX>
__global__ __launch_bounds__(64 * kMoeWaves) void k_moe_down(MoeArgs a, const MoeSlot* slots, const float* weights,
                                                             int n_slots) {
  // [waves][moe_down_rows(T)][kActStride], then the slots, then the weights
  extern __shared__ __attribute__((aligned(16))) char s_x[];
  __shared__ float total[kMoeWaves][kMoeMaxTokens][17];
  __shared__ int s_n;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n_lists = a.T * a.k;
  char* buf = s_x + wave * moe_down_rows(a.T) * kActStride;
  MoeSlot* s_slot = reinterpret_cast<MoeSlot*>(s_x + kMoeWaves * moe_down_rows(a.T) * kActStride);
  float* s_w = reinterpret_cast<float*>(s_slot + n_slots);
  if (tid == 0) s_n = 0;
  lds_barrier();
  if (tid < n_slots) {
    // Addresses come out of these: kept in range here too, so that a workspace that another
    // call wrote to meanwhile, which the interface forbids, gives wrong values at worst.
    MoeSlot v = slots[tid];
    v.expert = min(v.expert, static_cast<uint32_t>(a.E - 1));
    v.count = min(v.count, static_cast<uint32_t>(a.T));
    for (int c = 0; c < kMoeMaxTokens; ++c)
      v.token[c] = static_cast<uint8_t>(16 * min(v.token[c] >> 4, a.T - 1) + min(v.token[c] & 15, a.k - 1));
    s_slot[tid] = v;
    if (v.count) atomicMax(&s_n, tid + 1);  // the slots in use come first
  }
  if (tid < n_lists) s_w[tid] = weights[tid];
  for (int i = lane; i < kMoeMaxTokens * 17; i += 64) (&total[wave][0][0])[i] = 0.0f;
  lds_barrier();
  const int n = s_n;

  constexpr int UK = WeightFmt<MX>::UK;
  const int ks = (a.I + UK - 1) / UK, quads = (ks + 3) >> 2;
  const int items = n * quads, per = (items + kMoeWaves - 1) / kMoeWaves;
  const int end = min(items, per * (wave + 1));
  const unsigned plane = static_cast<unsigned>(n_lists) * a.I * 2u;  // bytes
  const __amdgpu_buffer_rsrc_t hr = make_rsrc(a.h, plane * 2u);
  const int r = lane & 15, g = lane >> 4;
  for (int i = per * wave; i < end;) {
    const int slot = i / quads;
    const int stop = min(end, (slot + 1) * quads);
    const MoeSlot& s = s_slot[slot];
    const size_t group = static_cast<size_t>(s.expert) * (a.D / 16) + blockIdx.x;
    const int count = __builtin_amdgcn_readfirstlane(static_cast<int>(s.count));
    v4f acc[2][1] = {};
    for (; i < stop; ++i) {
      const int q = i - slot * quads;
      WeightQuad<MX> w[1];
      w[0].load(a.w2, static_cast<const uint32_t*>(a.s2), group, ks, quads, q, lane);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int m = min(count - 8 * p, 8);  // tokens of this pass
        if (m <= 0) break;                    // wave-uniform
        ActQuad<MX> x;
        x.load(hr, q, a.I, 2 * m, lane, [&](int j) -> unsigned {
          if (j >= 2 * m) return kOOB;
          const unsigned e = s.token[8 * p + (j < m ? j : j - m)];
          return ((e >> 4) * a.k + (e & 15u)) * a.I * 2u + (j < m ? 0u : plane);
        });
        // operand rows 0-7 are the high parts, 8-15 the remainders; past the last token repeats
        const int row = min(r & 7, m - 1) + (r < 8 ? 0 : m);
        mma_quad<B16, MX, 1>(
            w, acc[p],
            [&](int piece) {
              wave_lds_fence();
              x.stage(piece, buf, 2 * m, lane, [](int j) { return j; });
              wave_lds_fence();
            },
            [&](int, int j, int v) { return act_operand<MX>(buf, row, j, v, lane); });
      }
    }
    float scale = 1.0f;
    if constexpr (!MX) scale = __fdiv_rn(static_cast<const float*>(a.s2)[group * 16 + r], 127.0f);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // rows 4 g + e (high) and 8 + 4 g + e (remainder) of one token are 32 lanes apart
        const float y = acc[p][0][e] + __shfl_xor(acc[p][0][e], 32, 64);
        const int c = 8 * p + 4 * (g & 1) + e;
        if (g < 2 && c < count) {
          const unsigned t = s.token[c] >> 4, place = s.token[c] & 15u;
          total[wave][t][r] += y * scale * s_w[t * a.k + place];
        }
      }
    }
  }
  lds_barrier();
  const int t = tid >> 4, f = tid & 15;
  if (t < a.T) {
    float y = 0.0f;
#pragma unroll
    for (int w = 0; w < kMoeWaves; ++w) y += total[w][t][f];
    static_cast<typename T::elem*>(a.Y)[static_cast<size_t>(t) * a.D + blockIdx.x * 16 + f] = T::round(y);
  }
}

template <class T, bool MX>
static hipError_t run(const MoeArgs& a, MoeSlot* slots, float* weights, hipStream_t s) {
  const int n_slots = a.E < a.T * a.k ? a.E : a.T * a.k;
  const size_t lds1 = static_cast<size_t>(kMoeWaves) * a.T * kActStride;
  const size_t lds2 = static_cast<size_t>(kMoeWaves) * moe_down_rows(a.T) * kActStride + n_slots * sizeof(MoeSlot) +
                      static_cast<size_t>(a.T) * a.k * sizeof(float);
  hipLaunchKernelGGL((k_moe_gate_up<T, MX>), dim3(a.I / 16, n_slots), dim3(64 * kMoeWaves), lds1, s, a, slots, weights);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_moe_down<T, MX>), dim3(a.D / 16), dim3(64 * kMoeWaves), lds2, s, a, slots, weights, n_slots);
  return hipGetLastError();
}

// Workspace: the slots, the weights, the hidden values.
size_t moe_workspace(int T, int I, int k) {
  return kMoeMaxSlots * (sizeof(MoeSlot) + sizeof(float)) + static_cast<size_t>(T) * k * I * 4;
}

hipError_t launch_moe(MoeArgs a, void* workspace, int type, bool mx4, hipStream_t s) {
  MoeSlot* slots = static_cast<MoeSlot*>(workspace);
  float* weights = reinterpret_cast<float*>(slots + kMoeMaxSlots);
  a.h = reinterpret_cast<uint16_t*>(weights + kMoeMaxSlots);
  if (type == kMxF16) return mx4 ? run<F16, true>(a, slots, weights, s) : run<F16, false>(a, slots, weights, s);
  return mx4 ? run<B16, true>(a, slots, weights, s) : run<B16, false>(a, slots, weights, s);
}

}  // namespace i8mm
