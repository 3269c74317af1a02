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

// What k_moe_gate_up leaves for k_moe_down: per chosen expert its index, the mask of its
// tokens and, four bits each, the place it has in each token's list.
struct MoeSlot {
  uint32_t expert, tokens, place_lo, place_hi;
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
  __shared__ int s_ids[kMoeMaxSlots];
  __shared__ float s_w[kMoeMaxSlots];
  __shared__ unsigned s_on[kMoeExpertWords], s_tokens;
  __shared__ int s_place[kMoeMaxTokens];
  __shared__ float red[kMoeWaves][2][16][17];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tok = lane & 15;
  if (tid < kMoeExpertWords) s_on[tid] = 0u;
  if (tid == kMoeExpertWords) s_tokens = 0u;
  for (int t = wave; t < a.T; t += kMoeWaves) moe_route(a, t, lane, s_ids + t * a.k, s_w + t * a.k);
  lds_barrier();
  const int n_lists = a.T * a.k;
  const int my_id = tid < n_lists ? s_ids[tid] : -1;
  if (my_id >= 0) atomicOr(&s_on[my_id >> 5], 1u << (my_id & 31));
  if (blockIdx.x == 0 && blockIdx.y == 0 && tid < n_lists) {
    weights[tid] = s_w[tid];
    if (a.ids) a.ids[tid] = my_id;
    if (a.weights) a.weights[tid] = s_w[tid];
  }
  lds_barrier();
  // this workgroup's expert: the blockIdx.y-th that is on
  const int word = lane < kMoeExpertWords ? static_cast<int>(s_on[lane]) : 0;
  const int upto = wave_prefix_sum(__builtin_popcount(static_cast<unsigned>(word)));
  const int slot = blockIdx.y;
  const uint64_t past = __ballot(upto > slot);
  if (past == 0) {  // fewer experts are on
    if (blockIdx.x == 0 && tid == 0) slots[slot] = MoeSlot{0u, 0u, 0u, 0u};
    return;
  }
  const int at = __builtin_ctzll(past);
  unsigned bits = static_cast<unsigned>(__builtin_amdgcn_readlane(word, at));
  int before = slot - (__builtin_amdgcn_readlane(upto, at) - __builtin_popcount(bits));
  while (before-- > 0) bits &= bits - 1;
  const int expert = 32 * at + __builtin_ctz(bits);
  if (my_id == expert) {
    const int t = tid / a.k;
    atomicOr(&s_tokens, 1u << t);
    s_place[t] = tid - t * a.k;
  }
  lds_barrier();
  const unsigned tokens = s_tokens;
  if (blockIdx.x == 0 && tid == 0) {
    uint64_t p = 0;
    for (int t = 0; t < a.T; ++t)
      if ((tokens >> t) & 1u) p |= static_cast<uint64_t>(s_place[t]) << (4 * t);
    slots[slot] = MoeSlot{static_cast<uint32_t>(expert), tokens, static_cast<uint32_t>(p), static_cast<uint32_t>(p >> 32)};
  }

  constexpr int UK = WeightFmt<MX>::UK;
  const int ks = (a.D + UK - 1) / UK, quads = (ks + 3) >> 2;
  const size_t gate = static_cast<size_t>(expert) * 2 * (a.I / 16) + blockIdx.x, up = gate + a.I / 16;
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.X, static_cast<unsigned>(((a.T - 1) * a.ldx + a.D) * 2));
  const unsigned row = static_cast<unsigned>(tok * a.ldx);
  const bool on = (tokens >> tok) & 1u;
  v4f acc[2] = {};
  for (int q = wave; q < quads; q += kMoeWaves) {
    WeightQuad<MX> wg, wu;
    ActQuad<MX> x;
    wg.load(a.w13, static_cast<const uint32_t*>(a.s13), gate, ks, quads, q, lane);
    wu.load(a.w13, static_cast<const uint32_t*>(a.s13), up, ks, quads, q, lane);
    x.load(q, lane, [&](int k) { return buf_load16(xr, on && k < a.D ? (row + k) * 2u : kOOB); });
    mma_quad<T, MX>(x, wg, acc[0]);
    mma_quad<T, MX>(x, wu, acc[1]);
  }
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int e = 0; e < 4; ++e) red[wave][p][4 * (lane >> 4) + e][tok] = acc[p][e];
  lds_barrier();
  const int t = tid >> 4, n = tid & 15;
  if (t < a.T && ((tokens >> t) & 1u)) {
    float g = 0.0f, u = 0.0f;
#pragma unroll
    for (int w = 0; w < kMoeWaves; ++w) {
      g += red[w][0][t][n];
      u += red[w][1][t][n];
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
    const size_t o = static_cast<size_t>(t * a.k + s_place[t]) * a.I + blockIdx.x * 16 + n;
    a.h[o] = __builtin_bit_cast(uint16_t, hi);
    a.h[static_cast<size_t>(n_lists) * a.I + o] = __builtin_bit_cast(uint16_t, lo);
  }
}

// The c-th set bit of m (c < 16), 32 or more if there is none.
__device__ __forceinline__ int nth_bit(unsigned m, int c) {
#pragma unroll
  for (int i = 0; i < kMoeMaxTokens - 1; ++i) m = i < c ? m & (m - 1) : m;
  return m ? __builtin_ctz(m) : 32;
}

template <class T, bool MX>
__global__ __launch_bounds__(64 * kMoeWaves) void k_moe_down(MoeArgs a, const MoeSlot* slots, const float* weights,
                                                             int n_slots) {
  __shared__ MoeSlot s_slot[kMoeMaxSlots];
  __shared__ float s_w[kMoeMaxSlots];
  __shared__ float total[kMoeWaves][kMoeMaxTokens][17];
  __shared__ int s_n;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n_lists = a.T * a.k;
  if (tid == 0) s_n = 0;
  lds_barrier();
  if (tid < n_slots) {
    const MoeSlot s = slots[tid];
    s_slot[tid] = s;
    if (s.tokens) atomicMax(&s_n, tid + 1);  // the slots in use come first
  }
  if (tid < n_lists) s_w[tid] = weights[tid];
  for (int i = lane; i < kMoeMaxTokens * 17; i += 64) (&total[wave][0][0])[i] = 0.0f;
  lds_barrier();
  const int n = s_n;

  constexpr int UK = WeightFmt<MX>::UK;
  const int ks = (a.I + UK - 1) / UK, quads = (ks + 3) >> 2;
  const int items = n * quads, per = (items + kMoeWaves - 1) / kMoeWaves;
  const int end = min(items, per * (wave + 1));
  const unsigned plane = static_cast<unsigned>(n_lists) * a.I;
  const __amdgpu_buffer_rsrc_t hr = make_rsrc(a.h, plane * 4u);
  const int r = lane & 15, g = lane >> 4;
  for (int i = per * wave; i < end;) {
    const int slot = i / quads;
    const int stop = min(end, (slot + 1) * quads);
    const MoeSlot s = s_slot[slot];
    const size_t group = static_cast<size_t>(s.expert) * (a.D / 16) + blockIdx.x;
    const uint64_t places = s.place_lo | (static_cast<uint64_t>(s.place_hi) << 32);
    const bool more = __builtin_popcount(s.tokens) > 8;
    // this lane's rows of the two passes of eight tokens: high parts in rows 0-7
    unsigned off[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int t = nth_bit(s.tokens, 8 * p + (r & 7));
      const unsigned list = t * a.k + (static_cast<unsigned>(places >> (4 * (t & 15))) & 15u);
      off[p] = t < 16 ? list * a.I + (r >> 3) * plane : kOOB;
    }
    v4f acc[2] = {};
    for (; i < stop; ++i) {
      const int q = i - slot * quads;
      WeightQuad<MX> w;
      w.load(a.w2, static_cast<const uint32_t*>(a.s2), group, ks, quads, q, lane);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        if (p == 1 && !more) break;  // wave-uniform
        ActQuad<MX> x;
        x.load(q, lane, [&](int k) { return buf_load16(hr, off[p] != kOOB && k < a.I ? (off[p] + k) * 2u : kOOB); });
        mma_quad<B16, MX>(x, w, acc[p]);
      }
    }
    float scale = 1.0f;
    if constexpr (!MX) scale = __fdiv_rn(static_cast<const float*>(a.s2)[group * 16 + r], 127.0f);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      if (p == 1 && !more) break;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // rows 4 g + e (high) and 8 + 4 g + e (remainder) of one token are 32 lanes apart
        const float y = acc[p][e] + __shfl_xor(acc[p][e], 32, 64);
        const int t = nth_bit(s.tokens, 8 * p + 4 * (g & 1) + e);
        if (g < 2 && t < 16) {
          const float w = s_w[t * a.k + (static_cast<int>(places >> (4 * t)) & 15)];
          total[wave][t][r] += y * scale * w;
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
  hipLaunchKernelGGL((k_moe_gate_up<T, MX>), dim3(a.I / 16, n_slots), dim3(64 * kMoeWaves), 0, s, a, slots, weights);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_moe_down<T, MX>), dim3(a.D / 16), dim3(64 * kMoeWaves), 0, s, a, slots, weights, n_slots);
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
