// Routing to experts: softmax or sigmoid scores, a balance bias that moves the
// choice but not the weights, expert groups, top-k, renormalised weights; and
// the gradient of the weights with respect to the logits.
//
// One warp per token; lane l holds experts l * VPL .. l * VPL + VPL - 1, so
// that the lowest lane among equals holds the lowest id.  The k-th largest of
// the 32 lanes' own maxima bounds the k-th largest key from below: k warp maxima
// (redux) find it, the keys that reach it (a few more than k) are packed one to a
// lane in order of their ids, and each counts those that go before it.  Against
// k rounds that each search a lane's VPL keys: 40 us for 92 at 32768 tokens of
// 256 experts, top-8, with bias and groups (37 without the host).  That is bound
// by instruction issue (about 880 a token, 71 % of the slots), not by the 19 MB
// it moves (2.8 us): 256 exponentials and reciprocals have to be exact to the bit
// for the choice to be that of the definition.  Softmax without a bias needs none
// of them for the choice: 20 us.
#include <float.h>
#include <math.h>

#include <type_traits>

#include "dtype.cuh"

namespace moe {

struct RouteArgs {
  const void* logits;
  long long ld;
  int T, E, k, score, n_group, topk_group, group_score, renorm;
  float scale;
  const float* bias;
  const uint8_t* mask;
  int32_t* ids;
  float* w;
  int32_t* load;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A logit as the choice sees it: NaN counts as -inf (not eligible).
template <typename TL>
__device__ __forceinline__ float load_logit(const TL* row, int e) {
  const float v = to_f32(row[e]);
  return v == v ? v : -INFINITY;
}

__device__ __forceinline__ float sigmoid_f32(float z) { return __frcp_rn(1.f + expf(-z)); }
// e^(z - top), also where both are +inf; 0 for z = -inf.
__device__ __forceinline__ float exp_below(float z, float top) {
  return z == -INFINITY ? 0.f : (z == top ? 1.f : expf(z - top));
}

// The warp's maximum (no NaN among the values).
__device__ __forceinline__ float redux_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// Lane's VPL logits of a row; NaN and what lies past E count as -inf.  `vec`:
// rows start where a lane's share can be read in one piece (up to 16 bytes).
template <int VPL, typename TL>
__device__ __forceinline__ void load_row(const TL* row, int lane, int E, bool vec, float (&z)[VPL]) {
  constexpr int kBytes = VPL * (int)sizeof(TL), kPiece = kBytes < 16 ? kBytes : 16;
  constexpr int kEach = kPiece / (int)sizeof(TL);
  if (kPiece > 2 && vec && (lane + 1) * VPL <= E) {
#pragma unroll
    for (int i = 0; i < kBytes / kPiece; ++i) {
      alignas(16) TL e[kEach];
      const TL* p = row + lane * VPL + i * kEach;
      if constexpr (kPiece == 16) *reinterpret_cast<uint4*>(e) = *reinterpret_cast<const uint4*>(p);
      else if constexpr (kPiece == 8) *reinterpret_cast<uint2*>(e) = *reinterpret_cast<const uint2*>(p);
      else if constexpr (kPiece == 4) *reinterpret_cast<uint32_t*>(e) = *reinterpret_cast<const uint32_t*>(p);
#pragma unroll
      for (int j = 0; j < kEach; ++j) z[i * kEach + j] = to_f32(e[j]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) z[i] = lane * VPL + i < E ? to_f32(row[lane * VPL + i]) : -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) z[i] = fmaxf(z[i], -INFINITY);   // NaN: the other operand
}

// The two largest of a group as its worth; -inf is an empty group's, so two biases of fp32's lowest
// value add up to that value.
__device__ __forceinline__ float sum_of_two(float m1, float m2) {
  return m2 > -INFINITY ? fmaxf(m1 + m2, -FLT_MAX) : m1;
}

// Lane g: what group g (of n_group times gs experts) is worth.  `lpg`: the lanes
// of a group, where a lane's experts belong to one group and a group's lanes are
// a power of two; else 0, and the groups are taken one after the other.
template <int VPL>
__device__ __forceinline__ float group_worth(const float (&val)[VPL], int lane, int E, int gs, int n_group, int lpg,
                                             int how) {
  float m1 = -INFINITY, m2 = -INFINITY;   // the two largest
  auto join = [&](int o) {
    const float o1 = __shfl_xor_sync(0xffffffffu, m1, o), o2 = __shfl_xor_sync(0xffffffffu, m2, o);
    m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
    m1 = fmaxf(m1, o1);
  };
  if (lpg) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      m2 = fmaxf(m2, fminf(m1, val[i]));
      m1 = fmaxf(m1, val[i]);
    }
    for (int o = 1; o < lpg; o <<= 1) join(o);
    if (how == MOE_GROUP_TOP2) m1 = sum_of_two(m1, m2);
    return __shfl_sync(0xffffffffu, m1, lane * lpg & 31);
  }
  float worth = -INFINITY;
  for (int g = 0; g < n_group; ++g) {
    m1 = m2 = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane * VPL + i;
      if (e >= g * gs && e < (g + 1) * gs) {
        m2 = fmaxf(m2, fminf(m1, val[i]));
        m1 = fmaxf(m1, val[i]);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) join(o);
    if (lane == g) worth = how == MOE_GROUP_TOP2 ? sum_of_two(m1, m2) : m1;
  }
  return worth;
}

constexpr int kRouteWarps = 4;
// Blocks an SM holds at once (64 to 168 registers a thread): the grid is that many times the SMs.
template <int VPL>
constexpr int kRouteBlocks = VPL <= 8 ? 8 : VPL == 16 ? 5 : 3;

// With more than 16 experts a lane its biases wait in shared memory, read from global
// memory in their order and laid out so that the lanes' reads meet no common bank:
// lane l's i-th at l * (VPL + 1) + i (4096 tokens of
// 1024 experts, softmax: 37.5 us read in place by every token, 25.2 so).
template <int VPL>
constexpr int kLaid = 32 * (VPL + 1);
template <int VPL>
constexpr bool kBiasLaid = VPL > 16;

template <int VPL, typename TL>
__global__ void __launch_bounds__(kRouteWarps * 32, kRouteBlocks<VPL>) route_kernel(const RouteArgs a, int vec) {
  extern __shared__ float laid_bias[];   // [kLaid], with kBiasLaid and a bias; then hist
  int* hist = reinterpret_cast<int*>(laid_bias + (kBiasLaid<VPL> && a.bias ? kLaid<VPL> : 0));   // [E] with a load
  __shared__ alignas(16) float c_key[kRouteWarps][32];
  __shared__ int c_id[kRouteWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int k = a.k, E = a.E;
  pdl_wait();
  pdl_launch_dependents();
  if (a.load)
    for (int e = threadIdx.x; e < E; e += kRouteWarps * 32) hist[e] = 0;
  if (kBiasLaid<VPL> && a.bias)
    for (int e = threadIdx.x; e < 32 * VPL; e += kRouteWarps * 32) laid_bias[e + e / VPL] = e < E ? a.bias[e] : 0.f;
  if (a.load || (kBiasLaid<VPL> && a.bias)) __syncthreads();
  const bool grouped = a.topk_group < a.n_group;
  const bool scored = a.bias || (grouped && a.group_score == MOE_GROUP_TOP2);
  const bool whole = a.score == MOE_SCORE_SOFTMAX && (scored || !a.renorm);   // the softmax's denominator is needed
  const int gs = E / a.n_group;
  // lanes of a group, where every lane's experts belong to one group
  const int lpg = gs % VPL == 0 && gs / VPL <= 32 && ((gs / VPL) & (gs / VPL - 1)) == 0 ? gs / VPL : 0;
  float bias[kBiasLaid<VPL> ? 1 : VPL];
  if (!kBiasLaid<VPL> && a.bias) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) bias[i % (kBiasLaid<VPL> ? 1 : VPL)] = lane * VPL + i < E ? a.bias[lane * VPL + i] : 0.f;
  }
  const long long step = (long long)gridDim.x * kRouteWarps;
  for (long long t = (long long)blockIdx.x * kRouteWarps + warp; t < a.T; t += step) {
    const TL* row = reinterpret_cast<const TL*>(a.logits) + t * a.ld;
    int my_id = -1, my_rank = lane;   // lane holds the my_rank-th choice
    float top = -INFINITY, den = 0.f;
    if (!a.mask || a.mask[t]) {
      float key[VPL];
      load_row<VPL>(row, lane, E, vec, key);
      if (whole) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) top = fmaxf(top, key[i]);
        top = redux_max(top);
        // the denominator, over neighbouring pairs: in the lane, then across lanes
        float ex[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) ex[i] = exp_below(key[i], top);
#pragma unroll
        for (int n = VPL / 2; n > 0; n /= 2)
#pragma unroll
          for (int i = 0; i < n; ++i) ex[i] = ex[2 * i] + ex[2 * i + 1];
        den = ex[0];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
      }
      float m1 = -INFINITY;   // lane g: what group g is worth
      if (scored) {
        float val[VPL];   // what groups are valued by; the key, where there is a bias
        // what is -inf gets its value below: an ordinary operand here, since a reciprocal of inf or a
        // quotient of 0 takes a slower way, and the whole warp with it (one token of 768 experts: 13.0 us, 9.2 so)
        if (a.score == MOE_SCORE_SIGMOID) {
#pragma unroll
          for (int i = 0; i < VPL; ++i) val[i] = sigmoid_f32(key[i] > -INFINITY ? key[i] : 0.f);
        } else {
#pragma unroll
          for (int i = 0; i < VPL; ++i) val[i] = __fdiv_rn(key[i] > -INFINITY ? exp_below(key[i], top) : 1.f, den);
        }
        if (a.bias) {
#pragma unroll
          for (int i = 0; i < VPL; ++i)
            val[i] += kBiasLaid<VPL> ? laid_bias[lane * (VPL + 1) + i] : bias[i % (kBiasLaid<VPL> ? 1 : VPL)];
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          val[i] = key[i] > -INFINITY ? val[i] : -INFINITY;
          if (a.bias) key[i] = val[i];
        }
        if (grouped) m1 = group_worth<VPL>(val, lane, E, gs, a.n_group, lpg, a.group_score);
      } else if (grouped) {
        m1 = group_worth<VPL>(key, lane, E, gs, a.n_group, lpg, a.group_score);
      }
      if (grouped) {
        // the topk_group largest, ties to the lower group; an empty group among them holds no key
        uint32_t keep = 0;
        float left = lane < a.n_group ? m1 : -INFINITY;
        for (int j = 0; j < a.topk_group; ++j) {
          const float m = redux_max(left);
          const int win = __ffs(__ballot_sync(0xffffffffu, left == m)) - 1;
          keep |= 1u << win;
          if (lane == win) left = -INFINITY;
        }
        if (lpg) {
          const bool in = keep >> (lane / lpg) & 1;
#pragma unroll
          for (int i = 0; i < VPL; ++i) key[i] = in ? key[i] : -INFINITY;
        } else {
#pragma unroll
          for (int i = 0; i < VPL; ++i) {
            const int e = lane * VPL + i;
            if (e < E && !(keep >> (e / gs) & 1)) key[i] = -INFINITY;
          }
        }
      }
      // a bound: the k-th largest of the lanes' maxima (lower yet where some are equal)
      float best = key[0];
#pragma unroll
      for (int i = 1; i < VPL; ++i) best = fmaxf(best, key[i]);
      float least = -INFINITY;
#pragma unroll 4
      for (int j = 0; j < k; ++j) {
        least = redux_max(best);
        best = best == least ? -INFINITY : best;
      }
      least = fmaxf(least, -FLT_MAX);   // what is -inf is not eligible
      // the keys that reach it, packed in order of their ids
      int n = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) n += key[i] >= least;
      int at = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += v;
      }
      const int all = __shfl_sync(0xffffffffu, at, 31);
      at -= n;
      if (all <= 32) {
        c_key[warp][lane] = -INFINITY;
        __syncwarp();
        if (n) {
#pragma unroll
          for (int i = 0; i < VPL; ++i)
            if (key[i] >= least) {
              c_key[warp][at] = key[i];
              c_id[warp][at++] = lane * VPL + i;
            }
        }
        __syncwarp();
        // a candidate's place: how many are larger, or equal with a lower id
        const float mine = c_key[warp][lane];
        const int id = c_id[warp][lane];
        int rank = 0;
        for (int i = 0; i < all; i += 4) {
          const float4 o = *reinterpret_cast<const float4*>(&c_key[warp][i]);
          rank += (o.x > mine || (o.x == mine && i < lane)) + (o.y > mine || (o.y == mine && i + 1 < lane)) +
                  (o.z > mine || (o.z == mine && i + 2 < lane)) + (o.w > mine || (o.w == mine && i + 3 < lane));
        }
        __syncwarp();
        // lanes without a candidate take the places after the last one, in order
        my_rank = lane < all ? rank : lane;
        my_id = lane < all && rank < k ? id : -1;
      } else {   // many equal keys, or a k near 32: round by round over all of them
        for (int j = 0; j < k; ++j) {
          float b = key[0];
#pragma unroll
          for (int i = 1; i < VPL; ++i) b = fmaxf(b, key[i]);
          const float m = redux_max(b);
          if (!(m > -INFINITY)) break;
          const int win = __ffs(__ballot_sync(0xffffffffu, b == m)) - 1;
          int id = 0;
          if (lane == win) {
            bool found = false;
#pragma unroll
            for (int i = 0; i < VPL; ++i)
              if (!found && key[i] == m) {
                found = true;
                id = lane * VPL + i;
                key[i] = -INFINITY;
              }
          }
          id = __shfl_sync(0xffffffffu, id, win);
          if (lane == j) my_id = id;
        }
      }
    }
    // weights, each lane its own choice's
    const float z = my_id >= 0 ? load_logit(row, my_id) : -INFINITY;
    float s;
    if (a.score == MOE_SCORE_SIGMOID) {
      s = my_id >= 0 ? sigmoid_f32(z) : 0.f;
    } else if (a.renorm) {
      s = exp_below(z, redux_max(z));
    } else {
      s = my_id >= 0 ? __fdiv_rn(exp_below(z, top), den) : 0.f;
    }
    if (a.renorm) {
      const float sum = warp_sum(s);
      s = sum > 0.f ? s / sum : 0.f;
    }
    if (my_rank < k) {
      a.ids[t * k + my_rank] = my_id;
      a.w[t * k + my_rank] = a.scale * s;
      if (a.load && my_id >= 0) atomicAdd(hist + my_id, 1);
    }
  }
  if (a.load) {
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kRouteWarps * 32)
      if (hist[e]) atomicAdd(a.load + e, hist[e]);
  }
}

struct RouteBwdArgs {
  const void* logits;
  long long ld;
  int T, E, k, score, renorm;
  float scale;
  const uint8_t* mask;
  const int32_t* ids;
  const float* dw;
  void* d;
  long long ld_d;
};

// GROUP lanes per token (k <= GROUP): the rows are written first (zeros), then the
// chosen experts' values over them.  16384 tokens of 256 experts, top-6,
// fp32: 6.2 us (17.9 MB: 2.65 us at the copy rate), the rest two dependent reads,
// ids and then their logits, and a launch.  `vec`: rows and their length allow 16-byte stores.
__device__ __forceinline__ float group_sum(float v, int width) {
  for (int o = width / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float group_max(float v, int width) {
  for (int o = width / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

template <typename TL, int GROUP>
__global__ void __launch_bounds__(128) route_bwd_kernel(const RouteBwdArgs a, int vec) {
  constexpr int kTokens = 32 / GROUP;   // of a warp
  const int lane = threadIdx.x & 31, sub = lane / GROUP, gl = lane % GROUP;
  pdl_wait();
  pdl_launch_dependents();
  const long long step = gridDim.x * 4LL * kTokens;
  for (long long t0 = (blockIdx.x * 4LL + (threadIdx.x >> 5)) * kTokens; t0 < a.T; t0 += step) {
    const long long t = t0 + sub;
    const TL* row = reinterpret_cast<const TL*>(a.logits) + t * a.ld;
    TL* d = reinterpret_cast<TL*>(a.d) + t * a.ld_d;
    const bool on = t < a.T && (!a.mask || a.mask[t]);
    int id = -1;
    float g = 0.f, z = -INFINITY;
    if (gl < a.k && on) {
      id = a.ids[t * a.k + gl];
      g = a.scale * a.dw[t * a.k + gl];
    }
    // while the ids are on their way
#pragma unroll
    for (int q = 0; q < kTokens; ++q) {
      if (t0 + q >= a.T) break;
      TL* dq = reinterpret_cast<TL*>(a.d) + (t0 + q) * a.ld_d;
      if (vec) {
        constexpr int kEach = 16 / (int)sizeof(TL);
        for (int e = lane * kEach; e < a.E; e += 32 * kEach)
          *reinterpret_cast<uint4*>(dq + e) = make_uint4(0, 0, 0, 0);
      } else {
        for (int e = lane; e < a.E; e += 32) dq[e] = from_f32<TL>(0.f);
      }
    }
    if (id >= 0 && id < a.E) z = load_logit(row, id);
    if (!(z > -INFINITY)) id = -1, g = 0.f;
    float q, c = 1.f;
    if (a.score == MOE_SCORE_SIGMOID) {
      q = id >= 0 ? sigmoid_f32(z) : 0.f;
      c = id >= 0 ? sigmoid_f32(-z) : 0.f;   // 1 - s without the cancellation
    } else {
      q = exp_below(z, group_max(z, GROUP));
    }
    float mean = 0.f;
    if (a.renorm) {
      const float sum = group_sum(q, GROUP);
      q = sum > 0.f ? q / sum : 0.f;
      mean = group_sum(q * g, GROUP);
    }
    const float dj = q * c * (g - mean);
    __syncwarp();   // the rows are written before the chosen experts' values
    if (id >= 0) d[id] = from_f32<TL>(dj);
  }
}

// Softmax weights that are not renormalised: every logit of a token has a gradient,
//   d z_e = p_e (g_e - sum_j g_j p_j),  g_e = 0 for experts not chosen.
// One warp per token, its row kept in registers between the softmax's sums and the
// gradient, a lane's share in pieces of 16 bytes or, where rows do not start for
// that, every 32nd element.  16384 tokens of 256 experts, fp32: 7.7 us (33.6 MB: 5.0
// at the copy rate; 14.8 with the row read again for each of its three uses).
template <int VPL, typename TL>
__global__ void __launch_bounds__(128) route_bwd_dense_kernel(const RouteBwdArgs a, int vec) {
  constexpr int kBytes = VPL * (int)sizeof(TL), kPiece = kBytes < 16 ? kBytes : 16;
  constexpr int kEach = kPiece / (int)sizeof(TL);
  const int lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  const long long step = gridDim.x * 4LL;
  for (long long t = blockIdx.x * 4LL + (threadIdx.x >> 5); t < a.T; t += step) {
    const TL* row = reinterpret_cast<const TL*>(a.logits) + t * a.ld;
    TL* d = reinterpret_cast<TL*>(a.d) + t * a.ld_d;
    const bool on = !a.mask || a.mask[t];
    int id = -1;
    float g = 0.f, z = -INFINITY, v[VPL];
    if (lane < a.k && on) {
      id = a.ids[t * a.k + lane];
      g = a.scale * a.dw[t * a.k + lane];
    }
    if (vec) {
      load_row<VPL>(row, lane, a.E, true, v);
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) v[i] = i * 32 + lane < a.E ? load_logit(row, i * 32 + lane) : -INFINITY;
    }
    if (id >= 0 && id < a.E) z = load_logit(row, id);
    if (!(z > -INFINITY)) id = -1, g = 0.f;
    float top = -INFINITY, den = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) top = fmaxf(top, v[i]);
    top = redux_max(top);
#pragma unroll
    for (int i = 0; i < VPL; ++i) den += v[i] = exp_below(v[i], top);
    den = warp_sum(den);
    const float p = id >= 0 ? exp_below(z, top) / den : 0.f, mean = warp_sum(g * p), dj = p * (g - mean);
    const bool some = on && den > 0.f;
    const float by = some ? -mean / den : 0.f;
    TL o[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) o[i] = from_f32<TL>(some ? v[i] * by : 0.f);
    if (!vec) {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (i * 32 + lane < a.E) d[i * 32 + lane] = o[i];
    } else if (kPiece > 2 && (lane + 1) * VPL <= a.E) {
#pragma unroll
      for (int i = 0; i < kBytes / kPiece; ++i) {
        alignas(16) TL q[kEach];
#pragma unroll
        for (int j = 0; j < kEach; ++j) q[j] = o[i * kEach + j];
        TL* at = d + lane * VPL + i * kEach;
        if constexpr (kPiece == 16) *reinterpret_cast<uint4*>(at) = *reinterpret_cast<const uint4*>(q);
        else if constexpr (kPiece == 8) *reinterpret_cast<uint2*>(at) = *reinterpret_cast<const uint2*>(q);
        else if constexpr (kPiece == 4) *reinterpret_cast<uint32_t*>(at) = *reinterpret_cast<const uint32_t*>(q);
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (lane * VPL + i < a.E) d[lane * VPL + i] = o[i];
    }
    __syncwarp();   // the row is written before the chosen experts' values
    if (id >= 0) d[id] = from_f32<TL>(dj);
  }
}

// f(constant VPL): experts of a lane, a power of two.
template <typename F>
static auto by_lane_share(int E, F f) {
  const int vpl = (E + 31) / 32;
  if (vpl <= 1) return f(std::integral_constant<int, 1>());
  if (vpl <= 2) return f(std::integral_constant<int, 2>());
  if (vpl <= 4) return f(std::integral_constant<int, 4>());
  if (vpl <= 8) return f(std::integral_constant<int, 8>());
  if (vpl <= 16) return f(std::integral_constant<int, 16>());
  if (vpl <= 32) return f(std::integral_constant<int, 32>());
  return f(std::integral_constant<int, 64>());
}
// Whether a lane's share of a row can be moved in pieces of up to 16 bytes.
template <int VPL, typename TL>
static int whole_pieces(const void* base, long long ld) {
  constexpr int kBytes = VPL * (int)sizeof(TL), kPiece = kBytes < 16 ? kBytes : 16;
  return (uintptr_t)base % kPiece == 0 && ld * (long long)sizeof(TL) % kPiece == 0;
}

template <typename TL>
static cudaError_t launch_route_bwd(const RouteBwdArgs& a, cudaStream_t s) {
  const bool dense = a.score == MOE_SCORE_SOFTMAX && !a.renorm;
  const int group = dense || a.k > 16 ? 32 : a.k > 8 ? 16 : 8;
  const long long warps = (a.T + 32LL / group - 1) / (32 / group), need = (warps + 3) / 4, most = device_sms() * 16LL;
  const dim3 grid((unsigned)(need < most ? need : most)), block(128);
  if (dense)
    return by_lane_share(a.E, [&](auto n) {
      constexpr int VPL = decltype(n)::value;
      return launch_pdl(route_bwd_dense_kernel<VPL, TL>, grid, block, 0, s, a,
                        (int)(whole_pieces<VPL, TL>(a.logits, a.ld) && whole_pieces<VPL, TL>(a.d, a.ld_d)));
    });
  const long long size = sizeof(TL);
  const int vec = (uintptr_t)a.d % 16 == 0 && a.ld_d * size % 16 == 0 && a.E * size % 16 == 0;
  if (group == 32) return launch_pdl(route_bwd_kernel<TL, 32>, grid, block, 0, s, a, vec);
  if (group == 16) return launch_pdl(route_bwd_kernel<TL, 16>, grid, block, 0, s, a, vec);
  return launch_pdl(route_bwd_kernel<TL, 8>, grid, block, 0, s, a, vec);
}

template <int VPL, typename TL>
static moe_status launch_route(const RouteArgs& a, cudaStream_t s) {
  const int vec = whole_pieces<VPL, TL>(a.logits, a.ld);
  const long long need = ((long long)a.T + kRouteWarps - 1) / kRouteWarps, most = device_sms() * (long long)kRouteBlocks<VPL>;
  ProfScope ps(MOE_K_ROUTE, s);
  cudaError_t e = launch_pdl(route_kernel<VPL, TL>, dim3((unsigned)(need < most ? need : most)),
                             dim3(kRouteWarps * 32), (kBiasLaid<VPL> && a.bias ? kLaid<VPL> * 4 : 0) + (a.load ? a.E * 4 : 0), s, a, vec);
  if (e != cudaSuccess) return cuda_fail(e, "route_kernel");
  return check_launch("route_kernel");
}

template <typename TL>
static moe_status route_by_size(const RouteArgs& a, cudaStream_t s) {
  return by_lane_share(a.E, [&](auto n) { return launch_route<decltype(n)::value, TL>(a, s); });
}

}  // namespace moe

using namespace moe;

static moe_status route_check(int dtype, int64_t ld, int T, int E, int k, int score) {
  MOE_ARG(T >= 0, "T must be >= 0");
  MOE_ARG(known_dtype(dtype), "unknown logits type %d", dtype);
  MOE_ARG(E >= 1 && E <= 2048, "E must be in [1, 2048] (got %d)", E);
  MOE_ARG(k >= 1 && k <= E && k <= 32, "k must be in [1, min(E, 32)] (got %d)", k);
  MOE_ARG(score == MOE_SCORE_SOFTMAX || score == MOE_SCORE_SIGMOID, "unknown score %d", score);
  MOE_ARG(ld >= E, "the logits' row distance must be >= E (got %lld)", (long long)ld);
  return MOE_OK;
}

extern "C" moe_status moe_route(const void* logits, int dtype, int64_t ld_logits, int T, int E, int k, int score,
                                const float* bias, int n_group, int topk_group, int group_score, int renorm,
                                float scale, const uint8_t* token_mask, int32_t* topk_ids, float* topk_w,
                                int32_t* load, cudaStream_t stream) {
  clear_error();
  moe_status st = route_check(dtype, ld_logits, T, E, k, score);
  if (st != MOE_OK) return st;
  MOE_ARG(n_group >= 1 && n_group <= 32 && E % n_group == 0, "n_group must be in [1, 32] and divide E (got %d)",
          n_group);
  MOE_ARG(topk_group >= 1 && topk_group <= n_group, "topk_group must be in [1, n_group] (got %d)", topk_group);
  MOE_ARG(group_score == MOE_GROUP_MAX || group_score == MOE_GROUP_TOP2, "unknown group score %d", group_score);
  if (T == 0) return MOE_OK;
  MOE_ARG(logits && topk_ids && topk_w, "null pointer");
  const RouteArgs a{logits, ld_logits, T,     E,    k,          score,    n_group, topk_group, group_score,
                    renorm, scale,     bias,  token_mask, topk_ids, topk_w, load};
  if (dtype == MOE_DT_F32) return route_by_size<float>(a, stream);
  if (dtype == MOE_DT_BF16) return route_by_size<__nv_bfloat16>(a, stream);
  return route_by_size<__half>(a, stream);
}

extern "C" moe_status moe_route_backward(const void* logits, int dtype, int64_t ld_logits, int T, int E, int k,
                                         int score, int renorm, float scale, const uint8_t* token_mask,
                                         const int32_t* topk_ids, const float* d_w, void* d_logits,
                                         int64_t ld_d_logits, cudaStream_t stream) {
  clear_error();
  moe_status st = route_check(dtype, ld_logits, T, E, k, score);
  if (st != MOE_OK) return st;
  MOE_ARG(ld_d_logits >= E, "the gradient's row distance must be >= E (got %lld)", (long long)ld_d_logits);
  if (T == 0) return MOE_OK;
  MOE_ARG(logits && topk_ids && d_w && d_logits, "null pointer");
  MOE_ARG(d_logits != logits, "d_logits must not be the logits");
  const RouteBwdArgs a{logits, ld_logits, T, E, k, score, renorm, scale, token_mask, topk_ids, d_w, d_logits,
                       ld_d_logits};
  ProfScope ps(MOE_K_ROUTE_BWD, stream);
  const cudaError_t e = dtype == MOE_DT_F32    ? launch_route_bwd<float>(a, stream)
                        : dtype == MOE_DT_BF16 ? launch_route_bwd<__nv_bfloat16>(a, stream)
                                               : launch_route_bwd<__half>(a, stream);
  if (e != cudaSuccess) return cuda_fail(e, "route_bwd_kernel");
  return check_launch("route_bwd_kernel");
}
