// Routing to experts: softmax or sigmoid scores, a balance bias that moves the
// choice but not the weights, expert groups, top-k, renormalised weights; and
// the gradient of the weights with respect to the logits.
//
// One warp per token; lane l holds experts l * VPL .. l * VPL + VPL - 1, so
// that the lowest lane among equals holds the lowest id.  Each of the k rounds
// takes the warp-wide maximum key; the lane that holds it drops it.
#include <math.h>

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

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
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

__device__ __forceinline__ float sigmoid_f32(float z) { return __fdiv_rn(1.f, 1.f + expf(-z)); }
// e^(z - top), also where both are +inf; 0 for z = -inf.
__device__ __forceinline__ float exp_below(float z, float top) {
  return z == -INFINITY ? 0.f : (z == top ? 1.f : expf(z - top));
}

template <int VPL, typename TL>
__global__ void __launch_bounds__(128) route_kernel(const RouteArgs a) {
  const int t = (int)((blockIdx.x * (size_t)blockDim.x + threadIdx.x) >> 5);
  const int lane = threadIdx.x & 31;
  if (t >= a.T) return;
  const int k = a.k, E = a.E;
  const TL* row = reinterpret_cast<const TL*>(a.logits) + (long long)t * a.ld;
  int my_id = -1;
  float top = -INFINITY, den = 0.f;
  if (!a.mask || a.mask[t]) {
    float key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane * VPL + i;
      key[i] = e < E ? load_logit(row, e) : -INFINITY;
      top = fmaxf(top, key[i]);
    }
    top = warp_max(top);
    const bool grouped = a.topk_group < a.n_group;
    const bool scored = a.bias || (grouped && a.group_score == MOE_GROUP_TOP2);
    if (a.score == MOE_SCORE_SOFTMAX && (scored || !a.renorm)) {
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
    float val[VPL];   // what groups are valued by, and the key where there is a bias
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      val[i] = key[i];
      if (scored && key[i] > -INFINITY) {
        const float s = a.score == MOE_SCORE_SIGMOID ? sigmoid_f32(key[i]) : __fdiv_rn(exp_below(key[i], top), den);
        val[i] = a.bias ? s + a.bias[lane * VPL + i] : s;
        if (a.bias) key[i] = val[i];
      }
    }
    if (grouped) {
      const int gs = E / a.n_group;
      float worth = -INFINITY;   // of group `lane`
      for (int g = 0; g < a.n_group; ++g) {
        float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          const int e = lane * VPL + i;
          if (e >= g * gs && e < (g + 1) * gs) {
            m2 = fmaxf(m2, fminf(m1, val[i]));
            m1 = fmaxf(m1, val[i]);
          }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const float o1 = __shfl_xor_sync(0xffffffffu, m1, o), o2 = __shfl_xor_sync(0xffffffffu, m2, o);
          m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
          m1 = fmaxf(m1, o1);
        }
        if (lane == g) worth = a.group_score == MOE_GROUP_MAX || m2 == -INFINITY ? m1 : m1 + m2;
      }
      int rank = 0;
      for (int g = 0; g < a.n_group; ++g) {
        const float o = __shfl_sync(0xffffffffu, worth, g);
        rank += o > worth || (o == worth && g < lane);
      }
      const uint32_t keep = __ballot_sync(0xffffffffu, lane < a.n_group && rank < a.topk_group);
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int e = lane * VPL + i;
        if (e < E && !((keep >> (e / gs)) & 1)) key[i] = -INFINITY;
      }
    }
    for (int j = 0; j < k; ++j) {
      float best = key[0];
#pragma unroll
      for (int i = 1; i < VPL; ++i) best = fmaxf(best, key[i]);
      const float m = warp_max(best);
      if (!(m > -INFINITY)) break;
      const int win = __ffs(__ballot_sync(0xffffffffu, best == m)) - 1;
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
  // weights: lane j holds the j-th choice
  const float z = my_id >= 0 ? load_logit(row, my_id) : -INFINITY;
  float s;
  if (a.score == MOE_SCORE_SIGMOID) {
    s = my_id >= 0 ? sigmoid_f32(z) : 0.f;
  } else if (a.renorm) {
    s = exp_below(z, warp_max(z));
  } else {
    s = my_id >= 0 ? __fdiv_rn(exp_below(z, top), den) : 0.f;
  }
  if (a.renorm) {
    const float sum = warp_sum(s);
    s = sum > 0.f ? s / sum : 0.f;
  }
  if (lane < k) {
    a.ids[(long long)t * k + lane] = my_id;
    a.w[(long long)t * k + lane] = a.scale * s;
    if (a.load && my_id >= 0) atomicAdd(a.load + my_id, 1);
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

template <typename TL>
__global__ void __launch_bounds__(128) route_bwd_kernel(const RouteBwdArgs a) {
  const int t = (int)((blockIdx.x * (size_t)blockDim.x + threadIdx.x) >> 5);
  const int lane = threadIdx.x & 31;
  if (t >= a.T) return;
  const TL* row = reinterpret_cast<const TL*>(a.logits) + (long long)t * a.ld;
  TL* d = reinterpret_cast<TL*>(a.d) + (long long)t * a.ld_d;
  int id = -1;
  float g = 0.f, z = -INFINITY;
  if (lane < a.k && (!a.mask || a.mask[t])) {
    id = a.ids[(long long)t * a.k + lane];
    if (id >= 0 && id < a.E) z = load_logit(row, id);
    if (z > -INFINITY) g = a.scale * a.dw[(long long)t * a.k + lane];
    else id = -1;
  }
  float dj;
  if (a.score == MOE_SCORE_SOFTMAX && !a.renorm) {
    float top = -INFINITY, den = 0.f;
    if (!a.mask || a.mask[t]) {
      for (int e = lane; e < a.E; e += 32) top = fmaxf(top, load_logit(row, e));
      top = warp_max(top);
      for (int e = lane; e < a.E; e += 32) den += exp_below(load_logit(row, e), top);
      den = warp_sum(den);
    }
    const float p = id >= 0 ? exp_below(z, top) / den : 0.f;
    const float mean = warp_sum(g * p);
    dj = p * (g - mean);
    for (int e = lane; e < a.E; e += 32)
      d[e] = from_f32<TL>(den > 0.f ? -mean * (exp_below(load_logit(row, e), top) / den) : 0.f);
  } else {
    float q, c = 1.f;
    if (a.score == MOE_SCORE_SIGMOID) {
      q = id >= 0 ? sigmoid_f32(z) : 0.f;
      c = id >= 0 ? sigmoid_f32(-z) : 0.f;   // 1 - s without the cancellation
    } else {
      q = exp_below(z, warp_max(z));
    }
    float mean = 0.f;
    if (a.renorm) {
      const float sum = warp_sum(q);
      q = sum > 0.f ? q / sum : 0.f;
      mean = warp_sum(q * g);
    }
    dj = q * c * (g - mean);
    for (int e = lane; e < a.E; e += 32) d[e] = from_f32<TL>(0.f);
  }
  __syncwarp();   // the row is written before the chosen experts' values
  if (id >= 0) d[id] = from_f32<TL>(dj);
}

template <int VPL, typename TL>
static moe_status launch_route(const RouteArgs& a, cudaStream_t s) {
  ProfScope ps(MOE_K_ROUTE, s);
  route_kernel<VPL, TL><<<(unsigned)((a.T + 3LL) / 4), 128, 0, s>>>(a);
  return check_launch("route_kernel");
}

template <typename TL>
static moe_status route_by_size(const RouteArgs& a, cudaStream_t s) {
  const int vpl = (a.E + 31) / 32;
  if (vpl <= 1) return launch_route<1, TL>(a, s);
  if (vpl <= 2) return launch_route<2, TL>(a, s);
  if (vpl <= 4) return launch_route<4, TL>(a, s);
  if (vpl <= 8) return launch_route<8, TL>(a, s);
  if (vpl <= 16) return launch_route<16, TL>(a, s);
  if (vpl <= 32) return launch_route<32, TL>(a, s);
  return launch_route<64, TL>(a, s);
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
  const unsigned grid = (unsigned)((T + 3LL) / 4);
  ProfScope ps(MOE_K_ROUTE_BWD, stream);
  if (dtype == MOE_DT_F32) route_bwd_kernel<float><<<grid, 128, 0, stream>>>(a);
  else if (dtype == MOE_DT_BF16) route_bwd_kernel<__nv_bfloat16><<<grid, 128, 0, stream>>>(a);
  else route_bwd_kernel<__half><<<grid, 128, 0, stream>>>(a);
  return check_launch("route_bwd_kernel");
}
