// Norms before and after a block, fused with the block's gate and residual
// scale, and their gradient:
//   r_y = (mean y^2 + eps)^-1/2,  v = y r_y g_post,  u = a x + gate v,
//   r_u = (mean u^2 + eps)^-1/2,  h = u r_u g_next.
// Gradient, with du, dh coming in and A = dh g_next:
//   D  = du + r_u (A - u r_u^2 mean(A u))           the gradient of u
//   dx = a D,  dgate = sum v D,  dg_next = sum dh u r_u
//   B  = gate D g_post,  dg_post = sum gate D y r_y
//   dy = r_y (B - y r_y^2 mean(B y))
//
// A row is held in the registers of a group of NT threads (a warp, or the whole
// block); thread i owns the same columns of every row, so the column sums of
// the gradient stay in its registers until the block is done.  Their partial
// sums go to the workspace, one row per block, and a second kernel adds them in
// block order.
#include <math.h>

#include "dtype.cuh"

namespace moe {

struct NormArgs {
  int T, H, w_dtype, gate_mode;
  float alpha, eps;
  const void *x, *y, *post, *gate, *next;
  long long ld_x, ld_y;
  void *x_out, *h;
  long long ld_xo, ld_h;
  // gradient
  const void *d_xo, *d_h;
  long long ld_dxo, ld_dh;
  void *d_x, *d_y;
  long long ld_dx, ld_dy;
  float *d_gate_token, *part;   // part: [blocks][3][H], post, gate, next
  int want_post, want_gate, want_next;
};

// VEC elements at p as fp32 (VEC 8: 16-byte accesses, p aligned).
template <int VEC, typename T>
__device__ __forceinline__ void load_vec(const T* p, float* f) {
  if constexpr (VEC == 1) {
    f[0] = to_f32(p[0]);
  } else {
    uint4 q[sizeof(T) / 2];
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) q[i] = reinterpret_cast<const uint4*>(p)[i];
    const T* e = reinterpret_cast<const T*>(q);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = to_f32(e[i]);
  }
}
template <int VEC, typename T>
__device__ __forceinline__ void store_vec(T* p, const float* f) {
  if constexpr (VEC == 1) {
    p[0] = from_f32<T>(f[0]);
  } else {
    uint4 q[sizeof(T) / 2];
    T* e = reinterpret_cast<T*>(q);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = from_f32<T>(f[i]);
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = q[i];
  }
}

// Sums of N values over the NT threads of a row, the same in all of them.
template <int NT, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*red)[N]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
  if constexpr (NT > 32) {
    const int wid = threadIdx.x >> 5;
    __syncthreads();   // the sums before these have been read
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int n = 0; n < N; ++n) red[wid][n] = v[n];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      v[n] = 0.f;
#pragma unroll
      for (int i = 0; i < NT / 32; ++i) v[n] += red[i][n];
    }
  }
}

template <int NT>
constexpr int kRowThreads = NT < 128 ? 128 : NT;   // threads of a block

template <typename TX, typename TY, int VEC, int NV, int NT>
__global__ void __launch_bounds__(kRowThreads<NT>) block_norm_kernel(const NormArgs a) {
  __shared__ float red[32][1];
  constexpr int kRows = kRowThreads<NT> / NT;   // rows a block works on at once
  const int tid = threadIdx.x % NT, H = a.H;
  for (long long t = (long long)blockIdx.x * kRows + threadIdx.x / NT; t < a.T; t += (long long)gridDim.x * kRows) {
    float u[NV][VEC];
    const TX* x = reinterpret_cast<const TX*>(a.x) + t * a.ld_x;
    float gt = 1.f;
    if (a.gate_mode == MOE_GATE_TOKEN) gt = load_any(a.gate, a.w_dtype, t);
    if (a.y) {
      const TY* y = reinterpret_cast<const TY*>(a.y) + t * a.ld_y;
      float ss[1] = {0.f};
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * NT + tid) * VEC;
#pragma unroll
        for (int j = 0; j < VEC; ++j) u[i][j] = 0.f;
        if (c < H) load_vec<VEC>(y + c, u[i]);
#pragma unroll
        for (int j = 0; j < VEC; ++j) ss[0] = fmaf(u[i][j], u[i][j], ss[0]);
      }
      float r = 1.f;
      if (a.post) {
        row_sums<NT>(ss, red);
        r = 1.f / sqrtf(ss[0] / (float)H + a.eps);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * NT + tid) * VEC;
        if (c >= H) continue;
        float xv[VEC];
        load_vec<VEC>(x + c, xv);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          float v = u[i][j] * r;
          if (a.post) v *= load_any(a.post, a.w_dtype, c + j);
          const float g = a.gate_mode == MOE_GATE_CHANNEL ? load_any(a.gate, a.w_dtype, c + j) : gt;
          u[i][j] = fmaf(g, v, a.alpha * xv[j]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * NT + tid) * VEC;
#pragma unroll
        for (int j = 0; j < VEC; ++j) u[i][j] = 0.f;
        if (c < H) load_vec<VEC>(x + c, u[i]);
#pragma unroll
        for (int j = 0; j < VEC; ++j) u[i][j] *= a.alpha;
      }
    }
    if (a.x_out) {
      TX* xo = reinterpret_cast<TX*>(a.x_out) + t * a.ld_xo;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * NT + tid) * VEC;
        if (c < H) store_vec<VEC>(xo + c, u[i]);
      }
    }
    if (a.next) {
      float ss[1] = {0.f};
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) ss[0] = fmaf(u[i][j], u[i][j], ss[0]);
      row_sums<NT>(ss, red);
      const float r = 1.f / sqrtf(ss[0] / (float)H + a.eps);
      TY* h = reinterpret_cast<TY*>(a.h) + t * a.ld_h;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * NT + tid) * VEC;
        if (c >= H) continue;
        float hv[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) hv[j] = u[i][j] * r * load_any(a.next, a.w_dtype, c + j);
        store_vec<VEC>(h + c, hv);
      }
    }
  }
}

template <typename TX, typename TY, int VEC, int NV, int NT>
__global__ void __launch_bounds__(kRowThreads<NT>) block_norm_bwd_kernel(const NormArgs a) {
  __shared__ float red1[32][1], red2[32][2];
  constexpr int kRows = kRowThreads<NT> / NT;
  const int tid = threadIdx.x % NT, H = a.H;
  const float inv_h = 1.f / (float)H;
  float acc_post[NV][VEC], acc_gate[NV][VEC], acc_next[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) acc_post[i][j] = acc_gate[i][j] = acc_next[i][j] = 0.f;
  for (long long t = (long long)blockIdx.x * kRows + threadIdx.x / NT; t < a.T; t += (long long)gridDim.x * kRows) {
    float y[NV][VEC], u[NV][VEC], d[NV][VEC];
    float gt = 1.f, ry = 1.f;
    if (a.gate_mode == MOE_GATE_TOKEN) gt = load_any(a.gate, a.w_dtype, t);
    const TX* x = reinterpret_cast<const TX*>(a.x) + t * a.ld_x;
    {
      float ss[1] = {0.f};
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * NT + tid) * VEC;
#pragma unroll
        for (int j = 0; j < VEC; ++j) y[i][j] = u[i][j] = d[i][j] = 0.f;
        if (c >= H) continue;
        if (a.y) load_vec<VEC>(reinterpret_cast<const TY*>(a.y) + t * a.ld_y + c, y[i]);
        if (a.d_xo) load_vec<VEC>(reinterpret_cast<const TX*>(a.d_xo) + t * a.ld_dxo + c, d[i]);
        load_vec<VEC>(x + c, u[i]);
#pragma unroll
        for (int j = 0; j < VEC; ++j) ss[0] = fmaf(y[i][j], y[i][j], ss[0]);
      }
      if (a.post) {
        row_sums<NT>(ss, red1);
        ry = 1.f / sqrtf(ss[0] * inv_h + a.eps);
      }
    }
    // from here y is n(y)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * NT + tid) * VEC;
      if (c >= H) continue;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        y[i][j] *= ry;
        u[i][j] *= a.alpha;
        if (a.y) {
          const float v = a.post ? y[i][j] * load_any(a.post, a.w_dtype, c + j) : y[i][j];
          const float g = a.gate_mode == MOE_GATE_CHANNEL ? load_any(a.gate, a.w_dtype, c + j) : gt;
          u[i][j] = fmaf(g, v, u[i][j]);
        }
      }
    }
    if (a.next) {
      float dh[NV][VEC];
      float s[2] = {0.f, 0.f};   // sum u^2, sum dh g_next u
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * NT + tid) * VEC;
#pragma unroll
        for (int j = 0; j < VEC; ++j) dh[i][j] = 0.f;
        if (c >= H) continue;
        load_vec<VEC>(reinterpret_cast<const TY*>(a.d_h) + t * a.ld_dh + c, dh[i]);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          s[0] = fmaf(u[i][j], u[i][j], s[0]);
          s[1] = fmaf(dh[i][j] * load_any(a.next, a.w_dtype, c + j), u[i][j], s[1]);
        }
      }
      row_sums<NT>(s, red2);
      const float ru = 1.f / sqrtf(s[0] * inv_h + a.eps);
      const float m = ru * ru * s[1] * inv_h;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * NT + tid) * VEC;
        if (c >= H) continue;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          d[i][j] = fmaf(ru, dh[i][j] * load_any(a.next, a.w_dtype, c + j) - u[i][j] * m, d[i][j]);
          acc_next[i][j] = fmaf(dh[i][j], u[i][j] * ru, acc_next[i][j]);
        }
      }
    }
    TX* dx = reinterpret_cast<TX*>(a.d_x) + t * a.ld_dx;
    float s[2] = {0.f, 0.f};   // sum B n(y), sum D v
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * NT + tid) * VEC;
      if (c >= H) continue;
      float o[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) o[j] = a.alpha * d[i][j];
      store_vec<VEC>(dx + c, o);
      if (!a.y) continue;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float p = a.post ? load_any(a.post, a.w_dtype, c + j) : 1.f;
        const float g = a.gate_mode == MOE_GATE_CHANNEL ? load_any(a.gate, a.w_dtype, c + j) : gt;
        const float dv = d[i][j] * y[i][j];
        s[1] = fmaf(dv, p, s[1]);
        acc_gate[i][j] = fmaf(dv, p, acc_gate[i][j]);
        acc_post[i][j] = fmaf(dv, g, acc_post[i][j]);
        s[0] = fmaf(dv, g * p, s[0]);
        d[i][j] *= g * p;   // B
      }
    }
    if (!a.y) continue;
    if (a.post || a.d_gate_token) row_sums<NT>(s, red2);
    if (a.d_gate_token && tid == 0) a.d_gate_token[t] = s[1];
    TY* dy = reinterpret_cast<TY*>(a.d_y) + t * a.ld_dy;
    const float m = a.post ? s[0] * inv_h : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * NT + tid) * VEC;
      if (c >= H) continue;
      float o[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) o[j] = ry * (d[i][j] - y[i][j] * m);
      store_vec<VEC>(dy + c, o);
    }
  }
  // the rows' partial column sums, one line of the workspace for each group of threads
  float* part = a.part + ((long long)blockIdx.x * kRows + threadIdx.x / NT) * 3 * H;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * NT + tid) * VEC;
    if (c >= H) continue;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      if (a.want_post) part[c + j] = acc_post[i][j];
      if (a.want_gate) part[H + c + j] = acc_gate[i][j];
      if (a.want_next) part[2 * H + c + j] = acc_next[i][j];
    }
  }
}

// Adds the lines of the workspace, in their order: blockIdx.y is the array.
__global__ void __launch_bounds__(256) column_sum_kernel(const float* part, int lines, int H, float* post, float* gate,
                                                         float* next) {
  float* out = blockIdx.y == 0 ? post : blockIdx.y == 1 ? gate : next;
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (!out || c >= H) return;
  float s = 0.f;
  for (int i = 0; i < lines; ++i) s += part[((long long)i * 3 + blockIdx.y) * H + c];
  out[c] = s;
}

// The (threads, vectors per thread) a row of H columns is held in.
struct RowShape {
  int vec, nv, nt;
};
static RowShape row_shape(int H, bool vec) {
  if (vec) {
    const int n = H / 8;
    if (n <= 32) return {8, 1, 32};
    if (n <= 128) return {8, 4, 32};
    if (n <= 256) return {8, 2, 128};
    if (n <= 512) return {8, 2, 256};
    if (n <= 1024) return {8, 2, 512};
    return {8, 2, 1024};
  }
  return H <= 1024 ? RowShape{1, 4, 256} : RowShape{1, 16, 1024};
}

// Blocks of the gradient kernel: what the workspace has lines for.
static int bwd_blocks(long long T, int rows) {
  const long long need = (T + rows - 1) / rows, most = device_sms() * 2;
  return (int)(need < most ? need : most);
}

template <typename TX, typename TY, int VEC, int NV, int NT>
static moe_status launch_norm(const NormArgs& a, bool bwd, cudaStream_t s) {
  constexpr int kRows = kRowThreads<NT> / NT;
  if (!bwd) {
    const long long need = ((long long)a.T + kRows - 1) / kRows;
    ProfScope ps(MOE_K_NORM, s);
    block_norm_kernel<TX, TY, VEC, NV, NT><<<(unsigned)(need < (1 << 20) ? need : 1 << 20), kRowThreads<NT>, 0, s>>>(a);
    return check_launch("block_norm_kernel");
  }
  ProfScope ps(MOE_K_NORM_BWD, s);
  block_norm_bwd_kernel<TX, TY, VEC, NV, NT><<<bwd_blocks(a.T, kRows), kRowThreads<NT>, 0, s>>>(a);
  return check_launch("block_norm_bwd_kernel");
}

template <typename TX, typename TY>
static moe_status norm_by_shape(const NormArgs& a, bool vec, bool bwd, cudaStream_t s) {
  const RowShape r = row_shape(a.H, vec);
  if (r.vec == 1) return r.nt == 256 ? launch_norm<TX, TY, 1, 4, 256>(a, bwd, s) : launch_norm<TX, TY, 1, 16, 1024>(a, bwd, s);
  if (r.nt == 32) return r.nv == 1 ? launch_norm<TX, TY, 8, 1, 32>(a, bwd, s) : launch_norm<TX, TY, 8, 4, 32>(a, bwd, s);
  if (r.nt == 128) return launch_norm<TX, TY, 8, 2, 128>(a, bwd, s);
  if (r.nt == 256) return launch_norm<TX, TY, 8, 2, 256>(a, bwd, s);
  if (r.nt == 512) return launch_norm<TX, TY, 8, 2, 512>(a, bwd, s);
  return launch_norm<TX, TY, 8, 2, 1024>(a, bwd, s);
}

static moe_status norm_by_type(const NormArgs& a, int xd, int yd, bool vec, bool bwd, cudaStream_t s) {
  if (xd == MOE_DT_BF16) return norm_by_shape<__nv_bfloat16, __nv_bfloat16>(a, vec, bwd, s);
  if (xd == MOE_DT_F16) return norm_by_shape<__half, __half>(a, vec, bwd, s);
  if (yd == MOE_DT_BF16) return norm_by_shape<float, __nv_bfloat16>(a, vec, bwd, s);
  if (yd == MOE_DT_F16) return norm_by_shape<float, __half>(a, vec, bwd, s);
  return norm_by_shape<float, float>(a, vec, bwd, s);
}

// Whether a tensor's rows can be read in 16-byte vectors.
static bool vec_ok(const void* p, long long ld, int dtype) {
  return !p || ((uintptr_t)p % 16 == 0 && ld * (long long)dtype_size(dtype) % 16 == 0);
}

static moe_status norm_check(int T, int H, int xd, int yd, int wd, const void* x, int64_t ld_x, const void* y,
                             int64_t ld_y, const void* post, const void* gate, int gate_mode) {
  MOE_ARG(T >= 0, "T must be >= 0");
  MOE_ARG(H >= 1 && H <= 16384, "H must be in [1, 16384] (got %d)", H);
  MOE_ARG(known_dtype(xd) && known_dtype(yd) && known_dtype(wd), "unknown type (x %d, y %d, weights %d)", xd, yd, wd);
  MOE_ARG(xd == yd || xd == MOE_DT_F32, "x must be of y's type or fp32");
  MOE_ARG(gate_mode >= MOE_GATE_NONE && gate_mode <= MOE_GATE_TOKEN, "unknown gate mode %d", gate_mode);
  if (T == 0) return MOE_OK;
  MOE_ARG(x, "null pointer");
  MOE_ARG(ld_x >= H && (!y || ld_y >= H), "a row distance is below H");
  MOE_ARG(y || (!post && gate_mode == MOE_GATE_NONE), "post_weight and gate need y");
  MOE_ARG((gate_mode == MOE_GATE_NONE) == !gate, "gate and gate_mode do not go together");
  return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_block_norm(int T, int H, int x_dtype, int y_dtype, int w_dtype, const void* x, int64_t ld_x,
                                     const void* y, int64_t ld_y, const void* post_weight, const void* gate,
                                     int gate_mode, float residual_scale, const void* next_weight, float eps,
                                     void* x_out, int64_t ld_x_out, void* h, int64_t ld_h, cudaStream_t stream) {
  clear_error();
  moe_status st = norm_check(T, H, x_dtype, y_dtype, w_dtype, x, ld_x, y, ld_y, post_weight, gate, gate_mode);
  if (st != MOE_OK || T == 0) return st;
  MOE_ARG(!next_weight == !h, "h and next_weight do not go together");
  MOE_ARG(x_out || h, "neither x_out nor h is asked for");
  MOE_ARG((!x_out || ld_x_out >= H) && (!h || ld_h >= H), "a row distance is below H");
  MOE_ARG(!x_out || x_out != x || ld_x_out == ld_x, "x_out in place needs x's row distance");
  NormArgs a = {};
  a.T = T, a.H = H, a.w_dtype = w_dtype, a.gate_mode = gate_mode, a.alpha = residual_scale, a.eps = eps;
  a.x = x, a.y = y, a.post = post_weight, a.gate = gate, a.next = next_weight;
  a.ld_x = ld_x, a.ld_y = ld_y, a.x_out = x_out, a.h = h, a.ld_xo = ld_x_out, a.ld_h = ld_h;
  const bool vec = H % 8 == 0 && vec_ok(x, ld_x, x_dtype) && vec_ok(y, ld_y, y_dtype) &&
                   vec_ok(x_out, ld_x_out, x_dtype) && vec_ok(h, ld_h, y_dtype);
  return norm_by_type(a, x_dtype, y_dtype, vec, false, stream);
}

extern "C" size_t moe_block_norm_backward_workspace(int T, int H) {
  if (T <= 0 || H <= 0) return 0;
  // the shapes of up to 4 rows a block have the most lines
  return (size_t)bwd_blocks(T, 1) * 4 * 3 * H * sizeof(float);
}

extern "C" moe_status moe_block_norm_backward(int T, int H, int x_dtype, int y_dtype, int w_dtype, const void* x,
                                              int64_t ld_x, const void* y, int64_t ld_y, const void* d_x_out,
                                              int64_t ld_d_x_out, const void* d_h, int64_t ld_d_h,
                                              const void* post_weight, const void* gate, int gate_mode,
                                              float residual_scale, const void* next_weight, float eps, void* d_x,
                                              int64_t ld_d_x, void* d_y, int64_t ld_d_y, float* d_post_weight,
                                              float* d_gate, float* d_next_weight, void* workspace,
                                              size_t workspace_bytes, cudaStream_t stream) {
  clear_error();
  moe_status st = norm_check(T, H, x_dtype, y_dtype, w_dtype, x, ld_x, y, ld_y, post_weight, gate, gate_mode);
  if (st != MOE_OK) return st;
  if (T == 0) {
    if (d_post_weight) MOE_CUDA(cudaMemsetAsync(d_post_weight, 0, H * sizeof(float), stream));
    if (d_gate && gate_mode == MOE_GATE_CHANNEL) MOE_CUDA(cudaMemsetAsync(d_gate, 0, H * sizeof(float), stream));
    if (d_next_weight) MOE_CUDA(cudaMemsetAsync(d_next_weight, 0, H * sizeof(float), stream));
    return MOE_OK;
  }
  MOE_ARG(d_x && !d_y == !y, "d_x is needed, and d_y exactly with y");
  MOE_ARG(!next_weight == !d_h, "d_h and next_weight do not go together");
  MOE_ARG(d_x_out || d_h, "neither d_x_out nor d_h is given");
  MOE_ARG((!d_post_weight || post_weight) && (!d_gate || gate) && (!d_next_weight || next_weight),
          "a gradient is asked for of a weight that is not there");
  MOE_ARG((!d_x_out || ld_d_x_out >= H) && (!d_h || ld_d_h >= H) && ld_d_x >= H && (!d_y || ld_d_y >= H),
          "a row distance is below H");
  MOE_ARG(d_x != d_x_out || ld_d_x == ld_d_x_out, "d_x in place needs d_x_out's row distance");
  MOE_ARG(!d_y || d_y != d_h || ld_d_y == ld_d_h, "d_y in place needs d_h's row distance");
  const bool sums = d_post_weight || d_next_weight || (d_gate && gate_mode == MOE_GATE_CHANNEL);
  MOE_ARG(!sums || (workspace && (uintptr_t)workspace % 16 == 0 &&
                    workspace_bytes >= moe_block_norm_backward_workspace(T, H)),
          "workspace missing, misaligned or too small (%zu bytes, %zu needed)", workspace_bytes,
          moe_block_norm_backward_workspace(T, H));
  NormArgs a = {};
  a.T = T, a.H = H, a.w_dtype = w_dtype, a.gate_mode = gate_mode, a.alpha = residual_scale, a.eps = eps;
  a.x = x, a.y = y, a.post = post_weight, a.gate = gate, a.next = next_weight;
  a.ld_x = ld_x, a.ld_y = ld_y;
  a.d_xo = d_x_out, a.d_h = d_h, a.ld_dxo = ld_d_x_out, a.ld_dh = ld_d_h;
  a.d_x = d_x, a.d_y = d_y, a.ld_dx = ld_d_x, a.ld_dy = ld_d_y;
  a.d_gate_token = gate_mode == MOE_GATE_TOKEN ? d_gate : nullptr;
  a.part = (float*)workspace;
  a.want_post = d_post_weight != nullptr, a.want_next = d_next_weight != nullptr;
  a.want_gate = d_gate && gate_mode == MOE_GATE_CHANNEL;
  const bool vec = H % 8 == 0 && vec_ok(x, ld_x, x_dtype) && vec_ok(y, ld_y, y_dtype) &&
                   vec_ok(d_x_out, ld_d_x_out, x_dtype) && vec_ok(d_h, ld_d_h, y_dtype) &&
                   vec_ok(d_x, ld_d_x, x_dtype) && vec_ok(d_y, ld_d_y, y_dtype);
  st = norm_by_type(a, x_dtype, y_dtype, vec, true, stream);
  if (st != MOE_OK || !sums) return st;
  const RowShape r = row_shape(H, vec);
  const int rows = (r.nt < 128 ? 128 : r.nt) / r.nt;
  column_sum_kernel<<<dim3((H + 255) / 256, 3), 256, 0, stream>>>(
      a.part, bwd_blocks(T, rows) * rows, H, d_post_weight, a.want_gate ? d_gate : nullptr, d_next_weight);
  return check_launch("column_sum_kernel");
}
