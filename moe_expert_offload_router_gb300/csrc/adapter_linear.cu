// A shared projection with low-rank adapters of many requests beside it:
//   out[t] = W x[t] + scale[a] B[a] (A[a] x[t]),  a = adapter_ids[t].
//
// A first kernel takes u[t] = scale[a] A[a] x[t] (fp32 [T, R], one warp per
// token); the projection's kernel adds B[a] u[t] to its sums before rounding.
#include <math.h>

#include "dtype.cuh"

namespace moe {

struct LinearArgs {
  int T, H, N, n, R, out_dtype;
  const void *x, *W, *A, *B;
  long long ld_x, ld_w, ld_out;
  const int32_t* ids;
  const float* scale;
  void* out;
  float* u;
  int32_t* err;
};

template <typename TE>
__global__ void __launch_bounds__(128) adapter_shrink_kernel(const LinearArgs a) {
  const int t = (int)((blockIdx.x * (size_t)blockDim.x + threadIdx.x) >> 5), lane = threadIdx.x & 31;
  if (t >= a.T) return;
  const int id = a.ids[t];
  if (id >= a.n && a.err && lane == 0) atomicCAS(a.err, MOE_OK, MOE_ERR_INVALID);
  if (id < 0 || id >= a.n) return;
  const TE* x = reinterpret_cast<const TE*>(a.x) + t * a.ld_x;
  const float c = a.scale ? a.scale[id] : 1.f;
  for (int r = 0; r < a.R; ++r) {
    const TE* row = reinterpret_cast<const TE*>(a.A) + ((long long)id * a.R + r) * a.H;
    float s = 0.f;
    for (int i = lane; i < a.H; i += 32) s = fmaf(to_f32(row[i]), to_f32(x[i]), s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) a.u[(long long)t * a.R + r] = c * s;
  }
}

// 64 tokens x 64 outputs per block of 256 threads, 4 x 4 per thread.
template <typename TE>
__global__ void __launch_bounds__(256) linear_kernel(const LinearArgs a) {
  __shared__ float xs[16][65], ws[16][65];
  const int t0 = blockIdx.y * 64, n0 = blockIdx.x * 64, tid = threadIdx.x;
  const int tx = tid % 16, ty = tid / 16;
  const TE* x = reinterpret_cast<const TE*>(a.x);
  const TE* W = reinterpret_cast<const TE*>(a.W);
  float acc[4][4] = {};
  for (int k0 = 0; k0 < a.H; k0 += 16) {
    for (int i = tid; i < 64 * 16; i += 256) {
      const int r = i / 16, c = i % 16;
      xs[c][r] = t0 + r < a.T && k0 + c < a.H ? to_f32(x[(t0 + r) * a.ld_x + k0 + c]) : 0.f;
      ws[c][r] = n0 + r < a.N && k0 + c < a.H ? to_f32(W[(n0 + r) * a.ld_w + k0 + c]) : 0.f;
    }
    __syncthreads();
    for (int c = 0; c < 16; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xs[c][ty * 4 + i], ws[c][tx * 4 + j], acc[i][j]);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = t0 + ty * 4 + i;
    if (t >= a.T) continue;
    const int id = a.n ? a.ids[t] : -1;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tx * 4 + j;
      if (n >= a.N) continue;
      float s = acc[i][j];
      if (id >= 0 && id < a.n) {
        const TE* b = reinterpret_cast<const TE*>(a.B) + ((long long)id * a.N + n) * a.R;
        for (int r = 0; r < a.R; ++r) s = fmaf(to_f32(b[r]), a.u[(long long)t * a.R + r], s);
      }
      const long long o = t * a.ld_out + n;
      if (a.out_dtype == MOE_DT_F32) reinterpret_cast<float*>(a.out)[o] = s;
      else reinterpret_cast<TE*>(a.out)[o] = from_f32<TE>(s);
    }
  }
}

template <typename TE>
static moe_status launch_linear(const LinearArgs& a, cudaStream_t s) {
  ProfScope ps(MOE_K_LINEAR, s);
  if (a.n) {
    adapter_shrink_kernel<TE><<<(unsigned)((a.T + 3LL) / 4), 128, 0, s>>>(a);
    const moe_status st = check_launch("adapter_shrink_kernel");
    if (st != MOE_OK) return st;
  }
  linear_kernel<TE><<<dim3((a.N + 63) / 64, (a.T + 63) / 64), 256, 0, s>>>(a);
  return check_launch("linear_kernel");
}

}  // namespace moe

using namespace moe;

extern "C" size_t moe_adapter_linear_workspace(int T, int H, int N, int n_adapters, int R) {
  if (T <= 0 || H <= 0 || N <= 0 || n_adapters <= 0 || R <= 0) return 0;
  return ((size_t)T * R * sizeof(float) + 15) / 16 * 16;
}

extern "C" moe_status moe_adapter_linear(int T, int H, int N, int dtype, int out_dtype, const void* x, int64_t ld_x,
                                         const void* W, int64_t ld_w, int n_adapters, int R, const void* lora_a,
                                         const void* lora_b, const int32_t* adapter_ids, const float* lora_scale,
                                         void* out, int64_t ld_out, void* workspace, size_t workspace_bytes,
                                         int32_t* d_error, cudaStream_t stream) {
  clear_error();
  MOE_ARG(T >= 0 && N >= 1, "T must be >= 0 and N >= 1 (got %d, %d)", T, N);
  MOE_ARG(H >= 8 && H % 8 == 0, "H must be a multiple of 8 (got %d)", H);
  MOE_ARG(dtype == MOE_DT_BF16 || dtype == MOE_DT_F16, "x and W must be bf16 or f16 (type %d)", dtype);
  MOE_ARG(out_dtype == dtype || out_dtype == MOE_DT_F32, "out must be of x's type or fp32 (type %d)", out_dtype);
  MOE_ARG(n_adapters >= 0, "n_adapters must be >= 0 (got %d)", n_adapters);
  MOE_ARG(!n_adapters || (R >= 8 && R <= 128 && R % 8 == 0), "R must be a multiple of 8 up to 128 (got %d)", R);
  if (T == 0) return MOE_OK;
  MOE_ARG(x && W && out, "null pointer");
  MOE_ARG(ld_x >= H && ld_w >= H && ld_out >= N, "a row distance is below the row's length");
  MOE_ARG((uintptr_t)x % 16 == 0 && (uintptr_t)W % 16 == 0 && ld_x % 8 == 0 && ld_w % 8 == 0,
          "x and W need rows on 16-byte boundaries");
  if (n_adapters) {
    MOE_ARG(lora_a && lora_b && adapter_ids, "null pointer");
    MOE_ARG((uintptr_t)lora_a % 16 == 0 && (uintptr_t)lora_b % 16 == 0, "lora_a and lora_b must be 16-byte aligned");
  }
  const size_t need = moe_adapter_linear_workspace(T, H, N, n_adapters, R);
  MOE_ARG(!need || (workspace && (uintptr_t)workspace % 16 == 0 && workspace_bytes >= need),
          "workspace missing, misaligned or too small (%zu bytes, %zu needed)", workspace_bytes, need);
  const LinearArgs a{T,    H,    N,      n_adapters, R,          out_dtype, x,  W, lora_a, lora_b, ld_x,
                     ld_w, ld_out, adapter_ids, lora_scale, out, (float*)workspace, d_error};
  return dtype == MOE_DT_BF16 ? launch_linear<__nv_bfloat16>(a, stream) : launch_linear<__half>(a, stream);
}
