// Norms before and after a block, fused with the block's gate and residual
// scale, and their gradient.  With w = gate * post_weight (per channel; for a
// gate per token w = post_weight and g_t the token's gate, else g_t = 1):
//   r_y = (mean y^2 + eps)^-1/2,  n = y r_y,  u = alpha x + g_t w n,
//   r_u = (mean u^2 + eps)^-1/2,  h = u r_u next.
// Gradient, with du, dh coming in, a = dh next and q = w n:
//   m  = r_u^2 mean(a u),  D = du + r_u (a - u m)          the gradient of u
//   dx = alpha D,  s = sum q D = sum q du + r_u (sum q a - m sum q u)
//   dy = r_y (g_t w D - n g_t mean(q D)),  d gate_t = s
//   E  = sum_t g_t D n:  d post = gate E,  d gate = post E;  d next = sum_t dh u r_u
// so a row takes two sums over its columns (five values in the second), and
// the three column gradients come from two column sums over the rows.
//
// Bound by HBM: x, y read and x_out, h written (forward: T = 8192, H = 4096 bf16,
// 268 MB in 43.9 us, 6.1 TB/s), x, y, du, dh read and dx, dy written (gradient: 403
// MB in 74.4 us with the column sums, 5.4 TB/s; its row kernel is as near to the
// issue slots as to HBM, hence the packed fp32 instructions).  A row is held in the registers of a group of NT
// threads (a warp, or the block), thread i owning the same columns of every
// row: its weights and its column sums stay in registers while the block walks
// over rows t, t + blocks, ...  Each thread copies its own columns of the next
// rows to shared memory (cp.async, a ring of S rows) and reads back nothing
// that another thread wrote, so the ring needs no barrier.  Partial column sums
// go to the workspace, one line a block; a second kernel adds them in block order.
#include <math.h>

#include <type_traits>

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
  float *d_gate_token, *part;   // part: [blocks][2][line], E and d next
  int sums;                     // whether a column sum is asked for
};

__host__ __device__ constexpr int column_line(int H) { return (H + 3) / 4 * 4; }

// Two fp32 values in one 64-bit register: Blackwell's packed fp32 instructions
// do both at once.  Columns are held as pairs (16-byte vectors of eight) or, in
// the unaligned form, as single floats, with the same operations.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 pack2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(F2 a) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(a.v));
  return f;
}
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ float mul(float a, float b) { return a * b; }
__device__ __forceinline__ float fma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float total(F2 a) {
  const float2 f = unpack2(a);
  return f.x + f.y;
}
__device__ __forceinline__ float total(float a) { return a; }
template <typename E>
__device__ __forceinline__ E splat(float f);
template <>
__device__ __forceinline__ F2 splat<F2>(float f) {
  return pack2(f, f);
}
template <>
__device__ __forceinline__ float splat<float>(float f) {
  return f;
}
template <int VEC>
using Elem = typename std::conditional<VEC == 8, F2, float>::type;
template <int VEC>
constexpr int kElems = VEC == 8 ? 4 : 1;

__device__ __forceinline__ void widen(const uint4 (&q)[2], const float*, F2* e) {
  e[0] = pack2(__uint_as_float(q[0].x), __uint_as_float(q[0].y));
  e[1] = pack2(__uint_as_float(q[0].z), __uint_as_float(q[0].w));
  e[2] = pack2(__uint_as_float(q[1].x), __uint_as_float(q[1].y));
  e[3] = pack2(__uint_as_float(q[1].z), __uint_as_float(q[1].w));
}
__device__ __forceinline__ void widen(const uint4 (&q)[1], const __nv_bfloat16*, F2* e) {
  const uint32_t w[4] = {q[0].x, q[0].y, q[0].z, q[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) e[i] = pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ void widen(const uint4 (&q)[1], const __half*, F2* e) {
  const uint32_t w[4] = {q[0].x, q[0].y, q[0].z, q[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    e[i] = pack2(f.x, f.y);
  }
}
__device__ __forceinline__ uint32_t narrow(float2 f, const __nv_bfloat16*) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t narrow(float2 f, const __half*) {
  const __half2 h = __floats2half2_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename T>
constexpr int kPieces = (int)sizeof(T) / 2;   // 16-byte pieces of eight elements

// Eight elements (16-byte aligned) or one at p, as fp32.
template <typename T>
__device__ __forceinline__ void load_vec(const T* p, F2* e) {
  uint4 q[kPieces<T>];
#pragma unroll
  for (int i = 0; i < kPieces<T>; ++i) q[i] = reinterpret_cast<const uint4*>(p)[i];
  widen(q, p, e);
}
template <typename T>
__device__ __forceinline__ void load_vec(const T* p, float* e) {
  e[0] = to_f32(p[0]);
}
template <typename T>
__device__ __forceinline__ void store_vec(T* p, const F2* e) {
  if constexpr (sizeof(T) == 4) {
    const float2 a = unpack2(e[0]), b = unpack2(e[1]), c = unpack2(e[2]), d = unpack2(e[3]);
    reinterpret_cast<float4*>(p)[0] = make_float4(a.x, a.y, b.x, b.y);
    reinterpret_cast<float4*>(p)[1] = make_float4(c.x, c.y, d.x, d.y);
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(narrow(unpack2(e[0]), p), narrow(unpack2(e[1]), p),
                                              narrow(unpack2(e[2]), p), narrow(unpack2(e[3]), p));
  }
}
template <typename T>
__device__ __forceinline__ void store_vec(T* p, const float* e) {
  p[0] = from_f32<T>(e[0]);
}

__device__ __forceinline__ void load_weight(const void* p, int dtype, int c, F2* e) {
  if ((uintptr_t)p % 16 == 0) {
    if (dtype == MOE_DT_F32) load_vec(reinterpret_cast<const float*>(p) + c, e);
    else if (dtype == MOE_DT_BF16) load_vec(reinterpret_cast<const __nv_bfloat16*>(p) + c, e);
    else load_vec(reinterpret_cast<const __half*>(p) + c, e);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      e[j] = pack2(load_any(p, dtype, c + 2 * j), load_any(p, dtype, c + 2 * j + 1));
  }
}
__device__ __forceinline__ void load_weight(const void* p, int dtype, int c, float* e) { e[0] = load_any(p, dtype, c); }

// The weights of VEC columns: w = gate * post (1 where absent), next.
template <int VEC, typename E>
__device__ __forceinline__ void load_weights(const NormArgs& a, int c, E* w, E* nx) {
#pragma unroll
  for (int j = 0; j < kElems<VEC>; ++j) w[j] = nx[j] = splat<E>(1.f);
  if (a.post) load_weight(a.post, a.w_dtype, c, w);
  if (a.gate_mode == MOE_GATE_CHANNEL) {
    E g[kElems<VEC>];
    load_weight(a.gate, a.w_dtype, c, g);
#pragma unroll
    for (int j = 0; j < kElems<VEC>; ++j) w[j] = mul(w[j], g[j]);
  }
  if (a.next) load_weight(a.next, a.w_dtype, c, nx);
}

// Sum of one value over the NT threads of a row, the same in all of them.  Sums
// in turn use two buffers, so that one barrier a sum is enough: a warp that
// writes a buffer again has passed the barrier after its last reads.
template <int NT, int M>
__device__ __forceinline__ float row_sum(float v, float (&buf)[2][M], int& turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (NT > 32) {
    constexpr int W = NT / 32;
    float* red = buf[turn];
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    F2 s = pack2(0.f, 0.f), r = s;
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const float4 f = reinterpret_cast<const float4*>(red)[i];
      s = add(s, pack2(f.x, f.y)), r = add(r, pack2(f.z, f.w));
    }
    v = total(add(s, r));
  }
  return v;
}

// Sums of five values.  The first four are halved on the way: at the first step
// a lane keeps two of them and hands on the other two, at the second one and
// one, so the butterfly moves 6 + 5 values instead of 20 + 5; lane l then holds
// value l / 8 of the warp.  Across warps the same.
__device__ __forceinline__ float halve4(const float (&v)[5], int lane) {
  const bool hi = lane & 16, mid = lane & 8;
  const float a = (hi ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[2], 16);
  const float b = (hi ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, hi ? v[1] : v[3], 16);
  return (mid ? b : a) + __shfl_xor_sync(0xffffffffu, mid ? a : b, 8);
}
template <int NT, int M>
__device__ __forceinline__ void row_sums5(float (&v)[5], float (&buf)[2][M], int& turn) {
  const int lane = threadIdx.x & 31;
  float q = halve4(v, lane), z = v[4];
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  if constexpr (NT > 32) {
    constexpr int W = NT / 32;   // 4, 8, 16 or 32
    float* red = buf[turn];      // [5][W]
    turn ^= 1;
    if ((lane & 7) == 0) red[(lane >> 3) * W + (threadIdx.x >> 5)] = q;
    if (lane == 1) red[4 * W + (threadIdx.x >> 5)] = z;
    __syncthreads();
    // eight lanes a value: lane l sums every eighth partial of value l / 8
    q = z = 0.f;
#pragma unroll
    for (int i = 0; i < W; i += 8) {
      const bool in = W >= 8 || (lane & 7) < W;
      if (in) q += red[(lane >> 3) * W + i + (lane & 7)], z += red[4 * W + i + (lane & 7)];
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
      q += __shfl_xor_sync(0xffffffffu, q, o);
      z += __shfl_xor_sync(0xffffffffu, z, o);
    }
  }
#pragma unroll
  for (int n = 0; n < 4; ++n) v[n] = __shfl_sync(0xffffffffu, q, n * 8);
  v[4] = z;
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(su32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int NT>
constexpr int kBlock = NT < 128 ? 128 : NT;   // threads of a block

// A thread's own slots of the ring: 16-byte pieces, [stage][piece][thread].
template <int NT, int PIECES>
struct Ring {
  uint8_t* base;
  __device__ __forceinline__ uint8_t* at(int stage, int piece) const {
    return base + ((size_t)(stage * PIECES + piece) * kBlock<NT> + threadIdx.x) * 16;
  }
};
template <typename T, typename R>
__device__ __forceinline__ void ring_copy(const R& ring, int stage, int piece, const T* src) {
#pragma unroll
  for (int i = 0; i < kPieces<T>; ++i) cp_async16(ring.at(stage, piece + i), reinterpret_cast<const uint4*>(src) + i);
}
template <typename T, typename R>
__device__ __forceinline__ void ring_load(const R& ring, int stage, int piece, F2* e) {
  uint4 q[kPieces<T>];
#pragma unroll
  for (int i = 0; i < kPieces<T>; ++i) q[i] = *reinterpret_cast<const uint4*>(ring.at(stage, piece + i));
  widen(q, (const T*)nullptr, e);
}

template <typename R>
__device__ __forceinline__ void put_slot(const R& slots, int piece, const F2* e) {
  const float2 a = unpack2(e[0]), b = unpack2(e[1]), c = unpack2(e[2]), d = unpack2(e[3]);
  *reinterpret_cast<float4*>(slots.at(0, piece)) = make_float4(a.x, a.y, b.x, b.y);
  *reinterpret_cast<float4*>(slots.at(0, piece + 1)) = make_float4(c.x, c.y, d.x, d.y);
}

// Threads an SM is to hold at once: 64 registers a thread are enough for eight
// columns of the forward, 128 for the rest.
template <int VEC, int NV, int NT, bool BWD>
constexpr int kResident = BWD || NV * VEC > 8 ? (kBlock<NT> > 512 ? kBlock<NT> : 512) : 1024;

// Rows of the ring: as many as the resident threads leave shared memory for, at
// most 4; 0: rows are loaded straight to registers (single elements, and the
// gradient's longest rows).
template <typename TX, typename TY, int VEC, int NV, int NT, bool BWD>
constexpr int ring_rows() {
  if (VEC == 1) return 0;
  const int bytes = NV * 8 * (int)(sizeof(TX) + sizeof(TY)) * (BWD ? 2 : 1), weights = BWD && NV > 1 ? NV * 64 : 0;
  const int most = (208 * 1024 / kResident<VEC, NV, NT, BWD> - weights) / bytes;
  return most < 0 ? 0 : most < 4 ? most : 4;
}

template <typename TX, typename TY, int VEC, int NV, int NT, int S>
__global__ void __launch_bounds__(kBlock<NT>, kResident<VEC, NV, NT, false> / kBlock<NT>)
    block_norm_kernel(const NormArgs a) {
  extern __shared__ uint8_t ring_smem[];
  __shared__ alignas(16) float red[2][32];
  using E = Elem<VEC>;
  constexpr int P = kElems<VEC>;
  constexpr int kRows = kBlock<NT> / NT;   // rows a block works on at once
  constexpr int kPX = kPieces<TX>, kP = kPieces<TX> + kPieces<TY>;
  const Ring<NT, NV * kP> ring{ring_smem};
  const int tid = threadIdx.x % NT, H = a.H;
  const long long step = (long long)gridDim.x * kRows;
  long long t = (long long)blockIdx.x * kRows + threadIdx.x / NT;
  pdl_wait();
  pdl_launch_dependents();
  const float inv_h = 1.f / (float)H;
  const bool has_y = a.y;
  // this thread's first column in the row to be fetched next, and in the rows written
  const int c0 = tid * VEC;
  const TX* x = reinterpret_cast<const TX*>(a.x) + t * a.ld_x + c0;
  const TY* y = reinterpret_cast<const TY*>(a.y) + (has_y ? t * a.ld_y + c0 : 0);
  TX* xo = reinterpret_cast<TX*>(a.x_out) + (a.x_out ? t * a.ld_xo + c0 : 0);
  TY* h = reinterpret_cast<TY*>(a.h) + (a.next ? t * a.ld_h + c0 : 0);
  auto advance = [&] {
    x += step * a.ld_x;
    if (has_y) y += step * a.ld_y;
  };
  auto fetch = [&](long long r, int stage) {
    if (r < a.T) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int o = i * NT * VEC;
        if (c0 + o >= H) continue;
        ring_copy<TX>(ring, stage, i * kP, x + o);
        if (has_y) ring_copy<TY>(ring, stage, i * kP + kPX, y + o);
      }
      advance();
    }
    cp_async_commit();
  };
  if constexpr (S > 0)
    for (int s = 0; s < S - 1; ++s) fetch(t + s * step, s);
  E w[NV][P], nx[NV][P];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * NT + tid) * VEC;
    if (c < H) load_weights<VEC>(a, c, w[i], nx[i]);
  }
  int stage = 0, turn = 0;
  for (; t < a.T; t += step) {
    E u[NV][P], v[NV][P];
    if constexpr (S > 0) {
      fetch(t + (S - 1) * step, (stage + S - 1) % S);
      cp_async_wait<S - 1>();
    }
    E ss = splat<E>(0.f);
    const float gt = a.gate_mode == MOE_GATE_TOKEN ? load_any(a.gate, a.w_dtype, t) : 1.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * NT + tid) * VEC;
#pragma unroll
      for (int j = 0; j < P; ++j) u[i][j] = v[i][j] = splat<E>(0.f);
      if (c >= H) continue;
      if constexpr (S > 0) {
        ring_load<TX>(ring, stage, i * kP, u[i]);
        if (has_y) ring_load<TY>(ring, stage, i * kP + kPX, v[i]);
      } else {
        load_vec(x + i * NT * VEC, u[i]);
        if (has_y) load_vec(y + i * NT * VEC, v[i]);
      }
#pragma unroll
      for (int j = 0; j < P; ++j) ss = fma(v[i][j], v[i][j], ss);
    }
    if constexpr (S > 0) stage = stage + 1 == S ? 0 : stage + 1;
    else advance();
    const float r = a.post ? gt * rsqrtf(fmaf(row_sum<NT>(total(ss), red, turn), inv_h, a.eps)) : gt;
    const E r2 = splat<E>(r), alpha = splat<E>(a.alpha);
    ss = splat<E>(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * NT + tid) * VEC;
      if (c >= H) continue;
#pragma unroll
      for (int j = 0; j < P; ++j) {
        u[i][j] = mul(u[i][j], alpha);
        if (has_y) u[i][j] = fma(mul(v[i][j], w[i][j]), r2, u[i][j]);
        ss = fma(u[i][j], u[i][j], ss);
      }
      if (a.x_out) store_vec(xo + i * NT * VEC, u[i]);
    }
    if (a.x_out) xo += step * a.ld_xo;
    if (a.next) {
      const E ru = splat<E>(rsqrtf(fmaf(row_sum<NT>(total(ss), red, turn), inv_h, a.eps)));
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * NT + tid) * VEC;
        if (c >= H) continue;
#pragma unroll
        for (int j = 0; j < P; ++j) u[i][j] = mul(mul(u[i][j], ru), nx[i][j]);
        store_vec(h + i * NT * VEC, u[i]);
      }
      h += step * a.ld_h;
    }
  }
}

// FULL: a post norm, a next norm, d_x_out given and no gate per token (a
// training step's usual call): nothing to ask for in the row loop.
template <typename TX, typename TY, int VEC, int NV, int NT, int S, bool FULL>
__global__ void __launch_bounds__(kBlock<NT>, kResident<VEC, NV, NT, true> / kBlock<NT>)
    block_norm_bwd_kernel(const NormArgs a) {
  extern __shared__ uint8_t ring_smem[];
  __shared__ alignas(16) float red[2][5 * 32];
  using E = Elem<VEC>;
  constexpr int P = kElems<VEC>;
  constexpr int kRows = kBlock<NT> / NT;
  constexpr int kPX = kPieces<TX>, kPY = kPieces<TY>, kP = 2 * kPX + 2 * kPY;
  constexpr bool kKeep = NV == 1;               // the weights stay in registers,
  constexpr bool kSlots = VEC == 8 && NV > 1;   // or as fp32 in slots of the thread's own in shared memory
  const Ring<NT, NV * kP> ring{ring_smem};
  const Ring<NT, NV * 4> slots{ring_smem + (size_t)S * NV * kP * 16 * kBlock<NT>};
  const int tid = threadIdx.x % NT, H = a.H;
  const float inv_h = 1.f / (float)H;
  const long long step = (long long)gridDim.x * kRows;
  long long t = (long long)blockIdx.x * kRows + threadIdx.x / NT;
  pdl_wait();
  pdl_launch_dependents();
  const bool has_y = FULL || a.y, has_du = FULL || a.d_xo, has_dh = FULL || a.d_h, post = FULL || a.post;
  const bool token = !FULL && a.gate_mode == MOE_GATE_TOKEN;
  // this thread's first column in the row to be fetched next, and in the rows written
  const int c0 = tid * VEC;
  const TX *x = reinterpret_cast<const TX*>(a.x) + t * a.ld_x + c0;
  const TX *du = reinterpret_cast<const TX*>(a.d_xo) + (has_du ? t * a.ld_dxo + c0 : 0);
  const TY *y = reinterpret_cast<const TY*>(a.y) + (has_y ? t * a.ld_y + c0 : 0);
  const TY *dh = reinterpret_cast<const TY*>(a.d_h) + (has_dh ? t * a.ld_dh + c0 : 0);
  TX* dx = reinterpret_cast<TX*>(a.d_x) + t * a.ld_dx + c0;
  TY* dy = reinterpret_cast<TY*>(a.d_y) + (has_y ? t * a.ld_dy + c0 : 0);
  auto advance = [&] {
    x += step * a.ld_x;
    if (has_y) y += step * a.ld_y;
    if (has_du) du += step * a.ld_dxo;
    if (has_dh) dh += step * a.ld_dh;
  };
  auto fetch = [&](long long r, int stage) {
    if (r < a.T) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int o = i * NT * VEC;
        if (c0 + o >= H) continue;
        ring_copy<TX>(ring, stage, i * kP, x + o);
        if (has_y) ring_copy<TY>(ring, stage, i * kP + kPX, y + o);
        if (has_du) ring_copy<TX>(ring, stage, i * kP + kPX + kPY, du + o);
        if (has_dh) ring_copy<TY>(ring, stage, i * kP + 2 * kPX + kPY, dh + o);
      }
      advance();
    }
    cp_async_commit();
  };
  if constexpr (S > 0)
    for (int s = 0; s < S - 1; ++s) fetch(t + s * step, s);
  E acc_e[NV][P], acc_n[NV][P], kw[NV][P], kn[NV][P];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * NT + tid) * VEC;
    if (kKeep && c < H) load_weights<VEC>(a, c, kw[i], kn[i]);
    if constexpr (kSlots) {
      if (c < H) {
        E w[P], nx[P];
        load_weights<VEC>(a, c, w, nx);
        put_slot(slots, i * 4, w);
        put_slot(slots, i * 4 + 2, nx);
      }
    }
#pragma unroll
    for (int j = 0; j < P; ++j) acc_e[i][j] = acc_n[i][j] = splat<E>(0.f);
  }
  int stage = 0, turn = 0;
  for (; t < a.T; t += step) {
    E n[NV][P], u[NV][P], d[NV][P], e[NV][P];   // n(y), u, du and then D, dh
    if constexpr (S > 0) {
      fetch(t + (S - 1) * step, (stage + S - 1) % S);
      cp_async_wait<S - 1>();
    }
    const float gt = token ? load_any(a.gate, a.w_dtype, t) : 1.f;
    E ss = splat<E>(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int o = i * NT * VEC;
#pragma unroll
      for (int j = 0; j < P; ++j) n[i][j] = u[i][j] = d[i][j] = e[i][j] = splat<E>(0.f);
      if (c0 + o >= H) continue;
      if constexpr (S > 0) {
        ring_load<TX>(ring, stage, i * kP, u[i]);
        if (has_y) ring_load<TY>(ring, stage, i * kP + kPX, n[i]);
        if (has_du) ring_load<TX>(ring, stage, i * kP + kPX + kPY, d[i]);
        if (has_dh) ring_load<TY>(ring, stage, i * kP + 2 * kPX + kPY, e[i]);
      } else {
        load_vec(x + o, u[i]);
        if (has_y) load_vec(y + o, n[i]);
        if (has_du) load_vec(du + o, d[i]);
        if (has_dh) load_vec(dh + o, e[i]);
      }
#pragma unroll
      for (int j = 0; j < P; ++j) ss = fma(n[i][j], n[i][j], ss);
    }
    if constexpr (S > 0) stage = stage + 1 == S ? 0 : stage + 1;
    else advance();
    const float ry = post ? rsqrtf(fmaf(row_sum<NT>(total(ss), red, turn), inv_h, a.eps)) : 1.f;
    E s2[5];   // of q du, u^2, a u, q a, q u
#pragma unroll
    for (int k = 0; k < 5; ++k) s2[k] = splat<E>(0.f);
    const E ry2 = splat<E>(has_y ? ry : 0.f), gt2 = splat<E>(gt), alpha = splat<E>(a.alpha);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * NT + tid) * VEC;
      if (c >= H) continue;
      E w[P], nx[P];
      if constexpr (kKeep) {
#pragma unroll
        for (int j = 0; j < P; ++j) w[j] = kw[i][j], nx[j] = kn[i][j];
      } else if constexpr (kSlots) {
        ring_load<float>(slots, 0, i * 4, w);
        ring_load<float>(slots, 0, i * 4 + 2, nx);
      } else {
        load_weights<VEC>(a, c, w, nx);
      }
#pragma unroll
      for (int j = 0; j < P; ++j) {
        n[i][j] = mul(n[i][j], ry2);
        const E q = mul(w[j], n[i][j]);
        u[i][j] = FULL ? fma(alpha, u[i][j], q) : fma(gt2, q, mul(alpha, u[i][j]));
        if (!has_dh) u[i][j] = splat<E>(0.f);   // without h nothing hangs on u
        s2[0] = fma(q, d[i][j], s2[0]);
        const E av = mul(e[i][j], nx[j]);
        s2[1] = fma(u[i][j], u[i][j], s2[1]);
        s2[2] = fma(av, u[i][j], s2[2]);
        s2[3] = fma(q, av, s2[3]);
        s2[4] = fma(q, u[i][j], s2[4]);
      }
    }
    float s[5];
#pragma unroll
    for (int k = 0; k < 5; ++k) s[k] = total(s2[k]);
    row_sums5<NT>(s, red, turn);
    const float ru = has_dh ? rsqrtf(fmaf(s[1], inv_h, a.eps)) : 0.f;
    const float m = ru * ru * s[2] * inv_h;
    const float sd = fmaf(ru, s[3] - m * s[4], s[0]);
    if (token && a.d_gate_token && tid == 0) a.d_gate_token[t] = sd;
    const E ru2 = splat<E>(ru), mm = splat<E>(-ru * m), mym = splat<E>(-ry * gt * sd * inv_h), ryo = splat<E>(ry);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * NT + tid) * VEC, o = i * NT * VEC;
      if (c >= H) continue;
      E w[P], nx[P];
      if constexpr (kKeep) {
#pragma unroll
        for (int j = 0; j < P; ++j) w[j] = kw[i][j], nx[j] = kn[i][j];
      } else if constexpr (kSlots) {
        ring_load<float>(slots, 0, i * 4, w);
        ring_load<float>(slots, 0, i * 4 + 2, nx);
      } else {
        load_weights<VEC>(a, c, w, nx);
      }
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const E er = mul(e[i][j], ru2);   // dh r_u
        d[i][j] = fma(er, nx[j], fma(u[i][j], mm, d[i][j]));
        acc_n[i][j] = fma(er, u[i][j], acc_n[i][j]);
        const E g = FULL ? d[i][j] : mul(gt2, d[i][j]);
        acc_e[i][j] = fma(g, n[i][j], acc_e[i][j]);
        const E b = mul(g, w[j]);
        n[i][j] = post ? fma(b, ryo, mul(n[i][j], mym)) : b;
        d[i][j] = mul(d[i][j], alpha);
      }
      store_vec(dx + o, d[i]);
      if (has_y) store_vec(dy + o, n[i]);
    }
    dx += step * a.ld_dx;
    if (has_y) dy += step * a.ld_dy;
  }
  if (!a.sums) return;
  // the block's column sums: one line of the workspace
  const int line = column_line(H);
  float* part = a.part + (long long)blockIdx.x * 2 * line;
  if constexpr (kRows == 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * NT + tid) * VEC;
      if (c >= H) continue;
      store_vec(part + c, acc_e[i]);
      store_vec(part + line + c, acc_n[i]);
    }
  } else {   // rows of one warp each: added in shared memory first, in row order
    __shared__ alignas(16) E sum[2][NT * NV * P];
    for (int r = 0; r < kRows; ++r) {
      if ((int)threadIdx.x / NT == r) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < P; ++j) {
            const int c = (i * NT + tid) * P + j;
            sum[0][c] = r ? add(sum[0][c], acc_e[i][j]) : acc_e[i][j];
            sum[1][c] = r ? add(sum[1][c], acc_n[i][j]) : acc_n[i][j];
          }
      }
      __syncthreads();
    }
    const float *f0 = reinterpret_cast<const float*>(sum[0]), *f1 = reinterpret_cast<const float*>(sum[1]);
    for (int c = threadIdx.x; c < H; c += kBlock<NT>) part[c] = f0[c], part[line + c] = f1[c];
  }
}

// Adds the blocks' lines in their order, 32 columns a block, eight threads a
// column of four each taking every eighth line: blockIdx.y 0: E, from which the
// post weight's and the gate's gradients, 1: the next weight's.
__global__ void __launch_bounds__(256) column_sum_kernel(const float* part, int lines, int H, const void* post,
                                                         const void* gate, int w_dtype, float* d_post, float* d_gate,
                                                         float* d_next) {
  __shared__ float4 sum[32][8];
  pdl_wait();
  pdl_launch_dependents();
  const int line = column_line(H), slice = threadIdx.x / 8, c = (blockIdx.x * 8 + threadIdx.x % 8) * 4;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < H) {
#pragma unroll 4
    for (int i = slice; i < lines; i += 32) {
      const float4 f = *reinterpret_cast<const float4*>(part + ((long long)i * 2 + blockIdx.y) * line + c);
      s.x += f.x, s.y += f.y, s.z += f.z, s.w += f.w;
    }
  }
  sum[slice][threadIdx.x % 8] = s;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  const int cc = blockIdx.x * 32 + threadIdx.x;
  if (cc >= H) return;
  float v = 0.f;
  for (int i = 0; i < 32; ++i) v += reinterpret_cast<const float*>(&sum[i][threadIdx.x / 4])[threadIdx.x % 4];
  if (blockIdx.y == 1) {
    if (d_next) d_next[cc] = v;
    return;
  }
  if (d_post) d_post[cc] = gate ? v * load_any(gate, w_dtype, cc) : v;
  if (d_gate) d_gate[cc] = post ? v * load_any(post, w_dtype, cc) : v;
}

// Blocks of the gradient kernel, which the workspace has a line for each: what
// fits the SMs at 512 threads each.
static int bwd_blocks(long long T, int rows, int threads) {
  const long long need = (T + rows - 1) / rows, most = (long long)device_sms() * (threads >= 512 ? 1 : 512 / threads);
  return (int)(need < most ? need : most);
}

template <bool BWD, typename TX, typename TY, int VEC, int NV, int NT>
static moe_status launch_norm(const NormArgs& a, int* lines, cudaStream_t s) {
  constexpr int kRows = kBlock<NT> / NT, S = ring_rows<TX, TY, VEC, NV, NT, BWD>();
  if constexpr (!BWD) {
    const long long need = ((long long)a.T + kRows - 1) / kRows, most = (long long)device_sms() * (kResident<VEC, NV, NT, false> / kBlock<NT>);
    constexpr size_t smem = (size_t)S * NV * 8 * (sizeof(TX) + sizeof(TY)) * kBlock<NT>;
    auto kernel = block_norm_kernel<TX, TY, VEC, NV, NT, S>;
    static char allowed[64];
    MOE_CUDA(allow_smem(kernel, smem, allowed));
    ProfScope ps(MOE_K_NORM, s);
    cudaError_t e = launch_pdl(kernel, dim3((unsigned)(need < most ? need : most)), dim3(kBlock<NT>), smem, s, a);
    if (e != cudaSuccess) return cuda_fail(e, "block_norm_kernel");
    return check_launch("block_norm_kernel");
  } else {
    constexpr size_t smem = ((size_t)S * NV * 16 * (sizeof(TX) + sizeof(TY)) + (VEC == 8 && NV > 1 ? NV * 64 : 0)) * kBlock<NT>;
    const bool full = VEC == 8 && a.post && a.d_h && a.d_xo && a.gate_mode != MOE_GATE_TOKEN;
    auto kernel = full ? block_norm_bwd_kernel<TX, TY, VEC, NV, NT, S, VEC == 8>
                       : block_norm_bwd_kernel<TX, TY, VEC, NV, NT, S, false>;
    static char allowed[2][64];
    MOE_CUDA(allow_smem(kernel, smem, allowed[full]));
    *lines = bwd_blocks(a.T, kRows, kBlock<NT>);
    cudaError_t e = launch_pdl(kernel, dim3(*lines), dim3(kBlock<NT>), smem, s, a);
    if (e != cudaSuccess) return cuda_fail(e, "block_norm_bwd_kernel");
    return check_launch("block_norm_bwd_kernel");
  }
}

// The shape a row is held in.  Rows of up to 512 columns (the gradient: 256) take
// one warp, with no barriers at all; longer ones the fewest threads that hold 8
// columns each.  The gradient of 16-bit rows takes 16 a thread from 1025 columns
// on: half the warps to add up, and two blocks an SM whose sums wait in turn (at
// T = 8192, H = 4096: 81.8 us with 8 columns a thread, 74.6 with 16).  Rows of fp32 leave no room for that ring; past 4096
// columns they take 16 as well, past 1024 threads the forward does.  Where rows
// cannot be read in 16-byte vectors: single elements, 4 to 16 a thread.
template <bool BWD, typename TX, typename TY>
static moe_status norm_by_shape(const NormArgs& a, bool vec, int* lines, cudaStream_t s) {
  const int H = a.H;
  constexpr bool kNarrow = sizeof(TX) + sizeof(TY) == 4;
  if (!vec) {
    if (H <= 512) return launch_norm<BWD, TX, TY, 1, 4, 128>(a, lines, s);
    if (H <= 2048) return launch_norm<BWD, TX, TY, 1, 8, 256>(a, lines, s);
    if (H <= 8192) return launch_norm<BWD, TX, TY, 1, 16, 512>(a, lines, s);
    return launch_norm<BWD, TX, TY, 1, 16, 1024>(a, lines, s);
  }
  if (H <= 256) return launch_norm<BWD, TX, TY, 8, 1, 32>(a, lines, s);
  if constexpr (!BWD)
    if (H <= 512) return launch_norm<BWD, TX, TY, 8, 2, 32>(a, lines, s);
  if (H <= 1024) return launch_norm<BWD, TX, TY, 8, 1, 128>(a, lines, s);
  if constexpr (BWD && kNarrow) {
    if (H <= 2048) return launch_norm<BWD, TX, TY, 8, 2, 128>(a, lines, s);
    if (H <= 4096) return launch_norm<BWD, TX, TY, 8, 2, 256>(a, lines, s);
  } else {
    if (H <= 2048) return launch_norm<BWD, TX, TY, 8, 1, 256>(a, lines, s);
    if (H <= 4096) return launch_norm<BWD, TX, TY, 8, 1, 512>(a, lines, s);
  }
  if constexpr (BWD) {
    if (H <= 8192) return launch_norm<BWD, TX, TY, 8, 2, 512>(a, lines, s);
  } else {
    if (H <= 8192) return launch_norm<BWD, TX, TY, 8, 1, 1024>(a, lines, s);
  }
  return launch_norm<BWD, TX, TY, 8, 2, 1024>(a, lines, s);
}

template <bool BWD>
static moe_status norm_by_type(const NormArgs& a, int xd, int yd, bool vec, int* lines, cudaStream_t s) {
  if (xd == MOE_DT_BF16) return norm_by_shape<BWD, __nv_bfloat16, __nv_bfloat16>(a, vec, lines, s);
  if (xd == MOE_DT_F16) return norm_by_shape<BWD, __half, __half>(a, vec, lines, s);
  if (yd == MOE_DT_BF16) return norm_by_shape<BWD, float, __nv_bfloat16>(a, vec, lines, s);
  if (yd == MOE_DT_F16) return norm_by_shape<BWD, float, __half>(a, vec, lines, s);
  return norm_by_shape<BWD, float, float>(a, vec, lines, s);
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
  return norm_by_type<false>(a, x_dtype, y_dtype, vec, nullptr, stream);
}

extern "C" size_t moe_block_norm_backward_workspace(int T, int H) {
  if (T <= 0 || H <= 0 || H > 16384) return 0;
  // one line of two sums a block; the narrowest blocks that norm_by_shape may take are the most
  return (size_t)bwd_blocks(T, 1, H <= 2048 ? 128 : H <= 4096 ? 256 : 512) * 2 * column_line(H) * sizeof(float);
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
  a.sums = sums;
  const bool vec = H % 8 == 0 && vec_ok(x, ld_x, x_dtype) && vec_ok(y, ld_y, y_dtype) &&
                   vec_ok(d_x_out, ld_d_x_out, x_dtype) && vec_ok(d_h, ld_d_h, y_dtype) &&
                   vec_ok(d_x, ld_d_x, x_dtype) && vec_ok(d_y, ld_d_y, y_dtype);
  int lines = 0;
  ProfScope ps(MOE_K_NORM_BWD, stream);
  st = norm_by_type<true>(a, x_dtype, y_dtype, vec, &lines, stream);
  if (st != MOE_OK || !sums) return st;
  const bool channel = gate_mode == MOE_GATE_CHANNEL;
  cudaError_t e = launch_pdl(column_sum_kernel, dim3((H + 31) / 32, next_weight ? 2 : 1), dim3(256), 0, stream,
                             (const float*)a.part, lines, H, post_weight, channel ? gate : nullptr, w_dtype,
                             d_post_weight, channel ? d_gate : nullptr, d_next_weight);
  if (e != cudaSuccess) return cuda_fail(e, "column_sum_kernel");
  return check_launch("column_sum_kernel");
}
