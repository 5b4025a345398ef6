// Products with 4-bit weights that share a scale (and a zero point) in groups of a row:
//   out[r, n] = sum_k x[r, k] (q[e, n, k] - z[e, n, k / g]) s[e, n, k / g],
// e the expert that row r belongs to (rows sorted by expert), or one matrix for all rows.
//
// q - z is a whole number that bf16 and f16 hold exactly, so the tensor cores' products
// are exact; a group's sum is taken in fp32 and multiplied by its scale in fp32. No
// weight is rounded: a scaled weight in 16 bits would add to the result's rounding about
// half as much again.
#include <math.h>

#include <type_traits>

#include "dtype.cuh"

namespace moe {

struct W4Args {
  int P, N, K, E, g, out_dtype;       // N: rows of a matrix (with swiglu gates, then ups)
  const void* x;
  long long ld_x, ld_out;             // elements
  const uint8_t *codes, *zeros;       // [E][N][K / 2]; [E][N][K / g] or null (8)
  const void* scales;                 // [E][N][K / g] of x's type
  const int32_t* offsets;             // [E + 1] or null (all P rows are expert 0's)
  void* out;
};

template <typename TE>
struct W4;
template <>
struct W4<__nv_bfloat16> {
  static constexpr uint32_t kMagic = 0x43004300u;   // 128: a nibble in its low bits is 128 + q
  static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  static __device__ __forceinline__ float scale(uint32_t packed) { return __uint_as_float(packed << 16); }
};
template <>
struct W4<__half> {
  static constexpr uint32_t kMagic = 0x64006400u;   // 1024
  static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
    const __half2 r = __hsub2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  static __device__ __forceinline__ float scale(uint32_t packed) {
    return __half2float(__ushort_as_half((unsigned short)packed));
  }
};

// Eight codes of a word less the zero point (`zero`: kMagic + z in both halves), as the
// pairs (0, 4), (1, 5), (2, 6), (3, 7): a nibble ORed into the mantissa of 128 (bf16) or
// 1024 (f16) is that number plus the code.
template <typename TE>
__device__ __forceinline__ void unpack(uint32_t w, uint32_t zero, uint32_t (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = W4<TE>::sub(((w >> (4 * i)) & 0x000f000fu) | W4<TE>::kMagic, zero);
}

template <typename TE>
__device__ __forceinline__ void w4_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  if constexpr (std::is_same<TE, __nv_bfloat16>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float silu_times(float gate, float up) { return gate / (1.f + expf(-gate)) * up; }

// WPL words of codes of one row's group for a lane: c * WPL words into the group.
template <int WPL>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[WPL]) {
  if constexpr (WPL == 4) {
    const uint4 v = ld_stream_v4(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (WPL == 2) {
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
  } else {
    asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(w[0]) : "l"(p));
  }
}

// Few rows of x to a matrix.  A warp multiplies 16 rows of weights by up to 8 rows of x
// (m16n8k16): lane (g, c) holds codes of rows g and g + 8, WPL words (8 WPL neighbouring
// codes) of each group, loaded straight from memory four groups ahead; which k a lane's
// codes are does not matter as long as x's fragment holds the same ones.  x lies in
// shared memory in the fragments' order.  The block's warps split the rows and, KS ways,
// the groups; the KS sums are added in order at the end.
constexpr int kChunkBytes = 64 * 1024;   // of x at a time

template <typename TE, int WPL, int KS>
__global__ void __launch_bounds__(256) w4_rows_kernel(const W4Args a, int swiglu) {
  extern __shared__ __align__(16) uint8_t w4_smem[];
  constexpr int kRowWarps = 8 / KS, kGroup = 32 * WPL;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int rw = warp % kRowWarps, ks = warp / kRowWarps;
  pdl_wait();
  pdl_launch_dependents();
  // the expert: with fewer rows than experts the y-th that has any
  int e = blockIdx.y, m0 = 0, m1 = a.P;
  if (a.offsets) {
    if (a.P < a.E) {
      __shared__ int found;
      __shared__ int ws[34];
      if (tid == 0) found = -1;
      int before = 0;
      __syncthreads();
      for (int b = 0; b < a.E; b += 256) {
        const int i = b + tid;
        const int any = i < a.E && a.offsets[i + 1] > a.offsets[i];
        int all;
        const int at = block_exclusive_scan(any, ws, &all);
        if (any && before + at == (int)blockIdx.y) found = i;
        before += all;
      }
      __syncthreads();
      e = found;
      if (e < 0) return;
    }
    m0 = max(a.offsets[e], 0), m1 = min(a.offsets[e + 1], a.P);
  }
  if (m0 >= m1) return;
  const int half = swiglu ? a.N / 2 : 8, outs = swiglu ? a.N / 2 : a.N;   // distance of a lane's two rows
  const int o0 = (blockIdx.x * kRowWarps + rw) * (swiglu ? 8 : 16);       // the warp's first output
  const int groups = a.K / kGroup, chunk = kChunkBytes / (kGroup * 16) & ~3;   // groups of x at a time
  const int r0 = min(o0 + g, a.N - 1), r1 = min(o0 + g + half, a.N - 1);
  const long long row0 = (long long)e * a.N + r0, row1 = (long long)e * a.N + r1;
  const uint8_t* w0 = a.codes + row0 * (a.K / 2) + c * (WPL * 4);
  const uint8_t* w1 = a.codes + row1 * (a.K / 2) + c * (WPL * 4);
  const unsigned short* s0 = reinterpret_cast<const unsigned short*>(a.scales) + row0 * groups;
  const unsigned short* s1 = reinterpret_cast<const unsigned short*>(a.scales) + row1 * groups;
  const uint8_t* z0 = a.zeros ? a.zeros + row0 * groups : nullptr;
  const uint8_t* z1 = a.zeros ? a.zeros + row1 * groups : nullptr;
  float* sums = reinterpret_cast<float*>(w4_smem);   // [KS - 1][rows warps][32][4], after the last chunk

  for (int t0 = m0; t0 < m1; t0 += 8) {
    const int m = min(8, m1 - t0);
    float acc[4] = {};
    for (int gb = 0; gb < groups; gb += chunk) {
      const int ge = min(groups, gb + chunk);
      // x's fragments: [group][word][lane] of 16 bytes, lane 4 i + c for row i of x
      __syncthreads();
      const int pieces = (ge - gb) * 4 * WPL;   // of 8 values
      for (int i = tid; i < pieces * m; i += 256) {
        const int t = i / pieces, q = i - t * pieces, in = q % (4 * WPL);
        const uint4 v = *reinterpret_cast<const uint4*>(reinterpret_cast<const TE*>(a.x) + (t0 + t) * a.ld_x +
                                                        (long long)gb * kGroup + q * 8);
        uint4 f;   // (0, 4), (1, 5), (2, 6), (3, 7)
        f.x = __byte_perm(v.x, v.z, 0x5410), f.y = __byte_perm(v.x, v.z, 0x7632);
        f.z = __byte_perm(v.y, v.w, 0x5410), f.w = __byte_perm(v.y, v.w, 0x7632);
        *reinterpret_cast<uint4*>(w4_smem + ((q / (4 * WPL) * WPL + in % WPL) * 32 + t * 4 + in / WPL) * 16) = f;
      }
      __syncthreads();
      const int n = ge - gb, i0 = gb + n * ks / KS, i1 = gb + n * (ks + 1) / KS;   // this warp's groups
      uint32_t q0[4][WPL], q1[4][WPL];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i0 + j < i1) {
          load_words<WPL>(w0 + (long long)(i0 + j) * (kGroup / 2), q0[j]);
          load_words<WPL>(w1 + (long long)(i0 + j) * (kGroup / 2), q1[j]);
        }
      for (int i = i0; i < i1; i += 4) {
        // scales and zero points of four groups, one to a lane c
        uint32_t p0 = 0, p1 = 0;
        if (i + c < i1) {
          p0 = s0[i + c] | (z0 ? (uint32_t)z0[i + c] : 8u) << 16;
          p1 = s1[i + c] | (z1 ? (uint32_t)z1[i + c] : 8u) << 16;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (i + j >= i1) break;
          const uint32_t b0 = __shfl_sync(0xffffffffu, p0, (lane & ~3) | j), b1 = __shfl_sync(0xffffffffu, p1, (lane & ~3) | j);
          const uint32_t k0 = W4<TE>::kMagic + (b0 >> 16) * 0x00010001u, k1 = W4<TE>::kMagic + (b1 >> 16) * 0x00010001u;
          float d[4] = {};
#pragma unroll
          for (int w = 0; w < WPL; ++w) {
            uint32_t u[4], v[4];
            unpack<TE>(q0[j][w], k0, u);
            unpack<TE>(q1[j][w], k1, v);
            const uint4 f = *reinterpret_cast<const uint4*>(w4_smem + (((i + j - gb) * WPL + w) * 32 + lane) * 16);
            w4_mma<TE>(d, u[0], v[0], u[1], v[1], f.x, f.y);
            w4_mma<TE>(d, u[2], v[2], u[3], v[3], f.z, f.w);
          }
          const float f0 = W4<TE>::scale(b0 & 0xffff), f1 = W4<TE>::scale(b1 & 0xffff);
          acc[0] = fmaf(f0, d[0], acc[0]), acc[1] = fmaf(f0, d[1], acc[1]);
          acc[2] = fmaf(f1, d[2], acc[2]), acc[3] = fmaf(f1, d[3], acc[3]);
          if (i + j + 4 < i1) {
            load_words<WPL>(w0 + (long long)(i + j + 4) * (kGroup / 2), q0[j]);
            load_words<WPL>(w1 + (long long)(i + j + 4) * (kGroup / 2), q1[j]);
          }
        }
      }
    }
    if (KS > 1) {
      __syncthreads();
      if (ks) *reinterpret_cast<float4*>(sums + ((ks - 1) * kRowWarps + rw) * 128 + lane * 4) = make_float4(acc[0], acc[1], acc[2], acc[3]);
      __syncthreads();
      if (ks == 0)
        for (int j = 1; j < KS; ++j) {
          const float4 o = *reinterpret_cast<const float4*>(sums + ((j - 1) * kRowWarps + rw) * 128 + lane * 4);
          acc[0] += o.x, acc[1] += o.y, acc[2] += o.z, acc[3] += o.w;
        }
    }
    if (KS == 1 || ks == 0) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (2 * c + i >= m) continue;
        const long long o = (t0 + 2 * c + i) * a.ld_out + o0 + g;
        auto put = [&](long long at, float v) {
          if (a.out_dtype == MOE_DT_F32) reinterpret_cast<float*>(a.out)[at] = v;
          else reinterpret_cast<TE*>(a.out)[at] = from_f32<TE>(v);
        };
        if (swiglu) {
          if (o0 + g < outs) put(o, silu_times(acc[i], acc[i + 2]));
        } else {
          if (o0 + g < outs) put(o, acc[i]);
          if (o0 + g + 8 < outs) put(o + 8, acc[i + 2]);
        }
      }
    }
  }
}

// --------------------------------------------------------------------- host --

template <typename TE, int WPL, int KS>
static moe_status launch_rows_kernel(const W4Args& a, int swiglu, cudaStream_t s) {
  auto kernel = w4_rows_kernel<TE, WPL, KS>;
  static char allowed[64];
  MOE_CUDA(allow_smem(kernel, kChunkBytes, allowed));
  const int outs = swiglu ? a.N / 2 : a.N, per = 8 / KS * (swiglu ? 8 : 16), tiles = (outs + per - 1) / per;
  const int experts = a.offsets && a.P < a.E ? a.P : a.E;
  const long long x = (long long)a.K * 16;   // 8 rows
  const size_t smem = x < 4096 ? 4096 : x < kChunkBytes ? (size_t)x : kChunkBytes;
  cudaError_t e = launch_pdl(kernel, dim3(tiles, experts), dim3(256), smem, s, a, swiglu);
  if (e != cudaSuccess) return cuda_fail(e, "w4_rows_kernel");
  return check_launch("w4_rows_kernel");
}
template <typename TE, int WPL>
static moe_status launch_split_rows(const W4Args& a, int swiglu, cudaStream_t s) {
  // few tiles: the groups are split over a block's warps, so that more blocks share the rows
  const long long tiles = ((long long)a.N + 127) / 128 * (a.offsets && a.P < a.E ? a.P : a.E);
  if (tiles * 2 >= device_sms() * 3) return launch_rows_kernel<TE, WPL, 1>(a, swiglu, s);
  return launch_rows_kernel<TE, WPL, 8>(a, swiglu, s);
}
template <typename TE>
static moe_status launch_w4(const W4Args& a, int swiglu, cudaStream_t s) {
  ProfScope ps(MOE_K_W4, s);
  if (a.g == 128) return launch_split_rows<TE, 4>(a, swiglu, s);
  if (a.g == 64) return launch_split_rows<TE, 2>(a, swiglu, s);
  return launch_split_rows<TE, 1>(a, swiglu, s);
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_w4_linear(int P, int N, int K, int E, int group, int dtype, int out_dtype, const void* x,
                                    int64_t ld_x, const uint8_t* codes, const void* scales, const uint8_t* zeros,
                                    const int32_t* offsets, int swiglu, void* out, int64_t ld_out, int32_t* d_error,
                                    cudaStream_t stream) {
  clear_error();
  MOE_ARG(P >= 0 && P <= 1 << 30, "rows must be in [0, 2^30] (got %d)", P);
  MOE_ARG(N >= 1 && N <= 1 << 24, "N must be in [1, 2^24] (got %d)", N);
  MOE_ARG(group == 32 || group == 64 || group == 128, "the group must be 32, 64 or 128 (got %d)", group);
  MOE_ARG(K >= group && K <= 1 << 24 && K % group == 0, "K must be a multiple of the group, at most 2^24 (got %d)", K);
  MOE_ARG(E >= 1 && E <= 65535, "E must be in [1, 65535] (got %d)", E);
  MOE_ARG((long long)E * N <= 0x7fffff00LL, "E * N must be below 2^31");
  MOE_ARG(dtype == MOE_DT_BF16 || dtype == MOE_DT_F16, "x must be bf16 or f16 (type %d)", dtype);
  MOE_ARG(out_dtype == dtype || out_dtype == MOE_DT_F32, "out must be of x's type or fp32 (type %d)", out_dtype);
  MOE_ARG(!swiglu || N % 2 == 0, "swiglu needs an even N (got %d)", N);
  MOE_ARG(offsets || E == 1, "E > 1 needs offsets");
  if (P == 0) return MOE_OK;
  MOE_ARG(x && codes && scales && out, "null pointer");
  MOE_ARG(ld_x >= K && ld_out >= (swiglu ? N / 2 : N), "a row distance is below the row's length");
  MOE_ARG((uintptr_t)x % 16 == 0 && ld_x % 8 == 0, "x needs rows on 16-byte boundaries");
  MOE_ARG((uintptr_t)codes % 16 == 0 && (uintptr_t)scales % 2 == 0, "codes must be 16-byte aligned");
  W4Args a = {P, N, K, E, group, out_dtype, x, ld_x, ld_out, codes, zeros, scales, offsets, out};
  return dtype == MOE_DT_BF16 ? launch_w4<__nv_bfloat16>(a, swiglu ? 1 : 0, stream)
                              : launch_w4<__half>(a, swiglu ? 1 : 0, stream);
}
