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
#include "four_of_row.h"
#include "tcgen05_issue.cuh"
#include "w4_tile.h"

namespace moe {

struct W4Args {
  int P, N, K, E, g, out_dtype;       // N: rows of a matrix (with swiglu gates, then ups)
  const void* x;
  long long ld_x, ld_out;             // elements
  const uint8_t *codes, *zeros;       // [E][N][K / 2]; [E][N][K / g] or null (8)
  const void* scales;                 // [E][N][K / g] of x's type
  const void *scales_end, *zeros_end;
  const int32_t* offsets;             // [E + 1] or null (all P rows are expert 0's)
  void* out;
  int32_t* err;
  int few;                            // experts of up to so many rows are w4_rows_kernel's, those of more w4_tile_kernel's
};

// A 16-bit float whose high bits are 0 is its low bits times the type's smallest number (2^-133 in
// bf16, 2^-24 in f16; with the lowest bit of the exponent among them too).  So a code, in the
// low four bits or the next four, is a number already, and one fused multiply-add brings it to
// (q - z) kUnit, exactly: no conversion, no bits of an exponent to put in.  1 / kUnit goes
// into the sums at the end.
template <typename TE>
struct W4;
template <>
struct W4<__nv_bfloat16> {
  static constexpr float kUp = 64.f;                                       // 1 / kUnit
  static constexpr uint32_t kLow = 0x7f007f00u, kHigh = 0x7d007d00u;       // 2^127, 2^123: codes in bits 0 to 3, 4 to 7
  static constexpr uint32_t kBoth = 0x7d007f00u;                           // one of each
  static __device__ __forceinline__ uint32_t fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
  }
  static __device__ __forceinline__ uint32_t offset(uint32_t z) {          // -z kUnit, twice
    const uint32_t h = __float_as_uint((float)z * (-1.f / kUp));           // 8 bits: exact
    return __byte_perm(h, h, 0x3232);
  }
  static __device__ __forceinline__ float scale(uint32_t packed) { return __uint_as_float(packed << 16); }
};
template <>
struct W4<__half> {
  static constexpr float kUp = 512.f;
  static constexpr uint32_t kLow = 0x78007800u, kHigh = 0x68006800u;       // 2^15, 2^11
  static constexpr uint32_t kBoth = 0x68007800u;
  static __device__ __forceinline__ uint32_t fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
  }
  static __device__ __forceinline__ uint32_t offset(uint32_t z) {
    const __half2 h = __float2half2_rn((float)z * (-1.f / kUp));
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float scale(uint32_t packed) {
    return __half2float(__ushort_as_half((unsigned short)packed));
  }
};

// Eight codes of a word less the zero point, times kUnit, as the pairs (0, 4), (1, 5), (2, 6), (3, 7).
template <typename TE>
__device__ __forceinline__ void unpack(uint32_t w, uint32_t offset, uint32_t (&v)[4]) {
  const uint32_t up = w >> 8;
  v[0] = W4<TE>::fma(w & 0x000f000fu, W4<TE>::kLow, offset);
  v[1] = W4<TE>::fma(w & 0x00f000f0u, W4<TE>::kHigh, offset);
  v[2] = W4<TE>::fma(up & 0x000f000fu, W4<TE>::kLow, offset);
  v[3] = W4<TE>::fma(up & 0x00f000f0u, W4<TE>::kHigh, offset);
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

// 16 bytes into another block's shared memory
__device__ __forceinline__ void st_cluster4(uint32_t to, const float (&v)[4]) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(to), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]) : "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t from) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(from) : "memory");
  return v;
}
__device__ __forceinline__ float silu_times(float gate, float up) { return gate / (1.f + expf(-gate)) * up; }

// 16 bytes of weights, read once a launch; 0 where there are none
__device__ __forceinline__ uint4 load_codes(bool in, const uint8_t* p) {
  uint4 w;
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\tmov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\t"
      "mov.u32 %3, 0;\n\t@q ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
      : "=&r"(w.x), "=&r"(w.y), "=&r"(w.z), "=&r"(w.w)
      : "l"(p), "r"((uint32_t)in));
  return w;
}

// 128 codes of a row lie in four lanes, 16 bytes to each as they were loaded, WPL words of every group wanted:
// lanes exchange words so that lane c holds WPL words of each group of 32 WPL, group by group.
template <int WPL>
__device__ __forceinline__ void deal_words(uint4 q, int c, uint32_t (&w)[4]) {
  w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
  if (WPL <= 2) {   // halves: lanes 0 and 1 hold the first 64 codes, 2 and 3 the others
    const bool up = c & 2;
    const uint32_t a = __shfl_xor_sync(0xffffffffu, up ? w[0] : w[2], 2), b = __shfl_xor_sync(0xffffffffu, up ? w[1] : w[3], 2);
    if (up) w[0] = a, w[1] = b;
    else w[2] = a, w[3] = b;
  }
  if (WPL == 1) {   // quarters
    const bool up = c & 1;
    const uint32_t a = __shfl_xor_sync(0xffffffffu, up ? w[0] : w[1], 1), b = __shfl_xor_sync(0xffffffffu, up ? w[2] : w[3], 1);
    if (up) w[0] = a, w[2] = b;
    else w[1] = a, w[3] = b;
  }
}
// Where x's values of word `in` of a step's 16 go: (word of the lane) * 32 + the lane's c.
template <int WPL>
__device__ __forceinline__ int word_place(int in) {
  if (WPL == 4) return (in & 3) * 32 + (in >> 2);
  if (WPL == 1) return (in >> 2) * 32 + (in & 3);
  const int lane = in >> 2 & 1, half = in >> 1 & 1;   // of the group's eight words: lanes 0, 2, 1, 3 hold two each
  return ((in >> 3) * 2 + (in & 1)) * 32 + lane + 2 * half;
}

// Few rows of x to a matrix.  A warp multiplies 16 rows of weights by up to 8 rows of x
// (m16n8k16), 128 products a step: lane (g, c) loads 16 bytes of codes of rows g and g + 8
// straight from memory, D steps ahead (four in groups of 128, two in smaller ones); which k a lane's codes
// are does not matter as long as x's fragment holds the same ones.  x lies in shared memory in the fragments'
// order.  Where the rows of weights alone would not fill the GPU, KS of the block's warps
// or a cluster of `splits` blocks share the steps, and the sums are added in order.
//
// Bound by HBM where there are codes enough: 512 rows of 256 experts, 4096 x 4096 (gates and
// ups) 369 us with the launch of tiles behind it, 5.3 TB/s; one row of 4096 x 4096 4.7 us with the codes in the L2 and 7 to 9
// from HBM, latency: x, the codes and a sum over the warps after each other.  Groups of 32
// take twice the instructions of groups of 128 (scales, zero points and sums for each): the
// same experts 618 us, 3.6 TB/s.  Scales come D steps ahead as the codes do; 80
// registers keep three blocks on an SM, more of them under way cost the third (556 us).
constexpr int kChunk = 32, kChunkBytes = kChunk * 2048;   // steps of x at a time
constexpr int kMaxSplits = 8;

template <typename TE, int WPL, int KS>
__global__ void __launch_bounds__(256, KS == 8 ? 2 : 3) w4_rows_kernel(const W4Args a, int swiglu, int lg, int x_bytes) {
  extern __shared__ __align__(16) uint8_t w4_smem[];
  constexpr int GP = 4 / WPL, kRowWarps = 8 / KS;   // groups of a step
  constexpr int D = WPL == 4 ? 4 : 2, NB = D * GP / 4;   // steps under way, scales of a lane for them
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int rw = warp % kRowWarps, ks = warp / kRowWarps;
  const int splits = 1 << lg, split = (int)blockIdx.x & (splits - 1), tile = (int)blockIdx.x >> lg;
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
  if (m0 >= m1 || m1 - m0 > a.few) return;   // all blocks of a cluster
  if (splits > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int half = swiglu ? a.N / 2 : 8, outs = swiglu ? a.N / 2 : a.N;   // distance of a lane's two rows
  const int o0 = (tile * kRowWarps + rw) * (swiglu ? 8 : 16);             // the warp's first output
  const int groups = a.K / (32 * WPL), all_steps = (a.K + 127) / 128;
  const int sb = all_steps * split >> lg, se = all_steps * (split + 1) >> lg;
  const int r0 = min(o0 + g, a.N - 1), r1 = min(o0 + g + half, a.N - 1);
  const long long row0 = (long long)e * a.N + r0, row1 = (long long)e * a.N + r1;
  const uint8_t* w0 = a.codes + row0 * (a.K / 2) + c * 16;
  const uint8_t* w1 = a.codes + row1 * (a.K / 2) + c * 16;
  const long long g0 = row0 * groups + c, g1 = row1 * groups + c;
  float* sums = reinterpret_cast<float*>(w4_smem + x_bytes);   // [splits * KS - 1][kRowWarps][32][4]

  for (int t0 = m0; t0 < m1; t0 += 8) {
    const int m = min(8, m1 - t0);
    float acc[4] = {};
    for (int cb = sb; cb < se; cb += kChunk) {
      const int ce = min(se, cb + kChunk), ib = cb + (ce - cb) * ks / KS, ie = cb + (ce - cb) * (ks + 1) / KS;   // this warp's
      uint4 q0[D], q1[D];
      auto codes = [&](int i, int j) {   // 0 past the row's end, where x is 0 too
        if constexpr (WPL == 4) {
          q0[j] = ld_stream_v4(w0 + (long long)i * 64);
          q1[j] = ld_stream_v4(w1 + (long long)i * 64);
        } else {
          const bool in = i * 128 + c * 32 < a.K;
          q0[j] = load_codes(in, w0 + (long long)i * 64);
          q1[j] = load_codes(in, w1 + (long long)i * 64);
        }
      };
      // scales and zero points of D steps' groups, every fourth one to a lane c, loaded D steps ahead
      uint32_t p0[NB], p1[NB], n0[NB], n1[NB];
      auto scales = [&](int i) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const int at = i * GP + 4 * b;
          n0[b] = n1[b] = 0;
          if (at + c < groups && i < ie) {
            const unsigned short* s = reinterpret_cast<const unsigned short*>(a.scales) + at;
            n0[b] = s[g0] | (a.zeros ? (uint32_t)a.zeros[g0 + at] : 8u) << 16;
            n1[b] = s[g1] | (a.zeros ? (uint32_t)a.zeros[g1 + at] : 8u) << 16;
          }
        }
      };
      // x's fragments: [step][word of a lane][lane] of 16 bytes, lane 4 i + c for row i of x
      __syncthreads();
      const int pieces = (ce - cb) * 16;   // of 8 values
      for (int i = tid; i < pieces * m; i += 256) {
        const int t = i / pieces, q = i - t * pieces;
        const long long k = (long long)cb * 128 + q * 8;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (k < a.K) v = *reinterpret_cast<const uint4*>(reinterpret_cast<const TE*>(a.x) + (t0 + t) * a.ld_x + k);
        uint4 f;   // (0, 4), (1, 5), (2, 6), (3, 7)
        f.x = __byte_perm(v.x, v.z, 0x5410), f.y = __byte_perm(v.x, v.z, 0x7632);
        f.z = __byte_perm(v.y, v.w, 0x5410), f.w = __byte_perm(v.y, v.w, 0x7632);
        *reinterpret_cast<uint4*>(w4_smem + ((q >> 4) * 128 + word_place<WPL>(q & 15) + t * 4) * 16) = f;
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < D; ++j)
        if (ib + j < ie) codes(ib + j, j);
      scales(ib);
      for (int i = ib; i < ie; i += D) {
#pragma unroll
        for (int b = 0; b < NB; ++b) p0[b] = n0[b], p1[b] = n1[b];
        scales(i + D);
#pragma unroll
        for (int j = 0; j < D; ++j) {
          if (i + j >= ie) break;
          uint32_t c0[4], c1[4];
          deal_words<WPL>(q0[j], c, c0);
          deal_words<WPL>(q1[j], c, c1);
#pragma unroll
          for (int h = 0; h < GP; ++h) {
            const int from = (lane & ~3) | ((j * GP + h) & 3);
            const uint32_t b0 = __shfl_sync(0xffffffffu, p0[(j * GP + h) / 4], from);
            const uint32_t b1 = __shfl_sync(0xffffffffu, p1[(j * GP + h) / 4], from);
            const uint32_t k0 = W4<TE>::offset(b0 >> 16), k1 = W4<TE>::offset(b1 >> 16);
            float d[4] = {};
#pragma unroll
            for (int w = h * WPL; w < (h + 1) * WPL; ++w) {
              uint32_t u[4], v[4];
              unpack<TE>(c0[w], k0, u);
              unpack<TE>(c1[w], k1, v);
              const uint4 f = *reinterpret_cast<const uint4*>(w4_smem + (((i + j - cb) * 4 + w) * 32 + lane) * 16);
              w4_mma<TE>(d, u[0], v[0], u[1], v[1], f.x, f.y);
              w4_mma<TE>(d, u[2], v[2], u[3], v[3], f.z, f.w);
            }
            const float f0 = W4<TE>::scale(b0 & 0xffff), f1 = W4<TE>::scale(b1 & 0xffff);
            acc[0] = fmaf(f0, d[0], acc[0]), acc[1] = fmaf(f0, d[1], acc[1]);
            acc[2] = fmaf(f1, d[2], acc[2]), acc[3] = fmaf(f1, d[3], acc[3]);
          }
          if (i + j + D < ie) codes(i + j + D, j);
        }
      }
    }
    if (splits > 1 || KS > 1) {
      float* to = sums + ((split * KS + ks - 1) * kRowWarps + rw) * 128 + lane * 4;
      if (splits > 1) {
        // into the first block's memory: once it has started, and once it has read the sums of the rows before
        if (t0 == m0) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        else cluster_sync();
        if (split) st_cluster4(cluster_addr(to, 0), acc);
        cluster_sync();
      } else {
        __syncthreads();
        if (ks) *reinterpret_cast<float4*>(to) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        __syncthreads();
      }
      if (split || ks) continue;
      for (int j = 0; j < splits * KS - 1; ++j) {
        const float4 o = *reinterpret_cast<const float4*>(sums + (j * kRowWarps + rw) * 128 + lane * 4);
        acc[0] += o.x, acc[1] += o.y, acc[2] += o.z, acc[3] += o.w;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] *= W4<TE>::kUp;
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

// ------------------------------------------------------------- tiles, tcgen05 --

// Waits for the phase of parity `parity`, at most a second or so.  A wait that gives up says so in
// *err, and ends the block's other waits.
static __device__ __noinline__ bool wait_long(uint64_t* b, uint32_t parity, int* err) {
  const uint64_t t0 = gtimer();
  while (*(volatile int*)err == MOE_OK) {
    if (mbar_try_wait(b, parity, 100000)) return true;
    if (gtimer() - t0 > 1000000000ull) atomicExch(err, MOE_ERR_TIMEOUT);
  }
  return false;
}
// `ready`: what an earlier test_wait said.  A test takes some 150 clocks whatever it finds, and three
// or four of them one after the other a third of a step: they are made early, under other work.
__device__ __forceinline__ bool wait_unless(bool ready, uint64_t* b, uint32_t parity, int* err) {
  return ready || mbar_try_wait(b, parity, 20000) || wait_long(b, parity, err);
}
// Arrives on a barrier of the pair.  What crosses the blocks here is in tensor memory, written or
// read before a tcgen05 fence: nothing of the block's other memory goes with the arrival, and
// a release at cluster scope, which waits for all of the thread's memory accesses, took 1300
// clocks a step.
__device__ __forceinline__ void arrive_pair(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// D [256 x n] over a pair of blocks (+)= A [256 x 16] (each block's 128 rows in its own tensor memory) B [n x 16]^T.
__device__ __forceinline__ void mma_k16_pair_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// Arrives on `bar` of the blocks of `mask` once this thread's MMAs so far have completed.
__device__ __forceinline__ void mma_commit_to(uint64_t* bar, uint32_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(su32(bar)),
      "h"((uint16_t)mask)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
// The same in the codes' own order, (0, 1), (2, 3), (4, 5), (6, 7): a byte of the low codes, one of
// the high ones, and zeros (the sign of a byte below 128) between them.
template <int I>
__device__ __forceinline__ uint32_t code_pair(uint32_t low, uint32_t high) {
  uint32_t p;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(p) : "r"(low), "r"(high), "n"(I | 0x80 | (4 + I) << 8 | 0x8000));
  return p;
}
template <typename TE>
__device__ __forceinline__ void unpack_in_order(uint32_t w, uint32_t offset, uint32_t* v) {
  const uint32_t low = w & 0x0f0f0f0fu, high = w & 0xf0f0f0f0u;
  v[0] = W4<TE>::fma(code_pair<0>(low, high), W4<TE>::kBoth, offset);
  v[1] = W4<TE>::fma(code_pair<1>(low, high), W4<TE>::kBoth, offset);
  v[2] = W4<TE>::fma(code_pair<2>(low, high), W4<TE>::kBoth, offset);
  v[3] = W4<TE>::fma(code_pair<3>(low, high), W4<TE>::kBoth, offset);
}

// Many rows of x to a matrix: persistent pairs of blocks (cta_group::2, a block per SM)
// over tiles of 256 rows of weights x NT rows of x.  A step is 128 products deep: each block
// brings its 128 rows of codes and half of the x rows by TMA; eight warps turn the codes
// into q - z straight into tensor memory, from where the MMAs read them as their A operand
// (through shared memory they would take twice the bandwidth that there is); one thread
// multiplies for both blocks into an accumulator for each group of the scales; and eight
// warps (sixteen at a width of 128) multiply each accumulator by its scales - a scale belongs to a tensor memory
// lane - and add it up in registers while the next ones fill.
//
// What bounds it is the way of a step through its four hands: codes, MMA, sums and back, each
// waiting on the other's barrier.  4001 x 4096 x 4096 in groups of 128 takes 146 us (0.92
// PFLOP/s), 0.65 us a step whose MMAs take some 0.27; without the sums 123.  Smaller groups hand
// over more accumulators: 222 us in groups of 64, 388 in groups of 32.  Two accumulators and
// four steps of codes in tensor memory were faster than three and two; a third set of four
// warps for the codes slower (174 us), and so were 64 columns of sums a thread.
struct LoadNc {
  template <typename T>
  __device__ __forceinline__ T operator()(const T* p) const {
    return __ldg(p);
  }
};
struct F32x2 {
  uint64_t v;
};
__device__ __forceinline__ F32x2 pair_of(float a, float b) {
  F32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 halves_of(F32x2 a) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(a.v));
  return f;
}
__device__ __forceinline__ F32x2 fma_pair(F32x2 a, F32x2 b, F32x2 c) {
  F32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// CUTS: rows of scales and zero points may be cut by their array's ends (Four).  At a width of 128 the second loops cost
// the first ones registers (4001 x 4096 x 4096 in groups of 128, 64 and 32: 149, 236 and 410 us with them, 146, 222 and
// 388 without), so arrays that start and end on whole words have an instance of their own; at 32 and 64 there is no
// difference.  Scales off an 8-byte boundary: 158, 273 and 497 us.
template <typename TE, int NT, int G, bool CUTS>
__global__ void __launch_bounds__(TileCfg<NT>::kThreads, 1)
    w4_tile_kernel(const __grid_constant__ CUtensorMap mC, const __grid_constant__ CUtensorMap mX,
                   const __grid_constant__ W4Args a, int swiglu, int lg) {
  using C = TileCfg<NT>;
  extern __shared__ uint8_t tile_raw[];
  __shared__ alignas(8) uint64_t full_c[kTileStages], full_x[kTileStages], empty[kTileStages], a_full[kAStages];
  __shared__ alignas(8) uint64_t acc_full[C::kBufs], acc_empty[C::kBufs];
  __shared__ uint32_t tmem_slot;
  __shared__ int s_err;
  __shared__ int ws[34];
  uint8_t* sm = reinterpret_cast<uint8_t*>(((uintptr_t)tile_raw + 1023) & ~(uintptr_t)1023);
  float* exchange = reinterpret_cast<float*>(sm + C::kRing);               // [kParts][16][64]
  int* first = reinterpret_cast<int*>(sm + C::kRing + C::kExchange);          // [E + 1]: an expert's first row
  int* cum = first + a.E + 1;                                              // [E + 1]: its first tile
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rank = blockIdx.x & 1;
  const int splits = 1 << lg, split = (int)(blockIdx.x >> 1) & (splits - 1), leader = split * 2;   // places in the cluster
  const int pair = blockIdx.x >> (1 + lg), pairs = gridDim.x >> (1 + lg);   // of all that share a tile
  if (tid == 0) {
    prefetch_map(&mC);
    prefetch_map(&mX);
    for (int i = 0; i < kTileStages; ++i) {
      mbar_init(&full_c[i], 1);
      mbar_init(&full_x[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kAStages; ++i) mbar_init(&a_full[i], 8);           // the leader's: four warps of each block
    for (int i = 0; i < C::kBufs; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 8 * C::kParts);
    }
    s_err = MOE_OK;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&tmem_slot)),
                 "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  pdl_wait();
  // the experts' tiles
  const int per = swiglu ? 128 : 256, outs = swiglu ? a.N / 2 : a.N, row_tiles = (outs + per - 1) / per;
  int tiles = 0;
  for (int b = 0; b < a.E; b += C::kThreads) {
    const int e = b + tid;
    int n = 0, lo = 0, hi = a.P;
    if (e < a.E) {
      if (a.offsets) lo = min(max(a.offsets[e], 0), a.P), hi = min(max(a.offsets[e + 1], 0), a.P);
      n = hi - lo > a.few ? (hi - lo + NT - 1) / NT * row_tiles : 0;
    }
    int all;
    const int at = block_exclusive_scan(n, ws, &all);
    if (e < a.E) {
      first[e] = lo, cum[e] = tiles + at;
      if (e == a.E - 1) first[a.E] = hi;
    }
    tiles += all;
  }
  if (tid == 0) cum[a.E] = tiles;
  if (lg) tiles = min(tiles, pairs);   // one each (the host counts them; offsets that do not ascend could make more)
  tc_fence_before();
  __syncwarp();
  cluster_sync();   // the barriers of both are there
  tc_fence_after();
  pdl_launch_dependents();   // both have their tensor memory: no launch behind this one can come between
  const uint32_t tmem = tmem_slot, tmem_a = tmem + kACols;
  const int all_steps = (a.K + 127) / 128, groups = a.K / G;
  const int sb = all_steps * split >> lg, se = all_steps * (split + 1) >> lg, steps = se - sb;   // this pair's
  bool ok = true;

  int e = 0;
  // a tile's rows of x and first output (of this block)
  struct Tile {
    int m0, m1, o0;
  };
  auto tile_at = [&](int tile) {
    while (cum[e + 1] <= tile) ++e;
    const int local = tile - cum[e], lo = first[e], hi = first[e + 1], tt = (hi - lo + NT - 1) / NT;
    const int rt = local / tt, m0 = lo + (local - rt * tt) * NT;
    return Tile{m0, hi < m0 + NT ? hi : m0 + NT, rt * per + rank * (per / 2)};
  };

  if (warp < 4) {
    if (warp == 0 && elect_one()) {
      RingPos r(kTileStages);
      bool wrapped = false;
      for (int tile = pair; tile < tiles && ok; tile += pairs) {
        const Tile t = tile_at(tile);
        const int row = e * a.N + t.o0, row2 = swiglu ? row + a.N / 2 : row + 64, x0 = t.m0 + rank * (NT / 2);
        for (int k = sb; k < se; ++k) {
          if (wrapped && !(ok = wait_unless(false, &empty[r.stage], r.parity ^ 1, &s_err))) break;
          uint8_t* st = sm + r.stage * C::kStage;
          mbar_expect_tx(&full_c[r.stage], kCodeBytes);
          tma_2d(st, &mC, k * 64, row, &full_c[r.stage]);
          tma_2d(st + kCodeBytes / 2, &mC, k * 64, row2, &full_c[r.stage]);
          if (rank == 0) mbar_expect_tx(&full_x[r.stage], NT * 256);
          const uint32_t bar = cluster_addr(&full_x[r.stage], leader);
          tma_2d_pair(st + kCodeBytes, &mX, k * 128, x0, bar);
          tma_2d_pair(st + kCodeBytes + NT / 2 * 128, &mX, k * 128 + 64, x0, bar);
          r.next();
          wrapped |= r.stage == 0;
        }
      }
    }
    if (warp == 1 && rank == 0 && elect_one()) {
      RingPos r(kTileStages), ar(kAStages), acc(C::kBufs);
      int used = 0;
      const uint32_t idesc = idesc_pair(NT, std::is_same<TE, __nv_bfloat16>::value);
      const uint64_t d0 = umma_desc_sw128(su32(sm));
      const uint32_t both = 3u << leader;
      bool x_there = false, a_there = false, acc_free = false;
      for (int tile = pair; tile < tiles && ok; tile += pairs) {
        for (int k = sb; k < se && ok; ++k) {
          const int last = min(a.K - k * 128, 128) / 16 - 1;
          ok = wait_unless(x_there, &full_x[r.stage], r.parity, &s_err) &&
               wait_unless(a_there, &a_full[ar.stage], ar.parity, &s_err);
          const uint64_t db = d0 + (uint32_t)((r.stage * C::kStage + kCodeBytes) / 16);
          const uint32_t ta = tmem_a + ar.stage * 64;
          uint64_t* done = &empty[r.stage];
          r.next();
          ar.next();
#pragma unroll
          for (int g = 0; g < 128 / G; ++g) {
            if (g * (G / 16) > last || !ok) break;
            if (used >= C::kBufs && !(ok = wait_unless(acc_free, &acc_empty[acc.stage], acc.parity ^ 1, &s_err))) break;
            tc_fence_after();
            const uint32_t d = tmem + acc.stage * NT;
#pragma unroll
            for (int i = 0; i < G / 16; ++i) {
              const int j = g * (G / 16) + i;
              mma_k16_pair_ta(d, ta + j * 8, db + (j >> 2) * (NT / 2 * 128 / 16) + (j & 3) * 2, idesc, i != 0);
            }
            uint64_t* full = &acc_full[acc.stage];
            acc.next();
            ++used;
            acc_free = test_wait(&acc_empty[acc.stage], acc.parity ^ 1);
            if ((g + 1) * (G / 16) > last) {
              x_there = test_wait(&full_x[r.stage], r.parity);
              a_there = test_wait(&a_full[ar.stage], ar.parity);
              mma_commit_to(done, both);   // first: no commit is under way once the last accumulator has been seen
            }
            mma_commit_to(full, both);
          }
        }
      }
    }
    __syncwarp();
    if (lg && pair < tiles) cluster_sync();   // the sums are there
  } else if (warp < 12) {
    // codes of row q * 32 + lane: four warps take the even steps, four the odd ones
    const int set = (warp - 4) >> 2, q = warp & 3, row = q * 32 + lane;
    const uint32_t lanes = (uint32_t)(q * 32) << 16, full_at = cluster_addr(&a_full[0], leader);
    constexpr int kGroups = 128 / G, kPer = 4 / kGroups;   // groups of a step, steps of four groups
    const uint8_t* codes = sm + row * 64;
    const int swizzle = ((row >> 1) & 3) << 4;
    bool codes_there = false;
    int n0 = 0;   // steps before the tile
    for (int tile = pair; tile < tiles && ok; tile += pairs, n0 += steps) {
      const Tile t = tile_at(tile);
      const int o = t.o0 + (swiglu ? row & 63 : row);
      const long long wr = (long long)e * a.N + (swiglu && row >= 64 ? a.N / 2 : 0) + min(o, outs - 1);
      const uint8_t* z_row = a.zeros ? a.zeros + wr * groups : nullptr;
      const int zs = a.zeros ? groups : 0;
      const int k0 = sb + ((n0 ^ set) & 1);   // these warps' first step of the tile
      auto tile_codes = [&](auto zeros) {
        zeros.fetch(k0 / kPer, LoadNc());
        int batch = -1;
        uint32_t z4 = 0x08080808u;
        for (int k = k0; k < se; k += 2) {
          if (k / kPer != batch) {
            batch = k / kPer;
            if (a.zeros) z4 = zeros.value(batch, LoadNc());
            zeros.fetch(kPer == 1 ? batch + 2 : batch + 1, LoadNc());
          }
          const int n = n0 + k - sb, st = n % kTileStages, as = n % kAStages, p = n - kAStages;
          ok = wait_unless(codes_there, &full_c[st], (n / kTileStages) & 1, &s_err);
          // the step that last used this A stage: its own ring stage is given back once it has been multiplied
          const bool free = p < 0 || test_wait(&empty[p % kTileStages], (p / kTileStages) & 1);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t v[32];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint4 w = *reinterpret_cast<const uint4*>(codes + st * C::kStage + (((h * 2 + i) << 4) ^ swizzle));
              const uint32_t offset = W4<TE>::offset(z4 >> ((k % kPer * kGroups + (h * 2 + i) * 32 / G) * 8) & 255);
              unpack_in_order<TE>(w.x, offset, v + 16 * i);
              unpack_in_order<TE>(w.y, offset, v + 16 * i + 4);
              unpack_in_order<TE>(w.z, offset, v + 16 * i + 8);
              unpack_in_order<TE>(w.w, offset, v + 16 * i + 12);
            }
            if (h == 0) {
              ok = __all_sync(0xffffffffu, ok && wait_unless(free, &empty[p % kTileStages], (p / kTileStages) & 1, &s_err));
              tc_fence_after();
            }
            if (ok) tmem_st32(tmem_a + lanes + as * 64 + h * 32, v);
          }
          if (!ok) return;
          codes_there = test_wait(&full_c[(n + 2) % kTileStages], ((n + 2) / kTileStages) & 1);
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_pair(full_at + as * 8);
        }
      };
      if (CUTS && __any_sync(0xffffffffu, Four<1>(z_row, zs).cut(a.zeros, a.zeros_end)))
        tile_codes(Four<1, CUTS>(z_row, zs));
      else
        tile_codes(Four<1>(z_row, zs));
    }
    __syncwarp();
    if (lg && pair < tiles) cluster_sync();   // the sums are there
  } else {
    // sums of row q * 32 + lane, columns from h * kCols
    constexpr int kCols = C::kCols;
    const int q = warp & 3, h = (warp - 12) >> 2, row = q * 32 + lane;
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    const uint32_t empty_at = cluster_addr(&acc_empty[0], leader);
    const int g0 = sb * (128 / G), mine = min(groups, se * (128 / G)) - g0;   // groups
    RingPos acc(C::kBufs);
    bool sums_there = false;
    for (int tile = pair; tile < tiles; tile += pairs) {   // a wait that gave up: NaN to the end
      const Tile t = tile_at(tile);
      const int o = t.o0 + (swiglu ? row & 63 : row);
      const long long wr = (long long)e * a.N + (swiglu && row >= 64 ? a.N / 2 : 0) + min(o, outs - 1);
      const TE* s_row = reinterpret_cast<const TE*>(a.scales) + wr * groups + g0;
      F32x2 total[kCols / 2];
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) total[i].v = 0;
      auto tile_sums = [&](auto scales) {
        scales.fetch(0, LoadNc());
        for (int b = 0; b * 4 < mine && ok; ++b) {
          const uint64_t s4 = scales.value(b, LoadNc());
          scales.fetch(b + 1, LoadNc());
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (b * 4 + j >= mine) break;
            const float s = W4<TE>::scale((uint32_t)(s4 >> (16 * j)) & 0xffff);
            ok = wait_unless(sums_there, &acc_full[acc.stage], acc.parity, &s_err);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            tc_fence_after();
            const F32x2 by = pair_of(s, s);
            const uint32_t at = tmem + lanes + acc.stage * NT + h * kCols, free_at = empty_at + acc.stage * 8;
            acc.next();
#pragma unroll
            for (int c = 0; c < kCols; c += 16) {
              uint32_t u[16];
              tmem_ld16(at + c, u);
              if (c + 16 >= kCols) {   // all of it is in registers
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_pair(free_at);
                sums_there = test_wait(&acc_full[acc.stage], acc.parity);
              }
#pragma unroll
              for (int i = 0; i < 16; i += 2)
                total[(c + i) / 2] = fma_pair(by, pair_of(__uint_as_float(u[i]), __uint_as_float(u[i + 1])), total[(c + i) / 2]);
            }
          }
        }
      };
      if (CUTS && __any_sync(0xffffffffu, Four<2>(s_row, mine).cut(a.scales, a.scales_end)))
        tile_sums(Four<2, CUTS>(s_row, mine));
      else
        tile_sums(Four<2>(s_row, mine));
      auto sum = [&](int i) {
        const float2 f = halves_of(total[i / 2]);
        return ok ? (i & 1 ? f.y : f.x) * W4<TE>::kUp : NAN;
      };
      const int rows = o < outs ? t.m1 - t.m0 - h * kCols : 0;   // of out that are there, from this warp's first
      long long at = (long long)(t.m0 + h * kCols) * a.ld_out + o;
      auto put = [&](int i, float v) {
        if (i < rows) {
          if (a.out_dtype == MOE_DT_F32) reinterpret_cast<float*>(a.out)[at] = v;
          else reinterpret_cast<TE*>(a.out)[at] = from_f32<TE>(v);
        }
        at += a.ld_out;
      };
      if (lg) {
        // sums into the ring's memory, which the last accumulator's products were the last to use: [column][row]; then
        // each pair reads a share of the columns from all, in order
        float* mem = reinterpret_cast<float*>(sm) + h * kCols * 128 + row;
#pragma unroll
        for (int i = 0; i < kCols; ++i) mem[i * 128] = sum(i);
        cluster_sync();
        const int per = kCols >> lg;
        at += (long long)split * per * a.ld_out;
        for (int i = split * per; i < (split + 1) * per; ++i) {
          float v = 0.f, up = 0.f;
          for (int j = 0; j < splits; ++j) {
            const uint32_t f = cluster_addr(mem + i * 128, j * 2 + rank);
            v += ld_cluster(f);
            if (swiglu && q < 2) up += ld_cluster(f + 64 * 4);
          }
          if (!swiglu) put(i, v);
          else if (q < 2) put(i, silu_times(v, up));
        }
      } else if (!swiglu) {
#pragma unroll
        for (int i = 0; i < kCols; ++i) put(i, sum(i));
      } else {
        // ups (rows 64 on) to the gates' threads, 16 columns at a time
        float* ex = exchange + h * 16 * 64 + (row & 63);
        auto meet = [&] { asm volatile("bar.sync %0, 128;" ::"r"(1 + h) : "memory"); };   // the four warps of these columns
#pragma unroll
        for (int c = 0; c < kCols; c += 16) {
          if (q >= 2)
#pragma unroll
            for (int i = 0; i < 16; ++i) ex[i * 64] = sum(c + i);
          meet();
          if (q < 2)
#pragma unroll
            for (int i = 0; i < 16; ++i) put(c + i, silu_times(sum(c + i), ex[i * 64]));
          meet();
        }
      }
    }
  }
  __syncwarp();
  if (!ok) {   // a wait gave up: leave the copies in flight time to land
    const uint64_t since = gtimer();
    while (gtimer() - since < 2000000ull) {
    }
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync();   // nothing of this block is used by the other any more
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
  if (tid == 0 && s_err != MOE_OK && a.err) atomicExch(a.err, MOE_ERR_TIMEOUT);
}

// --------------------------------------------------------------------- host --

// codes: rows of K / 2 bytes, boxes of 64 bytes x 64 rows, 64-byte swizzle
static moe_status map_codes(CUtensorMap* m, const W4Args& a) {
  auto fn = tensor_map_encoder();
  if (!fn) return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  cuuint64_t dims[2] = {(cuuint64_t)a.K / 2, (cuuint64_t)a.E * a.N};
  cuuint64_t strides[1] = {(cuuint64_t)a.K / 2};
  cuuint32_t box[2] = {64, 64};
  cuuint32_t es[2] = {1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(a.codes), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled (codes) failed: %d", (int)r);
  return MOE_OK;
}
// At most this many tiles: every expert's last one may be a part.
static long long most_tiles(const W4Args& a, int swiglu, int NT) {
  const int outs = swiglu ? a.N / 2 : a.N, per = swiglu ? 128 : 256;
  const long long of_x = a.offsets ? (long long)a.P / NT + (a.E < a.P / (a.few + 1) ? a.E : a.P / (a.few + 1)) : ((long long)a.P + NT - 1) / NT;
  return of_x * ((outs + per - 1) / per);
}
template <typename TE, int NT, int G, bool CUTS>
static cudaError_t allow_tiles() {
  static char allowed[64];
  return allow_smem(w4_tile_kernel<TE, NT, G, CUTS>, tile_smem<NT>(kMaxExperts), allowed);
}
// How many clusters of 2 << lg of the blocks, one to an SM, the device runs at once: a cluster's SMs are
// neighbours, and fewer fit than the SMs' number says (of eight 15, not 19).
static cudaError_t clusters_at_once(const void* kernel, int lg, int threads, size_t smem, int* n) {
  static int known[64][3];   // + 1; every instance has its SM to itself (kAloneBytes), so it is the same for all
  int dev;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int k = dev < 64 ? __atomic_load_n(&known[dev][lg], __ATOMIC_RELAXED) : 0;
  if (k == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2u << lg), cfg.blockDim = dim3(threads), cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2u << lg, attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr, cfg.numAttrs = 1;
    int got = 0;
    e = cudaOccupancyMaxActiveClusters(&got, kernel, &cfg);
    if (e != cudaSuccess) return e;
    k = got + 1;
    if (dev < 64) __atomic_store_n(&known[dev][lg], k, __ATOMIC_RELAXED);
  }
  *n = k - 1;
  return cudaSuccess;
}
// Few tiles: clusters of two or four pairs (1 << lg) share the steps of one each, where all of them run at once.  Measured,
// 57 rows of x, 4096 x 2048: 11.6 us by four, 18.7 by two, 23.4 by pairs.
static cudaError_t splits_of(const W4Args& a, long long most, const void* kernel, int threads, size_t smem, int* lg) {
  const int steps = (a.K + 127) / 128;
  for (*lg = 0; *lg < 2 && steps >= 4 << *lg; ++*lg) {   // two steps each at least
    int fit;
    const cudaError_t e = clusters_at_once(kernel, *lg + 1, threads, smem, &fit);
    if (e != cudaSuccess) return e;
    if (most > fit) break;
  }
  return cudaSuccess;
}
template <typename TE, int NT, int G, bool CUTS>
static moe_status launch_tiles(const W4Args& a, int dtype, int swiglu, cudaStream_t s) {
  CUtensorMap mC, mX;
  moe_status st = map_codes(&mC, a);
  if (st == MOE_OK) st = map_rows(&mX, a.x, dtype, a.K, a.P, a.ld_x, NT / 2);
  if (st != MOE_OK) return st;
  auto kernel = w4_tile_kernel<TE, NT, G, CUTS>;
  const cudaError_t allowed = allow_tiles<TE, NT, G, CUTS>();
  MOE_CUDA(allowed);
  const long long most = most_tiles(a, swiglu, NT);
  MOE_ARG(most <= 0x3fffffff, "too many tiles");
  const int pairs = device_sms() / 2;
  int lg;
  MOE_CUDA(splits_of(a, most, (const void*)kernel, TileCfg<NT>::kThreads, tile_smem<NT>(kMaxExperts), &lg));
  return launch_cluster(kernel, dim3((unsigned)(lg || most < pairs ? most : pairs) << (lg + 1)), TileCfg<NT>::kThreads, 2 << lg,
                        tile_smem<NT>(a.E), s, "w4_tile_kernel", mC, mX, a, swiglu, lg);
}
template <typename TE, int G>
static moe_status launch_tiles_of(const W4Args& a, int dtype, int swiglu, cudaStream_t s) {
  int nt = 128;
  if (a.offsets) {   // an expert's rows in one tile, most of the time
    const int mean = a.P / a.E;
    nt = mean > 64 ? 128 : mean > 32 || a.few ? 64 : 32;
  } else {
    // Rounds of tiles times steps times what a step of the width takes (5, 7 and 10 parts: measured 0.64, 0.9 and 1.26 us
    // in groups of 64), and 70 parts for the exchange of a split.  4096 x 4096 at widths of 32, 64 and 128, groups of 128:
    // 64 rows 13.6, 16.5 and 20.5 us, 128 rows 17.2, 17.1 and 20.8, 256 rows 29.7, 19.0 and 21.4, 512 rows 55, 33 and
    // 25.  The parts' ratios are near enough in groups of 128; in groups of 32 a narrow width can cost up to a seventh
    // more than the best one (100 rows 29.3 us at 32, which is taken, 25.7 at 64).
    const int steps = (a.K + 127) / 128, pairs = device_sms() / 2;
    long long least = 0;
    auto consider = [&](auto width, int part) {
      constexpr int NT = decltype(width)::value;
      const long long most = most_tiles(a, swiglu, NT);
      int lg;
      cudaError_t e = allow_tiles<TE, NT, G, true>();
      if (e == cudaSuccess)
        e = splits_of(a, most, (const void*)w4_tile_kernel<TE, NT, G, true>, TileCfg<NT>::kThreads, tile_smem<NT>(kMaxExperts), &lg);
      if (e != cudaSuccess) return e;
      const long long rounds = lg ? 1 : (most + pairs - 1) / pairs, cost = rounds * ((steps + (1 << lg) - 1) >> lg) * part + (lg ? 70 : 0);
      if (least == 0 || cost < least) least = cost, nt = NT;
      return cudaSuccess;
    };
    MOE_CUDA(consider(std::integral_constant<int, 32>(), 5));
    MOE_CUDA(consider(std::integral_constant<int, 64>(), 7));
    MOE_CUDA(consider(std::integral_constant<int, 128>(), 10));
  }
  if (nt == 64) return launch_tiles<TE, 64, G, true>(a, dtype, swiglu, s);
  if (nt == 32) return launch_tiles<TE, 32, G, true>(a, dtype, swiglu, s);
  const long long n_groups = (long long)a.E * a.N * (a.K / G);
  const bool cuts = ends_cut(a.scales, n_groups, 2) || (a.zeros && ends_cut(a.zeros, n_groups, 1));
  return cuts ? launch_tiles<TE, 128, G, true>(a, dtype, swiglu, s) : launch_tiles<TE, 128, G, false>(a, dtype, swiglu, s);
}

template <typename TE, int WPL, int KS>
static moe_status launch_rows_kernel(const W4Args& a, int swiglu, int lg, cudaStream_t s) {
  auto kernel = w4_rows_kernel<TE, WPL, KS>;
  static char allowed[64];
  MOE_CUDA(allow_smem(kernel, kChunkBytes + (kMaxSplits - 1) * 4096, allowed));
  const int outs = swiglu ? a.N / 2 : a.N, per = 8 / KS * (swiglu ? 8 : 16), tiles = (outs + per - 1) / per;
  const int experts = a.offsets && a.P < a.E ? a.P : a.E, steps = (a.K + 127) / 128;
  const int splits = 1 << lg, mine = (steps + splits - 1) / splits, x_bytes = (mine < kChunk ? mine : kChunk) * 2048;
  const size_t smem = x_bytes + (splits * KS - 1) * (8 / KS) * 512;
  MOE_ARG((long long)tiles * splits <= 0x7fffffffLL, "too many tiles");
  if (splits > 1)
    return launch_cluster(kernel, dim3(tiles * splits, experts), 256, splits, smem, s, "w4_rows_kernel", a, swiglu, lg, x_bytes);
  cudaError_t e = launch_pdl(kernel, dim3(tiles, experts), dim3(256), smem, s, a, swiglu, 0, x_bytes);
  if (e != cudaSuccess) return cuda_fail(e, "w4_rows_kernel");
  return check_launch("w4_rows_kernel");
}
template <typename TE, int WPL>
static moe_status launch_split_rows(const W4Args& a, int swiglu, cudaStream_t s) {
  // Blocks of 128 rows fill the GPU.  Else, with few rows of x, blocks of 16 whose warps split the groups (4096 x 4096,
  // one row: 4.8 us, clusters 6.4); with more of them a block would load more of x than of codes, so clusters share the
  // groups of 128 rows (8 rows: 6.5 us, blocks of 16 8.5; 8192 x 8192: 16 and 30).
  const long long tiles = ((long long)a.N + 127) / 128 * (a.offsets && a.P < a.E ? a.P : a.E);
  if (tiles >= device_sms()) return launch_rows_kernel<TE, WPL, 1>(a, swiglu, 0, s);
  if (a.P < (long long)a.E * 3) return launch_rows_kernel<TE, WPL, 8>(a, swiglu, 0, s);
  const int steps = (a.K + 127) / 128;
  int lg = 0;
  while (1 << lg < kMaxSplits && tiles << lg < device_sms() && steps >= 4 << lg) ++lg;
  return launch_rows_kernel<TE, WPL, 1>(a, swiglu, lg, s);
}
// Few rows to an expert on average can still be many to some, and w4_rows_kernel reads the codes again for every eight: such
// experts go to a launch of tiles behind it.  1802 rows of 2048 to 4096, 1500 of them one expert's of 256: 78 us, 1263
// without; where no expert has so many the launch costs 2 to 5 us (512 rows of 256 experts 185 us, 180 without), which a
// call of up to kFewInAll rows is spared: 64 rows that are all one expert's read its codes eight times, 119 us for 4096 x
// 4096 (13.6 as a dense product).
constexpr int kFewRows = 24, kFewInAll = 64;
template <typename TE>
static moe_status launch_w4(const W4Args& a, int dtype, int swiglu, cudaStream_t s) {
  ProfScope ps(MOE_K_W4, s);
  // Up to eight rows of x the kernel for few reads the codes once; experts have more than the mean too: 2048 x 2048, 256
  // experts, 8 rows to each 165 us (201 by tiles), 12 rows 219 (201).
  W4Args b = a;
  b.few = a.P >= (long long)a.E * (a.offsets ? 11 : 9) ? 0 : a.offsets && a.P > kFewInAll ? kFewRows : a.P;
  if (b.few) {
    const moe_status st = a.g == 128  ? launch_split_rows<TE, 4>(b, swiglu, s)
                          : a.g == 64 ? launch_split_rows<TE, 2>(b, swiglu, s)
                                      : launch_split_rows<TE, 1>(b, swiglu, s);
    if (st != MOE_OK || b.few == a.P) return st;
  }
  if (a.g == 128) return launch_tiles_of<TE, 128>(b, dtype, swiglu, s);
  if (a.g == 64) return launch_tiles_of<TE, 64>(b, dtype, swiglu, s);
  return launch_tiles_of<TE, 32>(b, dtype, swiglu, s);
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
  MOE_ARG(E >= 1 && E <= kMaxExperts, "E must be in [1, %d] (got %d)", kMaxExperts, E);
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
  const long long n_groups = (long long)E * N * (K / group);
  W4Args a = {P, N, K, E, group, out_dtype, x, ld_x, ld_out, codes, zeros, scales, (const char*)scales + n_groups * 2,
              zeros ? zeros + n_groups : nullptr, offsets, out, d_error, 0};
  return dtype == MOE_DT_BF16 ? launch_w4<__nv_bfloat16>(a, dtype, swiglu ? 1 : 0, stream)
                              : launch_w4<__half>(a, dtype, swiglu ? 1 : 0, stream);
}
