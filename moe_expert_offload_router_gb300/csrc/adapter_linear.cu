// A shared projection with low-rank adapters of many requests beside it:
//   out[t] = W x[t] + B[a] u[t],  u[t] = scale[a] A[a] x[t],  a = adapter_ids[t].
//
// u (fp32 [T, R]) comes from a first kernel; the projection's kernel starts
// beside it (programmatic dependent launch) and waits for it only before its
// epilogue or the steps that runs of one adapter add, where B[a] u is added to the
// tokens that name a: an adapter touches the tokens that name it and no others,
// whoever shares their tile.
//
// u enters that product as terms of x's type, its leading bits, the next ones, ...:
// with fp16 two (22 bits of a token's largest value; scaled by a power of two, or
// unscaled where they hold that many), with bf16 three (24 bits) for fp32 results and
// two (16 bits) for 16-bit ones.  A third term there changes nothing that a bf16 result
// can show: 4001 x 4096 x 4096, rank 32, is 1.662e-3 from 64 bits (its rounding) and
// 1.46e-4 from the rounded exact result with two as with three, in 107.6 us and 109.6.
//
// The projection runs on tcgen05 (kind::f16, fp32 accumulators in tensor
// memory) with the operands swapped: W's rows are the MMA's 128 rows and the
// tokens its N columns, so a decode batch of 16 tokens is one N = 16 tile and
// no row of the tensor core is spent on padding.
#include <math.h>

#include <type_traits>

#include "dtype.cuh"
#include "tcgen05_issue.cuh"

namespace moe {

struct LinearArgs {
  int T, H, N, n, R, out_dtype;
  const void *x, *W, *A, *B;
  long long ld_x, ld_w, ld_out;
  const int32_t* ids;
  const float* scale;
  void* out;
  float* u;            // [T, R]
  void* u_terms;       // [terms][T, R] of x's type: u's leading bits, the next ones, ... (large batches)
  int terms;
  int32_t* group;      // [T / 16] (large batches): the adapter that 16 tokens share, -1: none, or kMixed
  int32_t* err;
};

constexpr int kMixed = -2;   // a group of 16 tokens that do not share one adapter

template <typename TE>
struct Pair;   // two packed elements as fp32
template <>
struct Pair<__nv_bfloat16> {
  static __device__ __forceinline__ float2 f32(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
};
template <>
struct Pair<__half> {
  static __device__ __forceinline__ float2 f32(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
};

// ------------------------------------------------------------ u = scale A x --

// Few tokens: a block takes kDots ranks of one token, its four warps splitting H,
// so that every load of a row of 4096 is under way at once.  Every token reads its
// own R x H of A (from L2 where tokens share an adapter).  Latency: about 3 us for
// 64 tokens of rank 16, mostly under the projection's own start.
constexpr int kDots = 4;
template <typename TE>
__global__ void __launch_bounds__(128) adapter_dot_kernel(const LinearArgs a) {
  __shared__ float part[4][kDots];
  pdl_wait();
  pdl_launch_dependents();   // after the wait: the projection may read x from its start
  const int t = blockIdx.x, r0 = blockIdx.y * kDots, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int id = a.ids[t];
  if (id >= a.n && a.err && blockIdx.y == 0 && threadIdx.x == 0) atomicCAS(a.err, MOE_OK, MOE_ERR_INVALID);
  if (id < 0 || id >= a.n) return;
  const uint4* x = reinterpret_cast<const uint4*>(reinterpret_cast<const TE*>(a.x) + t * a.ld_x);
  const uint4* A = reinterpret_cast<const uint4*>(reinterpret_cast<const TE*>(a.A) + ((long long)id * a.R + r0) * a.H);
  const int nc = a.H / 8;   // 16-byte chunks of a row
  float s[kDots] = {};
#pragma unroll 4
  for (int c = threadIdx.x; c < nc; c += 128) {
    const uint4 xv = x[c];
    const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
    for (int r = 0; r < kDots; ++r) {
      const uint4 av = A[r * (long long)nc + c];
      const uint32_t aw[4] = {av.x, av.y, av.z, av.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 p = Pair<TE>::f32(xw[i]), q = Pair<TE>::f32(aw[i]);
        s[r] = fmaf(p.x, q.x, fmaf(p.y, q.y, s[r]));
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int r = 0; r < kDots; ++r) s[r] += __shfl_xor_sync(0xffffffffu, s[r], o);
  if (lane == 0)
#pragma unroll
    for (int r = 0; r < kDots; ++r) part[warp][r] = s[r];
  __syncthreads();
  if (threadIdx.x < kDots)
    a.u[(long long)t * a.R + r0 + threadIdx.x] =
        (a.scale ? a.scale[id] : 1.f) *
        ((part[0][threadIdx.x] + part[1][threadIdx.x]) + (part[2][threadIdx.x] + part[3][threadIdx.x]));
}

// -------------------------------------------------------------- projection --

// A tensor-core accumulator loses a little with every step (it truncates: 4.2e-6
// of the result over 4096 products, 0.5e-6 over 512), so a result kept in fp32
// takes at most this many 64-wide steps in one accumulator where there is room.
// A 16-bit result takes one over all of H: 4.2e-6 is a four-hundredth of bf16's
// rounding (1.66e-3) and a fiftieth of f16's (2.1e-4), while adding chunks up in
// registers holds the persistent kernel's tiles to 128 tokens (4001 x 4096 x 4096
// without adapters: fp32 results take 128 us, bf16 ones 80).
constexpr int kF32Chunk = 8;
constexpr int kRows = 128;          // outputs (W rows) of a tile
constexpr int kATile = kRows * 128; // bytes of a 64-wide K step of W

template <int NT>
struct SplitCfg {
  static constexpr int kStage = kATile + NT * 128;
  static constexpr int kStages = NT <= 64 ? 8 : 6;
  static constexpr int kSmem = kStages * kStage + 1024;
  static constexpr int kAcc = NT <= 64 ? 8 : 512 / NT;   // accumulators for fp32 results
  static constexpr int kCols = kAcc * NT;
  // u's three terms of all ranks, a row for each token (adapter_tiles)
  static constexpr int kTerms = 3 * NT * (128 * 2 + 16);
  static_assert(NT * kRows * 4 + kTerms <= kStages * kStage, "the partial sums and u's terms fit the stages");
};

template <typename TE>
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack_pair<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack_pair<__half>(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename TE>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
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

// Eight values of u (fp32, times `up`; zeros where not `in`) as three terms of x's type.
template <typename TE>
__device__ __forceinline__ void split_terms(const float* u, bool in, float up, uint32_t (&w)[3][4]) {
  float4 p = make_float4(0.f, 0.f, 0.f, 0.f), q = p;
  if (in) p = *reinterpret_cast<const float4*>(u), q = *reinterpret_cast<const float4*>(u + 4);
  float f[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
  if (!std::is_same<TE, __nv_bfloat16>::value)
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] *= up;
#pragma unroll
  for (int t = 0; t < 3; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[t][i] = pack_pair<TE>(f[2 * i], f[2 * i + 1]);
      const float2 r = Pair<TE>::f32(w[t][i]);
      f[2 * i] -= r.x, f[2 * i + 1] -= r.y;
    }
}
// Both m16 tiles of B's rows (A: rows g, g + 8, g + 16, g + 24) times u's first `terms` terms.
template <typename TE>
__device__ __forceinline__ void mma_terms(float (&d0)[4], float (&d1)[4], const uint4 (&A)[4],
                                          const uint32_t (&w)[3][4], int terms) {
#pragma unroll
  for (int t = 0; t < 3; ++t) {
    if (t == 2 && terms < 3) break;
    mma16816<TE>(d0, A[0].x, A[1].x, A[0].y, A[1].y, w[t][0], w[t][1]);
    mma16816<TE>(d1, A[2].x, A[3].x, A[2].y, A[3].y, w[t][0], w[t][1]);
    mma16816<TE>(d0, A[0].z, A[1].z, A[0].w, A[1].w, w[t][2], w[t][3]);
    mma16816<TE>(d1, A[2].z, A[3].z, A[2].w, A[3].w, w[t][2], w[t][3]);
  }
}

// The adapters' part of 32 outputs (from n0) x 16 tokens (from t0, `cols` of them
// there) by a warp; lane l holds the id of token l & 15 in `mine` (negative: none).
// Whatever the mixture: B[a] u is taken for every adapter that the tokens name,
// over all 16 columns, and a token keeps the column of its own; no value of
// another adapter is added to it, not even times 0.  u enters as terms of x's type
// (fp16: scaled by a power of two to below 2^14 first, so that it neither
// overflows nor loses its low bits).  Fragments come straight from memory: lane
// (g, c) loads 16 bytes of B at k = 32 i + 8 c of rows g and g + 8 and takes them
// as the k16 steps 2 i and 2 i + 1, u's eight values in the same order.
// sel[m][j]: rows 16 m + g (+ 8), columns 8 j + 2 c (+ 1), as m16n8 accumulators.
template <typename TE>
__device__ __forceinline__ void adapter_block(const LinearArgs& a, int mine, long long t0, int cols, int n0,
                                              float (&sel)[2][2][4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  constexpr bool kScaled = !std::is_same<TE, __nv_bfloat16>::value;
#pragma unroll
  for (int i = 0; i < 16; ++i) (&sel[0][0][0])[i] = 0.f;
  uint32_t left = __ballot_sync(0xffffffffu, mine >= 0) & 0xffff;
  const float* u[2];
  float up[2] = {1.f, 1.f}, down[2][2];   // of column g; of columns 2 c and 2 c + 1
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int col = j * 8 + g;
    u[j] = a.u + (t0 + (col < cols ? col : 0)) * a.R + c * 8;
    if (kScaled) {
      float top = 0.f;
      for (int k = 0; k + c * 8 < a.R; k += 32) {
        const float4 p = *reinterpret_cast<const float4*>(u[j] + k), q = *reinterpret_cast<const float4*>(u[j] + k + 4);
        top = fmaxf(fmaxf(fmaxf(fabsf(p.x), fabsf(p.y)), fmaxf(fabsf(p.z), fabsf(p.w))),
                    fmaxf(fmaxf(fmaxf(fabsf(q.x), fabsf(q.y)), fmaxf(fabsf(q.z), fabsf(q.w))), top));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      int e = (int)(__float_as_uint(top) >> 23 & 255) - 127 - 13;   // top in [2^13, 2^14) after the scale
      e = top == 0.f || e > 114 ? 0 : e < -100 ? -100 : e;
      up[j] = __uint_as_float((uint32_t)(127 - e) << 23);
      const float dn = __uint_as_float((uint32_t)(127 + e) << 23);
      down[j][0] = __shfl_sync(0xffffffffu, dn, c * 8);
      down[j][1] = __shfl_sync(0xffffffffu, dn, c * 8 + 4);
    }
  }
  // u's terms of the first 32 ranks, for all adapters; B's rows one adapter ahead
  uint32_t w0[2][3][4];
  const bool in0 = c * 8 < a.R;
#pragma unroll
  for (int j = 0; j < 2; ++j) split_terms<TE>(u[j], in0, up[j], w0[j]);
  auto row_of = [&](int id, int m) {
    const int n = n0 + m * 8 + g;
    return reinterpret_cast<const TE*>(a.B) + ((long long)id * a.N + (n < a.N ? n : a.N - 1)) * a.R + c * 8;
  };
  auto rows_at = [&](int id, int k, uint4 (&A)[4]) {
    const bool in = k + c * 8 < a.R;
#pragma unroll
    for (int m = 0; m < 4; ++m)
      A[m] = in ? *reinterpret_cast<const uint4*>(row_of(id, m) + k) : make_uint4(0, 0, 0, 0);
  };
  int id = left ? __shfl_sync(0xffffffffu, mine, __ffs(left) - 1) : 0;
  uint4 A[4];
  if (left) rows_at(id, 0, A);
  while (left) {
    const uint32_t who = __ballot_sync(0xffffffffu, mine == id) & 0xffff;
    left &= ~who;
    const int next = left ? __shfl_sync(0xffffffffu, mine, __ffs(left) - 1) : id;
    uint4 N[4];
    if (left) rows_at(next, 0, N);
    float d[2][2][4] = {};
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (who >> (j * 8) & 0xff) mma_terms<TE>(d[0][j], d[1][j], A, w0[j], a.terms);
    for (int k = 32; k < a.R; k += 32) {
      rows_at(id, k, A);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (!(who >> (j * 8) & 0xff)) continue;
        uint32_t w[3][4];
        split_terms<TE>(u[j] + k, k + c * 8 < a.R, up[j], w);
        mma_terms<TE>(d[0][j], d[1][j], A, w, a.terms);
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (who >> (j * 8 + 2 * c + i) & 1)
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            sel[m][j][i] += kScaled ? d[m][j][i] * down[j][i] : d[m][j][i];
            sel[m][j][i + 2] += kScaled ? d[m][j][i + 2] * down[j][i] : d[m][j][i + 2];
          }
    id = next;
#pragma unroll
    for (int m = 0; m < 4; ++m) A[m] = N[m];
  }
}
// The same into a warp's own [16][32] of shared memory, from where lane l takes output n0 + l.
template <typename TE>
__device__ __forceinline__ void adapter_turn(const LinearArgs& a, int t1, int n0, float* own) {
  const int lane = threadIdx.x & 31, cols = a.T - t1 < 16 ? a.T - t1 : 16;
  int mine = (lane & 15) < cols ? a.ids[t1 + (lane & 15)] : -1;
  if (mine >= a.n) mine = -1;
  float sel[2][2][4];
  adapter_block<TE>(a, mine, t1, cols, n0, sel);
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int m = 0; m < 2; ++m)
        own[(j * 8 + 2 * (lane & 3) + (k & 1)) * 32 + m * 16 + (lane >> 2) + (k & 2) * 4] = sel[m][j][k];
  __syncwarp();
}
// One column of 16 tokens (those below `left`).
template <typename T>
__device__ __forceinline__ void store16(T* o, long long ld, int left, const float* v, bool ok) {
  if (left >= 16 && ok) {
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j * ld] = from_f32<T>(v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (j < left) o[j * ld] = from_f32<T>(ok ? v[j] : NAN);
  }
}

template <typename TE>
__device__ __forceinline__ void store4(const LinearArgs& a, long long t, int n, const float* v) {
  if (a.out_dtype == MOE_DT_F32) {
    float* o = reinterpret_cast<float*>(a.out) + t * a.ld_out + n;
    if (n + 4 <= a.N && ((uintptr_t)o & 15) == 0) {
      *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      for (int j = 0; j < 4 && n + j < a.N; ++j) o[j] = v[j];
    }
  } else {
    TE* o = reinterpret_cast<TE*>(a.out) + t * a.ld_out + n;
    if (n + 4 <= a.N && ((uintptr_t)o & 7) == 0) {
      TE e[4] = {from_f32<TE>(v[0]), from_f32<TE>(v[1]), from_f32<TE>(v[2]), from_f32<TE>(v[3])};
      *reinterpret_cast<uint2*>(o) = *reinterpret_cast<const uint2*>(e);
    } else {
      for (int j = 0; j < 4 && n + j < a.N; ++j) o[j] = from_f32<TE>(v[j]);
    }
  }
}

// The adapters' part of a block of the split kernel.  Its tokens are put in order of
// their adapters, and a tile is up to eight of them that share one: a tile is
// multiplied by its own adapter's rows alone, so nothing of another one can reach a
// token, and B is read once for eight tokens of an adapter and not for each.
template <int NT>
struct AdapterTiles {
  int id[NT], start[NT];      // a token's adapter; the place of its tile, if it is the first of one
  int token[NT];              // in order of adapters
  int2 tile[NT];              // its first place and tokens (shifted by 8), its adapter
  float down[NT];             // fp16: what a place's product is multiplied by
  int tokens, tiles;

  // By threads 0 to 191: tokens t0 to t0 + share.
  __device__ __forceinline__ void fill(const LinearArgs& a, int i, int t0, int share) {
    int mine = 0x7fffffff, before = 0, less = 0, same = 0;
    if (i < share) {
      if (t0 + i < a.T) mine = a.ids[t0 + i];
      if (mine < 0 || mine >= a.n) mine = 0x7fffffff;
      id[i] = mine;
    }
    asm volatile("bar.sync 1, 192;" ::: "memory");
    int all = 0;
#pragma unroll 4
    for (int j = 0; i < share && j < share; ++j) {
      const int o = id[j];
      all += o != 0x7fffffff;
      less += o < mine;
      same += o == mine;
      before += o == mine && j < i;
    }
    const int place = less + before;
    const bool there = i < share && mine != 0x7fffffff, head = there && before % 8 == 0;
    if (there) token[place] = i;
    if (i < share) start[i] = head ? place : -1;
    asm volatile("bar.sync 1, 192;" ::: "memory");
    int at = 0, heads = 0;
#pragma unroll 4
    for (int j = 0; i < share && j < share; ++j) {
      at += start[j] >= 0 && start[j] < place;
      heads += start[j] >= 0;
    }
    if (head) tile[at] = make_int2(place | (same - before < 8 ? same - before : 8) << 8, mine);
    if (i == 0) tokens = all, tiles = heads;
  }
};
// u (fp32) enters as terms of x's type, which all threads first lay into shared
// memory (`room`) in the tiles' order; fp16 scaled by a power of two to below 2^14, so
// that it neither overflows nor loses its low bits.  A warp then takes 32 of the 128
// outputs and every other tile.  B comes straight from memory, kAhead steps of 32
// ranks ahead: lane (g, c) loads 16 bytes at k = 32 i + 8 c of rows g, g + 8, g + 16
// and g + 24 and takes them as the k16 steps 2 i and 2 i + 1, u's eight values in the
// same order.  `sums`: [share][128], made by fill_sums, to which the products are added.  The MMAs'
// latency bounds a tile: in four chains 57 tokens of 20 adapters of rank 40 to 2035
// outputs take 15.0 us, in two 17.0; two steps ahead 16.2, eight (more code) 16.9.
template <typename TE, int NT, typename F>
__device__ __forceinline__ void adapter_tiles(const LinearArgs& a, AdapterTiles<NT>& s, int t0, int n0, float* sums,
                                              uint8_t* room, F fill_sums) {
  constexpr bool kScaled = !std::is_same<TE, __nv_bfloat16>::value;
  constexpr int kAhead = 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3, half = warp >> 2;
  const int ld = a.R * 2 + 16, term = NT * ld;   // bytes of a token's row, of a term
  const int n1 = n0 + (warp & 3) * 32 + g, tiles = s.tiles;
  int row[4];   // of B, within an adapter's
#pragma unroll
  for (int m = 0; m < 4; ++m) row[m] = (n1 + m * 8 < a.N ? n1 + m * 8 : a.N - 1) * a.R + c * 8;
  uint4 A[kAhead][4];
  int lt = half, lk = 0;
  auto fetch = [&](uint4 (&X)[4]) {
    if (lt >= tiles) return;
    const TE* B = reinterpret_cast<const TE*>(a.B) + (long long)s.tile[lt].y * a.N * a.R + lk;
    const bool in = lk + c * 8 < a.R;
#pragma unroll
    for (int m = 0; m < 4; ++m) X[m] = in ? *reinterpret_cast<const uint4*>(B + row[m]) : make_uint4(0, 0, 0, 0);
    if ((lk += 32) >= a.R) lk = 0, lt += 2;
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) fetch(A[i]);
  pdl_wait();   // u
  const int width = a.R <= 16 ? 4 : a.R <= 32 ? 8 : a.R <= 64 ? 16 : 32;   // lanes of a token, four ranks each
  const int wl = lane & (width - 1), each = 32 / width;
#pragma unroll 4
  for (int p0 = warp * each; p0 < s.tokens; p0 += 8 * each) {
    const int p = p0 + lane / width;
    const bool in = p < s.tokens && wl * 4 < a.R;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (in) v = *reinterpret_cast<const float4*>(a.u + (long long)(t0 + s.token[p]) * a.R + wl * 4);
    float f[4] = {v.x, v.y, v.z, v.w};
    if (kScaled) {
      float top = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
      for (int o = 1; o < width; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      int e = (int)(__float_as_uint(top) >> 23 & 255) - 127 - 13;   // top in [2^13, 2^14) after the scale
      e = top == 0.f || e > 114 ? 0 : e < -100 ? -100 : e;
      const float up = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] *= up;
      if (in && wl == 0) s.down[p] = __uint_as_float((uint32_t)(127 + e) << 23);
    }
#pragma unroll
    for (int t = 0; t < 3; ++t) {
      if (t == 2 && a.terms < 3) break;
      const uint2 w = make_uint2(pack_pair<TE>(f[0], f[1]), pack_pair<TE>(f[2], f[3]));
      if (in) *reinterpret_cast<uint2*>(room + t * term + p * ld + wl * 8) = w;
      const float2 q = Pair<TE>::f32(w.x), r = Pair<TE>::f32(w.y);
      f[0] -= q.x, f[1] -= q.y, f[2] -= r.x, f[3] -= r.y;
    }
  }
  fill_sums();   // B's rows are on their way
  __syncthreads();
  int ct = half, ck = 0;
  float d[2][2][4] = {};   // by rows, by k16 step: four chains of MMAs
  while (ct < tiles) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (ct >= tiles) break;
      const int span = s.tile[ct].x, p = span & 255, len = span >> 8;
      const uint8_t* u = room + (p + (g < len ? g : 0)) * ld + (ck + c * 8) * 2;
      const bool in = ck + c * 8 < a.R;
#pragma unroll
      for (int t = 0; t < 3; ++t) {
        if (t == 2 && a.terms < 3) break;
        const uint4 w = in ? *reinterpret_cast<const uint4*>(u + t * term) : make_uint4(0, 0, 0, 0);
        mma16816<TE>(d[0][0], A[i][0].x, A[i][1].x, A[i][0].y, A[i][1].y, w.x, w.y);
        mma16816<TE>(d[1][0], A[i][2].x, A[i][3].x, A[i][2].y, A[i][3].y, w.x, w.y);
        mma16816<TE>(d[0][1], A[i][0].z, A[i][1].z, A[i][0].w, A[i][1].w, w.z, w.w);
        mma16816<TE>(d[1][1], A[i][2].z, A[i][3].z, A[i][2].w, A[i][3].w, w.z, w.w);
      }
      fetch(A[i]);
      if ((ck += 32) < a.R) continue;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (2 * c + j >= len) continue;
        float* at = sums + s.token[p + 2 * c + j] * kRows + (warp & 3) * 32 + g;
        const float by = kScaled ? s.down[p + 2 * c + j] : 1.f;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float v = d[m >> 1][0][(m & 1) * 2 + j] + d[m >> 1][1][(m & 1) * 2 + j];
          at[m * 8] += kScaled ? v * by : v;
        }
      }
#pragma unroll
      for (int m = 0; m < 16; ++m) (&d[0][0][0])[m] = 0.f;
      ck = 0, ct += 2;
    }
  }
}

// One tile of 128 outputs x NT tokens per cluster, whose blocks split H: each
// brings its share of W and x by TMA (as many 64-wide steps in flight as the
// stages hold: with H / cluster <= 512 the whole share), multiplies it, puts its
// fp32 sums into its own shared memory, and adds up the blocks' sums, in rank
// order, for its share of the tokens.  64 tokens to 2048 outputs, H = 4096: 7.2 us
// alone (19.5 MB), 12.1 with adapters; bound by what an SM takes in (W's 128 rows
// and x's 64 of 1024 columns: 390 KB) and the way there and back.
template <typename TE, int NT>
__global__ void __launch_bounds__(256) linear_split_kernel(const __grid_constant__ CUtensorMap mW,
                                                           const __grid_constant__ CUtensorMap mX,
                                                           const LinearArgs a, int early, int chunk) {
  using C = SplitCfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ alignas(8) uint64_t full[C::kStages], empty[C::kStages], done;
  __shared__ uint32_t tmem_slot;
  __shared__ int s_err;
  __shared__ AdapterTiles<NT> s_tiles;
  uint8_t* sm = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cs = gridDim.x, rank = blockIdx.x;   // the cluster spans the grid's x
  const int n0 = blockIdx.y * kRows, t0 = blockIdx.z * NT;
  const int nk = (a.H + 63) / 64, k0 = (int)((long long)nk * rank / cs), k1 = (int)((long long)nk * (rank + 1) / cs);

  if (threadIdx.x == 0) {
    prefetch_map(&mW);
    prefetch_map(&mX);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&done, 1);
    s_err = MOE_OK;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&tmem_slot)),
                 "r"(C::kCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  // beside adapter_*_kernel (early) everything but u is there already: that
  // kernel lets this one start only once the work before it has completed
  if (!early) pdl_wait();
  pdl_launch_dependents();

  if (warp == 0) {
    if (elect_one()) {
      RingPos r(C::kStages);
      for (int k = k0; k < k1; ++k) {
        if (k - k0 >= C::kStages && !wait_bar(&empty[r.stage], r.parity ^ 1, &s_err)) break;
        uint8_t* st = sm + r.stage * C::kStage;
        mbar_expect_tx(&full[r.stage], C::kStage);
        tma_2d(st, &mW, k * 64, n0, &full[r.stage]);
        tma_2d(st + kATile, &mX, k * 64, t0, &full[r.stage]);
        r.next();
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      const uint32_t idesc = idesc_f16(NT, std::is_same<TE, __nv_bfloat16>::value);
      const uint64_t d0 = umma_desc_sw128(su32(sm));
      RingPos r(C::kStages);
      uint32_t d = tmem;
      int in = 0;   // K steps in the accumulator
      for (int k = k0; k < k1; ++k) {
        if (!wait_bar(&full[r.stage], r.parity, &s_err)) break;
        tc_fence_after();
        const uint64_t da = d0 + (uint32_t)(r.stage * C::kStage / 16), db = da + kATile / 16;
#pragma unroll
        for (int j = 0; j < 4; ++j) mma_k16(d, da + 2 * j, db + 2 * j, idesc, in || j);
        mma_commit(&empty[r.stage]);
        r.next();
        if (++in == chunk) in = 0, d += NT;
      }
      mma_commit(&done);
    }
  } else if (early) {   // the adapters' rows of this block's outputs, on their way to L2 meanwhile
    s_tiles.fill(a, threadIdx.x - 64, t0 + rank * (NT / cs), NT / cs);
    asm volatile("bar.sync 1, 192;" ::: "memory");
    for (int i = threadIdx.x - 64; i < s_tiles.tiles * kRows; i += 192) {
      const int j = i / kRows, n = n0 + i % kRows;
      const char* row = reinterpret_cast<const char*>(a.B) + ((long long)s_tiles.tile[j].y * a.N + n) * a.R * 2;
      if (n < a.N && (j == 0 || s_tiles.tile[j].y != s_tiles.tile[j - 1].y) && (uintptr_t)row % 128 < (unsigned)a.R * 2) prefetch_l2(row);
    }
  }
  __syncwarp();
  const bool ok = __all_sync(0xffffffffu, wait_bar(&done, 0, &s_err)) && *(volatile int*)&s_err == MOE_OK;
  tc_fence_after();
  // sums -> shared memory [NT][128]: a warp reads its quadrant's 32 rows, 16 tokens at a time
  float* part = reinterpret_cast<float*>(sm);
  const int q = warp & 3;
#pragma unroll
  for (int ch = warp >> 2; ch < NT / 16; ch += 2) {
    float f[16];
    for (int b = 0; b * chunk < k1 - k0; ++b) {   // the accumulators in order
      uint32_t v[16];
      tmem_ld16(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * NT + ch * 16), v);
#pragma unroll
      for (int j = 0; j < 16; ++j) f[j] = b ? f[j] + __uint_as_float(v[j]) : __uint_as_float(v[j]);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) part[(ch * 16 + j) * kRows + q * 32 + lane] = ok ? f[j] : NAN;
  }
  if (!ok) {   // a wait gave up: leave the copies in flight time to land
    const uint64_t since = gtimer();
    while (gtimer() - since < 2000000ull) {
    }
  }
  tc_fence_before();
  __syncwarp();
  if (cs > 1) cluster_sync();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kCols));
  }
  if (!ok && threadIdx.x == 0 && a.err) atomicExch(a.err, MOE_ERR_TIMEOUT);
  // the blocks' sums of this block's share of the tokens, four outputs at a time; with adapters they go
  // back to their place in this block's own sums (which no other block reads)
  const int share = NT / cs;
  const uint32_t base = su32(part);
  auto sum = [&] {
    for (int i = threadIdx.x; i < share * (kRows / 4); i += 256) {
      const int tt = rank * share + i / (kRows / 4), nn = i % (kRows / 4) * 4;
      if (t0 + tt >= a.T || n0 + nn >= a.N) continue;
      float* own = part + tt * kRows + nn;
      float v[4] = {};
      for (int r = 0; r < cs; ++r) {
        const float4 f = cs > 1 ? ld_cluster4(base + (uint32_t)(tt * kRows + nn) * 4, r) : *reinterpret_cast<const float4*>(own);
        v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
      }
      if (a.n) *reinterpret_cast<float4*>(own) = make_float4(v[0], v[1], v[2], v[3]);
      else store4<TE>(a, t0 + tt, n0 + nn, v);
    }
  };
  if (!a.n) sum();
  else {
    adapter_tiles<TE, NT>(a, s_tiles, t0 + rank * share, n0, part + rank * share * kRows, sm + NT * kRows * 4, [&] {
      if (cs > 1) sum();
    });
    __syncthreads();
    for (int i = threadIdx.x; i < share * (kRows / 4); i += 256) {
      const int tt = rank * share + i / (kRows / 4), nn = i % (kRows / 4) * 4;
      if (t0 + tt < a.T && n0 + nn < a.N) store4<TE>(a, t0 + tt, n0 + nn, part + tt * kRows + nn);
    }
  }
  __syncwarp();
  if (cs > 1) cluster_sync();   // the others have read this block's sums
}

// u of a large batch: a cluster takes 128 tokens and splits H like
// linear_split_kernel, the MMA's 128 rows being A rows: those of as many of the
// adapters that the tokens name as fit (128 / R; a prompt's tokens name one or
// two, more take another pass).  Every row meets every token; a token takes the
// rows of its own adapter, so nothing else's values reach it.  For fp32 results the
// share of H goes through four accumulators of kF32Chunk steps, added up in
// registers, as often as it takes.  Bound by reading x
// (from a cold cache 67 MB at 8192 x 4096, rank 16, fp32 results: 23 us; 33 MB at
// 4001, rank 32, 16-bit results: 17 us).
constexpr int kShrinkTokens = 128;
constexpr int kShrinkStage = kATile + kShrinkTokens * 128;
constexpr int kShrinkStages = 6;
constexpr int kShrinkSmem = kShrinkStages * kShrinkStage + 1024;
constexpr int kShrinkAcc = 512 / kShrinkTokens;   // accumulators for fp32 results

template <typename TE, bool F32>
__global__ void __launch_bounds__(256, 1) adapter_shrink_kernel(const __grid_constant__ CUtensorMap mA,
                                                             const __grid_constant__ CUtensorMap mX,
                                                             const LinearArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ alignas(8) uint64_t full[kShrinkStages], empty[kShrinkStages], done;
  __shared__ uint32_t tmem_slot;
  __shared__ int s_err, s_id[kShrinkTokens], s_slot[kShrinkTokens], s_list[kShrinkTokens];
  __shared__ uint32_t s_top[kShrinkTokens];   // fp16: the largest |u| of a token, as bits
  __shared__ int s_first[kShrinkTokens], s_count[kShrinkTokens / 32];
  uint8_t* sm = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cs = gridDim.x, rank = blockIdx.x, t0 = blockIdx.y * kShrinkTokens;
  constexpr int cols = (F32 ? kShrinkAcc : 1) * kShrinkTokens;
  const int nk = (a.H + 63) / 64, k0 = (int)((long long)nk * rank / cs), k1 = (int)((long long)nk * (rank + 1) / cs);
  if (tid == 0) {
    prefetch_map(&mA);
    prefetch_map(&mX);
    for (int s = 0; s < kShrinkStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&done, 1);
    s_err = MOE_OK;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&tmem_slot)),
                 "r"(cols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();   // after the wait: the projection may read x from its start
  // x's first stages are on their way while the list of adapters is made
  const int early = k1 - k0 < kShrinkStages ? k1 - k0 : kShrinkStages;
  if (tid == 0) {
    for (int i = 0; i < early; ++i) {
      mbar_expect_only(&full[i], kShrinkTokens * 128);
      tma_2d(sm + i * kShrinkStage + kATile, &mX, (k0 + i) * 64, t0, &full[i]);
    }
  }
  __syncwarp();
  // the adapters that the tokens name, in order of their first token: first of a warp's tokens ...
  int mine = -1;
  bool first = false;
  if (tid < kShrinkTokens) {
    mine = t0 + tid < a.T ? a.ids[t0 + tid] : -1;
    if (mine >= a.n) {
      if (a.err && rank == 0) atomicCAS(a.err, MOE_OK, MOE_ERR_INVALID);
      mine = -1;
    }
    s_id[tid] = mine;
    const uint32_t same = __match_any_sync(0xffffffffu, mine);
    first = mine >= 0 && (same & ((1u << lane) - 1)) == 0;
    const uint32_t firsts = __ballot_sync(0xffffffffu, first);
    if (first) s_first[warp * 32 + __popc(firsts & ((1u << lane) - 1))] = mine;
    if (lane == 0) s_count[warp] = __popc(firsts);
    s_top[tid] = 0;
  }
  __syncthreads();
  // ... and of the warps before it
  if (tid < kShrinkTokens) {
    for (int w = 0; w < warp; ++w)
      for (int i = 0; i < s_count[w]; ++i) first = first && s_first[w * 32 + i] != mine;
  }
  const int total = __syncthreads_count(first);
  const uint32_t firsts = __ballot_sync(0xffffffffu, first);
  if (tid < kShrinkTokens && lane == 0) s_count[warp] = __popc(firsts);
  __syncthreads();
  if (first) {
    int at = __popc(firsts & ((1u << lane) - 1));
    for (int w = 0; w < warp; ++w) at += s_count[w];
    s_list[at] = mine;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid < kShrinkTokens) {
    int slot = -1;
    for (int i = 0; i < total; ++i) slot = s_list[i] == mine ? i : slot;
    s_slot[tid] = slot;
  }
  const uint32_t tmem = tmem_slot;
  const int per = kRows / a.R;
  bool ok = true;
  RingPos r(kShrinkStages);
  bool wrapped = false;
  uint32_t turn = 0;
  float* part = reinterpret_cast<float*>(sm);   // [tokens][128]
  const int share = kShrinkTokens / cs;
  for (int p = 0; p < total; p += per) {
    const int cnt = total - p < per ? total - p : per;
    float f[kShrinkTokens / 32][16];   // a warp's 32 rows, every other 16 tokens
    for (int kb = k0, ke; kb < k1; kb = ke) {
      ke = F32 && kb + kShrinkAcc * kF32Chunk < k1 ? kb + kShrinkAcc * kF32Chunk : k1;
      if (warp == 0) {
        if (elect_one()) {
          for (int k = kb; k < ke; ++k) {
            if (wrapped && !wait_bar(&empty[r.stage], r.parity ^ 1, &s_err)) break;
            uint8_t* st = sm + r.stage * kShrinkStage;
            const bool have = p == 0 && k - k0 < early;
            mbar_expect_tx(&full[r.stage], cnt * a.R * 128 + (have ? 0 : kShrinkTokens * 128));
            for (int i = 0; i < cnt; ++i) tma_2d(st + i * a.R * 128, &mA, k * 64, s_list[p + i] * a.R, &full[r.stage]);
            if (!have) tma_2d(st + kATile, &mX, k * 64, t0, &full[r.stage]);
            r.next();
            wrapped |= r.stage == 0;
          }
        }
      } else if (warp == 1) {
        if (elect_one()) {
          const uint32_t idesc = idesc_f16(kShrinkTokens, std::is_same<TE, __nv_bfloat16>::value);
          const uint64_t d0 = umma_desc_sw128(su32(sm));
          uint32_t d = tmem;
          int in = 0;   // K steps in the accumulator
          for (int k = kb; k < ke; ++k) {
            if (!wait_bar(&full[r.stage], r.parity, &s_err)) break;
            tc_fence_after();
            const uint64_t da = d0 + (uint32_t)(r.stage * (kShrinkStage / 16)), db = da + kATile / 16;
#pragma unroll
            for (int j = 0; j < 4; ++j) mma_k16(d, da + 2 * j, db + 2 * j, idesc, in || j);
            mma_commit(&empty[r.stage]);
            r.next();
            if (++in == kF32Chunk && F32) in = 0, d += kShrinkTokens;
          }
          mma_commit(&done);
        }
      }
      __syncwarp();
      ok = __all_sync(0xffffffffu, wait_bar(&done, turn, &s_err)) && *(volatile int*)&s_err == MOE_OK;
      turn ^= 1;
      tc_fence_after();
#pragma unroll
      for (int i = 0; i < kShrinkTokens / 32; ++i) {
        const int ch = (warp >> 2) + 2 * i;
        for (int b = 0; b == 0 || (F32 && b * kF32Chunk < ke - kb); ++b) {   // the accumulators in order
          uint32_t v[16];
          tmem_ld16(tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)(b * kShrinkTokens + ch * 16), v);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            f[i][j] = F32 && (b || kb > k0) ? f[i][j] + __uint_as_float(v[j]) : __uint_as_float(v[j]);
        }
      }
      if (F32 && ke < k1) {   // the accumulators are free again
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
      }
    }
#pragma unroll
    for (int i = 0; i < kShrinkTokens / 32; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j)
        part[(((warp >> 2) + 2 * i) * 16 + j) * kRows + (warp & 3) * 32 + lane] = ok ? f[i][j] : NAN;
    tc_fence_before();
    __syncwarp();
    cluster_sync();
    tc_fence_after();
    const int rq = a.R / 4;
    for (int i = tid; i < share * rq; i += 256) {
      const int tt = rank * share + i / rq, c = i % rq, slot = s_slot[tt] - p;
      if (slot < 0 || slot >= cnt) continue;
      const uint32_t at = su32(part) + (uint32_t)(tt * kRows + slot * a.R + c * 4) * 4;
      float v[4] = {};
      for (int k = 0; k < cs; ++k) {
        const float4 f = ld_cluster4(at, k);
        v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
      }
      const float sc = a.scale ? a.scale[s_id[tt]] : 1.f;
      const long long o = (long long)(t0 + tt) * a.R + c * 4;
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] *= sc;
        const uint32_t bits = __float_as_uint(fabsf(v[j]));   // in the numbers' order, inf and NaN last
        top = top > bits ? top : bits;
      }
      if (!std::is_same<TE, __nv_bfloat16>::value && a.group) atomicMax(&s_top[tt], top);
      *reinterpret_cast<float4*>(a.u + o) = make_float4(v[0], v[1], v[2], v[3]);
      for (int k = 0; a.group && k < a.terms; ++k) {
        TE e[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) e[j] = from_f32<TE>(v[j]), v[j] -= to_f32(e[j]);
        *reinterpret_cast<uint2*>(reinterpret_cast<TE*>(a.u_terms) + (long long)k * a.T * a.R + o) =
            *reinterpret_cast<const uint2*>(e);
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the sums' place goes back to the copies
    __syncwarp();
    cluster_sync();   // the others have read this block's sums
  }
  if (total == 0 && tid == 0) {   // nothing to multiply: x's first stages still have to land
    for (int i = 0; i < early; ++i) mbar_arrive(&full[i]);
    for (int i = 0; i < early && ok; ++i) ok = wait_bar(&full[i], 0, &s_err);
  }
  __syncthreads();
  // how the projection takes a group: together where all 16 (a last group's missing tokens
  // aside) share an adapter and fp16's terms, which are not scaled there, carry u: two of them are
  // off by at most 2^-25 (half of fp16's smallest step), that is 2^-22 of a token's largest |u|
  // from 2^-3 on, and the first one holds less than 2^15.  A token of u = 0 has nothing to carry.
  if (a.group && tid < share / 16) {
    const int g = rank * (share / 16) + tid, base = g * 16;
    if (t0 + base < a.T) {
      int id = s_id[base];
      bool fits = true;
      for (int i = 0; i < 16 && t0 + base + i < a.T; ++i) {
        id = s_id[base + i] == s_id[base] ? id : kMixed;
        const uint32_t top = s_top[base + i];
        fits = fits && (top == 0 || (top >= 0x3e000000u && top < 0x47000000u));   // 2^-3, 2^15
      }
      if (!std::is_same<TE, __nv_bfloat16>::value && id >= 0 && !fits) id = kMixed;
      a.group[t0 / 16 + g] = id;
    }
  }
  if (!ok) {   // a wait gave up: leave the copies in flight time to land
    const uint64_t since = gtimer();
    while (gtimer() - since < 2000000ull) {
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols));
  }
  if (tid == 0 && s_err != MOE_OK && a.err) atomicExch(a.err, MOE_ERR_TIMEOUT);
}

// Large batches: persistent pairs of blocks (clusters of two, one block per SM)
// over tiles of 256 outputs x NT tokens (NT <= 256, a multiple of 16).  An SM takes
// in about 64 bytes a clock, and a block of its own needs (128 + NT) rows of a K
// step for 128 x NT of output: it waits for its operands (0.33 us a step at NT =
// 224 where the MMAs take 0.23).  A pair's MMA (cta_group::2) reads half of the
// tokens' rows from each block, so each brings 128 rows of W and NT / 2 of x.
//
// In each block warp 0 brings its rows by TMA into a ring, and eight warps empty
// its 128 rows of the accumulators: two of 256 columns, so a tile's epilogue runs
// under the next tile's steps.  Warp 1 of the first block (the leader) multiplies
// for both; its barriers take both blocks' copies and both epilogues' releases,
// and its commits arrive in both.  Without adapters 145 us at 8192 x 4096 x 4096
// (1.89 PFLOP/s; the library's product 139), 80 at 4001 x 4096 x 4096 (71), whose
// tiles fill 3.79 of four rounds.
//
// An fp32 result of more than kF32Chunk steps: the epilogue adds the chunks up in
// registers, in order (CHUNKS; tiles of at most 128 tokens).
//
// Adapters: tokens come in groups of 16.  A run of groups that share one adapter
// gets more K steps at the end of its tile, over that run's columns alone: B[a]
// times u's leading bits, B[a] times the next ones.  A group of several adapters, or
// whose u fp16's terms do not carry unscaled, is done in the epilogue (adapter_block),
// but with CHUNKS, whose accumulators leave it no registers: adapter_mixed_kernel
// then adds to the fp32 results.
constexpr int kStreamStages = 8;   // at most: as many as fit 208 KB
constexpr int kStreamBytes = 208 * 1024;
constexpr int kStreamSmem = kStreamBytes + 8 * 2048 + 1024;
static_assert(kStreamSmem + 512 <= 232448, "shared memory per block");
constexpr int kStreamThreads = 320;   // TMA, MMA, eight epilogue warps

struct StreamPlan {
  int nt, stages, tiles_n, tiles;   // tokens of a tile, stages of the ring, tiles of 256 outputs, all tiles
  int nk, chunk;                    // K steps, K steps of an accumulator
  int blocks;
};

template <typename TE, bool CHUNKS>
__global__ void __launch_bounds__(kStreamThreads, 1)
    linear_stream_kernel(const __grid_constant__ CUtensorMap mW, const __grid_constant__ CUtensorMap mX,
                         const __grid_constant__ CUtensorMap mB, const __grid_constant__ CUtensorMap mU,
                         const __grid_constant__ LinearArgs a, const StreamPlan pl) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ alignas(8) uint64_t full[kStreamStages], empty[kStreamStages], acc_full[2], acc_empty[2];
  __shared__ uint32_t tmem_slot;
  __shared__ int s_err;
  uint8_t* sm = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  float* turn = reinterpret_cast<float*>(sm + kStreamBytes);   // the epilogue's, 2 KB a warp
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = blockIdx.x & 1;   // clusters of two along x
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  if (threadIdx.x == 0) {
    prefetch_map(&mW);
    prefetch_map(&mX);
    for (int s = 0; s < kStreamStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 16);   // the leader's: eight warps of each block
    }
    s_err = MOE_OK;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&tmem_slot)),
                 "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync();   // the barriers of both are there
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  if (!a.n) pdl_wait();   // as in linear_split_kernel
  pdl_launch_dependents();
  const int groups = pl.nt / 16;
  const uint32_t bytes = kATile + pl.nt * 64;   // of a stage in each block
  const int rchunks = (a.R + 63) / 64;
  bool ok = true;

  // the runs of groups that share an adapter among a tile's (lane g holds group
  // g's entry, kMixed past T): f(adapter, first group, groups)
  auto group_of = [&](int t0) { return lane < groups && t0 + lane * 16 < a.T ? a.group[t0 / 16 + lane] : kMixed; };
  // u and the groups are waited for once, as late as the first tile allows; later tiles load their
  // groups before their K steps
  bool there = false;
  int mine = kMixed;
  auto groups_early = [&](int t0) {
    if (there) mine = group_of(t0);
  };
  auto groups_now = [&](int t0) {
    if (there) return;
    pdl_wait();
    there = true;
    mine = group_of(t0);
  };
  auto runs = [&](int mine, auto f) {
    uint32_t left = __ballot_sync(0xffffffffu, mine >= 0);
    while (left) {
      const int g = __ffs(left) - 1, id = __shfl_sync(0xffffffffu, mine, g);
      const uint32_t other = ~__ballot_sync(0xffffffffu, mine == id) & ~((1u << g) - 1);   // 16 groups at most
      const int len = __ffs(other) - 1 - g;
      if (!f(id, g, len)) return;
      left &= ~(((1u << len) - 1) << g);
    }
  };

  if (warp == 0) {
    RingPos r(pl.stages);
    bool wrapped = false;
    const bool lead = elect_one();
    auto stage = [&](const CUtensorMap* ma, const CUtensorMap* mb, int ka, int rowa, int rowb) {
      if (wrapped && !wait_bar(&empty[r.stage], r.parity ^ 1, &s_err)) return false;
      uint8_t* st = sm + r.stage * bytes;
      if (rank == 0) mbar_expect_tx(&full[r.stage], 2 * bytes);
      const uint32_t bar = cluster_addr(&full[r.stage], 0);
      tma_2d_pair(st, ma, ka, rowa, bar);
      tma_2d_pair(st + kATile, mb, ka, rowb, bar);
      r.next();
      wrapped |= r.stage == 0;
      return true;
    };
    for (int tile = pair; tile < pl.tiles && ok; tile += pairs) {
      const int n0 = (tile % pl.tiles_n * 2 + rank) * kRows, t0 = tile / pl.tiles_n * pl.nt;
      groups_early(t0);
      if (lead)
        for (int k = 0; k < pl.nk && ok; ++k) ok = stage(&mW, &mX, k * 64, n0, t0 + rank * (pl.nt / 2));
      ok = __all_sync(0xffffffffu, ok);
      if (!a.n || !ok) continue;
      groups_now(t0);
      runs(mine, [&](int id, int g, int len) {   // the run's first half here, its second in the other block
        const int t1 = t0 + g * 16 + rank * len * 8;
        if (lead)
          for (int c = 0; c < rchunks && ok; ++c)
            for (int k = 0; k < a.terms && ok; ++k) ok = stage(&mB, &mU, c * 64, id * a.N + n0, k * a.T + t1);
        return ok = __all_sync(0xffffffffu, ok);
      });
    }
  } else if (warp == 1 && rank == 0) {
    RingPos r(pl.stages);
    RingPos acc(2);
    int used = 0;   // accumulators handed over so far (up to 2)
    const bool bf16 = std::is_same<TE, __nv_bfloat16>::value, lead = elect_one();
    const uint32_t idesc = idesc_pair(pl.nt, bf16);
    const uint64_t d0 = umma_desc_sw128(su32(sm));
    for (int tile = pair; tile < pl.tiles && ok; tile += pairs) {
      const int t0 = tile / pl.tiles_n * pl.nt;
      groups_early(t0);
      for (int k = 0; k < pl.nk && ok; k += pl.chunk) {
        const uint32_t d = tmem + acc.stage * 256;
        const int end = k + pl.chunk < pl.nk ? k + pl.chunk : pl.nk;
        if (lead) {
          if (used >= 2) ok = wait_bar(&acc_empty[acc.stage], acc.parity ^ 1, &s_err);
          tc_fence_after();
          for (int i = k; i < end && ok; ++i) {
            if (!(ok = wait_bar(&full[r.stage], r.parity, &s_err))) break;
            tc_fence_after();
            const uint64_t da = d0 + r.stage * (bytes / 16), db = da + kATile / 16;
#pragma unroll
            for (int j = 0; j < 4; ++j) mma_k16_pair(d, da + 2 * j, db + 2 * j, idesc, i != k || j);
            mma_commit_pair(&empty[r.stage]);
            r.next();
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        if (a.n && end == pl.nk && ok) {
          groups_now(t0);
          runs(mine, [&](int id, int g, int len) {
            if (lead) {
              const uint32_t id16 = idesc_pair(len * 16, bf16);
              for (int c = 0; c < a.terms * rchunks; ++c) {
                if (!(ok = wait_bar(&full[r.stage], r.parity, &s_err))) break;
                tc_fence_after();
                const uint64_t da = d0 + r.stage * (bytes / 16), db = da + kATile / 16;
                const int left = a.R - (c / a.terms) * 64, steps = left >= 64 ? 4 : (left + 15) / 16;
                for (int j = 0; j < steps; ++j) mma_k16_pair(d + g * 16, da + 2 * j, db + 2 * j, id16, 1);
                mma_commit_pair(&empty[r.stage]);
                r.next();
              }
            }
            return ok = __all_sync(0xffffffffu, ok);
          });
        }
        if (lead && ok) mma_commit_pair(&acc_full[acc.stage]);
        acc.next();
        ++used;
      }
    }
  } else if (warp >= 2) {
    constexpr int kHalf = CHUNKS ? 64 : 128;                  // tokens of the tile that a warp takes
    const int q = warp & 3, c0 = ((warp - 2) >> 2) * kHalf;   // its 32 outputs, its first token
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    RingPos acc(2);
    for (int tile = pair; tile < pl.tiles && ok; tile += pairs) {
      const int n = (tile % pl.tiles_n * 2 + rank) * kRows + q * 32 + lane, t0 = tile / pl.tiles_n * pl.nt;
      float v[CHUNKS ? kHalf : 16];
      groups_early(t0);
      auto columns = [&](int c, float* f, bool add) {   // 16 of the accumulator's columns
        uint32_t w[16];
        tmem_ld16(tmem + lanes + acc.stage * 256 + c0 + c * 16, w);
#pragma unroll
        for (int j = 0; j < 16; ++j) f[j] = add ? f[j] + __uint_as_float(w[j]) : __uint_as_float(w[j]);
      };
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(cluster_addr(&acc_empty[acc.stage], 0));
        acc.next();
      };
      if (CHUNKS) {
        for (int k = 0; k < pl.nk; k += pl.chunk) {
          if (!(ok = __all_sync(0xffffffffu, wait_bar(&acc_full[acc.stage], acc.parity, &s_err)))) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < kHalf / 16; ++c)
            if (c0 + c * 16 < pl.nt) columns(c, v + c * 16, k != 0);
          release();
        }
      } else {
        ok = __all_sync(0xffffffffu, wait_bar(&acc_full[acc.stage], acc.parity, &s_err));
        tc_fence_after();
      }
      if (a.n && !CHUNKS) groups_now(t0);
      const uint32_t mixed =
          a.n && !CHUNKS ? __ballot_sync(0xffffffffu, lane < groups && t0 + lane * 16 < a.T && mine == kMixed) >> (c0 / 16) : 0;
#pragma unroll
      for (int c = 0; c < kHalf / 16; ++c) {
        const int t1 = t0 + c0 + c * 16;
        if (c0 + c * 16 >= pl.nt || t1 >= a.T) break;
        float* f = CHUNKS ? v + c * 16 : v;
        if (!CHUNKS) columns(c, f, false);
        if (!CHUNKS && (mixed >> c & 1)) {
          float* own = turn + (warp - 2) * 512;
          adapter_turn<TE>(a, t1, n - lane, own);
#pragma unroll
          for (int j = 0; j < 16; ++j) f[j] += own[j * 32 + lane];
        }
        if (n < a.N) {
          const long long o = (long long)t1 * a.ld_out + n;
          if (CHUNKS || a.out_dtype == MOE_DT_F32)
            store16(reinterpret_cast<float*>(a.out) + o, a.ld_out, a.T - t1, f, ok);
          else
            store16(reinterpret_cast<TE*>(a.out) + o, a.ld_out, a.T - t1, f, ok);
        }
        __syncwarp();
      }
      if (!CHUNKS) release();
    }
  }
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
  if (threadIdx.x == 0 && s_err != MOE_OK && a.err) atomicExch(a.err, MOE_ERR_TIMEOUT);
  if (a.n) pdl_wait();
}

// The mixed groups' adapters, added to fp32 results: a block per 16 tokens and 128
// outputs, which ends at once where the group is not a mixed one.  6.7 us by
// itself for 8192 tokens in 8 runs, a launch and a chain of reads (8.3 with the sums
// read at the end); in the projection's epilogue this code took the
// registers that it adds its chunks up in (25.9 us for 20.9 even without adapters).
template <typename TE>
__global__ void __launch_bounds__(256) adapter_mixed_kernel(const LinearArgs a) {
  __shared__ alignas(16) uint8_t room[SplitCfg<16>::kTerms];
  __shared__ alignas(16) float sums[16 * kRows];
  __shared__ AdapterTiles<16> s_tiles;
  pdl_wait();
  pdl_launch_dependents();
  if (a.group[blockIdx.x] != kMixed) return;
  const int t0 = blockIdx.x * 16, n0 = blockIdx.y * kRows;
  if (threadIdx.x < 192) s_tiles.fill(a, threadIdx.x, t0, 16);
  const int n = threadIdx.x % kRows;
  float* o = reinterpret_cast<float*>(a.out) + (long long)t0 * a.ld_out + n0 + n;
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int t = threadIdx.x / kRows + 2 * j;
    v[j] = t0 + t < a.T && n0 + n < a.N ? o[t * a.ld_out] : 0.f;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) sums[(threadIdx.x / kRows + 2 * j) * kRows + n] = v[j];
  __syncthreads();
  adapter_tiles<TE, 16>(a, s_tiles, t0, n0, sums, room, [] {});
  __syncthreads();
#pragma unroll
  for (int j = threadIdx.x / kRows; j < 16; j += 2)
    if (t0 + j < a.T && n0 + n < a.N) o[j * a.ld_out] = sums[j * kRows + n];
}

// --------------------------------------------------------------------- host --

// Blocks that split H, of a call of so many tiles: while the blocks still fit the SMs at once and each
// keeps two steps; clusters of eight only where one of the eight GPCs takes each (16 of them: 13.4 us for
// 64 tokens to 2048 outputs, of four 8.9).
static int split_cluster(long long tiles, int nk) {
  int cs = 1;
  while (cs < (tiles <= 8 ? 8 : 4) && tiles * cs * 2 <= device_sms() && nk >= 4 * cs) cs *= 2;
  return cs;
}

template <typename TE, int NT>
static moe_status launch_split(const LinearArgs& a, int dtype, cudaStream_t s) {
  using C = SplitCfg<NT>;
  CUtensorMap mW, mX;
  moe_status st = map_rows(&mW, a.W, dtype, a.H, a.N, a.ld_w, kRows);
  if (st == MOE_OK) st = map_rows(&mX, a.x, dtype, a.H, a.T, a.ld_x, NT);
  if (st != MOE_OK) return st;
  auto kernel = linear_split_kernel<TE, NT>;
  static char allowed[64];
  MOE_CUDA(allow_smem(kernel, C::kSmem, allowed));
  const int tiles_n = (a.N + kRows - 1) / kRows, tiles_t = (a.T + NT - 1) / NT, nk = (a.H + 63) / 64;
  MOE_ARG(tiles_n <= 65535 && tiles_t <= 65535, "T or N too large");
  const int cs = split_cluster((long long)tiles_n * tiles_t, nk);
  // K steps of an accumulator: all of a block's for 16-bit results, else 8 or what its accumulators ask for
  const int most = (nk + cs - 1) / cs, each = (most + C::kAcc - 1) / C::kAcc;
  const int chunk = a.out_dtype != MOE_DT_F32 ? most : each > kF32Chunk ? each : kF32Chunk;
  return launch_cluster(kernel, dim3(cs, tiles_n, tiles_t), 256, cs, C::kSmem, s, "linear_split_kernel", mW, mX, a,
                        a.n ? 1 : 0, chunk);
}

// `beside`: the projection's blocks, which take an SM each as this kernel's do.
template <typename TE>
static moe_status launch_shrink(const LinearArgs& a, int dtype, long long beside, cudaStream_t s) {
  CUtensorMap mA, mX;
  moe_status st = map_rows(&mA, a.A, dtype, a.H, (uint64_t)a.n * a.R, a.H, a.R);
  if (st == MOE_OK) st = map_rows(&mX, a.x, dtype, a.H, a.T, a.ld_x, kShrinkTokens);
  if (st != MOE_OK) return st;
  const bool f32 = a.out_dtype == MOE_DT_F32;
  auto kernel = f32 ? adapter_shrink_kernel<TE, true> : adapter_shrink_kernel<TE, false>;
  static char allowed[2][64];
  MOE_CUDA(allow_smem(kernel, kShrinkSmem, allowed[f32]));
  const int tiles = (a.T + kShrinkTokens - 1) / kShrinkTokens, nk = (a.H + 63) / 64;
  MOE_ARG(tiles <= 65535, "T too large");
  // as many blocks as leave the projection's room to run at the same time (1599 tokens to 378 outputs, H = 4744:
  // 25.4 us, one after the other 31.7), else, or with more than 24 steps a block (1786 to 256, H = 4096: 24.7 us
  // beside it, 21.8 after it), as many as there are SMs
  auto cluster = [&](long long room) {
    int cs = 1;
    while (cs < 8 && (long long)tiles * cs * 2 <= room && nk >= 4 * cs) cs *= 2;
    return cs;
  };
  const long long free = device_sms() - beside;
  int cs = cluster(free);
  if (tiles > free || nk > 24 * cs) cs = cluster(device_sms());
  return launch_cluster(kernel, dim3(cs, tiles), 256, cs, kShrinkSmem, s, "adapter_shrink_kernel", mA, mX, a);
}

// Whether a call goes to the persistent pairs: once its tiles of 128 x 128 are
// more than the SMs (H = 4096, 192 tiles: 34.5 us split, 22.8 streamed; 128 tiles:
// 17.9 and 22.5, with adapters of rank 16 27.6 and 37.1, of mixed ones 27.5 and
// 50.7).  fp32 results from three quarters of the SMs on: the split kernel has
// accumulators for 512 products each only up to H = 2048 a block.
static bool large_batch(int T, int N, bool f32) {
  const long long tiles = ((long long)N + kRows - 1) / kRows * ((T + 127) / 128);
  return T > 128 && tiles * (f32 ? 4 : 3) >= device_sms() * 3LL + (f32 ? 0 : 1);
}

static StreamPlan stream_plan(const LinearArgs& a) {
  StreamPlan pl;
  pl.tiles_n = (a.N + 2 * kRows - 1) / (2 * kRows);
  pl.nk = (a.H + 63) / 64;
  const bool chunks = a.out_dtype == MOE_DT_F32 && pl.nk > kF32Chunk;
  pl.chunk = chunks ? kF32Chunk : pl.nk;
  // the tile that takes the least time: rounds of the pairs times a step's rows into an SM (128 of W and
  // NT / 2 of x, in units of half a row); among equals the one that leaves fewest pairs idle
  const int pairs = device_sms() / 2;
  long long best = -1;
  for (int nt = chunks ? 128 : 256; nt >= 64; nt -= 16) {
    const long long tiles = (long long)pl.tiles_n * ((a.T + nt - 1) / nt), cost = (tiles + pairs - 1) / pairs * (nt + 256);
    if (best < 0 || cost < best) best = cost, pl.nt = nt, pl.tiles = (int)tiles;
  }
  const int fit = kStreamBytes / (kATile + pl.nt * 64);
  pl.stages = fit < kStreamStages ? fit : kStreamStages;
  pl.blocks = 2 * (pl.tiles < pairs ? pl.tiles : pairs);
  return pl;
}

template <typename TE>
static moe_status launch_stream(const LinearArgs& a, const StreamPlan& pl, int dtype, cudaStream_t s) {
  CUtensorMap mW, mX, mB = {}, mU = {};
  const bool chunks = pl.chunk < pl.nk;
  moe_status st = map_rows(&mW, a.W, dtype, a.H, a.N, a.ld_w, kRows);
  if (st == MOE_OK) st = map_rows(&mX, a.x, dtype, a.H, a.T, a.ld_x, pl.nt / 2);
  if (a.n) {
    if (st == MOE_OK) st = map_rows(&mB, a.B, dtype, a.R, (uint64_t)a.n * a.N, a.R, kRows);
    if (st == MOE_OK) st = map_rows(&mU, a.u_terms, dtype, a.R, (uint64_t)a.terms * a.T, a.R, pl.nt / 2);
  }
  if (st != MOE_OK) return st;
  auto kernel = chunks ? linear_stream_kernel<TE, true> : linear_stream_kernel<TE, false>;
  static char allowed[2][64];
  MOE_CUDA(allow_smem(kernel, kStreamSmem, allowed[chunks]));
  st = launch_cluster(kernel, dim3(pl.blocks), kStreamThreads, 2, kStreamSmem, s,
                      "linear_stream_kernel", mW, mX, mB, mU, a, pl);
  if (st != MOE_OK || !chunks || !a.n) return st;
  MOE_ARG((a.N + kRows - 1) / kRows <= 65535, "N too large");
  cudaError_t e = launch_pdl(adapter_mixed_kernel<TE>, dim3((a.T + 15) / 16, (a.N + kRows - 1) / kRows), dim3(256), 0, s, a);
  if (e != cudaSuccess) return cuda_fail(e, "adapter_mixed_kernel");
  return check_launch("adapter_mixed_kernel");
}

template <typename TE>
static moe_status launch_linear(const LinearArgs& a, int dtype, cudaStream_t s) {
  ProfScope ps(MOE_K_LINEAR, s);
  moe_status st = MOE_OK;
  const bool large = large_batch(a.T, a.N, a.out_dtype == MOE_DT_F32);
  StreamPlan pl = {};
  if (large) pl = stream_plan(a);
  if (a.n) {
    // a dot per token and rank reads A again for every token, the tcgen05 kernel x again for every 128 / R
    // adapters among 128 tokens (which only the device knows): dots for a batch that may name many
    if (!large && (a.T <= 256 || (long long)a.T * a.R * a.H * 2 <= (64LL << 20))) {
      cudaError_t e = launch_pdl(adapter_dot_kernel<TE>, dim3(a.T, a.R / kDots), dim3(128), 0, s, a);
      if (e != cudaSuccess) return cuda_fail(e, "adapter_dot_kernel");
      st = check_launch("adapter_dot_kernel");
    } else {
      const long long tiles = (a.N + kRows - 1LL) / kRows * ((a.T + 127LL) / 128);
      st = launch_shrink<TE>(a, dtype, large ? pl.blocks : tiles * split_cluster(tiles, (a.H + 63) / 64), s);
    }
    if (st != MOE_OK) return st;
  }
  if (large) return launch_stream<TE>(a, pl, dtype, s);
  if (a.T <= 16) return launch_split<TE, 16>(a, dtype, s);
  if (a.T <= 32) return launch_split<TE, 32>(a, dtype, s);
  if (a.T <= 64) return launch_split<TE, 64>(a, dtype, s);
  return launch_split<TE, 128>(a, dtype, s);
}

// The workspace's parts: u, and for large batches u's 16-bit terms (room for three) and the groups' table.
struct LinearSpace {
  size_t u, terms, group, bytes;
};
static LinearSpace linear_space(int T, int N, int n, int R) {
  LinearSpace w = {};
  if (n <= 0) return w;
  auto take = [&](size_t b) {
    const size_t at = w.bytes;
    w.bytes += (b + 127) / 128 * 128;
    return at;
  };
  w.u = take((size_t)T * R * 4);
  if (large_batch(T, N, true)) {
    w.terms = take((size_t)T * R * 2 * 3);
    w.group = take(((size_t)T + 15) / 16 * 4);
  }
  return w;
}

}  // namespace moe

using namespace moe;

extern "C" size_t moe_adapter_linear_workspace(int T, int H, int N, int n_adapters, int R) {
  if (T <= 0 || H <= 0 || N <= 0 || n_adapters <= 0 || R <= 0) return 0;
  return linear_space(T, N, n_adapters, R).bytes;
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
  MOE_ARG((long long)n_adapters * N + 2 * kRows <= 0x7fffffffLL && (long long)n_adapters * R <= 0x7fffffffLL,
          "n_adapters * N and n_adapters * R must be below 2^31");
  MOE_ARG(T <= 1 << 29, "T must be at most 2^29 (got %d)", T);
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
  const LinearSpace w = linear_space(T, N, n_adapters, R);
  char* ws = (char*)workspace;
  LinearArgs a = {};
  a.T = T, a.H = H, a.N = N, a.n = n_adapters, a.R = R, a.out_dtype = out_dtype;
  a.x = x, a.W = W, a.A = lora_a, a.B = lora_b, a.ld_x = ld_x, a.ld_w = ld_w, a.ld_out = ld_out;
  a.ids = adapter_ids, a.scale = lora_scale, a.out = out, a.err = d_error;
  if (n_adapters) {
    a.u = (float*)(ws + w.u);
    if (large_batch(T, N, out_dtype == MOE_DT_F32)) a.u_terms = ws + w.terms, a.group = (int32_t*)(ws + w.group);
    a.terms = dtype == MOE_DT_BF16 && out_dtype == MOE_DT_F32 ? 3 : 2;
  }
  return dtype == MOE_DT_BF16 ? launch_linear<__nv_bfloat16>(a, dtype, stream)
                              : launch_linear<__half>(a, dtype, stream);
}
