// Tokens sorted by expert and back: the rows that grouped products read, the
// weighted sum of their results, and the gradients of both.
//
//   sort       pos[t, j] = the place of pair (t, j) among the pairs stably sorted by
//              expert, rows[pos[t, j]] = x[t]
//   combine    y[t] = base[t] + sum_j w[t, j] rows[pos[t, j]]; with neither weights
//              nor base the gradient of sort
//   combine'   d_rows[pos[t, j]] = w[t, j] d_y[t], d_w[t, j] = <d_y[t], rows[pos[t, j]]>
//
// All of them go by tokens, so a token's row is read (or written) once and its k rows
// once each: the bytes that the operator cannot do without.
#include <type_traits>

#include "dtype.cuh"

namespace moe {

constexpr int kMaxK = 64, kMaxE = 2048;

// ------------------------------------------------------------------- vectors --

template <int BYTES>
struct Bytes;
template <>
struct Bytes<16> {
  using T = uint4;
};
template <>
struct Bytes<8> {
  using T = uint2;
};
template <>
struct Bytes<4> {
  using T = uint32_t;
};
template <>
struct Bytes<2> {
  using T = uint16_t;
};

// V neighbouring elements of T, as they lie in memory (fp32: pieces of at most 16 bytes): loaded
// first and converted later, so that many loads are under way in few registers.
template <typename T, int V>
struct Vec {
  static constexpr int B = V * (int)sizeof(T), P = B > 16 ? 16 : B, E = P / (int)sizeof(T), N = V / E;
  using W = typename Bytes<P>::T;
  W w[N];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = reinterpret_cast<const W*>(p)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < N; ++i) reinterpret_cast<W*>(p)[i] = w[i];
  }
  __device__ __forceinline__ void get(float (&f)[V]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      T e[E];
      memcpy(e, &w[i], P);
#pragma unroll
      for (int j = 0; j < E; ++j) f[i * E + j] = to_f32(e[j]);
    }
  }
  __device__ __forceinline__ void set(const float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      T e[E];
#pragma unroll
      for (int j = 0; j < E; ++j) e[j] = from_f32<T>(f[i * E + j]);
      memcpy(&w[i], e, P);
    }
  }
};

// ---------------------------------------------------------------------- plan --

// The stable sort, by one cluster: block r takes an eighth of the pairs in order, each
// of its warps a run of them.  Counts by warp and expert in shared memory become, by
// sums over the warps before, the blocks before (read from their shared memory) and
// the experts before, the place of each run's first pair of an expert; then each warp
// places its pairs 32 at a time, the lanes that share an expert in order.
constexpr int kPlanBlocks = 8;
static int plan_warps(int E) { return E <= 1024 ? 32 : 16; }   // counts of 128 KB at most

__device__ __forceinline__ void plan_cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int ld_block(const int* p, uint32_t rank) {   // another block's shared memory
  uint32_t a;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(su32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

__global__ void __launch_bounds__(1024, 1) __cluster_dims__(kPlanBlocks, 1, 1)
    sort_plan_kernel(const int32_t* ids, int P, int E, int32_t* offsets, int32_t* pos, int32_t* err) {
  extern __shared__ __align__(16) uint8_t plan_smem[];
  __shared__ int ws[34];
  int* total = reinterpret_cast<int*>(plan_smem);   // [E]: of this block, read by the others
  int* base = total + E;                            // [E]
  int* cnt = base + E;                              // [warps][E]
  const int tid = threadIdx.x, NT = blockDim.x, warps = NT >> 5, warp = tid >> 5, lane = tid & 31;
  const int r = blockIdx.x;
  for (int i = tid; i < warps * E; i += NT) cnt[i] = 0;
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  // runs of whole steps of 32 pairs
  const long long steps = ((long long)P + 31) / 32, all = (long long)kPlanBlocks * warps, me = (long long)r * warps + warp;
  const long long s0 = steps * me / all, s1 = steps * (me + 1) / all;
  int* mine = cnt + warp * E;
  bool bad = false;
#pragma unroll 4
  for (long long s = s0; s < s1; ++s) {
    const long long p = s * 32 + lane;
    const int e = p < P ? ids[p] : -1;
    bad |= e >= E;
    if (e >= 0 && e < E) atomicAdd(&mine[e], 1);
  }
  if (bad && err) atomicExch(err, MOE_ERR_INVALID);
  __syncthreads();
  for (int e = tid; e < E; e += NT) {
    int t = 0;
    for (int w = 0; w < warps; ++w) {
      const int c = cnt[w * E + e];
      cnt[w * E + e] = t;
      t += c;
    }
    total[e] = t;
  }
  plan_cluster_sync();
  // experts in order, a run of neighbours to a thread
  const int per = (E + NT - 1) / NT, e0 = min(E, tid * per), e1 = min(E, e0 + per);
  int sum = 0;
  for (int e = e0; e < e1; ++e) {
    int before = 0, here = 0;
#pragma unroll
    for (int b = 0; b < kPlanBlocks; ++b) {
      const int c = ld_block(&total[e], b);
      before += b < r ? c : 0;
      here += c;
    }
    base[e] = sum + before;   // the pairs of the thread's earlier experts, of this one in earlier blocks
    sum += here;
  }
  int pairs;
  const int first = block_exclusive_scan(sum, ws, &pairs);
  int run = first;
  for (int e = e0; e < e1; ++e) {
    base[e] += first;
    if (r == 0) {
      int here = 0;
#pragma unroll
      for (int b = 0; b < kPlanBlocks; ++b) here += ld_block(&total[e], b);
      offsets[e] = run;
      run += here;
    }
  }
  if (r == 0 && tid == 0) offsets[E] = pairs;
  plan_cluster_sync();   // no block leaves while another reads its counts; base is complete
  for (long long s = s0; s < s1; ++s) {
    const long long p = s * 32 + lane;
    const int e = p < P ? ids[p] : -1;
    const bool in = e >= 0 && e < E;
    const unsigned peers = __match_any_sync(0xffffffffu, in ? e : -1);
    const int rank = __popc(peers & ((1u << lane) - 1));
    int at = -1;
    if (in) at = base[e] + mine[e] + rank;
    __syncwarp();
    if (in && rank == 0) mine[e] += __popc(peers);
    __syncwarp();
    if (p < P) pos[p] = at;
  }
}

// ---------------------------------------------------------------------- sort --

struct SortArgs {
  int T, k, nv;              // nv: vectors of a row
  const uint8_t* x;
  uint8_t* rows;
  long long ld_x, ld_rows;   // bytes
  const int32_t* pos;
};

// Neighbouring vectors of x's rows to a block, whatever their tokens: read once, written to
// the token's k rows.
constexpr int kItems = 2;   // vectors of a thread
template <int VB>
__global__ void __launch_bounds__(256) sort_rows_kernel(const SortArgs a) {
  using W = typename Bytes<VB>::T;
  pdl_wait();
  pdl_launch_dependents();
  const long long i0 = (long long)blockIdx.x * (256 * kItems);
  const long long t0 = i0 / a.nv;
  const int v0 = (int)(i0 - t0 * a.nv);
  W w[kItems];
  long long t[kItems];
  int v[kItems];
#pragma unroll
  for (int u = 0; u < kItems; ++u) {
    const unsigned at = (unsigned)v0 + u * 256 + threadIdx.x;
    const unsigned q = at / (unsigned)a.nv;
    t[u] = t0 + q, v[u] = (int)(at - q * a.nv);
    if (t[u] < a.T) w[u] = reinterpret_cast<const W*>(a.x + t[u] * a.ld_x)[v[u]];
  }
#pragma unroll
  for (int u = 0; u < kItems; ++u) {
    if (t[u] >= a.T) break;
    const int32_t* pos = a.pos + t[u] * a.k;
#pragma unroll 4
    for (int j = 0; j < a.k; ++j) {
      const int p = pos[j];
      if (p >= 0) reinterpret_cast<W*>(a.rows + p * a.ld_rows)[v[u]] = w[u];
    }
  }
}

// Few pairs: one launch, each block placing the pairs of its own tokens by counting, a warp to a pair,
// the pairs that come before it; the last block writes the offsets.  Latency: a launch and a
// round trip to memory more than the copy.
constexpr int kSmallPairs = 1024;
struct SmallSortArgs {
  SortArgs s;
  int E;
  const int32_t* ids;
  int32_t *offsets, *pos, *err;
};
template <int VB>
__global__ void __launch_bounds__(256) sort_small_kernel(const SmallSortArgs a) {
  using W = typename Bytes<VB>::T;
  __shared__ alignas(16) int ids[kSmallPairs];
  __shared__ int place[kSmallPairs], cnt[kMaxE], ws[34];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, k = a.s.k, P = a.s.T * k;
  pdl_wait();
  pdl_launch_dependents();
  const bool last = blockIdx.x == gridDim.x - 1;
  const long long i0 = (long long)blockIdx.x * (256 * kItems);
  const int t0 = last ? 0 : (int)(i0 / a.s.nv), v0 = (int)(i0 - (long long)t0 * a.s.nv);
  W w[kItems];
  int t[kItems], v[kItems];
#pragma unroll
  for (int u = 0; u < kItems; ++u) {
    const unsigned at = (unsigned)v0 + u * 256 + tid, q = at / (unsigned)a.s.nv;
    t[u] = last ? a.s.T : t0 + (int)min(q, (unsigned)a.s.T), v[u] = (int)(at - q * a.s.nv);
    if (t[u] < a.s.T) w[u] = reinterpret_cast<const W*>(a.s.x + t[u] * a.s.ld_x)[v[u]];
  }
  bool bad = false;
  for (int p = tid; p < kSmallPairs; p += 256) {
    int e = p < P ? a.ids[p] : -1;
    bad |= e >= a.E;
    ids[p] = e >= 0 && e < a.E ? e : kMaxE;   // without an expert: after all others
  }
  if (last) {
    if (bad && a.err) atomicExch(a.err, MOE_ERR_INVALID);
    for (int e = tid; e < a.E; e += 256) cnt[e] = 0;
  }
  __syncthreads();
  if (last) {
    for (int p = tid; p < P; p += 256)
      if (ids[p] < kMaxE) atomicAdd(&cnt[ids[p]], 1);
    __syncthreads();
    const int per = (a.E + 255) / 256, e0 = min(a.E, tid * per), e1 = min(a.E, e0 + per);
    int sum = 0, all;
    for (int e = e0; e < e1; ++e) sum += cnt[e];
    int run = block_exclusive_scan(sum, ws, &all);
    for (int e = e0; e < e1; ++e) {
      a.offsets[e] = run;
      run += cnt[e];
    }
    if (tid == 0) a.offsets[a.E] = all;
    return;
  }
  const int t1 = (int)min((long long)a.s.T - 1, (i0 + 256 * kItems - 1) / a.s.nv), p0 = t0 * k, n = (t1 - t0 + 1) * k;
  for (int i = warp; i < n; i += 8) {
    const int p = p0 + i, e = ids[p];
    int before = 0;
    for (int q = lane * 4; q < P; q += 128) {   // past the pairs: kMaxE
      const int4 o = *reinterpret_cast<const int4*>(ids + q);
      before += (o.x < e || (o.x == e && q < p)) + (o.y < e || (o.y == e && q + 1 < p)) +
                (o.z < e || (o.z == e && q + 2 < p)) + (o.w < e || (o.w == e && q + 3 < p));
    }
    before = __reduce_add_sync(0xffffffffu, before);
    if (lane == 0) {
      place[i] = e < kMaxE ? before : -1;
      if (v0 == 0 || i >= k) a.pos[p] = place[i];   // a token's first vector is this block's
    }
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kItems; ++u) {
    if (t[u] >= a.s.T) break;
    const int* mine = place + (t[u] - t0) * k;
#pragma unroll 4
    for (int j = 0; j < k; ++j) {
      const int p = mine[j];
      if (p >= 0) reinterpret_cast<W*>(a.s.rows + p * a.s.ld_rows)[v[u]] = w[u];
    }
  }
}

// ------------------------------------------------------------------- combine --

struct CombineArgs {
  int T, k, nv, n_rows;
  const void *rows, *base;
  void* y;
  long long ld_rows, ld_base, ld_y;   // elements
  const int32_t* pos;
  const float* w;
};

template <typename TR, typename TY, int V>
__global__ void __launch_bounds__(256) combine_rows_kernel(const CombineArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const long long i0 = (long long)blockIdx.x * 256;
  const long long t0 = i0 / a.nv;
  const unsigned at = (unsigned)(i0 - t0 * a.nv) + threadIdx.x, q = at / (unsigned)a.nv;
  const long long t = t0 + q;
  const long long c = (long long)(at - q * a.nv) * V;
  if (t >= a.T) return;
  const TR* rows = reinterpret_cast<const TR*>(a.rows) + c;
  const int32_t* pos = a.pos + t * a.k;
  const float* w = a.w ? a.w + t * a.k : nullptr;
  Vec<TY, V> base;
  if (a.base) base.load(reinterpret_cast<const TY*>(a.base) + t * a.ld_base + c);
  float s[V] = {};
#pragma unroll 1
  for (int j0 = 0; j0 < a.k; j0 += 8) {
    Vec<TR, V> r[8];
    float by[8];
    int p[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      p[j] = j0 + j < a.k ? pos[j0 + j] : -1;
      by[j] = j0 + j < a.k && w ? w[j0 + j] : 1.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (p[j] >= a.n_rows) p[j] = -1;
      if (p[j] >= 0) r[j].load(rows + p[j] * a.ld_rows);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float f[V];
      r[j].get(f);
      if (p[j] >= 0)
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = fmaf(by[j], f[i], s[i]);
    }
  }
  if (a.base) {
    float b[V];
    base.get(b);
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] += b[i];
  }
  Vec<TY, V> y;
  y.set(s);
  y.store(reinterpret_cast<TY*>(a.y) + t * a.ld_y + c);
}

// ---------------------------------------------------------- combine, backward --

struct CombineBwdArgs {
  int T, k, nv, n_rows;
  const void *dy, *rows;
  void* d_rows;
  long long ld_dy, ld_rows, ld_d_rows;   // elements
  const int32_t* pos;
  const float* w;
  float* dw;
};

// Eight sums over a warp, halving: lane l comes out with sum l >> 2 (a lane's eight values are dealt out, four
// to each half, then two, then one, 9 exchanges for 40).
__device__ __forceinline__ float sum8(float (&s)[8]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 4; n > 0; n >>= 1) {
    const bool up = lane & (n * 4);
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const float send = up ? s[j] : s[j + n], keep = up ? s[j + n] : s[j];
      s[j] = keep + __shfl_xor_sync(0xffffffffu, send, n * 4);
    }
  }
  float v = s[0];
  v += __shfl_xor_sync(0xffffffffu, v, 2);
  return v + __shfl_xor_sync(0xffffffffu, v, 1);
}

// G threads to a token; its k products go eight at a time, each thread holding the eight
// sums over its own columns.
template <typename TR, typename TY, int V, int G>
__global__ void __launch_bounds__(256) combine_bwd_kernel(const CombineBwdArgs a) {
  __shared__ float part[8][8];   // [warp][pair]
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, me = tid % G;
  const long long t = (long long)blockIdx.x * (256 / G) + tid / G;
  const bool there = t < a.T;
  const TY* dy = reinterpret_cast<const TY*>(a.dy) + t * a.ld_dy;
  const TR* rows = reinterpret_cast<const TR*>(a.rows);
  TR* d_rows = reinterpret_cast<TR*>(a.d_rows);
#pragma unroll 1
  for (int j0 = 0; j0 < a.k; j0 += 8) {
    int p[8];
    float by[8], s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      p[j] = there && j0 + j < a.k ? a.pos[t * a.k + j0 + j] : -1;
      by[j] = there && j0 + j < a.k && a.w ? a.w[t * a.k + j0 + j] : 1.f;
      s[j] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (p[j] >= a.n_rows) p[j] = -1;
    if (there)
      for (int v = me; v < a.nv; v += G) {
        Vec<TY, V> dv;
        Vec<TR, V> r[8];
        const long long c = (long long)v * V;
        dv.load(dy + c);
        if (a.dw)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (p[j] >= 0) r[j].load(rows + p[j] * a.ld_rows + c);
        float d[V];
        dv.get(d);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (p[j] < 0) continue;
          if (a.dw) {
            float f[V];
            r[j].get(f);
#pragma unroll
            for (int i = 0; i < V; ++i) s[j] = fmaf(d[i], f[i], s[j]);
          }
          float o[V];
#pragma unroll
          for (int i = 0; i < V; ++i) o[i] = by[j] * d[i];
          r[j].set(o);
          r[j].store(d_rows + p[j] * a.ld_d_rows + c);
        }
      }
    if (!a.dw) continue;
    const float mine = sum8(s);
    const int j = lane >> 2;
    if (G == 32) {
      if (there && (lane & 3) == 0 && j0 + j < a.k) a.dw[t * a.k + j0 + j] = mine;
    } else {
      __syncthreads();
      if ((lane & 3) == 0) part[warp][j] = mine;
      __syncthreads();
      if (there && me < 8 && j0 + me < a.k) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < G / 32; ++w) v += part[tid / G * (G / 32) + w][me];
        a.dw[t * a.k + j0 + me] = v;
      }
    }
  }
}

// ---------------------------------------------------------------------- host --

// Whether rows of `width` bytes, `ld` bytes apart, split into vectors of `v` bytes.
static bool splits(const void* p, long long ld, long long width, int v) {
  return ((uintptr_t)p | (uintptr_t)ld | (uintptr_t)width) % v == 0;
}

template <typename K, typename A>
static moe_status launch_rows(K kernel, long long blocks, cudaStream_t s, const char* name, const A& a) {
  MOE_ARG(blocks <= 0x7fffffffLL, "too many elements");
  cudaError_t e = launch_pdl(kernel, dim3((unsigned)blocks), dim3(256), 0, s, a);
  if (e != cudaSuccess) return cuda_fail(e, name);
  return check_launch(name);
}

template <typename TR, typename TY>
static moe_status launch_combine(CombineArgs a, int H, cudaStream_t s) {
  auto fits = [&](int v) {
    return splits(a.rows, a.ld_rows * (int)sizeof(TR), (long long)H * sizeof(TR), v * sizeof(TR) < 16 ? v * (int)sizeof(TR) : 16) &&
           splits(a.y, a.ld_y * (int)sizeof(TY), (long long)H * sizeof(TY), v * sizeof(TY) < 16 ? v * (int)sizeof(TY) : 16) &&
           (!a.base || splits(a.base, a.ld_base * (int)sizeof(TY), 0, v * sizeof(TY) < 16 ? v * (int)sizeof(TY) : 16));
  };
  const int v = H % 8 == 0 && fits(8) ? 8 : H % 2 == 0 && fits(2) ? 2 : 1;
  a.nv = H / v;
  const long long blocks = ((long long)a.T * a.nv + 255) / 256;
  const char* name = "combine_rows_kernel";
  if (v == 8) return launch_rows(combine_rows_kernel<TR, TY, 8>, blocks, s, name, a);
  if (v == 2) return launch_rows(combine_rows_kernel<TR, TY, 2>, blocks, s, name, a);
  return launch_rows(combine_rows_kernel<TR, TY, 1>, blocks, s, name, a);
}

template <typename TR, typename TY, int V>
static moe_status launch_bwd_v(CombineBwdArgs a, int H, cudaStream_t s) {
  a.nv = H / V;
  const char* name = "combine_bwd_kernel";
  auto blocks = [&](int G) { return ((long long)a.T + 256 / G - 1) / (256 / G); };
  if (a.nv <= 128) return launch_rows(combine_bwd_kernel<TR, TY, V, 32>, blocks(32), s, name, a);
  if (a.nv <= 512) return launch_rows(combine_bwd_kernel<TR, TY, V, 128>, blocks(128), s, name, a);
  return launch_rows(combine_bwd_kernel<TR, TY, V, 256>, blocks(256), s, name, a);
}
template <typename TR, typename TY>
static moe_status launch_bwd(const CombineBwdArgs& a, int H, cudaStream_t s) {
  auto fits = [&](int v) {
    const int r = v * sizeof(TR) < 16 ? v * (int)sizeof(TR) : 16, y = v * sizeof(TY) < 16 ? v * (int)sizeof(TY) : 16;
    return splits(a.d_rows, a.ld_d_rows * (int)sizeof(TR), 0, r) && splits(a.dy, a.ld_dy * (int)sizeof(TY), 0, y) &&
           (!a.dw || splits(a.rows, a.ld_rows * (int)sizeof(TR), 0, r));
  };
  if (H % 8 == 0 && fits(8)) return launch_bwd_v<TR, TY, 8>(a, H, s);
  if (H % 2 == 0 && fits(2)) return launch_bwd_v<TR, TY, 2>(a, H, s);
  return launch_bwd_v<TR, TY, 1>(a, H, s);
}

// f(element of the rows, element of the tokens) for the types of a call.
template <typename F>
static moe_status by_types(int rows, int y, F f) {
  if (rows == MOE_DT_F32) {
    if (y == MOE_DT_F32) return f(0.f, 0.f);
    if (y == MOE_DT_BF16) return f(0.f, __nv_bfloat16());
    return f(0.f, __half());
  }
  if (rows == MOE_DT_BF16) return f(__nv_bfloat16(), __nv_bfloat16());
  return f(__half(), __half());
}

static moe_status check_pairs(int T, int k, int H) {
  MOE_ARG(T >= 0, "T must be >= 0 (got %d)", T);
  MOE_ARG(k >= 1 && k <= kMaxK, "k must be in [1, %d] (got %d)", kMaxK, k);
  MOE_ARG(H >= 1, "H must be >= 1 (got %d)", H);
  MOE_ARG((long long)T * k < (1LL << 31) - 32, "too many pairs (%d x %d)", T, k);
  return MOE_OK;
}
static moe_status check_types(int rows, int y) {
  MOE_ARG(known_dtype(rows) && known_dtype(y), "unknown element type (%d, %d)", rows, y);
  MOE_ARG(rows == y || rows == MOE_DT_F32, "rows must be of the tokens' type or fp32 (types %d, %d)", rows, y);
  return MOE_OK;
}

static moe_status combine(int T, int k, int n_rows, int H, int rows_dtype, int y_dtype, const void* rows, int64_t ld_rows,
                          const int32_t* pos, const float* w, const void* base, int64_t ld_base, void* y, int64_t ld_y,
                          int kernel, cudaStream_t stream) {
  moe_status st = check_pairs(T, k, H);
  if (st == MOE_OK) st = check_types(rows_dtype, y_dtype);
  if (st != MOE_OK) return st;
  MOE_ARG(n_rows >= 0, "n_rows must be >= 0 (got %d)", n_rows);
  if (T == 0) return MOE_OK;
  MOE_ARG((rows || n_rows == 0) && pos && y, "null pointer");
  MOE_ARG(ld_rows >= H && ld_y >= H && (!base || ld_base >= H), "a row distance is below the row's length");
  MOE_ARG(base != y || ld_base == ld_y, "in place, base and y need the same row distance");
  ProfScope ps(kernel, stream);
  CombineArgs a = {T, k, 0, n_rows, rows, base, y, ld_rows, ld_base, ld_y, pos, w};
  return by_types(rows_dtype, y_dtype, [&](auto r, auto t) { return launch_combine<decltype(r), decltype(t)>(a, H, stream); });
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_sort_rows(int T, int k, int E, int H, int dtype, const void* x, int64_t ld_x,
                                    const int32_t* topk_ids, void* rows, int64_t ld_rows, int32_t* offsets,
                                    int32_t* pos, int32_t* d_error, cudaStream_t stream) {
  clear_error();
  moe_status st = check_pairs(T, k, H);
  if (st != MOE_OK) return st;
  MOE_ARG(E >= 1 && E <= kMaxE, "E must be in [1, %d] (got %d)", kMaxE, E);
  MOE_ARG(known_dtype(dtype), "unknown element type %d", dtype);
  MOE_ARG(offsets, "null pointer");
  if (T == 0) {
    MOE_CUDA(cudaMemsetAsync(offsets, 0, (size_t)(E + 1) * 4, stream));
    return MOE_OK;
  }
  MOE_ARG(x && topk_ids && rows && pos, "null pointer");
  MOE_ARG(ld_x >= H && ld_rows >= H, "a row distance is below the row's length");
  ProfScope ps(MOE_K_SORT_ROWS, stream);
  const int sz = (int)dtype_size(dtype);
  SortArgs a = {T, k, 0, (const uint8_t*)x, (uint8_t*)rows, ld_x * sz, ld_rows * sz, pos};
  const long long width = (long long)H * sz;
  auto fits = [&](int v) { return splits(x, a.ld_x, width, v) && splits(rows, a.ld_rows, 0, v); };
  const int v = fits(16) ? 16 : fits(4) ? 4 : 2, P = T * k;
  a.nv = (int)(width / v);
  const long long blocks = ((long long)T * a.nv + 256 * kItems - 1) / (256 * kItems);
  if (P <= kSmallPairs) {
    const SmallSortArgs m = {a, E, topk_ids, offsets, pos, d_error};
    const char* name = "sort_small_kernel";
    if (v == 16) return launch_rows(sort_small_kernel<16>, blocks + 1, stream, name, m);
    if (v == 4) return launch_rows(sort_small_kernel<4>, blocks + 1, stream, name, m);
    return launch_rows(sort_small_kernel<2>, blocks + 1, stream, name, m);
  }
  const int warps = plan_warps(E);
  const size_t smem = (size_t)(warps + 2) * E * 4;
  static char allowed[64];
  MOE_CUDA(allow_smem(sort_plan_kernel, (size_t)(16 + 2) * kMaxE * 4, allowed));   // more than 32 warps of 1024 experts
  cudaError_t e = launch_pdl(sort_plan_kernel, dim3(kPlanBlocks), dim3(warps * 32), smem, stream, topk_ids, P, E, offsets,
                             pos, d_error);
  if (e != cudaSuccess) return cuda_fail(e, "sort_plan_kernel");
  st = check_launch("sort_plan_kernel");
  if (st != MOE_OK) return st;
  const char* name = "sort_rows_kernel";
  if (v == 16) return launch_rows(sort_rows_kernel<16>, blocks, stream, name, a);
  if (v == 4) return launch_rows(sort_rows_kernel<4>, blocks, stream, name, a);
  return launch_rows(sort_rows_kernel<2>, blocks, stream, name, a);
}

extern "C" moe_status moe_sort_rows_backward(int T, int k, int n_rows, int H, int dtype, const void* d_rows,
                                             int64_t ld_d_rows, const int32_t* pos, void* d_x, int64_t ld_d_x,
                                             cudaStream_t stream) {
  clear_error();
  return combine(T, k, n_rows, H, dtype, dtype, d_rows, ld_d_rows, pos, nullptr, nullptr, 0, d_x, ld_d_x,
                 MOE_K_SORT_ROWS_BWD, stream);
}

extern "C" moe_status moe_combine_rows(int T, int k, int n_rows, int H, int rows_dtype, int y_dtype, const void* rows,
                                       int64_t ld_rows, const int32_t* pos, const float* w, const void* base,
                                       int64_t ld_base, void* y, int64_t ld_y, cudaStream_t stream) {
  clear_error();
  return combine(T, k, n_rows, H, rows_dtype, y_dtype, rows, ld_rows, pos, w, base, ld_base, y, ld_y,
                 MOE_K_COMBINE_ROWS, stream);
}

extern "C" moe_status moe_combine_rows_backward(int T, int k, int n_rows, int H, int rows_dtype, int y_dtype,
                                                const void* d_y, int64_t ld_d_y, const void* rows, int64_t ld_rows,
                                                const int32_t* pos, const float* w, void* d_rows, int64_t ld_d_rows,
                                                float* d_w, cudaStream_t stream) {
  clear_error();
  moe_status st = check_pairs(T, k, H);
  if (st == MOE_OK) st = check_types(rows_dtype, y_dtype);
  if (st != MOE_OK) return st;
  MOE_ARG(n_rows >= 0, "n_rows must be >= 0 (got %d)", n_rows);
  if (T == 0) return MOE_OK;
  MOE_ARG(d_y && pos && (n_rows == 0 || (d_rows && (!d_w || rows))), "null pointer");
  MOE_ARG(ld_d_y >= H && ld_d_rows >= H && (!d_w || ld_rows >= H), "a row distance is below the row's length");
  MOE_ARG(!d_w || d_rows != rows || ld_d_rows == ld_rows, "in place, rows and d_rows need the same row distance");
  ProfScope ps(MOE_K_COMBINE_ROWS_BWD, stream);
  CombineBwdArgs a = {T, k, 0, n_rows, d_y, rows, d_rows, ld_d_y, ld_rows, ld_d_rows, pos, w, d_w};
  return by_types(rows_dtype, y_dtype, [&](auto r, auto t) { return launch_bwd<decltype(r), decltype(t)>(a, H, stream); });
}
