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

// A load under a predicate, 0 without it: a branch for each of a token's rows would wait for one row's
// place before the next one's load (8192 tokens of 6 rows of 4096 bf16: 131 us with branches).
__device__ __forceinline__ void load_if(bool on, const uint4* p, uint4& w) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\tmov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\t"
      "mov.u32 %3, 0;\n\t@q ld.global.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
      : "=&r"(w.x), "=&r"(w.y), "=&r"(w.z), "=&r"(w.w)
      : "l"(p), "r"((uint32_t)on)
      : "memory");
}
__device__ __forceinline__ void load_if(bool on, const uint2* p, uint2& w) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %3, 0;\n\tmov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\t"
      "@q ld.global.v2.u32 {%0,%1}, [%2];\n\t}"
      : "=&r"(w.x), "=&r"(w.y)
      : "l"(p), "r"((uint32_t)on)
      : "memory");
}
__device__ __forceinline__ void load_if(bool on, const uint32_t* p, uint32_t& w) {
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\tmov.u32 %0, 0;\n\t@q ld.global.u32 %0, [%1];\n\t}"
               : "=&r"(w)
               : "l"(p), "r"((uint32_t)on)
               : "memory");
}
__device__ __forceinline__ void load_if(bool on, const uint16_t* p, uint16_t& w) {
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\tmov.u16 %0, 0;\n\t@q ld.global.u16 %0, [%1];\n\t}"
               : "=&h"(w)
               : "l"(p), "r"((uint32_t)on)
               : "memory");
}

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
  __device__ __forceinline__ void load(bool on, const T* p) {
#pragma unroll
    for (int i = 0; i < N; ++i) load_if(on, reinterpret_cast<const W*>(p) + i, w[i]);
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
  constexpr int kKeep = 8;   // steps whose ids stay in registers
  int kept[kKeep];
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {
    const long long p = (s0 + i) * 32 + lane;
    kept[i] = s0 + i < s1 && p < P ? ids[p] : -1;
  }
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {
    bad |= kept[i] >= E;
    if (kept[i] >= 0 && kept[i] < E) atomicAdd(&mine[kept[i]], 1);
  }
#pragma unroll 8
  for (long long s = s0 + kKeep; s < s1; ++s) {
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
  auto place = [&](long long s, int e) {
    const long long p = s * 32 + lane;
    const bool in = e >= 0 && e < E;
    const unsigned peers = __match_any_sync(0xffffffffu, in ? e : -1);
    const int rank = __popc(peers & ((1u << lane) - 1));
    int at = -1;
    if (in) at = base[e] + mine[e] + rank;
    __syncwarp();
    if (in && rank == 0) mine[e] += __popc(peers);
    __syncwarp();
    if (p < P) pos[p] = at;
  };
#pragma unroll
  for (int i = 0; i < kKeep; ++i)
    if (s0 + i < s1) place(s0 + i, kept[i]);
  for (long long s = s0 + kKeep; s < s1; s += kKeep) {
    int e[kKeep];
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
      const long long p = (s + i) * 32 + lane;
      e[i] = s + i < s1 && p < P ? ids[p] : -1;
    }
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
      if (s + i < s1) place(s + i, e[i]);
  }
}

// ---------------------------------------------------------------------- sort --

// How a kernel over tokens' rows is laid out: 2^lg threads to a token, each taking U of its vectors 2^lg apart
// (so that a token's places and weights are read once for all of them), `splits` blocks to a row.
struct RowMap {
  int lg, splits;
  long long blocks;
  RowMap() = default;
  RowMap(int T, int nv, int U) {
    lg = 0;
    while (lg < 8 && (long long)U << lg < nv) ++lg;
    splits = (int)((nv + ((long long)U << lg) - 1) / ((long long)U << lg));
    blocks = (((long long)T << lg) + 255) / 256 * splits;
  }
  // the thread's token and first vector
  __device__ __forceinline__ long long token(int& v, int U) const {
    const int group = (int)blockIdx.x / splits, split = (int)blockIdx.x - group * splits;
    v = (split * U << lg) + (int)(threadIdx.x & ((1u << lg) - 1));
    return ((long long)group << (8 - lg)) + (threadIdx.x >> lg);
  }
};

struct SortArgs {
  int T, k, nv;              // nv: vectors of a row
  const uint8_t* x;
  uint8_t* rows;
  long long ld_x, ld_rows;   // bytes
  const int32_t* pos;
  RowMap map;
};

// x's rows are read once and written to the token's k rows.  16 bytes a vector where rows allow it,
// else single elements, more of them to a thread.
template <int VB>
struct SortItems {
  static constexpr int U = VB == 16 ? 2 : 8;
};
template <int VB>
__global__ void __launch_bounds__(256) sort_rows_kernel(const SortArgs a) {
  using W = typename Bytes<VB>::T;
  constexpr int U = SortItems<VB>::U;
  int v;
  const long long t = a.map.token(v, U);
  if (t >= a.T) return;
  const int step = 1 << a.map.lg;
  // before the wait: sort_plan_kernel lets this one start once the work before itself has completed, and x is not its
  const W* x = reinterpret_cast<const W*>(a.x + t * a.ld_x) + v;
  W w[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (v + u * step < a.nv) w[u] = x[u * step];
  pdl_wait();
  pdl_launch_dependents();
  const int32_t* pos = a.pos + t * a.k;
  for (int j0 = 0; j0 < a.k; j0 += 8) {
    int p[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = j0 + j < a.k ? pos[j0 + j] : -1;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (p[j] < 0) continue;
      W* o = reinterpret_cast<W*>(a.rows + p[j] * a.ld_rows) + v;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (v + u * step < a.nv) o[u * step] = w[u];
    }
  }
}

// Few pairs: one launch, each block placing the pairs of its own tokens by counting, a warp to a pair,
// the pairs that come before it; the last block writes the offsets.  Latency: a launch and a
// round trip to memory more than the copy.
constexpr int kSmallPairs = 4096, kItems = 2;   // pairs; vectors of a thread
// Whether counting is quicker than sort_plan_kernel (which takes some 5 us): a block compares each of its own
// pairs with all of them.
static bool counts_pairs(int P, int k, int nv) {
  const long long own = (256 * kItems / nv + 1LL) * k;
  return P <= kSmallPairs && own * P <= 131072;
}
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
  for (int p = tid; p < (P + 127) / 128 * 128; p += 256) {
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
  RowMap map;
};

// J rows of U vectors at a time are under way in a thread.
template <typename TR, typename TY, int V, int U, int J>
__global__ void __launch_bounds__(256, V == 8 ? 4 : 3) combine_rows_kernel(const CombineArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  int v;
  const long long t = a.map.token(v, U);
  if (t >= a.T) return;
  const int step = 1 << a.map.lg;
  const TR* rows = reinterpret_cast<const TR*>(a.rows) + (long long)v * V;
  const int32_t* pos = a.pos + t * a.k;
  const float* w = a.w ? a.w + t * a.k : nullptr;
  bool in[U];
#pragma unroll
  for (int u = 0; u < U; ++u) in[u] = v + u * step < a.nv;
  Vec<TY, V> base[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    base[u].load(a.base && in[u], reinterpret_cast<const TY*>(a.base) + t * a.ld_base + (long long)(v + u * step) * V);
  float s[U][V] = {};
#pragma unroll 1
  for (int j0 = 0; j0 < a.k; j0 += J) {
    Vec<TR, V> r[J][U];
    int p[J];
    float by[J];
#pragma unroll
    for (int j = 0; j < J; ++j) p[j] = j0 + j < a.k ? pos[j0 + j] : -1;
#pragma unroll
    for (int j = 0; j < J; ++j) by[j] = w && j0 + j < a.k ? w[j0 + j] : 1.f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const bool on = p[j] >= 0 && p[j] < a.n_rows;
      if (!on) by[j] = 0.f;   // the row reads as 0, and its weight is not used
      const TR* row = rows + p[j] * a.ld_rows;
#pragma unroll
      for (int u = 0; u < U; ++u) r[j][u].load(on && in[u], row + u * step * V);
    }
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float f[V];
        r[j][u].get(f);
#pragma unroll
        for (int i = 0; i < V; ++i) s[u][i] = fmaf(by[j], f[i], s[u][i]);
      }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (!in[u]) continue;
    const long long c = (long long)(v + u * step) * V;
    float b[V];   // 0 without a base
    base[u].get(b);
#pragma unroll
    for (int i = 0; i < V; ++i) s[u][i] += b[i];
    Vec<TY, V> y;
    y.set(s[u]);
    y.store(reinterpret_cast<TY*>(a.y) + t * a.ld_y + c);
  }
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

// p[j] of an index that only the thread knows
template <int J>
__device__ __forceinline__ int p_of(const int (&p)[J], int j) {
  int v = -1;
#pragma unroll
  for (int i = 0; i < J; ++i) v = i == j ? p[i] : v;
  return v;
}
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

// G threads to a token; its k products go J at a time, each thread holding the J sums over its own
// columns, U vectors of J rows under way.  Many tokens: a warp to each, which needs no barrier; few: a block.
template <typename TR, typename TY, int V, int G, int J, int U>
__global__ void __launch_bounds__(256) combine_bwd_kernel(const CombineBwdArgs a) {
  __shared__ float part[8][8];   // [warp][pair]
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, me = tid % G;
  const long long t = (long long)blockIdx.x * (256 / G) + tid / G;
  if (t >= a.T) return;   // all of a token's threads
  const TY* dy = reinterpret_cast<const TY*>(a.dy) + t * a.ld_dy;
  const TR* rows = reinterpret_cast<const TR*>(a.rows);
  TR* d_rows = reinterpret_cast<TR*>(a.d_rows);
#pragma unroll 1
  for (int j0 = 0; j0 < a.k; j0 += J) {
    int p[J];
    float by[J], s[8] = {};
#pragma unroll
    for (int j = 0; j < J; ++j) p[j] = j0 + j < a.k ? a.pos[t * a.k + j0 + j] : -1;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      by[j] = j0 + j < a.k && a.w ? a.w[t * a.k + j0 + j] : 1.f;
      if (p[j] >= a.n_rows) p[j] = -1;
    }
    for (int v0 = me; v0 < a.nv; v0 += G * U) {
      Vec<TY, V> dv[U];
      Vec<TR, V> r[U][J];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool in = v0 + u * G < a.nv;
        const long long c = (long long)(v0 + u * G) * V;
        dv[u].load(in, dy + c);
        if (a.dw)
#pragma unroll
          for (int j = 0; j < J; ++j) r[u][j].load(in && p[j] >= 0, rows + p[j] * a.ld_rows + c);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (v0 + u * G >= a.nv) break;
        const long long c = (long long)(v0 + u * G) * V;
        float d[V];
        dv[u].get(d);
        if (a.dw)
#pragma unroll
          for (int j = 0; j < J; ++j) {   // a pair without a row: 0
            float f[V];
            r[u][j].get(f);
#pragma unroll
            for (int i = 0; i < V; ++i) s[j] = fmaf(d[i], f[i], s[j]);
          }
#pragma unroll
        for (int j = 0; j < J; ++j) {
          if (p[j] < 0) continue;
          float o[V];
#pragma unroll
          for (int i = 0; i < V; ++i) o[i] = by[j] * d[i];
          Vec<TR, V> out;
          out.set(o);
          out.store(d_rows + p[j] * a.ld_d_rows + c);
        }
      }
    }
    if (!a.dw) continue;
    const float sum = sum8(s);
    const int j = lane >> 2;
    if (G == 32) {
      if ((lane & 3) == 0 && j < J && j0 + j < a.k) a.dw[t * a.k + j0 + j] = p_of(p, j) >= 0 ? sum : 0.f;
    } else {
      auto meet = [&] { asm volatile("bar.sync %0, %1;" ::"r"(1 + tid / G), "n"(G) : "memory"); };   // a token's warps
      meet();
      if ((lane & 3) == 0) part[warp][j] = sum;
      meet();
      if (me < J && j0 + me < a.k) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < G / 32; ++w) v += part[tid / G * (G / 32) + w][me];
        a.dw[t * a.k + j0 + me] = p_of(p, me) >= 0 ? v : 0.f;
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
  const int v = H % 8 == 0 && fits(8) ? 8 : H % 2 == 0 && fits(2) ? 2 : 1, u = v == 8 ? 1 : v == 2 ? 4 : 8;
  a.nv = H / v;
  a.map = RowMap(a.T, a.nv, u);
  const char* name = "combine_rows_kernel";
  if (v == 8) return launch_rows(combine_rows_kernel<TR, TY, 8, 1, sizeof(TR) == 4 ? 4 : 8>, a.map.blocks, s, name, a);
  if (v == 2) return launch_rows(combine_rows_kernel<TR, TY, 2, 4, 4>, a.map.blocks, s, name, a);
  return launch_rows(combine_rows_kernel<TR, TY, 1, 8, 4>, a.map.blocks, s, name, a);
}

template <typename TR, typename TY, int V>
static moe_status launch_bwd_v(CombineBwdArgs a, int H, cudaStream_t s) {
  a.nv = H / V;
  const char* name = "combine_bwd_kernel";
  auto run = [&](auto g, auto u) {
    constexpr int G = decltype(g)::value, U = decltype(u)::value;
    const long long blocks = ((long long)a.T + 256 / G - 1) / (256 / G);
    return a.k <= 4 ? launch_rows(combine_bwd_kernel<TR, TY, V, G, 4, U>, blocks, s, name, a)
                    : launch_rows(combine_bwd_kernel<TR, TY, V, G, 8, U>, blocks, s, name, a);
  };
  using std::integral_constant;
  // Measured, vectors of eight (bf16): 8192 tokens of 6 rows of 4096 134 us by warps, 151 by blocks (warps without a
  // second vector under way 175); 512 tokens of 8 21 and 14 (17 with two vectors); 64 tokens 15.6 and 4.0 (3.6).
  // Single elements (fp32, 1021 tokens of 5 rows of 1001): 13.3 by warps, 11.7 by halves of a block, 15 by blocks.
  const int sms = device_sms();
  if (a.T >= 16 * sms || a.nv <= 32) return run(integral_constant<int, 32>(), integral_constant<int, V == 8 ? 2 : 4>());
  if constexpr (V < 8) {
    return run(integral_constant<int, 128>(), integral_constant<int, 4>());
  } else {
    // 32 bytes of an fp32 row are two loads already: 64 tokens of 8 rows of 4096 6.7 us (7.3 with a second vector), 200 13.4
    // (15.8).  By warps the second one pays for fp32 too: 4096 tokens of 6 rows 131 us, 141 without.
    if constexpr (sizeof(TR) == 2)
      if (a.T < 2 * sms) return run(integral_constant<int, 256>(), integral_constant<int, 2>());
    return run(integral_constant<int, 256>(), integral_constant<int, 1>());
  }
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
  CombineArgs a = {T, k, 0, n_rows, rows, base, y, ld_rows, ld_base, ld_y, pos, w, {}};
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
  SortArgs a = {T, k, 0, (const uint8_t*)x, (uint8_t*)rows, ld_x * sz, ld_rows * sz, pos, {}};
  const long long width = (long long)H * sz;
  auto fits = [&](int v) { return splits(x, a.ld_x, width, v) && splits(rows, a.ld_rows, 0, v); };
  const int v = fits(16) ? 16 : fits(4) ? 4 : 2, P = T * k;
  a.nv = (int)(width / v);
  const long long blocks = ((long long)T * a.nv + 256 * kItems - 1) / (256 * kItems);
  if (counts_pairs(P, k, a.nv)) {
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
  a.map = RowMap(T, a.nv, v == 16 ? SortItems<16>::U : SortItems<2>::U);
  if (v == 16) return launch_rows(sort_rows_kernel<16>, a.map.blocks, stream, name, a);
  if (v == 4) return launch_rows(sort_rows_kernel<4>, a.map.blocks, stream, name, a);
  return launch_rows(sort_rows_kernel<2>, a.map.blocks, stream, name, a);
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
