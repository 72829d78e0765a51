// Clipping by the global norm, over tensors in many separate buffers (the bucket
// tables of the scattered-tensor AllReduce, [CoCoNet] "Breaking the Computation and
// Communication Abstraction Barrier in Distributed Machine Learning Workloads", the
// section on scattered tensors):
//
//   norm = sqrt(sum of x^2 over all buckets),  out = x * min(1, max_norm / norm)
//
// in two launches: the first reads every bucket and leaves one sum of squares a
// block, the second joins those (every block for itself, in block order) and scales.
// With CLIP_SUM the first also sums the ranks' tensors and stores the sums, so the
// AllReduce's one pass gives the norm as well. Bound by HBM: the second pass walks
// backwards, and finds in L2 what the first touched last.
//
// Measured, from a graph: BERT-large's 335 million fp16 gradients of 8 ranks, averaged
// and clipped into one copy, 1087 us (the two passes' 7.4 GB at 6.8 TB/s); 12.6 million
// bf16 ones to fp32 23.2 us, where the two launches and what each waits for at its
// ends are half; 153 million fp32 ones 292 us. Zeros take as long as other numbers.
// Numbers of ranks without a kernel of their own: 75.6 million bf16 of 5 ranks to fp32
// 247 us (4.3 TB/s), bound by instructions: every load takes its address by shuffles.

#include <float.h>
#include <math.h>

#include <type_traits>

#include "internal.h"
#include "rows.h"

namespace coco {
namespace {

constexpr int kHeaderWords = 16;  // of a bucket table
constexpr int kThreads = 256, kWarps = kThreads / 32;

struct ClipArgs {
  const uint32_t* table;
  const uint32_t* out_table;
  int64_t nbuckets;
  int32_t nranks, out_nranks;
  float alpha, max_norm;
  float* norm;
  double* parts;
  int32_t nparts;
};

// The entries of ranks r0 .. r0 + n - 1 (three words each, n at most 10) of bucket b, a word a lane: one load brings all.
__device__ __forceinline__ uint32_t entry_words(const uint32_t* table, int64_t b, int nranks, int r0, int n) {
  const int lane = threadIdx.x & 31;
  return lane < 3 * n ? __ldg(table + kHeaderWords + (b * nranks + r0) * 3 + lane) : 0u;
}

// A rank's part of a bucket: the j-th entry of a warp's words.
struct Bucket {
  char* base;  // its first element
  int32_t len;
};

__device__ __forceinline__ uint32_t code_of(uint32_t words) { return __shfl_sync(0xffffffffu, words, 2); }

template <typename T>
__device__ __forceinline__ Bucket bucket_of(uint32_t words, int j) {
  const uint32_t lo = __shfl_sync(0xffffffffu, words, 3 * j), hi = __shfl_sync(0xffffffffu, words, 3 * j + 1);
  const uint32_t code = code_of(words);  // the same bucket and length for every rank
  Bucket r;
  r.base = reinterpret_cast<char*>((static_cast<uint64_t>(hi) << 32) | lo) +
           static_cast<int64_t>(code >> 10) * 1024 * sizeof(T);
  r.len = static_cast<int>(code & 1023u) + 1;
  return r;
}

// Consecutive elements that a lane takes at a time, 16 bytes of the wider of the two types: neighbouring lanes' loads and
// stores join without gaps. (Eight fp32 values a lane are two vectors 32 bytes apart from the next lane's: 12.6 million
// bf16 gradients to fp32 took 28.7 us with them.)
template <typename T, typename U>
constexpr int unit_of() { return sizeof(T) == 4 || sizeof(U) == 4 ? 4 : 8; }

template <typename T, int N>
struct Part {  // 8 values of 16 bits
  Chunk<T> c;
  __device__ __forceinline__ void load(const void* base, int i) { c.load(base, i); }
  __device__ __forceinline__ void get(float (&f)[8]) const { c.get(f); }
  __device__ __forceinline__ void put(const float (&f)[8]) { c.put(f); }
  __device__ __forceinline__ uint32_t bits() const { return (c.v.x | c.v.y | c.v.z | c.v.w) & 0x7fff7fffu; }  // 0: all zeros
  __device__ __forceinline__ void store(void* base, int i) const { static_cast<uint4*>(base)[i] = c.v; }
  __device__ __forceinline__ void store_stream(void* base, int i) const { c.store(base, i); }
};
template <>
struct Part<float, 4> {
  uint4 v;
  __device__ __forceinline__ void load(const void* base, int i) { v = ld_stream(static_cast<const uint4*>(base) + i); }
  __device__ __forceinline__ void get(float (&f)[4]) const {
    f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y); f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
  }
  __device__ __forceinline__ void put(const float (&f)[4]) {
    v = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
  __device__ __forceinline__ uint32_t bits() const { return (v.x | v.y | v.z | v.w) & 0x7fffffffu; }
  __device__ __forceinline__ void store(void* base, int i) const { static_cast<uint4*>(base)[i] = v; }
  __device__ __forceinline__ void store_stream(void* base, int i) const { __stcs(static_cast<uint4*>(base) + i, v); }
};
template <typename T>
struct Part<T, 4> {  // 4 values of 16 bits
  Chunk<T> c;        // (half of one)
  __device__ __forceinline__ void load(const void* base, int i) {
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(c.v.x), "=r"(c.v.y)
                 : "l"(static_cast<const uint2*>(base) + i));
    c.v.z = c.v.w = 0;
  }
  __device__ __forceinline__ void get(float (&f)[4]) const {
    float g[8];
    c.get(g);
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = g[j];
  }
  __device__ __forceinline__ void put(const float (&f)[4]) {
    const float g[8] = {f[0], f[1], f[2], f[3], 0.0f, 0.0f, 0.0f, 0.0f};
    c.put(g);
  }
  __device__ __forceinline__ uint32_t bits() const { return (c.v.x | c.v.y) & 0x7fff7fffu; }
  __device__ __forceinline__ void store(void* base, int i) const { static_cast<uint2*>(base)[i] = make_uint2(c.v.x, c.v.y); }
  __device__ __forceinline__ void store_stream(void* base, int i) const {
    __stcs(static_cast<uint2*>(base) + i, make_uint2(c.v.x, c.v.y));
  }
};

// A lane's unit i of a bucket that ends inside it or before it: its elements, and zeros past them. (Plain loads: it may
// have been written by this thread.)
template <typename T, int N>
__device__ __forceinline__ void load_end(const Bucket& b, int i, float (&f)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j)
    f[j] = i * N + j < b.len ? static_cast<float>(reinterpret_cast<const T*>(b.base)[i * N + j]) : 0.0f;
}

template <typename T, int N>
__device__ __forceinline__ void store_end(const Bucket& b, int i, const float (&f)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j)
    if (i * N + j < b.len) reinterpret_cast<T*>(b.base)[i * N + j] = static_cast<T>(f[j]);
}

template <int N>
__device__ __forceinline__ float add_squares(const float (&f)[N], float s) {
#pragma unroll
  for (int j = 0; j < N; ++j) s = fmaf(f[j], f[j], s);
  return s;
}

// The squares' sum of a lane's part of a bucket, s in fp32; taken again in fp64 where that has left fp32's range (past
// its largest number, or so low that squares were lost). `bits` is 0 where the values are all zeros, whose sum is right:
// gradients have them (words that a batch has not, experts without tokens), and walking them again took three to five times
// as long as the pass itself.
template <typename T, int N>
__device__ __forceinline__ double squares(const Bucket& b, float s, uint32_t bits) {
  if ((s >= 0x1p-80f && s <= FLT_MAX) || bits == 0) return s;
  double d = 0.0;
#pragma unroll 1
  for (int i = threadIdx.x & 31; i * N < b.len; i += 32) {
    float f[N];
    load_end<T>(b, i, f);
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (f[j] != 0.0f) d = fma(static_cast<double>(f[j]), static_cast<double>(f[j]), d);
  }
  return d;
}

// The block's sum, in thread 0 (fp64 units are few: the other threads do not need it).
__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int i = 1; i < kWarps; ++i) v += red[i];
  return v;
}

// A whole bucket's squares. With CLIP_SUM a unit is the sum over the ranks (NR of them, or any number four at a time).
template <typename T, typename U, int MODE, int NR>
__device__ __forceinline__ double squares_full(const ClipArgs& a, int64_t b, uint32_t words, uint32_t out_words) {
  constexpr int N = unit_of<T, U>(), UNITS = 1024 / N / 32;
  const int lane = threadIdx.x & 31;
  float s = 0.0f;
  uint32_t bits = 0;
  if constexpr (MODE != CLIP_SUM) {
    const Bucket k = bucket_of<T>(words, 0);
    Part<T, N> v[UNITS];
#pragma unroll
    for (int i = 0; i < UNITS; ++i) v[i].load(k.base, lane + 32 * i);
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      float f[N];
      v[i].get(f);
      s = add_squares(f, s);
      bits |= v[i].bits();
    }
    return squares<T, N>(k, s, bits);
  } else {
    const Bucket to = bucket_of<U>(out_words, 0);
    auto finish = [&](float (&f)[N], int i) {
#pragma unroll
      for (int j = 0; j < N; ++j) f[j] = static_cast<float>(static_cast<U>(f[j] * a.alpha));
      Part<U, N> o;
      o.put(f);
      o.store(to.base, lane + 32 * i);  // (not a streaming store: it is read again)
      s = add_squares(f, s);
      bits |= o.bits();
    };
    // Loads do not pass a store, so those of the next units are issued ahead of it: 32 a thread where the ranks are known
    // (BERT-large's 1095 us with 16, 1079 with 32; 75.6 million bf16 of three ranks to fp32 131 and 122), else the next four
    // ranks'.
    if constexpr (NR > 0) {
      constexpr int AHEAD = 32 / NR < UNITS ? 32 / NR : UNITS;
      const void* in[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) in[r] = bucket_of<T>(words, r).base;
      Part<T, N> raw[AHEAD][NR];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
#pragma unroll
        for (int r = 0; r < NR; ++r) raw[i][r].load(in[r], lane + 32 * i);
#pragma unroll
      for (int i = 0; i < UNITS; ++i) {
        float f[N], g[N];
        raw[i % AHEAD][0].get(f);
#pragma unroll
        for (int r = 1; r < NR; ++r) {
          raw[i % AHEAD][r].get(g);
#pragma unroll
          for (int j = 0; j < N; ++j) f[j] += g[j];
        }
        if (i + AHEAD < UNITS)
#pragma unroll
          for (int r = 0; r < NR; ++r) raw[i % AHEAD][r].load(in[r], lane + 32 * (i + AHEAD));
        finish(f, i);
      }
    } else {
      uint32_t eight = entry_words(a.table, b, a.nranks, 0, a.nranks < 8 ? a.nranks : 8);  // eight ranks' entries
      Part<T, N> next[4];
      auto fetch = [&](int i, int r0) {
        if (a.nranks > 8 && r0 % 8 == 0)
          eight = entry_words(a.table, b, a.nranks, r0, a.nranks - r0 < 8 ? a.nranks - r0 : 8);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (r0 + r < a.nranks) next[r].load(bucket_of<T>(eight, r0 % 8 + r).base, lane + 32 * i);
      };
      fetch(0, 0);
#pragma unroll 1
      for (int i = 0; i < UNITS; ++i) {
        float f[N], g[N];
#pragma unroll
        for (int j = 0; j < N; ++j) f[j] = -0.0f;  // (added to anything, it leaves that as it is)
#pragma unroll 1
        for (int r0 = 0; r0 < a.nranks; r0 += 4) {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (r0 + r < a.nranks) {
              next[r].get(g);
#pragma unroll
              for (int j = 0; j < N; ++j) f[j] += g[j];
            }
          const bool same = r0 + 4 < a.nranks;
          if (same || i + 1 < UNITS) fetch(same ? i : i + 1, same ? r0 + 4 : 0);
        }
        finish(f, i);
      }
    }
    return squares<U, N>(to, s, bits);
  }
}

// The same for the last bucket of a tensor, a unit and a rank at a time.
template <typename T, typename U, int MODE>
__device__ __forceinline__ double squares_end(const ClipArgs& a, int64_t b, uint32_t words, uint32_t out_words) {
  constexpr int N = unit_of<T, U>();
  const Bucket k = bucket_of<T>(words, 0), to = bucket_of<U>(out_words, 0);
  const int rounds = (k.len + 32 * N - 1) / (32 * N);
  float s = 0.0f;
  uint32_t bits = 0;
#pragma unroll 1
  for (int r0 = 0; r0 < rounds; ++r0) {
    const int i = (threadIdx.x & 31) + 32 * r0;
    float f[N];
    load_end<T>(k, i, f);
    if constexpr (MODE == CLIP_SUM) {
#pragma unroll 1
      for (int r = 1; r < a.nranks; ++r) {
        const Bucket kr = bucket_of<T>(entry_words(a.table, b, a.nranks, r, 1), 0);
        float g[N];
        load_end<T>(kr, i, g);
#pragma unroll
        for (int j = 0; j < N; ++j) f[j] += g[j];
      }
#pragma unroll
      for (int j = 0; j < N; ++j) f[j] = static_cast<float>(static_cast<U>(f[j] * a.alpha));
      store_end<U>(to, i, f);
    }
    s = add_squares(f, s);
#pragma unroll
    for (int j = 0; j < N; ++j) bits |= __float_as_uint(f[j]) << 1;
  }
  if constexpr (MODE == CLIP_SUM) return squares<U, N>(to, s, bits);
  else return squares<T, N>(k, s, bits);
}

// Two blocks an SM with CLIP_SUM, whose 128 registers hold a bucket's loads of eight ranks (three blocks: BERT-large's 1086
// -> 1188 us), and four with any number of ranks (19 million values of five, fp16 78 us with three and 50 with four, fp32 127
// and 85). Warps take buckets round-robin (those of every rank with CLIP_LOCAL), the next one's entries under way. With
// CLIP_SUM the ranks' tensors are added in rank order, scaled by alpha, rounded to U and stored to out's rank 0, and it is
// those values' norm. Where the two tables' tensors do not have a bucket in common, nothing is written and the norm is NaN.
template <typename T, typename U, int MODE, int NR>
__global__ void __launch_bounds__(kThreads, MODE == CLIP_SUM && NR > 0 ? 2 : 4)
    k_clip_squares(const __grid_constant__ ClipArgs a) {
  __shared__ double red[kWarps];
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
  const int64_t nwarps = static_cast<int64_t>(gridDim.x) * kWarps;
  const int64_t items = MODE == CLIP_LOCAL ? a.nbuckets * a.nranks : a.nbuckets;
  const bool two = a.table != a.out_table;
  const int n = MODE == CLIP_SUM && NR > 0 ? NR : 1;
  uint32_t words = 0, out_words = 0;
  auto fetch = [&](int64_t it) {  // (CLIP_LOCAL counts the entries themselves)
    words = MODE == CLIP_LOCAL ? entry_words(a.table, it, 1, 0, 1) : entry_words(a.table, it, a.nranks, 0, n);
    if (two) out_words = MODE == CLIP_LOCAL ? entry_words(a.out_table, it, 1, 0, 1)
                                            : entry_words(a.out_table, it, a.out_nranks, 0, 1);
    else out_words = words;
  };
  double sum = 0.0;
  if (warp < items) fetch(warp);
  for (int64_t it = warp; it < items; it += nwarps) {
    const uint32_t w = words, ow = out_words;
    if (it + nwarps < items) fetch(it + nwarps);
    const uint32_t code = code_of(w);
    if (code != code_of(ow)) sum = __longlong_as_double(0x7ff8000000000000ll);
    else if ((code & 1023u) == 1023u) sum += squares_full<T, U, MODE, NR>(a, it, w, ow);
    else sum += squares_end<T, U, MODE>(a, it, w, ow);
  }
  free_launches();
  sum = block_sum(sum, red);
  if (threadIdx.x == 0) a.parts[blockIdx.x] = sum;
}

template <typename X, typename U>
__device__ __forceinline__ void scale_full(const ClipArgs& a, int64_t b, uint32_t words, uint32_t out_words, int first,
                                           int last, float factor) {
  constexpr int N = unit_of<X, U>(), UNITS = 1024 / N / 32;
  const int lane = threadIdx.x & 31;
  const Bucket from = bucket_of<X>(words, 0);
  Part<X, N> v[UNITS];
#pragma unroll
  for (int i = 0; i < UNITS; ++i) v[i].load(from.base, lane + 32 * i);
#pragma unroll 1
  for (int r = first; r < last; ++r) {
    const Bucket to = bucket_of<U>(r ? entry_words(a.out_table, b, a.out_nranks, r, 1) : out_words, 0);
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      float f[N];
      v[i].get(f);
#pragma unroll
      for (int j = 0; j < N; ++j) f[j] *= factor;
      Part<U, N> o;
      o.put(f);
      o.store_stream(to.base, lane + 32 * i);
    }
  }
}

template <typename X, typename U>
__device__ __forceinline__ void scale_end(const ClipArgs& a, int64_t b, uint32_t words, uint32_t out_words, int first,
                                          int last, float factor) {
  constexpr int N = unit_of<X, U>();
  const Bucket from = bucket_of<X>(words, 0);
  const int rounds = (from.len + 32 * N - 1) / (32 * N);
#pragma unroll 1
  for (int r0 = 0; r0 < rounds; ++r0) {
    const int i = (threadIdx.x & 31) + 32 * r0;
    float f[N];
    load_end<X>(from, i, f);
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] *= factor;
#pragma unroll 1
    for (int r = first; r < last; ++r)
      store_end<U>(bucket_of<U>(r ? entry_words(a.out_table, b, a.out_nranks, r, 1) : out_words, 0), i, f);
  }
}

// Every block joins the sums of squares; block 0 writes the norm. Then out = x * factor, last buckets first; x is the
// ranks' own tensor (CLIP_LOCAL), rank 0's (CLIP_REPLICATED), or out's rank 0 (CLIP_SUM). `in_place`: where the factor is
// 1, the tensors that hold x already are left as they are.
template <typename T, typename U, int MODE>
__global__ void __launch_bounds__(kThreads, 4) k_clip_scale(const __grid_constant__ ClipArgs a, bool in_place) {
  __shared__ double red[kWarps];
  __shared__ float shared_factor;
  await_launches();
  double total = 0.0;
  for (int i = threadIdx.x; i < a.nparts; i += kThreads) total += a.parts[i];
  total = block_sum(total, red);
  if (threadIdx.x == 0) {
    const double norm = sqrt(total);
    if (blockIdx.x == 0) *a.norm = static_cast<float>(norm);
    const bool stay = a.max_norm == INFINITY || norm <= static_cast<double>(a.max_norm);  // (no limit: a NaN's too)
    shared_factor = stay ? 1.0f : static_cast<float>(a.max_norm / norm);
  }
  __syncthreads();
  const float factor = shared_factor;
  const bool keep = factor == 1.0f && (in_place || MODE == CLIP_SUM);
  if (keep && (MODE != CLIP_SUM || a.out_nranks == 1)) return;
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
  const int64_t nwarps = static_cast<int64_t>(gridDim.x) * kWarps;
  const int64_t items = MODE == CLIP_LOCAL ? a.nbuckets * a.nranks : a.nbuckets;
  using X = typename std::conditional<MODE == CLIP_SUM, U, T>::type;
  const bool two = a.table != a.out_table;
  const int first = MODE == CLIP_SUM && keep ? 1 : 0, last = MODE == CLIP_LOCAL ? 1 : a.out_nranks;
  uint32_t words = 0, out_words = 0;
  auto fetch = [&](int64_t it) {
    words = MODE == CLIP_LOCAL ? entry_words(a.table, it, 1, 0, 1) : entry_words(a.table, it, a.nranks, 0, 1);
    if (two) out_words = MODE == CLIP_LOCAL ? entry_words(a.out_table, it, 1, 0, 1)
                                            : entry_words(a.out_table, it, a.out_nranks, 0, 1);
    else out_words = words;
  };
  int64_t it = items - 1 - warp;
  if (it >= 0) fetch(it);
  for (; it >= 0; it -= nwarps) {
    const uint32_t w = words, ow = out_words;
    if (it >= nwarps) fetch(it - nwarps);
    const uint32_t code = code_of(w);
    if (code != code_of(ow)) continue;
    const uint32_t src = MODE == CLIP_SUM ? ow : w;
    if ((code & 1023u) == 1023u) scale_full<X, U>(a, it, src, ow, first, last, factor);
    else scale_end<X, U>(a, it, src, ow, first, last, factor);
  }
}

template <typename T, typename U, int MODE>
cudaError_t clip_go(const ClipLaunch& L, cudaStream_t s) {
  ClipArgs a;
  a.table = static_cast<const uint32_t*>(L.table);
  a.out_table = static_cast<const uint32_t*>(L.out_table);
  a.nbuckets = L.nbuckets;
  a.nranks = L.nranks;
  a.out_nranks = L.out_nranks;
  a.alpha = L.alpha;
  a.max_norm = L.max_norm;
  a.norm = L.norm;
  a.parts = L.parts;
  const int64_t items = MODE == CLIP_LOCAL ? L.nbuckets * L.nranks : L.nbuckets;
  const int64_t want = items ? (items + kWarps - 1) / kWarps : 1;
  int64_t most = static_cast<int64_t>(sm_count()) * 4;
  most = most < kClipMaxParts ? most : kClipMaxParts;
  a.nparts = static_cast<int32_t>(want < most ? want : most);
  if constexpr (MODE == CLIP_SUM) {
    cudaError_t e = with_ranks<2, 3, 4, 8>(L.nranks, [&](auto n) {
      k_clip_squares<T, U, MODE, n.value><<<a.nparts, kThreads, 0, s>>>(a);
      return cudaGetLastError();
    });
    if (e != cudaSuccess) return e;
  } else {
    k_clip_squares<T, U, MODE, 1><<<a.nparts, kThreads, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  count_launch();
  const cudaError_t e = launch_early(k_clip_scale<T, U, MODE>, dim3(a.nparts), dim3(kThreads), s, a,
                                     L.table == L.out_table);
  count_launch();
  return e;
}

template <typename T, typename U>
cudaError_t clip_mode(const ClipLaunch& L, cudaStream_t s) {
  switch (L.mode) {
    case CLIP_LOCAL: return clip_go<T, U, CLIP_LOCAL>(L, s);
    case CLIP_REPLICATED: return clip_go<T, U, CLIP_REPLICATED>(L, s);
    default: return clip_go<T, U, CLIP_SUM>(L, s);
  }
}

template <typename T>
cudaError_t clip_out(const ClipLaunch& L, cudaStream_t s) {
  switch (L.out_dtype) {
    case COCO_F32: return clip_mode<T, float>(L, s);
    case COCO_F16: return clip_mode<T, __half>(L, s);
    default: return clip_mode<T, __nv_bfloat16>(L, s);
  }
}

}  // namespace

cudaError_t launch_scattered_clip(const ClipLaunch& L, cudaStream_t s) {
  switch (L.dtype) {
    case COCO_F32: return clip_out<float>(L, s);
    case COCO_F16: return clip_out<__half>(L, s);
    default: return clip_out<__nv_bfloat16>(L, s);
  }
}

}  // namespace coco
