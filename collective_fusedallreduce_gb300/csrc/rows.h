// Rows held in registers: the pieces that the norms' and the experts' kernels share.
// A row belongs to `tpr` threads (a power of two, 32 to 1024), and a thread holds
// its 8-element chunks t, t + tpr, ... in fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "internal.h"

namespace coco {
namespace {

constexpr int kChunk = 8;         // elements a thread holds per step
constexpr int kBlockLanes = 16;   // lanes that hold the 128 columns of one scale
constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxFloor = 0x1p-100f;  // smallest block maximum a scale is made from: all-zero blocks stay finite

// ------------------------------------------------------------------ chunks

// (Not the non-coherent path, which is for memory that nothing writes while the kernel runs: outputs take inputs' places here,
// and a kernel placed early is on the device while the one ahead still stores what it will read. The times are the same.)
__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}

// Eight consecutive elements as loaded, and their conversions from and to fp32. Stores are streaming ones,
// which keeps outputs from displacing what is still to be read (the gradient, 8192 x 4096 fp16 on eight ranks: 118 to
// 116 us; in the quantiser the same cost 15 %, and it stores plainly).
template <typename T>
struct Chunk {
  uint4 v;
  __device__ __forceinline__ void load(const void* base, int64_t c) {
    v = ld_stream(static_cast<const uint4*>(base) + c);
  }
  __device__ __forceinline__ void load_cached(const void* base, int64_t c) {
    v = static_cast<const uint4*>(base)[c];
  }
  __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float (&f)[kChunk]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same<T, __half>::value) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
      } else {  // (bf16 is the upper half of fp32)
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
  __device__ __forceinline__ void put(const float (&f)[kChunk]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void store(void* base, int64_t c) const { __stcs(static_cast<uint4*>(base) + c, v); }
};

template <>
struct Chunk<float> {
  uint4 v, w;
  __device__ __forceinline__ void load(const void* base, int64_t c) {
    v = ld_stream(static_cast<const uint4*>(base) + 2 * c);
    w = ld_stream(static_cast<const uint4*>(base) + 2 * c + 1);
  }
  __device__ __forceinline__ void load_cached(const void* base, int64_t c) {
    v = static_cast<const uint4*>(base)[2 * c];
    w = static_cast<const uint4*>(base)[2 * c + 1];
  }
  __device__ __forceinline__ void zero() { v = w = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float (&f)[kChunk]) const {
    f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y); f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
    f[4] = __uint_as_float(w.x); f[5] = __uint_as_float(w.y); f[6] = __uint_as_float(w.z); f[7] = __uint_as_float(w.w);
  }
  __device__ __forceinline__ void put(const float (&f)[kChunk]) {
    v = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    w = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
  }
  __device__ __forceinline__ void store(void* base, int64_t c) const {
    __stcs(static_cast<uint4*>(base) + 2 * c, v);
    __stcs(static_cast<uint4*>(base) + 2 * c + 1, w);
  }
};

// The larger of two magnitudes; a NaN stays one, so that a block that holds one shows it in its scale.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float chunk_amax(const float (&f)[kChunk]) {
  float m = fabsf(f[0]);
#pragma unroll
  for (int j = 1; j < kChunk; ++j) m = max_nan(m, fabsf(f[j]));
  return m;
}

// The scale of a block whose largest magnitude is `amax`: the largest e4m3 value stands for that magnitude.
__device__ __forceinline__ float scale_of(float amax) { return __fdiv_rn(max_nan(amax, kAmaxFloor), kE4m3Max); }

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}

// Eight values over a block's scale, in e4m3 (round to nearest even). The quotient is the value times the
// scale's rounded reciprocal, corrected by its own residual (Markstein, "Computation of elementary functions on
// the IBM RISC System/6000 processor", 1990), which makes it the rounded quotient: with the product alone, some
// values fall on the other side of a rounding boundary. (With it some 30 of 33.5 million values still differ from the
// rounding in 64 bits, as they do where rows are divided: what fp32 leaves.) An infinite scale keeps the uncorrected
// product (0, or NaN for the infinity itself).
__device__ __forceinline__ uint2 to_e4m3(const float (&f)[kChunk], float scale) {
  const float inv = __frcp_rn(scale);
  const float s = inv == 0.0f ? 0.0f : -scale;
  const uint64_t inv2 = pack2(inv, inv), s2 = pack2(s, s);  // (two values an instruction)
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t f2 = pack2(f[2 * i], f[2 * i + 1]);
    uint64_t q2, r2;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q2) : "l"(f2), "l"(inv2));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r2) : "l"(q2), "l"(s2), "l"(f2));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(q2) : "l"(r2), "l"(inv2));
    float2 q;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(q.x), "=f"(q.y) : "l"(q2));
    h[i] = __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// The sum of `v` over the threads of a row (tpr of them, a power of two and at least a warp), the same
// value in each: within warps by shuffles, across warps through shared memory in warp order. Consecutive
// calls alternate between the two halves of `red` (`turn`), so one barrier a call is enough. OWN_BARRIERS: rows
// that share a block have a barrier each (named ones, from 1 on), so that they do not wait for one another.
template <bool OWN_BARRIERS>
__device__ __forceinline__ float row_sum(float v, int tpr, int slot, float (*red)[32], int turn) {
#pragma unroll
  for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  if (tpr == 32) return v;
  const int warp = threadIdx.x >> 5, warps = tpr >> 5;
  if ((threadIdx.x & 31) == 0) red[turn][warp] = v;
  // (one row a block, or more rows than there are named barriers: all threads together)
  if (!OWN_BARRIERS || blockDim.x == tpr || blockDim.x > 15 * tpr) __syncthreads();
  else asm volatile("bar.sync %0, %1;" ::"r"(1 + slot), "r"(tpr) : "memory");
  const int first = warp & ~(warps - 1);
  float s = red[turn][first];
  for (int i = 1; i < warps; ++i) s += red[turn][first + i];
  return s;
}

// The sum over the ranks' chunk c in rank order (fp32). NR: compile-time rank count, or 0.
template <typename T, int NR>
__device__ __forceinline__ void sum_ranks(const void* const* in, int nranks, int64_t c, float (&acc)[kChunk]) {
  if constexpr (NR > 0) {
    Chunk<T> raw[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) raw[r].load(in[r], c);
    raw[0].get(acc);
#pragma unroll
    for (int r = 1; r < NR; ++r) {
      float f[kChunk];
      raw[r].get(f);
#pragma unroll
      for (int j = 0; j < kChunk; ++j) acc[j] += f[j];
    }
  } else {
    Chunk<T> first;
    first.load(in[0], c);
    first.get(acc);
    for (int r0 = 1; r0 < nranks; r0 += 4) {
      Chunk<T> raw[4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (r0 + r < nranks) raw[r].load(in[r0 + r], c);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (r0 + r < nranks) {
          float f[kChunk];
          raw[r].get(f);
#pragma unroll
          for (int j = 0; j < kChunk; ++j) acc[j] += f[j];
        }
      }
    }
  }
}

// The same; any number of ranks (NR 0) goes four at a time, whose loads are all under way before the first addition, where
// sum_ranks loads one rank alone first. Which is better depends on what the last four hold: 8192 x 4096 bf16 normed on six
// ranks takes 132 us, and 137 with sum_ranks; on five 134 and 115.
template <typename T, int NR>
__device__ __forceinline__ void sum_all(const void* const* in, int nranks, int64_t c, float (&acc)[kChunk]) {
  if constexpr (NR > 0) {
    sum_ranks<T, NR>(in, nranks, c, acc);
  } else {
#pragma unroll
    for (int j = 0; j < kChunk; ++j) acc[j] = -0.0f;  // (added to anything, it leaves that as it is)
    for (int r0 = 0; r0 < nranks; r0 += 4) {
      Chunk<T> raw[4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (r0 + r < nranks) raw[r].load(in[r0 + r], c);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (r0 + r < nranks) {
          float f[kChunk];
          raw[r].get(f);
#pragma unroll
          for (int j = 0; j < kChunk; ++j) acc[j] += f[j];
        }
      }
    }
  }
}

// A chunk's eight values as four pairs, for instructions that take two values, each rounded as by itself. Half as many
// instructions, for twice as many registers in pairs: for the experts' rows, where a thread keeps little else, and not for
// the norms (two ranks to 8 bits 69 -> 83 us). A pair's product and the sum after it are contracted by the compiler.
struct Vec8 {
  uint64_t p[4];
};

__device__ __forceinline__ Vec8 splat8(float v) {
  const uint64_t q = pack2(v, v);
  return {{q, q, q, q}};
}
__device__ __forceinline__ Vec8 operator+(const Vec8& a, const Vec8& b) {
  Vec8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.p[i]) : "l"(a.p[i]), "l"(b.p[i]));
  return r;
}
__device__ __forceinline__ Vec8 operator*(const Vec8& a, const Vec8& b) {
  Vec8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.p[i]) : "l"(a.p[i]), "l"(b.p[i]));
  return r;
}
template <typename T>
__device__ __forceinline__ Vec8 values(const Chunk<T>& c) {
  float f[kChunk];
  c.get(f);
  return {{pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7])}};
}
__device__ __forceinline__ void unpack8(const Vec8& a, float (&f)[kChunk]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) asm("mov.b64 {%0, %1}, %2;" : "=f"(f[2 * i]), "=f"(f[2 * i + 1]) : "l"(a.p[i]));
}
// The sum of the eight values.
__device__ __forceinline__ float sum8(const Vec8& a) {
  float f[kChunk];
  unpack8(a, f);
  return ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
}
template <typename T>
__device__ __forceinline__ Chunk<T> rounded(const Vec8& a) {
  float f[kChunk];
  unpack8(a, f);
  Chunk<T> c;
  c.put(f);
  return c;
}

// Launches a kernel that may be placed on the device before the one ahead of it in the stream has ended. Its first
// statement is await_launches(): it reads and writes nothing before that kernel's end, so the order of their effects is the
// stream's, and what is saved is the launch. A kernel whose successor is known calls free_launches() when its last work is under way.
__device__ __forceinline__ void await_launches() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void free_launches() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, dim3 block, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// Calls f with the first of the numbers of ranks NS that nranks is, or with 0 (any number).
template <int... NS, typename F>
cudaError_t with_ranks(int nranks, F&& f) {
  cudaError_t e = cudaSuccess;
  const bool one = ((nranks == NS && (e = f(std::integral_constant<int, NS>()), true)) || ...);
  return one ? e : f(std::integral_constant<int, 0>());
}

// Threads of a row: a power of two that covers its chunks, at most 512, each with up to eight chunks (rows of up to
// 32768 columns).
struct RowShape {
  int tpr_log2, vpt, threads, rpb;
};
inline RowShape row_shape(int nchunks) {
  RowShape s;
  s.tpr_log2 = 5;
  while (s.tpr_log2 < 9 && (1 << s.tpr_log2) < nchunks) ++s.tpr_log2;
  const int tpr = 1 << s.tpr_log2;
  s.vpt = 1;
  while (s.vpt * tpr < nchunks) s.vpt *= 2;
  s.threads = tpr < 256 ? 256 : tpr;
  s.rpb = s.threads / tpr;
  return s;
}

}  // namespace
}  // namespace coco
