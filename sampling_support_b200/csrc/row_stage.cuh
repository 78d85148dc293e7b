// Rows staged in shared memory: helpers of the kernels whose cluster copies a
// row's slices into its CTAs' shared memory once and passes over that copy.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "common.cuh"

namespace vs {

using u64 = unsigned long long;

// Eight elements of a row from j (a multiple of 8; j + 8 <= the row's end).
template <typename T>
union Eight {
  uint4 q[sizeof(T) / 2];
  T e[8];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) q[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = q[i];
  }
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Largest of eight elements (NaN if there is one).
__device__ __forceinline__ float max8(const Eight<uint16_t>& v) {
  uint32_t m = 0xFF80FF80u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = reinterpret_cast<const uint32_t*>(v.q)[i];
    const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&m),
                                         *reinterpret_cast<const __nv_bfloat162*>(&w));
    m = *reinterpret_cast<const uint32_t*>(&r);
  }
  return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
}
__device__ __forceinline__ float max8(const Eight<uint32_t>& v) {
  float m = __uint_as_float(v.e[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max_nan(m, __uint_as_float(v.e[i]));
  return m;
}
__device__ __forceinline__ f32x2 pair_of(const Eight<uint16_t>& v, int i) {
  const uint32_t w = reinterpret_cast<const uint32_t*>(v.q)[i];
  return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ f32x2 pair_of(const Eight<uint32_t>& v, int i) {
  return pack2(__uint_as_float(v.e[2 * i]), __uint_as_float(v.e[2 * i + 1]));
}

template <typename T>
__device__ __forceinline__ T warp_sum(T x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ float warp_max_nan(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = max_nan(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(p)), "r"(rank));
  return r;
}
// The two largest group maxima seen (the first NaN once there is one), and
// where the first is.
struct TwoMax {
  float first = -kInf, second = -kInf;
  int at = 0;
  __device__ __forceinline__ void add(int g, float t) {
    at = t > first ? g : at;
    second = fmaxf(second, fminf(first, t));
    first = max_nan(first, t);
  }
};

// Block of T threads: n <= T E words from src in descending order to dst (room
// for T E; may be src), zeros behind them.  A bitonic network over E
// neighbouring words per thread: most of its steps stay in registers or go
// through the warp's shuffles, log2(T / 32) (log2(T / 32) + 1) / 2 of them
// through dst (a network through shared memory alone took 1.3 us a step for
// 4,096 words and 256 threads).
template <int T, int E>
__device__ __forceinline__ void block_sort(const u64* src, u64* dst, uint32_t n) {
  const uint32_t base = threadIdx.x * E;
  u64 e[E];
#pragma unroll
  for (int r = 0; r < E; ++r) e[r] = base + r < n ? src[base + r] : 0ull;
  auto order = [](u64& a, u64& b, bool descending) {
    const u64 x = a, y = b;
    const bool swap = (x < y) == descending;
    a = swap ? y : x;
    b = swap ? x : y;
  };
#pragma unroll
  for (int size = 2; size < E; size <<= 1)
#pragma unroll
    for (int step = size >> 1; step > 0; step >>= 1)
#pragma unroll
      for (int r = 0; r < E; ++r)
        if (!(r & step)) order(e[r], e[r + step], !(r & size));
#pragma unroll 1
  for (uint32_t size = E; size <= T * E; size <<= 1) {
    const bool descending = (base & size) == 0u;
#pragma unroll 1
    for (uint32_t step = size >> 1; step >= E; step >>= 1) {
      const bool larger = descending == ((base & step) == 0u);
      if (step < 32u * E) {
#pragma unroll
        for (int r = 0; r < E; ++r) {
          const u64 o = __shfl_xor_sync(0xffffffffu, e[r], step / E);
          e[r] = (e[r] < o) == larger ? o : e[r];
        }
      } else {
        cta_sync();
#pragma unroll
        for (int r = 0; r < E; ++r) dst[base + r] = e[r];
        cta_sync();
#pragma unroll
        for (int r = 0; r < E; ++r) {
          const u64 o = dst[(base ^ step) + r];
          e[r] = (e[r] < o) == larger ? o : e[r];
        }
      }
    }
#pragma unroll
    for (int step = E >> 1; step > 0; step >>= 1)
#pragma unroll
      for (int r = 0; r < E; ++r)
        if (!(r & step)) order(e[r], e[r + step], descending);
  }
  cta_sync();
#pragma unroll
  for (int r = 0; r < E; ++r) dst[base + r] = e[r];
  cta_sync();
}

// N 16-byte words into a peer's shared memory, counted on its barrier there.
template <int N>
__device__ __forceinline__ void push_words(uint32_t dst, uint32_t bar, const void* src) {
  const uint32_t* w = static_cast<const uint32_t*>(src);
#pragma unroll
  for (int i = 0; i < N; ++i)
    asm volatile(
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%2, %3, %4, %5}, [%1];" ::"r"(dst + 16u * i),
        "r"(bar), "r"(w[4 * i]), "r"(w[4 * i + 1]), "r"(w[4 * i + 2]), "r"(w[4 * i + 3])
        : "memory");
}

// Half of x - ref.  The difference itself may leave fp32 (logits at both ends of
// the type) where the difference over T does not; halving is exact, one rounding
// as for the difference, and the factor behind it doubles.
__device__ __forceinline__ float half_diff(float x, float ref) { return fmaf(0.5f, x, -0.5f * ref); }

// log2(e) / T, for T >= 2^-126 below 2^127: twice of it is finite.
__device__ __forceinline__ float exponent_factor(float t) { return fminf(kLog2e / t, 1.5e38f); }

// min-p's test, exp(z) >= m, on the exponential itself: the masses below are cut
// at 46 nats and m may be smaller.  A call of its own: in line at its places the
// sampling kernels spill more (64.5 against 63.3 us for 64 x 151,936 fp32).
static __device__ __noinline__ bool mass_reaches(double z, float m) { return exp(z) >= static_cast<double>(m); }

__device__ __forceinline__ double exp2_64th(int i) { return exp2(static_cast<double>(i) * (1.0 / 64.0)); }

// The masses of one row: w(v) = exp((v - vmax) / T) in fixed point, w * 2^fx.
// exp(z) = 2^(k/64) 2^(f/64), k = rint(64 z log2 e), |f| <= 1/2: a 64-entry
// table of 2^(i/64) and the Taylor polynomial of degree 4 in f ln2 / 64
// (remainder below 4e-14), the table-driven method of Tang (1989).  Ten fp64
// operations: 3.7 elements per clock and SM against 2.3 for exp().  The list
// kernel and the general one share it, and no operation is left to contraction,
// so that a row gets the same masses, and the same token, in every batch.
struct RowMass {
  double vmax;   // largest logit
  double inv_t;  // 1 / T
  double scale;  // 2^fx
  double c64;    // 64 log2(e) / T
  int fx;

  __device__ __forceinline__ void set(float v, float t, int shift) {
    vmax = static_cast<double>(v);
    inv_t = 1.0 / static_cast<double>(t);
    scale = static_cast<double>(1ull << shift);
    c64 = 92.332482616893656 * inv_t;  // 64 / ln 2
    fx = shift;
  }
  __device__ __forceinline__ double z(float v) const { return __dmul_rn(static_cast<double>(v) - vmax, inv_t); }
  __device__ __forceinline__ bool reaches(float v, float m) const { return mass_reaches(z(v), m); }
  __device__ __forceinline__ float logprob(float v, u64 mass) const {
    return static_cast<float>(__dsub_rn(z(v), log(static_cast<double>(mass) / scale)));
  }
  // w 2^fx, rounded; 0 from 46 nats on (there w 2^fx < 2^-16).  tab(i): 2^(i/64)
  template <typename Tab>
  __device__ __forceinline__ u64 fixed(float v, Tab&& tab) const {
    constexpr double kA = 0.010830424696249145;    // ln 2 / 64
    constexpr double kRound = 6755399441055744.0;  // 1.5 * 2^52: the integer lands in the low word
    const double d = static_cast<double>(v) - vmax;
    const double r = fma(d, c64, kRound);
    const int k = __double2loint(r);
    const double f = fma(d, c64, -(r - kRound));
    double p = fma(fma(fma(fma(f, kA * kA * kA * kA / 24.0, kA * kA * kA / 6.0), f, kA * kA / 2.0), f, kA), f, 1.0);
    p = __dmul_rn(p, tab(k & 63));
    const double w = __hiloint2double(__double2hiint(p) + (((k >> 6) + fx) << 20), __double2loint(p));
    // w 2^fx <= 2^50: adding 2^52 rounds it to an integer in the mantissa
    const double x = __dadd_rn(r >= kRound - 4247.0 ? w : 0.0, 4503599627370496.0);  // 46 nats in units of ln 2 / 64
    return static_cast<u64>(__double_as_longlong(x)) & 0xFFFFFFFFFFFFFull;
  }
};

// A thread's share of a staged slice, the groups of eight g0, g0 + step, ..:
// z = sum of 2^((l - m) c) below a reference m.  The first group's maximum
// serves as long as the sum stays moderate (a sum of powers of two keeps its
// relative precision whatever the reference), which saves a pass; one fused
// multiply-add per exponent, from m c rounded: the sum is z 2^-rest.  That
// holds for |m c| below kDirect (logits over T up to 2,839), where |rest| is at
// most 2^-13 and a caller may put it back to first order: the square is worth
// 4e-9.  Beyond (small T, common offsets, masks by a finite value) rest would
// reach whole powers of two: there, after masked first groups and before far
// larger values the thread's maximum and the differences come first.  A NaN or
// +inf comes out as m.  seen(g, group g) runs once for every group when it is given.
constexpr float kDirect = 4096.f;
struct SeenNone {
  template <typename T>
  __device__ __forceinline__ void operator()(int, const T&) const {}
};
template <typename Raw, typename Seen = SeenNone>
__device__ __forceinline__ void slice_sum(const Raw* buf, int g0, int groups, int step, float c, float& m, float& z,
                                          float& rest, Seen&& seen = Seen{}) {
  constexpr bool kSeen = !std::is_same_v<std::decay_t<Seen>, SeenNone>;
  m = -kInf;
  z = rest = 0.f;
  if (g0 >= groups) return;
  {
    Eight<Raw> v;
    v.load(buf + g0 * 8);
    m = max8(v);
  }
  const float mc = __fmul_rn(m, c);
  const bool direct = fabsf(mc) < kDirect;
  if (kSeen && !direct)
    for (int g = g0; g < groups; g += step) {
      Eight<Raw> v;
      v.load(buf + g * 8);
      seen(g, v);
    }
  if (direct) {
    const f32x2 c2 = pack2(c, c), m2 = pack2(-mc, -mc);
    f32x2 z2 = pack2(0.f, 0.f), y2 = pack2(0.f, 0.f);
    for (int g = g0; g < groups; g += step) {
      Eight<Raw> v;
      v.load(buf + g * 8);
      if (kSeen) seen(g, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float a, b;
        unpack2(fma2(pair_of(v, i), c2, m2), a, b);
        if (i & 1)
          y2 = add2(y2, pack2(ex2(a), ex2(b)));
        else
          z2 = add2(z2, pack2(ex2(a), ex2(b)));
      }
    }
    float a, b;
    unpack2(add2(z2, y2), a, b);
    z = a + b;
    rest = fmaf(m, c, -mc);
  }
  if (z > 0.f && z < 1e30f) return;
  z = rest = 0.f;
  m = -kInf;
  for (int g = g0; g < groups; g += step) {
    Eight<Raw> v;
    v.load(buf + g * 8);
    m = max_nan(m, max8(v));
  }
  if (m > -kInf && m < kInf)
    for (int g = g0; g < groups; g += step) {
      Eight<Raw> v;
      v.load(buf + g * 8);
#pragma unroll
      for (int i = 0; i < 8; ++i) z += ex2(half_diff(value_of(v.e[i]), m) * (2.f * c));
    }
}

// Cluster size of a staged kernel: slices of at most 40 KB, so that several
// CTAs share an SM and their phases overlap; smaller ones while the GPU has SMs
// to spare; 0 when eight slices do not fit shared memory.
inline int stage_cluster_size(int rows, int vocab, int esize) {
  constexpr int kMost = 8;
  const int64_t bytes = static_cast<int64_t>(vocab) * esize;
  int c = 1;
  while (c < kMost && bytes > c * (40 << 10)) c *= 2;
  while (c < kMost && 2ll * c * rows <= 148 && bytes > c * (8 << 10)) c *= 2;
  return (bytes + c - 1) / c <= (200 << 10) ? c : 0;
}

// Lets `kernel` use all of an SM's dynamic shared memory on the current device,
// once per device (the attribute call costs about as much host time as the
// launch).  All of it, not what one call needs: threads that set different
// sizes could take each other's grant back before the launch.
template <typename K>
cudaError_t allow_shared(K kernel, std::atomic<bool> (&granted)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && granted[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 << 10);
  if (e == cudaSuccess && dev < 64) granted[dev].store(true, std::memory_order_relaxed);
  return e;
}

// Launch `kernel` with clusters of c CTAs.  `behind`: an earlier kernel of the
// same call precedes, and this one waits for it where it reads what it wrote.
template <auto Kernel, typename... Args>
cudaError_t launch_cluster(unsigned grid, int c, int threads, size_t smem, bool behind, cudaStream_t s,
                           const Args&... args) {
  static std::atomic<bool> granted[64];
  const cudaError_t e = allow_shared(Kernel, granted);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = c;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = behind ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, Kernel, args...);
}

}  // namespace vs
