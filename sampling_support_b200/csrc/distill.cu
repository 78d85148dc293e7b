// vs_distill_fwd / vs_distill_bwd: Kullback-Leibler loss of a row's softmax
// against a teacher's top log-probabilities, and its gradient.
//
// With L the row's list (ids >= 0, the first of each), q = softmax(l / T) over
// the vocabulary and a_k the teacher's masses on L:
//   list mode:  a = softmax(lp) on L;  loss = sum_L a (log a - log q)
//               dl_j = (g / T) (q_j - a_j [j in L])
//   tail mode:  a = exp(lp), a_t = max(0, 1 - sum a), q_t = sum of q outside L
//               loss = sum_L a (log a - log q) + a_t (log a_t - log q_t)
//               dl_j = (g / T) (q_j - a_j)            j in L
//               dl_j = (g / T) r_j (q_t - a_t)        else, r_j = q_j / q_t
// (r_j on its own normaliser: q_j (1 - a_t / q_t) would divide by a q_t that
// may be tiny.)  The elements outside L are summed apart from the list, so a
// small q_t is a sum of its own and never a difference next to 1: each CTA
// marks its row's list in a bitmap of one byte per eight elements, which costs
// one shared load per 16-byte (bf16) vector of the pass.
//
// One cluster per row, one slice of the row per CTA: one pass for the
// statistics; with a gradient requested in the same call a second one from
// L2.  The backward kernel alone needs no exchange: (row, chunk) blocks read
// the saved row constants.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace vs {

namespace {

constexpr int kDThreads = 512;
constexpr int kDWarps = kDThreads / 32;
constexpr int kBThreads = 256;  // backward kernel

// Saved per-row state (VS_CTX_BYTES_PER_ROW bytes).
struct alignas(16) DistillCtx {
  float c;      // log2(e) / T
  float inv_t;  // 1 / T
  float ref;    // log2 normaliser of the dense part (the row's, or that outside the list)
  float coef;   // factor of the dense part: 1, or q_t - a_t
  float lse2;   // log2 sum_j 2^(l_j c)
  float tnorm;  // teacher: a_k = exp(lp_k - tnorm)
  uint32_t zero;  // no gradient (empty list, non-finite row)
  uint32_t dup;   // the list repeats an id
  uint32_t pad[8];
};
static_assert(sizeof(DistillCtx) == VS_CTX_BYTES_PER_ROW, "ctx layout");

__device__ __forceinline__ float grad_value(float v) { return v; }
__device__ __forceinline__ float grad_value(uint16_t v) { return value_of(v); }
template <typename G>
__device__ __forceinline__ G to_grad(float v) {
  if constexpr (sizeof(G) == 2)
    return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  else
    return v;
}

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

// Slot s of a list is its id's first occurrence.
__device__ __forceinline__ bool first_of(const int32_t* ids, int s) {
  const int32_t id = ids[s];
  for (int i = 0; i < s; ++i)
    if (ids[i] == id) return false;
  return true;
}

// Gradient of the elements [j0, j1) of a row (j0 a multiple of 8): the dense
// part of every element, then the listed ones whole.  The whole block calls.
// k.dup: a repeated id's later slots are skipped here.
template <typename Raw, typename G, bool ACC, int NT>
__device__ __forceinline__ void grad_pass(const Raw* __restrict__ row, G* __restrict__ out, int j0, int j1,
                                          const DistillCtx& k, float g, const int32_t* ids, const float* lp,
                                          int width) {
  const float scale = k.zero ? 0.f : g * k.inv_t;
  const float dense = scale * k.coef;
  // what the listed elements held before the accumulation
  constexpr int SLOTS = (VS_MAX_SUPPORT_WIDTH + NT - 1) / NT;
  float old[SLOTS];
  if constexpr (ACC) {
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      const int s = threadIdx.x + i * NT;
      const int id = s < width ? ids[s] : -1;
      old[i] = id >= j0 && id < j1 ? grad_value(out[id]) : 0.f;
    }
    cta_sync();
  }
  for (int j = j0 + static_cast<int>(threadIdx.x) * 8; j < j1; j += NT * 8) {
    if (j + 8 <= j1) {
      Eight<Raw> x;
      Eight<G> o;
      x.load(row + j);
      if constexpr (ACC) o.load(out + j);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float d = k.zero ? 0.f : dense * ex2(fmaf(value_of(x.e[i]), k.c, -k.ref));
        if constexpr (ACC) d += grad_value(o.e[i]);
        o.e[i] = to_grad<G>(d);
      }
      o.store(out + j);
    } else {
      for (int i = j; i < j1; ++i) {
        float d = k.zero ? 0.f : dense * ex2(fmaf(value_of(row[i]), k.c, -k.ref));
        if constexpr (ACC) d += grad_value(out[i]);
        out[i] = to_grad<G>(d);
      }
    }
  }
  cta_sync();
  if (k.zero) return;
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) {
    const int s = threadIdx.x + i * NT;
    const int id = s < width ? ids[s] : -1;
    if (id >= j0 && id < j1 && (!k.dup || first_of(ids, s))) {
      const float q = ex2(fmaf(value_of(row[id]), k.c, -k.lse2));
      float d = scale * (q - expf(lp[s] - k.tnorm));
      if constexpr (ACC) d += old[i];
      out[id] = to_grad<G>(d);
    }
  }
}

// Sum / maximum of three doubles over the block, in every thread: warp
// shuffles, one partial per warp, every thread combines them in warp order.
struct Three {
  double a, b, c;
};
template <bool MAX>
__device__ __forceinline__ double join(double x, double y) {
  return MAX ? fmax(x, y) : x + y;
}
template <bool MAX>
__device__ __forceinline__ Three block_three(Three v, Three* scratch) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.a = join<MAX>(v.a, __shfl_xor_sync(0xffffffffu, v.a, o));
    v.b = join<MAX>(v.b, __shfl_xor_sync(0xffffffffu, v.b, o));
    v.c = join<MAX>(v.c, __shfl_xor_sync(0xffffffffu, v.c, o));
  }
  cta_sync();  // the previous call's readers are done
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  cta_sync();
  v = scratch[0];
  for (int w = 1; w < kDWarps; ++w) {
    v.a = join<MAX>(v.a, scratch[w].a);
    v.b = join<MAX>(v.b, scratch[w].b);
    v.c = join<MAX>(v.c, scratch[w].c);
  }
  return v;
}

struct alignas(16) DistillShared {
  int32_t ids[VS_MAX_SUPPORT_WIDTH];
  float lp[VS_MAX_SUPPORT_WIDTH];
  Three red[kDWarps];
  double part[2];  // this CTA's (reference, sum) outside the list, read by the peers
  uint32_t part_bad;
  uint32_t status, dup;
};

// Online sum of 2^(l c - m) over a thread's elements.
struct Online {
  float v, m, z;  // largest logit, m = fl(v c), the sum
  uint32_t bad;
  template <typename Raw>
  __device__ __forceinline__ void add(const Raw (&r)[8], uint32_t listed, float c) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = value_of(r[i]);
    if (listed) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (listed >> i & 1u) x[i] = -kInf;
    }
    float t = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) t = fmaxf(t, x[i]);
    if (t > v) {
      const float mn = __fmul_rn(t, c);
      z = v == -kInf ? 0.f : z * ex2(m - mn);
      v = t;
      m = mn;
    }
    if (v == -kInf) {  // nothing but masked elements so far, or NaN
#pragma unroll
      for (int i = 0; i < 8; ++i) bad |= x[i] != x[i] ? 1u : 0u;
      return;
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += ex2(fmaf(x[i], c, -m));
    z += s;
  }
};

template <typename Raw, typename G, bool GRAD>
__global__ void __launch_bounds__(kDThreads) distill_fwd_kernel(DistillParams P) {
  extern __shared__ __align__(16) unsigned char d_smem[];
  DistillShared& sh = *reinterpret_cast<DistillShared*>(d_smem);
  uint32_t* marks = reinterpret_cast<uint32_t*>(d_smem + sizeof(DistillShared));
  const uint8_t* mark8 = reinterpret_cast<const uint8_t*>(marks);
  cg::cluster_group cl = cg::this_cluster();
  const int C = static_cast<int>(cl.num_blocks()), rank = static_cast<int>(cl.block_rank());
  const int row = static_cast<int>(blockIdx.x) / C;
  const int tid = threadIdx.x;
  const int V = P.vocab;
  const Raw* x = static_cast<const Raw*>(P.logits) + static_cast<int64_t>(row) * P.ld;
  const int j0 = min(V, rank * P.chunk), j1 = min(V, j0 + P.chunk);
  const float t = P.temperature ? P.temperature[row] : P.temperature_scalar;
  const bool fine = t > 0.f && t < kInf;
  const float c = fminf(kLog2e / t, 3e38f);

  // the list: marks over the whole vocabulary, repeats found on the way
  const int words = (V + 31) / 32;
  for (int i = tid; i < (words + 3) / 4; i += kDThreads) reinterpret_cast<uint4*>(marks)[i] = make_uint4(0u, 0u, 0u, 0u);
  if (tid == 0) {
    sh.status = 0u;
    sh.dup = 0u;
  }
  cta_sync();
  for (int s = tid; s < P.width; s += kDThreads) {
    int32_t id = P.ids[static_cast<int64_t>(row) * P.teacher_ld + s];
    if (id < -1 || id >= V) {
      atomicOr(&sh.status, VS_ROW_BAD_SUPPORT_ID);
      id = -1;
    }
    if (id >= 0) {
      const uint32_t bit = 1u << (id & 31);
      if (atomicOr(&marks[id >> 5], bit) & bit) sh.dup = 1u;
    }
    sh.ids[s] = id;
    sh.lp[s] = P.lp[static_cast<int64_t>(row) * P.teacher_ld + s];
  }
  cta_sync();
  if (sh.dup) {
    constexpr int SLOTS = (VS_MAX_SUPPORT_WIDTH + kDThreads - 1) / kDThreads;
    bool drop[SLOTS];
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      const int s = tid + i * kDThreads;
      drop[i] = s < P.width && sh.ids[s] >= 0 && !first_of(sh.ids, s);
    }
    cta_sync();
#pragma unroll
    for (int i = 0; i < SLOTS; ++i)
      if (drop[i]) sh.ids[tid + i * kDThreads] = -1;
    cta_sync();
  }

  // the slice outside the list
  Online o{-kInf, -kInf, 0.f, 0u};
  for (int j = j0 + tid * 8; j < j1; j += kDThreads * 8) {
    Eight<Raw> q;
    if (j + 8 <= j1)
      q.load(x + j);
    else
#pragma unroll
      for (int i = 0; i < 8; ++i) q.e[i] = j + i < j1 ? x[j + i] : static_cast<Raw>(sizeof(Raw) == 2 ? 0xFF80u : 0xFF800000u);
    o.add(q.e, mark8[j >> 3], c);
  }

  // the listed elements: teacher value and student value
  constexpr int SLOTS = (VS_MAX_SUPPORT_WIDTH + kDThreads - 1) / kDThreads;
  double lp[SLOTS], u[SLOTS];
  bool kept[SLOTS];
  Three mx{-kInf, -kInf, o.m};
  uint32_t bad = o.bad || !(o.z < kInf) ? 1u : 0u;  // this slice, and the list
  uint32_t any = 0u;
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) {
    const int s = tid + i * kDThreads;
    const int id = s < P.width ? sh.ids[s] : -1;
    kept[i] = id >= 0;
    lp[i] = u[i] = -kInf;
    if (kept[i]) {
      const float v = value_of(x[id]), l = sh.lp[s];
      bad |= !(v < kInf) || !(l < kInf) ? 1u : 0u;
      lp[i] = static_cast<double>(l);
      u[i] = static_cast<double>(v) * static_cast<double>(c);
      mx.a = fmax(mx.a, lp[i]);
      mx.b = fmax(mx.b, u[i]);
      any = 1u;
    }
  }
  mx = block_three<true>(mx, sh.red);
  const bool tail = P.tail != 0;
  const double toff = tail ? 0.0 : mx.a;
  Three sum{0.0, 0.0, o.z == 0.f ? 0.0 : static_cast<double>(o.z) * exp2(static_cast<double>(o.m) - mx.c)};
#pragma unroll
  for (int i = 0; i < SLOTS; ++i)
    if (kept[i]) {
      sum.a += lp[i] == -kInf ? 0.0 : exp(lp[i] - toff);
      sum.b += u[i] == -kInf ? 0.0 : exp2(u[i] - mx.b);
    }
  sum = block_three<false>(sum, sh.red);
  __syncwarp();
  bad = __syncthreads_or(bad) ? 1u : 0u;
  __syncwarp();
  any = __syncthreads_or(any) ? 1u : 0u;

  // the cluster's sums, in rank order
  double mr = mx.c, zr = sum.c;
  if (C > 1) {
    if (tid == 0) {
      sh.part[0] = mr;
      sh.part[1] = zr;
      sh.part_bad = bad;
    }
    __syncwarp();
    cl.sync();
    mr = -kInf;
    zr = 0.0;
    for (int r = 0; r < C; ++r) mr = fmax(mr, cl.map_shared_rank(sh.part, r)[0]);
    for (int r = 0; r < C; ++r) {
      const double* p = cl.map_shared_rank(sh.part, r);
      if (p[1] != 0.0) zr += p[1] * exp2(p[0] - mr);
      bad |= *cl.map_shared_rank(&sh.part_bad, r);
    }
  }
  const double m = fmax(mr, mx.b);
  const double z = (zr != 0.0 ? zr * exp2(mr - m) : 0.0) + (sum.b != 0.0 ? sum.b * exp2(mx.b - m) : 0.0);
  if (!(z > 0.0)) bad = 1u;  // every logit masked, or NaN
  const double lse2 = m + log2(z);
  const double lr2 = zr > 0.0 ? mr + log2(zr) : -kInf;
  const double at = tail ? fmax(0.0, 1.0 - sum.a) : 0.0;
  const double qt = zr > 0.0 ? exp2(lr2 - lse2) : 0.0;
  const bool empty = any == 0u || (!tail && !(sum.a > 0.0));
  const double tnorm = tail ? 0.0 : toff + log(sum.a);
  const bool live = fine && !bad && !empty;

  constexpr double kLn2d = 0.69314718055994530942;
  double loss = 0.0;
#pragma unroll
  for (int i = 0; i < SLOTS; ++i)
    if (kept[i] && live) {
      const double l = lp[i] - tnorm, a = exp(l);
      if (a > 0.0) loss += a * (l - kLn2d * (u[i] - lse2));
    }
  Three fin = block_three<false>(Three{loss, 0.0, 0.0}, sh.red);
  loss = fin.a;
  if (live && at > 0.0 && zr > 0.0) loss += at * (log(at) - kLn2d * (lr2 - lse2));

  DistillCtx k{};
  k.c = c;
  k.inv_t = 1.f / t;
  const bool outside = tail && zr > 0.0;
  k.ref = static_cast<float>(outside ? lr2 : lse2);
  k.coef = tail ? (outside ? static_cast<float>(qt - at) : 0.f) : 1.f;
  k.lse2 = static_cast<float>(lse2);
  k.tnorm = static_cast<float>(tnorm);
  k.zero = live ? 0u : 1u;
  k.dup = sh.dup;
  if (rank == 0 && tid == 0) {
    if (P.loss) P.loss[row] = (!fine || bad) ? __int_as_float(0x7FC00000) : (empty ? 0.f : static_cast<float>(loss));
    if (P.valid) P.valid[row] = live ? 1 : 0;
    if (P.status)
      P.status[row] = sh.status | (sh.dup ? VS_ROW_DUP_SUPPORT_ID : 0u) | (!fine ? VS_ROW_BAD_PARAM : bad ? VS_ROW_NONFINITE_INPUT : empty ? VS_ROW_EMPTY_SUPPORT : 0u);
    if (P.ctx) static_cast<DistillCtx*>(P.ctx)[row] = k;
  }
  if constexpr (GRAD) {
    k.dup = 0u;  // repeats are already off the shared list
    G* out = static_cast<G*>(P.dlogits) + static_cast<int64_t>(row) * P.grad_ld;
    const float g = P.g_loss ? P.g_loss[row] : 1.f;
    grad_pass<Raw, G, false, kDThreads>(x, out, j0, j1, k, g, sh.ids, sh.lp, P.width);
  }
  if (C > 1) {
    __syncwarp();
    cl.sync();  // peers may still read this CTA's sums
  }
}

template <typename Raw, typename G, bool ACC>
__global__ void __launch_bounds__(kBThreads) distill_bwd_kernel(DistillParams P, int nchunks) {
  const int row = static_cast<int>(blockIdx.x / nchunks), part = static_cast<int>(blockIdx.x % nchunks);
  const int j0 = min(P.vocab, part * P.chunk), j1 = min(P.vocab, j0 + P.chunk);
  const Raw* x = static_cast<const Raw*>(P.logits) + static_cast<int64_t>(row) * P.ld;
  G* out = static_cast<G*>(P.dlogits) + static_cast<int64_t>(row) * P.grad_ld;
  const DistillCtx k = static_cast<const DistillCtx*>(P.ctx)[row];
  const float g = P.g_loss ? P.g_loss[row] : 1.f;
  const int64_t at = static_cast<int64_t>(row) * P.teacher_ld;
  grad_pass<Raw, G, ACC, kBThreads>(x, out, j0, j1, k, g, P.ids + at, P.lp + at, P.width);
}

template <typename Raw, typename G, bool GRAD>
cudaError_t launch_fwd(const DistillParams& P, int c, cudaStream_t s) {
  const size_t smem = sizeof(DistillShared) + (static_cast<size_t>(P.vocab) + 127) / 128 * 16;
  cudaError_t e = cudaFuncSetAttribute(distill_fwd_kernel<Raw, G, GRAD>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(P.rows) * c);
  cfg.blockDim = dim3(kDThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = c;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, distill_fwd_kernel<Raw, G, GRAD>, P);
}

}  // namespace

cudaError_t launch_distill_fwd(DistillParams P, vs_dtype dtype, vs_dtype dl_dtype, cudaStream_t s) {
  const int c = row_cluster_size(P.rows, P.vocab);
  P.chunk = ((P.vocab + c - 1) / c + 31) / 32 * 32;
  const bool grad = P.dlogits != nullptr, half = dl_dtype == VS_BF16;
  if (dtype == VS_BF16) {
    if (!grad) return launch_fwd<uint16_t, float, false>(P, c, s);
    return half ? launch_fwd<uint16_t, uint16_t, true>(P, c, s) : launch_fwd<uint16_t, float, true>(P, c, s);
  }
  if (!grad) return launch_fwd<uint32_t, float, false>(P, c, s);
  return half ? launch_fwd<uint32_t, uint16_t, true>(P, c, s) : launch_fwd<uint32_t, float, true>(P, c, s);
}

cudaError_t launch_distill_bwd(DistillParams P, vs_dtype dtype, vs_dtype dl_dtype, bool acc, cudaStream_t s) {
  // chunks of at least 8,192 elements, enough of them for four blocks per SM
  int n = 1;
  const int want = 4 * 148;
  if (P.rows < want) n = (want + P.rows - 1) / P.rows;
  n = std::max(1, std::min(n, P.vocab / 8192));
  P.chunk = ((P.vocab + n - 1) / n + 31) / 32 * 32;
  n = (P.vocab + P.chunk - 1) / P.chunk;
  const unsigned grid = static_cast<unsigned>(P.rows) * n;
  const bool half = dl_dtype == VS_BF16;
#define VS_DISTILL_BWD(RAW)                                                                          \
  do {                                                                                               \
    if (half)                                                                                        \
      acc ? distill_bwd_kernel<RAW, uint16_t, true><<<grid, kBThreads, 0, s>>>(P, n)                 \
          : distill_bwd_kernel<RAW, uint16_t, false><<<grid, kBThreads, 0, s>>>(P, n);               \
    else                                                                                             \
      acc ? distill_bwd_kernel<RAW, float, true><<<grid, kBThreads, 0, s>>>(P, n)                    \
          : distill_bwd_kernel<RAW, float, false><<<grid, kBThreads, 0, s>>>(P, n);                  \
  } while (0)
  if (dtype == VS_BF16)
    VS_DISTILL_BWD(uint16_t);
  else
    VS_DISTILL_BWD(uint32_t);
#undef VS_DISTILL_BWD
  return cudaGetLastError();
}

}  // namespace vs
