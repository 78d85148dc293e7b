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
// small q_t is a sum of its own and never a difference next to 1.
//
// Two forward kernels, one cluster per row and one slice of the row per CTA.
// distill_stage_kernel copies its slice to shared memory, finds repeats with a
// hash table and takes the listed elements out of the copy; all passes, the
// gradient's too, run over that copy.  distill_fwd_kernel serves rows that eight
// CTAs' shared memory does not hold (above 819,200 bf16 or 409,600 fp32
// tokens): marks in a bitmap over the vocabulary, the row read from global
// memory, a second pass from L2 for the gradient.  The backward kernel needs no
// exchange: (row, chunk) blocks read the saved row constants.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "row_stage.cuh"

namespace vs {

namespace {

constexpr int kDThreads = 512;
constexpr int kDWarps = kDThreads / 32;
constexpr int kBThreads = 256;  // backward kernel

// Saved per-row state (VS_CTX_BYTES_PER_ROW bytes).
struct alignas(16) DistillCtx {
  float c;      // log2(e) / T
  float inv_t;  // 1 / T
  // an element's share is 2^((l - ref) c - lz): the differences of the logits come first (halved, with
  // twice the factor), so that l c and l - ref may overflow (rows at the type's ends)
  float ref, lz;    // of the dense part: the whole row's, or what lies outside the list
  float coef;       // factor of the dense part: 1, or q_t - a_t
  float rall, lall; // the whole row's
  // teacher: a_k = tnorm exp(lp_k - tref).  In list mode tref is the list's largest value, so that values of
  // any size keep their differences (the logarithm of the sum added to it would round them away)
  float tref, tnorm;
  uint32_t zero;    // no gradient (empty list, non-finite row)
  uint32_t dup;     // the list repeats an id
  uint32_t pad[5];
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
  const float dense = scale * k.coef, c2 = 2.f * k.c;
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
        float d = k.zero ? 0.f : dense * ex2(fmaf(half_diff(value_of(x.e[i]), k.ref), c2, -k.lz));
        if constexpr (ACC) d += grad_value(o.e[i]);
        o.e[i] = to_grad<G>(d);
      }
      o.store(out + j);
    } else {
      for (int i = j; i < j1; ++i) {
        float d = k.zero ? 0.f : dense * ex2(fmaf(half_diff(value_of(row[i]), k.ref), c2, -k.lz));
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
      const float q = ex2(fmaf(half_diff(value_of(row[id]), k.rall), c2, -k.lall));
      float d = scale * (q - k.tnorm * expf(lp[s] - k.tref));
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

// Online sum of 2^((l - v) c) over a thread's elements.
struct Online {
  float v, z;  // largest logit, the sum
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
      z = v == -kInf ? 0.f : z * ex2(half_diff(v, t) * (2.f * c));
      v = t;
    }
    if (v == -kInf) {  // nothing but masked elements so far, or NaN
#pragma unroll
      for (int i = 0; i < 8; ++i) bad |= x[i] != x[i] ? 1u : 0u;
      return;
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += ex2(half_diff(x[i], v) * (2.f * c));
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
  const bool fine = t >= kLeastT && t < kInf;
  const float c = exponent_factor(t);

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
  Online o{-kInf, 0.f, 0u};
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
  Three mx{-kInf, -kInf, o.v};
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
      u[i] = static_cast<double>(v);
      mx.a = fmax(mx.a, lp[i]);
      mx.b = fmax(mx.b, u[i]);
      any = 1u;
    }
  }
  mx = block_three<true>(mx, sh.red);
  const bool tail = P.tail != 0;
  const double toff = tail ? 0.0 : mx.a;
  const double cd = static_cast<double>(c);  // the same factor everywhere: its rounding cancels
  Three sum{0.0, 0.0, o.z == 0.f ? 0.0 : static_cast<double>(o.z) * exp2((static_cast<double>(o.v) - mx.c) * cd)};
#pragma unroll
  for (int i = 0; i < SLOTS; ++i)
    if (kept[i]) {
      sum.a += lp[i] == -kInf ? 0.0 : exp(lp[i] - toff);
      sum.b += u[i] == -kInf ? 0.0 : exp2((u[i] - mx.b) * cd);
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
      if (p[1] != 0.0) zr += p[1] * exp2((p[0] - mr) * cd);
      bad |= *cl.map_shared_rank(&sh.part_bad, r);
    }
  }
  const double m = fmax(mr, mx.b);
  const double z = (zr != 0.0 ? zr * exp2((mr - m) * cd) : 0.0) + (sum.b != 0.0 ? sum.b * exp2((mx.b - m) * cd) : 0.0);
  if (!(z > 0.0)) bad = 1u;  // every logit masked, or NaN
  const double lz = log2(z), lr = zr > 0.0 ? (mr - m) * cd + log2(zr) - lz : -kInf;  // log2 q_t
  const double at = tail ? fmax(0.0, 1.0 - sum.a) : 0.0;
  const double qt = zr > 0.0 ? exp2(lr) : 0.0;
  const bool empty = any == 0u || (!tail && !(sum.a > 0.0));
  const double tlog = tail ? 0.0 : log(sum.a);
  const bool live = fine && !bad && !empty;

  constexpr double kLn2d = 0.69314718055994530942;
  double loss = 0.0;
#pragma unroll
  for (int i = 0; i < SLOTS; ++i)
    if (kept[i] && live) {
      const double l = lp[i] - toff - tlog, a = exp(l);
      if (a > 0.0) loss += a * (l - kLn2d * ((u[i] - m) * cd - lz));
    }
  Three fin = block_three<false>(Three{loss, 0.0, 0.0}, sh.red);
  loss = fin.a;
  if (live && at > 0.0 && zr > 0.0) loss += at * (log(at) - kLn2d * lr);

  DistillCtx k{};
  k.c = c;
  k.inv_t = 1.f / t;
  const bool outside = tail && zr > 0.0;
  k.rall = static_cast<float>(m);
  k.lall = static_cast<float>(lz);
  k.ref = outside ? static_cast<float>(mr) : k.rall;
  k.lz = outside ? static_cast<float>(log2(zr)) : k.lall;
  k.coef = tail ? (outside ? static_cast<float>(qt - at) : 0.f) : 1.f;
  k.tref = static_cast<float>(toff);
  k.tnorm = tail ? 1.f : static_cast<float>(1.0 / sum.a);
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

// ---------------------------------------------------------------------------
// Rows whose slices fit shared memory: every CTA of the cluster copies its
// slice there once (a bulk asynchronous copy), and all passes read that copy,
// so a call reads each logit from HBM once and, with a gradient, writes it
// once.  The listed elements are taken out of the copy (set to -inf) before
// the sums.  Warp 0 goes through the teacher's list in fp64 while the other
// warps go through the slice; the CTAs' parts are pushed into the shared
// memory of those that need them (the leader's, with a gradient everyone's).
// A CTA holds its shared memory for a few microseconds of mostly latency, so
// the rate is that of the slots: 40 KB slices, five CTAs per SM.  Measured: loss
// and gradient of 2,048 x 151,936 bf16 in one call 261 us (4.8 TB/s of reads and
// writes), the loss alone of 4,096 such rows 291 us (4.3 TB/s).

constexpr int kSThreads = 256;
constexpr int kSWarps = kSThreads / 32;
constexpr int kSSlice = kSThreads - 32;  // threads of the slice passes
constexpr int kSMaxCluster = 8;

// One CTA's part of the row's sums of 2^((l - m) c): 48 bytes.  The loss is a
// difference of logarithms that may be near zero, so what is joined is in fp64
// from each thread's sum on, and so are the listed elements, which hold most
// of the mass: with fp32 there the loss was off by up to 1e-7, now by 1e-8.
struct alignas(16) DistillPart {
  float mr, ml;   // largest logit outside the list, and of its listed elements
  double zr, zl;  // the sums below them
  double w, wu;  // sums of the teacher's weight, and of it times (l - ml) c, over its listed elements
  uint32_t bad, pad;
};
static_assert(sizeof(DistillPart) == 48, "three 16-byte words");

// 2^x for |x| <= 1,000 to fp64's rounding: the Taylor polynomial of degree 12 in
// the fraction (remainder below (ln2 / 2)^13 / 13! = 2e-16), in pairs and fours,
// a shorter chain than exp2()'s; the list's warp is as long as the slice's
// passes.  Degree 8 left 2e-10, which 1 - sum a hands on whole: 2e-4 of a
// teacher's rest of 1e-6, and so of the gradient outside the list.
__device__ __forceinline__ double exp2_near(double x) {
  const double r = x + 6755399441055744.0;  // 1.5 * 2^52: the integer lands in the low word
  const double f = (x - (r - 6755399441055744.0)) * 0.69314718055994531, f2 = f * f, f4 = f2 * f2;
  const double lo = fma(f2, fma(f, 1.0 / 6.0, 0.5), 1.0 + f);
  const double mid = fma(f2, fma(f, 1.0 / 5040.0, 1.0 / 720.0), fma(f, 1.0 / 120.0, 1.0 / 24.0));
  const double hi = fma(f4, 1.0 / 479001600.0,
                        fma(f2, fma(f, 1.0 / 39916800.0, 1.0 / 3628800.0), fma(f, 1.0 / 362880.0, 1.0 / 40320.0)));
  const double p = fma(f4, fma(f4, hi, mid), lo);
  return __hiloint2double(__double2hiint(p) + (__double2loint(r) << 20), __double2loint(p));
}
// 2^x for x <= 0 to 3e-10 of itself (degree 8), 0 where it is small: the
// student's listed shares, whose sum enters the loss by its logarithm alone
// (degree 12 there too: a call of 8 x 1,024 7.5 instead of 6.9 us).
__device__ __forceinline__ double exp2_below(double x) {
  const double r = x + 6755399441055744.0;
  const double f = (x - (r - 6755399441055744.0)) * 0.69314718055994531, f2 = f * f;
  const double lo = fma(f2, fma(f, 1.0 / 6.0, 0.5), 1.0 + f);
  const double hi = fma(f2, fma(f2, 1.0 / 40320.0, fma(f, 1.0 / 5040.0, 1.0 / 720.0)), fma(f, 1.0 / 120.0, 1.0 / 24.0));
  const double p = fma(f2 * f2, hi, lo);
  return x >= -1000.0 ? __hiloint2double(__double2hiint(p) + (__double2loint(r) << 20), __double2loint(p)) : 0.0;
}

// 2^(d c - rest) for a part's distance d = x - ref <= 0 from the largest, |rest| at most
// 2^-13 (slice_sum): the product's rounding is put back (at d = -20 it would be
// worth 1e-6) and so is rest, both to first order.  What is left is the exponential's
// 2^-22, and nothing at d = 0; d is a distance of references, each the maximum of
// a thread's first group, so a part below the largest may hold much of the mass.
__device__ __forceinline__ double part_scale(float x, float ref, float c, float rest) {
  const float d = half_diff(x, ref), c2 = 2.f * c, p = __fmul_rn(d, c2);
  const float lo = fmaf(d, c2, -p) - rest;
  const float e = ex2(p);
  return e > 0.f ? static_cast<double>(e) * (1.0 + 0.69314718055994531 * static_cast<double>(lo)) : 0.0;
}

struct alignas(16) DistillStage {
  DistillPart parts[kSMaxCluster];  // from the CTA of each rank
  DistillCtx k;
  uint64_t bar, xbar;  // the slice's copy; the parts
  double s0, t1, tlog, at;
  float tref;
  float red_m[kSWarps];
  double red_z[kSWarps];
  uint32_t status, dup, any, bad;
};

// Room behind it: the list's ids, teacher values and student values, and a
// hash table of at least twice its width; then the slice.
__host__ __device__ inline int stage_width(int width) { return (width + 3) / 4 * 4; }
__host__ __device__ inline int stage_hash(int width) {
  int h = 64;
  while (h < 2 * width) h *= 2;
  return h;
}
__host__ __device__ inline size_t stage_fixed(int width) {
  return sizeof(DistillStage) + 12 * static_cast<size_t>(stage_width(width)) + 4 * static_cast<size_t>(stage_hash(width));
}

template <typename Raw, typename G, bool GRAD>
__global__ void __launch_bounds__(kSThreads, 5) distill_stage_kernel(DistillParams P) {
  extern __shared__ __align__(16) unsigned char d_smem[];
  DistillStage& sh = *reinterpret_cast<DistillStage*>(d_smem);
  const int W = P.width, W4 = stage_width(W), hsize = stage_hash(W);
  int32_t* ids = reinterpret_cast<int32_t*>(d_smem + sizeof(DistillStage));  // -1: pad, bad or repeated
  float* lps = reinterpret_cast<float*>(ids + W4);
  float* us = lps + W4;
  int32_t* hash = reinterpret_cast<int32_t*>(us + W4);
  Raw* buf = reinterpret_cast<Raw*>(hash + hsize);
  constexpr Raw kMasked = static_cast<Raw>(sizeof(Raw) == 2 ? 0xFF80u : 0xFF800000u);
  cg::cluster_group cl = cg::this_cluster();
  const int C = static_cast<int>(cl.num_blocks()), rank = static_cast<int>(cl.block_rank());
  const int row = static_cast<int>(blockIdx.x) / C;
  const int tid = threadIdx.x, lane = tid & 31;
  const int V = P.vocab;
  const Raw* x = static_cast<const Raw*>(P.logits) + static_cast<int64_t>(row) * P.ld;
  const int j0 = min(V, rank * P.chunk), j1 = min(V, j0 + P.chunk);
  const int n = j1 - j0, groups = (n + 7) / 8;  // of eight elements, the last one filled up with masked ones
  const uint32_t bytes = static_cast<uint32_t>(n / 8) * 8u * sizeof(Raw);

  if (tid == 0) {
    mbar_init(&sh.bar, 1);
    mbar_init(&sh.xbar, 1);
    fence_barrier_init();
    fence_proxy_async();
    if (GRAD || rank == 0) mbar_arrive_expect_tx(&sh.xbar, static_cast<uint32_t>(C * sizeof(DistillPart)));
    if (bytes) {
      mbar_arrive_expect_tx(&sh.bar, bytes);
      bulk_load_all(buf, x + j0, bytes, &sh.bar);
    }
    sh.status = sh.dup = sh.any = sh.bad = 0u;
  }
  // this thread's first slot of the list, on its way during the set-up
  const int64_t list_at = static_cast<int64_t>(row) * P.teacher_ld;
  const int32_t id0 = tid < W ? P.ids[list_at + tid] : -1;
  const float lp0 = tid < W ? P.lp[list_at + tid] : 0.f;
  // the parts' barriers are ready everywhere once every CTA has arrived here
  __syncwarp();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // ordered by the fence above
  const float t = P.temperature ? P.temperature[row] : P.temperature_scalar;
  const bool fine = t >= kLeastT && t < kInf;
  const float c = exponent_factor(t);
  const bool tail = P.tail != 0;
  for (int i = n / 8 * 8 + tid; i < groups * 8; i += kSThreads) buf[i] = i < n ? x[j0 + i] : kMasked;

  // the list, and whether it repeats an id
  for (int i = tid; i < hsize / 4; i += kSThreads) reinterpret_cast<int4*>(hash)[i] = make_int4(-1, -1, -1, -1);
  cta_sync();
  for (int s = tid; s < W; s += kSThreads) {
    int32_t id = s == tid ? id0 : P.ids[list_at + s];
    lps[s] = s == tid ? lp0 : P.lp[list_at + s];
    if (id < -1 || id >= V) {
      atomicOr(&sh.status, VS_ROW_BAD_SUPPORT_ID);
      id = -1;
    }
    ids[s] = id;
    if (id >= 0) {
      sh.any = 1u;
      uint32_t h = (static_cast<uint32_t>(id) * 2654435761u) >> 16 & (hsize - 1);
      for (int probe = 0; probe < hsize; ++probe) {  // at most half full: ends at a free place
        const int32_t old = atomicCAS(&hash[h], -1, id);
        if (old == -1) break;
        if (old == id) {
          sh.dup = 1u;
          break;
        }
        h = (h + 1) & (hsize - 1);
      }
    }
  }
  cta_sync();
  if (sh.dup) {
    constexpr int kSlots = (VS_MAX_SUPPORT_WIDTH + kSThreads - 1) / kSThreads;
    uint32_t drop = 0u;
    for (int i = 0; i < kSlots; ++i) {
      const int s = tid + i * kSThreads;
      if (s < W && ids[s] >= 0 && !first_of(ids, s)) drop |= 1u << i;
    }
    cta_sync();
    for (int i = 0; i < kSlots; ++i)
      if (drop >> i & 1u) ids[tid + i * kSThreads] = -1;
    cta_sync();
  }

  // take this slice's listed elements out of the copy
  if (bytes && !mbar_wait(&sh.bar, 0)) atomicOr(&sh.bad, 2u);
  __syncwarp();
  for (int s = tid; s < W; s += kSThreads) {  // repeats are off the list: no two slots name one element
    const int id = ids[s];
    float u = -kInf;
    if (id >= j0 && id < j1) {
      u = value_of(buf[id - j0]);
      buf[id - j0] = kMasked;
    }
    us[s] = u;
  }
  cta_sync();

  DistillPart mine{-kInf, -kInf, 0.0, 0.0, 0.0, 0.0, 0u, 0u};
  const double cd = static_cast<double>(c);  // the same factor everywhere: its rounding cancels
  if (tid < 32) {
    // the list: the teacher's sums s0 = sum w, t1 = sum w (lp - off) with w = exp(lp - off) over all of it, and
    // the student's over this slice's elements
    float off = -kInf;
    if (!tail)
      for (int s = lane; s < W; s += 32)
        if (ids[s] >= 0) off = fmaxf(off, lps[s]);
    off = tail ? 0.f : warp_max_nan(off);
    if (!(off > -kInf)) off = 0.f;
    float lmax = -kInf;
    for (int s = lane; s < W; s += 32)
      if (ids[s] >= j0 && ids[s] < j1) lmax = max_nan(lmax, us[s]);
    lmax = warp_max_nan(lmax);
    double s0 = 0.0, t1 = 0.0, ws = 0.0, wu = 0.0;
    uint32_t bad = lmax < kInf ? 0u : 1u;  // NaN or +inf
    double zl = 0.0;
    for (int s = lane; s < W; s += 32) {
      const int id = ids[s];
      if (id < 0) continue;
      const float l = lps[s], u = us[s];
      const bool own = id >= j0 && id < j1;
      bad |= !(l < kInf) ? 1u : 0u;
      if (l > -kInf) {
        const double below = static_cast<double>(l) - static_cast<double>(off), x2 = below * 1.4426950408889634;
        const double w = fabs(x2) <= 1000.0 ? exp2_near(x2) : exp(below);
        s0 += w;
        t1 += w * below;
        if (own && w > 0.0) {
          ws += w;
          if (lmax > -kInf) wu += w * ((static_cast<double>(u) - static_cast<double>(lmax)) * cd);
        }
      }
      if (own && lmax > -kInf) zl += exp2_below((static_cast<double>(u) - static_cast<double>(lmax)) * cd);
    }
    mine.ml = lmax;
    mine.zl = warp_sum(zl);
    mine.w = warp_sum(ws);
    mine.wu = warp_sum(wu);
    s0 = warp_sum(s0);
    t1 = warp_sum(t1);
    mine.bad = __reduce_or_sync(0xffffffffu, bad);
    if (lane == 0) {
      sh.s0 = s0;
      sh.t1 = t1;
      sh.tref = off;
      sh.tlog = tail ? 0.0 : log(s0);
      sh.at = tail ? fmax(0.0, 1.0 - s0) : 0.0;
    }
  } else {
    float m, z, rest;
    slice_sum(buf, tid - 32, groups, kSSlice, c, m, z, rest);
    const float wm = warp_max_nan(m);  // a NaN or +inf marks the part
    const double zw = warp_sum(z != 0.f ? z * part_scale(m, wm, c, rest) : 0.0);
    if (lane == 0) {
      sh.red_m[tid >> 5] = wm;
      sh.red_z[tid >> 5] = zw;
    }
  }
  cta_sync();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (tid < 32) {
    const bool in = lane > 0 && lane < kSWarps;
    const float m = in ? sh.red_m[lane] : -kInf;
    const double z = in ? sh.red_z[lane] : 0.0;
    mine.mr = warp_max_nan(m);
    mine.zr = warp_sum(z != 0.0 ? z * part_scale(m, mine.mr, c, 0.f) : 0.0);
    mine.bad |= sh.bad | (mine.mr < kInf ? 0u : 1u);
    if (lane < (GRAD ? C : 1)) push_words<sizeof(DistillPart) / 16>(peer_addr(&sh.parts[rank], lane), peer_addr(&sh.xbar, lane), &mine);
  }
  if (!GRAD && rank != 0) return;  // nothing is pushed here

  // the row's sums, by the first warp: lane r takes CTA r's part, a fixed tree
  if (tid < 32) {
    const bool got = mbar_wait(&sh.xbar, 0);
    __syncwarp();
    const DistillPart p = lane < C && got ? sh.parts[lane] : DistillPart{-kInf, -kInf, 0.0, 0.0, 0.0, 0.0, 0u, 0u};
    const float a = warp_max_nan(fmaxf(p.mr, -kInf)), b = warp_max_nan(fmaxf(p.mr, p.ml));
    // sums below the references (a: outside the list, b: the row)
    // (the gradient takes them in fp32, the loss in fp64 below)
    const float zrf = static_cast<float>(p.zr), zlf = static_cast<float>(p.zl);
    const float c2 = 2.f * c;
    const float za = warp_sum(zrf != 0.f ? zrf * ex2(half_diff(p.mr, a) * c2) : 0.f);
    const float zb = warp_sum((zrf != 0.f ? zrf * ex2(half_diff(p.mr, b) * c2) : 0.f) +
                              (zlf != 0.f ? zlf * ex2(half_diff(p.ml, b) * c2) : 0.f));
    uint32_t bad = __reduce_or_sync(0xffffffffu, p.bad) | (got ? 0u : 2u);
    if (!(zb > 0.f)) bad |= 1u;  // every logit masked, or NaN
    const bool empty = sh.any == 0u || (!tail && !(sh.s0 > 0.0));
    const bool live = fine && !bad && !empty;
    const bool outside = tail && za > 0.f;
    if (lane == 0) {
      DistillCtx k{};
      k.c = c;
      k.inv_t = 1.f / t;
      k.rall = b;
      k.lall = log2f(zb);
      k.ref = outside ? a : b;
      k.lz = outside ? log2f(za) : k.lall;
      k.coef = tail ? (outside ? static_cast<float>(static_cast<double>(exp2f(half_diff(a, b) * c2) * za / zb) - sh.at) : 0.f) : 1.f;
      k.tref = sh.tref;
      k.tnorm = tail ? 1.f : static_cast<float>(1.0 / sh.s0);
      k.zero = live ? 0u : 1u;
      k.dup = sh.dup;
      sh.k = k;
    }
    __syncwarp();
    if (GRAD) asm volatile("bar.arrive 1, %0;" ::"n"(kSThreads) : "memory");  // the other warps go on with the gradient
    if (rank == 0) {
      const double ad = static_cast<double>(a), bd = static_cast<double>(b);
      const double zad = warp_sum(p.zr != 0.0 ? p.zr * part_scale(p.mr, a, c, 0.f) : 0.0);
      const double zld = warp_sum(p.zl != 0.0 ? p.zl * exp2_below((static_cast<double>(p.ml) - bd) * cd) : 0.0);
      // sum of the teacher's weight times (l - b) c
      const double su = warp_sum(p.w > 0.0 ? p.wu + p.w * ((static_cast<double>(p.ml) - bd) * cd) : 0.0);
      const double lz = log2(zld + (zad > 0.0 ? zad * exp2_below((ad - bd) * cd) : 0.0));
      constexpr double kLn2d = 0.69314718055994530942;
      const double norm = tail ? 1.0 : 1.0 / sh.s0;  // a = w * norm
      double loss = (sh.t1 - sh.s0 * sh.tlog + kLn2d * (lz * sh.s0 - su)) * norm;
      if (tail && sh.at > 0.0 && zad > 0.0) {
        const double lq = (ad - bd) * cd + log2(zad) - lz;
        loss += sh.at * (log(sh.at) - kLn2d * lq);
      }
      if (lane == 0) {
        if (P.loss) P.loss[row] = (!fine || bad) ? __int_as_float(0x7FC00000) : (empty ? 0.f : static_cast<float>(loss));
        if (P.valid) P.valid[row] = live ? 1 : 0;
        if (P.status)
          P.status[row] = sh.status | (sh.dup ? VS_ROW_DUP_SUPPORT_ID : 0u) | (bad & 2u ? VS_ROW_DEVICE_TIMEOUT : 0u) |
                          (!fine ? VS_ROW_BAD_PARAM : bad ? VS_ROW_NONFINITE_INPUT : empty ? VS_ROW_EMPTY_SUPPORT : 0u);
        if (P.ctx) static_cast<DistillCtx*>(P.ctx)[row] = sh.k;
      }
    }
    __syncwarp();
  } else if (GRAD) {
    asm volatile("bar.sync 1, %0;" ::"n"(kSThreads) : "memory");
  }
  if constexpr (GRAD) {
    const DistillCtx k = sh.k;
    G* out = static_cast<G*>(P.dlogits) + static_cast<int64_t>(row) * P.grad_ld;
    const float scale = k.zero ? 0.f : (P.g_loss ? P.g_loss[row] : 1.f) * k.inv_t;
    const float dense = scale * k.coef;
    // one fused multiply-add per exponent: l c - (ref c + lz), the constant's rounding in the factor (at most
    // 2^(1/32): a larger constant's would overflow it, and there the differences come first)
    const double shift = static_cast<double>(k.ref) * k.c + static_cast<double>(k.lz);
    const float sf = static_cast<float>(shift);
    const bool wide = !(fabsf(sf) < 1048576.f);
    const float lead = wide ? dense : dense * exp2f(static_cast<float>(static_cast<double>(sf) - shift));
    const f32x2 c2 = pack2(k.c, k.c), s2 = pack2(-sf, -sf), d2 = pack2(lead, lead);
    for (int g = tid; g < groups; g += kSThreads) {
      Eight<Raw> v;
      v.load(buf + g * 8);
      float d[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float a, b;
        unpack2(fma2(pair_of(v, i), c2, s2), a, b);
        unpack2(mul2(pack2(ex2(a), ex2(b)), d2), d[2 * i], d[2 * i + 1]);
      }
      if (k.zero || wide) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          d[i] = k.zero ? 0.f : dense * ex2(fmaf(half_diff(value_of(v.e[i]), k.ref), 2.f * k.c, -k.lz));
      }
      const int j = j0 + g * 8;
      if (j + 8 <= j1) {
        Eight<G> o;
#pragma unroll
        for (int i = 0; i < 8; ++i) o.e[i] = to_grad<G>(d[i]);
        o.store(out + j);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (j + i < j1) out[j + i] = to_grad<G>(d[i]);
      }
    }
    cta_sync();
    if (!k.zero)
      for (int s = tid; s < W; s += kSThreads) {
        const int id = ids[s];
        if (id >= j0 && id < j1)
          out[id] = to_grad<G>(scale * (ex2(fmaf(half_diff(us[s], sh.k.rall), 2.f * sh.k.c, -sh.k.lall)) -
                                        sh.k.tnorm * expf(lps[s] - sh.k.tref)));
      }
  }
}

// Elementwise but for the list: bound by HBM.  4,096 x 151,936 bf16 in about 423
// us, 5.9 TB/s of reads and writes (a copy runs at 6.5).
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

}  // namespace

template <typename Raw, typename G, bool GRAD>
static cudaError_t launch_any(DistillParams P, cudaStream_t s) {
  const int c = stage_cluster_size(P.rows, P.vocab, sizeof(Raw));
  if (c == 0) {
    const int f = row_cluster_size(P.rows, P.vocab);
    P.chunk = ((P.vocab + f - 1) / f + 31) / 32 * 32;
    const size_t smem = sizeof(DistillShared) + (static_cast<size_t>(P.vocab) + 127) / 128 * 16;
    return launch_cluster<distill_fwd_kernel<Raw, G, GRAD>>(static_cast<unsigned>(P.rows) * f, f, kDThreads, smem,
                                                            false, s, P);
  }
  P.chunk = ((P.vocab + c - 1) / c + 31) / 32 * 32;
  const size_t smem = stage_fixed(P.width) + static_cast<size_t>(P.chunk) * sizeof(Raw);
  return launch_cluster<distill_stage_kernel<Raw, G, GRAD>>(static_cast<unsigned>(P.rows) * c, c, kSThreads, smem,
                                                            false, s, P);
}

cudaError_t launch_distill_fwd(DistillParams P, vs_dtype dtype, vs_dtype dl_dtype, cudaStream_t s) {
  const bool grad = P.dlogits != nullptr, half = dl_dtype == VS_BF16;
  if (dtype == VS_BF16) {
    if (!grad) return launch_any<uint16_t, float, false>(P, s);
    return half ? launch_any<uint16_t, uint16_t, true>(P, s) : launch_any<uint16_t, float, true>(P, s);
  }
  if (!grad) return launch_any<uint32_t, float, false>(P, s);
  return half ? launch_any<uint32_t, uint16_t, true>(P, s) : launch_any<uint32_t, float, true>(P, s);
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
