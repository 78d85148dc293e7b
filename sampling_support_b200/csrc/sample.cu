// vs_sample: one token per row from a given uniform number.
//
// With w_j = exp((l_j - max l) / T) and the row in the library's total order
// (logit descending, token id ascending), C_i the running sum of w:
//   n_k = top_k, n_p = the first i with C_i >= top_p C_{n_k},
//   n_m = the number of tokens with w >= min_p;  the support is the first
//   n = min(n_k, n_p, n_m) tokens;
//   token = the first i with C_i > u C_n,  logprob = log(w_i / C_n).
#include "internal.h"
#include "row_select.cuh"

namespace vs {

namespace {

// Largest top-k taken through the list of candidates above a floor (the
// k-th largest of the threads' maxima needs k of the 1,024 threads).
constexpr int kListTopK = 512;

__device__ __forceinline__ void write_none(const SampleParams& P, int row, uint32_t status) {
  P.token[row] = -1;
  if (P.logprob) P.logprob[row] = __int_as_float(0x7FC00000);
  if (P.support_size) P.support_size[row] = 0;
  if (P.status) P.status[row] = status;
}

__device__ __forceinline__ void write_row(const SampleParams& P, int row, double z, u64 mass, u64 n,
                                          const RsMass& M) {
  if (P.logprob) P.logprob[row] = static_cast<float>(z - log(static_cast<double>(mass) / M.scale));
  if (P.support_size) P.support_size[row] = static_cast<int32_t>(n);
  if (P.status) P.status[row] = 0u;
}

// The running mass that the row's number asks for: the first integer above
// u * mass, at most the mass itself (u = 1 takes the last token).
__device__ __forceinline__ u64 draw_target(float u, u64 mass) {
  const double x = floor(static_cast<double>(u) * static_cast<double>(mass));
  const u64 t = x >= static_cast<double>(mass) ? mass : static_cast<u64>(x) + 1ull;
  return t < mass ? t : mass;
}

template <typename Raw>
__global__ void __launch_bounds__(kRsThreads, 1) sample_kernel(SampleParams P) {
  extern __shared__ __align__(16) unsigned char rs_smem[];
  RsShared& sh = *reinterpret_cast<RsShared*>(rs_smem);
  __shared__ u64 s_mass;
  RsRow<Raw> R;
  const int row = static_cast<int>(blockIdx.x / cg::this_cluster().num_blocks());
  R.init(P.logits, row, P.ld, P.vocab, &sh);
  const bool lead = R.rank == 0 && threadIdx.x == 0;

  float t = P.temperature ? P.temperature[row] : P.temperature_scalar;
  int k = P.top_k ? P.top_k[row] : P.top_k_scalar;
  float p = P.top_p ? P.top_p[row] : P.top_p_scalar;
  float m = P.min_p ? P.min_p[row] : P.min_p_scalar;
  const float u = P.uniform[row];
  const bool fine = t >= 0.f && t < kInf && p > 0.f && m <= 1.f && u >= 0.f && u <= 1.f;

  uint32_t kmax, kmin, thread_max;
  const bool finite = rs_extremes(R, kmax, kmin, thread_max);
  if (!finite || !fine || kmax <= RsRow<Raw>::kMaskedKey) {
    if (lead)
      write_none(P, row, (finite ? 0u : VS_ROW_NONFINITE_INPUT) | (fine ? 0u : VS_ROW_BAD_PARAM) |
                             (finite && kmax <= RsRow<Raw>::kMaskedKey ? VS_ROW_EMPTY_SUPPORT : 0u));
    R.sync();  // peers read this CTA's extremes
    return;
  }
  if (t == 0.f) {  // greedy: the first token of the order
    t = 1.f;
    k = 1;
    p = 1.f;
    m = 0.f;
  }
  RsMass M;
  M.vmax = static_cast<double>(KeyTraits<Raw>::decode(kmax));
  M.inv_t = 1.0 / static_cast<double>(t);
  M.scale = static_cast<double>(1ull << P.fx_shift);

  if (k > 0 && k < P.vocab && k <= kListTopK) {
    const uint32_t floor_key = max(rs_topk_floor(R, thread_max, k), RsRow<Raw>::kMaskedKey + 1u);
    const uint32_t n_list = rs_collect(R, floor_key, kmax);
    if (n_list <= static_cast<uint32_t>(kRsCap)) {
      if (R.rank == 0) {
        const uint32_t nk = min(static_cast<uint32_t>(k), n_list);
        rs_sort(sh, n_list, nk);
        const uint32_t i = threadIdx.x;
        float v = 0.f;
        u64 w = 0ull;
        double wd = 0.0;
        if (i < nk) {
          v = KeyTraits<Raw>::decode(static_cast<uint32_t>(sh.sorted[i] >> 32));
          wd = exp(M.z(v));
          w = M.fx(v);
        }
        u64 upto, none;
        rs_scan(w, 0ull, upto, none, sh);
        upto += w;
        if (i == nk - 1) s_mass = upto;
        cta_sync();
        const u64 zk = s_mass;
        uint32_t n = nk;
        if (p < 1.f) {
          const u64 want = topp_target(p, static_cast<double>(zk));
          n = min(n, static_cast<uint32_t>(__syncthreads_count(i < nk && upto < want)) + 1u);
        }
        if (m > 0.f)
          n = min(n, static_cast<uint32_t>(__syncthreads_count(i < nk && wd >= static_cast<double>(m))));
        cta_sync();
        if (i == n - 1) s_mass = upto;
        cta_sync();
        const u64 zs = s_mass, want = draw_target(u, zs);
        if (i < n && upto - w < want && want <= upto) {
          P.token[row] = static_cast<int32_t>(~static_cast<uint32_t>(sh.sorted[i]));
          write_row(P, row, M.z(v), zs, n, M);
        }
      }
      return;  // rs_collect ended with a cluster barrier: nothing is read from peers after it
    }
  }

  RsBins B;
  B.vmax = KeyTraits<Raw>::decode(kmax);
  {
    // bins over the values whose mass is not zero in fixed point (46 nats), or over the row's own range
    const float range = fminf(B.vmax - KeyTraits<Raw>::decode(kmin), 46.f * t);
    B.s = range > 0.f ? fminf(static_cast<float>(kRsBins - 1) / range, 1e38f) : 0.f;
  }
  rs_hist(R, M, kRsBins, sh.rcnt, sh.rmass, [&](uint32_t, float v) { return B.of(v); });
  const RsMsg all = R.broadcast([&](RsMsg* msg) {
    if (threadIdx.x == 0) {
      msg->cnt = sh.rcnt[kRsBins - 1];
      msg->mass = sh.rmass[kRsBins - 1];
    }
  });
  u64 n = all.cnt, mass = all.mass;
  uint32_t last = kmin;  // the key that the support reaches down to
  if (k > 0 && static_cast<u64>(k) < n) {
    const RsHit h = rs_find(R, M, B, kmin, kmax, false, static_cast<u64>(k));
    n = h.cnt;
    mass = h.mass;
    last = h.key;
  }
  if (p < 1.f) {
    const RsHit h = rs_find(R, M, B, kmin, kmax, true, topp_target(p, static_cast<double>(mass)));
    if (h.cnt < n) {
      n = h.cnt;
      mass = h.mass;
      last = h.key;
    }
  }
  if (m > 0.f) {
    uint32_t lo = kmin, hi = kmax;  // the smallest key with w >= min_p
    while (lo < hi) {
      const uint32_t mid = lo + ((hi - lo) >> 1);
      if (exp(M.z(KeyTraits<Raw>::decode(mid))) >= static_cast<double>(m))
        hi = mid;
      else
        lo = mid + 1;
    }
    if (lo > last) {
      u64 cnt, above;
      rs_sum_above(R, M, lo, cnt, above);
      if (cnt < n) {
        n = cnt;
        mass = above;
      }
    }
  }
  const RsHit h = rs_find(R, M, B, kmin, kmax, true, draw_target(u, mass));
  if (h.tie)
    rs_ties(R, h.key, h.tie, [&](int id, u64 at) {
      if (at == h.tie - 1) P.token[row] = id;
    });
  if (lead) {
    if (!h.tie) P.token[row] = h.id;
    write_row(P, row, M.z(KeyTraits<Raw>::decode(h.key)), mass, n, M);
  }
  R.sync();  // peers may still read this CTA's words
}

}  // namespace

// Cluster size for `rows` rows of `vocab` elements: as many CTAs per row as
// the GPU's SMs hold at once, with at least 4,096 elements for each.
int row_cluster_size(int rows, int vocab) {
  int c = 1;
  while (c < kRsMaxCluster && 2ll * c * rows <= 148 && vocab / (2 * c) >= 4096) c *= 2;
  return c;
}

template <typename K, typename Params>
static cudaError_t launch_row(K kernel, const Params& P, cudaStream_t s) {
  const int c = row_cluster_size(P.rows, P.vocab);
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(sizeof(RsShared)));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(P.rows) * c);
  cfg.blockDim = dim3(kRsThreads);
  cfg.dynamicSmemBytes = sizeof(RsShared);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = c;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P);
}

cudaError_t launch_sample(const SampleParams& P, vs_dtype dtype, cudaStream_t s) {
  return dtype == VS_BF16 ? launch_row(sample_kernel<uint16_t>, P, s)
                          : launch_row(sample_kernel<uint32_t>, P, s);
}

namespace {

// vs_topk_logprob: the first k tokens of each row in the total order and
// their log-probabilities  z_j - log sum_i exp z_i,  z = l / T.
template <typename Raw>
__global__ void __launch_bounds__(kRsThreads, 1) topk_kernel(TopkParams P) {
  extern __shared__ __align__(16) unsigned char rs_smem[];
  RsShared& sh = *reinterpret_cast<RsShared*>(rs_smem);
  RsRow<Raw> R;
  const int row = static_cast<int>(blockIdx.x / cg::this_cluster().num_blocks());
  R.init(P.logits, row, P.ld, P.vocab, &sh);
  int32_t* ids = P.ids + static_cast<int64_t>(row) * P.out_ld;
  float* lps = P.logprob ? P.logprob + static_cast<int64_t>(row) * P.out_ld : nullptr;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float t = P.temperature ? P.temperature[row] : P.temperature_scalar;
  const bool fine = t > 0.f && t < kInf;

  uint32_t kmax, kmin, thread_max;
  const bool finite = rs_extremes(R, kmax, kmin, thread_max);
  const bool empty = finite && kmax <= RsRow<Raw>::kMaskedKey;
  if (!finite || !fine || empty) {
    if (R.rank == 0) {
      if (tid < P.k) {
        ids[tid] = -1;
        if (lps) lps[tid] = empty && fine ? -kInf : __int_as_float(0x7FC00000);
      }
      if (tid == 0 && P.status)
        P.status[row] = (finite ? 0u : VS_ROW_NONFINITE_INPUT) | (fine ? 0u : VS_ROW_BAD_PARAM) |
                        (empty ? VS_ROW_EMPTY_SUPPORT : 0u);
    }
    R.sync();
    return;
  }
  const float vmax = KeyTraits<Raw>::decode(kmax);

  // sum of 2^((l - max) log2(e) / T): fp32 per thread, fixed order across
  // the threads and the cluster
  const float c = kLog2e / t;
  if (lps) {
    float z = 0.f;
    R.each([&](int, const auto& r) {
#pragma unroll
      for (int i = 0; i < RsRow<Raw>::VEC; ++i) z += ex2((value_of(r[i]) - vmax) * c);
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    if (lane == 0) sh.fred[warp] = z;
    cta_sync();
    if (warp == 0) {
      z = sh.fred[lane];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
      if (lane == 0) sh.xf[0] = z;
    }
  }

  uint32_t n = 0u, nk = 0u;
  const uint32_t floor_key = max(rs_topk_floor(R, thread_max, P.k), RsRow<Raw>::kMaskedKey + 1u);
  n = rs_collect(R, floor_key, kmax);
  if (n > static_cast<uint32_t>(kRsCap)) {
    // too many elements share the floor: the k-th element exactly, then the
    // elements above it and its first equals
    RsMass M;
    M.vmax = static_cast<double>(vmax);
    M.inv_t = 1.0 / static_cast<double>(t);
    M.scale = static_cast<double>(1ull << P.fx_shift);
    RsBins B;
    B.vmax = vmax;
    const float range = B.vmax - KeyTraits<Raw>::decode(kmin);
    B.s = range > 0.f ? fminf(static_cast<float>(kRsBins - 1) / range, 1e38f) : 0.f;
    rs_hist(R, M, kRsBins, sh.rcnt, sh.rmass, [&](uint32_t, float v) { return B.of(v); });
    const RsHit h = rs_find(R, M, B, kmin, kmax, false, static_cast<u64>(P.k));
    n = h.key < kmax ? rs_collect(R, h.key + 1u, kmax) : 0u;
    u64* list = R.peer(sh.list, 0);
    rs_ties(R, h.key, static_cast<u64>(P.k) - n, [&](int id, u64 at) {
      list[n + at] = (static_cast<u64>(h.key) << 32) | static_cast<uint32_t>(~id);
    });
    n = static_cast<uint32_t>(P.k);
    R.sync();
  }
  nk = min(static_cast<uint32_t>(P.k), n);
  if (R.rank == 0) {
    float z = 0.f;
    if (lps)
      for (int r = 0; r < R.C; ++r) z += R.peer(sh.xf, r)[0];
    rs_sort(sh, n, nk);
    if (tid < P.k) {
      const bool in = static_cast<uint32_t>(tid) < nk;
      const u64 e = in ? sh.sorted[tid] : 0ull;
      ids[tid] = in ? static_cast<int32_t>(~static_cast<uint32_t>(e)) : -1;
      if (lps)
        lps[tid] = in ? (KeyTraits<Raw>::decode(static_cast<uint32_t>(e >> 32)) - vmax) / t - logf(z) : -kInf;
    }
    if (tid == 0 && P.status) P.status[row] = 0u;
  }
  R.sync();  // the leader reads the peers' sums
}

}  // namespace

cudaError_t launch_topk(const TopkParams& P, vs_dtype dtype, cudaStream_t s) {
  return dtype == VS_BF16 ? launch_row(topk_kernel<uint16_t>, P, s)
                          : launch_row(topk_kernel<uint32_t>, P, s);
}

}  // namespace vs
