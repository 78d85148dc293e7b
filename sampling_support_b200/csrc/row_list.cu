// Rows whose answer lies in their first k tokens: the list kernel behind
// vs_topk_logprob and behind vs_sample's rows with a small top-k.
//
// A cluster stages the row in its CTAs' shared memory (one bulk copy per
// slice, so the row is read from HBM once) and finds a floor that at least k
// elements reach: every thread's two largest group maxima are elements of their own,
// (all elements of a slice that is short) so a value that k of any CTA's maxima reach is a floor, and so is the smallest
// over the CTAs of values that ceil(k / C) of theirs reach.  The elements from the floor
// up (hardly more than k) are listed, gathered by the leader and sorted there.
// Top-k adds the row's sum of exponentials, taken in the same pass as the
// maxima; sampling cuts and draws from the sorted masses.
//
// Bound: a CTA holds its shared memory for several microseconds of mostly
// latency (copy, floor, exchange, listing), so with 40 KB slices and five CTAs
// per SM the rate is that of the slots: 191 us for k 64 of 2,048 x 151,936 bf16
// (3.3 TB/s), 16.6 us for k 257 of 61 x 50,021 fp32, 8 us for a call of a few
// rows, which is launch and latency.  No cluster barrier is waited for: the
// floors and the first listed elements of every CTA are pushed, and a CTA
// leaves once they are sent unless it has listed more.  Where the list
// overflows (crowds of equal values) the leader alone selects by digits of the
// key from the row in L2: some passes of one CTA, for rows that are rare.
#include <stddef.h>

#include <algorithm>

#include "internal.h"
#include "row_stage.cuh"
#include "select.cuh"

namespace vs {

namespace {

constexpr int kLThreads = 256;
constexpr int kLWarps = kLThreads / 32;
constexpr int kLMaxCluster = 8;
constexpr int kLTotal = 4096;  // listed elements per row, at most
constexpr int kLBins = 512;    // of the vector maxima, linear in the value below the largest
constexpr int kLShort = 4096;  // a slice of at most so many elements can bin them all
// Listed elements per CTA: 256 keep five CTAs on an SM, wide lists take 1,024
// (a CTA that lists alone holds k and what shares its floor's bin).
__host__ __device__ inline int list_local(int k, int c) { return k <= (c > 1 ? 256 : 192) ? 256 : 1024; }

struct alignas(16) ListPart {
  uint32_t kmax;         // largest key
  uint32_t kth, share;   // floors that k and ceil(k / C) of the maxima reach
  float m, z;            // sum of 2^((l - m) c)
  uint32_t pad[3];
};

// What a CTA pushes of its list: its length and its first elements, the rest
// (if any) stays for the leader to fetch.
constexpr int kLPush = 62;
struct alignas(16) ListPush {
  uint32_t n, pad[3];
  u64 e[kLPush];
};
static_assert(sizeof(ListPush) == 32 * 16, "one 16-byte store per lane");

struct alignas(16) ListStage {
  ListPart parts[kLMaxCluster];
  union {
    ListPush pushed[kLMaxCluster];  // leader: from the CTA of each rank
    struct {                        // before that: no CTA lists before it has this one's part
      uint32_t bins[kLBins];        // maxima per bin, and the smallest key of each
      uint32_t least[kLBins];
    };
  };
  ListPush mine;
  uint64_t bar, xbar, lbar, fbar;  // the slice's copy; the parts; the lists; (listed more) the leader has fetched
  uint64_t gbar[kLMaxCluster];     // leader: the rest of that CTA's list is written
  float2 red[kLWarps];
  uint32_t rmax[kLWarps], rmin[kLWarps];
  uint32_t bad;
};

// Shared memory behind it: this CTA's list (key << 32 | ~id) beyond mine.e,
// then the slice, later the leader's list and its sorted copy.
__host__ __device__ inline int list_total(int c, int local) { return c * local < kLTotal ? c * local : kLTotal; }
__host__ __device__ inline size_t list_more(int local) { return static_cast<size_t>(local - kLPush + 1) / 2 * 16; }
__host__ __device__ inline size_t list_room(int c, int local, size_t slice) {
  const size_t lists = static_cast<size_t>(list_total(c, local) + kListTopK) * sizeof(u64);
  return list_more(local) + (slice > lists ? slice : lists);
}

template <typename Raw>
struct ListKey {
  static constexpr uint32_t kMasked = sizeof(Raw) == 2 ? 0x007Fu : 0x007FFFFFu;  // key of -inf
  __device__ __forceinline__ static uint32_t of(float v) {
    return sizeof(Raw) == 2 ? key_of(static_cast<uint16_t>(__float_as_uint(v) >> 16)) : key_of(__float_as_uint(v));
  }
};

// One warp: the bin in which the running count of the block's maxima reaches k
// (lane l holds the counts c of kLBins / 32 bins, upto the sum through them);
// -1 when there are fewer.
__device__ __forceinline__ int bin_reaching(uint32_t upto, uint32_t mine, const uint32_t (&c)[kLBins / 32], uint32_t k) {
  const uint32_t hit = __ballot_sync(0xffffffffu, upto >= k);
  if (!hit) return -1;
  const int l = __ffs(hit) - 1;
  uint32_t run = upto - mine;
  int b = 0;
#pragma unroll
  for (int i = 0; i < kLBins / 32; ++i) {
    run += c[i];
    if (run < k) b = i + 1;
  }
  return __shfl_sync(0xffffffffu, b, l) + l * (kLBins / 32);
}

// Brings a list of n > 1,024 elements down to its largest, at least `keep` and
// at most 1,024 of them, in place: the smallest of those from counts over the
// words' range, 1,024 bins at a time, zooming into the bin that `keep` falls
// in as long as it holds too many (the words differ, so one of them does not).
// Returns how many stay.  Long lists come from vocabularies of a few thousand
// tokens with a k of that order, where the maxima give no floor: sorting 4,096
// elements there took most of 127 us (58 x 2,876 bf16, k 727).
__device__ __noinline__ uint32_t list_shrink(u64* list, uint32_t n, uint32_t keep, ListStage& sh) {
  constexpr int kBins = 2 * kLBins, kMost = 4 * kLThreads;
  static_assert(kBins == 1024 && offsetof(ListStage, least) == offsetof(ListStage, bins) + sizeof(sh.bins), "one array");
  uint32_t* bins = sh.bins;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t kmax = 0u, kmin = 0xFFFFFFFFu;
  for (uint32_t i = tid; i < n; i += kLThreads) {
    const uint32_t k = static_cast<uint32_t>(list[i] >> 32);
    kmax = max(kmax, k);
    kmin = min(kmin, k);
  }
  kmax = __reduce_max_sync(0xffffffffu, kmax);
  kmin = __reduce_min_sync(0xffffffffu, kmin);
  cta_sync();
  if (lane == 0) {
    sh.rmax[warp] = kmax;
    sh.rmin[warp] = kmin;
  }
  cta_sync();
  kmax = __reduce_max_sync(0xffffffffu, lane < kLWarps ? sh.rmax[lane] : 0u);
  kmin = __reduce_min_sync(0xffffffffu, lane < kLWarps ? sh.rmin[lane] : 0xFFFFFFFFu);
  u64 hi = static_cast<u64>(kmax) << 32 | 0xFFFFFFFFull, lo = static_cast<u64>(kmin) << 32;
  uint32_t before = 0u;  // elements above hi
  for (;;) {
    const int shift = max(0, 64 - __clzll(hi - lo) - 10);
    cta_sync();
    for (int i = tid; i < kBins; i += kLThreads) bins[i] = 0u;
    cta_sync();
    for (uint32_t i = tid; i < n; i += kLThreads) {
      const u64 w = list[i];
      if (w >= lo && w <= hi) atomicAdd(&bins[(hi - w) >> shift], 1u);
    }
    cta_sync();
    // every warp: first the 32 bins, then the one of them, in which the count reaches `keep`
    uint32_t sum = 0u;
#pragma unroll 8
    for (int i = 0; i < 32; ++i) sum += bins[lane * 32 + (i ^ lane)];
    uint32_t upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t a = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += a;
    }
    const int l = __ffs(__ballot_sync(0xffffffffu, before + upto >= keep) | 0x80000000u) - 1;
    before += __shfl_sync(0xffffffffu, upto - sum, l);
    const uint32_t c = bins[l * 32 + lane];
    uint32_t run = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t a = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += a;
    }
    const int b = __ffs(__ballot_sync(0xffffffffu, before + run >= keep) | 0x80000000u) - 1;
    const uint32_t through = before + __shfl_sync(0xffffffffu, run, b);
    before += __shfl_sync(0xffffffffu, run - c, b);
    hi -= static_cast<u64>(l * 32 + b) << shift;
    const u64 width = (1ull << shift) - 1ull;
    lo = hi - lo > width ? hi - width : lo;
    if (through <= static_cast<uint32_t>(kMost) || shift == 0) break;
  }
  // the elements from lo up, to the front: a round of them is read before its places are written
  if (tid == 0) sh.bad = 0u;
  for (uint32_t i0 = 0; i0 < n; i0 += kLThreads) {
    const u64 w = i0 + tid < n ? list[i0 + tid] : 0ull;
    cta_sync();
    const bool in = i0 + tid < n && w >= lo;
    const uint32_t at = in ? atomicAdd(&sh.bad, 1u) : 0u;
    if (in && at < static_cast<uint32_t>(kMost)) list[at] = w;
  }
  cta_sync();
  return min(sh.bad, static_cast<uint32_t>(kMost));
}

// The n listed elements in descending order at `out` (the first `keep`; room
// for kListTopK) or, for more than a block's worth, sorted in place.  Returns
// where they are.
__device__ __forceinline__ u64* list_sort(u64* list, u64* out, uint32_t n, uint32_t keep, ListStage& sh) {
  if (n <= kLThreads) {
    int bits = 3;
    while ((1u << bits) < n) ++bits;
    const int g = kLThreads >> bits;  // neighbouring lanes that share an element
    const uint32_t at = threadIdx.x / g;
    const u64 e = at < n ? list[at] : 0ull;
    uint32_t place = 0u;
    for (uint32_t o = threadIdx.x & (g - 1); o < n; o += g) place += list[o] > e ? 1u : 0u;
    for (int o = 1; o < g; o <<= 1) place += __shfl_xor_sync(0xffffffffu, place, o);
    if (at < n && (threadIdx.x & (g - 1)) == 0 && place < keep) out[place] = e;
    cta_sync();
    return out;
  }
  if (n > 4 * kLThreads) n = list_shrink(list, n, keep, sh);
  if (n <= 2 * kLThreads)
    block_sort<kLThreads, 2>(list, list, n);
  else
    block_sort<kLThreads, 4>(list, list, n);
  return list;
}
static_assert(kLThreads <= kListTopK && 4 * kLThreads >= VS_MAX_TOPK && 4 * kLThreads >= kListTopK,
              "the sorted copy's room, and what is sorted in place");

// vs_topk_logprob: rows[k] ids and log-probabilities.
struct TopkOp {
  using Params = TopkParams;
  static constexpr bool kSum = true;
  __device__ __forceinline__ static int k_of(const Params& P, int) { return P.k; }
  static int most(const Params& P) { return P.k; }
  __device__ __forceinline__ static float t_of(const Params& P, int row) {
    return P.temperature ? P.temperature[row] : P.temperature_scalar;
  }
  __device__ __forceinline__ static bool fine(const Params& P, int row) {
    const float t = t_of(P, row);
    return t >= kLeastT && t < kInf;
  }
  // no list: bad input, or every token masked
  __device__ __forceinline__ static void none(const Params& P, int row, uint32_t status) {
    int32_t* ids = P.ids + static_cast<int64_t>(row) * P.out_ld;
    float* lps = P.logprob ? P.logprob + static_cast<int64_t>(row) * P.out_ld : nullptr;
    const float lp = status == VS_ROW_EMPTY_SUPPORT ? -kInf : __int_as_float(0x7FC00000);
    for (int i = threadIdx.x; i < P.k; i += kLThreads) {
      ids[i] = -1;
      if (lps) lps[i] = lp;
    }
    if (threadIdx.x == 0 && P.status) P.status[row] = status;
  }
  template <typename Raw>
  __device__ __forceinline__ static void finish(const Params& P, int row, u64* sorted, u64*, uint32_t nk, float vmax,
                                                float z) {
    int32_t* ids = P.ids + static_cast<int64_t>(row) * P.out_ld;
    float* lps = P.logprob ? P.logprob + static_cast<int64_t>(row) * P.out_ld : nullptr;
    const float t = t_of(P, row), lz = logf(z);
    for (int i = threadIdx.x; i < P.k; i += kLThreads) {
      const bool in = static_cast<uint32_t>(i) < nk;
      const u64 e = in ? sorted[i] : 0ull;
      ids[i] = in ? static_cast<int32_t>(~static_cast<uint32_t>(e)) : -1;
      if (lps)
        lps[i] = in ? 2.f * (half_diff(KeyTraits<Raw>::decode(static_cast<uint32_t>(e >> 32)), vmax) / t) - lz : -kInf;
    }
    if (threadIdx.x == 0 && P.status) P.status[row] = 0u;
  }
};

// vs_sample's rows with a small top-k (greedy rows among them).
struct SampleOp {
  using Params = SampleParams;
  static constexpr bool kSum = false;
  static int most(const Params& P) { return P.top_k ? kListTopK : sample_list_k(P.vocab, 1.f, P.top_k_scalar); }
  __device__ __forceinline__ static float t_of(const Params& P, int row) {
    return P.temperature ? P.temperature[row] : P.temperature_scalar;
  }
  __device__ __forceinline__ static int k_of(const Params& P, int row) {
    return sample_list_k(P.vocab, t_of(P, row), P.top_k ? P.top_k[row] : P.top_k_scalar);
  }
  __device__ __forceinline__ static bool fine(const Params& P, int row) {
    const float t = t_of(P, row), p = P.top_p ? P.top_p[row] : P.top_p_scalar, m = P.min_p ? P.min_p[row] : P.min_p_scalar;
    const float u = P.uniform[row];
    return t >= 0.f && t < kInf && p > 0.f && m <= 1.f && u >= 0.f && u <= 1.f;
  }
  __device__ __forceinline__ static void none(const Params& P, int row, uint32_t status) {
    if (threadIdx.x != 0) return;
    P.token[row] = -1;
    if (P.logprob) P.logprob[row] = __int_as_float(0x7FC00000);
    if (P.support_size) P.support_size[row] = 0;
    if (P.status) P.status[row] = status;
  }
  // masses: room for nk words
  template <typename Raw>
  __device__ __forceinline__ static void finish(const Params& P, int row, u64* sorted, u64* masses, uint32_t nk,
                                                float vmax, float) {
    float t = t_of(P, row), p = P.top_p ? P.top_p[row] : P.top_p_scalar, m = P.min_p ? P.min_p[row] : P.min_p_scalar;
    if (t == 0.f) {
      t = 1.f;
      p = 1.f;
      m = 0.f;
    }
    RowMass M;
    M.set(vmax, t, P.fx_shift);
    auto value = [&](uint32_t i) { return KeyTraits<Raw>::decode(static_cast<uint32_t>(sorted[i] >> 32)); };
    for (uint32_t i = threadIdx.x; i < nk; i += kLThreads) masses[i] = M.fixed(value(i), [](int j) { return exp2_64th(j); });
    cta_sync();
    if (threadIdx.x >= 32) return;
    const int lane = threadIdx.x;
    // the first of n elements at which the running mass reaches want; sum: the mass through it
    auto cross = [&](uint32_t n, u64 want, u64& sum) {
      sum = 0ull;
      for (uint32_t i0 = 0; i0 < n; i0 += 32) {
        u64 s = i0 + lane < n ? masses[i0 + lane] : 0ull;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const u64 x = __shfl_up_sync(0xffffffffu, s, o);
          if (lane >= o) s += x;
        }
        s += sum;
        const uint32_t hit = __ballot_sync(0xffffffffu, i0 + lane < n && s >= want);
        if (hit) {
          const int l = __ffs(hit) - 1;
          sum = __shfl_sync(0xffffffffu, s, l);
          return i0 + l;
        }
        sum = __shfl_sync(0xffffffffu, s, 31);
      }
      return n - 1;
    };
    u64 mass;
    uint32_t n = nk;
    cross(n, ~0ull, mass);  // never reached: the total
    if (p < 1.f) n = cross(nk, topp_target(p, static_cast<double>(mass)), mass) + 1u;
    if (m > 0.f) {
      uint32_t keep = 0u;  // the order is by mass: those kept are the first ones
      for (uint32_t i = lane; i < n; i += 32) keep += M.reaches(value(i), m) ? 1u : 0u;
      n = __reduce_add_sync(0xffffffffu, keep);
      cross(n, ~0ull, mass);
    }
    u64 upto;
    const float u = P.uniform[row];
    const uint32_t at = u < 1.f ? cross(n, draw_target(u, mass), upto) : n - 1u;
    if (lane == 0) {
      P.token[row] = static_cast<int32_t>(~static_cast<uint32_t>(sorted[at]));
      if (P.logprob) P.logprob[row] = M.logprob(value(at), mass);
      if (P.support_size) P.support_size[row] = static_cast<int32_t>(n);
      if (P.status) P.status[row] = 0u;
    }
  }
};

// Wait (bounded) for a peer's release on this barrier's first phase.
__device__ __forceinline__ void wait_cluster(uint64_t* bar) {
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], 0;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_addr(bar))
        : "memory");
    if (ok) return;
  }
}

// f(first id, eight elements, those past the vocabulary masked) over the whole
// row in order, block by block of 8 kLThreads elements; the block's threads all
// call f (it may hold barriers) until it returns false in all of them.
template <typename Raw, typename F>
__device__ __forceinline__ void whole_row(const Raw* x, int vocab, F&& f) {
  constexpr Raw kMaskedRaw = static_cast<Raw>(sizeof(Raw) == 2 ? 0xFF80u : 0xFF800000u);
  for (int b = 0; b < vocab; b += 8 * kLThreads) {
    const int j = b + static_cast<int>(threadIdx.x) * 8;
    Eight<Raw> v;
    if (j + 8 <= vocab)
      v.load(x + j);
    else
#pragma unroll
      for (int i = 0; i < 8; ++i) v.e[i] = j + i < vocab ? x[j + i] : kMaskedRaw;
    if (!f(j, v)) return;
  }
}

// The leader alone, whole block: the row's first k tokens (it has more) into
// list, in any order.  The k-th key digit by digit, eight bits at a time, then
// the elements above it and its first equals.
template <typename Raw>
__device__ __noinline__ void list_by_digits(const Raw* x, int vocab, int k, u64* list, ListStage& sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t prefix = 0u, mask = 0u, need = static_cast<uint32_t>(k);
  for (int shift = KeyTraits<Raw>::kBits - 8; shift >= 0; shift -= 8) {
    cta_sync();
    if (tid < 256) sh.bins[tid] = 0u;
    cta_sync();
    whole_row(x, vocab, [&](int, const Eight<Raw>& v) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t key = key_of(v.e[i]);
        if (key > ListKey<Raw>::kMasked && (key & mask) == prefix) atomicAdd(&sh.bins[key >> shift & 255u], 1u);
      }
      return true;
    });
    cta_sync();
    // every warp: lane l holds the digits 255 - 8 l and down
    uint32_t c[8], sum = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = sh.bins[255 - 8 * lane - i];
      sum += c[i];
    }
    uint32_t upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t a = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += a;
    }
    const int l = __ffs(__ballot_sync(0xffffffffu, upto >= need) | 0x80000000u) - 1;
    uint32_t run = upto - sum, digit = 255u - 8u * lane, above = run;
    bool done = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      run += c[i];
      if (!done && run < need) {
        above = run;
        --digit;
      } else {
        done = true;
      }
    }
    need -= __shfl_sync(0xffffffffu, above, l);
    prefix |= (__shfl_sync(0xffffffffu, digit, l) & 255u) << shift;
    mask |= 255u << shift;
  }
  // need: how many of the key's own elements belong
  const uint32_t n_above = static_cast<uint32_t>(k) - need;
  cta_sync();
  if (tid == 0) sh.bins[0] = 0u;
  cta_sync();
  uint32_t taken = 0u;  // equals so far
  whole_row(x, vocab, [&](int j, const Eight<Raw>& v) {
    uint32_t eq = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t key = key_of(v.e[i]);
      if (key > prefix) {
        const uint32_t at = atomicAdd(&sh.bins[0], 1u);
        if (at < n_above) list[at] = static_cast<u64>(key) << 32 | static_cast<uint32_t>(~(j + i));
      }
      eq |= key == prefix ? 1u << i : 0u;
    }
    if (taken >= need) return true;  // the same in every thread
    uint32_t before = __popc(eq);
    const uint32_t mine = before;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t a = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += a;
    }
    cta_sync();
    if (lane == 31) sh.rmax[warp] = before;
    cta_sync();
    const uint32_t w = lane < kLWarps ? sh.rmax[lane] : 0u;
    const uint32_t all = __reduce_add_sync(0xffffffffu, w);
    uint32_t at = taken + before - mine + __reduce_add_sync(0xffffffffu, lane < warp ? w : 0u);
    for (; eq; eq &= eq - 1u, ++at)
      if (at < need) list[n_above + at] = static_cast<u64>(prefix) << 32 | static_cast<uint32_t>(~(j + __ffs(eq) - 1));
    taken += all;
    return true;
  });
  cta_sync();
}

template <typename Raw, typename Op>
__global__ void __launch_bounds__(kLThreads, 5) list_kernel(const __grid_constant__ typename Op::Params P, int chunk,
                                                            int local) {
  extern __shared__ __align__(16) unsigned char l_smem[];
  ListStage& sh = *reinterpret_cast<ListStage*>(l_smem);
  u64* more = reinterpret_cast<u64*>(l_smem + sizeof(ListStage));
  Raw* buf = reinterpret_cast<Raw*>(l_smem + sizeof(ListStage) + list_more(local));
  constexpr Raw kMaskedRaw = static_cast<Raw>(sizeof(Raw) == 2 ? 0xFF80u : 0xFF800000u);
  cg::cluster_group cl = cg::this_cluster();
  const int C = static_cast<int>(cl.num_blocks()), rank = static_cast<int>(cl.block_rank());
  const int row = static_cast<int>(blockIdx.x) / C;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // another kernel's rows need not wait for these
  const int k = Op::k_of(P, row);
  if (k <= 0) return;  // not a list row: the whole cluster leaves
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Raw* x = static_cast<const Raw*>(P.logits) + static_cast<int64_t>(row) * P.ld;
  const int j0 = min(P.vocab, rank * chunk), j1 = min(P.vocab, j0 + chunk);
  const int n = j1 - j0, groups = (n + 7) / 8;  // of eight elements, the last one filled up with masked ones
  const uint32_t bytes = static_cast<uint32_t>(n / 8) * 8u * sizeof(Raw);
  if (tid == 0) {
    mbar_init(&sh.bar, 1);
    mbar_init(&sh.xbar, 1);
    mbar_init(&sh.lbar, 1);
    mbar_init(&sh.fbar, 1);
    for (int r = 0; r < kLMaxCluster; ++r) mbar_init(&sh.gbar[r], 1);
    fence_barrier_init();
    fence_proxy_async();
    mbar_arrive_expect_tx(&sh.xbar, static_cast<uint32_t>(C * sizeof(ListPart)));
    if (bytes) {
      mbar_arrive_expect_tx(&sh.bar, bytes);
      bulk_load_all(buf, x + j0, bytes, &sh.bar);
    }
    if (rank == 0) mbar_arrive_expect_tx(&sh.lbar, static_cast<uint32_t>(C * sizeof(ListPush)));
    sh.mine.n = sh.bad = 0u;
  }
  __syncwarp();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // ordered by the fence above
  for (int i = n / 8 * 8 + tid; i < groups * 8; i += kLThreads) buf[i] = i < n ? x[j0 + i] : kMaskedRaw;
  for (int i = tid; i < kLBins; i += kLThreads) {
    sh.bins[i] = 0u;
    sh.least[i] = 0xFFFFFFFFu;
  }
  if (tid >= 64 && tid < 64 + kLPush) sh.mine.e[tid - 64] = 0ull;
  const bool fine = Op::fine(P, row);
  const float t = Op::t_of(P, row), c = exponent_factor(t);
  cta_sync();
  if (bytes && !mbar_wait(&sh.bar, 0)) atomicOr(&sh.bad, 1u);
  __syncwarp();

  // the thread's two largest groups, and its sum
  uint32_t mine, top[2];
  TwoMax two;
  {
    auto seen = [&](int g, const Eight<Raw>& v) { two.add(g, max8(v)); };
    if constexpr (Op::kSum) {
      float m, z, rest;
      slice_sum(buf, tid, groups, kLThreads, c, m, z, rest, seen);
      z *= ex2(-rest);
      const float wm = warp_max_nan(m);
      z = warp_sum(z != 0.f ? z * ex2(half_diff(m, wm) * (2.f * c)) : 0.f);
      if (lane == 0) sh.red[warp] = make_float2(wm, z);
    } else {
      for (int g = tid; g < groups; g += kLThreads) {
        Eight<Raw> v;
        v.load(buf + g * 8);
        seen(g, v);
      }
    }
    top[0] = ListKey<Raw>::of(two.first);
    top[1] = ListKey<Raw>::of(two.second);
    mine = two.first != two.first ? 0xFFFFFFFFu : top[0];
  }
  // a short slice gives all its elements to the bins when its maxima are too few for a near floor: a
  // share of a third of the groups still leaves a list of 1.2 times its length (bins for every
  // element cost 948 rows of 2,785 about 4 us)
  const bool every = groups * 8 <= kLShort && 3 * ((k + C - 1) / C) >= groups;
  auto candidates = [&](auto&& f) {
    if (!every) {
      f(top[0]);
      f(top[1]);
    } else {
      for (int g = tid; g < groups; g += kLThreads) {
        Eight<Raw> v;
        v.load(buf + g * 8);
#pragma unroll
        for (int i = 0; i < 8; ++i) f(key_of(v.e[i]));
      }
    }
  };
  {
    uint32_t low = 0xFFFFFFFFu;
    candidates([&](uint32_t key) {
      if (key > ListKey<Raw>::kMasked) low = min(low, key);
    });
    const uint32_t wmax = __reduce_max_sync(0xffffffffu, mine), wmin = __reduce_min_sync(0xffffffffu, low);
    if (lane == 0) {
      sh.rmax[warp] = wmax;
      sh.rmin[warp] = wmin;
    }
  }
  cta_sync();
  const uint32_t bmax = __reduce_max_sync(0xffffffffu, lane < kLWarps ? sh.rmax[lane] : 0u);
  const uint32_t bmin = __reduce_min_sync(0xffffffffu, lane < kLWarps ? sh.rmin[lane] : 0xFFFFFFFFu);
  if (bmax < KeyTraits<Raw>::kInfKey && bmax > ListKey<Raw>::kMasked) {
    // bins over the maxima's range, at most 100 below the largest (masks by a huge negative value)
    const float high = KeyTraits<Raw>::decode(bmax), range = fminf(high - KeyTraits<Raw>::decode(bmin), 100.f);
    const float per = range > 0.f ? fminf((kLBins - 1) / range, 1e30f) : 0.f;
    candidates([&](uint32_t key) {
      if (key > ListKey<Raw>::kMasked) {
        const int b = static_cast<int>(fminf((high - KeyTraits<Raw>::decode(key)) * per, kLBins - 1.f));
        atomicAdd(&sh.bins[b], 1u);
        atomicMin(&sh.least[b], key);
      }
    });
  }
  cta_sync();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (warp == 0) {
    ListPart part{};
    uint32_t cnt[kLBins / 32], sum = 0u;
#pragma unroll
    for (int i = 0; i < kLBins / 32; ++i) {
      cnt[i] = sh.bins[lane * (kLBins / 32) + i];
      sum += cnt[i];
    }
    uint32_t upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t a = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += a;
    }
    const int bk = bin_reaching(upto, sum, cnt, static_cast<uint32_t>(k));
    const int bs = bin_reaching(upto, sum, cnt, static_cast<uint32_t>((k + C - 1) / C));
    part.kth = bk < 0 ? 0u : sh.least[bk];
    part.share = bs < 0 ? 0u : sh.least[bs];
    part.kmax = bmax;
    if (sh.bad) part.kmax = 0xFFFFFFFFu;
    if constexpr (Op::kSum) {
      const float2 r = lane < kLWarps ? sh.red[lane] : make_float2(-kInf, 0.f);
      part.m = warp_max_nan(r.x);
      part.z = warp_sum(r.y != 0.f ? r.y * ex2(half_diff(r.x, part.m) * (2.f * c)) : 0.f);
    }
    if (lane < C)
      push_words<sizeof(ListPart) / 16>(peer_addr(&sh.parts[rank], lane), peer_addr(&sh.xbar, lane), &part);
  }
  const bool got = mbar_wait(&sh.xbar, 0);
  __syncwarp();
  const ListPart p = lane < C ? sh.parts[lane] : ListPart{0u, 0u, 0xFFFFFFFFu, -kInf, 0.f, {0u, 0u, 0u}};
  const uint32_t kmax = __reduce_max_sync(0xffffffffu, p.kmax);
  const uint32_t floor_key = max(max(__reduce_max_sync(0xffffffffu, p.kth), __reduce_min_sync(0xffffffffu, p.share)),
                                 ListKey<Raw>::kMasked + 1u);
  const bool finite = kmax < KeyTraits<Raw>::kInfKey && got, empty = finite && kmax <= ListKey<Raw>::kMasked;
  if (!finite || !fine || empty) {  // the same in every CTA
    if (rank == 0)
      Op::none(P, row, (finite ? 0u : VS_ROW_NONFINITE_INPUT) | (fine ? 0u : VS_ROW_BAD_PARAM) |
                           (empty ? VS_ROW_EMPTY_SUPPORT : 0u) | (got ? 0u : VS_ROW_DEVICE_TIMEOUT));
    return;
  }
  const float vmax = KeyTraits<Raw>::decode(kmax);

  // list the elements from the floor up
  if (top[0] >= floor_key) {
    const float low = KeyTraits<Raw>::decode(floor_key);
    // one group, as a rule; all of the thread's when a second one reaches the floor
    const bool one = top[1] < floor_key;
    for (int g = one ? two.at : tid; g < (one ? two.at + 1 : groups); g += kLThreads) {
      Eight<Raw> v;
      v.load(buf + g * 8);
      uint32_t hits = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) hits |= value_of(v.e[i]) >= low ? 1u << i : 0u;
      for (; hits; hits &= hits - 1u) {
        const int i = g * 8 + __ffs(hits) - 1;
        const uint32_t at = atomicAdd(&sh.mine.n, 1u);
        const u64 w = static_cast<u64>(ListKey<Raw>::of(value_of(buf[i]))) << 32 | static_cast<uint32_t>(~(j0 + i));
        if (at < kLPush)
          sh.mine.e[at] = w;
        else if (at < static_cast<uint32_t>(local))
          more[at - kLPush] = w;
      }
    }
  }
  cta_sync();
  if (warp == 0)
    push_words<1>(peer_addr(reinterpret_cast<char*>(&sh.pushed[rank]) + 16 * lane, 0), peer_addr(&sh.lbar, 0),
                  reinterpret_cast<const char*>(&sh.mine) + 16 * lane);
  if (tid == 0 && rank != 0 && sh.mine.n > static_cast<uint32_t>(kLPush))
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(peer_addr(&sh.gbar[rank], 0)) : "memory");
  if (rank != 0) {
    // leave, or stay until the leader has fetched what was not pushed
    if (sh.mine.n > static_cast<uint32_t>(kLPush)) mbar_wait(&sh.fbar, 0);
    return;
  }
  const bool all = mbar_wait(&sh.lbar, 0);
  __syncwarp();
  u64* list = reinterpret_cast<u64*>(buf);
  uint32_t cnt = lane < C && all ? sh.pushed[lane].n : 0u, upto = cnt;
#pragma unroll
  for (int o = 1; o < kLMaxCluster; o <<= 1) {
    const uint32_t a = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += a;
  }
  uint32_t total = __shfl_sync(0xffffffffu, upto, C - 1);
  const bool over = total > static_cast<uint32_t>(kLTotal) || __any_sync(0xffffffffu, cnt > static_cast<uint32_t>(local));
  for (int r = warp; r < C; r += kLWarps) {  // the warps share the peers' lists
    const uint32_t nc = __shfl_sync(0xffffffffu, cnt, r), at = __shfl_sync(0xffffffffu, upto, r) - nc;
    // also when nothing is read: this CTA must not leave before the peer's arrival is in
    if (r != 0 && nc > static_cast<uint32_t>(kLPush)) wait_cluster(&sh.gbar[r]);
    if (!over) {
      for (uint32_t i = lane; i < min(nc, static_cast<uint32_t>(kLPush)); i += 32) list[at + i] = sh.pushed[r].e[i];
      const u64* rest = cl.map_shared_rank(more, r);
      for (uint32_t i = kLPush + lane; i < nc; i += 32) list[at + i] = rest[i - kLPush];
    }
    __syncwarp();
    if (r != 0 && lane == 0 && nc > static_cast<uint32_t>(kLPush))
      asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(peer_addr(&sh.fbar, r)) : "memory");
  }
  cta_sync();
  if (!all) {
    Op::none(P, row, VS_ROW_DEVICE_TIMEOUT);
    return;
  }
  if (over) {  // more elements than k
    list_by_digits(x, P.vocab, k, list, sh);
    total = static_cast<uint32_t>(k);
  }
  const uint32_t nk = min(static_cast<uint32_t>(k), total);
  u64* spare = list + list_total(C, local);
  u64* sorted = list_sort(list, spare, total, nk, sh);
  float z = 0.f;
  if constexpr (Op::kSum)
    z = warp_sum(lane < C && p.z != 0.f ? p.z * ex2(half_diff(p.m, vmax) * (2.f * c)) : 0.f);
  Op::template finish<Raw>(P, row, sorted, sorted == list ? spare : list, nk, vmax, z);
}

template <typename Raw, typename Op>
cudaError_t launch_list(const typename Op::Params& P, cudaStream_t s, bool* done) {
  int c = stage_cluster_size(P.rows, P.vocab, sizeof(Raw));
  *done = c != 0;
  // wide lists: a CTA's share of k stays well below its 512 maxima (unless it bins all its elements:
  // 948 x 2,785 bf16, k 161: 26.7 us with one CTA per row, 39 with two) and below its list
  const int most = Op::most(P);
  while (c != 0 && c < kLMaxCluster && ((most > 128 * c && P.vocab > kLShort * c) || most > 768 * c)) c *= 2;
  if (c == 0) return cudaSuccess;
  const int chunk = ((P.vocab + c - 1) / c + 31) / 32 * 32;
  const int local = list_local(std::max(most, 1), c);
  const size_t smem = sizeof(ListStage) + list_room(c, local, static_cast<size_t>(chunk) * sizeof(Raw));
  return launch_cluster<list_kernel<Raw, Op>>(static_cast<unsigned>(P.rows) * c, c, kLThreads, smem, false, s, P, chunk,
                                              local);
}

}  // namespace

cudaError_t launch_sample_list(const SampleParams& P, vs_dtype dtype, cudaStream_t s, bool* done) {
  return dtype == VS_BF16 ? launch_list<uint16_t, SampleOp>(P, s, done) : launch_list<uint32_t, SampleOp>(P, s, done);
}

cudaError_t launch_topk_list(const TopkParams& P, vs_dtype dtype, cudaStream_t s, bool* done) {
  return dtype == VS_BF16 ? launch_list<uint16_t, TopkOp>(P, s, done) : launch_list<uint32_t, TopkOp>(P, s, done);
}

}  // namespace vs
