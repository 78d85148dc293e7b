// Exact selection inside one vocabulary row by a thread-block cluster: the
// machinery shared by the sampling kernel and the top-k kernel.
//
// The row's total order is (logit descending, token id ascending); a logit of
// -inf is a masked token and belongs to no set.  A selection asks for the
// element at which a running count, or a running sum of masses
// w_j = exp((l_j - max l) / T), first reaches a target.  Masses are 64-bit
// fixed point (RowMass), vocab * 2^fx <= 2^62: their sums are exact whatever
// the order, so every path of the kernels takes the same decisions.  Each mass is
// off by at most 2^-(fx+1) of the row's largest, a sum of n by n of these (2^-28
// for a full row of 151,936) and by 4e-14 of itself.  (A bf16 row that is drawn
// from by its values may count those within 2^-24 of zero as zeros, where that
// moves its sum by less than 2^-40.)
//
// The row is split into one contiguous slice per CTA of the cluster.  Every
// pass re-reads the slice (the first one from HBM, the others from L2, where a
// row of this size stays).  Rank 0 of the cluster (the leader) holds the
// cluster's bins; its first warp takes the decisions, without block barriers,
// and broadcasts what the next pass is to look for.
#pragma once

#include <cooperative_groups.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"
#include "row_stage.cuh"
#include "select.cuh"

namespace vs {

// 512 threads of up to 128 registers: 1,024 of 64 spill, and with the shared
// memory in use a spill goes to L2 (83 us against 36 for 128 rows of 151,936).
constexpr int kRsThreads = 512;
constexpr int kRsWarps = kRsThreads / 32;
constexpr int kRsLog = 9;
static_assert(kRsThreads == 1 << kRsLog, "threads");
constexpr int kRsMaxima = 2 * kRsThreads;  // two vector maxima per thread
constexpr int kRsZoomBins = 1024;  // bins of a zoom into one bin, linear in the key
constexpr int kRsCap = 4096;       // elements listed and sorted at once
constexpr int kRsMaxCluster = 8;

// Bins by the 16 leading bits of a logit (a bf16 value; an fp32 value cut off
// towards zero), in descending order of value: one bin for each magnitude in
// (2^-24, 2^17) of either sign.  Bin 0 holds what is larger, the last one what
// is smaller, the middle one what is nearer to zero.
constexpr uint32_t kKbLow = (127 - 24) << 7;  // leading bits of 2^-24
constexpr uint32_t kKbSpan = (24 + 17) << 7;  // bins on either side of the middle
constexpr int kKbBins = 2 * static_cast<int>(kKbSpan) + 1;
constexpr int kKbChunks = (kKbBins + 31) / 32;
constexpr int kKbAll = kKbChunks * 32;
constexpr int kKbPerLane = (kKbChunks + 31) / 32;  // chunks per lane of one warp

// What the leader asks of the cluster.
enum RsOp : uint32_t { kRsStop = 0, kRsCollect, kRsZoom, kRsSum, kRsTies };
struct RsMsg {
  uint32_t op, klo, khi, flag, key, pad;
  u64 a;
};

__device__ __forceinline__ const double* rs_tab();  // 2^(i/64), shared

// The masses of one row, with the table in shared memory.
struct RsMass : RowMass {
  __device__ __forceinline__ u64 fixed(float v) const {
    return RowMass::fixed(v, [](int i) { return rs_tab()[i]; });
  }
};

// A bin, the sums before it, and its own count and mass.
struct RsBin {
  int bin;
  u64 cnt, mass, n, m;
};

// The settings of one row's draw.
struct Settings {
  float t;
  int k;
  float p, m, u;
};

// The leader's state between two requests.  It lives in shared memory: only
// the first warp reads it, and registers held across the passes would spill.
struct RsDraw {
  Settings s;
  int phase;         // 0 top-k, 1 top-p, 2 min-p, 3 the draw
  uint32_t by_mass;  // what the search adds up
  u64 n, mass;       // the support so far
  u64 t;             // the running sum looked for
  uint32_t klo, khi; // the range under search
  RsBin f;           // the sums before it, its own
  uint32_t asked;    // the last request
  u64 got_cnt, got_mass;  // a kRsSum's answer
  // the drawn element
  uint32_t key;
  int32_t id;
};

// The slice of a row that a CTA holds.
struct RsGeo {
  const void* row;
  int vocab;
  int v0, v1;  // vectors of the slice
  int C, rank;
};

// What the phases below share.  Each phase is a function of its own that takes
// the row and the masses from here: in one piece the kernel keeps more live
// than its registers hold, and with this much shared memory a spill goes to L2.
struct RsShared {
  uint32_t cnt[kKbAll];  // this CTA's counts; in the leader, after the reduction, the cluster's
  union {
    struct {
      uint32_t lo[kKbAll], hi[kKbAll];  // the bins' masses
    };
    u64 w[kKbAll];  // leader, one value per bin: the mass of one token
  };
  u64 run_mass[32 * kKbPerLane + 1];  // leader: running sums before each chunk of 32 bins
  u64 run_cnt[32 * kKbPerLane + 1];
  u64 list[kRsCap];    // (key << 32 | ~id) of the collected elements, then their masses
  u64 sorted[kRsCap];  // the same elements in order
  uint32_t zcnt[kRsZoomBins], zlo[kRsZoomBins], zhi[kRsZoomBins];
  double tab[64];  // 2^(i/64)
  u64 sum_cnt, sum_mass;
  u64 scan_cnt[kRsWarps], scan_mass[kRsWarps];
  uint32_t red[kRsWarps][3];
  uint32_t wcount[kRsWarps];
  float fred[kRsWarps];
  uint16_t maxima[kRsMaxima];  // leading key bits of the threads' largest vectors
  uint32_t nlist;
  uint32_t x[8];  // this CTA's words of an exchange
  float xf[2];
  RsMsg msg[2];
  RsDraw draw;
  RsGeo geo;
  RsMass M;
  uint4 top[kRsThreads];  // each thread's RsTop
};

// The block's shared memory.
__device__ __forceinline__ RsShared& rs_shared() {
  extern __shared__ __align__(16) unsigned char rs_smem[];
  return *reinterpret_cast<RsShared*>(rs_smem);
}

__device__ __forceinline__ const double* rs_tab() { return rs_shared().tab; }

// The masses of a row with maximum v (or set later), by every thread: shared
// after the block's next barrier.
__device__ __forceinline__ void rs_set_masses(float v, float t, int shift) {
  RsShared& sh = rs_shared();
  if (threadIdx.x < 64) sh.tab[threadIdx.x] = exp2_64th(threadIdx.x);
  if (threadIdx.x == 64) sh.M.set(v, t, shift);
}

// The slice of one row that this CTA holds, and the cluster around it.
template <typename Raw>
struct RsRow {
  static constexpr int VEC = 16 / sizeof(Raw);
  static constexpr Raw kMaskedRaw = sizeof(Raw) == 2 ? Raw(0xFF80u) : Raw(0xFF800000u);
  static constexpr uint32_t kMaskedKey = sizeof(Raw) == 2 ? 0x007Fu : 0x007FFFFFu;  // key of -inf

  const Raw* row;
  int vocab;
  int v0, v1;  // vectors of this slice
  int C, rank;
  int turn;  // broadcast buffer in turn

  // Once per row, by every thread: the geometry, shared after the next barrier.
  __device__ __forceinline__ void init(const void* logits, int64_t r, int64_t ld, int vocab_) {
    cg::cluster_group cl = cg::this_cluster();
    C = static_cast<int>(cl.num_blocks());
    rank = static_cast<int>(cl.block_rank());
    row = static_cast<const Raw*>(logits) + r * ld;
    vocab = vocab_;
    turn = 0;
    const int nv = (vocab + VEC - 1) / VEC;
    const int per = (nv + C - 1) / C;
    v0 = min(nv, rank * per);
    v1 = min(nv, v0 + per);
    if (threadIdx.x == 0) rs_shared().geo = RsGeo{row, vocab, v0, v1, C, rank};
  }
  // The same from shared memory.
  __device__ __forceinline__ static RsRow get() {
    const RsGeo& g = rs_shared().geo;
    return RsRow{static_cast<const Raw*>(g.row), g.vocab, g.v0, g.v1, g.C, g.rank, 0};
  }

  __device__ __forceinline__ void sync() const {
    if (C == 1)
      cta_sync();
    else {
      __syncwarp();
      cg::this_cluster().sync();
    }
  }
  template <typename T>
  __device__ __forceinline__ T* peer(T* p, int r) const {
    return C == 1 ? p : cg::this_cluster().map_shared_rank(p, r);
  }
  // Lane c < C: CTA c's word; the other lanes `other`.  (All loads at once: a
  // loop over the peers would wait for each in turn.)
  template <typename T>
  __device__ __forceinline__ T from_peers(const T* p, T other) const {
    const int lane = threadIdx.x & 31;
    return lane < C ? *cg::this_cluster().map_shared_rank(p, lane) : other;
  }

  // Vector v of the row; elements at and beyond the vocabulary read as masked.
  __device__ __forceinline__ uint4 load(int v) const {
    if ((v + 1) * VEC <= vocab) return reinterpret_cast<const uint4*>(row)[v];
    union {
      uint4 q;
      Raw r[VEC];
    } u;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int j = v * VEC + i;
      u.r[i] = j < vocab ? row[j] : kMaskedRaw;
    }
    return u.q;
  }

  // f(vector index, its 16 bytes) over this slice's vectors.  The next U loads
  // are on their way while f works on the last U (few warps share an SM here:
  // loading and working in turn would leave each waiting for the other).  The
  // same thread gets the same vectors in every pass.
  template <int U, typename F>
  __device__ __forceinline__ void vectors(F&& f) const {
    static_assert(VS_MAX_ROW_VOCAB / 4 / kRsThreads <= 1 << 16, "a thread's vectors count in 16 bits");
    const int full = min(v1, vocab / VEC);  // whole vectors
    const uint4* p = reinterpret_cast<const uint4*>(row);
    int v = v0 + static_cast<int>(threadIdx.x);
    const int batches = max(0, full - v0) / (U * kRsThreads);  // complete for every thread: no predicates
    if (batches > 0) {
      uint4 q[U];
#pragma unroll
      for (int i = 0; i < U; ++i) q[i] = p[v + i * kRsThreads];
#pragma unroll 1
      for (int k = 1; k < batches; ++k) {
        uint4 cur[U];
#pragma unroll
        for (int i = 0; i < U; ++i) cur[i] = q[i];
#pragma unroll
        for (int i = 0; i < U; ++i) q[i] = p[v + (U + i) * kRsThreads];
#pragma unroll
        for (int i = 0; i < U; ++i) f(v + i * kRsThreads, cur[i]);
        v += U * kRsThreads;
      }
#pragma unroll
      for (int i = 0; i < U; ++i) f(v + i * kRsThreads, q[i]);
      v += U * kRsThreads;
    }
#pragma unroll 1
    for (; v < full; v += 4 * kRsThreads) {
      uint4 q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (v + i * kRsThreads < full) q[i] = p[v + i * kRsThreads];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (v + i * kRsThreads < full) f(v + i * kRsThreads, q[i]);
    }
    // the row's last, partial vector: the next one of the thread whose turn it is
    if (full < v1 && (full - v0) % kRsThreads == static_cast<int>(threadIdx.x)) f(full, load(full));
  }
  // f(first element id, raw values) over the same vectors.
  template <int U = 4, typename F>
  __device__ __forceinline__ void each(F&& f) const {
    vectors<U>([&](int v, const uint4& q) {
      Raw r[VEC];
      unpack(q, r);
      f(v * VEC, r);
    });
  }

  // Leader's message to every thread of the cluster.  `write` runs on the
  // leader's threads (exactly one of them fills the message).
  template <typename F>
  __device__ __forceinline__ RsMsg broadcast(F&& write) {
    RsMsg* m = &rs_shared().msg[turn];
    turn ^= 1;
    if (rank == 0) write(m);
    sync();
    return *peer(m, 0);
  }
};

// Bit i set where element i of a vector lies in [klo, khi] (keys), tested on
// the values: two comparisons per fp32 element or bf16 pair.
template <typename Raw>
struct RsRange {
  float lo, hi;
  uint32_t lo2, hi2;  // bf16, in both halves
  __device__ __forceinline__ RsRange(uint32_t klo, uint32_t khi) {
    lo = KeyTraits<Raw>::decode(klo);
    hi = KeyTraits<Raw>::decode(khi);
    lo2 = __byte_perm(__float_as_uint(lo), 0, 0x3232);
    hi2 = __byte_perm(__float_as_uint(hi), 0, 0x3232);
  }
  __device__ __forceinline__ uint32_t in(const uint4& q) const {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    uint32_t hits = 0u;
    if constexpr (sizeof(Raw) == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float v = __uint_as_float(w[i]);
        hits |= v >= lo && v <= hi ? 1u << i : 0u;
      }
    } else {
      uint32_t m[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162*>(&w[i]);
        m[i] = __hge2_mask(v, *reinterpret_cast<const __nv_bfloat162*>(&lo2)) &
               __hle2_mask(v, *reinterpret_cast<const __nv_bfloat162*>(&hi2));
      }
      if (m[0] | m[1] | m[2] | m[3]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) hits |= (m[i] & 1u) << (2 * i) | (m[i] >> 31) << (2 * i + 1);
      }
    }
    return hits;
  }
};

__device__ __forceinline__ uint32_t bmax2_nan(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                       *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// A thread's three largest vectors: the 16 leading key bits of a vector's
// maximum above the vector's turn in the thread's pass, descending; and the
// largest of the others.  With them the elements above a floor are found
// again by reading one to three vectors instead of the whole slice.
struct RsTop {
  uint32_t a, b, c, rest;
  __device__ __forceinline__ void add(uint32_t x) {
    uint32_t lo = min(a, x);
    a = max(a, x);
    x = lo;
    lo = min(b, x);
    b = max(b, x);
    x = lo;
    lo = min(c, x);
    c = max(c, x);
    rest = max(rest, lo);
  }
};

// The row's largest key (kMaskedKey: every token masked; kInfKey or more: it
// holds a NaN or +inf).  The two largest of each thread's vector maxima (their 16
// leading key bits) go to sh.maxima, its RsTop to sh.top.  The packed maximum lets a NaN through.
template <typename Raw>
__device__ __noinline__ uint32_t rs_max() {
  RsShared& sh = rs_shared();
  const RsRow<Raw> R = RsRow<Raw>::get();
  RsTop top{0u, 0u, 0u, 0u};
  uint32_t turn = 0u, thread_max = 0u;
  R.template vectors<8>([&](int, const uint4& q) {
    uint32_t k;
    if constexpr (sizeof(Raw) == 2) {
      uint32_t m = bmax2_nan(bmax2_nan(q.x, q.y), bmax2_nan(q.z, q.w));
      m = bmax2_nan(m, m >> 16 | m << 16) & 0xFFFFu;
      k = key_of(static_cast<uint16_t>(m));
      // a NaN comes out of the packed maximum as one of the largest or (sign set) smallest keys
      if (k < RsRow<Raw>::kMaskedKey) k = 0xFFFFu;
      thread_max = max(thread_max, k);
    } else {
      const float m = max_nan(max_nan(__uint_as_float(q.x), __uint_as_float(q.y)),
                              max_nan(__uint_as_float(q.z), __uint_as_float(q.w)));
      const uint32_t key = m != m ? 0xFFFFFFFFu : key_of(__float_as_uint(m));
      thread_max = max(thread_max, key);
      k = key >> 16;
    }
    top.add(k << 16 | turn);
    ++turn;
  });
  sh.top[threadIdx.x] = make_uint4(top.a, top.b, top.c, top.rest);
  reinterpret_cast<uint32_t*>(sh.maxima)[threadIdx.x] = __byte_perm(top.a, top.b, 0x7632);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t kmax = __reduce_max_sync(0xffffffffu, thread_max);
  if (lane == 0) sh.red[warp][0] = kmax;
  cta_sync();
  kmax = __reduce_max_sync(0xffffffffu, lane < kRsWarps ? sh.red[lane][0] : 0u);
  if (R.C > 1) {
    if (threadIdx.x == 0) sh.x[0] = kmax;
    R.sync();
    kmax = __reduce_max_sync(0xffffffffu, R.from_peers(&sh.x[0], 0u));
  }
  return kmax;
}

// The k-th largest of the block's maxima (0 when fewer threads have one) by one
// warp, bit by bit, from the highest bit in which they differ.
__device__ __forceinline__ uint32_t rs_warp_kth(const uint16_t* maxima, int k) {
  const int lane = threadIdx.x & 31;
  constexpr int N = kRsMaxima / 64;
  uint32_t a[N];  // two maxima each
  uint32_t mn = 0xFFFFu, mx = 0u;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    a[i] = reinterpret_cast<const uint32_t*>(maxima)[i * 32 + lane];
    mn = min(mn, min(a[i] & 0xFFFFu, a[i] >> 16));
    mx = max(mx, max(a[i] & 0xFFFFu, a[i] >> 16));
  }
  mn = __reduce_min_sync(0xffffffffu, mn);
  mx = __reduce_max_sync(0xffffffffu, mx);
  const int bits = 32 - __clz(mn ^ mx);  // the leading bits all share stay
  uint32_t t = mx >> bits << bits;
  for (int b = bits - 1; b >= 0; --b) {
    const uint32_t cand = t | (1u << b);
    uint32_t n = 0u;
#pragma unroll
    for (int i = 0; i < N; ++i) n += ((a[i] & 0xFFFFu) >= cand ? 1u : 0u) + ((a[i] >> 16) >= cand ? 1u : 0u);
    if (static_cast<int>(__reduce_add_sync(0xffffffffu, n)) >= k) t = cand;
  }
  return t;
}

// A lower bound of the row's k-th largest key from the threads' vector maxima
// (each is an element of its own), by their 16 leading key bits; k at most
// the number of maxima.  Two bounds hold: the k-th largest of any one CTA's,
// and the smallest over the C CTAs of their ceil(k / C)-th largest; the first
// is near when one slice holds the large values, the second when they are
// spread.  Ends with a barrier of the cluster; also clears the list.
template <typename Raw>
__device__ __noinline__ uint32_t rs_topk_floor(int k) {
  RsShared& sh = rs_shared();
  const RsRow<Raw> R = RsRow<Raw>::get();
  const int warp = threadIdx.x >> 5;
  if (warp == 0) {
    const uint32_t t = rs_warp_kth(sh.maxima, k);
    if (threadIdx.x == 0) {
      sh.x[2] = t;
      sh.nlist = 0u;
    }
  } else if (warp == 1 && R.C > 1) {
    const uint32_t s = rs_warp_kth(sh.maxima, (k + R.C - 1) / R.C);
    if ((threadIdx.x & 31) == 0) sh.x[3] = s;
  }
  R.sync();
  uint32_t t = sh.x[2];
  if (R.C > 1) {
    t = __reduce_max_sync(0xffffffffu, R.from_peers(&sh.x[2], 0u));
    t = max(t, __reduce_min_sync(0xffffffffu, R.from_peers(&sh.x[3], 0xFFFFFFFFu)));
  }
  return sizeof(Raw) == 2 ? t : t << 16;
}

// Collect the elements with klo <= key <= khi into the leader's list (sh.nlist
// cleared before, with a barrier).  Returns their number over the cluster; the
// list is complete only when that is at most kRsCap.  Every thread calls; the
// cluster is synchronised after.  With `top` (after rs_max, khi its result) a thread
// reads only those of its vectors that reach klo, when it has them noted.
template <typename Raw>
__device__ __noinline__ uint32_t rs_collect(bool top, uint32_t klo, uint32_t khi) {
  RsShared& sh = rs_shared();
  const RsRow<Raw> R = RsRow<Raw>::get();
  const RsRange<Raw> range(klo, khi);
  auto take = [&sh, range](int v, const uint4& q) {
    const uint32_t hits = range.in(q);
    if (hits) {
      Raw r[RsRow<Raw>::VEC];
      unpack(q, r);
#pragma unroll
      for (int i = 0; i < RsRow<Raw>::VEC; ++i)
        if (hits >> i & 1u) {
          const uint32_t at = atomicAdd(&sh.nlist, 1u);
          if (at < kRsCap)
            sh.list[at] = (static_cast<u64>(key_of(r[i])) << 32) | static_cast<uint32_t>(~(v * RsRow<Raw>::VEC + i));
        }
    }
  };
  const uint32_t lead = sizeof(Raw) == 2 ? klo : klo >> 16;
  const uint4 mine = top ? sh.top[threadIdx.x] : make_uint4(0u, 0u, 0u, 0xFFFFFFFFu);
  if (mine.w >> 16 >= lead) {
    R.template vectors<8>(take);
  } else {
    const uint32_t t[3] = {mine.x, mine.y, mine.z};
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (t[i] >> 16 >= lead) {
        const int v = R.v0 + static_cast<int>(threadIdx.x + (t[i] & 0xFFFFu) * kRsThreads);
        if (v < R.v1) take(v, R.load(v));
      }
  }
  R.sync();
  if (R.C == 1) return sh.nlist;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t n = R.from_peers(&sh.nlist, 0u);
  uint32_t upto = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t t = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += t;
  }
  const uint32_t total = __shfl_sync(0xffffffffu, upto, 31);
  if (R.rank == 0 && total <= kRsCap) {  // the warps share the peers' lists
    const int c = warp % R.C;
    const uint32_t nc = __shfl_sync(0xffffffffu, n, c), at = __shfl_sync(0xffffffffu, upto, c) - nc;
    const u64* src = R.peer(sh.list, c);
    if (c != 0)
      for (uint32_t i = (warp / R.C) * 32 + lane; i < nc; i += (kRsWarps / R.C) * 32) sh.list[at + i] = src[i];
  }
  R.sync();
  return total;
}
static_assert(kRsWarps % kRsMaxCluster == 0, "every peer's list has its warps");

// Leader: the first `keep` of the n collected elements in the total order
// (descending words: value, then smaller id), into sh.sorted.  Up to 512
// elements: an element's place is the number of larger ones, counted by a
// group of 512 / 2^ceil(log2 n) neighbouring lanes; more: a bitonic network.
static __device__ __noinline__ void rs_sort(uint32_t n, uint32_t keep) {
  RsShared& sh = rs_shared();
  int bits = kRsLog - 5;
  while ((1u << bits) < n) ++bits;
  if (bits <= kRsLog) {
    const int g = 1 << (kRsLog - bits);
    const uint32_t at = threadIdx.x >> (kRsLog - bits);
    const u64 e = at < n ? sh.list[at] : 0ull;
    uint32_t place = 0u;
    if (__any_sync(0xffffffffu, at < n)) {
      for (uint32_t o = threadIdx.x & (g - 1); o < n; o += g) place += sh.list[o] > e ? 1u : 0u;
      for (int o = 1; o < g; o <<= 1) place += __shfl_xor_sync(0xffffffffu, place, o);
      if (at < n && (threadIdx.x & (g - 1)) == 0 && place < keep) sh.sorted[place] = e;
    }
    cta_sync();
    return;
  }
  if (n <= 2 * kRsThreads)
    block_sort<kRsThreads, 2>(sh.list, sh.sorted, n);
  else if (n <= 4 * kRsThreads)
    block_sort<kRsThreads, 4>(sh.list, sh.sorted, n);
  else
    block_sort<kRsThreads, 8>(sh.list, sh.sorted, n);
}
static_assert(kRsCap == 8 * kRsThreads, "block_sort's room");

// Leader: the masses of the first n sorted elements, in sh.list.
template <typename Raw>
__device__ __forceinline__ void rs_list_masses(RsShared& sh, uint32_t n) {
  const RsMass M = sh.M;
  for (uint32_t i = threadIdx.x; i < n; i += kRsThreads)
    sh.list[i] = M.fixed(KeyTraits<Raw>::decode(static_cast<uint32_t>(sh.sorted[i] >> 32)));
  cta_sync();
}

// Inclusive running sum over a warp.
template <typename T>
__device__ __forceinline__ T rs_warp_scan(T x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T t = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += t;
  }
  return x;
}

// Sum of a value below 2^62 over a warp, in every lane: three 32-bit
// reductions of 21 bits each (32 of them add up to less than 2^32).
__device__ __forceinline__ u64 rs_warp_sum(u64 x) {
  constexpr uint32_t k21 = (1u << 21) - 1u;
  const u64 a = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(x) & k21);
  const u64 b = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(x >> 21) & k21);
  const u64 c = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(x >> 42));
  return a + (b << 21) + (c << 42);
}

// One warp: the first of n sorted elements at which `mass` (on top of it, the
// elements' masses) reaches t; mass becomes the sum through it.  n - 1 when
// the sum stays below.  n at most kRsCap.
__device__ __forceinline__ uint32_t rs_list_cross(const RsShared& sh, uint32_t n, u64 t, u64& mass) {
  const int lane = threadIdx.x & 31;
  for (uint32_t i0 = 0; i0 < n; i0 += 32) {
    const u64 s = mass + rs_warp_scan(i0 + lane < n ? sh.list[i0 + lane] : 0ull);
    const uint32_t hit = __ballot_sync(0xffffffffu, i0 + lane < n && s >= t);
    if (hit) {
      const int l = __ffs(hit) - 1;
      mass = __shfl_sync(0xffffffffu, s, l);
      return i0 + l;
    }
    mass = __shfl_sync(0xffffffffu, s, 31);
  }
  return n ? n - 1 : 0u;
}

// ---------------------------------------------------------------------------
// bins

// Two bf16 values' bins (16-bit halves) at once.
__device__ __forceinline__ uint32_t kb_pair(uint32_t w) {
  constexpr uint32_t kLo = kKbLow * 0x10001u, kHi = (kKbLow + kKbSpan) * 0x10001u;
  constexpr uint32_t kNeg = ((kKbSpan - kKbLow) & 0xFFFFu) * 0x10001u;  // t -> span - low + t
  constexpr uint32_t kDiff = ((2 * kKbLow + 1u) & 0xFFFFu) * 0x10001u;  // ~t -> span + low - t
  uint32_t t, nonneg;
  asm("max.u16x2 %0, %1, %2;" : "=r"(t) : "r"(w & 0x7FFF7FFFu), "r"(kLo));
  asm("min.u16x2 %0, %1, %2;" : "=r"(t) : "r"(t), "r"(kHi));
  asm("prmt.b32 %0, %1, 0, 0xBB99;" : "=r"(nonneg) : "r"(~w));  // each half's inverted sign, replicated
  t ^= nonneg;
  asm("add.u16x2 %0, %1, %2;" : "=r"(t) : "r"(t), "r"(kNeg));
  asm("add.u16x2 %0, %1, %2;" : "=r"(t) : "r"(t), "r"(nonneg & kDiff));
  return t;
}
// One value's bin from its 16 leading bits.
__device__ __forceinline__ int kb_one(uint32_t lead) {
  const int t = static_cast<int>(min(max(lead & 0x7FFFu, kKbLow), kKbLow + kKbSpan) - kKbLow);
  return static_cast<int>(kKbSpan) + ((lead & 0x8000u) ? t : -t);
}
template <typename Raw>
__device__ __forceinline__ int kb_of(Raw r) {
  return kb_one(sizeof(Raw) == 2 ? static_cast<uint32_t>(r) : static_cast<uint32_t>(r) >> 16);
}

// The keys [klo, khi] that bin b holds.
template <typename Raw>
__device__ __forceinline__ void kb_keys(int b, uint32_t& klo, uint32_t& khi) {
  constexpr int low = sizeof(Raw) == 2 ? 0 : 16;  // bits below the leading ones
  constexpr uint32_t ones = (1u << low) - 1u;
  const int d = static_cast<int>(kKbSpan) - b;
  auto key = [](uint32_t raw) { return key_of(static_cast<Raw>(raw)); };
  const uint32_t sign = sizeof(Raw) == 2 ? 0x8000u : 0x80000000u;
  if (d == 0) {
    klo = key(sign | (kKbLow << low | ones));
    khi = key(kKbLow << low | ones);
  } else if (d > 0) {
    klo = key((kKbLow + d) << low);
    khi = d == static_cast<int>(kKbSpan) ? KeyTraits<Raw>::kInfKey - 1u : key((kKbLow + d) << low | ones);
  } else {
    klo = d == -static_cast<int>(kKbSpan) ? RsRow<Raw>::kMaskedKey + 1u : key(sign | ((kKbLow - d) << low | ones));
    khi = key(sign | ((kKbLow - d) << low));
  }
}

// Clear the bins (counts, and masses where they are kept per bin).
template <bool MASS>
__device__ __forceinline__ void kb_clear(RsShared& sh) {
  constexpr uint4 zero = {0u, 0u, 0u, 0u};
  cta_sync();
  for (int i = threadIdx.x; i < kKbAll / 4; i += kRsThreads) {
    reinterpret_cast<uint4*>(sh.cnt)[i] = zero;
    if (MASS) {
      reinterpret_cast<uint4*>(sh.lo)[i] = zero;
      reinterpret_cast<uint4*>(sh.hi)[i] = zero;
    }
  }
  cta_sync();
}

// The cluster's sums of n bins into the leader's arrays, in place: each rank
// adds its share of the bins up over the peers and writes the leader's.
template <typename Raw, bool MASS>
__device__ __forceinline__ void kb_reduce(const RsRow<Raw>& R, uint32_t* cnt, uint32_t* lo, uint32_t* hi, int n) {
  R.sync();
  if (R.C == 1) return;
  const int per = (n + R.C - 1) / R.C;
  const int b0 = R.rank * per, b1 = min(n, b0 + per);
  for (int b = b0 + static_cast<int>(threadIdx.x); b < b1; b += kRsThreads) {
    uint32_t c = 0u;
    u64 m = 0ull;
#pragma unroll
    for (int r = 0; r < kRsMaxCluster; ++r)
      if (r < R.C) {
        c += R.peer(cnt, r)[b];
        if (MASS) m += (static_cast<u64>(R.peer(hi, r)[b]) << 32) + R.peer(lo, r)[b];
      }
    R.peer(cnt, 0)[b] = c;
    if (MASS) {
      R.peer(lo, 0)[b] = static_cast<uint32_t>(m);
      R.peer(hi, 0)[b] = static_cast<uint32_t>(m >> 32);
    }
  }
  R.sync();
}

// Counts of a row's values: one shared atomic per element.  A bf16 row's
// masked tokens are in the last bin too (those past the vocabulary among
// them), and so are NaNs with their sign set (the others are in bin 0).
template <typename Raw>
__device__ __noinline__ void kb_count() {
  RsShared& sh = rs_shared();
  const RsRow<Raw> R = RsRow<Raw>::get();
  kb_clear<false>(sh);
  const uint32_t base = smem_addr(sh.cnt);
  auto inc = [&](uint32_t b) { asm volatile("red.shared.add.u32 [%0], 1;" ::"r"(base + (b << 2)) : "memory"); };
  R.template vectors<8>([&](int, const uint4& q) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(Raw) == 2) {
        const uint32_t t = kb_pair(w[i]);
        inc(t & 0xFFFFu);
        inc(t >> 16);
      } else if (w[i] != RsRow<Raw>::kMaskedRaw) {
        inc(static_cast<uint32_t>(kb_of(w[i])));
      }
    }
  });
  kb_reduce<Raw, false>(R, sh.cnt, nullptr, nullptr, kKbAll);
}

// N elements' counts and masses into their bins (-1: none).  A mass goes in as
// two 32-bit words, the low word's carry taken from the value it replaced:
// 5.8 clocks per warp and SM measured for random bins, against 21 for a
// 64-bit shared atomic.  The N low words go out together: one after the other
// each would wait for its own carry.
template <int N>
__device__ __forceinline__ void rs_add(uint32_t* cnt, uint32_t* lo, uint32_t* hi, const int (&b)[N],
                                       const u64 (&w)[N]) {
  uint32_t old[N];
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (b[i] >= 0) {
      atomicAdd(&cnt[b[i]], 1u);
      old[i] = atomicAdd(&lo[b[i]], static_cast<uint32_t>(w[i]));
    }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (b[i] >= 0) {
      const uint32_t wl = static_cast<uint32_t>(w[i]);
      atomicAdd(&hi[b[i]], static_cast<uint32_t>(w[i] >> 32) + (old[i] + wl < wl ? 1u : 0u));
    }
}

// Counts and masses of a row's bins.
template <typename Raw>
__device__ __noinline__ void kb_masses() {
  RsShared& sh = rs_shared();
  const RsRow<Raw> R = RsRow<Raw>::get();
  kb_clear<true>(sh);
  const RsMass M = sh.M;
  R.template each<2>([&](int, const auto& r) {
    int b[RsRow<Raw>::VEC];
    u64 w[RsRow<Raw>::VEC];
#pragma unroll
    for (int i = 0; i < RsRow<Raw>::VEC; ++i) {
      w[i] = M.fixed(value_of(r[i]));
      b[i] = r[i] != RsRow<Raw>::kMaskedRaw ? kb_of(r[i]) : -1;
    }
    rs_add(sh.cnt, sh.lo, sh.hi, b, w);
  });
  kb_reduce<Raw, true>(R, sh.cnt, sh.lo, sh.hi, kKbAll);
}

// The same inside [klo, khi], linear in the key: kRsZoomBins bins of
// 2^shift keys, descending.
template <typename Raw>
__device__ __noinline__ void rs_zoom(uint32_t klo, uint32_t khi, int shift) {
  RsShared& sh = rs_shared();
  const RsRow<Raw> R = RsRow<Raw>::get();
  const RsMass M = sh.M;
  cta_sync();
  for (int b = threadIdx.x; b < kRsZoomBins; b += kRsThreads) sh.zcnt[b] = sh.zlo[b] = sh.zhi[b] = 0u;
  cta_sync();
  R.template each<4>([&](int, const auto& r) {
    int b[RsRow<Raw>::VEC];
    u64 w[RsRow<Raw>::VEC];
    bool any = false;
#pragma unroll
    for (int i = 0; i < RsRow<Raw>::VEC; ++i) {
      const uint32_t k = key_of(r[i]);
      const bool in = k >= klo && k <= khi;
      any |= in;
      b[i] = in ? static_cast<int>((khi - k) >> shift) : -1;
    }
    if (!any) return;
#pragma unroll
    for (int i = 0; i < RsRow<Raw>::VEC; ++i) w[i] = M.fixed(value_of(r[i]));
    rs_add(sh.zcnt, sh.zlo, sh.zhi, b, w);
  });
  kb_reduce<Raw, true>(R, sh.zcnt, sh.zlo, sh.zhi, kRsZoomBins);
}

// Leader, whole block: running sums of counts and masses before each chunk of
// 32 bins.  ONE: a bin holds one value, its mass is count * w and w is computed
// here; the row's maximum is the first bin's value (sh.M.vmax is set; false:
// there is none).  Ends with a block barrier.
template <typename Raw, bool ONE>
__device__ __noinline__ bool kb_chunks() {
  RsShared& sh = rs_shared();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int N = (32 * kKbPerLane + kRsWarps - 1) / kRsWarps;  // this warp's chunks: warp, warp + kRsWarps, ..
  static_assert(N <= 32, "one bit per chunk");
  uint32_t full = 0u;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int ch = warp + i * kRsWarps;
    const uint32_t n = ch < kKbChunks ? sh.cnt[ch * 32 + lane] : 0u;
    full |= __any_sync(0xffffffffu, n != 0u) ? 1u << i : 0u;
  }
  if (lane < N && !(full >> lane & 1u)) {
    const int ch = warp + lane * kRsWarps;
    if (ch < 32 * kKbPerLane) sh.run_cnt[ch + 1] = sh.run_mass[ch + 1] = 0ull;
  }
  RsMass M = sh.M;
  if (ONE) {
    if (lane == 0) sh.red[warp][0] = full ? static_cast<uint32_t>(warp + (__ffs(full) - 1) * kRsWarps) : 0xFFFFFFFFu;
    cta_sync();
    const uint32_t first = __reduce_min_sync(0xffffffffu, lane < kRsWarps ? sh.red[lane][0] : 0xFFFFFFFFu);
    if (first == 0xFFFFFFFFu) return false;
    const int b = static_cast<int>(first) * 32 + __ffs(__ballot_sync(0xffffffffu, sh.cnt[first * 32 + lane] != 0u)) - 1;
    uint32_t klo, khi;
    kb_keys<Raw>(b, klo, khi);
    if (b == static_cast<int>(kKbSpan)) khi = KeyTraits<Raw>::kBits == 16 ? 0x7FFFu : 0x7FFFFFFFu;  // zero
    M.vmax = static_cast<double>(KeyTraits<Raw>::decode(khi));
    if (threadIdx.x == 0) sh.M.vmax = M.vmax;
  }
  auto bin_mass = [&](int b) -> u64 {
    if (!ONE) return (static_cast<u64>(sh.hi[b]) << 32) + sh.lo[b];
    uint32_t klo, khi;
    kb_keys<Raw>(b, klo, khi);
    if (b == static_cast<int>(kKbSpan)) khi = KeyTraits<Raw>::kBits == 16 ? 0x7FFFu : 0x7FFFFFFFu;  // zero
    return M.fixed(KeyTraits<Raw>::decode(khi));
  };
  while (full) {  // the non-empty ones, two at a time (their chains of fp64 operations overlap)
    const int i = __ffs(full) - 1;
    full &= full - 1u;
    const int j = full ? __ffs(full) - 1 : i;
    full &= full - 1u;
    const int bi = (warp + i * kRsWarps) * 32 + lane, bj = (warp + j * kRsWarps) * 32 + lane;
    const uint32_t ni = sh.cnt[bi], nj = sh.cnt[bj];
    u64 wi = bin_mass(bi), wj = bin_mass(bj);
    if (ONE) {
      sh.w[bi] = wi;
      sh.w[bj] = wj;
      wi *= ni;
      wj *= nj;
    }
    const uint32_t ci = __reduce_add_sync(0xffffffffu, ni), cj = __reduce_add_sync(0xffffffffu, nj);
    wi = rs_warp_sum(wi);
    wj = rs_warp_sum(wj);
    if (lane == 0) {
      sh.run_cnt[(bi >> 5) + 1] = ci;
      sh.run_mass[(bi >> 5) + 1] = wi;
      sh.run_cnt[(bj >> 5) + 1] = cj;
      sh.run_mass[(bj >> 5) + 1] = wj;
    }
  }
  cta_sync();
  // running sums over the chunks, 32 to a warp
  static_assert(kKbPerLane <= kRsWarps, "a warp for every 32 chunks");
  u64 c = 0ull, m = 0ull;
  if (warp < kKbPerLane) {
    c = rs_warp_scan(sh.run_cnt[threadIdx.x + 1]);
    m = rs_warp_scan(sh.run_mass[threadIdx.x + 1]);
    if (lane == 31) {
      sh.scan_cnt[warp] = c;
      sh.scan_mass[warp] = m;
    }
  }
  cta_sync();
  if (warp < kKbPerLane) {
    c += rs_warp_sum(lane < warp ? sh.scan_cnt[lane] : 0ull);
    m += rs_warp_sum(lane < warp ? sh.scan_mass[lane] : 0ull);
    sh.run_cnt[threadIdx.x + 1] = c;
    sh.run_mass[threadIdx.x + 1] = m;
    if (threadIdx.x == 0) sh.run_cnt[0] = sh.run_mass[0] = 0ull;
  }
  cta_sync();
  return true;
}

// One warp: the bin at which the running count (by_mass: mass) reaches t.
template <bool ONE>
__device__ __noinline__ RsBin kb_find(bool by_mass, u64 t) {
  const RsShared& sh = rs_shared();
  const int lane = threadIdx.x & 31;
  const u64* run = by_mass ? sh.run_mass : sh.run_cnt;
  uint32_t below = 0u;  // chunks whose running sum stays below t
#pragma unroll
  for (int i = 0; i < kKbPerLane; ++i) below += run[i * 32 + lane + 1] < t ? 1u : 0u;
  const int ch = min(static_cast<int>(__reduce_add_sync(0xffffffffu, below)), kKbChunks - 1);
  const int b = ch * 32 + lane;
  const uint32_t n = sh.cnt[b];
  const u64 m = n == 0u ? 0ull : ONE ? sh.w[b] * n : (static_cast<u64>(sh.hi[b]) << 32) + sh.lo[b];
  RsBin f;
  int l;
  if (by_mass) {
    const u64 s = sh.run_mass[ch] + rs_warp_scan(m);
    l = __ffs(__ballot_sync(0xffffffffu, s >= t && n != 0u) | 0x80000000u) - 1;
    f.mass = __shfl_sync(0xffffffffu, s - m, l);
    f.cnt = sh.run_cnt[ch] + __reduce_add_sync(0xffffffffu, lane < l ? n : 0u);
  } else {
    const u64 c = sh.run_cnt[ch] + rs_warp_scan(n);
    l = __ffs(__ballot_sync(0xffffffffu, c >= t && n != 0u) | 0x80000000u) - 1;
    f.cnt = __shfl_sync(0xffffffffu, c - n, l);
    f.mass = sh.run_mass[ch] + rs_warp_sum(lane < l ? m : 0ull);
  }
  f.bin = ch * 32 + l;
  f.n = __shfl_sync(0xffffffffu, n, l);
  f.m = __shfl_sync(0xffffffffu, m, l);
  return f;
}

// One warp: the same among the zoom bins, on top of the sums (cnt, mass).
__device__ __forceinline__ RsBin rs_find_zoom(const RsShared& sh, bool by_mass, u64 t, u64 cnt, u64 mass) {
  const int lane = threadIdx.x & 31;
  RsBin f{0, cnt, mass, 0ull, 0ull};
  for (int b0 = 0; b0 < kRsZoomBins; b0 += 32) {
    const u64 n = sh.zcnt[b0 + lane], m = (static_cast<u64>(sh.zhi[b0 + lane]) << 32) + sh.zlo[b0 + lane];
    const u64 c = cnt + rs_warp_scan(n), s = mass + rs_warp_scan(m);
    const uint32_t hit = __ballot_sync(0xffffffffu, by_mass ? s - m < t && t <= s : c - n < t && t <= c);
    if (hit) {
      const int l = __ffs(hit) - 1;
      f.bin = b0 + l;
      f.n = __shfl_sync(0xffffffffu, n, l);
      f.m = __shfl_sync(0xffffffffu, m, l);
      f.cnt = __shfl_sync(0xffffffffu, c, l) - f.n;
      f.mass = __shfl_sync(0xffffffffu, s, l) - f.m;
      return f;
    }
    cnt = __shfl_sync(0xffffffffu, c, 31);
    mass = __shfl_sync(0xffffffffu, s, 31);
  }
  return f;
}

// Count and mass of the elements with klo <= key <= khi, to the leader's state.
template <typename Raw>
__device__ __noinline__ void rs_sum(uint32_t klo, uint32_t khi) {
  RsShared& sh = rs_shared();
  const RsRow<Raw> R = RsRow<Raw>::get();
  const RsMass M = sh.M;
  cta_sync();
  if (threadIdx.x == 0) sh.sum_cnt = sh.sum_mass = 0ull;
  cta_sync();
  const RsRange<Raw> range(klo, khi);
  u64 n = 0ull, s = 0ull;
  R.template vectors<4>([&](int, const uint4& q) {
    const uint32_t hits = range.in(q);
    if (hits) {
      Raw r[RsRow<Raw>::VEC];
      unpack(q, r);
#pragma unroll
      for (int i = 0; i < RsRow<Raw>::VEC; ++i)
        if (hits >> i & 1u) {
          n += 1u;
          s += M.fixed(value_of(r[i]));
        }
    }
  });
  if (n) {  // integer sums: any order
    atomicAdd(&sh.sum_cnt, n);
    atomicAdd(&sh.sum_mass, s);
  }
  R.sync();
  if (R.rank == 0 && threadIdx.x == 0) {
    u64 cnt = 0ull, mass = 0ull;
    for (int c = 0; c < R.C; ++c) {
      cnt += *R.peer(&sh.sum_cnt, c);
      mass += *R.peer(&sh.sum_mass, c);
    }
    sh.draw.got_cnt = cnt;
    sh.draw.got_mass = mass;
  }
  R.sync();
}

// How many of a vector's elements equal a value (the same key: +0 and -0 too).
template <typename Raw>
struct RsEqual {
  float v;
  uint32_t v2;  // bf16, in both halves
  __device__ __forceinline__ explicit RsEqual(uint32_t key) {
    v = KeyTraits<Raw>::decode(key);
    v2 = __byte_perm(__float_as_uint(v), 0, 0x3232);
  }
  __device__ __forceinline__ uint32_t count(const uint4& q) const {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    uint32_t n = 0u;
    if constexpr (sizeof(Raw) == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) n += __uint_as_float(w[i]) == v ? 1u : 0u;
    } else {
      uint32_t m[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        m[i] = __heq2_mask(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), *reinterpret_cast<const __nv_bfloat162*>(&v2));
      if (m[0] | m[1] | m[2] | m[3]) n = (__popc(m[0]) + __popc(m[1]) + __popc(m[2]) + __popc(m[3])) >> 4;
    }
    return n;
  }
  __device__ __forceinline__ uint32_t hits(const uint4& q) const {
    Raw r[16 / sizeof(Raw)];
    unpack(q, r);
    uint32_t h = 0u;
#pragma unroll
    for (int i = 0; i < static_cast<int>(16 / sizeof(Raw)); ++i) h |= value_of(r[i]) == v ? 1u << i : 0u;
    return h;
  }
};

// f(id, index) for the elements equal to `key` whose index (their place in
// the group in ascending id order, from 0) lies in [from, limit).  Each warp
// counts a contiguous run of vectors in steps of U blocks of 32 vectors, then
// only the steps that hold wanted indices are walked again in order.
template <typename Raw, typename F>
__device__ __forceinline__ void rs_ties(uint32_t key, u64 from, u64 limit, const F f) {
  constexpr int VEC = RsRow<Raw>::VEC, U = 8;
  RsShared& sh = rs_shared();
  const RsRow<Raw> R = RsRow<Raw>::get();
  uint32_t* counts = reinterpret_cast<uint32_t*>(sh.sorted);  // [warp][step]
  constexpr int kSteps = sizeof(sh.sorted) / sizeof(uint32_t) / kRsWarps;
  static_assert(VS_MAX_ROW_VOCAB / 4 / kRsWarps <= kSteps * U * 32, "step counts fit the sorted list");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (R.v1 - R.v0 + kRsWarps - 1) / kRsWarps;
  const int a = min(R.v1, R.v0 + warp * per), b = min(R.v1, a + per);
  const int whole = min(b, R.vocab / VEC);  // the run's whole vectors; one partial may follow
  const int steps = (b - a + U * 32 - 1) / (U * 32);
  const RsEqual<Raw> equal(key);
  const uint4* p = reinterpret_cast<const uint4*>(R.row);
  uint32_t n = 0u;
  cta_sync();  // the counts' room may still be read as a list
  for (int s = 0; s < steps; ++s) {
    const int v = a + s * U * 32 + lane;
    uint4 q[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (v + i * 32 < whole) q[i] = p[v + i * 32];
    uint32_t c = 0u;
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (v + i * 32 < whole) c += equal.count(q[i]);
    if (whole < b && whole >= v && (whole - v) % 32 == 0 && (whole - v) / 32 < U) c += equal.count(R.load(whole));
    c = __reduce_add_sync(0xffffffffu, c);
    if (lane == 0) counts[warp * kSteps + s] = c;
    n += c;
  }
  if (lane == 0) sh.wcount[warp] = n;
  cta_sync();
  u64 base = 0ull;
  if (R.C > 1) {
    if (warp == 0) {
      const uint32_t t = __reduce_add_sync(0xffffffffu, lane < kRsWarps ? sh.wcount[lane] : 0u);
      if (lane == 0) sh.x[4] = t;
    }
    R.sync();
    const uint32_t other = R.from_peers(&sh.x[4], 0u);
    base = __reduce_add_sync(0xffffffffu, lane < R.rank ? other : 0u);
  }
  base += __reduce_add_sync(0xffffffffu, lane < warp ? sh.wcount[lane] : 0u);
  if (base + n <= from || base >= limit) return;
  for (int s = 0; s < steps && base < limit; ++s) {
    const uint32_t here = counts[warp * kSteps + s];
    if (here == 0u || base + here <= from) {
      base += here;
      continue;
    }
    const int v = a + s * U * 32 + lane;
    uint32_t h[U];
#pragma unroll
    for (int i = 0; i < U; ++i) h[i] = v + i * 32 < b ? equal.hits(R.load(v + i * 32)) : 0u;
#pragma unroll 1
    for (int i = 0; i < U; ++i) {
      uint32_t hits = 0u;
#pragma unroll
      for (int k = 0; k < U; ++k) hits = k == i ? h[k] : hits;
      const uint32_t c = __popc(hits);
      const uint32_t incl = rs_warp_scan(c);
      u64 at = base + incl - c;
      for (; hits; hits &= hits - 1u) {
        if (at >= from && at < limit) f((v + i * 32) * VEC + __ffs(hits) - 1, at);
        ++at;
      }
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
}

// Of a bf16 row's last bin: the number of masked tokens (those past the
// vocabulary, which kb_count has counted too, among them); false when it holds
// a NaN.
static __device__ __noinline__ bool kb_masked(uint32_t* masked) {
  RsShared& sh = rs_shared();
  const RsRow<uint16_t> R = RsRow<uint16_t>::get();
  const RsEqual<uint16_t> equal(RsRow<uint16_t>::kMaskedKey);
  uint32_t n = 0u, top2 = 0u;
  R.vectors<8>([&](int, const uint4& q) {
    n += equal.count(q);
    asm("max.u16x2 %0, %0, %1;" : "+r"(top2) : "r"(q.x));
    asm("max.u16x2 %0, %0, %1;" : "+r"(top2) : "r"(q.y));
    asm("max.u16x2 %0, %0, %1;" : "+r"(top2) : "r"(q.z));
    asm("max.u16x2 %0, %0, %1;" : "+r"(top2) : "r"(q.w));
  });
  const uint32_t nan = (top2 & 0xFFFFu) > 0xFF80u || (top2 >> 16) > 0xFF80u ? 1u : 0u;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  n = __reduce_add_sync(0xffffffffu, n);
  const uint32_t any = __reduce_or_sync(0xffffffffu, nan);
  cta_sync();
  if (lane == 0) {
    sh.red[warp][1] = n;
    sh.red[warp][2] = any;
  }
  cta_sync();
  n = __reduce_add_sync(0xffffffffu, lane < kRsWarps ? sh.red[lane][1] : 0u);
  uint32_t bad = __reduce_or_sync(0xffffffffu, lane < kRsWarps ? sh.red[lane][2] : 0u);
  if (R.C > 1) {
    if (threadIdx.x == 0) {
      sh.x[6] = n;
      sh.x[7] = bad;
    }
    R.sync();
    n = __reduce_add_sync(0xffffffffu, R.from_peers(&sh.x[6], 0u));
    bad = __reduce_or_sync(0xffffffffu, R.from_peers(&sh.x[7], 0u));
  }
  *masked = n;
  return bad == 0u;
}

// Whether a bf16 row holds a value that is not zero but shares the zeros' bin.
static __device__ __noinline__ bool kb_tiny() {
  RsShared& sh = rs_shared();
  const RsRow<uint16_t> R = RsRow<uint16_t>::get();
  bool tiny = false;
  R.each<8>([&](int, const auto& r) {
#pragma unroll
    for (int i = 0; i < RsRow<uint16_t>::VEC; ++i) {
      const uint32_t a = r[i] & 0x7FFFu;
      tiny |= a - 1u < kKbLow;
    }
  });
  __syncwarp();
  tiny = __syncthreads_or(tiny);
  if (R.C > 1) {
    if (threadIdx.x == 0) sh.x[5] = tiny;
    R.sync();
    tiny = __reduce_or_sync(0xffffffffu, R.from_peers(&sh.x[5], 0u)) != 0u;
  }
  return tiny;
}

}  // namespace vs
