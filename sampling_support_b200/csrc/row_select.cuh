// Exact selection inside one vocabulary row by a thread-block cluster: the
// machinery shared by the sampling kernel and the top-k kernel.
//
// The row's total order is (logit descending, token id ascending); a logit of
// -inf is a masked token and belongs to no set.  A selection asks for the
// element at which a running count, or a running mass sum of
// w_j = exp((l_j - max l) / T), first reaches a target.  Masses are 64-bit
// fixed point, w * 2^fx with vocab * 2^fx <= 2^63, each w computed in fp64:
// every sum is exact whatever its order, and the decisions are those of the
// formula in 64 bits to about 2^-45 of the row's largest mass.
//
// The row is split into one contiguous slice per CTA of the cluster.  Every
// pass re-reads the slice (the first one from HBM, the others from L2, where a
// row of this size stays); rank 0 of the cluster (the leader) takes the
// decisions and broadcasts them.
#pragma once

#include <cooperative_groups.h>
#include <stdint.h>

#include "common.cuh"
#include "select.cuh"

namespace vs {

constexpr int kRsThreads = 1024;
constexpr int kRsWarps = kRsThreads / 32;
constexpr int kRsBins = 4096;      // level-0 bins, linear in the logit below the maximum
constexpr int kRsZoomBins = 1024;  // bins of a zoom into one bin, linear in the key
constexpr int kRsCap = 4096;       // elements listed and sorted at once
constexpr int kRsMaxCluster = 8;

// A decision of the leader, broadcast to the cluster.
struct RsMsg {
  uint32_t key, bin, flag;
  int32_t id;
  u64 n, cnt, mass;
};

struct RsShared {
  u64 hmass[kRsBins];      // this CTA's bins
  u64 rmass[kRsBins];      // leader: running sums over the cluster's level-0 bins
  u64 zmass[kRsZoomBins];  // leader: the same for a zoom
  u64 list[kRsCap];        // (key << 32 | ~id) of the collected elements
  u64 sorted[kRsCap];
  uint32_t hcnt[kRsBins];
  uint32_t rcnt[kRsBins];
  uint32_t zcnt[kRsZoomBins];
  u64 scan_a[kRsWarps], scan_b[kRsWarps];
  uint32_t red[kRsWarps][3];
  uint32_t wcount[kRsWarps];
  float fred[kRsWarps];
  uint32_t nlist;
  uint32_t x[8];  // this CTA's words of an exchange
  float xf[2];
  RsMsg msg[2];
};

// The slice of one row that this CTA holds, and the cluster around it.
template <typename Raw>
struct RsRow {
  static constexpr int VEC = 16 / sizeof(Raw);
  static constexpr Raw kMaskedRaw = sizeof(Raw) == 2 ? Raw(0xFF80u) : Raw(0xFF800000u);
  static constexpr uint32_t kMaskedKey = sizeof(Raw) == 2 ? 0x007Fu : 0x007FFFFFu;  // key of -inf

  const Raw* row;
  int vocab;
  int v0, v1;  // vectors of this slice
  RsShared* sh;
  int C, rank;
  int turn;  // broadcast buffer in turn

  __device__ void init(const void* logits, int64_t r, int64_t ld, int vocab_, RsShared* s) {
    cg::cluster_group cl = cg::this_cluster();
    C = static_cast<int>(cl.num_blocks());
    rank = static_cast<int>(cl.block_rank());
    row = static_cast<const Raw*>(logits) + r * ld;
    vocab = vocab_;
    sh = s;
    turn = 0;
    const int nv = (vocab + VEC - 1) / VEC;
    const int per = (nv + C - 1) / C;
    v0 = min(nv, rank * per);
    v1 = min(nv, v0 + per);
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

  // f(first element id, raw values) over this slice's vectors, four loads in
  // flight per thread.
  template <typename F>
  __device__ __forceinline__ void each(F&& f) const {
    constexpr int U = 4;
    for (int v = v0 + static_cast<int>(threadIdx.x); v < v1; v += U * kRsThreads) {
      uint4 q[U];
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (v + i * kRsThreads < v1) q[i] = load(v + i * kRsThreads);
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (v + i * kRsThreads < v1) {
          Raw r[VEC];
          unpack(q[i], r);
          f((v + i * kRsThreads) * VEC, r);
        }
    }
  }

  // Leader's message to every thread of the cluster.  `write` runs on the
  // leader's threads (exactly one of them fills the message).
  template <typename F>
  __device__ __forceinline__ RsMsg broadcast(F&& write) {
    RsMsg* m = &sh->msg[turn];
    turn ^= 1;
    if (rank == 0) write(m);
    sync();
    const RsMsg got = *peer(m, 0);
    return got;
  }
};

// Exclusive prefix sums of (a, b) over the block's threads, and the totals.
__device__ __forceinline__ void rs_scan(u64 a, u64 b, u64& ea, u64& eb, RsShared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 ia = a, ib = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 ta = __shfl_up_sync(0xffffffffu, ia, o), tb = __shfl_up_sync(0xffffffffu, ib, o);
    if (lane >= o) {
      ia += ta;
      ib += tb;
    }
  }
  cta_sync();  // the previous scan's readers are done
  if (lane == 31) {
    sh.scan_a[warp] = ia;
    sh.scan_b[warp] = ib;
  }
  cta_sync();
  if (warp == 0) {
    const u64 ta0 = sh.scan_a[lane], tb0 = sh.scan_b[lane];
    u64 xa = ta0, xb = tb0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 ya = __shfl_up_sync(0xffffffffu, xa, o), yb = __shfl_up_sync(0xffffffffu, xb, o);
      if (lane >= o) {
        xa += ya;
        xb += yb;
      }
    }
    sh.scan_a[lane] = xa - ta0;
    sh.scan_b[lane] = xb - tb0;
  }
  cta_sync();
  ea = sh.scan_a[warp] + ia - a;
  eb = sh.scan_b[warp] + ib - b;
}
static_assert(kRsWarps == 32, "rs_scan: one warp scans one total per warp");

// The masses of one row.
struct RsMass {
  double vmax;   // largest logit
  double inv_t;  // 1 / T
  double scale;  // 2^fx
  __device__ __forceinline__ double z(float v) const { return (static_cast<double>(v) - vmax) * inv_t; }
  __device__ __forceinline__ u64 fx(float v) const { return __double2ull_rn(exp(z(v)) * scale); }
};

// The element at which a target was reached, with the count and mass up to
// and including it.  tie > 0: the tie-th element (ascending id, from 1) of the
// group with this key; else `id` is known.
struct RsHit {
  uint32_t key;
  int32_t id;
  u64 tie, cnt, mass;
};

// Extremes of the row: largest and smallest unmasked key; false when it holds
// a NaN or +inf.  thread_max: this thread's own largest key.
template <typename Raw>
__device__ bool rs_extremes(RsRow<Raw>& R, uint32_t& kmax, uint32_t& kmin, uint32_t& thread_max) {
  RsShared& sh = *R.sh;
  uint32_t mx = 0u, mn = 0xFFFFFFFFu, bad = 0u;
  R.each([&](int, const auto& r) {
#pragma unroll
    for (int i = 0; i < RsRow<Raw>::VEC; ++i) {
      const uint32_t k = key_of(r[i]);
      bad |= (k >= KeyTraits<Raw>::kInfKey || k < RsRow<Raw>::kMaskedKey) ? 1u : 0u;
      mx = max(mx, k);
      if (k > RsRow<Raw>::kMaskedKey) mn = min(mn, k);
    }
  });
  thread_max = mx;
  mx = __reduce_max_sync(0xffffffffu, mx);
  mn = __reduce_min_sync(0xffffffffu, mn);
  bad = __reduce_or_sync(0xffffffffu, bad);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) {
    sh.red[warp][0] = mx;
    sh.red[warp][1] = mn;
    sh.red[warp][2] = bad;
  }
  cta_sync();
  if (warp == 0) {
    mx = __reduce_max_sync(0xffffffffu, sh.red[lane][0]);
    mn = __reduce_min_sync(0xffffffffu, sh.red[lane][1]);
    bad = __reduce_or_sync(0xffffffffu, sh.red[lane][2]);
    if (lane == 0) {
      sh.x[0] = mx;
      sh.x[1] = mn;
      sh.x[2] = bad;
    }
  }
  R.sync();
  kmax = 0u;
  kmin = 0xFFFFFFFFu;
  bad = 0u;
  for (int c = 0; c < R.C; ++c) {
    const uint32_t* x = R.peer(sh.x, c);
    kmax = max(kmax, x[0]);
    kmin = min(kmin, x[1]);
    bad |= x[2];
  }
  return bad == 0u;
}

// A lower bound of the row's k-th largest key: the k-th largest of the
// threads' own maxima in one CTA (each is an element of its own), the best
// over the cluster.  Found bit by bit, 16 leading bits of the key; 0 when a
// CTA has fewer than k threads with an element.
template <typename Raw>
__device__ uint32_t rs_topk_floor(RsRow<Raw>& R, uint32_t thread_max, int k) {
  constexpr int drop = sizeof(Raw) == 2 ? 0 : 16;
  const uint32_t mine = thread_max >> drop;
  uint32_t t = 0u;
  for (int b = 15; b >= 0; --b) {
    const uint32_t cand = t | (1u << b);
    __syncwarp();
    if (__syncthreads_count(mine >= cand) >= k) t = cand;
  }
  if (threadIdx.x == 0) R.sh->x[3] = t;
  R.sync();
  for (int c = 0; c < R.C; ++c) t = max(t, R.peer(R.sh->x, c)[3]);
  return t << drop;
}

// Collect the elements with klo <= key <= khi into the leader's list.
// Returns their number over the cluster; the list is complete only when that
// is at most kRsCap.  Every thread calls; the cluster is synchronised after.
template <typename Raw>
__device__ uint32_t rs_collect(RsRow<Raw>& R, uint32_t klo, uint32_t khi) {
  RsShared& sh = *R.sh;
  cta_sync();
  if (threadIdx.x == 0) sh.nlist = 0u;
  cta_sync();
  R.each([&](int j0, const auto& r) {
#pragma unroll
    for (int i = 0; i < RsRow<Raw>::VEC; ++i) {
      const uint32_t k = key_of(r[i]);
      if (k >= klo && k <= khi) {
        const uint32_t at = atomicAdd(&sh.nlist, 1u);
        if (at < kRsCap) sh.list[at] = (static_cast<u64>(k) << 32) | static_cast<uint32_t>(~(j0 + i));
      }
    }
  });
  R.sync();
  uint32_t total = 0u;
  for (int c = 0; c < R.C; ++c) total += *R.peer(&sh.nlist, c);
  if (R.rank == 0 && total <= kRsCap && R.C > 1) {
    uint32_t at = sh.nlist;
    for (int c = 1; c < R.C; ++c) {
      const uint32_t n = *R.peer(&sh.nlist, c);
      const u64* src = R.peer(sh.list, c);
      for (uint32_t i = threadIdx.x; i < n; i += kRsThreads) sh.list[at + i] = src[i];
      at += n;
    }
  }
  R.sync();
  return total;
}

// Leader: the first `keep` of the n collected elements in the total order
// (descending words: value, then smaller id), into sh.sorted.  Each element's
// place is the number of larger ones.
__device__ __forceinline__ void rs_sort(RsShared& sh, uint32_t n, uint32_t keep) {
  for (uint32_t i = threadIdx.x; i < n; i += kRsThreads) {
    const u64 e = sh.list[i];
    uint32_t place = 0u;
    for (uint32_t o = 0; o < n; ++o) place += sh.list[o] > e ? 1u : 0u;
    if (place < keep) sh.sorted[place] = e;
  }
  cta_sync();
}

// Level-0 bin of a value: linear in the distance below the maximum, so that
// it does not increase with the value.
struct RsBins {
  float vmax, s;
  __device__ __forceinline__ int of(float v) const {
    return static_cast<int>(fminf((vmax - v) * s, static_cast<float>(kRsBins - 1)));
  }
};

// The keys of level-0 bin b, within [kmin, kmax].
template <typename Raw>
__device__ void rs_bin_keys(const RsBins& B, int b, uint32_t kmin, uint32_t kmax, uint32_t& klo,
                            uint32_t& khi) {
  uint32_t lo = kmin, hi = kmax;  // smallest key whose bin is <= b
  while (lo < hi) {
    const uint32_t mid = lo + ((hi - lo) >> 1);
    if (B.of(KeyTraits<Raw>::decode(mid)) <= b)
      hi = mid;
    else
      lo = mid + 1;
  }
  klo = lo;
  lo = kmin;
  hi = kmax;  // largest key whose bin is >= b
  while (lo < hi) {
    const uint32_t mid = lo + ((hi - lo + 1) >> 1);
    if (B.of(KeyTraits<Raw>::decode(mid)) >= b)
      lo = mid;
    else
      hi = mid - 1;
  }
  khi = lo;
}

// Count and mass of every bin of this CTA's slice, then their sums over the
// cluster as running sums in the leader's (rcnt, rmass).
template <typename Raw, typename BinOf>
__device__ void rs_hist(RsRow<Raw>& R, const RsMass& M, int nb, uint32_t* rcnt, u64* rmass,
                        BinOf&& bin_of) {
  RsShared& sh = *R.sh;
  cta_sync();
  for (int b = threadIdx.x; b < nb; b += kRsThreads) {
    sh.hcnt[b] = 0u;
    sh.hmass[b] = 0ull;
  }
  cta_sync();
  R.each([&](int, const auto& r) {
#pragma unroll
    for (int i = 0; i < RsRow<Raw>::VEC; ++i) {
      const uint32_t k = key_of(r[i]);
      if (k > RsRow<Raw>::kMaskedKey) {
        const float v = value_of(r[i]);
        const int b = bin_of(k, v);
        if (b >= 0) {
          atomicAdd(&sh.hcnt[b], 1u);
          atomicAdd(&sh.hmass[b], M.fx(v));
        }
      }
    }
  });
  R.sync();
  const int per = (nb + R.C - 1) / R.C;
  const int b0 = R.rank * per, b1 = min(nb, b0 + per);
  uint32_t* oc = R.peer(rcnt, 0);
  u64* om = R.peer(rmass, 0);
  for (int b = b0 + static_cast<int>(threadIdx.x); b < b1; b += kRsThreads) {
    uint32_t n = 0u;
    u64 m = 0ull;
    for (int c = 0; c < R.C; ++c) {
      n += R.peer(sh.hcnt, c)[b];
      m += R.peer(sh.hmass, c)[b];
    }
    oc[b] = n;
    om[b] = m;
  }
  R.sync();
  if (R.rank == 0) {  // running sums: each thread its nb / kRsThreads bins
    const int q = nb / kRsThreads, f = threadIdx.x * q;
    u64 n = 0ull, m = 0ull, en, em;
    for (int i = 0; i < q; ++i) {
      n += rcnt[f + i];
      m += rmass[f + i];
    }
    rs_scan(n, m, en, em, sh);
    for (int i = 0; i < q; ++i) {
      en += rcnt[f + i];
      em += rmass[f + i];
      rcnt[f + i] = static_cast<uint32_t>(en);
      rmass[f + i] = em;
    }
  }
  cta_sync();
}
static_assert(kRsBins % kRsThreads == 0 && kRsZoomBins % kRsThreads == 0, "whole bins per thread");

// Leader: the bin at which the running count (by_mass: mass) reaches t, on
// top of (cnt0, mass0); fills the message with it, its element count and the
// sums before it.
__device__ __forceinline__ void rs_find_bin(RsMsg* m, const uint32_t* rcnt, const u64* rmass, int nb,
                                            bool by_mass, u64 t, u64 cnt0, u64 mass0) {
  for (int b = threadIdx.x; b < nb; b += kRsThreads) {
    const u64 cb = cnt0 + (b ? rcnt[b - 1] : 0u), ce = cnt0 + rcnt[b];
    const u64 mb = mass0 + (b ? rmass[b - 1] : 0ull), me = mass0 + rmass[b];
    if (by_mass ? (mb < t && t <= me) : (cb < t && t <= ce)) {
      m->bin = static_cast<uint32_t>(b);
      m->n = ce - cb;
      m->cnt = cb;
      m->mass = mb;
    }
  }
}

// The element at which the running count (by_mass: mass) of the whole row
// reaches t, 1 <= t <= the row's total, from the level-0 running sums.
template <typename Raw>
__device__ RsHit rs_find(RsRow<Raw>& R, const RsMass& M, const RsBins& B, uint32_t kmin, uint32_t kmax,
                         bool by_mass, u64 t) {
  RsShared& sh = *R.sh;
  RsMsg g = R.broadcast([&](RsMsg* m) { rs_find_bin(m, sh.rcnt, sh.rmass, kRsBins, by_mass, t, 0, 0); });
  uint32_t klo, khi;
  rs_bin_keys<Raw>(B, static_cast<int>(g.bin), kmin, kmax, klo, khi);
  while (g.n > kRsCap && klo < khi) {
    int shift = 0;
    while (((khi - klo) >> shift) >= static_cast<uint32_t>(kRsZoomBins)) ++shift;
    rs_hist(R, M, kRsZoomBins, sh.zcnt, sh.zmass, [&](uint32_t k, float) {
      return (k < klo || k > khi) ? -1 : static_cast<int>((khi - k) >> shift);
    });
    const u64 c0 = g.cnt, m0 = g.mass;
    g = R.broadcast([&](RsMsg* m) { rs_find_bin(m, sh.zcnt, sh.zmass, kRsZoomBins, by_mass, t, c0, m0); });
    const uint32_t top = khi - (g.bin << shift);
    const uint32_t width = (1u << shift) - 1u;
    klo = top - klo > width ? top - width : klo;
    khi = top;
  }
  RsHit h;
  if (klo == khi) {  // equal values: the place in the group by arithmetic
    const u64 w = M.fx(KeyTraits<Raw>::decode(klo));
    h.key = klo;
    h.id = -1;
    h.tie = by_mass ? (t - g.mass + w - 1) / w : t - g.cnt;
    h.cnt = g.cnt + h.tie;
    h.mass = g.mass + h.tie * w;
    return h;
  }
  const uint32_t n = rs_collect(R, klo, khi);
  const RsMsg a = R.broadcast([&](RsMsg* m) {
    rs_sort(sh, n, n);
    // running sums: kRsCap / kRsThreads consecutive elements per thread
    constexpr int Q = kRsCap / kRsThreads;
    const uint32_t f = threadIdx.x * Q;
    u64 w[Q], c = 0ull, s = 0ull, ec, es;
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      w[i] = f + i < n ? M.fx(KeyTraits<Raw>::decode(static_cast<uint32_t>(sh.sorted[f + i] >> 32))) : 0ull;
      c += f + i < n ? 1u : 0u;
      s += w[i];
    }
    rs_scan(c, s, ec, es, sh);
    ec += g.cnt;
    es += g.mass;
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      if (f + i < n) {
        const u64 before = by_mass ? es : ec;
        es += w[i];
        ec += 1u;
        if (before < t && t <= (by_mass ? es : ec)) {
          const u64 e = sh.sorted[f + i];
          m->key = static_cast<uint32_t>(e >> 32);
          m->id = static_cast<int32_t>(~static_cast<uint32_t>(e));
          m->cnt = ec;
          m->mass = es;
        }
      }
    }
  });
  h.key = a.key;
  h.id = a.id;
  h.tie = 0ull;
  h.cnt = a.cnt;
  h.mass = a.mass;
  return h;
}

// Count and mass of the elements with key >= kcut.
template <typename Raw>
__device__ void rs_sum_above(RsRow<Raw>& R, const RsMass& M, uint32_t kcut, u64& cnt, u64& mass) {
  RsShared& sh = *R.sh;
  u64 n = 0ull, s = 0ull;
  R.each([&](int, const auto& r) {
#pragma unroll
    for (int i = 0; i < RsRow<Raw>::VEC; ++i)
      if (key_of(r[i]) >= kcut) {
        n += 1u;
        s += M.fx(value_of(r[i]));
      }
  });
  u64 en, es;
  rs_scan(n, s, en, es, sh);
  if (threadIdx.x == kRsThreads - 1) {  // the last thread's inclusive sums are the block's
    sh.msg[R.turn].cnt = en + n;
    sh.msg[R.turn].mass = es + s;
  }
  R.sync();
  cnt = mass = 0ull;
  for (int c = 0; c < R.C; ++c) {
    const RsMsg* p = R.peer(&sh.msg[R.turn], c);
    cnt += p->cnt;
    mass += p->mass;
  }
  R.turn ^= 1;
}

// f(id, index) for every element equal to `key`, index = its place in the
// group in ascending id order, from 0; only for indices below `limit`.  Each
// warp counts a contiguous run of vectors, then the warps that hold indices
// below the limit walk their run again in order.
template <typename Raw, typename F>
__device__ void rs_ties(RsRow<Raw>& R, uint32_t key, u64 limit, F&& f) {
  constexpr int VEC = RsRow<Raw>::VEC;
  RsShared& sh = *R.sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (R.v1 - R.v0 + kRsWarps - 1) / kRsWarps;
  const int a = min(R.v1, R.v0 + warp * per), b = min(R.v1, a + per);
  uint32_t n = 0u;
  for (int v = a + lane; v < b; v += 32) {
    Raw r[VEC];
    unpack(R.load(v), r);
#pragma unroll
    for (int i = 0; i < VEC; ++i) n += key_of(r[i]) == key ? 1u : 0u;
  }
  n = __reduce_add_sync(0xffffffffu, n);
  cta_sync();
  if (lane == 0) sh.wcount[warp] = n;
  cta_sync();
  if (warp == 0) {
    const uint32_t t = __reduce_add_sync(0xffffffffu, sh.wcount[lane]);
    if (lane == 0) sh.x[4] = t;
  }
  R.sync();
  u64 base = 0ull;
  for (int c = 0; c < R.rank; ++c) base += R.peer(sh.x, c)[4];
  for (int w = 0; w < warp; ++w) base += sh.wcount[w];
  if (n == 0u || base >= limit) return;
  for (int v0 = a; v0 < b; v0 += 32) {
    const int v = v0 + lane;
    Raw r[VEC];
    uint32_t hits = 0u;
    if (v < b) {
      unpack(R.load(v), r);
#pragma unroll
      for (int i = 0; i < VEC; ++i) hits |= key_of(r[i]) == key ? 1u << i : 0u;
    }
    const uint32_t c = __popc(hits);
    uint32_t incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    u64 at = base + incl - c;
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (hits >> i & 1u) {
        if (at < limit) f(v * VEC + i, at);
        ++at;
      }
    base += __shfl_sync(0xffffffffu, incl, 31);
    if (base >= limit) break;
  }
}

}  // namespace vs
