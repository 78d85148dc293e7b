// vs_sample: one token per row from a given uniform number.
//
// With w_j = exp((l_j - max l) / T) and the row in the library's total order
// (logit descending, token id ascending), C_i the running sum of w:
//   n_k = top_k, n_p = the first i with C_i >= top_p C_{n_k},
//   n_m = the number of tokens with w >= min_p;  the support is the first
//   n = min(n_k, n_p, n_m) tokens;
//   token = the first i with C_i > u C_n (u = 1: the n-th),  logprob = log(w_i / C_n).
#include "internal.h"
#include "row_select.cuh"
#include "row_stage.cuh"

namespace vs {

namespace {

__device__ __forceinline__ void write_none(const SampleParams& P, int row, uint32_t status) {
  P.token[row] = -1;
  if (P.logprob) P.logprob[row] = __int_as_float(0x7FC00000);
  if (P.support_size) P.support_size[row] = 0;
  if (P.status) P.status[row] = status;
}

__device__ __forceinline__ void write_row(const SampleParams& P, int row, float v, u64 mass, u64 n, const RsMass& M) {
  if (P.logprob) P.logprob[row] = M.logprob(v, mass);
  if (P.support_size) P.support_size[row] = static_cast<int32_t>(n);
  if (P.status) P.status[row] = 0u;
}

// Leader: the support's cut and the drawn token from a list that holds at
// least the first nk tokens of the row.  The block sorts and takes the masses;
// its first warp decides.
template <typename Raw>
__device__ __noinline__ void draw_from_list(const SampleParams& P, int row, const Settings& s, uint32_t n_list) {
  RsShared& sh = rs_shared();
  const RsMass M = sh.M;
  const uint32_t nk = min(static_cast<uint32_t>(s.k), n_list);
  rs_sort(n_list, nk);
  rs_list_masses<Raw>(sh, nk);
  if (threadIdx.x >= 32) return;
  const int lane = threadIdx.x;
  u64 mass = 0ull;
  for (uint32_t i = lane; i < nk; i += 32) mass += sh.list[i];
  mass = rs_warp_sum(mass);
  uint32_t n = nk;
  if (s.p < 1.f) {
    u64 m = 0ull;
    n = rs_list_cross(sh, nk, topp_target(s.p, static_cast<double>(mass)), m) + 1u;
    mass = m;
  }
  if (s.m > 0.f) {
    uint32_t keep = 0u;  // the order is by mass: those kept are the first ones
    u64 m = 0ull;
    for (uint32_t i = lane; i < n; i += 32) {
      const float v = KeyTraits<Raw>::decode(static_cast<uint32_t>(sh.sorted[i] >> 32));
      if (M.reaches(v, s.m)) {
        ++keep;
        m += sh.list[i];
      }
    }
    n = __reduce_add_sync(0xffffffffu, keep);
    mass = rs_warp_sum(m);
  }
  u64 upto = 0ull;
  const uint32_t at = s.u < 1.f ? rs_list_cross(sh, n, draw_target(s.u, mass), upto) : n - 1u;
  if (lane == 0) {
    const u64 e = sh.sorted[at];
    P.token[row] = static_cast<int32_t>(~static_cast<uint32_t>(e));
    write_row(P, row, KeyTraits<Raw>::decode(static_cast<uint32_t>(e >> 32)), mass, n, M);
  }
}

// The smallest key in [lo, hi] that reaches min-p's m (hi does): the
// lanes of one warp test 32 keys at a time.
template <typename Raw>
__device__ __forceinline__ uint32_t first_above(const RsMass& M, float m, uint32_t lo, uint32_t hi) {
  const int lane = threadIdx.x & 31;
  while (lo < hi) {
    const uint32_t step = (hi - lo) / 32u + 1u;
    const uint32_t off = min(hi - lo, lane * step);
    const uint32_t yes = __ballot_sync(0xffffffffu, M.reaches(KeyTraits<Raw>::decode(lo + off), m));
    const int l = yes ? __ffs(yes) - 1 : 32;  // hi itself passes
    const uint32_t top = l == 32 ? hi : lo + min(hi - lo, l * step);
    lo = l == 0 ? lo : lo + min(hi - lo, (l - 1) * step) + 1u;
    hi = top;
    if (lo > hi) lo = hi;
  }
  return lo;
}

// The place, from 1, at which a group of tokens of mass w reaches d > 0 more:
// ceil(d / w), from a rounded quotient (at most 2^20 and off by less than one)
// and its corrections.
__device__ __forceinline__ u64 place_in_group(u64 d, u64 w) {
  u64 r = static_cast<u64>(fminf(static_cast<float>(d) / static_cast<float>(w), 2.f * VS_MAX_ROW_VOCAB));
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (r * w < d) ++r;
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (r > 1ull && (r - 1ull) * w >= d) --r;
  return r;
}

// One step of the leader's first warp: takes what the last request brought,
// goes on through the cuts (top-k, top-p, min-p, the draw) and fills the next
// request.  Each cut names a bin from the running sums; where the bin does not
// decide by itself, the cluster is asked to list its elements, to zoom into it
// when they are too many, or to add up a part of it.
template <typename Raw>
__device__ __noinline__ void draw_step(RsMsg* out) {
  RsShared& sh = rs_shared();
  const int lane = threadIdx.x & 31;
  RsDraw& d = sh.draw;
  const RsMass M = sh.M;
  const Settings s = d.s;
  int phase = d.phase;
  u64 n = d.n, mass = d.mass, t = d.t;
  bool by_mass = d.by_mass != 0u;
  uint32_t klo = d.klo, khi = d.khi, asked = d.asked;
  RsBin f = d.f;

  RsMsg q{kRsStop, 0u, 0u, 0u, 0u, 0u, 0ull};
  bool found = false, open = false;      // an element is known; a range is under search
  u64 cnt = 0ull, sum = 0ull, tie = 0ull;  // the sums through the element, its place in its group
  uint32_t key = 0u;
  int32_t id = -1;
  if (asked == kRsCollect) {
    uint32_t at;
    sum = f.mass;
    if (by_mass)
      at = rs_list_cross(sh, static_cast<uint32_t>(f.n), t, sum);
    else {
      at = min(static_cast<uint32_t>(t - f.cnt) - 1u, static_cast<uint32_t>(kRsCap - 1));
      u64 m = 0ull;
      for (uint32_t i = lane; i <= at; i += 32) m += sh.list[i];
      sum += rs_warp_sum(m);
    }
    found = true;
    cnt = f.cnt + at + 1u;
    key = static_cast<uint32_t>(sh.sorted[at] >> 32);
    id = static_cast<int32_t>(~static_cast<uint32_t>(sh.sorted[at]));
  } else if (asked == kRsZoom) {
    int shift = 0;
    while (((khi - klo) >> shift) >= static_cast<uint32_t>(kRsZoomBins)) ++shift;
    f = rs_find_zoom(sh, by_mass, t, f.cnt, f.mass);
    const uint32_t top = khi - (static_cast<uint32_t>(f.bin) << shift), width = (1u << shift) - 1u;
    klo = top - klo > width ? top - width : klo;
    khi = top;
    open = true;
  } else if (asked == kRsSum) {
    if (f.cnt + d.got_cnt < n) {
      n = f.cnt + d.got_cnt;
      mass = f.mass + d.got_mass;
    }
    phase = 3;
  }
  asked = kRsStop;
  while (asked == kRsStop) {
    if (!found && !open) {  // the next cut's bin
      if (phase == 0) {
        if (!(s.k > 0 && static_cast<u64>(s.k) < n)) {
          phase = 1;
          continue;
        }
        by_mass = false;
        t = static_cast<u64>(s.k);
      } else if (phase == 1) {
        if (!(s.p < 1.f)) {
          phase = 2;
          continue;
        }
        by_mass = true;
        t = topp_target(s.p, static_cast<double>(mass));
      } else if (phase == 2) {
        phase = 3;
        if (!(s.m > 0.f)) continue;
        // the first bin that does not pass whole, from the maximum's on (no mass is
        // asked for above the maximum, where there is none)
        const float top = static_cast<float>(M.vmax);
        const uint32_t ktop = KeyTraits<Raw>::kBits == 16 ? key_of(static_cast<uint16_t>(__float_as_uint(top) >> 16))
                                                          : key_of(__float_as_uint(top));
        const float vm = static_cast<float>(M.vmax + log(static_cast<double>(s.m)) / M.inv_t);
        int b = max(kb_one(__float_as_uint(top) >> 16), kb_one(__float_as_uint(vm) >> 16) - 2);
        for (; b < kKbBins; ++b) {
          kb_keys<Raw>(b, klo, khi);
          klo = min(klo, ktop);
          khi = min(khi, ktop);
          if (!M.reaches(KeyTraits<Raw>::decode(klo), s.m)) break;
        }
        if (b == kKbBins) continue;
        const int at = (b & ~31) + lane;
        const u64 c = sh.cnt[at];
        const u64 m = (static_cast<u64>(sh.hi[at]) << 32) + sh.lo[at];
        f.bin = b;
        f.cnt = sh.run_cnt[b >> 5] + rs_warp_sum(at < b ? c : 0ull);
        f.mass = sh.run_mass[b >> 5] + rs_warp_sum(at < b ? m : 0ull);
        f.n = __shfl_sync(0xffffffffu, c, b & 31);
        if (f.cnt >= n) continue;
        if (f.n == 0ull || !M.reaches(KeyTraits<Raw>::decode(khi), s.m)) {
          n = f.cnt;
          mass = f.mass;
          continue;
        }
        asked = q.op = kRsSum;
        q.klo = first_above<Raw>(M, s.m, klo, khi);
        q.khi = khi;
        break;
      } else {
        by_mass = s.u < 1.f;
        t = by_mass ? draw_target(s.u, mass) : n;
      }
      f = kb_find<false>(by_mass, t);
      if (phase == 1 && f.cnt >= n) {  // not before the top-k cut
        phase = 2;
        continue;
      }
      kb_keys<Raw>(f.bin, klo, khi);
      open = true;
    }
    if (!found) {  // inside the range
      if (klo == khi) {
        key = khi;
        const u64 w = M.fixed(KeyTraits<Raw>::decode(khi));
        tie = by_mass ? place_in_group(t - f.mass, w) : t - f.cnt;
        cnt = f.cnt + tie;
        sum = f.mass + tie * w;
      } else if (f.n == 1ull && phase < 3) {
        cnt = f.cnt + 1ull;
        sum = f.mass + f.m;
      } else {
        asked = q.op = f.n <= static_cast<u64>(kRsCap) ? kRsCollect : kRsZoom;
        q.klo = klo;
        q.khi = khi;
        break;
      }
    }
    // the cut's element is known
    found = open = false;
    if (phase == 3) {
      q.op = tie ? kRsTies : kRsStop;
      q.klo = key;
      q.a = tie;
      break;
    }
    if (cnt < n) {
      n = cnt;
      mass = sum;
    }
    ++phase;
  }
  if (lane == 0) {
    d.phase = phase;
    d.n = n;
    d.mass = mass;
    d.t = t;
    d.by_mass = by_mass;
    d.klo = klo;
    d.khi = khi;
    d.f = f;
    d.asked = asked;
    d.key = key;
    d.id = id;
    *out = q;
  }
  __syncwarp();
}

// The r-th token (from 1) of those with this key, into *token.
template <typename Raw>
__device__ __noinline__ void draw_tie(uint32_t key, u64 r, int32_t* token) {
  rs_ties<Raw>(key, r - 1ull, r, [token](int id, u64) { *token = id; });
}

// The cuts and the draw from the row's bins (kb_chunks done).
template <typename Raw>
__device__ __forceinline__ void draw_from_bins(const SampleParams& P, int row, const Settings& s, RsRow<Raw>& R) {
  RsShared& sh = rs_shared();
  if (R.rank == 0 && threadIdx.x == 0) {
    RsDraw& d = sh.draw;
    d.s = s;
    d.phase = 0;
    d.asked = kRsStop;
    d.n = sh.run_cnt[32 * kKbPerLane];
    d.mass = sh.run_mass[32 * kKbPerLane];
  }
  __syncwarp();
  for (;;) {
    const RsMsg msg = R.broadcast([&](RsMsg* out) {
      if (threadIdx.x < 32) draw_step<Raw>(out);
    });
    if (msg.op == kRsCollect) {
      cta_sync();
      if (threadIdx.x == 0) sh.nlist = 0u;
      R.sync();
      const uint32_t k = min(rs_collect<Raw>(false, msg.klo, msg.khi), static_cast<uint32_t>(kRsCap));
      if (R.rank == 0) {
        rs_sort(k, k);
        rs_list_masses<Raw>(sh, k);
      }
      continue;
    }
    if (msg.op == kRsZoom) {
      int shift = 0;
      while (((msg.khi - msg.klo) >> shift) >= static_cast<uint32_t>(kRsZoomBins)) ++shift;
      rs_zoom<Raw>(msg.klo, msg.khi, shift);
      continue;
    }
    if (msg.op == kRsSum) {
      rs_sum<Raw>(msg.klo, msg.khi);
      continue;
    }
    if (R.rank == 0 && threadIdx.x == 0) {
      const RsDraw& d = sh.draw;
      if (msg.op == kRsStop) P.token[row] = d.id;
      write_row(P, row, KeyTraits<Raw>::decode(d.key), d.mass, d.n, sh.M);
    }
    __syncwarp();
    if (msg.op == kRsTies) draw_tie<Raw>(msg.klo, msg.a, P.token + row);
    break;
  }
  R.sync();  // peers may still read this CTA's words
}

// Any row, any type, any setting.
template <typename Raw>
__device__ __forceinline__ void draw_general(const SampleParams& P, int row, const Settings& s, RsRow<Raw>& R,
                                             uint32_t kmax) {
  rs_set_masses(KeyTraits<Raw>::decode(kmax), s.t, P.fx_shift);
  kb_masses<Raw>();
  if (R.rank == 0) kb_chunks<Raw, false>();
  draw_from_bins<Raw>(P, row, s, R);
}

// The leader's first warp: the cuts and the draw of a bf16 row from the counts
// of its values.  A value's tokens have one mass and follow one another in the
// order, so the place inside a bin is arithmetic.  False: a cut falls into the
// zeros' bin, and it may hold other values (`middle`), or it weighs too much.
static __device__ __noinline__ bool draw_by_counts(bool middle) {
  RsShared& sh = rs_shared();
  RsDraw& d = sh.draw;
  const Settings s = d.s;
  const int lane = threadIdx.x & 31;
  u64 n = sh.run_cnt[32 * kKbPerLane], mass = sh.run_mass[32 * kKbPerLane];
  // the zeros' bin is taken as zeros as long as no cut falls into it and its mass, off by
  // at most 2^-24 / T of itself, moves the row's sum by less than 2^-40
  if (middle && static_cast<double>(sh.w[kKbSpan]) * sh.cnt[kKbSpan] * 65536.0 * sh.M.inv_t > static_cast<double>(mass))
    return false;
  auto lost = [&](const RsBin& f) { return middle && f.bin == static_cast<int>(kKbSpan); };
  if (s.k > 0 && static_cast<u64>(s.k) < n) {
    n = static_cast<u64>(s.k);
    const RsBin f = kb_find<true>(false, n);
    if (lost(f)) return false;
    mass = f.mass + (n - f.cnt) * sh.w[f.bin];
  }
  if (s.p < 1.f) {
    const u64 t = topp_target(s.p, static_cast<double>(mass));
    const RsBin f = kb_find<true>(true, t);
    if (lost(f)) return false;
    const u64 w = sh.w[f.bin], r = place_in_group(t - f.mass, w);
    if (f.cnt + r < n) {
      n = f.cnt + r;
      mass = f.mass + r * w;
    }
  }
  if (s.m > 0.f) {
    // the first bin, from the maximum's on, whose value does not pass
    const RsMass M = sh.M;
    const float top = static_cast<float>(M.vmax);
    const float vm = static_cast<float>(M.vmax + log(static_cast<double>(s.m)) / M.inv_t);
    const int b0 = kb_one(__float_as_uint(top) >> 16);
    int b = max(b0, kb_one(__float_as_uint(vm) >> 16) - 2);
    for (; b < kKbBins; ++b) {
      uint32_t klo, khi;
      kb_keys<uint16_t>(b, klo, khi);
      if (b == static_cast<int>(kKbSpan)) khi = 0x7FFFu;
      if (b > b0 && !M.reaches(KeyTraits<uint16_t>::decode(khi), s.m)) break;
    }
    if (b < kKbBins) {
      if (middle && (b == static_cast<int>(kKbSpan) || b == static_cast<int>(kKbSpan) + 1)) return false;
      const int at = (b & ~31) + lane;
      const uint32_t c = at < b ? sh.cnt[at] : 0u;
      const u64 cnt = sh.run_cnt[b >> 5] + __reduce_add_sync(0xffffffffu, c);
      if (cnt < n) {
        n = cnt;
        mass = sh.run_mass[b >> 5] + rs_warp_sum(c ? sh.w[at] * c : 0ull);
      }
    }
  }
  const bool by_mass = s.u < 1.f;
  const u64 t = by_mass ? draw_target(s.u, mass) : n;
  const RsBin f = kb_find<true>(by_mass, t);
  if (lost(f)) return false;
  if (lane == 0) {
    uint32_t klo, khi;
    kb_keys<uint16_t>(f.bin, klo, khi);
    d.key = f.bin == static_cast<int>(kKbSpan) ? 0x7FFFu : khi;
    d.t = by_mass ? place_in_group(t - f.mass, sh.w[f.bin]) : t - f.cnt;
    d.n = n;
    d.mass = mass;
  }
  __syncwarp();
  return true;
}

// A bf16 row from the counts of its values: one pass over the row (one shared
// atomic per element and no exponential), the decisions by the leader, and a
// second pass from L2 that finds the drawn token among those of its value.
// Returns false when the row needs the general path: values beyond the bins'
// range that matter.  `exact`: values next to zero matter too, so that a row
// whose list overflowed gets the list kernel's answer to the last unit.
__device__ __forceinline__ bool draw_by_value(const SampleParams& P, int row, const Settings& s, RsRow<uint16_t>& R,
                                              bool exact) {
  RsShared& sh = rs_shared();
  rs_set_masses(0.f, s.t, P.fx_shift);  // the maximum follows
  if (threadIdx.x == 0) sh.draw.s = s;
  cta_sync();  // and the geometry
  kb_count<uint16_t>();
  const RsMsg ends = R.broadcast([&](RsMsg* m) {
    if (threadIdx.x == 0) {
      m->flag = sh.cnt[0];
      m->klo = sh.cnt[kKbSpan];
      m->khi = sh.cnt[kKbBins - 1];
    }
  });
  if (ends.flag) return false;  // above 2^17, +inf or NaN
  uint32_t low = ends.khi;      // unmasked values of the last bin
  if (low) {
    uint32_t masked;
    if (!kb_masked(&masked)) return false;
    low -= masked;
    if (R.rank == 0 && threadIdx.x == 0) sh.cnt[kKbBins - 1] = low;
    __syncwarp();
  }
  bool chunks = false, middle = ends.klo != 0u;
  if (middle && exact) {
    if (kb_tiny()) return false;
    middle = false;
  }
  for (;;) {
    const RsMsg got = R.broadcast([&](RsMsg* msg) {
      uint32_t flag = 0u;
      if (!chunks) {
        cta_sync();
        if (!kb_chunks<uint16_t, true>())
          flag = 2u;  // every token masked
        else if (low && (s.u >= 1.f || sh.M.z(-131072.f) >= -46.0 || (s.m > 0.f && sh.M.reaches(-131072.f, s.m))))
          flag = 1u;  // the last bin's values have masses of their own, or min-p or the draw may tell them apart
      }
      if (threadIdx.x >= 32) return;
      if (flag == 0u && !draw_by_counts(middle)) flag = 3u;
      if (threadIdx.x == 0) {
        msg->flag = flag;
        msg->key = sh.draw.key;
        msg->a = sh.draw.t;
      }
      __syncwarp();
    });
    chunks = true;
    if (got.flag == 1u) return false;
    if (got.flag == 3u) {  // does the zeros' bin hold other values?
      if (kb_tiny()) return false;
      middle = false;
      continue;
    }
    if (R.rank == 0 && threadIdx.x == 0) {
      if (got.flag == 2u)
        write_none(P, row, VS_ROW_EMPTY_SUPPORT);
      else
        write_row(P, row, KeyTraits<uint16_t>::decode(got.key), sh.draw.mass, sh.draw.n, sh.M);
    }
    __syncwarp();
    if (got.flag == 0u) draw_tie<uint16_t>(got.key, got.a, P.token + row);
    R.sync();  // peers may still read this CTA's words
    return true;
  }
}

template <typename Raw>
__device__ __forceinline__ void sample_row(const SampleParams& P, int row) {
  RsRow<Raw> R;
  R.init(P.logits, row, P.ld, P.vocab);
  const bool lead = R.rank == 0 && threadIdx.x == 0;

  Settings s;
  s.t = P.temperature ? P.temperature[row] : P.temperature_scalar;
  s.k = P.top_k ? P.top_k[row] : P.top_k_scalar;
  s.p = P.top_p ? P.top_p[row] : P.top_p_scalar;
  s.m = P.min_p ? P.min_p[row] : P.min_p_scalar;
  s.u = P.uniform[row];
  const bool fine = s.t >= 0.f && s.t < kInf && s.p > 0.f && s.m <= 1.f && s.u >= 0.f && s.u <= 1.f;
  if (fine && s.t == 0.f) {  // greedy: the first token of the order
    s.t = 1.f;
    s.k = 1;
    s.p = 1.f;
    s.m = 0.f;
  }
  bool by_list = !P.lists && sample_list_k(P.vocab, s.t, s.k) > 0;
  bool by_value = sizeof(Raw) == 2 && fine && !by_list, crowd = false;
  for (;;) {
    if constexpr (sizeof(Raw) == 2) {
      if (by_value && draw_by_value(P, row, s, R, crowd)) return;
    }
    cta_sync();  // the geometry
    const uint32_t kmax = rs_max<Raw>();
    const bool finite = kmax < KeyTraits<Raw>::kInfKey;
    const bool empty = finite && kmax <= RsRow<Raw>::kMaskedKey;
    if (!finite || !fine || empty) {
      if (lead)
        write_none(P, row, (finite ? 0u : VS_ROW_NONFINITE_INPUT) | (fine ? 0u : VS_ROW_BAD_PARAM) |
                               (empty ? VS_ROW_EMPTY_SUPPORT : 0u));
      R.sync();  // peers read this CTA's maximum
      return;
    }
    if (by_list) {
      rs_set_masses(KeyTraits<Raw>::decode(kmax), s.t, P.fx_shift);
      const uint32_t floor_key = max(rs_topk_floor<Raw>(s.k), RsRow<Raw>::kMaskedKey + 1u);
      const uint32_t n_list = rs_collect<Raw>(true, floor_key, kmax);
      if (n_list <= static_cast<uint32_t>(kRsCap)) {
        if (R.rank == 0) draw_from_list<Raw>(P, row, s, n_list);
        return;  // rs_collect ended with a cluster barrier: nothing is read from peers after it
      }
      by_list = false;
      by_value = sizeof(Raw) == 2;
      crowd = true;
      if (by_value) continue;
    }
    draw_general(P, row, s, R, kmax);
    return;
  }
}

// One cluster per row, one CTA per SM.  Measured (device time): 128 x 151,936
// bf16 with top-p 37 us, 512 with mixed filters 116 us (1.3 TB/s), 64 x 151,936 fp32 over
// the whole vocabulary 63 us.  A bf16 row is bound by its one shared atomic per
// element and by the latency of what follows it (reduction, decision, the
// token among its equals, about 12 us); an fp32 row by its masses pass (24 us
// of the 63: the loads in flight that the registers allow, from L2).
// A list kernel before it may have its own share of the
// rows; nothing after this kernel may start before that one is done.
template <typename Raw>
__global__ void __launch_bounds__(kRsThreads, 1) sample_kernel(const __grid_constant__ SampleParams P) {
  const int row = static_cast<int>(blockIdx.x / cg::this_cluster().num_blocks());
  if (!P.lists || sample_list_k(P.vocab, P.temperature ? P.temperature[row] : P.temperature_scalar,
                                P.top_k ? P.top_k[row] : P.top_k_scalar) == 0)
    sample_row<Raw>(P, row);
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace

// Cluster size for `rows` rows of `vocab` elements: as many CTAs per row as
// the GPU's SMs hold at once, with at least 4,096 elements for each.
int row_cluster_size(int rows, int vocab) {
  int c = 1;
  while (c < kRsMaxCluster && 2ll * c * rows <= 148 && vocab / (2 * c) >= 4096) c *= 2;
  return c;
}

template <auto Kernel, typename Params>
static cudaError_t launch_rows(const Params& P, int clusters, int c, bool behind, cudaStream_t s) {
  return launch_cluster<Kernel>(static_cast<unsigned>(clusters) * c, c, kRsThreads, sizeof(RsShared), behind, s, P);
}

cudaError_t launch_sample(const SampleParams& Pin, vs_dtype dtype, cudaStream_t s) {
  SampleParams P = Pin;
  // Whether all rows have a small top-k, or (per-row settings) some may.  In the latter case the list
  // kernel runs first up to 16 rows: the general kernel lists as well, at more latency, but does not
  // hold up the rows without a top-k.  Device time in us, 151,936 bf16, list kernel first / general alone:
  //   rows   all top-k 50   half top-k 50   no top-k
  //      8   11.0 / 18.7    26.0 / 24.7     26.4 / 23.1
  //     32   12.4 / 18.1    34.7 / 26.7     28.7 / 26.7
  //    128   22.3 / 24.7    46.8 / 38.9     41.5 / 36.9
  // so 8 us are won where all have one, 3 lost where none has; from 32 rows on it is 2 to 6 against 2 to 8.
  const bool all = (!P.top_k && sample_list_k(P.vocab, 1.f, P.top_k_scalar) > 0) ||
                   (!P.temperature && P.temperature_scalar == 0.f);
  if (all || ((P.top_k || P.temperature) && P.rows <= 16)) {
    bool done = false;
    const cudaError_t e = launch_sample_list(P, dtype, s, &done);
    if (e != cudaSuccess || (all && done)) return e;
    P.lists = done;
  }
  const int c = row_cluster_size(P.rows, P.vocab);
  return dtype == VS_BF16 ? launch_rows<sample_kernel<uint16_t>>(P, P.rows, c, P.lists, s)
                          : launch_rows<sample_kernel<uint32_t>>(P, P.rows, c, P.lists, s);
}

namespace {

// More elements than a list holds lie above the floor: the k-th element's bin
// from counts, zoomed into until the bins down to it fit the list, or until
// it is one value, whose first tokens complete those above it.  Returns the
// list's length.
template <typename Raw>
__device__ __forceinline__ uint32_t topk_general(const TopkParams& P, RsRow<Raw>& R, float vmax, float t,
                                                 uint32_t kmax) {
  RsShared& sh = rs_shared();
  rs_set_masses(vmax, t, P.fx_shift);
  kb_count<Raw>();
  if (R.rank == 0) kb_chunks<Raw, true>();
  const u64 k = static_cast<u64>(P.k);
  RsBin f{0, 0ull, 0ull, 0ull, 0ull};
  uint32_t klo = 0u, khi = 0u;
  bool zoomed = false;
  for (;;) {
    const RsMsg msg = R.broadcast([&](RsMsg* out) {
      if (threadIdx.x >= 32) return;
      if (!zoomed) {
        f = kb_find<true>(false, k);
        kb_keys<Raw>(f.bin, klo, khi);
      } else {
        int shift = 0;
        while (((khi - klo) >> shift) >= static_cast<uint32_t>(kRsZoomBins)) ++shift;
        f = rs_find_zoom(sh, false, k, f.cnt, f.mass);
        const uint32_t top = khi - (static_cast<uint32_t>(f.bin) << shift), width = (1u << shift) - 1u;
        klo = top - klo > width ? top - width : klo;
        khi = top;
      }
      if (threadIdx.x == 0) {
        out->op = f.cnt + f.n <= static_cast<u64>(kRsCap) ? kRsCollect : klo == khi ? kRsTies : kRsZoom;
        out->klo = klo;
        out->khi = khi;
        out->a = f.cnt;
      }
    });
    zoomed = true;
    if (msg.op == kRsZoom) {
      int shift = 0;
      while (((msg.khi - msg.klo) >> shift) >= static_cast<uint32_t>(kRsZoomBins)) ++shift;
      rs_zoom<Raw>(msg.klo, msg.khi, shift);
      continue;
    }
    cta_sync();
    if (threadIdx.x == 0) sh.nlist = 0u;
    R.sync();
    if (msg.op == kRsCollect) {
      return rs_collect<Raw>(false, msg.klo, kmax);
    }
    const uint32_t above = msg.klo < kmax ? rs_collect<Raw>(false, msg.klo + 1u, kmax) : 0u;
    u64* list = R.peer(sh.list, 0);
    rs_ties<Raw>(msg.klo, 0ull, k - min(k, static_cast<u64>(above)), [=](int id, u64 at) {
      list[above + at] = (static_cast<u64>(msg.klo) << 32) | static_cast<uint32_t>(~id);
    });
    R.sync();
    return static_cast<uint32_t>(P.k);
  }
}

// vs_topk_logprob: the first k tokens of each row in the total order and
// their log-probabilities  z_j - log sum_i exp z_i,  z = l / T.
template <typename Raw>
__device__ __forceinline__ void topk_row(const TopkParams& P, int row) {
  RsShared& sh = rs_shared();
  RsRow<Raw> R;
  R.init(P.logits, row, P.ld, P.vocab);
  int32_t* ids = P.ids + static_cast<int64_t>(row) * P.out_ld;
  float* lps = P.logprob ? P.logprob + static_cast<int64_t>(row) * P.out_ld : nullptr;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float t = P.temperature ? P.temperature[row] : P.temperature_scalar;
  const bool fine = t >= kLeastT && t < kInf;

  cta_sync();  // the geometry
  const uint32_t kmax = rs_max<Raw>();
  const bool finite = kmax < KeyTraits<Raw>::kInfKey;
  const bool empty = finite && kmax <= RsRow<Raw>::kMaskedKey;
  if (!finite || !fine || empty) {
    if (R.rank == 0) {
      for (int i = tid; i < P.k; i += kRsThreads) {
        ids[i] = -1;
        if (lps) lps[i] = empty && fine ? -kInf : __int_as_float(0x7FC00000);
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
  const float c2 = 2.f * exponent_factor(t);
  if (lps) {
    float z = 0.f;
    R.each([&](int, const auto& r) {
#pragma unroll
      for (int i = 0; i < RsRow<Raw>::VEC; ++i) z += ex2(half_diff(value_of(r[i]), vmax) * c2);
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    if (lane == 0) sh.fred[warp] = z;
    cta_sync();
    if (warp == 0) {
      z = lane < kRsWarps ? sh.fred[lane] : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
      if (lane == 0) sh.xf[0] = z;
    }
  }

  uint32_t n = 0u, nk = 0u;
  const uint32_t floor_key = max(rs_topk_floor<Raw>(P.k), RsRow<Raw>::kMaskedKey + 1u);
  n = rs_collect<Raw>(true, floor_key, kmax);
  if (n > static_cast<uint32_t>(kRsCap)) n = topk_general(P, R, vmax, t, kmax);
  nk = min(static_cast<uint32_t>(P.k), n);
  if (R.rank == 0) {
    float z = 0.f;
    if (lps)
      for (int r = 0; r < R.C; ++r) z += R.peer(sh.xf, r)[0];
    rs_sort(n, nk);
    for (int i = tid; i < P.k; i += kRsThreads) {
      const bool in = static_cast<uint32_t>(i) < nk;
      const u64 e = in ? sh.sorted[i] : 0ull;
      ids[i] = in ? static_cast<int32_t>(~static_cast<uint32_t>(e)) : -1;
      if (lps)
        lps[i] = in ? 2.f * (half_diff(KeyTraits<Raw>::decode(static_cast<uint32_t>(e >> 32)), vmax) / t) - logf(z)
                    : -kInf;
    }
    if (tid == 0 && P.status) P.status[row] = 0u;
  }
  R.sync();  // the leader reads the peers' sums
}

// One cluster per row: vocabularies beyond the list kernel's shared memory.
template <typename Raw>
__global__ void __launch_bounds__(kRsThreads, 1) topk_kernel(const __grid_constant__ TopkParams P) {
  topk_row<Raw>(P, static_cast<int>(blockIdx.x / cg::this_cluster().num_blocks()));
}

}  // namespace

cudaError_t launch_topk(const TopkParams& P, vs_dtype dtype, cudaStream_t s) {
  bool done = false;
  const cudaError_t e = launch_topk_list(P, dtype, s, &done);
  if (e != cudaSuccess || done) return e;
  const int c = row_cluster_size(P.rows, P.vocab);
  return dtype == VS_BF16 ? launch_rows<topk_kernel<uint16_t>>(P, P.rows, c, false, s)
                          : launch_rows<topk_kernel<uint32_t>>(P, P.rows, c, false, s);
}

}  // namespace vs
