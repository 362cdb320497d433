// Truncated sampling: min-p, top-k and top-p on a row of logits, the draws
// from what is left, and the same truncation as -inf in the logits.
//
// A row's truncation is one threshold on its logits (M the largest, w(x) =
// exp((z(x) - M) / T)):
//   theta_m = M + T ln(min_p)
//   theta_k = the k-th largest z
//   theta_p = the largest z(x) with sum of w over A, z >= z(x), at least top_p
//             times the sum over A, where A = {z >= max(theta_m, theta_k)}
// and a draw is the smallest id whose cumulative weight among z >= theta
// exceeds u times their total.
//
// Weights.  Which id is drawn, and which token is the nucleus's last, turn on
// sums over the whole row next to a border, so weights are fixed-point integers
// (2^-35 of about the largest): sums are exact and the same in any order.  What
// is left is a weight's own error.  z c (c = log2(e) / T in two parts) is taken
// with its rounding error by an fma, whole powers leave exactly, and 2^g - 1 is
// added to 1 as an integer, so that a weight is off by about 2^-27 of itself
// (a plain exp2f((z - M) c) by 2^-20 at z - M = -20 T): few draws lie near enough
// to a border to differ from the same draws in 64 bits.
//
// Layout.  A cluster of up to eight CTAs takes a row; each keeps its part in
// shared memory, so the row is read once.  The ids that can matter are often
// few: min-p is a bound by itself, and with top-k up to the number of warps the
// k-th largest of the warps' maxima is one that at least k logits reach.  Where
// at most kList ids pass these bounds, they are gathered and one CTA sorts them and
// decides; else a histogram (2048 bins over the distance from M, added up over
// the cluster) finds the bin of the threshold, whose ids are gathered and
// sorted, or, if they are too many, put in finer bins.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace spec {
namespace {

constexpr int kT = 512;
constexpr int kW = kT / 32;
constexpr int kMaxC = 8;
constexpr int kBins = 2048;
constexpr int kList = kT;
constexpr float kPerBit = kBins / 37.5f;  // bins to a halving of the weight: weights end before the bins
constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds |x| < 2^22 to an integer

using u64 = unsigned long long;

struct Shared {
  union {
    unsigned hist[2][kBins];
    struct {           // where a list is put in order
      u64 pulled[kList];
      u64 ordered[kList];
      u64 cum[kList];
    } l;
  };
  u64 ex[2][2][kMaxC];   // values exchanged within the cluster, two sets in turn
  u64 red[kW];
  u64 seg[kW];           // weight of each warp's ids
  u64 list[kList];       // this CTA's gathered ids
  unsigned wmax[kMaxC * kW];  // the largest of every warp of the cluster (keys)
  unsigned n, lo, hi;    // ids gathered, the ends of their keys
  float bound, theta_m, sum_inv;
  double c;
};

constexpr size_t kSharedBytes = (sizeof(Shared) + 15) / 16 * 16;
constexpr size_t smem_bytes(int V, int C) {
  return kSharedBytes + (static_cast<size_t>((V + 3) / 4) + C - 1) / C * sizeof(float4);
}

// ---------------------------------------------------------------- cluster
SPEC_DEVINL unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
SPEC_DEVINL unsigned cluster_size() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
SPEC_DEVINL void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
SPEC_DEVINL uint32_t remote(const void* p, unsigned rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
SPEC_DEVINL void st_remote(uint32_t a, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
SPEC_DEVINL u64 ld_remote64(uint32_t a) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}
SPEC_DEVINL uint4 ld_remote4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

SPEC_DEVINL void st_remote32(uint32_t a, unsigned v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// Order-preserving key of a float that is not NaN.
SPEC_DEVINL unsigned key_of(float z) {
  const unsigned b = __float_as_uint(z);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
SPEC_DEVINL float key_value(unsigned k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }

SPEC_DEVINL u64 warp_sum64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
SPEC_DEVINL u64 warp_incl64(u64 v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  return v;
}

// floor(f x z) (+ 1 if that is not exact and up) of f in [0, 1] and z < 2^63, exactly.
SPEC_DEVINL u64 part_of(u64 z, float f, bool up) {
  const unsigned b = __float_as_uint(f);
  const int e = static_cast<int>(b >> 23);
  if (e == 0) return up && f > 0.f ? 1ull : 0ull;  // below 2^-126: less than one unit
  const u64 m = (b & 0x7FFFFFu) | 0x800000u;
  const int s = 150 - e;  // f = m 2^-s, 23 <= s <= 149
  const u64 lo = z * m, hi = __umul64hi(z, m);
  u64 q, rest;
  if (s < 64) {
    q = (hi << (64 - s)) | (lo >> s);
    rest = lo << (64 - s);
  } else if (s < 128) {
    q = s == 64 ? hi : hi >> (s - 64);
    rest = lo | (s == 64 ? 0ull : hi << (128 - s));
  } else {
    q = 0;
    rest = lo | hi;
  }
  return q + (up && rest ? 1ull : 0ull);
}

// ----------------------------------------------------------------- weights
// 2^31 (2^g - 1) for |g| <= 1/2 (a little over): g times a polynomial that meets
// (2^g - 1) / g at the six Chebyshev nodes of [-0.502, 0.502], 2^-27.5 of 2^g off
// at most; its first coefficient in two parts, so that the rounding of what is added
// to 1 is the last step's alone.
SPEC_DEVINL float exp2m1_scaled(float g) {
  constexpr float k31 = 2147483648.f;
  float r = 1.5453561e-4f * k31;
  r = fmaf(r, g, 1.33913236e-3f * k31);
  r = fmaf(r, g, 9.61808181e-3f * k31);
  r = fmaf(r, g, 5.55035625e-2f * k31);
  r = fmaf(r, g, 2.40226508e-1f * k31);
  r = fmaf(r, g, 5.7428755e-9f * k31);
  return fmaf(0.693147182f * k31, g, r * g);
}

// Where z c is too large for whole powers to leave it exactly in 32 bits: 64.
// (Few values of such a row are near enough to M to have a weight.)
__device__ __noinline__ void wide_power(float z, float M, double c, int* e, float* t) {
  const double d = z == M ? 0.0 : (static_cast<double>(z) - static_cast<double>(M)) * c;
  const double n = d < -200.0 ? -200.0 : rint(d);
  *e = static_cast<int>(n);
  *t = d < -200.0 ? 0.f : exp2m1_scaled(static_cast<float>(d - n));
}

struct Weights {
  float M, c_hi, c_lo, zlow, c_bin;
  int n0, b0;  // M's power, and its first bin, as the rounded sums' bits
  int off;     // 5 or 3: weights are in units of 2^-(30 + off) of about the largest
  bool wide;
  double c;

  // w = 2^e (1 + t 2^-31); -e at least 149 where z is further than that below M
  SPEC_DEVINL void power(float z, int& e, float& t) const {
    const float x = fmaxf(z, zlow), p = __fmul_rn(x, c_hi);  // (not to be contracted: the fma gives its rounding error)
    const float nb = __fadd_rn(p, kRound);
    const float g = __fadd_rn(p, kRound - nb) + fmaf(x, c_lo, fmaf(x, c_hi, -p));
    e = __float_as_int(nb) - n0;
    t = exp2m1_scaled(g);
  }
  // 2^(30 + off) w, to the nearest
  SPEC_DEVINL u64 units(int e, float t) const {
    const unsigned m = 0x80000000u + static_cast<unsigned>(__float2int_rn(t));
    const int sh = -off - e;  // of 2^31 (1 + t) to half units
    if (sh < 0) return static_cast<u64>(m) << (-1 - sh);
    unsigned h;
    asm("shr.b32 %0, %1, %2;" : "=r"(h) : "r"(m), "r"(sh));  // (0 from 32 on)
    return (h + 1u) >> 1;
  }
  SPEC_DEVINL u64 fixed(float z) const {
    int e;
    float t;
    if (wide)
      wide_power(z, M, c, &e, &t);
    else
      power(z, e, t);
    return units(e, t);
  }
  // of four at a time
  SPEC_DEVINL void fixed4(const float4& z, u64 (&x)[4]) const {
    if (wide) {
      x[0] = fixed(z.x);
      x[1] = fixed(z.y);
      x[2] = fixed(z.z);
      x[3] = fixed(z.w);
      return;
    }
    int e[4];
    float t[4];
    power(z.x, e[0], t[0]);
    power(z.y, e[1], t[1]);
    power(z.z, e[2], t[2]);
    power(z.w, e[3], t[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = units(e[i], t[i]);
  }
  SPEC_DEVINL float real(float z) const {
    int e;
    float t;
    if (wide)
      wide_power(z, M, c, &e, &t);
    else
      power(z, e, t);
    return e < -125 ? 0.f : fmaf(t, 4.65661287e-10f, 1.f) * __int_as_float((e + 127) << 23);
  }
};

// ------------------------------------------------------------------ kernel
struct RowSet {
  float T, top_p, min_p;
  int k;
};

SPEC_DEVINL RowSet row_set(const TruncParams& p, int row) {
  const unsigned s = static_cast<unsigned>(row) / static_cast<unsigned>(p.rows_per_set);
  RowSet r;
  r.T = p.d_T ? p.d_T[s] : p.T;
  r.k = p.d_k ? p.d_k[s] : p.k;
  r.top_p = p.d_p ? p.d_p[s] : p.top_p;
  r.min_p = p.d_mp ? p.d_mp[s] : p.min_p;
  return r;
}

template <bool BF16>
SPEC_DEVINL void load4(const void* row, int x, int V, bool vec, float (&v)[4]) {
  if (vec && x + 4 <= V) {
    if (BF16) {
      const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(row) + x);
      v[0] = bf16lo(w.x);
      v[1] = bf16hi(w.x);
      v[2] = bf16lo(w.y);
      v[3] = bf16hi(w.y);
    } else {
      const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(row) + x);
      v[0] = w.x;
      v[1] = w.y;
      v[2] = w.z;
      v[3] = w.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = -INFINITY;
      if (x + e < V)
        v[e] = BF16 ? bf16_to_f32(static_cast<const uint16_t*>(row)[x + e]) : static_cast<const float*>(row)[x + e];
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (!(v[e] >= -INFINITY)) v[e] = -INFINITY;  // NaN
}

template <bool BF16>
SPEC_DEVINL void store4(void* row, int x, int V, bool vec, const float (&v)[4]) {
  if (vec && x + 4 <= V) {
    if (BF16) {
      uint2 w;  // bf16 values, their bits as they were
      w.x = (__float_as_uint(v[0]) >> 16) | (__float_as_uint(v[1]) & 0xFFFF0000u);
      w.y = (__float_as_uint(v[2]) >> 16) | (__float_as_uint(v[3]) & 0xFFFF0000u);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(row) + x) = w;
    } else {
      *reinterpret_cast<float4*>(static_cast<float*>(row) + x) = make_float4(v[0], v[1], v[2], v[3]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (x + e < V) {
        if (BF16)
          static_cast<uint16_t*>(row)[x + e] = static_cast<uint16_t>(__float_as_uint(v[e]) >> 16);
        else
          static_cast<float*>(row)[x + e] = v[e];
      }
  }
}

template <bool BF16, bool FILTER>
struct Row {
  Shared& s;
  float4* const zs;  // this CTA's ids, in groups of four
  const TruncParams& p;
  const int tid, lane, warp, rank, C;
  int par = 0;
  int V, g0;   // the first group
  int i0, i1;  // this warp's groups, within the CTA's
  int limb;    // bits of the histogram's low part
  Weights w;

  SPEC_DEVINL Row(Shared& s_, float4* zs_, const TruncParams& p_)
      : s(s_), zs(zs_), p(p_), tid(threadIdx.x), lane(threadIdx.x & 31), warp(threadIdx.x >> 5),
        rank(static_cast<int>(cluster_rank())), C(static_cast<int>(cluster_size())) {}

  // f(first id, four logits) over the CTA's groups; a warp's are contiguous.
  template <class F>
  SPEC_DEVINL void each(F&& f) const {
#pragma unroll 2
    for (int i = i0 + lane; i < i1; i += 32) {
      const float4 v = zs[i];
      f(4 * (g0 + i), v);
    }
  }
  // f(first id, z) by single logits
  template <class F>
  SPEC_DEVINL void each1(F&& f) const {
    each([&](int x, const float4& v) {
      f(x, v.x);
      f(x + 1, v.y);
      f(x + 2, v.z);
      f(x + 3, v.w);
    });
  }

  // Two values of every CTA (held by warp 0) to every CTA of the cluster.
  SPEC_DEVINL const u64 (*exchange(u64 a, u64 b))[kMaxC] {
    par ^= 1;
    if (warp == 0 && lane < C) {
      st_remote(remote(&s.ex[par][0][rank], lane), a);
      st_remote(remote(&s.ex[par][1][rank], lane), b);
    }
    cluster_barrier();
    return s.ex[par];
  }
  // one of them, of each CTA, added up
  SPEC_DEVINL u64 total_of(const u64* v) const {
    u64 t = 0;
    for (int r = 0; r < C; ++r) t += v[r];
    return t;
  }

  SPEC_DEVINL void list_clear() {
    if (tid == 0) {
      s.n = 0;
      s.lo = 0xFFFFFFFFu;
      s.hi = 0;
    }
    __syncthreads();
  }
  // (the order of the list is of no account: what reads it puts it in order first)
  SPEC_DEVINL void list_add(float v, int id, bool ends) {
    const unsigned at = atomicAdd(&s.n, 1u), k = key_of(v);
    if (at < kList) s.list[at] = entry(k, id);
    if (ends) {
      atomicMin(&s.lo, k);
      atomicMax(&s.hi, k);
    }
  }
  // larger first, the lower id of equal ones
  SPEC_DEVINL static u64 entry(unsigned key, int id) { return (static_cast<u64>(key) << 32) | ~static_cast<unsigned>(id); }
  SPEC_DEVINL static float value_of(u64 x) { return key_value(static_cast<unsigned>(x >> 32)); }
  SPEC_DEVINL static int id_of(u64 x) { return static_cast<int>(~static_cast<unsigned>(x)); }

  // The cluster's lists (counts[r] entries of CTA r) to this CTA.
  SPEC_DEVINL void pull(const u64* counts, int n) {
    if (tid < n) {
      int r = 0, at = tid;
      while (at >= static_cast<int>(counts[r])) at -= static_cast<int>(counts[r++]);
      s.l.pulled[tid] = ld_remote64(remote(&s.list[at], r));
    }
    __syncthreads();
  }
  // ordered[0 .. n) = pulled by value and id, or (BY_ID) by id, by counting for each entry those
  // before it, a few threads an entry.
  template <bool BY_ID>
  SPEC_DEVINL void order(int n) {
    int lg = 0;
    while ((kT >> (lg + 1)) >= n && lg < 5) ++lg;
    const int i = tid >> lg, part = tid & ((1 << lg) - 1), step = 1 << lg;
    const u64 x = i < n ? s.l.pulled[i] : 0ull;
    int c = 0;
    if (i < n) {
#pragma unroll 8
      for (int j = part; j < n; j += step) {
        const u64 y = s.l.pulled[j];
        c += BY_ID ? (static_cast<unsigned>(y) > static_cast<unsigned>(x) ? 1 : 0) : (y > x ? 1 : 0);
      }
    }
    for (int o = 1; o < step; o <<= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    if (i < n && part == 0) s.l.ordered[c] = x;
    __syncthreads();
  }

  // cum[i] = inclusive sums of thread i's v, i < n; the total.
  SPEC_DEVINL u64 scan(int n, u64 v) {
    const u64 incl = warp_incl64(v, lane);
    if (lane == 31) s.red[warp] = incl;
    __syncthreads();
    u64 before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      const u64 x = s.red[i];
      if (i < warp) before += x;
      all += x;
    }
    if (tid < n) s.l.cum[tid] = before + incl;
    __syncthreads();
    return all;
  }
  // first i < n with cum[i] >= x (n if none); cum does not fall
  SPEC_DEVINL int find(int n, u64 x) const {
    int lo = 0, hi = n;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (s.l.cum[mid] >= x)
        hi = mid;
      else
        lo = mid + 1;
    }
    return lo;
  }

  // The largest value v with (MASS: weight, else number) of {lower <= z, z >= v}
  // at least the target: top_p of the whole, or k.  -inf if there is none.
  template <bool MASS>
  SPEC_DEVINL float select(float lower, float span, float top_p, int k) {
    // first bins: distance from M, linear (numbers: 256 to the span; weights: 54 to a halving); later
    // ones: keys khi down to klo
    const float scale = MASS ? fminf(w.c_hi, 1e28f) * kPerBit : (span > 0.f && span < 1e30f ? (kBins / 8) / span : 0.f);
    unsigned khi = 0xFFFFFFFFu, klo = 0;
    int shift = -1;
    u64 target = static_cast<u64>(k);
    auto in = [&](float v) {
      if (!(v >= lower) || v == -INFINITY) return false;
      if (shift < 0) return true;
      const unsigned kv = key_of(v);
      return kv >= klo && kv <= khi;
    };
    auto bin = [&](float v) -> int {
      if (shift >= 0) return static_cast<int>((khi - key_of(v)) >> shift);
      if (MASS && !w.wide) return min(w.b0 - __float_as_int(fmaf(fmaxf(v, w.zlow), w.c_bin, kRound)), kBins - 1);
      return min(static_cast<int>((w.M - v) * scale), kBins - 1);
    };
    __syncthreads();  // (hist lies where the last list was put in order)
    for (;;) {
      for (int i = tid; i < (MASS ? kBins / 2 : kBins / 4); i += kT)
        reinterpret_cast<uint4*>(s.hist)[i] = make_uint4(0, 0, 0, 0);
      list_clear();
      each([&](int, const float4& z) {
        const float v[4] = {z.x, z.y, z.z, z.w};
        if (MASS) {
          u64 x[4];
          w.fixed4(z, x);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (in(v[e])) {
              const int b = bin(v[e]);
              const unsigned lo = static_cast<unsigned>(x[e]) & ((1u << limb) - 1u),
                             hi = static_cast<unsigned>(x[e] >> limb);
              if (lo) atomicAdd(&s.hist[0][b], lo);
              if (hi) atomicAdd(&s.hist[1][b], hi);
            }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (in(v[e])) atomicAdd(&s.hist[0][bin(v[e])], 1u);
        }
      });
      cluster_barrier();
      // four bins a thread, each CTA its part of them
      const int per = kT / C;  // threads that have bins
      u64 q[4] = {0, 0, 0, 0};
      if (tid < per) {
        const int b0 = 4 * (rank * per + tid);
#pragma unroll 4
        for (int r = 0; r < C; ++r) {
          const uint4 lo = ld_remote4(remote(&s.hist[0][b0], r));
          const uint4 hi = MASS ? ld_remote4(remote(&s.hist[1][b0], r)) : make_uint4(0, 0, 0, 0);
          q[0] += lo.x + (static_cast<u64>(hi.x) << limb);
          q[1] += lo.y + (static_cast<u64>(hi.y) << limb);
          q[2] += lo.z + (static_cast<u64>(hi.z) << limb);
          q[3] += lo.w + (static_cast<u64>(hi.w) << limb);
        }
      }
      const u64 mine = q[0] + q[1] + q[2] + q[3];
      const u64 incl = warp_incl64(mine, lane);
      if (lane == 31) s.red[warp] = incl;
      __syncthreads();
      u64 excl = incl - mine, part = 0;
      for (int i = 0; i < kW; ++i) {
        if (i < warp) excl += s.red[i];
        part += s.red[i];
      }
      const u64(*ex)[kMaxC] = exchange(part, 0);
      u64 all = 0;
      for (int r = 0; r < C; ++r) {
        if (r < rank) excl += ex[0][r];
        all += ex[0][r];
      }
      if (shift < 0 && MASS) target = part_of(all, top_p, true);
      if (all < target) return -INFINITY;  // (the first time round only: fewer than k)
      // the bin that the target lies in, told to every CTA
      par ^= 1;
      if (tid < per && excl < target && target <= excl + mine) {
        int i = 0;
        while (excl + q[i] < target) excl += q[i++];
        const u64 b = 4 * (rank * per + tid) + i;
        for (int r = 0; r < C; ++r) {
          st_remote(remote(&s.ex[par][0][0], r), b);
          st_remote(remote(&s.ex[par][1][0], r), excl);
        }
      }
      cluster_barrier();
      const int b = static_cast<int>(s.ex[par][0][0]);
      target -= s.ex[par][1][0];
      each1([&](int x, float v) {
        if (bin(v) == b && in(v)) list_add(v, x, true);
      });
      __syncthreads();
      ex = exchange(s.n, (static_cast<u64>(s.lo) << 32) | s.hi);
      int n = 0;
      unsigned lo = 0xFFFFFFFFu, hi = 0;
      for (int r = 0; r < C; ++r) {
        n += static_cast<int>(ex[0][r]);
        lo = min(lo, static_cast<unsigned>(ex[1][r] >> 32));
        hi = max(hi, static_cast<unsigned>(ex[1][r]));
      }
      if (lo == hi) return key_value(lo);  // one value
      if (n <= kList) {  // (each CTA finds it for itself)
        pull(ex[0], n);
        order<false>(n);
        const float v = tid < n ? value_of(s.l.ordered[tid]) : 0.f;
        scan(n, tid < n ? (MASS ? w.fixed(v) : 1ull) : 0ull);
        return value_of(s.l.ordered[min(find(n, target), n - 1)]);
      }
      klo = lo;
      khi = hi;
      shift = 0;
      while (((khi - klo) >> shift) >= kBins) ++shift;
    }
  }

  // Every output of a row but its draws: value(z, id).
  template <class F>
  SPEC_DEVINL void write_row(int row, F&& value) {
    void* base;
    bool vec;
    if (FILTER) {
      base = static_cast<char*>(p.out) + static_cast<long long>(row) * p.out_ld * (BF16 ? 2 : 4);
      vec = (reinterpret_cast<uintptr_t>(base) & (BF16 ? 7 : 15)) == 0;
    } else {
      base = p.probs + static_cast<long long>(row) * p.probs_ld;
      vec = (reinterpret_cast<uintptr_t>(base) & 15) == 0;
    }
    each([&](int x, const float4& z) {
      const float v[4] = {value(z.x, x), value(z.y, x + 1), value(z.z, x + 2), value(z.w, x + 3)};
      store4 < BF16 && FILTER > (base, x, V, vec, v);
    });
  }
  SPEC_DEVINL void write_kept(int row, float theta, u64 total) {
    if (FILTER) {
      write_row(row, [&](float v, int) { return v >= theta ? v : -INFINITY; });
    } else if (p.probs) {
      if (tid == 0) s.sum_inv = static_cast<float>(static_cast<double>(1ull << (30 + w.off)) / static_cast<double>(total));
      __syncthreads();
      const float inv = s.sum_inv;
      write_row(row, [&](float v, int) { return v >= theta ? w.real(v) * inv : 0.f; });
    }
  }
  // one id alone (T = 0), or, id -1, a row with nothing to draw
  SPEC_DEVINL void write_single(int row, int only) {
    if (FILTER) {
      write_row(row, [&](float v, int x) { return only < 0 || x == only ? v : -INFINITY; });
    } else {
      if (rank == 0)
        for (int d = tid; d < p.draws; d += kT) p.tokens[static_cast<long long>(row) * p.draws + d] = only;
      if (p.probs) write_row(row, [&](float, int x) { return x == only ? 1.f : 0.f; });
    }
  }
  SPEC_DEVINL u64 draw_target(int row, int d, u64 total) const {
    const float u = p.u[static_cast<long long>(row) * p.draws + d];
    if (!(u > 0.f)) return 0;
    return u >= 1.f ? total - 1 : min(part_of(total, u, false), total - 1);
  }

  SPEC_DEVINL void run(int row) {
    V = p.V;
    const int groups = (V + 3) >> 2, per = (groups + C - 1) / C;
    g0 = rank * per;
    const int gn = max(0, min(per, groups - g0));
    const int wg = (gn + kT - 1) / kT * 32;
    i0 = min(warp * wg, gn);
    i1 = min(i0 + wg, gn);
    // a CTA's part of a bin fits two 32-bit counters: 2^14 ids of up to 2^35.5, or 2^15 of up to 2^33.5
    w.off = V <= 131072 ? 5 : 3;
    limb = V <= 131072 ? 18 : 17;
    const char* base = static_cast<const char*>(p.z) + static_cast<long long>(row) * p.ld * (BF16 ? 2 : 4);
    const bool vec = (reinterpret_cast<uintptr_t>(base) & (BF16 ? 7 : 15)) == 0;
    float top = -INFINITY;
    constexpr int kAhead = 8;  // loads on their way at once
    for (int i = i0 + lane; i < i1; i += 32 * kAhead) {
      float v[kAhead][4];
#pragma unroll
      for (int q = 0; q < kAhead; ++q)
        if (i + 32 * q < i1) load4<BF16>(base, 4 * (g0 + i + 32 * q), V, vec, v[q]);
#pragma unroll
      for (int q = 0; q < kAhead; ++q)
        if (i + 32 * q < i1) {
          zs[i + 32 * q] = make_float4(v[q][0], v[q][1], v[q][2], v[q][3]);
          top = fmaxf(top, fmaxf(fmaxf(v[q][0], v[q][1]), fmaxf(v[q][2], v[q][3])));
        }
    }
    const RowSet rs = row_set(p, row);
    const bool bad = !(rs.T >= 0.f) || rs.T > 3.4028234e38f || rs.k < 0 || !(rs.top_p > 0.f && rs.top_p <= 1.f) ||
                     !(rs.min_p >= 0.f && rs.min_p <= 1.f);
    list_clear();
    // every warp's maximum to every CTA
    const unsigned kt = __reduce_max_sync(0xffffffffu, key_of(top));
    if (lane < C) st_remote32(remote(&s.wmax[rank * kW + warp], lane), kt);
    cluster_barrier();
    const int nw = C * kW;  // (the lists' order of the keys)
    unsigned km = 0, kmin = 0xFFFFFFFFu;
    for (int i = lane; i < nw; i += 32) {
      km = max(km, s.wmax[i]);
      kmin = min(kmin, s.wmax[i]);
    }
    const float M = key_value(__reduce_max_sync(0xffffffffu, km));
    const float least = key_value(__reduce_min_sync(0xffffffffu, kmin));
    if (bad || M == -INFINITY) {
      if (rank == 0 && tid == 0) set_status(p.status, bad ? SPEC_DEV_BAD_PARAM : SPEC_DEV_EMPTY_MASK);
      write_single(row, -1);
      return;
    }
    if (rs.T == 0.f) {  // the lowest id of the largest
      each1([&](int x, float v) {
        if (v == M) atomicMin(&s.lo, static_cast<unsigned>(x));
      });
      __syncthreads();
      const u64(*ex)[kMaxC] = exchange(s.lo, 0);
      unsigned first = 0xFFFFFFFFu;
      for (int r = 0; r < C; ++r) first = min(first, static_cast<unsigned>(ex[0][r]));
      write_single(row, static_cast<int>(first));
      return;
    }
    // log2(e) / T in two parts
    const float c_hi = __fdiv_rn(1.44269502f, rs.T);
    const float far = fabsf(M) * c_hi;
    w.M = M;
    w.c_hi = c_hi;
    w.c_lo = __fdiv_rn(fmaf(-c_hi, rs.T, 1.44269502f) + 1.92596303e-8f, rs.T);
    w.wide = !(far < 70000.f) || !(c_hi < 1e30f) || !(c_hi > 1e-25f);
    w.zlow = w.wide ? 0.f : M - __fdividef(150.f, c_hi);
    w.n0 = __float_as_int(__fadd_rn(__fmul_rn(M, c_hi), kRound));
    w.c_bin = c_hi * kPerBit;
    w.b0 = __float_as_int(fmaf(M, w.c_bin, kRound));
    const bool top_k = rs.k > 0 && rs.k < V, top_p = rs.top_p < 1.f, few_k = top_k && rs.k <= nw;
    float lower = -INFINITY;
    if (rs.min_p > 0.f || w.wide || few_k || M == INFINITY) {
      if (tid == kT - 1) {
        s.c = 1.4426950408889634074 / static_cast<double>(rs.T);
        s.theta_m = M == INFINITY ? INFINITY
                    : rs.min_p > 0.f
                        ? __double2float_ru(static_cast<double>(M) + static_cast<double>(rs.T) * log(static_cast<double>(rs.min_p)))
                        : -INFINITY;
      }
      if (tid == 0) s.bound = -INFINITY;
      __syncthreads();
      // the k-th largest of the warps' maxima: that many logits at least reach it
      if (few_k) {
        const int lg = C == 8 ? 2 : C == 4 ? 3 : C == 2 ? 4 : 5;  // kT / nw threads a value
        const int i = tid >> lg;
        const unsigned mine = s.wmax[i];
        int c = 0;
#pragma unroll 8
        for (int j = tid & ((1 << lg) - 1); j < nw; j += 1 << lg) {
          const unsigned y = s.wmax[j];
          c += y > mine || (y == mine && j < i) ? 1 : 0;
        }
        for (int o = 1; o < 1 << lg; o <<= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
        if (c == rs.k - 1) s.bound = key_value(mine);
        __syncthreads();
      }
      w.c = s.c;
      lower = fmaxf(s.theta_m, s.bound);
    }
    const u64(*ex)[kMaxC];
    int n = kList + 1;
    if (lower > -INFINITY || V <= kList) {
      each([&](int x, const float4& v) {
        if (fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)) < lower) return;
        if (*const_cast<volatile unsigned*>(&s.n) > kList) return;  // too many already
        if (v.x >= lower && v.x > -INFINITY) list_add(v.x, x, false);
        if (v.y >= lower && v.y > -INFINITY) list_add(v.y, x + 1, false);
        if (v.z >= lower && v.z > -INFINITY) list_add(v.z, x + 2, false);
        if (v.w >= lower && v.w > -INFINITY) list_add(v.w, x + 3, false);
      });
      __syncthreads();
      ex = exchange(s.n, 0);
      n = static_cast<int>(total_of(ex[0]));
    }
    float theta = lower;
    u64 total = 0;
    if (n <= kList) {  // few: one CTA decides
      if (rank == 0) {
        pull(ex[0], n);
        const bool cut = top_k && n > rs.k;
        if (cut || top_p) {
          order<false>(n);
          if (cut) theta = value_of(s.l.ordered[rs.k - 1]);
          if (top_p) {
            const float v = tid < n ? value_of(s.l.ordered[tid]) : 0.f;
            const u64 all = scan(n, tid < n && v >= theta ? w.fixed(v) : 0ull);
            theta = fmaxf(theta, value_of(s.l.ordered[min(find(n, part_of(all, rs.top_p, true)), n - 1)]));
          }
          __syncthreads();  // ordered and cum are read before they are written again
        }
        if (!FILTER) {
          order<true>(n);
          const float v = tid < n ? value_of(s.l.ordered[tid]) : 0.f;
          total = scan(n, tid < n && v >= theta ? w.fixed(v) : 0ull);
          for (int d = tid; d < p.draws; d += kT)
            p.tokens[static_cast<long long>(row) * p.draws + d] =
                id_of(s.l.ordered[find(n, draw_target(row, d, total) + 1)]);
        }
      }
      ex = exchange(key_of(theta), total);  // (and no CTA leaves before its list is read)
      if (FILTER || p.probs) write_kept(row, key_value(static_cast<unsigned>(ex[0][0])), ex[1][0]);
      return;
    }
    if (top_k) theta = fmaxf(theta, select<false>(lower, M - least, 0.f, rs.k));
    if (top_p) theta = fmaxf(theta, select<true>(theta, 0.f, rs.top_p, 0));
    if (FILTER) {
      write_kept(row, theta, 0);
      cluster_barrier();  // no CTA leaves before its list is read
      return;
    }
    // the warps' weights, and the cluster's
    u64 sum = 0;
    each([&](int, const float4& v) {
      if (fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)) < theta) return;
      u64 x[4];
      w.fixed4(v, x);
      sum += (v.x >= theta ? x[0] : 0) + (v.y >= theta ? x[1] : 0) + (v.z >= theta ? x[2] : 0) +
             (v.w >= theta ? x[3] : 0);
    });
    sum = warp_sum64(sum);
    if (lane == 0) s.seg[warp] = sum;
    __syncthreads();
    sum = 0;
    for (int i = 0; i < kW; ++i) sum += s.seg[i];
    ex = exchange(sum, 0);
    u64 before = 0;
    for (int r = 0; r < C; ++r) {
      if (r < rank) before += ex[0][r];
      total += ex[0][r];
    }
    for (int d = warp; d < p.draws; d += kW) {
      u64 x = draw_target(row, d, total);
      if (x < before || x >= before + sum) continue;
      x -= before;
      // the warp's piece, then 128 ids, the lane and the id whose cumulative weight passes x
      int piece = 0;
      while (piece < kW - 1 && s.seg[piece] <= x) x -= s.seg[piece++];
      const int j1 = min((piece + 1) * wg, gn);
      for (int j = piece * wg; j < j1; j += 32) {
        const float4 v = j + lane < j1 ? zs[j + lane] : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        u64 f[4];
        w.fixed4(v, f);
        const u64 f0 = v.x >= theta ? f[0] : 0, f1 = v.y >= theta ? f[1] : 0, f2 = v.z >= theta ? f[2] : 0,
                  f3 = v.w >= theta ? f[3] : 0;
        const u64 t = f0 + f1 + f2 + f3, incl = warp_incl64(t, lane);
        const unsigned past = __ballot_sync(0xffffffffu, incl > x);
        if (past) {
          if (lane == __ffs(past) - 1) {
            const u64 y = x - (incl - t);
            const int e = y < f0 ? 0 : y < f0 + f1 ? 1 : y < f0 + f1 + f2 ? 2 : 3;
            p.tokens[static_cast<long long>(row) * p.draws + d] = 4 * (g0 + j + lane) + e;
          }
          break;
        }
        x -= __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    write_kept(row, theta, total);
  }
};

template <bool BF16, bool FILTER>
__global__ void __launch_bounds__(kT, 2) trunc_kernel(const TruncParams p) {
  extern __shared__ __align__(16) char smem[];
  grid_dep_wait();
  grid_dep_launch();
  Row<BF16, FILTER> r(*reinterpret_cast<Shared*>(smem), reinterpret_cast<float4*>(smem + kSharedBytes), p);
  r.run(static_cast<int>(blockIdx.x / static_cast<unsigned>(r.C)));
}

template <bool BF16, bool FILTER>
cudaError_t launch(const TruncParams& p, cudaLaunchConfig_t& cfg) {
  // the most a CTA of any call takes, asked for once per device
  static PerDevice<cudaError_t> set;
  cudaError_t e = cudaSuccess;
  if (!set.get(
          [] {
            return cudaFuncSetAttribute(trunc_kernel<BF16, FILTER>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        static_cast<int>(smem_bytes(kTruncMaxVocab, kMaxC)));
          },
          &e))
    return cudaErrorInvalidDevice;
  if (e != cudaSuccess) return e;
  return cudaLaunchKernelEx(&cfg, trunc_kernel<BF16, FILTER>, p);
}

}  // namespace

cudaError_t launch_trunc(const TruncParams& p, int sms, cudaStream_t stream) {
  const int groups = (p.V + 3) / 4;
  // as many CTAs as leave two to an SM, or, where SMs are left over, one for every
  // 512 groups: a row alone takes the less time the more share it
  int C = 1;
  while (C < kMaxC && (groups > C * kT * 8 || (groups > C * kT && p.rows * 2 * C <= sms))) C *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.rows) * C);
  cfg.blockDim = dim3(kT);
  cfg.dynamicSmemBytes = smem_bytes(p.V, C);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (p.bf16) return p.out ? launch<true, true>(p, cfg) : launch<true, false>(p, cfg);
  return p.out ? launch<false, true>(p, cfg) : launch<false, false>(p, cfg);
}

}  // namespace spec
