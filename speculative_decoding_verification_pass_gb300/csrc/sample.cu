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
// added to 1 as an integer, so that a weight is off by at most 2^-23.6 of itself
// (a plain exp2f((z - M) c) by 2^-20 at z - M = -20 T): few draws lie near enough
// to a border to differ from the same draws in 64 bits.
//
// Layout.  A cluster of one to eight CTAs takes a row, each CTA a part, each warp
// a part of that.  The row is read from memory once and, by the later passes, from
// the caches.  The ids that can matter are often few: min-p is a bound by
// itself, and with top-k up to 128 the k-th largest of the maxima of 128 parts of
// the row is one that at least k logits reach.  Where at most 256 ids pass these
// bounds, they are gathered and one CTA decides.  Else the ids are counted in 4096
// bins of the distance from M: a bin's weight is its number times the weight at its
// middle to within 0.24%, so the bins where the nucleus ends are known but for a few; one
// pass over the weights then gives their total, what lies above those bins, and
// the few ids in them, among which the threshold is found.  (Should it lie
// elsewhere, or the ids be too many, histograms of the weights part them by their
// bits.)
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace spec {
namespace {

using u64 = unsigned long long;

constexpr int kT = 512;
constexpr int kW = kT / 32;
constexpr int kMaxC = 8;
constexpr int kBins = 64;             // of a level
constexpr int kFine = kBins * kBins;  // of two
constexpr int kFar = kFine - 6;       // the last that a logit falls in, but for rounding
constexpr int kPieces = 8;            // of a warp's part, whose weights are kept
constexpr int kList = 1024;
constexpr int kFew = 256;              // candidates that one CTA decides about (by comparing each with each)
constexpr int kHeavyBits = 6;         // ids of more than 2^-6 of the largest weight are few, and weighed one by one
constexpr float kPerBit = kFar / 28.f;  // fine bins to a halving of the weight: 262144 ids past them weigh 2^-10
constexpr int kLarge = 5;  // weights above 2^-5 of the largest are few
constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds |x| < 2^22 to an integer

struct Shared {
  union {
    unsigned fine[kFine];
    struct {
      unsigned hist[2][kBins][32];  // a column a lane: no two lanes of a warp meet in a bank
      u64 bins[kMaxC][kBins];       // every CTA's
    } h;
    struct {
      u64 x[kList];  // the cluster's list
      u64 weight[kList];
      u64 targets[kTruncMaxDraws];
    } l;
  };
  u64 list[kList];           // this CTA's gathered ids
  u64 sums[kBins];
  u64 ex[2][4][kMaxC];       // values exchanged within the cluster, two sets in turn
  u64 red[kW];
  u64 seg[kW * kPieces];     // weights of the pieces
  unsigned wmax[kMaxC * kW]; // the largest of 128 parts of the row (keys)
  unsigned n, lo, hi;        // ids gathered, the ends of their keys
  float bound, theta_m, sum_inv;
  double c;
};

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
// The cluster's first barrier in two halves: no CTA writes to another's shared memory before that has started.
SPEC_DEVINL void cluster_started() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
SPEC_DEVINL void cluster_all_started() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
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
// N words in a row, of an address that is a multiple of as many (or of four)
template <int N>
SPEC_DEVINL void ld_remote_n(uint32_t a, unsigned (&v)[N]) {
  if constexpr (N == 1) {
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v[0]) : "r"(a) : "memory");
  } else if constexpr (N == 2) {
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(a) : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3])
                   : "r"(a + 4 * i)
                   : "memory");
  }
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
// Two fp32 values in one register pair, and operations on both at once.
SPEC_DEVINL u64 pair(float a, float b) {
  u64 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
SPEC_DEVINL float2 parts(u64 x) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(x));
  return f;
}
SPEC_DEVINL u64 both(float a) { return pair(a, a); }
SPEC_DEVINL u64 fma2(u64 a, u64 b, u64 c) {
  u64 r;
  asm("fma.rn.ftz.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
SPEC_DEVINL u64 mul2(u64 a, u64 b) {
  u64 r;
  asm("mul.rn.ftz.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 2^31 (2^g - 1) for |g| <= 1/2 (a little over): g times a polynomial that meets
// (2^g - 1) / g at the six Chebyshev nodes of [-0.502, 0.502], 2^-27.5 of 2^g off
// at most; its first coefficient in two parts, so that the rounding of what is added
// to 1 is the last step's alone.
SPEC_DEVINL u64 exp2m1_scaled(u64 g) {
  constexpr float k31 = 2147483648.f;
  u64 r = both(1.5453561e-4f * k31);
  r = fma2(r, g, both(1.33913236e-3f * k31));
  r = fma2(r, g, both(9.61808181e-3f * k31));
  r = fma2(r, g, both(5.55035625e-2f * k31));
  r = fma2(r, g, both(2.40226508e-1f * k31));
  r = fma2(r, g, both(5.7428755e-9f * k31));
  return fma2(both(0.693147182f * k31), g, mul2(r, g));
}

// Where z c is too large for whole powers to leave it exactly in 32 bits: 64.
// (Few values of such a row are near enough to M to have a weight.)  e, and t's bits: by address, they would
// lie in memory for every row (320 rows top-p 177 us, mixed filter 107; so 167 and 105).
__device__ __noinline__ int2 wide_power(float z, float M, double c) {
  const double d = z == M ? 0.0 : (static_cast<double>(z) - static_cast<double>(M)) * c;
  const double n = d < -200.0 ? -200.0 : rint(d);
  const float t = d < -200.0 ? 0.f : parts(exp2m1_scaled(both(static_cast<float>(d - n)))).x;
  return make_int2(static_cast<int>(n), __float_as_int(t));
}

__device__ u64 one_weight(float z, float M, float c_hi, float c_lo, float zlow, int n0, bool wide, double c);

struct Weights {
  float M, c_hi, c_lo, zlow;
  int n0;   // M's power, as the rounded sum's bits
  bool wide;
  double c;

  // w = 2^e (1 + t 2^-31) of two; -e at least 149 where z is further than that below M
  SPEC_DEVINL void power2(float a, float b, int (&e)[2], float (&t)[2]) const {
    const u64 x = pair(fmaxf(a, zlow), fmaxf(b, zlow)), c2 = both(c_hi), round = both(kRound);
    const u64 nb = fma2(x, c2, round);                   // the whole powers
    const u64 f = fma2(x, c2, fma2(nb, both(-1.f), round));  // what is left, with the product's rounding error
    const float2 n = parts(nb), r = parts(exp2m1_scaled(fma2(x, both(c_lo), f)));
    e[0] = __float_as_int(n.x) - n0;
    e[1] = __float_as_int(n.y) - n0;
    t[0] = r.x;
    t[1] = r.y;
  }
  SPEC_DEVINL void power4(const float4& z, int (&e)[4], float (&t)[4]) const {
    if (wide) {
      const float v[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int2 x = wide_power(v[i], M, c);
        e[i] = x.x;
        t[i] = __int_as_float(x.y);
      }
      return;
    }
    int e0[2], e1[2];
    float t0[2], t1[2];
    power2(z.x, z.y, e0, t0);
    power2(z.z, z.w, e1, t1);
    e[0] = e0[0];
    e[1] = e0[1];
    e[2] = e1[0];
    e[3] = e1[1];
    t[0] = t0[0];
    t[1] = t0[1];
    t[2] = t1[0];
    t[3] = t1[1];
  }
  // 2^35 w, to the nearest, of weights below 2^-5 (as most are: larger ones give 0 here, and all of
  // their weight in large)
  SPEC_DEVINL unsigned units(int e, float t) const {
    unsigned h;
    asm("shr.b32 %0, %1, %2;" : "=r"(h) : "r"(mantissa(t)), "r"(-kLarge - e));  // (0 from 32 on, and for less than 0)
    return (h + 1u) >> 1;
  }
  SPEC_DEVINL bool is_large(int e) const { return e > -kLarge; }
  SPEC_DEVINL u64 large(int e, float t) const { return static_cast<u64>(mantissa(t)) << (kLarge + e - 1); }
  SPEC_DEVINL static unsigned mantissa(float t) { return 0x80000000u + static_cast<unsigned>(__float2int_rn(t)); }
  SPEC_DEVINL u64 fixed(float z) const { return one_weight(z, M, c_hi, c_lo, zlow, n0, wide, c); }
  SPEC_DEVINL void fixed4(const float4& z, u64 (&x)[4]) const {
    int e[4];
    float t[4];
    power4(z, e, t);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = units(e[i], t[i]);
    if (max(max(e[0], e[1]), max(e[2], e[3])) > -kLarge) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (is_large(e[i])) x[i] = large(e[i], t[i]);
    }
  }
  SPEC_DEVINL static float real(int e, float t, float scale) {
    return e < -125 ? 0.f : fmaf(t, 4.65661287e-10f, 1.f) * __int_as_float((e + 127) << 23) * scale;
  }
};

// (A function of its own: it stands in many places where little goes through it.)
__device__ __noinline__ u64 one_weight(float z, float M, float c_hi, float c_lo, float zlow, int n0, bool wide,
                                       double c) {
  Weights w;
  w.M = M;
  w.c_hi = c_hi;
  w.c_lo = c_lo;
  w.zlow = zlow;
  w.n0 = n0;
  int e[2];
  float t[2];
  if (wide) {
    const int2 a = wide_power(z, M, c);
    e[0] = a.x;
    t[0] = __int_as_float(a.y);
  } else
    w.power2(z, z, e, t);
  return w.is_large(e[0]) ? w.large(e[0], t[0]) : w.units(e[0], t[0]);
}

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

// (A NaN stays one: no comparison below lets it through, and fmaxf passes it over.)
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
  float4* const zs;  // the CTA's groups in shared memory, or nullptr
  const TruncParams& p;
  const int tid, lane, warp, rank, C;
  int par = 0;
  const char* base;  // the row
  bool vec;
  int V, g0, gn;     // the CTA's groups of four ids: the first, and how many
  int i0, i1;        // the warp's, within the CTA's
  const float4* src; // where groups below full are to be had as they are
  int full;
  int iters, sub;    // rounds of the warp, of a piece
  Weights w;

  SPEC_DEVINL Row(Shared& s_, float4* zs_, const TruncParams& p_)
      : s(s_), zs(zs_), p(p_), tid(threadIdx.x), lane(threadIdx.x & 31), warp(threadIdx.x >> 5),
        rank(static_cast<int>(cluster_rank())), C(static_cast<int>(cluster_size())) {}

  // (of a group past the warp's: anything)
  SPEC_DEVINL float4 get(int i) const {
    float4 v;
    if (i < full)
      v = src[i];
    else
      v = fetch(i);
    return v;
  }
  SPEC_DEVINL float4 fetch(int i) const {
    float v[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    if (i < i1) load4<BF16>(base, 4 * (g0 + i), V, vec, v);
    return make_float4(v[0], v[1], v[2], v[3]);
  }
  // f(first id, four logits) over the CTA's groups (a warp's are contiguous), two loads ahead; after(round) by
  // whole warps
  template <class F, class G>
  SPEC_DEVINL void each(F&& f, G&& after) const {
    int i = i0 + lane;
    float4 a = get(i), b = get(i + 32);
    for (int j = 0; j < iters; ++j, i += 32) {
      const float4 v = a;
      a = b;
      b = get(i + 64);
      if (i < i1) f(4 * (g0 + i), v);
      after(j);
    }
  }
  template <class F>
  SPEC_DEVINL void each(F&& f) const {
    each(f, [](int) {});
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

  // Up to four values of every CTA (held by warp 0) to every CTA of the cluster.
  SPEC_DEVINL const u64 (*exchange(u64 a, u64 b = 0, u64 c = 0, u64 d = 0))[kMaxC] {
    par ^= 1;
    if (warp == 0 && lane < C) {
      st_remote(remote(&s.ex[par][0][rank], lane), a);
      st_remote(remote(&s.ex[par][1][rank], lane), b);
      st_remote(remote(&s.ex[par][2][rank], lane), c);
      st_remote(remote(&s.ex[par][3][rank], lane), d);
    }
    cluster_barrier();
    return s.ex[par];
  }
  // one of them, of each CTA, added up
  SPEC_DEVINL u64 total_of(const u64* v) const {
    u64 t = lane < C ? v[lane] : 0ull;
#pragma unroll
    for (int o = 1; o < kMaxC; o <<= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    return __shfl_sync(0xffffffffu, t, 0);
  }
  // the warps' values in v, added up (a whole warp)
  SPEC_DEVINL u64 warps_sum(const u64* v) const {
    u64 t = lane < kW ? v[lane] : 0ull;
#pragma unroll
    for (int o = 1; o < kW; o <<= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    return __shfl_sync(0xffffffffu, t, 0);
  }

  // the pieces' weights, added up (a whole warp)
  SPEC_DEVINL u64 pieces_sum() const {
    u64 t = 0;
#pragma unroll
    for (int i = 0; i < kW * kPieces; i += 32) t += s.seg[i + lane];
    return warp_sum64(t);
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
  SPEC_DEVINL void list_add(float v, int id) {
    const unsigned at = atomicAdd(&s.n, 1u);
    if (at < kList) s.list[at] = entry(key_of(v == 0.f ? 0.f : v), id);  // (-0 as 0)
  }
  // larger first, the lower id of equal ones
  SPEC_DEVINL static u64 entry(unsigned key, int id) { return (static_cast<u64>(key) << 32) | ~static_cast<unsigned>(id); }
  SPEC_DEVINL static float value_of(u64 x) { return key_value(static_cast<unsigned>(x >> 32)); }
  SPEC_DEVINL static int id_of(u64 x) { return static_cast<int>(~static_cast<unsigned>(x)); }

  // The cluster's lists (counts[r] entries of CTA r) to this CTA, with their weights (or 1 each); where its
  // own start.
  SPEC_DEVINL int pull(const u64* counts, int n, bool mass) {
    int own = 0;
    for (int r = 0; r < rank; ++r) own += static_cast<int>(counts[r]);
    for (int i = tid; i < n; i += kT) {
      int r = 0, at = i;
      while (at >= static_cast<int>(counts[r])) at -= static_cast<int>(counts[r++]);
      const u64 x = ld_remote64(remote(&s.list[at], r));
      s.l.x[i] = x;
      s.l.weight[i] = mass ? w.fixed(value_of(x)) : 1ull;
    }
    if (tid == 0) s.hi = 0;
    __syncthreads();
    return own;
  }
  // For each entry i of [from, from + some), by a few threads: then(i, the weights of those of the n for which
  // f(entry, another) holds, added up), by one of them.
  template <class F, class G>
  SPEC_DEVINL void over_list(int n, int from, int some, F&& f, G&& then) {
    int lg = 0;
    while ((kT >> (lg + 1)) >= some && lg < 5) ++lg;
    const int step = 1 << lg, part = tid & (step - 1);
    for (int i0 = 0; i0 < some; i0 += kT >> lg) {
      const int i = from + i0 + (tid >> lg);
      const bool mine = i < from + some;
      u64 sum = 0;
      if (mine) {
        const u64 x = s.l.x[i];
#pragma unroll 4
        for (int j = part; j < n; j += step) sum += f(x, s.l.x[j]) ? s.l.weight[j] : 0ull;
      }
      for (int o = 1; o < step; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (mine && part == 0) then(i, sum);
    }
  }
  // The key of the largest value of those entries whose weight and that of larger ones reach the target (0 if
  // none's does).
  SPEC_DEVINL unsigned reaches(int n, int from, int some, u64 target) {
    over_list(
        n, from, some, [](u64 x, u64 y) { return (y >> 32) >= (x >> 32); },
        [&](int i, u64 sum) {
          if (sum >= target) atomicMax(&s.hi, static_cast<unsigned>(s.l.x[i] >> 32));
        });
    __syncthreads();
    const unsigned key = s.hi;
    __syncthreads();  // (it is cleared for the next)
    return key;
  }
  // The largest of the threads' values, in every thread (set: 0 or 1 in turn).
  SPEC_DEVINL u64 block_max(u64 v, int set) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = max(v, static_cast<u64>(__shfl_xor_sync(0xffffffffu, v, o)));
    u64* const red = set ? s.seg : s.red;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    v = lane < kW ? red[lane] : 0ull;
#pragma unroll
    for (int o = 1; o < kW; o <<= 1) v = max(v, static_cast<u64>(__shfl_xor_sync(0xffffffffu, v, o)));
    return __shfl_sync(0xffffffffu, v, 0);
  }
  // A row whose n <= kFew candidates this CTA has pulled, with their weights: the threshold, the weight of what is
  // kept, and the draws.  Of each candidate: how many are larger, and the weight of the larger ones and of those
  // not smaller.  top-k keeps it if fewer than k are larger; top-p, if the larger ones' weight falls short of its
  // part of what top-k keeps, which is the most that ones not smaller than one of those weigh.
  SPEC_DEVINL u64 decide(int row, int n, int k, float top_p, float* theta) {
    int lg = 0;
    while ((kT >> (lg + 1)) >= n && lg < 5) ++lg;
    const int step = 1 << lg, part = tid & (step - 1), i = tid >> lg;
    const bool mine = i < n;
    u64 larger = 0, reached = 0;
    int rank_of = 0;
    const u64 x = mine ? s.l.x[i] : ~0ull;
    const unsigned key = static_cast<unsigned>(x >> 32);
    if (mine) {
#pragma unroll 4
      for (int j = part; j < n; j += step) {
        const unsigned other = static_cast<unsigned>(s.l.x[j] >> 32);
        const u64 y = s.l.weight[j];
        if (other > key) {
          larger += y;
          ++rank_of;
        }
        if (other >= key) reached += y;
      }
    }
    for (int o = 1; o < step; o <<= 1) {
      larger += __shfl_xor_sync(0xffffffffu, larger, o);
      reached += __shfl_xor_sync(0xffffffffu, reached, o);
      rank_of += __shfl_xor_sync(0xffffffffu, rank_of, o);
    }
    bool keep = mine && rank_of < k;
    u64 total = block_max(keep ? reached : 0ull, 0);
    if (top_p < 1.f) {
      keep = keep && larger < part_of(total, top_p, true);
      total = block_max(keep ? reached : 0ull, 1);
    }
    if (keep && part == 0 && reached == total) atomicMax(&s.hi, ~key);  // (the smallest: some may weigh nothing)
    if (FILTER) {
      __syncthreads();
      *theta = key_value(~s.hi);
      return total;
    }
    if (mine && part == 0 && !keep) s.l.weight[i] = 0;
    if (tid < p.draws) s.l.targets[tid] = draw_target(row, tid, total);
    __syncthreads();
    *theta = key_value(~s.hi);
    u64 sum = 0;  // cumulative weight in the order of ids
    if (mine) {
#pragma unroll 4
      for (int j = part; j < n; j += step)
        sum += static_cast<unsigned>(s.l.x[j]) >= static_cast<unsigned>(x) ? s.l.weight[j] : 0ull;
    }
    for (int o = 1; o < step; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (keep && part == 0)
      for (int d = 0; d < p.draws; ++d)
        if (s.l.targets[d] < sum && s.l.targets[d] >= sum - s.l.weight[i])
          p.tokens[static_cast<long long>(row) * p.draws + d] = id_of(x);
    return total;
  }
  // The same over the cluster's lists, each CTA its own entries.
  SPEC_DEVINL bool threshold(const u64* counts, int n, bool mass, u64 target, float* theta) {
    const int some = static_cast<int>(counts[rank]), own = pull(counts, n, mass);
    const unsigned key = some ? reaches(n, own, some, target) : 0u;
    const u64(*ex)[kMaxC] = exchange(key, 0);
    unsigned top = 0;
    for (int r = 0; r < C; ++r) top = max(top, static_cast<unsigned>(ex[0][r]));
    if (top) *theta = key_value(top);
    return top != 0;
  }

  // What every CTA has in hist to all of them, and there the bin that the target lies in (-1: beyond them
  // all), and the target less what lies above it.
  SPEC_DEVINL int find_bin(u64 target, u64* left) {
    __syncthreads();
    static_assert(kT == 8 * kBins && kMaxC == 8, "eight threads a bin");
    const int b = tid >> 3, part = tid & 7;
    const uint4 lo = *reinterpret_cast<const uint4*>(&s.h.hist[0][b][4 * part]);
    const uint4 hi = *reinterpret_cast<const uint4*>(&s.h.hist[1][b][4 * part]);
    u64 x = static_cast<u64>(lo.x) + lo.y + lo.z + lo.w + ((static_cast<u64>(hi.x) + hi.y + hi.z + hi.w) << kLimb);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (part < C) st_remote(remote(&s.h.bins[rank][b], part), x);
    cluster_barrier();
    x = part < C ? s.h.bins[part][b] : 0ull;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (part == 0) s.sums[b] = x;
    cluster_barrier();  // (every CTA has read its bins before they are written again)
    const u64 m0 = s.sums[2 * lane], m1 = s.sums[2 * lane + 1];
    const u64 incl = warp_incl64(m0 + m1, lane), before = incl - m0 - m1;
    const unsigned past = __ballot_sync(0xffffffffu, incl >= target);
    if (!past) return -1;
    const int at = __ffs(past) - 1;
    const bool second = before + m0 < target;
    *left = target - __shfl_sync(0xffffffffu, second ? before + m0 : before, at);
    return __shfl_sync(0xffffffffu, 2 * lane + second, at);
  }

  SPEC_DEVINL void hist_clear() {
    __syncthreads();
    for (int i = tid; i < static_cast<int>(sizeof(s.h.hist) / 16); i += kT)
      reinterpret_cast<uint4*>(s.h.hist)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
  }
  // What a lane adds to a counter fits it: at most 8192 ids, of up to 2^35.5 in weight.
  static constexpr int kLimb = 19;
  SPEC_DEVINL void hist_add(int b, u64 x) {
    atomicAdd(&s.h.hist[0][b][lane], static_cast<unsigned>(x) & ((1u << kLimb) - 1u));
    atomicAdd(&s.h.hist[1][b][lane], static_cast<unsigned>(x >> kLimb));
  }

  SPEC_DEVINL static u64 two(float a, float b) {
    return static_cast<u64>(__float_as_uint(a)) | static_cast<u64>(__float_as_uint(b)) << 32;
  }
  SPEC_DEVINL static float low_of(u64 x) { return __uint_as_float(static_cast<unsigned>(x)); }
  SPEC_DEVINL static float high_of(u64 x) { return __uint_as_float(static_cast<unsigned>(x >> 32)); }
  // Fine bins: distance from M, linear (weights: 146 to a halving; numbers: an eighth of them to the span), by
  // the bits of a sum rounded to a whole number, or, where that is too large, by a difference.
  struct Fine {
    float M, per, far, shift;  // (shift: of a bin's middle, in bins)
    int b0;
    bool by_sum;
    SPEC_DEVINL int operator()(float v) const {
      if (by_sum) return b0 - __float_as_int(fmaf(fmaxf(v, far), per, kRound));
      return min(static_cast<int>((M - v) * per), kFar);
    }
    // (MASS) the weight in a bin's middle, in 2^-36 of the largest
    SPEC_DEVINL float middle(int b) const {
      float w;  // (2^7 to 2^36: no number that a plain exp2f would have to look out for)
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(36.f - (static_cast<float>(b) + shift) * (1.f / kPerBit)));
      return w;
    }
    // The values between which bin b lies, but for rounding (slack: in bins).
    SPEC_DEVINL float upper(int b, float slack) const {
      if (b <= 0) return INFINITY;
      if (!by_sum) return M - __fdividef(static_cast<float>(b) - slack, per);
      return __fdividef((__int_as_float(b0) - kRound) - static_cast<float>(b) + (0.5f + slack), per);
    }
    SPEC_DEVINL float lower(int b, float slack) const {
      if (b >= kFar - 1) return -INFINITY;
      if (!by_sum) return M - __fdividef(static_cast<float>(b) + 1.f + slack, per);
      return __fdividef((__int_as_float(b0) - kRound) - static_cast<float>(b) - (0.5f + slack), per);
    }
  };
  template <bool MASS>
  SPEC_DEVINL Fine fine_bins(float span) const {
    Fine f;
    f.M = w.M;
    f.per = MASS ? fminf(w.c_hi, 1e28f) * kPerBit : (span > 0.f && span < 1e30f ? fminf((kFine / 8) / span, 1e30f) : 0.f);
    f.by_sum = !(MASS && w.wide) && fabsf(w.M) * f.per < 3.2e6f && f.per > 1e-25f;
    f.far = f.by_sum ? w.M - __fdividef(static_cast<float>(kFar), f.per) : 0.f;
    f.b0 = __float_as_int(fmaf(w.M, f.per, kRound));
    f.shift = f.by_sum ? fmaf(w.M, f.per, kRound - __int_as_float(f.b0)) : 0.5f;
    return f;
  }

  // All CTAs' ids in this thread's bins (every load on its way before the first is waited for).
  template <int CTAS>
  SPEC_DEVINL void counts_of(int b0, unsigned (&count)[kMaxC]) const {
    constexpr int kPer = kMaxC / CTAS;
    unsigned x[CTAS][kPer];
#pragma unroll
    for (int r = 0; r < CTAS; ++r) ld_remote_n<kPer>(remote(&s.fine[b0], r), x[r]);
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      count[q] = 0;
#pragma unroll
      for (int r = 0; r < CTAS; ++r) count[q] += x[r][q];
    }
  }

  // The fine bins [from, to] in which top_p of the weight of {z >= lower} ends, by the ids' numbers in them; or
  // (MASS false) the one of the k-th.  false: fewer than k.  A bin of n ids weighs n times its middle's weight
  // m, but for an error of about 0.0014 m sqrt(n) (ids lie anywhere in it); for the heavy ids, where a single one's
  // error counts, the difference is added up.  The end is looked for within three times the root of the errors'
  // squares, what may lie past the bins, and 2^-15 of the whole.
  template <bool MASS>
  SPEC_DEVINL bool count_bins(const Fine& fine, float lower, float top_p, int k, int* from, int* to) {
    constexpr int kHeavy = static_cast<int>(kHeavyBits * kPerBit);
    __syncthreads();  // (the bins lie where the last list was)
    for (int i = tid; i < kFine / 4; i += kT) reinterpret_cast<uint4*>(s.fine)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    const float heavy = w.M - __fdividef(kHeavyBits + 0.1f, w.c_hi);
    float extra = 0.f;  // heavy ids' weights less their bins' (in 2^-36)
    each([&](int, const float4& z) {
      const int b[4] = {fine(z.x), fine(z.y), fine(z.z), fine(z.w)};
      const float v[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (v[q] >= lower) atomicAdd(&s.fine[b[q]], 1u);
      if (MASS && fine.by_sum && fmaxf(fmaxf(z.x, z.y), fmaxf(z.z, z.w)) >= heavy) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (b[q] < kHeavy && v[q] >= lower)
            extra = fmaf(fine.middle(b[q]), fmaf(v[q] - w.M, fine.per, static_cast<float>(b[q]) + fine.shift), extra);
      }
    });
    cluster_barrier();
    // each CTA its part of the bins, a thread one to eight in a row
    static_assert(kFine == kMaxC * kT, "");
    const int per = kMaxC / C, b0 = (rank * kT + tid) * per;
    unsigned count[kMaxC];
    if (per == 1)
      counts_of<8>(b0, count);
    else if (per == 2)
      counts_of<4>(b0, count);
    else if (per == 4)
      counts_of<2>(b0, count);
    else
      counts_of<1>(b0, count);
    u64 v[kMaxC], mine = 0, first_bins = 0;  // (the latter: of heavy ids)
    float err = 0.f, err_heavy = 0.f;
#pragma unroll
    for (int q = 0; q < kMaxC; ++q) {
      v[q] = 0;
      if (q >= per) continue;
      const unsigned n = count[q];
      v[q] = n;
      if (MASS) {
        const float m = fine.middle(b0 + q), x = static_cast<float>(n) * m;
        if (b0 + q >= kFar - 1) {  // (anything further from M is counted there)
          v[q] = 0;
          err += x * x * 57000.f;  // (their whole weight, squared, over (3 x 0.0014)^2)
        } else {
          v[q] = n * static_cast<u64>(m);
          (b0 + q < kHeavy ? err_heavy : err) += x * m;
          if (b0 + q < kHeavy) first_bins += v[q];
        }
      }
      mine += v[q];
    }
    const u64 incl = warp_incl64(mine, lane);
    if (lane == 31) s.red[warp] = incl;
    if (MASS) {
      extra *= 0.693147181f / kPerBit;  // (2^d - 1 of less than half a bin)
      err = warp_sum(err);
      err_heavy = warp_sum(err_heavy);
      extra = warp_sum(extra);
      first_bins = warp_sum64(first_bins);
      if (lane == 0) {
        s.seg[warp] = first_bins;
        s.seg[kW + warp] = two(err, err_heavy);
        s.seg[2 * kW + warp] = two(extra, 0.f);
      }
    }
    __syncthreads();
    if (MASS && warp == 0) {
      first_bins = warps_sum(s.seg);
      const u64 e = lane < kW ? s.seg[kW + lane] : 0ull;
      err = warp_sum(low_of(e));
      err_heavy = warp_sum(high_of(e));
      extra = warp_sum(lane < kW ? low_of(s.seg[2 * kW + lane]) : 0.f);
    }
    const u64(*ex)[kMaxC] =
        exchange(warp == 0 ? warps_sum(s.red) : 0ull, two(err, err_heavy), two(extra, 0.f), first_bins);
    u64 excl = incl - mine;
    for (int i = 0; i < warp; ++i) excl += s.red[i];
    for (int r = 0; r < rank; ++r) excl += ex[0][r];
    const u64 all = total_of(ex[0]);
    u64 first = static_cast<u64>(k), last = first;
    if (MASS) {
      err = err_heavy = extra = 0.f;
      for (int r = 0; r < C; ++r) {
        err += low_of(ex[1][r]);
        err_heavy += high_of(ex[1][r]);
        extra += low_of(ex[2][r]);
      }
      const long long more = static_cast<long long>(extra);
      const u64 t = part_of(all + more, top_p, true) - more, off = (all >> 15) + static_cast<u64>(0.0042f * sqrtf(err));
      first = t > off ? t - off : 1ull;
      last = min(t + off, all);
      // among the heavy ids (which are few), or where those were not weighed
      if (!fine.by_sum || static_cast<long long>(t) <= 0 || first <= total_of(ex[3])) {
        const u64 t1 = part_of(all, top_p, true), off1 = off + static_cast<u64>(0.0042f * sqrtf(err + err_heavy));
        first = t1 > off1 ? t1 - off1 : 1ull;
        last = min(t1 + off1, all);
      }
    }
    if (all < first) return false;
    par ^= 1;
    int first_bin = -1, last_bin = -1;
#pragma unroll
    for (int q = 0; q < kMaxC; ++q) {
      if (q >= per) continue;
      const u64 next = excl + v[q];
      if (excl < first && first <= next) first_bin = b0 + q;
      if (excl < last && last <= next) last_bin = b0 + q;
      excl = next;
    }
    if (first_bin >= 0)
      for (int r = 0; r < C; ++r) st_remote(remote(&s.ex[par][0][0], r), first_bin);
    if (last_bin >= 0)
      for (int r = 0; r < C; ++r) st_remote(remote(&s.ex[par][1][0], r), last_bin);
    cluster_barrier();
    *from = static_cast<int>(s.ex[par][0][0]);
    *to = static_cast<int>(s.ex[par][1][0]);
    return true;
  }

  // The largest value v where the weight (MASS; else number) of the logits from v on, of those in [lower,
  // upper), reaches the target: false if it is less.
  template <bool MASS>
  SPEC_DEVINL bool refine(float lower, float upper, u64 target, float* theta) {
    // keys that are left (0 and -0 are equal, and so on the same side of a bound)
    auto end = [](float v) { return key_of(v == 0.f ? -0.f : v); };
    unsigned klo = max(end(lower), end(-INFINITY) + 1u), khi = upper == INFINITY ? end(INFINITY) : end(upper) - 1u;
    // f(id, z, key) for the logits there
    auto each_here = [&](auto&& fn) {
      each1([&](int x, float v) {
        const unsigned kv = key_of(v);
        if (kv - klo <= khi - klo) fn(x, v, kv);
      });
    };
    cluster_barrier();  // the bins of other CTAs, written to below, lie where their lists were
    for (;;) {
      list_clear();
      unsigned lo = 0xFFFFFFFFu, hi = 0;
      each_here([&](int x, float v, unsigned kv) {
        list_add(v, x);
        lo = min(lo, kv);
        hi = max(hi, kv);
      });
      lo = __reduce_min_sync(0xffffffffu, lo);
      hi = __reduce_max_sync(0xffffffffu, hi);
      if (lane == 0) {
        atomicMin(&s.lo, lo);
        atomicMax(&s.hi, hi);
      }
      __syncthreads();
      const u64(*ex)[kMaxC] = exchange((static_cast<u64>(s.lo) << 32) | s.hi, s.n);
      const int n = static_cast<int>(total_of(ex[1]));
      klo = 0xFFFFFFFFu;
      khi = 0;
      for (int r = 0; r < C; ++r) {
        klo = min(klo, static_cast<unsigned>(ex[0][r] >> 32));
        khi = max(khi, static_cast<unsigned>(ex[0][r]));
      }
      if (n == 0) return false;
      if (klo == khi) {  // one value
        const float v = key_value(klo);
        if (n * (MASS ? w.fixed(v) : 1ull) < target) return false;
        *theta = v;
        return true;
      }
      if (n <= kList) return threshold(ex[1], n, MASS, target, theta);
      // too many: bins of keys between the smallest and the largest
      int shift = 0;
      while (((khi - klo) >> shift) >= kBins) ++shift;
      hist_clear();
      each_here([&](int, float v, unsigned kv) { hist_add(static_cast<int>((khi - kv) >> shift), MASS ? w.fixed(v) : 1ull); });
      const int b = find_bin(target, &target);
      if (b < 0) return false;
      khi -= static_cast<unsigned>(b) << shift;
      klo = max(klo, khi - min(khi, (1u << shift) - 1u));
    }
  }

  // top_p's threshold of {z >= lower}.  true: seg holds what it keeps of the pieces' weights.
  SPEC_DEVINL bool nucleus(float lower, float top_p, float* theta) {
    const Fine fine = fine_bins<true>(0.f);
    int from = 0, to = kFine;
    count_bins<true>(fine, lower, top_p, 0, &from, &to);
    // (what follows holds for any two values: should the threshold not lie between them, it is found by itself)
    const float high = fine.upper(from, 0.f), low = fmaxf(lower, fine.lower(to, 0.f));
    const float large = w.wide ? lower : w.M - __fdividef(kLarge + 1.f, w.c_hi);  // no large weight below
    const float least = fminf(low, large);
    const float none = w.wide ? -INFINITY : w.M - __fdividef(38.f, w.c_hi);  // no weight from here down
    list_clear();
    u64 above = 0, all = 0;
    const bool some = lower > -INFINITY || w.wide;  // (else a NaN's power is 0, as -inf's)
    int left = sub, piece = warp * kPieces;
    each(
        [&](int x, const float4& z) {
          const float most = fmaxf(fmaxf(z.x, z.y), fmaxf(z.z, z.w));
          if (!(most >= none)) return;
          int e[4];
          float t[4];
          w.power4(z, e, t);
          const float v[4] = {z.x, z.y, z.z, z.w};
          unsigned u[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) u[q] = w.units(e[q], t[q]);
          if (some) {
#pragma unroll
            for (int q = 0; q < 4; ++q) u[q] = v[q] >= lower ? u[q] : 0u;
          }
          all += u[0] + u[1];  // (each below 2^31)
          all += u[2] + u[3];
          if (most < least) return;
          bool between = false;
          unsigned o[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            o[q] = v[q] >= high ? u[q] : 0u;
            between = between || (v[q] < high && v[q] >= low);
          }
          above += o[0] + o[1];
          above += o[2] + o[3];
          if (between) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (v[q] < high && v[q] >= low && v[q] > -INFINITY) list_add(v[q], x + q);
          }
          if (most < large) return;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (w.is_large(e[q]) && v[q] >= lower) {
              const u64 x1 = w.large(e[q], t[q]);
              all += x1;
              if (v[q] >= high) above += x1;
            }
        },
        [&](int j) {
          if (--left == 0 || j == iters - 1) {
            above = warp_sum64(above);
            if (lane == 0) s.seg[piece] = above;
            ++piece;
            left = sub;
            above = 0;
          }
        });
    for (; piece < (warp + 1) * kPieces; ++piece)
      if (lane == 0) s.seg[piece] = 0;
    all = warp_sum64(all);
    if (lane == 0) s.red[warp] = all;
    __syncthreads();
    if (warp == 0) {
      above = pieces_sum();
      all = warps_sum(s.red);
    }
    const u64(*ex)[kMaxC] = exchange(s.n, above, all);
    const int n = static_cast<int>(total_of(ex[0]));
    above = total_of(ex[1]);
    const u64 target = part_of(total_of(ex[2]), top_p, true);
    if (target > above) {
      if (n <= kList) {
        if (threshold(ex[0], n, true, target - above, theta)) {
          if constexpr (!FILTER) {
            for (int i = tid; i < static_cast<int>(s.n); i += kT) {  // what this CTA's list keeps, to its pieces' weights
              const u64 x = s.list[i];
              const float v = value_of(x);
              if (v >= *theta) {
                const int g = (id_of(x) >> 2) - g0, at = g / (32 * iters);
                atomicAdd(&s.seg[at * kPieces + (g - at * 32 * iters) / (32 * sub)], w.fixed(v));
              }
            }
            __syncthreads();
          }
          return true;
        }
      } else if (refine<true>(low, high, target - above, theta)) {
        return false;
      }
    }
    refine<true>(lower, INFINITY, target, theta);
    return false;
  }

  // The k-th largest of {lower <= z}, -inf if there are fewer.
  SPEC_DEVINL float kth(float lower, float span, int k) {
    const Fine fine = fine_bins<false>(span);
    int from, to;
    float theta = -INFINITY;
    if (!count_bins<false>(fine, lower, 0.f, k, &from, &to)) return theta;
    const float high = fine.upper(from, 0.3f), low = fmaxf(lower, fine.lower(to, 0.3f));
    list_clear();
    unsigned over = 0;
    each([&](int x, const float4& z) {
      if (fmaxf(fmaxf(z.x, z.y), fmaxf(z.z, z.w)) < low) return;
      const float v[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (v[q] >= high)
          ++over;
        else if (v[q] >= low && v[q] > -INFINITY)
          list_add(v[q], x + q);
      }
    });
    over = __reduce_add_sync(0xffffffffu, over);
    if (lane == 0) s.red[warp] = over;
    __syncthreads();
    const u64(*ex)[kMaxC] = exchange(s.n, warp == 0 ? warps_sum(s.red) : 0ull);
    const int n = static_cast<int>(total_of(ex[0]));
    const u64 above = total_of(ex[1]), target = static_cast<u64>(k);
    if (low == lower && above + n < target) return theta;  // fewer than k
    if (target > above) {
      if (n <= kList ? threshold(ex[0], n, false, target - above, &theta) : refine<false>(low, high, target - above, &theta))
        return theta;
    }
    refine<false>(lower, INFINITY, target, &theta);
    return theta;
  }

  // Every output of a row but its draws: value(first id, four logits, out).
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
      float v[4] = {z.x, z.y, z.z, z.w};
      value(x, z, v);
      store4 < BF16 && FILTER > (base, x, V, vec, v);
    });
  }
  SPEC_DEVINL void write_kept(int row, float theta, u64 total) {
    if (FILTER) {
      write_row(row, [&](int, const float4&, float (&v)[4]) {
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = v[q] >= theta ? v[q] : -INFINITY;
      });
    } else if (p.probs) {
      if (tid == 0) s.sum_inv = static_cast<float>(static_cast<double>(1ull << 35) / static_cast<double>(total));
      __syncthreads();
      const float inv = s.sum_inv;
      write_row(row, [&](int, const float4& z, float (&v)[4]) {
        if (fmaxf(fmaxf(z.x, z.y), fmaxf(z.z, z.w)) < theta) {
          v[0] = v[1] = v[2] = v[3] = 0.f;
          return;
        }
        int e[4];
        float t[4];
        w.power4(z, e, t);
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = v[q] >= theta ? Weights::real(e[q], t[q], inv) : 0.f;
      });
    }
  }
  // one id alone (T = 0), or, id -1, a row with nothing to draw
  SPEC_DEVINL void write_single(int row, int only) {
    if constexpr (!FILTER) {
      if (rank == 0)
        for (int d = tid; d < p.draws; d += kT) p.tokens[static_cast<long long>(row) * p.draws + d] = only;
    }
    if (FILTER || p.probs)
      write_row(row, [&](int x, const float4&, float (&v)[4]) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (FILTER)
            v[q] = only < 0 || x + q == only ? fmaxf(v[q], -INFINITY) : -INFINITY;
          else
            v[q] = x + q == only ? 1.f : 0.f;
        }
      });
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
    gn = max(0, min(per, groups - g0));
    iters = (gn + kT - 1) / kT;
    sub = max((iters + kPieces - 1) / kPieces, 4);
    i0 = min(warp * iters * 32, gn);
    i1 = min(i0 + iters * 32, gn);
    base = static_cast<const char*>(p.z) + static_cast<long long>(row) * p.ld * (BF16 ? 2 : 4);
    vec = (reinterpret_cast<uintptr_t>(base) & (BF16 ? 7 : 15)) == 0;
    src = zs ? zs : reinterpret_cast<const float4*>(base) + g0;
    full = zs ? i1 : !BF16 && vec ? min(i1, (V >> 2) - g0) : 0;
    const RowSet rs = row_set(p, row);
    float top = -INFINITY;
    constexpr int kAhead = 8;  // loads on their way at once
    for (int i = i0 + lane; i < i1; i += 32 * kAhead) {
      float4 v[kAhead];
#pragma unroll
      for (int q = 0; q < kAhead; ++q) v[q] = fetch(i + 32 * q);
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        if (zs && i + 32 * q < i1) zs[i + 32 * q] = v[q];
        top = fmaxf(top, fmaxf(fmaxf(v[q].x, v[q].y), fmaxf(v[q].z, v[q].w)));
      }
    }
    const bool bad = !(rs.T >= 0.f) || rs.T > 3.4028234e38f || rs.k < 0 || !(rs.top_p > 0.f && rs.top_p <= 1.f) ||
                     !(rs.min_p >= 0.f && rs.min_p <= 1.f);
    list_clear();
    // the maxima of parts of warps (of 4 C lanes each: 128 of them) to every CTA
    unsigned kt = key_of(top);
    const int group = 4 * C, in_warp = 32 / group;
    for (int o = 1; o < group; o <<= 1) kt = max(kt, __shfl_xor_sync(0xffffffffu, kt, o));
    cluster_all_started();
    if (lane % group < C) st_remote32(remote(&s.wmax[(rank * kW + warp) * in_warp + lane / group], lane % group), kt);
    cluster_barrier();
    constexpr int nw = kMaxC * kW;
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
    if (rs.T < 1.17549435e-38f) {  // (or what would be a subnormal) the lowest id of the largest
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
    // (c below 2^96: the paired steps take a subnormal z as 0, which moves a power by less than 2^-30)
    w.wide = !(far < 30000.f) || !(c_hi < 7.9e28f) || !(c_hi > 1e-25f);
    w.zlow = w.wide ? 0.f : M - __fdividef(150.f, c_hi);
    w.n0 = __float_as_int(fmaf(M, c_hi, kRound));
    const bool top_k = rs.k > 0 && rs.k < V, top_p = rs.top_p < 1.f, few_k = top_k && rs.k <= nw;
    float lower = -INFINITY;
    if (rs.min_p > 0.f || w.wide || few_k || M == INFINITY) {
      if (tid == kT - 1) {
        if (w.wide) s.c = 1.4426950408889634074 / static_cast<double>(rs.T);
        s.theta_m = M == INFINITY ? INFINITY
                    : rs.min_p > 0.f
                        ? __double2float_ru(static_cast<double>(M) + static_cast<double>(rs.T) * log(static_cast<double>(rs.min_p)))
                        : -INFINITY;
      }
      if (tid == 0) s.bound = -INFINITY;
      __syncthreads();
      // the k-th largest of those maxima: that many logits at least reach it
      if (few_k) {
        constexpr int kPer = kT / nw;  // threads a value
        const int i = tid / kPer;
        const unsigned mine = s.wmax[i];
        int c = 0;
#pragma unroll 8
        for (int j = tid % kPer; j < nw; j += kPer) {
          const unsigned y = s.wmax[j];
          c += y > mine || (y == mine && j < i) ? 1 : 0;
        }
#pragma unroll
        for (int o = 1; o < kPer; o <<= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
        if (c == rs.k - 1) s.bound = key_value(mine);
        __syncthreads();
      }
      w.c = s.c;
      lower = fmaxf(s.theta_m, s.bound);
    }
    const u64(*ex)[kMaxC];
    int n = kFew + 1;
    if ((lower > -INFINITY || V <= kFew) && !(FILTER && !top_k && !top_p)) {
      each([&](int x, const float4& v) {
        if (fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)) < lower) return;
        if (*const_cast<volatile unsigned*>(&s.n) > kFew) return;  // too many already
        if (v.x >= lower && v.x > -INFINITY) list_add(v.x, x);
        if (v.y >= lower && v.y > -INFINITY) list_add(v.y, x + 1);
        if (v.z >= lower && v.z > -INFINITY) list_add(v.z, x + 2);
        if (v.w >= lower && v.w > -INFINITY) list_add(v.w, x + 3);
      });
      __syncthreads();
      ex = exchange(s.n, 0);
      n = static_cast<int>(total_of(ex[0]));
    }
    float theta = lower;
    u64 total = 0;
    if (n <= kFew) {  // few: one CTA decides
      if (rank == 0) pull(ex[0], n, true);
      const bool alone = !FILTER && !p.probs;
      if (alone) cluster_barrier();  // no CTA leaves before its list is read
      if (rank == 0) total = decide(row, n, top_k ? rs.k : kT, rs.top_p, &theta);
      if (alone) return;
      ex = exchange(key_of(theta), total);
      write_kept(row, key_value(static_cast<unsigned>(ex[0][0])), ex[1][0]);
      return;
    }
    if (top_k) theta = fmaxf(theta, kth(lower, M - least, rs.k));
    bool weighed = false;
    if (top_p) {
      float v = theta;
      weighed = nucleus(theta, rs.top_p, &v);
      theta = fmaxf(theta, v);
    }
    if (FILTER) {
      write_kept(row, theta, 0);
      if (top_k || top_p) cluster_barrier();  // no CTA leaves before its list is read
      return;
    }
    // the pieces' weights, and the cluster's
    if (!weighed) {
      u64 sum = 0;
      int left = sub, piece = warp * kPieces;
      each(
          [&](int, const float4& v) {
            if (fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)) < theta) return;
            u64 x[4];
            w.fixed4(v, x);
            sum += (v.x >= theta ? x[0] : 0) + (v.y >= theta ? x[1] : 0) + (v.z >= theta ? x[2] : 0) +
                   (v.w >= theta ? x[3] : 0);
          },
          [&](int j) {
            if (--left == 0 || j == iters - 1) {
              sum = warp_sum64(sum);
              if (lane == 0) s.seg[piece] = sum;
              ++piece;
              left = sub;
              sum = 0;
            }
          });
      for (; piece < (warp + 1) * kPieces; ++piece)
        if (lane == 0) s.seg[piece] = 0;
      __syncthreads();
    }
    const u64 sum = pieces_sum();
    ex = exchange(sum);
    u64 before = 0;
    for (int r = 0; r < rank; ++r) before += ex[0][r];
    total = total_of(ex[0]);
    for (int d = warp; d < p.draws; d += kW) {
      u64 x = draw_target(row, d, total);
      if (x < before || x >= before + sum) continue;
      x -= before;
      // the piece, then 128 ids, the lane and the id whose cumulative weight passes x
      int piece = 0;
      for (; piece < kW * kPieces; piece += 32) {
        const u64 c = s.seg[piece + lane], incl = warp_incl64(c, lane);
        const unsigned past = __ballot_sync(0xffffffffu, incl > x);
        if (past) {
          const int at = __ffs(past) - 1;
          x -= __shfl_sync(0xffffffffu, incl - c, at);
          piece += at;
          break;
        }
        x -= __shfl_sync(0xffffffffu, incl, 31);
      }
      const int j0 = piece / kPieces * 32 * iters + piece % kPieces * 32 * sub,
                j1 = min(min(j0 + 32 * sub, (piece / kPieces + 1) * 32 * iters), gn);
      for (int j = j0; j < j1; j += 32) {
        float v[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if (j + lane < j1) load4<BF16>(base, 4 * (g0 + j + lane), V, vec, v);
        u64 f[4];
        w.fixed4(make_float4(v[0], v[1], v[2], v[3]), f);
        const u64 f0 = v[0] >= theta ? f[0] : 0, f1 = v[1] >= theta ? f[1] : 0, f2 = v[2] >= theta ? f[2] : 0,
                  f3 = v[3] >= theta ? f[3] : 0;
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

// What bounds it: with many rows instruction issue (320 rows of 128256, top-p alone: 143 us, 164 MB read once
// from memory; 97 million warp instructions, 65% of the issue slots of busy cycles; filter of as many rows with
// settings of their own 106 us for 328 MB, 51%); with few, the chain of cluster barriers between phases (one row,
// top-k 50 and top-p 0.95: 9.6 us).  64 registers, so that two CTAs fit an SM; three of 40 spilled and gained
// nothing, and logits kept in registers spill too (three times the time of shared memory).
template <bool BF16, bool FILTER>
__global__ void __launch_bounds__(kT, 2) trunc_kernel(const TruncParams p) {
  extern __shared__ __align__(16) char smem[];
  cluster_started();
  grid_dep_wait();
  grid_dep_launch();
  Row<BF16, FILTER> r(*reinterpret_cast<Shared*>(smem),
                      p.resident ? reinterpret_cast<float4*>(smem + sizeof(Shared)) : nullptr, p);
  r.run(static_cast<int>(blockIdx.x / static_cast<unsigned>(r.C)));
}

static_assert(sizeof(Shared) % 16 == 0, "");
constexpr int kResident = 4096;  // groups of a CTA that stay in shared memory, with room for two CTAs on an SM

template <bool BF16, bool FILTER>
cudaError_t launch(const TruncParams& p, cudaLaunchConfig_t& cfg) {
  // the most a CTA takes, asked for once per device
  static PerDevice<cudaError_t> set;
  cudaError_t e = cudaSuccess;
  if (!set.get(
          [] {
            return cudaFuncSetAttribute(trunc_kernel<BF16, FILTER>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        static_cast<int>(sizeof(Shared) + (kResident + 1) * sizeof(float4)));
          },
          &e))
    return cudaErrorInvalidDevice;
  if (e != cudaSuccess) return e;
  return cudaLaunchKernelEx(&cfg, trunc_kernel<BF16, FILTER>, p);
}

}  // namespace

cudaError_t launch_trunc(TruncParams p, int sms, cudaStream_t stream) {
  const int groups = (p.V + 3) / 4;
  // As many CTAs as keep the row in shared memory, two to an SM, or, where SMs are left over, one for
  // every 512 groups: a row alone takes the less time the more share it.  Of so many rows that their CTAs
  // take turns, fewer: what a cluster's CTAs wait for one another costs more then than reading the row
  // again from the caches, and the more so the longer a row's chain of passes (a filter's is shorter).
  // fp32 rows of 128256, us with eight / four / two CTAs a row (bf16 rows go by the same rule, as they are
  // kept as fp32: 320 of them 183, 184 and 156 us for the three lines below, with two, two and four CTAs):
  //                            38 rows           64                152               320
  //   draws, top-p alone       43 / 38 / 43      56 / 43 / 50      115 / 85 / 68     232 / 168 / 144
  //   draws, mixed, probs      31 / 38 / 52      43 / 40 / 53      91 / 83 / 85      163 / 129 / 136
  //   filter, mixed            24 / 32 / 46      30 / 34 / 46      69 / 64 / 71      125 / 104 / 119
  int C = 1;
  while (C < kMaxC && (groups > C * kResident || (groups > C * 512 && p.rows * C <= sms))) C *= 2;
  if (C == 8 && p.rows * 8 > (p.out ? 4 : 2) * sms) C = 4;
  if (C == 4 && p.rows * 4 > 3 * sms && !p.out) C = 2;
  const int per = (groups + C - 1) / C;
  p.resident = per <= kResident;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.rows) * C);
  cfg.blockDim = dim3(kT);
  cfg.dynamicSmemBytes = sizeof(Shared) + (p.resident ? (per + 1) * sizeof(float4) : 0);
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
