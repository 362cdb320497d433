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
// decides.  Else the ids are counted in 4096 bins of the distance from M: a bin's
// weight is its number times the weight at its middle to within 0.32%, so the bins
// where the nucleus ends are known but for a few; one pass over the weights then
// gives their total, what lies above those bins, and the few ids in them, among
// which the threshold is found.  (Should it lie elsewhere, or the ids be too
// many, histograms of the weights themselves part them, bin by bin.)
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
constexpr int kList = kT;
constexpr float kPerBit = kFar / 37.4f;  // fine bins to a halving of the weight: weights end before the bins
constexpr u64 kMassMask = (1ull << 54) - 1;
constexpr unsigned kManyIds = 1023;   // counts end there
constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds |x| < 2^22 to an integer

struct Shared {
  union {
    unsigned hist[2][kBins][32];  // a column a lane: no two lanes of a warp meet in a bank
    unsigned fine[kFine];
    struct {
      u64 x[kList];      // the cluster's list
      u64 weight[kList];
      u64 targets[kTruncMaxDraws];
    } l;
  };
  u64 bins[2][kMaxC][kBins];  // every CTA's bins: weight, and in the upper ten bits the number of ids; two sets in turn
  u64 sums[kBins];
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
SPEC_DEVINL uint32_t ld_remote32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
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
SPEC_DEVINL u64 add2(u64 a, u64 b) {
  u64 r;
  asm("add.rn.ftz.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
SPEC_DEVINL u64 neg2(u64 a) { return a ^ 0x8000000080000000ull; }

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
// (Few values of such a row are near enough to M to have a weight.)
__device__ __noinline__ void wide_power(float z, float M, double c, int* e, float* t) {
  const double d = z == M ? 0.0 : (static_cast<double>(z) - static_cast<double>(M)) * c;
  const double n = d < -200.0 ? -200.0 : rint(d);
  *e = static_cast<int>(n);
  *t = d < -200.0 ? 0.f : parts(exp2m1_scaled(both(static_cast<float>(d - n)))).x;
}

struct Weights {
  float M, c_hi, c_lo, zlow;
  int n0;   // M's power, as the rounded sum's bits
  int off;  // 5 or 2: weights are in units of 2^-(30 + off) of about the largest
  bool wide;
  double c;

  // w = 2^e (1 + t 2^-31) of two; -e at least 149 where z is further than that below M
  SPEC_DEVINL void power2(float a, float b, int (&e)[2], float (&t)[2]) const {
    const u64 x = pair(fmaxf(a, zlow), fmaxf(b, zlow)), c2 = both(c_hi);
    const u64 p = mul2(x, c2);
    const u64 nb = add2(p, both(kRound));
    const u64 rest = fma2(x, both(c_lo), fma2(x, c2, neg2(p)));  // the product's rounding error, and c's
    const u64 g = add2(add2(p, add2(both(kRound), neg2(nb))), rest);
    const float2 n = parts(nb), f = parts(exp2m1_scaled(g));
    e[0] = __float_as_int(n.x) - n0;
    e[1] = __float_as_int(n.y) - n0;
    t[0] = f.x;
    t[1] = f.y;
  }
  SPEC_DEVINL void power4(const float4& z, int (&e)[4], float (&t)[4]) const {
    if (wide) {
      wide_power(z.x, M, c, e, t);
      wide_power(z.y, M, c, e + 1, t + 1);
      wide_power(z.z, M, c, e + 2, t + 2);
      wide_power(z.w, M, c, e + 3, t + 3);
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
  // 2^(30 + off) w, to the nearest, of weights below 2^-off (as most are: larger ones give 0 here, and
  // all of their weight in large)
  SPEC_DEVINL unsigned units(int e, float t) const {
    unsigned h;
    asm("shr.b32 %0, %1, %2;" : "=r"(h) : "r"(mantissa(t)), "r"(-off - e));  // (0 from 32 on, and for less than 0)
    return (h + 1u) >> 1;
  }
  SPEC_DEVINL bool is_large(int e) const { return e > -off; }
  SPEC_DEVINL u64 large(int e, float t) const { return static_cast<u64>(mantissa(t)) << (off + e - 1); }
  SPEC_DEVINL static unsigned mantissa(float t) { return 0x80000000u + static_cast<unsigned>(__float2int_rn(t)); }
  SPEC_DEVINL u64 fixed(float z) const {
    int e[4];
    float t[4];
    power4(make_float4(z, z, z, z), e, t);
    return is_large(e[0]) ? large(e[0], t[0]) : units(e[0], t[0]);
  }
  SPEC_DEVINL void fixed4(const float4& z, u64 (&x)[4]) const {
    int e[4];
    float t[4];
    power4(z, e, t);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = units(e[i], t[i]);
    if (max(max(e[0], e[1]), max(e[2], e[3])) > -off) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (is_large(e[i])) x[i] = large(e[i], t[i]);
    }
  }
  SPEC_DEVINL static float real(int e, float t, float scale) {
    return e < -125 ? 0.f : fmaf(t, 4.65661287e-10f, 1.f) * __int_as_float((e + 127) << 23) * scale;
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
    v[e] = fmaxf(v[e], -INFINITY);  // (NaN)
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
  int i0, i1, wg;  // this warp's groups, within the CTA's, and their number a warp
  int limb, cnt_at;  // bits of the histogram's low part, and above which it counts ids in the other
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
  SPEC_DEVINL void list_add(float v, int id) {
    const unsigned at = atomicAdd(&s.n, 1u);
    if (at < kList) s.list[at] = entry(key_of(v), id);
  }
  // larger first, the lower id of equal ones
  SPEC_DEVINL static u64 entry(unsigned key, int id) { return (static_cast<u64>(key) << 32) | ~static_cast<unsigned>(id); }
  SPEC_DEVINL static float value_of(u64 x) { return key_value(static_cast<unsigned>(x >> 32)); }
  SPEC_DEVINL static int id_of(u64 x) { return static_cast<int>(~static_cast<unsigned>(x)); }

  // The cluster's lists (counts[r] entries of CTA r) to this CTA, with their weights (or 1 each).
  SPEC_DEVINL void pull(const u64* counts, int n, bool mass) {
    if (tid < n) {
      int r = 0, at = tid;
      while (at >= static_cast<int>(counts[r])) at -= static_cast<int>(counts[r++]);
      const u64 x = ld_remote64(remote(&s.list[at], r));
      s.l.x[tid] = x;
      s.l.weight[tid] = mass ? w.fixed(value_of(x)) : 1ull;
    }
    if (tid == 0) s.hi = 0;
    __syncthreads();
  }
  // A few threads an entry: f(entry, another, its weight) of all, added up (in each of them).
  template <class F>
  SPEC_DEVINL void over_list(int n, int& i, bool& first, u64& sum, F&& f) {
    int lg = 0;
    while ((kT >> (lg + 1)) >= n && lg < 5) ++lg;
    const int step = 1 << lg, part = tid & (step - 1);
    i = tid >> lg;
    first = part == 0;
    sum = 0;
    if (i < n) {
      const u64 x = s.l.x[i];
#pragma unroll 4
      for (int j = part; j < n; j += step) sum += f(x, s.l.x[j]) ? s.l.weight[j] : 0ull;
    }
    for (int o = 1; o < step; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  // The largest value of the list whose weight and that of larger ones reach the target (false if none's does).
  SPEC_DEVINL bool reaches(int n, u64 target, float* v) {
    int i;
    bool first;
    u64 sum;
    over_list(n, i, first, sum, [](u64 x, u64 y) { return (y >> 32) >= (x >> 32); });
    if (i < n && first && sum >= target) atomicMax(&s.hi, static_cast<unsigned>(s.l.x[i] >> 32));
    __syncthreads();
    const unsigned key = s.hi;
    __syncthreads();  // (it is cleared for the next)
    if (key) *v = key_value(key);
    return key != 0;
  }

  // What every CTA has in hist to all of them, and there the bin that the target lies in: the bin, the
  // target less what lies above it, and the ids in it (at most kManyIds).
  struct Found {
    int bin;
    u64 target;
    int n;
  };
  template <bool MASS, class F>
  SPEC_DEVINL Found find_bin(F&& target_of) {
    par ^= 1;
    __syncthreads();
    static_assert(kT == 8 * kBins && kMaxC == 8, "eight threads a bin");
    const int b = tid >> 3, part = tid & 7;
    const uint4 lo = *reinterpret_cast<const uint4*>(&s.hist[0][b][4 * part]);
    u64 x = static_cast<u64>(lo.x) + lo.y + lo.z + lo.w;
    unsigned n = 0;
    if (MASS) {
      const uint4 hi = *reinterpret_cast<const uint4*>(&s.hist[1][b][4 * part]);
      const unsigned m = (1u << cnt_at) - 1u;
      x += static_cast<u64>((hi.x & m) + (hi.y & m) + (hi.z & m) + (hi.w & m)) << limb;
      n = (hi.x >> cnt_at) + (hi.y >> cnt_at) + (hi.z >> cnt_at) + (hi.w >> cnt_at);
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      x += __shfl_xor_sync(0xffffffffu, x, o);
      if (MASS) n += __shfl_xor_sync(0xffffffffu, n, o);
    }
    if (!MASS) n = static_cast<unsigned>(x);
    if (part < C) st_remote(remote(&s.bins[par][rank][b], part), x | static_cast<u64>(min(n, kManyIds)) << 54);
    cluster_barrier();
    x = part < C ? s.bins[par][part][b] : 0ull;
    n = static_cast<unsigned>(x >> 54);
    x &= kMassMask;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      x += __shfl_xor_sync(0xffffffffu, x, o);
      n += __shfl_xor_sync(0xffffffffu, n, o);
    }
    if (part == 0) s.sums[b] = x | static_cast<u64>(min(n, kManyIds)) << 54;
    __syncthreads();
    const u64 p0 = s.sums[2 * lane], p1 = s.sums[2 * lane + 1], m0 = p0 & kMassMask, m1 = p1 & kMassMask;
    const u64 incl = warp_incl64(m0 + m1, lane), before = incl - m0 - m1;
    const u64 target = target_of(__shfl_sync(0xffffffffu, incl, 31));
    const unsigned past = __ballot_sync(0xffffffffu, incl >= target);
    if (!past) return {-1, target, 0};
    const int at = __ffs(past) - 1;
    const bool second = before + m0 < target;
    Found f;
    f.bin = __shfl_sync(0xffffffffu, 2 * lane + second, at);
    f.target = target - __shfl_sync(0xffffffffu, second ? before + m0 : before, at);
    f.n = static_cast<int>(__shfl_sync(0xffffffffu, static_cast<unsigned>((second ? p1 : p0) >> 54), at));
    return f;
  }

  SPEC_DEVINL void hist_clear() {
    for (int i = tid; i < static_cast<int>(sizeof(s.hist) / 16); i += kT)
      reinterpret_cast<uint4*>(s.hist)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
  }
  // one id of weight x
  SPEC_DEVINL void hist_add(int b, u64 x) {
    atomicAdd(&s.hist[0][b][lane], static_cast<unsigned>(x) & ((1u << limb) - 1u));
    atomicAdd(&s.hist[1][b][lane], static_cast<unsigned>(x >> limb) + (1u << cnt_at));
  }

  // Fine bins: distance from M, linear (weights: 109 to a halving; numbers: an eighth of them to the span), by
  // the bits of a sum rounded to a whole number, or, where that is too large, by a difference.
  struct Fine {
    float M, per, far;
    int b0;
    bool by_sum;
    SPEC_DEVINL int operator()(float v) const {
      if (by_sum) return b0 - __float_as_int(fmaf(fmaxf(v, far), per, kRound));
      return min(static_cast<int>((M - v) * per), kFar);
    }
  };
  template <bool MASS>
  SPEC_DEVINL Fine fine_bins(float span) const {
    Fine f;
    f.M = w.M;
    f.per = MASS ? fminf(w.c_hi, 1e28f) * kPerBit : (span > 0.f && span < 1e30f ? (kFine / 8) / span : 0.f);
    f.by_sum = !(MASS && w.wide) && fabsf(w.M) * f.per < 3.2e6f && f.per > 1e-25f;
    f.far = f.by_sum ? w.M - __fdividef(static_cast<float>(kFar), f.per) : 0.f;
    f.b0 = __float_as_int(fmaf(w.M, f.per, kRound));
    return f;
  }

  // The fine bins [from, to] between which top_p of the weight of {z >= lower} ends by the ids' numbers in
  // them, give or take 2^-13 of it; or (MASS false) the one of the k-th.  false: fewer than k.
  template <bool MASS>
  SPEC_DEVINL bool count_bins(const Fine& fine, float lower, float top_p, int k, int* from, int* to) {
    __syncthreads();  // (the bins lie where the last list was)
    for (int i = tid; i < kFine / 4; i += kT) reinterpret_cast<uint4*>(s.fine)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    each([&](int, const float4& z) {
      const int b[4] = {fine(z.x), fine(z.y), fine(z.z), fine(z.w)};
      const float v[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (v[q] >= lower && v[q] > -INFINITY) atomicAdd(&s.fine[b[q]], 1u);
    });
    cluster_barrier();
    // each CTA its part of the bins, a thread one to eight in a row
    const int per = 8 / C, b0 = (rank * kT + tid) * per;
    u64 v[8], mine = 0;
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = 0;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if (q >= per) break;
      unsigned n = 0;
#pragma unroll
      for (int r = 0; r < kMaxC; ++r)
        if (r < C) n += ld_remote32(remote(&s.fine[b0 + q], r));
      v[q] = MASS ? n * static_cast<u64>(__float2ull_rn(exp2f(36.f - static_cast<float>(b0 + q) * (1.f / kPerBit)))) : n;
      mine += v[q];
    }
    const u64 incl = warp_incl64(mine, lane);
    if (lane == 31) s.red[warp] = incl;
    __syncthreads();
    u64 excl = incl - mine, part = 0;
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      const u64 x = s.red[i];
      if (i < warp) excl += x;
      part += x;
    }
    const u64(*ex)[kMaxC] = exchange(part, 0);
    u64 all = 0;
    for (int r = 0; r < C; ++r) {
      if (r < rank) excl += ex[0][r];
      all += ex[0][r];
    }
    u64 first = static_cast<u64>(k), last = first;
    if (MASS) {
      const u64 t = part_of(all, top_p, true);
      first = max(t - (t >> 13), static_cast<u64>(1));
      last = min(t + (t >> 13), all);
    }
    if (all < first) return false;
    par ^= 1;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if (q >= per) break;
      const u64 next = excl + v[q];
      if (excl < first && first <= next)
        for (int r = 0; r < C; ++r) st_remote(remote(&s.ex[par][0][0], r), b0 + q);
      if (excl < last && last <= next)
        for (int r = 0; r < C; ++r) st_remote(remote(&s.ex[par][1][0], r), b0 + q);
      excl = next;
    }
    cluster_barrier();
    *from = static_cast<int>(s.ex[par][0][0]);
    *to = static_cast<int>(s.ex[par][1][0]);
    return true;
  }

  // top_p's threshold and, for the draws, seg (this warp's part of what it keeps): false where the bins by
  // numbers did not hold it, or too many ids.
  SPEC_DEVINL bool nucleus(float lower, float top_p, float* theta) {
    const Fine fine = fine_bins<true>(0.f);
    int from, to;
    count_bins<true>(fine, lower, top_p, 0, &from, &to);
    list_clear();
    u64 above = 0, rest = 0;
    each([&](int x, const float4& z) {
      int e[4];
      float t[4];
      w.power4(z, e, t);
      const float v[4] = {z.x, z.y, z.z, z.w};
      u64 u[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) u[q] = w.units(e[q], t[q]);
      if (max(max(e[0], e[1]), max(e[2], e[3])) > -w.off) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (w.is_large(e[q])) u[q] = w.large(e[q], t[q]);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int b = fine(v[q]);
        if (v[q] >= lower) {
          if (b < from)
            above += u[q];
          else
            rest += u[q];
          if (b >= from && b <= to && v[q] > -INFINITY) list_add(v[q], x + q);
        }
      }
    });
    above = warp_sum64(above);
    rest = warp_sum64(rest);
    if (lane == 0) {
      s.seg[warp] = above;
      s.red[warp] = rest;
    }
    __syncthreads();
    above = rest = 0;
    for (int i = 0; i < kW; ++i) {
      above += s.seg[i];
      rest += s.red[i];
    }
    const unsigned mine = min(s.n, kManyIds);
    const u64(*ex)[kMaxC] = exchange(above, rest | static_cast<u64>(mine) << 54);
    above = rest = 0;
    int n = 0;
    u64* counts = s.sums;
    for (int r = 0; r < C; ++r) {
      above += ex[0][r];
      rest += ex[1][r] & kMassMask;
      n += static_cast<int>(ex[1][r] >> 54);
    }
    if (tid < C) counts[tid] = ex[1][tid] >> 54;
    const u64 target = part_of(above + rest, top_p, true);
    if (n == 0 || n > kList || target <= above) return false;
    __syncthreads();
    pull(counts, n, true);
    if (!reaches(n, target - above, theta)) return false;
    if (!FILTER) {  // what this CTA's part of the list keeps, to its warps' weights
      if (tid < static_cast<int>(mine)) {
        const u64 x = s.list[tid];
        const float v = value_of(x);
        if (v >= *theta) atomicAdd(&s.seg[((id_of(x) >> 2) - g0) / wg], w.fixed(v));
      }
      __syncthreads();
    }
    return true;
  }

  // The k-th largest of {lower <= z}, -inf if there are fewer: false where too many ids lie near it.
  SPEC_DEVINL bool kth(float lower, float span, int k, float* theta) {
    const Fine fine = fine_bins<false>(span);
    int from, to;
    *theta = -INFINITY;
    if (!count_bins<false>(fine, lower, 0.f, k, &from, &to)) return true;
    list_clear();
    unsigned over = 0;
    each([&](int x, const float4& z) {
      const float v[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int b = fine(v[q]);
        if (b <= from && v[q] >= lower && v[q] > -INFINITY) {
          if (b < from)
            ++over;
          else
            list_add(v[q], x + q);
        }
      }
    });
    over = __reduce_add_sync(0xffffffffu, over);
    if (lane == 0) s.red[warp] = over;
    __syncthreads();
    u64 above = 0;
    for (int i = 0; i < kW; ++i) above += s.red[i];
    const u64(*ex)[kMaxC] = exchange(s.n, above);
    const int n = static_cast<int>(total_of(ex[0]));
    above = total_of(ex[1]);
    if (n > kList) return false;
    pull(ex[0], n, false);
    return reaches(n, static_cast<u64>(k) - above, theta);
  }

  // The largest value v with (MASS: weight, else number) of {lower <= z, z >= v}
  // at least the target: top_p of the whole, or k.  -inf if there is none.
  template <bool MASS>
  SPEC_DEVINL float select(float lower, float span, float top_p, int k) {
    const Fine fine = fine_bins<MASS>(span);
    __syncthreads();  // (hist lies where the last list was put in order)
    hist_clear();
    each([&](int, const float4& z) {
      const float v[4] = {z.x, z.y, z.z, z.w};
      const int at[4] = {fine(z.x) / kBins, fine(z.y) / kBins, fine(z.z) / kBins, fine(z.w) / kBins};
      if (!MASS) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (v[q] >= lower) atomicAdd(&s.hist[0][at[q]][lane], 1u);
        return;
      }
      int e[4];
      float t[4];
      w.power4(z, e, t);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (v[q] >= lower) {
          const unsigned x = w.units(e[q], t[q]);
          atomicAdd(&s.hist[0][at[q]][lane], x & ((1u << limb) - 1u));
          atomicAdd(&s.hist[1][at[q]][lane], (x >> limb) + (1u << cnt_at));
        }
      if (max(max(e[0], e[1]), max(e[2], e[3])) > -w.off) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (w.is_large(e[q]) && v[q] >= lower) {
            const u64 x = w.large(e[q], t[q]);
            atomicAdd(&s.hist[0][at[q]][lane], static_cast<unsigned>(x) & ((1u << limb) - 1u));
            atomicAdd(&s.hist[1][at[q]][lane], static_cast<unsigned>(x >> limb));
          }
      }
    });
    Found f = find_bin<MASS>([&](u64 all) { return MASS ? part_of(all, top_p, true) : static_cast<u64>(k); });
    if (f.bin < 0) return -INFINITY;  // (fewer than k)
    unsigned from = f.bin * kBins, width = kBins;  // the fine bins that the threshold lies in
    unsigned khi = 0xFFFFFFFFu, klo = 1;           // and the keys
    // f(id, z) for the logits there
    auto each_here = [&](auto&& fn) {
      each([&](int x, const float4& z) {
        const bool h0 = fine(z.x) - from < width, h1 = fine(z.y) - from < width, h2 = fine(z.z) - from < width,
                   h3 = fine(z.w) - from < width;
        if (!(h0 || h1 || h2 || h3)) return;
        const bool h[4] = {h0, h1, h2, h3};
        const float v[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const unsigned kv = key_of(v[q]);
          if (h[q] && v[q] >= lower && v[q] > -INFINITY && kv >= klo && kv <= khi) fn(x + q, v[q]);
        }
      });
    };
    if (f.n > kList) {
      hist_clear();
      each_here([&](int, float v) {
        if (MASS)
          hist_add(fine(v) - from, w.fixed(v));
        else
          atomicAdd(&s.hist[0][fine(v) - from][lane], 1u);
      });
      const u64 target = f.target;
      f = find_bin<MASS>([&](u64) { return target; });
      from += f.bin;
      width = 1;
    }
    for (;;) {
      list_clear();
      each_here([&](int x, float v) { list_add(v, x); });
      __syncthreads();
      const u64(*ex)[kMaxC] = exchange(s.n, 0);
      const int n = static_cast<int>(total_of(ex[0]));
      if (n <= kList) {  // (each CTA finds it for itself)
        pull(ex[0], n, MASS);
        float v = lower;
        reaches(n, f.target, &v);
        return v;
      }
      // still too many: bins of keys between the smallest and the largest
      each_here([&](int, float v) {
        const unsigned kv = key_of(v);
        atomicMin(&s.lo, kv);
        atomicMax(&s.hi, kv);
      });
      __syncthreads();
      ex = exchange(s.lo, s.hi);
      klo = 0xFFFFFFFFu;
      khi = 0;
      for (int r = 0; r < C; ++r) {
        klo = min(klo, static_cast<unsigned>(ex[0][r]));
        khi = max(khi, static_cast<unsigned>(ex[1][r]));
      }
      if (klo == khi) return key_value(klo);  // one value
      int shift = 0;
      while (((khi - klo) >> shift) >= kBins) ++shift;
      hist_clear();
      each_here([&](int, float v) {
        const int b = static_cast<int>((khi - key_of(v)) >> shift);
        if (MASS)
          hist_add(b, w.fixed(v));
        else
          atomicAdd(&s.hist[0][b][lane], 1u);
      });
      const u64 target = f.target;
      f = find_bin<MASS>([&](u64) { return target; });
      khi -= static_cast<unsigned>(f.bin) << shift;
      klo = max(klo, khi - min(khi, (1u << shift) - 1u));
    }
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
      if (tid == 0) s.sum_inv = static_cast<float>(static_cast<double>(1ull << (30 + w.off)) / static_cast<double>(total));
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
    if (!FILTER && rank == 0)
      for (int d = tid; d < p.draws; d += kT) p.tokens[static_cast<long long>(row) * p.draws + d] = only;
    if (FILTER || p.probs)
      write_row(row, [&](int x, const float4&, float (&v)[4]) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (FILTER)
            v[q] = only < 0 || x + q == only ? v[q] : -INFINITY;
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
    const int gn = max(0, min(per, groups - g0));
    wg = (gn + kT - 1) / kT * 32;
    i0 = min(warp * wg, gn);
    i1 = min(i0 + wg, gn);
    // What a lane adds to a bin fits its two counters: 512 ids of up to 2^35.5 (23 bits low; 12.5 + 9 high, and
    // 10 for their number), or 1024 of up to 2^32.5 (22; 10.5 + 10, and 11)
    w.off = V <= 131072 ? 5 : 2;
    limb = V <= 131072 ? 23 : 22;
    cnt_at = V <= 131072 ? 22 : 21;
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
    w.wide = !(far < 30000.f) || !(c_hi < 1e30f) || !(c_hi > 1e-25f);
    w.zlow = w.wide ? 0.f : M - __fdividef(150.f, c_hi);
    w.n0 = __float_as_int(__fadd_rn(__fmul_rn(M, c_hi), kRound));
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
    if (n <= kList) {  // few: one CTA decides
      if (rank == 0) {
        pull(ex[0], n, false);
        if (top_k && n > rs.k) reaches(n, rs.k, &theta);
        if (top_p || !FILTER) {
          u64 x = 0;
          if (tid < n) {
            const float v = value_of(s.l.x[tid]);
            x = v >= theta ? w.fixed(v) : 0ull;
            s.l.weight[tid] = x;
          }
          x = warp_sum64(x);
          if (lane == 0) s.red[warp] = x;
          if (tid == 0) s.hi = 0;
          __syncthreads();
          for (int i = 0; i < kW; ++i) total += s.red[i];
        }
        if (top_p) {
          float v = theta;
          reaches(n, part_of(total, rs.top_p, true), &v);
          if (!FILTER && v > theta) {  // weights of what is cut now go
            u64 x = 0;
            if (tid < n) {
              x = value_of(s.l.x[tid]) >= v ? s.l.weight[tid] : 0ull;
              s.l.weight[tid] = x;
            }
            x = warp_sum64(x);
            if (lane == 0) s.red[warp] = x;
            __syncthreads();
            total = 0;
            for (int i = 0; i < kW; ++i) total += s.red[i];
          }
          theta = fmaxf(theta, v);
        }
        if (!FILTER) {
          if (tid < p.draws) s.l.targets[tid] = draw_target(row, tid, total);
          __syncthreads();
          int i;
          bool first;
          u64 sum;  // cumulative weight in the order of ids
          over_list(n, i, first, sum, [](u64 x, u64 y) { return static_cast<unsigned>(y) >= static_cast<unsigned>(x); });
          if (i < n && first)
            for (int d = 0; d < p.draws; ++d)
              if (s.l.targets[d] < sum && s.l.targets[d] >= sum - s.l.weight[i])
                p.tokens[static_cast<long long>(row) * p.draws + d] = id_of(s.l.x[i]);
        }
      }
      ex = exchange(key_of(theta), total);  // (and no CTA leaves before its list is read)
      if (FILTER || p.probs) write_kept(row, key_value(static_cast<unsigned>(ex[0][0])), ex[1][0]);
      return;
    }
    if (top_k) {
      float v;
      if (!kth(lower, M - least, rs.k, &v)) v = select<false>(lower, M - least, 0.f, rs.k);
      theta = fmaxf(theta, v);
    }
    bool weighed = false;
    if (top_p) {
      float v;
      weighed = nucleus(theta, rs.top_p, &v);
      if (!weighed) v = select<true>(theta, 0.f, rs.top_p, 0);
      theta = fmaxf(theta, v);
    }
    if (FILTER) {
      write_kept(row, theta, 0);
      cluster_barrier();  // no CTA leaves before its list is read
      return;
    }
    // the warps' weights, and the cluster's
    u64 sum = 0;
    if (!weighed) {
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
    }
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
  while (C < kMaxC && (groups > C * kT * 8 || (groups > C * kT && p.rows * C <= sms))) C *= 2;
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
