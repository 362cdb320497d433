// Attention of n new positions over the 8-bit paged KV cache (kv8_attention_wide.cu
// takes the calls with many query rows).
//   s_j = scale * q . (ks_j k_j),  o = sum_j p_j vs_j v_j / sum_j p_j,
//   p_j = exp(s_j - max s) over the slots that the row's token may see
// (the cached ones, and of the new ones its own and earlier, or those of its
// ancestor mask); a row that sees nothing is zero.
//
// The cache is read once, by TMA, into shared memory, and enters the tensor
// cores as it is stored: both products are tcgen05.mma kind::f8f6f4 with e4m3
// operands and fp32 accumulators in TMEM, so no key or value is ever
// converted.  The other operand is split into e4m3 pieces that add up to it:
//   q row = 2^k (hi + 2^-5 lo)       bf16 has 8 significant bits, a piece 4: exact for
//                                    elements down to 2^-14 of the row's largest (at
//                                    2^7 or more), below off by 2^-22 of it at most
//   p     = hi + 2^-4 mid + 2^-8 lo  an fp16 weight's 11 bits, in steps of 2^-17 at the least
// and the pieces lie side by side in the N dimension, so a tile of keys or
// values is read from shared memory once whatever their number.
//
// One CTA takes the RT query rows (n tokens x the query heads of a KV head) of
// one (sequence, KV head) over a run of 128-key tiles; the runs of one row tile
// are a thread-block cluster, whose CTAs merge their partial sums through
// distributed shared memory: no workspace, no second launch.
//   S^T [128 keys][RT hi | RT lo]          = K [keys][hd] x Q^T
//   O^T [128 dims][RT hi | mid | lo]      += V^T [dims][keys] x P
// Thread t of the four softmax warps owns TMEM lane t: key t of S^T, then
// dimension t of O^T.  A key's scales so belong to one thread: ks multiplies its
// scores, and vs enters as an exponent,
//   p'_j = p_j vs_j = 2^(s_j + log2 vs_j - M),
// which keeps the weights that enter the product in the pieces' range; the sum
// of the p_j themselves adds p'_j / vs_j in fp32.  The reference M of a row
// need not be its maximum: the pieces hold weights up to 448, so M is set to put
// the maximum of the first tile at 2^2 and raised only when a weight would pass
// 2^8.75 (one barrier per tile asks whether any does).  Until then O^T adds
// up in TMEM and no thread reads it.
//
// With a row's largest weight at 2^2 the pieces' last step, 2^-17, is 2^-19 of it,
// and in a long context that many keys may each have less.  Rounded to nearest,
// weights that are alike would all go the same way, say to zero where together they
// are half of the row, while the sum of the p_j keeps them.  So a weight is rounded
// up or down by a fixed pattern of slot numbers (slot_dither), and n errors add up
// to about sqrt(n) of them.  Measured against rounding to nearest, batch 64 and 16:
// the pattern 51.7 to 52.1 us and 23.7 to 23.8; a fourth piece 54.0 and 25.5; maxima
// at 2^4 and M set anew every 16 tiles 54.2 and 24.9.
//
// Why 11 bits: the output is bf16, 8 bits.  Errors of 2^-11 of the weights at the most
// move it by a small part of its own rounding, which falls the other way in a few
// percent of the elements; two fp16 values a weight would double the pieces.
//
// After the softmax's four warps one issues the TMA loads of K, one those of V,
// one the score MMAs and one the products: one thread for both of either kind had
// less time a tile than its waits and issues took.  S and P are double-buffered,
// so the scores of tile i + 1 and the products of tile i - 1 run beside the
// softmax of tile i.
//
// Why two CTAs an SM (113 KB and 128 registers a thread each): a tile is one
// chain of score, weights and product, and another CTA's chain fills its gaps.
// Where the clusters are too few for that (one KV head's tiles are shared by 16
// CTAs at the most), a CTA has an SM to itself and two groups of softmax warps (NG
// = 2), one for the even and one for the odd tiles of its run, each with its own
// M, sums, O and issuing warps; their sums are put together at the end.  (Groups
// that share a tile, half the rows each, took the time of one.)
//
// What bounds it, with what it measured (152 SMs; 32 query heads on 8 KV heads,
// head dim 128 and 5 tokens a sequence unless it says otherwise; device time of
// a launch inside a graph):
//   64 sequences, 309 MB of cache: 52 us, 5.9 TB/s; in its loop it runs at the
//     copy bandwidth, the rest is the second wave's prologue and the tail
//   16 sequences, 77 MB: 24 us, 3.2 TB/s; ~7 us of setup and end, and tiles
//     that do not divide evenly over the SMs
//   1 sequence of 131000 slots: 1 token 44.6 us, 6.0 TB/s, 5 tokens 57 us; 12 CTAs
//     for each of the 8 KV heads, so 96 of the SMs take part (a cluster lies
//     within a group of SMs, and 8 of 16 do not fit at once)
//   1 sequence of 2048: 8.4 us, the latency of one tile, the merge and a launch
//   1 sequence x 32 tokens at 4000 slots: 15.3 us; the softmax threads' chain,
//     with conversions to e4m3 at a quarter rate (for more rows: the other kernel)
#include "kv8_attn.cuh"

namespace spec {
namespace {

constexpr int kSoft = 128;                  // threads of a softmax group
// The warps of a CTA with NG groups: those of the groups, K and V loader, and S
// and O issuer of each group.
template <int NG>
struct Warps {
  static constexpr int kLoadK = 4 * NG, kLoadV = kLoadK + 1, kIssue = kLoadK + 2, kAll = kIssue + 2 * NG;
};
constexpr int kPSpan = 32;                  // bytes of a key's row in one span of P
// The kernel for many query rows takes over where a KV head has more than 64 of
// them and the call's (128 rows x 128 keys) at full capacity are 448 or more:
// below, its longer prologue and merge cost more than its cheaper tiles save.
// Measured, this kernel / that one in us (32 heads on 8, head dim 128, 4000 slots
// but where it says): 1 x 32 tokens (256) 15.3 / 15.1, 1 x 64 (512) 18.7 / 18.1,
// 1 x 96 (792) 29.6 / 19.2, 1 x 128 (1056) 31.5 / 22.1, 16 x 32 (4096) 75 / 51,
// 4 x 64 at 700 (384) 13.6 / 15.4, 4 x 128 at 700 (896) 25.7 / 16.7, head dim 64
// 4 x 32 at 1900 (480) 15.5 / 12.1; 64 rows a head: 16 x 16 tokens 45 / 50,
// 64 x 16 141 / 149.  (Capacity and not length, which the host does not know: the
// 4 x 64 tokens at 700 slots in a table of 32768 take the other kernel and 15.1 us.)
constexpr int kWideRows = 64, kWideWork = 448;
constexpr float kTopExp = 8.75f;            // 2^8.75 < 448: weights that fit e4m3
constexpr float kStartExp = 2.f;            // exponent of a row's maximum where M is set
constexpr float kLift = 4.f;                // exponents are kept this much higher: fp16 then holds small weights too

// N columns of the thread's lane at each of two places, ready for use.
template <int N>
SPEC_DEVINL void tmem_ld2(uint32_t ta, uint32_t tb, uint32_t (&a)[N], uint32_t (&b)[N]) {
  if constexpr (N == 8) {
    tmem_ld_x8(ta, a);
    tmem_ld_x8(tb, b);
  } else {
    tmem_ld_x16(ta, a);
    tmem_ld_x16(tb, b);
  }
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(a[i]), "+r"(b[i]));  // no use moves above the wait
}
SPEC_DEVINL void tmem_ld_wait(uint32_t (&a)[8], uint32_t (&b)[8], uint32_t (&c)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) asm volatile("" : "+r"(a[i]), "+r"(b[i]), "+r"(c[i]));
}

SPEC_DEVINL uint32_t f16x2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
SPEC_DEVINL uint32_t f16x2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
SPEC_DEVINL uint32_t f16x2_to_e4m3x2(uint32_t a) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(a));
  return r;
}
// Two fp16 numbers in [-1/2, 1/2) of the last piece's smallest step (2^-9), made of
// slot t by two rounds of multiply and xor-shift: in any stretch of slots, and in
// every k'th of them, as evenly spread as random ones.
SPEC_DEVINL uint32_t slot_dither(int t) {
  uint32_t h = static_cast<uint32_t>(t) * 0x9E3779B1u;
  h = (h ^ (h >> 15)) * 0x85EBCA77u;
  h ^= h >> 15;
  return f16x2_fma((h & 0x03FF03FFu) | 0x3C003C00u, 0x18001800u, 0x9A009A00u);  // ([1, 2) - 1.5) 2^-9
}
// ... and of chunk c of key i's row of P, which is cut into spans of 32 bytes
// ([128 keys][32 bytes] each): three pieces of 24 rows then take 96 bytes a key
// where a 128-byte span would take 128.
SPEC_DEVINL uint32_t p_off(int i, int c) { return (c >> 1) * (kTile * kPSpan) + swz_off<kPSpan>(i, c & 1); }

// Named barrier that also tells every thread whether any of them raised v.
SPEC_DEVINL bool named_bar_any(int id, int nthreads, bool v) {
  int any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 q, %3, 0;\n\t"
      "barrier.cta.red.or.pred p, %1, %2, q;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(any)
      : "r"(id), "r"(nthreads), "r"(v ? 1 : 0)
      : "memory");
  return any != 0;
}

// Reduce RT values per lane (a multiple of 8) over the warp's 32 lanes with op;
// lane l < RT then holds the result of value l.  Halving: each step sends half
// of what is left, first within groups of 8 values, then across the groups.
template <int RT, class Op>
SPEC_DEVINL float warp_rows_reduce(const float (&v)[RT], float none, Op op) {
  const int lane = threadIdx.x & 31;
  float g[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (q >= RT / 8) {
      g[q] = none;
      continue;
    }
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = v[8 * q + i];
#pragma unroll
    for (int o = 4; o >= 1; o >>= 1) {
      const bool upper = (lane & o) != 0;
#pragma unroll
      for (int i = 0; i < o; ++i) {
        const float send = upper ? x[i] : x[i + o];
        const float keep = upper ? x[i + o] : x[i];
        x[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, o));
      }
    }
    g[q] = x[0];
  }
  const bool up16 = (lane & 16) != 0, up8 = (lane & 8) != 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float send = up16 ? g[i] : g[i + 2];
    const float keep = up16 ? g[i + 2] : g[i];
    g[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, 16));
  }
  const float send = up8 ? g[0] : g[1];
  const float keep = up8 ? g[1] : g[0];
  return op(keep, __shfl_xor_sync(0xffffffffu, send, 8));
}

template <int HD, int RT, int NG>
struct AttSmem {
  static constexpr int kMaxStages = NG > 1 ? 6 : 5;  // of K, and of V
  static constexpr uint32_t kTileB = kTile * HD;  // bytes of a K or V tile
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kP = kQ + 2 * RT * HD;
  static constexpr uint32_t kPB = (3 * RT + kPSpan - 1) / kPSpan * (kTile * kPSpan);  // bytes of one P buffer
  static constexpr uint32_t kK = kP + 2 * NG * kPB;
  // then nk K tiles, nv V tiles and Misc
  struct Misc {
    uint64_t full_k[kMaxStages], full_v[kMaxStages], empty_k[kMaxStages], empty_v[kMaxStages];
    uint64_t s_full[2 * NG], s_free[2 * NG], p_full[2 * NG], o_full[2 * NG], drain[2 * NG];
    uint64_t anc[RT];
    alignas(16) float red[4 * NG][RT];   // per-warp maxima (sums at the end); this and the next two are read as float4
    float mneg[4 * NG][RT];              // each warp's copy of kLift - M
    float cq[RT];                   // score factor of a row: 2^k scale log2(e)
    alignas(16) float stat[2][RT];  // this CTA's M and sum per row
    float part[NG][2][RT];          // ... a group's, and then the factor of its O
    alignas(16) long long out[RT];  // where the row's output starts, -1: no such row
    union {                         // before the loop, and from it on
      alignas(16) int len[kSortSeqs];
      uint32_t nan[RT][HD / 32];  // outputs that a NaN value code reaches
    };
    uint32_t tmem;
    alignas(8) int pages[2][16];  // page ids of the 8 tiles being loaded, of K and of V
    int seq, seq_len, unit, unfit, abort, any_nan;
  };
  // partial sums [RT][HD] fp32, over the K ring once every MMA is done
  static constexpr uint32_t kO = kK;
  static_assert(offsetof(Misc, mneg) % 16 == 0 && offsetof(Misc, cq) % 16 == 0 && alignof(Misc) == 16 && kK % 1024 == 0,
                "row arrays are read as float4");
  static_assert(RT * HD * 4 <= 4 * kTileB, "the partial sums lie over a ring of two stages or more");
  static constexpr uint32_t bytes(int nk, int nv) { return kK + (nk + nv) * kTileB + sizeof(Misc); }
  static constexpr int kNO = (3 * RT + 15) / 16 * 16;              // O columns (M = 128 takes multiples of 16)
  static constexpr int kGroupCols = 4 * RT + kNO;  // a group's two S buffers and O
  static constexpr uint32_t kTmemCols = NG * (RT >= 24 ? 256 : (RT == 16 ? 128 : 64));
  static_assert(NG * kGroupCols <= static_cast<int>(kTmemCols), "the groups' columns");
};

struct AttMaps {
  CUtensorMap k, v;
};

// kLo: the bf16 residual of o is written too (a kernel of its own: as a branch,
// its code cost batch 64 5%).
template <int HD, int RT, bool kLo, int NG>
__global__ void __launch_bounds__(32 * Warps<NG>::kAll, 3 - NG)
    kv8_attention_kernel(const __grid_constant__ AttMaps maps, const Kv8AttnParams p, const int csize, const int NK,
                         const int NV, const int share) {
  using S = AttSmem<HD, RT, NG>;
  using W = Warps<NG>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t base = smem_u32(smem_raw);  // swizzled tiles lie on their own span's boundaries
  const uint32_t ring_k = base + S::kK, ring_v = ring_k + NK * S::kTileB;
  auto& sm = *reinterpret_cast<typename S::Misc*>(smem_raw + (ring_v + NV * S::kTileB - smem_u32(smem_raw)));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x % csize, rtile = blockIdx.x / csize, h = blockIdx.y;
  const int G = p.G, R = p.n * G, rbase = rtile * RT;

  if (tid == 0) {
    for (int i = 0; i < S::kMaxStages; ++i) {
      mbar_init(&sm.full_k[i], 1);
      mbar_init(&sm.full_v[i], 1);
      mbar_init(&sm.empty_k[i], 1);
      mbar_init(&sm.empty_v[i], 1);
    }
    for (int i = 0; i < 2 * NG; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.s_free[i], kSoft);
      mbar_init(&sm.p_full[i], kSoft);
      mbar_init(&sm.o_full[i], 1);
      mbar_init(&sm.drain[i], 1);
    }
    fence_mbar_init();
    sm.abort = 0;
    sm.any_nan = 0;
  }
  if (tid == 32 * W::kLoadK) {
    prefetch_tmap(&maps.k);
    prefetch_tmap(&maps.v);
  }
  if (warp == W::kAll - 1) {
    tmem_alloc(&sm.tmem, S::kTmemCols);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();  // barriers and TMEM set up
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  grid_dep_wait();

  // Which sequence, and how many of the cluster's CTAs share its tiles (the CTAs
  // that a short sequence does not need leave).
  const int cap = p.max_pages * kPageSlots;
  const int slots = csize > 1 ? share / (p.Hkv * (gridDim.x / csize)) : 0;  // CTAs of the GPU per KV head and row tile
  const AttPick pick = att_pick(p, csize > 1, slots, sm);
  const int b = pick.b;
  // ---- the query rows: row r = token r / G, head h * G + r % G (loads on their
  // way before the length is known)
  constexpr int TPR = RT <= 16 && HD == 128 ? 8 : 4;  // threads per query row
  constexpr int E = HD / TPR;                         // ... and their elements
  static_assert(RT * TPR <= kSoft && RT * TPR % 32 == 0 && E % 16 == 0, "whole warps, 16 elements a thread");
  const int qr = tid / TPR, qpart = tid % TPR;
  uint4 qw[E / 8];
  long long out_at = -1;
  unsigned long long am = 0ull;
  if (tid < RT * TPR) {
    const int rr = rbase + qr, tok = rr / G, head = h * G + rr - tok * G;
#pragma unroll
    for (int c = 0; c < E / 8; ++c) qw[c] = make_uint4(0, 0, 0, 0);
    if (rr < R) {
      const long long m = static_cast<long long>(b) * p.n + tok;
      const uint16_t* q = p.q + m * p.q_ld + head * HD + qpart * E;
#pragma unroll
      for (int c = 0; c < E / 8; ++c) qw[c] = *reinterpret_cast<const uint4*>(q + c * 8);
      if (qpart == 0 && p.anc) am = p.anc[m];
      out_at = m * p.o_ld + head * HD;
    }
  }

  const bool sorted = pick.sorted;
  const int L = sorted ? sm.seq_len : p.base[b];
  const bool over = L < 0 || L > cap - p.n;
  const int T = over ? 0 : L + p.n;  // slots [0, T)
  const int tiles = (T + kTile - 1) / kTile;
  int C = 1, i0 = 0, nt = tiles;  // CTAs that share the tiles; this one's
  if (csize > 1) {
    const int unit = sorted ? sm.unit : max(kMinTiles, p.B > 1 ? 0 : (tiles + slots - 1) / max(slots, 1));
    C = min(csize, max(1, (tiles + unit - 1) / unit));
    if (rank >= C) {  // (its peers' barriers go on without it)
      if (warp == W::kAll - 1) tmem_dealloc(tmem, S::kTmemCols);
      return;
    }
    i0 = tiles * rank / C;  // (tiles * C <= 2^13 * 2^4)
    nt = tiles * (rank + 1) / C - i0;
  }
  const int32_t* table = p.table + static_cast<long long>(b) * p.max_pages;
  const auto page_of = [&](int t) {  // the page of slot t, clamped into the pool
    const int pg = table[min(t / kPageSlots, p.max_pages - 1)];
    if (pg < 0 || pg >= p.n_pages) {
      if (t < T) set_status(p.status, SPEC_DEV_BAD_PAGE);
      return pg < 0 ? 0 : p.n_pages - 1;
    }
    return pg;
  };

  // ---- ... as e4m3 pieces
  if (tid < RT * TPR) {
    float x[E];
#pragma unroll
    for (int c = 0; c < E / 8; ++c) {
      const uint32_t v[4] = {qw[c].x, qw[c].y, qw[c].z, qw[c].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[8 * c + 2 * k] = bf16lo(v[k]);
        x[8 * c + 2 * k + 1] = bf16hi(v[k]);
      }
    }
    float mx = 0.f;
    bool odd = false;  // an infinite or NaN element: the whole row is NaN
#pragma unroll
    for (int k = 0; k < E; ++k) {
      odd |= !(fabsf(x[k]) <= 3.402823466e38f);
      mx = fmaxf(mx, fabsf(x[k]));
    }
#pragma unroll
    for (int o = 1; o < TPR; o <<= 1) {
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      odd |= __shfl_xor_sync(0xffffffffu, odd ? 1 : 0, o) != 0;
    }
    // 2^-k brings the largest element into [128, 256) (k at least -100: a row
    // of smaller elements scores zero to fp32's last bit anyway)
    const int k2 = max(static_cast<int>(__float_as_uint(mx) >> 23) - 127 - 7, -100);
    const float down = __uint_as_float(static_cast<uint32_t>(127 - k2) << 23);
#pragma unroll
    for (int c = 0; c < E / 16; ++c) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float a = odd ? 0.f : x[16 * c + 2 * k] * down, d = odd ? 0.f : x[16 * c + 2 * k + 1] * down;
        const uint32_t w = e4m3x2(a, d);
        const float2 f = e4m3x2_to_f32(w);
        const uint32_t u = e4m3x2((a - f.x) * 32.f, (d - f.y) * 32.f);
        if (k & 1) {
          hi[k / 2] |= w << 16;
          lo[k / 2] |= u << 16;
        } else {
          hi[k / 2] = w;
          lo[k / 2] = u;
        }
      }
      const int ch = qpart * (E / 16) + c;
      st_shared_v4(base + S::kQ + swz_off<HD>(qr, ch), hi[0], hi[1], hi[2], hi[3]);
      st_shared_v4(base + S::kQ + swz_off<HD>(RT + qr, ch), lo[0], lo[1], lo[2], lo[3]);
    }
    if (qpart == 0) {
#pragma unroll
      for (int c = 0; c < 4 * NG; ++c) sm.mneg[c][qr] = -kNoRef;
      sm.cq[qr] = odd ? __uint_as_float(0x7FC00000u)
                      : p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + k2) << 23);
      sm.out[qr] = out_at;
      sm.anc[qr] = am;
#pragma unroll
      for (int c = 0; c < HD / 32; ++c) sm.nan[qr][c] = 0u;
    }
    fence_async_smem();
  }
  // q and the row arrays are ready (the loading warps need neither)
  if (warp != W::kLoadK && warp != W::kLoadV) named_bar(3, NG * (kSoft + 64));
  tc_fence_after();

  float mrun = kNoRef;  // lane r: row r's reference M

  if (warp == W::kLoadK || warp == W::kLoadV) {
    // ------------------------------------------- TMA: the tiles of K, or of V
    const bool is_k = warp == W::kLoadK;
    const int entries = (T + kPageSlots - 1) / kPageSlots - 2 * i0;  // pages from this CTA's first slot on
    const auto page_at = [&](int e) { return e < entries ? page_of(i0 * kTile + e * kPageSlots) : 0; };
    att_load_tiles<HD>(is_k ? &maps.k : &maps.v, is_k ? sm.full_k : sm.full_v, is_k ? sm.empty_k : sm.empty_v,
                       sm.pages[is_k ? 0 : 1], is_k ? ring_k : ring_v, is_k ? NK : NV, nt, entries, p.Hkv, h,
                       &sm.abort, page_at);
  } else if (warp >= W::kIssue) {
    // ------------------------------------- MMA issuers: scores, products
    // An MMA of N columns holds the pipe for 32 + N / 4 cycles (M = 128, K =
    // 32), and its thread for 57 to 92 at any N, so the two products of a tile
    // come from two threads.
    if (lane == 0) {
      const int g = (warp - W::kIssue) / 2;  // of group g: its j'th tile is the CTA's NG j + g
      const bool scores = (warp - W::kIssue) % 2 == 0;
      const int stages = scores ? NK : NV;
      const uint32_t tg = tmem + g * S::kGroupCols;
      Ring ring;
      if (g) ring.next(stages);
      bool ok = true;
      const uint64_t a0 = scores ? sdesc_rows<HD>(ring_k, 16) : sdesc_rows<HD>(ring_v, 0);
      const uint64_t b0 = scores ? sdesc_rows<HD>(base + S::kQ, 16)
                                 : sdesc_rows<kPSpan>(base + S::kP + g * 2 * S::kPB, kTile * kPSpan);
      const int ntg = (nt + NG - 1 - g) / NG;
      for (int j = 0; j < ntg; ++j) {
        const int buf = j & 1, at = 2 * g + buf;
        const uint64_t a = a0 + static_cast<uint32_t>(ring.s) * (S::kTileB >> 4);
        if (scores) {
          ok = (j < 2 || mbar_wait(&sm.s_free[at], static_cast<uint32_t>((j / 2 - 1) & 1), &sm.abort)) &&
               mbar_wait(&sm.full_k[ring.s], ring.par, &sm.abort);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < HD / 32; ++kk)
            umma_e4m3(tg + buf * 2 * RT, a + kk * 2, b0 + kk * 2, idesc_e4m3(kTile, 2 * RT, false, false),
                      kk > 0 ? 1u : 0u);
          umma_commit(&sm.s_full[at]);
          umma_commit(&sm.empty_k[ring.s]);
        } else {
          ok = mbar_wait(&sm.full_v[ring.s], ring.par, &sm.abort) &&
               mbar_wait(&sm.p_full[at], static_cast<uint32_t>((j >> 1) & 1), &sm.abort);
          if (!ok) break;
          tc_fence_after();
          const uint64_t bp = b0 + static_cast<uint32_t>(buf) * (S::kPB >> 4);
#pragma unroll
          for (int kk = 0; kk < kTile / 32; ++kk)
            // head dim 64: the 128 rows of the A operand are the 64 dimensions twice
            umma_e4m3(tg + 4 * RT, a + kk * (32 * HD >> 4), bp + kk * (32 * kPSpan >> 4),
                      idesc_e4m3(kTile, S::kNO, true, true), j > 0 || kk > 0 ? 1u : 0u);
          umma_commit(&sm.o_full[at]);
          umma_commit(&sm.empty_v[ring.s]);
        }
#pragma unroll
        for (int k = 0; k < NG; ++k) ring.next(stages);
      }
      if (!ok) {  // MMAs in flight end before TMEM and shared memory go
        int none = 0;
        umma_commit(&sm.drain[2 * g + (scores ? 0 : 1)]);
        mbar_wait(&sm.drain[2 * g + (scores ? 0 : 1)], 0, &none);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------- softmax and accumulation
    // A wait that gives up sets the abort flag; the threads leave the loop
    // together at its barrier.
    const int g = NG > 1 ? warp / 4 : 0, st = tid - g * kSoft;  // group, key (then dimension) of the thread
    const uint32_t tg = tmem + (static_cast<uint32_t>(warp % 4 * 32) << 16) + g * S::kGroupCols;
    const int bar = 1 + 3 * g;                // the group's two named barriers, bar and bar + 1
    const int ntg = (nt + NG - 1 - g) / NG;   // its tiles
    const int sub = (st % kPageSlots) / kKv8Block;
    const auto scale_at = [&](int pg) { return (static_cast<long long>(pg) * p.Hkv + h) * kKv8Sub + sub; };
    const auto seen = [&](int t) {  // bit r: row rbase + r sees slot t
      if (t < L) return 0xFFFFFFFFu;
      if (t >= T) return 0u;
      const int k = t - L;
      if (p.anc) {
        uint32_t m = 0u;
        if (k < 64)
#pragma unroll 1
          for (int r = 0; r < RT; ++r) m |= static_cast<uint32_t>((sm.anc[r] >> k) & 1ull) << r;
        return m;
      }
      const int first = k * G - rbase;  // row rr (token rr / G) sees new slot k iff rr >= k * G
      return first <= 0 ? 0xFFFFFFFFu : (first >= 32 ? 0u : 0xFFFFFFFFu << first);
    };
    // the pages that the new slots lie on, looked at in the end
    const int new_pages = over ? 0 : (T - 1) / kPageSlots - L / kPageSlots + 1;
    const int new_page = tid < new_pages ? table[L / kPageSlots + tid] : 0;
    // rows r .. r + 7 of O, the pieces put together
    const auto o_rows = [&](int r, float (&o)[8]) {
      uint32_t w[3][8];
#pragma unroll
      for (int q = 0; q < 3; ++q) tmem_ld_x8(tg + (4 + q) * RT + r, w[q]);
      tmem_ld_wait(w[0], w[1], w[2]);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        o[k] = fmaf(__uint_as_float(w[2][k]), 0.00390625f,
                    fmaf(__uint_as_float(w[1][k]), 0.0625f, __uint_as_float(w[0][k])));
    };
    float l[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) l[r] = 0.f;
    // this thread's scales, one tile ahead, and its page, two ahead (the TMA
    // warp flags ids outside the pool; here they are clamped)
    const int last_page = p.max_pages - 1;
    const auto page_id = [&](int i) { return table[min(((i0 + NG * i + g) * kTile + st) / kPageSlots, last_page)]; };
    const auto scale_of = [&](const float* sc, int pg) {
      return sc[scale_at(min(max(pg, 0), p.n_pages - 1))];
    };
    int pg1 = ntg > 0 ? page_id(0) : 0;
    float ks_n = ntg > 0 ? scale_of(p.ks, pg1) : 1.f, vs_n = ntg > 0 ? scale_of(p.vs, pg1) : 1.f;
    pg1 = ntg > 1 ? page_id(1) : 0;
    bool stopped = false;
    Ring vring;
    if (g) vring.next(NV);
    for (int i = 0; i < ntg; ++i) {  // the group's i'th tile
      const int buf = i & 1, t0 = (i0 + NG * i + g) * kTile, t = t0 + st;
      const float ks = ks_n, vs = vs_n;
      if (i + 1 < ntg) {
        ks_n = scale_of(p.ks, pg1);
        vs_n = scale_of(p.vs, pg1);
        pg1 = page_id(i + 2);
      }
      const uint32_t dither2 = slot_dither(t);
      const bool none = t >= T;  // past the end: no scale to read
      const float lvs = none ? 0.f : static_cast<float>(static_cast<int>(__float_as_uint(vs) >> 23) - 127);
      const float ivs = none ? 0.f : pow2_inv(vs) * 0.0625f;  // (of weights that are 2^kLift too large)
      const bool masked = t0 + kTile > L;  // the tile holds slots that some row does not see
      const uint32_t vis = masked ? seen(t) : 0xFFFFFFFFu;
      mbar_wait(&sm.s_full[2 * g + buf], static_cast<uint32_t>((i >> 1) & 1), &sm.abort);
      tc_fence_after();
      float s[RT];
      const auto scores = [&] {  // s_j + log2 vs_j of this key for the tile's rows
        const float2 ks2 = make_float2(ks, ks), lvs2 = make_float2(lvs, lvs);
        constexpr int GR = RT >= 24 ? 8 : RT;  // rows at a time (registers)
#pragma unroll
        for (int r0 = 0; r0 < RT; r0 += GR) {
          uint32_t hi[GR], lo[GR];
          tmem_ld2(tg + buf * 2 * RT + r0, tg + buf * 2 * RT + RT + r0, hi, lo);
#pragma unroll
          for (int r = 0; r < GR; r += 4) {
            const float4 c = *reinterpret_cast<const float4*>(sm.cq + r0 + r);
#pragma unroll
            for (int q = 0; q < 4; q += 2) {
              const float2 u = fma2(make_float2(__uint_as_float(lo[r + q]), __uint_as_float(lo[r + q + 1])),
                                    make_float2(0.03125f, 0.03125f),
                                    make_float2(__uint_as_float(hi[r + q]), __uint_as_float(hi[r + q + 1])));
              const float2 x = fma2(mul2(u, ks2), q ? make_float2(c.z, c.w) : make_float2(c.x, c.y), lvs2);
              s[r0 + r + q] = x.x;
              s[r0 + r + q + 1] = x.y;
            }
          }
        }
        if (masked) {
#pragma unroll
          for (int r = 0; r < RT; ++r) s[r] = (vis >> r) & 1u ? s[r] : -INFINITY;
        }
      };
      const auto exponents = [&] {  // s - M + kLift, and the largest of them
        float top = -INFINITY;
#pragma unroll
        for (int r = 0; r < RT; r += 4) {
          const float4 m = *reinterpret_cast<const float4*>(&sm.mneg[warp][r]);
          const float2 a = add2(make_float2(s[r], s[r + 1]), make_float2(m.x, m.y));
          const float2 c = add2(make_float2(s[r + 2], s[r + 3]), make_float2(m.z, m.w));
          s[r] = a.x, s[r + 1] = a.y, s[r + 2] = c.x, s[r + 3] = c.y;
          top = fmaxf(fmaxf(top, fmaxf(a.x, a.y)), fmaxf(c.x, c.y));
        }
        return top;
      };
      scores();
      if (masked) {
        // Value rows that not every query row sees: zero past the end (pages
        // hold anything there), and NaN codes of new slots taken out (a weight
        // of 0 would not clear them) and noted for the rows that see them.
        // (The products of tile i - 2 are waited for first: the stage's last fill is
        // then a past one, else this fill's parity would also name the one before.)
        const uint32_t vt = ring_v + vring.s * S::kTileB;
        if (i >= 2)
          mbar_wait(&sm.o_full[2 * g + buf], static_cast<uint32_t>(((i >> 1) - 1) & 1), &sm.abort);
        mbar_wait(&sm.full_v[vring.s], vring.par, &sm.abort);
        const uint32_t row0 = max(L - t0, 0), row1 = min(T - t0, kTile);
        for (uint32_t a = vt + row1 * HD + st * 16; a < vt + kTile * HD; a += kSoft * 16) st_shared_v4(a, 0, 0, 0, 0);
        for (uint32_t a = vt + row0 * HD + st * 16; a < vt + row1 * HD; a += kSoft * 16) {
          uint32_t w[4];
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                       : "r"(a)
                       : "memory");
          uint32_t hit = 0u;  // bytes 0x7F (but for the sign): the NaN codes
#pragma unroll
          for (int k = 0; k < 4; ++k) hit |= ((w[k] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
          if (!hit) continue;
          sm.any_nan = 1;
          const int row = static_cast<int>((a - vt) / HD);
          const int c = static_cast<int>(swz_off<HD>(row, (a - vt) % HD / 16) % HD) / 16;  // (its own inverse)
          const uint32_t m = seen(t0 + row);
#pragma unroll 1
          for (int k = 0; k < 16; ++k) {
            uint32_t byte;
            asm volatile("ld.shared.u8 %0, [%1];" : "=r"(byte) : "r"(a + k) : "memory");
            if ((byte & 0x7Fu) != 0x7Fu) continue;
            asm volatile("st.shared.u8 [%0], %1;" ::"r"(a + k), "r"(0) : "memory");
            const int d = c * 16 + k;
#pragma unroll 1
            for (int r = 0; r < RT; ++r)
              if ((m >> r) & 1u) atomicOr(&sm.nan[r][d / 32], 1u << (d % 32));
          }
        }
      }
      // ---- does any exponent pass the pieces' range?
      // (the first tile sets M)
      if (i == 0 || named_bar_any(bar, kSoft, exponents() > kTopExp + kLift || *static_cast<volatile int*>(&sm.abort) != 0)) {
        // raise M to each row's maximum (at 2^2); what is summed so far shrinks by alpha
        if (i && named_bar_any(bar + 1, kSoft, *static_cast<volatile int*>(&sm.abort) != 0)) {
          stopped = true;
          break;
        }
        if (i) scores();
        float alpha = 1.f;  // lane r: row r's
        const float m = warp_rows_reduce(s, -INFINITY, [](float a, float c) { return fmaxf(a, c); });
        if (lane < RT) sm.red[warp][lane] = m;
        named_bar(bar, kSoft);
        if (lane < RT) {
          const float mt = fmaxf(fmaxf(sm.red[4 * g][lane], sm.red[4 * g + 1][lane]),
                                 fmaxf(sm.red[4 * g + 2][lane], sm.red[4 * g + 3][lane]));
          const float mn = fmaxf(mrun, mt - kStartExp);
          alpha = exp2f(mrun - mn);
          sm.mneg[warp][lane] = kLift - mn;
          mrun = mn;
        }
        __syncwarp();
        if (i) {  // O and l shrink with it (O's pieces become one)
          mbar_wait(&sm.o_full[2 * g + ((i - 1) & 1)], static_cast<uint32_t>(((i - 1) >> 1) & 1), &sm.abort);
          tc_fence_after();
#pragma unroll
          for (int r = 0; r < RT; r += 8) {
            float o[8];
            o_rows(r, o);
            uint32_t w[8], z[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float a = __shfl_sync(0xffffffffu, alpha, r + k);
              l[r + k] *= a;
              w[k] = __float_as_uint(o[k] * a);
              z[k] = 0u;
            }
            tmem_st_x8(tg + 4 * RT + r, w);
            tmem_st_x8(tg + 5 * RT + r, z);
            tmem_st_x8(tg + 6 * RT + r, z);
          }
          tmem_st_wait();
        }
        exponents();
      }
      tc_fence_before();
      mbar_arrive(&sm.s_free[2 * g + buf]);
      // ---- weights and their sums; P: this key's row, hi | mid | lo
      uint32_t w[3][RT / 4];
#pragma unroll
      for (int r = 0; r < RT; r += 2) {
        const float2 e = make_float2(exp2f(s[r]), exp2f(s[r + 1]));
        const float2 sum = fma2(e, make_float2(ivs, ivs), make_float2(l[r], l[r + 1]));
        l[r] = sum.x, l[r + 1] = sum.y;
        // p = hi + mid / 16 + lo / 256, each the nearest e4m3 of what is left times 1, 16
        // and 256 (f is 16 p; fp16 holds every difference exactly), the last with the
        // slot's number added (zero plus half a step at the most stays zero)
        const uint32_t f = f16x2(e.x, e.y);
        const uint32_t u0 = f16x2_to_e4m3x2(f16x2_mul(f, 0x2C002C00u));            // / 16
        const uint32_t f1 = f16x2_fma(e4m3x2_to_f16x2(u0), 0xCC00CC00u, f);        // - 16 hi
        const uint32_t u1 = f16x2_to_e4m3x2(f1);
        const uint32_t f2 = f16x2_fma(e4m3x2_to_f16x2(u1), 0xBC00BC00u, f1);       // - mid
        const uint32_t u2 = f16x2_to_e4m3x2(f16x2_fma(f2, 0x4C004C00u, dither2));  // x 16
        w[0][r / 4] = r % 4 ? w[0][r / 4] | (u0 << 16) : u0;
        w[1][r / 4] = r % 4 ? w[1][r / 4] | (u1 << 16) : u1;
        w[2][r / 4] = r % 4 ? w[2][r / 4] | (u2 << 16) : u2;
      }
      // P of tile i - 2 has been read
      if (i >= 2) mbar_wait(&sm.o_full[2 * g + buf], static_cast<uint32_t>(((i >> 1) - 1) & 1), &sm.abort);
      const uint32_t pbuf = base + S::kP + (2 * g + buf) * S::kPB;
      const auto word = [&](int k) { return w[k / (RT / 4)][k % (RT / 4)]; };
#pragma unroll
      for (int c = 0; c < 3 * RT / 16; ++c)
        st_shared_v4(pbuf + p_off(st, c), word(4 * c), word(4 * c + 1), word(4 * c + 2), word(4 * c + 3));
      if constexpr (3 * RT % 16 != 0) {
        constexpr int c = 3 * RT / 16;
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(pbuf + p_off(st, c)), "r"(word(4 * c)),
                     "r"(word(4 * c + 1))
                     : "memory");
      }
      fence_async_smem();
      tc_fence_before();
      mbar_arrive(&sm.p_full[2 * g + buf]);
#pragma unroll
      for (int k = 0; k < NG; ++k) vring.next(NV);
    }
    // the next launch may start now: earlier, its blocks would take the places that
    // free first and lie unevenly over the SMs (batch 16 25.4 us against 23.6)
    grid_dep_launch();
    // ---- this CTA's row sums
    const float ls = warp_rows_reduce(l, 0.f, [](float a, float c) { return a + c; });
    // (and the last maxima have been read)
    const bool bad_page = named_bar_any(bar + 1, kSoft, new_page < 0 || new_page >= p.n_pages);
    const bool unfit = over || bad_page;  // zero rows
    if (tid == 0) {
      sm.unfit = unfit;
      if (unfit) set_status(p.status, over ? SPEC_DEV_KV_OVERFLOW : SPEC_DEV_BAD_PAGE);
    }
    if (lane < RT) sm.red[warp][lane] = ls;
    named_bar(bar, kSoft);
    float lt = 0.f;
    if (st < RT) {
      lt = (sm.red[4 * g][st] + sm.red[4 * g + 1][st]) + (sm.red[4 * g + 2][st] + sm.red[4 * g + 3][st]);
      sm.part[g][0][st] = mrun;
      sm.part[g][1][st] = lt;
    }
    if constexpr (NG > 1) {  // the groups' sums at a common M
      named_bar(7, NG * kSoft);
      float mine = 1.f;
      if (st < RT) {
        const float m = fmaxf(mrun, sm.part[g ^ 1][0][st]);
        mine = exp2f(mrun - m);
        lt = fmaf(mine, lt, exp2f(sm.part[g ^ 1][0][st] - m) * sm.part[g ^ 1][1][st]);
        mrun = m;
      }
      named_bar(7, NG * kSoft);  // (both have read the other's)
      if (st < RT) sm.part[g][0][st] = mine;
    }
    if (tid < RT) {
      sm.stat[0][tid] = C > 1 ? mrun : (lt == 0.f || unfit ? 0.f : 1.f / lt);  // alone: the factor of a row
      sm.stat[1][tid] = lt;
    }
    if (C == 1 || NG > 1) named_bar(bar, kSoft);
    // ---- O: dimension tid of every row, to the output, or to shared memory for the merge
    if (ntg && !stopped) {
      mbar_wait(&sm.o_full[2 * g + ((ntg - 1) & 1)], static_cast<uint32_t>(((ntg - 1) >> 1) & 1), &sm.abort);
      tc_fence_after();
    }
    float acc[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[r] = 0.f;
    if (ntg) {
#pragma unroll
      for (int r = 0; r < RT; r += 8) {
        float o[8];
        o_rows(r, o);
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[r + k] = o[k];
      }
    }
    if constexpr (NG > 1) {  // the second group's O to the first
      named_bar(7, NG * kSoft);  // (every MMA is done with the tiles that it lies over)
      const uint32_t mine = base + S::kO + st * 4;
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[r] *= sm.part[g][0][r];
      if (g && st < HD) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(mine + r * HD * 4), "f"(acc[r]) : "memory");
      }
      named_bar(7, NG * kSoft);
      if (!g && st < HD) {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          float x;
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(mine + r * HD * 4) : "memory");
          acc[r] += x;
        }
      }
    }
    if (sm.any_nan && tid < HD) {
#pragma unroll
      for (int r = 0; r < RT; ++r)
        if ((sm.nan[r][tid / 32] >> (tid % 32)) & 1u) acc[r] = __uint_as_float(0x7FC00000u);
    }
    if (tid < HD) {
      if (C > 1) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(base + S::kO + (r * HD + tid) * 4), "f"(acc[r]) : "memory");
      } else {
        uint16_t* o = p.o + tid;
#pragma unroll
        for (int r = 0; r < RT; r += 2) {
          const float2 f = *reinterpret_cast<const float2*>(&sm.stat[0][r]);
          const longlong2 at = *reinterpret_cast<const longlong2*>(&sm.out[r]);
          // (a factor of zero is a row that sees nothing, whatever its sum holds)
          const float x = f.x == 0.f ? 0.f : acc[r] * f.x, y = f.y == 0.f ? 0.f : acc[r + 1] * f.y;
          const uint32_t u = bf16x2(x, y);
          if (at.x >= 0) o[at.x] = static_cast<uint16_t>(u);
          if (at.y >= 0) o[at.y] = static_cast<uint16_t>(u >> 16);
          acc[r] = x - bf16lo(u);
          acc[r + 1] = y - bf16hi(u);
        }
        if constexpr (kLo) {
          o = p.o_lo + tid;
#pragma unroll
          for (int r = 0; r < RT; r += 2) {
            const longlong2 at = *reinterpret_cast<const longlong2*>(&sm.out[r]);
            const uint32_t u = bf16x2(acc[r], acc[r + 1]);
            if (at.x >= 0) o[at.x] = static_cast<uint16_t>(u);
            if (at.y >= 0) o[at.y] = static_cast<uint16_t>(u >> 16);
          }
        }
      }
    }
  }

  __syncwarp();
  if (C > 1) {
    const int rows = min(RT, R - rbase);
    // ---- merge: the cluster's CTAs share the (row, 4 dimensions) items
    __syncwarp();
    cluster_sync_all();
    const uint32_t stat = smem_u32(&sm.stat[0][0]);
    for (int e = rank * 32 * W::kAll + tid; e < rows * (HD / 4); e += C * 32 * W::kAll) {
      const int r = e / (HD / 4), d = e % (HD / 4) * 4;
      // every peer's reference, sum and four partial sums, all loads in flight together
      float mc[kMaxCluster], lc[kMaxCluster];
      float4 x[kMaxCluster];
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        mc[c] = kNoRef;
        lc[c] = 0.f;
        x[c] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c < C) {
          mc[c] = peer_f32(peer_addr(stat + r * 4, c));
          lc[c] = peer_f32(peer_addr(stat + (RT + r) * 4, c));
          x[c] = peer_f32x4(peer_addr(base + S::kO + (r * HD + d) * 4, c));
        }
      }
      float m = kNoRef, lt = 0.f;
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) m = fmaxf(m, mc[c]);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        if (c >= C) break;
        const float w = exp2f(mc[c] - m);  // 1 if no CTA has seen a slot: their sums are zero
        lt = fmaf(w, lc[c], lt);
        o.x = fmaf(w, x[c].x, o.x);
        o.y = fmaf(w, x[c].y, o.y);
        o.z = fmaf(w, x[c].z, o.z);
        o.w = fmaf(w, x[c].w, o.w);
      }
      const bool zero = lt == 0.f || sm.unfit;  // a row that sees nothing
      const float inv = 1.f / lt;
      o.x = zero ? 0.f : o.x * inv;
      o.y = zero ? 0.f : o.y * inv;
      o.z = zero ? 0.f : o.z * inv;
      o.w = zero ? 0.f : o.w * inv;
      const uint2 u = make_uint2(bf16x2(o.x, o.y), bf16x2(o.z, o.w));
      *reinterpret_cast<uint2*>(p.o + sm.out[r] + d) = u;
      if constexpr (kLo)
        *reinterpret_cast<uint2*>(p.o_lo + sm.out[r] + d) = make_uint2(
            bf16x2(o.x - bf16lo(u.x), o.y - bf16hi(u.x)), bf16x2(o.z - bf16lo(u.y), o.w - bf16hi(u.y)));
    }
    __syncwarp();
    cluster_sync_all();  // peers' shared memory stays until every CTA has read it
  }
  if (tid == 0 && sm.abort) set_status(p.status, SPEC_DEV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == W::kAll - 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmemCols);
  }
}

template <int HD, int RT, bool kLo, int NG>
cudaError_t launch_tile(const Kv8AttnParams& p, cudaStream_t stream) {
  using S = AttSmem<HD, RT, NG>;
  constexpr int kThreads = 32 * Warps<NG>::kAll, kSmem = NG > 1 ? kSmemCta : kSmemHalf;
  static PerDevice<AttSetup> setup;
  AttSetup s{};
  if (!setup.get([] { return att_setup(kv8_attention_kernel<HD, RT, kLo, NG>, kThreads, kSmem); }, &s))
    return cudaErrorInvalidDevice;
  if (s.err != cudaSuccess) return s.err;
  const int R = p.n * p.G, rtiles = (R + RT - 1) / RT;
  const int c = att_cluster(p, rtiles, s, 3 - NG);
  // Two groups a CTA where every CTA has an SM to itself and four tiles or more at
  // full capacity.  One group / two in us, 8 KV heads: 1 token at 131000 slots 51.4
  // / 44.6, 5 tokens 75.6 / 57.1, at 16000 16.8 / 15.0; with two tiles a CTA, 5
  // tokens at 2048 8.4 / 9.1, one KV head at 4000 8.0 / 9.1.  Short contexts in wide
  // tables take the two groups too: 2 x 5 tokens at 300 slots 7.2 us in a table of 320
  // slots, 8.4 in one of 32768; 1 token at 8000 9.1 and 8.2.
  if constexpr (NG == 1) {
    const int tiles = (p.max_pages * kPageSlots + kTile - 1) / kTile;
    if (static_cast<long long>(p.B) * p.Hkv * rtiles * c <= s.sms && tiles >= 4 * c)
      return launch_tile<HD, RT, kLo, 2>(p, stream);
  }
  const int fit = static_cast<int>((kSmem - S::bytes(0, 0)) / S::kTileB);
  // With two groups the counts are even: a stage then holds tiles of one group
  // only.  (A group that saw every other fill of a stage could take a past fill,
  // whose parity is the same, for the one that it waits for.)
  constexpr int kEven = ~(NG - 1);
  const int nk = std::min(fit / 2, S::kMaxStages) & kEven, nv = std::min(fit - nk, S::kMaxStages) & kEven;
  const uint32_t bytes = std::max<uint32_t>(S::bytes(nk, nv), NG > 1 ? kSmemAlone : 0);
  AttMaps maps;
  const long long rows = static_cast<long long>(p.n_pages) * p.Hkv * kPageSlots;
  if (!page_map(&maps.k, p.kc, rows, HD) || !page_map(&maps.v, p.vc, rows, HD)) return cudaErrorInvalidValue;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = att_config(dim3(rtiles * c, p.Hkv, p.B), kThreads, bytes, stream, attr, c);
  return cudaLaunchKernelEx(&cfg, kv8_attention_kernel<HD, RT, kLo, NG>, maps, p, c, nk, nv, (3 - NG) * s.sms);
}

template <int HD, bool kLo>
cudaError_t launch_rows(const Kv8AttnParams& p, cudaStream_t stream) {
  // the row tile that leaves the fewest rows empty, the larger of equal ones
  const int R = p.n * p.G;
  int best = 32;
  for (int rt = 24; rt >= 8; rt -= 8)
    if ((R + rt - 1) / rt * rt < (R + best - 1) / best * best) best = rt;
  switch (best) {
    case 8: return launch_tile<HD, 8, kLo, 1>(p, stream);
    case 16: return launch_tile<HD, 16, kLo, 1>(p, stream);
    case 24: return launch_tile<HD, 24, kLo, 1>(p, stream);
    default: return launch_tile<HD, 32, kLo, 1>(p, stream);
  }
}

}  // namespace

cudaError_t launch_kv8_attention(const Kv8AttnParams& p, cudaStream_t stream) {
  const long long R = static_cast<long long>(p.n) * p.G;
  const long long tiles = (static_cast<long long>(p.max_pages) * kPageSlots + kTile - 1) / kTile;
  if (R > kWideRows && (R + 127) / 128 * p.Hkv * p.B * tiles >= kWideWork) return launch_kv8_attention_wide(p, stream);
  if (p.o_lo) return p.hd == 128 ? launch_rows<128, true>(p, stream) : launch_rows<64, true>(p, stream);
  return p.hd == 128 ? launch_rows<128, false>(p, stream) : launch_rows<64, false>(p, stream);
}

}  // namespace spec
