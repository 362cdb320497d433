// Attention over the 8-bit paged KV cache for many query rows (prefill chunks,
// large trees): the same formulas as the kernel for few rows, but a tile is
// 128 query rows x 128 keys with a row per softmax thread.
//   S [128 rows][64 keys]   = (Q hi + Q lo) x K^T   kind::f8f6f4, K as stored, hi e4m3, lo e5m2
//   O [128 rows][hd dims]  += P x V                 kind::f16, P from TMEM
// With few rows a weight can afford three e4m3 pieces, since there the tile of
// values is what costs.  With many the pieces cost, and it is cheaper to widen
// the values once a tile, e4m3 to fp16 (exact), for all 128 rows: four warps do
// that, straight from global memory into a swizzled tile.  A weight is then one
// fp16, with the 11 bits that the three pieces hold (why so few: there), rounded to
// nearest: where the row's largest is 2^4 or more, the smallest step is 2^-28 of it.
//   p'_j = 2^(s_j + log2 vs_j - M),  l = sum over blocks of (sum of p'_j) / vs
// A block's 16 keys are 16 neighbouring columns, so its two scales enter as the
// two constants of one multiply-add per score.  M is a row's own (one thread
// knows it) and is raised only when a weight would pass 2^15; the row's warp then
// scales its rows of O.  P takes the place of the scores it came from.
//
// A CTA has an SM to itself.  Two softmax groups of four warps take the even and
// the odd tiles of its run over the keys, each with an M, l and O of its own and
// a warp that issues its MMAs, half a turn apart; a group has two score buffers of
// half a tile, so the tensor cores work on the next half during its softmax.
// (Two CTAs an SM of one group each: 2700 cycles a tile and SM, 128-register
// threads could not be had; two groups with a row tile each, of 256 rows: 3000,
// and twice the prologue and merge; so: 2400.)  At the end the groups' sums are put
// together in shared memory, and those of the cluster's CTAs, whose runs share a
// row tile, through distributed shared memory.
//
// What bounds it: the latency of a group's chain (scores, TMEM load, largest,
// weights, TMEM store, products); of the SM's cycles the tensor pipe is busy 41%,
// the issue slots 38%, and nothing else more.  32 heads on 8, head dim 128: 128
// tokens at 4000 slots 21.9 us (4.3 us of products at the measured bf16 rate), of
// which ~10 are prologue, merge and a launch; at 131000 slots 322 us, 0.43 of that
// rate; four sequences of 128 at 700 16.7 us; head dim 64 at 1900 19.3 us.
#include "kv8_attn.cuh"

namespace spec {
namespace {

constexpr int kRows = 128;               // query rows of a tile
constexpr int kGroups = 2;               // softmax groups of four warps, a thread per row: even and odd tiles
constexpr int kSoftW = kGroups * kRows;  // softmax threads
constexpr int kHalf = kTile / 2;         // keys of a score buffer (a group has two)
constexpr int kWiden = 128;              // threads that widen the values
constexpr int kWLoadK = 12;              // the warp that loads K,
constexpr int kWIssue = 13;              // ... and the first of the issuing ones
constexpr int kWideThreads = 32 * (kWIssue + kGroups);
constexpr float kWTop = 15.f;   // a weight stays below 2^15: fp16's largest is 2^16
constexpr float kWStart = 4.f;  // exponent of a row's maximum where M is set

// D[tmem] (+)= A[tmem] * B[smem] of fp16 operands, issued by one thread.
SPEC_DEVINL void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
SPEC_DEVINL void tmem_ld_x32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
template <int N>
SPEC_DEVINL void ld_pin(uint32_t (&a)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(a[i]));  // no use moves above the wait before it
}
template <int N>
SPEC_DEVINL void ld_wait(uint32_t (&a)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  ld_pin(a);
}
// Two fp32 values to two e5m2 codes (nearest), `a` in the low byte.
SPEC_DEVINL uint32_t e5m2x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
constexpr uint32_t kIdescE5m2A = 1u << 7;  // instruction descriptor: operand A is e5m2
SPEC_DEVINL float2 peer_f32x2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a));
  return v;
}
SPEC_DEVINL uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
SPEC_DEVINL float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

template <int HD>
struct WideSmem {
  static constexpr int kStages = 4;  // of K
  static constexpr uint32_t kTileB = kTile * HD;
  static constexpr uint32_t kQ = 0;  // [hi | lo][rows][HD] e4m3
  static constexpr uint32_t kK = kQ + 2 * kRows * HD;
  static constexpr uint32_t kVB = 2 * kTileB;            // a group's value tile: [HD / 64][keys][64] fp16
  static constexpr uint32_t kV = kK + kStages * kTileB;
  static constexpr uint32_t kMisc = kV + 2 * kVB;
  struct Misc {
    uint64_t full_k[kStages], empty_k[kStages];
    uint64_t c_full[kGroups], v_full[kGroups], drain[kGroups], second;
    uint64_t s_full[kGroups][2], p_full[kGroups][2], o_full[kGroups][2];  // of a tile's halves
    // of a tile's blocks: the keys' scale, log2 of the values'
    alignas(16) float2 scale[kGroups][kTile / kKv8Block];
    uint64_t anc[kRows];
    float cq[kRows];                // score factor of a row: 2^k scale log2(e)
    float2 part[kGroups][kRows];    // a group's M and sum per row,
    alignas(8) float2 stat[kRows];  // ... and the CTA's
    uint32_t nan[kRows][HD / 32];   // outputs that a NaN value code reaches
    alignas(16) int len[kSortSeqs];
    uint32_t tmem;
    alignas(8) int pages[16];
    int seq, seq_len, unit, unfit, abort, any_nan;
  };
  // partial sums [rows][HD] fp32 and after them the merge's weights [cluster][rows],
  // over the tiles once every MMA is done
  static constexpr uint32_t kO = 0, kW = kRows * HD * 4;
  static constexpr uint32_t kBytes = std::max<uint32_t>(kMisc + sizeof(Misc), kSmemAlone);
  static_assert(kW + kMaxCluster * kRows * 4 <= kMisc, "they lie within the tiles");
  static_assert(kBytes <= kSmemCta && kMisc % 16 == 0, "");
  static_assert(kK % 1024 == 0 && kV % 1024 == 0, "swizzled tiles lie on their own span's boundaries");
  static constexpr uint32_t kTmemCols = 512;  // a group's S (then P) 128 each, O HD each
};

template <int HD, bool kLo>
__global__ void __launch_bounds__(kWideThreads, 1)
    kv8_attention_wide_kernel(const __grid_constant__ CUtensorMap kmap, const Kv8AttnParams p, const int csize,
                              const int share) {
  using S = WideSmem<HD>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t base = smem_u32(smem_raw);
  auto& sm = *reinterpret_cast<typename S::Misc*>(smem_raw + S::kMisc);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x % csize, rtile = blockIdx.x / csize, h = blockIdx.y;
  const int G = p.G, R = p.n * G, rbase = rtile * kRows;

  if (tid == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&sm.full_k[i], 1);
      mbar_init(&sm.empty_k[i], 1);
    }
    for (int g = 0; g < kGroups; ++g) {
      mbar_init(&sm.c_full[g], 1);
      mbar_init(&sm.v_full[g], kWiden);
      mbar_init(&sm.drain[g], 1);
      for (int u = 0; u < 2; ++u) {
        mbar_init(&sm.s_full[g][u], 1);
        mbar_init(&sm.p_full[g][u], kRows);
        mbar_init(&sm.o_full[g][u], 1);
      }
    }
    mbar_init(&sm.second, 1);
    fence_mbar_init();
    sm.abort = 0;
    sm.any_nan = 0;
  }
  if (tid == 32 * kWLoadK) prefetch_tmap(&kmap);
  if (warp == kWIssue) {
    tmem_alloc(&sm.tmem, S::kTmemCols);
    tmem_relinquish();
    tc_fence_before();
  }
  if (tid < kRows)
#pragma unroll
    for (int c = 0; c < HD / 32; ++c) sm.nan[tid][c] = 0u;
  __syncthreads();  // barriers and TMEM set up
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  grid_dep_wait();

  const int cap = p.max_pages * kPageSlots;
  const int slots = csize > 1 ? share / (p.Hkv * (gridDim.x / csize)) : 0;  // CTAs of the GPU per KV head and row tile
  const AttPick pick = att_pick(p, csize > 1, slots, sm);
  const int b = pick.b, L = pick.sorted ? sm.seq_len : p.base[b];
  // ---- the query rows: row r = token r / G, head h * G + r % G; HD / 8 lanes
  // each, so that a warp reads whole rows
  constexpr int LPR = HD / 8, RPW = 32 / LPR;  // lanes of a row, rows of a warp at a time
  constexpr int RP = kSoftW / 32 * RPW;        // ... of the softmax warps
  constexpr int NQ = kRows / RP;               // a lane's loads, all under way together
  const int ql = lane % LPR, q0 = warp * RPW + lane / LPR;
  const auto row_at = [&](int r, long long ld) {  // where row r (of the tile) starts
    const int rr = rbase + r, tok = rr / G;
    return (static_cast<long long>(b) * p.n + tok) * ld + (h * G + rr - tok * G) * HD;
  };
  uint4 qw[NQ];
  if (tid < kSoftW) {
#pragma unroll
    for (int k = 0; k < NQ; ++k) {
      const int r = k * RP + q0;
      qw[k] = make_uint4(0, 0, 0, 0);
      if (rbase + r < R) qw[k] = *reinterpret_cast<const uint4*>(p.q + row_at(r, p.q_ld) + ql * 8);
    }
    if (p.anc && tid < kRows) {
      const int rr = min(rbase + tid, R - 1);
      sm.anc[tid] = p.anc[static_cast<long long>(b) * p.n + rr / G] & (p.n < 64 ? (1ull << p.n) - 1 : ~0ull);
    }
  }

  const bool over = L < 0 || L > cap - p.n;
  const int T = over ? 0 : L + p.n;  // slots [0, T)
  const int tiles = (T + kTile - 1) / kTile;
  int C = 1, i0 = 0, nt = tiles;  // CTAs that share the tiles; this one's
  if (csize > 1) {
    const int unit = pick.sorted ? sm.unit : max(kMinTiles, p.B > 1 ? 0 : (tiles + slots - 1) / max(slots, 1));
    C = min(csize, max(1, (tiles + unit - 1) / unit));
    if (rank >= C) {  // (its peers' barriers go on without it)
      if (warp == kWIssue) tmem_dealloc(tmem, S::kTmemCols);
      return;
    }
    i0 = tiles * rank / C;  // (tiles * C <= 2^13 * 2^4)
    nt = tiles * (rank + 1) / C - i0;
  }
  const int32_t* table = p.table + static_cast<long long>(b) * p.max_pages;
  const auto page_of = [&](int t) {  // the page of slot t, clamped into the pool
    const int pg = table[min(t / kPageSlots, p.max_pages - 1)];
    return min(max(pg, 0), p.n_pages - 1);
  };

  // ---- ... as pieces, 2^k (hi + lo).  What hi (4 bits) leaves of an element's 8 bits
  // is a whole number of its last bit, 8 at most, which lo (3 bits) holds: exact for
  // elements down to 2^-13 of the row's largest (at 2^7 or more), below off by e5m2's
  // rounding of 2^-10 (half of hi's smallest step) or less, 2^-21 of the largest.
  if (tid < kSoftW) {
    // the row's largest magnitude, as bf16 bits: those order as integers, with
    // infinities and NaN (which make the row NaN) above all finite values
    uint32_t mx[NQ];
#pragma unroll
    for (int k = 0; k < NQ; ++k)
      mx[k] = max_u16x2(max_u16x2(qw[k].x & 0x7FFF7FFFu, qw[k].y & 0x7FFF7FFFu),
                        max_u16x2(qw[k].z & 0x7FFF7FFFu, qw[k].w & 0x7FFF7FFFu));
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1)
#pragma unroll
      for (int k = 0; k < NQ; ++k) mx[k] = max_u16x2(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], o));
#pragma unroll
    for (int k = 0; k < NQ; ++k) {
      const int r = k * RP + q0;
      const uint32_t v[4] = {qw[k].x, qw[k].y, qw[k].z, qw[k].w};
      const int top = static_cast<int>(max(mx[k] & 0xFFFFu, mx[k] >> 16) >> 7);  // its exponent
      // 2^-k brings the largest element into [128, 256) (k at least -100: a row
      // of smaller elements scores zero to fp32's last bit anyway)
      const int k2 = top == 255 ? 0 : max(top - 127 - 7, -100);
      const float down = __uint_as_float(top == 255 ? 0x7FC00000u : static_cast<uint32_t>(127 - k2) << 23);
      uint32_t hi[2], lo[2];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = bf16lo(v[j]) * down, d = bf16hi(v[j]) * down;
        const uint32_t w = e4m3x2(a, d);
        const float2 f = e4m3x2_to_f32(w);
        const uint32_t u = e5m2x2(a - f.x, d - f.y);
        hi[j / 2] = j & 1 ? hi[j / 2] | (w << 16) : w;
        lo[j / 2] = j & 1 ? lo[j / 2] | (u << 16) : u;
      }
      const uint32_t to = base + S::kQ + swz_off<HD>(r, ql / 2) + ql % 2 * 8;
      asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(to), "r"(hi[0]), "r"(hi[1]) : "memory");
      asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(to + kRows * HD), "r"(lo[0]), "r"(lo[1]) : "memory");
      if (ql == 0) sm.cq[r] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + k2) << 23);
    }
    fence_async_smem();
  }
  if (warp != kWLoadK) named_bar(3, kWideThreads - 32);  // q and the row arrays are ready
  tc_fence_after();

  if (warp == kWLoadK) {
    // ------------------------------------------- TMA: the tiles of K
    const int entries = (T + kPageSlots - 1) / kPageSlots - 2 * i0;  // pages from this CTA's first slot on
    const auto page_at = [&](int e) {
      if (e >= entries) return 0;
      const int pg = table[min((i0 * kTile + e * kPageSlots) / kPageSlots, p.max_pages - 1)];
      if (pg < 0 || pg >= p.n_pages) set_status(p.status, SPEC_DEV_BAD_PAGE);
      return min(max(pg, 0), p.n_pages - 1);
    };
    att_load_tiles<HD>(&kmap, sm.full_k, sm.empty_k, sm.pages, base + S::kK, S::kStages, nt, entries, p.Hkv, h,
                       &sm.abort, page_at);
  } else if (warp >= kWIssue) {
    // ------------------------------------------- MMAs of a group
    const int g = warp - kWIssue;
    if (lane == 0) {
      bool ok = true;
      const uint64_t aq = sdesc_rows<HD>(base + S::kQ, 16), bk0 = sdesc_rows<HD>(base + S::kK, 16);
      const uint64_t bv = sdesc_rows<128>(base + S::kV + g * S::kVB, kTile * 128);
      const uint32_t ts = tmem + g * kTile, to = tmem + kGroups * kTile + g * HD;
      // The second group starts behind the first: its MMAs run beside the other's
      // softmax, and the other way round.
      if (g && nt > 1) ok = mbar_wait(&sm.second, 0, &sm.abort);
      // Scores of half u of the group's j'th tile; they take the place of the
      // weights of the half before the last, whose products must be done.
      const auto issue_scores = [&](int j, int u) {
        const int i = kGroups * j + g;
        ok = (j == 0 || mbar_wait(&sm.o_full[g][u], static_cast<uint32_t>((j - 1) & 1), &sm.abort)) &&
             (u || mbar_wait(&sm.full_k[i % S::kStages], static_cast<uint32_t>((i / S::kStages) & 1), &sm.abort));
        if (!ok) return;
        tc_fence_after();
        const uint64_t bk = bk0 + static_cast<uint32_t>(i % S::kStages * S::kTileB + u * kHalf * HD >> 4);
#pragma unroll
        for (int kk = 0; kk < HD / 32; ++kk)
#pragma unroll
          for (int piece = 0; piece < 2; ++piece)
            umma_e4m3(ts + u * kHalf, aq + piece * (kRows * HD >> 4) + kk * 2, bk + kk * 2,
                      idesc_e4m3(kRows, kHalf, false, false) | (piece ? kIdescE5m2A : 0u), kk + piece > 0 ? 1u : 0u);
        umma_commit(&sm.s_full[g][u]);
        if (u) umma_commit(&sm.empty_k[i % S::kStages]);
      };
      const int ntg = (nt + 1 - g) / 2;
      if (ntg && ok) issue_scores(0, 0);
      for (int t = 0; t < 2 * ntg && ok; ++t) {
        const int j = t >> 1, u = t & 1;
        if (t + 1 < 2 * ntg) issue_scores((t + 1) >> 1, (t + 1) & 1);
        if (!ok) break;
        ok = mbar_wait(&sm.v_full[g], static_cast<uint32_t>(j & 1), &sm.abort) &&
             mbar_wait(&sm.p_full[g][u], static_cast<uint32_t>(j & 1), &sm.abort);
        if (!ok) break;
        if (g == 0 && t == 0) mbar_arrive(&sm.second);
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kHalf / 16; ++kk)  // (the same descriptor bits name fp16 in this kind)
          umma_f16_ts(to, ts + u * kHalf + kk * 8, bv + (u * kHalf + kk * 16) * (128 >> 4),
                      idesc_e4m3(kRows, HD, false, true), t + kk > 0 ? 1u : 0u);
        umma_commit(&sm.o_full[g][u]);
      }
      if (!ok) {  // MMAs in flight end before TMEM and shared memory go
        int none = 0;
        umma_commit(&sm.drain[g]);
        mbar_wait(&sm.drain[g], 0, &none);
      }
    }
    __syncwarp();
  } else if (warp >= kSoftW / 32) {
    // ------------------------------------------- V: e4m3 codes to an fp16 tile
    constexpr int TR = HD / 16;      // threads per key row
    constexpr int RV = kWiden / TR;  // rows at a time
    constexpr int IT = kTile / RV;
    const int w = tid - kSoftW, ch = w % TR, r0 = w / TR;
    const uint8_t* vc = p.vc + ch * 16;
    uint4 x[IT];
    const auto load = [&](int i) {
      const int t0 = (i0 + i) * kTile;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const long long page = page_of(t0 + half * kPageSlots);
#pragma unroll
        for (int k = half * IT / 2; k < (half + 1) * IT / 2; ++k) {
          const int row = r0 + k * RV;
          x[k] = make_uint4(0, 0, 0, 0);  // past the end: zero
          if (t0 + row < T)
            x[k] = __ldcs(
                reinterpret_cast<const uint4*>(vc + ((page * p.Hkv + h) * kPageSlots + row % kPageSlots) * HD));
        }
      }
    };
    const auto seen = [&](int r, int k) {  // row r of the tile sees new slot k
      return p.anc ? k < 64 && ((sm.anc[r] >> k) & 1ull) != 0 : rbase + r >= k * G;
    };
    // lane k of the first warp: the scales of the tile's block k
    float2 sc = make_float2(1.f, 1.f);
    const auto load_scale = [&](int i) {
      const int t = (i0 + i) * kTile + lane * kKv8Block;
      sc = make_float2(1.f, 1.f);
      if (t >= T) return;
      const long long at = (static_cast<long long>(page_of(t)) * p.Hkv + h) * kKv8Sub + t % kPageSlots / kKv8Block;
      sc = make_float2(p.ks[at], p.vs[at]);
    };
    const bool scales = w < kTile / kKv8Block;
    if (nt) {
      if (scales) load_scale(0);
      load(0);
    }
    for (int i = 0; i < nt; ++i) {
      // the group's last products have read its tile and scales (and its softmax, before them)
      const bool ok = i < 2 || mbar_wait(&sm.o_full[i & 1][1], static_cast<uint32_t>(((i >> 1) - 1) & 1), &sm.abort);
      if (__any_sync(0xffffffffu, !ok)) break;
      if (w < 32) {
        if (scales)
          sm.scale[i & 1][lane] =
              make_float2(sc.x, static_cast<float>(static_cast<int>(__float_as_uint(sc.y) >> 23) - 127));
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.c_full[i & 1]);
      }
      const int t0 = (i0 + i) * kTile;
      if (t0 + kTile > L) {
        // NaN codes of slots that not every row sees are taken out (a weight of 0
        // would not clear them) and noted for the rows that see them.
#pragma unroll
        for (int k = 0; k < IT; ++k) {
          const int t = t0 + r0 + k * RV;
          if (t < L) continue;
          uint32_t c[4] = {x[k].x, x[k].y, x[k].z, x[k].w}, hit = 0u;
#pragma unroll
          for (int q = 0; q < 4; ++q) hit |= ((c[q] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
          if (!hit) continue;
          sm.any_nan = 1;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
#pragma unroll 1
            for (int e = 0; e < 4; ++e) {
              if (((c[q] >> (8 * e)) & 0x7Fu) != 0x7Fu) continue;
              c[q] &= ~(0xFFu << (8 * e));
              const int d = ch * 16 + q * 4 + e;
#pragma unroll 1
              for (int r = 0; r < kRows; ++r)
                if (seen(r, t - L)) atomicOr(&sm.nan[r][d / 32], 1u << (d % 32));
            }
          }
          x[k] = make_uint4(c[0], c[1], c[2], c[3]);
        }
      }
#pragma unroll
      for (int k = 0; k < IT; ++k) {
        const int row = r0 + k * RV;
        const uint32_t c[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
        uint32_t f[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          f[2 * q] = e4m3x2_to_f16x2(c[q]);
          f[2 * q + 1] = e4m3x2_to_f16x2(c[q] >> 16);
        }
        const uint32_t span = base + S::kV + (i & 1) * S::kVB + ch / 4 * (kTile * 128);
        // (the lanes of the second span write their second half first: other banks)
        const int flip = ch / 4;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int g = j ^ flip;
          st_shared_v4(span + swz_off<128>(row, ch % 4 * 2 + g), g ? f[4] : f[0], g ? f[5] : f[1], g ? f[6] : f[2],
                       g ? f[7] : f[3]);
        }
      }
      fence_async_smem();
      mbar_arrive(&sm.v_full[i & 1]);
      if (i + 1 < nt) {
        if (scales) load_scale(i + 1);
        load(i + 1);
      }
    }
  } else {
    // ------------------------------------------- softmax: thread = row
    const int g = warp / 4, row = tid % kRows;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp % 4 * 32) << 16);
    const uint32_t ts = lanes + g * kTile, to = lanes + kGroups * kTile + g * HD;
    const int ntg = (nt + 1 - g) / 2;  // the group's tiles
    const int tok = min(rbase + row, R - 1) / G;
    const float cq = sm.cq[row];
    float M = kNoRef, l = 0.f;
    // the columns of 16 slots from t on that the row sees
    const auto seen16 = [&](int t) {
      if (!p.anc) {
        const int lim = L + tok + 1 - t;
        return lim <= 0 ? 0u : (lim >= 16 ? 0xFFFFu : (1u << lim) - 1u);
      }
      const unsigned long long am = sm.anc[row];
      const int off = t - L;
      if (off <= -16) return 0xFFFFu;
      if (off < 0) return ((1u << -off) - 1u) | static_cast<uint32_t>((am << -off) & 0xFFFFull);
      return off < 64 ? static_cast<uint32_t>(am >> off) & 0xFFFFu : 0u;
    };
    bool stopped = false;
    for (int i = 0; i < 2 * ntg; ++i) {  // half u of the group's j'th tile
      const int j = i >> 1, u = i & 1;
      const int t0 = (i0 + kGroups * j + g) * kTile + u * kHalf;
      const bool masked = t0 + kHalf > L;  // it holds slots that some row does not see
      const uint32_t tsu = ts + u * kHalf;
      const bool ok = mbar_wait(&sm.c_full[g], static_cast<uint32_t>(j & 1), &sm.abort) &&
                      mbar_wait(&sm.s_full[g][u], static_cast<uint32_t>(j & 1), &sm.abort);
      if (__any_sync(0xffffffffu, !ok)) {
        stopped = true;
        break;
      }
      tc_fence_after();
      // (never zero: a masked score of -inf stays that)
      const auto factor = [&](float ks) { return fmaxf(ks * cq, 1.17549435e-38f); };
      const float4* const scale = reinterpret_cast<const float4*>(sm.scale[g] + u * (kHalf / kKv8Block));
      uint32_t x[2][32];
      tmem_ld_x32(tsu, x[0]);
      tmem_ld_x32(tsu + 32, x[1]);
      ld_wait(x[0]);
      ld_pin(x[1]);
      if (masked) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int q = 0; q < 32; q += 16) {
            const uint32_t vis = seen16(t0 + 32 * k + q);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[k][q + e] = (vis >> e) & 1u ? x[k][q + e] : 0xFF800000u;
          }
      }
      // ---- the row's largest exponent.  (Eight chains: with two warps a scheduler,
      // a chain's latency is what a row costs.)
      float top = -INFINITY;
      {
        float m[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) m[k] = -INFINITY;
#pragma unroll
        for (int e = 0; e < 8; e += 2)
#pragma unroll
          for (int k = 0; k < 8; ++k)
            m[k] = max3(m[k], __uint_as_float(x[k / 4][k % 4 * 8 + e]), __uint_as_float(x[k / 4][k % 4 * 8 + e + 1]));
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float4 sc = scale[k];
          top = max3(top, fmaf(fmaxf(m[4 * k], m[4 * k + 1]), factor(sc.x), sc.y),
                     fmaf(fmaxf(m[4 * k + 2], m[4 * k + 3]), factor(sc.z), sc.w));
        }
      }
      // ---- raise M (at first: set it); O and l shrink with it
      if (__any_sync(0xffffffffu, i == 0 || top - M > kWTop)) {
        const float mn = fmaxf(M, top - kWStart), alpha = exp2f(M - mn);
        M = mn;
        l *= alpha;
        if (i) {  // the products so far must be in O
          mbar_wait(&sm.o_full[g][u ^ 1], static_cast<uint32_t>(((i - 1) >> 1) & 1), &sm.abort);
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < HD; c += 16) {
            uint32_t o[16];
            tmem_ld_x16(to + c, o);
            ld_wait(o);
#pragma unroll
            for (int q = 0; q < 16; q += 8) {
              uint32_t z[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) z[e] = __float_as_uint(__uint_as_float(o[q + e]) * alpha);
              tmem_st_x8(to + c + q, z);
            }
          }
          tmem_st_wait();
        }
      }
      // ---- weights, their sums, and P over the scores
#pragma unroll
      for (int h2 = 0; h2 < 2; ++h2) {
        const float4 sc = scale[h2];
        const float a[2] = {factor(sc.x), factor(sc.z)}, lv[2] = {sc.y, sc.w};
        float2 sum[2][2];
        uint32_t w[2][8];
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float2 s2 = make_float2(__uint_as_float(x[h2][k * 16 + e]), __uint_as_float(x[h2][k * 16 + e + 1]));
            const float2 y = fma2(s2, make_float2(a[k], a[k]), make_float2(lv[k] - M, lv[k] - M));
            const float2 p2 = make_float2(exp2f(y.x), exp2f(y.y));
            sum[k][e / 2 % 2] = e < 4 ? p2 : add2(sum[k][e / 2 % 2], p2);
            w[k][e / 2] = f16x2(p2.x, p2.y);
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float2 t = add2(sum[k][0], sum[k][1]);
          l = fmaf(t.x + t.y, __uint_as_float(static_cast<uint32_t>(127 - static_cast<int>(lv[k])) << 23), l);
          tmem_st_x8(tsu + h2 * 16 + k * 8, w[k]);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&sm.p_full[g][u]);
    }
    grid_dep_launch();
    // the pages that the new slots lie on
    const int new_pages = over ? 0 : (T - 1) / kPageSlots - L / kPageSlots + 1;
    bool bad = false;
    if (lane < new_pages) {
      const int pg = table[L / kPageSlots + lane];
      bad = pg < 0 || pg >= p.n_pages;
    }
    const bool unfit = over || __any_sync(0xffffffffu, bad);  // zero rows
    if (tid == 0) {
      sm.unfit = unfit;
      if (unfit) set_status(p.status, over ? SPEC_DEV_KV_OVERFLOW : SPEC_DEV_BAD_PAGE);
    }
    if (ntg && !stopped) {
      mbar_wait(&sm.o_full[g][1], static_cast<uint32_t>((ntg - 1) & 1), &sm.abort);
      mbar_wait(&sm.v_full[g], static_cast<uint32_t>((ntg - 1) & 1), &sm.abort);  // (sm.nan)
      tc_fence_after();
    }
    // ---- the two groups' sums of a row, put together: each hands the other half of
    // its dimensions and ends with the other half
    sm.part[g][row] = make_float2(M, l);
    named_bar(4, kSoftW);  // (and the MMAs are done with the tiles, which the sums replace)
    const float2 other = sm.part[g ^ 1][row];
    const float m = fmaxf(M, other.x);
    const float w = exp2f(M - m), lt = fmaf(exp2f(other.x - m), other.y, w * l);
    const bool nans = sm.any_nan != 0, live = rbase + row < R;
    const long long at = live ? row_at(row, p.o_ld) : 0;
    const float inv = lt == 0.f || unfit ? 0.f : 1.f / lt;
    if (g == 0) sm.stat[row] = make_float2(m, lt);
    const auto o_cols = [&](int c, uint32_t (&o)[32]) {  // dimensions c .. c + 31, at the common M
#pragma unroll
      for (int j = 0; j < 32; ++j) o[j] = 0u;
      if (ntg) {
        tmem_ld_x32(to + c, o);
        ld_wait(o);
      }
#pragma unroll
      for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * w);
    };
    // (chunks of a row in another order per row: other banks)
    const auto chunk = [&](int c) { return base + S::kO + row * HD * 4 + ((c ^ (row & 7)) << 4); };
#pragma unroll
    for (int c = (g ^ 1) * (HD / 2), e = c + HD / 2; c < e; c += 32) {
      uint32_t o[32];
      o_cols(c, o);
#pragma unroll
      for (int q = 0; q < 8; ++q) st_shared_v4(chunk(c / 4 + q), o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
    }
    named_bar(4, kSoftW);
#pragma unroll
    for (int c = g * (HD / 2), e = c + HD / 2; c < e; c += 32) {
      uint32_t o[32];
      o_cols(c, o);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        float4 x;
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                     : "r"(chunk(c / 4 + q))
                     : "memory");
        const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) o[4 * q + j] = __float_as_uint(__uint_as_float(o[4 * q + j]) + y[j]);
      }
      if (nans) {
        const uint32_t bits = sm.nan[row][c / 32];
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if ((bits >> j) & 1u) o[j] = 0x7FC00000u;
      }
      if (C > 1) {
#pragma unroll
        for (int q = 0; q < 8; ++q) st_shared_v4(chunk(c / 4 + q), o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
      } else if (live) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t y[4], z[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // (a factor of zero is a row that sees nothing, whatever its sum holds)
            const float x0 = inv == 0.f ? 0.f : __uint_as_float(o[8 * q + 2 * j]) * inv;
            const float x1 = inv == 0.f ? 0.f : __uint_as_float(o[8 * q + 2 * j + 1]) * inv;
            y[j] = bf16x2(x0, x1);
            z[j] = bf16x2(x0 - bf16lo(y[j]), x1 - bf16hi(y[j]));
          }
          *reinterpret_cast<uint4*>(p.o + at + c + 8 * q) = make_uint4(y[0], y[1], y[2], y[3]);
          if constexpr (kLo) *reinterpret_cast<uint4*>(p.o_lo + at + c + 8 * q) = make_uint4(z[0], z[1], z[2], z[3]);
        }
      }
    }
  }

  __syncwarp();
  if (C > 1) {
    cluster_sync_all();
    // ---- merge: each row's weight of every CTA, 2^(M - max M) / sum
    float* const wt = reinterpret_cast<float*>(smem_raw + S::kW);
    if (tid < kRows) {
      const uint32_t stat = smem_u32(&sm.stat[tid]);
      float2 ml[kMaxCluster];  // (all loads under way together)
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) ml[c] = c < C ? peer_f32x2(peer_addr(stat, c)) : make_float2(kNoRef, 0.f);
      float m = kNoRef, lt = 0.f;
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) m = fmaxf(m, ml[c].x);
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        ml[c].x = exp2f(ml[c].x - m);  // 1 if no CTA has seen a slot: their sums are zero
        lt = fmaf(ml[c].x, ml[c].y, lt);
      }
      const bool zero = lt == 0.f || sm.unfit;  // a row that sees nothing
      const float inv = 1.f / lt;
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c)
        if (c < C) wt[c * kRows + tid] = zero ? -1.f : ml[c].x * inv;
    }
    __syncthreads();
    // ... then the cluster's CTAs share the (row, 4 dimensions) items
    const int rows = min(kRows, R - rbase);
    for (int e = rank * kWideThreads + tid; e < rows * (HD / 4); e += C * kWideThreads) {
      const int r = e / (HD / 4), d = e % (HD / 4);
      const uint32_t src = base + S::kO + r * HD * 4 + ((d ^ (r & 7)) << 4);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int c0 = 0; c0 < kMaxCluster; c0 += 8) {
        if (c0 >= C) break;
        float4 x[8];
#pragma unroll
        for (int c = 0; c < 8; ++c)
          x[c] = c0 + c < C ? peer_f32x4(peer_addr(src, c0 + c)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float w = c0 + c < C ? wt[(c0 + c) * kRows + r] : 0.f;
          o.x = fmaf(w, x[c].x, o.x);
          o.y = fmaf(w, x[c].y, o.y);
          o.z = fmaf(w, x[c].z, o.z);
          o.w = fmaf(w, x[c].w, o.w);
        }
      }
      if (wt[r] < 0.f) o = make_float4(0.f, 0.f, 0.f, 0.f);
      const long long at = row_at(r, p.o_ld) + d * 4;
      const uint2 u = make_uint2(bf16x2(o.x, o.y), bf16x2(o.z, o.w));
      *reinterpret_cast<uint2*>(p.o + at) = u;
      if constexpr (kLo)
        *reinterpret_cast<uint2*>(p.o_lo + at) = make_uint2(bf16x2(o.x - bf16lo(u.x), o.y - bf16hi(u.x)),
                                                            bf16x2(o.z - bf16lo(u.y), o.w - bf16hi(u.y)));
    }
    __syncwarp();
    cluster_sync_all();  // peers' shared memory stays until every CTA has read it
  }
  if (tid == 0 && sm.abort) set_status(p.status, SPEC_DEV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == kWIssue) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmemCols);
  }
}

template <int HD, bool kLo>
cudaError_t launch_wide(const Kv8AttnParams& p, cudaStream_t stream) {
  using S = WideSmem<HD>;
  static PerDevice<AttSetup> setup;
  AttSetup s{};
  if (!setup.get([] { return att_setup(kv8_attention_wide_kernel<HD, kLo>, kWideThreads, S::kBytes); }, &s))
    return cudaErrorInvalidDevice;
  if (s.err != cudaSuccess) return s.err;
  const int rtiles = (p.n * p.G + kRows - 1) / kRows, c = att_cluster(p, rtiles, s, 1);
  CUtensorMap kmap;
  if (!page_map(&kmap, p.kc, static_cast<long long>(p.n_pages) * p.Hkv * kPageSlots, HD)) return cudaErrorInvalidValue;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg =
      att_config(dim3(rtiles * c, p.Hkv, p.B), kWideThreads, S::kBytes, stream, attr, c);
  return cudaLaunchKernelEx(&cfg, kv8_attention_wide_kernel<HD, kLo>, kmap, p, c, s.sms);
}

}  // namespace

cudaError_t launch_kv8_attention_wide(const Kv8AttnParams& p, cudaStream_t stream) {
  if (p.o_lo) return p.hd == 128 ? launch_wide<128, true>(p, stream) : launch_wide<64, true>(p, stream);
  return p.hd == 128 ? launch_wide<128, false>(p, stream) : launch_wide<64, false>(p, stream);
}

}  // namespace spec
