// Attention of n new positions over the 8-bit paged KV cache.
//   s_j = scale * q . (ks_j k_j),  o = sum_j p_j vs_j v_j / sum_j p_j,
//   p_j = exp(s_j - max s) over the slots that the row's token may see
// (the cached ones, and of the new ones its own and earlier, or those of its
// ancestor mask); a row that sees nothing is zero.
//
// The cache is read once, by TMA, into shared memory, and enters the tensor
// cores as it is stored: both products are tcgen05.mma kind::f8f6f4 with e4m3
// operands and fp32 accumulators in TMEM, so no key or value is ever
// converted.  The other operand is split into e4m3 pieces that add up to it:
//   q row = 2^k (hi + lo)            bf16 has 8 significant bits, a piece 4: exact but
//                                    for elements 2^-18 below the row's largest
//   p     = 2^-7 (hi + mid + lo)     an fp16 weight's 11 bits (2^-17 of the row's
//                                    reference at the least)
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
// need not be its maximum: weights up to 2^1.8 M fit the pieces, so M is set
// one above the maximum of the first tile and raised only when a score passes
// it by 1.75 (one barrier per tile asks whether any did).  Until then O^T adds
// up in TMEM and no thread reads it.  Warp 4 issues the TMA loads, warp 5 the
// MMAs; S and P are double-buffered, so the scores of tile i + 1 and the
// products of tile i - 1 run beside the softmax of tile i.
#include <cudaTypedefs.h>

#include <algorithm>

#include "internal.h"
#include "kv8_common.cuh"

namespace spec {
namespace {

constexpr int kTile = 128;                  // keys per tile
constexpr int kSoft = 128;                  // softmax threads
constexpr int kAttThreads = kSoft + 64;     // + TMA warp + MMA warp
constexpr int kPRow = 128;                  // bytes of a key's row of P
constexpr int kMaxCluster = 16;
constexpr float kTopExp = 8.75f;            // 2^8.75 < 448: weights times 2^7 that fit e4m3
constexpr float kNoRef = -3.402823466e38f;  // M of a row that has seen no slot: any score passes it

SPEC_DEVINL void tmem_ld_x8(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
}
SPEC_DEVINL void tmem_ld_x16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
SPEC_DEVINL void tmem_ld_x32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// N consecutive columns of the thread's lane (N a multiple of 8), ready for use.
template <int N>
SPEC_DEVINL void tmem_ld(uint32_t taddr, uint32_t (&r)[N]) {
  int at = 0;
#pragma unroll
  for (; at + 32 <= N; at += 32) tmem_ld_x32(taddr + at, r + at);
  if constexpr (N % 32 >= 16) {
    tmem_ld_x16(taddr + at, r + at);
    at += 16;
  }
  if constexpr (N % 16 >= 8) tmem_ld_x8(taddr + at, r + at);
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));  // no use moves above the wait
}

// Two fp32 operations in one instruction.
SPEC_DEVINL float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.ftz.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
SPEC_DEVINL float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.ftz.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
SPEC_DEVINL float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.ftz.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
// fp16 pairs: two fp32 rounded, the difference, to e4m3 and back (`a` low).
SPEC_DEVINL uint32_t f16x2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
SPEC_DEVINL uint32_t f16x2_sub(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
SPEC_DEVINL uint32_t f16x2_to_e4m3x2(uint32_t a) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(a));
  return r;
}
SPEC_DEVINL uint32_t e4m3x2_to_f16x2(uint32_t a) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(a)));
  return r;
}

// D[tmem] (+)= A[smem] * B[smem] of e4m3 operands, issued by one thread.
SPEC_DEVINL void umma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor of kind::f8f6f4, e4m3 x e4m3 -> fp32, M x N; tra / trb:
// operand stored MN-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, bool tra, bool trb) {
  return (1u << 4) | (tra ? 1u << 15 : 0u) | (trb ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}
// Shared-memory descriptor of rows of ROWB bytes (128 or 64) with the swizzle
// of that span: 8-row groups ROWB * 8 apart (stride offset); lbo: distance
// between two spans along an MN-major operand's own dimension.
template <int ROWB>
SPEC_DEVINL uint64_t sdesc_rows(uint32_t saddr, uint32_t lbo) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>((ROWB * 8) >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(ROWB == 128 ? 2 : 4) << 61;
  return d;
}
// Byte offset of 16-byte chunk c of row i in such rows.
template <int ROWB>
SPEC_DEVINL uint32_t swz_off(int i, int c) {
  if constexpr (ROWB == 128)
    return static_cast<uint32_t>(i * 128 + ((c ^ (i & 7)) << 4));
  else
    return static_cast<uint32_t>(i * 64 + ((c ^ ((i >> 1) & 3)) << 4));
}

SPEC_DEVINL void st_shared_v4(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
SPEC_DEVINL void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
SPEC_DEVINL void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
SPEC_DEVINL uint32_t peer_addr(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
SPEC_DEVINL float peer_f32(uint32_t a) {
  float v;
  asm("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}
SPEC_DEVINL float4 peer_f32x4(uint32_t a) {
  float4 v;
  asm("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}

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

template <int HD, int RT>
struct AttSmem {
  static constexpr int kStages = HD == 128 ? 2 : 4;
  static constexpr uint32_t kTileB = kTile * HD;  // bytes of a K or V tile
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kP = kQ + 2 * RT * HD;
  static constexpr uint32_t kPB = kTile * kPRow;  // bytes of one P buffer
  static constexpr uint32_t kK = kP + 2 * kPB;
  static constexpr uint32_t kV = kK + kStages * kTileB;
  static constexpr uint32_t kMisc = kV + kStages * kTileB;
  struct Misc {
    uint64_t full_k[kStages], full_v[kStages], empty_k[kStages], empty_v[kStages];
    uint64_t s_full[2], s_free[2], p_full[2], o_full[2], drain;
    uint64_t anc[RT];
    alignas(16) float red[4][RT];  // per-warp maxima (sums at the end); this and the next three are read as float4
    float mneg[4][RT];         // each warp's copy of 7 - M
    float alpha[4][RT];        // ... and of the factor of a rise of M
    float cq[RT];              // score factor of a row: 2^k scale log2(e)
    float stat[2][RT];         // this CTA's M' and sum
    float peer[2][kMaxCluster][RT];
    uint32_t nan[RT][HD / 32]; // outputs that a NaN value code reaches
    uint32_t tmem;
    int abort, any_nan, fresh;  // fresh: the tile whose products start O from zero
  };
  // partial sums [RT][HD] fp32, over the K ring once every MMA is done
  static constexpr uint32_t kO = kK;
  static_assert(offsetof(Misc, mneg) % 16 == 0 && offsetof(Misc, alpha) % 16 == 0 && offsetof(Misc, cq) % 16 == 0 &&
                    alignof(Misc) == 16 && kMisc % 1024 == 0,
                "row arrays are read as float4");
  static_assert(RT * HD * 4 <= 2 * kStages * kTileB, "the partial sums lie over the ring");
  static constexpr uint32_t kBytes = kMisc + sizeof(Misc) + 1024;  // + alignment of the base
  static constexpr int kNO = (3 * RT + 15) / 16 * 16;              // O columns (M = 128 takes multiples of 16)
  static constexpr uint32_t kTmemCols = RT >= 24 ? 256 : (RT == 16 ? 128 : 64);
  static_assert(4 * RT + kNO <= static_cast<int>(kTmemCols), "two S buffers and O");
};

struct AttMaps {
  CUtensorMap k, v;
};

template <int HD, int RT>
__global__ void __launch_bounds__(kAttThreads, 2)
    kv8_attention_kernel(const __grid_constant__ AttMaps maps, const Kv8AttnParams p, const int C) {
  using S = AttSmem<HD, RT>;
  constexpr int NS = S::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  auto& sm = *reinterpret_cast<typename S::Misc*>(smem_raw + (base - smem_u32(smem_raw)) + S::kMisc);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x % C, rtile = blockIdx.x / C, h = blockIdx.y, b = blockIdx.z;
  const int G = p.H / p.Hkv, R = p.n * G, rbase = rtile * RT;

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&sm.full_k[i], 1);
      mbar_init(&sm.full_v[i], 1);
      mbar_init(&sm.empty_k[i], 1);
      mbar_init(&sm.empty_v[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.s_free[i], kSoft);
      mbar_init(&sm.p_full[i], kSoft);
      mbar_init(&sm.o_full[i], 1);
    }
    mbar_init(&sm.drain, 1);
    fence_mbar_init();
    sm.abort = 0;
    sm.any_nan = 0;
    sm.fresh = 0;
  }
  if (warp == 4) {
    if (lane == 0) {
      prefetch_tmap(&maps.k);
      prefetch_tmap(&maps.v);
    }
    __syncwarp();
    tmem_alloc(&sm.tmem, S::kTmemCols);
    tmem_relinquish();
  }
  grid_dep_wait();
  grid_dep_launch();

  const int L = p.base[b];
  const int32_t unfit = kv8_fit(L, p.n, p.table, p.max_pages, p.n_pages, b);
  if (unfit && tid == 0) set_status(p.status, unfit);
  const int T = unfit ? 0 : L + p.n;  // slots [0, T)
  const int tiles = (T + kTile - 1) / kTile;
  const int i0 = static_cast<int>(static_cast<long long>(tiles) * rank / C);
  const int nt = static_cast<int>(static_cast<long long>(tiles) * (rank + 1) / C) - i0;  // this CTA's tiles
  const int32_t* table = p.table + static_cast<long long>(b) * p.max_pages;
  const auto page_of = [&](int t) {  // the page of slot t, clamped into the pool
    const int pg = __ldg(table + min(t / kPageSlots, p.max_pages - 1));
    if (pg < 0 || pg >= p.n_pages) {
      if (t < T) set_status(p.status, SPEC_DEV_BAD_PAGE);
      return pg < 0 ? 0 : p.n_pages - 1;
    }
    return pg;
  };

  // ---- the query rows as e4m3 pieces: row r = token r / G, head h * G + r % G
  constexpr int TPR = RT <= 16 && HD == 128 ? 8 : 4;  // threads per query row
  static_assert(RT * TPR <= kSoft && RT * TPR % 32 == 0 && HD / TPR % 16 == 0, "whole warps, 16 elements a thread");
  if (tid < RT * TPR) {
    constexpr int E = HD / TPR;  // elements per thread
    const int r = tid / TPR, part = tid % TPR, rr = rbase + r;
    float x[E];
#pragma unroll
    for (int c = 0; c < E / 8; ++c) {
      uint4 w = make_uint4(0, 0, 0, 0);
      if (rr < R)
        w = *reinterpret_cast<const uint4*>(p.q + (static_cast<long long>(b) * p.n + rr / G) * p.q_ld +
                                            (h * G + rr % G) * HD + part * E + c * 8);
      const uint32_t v[4] = {w.x, w.y, w.z, w.w};
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
        const uint32_t u = e4m3x2(a - f.x, d - f.y);
        if (k & 1) {
          hi[k / 2] |= w << 16;
          lo[k / 2] |= u << 16;
        } else {
          hi[k / 2] = w;
          lo[k / 2] = u;
        }
      }
      const int ch = part * (E / 16) + c;
      st_shared_v4(base + S::kQ + swz_off<HD>(r, ch), hi[0], hi[1], hi[2], hi[3]);
      st_shared_v4(base + S::kQ + swz_off<HD>(RT + r, ch), lo[0], lo[1], lo[2], lo[3]);
    }
    if (part == 0) {
#pragma unroll
      for (int c = 0; c < 4; ++c) sm.mneg[c][r] = -kNoRef;
      sm.cq[r] = odd ? __uint_as_float(0x7FC00000u)
                     : p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + k2) << 23);
      sm.anc[r] = (p.anc && rr < R) ? p.anc[static_cast<long long>(b) * p.n + rr / G] : 0ull;
#pragma unroll
      for (int c = 0; c < HD / 32; ++c) sm.nan[r][c] = 0u;
    }
    fence_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;

  float acc[RT], l[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) acc[r] = l[r] = 0.f;
  float mrun = kNoRef;  // lane r: row r's reference M

  if (warp == 4) {
    // ------------------------------------------------------- TMA producer
    if (lane == 0) {
      const uint64_t pol = l2_policy_evict_first();
      int issued = 0;
      const auto load = [&](const CUtensorMap* m, uint32_t dst, uint64_t* bar, int i) {
        const int t = (i0 + i) * kTile;
        const int np = T - t > kPageSlots ? 2 : 1;  // a page past the end is not read
        mbar_arrive_expect_tx(bar, static_cast<uint32_t>(np * kPageSlots * HD));
        for (int g = 0; g < np; ++g)
          tma_load_2d_s(dst + g * kPageSlots * HD, m, bar, 0, (page_of(t + g * kPageSlots) * p.Hkv + h) * kPageSlots,
                        pol);
      };
      for (int i = 0; i < nt; ++i) {
        const int s = i % NS;
        const uint32_t par = static_cast<uint32_t>((i / NS - 1) & 1);
        if (i >= NS && !mbar_wait(&sm.empty_k[s], par, &sm.abort)) break;
        load(&maps.k, base + S::kK + s * S::kTileB, &sm.full_k[s], i);
        issued = 2 * i + 1;
        if (i >= NS && !mbar_wait(&sm.empty_v[s], par, &sm.abort)) break;
        load(&maps.v, base + S::kV + s * S::kTileB, &sm.full_v[s], i);
        issued = 2 * i + 2;
      }
      if (sm.abort) {  // loads in flight land before the CTA leaves (bounded as every wait)
        int none = 0;
        for (int k = max(0, issued - 2 * NS); k < issued; ++k) {
          const int i = k / 2;
          mbar_wait(k & 1 ? &sm.full_v[i % NS] : &sm.full_k[i % NS], static_cast<uint32_t>((i / NS) & 1), &none);
        }
      }
    }
    __syncwarp();
  } else if (warp == 5) {
    // --------------------------------------------------------- MMA issuer
    if (lane == 0) {
      constexpr uint32_t id_s = idesc_e4m3(kTile, 2 * RT, false, false);
      constexpr uint32_t id_o = idesc_e4m3(kTile, S::kNO, true, true);
      const auto issue_o = [&](int i) {
        const int s = i % NS;
        if (!mbar_wait(&sm.full_v[s], static_cast<uint32_t>((i / NS) & 1), &sm.abort)) return false;
        if (!mbar_wait(&sm.p_full[i & 1], static_cast<uint32_t>((i >> 1) & 1), &sm.abort)) return false;
        tc_fence_after();
        const bool fresh = *static_cast<volatile int*>(&sm.fresh) == i;
#pragma unroll
        for (int kk = 0; kk < kTile / 32; ++kk)
          // head dim 64: the 128 rows of the A operand are the 64 dimensions twice
          umma_e4m3(tmem + 4 * RT, sdesc_rows<HD>(base + S::kV + s * S::kTileB + kk * 32 * HD, 0),
                    sdesc_rows<kPRow>(base + S::kP + (i & 1) * S::kPB + kk * 32 * kPRow, 0), id_o,
                    kk > 0 || !fresh ? 1u : 0u);
        umma_commit(&sm.empty_v[s]);
        umma_commit(&sm.o_full[i & 1]);
        return true;
      };
      bool ok = true;
      for (int i = 0; i < nt && ok; ++i) {
        const int s = i % NS;
        ok = mbar_wait(&sm.full_k[s], static_cast<uint32_t>((i / NS) & 1), &sm.abort) &&
             (i < 2 || mbar_wait(&sm.s_free[i & 1], static_cast<uint32_t>((i / 2 - 1) & 1), &sm.abort));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < HD / 32; ++kk)
          umma_e4m3(tmem + (i & 1) * 2 * RT, sdesc_rows<HD>(base + S::kK + s * S::kTileB + kk * 32, 16),
                    sdesc_rows<HD>(base + S::kQ + kk * 32, 16), id_s, kk > 0 ? 1u : 0u);
        umma_commit(&sm.empty_k[s]);
        umma_commit(&sm.s_full[i & 1]);
        if (i) ok = issue_o(i - 1);
      }
      if (ok && nt) ok = issue_o(nt - 1);
      if (!ok) {  // MMAs in flight end before TMEM and shared memory go
        int none = 0;
        umma_commit(&sm.drain);
        mbar_wait(&sm.drain, 0, &none);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------- softmax and accumulation
    // A wait that gives up sets the abort flag; the threads leave the loop
    // together at its barrier.
    const uint32_t lane_addr = static_cast<uint32_t>(warp * 32) << 16;
    const Kv8Map map{p.table, p.max_pages, p.n_pages, p.Hkv, HD};
    const int sub = (tid % kPageSlots) / kKv8Block;
    const auto scale_at = [&](int pg) { return (static_cast<long long>(pg) * p.Hkv + h) * kKv8Sub + sub; };
    const auto add_o = [&](int i) {  // acc += what O holds, tile i's products the last
      mbar_wait(&sm.o_full[i & 1], static_cast<uint32_t>((i >> 1) & 1), &sm.abort);
      tc_fence_after();
      uint32_t o[RT];
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        tmem_ld(tmem + lane_addr + (4 + q) * RT, o);
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[r] += __uint_as_float(o[r]);
      }
    };
    // this thread's scales, one tile ahead, and its page, two ahead
    int pg1 = nt > 0 ? page_of(i0 * kTile + tid) : 0;
    float ks_n = nt > 0 ? __ldg(p.ks + scale_at(pg1)) : 1.f, vs_n = nt > 0 ? __ldg(p.vs + scale_at(pg1)) : 1.f;
    pg1 = nt > 1 ? page_of((i0 + 1) * kTile + tid) : 0;
    bool stopped = false;
    for (int i = 0; i < nt; ++i) {
      const int buf = i & 1, t0 = (i0 + i) * kTile, t = t0 + tid;
      const float ks = ks_n, vs = vs_n;
      if (i + 1 < nt) {
        ks_n = __ldg(p.ks + scale_at(pg1));
        vs_n = __ldg(p.vs + scale_at(pg1));
        if (i + 2 < nt) pg1 = page_of(t0 + 2 * kTile + tid);
      }
      const bool none = t >= T;  // past the end: no scale to read
      const float lvs = none ? 0.f : static_cast<float>(static_cast<int>(__float_as_uint(vs) >> 23) - 127);
      const float ivs = none ? 0.f : pow2_inv(vs);
      const bool masked = t0 + kTile > L;  // the tile holds slots that some row does not see
      uint32_t vis = 0xFFFFFFFFu;          // bit r: row rbase + r sees slot t
      if (masked && t >= L) {
        const int k = t - L;
        if (t >= T) {
          vis = 0u;
        } else if (p.anc) {
          vis = 0u;
          if (k < 64)
            for (int r = 0; r < RT; ++r) vis |= static_cast<uint32_t>((sm.anc[r] >> k) & 1ull) << r;
        } else {  // row rr (token rr / G) sees new slot k iff rr >= k * G
          const int first = k * G - rbase;
          if (first > 0) vis = first >= 32 ? 0u : 0xFFFFFFFFu << first;
        }
      }
      mbar_wait(&sm.s_full[buf], static_cast<uint32_t>((i >> 1) & 1), &sm.abort);
      tc_fence_after();
      float s[RT];
      const auto scores = [&] {  // s_j + log2 vs_j of this key for the tile's rows
        uint32_t w[2 * RT];
        tmem_ld(tmem + lane_addr + buf * 2 * RT, w);
        const float2 ks2 = make_float2(ks, ks), lvs2 = make_float2(lvs, lvs);
#pragma unroll
        for (int r = 0; r < RT; r += 4) {
          const float4 c = *reinterpret_cast<const float4*>(sm.cq + r);
#pragma unroll
          for (int q = 0; q < 4; q += 2) {
            const float2 u = add2(make_float2(__uint_as_float(w[r + q]), __uint_as_float(w[r + q + 1])),
                                  make_float2(__uint_as_float(w[RT + r + q]), __uint_as_float(w[RT + r + q + 1])));
            const float2 x = fma2(mul2(u, ks2), q ? make_float2(c.z, c.w) : make_float2(c.x, c.y), lvs2);
            s[r + q] = x.x;
            s[r + q + 1] = x.y;
          }
        }
        if (masked) {
#pragma unroll
          for (int r = 0; r < RT; ++r) s[r] = (vis >> r) & 1u ? s[r] : -INFINITY;
        }
      };
      const auto exponents = [&] {  // s - M + 7, and the largest of them
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
        // This thread's value row, if not every row sees it: zero past the
        // end (pages hold anything there), and NaN codes taken out (their
        // weight of 0 would not clear them) and noted for the rows that see them.
        const uint32_t vt = base + S::kV + (i % NS) * S::kTileB;
        mbar_wait(&sm.full_v[i % NS], static_cast<uint32_t>((i / NS) & 1), &sm.abort);
        if (t >= L) {
#pragma unroll 1
          for (int c = 0; c < HD / 16; ++c) {
            const uint32_t a = vt + swz_off<HD>(tid, c);
            if (t >= T) {
              st_shared_v4(a, 0, 0, 0, 0);
              continue;
            }
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
              uint32_t w;
              asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(a + 4 * k) : "memory");
              const uint32_t m = w & 0x7F7F7F7Fu;
              const uint32_t hit = (m + 0x01010101u) & 0x80808080u;  // bytes 0x7F: the NaN codes
              if (!hit) continue;
              sm.any_nan = 1;
              for (int q = 0; q < 4; ++q) {
                if (!((hit >> (8 * q + 7)) & 1u)) continue;
                w &= ~(0xFFu << (8 * q));
                const int d = c * 16 + k * 4 + q;
                for (int r = 0; r < RT; ++r)
                  if ((vis >> r) & 1u) atomicOr(&sm.nan[r][d / 32], 1u << (d % 32));
              }
              asm volatile("st.shared.b32 [%0], %1;" ::"r"(a + 4 * k), "r"(w) : "memory");
            }
          }
        }
      }
      // ---- does any exponent pass the pieces' range?
      const bool raise = exponents() > kTopExp;
      if (named_bar_any(1, kSoft, raise || *static_cast<volatile int*>(&sm.abort) != 0)) {
        // raise M to one above each row's maximum; what is summed so far shrinks by alpha
        if (named_bar_any(2, kSoft, *static_cast<volatile int*>(&sm.abort) != 0)) {
          stopped = true;
          break;
        }
        scores();
        const float m = warp_rows_reduce(s, -INFINITY, [](float a, float c) { return fmaxf(a, c); });
        if (lane < RT) sm.red[warp][lane] = m;
        named_bar(1, kSoft);
        if (lane < RT) {
          const float mt = fmaxf(fmaxf(sm.red[0][lane], sm.red[1][lane]), fmaxf(sm.red[2][lane], sm.red[3][lane]));
          const float mn = fmaxf(mrun, mt + 1.f);
          sm.alpha[warp][lane] = exp2f(mrun - mn);
          sm.mneg[warp][lane] = 7.f - mn;
          mrun = mn;
        }
        __syncwarp();
        if (i) add_o(i - 1);
        if (tid == 0) sm.fresh = i;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const float a = sm.alpha[warp][r];
          acc[r] *= a;
          l[r] *= a;
        }
        exponents();
      }
      tc_fence_before();
      mbar_arrive(&sm.s_free[buf]);
      // ---- weights (times 2^7) and their sums; P: this key's row, hi | mid | lo
      uint32_t w[3][RT / 4];
#pragma unroll
      for (int r = 0; r < RT; r += 2) {
        const float2 e = make_float2(exp2f(s[r]), exp2f(s[r + 1]));
        const float2 sum = fma2(e, make_float2(ivs, ivs), make_float2(l[r], l[r + 1]));
        l[r] = sum.x, l[r + 1] = sum.y;
        uint32_t f = f16x2(e.x, e.y);
#pragma unroll
        for (int q = 0; q < 3; ++q) {
          const uint32_t u = f16x2_to_e4m3x2(f);
          if (q < 2) f = f16x2_sub(f, e4m3x2_to_f16x2(u));
          w[q][r / 4] = r % 4 ? w[q][r / 4] | (u << 16) : u;
        }
      }
      // P of tile i - 2 has been read
      if (i >= 2) mbar_wait(&sm.o_full[buf], static_cast<uint32_t>(((i >> 1) - 1) & 1), &sm.abort);
      const uint32_t prow = base + S::kP + buf * S::kPB;
      const auto word = [&](int k) { return w[k / (RT / 4)][k % (RT / 4)]; };
#pragma unroll
      for (int c = 0; c < 3 * RT / 16; ++c)
        st_shared_v4(prow + swz_off<kPRow>(tid, c), word(4 * c), word(4 * c + 1), word(4 * c + 2), word(4 * c + 3));
      if constexpr (3 * RT % 16 != 0) {
        constexpr int c = 3 * RT / 16;
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(prow + swz_off<kPRow>(tid, c)), "r"(word(4 * c)),
                     "r"(word(4 * c + 1))
                     : "memory");
      }
      fence_async_smem();
      tc_fence_before();
      mbar_arrive(&sm.p_full[buf]);
    }
    if (nt && !stopped) add_o(nt - 1);
    // ---- this CTA's row sums
    const float ls = warp_rows_reduce(l, 0.f, [](float a, float c) { return a + c; });
    named_bar(1, kSoft);  // the last tile's maxima have been read
    if (lane < RT) sm.red[warp][lane] = ls;
    named_bar(1, kSoft);
    if (tid < RT) {
      sm.stat[0][tid] = mrun;
      sm.stat[1][tid] = (sm.red[0][tid] + sm.red[1][tid]) + (sm.red[2][tid] + sm.red[3][tid]);
    }
    if (sm.any_nan && tid < HD) {
#pragma unroll
      for (int r = 0; r < RT; ++r)
        if ((sm.nan[r][tid / 32] >> (tid % 32)) & 1u) acc[r] = __uint_as_float(0x7FC00000u);
    }
    if (tid < HD) {
#pragma unroll
      for (int r = 0; r < RT; ++r)
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(base + S::kO + (r * HD + tid) * 4), "f"(acc[r]) : "memory");
    }
  }

  // ---- merge: the cluster's CTAs share the (row, 4 dimensions) items
  __syncwarp();
  if (C > 1)
    cluster_sync_all();
  else
    __syncthreads();
  const uint32_t stat = smem_u32(&sm.stat[0][0]);
  for (int e = tid; e < 2 * C * RT; e += kAttThreads) {
    const int which = e / (C * RT), c = (e / RT) % C, r = e % RT;
    const uint32_t a = stat + (which * RT + r) * 4;
    sm.peer[which][c][r] = C > 1 ? peer_f32(peer_addr(a, c)) : sm.stat[which][r];
  }
  __syncthreads();
  const int rows = min(RT, R - rbase);
  for (int e = rank * kAttThreads + tid; e < rows * (HD / 4); e += C * kAttThreads) {
    const int r = e / (HD / 4), d = e % (HD / 4) * 4;
    const uint32_t a = base + S::kO + (r * HD + d) * 4;
    float m = kNoRef;
    for (int c = 0; c < C; ++c) m = fmaxf(m, sm.peer[0][c][r]);
    float lt = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = 0; c < C; ++c) {
      const float mc = sm.peer[0][c][r];
      const float w = exp2f(mc - m);  // 1 if no CTA has seen a slot: their sums are zero
      const float4 x = peer_f32x4(C > 1 ? peer_addr(a, c) : peer_addr(a, 0));
      lt = fmaf(w, sm.peer[1][c][r], lt);
      o.x = fmaf(w, x.x, o.x);
      o.y = fmaf(w, x.y, o.y);
      o.z = fmaf(w, x.z, o.z);
      o.w = fmaf(w, x.w, o.w);
    }
    const float inv = lt == 0.f ? 0.f : 1.f / lt;  // a row that sees nothing is zero
    const int rr = rbase + r;
    uint2 u;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u.x) : "f"(o.y * inv), "f"(o.x * inv));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u.y) : "f"(o.w * inv), "f"(o.z * inv));
    *reinterpret_cast<uint2*>(p.o + (static_cast<long long>(b) * p.n + rr / G) * p.o_ld + (h * G + rr % G) * HD + d) =
        u;
  }
  if (C > 1) cluster_sync_all();  // peers' shared memory stays until every CTA has read it
  if (tid == 0 && sm.abort) set_status(p.status, SPEC_DEV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmemCols);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 tmap_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// One layer's codes as [rows][hd] bytes, boxes of one page of one head (64 rows).
bool page_map(CUtensorMap* m, const void* codes, long long rows, int hd) {
  const auto fn = tmap_encoder();
  if (!fn) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(hd), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(hd)};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(hd), kPageSlots};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, hd == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct AttSetup {
  cudaError_t err;
  int max_cluster;  // largest cluster size that can be placed
  int sms;
};

cudaLaunchConfig_t att_config(dim3 grid, uint32_t smem, cudaStream_t stream, cudaLaunchAttribute (&attr)[2], int C) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kAttThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

template <int HD, int RT>
cudaError_t launch_tile(const Kv8AttnParams& p, cudaStream_t stream) {
  constexpr uint32_t smem = AttSmem<HD, RT>::kBytes;
  static PerDevice<AttSetup> setup;
  AttSetup s{};
  if (!setup.get(
          [] {
            AttSetup r{cudaSuccess, 1, 0};
            int dev = 0;
            if ((r.err = cudaGetDevice(&dev)) != cudaSuccess) return r;
            if ((r.err = cudaDeviceGetAttribute(&r.sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return r;
            const auto fn = kv8_attention_kernel<HD, RT>;
            if ((r.err = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                              static_cast<int>(smem))) != cudaSuccess)
              return r;
            if ((r.err = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess)
              return r;
            for (int c = kMaxCluster; c > 1; c /= 2) {
              cudaLaunchAttribute attr[2];
              cudaLaunchConfig_t cfg = att_config(dim3(c), smem, nullptr, attr, c);
              cfg.numAttrs = 1;
              int n = 0;
              if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) == cudaSuccess && n > 0) {
                r.max_cluster = c;
                break;
              }
            }
            return r;
          },
          &s))
    return cudaErrorInvalidDevice;
  if (s.err != cudaSuccess) return s.err;
  const int R = p.n * (p.H / p.Hkv), rtiles = (R + RT - 1) / RT;
  // as many CTAs per row tile as keep two resident per SM, and no more than tiles
  const long long groups = static_cast<long long>(p.B) * p.Hkv * rtiles;
  const int tiles = (p.max_pages * kPageSlots + kTile - 1) / kTile;
  int C = 1;
  while (2 * C <= s.max_cluster && 2 * C <= tiles && groups * 2 * C <= 2ll * s.sms) C *= 2;
  AttMaps maps;
  const long long rows = static_cast<long long>(p.n_pages) * p.Hkv * kPageSlots;
  if (!page_map(&maps.k, p.kc, rows, HD) || !page_map(&maps.v, p.vc, rows, HD)) return cudaErrorInvalidValue;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = att_config(dim3(C * rtiles, p.Hkv, p.B), smem, stream, attr, C);
  return cudaLaunchKernelEx(&cfg, kv8_attention_kernel<HD, RT>, maps, p, C);
}

template <int HD>
cudaError_t launch_rows(const Kv8AttnParams& p, cudaStream_t stream) {
  // the row tile that leaves the fewest rows empty, the larger of equal ones
  const int R = p.n * (p.H / p.Hkv);
  int best = 32;
  for (int rt = 24; rt >= 8; rt -= 8)
    if ((R + rt - 1) / rt * rt < (R + best - 1) / best * best) best = rt;
  switch (best) {
    case 8: return launch_tile<HD, 8>(p, stream);
    case 16: return launch_tile<HD, 16>(p, stream);
    case 24: return launch_tile<HD, 24>(p, stream);
    default: return launch_tile<HD, 32>(p, stream);
  }
}

}  // namespace

cudaError_t launch_kv8_attention(const Kv8AttnParams& p, cudaStream_t stream) {
  return p.hd == 128 ? launch_rows<128>(p, stream) : launch_rows<64>(p, stream);
}

}  // namespace spec
