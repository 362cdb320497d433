// What the attention kernels over the 8-bit cache share: TMEM, packed
// arithmetic and descriptors, which tiles a CTA takes, the tile loader, and on
// the host the tensor maps and the launch's clusters.
#pragma once

#include <algorithm>
#include <climits>

#include "internal.h"
#include "kv8_common.cuh"

namespace spec {
namespace {

constexpr int kTile = 128;           // keys per tile
constexpr int kMaxCluster = 16;
// Sequences that are put in order of length, a thread each among the first 96 (a
// multiple of 4); of more, the waves are many enough that their order counts
// for little, and each CTA would pay for the search.
constexpr int kSortSeqs = 96;
constexpr int kMinTiles = 2;         // tiles of a CTA at least, where they are shared
constexpr int kSmemCta = 227 * 1024;   // dynamic shared memory of a CTA alone on its SM,
constexpr int kSmemHalf = 113 * 1024;  // ... and of two (1 KB of each CTA's share is the system's)
// ... of a CTA that takes an SM's TMEM for itself and whose cluster waits for it: it
// shares its SM with no CTA that could hold TMEM while waiting for another (none
// of those needs less than 67 KB)
constexpr int kSmemAlone = 160 * 1024;
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
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
SPEC_DEVINL void tmem_st_x8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
SPEC_DEVINL void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

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
// Two fp32 values to bf16 (`a` low; infinities and NaN kept).
SPEC_DEVINL uint32_t bf16x2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
// fp16 pairs: two fp32 rounded, product, a b + c, to e4m3 and back (`a` low).
SPEC_DEVINL uint32_t f16x2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
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
// Shared-memory descriptor of rows of ROWB bytes (128, 64 or 32) with the swizzle
// of that span: 8-row groups ROWB * 8 apart (stride offset); lbo: distance
// between two spans along an MN-major operand's own dimension.
template <int ROWB>
SPEC_DEVINL uint64_t sdesc_rows(uint32_t saddr, uint32_t lbo) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>((ROWB * 8) >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(ROWB == 128 ? 2 : (ROWB == 64 ? 4 : 6)) << 61;
  return d;
}
// Byte offset of 16-byte chunk c of row i in such rows.
template <int ROWB>
SPEC_DEVINL uint32_t swz_off(int i, int c) {
  if constexpr (ROWB == 128) return static_cast<uint32_t>(i * 128 + ((c ^ (i & 7)) << 4));
  if constexpr (ROWB == 64) return static_cast<uint32_t>(i * 64 + ((c ^ ((i >> 1) & 3)) << 4));
  return static_cast<uint32_t>(i * 32 + ((c ^ ((i >> 2) & 1)) << 4));
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
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}
SPEC_DEVINL float4 peer_f32x4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a));
  return v;
}

// A place in the ring: stage and the parity of the fill being awaited there
// (counted along: a division by a stage count known only at run time costs the
// one issuing thread ~100 cycles).
struct Ring {
  int s = 0;
  uint32_t par = 0;
  SPEC_DEVINL void next(int stages) {
    if (++s == stages) {
      s = 0;
      par ^= 1u;
    }
  }
};


// Which sequence block z takes.  With the lengths at hand (up to kSortSeqs), the
// longest sequences go first (blocks start in index order: block z takes the
// sequence with z longer ones), and `unit` is the tiles of a CTA at which all
// tiles fill the GPU once.  Every thread calls it; sm has len, seq, seq_len, unit.
struct AttPick {
  int b;
  bool sorted;  // sm.seq_len and sm.unit are set
};
SPEC_DEVINL int att_tiles(const Kv8AttnParams& p, int len) {
  return len < 0 || len > p.max_pages * kPageSlots - p.n ? 0 : (len + p.n + kTile - 1) / kTile;
}
template <class Misc>
SPEC_DEVINL AttPick att_pick(const Kv8AttnParams& p, bool shared, int slots, Misc& sm) {
  const int tid = threadIdx.x;
  AttPick a{static_cast<int>(blockIdx.z), p.B > 1 && p.B <= kSortSeqs};
  if (!a.sorted) return a;
  if (tid < kSortSeqs) sm.len[tid] = tid < p.B ? p.base[tid] : INT_MIN;  // (no length, after all others)
  __syncthreads();
  if (tid < p.B) {
    const int mine = sm.len[tid];
    int before = 0, total = 0;
    for (int j = 0; j < p.B; j += 4) {
      const int4 v = *reinterpret_cast<const int4*>(&sm.len[j]);
      const int o[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) before += o[k] > mine || (o[k] == mine && j + k < tid);
      if (shared)
#pragma unroll
        for (int k = 0; k < 4; ++k) total += att_tiles(p, o[k]);
    }
    if (before == static_cast<int>(blockIdx.z)) {
      sm.seq = tid;
      sm.seq_len = mine;
      if (shared) sm.unit = max(kMinTiles, (total + slots - 1) / max(slots, 1));
    }
  }
  __syncthreads();
  a.b = sm.seq;
  return a;
}

// One warp: the pages of tiles i0 .. i0 + nt - 1 into a ring of tiles.  Page ids
// come 16 at a time (8 tiles), the next 16 on their way: a lookup per page in
// line with the loads took ~500 cycles each.  page_at(e): the page of entry e
// counted from the first tile (0 past the last of the `entries`).
template <int HD, class PageAt>
SPEC_DEVINL void att_load_tiles(const CUtensorMap* map, uint64_t* full, uint64_t* empty, int* pages, uint32_t ring,
                                int stages, int nt, int entries, int Hkv, int h, int* abort, PageAt page_at) {
  const int lane = threadIdx.x & 31;
  const uint64_t pol = l2_policy_evict_first();
  int next = nt > 0 && lane < 16 ? page_at(lane) : 0;
  Ring r;
  bool ok = true;
  int i = 0, issued = 0;
  while (i < nt && ok) {
    __syncwarp();
    if (lane < 16) {
      pages[lane] = next;
      next = page_at(2 * i + 16 + lane);
    }
    __syncwarp();
    const int end = min(i + 8, nt);
    if (lane == 0) {
      for (int k = 0; i + k < end; ++k) {
        if (i + k >= stages && !mbar_wait(&empty[r.s], r.par ^ 1u, abort)) {
          ok = false;
          break;
        }
        const bool two = entries - 2 * (i + k) > 1;  // a page past the end is not read
        const int2 pg = *reinterpret_cast<const int2*>(&pages[2 * k]);
        const uint32_t dst = ring + r.s * (kTile * HD);
        mbar_arrive_expect_tx(&full[r.s], (two ? 2u : 1u) * kPageSlots * HD);
        tma_load_2d_s(dst, map, &full[r.s], 0, (pg.x * Hkv + h) * kPageSlots, pol);
        if (two) tma_load_2d_s(dst + kPageSlots * HD, map, &full[r.s], 0, (pg.y * Hkv + h) * kPageSlots, pol);
        r.next(stages);
        ++issued;
      }
    }
    ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
    i = end;
  }
  if (lane == 0 && *static_cast<volatile int*>(abort)) {  // loads in flight land before the CTA leaves (bounded too)
    int none = 0;
    for (int k = max(0, issued - stages); k < issued; ++k)
      mbar_wait(&full[k % stages], static_cast<uint32_t>((k / stages) & 1), &none);
  }
  __syncwarp();
}

// ------------------------------------------------------------------ host
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
  int active[kMaxCluster + 1];  // clusters of each size that can run at once, a CTA an SM
  int sms;
};

cudaLaunchConfig_t att_config(dim3 grid, int threads, uint32_t smem, cudaStream_t stream,
                              cudaLaunchAttribute (&attr)[2], int C) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
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

// Set up once per device: shared-memory limit, cluster permission, how many
// clusters of CTAs of `smem` bytes fit (the query places one CTA on an SM even
// where two fit; twice as many clusters were seen to run then).
template <class F>
AttSetup att_setup(F fn, int threads, int smem) {
  AttSetup r{cudaSuccess, {}, 0};
  int dev = 0;
  if ((r.err = cudaGetDevice(&dev)) != cudaSuccess) return r;
  if ((r.err = cudaDeviceGetAttribute(&r.sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return r;
  if ((r.err = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemCta)) != cudaSuccess)
    return r;
  if ((r.err = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess) return r;
  for (int c = 1; c <= kMaxCluster; ++c) {
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = att_config(dim3(c), threads, smem, nullptr, attr, c);
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess) {
      cudaGetLastError();  // (a size that does not fit is no error of the call)
      continue;
    }
    r.active[c] = n;
  }
  return r;
}

// CTAs of a cluster (one per row tile): the most, up to 16, with which all of the
// clusters run at once, each CTA with two tiles at least at full capacity.  (More
// than the GPU holds, the surplus leaving at once, costs more than the even
// shares give: batch 16 29 us against 21.  A cluster lies within a group of
// SMs: 16 clusters of 16, two CTAs an SM, do not fit although their CTAs would.)
int att_cluster(const Kv8AttnParams& p, int rtiles, const AttSetup& s, int per_sm) {
  const long long groups = static_cast<long long>(p.B) * p.Hkv * rtiles;
  const int tiles = (p.max_pages * kPageSlots + kTile - 1) / kTile;
  int c = 1;
  for (int k = 2; k <= kMaxCluster && k * kMinTiles <= tiles; ++k)
    if (groups <= static_cast<long long>(per_sm) * s.active[k]) c = k;
  return c;
}

}  // namespace
}  // namespace spec
