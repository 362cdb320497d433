// The 8-bit paged KV cache: append with rotation, draft-tree commit and
// length updates.  (Attention over it is in kv8_attention.cu.)
#include "internal.h"
#include "kv8_common.cuh"

namespace spec {
namespace {

// ------------------------------------------------------------------ rotary
// Frequency of pair i in turns per position, split as hi + lo floats:
//   f = theta^(-2i / rd) / 2 pi
// scaled for long contexts by `factor`: every frequency divided by it
// (orig_len = 0), or, by wavelength, kept where orig_len * f >= high_freq
// turns, divided where <= low_freq, and mixed linearly between.
__global__ void kv8_rope_kernel(float2* dst, int rd, double theta, double factor, double low, double high,
                                int orig_len) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= rd / 2) return;
  const double two_pi = 6.283185307179586;
  double f = pow(theta, -2.0 * i / rd) / two_pi;
  if (factor != 1.0) {
    double w = 0.0;
    if (orig_len > 0) {
      w = (orig_len * f - low) / (high - low);
      w = w < 0.0 ? 0.0 : (w > 1.0 ? 1.0 : w);
    }
    f = f * w + f / factor * (1.0 - w);
  }
  const float hi = static_cast<float>(f);
  dst[i] = make_float2(hi, static_cast<float>(f - static_cast<double>(hi)));
}

// ------------------------------------------------------------------ append
// Every input may come from the launch before, which this one overlaps up to
// its wait, so none is read through the read-only path (that is for data that
// nothing writes while the kernel runs; the frequencies are such).
//
// A warp takes one token's q and a few of its heads; a CTA takes one block of 16
// slots of k or v of one (sequence, KV head), so that it sees every row that the
// block's scale depends on:
//   s = max over the block's new rows of the smallest 2^e with |x| <= 448 2^e
//   (and the scale it has, if it holds rows from before),
//   code = e4m3(x / s); rows held before are re-rounded when s has grown.
// A row is spread over hd / 4 lanes, each with two rotary pairs (p, p + 1), so
// the rotation needs no exchange: half layout dims (p, p + 1) and
// (p + rd/2, p + 1 + rd/2), interleaved layout or unrotated dims 2p .. 2p + 3.
// What bounds it is latency: the launch and one chain of length, page, rows,
// rotation and store (the bytes of the largest measured call, 8.9 MB, take 1.3
// us).  So every row of a warp is on its way at once, before the pages are
// looked at, and a block's rows are spread over four warps: a warp that took all
// 16 was a long stretch of code that ran once, and fetching it cost more than
// the work (1 x 5 tokens 5.2 us, now 2.6; two warps 3.4; eight take 64 x 5 from 6.0
// to 7.9).  Device time inside a graph, 32 query heads on 8 KV heads: 1 sequence
// x 5 tokens of head dim 128 2.6 us, 64 x 5 6.0 us, 4 x 128 tokens of head dim 64
// in fp32 4.7 us.
constexpr int kAppWarps = 4;
constexpr int kAppThreads = 32 * kAppWarps;
constexpr int kAppHeads = 4;  // head rows per lane of a q unit

SPEC_DEVINL float2 load2(const void* p, long long i, int f32) {
  if (f32) return *reinterpret_cast<const float2*>(static_cast<const float*>(p) + i);
  const uint32_t w = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p) + i);
  return make_float2(bf16lo(w), bf16hi(w));
}

// Sine and cosine of pos turns x (fr.x + fr.y): pos * fr.x = t + its rounding
// error exactly (fma), whole turns leave exactly, and the half-turn functions
// take the reduced angle within 2 ulps, so that a rotated value is off by
// little more than its own fp32 rounding at any position.  (A code is a
// rounding to 4 bits: a coarser angle moves values over its borders.)
SPEC_DEVINL void kv8_sincos(int pos, float2 fr, float* sn, float* cs) {
  const float fp = static_cast<float>(pos);
  const float t = fp * fr.x;
  const float terr = fmaf(fp, fr.x, -t) + fp * fr.y;
  sincospif(2.f * ((t - rintf(t)) + terr), sn, cs);
}

// bf16 bits of a value that may be infinite or NaN.
SPEC_DEVINL uint32_t bf16_any(float x) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(0.f), "f"(x));
  return r & 0xFFFFu;
}

struct Pair4 {  // dims d0, d0 + 1 and d1, d1 + 1 of one row
  int d0, d1;
  bool rot, inter;
  int i0;  // first pair's frequency index
};
SPEC_DEVINL Pair4 pair4(int li, int rd, int inter) {
  Pair4 q;
  q.i0 = 2 * li;
  q.rot = q.i0 < rd / 2;
  q.inter = inter || !q.rot;
  q.d0 = q.inter ? 4 * li : 2 * li;
  q.d1 = q.inter ? q.d0 + 2 : q.d0 + rd / 2;
  return q;
}
SPEC_DEVINL void rotate4(const Pair4& q, float (&x)[4], const float (&c)[2], const float (&s)[2]) {
  if (!q.rot) return;
  if (q.inter) {  // pairs (x0, x1), (x2, x3)
    const float a0 = x[0], a1 = x[2];
    x[0] = a0 * c[0] - x[1] * s[0];
    x[1] = x[1] * c[0] + a0 * s[0];
    x[2] = a1 * c[1] - x[3] * s[1];
    x[3] = x[3] * c[1] + a1 * s[1];
  } else {  // pairs (x0, x2), (x1, x3)
    const float a0 = x[0], a1 = x[1];
    x[0] = a0 * c[0] - x[2] * s[0];
    x[2] = x[2] * c[0] + a0 * s[0];
    x[1] = a1 * c[1] - x[3] * s[1];
    x[3] = x[3] * c[1] + a1 * s[1];
  }
}

template <int HD>
__global__ void __launch_bounds__(kAppThreads) kv8_append_kernel(const Kv8AppendParams p) {
  constexpr int LPR = HD / 4, RPW = 32 / LPR;
  constexpr int RPC = RPW * kAppWarps, IT = kKv8Block / RPC;  // rows of a CTA at a time
  __shared__ float s_max[kAppWarps];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, li = lane % LPR;
  const Pair4 pr = pair4(li, p.rd, p.inter);
  float2 fr[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) fr[k] = pr.rot ? __ldg(p.rope + pr.i0 + k) : make_float2(0.f, 0.f);
  const long long kv_units = 2ll * p.B * p.Hkv * p.nb;
  if (blockIdx.x >= kv_units) {  // ---- q: rotate and round to bf16
    const long long u = (blockIdx.x - kv_units) * kAppWarps + warp;
    const int sub = lane / LPR;
    const int groups = (p.H + kAppHeads * RPW - 1) / (kAppHeads * RPW);
    const int m = static_cast<int>(u / groups), g = static_cast<int>(u % groups);
    if (m >= p.B * p.n) return;
    const int b = m / p.n;
    float x[kAppHeads][4];
#pragma unroll
    for (int k = 0; k < kAppHeads; ++k) {
      const int h = (g * kAppHeads + k) * RPW + sub;
      if (h < p.H) {
        const long long at = static_cast<long long>(m) * p.q_ld + h * HD;
        const float2 a = load2(p.q, at + pr.d0, p.f32), c = load2(p.q, at + pr.d1, p.f32);
        x[k][0] = a.x, x[k][1] = a.y, x[k][2] = c.x, x[k][3] = c.y;
      }
    }
    const int pos = p.base[b] + (p.depth ? p.depth[m] : m - b * p.n);
    float cs[2], sn[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) kv8_sincos(pos, fr[k], &sn[k], &cs[k]);
#pragma unroll
    for (int k = 0; k < kAppHeads; ++k) {
      const int h = (g * kAppHeads + k) * RPW + sub;
      if (h >= p.H) continue;
      rotate4(pr, x[k], cs, sn);
      uint16_t* o = p.q_out + (static_cast<long long>(m) * p.H + h) * HD;
      *reinterpret_cast<uint32_t*>(o + pr.d0) = bf16_any(x[k][0]) | (bf16_any(x[k][1]) << 16);
      *reinterpret_cast<uint32_t*>(o + pr.d1) = bf16_any(x[k][2]) | (bf16_any(x[k][3]) << 16);
    }
    return;
  }
  // ---- one block of 16 slots of k (which 0) or v (1)
  int u = blockIdx.x;
  const int which = u & 1;
  u >>= 1;
  const int h = u % p.Hkv;
  u /= p.Hkv;
  const int blk_i = u % p.nb, b = u / p.nb;
  const int row0 = warp * RPW + lane / LPR;  // the thread's rows: row0 + i RPC
  const int L = p.base[b];
  if (p.seq_ok && !p.seq_ok[b]) return;  // flagged when the pass began
  if (L < 0 || L > p.max_pages * kPageSlots - p.n) {
    if (threadIdx.x == 0) set_status(p.status, SPEC_DEV_KV_OVERFLOW);
    return;
  }
  const int slot0 = (L / kKv8Block + blk_i) * kKv8Block;  // the block's first slot
  if (slot0 >= L + p.n) return;
  const void* src = which ? p.v : p.k;
  const long long ld = which ? p.v_ld : p.k_ld;
  const Pair4 at = which ? pair4(li, 0, 1) : pr;
  float x[IT][4];  // (on their way before the pages are looked at)
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int j = slot0 + i * RPC + row0 - L;  // the row's token
    x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.f;
    if (j >= 0 && j < p.n) {
      const long long o = (static_cast<long long>(b) * p.n + j) * ld + h * HD;
      const float2 a = load2(src, o + at.d0, p.f32), c = load2(src, o + at.d1, p.f32);
      x[i][0] = a.x, x[i][1] = a.y, x[i][2] = c.x, x[i][3] = c.y;
    }
  }
  int page;
  if (const int32_t bad = kv8_fit_warp(L, p.n, p.table, p.max_pages, p.n_pages, b, slot0, &page)) {
    if (threadIdx.x == 0) set_status(p.status, bad);
    return;
  }
  const Kv8Map map{p.table, p.max_pages, p.n_pages, p.Hkv, HD};
  float* sp = (which ? p.vs : p.ks) + map.scale(page, h, slot0);
  const int kept = max(0, L - slot0);  // rows the block holds from before
  const float s_held = kept ? *sp : 0.f;
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int j = slot0 + i * RPC + row0 - L;
    if (at.rot && j >= 0 && j < p.n) {
      const int pos = L + (p.depth ? p.depth[b * p.n + j] : j);
      float cs[2], sn[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) kv8_sincos(pos, fr[k], &sn[k], &cs[k]);
      rotate4(at, x[i], cs, sn);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float a = fabsf(x[i][k]);
      if (a <= 3.402823466e38f) amax = fmaxf(amax, a);  // finite values alone set the scale
    }
  }
  amax = warp_max(amax);
  if (lane == 0) s_max[warp] = amax;
  __syncthreads();  // (and every thread has read the scale before it is replaced)
#pragma unroll
  for (int k = 0; k < kAppWarps; ++k) amax = fmaxf(amax, s_max[k]);
  uint8_t* codes = (which ? p.vc : p.kc) + map.row(page, h, slot0);
  const float s_new = kv8_scale(amax);
  const float s = kept ? fmaxf(s_new, s_held) : s_new;
  const float s_old = kept ? s_held : s;
  const float inv = pow2_inv(s), ratio = s_old * inv;
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int r = i * RPC + row0, j = slot0 + r - L;
    uint8_t* row = codes + static_cast<long long>(r) * HD;
    if (j >= 0 && j < p.n) {
      const uint32_t w = e4m3x4(x[i][0] * inv, x[i][1] * inv, x[i][2] * inv, x[i][3] * inv);
      if (at.inter) {
        *reinterpret_cast<uint32_t*>(row + at.d0) = w;
      } else {
        *reinterpret_cast<uint16_t*>(row + at.d0) = static_cast<uint16_t>(w);
        *reinterpret_cast<uint16_t*>(row + at.d1) = static_cast<uint16_t>(w >> 16);
      }
    } else if (r < kept && ratio < 1.f) {
      uint32_t* w = reinterpret_cast<uint32_t*>(row + 4 * li);
      *w = kv8_rescale4(*w, ratio);
    }
  }
  if (threadIdx.x == 0) *sp = s;
}

// ------------------------------------------------------------------ commit
// Moves the accepted path's rows L0 + path[d - 1] -> L0 + d (d = 1 .. m) of one
// (sequence, KV head), keys and values, in up to kMoveLayers layers.  A
// destination block's scale is the largest of those its rows come with: the
// rows moved in, and its own if it keeps rows (slots up to the root, L0).
// Every row of a layer is read before any is written: rows and scales go
// through registers and shared memory.  What bounds it is the chain of round
// trips (length, path, page, row); a path of a few rows leaves a thread one
// 16-byte word a layer, so a CTA takes a few layers at once.  With the length
// update and a copy that puts the lengths back, 1 sequence of 7 nodes / 16 of 33,
// 32 layers: eight layers of eight words a thread 6.8 / 9.9 us, four of four 6.2 /
// 9.0, two of eight (128 threads) 6.3 / 11.0; one layer a CTA took 16.4 for the 16.
constexpr int kMoveThreads = 256;
constexpr int kMoveLayers = 4;
constexpr int kMoveWords = 4;                                                 // 16-byte words per thread
constexpr int kMoveBlocks = (kTreeMaxNodes + 2 * kKv8Block - 2) / kKv8Block;  // blocks n slots can touch

// 0 when the path of sequence b can be committed, else the status bit (the
// same for every lane of the warp).
SPEC_DEVINL int32_t kv8_path_bad(const Kv8CommitParams& p, int b, int len, int m) {
  static_assert(kTreeMaxNodes <= 64, "two nodes a lane");
  if (m < 0 || m >= p.n) return SPEC_DEV_BAD_TREE;
  const int32_t* path = p.path + static_cast<long long>(b) * p.n;
  const int lane = threadIdx.x & 31;
  bool bad = false;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int d = lane + 32 * k;
    if (d < m) {
      const int s = path[d];
      bad |= s <= (d ? path[d - 1] : 0) || s >= p.n;
    }
  }
  if (__any_sync(0xffffffffu, bad)) return SPEC_DEV_BAD_TREE;
  if (len < p.n) return SPEC_DEV_KV_OVERFLOW;
  int page;
  return kv8_fit_warp(len - p.n, p.n, p.table, p.max_pages, p.n_pages, b, len - p.n, &page);
}

template <int HD>
__global__ void __launch_bounds__(kMoveThreads) kv8_commit_kernel(const Kv8CommitParams p) {
  constexpr int VEC = HD / 16;  // 16-byte words per row
  static_assert(2 * (kTreeMaxNodes - 1) * VEC <= kMoveWords * kMoveThreads, "a layer fits the registers");
  __shared__ float s_src[kMoveLayers][2][kTreeMaxNodes], s_dst[kMoveLayers][2][kMoveBlocks], s_own[kMoveLayers][2];
  grid_dep_wait();
  grid_dep_launch();
  const int b = blockIdx.x / p.Hkv, h = blockIdx.x % p.Hkv;
  const int tid = threadIdx.x;
  const int len = p.len[b], m = p.n_acc[b];
  if (m <= 0 || kv8_path_bad(p, b, len, m)) return;  // the length update reports it
  const int L0 = len - p.n;
  const int32_t* path = p.path + static_cast<long long>(b) * p.n;
  const Kv8Map map{p.table, p.max_pages, p.n_pages, p.Hkv, HD};
  const long long layer_rows = static_cast<long long>(p.n_pages) * p.Hkv * kPageSlots;
  const auto codes = [&](int side, int layer) { return (side ? p.vc : p.kc) + layer * layer_rows * HD; };
  const auto scales = [&](int side, int layer) { return (side ? p.vs : p.ks) + layer * (layer_rows / kKv8Block); };
  const int per_side = m * VEC, per_layer = 2 * per_side;
  const int blk0 = L0 / kKv8Block, nblk = (L0 + m) / kKv8Block - blk0 + 1;
  const int last = min(p.L, static_cast<int>(blockIdx.y + 1) * kMoveLayers);
  const int at_once = min(kMoveLayers, kMoveWords * kMoveThreads / per_layer);
  for (int layer0 = blockIdx.y * kMoveLayers; layer0 < last; layer0 += at_once) {
    const int nl = min(at_once, last - layer0);
    uint4 w[kMoveWords];
#pragma unroll
    for (int k = 0; k < kMoveWords; ++k) {
      const int e = tid + k * kMoveThreads;
      if (e < nl * per_layer) {
        const int l = e / per_layer, f = e - l * per_layer, side = f >= per_side, rem = f - side * per_side;
        const int src = L0 + path[rem / VEC];
        w[k] = reinterpret_cast<const uint4*>(codes(side, layer0 + l) + map.row(map.page(b, src), h, src))[rem % VEC];
      }
    }
    for (int e = tid; e < nl * 2 * m; e += kMoveThreads) {
      const int l = e / (2 * m), f = e - l * 2 * m, side = f >= m, d = f - side * m;
      const int src = L0 + path[d];
      s_src[l][side][d] = scales(side, layer0 + l)[map.scale(map.page(b, src), h, src)];
    }
    if (tid < 2 * nl) s_own[tid / 2][tid % 2] = scales(tid % 2, layer0 + tid / 2)[map.scale(map.page(b, L0), h, L0)];
    __syncthreads();
    for (int e = tid; e < nl * 2 * nblk; e += kMoveThreads) {
      const int l = e / (2 * nblk), f = e - l * 2 * nblk, side = f >= nblk, i = f - side * nblk;
      const int d0 = max(1, (blk0 + i) * kKv8Block - L0), d1 = min(m, (blk0 + i + 1) * kKv8Block - 1 - L0);
      float s = i == 0 ? s_own[l][side] : 0.f;  // the root's block keeps rows
      for (int d = d0; d <= d1; ++d) s = fmaxf(s, s_src[l][side][d - 1]);
      s_dst[l][side][i] = s;
      if (d0 <= d1) {
        const int t = (blk0 + i) * kKv8Block;
        scales(side, layer0 + l)[map.scale(map.page(b, t), h, t)] = s;
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kMoveWords; ++k) {
      const int e = tid + k * kMoveThreads;
      if (e >= nl * per_layer) continue;
      const int l = e / per_layer, f = e - l * per_layer, side = f >= per_side, rem = f - side * per_side;
      const int d = rem / VEC + 1;
      const float ratio = s_src[l][side][d - 1] * pow2_inv(s_dst[l][side][(L0 + d) / kKv8Block - blk0]);
      uint4 v = w[k];
      if (ratio < 1.f)
        v = make_uint4(kv8_rescale4(v.x, ratio), kv8_rescale4(v.y, ratio), kv8_rescale4(v.z, ratio),
                       kv8_rescale4(v.w, ratio));
      reinterpret_cast<uint4*>(codes(side, layer0 + l) + map.row(map.page(b, L0 + d), h, L0 + d))[rem % VEC] = v;
    }
    // rows that the root's block holds, if its scale has grown
    const int t0 = blk0 * kKv8Block, kept = L0 - t0 + 1;
    for (int e = tid; e < nl * 2 * kept * VEC; e += kMoveThreads) {
      const int l = e / (2 * kept * VEC), f = e - l * 2 * kept * VEC;
      const int side = f >= kept * VEC, rem = f - side * kept * VEC;
      const float ratio = s_own[l][side] * pow2_inv(s_dst[l][side][0]);
      if (ratio >= 1.f) continue;
      const int t = t0 + rem / VEC;
      uint4* a = reinterpret_cast<uint4*>(codes(side, layer0 + l) + map.row(map.page(b, t), h, t)) + rem % VEC;
      const uint4 v = *a;
      *a = make_uint4(kv8_rescale4(v.x, ratio), kv8_rescale4(v.y, ratio), kv8_rescale4(v.z, ratio),
                      kv8_rescale4(v.w, ratio));
    }
    __syncthreads();  // the scales in shared memory are the next layers'
  }
}

// len = L0 + 1 + m, after the copies (a launch of its own: they read len); a
// warp per sequence.
__global__ void kv8_commit_len_kernel(const Kv8CommitParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const int b = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
  if (b >= p.B) return;
  const int len = p.len[b], m = p.n_acc[b];
  const int32_t bad = kv8_path_bad(p, b, len, m);
  if (threadIdx.x % 32) return;
  if (bad)
    set_status(p.status, bad);
  else
    p.len[b] = len - p.n + 1 + m;
}

// len += n for every sequence whose slots and pages (all of [0, len + n)) are
// in order; a warp per sequence, which looks at 32 pages at a time: 2.0 us for 64
// sequences of 4000 slots, 4.7 us for one of 131000 (2048 pages).
__global__ void kv8_advance_kernel(int32_t* len, const int32_t* table, int B, int n, int max_pages, int n_pages,
                                   int32_t* status) {
  grid_dep_wait();
  grid_dep_launch();
  const int b = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32, lane = threadIdx.x % 32;
  if (b >= B) return;
  const int L = len[b];
  int32_t bad = L < 0 || L > max_pages * kPageSlots - n ? SPEC_DEV_KV_OVERFLOW : 0;
  if (!bad) {
    const int32_t* row = table + static_cast<long long>(b) * max_pages;
    const int np = (L + n + kPageSlots - 1) / kPageSlots;
    bool out = false;
#pragma unroll 4
    for (int j = lane; j < np; j += 32) out |= row[j] < 0 || row[j] >= n_pages;
    if (__any_sync(0xffffffffu, out)) bad = SPEC_DEV_BAD_PAGE;
  }
  if (lane) return;
  if (bad)
    set_status(status, bad);
  else
    len[b] = L + n;
}

template <class... A>
cudaError_t launch_dep(void (*fn)(A...), dim3 grid, int threads, cudaStream_t stream, A... a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, a...);
}

}  // namespace

cudaError_t launch_kv8_rope(float2* dst, int rd, double theta, double factor, double low, double high, int orig_len,
                            cudaStream_t stream) {
  kv8_rope_kernel<<<(rd / 2 + 63) / 64, 64, 0, stream>>>(dst, rd, theta, factor, low, high, orig_len);
  return cudaGetLastError();
}

cudaError_t launch_kv8_append(const Kv8AppendParams& p, cudaStream_t stream) {
  const int rpw = 32 / (p.hd / 4);
  const long long q_units = static_cast<long long>(p.B) * p.n * ((p.H + kAppHeads * rpw - 1) / (kAppHeads * rpw));
  const long long grid = 2ll * p.B * p.Hkv * p.nb + (q_units + kAppWarps - 1) / kAppWarps;
  if (grid > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  return launch_dep(p.hd == 128 ? kv8_append_kernel<128> : kv8_append_kernel<64>, dim3(static_cast<unsigned>(grid)),
                    kAppThreads, stream, p);
}

cudaError_t launch_kv8_commit(const Kv8CommitParams& p, cudaStream_t stream) {
  if (p.n > 1) {
    const cudaError_t e = launch_dep(p.hd == 128 ? kv8_commit_kernel<128> : kv8_commit_kernel<64>,
                                     dim3(p.B * p.Hkv, (p.L + kMoveLayers - 1) / kMoveLayers), kMoveThreads, stream, p);
    if (e != cudaSuccess) return e;
  }
  return launch_dep(kv8_commit_len_kernel, dim3((p.B + 3) / 4), 128, stream, p);
}

cudaError_t launch_kv8_advance(int32_t* len, const int32_t* table, int B, int n, int max_pages, int n_pages,
                               int32_t* status, cudaStream_t stream) {
  return launch_dep(kv8_advance_kernel, dim3((B + 3) / 4), 128, stream, len, table, B, n, max_pages, n_pages,
                    status);
}

}  // namespace spec
