// Attention of n new positions over the 8-bit paged KV cache.
//   s_j = scale * q . (ks_j k_j),  o = sum_j p_j vs_j v_j / sum_j p_j,
//   p_j = exp(s_j - max s) over the slots that the row's token may see
// (the cached ones, and of the new ones its own and earlier, or those of its
// ancestor mask); a row that sees nothing is zero.
#include "internal.h"
#include "kv8_common.cuh"

namespace spec {
namespace {

// One CTA per (sequence, query row): a thread scores one key of a block of
// 128, then owns one output dimension.
constexpr int kRowThreads = 128;

template <int HD>
__global__ void __launch_bounds__(kRowThreads) kv8_attention_kernel(const Kv8AttnParams p) {
  __shared__ float sq[HD], sp[kRowThreads], red[4];
  grid_dep_wait();
  grid_dep_launch();
  const int row = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;  // row = token j, head hq
  const int j = row / p.H, hq = row % p.H, h = hq / (p.H / p.Hkv);
  const int L = p.base[b];
  const long long m = static_cast<long long>(b) * p.n + j;
  uint16_t* out = p.o + m * p.o_ld + hq * HD;
  const int32_t bad = kv8_fit(L, p.n, p.table, p.max_pages, p.n_pages, b);
  if (bad) {
    if (tid == 0) set_status(p.status, bad);
    if (tid < HD) out[tid] = 0;
    return;
  }
  const Kv8Map map{p.table, p.max_pages, p.n_pages, p.Hkv, HD};
  if (tid < HD) sq[tid] = bf16_to_f32(p.q[m * p.q_ld + hq * HD + tid]) * p.scale_log2;
  const uint64_t am = p.anc ? p.anc[m] : 0ull;
  __syncthreads();
  float mx = -INFINITY, l = 0.f, acc = 0.f;
  const int T = L + p.n;
  for (int t0 = 0; t0 < T; t0 += kRowThreads) {
    const int t = t0 + tid;
    const bool see = t < T && key_visible(t, L, j, p.anc, am);
    float s = -INFINITY;
    if (see) {
      const int pg = map.page(b, t);
      const uint32_t* k = reinterpret_cast<const uint32_t*>(p.kc + map.row(pg, h, t));
      float d = 0.f;
      for (int c = 0; c < HD / 4; ++c) {
        const float2 x = e4m3x2_to_f32(k[c]), y = e4m3x2_to_f32(k[c] >> 16);
        d += x.x * sq[4 * c] + x.y * sq[4 * c + 1] + y.x * sq[4 * c + 2] + y.y * sq[4 * c + 3];
      }
      s = d * p.ks[map.scale(pg, h, t)];
    }
    float w = warp_max(s);
    if ((tid & 31) == 0) red[tid >> 5] = w;
    __syncthreads();
    const float mn = fmaxf(mx, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float alpha = mx == -INFINITY ? 0.f : exp2f(mx - mn);
    mx = mn;
    const float e = see ? exp2f(s - mn) : 0.f;
    sp[tid] = e;
    l = l * alpha + e;
    __syncthreads();
    if (tid < HD) {
      acc *= alpha;
      for (int i = 0; i < min(kRowThreads, T - t0); ++i) {
        if (!key_visible(t0 + i, L, j, p.anc, am)) continue;
        const int pg = map.page(b, t0 + i);
        const float v = e4m3x2_to_f32(p.vc[map.row(pg, h, t0 + i) + tid]).x;
        acc += sp[i] * v * p.vs[map.scale(pg, h, t0 + i)];
      }
    }
    __syncthreads();
  }
  l = warp_sum(l);
  if ((tid & 31) == 0) red[tid >> 5] = l;
  __syncthreads();
  const float lt = (red[0] + red[1]) + (red[2] + red[3]);
  if (tid < HD) {
    const float o = lt == 0.f ? 0.f : acc / lt;
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(0.f), "f"(o));
    out[tid] = static_cast<uint16_t>(r);
  }
}

}  // namespace

cudaError_t launch_kv8_attention(const Kv8AttnParams& p, cudaStream_t stream) {
  if (p.hd == 128)
    kv8_attention_kernel<128><<<dim3(p.n * p.H, p.B), kRowThreads, 0, stream>>>(p);
  else
    kv8_attention_kernel<64><<<dim3(p.n * p.H, p.B), kRowThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace spec
