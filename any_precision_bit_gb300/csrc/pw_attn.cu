// pw_attn.cu -- attention over the paged key/value cache.
#include <cuda_runtime.h>

#include "pw_attn.h"
#include "pw_device.cuh"

namespace pw {

template <bool BF>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (BF) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  const __half2 h = *reinterpret_cast<const __half2 *>(&w);
  return __half22float2(h);
}
template <bool BF>
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
  uint32_t r;
  if (BF)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// One row (token t, query head h) over the keys [lo, hi) of its table row, by one warp: lane l
// holds elements 4 l .. 4 l + 3 of the head.  The running maximum and sum of a softmax in fp32;
// only visible keys and values are read.  acc is the normalised output, *lse the natural
// log-sum-exp (-inf and zeros for a row without keys).
template <bool BF>
__device__ void row_attention(const AttnArgs &a, int t, int h, int lo, int hi, int trow, int pos, float (&acc)[4],
                              float *lse) {
  const int lane = threadIdx.x & 31, d = 4 * lane;
  const bool mine = d < a.D;
  float qf[4] = {0.f, 0.f, 0.f, 0.f};
  if (mine) {
    const uint2 w = *reinterpret_cast<const uint2 *>(a.q + t * a.q_token + h * a.q_head + d);
    const float2 x = unpack2<BF>(w.x), y = unpack2<BF>(w.y);
    qf[0] = x.x, qf[1] = x.y, qf[2] = y.x, qf[3] = y.y;
  }
  const int hk = h / a.G, mask = (1 << a.log_bt) - 1;
  const float slope = a.slopes ? a.slopes[h] : 0.f;
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = 0.f;
  for (int j = lo; j < hi; ++j) {
    const int page = j >> a.log_bt;
    const int id = trow >= 0 && page < a.table_stride ? a.table[(size_t)trow * a.table_stride + page] : -1;
    uint2 kw{0u, 0u}, vw{0u, 0u};
    if (mine && id >= 0 && id < a.n_blocks) {
      const int64_t at = id * a.block_stride + (j & mask) * a.token_stride + hk * a.head_stride + d;
      kw = *reinterpret_cast<const uint2 *>(a.kc + at);
      vw = *reinterpret_cast<const uint2 *>(a.vc + at);
    }
    const float2 k0 = unpack2<BF>(kw.x), k1 = unpack2<BF>(kw.y);
    float s = qf[0] * k0.x + qf[1] * k0.y + qf[2] * k1.x + qf[3] * k1.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    s *= a.scale;
    if (a.softcap > 0.f) s = a.softcap * tanhf(s / a.softcap);
    if (a.slopes) s -= slope * fabsf((float)(pos - j));
    const float mn = fmaxf(m, s), ms = mn == -INFINITY ? 0.f : mn;
    const float f = expf(m - ms), p = expf(s - ms);
    m = mn;
    l = l * f + p;
    const float2 v0 = unpack2<BF>(vw.x), v1 = unpack2<BF>(vw.y);
    acc[0] = acc[0] * f + p * v0.x;
    acc[1] = acc[1] * f + p * v0.y;
    acc[2] = acc[2] * f + p * v1.x;
    acc[3] = acc[3] * f + p * v1.y;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] *= inv;
  *lse = m + logf(l);
}

template <bool BF>
__global__ void __launch_bounds__(256) attn_rows_kernel(AttnArgs a) {
  const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (w >= (long long)a.n_tokens * a.Hq) return;
  const int t = (int)(w / a.Hq), h = (int)(w - (long long)t * a.Hq), lane = threadIdx.x & 31;
  const RowBound b = a.bounds[t];
  float acc[4], lse;
  row_attention<BF>(a, t, h, b.lo, b.hi, b.trow, b.pos, acc, &lse);
  if (4 * lane < a.D) {
    const uint2 out{pack_pair<BF>(acc[0], acc[1]), pack_pair<BF>(acc[2], acc[3])};
    *reinterpret_cast<uint2 *>(a.o + t * a.o_token + h * a.o_head + 4 * lane) = out;
  }
  if (a.lse && lane == 0) a.lse[w] = lse;
}

int launch_attn(const AttnArgs &a, int bf16, void *stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const long long rows = (long long)a.n_tokens * a.Hq;
  const unsigned grid = (unsigned)((rows + 7) / 8);
  if (bf16)
    attn_rows_kernel<true><<<grid, 256, 0, st>>>(a);
  else
    attn_rows_kernel<false><<<grid, 256, 0, st>>>(a);
  return (int)cudaGetLastError();
}

}  // namespace pw
