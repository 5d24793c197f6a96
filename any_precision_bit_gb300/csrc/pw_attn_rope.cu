// pw_attn_rope.cu -- norms and rotation of queries and keys, and the cache write, in one pass over a step's rows.
//
// A head x of q or k becomes y = x rsqrt(mean x^2 + eps) gain, and each of its pairs (a, b) becomes s (a cos f - b sin f,
// a sin f + b cos f), f = p inv_freq.  The host turns inv_freq / 2 pi into a 64-bit fraction of a turn, so that the product
// with the integer position modulo 2^64 is the angle's fraction of a turn at any position, exactly; in fp32 the product alone is
// off by 2^-24 p radians.  Its upper 32 bits give the nearest quarter turn and a rest of at most 1/8 turn for two short
// polynomials.
#include <cuda_runtime.h>

#include "pw_attn.h"
#include "pw_device.cuh"

namespace pw {

constexpr int kRopeThreads = 256;

// Sine and cosine of 2 pi h 2^-32: their Taylor polynomials in x, |x| <= pi / 4 (x^11 / 11! < 2^-29, x^10 / 10! < 2^-25),
// turned back by quarters.
__device__ __forceinline__ void sincos_turn(uint32_t h, float &s, float &c) {
  const uint32_t quarter = (h + 0x20000000u) >> 30;
  const float x = (float)(int)(h - (quarter << 30)) * 1.46291807926715968e-9f, u = x * x;  // 2 pi 2^-32
  float ps = fmaf(u, 2.755731922e-6f, -1.984126984e-4f);
  ps = fmaf(ps, u, 8.333333333e-3f);
  ps = fmaf(ps, u, -1.666666667e-1f);
  ps = fmaf(ps * u, x, x);
  float pc = fmaf(u, 2.480158730e-5f, -1.388888889e-3f);
  pc = fmaf(pc, u, 4.166666667e-2f);
  pc = fmaf(pc, u, -0.5f);
  pc = fmaf(pc, u, 1.f);
  const float a = quarter & 1 ? pc : ps, b = quarter & 1 ? ps : pc;
  s = quarter & 2 ? -a : a;
  c = (quarter + 1) & 2 ? -b : b;
}

template <bool BF>
__device__ __forceinline__ float2 to_floats(uint32_t w) {
  if (BF) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  const __half2 h = *reinterpret_cast<const __half2 *>(&w);
  return __half22float2(h);
}
template <bool BF>
__device__ __forceinline__ uint32_t from_floats(float lo, float hi) {
  uint32_t r;
  if (BF)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// P elements, in one load or store.
template <int P>
struct Piece16 {
  uint32_t w[P / 2];
};
template <int P>
__device__ __forceinline__ Piece16<P> load_piece(const uint16_t *p) {
  Piece16<P> r;
  if constexpr (P == 8) {
    const uint4 x = *reinterpret_cast<const uint4 *>(p);
    r.w[0] = x.x, r.w[1] = x.y, r.w[2] = x.z, r.w[3] = x.w;
  } else {
    const uint2 x = *reinterpret_cast<const uint2 *>(p);
    r.w[0] = x.x, r.w[1] = x.y;
  }
  return r;
}
template <int P>
__device__ __forceinline__ void store_piece(uint16_t *p, const Piece16<P> &r) {
  if constexpr (P == 8)
    *reinterpret_cast<uint4 *>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
  else
    *reinterpret_cast<uint2 *>(p) = make_uint2(r.w[0], r.w[1]);
}

// GL lanes to a head, each with two pieces of P elements: the two halves of P pairs (IL: or, side by side, 2 P elements that
// are P pairs).  A warp takes U of its 32 / GL heads at a time, all of them heads of q, or of k, or of v; `parts` warps
// share a token's.
template <bool BF, int P, int GL, bool IL>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a, int parts) {
  constexpr int U = 2, kHeads = 32 / GL * U;  // heads that a warp takes at a time
  const int lane = threadIdx.x & 31, sub = lane / GL, l = lane % GL;
  const unsigned item = blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);  // at most 2^20 tokens, 768 parts
  const int t = (int)(item / (unsigned)parts), part = (int)(item - (unsigned)t * parts);
  // this lane's pieces, and whether they are turned
  const int rot_lanes = IL ? 0 : a.rot / (2 * P);
  const bool turn0 = IL ? 2 * P * l < a.rot : l < rot_lanes, turn1 = IL ? 2 * P * l + P < a.rot : turn0;
  const int at0 = !IL && turn0 ? P * l : 2 * P * l;  // (behind the turned ones: rot + 2 P (l - rot / 2 P))
  const int at1 = !IL && turn0 ? a.rot / 2 + P * l : 2 * P * l + P;
  const bool has0 = at0 < a.D, has1 = at1 < a.D;
  pdl_trigger();
  uint64_t f[P];
  int axis[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {  // (set long before this launch)
    const bool on = IL && i >= P / 2 ? turn1 : turn0;
    f[i] = on ? a.table->turn[P * l + i] : 0;
    axis[i] = on ? a.table->axis[P * l + i] : 0;
  }
  pdl_wait();
  if (t >= a.n_tokens) return;
  const int64_t slot = a.slot[t];
  if (slot < 0) return;
  const bool stored = slot >> a.log_bt < a.n_blocks;
  const int64_t place = (slot >> a.log_bt) * a.block_stride + (slot & (a.bt - 1)) * a.token_stride;
  float sn[P], cs[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int p = a.pos[axis[i] * a.pos_axis + t];
    sincos_turn((uint32_t)(f[i] * (uint64_t)(int64_t)p >> 32), sn[i], cs[i]);
    sn[i] *= a.scale;
    cs[i] *= a.scale;
  }
  const int nq = (a.Hq + kHeads - 1) / kHeads, nk = (a.Hkv + kHeads - 1) / kHeads;
  for (int c = part; c < nq + 2 * nk; c += parts) {
    const int kind = c < nq ? 0 : c < nq + nk ? 1 : 2;
    const int h0 = (kind == 0 ? c : kind == 1 ? c - nq : c - nq - nk) * kHeads + sub, H = kind == 0 ? a.Hq : a.Hkv;
    const uint16_t *src = kind == 0 ? a.q + t * a.q_token : kind == 1 ? a.k + t * a.k_token : a.v + t * a.v_token;
    const int64_t src_head = kind == 0 ? a.q_head : kind == 1 ? a.k_head : a.v_head;
    uint16_t *dst = kind == 0 ? a.qo + t * a.qo_token : kind == 1 ? a.kc + place : a.vc + place;
    const int64_t dst_head = kind == 0 ? a.qo_head : a.head_stride;
    Piece16<P> x[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * (32 / GL);
      x[u][0] = x[u][1] = Piece16<P>{};
      if (h < H && has0) x[u][0] = load_piece<P>(src + h * src_head + at0);
      if (h < H && has1) x[u][1] = load_piece<P>(src + h * src_head + at1);
    }
    const bool norm = kind == 0 ? a.norm_q : kind == 1 && a.norm_k;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * (32 / GL);
      if (kind < 2) {
        float y[2][P];
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int i = 0; i < P; i += 2) {
            const float2 z = to_floats<BF>(x[u][s].w[i / 2]);
            y[s][i] = z.x, y[s][i + 1] = z.y;
          }
        if (norm) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < P; ++i) ss = fmaf(y[0][i], y[0][i], fmaf(y[1][i], y[1][i], ss));
#pragma unroll
          for (int o = 1; o < GL; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float r = rsqrtf(fmaf(ss, a.inv_d, a.eps));
          const float *g = a.table->gain[kind];
#pragma unroll
          for (int i = 0; i < P; ++i) {
            if (has0) y[0][i] *= r * g[at0 + i];
            if (has1) y[1][i] *= r * g[at1 + i];
          }
        }
        if (IL) {
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < P; i += 2) {
              if (!(s ? turn1 : turn0)) continue;  // (0 times what is not turned may be NaN)
              const int j = s * (P / 2) + i / 2;
              const float p = y[s][i], q = y[s][i + 1];
              y[s][i] = fmaf(p, cs[j], -q * sn[j]);
              y[s][i + 1] = fmaf(p, sn[j], q * cs[j]);
            }
        } else if (turn0) {
#pragma unroll
          for (int i = 0; i < P; ++i) {
            const float p = y[0][i], q = y[1][i];
            y[0][i] = fmaf(p, cs[i], -q * sn[i]);
            y[1][i] = fmaf(p, sn[i], q * cs[i]);
          }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int i = 0; i < P; i += 2) x[u][s].w[i / 2] = from_floats<BF>(y[s][i], y[s][i + 1]);
      }
      if (h < H && (kind == 0 || stored)) {
        if (has0) store_piece<P>(dst + h * dst_head + at0, x[u][0]);
        if (has1) store_piece<P>(dst + h * dst_head + at1, x[u][1]);
      }
    }
  }
}

template <bool BF, int P, int GL, bool IL>
static int launch_one(const RopeArgs &a, cudaStream_t st) {
  constexpr int kHeads = 32 / GL * 2;
  const int parts = (a.Hq + kHeads - 1) / kHeads + 2 * ((a.Hkv + kHeads - 1) / kHeads);
  const int64_t warps = (int64_t)a.n_tokens * parts, per = kRopeThreads / 32;
  return (int)launch_pdl(rope_kernel<BF, P, GL, IL>, dim3((unsigned)((warps + per - 1) / per)), dim3(kRopeThreads), 0, st, a,
                         parts);
}
template <bool BF>
static int launch_type(const RopeArgs &a, cudaStream_t st) {
  if (a.interleaved) {
    const int lanes = (a.D + 15) / 16;
    return lanes <= 4 ? launch_one<BF, 8, 4, true>(a, st) : launch_one<BF, 8, 8, true>(a, st);
  }
  // halves of whole 16-byte pieces, or of 8-byte ones
  if (a.rot % 16 == 0) {
    const int lanes = a.rot / 16 + (a.D - a.rot + 15) / 16;
    return lanes <= 4 ? launch_one<BF, 8, 4, false>(a, st) : launch_one<BF, 8, 8, false>(a, st);
  }
  return launch_one<BF, 4, 16, false>(a, st);
}

int launch_rope(const RopeArgs &a, int bf16, void *stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return bf16 ? launch_type<true>(a, st) : launch_type<false>(a, st);
}

}  // namespace pw
