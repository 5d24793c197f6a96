// pw_attn_rope.cu -- norms and rotation of queries and keys, and the cache write, in one pass over a step's rows.
//
// A head x of q or k becomes y = x rsqrt(mean x^2 + eps) gain, and each of its pairs (a, b) becomes s (a cos f - b sin f,
// a sin f + b cos f), f = p inv_freq.  The host turns inv_freq / 2 pi into the nearest 64-bit fraction of a turn, off by at most 2^-65,
// so that the product with the integer position modulo 2^64 is the angle's fraction of a turn to 2^-34 at any position; in fp32 the
// product alone is off by 2^-24 p radians.  Its upper 32 bits give the nearest quarter turn and a rest of at most 1/8 turn for
// two short polynomials.  What was cut off is less than 2^-31.6 of a turn, 2 10^-9; with the polynomials' fp32 steps sine and cosine are
// off by less than 2^-22 (2^-23.3 at most among 4 10^7 random angles, the same steps restated on the host).
#include <cuda_runtime.h>

#include "pw_attn.h"
#include "pw_device.cuh"

namespace pw {

constexpr int kRopeThreads = 128;

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

// 2 N floats as pairs, or zeros.
template <int N>
__device__ __forceinline__ void load_pairs(const float *p, bool there, uint64_t (&out)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float4 x = there ? *reinterpret_cast<const float4 *>(p + 2 * i) : make_float4(0.f, 0.f, 0.f, 0.f);
    out[i] = pair(x.x, x.y);
    out[i + 1] = pair(x.z, x.w);
  }
}

// A CTA takes a few tokens.  Their angles' sines and cosines, which all heads share, come first, to shared memory (computed by
// every warp for its heads they were a third of the instructions); the rows' first loads are under way by then.  GL lanes
// have a head, each two pieces of P elements: the two halves of P pairs (IL: or, side by side, 2 P elements that are P
// pairs).  A warp takes kRopeHeads heads for each GL lanes at a time, all of q, or of k, or of v, so that it has one kind of
// address and of work.
//
// Memory bounds it where heads are many: 8205 tokens of 32/8 heads of 128 with norms, 202 MB, take 37.3 us (5.4 TB/s;
// interleaved 38.7), 30000 tokens 121 us (6.1 TB/s, 90 % of a copy's rate: the rest of the shorter kernel is its beginning and end),
// 5003 of 16/16 heads of 96, 92 MB, 17.6 us.  With few heads most places of a chunk are empty, one key/value head in 16 or 32:
// 8/1 heads of 128 and 16/2 of 64 2.5 to 3.0 TB/s; heads of 72 fill five lanes of eight, 28/4 of them 2.8 to 3.2.
// The first two by 2 heads at a time 39 and 21 us, by 3 or 6 CTAs an SM 38 to 41 and 19; one token to a CTA 39 and 21, 5 or 8 tokens 42 and 18 to 20, where the last CTAs
// run alone.  With the slot's, the positions' and the rows' loads behind each other it took 62 us.
constexpr int kRopeHeads = 4, kRopeTokens = 4, kPairs = 64, kRopeCtas = 5;
template <bool BF, int P, int GL, bool IL>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) rope_kernel(const __grid_constant__ RopeArgs a, int tokens) {
  constexpr int U = kRopeHeads, S = 32 / GL, Q = P / 2;
  __shared__ __align__(16) float cos_of[kRopeTokens][kPairs], sin_of[kRopeTokens][kPairs];
  const int lane = threadIdx.x & 31, sub = lane / GL, l = lane % GL, pair_of = threadIdx.x % kPairs;
  // this lane's pieces, and whether they are turned
  const bool turn0 = 2 * P * l < a.rot, turn1 = IL ? 2 * P * l + P < a.rot : turn0;
  const int at0 = !IL && turn0 ? P * l : 2 * P * l;  // (behind the turned ones: rot + 2 P (l - rot / 2 P))
  const int at1 = !IL && turn0 ? a.rot / 2 + P * l : 2 * P * l + P;
  const bool has0 = at0 < a.D, has1 = at1 < a.D;
  const int t0 = blockIdx.x * tokens, n = min(tokens, a.n_tokens - t0);
  pdl_trigger();
  uint64_t turn = 0;
  int axis = 0;
  if (pair_of < a.rot / 2) {  // (set long before this launch)
    turn = a.table->turn[pair_of];
    axis = a.table->axis[pair_of];
  }
  pdl_wait();
  // this warp's share of the work: chunks of S U heads of q, k and v, token by token
  const int nq = (a.Hq + S * U - 1) / (S * U), nk = (a.Hkv + S * U - 1) / (S * U);
  int tok = 0, chunk = threadIdx.x >> 5;
  Piece16<P> x[U][2];
  int64_t slot = -1;
  int kind = 0, left = 0;  // q, k or v; heads from this lane's first one on
  auto load = [&] {
    while (chunk >= nq + 2 * nk) {
      chunk -= nq + 2 * nk;
      ++tok;
    }
    if (tok >= n) return;
    const int64_t t = t0 + tok;
    kind = chunk < nq ? 0 : chunk < nq + nk ? 1 : 2;
    const int h = (kind == 0 ? chunk : kind == 1 ? chunk - nq : chunk - nq - nk) * (S * U) + sub;
    left = (kind == 0 ? a.Hq : a.Hkv) - h;
    const int64_t head = kind == 0 ? a.q_head : kind == 1 ? a.k_head : a.v_head;
    const uint16_t *src = (kind == 0 ? a.q + t * a.q_token : kind == 1 ? a.k + t * a.k_token : a.v + t * a.v_token) + h * head;
    slot = a.slot[t];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      x[u][0] = x[u][1] = Piece16<P>{};
      if (u * S < left && has0) x[u][0] = load_piece<P>(src + at0);
      if (u * S < left && has1) x[u][1] = load_piece<P>(src + at1);
      src += S * head;
    }
  };
  load();
  if (pair_of < a.rot / 2)
    for (int k = threadIdx.x / kPairs; k < n; k += kRopeThreads / kPairs) {
      float s, c;
      sincos_turn((uint32_t)(turn * (uint64_t)(int64_t)a.pos[axis * a.pos_axis + t0 + k] >> 32), s, c);
      sin_of[k][pair_of] = s * a.scale;
      cos_of[k][pair_of] = c * a.scale;
    }
  __syncthreads();
  while (tok < n) {
    if (kind < 2) {
      // pairs of pairs: cosines, sines, and the gains of either piece
      uint64_t cs[Q], sn[Q], minus_sn[Q], g[2][Q];
      load_pairs<Q>(&cos_of[tok][P * l], turn0, cs);
      load_pairs<Q>(&sin_of[tok][P * l], turn0, sn);
#pragma unroll
      for (int i = 0; i < Q; ++i) minus_sn[i] = sn[i] ^ 0x8000000080000000ull;
      const bool norm = kind ? a.norm_k : a.norm_q;
      if (norm) {
        load_pairs<Q>(a.table->gain[kind] + at0, has0, g[0]);
        load_pairs<Q>(a.table->gain[kind] + at1, has1, g[1]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!__any_sync(0xffffffffu, u * S < left)) break;
        uint64_t y[2][Q];
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int i = 0; i < Q; ++i) {
            const float2 z = unpack2<BF>(x[u][s].w[i]);
            y[s][i] = pair(z.x, z.y);
          }
        if (norm) {
          uint64_t sq = 0;
#pragma unroll
          for (int i = 0; i < Q; ++i) sq = fma2(y[0][i], y[0][i], fma2(y[1][i], y[1][i], sq));
          float ss, s1;
          unpair(sq, ss, s1);
          ss += s1;
#pragma unroll
          for (int o = 1; o < GL; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float r = rsqrtf(fmaf(ss, a.inv_d, a.eps));
          const uint64_t rr = pair(r, r);
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < Q; ++i) y[s][i] = mul2(y[s][i], mul2(rr, g[s][i]));
        }
        if (IL) {
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < Q; ++i) {
              if (!(s ? turn1 : turn0)) continue;  // (0 times what is not turned may be NaN)
              const int j = s * Q + i;
              float p, q, c0, c1, s0, s1;
              unpair(y[s][i], p, q);
              unpair(cs[j / 2], c0, c1);
              unpair(sn[j / 2], s0, s1);
              const float c = j & 1 ? c1 : c0, z = j & 1 ? s1 : s0;
              y[s][i] = pair(fmaf(p, c, -q * z), fmaf(p, z, q * c));
            }
        } else if (turn0) {
#pragma unroll
          for (int i = 0; i < Q; ++i) {
            const uint64_t p = y[0][i], q = y[1][i];
            y[0][i] = fma2(p, cs[i], mul2(q, minus_sn[i]));
            y[1][i] = fma2(p, sn[i], mul2(q, cs[i]));
          }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int i = 0; i < Q; ++i) {
            float p, q;
            unpair(y[s][i], p, q);
            x[u][s].w[i] = pack_pair<BF>(p, q);
          }
      }
    }
    const int64_t t = t0 + tok, block = slot >> a.log_bt, head = kind == 0 ? a.qo_head : a.head_stride;
    const int h = (kind == 0 ? a.Hq : a.Hkv) - left;
    uint16_t *dst = (kind == 0 ? a.qo + t * a.qo_token
                               : (kind == 1 ? a.kc : a.vc) + block * a.block_stride + (slot & (a.bt - 1)) * a.token_stride) +
                    h * head;
    if (slot >= 0 && (kind == 0 || block < a.n_blocks)) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u * S < left && has0) store_piece<P>(dst + at0, x[u][0]);
        if (u * S < left && has1) store_piece<P>(dst + at1, x[u][1]);
        dst += S * head;
      }
    }
    chunk += kRopeThreads / 32;
    load();
  }
}

template <bool BF, int P, int GL, bool IL>
static int launch_one(const RopeArgs &a, cudaStream_t st) {
  // As few tokens to a CTA as keep the SMs in work, for the shortest way, and no more than make the tables worth their while.  Both
  // borders are measured: tokens and us with 1, 2 and 4 to a CTA on 152 SMs,
  //            1200             2432             4000             4864             8000
  //   32/8 x 128  9.1 8.2 12.1  14.9 14.3 13.8   21.3 20.2 23.0   25.0 24.7 24.5   38.2 36.7 36.5
  //   16/16 x 96  8.3 7.7 9.7   13.8 13.5 10.9   19.8 19.1 17.4   23.0 23.4 19.0   34.4 34.4 28.0
  //   8/1 x 128   4.5 4.0 5.4   9.2 7.9 6.4      14.0 11.9 10.8   16.3 14.5 11.5   24.8 21.3 16.7
  //   28/4 x 72   8.5 8.7 14.7  13.3 13.2 15.9   18.2 16.2 16.3   21.7 19.9 23.5   33.0 29.3 29.8
  // (600 tokens: 1 is the best of all four by a third; halves of a head)
  const int tokens = a.n_tokens >= a.sms * 8 * kRopeTokens ? kRopeTokens : a.n_tokens >= a.sms * 16 ? 2 : 1;
  return (int)launch_pdl(rope_kernel<BF, P, GL, IL>, dim3((a.n_tokens + tokens - 1) / tokens), dim3(kRopeThreads), 0, st, a,
                         tokens);
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
