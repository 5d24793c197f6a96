// pw_kv_pages.cu -- keys and values that change their place: an accepted path of drafted tokens moves to the front of its
// tree, and blocks are copied and renamed.  All layers' caches in one launch (of at most kMoveCaches).
#include <cuda_runtime.h>
#include <limits.h>

#include "pw_attn.h"
#include "pw_device.cuh"

namespace pw {

constexpr int kKeepThreads = 128;

// A CTA moves one request's tokens in one cache, a layer's keys or values.  Ids and addresses come once for the CTA; a thread then
// has 16 bytes of a token and goes through the moves in ascending order, four loads ahead of their stores: a place lies
// at or before where its token comes from, and so before everything that is loaded later.  96 requests' paths of up to 6
// tokens in 32 caches, 23.5 MB moved, take 5.5 to 5.9 us: latency (ids, addresses, and two rounds of loads in turn).
__global__ void __launch_bounds__(kKeepThreads) kv_keep_kernel(const __grid_constant__ KeepArgs a,
                                                               const __grid_constant__ MoveCaches m) {
  __shared__ int from[PW_TREE_NODES], end;
  __shared__ int64_t src[PW_TREE_NODES], dst[PW_TREE_NODES];
  __shared__ int n_moves, warp_moves[kKeepThreads / 32];
  const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint16_t *base = m.base[blockIdx.y];
  pdl_trigger();
  pdl_wait();
  const long long cap = (long long)a.table_stride * a.bt;
  const int kv = (int)min((long long)max(a.kv_len[r], 0), min(cap, (long long)INT_MAX));
  const int tl = a.tree_len[r], row = a.rows ? a.rows[r] : r;
  int n = a.n_keep[r], bad = 0;
  const bool tree = tl >= 0 && tl <= PW_TREE_NODES && tl <= kv, there = row >= 0 && row < a.table_rows;
  if (!tree || n < 0 || n > tl || n > a.keep_stride) {
    bad = kAttnErrTree;
    n = 0;
  }
  if (!there) {
    bad |= kAttnErrBlock;
    n = 0;
  }
  const int start = tree ? kv - tl : kv;
  if (tid == 0) {
    end = n;
    n_moves = 0;
  }
  for (int i = tid; i < n; i += kKeepThreads) from[i] = a.keep[(size_t)r * a.keep_stride + i];
  __syncthreads();
  for (int i = tid; i < n; i += kKeepThreads)
    if (from[i] <= (i ? from[i - 1] : -1) || from[i] >= tl) atomicMin(&end, i);
  __syncthreads();
  if (end < n) bad |= kAttnErrTree;
  n = end;
  if (a.ctx_out && blockIdx.y == 0 && tid == 0) a.ctx_out[r] = start + n;
  // the moves of tokens that are not in their place, in order
  auto address = [&](int p) {
    const int id = a.table[(size_t)row * a.table_stride + (p >> a.log_bt)];
    return id >= 0 && id < a.n_blocks ? id * m.block_stride + (p & (a.bt - 1)) * m.token_stride : (int64_t)-1;
  };
  for (int i0 = 0; i0 < n; i0 += kKeepThreads) {
    const int i = i0 + tid;
    int64_t s = -1, d = -1;
    if (i < n && from[i] != i) {
      s = address(start + from[i]);
      d = address(start + i);
      if (s < 0 || d < 0) bad |= kAttnErrBlock;
    }
    const bool move = s >= 0 && d >= 0;
    const unsigned who = __ballot_sync(0xffffffffu, move);
    if (lane == 0) warp_moves[warp] = __popc(who);
    __syncthreads();
    int at = n_moves + __popc(who & ((1u << lane) - 1u));
    for (int w = 0; w < warp; ++w) at += warp_moves[w];
    if (move) {
      src[at] = s;
      dst[at] = d;
    }
    __syncthreads();
    if (tid == 0)
      for (int w = 0; w < kKeepThreads / 32; ++w) n_moves += warp_moves[w];
    __syncthreads();
  }
  if (bad) atomicOr(a.err, bad);
  const int moves = n_moves, vec = a.head_dim / 8;
  for (int p = tid; p < a.n_heads * vec; p += kKeepThreads) {
    const int h = p / vec;
    uint16_t *col = base + h * m.head_stride + 8 * (p - h * vec);
    for (int i = 0; i < moves; i += 4) {
      uint4 x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i + k < moves) x[k] = *reinterpret_cast<const uint4 *>(col + src[i + k]);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i + k < moves) *reinterpret_cast<uint4 *>(col + dst[i + k]) = x[k];
    }
  }
}

int launch_keep(const KeepArgs &a, const MoveCaches &m, int n_caches, void *stream) {
  return (int)launch_pdl(kv_keep_kernel, dim3(a.R, n_caches), dim3(kKeepThreads), 0, reinterpret_cast<cudaStream_t>(stream), a, m);
}

// A CTA copies a part of one block of one cache, kCopyPieces pieces of 16 bytes a thread.  The pieces are
// numbered in the order in which they lie in memory where the block is one run of it (`whole`), else token by token.  700
// blocks of 32 KB in 24 caches, 1.1 GB moved, take 163 us, a copy's rate.  CTAs behind the copies' rename the table's entries
// where pairs are few (3 pairs with a launch of its own for that: 1.5 us later).
constexpr int kCopyThreads = 256, kCopyPieces = 8, kRenameEntries = 16;  // entries of a thread
__device__ void rename_few(const CopyArgs &a, int64_t e0) {
  __shared__ int src[kRenamePairs], dst[kRenamePairs];
  if ((int)threadIdx.x < a.n) {
    const int s = a.src[threadIdx.x], d = a.dst[threadIdx.x];
    const bool good = s >= 0 && s < a.n_blocks && d >= 0 && d < a.n_blocks;
    src[threadIdx.x] = good ? s : -1;
    dst[threadIdx.x] = d;
  }
  __syncthreads();
  for (int k = 0; k < kRenameEntries; ++k) {
    const int64_t e = e0 + k * kCopyThreads + threadIdx.x;
    const int id = e < a.entries ? a.table[e] : -1;
    if (id < 0) continue;
    for (int i = 0; i < a.n; ++i)
      if (src[i] == id) {
        a.table[e] = dst[i];
        break;
      }
  }
}
__global__ void __launch_bounds__(kCopyThreads) kv_copy_kernel(const __grid_constant__ CopyArgs a,
                                                               const __grid_constant__ MoveCaches m, int splits) {
  uint16_t *base = m.base[blockIdx.y];
  const int pair = blockIdx.x / splits, split = blockIdx.x - pair * splits;
  const int vec = a.head_dim / 8, row = a.n_heads * vec, total = a.bt * row;
  const bool whole = (m.head_stride == a.head_dim && m.token_stride == (int64_t)a.n_heads * a.head_dim) ||
                     (m.token_stride == a.head_dim && m.head_stride == (int64_t)a.bt * a.head_dim);
  pdl_trigger();
  pdl_wait();
  if (pair >= a.n) {
    if (blockIdx.y == 0) rename_few(a, (int64_t)(blockIdx.x - a.n * splits) * (kCopyThreads * kRenameEntries));
    return;
  }
  const int s = a.src[pair], d = a.dst[pair];
  const bool good = s >= 0 && s < a.n_blocks && d >= 0 && d < a.n_blocks;
  if (blockIdx.y == 0 && split == 0 && threadIdx.x == 0) {
    if (!good) atomicOr(a.err, kAttnErrCopy);
    if (a.where && good) a.where[s] = pair;
  }
  if (!good) return;
  const uint16_t *from = base + s * m.block_stride;
  uint16_t *to = base + d * m.block_stride;
  const int p0 = split * (kCopyThreads * kCopyPieces) + threadIdx.x;
  int64_t at[kCopyPieces];
  uint4 x[kCopyPieces];
#pragma unroll
  for (int k = 0; k < kCopyPieces; ++k) {
    const int p = p0 + k * kCopyThreads;
    at[k] = 8 * (int64_t)p;
    if (!whole) {
      const int t = p / row, q = p - t * row, h = q / vec;
      at[k] = t * m.token_stride + h * m.head_stride + 8 * (q - h * vec);
    }
    if (p < total) x[k] = *reinterpret_cast<const uint4 *>(from + at[k]);
  }
#pragma unroll
  for (int k = 0; k < kCopyPieces; ++k)
    if (p0 + k * kCopyThreads < total) *reinterpret_cast<uint4 *>(to + at[k]) = x[k];
}

int launch_copy(const CopyArgs &a, const MoveCaches &m, int n_caches, void *stream) {
  const int per = kCopyThreads * kCopyPieces;
  const int splits = (a.bt * a.n_heads * (a.head_dim / 8) + per - 1) / per;
  const int64_t each = kCopyThreads * kRenameEntries, rename = a.table ? (a.entries + each - 1) / each : 0;
  return (int)launch_pdl(kv_copy_kernel, dim3((unsigned)(a.n * splits + rename), n_caches), dim3(kCopyThreads), 0,
                         reinterpret_cast<cudaStream_t>(stream), a, m, splits);
}

// Table entries that name a source name its copy from now on.  where[id] is the number of a pair with this source, or
// anything (left by an earlier call): the pair itself says which.
__global__ void __launch_bounds__(256) kv_rename_kernel(CopyArgs a) {
  pdl_trigger();
  pdl_wait();
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < a.entries; e += (int64_t)gridDim.x * 256) {
    const int id = a.table[e];
    if (id < 0 || id >= a.n_blocks) continue;
    const int pair = a.where[id];
    if (pair < 0 || pair >= a.n || a.src[pair] != id) continue;
    const int d = a.dst[pair];
    if (d >= 0 && d < a.n_blocks) a.table[e] = d;
  }
}

int launch_rename(const CopyArgs &a, void *stream) {
  const int64_t ctas = (a.entries + 255) / 256;
  return (int)launch_pdl(kv_rename_kernel, dim3((unsigned)(ctas < 1216 ? ctas : 1216)), dim3(256), 0,
                         reinterpret_cast<cudaStream_t>(stream), a);
}

}  // namespace pw
