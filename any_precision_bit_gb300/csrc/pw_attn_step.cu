// pw_attn_step.cu -- what an engine step needs around its attention: block tables and slot
// maps from the request lengths, the division of the attention work, and the cache write.
#include <cuda_runtime.h>
#include <limits.h>

#include "pw_attn.h"
#include "pw_device.cuh"

namespace pw {

constexpr int kStepThreads = 256;

// Exclusive prefix sum over the block of one value per thread; *total gets the sum.
template <int THREADS>
__device__ __forceinline__ long long block_scan(long long v, long long *total) {
  __shared__ long long ws[THREADS / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long inc = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += u;
  }
  __syncthreads();  // ws of an earlier call has been read
  if (lane == 31) ws[warp] = inc;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    const long long s = ws[w];
    if (w < warp) before += s;
    all += s;
  }
  *total = all;
  return before + inc - v;
}

// The largest i in [0, n) with cum[i] <= t (cum ascending, cum[0] <= t): with equal entries
// the last of them, so that empty segments are skipped.
__device__ __forceinline__ int seg_of(const int *cum, int n, int t) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cum[mid] <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ int sat(long long v) { return v > INT_MAX ? INT_MAX : (int)v; }

// Block tables and slot maps.  Two exclusive sums over the requests, of the new tokens
// (q_start) and of the blocks they open, locate everything else: a token's request and an
// opened block's request are binary searches in them.  Every CTA computes both sums for
// itself in shared memory (R <= 4096: 16 lengths a thread, which its neighbours have put
// into L2) and then does its share of the requests, opened blocks and tokens, so one launch
// without any hand-over between CTAs is enough; the sums cost a CTA less than a second
// launch would.
__global__ void __launch_bounds__(kStepThreads) kv_map_kernel(MapArgs a) {
  extern __shared__ int sh[];
  int *qs = sh, *bs = sh + a.R + 1;
  const int tid = threadIdx.x;
  pdl_trigger();
  pdl_wait();
  const int per = (a.R + kStepThreads - 1) / kStepThreads;
  const int r0 = min(a.R, tid * per), r1 = min(a.R, r0 + per);
  const long long cap = (long long)a.table_stride * a.bt;
  long long nt = 0, nb = 0;
  int bad = 0;
  for (int r = r0; r < r1; ++r) {
    const long long c = a.ctx_len[r], n = a.new_len[r];
    qs[r] = (int)nt;  // sums within the thread, at most INT_MAX; the threads before are added below
    bs[r] = sat(nb);
    // a request with a bad length brings nothing
    if (c < 0 || n < 0 || c + n > cap) {
      bad |= kAttnErrLen;
    } else {
      nt = min(nt + n, (long long)INT_MAX);
      nb += (c + n + a.bt - 1) / a.bt - (c + a.bt - 1) / a.bt;
    }
  }
  long long tot_t, tot_b;
  const long long t0 = block_scan<kStepThreads>(nt, &tot_t);
  const long long b0 = block_scan<kStepThreads>(nb, &tot_b);
  for (int r = r0; r < r1; ++r) {
    qs[r] = sat(qs[r] + t0);
    bs[r] = sat(bs[r] + b0);
  }
  if (tid == 0) {
    qs[a.R] = sat(tot_t);
    bs[a.R] = sat(tot_b);
  }
  __syncthreads();
  const int n_new = min(qs[a.R], a.n_tokens), n_open = bs[a.R];
  if (tot_t > a.n_tokens) bad |= kAttnErrTokens;
  if (n_open > a.n_ids) bad |= kAttnErrIds;
  const int gid = blockIdx.x * kStepThreads + tid, step = gridDim.x * kStepThreads;
  for (int r = gid; r <= a.R; r += step) {
    a.q_start[r] = min(qs[r], a.n_tokens);
    if (r < a.R) a.kv_len[r] = a.ctx_len[r] < 0 ? 0 : sat(min(cap, (long long)a.ctx_len[r] + (qs[r + 1] - qs[r])));
    const int row = r < a.R && a.rows ? a.rows[r] : 0;
    if (row < 0 || row >= a.table_rows) bad |= kAttnErrBlock;
  }
  for (long long j = gid; j < n_open; j += step) {  // (n_open may be anything below 2^31)
    const int i = (int)j, r = seg_of(bs, a.R, i);
    const int row = a.rows ? a.rows[r] : r;
    const int page = (a.ctx_len[r] + a.bt - 1) / a.bt + i - bs[r];
    int id = i < a.n_ids ? a.new_ids[i] : -1;
    if (id < 0 || id >= a.n_blocks) {
      if (i < a.n_ids) bad |= kAttnErrBlock;
      id = -1;
    }
    if (row >= 0 && row < a.table_rows) a.table[(size_t)row * a.table_stride + page] = id;
  }
  for (int t = gid; t < a.n_tokens; t += step) {
    long long slot = -1;
    int pos = -1;
    if (t < n_new) {
      const int r = seg_of(qs, a.R, t);
      const int row = a.rows ? a.rows[r] : r;
      const int c = a.ctx_len[r], held = (c + a.bt - 1) / a.bt;
      pos = c + t - qs[r];
      const int page = pos / a.bt;
      int id = -1;
      if (page < held) {  // a cached block's free end: an entry no thread writes
        if (row >= 0 && row < a.table_rows) id = a.table[(size_t)row * a.table_stride + page];
      } else {
        const int i = bs[r] + page - held;
        if (i < a.n_ids) id = a.new_ids[i];
      }
      if (id >= 0 && id < a.n_blocks)
        slot = (long long)id * a.bt + pos % a.bt;
      else if (page < held)
        bad |= kAttnErrBlock;
    }
    a.slot[t] = slot;
    a.pos[t] = pos;
  }
  if (bad) atomicOr(a.err, bad);
}

int launch_kv_map(const MapArgs &a, void *stream) {
  const int work = max(max(a.n_tokens, a.n_ids), a.R);
  const int grid = max(1, min(148, (work + 4 * kStepThreads - 1) / (4 * kStepThreads)));
  const size_t smem = 2 * sizeof(int) * (size_t)(a.R + 1);
  return (int)launch_pdl(kv_map_kernel, dim3(grid), dim3(kStepThreads), smem, reinterpret_cast<cudaStream_t>(stream), a);
}

// The keys that each row sees (the masks are intervals, so one pair per token).
__global__ void __launch_bounds__(kStepThreads) attn_bounds_kernel(PlanArgs a) {
  const long long cap = (long long)a.table_stride * a.bt;
  const int t = blockIdx.x * kStepThreads + threadIdx.x;
  pdl_trigger();
  pdl_wait();
  if (t >= a.n_tokens) return;
  RowBound b{0, 0, -1, 0};
  if (t < a.q_start[a.R]) {
    const int r = seg_of(a.q_start, a.R, t);
    const int kv = (int)min((long long)a.kv_len[r], cap);
    const int row = a.rows ? a.rows[r] : r;
    b.pos = a.ctx_len[r] + t - a.q_start[r];
    b.trow = row >= 0 && row < a.table_rows ? row : -1;
    b.hi = b.pos + 1;
    if (a.bidir_len) b.hi = max(b.hi, a.bidir_len[r]);
    b.hi = min(b.hi, kv);
    if (a.window > 0) b.lo = max(0, b.pos - a.window + 1);
    if (a.doc_start) b.lo = max(b.lo, a.doc_start[t]);
    b.lo = min(b.lo, b.hi);
    if (b.hi <= 0) b.lo = b.hi = 0;
  }
  a.bounds[t] = b;
}

int launch_attn_bounds(const PlanArgs &a, void *stream) {
  return (int)launch_pdl(attn_bounds_kernel, dim3((a.n_tokens + kStepThreads - 1) / kStepThreads), dim3(kStepThreads), 0,
                         reinterpret_cast<cudaStream_t>(stream), a);
}

// The same for a step with trees.  The first R blocks of threads take a request's tree each, a thread a node; the others take the
// rows that stand in no tree as attn_bounds_kernel does.  A node's way up is in descending order (a parent comes before its children), so
// that one word of its visible nodes after the other is finished; the parents lie in shared memory.
__device__ __forceinline__ int tree_of(const TreeArgs &a, int r, int kv) {
  const int tl = a.tree_len[r];
  return tl > 0 && tl <= PW_TREE_NODES && tl <= a.parent_stride && tl <= kv ? tl : 0;
}
// One of them (`block`), in two phases with a meeting of the CTA between them: parents to shared memory, and the rows.
__device__ __forceinline__ void tree_parents(const TreeArgs &x, int block, int tid, int *parent) {
  const PlanArgs &a = x.plan;
  if (block >= a.R) return;
  const int kv = (int)min((long long)a.kv_len[block], (long long)a.table_stride * a.bt), tl = tree_of(x, block, kv);
  if (tl != x.tree_len[block] && tid == 0) atomicOr(x.err, kAttnErrTree);
  if (tid >= tl) return;
  int p = x.parent[(size_t)block * x.parent_stride + tid];
  if (p < -1 || p >= tid) {
    atomicOr(x.err, kAttnErrTree);
    p = -1;
  }
  parent[tid] = p;
}
__device__ __forceinline__ void tree_rows(const TreeArgs &x, int block, int tid, const int *parent) {
  const PlanArgs &a = x.plan;
  const long long cap = (long long)a.table_stride * a.bt;
  if (block < a.R) {
    const int r = block, kv = (int)min((long long)a.kv_len[r], cap), tl = tree_of(x, r, kv);
    const int start = kv - tl, q0 = max(a.q_start[r], 0), q1 = min(a.q_start[r + 1], a.n_tokens);
    const int t = q0 + (start + tid - a.ctx_len[r]);
    if (tid >= tl || t < q0 || t >= q1) return;
    uint32_t word[kTreeWords];
    int node = tid, depth = 0;  // nodes passed so far
#pragma unroll
    for (int w = kTreeWords - 1; w >= 0; --w) {
      uint32_t bits = 0;
      while (node >= 32 * w) {  // (a root's parent is below every word)
        if (a.window <= 0 || depth < a.window) bits |= 1u << (node & 31);
        ++depth;
        node = parent[node];
      }
      word[w] = bits;
    }
    uint4 *seen = reinterpret_cast<uint4 *>(x.seen + (size_t)t * kTreeWords);
    seen[0] = make_uint4(word[0], word[1], word[2], word[3]);
    seen[1] = make_uint4(word[4], word[5], word[6], word[7]);
    RowBound b;
    b.pos = start + depth - 1;
    b.hi = start + tid + 1;
    // (an ancestor within the window has no lower place than its position, which is not below this)
    b.lo = a.window > 0 ? max(0, b.pos - a.window + 1) : 0;
    b.trow = start;
    a.bounds[t] = b;
    if (x.pos) x.pos[t] = b.pos;
    return;
  }
  const int t = (block - a.R) * kTreeRows + tid;
  if (t >= a.n_tokens) return;
  RowBound b{0, 0, INT_MAX, -1};
  if (t < a.q_start[a.R]) {
    const int r = seg_of(a.q_start, a.R, t);
    const int kv = (int)min((long long)a.kv_len[r], cap), tl = tree_of(x, r, kv);
    b.pos = a.ctx_len[r] + t - a.q_start[r];
    if (tl && b.pos >= kv - tl && b.pos < kv) return;  // a node's row
    b.hi = min(b.pos + 1, kv);
    if (a.window > 0) b.lo = max(0, b.pos - a.window + 1);
    b.lo = min(b.lo, b.hi);
    if (b.hi <= 0) b.lo = b.hi = 0;
  }
  a.bounds[t] = b;
  if (x.pos) x.pos[t] = b.pos;
}
__global__ void __launch_bounds__(kTreeRows) tree_bounds_kernel(TreeArgs x) {
  static_assert(kTreeRows == PW_TREE_NODES && kTreeWords == 8, "a thread a node, two 16-byte stores");
  __shared__ int parent[PW_TREE_NODES];
  pdl_trigger();
  pdl_wait();
  tree_parents(x, blockIdx.x, threadIdx.x, parent);
  __syncthreads();
  tree_rows(x, blockIdx.x, threadIdx.x, parent);
}

int launch_tree_bounds(const TreeArgs &a, void *stream) {
  return (int)launch_pdl(tree_bounds_kernel, dim3(tree_blocks(a)), dim3(kTreeRows), 0, reinterpret_cast<cudaStream_t>(stream), a);
}

// Segments of a list: requests (and, behind them, the rows that are padding), or groups.
struct Segment {
  int tok0, tok1, trow, klo, khi, merge;
};

__device__ __forceinline__ Segment segment_of(const PlanArgs &a, int i) {
  Segment g{0, 0, -1, 0, 0, 0};
  const int n = min(max(a.q_start[a.R], 0), a.n_tokens);
  const int cap = (int)min((long long)a.table_stride * a.bt, (long long)INT_MAX);
  int r = i;
  if (a.of_groups) {
    r = min(max(a.group_start[i], 0), a.R);
    const int e = min(max(a.group_start[i + 1], r), a.R);
    g.tok0 = min(max(a.q_start[r], 0), n);
    g.tok1 = min(max(a.q_start[e], g.tok0), n);
    g.khi = min(max(a.shared_len[i], 0), cap);
    if (r == a.R) return g;
  } else if (i == a.R) {  // padding rows: no keys
    g.tok0 = n;
    g.tok1 = a.n_tokens;
    return g;
  } else {
    g.tok0 = min(max(a.q_start[r], 0), n);
    g.tok1 = min(max(a.q_start[r + 1], g.tok0), n);
    g.khi = min(max(a.kv_len[r], 0), cap);
    if (a.n_groups) {
      g.klo = min(max(a.shared_len[seg_of(a.group_start, a.n_groups, r)], 0), g.khi);
      g.merge = 1;
    }
  }
  const int row = a.rows ? a.rows[r] : r;
  g.trow = row >= 0 && row < a.table_rows ? row : -1;
  return g;
}

// One list of work, by one CTA: tiles per segment and their sum; per tile (one warp each) the key
// tiles that some row of it sees; their sum; and where each of the forward's CTAs begins.
constexpr int kListThreads = 1024;
constexpr int kListTiles = 1024;  // with at most so many tiles their sums are searched in shared memory
__device__ __forceinline__ void lay_out_list(const PlanArgs &a, int *cum_tiles) {
  __shared__ int near_cum[kListTiles + 1];
  const int tid = threadIdx.x;
  const int n_seg = a.of_groups ? a.n_groups : a.R + 1;
  const int tt = a.list.tpt * a.list.streams;
  auto units_of = [&](const AttnTile &t) { return t.ntok > a.list.tpt ? a.list.two : a.list.one; };  // of a key tile
  long long before = 0;
  for (int s0 = 0; s0 < n_seg; s0 += kListThreads) {
    const int s = s0 + tid;
    int n = 0;
    if (s < n_seg) {
      const Segment g = segment_of(a, s);
      n = (g.tok1 - g.tok0 + tt - 1) / tt;
    }
    long long total;
    const long long at = block_scan<kListThreads>(n, &total);
    if (s < n_seg) cum_tiles[s] = (int)(before + at);
    before += total;
  }
  const int n_tiles = (int)min(before, (long long)a.list.max_tiles);
  __syncthreads();
  // lanes that look through a tile's tokens: one where they are few (a decode step's), else as many as leave one round of
  // tiles, or four, with eight loads a lane under way (32 lanes each and one load at a time: 96 tiles of 64 tokens 13.7 us for
  // the whole plan instead of 11.2, a prompt of 8192 13 instead of 10.2)
  int wide = tt > 4 ? 32 : 1;
  while (wide > 4 && n_tiles * wide > kListThreads) wide >>= 1;
  for (int i0 = 0; i0 < n_tiles; i0 += kListThreads / wide) {
    const int i = i0 + tid / wide;
    const bool some = i < n_tiles;
    const int s = some ? seg_of(cum_tiles, n_seg, i) : 0;
    const Segment g = segment_of(a, s);
    AttnTile t;
    t.tok0 = g.tok0 + (i - cum_tiles[s]) * tt;
    t.ntok = some ? min(tt, g.tok1 - t.tok0) : 0;
    t.trow = g.trow;
    t.klo = g.klo;
    t.khi = g.khi;
    t.merge = g.merge;
    int lo = INT_MAX, hi = 0;
    constexpr int kAhead = 8;  // rows whose bounds are under way at once
    for (int j0 = tid & (wide - 1); j0 < t.ntok; j0 += kAhead * wide) {
      int2 b[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int j = j0 + k * wide;
        b[k] = j < t.ntok ? *reinterpret_cast<const int2 *>(a.bounds + t.tok0 + j) : make_int2(0, 0);  // lo and hi
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int l = max(b[k].x, g.klo), h = min(b[k].y, g.khi);
        if (l < h) {
          lo = min(lo, l);
          hi = max(hi, h);
        }
      }
    }
    for (int o = wide >> 1; o > 0; o >>= 1) {
      lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    t.kv0 = hi > 0 ? lo / kAttnKeys : g.klo / kAttnKeys;
    t.kv1 = hi > 0 ? (hi - 1) / kAttnKeys + 1 : t.kv0 + 1;
    if (some && (tid & (wide - 1)) == 0) {
      a.list.tiles[i] = t;
      a.list.cum[i + 1] = (t.kv1 - t.kv0) * units_of(t) + a.list.piece_cost;
    }
  }
  __syncthreads();
  before = 0;
  for (int i0 = 0; i0 < n_tiles; i0 += kListThreads) {
    const int i = i0 + tid;
    const int n = i < n_tiles ? a.list.cum[i + 1] : 0;
    long long total;
    const long long at = block_scan<kListThreads>(n, &total);
    if (i < n_tiles) {
      a.list.cum[i + 1] = sat(before + at + n);
      if (n_tiles <= kListTiles) near_cum[i + 1] = sat(before + at + n);
    }
    before += total;
  }
  const int *cum = n_tiles <= kListTiles ? near_cum : a.list.cum;
  if (tid == 0) {
    near_cum[0] = 0;
    a.list.cum[0] = 0;
    a.list.meta[0] = n_tiles;
    a.list.meta[1] = sat(before);
  }
  __syncthreads();
  const long long W = before * a.n_kv_heads;  // (0 for groups without new tokens)
  // (a share is a key tile's units at least, so that every CTA between a (tile, head)'s first and last has a piece of it)
  const long long P = max(1LL, min((long long)a.ctas, W / a.list.two));
  // CTAs of the first and the last key tile of a (tile, head) whose units begin at ub
  auto ctas_of = [&](long long ub, int cost, int units) {
    return make_int2((int)(((ub + a.list.piece_cost + 1) * P - 1) / W), (int)(((ub + cost - units + 1) * P - 1) / W));
  };
  __shared__ int n_splits;
  if (tid == 0) n_splits = 0;
  __syncthreads();
  for (int c = tid; c < a.ctas; c += kListThreads) {
    const long long u0 = min(c * W / P, W), u1 = min((c + 1) * W / P, W);
    AttnStart st{0, 0, 0, (int)(u1 - u0), {}, {0, 0}, {0, 0}};
    // the (tile, head) of a unit, and the CTAs of its first and last key tiles
    auto find = [&](long long u, int &tile, int &head, int &off) {
      int lo = 0, hi = n_tiles - 1;  // the last tile whose units begin at or before u
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((long long)cum[mid] * a.n_kv_heads <= u)
          lo = mid;
        else
          hi = mid - 1;
      }
      const int cost = cum[lo + 1] - cum[lo];
      const long long rem = u - (long long)cum[lo] * a.n_kv_heads;
      tile = lo;
      head = (int)(rem / cost);
      off = (int)(rem - (long long)head * cost);
      return ctas_of(u - off, cost, a.list.two > 1 ? units_of(a.list.tiles[lo]) : 1);
    };
    if (u1 > u0) {
      st.first = find(u0, st.tile, st.head, st.off);
      int tile, head, off;
      st.last = find(u1 - 1, tile, head, off);
      st.t = a.list.tiles[st.tile];
      if (st.last.x == c && st.last.y > c)  // split, from here on (their order does not matter)
        a.list.splits[atomicAdd(&n_splits, 1)] = AttnSplit{a.list.tiles[tile], head, c, st.last.y, 0};
    }
    a.list.start[c] = st;
  }
  __syncthreads();
  if (tid == 0) {
    a.list.meta[2] = n_splits;
    if (!a.of_groups) *a.shape_out = a.shape;
  }
}
__global__ void __launch_bounds__(kListThreads) attn_list_kernel(PlanArgs a) {
  extern __shared__ int cum_tiles[];
  pdl_trigger();
  pdl_wait();
  lay_out_list(a, cum_tiles);
}
// Bounds and list of a small step with trees.
__global__ void __launch_bounds__(kListThreads) tree_list_kernel(TreeArgs x) {
  extern __shared__ int cum_tiles[];
  constexpr int kBlocks = kListThreads / kTreeRows;
  __shared__ int parent[kBlocks][PW_TREE_NODES];
  const int blocks = x.plan.R + (x.plan.n_tokens + kTreeRows - 1) / kTreeRows, part = threadIdx.x / kTreeRows;
  pdl_trigger();
  pdl_wait();
  for (int b0 = 0; b0 < blocks; b0 += kBlocks) {
    const int block = b0 + part;
    if (block < blocks) tree_parents(x, block, threadIdx.x % kTreeRows, parent[part]);
    __syncthreads();
    if (block < blocks) tree_rows(x, block, threadIdx.x % kTreeRows, parent[part]);
    __syncthreads();
  }
  lay_out_list(x.plan, cum_tiles);
}

int launch_attn_list(const PlanArgs &a, void *stream) {
  const int n_seg = a.of_groups ? a.n_groups : a.R + 1;
  return (int)launch_pdl(attn_list_kernel, dim3(1), dim3(kListThreads), sizeof(int) * (size_t)n_seg,
                         reinterpret_cast<cudaStream_t>(stream), a);
}

int launch_tree_list(const TreeArgs &a, void *stream) {
  return (int)launch_pdl(tree_list_kernel, dim3(1), dim3(kListThreads), sizeof(int) * (size_t)(a.plan.R + 1),
                         reinterpret_cast<cudaStream_t>(stream), a);
}

// The cache write.  A token is 2 n_heads head_dim elements, of k and then of v, in pieces of 16 bytes; a
// thread keeps its piece and goes through the tokens four at a time, so that the divisions that find the
// piece are done once and four loads are under way together.  Consecutive threads take consecutive pieces:
// reads and writes are whole runs of a head, or of all heads where the cache keeps them side by side.
constexpr int kAppendTokens = 4;
__global__ void __launch_bounds__(kStepThreads) attn_append_kernel(AppendArgs a, int lanes) {
  const int vec = a.head_dim / 8, row = a.n_heads * vec;
  const int sub = threadIdx.x / lanes, per = kStepThreads / lanes;  // token within the block's `per` tokens
  pdl_trigger();
  pdl_wait();
  if (sub >= per) return;
  const int stride = gridDim.x * per;
  for (int w = threadIdx.x - sub * lanes; w < 2 * row; w += lanes) {
    const bool val = w >= row;
    const int x = val ? w - row : w, h = x / vec, c = 8 * (x - h * vec);
    const uint16_t *src = val ? a.v + h * a.v_head + c : a.k + h * a.k_head + c;
    uint16_t *dst = (val ? a.vc : a.kc) + h * a.head_stride + c;
    const int64_t step = val ? a.v_token : a.k_token;
    for (int t0 = blockIdx.x * per + sub; t0 < a.n_tokens; t0 += kAppendTokens * stride) {
      int64_t slot[kAppendTokens];
      uint4 data[kAppendTokens];
#pragma unroll
      for (int i = 0; i < kAppendTokens; ++i) {
        const int64_t t = t0 + (int64_t)i * stride;
        slot[i] = t < a.n_tokens ? a.slot[t] : -1;
        if (slot[i] >> a.log_bt >= a.n_blocks) slot[i] = -1;
        if (slot[i] >= 0) data[i] = *reinterpret_cast<const uint4 *>(src + t * step);
      }
#pragma unroll
      for (int i = 0; i < kAppendTokens; ++i)
        if (slot[i] >= 0)
          *reinterpret_cast<uint4 *>(dst + (slot[i] >> a.log_bt) * a.block_stride + (slot[i] & (a.bt - 1)) * a.token_stride) =
              data[i];
    }
  }
}

int launch_attn_append(const AppendArgs &a, void *stream) {
  const int pieces = 2 * a.n_heads * (a.head_dim / 8);
  const int lanes = pieces < kStepThreads ? pieces : kStepThreads, per = kStepThreads / lanes;
  // enough blocks to fill the SMs; a step of few tokens gets one token (of each `per`) a block
  const int want = (a.n_tokens + per - 1) / per, most = 152 * 8;
  return (int)launch_pdl(attn_append_kernel, dim3(want < most ? want : most), dim3(kStepThreads), 0,
                         reinterpret_cast<cudaStream_t>(stream), a, lanes);
}

}  // namespace pw
