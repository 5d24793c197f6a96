// pw_attn.h -- structures of the paged-attention kernels and their launchers.
#pragma once
#include <stdint.h>

#include "../../include/pw.h"
#include <cuda_runtime.h>

#include "pw_internal.h"

namespace pw {

constexpr int kAttnKeys = 128;         // keys of one key/value tile, the unit of work
constexpr int kAttnRows = 128;         // query rows of one tile (tensor-memory lanes of an MMA)
constexpr int kAttnMaxRequests = 4096;
// Two forms of the kernel:
//   kTwo     two 128-row tiles share each key tile: while one tile's scores are in the softmax the
//            tensor cores work on the other's;
//   kSpread  one tile of at most 16 rows, which is held four times, once in each lane quarter of tensor
//            memory: quarter w keeps a softmax over keys 32 w .. 32 w + 31 of every key tile (its
//            probabilities of the other keys are zeros), and the four results are added at the end.  Four
//            warps then share the few rows (eight or sixteen scores a thread), the scores of the next key
//            tile are computed during a softmax, and four more warps finish a piece during the next.
// Measured with one form and the other, 64 requests (us, launch included): 4 rows behind 256 .. 8192 keys 189 in
// kSpread and 201 in kTwo, behind 16 .. 700 keys 36 and 46; 4 rows of 64 with capped scores behind up to 4096
// keys 126 and 249; 16 rows behind as many 111 and 120; 32 rows, where kSpread has no second query buffer, 65 and 64.
enum { kTwo = 2, kSpread = 4 };
constexpr int kSpreadRows = 16;

// tanh(y) = y P(y^2) with P of degree 4, fitted at Chebyshev nodes on |y| <= 1/2; largest error 3.8e-8.
constexpr double kTanhPoly[5] = {1.0, -0.3333307206630707, 0.13324828445911407, -0.05298924073576927, 0.017141319811344147};

// Findings of the device side, reported by pw_attn_check.
enum {
  kAttnErrWait = 1,    // a bounded wait expired
  kAttnErrLen = 2,     // a negative length, or more tokens than a table row can hold
  kAttnErrTokens = 4,  // new tokens beyond n_tokens
  kAttnErrIds = 8,     // fewer new ids than opened blocks
  kAttnErrBlock = 16,  // a block id or a table row out of range
  kAttnErrPlan = 32,   // a forward met a plan of another shape than it was launched for
};

// What a forward's launch takes from the plan by value, beside the lists that lie on the device.  The plan's
// kernels leave it beside the lists; a launch that finds another one there (a captured forward replayed after the
// plan was laid out again, or a captured plan that has not been replayed) would read past its tiles, the rows of
// q and o or the table, so it writes nothing and reports kAttnErrPlan.
struct alignas(16) AttnShape {
  int tpt, streams;              // of the requests' list (streams 0: never laid out)
  int group_tpt, group_streams;  // of the groups' (0: no groups)
  int n_tokens, table_stride;
  const int *table;
};
static_assert(sizeof(AttnShape) == 32, "two 16-byte loads");

// Keys a row may see, and where: [lo, hi) of table row trow (-1: none), at position pos.
struct RowBound {
  int lo, hi, trow, pos;
};

// A tile of query rows of one segment (a request's keys, or a group's shared prefix): tokens
// tok0 .. tok0 + ntok - 1, each with its G = n_heads / n_kv_heads heads, against the keys
// [klo, khi) of table row trow, of which the tiles kv0 .. kv1 - 1 (128 keys each) hold some
// that a row of the tile sees; kv1 > kv0 always (a tile without visible keys runs one tile of
// masked keys, and so gets its zeros).
struct AttnTile {
  int tok0, ntok, trow, klo, khi, kv0, kv1;
  int merge;  // the rows also have a result over their group's shared prefix
};

// Where a CTA's share of the work begins.
struct AttnStart {
  int tile, head, off, n;  // unit `off` of (tile, head); n units in all
  AttnTile t;              // the tile
  // CTAs of the first and the last key tile of the (tile, head) that the CTA begins in, and of the one that it
  // ends in
  int2 first, last;
};

// A (tile, head) that is split among the CTAs c0 .. c1, c1 > c0.
struct AttnSplit {
  AttnTile t;
  int head, c0, c1, pad;
};

// One list of work.  In the order (tile, head), each has piece_cost units without keys and then one for
// each of its key tiles; of the W units CTA c takes [c W / P, (c + 1) W / P), P the number of CTAs or W if that is less (the rest idle).
struct AttnList {
  AttnTile *tiles;
  int *cum;          // [tiles + 1] units of one head before each tile
  AttnStart *start;  // [P]
  AttnSplit *splits; // [P], of which meta[2] are set
  int *meta;         // [0] tiles, [1] units of one head, [2] splits
  int tpt;           // tokens of one 128-row tile
  int streams;       // 128-row tiles of one AttnTile (1 or 2)
  int piece_cost;    // units that a (tile, head) counts for beside its key tiles when the work is divided: the
                     // queries' way in, the pipeline's filling and draining, the result's way out
  int max_tiles;
};

struct PlanArgs {
  int R, n_tokens, table_rows, table_stride, bt;
  const int *ctx_len, *rows, *q_start, *kv_len;
  const int *doc_start, *bidir_len;
  int window;
  int n_groups;
  const int *group_start, *shared_len;
  RowBound *bounds;
  AttnList list;
  int of_groups;  // the list of the groups' shared prefixes, not of the requests
  AttnShape shape, *shape_out;  // left by the kernel that lays out the requests' list, the plan's last
  int ctas, n_kv_heads;
};

struct MapArgs {
  int R, n_tokens, table_rows, table_stride, bt, n_blocks, n_ids;
  const int *ctx_len, *new_len, *rows, *new_ids;
  int *table, *q_start, *kv_len, *pos;
  int64_t *slot;
  int *err;
};

struct AppendArgs {
  const uint16_t *k, *v;
  int64_t k_token, k_head, v_token, v_head;
  uint16_t *kc, *vc;
  int64_t block_stride, token_stride, head_stride;
  const int64_t *slot;
  int n_tokens, n_heads, head_dim, bt, log_bt, n_blocks;
};

// Tensor maps of one forward launch: boxes of 64 elements of a head by (Q) the G heads of a
// key/value head by a tile's tokens, or (K, V) the tokens of a block; 128-byte swizzle, the K-major
// operand layout of the MMAs.  Elements past head_dim, tokens past n_tokens and blocks past n_blocks
// read as zeros.
struct AttnMaps {
  TmaDesc q, k, v;
};

struct AttnArgs {
  const RowBound *bounds;
  AttnList list;
  AttnShape shape;           // as launched
  const AttnShape *planned;  // as laid out
  int ctas, device;
  const int *table;
  int table_stride, n_tokens, n_blocks, log_bt;
  int Hq, Hkv, G, D;
  unsigned g_magic;  // ceil(65536 / G)
  int box_tokens;  // tokens of one Q box
  const uint16_t *q;
  int64_t q_token, q_head;
  uint16_t *o;
  int64_t o_token, o_head;
  const uint16_t *kc, *vc;
  int64_t block_stride, token_stride, head_stride;
  float *lse;
  float scale, softcap;
  float scale2, inv_cap, cap2;  // scale log2 e, scale / softcap, softcap log2 e
  float cap_poly[5];            // cap2 tanh(inv_cap x) as x times a polynomial of x^2
  const float *slopes;
  // Results over a shared prefix, normalised, and their log2-sum-exp2: written (to_prefix) or merged
  // into the rows of tiles with `merge`.
  float *prefix_o, *prefix_lse;  // [n_tokens][Hq][D], [n_tokens][Hq]
  int to_prefix, after_prefix;
  int join;  // pieces of split tiles are added up by attn_join_kernel, not by the last of their CTAs
  // Partial results of split tiles: two slots a CTA (its last piece and its first) and stream.
  float *part_o;    // [ctas][2][streams][head_dim padded / 4][128][4]
  float2 *part_ml;  // [ctas][2][streams][128] running maximum and sum
  uint32_t *part_odd;  // [ctas][2][streams][128] bit g: columns 4 g .. 4 g + 3 of a row's piece are not finite (with `join`)
  int *counters;    // [ctas][2] arrived pieces of the split tile whose first piece is the CTA's last,
                    // per stream; zero between launches
  uint32_t *marks;  // a bit for each row [n_tokens][Hq]: to be computed again by attn_kernel; zero between launches
  int *err;
  long long wait_cycles;  // bounded device waits give up after this many SM cycles
  int withhold;           // testing: see produce()
};

int launch_kv_map(const MapArgs &a, void *stream);
int launch_attn_bounds(const PlanArgs &a, void *stream);
int launch_attn_list(const PlanArgs &a, void *stream);
int launch_attn_append(const AppendArgs &a, void *stream);
int launch_attn(const AttnArgs &a, const AttnMaps &maps, int bf16, void *stream);

}  // namespace pw
