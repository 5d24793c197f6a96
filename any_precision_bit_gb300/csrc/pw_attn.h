// pw_attn.h -- structures of the paged-attention kernels and their launchers.
#pragma once
#include <stdint.h>

#include "../../include/pw.h"
#include "pw_internal.h"

namespace pw {

constexpr int kAttnKeys = 128;         // keys of one key/value tile, the unit of work
constexpr int kAttnRows = 128;         // query rows of one tile (tensor-memory lanes of an MMA)
constexpr int kAttnMaxRequests = 4096;

// Findings of the device side, reported by pw_attn_check.
enum {
  kAttnErrWait = 1,    // a bounded wait expired
  kAttnErrLen = 2,     // a negative length, or more tokens than a table row can hold
  kAttnErrTokens = 4,  // new tokens beyond n_tokens
  kAttnErrIds = 8,     // fewer new ids than opened blocks
  kAttnErrBlock = 16,  // a block id or a table row out of range
};

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
  int tile, head, off, n;  // key tile `off` of (tile, head); n key tiles in all
};

// One list of work.  The units are key tiles, in the order (tile, head, key tile); CTA c of P
// takes the units [c W / P, (c + 1) W / P) of the W.
struct AttnList {
  AttnTile *tiles;
  int *cum;          // [tiles + 1] key tiles of one head before each tile
  AttnStart *start;  // [P]
  int *meta;         // [0] tiles, [1] key tiles of one head
  int tpt;           // tokens of one 128-row tile
  int streams;       // 128-row tiles of one AttnTile (1 or 2)
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

struct AttnArgs {
  const RowBound *bounds;
  const int *table;
  int table_stride, n_tokens, n_blocks, log_bt;
  int Hq, Hkv, G, D;
  const uint16_t *q;
  int64_t q_token, q_head;
  uint16_t *o;
  int64_t o_token, o_head;
  const uint16_t *kc, *vc;
  int64_t block_stride, token_stride, head_stride;
  float *lse;
  float scale, softcap;
  const float *slopes;
  int *err;
  long long wait_cycles;
};

int launch_kv_map(const MapArgs &a, void *stream);
int launch_attn_plan(const PlanArgs &a, int want_bounds, void *stream);
int launch_attn_append(const AppendArgs &a, void *stream);
int launch_attn(const AttnArgs &a, int bf16, void *stream);

}  // namespace pw
