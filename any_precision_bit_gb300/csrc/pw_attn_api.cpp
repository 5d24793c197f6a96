// pw_attn_api.cpp -- host side of the paged-attention calls of include/pw.h: the handle, its
// argument checks and launches.  Nothing is allocated after creation.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <new>
#include <tuple>
#include <vector>

#include "pw_attn.h"

using namespace pw;

namespace {

// Measured (us), pieces added up by the last CTA to arrive and by attn_join_kernel.  Two tiles: 64 new tokens behind
// 32000 71 and 39, 100 behind 1000 28 and 16, 256 behind 32000 (4 pieces a tile) 104 and 96, 700 in three
// requests (1.5 pieces) 28.8 and 31.7.  Few rows: one request behind 131000 with one key/value head 55 and 23, behind
// 32000 with two 32 and 16, with four 28 and 21; with eight (8 pieces by this count) behind 517 10.9 and 12.4.
constexpr int kJoinTwo = 2, kJoinSpread = 16;

// Where heads stand side by side in a cache and do not fill 256 bytes, a copy that has L2 fetch 256 bytes brings part of
// the next head, too, whose turn on this SM comes a whole row of keys later.  While all SMs' keys of a head fit into
// this many bytes of L2 that is a gain; beyond, most of it is fetched twice and 64 bytes are better.  Measured, 80
// requests of 16 heads of 64 and a window (us, 256 and 64 bytes): 300 keys 46 and 49, 1024 (40 MB) 94 and 97, 1500
// (58 MB) 130 and 124, 4096 339 and 275; 8 heads of 96: 300 keys 42 and 42, 1024 (60 MB) 87 and 77, 3000 212 and 162.
// Rows of 256 bytes, or heads outermost: both alike (8 heads of 128 212 and 214).
constexpr int64_t kReuseBytes = 48 << 20;

// A forward over shared prefixes begins its last kernel while the one before adds results up, or computes rows again
// there: at most 32 rows a warp in each of 16 pieces of work, at 0.24 us a key alone and 0.4 us with all warps at it.
// That kernel's waits last so many SM cycles longer for each key that a row may see (16384 keys: 4 s).  (Waiting for the
// other kernel in the waits themselves made prefix-64 1.4 us slower.)
constexpr int64_t kRedoCycles = 32 * 16 * 1024;

pw_status bad(const char *msg) { return report(nullptr, PW_ERR_INVALID, msg); }
pw_status cuda_failed(const char *what, int e) {
  cudaGetLastError();
  char buf[256];
  snprintf(buf, sizeof buf, "%s failed: %s", what, cudaGetErrorString((cudaError_t)e));
  return report(nullptr, PW_ERR_CUDA, buf);
}

// Tensor map of 16-bit elements with the 128-byte swizzle: dim[0] contiguous, the others `stride` elements
// apart, boxes of box[] elements (64 along dim 0); what lies outside reads as zeros.
bool encode_map(TmaDesc *out, const void *base, int rank, const cuuint64_t *dim, const int64_t *stride,
                const cuuint32_t *box, CUtensorMapL2promotion fetch = CU_TENSOR_MAP_L2_PROMOTION_L2_256B) {
  using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode fn = []() -> Encode {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    return reinterpret_cast<Encode>(p);
  }();
  if (!fn) return false;
  const cuuint32_t one[4] = {1, 1, 1, 1};
  cuuint64_t bytes[3];
  for (int i = 0; i + 1 < rank; ++i) bytes[i] = (cuuint64_t)stride[i] * 2;
  return fn(reinterpret_cast<CUtensorMap *>(out), CU_TENSOR_MAP_DATA_TYPE_UINT16, (cuuint32_t)rank,
            const_cast<void *>(base), dim, bytes, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, fetch,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Layer {
  uint16_t *k = nullptr, *v = nullptr;
  TmaDesc map_k[2], map_v[2];  // L2 fetches 256 bytes, or 64 (see kReuseBytes)
  int64_t block_stride = 0, token_stride = 0, head_stride = 0;
  // its rotation; rope.table is null before pw_attn_set_rope
  RopeArgs rope{};
  int rope_axes = 0;
};

// A cache of keys or of values.
struct CacheRef {
  uint16_t *base;
  int64_t block_stride, token_stride, head_stride;
  auto strides() const { return std::tie(block_stride, token_stride, head_stride); }
};

struct Plan {
  bool set = false;
  pw_kv_step step{};
  int64_t reach = 0;           // keys that a row sees at most
  RowBound *bounds = nullptr;  // [max_tokens]
  AttnShape *shape = nullptr;  // as laid out on the device
  uint32_t *seen = nullptr;    // [max_tree_tokens][kTreeWords]
  bool tree = false;           // laid out by pw_attn_plan_tree
  AttnList requests{}, groups{};

  AttnShape launch_shape() const {
    AttnShape s{requests.tpt, requests.streams + (tree ? kTreeShape * requests.two : 0), 0, 0, step.n_tokens, step.table_stride, step.table};
    if (step.n_groups) {
      s.group_tpt = groups.tpt;
      s.group_streams = groups.streams + (tree ? kTreeShape * groups.two : 0);
    }
    return s;
  }
};

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool good_stride(int64_t s) { return s > 0 && s % 8 == 0; }

int log2_of(int v) {
  int l = 0;
  while ((1 << l) < v) ++l;
  return l;
}

// f / 2 pi modulo one turn, in units of 2^-64 to the nearest (f finite): for f = m 2^e with a whole m the bits of 1 / 2 pi from the
// (e + 1)st behind the point on, all that is left of 2^e / 2 pi, times m (the reduction of Payne and Hanek, 1983).  128 of
// those bits are enough: m < 2^53.  (In double f / 2 pi has 53 bits at best, which 2^31 positions later is 2^-22 of a turn and
// more; negative and large f lose more than that.)
uint64_t turn_of(double f) {
  static const uint64_t kBits[18] = {  // of 1 / 2 pi behind the point, computed by Machin's formula
    0x28be60db9391054a, 0x7f09d5f47d4d3770, 0x36d8a5664f10e410, 0x7f9458eaf7aef158, 0x6dc91b8e909374b8,
    0x01924bba82746487, 0x3f877ac72c4a69cf, 0xba208d7d4baed121, 0x3a671c09ad17df90, 0x4e64758e60d4ce7d,
    0x272117e2ef7e4a0e, 0xc7fe25fff7816603, 0xfbcbc462d6829b47, 0xdb4d9fb3c9f2c26d, 0xd3d18fd9a797fa8b,
    0x5d49eeb1faf97c5e, 0xcf41ce7de294a4ba, 0x9afed7ec47e35742};
  using u128 = unsigned __int128;
  int e;
  const double m = std::frexp(std::fabs(f), &e);
  const uint64_t whole = (uint64_t)std::ldexp(m, 53);
  e -= 53;  // at most 971: 128 bits from there on are in the table
  const int at = e >= 0 ? e / 64 : -((63 - e) / 64), shift = e - 64 * at;
  auto word = [&](int i) { return i >= 0 && i < 18 ? kBits[i] : 0; };
  auto from = [&](int i) { return shift ? word(i) << shift | word(i + 1) >> (64 - shift) : word(i); };
  const u128 turns = ((u128)from(at) << 64 | from(at + 1)) * whole;
  const uint64_t turn = (uint64_t)((turns + ((u128)1 << 63)) >> 64);
  return f < 0 ? 0 - turn : turn;
}

// Makes the handle's device current for a call and puts the caller's back.
struct OnDevice {
  int before = -1;
  bool ok;
  explicit OnDevice(int dev) {
    ok = cudaGetDevice(&before) == cudaSuccess && (before == dev || cudaSetDevice(dev) == cudaSuccess);
    if (before == dev) before = -1;
  }
  ~OnDevice() {
    if (before >= 0) cudaSetDevice(before);
  }
};

}  // namespace

struct pw_attn {
  pw_attn_desc d{};
  int sm_count = 0;
  std::vector<Layer> layers;
  std::vector<Plan> plans;
  std::vector<void *> allocs;
  std::vector<CacheRef> caches;  // what the layers are bound to, each once; empty since a layer was bound anew
  bool caches_mixed = false;     // some of them begin at one address with other strides
  int *err = nullptr;
  float *part_o = nullptr, *prefix_o = nullptr, *prefix_lse = nullptr;
  float2 *part_ml = nullptr;
  int *counters = nullptr;
  uint32_t *marks = nullptr, *part_odd = nullptr;
  RopeTable *rope = nullptr;  // [L]
  int *where = nullptr;       // [n_blocks] see CopyArgs
  size_t mark_words = 0;
  long long wait_cycles = kWaitCyclesDefault;
  int fault_withhold = 0;  // testing: the next forward withholds one device barrier arrival
};

namespace {

pw_status check_step(const pw_attn *a, const pw_kv_step *s) {
  if (!a || !s) return bad("null argument");
  if (s->R < 1 || s->R > a->d.max_requests) return bad("R must be in 1..max_requests");
  if (s->n_tokens < 1 || s->n_tokens > a->d.max_tokens) return bad("n_tokens must be in 1..max_tokens");
  if (s->max_new < 0) return bad("max_new must not be negative");
  if (s->table_rows < 1 || s->table_stride < 1) return bad("the table needs rows and entries");
  if (!s->rows && s->table_rows < s->R) return bad("without `rows` the table needs a row for each request");
  if ((int64_t)s->table_stride * a->d.block_tokens > INT32_MAX) return bad("a table row holds 2^31 tokens or more");
  if (!s->ctx_len || !s->new_len || !s->table || !s->q_start || !s->kv_len || !s->slot || !s->pos)
    return bad("null pointer in the step");
  if (s->n_groups < 0 || s->n_groups > s->R) return bad("n_groups must be in 0..R");
  if (s->n_groups > 0) {
    if (!s->group_start || !s->shared_len) return bad("groups without group_start or shared_len");
    if (s->n_tokens > a->d.max_shared_tokens) return bad("n_tokens of a step with groups exceeds max_shared_tokens");
  }
  return PW_OK;
}

template <class T>
bool alloc(pw_attn *a, T **p, size_t n) {
  void *q = nullptr;
  if (cudaMalloc(&q, n * sizeof(T) + 16) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  a->allocs.push_back(q);  // capacity reserved at creation
  *p = static_cast<T *>(q);
  return true;
}

pw_status create(const pw_attn_desc &d, pw_attn *a) {
  a->d = d;
  a->layers.resize((size_t)d.L);
  a->plans.resize((size_t)d.n_plans);
  a->allocs.reserve(16 + 14 * (size_t)d.n_plans);
  a->caches.reserve(2 * (size_t)d.L);
  int e = cudaDeviceGetAttribute(&a->sm_count, cudaDevAttrMultiProcessorCount, d.device);
  if (e) return cuda_failed("cudaDeviceGetAttribute", e);
  const size_t ctas = (size_t)a->sm_count, dp = d.head_dim > 64 ? 128 : 64;
  a->mark_words = ((size_t)d.max_tokens * d.n_heads + 31) / 32;
  bool ok = alloc(a, &a->marks, a->mark_words) && alloc(a, &a->err, 1) && alloc(a, &a->counters, 2 * ctas) &&
            alloc(a, &a->part_o, ctas * 4 * kAttnRows * dp) && alloc(a, &a->part_ml, ctas * 4 * kAttnRows) &&
            alloc(a, &a->part_odd, ctas * 4 * kAttnRows) && alloc(a, &a->rope, (size_t)d.L) &&
            alloc(a, &a->where, (size_t)d.n_blocks);
  if (d.max_shared_tokens > 0)
    ok = ok && alloc(a, &a->prefix_o, (size_t)d.max_shared_tokens * d.n_heads * d.head_dim) &&
         alloc(a, &a->prefix_lse, (size_t)d.max_shared_tokens * d.n_heads);
  // a tile holds a token at least, but the last of each segment may be short: requests and the padding, or groups
  for (Plan &p : a->plans) {
    ok = ok && alloc(a, &p.bounds, (size_t)d.max_tokens) && alloc(a, &p.shape, 1);
    if (d.max_tree_tokens > 0) ok = ok && alloc(a, &p.seen, (size_t)d.max_tree_tokens * kTreeWords);
    for (AttnList *l : {&p.requests, &p.groups}) {
      if (l == &p.groups && d.max_shared_tokens == 0) continue;
      if (l == &p.groups) {
        // full tiles of at least 128 / G tokens (or of all a step's), and the short last one of each group
        const int G = d.n_heads / d.n_kv_heads;
        l->max_tiles = d.max_shared_tokens / std::min(kAttnRows / G, d.max_shared_tokens) + d.max_requests;
      } else {
        l->max_tiles = d.max_tokens + d.max_requests + 1;
      }
      ok = ok && alloc(a, &l->tiles, (size_t)l->max_tiles + 1) && alloc(a, &l->cum, (size_t)l->max_tiles + 1) &&
           alloc(a, &l->start, ctas) && alloc(a, &l->meta, 3) && alloc(a, &l->splits, ctas);
    }
  }
  if (!ok) return report(nullptr, PW_ERR_OOM, "device memory exhausted");
  if ((e = cudaMemset(a->err, 0, sizeof(int))) || (e = cudaMemset(a->counters, 0, 2 * ctas * sizeof(int))) ||
      (e = cudaMemset(a->marks, 0, a->mark_words * sizeof(uint32_t))) ||
      (e = cudaMemset(a->where, 0, (size_t)d.n_blocks * sizeof(int))))
    return cuda_failed("cudaMemset", e);
  for (Plan &p : a->plans)
    if ((e = cudaMemset(p.shape, 0, sizeof(AttnShape)))) return cuda_failed("cudaMemset", e);
  if ((e = cudaDeviceSynchronize())) return cuda_failed("cudaDeviceSynchronize", e);
  return PW_OK;
}

// Lists the caches of all layers, each once: layers may share them, and keys and values may be one.
pw_status list_caches(pw_attn *a) {
  if (!a->caches.empty()) return PW_OK;
  for (const Layer &l : a->layers)
    if (!l.k) return report(nullptr, PW_ERR_STATE, "a layer's cache is not bound");
  for (const Layer &l : a->layers)
    for (uint16_t *base : {l.k, l.v})  // (strides along a length of one say nothing; the room is reserved at creation)
      a->caches.push_back(CacheRef{base, a->d.n_blocks > 1 ? l.block_stride : 0, l.token_stride,
                                   a->d.n_kv_heads > 1 ? l.head_stride : a->d.head_dim});
  auto at = [](const CacheRef &c) { return reinterpret_cast<uintptr_t>(c.base); };
  auto meet = [](const CacheRef &x, const CacheRef &y) { return x.base == y.base; };
  auto same = [&](const CacheRef &x, const CacheRef &y) { return meet(x, y) && x.strides() == y.strides(); };
  std::sort(a->caches.begin(), a->caches.end(), [&](const CacheRef &x, const CacheRef &y) {
    return at(x) != at(y) ? at(x) < at(y) : x.strides() < y.strides();
  });
  a->caches.erase(std::unique(a->caches.begin(), a->caches.end(), same), a->caches.end());
  a->caches_mixed = std::adjacent_find(a->caches.begin(), a->caches.end(), meet) != a->caches.end();
  std::sort(a->caches.begin(), a->caches.end(), [&](const CacheRef &x, const CacheRef &y) {
    return x.strides() != y.strides() ? x.strides() < y.strides() : at(x) < at(y);
  });
  return PW_OK;
}

// The listed caches, at most kMoveCaches of the same strides a launch: launch(caches, their number, whether they are the first).
template <class F>
pw_status for_caches(const pw_attn *a, const char *what, F launch) {
  MoveCaches m;
  const std::vector<CacheRef> &c = a->caches;
  int n = 0;
  for (size_t at = 0; at < c.size(); at += (size_t)n) {
    for (n = 0; n < kMoveCaches && at + n < c.size() && c[at + n].strides() == c[at].strides(); ++n) m.base[n] = c[at + n].base;
    std::tie(m.block_stride, m.token_stride, m.head_stride) = c[at].strides();
    if (int e = launch(m, n, at == 0)) return cuda_failed(what, e);
  }
  return PW_OK;
}

// pw_attn_plan, or with a tree pw_attn_plan_tree.
pw_status lay_out(pw_attn *a, int plan, const pw_kv_step *s, int window, const int32_t *doc_start,
                  const int32_t *bidir_len, const pw_tree *tree, pw_stream stream) {
  if (pw_status st = check_step(a, s)) return st;
  if (plan < 0 || plan >= a->d.n_plans) return bad("plan out of range");
  if (window < 0) return bad("window must not be negative");
  PlanArgs g{};
  g.R = s->R;
  g.n_tokens = s->n_tokens;
  g.table_rows = s->table_rows;
  g.table_stride = s->table_stride;
  g.bt = a->d.block_tokens;
  g.ctx_len = s->ctx_len;
  g.rows = s->rows;
  g.q_start = s->q_start;
  g.kv_len = s->kv_len;
  g.doc_start = doc_start;
  g.bidir_len = bidir_len;
  g.window = window;
  g.n_groups = s->n_groups;
  g.group_start = s->group_start;
  g.shared_len = s->shared_len;
  g.ctas = a->sm_count;
  g.n_kv_heads = a->d.n_kv_heads;
  const int G = a->d.n_heads / a->d.n_kv_heads, most = kAttnRows / G;
  auto shape = [&](AttnList &l, int tokens) {
    tokens = std::max(tokens, 1);
    l.streams = (int64_t)tokens * G > kSpreadRows ? 2 : 1;  // the kernel's form: see pw_attn.h
    l.tpt = std::min(most, tokens);
    // measured: two tiles, 8192-token prompt 479, 417, 395, 397, 401 us at 1 to 5 and packed chunks 66, 66, 68,
    // 71, 73 us; few rows, 160 windowed requests 137, 137, 138 us at 1 to 3
    l.piece_cost = l.streams == 2 ? 3 : 2;
    l.one = l.two = 1;
    // Where some tiles hold two 128-row tiles and others one: a key tile of the latter, which the streams take in turns, is
    // memory's or the copies' more often than theirs.
    // Measured, weights 1 : 1, 2 : 3 and 1 : 2 (us): prompt chunks among trees 54, 47 and 46, 32 trees of up to 33 nodes 122,
    // 109 and 112, of up to 64 127, 130 and 153; a piece at 6, 9 and 12: chunks among trees 47.7, 47.1 and 47.8.
    if (tree && l.streams == 2 && tokens > most) {
      l.one = 2;
      l.two = 3;
      l.piece_cost = 8;
    }
  };
  // The lists sum up key tiles (and a piece's cost) over all tiles of rows in 31 bits, as they do an SM's share over
  // the heads.
  const int64_t keys = ((int64_t)s->table_stride * a->d.block_tokens + kAttnKeys - 1) / kAttnKeys;
  auto countable = [&](const AttnList &l, int segments) {
    const int64_t sum = (s->n_tokens / (l.tpt * l.streams) + (int64_t)segments) * (keys * l.two + l.piece_cost);
    return sum <= INT32_MAX && sum * a->d.n_kv_heads / a->sm_count < INT32_MAX;
  };
  AttnList requests = a->plans[(size_t)plan].requests, groups = a->plans[(size_t)plan].groups;
  shape(requests, s->max_new);
  shape(groups, s->n_tokens);
  if (!countable(requests, s->R + 1) || (s->n_groups && !countable(groups, s->n_groups)))
    return bad("table_stride is too long for this many tokens (2^31 key tiles or more)");
  OnDevice dev(a->d.device);
  Plan &p = a->plans[(size_t)plan];
  p.reach = std::min((int64_t)s->table_stride * a->d.block_tokens,
                     window ? (int64_t)window + s->max_new + (tree ? PW_TREE_NODES : 0) : INT64_MAX);
  p.set = false;
  p.tree = tree != nullptr;
  p.requests = requests;
  p.groups = groups;
  p.step = *s;
  g.bounds = p.bounds;
  g.shape = p.launch_shape();
  g.shape_out = p.shape;
  int e;
  if (tree) {
    TreeArgs t{g, tree->tree_len, tree->parent, tree->parent_stride, tree->pos, p.seen, a->err};
    if (!s->n_groups && tree_blocks(t) <= kTreeListBlocks) {
      t.plan.list = p.requests;
      if ((e = launch_tree_list(t, stream))) return cuda_failed("pw_attn_plan_tree launch", e);
      p.set = true;
      return PW_OK;
    }
    e = launch_tree_bounds(t, stream);
  } else {
    e = launch_attn_bounds(g, stream);
  }
  if (!e && s->n_groups) {
    g.of_groups = 1;
    g.list = p.groups;
    e = launch_attn_list(g, stream);
  }
  g.of_groups = 0;
  g.list = p.requests;
  if (!e) e = launch_attn_list(g, stream);
  if (e) return cuda_failed("pw_attn_plan launch", e);
  p.set = true;
  return PW_OK;
}

}  // namespace

extern "C" {

pw_status pw_attn_create(const pw_attn_desc *desc, pw_attn **out) {
  if (!desc || !out) return bad("null argument");
  *out = nullptr;
  const pw_attn_desc &d = *desc;
  if (d.L < 1 || d.L > 4096) return bad("L must be in 1..4096");
  if (d.n_kv_heads < 1 || d.n_heads < d.n_kv_heads || d.n_heads % d.n_kv_heads || d.n_heads > 1024)
    return bad("n_heads must be a multiple of n_kv_heads, at most 1024");
  if (d.n_heads / d.n_kv_heads > kAttnRows) return bad("at most 128 query heads share a key/value head");
  if (d.head_dim < 8 || d.head_dim % 8 || d.head_dim > 128) return bad("head_dim must be a multiple of 8 in 8..128");
  if (d.dtype != PW_BF16 && d.dtype != PW_FP16) return bad("dtype must be PW_BF16 or PW_FP16");
  if (d.n_blocks < 1) return bad("n_blocks must be positive");
  if (d.block_tokens != 16 && d.block_tokens != 32 && d.block_tokens != 64 && d.block_tokens != 128)
    return bad("block_tokens must be 16, 32, 64 or 128");
  if (d.max_requests < 1 || d.max_requests > kAttnMaxRequests) return bad("max_requests must be in 1..4096");
  if (d.max_tokens < 1 || d.max_tokens > (1 << 20)) return bad("max_tokens must be in 1..2^20");
  if (d.max_shared_tokens < 0 || d.max_shared_tokens > d.max_tokens)
    return bad("max_shared_tokens must be in 0..max_tokens");
  if (d.max_tree_tokens < 0 || d.max_tree_tokens > d.max_tokens) return bad("max_tree_tokens must be in 0..max_tokens");
  if (d.n_plans < 1 || d.n_plans > 16) return bad("n_plans must be in 1..16");
  OnDevice dev(d.device);
  if (!dev.ok) return cuda_failed("cudaSetDevice", cudaGetLastError());
  pw_attn *a = new (std::nothrow) pw_attn;
  if (!a) return report(nullptr, PW_ERR_OOM, "host memory exhausted");
  pw_status st;
  try {
    st = create(d, a);
  } catch (...) {
    st = report(nullptr, PW_ERR_OOM, "host memory exhausted");
  }
  if (st) {
    for (void *p : a->allocs) cudaFree(p);
    delete a;
    return st;
  }
  *out = a;
  return PW_OK;
}

void pw_attn_destroy(pw_attn *a) {
  if (!a) return;
  OnDevice dev(a->d.device);
  cudaDeviceSynchronize();
  for (void *p : a->allocs) cudaFree(p);
  delete a;
}

pw_status pw_attn_bind(pw_attn *a, int layer, void *k, void *v, int64_t block_stride, int64_t token_stride,
                       int64_t head_stride) {
  if (!a || !k || !v) return bad("null argument");
  if (layer < 0 || layer >= a->d.L) return bad("layer out of range");
  if (!aligned16(k) || !aligned16(v)) return bad("cache addresses must be multiples of 16 bytes");
  if (!good_stride(block_stride) || !good_stride(token_stride) || !good_stride(head_stride))
    return bad("cache strides must be positive multiples of 8 elements");
  OnDevice dev(a->d.device);
  const pw_attn_desc &d = a->d;
  const cuuint64_t dim[4] = {(cuuint64_t)d.head_dim, (cuuint64_t)d.block_tokens, (cuuint64_t)d.n_kv_heads,
                             (cuuint64_t)d.n_blocks};
  const int64_t stride[3] = {token_stride, head_stride, block_stride};
  const cuuint32_t box[4] = {64, (cuuint32_t)d.block_tokens, 1, 1};
  Layer n = a->layers[(size_t)layer], &l = a->layers[(size_t)layer];
  for (int i = 0; i < 2; ++i) {
    const auto fetch = i ? CU_TENSOR_MAP_L2_PROMOTION_L2_64B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
    if (!encode_map(&n.map_k[i], k, 4, dim, stride, box, fetch) || !encode_map(&n.map_v[i], v, 4, dim, stride, box, fetch))
      return bad("no tensor map can describe this cache (address or strides)");
  }
  l = n;
  l.k = static_cast<uint16_t *>(k);
  l.v = static_cast<uint16_t *>(v);
  l.block_stride = block_stride;
  l.token_stride = token_stride;
  l.head_stride = head_stride;
  a->caches.clear();
  return PW_OK;
}

pw_status pw_kv_map(pw_attn *a, const pw_kv_step *s, const int32_t *new_ids, int n_ids, pw_stream stream) {
  if (pw_status st = check_step(a, s)) return st;
  if (n_ids < 0 || (n_ids > 0 && !new_ids)) return bad("n_ids ids are needed");
  OnDevice dev(a->d.device);
  MapArgs m{};
  m.R = s->R;
  m.n_tokens = s->n_tokens;
  m.table_rows = s->table_rows;
  m.table_stride = s->table_stride;
  m.bt = a->d.block_tokens;
  m.n_blocks = a->d.n_blocks;
  m.n_ids = n_ids;
  m.ctx_len = s->ctx_len;
  m.new_len = s->new_len;
  m.rows = s->rows;
  m.new_ids = new_ids;
  m.table = s->table;
  m.q_start = s->q_start;
  m.kv_len = s->kv_len;
  m.pos = s->pos;
  m.slot = s->slot;
  m.err = a->err;
  if (int e = launch_kv_map(m, stream)) return cuda_failed("pw_kv_map launch", e);
  return PW_OK;
}

pw_status pw_attn_plan(pw_attn *a, int plan, const pw_kv_step *s, int window, const int32_t *doc_start,
                       const int32_t *bidir_len, pw_stream stream) {
  return lay_out(a, plan, s, window, doc_start, bidir_len, nullptr, stream);
}

pw_status pw_attn_plan_tree(pw_attn *a, int plan, const pw_kv_step *s, int window, const pw_tree *tree, pw_stream stream) {
  if (!a || !s || !tree || !tree->tree_len || !tree->parent) return bad("null argument");
  if (tree->parent_stride < 1) return bad("parent_stride must be positive");
  if (s->n_tokens > a->d.max_tree_tokens) return bad("n_tokens of a step with trees exceeds max_tree_tokens");
  // (the kernels put the tree of a row that is in none at INT_MAX, behind every key)
  if ((int64_t)s->table_stride * a->d.block_tokens > INT32_MAX - 1024) return bad("a table row holds nearly 2^31 tokens");
  return lay_out(a, plan, s, window, nullptr, nullptr, tree, stream);
}

pw_status pw_attn_append(pw_attn *a, int layer, const pw_kv_step *s, const void *k, int64_t k_token,
                         int64_t k_head, const void *v, int64_t v_token, int64_t v_head, pw_stream stream) {
  if (pw_status st = check_step(a, s)) return st;
  if (!k || !v) return bad("null argument");
  if (layer < 0 || layer >= a->d.L) return bad("layer out of range");
  if (!aligned16(k) || !aligned16(v)) return bad("k and v must be multiples of 16 bytes");
  if (k_token % 8 || k_head % 8 || v_token % 8 || v_head % 8) return bad("strides must be multiples of 8 elements");
  const Layer &l = a->layers[(size_t)layer];
  if (!l.k) return report(nullptr, PW_ERR_STATE, "the layer's cache is not bound");
  OnDevice dev(a->d.device);
  AppendArgs g{};
  g.k = static_cast<const uint16_t *>(k);
  g.v = static_cast<const uint16_t *>(v);
  g.k_token = k_token;
  g.k_head = k_head;
  g.v_token = v_token;
  g.v_head = v_head;
  g.kc = l.k;
  g.vc = l.v;
  g.block_stride = l.block_stride;
  g.token_stride = l.token_stride;
  g.head_stride = l.head_stride;
  g.slot = s->slot;
  g.n_tokens = s->n_tokens;
  g.n_heads = a->d.n_kv_heads;
  g.head_dim = a->d.head_dim;
  g.bt = a->d.block_tokens;
  g.log_bt = log2_of(a->d.block_tokens);
  g.n_blocks = a->d.n_blocks;
  if (int e = launch_attn_append(g, stream)) return cuda_failed("pw_attn_append launch", e);
  return PW_OK;
}

pw_status pw_attn_forward(pw_attn *a, int layer, int plan, const void *q, int64_t q_token, int64_t q_head,
                          void *o, int64_t o_token, int64_t o_head, float *lse, float scale, float softcap,
                          const float *slopes, pw_stream stream) {
  if (!a || !q || !o) return bad("null argument");
  if (layer < 0 || layer >= a->d.L) return bad("layer out of range");
  if (plan < 0 || plan >= a->d.n_plans) return bad("plan out of range");
  if (!aligned16(q) || !aligned16(o)) return bad("q and o must be multiples of 16 bytes");
  if (!good_stride(q_token) || !good_stride(q_head) || !good_stride(o_token) || !good_stride(o_head))
    return bad("strides of q and o must be positive multiples of 8 elements");
  if (!std::isfinite(scale)) return bad("scale must be finite");
  if (!(softcap >= 0.f) || !std::isfinite(softcap)) return bad("softcap must be finite and not negative");
  const Layer &l = a->layers[(size_t)layer];
  const Plan &p = a->plans[(size_t)plan];
  if (!l.k) return report(nullptr, PW_ERR_STATE, "the layer's cache is not bound");
  if (!p.set) return report(nullptr, PW_ERR_STATE, "the plan was never set");
  OnDevice dev(a->d.device);
  AttnArgs g{};
  g.bounds = p.bounds;
  g.shape = p.launch_shape();
  g.planned = p.shape;
  g.table = p.step.table;
  g.table_stride = p.step.table_stride;
  g.n_tokens = p.step.n_tokens;
  g.n_blocks = a->d.n_blocks;
  g.log_bt = log2_of(a->d.block_tokens);
  g.device = a->d.device;
  g.Hq = a->d.n_heads;
  g.Hkv = a->d.n_kv_heads;
  g.G = g.Hq / g.Hkv;
  g.D = a->d.head_dim;
  g.g_magic = (65536u + (unsigned)g.G - 1u) / (unsigned)g.G;
  g.q = static_cast<const uint16_t *>(q);
  g.q_token = q_token;
  g.q_head = q_head;
  g.o = static_cast<uint16_t *>(o);
  g.o_token = o_token;
  g.o_head = o_head;
  g.kc = l.k;
  g.vc = l.v;
  g.block_stride = l.block_stride;
  g.token_stride = l.token_stride;
  g.head_stride = l.head_stride;
  g.lse = lse;
  g.scale = scale;
  g.softcap = softcap;
  g.slopes = slopes;
  g.scale2 = scale * 1.4426950408889634f;
  g.cap2 = softcap * 1.4426950408889634f;
  g.inv_cap = softcap > 0.f ? std::clamp(scale / softcap, -FLT_MAX, FLT_MAX) : 0.f;  // (0 scores stay 0)
  double power = (double)g.cap2 * g.inv_cap;
  for (int i = 0; i < 5; ++i, power *= (double)g.inv_cap * g.inv_cap) g.cap_poly[i] = (float)(kTanhPoly[i] * power);
  g.marks = a->marks;
  g.err = a->err;
  g.wait_cycles = a->wait_cycles;
  g.withhold = a->fault_withhold;
  a->fault_withhold = 0;
  g.part_o = a->part_o;
  g.part_ml = a->part_ml;
  g.part_odd = a->part_odd;
  g.counters = a->counters;
  g.ctas = a->sm_count;
  g.seen = p.tree ? p.seen : nullptr;
  AttnMaps maps;
  const bool apart = l.token_stride != g.D && g.D % 128;
  const int fetch = apart && p.reach * g.D * 4 * a->sm_count > kReuseBytes;
  maps.k = l.map_k[fetch];
  maps.v = l.map_v[fetch];
  const cuuint64_t dim[3] = {(cuuint64_t)g.D, (cuuint64_t)g.Hq, (cuuint64_t)g.n_tokens};
  const int64_t stride[2] = {q_head, q_token};
  auto launch = [&](const AttnList &list) -> pw_status {
    g.list = list;
    g.box_tokens = list.tpt;
    const cuuint32_t box[3] = {64, (cuuint32_t)g.G, (cuuint32_t)list.tpt};
    if (!encode_map(&maps.q, q, 3, dim, stride, box)) return bad("no tensor map can describe q (address or strides)");
    if (int e = launch_attn(g, maps, a->d.dtype == PW_BF16, stream)) return cuda_failed("pw_attn_forward launch", e);
    return PW_OK;
  };
  if (p.step.n_groups) {
    g.prefix_o = a->prefix_o;
    g.prefix_lse = a->prefix_lse;
    g.to_prefix = g.join = 1;
    if (pw_status st = launch(p.groups)) return st;
    g.to_prefix = 0;
    g.after_prefix = 1;
    g.wait_cycles += p.reach * kRedoCycles;
  }
  // Where tiles are few, each is split among many CTAs, and a kernel of its own adds up the pieces: from so many
  // pieces a tile on average.
  const int tiles = p.step.n_tokens / (p.requests.tpt * p.requests.streams) + p.step.R;
  g.join = (int64_t)tiles * g.Hkv * (p.requests.streams == 2 ? kJoinTwo : kJoinSpread) <= g.ctas;
  return launch(p.requests);
}

pw_status pw_attn_set_rope(pw_attn *a, int layer, const pw_rope_desc *r) {
  if (!a || !r) return bad("null argument");
  if (layer < 0 || layer >= a->d.L) return bad("layer out of range");
  if (r->rot_dim < 0 || r->rot_dim % 8 || r->rot_dim > a->d.head_dim)
    return bad("rot_dim must be a multiple of 8 in 0..head_dim");
  if (r->n_axes < 1 || r->n_axes > 4) return bad("n_axes must be in 1..4");
  if (r->rot_dim && !r->inv_freq) return bad("null argument");
  if (!std::isfinite(r->scale)) return bad("scale must be finite");
  if (!(r->eps >= 0.f) || !std::isfinite(r->eps)) return bad("eps must be finite and not negative");
  RopeTable t{};
  for (int i = 0; i < r->rot_dim / 2; ++i) {
    if (!std::isfinite(r->inv_freq[i])) return bad("inv_freq must be finite");
    if (r->axis && (r->axis[i] < 0 || r->axis[i] >= r->n_axes)) return bad("axis must be in 0..n_axes - 1");
    t.turn[i] = turn_of(r->inv_freq[i]);  // (whole turns fall away, since positions are whole numbers)
    t.axis[i] = r->axis ? r->axis[i] : 0;
  }
  OnDevice dev(a->d.device);
  if (!dev.ok) return cuda_failed("cudaSetDevice", cudaGetLastError());
  if (int e = cudaDeviceSynchronize()) return cuda_failed("cudaDeviceSynchronize", e);
  const float *gains[2] = {r->q_gain, r->k_gain};
  for (int i = 0; i < 2; ++i)
    if (gains[i])
      if (int e = cudaMemcpy(t.gain[i], gains[i], sizeof(float) * (size_t)a->d.head_dim, cudaMemcpyDefault))
        return cuda_failed("cudaMemcpy", e);
  RopeTable *table = a->rope + layer;
  if (int e = cudaMemcpy(table, &t, sizeof t, cudaMemcpyHostToDevice)) return cuda_failed("cudaMemcpy", e);
  // (the copy may return while its bytes are on their way, on a stream that the caller's need not wait for)
  if (int e = cudaDeviceSynchronize()) return cuda_failed("cudaDeviceSynchronize", e);
  Layer &l = a->layers[(size_t)layer];
  l.rope_axes = r->n_axes;
  l.rope.table = table;
  l.rope.rot = r->rot_dim;
  l.rope.interleaved = r->interleaved != 0;
  l.rope.norm_q = r->q_gain != nullptr;
  l.rope.norm_k = r->k_gain != nullptr;
  l.rope.scale = r->scale;
  l.rope.eps = r->eps;
  return PW_OK;
}

pw_status pw_attn_rope_append(pw_attn *a, int layer, const pw_kv_step *s, const void *q, int64_t q_token, int64_t q_head,
                              void *q_out, int64_t qo_token, int64_t qo_head, const void *k, int64_t k_token, int64_t k_head,
                              const void *v, int64_t v_token, int64_t v_head, const int32_t *pos, pw_stream stream) {
  if (pw_status st = check_step(a, s)) return st;
  if (!q || !q_out || !k || !v) return bad("null argument");
  if (layer < 0 || layer >= a->d.L) return bad("layer out of range");
  if (!aligned16(q) || !aligned16(q_out) || !aligned16(k) || !aligned16(v))
    return bad("q, q_out, k and v must be multiples of 16 bytes");
  for (int64_t stride : {q_token, q_head, qo_token, qo_head, k_token, k_head, v_token, v_head})
    if (stride % 8) return bad("strides must be multiples of 8 elements");
  const Layer &l = a->layers[(size_t)layer];
  if (!l.k) return report(nullptr, PW_ERR_STATE, "the layer's cache is not bound");
  if (!l.rope.table) return report(nullptr, PW_ERR_STATE, "the layer's rotation was never set");
  OnDevice dev(a->d.device);
  RopeArgs g = l.rope;
  g.q = static_cast<const uint16_t *>(q);
  g.q_token = q_token;
  g.q_head = q_head;
  g.qo = static_cast<uint16_t *>(q_out);
  g.qo_token = qo_token;
  g.qo_head = qo_head;
  g.k = static_cast<const uint16_t *>(k);
  g.k_token = k_token;
  g.k_head = k_head;
  g.v = static_cast<const uint16_t *>(v);
  g.v_token = v_token;
  g.v_head = v_head;
  g.kc = l.k;
  g.vc = l.v;
  g.block_stride = l.block_stride;
  g.token_stride = l.token_stride;
  g.head_stride = l.head_stride;
  g.slot = s->slot;
  g.pos = pos ? pos : s->pos;
  g.pos_axis = pos ? s->n_tokens : 0;
  g.n_tokens = s->n_tokens;
  g.sms = a->sm_count;
  g.Hq = a->d.n_heads;
  g.Hkv = a->d.n_kv_heads;
  g.D = a->d.head_dim;
  g.inv_d = 1.f / (float)a->d.head_dim;
  g.bt = a->d.block_tokens;
  g.log_bt = log2_of(a->d.block_tokens);
  g.n_blocks = a->d.n_blocks;
  if (int e = launch_rope(g, a->d.dtype == PW_BF16, stream)) return cuda_failed("pw_attn_rope_append launch", e);
  return PW_OK;
}

pw_status pw_kv_keep(pw_attn *a, const pw_kv_step *s, const int32_t *tree_len, const int32_t *keep, int keep_stride,
                     const int32_t *n_keep, int32_t *ctx_out, pw_stream stream) {
  if (pw_status st = check_step(a, s)) return st;
  if (!tree_len || !keep || !n_keep) return bad("null argument");
  if (keep_stride < 1) return bad("keep_stride must be positive");
  if (pw_status st = list_caches(a)) return st;
  if (a->caches_mixed) return report(nullptr, PW_ERR_STATE, "two layers' caches begin at one address with other strides");
  OnDevice dev(a->d.device);
  KeepArgs g{};
  g.R = s->R;
  g.table_rows = s->table_rows;
  g.table_stride = s->table_stride;
  g.keep_stride = keep_stride;
  g.bt = a->d.block_tokens;
  g.log_bt = log2_of(a->d.block_tokens);
  g.n_blocks = a->d.n_blocks;
  g.n_heads = a->d.n_kv_heads;
  g.head_dim = a->d.head_dim;
  g.rows = s->rows;
  g.table = s->table;
  g.kv_len = s->kv_len;
  g.tree_len = tree_len;
  g.keep = keep;
  g.n_keep = n_keep;
  g.err = a->err;
  return for_caches(a, "pw_kv_keep launch", [&](const MoveCaches &m, int n, bool first) {
    g.ctx_out = first ? ctx_out : nullptr;
    return launch_keep(g, m, n, stream);
  });
}

pw_status pw_kv_copy(pw_attn *a, const int32_t *src, const int32_t *dst, int n, int32_t *table, int table_rows, int table_stride,
                     pw_stream stream) {
  if (!a) return bad("null argument");
  if (n < 0 || (n > 0 && (!src || !dst))) return bad("n pairs are needed");
  if ((table || table_rows || table_stride) && (!table || table_rows < 1 || table_stride < 1))
    return bad("the table needs rows and entries");
  if (n > a->d.n_blocks) return bad("more pairs than the cache has blocks");
  if ((int64_t)n * ((int64_t)a->d.block_tokens * a->d.n_kv_heads * a->d.head_dim / 16384 + 1) > INT32_MAX - 1024)
    return bad("too many pairs for one call");
  if (pw_status st = list_caches(a)) return st;
  if (!n) return PW_OK;
  OnDevice dev(a->d.device);
  CopyArgs g{};
  g.src = src;
  g.dst = dst;
  g.n = n;
  g.n_blocks = a->d.n_blocks;
  g.bt = a->d.block_tokens;
  g.n_heads = a->d.n_kv_heads;
  g.head_dim = a->d.head_dim;
  g.err = a->err;
  g.entries = (int64_t)table_rows * table_stride;
  const bool few = n <= kRenamePairs && g.entries <= (1 << 20);
  pw_status st = for_caches(a, "pw_kv_copy launch", [&](const MoveCaches &m, int caches, bool first) {
    g.table = first && few ? table : nullptr;
    g.where = first && table && !few ? a->where : nullptr;
    return launch_copy(g, m, caches, stream);
  });
  if (st || !table || few) return st;
  g.table = table;
  g.where = a->where;
  if (int e = launch_rename(g, stream)) return cuda_failed("pw_kv_copy launch", e);
  return PW_OK;
}

pw_status pw_attn_set_fault(pw_attn *a, int kind, int n) {
  if (!a) return bad("null argument");
  if (n < 0 || (kind != 4 && kind != 5)) return bad("kind 4 or 5 and n >= 0");
  if (kind == 4) {
    a->fault_withhold = n != 0;
  } else {
    // cycles at the highest SM clock, so the wait lasts at least n microseconds
    a->wait_cycles = n ? 2100LL * n : kWaitCyclesDefault;
  }
  return PW_OK;
}

pw_status pw_attn_check(pw_attn *a, pw_stream stream) {
  if (!a) return bad("null argument");
  OnDevice dev(a->d.device);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int bits = 0, e;
  if ((e = cudaMemcpyAsync(&bits, a->err, sizeof bits, cudaMemcpyDeviceToHost, st)))
    return cuda_failed("cudaMemcpyAsync", e);
  if ((e = cudaStreamSynchronize(st))) return cuda_failed("cudaStreamSynchronize", e);
  if (!bits) return PW_OK;
  if ((e = cudaMemsetAsync(a->err, 0, sizeof bits, st)) ||
      (e = cudaMemsetAsync(a->counters, 0, 2 * sizeof(int) * (size_t)a->sm_count, st)) ||
      (e = cudaMemsetAsync(a->marks, 0, a->mark_words * sizeof(uint32_t), st)) ||
      (e = cudaStreamSynchronize(st)))
    return cuda_failed("cudaMemsetAsync", e);
  if (bits & kAttnErrWait) return report(nullptr, PW_ERR_TIMEOUT, "a bounded device wait expired; outputs are invalid");
  char buf[512];
  constexpr int kMapErrs = kAttnErrLen | kAttnErrTokens | kAttnErrIds | kAttnErrBlock;
  snprintf(buf, sizeof buf, "%s%s%s%s%s%s%s%s", bits & kMapErrs ? "pw_kv_map or pw_kv_keep found:" : "",
           bits & kAttnErrLen ? " a length out of range;" : "",
           bits & kAttnErrTokens ? " more new tokens than n_tokens;" : "",
           bits & kAttnErrIds ? " fewer new ids than opened blocks;" : "",
           bits & kAttnErrBlock ? " a block id or table row out of range;" : "",
           bits & kAttnErrPlan ? " a forward's plan is laid out for other tile sizes, n_tokens, table or groups than it was "
                                 "launched with: it wrote nothing;" : "",
           bits & kAttnErrTree ? " a tree's length or parent, or a node to be kept, out of range;" : "",
           bits & kAttnErrCopy ? " pw_kv_copy met a block id out of range" : "");
  return report(nullptr, PW_ERR_STATE, buf);
}

}  // extern "C"
