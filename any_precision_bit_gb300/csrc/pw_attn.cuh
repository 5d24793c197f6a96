// pw_attn.cuh -- attention over the paged key/value cache: the kernel and its launch, instantiated form by
// form in pw_attn_two.cu and pw_attn_spread.cu, and for trees of drafted tokens (TREE) in pw_attn_two_tree.cu and
// pw_attn_spread_tree.cu.
//
// For a query row q with keys lo <= j < hi, x_j = scale q.k_j (capped, biased) and o = sum_j e^{x_j} v_j / sum_j
// e^{x_j}, in one pass over the keys: with m a running reference, l = sum 2^{x_j log2 e - m} and O = sum
// 2^{x_j log2 e - m} v_j; where the maximum outgrows m, l and O are scaled by 2^{m - m'}.  Two partial results of a
// row join in the same way.
//
// A CTA (one to an SM) goes through its share of the units (a tile of 128 keys against a tile of query rows of one
// key/value head, see AttnList).  Warps have roles: producers copy queries, keys and values to shared memory block by
// block (TMA through the block table, 128-byte swizzle); one warp issues S = Q K^T and O += P V, S, P and O in tensor
// memory (S and P share columns); softmax warps turn S into P; and a piece of a tile's keys ends in the
// result, or in a partial one that is added up with the others' (the last CTA to arrive, or attn_join_kernel).
//
// Memory bounds the few-row form: 64 rows of 4 behind 0.26 to 8 thousand keys move 1.13 GB in 172 to 178 us, 6.4 to
// 6.6 TB/s; two producer warps (one for K, one for V) reached 5.2 TB/s, the copies' issue being their limit.  The
// two-tile form runs an 8192-token prompt of 32/8 heads of 128 at 1.42 PFLOP/s (388 us): a stream waits for its own
// products (512 + 512 cycles and 350 of latency) behind its softmax (1800 cycles), and tensor memory has no room for
// a second buffer of 128 scores beside two streams' S and O.
#pragma once
#include <cuda_runtime.h>
#include <limits.h>

#include <atomic>
#include <type_traits>

#include "pw_attn.h"
#include "pw_device.cuh"
#include "pw_tc.cuh"

// Code that hardly ever runs is kept out of line, since the instructions of the roles of a CTA share their
// cache; but not in kTwo, whose warps trade registers, which excludes calls.
#ifndef PW_RARE
#define PW_RARE __noinline__
#endif

namespace pw {

// ------------------------------------------------------------------ the tensor-core kernel
constexpr int kSmemRing = 227 * 1024 - 3072;  // dynamic shared memory: query tiles and the K/V ring
constexpr uint32_t kTmemColsAttn = 512;
constexpr uint32_t kSpinNs = 2000;

constexpr int kJoinRows = 8;  // rows added up at a time

template <int FORM, int DP>
struct Cfg {
  static constexpr int NS = FORM == kTwo ? 2 : 1;
  static constexpr int kHalves = DP / 64;             // 64-element column blocks of a head
  static constexpr int kHalfBytes = 128 * 128;        // 128 rows of 128 bytes
  static constexpr int kTileBytes = kHalves * kHalfBytes;
  // kSpread: the quarters' results side by side, rows padded against bank conflicts
  static constexpr int kScratchRow = DP + 4;
  static constexpr int kScratch = FORM == kSpread ? 4 * kJoinRows * kScratchRow * 4 + 2 * 4 * 32 * 8 : 0;
  static constexpr int kStages = (kSmemRing - NS * kTileBytes - kScratch) / kTileBytes;
  static constexpr int kScratchAt = (NS + kStages) * kTileBytes;
  static constexpr int kSmem = kScratchAt + kScratch;
  static constexpr int kSoftWarps = 4 * NS;
  // kSpread: four warps add up and write out a piece while the softmax warps are at the next; its outputs
  // take turns in two accumulators for that (kTwo has no tensor memory left to do so)
  static constexpr int kFinishWarps = FORM == kSpread ? 4 : 0;
  static constexpr int kProdWarp = kSoftWarps + kFinishWarps;
  // Producer warps: one for the keys and one for the values, two for each where the memory sets the pace (a
  // tensor copy takes its lane about 60 cycles, and 16-token blocks make 32 of them for a key tile).
  static constexpr int kProducers = FORM == kSpread ? 4 : 2;
  static constexpr int kMmaWarp = kProdWarp + kProducers;
  // and (two tiles) an idle warp that completes its warpgroup
  static constexpr int kThreads = FORM == kTwo ? 384 : 32 * (kMmaWarp + 1);
};
// Two tiles: 384 threads of 168 registers at launch, of which the softmax warps, which hold 128 scores
// each, need more: 256 x 216 + 128 x 72 = 384 x 168.
constexpr int kRegsSoft = 216, kRegsOther = 72;
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}

// A piece of work as the producer hands it to the other warps: consecutive key tiles of one (tile, head).
struct Piece {
  int n, first;  // key tiles, and the first one (n = 0: no more pieces)
  int head, tok0, ntok, trow, klo, khi;  // as in AttnTile; head of the keys
  int fresh;     // other rows than the last piece's
  int merge;     // merge with the rows' results over their shared prefix
  int c0, c1;    // CTAs of the (tile, head)'s first and last key tile; equal: the piece is all of it
};
constexpr int kPieces = 4;  // pieces handed over ahead

// mbarriers
template <int STAGES>
struct Bars {
  enum {
    kFull = 0,               // a stage's keys or values have landed
    kEmpty = STAGES,         // ... have been read by the MMAs
    kQF = 2 * STAGES,        // a query buffer has landed
    kQE = kQF + 2,           // ... its last scores are issued and done
    kSF = kQE + 2,           // scores are in tensor memory (kTwo: of a stream; kSpread: of even and odd key tiles)
    kPF = kSF + 2,           // probabilities are (four warps)
    kPE = kPF + 2,           // kTwo: those of the first keys
    kOD = kPE + 2,           // P V done: kTwo, a stream's last of a piece; kSpread, of an even or odd key tile
    kOF = kOD + 2,           // kSpread: an output accumulator holds a piece's result
    kOE = kOF + 2,           // ... has been read
    kML = kOE + 2,           // ... the piece's maxima and sums are in shared memory
    kJoin = kML + 2,         // four warps meet (a stream's, or the finishing warps)
    kDF = kJoin + 2,         // a piece has been handed over
    kDE = kDF + kPieces,     // ... every reader is done with it
    kDrain = kDE + kPieces,  // the MMA warp's last commit
    kMerge,                  // TREE, kTwo: the softmax warps of both streams meet
    kNum
  };
};

// Bounded wait on an mbarrier phase: false once the launch's limit is over or another warp has given up.
static __device__ PW_RARE bool wait_slow(uint32_t bar, uint32_t parity, volatile int *abort_flag, int *err,
                                       long long cycles) {
  const long long t0 = clock64();
  for (;;) {
    if (mbar_try_wait_sleep(bar, parity, kSpinNs)) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > cycles) break;
  }
  *abort_flag = 1;
  atomicOr(err, kAttnErrWait);
  return false;
}
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int *abort_flag, const AttnArgs &a) {
  return mbar_try_wait(bar, parity) || wait_slow(bar, parity, abort_flag, a.err, a.wait_cycles);
}
__device__ __forceinline__ bool wait_for_all(uint32_t bar, uint32_t parity, volatile int *abort_flag, const AttnArgs &a) {
  return __all_sync(0xffffffffu, wait_for(bar, parity, abort_flag, a));
}

// A CTA's way through its units: pieces of consecutive key tiles of one (tile, head).  The tile after
// the current one is fetched ahead of its use.
__device__ __forceinline__ AttnTile load_tile(const AttnTile *p) {
  const int4 x = reinterpret_cast<const int4 *>(p)[0], y = reinterpret_cast<const int4 *>(p)[1];
  AttnTile t;
  t.tok0 = x.x, t.ntok = x.y, t.trow = x.z, t.klo = x.w;
  t.khi = y.x, t.kv0 = y.y, t.kv1 = y.z, t.merge = y.w;
  return t;
}
// Slot of a split tile's piece among the partial results: a CTA's last piece, if it begins its tile, or its first.
__device__ __forceinline__ size_t part_slot(int cta, int c0, int streams, int s) {
  return ((size_t)cta * 2 + (cta == c0 ? 1 : 0)) * streams + s;
}
template <bool TREE>
struct Walk {
  int tile, head, off, left;  // off and left in units
  int cost;                   // units that lead each (tile, head)
  int tpt, one, two;
  AttnTile t, ahead;
  int j0, n;  // first key tile of this piece within the tile's, and their number
  int2 first_ctas, last_ctas;  // see AttnStart
  bool fresh; // the tile is another than the last piece's
  __device__ __forceinline__ Walk(const AttnArgs &a, bool fits) {
    const AttnStart *s = a.list.start + blockIdx.x;
    const int4 x = *reinterpret_cast<const int4 *>(s);
    t = load_tile(&s->t);
    tile = x.x, head = x.y, off = x.z, left = fits ? x.w : 0;
    first_ctas = s->first, last_ctas = s->last;
    cost = a.list.piece_cost;
    tpt = a.list.tpt;
    one = a.list.one, two = a.list.two;
    fresh = true;
    if (left > 0) ahead = load_tile(a.list.tiles + tile + 1);
  }
  __device__ __forceinline__ int units() const { return TREE ? (t.ntok > tpt ? two : one) : 1; }  // of a key tile
  __device__ __forceinline__ bool load(const AttnArgs &a) {
    for (;;) {
      if (off < cost) {
        const int skip = min(cost - off, left);
        off += skip;
        left -= skip;
      }
      if (left <= 0) return false;
      const int u = units(), o = off - cost;
      j0 = (o + u - 1) / u;
      n = min(t.kv1 - t.kv0, (o + left + u - 1) / u) - j0;
      if (!TREE || n > 0) return true;
      const bool f = fresh;  // the rest of a key tile that is the CTA's before
      next(a);
      fresh = fresh || f;
    }
  }
  __device__ __forceinline__ void next(const AttnArgs &a) {
    const int all = (t.kv1 - t.kv0) * units(), used = min(left, all - (off - cost));
    left -= used;
    off += used;
    fresh = false;
    if (off == all + cost) {
      off = 0;
      if (++head == a.Hkv) {
        head = 0;
        ++tile;
        fresh = true;
        t = ahead;
        if (left > 0) ahead = load_tile(a.list.tiles + tile + 1);
      }
    }
  }
  __device__ __forceinline__ int first() const { return t.kv0 + j0; }
  __device__ __forceinline__ void describe(const AttnArgs &a, Piece *p) const {
    int2 c = make_int2(0, 0);
    // a piece that lacks its tile's beginning is the CTA's first, one that lacks only its end the last
    if (n != t.kv1 - t.kv0) c = j0 > 0 ? first_ctas : last_ctas;
    *p = Piece{n, first(), head, t.tok0, t.ntok, t.trow, t.klo, t.khi, fresh, t.merge && !a.to_prefix, c.x, c.y};
  }
};

// The plan on the device is the one that this launch was made for.
__device__ __forceinline__ bool plan_fits(const AttnArgs &a) {
  const int4 x = reinterpret_cast<const int4 *>(a.planned)[0], y = reinterpret_cast<const int4 *>(a.planned)[1];
  const AttnShape &s = a.shape;
  const uint64_t table = (uint64_t)(uint32_t)y.z | (uint64_t)(uint32_t)y.w << 32;
  return x.x == s.tpt && x.y == s.streams && x.z == s.group_tpt && x.w == s.group_streams && y.x == s.n_tokens &&
         y.y == s.table_stride && table == reinterpret_cast<uint64_t>(s.table);
}

// Position in the ring of K/V stages.
template <int STAGES>
struct Ring {
  uint32_t st = 0, ph = 0;
  __device__ __forceinline__ void next() {
    if (++st == STAGES) {
      st = 0;
      ph ^= 1;
    }
  }
};

// Query buffers.  kSpread keeps a second box (of at most 16 rows) behind the first in each quarter's 32 rows, so
// that the next piece's queries are loaded while the current one's are in use.  (The MMAs read 128 rows from
// either; what lies between or behind a box's rows gives scores of rows that nobody has.)
template <int FORM>
constexpr uint32_t kQBuffers = FORM == kSpread ? 2 : 1;
constexpr uint32_t kQBufferStep = kSpreadRows * 128;  // bytes between the two

// A producer warp: the keys (kv = 0) or values of every key tile, or every other box of them; the last of
// the warps also loads the queries and hands the pieces over.
template <int FORM, int DP, bool TREE>
__device__ void produce(const AttnArgs &a, const AttnMaps &maps, int self, Piece *piece, uint32_t sm, uint32_t bars,
                        volatile int *abort_flag) {
  using C = Cfg<FORM, DP>;
  constexpr int NS = C::NS;
  using B = Bars<C::kStages>;
  constexpr int kShare = C::kProducers / 2;  // warps that share a tile's boxes
  const int lane = threadIdx.x & 31, kv = self / kShare, share = self % kShare;
  const bool leads = self == C::kProducers - 1;  // values are needed later than keys
  const int bt = 1 << a.log_bt, ppt = kAttnKeys >> a.log_bt;  // blocks of a key tile
  const int page = lane % ppt, half = lane / ppt;             // this lane's box
  const bool mine = half < C::kHalves;
  const bool loads = mine && lane % kShare == share;
  const uint32_t ring = sm + NS * C::kTileBytes;
  const uint32_t at = (uint32_t)(half * C::kHalfBytes + page * bt * 128);
  constexpr uint32_t nq = kQBuffers<FORM>;
  const void *map = kv ? &maps.v : &maps.k;
  uint32_t tiles = 0, pieces = 0;
  Ring<C::kStages> r;
  if (kv) r.next();
  // (where the plan does not fit there are no pieces, and the other warps find none)
  const bool fits = plan_fits(a);
  Walk<TREE> w(a, fits);
  if (!fits && leads) {
    if (a.after_prefix) pdl_wait();  // as every launch before its end
    if (lane == 0) atomicOr(a.err, kAttnErrPlan);
    __syncwarp();
  }
  bool ok = true;
  // the block of this lane's box of a key tile; -1: none of its keys counts
  auto block_of = [&](const AttnTile &t, int kt) {
    const int key0 = kt * kAttnKeys + page * bt;
    if (!mine || key0 >= t.khi || key0 + bt <= t.klo) return -1;
    const int p = key0 >> a.log_bt;
    int id = -1;
    if (t.trow >= 0 && p < a.table_stride) id = a.table[(size_t)t.trow * a.table_stride + p];
    return id >= 0 && id < a.n_blocks ? id : a.n_blocks;  // out of the map's range: zeros
  };
  bool more = w.load(a);
  int id = more ? block_of(w.t, w.first()) : -1;
  // hand over piece `i`, the one the walk is at (or the end)
  auto publish = [&](uint32_t i) {
    const uint32_t d = i % kPieces;
    const bool y = wait_for_all(bars + 8 * (B::kDE + d), ((i / kPieces) & 1) ^ 1, abort_flag, a);
    if (y && lane == 0) {
      if (more)
        w.describe(a, piece + d);
      else
        piece[d].n = 0;
      // (testing: CTA 0's first piece is never announced, and the waits for it expire)
      if (!(a.withhold && blockIdx.x == 0 && i == 0)) mbar_arrive(bars + 8 * (B::kDF + d));
    }
    return y;
  };
  while (more && ok) {
    if (leads) {
      const uint32_t qb = pieces % nq;
      if (!(ok = publish(pieces))) break;
      ok = wait_for_all(bars + 8 * (B::kQE + qb), ((pieces / nq) & 1) ^ 1, abort_flag, a);
      if (!ok) break;
      const int ns = FORM == kTwo && w.t.ntok > a.list.tpt ? 2 : 1;
      if (lane == 0) {
        const int copies = FORM == kSpread ? 4 : ns;
        mbar_arrive_expect_tx(bars + 8 * (B::kQF + qb), (uint32_t)(copies * C::kHalves * a.box_tokens * a.G * 128));
        for (int s = 0; s < copies; ++s)
          for (int h = 0; h < C::kHalves; ++h)
            tma_load_3d(sm + s * (FORM == kSpread ? 32 * 128 : C::kTileBytes) + h * C::kHalfBytes +
                            qb * kQBufferStep,
                        &maps.q, 64 * h, w.head * a.G, FORM == kSpread ? w.t.tok0 : w.t.tok0 + s * a.list.tpt,
                        bars + 8 * (B::kQF + qb));
      }
    }
    ++pieces;
    const int n = w.n, head = w.head;
    for (int j = 0; j < n; ++j) {
      const int cur = id;
      if (j + 1 < n) {
        id = block_of(w.t, w.first() + j + 1);
      } else {  // the next piece's first
        w.next(a);
        more = w.load(a);
        id = more ? block_of(w.t, w.first()) : -1;
      }
      const uint32_t bytes = (uint32_t)(__popc(__ballot_sync(0xffffffffu, cur >= 0)) * bt * 128);
      ok = wait_for_all(bars + 8 * (B::kEmpty + r.st), r.ph ^ 1, abort_flag, a);
      if (!ok) break;
      // the barrier's one arrival brings the bytes of all boxes; those of the warp beside may land before it
      if (share == 0 && lane == 0) mbar_arrive_expect_tx(bars + 8 * (B::kFull + r.st), bytes);
      __syncwarp();
      if (loads && cur >= 0)
        tma_load_4d(ring + r.st * C::kTileBytes + at, map, 64 * half, 0, head, cur, bars + 8 * (B::kFull + r.st));
      ++tiles;
      r.next();
      r.next();
    }
  }
  if (leads && ok) ok = publish(pieces);
  if (!ok) {  // given up: wait for what was issued before the shared memory goes away
    const long long t0 = clock64();
    auto drain = [&](uint32_t bar, uint32_t par) {
      while (!mbar_try_wait_sleep(bar, par, kSpinNs) && clock64() - t0 <= a.wait_cycles) {
      }
    };
    for (uint32_t t = tiles > (uint32_t)C::kStages ? tiles - C::kStages : 0; t < tiles; ++t) {
      const uint32_t f = 2 * t + kv;
      if (f + C::kStages >= 2 * tiles + kv) drain(bars + 8 * (B::kFull + f % C::kStages), (f / C::kStages) & 1);
    }
    if (leads)
      for (uint32_t q = pieces > nq ? pieces - nq : 0; q < pieces; ++q)
        drain(bars + 8 * (B::kQF + q % nq), (q / nq) & 1);
  }
}

// kTwo: 16-key steps of a key tile whose probabilities are handed over early.
constexpr int kEarly = 6;

// S = Q K^T (128 rows by 128 keys) and O += P V (P in tensor memory), issued by an elected lane of the
// converged warp, so that the operands stay in the uniform datapath: issued by a lane that ran the loop
// alone an MMA took 150 cycles, against the 64 that the tensor cores need for one.  The descriptors' low
// words (address and leading offset) are kept as numbers to which a step's offset is added.
template <int FORM, int DP, bool BF>
struct Mma {
  using C = Cfg<FORM, DP>;
  static constexpr uint32_t kHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // 1 KB atoms, version 1, 128-byte swizzle
  static constexpr uint32_t kIdesc = (1u << 4) | ((128u >> 4) << 24) | (BF ? (1u << 7) | (1u << 10) : 0u);
  static __device__ __forceinline__ uint32_t lo_k(uint32_t addr) { return (addr >> 4) | (1u << 16); }
  static __device__ __forceinline__ uint32_t lo_mn(uint32_t addr) { return (addr >> 4) | ((C::kHalfBytes >> 4) << 16); }
  static __device__ __forceinline__ uint64_t desc(uint32_t lo) { return (uint64_t)lo | ((uint64_t)kHi << 32); }
  static __device__ __forceinline__ void qk(uint32_t tmem_s, uint32_t q, uint32_t k) {
    constexpr uint32_t idesc = kIdesc | ((kAttnKeys >> 3) << 17);
#pragma unroll
    for (int i = 0; i < DP / 16; ++i) {
      const uint32_t off = (uint32_t)((i / 4) * C::kHalfBytes + (i % 4) * 32) >> 4;
      tc_mma_f16(tmem_s, desc(q + off), desc(k + off), idesc, i > 0);
    }
  }
  // steps (of 16 keys) from .. to - 1
  template <int FROM = 0, int TO = kAttnKeys / 16>
  static __device__ __forceinline__ void pv(uint32_t tmem_o, uint32_t tmem_p, uint32_t v, uint32_t accumulate) {
    constexpr uint32_t idesc = kIdesc | ((DP >> 3) << 17) | (1u << 16);  // B contiguous along N
#pragma unroll
    for (int i = FROM; i < TO; ++i)
      tc_mma_f16_ta(tmem_o, tmem_p + 8 * i, desc(v + i * (2048 >> 4)), idesc, i > 0 ? 1u : accumulate);
  }
};

// Trees are small, and often one 128-row tile holds one (of at most 32 nodes with four query heads to a key/value head).
// The two streams of kTwo then take every other key tile of the same rows, each with maxima, sums and outputs of its own,
// which stream 0 adds up at the end of a piece: one's products run during the other's softmax again.  Measured (us, without and
// with): 64 trees of up to 32 nodes behind up to 4000 tokens, heads of 64 90 and 72, of 128 115 and 108 (memory: 86); 8 of up to
// 24 behind up to 8000, heads of 64, capped 47 and 36; one of 24 11.0 both.
template <bool TREE>
__device__ __forceinline__ bool alternates(bool two, int n) {
  return TREE && !two && n > 1;
}

template <int FORM, int DP, bool BF, bool TREE>
__device__ void issue(const AttnArgs &a, const volatile Piece *piece, uint32_t sm, uint32_t bars, uint32_t tmem, volatile int *abort_flag) {
  using C = Cfg<FORM, DP>;
  constexpr int NS = C::NS;
  using B = Bars<C::kStages>;
  using M = Mma<FORM, DP, BF>;
  constexpr uint32_t kStep = C::kTileBytes >> 4;
  constexpr bool SP = FORM == kSpread;
  const uint32_t ring_k = M::lo_k(sm + NS * C::kTileBytes), ring_v = M::lo_mn(sm + NS * C::kTileBytes);
  const uint32_t o0 = tmem + 256;
  constexpr uint32_t nq = kQBuffers<FORM>;
  Ring<C::kStages> r;  // the next stage to be read
  uint32_t pieces = 0, it = 0, p_par = 0, p2_par = 0;
  bool ok = true;
  auto wait = [&](uint32_t bar, uint32_t par) {
    const bool y = wait_for_all(bars + 8 * bar, par, abort_flag, a);
    tc_fence_after();
    return y;
  };
  auto full = [&](const Ring<C::kStages> &x) { return wait(B::kFull + x.st, x.ph); };
  auto release = [&](uint32_t st) { tc_commit(bars + 8 * (B::kEmpty + st)); };
  // the next piece's key tiles and whether its second tile has rows; false at the end or when giving up
  auto next_piece = [&](uint32_t i, int &n, bool &two) {
    const uint32_t d = i % kPieces;
    if (!(ok = wait(B::kDF + d, (i / kPieces) & 1))) return false;
    n = __shfl_sync(0xffffffffu, piece[d].n, 0);
    two = !SP && __shfl_sync(0xffffffffu, piece[d].ntok, 0) > a.list.tpt;
    if (n == 0) return false;
    if (elect_one()) mbar_arrive(bars + 8 * (B::kDE + d));
    __syncwarp();
    return ok = wait(B::kQF + i % nq, (i / nq) & 1);
  };
  int n = 0;
  bool two = false;
  bool more_pieces = next_piece(0, n, two);
  if constexpr (!SP) {
    for (; more_pieces; more_pieces = next_piece(++pieces, n, two)) {
      const uint32_t q0 = M::lo_k(sm);
      if (alternates<TREE>(two, n)) {  // stream t & 1 has the key tile t
        Ring<C::kStages> rk = r, rv = r;
        rv.next();
        auto scores = [&](int t) {
          if (!(ok = full(rk))) return false;
          const uint32_t st = rk.st, u = t & 1;
          rk.next();
          rk.next();
          if (elect_one()) {
            M::qk(tmem + 128 * u, q0, ring_k + st * kStep);
            tc_commit(bars + 8 * (B::kSF + u));
            release(st);
            if (t + 1 == n) tc_commit(bars + 8 * B::kQE);
          }
          __syncwarp();
          return true;
        };
        if (!scores(0) || !scores(1)) break;
        for (int t = 0; t < n; ++t) {
          const uint32_t u = t & 1, par = u ? p2_par : p_par;
          if (!(ok = full(rv))) break;
          const uint32_t v_st = rv.st, v = ring_v + v_st * kStep;
          rv.next();
          rv.next();
          if (!(ok = wait(B::kPE + u, par))) break;
          if (elect_one()) M::template pv<0, kEarly>(o0 + 128 * u, tmem + 128 * u, v, t > 1);
          __syncwarp();
          if (!(ok = wait(B::kPF + u, par))) break;
          if (u)
            p2_par ^= 1;
          else
            p_par ^= 1;
          if (elect_one()) {
            M::template pv<kEarly, kAttnKeys / 16>(o0 + 128 * u, tmem + 128 * u, v, 1);
            if (t + 2 >= n) tc_commit(bars + 8 * (B::kOD + u));
            release(v_st);
          }
          __syncwarp();
          if (t + 2 < n && !scores(t + 2)) break;
        }
        if (!ok) break;
        r = rk;
        continue;
      }
      if (!(ok = full(r))) break;
      uint32_t k_st = r.st;
      r.next();
      if (elect_one()) {
        M::qk(tmem, q0, ring_k + k_st * kStep);
        tc_commit(bars + 8 * B::kSF);
        if (two) {
          M::qk(tmem + 128, q0 + kStep, ring_k + k_st * kStep);
          tc_commit(bars + 8 * (B::kSF + 1));
        }
        release(k_st);
        if (n == 1) tc_commit(bars + 8 * B::kQE);
      }
      __syncwarp();
      for (int j = 0; j < n; ++j) {
        const bool more = j + 1 < n;
        if (!(ok = full(r))) break;
        const uint32_t v_st = r.st, v = ring_v + v_st * kStep;
        r.next();
        if (more) {
          if (!(ok = full(r))) break;
          k_st = r.st;
          r.next();
        }
        // the product with the first keys' probabilities while the softmax is at the last ones'
        if (!(ok = wait(B::kPE, p_par))) break;
        if (elect_one()) M::template pv<0, kEarly>(o0, tmem, v, j > 0);
        __syncwarp();
        if (!(ok = wait(B::kPF, p_par))) break;
        if (elect_one()) {
          M::template pv<kEarly, kAttnKeys / 16>(o0, tmem, v, 1);
          if (more) {
            M::qk(tmem, q0, ring_k + k_st * kStep);
            tc_commit(bars + 8 * B::kSF);
          } else {
            tc_commit(bars + 8 * B::kOD);
          }
          if (!two) {
            release(v_st);
            if (more) release(k_st);
            if (j + 2 == n) tc_commit(bars + 8 * B::kQE);
          }
        }
        __syncwarp();
        if (two) {
          if (!(ok = wait(B::kPE + 1, p2_par))) break;
          if (elect_one()) M::template pv<0, kEarly>(o0 + 128, tmem + 128, v, j > 0);
          __syncwarp();
          if (!(ok = wait(B::kPF + 1, p2_par))) break;
          p2_par ^= 1;
          if (elect_one()) {
            M::template pv<kEarly, kAttnKeys / 16>(o0 + 128, tmem + 128, v, 1);
            if (more) {
              M::qk(tmem + 128, q0 + kStep, ring_k + k_st * kStep);
              tc_commit(bars + 8 * (B::kSF + 1));
            } else {
              tc_commit(bars + 8 * (B::kOD + 1));
            }
            release(v_st);
            if (more) release(k_st);
            if (j + 2 == n) tc_commit(bars + 8 * B::kQE);
          }
          __syncwarp();
        }
        p_par ^= 1;
      }
      if (!ok) break;
    }
  } else {
    // The scores of the next key tile, be it of the next piece, are issued before the wait for this tile's
    // probabilities.
    uint32_t k_st = 0;
    int j = 0;  // key tile of the piece
    auto scores = [&](uint32_t buf, bool last_of_piece, uint32_t qb) {  // of the tile whose keys come next
      if (!(ok = full(r))) return;
      k_st = r.st;
      r.next();
      if (elect_one()) {
        M::qk(tmem + 128 * buf, M::lo_k(sm + qb * kQBufferStep), ring_k + k_st * kStep);
        tc_commit(bars + 8 * (B::kSF + buf));
        release(k_st);
        if (last_of_piece) tc_commit(bars + 8 * (B::kQE + qb));
      }
      __syncwarp();
    };
    if (more_pieces) scores(0, n == 1, 0);
    while (ok && more_pieces) {
      const uint32_t b = it & 1, ob = pieces & 1;  // score buffer, output accumulator
      const Ring<C::kStages> rv = r;                        // this tile's values follow its keys
      r.next();
      const bool first = j == 0, last = j + 1 == n;
      uint32_t of_piece = pieces;
      if (last) {
        more_pieces = next_piece(++of_piece, n, two);
        if (!ok) break;
        j = 0;
      } else {
        ++j;
      }
      if (more_pieces) scores(b ^ 1, j + 1 == n, of_piece % nq);
      if (!ok || !(ok = full(rv))) break;
      if (first && !(ok = wait(B::kOE + ob, ((pieces >> 1) & 1) ^ 1))) break;
      if (!(ok = wait(B::kPF + b, (it >> 1) & 1))) break;
      if (elect_one()) {
        M::pv(o0 + 128 * ob, tmem + 128 * b, ring_v + rv.st * kStep, !first);
        tc_commit(bars + 8 * (B::kOD + b));
        if (last) tc_commit(bars + 8 * (B::kOF + ob));
        release(rv.st);
      }
      __syncwarp();
      pieces = of_piece;
      ++it;
    }
  }
  // nothing of the tensor cores is in flight when tensor memory is freed
  if (elect_one()) tc_commit(bars + 8 * B::kDrain);
  __syncwarp();
  const long long t0 = clock64();
  while (!mbar_try_wait_sleep(bars + 8 * B::kDrain, 0, kSpinNs) && clock64() - t0 <= a.wait_cycles) {
  }
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
// row / G for the rows of a tile: a multiplication by ceil(65536 / G) is exact below 65536 / G.
__device__ __forceinline__ int over_g(const AttnArgs &a, int row) { return (int)((uint32_t)row * a.g_magic >> 16); }
__device__ __forceinline__ bool finite(float v) { return fabsf(v) <= 3.4028234e38f; }

// What happens to the scores besides a positive scale.
enum { kPlain, kCapped, kGeneral };

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}
__device__ __forceinline__ float max_nan(float x, float y, float z) {  // NaN if one of them is
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}
template <int N>
__device__ __forceinline__ float max_of(const float (&x)[N]) {
  float m[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
  for (int i = 4; i + 8 <= N; i += 8)
#pragma unroll
    for (int k = 0; k < 4; ++k) m[k] = max3(m[k], x[i + 2 * k], x[i + 2 * k + 1]);
#pragma unroll
  for (int k = 0; k < 4; ++k) m[k] = fmaxf(m[k], x[N - 4 + k]);  // N = 4 + 8 j + 4
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

template <int N>
__device__ __forceinline__ float largest_magnitude(const float (&x)[N]) {
  float top[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < N; i += 8)
#pragma unroll
    for (int k = 0; k < 4; ++k) top[k] = max3(top[k], fabsf(x[i + 2 * k]), fabsf(x[i + 2 * k + 1]));
  return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
}

// Trees of drafted tokens.  Bits of the keys from .. from + 31, `from` counted from the tree's first node: those that the
// row of these words sees.  Keys before the tree count as `before`, all ones or zeros.
__device__ __forceinline__ uint32_t tree_bits(const uint32_t *seen, int from, uint32_t before) {
  if (from <= -32) return before;
  if (from >= PW_TREE_NODES) return 0;
  const int w = from >> 5;
  return __funnelshift_r(w < 0 ? before : seen[w], w + 1 < kTreeWords ? seen[w + 1] : 0u, from & 31);
}
// Nodes that the row sees among the first n of its tree.  (A node's distance from one of its ancestors is the number of its
// ancestors behind that one, with itself and without that one: nodes ascend along a path.)
__device__ __forceinline__ int tree_count(const uint32_t *seen, int n) {
  int c = 0;
#pragma unroll
  for (int w = 0; w < kTreeWords; ++w) {
    const int m = min(max(n - 32 * w, 0), 32);
    if (m > 0) c += __popc(seen[w] & (m == 32 ? 0xffffffffu : (1u << m) - 1u));
  }
  return c;
}
// The row of a token that is in a tree; rows in none have their tree behind every key.
__device__ __forceinline__ const uint32_t *tree_row(const AttnArgs &a, int tok) { return a.seen + (size_t)tok * kTreeWords; }

// kGeneral: scores of the keys base + i to log2 units with cap and bias.  tanh(y) is a polynomial
// (kTanhPoly, |y| <= 1/2) on the multiply-add pipe; a warp that meets a larger |y| takes 1 - 2 / (1 + e^(2y)) for the tile, with two special-function
// operations for each score.  (tanh itself in one such operation is off by 2^-11: capped scores, and so
// probabilities, would lose as much.)
// Scores are consecutive keys, or (PAIRS) pairs of them eight apart.
template <int N, bool PAIRS = false>
__device__ __forceinline__ void transform(const AttnArgs &a, float (&x)[N], bool valid, float slope, float d0) {
  if (a.softcap > 0.f) {
    const float inv = a.inv_cap, cap2 = a.cap2;
    const float most = largest_magnitude(x) * fabsf(inv);
    if (__any_sync(0xffffffffu, valid && !(most <= 0.5f))) {
      const float t2 = 2.f * kLog2e * inv;
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = cap2 - 2.f * cap2 * rcp(ex2(x[i] * t2) + 1.f);
    } else {
      const uint64_t s = pair(inv, inv);
      constexpr float p1 = (float)kTanhPoly[1], p2 = (float)kTanhPoly[2], p3 = (float)kTanhPoly[3], p4 = (float)kTanhPoly[4];
      const float c1 = p1 * cap2, c2 = p2 * cap2, c3 = p3 * cap2, c4 = p4 * cap2;
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const uint64_t y = mul2(pair(x[i], x[i + 1]), s), u = mul2(y, y);
        uint64_t r = fma2(pair(c4, c4), u, pair(c3, c3));
        r = fma2(r, u, pair(c2, c2));
        r = fma2(r, u, pair(c1, c1));
        r = fma2(r, u, pair(cap2, cap2));
        unpair(mul2(r, y), x[i], x[i + 1]);
      }
    }
  } else {
    const uint64_t s = pair(a.scale2, a.scale2);
#pragma unroll
    for (int i = 0; i < N; i += 2) unpair(mul2(pair(x[i], x[i + 1]), s), x[i], x[i + 1]);
  }
  if (a.slopes) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = fmaf(-slope, fabsf(d0 - (float)(PAIRS ? 8 * (i / 2) + i % 2 : i)), x[i]);
  }
}

// Keys outside [lo, hi) (relative to the first score) get `value`.
template <int N>
__device__ __forceinline__ void mask_out(float (&x)[N], int lo, int hi, float value) {
#pragma unroll
  for (int c = 0; c < N / 32; ++c) {
    const int l = min(max(lo - 32 * c, 0), 32), h = min(max(hi - 32 * c, 0), 32);
    // bits l .. h - 1 (none if h <= l)
    const uint32_t below_h = h == 32 ? 0xffffffffu : (1u << h) - 1u, below_l = l == 32 ? 0xffffffffu : (1u << l) - 1u;
    const uint32_t seen = below_h & ~below_l;
#pragma unroll
    for (int i = 0; i < 32; ++i) x[32 * c + i] = seen >> i & 1u ? x[32 * c + i] : value;
  }
}

template <int N>
struct Words {
  uint32_t w[N];
};
// The same for rows in a tree: also the keys whose bit in `seen` is not set.
template <int N>
__device__ __forceinline__ void mask_tree(float (&x)[N], int lo, int hi, const Words<N / 32> &seen, float value) {
#pragma unroll
  for (int c = 0; c < N / 32; ++c) {
    const int l = min(max(lo - 32 * c, 0), 32), h = min(max(hi - 32 * c, 0), 32);
    const uint32_t below_h = h == 32 ? 0xffffffffu : (1u << h) - 1u, below_l = l == 32 ? 0xffffffffu : (1u << l) - 1u;
    const uint32_t bits = below_h & ~below_l & seen.w[c];
#pragma unroll
    for (int i = 0; i < 32; ++i) x[32 * c + i] = bits >> i & 1u ? x[32 * c + i] : value;
  }
}

// kCapped: N raw scores to exponents cap(x) - m.  With the scale folded into the polynomial's coefficients
// (a.cap_poly) that is six operations a pair, the last of which subtracts m: the maximum of capped scores is the
// cap of the largest, so that m is known before.
__device__ __forceinline__ float cap_one(const AttnArgs &a, float x, bool wide) {
  if (wide) return a.cap2 - 2.f * a.cap2 * rcp(ex2(x * (2.f * kLog2e) * a.inv_cap) + 1.f);
  const float u = x * x;
  return x * fmaf(fmaf(fmaf(fmaf(a.cap_poly[4], u, a.cap_poly[3]), u, a.cap_poly[2]), u, a.cap_poly[1]), u, a.cap_poly[0]);
}
template <int N>
__device__ __forceinline__ void cap_exponents(const AttnArgs &a, float (&x)[N], bool wide, float m) {
  if (wide) {
    const float t2 = 2.f * kLog2e * a.inv_cap, top = a.cap2 - m;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = fmaf(-2.f * a.cap2, rcp(ex2(x[i] * t2) + 1.f), top);
  } else {
    const uint64_t k4 = pair(a.cap_poly[4], a.cap_poly[4]), k3 = pair(a.cap_poly[3], a.cap_poly[3]),
                   k2 = pair(a.cap_poly[2], a.cap_poly[2]), k1 = pair(a.cap_poly[1], a.cap_poly[1]),
                   k0 = pair(a.cap_poly[0], a.cap_poly[0]), neg_m = pair(-m, -m);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const uint64_t y = pair(x[i], x[i + 1]), u = mul2(y, y);
      const uint64_t r = fma2(fma2(fma2(fma2(k4, u, k3), u, k2), u, k1), u, k0);
      unpair(fma2(r, y, neg_m), x[i], x[i + 1]);
    }
  }
}
// The maximum subtracted from the scores is renewed only when it has grown by a factor of 2^8: until then the
// accumulator stays untouched.  fp16 probabilities lie as high as its range allows, in 2^7 .. 2^15 for the largest, so
// that what is 2^-21 of it still has all its bits and 2^-32 of it is not lost: many small ones behind a large one (of
// a small value) make up the result.
template <bool BF>
constexpr float kAbove = BF ? 0.f : 7.f;

// Zeros for the value of a key tile's key `thread`, where it lies outside [klo, khi).
template <class C>
__device__ __forceinline__ void hide_value(uint8_t *v, int thread, int base, int klo, int khi) {
  if (base + thread < klo || base + thread >= khi) {
#pragma unroll
    for (int h = 0; h < C::kHalves; ++h)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *reinterpret_cast<uint4 *>(v + h * C::kHalfBytes + thread * 128 + 16 * i) = make_uint4(0, 0, 0, 0);
  }
  fence_async_smem();
}
// N scores to probabilities, packed, and their sum in pairs: 2^(x scale - m) (kPlain), 2^(x - m) (kGeneral), or 2^x of
// exponents (kCapped).
template <bool BF, int MODE, int N>
__device__ __forceinline__ void exponentials(const float *x, uint64_t scale, uint64_t neg_m, uint32_t (&pk)[N / 2],
                                             uint64_t (&sum)[2]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    float p, q;
    const uint64_t y = pair(x[i], x[i + 1]);
    unpair(MODE == kCapped ? y : MODE == kGeneral ? add2(y, neg_m) : fma2(y, scale, neg_m), p, q);
    p = ex2(p);
    q = ex2(q);
    sum[i / 2 & 1] = add2(sum[i / 2 & 1], pair(p, q));
    pk[i / 2] = pack_pair<BF>(p, q);
  }
}

// How a row's unscaled output v becomes its result: v * inv + w2 * (the row's result over its group's
// shared prefix, where it has one).  m and l are the row's maximum (log2 units) and sum.
struct RowOut {
  float inv, w2, lse2;
  size_t at;  // the row in [n_tokens][Hq] order
};
__device__ __forceinline__ RowOut row_out(const AttnArgs &a, int tok, int head, bool merge, float pl, float m, float l) {
  RowOut r;
  r.at = (size_t)tok * a.Hq + head;
  r.inv = l == 0.f ? 0.f : rcp(l);
  r.lse2 = l == 0.f ? -INFINITY : m + lg2(l);
  r.w2 = 0.f;
  if (merge) {  // pl: the row's log2-sum-exp2 over the prefix
    const float mx = fmaxf(pl, r.lse2), ms = mx == -INFINITY ? 0.f : mx;
    const float e1 = ex2(r.lse2 - ms), e2 = ex2(pl - ms), sum = e1 + e2;
    const float is = sum == 0.f ? 0.f : rcp(sum);
    r.inv *= e1 * is;
    r.w2 = e2 * is;
    r.lse2 = sum == 0.f ? -INFINITY : ms + lg2(sum);
  }
  return r;
}
// The largest magnitude of the first n of N elements (n a multiple of 8, or N = 4), NaN if one of them is.  (Columns
// past head_dim are zeros, or NaN times them: not looked at.)
template <int N>
__device__ __forceinline__ float largest_before(const float *v, int n) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < N; i += 8) {
    float t8 = max_nan(max_nan(fabsf(v[i]), fabsf(v[i + 1]), fabsf(v[i + 2])), fabsf(v[i + 3]), top);
    if constexpr (N % 8 == 0)
      t8 = max_nan(max_nan(fabsf(v[i + 4]), fabsf(v[i + 5]), fabsf(v[i + 6])), fabsf(v[i + 7]), t8);
    if (i < n) top = t8;
  }
  return top;
}
// N consecutive elements from column c of a row; false if one is not finite (by the row's own keys: its result over a
// shared prefix may be).
// `ready`: the row's result over the prefix from column c on, or null to load it here where it counts.  hold: what is
// not finite is not stored.
template <int N, bool BF>
__device__ __forceinline__ bool store_cols(const AttnArgs &a, const RowOut &r, int tok, int head, int c, float (&v)[N],
                                           const float4 *ready = nullptr, bool hold = false) {
  static_assert(N % 4 == 0, "stores of 8 or 16 bytes");
  if (c >= a.D) return true;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] *= r.inv;
  const bool fin = finite(largest_before<N>(v, a.D - c));
  if (hold && !fin) return false;
  if (r.w2 != 0.f) {
    const float *po = a.prefix_o + r.at * a.D + c;
#pragma unroll
    for (int i = 0; i < N; i += 4)
      if (c + i < a.D) {
        const float4 x = ready ? ready[i / 4] : *reinterpret_cast<const float4 *>(po + i);
        v[i] = fmaf(r.w2, x.x, v[i]);
        v[i + 1] = fmaf(r.w2, x.y, v[i + 1]);
        v[i + 2] = fmaf(r.w2, x.z, v[i + 2]);
        v[i + 3] = fmaf(r.w2, x.w, v[i + 3]);
      }
  }
  if (a.to_prefix) {
    float *d = a.prefix_o + r.at * a.D + c;
#pragma unroll
    for (int i = 0; i < N; i += 4)
      if (c + i < a.D) *reinterpret_cast<float4 *>(d + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else {
    uint16_t *d = a.o + tok * a.o_token + head * a.o_head + c;
    if constexpr (N % 8 == 0) {
#pragma unroll
      for (int i = 0; i < N; i += 8)
        if (c + i < a.D)
          *reinterpret_cast<uint4 *>(d + i) =
              make_uint4(pack_pair<BF>(v[i], v[i + 1]), pack_pair<BF>(v[i + 2], v[i + 3]),
                         pack_pair<BF>(v[i + 4], v[i + 5]), pack_pair<BF>(v[i + 6], v[i + 7]));
    } else {
      *reinterpret_cast<uint2 *>(d) = make_uint2(pack_pair<BF>(v[0], v[1]), pack_pair<BF>(v[2], v[3]));
    }
  }
  return fin;
}
__device__ __forceinline__ void store_lse(const AttnArgs &a, const RowOut &r) {
  if (a.to_prefix)
    a.prefix_lse[r.at] = r.lse2;
  else if (a.lse)
    a.lse[r.at] = r.lse2 * kLn2;
}

// One row (token t, query head h) over the keys [lo, hi) of its table row, by one warp, for rows that the
// tensor cores cannot do (see redo_row): o = sum_j 2^{x_j log2 e - lse2} v_j, whose weights add up to one (large values
// keep within fp32 however many keys they meet).  Eight lanes share a key, lane l its elements 8 (l % 8) .. + 7 and 64 + 8
// (l % 8) .. + 7, and 4 KEYS keys are under way at a time, KEYS to each quarter of the warp.  Only visible keys and
// values count.  acc is the output in all lanes (zeros for a row without keys).
template <bool BF, int KEYS, bool TREE>
__device__ void row_attention(const AttnArgs &a, int t, int h, int lo, int hi, int trow, int pos, int tree0, float lse2,
                              float (&acc)[16]) {
  const int lane = threadIdx.x & 31, sub = lane >> 3, d = 8 * (lane & 7);
  const int hk = h / a.G, mask = (1 << a.log_bt) - 1;
  auto spread = [](const uint4 &w, float *x) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 y = unpack2<BF>(u[i]);
      x[2 * i] = y.x;
      x[2 * i + 1] = y.y;
    }
  };
  // Loads are made from the cache's or the table's beginning where there is nothing to load, and replaced by zeros: no
  // branch keeps one from being issued behind another.
  const bool has[2] = {d < a.D, d + 64 < a.D};
  const int col[2] = {has[0] ? d : 0, has[1] ? d + 64 : 0};
  auto zeros_but = [](bool keep, uint4 w) { return keep ? w : make_uint4(0, 0, 0, 0); };
  float q[16];
#pragma unroll
  for (int half = 0; half < 2; ++half)
    spread(zeros_but(has[half], *reinterpret_cast<const uint4 *>(a.q + t * a.q_token + h * a.q_head + col[half])), q + 8 * half);
  const int *table = a.table + (trow >= 0 ? (size_t)trow * a.table_stride : 0);
  const float slope = a.slopes ? a.slopes[h] : 0.f;
  // what the row sees of its tree's nodes; all in all
  auto node_seen = [&](int j) { return tree_row(a, t)[(j - tree0) >> 5] >> (j - tree0 & 31) & 1u; };
  const int nodes = TREE && hi > tree0 && a.slopes ? tree_count(tree_row(a, t), PW_TREE_NODES) : 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
#pragma unroll 1
  for (int j0 = lo; j0 < hi; j0 += 4 * KEYS) {
    uint4 k[KEYS][2], v[KEYS][2];
    int id[KEYS];
    bool there[KEYS];
#pragma unroll
    for (int u = 0; u < KEYS; ++u) {
      const int j = j0 + 4 * u + sub, page = j >> a.log_bt;
      const bool in = j < hi && trow >= 0 && page < a.table_stride && !(TREE && j >= tree0 && !node_seen(j));
      id[u] = table[in ? page : 0];
      there[u] = in && id[u] >= 0 && id[u] < a.n_blocks;
    }
#pragma unroll
    for (int u = 0; u < KEYS; ++u) {
      const int64_t at = there[u] ? id[u] * a.block_stride + ((j0 + 4 * u + sub) & mask) * a.token_stride + hk * a.head_stride : 0;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        k[u][half] = *reinterpret_cast<const uint4 *>(a.kc + at + col[half]);
        v[u][half] = *reinterpret_cast<const uint4 *>(a.vc + at + col[half]);
      }
    }
#pragma unroll
    for (int u = 0; u < KEYS; ++u) {
      const int j = j0 + 4 * u + sub;
      float x[16], y = 0.f;
#pragma unroll
      for (int half = 0; half < 2; ++half) spread(zeros_but(there[u] && has[half], k[u][half]), x + 8 * half);
#pragma unroll
      for (int i = 0; i < 16; ++i) y = fmaf(q[i], x[i], y);
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
      y *= a.scale;
      if (a.softcap > 0.f) y = a.softcap * tanhf(y / a.softcap);
      float away = fabsf((float)(pos - j));
      bool seen = j < hi;
      if (TREE && seen && j >= tree0) {
        seen = node_seen(j);
        if (a.slopes) away = (float)(nodes - tree_count(tree_row(a, t), j - tree0 + 1));
      }
      if (a.slopes) y -= slope * away;
      const float w = seen ? ex2(fmaf(y, kLog2e, -lse2)) : 0.f;
#pragma unroll
      for (int half = 0; half < 2; ++half) spread(zeros_but(there[u] && has[half], v[u][half]), x + 8 * half);
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[i] = fmaf(w, x[i], acc[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {  // the quarters' together
    acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], 8);
    acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], 16);
  }
}

// A row whose sum is finite but whose output is not: a value is infinite or NaN, possibly one that the row
// does not see (0 times it in the product with v).  Again, from the row's visible keys alone, by the warp.
// merge: over the shared prefix too.  lse2: the row's log2-sum-exp2, which is right.  Columns 4 g .. 4 g + 3 are written for the bits g of `groups`.
template <bool BF, int KEYS, bool TREE>
static __device__ PW_RARE void redo_row(const AttnArgs &a, int tok, int head, int klo, int khi, int trow, bool merge,
                                        float lse2, uint32_t groups = ~0u) {
  const int lane = threadIdx.x & 31;
  const RowBound b = a.bounds[tok];
  float acc[16];
  row_attention<BF, KEYS, TREE>(a, tok, head, merge ? b.lo : max(b.lo, klo), merge ? b.hi : min(b.hi, khi), trow, b.pos,
                                b.trow, lse2, acc);
  if (lane >= 8) return;
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    const int c = i / 8 * 64 + 8 * lane + i % 8;
    if (c >= a.D || !(groups >> (c / 4) & 1u)) continue;
    if (a.to_prefix)
      *reinterpret_cast<float4 *>(a.prefix_o + ((size_t)tok * a.Hq + head) * a.D + c) =
          make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
    else
      *reinterpret_cast<uint2 *>(a.o + tok * a.o_token + head * a.o_head + c) =
          make_uint2(pack_pair<BF>(acc[i], acc[i + 1]), pack_pair<BF>(acc[i + 2], acc[i + 3]));
  }
}

// Such a row takes as long as its keys are many, and a pipeline of bounded waits cannot stop for it: within
// attn_kernel it is marked, once its output is written, and computed again when the CTA's pieces are done.  Until then
// the first four bytes of the output hold its lse2 (results over a shared prefix have theirs beside them).
__device__ __forceinline__ float *marked_lse(const AttnArgs &a, int tok, int head) {
  return a.to_prefix ? a.prefix_lse + (size_t)tok * a.Hq + head
                     : reinterpret_cast<float *>(a.o + tok * a.o_token + head * a.o_head);
}
static __device__ __forceinline__ void mark_row(const AttnArgs &a, int tok, int head, float lse2, volatile int *marked) {
  const size_t at = (size_t)tok * a.Hq + head;
  *marked_lse(a, tok, head) = lse2;
  __threadfence();  // another CTA that has a piece of the tile may be the one that takes the row
  atomicOr(a.marks + (at >> 5), 1u << (at & 31));
  *marked = 1;
}
// By the first `warps` of a CTA whose pieces are done, rows dealt out among them.  A CTA looks at the rows of all its pieces;
// the one that finished a tile has a piece of it, and whoever clears a row's mark computes it.
template <bool BF, int KEYS, bool TREE>
static __device__ PW_RARE void redo_marked(const AttnArgs &a, int warps) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Walk<TREE> w(a, true);
  while (w.load(a)) {
    const AttnTile t = w.t;
    const bool merge = t.merge && !a.to_prefix;
    const int rows = t.ntok * a.G;
    for (int r0 = 0; r0 < rows; r0 += 32 * warps) {
      const int r = r0 + lane * warps + warp, tok = t.tok0 + r / a.G, head = w.head * a.G + r % a.G;
      bool mine = false;
      float lse2 = 0.f;
      if (r < rows) {
        const size_t at = (size_t)tok * a.Hq + head;
        const uint32_t bit = 1u << (at & 31);
        mine = (__ldcg(a.marks + (at >> 5)) & bit) && (atomicAnd(a.marks + (at >> 5), ~bit) & bit);
        if (mine) {
          __threadfence();
          lse2 = __ldcg(marked_lse(a, tok, head));
        }
      }
      unsigned flagged = __ballot_sync(0xffffffffu, mine);
      __syncwarp();
      while (flagged) {
        const int src = __ffs(flagged) - 1;
        flagged &= flagged - 1;
        redo_row<BF, KEYS, TREE>(a, __shfl_sync(0xffffffffu, tok, src), __shfl_sync(0xffffffffu, head, src), t.klo, t.khi, t.trow,
                           merge, __shfl_sync(0xffffffffu, lse2, src));
      }
    }
    w.next(a);
  }
}

// Bit i of sixteen as bit 2 i.
__device__ __forceinline__ uint32_t every_other(uint32_t x) {
  x = (x | x << 8) & 0x00ff00ffu;
  x = (x | x << 4) & 0x0f0f0f0fu;
  x = (x | x << 2) & 0x33333333u;
  return (x | x << 1) & 0x55555555u;
}

// Four warps that finish a row tile together.
template <int STAGES>
struct Group {
  uint32_t bars;
  int s;           // stream
  uint32_t joins;  // meetings so far
  volatile int *abort_flag;
  // all four meet (bounded, as every wait)
  __device__ __forceinline__ bool join(const AttnArgs &a) {
    const uint32_t bar = bars + 8 * (Bars<STAGES>::kJoin + s);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
    return wait_for_all(bar, joins++ & 1, abort_flag, a);
  }
  // A split tile's piece has been written: true for the last of its CTAs to come here, which may read them all.
  __device__ __forceinline__ bool last_to_arrive(const AttnArgs &a, int c0, int c1, int thread,
                                                 volatile int *last_flag, bool &ok) {
    if (!(ok = join(a))) return false;
    if (thread == 0) {
      int *cnt = a.counters + 2 * c0 + s;
      // releases the group's writes, which the meeting has made visible to this thread, and acquires the others'
      int before;
      asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;\n" : "=r"(before) : "l"(cnt) : "memory");
      const int last = before == c1 - c0;
      if (last) *cnt = 0;
      last_flag[s] = last;
    }
    if (!(ok = join(a))) return false;
    return last_flag[s] != 0;
  }
};

// kTwo: the softmax warps of two streams, which write their rows' results, too.
template <int DP, bool BF, int MODE, bool TREE>
__device__ void soften(const AttnArgs &a, const volatile Piece *piece, uint8_t *smp, uint32_t bars, uint32_t tmem,
                       volatile int *abort_flag, volatile int *last_flag, volatile int *marked, volatile float2 *other) {
  using C = Cfg<kTwo, DP>;
  using B = Bars<C::kStages>;
  constexpr int NS = C::NS;
  constexpr int NC = 128;  // scores of a key tile that a thread takes
  // Of which this many at a time.  Capped and biased scores go through tensor memory once more, in two halves:
  // all 128 at a time their arithmetic spilled registers and filled the instruction cache (chunks-docs-cap
  // 70.7 us, in halves 67.9); plain scores lose more by the second read (prompt-8192 413 us, in halves 444).
  constexpr int CH = MODE != kPlain ? 64 : 128;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int s = warp >> 2, quarter = warp & 3, thread = 32 * quarter + lane;
  const int row = thread;
  const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
  uint32_t it = 0;        // key tiles of this stream so far
  Ring<C::kStages> rv;    // the current tile's V
  rv.next();
  uint32_t o_done = 0;    // pieces of this stream so far
  uint32_t o1_done = 0;   // (TREE) of stream 1
  uint32_t merges = 0;
  Group<C::kStages> group{bars, s, 0, abort_flag};
  auto merge_meet = [&] {  // all eight warps, bounded as every wait
    __syncwarp();
    if (lane == 0) mbar_arrive(bars + 8 * B::kMerge);
    return wait_for_all(bars + 8 * B::kMerge, merges++ & 1, abort_flag, a);
  };
  constexpr int kPart = DP * 128;
  auto slot_of = [&](int c, int c0) { return part_slot(c, c0, NS, s); };
  const float sl2 = a.scale2;
  const int row_t = over_g(a, row), row_h = row - row_t * a.G;  // the row's token in its tile, and head
  // the row in a tile of ntok tokens: a stream of its own, or (TREE) the same in both
  auto tok_of = [&](int ntok) { return (TREE && ntok <= a.list.tpt ? 0 : s * a.list.tpt) + row_t; };
  uint32_t pieces = 0;
  bool ok = wait_for_all(bars + 8 * B::kDF, 0, abort_flag, a);
  const RowBound nobody{0, 0, TREE ? INT_MAX : -1, 0};
  RowBound rb = nobody, rb_ahead = nobody;
  // the row's keys in a piece, fetched while the piece before is in work
  auto bound_of = [&](const volatile Piece &x) {
    if (x.n == 0 || !x.fresh) return rb;
    const int nt = x.ntok, r = tok_of(nt);
    return r < min(nt, (s + 1) * a.list.tpt) ? a.bounds[x.tok0 + r] : nobody;
  };
  if (ok) rb_ahead = bound_of(piece[0]);
  for (; ok; ++pieces) {
    const volatile Piece &w = piece[pieces % kPieces];
    const int n = w.n, first = w.first;
    if (n == 0) break;
    const int row_tok = tok_of(w.ntok);
    const bool alt = alternates<TREE>(w.ntok > a.list.tpt, n);
    const int ntok = alt ? w.ntok : min(a.list.tpt, w.ntok - s * a.list.tpt), nrows = ntok * a.G;
    if (TREE && (alt || w.ntok > a.list.tpt)) ++o1_done;
    rb = rb_ahead;
    const uint32_t dn = (pieces + 1) % kPieces;
    if (ntok <= 0) {
      for (int i = 0; i < 2 * n; ++i) rv.next();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 8 * (B::kDE + pieces % kPieces));
      if (!(ok = wait_for_all(bars + 8 * (B::kDF + dn), ((pieces + 1) / kPieces) & 1, abort_flag, a))) break;
      rb_ahead = bound_of(piece[dn]);
      continue;
    }
    const bool valid = row < nrows;
    const int klo = w.klo, khi = w.khi, lo = max(rb.lo, klo), hi = min(rb.hi, khi);
    const bool active = 32 * quarter < nrows;
    const float slope = MODE == kGeneral && a.slopes && valid ? a.slopes[w.head * a.G + row_h] * kLog2e : 0.f;
    const uint32_t tmem_o = tmem + 256 + 128 * (uint32_t)s + lanes, ts = tmem + 128 * (uint32_t)s + lanes;
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < n; ++j, rv.next(), rv.next()) {
      if (alt && (j & 1) != s) continue;
      const int base = (first + j) * kAttnKeys;
      if (!(ok = wait_for_all(bars + 8 * (B::kSF + s), it++ & 1, abort_flag, a))) break;
      tc_fence_after();
      if ((s == 0 || alt) && (base < klo || base + kAttnKeys > khi)) {
        // keys outside the segment (unwritten cache, blocks not loaded): their values must be zeros, since 0
        // times what the memory holds may be NaN
        if (!(ok = wait_for_all(bars + 8 * (B::kFull + rv.st), rv.ph, abort_flag, a))) break;
        hide_value<C>(smp + (NS + rv.st) * C::kTileBytes, thread, base, klo, khi);
        __syncwarp();  // a warp without rows arrives below by one lane for all of them
      }
      if (active) {
        const int l0 = lo - base, h0 = hi - base;
        // (a row in a tree sees all keys up to the tree, and few of the tree's)
        const int t0 = TREE ? rb.trow - base : 0;
        const bool edge = __any_sync(0xffffffffu, valid && (l0 > 0 || (TREE ? min(h0, t0) : h0) < NC));
        uint32_t nodes[NC / 32];
        if (TREE && edge) {
          const uint32_t *of_row = tree_row(a, w.tok0 + row_tok);
#pragma unroll
          for (int c = 0; c < NC / 32; ++c) nodes[c] = tree_bits(of_row, 32 * c - t0, 0xffffffffu);
        }
        // (without a run-time index, which would put them in memory)
        auto nodes_from = [&](int c) {
          Words<CH / 32> r;
#pragma unroll
          for (int i = 0; i < CH / 32; ++i) r.w[i] = CH < NC && c ? nodes[(NC - CH) / 32 + i] : nodes[i];
          return r;
        };
        auto hide = [&](float (&y)[CH], int c, float value) {
          if constexpr (TREE)
            mask_tree<CH>(y, l0 - c, h0 - c, nodes_from(c), value);
          else
            mask_out<CH>(y, l0 - c, h0 - c, value);
        };
        float x[CH], mx = -INFINITY;
        auto load = [&](int c) {
#pragma unroll
          for (int i = 0; i < CH; i += 32) tmem_ld32(ts + c + i, reinterpret_cast<uint32_t *>(x) + i);
          tmem_wait_ld();
        };
        float top = 0.f;
#pragma unroll 1
        for (int c = 0; c < NC; c += CH) {
          load(c);
          // (hidden scores, which may come from unwritten memory, have no say in how the tile's are capped)
          if (MODE != kPlain && edge && a.softcap > 0.f) hide(x, c, 0.f);
          if (MODE == kCapped) top = fmaxf(top, largest_magnitude(x));
          if (MODE == kGeneral) transform<CH>(a, x, valid, slope, (float)(rb.pos - base - c));
          if (TREE && MODE == kGeneral && edge && a.slopes && t0 < c + CH) {
            // distances along the tree instead of those between the places in the cache
            const uint32_t *of_row = tree_row(a, w.tok0 + row_tok);
            int behind = tree_count(of_row, PW_TREE_NODES) - tree_count(of_row, c - t0);
            const float d0 = (float)(rb.pos - base - c);
            const Words<CH / 32> mine = nodes_from(c);
#pragma unroll
            for (int i = 0; i < CH; ++i) {
              if (c + i < t0) continue;
              behind -= mine.w[i / 32] >> (i & 31) & 1u;
              x[i] = fmaf(slope, fabsf(d0 - (float)i) - (float)behind, x[i]);
            }
          }
          if (edge) hide(x, c, -INFINITY);
          mx = fmaxf(mx, max_of<CH>(x));
          if (MODE == kGeneral && CH < NC) {
#pragma unroll
            for (int i = 0; i < CH; i += 32) tmem_st32(ts + c + i, reinterpret_cast<uint32_t *>(x) + i);
          }
        }
        if (MODE == kGeneral && CH < NC) tmem_wait_st();
        const bool wide = MODE == kCapped && __any_sync(0xffffffffu, valid && !(top * a.inv_cap <= 0.5f));
        if (MODE == kPlain) mx *= a.scale2;
        if (MODE == kCapped) mx = mx == -INFINITY ? mx : cap_one(a, mx, wide);
        if (!valid) mx = INFINITY;  // rows of nobody: no rescaling on their account
        mx -= kAbove<BF>;
        if (j == (alt ? s : 0)) {
          m = mx;
        } else if (__any_sync(0xffffffffu, mx > m + 8.f)) {
          // (these scores were issued behind the product before, which is therefore done)
          const float mn = fmaxf(m, mx), f = mn == -INFINITY ? 1.f : ex2(m - mn);
          m = mn;
          l *= f;
#pragma unroll 1
          for (int c = 0; c < DP / 32; ++c) {
            float o[32];
            tmem_ld32(tmem_o + 32 * c, reinterpret_cast<uint32_t *>(o));
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= f;
            tmem_st32(tmem_o + 32 * c, reinterpret_cast<uint32_t *>(o));
          }
        }
        const float ms = m == -INFINITY ? 0.f : m;
        const uint64_t scale = pair(sl2, sl2), neg_m = pair(-ms, -ms);
        uint64_t sum[2] = {0, 0};
#pragma unroll 1
        for (int c0 = 0; c0 < NC; c0 += CH) {
          if (CH < NC) load(c0);  // (kGeneral: as transformed)
          if (MODE == kCapped) {
            cap_exponents<CH>(a, x, wide, ms);
            if (edge) hide(x, c0, -INFINITY);
          }
#pragma unroll
          for (int c = 0; c < CH / 32; ++c) {
            uint32_t pk[16];
            exponentials<BF, MODE, 32>(x + 32 * c, scale, neg_m, pk, sum);
            tmem_st16(ts + c0 / 2 + 16 * c, pk);
            if (c0 / 16 + 2 * (c + 1) == kEarly) {
              tmem_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(bars + 8 * (B::kPE + s));
            }
          }
        }
        float s0, s1;
        unpair(add2(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
        tmem_wait_st();
      } else if (lane == 0) {
        mbar_arrive(bars + 8 * (B::kPE + s));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 8 * (B::kPF + s));
    }
    if (!ok) break;
    // the next piece has been handed over: its first scores may be on their way
    if (!(ok = wait_for_all(bars + 8 * (B::kDF + dn), ((pieces + 1) / kPieces) & 1, abort_flag, a))) break;
    rb_ahead = bound_of(piece[dn]);
    // the piece's last product
    if (!(ok = wait_for_all(bars + 8 * (B::kOD + s), o_done++ & 1, abort_flag, a))) break;
    tc_fence_after();
    if (TREE && alt) {
      if (s == 1 && valid) {
        other[row].x = m;
        other[row].y = l;
      }
      if (!(ok = merge_meet())) break;
      if (s == 0) {
        if (!(ok = wait_for_all(bars + 8 * (B::kOD + 1), (o1_done - 1) & 1, abort_flag, a))) break;
        tc_fence_after();
        if (active) {
          const float m1 = other[row].x, l1 = other[row].y, mm = fmaxf(m, m1), ms = mm == -INFINITY ? 0.f : mm;
          const float f0 = ex2(m - ms), f1 = ex2(m1 - ms);
          m = mm;
          l = fmaf(l1, f1, l * f0);
#pragma unroll 1
          for (int c = 0; c < DP / 32; ++c) {
            float o[32], o1[32];
            __syncwarp();
            tmem_ld32(tmem_o + 32 * c, reinterpret_cast<uint32_t *>(o));
            tmem_ld32(tmem_o + 128 + 32 * c, reinterpret_cast<uint32_t *>(o1));
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = fmaf(o1[i], f1, o[i] * f0);
            tmem_st32(tmem_o + 32 * c, reinterpret_cast<uint32_t *>(o));
          }
          tmem_wait_st();
        }
        tc_fence_before();
      }
      if (!(ok = merge_meet())) break;  // stream 1's outputs have been read
      if (s == 1) {
        if (lane == 0) mbar_arrive(bars + 8 * (B::kDE + pieces % kPieces));
        continue;
      }
    }
    if (a.after_prefix) pdl_wait();  // (returns at once but the first time)
    auto from_tmem = [&](int c, float (&v)[32]) {
      __syncwarp();  // a load of the whole warp: lanes without a row come from other branches
      tmem_ld32(tmem_o + 32 * c, reinterpret_cast<uint32_t *>(v));
      tmem_wait_ld();
    };
    const bool merge = w.merge;
    const int c0 = w.c0, c1 = w.c1;
    bool out = true;  // this CTA writes the result
    if (c0 != c1) {
      // a piece of a tile: its partial result goes to this CTA's slot, and whoever arrives last adds all up, in
      // tensor memory again (or attn_join_kernel does)
      const size_t my = slot_of(blockIdx.x, c0);
      if (active) {
        uint32_t odd = 0;
#pragma unroll 1
        for (int c = 0; c < DP / 32; ++c) {
          float v[32];
          from_tmem(c, v);
          if (a.join) {
            uint32_t o = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) o |= finite(largest_before<4>(v + 4 * i, 4)) ? 0u : 1u << i;
            odd |= o << (8 * c);
          }
          if (valid) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              __stcg(reinterpret_cast<float4 *>(a.part_o + my * kPart + ((8 * c + i / 4) * 128 + row) * 4),
                     make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]));
          }
        }
        if (valid) {
          __stcg(a.part_ml + my * 128 + row, make_float2(m, l));
          if (a.join) a.part_odd[my * 128 + row] = odd;
        }
      }
      out = !a.join && group.last_to_arrive(a, c0, c1, thread, last_flag, ok);
      if (!ok) break;
      if (out && active) {
        m = -INFINITY;
        l = 0.f;
        if (valid)
          for (int p = c0; p <= c1; ++p) m = fmaxf(m, __ldcg(a.part_ml + slot_of(p, c0) * 128 + row).x);
        const float ms = m == -INFINITY ? 0.f : m;
        if (valid)
          for (int p = c0; p <= c1; ++p) {
            const float2 y = __ldcg(a.part_ml + slot_of(p, c0) * 128 + row);
            l = fmaf(ex2(y.x - ms), y.y, l);
          }
#pragma unroll 1
        for (int c = 0; c < DP / 32; ++c) {
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0.f;
          if (valid)
#pragma unroll 1
            for (int p = c0; p <= c1; ++p) {
              const size_t at = slot_of(p, c0);
              const float f = ex2(__ldcg(a.part_ml + at * 128 + row).x - ms);
              const float4 *src = reinterpret_cast<const float4 *>(a.part_o + at * kPart) + 8 * c * 128 + row;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float4 y = __ldcg(src + i * 128);
                v[4 * i] = fmaf(f, y.x, v[4 * i]);
                v[4 * i + 1] = fmaf(f, y.y, v[4 * i + 1]);
                v[4 * i + 2] = fmaf(f, y.z, v[4 * i + 2]);
                v[4 * i + 3] = fmaf(f, y.w, v[4 * i + 3]);
              }
            }
          __syncwarp();
          tmem_st32(tmem_o + 32 * c, reinterpret_cast<uint32_t *>(v));
        }
        tmem_wait_st();
      }
    }
    if (out && active) {  // a thread's row, 32 columns at a time
      const int tok = w.tok0 + row_tok, head = w.head * a.G + row_h;
      RowOut ro{};
      if (valid) ro = row_out(a, tok, head, merge, merge ? a.prefix_lse[(size_t)tok * a.Hq + head] : 0.f, m, l);
      bool fin = true;
#pragma unroll 1
      for (int c = 0; c < DP / 32; ++c) {
        float v[32];
        from_tmem(c, v);
        if (valid) fin = store_cols<32, BF>(a, ro, tok, head, 32 * c, v) && fin;
      }
      if (valid) store_lse(a, ro);
      if (valid && !fin && finite(l)) mark_row(a, tok, head, ro.lse2, marked);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(bars + 8 * (B::kDE + pieces % kPieces));
  }
}

// kSpread: the softmax warps.  A quarter's 16 rows by its 32 keys lie over its warp as the tensor cores' fragments:
// thread t holds eight scores of row t / 4 and, where a tile has more than eight rows, eight of the row eight
// below.  (A lane a row, half of a warp's lanes or more would have nothing to do.)  Four threads share a row: its
// maximum is made common to them when it is renewed, which each of them may ask for, and its sum at a piece's end.
template <int DP, bool BF, int MODE, bool TREE>
__device__ void soften_few(const AttnArgs &a, const volatile Piece *piece, uint8_t *smp, uint32_t bars, uint32_t tmem,
                           volatile int *abort_flag) {
  using C = Cfg<kSpread, DP>;
  using B = Bars<C::kStages>;
  const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3, thread = 32 * quarter + lane;
  const int col0 = 32 * quarter + 2 * (lane & 3);  // this thread's keys: col0 + 8 k and the one after, k = 0 .. 3
  const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
  uint32_t it = 0, pieces = 0;  // key tiles, pieces so far
  Ring<C::kStages> rv;          // the current tile's V
  rv.next();
  // P V of key tile t is complete.  Even and odd tiles have a barrier each: when this is asked the tile before on
  // the same barrier is known to be complete (the scores of tile t or t + 1 were issued behind it) and the one after
  // waits for this thread, so the parity cannot be mistaken.
  auto product_done = [&](uint32_t t) {
    return wait_for_all(bars + 8 * (B::kOD + (t & 1)), (t >> 1) & 1, abort_flag, a);
  };
  int row_t[2], row_h[2];  // the rows' tokens in their tile, and heads
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int row = lane / 4 + 8 * h;
    row_t[h] = over_g(a, row);
    row_h[h] = row - row_t[h] * a.G;
  }
  bool ok = wait_for_all(bars + 8 * B::kDF, 0, abort_flag, a);
  const RowBound nobody{0, 0, TREE ? INT_MAX : -1, 0};
  RowBound rb[2] = {nobody, nobody}, ahead[2] = {nobody, nobody};
  // the rows' keys in a piece, fetched while the piece before is in work
  auto fetch = [&](const volatile Piece &x) {
    const bool fresh = x.n != 0 && x.fresh;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      ahead[h] = rb[h];
      if (fresh) ahead[h] = row_t[h] < x.ntok ? a.bounds[x.tok0 + row_t[h]] : nobody;
    }
  };
  if (ok) fetch(piece[0]);
  for (; ok; ++pieces) {
    const volatile Piece &w = piece[pieces % kPieces];
    const int n = w.n, first = w.first;
    if (n == 0) break;
    const int ntok = w.ntok, klo = w.klo, khi = w.khi;
    const bool both = ntok * a.G > 8;
    bool valid[2];
    int lo[2], hi[2];
    float slope[2], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      rb[h] = ahead[h];
      valid[h] = row_t[h] < ntok;
      lo[h] = max(rb[h].lo, klo);
      hi[h] = min(rb[h].hi, khi);
      slope[h] = MODE == kGeneral && a.slopes && valid[h] ? a.slopes[w.head * a.G + row_h[h]] * kLog2e : 0.f;
    }
    const uint32_t tmem_o = tmem + 256 + 128 * (pieces & 1) + lanes;
    // The scores s of a key tile, of the first eight rows or of all sixteen.
    auto tile = [&](auto rows, const uint32_t (&sc)[16], uint32_t ts, int base, bool begins) {
      constexpr int H = decltype(rows)::value;
      float x[H][8], mx[H];
      uint32_t seen[H];  // bits 8 k + e: this thread's keys that the row sees
      bool edge = false, wide = false;
#pragma unroll
      for (int h = 0; h < H; ++h) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[h][i] = __uint_as_float(sc[4 * (i / 2) + 2 * h + i % 2]);
        const int l0 = lo[h] - base - 32 * quarter, h0 = hi[h] - base - 32 * quarter;
        const int from = min(max(l0, 0), 32), to = min(max(h0, 0), 32);
        const uint32_t below_to = to == 32 ? 0xffffffffu : (1u << to) - 1u;
        const uint32_t below_from = from == 32 ? 0xffffffffu : (1u << from) - 1u;
        const int t0 = TREE ? rb[h].trow - base - 32 * quarter : 0;
        uint32_t all = below_to & ~below_from;
        if (TREE && t0 < 32) all &= tree_bits(tree_row(a, w.tok0 + row_t[h]), -t0, 0xffffffffu);
        seen[h] = all >> (2 * (lane & 3));
        edge = edge || (valid[h] && (l0 > 0 || (TREE ? min(h0, t0) : h0) < 32));
      }
      edge = __any_sync(0xffffffffu, edge);
      auto hide = [&](int h, float value) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[h][i] = seen[h] >> (8 * (i / 2) + i % 2) & 1u ? x[h][i] : value;
      };
#pragma unroll
      for (int h = 0; h < H; ++h) {
        // (hidden scores, which may come from unwritten memory, have no say in how the tile's are capped)
        if (MODE != kPlain && edge && a.softcap > 0.f) hide(h, 0.f);
        if (MODE == kCapped) wide = wide || (valid[h] && !(largest_magnitude(x[h]) * a.inv_cap <= 0.5f));
        if (MODE == kGeneral) transform<8, true>(a, x[h], valid[h], slope[h], (float)(rb[h].pos - base - col0));
        if (TREE && MODE == kGeneral && a.slopes && rb[h].trow < base + 32 * (quarter + 1)) {
          // distances along the tree instead of those between the places in the cache
          const uint32_t *of_row = tree_row(a, w.tok0 + row_t[h]);
          const int from = base + 32 * quarter - rb[h].trow;
          const int behind = tree_count(of_row, PW_TREE_NODES) - tree_count(of_row, from);
          const uint32_t nodes = tree_bits(of_row, from, 0);
          const float d0 = (float)(rb[h].pos - base - col0);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int b = 8 * (i / 2) + i % 2, key = 2 * (lane & 3) + b;
            if (key + from >= 0)
              x[h][i] = fmaf(slope[h], fabsf(d0 - (float)b) - (float)(behind - __popc(nodes & (2u << key) - 1u)), x[h][i]);
          }
        }
        if (edge) hide(h, -INFINITY);
        mx[h] = max_of(x[h]);
      }
      if (MODE == kCapped) wide = __any_sync(0xffffffffu, wide);
      bool grown = false;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        if (MODE == kPlain) mx[h] *= a.scale2;
        if (MODE == kCapped) mx[h] = mx[h] == -INFINITY ? mx[h] : cap_one(a, mx[h], wide);
        mx[h] -= kAbove<BF>;
        if (!valid[h]) mx[h] = -INFINITY;  // rows of nobody: no rescaling on their account
        grown = grown || mx[h] > m[h] + 8.f;
      }
      if (begins || __any_sync(0xffffffffu, grown)) {
        float f[2] = {1.f, 1.f};
#pragma unroll
        for (int h = 0; h < H; ++h) {
          mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
          mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
          const float mn = fmaxf(m[h], mx[h]);
          f[h] = mn == -INFINITY ? 1.f : ex2(m[h] - mn);
          m[h] = mn;
          l[h] *= f[h];
        }
        if (!begins) {
          if (!(ok = product_done(it - 1))) return;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < DP / 32; ++c) {
            uint32_t o[16];
            tmem_ld_16x32(tmem_o + 32 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f[i / 2 % 2]);
            tmem_st_16x32(tmem_o + 32 * c, o);
          }
        }
      }
      uint32_t p[8] = {};
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const float ms = m[h] == -INFINITY ? 0.f : m[h];
        if (MODE == kCapped) {
          cap_exponents<8>(a, x[h], wide, ms);
          if (edge) hide(h, -INFINITY);
        }
        uint32_t pk[4];
        uint64_t sum[2] = {0, 0};
        exponentials<BF, MODE, 8>(x[h], pair(a.scale2, a.scale2), pair(-ms, -ms), pk, sum);
#pragma unroll
        for (int i = 0; i < 4; ++i) p[2 * i + h] = pk[i];
        float s0, s1;
        unpair(add2(sum[0], sum[1]), s0, s1);
        l[h] += s0 + s1;
      }
      const uint32_t none[8] = {};
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (q != quarter) tmem_st_16x16(ts + 16 * q, none);
      tmem_st_16x16(ts + 16 * quarter, p);
      tmem_wait_st();
    };
    for (int j = 0; j < n; ++j, ++it, rv.next(), rv.next()) {
      const uint32_t buf = it & 1, ts = tmem + 128 * buf + lanes;
      const int base = (first + j) * kAttnKeys;
      if (!(ok = wait_for_all(bars + 8 * (B::kSF + buf), (it >> 1) & 1, abort_flag, a))) break;
      tc_fence_after();
      if (base < klo || base + kAttnKeys > khi) {
        // keys outside the segment (unwritten cache, blocks not loaded): their values must be zeros, since 0
        // times what the memory holds may be NaN
        if (!(ok = wait_for_all(bars + 8 * (B::kFull + rv.st), rv.ph, abort_flag, a))) break;
        hide_value<C>(smp + (1 + rv.st) * C::kTileBytes, thread, base, klo, khi);
        __syncwarp();
      }
      uint32_t sc[16];
      tmem_ld_16x32(ts + 32 * quarter, sc);
      tmem_wait_ld();
      if (both)
        tile(std::integral_constant<int, 2>{}, sc, ts, base, j == 0);
      else
        tile(std::integral_constant<int, 1>{}, sc, ts, base, j == 0);
      if (!ok) break;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 8 * (B::kPF + buf));
    }
    if (!ok) break;
    // the next piece has been handed over: its first scores may be on their way
    const uint32_t dn = (pieces + 1) % kPieces;
    if (!(ok = wait_for_all(bars + 8 * (B::kDF + dn), ((pieces + 1) / kPieces) & 1, abort_flag, a))) break;
    fetch(piece[dn]);
    const uint32_t ob = pieces & 1;  // the rest is the finishing warps' work
    float2 *ml = reinterpret_cast<float2 *>(smp + C::kScratchAt + 4 * kJoinRows * C::kScratchRow * 4) + ob * 4 * 32;
    if (!(ok = wait_for_all(bars + 8 * (B::kOE + ob), ((pieces >> 1) & 1) ^ 1, abort_flag, a))) break;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      if ((lane & 3) == 0) ml[32 * quarter + lane / 4 + 8 * h] = make_float2(m[h], l[h]);
    }
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(bars + 8 * (B::kML + ob));
      mbar_arrive(bars + 8 * (B::kDE + pieces % kPieces));
    }
  }
}

// kSpread: the finishing warps.  Eight rows at a time: the quarters lay their rows side by side, then sixteen
// threads to a row add them, relative to the largest of their maxima.
template <int DP, bool BF>
__device__ void finish(const AttnArgs &a, const volatile Piece *piece, uint8_t *smp, uint32_t bars, uint32_t tmem,
                       volatile int *abort_flag, volatile int *last_flag, volatile int *marked) {
  using C = Cfg<kSpread, DP>;
  using B = Bars<C::kStages>;
  const int quarter = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31, thread = 32 * quarter + lane;
  float *sh = reinterpret_cast<float *>(smp + C::kScratchAt);
  constexpr int V = DP / 16, kPart = DP * 128, kBatch = 8;
  const int c = (thread & 15) * V;  // this thread's columns c .. c + V - 1
  auto slot_of = [&](int cta, int c0) { return part_slot(cta, c0, 1, 0); };
  Group<C::kStages> group{bars, 0, 0, abort_flag};
  bool ok = true;
  const int row0 = thread >> 4, tok0 = over_g(a, row0), head0 = row0 - tok0 * a.G;  // the first eight rows: this thread's
  // their results over the shared prefix, fetched a piece ahead where the next one is known by then
  float pl = 0.f;
  float4 po[V / 4];
  uint32_t fetched = 0;  // pieces up to here
  auto fetch = [&](const volatile Piece &w) {
    if (w.n && w.merge && row0 < w.ntok * a.G && c < a.D) {
      const size_t at = (size_t)(w.tok0 + tok0) * a.Hq + w.head * a.G + head0;
      pl = a.prefix_lse[at];
#pragma unroll
      for (int i = 0; i < V / 4; ++i) po[i] = *reinterpret_cast<const float4 *>(a.prefix_o + at * a.D + c + 4 * i);
    }
    ++fetched;
  };
  if (a.after_prefix) pdl_wait();
  for (uint32_t pieces = 0; ok; ++pieces) {
    const uint32_t d = pieces % kPieces, ob = pieces & 1, par = (pieces >> 1) & 1;
    if (!wait_for_all(bars + 8 * (B::kDF + d), (pieces / kPieces) & 1, abort_flag, a)) break;
    const volatile Piece &w = piece[d];
    if (w.n == 0) break;
    const int nrows = w.ntok * a.G, c0 = w.c0, c1 = w.c1;
    const bool merge = w.merge;
    const float2 *ml = reinterpret_cast<const float2 *>(sh + 4 * kJoinRows * C::kScratchRow) + ob * 4 * 32;
    if (fetched == pieces) fetch(w);
    if (!(ok = wait_for_all(bars + 8 * (B::kML + ob), par, abort_flag, a))) break;
    if (!(ok = wait_for_all(bars + 8 * (B::kOF + ob), par, abort_flag, a))) break;
    tc_fence_after();
    const uint32_t tmem_o = tmem + 256 + 128 * ob + ((uint32_t)(32 * quarter) << 16);
    auto from_tmem = [&](int k, float (&v)[32]) {
      __syncwarp();
      tmem_ld32(tmem_o + 32 * k, reinterpret_cast<uint32_t *>(v));
      tmem_wait_ld();
    };
    for (int r0 = 0; r0 < nrows && ok; r0 += kJoinRows) {
      if (r0 > 0 && !(ok = group.join(a))) break;  // the rows before have been read
#pragma unroll
      for (int k = 0; k < DP / 32; ++k) {
        float v[32];
        from_tmem(k, v);
        if (lane >= r0 && lane < r0 + kJoinRows) {
          float4 *d = reinterpret_cast<float4 *>(sh + (quarter * kJoinRows + lane - r0) * C::kScratchRow + 32 * k);
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
      }
      if (!(ok = group.join(a))) break;
      const int rr = r0 + (thread >> 4);  // this thread's row and columns c .. c + V - 1
      const bool mine = rr < nrows;
      float mm = -INFINITY, ll = 0.f, v[V];
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = 0.f;
      if (mine) {
#pragma unroll
        for (int q = 0; q < 4; ++q) mm = fmaxf(mm, ml[q * 32 + rr].x);
        const float ms = mm == -INFINITY ? 0.f : mm;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 y = ml[q * 32 + rr];
          const float f = ex2(y.x - ms);
          ll = fmaf(f, y.y, ll);
          const float4 *p = reinterpret_cast<const float4 *>(sh + (q * kJoinRows + rr - r0) * C::kScratchRow + c);
#pragma unroll
          for (int i = 0; i < V; i += 4) {
            const float4 z = p[i / 4];
            v[i] = fmaf(f, z.x, v[i]);
            v[i + 1] = fmaf(f, z.y, v[i + 1]);
            v[i + 2] = fmaf(f, z.z, v[i + 2]);
            v[i + 3] = fmaf(f, z.w, v[i + 3]);
          }
        }
      }
      bool last = c0 == c1;
      if (!last) {
        const size_t my = slot_of(blockIdx.x, c0);
        // the threads of a row, one half of the warp, with columns that are not finite
        uint32_t odd[V / 4];
#pragma unroll
        for (int i = 0; i < V / 4; ++i)
          odd[i] = __ballot_sync(0xffffffffu, !finite(largest_before<4>(v + 4 * i, 4))) >> (lane & 16) & 0xffffu;
        if (mine) {
#pragma unroll
          for (int i = 0; i < V; i += 4)
            __stcg(reinterpret_cast<float4 *>(a.part_o + my * kPart + ((c + i) / 4 * 128 + rr) * 4),
                   make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]));
          if (c == 0) {
            __stcg(a.part_ml + my * 128 + rr, make_float2(mm, ll));
            if (a.join) a.part_odd[my * 128 + rr] = V == 4 ? odd[0] : every_other(odd[0]) | every_other(odd[V / 4 - 1]) << 1;
          }
        }
        if (a.join || r0 + kJoinRows < nrows) continue;
        last = group.last_to_arrive(a, c0, c1, thread, last_flag, ok);
        if (!ok) break;
      }
      // whole tiles: these eight rows; split tiles: once all pieces are there, all rows
      for (int q0 = c0 == c1 ? r0 : 0; last && q0 < (c0 == c1 ? min(nrows, r0 + kJoinRows) : nrows); q0 += kJoinRows) {
        int slot = thread >> 4, share = 0;  // (row, share of its pieces)
        if (c0 != c1) {
          // running maximum and sums, eight pieces under way; where rows are few, several threads share one's pieces
          const int shares = nrows > 4 ? 1 : nrows > 2 ? 2 : nrows > 1 ? 4 : 8, rows = kJoinRows / shares;
          share = slot / rows;
          slot -= share * rows;
          const int ro = q0 + slot;
          mm = -INFINITY;
          ll = 0.f;
#pragma unroll
          for (int i = 0; i < V; ++i) v[i] = 0.f;
          if (ro < nrows) {
#pragma unroll 1
            for (int p0 = c0 + share; p0 <= c1; p0 += kBatch * shares) {
              float2 y[kBatch];
              float4 z[kBatch][V / 4];
#pragma unroll
              for (int k = 0; k < kBatch; ++k) {
                y[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
                for (int i = 0; i < V / 4; ++i) z[k][i] = make_float4(0.f, 0.f, 0.f, 0.f);
                const int p = p0 + k * shares;
                if (p <= c1) {
                  const size_t at = slot_of(p, c0);
                  y[k] = __ldcg(a.part_ml + at * 128 + ro);
#pragma unroll
                  for (int i = 0; i < V / 4; ++i)
                    z[k][i] = __ldcg(reinterpret_cast<const float4 *>(a.part_o + at * kPart + ((c / 4 + i) * 128 + ro) * 4));
                }
              }
              float mn = mm;
#pragma unroll
              for (int k = 0; k < kBatch; ++k) mn = fmaxf(mn, y[k].x);
              const float ms = mn == -INFINITY ? 0.f : mn, keep = ex2(mm - ms);
              ll *= keep;
#pragma unroll
              for (int i = 0; i < V; ++i) v[i] *= keep;
#pragma unroll
              for (int k = 0; k < kBatch; ++k) {
                const float f = ex2(y[k].x - ms);
                ll = fmaf(f, y[k].y, ll);
#pragma unroll
                for (int i = 0; i < V; i += 4) {
                  v[i] = fmaf(f, z[k][i / 4].x, v[i]);
                  v[i + 1] = fmaf(f, z[k][i / 4].y, v[i + 1]);
                  v[i + 2] = fmaf(f, z[k][i / 4].z, v[i + 2]);
                  v[i + 3] = fmaf(f, z[k][i / 4].w, v[i + 3]);
                }
              }
              mm = mn;
            }
          }
          if (shares > 1) {  // the shares' sums side by side, as the quarters' before
            float2 *share_ml = reinterpret_cast<float2 *>(sh + kJoinRows * C::kScratchRow);
            if (share > 0) {
#pragma unroll
              for (int i = 0; i < V; i += 4)
                *reinterpret_cast<float4 *>(sh + (share * rows + slot) * C::kScratchRow + c + i) =
                    make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
              if (c == 0) share_ml[share * rows + slot] = make_float2(mm, ll);
            }
            if (!(ok = group.join(a))) break;
            if (share == 0) {
              float mn = mm;
#pragma unroll 1
              for (int k = 1; k < shares; ++k) mn = fmaxf(mn, share_ml[k * rows + slot].x);
              const float ms = mn == -INFINITY ? 0.f : mn, keep = ex2(mm - ms);
              ll *= keep;
#pragma unroll
              for (int i = 0; i < V; ++i) v[i] *= keep;
#pragma unroll 1
              for (int k = 1; k < shares; ++k) {
                const float2 y = share_ml[k * rows + slot];
                const float f = ex2(y.x - ms);
                ll = fmaf(f, y.y, ll);
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] = fmaf(f, sh[(k * rows + slot) * C::kScratchRow + c + i], v[i]);
              }
              mm = mn;
            }
          }
        }
        const int ro = q0 + slot;
        const bool use = share == 0 && ro < nrows;
        const bool near = q0 == 0;  // fetched above
        const int ro_t = over_g(a, ro), tok = w.tok0 + ro_t, head = w.head * a.G + ro - ro_t * a.G;
        bool again = false;
        if (use) {
          if (merge && !near) pl = a.prefix_lse[(size_t)tok * a.Hq + head];
          const RowOut out = row_out(a, tok, head, merge, pl, mm, ll);
          again = !store_cols<V, BF>(a, out, tok, head, c, v, near ? po : nullptr) && finite(ll);
          if (c == 0) store_lse(a, out);
        }
        const unsigned flagged = __ballot_sync(0xffffffffu, again);
        if (__builtin_expect(flagged != 0, 0)) {
          __syncwarp();  // the row's stores come before its mark
          if (lane % 16 == 0 && (flagged >> lane & 0xffffu)) {
            const int rw = q0 + 2 * quarter + lane / 16, rw_t = rw / a.G;
            const int rw_tok = w.tok0 + rw_t, rw_head = w.head * a.G + rw - rw_t * a.G;
            mark_row(a, rw_tok, rw_head, row_out(a, rw_tok, rw_head, merge, pl, mm, ll).lse2, marked);
          }
        }
      }
    }
    if (!ok) break;
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(bars + 8 * (B::kOE + ob));
      mbar_arrive(bars + 8 * (B::kDE + d));
    }
    const uint32_t dn = (pieces + 1) % kPieces;
    if (__all_sync(0xffffffffu, mbar_try_wait(bars + 8 * (B::kDF + dn), ((pieces + 1) / kPieces) & 1))) fetch(piece[dn]);
    ok = group.join(a);  // the shared rows have been read
  }
}

// Rows of this warp whose columns are not finite: bit `it` of `todo` for the CTA's piece of work number `it`.  Those columns
// were not stored.  Where pieces of the row are not finite, all CTAs that have such columns of it find the same ones, and
// one of them computes the row, once; where only the sum overflowed each does so for its columns.
template <int COLS, bool BF, bool TREE>
static __device__ __noinline__ void redo_join(const AttnArgs &a, unsigned todo, int streams) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int it = 0; it < 16; ++it) {
    const int i = blockIdx.x + it * gridDim.x, col = i % COLS, s = i / COLS % streams;
#pragma unroll 1
    for (unsigned left = __ballot_sync(0xffffffffu, todo >> it & 1u); left; left &= left - 1) {
      const AttnSplit *sp = a.list.splits + i / (streams * COLS);
      const AttnTile t = load_tile(&sp->t);
      const int row = (threadIdx.x & ~31) + __ffs(left) - 1, row_t = over_g(a, row);
      uint32_t odd = 0;
      for (int p = sp->c0 + lane; p <= sp->c1; p += 32) odd |= a.part_odd[part_slot(p, sp->c0, streams, s) * 128 + row];
      odd = __reduce_or_sync(0xffffffffu, odd) & (0xffffffffu >> (32 - a.D / 4));
      uint32_t groups = 1u << col;
      if (odd & groups) {
        groups = odd;
        for (int k = row % __popc(odd); k > 0; --k) odd &= odd - 1;  // rows are dealt out among the CTAs
        if (__ffs(odd) - 1 != col) continue;
      }
      const int tok = t.tok0 + s * a.list.tpt + row_t, head = sp->head * a.G + row - row_t * a.G;
      const bool merge = t.merge && !a.to_prefix;
      float m = -INFINITY, l = 0.f;
      for (int p = sp->c0; p <= sp->c1; ++p) m = fmaxf(m, __ldcg(a.part_ml + part_slot(p, sp->c0, streams, s) * 128 + row).x);
      for (int p = sp->c0; p <= sp->c1; ++p) {
        const float2 y = __ldcg(a.part_ml + part_slot(p, sp->c0, streams, s) * 128 + row);
        l = fmaf(ex2(y.x - (m == -INFINITY ? 0.f : m)), y.y, l);
      }
      const float lse2 = row_out(a, tok, head, merge, merge ? a.prefix_lse[(size_t)tok * a.Hq + head] : 0.f, m, l).lse2;
      redo_row<BF, 1, TREE>(a, tok, head, t.klo, t.khi, t.trow, merge, lse2, groups);
    }
  }
}
// The sum of each split tile's pieces, where tiles are few and their pieces many: one CTA of the attention
// kernel adding up a tile's (18 pieces of 64 KB for 256 rows over a prefix of 4096 keys) took longer than the
// products.  Here a CTA takes 4 columns of a tile's rows at a time, a thread a row, with eight pieces under way;
// of kSpread's 16 rows eight threads share each, its pieces dealt out among them.  (At most 72 registers, so that the
// next kernel's CTAs find room beside these; rows to be computed again take few keys at a time for it, and are done
// behind the loop.  With the 128 registers that four times as many keys take, 64 requests behind a shared prefix of
// 4096 were 4 us slower.)
template <int FORM, int DP, bool BF, bool TREE>
static __global__ void __launch_bounds__(128, 7) attn_join_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int kBatch = 8, kCols = DP / 4;
  constexpr int kRows = FORM == kSpread ? kSpreadRows : 128, kShare = 128 / kRows;
  __shared__ float4 sum_v[kShare][kRows];
  __shared__ float2 sum_ml[kShare][kRows];
  pdl_trigger();
  pdl_wait();
  if (!plan_fits(a)) return;  // (reported by attn_kernel)
  const int streams = FORM == kTwo ? 2 : 1, share = threadIdx.x / kRows, row = threadIdx.x % kRows, row_t = over_g(a, row), row_h = row - row_t * a.G;
  const int n = a.list.meta[2] * streams * kCols;
  // Rows to be computed again, by this CTA's tiles: what is done for them stays out of this loop's registers.
  unsigned todo = 0;
#pragma unroll 1
  for (int i = blockIdx.x, it = 0; i < n; i += gridDim.x, ++it) {
    const int c = i % kCols * 4, s = i / kCols % streams;
    const AttnSplit *sp = a.list.splits + i / (streams * kCols);
    const AttnTile t = load_tile(&sp->t);
    const int4 x = *reinterpret_cast<const int4 *>(&sp->head);
    const int c0 = x.y, c1 = x.z, tok = t.tok0 + s * a.list.tpt + row_t, h = x.x * a.G + row_h;
    const bool valid = row < min(a.list.tpt, t.ntok - s * a.list.tpt) * a.G && c < a.D, merge = t.merge && !a.to_prefix;
    float pl = 0.f, m = -INFINITY, l = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
    if (valid) {
      // pieces of this thread: the CTAs c0 + share, c0 + share + kShare, ...; all but c0's are their CTAs' first (see
      // part_slot), two slots apart
      const int step = 2 * streams * kShare;
      auto load = [&](size_t at, float2 &y, float4 &z) {
        y = __ldcg(a.part_ml + at * 128 + row);
        z = __ldcg(reinterpret_cast<const float4 *>(a.part_o + at * (DP * 128)) + c / 4 * 128 + row);
      };
      float2 y0 = make_float2(-INFINITY, 0.f);
      float4 v0 = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c0 + share <= c1) load(part_slot(c0 + share, c0, streams, s), y0, v0);
      const size_t next = part_slot(c0 + share + kShare, c0, streams, s);
      if (merge && share == 0) pl = a.prefix_lse[(size_t)tok * a.Hq + h];
      m = y0.x;
      l = y0.y;
      v[0] = v0.x, v[1] = v0.y, v[2] = v0.z, v[3] = v0.w;
      size_t at = next;
#pragma unroll 1
      for (int p = c0 + share + kShare; p <= c1; p += kBatch * kShare, at += kBatch * step) {
        float2 y[kBatch];
        float4 z[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          y[k] = make_float2(-INFINITY, 0.f);
          z[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (p + k * kShare <= c1) load(at + k * step, y[k], z[k]);
        }
        float mn = m;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) mn = fmaxf(mn, y[k].x);
        const float ms = mn == -INFINITY ? 0.f : mn, keep = ex2(m - ms);
        l *= keep;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] *= keep;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const float f = ex2(y[k].x - ms);
          l = fmaf(f, y[k].y, l);
          v[0] = fmaf(f, z[k].x, v[0]);
          v[1] = fmaf(f, z[k].y, v[1]);
          v[2] = fmaf(f, z[k].z, v[2]);
          v[3] = fmaf(f, z[k].w, v[3]);
        }
        m = mn;
      }
      if (kShare > 1) {
        sum_ml[share][row] = make_float2(m, l);
        sum_v[share][row] = make_float4(v[0], v[1], v[2], v[3]);
      }
    }
    if (kShare > 1) {
      __syncthreads();
      if (valid && share == 0) {
        float mn = m;
#pragma unroll
        for (int k = 1; k < kShare; ++k) mn = fmaxf(mn, sum_ml[k][row].x);
        const float ms = mn == -INFINITY ? 0.f : mn, keep = ex2(m - ms);
        l *= keep;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] *= keep;
#pragma unroll
        for (int k = 1; k < kShare; ++k) {
          const float2 y = sum_ml[k][row];
          const float4 z = sum_v[k][row];
          const float f = ex2(y.x - ms);
          l = fmaf(f, y.y, l);
          v[0] = fmaf(f, z.x, v[0]);
          v[1] = fmaf(f, z.y, v[1]);
          v[2] = fmaf(f, z.z, v[2]);
          v[3] = fmaf(f, z.w, v[3]);
        }
        m = mn;
      }
      __syncthreads();
    }
    if (valid && share == 0) {
      const RowOut out = row_out(a, tok, h, merge, pl, m, l);
      const bool sums = finite(l);
      if (!store_cols<4, BF>(a, out, tok, h, c, v, nullptr, sums) && sums) todo |= 1u << it;
      if (c == 0) store_lse(a, out);
    }
  }
  if (__any_sync(0xffffffffu, todo != 0)) redo_join<kCols, BF, TREE>(a, todo, streams);
}

template <int FORM, int DP, bool BF, int MODE, bool TREE>
__global__ void __launch_bounds__(Cfg<FORM, DP>::kThreads, 1) attn_kernel(const __grid_constant__ AttnMaps maps,
                                                                       const __grid_constant__ AttnArgs a) {
  using C = Cfg<FORM, DP>;
  using B = Bars<C::kStages>;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(8) uint64_t bar_mem[B::kNum];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag, last_flag[2], marked;
  __shared__ Piece piece[kPieces];
  __shared__ float2 other[TREE && FORM == kTwo ? kAttnRows : 1];  // maxima and sums of stream 1, where it has the same rows
  const int warp = threadIdx.x >> 5;
  const uint32_t bars = smem_u32(bar_mem), sm = smem_u32(smem);
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(bars + 8 * (B::kFull + i), 1);
      mbar_init(bars + 8 * (B::kEmpty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars + 8 * (B::kQF + i), 1);
      mbar_init(bars + 8 * (B::kQE + i), 1);
      mbar_init(bars + 8 * (B::kSF + i), 1);
      mbar_init(bars + 8 * (B::kPF + i), 4);
      mbar_init(bars + 8 * (B::kOD + i), 1);
      mbar_init(bars + 8 * (B::kJoin + i), 4);
      mbar_init(bars + 8 * (B::kOF + i), 1);
      mbar_init(bars + 8 * (B::kOE + i), 4);
      mbar_init(bars + 8 * (B::kML + i), 4);
      mbar_init(bars + 8 * (B::kPE + i), 4);
    }
    mbar_init(bars + 8 * B::kDrain, 1);
    mbar_init(bars + 8 * B::kMerge, 8);
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(bars + 8 * (B::kDF + i), 1);
      mbar_init(bars + 8 * (B::kDE + i), C::kProdWarp + 1);  // the softmax and finishing warps and the MMA warp
    }
    marked = 0;
    abort_flag = (sm & 1023u) != 0u;  // the swizzled tiles are 1 KB-aligned
    if (abort_flag) atomicOr(a.err, kAttnErrWait);
    fence_mbar_init();
  }
  if (warp == C::kMmaWarp) {
    tmem_alloc(smem_u32(&tmem_slot), kTmemColsAttn);
    tmem_relinquish();
  }
  if (threadIdx.x == 32 * C::kProdWarp) {
    prefetch_tensormap(&maps.q);
    prefetch_tensormap(&maps.k);
    prefetch_tensormap(&maps.v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  // Set up before the previous kernels of the stream have finished; what they wrote is read from here on.  Behind
  // the kernels over the shared prefixes only the finishing code waits: those kernels write nothing that the
  // others read, and whatever ran before them is complete, since the first of them lets its successor begin only
  // at its end.  (At its end, because the successor's many small CTAs would otherwise crowd the SMs that are done
  // first.)
  if (!a.join) pdl_trigger();
  if (!a.after_prefix) pdl_wait();
  if (warp < C::kSoftWarps) {
    if (FORM == kTwo) regs_inc<kRegsSoft>();
    if (!abort_flag) {
      if constexpr (FORM == kSpread)
        soften_few<DP, BF, MODE, TREE>(a, piece, smem, bars, tmem, &abort_flag);
      else
        soften<DP, BF, MODE, TREE>(a, piece, smem, bars, tmem, &abort_flag, last_flag, &marked, other);
    }
    if constexpr (FORM == kTwo) {  // (here, where a warp has the registers for it)
      static_assert(FORM != kTwo || C::kSoftWarps == 8, "a barrier of 256 threads");
      __syncwarp();
      asm volatile("bar.sync 1, 256;\n" ::: "memory");
      if (__all_sync(0xffffffffu, marked && !abort_flag)) redo_marked<BF, 2, TREE>(a, C::kSoftWarps);
    }
  } else if (warp < C::kProdWarp) {
    if constexpr (FORM == kSpread) {
      if (!abort_flag) finish<DP, BF>(a, piece, smem, bars, tmem, &abort_flag, last_flag, &marked);
    }
  } else {
    if (FORM == kTwo) regs_dec<kRegsOther>();
    if (abort_flag) {
    } else if (warp < C::kMmaWarp) {
      produce<FORM, DP, TREE>(a, maps, warp - C::kProdWarp, piece, sm, bars, &abort_flag);
    } else if (warp == C::kMmaWarp) {
      issue<FORM, DP, BF, TREE>(a, piece, sm, bars, tmem, &abort_flag);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemColsAttn);
    __syncwarp();
  }
  if (FORM == kSpread && __all_sync(0xffffffffu, marked && !abort_flag)) redo_marked<BF, 1, TREE>(a, C::kThreads / 32);
}

template <int FORM, int DP, bool BF, int MODE, bool TREE>
static int launch_one(const AttnArgs &a, const AttnMaps &maps, cudaStream_t st) {
  using C = Cfg<FORM, DP>;
  static_assert(C::kStages >= 4, "two key tiles in flight");
  auto kern = attn_kernel<FORM, DP, BF, MODE, TREE>;
  static std::atomic<uint64_t> done{0};  // devices whose limit has been raised
  const uint64_t bit = 1ull << (a.device & 63);
  if (!(done.load(std::memory_order_relaxed) & bit)) {
    if (cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem)) return (int)e;
    if (a.device < 64) done.fetch_or(bit, std::memory_order_relaxed);
  }
  if (cudaError_t e = launch_pdl(kern, dim3(a.ctas), dim3(C::kThreads), (size_t)C::kSmem, st, maps, a)) return (int)e;
  if (!a.join) return 0;
  // (a split ends a CTA's share, so that there are at most a.ctas of them with two streams of 32 column groups each: not
  // more than 16 pieces of work for a CTA here, as redo_join counts on)
  return (int)launch_pdl(attn_join_kernel<FORM, DP, BF, TREE>, dim3(4 * a.ctas), dim3(128), 0, st, a);
}

template <int FORM, int DP, bool BF, bool TREE>
static int launch_mode(const AttnArgs &a, const AttnMaps &maps, cudaStream_t st) {
  // kPlain folds a positive scale into the exponent's multiply-add; caps alone have the form above (for scales whose
  // ninth power is far from what fp32 holds), and everything else transforms the scores first
  if (!(a.softcap > 0.f) && !a.slopes && a.scale > 0.f) return launch_one<FORM, DP, BF, kPlain, TREE>(a, maps, st);
  if (!a.slopes && a.inv_cap >= 1e-3f && a.inv_cap <= 1e2f) return launch_one<FORM, DP, BF, kCapped, TREE>(a, maps, st);
  return launch_one<FORM, DP, BF, kGeneral, TREE>(a, maps, st);
}
template <int FORM, int DP, bool TREE>
static int launch_type(const AttnArgs &a, const AttnMaps &maps, int bf16, cudaStream_t st) {
  return bf16 ? launch_mode<FORM, DP, true, TREE>(a, maps, st) : launch_mode<FORM, DP, false, TREE>(a, maps, st);
}

template <int FORM, bool TREE>
int launch_form(const AttnArgs &a, const AttnMaps &maps, int bf16, cudaStream_t st) {
  return a.D > 64 ? launch_type<FORM, 128, TREE>(a, maps, bf16, st) : launch_type<FORM, 64, TREE>(a, maps, bf16, st);
}

}  // namespace pw
