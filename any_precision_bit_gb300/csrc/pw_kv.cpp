// pw_kv.cpp -- KV-block allocator sharing the device budget with the weight pages (host).
//
// PagedWeight Sec. 3.3 (asynchronous page movement): the planner follows the free KV
// blocks, the allocator headroom and the pending KV growth, and the GPU pages an offload
// retires become headroom the KV blocks can take.  Sec. 3.2, Eq. 7: the free-block count
// F_blk against the reserve T_blk sets the bytes the planner must release.  Here one budget
// S holds the weight pages (W bytes) and the KV blocks (B bytes each):
//   C = floor(max(0, S - W) / B),  F_blk = C - U - P,  headroom = S - W - U B,
// with U the blocks held and P the blocks announced as pending growth.  A grow draws on the
// request's own announcement first and must otherwise fit in F_blk; it is all or nothing.
// Ids are logical and the lowest free one is granted first: ids below the high-water mark
// that were released are kept in an ordered set, so memory grows with the ids in use, not
// with the budget.  Requests may share blocks (a fork holds its parent's); a shared block counts once, and comes free with
// its last holder.
#include <stdint.h>

#include <iterator>
#include <new>
#include <set>
#include <unordered_map>
#include <vector>

#include "../../include/pw.h"

struct pw_kv {
  int64_t S = 0, B = 0, W = 0;
  int64_t n_ids = 0;
  pw_ctx *ctx = nullptr;  // W is read from here when set
  int64_t U = 0, P = 0;
  int32_t next_id = 0;              // ids >= next_id were never granted
  std::set<int32_t> freed;          // released ids below next_id
  std::unordered_map<int64_t, std::vector<int32_t>> held;
  std::unordered_map<int32_t, int64_t> sharers;  // of a block that several requests hold: how many
  std::unordered_map<int64_t, int64_t> announced;
};

namespace {

pw_status refresh_weights(pw_kv *kv) {
  if (!kv->ctx) return PW_OK;
  pw_mem_info mi;
  if (pw_status st = pw_memory(kv->ctx, &mi)) return st;
  kv->W = mi.held_bytes;
  return PW_OK;
}

int64_t capacity(const pw_kv *kv) { return kv->S > kv->W ? (kv->S - kv->W) / kv->B : 0; }

int32_t take_lowest(pw_kv *kv) {
  if (!kv->freed.empty()) {
    const int32_t id = *kv->freed.begin();
    kv->freed.erase(kv->freed.begin());
    return id;
  }
  return kv->next_id++;
}

// The high-water mark comes back down over released ids at its top.
void lower_mark(pw_kv *kv) {
  while (kv->next_id > 0 && !kv->freed.empty() && *kv->freed.rbegin() == kv->next_id - 1) {
    kv->freed.erase(std::prev(kv->freed.end()));
    --kv->next_id;
  }
}

// One holder less of a block that several requests hold; false if it is one request's alone.
bool leave(pw_kv *kv, int32_t id) {
  auto it = kv->sharers.find(id);
  if (it == kv->sharers.end()) return false;
  if (--it->second == 1) kv->sharers.erase(it);
  return true;
}

// The blocks behind the first n_keep of a request's are returned; how many are free now.  Where memory for the free ids
// runs out nothing changes: those that were entered are taken out again, and what comes behind allocates nothing.
bool give_back(pw_kv *kv, std::vector<int32_t> &ids, int64_t n_keep, int64_t *n) {
  if ((int64_t)ids.size() <= n_keep) return true;
  const size_t keep = (size_t)n_keep;
  size_t i = keep;
  try {
    for (; i < ids.size(); ++i)
      if (!kv->sharers.count(ids[i])) {
        kv->freed.insert(ids[i]);
        ++*n;
      }
  } catch (...) {
    while (i-- > keep) kv->freed.erase(ids[i]);
    return false;
  }
  for (i = keep; i < ids.size(); ++i) leave(kv, ids[i]);
  kv->U -= *n;
  ids.resize(keep);
  return true;
}

// A grow's room: the part of n blocks that request r's announcement covers, or -1 where the others do not fit.
int64_t covered(const pw_kv *kv, int64_t request, int64_t n) {
  auto it = kv->announced.find(request);
  const int64_t own = it == kv->announced.end() ? 0 : it->second, c = n < own ? n : own;
  return n - c > capacity(kv) - kv->U - kv->P ? -1 : c;
}

}  // namespace

extern "C" pw_status pw_kv_create(int64_t budget_bytes, int64_t block_bytes, pw_kv **out) {
  if (!out || budget_bytes < 0 || block_bytes <= 0 || budget_bytes / block_bytes >= (int64_t(1) << 31))
    return PW_ERR_INVALID;
  pw_kv *kv = new (std::nothrow) pw_kv;
  if (!kv) return PW_ERR_OOM;
  kv->S = budget_bytes;
  kv->B = block_bytes;
  kv->n_ids = budget_bytes / block_bytes;
  *out = kv;
  return PW_OK;
}

extern "C" void pw_kv_destroy(pw_kv *kv) { delete kv; }

extern "C" pw_status pw_kv_set_weight_bytes(pw_kv *kv, int64_t weight_bytes) {
  if (!kv || weight_bytes < 0) return PW_ERR_INVALID;
  kv->ctx = nullptr;
  kv->W = weight_bytes;
  return PW_OK;
}

extern "C" pw_status pw_kv_attach(pw_kv *kv, pw_ctx *ctx) {
  if (!kv) return PW_ERR_INVALID;
  kv->ctx = ctx;
  if (pw_status st = refresh_weights(kv)) {
    kv->ctx = nullptr;
    return st;
  }
  return PW_OK;
}

extern "C" pw_status pw_kv_announce(pw_kv *kv, int64_t request, int64_t n_blocks) {
  if (!kv || n_blocks < 0) return PW_ERR_INVALID;
  auto it = kv->announced.find(request);
  const int64_t old = it == kv->announced.end() ? 0 : it->second;
  if (n_blocks == 0) {
    if (it != kv->announced.end()) kv->announced.erase(it);
  } else {
    try {
      kv->announced[request] = n_blocks;
    } catch (...) {
      return PW_ERR_OOM;
    }
  }
  kv->P += n_blocks - old;
  return PW_OK;
}

extern "C" pw_status pw_kv_grow(pw_kv *kv, int64_t request, int64_t n_blocks, int32_t *ids_out) {
  if (!kv || n_blocks < 0) return PW_ERR_INVALID;
  if (pw_status st = refresh_weights(kv)) return st;
  const int64_t c = covered(kv, request, n_blocks);
  if (c < 0) return PW_ERR_OOM;
  // U + n <= C <= n_ids, so the ids below n_ids suffice
  std::vector<int32_t> *held;
  try {
    held = &kv->held[request];
    held->reserve(held->size() + (size_t)n_blocks);
  } catch (...) {
    return PW_ERR_OOM;
  }
  std::vector<int32_t> &mine = *held;
  for (int64_t k = 0; k < n_blocks; ++k) {
    const int32_t id = take_lowest(kv);
    mine.push_back(id);
    if (ids_out) ids_out[k] = id;
  }
  kv->U += n_blocks;
  if (c > 0) pw_kv_announce(kv, request, kv->announced[request] - c);
  return PW_OK;
}

extern "C" pw_status pw_kv_release(pw_kv *kv, int64_t request, int64_t *n_released) {
  if (!kv) return PW_ERR_INVALID;
  int64_t n = 0;
  auto it = kv->held.find(request);
  if (it != kv->held.end()) {
    if (!give_back(kv, it->second, 0, &n)) return PW_ERR_OOM;
    kv->held.erase(it);
  }
  lower_mark(kv);
  pw_kv_announce(kv, request, 0);
  if (n_released) *n_released = n;
  return PW_OK;
}

extern "C" pw_status pw_kv_fork(pw_kv *kv, int64_t parent, int64_t child, int64_t n_blocks) {
  if (!kv || n_blocks < 0 || parent == child) return PW_ERR_INVALID;
  auto from = kv->held.find(parent), to = kv->held.find(child);
  if (n_blocks > (from == kv->held.end() ? 0 : (int64_t)from->second.size())) return PW_ERR_INVALID;
  if (to != kv->held.end() && !to->second.empty()) return PW_ERR_STATE;
  if (n_blocks == 0) return PW_OK;
  try {
    std::vector<int32_t> ids(from->second.begin(), from->second.begin() + n_blocks);
    for (int32_t id : ids) kv->sharers.emplace(id, 1);  // (of one that is not shared yet: its holder)
    kv->held[child] = std::move(ids);
  } catch (...) {
    for (int64_t i = 0; i < n_blocks; ++i) {
      auto it = kv->sharers.find(from->second[(size_t)i]);
      if (it != kv->sharers.end() && it->second == 1) kv->sharers.erase(it);
    }
    return PW_ERR_OOM;
  }
  for (int32_t id : kv->held[child]) ++kv->sharers[id];
  return PW_OK;
}

extern "C" pw_status pw_kv_unshare(pw_kv *kv, int64_t request, int64_t index, int32_t *src, int32_t *dst) {
  if (!kv || !src || !dst || index < 0) return PW_ERR_INVALID;
  if (pw_status st = refresh_weights(kv)) return st;
  auto it = kv->held.find(request);
  if (it == kv->held.end() || index >= (int64_t)it->second.size()) return PW_ERR_INVALID;
  int32_t &id = it->second[(size_t)index];
  if (kv->sharers.find(id) == kv->sharers.end()) {
    *src = *dst = id;
    return PW_OK;
  }
  const int64_t c = covered(kv, request, 1);
  if (c < 0) return PW_ERR_OOM;
  *src = id;
  leave(kv, id);
  *dst = id = take_lowest(kv);
  ++kv->U;
  if (c > 0) pw_kv_announce(kv, request, kv->announced[request] - c);
  return PW_OK;
}

extern "C" pw_status pw_kv_trim(pw_kv *kv, int64_t request, int64_t n_keep, int64_t *n_released) {
  if (!kv || n_keep < 0) return PW_ERR_INVALID;
  int64_t n = 0;
  auto it = kv->held.find(request);
  if (it != kv->held.end() && !give_back(kv, it->second, n_keep, &n)) return PW_ERR_OOM;
  lower_mark(kv);
  if (n_released) *n_released = n;
  return PW_OK;
}

extern "C" pw_status pw_kv_compact(pw_kv *kv, int64_t limit, int32_t *src, int32_t *dst, int64_t capacity_out, int64_t *n) {
  if (!kv || !n || limit < kv->U || capacity_out < 0 || (capacity_out > 0 && (!src || !dst))) return PW_ERR_INVALID;
  try {
    std::set<int32_t> used, above;
    for (const auto &h : kv->held) used.insert(h.second.begin(), h.second.end());
    for (int32_t id : used)
      if (id >= limit) above.insert(id);
    *n = (int64_t)above.size();
    if (*n > capacity_out) return PW_ERR_INVALID;
    std::unordered_map<int32_t, int32_t> to;
    std::set<int32_t> freed;
    int32_t place = 0;
    for (int32_t id : above) {
      while (used.count(place)) ++place;
      to[id] = place++;
    }
    // what the moves leave free, below the new high-water mark
    for (const auto &m : to) {
      used.erase(m.first);
      used.insert(m.second);
    }
    const int32_t top = used.empty() ? 0 : *used.rbegin() + 1;
    int32_t at = 0;
    for (int32_t id : used) {
      for (; at < id; ++at) freed.insert(at);
      at = id + 1;
    }
    std::unordered_map<int32_t, int64_t> sharers;
    for (const auto &s : kv->sharers) {
      auto m = to.find(s.first);
      sharers[m == to.end() ? s.first : m->second] = s.second;
    }
    // (nothing below throws)
    int64_t i = 0;
    for (int32_t id : above) {
      src[i] = id;
      dst[i++] = to.find(id)->second;
    }
    for (auto &h : kv->held)
      for (int32_t &id : h.second) {
        auto m = to.find(id);
        if (m != to.end()) id = m->second;
      }
    kv->sharers.swap(sharers);
    kv->freed.swap(freed);
    kv->next_id = top;
  } catch (...) {
    return PW_ERR_OOM;
  }
  return PW_OK;
}

extern "C" pw_status pw_kv_request(const pw_kv *kv, int64_t request, int64_t *held, int64_t *announced) {
  if (!kv) return PW_ERR_INVALID;
  if (held) {
    auto it = kv->held.find(request);
    *held = it == kv->held.end() ? 0 : (int64_t)it->second.size();
  }
  if (announced) {
    auto it = kv->announced.find(request);
    *announced = it == kv->announced.end() ? 0 : it->second;
  }
  return PW_OK;
}

extern "C" pw_status pw_kv_blocks(const pw_kv *kv, int64_t request, int32_t *ids_out, int64_t capacity_out,
                                  int64_t *n) {
  if (!kv || !n || capacity_out < 0 || (capacity_out > 0 && !ids_out)) return PW_ERR_INVALID;
  auto it = kv->held.find(request);
  *n = it == kv->held.end() ? 0 : (int64_t)it->second.size();
  for (int64_t k = 0; k < *n && k < capacity_out; ++k) ids_out[k] = it->second[(size_t)k];
  return PW_OK;
}

extern "C" pw_status pw_kv_get_stats(pw_kv *kv, pw_kv_stats *out) {
  if (!kv || !out) return PW_ERR_INVALID;
  if (pw_status st = refresh_weights(kv)) return st;
  out->budget_bytes = kv->S;
  out->block_bytes = kv->B;
  out->weight_bytes = kv->W;
  out->capacity_blocks = capacity(kv);
  out->used_blocks = kv->U;
  out->pending_blocks = kv->P;
  out->free_blocks = out->capacity_blocks - kv->U - kv->P;
  out->headroom_bytes = kv->S - kv->W - kv->U * kv->B;
  return PW_OK;
}
