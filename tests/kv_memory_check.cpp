// Host check of the KV-block allocator where host memory runs out (compiled and run by test_kv_memory_host.py).
//
// Random operations run on two allocators.  On the first, every allocation of memory within a call fails once, the first,
// then the second and so on, until the call succeeds: each failed call reports PW_ERR_OOM and leaves what the allocator
// tells of itself as it was.  The second runs the operation once with all the memory it wants; results and states agree.
#include <cstdio>
#include <cstdlib>
#include <map>
#include <new>
#include <vector>

#include "../any_precision_bit_gb300/csrc/pw_kv.cpp"

static long countdown = -1;  // allocations until one fails; below zero none does
static bool failed = false;
void *operator new(size_t n) {
  if (countdown == 0) {
    failed = true;
    throw std::bad_alloc();
  }
  if (countdown > 0) --countdown;
  void *p = std::malloc(n ? n : 1);
  if (!p) std::abort();
  return p;
}
void operator delete(void *p) noexcept { std::free(p); }
void operator delete(void *p, size_t) noexcept { std::free(p); }

extern "C" pw_status pw_memory(pw_ctx *, pw_mem_info *) { return PW_ERR_INVALID; }

static unsigned rng_state = 2463534242u;
static int rnd(int n) {  // uniform in [0, n)
  rng_state = rng_state * 1664525u + 1013904223u;
  return (int)((rng_state >> 8) % (unsigned)n);
}

constexpr int kRequests = 8;
using State = std::vector<int64_t>;
static State state_of(pw_kv *kv) {
  State s;
  pw_kv_stats st;
  pw_kv_get_stats(kv, &st);
  for (int64_t v : {st.capacity_blocks, st.used_blocks, st.pending_blocks, st.free_blocks}) s.push_back(v);
  for (int r = 0; r < kRequests; ++r) {
    int64_t held, announced, n;
    pw_kv_request(kv, r, &held, &announced);
    std::vector<int32_t> ids((size_t)held + 1);
    pw_kv_blocks(kv, r, ids.data(), held, &n);
    s.push_back(held);
    s.push_back(announced);
    s.insert(s.end(), ids.begin(), ids.begin() + held);
  }
  return s;
}

// One operation: its status, and all that it answers.
struct Op {
  int kind, r, p, n;
};
static pw_status run(pw_kv *kv, const Op &o, State *out) {
  out->clear();
  int64_t n = -1;
  int32_t a[128], b[128];
  pw_status st;
  switch (o.kind) {
    case 0:
      st = pw_kv_release(kv, o.r, &n);
      break;
    case 1:
      st = pw_kv_trim(kv, o.r, o.n, &n);
      break;
    case 2:
      st = pw_kv_grow(kv, o.r, o.n, a);
      if (!st) out->insert(out->end(), a, a + o.n);
      break;
    case 3:
      st = pw_kv_fork(kv, o.p, o.r, o.n);
      break;
    case 4:
      st = pw_kv_unshare(kv, o.r, o.n, a, b);
      if (!st) out->insert(out->end(), {a[0], b[0]});
      break;
    case 5:
      st = pw_kv_compact(kv, 60, a, b, 128, &n);
      for (int64_t i = 0; !st && i < n; ++i) out->insert(out->end(), {a[i], b[i]});
      break;
    default:
      st = pw_kv_announce(kv, o.r, o.n);
      break;
  }
  out->push_back(n);
  return st;
}

// argv[1] has a 1 or a 0 for each kind of operation: whether its memory fails.
int main(int argc, char **argv) {
  std::map<int, int> shortages;
  for (int trial = 0; trial < 20; ++trial) {
    pw_kv *one = nullptr, *two = nullptr;
    if (pw_kv_create(100 * 8, 8, &one) || pw_kv_create(100 * 8, 8, &two)) return 2;
    for (int step = 0; step < 300; ++step) {
      const Op o{rnd(7), rnd(kRequests), rnd(kRequests), rnd(12)};
      const bool tried = argv[1][o.kind] == '1';
      State got, want;
      pw_status st = PW_OK;
      for (long k = 0;; ++k) {
        const State before = state_of(one);
        got.reserve(256);
        failed = false;
        countdown = tried ? k : -1;
        try {
          st = run(one, o, &got);
        } catch (...) {
          countdown = -1;
          std::printf("FAIL operation %d threw (trial %d, step %d)\n", o.kind, trial, step);
          return 1;
        }
        countdown = -1;
        if (!failed) break;
        ++shortages[o.kind];
        if (st != PW_ERR_OOM || state_of(one) != before) {
          std::printf("FAIL operation %d out of memory: status %d, state %s (trial %d, step %d)\n", o.kind, st,
                      state_of(one) == before ? "as before" : "changed", trial, step);
          return 1;
        }
      }
      const pw_status wanted = run(two, o, &want);
      if (st != wanted || got != want || state_of(one) != state_of(two)) {
        std::printf("FAIL operation %d differs (trial %d, step %d)\n", o.kind, trial, step);
        return 1;
      }
    }
    pw_kv_destroy(one);
    pw_kv_destroy(two);
  }
  for (int kind = 0; kind < 7; ++kind)
    if (argv[1][kind] == '1' && !shortages[kind]) {
      std::printf("FAIL operation %d never ran out of memory\n", kind);
      return 1;
    }
  std::puts("ok");
  return 0;
}
