"""Shared blocks, trimmed requests and compaction of the KV-block allocator (host only) against the oracle's accounting."""
import numpy as np
import pytest

from oracle import kv as okv

pw = pytest.importorskip("any_precision_bit_gb300")


@pytest.fixture(scope="module", autouse=True)
def built():
    from any_precision_bit_gb300 import _build
    _build.build()


@pytest.fixture
def kv():
    h = pw.pw_kv_create(100 * 8, 8)
    yield h
    pw.pw_kv_destroy(h)


def ids(kv, r):
    return pw.pw_kv_blocks(kv, r).tolist()


def refused(status, f, *args):
    with pytest.raises(pw.PwError) as e:
        f(*args)
    assert e.value.status == status


def used(kv):
    return pw.pw_kv_get_stats(kv)["used_blocks"]


def test_a_fork_by_hand(kv):
    pw.pw_kv_grow(kv, 1, 4)
    pw.pw_kv_fork(kv, 1, 2, 3)
    pw.pw_kv_fork(kv, 2, 3, 1)
    assert ids(kv, 2) == [0, 1, 2] and ids(kv, 3) == [0] and used(kv) == 4
    assert pw.pw_kv_unshare(kv, 2, 2) == (2, 4) and ids(kv, 2) == [0, 1, 4] and used(kv) == 5
    assert pw.pw_kv_unshare(kv, 2, 2) == (4, 4) and pw.pw_kv_unshare(kv, 1, 3) == (3, 3)
    assert pw.pw_kv_unshare(kv, 1, 2) == (2, 2)  # the fork has its own now
    assert pw.pw_kv_release(kv, 1) == 2 and used(kv) == 3  # 0 and 1 are still held
    assert pw.pw_kv_trim(kv, 2, 1) == 2 and ids(kv, 2) == [0] and used(kv) == 1
    assert pw.pw_kv_trim(kv, 2, 5) == 0 and pw.pw_kv_trim(kv, 77, 0) == 0
    assert pw.pw_kv_release(kv, 2) == 0 and pw.pw_kv_release(kv, 3) == 1 and used(kv) == 0


def test_compaction_by_hand(kv):
    for r in range(5):
        pw.pw_kv_grow(kv, r, 3)
    pw.pw_kv_fork(kv, 4, 9, 2)
    pw.pw_kv_release(kv, 0)
    pw.pw_kv_release(kv, 2)
    src, dst = pw.pw_kv_compact(kv, 9)
    assert src.tolist() == [9, 10, 11, 12, 13, 14] and dst.tolist() == [0, 1, 2, 6, 7, 8]
    assert ids(kv, 3) == [0, 1, 2] and ids(kv, 4) == [6, 7, 8] and ids(kv, 9) == [6, 7] and ids(kv, 1) == [3, 4, 5]
    assert pw.pw_kv_compact(kv, 9)[0].size == 0
    assert pw.pw_kv_grow(kv, 5, 1).tolist() == [9]  # the mark came down
    assert pw.pw_kv_unshare(kv, 9, 0) == (6, 10)


def test_refusals(kv):
    pw.pw_kv_grow(kv, 1, 4)
    refused(pw.PW_ERR_INVALID, pw.pw_kv_fork, kv, 1, 2, 5)
    refused(pw.PW_ERR_INVALID, pw.pw_kv_fork, kv, 7, 2, 1)
    refused(pw.PW_ERR_INVALID, pw.pw_kv_fork, kv, 1, 1, 2)
    refused(pw.PW_ERR_INVALID, pw.pw_kv_fork, kv, 1, 2, -1)
    pw.pw_kv_fork(kv, 1, 2, 2)
    refused(pw.PW_ERR_STATE, pw.pw_kv_fork, kv, 1, 2, 1)
    pw.pw_kv_fork(kv, 7, 8, 0)
    for index in (-1, 2):
        refused(pw.PW_ERR_INVALID, pw.pw_kv_unshare, kv, 2, index)
    refused(pw.PW_ERR_INVALID, pw.pw_kv_unshare, kv, 7, 0)
    refused(pw.PW_ERR_INVALID, pw.pw_kv_trim, kv, 1, -1)
    refused(pw.PW_ERR_INVALID, pw.pw_kv_compact, kv, 3)
    pw.pw_kv_set_weight_bytes(kv, 96 * 8)  # four blocks in all, all in use
    refused(pw.PW_ERR_OOM, pw.pw_kv_unshare, kv, 2, 0)
    assert ids(kv, 2) == [0, 1] and used(kv) == 4
    pw.pw_kv_set_weight_bytes(kv, 95 * 8)
    pw.pw_kv_announce(kv, 2, 1)
    refused(pw.PW_ERR_OOM, pw.pw_kv_unshare, kv, 1, 0)  # the free one is announced
    assert pw.pw_kv_unshare(kv, 2, 0) == (0, 4) and pw.pw_kv_request(kv, 2) == (2, 0)
    lib, n = pw.lib(), pw.C.c_int64(-1)
    pw.pw_kv_release(kv, 1)
    assert lib.pw_kv_compact(kv, 2, None, None, 0, pw.C.byref(n)) == pw.PW_ERR_INVALID and n.value == 1
    assert ids(kv, 2) == [4, 1]
    for f in (lambda: lib.pw_kv_fork(None, 1, 2, 1), lambda: lib.pw_kv_unshare(kv, 2, 0, None, None),
              lambda: lib.pw_kv_trim(None, 1, 0, None), lambda: lib.pw_kv_compact(kv, 2, None, None, 0, None),
              lambda: lib.pw_kv_compact(kv, 2, None, None, 1, pw.C.byref(n))):
        assert f() == pw.PW_ERR_INVALID


@pytest.mark.parametrize("seed", range(12))
def test_random_operations(seed):
    rng = np.random.default_rng(seed)
    S, B = 60 * 8, 8
    lib, ora = pw.pw_kv_create(S, B), okv.KVAllocator(S, B)

    def both(f, g):
        try:
            want = g()
        except okv.KVError:
            with pytest.raises(pw.PwError):
                f()
            return
        got = f()
        got = [x.tolist() for x in got] if isinstance(got, tuple) and hasattr(got[0], "tolist") else got
        got = got.tolist() if hasattr(got, "tolist") else got
        if want is not None:
            assert got == want
    try:
        for _ in range(400):
            r, p, n = int(rng.integers(0, 8)), int(rng.integers(0, 8)), int(rng.integers(0, 9))
            op = rng.choice(["grow", "grow", "release", "announce", "weights", "fork", "fork", "unshare", "unshare", "trim", "compact"])
            if op == "grow":
                both(lambda: pw.pw_kv_grow(lib, r, n), lambda: ora.grow(r, n))
            elif op == "release":
                both(lambda: pw.pw_kv_release(lib, r), lambda: ora.release(r))
            elif op == "announce":
                both(lambda: pw.pw_kv_announce(lib, r, n), lambda: ora.announce(r, n))
            elif op == "weights":
                w = int(rng.integers(0, S))
                both(lambda: pw.pw_kv_set_weight_bytes(lib, w), lambda: ora.set_weight_bytes(w))
            elif op == "fork":
                both(lambda: pw.pw_kv_fork(lib, p, r, n), lambda: ora.fork(p, r, n))
            elif op == "unshare":
                both(lambda: pw.pw_kv_unshare(lib, r, n), lambda: ora.unshare(r, n))
            elif op == "trim":
                both(lambda: pw.pw_kv_trim(lib, r, n), lambda: ora.trim(r, n))
            else:
                limit = ora.used() + int(rng.integers(-1, 6))
                both(lambda: pw.pw_kv_compact(lib, limit), lambda: [list(x) for x in zip(*ora.compact(limit))] or [[], []])
            assert pw.pw_kv_get_stats(lib) == ora.stats()
            for q in range(8):
                assert ids(lib, q) == ora.blocks(q) and pw.pw_kv_request(lib, q) == ora.request(q)
    finally:
        pw.pw_kv_destroy(lib)
