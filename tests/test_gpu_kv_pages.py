"""Kept paths and copied blocks: bit by bit what plain indexing gives, in every layer, and nothing else touched."""
import numpy as np
import pytest

from oracle import attn as oa
from tree_helpers import random_tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from any_precision_bit_gb300 import _build
    _build.build()


class Cache:
    """Caches of L layers with a table of requests of kv_len tokens, blocks in random order; elements are random bits."""

    def __init__(self, kv_len, L=2, Hkv=2, D=64, bt=16, layout="nhd", rows=None, spare=4, seed=0):
        import torch

        import any_precision_bit_gb300 as pw
        self.torch, self.pw = torch, pw
        self.kv_len, self.L, self.bt, self.rows = list(kv_len), L, bt, rows
        R = len(kv_len)
        rng = np.random.default_rng(seed)
        pages = [-(-n // bt) for n in kv_len]
        nb = self.nb = sum(pages) + spare
        perm = rng.permutation(nb).astype(np.int32)
        self.used = perm[:sum(pages)]
        self.free = perm[sum(pages):]
        table = np.full((R if rows is None else max(rows) + 1, max(pages) + 1), -1, dtype=np.int32)
        at = 0
        for r, n in enumerate(pages):
            table[r if rows is None else rows[r], :n] = perm[at:at + n]
            at += n
        self.table0 = table
        shape = {"nhd": (L, 2, nb, bt, Hkv, D), "hnd": (L, 2, nb, Hkv, bt, D), "apart": (L, 2, nb, bt, Hkv + 1, D + 8)}[layout]
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.store = torch.randint(-32768, 32768, shape, dtype=torch.int16, device="cuda", generator=g).view(torch.bfloat16)
        self.cache = self.store.transpose(3, 4) if layout == "hnd" else self.store[..., :Hkv, :D]
        i32 = lambda a: torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
        self.i32 = i32
        self.table = i32(table)
        self.attn = pw.pw_attn_create(pw.pw_attn_desc(L=L, n_heads=Hkv, n_kv_heads=Hkv, head_dim=D, dtype=0, n_blocks=nb,
                                                      block_tokens=bt, max_requests=R, max_tokens=1, n_plans=1, device=0))
        for layer in range(L):
            pw.pw_attn_bind(self.attn, layer, self.cache[layer, 0], self.cache[layer, 1])
        one = i32([0])
        self.kv = i32(kv_len)
        self.step = pw.pw_make_step(i32(kv_len), i32([0] * R), self.table, i32([0] * (R + 1)), self.kv,
                                    torch.zeros(1, dtype=torch.int64, device="cuda"), one, max_new=1,
                                    rows=None if rows is None else i32(rows))

    def bits(self):
        self.torch.cuda.synchronize()
        return self.store.view(self.torch.int16).cpu().numpy().copy()

    def views(self, bits):  # [L][2][nb][bt][Hkv][D] of an array like the store
        t = self.cache
        offset = t.storage_offset()
        return np.lib.stride_tricks.as_strided(bits.reshape(-1)[offset:], t.shape, [2 * s for s in t.stride()])

    def expect_kept(self, before, tree_len, paths):
        want = before.copy()
        view, old, ctx = self.views(want), self.views(before), None
        for layer in range(self.L):
            for kind in range(2):
                view[layer, kind], ctx = oa.keep(old[layer, kind], self.table0, self.kv_len, tree_len, paths, self.bt, self.rows)
        return want, ctx

    def keep(self, tree_len, paths, stream=None):
        width = max([len(p) for p in paths] + [1])
        flat = np.full((len(paths), width), 77, dtype=np.int32)
        for r, p in enumerate(paths):
            flat[r, :len(p)] = p
        ctx = self.i32([-5] * len(paths))
        args = self.i32(tree_len), self.i32(flat), self.i32([len(p) for p in paths])
        self.torch.cuda.synchronize()
        self.pw.pw_kv_keep(self.attn, self.step, *args, ctx_out=ctx, stream=stream)
        self.torch.cuda.synchronize()
        return ctx.tolist()

    def compare_kept(self, tree_len, paths):
        before = self.bits()
        ctx = self.keep(tree_len, paths)
        self.pw.pw_attn_check(self.attn)
        want, want_ctx = self.expect_kept(before, tree_len, paths)
        assert np.array_equal(self.bits(), want) and ctx == want_ctx.tolist()

    def close(self):
        self.pw.pw_attn_destroy(self.attn)


def path_to(tree, node):
    path = []
    while node >= 0:
        path.append(node)
        node = tree[node]
    return path[::-1]


@pytest.mark.parametrize("layout,D,bt", [("nhd", 64, 16), ("hnd", 64, 32), ("apart", 72, 16), ("nhd", 8, 128), ("nhd", 128, 64)])
@pytest.mark.parametrize("L", [1, 3])
def test_paths(layout, D, bt, L):
    rng = np.random.default_rng(D)
    kv = [100, 33, 256, 5, 400, 70]
    nodes = [20, 33, 256, 0, 200, 1]
    paths = []
    for n in nodes:
        paths.append(path_to(random_tree(n, n), int(rng.integers(n // 2, n))) if n else [])
    s = Cache(kv, L=L, D=D, bt=bt, layout=layout)
    try:
        s.compare_kept(nodes, paths)
    finally:
        s.close()


@pytest.mark.parametrize("path", [[], [0], [5], [0, 1, 2, 3], [0, 2], [1, 2, 3, 4, 5, 6, 7, 8, 9], list(range(1, 60)), list(range(0, 60, 2)),
                                  list(range(59, 60)), list(range(60))], ids=lambda p: f"{len(p)}-{sum(p)}")
def test_moves_that_overlap(path):
    s = Cache([137, 60], Hkv=3, D=40, rows=[3, 1])
    try:
        s.compare_kept([60, 60], [path, path[:len(path) // 2]])
    finally:
        s.close()


def test_more_layers_than_one_launch_takes():
    s = Cache([40, 60], L=130, Hkv=1, D=8)
    try:
        s.compare_kept([20, 30], [[0, 5, 19], [2, 3, 29]])
        before = s.bits()
        src, dst = s.i32(s.used[:3]), s.i32(s.free[:3])
        s.torch.cuda.synchronize()
        s.pw.pw_kv_copy(s.attn, src, dst, table=s.table)
        want = before.copy()
        want[:, :, s.free[:3]] = before[:, :, s.used[:3]]
        assert np.array_equal(s.bits(), want)
    finally:
        s.close()


@pytest.mark.parametrize("L", [4, 150])
def test_caches_that_several_layers_share(L):
    """Layers bound to caches of others, and keys that are the values: each cache is moved once, more of them than a launch
    takes among them."""
    s = Cache([90, 50, 130], L=L, Hkv=2, D=16)
    nodes, paths = [40, 30, 100], [[1, 3, 4, 9, 30], [1, 3], list(range(1, 100, 2))]
    bind = lambda layer, k, v: s.pw.pw_attn_bind(s.attn, layer, k, v)  # noqa: E731
    try:
        bind(1, s.cache[0, 0], s.cache[0, 1])  # as layer 0
        bind(2, s.cache[0, 1], s.cache[0, 0])  # the other way round
        bind(3, s.cache[3, 0], s.cache[3, 0])  # one for both
        untouched = [(1, 0), (1, 1), (2, 0), (2, 1), (3, 1)]
        for _ in range(2):
            before = s.bits()
            ctx = s.keep(nodes, paths)
            s.pw.pw_attn_check(s.attn)
            want, want_ctx = s.expect_kept(before, nodes, paths)
            for at in untouched:
                want[at] = before[at]
            assert np.array_equal(s.bits(), want) and ctx == want_ctx.tolist()
            before = s.bits()
            src, dst = s.i32(s.used[:3]), s.i32(s.free[:3])
            s.torch.cuda.synchronize()
            s.pw.pw_kv_copy(s.attn, src, dst)
            want = before.copy()
            want[:, :, s.free[:3]] = before[:, :, s.used[:3]]
            for at in untouched:
                want[at] = before[at]
            assert np.array_equal(s.bits(), want)
            # bound again: the caches are listed anew
            bind(1, s.cache[1, 0], s.cache[1, 1])
            untouched = [(2, 0), (2, 1), (3, 1)]
    finally:
        s.close()


def test_layers_of_different_strides():
    """Heads outermost in one layer, tokens in the others: each is moved by its own strides, and the table renamed once."""
    s = Cache([90, 50], L=4, Hkv=2, D=16)
    try:
        hnd = s.cache[1].reshape(2, s.nb, 2, s.bt, 16).transpose(2, 3)
        s.pw.pw_attn_bind(s.attn, 1, hnd[0], hnd[1])
        view = lambda bits: bits[1].reshape(2, s.nb, 2, s.bt, 16).transpose(0, 1, 3, 2, 4)  # noqa: E731
        nodes, paths = [40, 30], [[1, 3, 4, 9, 30], [1, 3]]
        before = s.bits()
        ctx = s.keep(nodes, paths)
        s.pw.pw_attn_check(s.attn)
        want, want_ctx = s.expect_kept(before, nodes, paths)
        want[1] = before[1]
        for kind in range(2):
            view(want)[kind], _ = oa.keep(view(before)[kind], s.table0, s.kv_len, nodes, paths, s.bt)
        assert np.array_equal(s.bits(), want) and ctx == want_ctx.tolist()
        before = s.bits()
        src, dst = s.i32(s.used[:2]), s.i32(s.free[:2])
        s.torch.cuda.synchronize()
        s.pw.pw_kv_copy(s.attn, src, dst, table=s.table)
        want, renamed = before.copy(), s.table0.copy()
        want[:, :, s.free[:2]] = before[:, :, s.used[:2]]
        for a, b in zip(s.used[:2], s.free[:2]):
            renamed[s.table0 == a] = b
        assert np.array_equal(s.bits(), want) and np.array_equal(s.table.cpu().numpy(), renamed)
    finally:
        s.close()


def test_shared_caches_of_other_strides_are_refused():
    s = Cache([40], L=2, Hkv=2, D=16)
    try:
        k, v = s.cache[0, 0], s.cache[0, 1]
        a, b = ((s.bt * 2 * 16, 16, s.bt * 16, 1), k.shape)
        s.pw.pw_attn_bind(s.attn, 1, k.as_strided(b, a, k.storage_offset()), v.as_strided(b, a, v.storage_offset()))
        before = s.bits()
        with pytest.raises(s.pw.PwError) as e:
            s.keep([20], [[3, 5]])
        assert e.value.status == s.pw.PW_ERR_STATE and "strides" in str(e.value)
        assert np.array_equal(s.bits(), before)
        s.pw.pw_attn_bind(s.attn, 1, s.cache[1, 0], s.cache[1, 1])
        s.compare_kept([20], [[3, 5]])
    finally:
        s.close()


def test_paths_that_are_wrong_are_reported():
    s = Cache([100, 100, 100], D=8)
    good = [3, 7, 12]
    try:
        for path, kept in (([3, 3, 12], 1), ([3, 2, 12], 1), ([3, 7, 20], 2), ([-1, 4, 5], 0), ([25, 26, 27], 0)):
            before = s.bits()
            ctx = s.keep([20] * 3, [good, path, good])
            with pytest.raises(s.pw.PwError) as e:
                s.pw.pw_attn_check(s.attn)
            assert e.value.status == s.pw.PW_ERR_STATE and "kept" in str(e.value)
            want, want_ctx = s.expect_kept(before, [20] * 3, [good, path[:kept], good])
            assert np.array_equal(s.bits(), want) and ctx == want_ctx.tolist()
        for length, n in ((-1, 3), (257, 3), (101, 3), (20, -1), (20, 4), (2, 3)):
            before = s.bits()
            args = s.i32([20, length, 20]), s.i32([good] * 3), s.i32([3, n, 3])
            s.torch.cuda.synchronize()
            s.pw.pw_kv_keep(s.attn, s.step, *args)
            with pytest.raises(s.pw.PwError):
                s.pw.pw_attn_check(s.attn)
            want, _ = s.expect_kept(before, [20] * 3, [good, [], good])
            assert np.array_equal(s.bits(), want)
        before = s.bits()
        s.table[1, 5] = s.nb  # tokens 80 .. 95 of the second request have no place
        s.keep([20] * 3, [good] * 3)
        with pytest.raises(s.pw.PwError):
            s.pw.pw_attn_check(s.attn)
        want, _ = s.expect_kept(before, [20] * 3, [good, [], good])
        assert np.array_equal(s.bits(), want)
    finally:
        s.close()


@pytest.mark.parametrize("layout,D,bt", [("nhd", 64, 16), ("hnd", 64, 32), ("apart", 72, 16), ("nhd", 8, 128), ("nhd", 128, 128)])
@pytest.mark.parametrize("n", [1, 2, 37, 64, 65, 150])
def test_copies(layout, D, bt, n):
    s = Cache([160 * bt, 3 * bt], D=D, bt=bt, layout=layout, spare=160)
    try:
        rng = np.random.default_rng(n)
        src, dst = rng.choice(s.used, n, replace=False), s.free[:n]
        for table in (None, s.table):
            before = s.bits()
            args = s.i32(src), s.i32(dst)
            s.torch.cuda.synchronize()
            s.pw.pw_kv_copy(s.attn, *args, table=table)
            want = before.copy()
            s.views(want)[:, :, dst] = s.views(before)[:, :, src]
            assert np.array_equal(s.bits(), want)
            s.pw.pw_attn_check(s.attn)
        renamed = s.table0.copy()
        for a, b in zip(src, dst):
            renamed[s.table0 == a] = b
        assert np.array_equal(s.table.cpu().numpy(), renamed)
        # another call, whose blocks were sources and copies before
        args = s.i32(dst), s.i32(src)
        s.torch.cuda.synchronize()
        s.pw.pw_kv_copy(s.attn, *args, table=s.table)
        assert np.array_equal(s.table.cpu().numpy(), s.table0)
    finally:
        s.close()


def test_one_block_to_several_and_none_at_all():
    s = Cache([64])
    try:
        before = s.bits()
        args = s.i32([s.used[0]] * 3), s.i32(s.free[:3])
        s.torch.cuda.synchronize()
        s.pw.pw_kv_copy(s.attn, *args)
        want = before.copy()
        want[:, :, s.free[:3]] = before[:, :, s.used[:1]]
        assert np.array_equal(s.bits(), want)
        s.pw.pw_kv_copy(s.attn, s.i32([]), s.i32([]), table=s.table)
        assert np.array_equal(s.bits(), want) and np.array_equal(s.table.cpu().numpy(), s.table0)
    finally:
        s.close()


def test_copies_of_bad_ids_are_reported():
    s = Cache([64])
    try:
        before = s.bits()
        args = s.i32([s.used[0], -1, s.nb, s.used[1], s.used[2]]), s.i32([s.free[0], s.free[1], s.free[2], -3, 1 << 30])
        s.torch.cuda.synchronize()
        s.pw.pw_kv_copy(s.attn, *args, table=s.table)
        with pytest.raises(s.pw.PwError) as e:
            s.pw.pw_attn_check(s.attn)
        assert e.value.status == s.pw.PW_ERR_STATE and "pw_kv_copy" in str(e.value)
        want, renamed = before.copy(), s.table0.copy()
        want[:, :, s.free[0]] = before[:, :, s.used[0]]
        renamed[renamed == s.used[0]] = s.free[0]
        assert np.array_equal(s.bits(), want) and np.array_equal(s.table.cpu().numpy(), renamed)
        s.pw.pw_attn_check(s.attn)
    finally:
        s.close()


def test_offsets_beyond_32_bits():
    """Blocks 2^31 elements apart: a rotation's cache write, a kept path and a copy."""
    import torch

    import any_precision_bit_gb300 as pw
    far = 1 << 31
    store = torch.empty(2 * far + 4096, dtype=torch.bfloat16, device="cuda")
    k = store.as_strided((3, 16, 1, 64), (far, 64, 64, 1))
    v = store.as_strided((3, 16, 1, 64), (far, 64, 64, 1), 2048)
    k.zero_(), v.zero_()
    i32 = lambda a: torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    attn = pw.pw_attn_create(pw.pw_attn_desc(L=1, n_heads=1, n_kv_heads=1, head_dim=64, dtype=0, n_blocks=3, block_tokens=16,
                                             max_requests=1, max_tokens=20, n_plans=1, device=0))
    try:
        pw.pw_attn_bind(attn, 0, k, v)
        pw.pw_attn_set_rope(attn, 0, [])
        table, slot = i32([[2, 1]]), torch.tensor([*range(32, 48), *range(16, 20)]).cuda()
        step = pw.pw_make_step(i32([0]), i32([20]), table, i32([0, 20]), i32([20]), slot, i32(range(20)), max_new=20)
        x = torch.randn(3, 20, 1, 64, device="cuda").bfloat16()
        q_out = torch.empty_like(x[0])
        pw.pw_attn_rope_append(attn, 0, step, x[0], q_out, x[1], x[2])
        pw.pw_kv_keep(attn, step, i32([8]), i32([[0, 2, 7]]), i32([3]))
        pw.pw_kv_copy(attn, i32([2]), i32([0]), table=table)
        pw.pw_attn_check(attn)
        assert torch.equal(q_out, x[0]) and table.tolist() == [[0, 1]]
        for c, new in ((k, x[1]), (v, x[2])):
            want = new.clone()
            want[13], want[14] = new[14], new[19]
            assert torch.equal(c[2], want[:16]) and torch.equal(c[0], want[:16]) and torch.equal(c[1, :4], want[16:])
            assert not c[1, 4:].any()
    finally:
        pw.pw_attn_destroy(attn)


def test_captured_calls():
    import torch
    s = Cache([100, 100], D=64)
    try:
        tl, keep, n, ctx = s.i32([20, 20]), s.i32([[3, 7, 12], [0, 0, 0]]), s.i32([3, 0]), s.i32([0, 0])
        src, dst = s.i32(s.used[:1]), s.i32(s.free[:1])
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        before = s.bits()
        with torch.cuda.graph(graph, stream=stream):
            s.pw.pw_kv_keep(s.attn, s.step, tl, keep, n, ctx_out=ctx, stream=stream)
            s.pw.pw_kv_copy(s.attn, src, dst, table=s.table, stream=stream)
        assert np.array_equal(s.bits(), before)
        keep[1] = torch.tensor([1, 2, 19], dtype=torch.int32)
        n[1] = 2
        src.fill_(int(s.used[1]))
        torch.cuda.synchronize()
        graph.replay()
        want, want_ctx = s.expect_kept(before, [20, 20], [[3, 7, 12], [1, 2]])
        want[:, :, s.free[0]] = want[:, :, s.used[1]]
        assert np.array_equal(s.bits(), want) and ctx.tolist() == want_ctx.tolist()
        assert int(s.table[0, 1]) == s.free[0]
    finally:
        s.close()


def test_tensors_made_for_a_call_on_another_stream():
    """While that stream is busy their memory is not given out again."""
    import torch
    s = Cache([100, 100], D=64)
    stream = torch.cuda.Stream()

    def addresses(call):
        t = torch.zeros(2000, dtype=torch.int32, device="cuda")  # (of a size that nothing else here has)
        at = t.data_ptr()
        call(t)
        del t
        return at, torch.zeros(2000, dtype=torch.int32, device="cuda").data_ptr()
    try:
        first, second = addresses(lambda t: None)
        assert first == second  # as a rule it comes back at once
        none, used, free = s.i32([0, 0]), s.i32(s.used[:2]), s.i32(s.free[:2])
        for call in (lambda t: s.pw.pw_kv_keep(s.attn, s.step, none, t.view(2, 1000), none, stream=stream),
                     lambda t: s.pw.pw_kv_copy(s.attn, used, free, table=t.view(2, 1000), stream=stream)):
            torch.cuda.synchronize()
            with torch.cuda.stream(stream):
                torch.cuda._sleep(200_000_000)
            first, second = addresses(call)
            assert first != second
        torch.cuda.synchronize()
        s.pw.pw_attn_check(s.attn)
    finally:
        torch.cuda.synchronize()
        s.close()


def test_refusals():
    import torch
    s = Cache([40])
    pw = s.pw
    try:
        one, two = s.i32([0]), s.i32([[0]])
        other = pw.pw_attn_create(pw.pw_attn_desc(L=2, n_heads=2, n_kv_heads=2, head_dim=64, dtype=0, n_blocks=s.nb, block_tokens=16,
                                                  max_requests=1, max_tokens=1, n_plans=1, device=0))
        pw.pw_attn_bind(other, 0, s.cache[0, 0], s.cache[0, 1])
        for call in (lambda: pw.pw_kv_keep(other, s.step, one, two, one), lambda: pw.pw_kv_copy(other, one, one)):
            with pytest.raises(pw.PwError) as e:
                call()
            assert e.value.status == pw.PW_ERR_STATE
        pw.pw_attn_destroy(other)
        for call in (lambda: pw.pw_kv_keep(s.attn, s.step, one.long(), two, one), lambda: pw.pw_kv_keep(s.attn, s.step, one, two.cpu(), one),
                     lambda: pw.pw_kv_keep(s.attn, s.step, one, two, one[:0]), lambda: pw.pw_kv_copy(s.attn, s.i32([0, 1]), one),
                     lambda: pw.pw_kv_copy(s.attn, one, one, table=s.table.long()),
                     lambda: pw.pw_kv_copy(s.attn, one, one, table=s.table[:, ::2])):
            with pytest.raises(ValueError):
                call()
        many = torch.zeros(s.nb + 1, dtype=torch.int32, device="cuda")
        with pytest.raises(pw.PwError) as e:
            pw.pw_kv_copy(s.attn, many, many)
        assert e.value.status == pw.PW_ERR_INVALID
        with pytest.raises(pw.PwError):
            pw.pw_kv_copy(s.attn, one, one, table=s.table[:0])
        with pytest.raises(pw.PwError):
            pw.pw_kv_keep(s.attn, s.step, one, two[:, :0], one)
    finally:
        s.close()
