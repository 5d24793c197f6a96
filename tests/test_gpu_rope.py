"""Norms, rotation and cache write in one pass against the float64 oracle."""
from fractions import Fraction

import numpy as np
import pytest

from attn_helpers import UNIT
from oracle import attn as oa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from any_precision_bit_gb300 import _build
    _build.build()


def freqs(rot, theta=10000.0):
    return theta ** (-np.arange(0, rot, 2) / max(rot, 1))


class Rope:
    """A step of n tokens at random slots of a cache that holds NaN."""

    def __init__(self, n, Hq=4, Hkv=2, D=64, dtype="bf16", bt=16, seed=0, layout="nhd", skip=(), top=100, L=1, scale=1.0):
        import torch

        import any_precision_bit_gb300 as pw
        self.torch, self.pw = torch, pw
        self.n, self.Hq, self.Hkv, self.D, self.bt, self.dtype = n, Hq, Hkv, D, bt, dtype
        dt = self.dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
        rng, g = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
        nb = self.nb = -(-n // bt) + 2
        self.slots = rng.permutation(nb * bt)[:n].astype(np.int64)
        self.slots[list(skip)] = -1
        self.where = rng.integers(0, top, n).astype(np.int32)
        qkv = (scale * torch.randn(n, Hq + 2 * Hkv, D, generator=g)).to(dt).cuda()
        self.q, self.k, self.v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        shape = (L, 2, nb, bt, Hkv, D) if layout == "nhd" else (L, 2, nb, Hkv, bt, D)
        self.cache = torch.full(shape, float("nan"), dtype=dt, device="cuda")
        if layout != "nhd":
            self.cache = self.cache.transpose(3, 4)
        self.out = torch.full((n, Hq, 2, D), float("nan"), dtype=dt, device="cuda")
        i32 = lambda a: torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
        self.slot, self.pos = torch.as_tensor(self.slots).cuda(), i32(self.where)
        self.step = pw.pw_make_step(i32([0]), i32([n]), i32(np.zeros((1, nb))), i32([0, n]), i32([n]), self.slot, self.pos, max_new=n)
        self.attn = pw.pw_attn_create(pw.pw_attn_desc(
            L=L, n_heads=Hq, n_kv_heads=Hkv, head_dim=D, dtype=pw.PW_BF16 if dtype == "bf16" else pw.PW_FP16, n_blocks=nb,
            block_tokens=bt, max_requests=1, max_tokens=n, n_plans=1, device=0))
        for layer in range(L):
            pw.pw_attn_bind(self.attn, layer, self.cache[layer, 0], self.cache[layer, 1])

    def compare(self, rot=None, pos=None, layer=0, q_out=None, **kw):
        """q and the cache: half a step of the result and fp32 sums of D squares, sines and cosines before it, counted in
        2^-24 of the magnitudes that make up an element; fp16 subnormals half of their step 2^-24."""
        t, pw = self.torch, self.pw
        freq = kw.pop("freq", None)
        freq = freqs(self.D if rot is None else rot) if freq is None else freq
        before = self.q.clone()
        out = self.out[:, :, 0] if q_out is None else q_out
        pw.pw_attn_set_rope(self.attn, layer, freq, **kw)
        t.cuda.synchronize()
        pw.pw_attn_rope_append(self.attn, layer, self.step, self.q, out, self.k, self.v,
                               pos=None if pos is None else t.as_tensor(np.asarray(pos, dtype=np.int32)).cuda())
        pw.pw_attn_check(self.attn)
        n_axes = kw.pop("n_axes", 1)
        places = np.stack([self.where] * n_axes) if pos is None else pos
        gains = {"q": kw.pop("q_gain", None), "k": kw.pop("k_gain", None)}
        kw.setdefault("eps", 1e-6)
        some, u = self.slots >= 0, UNIT[self.dtype]
        f = lambda x: x.float().cpu().numpy()  # noqa: E731
        held = f(self.cache[layer]).reshape(2, self.nb * self.bt, self.Hkv, self.D)

        def near(got, x, gain):
            gain = None if gain is None else f(gain) if hasattr(gain, "cpu") else gain
            want, mag = oa.rotate(f(x)[some], np.asarray(places)[:, some], freq, gain=gain, **kw)
            err = np.abs(got - want)
            lim = u * np.abs(want) + (self.D / 2 + 16) * 2.0 ** -24 * mag + 2.0 ** -25
            assert (err <= lim).all(), (float((err / lim).max()), np.argwhere(err > lim)[:4].tolist())
        near(f(out)[some], before, gains["q"])
        near(held[0][self.slots[some]], self.k, gains["k"])
        assert np.array_equal(held[1][self.slots[some]], f(self.v)[some])
        rest = np.ones(self.nb * self.bt, dtype=bool)
        rest[self.slots[some]] = False
        assert np.isnan(held[:, rest]).all(), "wrote beside the slots"
        if q_out is None:
            assert bool(t.isnan(self.out[:, :, 1].float()).all()), "wrote beside q_out"
            assert np.isnan(f(out)[~some]).all(), "wrote a row that is skipped"

    def close(self):
        self.pw.pw_attn_destroy(self.attn)


def run(n, make=None, **kw):
    s = Rope(n, **(make or {}))
    try:
        s.compare(**kw)
    finally:
        s.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(8, 8), (24, 24), (32, 32), (40, 16), (64, 64), (64, 32), (72, 72), (72, 64), (72, 8), (80, 80),
                                   (96, 48), (104, 88), (120, 112), (120, 120), (128, 128), (128, 64), (128, 8), (128, 0),
                                   (128, 120)])
def test_head_dims(D, rot, interleaved, dtype):
    gain = np.random.default_rng(D).normal(1, 0.2, (2, D))
    run(9, dict(D=D, dtype=dtype), rot=rot, interleaved=interleaved)
    run(9, dict(D=D, dtype=dtype), rot=rot, interleaved=interleaved, q_gain=gain[0], k_gain=gain[1])


@pytest.mark.parametrize("n", [1, 2, 3, 17, 100, 1001])
@pytest.mark.parametrize("heads", [(1, 1), (3, 3), (8, 1), (10, 2), (32, 8), (40, 20)], ids=str)
def test_rows_and_heads(n, heads):
    ones = np.ones(64)
    run(n, dict(Hq=heads[0], Hkv=heads[1], top=5000, seed=n), q_gain=ones, k_gain=0.5 * ones, eps=1e-5)


@pytest.mark.parametrize("make", [dict(bt=128), dict(bt=64, layout="hnd"), dict(skip=(0, 7, 8, 20)), dict(skip=tuple(range(21)))],
                         ids=str)
def test_layouts_and_skipped_rows(make):
    run(21, make)
    run(21, {**make, "D": 72}, q_gain=np.ones(72))


@pytest.mark.parametrize("top", [1, 1 << 20, (1 << 31) - 1])
@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(top, interleaved):
    pos = np.array([[0, 1, top - 1, top // 3, top // 7 * 2, -top + 1, -1]])
    run(7, dict(D=128, dtype="fp16"), pos=pos, interleaved=interleaved)
    run(7, dict(D=128, dtype="fp16"), pos=pos, interleaved=interleaved, freq=-freqs(128, 500000.0) * 3)


def two_pi(bits=1400):
    """2 pi as a fraction, by Machin's formula."""
    def atan_of_inverse(n):
        x = total = (1 << bits) // n
        k, sign = 1, -1
        while x:
            x //= n * n
            k += 2
            total += sign * (x // k)
            sign = -sign
        return total
    return Fraction(8 * (4 * atan_of_inverse(5) - atan_of_inverse(239)), 1 << bits)


@pytest.mark.parametrize("sign", [1, -1])
def test_angles_far_away(sign):
    """Sines of angles next to a multiple of pi, which show an angle to a small part of fp32's step: for each frequency the
    position among the farthest 200000 whose sine is the smallest.  The angle is off by what 32 bits of a turn cut off and
    2^31 / 2 steps of 2^-64; sine, scale and result are rounded once or a few times, relative to a sine that small."""
    some = [1.0, 0.3, 2.5, 7.0, 1000.0, 1e5, 1e12, 1e30, 1e300, 2.0 ** 53, 2.0 ** 100 / 3, 5e-324]
    freq = np.array([sign * f for f in [*some, *freqs(128)[:26], *freqs(128, 5e5)[:26]]])
    turn, top, places, want = two_pi(), (1 << 31) - 1, [], []
    near = top - np.arange(200000, dtype=np.uint64)
    for f in freq:
        part = Fraction(float(f)) / turn % 1
        angle = (near * np.uint64(int(part * 2 ** 64))) & np.uint64(2 ** 63 - 1)  # modulo half a turn
        p = int(near[np.argmin(np.minimum(angle, np.uint64(2 ** 63) - angle))])
        halves = 2 * part * p
        whole = round(halves)
        places.append(p)
        want.append((-1) ** whole * np.sin(float((halves - whole) * turn / 2)))
    want, n = np.array(want), len(freq)
    s = Rope(n, Hq=1, Hkv=1, D=128, dtype="fp16")
    try:
        for x in (s.q, s.k):
            x[..., :64], x[..., 64:] = 1, 0
        for way in (1, -1):
            pos = s.torch.as_tensor(way * np.array([places], dtype=np.int32)).cuda()
            s.pw.pw_attn_set_rope(s.attn, 0, freq, scale=1024.0)
            s.torch.cuda.synchronize()
            s.pw.pw_attn_rope_append(s.attn, 0, s.step, s.q, s.out[:, :, 0], s.k, s.v, pos=pos)
            s.pw.pw_attn_check(s.attn)
            held = s.cache[0, 0].reshape(-1, 1, 128)[s.slot]
            for got in (s.out[:, 0, 0], held[:, 0]):
                err = np.abs(got.double().cpu().numpy()[np.arange(n), 64 + np.arange(n)] / 1024 - way * want)
                lim = 2 * np.pi * (2.0 ** -32 + 2.0 ** -33) + (2.0 ** -11 + 2.0 ** -22) * np.abs(want) + 2.0 ** -35
                assert (err <= lim).all(), (freq[err > lim].tolist(), err[err > lim].tolist(), lim[err > lim].tolist())
    finally:
        s.close()


@pytest.mark.parametrize("n_axes", [2, 3, 4])
@pytest.mark.parametrize("interleaved", [False, True])
def test_several_axes(n_axes, interleaved):
    rng = np.random.default_rng(n_axes)
    for D in (72, 80, 128):
        axis = rng.integers(0, n_axes, D // 2)
        run(13, dict(D=D), pos=rng.integers(0, 4000, (n_axes, 13)), axis=axis, n_axes=n_axes, interleaved=interleaved)
    run(13, dict(D=64), axis=rng.integers(0, n_axes, 32), n_axes=n_axes)  # the step's positions on every axis


def test_scale_and_one_norm_alone():
    run(5, rot=32, scale=1.3)
    run(5, q_gain=np.full(64, 2.0))
    run(5, k_gain=np.full(64, 2.0), eps=0.0)
    run(5, dict(scale=1e-4), q_gain=np.ones(64), k_gain=np.ones(64), eps=1e-6)  # eps counts as much as the squares do


def test_gains_on_the_device_and_a_rotation_set_again():
    import torch
    s = Rope(6, L=3)
    try:
        s.compare(q_gain=torch.full((64,), 1.5, device="cuda"), k_gain=torch.arange(64, dtype=torch.float32, device="cuda"))
        s.cache.fill_(float("nan"))
        s.out.fill_(float("nan"))
        s.compare(rot=16, interleaved=True)
        s.out.fill_(float("nan"))
        s.compare(layer=2, rot=8)
    finally:
        s.close()


@pytest.mark.parametrize("kind", [dict(), dict(rot=32), dict(interleaved=True)], ids=str)
def test_in_place(kind):
    s = Rope(11, D=72)
    try:
        s.compare(q_out=s.q, q_gain=np.ones(72), **kind)
    finally:
        s.close()


def test_what_is_not_turned_stays_as_it_is():
    """Infinities and NaN beside the turned elements, without a norm."""
    import torch
    for interleaved in (False, True):
        s = Rope(4, D=128)
        try:
            s.q[:, :, 70] = float("inf")
            s.k[:, :, 127] = float("-inf")
            s.k[:, :, 100] = float("nan")
            s.v[:, :, 3] = float("nan")
            s.pw.pw_attn_set_rope(s.attn, 0, freqs(64), interleaved=interleaved)
            torch.cuda.synchronize()
            s.pw.pw_attn_rope_append(s.attn, 0, s.step, s.q, s.out[:, :, 0], s.k, s.v)
            torch.cuda.synchronize()
            held = s.cache[0].reshape(2, -1, 2, 128)[:, s.slot]
            assert torch.equal(s.out[:, :, 0, 64:], s.q[:, :, 64:])
            assert torch.equal(held[0][..., 64:].nan_to_num(nan=7.0), s.k[..., 64:].nan_to_num(nan=7.0))
            assert torch.equal(held[1].nan_to_num(nan=7.0), s.v.nan_to_num(nan=7.0))
            assert bool(torch.isfinite(s.out[:, :, 0, :64]).all() and torch.isfinite(held[0][..., :64]).all())
        finally:
            s.close()


def test_a_rotation_holds_for_every_stream_once_it_is_set():
    """Launches on a stream that waits for no other, right behind pw_attn_set_rope."""
    import torch
    s = Rope(300, D=128)
    stream = torch.cuda.Stream()
    gain = np.random.default_rng(0).normal(1, 0.2, (12, 128))
    torch.cuda.synchronize()
    try:
        for k in range(12):
            s.pw.pw_attn_set_rope(s.attn, 0, freqs(128) * (k + 1), q_gain=gain[k], k_gain=gain[k])
            s.pw.pw_attn_rope_append(s.attn, 0, s.step, s.q, s.out[:, :, 0], s.k, s.v, stream=stream)
            torch.cuda.synchronize()
            got, held = s.out[:, :, 0].clone(), s.cache[0].clone()
            torch.cuda.synchronize()
            s.pw.pw_attn_rope_append(s.attn, 0, s.step, s.q, s.out[:, :, 0], s.k, s.v, stream=stream)
            torch.cuda.synchronize()
            assert torch.equal(got, s.out[:, :, 0])
            assert torch.equal(held.nan_to_num(nan=7.0), s.cache[0].nan_to_num(nan=7.0))
    finally:
        s.close()


def test_a_captured_call_on_a_stream_of_its_own():
    import torch
    s = Rope(10, D=128)
    try:
        s.pw.pw_attn_set_rope(s.attn, 0, freqs(128))
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            s.pw.pw_attn_rope_append(s.attn, 0, s.step, s.q, s.out[:, :, 0], s.k, s.v, stream=stream)
        assert bool(torch.isnan(s.out.float()).all())
        for k in range(2):
            s.pos.add_(17)
            graph.replay()
            torch.cuda.synchronize()
            got, held = s.out[:, :, 0].clone(), s.cache[0].clone()
            s.pw.pw_attn_rope_append(s.attn, 0, s.step, s.q, s.out[:, :, 0], s.k, s.v)
            torch.cuda.synchronize()
            assert torch.equal(got, s.out[:, :, 0])
            assert torch.equal(held.nan_to_num(nan=7.0), s.cache[0].nan_to_num(nan=7.0))
    finally:
        s.close()


def test_refusals():
    import torch
    s = Rope(3, L=2, D=72)
    pw = s.pw
    try:
        def call(layer=0, **kw):
            a = dict(q=s.q, q_out=s.out[:, :, 0], k=s.k, v=s.v, pos=None)
            a.update(kw)
            pw.pw_attn_rope_append(s.attn, layer, s.step, a["q"], a["q_out"], a["k"], a["v"], pos=a["pos"])
        with pytest.raises(pw.PwError) as e:
            call()
        assert e.value.status == pw.PW_ERR_STATE
        for kw in (dict(inv_freq=freqs(10)), dict(inv_freq=freqs(80)), dict(inv_freq=[np.inf] * 4), dict(inv_freq=[np.nan] * 4),
                   dict(n_axes=0), dict(n_axes=5), dict(axis=[1] * 36), dict(axis=[-1] * 36), dict(scale=np.inf), dict(eps=-1.0),
                   dict(eps=np.nan), dict(layer=2), dict(layer=-1)):
            with pytest.raises(pw.PwError) as e:
                pw.pw_attn_set_rope(s.attn, **{**dict(layer=0, inv_freq=freqs(72)), **kw})
            assert e.value.status == pw.PW_ERR_INVALID, kw
        for kw in (dict(axis=[0] * 3), dict(q_gain=np.ones(71)), dict(k_gain=torch.ones(71, device="cuda")),
                   dict(q_gain=torch.ones(72, device="cuda", dtype=torch.float64))):
            with pytest.raises(ValueError):
                pw.pw_attn_set_rope(s.attn, **{**dict(layer=0, inv_freq=freqs(72)), **kw})
        pw.pw_attn_set_rope(s.attn, 0, freqs(72), n_axes=3, axis=[2] * 36)
        one = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
        for kw in (dict(q=s.k), dict(k=s.q), dict(q_out=s.out[:, :, 0].half()), dict(v=s.v.cpu()), dict(pos=one(8)), dict(q=s.q[:2])):
            with pytest.raises(ValueError):
                call(**kw)
        flat = torch.zeros(4000, dtype=s.dt, device="cuda")
        with pytest.raises(pw.PwError):  # strides and addresses of whole 16-byte pieces
            call(q=flat.as_strided((3, 4, 72), (292, 73, 1)))
        with pytest.raises(pw.PwError):
            call(q=flat[1:].as_strided((3, 4, 72), (320, 80, 1)))
        with pytest.raises(pw.PwError) as e:
            call(layer=1)
        assert e.value.status == pw.PW_ERR_STATE
        call(pos=one(9))
        torch.cuda.synchronize()
    finally:
        s.close()
