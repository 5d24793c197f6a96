"""What may change between the calls of a step, and what is reported when it may not."""
import numpy as np
import pytest

from attn_helpers import Step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from any_precision_bit_gb300 import _build
    _build.build()


@pytest.mark.parametrize("new", [[1, 1, 1], [70, 4, 1]])
@pytest.mark.parametrize("groups", [False, True])
def test_a_block_moved_between_plan_and_forward(new, groups):
    """Copied to another block and its table entry changed, as a server does before it writes to a block that
    requests share: the forward reads the table as it is then, in every key tile alike."""
    kw = dict(group_start=[0, 3], prefix=64) if groups else {}
    s = Step([100, 400, 70], new, Hq=4, Hkv=2, D=64, **kw)
    s.map_and_append()
    s.pw.pw_attn_plan(s.attn, 0, s.step)
    before = s.forward()
    # the first block of every request (of the group) to a block that nobody has
    used = set(int(b) for b in s.table.cpu().numpy().ravel())
    spare = [b for b in range(s.n_blocks) if b not in used]
    if groups:
        spare = spare[:1] * 3
    for r, to in zip(range(3), spare):
        at = int(s.table[r, 0])
        for c in s.kv:
            c[to] = c[at]
    for r, to in zip(range(3), spare):
        at = int(s.table[r, 0])
        for c in s.kv:
            if at not in spare:
                c[at] = float("nan")
        s.table[r, 0] = to
    o = s.torch.empty(s.N, s.Hq, s.D, dtype=s.dt, device="cuda")
    s.torch.cuda.synchronize()
    s.pw.pw_attn_forward(s.attn, 0, 0, s.q, o)
    s.pw.pw_attn_check(s.attn)
    assert np.array_equal(o.float().cpu().numpy(), before[0])
    s.close()
