"""examples/draft_steps.py: rotation, trees, kept paths, forked, trimmed and compacted blocks, as a server calls them."""
import os
import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def draft():
    from any_precision_bit_gb300 import _build
    _build.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import draft_steps
    return draft_steps


def test_runs_and_repeats(draft):
    import torch
    a, b = draft.main(), draft.main()
    assert a[0] == b[0] and a[2] == b[2] and a[3] == b[3] > 0
    assert max(a[2]) > 1  # some draft was accepted: paths were moved
    for r in a[0]:
        assert len(a[1][r]) == len(a[0][r]) - 1
        assert all(torch.equal(x, y) for x, y in zip(a[1][r], b[1][r]))


@pytest.mark.parametrize("seed", [0, 1])
def test_every_kept_token_is_the_prompt_of_all_tokens(draft, seed):
    """The hidden states of all kept tokens, whatever trees, forks and moves brought them about, are those of the same
    tokens as one prompt: within the rounding of two bf16 layers (3 %, of which a step that sums in another order uses
    a part), and far from what a wrong key, position or block would leave of them (a key less changes a row by 1 / sqrt(its
    keys) of the attention's part)."""
    import torch
    tokens, seen, _, _ = draft.main(seed=seed)
    for r in tokens:
        s = draft.Server(max_requests=1, max_tokens=256, n_blocks=32, seed=seed)
        s.admit(9, tokens[r][:-1])
        want, got = torch.stack(s.seen[9]), torch.stack(seen[r])
        s.close()
        err = (got - want).norm(dim=1) / want.norm(dim=1)
        assert got.shape == want.shape and err.max() < 0.03, (r, float(err.max()), int(err.argmax()))
