"""pw_attn_create's checks of its shapes (no GPU is touched)."""
import pytest

pw = pytest.importorskip("any_precision_bit_gb300")


@pytest.fixture(scope="module", autouse=True)
def built():
    from any_precision_bit_gb300 import _build
    _build.build()


GOOD = dict(L=1, n_heads=4, n_kv_heads=2, head_dim=64, dtype=0, n_blocks=10, block_tokens=16, max_requests=2,
            max_tokens=8, max_shared_tokens=0, n_plans=1, device=0)


@pytest.mark.parametrize("change", [
    dict(L=0), dict(n_heads=5), dict(n_heads=0, n_kv_heads=0), dict(n_heads=258, n_kv_heads=2), dict(head_dim=0),
    dict(head_dim=12), dict(head_dim=136), dict(dtype=2), dict(n_blocks=0), dict(block_tokens=8),
    dict(block_tokens=48), dict(max_requests=0), dict(max_requests=4097), dict(max_tokens=0),
    dict(max_tokens=(1 << 20) + 1), dict(max_shared_tokens=9), dict(max_shared_tokens=-1), dict(n_plans=0),
    dict(n_plans=17)], ids=str)
def test_create_refuses(change):
    with pytest.raises(pw.PwError) as e:
        pw.pw_attn_create(pw.pw_attn_desc(**{**GOOD, **change}))
    assert e.value.status == pw.PW_ERR_INVALID and str(e.value)
