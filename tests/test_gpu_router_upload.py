"""A router that was just set is the one that the next forward uses, whatever stream it runs on."""
import numpy as np
import pytest

import synthetic as syn

from gpu_helpers import LayerData, make_ctx

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
pw = pytest.importorskip("any_precision_bit_gb300")


@pytest.mark.parametrize("where", ["host", "device"])
def test_forwards_right_behind_a_router_that_is_set_again(where):
    from any_precision_bit_gb300 import _build
    _build.build()
    shape = syn.SHAPES["tiny"]
    T = shape.decode_T[0]
    data = LayerData(shape, 3, 0, T, tiny=True)
    ctx = make_ctx(pw, shape, max_tokens=T)
    rng = np.random.default_rng(0)
    try:
        data.load(pw, ctx)
        x = torch.from_numpy(data.x.view(np.int16)).cuda()
        ids, again = (torch.zeros((T, shape.K), dtype=torch.int32, device="cuda") for _ in range(2))
        y, stream = torch.zeros_like(x), torch.cuda.Stream()
        torch.cuda.synchronize()
        for _ in range(8):
            Wr, bias = data.Wr[rng.permutation(shape.E)].copy(), data.bias
            if where == "device":
                Wr = torch.from_numpy(Wr).cuda()
            pw.pw_set_router(ctx, 0, Wr, bias)
            pw.pw_moe_forward(ctx, 0, x, T, y, ids, None, 0, stream.cuda_stream)
            torch.cuda.synchronize()
            pw.pw_moe_forward(ctx, 0, x, T, y, again, None, 0, stream.cuda_stream)
            torch.cuda.synchronize()
            assert torch.equal(ids, again)
    finally:
        pw.pw_destroy(ctx)
