"""Expired waits of the serving kernels, without a fault: operands of one launch are withheld on
purpose; the launch must report the timeout, return, and leave the context usable."""
import time

import pytest
import torch

from dropless_mixture_experts_dmoe_b200 import binding as B

from test_few_gpu import make, outputs, run, same
from test_mx4_gpu import setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nth", [1, 2], ids=["first product", "second product"])
@pytest.mark.parametrize("shape", [(600, 256, 384, 8, 2, 0), (3000, 640, 256, 40, 6, 0),
                                   (300, 256, 1152, 8, 2, 0)],
                         ids=lambda s: "-".join(map(str, s)))
def test_mx4_forward_stalled_product(shape, nth):
    """Units in rounds and in shares, the second product with its rows resident and (ffn 1152)
    streamed.  Epilogue warps of the second product meet in pairs, which may not part where the
    waits expire."""
    dims, x, lg, w, bufs = setup(shape)
    y, y2 = torch.empty_like(x), torch.empty_like(x)
    B.dmoe_sparse_map(dims, lg, bufs.map, bufs.ws_map)
    B.dmoe_mx4_forward(dims, x, *w, bufs.map, y, bufs.ws)
    torch.cuda.synchronize()
    assert int(bufs.map.status.item()) == 0
    for _ in range(5):
        B.dmoe_debug_inject_stall(nth)
        t0 = time.time()
        B.dmoe_mx4_forward(dims, x, *w, bufs.map, y2, bufs.ws)
        torch.cuda.synchronize()
        assert time.time() - t0 < 10.0
        assert int(bufs.map.status.item()) == B.STATUS_TIMEOUT
        B.dmoe_sparse_map(dims, lg, bufs.map, bufs.ws_map)
        B.dmoe_mx4_forward(dims, x, *w, bufs.map, y2, bufs.ws)
        torch.cuda.synchronize()
        assert int(bufs.map.status.item()) == 0
        assert torch.equal(y.view(torch.int16), y2.view(torch.int16))


@pytest.mark.parametrize("nth", [1, 2], ids=["first product", "second product"])
@pytest.mark.parametrize("mx4", [False, True], ids=["bf16", "mx4"])
@pytest.mark.parametrize("shape", [(1, 1024, 512, 8, 2),     # routed in the products, few stages
                                   (3, 4096, 2048, 4, 2),    # rings that wrap
                                   (40, 2048, 1024, 16, 4),  # rows copied by four loading warps
                                   (128, 512, 2048, 3, 2)],  # many columns per expert
                         ids=lambda s: "-".join(map(str, s)))
def test_few_stalled_product(shape, mx4, nth):
    """Every multiplying warp's first wait expires; the loading warps stop and drain; y is whatever it
    is, the status says so, the next call is right."""
    d = make(shape, seed=41, mx4=mx4)
    bufs, yg = outputs(d)
    run(d, bufs, yg[:-1])
    torch.cuda.synchronize()
    assert int(bufs.status.item()) == 0
    for _ in range(3):
        bufs2, yg2 = outputs(d)
        torch.cuda.synchronize()
        B.dmoe_debug_inject_stall(nth)
        t0 = time.time()
        run(d, bufs2, yg2[:-1])
        torch.cuda.synchronize()
        assert time.time() - t0 < 10.0
        assert int(bufs2.status.item()) == B.STATUS_TIMEOUT
        assert (yg2[-1] == 7.0).all()
        assert torch.equal(bufs.top_experts, bufs2.top_experts)
        bufs2.status.zero_()
        run(d, bufs2, yg2[:-1])
        torch.cuda.synchronize()
        assert int(bufs2.status.item()) == 0
        assert same(yg, yg2)
