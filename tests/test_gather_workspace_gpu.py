"""The gather products in a workspace made for more rows, or of just the size asked for."""
import numpy as np
import pytest
import torch

import combine_moe_route_topk_amd as moe
from tests.gpu_util import DEV, to_dev
from tests.test_int4_gpu import BF16, F32, _bits, _case, _check, _dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,e", [((16385, 16384, 100, 3), 1024), ((700, 640), 5)])
def test_int4_products_of_fewer_rows(rows, e):
    size = moe.moe_gather_gemm_int4_workspace_bytes(rows[0], e)
    buf = torch.full((size + 4096,), 255, dtype=torch.uint8, device=DEV)
    for r in rows:
        case = _case(r, e, 32, 4, 32)
        x, ex, w, _ = case
        y = moe.moe_gather_gemm_int4(to_dev(_bits(x)), to_dev(ex), *_dev(w, BF16), out_dtype=F32, workspace=buf[:size])
        _check(y, case, F32)
        assert (buf[size:] == 255).all()


def test_mxfp4_products_of_fewer_rows():
    e, n, k, most = 1024, 32, 128, 16385
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    x = torch.randn((most, k), generator=g, device=DEV).to(BF16)
    ex = torch.randint(0, e, (most,), generator=g, device=DEV, dtype=torch.int32)
    q, s = moe.moe_quantize_mxfp4(x)
    w, ws = [t.view(e, n, -1) for t in moe.moe_quantize_mxfp4(torch.randn((e * n, k), generator=g, device=DEV).to(BF16))]
    size = moe.moe_gather_gemm_mxfp4_workspace_bytes(most, e)
    buf = torch.full((size + 4096,), 255, dtype=torch.uint8, device=DEV)
    for r in (most, most - 1):
        args = (q[:r], s[:r], ex[:r], w, ws)
        assert torch.equal(moe.moe_gather_gemm_mxfp4(*args, workspace=buf[:size]), moe.moe_gather_gemm_mxfp4(*args))
        assert (buf[size:] == 255).all()
