"""moe_balance_loss in a workspace made for a larger batch, or of just the size asked for."""
import numpy as np
import pytest
import torch

import combine_moe_route_topk_amd as moe
from tests.gpu_util import DEV, to_dev
from tests.test_balance_gpu import _check_forward, _inputs

pytestmark = pytest.mark.gpu
NAMES = ("loss", "z_loss", "counts", "probs", "tokens")


def _even(n, b):
    return None if b == 1 else np.linspace(0, n, b + 1).astype(np.int32)


@pytest.mark.parametrize("most,less,e", [((20000, 1), (16384, 1), 64), ((4096, 2048), (4095, 2048), 60),
                                         ((2500, 40), (2339, 20), 256), ((1000, 700), (999, 500), 16)])
def test_smaller_batches_in_the_workspace_of_the_largest(most, less, e):
    ws = torch.empty(moe.moe_balance_loss_workspace_bytes(most[0], e, most[1]), dtype=torch.uint8, device=DEV)
    for n, b in (most, less, (17, 2)):
        rng, logits, idx = _inputs(n, e, 2, n)
        offs = _even(n, b)
        ws.fill_(255)
        got = moe.moe_balance_loss(to_dev(logits), to_dev(idx), None if offs is None else to_dev(offs), workspace=ws)
        _check_forward(got, logits, idx, offs, None)


@pytest.mark.parametrize("n,e,b", [(300, 7, 1), (4095, 60, 2048), (1999, 8, 1000), (2339, 256, 20), (5, 16, 900)])
def test_nothing_is_written_behind_the_workspace(n, e, b):
    size = moe.moe_balance_loss_workspace_bytes(n, e, b)
    buf = torch.full((size + 4096,), 255, dtype=torch.uint8, device=DEV)
    rng, logits, idx = _inputs(n, e, 2, n)
    offs = _even(n, b)
    args = (to_dev(logits), to_dev(idx), None if offs is None else to_dev(offs))
    got = moe.moe_balance_loss(*args, workspace=buf[:size])
    assert (buf[size:] == 255).all()
    want = moe.moe_balance_loss(*args)
    for name in NAMES:
        assert torch.equal(getattr(got, name), getattr(want, name)), name
