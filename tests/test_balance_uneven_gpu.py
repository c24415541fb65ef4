"""Balance loss of packed batches whose sequences differ widely: one long among many short or
empty ones, and offsets padded to a fixed number of sequences.

Tolerances as in test_balance_gpu: chunks are 16 tokens or fewer here, one to a team, and the
longest sequence has 1500 slots: 1 + 16 + 47 + 32 + 16 additions, below the 150 allowed there."""
import numpy as np
import pytest
import torch

import combine_moe_route_topk_amd as moe
from tests.gpu_util import DEV, to_dev, to_np
from tests.test_balance_gpu import _check_backward, _check_forward, _inputs, _run

pytestmark = pytest.mark.gpu


def _layout(kind, n, b, rng):
    short = rng.integers(0, 4, b)
    if kind == "long first":
        short[0] = n - short[1:].sum()
    elif kind == "long inside":
        short[b // 2] = n - short.sum() + short[b // 2]
    elif kind == "empty before the last tokens":
        short[:] = 0
        short[0], short[-1] = n - 9, 9
    elif kind == "padded behind, tokens left over":       # offsets repeat a value below n
        short[:] = 0
        short[:3] = (n - 50) // 4, (n - 50) // 4, (n - 50) // 2
    elif kind == "padded behind":
        short[:] = 0
        short[:2] = n - 100, 100
    elif kind == "all empty":
        short[:] = 0
        return np.concatenate([[n // 2], n // 2 + np.cumsum(short)]).astype(np.int32)
    return np.concatenate([[0], np.cumsum(short)]).astype(np.int32)


KINDS = ["long first", "long inside", "empty before the last tokens", "padded behind, tokens left over",
         "padded behind", "all empty"]


# few sequences: the sums of 32 experts each meet by a ticket; many: a workgroup takes all
# experts of a sequence; with 1500 of them chunks are 6 tokens
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,e,b", [(9000, 96, 5), (9000, 97, 260), (9000, 96, 260), (9000, 64, 1500), (500, 1000, 130)])
def test_uneven_sequences(n, e, b, kind):
    k = 4
    rng, logits, idx = _inputs(n, e, k, n + b)
    offs = _layout(kind, n, b, rng)
    assert offs.size == b + 1 and (np.diff(offs) >= 0).all() and 0 <= offs[-1] <= n
    mask = rng.random(n) < 0.9
    for m in (None, mask):
        got = _run(logits, idx, offs, m)
        want = _check_forward(got, logits, idx, offs, m)
        assert want["tokens"].sum() == (offs[-1] - offs[0] if m is None else m[offs[0]:offs[-1]].sum())
    again = _run(logits, idx, offs, mask)
    for name in ("loss", "z_loss", "counts", "probs", "tokens"):
        assert torch.equal(getattr(got, name), getattr(again, name)), name
    dl, dz = rng.standard_normal(b).astype(np.float32), rng.standard_normal(b).astype(np.float32)
    out = torch.full((n, e), 7.0, device=DEV)
    moe.moe_balance_loss_backward(to_dev(logits), got.counts, got.tokens, k, to_dev(dl), to_dev(dz),
                                  seq_offsets=to_dev(offs), token_mask=to_dev(mask), d_logits=out)
    _check_backward(out, logits, want["counts"], want["tokens"], k, dl, dz, offs, mask)
    outside = np.ones(n, bool)
    outside[offs[0]:offs[-1]] = False
    assert (to_np(out)[outside] == 0).all()


def test_two_calls_at_once():
    """Two streams, each with its own workspace."""
    sets = []
    for n, e, b in ((5000, 256, 20), (3000, 64, 500)):
        rng, logits, idx = _inputs(n, e, 4, n)
        sets.append((to_dev(logits), to_dev(idx), to_dev(_layout("long inside", n, b, rng))))
    want = [moe.moe_balance_loss(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[moe.moe_balance_loss(*s, stream=st) for s, st in zip(sets, streams)] for _ in range(3)]
    torch.cuda.synchronize()
    for turn in got:
        for g, w in zip(turn, want):
            for name in ("loss", "z_loss", "counts", "probs", "tokens"):
                assert torch.equal(getattr(g, name), getattr(w, name)), name
