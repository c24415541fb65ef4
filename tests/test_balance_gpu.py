"""Balance loss, per-expert counts and their gradient against the float64 oracle.

Tolerances, with u = 2^-24 (half an fp32 step).  A probability p = exp(l - m) / S:
the difference errs by u |l - m|, the exponential by 2 u (one step), S by one
rounding per addition (at most 16 in a lane and 6 between lanes) on top of its
terms' errors, and reciprocal and product by 3 u: within (2 D + 40) u relatively,
D the largest finite |l - m| that matters (terms below exp(-88) are below 2^-126
and are allowed as an absolute error).  Sums over tokens add at most one rounding
per addition along the longest chain: 64 tokens in a team, 16 teams, 16 slots in a
thread, 32 rows, 16 roundings of the scaling: 150 u.  All terms are positive, so
probs and loss are within R = (2 D + 40 + 150 + E / 8) u, E / 8 for the sum over
experts (32 in a lane and 8 parts, generously).
log-sum-exp: S within (D + 40) u gives that absolutely, the logarithm one step of
its value, the sum one rounding: delta = u (D + 44 + 2 log E + 2 |m|);
z within mean(2 |lse| delta + delta^2) + 150 u z.
The gradient p (u_e - sum p u + f lse): u_e errs by 5 u, the dot product by
(R + 24 u) sum p |u|, the rest by a rounding each:
    p (R + 64 u) (|u_e| + sum p |u| + |f| |lse|) + p |f| delta.
"""
import numpy as np
import pytest
import torch

import combine_moe_route_topk_amd as moe
from oracle.balance import balance, balance_backward, softmax
from tests.gpu_util import DEV, to_dev, to_np

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _errors(logits):
    p, lse, live = softmax(logits)
    with np.errstate(invalid="ignore"):
        top = np.where(np.isfinite(logits.max(1)), logits.max(1), 0.0)
        gap = np.where(np.isfinite(logits), top[:, None] - logits, 0.0)
    d = float(np.minimum(gap, 90.0).max(initial=0.0))
    e = logits.shape[1]
    r = (2 * d + 190 + e / 8) * U
    delta = U * (d + 44 + 2 * np.log(e) + 2 * np.abs(top))
    return p, lse, live, r, delta


def _check_forward(got, logits, idx, offs, mask):
    want = balance(logits, idx, offs, mask)
    p, lse, live, r, delta = _errors(logits)
    assert np.array_equal(to_np(got.counts), want["counts"])
    assert np.array_equal(to_np(got.tokens), want["tokens"])
    tiny = 2.0 ** -126
    assert (np.abs(to_np(got.probs) - want["probs"]) <= r * want["probs"] + tiny).all()
    assert (np.abs(to_np(got.loss) - want["loss"]) <= r * want["loss"] + tiny).all()
    keep = live if mask is None else live & mask.astype(bool)
    lim = float((2 * np.abs(lse[keep]) * delta[keep] + delta[keep] ** 2).max(initial=0.0))   # a mean is below the largest
    assert (np.abs(to_np(got.z_loss) - want["z_loss"]) <= lim + 150 * U * want["z_loss"]).all()
    return want


def _check_backward(got, logits, counts, tokens, k, dl, dz, offs, mask):
    want = balance_backward(logits, counts, tokens, k, dl, dz, offs, mask)
    n, e = logits.shape
    p, lse, live, r, delta = _errors(logits)
    seqs = [0, n] if offs is None else list(offs)
    bound = np.zeros((n, e))
    for b, (lo, hi) in enumerate(zip(seqs[:-1], seqs[1:])):
        m = max(int(tokens[b]), 1)
        u = dl[b] * (e * np.asarray(counts[b], np.float64) - k * m) / (k * float(m) ** 2)
        f = abs(2.0 * dz[b] / m)
        q = p[lo:hi]
        with np.errstate(invalid="ignore"):
            z = np.where(live[lo:hi], np.abs(lse[lo:hi]), 0.0)
        size = np.abs(u) + (q * np.abs(u)).sum(1, keepdims=True) + f * z[:, None]
        bound[lo:hi] = q * ((r + 64 * U) * size + f * delta[lo:hi, None])
    g = to_np(got)
    assert (np.abs(g - want) <= bound + 2.0 ** -126).all(), np.max(np.abs(g - want) - bound)
    return want


def _inputs(n, e, k, seed, spread=1.0):
    rng = np.random.default_rng(seed)
    logits = (rng.standard_normal((n, e)) * spread).astype(np.float32)
    idx = np.argsort(-logits, axis=1, kind="stable")[:, :k].astype(np.int32)
    return rng, logits, idx


def _offsets(kind, n, rng):
    if kind == "none":
        return None
    if kind == "whole":
        return np.array([0, n], np.int32)
    if kind == "ragged":                     # empty ones among them, rows before the first and behind the last
        cut = np.sort(rng.integers(0, n + 1, 7))
        return np.concatenate([cut[:3], cut[2:]]).astype(np.int32)
    # more sequences than tokens
    return np.sort(rng.integers(0, n + 1, 2 * n + 3)).astype(np.int32)


def _run(logits, idx, offs, mask):
    return moe.moe_balance_loss(to_dev(logits), to_dev(idx), seq_offsets=None if offs is None else to_dev(offs),
                                token_mask=None if mask is None else to_dev(mask))


SIZES = [(1, 1, 1), (1, 8, 2), (16, 8, 2), (63, 64, 8), (64, 65, 3), (65, 256, 8), (300, 60, 6), (1000, 256, 8),
         (517, 130, 1), (40, 512, 4), (33, 1000, 64), (200, 1024, 8), (2049, 128, 2), (9000, 7, 3)]


@pytest.mark.parametrize("kind", ["none", "whole", "ragged", "many"])
@pytest.mark.parametrize("n,e,k", SIZES)
def test_loss_counts_and_gradient(n, e, k, kind):
    rng, logits, idx = _inputs(n, e, k, n + e)
    offs = _offsets(kind, n, rng)
    for mask in (None, (rng.random(n) < 0.7).astype(np.uint8)):
        got = _run(logits, idx, offs, mask)
        want = _check_forward(got, logits, idx, offs, mask)
        b = want["loss"].size
        dl, dz = rng.standard_normal(b).astype(np.float32), rng.standard_normal(b).astype(np.float32)
        args = (to_dev(logits), got.counts, got.tokens, k, to_dev(dl))
        kw = dict(seq_offsets=None if offs is None else to_dev(offs), token_mask=None if mask is None else to_dev(mask))
        g = moe.moe_balance_loss_backward(*args, to_dev(dz), **kw)
        _check_backward(g, logits, want["counts"], want["tokens"], k, dl, dz, offs, mask)
        g0 = moe.moe_balance_loss_backward(*args, **kw)
        _check_backward(g0, logits, want["counts"], want["tokens"], k, dl, 0 * dz, offs, mask)
        # added to another gradient: one more rounding
        base = to_dev(rng.standard_normal((n, e)).astype(np.float32))
        acc = base.clone()
        assert moe.moe_balance_loss_backward(*args, to_dev(dz), **kw, d_logits=acc, accumulate=True) is acc
        assert torch.equal(acc, base + g)


def test_prefill_size_packed():
    n, e, k = 20011, 256, 8
    rng, logits, idx = _inputs(n, e, k, 5)
    offs = np.sort(rng.integers(0, n + 1, 30)).astype(np.int32)
    mask = rng.random(n) < 0.9
    got = _run(logits, idx, offs, mask)
    want = _check_forward(got, logits, idx, offs, mask)
    again = _run(logits, idx, offs, mask)
    for name in ("loss", "z_loss", "counts", "probs", "tokens"):
        assert torch.equal(getattr(got, name), getattr(again, name))       # the same bits every time
    dl = np.full(29, 0.01, np.float32)
    g = moe.moe_balance_loss_backward(to_dev(logits), got.counts, got.tokens, k, to_dev(dl), to_dev(dl),
                                      seq_offsets=to_dev(offs), token_mask=to_dev(mask))
    _check_backward(g, logits, want["counts"], want["tokens"], k, dl, dl, offs, mask)


def test_no_tokens():
    z = torch.zeros
    for offs in (None, z(4, dtype=torch.int32, device=DEV)):
        b = 1 if offs is None else 3
        out = moe.BalanceLoss(z(b, device=DEV) + 7, z(b, device=DEV) + 7, z((b, 8), dtype=torch.int32, device=DEV) + 7,
                              z((b, 8), device=DEV) + 7, z(b, dtype=torch.int32, device=DEV) + 7)
        r = moe.moe_balance_loss(z((0, 8), device=DEV), z((0, 2), dtype=torch.int32, device=DEV), offs, out=out)
        for t in (r.loss, r.z_loss, r.counts, r.probs, r.tokens):
            assert (t == 0).all()
        g = moe.moe_balance_loss_backward(z((0, 8), device=DEV), r.counts, r.tokens, 2, r.loss, seq_offsets=offs)
        assert g.shape == (0, 8)


@pytest.mark.parametrize("n", [40, 700])
def test_everything_masked_and_empty_rows(n):
    rng, logits, idx = _inputs(n, 60, 4, n)
    dl = np.ones(1, np.float32)
    r = _run(logits, idx, None, np.zeros(n, np.uint8))
    for t in (r.loss, r.z_loss, r.counts, r.probs, r.tokens):
        assert (t == 0).all()
    g = moe.moe_balance_loss_backward(to_dev(logits), r.counts, r.tokens, 4, to_dev(dl), to_dev(dl),
                                      token_mask=to_dev(np.zeros(n, np.uint8)))
    assert (g == 0).all()
    # masked experts, rows whose experts are all masked, and the type's lowest value instead
    logits[:, 5] = -np.inf
    logits[3::7] = -np.inf
    logits[4, :] = np.finfo(np.float32).min / 8
    logits[5, 10:] = np.finfo(np.float32).min
    r = _run(logits, idx, None, None)
    live = (logits > -np.inf).any(1)
    assert int(r.tokens[0]) == live.sum()
    keep = live & (np.arange(n) != 4)        # the square of row 4's log-sum-exp overflows
    assert torch.isinf(r.z_loss[0])
    want = balance(logits, idx)
    assert np.array_equal(to_np(r.counts), want["counts"])
    assert np.allclose(to_np(r.probs), want["probs"], rtol=1e-5, atol=2.0 ** -126)
    r = _run(logits, idx, None, keep.astype(np.uint8))
    _check_forward(r, logits, idx, None, keep.astype(np.uint8))
    g = moe.moe_balance_loss_backward(to_dev(logits), r.counts, r.tokens, 4, to_dev(dl), to_dev(dl),
                                      token_mask=to_dev(keep.astype(np.uint8)))
    w = _check_backward(g, logits, to_np(r.counts), to_np(r.tokens), 4, dl, dl, None, keep.astype(np.uint8))
    assert (to_np(g)[~keep] == 0).all() and (w[~keep] == 0).all() and (to_np(g)[:, 5] == 0).all()


def test_nan_and_infinity_stay_in_their_sequence_and_row():
    n, e, k = 600, 64, 2
    rng, logits, idx = _inputs(n, e, k, 9)
    offs = np.array([0, 100, 350, 600], np.int32)
    clean = _run(logits, idx, offs, None)
    bad = logits.copy()
    bad[120, 7], bad[130, 9] = np.nan, np.inf
    got = _run(bad, idx, offs, None)
    assert torch.equal(got.counts, clean.counts) and torch.equal(got.tokens, clean.tokens)
    for name in ("loss", "z_loss", "probs"):
        a, b = getattr(got, name), getattr(clean, name)
        assert torch.isnan(a[1]).all() and torch.equal(a[[0, 2]], b[[0, 2]]), name
    # in masked places they do nothing
    mask = np.ones(n, np.uint8)
    mask[[120, 130]] = 0
    want = _run(logits, idx, offs, mask)
    got = _run(bad, idx, offs, mask)
    for name in ("loss", "z_loss", "counts", "probs", "tokens"):
        assert torch.equal(getattr(got, name), getattr(want, name)), name
    dl = to_dev(np.ones(3, np.float32))
    kw = dict(seq_offsets=to_dev(offs))
    a = moe.moe_balance_loss_backward(to_dev(bad), clean.counts, clean.tokens, k, dl, dl, **kw)
    b = moe.moe_balance_loss_backward(to_dev(logits), clean.counts, clean.tokens, k, dl, dl, **kw)
    rows = np.ones(n, bool)
    rows[[120, 130]] = False
    assert torch.isnan(a[[120, 130]]).all() and torch.equal(a[to_dev(rows)], b[to_dev(rows)])


def test_dropped_and_repeated_ids():
    n, e, k = 500, 16, 4
    rng, logits, idx = _inputs(n, e, k, 3)
    idx[::3, 1] = -1
    idx[1::5, 2] = e
    idx[2::5, 0] = 2**31 - 1
    idx[:, 3] = idx[:, 1]                    # an id twice in a row
    for m in (n, 37):
        _check_forward(_run(logits[:m], idx[:m], None, None), logits[:m], idx[:m], None, None)


def test_offsets_that_run_over_read_nothing_outside():
    """Offsets past the tokens, negative or falling: no fault, the counts stay within the tokens."""
    rng, logits, idx = _inputs(300, 8, 2, 1)
    for offs in ([-5, 100, 4000], [200, 100, 300], [2**31 - 1, -2**31, 7], [-9, -3, -1], [400, 500, 600]):
        r = _run(logits, idx, np.array(offs, np.int64).astype(np.int32), None)
        moe.moe_balance_loss_backward(to_dev(logits), r.counts.clamp(0, 10), r.tokens.clamp(0, 10), 2, r.loss,
                                      seq_offsets=to_dev(np.array(offs, np.int64).astype(np.int32)))
        torch.cuda.synchronize()
    r = _run(logits, idx, np.array([-5, 100, 4000], np.int32), None)
    _check_forward(r, logits, idx, np.array([0, 100, 300]), None)


@pytest.mark.parametrize("e", [8, 64, 256, 512])
def test_logits_off_a_16_byte_boundary(e):
    n, k = 77, 2
    rng, logits, idx = _inputs(n, e, k, e)
    for shift in (1, 2, 3):
        flat = torch.empty(n * e + shift, device=DEV)
        view = flat[shift:].view(n, e)
        view.copy_(to_dev(logits))
        r = moe.moe_balance_loss(view, to_dev(idx))
        _check_forward(r, logits, idx, None, None)
        out = torch.full((n * e + shift + 5,), 7.0, device=DEV)
        dl = np.ones(1, np.float32)
        moe.moe_balance_loss_backward(view, r.counts, r.tokens, k, to_dev(dl), d_logits=out[shift:-5].view(n, e))
        _check_backward(out[shift:-5].view(n, e), logits, to_np(r.counts), to_np(r.tokens), k, dl, 0 * dl, None, None)
        assert (out[:shift] == 7).all() and (out[-5:] == 7).all()


@pytest.mark.parametrize("n", [40, 1500])
def test_stable_at_large_logits(n):
    rng, logits, idx = _inputs(n, 60, 4, n, spread=30.0)
    logits += np.float32(500.0)
    r = _run(logits, idx, None, None)
    w = _check_forward(r, logits, idx, None, None)
    dl = np.ones(1, np.float32)
    g = moe.moe_balance_loss_backward(to_dev(logits), r.counts, r.tokens, 4, to_dev(dl), to_dev(dl))
    _check_backward(g, logits, w["counts"], w["tokens"], 4, dl, dl, None, None)


def test_parts_of_a_batch():
    """Counts and tokens summed over two parts: their gradients are the whole's rows."""
    n, e, k = 900, 64, 4
    rng, logits, idx = _inputs(n, e, k, 4)
    dl = to_dev(np.array([0.5], np.float32))
    parts = [slice(0, 333), slice(333, 900)]
    rs = [_run(logits[s], idx[s], None, None) for s in parts]
    counts, tokens = rs[0].counts + rs[1].counts, rs[0].tokens + rs[1].tokens
    whole = _run(logits, idx, None, None)
    assert torch.equal(counts, whole.counts) and torch.equal(tokens, whole.tokens)
    g = moe.moe_balance_loss_backward(to_dev(logits), counts, tokens, k, dl, dl)
    for s in parts:
        assert torch.equal(moe.moe_balance_loss_backward(to_dev(logits[s]), counts, tokens, k, dl, dl), g[s])


def test_gradient_against_differences_of_the_loss():
    """The kernel's own loss along random directions, the ids held: d/dh L(l + h v).
    fp32 losses of about 1.2 leave 2^-23 / h of noise in the quotient, the third
    derivative h^2: with h = 2^-6 they are 2^-17 and about 2^-12."""
    n, e, k = 30, 12, 2
    rng, logits, idx = _inputs(n, e, k, 8)
    r = _run(logits, idx, None, None)
    one = to_dev(np.ones(1, np.float32))
    g = to_np(moe.moe_balance_loss_backward(to_dev(logits), r.counts, r.tokens, k, one)).astype(np.float64)
    h = 2.0 ** -6
    for _ in range(5):
        v = rng.standard_normal((n, e)).astype(np.float32)
        hi, lo = (_run((logits + s * np.float32(h) * v).astype(np.float32), idx, None, None) for s in (1, -1))
        assert float(hi.loss - lo.loss) / (2 * h) == pytest.approx((g * v).sum(), abs=2.0 ** -11)


def test_graph_replays_and_shared_workspace():
    """Two captured calls that share a workspace, on inputs that change between
    replays, with eager work in between."""
    shapes = [(700, 256, 8, 5), (50, 60, 4, 1)]
    ws = torch.empty(max(moe.moe_balance_loss_workspace_bytes(n, e, b) for n, e, k, b in shapes),
                     dtype=torch.uint8, device=DEV)
    sets, graphs = [], []
    for n, e, k, b in shapes:
        rng, logits, idx = _inputs(n, e, k, n)
        offs = None if b == 1 else to_dev(np.sort(rng.integers(0, n + 1, b + 1)).astype(np.int32))
        s = dict(l=to_dev(logits), i=to_dev(idx), o=offs, k=k, dl=torch.ones(b, device=DEV), g=torch.empty((n, e), device=DEV))
        s["out"] = moe.moe_balance_loss(s["l"], s["i"], offs, workspace=ws)
        sets.append(s)
    torch.cuda.synchronize()

    def step(s):
        moe.moe_balance_loss(s["l"], s["i"], s["o"], out=s["out"], workspace=ws)
        moe.moe_balance_loss_backward(s["l"], s["out"].counts, s["out"].tokens, s["k"], s["dl"], s["dl"],
                                      seq_offsets=s["o"], d_logits=s["g"])

    for s in sets:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step(s)
        graphs.append(gr)
    for rep in range(4):
        for s, gr in zip(sets, graphs):
            s["l"].mul_(1.1)
            for t in (s["out"].loss, s["out"].counts, s["out"].probs, s["g"]):
                t.fill_(7)
            ws.fill_(255)
            gr.replay()
            got = [t.clone() for t in (s["out"].loss, s["out"].z_loss, s["out"].counts, s["out"].probs, s["out"].tokens, s["g"])]
            torch.cuda.synchronize()
            step(s)
            want = (s["out"].loss, s["out"].z_loss, s["out"].counts, s["out"].probs, s["out"].tokens, s["g"])
            for a, b in zip(got, want):
                assert torch.equal(a, b), rep


def test_on_another_stream():
    rng, logits, idx = _inputs(3000, 256, 8, 2)
    l, i = to_dev(logits), to_dev(idx)
    want = moe.moe_balance_loss(l, i)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for _ in range(3):
        got = moe.moe_balance_loss(l, i, stream=st)
        g = moe.moe_balance_loss_backward(l, got.counts, got.tokens, 8, want.loss, stream=st)
        st.synchronize()
        assert torch.equal(got.loss, want.loss) and torch.equal(got.counts, want.counts)
        assert torch.equal(g, moe.moe_balance_loss_backward(l, want.counts, want.tokens, 8, want.loss))


def test_refusals():
    l, i = torch.zeros((16, 8), device=DEV), torch.zeros((16, 2), dtype=torch.int32, device=DEV)
    offs = torch.tensor([0, 4, 16], dtype=torch.int32, device=DEV)
    r = moe.moe_balance_loss(l, i, offs)
    with pytest.raises(TypeError, match="logits"):
        moe.moe_balance_loss(l.bfloat16(), i)
    with pytest.raises(TypeError, match="topk_idx"):
        moe.moe_balance_loss(l, i.long())
    with pytest.raises(ValueError, match="topk_idx"):
        moe.moe_balance_loss(l, i[:15])
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_balance_loss(torch.zeros((8, 16), device=DEV).t(), i)
    with pytest.raises(ValueError, match="seq_offsets"):
        moe.moe_balance_loss(l, i, offs[:1])
    with pytest.raises(TypeError, match="seq_offsets"):
        moe.moe_balance_loss(l, i, offs.long())
    with pytest.raises(ValueError, match="token_mask"):
        moe.moe_balance_loss(l, i, token_mask=torch.ones(15, dtype=torch.bool, device=DEV))
    with pytest.raises(TypeError, match="token_mask"):
        moe.moe_balance_loss(l, i, token_mask=torch.ones(16, device=DEV))
    with pytest.raises(ValueError, match="out.loss"):
        moe.moe_balance_loss(l, i, out=r)                    # two sequences' outputs for one
    with pytest.raises(moe.MoeError, match="MOE_ERR_WORKSPACE"):
        moe.moe_balance_loss(l, i, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(moe.MoeError, match="k="):
        moe.moe_balance_loss(l, torch.zeros((16, 9), dtype=torch.int32, device=DEV))
    one = torch.ones(2, device=DEV)
    b = lambda **kw: moe.moe_balance_loss_backward(**{**dict(logits=l, counts=r.counts, tokens=r.tokens, k=2, d_loss=one,
                                                             seq_offsets=offs), **kw})
    b()
    with pytest.raises(ValueError, match="counts"):
        b(counts=r.counts[:1])
    with pytest.raises(ValueError, match="d_loss"):
        b(d_loss=one[:1])
    with pytest.raises(ValueError, match="d_z_loss"):
        b(d_z_loss=one[:1])
    with pytest.raises(ValueError, match="accumulate"):
        b(accumulate=True)
    with pytest.raises(ValueError, match="d_logits"):
        b(d_logits=torch.zeros((15, 8), device=DEV))
    with pytest.raises(moe.MoeError, match="k="):
        b(k=0)
