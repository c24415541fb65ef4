"""Balance loss and 4-bit integer operators where elements lie past 2^31 and 2^32: the last
rows against the oracle, or against the same rows alone."""
import numpy as np
import pytest
import torch

import combine_moe_route_topk_amd as moe
from tests.gpu_util import DEV, as_f32, to_dev, to_np
from tests.test_balance_gpu import _check_backward, _check_forward
from tests.test_int4_gpu import BF16, F32, _case, _check, _dev

pytestmark = pytest.mark.gpu


def test_balance_loss_of_two_billion_logits():
    n, e, k, last = (1 << 21) + 777, 1024, 2, 300
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    logits = torch.randn((n, e), generator=g, device=DEV)
    idx = torch.randint(0, e, (n, k), generator=g, device=DEV, dtype=torch.int32)
    offs = torch.tensor([0, n - last, n], dtype=torch.int32, device=DEV)
    got = moe.moe_balance_loss(logits, idx, offs)
    assert got.tokens.tolist() == [n - last, last]
    assert torch.equal(got.counts[0], torch.bincount(idx[:n - last].reshape(-1), minlength=e).int())
    hl, hi = to_np(logits[n - last:]), to_np(idx[n - last:])
    tail = moe.BalanceLoss(*(getattr(got, f)[1:] for f in ("loss", "z_loss", "counts", "probs", "tokens")))
    want = _check_forward(tail, hl, hi, None, None)
    dl, dz = np.array([0.0, 0.5], np.float32), np.array([0.0, -0.25], np.float32)
    d = moe.moe_balance_loss_backward(logits, got.counts, got.tokens, k, to_dev(dl), to_dev(dz), seq_offsets=offs)
    _check_backward(d[n - last:], hl, want["counts"], want["tokens"], k, dl[1:], dz[1:], None, None)
    assert not torch.any(d[n - last - 4096:n - last])


@pytest.mark.parametrize("affine", [False, True])
def test_quantising_four_billion_elements(affine):
    r, k = (1 << 18) + 5, 1 << 14                            # 2^32 + 81920 elements
    x = torch.empty((r, k), dtype=BF16, device=DEV)
    for r0 in range(0, r, 1 << 15):
        x[r0:r0 + (1 << 15)].normal_()
    c, s, b = moe.moe_quantize_int4(x, 128, affine=affine)
    v = moe.moe_dequant_int4(c, s, b)
    for rows in (slice(0, 9), slice((1 << 17) - 4, (1 << 17) + 4), slice(r - 9, r)):
        cs, ss, bs = moe.moe_quantize_int4(x[rows], 128, affine=affine)
        assert torch.equal(c[rows], cs) and torch.equal(s[rows], ss) and (not affine or torch.equal(b[rows], bs))
        assert torch.equal(v[rows], moe.moe_dequant_int4(cs, ss, bs))


def test_products_of_two_billion_elements_of_rows():
    r, e, k, n = (1 << 18) + 100, 3, 8192, 8                 # 2^31 + 819200 elements of x
    _, _, w, _ = _case(4, e, k, n, 128, True, BF16)
    x = torch.empty((r, k), dtype=BF16, device=DEV)
    for r0 in range(0, r, 1 << 15):
        x[r0:r0 + (1 << 15)].normal_()
    ex = (torch.arange(r, device=DEV) % e).int()
    y = moe.moe_gather_gemm_int4(x, ex, *_dev(w, BF16), out_dtype=F32)
    pick = torch.cat([torch.arange(0, 40), torch.arange(r - 150, r)]).to(DEV)
    _check(y[pick], (as_f32(to_np(x[pick])), to_np(ex[pick]), w, None), F32)


def test_products_into_four_billion_bytes_of_y():
    r, e, k, n = 70000, 2, 32, 16001                         # 1.12e9 elements of y, 4.48 GB
    case = _case(r, e, k, n, 32, False, BF16)
    y = moe.moe_gather_gemm_int4(to_dev(np.ascontiguousarray(case[0])).to(BF16), to_dev(case[1]), *_dev(case[2], BF16), out_dtype=F32)
    pick = np.r_[0:20, 33000:33020, r - 40:r]
    _check(y[to_dev(pick)], (case[0][pick], case[1][pick], case[2], None), F32)
