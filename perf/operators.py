"""Measured cases of the training and MXFP4 operators of the MoE token path.

Operators: the gradients of routing, dispatch and combine, and the microscaled
4-bit (MXFP4) quantisation and expert products.  ``run`` computes a case either
in plain torch operations (``own`` false) or through the framework's calls
(``own`` true); ``exact`` is the same result from the definition in float64.

N tokens, D hidden size, E experts, k experts per token, R = N*k dispatched
rows.  MXFP4: E2M1 codes, two per byte (even element in the low nibble), one
E8M0 scale byte per 32 elements.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
BLOCK = 32


def listed():
    return [
        # training step over a prefill-sized batch: 4096 tokens, hidden 7168, top-8 of 256 experts
        dict(name="combine_backward_prefill", op="combine_backward", n=4096, d=7168, k=8, e=256, y="bf16", g="bf16", drop=0.0),
        # a ragged fp32 micro-batch with 5% of the pairs dropped (capacity), gradient from a bf16 residual
        dict(name="combine_backward_ragged", op="combine_backward", n=513, d=4100, k=2, e=8, y="f32", g="bf16", drop=0.05),
        # an 8-expert, top-2 layer of hidden 4096 over 8192 tokens
        dict(name="dispatch_backward_top2", op="dispatch_backward", n=8192, d=4096, k=2, e=8, y="bf16", g="bf16", drop=0.0),
        # the smallest layer, where the launch counts: 16 tokens of 64 floats
        dict(name="dispatch_backward_tiny", op="dispatch_backward", n=16, d=64, k=2, e=8, y="f32", g="f32", drop=0.0),
        # router gradient of the prefill batch, weights renormalised over the chosen experts
        dict(name="route_backward_top8", op="route_backward", n=4096, e=256, k=8, renorm=True),
        # full-softmax router weights (the gradient reaches every expert), long batch
        dict(name="route_backward_softmax", op="route_backward", n=32768, e=256, k=4, renorm=False),
        # activations between the two products of an 8-expert layer: 16384 rows of 14336
        dict(name="quantize_ffn_rows", op="quantize", r=16384, kk=14336, x="bf16"),
        # hidden states of a decode batch in fp32
        dict(name="quantize_decode", op="quantize", r=128, kk=7168, x="f32"),
        # gate and up product of an 8-expert layer over 8192 tokens, top-2 (F = 14336)
        dict(name="grouped_glu_8_experts", op="grouped", r=16384, e=8, kk=4096, n=14336, glu=True, skew=0.0),
        # 256 experts with 32 rows each: the weights are most of the bytes
        dict(name="grouped_256_experts", op="grouped", r=8192, e=256, kk=7168, n=4096, glu=False, skew=0.0),
        # decode batch: 128 tokens, top-8 of 256 experts, F = 2048, rows in token order
        dict(name="gather_glu_decode", op="gather", r=1024, e=256, kk=7168, n=2048, glu=True, skew=0.0),
        # a single token: its 8 rows through the down product
        dict(name="gather_single_token", op="gather", r=8, e=256, kk=2048, n=7168, glu=False, skew=0.0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["combine_backward", "dispatch_backward", "route_backward", "quantize", "grouped", "gather"])
    if op in ("combine_backward", "dispatch_backward"):
        d = _log_int(rng, 64, 7168)
        if rng.random() < 0.6:                    # most hidden sizes are multiples of 8
            d = d // 8 * 8
        e = rng.choice([8, 64, 256])
        return dict(op=op, n=_log_int(rng, 1, 4096), d=d, k=rng.randint(1, 8), e=e,
                    y=rng.choice(["f32", "bf16"]) if d * 2 <= 7168 else "bf16",
                    g=rng.choice(["f32", "bf16"]) if d * 2 <= 7168 else "bf16", drop=rng.choice([0.0, 0.1]))
    if op == "route_backward":
        return dict(op=op, n=_log_int(rng, 1, 32768), e=rng.randint(8, 256), k=rng.randint(1, 8),
                    renorm=rng.random() < 0.5)
    if op == "quantize":
        return dict(op=op, r=_log_int(rng, 1, 16384), kk=BLOCK * _log_int(rng, 1, 448 // 2),
                    x=rng.choice(["f32", "bf16"]))
    if op == "grouped":
        return dict(op=op, r=_log_int(rng, 1, 8192), e=rng.choice([4, 8, 16, 32, 64]), kk=128 * _log_int(rng, 1, 56),
                    n=8 * _log_int(rng, 8, 512), glu=rng.random() < 0.5, skew=rng.choice([0.0, 0.5]))
    return dict(op=op, r=_log_int(rng, 1, 1024), e=rng.choice([8, 32, 128]), kk=128 * _log_int(rng, 1, 56),
                n=8 * _log_int(rng, 8, 512), glu=rng.random() < 0.5, skew=rng.choice([0.0, 0.5]))


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, scale=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * scale


def _routing(g, n, e, k, skew=0.0):
    """Router logits (popularity falling as a power of a seeded rank) and their top-k."""
    rank = torch.randperm(e, generator=g, device=DEV).float()
    logits = _randn(g, n, e) - skew * torch.log1p(rank)
    top, idx = torch.topk(logits, k, dim=1)
    return logits, idx.int(), top


def _positions(g, n, e, k, drop):
    """Row of every pair after a stable sort by expert; dropped pairs hold -1."""
    _, idx, _ = _routing(g, n, e, min(k, e), 1.1)
    order = torch.argsort(idx.reshape(-1), stable=True)
    pos = torch.empty(n * k, dtype=torch.int32, device=DEV)
    pos[order] = torch.arange(n * k, dtype=torch.int32, device=DEV)
    if drop:
        gone = torch.rand(n * k, generator=g, device=DEV) < drop
        pos = torch.where(gone, torch.full_like(pos, -1), pos)
    return pos


def _encode(x):
    """MXFP4 codes and scales of x [..., K] float32 (used to make operands)."""
    shape = x.shape
    b = x.reshape(-1, BLOCK)
    byte = torch.frexp(b.abs().amax(1, keepdim=True))[1] - 1 - 2 + 127   # floor(log2 amax) - 2, biased
    byte = byte.clamp(0, 254)
    v = torch.ldexp(b, 127 - byte)
    step = torch.exp2((torch.frexp(v)[1] - 1).clamp(0, 2).float() - 1)    # grid of E2M1 at this size
    q = (torch.round(v.abs() / step) * step).clamp(max=6.0)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=x.device)
    code = (torch.searchsorted(grid, q) + 8 * (v < 0)).to(torch.uint8).view(-1, 2)
    packed = (code[:, 0] | (code[:, 1] << 4)).reshape(*shape[:-1], shape[-1] // 2)
    return packed, byte.to(torch.uint8).reshape(*shape[:-1], shape[-1] // BLOCK)


def _activations(g, r, k):
    """Rows with a few loud channels, as hidden states have them."""
    loud = 1.0 + 7.0 * (torch.rand(k, generator=g, device=DEV) < 0.01).float()
    return _randn(g, r, k) * loud


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "combine_backward":
        n, d, k = case["n"], case["d"], case["k"]
        return dict(op=op, k=k, pos=_positions(g, n, case["e"], k, case["drop"]),
                    w=torch.softmax(_randn(g, n, k), 1),
                    g=_randn(g, n, d).to(DTYPES[case["g"]]), y=_randn(g, n * k, d).to(DTYPES[case["y"]]),
                    # rows of dropped pairs have gradient zero and are not written
                    d_y=torch.zeros((n * k, d), dtype=DTYPES[case["y"]], device=DEV))
    if op == "dispatch_backward":
        n, d, k = case["n"], case["d"], case["k"]
        return dict(op=op, k=k, pos=_positions(g, n, case["e"], k, case["drop"]),
                    rows=_randn(g, n * k, d).to(DTYPES[case["y"]]), out=DTYPES[case["g"]])
    if op == "route_backward":
        logits, idx, top = _routing(g, case["n"], case["e"], case["k"], 1.1)
        w = torch.softmax(top, 1) if case["renorm"] else torch.exp(top - torch.logsumexp(logits, 1, keepdim=True))
        return dict(op=op, e=case["e"], renorm=case["renorm"], logits=logits, idx=idx, w=w.contiguous(),
                    g=_randn(g, case["n"], case["k"]))
    if op == "quantize":
        return dict(op=op, x=_activations(g, case["r"], case["kk"]).to(DTYPES[case["x"]]))
    def weights(e, n, k):
        codes = torch.empty((e, n, k // 2), dtype=torch.uint8, device=DEV)
        scales = torch.empty((e, n, k // BLOCK), dtype=torch.uint8, device=DEV)
        for i in range(e):                        # one expert at a time bounds the float32 temporaries
            codes[i], scales[i] = _encode(_randn(g, n, k, scale=0.02))
        return codes, scales

    rows, row_scales = _encode(_activations(g, case["r"], case["kk"]))
    _, idx, _ = _routing(g, case["r"], case["e"], 1, case["skew"])
    expert = idx.reshape(-1)
    if op == "grouped":
        expert = torch.sort(expert).values
    counts = torch.bincount(expert.long(), minlength=case["e"])
    offs = torch.zeros(case["e"] + 1, dtype=torch.int32, device=DEV)
    offs[1:] = torch.cumsum(counts, 0).int()
    s = dict(op=op, rows=rows, row_scales=row_scales, expert=expert.contiguous(), offs=offs,
             most=int(counts.max()), w=weights(case["e"], case["n"], case["kk"]), up=(None, None))
    if case["glu"]:
        s["up"] = weights(case["e"], case["n"], case["kk"])
    return s


# ---------------------------------------------------------------- plain forms

def _decode(codes, scales):
    """float32 values of MXFP4 codes and scales (scale bytes below 255)."""
    c = torch.arange(16, device=codes.device)
    mag = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    one = torch.where(c >= 8, -mag[c % 8], mag[c % 8])
    b = torch.arange(256, device=codes.device)
    pair = torch.stack((one[b % 16], one[b // 16]), 1)                # both values of a byte
    v = pair[codes.int()].reshape(*scales.shape, BLOCK)
    v *= torch.ldexp(torch.ones((), device=codes.device), scales.int() - 127).unsqueeze(-1)
    return v.reshape(*codes.shape[:-1], codes.shape[-1] * 2)


def _product(s, w):
    """Every row times its expert's weights, float32 [R, N]."""
    codes, scales = w
    x = _decode(s["rows"], s["row_scales"])
    if x.shape[0] * 4 <= codes.shape[0]:          # few rows: only their experts' weights
        e = s["expert"].long()
        return torch.bmm(_decode(codes[e], scales[e]), x.unsqueeze(-1)).squeeze(-1)
    # rows bucketed by expert into [E, most, K], one batched product, and back
    order = torch.argsort(s["expert"], stable=True)
    e = s["expert"][order].long()
    slot = torch.arange(x.shape[0], device=x.device) - s["offs"][e]
    bucket = torch.zeros((codes.shape[0], s["most"], x.shape[1]), device=x.device)
    bucket[e, slot] = x[order]
    prod = torch.bmm(_decode(codes, scales), bucket.transpose(1, 2).contiguous())   # [E, N, most]
    out = torch.empty((x.shape[0], codes.shape[1]), device=x.device)
    out[order] = prod.transpose(1, 2)[e, slot]
    return out


def _plain(s):
    op = s["op"]
    if op == "combine_backward":
        k, pos = s["k"], s["pos"].long()
        ok = (pos >= 0) & (pos < pos.numel())
        gt = s["g"].float().repeat_interleave(k, 0)
        d_y = torch.zeros((pos.numel() + 1, gt.shape[1]), device=gt.device)
        d_y[torch.where(ok, pos, pos.numel())] = gt * s["w"].reshape(-1, 1)
        d_w = torch.where(ok, (gt * s["y"].float()[pos.clamp(min=0)]).sum(1), 0.0)
        return d_y[:-1].to(s["y"].dtype), d_w.view_as(s["w"])
    if op == "dispatch_backward":
        pos = s["pos"].long()
        ok = (pos >= 0) & (pos < pos.numel())
        v = torch.where(ok.unsqueeze(1), s["rows"].float()[pos.clamp(min=0)], 0.0)
        return v.view(-1, s["k"], v.shape[1]).sum(1).to(s["out"])
    if op == "route_backward":
        wd = s["w"] * s["g"]
        total = wd.sum(1, keepdim=True)
        idx = s["idx"].long()
        if s["renorm"]:
            d = torch.zeros((idx.shape[0], s["e"]), device=wd.device)
            return d.scatter_(1, idx, wd - s["w"] * total)
        p = torch.exp(s["logits"] - torch.logsumexp(s["logits"], 1, keepdim=True))
        return (-p * total).scatter_add_(1, idx, wd)
    if op == "quantize":
        x = s["x"].float()
        b = x.reshape(-1, BLOCK)
        scale = torch.exp2((torch.frexp(b.abs().amax(1, keepdim=True))[1] - 3).clamp(min=-127).float())
        v = b / scale
        step = torch.exp2((torch.frexp(v)[1] - 1).clamp(0, 2).float() - 1)    # grid of E2M1 at this size
        q = (torch.round(v / step) * step).clamp(-6.0, 6.0)
        return (q * scale).reshape(x.shape).to(torch.bfloat16)
    y = _product(s, s["w"])
    if s["up"][0] is not None:
        y = y / (1.0 + torch.exp(-y)) * _product(s, s["up"])
    return y.to(torch.bfloat16)


def run(state):
    if not own:
        return _plain(state)
    import combine_moe_route_topk_amd as moe
    s, op = state, state["op"]
    if op == "combine_backward":
        return moe.moe_combine_backward(s["g"], s["y"], s["pos"], s["w"], d_y=s["d_y"])
    if op == "dispatch_backward":
        return moe.moe_dispatch_backward(s["rows"], s["pos"], s["k"], out_dtype=s["out"])
    if op == "route_backward":
        return moe.moe_route_topk_backward(s["idx"], s["w"], s["g"], s["e"], renormalize=s["renorm"],
                                           logits=None if s["renorm"] else s["logits"])
    if op == "quantize":
        codes, scales = moe.moe_quantize_mxfp4(s["x"])
        return moe.moe_dequant_mxfp4(codes, scales)
    if op == "grouped":
        return moe.moe_grouped_gemm_mxfp4(s["rows"], s["row_scales"], s["offs"], s["w"][0], s["w"][1],
                                          w_up=s["up"][0], w_up_scales=s["up"][1])
    return moe.moe_gather_gemm_mxfp4(s["rows"], s["row_scales"], s["expert"], s["w"][0], s["w"][1],
                                     w_up=s["up"][0], w_up_scales=s["up"][1])


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op in ("combine_backward", "dispatch_backward"):
        n, d, nk = case["n"], case["d"], case["n"] * case["k"]
        keep = 1.0 - case["drop"]
        y, g = SIZE[case["y"]], SIZE[case["g"]]
        if op == "combine_backward":              # y read, d_y written; d_out read; dst, w, d_w
            return dict(bytes=keep * 2 * nk * d * y + n * d * g + 12 * nk, flops=3 * nk * d)
        return dict(bytes=keep * nk * d * y + n * d * g + 4 * nk, flops=nk * d)
    if op == "route_backward":
        n, e, k = case["n"], case["e"], case["k"]
        return dict(bytes=n * e * 4 * (1 if case["renorm"] else 2) + 12 * n * k, flops=4 * n * k + (0 if case["renorm"] else 3 * n * e))
    if op == "quantize":                          # x to codes and scales, and these to bf16 values
        m = case["r"] * case["kk"]
        return dict(bytes=m * SIZE[case["x"]] + 2 * m * (1 / 2 + 1 / 32) + 2 * m, flops=4 * m)
    r, e, kk, n = case["r"], case["e"], case["kk"], case["n"]
    # experts that expect at least one row: E (1 - (1 - 1/E)^R), for even popularity
    active = e * (1.0 - (1.0 - 1.0 / e) ** r)
    mats = 2 if case["glu"] else 1
    per = kk * (1 / 2 + 1 / 32)
    return dict(bytes=r * per + mats * active * n * per + 2 * r * n, flops=2.0 * mats * r * kk * n)


# ---------------------------------------------------------------- the definitions in float64

def _values64(codes, scales):
    c = torch.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1).to(torch.int32)
    exp, man = (c >> 1) & 3, (c & 1).double()
    mag = torch.where(exp == 0, 0.5 * man, (1.0 + 0.5 * man) * torch.exp2(exp.double() - 1.0))
    mag = torch.where(c >= 8, -mag, mag)
    return mag * torch.exp2(scales.double() - 127.0).repeat_interleave(BLOCK, -1)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "combine_backward":
        k, nk = s["k"], s["pos"].numel()
        d_y = torch.zeros((nk, case["d"]), dtype=torch.float64, device=DEV)
        d_w = torch.zeros((case["n"], k), dtype=torch.float64, device=DEV)
        for j in range(k):
            pos = s["pos"].view(-1, k)[:, j].long()
            tok = torch.nonzero(pos >= 0).squeeze(1)
            gj, wj = s["g"][tok].double(), s["w"][tok, j].double()
            d_y[pos[tok]] = wj.unsqueeze(1) * gj
            d_w[tok, j] = (gj * s["y"][pos[tok]].double()).sum(1)
        return d_y, d_w
    if op == "dispatch_backward":
        out = torch.zeros((case["n"], case["d"]), dtype=torch.float64, device=DEV)
        for j in range(s["k"]):
            pos = s["pos"].view(-1, s["k"])[:, j].long()
            tok = torch.nonzero(pos >= 0).squeeze(1)
            out[tok] += s["rows"][pos[tok]].double()
        return out
    if op == "route_backward":
        # the Jacobian of the softmax, from the weights that the forward pass handed out
        idx, w, gw = s["idx"].long(), s["w"].double(), s["g"].double()
        onehot = torch.zeros((case["n"], case["e"]), dtype=torch.float64, device=DEV)
        up = onehot.scatter(1, idx, gw)
        p = onehot.scatter(1, idx, w) if case["renorm"] else torch.softmax(s["logits"].double(), 1)
        return p * (up - (p * up).sum(1, keepdim=True))
    if op == "quantize":
        x = s["x"]
        out = torch.empty(x.shape, dtype=torch.float64, device=DEV)
        grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=DEV)
        for r0 in range(0, x.shape[0], 1024):
            b = x[r0:r0 + 1024].double().reshape(-1, BLOCK)
            e = torch.floor(torch.log2(b.abs().amax(1, keepdim=True))) - 2.0
            scale = torch.exp2(torch.clamp(e, min=-127.0))
            v = (b / scale).abs()
            lo = torch.searchsorted(grid, v.clamp(max=6.0), right=True).sub(1).clamp(max=6)
            a, c = grid[lo], grid[lo + 1]
            up = ((v - a) > (c - v)) | (((v - a) == (c - v)) & (lo % 2 == 1))
            q = torch.where(up, c, a)
            out[r0:r0 + 1024] = (torch.sign(b) * q * scale).reshape(-1, x.shape[1])
        return out
    y = torch.empty((case["r"], case["n"]), dtype=torch.float64, device=DEV)
    for i in torch.unique(s["expert"]).tolist():
        sel = torch.nonzero(s["expert"] == i).squeeze(1)
        x = _values64(s["rows"][sel], s["row_scales"][sel])
        v = x @ _values64(s["w"][0][i], s["w"][1][i]).t()
        if case["glu"]:
            v = v * torch.sigmoid(v) * (x @ _values64(s["up"][0][i], s["up"][1][i]).t())
        y[sel] = v
    return y
