"""Measured cases of the router's balance loss and the 4-bit integer experts.

Operators: the load-balance and z losses of a softmax top-k router with its
per-expert counts, their gradient, the quantisation of weights to 4-bit
integers with group scales, and the experts' products with such weights over
rows in any order.  ``run`` computes a case either in plain torch operations
(``own`` false) or through the framework's calls (``own`` true); ``exact`` is
the same result from the definition in float64.

N tokens, E experts, k experts per token, B sequences; R rows, K and N the
inner and outer size of an expert's weights, g weights per scale.  Codes are
two to a byte, the even element in the low nibble; a weight is s (q - 8), or
s q + b with biases.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


def listed():
    return [
        # router of a prefill batch: 4096 tokens of one sequence, top-8 of 256 experts
        dict(name="balance_prefill", op="balance", n=4096, e=256, k=8, seqs=1, pad=0.0),
        # a packed training batch: 37 sequences of uneven length over 32768 tokens, a tenth of them padding
        dict(name="balance_packed", op="balance", n=32768, e=256, k=8, seqs=37, pad=0.1),
        # the smallest layer, where the launch counts: 16 tokens, top-2 of 8 experts
        dict(name="balance_tiny", op="balance", n=16, e=8, k=2, seqs=1, pad=0.0),
        # the gradient of the prefill batch
        dict(name="balance_backward_prefill", op="balance_backward", n=4096, e=256, k=8, seqs=1, pad=0.0),
        # the gradient of the packed batch
        dict(name="balance_backward_packed", op="balance_backward", n=32768, e=256, k=8, seqs=37, pad=0.1),
        # loading a layer: the gate weights of 8 experts (14336 x 4096 each) to 4 bits, and back
        dict(name="quantize4_experts", op="quantize4", r=114688, kk=4096, x="bf16", g=128, affine=False, s="bf16"),
        # a shared expert's fp32 weights of odd height, small groups with biases
        dict(name="quantize4_affine", op="quantize4", r=2113, kk=7168, x="f32", g=32, affine=True, s="f32"),
        # decode batch: 128 tokens, top-8 of 256 experts, gate and up products of F = 2048, rows in token order
        dict(name="gather4_glu_decode", op="gather4", r=1024, e=256, kk=7168, n=2048, glu=True, g=128, affine=False, s="bf16", y="bf16", skew=0.0),
        # a single token: its 8 rows through the down product
        dict(name="gather4_single_token", op="gather4", r=8, e=256, kk=2048, n=7168, glu=False, g=128, affine=False, s="bf16", y="bf16", skew=0.0),
        # one row through one dense (shared) expert of odd width
        dict(name="gather4_shared_expert", op="gather4", r=1, e=1, kk=7168, n=2113, glu=False, g=64, affine=True, s="bf16", y="bf16", skew=0.0),
        # 64 tokens, top-2 of 8 experts: 16 rows per expert, small groups with biases
        dict(name="gather4_glu_8_experts", op="gather4", r=128, e=8, kk=4096, n=14336, glu=True, g=32, affine=True, s="bf16", y="bf16", skew=0.0),
        # down product of a small batch into an fp32 residual, fp32 scales, uneven experts
        dict(name="gather4_down_f32", op="gather4", r=48, e=8, kk=14336, n=4096, glu=False, g=64, affine=False, s="f32", y="f32", skew=0.5),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["balance", "balance_backward", "quantize4", "gather4", "gather4"])
    if op in ("balance", "balance_backward"):
        e = rng.choice([8, 60, 64, 128, 160, 256])
        return dict(op=op, n=_log_int(rng, 1, 32768), e=e, k=rng.randint(1, 8), seqs=_log_int(rng, 1, 64),
                    pad=rng.choice([0.0, 0.2]))
    g, affine, s = rng.choice([32, 64, 128]), rng.random() < 0.5, rng.choice(["bf16", "f32"])
    kk = g * _log_int(rng, 1, 7168 // g)
    if op == "quantize4":
        return dict(op=op, r=_log_int(rng, 1, 16384), kk=kk, x=rng.choice(["f32", "bf16"]), g=g, affine=affine, s=s)
    return dict(op=op, r=_log_int(rng, 1, 512), e=rng.choice([1, 8, 32, 128]), kk=kk, n=_log_int(rng, 64, 4096),
                glu=rng.random() < 0.5, g=g, affine=affine, s=s, y=rng.choice(["bf16", "bf16", "f32"]),
                skew=rng.choice([0.0, 0.5]))


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, scale=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * scale


def _logits(g, n, e, skew):
    """Router logits, popularity falling as a power of a seeded rank."""
    rank = torch.randperm(e, generator=g, device=DEV).float()
    return _randn(g, n, e) - skew * torch.log1p(rank)


def _code_values(codes):
    """Codes [..., K/2] as numbers 0 .. 15 [..., K] (uint8)."""
    return torch.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], codes.shape[-1] * 2)


def _weights(g, case, e):
    """Codes, scales and biases of e experts, one at a time to bound the float32 temporaries."""
    n, kk, grp = case["n"], case["kk"], case["g"]
    codes = torch.empty((e, n, kk // 2), dtype=torch.uint8, device=DEV)
    scales = torch.empty((e, n, kk // grp), dtype=DTYPES[case["s"]], device=DEV)
    biases = torch.empty_like(scales) if case["affine"] else None
    for i in range(e):
        w = _randn(g, n, kk // grp, grp, scale=0.02)
        if case["affine"]:
            lo, hi = w.amin(-1), w.amax(-1)
            scales[i], biases[i] = (hi - lo) / 15, lo
            q = torch.round((w - biases[i].float().unsqueeze(-1)) / scales[i].float().unsqueeze(-1))
        else:
            scales[i] = w.abs().amax(-1) / 7
            q = torch.round(w / scales[i].float().unsqueeze(-1)) + 8
        q = q.clamp(0, 15).to(torch.uint8).view(n, kk // 2, 2)
        codes[i] = q[..., 0] | (q[..., 1] << 4)
    return codes, scales, biases


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op in ("balance", "balance_backward"):
        n, e, k, b = case["n"], case["e"], min(case["k"], case["e"]), case["seqs"]
        logits = _logits(g, n, e, 0.5)
        idx = torch.topk(logits, k, dim=1).indices.int()
        s = dict(op=op, logits=logits, idx=idx, k=k, offs=None, mask=None)
        if b > 1:                                 # uneven sequences; what is behind the last one is in none
            cut = torch.sort(torch.randint(0, n + 1, (b + 1,), generator=g, device=DEV)).values
            cut[0] = 0
            s["offs"] = cut.int()
        if case["pad"]:
            s["mask"] = torch.rand(n, generator=g, device=DEV) >= case["pad"]
        if op == "balance_backward":              # what the forward pass handed out, and the gradients of its losses
            seq, valid = _sequence(s)
            s["tokens"] = torch.bincount(seq[valid], minlength=b).int()
            where = (seq.unsqueeze(1) * e + idx.long())[valid]
            s["counts"] = torch.bincount(where.reshape(-1), minlength=b * e).view(b, e).int()
            s["d_loss"] = torch.full((b,), 0.01 / b, device=DEV) * (1.0 + torch.rand(b, generator=g, device=DEV))
            s["d_z"] = torch.full((b,), 0.001 / b, device=DEV) * (1.0 + torch.rand(b, generator=g, device=DEV))
        return s
    if op == "quantize4":
        x = _randn(g, case["r"], case["kk"], scale=0.02).to(DTYPES[case["x"]])
        return dict(op=op, x=x, g=case["g"], affine=case["affine"], s=DTYPES[case["s"]])
    # hidden states with a few loud channels, and the expert of every row
    loud = 1.0 + 7.0 * (torch.rand(case["kk"], generator=g, device=DEV) < 0.01).float()
    rows = (_randn(g, case["r"], case["kk"]) * loud).to(torch.bfloat16)
    expert = _logits(g, case["r"], case["e"], case["skew"]).argmax(1).int()
    s = dict(op=op, rows=rows, expert=expert, y=DTYPES[case["y"]], w=_weights(g, case, case["e"]),
             up=(None, None, None), most=int(torch.bincount(expert.long()).max()))
    if case["glu"]:
        s["up"] = _weights(g, case, case["e"])
    return s


# ---------------------------------------------------------------- plain forms

def _sequence(s):
    """The sequence of every token, and which tokens count."""
    n = s["logits"].shape[0]
    t = torch.arange(n, device=DEV)
    if s["offs"] is None:
        seq, valid = torch.zeros_like(t), torch.ones_like(t, dtype=torch.bool)
    else:
        offs = s["offs"].long()
        seq = torch.searchsorted(offs, t, right=True) - 1
        valid = (seq >= 0) & (seq < offs.numel() - 1)
        seq = seq.clamp(0, offs.numel() - 2)
    return seq, valid if s["mask"] is None else valid & s["mask"]


def _softmax(logits):
    top = logits.amax(1, keepdim=True)
    ex = torch.exp(logits - top)
    total = ex.sum(1, keepdim=True)
    return ex / total, (top + torch.log(total)).squeeze(1)


def _dequant(codes, scales, biases):
    q = _code_values(codes).view(*scales.shape, -1).float()
    s = scales.float().unsqueeze(-1)
    w = (q - 8.0) * s if biases is None else q * s + biases.float().unsqueeze(-1)
    return w.reshape(*codes.shape[:-1], codes.shape[-1] * 2)


def _product(s, w):
    """Every row times its expert's weights, float32 [R, N]."""
    codes, scales, biases = w
    x, e = s["rows"].float(), s["expert"].long()
    if x.shape[0] * 4 <= codes.shape[0]:          # few rows: only their experts' weights
        v = _dequant(codes[e], scales[e], None if biases is None else biases[e])
        return torch.bmm(v, x.unsqueeze(-1)).squeeze(-1)
    # rows bucketed by expert into [E, K, most], one batched product, and back
    order = torch.argsort(e, stable=True)
    es = e[order]
    first = torch.searchsorted(es, torch.arange(codes.shape[0], device=DEV))
    slot = torch.arange(x.shape[0], device=DEV) - first[es]
    bucket = torch.zeros((codes.shape[0], s["most"], x.shape[1]), device=DEV)
    bucket[es, slot] = x[order]
    prod = torch.bmm(_dequant(codes, scales, biases), bucket.transpose(1, 2).contiguous())   # [E, N, most]
    out = torch.empty((x.shape[0], codes.shape[1]), device=DEV)
    out[order] = prod.transpose(1, 2)[es, slot]
    return out


def _plain(s):
    op = s["op"]
    if op == "balance":
        e, k = s["logits"].shape[1], s["k"]
        b = 1 if s["offs"] is None else s["offs"].numel() - 1
        seq, valid = _sequence(s)
        p, lse = _softmax(s["logits"])
        # sums over a sequence's tokens as products with its members
        member = ((seq == torch.arange(b, device=DEV).unsqueeze(1)) & valid).float()         # [B, N]
        chosen = torch.zeros_like(p).scatter_add_(1, s["idx"].long(), torch.ones_like(p[:, :k]))
        counts, tokens = torch.mm(member, chosen).int(), member.sum(1).int()                 # below 2^24: exact
        n = tokens.float().clamp(min=1.0).unsqueeze(1)
        probs, z = torch.mm(member, p) / n, torch.mv(member, lse * lse)
        loss = (counts * probs).sum(1) * e / (k * n.squeeze(1))
        return loss, z / n.squeeze(1), counts, probs, tokens
    if op == "balance_backward":
        e, k = s["logits"].shape[1], s["k"]
        seq, valid = _sequence(s)
        p, lse = _softmax(s["logits"])
        n = s["tokens"].float().clamp(min=1.0)
        # counts less their mean, which the softmax's Jacobian takes away
        u = s["counts"].float() - k * n.unsqueeze(1) / e
        u = (u * (s["d_loss"] * e / (k * n * n)).unsqueeze(1))[seq]
        zs = (s["d_z"] * 2.0 / n)[seq] * lse
        d = p * (u - (p * u).sum(1, keepdim=True) + zs.unsqueeze(1))
        return torch.where(valid.unsqueeze(1), d, 0.0)
    if op == "quantize4":
        x = s["x"].float().view(s["x"].shape[0], -1, s["g"])
        if s["affine"]:
            biases = x.amin(-1)
            scales = ((x.amax(-1) - biases) / 15.0).to(s["s"])
            biases = biases.to(s["s"])
            off = x.double() - biases.double().unsqueeze(-1)       # 64 bits: values next to a border
        else:
            biases = None
            scales = (x.abs().amax(-1) / 7.0).to(s["s"])
            off = x.double()
        sc = scales.double().unsqueeze(-1)
        q = torch.round(off / torch.where(sc == 0, 1.0, sc))
        if s["affine"]:
            q = q.clamp(0.0, 15.0).float()
            v = q * scales.float().unsqueeze(-1) + biases.float().unsqueeze(-1)
        else:
            v = q.clamp(-8.0, 7.0).float() * scales.float().unsqueeze(-1)
        v = v.view(s["x"].shape).to(torch.bfloat16)
        return (v, scales) if biases is None else (v, scales, biases)
    y = _product(s, s["w"])
    if s["up"][0] is not None:
        y = y / (1.0 + torch.exp(-y)) * _product(s, s["up"])
    return y.to(s["y"])


def run(state):
    if not own:
        return _plain(state)
    import combine_moe_route_topk_amd as moe
    s, op = state, state["op"]
    if op == "balance":
        r = moe.moe_balance_loss(s["logits"], s["idx"], seq_offsets=s["offs"], token_mask=s["mask"])
        return r.loss, r.z_loss, r.counts, r.probs, r.tokens
    if op == "balance_backward":
        return moe.moe_balance_loss_backward(s["logits"], s["counts"], s["tokens"], s["k"], s["d_loss"], s["d_z"],
                                             seq_offsets=s["offs"], token_mask=s["mask"])
    if op == "quantize4":
        codes, scales, biases = moe.moe_quantize_int4(s["x"], s["g"], affine=s["affine"], scale_dtype=s["s"])
        v = moe.moe_dequant_int4(codes, scales, biases)
        return (v, scales) if biases is None else (v, scales, biases)
    return moe.moe_gather_gemm_int4(s["rows"], s["expert"], *s["w"], w_up=s["up"][0], w_up_scales=s["up"][1],
                                    w_up_biases=s["up"][2], out_dtype=s["y"])


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op in ("balance", "balance_backward"):
        n, e, k, b = case["n"], case["e"], min(case["k"], case["e"]), case["seqs"]
        mask = n if case["pad"] else 0
        if op == "balance":                       # logits, ids, mask; counts, probs and three numbers a sequence
            return dict(bytes=4 * n * e + 4 * n * k + mask + 8 * b * e + 12 * b, flops=4 * n * e)
        return dict(bytes=8 * n * e + mask + 4 * b * e + 12 * b, flops=7 * n * e)
    if op == "quantize4":                         # x to codes and scales, and these to bf16 values
        m = case["r"] * case["kk"]
        sc = SIZE[case["s"]] * (2 if case["affine"] else 1) / case["g"]
        return dict(bytes=m * SIZE[case["x"]] + 2 * m * (1 / 2 + sc) + 2 * m, flops=5 * m)
    r, e, kk, n = case["r"], case["e"], case["kk"], case["n"]
    # experts that expect at least one row: E (1 - (1 - 1/E)^R), for even popularity
    active = e * (1.0 - (1.0 - 1.0 / e) ** r)
    mats = 2 if case["glu"] else 1
    per = kk * (1 / 2 + SIZE[case["s"]] * (2 if case["affine"] else 1) / case["g"])
    return dict(bytes=2 * r * kk + mats * active * n * per + r * n * SIZE[case["y"]], flops=2.0 * mats * r * kk * n)


# ---------------------------------------------------------------- the definitions in float64

def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("balance", "balance_backward"):
        n, e, k, b = case["n"], case["e"], s["k"], case["seqs"]
        offs = [0, n] if s["offs"] is None else s["offs"].tolist()
        keep = torch.ones(n, dtype=torch.bool, device=DEV) if s["mask"] is None else s["mask"]
        loss, z = torch.zeros((2, b), dtype=torch.float64, device=DEV)
        probs = torch.zeros((b, e), dtype=torch.float64, device=DEV)
        counts = torch.zeros((b, e), dtype=torch.int32, device=DEV)
        tokens = torch.zeros(b, dtype=torch.int32, device=DEV)
        grad = torch.zeros((n, e), dtype=torch.float64, device=DEV)
        for i in range(b):
            t = torch.arange(offs[i], offs[i + 1], device=DEV)
            t = t[keep[t]]
            if not t.numel():
                continue
            l = s["logits"][t].double()
            p, lse = torch.softmax(l, 1), torch.logsumexp(l, 1)
            c = torch.bincount(s["idx"][t].long().reshape(-1), minlength=e)
            frac = c.double() * e / (k * t.numel())
            if op == "balance_backward":
                # the Jacobian of the softmax, the counts standing for constants
                up = frac * s["d_loss"][i].double() / t.numel()
                g = p * (up - (p * up).sum(1, keepdim=True))
                grad[t] = g + p * (lse * 2.0 * s["d_z"][i].double() / t.numel()).unsqueeze(1)
                continue
            tokens[i], counts[i], probs[i] = t.numel(), c.int(), p.mean(0)
            loss[i], z[i] = (frac * p.mean(0)).sum(), (lse * lse).mean()
        return grad if op == "balance_backward" else (loss, z, counts, probs, tokens)
    if op == "quantize4":
        grp, r = case["g"], case["r"]
        out = torch.empty(s["x"].shape, dtype=torch.float64, device=DEV)
        scales, biases = torch.empty((2, r, case["kk"] // grp), dtype=torch.float64, device=DEV)
        for r0 in range(0, r, 4096):
            x = s["x"][r0:r0 + 4096].double().reshape(-1, grp)
            # the scale is held in 32 bits before its own rounding
            if case["affine"]:
                lo, hi = x.min(1).values, x.max(1).values
                sc = ((hi - lo).float() / 15.0).to(s["s"]).double()
                base, zero = lo.to(s["s"]).double(), 0
            else:
                sc = (x.abs().max(1).values.float() / 7.0).to(s["s"]).double()
                base, zero = torch.zeros_like(sc), 8
            v = (x - base.unsqueeze(1)) / sc.clamp(min=1e-300).unsqueeze(1) + zero
            lo = torch.floor(v)
            up = ((v - lo) > 0.5) | (((v - lo) == 0.5) & (lo % 2 == 1))
            q = (lo + up).clamp(0, 15) - zero
            out[r0:r0 + 4096] = (q * sc.unsqueeze(1) + base.unsqueeze(1)).reshape(-1, case["kk"])
            scales[r0:r0 + 4096] = sc.view(-1, case["kk"] // grp)
            biases[r0:r0 + 4096] = base.view(-1, case["kk"] // grp)
        return (out, scales, biases) if case["affine"] else (out, scales)
    y = torch.empty((case["r"], case["n"]), dtype=torch.float64, device=DEV)

    def weight(w, i):
        q = torch.stack((w[0][i] % 16, w[0][i] // 16), -1).view(*w[1][i].shape, case["g"]).double()
        sc = w[1][i].double().unsqueeze(-1)
        v = sc * q + (-8.0 * sc if w[2] is None else w[2][i].double().unsqueeze(-1))
        return v.view(case["n"], case["kk"])

    for i in torch.unique(s["expert"]).tolist():
        sel = torch.nonzero(s["expert"] == i).squeeze(1)
        x = s["rows"][sel].double()
        v = x @ weight(s["w"], i).t()
        if case["glu"]:
            v = v * torch.sigmoid(v) * (x @ weight(s["up"], i).t())
        y[sel] = v
    return y
