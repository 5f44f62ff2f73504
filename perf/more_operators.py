"""Training through a layer on int8 weights, as workloads: attention of packed sequences with its gradient,
rotary positions with several axes and their gradient, layer norm with its gradients, and the norm and clipping
of a model's gradients. Each in a plain torch form and through the package's entry points.

A case names its operator (``op``):
  attend  ``hq`` query and ``hk`` key/value heads of ``dim`` channels, ``seqs`` sequences of ``lo`` to ``hi``
          tokens packed one after the other, ``causal``, ``window`` and ``sinks``
  rope    ``rows`` tokens of ``hq`` and ``hk`` heads, the first ``rot`` channels turned; ``sections``: how many
          pairs follow each axis ("16,24,24"), in blocks or in turns (``turns``)
  norm    ``rows`` of ``width`` channels; ``affine``: weight and bias in the type of x, in fp32, or none
  clip    ``tensors`` gradients of ``lo`` to ``hi`` values, written back in their type or in fp32 (``wide``)
and the type; ``train``: the gradients too. Lengths are a function of the case alone; values come from the seed.
"""
from __future__ import annotations

import math
import random

import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5


def _attend(name, hq, hk, dim, seqs, lo, hi, dtype, causal=True, window=0, sinks=0, train=True):
    return {"name": name, "op": "attend", "hq": hq, "hk": hk, "dim": dim, "seqs": seqs, "lo": lo, "hi": hi,
            "dtype": dtype, "causal": causal, "window": window, "sinks": sinks, "train": train}


def _rope(name, rows, hq, hk, dim, rot, sections, dtype, turns=False, interleaved=False, train=True):
    return {"name": name, "op": "rope", "rows": rows, "hq": hq, "hk": hk, "dim": dim, "rot": rot,
            "sections": sections, "turns": turns, "interleaved": interleaved, "dtype": dtype, "train": train}


def _norm(name, rows, width, dtype, affine, train=True):
    return {"name": name, "op": "norm", "rows": rows, "width": width, "dtype": dtype, "affine": affine,
            "train": train}


def _clip(name, tensors, lo, hi, dtype, wide):
    return {"name": name, "op": "clip", "tensors": tensors, "lo": lo, "hi": hi, "dtype": dtype, "wide": wide}


def listed():
    return [
        # a step on a few short texts with a small model: latency only
        _attend("attend_notes", 8, 2, 64, 3, 5, 60, "fp16"),
        # prompts of several users scored in one call, no gradient
        _attend("attend_score", 32, 8, 128, 4, 700, 8192, "bf16", train=False),
        # a training step on documents of different lengths packed into one row
        _attend("attend_documents", 32, 8, 128, 6, 300, 4096, "bf16"),
        # the same with a sliding window and sinks, a key/value head of its own for every query head
        _attend("attend_window", 16, 16, 64, 9, 100, 6000, "fp16", window=500, sinks=4),
        # images of different sizes, every patch sees all of its image
        _attend("attend_images", 16, 16, 80, 20, 200, 1500, "bf16", causal=False),
        # one token of a served model with three axes: latency only
        _rope("rope_token", 1, 32, 8, 128, 128, "16,24,24", "bf16", train=False),
        # frames of a video: time, height and width
        _rope("rope_frames", 16000, 32, 8, 128, 128, "24,20,20", "bf16", turns=True),
        # one token of a served model: latency only
        _norm("norm_token", 1, 4096, "fp16", "same", train=False),
        # a training step, parameters kept in fp32
        _norm("norm_step", 8190, 4096, "bf16", "fp32"),
        # an odd width, as after pruning
        _norm("norm_odd", 1700, 1001, "fp16", "same"),
        # only a model's norms are trained: latency only
        _clip("clip_norms", 65, 4096, 4096, "fp32", False),
        # adapters on every layer of a model: many tensors, written as the optimizer's fp32
        _clip("clip_adapters", 448, 4096, 180000, "bf16", True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "rope", "norm", "clip"])
    dtype = rng.choice(["fp16", "bf16"])
    if op == "attend":
        hk = rng.choice([1, 2, 4, 8, 8, 16])
        hq = hk * rng.choice([1, 2, 3, 4, 5, 8] if hk <= 8 else [1, 2])
        dim = rng.choice([40, 64, 72, 80, 96, 128, 128, 128])
        seqs = _log_int(rng, 1, 40)
        most = int(math.sqrt(7.0e10 / (seqs * hq * dim)))  # no case costs more than the largest listed one
        hi = _log_int(rng, 16, max(17, min(8192, most)))
        lo = max(1, _log_int(rng, max(1, hi // 16), hi))
        causal = rng.random() < 0.75
        window = sinks = 0
        if causal and rng.random() < 0.4:
            window, sinks = _log_int(rng, 8, max(9, hi)), rng.choice([0, 1, 4, 70])
        return _unnamed(_attend("", hq, hk, dim, seqs, lo, hi, dtype, causal, window, sinks, rng.random() < 0.7))
    if op == "rope":
        hk = rng.choice([1, 2, 4, 8, 16])
        hq = hk * rng.choice([1, 2, 4, 7])
        dim = rng.choice([64, 72, 80, 96, 128])
        rot = rng.choice([dim, dim, dim // 2])
        pairs, axes = rot // 2, rng.choice([1, 2, 3, 3])
        cuts = sorted(rng.sample(range(1, pairs), axes - 1)) + [pairs]
        sections = ",".join(str(b - a) for a, b in zip([0] + cuts, cuts))
        rows = _log_int(rng, 1, max(2, 80_000_000 // ((hq + hk) * dim)))
        return _unnamed(_rope("", rows, hq, hk, dim, rot, sections, dtype, rng.random() < 0.4, rng.random() < 0.4,
                              rng.random() < 0.7))
    if op == "norm":
        width = rng.choice([64, 768, 1024, 2048, 4096, 8192, rng.randint(33, 9000)])
        rows = _log_int(rng, 1, 33_000_000 // width)
        return _unnamed(_norm("", rows, width, rng.choice(["fp16", "bf16", "fp32"]),
                              rng.choice(["same", "same", "fp32", "none"]), rng.random() < 0.7))
    hi = _log_int(rng, 100, 2_000_000)
    lo = _log_int(rng, 1, hi)
    tensors = _log_int(rng, 1, min(600, max(2, 28_000_000 // hi)))
    return _unnamed(_clip("", tensors, lo, hi, rng.choice(["fp16", "bf16", "fp32"]), rng.random() < 0.5))


def _unnamed(case):
    del case["name"]
    return case


def _lengths(case):
    """Tokens of each sequence, or values of each gradient (these spread over their logarithm)."""
    if case["op"] == "attend":
        rng = random.Random("%(seqs)d %(lo)d %(hi)d" % case)
        return [rng.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
    rng = random.Random("%(tensors)d %(lo)d %(hi)d" % case)
    return [_log_int(rng, case["lo"], case["hi"]) for _ in range(case["tensors"])]


def _starts(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return at


def _sections(case):
    """The axis of every pair."""
    left = [int(s) for s in case["sections"].split(",")]
    if not case["turns"]:
        return [a for a, n in enumerate(left) for _ in range(n)]
    axis, a = [], 0
    while sum(left):
        if left[a]:
            left[a] -= 1
            axis.append(a)
        a = (a + 1) % len(left)
    return axis


def _pairs(n, case):
    """How many (row, token) pairs a sequence of n tokens has."""
    if not case["causal"]:
        return n * n
    w, s = case["window"], case["sinks"]
    if not w:
        return n * (n + 1) // 2
    return sum(min(p + 1, w) + min(s, max(0, p + 1 - w)) for p in range(n))


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "attend":
        lens, hq, hk, D = _lengths(case), case["hq"], case["hk"], case["dim"]
        T, pairs = sum(lens), sum(_pairs(n, case) for n in lens)
        # q, k, v in, o out; with the gradient do in, dq, dk, dv out; two products forward, five backward
        nbytes, flops = T * D * 2 * (2 * hq + 2 * hk), 4 * pairs * hq * D
        if case["train"]:
            nbytes, flops = nbytes + T * D * 2 * (2 * hq + 2 * hk), flops + 10 * pairs * hq * D
        return {"bytes": nbytes, "flops": flops}
    if case["op"] == "rope":
        n = case["rows"] * (case["hq"] + case["hk"])
        passes = 2 if case["train"] else 1
        return {"bytes": passes * n * case["dim"] * 4, "flops": passes * n * case["rot"] * 3}
    if case["op"] == "norm":
        n = case["rows"] * case["width"]
        par = 0 if case["affine"] == "none" else 2 * case["width"] * (4 if case["affine"] == "fp32" else size)
        if not case["train"]:
            return {"bytes": 2 * n * size + par, "flops": 8 * n}
        return {"bytes": 4 * n * size + 2 * par, "flops": 20 * n}  # x, dy in; y, dx out
    n = sum(_lengths(case))
    return {"bytes": n * (size + (4 if case["wide"] else size)), "flops": 3 * n}


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 1000003 + 29)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    dt = TYPES[case["dtype"]]
    st = {"case": case}
    if case["op"] == "attend":
        lens, hq, hk, D = _lengths(case), case["hq"], case["hk"], case["dim"]
        T = sum(lens)
        # one projection's output holds q, k and v of a token side by side; a few channels of a key head are
        # much larger than the rest, as trained models have them
        ks = torch.exp(0.5 * normal(hk, D))
        ks[:, torch.randperm(D, generator=g, device=dev)[:max(1, D // 32)]] *= 6.0
        qkv = normal(T, (hq + 2 * hk) * D)
        qkv[:, hq * D:(hq + hk) * D] *= ks.reshape(-1)
        qkv[:, :hq * D] *= (1.0 / ks).repeat_interleave(hq // hk, 0).reshape(-1)
        qkv = qkv.to(dt)
        st["q"] = qkv[:, :hq * D].view(T, hq, D)
        st["k"] = qkv[:, hq * D:(hq + hk) * D].view(T, hk, D)
        st["v"] = qkv[:, (hq + hk) * D:].view(T, hk, D)
        # gradients of tokens differ by orders of magnitude
        st["do"] = (normal(T, hq, D) * 10.0 ** (1.5 * normal(T, 1, 1).clamp(-2, 1) - 1.0)).to(dt)
        st["lens"] = lens
        if own:
            import mixed_precision_int8_amd as m8
            st["batch"] = m8.PackedRows(torch.tensor(_starts(lens), dtype=torch.int32, device=dev), T,
                                        max_len=max(lens))
    elif case["op"] == "rope":
        T, D, rot, axis = case["rows"], case["dim"], case["rot"], _sections(case)
        axes = max(axis) + 1
        qkv = normal(T, (case["hq"] + 2 * case["hk"]) * D).to(dt)
        st["q"] = qkv[:, :case["hq"] * D].view(T, case["hq"], D)
        st["k"] = qkv[:, case["hq"] * D:(case["hq"] + case["hk"]) * D].view(T, case["hk"], D)
        st["dq"], st["dk"] = normal(T, case["hq"], D).to(dt), normal(T, case["hk"], D).to(dt)
        reach = 6000
        # the first axis is time (it may be far), the others are places in a frame
        most = torch.tensor([reach] + [90] * (axes - 1), device=dev)
        st["pos"] = (torch.rand((T, axes), generator=g, device=dev) * most).to(torch.int32)
        f = 10000.0 ** (-2.0 * torch.arange(rot // 2, device=dev, dtype=torch.float64) / rot)
        angle = torch.arange(reach, device=dev, dtype=torch.float64)[:, None] * f
        st["table"] = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)
        st["axis"] = axis
        st["axis_dev"] = torch.tensor(axis, device=dev)
    elif case["op"] == "norm":
        N, K = case["rows"], case["width"]
        x = normal(N, K) * torch.exp(0.5 * normal(N, 1)) + 0.3 * normal(N, 1)
        x[:, torch.randperm(K, generator=g, device=dev)[:max(1, K // 500)]] *= 20.0  # outlier channels
        st["x"], st["dy"] = x.to(dt), (normal(N, K) * 0.1).to(dt)
        st["w"] = st["b"] = None
        if case["affine"] != "none":
            at = torch.float32 if case["affine"] == "fp32" else dt
            st["w"], st["b"] = (1.0 + 0.2 * normal(K)).to(at), (0.1 * normal(K)).to(at)
    else:
        lens = _lengths(case)
        flat = normal(sum(lens)).to(dt)
        # gradients of one backward pass, as they lie in memory (16-byte aligned), of different sizes
        st["grads"] = [(p * float(10.0 ** ((i * 7) % 5 - 3))).clone() for i, p in enumerate(flat.split(lens))]
        # what the optimizer reads: one buffer, every tensor's part at a multiple of 64 values
        at = _starts([-(-n // 64) * 64 for n in lens])
        st["flat"] = torch.zeros(at[-1], dtype=torch.float32 if case["wide"] else dt, device=dev)
        st["outs"] = [st["flat"][a:a + n] for a, n in zip(at, lens)]
        st["max_norm"], st["scale"] = 1.0, 1.0 / 64.0
        if own:
            import mixed_precision_int8_amd as m8
            st["set"] = m8.GradientSet(st["grads"], out=st["outs"])
    return st


# ---- the plain forms


def _visible(n, case, dev):
    i, j = torch.arange(n, device=dev)[:, None], torch.arange(n, device=dev)[None]
    if not case["causal"]:
        return torch.ones((n, n), dtype=torch.bool, device=dev)
    see = j <= i
    if case["window"]:
        see &= (j > i - case["window"]) | (j < case["sinks"])
    return see


def _plain_attend(st):
    case = st["case"]
    hq, hk, D, dt = case["hq"], case["hk"], case["dim"], TYPES[case["dtype"]]
    G, scale = hq // hk, 1.0 / math.sqrt(D)
    o, dq = torch.empty_like(st["do"]), torch.empty_like(st["do"])
    dk = torch.empty((len(st["do"]), hk, D), dtype=dt, device=o.device)
    dv = torch.empty_like(dk)
    at = 0
    for n in st["lens"]:
        rows = slice(at, at + n)
        at += n
        # [hk, G n, D]: the rows of a group side by side
        q = st["q"][rows].float().view(n, hk, G, D).permute(1, 2, 0, 3).reshape(hk, G * n, D)
        k, v = st["k"][rows].float().transpose(0, 1), st["v"][rows].float().transpose(0, 1)
        s = torch.matmul(q, k.transpose(1, 2)).mul_(scale)
        see = _visible(n, case, q.device)
        s.view(hk, G, n, n).masked_fill_(~see, -math.inf)
        p = s.sub_(s.amax(-1, keepdim=True)).exp_()
        p /= p.sum(-1, keepdim=True)
        out = torch.matmul(p, v)
        o[rows] = out.view(hk, G, n, D).permute(2, 0, 1, 3).reshape(n, hq, D).to(dt)
        if not case["train"]:
            continue
        do = st["do"][rows].float().view(n, hk, G, D).permute(1, 2, 0, 3).reshape(hk, G * n, D)
        dv[rows] = torch.matmul(p.transpose(1, 2), do).transpose(0, 1).to(dt)
        ds = torch.matmul(do, v.transpose(1, 2))
        ds.sub_((do * out).sum(-1, keepdim=True)).mul_(p).mul_(scale)
        dk[rows] = torch.matmul(ds.transpose(1, 2), q).transpose(0, 1).to(dt)
        dq[rows] = torch.matmul(ds, k).view(hk, G, n, D).permute(2, 0, 1, 3).reshape(n, hq, D).to(dt)
        del ds
    return {"o": o, "dq": dq, "dk": dk, "dv": dv} if case["train"] else {"o": o}


def _turn(x, cos, sin, case, dt):
    rot = case["rot"]
    x = x.float()
    if case["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1).to(dt)


def _plain_rope(st):
    case, dt, half = st["case"], TYPES[st["case"]["dtype"]], st["case"]["rot"] // 2
    at = st["pos"].long()[:, st["axis_dev"]]                                   # [T, pairs]
    cos = st["table"][:, :half].gather(0, at)[:, None]
    sin = st["table"][:, half:].gather(0, at)[:, None]
    out = {"q": _turn(st["q"], cos, sin, case, dt), "k": _turn(st["k"], cos, sin, case, dt)}
    if case["train"]:
        out["dq"], out["dk"] = _turn(st["dq"], cos, -sin, case, dt), _turn(st["dk"], cos, -sin, case, dt)
    return out


def _plain_norm(st):
    x, dt = st["x"].float(), st["x"].dtype
    x = x - x.mean(-1, keepdim=True)
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    x *= r
    w = None if st["w"] is None else st["w"].float()
    out = {"y": (x if w is None else x * w + st["b"].float()).to(dt)}
    if st["case"]["train"]:
        dy = st["dy"].float()
        if w is not None:
            out["dw"], out["db"] = (dy * x).sum(0).to(st["w"].dtype), dy.sum(0).to(st["w"].dtype)
            dy = dy * w
        dy = dy - dy.mean(-1, keepdim=True) - x * (dy * x).mean(-1, keepdim=True)
        out["dx"] = (dy * r).to(dt)
    return out


def _plain_clip(st):
    squares = torch.stack([p.double().square().sum() for p in st["grads"]])
    norm = (squares.sum().sqrt() * st["scale"]).float()
    f = (st["scale"] * (st["max_norm"] / (norm.double() + 1e-6)).clamp(max=1.0)).float()
    for p, o in zip(st["grads"], st["outs"]):
        o.copy_(p.float() * f)
    return {"norm": norm, "grads": st["flat"]}


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return {"attend": _plain_attend, "rope": _plain_rope, "norm": _plain_norm, "clip": _plain_clip}[op](state)
    import mixed_precision_int8_amd as m8
    if op == "attend":
        how = {"causal": case["causal"], "window": case["window"], "sinks": case["sinks"]}
        q, k, v = state["q"], state["k"], state["v"]
        o, lse = m8.llmint8_attention(state["batch"], q, k, v, **how)
        if not case["train"]:
            return {"o": o}
        dq, dk, dv = m8.llmint8_attention_backward(state["batch"], q, k, v, o, lse, state["do"], **how)
        return {"o": o, "dq": dq, "dk": dk, "dv": dv}
    if op == "rope":
        table, pos, axis = state["table"], state["pos"], state["axis"]
        q, k = m8.llmint8_rope(table, pos, axis, state["q"], state["k"], interleaved=case["interleaved"])
        if not case["train"]:
            return {"q": q, "k": k}
        dq, dk = m8.llmint8_rope(table, pos, axis, state["dq"], state["dk"], interleaved=case["interleaved"],
                                 inverse=True)
        return {"q": q, "k": k, "dq": dq, "dk": dk}
    if op == "norm":
        x, w, b = state["x"], state["w"], state["b"]
        y, stats = m8.llmint8_layer_norm(x, w, b, eps=EPS, stats=case["train"])
        if not case["train"]:
            return {"y": y}
        dx, dw, db = m8.llmint8_layer_norm_backward(state["dy"], x, stats, w)
        return {"y": y, "dx": dx} if w is None else {"y": y, "dw": dw, "db": db, "dx": dx}
    norm = m8.llmint8_grad_norm(state["set"], scale=state["scale"])
    m8.llmint8_grad_clip(state["set"], norm, state["max_norm"], scale=state["scale"])
    return {"norm": norm, "grads": state["flat"]}


# ---- the definitions in 64 bits


def _exact_attend(case, st):
    """Sequence by sequence and key/value head by head; the gradients are those of the graph of the forward."""
    hq, hk, D = case["hq"], case["hk"], case["dim"]
    G, at, parts = hq // hk, _starts(st["lens"]), []
    for b, n in enumerate(st["lens"]):
        i = torch.arange(n, device=st["q"].device)
        hidden = torch.zeros((n, n), dtype=torch.bool, device=i.device)
        if case["causal"]:
            back = i[:, None] - i[None]
            hidden |= back < 0
            if case["window"]:
                hidden |= (back >= case["window"]) & (i[None] >= case["sinks"])
        heads = []
        for h in range(hk):
            q = st["q"][at[b]:at[b + 1], h * G:(h + 1) * G].double().transpose(0, 1).contiguous()
            k, v = (st[x][at[b]:at[b + 1], h].double() for x in "kv")
            leaves = [t.requires_grad_(case["train"]) for t in (q, k, v)]
            with torch.enable_grad():
                s = torch.einsum("gic,jc->gij", q, k) / math.sqrt(D)
                o = torch.einsum("gij,jc->igc", torch.softmax(s.masked_fill(hidden, -math.inf), -1), v)
            grads = ()
            if case["train"]:
                grads = torch.autograd.grad(o, leaves, st["do"][at[b]:at[b + 1], h * G:(h + 1) * G].double())
                grads = (grads[0].transpose(0, 1), grads[1][:, None], grads[2][:, None])
            heads.append((o.detach(), *grads))
        parts.append([torch.cat(x, 1) for x in zip(*heads)])
    return dict(zip(("o", "dq", "dk", "dv"), (torch.cat(x) for x in zip(*parts))))


def _exact_rope(case, st):
    rot, half = case["rot"], case["rot"] // 2
    pos = st["pos"].long()
    factor = torch.empty((case["rows"], 1, half), dtype=torch.complex128, device=pos.device)
    for i, a in enumerate(st["axis"]):
        row = st["table"][pos[:, a]].double()
        factor[:, 0, i] = torch.complex(row[:, i], row[:, half + i])
    first = slice(0, rot, 2) if case["interleaved"] else slice(0, half)
    second = slice(1, rot, 2) if case["interleaved"] else slice(half, rot)

    def turned(x, f):
        y = x.double()
        z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * f
        y[..., first], y[..., second] = z.real, z.imag
        return y

    out = {n: turned(st[n], factor) for n in "qk"}
    if case["train"]:
        out.update({n: turned(st[n], factor.conj()) for n in ("dq", "dk")})
    return out


def _exact_norm(case, st):
    leaves = {"x": st["x"].double().requires_grad_()}
    if st["w"] is not None:
        leaves.update(w=st["w"].double().requires_grad_(), b=st["b"].double().requires_grad_())
    with torch.enable_grad():
        var, mean = torch.var_mean(leaves["x"], -1, unbiased=False, keepdim=True)
        y = (leaves["x"] - mean) / torch.sqrt(var + EPS)
        if st["w"] is not None:
            y = y * leaves["w"] + leaves["b"]
    out = {"y": y.detach()}
    if case["train"]:
        grads = torch.autograd.grad(y, list(leaves.values()), st["dy"].double())
        out.update({"d" + n: g for n, g in zip(leaves, grads)})
    return out


def _exact_clip(case, st):
    flat = torch.cat([p.double() for p in st["grads"]])
    norm = torch.linalg.vector_norm(flat) * st["scale"]
    flat = flat * (st["scale"] * min(1.0, st["max_norm"] / (float(norm) + 1e-6)))
    parts = [torch.nn.functional.pad(p, (0, -len(p) % 64)) for p in flat.split([p.numel() for p in st["grads"]])]
    return {"norm": norm, "grads": torch.cat(parts)}


def exact(case, seed):
    if work(case)["flops"] > 4e12:
        return None
    st = prepare(case, seed)
    return {"attend": _exact_attend, "rope": _exact_rope, "norm": _exact_norm, "clip": _exact_clip}[case["op"]](case, st)
