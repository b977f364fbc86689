"""Cases for timing and comparing the serving operators beside the ternary projections.

Three operators, each in a plain form (elementary torch operations in 32 bits, angles in 64) and as
the calls a user makes of this package:

* ``append``     rotate the new tokens' queries and keys (optionally after an RMSNorm of each head)
                 and append keys and values to a paged cache: ``bitnet_rope_append``
* ``attention``  causal attention of the new tokens over the paged cache, from one token per
                 sequence to whole prompts: ``bitnet_attention``
* ``linear_w8``  the product of int8 activation codes with int8 weight codes, a scale per token and
                 per output channel, for the layers that are not ternary: ``bitnet_linear_w8``

Head layouts are the 2B model's (20 query and 5 key/value heads of 128), the 512-wide model's (8
heads of 64) and generic ones; widths are the 2B model's 2560 / 6912 and its 128256 vocabulary.
``own`` selects which form ``run`` computes.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32, "i32": torch.int32}
_THETA = 500000.0


def listed():
    return [
        # one new token of one conversation: the call whose latency counts
        dict(name="append 1 token", op="append", dtype="bf16", batch=1, new=1, kv=1024, ragged=0,
             qh=20, kvh=5, dim=128, page=64, interleaved=False, norm=False),
        # a prompt step of three requests on the 2B model's heads
        dict(name="append 4096 tokens", op="append", dtype="bf16", batch=3, new=1900, kv=3900,
             ragged=1, qh=20, kvh=5, dim=128, page=64, interleaved=False, norm=False),
        # fp32 activations of the 512-wide model, heads normalised, pairs interleaved, odd lengths
        dict(name="append fp32 head norms", op="append", dtype="f32", batch=9, new=117, kv=700,
             ragged=2, qh=8, kvh=8, dim=64, page=16, interleaved=True, norm=True),
        # one token of one conversation over a short history
        dict(name="attention 1 token", op="attention", dtype="bf16", batch=1, new=1, kv=715,
             ragged=0, qh=20, kvh=5, dim=128, page=64),
        # a decode step of a served batch with histories of mixed length
        dict(name="attention decode batch", op="attention", dtype="bf16", batch=32, new=1, kv=4096,
             ragged=3, qh=20, kvh=5, dim=128, page=16),
        # decode over long documents, two at once
        dict(name="attention decode long", op="attention", dtype="bf16", batch=2, new=1, kv=131071,
             ragged=4, qh=20, kvh=5, dim=128, page=128),
        # chunks of several prompts over caches that already hold part of them
        dict(name="attention chunks", op="attention", dtype="bf16", batch=4, new=512, kv=4000,
             ragged=5, qh=20, kvh=5, dim=128, page=32),
        # a whole prompt of the 2B model's context
        dict(name="attention prompt 4096", op="attention", dtype="bf16", batch=1, new=4096, kv=4096,
             ragged=0, qh=20, kvh=5, dim=128, page=64),
        # the 512-wide model's eight sequences of 128 tokens in fp32
        dict(name="attention fp32 8x128", op="attention", dtype="f32", batch=8, new=128, kv=128,
             ragged=0, qh=8, kvh=8, dim=64, page=16),
        # the output head for one token
        dict(name="w8 head 1 token", op="linear_w8", out="f32", m=1, n=128256, k=2560, silu=False,
             residual=False),
        # a small served batch through a square projection with its residual
        dict(name="w8 37 tokens residual", op="linear_w8", out="bf16", m=37, n=2560, k=2560,
             silu=False, residual=True),
        # a prompt through the wide projection
        dict(name="w8 4096 tokens", op="linear_w8", out="bf16", m=4096, n=6912, k=2560, silu=False,
             residual=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "linear_w8"])
    if op == "linear_w8":
        m = _log(rng, 1, 4096)
        k = 16 * _log(rng, 4, 432)
        n = min(_log(rng, 64, 130000), max(64, 4096 * 6912 * 2560 // (m * k)),
                max(64, 400_000_000 // k))
        out = rng.choice(["bf16", "f32", "i32"])
        return dict(op=op, out=out, m=m, n=n, k=k, silu=out != "i32" and rng.random() < 0.25,
                    residual=out != "i32" and rng.random() < 0.4)
    qh, kvh, dim = rng.choice([(20, 5, 128), (20, 5, 128), (8, 8, 64), (8, 2, 128), (12, 4, 96),
                               (8, 1, 64), (6, 6, 128)])
    case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), batch=_log(rng, 1, 48), new=1,
                kv=0, ragged=rng.randrange(1, 1 << 20), qh=qh, kvh=kvh, dim=dim,
                page=rng.choice([16, 32, 48, 64, 128]))
    if op == "append":
        case["new"] = _log(rng, 1, max(1, 4096 // case["batch"]))
        case["kv"] = case["new"] + _log(rng, 1, 4096)
        case["interleaved"] = rng.random() < 0.3
        case["norm"] = rng.random() < 0.4
        return case
    if rng.random() < 0.5:                       # a decode step (one to a few new tokens)
        case["new"] = rng.choice([1, 1, 1, 2, 5])
        case["kv"] = _log(rng, 8, max(9, min(131071, 160_000 // case["batch"])))
        case["kv"] = max(case["kv"], case["new"])
    else:                                        # a chunk of a prompt
        case["batch"] = min(case["batch"], 8)
        case["new"] = _log(rng, 6, 2048 // case["batch"])
        case["kv"] = case["new"] + _log(rng, 1, 2048)
    return case


def _lengths(case):
    """(new tokens, length after appending) of each sequence: whole numbers from the case alone."""
    if not case["ragged"]:
        return [case["new"]] * case["batch"], [case["kv"]] * case["batch"]
    r = random.Random(case["ragged"])
    new = [max(1, int(case["new"] * r.uniform(0.25, 1.0))) for _ in range(case["batch"])]
    kv = [max(n, int(case["kv"] * r.uniform(0.3, 1.0))) for n in new]
    return new, kv


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed) & 0x7FFFFFFF)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=dev) * std

    if case["op"] == "linear_w8":
        m, n, k = case["m"], case["n"], case["k"]
        s = {"op": "linear_w8", "case": dict(case)}
        # absmax codes of normal values: 127 at each row's largest value
        for key, rows in (("x", m), ("w", n)):
            v = normal(rows, k)
            scale = 127.0 / v.abs().amax(dim=1)
            s[key + "q"] = torch.round(v * scale[:, None]).clamp_(-128, 127).to(torch.int8)
            s[key + "s"] = scale * (50.0 if key == "w" else 1.0)      # weights of std 0.02
        s["res"] = normal(m, n).to(_DT[case["out"]]) if case["residual"] else None
        return s

    new, kv = _lengths(case)
    B, page, D, qh, kvh = case["batch"], case["page"], case["dim"], case["qh"], case["kvh"]
    dt = _DT[case["dtype"]]
    pages = [-(-t // page) for t in kv]
    total = sum(pages) + 3
    # the cache's pages in use, scattered; unused entries of the table are -1
    perm = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    table = torch.full((B, max(pages) + 1), -1, dtype=torch.int32, device=dev)
    at = 0
    for b in range(B):
        table[b, : pages[b]] = perm[at: at + pages[b]]
        at += pages[b]
    cu = [0]
    for t in new:
        cu.append(cu[-1] + t)
    M = cu[-1]
    s = {"op": case["op"], "case": dict(case), "m": M, "max_new": max(new), "max_kv": max(kv),
         "cu": torch.tensor(cu, dtype=torch.int32, device=dev),
         "len": torch.tensor(kv, dtype=torch.int32, device=dev), "table": table,
         "kc": normal(total, kvh, page, D).to(torch.bfloat16),
         "vc": normal(total, kvh, page, D).to(torch.bfloat16),
         "q": normal(M, qh * D).to(dt)}
    if case["op"] == "append":
        s["k"] = normal(M, kvh * D, std=2.0).to(dt)
        s["v"] = normal(M, kvh * D).to(dt)
        i = torch.arange(D // 2, dtype=torch.float64, device=dev)
        s["inv_freq"] = (_THETA ** (-2.0 * i / D)).float()
        s["qg"] = s["kg"] = None
        if case["norm"]:
            s["qg"] = 1.0 + 0.1 * normal(D)
            s["kg"] = 1.0 + 0.1 * normal(D)
    return s


# ------------------------------------------------------------------- plain forms

def _places(s):
    """For every row: its sequence, and its position in it."""
    r = torch.arange(s["m"], device=s["cu"].device, dtype=torch.int32)
    b = torch.searchsorted(s["cu"][1:], r, right=True)
    n = s["cu"][1:] - s["cu"][:-1]
    return b, (s["len"][b] - n[b] + r - s["cu"][b]).long()


def _rotate(x, heads, pos, s, gain):
    c = s["case"]
    D = c["dim"]
    x = x.float().view(-1, heads, D)
    if c["norm"]:
        x = x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + 1e-5) * gain
    a = pos.double()[:, None] * s["inv_freq"].double()[None, :]
    cos, sin = a.cos().float()[:, None, :], a.sin().float()[:, None, :]
    if c["interleaved"]:
        p, q = x[..., 0::2], x[..., 1::2]
        return torch.stack((p * cos - q * sin, q * cos + p * sin), dim=-1).flatten(-2)
    p, q = x[..., : D // 2], x[..., D // 2:]
    return torch.cat((p * cos - q * sin, q * cos + p * sin), dim=-1)


def _append_plain(s):
    c = s["case"]
    b, pos = _places(s)
    q = _rotate(s["q"], c["qh"], pos, s, s["qg"]).to(s["q"].dtype).view(s["m"], -1)
    k = _rotate(s["k"], c["kvh"], pos, s, s["kg"])
    page = s["table"][b, pos // c["page"]].long()
    slot = pos % c["page"]
    s["kc"][page, :, slot] = k.to(torch.bfloat16)
    s["vc"][page, :, slot] = s["v"].view(-1, c["kvh"], c["dim"]).to(torch.bfloat16)
    return {"q": q, "k_cache": s["kc"], "v_cache": s["vc"]}


def _attention_plain(s):
    c = s["case"]
    B, D, kvh, page = c["batch"], c["dim"], c["kvh"], c["page"]
    G, n, L = c["qh"] // kvh, s["max_new"], s["max_kv"]
    dev = s["q"].device
    table = s["table"][:, : -(-L // page)].clamp(min=0).long()
    k = s["kc"][table].float().transpose(1, 2).reshape(B, kvh, -1, D)     # keys by sequence
    v = s["vc"][table].float().transpose(1, 2).reshape(B, kvh, -1, D)
    i = torch.arange(n, device=dev)
    news = s["cu"][1:] - s["cu"][:-1]
    rows = (s["cu"][:-1, None] + i[None, :]).clamp(max=s["m"] - 1).long()
    q = s["q"].float()[rows].view(B, n, kvh, G, D).permute(0, 2, 3, 1, 4).reshape(B, kvh, G * n, D)
    z = (q * (1.0 / math.sqrt(D))) @ k.transpose(-1, -2)
    pos = (s["len"] - news)[:, None] + i[None, :]                          # [B][n]
    seen = torch.arange(k.shape[2], device=dev)[None, None, :] <= pos[:, :, None]
    z = z.view(B, kvh, G, n, -1).masked_fill(~seen[:, None, None], float("-inf"))
    z = z - z.amax(dim=-1, keepdim=True)
    p = z.exp()
    o = (p.view(B, kvh, G * n, -1) @ v).view(B, kvh, G, n, D) / p.sum(dim=-1, keepdim=True)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, -1)
    b, _ = _places(s)
    r = torch.arange(s["m"], device=dev) - s["cu"][b]
    return o[b, r].to(s["q"].dtype)


def _linear_w8_plain(s):
    c = s["case"]
    if c["out"] == "i32":       # whole numbers: sums may pass what 32-bit floats hold exactly
        return (s["xq"].double() @ s["wq"].double().t()).to(torch.int32)
    y = (s["xq"].float() @ s["wq"].float().t()) / (s["xs"][:, None] * s["ws"][None, :])
    if c["silu"]:
        y = y / (1.0 + torch.exp(-y))
    if s["res"] is not None:
        y = y + s["res"].float()
    return y.to(_DT[c["out"]])


# ---------------------------------------------------------- the package's calls

def _append_own(s):
    import ternary_weight_token_b200 as bn

    c = s["case"]
    q = torch.empty_like(s["q"])
    bn.bitnet_rope_append(
        s["q"], s["k"], s["v"], s["inv_freq"], s["cu"], s["len"], s["table"], s["kc"], s["vc"], q,
        rope=bn.BITNET_ROPE_INTERLEAVED if c["interleaved"] else bn.BITNET_ROPE_HALF,
        head_norm=c["norm"], q_gain=s["qg"], k_gain=s["kg"], eps=1e-5)
    return {"q": q, "k_cache": s["kc"], "v_cache": s["vc"]}


def _attention_own(s):
    import ternary_weight_token_b200 as bn

    c = s["case"]
    if "ws" not in s:           # kept from step to step, as a server does
        s["ws"] = bn.alloc_attention_workspace(s["m"], c["batch"], c["qh"], c["kvh"], c["dim"])
    o = torch.empty_like(s["q"])
    bn.bitnet_attention(s["q"], s["cu"], s["len"], s["table"], s["kc"], s["vc"], o, s["ws"])
    return o


def _linear_w8_own(s):
    import ternary_weight_token_b200 as bn

    c = s["case"]
    y = torch.empty((c["m"], c["n"]), dtype=_DT[c["out"]], device=s["xq"].device)
    bn.bitnet_linear_w8(s["xq"], s["xs"], s["wq"], s["ws"], y, silu=c["silu"], residual=s["res"])
    return y


def run(state):
    op = state["op"]
    if own:
        if op == "append":
            return _append_own(state)
        return _attention_own(state) if op == "attention" else _linear_w8_own(state)
    if op == "append":
        return _append_plain(state)
    return _attention_plain(state) if op == "attention" else _linear_w8_plain(state)


# ------------------------------------------------------------------ work and values

def work(case):
    if case["op"] == "linear_w8":
        m, n, k = case["m"], case["n"], case["k"]
        size = 2 if case["out"] == "bf16" else 4
        return {"bytes": m * k + n * k + 4 * (m + n) + m * n * size * (2 if case["residual"] else 1),
                "flops": 2 * m * n * k}
    new, kv = _lengths(case)
    M, D, qh, kvh = sum(new), case["dim"], case["qh"], case["kvh"]
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "append":
        return {"bytes": M * D * (2 * qh * size + 2 * kvh * (size + 2)) + 4 * M,
                "flops": M * D * (qh + kvh) * (7 if case["norm"] else 3)}
    pairs = sum(n * t - n * (n - 1) // 2 for n, t in zip(new, kv))
    return {"bytes": 2 * M * qh * D * size + 4 * sum(kv) * kvh * D,
            "flops": 4 * pairs * qh * D}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear_w8":
        if case["out"] == "i32":
            return None
        out = []
        x = s["xq"].double()
        for j in range(0, case["n"], 16384):
            y = torch.einsum("mk,nk->mn", x, s["wq"][j: j + 16384].double())
            y = y / s["xs"].double()[:, None] / s["ws"][j: j + 16384].double()[None, :]
            if case["silu"]:
                y = y * torch.sigmoid(y)
            if s["res"] is not None:
                y = y + s["res"][:, j: j + 16384].double()
            out.append(y)
        return torch.cat(out, dim=1)
    new, kv = _lengths(case)
    D, qh, kvh, page = case["dim"], case["qh"], case["kvh"], case["page"]
    if case["op"] == "append":
        q_rows, at = [], 0
        kc, vc = s["kc"].double(), s["vc"].double()
        f = s["inv_freq"].double()
        for b, (n, t) in enumerate(zip(new, kv)):
            pos = torch.arange(t - n, t, device="cuda")
            turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                               torch.outer(pos.double(), f))[:, None, :]
            done = []
            for x, heads, gain in ((s["q"], qh, s["qg"]), (s["k"], kvh, s["kg"])):
                y = x[at: at + n].double().reshape(n, heads, D)
                if case["norm"]:
                    y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / D + 1e-5) * gain.double()
                if case["interleaved"]:
                    z = torch.view_as_complex(y.reshape(n, heads, D // 2, 2).contiguous()) * turn
                    done.append(torch.view_as_real(z).reshape(n, heads, D))
                else:
                    z = torch.complex(y[..., : D // 2], y[..., D // 2:]) * turn
                    done.append(torch.cat((z.real, z.imag), dim=-1))
            q_rows.append(done[0].reshape(n, -1))
            where = s["table"][b].long()[pos // page]
            kc[where, :, pos % page] = done[1]
            vc[where, :, pos % page] = s["v"][at: at + n].double().reshape(n, kvh, D)
            at += n
        return {"q": torch.cat(q_rows), "k_cache": kc, "v_cache": vc}
    out = torch.empty(s["m"], qh, D, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, t) in enumerate(zip(new, kv)):
        used = s["table"][b, : -(-t // page)].long()
        for h in range(kvh):
            k = s["kc"][used, h].reshape(-1, D)[:t].double()
            v = s["vc"][used, h].reshape(-1, D)[:t].double()
            for g in range(h * (qh // kvh), (h + 1) * (qh // kvh)):
                x = s["q"][at: at + n].view(n, qh, D)[:, g].double()
                z = torch.einsum("nd,td->nt", x, k) / math.sqrt(D)
                if n > 1:
                    hide = torch.ones(n, t, dtype=torch.bool, device="cuda").triu(t - n + 1)
                    z = z.masked_fill(hide, float("-inf"))
                out[at: at + n, g] = torch.softmax(z, dim=-1) @ v
        at += n
    return out.view(s["m"], qh * D)
