"""64-bit references and inputs of the serving operators (paged cache, attention, int8 product):
plain torch on the CPU, from the definitions in include/bitnet.h."""
import torch

BF, F32 = torch.bfloat16, torch.float32


def batch(lens, page, kvh, D, seed=0, spare=3, table_extra=2, pad_rows=0, fill=None):
    """A paged batch: `lens` holds (new tokens, cached length) per sequence.  Pages are scattered,
    unused table entries -1, and with `fill` every slot beyond a sequence's length holds it."""
    g = torch.Generator().manual_seed(seed)
    pages = [-(-max(t, 0) // page) for _, t in lens]
    total = sum(pages) + spare
    perm = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(pages, default=0) + table_extra), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
    cu = [0]
    for n, _ in lens:
        cu.append(cu[-1] + n)
    kc = torch.randn(total, kvh, page, D, generator=g).to(BF)
    vc = torch.randn(total, kvh, page, D, generator=g).to(BF)
    if fill is not None:
        used = torch.zeros(total, page, dtype=torch.bool)
        for b, (_, t) in enumerate(lens):
            for j in range(max(t, 0)):
                used[table[b, j // page].long(), j % page] = True
        for c in (kc, vc):
            c.permute(0, 2, 1, 3)[~used] = fill
    return {"lens": lens, "M": cu[-1] + pad_rows, "cu": torch.tensor(cu, dtype=torch.int32),
            "len": torch.tensor([t for _, t in lens], dtype=torch.int32), "table": table,
            "kc": kc, "vc": vc, "page": page, "kvh": kvh, "D": D, "g": g}


def attention(s, q, qh, scale):
    """(o, tol basis a = sum p |v| / sum p, largest sum |q k| scale) in 64 bits; rows of no
    sequence are NaN."""
    D, kvh, page = s["D"], s["kvh"], s["page"]
    G = qh // kvh
    o = torch.full((s["M"], qh, D), float("nan"), dtype=torch.float64)
    a = torch.zeros_like(o)
    smax = 0.0
    cu = s["cu"].tolist()
    for b, (n, t) in enumerate(s["lens"]):
        if n == 0:
            continue
        x = q[cu[b]:cu[b] + n].double().view(n, kvh, G, D)
        used = s["table"][b, :-(-t // page)].long()
        k = s["kc"][used].double().transpose(0, 1).reshape(kvh, -1, D)[:, :t]
        v = s["vc"][used].double().transpose(0, 1).reshape(kvh, -1, D)[:, :t]
        z = torch.einsum("nhgd,htd->hgnt", x, k) * scale
        if t > 0:
            smax = max(smax, float(torch.einsum("nhgd,htd->hgnt", x.abs(), k.abs()).max()
                                   * abs(scale)))
        seen = torch.arange(t)[None, :] <= (t - n + torch.arange(n))[:, None]
        z = z.masked_fill(~seen, float("-inf"))
        m = z.amax(dim=-1, keepdim=True) if t > 0 else z.sum(dim=-1, keepdim=True)
        p = torch.where(seen, torch.exp(z - torch.where(m.isinf(), torch.zeros_like(m), m)),
                        torch.zeros_like(z))
        l = p.sum(dim=-1, keepdim=True)
        p = p / torch.where(l > 0, l, torch.ones_like(l))
        o[cu[b]:cu[b] + n] = torch.einsum("hgnt,htd->nhgd", p, v).reshape(n, qh, D)
        a[cu[b]:cu[b] + n] = torch.einsum("hgnt,htd->nhgd", p, v.abs()).reshape(n, qh, D)
    return o.view(s["M"], -1), a.view(s["M"], -1), smax


def attention_tolerance(dtype, o, a, smax, D):
    """Bounds of the roundings.  Scores: a matrix instruction adds 16 products with one
    truncation (2^-23 of the partial sums, at most smax), D / 16 times per term (one term of q for
    bf16, three for fp32); the error enters numerator and denominator.  exp2 adds 2^-21 with its
    argument's rounding.  Probabilities: bf16 2^-8, fp32 (three terms) 2^-24.  The output's rounding:
    2^-8 or 2^-24 of its value."""
    terms = 3 if dtype == F32 else 1
    score = 2 * 1.4427 * terms * (D / 16) * 2.0 ** -23 * smax + 2.0 ** -20
    if dtype == F32:
        return a * (2.0 ** -24 + score) + o.abs() * 2.0 ** -24 + 1e-30
    return a * (2.0 ** -8 + score) + o.abs() * 2.0 ** -8 + 1e-30


def rope(x, heads, D, pos, inv_freq, interleaved, norm, gain, eps):
    """(rotated heads, tolerance basis: the pair's length) in 64 bits."""
    y = x.double().reshape(-1, heads, D)
    if norm:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
        if gain is not None:
            y = y * gain.double()
    rot = 2 * inv_freq.numel()
    a = pos.double()[:, None] * inv_freq.double()[None, :]
    c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]
    out, size = y.clone(), y.abs()
    if rot:
        if interleaved:
            i, j = torch.arange(0, rot, 2), torch.arange(1, rot, 2)
        else:
            i, j = torch.arange(rot // 2), torch.arange(rot // 2, rot)
        out[..., i] = y[..., i] * c - y[..., j] * s
        out[..., j] = y[..., j] * c + y[..., i] * s
        size = size.clone()
        size[..., i] = size[..., j] = torch.hypot(y[..., i], y[..., j])
    return out, size


def rope_tolerance(dtype, out, size, norm):
    """fp32 steps: cosine and sine 2^-23 with the reduced angle's rounding, two products and a sum
    (2^-24 each) on the pair's length; the norm adds a sum of up to 256 squares (a lane's 16 and
    its 5 shuffle steps, halved by the root), a division, a root and two products: 2^-19.  Then
    the output's rounding."""
    step = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    return out.abs() * step + size * (2.0 ** -21 + (2.0 ** -19 if norm else 0.0)) + 1e-30


def linear_w8(xq, xs, wq, ws, silu=False, residual=None):
    acc = xq.double() @ wq.double().t()
    y = acc / (xs.double()[:, None] * ws.double()[None, :])
    if silu:
        y = y * torch.sigmoid(y)
    if residual is not None:
        y = y + residual.double()
    return acc.to(torch.int64), y


# ------------------------------------------------- inputs that show single steps

def one_key_scores(lens, page, qh, kvh, D, lo, hi, seed=0):
    """A paged batch and fp32 queries whose rows weigh two keys: position 0 with score 0 and value
    0, position 1 with a score z in [-hi, -lo] of 24 bits and value 1; the rest score -120 (weight
    2^-173) with value 0.  So o = 2^x / (1 + 2^x), x = z log2 e, in every element, each score is one
    product, and a term of q or of the probability that is left out shows at its full size.
    Returns (batch, q, z [M][qh]); rows before position 1 have o = 0."""
    s = batch(lens, page, kvh, D, seed=seed, fill=float("nan"))
    s["kc"].zero_()
    s["vc"].zero_()
    for b, (_, t) in enumerate(lens):
        used = s["table"][b, :-(-t // page)].long()
        s["kc"][used, :, :, 1] = 1.0
        s["kc"][used[0], :, 0, 1] = 0.0
        if t > 1:
            at = (used[1 // page], slice(None), 1 % page)
            s["kc"][at] = 0.0
            s["kc"][(*at, 0)] = 1.0
            s["vc"][at] = 1.0
    z = -(lo + (hi - lo) * torch.rand(s["M"], qh, generator=s["g"]))
    q = torch.zeros(s["M"], qh, D)
    q[..., 0], q[..., 1] = z, -120.0
    return s, q.view(s["M"], -1), z.double()


def one_key_tolerance(z):
    """Relative bound on o, in units of 2^-24.  z: its three products are added with a truncation
    of 2^-23 each (6), the factor and the product with it are rounded and so is the difference to
    the maximum (3).  p: exp2 within 2^-22 (4), the three products with v truncated (6), its own
    24 bits, the sums, the reciprocal and the last product (8)."""
    return (z.abs() * 9 + 18) * 2.0 ** -24


def terms(x, n):
    """What n bf16 terms of fp32 values hold."""
    x, out = x.float(), torch.zeros_like(x, dtype=torch.float64)
    for _ in range(n):
        t = x.to(BF).float()
        out += t.double()
        x = x - t
    return out


def block_counts(lens, page, kvh, D, seed=0):
    """A paged batch for queries of zeros: every key weighs the same, and the value of position j
    is 1 in channel (j // 64) % D.  So a row at position p has o[d] = (its positions of channel d)
    / (p + 1) with sums of whole numbers, and a block lost, doubled or taken from another page
    shows.  Returns (batch, o [M][D] in 64 bits)."""
    s = batch(lens, page, kvh, D, seed=seed, fill=float("nan"))
    rows = []
    for b, (n, t) in enumerate(lens):
        j = torch.arange(t)
        hot = torch.zeros(t, D, dtype=torch.float64)
        hot[j, (j // 64) % D] = 1.0
        if t:
            s["vc"][s["table"][b].long()[j // page], :, j % page] = hot[:, None].to(BF)
        upto = torch.cat([torch.zeros(1, D, dtype=torch.float64), hot.cumsum(0)])
        p1 = (t - n + torch.arange(n) + 1).clamp(min=0)
        rows.append(upto[p1] / p1.clamp(min=1)[:, None])
    return s, torch.cat(rows)
