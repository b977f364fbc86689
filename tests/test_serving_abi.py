"""CPU checks of the serving operators' boundary: bad arguments are refused on the host before any
device is touched, and the references of the GPU tests agree with hand-derived values."""
import ctypes

import pytest
import torch

import ternary_weight_token_b200 as bn
from tests import serving_ref as ref

FAKE, FAKE2 = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x20000)
ODD8, ODD2 = ctypes.c_void_p(0x10008), ctypes.c_void_p(0x10002)
INVALID, UNSUPPORTED = bn.BITNET_ERR_INVALID_ARG, bn.BITNET_ERR_UNSUPPORTED


def w8(**kw):
    a = dict(Xq=FAKE, xs=FAKE, Wq=FAKE, ws=FAKE, M=4, N=8, K=64, Y=FAKE2, epi=0, res=None)
    a.update(kw)
    return bn.library().bitnet_linear_w8(a["Xq"], a["xs"], a["Wq"], a["ws"], a["M"], a["N"],
                                         a["K"], a["Y"], a["epi"], a["res"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(K=17), INVALID), (dict(K=0), INVALID), (dict(K=16400), INVALID),
    (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(Xq=None), INVALID),
    (dict(ws=None), INVALID), (dict(xs=None), INVALID), (dict(Wq=ODD8), INVALID),
    (dict(Y=ODD8), INVALID), (dict(epi=7), INVALID), (dict(epi=0x40), INVALID),
    (dict(epi=bn.BITNET_LAUNCH_PDL), INVALID), (dict(epi=bn.BITNET_LAUNCH_PDL_INPUTS), INVALID),
    (dict(epi=bn.BITNET_I32 | bn.BITNET_EPI_SILU), UNSUPPORTED),
    (dict(epi=bn.BITNET_EPI_RESIDUAL), INVALID), (dict(res=FAKE), INVALID),
    (dict(M=0), bn.BITNET_OK), (dict(N=0), bn.BITNET_OK),
])
def test_linear_w8_rejects_bad_arguments(kw, code):
    assert w8(**kw) == code
    assert (bn.bitnet_last_error() == "") == (code == bn.BITNET_OK)


def append(**kw):
    a = dict(Q=FAKE, ldq=512, K=FAKE, ldk=128, V=FAKE, ldv=128, dtype=1, M=4, qh=8, kvh=2, D=64,
             inv=FAKE, rot=64, flags=0, qg=None, kg=None, eps=1e-5, batch=1, cu=FAKE, len=FAKE,
             table=FAKE, stride=4, kc=FAKE, vc=FAKE, pages=9, page=16, out=FAKE2)
    a.update(kw)
    return bn.library().bitnet_rope_append(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(dtype=5), dict(M=-1), dict(batch=-1), dict(qh=7), dict(kvh=0), dict(qh=1),
    dict(D=0), dict(D=24), dict(D=272), dict(rot=72), dict(rot=8), dict(rot=-16), dict(flags=4),
    dict(qg=FAKE), dict(kg=FAKE), dict(flags=2, eps=-1.0), dict(flags=2, eps=float("nan")),
    dict(ldq=504), dict(ldk=132), dict(ldv=64), dict(stride=0), dict(pages=0), dict(page=8),
    dict(page=24), dict(stride=1 << 27), dict(Q=None), dict(K=None), dict(V=None), dict(inv=None),
    dict(cu=None), dict(len=None), dict(table=None), dict(kc=None), dict(vc=None), dict(out=None),
    dict(Q=ODD8), dict(kc=ODD8), dict(out=ODD8), dict(cu=ODD2), dict(table=ODD2),
    dict(flags=2, qg=ODD2), dict(ldq=1024, out=FAKE), dict(M=1 << 30),
])
def test_rope_append_rejects_bad_arguments(kw):
    assert append(**kw) == INVALID
    assert bn.bitnet_last_error() != ""


def test_rope_append_empty_is_a_noop():
    assert append(M=0, Q=None) == bn.BITNET_OK
    assert append(batch=0, cu=None) == bn.BITNET_OK


def attend(**kw):
    a = dict(Q=FAKE, dtype=1, M=4, qh=8, kvh=2, D=64, scale=0.125, batch=1, cu=FAKE, len=FAKE,
             table=FAKE, stride=4, kc=FAKE, vc=FAKE, pages=9, page=16, out=FAKE2, ws=FAKE,
             bytes=bn.bitnet_attention_workspace_size(4, 1, 8, 2, 64))
    a.update(kw)
    return bn.library().bitnet_attention(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), INVALID), (dict(M=-1), INVALID), (dict(batch=-1), INVALID),
    (dict(qh=7), INVALID), (dict(kvh=0), INVALID), (dict(D=24), INVALID), (dict(D=272), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(stride=0), INVALID), (dict(pages=0), INVALID), (dict(page=8), INVALID),
    (dict(page=40), INVALID), (dict(stride=1 << 27), INVALID), (dict(Q=None), INVALID),
    (dict(cu=None), INVALID), (dict(len=None), INVALID), (dict(table=None), INVALID),
    (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(out=None), INVALID),
    (dict(Q=ODD8), INVALID), (dict(vc=ODD8), INVALID), (dict(out=ODD8), INVALID),
    (dict(len=ODD2), INVALID), (dict(ws=ODD8), INVALID), (dict(M=1 << 30), INVALID),
    (dict(ws=None), bn.BITNET_ERR_WORKSPACE), (dict(bytes=16), bn.BITNET_ERR_WORKSPACE),
    (dict(M=0, Q=None), bn.BITNET_OK), (dict(batch=0, cu=None), bn.BITNET_OK),
])
def test_attention_rejects_bad_arguments(kw, code):
    assert attend(**kw) == code


def test_attention_refuses_the_queries_buffer_as_output():
    assert attend(out=FAKE) == INVALID
    assert "buffer" in bn.bitnet_last_error()


@pytest.mark.parametrize("at", [0x10000 + 16, 0x10000 - 16, 0x10000 + 4 * 1024 - 16,
                                0x10000 - 4 * 1024 + 16])
def test_attention_refuses_outputs_that_overlap_the_queries(at):
    """4 rows of 1024 bytes on each side: every row is read while others are written."""
    assert attend(out=ctypes.c_void_p(at)) == INVALID
    assert "overlap" in bn.bitnet_last_error()


@pytest.mark.parametrize("kw", [
    dict(Q=0x20000 + 16), dict(Q=0x20000 - 16), dict(K=0x20000), dict(V=0x20000 + 4080),
    dict(K=0x20000 - 256 * 4 + 16), dict(V=0x20000 - 256 * 4 + 16),
    # rows 4096 bytes apart (2048 elements): the output lies between two, and reaches the next
    dict(Q=0x20000 - 1024, ldq=2048, K=0x20000 - 256 + 16, ldk=2048),
    dict(V=0x20000 - 2560, ldv=2048),
])
def test_rope_append_refuses_outputs_that_overlap_its_inputs(kw):
    """Output of 4 rows of 1024 bytes at 0x20000; keys and values have rows of 256 bytes."""
    kw = {k: ctypes.c_void_p(v) if k in "QKV" else v for k, v in kw.items()}
    assert append(**kw) == INVALID
    assert "overlap" in bn.bitnet_last_error()


def test_attention_workspace_serves_smaller_calls():
    size = bn.bitnet_attention_workspace_size
    for qh, kvh, D in ((20, 5, 128), (8, 8, 64), (4, 2, 256), (20, 1, 96)):
        sizes = [size(M, B, qh, kvh, D) for M in (1, 2, 16, 17, 100, 5000) for B in (1,)]
        assert sizes == sorted(sizes) and sizes[0] > 0
        assert size(64, 8, qh, kvh, D) >= size(64, 3, qh, kvh, D)
    assert size(-1, 1, 8, 2, 64) == 0 and size(1, 1, 7, 2, 64) == 0


def test_binding_refuses_host_tensors():
    t = torch.zeros((4, 64))
    with pytest.raises(ValueError):
        bn.bitnet_linear_w8(t.to(torch.int8), t[:, 0], t.to(torch.int8), t[:, 0], t)
    i = torch.zeros(2, dtype=torch.int32)
    c = torch.zeros((2, 1, 16, 16), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        bn.bitnet_attention(t, i, i[:1], i[None], c, c, t, t)
    with pytest.raises(ValueError):
        bn.bitnet_rope_append(t, t, t, t[0], i, i[:1], i[None], c, c, t)


@pytest.mark.parametrize("kw", [
    dict(epilogue=bn.BITNET_F32),
    dict(epilogue=bn.BITNET_F32 | bn.BITNET_EPI_RESIDUAL, residual=torch.zeros(4, 8)),
])
def test_linear_w8_refuses_a_silu_that_the_epilogue_leaves_out(kw):
    """The flags of an explicit epilogue are all that the call takes: a SiLU asked for beside one
    without it would be left out silently.  (A residual without its flag, or the flag without a
    residual, is refused by the library.)"""
    q, s = torch.zeros((4, 64), dtype=torch.int8), torch.ones(4)
    kw["silu"] = True
    with pytest.raises(ValueError, match="silu"):
        bn.bitnet_linear_w8(q, s, torch.zeros((8, 64), dtype=torch.int8), torch.ones(8),
                            torch.zeros(4, 8), **kw)


# ------------------------------------------------------ the references' own pins

def test_reference_attention_by_hand():
    """Two keys with scores 0 and ln 3: weights 1/4 and 3/4; the first row sees one key."""
    s = ref.batch([(2, 2)], 16, 1, 16, seed=0, fill=float("nan"))
    page = int(s["table"][0, 0])
    s["kc"][page, 0, :2] = 0
    s["kc"][page, 0, 1, 0] = 1
    s["vc"][page, 0, 0], s["vc"][page, 0, 1] = 2.0, 6.0
    q = torch.zeros(2, 16, dtype=torch.float64)
    q[:, 0] = torch.log(torch.tensor(3.0, dtype=torch.float64))
    o, a, smax = ref.attention(s, q, 1, 1.0)
    assert torch.allclose(o[0], torch.full((16,), 2.0, dtype=torch.float64), rtol=1e-14)
    assert torch.allclose(o[1], torch.full((16,), 5.0, dtype=torch.float64), rtol=1e-14)


def test_reference_rope_by_hand():
    """A quarter turn maps (x, y) to (-y, x); scores depend on the distance alone."""
    inv = torch.tensor([torch.pi / 2] * 8)
    x = torch.arange(16.0)[None]
    y, _ = ref.rope(x, 1, 16, torch.tensor([1]), inv, False, False, None, 0)
    assert torch.allclose(y[0, 0, :8], -x[0, 8:].double(), atol=1e-5)
    y, _ = ref.rope(x, 1, 16, torch.tensor([1]), inv, True, False, None, 0)
    assert torch.allclose(y[0, 0, 0::2], -x[0, 1::2].double(), atol=1e-5)
    f = torch.rand(8)
    a, b = torch.randn(1, 16), torch.randn(1, 16)
    dots = [(ref.rope(a, 1, 16, torch.tensor([p]), f, False, False, None, 0)[0] *
             ref.rope(b, 1, 16, torch.tensor([p + 7]), f, False, False, None, 0)[0]).sum()
            for p in (0, 1000)]
    assert torch.allclose(dots[0], dots[1], rtol=1e-9)


@pytest.mark.parametrize("lo,hi,what", [(4, 12, "q"), (0.25, 3, "p")])
def test_one_key_bound_tells_two_terms_from_three(lo, hi, what):
    """With two bf16 terms of the queries, or of the probabilities, some of 500 rows leave the
    bound; with three all stay far inside it."""
    s, q, z = ref.one_key_scores([(100, 130)], 16, 5, 1, 64, lo, hi)
    o, _, _ = ref.attention(s, q, 5, 1.0)
    want = torch.sigmoid(z)
    assert torch.allclose(o.view(100, 5, 64), want[..., None].expand(-1, -1, 64), rtol=1e-12)
    worst = {}
    for n in (2, 3):
        x = ref.terms(z, n) if what == "q" else z
        p = torch.exp(x)
        held = ref.terms(p, n) if what == "p" else p
        worst[n] = ((held / (1 + p) - want).abs() / want / ref.one_key_tolerance(z)).max()
    assert worst[2] > 3 and worst[3] < 0.1, worst


@pytest.mark.parametrize("t", [3000, 70001])
def test_block_counts_show_a_lost_block(t):
    """The 64-bit reference gives the counts, and a block of 64 less moves an element by more than
    the bf16 bound, a single key by more than the fp32 bound."""
    s, want = ref.block_counts([(2, t)], 128, 1, 128)
    o, _, _ = ref.attention(s, torch.zeros(2, 128), 1, 1.0)
    assert torch.allclose(o, want, rtol=1e-12)
    p = torch.tensor([t - 1, t], dtype=torch.float64)[:, None]
    count = want * p
    for lost, bound in ((64, 2.0 ** -8 + 3 * 2.0 ** -24), (1, 3 * 2.0 ** -24)):
        d = 5                                            # a channel that loses `lost` keys
        less = (count[:, d] - lost) / (p[:, 0] - lost)
        assert ((less - want[:, d]).abs() > 2 * want[:, d] * bound).all()
