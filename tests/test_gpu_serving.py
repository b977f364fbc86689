"""GPU tests of the serving operators against 64-bit references: the append with rotation, the
attention over the paged cache, the int8 product, and a decode step that uses them together."""
import pytest
import torch

import ternary_weight_token_b200 as bn
from tests import serving_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def cuda(s):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}


def close(got, want, tol, what):
    err = (got.double().cpu() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float((err / tol)[bad].max())} times the bound")


# ------------------------------------------------------------------- attention

def run_attention(s, q, qh, scale=None, ws=None, out=None, stream=None):
    d = cuda(s)
    o = torch.full_like(q, 7.0) if out is None else out
    if ws is None:
        ws = bn.alloc_attention_workspace(s["M"], len(s["lens"]), qh, s["kvh"], s["D"])
        ws.fill_(0xFF)                                  # NaN and -1 everywhere
    torch.cuda.synchronize()
    bn.bitnet_attention(q, d["cu"], d["len"], d["table"], d["kc"], d["vc"], o, ws, scale=scale,
                        stream=stream)
    torch.cuda.synchronize()
    assert bn.bitnet_check_device_error() == bn.BITNET_OK
    return o


def check_attention(lens, qh, kvh, D, page, dtype, seed=0, scale=None, pad_rows=0,
                    fill=float("nan")):
    s = ref.batch(lens, page, kvh, D, seed=seed, pad_rows=pad_rows, fill=fill)
    q = torch.randn(s["M"], qh * D, generator=s["g"]).to(dtype)
    got = run_attention(s, q.cuda(), qh, scale)
    o, a, smax = ref.attention(s, q, qh, D ** -0.5 if scale is None else scale)
    rows = int(s["cu"][-1])
    close(got[:rows], o[:rows], ref.attention_tolerance(dtype, o, a, smax, D)[:rows], "attention")
    assert torch.all(got[rows:] == 7.0), "rows behind the last sequence changed"


DECODE = [
    ([(1, 1)], 20, 5, 128, 16),
    ([(1, 715)], 20, 5, 128, 64),
    ([(1, 64), (1, 65), (1, 63), (1, 1), (1, 129)], 20, 5, 128, 16),
    ([(1, 300)] * 3, 8, 8, 64, 48),
    ([(1, 257), (1, 33)], 8, 1, 64, 32),
    ([(1, 1000)], 20, 1, 128, 16),
    ([(1, 515), (2, 77), (1, 5)], 12, 4, 96, 16),
    ([(1, 130)], 4, 2, 256, 16),
    ([(1, 90), (1, 17)], 3, 1, 16, 16),
    ([(1, 90), (1, 17)], 6, 6, 80, 112),
    ([(1, 70001), (1, 3000)], 20, 5, 128, 128),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", DECODE, ids=str)
def test_attention_decode(case, dtype):
    check_attention(*case, dtype)


CHUNK = [
    ([(17, 17)], 20, 5, 128, 16),
    ([(128, 128)] * 2, 8, 8, 64, 16),
    ([(65, 130), (1, 400), (33, 33)], 20, 5, 128, 32),
    ([(40, 1000)], 20, 5, 128, 64),
    ([(130, 9000)], 8, 2, 128, 128),
    ([(5, 200), (0, 60), (64, 64)], 7, 1, 64, 16),
    ([(21, 50)], 12, 4, 96, 48),
    ([(21, 50)], 2, 1, 256, 16),
    ([(300, 333)], 4, 4, 32, 16),
    ([(700, 700), (257, 1300)], 20, 5, 128, 64),
    ([(511, 511), (3, 900), (129, 200)], 6, 6, 64, 16),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", CHUNK, ids=str)
def test_attention_chunks(case, dtype):
    check_attention(*case, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", [[(3, 0)], [(5, 2)], [(0, 10), (4, 1), (1, 0), (2, 40)],
                                  [(100, 30), (1, 20)]], ids=str)
def test_attention_rows_without_keys_are_zero(lens, dtype):
    check_attention(lens, 8, 2, 64, 16, dtype, pad_rows=3)
    check_attention(lens, 20, 5, 128, 16, dtype, pad_rows=3)


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0])
def test_attention_scales(scale):
    check_attention([(1, 200), (20, 90)], 8, 2, 64, 16, BF, scale=scale)
    check_attention([(40, 200), (150, 150)], 8, 2, 128, 16, BF, scale=scale)


def test_attention_large_scores_keep_the_running_maximum():
    """Scores of hundreds, rising along the keys, so that the maximum moves at every block."""
    for n, t in ((1, 900), (60, 900)):
        s = ref.batch([(n, t)], 16, 2, 64, seed=5, fill=float("nan"))
        q = torch.ones(n, 8 * 64).to(BF)
        used = s["table"][0, :-(-t // 16)].long()
        ramp = (torch.arange(len(used) * 16) * 0.5).view(-1, 1, 16, 1)
        s["kc"][used] = torch.where(ramp < t * 0.5, ramp, float("nan")).expand(
            -1, 2, 16, 64).to(BF)
        got = run_attention(s, q.cuda(), 8, 0.05)
        o, a, smax = ref.attention(s, q, 8, 0.05)
        close(got, o, ref.attention_tolerance(BF, o, a, smax, 64), "attention")


@pytest.mark.parametrize("D", [16, 48, 80, 112])
@pytest.mark.parametrize("page", [16, 48, 256])
def test_attention_chunks_of_other_head_widths(D, page):
    check_attention([(70, 170), (31, 31), (1, 400)], 6, 2, D, page, BF)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_long_history_of_a_chunk(dtype):
    """Few items over many keys: every one is cut into many shares."""
    check_attention([(40, 20011)], 8, 8, 64, 32, dtype)
    check_attention([(9, 6000), (90, 133)], 20, 1, 96, 16, dtype)
    check_attention([(300, 4000), (2, 2)], 20, 5, 128, 64, dtype)


@pytest.mark.parametrize("case", [
    ([(1, 1 + i % 9) for i in range(60)] + [(1500, 1500)], 64, 64, 64, 16),
    ([(300, 4000)] + [(2, 2 + i % 7) for i in range(30)], 20, 5, 128, 64),
    ([(1, 1 + 3 * i) for i in range(30)] + [(129, 300), (40, 0), (2, 140)], 20, 20, 128, 16),
    ([(0, 9), (33, 129)] * 40, 4, 4, 128, 32),
], ids=["decode among a prompt", "short after cut", "odd tiles", "empty between"])
def test_attention_many_short_items_on_the_tensor_cores(case):
    """CTAs run through many items in a row that have one row tile or one block."""
    for _ in range(3):
        check_attention(*case, BF)


@pytest.mark.parametrize("case", [
    ([(300, 9000)], 20, 5, 128, 64),
    ([(300, 9000), (2, 2), (40, 0), (40, 3000), (130, 5000)], 20, 5, 128, 32),
    ([(129, 7000), (100, 5500)], 8, 8, 128, 128),
    ([(33, 20000), (1, 30), (257, 4100)], 6, 2, 128, 16),
    ([(257, 9001), (64, 64), (500, 6100)], 12, 4, 96, 48),
], ids=str)
def test_attention_cut_items_repeat_bit_for_bit(case):
    """Equal shares: a CTA's part of one item is followed by others without a barrier between its
    warps, so every run has to give the bits of the first, which is compared with 64 bits."""
    lens, qh, kvh, D, page = case
    s = ref.batch(lens, page, kvh, D, seed=31, fill=float("nan"))
    q = torch.randn(s["M"], qh * D, generator=s["g"]).to(BF)
    o, a, smax = ref.attention(s, q, qh, D ** -0.5)
    d, qd = cuda(s), q.cuda()
    ws = bn.alloc_attention_workspace(s["M"], len(lens), qh, kvh, D)
    runs = torch.full((60, *q.shape), 7.0, dtype=BF, device="cuda")
    for out in runs:
        ws.fill_(0xFF)
        bn.bitnet_attention(qd, d["cu"], d["len"], d["table"], d["kc"], d["vc"], out, ws)
    torch.cuda.synchronize()
    assert bn.bitnet_check_device_error() == bn.BITNET_OK
    close(runs[0], o, ref.attention_tolerance(BF, o, a, smax, D), "attention")
    other = [i for i in range(len(runs)) if not torch.equal(runs[i], runs[0])]
    assert not other, f"runs {other} differ from the first"


ONE_KEY = [([(1, 300), (1, 2)], 20, 5, 128, 16), ([(1, 715)], 8, 1, 64, 64),   # 8 rows, 8 heads
           ([(3, 500), (2, 40)], 20, 5, 128, 16), ([(2, 90)], 8, 1, 256, 16),  # 16 rows
           ([(128, 128), (70, 333)], 8, 8, 64, 16), ([(40, 1000)], 20, 5, 128, 32),
           ([(1, 9000)], 20, 5, 128, 128), ([(33, 6000)], 4, 2, 96, 48)]


@pytest.mark.parametrize("lo,hi", [(4, 12), (0.25, 3)])
@pytest.mark.parametrize("case", ONE_KEY, ids=str)
def test_attention_fp32_holds_queries_and_probabilities_in_24_bits(case, lo, hi):
    """Two terms of q or of p in place of three pass the bound three times over (a CPU test of the
    bound shows it)."""
    lens, qh, kvh, D, page = case
    s, q, z = ref.one_key_scores(lens, page, qh, kvh, D, lo, hi, seed=50)
    got = run_attention(s, q.cuda(), qh, scale=1.0).double().cpu().view(s["M"], qh, D)
    pos = torch.cat([torch.arange(t - n, t) for n, t in lens])
    want = torch.where(pos[:, None] >= 1, torch.sigmoid(z), torch.zeros_like(z))[..., None]
    close(got, want.expand(-1, -1, D),
          (want * ref.one_key_tolerance(z)[..., None]).expand(-1, -1, D) + 1e-30, "one key")


COUNTS = [
    ([(1, 70001), (1, 3000)], 20, 5, 128, 128),
    ([(1, 1 + (i * 911) % 2500) for i in range(300)] + [(1, 30000)], 4, 1, 64, 32),
    ([(2, 1000), (1, 64), (1, 1), (2, 65), (1, 4097)], 20, 5, 128, 16),
    ([(1, 90), (1, 17), (1, 3001)], 6, 6, 80, 112),
    ([(4, 130), (4, 7000)], 4, 2, 256, 16),
    ([(300, 9000)], 20, 5, 128, 64),
    ([(300, 9000), (2, 2), (40, 0), (40, 3000), (130, 5000)], 20, 5, 128, 32),
    ([(33, 20000), (1, 30), (257, 4100)], 6, 2, 128, 16),
    ([(257, 9001), (64, 64), (500, 6100)], 12, 4, 96, 48),
    ([(40, 20011)], 8, 8, 64, 32),
    ([(130, 9000)], 8, 2, 128, 128),
    ([(700, 700), (257, 1300)], 20, 5, 128, 64),
    ([(21, 2050)], 2, 1, 256, 16),
    ([(1500, 1500)] + [(1, 1 + i % 9) for i in range(60)], 64, 64, 64, 16),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", COUNTS, ids=[str(c)[:60] for c in COUNTS])
def test_attention_counts_every_block_once(case, dtype):
    """Equal weights over one-hot values: sums are whole numbers, so what is left is the quotient's
    two roundings (2^-24 each, and one for the reciprocal) and the output's."""
    lens, qh, kvh, D, page = case
    s, want = ref.block_counts(lens, page, kvh, D, seed=60)
    q = torch.zeros(s["M"], qh * D, dtype=dtype, device="cuda")
    got = run_attention(s, q, qh).view(s["M"], qh, D)
    want = want[:, None].expand(-1, qh, -1)
    close(got, want, want * (3 * 2.0 ** -24 + (2.0 ** -8 if dtype == BF else 0.0)), "counts")


def test_attention_ten_new_tokens_each():
    """More than 16 rows a sequence, all in one tile; then 9 to 16 rows."""
    check_attention([(10, 500)] * 7, 20, 5, 128, 16, BF)
    check_attention([(3, 500 + 7 * i) for i in range(9)], 20, 5, 128, 16, BF)
    check_attention([(3, 500 + 7 * i) for i in range(9)], 20, 5, 128, 16, F32)


@pytest.mark.parametrize("n", [1, 3, 90])
def test_offsets_past_32_bits(n):
    """Pages whose elements lie past 2^31 in the caches."""
    kvh, D, page, qh = 5, 128, 16, 20
    pages = 2 ** 31 // (kvh * page * D) + 40
    s = ref.batch([(n, 300)], page, kvh, D, seed=12, spare=0)
    q, k, v = (torch.randn(n, h * D, generator=s["g"]).to(BF) for h in (qh, kvh, kvh))
    inv = torch.rand(D // 2, generator=s["g"])
    d = cuda(s)
    used = s["kc"].shape[0]
    big = {}
    for key in ("kc", "vc"):
        big[key] = torch.empty(pages, kvh, page, D, dtype=BF, device="cuda")
        big[key][pages - used:] = d[key]
    table = torch.where(d["table"] >= 0, d["table"] + (pages - used), d["table"])
    small_q, big_q = torch.empty_like(q, device="cuda"), torch.empty_like(q, device="cuda")
    args = (q.cuda(), k.cuda(), v.cuda(), inv.cuda(), d["cu"], d["len"])
    bn.bitnet_rope_append(*args, d["table"], d["kc"], d["vc"], small_q)
    bn.bitnet_rope_append(*args, table, big["kc"], big["vc"], big_q)
    assert torch.equal(small_q, big_q)
    for key in ("kc", "vc"):
        assert torch.equal(big[key][pages - used:], d[key])
    ws = bn.alloc_attention_workspace(n, 1, qh, kvh, D)
    o1, o2 = torch.empty_like(small_q), torch.empty_like(small_q)
    bn.bitnet_attention(small_q, d["cu"], d["len"], d["table"], d["kc"], d["vc"], o1, ws)
    bn.bitnet_attention(big_q, d["cu"], d["len"], table, big["kc"], big["vc"], o2, ws)
    assert torch.equal(o1, o2)
    assert bn.bitnet_check_device_error() == bn.BITNET_OK
    now = {**s, "kc": d["kc"].cpu(), "vc": d["vc"].cpu()}
    want, a, smax = ref.attention(now, small_q.cpu(), qh, D ** -0.5)
    close(o1, want, ref.attention_tolerance(BF, want, a, smax, D), "attention")


def test_attention_two_streams_at_once():
    """Calls with workspaces of their own may overlap."""
    cases = [ref.batch([(1, 9000), (1, 4000)], 16, 5, 128, seed=20),
             ref.batch([(300, 900)], 16, 5, 128, seed=21)]
    streams = [torch.cuda.Stream() for _ in cases]
    work = []
    for s in cases:
        q = torch.randn(s["M"], 2560, generator=s["g"]).to(BF).cuda()
        work.append((cuda(s), q, torch.empty_like(q),
                     bn.alloc_attention_workspace(s["M"], len(s["lens"]), 20, 5, 128)))
    alone = [run_attention(s, w[1], 20) for s, w in zip(cases, work)]
    for _ in range(10):
        for st, (d, q, o, ws) in zip(streams, work):
            bn.bitnet_attention(q, d["cu"], d["len"], d["table"], d["kc"], d["vc"], o, ws,
                                stream=st)
    torch.cuda.synchronize()
    for want, w in zip(alone, work):
        assert torch.equal(want, w[2])


def test_attention_many_sequences_cut_into_shares():
    lens = [(1, 1 + (i * 911) % 2500) for i in range(300)] + [(1, 30000)]
    check_attention(lens, 4, 1, 64, 32, BF)


def test_attention_many_sequences():
    lens = [(1 if i % 3 else 0, 1 + (i * 37) % 150) for i in range(400)]
    check_attention(lens, 4, 2, 64, 16, BF)


def test_attention_replays_follow_the_lengths():
    """A captured call serves a cache that grows between replays, and two captured calls may share
    one workspace in order."""
    lens = [(1, 2000), (1, 1500)]
    s = ref.batch(lens, 16, 5, 128, seed=3)
    q = torch.randn(2, 2560, generator=s["g"]).to(BF)
    d, qd = cuda(s), q.cuda()
    o1, o2 = torch.empty_like(qd), torch.empty_like(qd)
    ws = bn.alloc_attention_workspace(2, 2, 20, 5, 128)
    stream = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(stream):
        for o in (o1, o2):
            call = lambda: bn.bitnet_attention(qd, d["cu"], d["len"], d["table"], d["kc"],
                                               d["vc"], o, ws)
            call()
            stream.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                call()
            graphs.append(g)
    for t0, t1 in ((2000, 1500), (1, 1500), (700, 64)):
        d["len"].copy_(torch.tensor([t0, t1], dtype=torch.int32))
        o1.fill_(9.0)
        o2.fill_(9.0)
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        s["lens"] = [(1, t0), (1, t1)]
        o, a, smax = ref.attention(s, q, 20, 128 ** -0.5)
        tol = ref.attention_tolerance(BF, o, a, smax, 128)
        close(o1, o, tol, "first graph")
        close(o2, o, tol, "second graph")


def test_attention_calls_in_a_row_share_a_workspace():
    """Small and cut calls in turn, nothing between them: a call's plan and sums stay until its
    join has read them."""
    work, ws_m = [], 0
    for lens, page, seed in (([(1, 700), (2, 50)], 16, 17), ([(129, 9000), (257, 7000)], 32, 18),
                             ([(20, 300)], 16, 19)):
        s = ref.batch(lens, page, 5, 128, seed=seed)
        q = torch.randn(s["M"], 2560, generator=s["g"]).to(BF).cuda()
        work.append((cuda(s), q, run_attention(s, q, 20)))
        ws_m = max(ws_m, s["M"])
    ws = bn.alloc_attention_workspace(ws_m, 2, 20, 5, 128)
    outs = [[torch.full_like(q, 7.0) for _, q, _ in work] for _ in range(20)]
    torch.cuda.synchronize()
    for row in outs:
        for (d, q, _), o in zip(work, row):
            bn.bitnet_attention(q, d["cu"], d["len"], d["table"], d["kc"], d["vc"], o, ws)
    torch.cuda.synchronize()
    assert bn.bitnet_check_device_error() == bn.BITNET_OK
    for row in outs:
        for (_, _, want), o in zip(work, row):
            assert torch.equal(o, want)


def test_attention_same_bits_twice():
    s = ref.batch([(1, 5000), (3, 900)], 16, 5, 128, seed=8)
    q = torch.randn(4, 2560, generator=s["g"]).to(BF).cuda()
    assert torch.equal(run_attention(s, q, 20), run_attention(s, q, 20))


def test_attention_on_a_side_stream():
    s = ref.batch([(1, 5000), (9, 900)], 16, 5, 128, seed=9)
    q = torch.randn(10, 2560, generator=s["g"]).to(BF).cuda()
    want = run_attention(s, q, 20)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(run_attention(s, q, 20, stream=side), want)


@pytest.mark.parametrize("n", [1, 200])
def test_attention_reports_pages_out_of_range(n):
    s = ref.batch([(n, 300), (1, 40)], 16, 2, 64, seed=2)
    for bad in (-1, 1 << 20):
        d = cuda(s)
        d["table"][0, 3] = bad
        q = torch.randn(n + 1, 512, generator=s["g"]).to(BF)
        o = torch.empty(n + 1, 512, dtype=BF, device="cuda")
        ws = bn.alloc_attention_workspace(n + 1, 2, 8, 2, 64)
        bn.bitnet_attention(q.cuda(), d["cu"], d["len"], d["table"], d["kc"], d["vc"], o, ws)
        assert bn.bitnet_check_device_error() == bn.BITNET_ERR_INVALID_ARG
        assert bn.bitnet_check_device_error() == bn.BITNET_OK
        want, a, smax = ref.attention(s, q, 8, 0.125)    # the other sequence is unharmed
        close(o[n:], want[n:], ref.attention_tolerance(BF, want, a, smax, 64)[n:], "other")


@pytest.mark.parametrize("n", [1, 200])
def test_attention_reports_lengths_out_of_range(n):
    s = ref.batch([(n, 300)], 16, 2, 64, seed=2)
    q = torch.randn(n, 512, generator=s["g"]).to(BF).cuda()
    o = torch.empty_like(q)
    ws = bn.alloc_attention_workspace(n, 1, 8, 2, 64)
    for key, value in (("len", [100000]), ("len", [-5]), ("cu", [0, n + 7]), ("cu", [4, 2])):
        d = cuda(s)
        d[key] = torch.tensor(value, dtype=torch.int32, device="cuda")
        bn.bitnet_attention(q, d["cu"], d["len"], d["table"], d["kc"], d["vc"], o, ws)
        assert bn.bitnet_check_device_error() == bn.BITNET_ERR_INVALID_ARG
    assert bn.bitnet_check_device_error() == bn.BITNET_OK


# ---------------------------------------------------------------------- append

APPEND = [
    # lens, qh, kvh, D, page, rot
    ([(1, 1)], 20, 5, 128, 16, 128),
    ([(1, 1025), (1, 3), (1, 64)], 20, 5, 128, 64, 128),
    ([(7, 40), (0, 5), (33, 33)], 8, 8, 64, 16, 64),
    ([(3, 30), (50, 77)], 12, 4, 96, 48, 96),
    ([(5, 9)], 4, 1, 256, 16, 64),
    ([(5, 9), (17, 100001)], 3, 3, 16, 32, 16),
    ([(20, 21)], 6, 2, 80, 16, 32),
    ([(12, 900)], 2, 2, 64, 16, 0),
    ([(1500, 2000), (1000, 1000)], 8, 2, 128, 64, 128),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved,norm", [(False, False), (True, False), (False, True),
                                              (True, True)])
@pytest.mark.parametrize("case", APPEND, ids=str)
def test_rope_append(case, interleaved, norm, dtype):
    lens, qh, kvh, D, page, rot = case
    s = ref.batch(lens, page, kvh, D, seed=1, pad_rows=2)
    g, M = s["g"], s["M"]
    # one fused projection: strided rows
    qkv = torch.randn(M, (qh + 2 * kvh) * D + 8, generator=g).to(dtype)
    cuts = (qh * D, (qh + kvh) * D, (qh + 2 * kvh) * D)
    q, k, v = qkv[:, :cuts[0]], qkv[:, cuts[0]:cuts[1]], qkv[:, cuts[1]:cuts[2]]
    inv = (500000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / max(rot, 1))).float()
    qg = 1 + 0.2 * torch.randn(D, generator=g) if norm else None
    kg = None                                         # all ones
    d, f = cuda(s), qkv.cuda()
    out = torch.full((M, qh * D), 7.0, dtype=dtype, device="cuda")
    bn.bitnet_rope_append(f[:, :cuts[0]], f[:, cuts[0]:cuts[1]], f[:, cuts[1]:cuts[2]],
                          inv.cuda(), d["cu"], d["len"], d["table"], d["kc"], d["vc"], out,
                          rope=int(interleaved), head_norm=norm,
                          q_gain=None if qg is None else qg.cuda(), eps=1e-5)
    torch.cuda.synchronize()
    assert bn.bitnet_check_device_error() == bn.BITNET_OK
    kc, vc = s["kc"].double(), s["vc"].double()
    ktol = torch.zeros_like(kc)
    cu = s["cu"].tolist()
    for b, (n, t) in enumerate(lens):
        r = slice(cu[b], cu[b] + n)
        pos = torch.arange(t - n, t)
        want, size = ref.rope(q[r], qh, D, pos, inv, interleaved, norm, qg, 1e-5)
        close(out[r].view(n, qh, D), want, ref.rope_tolerance(dtype, want, size, norm), "q")
        want, size = ref.rope(k[r], kvh, D, pos, inv, interleaved, norm, kg, 1e-5)
        at = s["table"][b].long()[pos // page]
        kc[at, :, pos % page] = want
        ktol[at, :, pos % page] = ref.rope_tolerance(BF, want, size, norm)
        vc[at, :, pos % page] = v[r].reshape(n, kvh, D).to(BF).double()
    assert torch.all(out[cu[-1]:] == 7.0), "rows behind the last sequence changed"
    close(d["kc"], kc, ktol, "k cache")
    assert torch.equal(d["vc"].double().cpu(), vc), "v cache"


def test_rope_append_in_place_and_without_a_place():
    """Q_out may be Q; tokens at negative positions and padding rows are left out."""
    s = ref.batch([(6, 4), (2, 0), (1, 17)], 16, 2, 64, seed=4, pad_rows=1)
    M, g = s["M"], s["g"]
    q, k, v = (torch.randn(M, h * 64, generator=g).to(BF) for h in (8, 2, 2))
    inv = torch.rand(32, generator=g)
    d, qd = cuda(s), q.cuda()
    bn.bitnet_rope_append(qd, k.cuda(), v.cuda(), inv.cuda(), d["cu"], d["len"], d["table"],
                          d["kc"], d["vc"], qd)
    torch.cuda.synchronize()
    assert bn.bitnet_check_device_error() == bn.BITNET_OK
    want, tol = q.double(), torch.zeros(M, 512, dtype=torch.float64)
    kc = s["kc"].double()
    ktol = torch.zeros_like(kc)
    for r, (b, p) in {2: (0, 0), 3: (0, 1), 4: (0, 2), 5: (0, 3), 8: (2, 16)}.items():
        y, size = ref.rope(q[r:r + 1], 8, 64, torch.tensor([p]), inv, False, False, None, 0)
        want[r], tol[r] = y.view(-1), ref.rope_tolerance(BF, y, size, False).view(-1)
        y, size = ref.rope(k[r:r + 1], 2, 64, torch.tensor([p]), inv, False, False, None, 0)
        page = int(s["table"][b, p // 16])
        kc[page, :, p % 16], ktol[page, :, p % 16] = y[0], ref.rope_tolerance(BF, y, size, False)[0]
    close(qd, want, tol, "q in place")
    close(d["kc"], kc, ktol, "k cache")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 32])
def test_rope_append_passes_the_rest_of_a_head_as_it_is(rot, interleaved, dtype):
    """Elements past rot_dim keep their bits, infinities and negative zeros too."""
    qh, kvh, D, M = 4, 2, 96, 5
    s = ref.batch([(M, 20)], 16, kvh, D, seed=14)
    g = s["g"]
    q, k, v = (torch.randn(M, h, D, generator=g) for h in (qh, kvh, kvh))
    for x in (q, k):
        x[..., rot:].masked_fill_(torch.rand(M, x.shape[1], D - rot, generator=g) < 0.2, -0.0)
        x[..., rot:].masked_fill_(torch.rand(M, x.shape[1], D - rot, generator=g) < 0.2,
                                  float("inf"))
        x[..., rot:].masked_fill_(torch.rand(M, x.shape[1], D - rot, generator=g) < 0.2,
                                  -float("inf"))
    q, k, v = (x.to(dtype).cuda() for x in (q, k, v))
    d, out = cuda(s), torch.empty(M, qh * D, dtype=dtype, device="cuda")
    inv = torch.rand(rot // 2, generator=g).cuda()
    bn.bitnet_rope_append(q.view(M, -1), k.view(M, -1), v.view(M, -1), inv, d["cu"], d["len"],
                          d["table"], d["kc"], d["vc"], out, rope=int(interleaved))
    assert bn.bitnet_check_device_error() == bn.BITNET_OK

    def bits(x):
        return x.contiguous().view(torch.int16 if x.dtype == BF else torch.int32)
    assert torch.equal(bits(out.view(M, qh, D)[..., rot:]), bits(q[..., rot:]))
    pos = torch.arange(15, 20, device="cuda")
    now = d["kc"][d["table"][0].long()[pos // 16], :, pos % 16]
    assert torch.equal(bits(now[..., rot:]), bits(k[..., rot:].to(BF)))
    assert torch.isfinite(out.view(M, qh, D)[..., :rot]).all()


def test_outputs_beside_the_inputs_in_one_buffer():
    """Neighbours, and an output between the rows of its inputs, are no overlap."""
    M, qh, kvh, D = 3, 4, 2, 64
    s = ref.batch([(M, 40)], 16, kvh, D, seed=15)
    g = s["g"]
    rows = torch.randn(M, 8192, generator=g).to(BF).cuda()      # q, k, v and room per row
    q, k, v = rows[:, :256], rows[:, 256:384], rows[:, 384:512]
    spare = rows.view(-1)[512:512 + M * 256].view(M, 256)
    inv = torch.rand(32, generator=g).cuda()
    d, e = cuda(s), cuda(s)
    apart = torch.empty(M, 256, dtype=BF, device="cuda")
    bn.bitnet_rope_append(q, k, v, inv, d["cu"], d["len"], d["table"], d["kc"], d["vc"], apart)
    bn.bitnet_rope_append(q, k, v, inv, e["cu"], e["len"], e["table"], e["kc"], e["vc"], spare)
    assert torch.equal(spare, apart) and torch.equal(d["kc"], e["kc"])
    both = torch.empty(2 * M, 256, dtype=BF, device="cuda")
    both[:M] = apart
    ws = bn.alloc_attention_workspace(M, 1, qh, kvh, D)
    bn.bitnet_attention(both[:M], d["cu"], d["len"], d["table"], d["kc"], d["vc"], both[M:], ws)
    assert torch.equal(both[:M], apart)
    assert torch.equal(both[M:], run_attention({**s, "kc": d["kc"], "vc": d["vc"]}, apart, qh))


def test_rope_append_reports_pages_out_of_range():
    s = ref.batch([(4, 40), (1, 10)], 16, 2, 64, seed=4)
    q, k, v = (torch.randn(5, h * 64, generator=s["g"]).to(BF).cuda() for h in (8, 2, 2))
    inv = torch.rand(32, generator=s["g"]).cuda()
    for key, at, value in (("table", (0, 2), -1), ("table", (0, 2), 1 << 28), ("len", (0,), 9999)):
        d = cuda(s)
        before = d["kc"].clone()
        d[key][at] = value
        bn.bitnet_rope_append(q, k, v, inv, d["cu"], d["len"], d["table"], d["kc"], d["vc"],
                              torch.empty_like(q))
        assert bn.bitnet_check_device_error() == bn.BITNET_ERR_INVALID_ARG
        changed = (d["kc"] != before).any(dim=-1).any(dim=1).nonzero().tolist()
        assert changed == [[int(s["table"][1, 0]), 9]], "only the good sequence's slot"
    assert bn.bitnet_check_device_error() == bn.BITNET_OK


BAD_TABLES = [
    # lengths, cu_q, kv_len, sequences whose tokens are still appended
    ([(4, 40), (3, 10)], None, [-5, 10], [1]),
    ([(4, 40), (3, 10)], None, [40, 400000], [0]),
    ([(4, 40), (3, 10)], [0, 4, 14], None, [0]),
    ([(7, 40)], [0, 14], None, []),
    ([(7, 40)], [4, 2], None, []),
    ([(7, 40)], [-3, 7], None, []),
    ([(4, 40), (3, 10)], [0, 7, 4], None, [0]),
    ([(7, 40), (0, 10)], None, [40, -1], [0]),          # no row names that sequence
    ([(7, 40), (0, 10)], [0, 7, 9], None, [0]),
    ([(1, 5)] * 500 + [(0, 1)], None, [5] * 500 + [-1], range(500)),
]


@pytest.mark.parametrize("lens,cu,kv,good", BAD_TABLES, ids=range(len(BAD_TABLES)))
def test_rope_append_reports_rows_and_lengths_out_of_range(lens, cu, kv, good):
    """A sequence whose rows or length are out of range leaves the cache as it is, and is recorded,
    as the attention over the same tables does."""
    s = ref.batch(lens, 16, 2, 64, seed=4)
    M, g = s["M"], s["g"]
    q, k, v = (torch.randn(M, h * 64, generator=g).to(BF).cuda() for h in (8, 2, 2))
    d = cuda(s)
    kc, vc = d["kc"].clone(), d["vc"].clone()
    if cu is not None:
        d["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    if kv is not None:
        d["len"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
    bn.bitnet_rope_append(q, k, v, torch.rand(32, generator=g).cuda(), d["cu"], d["len"],
                          d["table"], d["kc"], d["vc"], torch.empty_like(q))
    assert bn.bitnet_check_device_error() == bn.BITNET_ERR_INVALID_ARG
    at, ln = d["cu"].tolist(), d["len"].tolist()
    slots = set()
    for b in good:
        for pos in range(ln[b] - (at[b + 1] - at[b]), ln[b]):
            slots.add((int(s["table"][b, pos // 16]), pos % 16))
    for now, before in ((d["kc"], kc), (d["vc"], vc)):
        changed = (now != before).any(dim=-1).any(dim=1).nonzero().tolist()
        assert {tuple(c) for c in changed} == slots
    ws = bn.alloc_attention_workspace(M, len(lens), 8, 2, 64)
    bn.bitnet_attention(q, d["cu"], d["len"], d["table"], d["kc"], d["vc"], torch.empty_like(q), ws)
    assert bn.bitnet_check_device_error() == bn.BITNET_ERR_INVALID_ARG
    assert bn.bitnet_check_device_error() == bn.BITNET_OK


def test_binding_refuses_wrong_tensors():
    """Types, shapes, layouts and devices are checked before anything is launched."""
    s = ref.batch([(2, 20), (1, 9)], 16, 2, 64, seed=1)
    d = cuda(s)
    q, k, v, o = (torch.zeros(3, h * 64, dtype=BF, device="cuda") for h in (8, 2, 2, 8))
    inv = torch.rand(32, device="cuda")
    ws = bn.alloc_attention_workspace(3, 2, 8, 2, 64)
    good = dict(Q=q, cu_q=d["cu"], kv_len=d["len"], block_table=d["table"], k_cache=d["kc"],
                v_cache=d["vc"], O=o, workspace=ws)
    bn.bitnet_attention(**good)
    bad = dict(Q=q[:, :500], cu_q=d["cu"].long(), kv_len=d["len"].float(), O=o.float(),
               block_table=d["table"][:1], k_cache=d["kc"][:, :, :, :32], workspace=ws.cpu(),
               v_cache=d["vc"][:2])
    for key, t in list(bad.items()) + [("cu_q", d["cu"][:2]), ("kv_len", d["len"].cpu()),
                                       ("Q", q.t().contiguous().t()), ("k_cache", d["kc"][0]),
                                       ("block_table", d["table"].t().contiguous().t())]:
        with pytest.raises(ValueError):
            bn.bitnet_attention(**{**good, key: t})
    good = dict(Q=q, K=k, V=v, inv_freq=inv, cu_q=d["cu"], kv_len=d["len"],
                block_table=d["table"], k_cache=d["kc"], v_cache=d["vc"], Q_out=o)
    for key, t in (("K", k.float()), ("K", q), ("V", v[:2]), ("Q", q.cpu()), ("Q_out", o[:, :64]),
                   ("inv_freq", inv.double()), ("q_gain", inv), ("k_gain", torch.ones(64)),
                   ("V", v.t().contiguous().t()), ("Q", q[:, None])):
        with pytest.raises(ValueError):
            bn.bitnet_rope_append(**{**good, key: t}, head_norm=True)
    xq, xs, wq, wsc, _ = (t.cuda() if isinstance(t, torch.Tensor) else t for t in codes(3, 5, 32, 0))
    y = torch.zeros(3, 5, device="cuda")
    good = dict(Xq=xq, x_scale=xs, Wq=wq, w_scale=wsc, Y=y)
    for key, t in (("Xq", xq.float()), ("Wq", wq[:, :16]), ("x_scale", xs[:2]), ("Y", y.t()),
                   ("w_scale", wsc.double()), ("Y", y.half()), ("residual", y.to(BF)),
                   ("residual", y.cpu()), ("epilogue", bn.BITNET_BF16), ("Wq", wq[0])):
        with pytest.raises(ValueError):
            bn.bitnet_linear_w8(**{**good, key: t})
    assert bn.bitnet_check_device_error() == bn.BITNET_OK


# ------------------------------------------------------------------ int8 product

W8 = [(1, 1, 16), (1, 128, 128), (3, 130, 144), (16, 257, 2560), (17, 64, 272), (33, 1000, 64),
      (64, 129, 6912), (65, 127, 512), (128, 384, 2560), (129, 96, 1040), (300, 333, 400),
      (513, 1031, 16384), (1, 128256, 256), (700, 2560, 2560), (5, 40, 16384), (9, 6912, 2560)]


def codes(M, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    xq = torch.randint(-127, 128, (M, K), generator=g, dtype=torch.int8)
    wq = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8)
    return xq, torch.rand(M, generator=g) * 50 + 5, wq, torch.rand(N, generator=g) * 900 + 50, g


@pytest.mark.parametrize("shape", W8, ids=str)
def test_linear_w8(shape):
    M, N, K = shape
    xq, xs, wq, ws, g = codes(M, N, K, 3)
    dev = [t.cuda() for t in (xq, xs, wq, ws)]
    acc, y = ref.linear_w8(xq, xs, wq, ws)
    for dtype in (torch.int32, F32, BF):
        out = torch.full((M, N), 7, dtype=dtype, device="cuda")
        bn.bitnet_linear_w8(*dev, out)
        if dtype == torch.int32:
            assert torch.equal(out.cpu().long(), acc)
        else:
            # the sum to fp32, two reciprocals, their product, the last product: 2^-24 each
            close(out, y, y.abs() * (5 * 2.0 ** -24 + (2.0 ** -8 if dtype == BF else 0)), "y")
    assert bn.bitnet_check_device_error() == bn.BITNET_OK


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("silu,in_place", [(True, None), (False, False), (True, False),
                                           (False, True)])
@pytest.mark.parametrize("shape", [(1, 200, 256), (37, 640, 512), (300, 333, 400)], ids=str)
def test_linear_w8_epilogues(shape, silu, in_place, dtype):
    M, N, K = shape
    xq, xs, wq, ws, g = codes(M, N, K, 4)
    res = None if in_place is None else torch.randn(M, N, generator=g).to(dtype)
    out = res.cuda() if in_place else torch.empty(M, N, dtype=dtype, device="cuda")
    r = None if res is None else out if in_place else res.cuda()
    bn.bitnet_linear_w8(*(t.cuda() for t in (xq, xs, wq, ws)), out, silu=silu, residual=r)
    _, y0 = ref.linear_w8(xq, xs, wq, ws)
    _, y = ref.linear_w8(xq, xs, wq, ws, silu, res)
    # 5 steps on y0; the SiLU carries them with |d silu / dy| <= 1.1 and y's own size, and adds an
    # exponential (2 ulp), a sum and a quotient (2 ulp); the residual sum one step of the result
    tol = y0.abs() * 2.0 ** -24 * (6 + (8 if silu else 0)) + y.abs() * 2.0 ** -24
    if dtype == BF:
        tol = tol + y.abs() * 2.0 ** -8
    close(out, y, tol, "epilogue")


def test_linear_w8_extreme_codes_are_exact():
    K = 16384
    xq = torch.full((2, K), -128, dtype=torch.int8, device="cuda")
    wq = torch.full((3, K), -128, dtype=torch.int8, device="cuda")
    wq[1] = 127
    out = torch.empty(2, 3, dtype=torch.int32, device="cuda")
    bn.bitnet_linear_w8(xq, torch.ones(2, device="cuda"), wq, torch.ones(3, device="cuda"), out)
    assert out.tolist() == [[K * 128 * 128, -K * 128 * 127, K * 128 * 128]] * 2


def test_linear_w8_takes_the_quantiser_s_codes():
    """Weights and activations through bitnet_quant_act, the output near the unquantised one."""
    g = torch.Generator().manual_seed(0)
    X, W = torch.randn(20, 512, generator=g), torch.randn(300, 512, generator=g) * 0.02
    xq, xs, rs = bn.alloc_quant(20, 512)
    wq, ws, _ = bn.alloc_quant(300, 512)
    bn.bitnet_quant_act(X.cuda(), xq, xs, rs)
    bn.bitnet_quant_act(W.cuda(), wq, ws)
    Y = torch.empty(20, 300, device="cuda")
    bn.bitnet_linear_w8(xq, xs, wq, ws, Y)
    _, y = ref.linear_w8(xq.cpu(), xs.cpu(), wq.cpu(), ws.cpu())
    close(Y, y, y.abs() * 5 * 2.0 ** -24, "y")
    # a code is off by half a step at most: |x| / 254 of the row's largest on each side
    dx, dw = X.abs().amax(1) / 254, W.abs().amax(1) / 254
    lim = (dx[:, None] * W.abs().sum(1)[None] + dw[None] * X.abs().sum(1)[:, None] +
           512 * dx[:, None] * dw[None]).double()
    close(Y, X.double() @ W.double().t(), lim + y.abs() * 2.0 ** -20, "against the fp product")


# ----------------------------------------------------------- a step of a block

@pytest.mark.parametrize("new", [1, 3])
def test_decode_step_of_a_block(new):
    """q/k/v projections -> append -> attention -> block tail -> 8-bit head on one stream, for
    three requests, each operator against 64 bits on the values it got, and again as a graph."""
    H, I, qh, kvh, D, vocab = 512, 1024, 8, 2, 64, 1000
    lens = [(new, 50 + new), (new, new), (new, 333)]
    s = ref.batch(lens, 16, kvh, D, seed=6)
    M, g = s["M"], s["g"]
    d = cuda(s)
    x = torch.randn(M, H, generator=g).to(BF).cuda()
    packed = {}
    for name, (n, k) in {"q": (H, H), "k": (kvh * D, H), "v": (kvh * D, H), "o": (H, H),
                         "gate": (I, H), "up": (I, H), "down": (H, I)}.items():
        P, gamma, ws = bn.alloc_packed(n, k)
        bn.bitnet_pack_weights((torch.randn(n, k, generator=g) * 0.02).cuda(), P, gamma, ws)
        packed[name] = (P, gamma)
    wq, wscale, _ = bn.alloc_quant(vocab, H)
    bn.bitnet_quant_act((torch.randn(vocab, H, generator=g) * 0.02).cuda(), wq, wscale)
    inv = (500000.0 ** (-torch.arange(D // 2, dtype=torch.float64) * 2 / D)).float().cuda()
    xq, xs, xr = bn.alloc_quant(M, H)
    q, k, v = (torch.empty(M, h * D, dtype=BF, device="cuda") for h in (qh, kvh, kvh))
    qr, o, y = torch.empty_like(q), torch.empty_like(q), torch.empty_like(x)
    yq, ys, yr = bn.alloc_quant(M, H)
    logits = torch.empty(M, vocab, device="cuda")
    aws = bn.alloc_attention_workspace(M, 3, qh, kvh, D)
    tws = bn.alloc_block_tail_workspace(M, H, I)

    def attend():
        bn.bitnet_quant_act(x, xq, xs, xr, prelude=bn.BITNET_PRELUDE_RMSNORM)
        bn.bitnet_linear_multi(xq, xs, xr, [packed[n][0] for n in "qkv"],
                               [packed[n][1] for n in "qkv"], H, [q, k, v])
        bn.bitnet_rope_append(q, k, v, inv, d["cu"], d["len"], d["table"], d["kc"], d["vc"], qr)
        bn.bitnet_attention(qr, d["cu"], d["len"], d["table"], d["kc"], d["vc"], o, aws)

    def finish():
        bn.bitnet_block_tail(o, x, *packed["o"], *packed["gate"], *packed["up"],
                             *packed["down"], y, tws)
        bn.bitnet_quant_act(y, yq, ys, yr, prelude=bn.BITNET_PRELUDE_RMSNORM)
        bn.bitnet_linear_w8(yq, ys, wq, wscale, logits)

    attend()
    finish()
    torch.cuda.synchronize()
    assert bn.bitnet_check_device_error() == bn.BITNET_OK
    now = {**s, "kc": d["kc"].cpu(), "vc": d["vc"].cpu()}
    want, a, smax = ref.attention(now, qr.cpu(), qh, D ** -0.5)
    close(o, want, ref.attention_tolerance(BF, want, a, smax, D), "attention")
    pos = torch.cat([torch.arange(t - n, t) for n, t in lens])
    want, size = ref.rope(q.cpu(), qh, D, pos, inv.cpu(), False, False, None, 0)
    close(qr.view(M, qh, D), want, ref.rope_tolerance(BF, want, size, False), "q")
    _, want = ref.linear_w8(yq.cpu(), ys.cpu(), wq.cpu(), wscale.cpu())
    close(logits, want, want.abs() * 5 * 2.0 ** -24, "logits")
    assert torch.isfinite(y.float()).all()

    first = (o.clone(), logits.clone())
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            attend()
    for t in (q, k, v, qr, o):
        t.fill_(float("nan"))
    torch.cuda.synchronize()
    graph.replay()
    finish()
    torch.cuda.synchronize()
    assert torch.equal(o, first[0]) and torch.equal(logits, first[1])


@pytest.mark.parametrize("between", ["append", "attention", "linear_w8"])
@pytest.mark.parametrize("M", [1, 5, 16])
def test_early_reading_calls_look_past_one_launch_at_most(M, between):
    """bitnet_linear with BITNET_LAUNCH_PDL_INPUTS reads its inputs while the launch before it runs.
    That launch may be one of the serving calls, which does not write them, behind the quantiser
    or the packing that does: each round has other activations and other weights."""
    K, N, rounds = 6912, 2560, 12
    g = torch.Generator().manual_seed(40 + M)
    W = [(torch.randn(N, K, generator=g) * 0.02).cuda() for _ in range(2)]
    X = (torch.randn(rounds, M, K, generator=g) * 3).cuda()
    s = ref.batch([(1, 70)] * M, 16, 5, 128, seed=41)
    d = cuda(s)
    q, k, v = (torch.randn(M, h * 128, generator=g).to(BF).cuda() for h in (20, 5, 5))
    qo, o = torch.empty_like(q), torch.empty_like(q)
    inv = torch.rand(64, generator=g).cuda()
    aws = bn.alloc_attention_workspace(M, M, 20, 5, 128)
    wq = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8).cuda()
    wsc, other = torch.rand(N, generator=g).cuda() + 1, torch.empty(M, N, device="cuda")
    P, gamma, pws = bn.alloc_packed(N, K)
    xq, xs, xr = bn.alloc_quant(M, K)
    xq2, xs2, _ = bn.alloc_quant(M, K)
    bn.bitnet_quant_act(X[0], xq2, xs2)

    def middle():
        if between == "append":
            bn.bitnet_rope_append(q, k, v, inv, d["cu"], d["len"], d["table"], d["kc"], d["vc"], qo)
        elif between == "attention":
            bn.bitnet_attention(q, d["cu"], d["len"], d["table"], d["kc"], d["vc"], o, aws)
        else:
            bn.bitnet_linear_w8(xq2, xs2, wq, wsc, other)

    def steps(flags, wait):
        out = torch.empty(rounds, 2, M, N, device="cuda")
        for i in range(rounds):
            bn.bitnet_pack_weights(W[i % 2], P, gamma, pws)
            wait()
            bn.bitnet_quant_act(X[i], xq, xs, xr)
            wait()
            middle()
            wait()
            bn.bitnet_linear(xq, xs, xr, P, gamma, K, out[i, 0], epilogue=bn.BITNET_F32 | flags)
            wait()
            bn.bitnet_pack_weights(W[1 - i % 2], P, gamma, pws)
            wait()
            middle()
            wait()
            bn.bitnet_linear(xq, xs, xr, P, gamma, K, out[i, 1], epilogue=bn.BITNET_F32 | flags)
            wait()
        torch.cuda.synchronize()
        assert bn.bitnet_check_device_error() == bn.BITNET_OK
        return out

    want = steps(0, torch.cuda.synchronize)
    for flags in (bn.BITNET_LAUNCH_PDL, bn.BITNET_LAUNCH_PDL_INPUTS):
        assert torch.equal(steps(flags, lambda: None), want)
