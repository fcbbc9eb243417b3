"""Attention of new tokens over a shared prefix and each request's own rows
(fa_decode) against the definition in 64 bits.

Tolerance (u: half a step of the input type): each weight is rounded to the
type before the product with V, so o is off by at most u A, A = the weighted
mean of |v|; the final rounding adds u |o|.  Scores are fp32 sums of at most
128 products (relative error below 2^-16 of the weight at these magnitudes),
exponentials are off by 2^-22: 4e-5 A.  L = log of an fp32 sum: 4e-5, plus
2^-23 |L|.
"""

from __future__ import annotations

import math

import pytest
import torch

from exact_attention_83_gb300 import fa

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
SLACK = 4e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fa.load_library()


def make(B, Hq, Hkv, Nq, D, P, S, lens, dtype="bf16", layout="bhnd", seed=0, poison=True):
    """Inputs; rows past each request's length hold NaN (they are never read)."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = DT[dtype]

    def heads(B, H, N):
        if layout == "bnhd":
            return torch.randn(B, N, H, D, generator=g, device=DEV).to(dt).permute(0, 2, 1, 3)
        return torch.randn(B, H, N, D, generator=g, device=DEV).to(dt)

    t = dict(q=heads(B, Hq, Nq), kp=heads(1, Hkv, P)[0], vp=heads(1, Hkv, P)[0], k=heads(B, Hkv, S),
             v=heads(B, Hkv, S), lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    if poison:
        for b, n in enumerate(lens):
            t["k"][b, :, max(n, 0):] = float("nan")
            t["v"][b, :, max(n, 0):] = float("nan")
    return t


def reference(t, causal=True, scale=None):
    B, Hq, Nq, D = t["q"].shape
    Hkv = t["k"].shape[1]
    G = Hq // Hkv
    scale = 1 / math.sqrt(D) if scale is None else scale
    o, a = (torch.zeros(B, Hq, Nq, D, dtype=torch.float64, device=DEV) for _ in range(2))
    lse = torch.full((B, Hq, Nq), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(t["lens"].tolist()):
        for tok in range(Nq):
            seen = max(0, min(n, n - Nq + tok + 1) if causal else n)
            keys = torch.cat([t["kp"].double(), t["k"][b, :, :seen].double()], 1)
            vals = torch.cat([t["vp"].double(), t["v"][b, :, :seen].double()], 1)
            if keys.shape[1] == 0:
                continue
            s = torch.einsum("hgd,hnd->hgn", t["q"][b, :, tok].double().reshape(Hkv, G, D), keys) * scale
            lse[b, :, tok] = torch.logsumexp(s, -1).reshape(Hq)
            p = torch.softmax(s, -1)
            o[b, :, tok] = torch.einsum("hgn,hnd->hgd", p, vals).reshape(Hq, D)
            a[b, :, tok] = torch.einsum("hgn,hnd->hgd", p, vals.abs()).reshape(Hq, D)
    return o, lse, a


def check(t, got, causal=True, scale=None, rows=None):
    o, lse = got
    ro, rl, ra = reference(t, causal, scale)
    u = torch.finfo(t["q"].dtype).eps / 2
    if rows is not None:
        o, lse, ro, rl, ra = (x[rows] for x in (o, lse, ro, rl, ra))
    none = torch.isneginf(rl)
    assert (torch.isneginf(lse) == none).all()
    assert (o[none] == 0).all()
    el = (lse.double() - rl).abs()[~none]
    assert (el <= SLACK + 2**-23 * rl[~none].abs()).all(), f"lse {float(el.max()):.3e}"
    lim = (u + SLACK) * ra + u * ro.abs() + torch.finfo(t["q"].dtype).smallest_normal
    err = (o.double() - ro).abs()
    assert (err <= lim).all(), f"o worst ratio {float((err / lim).nan_to_num(9e9).max()):.3f}"


def run(t, **kw):
    got = fa.attention_decode(t["q"], t["kp"], t["vp"], t["k"], t["v"], t["lens"], **kw)
    torch.cuda.synchronize()
    assert fa.device_status() == 0
    return got


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("layout", ["bhnd", "bnhd"])
@pytest.mark.parametrize("D", [16, 32, 64, 128])
def test_types_layouts_head_dims(D, layout, dtype):
    t = make(3, 8, 2, 1, D, 200, 70, [70, 1, 33], dtype, layout)
    check(t, run(t))


@pytest.mark.parametrize("P", [0, 1, 127, 128, 129, 255, 256, 257, 384, 1000, 5000])
def test_prefix_lengths(P):
    t = make(2, 4, 2, 1, 128, P, 40, [40, 3], seed=P)
    check(t, run(t))
    t = make(2, 4, 4, 1, 64, P, 40, [40, 0], "fp16", seed=P)
    check(t, run(t))


@pytest.mark.parametrize("S,lens", [(0, [0, 0, 0]), (1, [1, 0, 1]), (16, [15, 16, 0]), (17, [17, 16, 1]),
                                    (64, [63, 64, 33]), (65, [65, 64, 1]), (300, [129, 300, 0]),
                                    (2000, [2000, 1, 777]), (5001, [4999, 5001, 2])])
@pytest.mark.parametrize("P", [0, 130])
def test_own_lengths(S, lens, P):
    """Lengths of zero and one, ragged ends, clusters of several blocks."""
    t = make(3, 4, 2, 1, 128, P, S, lens, seed=S)
    check(t, run(t))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (16, 16), (12, 4), (5, 1), (8, 1), (20, 1), (40, 2)])
@pytest.mark.parametrize("Nq", [1, 2, 5, 16])
def test_grouped_heads_and_drafted_tokens(Hq, Hkv, Nq):
    """Row tiles of 16 with ragged ends: up to 320 rows of one request."""
    for causal in (True, False):
        t = make(2, Hq, Hkv, Nq, 64, 150, 90, [90, max(Nq - 1, 1)], seed=Hq * 17 + Nq)
        check(t, run(t, causal=causal), causal)


@pytest.mark.parametrize("B,Hq,Hkv,Nq", [(127, 1, 1, 1), (128, 1, 1, 1), (129, 1, 1, 1), (64, 4, 1, 1), (65, 4, 1, 1),
                                         (90, 6, 2, 1), (33, 8, 1, 2), (3, 1, 1, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_row_tiles_of_the_prefix(B, Hq, Hkv, Nq, D):
    """One row tile (two key streams), two, an odd number, ragged ends."""
    t = make(B, Hq, Hkv, Nq, D, 700, 20, [1 + i % 20 for i in range(B)], seed=B)
    check(t, run(t))


def test_many_ranges_of_a_long_prefix():
    t = make(1, 4, 1, 1, 128, 50000, 10, [10], seed=4)
    check(t, run(t))
    t = make(40, 8, 1, 1, 64, 20011, 10, [10] * 40, "fp16", seed=5)
    check(t, run(t))


@pytest.mark.parametrize("Nq", [1, 4])
def test_tokens_before_the_first_own_row(Nq):
    """More new tokens than own rows: the early ones see the prefix alone, or,
    without a prefix, nothing at all."""
    for P in (0, 100):
        t = make(3, 4, 2, Nq, 64, P, 8, [1, 0, 8], seed=P)
        check(t, run(t))


@pytest.mark.parametrize("gain", [0.0, 30.0, -30.0])
def test_extreme_scores(gain):
    """All scores equal, and scores of several hundred that grow along the keys
    (the running maximum moves at every tile) or fall."""
    t = make(2, 4, 1, 1, 64, 600, 300, [300, 150], seed=8)
    ramp = torch.linspace(0.1, 4, 600, device=DEV)[:, None]
    t["kp"] = (gain * ramp * torch.ones(64, device=DEV) / 8).to(torch.bfloat16)[None].contiguous()
    t["q"] = torch.ones_like(t["q"])
    check(t, run(t))


def test_infinite_values_in_masked_places():
    """Drafted tokens do not see later own keys: an infinite key there is a
    score of -inf for none of them."""
    t = make(1, 4, 2, 3, 64, 50, 10, [10], seed=3)
    t["k"][0, :, 9] = float("inf")
    o, lse = run(t)
    t2 = dict(t, k=t["k"].clone())
    t2["k"][0, :, 9] = 0
    o2, lse2 = run(t2)
    assert torch.equal(o[:, :, :2], o2[:, :, :2]) and torch.equal(lse[:, :, :2], lse2[:, :, :2])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,Hq", [(2, 2), (140, 2)])
def test_prefix_keys_with_scores_of_minus_infinity(B, Hq, D):
    """Keys that hold -inf where every query is positive weigh nothing: whole
    tiles and ranges of the prefix, its whole, and own rows too."""
    for dead in (300, 900):
        t = make(B, Hq, 1, 1, D, 900, 40, [1 + i % 40 for i in range(B)], seed=dead + B)
        t["q"][..., 3] = t["q"][..., 3].abs() + 0.5
        t["kp"][:, :dead, 3] = -math.inf
        t["k"][:, :, 20:30, 3] = -math.inf
        check(t, run(t))


def test_bad_lengths_are_reported_and_skipped():
    t = make(4, 4, 2, 1, 64, 100, 20, [20, 21, -1, 7], seed=1, poison=False)
    o = torch.full_like(t["q"], 7.0)
    lse = torch.full(t["q"].shape[:3], 7.0, device=DEV)
    ws = torch.empty(fa.decode_workspace_bytes(t["q"], t["kp"], t["k"]) // 4, device=DEV)
    fa.decode(t["q"], t["kp"], t["vp"], t["k"], t["v"], t["lens"], o, lse, workspace=ws)
    torch.cuda.synchronize()
    assert fa.device_status() == 13 and fa.device_status() == 0
    assert (o[1:3] == 7).all() and (lse[1:3] == 7).all()
    t["lens"] = torch.tensor([20, 0, 0, 7], dtype=torch.int32, device=DEV)
    check(t, (o, lse), rows=[0, 3])


def test_strided_views_and_scale():
    """Caches that are slices of wider buffers, outputs with strides, a scale."""
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    buf = torch.randn(3, 50, 2, 4, 64, generator=g, device=DEV).bfloat16()   # [B, S, k|v, Hkv, D]
    pre = torch.randn(77, 2, 4, 64, generator=g, device=DEV).bfloat16()
    t = dict(q=torch.randn(3, 1, 8, 192, generator=g, device=DEV).bfloat16()[..., 64:128].permute(0, 2, 1, 3),
             k=buf[:, :, 0].permute(0, 2, 1, 3), v=buf[:, :, 1].permute(0, 2, 1, 3),
             kp=pre[:, 0].transpose(0, 1), vp=pre[:, 1].transpose(0, 1),
             lens=torch.tensor([50, 2, 31], dtype=torch.int32, device=DEV))
    out = torch.full((3, 8, 1, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(3, 8, 1, device=DEV)
    ws = torch.full((fa.decode_workspace_bytes(t["q"], t["kp"], t["k"]) // 4,), float("nan"), device=DEV)
    fa.decode(t["q"], t["kp"], t["vp"], t["k"], t["v"], t["lens"], out[..., 64:], lse, True, 0.3, workspace=ws)
    torch.cuda.synchronize()
    check(t, (out[..., 64:], lse), scale=0.3)
    assert (out[..., :64] == 7).all()


def test_repeats_bitwise_and_on_a_side_stream():
    t = make(20, 8, 2, 1, 128, 3000, 200, [(37 * i) % 200 + 1 for i in range(20)], seed=2)
    a = run(t)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b = fa.attention_decode(t["q"], t["kp"], t["vp"], t["k"], t["v"], t["lens"])
    s.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_captured_graph_follows_lengths_and_values():
    t = make(5, 8, 2, 1, 64, 400, 100, [5, 1, 100, 50, 0], seed=2, poison=False)
    args = (t["q"], t["kp"], t["vp"], t["k"], t["v"], t["lens"])
    run(t)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fa.attention_decode(*args)
    for step in range(3):
        t["lens"] += 1
        t["lens"].clamp_(max=100)
        t["q"].copy_(torch.randn_like(t["q"]))
        graph.replay()
        torch.cuda.synchronize()
        check(t, got)


def test_two_calls_at_once():
    """Two streams, each with its own workspace."""
    ts = [make(30, 8, 2, 1, 128, 6000, 300, [300] * 30, seed=i) for i in range(2)]
    ref = [run(t) for t in ts]
    streams = [torch.cuda.Stream() for _ in ts]
    torch.cuda.synchronize()
    got = []
    for t, s in zip(ts, streams):
        with torch.cuda.stream(s):
            for _ in range(5):
                r = fa.attention_decode(t["q"], t["kp"], t["vp"], t["k"], t["v"], t["lens"])
            got.append(r)
    torch.cuda.synchronize()
    for a, b in zip(ref, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_own_rows_past_32_bit_offsets():
    """A cache whose last requests lie past 2^31 elements (8.6 GB each of K, V)."""
    B, Hkv, S, D = 33, 8, 131072, 128
    assert B * Hkv * S * D > 2**32
    k = torch.zeros(B, Hkv, S, D, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros(B, Hkv, S, D, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    small = make(1, 8, 8, 1, D, 64, 500, [500], seed=9)
    k[-1, :, :500], v[-1, :, :500] = small["k"][0], small["v"][0]
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    lens[-1] = 500
    q = small["q"].expand(B, 8, 1, D).contiguous()
    o, lse = fa.attention_decode(q, small["kp"], small["vp"], k, v, lens)
    torch.cuda.synchronize()
    check(small, (o[-1:], lse[-1:]))


@pytest.mark.parametrize("Hq,Hkv,Nq", [(4, 1, 1), (8, 2, 3), (20, 1, 2)])
@pytest.mark.parametrize("P", [0, 300])
def test_chunks_of_long_requests(P, Hq, Hkv, Nq):
    """Few requests with many rows: chunks that end inside, at and behind a
    length, lengths of zero and one among them, and lengths out of range."""
    S = 4096
    lens = [4096, 0, 1, 512, 513, 1023, 3000]
    for D, dtype in ((128, "bf16"), (64, "fp16")):
        t = make(7, Hq, Hkv, Nq, D, P, S, lens, dtype, seed=Nq)
        assert fa.decode_workspace_bytes(t["q"], t["kp"], t["k"]) > fa.decode_workspace_bytes(
            t["q"], t["kp"], t["k"][:, :, :64])        # it is cut into chunks
        check(t, run(t))
    o, lse = torch.full_like(t["q"], 7.0), torch.full(t["q"].shape[:3], 7.0, device=DEV)
    ws = torch.full((fa.decode_workspace_bytes(t["q"], t["kp"], t["k"]) // 4,), float("nan"), device=DEV)
    t["lens"][1], t["lens"][4] = -3, S + 1
    fa.decode(t["q"], t["kp"], t["vp"], t["k"], t["v"], t["lens"], o, lse, workspace=ws)
    torch.cuda.synchronize()
    assert fa.device_status() == 13
    assert all((x[i] == 7).all() for x in (o, lse) for i in (1, 4))
    t["lens"][1] = t["lens"][4] = 0
    check(t, (o, lse), rows=[0, 2, 3, 5, 6])


@pytest.mark.parametrize("B", [200, 256, 257, 300])
def test_more_requests_than_blocks(B):
    """Many more blocks than run at once, with equal lengths and lengths out of
    range among them."""
    S = 120
    lens = [(i * 37) % 121 for i in range(B)]
    t = make(B, 8, 8, 1, 64, 40, S, lens, "fp16", seed=B)
    check(t, run(t))
    t["lens"][3], t["lens"][B - 1] = 2**31 - 1, -2**31
    o, lse = fa.attention_decode(t["q"], t["kp"], t["vp"], t["k"], t["v"], t["lens"])
    torch.cuda.synchronize()
    assert fa.device_status() == 13
    t["lens"][3] = t["lens"][B - 1] = 0
    check(t, (o, lse), rows=[i for i in range(B) if i not in (3, B - 1)])


@pytest.mark.parametrize("B,Hkv,D,S", [(128, 3, 128, 1024), (100, 8, 64, 2100), (127, 4, 128, 1200)])
@pytest.mark.parametrize("P", [0, 40])
def test_requests_taken_by_falling_length(B, Hkv, D, S, P):
    lens = [(i * 37) % 121 for i in range(B)]
    lens[5], lens[70], lens[B - 1] = S, S - 1, S
    t = make(B, Hkv, Hkv, 1, D, P, S, lens, "fp16", seed=B)
    check(t, run(t))
    t["lens"][3], t["lens"][B - 2] = 2**31 - 1, -2**31
    o, lse = fa.attention_decode(t["q"], t["kp"], t["vp"], t["k"], t["v"], t["lens"])
    torch.cuda.synchronize()
    assert fa.device_status() == 13
    t["lens"][3] = t["lens"][B - 2] = 0
    check(t, (o, lse), rows=[i for i in range(B) if i not in (3, B - 2)])


@pytest.mark.parametrize("B,Hq,Hkv,D,P,S", [(64, 32, 8, 128, 16384, 1024), (128, 8, 8, 64, 9000, 1200),
                                            (33, 16, 8, 128, 20000, 2048)])
def test_own_rows_beside_a_long_prefix(B, Hq, Hkv, D, P, S):
    """Both kernels at once and a join behind them: requests without own rows, a
    bad length, and a second call right behind the first in the same workspace."""
    lens = [(i * 131) % (S + 1) for i in range(B)]
    lens[B - 1] = 0
    t = make(B, Hq, Hkv, 1, D, P, S, lens, seed=B, poison=False)
    args = (t["q"], t["kp"], t["vp"], t["k"], t["v"], t["lens"])
    ws = torch.full((fa.decode_workspace_bytes(t["q"], t["kp"], t["k"]) // 4,), math.nan, device=DEV)
    got = fa.attention_decode(*args, workspace=ws)
    q2 = t["q"].flip(0)
    again = fa.attention_decode(q2, *args[1:], workspace=ws)
    third = fa.attention_decode(*args, workspace=ws)
    torch.cuda.synchronize()
    assert fa.device_status() == 0
    assert torch.equal(got[0], third[0]) and torch.equal(got[1], third[1])
    check(t, got)
    check(dict(t, q=q2), again)
    t["lens"][0] = -1
    o, lse = torch.full_like(got[0], 7.0), torch.full_like(got[1], 7.0)
    fa.decode(*args, o, lse, workspace=ws)
    torch.cuda.synchronize()
    assert fa.device_status() == 13
    assert (o[0] == 7).all() and (lse[0] == 7).all()
    assert torch.equal(o[1:], got[0][1:]) and torch.equal(lse[1:], got[1][1:])


def test_captured_graph_of_chunks_and_one_workspace_for_two_graphs_in_turn():
    t = make(2, 4, 2, 1, 64, 200, 3000, [3000, 10], seed=2, poison=False)
    args = (t["q"], t["kp"], t["vp"], t["k"], t["v"], t["lens"])
    ws = torch.empty(fa.decode_workspace_bytes(t["q"], t["kp"], t["k"]) // 4, device=DEV)
    fa.attention_decode(*args, workspace=ws)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = fa.attention_decode(*args, workspace=ws)
        graphs.append((g, out))
    for step in range(4):
        t["lens"].copy_(torch.tensor([3000 - 900 * step, 10 + 990 * step], dtype=torch.int32))
        t["q"].copy_(torch.randn_like(t["q"]))
        g, out = graphs[step % 2]
        g.replay()
        torch.cuda.synchronize()
        check(t, out)
