"""Packed sequences behind one shared prefix (fa_fwd_prefix / fa_bwd_prefix)
against the definition in 64 bits, forward and gradients.

Tolerance (u: half a step of the input type; 0 for fp32), elementwise, from
magnitude sums of the terms of each product:
 * o: each weight is rounded to the type before P V: u A with A = sum P |v|,
   then the result: u |o|;
 * the gradients take P and dS = P (dP - Delta) rounded to the type (u of their
   magnitudes M), and Delta is formed from the rounded o: |dO| u |o| summed over
   d, carried through P; then the result's own rounding;
 * fp32 arithmetic: scores are sums of at most 128 products, exponentials off by
   2^-22; 6e-5 of the magnitudes covers chains of thousands of additions here.
"""

from __future__ import annotations

import math

import pytest
import torch

from exact_attention_83_gb300 import fa

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SLACK = 6e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fa.load_library()
    fa.set_path(fa.FA_PATH_AUTO)
    yield
    fa.set_path(fa.FA_PATH_AUTO)


def make(lq, lk, Hq, Hkv, D, P, dtype="bf16", seed=0, lead=0, tail=0):
    """Inputs with `lead` rows before the first and `tail` behind the last
    sequence, which hold NaN."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = DT[dtype]

    def packed(lens, H):
        t = torch.full((lead + sum(lens) + tail, H, D), float("nan"), device=DEV, dtype=dt)
        t[lead:lead + sum(lens)] = torch.randn(sum(lens), H, D, generator=g, device=DEV).to(dt)
        return t

    def cu(lens):
        return torch.tensor([lead + sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=DEV)

    return dict(q=packed(lq, Hq), k=packed(lk, Hkv), v=packed(lk, Hkv), do=packed(lq, Hq),
                kp=torch.randn(P, Hkv, D, generator=g, device=DEV).to(dt),
                vp=torch.randn(P, Hkv, D, generator=g, device=DEV).to(dt), cq=cu(lq), ck=cu(lk),
                mq=max(max(lq), 1), mk=max(max(lk), 1))


def reference(t, causal, scale=None, rounded_delta=True):
    """Values and magnitudes, {name: (value, bound without the final rounding)}."""
    Tq, Hq, D = t["q"].shape
    Tk, Hkv, _ = t["k"].shape
    P, G = t["kp"].shape[0], Hq // Hkv
    scale = 1 / math.sqrt(D) if scale is None else scale
    dt = t["q"].dtype
    u = torch.finfo(dt).eps / 2 if dt != torch.float32 else 0.0
    f = dict(dtype=torch.float64, device=DEV)
    val = dict(o=torch.zeros(Tq, Hq, D, **f), lse=torch.full((Hq, Tq), -math.inf, **f), dq=torch.zeros(Tq, Hq, D, **f),
               dk=torch.zeros(Tk, Hkv, D, **f), dv=torch.zeros(Tk, Hkv, D, **f), dkp=torch.zeros(P, Hkv, D, **f),
               dvp=torch.zeros(P, Hkv, D, **f))
    bnd = {n: torch.zeros_like(x) for n, x in val.items()}
    cq, ck = t["cq"].tolist(), t["ck"].tolist()
    for b in range(len(cq) - 1):
        r, c = slice(cq[b], cq[b + 1]), slice(ck[b], ck[b + 1])
        nq, nk = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
        if nq == 0:
            continue
        for h in range(Hq):
            hk = h // G
            q, do = t["q"][r, h].double(), t["do"][r, h].double()
            keys = torch.cat([t["kp"][:, hk].double(), t["k"][c, hk].double()])
            vals = torch.cat([t["vp"][:, hk].double(), t["v"][c, hk].double()])
            if keys.shape[0] == 0:
                continue
            s = q @ keys.T * scale
            if causal:
                i, j = torch.arange(nq, device=DEV)[:, None], torch.arange(nk, device=DEV)[None]
                s[:, P:] = s[:, P:].masked_fill(j > i, -math.inf)
            lse = torch.logsumexp(s, -1)
            none = torch.isneginf(lse)
            p = torch.where(none[:, None], 0.0, torch.exp(s - torch.where(none, 0.0, lse)[:, None]))
            o = p @ vals
            val["o"][r, h], val["lse"][h, r] = o, lse
            bnd["o"][r, h] = (u + SLACK) * (p @ vals.abs())
            dp = do @ vals.T
            delta = (do * o).sum(-1, keepdim=True)
            # Delta from the rounded o: u |o| and the product error, per element
            ddelta = (do.abs() * (bnd["o"][r, h] + u * o.abs())).sum(-1, keepdim=True)
            ds = p * (dp - delta)
            mds = p * (do.abs() @ vals.abs().T + (do * o).abs().sum(-1, keepdim=True))
            eds = u * ds.abs() + SLACK * mds + (p * ddelta if rounded_delta else 0.0)
            val["dq"][r, h] = ds @ keys * scale
            bnd["dq"][r, h] = eds @ keys.abs() * scale
            dk, ek = ds.T @ q * scale, eds.T @ q.abs() * scale
            dv, ev = p.T @ do, (u + SLACK) * (p.T @ do.abs())
            val["dkp"][:, hk] += dk[:P]; bnd["dkp"][:, hk] += ek[:P]
            val["dvp"][:, hk] += dv[:P]; bnd["dvp"][:, hk] += ev[:P]
            val["dk"][c, hk] += dk[P:]; bnd["dk"][c, hk] += ek[P:]
            val["dv"][c, hk] += dv[P:]; bnd["dv"][c, hk] += ev[P:]
    return val, bnd


def run(t, causal, scale=None, train=True):
    """Outputs start at 7: rows of no sequence must keep it."""
    Hq, Tq = t["q"].shape[1], t["q"].shape[0]
    o, lse = torch.full_like(t["q"], 7.0), torch.full((Hq, Tq), 7.0, device=DEV)
    args = (t["cq"], t["ck"], t["mq"], t["mk"], causal, scale)
    fa.fwd_prefix(t["q"], t["k"], t["v"], t["kp"], t["vp"], o, lse, *args)
    got = dict(o=o, lse=lse)
    if train:
        delta = torch.empty_like(lse)
        fa.bwd_preprocess(fa._as4(o, True), fa._as4(t["do"], True), delta)
        for n, ref in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dkp", "kp"), ("dvp", "vp")):
            got[n] = torch.full_like(t[ref], 7.0)
        fa.bwd_prefix(t["q"], t["k"], t["v"], t["kp"], t["vp"], t["do"], lse, delta, got["dq"], got["dk"], got["dv"],
                      got["dkp"], got["dvp"], *args)
    torch.cuda.synchronize()
    assert fa.device_status() == 0
    return got


def check(t, got, causal, scale=None, rounded_delta=True):
    val, bnd = reference(t, causal, scale, rounded_delta)
    dt = t["q"].dtype
    u = torch.finfo(dt).eps / 2
    rows = dict(q=slice(int(t["cq"][0]), int(t["cq"][-1])), k=slice(int(t["ck"][0]), int(t["ck"][-1])))
    for n, g in got.items():
        r, e = val[n], bnd[n]
        if n == "lse":
            g, r = g[:, rows["q"]].double(), r[:, rows["q"]]
            none = torch.isneginf(r)
            assert (torch.isneginf(g) == none).all()
            g, r = g.masked_fill(none, 0), r.masked_fill(none, 0)
            assert ((g - r).abs() <= SLACK + 2**-23 * r.abs()).all(), float((g - r).abs().max())
            continue
        if n in ("o", "dq", "dk", "dv"):
            own = rows["q" if n in ("o", "dq") else "k"]
            for side in (g[:own.start], g[own.stop:]):
                assert (side == 7).all(), f"{n}: rows of no sequence were written"
            g, r, e = g[own], r[own], e[own]
        err = (g.double() - r).abs()
        lim = e + u * (r.abs() + e) + 1e-6
        assert (err <= lim).all(), f"{n}: worst ratio {float((err / lim).nan_to_num(9e9).max()):.3f}"


def both(t, causal=True, scale=None):
    check(t, run(t, causal, scale), causal, scale)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("D", [16, 32, 64, 128])
def test_types_and_head_dims(D, dtype, causal):
    both(make((70, 1, 130, 0, 33), (70, 1, 130, 0, 33), 4, 2, D, 200, dtype, seed=D), causal)


@pytest.mark.parametrize("P", [0, 1, 63, 64, 65, 127, 128, 129, 256, 300, 1000])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64), ("fp32", 64)])
def test_prefix_lengths(P, dtype, D):
    both(make((140, 20), (140, 20), 2, 1, D, P, dtype, seed=P))


@pytest.mark.parametrize("lens", [(1,), (2, 1), (127,), (128,), (129, 256, 255), (300, 5, 640), (1, 1, 1, 1, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_sequence_lengths(lens, D):
    both(make(lens, lens, 4, 2, D, 150, seed=sum(lens)))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("fp32", 32)])
def test_key_lengths_that_differ(dtype, D, causal):
    """More own keys than queries and the other way, sequences with no key or no
    query of their own."""
    both(make((100, 0, 300, 7), (40, 130, 0, 400), 4, 4, D, 90, dtype, seed=1), causal)
    both(make((100, 0, 300, 7), (40, 130, 0, 400), 4, 4, D, 0, dtype, seed=2), causal)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 1), (6, 2), (5, 5), (16, 2)])
@pytest.mark.parametrize("D", [64, 128])
def test_grouped_heads(Hq, Hkv, D):
    both(make((200, 61), (200, 61), Hq, Hkv, D, 260, seed=Hq))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64), ("bf16", 32), ("fp32", 64)])
def test_rows_of_no_sequence(dtype, D, causal):
    """Rows before the first and behind the last sequence hold NaN (a padded
    batch, uninitialised memory): nothing of them reaches a result, and what
    the outputs hold there stays."""
    both(make((70, 129, 1), (70, 129, 1), 4, 2, D, 75, dtype, seed=3, lead=8, tail=40), causal)
    both(make((50, 3), (20, 77), 2, 2, D, 200, dtype, seed=4, lead=16, tail=200), causal)


def test_many_sequences_and_a_long_prefix():
    lens = tuple((37 * i) % 90 + 1 for i in range(40))
    both(make(lens, lens, 4, 1, 64, 2100, seed=5))
    both(make((1500, 700), (1500, 700), 2, 1, 128, 3000, seed=6))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64), ("bf16", 32)])
def test_one_long_sequence_among_short_ones(dtype, D, causal):
    """Far fewer tiles than sequences x the longest one's; some are empty."""
    lens = [(i * 37) % 7 for i in range(140)]
    lens[0], lens[129], lens[139] = 0, 700, 0
    both(make(lens, lens, 4, 2, D, 70, dtype, seed=17, lead=2, tail=3), causal)


@pytest.mark.parametrize("n", [511, 512, 513])
def test_sequence_counts_around_the_limit_of_the_packed_order(n):
    lens = [1 + i % 3 for i in range(n)]
    lens[n // 2] = 400
    both(make(lens, lens, 2, 1, 64, 40, "bf16", seed=18))


def test_long_sequences_of_unequal_length_and_many_heads():
    lens = (900, 3, 128, 0, 257, 512)
    both(make(lens, lens, 12, 6, 128, 200, "bf16", seed=19))


@pytest.mark.parametrize("D", [64, 128])
def test_bad_keys_of_an_empty_sequence_are_reported(D):
    """Sequences before the bad one keep their rows."""
    lens = [5, 300, 0, 4, 4, 4, 4, 4, 4]
    t = make(lens, lens, 2, 2, D, 30, "bf16", seed=20)
    o = run(t, True, train=False)["o"]
    bad = t["ck"].clone()
    bad[3] = 100000
    got, _ = fa.attention_prefix_fwd(t["q"], t["k"], t["v"], t["kp"], t["vp"], t["cq"], bad, t["mq"], t["mk"], True)
    torch.cuda.synchronize()
    assert fa.device_status() == 13 and fa.device_status() == 0
    assert torch.equal(got[:305], o[:305])


@pytest.mark.parametrize("P", [0, 1, 3, 31, 32, 63, 65, 129])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64), ("bf16", 32)])
def test_short_prefixes_of_many_sequences(P, dtype, D):
    """Too much for the FFMA kernels to pay: the tensor-core kernels at prefixes
    of up to two tiles."""
    lens = [(i * 41) % 150 for i in range(24)]
    t = make(lens, lens, 8, 4, D, P, dtype, seed=21, lead=3, tail=5)
    both(t)
    both(t, False)


@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (4, 1), (6, 1), (16, 2), (7, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_walks_shared_by_clusters(Hq, Hkv, D):
    """Few key tiles and many query rows: clusters of up to eight, for the own and
    the prefix's keys."""
    lens = (300, 1, 403, 130, 77, 260)
    t = make(lens, lens, Hq, Hkv, D, 450, "bf16", seed=24, lead=1, tail=2)
    both(t)
    both(t, False)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64), ("bf16", 32), ("fp16", 16)])
@pytest.mark.parametrize("n,P", [(1, 1), (3, 11), (40, 11), (40, 0), (30, 2)])
def test_gradients_of_rows_with_few_keys(n, P, dtype, D, causal):
    """At most 32 keys per row: Delta comes without the rounding of o, so the
    gradients' bound has no term for it; few rows (FFMA) and many (tensor cores)."""
    lens = [1 + (7 * i + n) % 20 for i in range(n)] if n > 1 else [1]
    t = make(lens, lens, 8, 4, D, P, dtype, seed=22, lead=2, tail=1)
    args = (t["cq"], t["ck"], t["mq"], t["mk"], causal)
    o, lse = fa.attention_prefix_fwd(t["q"], t["k"], t["v"], t["kp"], t["vp"], *args)
    delta = torch.full_like(lse, 7.0)
    fa.bwd_prefix_delta(t["q"], t["k"], t["v"], t["kp"], t["vp"], o, t["do"], lse, delta, *args)
    grads = [torch.full_like(t[x], 7.0) for x in ("q", "k", "v", "kp", "vp")]
    ts = (t["q"], t["k"], t["v"], t["kp"], t["vp"])
    fa.bwd_prefix(*ts, t["do"], lse, delta, grads[0], grads[1], grads[2], grads[3], grads[4], *args)
    torch.cuda.synchronize()
    assert fa.device_status() == 0
    check(t, dict(zip(("dq", "dk", "dv", "dkp", "dvp"), grads)), causal, rounded_delta=False)


def test_few_keys_of_unequal_sequences_keep_rowsum_elsewhere():
    """Rows above 32 keys take fa_bwd_preprocess's delta, bit for bit."""
    lens = [100, 5, 0, 33, 20]
    t = make(lens, lens, 4, 2, 64, 12, "bf16", seed=23)
    for causal in (True, False):
        args = (t["cq"], t["ck"], t["mq"], t["mk"], causal)
        o, lse = fa.attention_prefix_fwd(t["q"], t["k"], t["v"], t["kp"], t["vp"], *args)
        plain, delta = torch.empty_like(lse), torch.empty_like(lse)
        fa.bwd_preprocess(fa._as4(o, True), fa._as4(t["do"], True), plain)
        fa.bwd_prefix_delta(t["q"], t["k"], t["v"], t["kp"], t["vp"], o, t["do"], lse, delta, *args)
        few = torch.zeros(sum(lens), dtype=torch.bool, device=DEV)
        at = 0
        for n in lens:
            keys = 12 + (torch.arange(n, device=DEV) + 1 if causal else torch.full((n,), n, device=DEV))
            few[at:at + n] = keys <= 32
            at += n
        assert torch.equal(delta[:, ~few], plain[:, ~few])
        assert 20 <= int(few.sum()) < 120
        u = 2.0**-8
        mag = (t["do"].float().abs() * o.float().abs()).sum(-1).T
        assert ((delta - plain).abs() <= 4 * u * mag + 1e-2)[:, few].all()


def test_scale_strides_and_slices():
    """Rows of a fused projection [rows, 3, H, D] and a prefix that is a slice of
    a longer cache."""
    t = make((90, 33), (90, 33), 2, 2, 64, 100, seed=7)
    qkv = torch.stack([t["q"], t["k"], t["v"]], 1)
    cache = torch.randn(300, 2, 4, 64, device=DEV).bfloat16()
    t.update(q=qkv[:, 0], k=qkv[:, 1], v=qkv[:, 2], kp=cache[50:150, 0, 1:3], vp=cache[50:150, 1, 1:3])
    both(t, True, 0.2)


def test_ffma_path():
    """The FFMA kernels for 16-bit inputs too."""
    fa.set_path(fa.FA_PATH_FFMA)
    try:
        both(make((70, 1, 130), (70, 1, 130), 4, 2, 64, 100, "bf16", seed=8, tail=9))
    finally:
        fa.set_path(fa.FA_PATH_AUTO)


def test_large_scores():
    """The running maximum moves between prefix and own keys."""
    t = make((150, 20), (150, 20), 2, 1, 64, 300, seed=9)
    t["k"] *= 12
    both(t)
    t = make((150, 20), (150, 20), 2, 1, 128, 300, seed=10)
    t["kp"] *= 12
    both(t)


def test_equals_attention_over_concatenated_keys():
    """One sequence: the same as attention over prefix and own keys joined, with
    the queries shifted (non-causal, so that only the joining differs)."""
    t = make((200,), (200,), 4, 2, 128, 256, seed=11)
    got = run(t, False)
    k, v = torch.cat([t["kp"], t["k"]]), torch.cat([t["vp"], t["v"]])
    cu = torch.tensor([0, 456], dtype=torch.int32, device=DEV)
    o, lse = fa.attention_ex_fwd(t["q"], k, v, False, cu_seqlens_q=t["cq"], cu_seqlens_k=cu, max_seqlen_q=200,
                                 max_seqlen_k=456)
    # 256 prefix keys fill whole tiles: the same tiles in the same order
    assert torch.equal(got["o"], o) and torch.equal(got["lse"], lse)


def test_bad_offsets_are_reported():
    t = make((40, 30, 20), (40, 30, 20), 2, 2, 64, 50, seed=12)
    t["cq"] = torch.tensor([0, 40, 30, 90], dtype=torch.int32, device=DEV)
    o, lse = torch.full_like(t["q"], 7.0), torch.full((2, 90), 7.0, device=DEV)
    fa.fwd_prefix(t["q"], t["k"], t["v"], t["kp"], t["vp"], o, lse, t["cq"], t["ck"], 40, 40, True)
    torch.cuda.synchronize()
    assert fa.device_status() == 13 and fa.device_status() == 0


def test_autograd_and_repeats():
    t = make((90, 133), (90, 133), 4, 2, 64, 180, seed=13)
    names = ("q", "k", "v", "kp", "vp")
    leaves = [t[n].clone().requires_grad_() for n in names]
    q, k, v, kp, vp = leaves
    args = (t["cq"], t["ck"], t["mq"], t["mk"])
    o = fa.attention_varlen_prefix(q, k, v, kp, vp, *args)
    got = torch.autograd.grad(o, leaves, t["do"])
    o2, lse = fa.attention_prefix_fwd(*(t[n] for n in names), *args)
    ref = fa.attention_prefix_bwd(*(t[n] for n in names), o2, lse, t["do"], *args)
    assert torch.equal(o, o2)
    assert all(torch.equal(a, b) for a, b in zip(got, (ref[0], ref[1], ref[2], ref[3], ref[4])))
    # expanded gradients, and a prefix expanded over heads
    o = fa.attention_varlen_prefix(q, k, v, kp, vp, *args)
    got = torch.autograd.grad(o.sum(), leaves)
    ref = fa.attention_prefix_bwd(*(t[n] for n in names), o2, lse, torch.ones_like(o2), *args)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    one = kp.detach()[:, :1].clone().requires_grad_()
    o = fa.attention_varlen_prefix(q, k, v, one.expand(-1, 2, -1), vp, *args)
    (g1,) = torch.autograd.grad(o, one, t["do"])
    full = one.detach().expand(-1, 2, -1).contiguous().requires_grad_()
    o = fa.attention_varlen_prefix(q, k, v, full, vp, *args)
    (g2,) = torch.autograd.grad(o, full, t["do"])
    assert torch.equal(g1, g2.sum(1, keepdim=True))


def test_gradient_matches_differences():
    """fp32 inputs, along random directions: differences of the 64-bit
    definition's loss would test the reference; these test the kernels' own
    forward (rounding 1e-6 of the summed magnitudes over the step)."""
    t = make((40, 9), (40, 9), 2, 1, 32, 50, "fp32", seed=14)
    names = ("q", "k", "v", "kp", "vp")
    args = (t["cq"], t["ck"], t["mq"], t["mk"])

    def loss(x):
        o, _ = fa.attention_prefix_fwd(*(x[n] for n in names), *args)
        return float((o.double() * t["do"].double()).sum())

    o, lse = fa.attention_prefix_fwd(*(t[n] for n in names), *args)
    grads = dict(zip(("q", "k", "v", "kp", "vp"),
                     fa.attention_prefix_bwd(*(t[n] for n in names), o, lse, t["do"], *args)))
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    for n in names:
        d = torch.randn(t[n].shape, generator=g, device=DEV)
        d /= d.norm()
        h = 2e-2
        num = (loss(dict(t, **{n: t[n] + h * d})) - loss(dict(t, **{n: t[n] - h * d}))) / (2 * h)
        want = float((grads[n].double() * d.double()).sum())
        assert abs(num - want) < 2e-3 * max(1.0, float(grads[n].norm())), (n, num, want)


def test_graph_and_side_stream():
    """A captured forward and backward, replayed on new values, while an eager
    graph of the same tensors is alive; and another stream."""
    t = make((90, 133), (90, 133), 4, 2, 64, 180, seed=15)
    names = ("q", "k", "v", "kp", "vp")
    args = (t["cq"], t["ck"], t["mq"], t["mk"])

    def step():
        o, lse = fa.attention_prefix_fwd(*(t[n] for n in names), *args)
        return (o, *fa.attention_prefix_bwd(*(t[n] for n in names), o, lse, t["do"], *args))

    ref = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = step()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    t["q"].copy_(torch.randn(t["q"].shape, device=DEV))
    t["kp"].copy_(torch.randn(t["kp"].shape, device=DEV))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_rotation_then_prompt_then_decode():
    """The operators together, as a model uses them: a document's keys are
    rotated once; questions behind it run as packed sequences; then one token
    each is decoded over the same prefix and the questions' cached keys.  The
    decoded token equals the last row of the packed run with that token."""
    g = torch.Generator(device=DEV)
    g.manual_seed(16)
    D, Hq, Hkv, P, lens = 64, 8, 2, 300, [45, 1, 130]
    dt = torch.bfloat16
    freq = (10000.0 ** (-torch.arange(D // 2, device=DEV) / (D // 2))).float()
    qw, kw = (1 + 0.1 * torch.randn(D, generator=g, device=DEV) for _ in range(2))
    doc_k, doc_v = (torch.randn(P, Hkv, D, generator=g, device=DEV).to(dt) for _ in range(2))
    _, kp = fa.qk_norm_rotary_fwd(doc_k, doc_k, qw, kw, torch.arange(P, device=DEV), freq)
    total = sum(lens)
    q, k, v = (torch.randn(total, H, D, generator=g, device=DEV).to(dt).requires_grad_() for H in (Hq, Hkv, Hkv))
    cu = torch.tensor([0, 45, 46, 176], dtype=torch.int32, device=DEV)
    pos = torch.cat([torch.arange(P, P + n, device=DEV) for n in lens])
    kp_leaf = kp.clone().requires_grad_()
    wq, wk = qw.clone().requires_grad_(), kw.clone().requires_grad_()
    o = fa.attention_varlen_prefix(q, k, v, kp_leaf, doc_v, cu, cu, 130, 130,
                                   rotary=fa.Rotary(pos, freq, None, False, wq, wk))
    grads = torch.autograd.grad(o, (q, k, v, kp_leaf, wq, wk), torch.randn(o.shape, generator=g, device=DEV).to(dt))
    assert all(torch.isfinite(x).all() and (x != 0).any() for x in grads)
    # caches as a server keeps them: the rotated keys of each question
    qr, kr = fa.qk_norm_rotary_fwd(q.detach(), k.detach(), qw, kw, pos, freq)
    S = 160
    kc, vc = (torch.full((3, Hkv, S, D), float("nan"), device=DEV, dtype=dt) for _ in range(2))
    at = 0
    for b, n in enumerate(lens):
        kc[b, :, :n], vc[b, :, :n] = kr[at:at + n].transpose(0, 1), v.detach()[at:at + n].transpose(0, 1)
        at += n
    last = cu[1:].long() - 1
    od, _ = fa.attention_decode(qr[last][:, :, None], kp.transpose(0, 1), doc_v.transpose(0, 1), kc, vc,
                                torch.tensor(lens, dtype=torch.int32, device=DEV))
    u = 2.0**-8
    want = o.detach()[last].float()
    # both round P (u of a weighted mean of |v|, below 1 here) and the result
    assert ((od[:, :, 0].float() - want).abs() <= 2 * u * (1 + want.abs())).all()
