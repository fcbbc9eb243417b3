"""Rotation of query and key heads by positions with one or several axes, and
the norm of heads in the same pass, against the definitions in 64 bits.

Tolerances, from the arithmetic of the kernels (u: half a step of the output
type; fp32 rounding 2^-24 = 6e-8):
 * a rotated element a cos - b sin: the angle's fraction of a turn is rounded
   once to fp32 (9.4e-8 rad at most), sine and cosine are off by two steps
   (2.4e-7), products and sum round three times (1.8e-7): below
   ROT = 8e-7 (|a| + |b|), then one rounding u |result|;
 * the norm's sum of D <= 128 squares is 16 sequential additions and three
   exchanges, rsqrt two steps: rstd is off by less than 24 roundings (1.5e-6)
   relative, each product one more: NORM = 3e-6 relative on what it scales;
 * the gradient's mean of D products the same: GRAD = 6e-6 on the sum of the
   magnitudes of its terms;
 * a weight's gradient adds rows in chains no longer than 200 here (1.2e-5 of
   the sum of magnitudes) plus the terms' own error: DW = 2.5e-5.
"""

from __future__ import annotations

import pytest
import torch

from exact_attention_83_gb300 import fa

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
ROT, NORM, GRAD, DW = 8e-7, 3e-6, 6e-6, 2.5e-5
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fa.load_library()


def _heads(g, B, H, N, D, dt, layout):
    if layout == "bhnd":
        return torch.randn(B, H, N, D, generator=g, device=DEV).to(dt)
    if layout == "bnhd":
        return torch.randn(B, N, H, D, generator=g, device=DEV).to(dt).permute(0, 2, 1, 3)
    if layout == "packed":
        return torch.randn(N, H, D, generator=g, device=DEV).to(dt)
    # every other head and row of a wider buffer, as a fused projection leaves them
    return torch.randn(B, 2 * H, N, 2 * D, generator=g, device=DEV).to(dt)[:, ::2, :, :D]


def _angles(pos, freq, sections, packed):
    """[(B,) 1, N, pairs] (or [N, 1, pairs] packed) angles in 64 bits."""
    axis = torch.tensor([a for a, n in enumerate(sections) for _ in range(n)], device=DEV)
    ang = pos.double()[axis].movedim(0, -1) * freq.double()
    return ang[:, None]


def _rot(x, ang, interleaved):
    n = ang.shape[-1]
    c, s = ang.cos(), ang.sin()
    y = x.clone()
    ia, ib = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = a * s + b * c
    return y


def _pair_mag(x, n, interleaved):
    """|a| + |b| on both elements of each rotated pair, 0 elsewhere."""
    m = torch.zeros_like(x)
    ia, ib = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    m[..., ia] = m[..., ib] = x[..., ia].abs() + x[..., ib].abs()
    return m


def _close(name, got, ref, bound, dt):
    u = torch.finfo(dt).eps / 2
    # a result below the type's normal numbers rounds by half a subnormal step
    tiny = torch.finfo(dt).smallest_normal * u
    err = (got.double() - ref).abs()
    lim = bound + u * (ref.abs() + bound) + tiny
    bad = ~(err <= lim)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()}, worst {float((err - lim).max()):.3e}"


def _check(dtype, B, N, Hq, Hkv, D, sections, interleaved, layout, norm, pos=None, w32=True, seed=0,
           pos_dtype=torch.int64):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt, A, n = DT[dtype], len(sections), sum(sections)
    q, k = _heads(g, B, Hq, N, D, dt, layout), _heads(g, B, Hkv, N, D, dt, layout)
    dqo, dko = _heads(g, B, Hq, N, D, dt, layout), _heads(g, B, Hkv, N, D, dt, layout)
    packed = layout == "packed"
    if pos is None:
        pos = torch.randint(-1000, 200000, (A, N) if packed else (A, B, N), generator=g, device=DEV)
    pos = pos.to(pos_dtype)
    freq = (500000.0 ** (-torch.arange(n, device=DEV) / n)).float()
    ang = _angles(pos, freq, sections, packed)
    wdt = torch.float32 if w32 else dt
    ws = [(1 + 0.2 * torch.randn(D, generator=g, device=DEV)).to(wdt) for _ in range(2)]
    if norm:
        outs = fa.qk_norm_rotary_fwd(q, k, *ws, pos, freq, sections, interleaved, EPS)
        grads = fa.qk_norm_rotary_bwd(q, k, *ws, dqo, dko, pos, freq, sections, interleaved, EPS)
    else:
        outs = fa.rotary_fwd(q, k, pos, freq, sections, interleaved)
        grads = fa.rotary_bwd(dqo, dko, pos, freq, sections, interleaved)
    assert fa.device_status() == 0
    for i, (x, go, w) in enumerate(((q, dqo, ws[0]), (k, dko, ws[1]))):
        x, go, w = x.double(), go.double(), w.double()
        g0 = _rot(go, -ang, interleaved)
        gmag = ROT * _pair_mag(go, n, interleaved)
        if not norm:
            _close(f"out{i}", outs[i], _rot(x, ang, interleaved), ROT * _pair_mag(x, n, interleaved), dt)
            _close(f"grad{i}", grads[i], g0, gmag, dt)
            continue
        rstd = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
        xh = x * rstd
        y = xh * w
        _close(f"out{i}", outs[i], _rot(y, ang, interleaved),
               ROT * _pair_mag(y, n, interleaved) + NORM * (y.abs() + _pair_mag(y, n, interleaved)), dt)
        gw = g0 * w
        mean = (gw * xh).mean(-1, keepdim=True)
        ref = rstd * (gw - xh * mean)
        mag = (gw.abs() + gmag / ROT * w.abs())
        magm = (mag * xh.abs()).mean(-1, keepdim=True)
        _close(f"grad{i}", grads[i], ref, GRAD * rstd * (mag + xh.abs() * magm), dt)
        red = [d for d in range(x.dim() - 1)]
        dw = (g0 * xh).sum(red)
        dwmag = ((g0.abs() + gmag / ROT) * xh.abs()).sum(red)
        err = (grads[2 + i].double() - dw).abs()
        assert (err <= DW * dwmag + 1e-30).all(), f"dw{i}: {float((err / dwmag).max()):.3e}"


LAYOUTS = ["bhnd", "bnhd", "packed", "sliced"]


@pytest.mark.parametrize("norm", [False, True], ids=["rot", "norm"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("interleaved", [False, True])
def test_layouts(dtype, layout, interleaved, norm):
    _check(dtype, 1 if layout == "packed" else 2, 77, 6, 2, 64, [8, 12, 12], interleaved, layout, norm)


@pytest.mark.parametrize("norm", [False, True], ids=["rot", "norm"])
@pytest.mark.parametrize("D,sections", [(16, [8]), (32, [8]), (32, [5, 11]), (64, [16]), (64, [1, 2, 3, 2]),
                                        (128, [64]), (128, [16, 24, 24]), (128, [8]), (128, [40])])
@pytest.mark.parametrize("interleaved", [False, True])
def test_head_dims_and_partial_rotation(D, sections, interleaved, norm):
    _check("bf16", 2, 33, 5, 3, D, sections, interleaved, "bhnd", norm, seed=D)
    _check("fp32", 1, 9, 1, 7, D, sections, interleaved, "bnhd", norm, seed=D + 1)


@pytest.mark.parametrize("norm", [False, True], ids=["rot", "norm"])
@pytest.mark.parametrize("N", [1, 2, 7, 8, 9, 255, 2049])
def test_lengths(N, norm):
    _check("bf16", 1, N, 4, 1, 128, [64], False, "packed", norm, seed=N)
    _check("fp16", 3, N, 1, 1, 64, [16, 16], True, "bhnd", norm, seed=N)


def test_norm_weights_of_the_heads_type():
    for dtype in ("bf16", "fp16"):
        _check(dtype, 2, 50, 4, 2, 64, [32], False, "bhnd", True, w32=False)


def test_far_and_negative_positions():
    """The angle of a far position keeps its fraction of a turn: fp32 products
    would be off by tenths of a radian here."""
    pos = torch.tensor([0, 1, -1, 10**6, -10**6, 12345678, 2**30 - 1, -2**30], device=DEV)
    _check("fp32", 1, len(pos), 2, 2, 64, [32], False, "packed", False, pos=pos[None])
    _check("fp32", 1, len(pos), 2, 2, 64, [32], False, "packed", False, pos=pos[None],
           pos_dtype=torch.int32)


def test_frequencies_of_all_magnitudes():
    """inv_freq from 2^-40 to 2^20, both signs: the turn's fraction is exact."""
    n = 32
    freq = torch.tensor([(1.37 * (-1) ** i) * 2.0 ** e for i, e in enumerate(
        [-40, -30, -24, -23, -22, -10, -3, -1, 0, 1, 2, 3, 5, 8, 12, 16, 17, 18, 19, 20, -126, -140, -12,
         -13, -14, -15, -16, -17, 4, 6, 7, 9])], device=DEV, dtype=torch.float32)
    pos = torch.tensor([[0, 1, 2, -3, 977, 65537, 1000003, 2**35 + 12345]], device=DEV)
    x = torch.randn(8, 2, 64, device=DEV)
    y, _ = fa.rotary_fwd(x, x, pos, freq)
    # the reference's own angles: exact integers of 2^-k turns are out of a
    # double's reach for the largest products, so reduce with exact integers
    import math
    from fractions import Fraction
    PI = Fraction(314159265358979323846264338327950288419716939937510, 10**50)
    for t, p in enumerate(pos[0].tolist()):
        for i, f in enumerate(freq.tolist()):
            turn = Fraction(f) * p / (2 * PI)
            ang = float((turn - round(turn)) * 2 * PI)
            a, b = float(x[t, 0, i]), float(x[t, 0, n + i])
            tol = (ROT + 2**-24) * (abs(a) + abs(b)) * 1.01
            assert abs(float(y[t, 0, i]) - (a * math.cos(ang) - b * math.sin(ang))) <= tol, (p, f)
            assert abs(float(y[t, 0, n + i]) - (a * math.sin(ang) + b * math.cos(ang))) <= tol, (p, f)


def test_shared_positions_and_short_forms():
    """[N] and [B, N] with one axis, [A, 1, N] shared over the batch."""
    q, k = torch.randn(2, 3, 11, 64, device=DEV), torch.randn(2, 1, 11, 64, device=DEV)
    freq = (100.0 ** (-torch.arange(32, device=DEV) / 32)).float()
    n = torch.arange(11, device=DEV)
    full = n.expand(1, 2, 11).contiguous()
    ref = fa.rotary_fwd(q, k, full, freq)
    for pos in (n, n[None].expand(2, 11), n[None, None], n.int(), full.expand(1, 2, 11)):
        got = fa.rotary_fwd(q, k, pos, freq)
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    pos = torch.stack([n, 2 * n])[:, None]
    a = fa.rotary_fwd(q, k, pos, freq, [20, 12])
    b = fa.rotary_fwd(q, k, pos.expand(2, 2, 11).contiguous(), freq, [20, 12])
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_zero_rows_and_in_place():
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    q, k = _heads(g, 2, 4, 30, 64, torch.bfloat16, "bhnd"), _heads(g, 2, 2, 30, 64, torch.bfloat16, "bnhd")
    q[1, 2] = 0
    w = torch.ones(64, device=DEV)
    freq, pos = torch.rand(32, device=DEV), torch.arange(30, device=DEV)
    out = fa.qk_norm_rotary_fwd(q, k, w, w, pos, freq)
    assert (out[0][1, 2] == 0).all() and torch.isfinite(out[0]).all()
    rot = fa.rotary_fwd(q, k, pos, freq)
    q2, k2 = q.clone(), k.clone(memory_format=torch.preserve_format)
    assert k2.stride() == k.stride()
    fa.rotary_fwd(q2, k2, pos, freq, out=(q2, k2))
    assert torch.equal(q2, rot[0]) and torch.equal(k2, rot[1])
    dq, dk = fa.rotary_bwd(out[0], out[1], pos, freq)
    g0, g1 = out[0].clone(), out[1].clone()
    fa.rotary_bwd(g0, g1, pos, freq, out=(g0, g1))
    assert torch.equal(g0, dq) and torch.equal(g1, dk)
    q3, k3 = q.clone(), k.clone(memory_format=torch.preserve_format)
    fa.qk_norm_rotary_fwd(q3, k3, w, w, pos, freq, out=(q3, k3))
    assert torch.equal(q3, out[0]) and torch.equal(k3, out[1])


def test_rows_of_a_wider_buffer_are_left_alone():
    """Outputs with strides: what lies between their rows is not written."""
    buf = torch.full((2, 9, 3, 96), 7.0, device=DEV, dtype=torch.float16)
    q = torch.randn(2, 3, 9, 64, device=DEV).half()
    out = buf[..., :64].permute(0, 2, 1, 3)
    freq, pos = torch.rand(16, device=DEV), torch.arange(9, device=DEV)
    got = fa.rotary_fwd(q, q, pos, freq, out=(out, torch.empty_like(q)))
    assert torch.equal(got[0], got[1]) and (buf[..., 64:] == 7).all()


def test_autograd_matches_the_calls_and_differences():
    """Gradients through autograd equal the explicit calls, also for expanded
    incoming gradients; and differences of the forward in fp32."""
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    q = torch.randn(2, 4, 12, 32, generator=g, device=DEV).requires_grad_()
    k = torch.randn(2, 2, 12, 32, generator=g, device=DEV).requires_grad_()
    qw = (1 + 0.1 * torch.randn(32, generator=g, device=DEV)).requires_grad_()
    kw = (1 + 0.1 * torch.randn(32, generator=g, device=DEV)).requires_grad_()
    freq, pos = torch.rand(16, device=DEV), torch.arange(12, device=DEV)
    cq, ck = torch.randn(2, 4, 12, 32, generator=g, device=DEV), torch.randn(2, 2, 12, 32, generator=g, device=DEV)

    def loss(q, k, qw, kw):
        a, b = fa.qk_norm_rotary(q, k, qw, kw, pos, freq, None, False, EPS)
        return (a * cq).sum() + (b * ck).sum()

    got = torch.autograd.grad(loss(q, k, qw, kw), (q, k, qw, kw))
    ref = fa.qk_norm_rotary_bwd(q.detach(), k.detach(), qw.detach(), kw.detach(), cq, ck, pos, freq, None,
                                False, EPS)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    # central differences along a random direction: truncation O(h^2), the
    # forward's rounding 1e-6 of the summed magnitudes over 2 h
    h = 2e-2
    for i, x in enumerate((q, k, qw, kw)):
        d = torch.randn(x.shape, generator=g, device=DEV)
        d /= d.norm()
        args = [t.detach() for t in (q, k, qw, kw)]
        lo, hi = list(args), list(args)
        lo[i], hi[i] = args[i] - h * d, args[i] + h * d
        num = float((loss(*hi).double() - loss(*lo).double()) / (2 * h))
        assert abs(num - float((got[i] * d).sum())) < 2e-2, i
    # expanded gradients: of a sum, and broadcast over heads
    a, b = fa.rotary(q, k, pos, freq)
    (gq,) = torch.autograd.grad(a.sum(), q, retain_graph=True)
    exp = fa.rotary_bwd(torch.ones_like(q), torch.ones_like(k), pos, freq)[0]
    assert torch.equal(gq, exp)
    a, b = fa.rotary(q, k, pos, freq)
    (gq,) = torch.autograd.grad((a.sum(1) * cq[:, 0]).sum(), q)
    exp = fa.rotary_bwd(cq[:, :1].expand(2, 4, 12, 32).contiguous(), torch.zeros_like(k), pos, freq)[0]
    assert torch.equal(gq, exp)
    # expanded inputs get the sum over what they were expanded to
    k1 = torch.randn(2, 1, 12, 32, generator=g, device=DEV).requires_grad_()
    _, b = fa.rotary(q, k1.expand(2, 4, 12, 32), pos, freq)
    (gk,) = torch.autograd.grad((b * cq).sum(), k1)
    exp = fa.rotary_bwd(cq, cq, pos, freq)[1].sum(1, keepdim=True)
    assert torch.allclose(gk, exp, rtol=0, atol=1e-5)
    with pytest.raises(RuntimeError):
        a, b = fa.rotary(q, k, pos, freq)
        (gq,) = torch.autograd.grad((a * a).sum(), q, create_graph=True)
        gq.sum().backward()


def test_weight_gradients_do_not_depend_on_the_schedule():
    g = torch.Generator(device=DEV)
    g.manual_seed(9)
    q, k = _heads(g, 1, 8, 5000, 64, torch.bfloat16, "packed"), _heads(g, 1, 2, 5000, 64, torch.bfloat16, "packed")
    w, freq, pos = torch.ones(64, device=DEV), torch.rand(32, device=DEV), torch.arange(5000, device=DEV)
    a = fa.qk_norm_rotary_bwd(q, k, w, w, q, k, pos, freq)
    b = fa.qk_norm_rotary_bwd(q, k, w, w, q, k, pos, freq)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_side_stream_and_graph():
    """Another stream than the default, and a captured call replayed on new
    values."""
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    q, k = _heads(g, 2, 4, 40, 64, torch.bfloat16, "bhnd"), _heads(g, 2, 2, 40, 64, torch.bfloat16, "bhnd")
    w, freq, pos = torch.ones(64, device=DEV), torch.rand(32, device=DEV), torch.arange(40, device=DEV)
    ref = fa.qk_norm_rotary_bwd(q, k, w, w, q, k, pos, freq)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = fa.qk_norm_rotary_bwd(q, k, w, w, q, k, pos, freq)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fa.qk_norm_rotary_bwd(q, k, w, w, q, k, pos, freq)
        fwd = fa.qk_norm_rotary_fwd(q, k, w, w, pos, freq)
    q.copy_(torch.randn(q.shape, generator=g, device=DEV))
    pos += 100
    graph.replay()
    torch.cuda.synchronize()
    ref = fa.qk_norm_rotary_bwd(q, k, w, w, q, k, pos, freq)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    assert all(torch.equal(a, b) for a, b in zip(fwd, fa.qk_norm_rotary_fwd(q, k, w, w, pos, freq)))


def test_attention_applies_the_rotation_first():
    """attention_gqa and attention_varlen with rotary= are the rotation and then
    the attention, forward and gradients."""
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    q, k, v = (_heads(g, 2, H, 70, 64, torch.bfloat16, "bhnd").requires_grad_() for H in (4, 2, 2))
    qw, kw = (torch.rand(64, device=DEV).requires_grad_() for _ in range(2))
    rot = fa.Rotary(torch.arange(70, device=DEV), torch.rand(24, device=DEV), None, False, qw, kw)
    o = fa.attention_gqa(q, k, v, causal=True, rotary=rot)
    do = torch.randn(o.shape, generator=g, device=DEV).bfloat16()
    got = torch.autograd.grad(o, (q, k, v, qw, kw), do)
    q2, k2 = fa.qk_norm_rotary(q, k, qw, kw, rot.positions, rot.inv_freq)
    o2 = fa.attention_gqa(q2, k2, v, causal=True)
    assert torch.equal(o, o2)
    ref = torch.autograd.grad(o2, (q, k, v, qw, kw), do)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    cu = torch.tensor([0, 30, 70], dtype=torch.int32, device=DEV)
    qp, kp, vp = (t.detach()[0].transpose(0, 1).contiguous() for t in (q, k, v))
    o = fa.attention_varlen(qp, kp, vp, cu, cu, 40, 40, causal=True, rotary=rot)
    q2, k2 = fa.qk_norm_rotary_fwd(qp, kp, qw.detach(), kw.detach(), rot.positions, rot.inv_freq)
    assert torch.equal(o, fa.attention_varlen(q2, k2, vp, cu, cu, 40, 40, causal=True))


def test_positions_changed_before_the_backward_are_an_error():
    """A decode loop that advances its positions in place must not change the
    gradient of an earlier call in silence."""
    q = torch.randn(2, 4, 12, 32, device=DEV, requires_grad=True)
    pos, freq = torch.arange(12, device=DEV), torch.rand(16, device=DEV)
    a, b = fa.rotary(q, q.detach(), pos, freq)
    pos += 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        a.sum().backward()


def test_several_calls_at_once():
    """Two streams; each call allocates its own workspace."""
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    xs = [(_heads(g, 1, 16, 3000, 128, torch.bfloat16, "packed"), _heads(g, 1, 4, 3000, 128, torch.bfloat16, "packed"))
          for _ in range(2)]
    w, freq, pos = torch.rand(128, device=DEV), torch.rand(64, device=DEV), torch.arange(3000, device=DEV)
    ref = [fa.qk_norm_rotary_bwd(q, k, w, w, q, k, pos, freq) for q, k in xs]
    torch.cuda.synchronize()
    got = []
    for q, k in xs:
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(4):
                r = fa.qk_norm_rotary_bwd(q, k, w, w, q, k, pos, freq)
            got.append(r)
    torch.cuda.synchronize()
    for a, b in zip(ref, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (33, 7), (100, 3)])
@pytest.mark.parametrize("D", [16, 64, 128])
def test_head_counts_and_tiles(D, Hq, Hkv, interleaved):
    """Fewer heads than a warp has rows, heads that leave lanes over, and lengths
    around every tile size."""
    for N in (3, 17, 130):
        _check("bf16", 2, N, Hq, Hkv, D, [8] if D == 16 else [8, D // 2 - 8], interleaved, "bnhd", True, seed=Hq + N)
