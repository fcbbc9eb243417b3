"""Measured cases of the operators around attention over a shared prefix.

Four operators, each with its plain form (elementary torch operations in 32
bits, angles in 64), its calls of the framework, and its definition in 64 bits:

  decode     one or a few query tokens per request; every request's keys are a
             prefix that the whole batch shares, followed by its own cache rows
             (the first seq_lens[b] of the rows allocated)
  prompt     packed sequences that follow one shared prefix: every query sees
             the whole prefix and, causally, its own sequence; forward and, for
             training, the gradients of everything
  rotary     rotation of query and key heads by positions with one or several
             axes (time, height, width), and its gradient
  qk_norm    RMS norm of every query and key head, times a weight, with the
             rotation in the same pass; gradients of inputs and weights

`own` chooses between the plain forms (False) and the framework's calls (True).
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
_DEV = "cuda"
_EPS = 1e-6


# --------------------------------------------------------------------- cases


def listed():
    return [
        # A handful of chats behind a short system prompt, one token each: the
        # step is all latency.
        dict(name="decode-fp16-B4-H16-P512", op="decode", dtype="fp16", B=4, Hq=16, Hkv=16, Nq=1,
             D=64, P=512, S=128, layout="bhnd"),
        # Drafted tokens checked four at a time, three query heads to a
        # key/value head, a prefix that ends inside a tile, token-major caches.
        dict(name="decode-bf16-B7-Nq4-P1537", op="decode", dtype="bf16", B=7, Hq=12, Hkv=4, Nq=4,
             D=64, P=1537, S=333, layout="bnhd"),
        # An ordinary serving batch over a long tool description.
        dict(name="decode-bf16-B32-gqa-P8192", op="decode", dtype="bf16", B=32, Hq=32, Hkv=8, Nq=1,
             D=128, P=8192, S=512, layout="bhnd"),
        # The largest serving batch over a whole document.
        dict(name="decode-bf16-B128-gqa-P16384", op="decode", dtype="bf16", B=128, Hq=32, Hkv=8,
             Nq=1, D=128, P=16384, S=1024, layout="bhnd"),
        # A few short continuations in full precision, as a test or a probe of
        # a trained model runs them.
        dict(name="prompt-fp32-3seq-P200-train", op="prompt", dtype="fp32", seqs=3, N=130, Hq=4,
             Hkv=2, D=64, P=200, train=True),
        # Prefill of many questions about one document (no gradient).
        dict(name="prompt-fp16-24seq-P2048", op="prompt", dtype="fp16", seqs=24, N=257, Hq=16,
             Hkv=16, D=64, P=2048, train=False),
        # A training step over sampled answers to one long prompt.
        dict(name="prompt-bf16-16seq-gqa-P4096-train", op="prompt", dtype="bf16", seqs=16, N=512,
             Hq=32, Hkv=8, D=128, P=4096, train=True),
        # The new tokens of a video model's serving step: three axes.
        dict(name="rotary-bf16-T32-axes3", op="rotary", dtype="bf16", B=1, N=32, Hq=16, Hkv=16, D=64,
             sections="8,12,12", interleaved=False, layout="packed", train=False),
        # Image patches with two axes through a training step, pairs side by side.
        dict(name="rotary-fp16-B4-N4096-axes2-train", op="rotary", dtype="fp16", B=4, N=4096, Hq=16,
             Hkv=16, D=64, sections="16,16", interleaved=True, layout="bhnd", train=True),
        # One decode step's new tokens.
        dict(name="qk_norm-bf16-T32", op="qk_norm", dtype="bf16", B=1, N=32, Hq=32, Hkv=8, D=128,
             sections="64", interleaved=False, layout="packed", train=False),
        # An odd batch with half of each head rotated.
        dict(name="qk_norm-fp16-B3-N1001-partial-train", op="qk_norm", dtype="fp16", B=3, N=1001,
             Hq=12, Hkv=4, D=64, sections="16", interleaved=False, layout="bnhd", train=True),
        # A training step's whole sequence.
        dict(name="qk_norm-bf16-T16384-gqa-train", op="qk_norm", dtype="bf16", B=1, N=16384, Hq=32,
             Hkv=8, D=128, sections="64", interleaved=False, layout="packed", train=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "prompt", "rotary", "qk_norm"])
    half = rng.choice(["bf16", "fp16"])
    if op == "decode":
        Hkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 3, 4, 8])
        return dict(op=op, dtype=half, B=_log_int(rng, 1, 128), Hq=Hkv * G, Hkv=Hkv,
                    Nq=rng.choice([1, 1, 1, 2, 5]), D=rng.choice([64, 128]),
                    P=_log_int(rng, 1, 8192), S=_log_int(rng, 1, 1024),
                    layout=rng.choice(["bhnd", "bnhd"]))
    if op == "prompt":
        Hkv = rng.choice([1, 2, 4])
        G = rng.choice([1, 2, 3, 4])
        dtype = rng.choice([half, half, "fp32"])
        big = dtype != "fp32"
        return dict(op=op, dtype=dtype, seqs=_log_int(rng, 1, 16 if big else 4),
                    N=_log_int(rng, 1, 512 if big else 200), Hq=Hkv * G, Hkv=Hkv,
                    D=rng.choice([32, 64, 128]), P=_log_int(rng, 1, 4096 if big else 512),
                    train=rng.choice([True, False]))
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4])
    D = rng.choice([64, 128])
    pairs = rng.choice([D // 2, D // 2, D // 4])
    axes = rng.choice([1, 2, 3])
    if axes == 1:
        sections = [pairs]
    elif axes == 2:
        a = rng.randint(1, pairs - 1)
        sections = [a, pairs - a]
    else:
        a = rng.randint(1, pairs - 2)
        b = rng.randint(1, pairs - a - 1)
        sections = [a, b, pairs - a - b]
    B = rng.choice([1, 2, 3])
    return dict(op=op, dtype=rng.choice([half, half, "fp32"]), B=B, N=_log_int(rng, 1, 4096 // B),
                Hq=Hkv * G, Hkv=Hkv, D=D, sections=",".join(str(s) for s in sections),
                interleaved=rng.choice([True, False]), layout=rng.choice(["bhnd", "bnhd"]),
                train=rng.choice([True, False]))


# ------------------------------------------------------------- what a case is


def _lens(count, most):
    """`count` lengths from 1 to `most`, spread evenly, the first one `most`."""
    step = (math.sqrt(5.0) - 1.0) / 2.0
    return [max(1, math.ceil(most * (1.0 - (i * step) % 1.0))) for i in range(count)]


def _own_lens(case):
    """Own cache rows of each request: at least the new tokens, where they fit."""
    return [max(n, min(case["Nq"], case["S"])) for n in _lens(case["B"], case["S"])]


def _sections(case):
    return [int(s) for s in case["sections"].split(",")]


def _causal_pairs(n):
    return n * (n + 1) // 2


def work(case):
    e = _SIZE[case["dtype"]]
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    if case["op"] == "decode":
        B, Nq, P = case["B"], case["Nq"], case["P"]
        lens = _own_lens(case)
        kv = 2 * Hkv * D * e * (P + sum(lens))
        qo = B * Hq * Nq * (2 * D * e + 4)
        pairs = sum(Nq * P + sum(max(0, n - Nq + t + 1) for t in range(Nq)) for n in lens)
        return {"bytes": kv + qo + 4 * B, "flops": 4 * pairs * Hq * D}
    if case["op"] == "prompt":
        lens = _lens(case["seqs"], case["N"])
        total, P = sum(lens), case["P"]
        pairs = sum(n * P + _causal_pairs(n) for n in lens)
        q, kv = total * Hq * D * e, 2 * (total + P) * Hkv * D * e
        fwd = 2 * q + kv + 4 * total * Hq
        if not case["train"]:
            return {"bytes": fwd, "flops": 4 * pairs * Hq * D}
        # the gradient reads dO and writes dQ, dK, dV
        return {"bytes": fwd + 2 * q + kv, "flops": 14 * pairs * Hq * D}
    rows = case["B"] * case["N"]
    elems = rows * (Hq + Hkv) * D
    pairs = sum(_sections(case))
    extra = 8 * rows * len(_sections(case)) + 4 * pairs
    rot = 6 * rows * (Hq + Hkv) * pairs
    if case["op"] == "rotary":
        k = 2 if case["train"] else 1
        return {"bytes": k * 2 * elems * e + extra, "flops": k * rot}
    if case["train"]:
        # forward: read, write; backward: read input and gradient, write
        return {"bytes": 5 * elems * e + extra + 16 * D, "flops": 2 * rot + 14 * elems}
    return {"bytes": 2 * elems * e + extra + 8 * D, "flops": rot + 4 * elems}


# -------------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device=_DEV, dtype=torch.float32) * scale).to(dtype)


def _heads(g, B, H, N, D, dtype, layout, scale=1.0):
    """[B, H, N, D] values, stored head-major or token-major."""
    if layout == "bnhd":
        return _randn(g, (B, N, H, D), dtype, scale).permute(0, 2, 1, 3)
    return _randn(g, (B, H, N, D), dtype, scale)


def _positions(case, g):
    """int64 positions [A, B, N] or [A, N]: text positions that start far into
    a long context, or coordinates of a grid."""
    A, B, N = len(_sections(case)), case["B"], case["N"]
    start = torch.randint(0, 100000, (B, 1), generator=g, device=_DEV)
    i = torch.arange(N, device=_DEV)
    if A == 1:
        pos = (start + i)[None]
    else:
        side = max(1, math.isqrt(N))
        axes = [(i // side) % side, i % side] if A == 2 else [i // (side * 4), (i // side) % 4, i % side]
        pos = torch.stack([a.expand(B, N) for a in axes]) + (start[None] if A == 3 else 0)
    return pos.reshape(A, N).contiguous() if case["layout"] == "packed" else pos.contiguous()


def prepare(case, seed):
    g = _gen(seed)
    dt = _DT[case["dtype"]]
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    st = {"case": case}
    if case["op"] == "decode":
        B, Nq, P, S, lay = case["B"], case["Nq"], case["P"], case["S"], case["layout"]
        lens = torch.tensor(_own_lens(case), dtype=torch.int32, device=_DEV)
        lens = lens[torch.randperm(B, generator=g, device=_DEV)].contiguous()
        st.update(q=_heads(g, B, Hq, Nq, D, dt, lay), lens=lens,
                  kp=_heads(g, 1, Hkv, P, D, dt, lay)[0], vp=_heads(g, 1, Hkv, P, D, dt, lay)[0],
                  k=_heads(g, B, Hkv, S, D, dt, lay), v=_heads(g, B, Hkv, S, D, dt, lay))
        return st
    if case["op"] == "prompt":
        lens, P = _lens(case["seqs"], case["N"]), case["P"]
        total = sum(lens)
        cu = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).to(_DEV)
        st.update(q=_randn(g, (total, Hq, D), dt), k=_randn(g, (total, Hkv, D), dt),
                  v=_randn(g, (total, Hkv, D), dt), kp=_randn(g, (P, Hkv, D), dt),
                  vp=_randn(g, (P, Hkv, D), dt), cu=cu, lens=lens, most=max(lens))
        if case["train"]:
            st["do"] = _randn(g, (total, Hq, D), dt)
        return st
    B, N, lay = case["B"], case["N"], case["layout"]
    for name, H in (("q", Hq), ("k", Hkv)):
        if lay == "packed":
            st[name] = _randn(g, (N, H, D), dt)
        else:
            st[name] = _heads(g, B, H, N, D, dt, lay)
        if case["train"]:
            st["d" + name] = (_randn(g, (N, H, D), dt) if lay == "packed"
                              else _heads(g, B, H, N, D, dt, lay))
    sections = _sections(case)
    pairs = sum(sections)
    st["inv_freq"] = (10000.0 ** (-torch.arange(pairs, device=_DEV, dtype=torch.float64) / pairs)).float()
    st["positions"] = _positions(case, g)
    st["sections"] = sections
    if case["op"] == "qk_norm":
        st["qw"] = 1.0 + 0.1 * torch.randn(D, generator=g, device=_DEV)
        st["kw"] = 1.0 + 0.1 * torch.randn(D, generator=g, device=_DEV)
    return st


# --------------------------------------------------------------- plain forms


def _plain_decode(st):
    case = st["case"]
    B, Hq, Hkv, Nq, D = case["B"], case["Hq"], case["Hkv"], case["Nq"], case["D"]
    P, S, G = case["P"], case["S"], Hq // Hkv
    scale = 1.0 / math.sqrt(D)
    q = st["q"].float().reshape(B, Hkv, G * Nq, D)
    kp, vp, k, v = (st[n].float() for n in ("kp", "vp", "k", "v"))
    sp = torch.matmul(q, kp.transpose(-1, -2)) * scale                  # [B, Hkv, G Nq, P]
    so = torch.matmul(q, k.transpose(-1, -2)) * scale                   # [B, Hkv, G Nq, S]
    last = st["lens"].long()[:, None] - Nq + torch.arange(Nq, device=_DEV)   # [B, Nq]
    keep = torch.arange(S, device=_DEV)[None, None, :] <= last[:, :, None]
    keep = keep[:, None, None].expand(B, 1, G, Nq, S).reshape(B, 1, G * Nq, S)
    s = torch.cat([sp, torch.where(keep, so, torch.full_like(so, -math.inf))], -1)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    z = p.sum(-1, keepdim=True)
    o = (torch.matmul(p[..., :P], vp) + torch.matmul(p[..., P:], v)) / z
    lse = (m + torch.log(z)).squeeze(-1)
    return [o.reshape(B, Hq, Nq, D).to(st["q"].dtype), lse.reshape(B, Hq, Nq)]


def _plain_prompt(st):
    case = st["case"]
    Hq, Hkv, D, P = case["Hq"], case["Hkv"], case["D"], case["P"]
    G, scale, train = Hq // Hkv, 1.0 / math.sqrt(case["D"]), case["train"]
    q, k, v, kp, vp = (st[n].float().transpose(0, 1) for n in ("q", "k", "v", "kp", "vp"))
    if train:
        do = st["do"].float().transpose(0, 1)
        dkp, dvp = torch.zeros_like(kp), torch.zeros_like(vp)
    outs = {n: [] for n in ("o", "lse", "dq", "dk", "dv")}
    at = 0
    for n in st["lens"]:
        rows = slice(at, at + n)
        at += n
        keys = torch.cat([kp, k[:, rows]], 1)                           # [Hkv, P + n, D]
        vals = torch.cat([vp, v[:, rows]], 1)
        qs = q[:, rows].reshape(Hkv, G, n, D)
        s = torch.matmul(qs, keys[:, None].transpose(-1, -2)) * scale   # [Hkv, G, n, P + n]
        i = torch.arange(n, device=_DEV)
        keep = torch.cat([torch.ones(n, P, dtype=torch.bool, device=_DEV), i[None] <= i[:, None]], 1)
        s = torch.where(keep, s, torch.full_like(s, -math.inf))
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - m)
        z = p.sum(-1, keepdim=True)
        p = p / z
        o = torch.matmul(p, vals[:, None])
        outs["o"].append(o.reshape(Hq, n, D).transpose(0, 1))
        outs["lse"].append((m + torch.log(z)).reshape(Hq, n))
        if train:
            g = do[:, rows].reshape(Hkv, G, n, D)
            dp = torch.matmul(g, vals[:, None].transpose(-1, -2))
            ds = p * (dp - (g * o).sum(-1, keepdim=True)) * scale
            dkeys = torch.matmul(ds.transpose(-1, -2), qs).sum(1)
            dvals = torch.matmul(p.transpose(-1, -2), g).sum(1)
            dkp += dkeys[:, :P]
            dvp += dvals[:, :P]
            outs["dq"].append(torch.matmul(ds, keys[:, None]).reshape(Hq, n, D).transpose(0, 1))
            outs["dk"].append(dkeys[:, P:].transpose(0, 1))
            outs["dv"].append(dvals[:, P:].transpose(0, 1))
    dt = st["q"].dtype
    res = [torch.cat(outs["o"]).to(dt), torch.cat(outs["lse"], 1)]
    if train:
        res += [torch.cat(outs[n]).to(dt) for n in ("dq", "dk", "dv")]
        res += [dkp.transpose(0, 1).to(dt), dvp.transpose(0, 1).to(dt)]
    return res


def _angles(st):
    """Angles in 64 bits, [.., rows, pairs] before the head axis is put in."""
    pos = st["positions"].double()
    axis = [a for a, n in enumerate(st["sections"]) for _ in range(n)]
    per_pair = pos[torch.tensor(axis, device=_DEV)]                     # [pairs, (B,) N]
    return per_pair.movedim(0, -1) * st["inv_freq"].double()


def _cos_sin(st):
    ang = _angles(st)
    # [N, 1, pairs] beside packed heads, [B, 1, N, pairs] beside [B, H, N, D]
    ang = ang.unsqueeze(1)
    return ang.cos().float(), ang.sin().float()


def _rotate(x, cos, sin, interleaved):
    pairs = cos.shape[-1]
    if interleaved:
        a, b = x[..., 0:2 * pairs:2], x[..., 1:2 * pairs:2]
        rot = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :pairs], x[..., pairs:2 * pairs]
        rot = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([rot, x[..., 2 * pairs:]], -1)


def _plain_rotary(st):
    case = st["case"]
    cos, sin = _cos_sin(st)
    il = case["interleaved"]
    outs = [_rotate(st[n].float(), cos, sin, il).to(st[n].dtype) for n in ("q", "k")]
    if case["train"]:
        outs += [_rotate(st[n].float(), cos, -sin, il).to(st[n].dtype) for n in ("dq", "dk")]
    return outs


def _plain_qk_norm(st):
    case = st["case"]
    cos, sin = _cos_sin(st)
    il = case["interleaved"]
    outs, grads, wgrads = [], [], []
    for n in ("q", "k"):
        x, w = st[n].float(), st[n + "w"]
        rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS)
        xh = x * rstd
        outs.append(_rotate(xh * w, cos, sin, il).to(st[n].dtype))
        if case["train"]:
            dy = _rotate(st["d" + n].float(), cos, -sin, il)
            gw = dy * w
            dx = rstd * (gw - xh * (gw * xh).mean(-1, keepdim=True))
            grads.append(dx.to(st[n].dtype))
            wgrads.append((dy * xh).reshape(-1, x.shape[-1]).sum(0))
    return outs + grads + wgrads


# ---------------------------------------------------------- framework's calls


def _own_decode(st):
    from exact_attention_83_gb300 import fa
    return list(fa.attention_decode(st["q"], st["kp"], st["vp"], st["k"], st["v"], st["lens"],
                                    causal=True))


def _own_prompt(st):
    from exact_attention_83_gb300 import fa
    cu, most = st["cu"], st["most"]
    args = (st["q"], st["k"], st["v"], st["kp"], st["vp"])
    o, lse = fa.attention_prefix_fwd(*args, cu, cu, most, most, causal=True)
    if not st["case"]["train"]:
        return [o, lse]
    return [o, lse, *fa.attention_prefix_bwd(*args, o, lse, st["do"], cu, cu, most, most,
                                             causal=True)]


def _own_rotary(st):
    from exact_attention_83_gb300 import fa
    rot = (st["positions"], st["inv_freq"], st["sections"], st["case"]["interleaved"])
    outs = list(fa.rotary_fwd(st["q"], st["k"], *rot))
    if st["case"]["train"]:
        outs += fa.rotary_bwd(st["dq"], st["dk"], *rot)
    return outs


def _own_qk_norm(st):
    from exact_attention_83_gb300 import fa
    rot = (st["positions"], st["inv_freq"], st["sections"], st["case"]["interleaved"])
    args = (st["q"], st["k"], st["qw"], st["kw"])
    outs = list(fa.qk_norm_rotary_fwd(*args, *rot, eps=_EPS))
    if st["case"]["train"]:
        outs += fa.qk_norm_rotary_bwd(*args, st["dq"], st["dk"], *rot, eps=_EPS)
    return outs


_PLAIN = {"decode": _plain_decode, "prompt": _plain_prompt, "rotary": _plain_rotary,
          "qk_norm": _plain_qk_norm}
_OWN = {"decode": _own_decode, "prompt": _own_prompt, "rotary": _own_rotary,
        "qk_norm": _own_qk_norm}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------- definition in 64 bits


def _exact_decode(st):
    """Request by request: softmax over the keys that a query sees."""
    case = st["case"]
    Hq, Hkv, Nq, D = case["Hq"], case["Hkv"], case["Nq"], case["D"]
    G = Hq // Hkv
    kp, vp = st["kp"].double(), st["vp"].double()
    o = torch.empty(case["B"], Hq, Nq, D, dtype=torch.float64, device=_DEV)
    lse = torch.empty(case["B"], Hq, Nq, dtype=torch.float64, device=_DEV)
    for b, n in enumerate(st["lens"].tolist()):
        for t in range(Nq):
            own_keys = max(0, n - Nq + t + 1)
            keys = torch.cat([kp, st["k"][b, :, :own_keys].double()], 1)
            vals = torch.cat([vp, st["v"][b, :, :own_keys].double()], 1)
            q = st["q"][b, :, t].double().reshape(Hkv, G, D)
            s = torch.einsum("hgd,hnd->hgn", q, keys) / math.sqrt(D)
            lse[b, :, t] = torch.logsumexp(s, -1).reshape(Hq)
            o[b, :, t] = torch.einsum("hgn,hnd->hgd", torch.softmax(s, -1), vals).reshape(Hq, D)
    return [o, lse]


def _exact_prompt(st):
    """Head by head and sequence by sequence, the gradient by differentiation
    of sum(dO o O)."""
    case = st["case"]
    Hq, Hkv, D, P, train = case["Hq"], case["Hkv"], case["D"], case["P"], case["train"]
    G = Hq // Hkv
    total = st["q"].shape[0]
    f64 = dict(dtype=torch.float64, device=_DEV)
    o, lse = torch.empty(total, Hq, D, **f64), torch.empty(Hq, total, **f64)
    grads = {n: torch.zeros(st[n].shape, **f64) for n in ("q", "k", "v", "kp", "vp")}
    for h in range(Hq):
        hk = h // G
        at = 0
        for n in st["lens"]:
            rows = slice(at, at + n)
            at += n
            x = {"q": st["q"][rows, h], "k": st["k"][rows, hk], "v": st["v"][rows, hk],
                 "kp": st["kp"][:, hk], "vp": st["vp"][:, hk]}
            x = {key: t.double().requires_grad_(train) for key, t in x.items()}
            s = torch.cat([x["q"] @ x["kp"].T, x["q"] @ x["k"].T], 1) / math.sqrt(D)
            hide = torch.ones(n, n, dtype=torch.bool, device=_DEV).triu(1)
            s = s.masked_fill(torch.cat([hide.new_zeros(n, P), hide], 1), -math.inf)
            oh = torch.softmax(s, -1) @ torch.cat([x["vp"], x["v"]])
            o[rows, h], lse[h, rows] = oh.detach(), torch.logsumexp(s.detach(), -1)
            if train:
                got = torch.autograd.grad(oh, list(x.values()), st["do"][rows, h].double())
                grads["q"][rows, h] = got[0]
                grads["k"][rows, hk] += got[1]
                grads["v"][rows, hk] += got[2]
                grads["kp"][:, hk] += got[3]
                grads["vp"][:, hk] += got[4]
    return [o, lse] + ([grads[n] for n in ("q", "k", "v", "kp", "vp")] if train else [])


def _turn(x, st, sign):
    """The rotation as a product of complex numbers."""
    il = st["case"]["interleaved"]
    parts = []
    for a, f in enumerate(torch.split(st["inv_freq"], st["sections"])):
        parts.append(st["positions"][a].double()[..., None] * f.double())
    ang = torch.cat(parts, -1)
    ang = ang[:, None]
    n = ang.shape[-1]
    z = torch.polar(torch.ones_like(ang), sign * ang)
    if il:
        w = torch.view_as_complex(x[..., :2 * n].unflatten(-1, (n, 2)).contiguous()) * z
        return torch.cat([torch.view_as_real(w).flatten(-2), x[..., 2 * n:]], -1)
    w = torch.complex(x[..., :n].contiguous(), x[..., n:2 * n].contiguous()) * z
    return torch.cat([w.real, w.imag, x[..., 2 * n:]], -1)


def _exact_rotary(st):
    outs = [_turn(st[n].double(), st, 1.0) for n in ("q", "k")]
    if st["case"]["train"]:
        outs += [_turn(st[n].double(), st, -1.0) for n in ("dq", "dk")]
    return outs


def _exact_qk_norm(st):
    """Gradients by differentiation of the definition."""
    train = st["case"]["train"]
    outs, dxs, dws = [], [], []
    for n in ("q", "k"):
        x = st[n].double().requires_grad_(train)
        w = st[n + "w"].double().requires_grad_(train)
        y = _turn(x / torch.sqrt(x.square().mean(-1, keepdim=True) + _EPS) * w, st, 1.0)
        outs.append(y.detach())
        if train:
            dx, dw = torch.autograd.grad(y, (x, w), st["d" + n].double())
            dxs.append(dx)
            dws.append(dw)
    return outs + dxs + dws


def exact(case, seed):
    st = prepare(case, seed)
    return {"decode": _exact_decode, "prompt": _exact_prompt, "rotary": _exact_rotary,
            "qk_norm": _exact_qk_norm}[case["op"]](st)
