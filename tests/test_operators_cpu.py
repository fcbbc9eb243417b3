"""Argument checks of the rotation and decode entry points that need no GPU:
invalid arguments give the documented status before any device work."""

from __future__ import annotations

import ctypes

import pytest
import torch

from exact_attention_83_gb300 import build as fabuild
from exact_attention_83_gb300 import fa

FAKE = 0x100000          # 16-byte aligned, never dereferenced
S4 = ctypes.c_int64 * 4


@pytest.fixture(scope="module")
def lib():
    fabuild.build()
    return fa.load_library()


def _rot(**kw):
    pr = fa.RotaryProblem()
    d = dict(B=2, N=10, Hq=4, Hkv=2, D=64, dtype=2, interleaved=0, n_axes=1, sections=(32, 0, 0, 0),
             inv_freq=FAKE, positions=FAKE, pos_stride=(0, 0, 1), positions_64=1, weight_f32=1,
             q_weight=None, k_weight=None, eps=1e-6)
    d.update(kw)
    for name, v in d.items():
        if name in ("sections", "pos_stride"):
            for i, x in enumerate(v):
                getattr(pr, name)[i] = x
        else:
            setattr(pr, name, v)
    return pr


ST = S4(4 * 640, 640, 64, 1)


def _fwd(lib, pr, q=FAKE, sq=ST, sko=ST):
    return lib.fa_rotary_fwd(ctypes.byref(pr) if pr is not None else None, q, sq, FAKE, ST, FAKE, ST,
                             FAKE, sko, None)


def test_rotary_validation(lib):
    assert _fwd(lib, None) == 1
    for kw, code in ((dict(B=0), 2), (dict(N=0), 2), (dict(Hq=0), 2), (dict(Hkv=0), 2), (dict(D=48), 3),
                     (dict(dtype=5), 4), (dict(n_axes=0), 11), (dict(n_axes=5), 11),
                     (dict(sections=(12, 0, 0, 0)), 11), (dict(sections=(40, 0, 0, 0)), 11),
                     (dict(n_axes=2), 11), (dict(n_axes=2, sections=(40, -8, 0, 0)), 11),
                     (dict(inv_freq=None), 1), (dict(positions=None), 1), (dict(positions=FAKE + 4), 6),
                     (dict(inv_freq=FAKE + 2), 6), (dict(pos_stride=(0, -1, 1)), 5),
                     (dict(q_weight=FAKE), 1), (dict(q_weight=FAKE, k_weight=FAKE + 2), 6),
                     (dict(q_weight=FAKE, k_weight=FAKE, eps=-1.0), 11),
                     (dict(q_weight=FAKE, k_weight=FAKE, eps=float("nan")), 11),
                     (dict(Hq=1 << 21), 2)):
        assert _fwd(lib, _rot(**kw)) == code, kw
    assert _fwd(lib, _rot(positions=FAKE + 4, positions_64=0), q=None) == 1     # int32 positions: aligned
    assert _fwd(lib, _rot(), q=FAKE + 8) == 6
    assert _fwd(lib, _rot(), sq=S4(4 * 640, 640, 64, 2)) == 5
    assert _fwd(lib, _rot(), sq=S4(4 * 640, 0, 64, 1)) == 5       # broadcast heads
    assert _fwd(lib, _rot(), sko=S4(4 * 640, 640, 0, 1)) == 5
    assert _fwd(lib, _rot(), sq=S4(4 * 640, 640, 68, 1)) == 6


def test_rotary_gradient_validation(lib):
    norm = dict(q_weight=FAKE, k_weight=FAKE)
    assert lib.fa_rotary_bwd_workspace_bytes(ctypes.byref(_rot())) == 0
    assert lib.fa_rotary_bwd_workspace_bytes(None) == 0
    need = lib.fa_rotary_bwd_workspace_bytes(ctypes.byref(_rot(**norm)))
    assert need > 0 and need % (64 * 4) == 0

    def bwd(pr, q=FAKE, dwq=FAKE, ws=FAKE, nbytes=need, dk=FAKE):
        return lib.fa_rotary_bwd(ctypes.byref(pr), q, ST, FAKE, ST, FAKE, ST, FAKE, ST, FAKE, ST, dk, ST,
                                 dwq, FAKE, ws, nbytes, None)

    assert bwd(_rot(**norm), q=None) == 1
    assert bwd(_rot(**norm), dwq=None) == 1
    assert bwd(_rot(**norm), dwq=FAKE + 4) == 6
    assert bwd(_rot(**norm), ws=None) == 1
    assert bwd(_rot(**norm), nbytes=need - 1) == 12
    assert bwd(_rot(), q=None, dwq=None, ws=None, nbytes=0, dk=None) == 1      # only dk is missing


def _dec(**kw):
    pr = fa.DecodeProblem()
    d = dict(B=2, Hq=4, Hkv=2, Nq=1, D=64, P=100, S=10, seq_lens=FAKE, causal=1, scale=0.125, dtype=2)
    d.update(kw)
    for name, v in d.items():
        setattr(pr, name, v)
    return pr


def _decode(lib, pr, q=FAKE, kp=FAKE, k=FAKE, lse=FAKE, ws=FAKE, nbytes=1 << 40, sk=S4(2 * 640, 640, 64, 1),
            skp=S4(0, 6400, 64, 1)):
    st = S4(256, 64, 64, 1)
    return lib.fa_decode(ctypes.byref(pr) if pr is not None else None, q, st, kp, skp, FAKE, skp, k, sk, FAKE,
                         sk, FAKE, st, lse, ws, nbytes, None)


def test_decode_validation(lib):
    assert _decode(lib, None) == 1
    for kw, code in ((dict(dtype=0), 4), (dict(dtype=9), 4), (dict(B=0), 2), (dict(Hkv=3), 2), (dict(Nq=0), 2),
                     (dict(Nq=17), 2), (dict(P=-1), 2), (dict(S=-1), 2), (dict(D=96), 3), (dict(scale=0.0), 10),
                     (dict(seq_lens=None), 1), (dict(seq_lens=FAKE + 2), 6), (dict(B=1 << 31), 2),
                     (dict(S=1 << 31), 2), (dict(P=1 << 31), 2)):
        assert _decode(lib, _dec(**kw)) == code, kw
        assert lib.fa_decode_workspace_bytes(ctypes.byref(_dec(**kw))) == 0, kw
    assert _decode(lib, _dec(), q=None) == 1
    assert _decode(lib, _dec(), kp=None) == 1
    assert _decode(lib, _dec(), k=None) == 1
    assert _decode(lib, _dec(), lse=None) == 1
    assert _decode(lib, _dec(), ws=None) == 1
    assert _decode(lib, _dec(), ws=FAKE + 4) == 6
    assert _decode(lib, _dec(), sk=S4(0, 640, 64, 1)) == 5          # one cache for two requests
    assert _decode(lib, _dec(), skp=S4(0, 0, 64, 1)) == 5           # one prefix head for two
    need = lib.fa_decode_workspace_bytes(ctypes.byref(_dec()))
    assert need > 0 and _decode(lib, _dec(), nbytes=need - 1) == 12
    # without a prefix: no workspace; without own rows: no lengths, no cache
    assert lib.fa_decode_workspace_bytes(ctypes.byref(_dec(P=0))) == 0
    assert _decode(lib, _dec(P=0), kp=None, ws=None, nbytes=0, lse=None) == 1
    assert _decode(lib, _dec(S=0, seq_lens=None), k=None, lse=FAKE + 4) == 6


def test_python_refusals():
    """The binding refuses tensors that are not on a GPU, and shapes that do not
    fit, before it calls the library."""
    x = torch.zeros(2, 4, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        fa.rotary_fwd(x, x, torch.arange(8), torch.ones(32))
    with pytest.raises(TypeError):
        fa.attention_decode(x, x[0], x[0], x, x, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="no gradient"):
        fa.rotary(x, x, torch.arange(8), torch.ones(32, requires_grad=True))


def test_packed_structs_have_the_c_layout():
    """The binding's packed bytes are the ctypes mirrors of the C structs, field
    by field."""
    pr = _rot(n_axes=3, sections=(8, 12, 12, 0), interleaved=1, pos_stride=(7, 5, 3), weight_f32=1,
              q_weight=FAKE + 16, k_weight=FAKE + 32, eps=0.25)
    raw = fa._PACK_ROTARY(2, 10, 4, 2, 64, 2, 1, 3, 8, 12, 12, 0, FAKE, FAKE, 7, 5, 3, 1, 1, FAKE + 16,
                          FAKE + 32, 0.25)
    assert raw == bytes(pr)
    raw = fa._PACK_DECODE(2, 4, 2, 1, 64, 100, 10, FAKE, 1, 0.125, 2)
    assert raw[:76] == bytes(_dec())[:76] and len(raw) == len(bytes(_dec()))
    pr = _packed()
    pr.seed, pr.offset = 5, 6
    raw = fa._PACK_PROBLEM(3, 4, 2, 40, 50, 64, FAKE, FAKE, 100, 120, 1, 0.125, 2, 0.0, 5, 6, 0)
    assert raw == bytes(pr)


def _packed(**kw):
    pr = fa.Problem()
    d = dict(B=3, Hq=4, Hkv=2, Nq=40, Nk=50, D=64, cu_seqlens_q=FAKE, cu_seqlens_k=FAKE, total_q=100,
             total_k=120, causal=1, scale=0.125, dtype=2)
    d.update(kw)
    for name, v in d.items():
        setattr(pr, name, v)
    return pr


def test_prefix_validation(lib):
    st = S4(0, 64, 256, 1)

    def fwd(pr, P=70, q=FAKE, kp=FAKE, skp=st, so=st, lse=FAKE):
        return lib.fa_fwd_prefix(ctypes.byref(pr) if pr is not None else None, P, q, st, kp, skp, FAKE, st,
                                 FAKE, st, FAKE, st, FAKE, so, lse, None)

    def bwd(pr, P=70, dkp=FAKE, sdk=st, delta=FAKE, dq=FAKE):
        return lib.fa_bwd_prefix(ctypes.byref(pr), P, FAKE, st, FAKE, st, FAKE, st, FAKE, st, FAKE, st, FAKE,
                                 st, FAKE, delta, dq, st, dkp, st, FAKE, st, FAKE, sdk, FAKE, st, None)

    def delta(pr, P=70, q=FAKE, kp=FAKE, o=FAKE, so=st, lse=FAKE, out=FAKE):
        return lib.fa_bwd_prefix_delta(ctypes.byref(pr) if pr is not None else None, P, q, st, kp, st, FAKE, st,
                                       FAKE, st, FAKE, st, o, so, FAKE, st, lse, out, None)

    assert delta(None) == 1
    assert delta(_packed(D=96)) == 3 and delta(_packed(), P=-1) == 2
    assert delta(_packed(), q=None) == 1 and delta(_packed(), kp=None) == 1
    assert delta(_packed(), o=None) == 1 and delta(_packed(), lse=None) == 1 and delta(_packed(), out=None) == 1
    assert delta(_packed(), out=FAKE + 4) == 6 and delta(_packed(), so=S4(0, 0, 256, 1)) == 5

    assert fwd(None) == 1
    for call in (fwd, bwd):
        for kw, code in ((dict(dtype=9), 4), (dict(Hkv=3), 2), (dict(D=48), 3), (dict(scale=0.0), 10),
                         (dict(cu_seqlens_k=None), 2), (dict(cu_seqlens_q=None, cu_seqlens_k=None), 2),
                         (dict(dropout_p=0.1), 11), (dict(total_q=0), 2)):
            assert call(_packed(**kw)) == code, kw
        assert call(_packed(), P=-1) == 2
        assert call(_packed(), P=1 << 31) == 2
        assert call(_packed(Nk=1 << 30), P=(1 << 30) + 5) == 2
    assert fwd(_packed(), q=None) == 1
    assert fwd(_packed(), kp=None) == 1
    assert fwd(_packed(), kp=FAKE + 8) == 6
    assert fwd(_packed(), skp=S4(0, 0, 256, 1)) == 5
    assert fwd(_packed(), so=S4(0, 64, 0, 1)) == 5
    assert fwd(_packed(), lse=None) == 1
    assert fwd(_packed(), P=0, kp=None, lse=None) == 1           # without a prefix its pointers are ignored
    assert bwd(_packed(), dkp=None) == 1
    assert bwd(_packed(), sdk=S4(0, 64, 250, 1)) == 6
    assert bwd(_packed(), delta=None) == 1
    assert bwd(_packed(), P=0, dkp=None, dq=None) == 1
