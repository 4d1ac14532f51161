"""What the behaviour-history entry points refuse, on the host, before anything
is enqueued (no GPU work: the pointers are never dereferenced)."""
import ctypes

import pytest

from deep_learning_recommendation_amd import _lib as C

F, BF, I8 = C.DLRM_F32, C.DLRM_BF16, C.DLRM_I8
P, ODD4, ODD2 = 0x10000, 0x10004, 0x10002
INV, WS, UNS, OK = C.DLRM_E_INVALID, C.DLRM_E_WORKSPACE, C.DLRM_E_UNSUPPORTED, C.DLRM_OK


def change(base, **kw):
    return [kw.get(k, v) for k, v in base.items()]


EMBED = dict(table=P, td=BF, rows=100, d=64, tok=P, n=10, scale=1.0, out=P, od=BF, ld=64, st=None)


@pytest.mark.parametrize("kw", [dict(table=None), dict(tok=None), dict(out=None), dict(td=I8), dict(od=7), dict(rows=0),
                                dict(d=6), dict(d=2048), dict(d=0), dict(n=-1), dict(ld=60), dict(ld=66), dict(table=ODD4),
                                dict(out=ODD2), dict(td=F, table=0x10008)])
def test_token_embed_fwd(kw):
    assert C.lib().dlrm_token_embed_fwd(*change(EMBED, **kw)) == INV


def test_token_embed_fwd_nothing_to_do():
    assert C.lib().dlrm_token_embed_fwd(*change(EMBED, n=0, tok=None, out=None)) == OK


GRAD = dict(tok=P, n=10, dout=P, dd=BF, ld=64, rows=100, d=64, scale=1.0, dT=P, add=0, ws=P, nws=1 << 24, st=None)


@pytest.mark.parametrize("kw,status", [(dict(tok=None), INV), (dict(dout=None), INV), (dict(dT=None), INV), (dict(dT=ODD4), INV),
                                       (dict(dd=I8), INV), (dict(ld=32), INV), (dict(rows=0), INV), (dict(d=10), INV),
                                       (dict(n=1 << 31), INV), (dict(n=-1), INV), (dict(rows=0xFFFFFFFF), UNS),
                                       (dict(ws=None), WS), (dict(nws=256), WS), (dict(ws=P + 64), INV),
                                       (dict(dout=ODD2), INV)])
def test_token_embed_bwd(kw, status):
    assert C.lib().dlrm_token_embed_bwd(*change(GRAD, **kw)) == status


DROP = dict(x=P, xl=64, y=P, yl=64, t=BF, rows=10, cols=64, p=0.5, rng=P, st=None)


@pytest.mark.parametrize("kw,status", [(dict(x=None), INV), (dict(y=None), INV), (dict(rng=None), INV), (dict(xl=63), INV),
                                       (dict(yl=63), INV), (dict(yl=65), INV), (dict(t=I8), INV), (dict(p=-0.1), INV),
                                       (dict(p=1.1), INV), (dict(p=float("nan")), INV), (dict(cols=0), INV),
                                       (dict(rows=-1), INV), (dict(x=P + 1, y=P + 1), INV), (dict(t=F, x=ODD2, y=ODD2), INV),
                                       (dict(rng=P + 4), INV), (dict(rows=1 << 40), UNS), (dict(rows=0, x=None), OK)])
def test_dropout(kw, status):
    assert C.lib().dlrm_dropout(*change(DROP, **kw)) == status


NORM = dict(x=P, xl=64, r=2 * P, rl=64, t=BF, w=P, n=10, d=64, eps=1e-6, p=0.5, rng=P, h=3 * P, hl=64, y=4 * P, yt=BF, yl=64,
            sb=None, rstd=P, st=None)


@pytest.mark.parametrize("kw,status", [(dict(x=None), INV), (dict(w=None), INV), (dict(y=None), INV), (dict(rng=None), INV),
                                       (dict(yt=I8), INV), (dict(yt=F), INV), (dict(t=I8, yt=I8), INV), (dict(d=0), INV),
                                       (dict(d=16385, xl=1 << 15, rl=1 << 15, hl=1 << 15, yl=1 << 15), INV),
                                       (dict(xl=60), INV), (dict(rl=60), INV), (dict(hl=60), INV), (dict(yl=60), INV),
                                       (dict(eps=-1.0), INV), (dict(p=2.0), INV), (dict(n=-1), INV), (dict(x=P + 1), INV),
                                       (dict(h=P, hl=128), INV), (dict(h=2 * P, hl=128), INV), (dict(n=1 << 40), UNS),
                                       (dict(n=0, x=None), OK)])
def test_add_rmsnorm_fwd(kw, status):
    assert C.lib().dlrm_add_rmsnorm_fwd(*change(NORM, **kw)) == status


NBWD = dict(dy=P, dyl=64, dh=2 * P, dhl=64, h=3 * P, hl=64, t=BF, w=P, rstd=P, n=10, d=64, p=0.5, rng=P, dx=4 * P, dxl=64,
            dr=5 * P, drl=64, dw=P, ws=P, nws=1 << 24, st=None)


@pytest.mark.parametrize("kw,status", [(dict(dy=None), INV), (dict(h=None), INV), (dict(w=None), INV), (dict(rstd=None), INV),
                                       (dict(dw=None), INV), (dict(dx=None, dr=None), INV), (dict(rng=None), INV),
                                       (dict(dyl=1), INV), (dict(dhl=1), INV), (dict(hl=1), INV), (dict(dxl=1), INV),
                                       (dict(drl=1), INV), (dict(t=I8), INV), (dict(dx=5 * P), INV), (dict(dr=3 * P), INV),
                                       (dict(dx=P, dxl=128), INV), (dict(dr=2 * P, drl=128), INV), (dict(ws=None), WS),
                                       (dict(nws=0), WS), (dict(ws=P + 8), INV), (dict(d=0), INV), (dict(p=-1.0), INV),
                                       (dict(n=1 << 40), UNS)])
def test_add_rmsnorm_bwd(kw, status):
    assert C.lib().dlrm_add_rmsnorm_bwd(*change(NBWD, **kw)) == status


def _s(name, p=P):
    return {name: p, name + "t": 384, name + "h": 64}


ATT = dict(**_s("q"), **_s("k"), **_s("v"), t=BF, off=P, B=4, H=2, m=100, dk=64, dv=64, lam=P, sc=1.0, s0=None,
           **_s("o"), s=None, ws=P, nws=1 << 40, st=None)
ATTB = dict(**_s("q"), **_s("k"), **_s("v"), **_s("do"), t=BF, off=P, B=4, H=2, m=100, dk=64, dv=64, lam=P, sc=1.0, s0=None,
            ds=None, **_s("dq"), **_s("dkk"), **_s("dvv"), ds0=P, ws=P, nws=1 << 40, st=None)
SHAPE_REFUSALS = [dict(off=None), dict(lam=None), dict(B=0), dict(H=0), dict(m=-1), dict(dk=4), dict(dk=136), dict(dk=20),
                  dict(dv=12), dict(dv=0), dict(t=I8), dict(q=None), dict(k=None), dict(v=None), dict(q=P + 8),
                  dict(kt=100), dict(vh=60), dict(s0=P + 8), dict(ws=P + 8)]


@pytest.mark.parametrize("kw", SHAPE_REFUSALS + [dict(o=None), dict(ot=12), dict(s=P + 4)])
def test_linattn_fwd(kw):
    assert C.lib().dlrm_linattn_fwd(*change(ATT, **kw)) == INV


@pytest.mark.parametrize("kw", SHAPE_REFUSALS + [dict(do=None), dict(dq=None), dict(dkk=None), dict(dvv=None), dict(dqt=3),
                                                 dict(ds=P), dict(ds=P + 4), dict(ds0=P + 4)])
def test_linattn_bwd(kw):
    assert C.lib().dlrm_linattn_bwd(*change(ATTB, **kw)) == INV


def test_linattn_too_many_histories():
    assert C.lib().dlrm_linattn_fwd(*change(ATT, B=1 << 30)) == UNS
    assert C.lib().dlrm_linattn_bwd(*change(ATTB, B=1 << 30)) == UNS


def test_linattn_workspace():
    """A long history is cut into segments whose states need room."""
    lib = C.lib()
    for size, call, base in ((lib.dlrm_linattn_workspace_size, lib.dlrm_linattn_fwd, ATT),
                             (lib.dlrm_linattn_bwd_workspace_size, lib.dlrm_linattn_bwd, ATTB)):
        need = size(1, 1, 100000, 64, 64)
        assert need % 256 == 0 and size(4, 2, -1, 64, 64) == 0 and size(0, 2, 100, 64, 64) == 0
        if need:
            assert call(*change(base, B=1, H=1, m=100000, nws=need - 1)) == WS
            assert call(*change(base, B=1, H=1, m=100000, ws=None)) == WS


STEP = dict(**_s("q"), **_s("k"), **_s("v"), t=BF, B=4, H=2, dk=64, dv=64, lam=P, sc=1.0, s=P, slots=None, **_s("o"), st=None)


@pytest.mark.parametrize("kw", [dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(lam=None), dict(s=None),
                                dict(s=P + 8), dict(t=I8), dict(H=0), dict(B=-1), dict(dk=4), dict(dv=129), dict(dv=136),
                                dict(qt=9), dict(oh=4), dict(q=P + 2)])
def test_linattn_step(kw):
    assert C.lib().dlrm_linattn_step(*change(STEP, **kw)) == INV


def test_linattn_step_limits():
    assert C.lib().dlrm_linattn_step(*change(STEP, B=0, q=None)) == OK
    assert C.lib().dlrm_linattn_step(*change(STEP, B=1 << 30)) == UNS


def test_bindings_want_contiguous_heads():
    import torch

    t = torch.zeros(4, 6, 8)
    assert C._heads(t[:, ::2])[1:] == (48, 16)
    with pytest.raises(ValueError):
        C._heads(t[:, :, ::2])
    with pytest.raises(ValueError):
        C._heads(t[0])
    assert ctypes.sizeof(ctypes.c_void_p) == 8


def test_bindings_refuse_mixed_types():
    """An array read as another type would be read past its end, so the
    bindings compare types before the call."""
    import torch

    f, b, i = torch.zeros(2, 2, 8), torch.zeros(2, 2, 8, dtype=torch.bfloat16), torch.zeros(8, dtype=torch.int64)
    half, short = f.half(), i.int()
    calls = [
        lambda: C.dlrm_token_embed_fwd(half, 2, 8, i, 2, 1.0, f, 8),
        lambda: C.dlrm_token_embed_fwd(f, 2, 8, short, 2, 1.0, f, 8),
        lambda: C.dlrm_token_embed_fwd(f, 2, 8, i, 2, 1.0, half, 8),
        lambda: C.dlrm_token_embed_bwd(short, 2, f, 8, 2, 8, 1.0, f, False, f),
        lambda: C.dlrm_token_embed_bwd(i, 2, f, 8, 2, 8, 1.0, b, False, f),
        lambda: C.dlrm_dropout(f, 8, b, 8, 2, 8, 0.5, i),
        lambda: C.dlrm_dropout(half, 8, half, 8, 2, 8, 0.5, i),
        lambda: C.dlrm_dropout(f, 8, f, 8, 2, 8, 0.5, short),
        lambda: C.dlrm_add_rmsnorm_fwd(f, 8, b, 8, f, 2, 8, 0.1, 0.0, None, None, 0, f, 8, None, None),
        lambda: C.dlrm_add_rmsnorm_fwd(f, 8, None, 8, b, 2, 8, 0.1, 0.0, None, None, 0, f, 8, None, None),
        lambda: C.dlrm_add_rmsnorm_fwd(f, 8, None, 8, f, 2, 8, 0.1, 0.0, None, b, 8, f, 8, None, None),
        lambda: C.dlrm_add_rmsnorm_fwd(f, 8, None, 8, f, 2, 8, 0.1, 0.0, None, None, 0, b, 8, None, None),
        lambda: C.dlrm_add_rmsnorm_fwd(f, 8, None, 8, f, 2, 8, 0.1, 0.0, None, None, 0, f, 8, None, b),
        lambda: C.dlrm_add_rmsnorm_bwd(f, 8, None, 0, f, 8, f, f, 2, 8, 0.0, None, b, 8, None, 0, f, f),
        lambda: C.dlrm_add_rmsnorm_bwd(b, 8, b, 8, f, 8, f, f, 2, 8, 0.0, None, b, 8, None, 0, f, f),
        lambda: C.dlrm_linattn_fwd(f, b, f, i, 1, 2, 2, 8, 8, f, 1.0, None, f, None, None),
        lambda: C.dlrm_linattn_fwd(f, f, f, short, 1, 2, 2, 8, 8, f, 1.0, None, f, None, None),
        lambda: C.dlrm_linattn_fwd(b, b, b, i, 1, 2, 2, 8, 8, b, 1.0, None, b, None, None),
        lambda: C.dlrm_linattn_fwd(b, b, b, i, 1, 2, 2, 8, 8, f, 1.0, b, b, None, None),
        lambda: C.dlrm_linattn_bwd(b, b, b, b, i, 1, 2, 2, 8, 8, f, 1.0, None, None, b, f, b, None, None),
        lambda: C.dlrm_linattn_step(f, f, f, 2, 2, 8, 8, f, 1.0, b, None, f),
        lambda: C.dlrm_linattn_step(f, f, f, 2, 2, 8, 8, f, 1.0, f, short, f),
        lambda: C.dlrm_linattn_step(f, f, f, 2, 2, 8, 8, f, 1.0, f, None, b),
    ]
    for n, call in enumerate(calls):
        with pytest.raises(TypeError):
            call()
            pytest.fail(f"call {n} was not refused")


@pytest.mark.parametrize("stride", [-8, 1 << 22])
@pytest.mark.parametrize("which", ["qt", "kt", "vt", "ot"])
def test_linattn_row_strides(which, stride):
    assert C.lib().dlrm_linattn_step(*change(STEP, **{which: stride})) == INV
