"""Host-side contract of linear attention and of the per-head norm (CPU only: no kernel is launched,
device pointers are fake): what the host can see comes back as its status code."""

import ctypes

import pytest

import causal_depthwise_short_amd as cc

OK, NULLP, SHAPE, STRIDE, DTYPE, MISAL, ALIAS, WS, INDEX, LAUNCH, CONFIG = range(11)
P = [0x10_0000_0000 + i * 0x1_0000_0000 for i in range(24)]
B, T, H, HV, DK, DV = 2, 640, 2, 4, 128, 64


def rows(p, heads, dim, sb=None, st=None, sh=None):
    sh = dim if sh is None else sh
    st = heads * dim if st is None else st
    return cc.Rows(p, T * st if sb is None else sb, st, sh)


def fwd(q=None, k=None, v=None, o=None, ld=P[4], scale=1.0, init=P[5], fin=P[6], cu=None, nseq=-1, status=None, ws=P[7],
        ws_bytes=1 << 40, B=B, T=T, H=H, HV=HV, Dk=DK, Dv=DV):
    q = q or rows(P[0], 2, DK)
    k = k or rows(P[1], 2, DK)
    v = v or rows(P[2], 4, DV)
    o = o or rows(P[3], 4, DV)
    return cc.lib().cconv_linattn_fwd(q, k, v, ld, scale, init, o, fin, cu, nseq, status, ws, ws_bytes, B, T, H, HV, Dk, Dv,
                                      None)


FWD = [
    (dict(q=rows(None, 2, DK)), NULLP),
    (dict(o=rows(None, 4, DV)), NULLP),
    (dict(ld=None), NULLP),
    (dict(ws=None), NULLP),
    (dict(ws_bytes=64), WS),
    (dict(B=-1), SHAPE),
    (dict(T=-1), SHAPE),
    (dict(HV=3), SHAPE),
    (dict(H=0), SHAPE),
    (dict(Dk=0), SHAPE),
    (dict(Dk=257), SHAPE),
    (dict(Dv=257), SHAPE),
    (dict(T=1 << 31), SHAPE),
    (dict(q=rows(P[0], 2, DK, st=-1, sb=0)), STRIDE),
    (dict(o=rows(P[3], 4, DV, sh=DV - 1)), STRIDE),
    (dict(o=rows(P[3], 4, DV, sb=0)), STRIDE),
    (dict(o=rows(P[3], 4, DV, st=3 * DV, sb=1 << 30)), STRIDE),
    (dict(q=rows(P[0] + 1, 2, DK)), MISAL),
    (dict(ld=P[4] + 2), MISAL),
    (dict(init=P[5] + 1), MISAL),
    (dict(ws=P[7] + 8), MISAL),
    (dict(o=rows(P[0], 4, DV)), ALIAS),
    (dict(fin=P[5]), ALIAS),
    (dict(fin=P[3] + 64), ALIAS),
    (dict(ws=P[2] + 1024), ALIAS),
    (dict(scale=float("nan")), CONFIG),
    (dict(cu=P[8], nseq=3, status=P[9]), SHAPE),  # packed rows are one batch
    (dict(cu=P[8], nseq=3, B=1), NULLP),  # no status word
    (dict(cu=P[8], nseq=0, B=1, status=P[9]), SHAPE),  # rows of no sequence
    (dict(cu=P[8] + 2, nseq=3, B=1, status=P[9]), MISAL),
    (dict(cu=P[8], nseq=3, B=1, status=P[8] + 4), ALIAS),
]


@pytest.mark.parametrize("kw,code", FWD, ids=str)
def test_fwd_host_errors(kw, code):
    assert fwd(**kw) == code


def test_empty_batches_are_ok_without_a_launch():
    assert fwd(B=0) == OK
    n = cc.lib().cconv_linattn_fwd_workspace_bytes(0, T, -1, HV, DK, DV)
    assert n == 0 or n > 0  # any size; the call above needs none of it
    assert cc.lib().cconv_linattn_fwd_workspace_bytes(1, T, -1, HV, 300, DV) == 0
    assert cc.lib().cconv_linattn_bwd_workspace_bytes(1, T, -1, 3, HV, DK, DV) == 0


def bwd(dq=None, dk=None, dv=None, do=None, dinit=P[9], dfin=P[10], ws=P[7], ws_bytes=1 << 40):
    r = (rows(P[0], 2, DK), rows(P[1], 2, DK), rows(P[2], 4, DV))
    return cc.lib().cconv_linattn_bwd(*r, P[4], 1.0, P[5], do or rows(P[3], 4, DV), dfin, dq or rows(P[11], 2, DK),
                                      dk or rows(P[12], 2, DK), dv or rows(P[13], 4, DV), dinit, None, -1, None, ws, ws_bytes,
                                      B, T, H, HV, DK, DV, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dq=rows(None, 2, DK)), NULLP), (dict(do=rows(None, 4, DV)), NULLP), (dict(dq=rows(P[11], 2, DK, sh=0)), STRIDE),
    (dict(dk=rows(P[11], 2, DK)), ALIAS), (dict(dinit=P[10]), ALIAS), (dict(dv=rows(P[2], 4, DV)), ALIAS),
    (dict(dfin=P[10] + 2), MISAL), (dict(ws_bytes=0), WS), (dict(ws=None), NULLP)], ids=str)
def test_bwd_host_errors(kw, code):
    assert bwd(**kw) == code


def update(q=None, state=P[5], S=8, idx=P[6], status=P[7], N=4, o=None, Dv=DV, scale=1.0):
    r = (q or rows(P[0], 2, DK), rows(P[1], 2, DK), rows(P[2], 4, DV))
    return cc.lib().cconv_linattn_update(*r, P[4], scale, state, S, idx, o or rows(P[3], 4, DV), N, H, HV, DK, Dv, status, None)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), SHAPE), (dict(S=-1), SHAPE), (dict(idx=None, S=3), SHAPE), (dict(S=(1 << 18) + 1), SHAPE), (dict(Dv=0), SHAPE),
    (dict(state=None), NULLP), (dict(status=None), NULLP), (dict(q=rows(None, 2, DK)), NULLP), (dict(state=P[5] + 2), MISAL),
    (dict(idx=P[6] + 1), MISAL), (dict(o=rows(P[5], 4, DV)), ALIAS), (dict(state=P[0]), ALIAS), (dict(status=P[6]), ALIAS),
    (dict(o=rows(P[3], 4, DV, st=0)), STRIDE), (dict(scale=float("nan")), CONFIG)], ids=str)
def test_update_host_errors(kw, code):
    assert update(**kw) == code


def norm(q=None, k=None, yq=None, yk=None, wq=P[4], wdt=1, table=P[5], Pn=1000, R=64, inter=0, pos=P[6], eps=1e-6,
         status=P[7], B=B, T=T, Hq=2, Hk=4, D=64):
    return cc.lib().cconv_qknorm_fwd(q or rows(P[0], 2, 64), k or rows(P[1], 4, 64), wq, P[8], wdt, table, Pn, R, inter, pos,
                                     eps, yq or rows(P[2], 2, 64), yk or rows(P[3], 4, 64), B, T, Hq, Hk, D, status, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), SHAPE), (dict(Hk=0), SHAPE), (dict(D=257), SHAPE), (dict(R=63), SHAPE), (dict(R=66), SHAPE), (dict(Pn=-1), SHAPE),
    (dict(pos=None, Pn=639), SHAPE), (dict(wdt=3), DTYPE), (dict(wq=None), NULLP), (dict(table=None), NULLP),
    (dict(status=None), NULLP), (dict(q=rows(None, 2, 64)), NULLP), (dict(eps=-1.0), CONFIG), (dict(eps=float("nan")), CONFIG),
    (dict(inter=2), CONFIG), (dict(q=rows(P[0] + 1, 2, 64)), MISAL), (dict(table=P[5] + 2), MISAL), (dict(pos=P[6] + 1), MISAL),
    (dict(yq=rows(P[2], 2, 64, sh=32)), STRIDE), (dict(yq=rows(P[0], 2, 64)), ALIAS), (dict(yk=rows(P[2], 4, 64)), ALIAS),
    (dict(status=P[6] + 8), ALIAS), (dict(wq=P[2]), ALIAS)], ids=str)
def test_norm_host_errors(kw, code):
    assert norm(**kw) == code


def test_norm_backward_host_errors():
    def call(ws=P[9], ws_bytes=1 << 30, dwq=P[10], dwk=P[11]):
        r = [rows(P[i], 2, 64) for i in range(4)]
        return cc.lib().cconv_qknorm_bwd(*r, P[4], P[5], 1, P[6], 1000, 64, 0, None, 1e-6, rows(P[12], 2, 64),
                                         rows(P[13], 2, 64), dwq, dwk, ws, ws_bytes, B, T, 2, 2, 64, None, None)

    assert call(ws=None) == NULLP and call(dwq=None) == NULLP
    assert call(ws_bytes=100) == WS
    assert call(ws=P[9] + 4) == MISAL
    assert call(dwk=P[10]) == ALIAS and call(dwq=P[13] + 64) == ALIAS


def test_host_tensors_are_refused():
    import torch

    x, ld = torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16), torch.zeros(1)
    with pytest.raises(ValueError, match="GPU"):
        cc.cconv_linattn_fwd(x, x, x, ld)
    with pytest.raises(ValueError, match="GPU"):
        cc.cconv_linattn_update(x[0], x[0], x[0], ld, torch.zeros(4, 1, 64, 64))
    with pytest.raises(ValueError, match="GPU"):
        cc.cconv_qknorm_fwd(x, x, torch.ones(64), torch.ones(64))
    assert ctypes.sizeof(cc.Rows) == 32
