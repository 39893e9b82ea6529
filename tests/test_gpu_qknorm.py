"""GPU tests of the per-head norm with rotation (cconv_qknorm_fwd / _bwd) against the float64 oracle.

Tolerances: everything runs in fp32 and is rounded once to bf16 (u = eps/2 = 2^-8 of the value). A norm
sums at most 256 squares (relative 2^-16 at most, far less for positive terms), and a turned channel adds
two products, so |gpu - ref| <= u |ref| + 2^-16 * (the terms' absolute values). dw sums fp32 terms over
all rows and heads: at most 2^-16 of their absolute values, plus its own rounding in bf16.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import causal_depthwise_short_amd as cc
from oracle import layer
from parity import bits, canaries_intact, guarded

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0**-8


def f64(t):
    return t.detach().float().cpu().double().numpy()


def table_of(P, R):
    if not R:
        return None
    inv = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    angle = torch.arange(P, dtype=torch.float64)[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], -1).float()


# B, T, Hq, Hk, D, R
SHAPES = [(1, 1, 1, 1, 128, 128), (2, 3, 4, 1, 128, 64), (16, 1, 16, 16, 128, 128), (1, 37, 6, 2, 80, 40), (2, 19, 3, 3, 80, 20),
          (1, 11, 5, 1, 66, 22), (1, 9, 2, 2, 72, 0), (1, 8, 3, 1, 256, 256), (1, 8, 1, 1, 256, 128), (1, 6, 2, 1, 96, 96),
          (1, 5, 3, 2, 129, 64), (1, 4, 1, 1, 255, 10), (3, 7, 2, 2, 1, 0), (1, 5, 2, 1, 2, 2), (1, 6, 1, 1, 64, 6),
          (1, 1500, 2, 1, 64, 64)]


def sides(shape, seed, fused):
    B, T, Hq, Hk, D, _ = shape
    g = torch.Generator().manual_seed(seed)
    if fused:  # slices of one projection's rows
        x = torch.randn(B, T, (Hq + 2 * Hk) * D, generator=g).to(torch.bfloat16)
        d = x.to(DEV)
        cut = lambda x: (x[:, :, :Hq * D].unflatten(-1, (Hq, D)), x[:, :, Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D)))  # noqa: E731
        return cut(x), cut(d), g
    q = torch.randn(B, T, Hq, D, generator=g).to(torch.bfloat16)
    k = torch.randn(B, T, Hk, D, generator=g).to(torch.bfloat16)
    return (q, k), (q.to(DEV), k.to(DEV)), g


def turned_size(x, w, table, pos, eps, inter):
    """The sum of the absolute values of the (at most two) products of each output."""
    t = None if table is None else np.abs(table)
    y = np.abs(layer.qknorm(x, w, None, None, eps, inter))
    if t is None:
        return y
    B, T, H, D = y.shape
    p = np.tile(np.arange(T), B) if pos is None else np.asarray(pos).reshape(-1)
    m = np.abs(layer._rotation(np.asarray(table, dtype=np.float64), p, table.shape[1], D, inter))
    return np.einsum("rij,rhj->rhi", m, y.reshape(B * T, H, D)).reshape(y.shape)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("wdt", [torch.float32, torch.bfloat16])
def test_forward_and_backward(shape, interleaved, wdt):
    B, T, Hq, Hk, D, R = shape
    (q, k), (qd, kd), g = sides(shape, D + T, fused=T % 2 == 1)
    wq, wk = ((1 + 0.1 * torch.randn(D, generator=g)).to(wdt) for _ in range(2))
    P = T + 90
    tab = table_of(P, R)
    pos = torch.randint(0, P, (B, T), generator=g, dtype=torch.int32) if T != 37 else None
    dyq, dyk = (torch.randn(x.shape, generator=g).to(torch.bfloat16) for x in (q, k))
    on = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    args = dict(positions=on(pos), eps=1e-5, interleaved=interleaved)
    yq, yk, st = cc.cconv_qknorm_fwd(qd, kd, on(wq), on(wk), on(tab), **args)
    got = cc.cconv_qknorm_bwd(qd, kd, on(dyq), on(dyk), on(wq), on(wk), on(tab), **args)
    assert (st is None) == (pos is None or R == 0)
    if st is not None:
        assert int(st) == 0 and int(got[4]) == 0
    t64, p = (None if tab is None else f64(tab)), (None if pos is None else pos.numpy())
    for name, x, w, y, dy, dx, dw in (("q", q, wq, yq, dyq, got[0], got[2]), ("k", k, wk, yk, dyk, got[1], got[3])):
        x, w, dy = f64(x), f64(w), f64(dy)
        ref, size = layer.qknorm(x, w, t64, p, 1e-5, interleaved), turned_size(x, w, t64, p, 1e-5, interleaved)
        assert np.all(np.abs(f64(y) - ref) <= U * np.abs(ref) + 2.0**-16 * size + 1e-30), name
        rdx, rdw = layer.qknorm_bwd(x, w, t64, p, 1e-5, interleaved, dy)
        s = np.sqrt(np.mean(x * x, -1, keepdims=True) + 1e-5)
        u = np.sqrt(2) * np.sqrt(np.mean(dy * dy, -1, keepdims=True) * D)  # bounds a row's turned gradients
        big = np.max(np.abs(w)) * u / s  # and with them every term of dx
        assert np.all(np.abs(f64(dx) - rdx) <= U * np.abs(rdx) + 2.0**-16 * 2 * big + 1e-30), name
        sw = (u * np.abs(x / s)).reshape(-1, D).sum(0)
        assert np.all(np.abs(f64(dw) - rdw) <= (U if wdt == torch.bfloat16 else 0) * np.abs(rdw) + 2.0**-16 * sw + 1e-30), name
    again = cc.cconv_qknorm_bwd(qd, kd, on(dyq), on(dyk), on(wq), on(wk), on(tab), **args)
    for a, b in zip(got[:4], again[:4]):
        assert torch.equal(bits(a), bits(b)), "a second call differs"


def test_special_values():
    """Zero heads, infinities and NaN stay in their own head, and in unrotated channels alone."""
    x = torch.randn(1, 4, 3, 80, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    x[0, 0, 0] = 0
    x[0, 1, 1, 70] = float("inf")
    x[0, 2, 2, 3] = float("nan")
    one, tab = torch.ones(80, device=DEV), table_of(9, 40).to(DEV)
    for inter in (False, True):
        y, _, _ = cc.cconv_qknorm_fwd(x.to(DEV), x[:, :, :1].to(DEV), one, one, tab, interleaved=inter)
        y = y.cpu()
        assert not y[0, 0, 0].any()
        odd = torch.isnan(y[0, 1, 1])
        assert odd[70] and int(odd.sum()) == 1 and not y[0, 1, 1][~odd].any()
        assert torch.isnan(y[0, 2, 2]).all()
        y[0, 1, 1] = y[0, 2, 2] = 0
        assert torch.isfinite(y).all()


def test_no_rows():
    e = torch.empty(2, 0, 3, 64, dtype=torch.bfloat16, device=DEV)
    w, tab = torch.ones(64, device=DEV), table_of(4, 64).to(DEV)
    pos = torch.empty(2, 0, dtype=torch.int32, device=DEV)
    y, _, st = cc.cconv_qknorm_fwd(e, e, w, w, tab, positions=pos)
    assert y.shape == e.shape and int(st) == 0
    *_, dwq, dwk, st = cc.cconv_qknorm_bwd(e, e, e, e, w, w, tab, positions=pos)
    assert not dwq.any() and not dwk.any() and int(st) == 0


@pytest.mark.parametrize("T", [5, 3000])
@pytest.mark.parametrize("bad", [-1, 4000, 2**31 - 1])
def test_bad_positions_write_nothing(T, bad):
    x = torch.randn(1, T, 2, 64, device=DEV).to(torch.bfloat16)
    w, tab = torch.ones(64, device=DEV), table_of(4000, 64).to(DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)[None].contiguous()
    pos[0, T - 1] = bad
    outs = [torch.full_like(x, 7.0) for _ in range(4)]
    dw = [torch.full((64,), 7.0, device=DEV) for _ in range(2)]
    _, _, st = cc.cconv_qknorm_fwd(x, x, w, w, tab, positions=pos, yq=outs[0], yk=outs[1])
    *_, st2 = cc.cconv_qknorm_bwd(x, x, x, x, w, w, tab, positions=pos, dq=outs[2], dk=outs[3], dwq=dw[0], dwk=dw[1])
    assert int(st) == 8 and int(st2) == 8
    for o in (*outs, *dw):
        assert bool((o == 7.0).all())


def test_rows_past_32_bit_offsets():
    """2.2e9 elements a tensor: the last rows come out as they do alone, bit for bit."""
    T, H = 270000, 64
    x = torch.randn(1, 64, H, 128, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(DEV)
    big = torch.zeros(1, T, H, 128, dtype=torch.bfloat16, device=DEV)
    assert big.numel() > 2**31
    big[:, -64:] = x
    w, tab = torch.ones(128, device=DEV), table_of(T, 64).to(DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)[None]
    k, kp = big[:, :, :1], x[:, :, :1]
    yq, yk, st = cc.cconv_qknorm_fwd(big, k, w, w, tab, positions=pos)
    zq, zk, _ = cc.cconv_qknorm_fwd(x, kp, w, w, tab, positions=pos[:, -64:].contiguous())
    assert int(st) == 0 and torch.equal(bits(yq[:, -64:]), bits(zq)) and torch.equal(bits(yk[:, -64:]), bits(zk))
    del yq
    dq, dk, _, _, _ = cc.cconv_qknorm_bwd(big, k, big, k, w, w, tab, positions=pos)
    eq, ek, _, _, _ = cc.cconv_qknorm_bwd(x, kp, x, kp, w, w, tab, positions=pos[:, -64:].contiguous())
    assert torch.equal(bits(dq[:, -64:]), bits(eq)) and torch.equal(bits(dk[:, -64:]), bits(ek))


def test_outputs_in_wider_rows_and_guards():
    x = torch.randn(2, 5, 3, 96, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).to(DEV)
    w, tab = torch.ones(96, device=DEV), table_of(8, 32).to(DEV)
    yq, yk, _ = cc.cconv_qknorm_fwd(x, x, w, w, tab)
    wide = torch.full((2, 5, 4, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    view = wide[:, :, :3, 16:112]
    g, buf, lo, hi = guarded(x.shape, torch.bfloat16, DEV)
    cc.cconv_qknorm_fwd(x, x, w, w, tab, yq=view, yk=g)
    assert torch.equal(bits(view), bits(yq)) and torch.equal(bits(g), bits(yk)) and canaries_intact(buf, lo, hi)
    wide[:, :, :3, 16:112] = 7.0
    assert bool((wide == 7.0).all())


def test_graph_replays_equal_the_eager_calls():
    g = torch.Generator().manual_seed(5)
    x = torch.randn(2, 700, 4, 128, generator=g).to(torch.bfloat16).to(DEV)
    dy, w, tab = x.clone(), torch.ones(128, device=DEV), table_of(4096, 128).to(DEV)
    pos = torch.randint(0, 4096, (2, 700), generator=g, dtype=torch.int32).to(DEV)

    def call():
        a = cc.cconv_qknorm_fwd(x, x, w, w, tab, positions=pos)[:2]
        return (*a, *cc.cconv_qknorm_bwd(x, x, dy, dy, w, w, tab, positions=pos)[:4])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    for r in range(3):
        x.copy_(torch.randn(x.shape, generator=g).to(torch.bfloat16))
        dy.copy_(torch.randn(x.shape, generator=g).to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, call()):
            assert torch.equal(bits(a), bits(b)), r


def test_binding_refusals():
    x = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16, device=DEV)
    w, tab = torch.ones(64, device=DEV), table_of(8, 64).to(DEV)
    for bad, kw in (((x.float(), x, w, w, tab), {}), ((x, x[:, :3], w, w, tab), {}), ((x, x, w[:32], w, tab), {}),
                    ((x, x, w, w.bfloat16(), tab), {}), ((x, x, w, w, tab.double()), {}), ((x.cpu(), x, w, w, tab), {}),
                    ((x, x, w, w, tab), dict(positions=torch.zeros(1, 3, dtype=torch.int32, device=DEV)))):
        with pytest.raises(ValueError):
            cc.cconv_qknorm_fwd(*bad, **kw)
    with pytest.raises(cc.CconvError, match="BAD_SHAPE"):  # an odd number of rotated channels
        cc.cconv_qknorm_fwd(x, x, w, w, tab[:, :63].contiguous())
    with pytest.raises(cc.CconvError, match="BAD_SHAPE"):  # more rows than positions
        cc.cconv_qknorm_fwd(x, x, w, w, tab[:3])
    with pytest.raises(cc.CconvError, match="ALIASING"):
        cc.cconv_qknorm_fwd(x, x, w, w, tab, yq=x)
    with pytest.raises(cc.CconvError, match="BAD_CONFIG"):
        cc.cconv_qknorm_fwd(x, x, w, w, tab, eps=-1.0)
