"""GPU tests of linear attention with a decay for each head (cconv_linattn_fwd / _bwd / _update)
against the float64 oracle.

Tolerances, from the roundings the header states (u = eps/2 of bf16 = 2^-8 relative, w = 2^-24 of fp32):
  * o, dq, dk, dv. The scores and the state are rounded to bf16 as operands of a matrix product (their
    terms move by at most u each), sums run in fp32 over at most a few hundred terms at a time (256 w =
    2^-16 of the terms' absolute values), then the result is rounded to bf16 (u of itself):
        |gpu - ref| <= u |ref| + (u + 2^-14) * size,   size = the sum of the terms' absolute values.
    Where errors are random (Gaussian inputs), rms errors add in squares: a rounding's rms is at most
    u / sqrt(3), the operands' and the result's together sqrt(2) u / sqrt(3) = 0.82 u of the norm:
        ||gpu - ref|| <= u ||ref||.
  * states (fp32). The weighted rows enter as a sum of two bf16 values: the second holds what the first
    rounds off (u) to within its own rounding (u), so a term moves by at most u^2 = 2^-16, by rms
    u^2 / 3. Sums and decays in fp32: 2^-16 of the absolute values.
        |gpu - ref| <= 2^-15 * size,   ||gpu - ref|| <= 2^-17 ||ref|| + 2^-20 * ||size|| / sqrt(terms)
    (the last: fp32 accumulation, which does not shrink with cancelling terms).
  * the single-token step runs in fp32 throughout: states to 8 w of their terms, o to one bf16 rounding
    plus 2^-16 of its terms.
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
    return None if t is None else t.detach().float().cpu().double().numpy()


def close(gpu, ref, size, what, norm=True):
    g = f64(gpu)
    assert g.shape == ref.shape, what
    err = np.abs(g - ref)
    lim = U * np.abs(ref) + (U + 2.0**-14) * size + 1e-30
    assert np.all(err <= lim), f"{what}: {np.max(err / lim):.2f} of the elementwise bound"
    if norm and ref.size >= 256:
        assert np.linalg.norm(g - ref) <= U * np.linalg.norm(ref), \
            f"{what}: relative norm {np.linalg.norm(g - ref) / np.linalg.norm(ref):.2e}"


def close_state(gpu, ref, size, what):
    g = f64(gpu)
    assert g.shape == ref.shape, what
    err = np.abs(g - ref)
    lim = 2.0**-15 * size + 1e-30
    assert np.all(err <= lim), f"{what}: {np.max(err / lim):.2f} of the elementwise bound"
    if ref.size >= 256:
        lim = 2.0**-17 * np.linalg.norm(ref) + 2.0**-20 * np.linalg.norm(size)
        assert np.linalg.norm(g - ref) <= lim, f"{what}: {np.linalg.norm(g - ref) / lim:.2f} of the norm bound"


def make(shape_q, shape_v, seed, decay="mixed", slice_v=False):
    """q, k, v in bf16 on the GPU; v a slice of wider rows when slice_v."""
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)  # noqa: E731
    q, k = n(*shape_q), n(*shape_q)
    if slice_v:
        wide = n(*shape_v[:-2], shape_v[-2] * shape_v[-1] + 24)
        v = wide[..., 24:].unflatten(-1, shape_v[-2:])
    else:
        v = n(*shape_v)
    HV = shape_v[-2]
    if decay == "mixed":
        ld = -torch.exp2(-8.0 * (torch.arange(HV) + 1) / HV)
        if HV > 1:
            ld[-1] = 0.0
    elif decay == "strong":
        ld = -40.0 * torch.rand(HV, generator=g)
    else:
        ld = torch.full((HV,), decay)
    return q, k, v, ld.float(), g


def run_fwd(q, k, v, ld, scale, init, **kw):
    d = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    vd = v.to(DEV) if v.is_contiguous() else _on_device(v)
    o, fin, st = cc.cconv_linattn_fwd(d(q), d(k), vd, d(ld), scale=scale, init_state=d(init), want_final_state=True, **kw)
    torch.cuda.synchronize()
    return o, fin, st


def _on_device(v):
    """The same strided view on the device (its base goes whole)."""
    base = v._base.to(DEV)
    return base.as_strided(v.shape, v.stride(), v.storage_offset())


SHAPES = [
    # B, T, H, HV, Dk, Dv
    (1, 1, 1, 1, 128, 128), (2, 15, 1, 2, 64, 64), (1, 16, 2, 2, 64, 128), (1, 17, 2, 4, 128, 64), (1, 63, 1, 1, 128, 128),
    (2, 64, 1, 1, 128, 128), (1, 65, 3, 3, 96, 80), (1, 127, 1, 2, 100, 60), (1, 128, 2, 2, 33, 47), (1, 129, 1, 3, 72, 136),
    (1, 200, 1, 1, 256, 256), (2, 300, 1, 2, 128, 256), (1, 700, 1, 1, 128, 128), (1, 577, 2, 2, 256, 64), (1, 5, 1, 1, 1, 1),
    (1, 70, 1, 1, 8, 200), (1, 1100, 1, 2, 64, 64),
    # several segments of every width and kind of load
    (1, 650, 1, 1, 64, 128), (1, 651, 1, 2, 128, 64), (1, 520, 2, 2, 100, 60), (1, 521, 1, 1, 33, 47), (2, 523, 1, 3, 72, 136),
    (1, 449, 1, 1, 256, 256), (1, 450, 1, 1, 40, 256),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("init", [False, True])
def test_forward(shape, init):
    B, T, H, HV, Dk, Dv = shape
    q, k, v, ld, g = make((B, T, H, Dk), (B, T, HV, Dv), T, slice_v=bool(T % 2))
    S0 = torch.randn(B, HV, Dk, Dv, generator=g) if init else None
    scale = Dk**-0.5
    o, fin, st = run_fwd(q, k, v, ld, scale, S0)
    assert st is None
    ref, S = layer.linattn(f64(q), f64(k), f64(v), f64(ld), scale, f64(S0))
    so, sS = layer.linattn_size(f64(q), f64(k), f64(v), f64(ld), scale, f64(S0))
    close(o, ref, so, "o")
    close_state(fin, S, sS, "final state")


@pytest.mark.parametrize("decay", ["strong", 0.0, float("-inf"), -1e-4])
def test_forward_decays(decay):
    q, k, v, ld, g = make((1, 330, 2, 128), (1, 330, 2, 128), 3, decay)
    S0 = torch.randn(1, 2, 128, 128, generator=g)
    o, fin, _ = run_fwd(q, k, v, ld, 0.5, S0)
    ref, S = layer.linattn(f64(q), f64(k), f64(v), f64(ld), 0.5, f64(S0))
    so, sS = layer.linattn_size(f64(q), f64(k), f64(v), f64(ld), 0.5, f64(S0))
    close(o, ref, so, "o")
    close_state(fin, S, sS, "final state")


def test_zero_rows_and_empty_batches():
    q, k, v, ld, g = make((2, 0, 1, 64), (2, 0, 1, 64), 1)
    S0 = torch.randn(2, 1, 64, 64, generator=g)
    o, fin, _ = run_fwd(q, k, v, ld, 1.0, S0)
    assert o.shape == (2, 0, 1, 64) and torch.equal(fin.cpu(), S0)
    _, fin, _ = run_fwd(q, k, v, ld, 1.0, None)
    assert not fin.any()
    *_, dS, _ = cc.cconv_linattn_bwd(q.to(DEV), k.to(DEV), v.to(DEV), ld.to(DEV), v.to(DEV), d_final_state=S0.to(DEV),
                                     want_d_init_state=True)
    assert torch.equal(dS.cpu(), S0)
    q, k, v, ld, g = make((0, 5, 1, 64), (0, 5, 1, 64), 1)
    o, fin, _ = run_fwd(q, k, v, ld, 1.0, None)
    assert o.shape == (0, 5, 1, 64) and fin.shape == (0, 1, 64, 64)


PACKED = [[0, 1], [0, 0, 64, 64, 65, 300, 300], [0, 700, 701, 1400], [0, 256, 512, 600], [0, 0, 0], [0, 130, 387, 387, 640, 2000]]


@pytest.mark.parametrize("cu", PACKED, ids=str)
@pytest.mark.parametrize("dims", [(2, 4, 128, 128), (1, 1, 96, 72)], ids=str)
def test_packed(cu, dims):
    H, HV, Dk, Dv = dims
    T, n = cu[-1], len(cu) - 1
    q, k, v, ld, g = make((T, H, Dk), (T, HV, Dv), T + n)
    S0 = torch.randn(n, HV, Dk, Dv, generator=g)
    do, F = torch.randn(T, HV, Dv, generator=g).to(torch.bfloat16), torch.randn(n, HV, Dk, Dv, generator=g)
    c = torch.tensor(cu, dtype=torch.int32, device=DEV)
    o, fin, st = run_fwd(q, k, v, ld, 0.1, S0, cu_seqlens=c)
    dq, dk, dv, dS, st2 = cc.cconv_linattn_bwd(q.to(DEV), k.to(DEV), v.to(DEV), ld.to(DEV), do.to(DEV), scale=0.1,
                                               init_state=S0.to(DEV), d_final_state=F.to(DEV), want_d_init_state=True,
                                               cu_seqlens=c)
    assert int(st) == 0 and int(st2) == 0
    for i in range(n):
        s = slice(cu[i], cu[i + 1])
        a = tuple(f64(x[s])[None] for x in (q, k, v))
        ini, dd, FF = f64(S0[i])[None], f64(do[s])[None], f64(F[i])[None]
        ref, S = layer.linattn(*a, f64(ld), 0.1, ini)
        so, sS = layer.linattn_size(*a, f64(ld), 0.1, ini)
        close(o[s][None], ref, so, f"o of {i}")
        close_state(fin[i][None], S, sS, f"state of {i}")
        r = layer.linattn_bwd(*a, f64(ld), 0.1, dd, ini, FF)
        z = layer.linattn_bwd_size(*a, f64(ld), 0.1, dd, ini, FF)
        for name, have, want, size in zip(("dq", "dk", "dv"), (dq, dk, dv), r, z):
            close(have[s][None], want, size, f"{name} of {i}")
        close_state(dS[i][None], r[3], z[3], f"d_init of {i}")


@pytest.mark.parametrize("cu", [[1, 10], [0, 7, 5, 10], [0, 9], [0, 11], [0, -3, 10]], ids=str)
def test_bad_offsets_write_nothing(cu):
    q, k, v, ld, _ = make((10, 1, 64), (10, 1, 64), 5)
    c = torch.tensor(cu, dtype=torch.int32, device=DEV)
    o = torch.full(v.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    fin = torch.full((len(cu) - 1, 1, 64, 64), 7.0, device=DEV)
    a = [x.to(DEV) for x in (q, k, v, ld)]
    _, _, st = cc.cconv_linattn_fwd(*a, o=o, final_state=fin, cu_seqlens=c)
    dq, dk, dv = (torch.full_like(o, 7.0) for _ in range(3))
    *_, st2 = cc.cconv_linattn_bwd(*a, a[2], dq=dq, dk=dk, dv=dv, d_init_state=fin, cu_seqlens=c)
    assert int(st) == 8 and int(st2) == 8
    for x in (o, fin, dq, dk, dv):
        assert bool((x == 7.0).all())


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("states", [False, True])
def test_backward(shape, states):
    B, T, H, HV, Dk, Dv = shape
    q, k, v, ld, g = make((B, T, H, Dk), (B, T, HV, Dv), T + 1, slice_v=bool(T % 2))
    do = torch.randn(v.shape, generator=g).to(torch.bfloat16)
    S0, F = (torch.randn(B, HV, Dk, Dv, generator=g) if states else None for _ in range(2))
    scale = Dk**-0.5
    d = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    vd = v.to(DEV) if v.is_contiguous() else _on_device(v)
    dq, dk, dv, dS, _ = cc.cconv_linattn_bwd(d(q), d(k), vd, d(ld), d(do), scale=scale, init_state=d(S0),
                                             d_final_state=d(F), want_d_init_state=True)
    a = (f64(q), f64(k), f64(v), f64(ld), scale, f64(do), f64(S0), f64(F))
    r, z = layer.linattn_bwd(*a), layer.linattn_bwd_size(*a)
    for name, have, want, size in zip(("dq", "dk", "dv"), (dq, dk, dv), r, z):
        close(have, want, size, name)
    close_state(dS, r[3], z[3], "d_init")
    again = cc.cconv_linattn_bwd(d(q), d(k), vd, d(ld), d(do), scale=scale, init_state=d(S0), d_final_state=d(F),
                                 want_d_init_state=True)
    for x, y in zip((dq, dk, dv, dS), again):
        assert torch.equal(bits(x), bits(y)), "a second call differs"


def test_broadcast_and_head_major_inputs():
    """Strides other than the usual: heads before rows, one query row for all, a batch of stride 0."""
    g = torch.Generator().manual_seed(2)
    q = torch.randn(2, 3, 90, 64, generator=g).to(torch.bfloat16).to(DEV).transpose(1, 2)
    k = torch.randn(1, 90, 3, 64, generator=g).to(torch.bfloat16).to(DEV).expand(2, 90, 3, 64)
    v = torch.randn(2, 1, 3, 64, generator=g).to(torch.bfloat16).to(DEV).expand(2, 90, 3, 64)
    ld = torch.tensor([-0.3, -0.01, 0.0], device=DEV)
    o = torch.empty(2, 3, 90, 64, dtype=torch.bfloat16, device=DEV).transpose(1, 2)
    cc.cconv_linattn_fwd(q, k, v, ld, o=o)
    a = (f64(q), f64(k), f64(v), f64(ld), 1.0)
    close(o, layer.linattn(*a)[0], layer.linattn_size(*a)[0], "o")


def test_later_rows_do_not_reach_earlier_ones():
    """Infinities and NaN in rows after t leave the outputs up to t as they were, bit for bit; so with
    gradients and the rows before t."""
    q, k, v, ld, g = make((1, 150, 1, 128), (1, 150, 1, 128), 9)
    a = [x.to(DEV) for x in (q, k, v, ld)]
    do = torch.randn(v.shape, generator=g).to(torch.bfloat16).to(DEV)
    o, _, _ = cc.cconv_linattn_fwd(*a)
    dq, dk, dv, _, _ = cc.cconv_linattn_bwd(*a, do)
    for t in (70, 100, 127, 128, 149):
        for bad in (float("nan"), float("inf"), float("-inf")):
            b = [x.clone() for x in a[:3]]
            b[1][:, t:, :, 5] = bad
            b[2][:, t:, :, 7] = bad
            b[0][:, t:, :, 0] = bad
            p, _, _ = cc.cconv_linattn_fwd(*b, a[3])
            # a chunk with such rows is summed in another order: equal to 2^-16 of its terms and a rounding
            near = lambda x, y: np.all(np.abs(f64(x) - f64(y)) <= 2 * U * np.abs(f64(y)) + 2.0**-6)  # noqa: E731
            assert torch.isfinite(p[:, :t]).all() and near(p[:, :t], o[:, :t]), t
            eq, _, _, _, _ = cc.cconv_linattn_bwd(*b, a[3], do)
            assert torch.isfinite(eq[:, :t]).all(), t
    for t in (1, 30, 64, 100):
        b = [x.clone() for x in a[:3]]
        for x in b:
            x[:, :t, :, 5] = float("nan")
        _, ek, ev, _, _ = cc.cconv_linattn_bwd(*b, a[3], do)
        assert torch.isfinite(ek[:, t:]).all() and torch.isfinite(ev[:, t:]).all(), t


def test_infinite_value_reaches_its_own_channel_alone():
    q, k, v, ld, _ = make((1, 40, 1, 64), (1, 40, 1, 64), 4)
    k, q = k.abs() + 0.5, q.abs() + 0.5
    v[0, 20, 0, 7] = float("inf")
    o, fin, _ = run_fwd(q, k, v, ld, 1.0, None)
    o, fin = o.cpu(), fin.cpu()
    assert bool((o[0, 20:, 0, 7] == float("inf")).all()) and torch.isfinite(o[0, :20]).all()
    o[..., 7] = 0
    assert torch.isfinite(o).all()
    assert bool((fin[0, 0, :, 7] == float("inf")).all())


def test_writes_only_its_outputs():
    for Dk, Dv, T in ((128, 128, 100), (33, 47, 67)):
        q, k, v, ld, _ = make((2, T, 2, Dk), (2, T, 2, Dv), 11)
        o, bo, lo, ho = guarded((2, T, 2, Dv), torch.bfloat16, DEV)
        fin, bf, lf, hf = guarded((2, 2, Dk, Dv), torch.float32, DEV)
        need = cc.cconv_linattn_fwd_workspace_bytes(2, T, 2, Dk, Dv)
        ws, bw, lw, hw = guarded(((need + 3) // 4,), torch.float32, DEV)
        a = [x.to(DEV) for x in (q, k, v, ld)]
        cc.cconv_linattn_fwd(*a, o=o, final_state=fin, workspace=ws)
        outs = [guarded(x.shape, torch.bfloat16, DEV) for x in (q, k, v)]
        cc.cconv_linattn_bwd(*a, a[2], dq=outs[0][0], dk=outs[1][0], dv=outs[2][0], d_init_state=fin)
        torch.cuda.synchronize()
        assert canaries_intact(bo, lo, ho) and canaries_intact(bf, lf, hf) and canaries_intact(bw, lw, hw)
        assert all(canaries_intact(b, lo, hi) for _, b, lo, hi in outs)


# ---- single tokens -------------------------------------------------------------------------

STEPS = [(1, 1, 1, 1, 128, 128), (3, 5, 2, 4, 128, 128), (33, 40, 1, 2, 64, 128), (17, 17, 3, 3, 33, 47), (4, 9, 1, 3, 256, 256),
         (6, 6, 2, 2, 100, 60), (300, 300, 1, 1, 16, 8), (2, 3, 1, 1, 1, 1), (40, 64, 4, 8, 72, 136)]


@pytest.mark.parametrize("shape", STEPS, ids=str)
@pytest.mark.parametrize("indexed", [False, True])
def test_step(shape, indexed):
    N, S, H, HV, Dk, Dv = shape
    q, k, v, ld, g = make((N, H, Dk), (N, HV, Dv), N, slice_v=True)
    pool = torch.randn(S, HV, Dk, Dv, generator=g)
    idx = None
    if indexed:
        idx = torch.randperm(S, generator=g)[:N].to(torch.int32)
        idx[1::4] = -1
    pd = pool.to(DEV)
    o, st = cc.cconv_linattn_update(q.to(DEV), k.to(DEV), _on_device(v), ld.to(DEV), pd,
                                    None if idx is None else idx.to(DEV), scale=0.3)
    assert int(st) == 0
    ids = None if idx is None else idx.numpy()
    ref, want = layer.linattn_step(f64(q), f64(k), f64(v), f64(ld), 0.3, f64(pool), ids)
    so, sw = layer.linattn_step(*(np.abs(f64(x)) for x in (q, k, v)), f64(ld), 0.3, np.abs(f64(pool)), ids)
    assert np.all(np.abs(f64(pd) - want) <= 8 * 2.0**-24 * sw)
    assert np.all(np.abs(f64(o) - ref) <= U * np.abs(ref) + 2.0**-16 * so + 1e-30)
    if indexed:
        untouched = sorted(set(range(S)) - set(ids.tolist()))
        assert torch.equal(pd.cpu()[untouched], pool[untouched])
        assert not o.cpu()[1::4].any()


@pytest.mark.parametrize("bad", [[0, 5], [2, 2], [-2, 1], [1, 2**31 - 1]])
def test_step_bad_slots_write_nothing(bad):
    q, k, v, ld, g = make((2, 1, 64), (2, 1, 64), 1)
    pool = torch.randn(5, 1, 64, 64, generator=g)
    pd = pool.to(DEV)
    _, st = cc.cconv_linattn_update(q.to(DEV), k.to(DEV), v.to(DEV), ld.to(DEV), pd,
                                    torch.tensor(bad, dtype=torch.int32, device=DEV))
    assert int(st) == 8 and torch.equal(pd.cpu(), pool)


def test_step_empty():
    q, k, v, ld, _ = make((0, 1, 64), (0, 1, 64), 1)
    o, st = cc.cconv_linattn_update(q.to(DEV), k.to(DEV), v.to(DEV), ld.to(DEV), torch.zeros(2, 1, 64, 64, device=DEV))
    assert o.shape == (0, 1, 64) and int(st) == 0


def test_prompt_then_tokens_equals_the_longer_prompt():
    q, k, v, ld, g = make((2, 90, 2, 128), (2, 90, 4, 128), 8)
    a = [x.to(DEV) for x in (q, k, v)]
    ld = ld.to(DEV)
    o, fin, _ = cc.cconv_linattn_fwd(*a, ld, want_final_state=True)
    head = [x[:, :80] for x in a]
    _, S, _ = cc.cconv_linattn_fwd(*head, ld, want_final_state=True)
    for t in range(80, 90):
        y, _ = cc.cconv_linattn_update(a[0][:, t], a[1][:, t], a[2][:, t], ld, S)
        args = (f64(q)[:, :t + 1], f64(k)[:, :t + 1], f64(v)[:, :t + 1], f64(ld), 1.0)
        close(y[:, None], layer.linattn(*args)[0][:, -1:], layer.linattn_size(*args)[0][:, -1:], f"token {t}")
    args = (f64(q), f64(k), f64(v), f64(ld), 1.0)
    close_state(S, layer.linattn(*args)[1], layer.linattn_size(*args)[1], "state")
    close_state(fin, layer.linattn(*args)[1], layer.linattn_size(*args)[1], "state")


# ---- offsets past 32 bits ------------------------------------------------------------------


def test_rows_past_32_bit_offsets():
    """2.2e9 elements a tensor: the last rows of a long sequence with fast decays equal those of its tail alone
    (rows 1024 back weigh e^-512), forwards and backwards."""
    T, H, tail, keep = 270000, 64, 1600, 400
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    x = torch.empty(1, T, H, 128, dtype=torch.bfloat16, device=DEV)
    assert x.numel() > 2**31
    for i in range(0, T, 30000):
        x[:, i:i + 30000] = torch.randn(1, 30000, H, 128, generator=g, device=DEV).to(torch.bfloat16)
    ld = torch.full((H,), -0.5, device=DEV)
    o, fin, _ = cc.cconv_linattn_fwd(x, x, x, ld, want_final_state=True)
    y = x[:, -tail:]
    p, f2, _ = cc.cconv_linattn_fwd(y, y, y, ld, want_final_state=True)
    # each side rounds its scores, its state and its result: 2 * 0.82 u of the norm at most
    a, b = o[:, -keep:].float(), p[:, -keep:].float()
    assert float((a - b).norm()) <= 2 * U * float(b.norm())
    assert float((fin - f2).norm()) <= 2.0**-16 * float(f2.norm())
    del o
    got = cc.cconv_linattn_bwd(x, x, x, ld, x, want_d_init_state=False)[:3]
    want = cc.cconv_linattn_bwd(y, y, y, ld, y)[:3]
    for a, b in zip(got, want):
        a, b = a[:, -keep:].float(), b[:, -keep:].float()
        assert float((a - b).norm()) <= 2 * U * float(b.norm())


def test_pool_past_32_bit_offsets():
    pool = torch.zeros(2200, 32, 128, 128, device=DEV)
    assert pool.numel() * 4 > 2**32
    q, k, v, ld, _ = make((2, 32, 128), (2, 32, 128), 3)
    idx = torch.tensor([2199, 7], dtype=torch.int32, device=DEV)
    o, st = cc.cconv_linattn_update(q.to(DEV), k.to(DEV), v.to(DEV), ld.to(DEV), pool, idx)
    assert int(st) == 0
    want = f64(k)[..., :, None] * f64(v)[..., None, :]
    for n, i in enumerate((2199, 7)):  # a product of two bf16 values is exact in fp32
        assert np.array_equal(f64(pool[i]), want[n])
        pool[i] = 0
    assert not pool.any()


# ---- streams and graphs --------------------------------------------------------------------


def test_graph_replays_equal_the_eager_calls():
    T, n = 600, 3
    q, k, v, ld, g = make((T, 2, 128), (T, 4, 128), 21)
    a = [x.to(DEV) for x in (q, k, v)]
    ld = ld.to(DEV)
    cu = torch.tensor([0, 10, 10, T], dtype=torch.int32, device=DEV)
    S0 = torch.randn(n, 4, 128, 128, generator=g).to(DEV)
    do = torch.randn(v.shape, generator=g).to(torch.bfloat16).to(DEV)

    def call():
        o, fin, _ = cc.cconv_linattn_fwd(*a, ld, init_state=S0, want_final_state=True, cu_seqlens=cu)
        dq, dk, dv, dS, _ = cc.cconv_linattn_bwd(*a, ld, do, init_state=S0, want_d_init_state=True, cu_seqlens=cu)
        return o, fin, dq, dk, dv, dS

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    for r in range(3):
        for x in (*a, do):
            x.copy_(torch.randn(x.shape, generator=g).to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(held, call()):
            assert torch.equal(bits(x), bits(y)), r


def test_another_stream():
    q, k, v, ld, _ = make((1, 300, 1, 128), (1, 300, 1, 128), 13)
    a = [x.to(DEV) for x in (q, k, v, ld)]
    want, _, _ = cc.cconv_linattn_fwd(*a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, _, _ = cc.cconv_linattn_fwd(*a, o=torch.empty_like(want), stream=s)
    s.synchronize()
    assert torch.equal(bits(got), bits(want))


def test_memory_of_a_call_on_another_stream_is_not_reused_under_it():
    """What a call allocates belongs to the current stream, its work to another: the allocator must not hand the
    workspace out again before that work is done. The other stream is held up by long products first; were the
    workspace free, the fills below would take its place and write into it."""
    q, k, v, ld, _ = make((1, 4096, 1, 128), (1, 4096, 1, 128), 17)
    a = [x.to(DEV) for x in (q, k, v, ld)]
    want, fin, _ = cc.cconv_linattn_fwd(*a, want_final_state=True)
    need = cc.cconv_linattn_fwd_workspace_bytes(1, 4096, 1, 128, 128)
    assert need > 0
    m = torch.randn(4096, 4096, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(20):
            m = m @ m * 1e-3
    got, gfin, _ = cc.cconv_linattn_fwd(*a, want_final_state=True, stream=s)
    junk = [torch.full((need,), 255, dtype=torch.uint8, device=DEV) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(bits(got), bits(want)) and torch.equal(bits(gfin), bits(fin)) and len(junk) == 4


def test_binding_refusals():
    q, k, v, ld, _ = make((1, 8, 2, 64), (1, 8, 4, 64), 1)
    a = [x.to(DEV) for x in (q, k, v, ld)]
    with pytest.raises(ValueError, match="bf16"):
        cc.cconv_linattn_fwd(a[0].float(), *a[1:])
    with pytest.raises(ValueError, match="shape"):
        cc.cconv_linattn_fwd(a[0], a[1][:, :7], *a[2:])
    with pytest.raises(ValueError, match="log_decay"):
        cc.cconv_linattn_fwd(*a[:3], a[3][:2])
    with pytest.raises(ValueError, match="init_state"):
        cc.cconv_linattn_fwd(*a, init_state=torch.zeros(1, 4, 64, 32, device=DEV))
    with pytest.raises(ValueError, match="GPU"):
        cc.cconv_linattn_fwd(q, *a[1:])
    with pytest.raises(cc.CconvError, match="BAD_SHAPE"):  # value heads must be a multiple of the others
        cc.cconv_linattn_fwd(a[0], a[1], a[2][:, :, :3], a[3][:3].clone())
    with pytest.raises(cc.CconvError, match="ALIASING"):
        cc.cconv_linattn_fwd(*a, o=a[2])
    with pytest.raises(cc.CconvError, match="WORKSPACE"):
        big = torch.zeros(1, 2048, 1, 64, dtype=torch.bfloat16, device=DEV)
        cc.cconv_linattn_fwd(big, big, big, a[3][:1].clone(), o=torch.empty_like(big),
                             workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="state"):
        cc.cconv_linattn_update(a[0][0], a[1][0], a[2][0], a[3], torch.zeros(8, 4, 64, 64, device=DEV, dtype=torch.bfloat16))
