"""The layer example on the GPU: its gradients against float64 differences of the same layer on the CPU
oracle, a falling loss, and prefill plus decode against the full forward."""

from __future__ import annotations

import importlib.util
from pathlib import Path

import numpy as np
import pytest
import torch

import oracle
from oracle import layer as ref

pytestmark = pytest.mark.gpu
_spec = importlib.util.spec_from_file_location(
    "linear_attention_layer", Path(__file__).resolve().parent.parent / "examples" / "linear_attention_layer.py")
ex = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(ex)


def test_loss_falls():
    layer = ex.Layer(width=256, H=2, HV=4, Dk=64, Dv=64, positions=512)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.randn(2, 300, 256, generator=g, device="cuda")
    losses = ex.train(layer, x, torch.roll(x, 2, 1), steps=15)
    assert losses[-1] < 0.9 * losses[0], losses


def test_serving_equals_the_full_forward():
    layer = ex.Layer(width=256, H=2, HV=4, Dk=128, Dv=64, positions=512)
    made, full = ex.serve(layer, [3, 130, 1, 64], tokens=6)
    for m, f in zip(made, full):
        # five bf16 roundings a side (projection, convolution, norm, attention's operands, output), each of
        # rms at most 2^-8 / sqrt(3): 2 * sqrt(5) * 2^-8 / sqrt(3) = 0.010 of the norm if all differed
        assert float((m.float() - f.float()).norm() / f.float().norm()) < 0.0102


def _loss64(w, x, dy, layer):
    """sum(y * dy) of the layer in float64."""
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    z = f(x) @ w["w_in"]
    _, rows = oracle.fwd(torch.from_numpy(z).float(), torch.from_numpy(w["taps"]).float(), None)
    rows = np.asarray(rows, dtype=np.float64)
    a, b = layer.H * layer.Dk, 2 * layer.H * layer.Dk
    B, T = rows.shape[:2]
    q, k, v = (rows[..., s].reshape(B, T, -1, d) for s, d in ((slice(0, a), layer.Dk), (slice(a, b), layer.Dk), (slice(b, None), layer.Dv)))
    tab = f(layer.table)
    qn, kn = ref.qknorm(q, w["wq"], tab, None, 1e-6, False), ref.qknorm(k, w["wk"], tab, None, 1e-6, False)
    o, _ = ref.linattn(qn, kn, v, f(layer.log_decay), layer.scale)
    return float(((o.reshape(B, T, -1) @ w["w_out"]) * f(dy)).sum())


def test_gradients_against_differences():
    layer = ex.Layer(width=64, H=1, HV=2, Dk=16, Dv=16, positions=64)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    x = torch.randn(1, 40, 64, generator=g, device="cuda")
    y, saved = layer.forward(x)
    dy = torch.randn(y.shape, generator=g, device="cuda").to(torch.bfloat16)
    grads = layer.backward(saved, dy)
    w = {n: t.double().cpu().numpy() for n, t in layer.w.items()}
    rng = np.random.default_rng(0)
    for name in w:
        d = rng.standard_normal(w[name].shape)
        got = float((grads[name].double().cpu().numpy() * d).sum())
        step = 1e-3 * np.sqrt(np.mean(w[name] ** 2))
        up, down = dict(w), dict(w)
        up[name], down[name] = w[name] + step * d, w[name] - step * d
        want = (_loss64(up, x, dy, layer) - _loss64(down, x, dy, layer)) / (2 * step)
        # along a random direction the gradient's bf16 roundings (about ten stages of rms 2^-8 / sqrt(3)
        # each) add up like the gradient itself: a few hundredths of its norm times the direction's
        scale = float(grads[name].double().norm())
        assert abs(got - want) <= 10 * 2.0**-8 * max(abs(want), 4 * scale), name
