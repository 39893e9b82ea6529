"""Cases, plain forms and exact values of the layer's operators around the short convolution:
linear attention with a decay for each head (training, prompts, packed prompts, single tokens)
and the per-head norm of queries and keys with the position rotation in the same pass.

``run`` computes the plain form in 32-bit torch operations, or, with ``own`` set, calls the
library. ``exact`` computes the same outputs in 64 bits by other means: linear attention token by
token from its recurrence, the rotation as a product of complex numbers.

Linear attention, for each value head with decay a = exp(log_decay), query/key head h = hv // (HV/H):

    S_t = a S_{t-1} + k_t^T v_t        o_t = scale * q_t S_t

Norm and rotation, for each head: y = x / sqrt(mean(x^2) + eps) * weight, then its first R
channels are rotated in pairs by the angle of the row's position.
"""

import math
import random

import torch

own = False

EPS = 1e-6
CHUNK = 64


def listed():
    return [
        # one sequence being generated: one token through one layer, where the call's latency counts
        dict(name="linattn_token_1", op="linattn", form="token", N=1, S=8, H=16, HV=16, Dk=128, Dv=128),
        # a full serving batch, value heads grouped over query/key heads, some rows padding
        dict(name="linattn_token_192", op="linattn", form="token", N=192, S=208, H=16, HV=32, Dk=128, Dv=128),
        # a short chat prompt of one user, small heads
        dict(name="linattn_prompt_77", op="linattn", form="prompt", B=1, T=77, H=8, HV=8, Dk=64, Dv=64),
        # one long document: few heads, so the time axis is the only parallelism
        dict(name="linattn_prompt_32768", op="linattn", form="prompt", B=1, T=32768, H=16, HV=16, Dk=128, Dv=128),
        # a serving engine's prefill: prompts of very different lengths packed along time, each
        # continuing from a state (a cached prefix) and leaving one for decoding
        dict(name="linattn_packed_12288", op="linattn", form="packed", nseq=24, T=12288, H=8, HV=16, Dk=128, Dv=128),
        # a training step of one layer: forward and backward at a pretraining length
        dict(name="linattn_train_4x8192", op="linattn", form="train", B=4, T=8192, H=32, HV=32, Dk=128, Dv=128),
        # a small training step with grouped heads, head widths off the tile sizes, an odd length
        # and a state carried in and out (truncated backpropagation through time)
        dict(name="linattn_train_odd", op="linattn", form="train", B=3, T=1021, H=5, HV=10, Dk=96, Dv=72),
        # the norm and rotation of one decoding step of a small batch at far positions
        dict(name="qknorm_token_16", op="qknorm", form="forward", B=16, T=1, Hq=16, Hk=16, D=128, R=128, P=131072,
             interleaved=False),
        # a long prompt, few key heads
        dict(name="qknorm_prompt_16384", op="qknorm", form="forward", B=1, T=16384, Hq=32, Hk=8, D=128, R=128,
             P=32768, interleaved=False),
        # a training step: forward and backward with the gradients of both weights
        dict(name="qknorm_train_4x8192", op="qknorm", form="train", B=4, T=8192, Hq=32, Hk=32, D=128, R=128, P=8192,
             interleaved=False),
        # a small training step with neighbouring pairs, half of each head rotated, an odd length
        dict(name="qknorm_train_odd", op="qknorm", form="train", B=2, T=1531, Hq=6, Hk=2, D=80, R=40, P=2048,
             interleaved=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.62:
        form = rng.choice(["token", "prompt", "packed", "train"])
        H = rng.choice([1, 2, 3, 4, 5, 6, 8, 12, 16])
        HV = H * rng.choice([1, 1, 1, 2, 2, 3] if H <= 8 else [1, 1, 2])
        Dk, Dv = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (128, 256), (256, 256), (96, 80), (128, 64),
                             (72, 136), (100, 60), (33, 47)])
        wide = max(1.0, Dk * Dv / 16384.0)
        if form == "token":
            N = _log_int(rng, 1, max(2, int(192 * 32 / HV / wide / 2)))
            N = min(N, 512)
            return dict(op="linattn", form=form, N=N, S=N + rng.randrange(0, 9), H=H, HV=HV, Dk=Dk, Dv=Dv)
        most = int((524288 if form == "prompt" else 262144) / HV / wide)
        if form == "packed":
            T = _log_int(rng, 200, max(400, most))
            return dict(op="linattn", form=form, nseq=rng.randrange(1, 33), T=T, H=H, HV=HV, Dk=Dk, Dv=Dv)
        B = rng.choice([1, 1, 2, 3, 4, 7])
        T = _log_int(rng, 1, max(64, min(32768, most // B)))
        return dict(op="linattn", form=form, B=B, T=T, H=H, HV=HV, Dk=Dk, Dv=Dv)
    form = rng.choice(["forward", "train"])
    D, R = rng.choice([(128, 128), (128, 64), (64, 64), (256, 128), (256, 256), (96, 96), (80, 40), (80, 20),
                       (72, 0), (66, 22)])
    Hq = rng.choice([1, 2, 4, 6, 8, 12, 16, 32])
    Hk = rng.choice([h for h in (1, 2, 4, 6, 8, 12, 16) if h <= Hq])
    B = rng.choice([1, 2, 3, 4, 8, 16])
    most = int((80e6 if form == "forward" else 60e6) / (Hq + Hk) / D / B)
    T = _log_int(rng, 1, max(8, min(16384, most)))
    return dict(op="qknorm", form=form, B=B, T=T, Hq=Hq, Hk=Hk, D=D, R=R, P=T + rng.randrange(1, 5000),
                interleaved=rng.random() < 0.5)


# ---------------------------------------------------------------------------------------------
# inputs


def _decays(HV, g):
    """log_decay of each head: geometric slopes from 1/2 down to 2^-8, one head without a decay."""
    s = -torch.exp2(-8.0 * (torch.arange(HV, dtype=torch.float64) + 1) / HV)
    if HV > 2:
        s[-1] = 0.0
    return s.to(torch.float32).to(g.device)


def _normal(g, *shape, size=1.0):
    return (torch.randn(*shape, generator=g, device=g.device) * size).to(torch.bfloat16)


def _unit(g, *shape):
    """Rows of root mean square 1, as the norm leaves them."""
    x = torch.randn(*shape, generator=g, device=g.device)
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)).to(torch.bfloat16)


def _values(g, B, T, H, HV, Dk, Dv):
    """v as the short convolution of a fused projection leaves it: a slice of rows q | k | v after SiLU."""
    x = torch.randn(B, T, 2 * H * Dk + HV * Dv, generator=g, device=g.device)
    x = (x * torch.sigmoid(x)).to(torch.bfloat16)
    return x[:, :, 2 * H * Dk:].unflatten(-1, (HV, Dv))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c, s = case, {"case": case}
    if c["op"] == "linattn":
        H, HV, Dk, Dv = c["H"], c["HV"], c["Dk"], c["Dv"]
        s["log_decay"] = _decays(HV, g)
        s["scale"] = Dk ** -0.5
        if c["form"] == "token":
            N, S = c["N"], c["S"]
            s["q"], s["k"] = _unit(g, N, H, Dk), _unit(g, N, H, Dk)
            s["v"] = _values(g, N, 1, H, HV, Dk, Dv)[:, 0]
            s["pool"] = torch.randn(S, HV, Dk, Dv, generator=g, device="cuda")
            idx = torch.randperm(S, generator=g, device="cuda")[:N].to(torch.int32)
            if N >= 16:
                idx[5::16] = -1  # padding rows of a fixed-size batch
            s["indices"] = idx
            s["rows"] = None
            return s
        B, T = c.get("B", 1), c["T"]
        s["q"], s["k"] = _unit(g, B, T, H, Dk), _unit(g, B, T, H, Dk)
        s["v"] = _values(g, B, T, H, HV, Dk, Dv)
        if c["form"] == "packed":
            r = random.Random(seed)
            cuts = sorted(r.randrange(0, T + 1) for _ in range(c["nseq"] - 1))
            s["cu"] = torch.tensor([0, *cuts, T], dtype=torch.int32, device="cuda")
            s["q"], s["k"], s["v"] = s["q"][0], s["k"][0], s["v"][0]
            s["init"] = torch.randn(c["nseq"], HV, Dk, Dv, generator=g, device="cuda")
        if c["form"] == "train":
            s["do"] = _normal(g, B, T, HV, Dv, size=0.01)
            s["init"] = torch.randn(B, HV, Dk, Dv, generator=g, device="cuda")
            s["dfinal"] = torch.randn(B, HV, Dk, Dv, generator=g, device="cuda") * 0.01
        return s
    B, T, Hq, Hk, D, R = c["B"], c["T"], c["Hq"], c["Hk"], c["D"], c["R"]
    x = torch.randn(B, T, (Hq + 2 * Hk) * D, generator=g, device="cuda")
    x = (x * torch.sigmoid(x)).to(torch.bfloat16)  # rows q | k | v after the short convolution
    s["q"] = x[:, :, :Hq * D].unflatten(-1, (Hq, D))
    s["k"] = x[:, :, Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D))
    s["wq"] = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
    s["wk"] = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
    s["table"] = None
    if R:
        inv = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)
        angle = torch.arange(c["P"], dtype=torch.float64, device="cuda")[:, None] * inv
        s["table"] = torch.cat([angle.cos(), angle.sin()], -1).to(torch.float32)
    if c["form"] == "train":
        s["positions"] = None
        s["dyq"], s["dyk"] = _normal(g, B, T, Hq, D, size=0.01), _normal(g, B, T, Hk, D, size=0.01)
    else:
        first = torch.randint(0, c["P"] - T + 1, (B, 1), generator=g, device="cuda")
        s["positions"] = (first + torch.arange(T, device="cuda")).to(torch.int32)
    return s


# ---------------------------------------------------------------------------------------------
# the plain form


def _decay(log_decay, steps):
    """exp(log_decay * steps) where steps >= 0, else 0: [HV, *steps.shape], angles and products in 64 bits."""
    e = torch.exp(log_decay.double().view(-1, *[1] * steps.dim()) * steps.clamp(min=0).double())
    return torch.where(steps >= 0, e, torch.zeros((), dtype=torch.float64, device=e.device)).float()


def _walk(q, k, v, log_decay, starts, lens, first, alpha, beta, shift, reverse):
    """out_i = alpha sum_{j <= i} a^(i-j) (q_i . k_j) v_j + beta a^(i+shift) (q_i first) over the rows of each
    sequence, in chunks, and sum_j a^(len-1-j) k_j^T v_j; q, k, v [rows, HV, .]; first [nseq, HV, ., .].
    With reverse, rows count from each sequence's end."""
    dev, n = q.device, lens.numel()
    per = (lens + CHUNK - 1) // CHUNK
    nc = q.shape[0] // CHUNK + n  # at least as many chunks as there are
    base = torch.cumsum(per, 0) - per
    c = torch.arange(nc, device=dev)
    seq = (torch.searchsorted(base + per, c, right=True)).clamp(max=n - 1)
    off = (c - base[seq]) * CHUNK  # the chunk's first row within its sequence
    r = torch.arange(CHUNK, device=dev)
    at = off[:, None] + r
    real = (at < lens[seq][:, None]) & (c < per.sum())[:, None]
    rows = starts[seq][:, None] + torch.where(torch.full_like(at, reverse, dtype=torch.bool), lens[seq][:, None] - 1 - at, at)
    total = q.shape[0]
    rows = torch.where(real, rows, torch.full_like(rows, total))  # no row: the one past the last
    pick = lambda x: torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, 1))[rows].permute(2, 0, 1, 3).contiguous()  # noqa: E731
    Q, K, V = pick(q), pick(k), pick(v)  # [HV, chunks, CHUNK, .]
    count = real.sum(-1)
    tail = _decay(log_decay, torch.where(real, count[:, None] - 1 - r, -1))  # decay to the chunk's last row
    kv = torch.matmul(K.transpose(-1, -2).contiguous(), V * tail[..., None])  # [HV, chunks, Dk, Dv]
    begin, end = off, off + count
    before = (seq[:, None] == seq) & (c[:, None] > c) & (c < per.sum())
    carry = _decay(log_decay, torch.where(before, begin[:, None] - end, -1))
    into = torch.matmul(carry, kv.flatten(2)).view_as(kv)  # each chunk's state before its first row
    P = torch.matmul(Q, K.transpose(-1, -2).contiguous()) * _decay(log_decay, r[:, None] - r)[:, None]
    mid = torch.matmul(Q, into) * _decay(log_decay, r + 1)[:, None, :, None]
    out = (torch.matmul(P, V) + mid) * alpha
    final = torch.where((seq == torch.arange(n, device=dev)[:, None]) & (c < per.sum()), lens[:, None] - end, -1)
    last = torch.matmul(_decay(log_decay, final), kv.flatten(2)).view(kv.shape[0], n, *kv.shape[2:]).transpose(0, 1)
    if first is not None:
        S = first.float()[seq].transpose(0, 1)
        out = out + torch.matmul(Q, S) * (_decay(log_decay, at + shift) * beta)[..., None]
    full = torch.empty(total + 1, q.shape[1], v.shape[2], device=dev)
    full[rows] = out.permute(1, 2, 0, 3)
    return full[:total], last


def _grouped(x, HV):
    return x.repeat_interleave(HV // x.shape[-2], dim=-2)


def _linattn_rows(s):
    """The rows of all sequences as one list, and where each starts."""
    c = s["case"]
    if c["form"] == "packed":
        cu = s["cu"].long()
        return (lambda x: x), cu[:-1], cu[1:] - cu[:-1]
    lens = torch.full((c["B"],), c["T"], device=s["q"].device)
    return (lambda x: x.flatten(0, 1)), torch.arange(c["B"], device=lens.device) * c["T"], lens


def _plain_linattn(s):
    c, g, scale = s["case"], s["log_decay"], s["scale"]
    HV = c["HV"]
    if c["form"] == "token":
        idx = s["indices"].long()
        live = (idx >= 0).nonzero()[:, 0]
        q, k, v = (_grouped(x[live], HV).float() for x in (s["q"], s["k"], s["v"]))
        S = s["pool"][idx[live]] * torch.exp(g)[:, None, None] + k[..., None] * v[..., None, :]
        s["pool"][idx[live]] = S
        o = torch.zeros(c["N"], HV, c["Dv"], device=q.device)
        o[live] = (q[..., None] * S).sum(-2) * scale
        return o.to(torch.bfloat16), s["pool"]
    flat, starts, lens = _linattn_rows(s)
    q, k, v = _grouped(flat(s["q"]), HV), _grouped(flat(s["k"]), HV), flat(s["v"])
    S0 = s.get("init")
    o, last = _walk(q, k, v, g, starts, lens, S0, scale, scale, 1, False)
    if S0 is not None:
        last = last + S0 * _decay(g, lens).T[..., None, None]
    o = o.to(torch.bfloat16).view(s["v"].shape)
    if c["form"] != "train":
        return o, last
    do, F = flat(s["do"]), s["dfinal"]
    T = lambda x: x.transpose(-1, -2)  # noqa: E731
    dq, _ = _walk(do, v, k, g, starts, lens, T(S0), scale, scale, 1, False)
    dk, _ = _walk(v, do, q, g, starts, lens, T(F), scale, 1.0, 0, True)
    dv, R = _walk(k, q, do, g, starts, lens, F, scale, 1.0, 0, True)
    dS0 = R * scale * _decay(g, torch.ones_like(lens)).T[..., None, None] + F * _decay(g, lens).T[..., None, None]
    shared = lambda x: x.unflatten(1, (c["H"], HV // c["H"])).sum(2).to(torch.bfloat16).view(s["q"].shape)  # noqa: E731
    return o, last, shared(dq), shared(dk), dv.to(torch.bfloat16).view(s["v"].shape), dS0


def _turn(x, cos, sin, R, interleaved, back=False):
    """x with its first R channels rotated (back: by the negative angle)."""
    sin = -sin if back else sin
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., R:]], -1)


def _plain_qknorm(s):
    c = s["case"]
    R = c["R"]
    if R:
        rows = s["table"][:c["T"]][None] if s["positions"] is None else s["table"][s["positions"].long()]
        cos, sin = rows[..., None, :R // 2], rows[..., None, R // 2:]
    turn = lambda x, back=False: _turn(x, cos, sin, R, c["interleaved"], back) if R else x  # noqa: E731

    def forward(x, w):
        x = x.float()
        unit = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        return turn(unit * w).to(torch.bfloat16)

    def backward(x, w, dy):
        x = x.float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        unit, u = x * r, turn(dy.float(), True)
        du = u * w
        dx = r * (du - unit * (du * unit).mean(-1, keepdim=True))
        return dx.to(torch.bfloat16), (u * unit).sum((0, 1, 2))

    y = forward(s["q"], s["wq"]), forward(s["k"], s["wk"])
    if c["form"] == "forward":
        return y
    (dq, dwq), (dk, dwk) = backward(s["q"], s["wq"], s["dyq"]), backward(s["k"], s["wk"], s["dyk"])
    return (*y, dq, dk, dwq, dwk)


# ---------------------------------------------------------------------------------------------
# the library's calls


def _own_linattn(s):
    import causal_depthwise_short_amd as cc

    c, g, scale = s["case"], s["log_decay"], s["scale"]
    if c["form"] == "token":
        o, _ = cc.cconv_linattn_update(s["q"], s["k"], s["v"], g, s["pool"], s["indices"], scale=scale)
        return o, s["pool"]
    if c["form"] == "packed":
        o, last, _ = cc.cconv_linattn_fwd(s["q"], s["k"], s["v"], g, scale=scale, init_state=s["init"],
                                          want_final_state=True, cu_seqlens=s["cu"])
        return o, last
    o, last, _ = cc.cconv_linattn_fwd(s["q"], s["k"], s["v"], g, scale=scale, init_state=s.get("init"),
                                      want_final_state=True)
    if c["form"] == "prompt":
        return o, last
    dq, dk, dv, dS0, _ = cc.cconv_linattn_bwd(s["q"], s["k"], s["v"], g, s["do"], scale=scale, init_state=s["init"],
                                              d_final_state=s["dfinal"], want_d_init_state=True)
    return o, last, dq, dk, dv, dS0


def _own_qknorm(s):
    import causal_depthwise_short_amd as cc

    kw = dict(positions=s["positions"], eps=EPS, interleaved=s["case"]["interleaved"])
    yq, yk, _ = cc.cconv_qknorm_fwd(s["q"], s["k"], s["wq"], s["wk"], s["table"], **kw)
    if s["case"]["form"] == "forward":
        return yq, yk
    dq, dk, dwq, dwk, _ = cc.cconv_qknorm_bwd(s["q"], s["k"], s["dyq"], s["dyk"], s["wq"], s["wk"], s["table"], **kw)
    return yq, yk, dq, dk, dwq, dwk


def run(state):
    if state["case"]["op"] == "linattn":
        return _own_linattn(state) if own else _plain_linattn(state)
    return _own_qknorm(state) if own else _plain_qknorm(state)


# ---------------------------------------------------------------------------------------------
# the work and the exact values


def work(case):
    c = case
    if c["op"] == "linattn":
        H, HV, Dk, Dv = c["H"], c["HV"], c["Dk"], c["Dv"]
        state = HV * Dk * Dv
        if c["form"] == "token":
            live = c["N"] - len(range(5, c["N"], 16)) * (c["N"] >= 16)
            return {"bytes": live * (8 * state + 2 * (2 * H * Dk + HV * Dv)) + 2 * c["N"] * HV * Dv + 4 * c["N"],
                    "flops": live * 5 * state}
        B, rows = c.get("B", 1), c.get("B", 1) * c["T"]
        qk, v = 2 * rows * H * Dk, 2 * rows * HV * Dv
        if c["form"] == "train":
            return {"bytes": 4 * qk + 4 * v + 16 * B * state, "flops": rows * 14 * state}
        nseq, init = c.get("nseq", B), c["form"] == "packed"
        return {"bytes": 2 * qk + 2 * v + 4 * (1 + init) * nseq * state, "flops": rows * 4 * state}
    rows, D = c["B"] * c["T"], c["D"]
    x = 2 * rows * (c["Hq"] + c["Hk"]) * D
    table = 4 * c["R"] * min(c["P"], rows)
    if c["form"] == "forward":
        return {"bytes": 2 * x + table + 8 * D + 4 * rows, "flops": 4 * x}
    return {"bytes": 4 * x + table + 16 * D, "flops": 13 * x}


def _exact_linattn(s):
    """The recurrence itself, one token after the other, all sequences and heads at once, in 64 bits."""
    c, scale = s["case"], s["scale"]
    HV, grp = c["HV"], c["HV"] // c["H"]
    a = s["log_decay"].double().exp()[:, None, None]
    if c["form"] == "token":
        pool, o = s["pool"].double(), torch.zeros(c["N"], HV, c["Dv"], dtype=torch.float64, device="cuda")
        for n, i in enumerate(s["indices"].tolist()):
            if i >= 0:
                k, q = (s[x][n].double().repeat_interleave(grp, 0) for x in "kq")
                pool[i] = pool[i] * a + torch.einsum("hd,he->hde", k, s["v"][n].double())
                o[n] = scale * torch.einsum("hd,hde->he", q, pool[i])
        return o, pool
    if c["form"] == "packed":
        cu = s["cu"].tolist()
        lens = [y - x for x, y in zip(cu, cu[1:])]
        wide = lambda x: torch.nn.utils.rnn.pad_sequence([x[i:j] for i, j in zip(cu, cu[1:])], batch_first=True)  # noqa: E731
    else:
        lens, wide = [c["T"]] * c["B"], (lambda x: x)
    q, k, v = (wide(s[x]) for x in "qkv")
    n, most = q.shape[:2]
    if most * n * HV > 3e6:
        return None
    at = torch.tensor(lens, device="cuda")
    S = torch.zeros(n, HV, c["Dk"], c["Dv"], dtype=torch.float64, device="cuda")
    S = S + s["init"].double() if "init" in s else S
    do = wide(s["do"]) if c["form"] == "train" else None
    o = torch.zeros(n, most, HV, c["Dv"], dtype=torch.float64, device="cuda")
    dq = torch.zeros(n, most, HV, c["Dk"], dtype=torch.float64, device="cuda") if do is not None else None
    row = lambda x, t: x[:, t].double().repeat_interleave(HV // x.shape[2], 1)  # noqa: E731
    for t in range(most):
        new = a * S
        new.addcmul_(row(k, t)[..., None], row(v, t)[..., None, :])
        S = new if c["form"] != "packed" else torch.where((t < at).view(-1, 1, 1, 1), new, S)
        o[:, t] = scale * torch.matmul(row(q, t)[..., None, :], S)[..., 0, :]
        if do is not None:
            dq[:, t] = scale * torch.matmul(S, row(do, t)[..., None])[..., 0]
    if c["form"] == "packed":
        return torch.cat([o[i, :m] for i, m in enumerate(lens)]), S
    if do is None:
        return o, S
    dk, dv = torch.zeros_like(dq), torch.zeros_like(o)
    G = s["dfinal"].double()
    for t in reversed(range(most)):  # G: the gradient of the state after token t
        G = G + scale * row(q, t)[..., None] * row(do, t)[..., None, :]
        dk[:, t] = torch.matmul(G, row(v, t)[..., None])[..., 0]
        dv[:, t] = torch.matmul(row(k, t)[..., None, :], G)[..., 0, :]
        G = a * G
    both = lambda x: x.unflatten(2, (c["H"], grp)).sum(3)  # noqa: E731
    return o, S, both(dq), both(dk), dv, G


def _exact_qknorm(s):
    c = s["case"]
    B, T, R = c["B"], c["T"], c["R"]
    at = torch.arange(T, device="cuda").expand(B, T) if s["positions"] is None else s["positions"].long()
    if R:
        row = s["table"].double()[at]
        z = torch.complex(row[..., :R // 2], row[..., R // 2:])[:, :, None]

    def turned(x, z):
        pairs = x[..., :R].unflatten(-1, (R // 2, 2)) if c["interleaved"] else x[..., :R].unflatten(-1, (2, R // 2)).transpose(-1, -2)
        p = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
        return torch.cat([(p if c["interleaved"] else p.transpose(-1, -2)).flatten(-2), x[..., R:]], -1)

    outs, grads, sums = [], [], []
    for x, w, dy in ((s["q"], s["wq"], s.get("dyq")), (s["k"], s["wk"], s.get("dyk"))):
        x, w = x.double(), w.double()
        size = (torch.linalg.vector_norm(x, dim=-1, keepdim=True).square() / c["D"] + EPS).sqrt()
        y = x / size * w
        outs.append(turned(y, z) if R else y)
        if dy is not None:
            u = dy.double()
            u = turned(u, z.conj()) if R else u
            sums.append((u * x / size).flatten(0, 2).sum(0))
            along = (u * w * x).sum(-1, keepdim=True) / (c["D"] * size.square())
            grads.append((u * w - along * x) / size)
    return (*outs, *grads, *sums)


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_linattn(s) if case["op"] == "linattn" else _exact_qknorm(s)
