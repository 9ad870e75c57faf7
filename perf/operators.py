"""Measured cases of the operators that serve a recurrent block: the root-mean-square norm
with the residual's addition (8-bit output with scales), the short causal convolution, the
selective state space scan (prompts and single tokens) and the product of a few rows with
4-bit weights.

``listed`` and ``draw`` give cases, ``prepare`` what a program holds before the call, ``run``
one call: the framework's entry points when ``own`` is true, else the same operator in plain
torch operations in 32 bits.  ``exact`` is the operator's definition in 64 bits.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "i8": torch.int8,
       "e4m3": torch.float8_e4m3fn}
_EPS = 1e-5


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # a decode batch of 64 sequences at d_model 2048: latency
        dict(name="norm_decode", op="norm", rows=64, d=2048, x="bf16", res=True, y="i8", group=0),
        # the rows of a prompt batch, 8 x 4096 at d_model 2048, for 8-bit products
        dict(name="norm_prompt", op="norm", rows=32768, d=2048, x="bf16", res=True, y="e4m3",
             group=128),
        # a prompt batch through the convolution: 4096 channels (d_model 2048, expanded twice)
        dict(name="conv_prompt", op="conv", B=8, L=4096, D=4096, W=4, x="bf16", ragged=False,
             state=False),
        # a padded batch of odd sizes that goes on from states, fp32
        dict(name="conv_ragged", op="conv", B=3, L=1021, D=1030, W=3, x="f32", ragged=True,
             state=True),
        # one token of 64 sequences
        dict(name="conv_step", op="conv", B=64, L=1, D=4096, W=4, x="bf16", ragged=False,
             state=True),
        # the same prompt batch through the scan
        dict(name="scan_prompt", op="scan", B=8, L=4096, D=4096, N=16, G=1, x="bf16", gate=True,
             ragged=False, state=False),
        # one long sequence on few channels
        dict(name="scan_long", op="scan", B=1, L=16384, D=1024, N=16, G=1, x="bf16", gate=True,
             ragged=False, state=False),
        # a padded batch of odd sizes that goes on from states, fp32, two groups
        dict(name="scan_ragged", op="scan", B=3, L=777, D=520, N=24, G=2, x="f32", gate=False,
             ragged=True, state=True),
        # one token of 64 sequences
        dict(name="scan_step", op="scan", B=64, L=1, D=4096, N=16, G=1, x="bf16", gate=True,
             ragged=False, state=True),
        # the layer's projection (d_model 2048 to 8 heads of 2 x 256 + 2 x 512) for one token
        dict(name="w4_token", op="w4", M=1, K=2048, N=12288, group=128, x="bf16", zeros=False),
        # the output projection for a few fp32 rows, small groups with zero points
        dict(name="w4_fp32", op="w4", M=5, K=4096, N=2048, group=32, x="f32", zeros=True),
        # a large feed-forward product for a decode batch whose rows are 8-bit (the norm's output)
        dict(name="w4_batch", op="w4", M=16, K=8192, N=28672, group=128, x="i8", zeros=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "conv", "scan", "w4"])
    x = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        y = rng.choice(["f32", "bf16", "i8", "e4m3"])
        group = rng.choice([0, 32, 64, 128]) if y in ("i8", "e4m3") else 0
        d = _log(rng, 64, 8192)
        if group:
            d = max(group, d // group * group)
        rows = _log(rng, 1, min(32768, max(1, 67108864 // d)))
        return dict(op=op, rows=rows, d=d, x=x, res=rng.random() < 0.7, y=y, group=group)
    if op == "conv":
        step = rng.random() < 0.25
        D = _log(rng, 64, 8192)
        B = _log(rng, 1, 256) if step else _log(rng, 1, 16)
        L = 1 if step else _log(rng, 2, min(16384, max(2, 100000000 // (B * D))))
        return dict(op=op, B=B, L=L, D=D, W=rng.choice([2, 3, 4]), x=x,
                    ragged=not step and rng.random() < 0.5, state=step or rng.random() < 0.5)
    if op == "scan":
        step = rng.random() < 0.25
        N = rng.choice([8, 16, 16, 16, 24, 32, 64])
        G = rng.choice([1, 1, 1, 2, 4])
        D = max(1, _log(rng, 64, 8192) // G) * G
        B = _log(rng, 1, 256) if step else _log(rng, 1, 8)
        L = 1 if step else _log(rng, 2, min(32768, max(2, 1000000000 // (B * D * N))))
        return dict(op=op, B=B, L=L, D=D, N=N, G=G, x=x, gate=rng.random() < 0.6,
                    ragged=not step and rng.random() < 0.5, state=step or rng.random() < 0.5)
    group = rng.choice([32, 64, 128])
    K = max(group, _log(rng, 256, 16384) // group * group)
    N = _log(rng, 128, min(32768, 117440512 // K))
    return dict(op=op, M=_log(rng, 1, 64), K=K, N=N, group=group,
                x=rng.choice(["bf16", "bf16", "f32", "i8", "e4m3"]), zeros=rng.random() < 0.4)


# ----------------------------------------------------------------------------- inputs
def _randn(shape, gen, scale=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def _lengths(B, L, ragged, gen):
    """Valid rows of every sequence of a padded batch, or None for a full one."""
    if not ragged:
        return None
    n = torch.randint(0, L + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    n[-1] = L
    return n


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op, dt = case["op"], _DT[case["x"]]
    st = dict(case=dict(case))
    if op == "norm":
        M, d = case["rows"], case["d"]
        st["x"] = _randn((M, d), gen, 1.0, dt)
        st["w"] = 1.0 + _randn((d,), gen, 0.2)
        # the residual stream of a deep model: larger than what a block adds
        st["r"] = _randn((M, d), gen, 3.0, dt) if case["res"] else None
        st["r_out"] = torch.zeros(M, d, device="cuda", dtype=dt) if case["res"] else None
        st["y"] = torch.zeros(M, d, device="cuda", dtype=_DT[case["y"]])
        st["scales"] = None
        if case["y"] in ("i8", "e4m3"):
            st["scales"] = torch.zeros(M, d // (case["group"] or d), device="cuda")
    elif op == "conv":
        B, L, D, W = case["B"], case["L"], case["D"], case["W"]
        # the channels are the first half of the rows of the input projection
        st["x"] = _randn((B, L, 2 * D), gen, 1.0, dt)[..., :D]
        st["w"] = _randn((D, W), gen, W ** -0.5)
        st["bias"] = _randn((D,), gen, 0.1)
        st["lengths"] = _lengths(B, L, case["ragged"], gen)
        st["state"] = _randn((B, W - 1, D), gen, 1.0, dt) if case["state"] else None
        # a single token's state is updated in place, a prompt's goes to a buffer of its own
        st["state_out"] = st["state"] if L == 1 and case["state"] else \
            torch.zeros(B, W - 1, D, device="cuda", dtype=dt)
        st["y"] = torch.zeros(B, L, D, device="cuda", dtype=dt)
    elif op == "scan":
        B, L, D, N, G = (case[k] for k in ("B", "L", "D", "N", "G"))
        st["u"] = _randn((B, L, D), gen, 1.0, dt)
        # step sizes log-uniform over 0.001 .. 0.1 by channel, moved by the token
        step = torch.exp(torch.rand(D, generator=gen, device="cuda") * math.log(100.0)
                         + math.log(0.001))
        st["dt_bias"] = step + torch.log(-torch.expm1(-step))
        st["delta"] = _randn((B, L, D), gen, 0.5, dt)
        st["A"] = -(torch.arange(1, N + 1, device="cuda", dtype=torch.float32)
                    * torch.exp(_randn((D, N), gen, 0.1)))
        # B and C are columns of the rows of one projection, beside the step's low-rank part
        rank = 8 * ((D + 127) // 128)
        proj = _randn((B, L, rank + 2 * G * N), gen, 1.0, dt)
        st["B"] = proj[..., rank:rank + G * N].unflatten(-1, (G, N))
        st["C"] = proj[..., rank + G * N:].unflatten(-1, (G, N))
        st["skip"] = 1.0 + _randn((D,), gen, 0.1)
        # the gate is the second half of the rows of the input projection
        st["z"] = _randn((B, L, 2 * D), gen, 1.0, dt)[..., D:] if case["gate"] else None
        st["lengths"] = _lengths(B, L, case["ragged"], gen)
        st["state"] = _randn((B, D, N), gen, 0.3) if case["state"] else None
        st["state_out"] = st["state"] if L == 1 and case["state"] else \
            torch.zeros(B, D, N, device="cuda")
        st["y"] = torch.zeros(B, L, D, device="cuda", dtype=dt)
    else:
        M, K, N, g = (case[k] for k in ("M", "K", "N", "group"))
        st["wq"] = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda",
                                 dtype=torch.uint8)
        st["s"] = ((torch.rand((N, K // g), generator=gen, device="cuda") + 0.5)
                   * (0.25 * K ** -0.5)).to(torch.bfloat16)
        st["z"] = torch.randint(6, 11, (N, K // g), generator=gen, device="cuda",
                                dtype=torch.uint8) if case["zeros"] else None
        x = _randn((M, K), gen)
        st["xs"] = None
        if case["x"] in ("i8", "e4m3"):
            top = 127.0 if case["x"] == "i8" else 448.0
            st["xs"] = x.abs().amax(-1, keepdim=True) / top
            x = x / st["xs"]
            x = torch.round(x) if case["x"] == "i8" else x
        st["x"] = x.to(dt)
        st["y"] = torch.zeros(M, N, device="cuda",
                              dtype=torch.float32 if case["x"] == "f32" else torch.bfloat16)
    return st


# ----------------------------------------------------------------------------- one pass
def run(st):
    return _RUN[st["case"]["op"]](st)


def _values(codes, scales):
    """What 8-bit rows with scales stand for, as a bf16 operand of the next product."""
    M, d = codes.shape
    v = codes.float().view(M, scales.shape[1], -1) * scales[:, :, None]
    return v.view(M, d).to(torch.bfloat16)


def _run_norm(st):
    c = st["case"]
    if own:
        from retentive_network_scale_b200 import retention as R
        R.ret_rms_norm(st["x"], st["y"], weight=st["w"], residual=st["r"],
                       residual_out=st["r_out"], scales=st["scales"], eps=_EPS)
        y, scales = st["y"], st["scales"]
    else:
        s = st["x"].float()
        if c["res"]:
            s = s + st["r"].float()
            st["r_out"].copy_(s)
        y = s * torch.rsqrt((s * s).mean(-1, keepdim=True) + _EPS) * st["w"]
        scales = None
        if c["y"] in ("i8", "e4m3"):
            M, d = y.shape
            y = y.view(M, st["scales"].shape[1], -1)
            scales = y.abs().amax(-1) / (127.0 if c["y"] == "i8" else 448.0)
            y = (y / torch.where(scales > 0, scales, 1.0)[:, :, None]).view(M, d)
            y = torch.round(y) if c["y"] == "i8" else y
        y = y.to(_DT[c["y"]])
    out = {"y": y if scales is None else _values(y, scales), "scales": scales}
    if c["res"]:
        out["residual"] = st["r_out"]
    return out


def _swish(v):
    return v / (1.0 + torch.exp(-v))


def _valid(st, L):
    """[B, L, 1]: the rows that belong to their sequence."""
    n = st["lengths"]
    return torch.arange(L, device="cuda")[None, :, None] < n[:, None, None]


def _run_conv(st):
    c = st["case"]
    if own:
        from retentive_network_scale_b200 import retention as R
        R.ret_causal_conv(st["x"], st["w"], st["y"], bias=st["bias"], swish=True,
                          lengths=st["lengths"], state_in=st["state"],
                          state_out=st["state_out"])
        return {"y": st["y"], "state": st["state_out"]}
    B, L, D, W = c["B"], c["L"], c["D"], c["W"]
    before = st["state"] if st["state"] is not None else \
        torch.zeros(B, W - 1, D, device="cuda", dtype=st["x"].dtype)
    rows = torch.cat([before, st["x"]], 1)
    y = _swish(st["bias"] + torch.stack([rows[:, k:k + L].float() * st["w"][:, k]
                                         for k in range(W)]).sum(0))
    if st["lengths"] is None:
        last = rows[:, L:]
    else:
        y = torch.where(_valid(st, L), y, 0.0)
        at = st["lengths"].long()[:, None] + torch.arange(W - 1, device="cuda")
        last = torch.gather(rows, 1, at[:, :, None].expand(B, W - 1, D))
    st["state_out"].copy_(last)
    return {"y": y.to(st["x"].dtype), "state": st["state_out"]}


def _run_scan(st):
    c = st["case"]
    if own:
        from retentive_network_scale_b200 import retention as R
        R.ret_selective_scan(st["u"], st["delta"], st["A"], st["B"], st["C"], st["y"],
                             skip=st["skip"], Z=st["z"], delta_bias=st["dt_bias"], softplus=True,
                             lengths=st["lengths"], state_in=st["state"],
                             state_out=st["state_out"])
        return {"y": st["y"], "state": st["state_out"]}
    L, D, G = c["L"], c["D"], c["G"]
    u = st["u"].float()
    d = st["delta"].float() + st["dt_bias"]
    d = torch.clamp(d, min=0.0) + torch.log1p(torch.exp(-d.abs()))
    if st["lengths"] is not None:
        d = torch.where(_valid(st, L), d, 0.0)
    a = torch.exp(d[..., None] * st["A"])
    Bm = st["B"].float().repeat_interleave(D // G, 2)
    h = (d * u)[..., None] * Bm
    del Bm
    if st["state"] is not None:
        h[:, 0] += a[:, 0] * st["state"]
    # inclusive scan of h_t = a_t h_{t-1} + b_t by doubling
    n = 1
    while n < L:
        h[:, n:] += a[:, n:] * h[:, :-n]
        if 2 * n < L:
            a[:, n:] *= a[:, :-n].clone()
        n *= 2
    del a
    y = (h * st["C"].float().repeat_interleave(D // G, 2)).sum(-1) + st["skip"] * u
    if st["z"] is not None:
        y = y * _swish(st["z"].float())
    if st["lengths"] is not None:
        y = torch.where(_valid(st, L), y, 0.0)
    st["state_out"].copy_(h[:, -1])
    return {"y": y.to(st["u"].dtype), "state": st["state_out"]}


def _run_w4(st):
    c = st["case"]
    if own:
        from retentive_network_scale_b200 import retention as R
        R.ret_matvec_w4(st["x"], st["wq"], st["s"], st["y"], zeros=st["z"], x_scales=st["xs"])
        return st["y"]
    N, K, g = c["N"], c["K"], c["group"]
    q = torch.stack([st["wq"] & 15, st["wq"] >> 4], -1).view(N, K // g, g).float()
    z = st["z"].float()[:, :, None] if st["z"] is not None else 8.0
    w = ((q - z) * st["s"].float()[:, :, None]).view(N, K)
    y = st["x"].float() @ w.t()
    if st["xs"] is not None:
        y = y * st["xs"]
    return y.to(st["y"].dtype)


_RUN = dict(norm=_run_norm, conv=_run_conv, scan=_run_scan, w4=_run_w4)


# ----------------------------------------------------------------------------- work
_SIZE = {"f32": 4, "bf16": 2, "i8": 1, "e4m3": 1}


def work(case):
    op, xs = case["op"], _SIZE[case["x"]]
    if op == "norm":
        n, ys = case["rows"] * case["d"], _SIZE[case["y"]]
        groups = case["rows"] * (case["d"] // (case["group"] or case["d"])) if ys == 1 else 0
        return dict(bytes=n * (xs * (3 if case["res"] else 1) + ys) + 4 * (groups + case["d"]),
                    flops=6 * n)
    if op == "conv":
        n, W = case["B"] * case["L"] * case["D"], case["W"]
        held = case["B"] * case["D"] * (W - 1) * xs * (2 if case["state"] else 1)
        return dict(bytes=2 * n * xs + held + 4 * case["D"] * (W + 1), flops=(2 * W + 4) * n)
    if op == "scan":
        B, L, D, N, G = (case[k] for k in ("B", "L", "D", "N", "G"))
        n = B * L * D
        held = 4 * B * D * N * (2 if case["state"] else 1)
        return dict(bytes=n * xs * (4 if case["gate"] else 3) + 2 * B * L * G * N * xs + held
                    + 4 * D * (N + 2), flops=n * (7 * N + 10))
    M, K, N, g = (case[k] for k in ("M", "K", "N", "group"))
    return dict(bytes=N * K // 2 + N * (K // g) * (3 if case["zeros"] else 2) + M * K * xs
                + M * N * (4 if case["x"] == "f32" else 2), flops=2 * M * N * K)


# ----------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        s = st["x"].double()
        if case["res"]:
            s = s + st["r"].double()
        y = s / torch.sqrt((s ** 2).mean(-1, keepdim=True) + _EPS) * st["w"].double()
        out = {"y": y, "scales": None}
        if case["y"] in ("i8", "e4m3"):
            t = y.unflatten(-1, (-1, case["group"] or case["d"]))
            scale = t.abs().amax(-1) / (127.0 if case["y"] == "i8" else 448.0)
            t = t / scale[..., None]
            t = torch.round(t) if case["y"] == "i8" else t.to(torch.float8_e4m3fn).double()
            out = {"y": (t * scale[..., None]).flatten(-2), "scales": scale}
        if case["res"]:
            out["residual"] = s
        return out
    if op == "conv":
        B, L, D, W = (case[k] for k in ("B", "L", "D", "W"))
        x, w = st["x"].double(), st["w"].double()
        held = st["state"].double() if case["state"] else \
            torch.zeros(B, W - 1, D, device="cuda", dtype=torch.float64)
        y = torch.zeros(B, L, D, device="cuda", dtype=torch.float64)
        state = torch.empty_like(held)
        for b in range(B):
            n = L if st["lengths"] is None else int(st["lengths"][b])
            rows = torch.cat([held[b], x[b, :n]])
            state[b] = rows[n:]
            acc = st["bias"].double().expand(n, D).clone()
            for k in range(W):
                acc += w[:, k] * rows[k:k + n]
            y[b, :n] = acc * torch.sigmoid(acc)
        return {"y": y, "state": state}
    if op == "scan":
        B, L, D, N, G = (case[k] for k in ("B", "L", "D", "N", "G"))
        A, skip = st["A"].double(), st["skip"].double()
        h = st["state"].double().clone() if case["state"] else \
            torch.zeros(B, D, N, device="cuda", dtype=torch.float64)
        y = torch.zeros(B, L, D, device="cuda", dtype=torch.float64)
        for t in range(L):
            u = st["u"][:, t].double()
            d = torch.logaddexp(st["delta"][:, t].double() + st["dt_bias"].double(),
                                torch.zeros((), device="cuda", dtype=torch.float64))
            Bt = st["B"][:, t].double().repeat_interleave(D // G, 1)
            Ct = st["C"][:, t].double().repeat_interleave(D // G, 1)
            new = torch.exp(d[:, :, None] * A) * h + (d * u)[:, :, None] * Bt
            o = torch.einsum("bdn,bdn->bd", new, Ct) + skip * u
            if case["gate"]:
                z = st["z"][:, t].double()
                o = o * z * torch.sigmoid(z)
            if st["lengths"] is None:
                h, y[:, t] = new, o
            else:
                live = t < st["lengths"]
                h = torch.where(live[:, None, None], new, h)
                y[:, t] = torch.where(live[:, None], o, 0.0)
        return {"y": y, "state": h}
    M, K, N, g = (case[k] for k in ("M", "K", "N", "group"))
    x = st["x"].double()
    if st["xs"] is not None:
        x = x * st["xs"].double()
    y = torch.empty(M, N, device="cuda", dtype=torch.float64)
    for n in range(0, N, 2048):
        rows = slice(n, min(n + 2048, N))
        w = torch.empty(rows.stop - n, K, device="cuda", dtype=torch.float64)
        w[:, 0::2] = (st["wq"][rows] % 16).double()
        w[:, 1::2] = (st["wq"][rows] // 16).double()
        zero = st["z"][rows].double() if case["zeros"] else torch.full_like(
            st["s"][rows], 8.0, dtype=torch.float64)
        w -= zero.repeat_interleave(g, 1)
        w *= st["s"][rows].double().repeat_interleave(g, 1)
        y[:, rows] = x @ w.t()
    return y
