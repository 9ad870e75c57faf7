"""Plain 64-bit forms of the operators around the mixers (root-mean-square norm,
causal convolution, selective scan, 4-bit product), with the bounds their fp32
kernels are held to.  Host tensors in, host fp64 tensors out.

A rounding to bf16 is off by at most 2^-8 of the value (half a step), to e4m3 by
2^-4 (or half the smallest step, 2^-10, of the scale), to an integer code by 1/2.
"""
import torch

BF16 = 2.0 ** -8


def rounded(y, dtype):
    """Allowance of the one rounding of an output to its type."""
    return y.abs() * (BF16 if dtype == torch.bfloat16 else 2.0 ** -24)


def within(got, ref, bound):
    """Every element within its bound (an exact value where it is 0); returns
    the largest excess ratio for the message."""
    err = (got.double().cpu() - ref).abs()
    return float((err / (bound + 1e-300)).max()) if err.numel() else 0.0


def rms_norm(x, w=None, r=None, eps=1e-5):
    s = x.double() + (r.double() if r is not None else 0.0)
    y = s / torch.sqrt((s * s).mean(-1, keepdim=True) + eps)
    return s, y * w.double() if w is not None else y


# The sum of d <= 16384 squares runs through at most 16 additions of a thread,
# 5 of a warp and 32 of a row, so its relative error is at most 54 * 2^-24, half
# of that after the root; the reciprocal root (2 units), s, w and the products
# add fewer than 8.  Below 2^-18.
NORM = 2.0 ** -18


def swish(v):
    return v * torch.sigmoid(v)


def causal_conv(x, w, bias=None, act=True, lengths=None, state=None):
    """Returns (y, state, bound of y); rows past a sequence's length are NaN."""
    B, L, D = x.shape
    W = w.shape[1]
    x, w = x.double(), w.double()
    held = state.double() if state is not None else torch.zeros(B, W - 1, D, dtype=torch.float64)
    y = torch.full((B, L, D), float("nan"), dtype=torch.float64)
    tol, out = torch.zeros_like(y), torch.empty_like(held)
    for b in range(B):
        n = L if lengths is None else min(max(int(lengths[b]), 0), L)
        rows = torch.cat([held[b], x[b, :n]])
        out[b] = rows[n:]
        v = (bias.double() if bias is not None else torch.zeros(D, dtype=torch.float64)).expand(n, D).clone()
        mag = v.abs()
        for k in range(W):
            v += w[:, k] * rows[k:k + n]
            mag += (w[:, k] * rows[k:k + n]).abs()
        y[b, :n] = swish(v) if act else v
        # W + 1 roundings of the sum, times the swish's slope (at most 1.1); the
        # fast exponential's argument is off by |v| 2^-23, and it, the sum and
        # the quotient by a few units more
        tol[b, :n] = 1.1 * (W + 2) * 2.0 ** -24 * mag + (y[b, :n].abs() * (4 + v.abs()) * 2.0 ** -22 if act else 0)
    return y, out, tol


def selective_scan(u, delta, A, Bm, Cm, skip=None, z=None, bias=None, softplus=True, lengths=None,
                   state=None, per=2.0 ** -22):
    """Returns (y, state, bound of y, bound of the state); Bm, Cm [B,L,G,N].
    Rows past a sequence's length are NaN.

    The bound follows the recurrence: with H the state's magnitude (the same
    recurrence on |b_t|), e the allowance,
        e_t = a_t (e_{t-1} + H_{t-1} (2 per + p per)) + |b_t| 16 per,
    p = |d_t A| being the exponent: the exponential is within 2 units (2 per),
    its argument, a product of rounded d, A and log2 e, within a few units
    of p, and b_t = d u B (softplus included) within 16."""
    B, L, D = u.shape
    N = A.shape[1]
    rep = D // Bm.shape[2]
    A = A.double()
    h = state.double().clone() if state is not None else torch.zeros(B, D, N, dtype=torch.float64)
    H, e = h.abs(), torch.zeros_like(h)
    y = torch.full((B, L, D), float("nan"), dtype=torch.float64)
    tol = torch.zeros_like(y)
    for t in range(L):
        live = torch.ones(B, dtype=torch.bool) if lengths is None else t < lengths.cpu().long()
        ut = u[:, t].double()
        d = delta[:, t].double() + (bias.double() if bias is not None else 0.0)
        if softplus:
            d = torch.logaddexp(d, torch.zeros((), dtype=torch.float64))
        Bt = Bm[:, t].double().repeat_interleave(rep, 1)
        Ct = Cm[:, t].double().repeat_interleave(rep, 1)
        p = d[..., None] * A
        a, b = torch.exp(p), (d * ut)[..., None] * Bt
        h2 = a * h + b
        e2 = a * (e + H * (2 * per + 8 * p.abs() * per)) + b.abs() * 16 * per
        H2 = a * H + b.abs()
        keep = live[:, None, None]
        h, e, H = torch.where(keep, h2, h), torch.where(keep, e2, e), torch.where(keep, H2, H)
        s = skip.double() * ut if skip is not None else torch.zeros_like(ut)
        o = (Ct * h).sum(-1) + s
        # the sum over N states (and the gate's few units)
        eo = (Ct.abs() * e).sum(-1) + ((Ct.abs() * H).sum(-1) + s.abs()) * (N + 4) * 2.0 ** -24
        if z is not None:
            zt = z[:, t].double()
            o, eo = o * swish(zt), (eo + o.abs() * (4 + zt.abs()) * 2.0 ** -22) * swish(zt).abs()
        y[:, t] = torch.where(live[:, None], o, y[:, t])
        tol[:, t] = torch.where(live[:, None], eo, tol[:, t])
    return y, h, tol, e + H * 2.0 ** -23


def dequantise_w4(wq, scales, zeros=None):
    """fp64 weights [N, K]."""
    wq = wq.cpu()
    N, half = wq.shape
    q = torch.stack([wq & 15, wq >> 4], -1).view(N, 2 * half).double()
    g = 2 * half // scales.shape[1]
    z = zeros.cpu().double().repeat_interleave(g, 1) if zeros is not None else 8.0
    return (q - z) * scales.cpu().double().repeat_interleave(g, 1)


def matvec_w4(x, wq, scales, zeros=None, x_scales=None):
    """Returns (y, bound): exact products, summed in fp32 in chains of at most
    8 per group, K / 1024 groups and 8 parts (for the sizes tested under 40
    additions, each within 2^-22 of the terms' magnitude)."""
    x = x.cpu().double()
    if x_scales is not None:
        x = x * x_scales.cpu().double().repeat_interleave(x.shape[1] // x_scales.shape[1], 1)
    w = dequantise_w4(wq, scales, zeros)
    return x @ w.t(), (x.abs() @ w.abs().t()) * 1e-5
