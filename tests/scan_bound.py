"""The selective scan in 64 bits on the GPU, with the error bound that the fp32
kernels' roundings add up to, counted one by one (block_ref's bound is several times
wider, since it takes one unit for all).  u = 2^-24 is half a unit in the last place.

    x = delta + bias            u |x|
    softplus(x)                 e^-|x|: its argument is off by 2 u |x| (log2 e, the
                                product), the exponential 4 u; the polynomial 0.5 u
                                and 2 u of its additions; the last sum u.  With
                                sigmoid <= softplus: (3 |x| + 7.5) u of d
    p = d A log2 e              3 u of p more (log2 e, two products)
    exp(p)                      4 u, and |p| times p's
    d u B                       3 products: 3 u more than d
    h = exp(p) h + d u B        u of h

Where the sequence is cut into segments the sum of a segment's d is added up in tiles
of 16 rows, and `cut` (16 and the tiles of a segment) roundings of it go into the
exponent of the segment's decay."""
import torch

U = 2.0 ** -24


def selective_scan(u, delta, A, Bm, Cm, skip=None, z=None, bias=None, softplus=True, lengths=None,
                   state=None, cut=0):
    """As block_ref.selective_scan; everything on the GPU."""
    dev = lambda t: None if t is None else t.cuda().double()  # noqa: E731
    u, delta, A, Bm, Cm, skip, z, bias, state = map(dev, (u, delta, A, Bm, Cm, skip, z, bias, state))
    B, L, D = u.shape
    N, rep = A.shape[1], D // Bm.shape[2]
    x = delta + bias if bias is not None else delta
    d = torch.logaddexp(x, torch.zeros_like(x)) if softplus else x
    rel = 3 * x.abs() + 7.5 if softplus else torch.ones_like(x)
    # a step of 0 (x = -inf) is exact; no 0 * inf
    rel = torch.where(d == 0, 0.0, rel)
    live = torch.ones(B, L, dtype=torch.bool, device="cuda")
    if lengths is not None:
        live = torch.arange(L, device="cuda")[None] < lengths.cuda()[:, None]
    h = state.clone() if state is not None else torch.zeros(B, D, N, device="cuda", dtype=torch.float64)
    H, e = h.abs(), torch.zeros_like(h)
    ys, tols = [], []
    for t in range(L):
        Bt, Ct = Bm[:, t].repeat_interleave(rep, 1), Cm[:, t].repeat_interleave(rep, 1)
        p = d[:, t, :, None] * A
        a, b = torch.exp(p), (d[:, t] * u[:, t])[..., None] * Bt
        r = rel[:, t, :, None]
        H2 = a * H + b.abs()
        e2 = a * (e + H * (4 + p.abs() * (r + 3 + cut)) * U) + b.abs() * (r + 3) * U + H2 * U
        on = live[:, t, None, None]
        h, H, e = torch.where(on, a * h + b, h), torch.where(on, H2, H), torch.where(on, e2, e)
        ys.append((Ct * h).sum(-1))
        # a chain of at most 16 products, the sum of a pair and of 8 threads
        tols.append((Ct.abs() * e).sum(-1) + (Ct.abs() * H).sum(-1) * min(N + 3, 27) * U)
    y, tol = torch.stack(ys, 1), torch.stack(tols, 1)
    if skip is not None:
        y, tol = y + skip * u, tol + (skip * u).abs() * U
    tol = tol + y.abs() * U
    if z is not None:
        gate = z * torch.sigmoid(z)
        # exponent 2 u |z|, exponential 4 u, sum u, quotient 4 u, product u
        y, tol = y * gate, tol * gate.abs() + (y * gate).abs() * (2 * z.abs() + 10) * U
    y = torch.where(live[..., None], y, float("nan"))
    return y, h, torch.where(live[..., None], tol, 0.0), e
