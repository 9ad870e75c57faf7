"""Every form of the kernels of the operators around the mixers at sizes that take
it: long runs of the convolution, several steps a thread of the norm, sequences cut
into segments for every layout of the scan's states.  References in 64 bits on the
GPU, bounds as in block_ref and scan_bound."""
import pytest
import torch

import block_ref as ref
import scan_bound
from retentive_network_scale_b200 import retention as R
from test_gpu_block_ops import rt, scan_case, strided

pytestmark = pytest.mark.gpu
F32, BF16, I8, E4M3 = torch.float32, torch.bfloat16, torch.int8, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from retentive_network_scale_b200 import build
    build.build()
    R.load_library()
    yield
    torch.cuda.synchronize()
    assert R.ret_last_device_status() == 0


def randn(shape, seed, scale=1.0, dtype=F32):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def widened(t, pad, off):
    wide = torch.full(t.shape[:-1] + (t.shape[-1] + pad,), 7.0, device="cuda").to(t.dtype)
    out = wide[..., off:off + t.shape[-1]]
    out.copy_(t)
    return out


def ratio(got, want, bound):
    """The largest error in units of its bound (0 / 0 is none)."""
    err = (got.double() - want).abs()
    return float((err / (bound + 1e-300)).max())


# ------------------------------------------------------------------------ convolution
# rows of a thread in bf16: 32, 32, 64 (one channel a thread), 128, 128 (four channels),
# 64 (unaligned)
@pytest.mark.parametrize("B,L,D,pad,off", [(8, 1021, 2048, 0, 0), (8, 1021, 1030, 2, 0), (8, 1021, 1031, 0, 0),
                                           (3, 4099, 4100, 0, 0), (8, 2400, 4096, 4096, 0), (8, 1021, 1030, 3, 1)])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_causal_conv_long_runs(B, L, D, pad, off, W, dtype):
    x, w, bias = randn((B, L, D), 1, 1.0, dtype), randn((D, W), 2, W ** -0.5), randn((D,), 3, 0.3)
    state = randn((B, W - 1, D), 4, 1.0, dtype)
    for lens in (None, ([L, L - 1, 0, 129, 128, 127, 33, 1])[:B]):
        held = state.clone() if lens else None
        n = torch.tensor(lens or [L] * B, device="cuda", dtype=torch.int32)
        live = (torch.arange(L, device="cuda")[None] < n[:, None])[..., None]
        rows = torch.cat([state if lens else torch.zeros_like(state), x], 1).double()
        v = bias.double().expand(B, L, D).clone()
        mag = v.abs()
        for k in range(W):
            v += w[:, k].double() * rows[:, k:k + L]
            mag += (w[:, k].double() * rows[:, k:k + L]).abs()
        want = v * torch.sigmoid(v)
        tol = 1.1 * (W + 2) * 2.0 ** -24 * mag + want.abs() * (4 + v.abs()) * 2.0 ** -22 + ref.rounded(want, dtype)
        del v, mag
        y, end = torch.full((B, L, D), 5.0, device="cuda", dtype=dtype), torch.empty_like(state)
        xs = torch.where(live, x, float("nan"))                 # rows that must not be read
        R.ret_causal_conv(widened(xs, pad, off), w, y, bias=bias, lengths=n if lens else None, state_in=held,
                          state_out=held if lens else end)
        assert bool((y.masked_select(~live) == 5.0).all())
        assert ratio(torch.where(live, y, 0), torch.where(live, want, 0.0), tol) <= 1
        at = n.long()[:, None] + torch.arange(W - 1, device="cuda")
        last = torch.gather(rows, 1, at[:, :, None].expand(B, W - 1, D))
        assert torch.equal((held if lens else end).double(), last)


# ------------------------------------------------------------------------ norm
@pytest.mark.parametrize("rows,d", [(1200, 264), (1187, 320), (1200, 2048), (1201, 2056), (1200, 8192), (1187, 8224)])
@pytest.mark.parametrize("pad,off", [(0, 0), (8, 8), (3, 1)])
@pytest.mark.parametrize("xt,rtype", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
def test_rms_norm_many_rows(rows, d, pad, off, xt, rtype):
    x, w, r = randn((rows, d), 5, 1.0, xt), 1 + randn((d,), 6, 0.2), randn((rows, d), 7, 3.0, rtype)
    xs = widened(x, pad, off)
    s = x.double() + r.double()
    want = s / torch.sqrt((s * s).mean(-1, keepdim=True) + 1e-5) * w.double()
    plain = s / torch.sqrt((s * s).mean(-1, keepdim=True) + 1e-5)
    for yt in (F32, BF16):
        y, held = torch.full((rows, d), 9.0, device="cuda", dtype=yt), r.clone()
        R.ret_rms_norm(xs, y, weight=w, residual=held, residual_out=held)           # in place
        assert ratio(y, want, ref.NORM * want.abs() + ref.rounded(want, yt)) <= 1
        assert ratio(held, s, 2.0 ** -24 * s.abs() + ref.rounded(s, rtype)) <= 1
    R.ret_rms_norm(xs, y, residual=r)
    assert ratio(y, plain, ref.NORM * plain.abs() + ref.rounded(plain, BF16)) <= 1
    for yt in (I8, E4M3):
        for group in [0] + [g for g in (32, 64, 128) if d % g == 0]:
            y, held = torch.full((rows, d), 1.0, device="cuda").to(yt), r.clone()
            sc = torch.full((rows, d // (group or d)), -1.0, device="cuda")
            R.ret_rms_norm(xs, y, weight=w, residual=held, residual_out=held, scales=sc)
            g, top = group or d, 127.0 if yt == I8 else 448.0
            scale = want.view(rows, d // g, g).abs().amax(-1) / top
            assert ratio(sc, scale, ref.NORM * scale) <= 1
            step = scale.repeat_interleave(g, 1)
            got = y.float().double() * sc.double().repeat_interleave(g, 1)
            half = 0.5 * step if yt == I8 else torch.maximum(want.abs() * 2.0 ** -4, step * 2.0 ** -10)
            # 4 NORM: the code is taken of a value and with a scale that are each off
            assert ratio(got, want, half + 4 * ref.NORM * (want.abs() + step)) <= 1
            assert ratio(held, s, 2.0 ** -24 * s.abs() + ref.rounded(s, rtype)) <= 1


# ------------------------------------------------------------------------ scan
def scan_and_check(c, dtype, lens, gate=True, state=True, pad=0, off=0, in_place=True, cut=0):
    B, L, D = c["u"].shape
    N = c["A"].shape[1]
    n = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    u, delta, z, bm, cm = (c[k].clone() for k in ("u", "delta", "z", "Bm", "Cm"))
    if lens is not None:
        for b in range(B):                                      # rows that must not be read
            for t in (u, delta, z, bm, cm):
                t[b, lens[b]:] = float("nan")
    y = torch.full((B, L, D), 5.0, device="cuda", dtype=dtype)
    held = c["s0"].cuda() if state else torch.full((B, D, N), 8.0, device="cuda")
    out = held if in_place or not state else torch.full_like(held, 8.0)
    flat = lambda t: strided(t.flatten(2), pad, off).unflatten(2, t.shape[2:])  # noqa: E731
    R.ret_selective_scan(strided(u, pad, off), strided(delta, pad, off), c["A"].cuda(), flat(bm), flat(cm), y,
                         skip=c["skip"].cuda(), Z=strided(z, pad, off) if gate else None,
                         delta_bias=c["bias"].cuda(), lengths=None if n is None else n.cuda(),
                         state_in=held if state else None, state_out=out)
    want, last, tol, stol = scan_bound.selective_scan(
        c["u"], c["delta"], c["A"], c["Bm"], c["Cm"], c["skip"], c["z"] if gate else None, c["bias"], True, n,
        c["s0"] if state else None, cut=cut)
    dead = torch.isnan(want)
    assert bool((y[dead] == 5.0).all())
    want = torch.where(dead, 0.0, want)
    worst = ratio(torch.where(dead, 0.0, y.double()), want, tol + ref.rounded(want, dtype)), ratio(out, last, stol)
    assert max(worst) <= 1, worst
    return worst


@pytest.mark.parametrize("D,N,G,pad,off", [(8, 5, 1, 0, 0), (34, 5, 2, 3, 1), (48, 8, 2, 8, 8), (48, 16, 2, 8, 8),
                                           (40, 16, 1, 1, 1), (48, 24, 2, 8, 8), (33, 24, 3, 1, 0), (64, 64, 1, 0, 0),
                                           (20, 64, 2, 5, 3), (32, 128, 2, 0, 0), (18, 128, 1, 8, 0), (24, 100, 1, 2, 1)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("L,cut", [(270, 16 + 5), (530, 16 + 5), (1040, 16 + 5)])
def test_scan_in_segments_of_every_layout(D, N, G, pad, off, dtype, L, cut):
    """Few channels, 4, 8 or 16 segments: among the sequences one without rows, one
    that ends in the first segment, and one that leaves the last ones empty."""
    c = scan_case(4, L, D, N, G, dtype, seed=61)
    scan_and_check(c, dtype, [L, 0, 7, L // 2 + 3], pad=pad, off=off, cut=cut)
    if L == 270:
        scan_and_check(c, dtype, None, gate=False, state=False, pad=pad, off=off, cut=cut)
        scan_and_check(c, dtype, [0, 0, 0, L - 1], in_place=False, pad=pad, off=off, cut=cut)


@pytest.mark.parametrize("L", [1, 8, 9, 100])
@pytest.mark.parametrize("D,N,G,pad,off", [(70, 16, 2, 0, 0), (33, 1, 1, 3, 1), (40, 24, 1, 0, 0), (34, 64, 1, 0, 0),
                                           (35, 128, 1, 2, 1)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scan_within_its_counted_roundings(D, N, G, pad, off, dtype, L):
    c = scan_case(3, L, D, N, G, dtype, seed=62)
    scan_and_check(c, dtype, None, pad=pad, off=off)
    scan_and_check(c, dtype, [L, 0, (L + 1) // 2], gate=False, pad=pad, off=off)


@pytest.mark.parametrize("L", [6, 8])
@pytest.mark.parametrize("B,D,N,G", [(8, 4096, 16, 1), (12, 4100, 5, 2), (13, 1030, 64, 1), (7, 1032, 128, 4)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scan_of_a_few_rows_and_many_channels(B, D, N, G, dtype, L):
    """(as many as the kernel of few rows takes 6 to 8 of)"""
    c = scan_case(B, L, D, N, G, dtype, seed=63)
    scan_and_check(c, dtype, None, gate=False)
    scan_and_check(c, dtype, [L, 0, 1, L - 1, 5, 2, 3] + [L] * (B - 7), in_place=False, pad=1)


# ------------------------------------------------------------------------ together
@pytest.mark.parametrize("T", [1, 3])
def test_norm_and_4_bit_products_around_the_recurrent_step(T):
    """A retention layer that decodes with 4-bit weights: norm with the residual to
    8-bit rows, one product for q, k, v and the gate, the recurrent step, GroupNorm
    and gate, the output product, over several calls on a carried state.  The
    recurrent step takes dense heads, so the product's columns are copied apart."""
    B, H, dk, dv, dm, g = 3, 4, 64, 128, 256, 64
    n, gamma, eps = H * (2 * dk + 2 * dv), [0.9, 0.95, 0.98, 1.0], 1e-5
    w_in = R.ret_quantize_w4(rt((dm, n), 71, dm ** -0.5).cuda(), g)
    w_out = R.ret_quantize_w4(rt((H * dv, dm), 72, (H * dv) ** -0.5).cuda(), g, zeros=True)
    wn = 1 + rt((dm,), 73, 0.1)
    state = torch.zeros(B, H, dk, dv, device="cuda")
    S = torch.zeros(B, H, dk, dv, dtype=torch.float64)
    deq = lambda w: ref.dequantise_w4(*w).t()  # noqa: E731
    for call in range(3):
        x, r = rt((B, T, dm), 74 + call), rt((B, T, dm), 84 + call)
        code, sc = torch.empty(B, T, dm, device="cuda", dtype=I8), torch.empty(B, T, 1, device="cuda")
        ro = torch.empty(B, T, dm, device="cuda")
        R.ret_rms_norm(x.cuda(), code, weight=wn.cuda(), residual=r.cuda(), residual_out=ro, scales=sc)
        p = torch.empty(B * T, n, device="cuda")
        R.ret_matvec_w4(code.view(B * T, dm), *w_in[:2], p, x_scales=sc.view(B * T, 1))
        heads = [t.contiguous() for t in p.view(B, T, n).split([H * dk, H * dk, H * dv, H * dv], -1)]
        q, k, v = (t.view(B, T, H, -1).transpose(1, 2).contiguous() for t in heads[:3])
        o, y = torch.empty(B, H, T, dv, device="cuda"), torch.empty(B, T, H * dv, device="cuda")
        R.ret_recurrent_step(q, k, v, state, o, gamma, pos=call * T)
        R.ret_gate_norm(o, heads[3], y, eps)
        out = torch.empty(B * T, dm, device="cuda")
        R.ret_matvec_w4(y.view(B * T, H * dv), *w_out[:2], out, zeros=w_out[2])
        # in 64 bits, from the codes the norm gave
        p64 = (code.cpu().double() * sc.cpu().double()) @ deq(w_in)
        q64, k64, v64, g64 = (t.view(B, T, H, -1) for t in p64.split([H * dk, H * dk, H * dv, H * dv], -1))
        o64 = torch.empty(B, T, H, dv, dtype=torch.float64)
        for t in range(T):
            S = S * torch.tensor(gamma, dtype=torch.float64)[:, None, None] + k64[:, t, :, :, None] * v64[:, t, :, None]
            o64[:, t] = (q64[:, t, :, :, None] * S).sum(-2)
        o64 = (o64 - o64.mean(-1, keepdim=True)) / torch.sqrt(o64.var(-1, unbiased=False, keepdim=True) + eps)
        want = (o64 * ref.swish(g64)).reshape(B * T, H * dv) @ deq(w_out)
        # five fp32 stages, each within 1e-5 of its terms' magnitude
        assert float((out.cpu().double() - want).abs().max()) <= 1e-4 * float(want.abs().max())
        assert float((state.cpu().double() - S).abs().max()) <= 1e-4 * float(S.abs().max())
        s64, _ = ref.rms_norm(x, wn, r)
        assert ref.within(ro, s64, 2.0 ** -23 * s64.abs()) <= 1
