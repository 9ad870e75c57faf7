"""The operators around the mixers on the GPU against their plain 64-bit forms
(block_ref): sizes where vector pieces, tiles, groups and warps end, strided and
unaligned rows, padded batches, empty ones, values that are not finite, in-place
states, streams, captured graphs, and a run of them as a block serves."""
import pytest
import torch

import block_ref as ref
from retentive_network_scale_b200 import retention as R
from retentive_network_scale_b200.synth import random_tensor

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from retentive_network_scale_b200 import build
    build.build()
    R.load_library()
    yield
    torch.cuda.synchronize()
    assert R.ret_last_device_status() == 0


def rt(shape, seed, scale=1.0, dtype=F32):
    return random_tensor(shape, seed, scale).to(dtype)


def strided(t, pad, offset=0):
    """t as columns offset.. of rows that are `pad` elements longer, on the GPU."""
    wide = torch.full(t.shape[:-1] + (t.shape[-1] + pad,), 7.0, device="cuda").to(t.dtype)
    out = wide[..., offset:offset + t.shape[-1]]
    out.copy_(t)
    return out


# ------------------------------------------------------------------------ norm
@pytest.mark.parametrize("rows,d,pad,off", [(1, 1, 0, 0), (3, 37, 0, 0), (5, 64, 8, 8), (2, 256, 1, 1),
                                            (70, 512, 0, 0), (9, 2048, 0, 0), (4, 2056, 24, 16),
                                            (3, 5120, 0, 0), (2, 16384, 0, 0)])
@pytest.mark.parametrize("xt,rtype,yt", [(BF16, BF16, BF16), (F32, F32, F32), (BF16, F32, F32),
                                         (F32, BF16, BF16), (BF16, None, F32)])
def test_rms_norm(rows, d, pad, off, xt, rtype, yt):
    x, w = rt((rows, d), 1, 1.0, xt), 1 + rt((d,), 2, 0.2)
    r = None if rtype is None else rt((rows, d), 3, 3.0, rtype)
    y = torch.full((rows, d), 9.0, device="cuda", dtype=yt)
    rg = None if r is None else r.cuda()
    ro = None if r is None else torch.empty_like(rg)
    R.ret_rms_norm(strided(x, pad, off), y, weight=w.cuda(), residual=rg, residual_out=ro)
    s, want = ref.rms_norm(x, w, r)
    assert ref.within(y, want, ref.NORM * want.abs() + ref.rounded(want, yt)) <= 1
    if r is not None:
        # one fp32 addition, then the rounding
        assert ref.within(ro, s, 2.0 ** -24 * s.abs() + ref.rounded(s, rtype)) <= 1
        R.ret_rms_norm(strided(x, pad, off), y, residual=rg, residual_out=rg)   # in place, no weight
        assert torch.equal(rg, ro)


@pytest.mark.parametrize("rows,d,group", [(1, 32, 0), (3, 100, 0), (5, 96, 32), (4, 320, 64),
                                          (7, 2048, 128), (2, 2048, 0), (3, 8192, 32), (2, 16384, 128)])
@pytest.mark.parametrize("xt", [BF16, F32])
@pytest.mark.parametrize("yt", [torch.int8, torch.float8_e4m3fn])
def test_rms_norm_codes(rows, d, group, xt, yt):
    x, w, r = rt((rows, d), 4, 1.0, xt), 1 + rt((d,), 5, 0.2), rt((rows, d), 6, 2.0, xt)
    g = group or d
    y = torch.empty(rows, d, device="cuda", dtype=yt)
    sc = torch.full((rows, d // g), -1.0, device="cuda")
    R.ret_rms_norm(x.cuda(), y, weight=w.cuda(), residual=r.cuda(), scales=sc)
    _, want = ref.rms_norm(x, w, r)
    top = 127.0 if yt == torch.int8 else 448.0
    grp = want.view(rows, d // g, g)
    scale = grp.abs().amax(-1) / top
    assert ref.within(sc, scale, ref.NORM * scale) <= 1
    codes = y.float().cpu().double()
    assert float(codes.abs().max()) <= top
    got = (codes.view(rows, d // g, g) * sc.cpu().double()[..., None]).view(rows, d)
    step = scale.repeat_interleave(g, 1)
    half = 0.5 * step if yt == torch.int8 else torch.maximum(want.abs() * 2.0 ** -4, step * 2.0 ** -10)
    # 4 NORM: the code is taken of a value and with a scale that are each off
    assert ref.within(got, want, half + 4 * ref.NORM * (want.abs() + step)) <= 1


def test_rms_norm_codes_of_zero_and_non_finite_rows():
    d, g = 256, 64
    x = rt((5, d), 7)
    x[0] = 0.0
    x[1, g:2 * g] = 0.0
    x[2, 3] = float("nan")
    x[3, 5] = float("inf")
    w = torch.ones(d)
    w[130] = float("inf")       # channel of group 2 in every row
    for yt in (torch.int8, torch.float8_e4m3fn):
        y = torch.empty(5, d, device="cuda", dtype=yt)
        sc = torch.empty(5, d // g, device="cuda")
        R.ret_rms_norm(x.cuda(), y, weight=torch.ones(d, device="cuda"), scales=sc)
        c, s = y.float().cpu(), sc.cpu()
        assert bool((c[0] == 0).all()) and bool((s[0] == 0).all())
        assert bool((c[1, g:2 * g] == 0).all()) and float(s[1, 1]) == 0 and float(s[1, 0]) > 0
        assert bool(torch.isnan(s[2]).all())            # the sum of squares is NaN
        assert bool(torch.isnan(s[3, 0]))               # infinity over an infinite norm
        assert bool(torch.isfinite(s[4]).all())
        R.ret_rms_norm(x.cuda(), y, weight=w.cuda(), scales=sc)
        s = sc.cpu()
        assert bool(torch.isnan(s[4, 2])) and bool(torch.isfinite(s[4, [0, 1, 3]]).all())
        whole = torch.empty(5, 1, device="cuda")
        R.ret_rms_norm(x.cuda(), y, weight=w.cuda(), scales=whole)
        assert bool(torch.isnan(whole[4])) and bool((y[4].float() == 0).all())


def test_rms_norm_empty_and_refusals():
    x = torch.empty(0, 64, device="cuda")
    R.ret_rms_norm(x, torch.empty_like(x))
    x = torch.ones(2, 64, device="cuda")
    y = torch.empty_like(x)
    with pytest.raises(ValueError):
        R.ret_rms_norm(x, y, scales=torch.empty(2, 1, device="cuda"))
    with pytest.raises(ValueError):
        R.ret_rms_norm(x, y.to(torch.int8))
    with pytest.raises(ValueError):
        R.ret_rms_norm(x.t(), y.t())
    with pytest.raises(ValueError):
        R.ret_rms_norm(x[:1].expand(2, 64), y)          # rows on top of each other
    with pytest.raises(R.RetentionError):
        R.ret_rms_norm(x, y, eps=-1.0)


# ------------------------------------------------------------------------ convolution
LENS = {"full": None, "padded": [0, 1, 33, 70], "outside": [-5, 1000, 2, 64]}


@pytest.mark.parametrize("L", [1, 2, 3, 31, 32, 33, 70])
@pytest.mark.parametrize("D,pad,off", [(8, 0, 0), (264, 8, 8), (37, 3, 1), (66, 2, 0), (1024, 1024, 0)])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_causal_conv(L, D, pad, off, W, dtype):
    B = 4
    x, w = rt((B, L, D), 11, 1.0, dtype), rt((D, W), 12, W ** -0.5)
    bias, s0 = rt((D,), 13, 0.3), rt((B, W - 1, D), 14, 1.0, dtype)
    for name, lens in LENS.items():
        for state in (None, s0):
            act = name != "outside"
            n = None if lens is None else torch.tensor(lens, dtype=torch.int32)
            want, last, tol = ref.causal_conv(x, w, bias if act else None, act, n, state)
            xs = x.clone()
            if n is not None:
                for b in range(B):
                    xs[b, max(0, lens[b]):] = float("nan")      # rows that must not be read
            y = torch.full((B, L, D), 5.0, device="cuda", dtype=dtype)
            held = torch.full((B, W - 1, D), 8.0, device="cuda", dtype=dtype) if state is None else state.cuda()
            R.ret_causal_conv(strided(xs, pad, off), w.cuda(), y, bias=bias.cuda() if act else None,
                              swish=act, lengths=None if n is None else n.cuda(),
                              state_in=None if state is None else held, state_out=held)
            dead = torch.isnan(want)
            assert bool((y.cpu()[dead] == 5.0).all())
            assert ref.within(torch.where(dead, 0.0, y.cpu().double()), torch.where(dead, 0.0, want),
                              tol + ref.rounded(torch.where(dead, 0.0, want), dtype)) <= 1
            assert torch.equal(held.cpu().double(), last)


def test_causal_conv_tokens_follow_the_prompt():
    B, L, D, W = 3, 45, 96, 4
    x, w, bias = rt((B, L, D), 15).cuda(), rt((D, W), 16).cuda(), rt((D,), 17).cuda()
    full = torch.empty(B, L, D, device="cuda")
    end = torch.empty(B, W - 1, D, device="cuda")
    R.ret_causal_conv(x, w, full, bias=bias, state_out=end)
    part, state = torch.empty(B, 33, D, device="cuda"), torch.empty(B, W - 1, D, device="cuda")
    R.ret_causal_conv(x[:, :33].contiguous(), w, part, bias=bias, state_out=state)
    assert torch.equal(part, full[:, :33])
    for t in range(33, L):
        y = torch.empty(B, 1, D, device="cuda")
        R.ret_causal_conv(x[:, t:t + 1].contiguous(), w, y, bias=bias, state_in=state, state_out=state)
        assert torch.equal(y[:, 0], full[:, t])
    assert torch.equal(state, end)


# ------------------------------------------------------------------------ scan
def scan_case(B, L, D, N, G, dtype, seed=21):
    u, delta = rt((B, L, D), seed, 1.0, dtype), rt((B, L, D), seed + 1, 1.0, dtype)
    A = -(torch.arange(1, N + 1).float() * torch.exp(rt((D, N), seed + 2, 0.3)))
    bm, cm = rt((B, L, G, N), seed + 3, 1.0, dtype), rt((B, L, G, N), seed + 4, 1.0, dtype)
    skip, z = rt((D,), seed + 5), rt((B, L, D), seed + 6, 1.0, dtype)
    bias, s0 = rt((D,), seed + 7, 1.0) - 3.0, rt((B, D, N), seed + 8)
    return dict(u=u, delta=delta, A=A, Bm=bm, Cm=cm, skip=skip, z=z, bias=bias, s0=s0)


def run_scan(c, dtype, gate=True, state=True, softplus=True, bare=False, lens=None, pad=0, off=0, in_place=True,
             stream=None):
    B, L, D = c["u"].shape
    N = c["A"].shape[1]
    n = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    u, delta, z = (c[k].clone() for k in ("u", "delta", "z"))
    if n is not None:
        for b in range(B):
            for t in (u, delta, z):
                t[b, max(0, lens[b]):] = float("nan")           # rows that must not be read
    bm = strided(c["Bm"].flatten(2), pad, off).unflatten(2, c["Bm"].shape[2:])
    cm = strided(c["Cm"].flatten(2), pad, off).unflatten(2, c["Cm"].shape[2:])
    y = torch.full((B, L, D), 5.0, device="cuda", dtype=dtype)
    held = c["s0"].cuda() if state else torch.full((B, D, N), 8.0, device="cuda")
    out = held if in_place or not state else torch.full_like(held, 8.0)
    R.ret_selective_scan(strided(u, pad, off), strided(delta, pad, off), c["A"].cuda(), bm, cm, y,
                         skip=None if bare else c["skip"].cuda(), Z=strided(z, pad, off) if gate else None,
                         delta_bias=None if bare else c["bias"].cuda(), softplus=softplus,
                         lengths=None if n is None else n.cuda(), state_in=held if state else None,
                         state_out=out, stream=stream)
    return y, out


def check_scan(c, dtype, gate=True, state=True, softplus=True, bare=False, lens=None, **kw):
    y, out = run_scan(c, dtype, gate, state, softplus, bare, lens, **kw)
    want, last, tol, stol = ref.selective_scan(
        c["u"], c["delta"], c["A"], c["Bm"], c["Cm"], None if bare else c["skip"], c["z"] if gate else None,
        None if bare else c["bias"], softplus, None if lens is None else torch.tensor(lens),
        c["s0"] if state else None)
    dead = torch.isnan(want)
    assert bool((y.cpu()[dead] == 5.0).all())
    want = torch.where(dead, 0.0, want)
    assert ref.within(torch.where(dead, 0.0, y.cpu().double()), want, tol + ref.rounded(want, dtype)) <= 1
    assert ref.within(out, last, stol) <= 1


@pytest.mark.parametrize("L", [1, 2, 31, 33, 100])
@pytest.mark.parametrize("D,N,G,pad,off", [(8, 16, 1, 0, 0), (70, 16, 2, 0, 0), (33, 1, 1, 3, 1),
                                           (96, 5, 3, 8, 8), (40, 8, 1, 0, 0), (36, 24, 2, 1, 0),
                                           (34, 64, 1, 0, 0), (35, 100, 1, 2, 1), (4, 128, 4, 0, 0),
                                           (160, 16, 2, 0, 0), (48, 32, 3, 8, 8), (32, 120, 2, 8, 0)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_selective_scan(L, D, N, G, pad, off, dtype):
    c = scan_case(3, L, D, N, G, dtype)
    check_scan(c, dtype, pad=pad, off=off)
    check_scan(c, dtype, gate=False, state=False, pad=pad, off=off, lens=[0, L, (L + 1) // 2])
    check_scan(c, dtype, lens=[1, 0, L + 7], in_place=False)
    # the step as it is (delta made positive), no bias, no skip
    c2 = dict(c, delta=(c["delta"].float().abs() * 0.1).to(dtype))
    check_scan(c2, dtype, softplus=False, bare=True, state=False)


@pytest.mark.parametrize("B,L,D", [(1, 2000, 16), (2, 1500, 40), (1, 700, 300)])
def test_selective_scan_long(B, L, D):
    """Few channels and many rows."""
    for dtype in (F32, BF16):
        c = scan_case(B, L, D, 16, 1, dtype, seed=31)
        check_scan(c, dtype)
        check_scan(c, dtype, state=False, gate=False, lens=[L - 3] + [5] * (B - 1))


def test_selective_scan_growing_states():
    """A above 0 (states that grow), and 0 (that only add up), in one piece and
    in segments."""
    for L, D in ((60, 40), (1100, 8)):
        c = scan_case(2, L, D, 16, 1, F32, seed=45)
        c["A"][:, 0] = 0.0
        c["A"][:, 1] = 0.01
        c["A"][:, 2:] *= 0.1
        check_scan(c, F32, lens=[L, L - 30])


def test_a_call_with_no_rows_passes_the_state_on():
    s0 = rt((2, 8, 16), 46).cuda()
    out = torch.empty_like(s0)
    u, bm = torch.empty(2, 0, 8, device="cuda"), torch.empty(2, 0, 16, device="cuda")
    A = -torch.ones(8, 16, device="cuda")
    R.ret_selective_scan(u, u, A, bm, bm, u, state_in=s0, state_out=out)
    assert torch.equal(out, s0)
    R.ret_selective_scan(u, u, A, bm, bm, u, state_out=out)
    assert bool((out == 0).all())
    held = rt((2, 3, 8), 47).cuda()
    end = torch.empty_like(held)
    R.ret_causal_conv(u, torch.ones(8, 4, device="cuda"), u, state_in=held, state_out=end)
    assert torch.equal(end, held)


def test_operands_of_the_scan_at_both_ends_of_an_allocation():
    """Unaligned rows whose first and last elements are an allocation's: what
    lies before and behind them in the aligned words does not matter."""
    B, L, D, N = 1, 21, 13, 3
    c = scan_case(B, L, D, N, 1, BF16, seed=48)
    check_scan(c, BF16)
    wide = torch.full((L * D + 3,), float("nan"), device="cuda", dtype=BF16)
    u = wide[3:].view(1, L, D)
    u.copy_(c["u"])
    y, want = torch.empty(1, L, D, device="cuda", dtype=BF16), torch.empty(1, L, D, device="cuda", dtype=BF16)
    g = {k: v.cuda() for k, v in c.items()}
    R.ret_selective_scan(u, g["delta"], g["A"], g["Bm"], g["Cm"], y)
    R.ret_selective_scan(g["u"], g["delta"], g["A"], g["Bm"], g["Cm"], want)
    assert torch.equal(y, want)


def test_selective_scan_extreme_steps():
    """Steps of 0 (delta -inf: the state stays), of 10^4 (it is forgotten), and
    softplus far from 0."""
    c = scan_case(2, 40, 24, 16, 1, F32, seed=41)
    c["delta"][0, 7] = float("-inf")
    c["delta"][0, 20] = 1e4
    c["delta"][1, 5] = 80.0
    c["delta"][1, 6] = -60.0
    check_scan(c, F32)


def test_selective_scan_tokens_follow_the_prompt():
    B, L, D, N = 2, 50, 40, 16
    c = scan_case(B, L, D, N, 1, F32, seed=51)
    full, end = run_scan(c, F32)
    cut = lambda a, b: {k: (v[:, a:b].contiguous() if v.dim() > 2 and k != "s0" else v) for k, v in c.items()}  # noqa: E731
    y0, state = run_scan(cut(0, 35), F32)
    ys = [y0]
    for t in range(35, L):
        ct = dict(cut(t, t + 1), s0=state.cpu())
        y, state = run_scan(ct, F32)
        ys.append(y)
    want, last, tol, stol = ref.selective_scan(c["u"], c["delta"], c["A"], c["Bm"], c["Cm"], c["skip"], c["z"],
                                               c["bias"], True, None, c["s0"])
    assert ref.within(torch.cat(ys, 1), want, tol + ref.rounded(want, F32)) <= 1
    assert ref.within(full, want, tol + ref.rounded(want, F32)) <= 1
    assert ref.within(state, last, stol) <= 1 and ref.within(end, last, stol) <= 1


# ------------------------------------------------------------------------ 4-bit product
def w4_case(N, K, g, zeros, seed=61):
    gen = torch.Generator().manual_seed(seed)
    wq = torch.randint(0, 256, (N, K // 2), generator=gen, dtype=torch.uint8)
    s = (torch.rand((N, K // g), generator=gen) + 0.5).bfloat16()
    z = torch.randint(0, 16, (N, K // g), generator=gen, dtype=torch.uint8) if zeros else None
    return wq, s, z


def x_case(M, K, xt, xg, seed=62):
    x = rt((M, K), seed)
    if xt in (F32, BF16):
        return x.to(xt), None
    top = 127.0 if xt == torch.int8 else 448.0
    xs = x.view(M, K // xg, xg).abs().amax(-1) / top
    v = x / xs.repeat_interleave(xg, 1)
    return (torch.round(v) if xt == torch.int8 else v).to(xt), xs


@pytest.mark.parametrize("M", [1, 2, 3, 7, 8, 9, 16, 17, 40, 64])
@pytest.mark.parametrize("N,K,g,zeros", [(16, 128, 128, False), (1, 32, 32, False), (50, 1056, 32, True),
                                         (33, 704, 64, False), (130, 2048, 128, True), (24, 192, 64, True)])
@pytest.mark.parametrize("xt", [F32, BF16, torch.int8, torch.float8_e4m3fn])
def test_matvec_w4(M, N, K, g, zeros, xt):
    wq, s, z = w4_case(N, K, g, zeros)
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    for xg in ((K, g) if xt not in (F32, BF16) else (K,)):
        x, xs = x_case(M, K, xt, xg)
        want, tol = ref.matvec_w4(x.float(), wq, s, z, xs)
        yt = F32 if M % 2 else BF16
        y = torch.full((M, N), 7.0, device="cuda", dtype=yt)
        R.ret_matvec_w4(x.cuda(), wq.cuda(), s.cuda(), y, zeros=cuda(z), x_scales=cuda(xs))
        assert ref.within(y, want, tol + ref.rounded(want, yt)) <= 1


@pytest.mark.parametrize("M,N,K,g", [(1, 2050, 8192, 128), (5, 4096, 4096, 32), (33, 1024, 9216, 64)])
@pytest.mark.parametrize("xt", [F32, BF16, torch.int8])
def test_matvec_w4_large_and_strided(M, N, K, g, xt):
    wq, s, z = w4_case(N, K, g, True, seed=63)
    x, xs = x_case(M, K, xt, K, seed=64)
    want, tol = ref.matvec_w4(x.float(), wq, s, z, xs)
    for pad, off in ((0, 0), (3, 1)):
        y = torch.empty(M, N, device="cuda")
        R.ret_matvec_w4(strided(x, pad, off), wq.cuda(), s.cuda(), y, zeros=z.cuda(),
                        x_scales=None if xs is None else xs.cuda())
        assert ref.within(y, want, tol) <= 1


def test_matvec_w4_repeats_bit_for_bit_and_keeps_infinities():
    wq, s, z = w4_case(300, 2048, 128, True, seed=65)
    wq, s, z = wq.cuda(), s.cuda(), z.cuda()
    x = rt((3, 2048), 66).cuda()
    x[1, 5] = float("inf")
    x[2, 6] = float("nan")
    y, y2 = torch.empty(3, 300, device="cuda"), torch.empty(3, 300, device="cuda")
    R.ret_matvec_w4(x, wq, s, y, zeros=z)
    R.ret_matvec_w4(x, wq, s, y2, zeros=z)
    assert torch.equal(y[0], y2[0]) and bool(torch.isfinite(y[0]).all())
    w5 = ref.dequantise_w4(wq, s, z)[:, 5]
    got = y[1].cpu().double()
    assert bool((got[w5 > 0] == float("inf")).all()) and bool((got[w5 < 0] == float("-inf")).all())
    assert bool(torch.isnan(got[w5 == 0]).all()) and bool(torch.isnan(y[2]).all())
    e = torch.empty(0, 300, device="cuda")
    R.ret_matvec_w4(x[:0], wq, s, e, zeros=z)


@pytest.mark.parametrize("wt", [F32, BF16])
@pytest.mark.parametrize("zeros", [False, True])
def test_quantize_w4(wt, zeros):
    K, N, g = 384, 70, 64
    W = rt((K, N), 67, 0.5, wt)
    W[:g, 3] = 0.0                                              # an all-zero group
    W[g:2 * g, 4] = W[g:2 * g, 4].abs() + 0.25                  # one of one sign
    wq, s, z = R.ret_quantize_w4(strided(W, 5, 2), g, zeros=zeros)
    assert (z is not None) == zeros
    got = ref.dequantise_w4(wq, s, z).t()
    t = W.double().view(K // g, g, N)
    lo, hi = t.amin(1).clamp(max=0), t.amax(1).clamp(min=0)
    step = ((hi - lo) / 15 if zeros else torch.maximum(hi, -lo) / 7)
    # half a step; the scale's rounding (2^-8) moves the far end of the range by
    # up to 15 * 2^-8 of a step, and the zero point's by half a step
    tol = step * (0.5 + 15 * ref.BF16 + (0.5 if zeros else 0.0)) + 1e-6
    assert ref.within(got, W.double(), tol.repeat_interleave(g, 0)) <= 1
    assert bool((got[:g, 3] == 0).all())


# ------------------------------------------------------------------------ all of them
def test_offsets_past_32_bits():
    """Operands of more than 2^31 elements: the last rows are checked."""
    D, L = 8192, 270000                                         # 2.2e9 elements
    x = torch.zeros(1, L, D, device="cuda", dtype=BF16)
    tail = rt((1, 64, D), 71, 1.0, BF16)
    x[:, -64:] = tail.cuda()
    y = torch.empty_like(x)
    w, bias = rt((D, 4), 72), rt((D,), 73)
    R.ret_causal_conv(x, w.cuda(), y, bias=bias.cuda())
    want, _, tol = ref.causal_conv(tail, w, bias, True, None, torch.zeros(1, 3, D, dtype=BF16))
    assert ref.within(y[:, -64:], want, tol + ref.rounded(want, BF16)) <= 1
    R.ret_rms_norm(x[0], y[0])
    _, want = ref.rms_norm(tail[0])
    assert ref.within(y[0, -64:], want, ref.NORM * want.abs() + ref.rounded(want, BF16)) <= 1
    # the scan from a zero state: rows of zeros leave it at zero
    bm = torch.ones(1, L, 1, 4, device="cuda", dtype=BF16)
    A = -(1 + rt((D, 4), 74).abs())
    R.ret_selective_scan(x, x, A.cuda(), bm, bm, y)
    one = torch.ones(1, 64, 1, 4, dtype=BF16)
    want, _, tol, _ = ref.selective_scan(tail, tail, A, one, one)
    assert ref.within(y[:, -64:], want, tol + ref.rounded(want, BF16)) <= 1


def test_streams_and_captured_graphs():
    """Each call on a stream of its own gives what the default stream gives,
    bit for bit, and so does a captured graph replayed on new inputs."""
    c = scan_case(2, 300, 64, 16, 1, BF16, seed=81)
    g = {k: v.cuda() for k, v in c.items()}
    wq, s, _ = (t.cuda() if t is not None else None for t in w4_case(64, 64, 64, False))
    w, wn = rt((64, 4), 82).cuda(), rt((64,), 83).cuda()
    x = torch.empty(2, 300, 64, device="cuda", dtype=BF16)

    def chain(stream=None):
        n = torch.empty(600, 64, device="cuda", dtype=torch.int8)
        sc = torch.empty(600, 1, device="cuda")
        R.ret_rms_norm(x.view(600, 64), n, weight=wn, scales=sc, stream=stream)
        p = torch.empty(64, 64, device="cuda", dtype=BF16)
        R.ret_matvec_w4(n[:64], wq, s, p, x_scales=sc[:64], stream=stream)
        v, y = torch.empty_like(x), torch.empty_like(x)
        R.ret_causal_conv(x, w, v, stream=stream)
        end = torch.empty_like(g["s0"])
        R.ret_selective_scan(v, g["delta"], g["A"], g["Bm"], g["Cm"], y, skip=g["skip"], Z=g["z"],
                             delta_bias=g["bias"], state_in=g["s0"], state_out=end, stream=stream)
        return sc, n, p, v, y, end

    x.copy_(c["u"])
    want = chain()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = chain(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    x.zero_()
    with torch.cuda.graph(graph):
        held = chain()
    x.copy_(c["u"])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, held))


def test_calls_of_two_host_threads():
    """Calls of different sizes of the same kernels at once, each thread on a
    stream of its own."""
    import threading
    jobs, bad = [], []
    for K, M, L in ((256, 3, 40), (8192, 3, 400)):
        wq, s, _ = w4_case(48, K, 128, False, seed=85)
        x = x_case(M, K, BF16, K, seed=86)[0].cuda()
        c = scan_case(1, L, 24, 16, 1, F32, seed=87)
        jobs.append((x, wq.cuda(), s.cuda(), {k: v.cuda() for k, v in c.items()}))
    torch.cuda.synchronize()

    def work(x, wq, s, c):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            y = [torch.empty(x.shape[0], 48, device="cuda") for _ in range(40)]
            z = [torch.empty_like(c["u"]) for _ in range(40)]
            try:
                for a, b in zip(y, z):
                    R.ret_matvec_w4(x, wq, s, a)
                    R.ret_selective_scan(c["u"], c["delta"], c["A"], c["Bm"], c["Cm"], b)
                stream.synchronize()
                if not all(torch.equal(a, y[0]) for a in y) or not all(torch.equal(b, z[0]) for b in z):
                    bad.append("results differ")
            except Exception as e:  # noqa: BLE001 -- handed to the test's own thread
                bad.append(repr(e))

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad


def test_block_serves_a_prompt_and_then_tokens():
    """A block of the operators: norm with the residual, 4-bit projections of
    its 8-bit rows, convolution, scan, 4-bit output projection.  A prompt of 12
    tokens and then single tokens give what the whole sequence gives, and both
    are near the same block in 64 bits on the same codes."""
    B, L, dm, D, N, W, g = 2, 20, 128, 256, 16, 4, 64
    dev = lambda t: t.cuda()  # noqa: E731
    w_in, s_in, _ = R.ret_quantize_w4(dev(rt((dm, 2 * D), 91, dm ** -0.5)), g)
    w_x, s_x, _ = R.ret_quantize_w4(dev(rt((D, D + 2 * N), 92, D ** -0.5)), g)
    w_out, s_out, _ = R.ret_quantize_w4(dev(rt((D, dm), 93, D ** -0.5)), g)
    wn, wc, bc = 1 + rt((dm,), 94, 0.1), rt((D, W), 95, 0.5), rt((D,), 96, 0.1)
    A = -torch.arange(1, N + 1).float().expand(D, N).contiguous()
    skip, bias = torch.ones(D), rt((D,), 97, 0.5) - 3
    x, r = rt((B, L, dm), 98), rt((B, L, dm), 99)

    def block(xs, rs, conv_state, state):
        n = xs.shape[1]
        code = torch.empty(B, n, dm, device="cuda", dtype=torch.int8)
        sc = torch.empty(B, n, 1, device="cuda")
        ro = torch.empty_like(rs)
        R.ret_rms_norm(xs, code, weight=dev(wn), residual=rs, residual_out=ro, scales=sc)
        xz = torch.empty(B * n, 2 * D, device="cuda")
        R.ret_matvec_w4(code.view(B * n, dm), w_in, s_in, xz, x_scales=sc.view(B * n, 1))
        xz = xz.view(B, n, 2 * D)
        u = torch.empty(B, n, D, device="cuda")
        R.ret_causal_conv(xz[..., :D], dev(wc), u, bias=dev(bc), state_in=conv_state, state_out=conv_state)
        p = torch.empty(B * n, D + 2 * N, device="cuda")
        R.ret_matvec_w4(u.view(B * n, D), w_x, s_x, p)
        p = p.view(B, n, D + 2 * N)
        y = torch.empty(B, n, D, device="cuda")
        R.ret_selective_scan(u, p[..., :D], dev(A), p[..., D:D + N], p[..., D + N:], y, skip=dev(skip),
                             Z=xz[..., D:], delta_bias=dev(bias), state_in=state, state_out=state)
        out = torch.empty(B * n, dm, device="cuda")
        R.ret_matvec_w4(y.view(B * n, D), w_out, s_out, out)
        return out.view(B, n, dm), ro, code, sc

    zero = lambda: (torch.zeros(B, W - 1, D, device="cuda"), torch.zeros(B, D, N, device="cuda"))  # noqa: E731
    cs, hs = zero()
    full, ro, code, sc = block(dev(x), dev(r), cs, hs)
    c2, h2 = zero()
    outs = [block(dev(x[:, :12].contiguous()), dev(r[:, :12].contiguous()), c2, h2)[0]]
    for t in range(12, L):
        outs.append(block(dev(x[:, t:t + 1].contiguous()), dev(r[:, t:t + 1].contiguous()), c2, h2)[0])
    # the same block in 64 bits, from the codes the norm gave
    xq = code.cpu().double() * sc.cpu().double()
    xz = xq @ ref.dequantise_w4(w_in, s_in).t()
    u, last, _ = ref.causal_conv(xz[..., :D], wc, bc)
    p = u @ ref.dequantise_w4(w_x, s_x).t()
    y, h, _, _ = ref.selective_scan(u, p[..., :D], A, p[..., D:D + N, None].transpose(2, 3),
                                    p[..., D + N:, None].transpose(2, 3), skip, xz[..., D:], bias)
    want = y @ ref.dequantise_w4(w_out, s_out).t()
    size = float(want.abs().max())
    # five fp32 stages, each within 1e-5 of its terms' magnitude
    for got in (full, torch.cat(outs, 1)):
        assert float((got.cpu().double() - want).abs().max()) <= 1e-4 * size
    for got in (hs, h2):
        assert float((got.cpu().double() - h).abs().max()) <= 1e-4 * float(h.abs().max())
    assert float((cs.cpu().double() - last).abs().max()) <= 1e-4 * float(last.abs().max())
    s64, _ = ref.rms_norm(x, wn, r)
    assert ref.within(ro, s64, 2.0 ** -23 * s64.abs()) <= 1
