"""kq_rmsnorm_quant: the residual's addition, the root-mean-square norm and INT8 codes.

The reference is the formula in 64 bits. Bounds, from the kernel's arithmetic (fp32, every
step rounded once, half a step is 2^-24):
- h = x + r: one rounding; the sum of squares: at most 64 additions in a thread, 6 + 16 over
  the workgroup, so 90 roundings, half of which reach the root; the root, the division by n,
  the addition of eps and the reciprocal add 4, u = h w one, y = u r one. Together
  |y - y64| <= 60 * 2^-24 * |y64| =: YREL |y64|.
- a 16-bit output adds half a step of its type, eps / 2 (relative), or half the type's
  smallest step near zero.
- the step: YREL, one rounding each of clip * a and / 127, and half a step of its type.
- the codes: against the step the call stored, v = y64 / s, the code is the nearest integer to
  a number within YREL + 2 * 2^-24 of v: |q - clamp(v)| <= 0.5 + |v| (YREL + 2^-23).
For fp32 rows `normed` is y itself, so there the codes and steps are bit-exact against the
oracle's quantizer."""
import math

import numpy as np
import pytest

from kronecker_factored_transforms_amd import binding as B
from oracle import kq_oracle as O

YREL = 60 * 2.0 ** -24
DTYPES = ["bf16", "fp16", "fp32"]


def _dt(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def _half_step(dt):
    """(relative, absolute) rounding of one conversion to dt"""
    import torch
    f = torch.finfo(dt)
    return f.eps / 2, f.smallest_normal * f.eps / 2


def _inputs(T, n, dt, residual, gpu, seed, pad=0, scale=1.0):
    import torch
    g = torch.Generator().manual_seed(seed)

    def rows():
        return (scale * torch.randn((T, n + pad), generator=g)).to(dt).to(gpu)[:, :n]
    x = rows()
    r = rows() if residual else None
    w = (1 + 0.3 * torch.randn(n, generator=g)).to(dt).to(gpu)
    return x, r, w


def _check(x, r, w, eps, alpha, sdt, o, codes=True, normed=True):
    import torch
    dt = x.dtype
    h = x.double() + (r.double() if r is not None else 0)
    if r is not None:
        assert torch.equal(o.residual, (x.float() + r.float()).to(dt))
    ms = (h * h).mean(1, keepdim=True) + eps
    y = torch.where(ms > 0, h * w.double() / torch.sqrt(ms), torch.zeros_like(h))
    rel, tiny = _half_step(dt)
    if normed:
        err = (o.normed.double() - y).abs()
        bound = y.abs() * (YREL + (rel if dt != torch.float32 else 0)) * (1 + 2 ** -6) + tiny
        assert bool((err <= bound).all()), float((err - bound).max())
    if codes:
        clip = float(O.clip_ratio(alpha))
        s = o.scales.double()
        want = clip * y.abs().amax(1) / 127
        srel, stiny = _half_step(o.scales.dtype)
        assert bool(((s - want).abs() <= want * (YREL + 2 ** -23 + srel) * 1.01 + stiny).all())
        q = o.codes.view(torch.int8).double()
        live = s > 0
        assert bool((q[~live] == 0).all())
        v = y[live] / s[live, None]
        err = (q[live] - v.clamp(-128, 127)).abs()
        assert bool((err <= 0.5 + v.abs() * (YREL + 2 ** -23)).all()), float(err.max())
        if dt == torch.float32 and normed:  # the very y that was quantized
            qo, so = O.quantize_per_token(o.normed.cpu().numpy(), np.float32(clip),
                                          "fp16" if sdt == torch.float16 else "fp32", bits=8)
            assert np.array_equal(o.codes.cpu().numpy().view(np.int8), qo.astype(np.int8))
            assert np.array_equal(o.scales.cpu().numpy().view(np.uint8), so.view(np.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 7, 8, 64, 500, 512, 520, 2048, 2051, 4096, 5121, 8192, 11008, 16392,
                               32776, 65536])
def test_rows_of_every_length(gpu, n, dtype):
    import torch
    dt = _dt(dtype)
    T = 37 if n < 20000 else 5
    x, r, w = _inputs(T, n, dt, True, gpu, n)
    o = B.rmsnorm_quant(x, w, residual=r, normed=True, alpha=3.0)
    torch.cuda.synchronize()
    _check(x, r, w, 1e-5, 3.0, torch.float16, o)
    # the same rows, asked for one output at a time: the same bits
    a = B.rmsnorm_quant(x, w, residual=r, alpha=3.0)
    b = B.rmsnorm_quant(x, w, residual=r, codes=False, normed=True)
    assert a.normed is None and b.codes is None and b.scales is None
    assert torch.equal(a.codes, o.codes) and torch.equal(a.scales, o.scales)
    assert torch.equal(b.normed, o.normed) and torch.equal(b.residual, o.residual)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 3, 4, 5, 1000])
@pytest.mark.parametrize("n", [40, 4096])
def test_no_residual_fp32_steps(gpu, T, n):
    import torch
    x, _, w = _inputs(T, n, torch.bfloat16, False, gpu, T + n)
    o = B.rmsnorm_quant(x, w, scale_dtype="fp32", normed=True, eps=0.0)
    torch.cuda.synchronize()
    assert o.residual is None and o.scales.dtype == torch.float32
    _check(x, None, w, 0.0, math.inf, torch.float32, o)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,pad", [(4096, 8), (4096, 3), (100, 5), (8192, 1)])
def test_rows_inside_wider_ones(gpu, n, pad, dtype):
    """Strides that keep 16-byte alignment and strides that do not; nothing is written between
    the rows."""
    import torch
    dt = _dt(dtype)
    T = 33
    x, r, w = _inputs(T, n, dt, True, gpu, 5, pad=pad)
    big = torch.full((T, 2 * (n + pad)), 7.0, dtype=dt, device=gpu)  # both outputs in one buffer
    out = B.NormQuant(None, None, big[:, :n], big[:, n + pad:2 * n + pad])
    o = B.rmsnorm_quant(x, w, residual=r, normed=True, out=out)
    torch.cuda.synchronize()
    _check(x, r, w, 1e-5, math.inf, torch.float16, o)
    assert bool((big[:, n:n + pad] == 7).all()) and bool((big[:, 2 * n + pad:] == 7).all())
    c = B.rmsnorm_quant(x.contiguous(), w, residual=r.contiguous(), normed=True)
    assert torch.equal(c.codes, o.codes) and torch.equal(c.normed, o.normed)


@pytest.mark.gpu
def test_in_place(gpu):
    import torch
    for n in (4096, 1003):
        x, r, w = _inputs(50, n, torch.bfloat16, True, gpu, 9)
        want = B.rmsnorm_quant(x, w, residual=r, normed=True)
        x1, r1 = x.clone(), r.clone()
        o = B.rmsnorm_quant(x1, w, residual=r1, normed=True, out=B.NormQuant(None, None, r1, x1))
        assert torch.equal(r1, want.residual) and torch.equal(x1, want.normed)
        assert torch.equal(o.codes, want.codes)
        x2 = x.clone()
        o = B.rmsnorm_quant(x2, w, residual=r, out=B.NormQuant(None, None, x2, None))
        assert torch.equal(x2, want.residual) and torch.equal(o.scales, want.scales)


@pytest.mark.gpu
def test_rows_of_zeros_and_of_extremes(gpu):
    """Zero rows (with and without eps), rows of one large value, tiny and huge rows."""
    import torch
    n = 1024
    x = torch.zeros((6, n), dtype=torch.float32, device=gpu)
    x[1, 17] = 1e15
    x[2] = 1e-30
    x[3] = torch.linspace(-1, 1, n) * 1e17
    x[4, ::2] = -3.0
    w = torch.ones(n, dtype=torch.float32, device=gpu)
    for eps in (0.0, 1e-6):
        o = B.rmsnorm_quant(x, w, eps=eps, scale_dtype="fp32", normed=True)
        torch.cuda.synchronize()
        rows = [0, 1, 3, 4, 5] if eps == 0.0 else range(6)  # 1e-30 squared is 0 in fp32
        for t in rows:
            _check(x[t:t + 1], None, w, eps, math.inf, torch.float32,
                   B.NormQuant(o.codes[t:t + 1], o.scales[t:t + 1], None, o.normed[t:t + 1]))
        assert not o.codes[0].any() and float(o.scales[0]) == 0 and not o.normed[0].any()
    o = B.rmsnorm_quant(x, w, alpha=-math.inf)
    assert not o.codes.any() and not o.scales.any()


@pytest.mark.gpu
def test_many_rows(gpu):
    """More rows than one grid takes at once, each equal to its copy in a small call."""
    import torch
    x, r, w = _inputs(64, 264, torch.bfloat16, True, gpu, 3)
    T = 70001
    xs, rs = x.repeat(T // 64 + 1, 1)[:T], r.repeat(T // 64 + 1, 1)[:T]
    a, b = B.rmsnorm_quant(xs, w, residual=rs, normed=True), B.rmsnorm_quant(x, w, residual=r, normed=True)
    k = torch.arange(T, device=gpu) % 64
    for u, v in zip(a, b):
        assert torch.equal(u, v[k])


@pytest.mark.gpu
@pytest.mark.slow
def test_rows_past_four_gigabytes(gpu):
    import torch
    n, T = 65536, 36000  # 4.7 GB of bf16
    x = torch.empty((T, n), dtype=torch.bfloat16, device=gpu)
    part, _, w = _inputs(100, n, torch.bfloat16, False, gpu, 8)
    for i in range(0, T, 100):
        x[i:i + 100] = part
    o = B.rmsnorm_quant(x, w)
    small = B.rmsnorm_quant(part, w)
    for i in range(0, T, 100):
        assert torch.equal(o.codes[i:i + 100], small.codes), i
        assert torch.equal(o.scales[i:i + 100], small.scales), i


@pytest.mark.gpu
def test_another_stream_and_a_captured_call(gpu):
    import torch
    x, r, w = _inputs(300, 4096, torch.bfloat16, True, gpu, 1)
    want = B.rmsnorm_quant(x, w, residual=r, normed=True)
    torch.cuda.synchronize()
    for st in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        o = B.rmsnorm_quant(x, w, residual=r, normed=True, stream=st)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(o, want))
    g = torch.cuda.CUDAGraph()
    xi, ri = x.clone(), r.clone()
    with torch.cuda.graph(g):
        o = B.rmsnorm_quant(xi, w, residual=ri, normed=True)
    for i in range(4):
        xi.copy_(x.roll(i, 0))
        ri.copy_(r.roll(i, 0))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b.roll(i, 0)) for a, b in zip(o, want))


# --------------------------------------------------------------------- refusals (no GPU)
def _raw(**kw):
    a = dict(x=0x10000, ldx=64, res=0x20000, ldr=64, w=0x30000, T=4, n=64, xd=B.KQ_BF16, eps=1e-5,
             alpha=1.0, sd=B.KQ_FP16, ro=0x40000, ldres=64, y=0x50000, ldy=64, q=0x60000, s=0x70000)
    a.update(kw)
    return B.lib().kq_rmsnorm_quant(a["x"], a["ldx"], a["res"], a["ldr"], a["w"], a["T"], a["n"], a["xd"],
                                    a["eps"], a["alpha"], a["sd"], a["ro"], a["ldres"], a["y"], a["ldy"],
                                    a["q"], a["s"], None)


def test_refusals():
    assert _raw(T=0) == B.KQ_OK
    for kw in (dict(T=-1), dict(n=0), dict(xd=5), dict(sd=B.KQ_BF16), dict(eps=-1.0), dict(eps=math.nan),
               dict(eps=math.inf), dict(alpha=math.nan), dict(x=None), dict(w=None), dict(s=None),
               dict(q=None), dict(q=None, s=None, y=None), dict(res=None), dict(ldx=63), dict(ldr=63),
               dict(ldres=63), dict(ldy=63), dict(T=1 << 40), dict(ldx=1 << 62),
               dict(y=0x40000),            # two outputs in one place
               dict(ro=0x10080), dict(ro=0x20002), dict(ro=0x10000, ldres=128),  # inputs, not in place
               dict(y=0x20000), dict(q=0x10000), dict(ro=0x30000), dict(s=0x60010)):
        assert _raw(**kw) == B.KQ_ERR_INVALID_ARG, kw
    assert _raw(n=65537, ldx=65537, ldr=65537, ldres=65537, ldy=65537) == B.KQ_ERR_UNSUPPORTED
    for kw in (dict(x=0x10001), dict(res=0x20001), dict(w=0x30001), dict(ro=0x40001), dict(y=0x50001),
               dict(s=0x70001), dict(sd=B.KQ_FP32, s=0x70002)):
        assert _raw(**kw) == B.KQ_ERR_ALIGNMENT, kw


def test_host_tensors_are_refused():
    import torch
    with pytest.raises(ValueError):
        B.rmsnorm_quant(torch.zeros((2, 8)), torch.ones(8))


@pytest.mark.gpu
def test_tensors_that_do_not_fit_are_refused(gpu):
    import torch
    x, r, w = _inputs(4, 64, torch.bfloat16, True, gpu, 1)
    bad = [dict(weight=w[:63]), dict(weight=w.float()), dict(residual=r[:3]), dict(residual=r.float()),
           dict(residual=r.t().contiguous().t()), dict(scale_dtype="bf16"), dict(codes=False),
           dict(residual=r.cpu()), dict(x=x[:, ::2]), dict(x=x[:1].expand(4, 64)),
           dict(out=B.NormQuant(torch.empty((4, 63), dtype=torch.uint8, device=gpu), None, None, None)),
           dict(out=B.NormQuant(None, torch.empty(4, device=gpu), None, None)),
           dict(out=B.NormQuant(None, None, r[:2], None))]
    for kw in bad:
        a = dict(x=x, weight=w, residual=r)
        a.update(kw)
        with pytest.raises(ValueError):
            B.rmsnorm_quant(**a)
    e = B.rmsnorm_quant(x[:0], w, residual=r[:0], normed=True)
    assert e.codes.shape == (0, 64) and e.normed.shape == (0, 64)


def test_strides_whose_rows_leave_64_bits_are_refused():
    for name in ("ldx", "ldr", "ldres", "ldy"):
        assert _raw(**{name: 1 << 40, "T": 1 << 30}) == B.KQ_ERR_INVALID_ARG, name
