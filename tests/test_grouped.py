"""kq_grouped_gemm: INT4 and INT8 products grouped by expert, with ragged sizes.

The integer sums are exact and each output is two fp32 roundings and one conversion, so every
output is compared bit for bit with the same steps in NumPy (the sums in 64 bits)."""
import numpy as np
import pytest

from kronecker_factored_transforms_amd import binding as B
from oracle import kq_oracle as O


def _pack(q, bits):
    return O.pack_int4(q) if bits == 4 else q.view(np.uint8)


def _case(rng, T, K, E, N, counts, bits, sdt, rows=True, extremes=False):
    lo, hi = (-8, 8) if bits == 4 else (-128, 128)
    if extremes:  # the lowest code everywhere: the largest sums there are
        qx, qw = np.full((T, K), lo, np.int8), np.full((E, N, K), lo, np.int8)
    else:
        qx = rng.integers(lo, hi, (T, K)).astype(np.int8)
        qw = rng.integers(lo, hi, (E, N, K)).astype(np.int8)
    sx = rng.uniform(1e-3, 0.5, T).astype(sdt)
    sw = rng.uniform(1e-3, 0.5, (E, N)).astype(sdt)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    src = rng.integers(0, T, int(off[-1])).astype(np.int32) if rows else None
    return qx, qw, sx, sw, off, src


def _want(qx, qw, sx, sw, off, src, out, R):
    """out [R, N] fp32 before its conversion, NaN where no row is written."""
    want = np.full((R, qw.shape[1]), np.nan, np.float32)
    for e in range(qw.shape[0]):
        i, j = int(off[e]), int(off[e + 1])
        if j <= i:
            continue
        t = np.arange(i, j) if src is None else src[i:j]
        live = (t >= 0) & (t < qx.shape[0])
        t = t[live]
        acc = qx[t].astype(np.float64) @ qw[e].astype(np.float64).T
        assert np.abs(acc).max(initial=0) < 2 ** 31
        want[np.arange(i, j)[live]] = (acc.astype(np.int64).astype(np.float32) * sx[t].astype(np.float32)[:, None]
                                       * sw[e].astype(np.float32)[None])
    return want


def _run(gpu, case, bits, out_dtype, R, fill=-7.0, **kw):
    import torch
    qx, qw, sx, sw, off, src = case
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(gpu)  # noqa: E731
    odt = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}[out_dtype]
    out = torch.full((R, qw.shape[1]), fill, dtype=odt, device=gpu)
    wq = dev(_pack(qw.reshape(-1, qw.shape[2]), bits)).view(qw.shape[0], qw.shape[1], -1)
    B.grouped_gemm(dev(_pack(qx, bits)), dev(sx), wq, dev(sw), dev(off),
                   rows=None if src is None else dev(src), bits=bits, out_dtype=out_dtype, out=out, **kw)
    torch.cuda.synchronize()
    return out


def _same(out, want, fill=-7.0):
    import torch
    w = torch.from_numpy(want)
    w = torch.where(w.isnan(), torch.full_like(w, fill), w).to(out.dtype)
    got = out.cpu()
    bad = (got != w).nonzero()
    assert not len(bad), (len(bad), bad[0].tolist(), got[tuple(bad[0])], w[tuple(bad[0])])


COUNTS = {
    "one": [1], "decode": [1, 0, 3, 0, 0, 2, 1], "empty ends": [0, 5, 0], "tile": [16, 32, 64, 15, 17],
    "ragged": [70, 1, 0, 33, 130], "long": [300, 2, 513], "many": [i % 5 for i in range(200)],
}


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("name", COUNTS)
@pytest.mark.parametrize("N,K", [(1, 32), (52, 256), (33, 1056), (260, 544), (512, 2048)])
def test_ragged_groups(gpu, name, bits, N, K):
    counts = COUNTS[name]
    rng = np.random.default_rng(N + K + bits + len(counts))
    R = sum(counts) + 3  # three rows behind the last group: left as they were
    case = _case(rng, 41, K, len(counts), N, counts, bits, np.float16)
    src = np.concatenate([case[5], [0, 0, 0]]).astype(np.int32)
    case = (*case[:5], src)
    _same(_run(gpu, case, bits, "fp32", R), _want(*case, None, R))


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("out_dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("sdt", [np.float16, np.float32])
@pytest.mark.parametrize("counts", [[3, 0, 9], [300, 77, 512, 0, 1]])
def test_types(gpu, bits, out_dtype, sdt, counts):
    rng = np.random.default_rng(8)
    R = sum(counts)
    case = _case(rng, R, 640, len(counts), 390, counts, bits, sdt, rows=False)
    _same(_run(gpu, case, bits, out_dtype, R), _want(*case, None, R))


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("counts", [[5, 2], [257, 300]])
def test_largest_sums(gpu, bits, counts):
    """Every code the lowest one, at the longest K: the sums the int32 range has to hold."""
    rng = np.random.default_rng(1)
    case = _case(rng, 9, 65536, 2, 20, counts, bits, np.float32, extremes=True)
    _same(_run(gpu, case, bits, "fp32", sum(counts)), _want(*case, None, sum(counts)))


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("counts", [[4, 6, 3], [260, 300, 90]])
def test_padding_rows_and_repeated_rows(gpu, bits, counts):
    """Source rows outside xq are padding (their outputs stay), the same source row twice."""
    rng = np.random.default_rng(2)
    R = sum(counts)
    case = _case(rng, 12, 256, 3, 100, counts, bits, np.float32)
    src = case[5].copy()
    src[1], src[-1], src[counts[0]] = -1, 12, 2 ** 31 - 1
    src[3] = src[2]
    case = (*case[:5], src)
    _same(_run(gpu, case, bits, "bf16", R), _want(*case, None, R))


@pytest.mark.gpu
def test_offsets_out_of_range_stay_inside(gpu):
    """Ends outside 0 .. R count as the nearer end, a decrease as an empty group."""
    rng = np.random.default_rng(3)
    case = list(_case(rng, 8, 128, 4, 40, [2, 2, 2, 2], 8, np.float32))
    case[4] = np.array([-5, 3, 2, 2, 900], np.int32)
    clean = np.array([0, 3, 2, 2, 8], np.int32)
    want = _want(*case[:4], clean, case[5], None, 8)  # group 1: 3 .. 2 is empty
    out = _run(gpu, tuple(case), 8, "fp32", 8).cpu().numpy()
    assert np.array_equal(out[:2], want[:2]) and np.array_equal(out[3:], want[3:])


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("counts", [[3, 2], [280, 100]])
def test_strides(gpu, bits, counts):
    """Rows of codes, experts and outputs inside wider buffers."""
    import torch
    rng = np.random.default_rng(4)
    R, N, K = sum(counts), 70, 384
    qx, qw, sx, sw, off, src = _case(rng, R, K, 2, N, counts, bits, np.float16, rows=False)
    rb = K * bits // 8
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(gpu)  # noqa: E731
    xq = torch.full((R, rb + 48), 0x5A, dtype=torch.uint8, device=gpu)
    xq[:, :rb] = dev(_pack(qx, bits))
    wq = torch.full((2, N + 3, rb + 16), 0x5A, dtype=torch.uint8, device=gpu)
    wq[:, :N, :rb] = dev(_pack(qw.reshape(-1, K), bits)).view(2, N, rb)
    for odt in (torch.float32, torch.bfloat16):
        for lead in (1, 8):
            big = torch.full((R, N + 24), 3.0, dtype=odt, device=gpu)
            B.grouped_gemm(xq[:, :rb], dev(sx), wq[:, :N, :rb], dev(sw), dev(off), bits=bits,
                           out_dtype=odt, out=big[:, lead:lead + N])
            torch.cuda.synchronize()
            _same(big[:, lead:lead + N], _want(qx, qw, sx, sw, off, None, None, R))
            assert bool((big[:, :lead] == 3).all()) and bool((big[:, lead + N:] == 3).all())


def _counts(rng, E, mean):
    """Ragged groups around a mean, an empty one and a single row among them."""
    c = rng.integers(mean // 2, mean * 3 // 2, E)
    c[1], c[2] = 0, 1
    return [int(v) for v in c]


# One shape for each kernel and number of steps in LDS, by the rule that picks them: enough 256 x
# 256 tiles; 128 x 128 tiles, more than 256 of them and fewer; few rows over many groups; tiny N.
PICKED = {"tiles256": (16, 170, 2053), "tiles128": (40, 50, 1003), "few tiles128": (6, 60, 1500),
          "rows of decode": (30, 5, 3100), "stream": (9, 7, 700), "stream32": (3, 400, 70)}


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("out_dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("name", PICKED)
@pytest.mark.parametrize("K", [32, 512, 1056])
def test_every_kernel(gpu, name, K, out_dtype, bits):
    E, mean, N = PICKED[name]
    rng = np.random.default_rng(E + K + bits)
    counts = _counts(rng, E, mean)
    R = sum(counts) + 2
    case = _case(rng, 500, K, E, N, counts, bits, np.float16 if bits == 4 else np.float32)
    src = np.concatenate([case[5], [0, 0]]).astype(np.int32)
    src[::37] = -1  # padding rows
    case = (*case[:5], src)
    _same(_run(gpu, case, bits, out_dtype, R), _want(*case, None, R))


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("name", ["tiles256", "tiles128", "few tiles128", "stream"])
def test_every_kernel_largest_sums_and_odd_rows(gpu, name, bits):
    """The largest sums of a long K (the kernels' last step cut short), and outputs at odd
    addresses."""
    import torch
    E, mean, N = PICKED[name]
    rng = np.random.default_rng(E)
    counts = _counts(rng, E, mean)
    R, Kc = sum(counts), 16384 + 32
    qx, qw, sx, sw, off, src = _case(rng, 4, Kc, E, N, counts, bits, np.float32, extremes=True)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(gpu)  # noqa: E731
    big = torch.full((R, N + 3), 3.0, dtype=torch.bfloat16, device=gpu)
    wq = dev(_pack(qw.reshape(-1, Kc), bits)).view(E, N, -1)
    B.grouped_gemm(dev(_pack(qx, bits)), dev(sx), wq, dev(sw), dev(off), rows=dev(src), bits=bits,
                   out_dtype="bf16", out=big[:, 1:N + 1])
    torch.cuda.synchronize()
    lo = -8 if bits == 4 else -128
    e = np.repeat(np.arange(E), counts)  # every sum is the same: K lo^2
    want = np.float32(Kc * lo * lo) * sx[src][:, None] * sw[e]
    _same(big[:, 1:N + 1], want)
    assert bool((big[:, 0] == 3).all()) and bool((big[:, N + 1:] == 3).all())


@pytest.mark.gpu
def test_one_group_is_the_dense_product(gpu):
    """One group of all rows: kq_int4_gemm's result, bit for bit."""
    import torch
    g = torch.Generator().manual_seed(6)
    T, N, K = 300, 264, 1024
    xq = torch.randint(0, 256, (T, K // 2), generator=g, dtype=torch.uint8).to(gpu)
    wq = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8).to(gpu)
    sx, sw = torch.rand(T, generator=g).to(gpu), torch.rand(N, generator=g).to(gpu)
    off = torch.tensor([0, T], dtype=torch.int32, device=gpu)
    for dt in ("fp32", "bf16"):
        a = B.grouped_gemm(xq, sx, wq[None], sw[None], off, bits=4, out_dtype=dt)
        assert torch.equal(a, B.int4_gemm(xq, sx, wq, sw, dt))


@pytest.mark.gpu
@pytest.mark.slow
@pytest.mark.parametrize("counts", [[3, 0, 2], [200, 0, 300]])
def test_weights_past_four_gigabytes(gpu, counts):
    """Three experts of 2.2 GB each, of which the last is used: 64-bit offsets."""
    import torch
    N, K = 34000, 65536
    w = torch.randint(0, 256, (1, K), dtype=torch.uint8, generator=torch.Generator().manual_seed(1)).to(gpu)
    wq = torch.empty((3, N, K), dtype=torch.uint8, device=gpu)
    for e in range(3):
        wq[e] = w.roll(e, 1)
    wq[2, N - 1] = w[0].flip(0)
    x = torch.randint(0, 256, (4, K), dtype=torch.uint8, generator=torch.Generator().manual_seed(2)).to(gpu)
    R = sum(counts)
    rows = (torch.arange(R, device=gpu) % 4).to(torch.int32)
    off = torch.tensor([0, counts[0], counts[0], R], dtype=torch.int32, device=gpu)
    out = B.grouped_gemm(x, torch.ones(4, device=gpu), wq, torch.ones((3, N), device=gpu), off, rows=rows, bits=8)
    xs = x.view(torch.int8).double()[rows.long()]
    first = (xs[:counts[0]] * w[0].view(torch.int8).double()).sum(1)
    last = (xs[counts[0]:] * w[0].roll(2).view(torch.int8).double()).sum(1)
    end = (xs[counts[0]:] * w[0].flip(0).view(torch.int8).double()).sum(1)
    assert torch.equal(out[:counts[0]].double(), first.float().double()[:, None].expand(-1, N))
    assert torch.equal(out[counts[0]:, :-1].double(), last.float().double()[:, None].expand(-1, N - 1))
    assert torch.equal(out[counts[0]:, -1].double(), end.float().double())


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 8])
def test_another_stream_and_a_captured_call(gpu, bits):
    """A captured call follows the offsets and rows of each replay."""
    import torch
    rng = np.random.default_rng(5)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(gpu)  # noqa: E731
    sets = [[100, 0, 20, 7], [0, 127, 0, 0], [31, 32, 33, 31], [1, 1, 1, 124]]
    cases = [_case(rng, 50, 512, 4, 136, c, bits, np.float32) for c in sets]
    for c in cases[1:]:  # one weight, as a layer has
        c[1][:], c[3][:] = cases[0][1], cases[0][3]
    qw, sw = cases[0][1], cases[0][3]
    wq, swd = dev(_pack(qw.reshape(-1, 512), bits)).view(4, 136, -1), dev(sw)
    args = [(dev(_pack(c[0], bits)), dev(c[2]), dev(c[4]), dev(c[5])) for c in cases]
    buf = [a.clone() for a in args[0]]
    out = torch.empty((127, 136), dtype=torch.bfloat16, device=gpu)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    o = B.grouped_gemm(buf[0], buf[1], wq, swd, buf[2], rows=buf[3], bits=bits, out_dtype="bf16", stream=st)
    torch.cuda.synchronize()
    _same(o, _want(*cases[0], None, 127))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.grouped_gemm(buf[0], buf[1], wq, swd, buf[2], rows=buf[3], bits=bits, out_dtype="bf16", out=out)
    for i in (0, 1, 2, 3, 1):
        for b, a in zip(buf, args[i]):
            b.copy_(a)
        out.fill_(-7.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        _same(out, _want(*cases[i], None, 127))


# --------------------------------------------------------------------- refusals (no GPU)
def _raw(**kw):
    a = dict(xq=0x1000, ldxq=128, sx=0x2000, T=8, rows=0x3000, R=16, wq=0x4000, ldwq=128, ldwe=128 * 32,
             sw=0x5000, N=32, K=256, E=4, off=0x6000, bits=4, sd=B.KQ_FP16, od=B.KQ_BF16, out=0x7000, ldo=32)
    a.update(kw)
    return B.lib().kq_grouped_gemm(a["xq"], a["ldxq"], a["sx"], a["T"], a["rows"], a["R"], a["wq"], a["ldwq"],
                                   a["ldwe"], a["sw"], a["N"], a["K"], a["E"], a["off"], a["bits"], a["sd"],
                                   a["od"], a["out"], a["ldo"], None)


def test_refusals():
    assert _raw(R=0) == B.KQ_OK and _raw(N=0) == B.KQ_OK
    for kw in (dict(T=-1), dict(R=-1), dict(N=-1), dict(K=0), dict(E=0), dict(bits=5), dict(sd=B.KQ_BF16),
               dict(od=9), dict(rows=None, R=9), dict(xq=None), dict(sx=None), dict(wq=None), dict(sw=None),
               dict(off=None), dict(out=None), dict(T=0), dict(ldxq=112), dict(ldwq=112), dict(ldo=31),
               dict(ldwe=128 * 31 + 112), dict(bits=8)):
        assert _raw(**kw) == B.KQ_ERR_INVALID_ARG, kw
    for kw in (dict(K=258, ldxq=144, ldwq=144), dict(K=65536 + 256), dict(E=4097), dict(R=1 << 31),
               dict(T=1 << 31), dict(N=1 << 31, ldo=1 << 31), dict(ldwq=1 << 40), dict(ldwe=1 << 50),
               dict(K=24, bits=8)):
        assert _raw(**kw) == B.KQ_ERR_UNSUPPORTED, kw
    for kw in (dict(xq=0x1008), dict(wq=0x4004), dict(ldxq=136), dict(ldwq=136, ldwe=136 * 32), dict(ldwe=128 * 32 + 8),
               dict(sx=0x2001), dict(sw=0x5002, sd=B.KQ_FP32), dict(out=0x7001), dict(rows=0x3002),
               dict(off=0x6001)):
        assert _raw(**kw) == B.KQ_ERR_ALIGNMENT, kw


def test_host_tensors_are_refused():
    import torch
    z = torch.zeros
    with pytest.raises(ValueError):
        B.grouped_gemm(z((2, 16), dtype=torch.uint8), z(2), z((1, 4, 16), dtype=torch.uint8), z((1, 4)),
                       z(2, dtype=torch.int32))


@pytest.mark.gpu
def test_tensors_that_do_not_fit_are_refused(gpu):
    import torch
    u8, i32 = torch.uint8, torch.int32
    ok = dict(xq=torch.zeros((6, 32), dtype=u8, device=gpu), sx=torch.ones(6, device=gpu),
              wq=torch.zeros((2, 8, 32), dtype=u8, device=gpu), sw=torch.ones((2, 8), device=gpu),
              offsets=torch.tensor([0, 3, 6], dtype=i32, device=gpu))
    bad = [dict(xq=torch.zeros((6, 16), dtype=u8, device=gpu)), dict(sx=torch.ones(5, device=gpu)),
           dict(sx=torch.ones(6, dtype=torch.float16, device=gpu)), dict(sw=torch.ones((2, 7), device=gpu)),
           dict(offsets=torch.zeros(2, dtype=i32, device=gpu)), dict(offsets=torch.zeros(3, device=gpu)),
           dict(rows=torch.zeros(6, device=gpu)), dict(bits=3), dict(wq=ok["wq"].cpu()),
           dict(wq=ok["wq"][0]), dict(wq=ok["wq"][:1].expand(2, 8, 32)), dict(offsets=ok["offsets"].cpu()),
           dict(out=torch.empty((5, 8), device=gpu)), dict(out=torch.empty((6, 8), dtype=torch.float16, device=gpu))]
    for kw in bad:
        with pytest.raises(ValueError):
            B.grouped_gemm(**{**ok, "bits": 8, **kw})
    assert B.grouped_gemm(**ok, rows=torch.zeros(0, dtype=i32, device=gpu), bits=8).shape == (0, 8)


def test_outputs_over_inputs_are_refused():
    apart = dict(xq=0x10000, sx=0x20000, rows=0x30000, wq=0x40000, sw=0x50000, off=0x60000)
    for name, at in apart.items():
        assert _raw(**{**apart, "out": at}) == B.KQ_ERR_INVALID_ARG, name
    # the last value of 16 rows of 32 (0x400 bytes), the last weight of 4 experts (0x4000 bytes)
    assert _raw(**{**apart, "out": 0x20000 - 0x3fe}) == B.KQ_ERR_INVALID_ARG
    assert _raw(**{**apart, "out": 0x44000 - 2}) == B.KQ_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("mean", [2, 70, 300])
def test_decreasing_offsets_stay_inside(gpu, mean, bits):
    """Groups that overlap leave unspecified rows, but none outside the groups' range."""
    import torch
    rng = np.random.default_rng(mean + bits)
    E, R = 6, 6 * mean
    case = _case(rng, R, 512, E, 300, [mean] * E, bits, np.float32)
    off = np.array([mean, 4 * mean, 2 * mean, 5 * mean, 3 * mean, 3 * mean, 4 * mean], np.int32)
    out = _run(gpu, (*case[:4], off, case[5]), bits, "fp32", R).cpu()
    assert (out[:mean] == -7.0).all() and (out[5 * mean:] == -7.0).all()
    assert torch.isfinite(out).all()
