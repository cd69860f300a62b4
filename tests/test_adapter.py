"""kq_adapter_add: low-rank adapters of many requests beside a shared projection.

The reference is the formula in 64 bits: out = base + s B (A x). Bounds, with u = 2^-24 (half a
step of fp32), all sums of magnitudes M2 = |B| (|A| |x|) and Mh = |A| |x|:
- h = A x, K products in fp32 in some order: at most (K + 16) u Mh, then one rounding for s;
- the two 16-bit terms leave at most 2^-16 of the largest |h| of the token (fp16: the second
  term's smallest step, 2^-24 after the largest is brought to 2^14 or more, is far below it);
- B h, 2 r products in fp32: at most (2 r + 2) u (|B| |h|) <= (2 r + 2) u M2;
- the sum with base: one fp32 rounding; the output: eps / 2 of its type, relative.
So |out - ref| <= eps/2 |ref| + 2 ((K + 2 r + 20) u + 2^-16) M, where M also takes the largest
|h| for every rank. As the worst orders do not occur, a second bound is held on the norm: the
output's rounding (eps / 2) plus 1e-4 of the adapter's part."""
import pytest

from kronecker_factored_transforms_amd import binding as B


def _dt(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16}[name]


def _inputs(gpu, T, K, N, r, L, dtype, seed=0, adapter=None, gain=1.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    dt = _dt(dtype)
    x = torch.randn((T, K), generator=g).to(dt)
    A = (gain * torch.randn((L, r, K), generator=g) / K ** 0.5).to(dt)
    Bm = (torch.randn((L, N, r), generator=g) / r ** 0.5).to(dt)
    base = torch.randn((T, N), generator=g).to(dt)
    s = 0.25 + torch.rand(L, generator=g)
    if adapter is None:
        adapter = torch.randint(-1, L, (T,), generator=g)
    return [t.to(gpu) for t in (x, A, Bm, torch.as_tensor(adapter, dtype=torch.int32), base, s)]


def _check(x, A, Bm, ad, base, s, out):
    import torch
    T, K = x.shape
    L, N, r = Bm.shape
    eps = torch.finfo(out.dtype).eps
    ref = torch.zeros((T, N), dtype=torch.float64, device=x.device) if base is None else base.double()
    mag = torch.zeros_like(ref)
    part = torch.zeros_like(ref)
    for a in range(L):
        at = (ad == a).nonzero()[:, 0]
        if not at.numel():
            continue
        h = x[at].double() @ A[a].double().t()
        mh = x[at].double().abs() @ A[a].double().abs().t()
        k = 1.0 if s is None else float(s[a])
        part[at] = k * (h @ Bm[a].double().t())
        m2 = mh @ Bm[a].double().abs().t()
        top = h.abs().amax(1, keepdim=True) * Bm[a].double().abs().sum(1)[None]
        mag[at] = abs(k) * ((K + 2 * r + 20) * 2.0 ** -24 * m2 + 2.0 ** -16 * top)
    ref = ref + part
    none = (ad < 0) | (ad >= L)
    if base is not None:
        assert torch.equal(out[none], base[none])
    else:
        assert not out[none].any()
    err = (out.double() - ref).abs()
    tiny = torch.finfo(out.dtype).smallest_normal * eps / 2
    bound = eps / 2 * ref.abs() * (1 + 2 ** -6) + 2 * mag + tiny
    assert bool((err <= bound).all()), (float((err - bound).max()), (err > bound).sum().item())
    # each output's conversion is off by eps / 2 |ref| or, below the type's normal range, by half
    # its smallest step (fp16: 2^-25): over n outputs eps / 2 ||ref|| + sqrt(n) 2^-25 in norm
    assert float(err.norm()) <= eps / 2 * float(ref.norm()) + 1e-4 * float(part.norm()) + tiny * err.numel() ** 0.5


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("r", [8, 16, 24, 32, 40, 64, 104, 128, 200, 256])
@pytest.mark.parametrize("T", [1, 16, 37])
def test_ranks_and_tokens(gpu, dtype, r, T):
    a = _inputs(gpu, T, 520, 264, r, 5, dtype, seed=r + T)
    _check(*a, B.adapter_add(*a[:4], base=a[4], scaling=a[5]))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,K,N,r,L", [(1, 8, 8, 8, 1), (5, 8192, 16, 16, 3), (64, 4096, 4096, 16, 64),
                                       (333, 1000, 1096, 40, 7), (3, 16, 5000, 128, 2), (700, 2048, 512, 64, 2),
                                       (2000, 1024, 776, 16, 3), (17, 11008, 4096, 32, 9)])
def test_shapes(gpu, dtype, T, K, N, r, L):
    a = _inputs(gpu, T, K, N, r, L, dtype, seed=T + K)
    _check(*a, B.adapter_add(*a[:4], base=a[4], scaling=a[5]))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("r", [8, 16, 32, 56, 64, 120, 128, 256])
@pytest.mark.parametrize("T", [1024, 1337, 4096, 4133])
def test_many_tokens(gpu, T, r, dtype):
    """The two ways of many tokens (parts joined in between; K whole), prompts whose ends fall
    inside tiles of 16 and 32."""
    import torch
    seg = torch.arange(T) // 205 % 5 - 1
    a = _inputs(gpu, T, 328, 200, r, 4, dtype, seed=r + T, adapter=seg)
    _check(*a, B.adapter_add(*a[:4], base=a[4], scaling=a[5]))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,gain", [("bf16", 1.0), ("fp16", 1e-5), ("fp16", 200.0)])
@pytest.mark.parametrize("T", [1500, 5000])
def test_many_tokens_in_any_order(gpu, T, dtype, gain):
    """Every adapter in every tile, K past one step per wave, h of any size."""
    a = _inputs(gpu, T, 2056, 136, 24, 19, dtype, seed=T, gain=gain)
    _check(*a, B.adapter_add(*a[:4], base=a[4], scaling=a[5]))
    base = a[4].clone()
    out = B.adapter_add(*a[:4], base=base, scaling=a[5], out=base)
    _check(*a, out)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [40, 900, 1100, 4200])
def test_orders_of_adapters(gpu, T):
    """All tokens on one adapter, none on any, every token another, and segments whose ends
    fall inside tiles; numbers outside 0 .. L-1 name none."""
    import torch
    L = 48
    seg = torch.arange(T) // 13 % L
    seg[::29] = -1
    orders = [torch.zeros(T), torch.full((T,), -1), torch.arange(T) % L, seg,
              torch.where(torch.arange(T) % 2 == 0, 2 ** 31 - 1, 5), torch.full((T,), L),
              torch.full((T,), -2 ** 31)]
    for i, o in enumerate(orders):
        a = _inputs(gpu, T, 768, 392, 16, L, "bf16", seed=i, adapter=o)
        _check(*a, B.adapter_add(*a[:4], base=a[4], scaling=a[5]))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("gain", [1e-6, 1e-3, 300.0])
def test_sizes_of_the_low_rank_vector(gpu, dtype, gain):
    """h far below and above fp16's comfortable range: the two terms keep their bits."""
    a = _inputs(gpu, 50, 640, 256, 32, 4, dtype, seed=3, gain=gain)
    _check(*a[:4], None, a[5], B.adapter_add(*a[:4], scaling=a[5]))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [30, 600])
def test_no_base_no_scaling_and_in_place(gpu, T):
    import torch
    x, A, Bm, ad, base, s = _inputs(gpu, T, 512, 328, 16, 3, "bf16", seed=4)
    _check(x, A, Bm, ad, base, None, B.adapter_add(x, A, Bm, ad, base=base))
    _check(x, A, Bm, ad, None, s, B.adapter_add(x, A, Bm, ad, scaling=s))
    want = B.adapter_add(x, A, Bm, ad, base=base, scaling=s)
    b = base.clone()
    assert B.adapter_add(x, A, Bm, ad, base=b, scaling=s, out=b) is b
    assert torch.equal(b, want)
    again = B.adapter_add(x, A, Bm, ad, base=base, scaling=s)
    assert torch.equal(again, want)  # no order that changes


@pytest.mark.gpu
@pytest.mark.parametrize("T", [20, 500, 1200, 4111])
def test_strides(gpu, T):
    import torch
    x, A, Bm, ad, base, s = _inputs(gpu, T, 264, 136, 24, 3, "fp16", seed=5)
    xw = torch.full((T, 264 + 16), float("nan"), dtype=x.dtype, device=gpu)
    xw[:, 8:272] = x
    bw = torch.full((T, 136 + 24), 9.0, dtype=x.dtype, device=gpu)
    bw[:, 16:152] = base
    want = B.adapter_add(x, A, Bm, ad, base=base, scaling=s)
    out = torch.full((T, 160), 5.0, dtype=x.dtype, device=gpu)
    B.adapter_add(xw[:, 8:272], A, Bm, ad, base=bw[:, 16:152], scaling=s, out=out[:, 8:144])
    assert torch.equal(out[:, 8:144], want)
    assert bool((out[:, :8] == 5).all()) and bool((out[:, 144:] == 5).all())
    B.adapter_add(xw[:, 8:272], A, Bm, ad, base=bw[:, 16:152], scaling=s, out=bw[:, 16:152])
    assert torch.equal(bw[:, 16:152], want) and bool((bw[:, :16] == 9).all()) and bool((bw[:, 152:] == 9).all())


@pytest.mark.gpu
@pytest.mark.parametrize("T", [16, 48, 800, 1030, 4100])
def test_what_is_not_finite_stays_with_its_own_tokens(gpu, T):
    """NaN and infinities in one adapter, and in one token's row, reach no other token."""
    import torch
    x, A, Bm, ad, base, s = _inputs(gpu, T, 256, 136, 16, 4, "bf16", seed=6, adapter=torch.arange(T) % 4)
    want = B.adapter_add(x, A, Bm, ad, base=base, scaling=s)
    A2, B2, x2, s2 = A.clone(), Bm.clone(), x.clone(), s.clone()
    A2[1, 3, 7] = float("nan")
    A2[1, 4] = float("inf")
    B2[2, 5] = float("nan")
    B2[2, 6] = float("-inf")
    s2[1] = float("inf")
    x2[3] = float("nan")
    out = B.adapter_add(x2, A2, B2, ad, base=base, scaling=s2)
    ok = (ad == 0) | ((ad == 3) & (torch.arange(T, device=gpu) != 3))
    assert torch.equal(out[ok], want[ok])
    two = ad == 2
    cols = torch.ones(136, dtype=torch.bool, device=gpu)
    cols[5:7] = False
    assert torch.equal(out[two][:, cols], want[two][:, cols])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [70, 1025, 4097])
def test_another_stream_and_captured_calls(gpu, T):
    """Two graphs in turn, each with a workspace of its own, follow the adapters of each replay."""
    import torch
    L = 6
    sets = [_inputs(gpu, T, 512, 264, 16, L, "bf16", seed=i) for i in range(4)]
    x, A, Bm, ad, base, s = sets[0]
    want = [B.adapter_add(t[0], A, Bm, t[3], base=t[4], scaling=s) for t in sets]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    o = B.adapter_add(x, A, Bm, ad, base=base, scaling=s, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(o, want[0])
    bufs, outs, graphs = [], [], []
    for _ in range(2):
        xi, ai, bi = x.clone(), ad.clone(), base.clone()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(B.adapter_add(xi, A, Bm, ai, base=bi, scaling=s))
        bufs.append((xi, ai, bi))
        graphs.append(g)
    for i in range(4):
        for k in range(2):
            t = sets[(i + k) % 4]
            for b, v in zip(bufs[k], (t[0], t[3], t[4])):
                b.copy_(v)
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for k in range(2):
            assert torch.equal(outs[k], want[(i + k) % 4])


@pytest.mark.gpu
@pytest.mark.slow
def test_adapters_past_four_gigabytes(gpu):
    """Adapters whose matrices lie beyond 2^32 bytes."""
    import torch
    L, r, K, N = 1100, 256, 8192, 64
    A = torch.zeros((L, r, K), dtype=torch.bfloat16, device=gpu)  # 4.6 GB
    x, A0, B0, _, base, _ = _inputs(gpu, 20, K, N, r, 2, "bf16", seed=7)
    A[0], A[L - 1] = A0[0], A0[1]
    Bm = torch.zeros((L, N, r), dtype=torch.bfloat16, device=gpu)
    Bm[0], Bm[L - 1] = B0[0], B0[1]
    ad = torch.tensor([0, L - 1] * 10, dtype=torch.int32, device=gpu)
    small = B.adapter_add(x, A0, B0, torch.tensor([0, 1] * 10, dtype=torch.int32, device=gpu), base=base)
    assert torch.equal(B.adapter_add(x, A, Bm, ad, base=base), small)


# --------------------------------------------------------------------- refusals (no GPU)
def _raw(**kw):
    a = dict(x=0x10000, ldx=64, A=0x20000, B=0x30000, ad=0x40000, s=0x50000, base=0x60000, ldb=32, T=4, K=64,
             N=32, r=16, L=2, dt=B.KQ_BF16, out=0x70000, ldo=32, ws=0x80000, wsb=1 << 20)
    a.update(kw)
    return B.lib().kq_adapter_add(a["x"], a["ldx"], a["A"], a["B"], a["ad"], a["s"], a["base"], a["ldb"], a["T"],
                                  a["K"], a["N"], a["r"], a["L"], a["dt"], a["out"], a["ldo"], a["ws"], a["wsb"],
                                  None)


def test_refusals():
    assert _raw(T=0) == B.KQ_OK and _raw(N=0) == B.KQ_OK
    for kw in (dict(T=-1), dict(K=0), dict(N=-8), dict(r=0), dict(L=0), dict(dt=B.KQ_FP32), dict(x=None),
               dict(A=None), dict(B=None), dict(ad=None), dict(out=None), dict(ldx=56), dict(ldb=24),
               dict(ldo=24), dict(out=0x10000), dict(out=0x60010), dict(out=0x60000, ldo=64), dict(out=0x30000),
               dict(out=0x20000)):
        assert _raw(**kw) == B.KQ_ERR_INVALID_ARG, kw
    for kw in (dict(K=60), dict(N=36, ldb=40, ldo=40), dict(r=12), dict(r=264), dict(K=(1 << 20) + 8),
               dict(N=(1 << 20) + 8), dict(T=(1 << 27) + 1), dict(ldx=1 << 40)):
        assert _raw(**kw) == B.KQ_ERR_UNSUPPORTED, kw
    for kw in (dict(x=0x10008), dict(A=0x20002), dict(B=0x30008), dict(ad=0x40002), dict(s=0x50001),
               dict(base=0x60008), dict(out=0x70008), dict(ldx=68), dict(ldb=36), dict(ldo=36), dict(ws=0x80010)):
        assert _raw(**kw) == B.KQ_ERR_ALIGNMENT, kw
    need = B.kq_adapter_workspace_size(4, 64, 16)
    assert need >= 4 * 16 * 4 and need % 256 == 0
    assert _raw(ws=None) == B.KQ_ERR_WORKSPACE and _raw(wsb=need - 1) == B.KQ_ERR_WORKSPACE
    assert B.kq_adapter_workspace_size(0, 64, 16) == 0
    for T, K, r in ((-1, 64, 16), (4, 0, 16), (4, 64, 0), (4, 60, 16), (4, 64, 512)):
        with pytest.raises(B.KqError):
            B.kq_adapter_workspace_size(T, K, r)


def test_host_tensors_are_refused():
    import torch
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ValueError):
        B.adapter_add(z(2, 16), z(1, 8, 16), z(1, 8, 8), torch.zeros(2, dtype=torch.int32))


@pytest.mark.gpu
def test_tensors_that_do_not_fit_are_refused(gpu):
    import torch
    x, A, Bm, ad, base, s = _inputs(gpu, 6, 64, 32, 16, 3, "bf16")
    ok = dict(x=x, A=A, B=Bm, adapter=ad, base=base, scaling=s)
    bad = [dict(x=x.float()), dict(A=A[:, :, :56]), dict(A=A.half()), dict(B=Bm[:2]), dict(B=Bm.transpose(1, 2)),
           dict(adapter=ad.long()), dict(adapter=ad[:5]), dict(base=base[:, :24]), dict(base=base.half()),
           dict(scaling=s.half()), dict(scaling=s[:2]), dict(out=torch.empty((6, 24), dtype=x.dtype, device=gpu)),
           dict(workspace=torch.empty(16, dtype=torch.uint8, device=gpu)), dict(x=x.cpu()), dict(adapter=ad.cpu()),
           dict(base=base[:1].expand(6, 32))]
    for kw in bad:
        with pytest.raises(ValueError):
            B.adapter_add(**{**ok, **kw})
    assert B.adapter_add(x[:0], A, Bm, ad[:0], base=base[:0]).shape == (0, 32)


def test_workspace_over_other_arguments_is_refused():
    for at in (0x10000, 0x20000, 0x30000, 0x40000, 0x50000, 0x60000, 0x70000):
        assert _raw(ws=at) == B.KQ_ERR_INVALID_ARG, hex(at)
    # 4 tokens of 16 ranks in fp32, one part: 0x100 bytes, so its last 16 are the first of out
    assert _raw(ws=0x80000 - 0x100, out=0x80000 - 0x10) == B.KQ_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,K,N,r,L", [(1, 64, 8, 8, 1), (1, 4096, 4096, 32, 64), (1, 8, 32768, 16, 2),
                                       (1, 8, 32776, 16, 2), (4, 1032, 1000, 8, 9), (16, 2040, 136, 16, 4),
                                       (16, 1000, 264, 32, 4), (3, 4104, 72, 8, 3), (16, 8192, 520, 8, 2),
                                       (16, 1016, 136, 16, 4), (16, 512, 264, 32, 4), (2, 2048, 72, 16, 3)])
def test_few_tokens(gpu, T, K, N, r, L, dtype):
    for seed in range(2):
        x, A, Bm, ad, base, s = _inputs(gpu, T, K, N, r, L, dtype, seed=seed)
        _check(x, A, Bm, ad, base, s, B.adapter_add(x, A, Bm, ad, base=base, scaling=s))
        none = ad.clone()
        none[::2] = -1
        _check(x, A, Bm, none, base, s, B.adapter_add(x, A, Bm, none, base=base, scaling=s, out=base.clone()))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 5, 16])
def test_few_tokens_that_are_not_finite(gpu, T):
    """Infinities and NaN of one token, of one adapter, stay with the tokens that have them."""
    import torch
    x, A, Bm, ad, base, s = _inputs(gpu, T, 512, 264, 16, 4, "bf16", seed=T)
    ad.copy_(torch.arange(T, device=ad.device) % 4 - 1)
    want = B.adapter_add(x, A, Bm, ad, base=base, scaling=s)
    A[2, 3, 7], Bm[2, 5, 1] = float("inf"), float("nan")
    x2 = x.clone()
    x2[T // 2, 9] = float("nan")
    out = B.adapter_add(x2, A, Bm, ad, base=base, scaling=s)
    touched = (ad == 2) | ((torch.arange(T, device=ad.device) == T // 2) & (ad >= 0))
    assert torch.equal(out[~touched], want[~touched])
    assert not torch.isfinite(out[touched]).all(1).any()


@pytest.mark.gpu
def test_few_tokens_in_a_graph(gpu):
    import torch
    x, A, Bm, ad, base, s = _inputs(gpu, 4, 1024, 1024, 16, 4, "fp16", seed=9)
    out = torch.empty_like(base)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        B.adapter_add(x, A, Bm, ad, base=base, scaling=s, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.adapter_add(x, A, Bm, ad, base=base, scaling=s, out=out)
    for k in range(4):
        x.copy_(torch.randn_like(x))
        ad.copy_((ad + k) % 5 - 1)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        _check(x, A, Bm, ad, base, s, got)
        assert torch.equal(got, B.adapter_add(x, A, Bm, ad, base=base, scaling=s))
