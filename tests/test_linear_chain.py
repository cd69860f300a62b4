"""The operators around a linear layer as they are used together: the norm in front of it (INT8
codes for W8A8 experts, normed rows for the transform plan of a W4A4 projection), the products,
and the adapters beside the projection. Each step is checked against the oracle or the formula on
the step's own inputs, and the whole chain is captured into one graph and replayed."""
import numpy as np
import pytest

import kqtest as K
from kronecker_factored_transforms_amd import binding as B
from kronecker_factored_transforms_amd import synth as S
from oracle import kq_oracle as O

pytestmark = pytest.mark.gpu


def _layer(gpu, T, seed=3):
    import torch
    g = torch.Generator().manual_seed(seed)
    n, N, E, top, F, L, r = 4096, 512, 6, 2, 392, 3, 16
    inp = S.make("attn_n4096", T=4)
    _, P1, P2, _ = K.device_inputs(inp, gpu)
    bf = torch.bfloat16
    w = dict(
        norm=(1 + 0.1 * torch.randn(n, generator=g)).to(bf).to(gpu),
        plan=B.Plan(P1, P2, None, 3.0),
        wplan=B.Plan(B.weight_factor(P1), B.weight_factor(P2), None, float("inf")),
        proj=(torch.randn((N, n), generator=g) / n ** 0.5).to(bf).to(gpu),
        eq=torch.randint(0, 256, (E, F, n), generator=g, dtype=torch.uint8).to(gpu),
        es=(0.001 + 0.001 * torch.rand((E, F), generator=g)).half().to(gpu),
        A=(torch.randn((L, r, n), generator=g) / n ** 0.5).to(bf).to(gpu),
        Bm=(torch.randn((L, N, r), generator=g) / r ** 0.5).to(bf).to(gpu),
        sc=torch.rand(L, generator=g).to(gpu))
    w["wq"], w["ws"] = w["wplan"](w["proj"])

    def batch(seed):
        g = torch.Generator().manual_seed(seed)
        expert = torch.rand((T, E), generator=g).topk(top, 1).indices.reshape(-1)
        order = torch.argsort(expert, stable=True)
        off = torch.cat([torch.zeros(1, dtype=torch.int64), torch.bincount(expert, minlength=E).cumsum(0)])
        return [t.to(gpu) for t in (torch.randn((T, n), generator=g).to(bf), torch.randn((T, n), generator=g).to(bf),
                                    (order // top).int(), off.int(), torch.randint(-1, L, (T,), generator=g).int())]

    def run(x, res, rows, off, ad):
        o = B.rmsnorm_quant(x, w["norm"], residual=res, alpha=4.0, normed=True)
        experts = B.grouped_gemm(o.codes, o.scales, w["eq"], w["es"], off, rows=rows, bits=8, out_dtype="bf16")
        xq, xs = w["plan"](o.normed)
        base = B.int4_gemm(xq, xs, w["wq"], w["ws"], "bf16")
        out = B.adapter_add(o.normed, w["A"], w["Bm"], ad, base=base, scaling=w["sc"])
        return dict(o=o, experts=experts, xq=xq, xs=xs, base=base, out=out)
    return w, batch, run


@pytest.mark.parametrize("T", [1, 37, 300])
def test_each_step_of_the_chain(gpu, T):
    import torch
    w, batch, run = _layer(gpu, T)
    x, res, rows, off, ad = batch(1)
    y = run(x, res, rows, off, ad)
    torch.cuda.synchronize()
    o = y["o"]
    assert torch.equal(o.residual, (x.float() + res.float()).bfloat16())
    # the experts' product of the call's own codes, bit for bit
    q, s = o.codes.cpu().numpy().view(np.int8), o.scales.cpu().numpy().astype(np.float32)
    src, ends = rows.cpu().numpy(), off.cpu().numpy()
    for e in range(w["eq"].shape[0]):
        t = src[ends[e]:ends[e + 1]]
        acc = q[t].astype(np.int64) @ w["eq"][e].cpu().numpy().view(np.int8).astype(np.int64).T
        want = acc.astype(np.float32) * s[t][:, None] * w["es"][e].float().cpu().numpy()[None]
        assert torch.equal(y["experts"][ends[e]:ends[e + 1]].cpu(), torch.from_numpy(want).bfloat16()), e
    # the projection of the call's own codes, bit for bit
    want = O.int4_gemm(y["xq"].cpu().numpy(), K.np_scales(y["xs"]), w["wq"].cpu().numpy(), K.np_scales(w["ws"]))
    assert torch.equal(y["base"].cpu(), torch.from_numpy(want).bfloat16())
    # the adapters on the projection's rows: half a bf16 step of the 64-bit formula, and 2^-12 of
    # the adapter's part for its sums (4096 products, 2^-24 each in the worst order)
    xn, ref = o.normed.double(), y["base"].double()
    part = torch.zeros_like(ref)
    for a in range(3):
        at = ad == a
        part[at] = float(w["sc"][a]) * ((xn[at] @ w["A"][a].double().t()) @ w["Bm"][a].double().t())
    err = (y["out"].double() - (ref + part)).abs()
    assert bool((err <= 2.0 ** -8 * (1 + 2 ** -6) * (ref + part).abs() + 2.0 ** -12 * part.abs().amax()).all())
    assert torch.equal(y["out"][ad < 0], y["base"][ad < 0])


def test_the_chain_in_one_graph(gpu):
    import torch
    w, batch, run = _layer(gpu, 50)
    sets = [batch(i) for i in range(4)]
    want = [run(*s) for s in sets]
    torch.cuda.synchronize()
    bufs = [t.clone() for t in sets[0]]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = run(*bufs)
    for i in (0, 1, 2, 3, 1):
        for b, t in zip(bufs, sets[i]):
            b.copy_(t)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for k in ("experts", "base", "out", "xq"):
            assert torch.equal(y[k], want[i][k]), (i, k)
        assert torch.equal(y["o"].codes, want[i]["o"].codes)
