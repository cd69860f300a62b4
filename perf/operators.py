"""The operators around a quantized linear layer, as they are measured.

Three operators stand beside the fused transform and its INT4 product:

- "norm": the residual's addition, the root-mean-square norm and INT8 codes with a step per
  token (optionally the normed row too, which a transform plan then takes);
- "experts": products of INT4 or INT8 codes grouped by expert, with ragged sizes;
- "adapters": low-rank adapters of many requests at once, beside a shared projection.

`run` computes each in plain torch operations, or, where `own` is true, by the framework's
calls. Codes are returned as the values they stand for (code times step).
"""
import math

import torch

own = False

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-5


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # the norm in front of a layer for one token being generated: latency
        dict(name="norm_token", op="norm", T=1, n=4096, dtype="bf16", step="fp16", residual=True,
             normed=False, alpha=math.inf, pad=0),
        # a long prompt (or a full batch of them) at hidden size 8192
        dict(name="norm_prompt", op="norm", T=16384, n=8192, dtype="bf16", step="fp16", residual=True,
             normed=False, alpha=3.0, pad=0),
        # the norm of a layer that also feeds a transform plan: codes and normed rows, ragged batch
        dict(name="norm_both", op="norm", T=1001, n=7168, dtype="fp16", step="fp16", residual=True,
             normed=True, alpha=math.inf, pad=8),
        # fp32 rows of an odd length inside wider ones, no residual: calibration
        dict(name="norm_odd", op="norm", T=777, n=5121, dtype="fp32", step="fp32", residual=False,
             normed=True, alpha=2.0, pad=3),
        # one token through two of eight experts: the weights' stream, latency
        dict(name="experts_token", op="experts", bits=8, T=1, top=2, E=8, N=4096, K=4096, step="fp16",
             out="bf16"),
        # a decode batch over many experts, a few rows each: every expert's weights once
        dict(name="experts_decode", op="experts", bits=4, T=64, top=4, E=64, N=4096, K=7168,
             step="fp16", out="bf16"),
        # a short prompt over sixteen experts, about 190 ragged rows each, W8A8, fp32 out
        dict(name="experts_ragged", op="experts", bits=8, T=1531, top=2, E=16, N=11008, K=4096,
             step="fp32", out="fp32"),
        # a prefill over eight experts, up projection, W4A4: bound by the matrix cores
        dict(name="experts_prompt", op="experts", bits=4, T=8192, top=2, E=8, N=14336, K=4096,
             step="fp16", out="bf16"),
        # one token of one request beside a 4096 x 4096 projection: latency
        dict(name="adapters_token", op="adapters", T=1, requests=1, L=4, r=16, K=4096, N=4096,
             dtype="bf16"),
        # a decode batch whose requests use 32 adapters in any order, some none
        dict(name="adapters_decode", op="adapters", T=128, requests=128, L=32, r=16, K=8192, N=8192,
             dtype="bf16"),
        # prompts of six requests, ranks of 64, up projection: the output's read and write
        dict(name="adapters_prompt", op="adapters", T=8192, requests=6, L=8, r=64, K=4096, N=14336,
             dtype="bf16"),
        # a mixed batch (prompts and single tokens), fp16, a rank and widths off the tiles
        dict(name="adapters_mixed", op="adapters", T=777, requests=40, L=12, r=40, K=7168, N=2120,
             dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["norm", "experts", "adapters"])
    if op == "norm":
        T, n = _log(rng, 1, 16384), _log(rng, 64, 16384)
        if rng.random() < 0.6:
            n = -(-n // 8) * 8
        T = min(T, (1 << 27) // n)
        return dict(op=op, T=T, n=n, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    step=rng.choice(["fp16", "fp32"]), residual=rng.random() < 0.7,
                    normed=rng.random() < 0.4, alpha=rng.choice([math.inf, 2.0, 4.0]),
                    pad=rng.choice([0, 0, 8, 5]))
    if op == "experts":
        bits = rng.choice([4, 8])
        E = _log(rng, 2, 128)
        top = min(E, rng.choice([1, 2, 4, 6]))
        T = _log(rng, 1, 8192)
        K, N = _log(rng, 256, 14336) // 32 * 32, _log(rng, 64, 14336)
        if rng.random() < 0.7:
            N = -(-N // 8) * 8
        while E * N * K * bits > 1 << 32 or T * top * N * K > 10**12:
            E, T, N = max(2, E * 3 // 4), max(1, T * 3 // 4), max(64, N * 3 // 4 // 8 * 8)
            top = min(E, top)
        return dict(op=op, bits=bits, T=T, top=top, E=E, N=N, K=K, step=rng.choice(["fp16", "fp32"]),
                    out=rng.choice(["bf16", "fp16", "fp32"]))
    T, L, r = _log(rng, 1, 8192), _log(rng, 1, 64), 8 * rng.randint(1, 16)
    requests = _log(rng, 1, T)
    K, N = 8 * _log(rng, 32, 1792), 8 * _log(rng, 32, 1792)
    while T * L * r * (K + N) > 7 * 10**10:
        T, L = max(1, T * 3 // 4), max(1, L * 3 // 4)
        requests = min(requests, T)
    return dict(op=op, T=T, requests=requests, L=L, r=r, K=K, N=N, dtype=rng.choice(["bf16", "fp16"]))


# ----------------------------------------------------------------------------- inputs
def _rows(g, T, n, dtype, pad):
    """T rows of n values inside rows of n + pad, as a slice of a wider activation is."""
    return torch.randn((T, n + pad), generator=g, device=DEV).to(dtype)[:, :n]


def _codes(g, shape, bits):
    """Packed codes of normal values quantized by their largest magnitude (about 4 deviations):
    two INT4 codes to a byte, the even one in the low nibble, or one INT8 code."""
    if bits == 8:
        out = torch.empty(shape, dtype=torch.int8, device=DEV)
        for part in out.view(-1).split(1 << 27):
            part.copy_(torch.randn(part.shape, generator=g, device=DEV).mul_(32).round_().clamp_(-128, 127))
        return out.view(torch.uint8)
    lo = torch.empty((*shape[:-1], shape[-1] // 2), dtype=torch.uint8, device=DEV)
    for part in lo.view(-1).split(1 << 27):
        q = [torch.randn(part.shape, generator=g, device=DEV).mul_(1.8).round_().clamp_(-8, 7).to(torch.int16)
             for _ in range(2)]
        part.copy_((q[0] & 15) | ((q[1] & 15) << 4))
    return lo


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] == "norm":
        dt = TYPES[case["dtype"]]
        x = _rows(g, case["T"], case["n"], dt, case["pad"])
        # a few channels of a residual stream are far larger than the others
        r = _rows(g, case["T"], case["n"], dt, case["pad"]) if case["residual"] else None
        if r is not None:
            r[:, :: max(1, case["n"] // 4)] *= 30
        w = (1 + 0.2 * torch.randn(case["n"], generator=g, device=DEV)).to(dt)
        values = torch.empty((case["T"], case["n"]), dtype=torch.bfloat16 if case["step"] == "fp32" else torch.float16,
                             device=DEV)
        s.update(x=x, r=r, w=w, values=values)
    elif case["op"] == "experts":
        T, E, top, N, K, bits = (case[k] for k in ("T", "E", "top", "N", "K", "bits"))
        sdt = TYPES[case["step"]]
        s["xq"], s["wq"] = _codes(g, (T, K), bits), _codes(g, (E, N, K), bits)
        s["sx"] = (0.02 + 0.03 * torch.rand(T, generator=g, device=DEV)).to(sdt)
        s["sw"] = (0.002 + 0.002 * torch.rand((E, N), generator=g, device=DEV)).to(sdt)
        # routing: some experts are more popular than others; rows sorted by expert
        logits = torch.randn((T, E), generator=g, device=DEV) + 0.5 * torch.randn(E, generator=g, device=DEV)
        expert = logits.topk(top, dim=1).indices.reshape(-1)
        order = torch.argsort(expert, stable=True)
        counts = torch.bincount(expert, minlength=E)
        s["rows"] = (order // top).to(torch.int32)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["most"] = int(counts.max())
    else:
        T, L, r, K, N = (case[k] for k in ("T", "L", "r", "K", "N"))
        dt = TYPES[case["dtype"]]
        s["x"] = torch.randn((T, K), generator=g, device=DEV).to(dt)
        s["A"] = (torch.randn((L, r, K), generator=g, device=DEV) / math.sqrt(K)).to(dt)
        s["B"] = (torch.randn((L, N, r), generator=g, device=DEV) / math.sqrt(r)).to(dt)
        s["scaling"] = 0.5 + torch.rand(L, generator=g, device=DEV)
        s["base"] = torch.randn((T, N), generator=g, device=DEV).to(dt)
        # each request's tokens stand together; about one request in nine has no adapter
        which = torch.randint(0, L, (case["requests"],), generator=g, device=DEV)
        which[torch.rand(case["requests"], generator=g, device=DEV) < 0.11] = -1
        cuts = torch.randint(0, case["requests"], (T,), generator=g, device=DEV).sort().values
        s["adapter"] = which[cuts].to(torch.int32)
    return s


# -------------------------------------------------------------------------- one pass
def _plain_norm(s):
    h = s["x"].float() if s["r"] is None else s["x"].float() + s["r"].float()
    rstd = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS)
    y = h * s["w"].float() * rstd
    clip = 1 / (1 + math.exp(-s["alpha"]))
    step = (clip * y.abs().amax(-1, keepdim=True) / 127).to(TYPES[s["step"]])
    inv = torch.where(step > 0, 1 / step.float(), torch.zeros_like(y[:, :1]))
    q = (y * inv).round().clamp(-128, 127)
    s["values"].copy_(q * step.float())
    return dict(values=s["values"], scales=step[:, 0],
                residual=None if s["r"] is None else h.to(s["x"].dtype),
                normed=y.to(s["x"].dtype) if s["normed"] else None)


def _numbers(codes, bits):
    """The codes as fp32 numbers."""
    if bits == 8:
        return codes.view(torch.int8).float()
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    return ((q ^ 8).to(torch.int8) - 8).float()


def _plain_experts(s):
    # every group padded to the longest one, and one batched product
    R, E = s["rows"].numel(), s["E"]
    at = torch.arange(R, device=DEV, dtype=torch.int32)
    e = torch.searchsorted(s["offsets"], at, right=True) - 1
    place = at - s["offsets"][e]
    x = _numbers(s["xq"], s["bits"])[s["rows"]]
    padded = x.new_zeros((E, s["most"], s["K"]))
    padded[e, place] = x
    prod = torch.bmm(padded, _numbers(s["wq"], s["bits"]).transpose(1, 2).contiguous())
    out = prod[e, place] * s["sx"].float()[s["rows"], None] * s["sw"].float()[e]
    return out.to(TYPES[s["out"]])


def _plain_adapters(s):
    # all adapters' products, those that are not a token's own masked out between the two
    L, r, K, N = s["L"], s["r"], s["K"], s["N"]
    h = (s["x"].float() @ s["A"].float().view(L * r, K).t()).view(-1, L, r)
    mine = s["adapter"][:, None] == torch.arange(L, device=DEV, dtype=torch.int32)
    h = h * (mine * s["scaling"])[:, :, None]
    d = h.reshape(-1, L * r) @ s["B"].float().transpose(1, 2).reshape(L * r, N)
    return (s["base"].float() + d).to(s["base"].dtype)


def run(state):
    s = state
    if own:
        from kronecker_factored_transforms_amd import binding as kq
        if s["op"] == "norm":
            o = kq.rmsnorm_quant(s["x"], s["w"], residual=s["r"], eps=EPS, alpha=s["alpha"],
                                 scale_dtype=s["step"], normed=s["normed"])
            torch.mul(o.codes.view(torch.int8), o.scales[:, None], out=s["values"])
            return dict(values=s["values"], scales=o.scales, residual=o.residual, normed=o.normed)
        if s["op"] == "experts":
            return kq.grouped_gemm(s["xq"], s["sx"], s["wq"], s["sw"], s["offsets"], rows=s["rows"],
                                   bits=s["bits"], out_dtype=s["out"])
        return kq.adapter_add(s["x"], s["A"], s["B"], s["adapter"], base=s["base"], scaling=s["scaling"])
    if s["op"] == "norm":
        return _plain_norm(s)
    return _plain_experts(s) if s["op"] == "experts" else _plain_adapters(s)


# ------------------------------------------------------------------------------ work
def work(case):
    if case["op"] == "norm":
        es = 4 if case["dtype"] == "fp32" else 2
        T, n = case["T"], case["n"]
        passes = 1 + 2 * case["residual"] + case["normed"]
        return {"bytes": T * n * (passes * es + 1) + n * es + T * (4 if case["step"] == "fp32" else 2),
                "flops": 6 * T * n}
    if case["op"] == "experts":
        T, E, N, K, R = case["T"], case["E"], case["N"], case["K"], case["T"] * case["top"]
        ss, os_ = (4 if case[k] == "fp32" else 2 for k in ("step", "out"))
        used = E * (1 - (1 - 1 / E) ** R)  # experts that some row chose, were the choice even
        return {"bytes": int((T * K + used * N * K) * case["bits"] / 8 + (T + used * N) * ss + R * N * os_),
                "flops": 2 * R * N * K}
    T, r, K, N = case["T"], case["r"], case["K"], case["N"]
    used = case["L"] * (1 - (1 - 1 / case["L"]) ** case["requests"])
    return {"bytes": int(2 * (T * K + used * r * (K + N) + 2 * T * N) + 4 * T),
            "flops": 2 * T * r * (K + N)}


# ----------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f8 = torch.float64
    if case["op"] == "norm":
        x = s["x"].to(f8)
        if s["r"] is not None:
            x += s["r"].to(f8)
        y = x * s["w"].to(f8) / torch.sqrt(torch.linalg.vector_norm(x, dim=1, keepdim=True) ** 2 / case["n"] + EPS)
        top = torch.maximum(y.amax(1), -y.amin(1)) / (1 + math.exp(-case["alpha"]))
        step = (top / 127).to(TYPES[case["step"]]).to(f8)
        q = torch.clamp(torch.round(y / step.clamp_min(1e-300)[:, None]), -128, 127) * (step > 0)[:, None]
        return dict(values=q * step[:, None], scales=step, residual=None if s["r"] is None else x,
                    normed=y if case["normed"] else None)
    if case["op"] == "experts":
        b, N = case["bits"], case["N"]
        rows, ends = s["rows"].long(), s["offsets"].tolist()

        def value(c):  # two's complement of b bits
            if b == 8:
                v = c.to(f8)
                return v - 256 * (v > 127)
            v = torch.empty((*c.shape[:-1], 2 * c.shape[-1]), dtype=f8, device=DEV)
            v[..., 0::2] = (c % 16).to(f8)
            v[..., 1::2] = torch.div(c, 16, rounding_mode="floor").to(f8)
            return v - 16 * (v > 7)

        out = torch.empty((rows.numel(), N), dtype=f8, device=DEV)
        for e in range(case["E"]):
            i, j = ends[e], ends[e + 1]
            if j > i:
                x = value(s["xq"][rows[i:j]]) * s["sx"][rows[i:j]].to(f8)[:, None]
                out[i:j] = x @ (value(s["wq"][e]) * s["sw"][e].to(f8)[:, None]).t()
        return out
    out = s["base"].to(f8)
    for a in range(case["L"]):
        at = (s["adapter"] == a).nonzero()[:, 0]
        if at.numel():
            low = s["x"][at].to(f8) @ s["A"][a].to(f8).t()
            out[at] += float(s["scaling"][a]) * (low @ s["B"][a].to(f8).t())
    return out
