"""Feed-forward operators measured here: the gated block over N:M weights with its
backward pass, and microscaled 4-bit floating point (quantisation, product and
gated product).

Gated block (weight W [2F][k], gate rows first, masked to N:M):
    p = X Wm^T * scale + bias,   y[t, f] = act(p[t, f]) * p[t, F + f]
and from p, X and dY the gradients of X, of Wm and of the bias.

Microscaled 4-bit floating point: blocks of 32 values along k share a power of two
2^e, e = floor(log2(max |x|)) - 2 (at least -127); each value is x / 2^e rounded
half to even onto {0, 0.5, 1, 1.5, 2, 3, 4, 6} with its sign, at most 6.
"""
import math

import torch

own = False

ACTS = ("silu", "gelu", "relu", "none")
DT = {"int8": torch.int8, "fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
OUT = {"fp16": "float16", "bf16": "bfloat16", "fp32": "float32"}
PATTERNS = ((1, 4), (2, 4), (2, 8), (4, 8), (4, 4))


def listed():
    return [
        # one image of a ViT-B (197 tokens) through an int8 gated block: launch latency counts
        dict(name="gated int8 T197", op="gated", dt="int8", T=197, k=768, F=2048, N=2, M=4, act="gelu", out="fp16",
             bias=True, save=False),
        # a training forward at ViT-L's width, batch 32, which saves the pre-activations
        dict(name="gated bf16 T6304 saved", op="gated", dt="bf16", T=6304, k=1024, F=4096, N=2, M=4, act="silu",
             out="bf16", bias=False, save=True),
        # a Swin stage with ragged tokens and channels, 4:8
        dict(name="gated fp16 ragged", op="gated", dt="fp16", T=1003, k=384, F=1030, N=4, M=8, act="relu", out="fp32",
             bias=True, save=True),
        # the training step's backward pass at ViT-L's width, batch 32
        dict(name="backward bf16 T6304", op="backward", dt="bf16", T=6304, k=1024, F=4096, N=2, M=4, act="silu",
             bias=False),
        # a small ragged fine-tuning batch, with the gradient of the bias
        dict(name="backward fp16 ragged", op="backward", dt="fp16", T=1379, k=768, F=2051, N=1, M=4, act="gelu",
             bias=True),
        # ViT-B activations of batch 64 to 4 bits and back
        dict(name="quantise bf16 T12608", op="quantise", dt="bf16", T=12608, k=768),
        # few rows of a long odd width in full precision
        dict(name="quantise fp32 ragged", op="quantise", dt="fp32", T=333, k=4128),
        # one token against a 4-bit weight: latency
        dict(name="mx one token", op="mx", dt="bf16", T=1, k=1024, n=4096, N=4, M=4, act="none", out="bf16",
             bias=False),
        # the first feed-forward layer of a ViT-L at batch 64, quantised on the way in
        dict(name="mx bf16 T12608", op="mx", dt="bf16", T=12608, k=1024, n=4096, N=4, M=4, act="gelu", out="bf16",
             bias=True),
        # a long reduction with ragged tokens and channels, the weight pruned 2:4 before it is quantised
        dict(name="mx fp16 ragged", op="mx", dt="fp16", T=515, k=4096, n=1001, N=2, M=4, act="none", out="fp32",
             bias=True),
        # the gated block of one image in 4 bits
        dict(name="mx gated T197", op="mx_gated", dt="fp16", T=197, k=768, F=2048, N=4, M=4, act="gelu", out="fp16",
             bias=True),
        # and of a batch of 32
        dict(name="mx gated T6304", op="mx_gated", dt="bf16", T=6304, k=1024, F=4096, N=2, M=4, act="silu",
             out="bf16", bias=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("gated", "backward", "quantise", "mx", "mx_gated"))
    N, M = rng.choice(PATTERNS)
    act = rng.choice(ACTS)
    bias = rng.random() < 0.5
    if op == "gated":
        dt = rng.choice(("int8", "fp16", "bf16"))
        return dict(op=op, dt=dt, T=_log(rng, 1, 6304), k=16 * _log(rng, 4, 64), F=_log(rng, 24, 4096), N=N, M=M,
                    act=act, out=rng.choice(("fp16", "bf16", "fp32")), bias=bias,
                    save=dt != "int8" and rng.random() < 0.5)
    if op == "backward":
        return dict(op=op, dt=rng.choice(("fp16", "bf16")), T=_log(rng, 1, 6304), k=16 * _log(rng, 4, 64),
                    F=_log(rng, 24, 4096), N=N, M=M, act=act, bias=bias)
    if op == "quantise":
        return dict(op=op, dt=rng.choice(("fp16", "bf16", "fp32")), T=_log(rng, 1, 12608), k=32 * _log(rng, 1, 128))
    dt = rng.choice(("fp16", "bf16", "fp32"))
    out = rng.choice(("fp16", "bf16", "fp32"))
    if op == "mx":
        return dict(op=op, dt=dt, T=_log(rng, 1, 6304), k=32 * _log(rng, 2, 64), n=_log(rng, 24, 4096), N=N, M=M,
                    act=rng.choice(("none", "gelu")), out=out, bias=bias)
    return dict(op=op, dt=dt, T=_log(rng, 1, 6304), k=32 * _log(rng, 2, 32), F=_log(rng, 24, 4096), N=N, M=M, act=act,
                out=out, bias=bias)


# ------------------------------------------------------------------ plain forms

def _mask(W, N, M):
    """W with all but the N largest |w| of every M along a row set to zero (ties keep the lower position)."""
    if N == M:
        return W
    g = W.reshape(W.shape[0], -1, M)
    order = torch.sort(g.float().abs(), dim=2, descending=True, stable=True).indices[..., :N]
    keep = torch.zeros(g.shape, dtype=torch.bool, device=W.device).scatter_(2, order, True)
    return torch.where(keep, g, torch.zeros_like(g)).reshape(W.shape)


def _mx(x):
    """The values that x [rows, k] stands for in microscaled 4-bit floating point, in fp32."""
    b = x.float().reshape(x.shape[0], -1, 32)
    top = b.abs().amax(dim=2, keepdim=True)
    e = torch.clamp(torch.frexp(top).exponent - 3, min=-127)
    y = b * _pow2(-e)
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = torch.clamp(torch.round(a / step) * step, max=6.0)
    return (torch.copysign(q, y) * _pow2(e)).reshape(x.shape)


def _pow2(e):
    """2^e, exactly (the exponent field of a 64-bit number), in fp32."""
    return ((e.long() + 1023) << 52).view(torch.float64).float()


def _act(v, act):
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    return torch.clamp(v, min=0) if act == "relu" else v


def _slope(v, act):
    if act == "silu":
        s = 1 / (1 + torch.exp(-v))
        return s * (1 + v * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(v * math.sqrt(0.5))) + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)
    return (v > 0).to(v.dtype) if act == "relu" else torch.ones_like(v)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, dt, T, k = case["op"], DT[case["dt"]], case["T"], case["k"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    st = {"case": case}
    if dt == torch.int8:
        st["X"] = torch.randint(-128, 128, (T, k), generator=g, device="cuda").to(dt)
    else:
        X = normal(T, k)
        X *= 1 + 15 * (torch.rand((1, k), generator=g, device="cuda") < 0.01)  # a few outlier features
        st["X"] = X.to(dt)
    if op == "quantise":
        return st
    rows = 2 * case["F"] if "F" in case else case["n"]
    if dt == torch.int8:
        W = torch.randint(-127, 128, (rows, k), generator=g, device="cuda").to(dt)
        st["scale"] = (0.5 + torch.rand(rows, generator=g, device="cuda")) / (73 * 73 * math.sqrt(k * case["N"] / case["M"]))
    else:
        W = (normal(rows, k) / math.sqrt(k)).to(dt)
        st["scale"] = None
    st["bias"] = 0.1 * normal(rows) if case["bias"] else None
    st["Wm"] = _mask(W, case["N"], case["M"])
    if op in ("mx", "mx_gated"):
        st["Wm"] = _mx(st["Wm"])
    if op == "backward":
        p = torch.matmul(st["X"], st["Wm"].t())
        st["P"] = p if st["bias"] is None else (p + st["bias"]).to(dt)
        st["dY"] = (0.1 * normal(T, case["F"])).to(dt)
    if own:
        import structured_sparse_gemm_compress_b200 as nm
        if op in ("mx", "mx_gated"):
            st["h"] = nm.nm_compress_mx(W, case["N"], case["M"], gated=op == "mx_gated")
        else:
            st["h"] = nm.nm_compress_gated(W, case["N"], case["M"])
    return st


def _run_own(st):
    import structured_sparse_gemm_compress_b200 as nm
    case = st["case"]
    op = case["op"]
    if op == "quantise":
        Q, S = nm.nm_mx_quantize(st["X"])
        return {"values": nm.nm_mx_dequantize(Q, S, dtype=st["X"].dtype)}
    if op == "backward":
        dX, dW, dbias = nm.nm_gated_backward(st["h"], st["X"], st["P"], st["dY"], act=case["act"],
                                             bias_grad=case["bias"])
        return {"dX": dX, "dW": dW, **({"dbias": dbias} if case["bias"] else {})}
    kw = dict(scale=st["scale"], bias=st["bias"], act=case["act"], out=OUT[case["out"]])
    if op == "gated":
        P = None
        if case["save"]:
            P = torch.empty((case["T"], 2 * case["F"]), dtype=st["X"].dtype, device="cuda")
        Y = nm.nm_spmm_gated(st["h"], st["X"], P=P, **kw)
        return {"Y": Y, "P": P} if case["save"] else {"Y": Y}
    Q, S = nm.nm_mx_quantize(st["X"])
    return {"Y": (nm.nm_spmm_mx_gated if op == "mx_gated" else nm.nm_spmm_mx)(st["h"], Q, S, **kw)}


def run(state):
    if own:
        return _run_own(state)
    case, X = state["case"], state["X"]
    op = case["op"]
    if op == "quantise":
        return {"values": _mx(X).to(X.dtype)}
    W = state["Wm"].float()
    if op == "backward":
        F = case["F"]
        p, dy = state["P"].float(), state["dY"].float()
        gate, up = p[:, :F], p[:, F:]
        dp = torch.cat((dy * up * _slope(gate, case["act"]), dy * _act(gate, case["act"])), dim=1)
        out = {"dX": (dp @ W).to(X.dtype), "dW": (dp.t() @ X.float()).to(X.dtype)}
        if case["bias"]:
            out["dbias"] = dp.sum(dim=0)
        return out
    p = (_mx(X) if op in ("mx", "mx_gated") else X.float()) @ W.t()
    if state["scale"] is not None:
        p = p * state["scale"]
    if state["bias"] is not None:
        p = p + state["bias"]
    out = DT[case["out"]]
    if op == "mx":
        return {"Y": _act(p, case["act"]).to(out)}
    F = case["F"]
    y = (_act(p[:, :F], case["act"]) * p[:, F:]).to(out)
    return {"Y": y, "P": p.to(X.dtype)} if case.get("save") else {"Y": y}


# ------------------------------------------------------------------ 64 bits

def _mx64(x):
    """Microscaled values in 64 bits, each the nearest of the eight magnitudes by comparison with their midpoints."""
    b = x.double().unflatten(1, (-1, 32))
    top = b.abs().max(dim=2, keepdim=True).values
    # the largest power of two that is at most the block's maximum, found in a table; two steps below it is the unit
    table = torch.tensor([2.0 ** i for i in range(-125, 128)], dtype=torch.float64, device=x.device)
    unit = table[(torch.bucketize(top, table, right=True) - 1).clamp(min=0)] / 4
    a = (b / unit).abs()
    levels = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
    q = torch.zeros_like(a)
    for i in range(1, 8):
        mid = 0.5 * (levels[i - 1] + levels[i])
        # a value on a midpoint goes to the level of even mantissa, i.e. of even index
        up = a >= mid if i % 2 == 0 else a > mid
        q = torch.where(up, torch.full_like(q, levels[i]), q)
    return (torch.sign(b) * q * unit).flatten(1)


def _act64(v, act):
    if act == "silu":
        return v * torch.special.expit(v)
    if act == "gelu":
        return v * torch.special.ndtr(v)
    return v * (v > 0) if act == "relu" else v


def _slope64(v, act):
    if act == "silu":
        s = torch.special.expit(v)
        return s + v * s * torch.special.expit(-v)
    if act == "gelu":
        return torch.special.ndtr(v) + v * torch.exp(-v * v / 2) * (2 * math.pi) ** -0.5
    return (v > 0).double() if act == "relu" else torch.ones_like(v)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantise":
        return {"values": _mx64(st["X"])}
    W = st["Wm"].double()
    if op == "backward":
        p, dy = st["P"].double(), st["dY"].double()
        gate, up = p.tensor_split(2, dim=1)
        dgate, dup = dy * up * _slope64(gate, case["act"]), dy * _act64(gate, case["act"])
        F, X = case["F"], st["X"].double()
        out = {"dX": dgate @ W[:F] + dup @ W[F:], "dW": torch.cat((dgate.t() @ X, dup.t() @ X))}
        if case["bias"]:
            out["dbias"] = torch.cat((dgate.sum(0), dup.sum(0)))
        return out
    X = _mx64(st["X"]) if op in ("mx", "mx_gated") else st["X"].double()
    p = X @ W.t()
    if st["scale"] is not None:
        p = p * st["scale"].double()
    if st["bias"] is not None:
        p = p + st["bias"].double()
    if op == "mx":
        return {"Y": _act64(p, case["act"])}
    gate, up = p.tensor_split(2, dim=1)
    y = _act64(gate, case["act"]) * up
    return {"Y": y, "P": p} if case.get("save") else {"Y": y}


def work(case):
    """Inputs read once, outputs written once; products count the kept weights only."""
    op, T, k = case["op"], case["T"], case["k"]
    size = {"int8": 1, "fp16": 2, "bf16": 2, "fp32": 4}
    es = size[case["dt"]]
    if op == "quantise":  # values in and out; the 4-bit form and its scales written and read between
        return {"bytes": 2 * T * k * es + 2 * (T * k / 2 + T * k / 32), "flops": 8 * T * k}
    kept = case["N"] / case["M"]
    rows = 2 * case["F"] if "F" in case else case["n"]
    cols = case["F"] if "F" in case else rows
    vec = 4 * rows * ((1 if case["bias"] else 0) + (1 if case["dt"] == "int8" else 0))
    if op == "backward":
        nbytes = es * (2 * T * k + T * rows + T * cols + rows * k * (1 + kept)) + vec
        return {"bytes": nbytes, "flops": 2 * T * rows * k * (1 + kept)}
    out = T * cols * size[case["out"]]
    if op == "gated":
        weight = rows * k * kept * (es + (0 if case["N"] == case["M"] else math.log2(case["M"]) / 8))
        saved = T * rows * es if case["save"] else 0
        return {"bytes": T * k * es + weight + out + saved + vec, "flops": 2 * T * rows * k * kept}
    weight = rows * k * (1 / 2 + 1 / 32)
    between = 2 * T * k * (1 / 2 + 1 / 32)  # the 4-bit activation, written and read
    return {"bytes": T * k * es + between + weight + out + vec, "flops": 2 * T * rows * k * kept}
