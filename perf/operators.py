"""The grouped and 8-bit matrix products: measured cases, plain forms and
64-bit definitions.

Operators (``op`` of a case):

* ``matmul``    c[r, n] = sum_k a[r, k] w[e, n, k] for the rows r of expert
                e's queue [offsets[e], offsets[e + 1])
* ``backward``  da[r, k] = sum_n dc[r, n] w[e, n, k] and
                dw[e, n, k] = sum over the queue's rows of dc[r, n] a[r, k]
* ``quantize``  8-bit integer codes and one float32 scale for each row
* ``int8``      c[r, n] = (sum_k qa[r, k] qw[e, n, k]) sa[r] sw[e, n]; with
                E = 0 the product is dense (no queues, one weight matrix)

The queues come from a routing: T tokens pick k of E experts each, by the k
largest of random logits plus ``skew`` times a falling bias, so that
queue lengths are ragged and some experts stay empty.
"""
import math

import torch

own = False

# bytes per element of the types a case names
SIZE = {"bf16": 2, "f32": 4}
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token of a 128-expert layer through the fused gate and up
        # weights: 8 rows, each in a queue of its own; the weights' bytes are all
        dict(name="matmul one token", op="matmul", T=1, k=8, E=128, N=1536, K=2048, dtype="bf16", skew=0.0),
        # a decoding batch of 64 through a 64-expert layer's down projection
        dict(name="matmul batch 64", op="matmul", T=64, k=6, E=64, N=2048, K=1408, dtype="bf16", skew=0.5),
        # a short prompt, widths that no tile divides
        dict(name="matmul odd widths", op="matmul", T=1001, k=2, E=8, N=1000, K=520, dtype="bf16", skew=0.5),
        # prefill of an 8-expert layer, one of its 4096 x 14336 matrices
        dict(name="matmul prefill", op="matmul", T=8192, k=2, E=8, N=14336, K=4096, dtype="bf16", skew=0.3),
        # a small layer kept in float32
        dict(name="matmul f32", op="matmul", T=256, k=2, E=8, N=256, K=128, dtype="f32", skew=0.3),
        # a training step's gradients, 128 experts of width 768
        dict(name="backward training", op="backward", T=32768, k=8, E=128, N=768, K=2048, dtype="bf16", skew=0.5),
        # the gradients of the short prompt
        dict(name="backward odd widths", op="backward", T=1001, k=2, E=8, N=1000, K=520, dtype="bf16", skew=0.5),
        # a mid-sized layer's gradients in float32
        dict(name="backward f32", op="backward", T=2048, k=2, E=16, N=512, K=1024, dtype="f32", skew=0.3),
        # the tokens of a training batch
        dict(name="quantize tokens", op="quantize", T=32768, K=2048, dtype="bf16"),
        # a small weight matrix kept in float32, rows of an odd number of words
        dict(name="quantize f32", op="quantize", T=1408, K=1040, dtype="f32"),
        # a decoding batch of 16 through a dense projection
        dict(name="int8 dense batch 16", op="int8", T=16, k=1, E=0, N=4096, K=4096, dtype="bf16", skew=0.0),
        # prefill of the 8-expert layer in 8 bits
        dict(name="int8 prefill", op="int8", T=8192, k=2, E=8, N=14336, K=4096, dtype="bf16", skew=0.3),
    ]


def _log(rng, low, high):
    return math.exp(rng.uniform(math.log(low), math.log(high)))


def draw(rng):
    while True:
        op = rng.choice(["matmul", "matmul", "backward", "quantize", "int8", "int8"])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        # rows of every operand are whole 16-byte words
        T = int(_log(rng, 1, 40000))
        K = 16 * int(_log(rng, 4, 500)) if op in ("int8", "quantize") else 8 * int(_log(rng, 8, 1000))
        if op == "quantize":
            if T * K <= 32768 * 2048:
                return dict(op=op, T=T, K=K, dtype=dtype)
            continue
        N = 8 * int(_log(rng, 8, 1800))
        E = int(_log(rng, 1, 257))
        if op == "int8" and rng.random() < 0.3:
            E = 0
        k = min(rng.choice([1, 2, 4, 6, 8]), max(E, 1))
        rows = T * k
        flops = 2.0 * rows * N * K * (2 if op == "backward" else 1)
        # (float32 products run on a sixteenth of the rate)
        most = 1.0e11 if dtype == "f32" and op != "int8" else 1.9e12
        if flops > most or max(E, 1) * N * K > 5.0e8 or rows * max(N, K) > 2.5e8:
            continue
        return dict(op=op, T=T, k=k, E=E, N=N, K=K, dtype=dtype, skew=rng.choice([0.0, 0.3, 0.5, 1.0]))


def _active(case):
    """Experts that get a row, as the routing gives them on average (of
    equally likely experts)."""
    E, k, T = case["E"], case["k"], case["T"]
    return 1 if E == 0 else E * (1.0 - (1.0 - k / E) ** T)


def work(case):
    T, K, b = case["T"], case["K"], SIZE[case["dtype"]]
    if case["op"] == "quantize":
        return {"bytes": T * K * (b + 1) + 4 * T, "flops": 3 * T * K}
    rows, N = T * case["k"], case["N"]
    mats = _active(case)
    if case["op"] == "matmul":
        return {"bytes": b * (rows * K + rows * N + mats * N * K), "flops": 2 * rows * N * K}
    if case["op"] == "backward":
        return {"bytes": b * (2 * rows * K + rows * N + (mats + case["E"]) * N * K), "flops": 4 * rows * N * K}
    return {"bytes": rows * K + 4 * rows + mats * (N * K + 4 * N) + rows * N * b, "flops": 2 * rows * N * K}


def _codes(g, rows, cols):
    """Codes and scales of a matrix of normal values: each row's largest
    value has the code 127 or -127."""
    codes = torch.empty(rows, cols, dtype=torch.int8, device="cuda")
    scales = torch.empty(rows, dtype=torch.float32, device="cuda")
    step = max(1, (1 << 27) // cols)
    for r in range(0, rows, step):
        v = torch.randn(min(step, rows - r), cols, generator=g, device="cuda")
        s = v.abs().amax(1) / 127
        codes[r:r + step] = (v / s[:, None]).round().clamp(-127, 127).to(torch.int8)
        scales[r:r + step] = s
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = TORCH[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dt)

    st = dict(case)
    T, K = case["T"], case["K"]
    if case["op"] == "quantize":
        # tokens differ in size by orders of magnitude, some channels stand out
        x = torch.randn(T, K, generator=g, device="cuda") * torch.exp(torch.randn(T, 1, generator=g, device="cuda"))
        x *= torch.where(torch.rand(K, generator=g, device="cuda") < 0.01, 20.0, 1.0)
        st["x"] = x.to(dt)
        return st
    E, N, k = case["E"], case["N"], case["k"]
    rows = T * k
    if E > 0:
        logits = torch.randn(T, E, generator=g, device="cuda") - case["skew"] * torch.log1p(
            torch.arange(E, device="cuda", dtype=torch.float32))
        ids = torch.topk(logits, k, dim=1).indices
        counts = torch.bincount(ids.reshape(-1), minlength=E)
        offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        offsets[1:] = torch.cumsum(counts, 0)
        st["offsets"] = offsets
        # (the plain forms walk the queues on the host)
        st["bounds"] = offsets.tolist()
    if case["op"] == "int8":
        st["a"], st["sa"] = _codes(g, rows, K)
        w, sw = _codes(g, max(E, 1) * N, K)
        sw *= 1.0 / math.sqrt(K)
        st["w"] = w.view(E, N, K) if E > 0 else w
        st["sw"] = sw.view(E, N) if E > 0 else sw
        return st
    st["a"] = normal(rows, K)
    st["w"] = normal(E, N, K).mul_(1.0 / math.sqrt(K))
    if case["op"] == "backward":
        st["dc"] = normal(rows, N)
    return st


def _queues(st):
    """(expert, first row, end) of every queue that has rows.  Queues differ
    in length, so no one torch product covers them all; padding them to the
    longest would multiply the work by the longest over the mean."""
    b = st["bounds"]
    return [(e, b[e], b[e + 1]) for e in range(st["E"]) if b[e + 1] > b[e]]


def run(st):
    op = st["op"]
    if own:
        import mixture_experts_layer_exclusive_amd as moe
        if op == "matmul":
            return moe.grouped_matmul(st["a"], st["w"], st["offsets"])
        if op == "backward":
            g = moe.grouped_matmul_backward(st["a"], st["w"], st["offsets"], st["dc"])
            return {"da": g["da"], "dw": g["dw"]}
        if op == "quantize":
            codes, scales = moe.quantize_rows_int8(st["x"])
            return {"codes": codes, "scales": scales}
        return moe.grouped_matmul_int8(st["a"], st["sa"], st["w"], st["sw"], st.get("offsets"),
                                       out_dtype=TORCH[st["dtype"]])
    if op == "quantize":
        # (in 64 bits: codes next to a border; each quotient is rounded to
        # float32 first, as the operator defines it)
        x = st["x"].double()
        scales = (x.abs().amax(1) / 127).float()
        codes = (x / scales.double()[:, None]).float().round()
        return {"codes": codes.to(torch.int8), "scales": scales}
    if op == "int8" and st["E"] == 0:
        c = st["a"].float() @ st["w"].float().t()
        return (c * st["sa"][:, None] * st["sw"]).to(TORCH[st["dtype"]])
    a, w = st["a"], st["w"]
    if op == "backward":
        dc = st["dc"]
        da, dw = torch.empty_like(a), torch.zeros_like(w)
        for e, lo, hi in _queues(st):
            d = dc[lo:hi].float()
            da[lo:hi] = d @ w[e].float()
            dw[e] = d.t() @ a[lo:hi].float()
        return {"da": da, "dw": dw}
    c = torch.empty(a.shape[0], st["N"], dtype=TORCH[st["dtype"]], device=a.device)
    for e, lo, hi in _queues(st):
        v = a[lo:hi].float() @ w[e].float().t()
        if op == "int8":
            v = v * st["sa"][lo:hi, None] * st["sw"][e]
        c[lo:hi] = v
    return c


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = st["x"].double()
        m = torch.maximum(x.amax(1), -x.amin(1))
        s = torch.div(m, 127.0).to(torch.float32)
        # the operator's scale is this float32 number, its quotient a float32
        q = torch.div(x, s.to(torch.float64).unsqueeze(1)).to(torch.float32)
        return {"codes": torch.round(q).to(torch.int8), "scales": torch.div(m, 127.0)}
    a, w = st["a"], st["w"]
    E = max(case["E"], 1)
    cuts = st["bounds"] if case["E"] > 0 else [0, a.shape[0]]
    sizes = [cuts[e + 1] - cuts[e] for e in range(E)]
    w = w.reshape(E, case["N"], case["K"])
    if op == "backward":
        da, dw = [], []
        for ae, de, we in zip(a.split(sizes), st["dc"].split(sizes), w):
            dt = de.double()
            da.append(torch.matmul(we.double().t(), dt.t()).t())
            dw.append(torch.matmul(ae.double().t(), dt).t().contiguous())
        return {"da": torch.cat(da), "dw": torch.stack(dw)}
    out = [torch.matmul(we.double(), ae.double().t()).t() for ae, we in zip(a.split(sizes), w)]
    if op == "int8":
        sa, sw = st["sa"].double(), st["sw"].double().reshape(E, -1)
        out = [o * torch.outer(s, t) for o, s, t in zip(out, sa.split(sizes), sw)]
    return torch.cat(out)
