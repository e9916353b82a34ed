"""Routing with scores, balance bias and groups, its gradient, the combine's
gradient, and 4-bit microscaled floats with their product by expert: measured
cases, plain forms and 64-bit definitions.

Operators (``op`` of a case):

* ``route``      scores s[t, e] = sigmoid(l[t, e]), or softmax over the experts;
                 of the ``kept`` best of ``groups`` groups (a group's value: the
                 sum of its ``top`` best s + bias), the k largest s + bias,
                 equal ones to the lower expert; gates scale * s of the chosen,
                 over their sum with ``renorm``; with ``sums`` also the sum of
                 s over the tokens
* ``route_back`` the logits' gradient for the gates' and the score sums'
* ``combine_back`` for y[t] = sum_j gates[t, j] y_perm[pos[t, j]]:
                 dy_perm[pos[t, j]] = gates[t, j] dy[t], dgates[t, j] = dy[t] . y_perm[pos[t, j]]
* ``quantize``   4-bit codes (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives)
                 with a power of two for each 32 values of a row, 2^(floor(log2
                 max) - 2), and back to numbers
* ``product``    c[r, n] = sum_k a[r, k] w[e, n, k] of such numbers for the rows r
                 of expert e's queue [offsets[e], offsets[e + 1]); with E = 0
                 the product is dense (no queues, one weight matrix)
"""
import math

import torch

own = False

# bytes per element of the types a case names
SIZE = {"bf16": 2, "f32": 4}
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
# the values of the 4-bit codes
VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def listed():
    return [
        # one token of a 256-expert layer whose experts lie in 8 groups
        dict(name="route one token", op="route", T=1, E=256, k=8, score="sigmoid", bias=True, groups=8, kept=4, top=2,
             renorm=True, scale=2.5, sums=False),
        # a training batch of that layer, with the score sums of a balance loss
        dict(name="route training", op="route", T=32768, E=256, k=8, score="sigmoid", bias=True, groups=8, kept=4,
             top=2, renorm=True, scale=2.5, sums=True),
        # a short prompt, softmax scores kept as they are, experts that no word divides
        dict(name="route_back odd", op="route_back", T=1001, E=62, k=6, score="softmax", renorm=False, scale=1.0,
             sums=True),
        # the gradient of the training batch
        dict(name="route_back training", op="route_back", T=32768, E=256, k=8, score="sigmoid", renorm=True, scale=2.5,
             sums=True),
        # a short prompt's combine kept in float32
        dict(name="combine_back f32", op="combine_back", T=1001, k=2, d=520, dtype="f32"),
        # a training step's combine, 8 experts per token
        dict(name="combine_back training", op="combine_back", T=32768, k=8, d=2048, dtype="bf16"),
        # a decoding batch's activations
        dict(name="quantize batch 16", op="quantize", T=16, K=4096, dtype="bf16"),
        # the tokens of a training batch
        dict(name="quantize tokens", op="quantize", T=32768, K=2048, dtype="bf16"),
        # one token of a 128-expert layer through the fused gate and up weights:
        # 8 rows, each in a queue of its own; the weights' bytes are all
        dict(name="product one token", op="product", T=1, k=8, E=128, N=1536, K=2048, dtype="bf16", skew=0.0),
        # a decoding batch of 64 through a 64-expert layer's down projection
        dict(name="product batch 64", op="product", T=64, k=6, E=64, N=2048, K=1408, dtype="bf16", skew=0.5),
        # a short prompt, widths that no tile divides, a float32 result
        dict(name="product odd widths", op="product", T=1001, k=2, E=8, N=1000, K=544, dtype="f32", skew=0.5),
        # prefill of an 8-expert layer, one of its 4096 x 14336 matrices
        dict(name="product prefill", op="product", T=8192, k=2, E=8, N=14336, K=4096, dtype="bf16", skew=0.3),
    ]


def _log(rng, low, high):
    return math.exp(rng.uniform(math.log(low), math.log(high)))


def draw(rng):
    while True:
        op = rng.choice(["route", "route_back", "combine_back", "quantize", "product", "product"])
        T = int(_log(rng, 1, 40000))
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if op in ("route", "route_back"):
            groups = rng.choice([1, 1, 2, 4, 8])
            size = int(_log(rng, 2, 256 / groups + 0.99))
            E = groups * size
            k = min(rng.choice([1, 2, 4, 6, 8, 12]), E)
            kept = rng.randint(min(groups, -(-k // size)), groups)
            c = dict(op=op, T=T, E=E, k=k, score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.6,
                     scale=rng.choice([1.0, 2.5]), sums=rng.random() < 0.5)
            if T * E > 32768 * 256:
                continue
            if op == "route":
                c.update(bias=rng.random() < 0.6, groups=groups, kept=kept, top=rng.choice([1, 2]))
            return c
        if op == "combine_back":
            # (the combine takes bf16 rows of whole 128-byte lines, float32 rows of any length)
            d = 64 * int(_log(rng, 1, 129)) if dtype == "bf16" else int(_log(rng, 8, 8192))
            k = rng.choice([1, 2, 4, 6, 8])
            if T * k * d > 32768 * 8 * 2048 // 2:
                continue
            return dict(op=op, T=T, k=k, d=d, dtype=dtype)
        # rows of codes are whole 16-byte words
        K = 32 * int(_log(rng, 2, 300))
        if op == "quantize":
            if T * K <= 32768 * 2048:
                return dict(op=op, T=T, K=K, dtype=dtype)
            continue
        N = 8 * int(_log(rng, 8, 1800))
        E = 0 if rng.random() < 0.25 else int(_log(rng, 1, 257))
        k = min(rng.choice([1, 2, 4, 6, 8]), max(E, 1))
        rows = T * k
        if 2.0 * rows * N * K > 1.9e12 or max(E, 1) * N * K > 5.0e8 or rows * max(N, K) > 2.5e8:
            continue
        return dict(op=op, T=T, k=k, E=E, N=N, K=K, dtype=dtype, skew=rng.choice([0.0, 0.3, 0.5, 1.0]))


def work(case):
    op, T = case["op"], case["T"]
    if op in ("route", "route_back"):
        E, k = case["E"], case["k"]
        if op == "route":
            return {"bytes": 4 * (T * E + 2 * T * k + (E if case["bias"] else 0) + (E if case["sums"] else 0)),
                    "flops": 8 * T * E}
        return {"bytes": 4 * (2 * T * E + 2 * T * k + (E if case["sums"] else 0)), "flops": 8 * T * E}
    if op == "combine_back":
        k, d, b = case["k"], case["d"], SIZE[case["dtype"]]
        return {"bytes": b * d * T * (1 + 2 * k) + 12 * T * k, "flops": 3 * T * k * d}
    K = case["K"]
    if op == "quantize":
        # codes, scales, and the numbers they stand for
        return {"bytes": T * K * SIZE[case["dtype"]] + T * K // 2 + T * K // 32 + 2 * T * K, "flops": 4 * T * K}
    E, N, k = case["E"], case["N"], case["k"]
    rows = T * k
    # experts that get a row, as the routing gives them on average (of equally
    # likely experts)
    mats = 1 if E == 0 else E * (1.0 - (1.0 - k / E) ** T)
    return {"bytes": (rows * K + mats * N * K) * (0.5 + 1 / 32) + rows * N * SIZE[case["dtype"]],
            "flops": 2 * rows * N * K}


def _quantized(g, rows, cols):
    """Codes [rows, cols / 2], two to a byte, the even column in the low half,
    and scale bytes [ceil(cols / 256), rows, 8] (2^(byte - 127), block b of a
    row at [b / 8, row, b % 8]) of a matrix of normal values whose columns
    differ in size."""
    blocks = cols // 32
    codes = torch.empty(rows, cols // 2, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, -(-blocks // 8) * 8), 127, dtype=torch.uint8, device="cuda")
    size = torch.exp(0.5 * torch.randn(blocks, 1, generator=g, device="cuda"))
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    step = max(1, (1 << 26) // cols)
    for r in range(0, rows, step):
        v = torch.randn(min(step, rows - r), blocks, 32, generator=g, device="cuda") * size
        e = torch.frexp(v.abs().amax(2)).exponent - 3
        c = torch.bucketize(torch.ldexp(v.abs(), -e[:, :, None]), borders) + 8 * (v < 0)
        c = c.to(torch.uint8).view(-1, cols // 2, 2)
        codes[r:r + step] = c[:, :, 0] | (c[:, :, 1] << 4)
        scales[r:r + step, :blocks] = (e + 127).to(torch.uint8)
    return codes, scales.view(rows, -1, 8).transpose(0, 1).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    st = dict(case)
    op, T = case["op"], case["T"]
    if op in ("route", "route_back"):
        E, k = case["E"], case["k"]
        st["logits"] = 2.0 * normal(T, E)
        if op == "route":
            st["balance"] = 0.1 * normal(E) if case["bias"] else None
        else:
            st["ids"] = torch.topk(normal(T, E) + st["logits"], k, dim=1).indices.to(torch.int32)
            st["dgates"] = normal(T, k)
            st["dsums"] = normal(E) / T if case["sums"] else None
        return st
    if op == "combine_back":
        k, d, dt = case["k"], case["d"], TORCH[case["dtype"]]
        st["dy"] = torch.randn(T, d, generator=g, device="cuda", dtype=dt)
        st["y_perm"] = torch.randn(T * k, d, generator=g, device="cuda", dtype=dt)
        gates = torch.softmax(normal(T, k), 1)
        # queues of k experts' tokens
        pick = torch.rand(T, 4 * k, generator=g, device="cuda").topk(k, dim=1).indices.reshape(-1)
        order = torch.sort(pick, stable=True).indices
        pos = torch.empty(T * k, dtype=torch.int32, device="cuda")
        pos[order] = torch.arange(T * k, dtype=torch.int32, device="cuda")
        st["gates"], st["pos"] = gates, pos
        return st
    K = case["K"]
    if op == "quantize":
        # tokens differ in size by orders of magnitude, some channels stand out
        x = normal(T, K) * torch.exp(normal(T, 1))
        x *= torch.where(torch.rand(K, generator=g, device="cuda") < 0.01, 20.0, 1.0)
        st["x"] = x.to(TORCH[case["dtype"]])
        return st
    E, N, k = case["E"], case["N"], case["k"]
    if E > 0:
        logits = normal(T, E) - case["skew"] * torch.log1p(torch.arange(E, device="cuda", dtype=torch.float32))
        counts = torch.bincount(torch.topk(logits, k, dim=1).indices.reshape(-1), minlength=E)
        offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        offsets[1:] = torch.cumsum(counts, 0)
        st["offsets"] = offsets
        # (the plain form walks the queues on the host)
        st["bounds"] = offsets.tolist()
    st["a"], st["sa"] = _quantized(g, T * k, K)
    w, sw = _quantized(g, max(E, 1) * N, K)
    st["w"] = w.view(E, N, K // 2) if E > 0 else w
    st["sw"] = sw.view(-1, E, N, 8) if E > 0 else sw
    return st


def _numbers(codes, scales):
    """The float32 numbers of codes [rows, K / 2] with scales [.., rows, 8]."""
    rows, K = codes.shape[0], 2 * codes.shape[1]
    table = torch.tensor(VALUES, device=codes.device)
    v = table[torch.stack([codes & 15, codes >> 4], 2).int()].view(rows, K // 32, 32)
    e = scales.transpose(0, 1).reshape(rows, -1)[:, :K // 32].int() - 127
    return torch.ldexp(v, e[:, :, None]).view(rows, K)


def _scores(st, dtype):
    l = st["logits"].to(dtype)
    return torch.sigmoid(l) if st["score"] == "sigmoid" else torch.softmax(l, 1)


def run(st):
    op = st["op"]
    if own:
        import mixture_experts_layer_exclusive_amd as moe
        if op == "route":
            return _named(moe.route_scored(st["k"], logits=st["logits"], score=st["score"], bias=st["balance"],
                                           groups=st["groups"], groups_kept=st["kept"], group_top=st["top"],
                                           renormalise=st["renorm"], scale=st["scale"], with_score_sums=st["sums"]))
        if op == "route_back":
            return moe.route_scored_backward(st["logits"], st["ids"], st["dgates"], score=st["score"],
                                             renormalise=st["renorm"], scale=st["scale"], dscore_sums=st["dsums"])
        if op == "combine_back":
            g = moe.combine_backward(st["dy"], st["pos"], st["gates"], y_perm=st["y_perm"])
            return {"dy_perm": g["dy_perm"], "dgates": g["dgates"]}
        if op == "quantize":
            codes, scales = moe.quantize_rows_mxfp4(st["x"])
            return moe.dequantize_rows_mxfp4(codes, scales)
        return moe.grouped_matmul_mxfp4(st["a"], st["sa"], st["w"], st["sw"], st.get("offsets"),
                                        out_dtype=TORCH[st["dtype"]])
    if op == "route":
        # (in 64 bits: scores next to each other decide the order)
        s = _scores(st, torch.float64)
        T, E = s.shape
        c = s if st["balance"] is None else s + st["balance"].double()
        if st["kept"] < st["groups"]:
            per = c.view(T, st["groups"], -1)
            value = per.topk(min(st["top"], per.shape[2]), 2).values.sum(2)
            best = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :st["kept"]]
            out = torch.ones_like(value, dtype=torch.bool).scatter_(1, best, False)
            c = per.masked_fill(out[:, :, None], -math.inf).view(T, E)
        ids = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :st["k"]]
        gates = st["scale"] * s.gather(1, ids)
        if st["renorm"]:
            gates = gates / s.gather(1, ids).sum(1, keepdim=True)
        return {"ids": ids.to(torch.int32), "gates": gates.float(),
                "sums": s.sum(0).float() if st["sums"] else None}
    if op == "route_back":
        s = _scores(st, torch.float32)
        ids = st["ids"].long()
        chosen, dg = s.gather(1, ids), st["scale"] * st["dgates"]
        if st["renorm"]:
            total = chosen.sum(1, keepdim=True)
            dg = (dg - (dg * chosen).sum(1, keepdim=True) / total) / total
        ds = torch.zeros_like(s) if st["dsums"] is None else st["dsums"].expand_as(s).clone()
        ds.scatter_add_(1, ids, dg)
        if st["score"] == "sigmoid":
            return ds * s * torch.sigmoid(-st["logits"])
        return s * (ds - (s * ds).sum(1, keepdim=True))
    if op == "combine_back":
        T, d = st["dy"].shape
        dy, pos = st["dy"].float()[:, None, :], st["pos"].long()
        dgates = (st["y_perm"][pos].float().view(T, -1, d) * dy).sum(2)
        dy_perm = torch.empty_like(st["y_perm"])
        dy_perm[pos] = (st["gates"][:, :, None] * dy).to(dy_perm.dtype).view(-1, d)
        return {"dy_perm": dy_perm, "dgates": dgates}
    if op == "quantize":
        x = st["x"].float().view(st["T"], -1, 32)
        scale = torch.frexp(x.abs().amax(2, keepdim=True)).exponent - 3
        q = torch.ldexp(x.abs(), -scale).clamp_max(6.0)
        step = torch.where(q < 2.0, 0.5, torch.where(q < 4.0, 1.0, 2.0))
        q = torch.copysign((q / step).round() * step, x)
        return torch.ldexp(q, scale).view(st["T"], -1).to(torch.bfloat16)
    a, w, dt = _numbers(st["a"], st["sa"]), st["w"], TORCH[st["dtype"]]
    if st["E"] == 0:
        return (a @ _numbers(w, st["sw"]).t()).to(dt)
    c = torch.empty(a.shape[0], st["N"], dtype=dt, device=a.device)
    # (queues differ in length, so no one torch product covers them all; padding
    # them to the longest would multiply the work by the longest over the mean)
    b = st["bounds"]
    for e, lo, hi in [(e, b[e], b[e + 1]) for e in range(st["E"]) if b[e + 1] > b[e]]:
        c[lo:hi] = a[lo:hi] @ _numbers(w[e], st["sw"][:, e]).t()
    return c


def _named(routed):
    return {"ids": routed[0], "gates": routed[1], "sums": routed[3] if len(routed) > 3 else None}


def _exact_numbers(codes, scales):
    """(in 64 bits, from sign, exponent and fraction of each code)"""
    both = torch.cat([codes.unsqueeze(2) % 16, codes.unsqueeze(2) // 16], 2).reshape(codes.shape[0], -1).long()
    exponent, odd = (both % 8) // 2, (both % 2).double()
    size = torch.where(exponent == 0, odd / 2, (1 + odd / 2) * 2.0 ** (exponent - 1).double())
    blocks = both.shape[1] // 32
    power = torch.cat(list(scales), 1)[:, :blocks].double() - 127
    return torch.where(both >= 8, -size, size) * torch.exp2(power).repeat_interleave(32, 1)


def exact(case, seed):
    st = prepare(case, seed)
    op, T = case["op"], case["T"]
    if op in ("route", "route_back"):
        l = st["logits"].double()
        if case["score"] == "sigmoid":
            s = 1.0 / (1.0 + torch.exp(-l))
        else:
            s = torch.exp(l - torch.logsumexp(l, 1, keepdim=True))
        if op == "route":
            c = s + (0.0 if st["balance"] is None else st["balance"].double())
            if case["kept"] < case["groups"]:
                per = c.reshape(T * case["groups"], -1)
                first = per.amax(1)
                if case["top"] == 2 and per.shape[1] > 1:
                    at = per.argmax(1, keepdim=True)
                    first = first + per.scatter(1, at, -math.inf).amax(1)
                rank = torch.argsort(torch.argsort(-first.view(T, -1), dim=1, stable=True), dim=1)
                c = torch.where((rank < case["kept"]).repeat_interleave(c.shape[1] // case["groups"], 1), c, -math.inf)
            ids = torch.argsort(-c, dim=1, stable=True)[:, :case["k"]]
            gates = torch.take_along_dim(s, ids, 1)
            if case["renorm"]:
                gates = gates / torch.linalg.vector_norm(gates, 1, dim=1, keepdim=True)
            return {"ids": ids.to(torch.int32), "gates": case["scale"] * gates,
                    "sums": torch.ones(T, dtype=torch.float64, device=s.device) @ s if case["sums"] else None}
        # each gate's derivatives by the scores, then the scores' by the logits
        ids = st["ids"].long()
        hot = torch.zeros(T, s.shape[1], dtype=torch.float64, device=s.device)
        hot.scatter_(1, ids, 1.0)
        dgates = torch.zeros_like(hot).scatter_(1, ids, case["scale"] * st["dgates"].double())
        by_score = dgates
        if case["renorm"]:
            total = (hot * s).sum(1)
            mean = torch.einsum("te,te->t", dgates, s) / total
            by_score = hot * (dgates - mean[:, None]) / total[:, None]
        if case["sums"]:
            by_score = by_score + st["dsums"].double()
        if case["score"] == "sigmoid":
            return by_score * s * (1.0 - s)
        return by_score * s - s * torch.einsum("te,te->t", by_score, s)[:, None]
    if op == "combine_back":
        pos = st["pos"].long()
        token = torch.empty_like(pos)
        token[pos] = torch.arange(pos.numel(), device=pos.device) // case["k"]
        gate = torch.empty(pos.numel(), dtype=torch.float64, device=pos.device)
        gate[pos] = st["gates"].double().reshape(-1)
        dot = torch.empty_like(gate)
        dy_perm = torch.empty(pos.numel(), case["d"], dtype=torch.float64, device=pos.device)
        step = 1 << 15
        for r in range(0, pos.numel(), step):
            dy = st["dy"][token[r:r + step]].double()
            dot[r:r + step] = torch.linalg.vecdot(dy, st["y_perm"][r:r + step].double())
            dy_perm[r:r + step] = dy * gate[r:r + step, None]
        return {"dy_perm": dy_perm, "dgates": dot[pos].view(T, case["k"])}
    if op == "quantize":
        x = st["x"].double().view(-1, 32)
        unit = torch.exp2(torch.floor(torch.log2(x.abs().amax(1, keepdim=True))) - 2)
        # the number of borders passed; a border itself belongs to the even code
        q = x.abs() / unit
        code = torch.zeros_like(q, dtype=torch.int64)
        for i, border in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
            code += (q >= border) if i % 2 else (q > border)
        value = torch.tensor(VALUES[:8], dtype=torch.float64, device=x.device)[code]
        return (torch.sign(x) * value * unit).view(T, -1)
    a = _exact_numbers(st["a"], st["sa"])
    if case["E"] == 0:
        return torch.matmul(_exact_numbers(st["w"], st["sw"]), a.t()).t()
    b = st["bounds"]
    parts = a.split([b[e + 1] - b[e] for e in range(case["E"])])
    return torch.cat([torch.matmul(_exact_numbers(w, st["sw"][:, e]), p.t()).t() if p.shape[0] else
                      a.new_empty(0, case["N"]) for e, (p, w) in enumerate(zip(parts, st["w"]))])
