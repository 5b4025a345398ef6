"""The operators between routing and a layer's output, as cases to be timed and compared: tokens sorted by expert and
back with their weights, the gradients of both, and the products of 4-bit weights with group scales that run between
them or as a dense projection.

Where ``own`` is false, ``run`` computes them from elementary torch operations in 32 bits; where it is true, it
makes the calls of this package."""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def sort(name, T, k, E, H, dtype="bf16", pad=0.0, wide=0, op="sort"):
    """T tokens sorted by their k of E experts; `pad`: share of pairs without an expert, `wide`: columns between rows."""
    return dict(name=name, op=op, T=T, k=k, E=E, H=H, dtype=dtype, pad=pad, wide=wide)


def combine(name, T, k, E, H, rows="bf16", y="bf16", pad=0.0, weights=True, base=False, wide=0, op="combine"):
    """The way back; `rows`, `y`: types of the experts' rows and of the result, `base`: what the sum is added to."""
    return dict(name=name, op=op, T=T, k=k, E=E, H=H, rows=rows, y=y, pad=pad, weights=weights, base=base, wide=wide)


def linear(name, T, K, N, g, k=0, E=1, dtype="bf16", out="bf16", zeros=True, swiglu=False, pad=0.0, wide=0):
    """Products with 4-bit weights [E, N, K] and a scale for g neighbours of a row; k > 0: T tokens sorted by their k of
    E experts, else T tokens through one matrix; `swiglu`: the first half of the outputs gates the second."""
    return dict(name=name, op="linear", T=T, k=k, E=E, K=K, N=N, g=g, dtype=dtype, out=out, zeros=zeros, swiglu=swiglu,
                pad=pad, wide=wide)


def listed():
    return [
        # one token of the 256-expert, top-8 layer: a lone user's decode step
        sort("sort, one token", 1, 8, 256, 4096),
        # the decode batch of the headline workload, some of its tokens padding
        sort("sort, decode", 64, 8, 256, 4096, pad=0.05),
        # the prompt of the prefill workload, top-6
        sort("sort, prompt", 8192, 6, 256, 4096),
        # its gradient: a token's rows summed
        sort("sort gradient", 8192, 6, 256, 4096, op="sort_grad"),
        # the decode batch back in token order onto the shared expert's output, rows kept in 32 bits
        combine("combine, decode", 64, 8, 256, 4096, rows="f32", base=True),
        # ragged: a width that no vector divides, 32 bits, pairs left out
        combine("combine, ragged", 1021, 5, 40, 1001, rows="f32", y="f32", pad=0.1, base=True),
        # training: the gradient of the way back over a batch, with respect to rows and weights
        combine("combine gradient", 8192, 6, 256, 4096, op="combine_grad"),
        # one token through a square projection: a lone user's decode step
        linear("4 bits, one token", 1, 4096, 4096, 128),
        # a ragged decode batch through a projection to the intermediate size, no zero points, results in 32 bits
        linear("4 bits, batch", 57, 4096, 2048, 64, dtype="f16", out="f32", zeros=False),
        # the gates and ups of the decode batch's experts: 512 rows over 256 experts
        linear("4 bits, decode experts", 64, 4096, 4096, 128, k=8, E=256, swiglu=True),
        # the experts' way down for a prompt of 4096 tokens: about 96 rows to an expert
        linear("4 bits, prompt experts", 4096, 2048, 4096, 128, k=6, E=256),
        # a dense projection of several prompts, none of them a multiple of a tile
        linear("4 bits, prompt", 4001, 4096, 4096, 128),
    ]


def spread(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["sort", "sort", "sort_grad", "combine", "combine", "combine_grad", "linear", "linear", "linear",
                     "linear"])
    if op != "linear":
        E = rng.choice([256, spread(rng, 4, 1024)])
        k = rng.randint(1, min(12, E))
        H = rng.choice([4096, 2048, 8 * spread(rng, 8, 1024), spread(rng, 64, 8192)])
        T = spread(rng, 1, 8192 * 6 * 4096 // (max(H, 1024) * max(k, 4)))
        pad, wide = rng.choice([0.0, 0.0, 0.1, 0.6]), rng.choice([0, 0, 64, 7])
        x, y = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("f32", "bf16"),
                           ("f32", "f16")])
        if x == "f32":
            T = max(1, T // 2)
        if op in ("sort", "sort_grad"):
            c = sort("", T, k, E, H, dtype=x, pad=pad, wide=wide, op=op)
        else:
            c = combine("", T, k, E, H, rows=x, y=y, pad=pad, weights=op == "combine_grad" or rng.random() < 0.8,
                        base=op == "combine" and rng.random() < 0.5, wide=wide, op=op)
    else:
        g = rng.choice([32, 64, 128, 128])
        swiglu = rng.random() < 0.3
        if rng.random() < 0.5:
            E, k, pad = 1, 0, 0.0
            K = g * spread(rng, 1, 8192 // g)
            N = rng.choice([256, 2048, 4096, spread(rng, 16, 8192)])
            T = spread(rng, 1, 4096)
            rows = T
        else:
            E = rng.choice([8, 64, 256, spread(rng, 2, 256)])
            k, pad = rng.randint(1, min(8, E)), rng.choice([0.0, 0.1])
            K = g * spread(rng, max(1, 256 // g), 4096 // g)
            N = rng.choice([1024, 4096, spread(rng, 64, 4096)])
            T = spread(rng, 1, 4096)
            rows = T * k
        most = 4001 * 4096 * 4096
        if rows * K * N > most:
            T = max(1, T * most // (rows * K * N))
        dtype = rng.choice(["bf16", "bf16", "f16"])
        c = linear("", T, K, N + N % 2 if swiglu else N, g, k=k, E=E, dtype=dtype, out=rng.choice([dtype, dtype, "f32"]),
                   zeros=rng.random() < 0.6, swiglu=swiglu, pad=pad, wide=rng.choice([0, 0, 64]))
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------------------- inputs --


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.float32, by=1.0):
        return torch.randn(*shape, device="cuda", generator=g).mul_(by).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=g)

    def matrix(n, width, dtype, by=1.0):
        """[n, width] with the case's columns between its rows."""
        return normal(n, width + case["wide"], dtype=dtype, by=by)[:, :width]

    s = dict(case)
    T, k, E = case["T"], case["k"], case["E"]
    if k:
        # balanced routing: every token its k experts, in the order of their scores
        ids = torch.topk(uniform(T, E), k, dim=1)[1].to(torch.int32)
        if case["pad"]:
            ids = torch.where(uniform(T, k) < case["pad"], -1, ids)
        s["ids"] = ids
        s["offsets"], s["pos"], _ = plan(ids, E)
    P = T * max(k, 1)
    if case["op"] in ("sort", "sort_grad"):
        H, dt = case["H"], DT[case["dtype"]]
        if case["op"] == "sort":
            s["x"] = matrix(T, H, dt)
            s["out"] = torch.zeros(P, H, dtype=dt, device="cuda")
            s["offsets"], s["pos"] = torch.empty_like(s["offsets"]), torch.empty_like(s["pos"])
        else:
            s["d_rows"] = matrix(P, H, dt, by=0.02)
            s["out"] = torch.empty(T, H, dtype=dt, device="cuda")
    elif case["op"] in ("combine", "combine_grad"):
        H, rd, yd = case["H"], DT[case["rows"]], DT[case["y"]]
        s["rows_in"] = matrix(P, H, rd, by=0.3)
        s["w"] = torch.softmax(normal(T, k), dim=1) if case["weights"] else None
        if case["op"] == "combine":
            s["base_in"] = matrix(T, H, yd, by=0.3) if case["base"] else None
            s["out"] = torch.empty(T, H, dtype=yd, device="cuda")
        else:
            s["d_y"] = matrix(T, H, yd, by=0.02)
            s["d_rows"] = torch.zeros(P, H, dtype=rd, device="cuda")
            s["d_w"] = torch.empty(T, k, device="cuda")
    else:
        K, N, dt = case["K"], case["N"], DT[case["dtype"]]
        # weights as a quantiser leaves them: codes that fill their range, scales about sigma / 4 for sigma = K^-0.5
        s["x"] = matrix(P, K, dt)
        s["codes"] = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
        s["scales"] = ((0.5 + uniform(E, N, K // case["g"])) * (0.25 * K ** -0.5)).to(dt)
        s["z"] = None
        if case["zeros"]:
            s["z"] = torch.randint(5, 12, (E, N, K // case["g"]), dtype=torch.uint8, device="cuda", generator=g)
        s["out"] = torch.zeros(P, N // 2 if case["swiglu"] else N, dtype=DT[case["out"]], device="cuda")
        s["bounds"] = s["offsets"].tolist() if k else [0, P]
        if not k:
            s["offsets"] = None
    return s


# ------------------------------------------------------------------------------------------------ plain forms --


def plan(ids, E):
    """(offsets [E + 1], pos [T, k]: a pair's row or -1, the pair of every row; pairs without an expert come last)."""
    flat = ids.flatten().long()
    key = torch.where(flat < 0, E, flat)
    pair = torch.sort(key, stable=True)[1]
    pos = torch.empty_like(pair).scatter_(0, pair, torch.arange(pair.numel(), device=ids.device))
    pos = torch.where(flat < 0, -1, pos).to(torch.int32).view_as(ids)
    count = torch.zeros(E + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = torch.cumsum(count[:E], 0)
    return offsets, pos, pair


def taken(s, rows):
    """A token's rows [T, k, H] in 32 bits, 0 where a pair has none."""
    on = (s["pos"] >= 0)[..., None]
    return torch.where(on, rows[s["pos"].clamp(min=0).long()].float(), 0.0)


def weights(s, a, b):
    """Rows a to b of all experts' weights [b - a, N, K], in 32 bits."""
    c = s["codes"][a:b]
    q = torch.stack([c & 15, c >> 4], -1).flatten(-2).float().unflatten(-1, (-1, s["g"]))
    z = 8.0 if s["z"] is None else s["z"][a:b].float()[..., None]
    return ((q - z) * s["scales"][a:b].float()[..., None]).flatten(-2)


def run(s):
    op = s["op"]
    if own:
        import moe_expert_offload_router_gb300 as M
        if op == "sort":
            rows, offsets, pos = M.moe_sort_rows(s["x"], s["ids"], s["E"], rows=s["out"], offsets=s["offsets"],
                                                 pos=s["pos"])
            return {"rows": rows, "offsets": offsets, "pos": pos}
        if op == "sort_grad":
            return M.moe_sort_rows_backward(s["d_rows"], s["pos"], d_x=s["out"])
        if op == "combine":
            return M.moe_combine_rows(s["rows_in"], s["pos"], s["w"], s["base_in"], y=s["out"])
        if op == "combine_grad":
            d_rows, d_w = M.moe_combine_rows_backward(s["d_y"], s["rows_in"], s["pos"], s["w"], d_rows=s["d_rows"],
                                                      d_w=s["d_w"])
            return {"d_rows": d_rows, "d_w": d_w}
        if s["k"]:
            return M.moe_w4_linear(s["x"], s["codes"], s["scales"], s["z"], s["offsets"], swiglu=s["swiglu"],
                                   out=s["out"])
        return M.moe_w4_linear(s["x"], s["codes"][0], s["scales"][0], None if s["z"] is None else s["z"][0],
                               swiglu=s["swiglu"], out=s["out"])
    if op == "sort":
        offsets, pos, pair = plan(s["ids"], s["E"])
        on = torch.arange(pair.numel(), device=pair.device) < offsets[-1]
        return {"rows": torch.where(on[:, None], s["x"][pair // s["k"]], 0.0), "offsets": offsets, "pos": pos}
    if op == "sort_grad":
        return taken(s, s["d_rows"]).sum(1).to(DT[s["dtype"]])
    if op == "combine":
        rows = taken(s, s["rows_in"])
        y = (rows if s["w"] is None else rows * s["w"][..., None]).sum(1)
        return (y if s["base_in"] is None else s["base_in"].float() + y).to(DT[s["y"]])
    if op == "combine_grad":
        d, P = s["d_y"].float()[:, None], s["pos"].numel()
        to = torch.where(s["pos"] < 0, P, s["pos"].long()).flatten()
        d_rows = torch.zeros(P + 1, s["H"], dtype=DT[s["rows"]], device=d.device)
        d_rows.index_copy_(0, to, (d * s["w"][..., None]).flatten(0, 1).to(d_rows.dtype))
        return {"d_rows": d_rows[:P], "d_w": (d * taken(s, s["rows_in"])).sum(-1)}
    x, out = s["x"].float(), torch.zeros_like(s["out"])
    for e in range(s["E"]):
        a, b = s["bounds"][e], s["bounds"][e + 1]
        if a < b:
            o = x[a:b] @ weights(s, e, e + 1)[0].T
            if s["swiglu"]:
                gate, up = o[:, :s["N"] // 2], o[:, s["N"] // 2:]
                o = gate / (1 + torch.exp(-gate)) * up
            out[a:b] = o.to(out.dtype)
    return out


def work(case):
    T, k = case["T"], case["k"]
    n = T * max(k, 1) * (1 - case["pad"])   # rows with an expert
    if case["op"] in ("sort", "sort_grad"):
        # every token is read (written) once, every row written (read) once
        b = SIZE[case["dtype"]] * case["H"] * (T + n) + 4 * T * k
        return {"bytes": b + (4 * T * k + 4 * case["E"] if case["op"] == "sort" else 0), "flops": n * case["H"]}
    if case["op"] in ("combine", "combine_grad"):
        H, r, y = case["H"], SIZE[case["rows"]], SIZE[case["y"]]
        if case["op"] == "combine":
            return {"bytes": n * H * r + T * H * y * (1 + case["base"]) + T * k * (4 + 4 * case["weights"]),
                    "flops": 2 * n * H}
        return {"bytes": 2 * n * H * r + T * H * y + 12 * T * k, "flops": 3 * n * H}
    K, N, z = case["K"], case["N"], SIZE[case["dtype"]]
    share = k * (1 - case["pad"]) / case["E"] if k else 1.0
    used = case["E"] * (1 - (1 - share) ** T)   # experts that balanced routing of T tokens reaches
    weight = N * K / 2 + N * (K // case["g"]) * (z + case["zeros"])
    out = N // 2 if case["swiglu"] else N
    return {"bytes": used * weight + n * (K * z + out * SIZE[case["out"]]), "flops": 2 * n * N * K}


# ------------------------------------------------------------------------------------------ in 64 bits, apart --


def exact(case, seed):
    """The definitions in 64 bits, expert by expert and rank by rank, not from the plain form above."""
    s = prepare(case, seed)
    f = torch.float64
    T, k = case["T"], case["k"]
    if case["op"] == "sort":
        rows = torch.zeros(T * k, case["H"], dtype=f, device="cuda")
        at = 0
        for e in torch.unique(s["ids"][s["ids"] >= 0]).tolist():
            token = torch.nonzero(s["ids"] == e)[:, 0]   # in the order of the pairs
            rows[at:at + token.numel()] = s["x"][token].to(f)
            at += token.numel()
        return {"rows": rows, "offsets": None, "pos": None}
    if case["op"] in ("sort_grad", "combine"):
        source = s["d_rows"] if case["op"] == "sort_grad" else s["rows_in"]
        y = torch.zeros(T, case["H"], dtype=f, device="cuda")
        if s.get("base_in") is not None:
            y += s["base_in"]
        for j in range(k):
            t = torch.nonzero(s["pos"][:, j] >= 0)[:, 0]
            part = source[s["pos"][t, j].long()].to(f)
            y[t] += part if s.get("w") is None else part * s["w"][t, j, None].to(f)
        return y
    if case["op"] == "combine_grad":
        d_rows = torch.zeros(T * k, case["H"], dtype=f, device="cuda")
        d_w = torch.zeros(T, k, dtype=f, device="cuda")
        for j in range(k):
            t = torch.nonzero(s["pos"][:, j] >= 0)[:, 0]
            r, d = s["pos"][t, j].long(), s["d_y"][t].to(f)
            d_rows[r] = d * s["w"][t, j, None].to(f)
            d_w[t, j] = torch.linalg.vecdot(d, s["rows_in"][r].to(f))
        return {"d_rows": d_rows, "d_w": d_w}
    out = torch.zeros(s["out"].shape, dtype=f, device="cuda")
    begin = 0
    for e in range(case["E"]):
        n = int((s["ids"] == e).sum()) if k else T
        if n == 0:
            continue
        W = torch.empty(case["N"], case["K"], dtype=f, device="cuda")
        W[:, 0::2] = torch.remainder(s["codes"][e], 16)
        W[:, 1::2] = torch.div(s["codes"][e], 16, rounding_mode="floor")
        W -= 8 if s["z"] is None else s["z"][e].to(f).repeat_interleave(case["g"], 1)
        W *= s["scales"][e].to(f).repeat_interleave(case["g"], 1)
        o = torch.matmul(s["x"][begin:begin + n].to(f), W.mT)
        if case["swiglu"]:
            gate, up = o.chunk(2, 1)
            o = torch.nn.functional.silu(gate) * up
        out[begin:begin + n] = o
        begin += n
    return out
