"""The operators around the routed expert layer, as cases to be timed and compared: routing to experts and its
gradient, the norms before and after the block with gate and residual scale and their gradient, and the shared
projection with low-rank adapters of many requests beside it.

Where ``own`` is false, ``run`` computes them from elementary torch operations in 32 bits; where it is true, it
makes the calls of this package."""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6


def route(name, T, E, k, score, bias=False, G=1, tg=1, group="top2", renorm=True, scale=1.0, dtype="f32", off=0,
          pad=0.0, load=False, op="route"):
    """Routing of T tokens over E experts; `off`: experts switched off by a logit of -inf, `pad`: share of padding."""
    return dict(name=name, op=op, T=T, E=E, k=k, score=score, bias=bias, G=G, tg=tg, group=group, renorm=renorm,
                scale=scale, dtype=dtype, off=off, pad=pad, load=load)


def norm(name, T, H, x, y, post=True, gate="vector", nxt=True, alpha=1.0, wide=0, w="f32", op="norm"):
    """Norms around a block of T tokens; `x`, `y`: types of the residual stream and of the block's output, `wide`:
    columns between the rows of y, `w`: the weights' type."""
    return dict(name=name, op=op, T=T, H=H, x=x, y=y, post=post, gate=gate, next=nxt, alpha=alpha, wide=wide, w=w)


def linear(name, T, H, N, r, n, order, dtype="bf16", out="bf16", wide=0):
    """A projection of T tokens with n adapters of rank r; `order`: a request for every token ("mixed") or requests
    of many tokens one after the other ("runs"); about one token or run in eight has no adapter."""
    return dict(name=name, op="linear", T=T, H=H, N=N, r=r, n=n, order=order, dtype=dtype, out=out, wide=wide)


def listed():
    return [
        # one token of the 256-expert, top-8 layer: a lone user's decode step
        route("route, one token", 1, 256, 8, "softmax"),
        # the decode batch of the headline workload under balanced routing: bias, 4 of 8 groups
        route("route, decode groups", 64, 256, 8, "sigmoid", bias=True, G=8, tg=4, scale=2.5),
        # a long prompt (or many) with padding at its end, router logits in 16 bits, load counted for the balance bias
        route("route, prompt groups", 32768, 256, 8, "sigmoid", bias=True, G=8, tg=4, scale=2.5, dtype="bf16",
              pad=0.03, load=True),
        # the router's gradient for one training batch, top-6
        route("route gradient", 16384, 256, 6, "sigmoid", scale=2.5, op="route_grad"),
        # a decode batch through one block of the 43-layer stack
        norm("norm, decode", 16, 4096, "bf16", "bf16"),
        # a prompt of the prefill workload
        norm("norm, prompt", 8192, 4096, "bf16", "bf16", alpha=0.5),
        # ragged: the stream kept in 32 bits, a width that no vector divides, a gate for each token
        norm("norm, ragged", 1021, 1001, "f32", "bf16", gate="token", w="bf16"),
        # training: the gradient of one block's norms over a batch
        norm("norm gradient", 8192, 4096, "bf16", "bf16", op="norm_grad"),
        # the router's projection for a decode batch, each token its own request
        linear("gate, decode", 16, 4096, 256, 16, 8, "mixed", out="f32"),
        # a dense projection to the intermediate size for the T = 64 decode batch, 32 adapters in it
        linear("projection, decode", 64, 4096, 2048, 16, 32, "mixed"),
        # the router's projection of the T = 8192 prefill batch
        linear("gate, prompt", 8192, 4096, 256, 16, 8, "runs", out="f32"),
        # a dense projection of several prompts, none of them a multiple of a tile
        linear("projection, prompt", 4001, 4096, 4096, 32, 8, "runs"),
    ]


def spread(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["route", "route", "route_grad", "norm", "norm", "norm_grad", "linear", "linear", "linear"])
    if op in ("route", "route_grad"):
        G = rng.choice([1, 1, 2, 4, 8])
        E = G * spread(rng, 8, 1024 // G if G == 1 else 64)
        T = spread(rng, 1, (16384 if op == "route_grad" else 32768) * 256 // max(E, 256))
        tg = rng.randint(1, G)
        k = rng.randint(1, min(12, tg * (E // G)))
        c = route("", T, E, k, rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, G=G, tg=tg,
                  group=rng.choice(["top2", "max"]), renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]),
                  dtype=rng.choice(["f32", "f32", "bf16", "f16"]), off=rng.choice([0, 0, E // 5]),
                  pad=rng.choice([0.0, 0.1]), load=op == "route" and rng.random() < 0.3, op=op)
    elif op in ("norm", "norm_grad"):
        H = rng.choice([4096, 2048, 8 * spread(rng, 8, 1024), spread(rng, 64, 8192)])
        T = spread(rng, 1, 8192 * 4096 // max(H, 4096))
        x, y = rng.choice([("bf16", "bf16"), ("f16", "f16"), ("f32", "bf16"), ("f32", "f16"), ("f32", "f32")])
        if x == "f32":
            T = max(1, T // 2)
        c = norm("", T, H, x, y, post=rng.random() < 0.7, gate=rng.choice(["none", "vector", "token"]),
                 nxt=rng.random() < 0.8, alpha=rng.choice([1.0, 0.5, 0.22]), wide=rng.choice([0, 0, 64, 7]),
                 w=rng.choice(["f32", x]), op=op)
    else:
        T = spread(rng, 1, 8192)
        H = rng.choice([4096, 2048, 8 * spread(rng, 32, 1024)])
        N = rng.choice([256, 2048, 4096, spread(rng, 32, 4096)])
        most = 4001 * 4096 * 4096
        while T * H * N > most:
            T = max(1, most // (H * N))
        c = linear("", T, H, N, 8 * rng.randint(1, 8), spread(rng, 1, 48), "runs" if T > 256 else "mixed",
                   dtype=rng.choice(["bf16", "bf16", "f16"]), out=rng.choice(["same", "f32"]),
                   wide=rng.choice([0, 0, 64]))
        c["out"] = c["dtype"] if c["out"] == "same" else "f32"
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

    s = dict(case)
    T = case["T"]
    if case["op"] in ("route", "route_grad"):
        E, k, dt = case["E"], case["k"], DT[case["dtype"]]
        logits = normal(T, E, by=1.5) + normal(1, E, by=0.5)
        if case["off"]:
            logits[:, torch.randperm(E, device="cuda", generator=g)[:case["off"]]] = -math.inf
        s["logits"] = logits.to(dt)
        s["mask"] = None
        if case["pad"]:
            s["mask"] = (uniform(T) >= case["pad"]).to(torch.uint8)
            s["logits"][s["mask"] == 0] = math.nan   # what padding holds is not to matter
        # a bias moves by steps of 0.001 towards balance
        s["b"] = torch.round(normal(E, by=40.0)) * 0.001 if case["bias"] else None
        s["ids"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
        s["w"] = torch.empty(T, k, device="cuda")
        s["count"] = torch.zeros(E, dtype=torch.int32, device="cuda") if case["load"] else None
        if case["op"] == "route_grad":
            s["ids"].copy_(choose(s)[0])
            s["dw"] = normal(T, k, by=0.1)
            s["dlogits"] = torch.empty(T, E, dtype=dt, device="cuda")
    elif case["op"] in ("norm", "norm_grad"):
        H, xd, yd, wd = case["H"], DT[case["x"]], DT[case["y"]], DT[case["w"]]
        s["xs"] = normal(T, H, dtype=xd, by=2.0)
        s["ys"] = normal(T, H + case["wide"], dtype=yd, by=0.3)[:, :H]
        s["gp"] = (1.0 + normal(H, by=0.1)).to(wd) if case["post"] else None
        s["gn"] = (1.0 + normal(H, by=0.1)).to(wd) if case["next"] else None
        s["gt"] = {"none": None, "vector": normal(H, by=0.5).to(wd), "token": uniform(T, 1).to(wd)}[case["gate"]]
        if case["op"] == "norm":
            s["xo"] = torch.empty(T, H, dtype=xd, device="cuda")
            s["h"] = torch.empty(T, H, dtype=yd, device="cuda") if case["next"] else None
        else:
            s["du"] = normal(T, H, dtype=xd, by=0.02)
            s["dh"] = normal(T, H, dtype=yd, by=0.02) if case["next"] else None
            s["dx"] = torch.empty(T, H, dtype=xd, device="cuda")
            s["dy"] = torch.empty(T, H, dtype=yd, device="cuda")
    else:
        H, N, r, n, dt = case["H"], case["N"], case["r"], case["n"], DT[case["dtype"]]
        s["xs"] = normal(T, H + case["wide"], dtype=dt)[:, :H]
        s["W"] = normal(N, H, dtype=dt, by=H ** -0.5)
        s["A"] = normal(n, r, H, dtype=dt, by=H ** -0.5)
        s["B"] = normal(n, N, r, dtype=dt, by=0.3 * r ** -0.5)
        s["c"] = 0.5 + uniform(n)
        if case["order"] == "mixed":
            a = torch.randint(0, n, (T,), device="cuda", generator=g)
            s["a"] = torch.where(uniform(T) < 0.125, -1, a).to(torch.int32)
        else:
            run = torch.cumsum((uniform(T) < 16.0 / T).to(torch.int64), 0)   # about 16 requests
            of = torch.randint(0, n, (T + 1,), device="cuda", generator=g)
            of = torch.where(uniform(T + 1) < 0.125, -1, of)
            s["a"] = of[run].to(torch.int32)
        s["o"] = torch.empty(T, N, dtype=DT[case["out"]], device="cuda")
    return s


# ------------------------------------------------------------------------------------------------ plain forms --


def pair_sum(v):
    """The sum over the last axis in neighbouring pairs: the order that the softmax's denominator is defined in."""
    n = 1 << (v.shape[-1] - 1).bit_length()
    v = torch.nn.functional.pad(v, (0, n - v.shape[-1]))
    while v.shape[-1] > 1:
        v = v[..., 0::2] + v[..., 1::2]
    return v[..., 0]


def scores(s, wide=torch.float32):
    """(logits with -inf where an expert cannot be taken, scores) in `wide`."""
    z = s["logits"].to(wide)
    out = torch.isnan(z)
    if s["mask"] is not None:
        out = out | (s["mask"] == 0)[:, None]
    z = torch.where(out, -math.inf, z)
    if s["score"] == "sigmoid":
        return z, 1 / (1 + torch.exp(-z))
    top = z.amax(-1, keepdim=True)
    e = torch.where(z == -math.inf, 0.0, torch.exp(z - top))
    den = (pair_sum(e) if wide == torch.float32 else e.sum(-1))[:, None]
    return z, torch.where(den > 0, e / den, 0.0)


def choose(s, wide=torch.float32):
    """(ids with -1 where no expert is left, scores of the chosen, 0 there)."""
    T, E, k, G = s["T"], s["E"], s["k"], s["G"]
    z, p = scores(s, wide)
    can = z > -math.inf
    key = z if s["b"] is None else torch.where(can, p + s["b"].to(wide), -math.inf)
    if s["tg"] < G:
        if s["group"] == "max":
            worth = key.view(T, G, E // G).amax(-1)
        else:
            v = torch.where(can, p if s["b"] is None else key, -math.inf).view(T, G, E // G)
            two = torch.sort(v, dim=-1, descending=True)[0][..., :2]
            two = torch.where(two[..., :1] == -math.inf, two, torch.where(two == -math.inf, 0.0, two))
            worth = two.sum(-1)
        best = torch.sort(worth, dim=-1, descending=True, stable=True)[1][:, :s["tg"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=z.device).scatter_(1, best, True)
        key = torch.where(keep.repeat_interleave(E // G, 1), key, -math.inf)
    val, ids = torch.sort(key, dim=-1, descending=True, stable=True)
    val, ids = val[:, :k], ids[:, :k]
    none = val == -math.inf
    return torch.where(none, -1, ids).to(torch.int32), torch.where(none, 0.0, p.gather(1, ids))


def weights(s, wide=torch.float32):
    ids, p = choose(s, wide)
    if s["renorm"]:
        den = p.sum(-1, keepdim=True)
        p = torch.where(den > 0, p / den, 0.0)
    return ids, s["scale"] * p


def route_gradient(s, wide=torch.float32):
    """d logits of the weights, for given ids."""
    z, p = scores(s, wide)
    ids = s["ids"].long()
    on = ids >= 0
    at = ids.clamp(min=0)
    gr = torch.where(on, s["dw"].to(wide), 0.0) * s["scale"]
    pj = torch.where(on, p.gather(1, at), 0.0)
    sharp = 1 / (1 + torch.exp(z.gather(1, at))) if s["score"] == "sigmoid" else 1.0   # 1 - sigmoid
    d = torch.zeros_like(z)
    if s["renorm"]:
        den = pj.sum(-1, keepdim=True)
        q = torch.where(den > 0, pj / den, 0.0)
        dj = q * sharp * (gr - (q * gr).sum(-1, keepdim=True))
    elif s["score"] == "sigmoid":
        dj = pj * sharp * gr
    else:
        dj = pj * gr
        d = -p * dj.sum(-1, keepdim=True)
    return d.scatter_add_(1, at, torch.where(on, dj, 0.0))


def block(s, wide=torch.float32):
    """(y^, r_y, v, u, r_u) of the block's norms."""
    x, y = s["xs"].to(wide), s["ys"].to(wide)
    ry = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) if s["post"] else 1.0
    yn = y * ry
    v = yn * s["gp"].to(wide) if s["post"] else yn
    u = s["alpha"] * x + (v if s["gt"] is None else s["gt"].to(wide) * v)
    return yn, ry, v, u, torch.rsqrt((u * u).mean(-1, keepdim=True) + EPS)


def block_gradient(s, wide=torch.float32):
    yn, ry, v, u, ru = block(s, wide)
    un = u * ru
    du, d = s["du"].to(wide), {}
    if s["next"]:
        dh = s["dh"].to(wide)
        a = dh * s["gn"].to(wide)
        du = du + ru * (a - un * (a * un).mean(-1, keepdim=True))
        d["next"] = (dh * un).sum(0)
    dv = du
    if s["gt"] is not None:
        dv = du * s["gt"].to(wide)
        d["gate"] = (du * v).sum(0) if s["gate"] == "vector" else (du * v).sum(-1, keepdim=True)
    dy = dv
    if s["post"]:
        b = dv * s["gp"].to(wide)
        d["post"] = (dv * yn).sum(0)
        dy = ry * (b - yn * (b * yn).mean(-1, keepdim=True))
    return {"dx": s["alpha"] * du, "dy": dy, **d}


def project(s, wide=torch.float32):
    T, H, N, r, n = (s[m] for m in ("T", "H", "N", "r", "n"))
    x = s["xs"].to(wide)
    low = (x @ s["A"].to(wide).view(n * r, H).T).view(T, n, r)
    mine = s["a"][:, None] == torch.arange(n, device=x.device, dtype=torch.int32)
    low = low * (mine * s["c"].to(wide))[..., None]
    return x @ s["W"].to(wide).T + low.view(T, n * r) @ s["B"].to(wide).transpose(1, 2).reshape(n * r, N)


# ---------------------------------------------------------------------------------------------------- one pass --


def run(s):
    op = s["op"]
    if own:
        import moe_expert_offload_router_gb300 as M
        if op in ("route", "route_grad"):
            score = M.MOE_SCORE_SIGMOID if s["score"] == "sigmoid" else M.MOE_SCORE_SOFTMAX
            if op == "route_grad":
                return M.moe_route_backward(s["logits"], s["ids"], s["dw"], score=score, renorm=s["renorm"],
                                            scale=s["scale"], token_mask=s["mask"], d_logits=s["dlogits"])
            if s["load"]:
                s["count"].zero_()
            M.moe_route(s["logits"], s["k"], score=score, bias=s["b"], n_group=s["G"], topk_group=s["tg"],
                        group_score=M.MOE_GROUP_TOP2 if s["group"] == "top2" else M.MOE_GROUP_MAX,
                        renorm=s["renorm"], scale=s["scale"], token_mask=s["mask"], topk_ids=s["ids"],
                        topk_w=s["w"], load=s["count"])
            return {"ids": s["ids"], "w": s["w"], "load": s["count"]}
        if op == "norm":
            x, h = M.moe_block_norm(s["xs"], s["ys"], post_weight=s["gp"], gate=s["gt"], residual_scale=s["alpha"],
                                    next_weight=s["gn"], eps=EPS, x_out=s["xo"], h=s["h"])
            return {"x": x, "h": h}
        if op == "norm_grad":
            dx, dy, dp, dg, dn = M.moe_block_norm_backward(
                s["xs"], s["ys"], s["du"], s["dh"], post_weight=s["gp"], gate=s["gt"], residual_scale=s["alpha"],
                next_weight=s["gn"], eps=EPS, d_x=s["dx"], d_y=s["dy"])
            return {"dx": dx, "dy": dy, "post": dp, "gate": dg, "next": dn}
        return M.moe_adapter_linear(s["xs"], s["W"], s["A"], s["B"], s["a"], s["c"], out=s["o"])
    if op == "route":
        ids, w = weights(s)
        load = torch.bincount(ids[ids >= 0], minlength=s["E"]).to(torch.int32) if s["load"] else None
        return {"ids": ids, "w": w, "load": load}
    if op == "route_grad":
        return route_gradient(s).to(s["logits"].dtype)
    if op == "norm":
        _, _, _, u, ru = block(s)
        h = (u * ru * s["gn"].float()).to(DT[s["y"]]) if s["next"] else None
        return {"x": u.to(DT[s["x"]]), "h": h}
    if op == "norm_grad":
        d = block_gradient(s)
        return {"dx": d["dx"].to(DT[s["x"]]), "dy": d["dy"].to(DT[s["y"]]),
                **{m: d.get(m) for m in ("post", "gate", "next")}}
    return project(s).to(DT[s["out"]])


def work(case):
    T = case["T"]
    if case["op"] in ("route", "route_grad"):
        E, k, z = case["E"], case["k"], SIZE[case["dtype"]]
        if case["op"] == "route":
            return {"bytes": T * (E * z + 8 * k) + (4 * E if case["bias"] else 0) + (4 * E if case["load"] else 0),
                    "flops": T * E * 4}
        read = E if case["score"] == "softmax" and not case["renorm"] else min(E, k)
        return {"bytes": T * (E * z + read * z + 8 * k), "flops": T * (E + 10 * k)}
    if case["op"] in ("norm", "norm_grad"):
        H, x, y, w = case["H"], SIZE[case["x"]], SIZE[case["y"]], SIZE[case["w"]]
        vec = H * (case["post"] + case["next"] + (case["gate"] == "vector"))
        if case["op"] == "norm":
            return {"bytes": T * H * (2 * x + y + case["next"] * y) + vec * w, "flops": 10 * T * H}
        return {"bytes": T * H * (3 * x + 2 * y + case["next"] * y) + vec * (w + 4), "flops": 30 * T * H}
    H, N, r, z = case["H"], case["N"], case["r"], SIZE[case["dtype"]]
    used = min(case["n"], T)
    return {"bytes": z * (T * H + N * H + used * r * (H + N)) + T * N * SIZE[case["out"]] + 4 * T,
            "flops": 2 * T * N * H + 2 * T * r * (H + N)}


# ------------------------------------------------------------------------------------------ in 64 bits, apart --


def exact(case, seed):
    """The definitions in 64 bits, written row by row of the formula and not from the plain form above."""
    s = prepare(case, seed)
    f = torch.float64
    if case["op"] in ("route", "route_grad"):
        E, k, G = case["E"], case["k"], case["G"]
        z = s["logits"].to(f)
        z = torch.where(torch.isnan(z), torch.full_like(z, -math.inf), z)
        if s["mask"] is not None:
            z = z.masked_fill((s["mask"] == 0)[:, None], -math.inf)
        can = torch.isfinite(z)
        p = torch.sigmoid(z) if case["score"] == "sigmoid" else torch.nan_to_num(torch.softmax(z, -1), nan=0.0)
        if case["op"] == "route_grad":
            leaf = torch.where(can, z, torch.full_like(z, -700.0)).requires_grad_(True)
            q = torch.sigmoid(leaf) if case["score"] == "sigmoid" else torch.softmax(leaf, -1)
            on = s["ids"] >= 0
            q = q.gather(1, s["ids"].long().clamp(min=0)) * on
            if case["renorm"]:
                q = q / q.sum(-1, keepdim=True).clamp(min=1e-300)
            q.backward(case["scale"] * s["dw"].to(f) * on)
            return leaf.grad * can
        rank = z if s["b"] is None else (p + s["b"].to(f)).masked_fill(~can, -math.inf)
        if case["tg"] < G:
            of = (rank if case["group"] == "max" or s["b"] is not None else p.masked_fill(~can, -math.inf))
            of = of.unflatten(1, (G, E // G)).topk(min(2, E // G), -1)[0]
            worth = of[..., 0]
            if case["group"] == "top2" and of.shape[-1] == 2:
                worth = worth + of[..., 1].clamp(min=-1e30).masked_fill(of[..., 1] == -math.inf, 0.0)
            order = torch.argsort(worth, dim=1, descending=True, stable=True)
            place = torch.argsort(order, dim=1)
            rank = rank.masked_fill((place >= case["tg"]).repeat_interleave(E // G, 1), -math.inf)
        at = torch.argsort(rank, dim=1, descending=True, stable=True)[:, :k]
        q = p.gather(1, at).masked_fill(rank.gather(1, at) == -math.inf, 0.0)
        if case["renorm"]:
            q = q / q.sum(-1, keepdim=True).clamp(min=1e-300)
        return {"ids": None, "w": case["scale"] * q, "load": None}
    if case["op"] in ("norm", "norm_grad"):
        t = {m: s[m].to(f) if s[m] is not None else None for m in ("xs", "ys", "gp", "gn", "gt")}
        if case["op"] == "norm_grad":
            t = {m: None if v is None else v.detach().requires_grad_(True) for m, v in t.items()}
        v = t["ys"]
        if t["gp"] is not None:
            v = v / torch.sqrt(v.pow(2).mean(1, keepdim=True) + EPS) * t["gp"]
        u = t["xs"] * case["alpha"] + (v if t["gt"] is None else v * t["gt"])
        h = None if t["gn"] is None else u / torch.sqrt(u.pow(2).mean(1, keepdim=True) + EPS) * t["gn"]
        if case["op"] == "norm":
            return {"x": u, "h": h}
        total = (u * s["du"].to(f)).sum()
        if h is not None:
            total = total + (h * s["dh"].to(f)).sum()
        total.backward()
        grad = {m: None if v is None else v.grad for m, v in t.items()}
        return {"dx": grad["xs"], "dy": grad["ys"], "post": grad["gp"], "gate": grad["gt"], "next": grad["gn"]}
    out = torch.empty(case["T"], case["N"], dtype=f, device="cuda")
    x, W = s["xs"].to(f), s["W"].to(f)
    torch.matmul(x, W.T, out=out)
    for a in range(case["n"]):
        rows = torch.nonzero(s["a"] == a)[:, 0]
        if rows.numel():
            out[rows] += float(s["c"][a]) * ((x[rows] @ s["A"][a].to(f).T) @ s["B"][a].to(f).T)
    return out
