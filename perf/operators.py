"""The layer's training operators on inputs as they occur: group-limited
routing, its gradient, and the Newton-Schulz orthogonalisation of weight
gradients.

``listed()`` gives the cases that are timed, ``draw()`` further ones of the
same ranges; ``run()`` is one pass, in plain torch operations (``own`` false)
or through the library's entry points (``own`` true), and ``exact()`` the same
outputs from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

F32, BF16 = "f32", "bf16"
_TORCH = {F32: torch.float32, BF16: torch.bfloat16}
_SIZE = {F32: 4, BF16: 2}
COEFFS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7
INF = float("inf")


# ---------------------------------------------------------------- the cases
def _route(name, op, T, E, k, groups, topk_group, group_score=2, gate="sigmoid", space=1,
           norm=True, scale=1.0, dtype=F32, bias=True, padded=0.0, disabled=0, pad_cols=0):
    """A routing call: op "route" or "route_bwd"; groups consecutive expert
    groups of which a token uses topk_group; padded: share of padding tokens;
    disabled: experts switched off by a bias of -inf; pad_cols: columns behind
    each row's logits (a row stride above E)."""
    return dict(name=name, op=op, T=T, E=E, k=k, groups=groups, topk_group=topk_group,
                group_score=group_score, gate=gate, space=space, norm=norm, scale=scale,
                dtype=dtype, bias=bias, padded=padded, disabled=disabled, pad_cols=pad_cols)


def _ortho(name, batch, rows, cols, dtype=BF16, out=BF16, steps=5, rank=0):
    """An orthogonalised batch of gradients [batch, rows, cols]; rank > 0: the
    gradients have that many strong directions over a weak full-rank part."""
    return dict(name=name, op="ortho", batch=batch, rows=rows, cols=cols, dtype=dtype, out=out,
                steps=steps, rank=rank)


def listed():
    return [
        # one token of a decode step, 64 experts in 8 groups
        _route("route_one_token", "route", 1, 64, 6, 8, 3, scale=2.5),
        # a decode batch with bf16 gate outputs, groups ranked by their best expert
        _route("route_decode_batch", "route", 200, 160, 6, 8, 3, group_score=1, gate="softmax",
               norm=False, scale=16.0, dtype=BF16, bias=False),
        # the 128-expert top-8 layer's 16384 tokens
        _route("route_train", "route", 16384, 128, 8, 8, 4, scale=1.0),
        # a long prefill of padded sequences, 256 experts, two switched off
        _route("route_long", "route", 131072, 256, 8, 8, 4, scale=2.5, padded=0.1, disabled=2),
        # odd token count, bf16 logits in a wider buffer, softmax gate
        _route("route_bwd_odd", "route_bwd", 4099, 96, 6, 6, 2, gate="softmax", dtype=BF16,
               pad_cols=8, padded=0.05),
        # gradient of the 16384-token layer's routing
        _route("route_bwd_train", "route_bwd", 16384, 128, 8, 8, 4, gate="softmax"),
        # gradient of the long one
        _route("route_bwd_long", "route_bwd", 131072, 256, 8, 8, 4, scale=2.5, padded=0.1),
        # the router weight's fp32 gradient [E, d] of the 128-expert layer
        _ortho("ortho_router", 1, 128, 2048, dtype=F32, out=F32),
        # odd sizes, fp32 in and out
        _ortho("ortho_odd", 3, 333, 517, dtype=F32, out=F32, rank=24),
        # the 16-expert d = 640 layer's down weights (stored taller than wide)
        _ortho("ortho_experts16", 16, 1024, 640, rank=40),
        # the 128-expert layer's gate weights
        _ortho("ortho_experts128", 128, 768, 2048, rank=64),
        # wide experts' down weights, four experts at a time, from an fp32 momentum
        _ortho("ortho_wide", 4, 5120, 4352, dtype=F32, rank=200),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "route_bwd", "route_bwd", "ortho", "ortho"])
    if op != "ortho":
        T = _log_int(rng, 1, 131072)
        groups = rng.choice([1, 2, 4, 6, 8, 16])
        per = rng.randint(2, 256 // groups) if groups > 1 else rng.randint(8, 256)
        E = groups * per
        topk_group = rng.randint(1, groups)
        k = rng.randint(1, min(16, topk_group * per))
        gate = rng.choice(["sigmoid", "softmax"])
        space = rng.choice([0, 1])
        case = _route(None, op, T, E, k, groups, topk_group, group_score=rng.choice([1, 2]),
                      gate=gate, space=space, norm=rng.choice([True, True, False]),
                      scale=rng.choice([1.0, 2.5, 16.0]), dtype=rng.choice([F32, BF16]),
                      bias=rng.choice([True, False]), padded=rng.choice([0.0, 0.1]),
                      disabled=rng.choice([0, 0, 1, 3]), pad_cols=rng.choice([0, 0, 3, 8]))
        if not case["bias"]:
            case["disabled"] = 0
    else:
        batch = _log_int(rng, 1, 64)
        side = _log_int(rng, 16, 2600)
        other = _log_int(rng, max(16, side // 4), min(5120, side * 4))
        rows, cols = (side, other) if rng.random() < 0.5 else (other, side)
        # no more work than the largest listed case
        m, n = min(rows, cols), max(rows, cols)
        batch = max(1, min(batch, int(4 * 4352 * 4352 * 5120 / (3.0 * m * m * n)),
                           int(2.0e8 / (rows * cols))))
        out = rng.choice([BF16, BF16, F32])
        case = _ortho(None, batch, rows, cols, dtype=rng.choice([BF16, F32]), out=out,
                      steps=rng.choice([3, 5, 5, 6]), rank=rng.choice([0, max(1, m // 16)]))
    del case["name"]
    return case


# --------------------------------------------------------------- the inputs
def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 2654435761 % (1 << 40) + 17)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float32)
    uni = lambda *s: torch.rand(*s, generator=g, device="cuda", dtype=torch.float32)
    if case["op"] == "ortho":
        b, r, c = case["batch"], case["rows"], case["cols"]
        G = rnd(b, r, c)
        if case["rank"]:
            # decaying strong directions over noise, as accumulated gradients have
            q = case["rank"]
            s = 6.0 * torch.exp(-3.0 * torch.arange(q, device="cuda", dtype=torch.float32) / q)
            G = G * 0.5 + torch.matmul(rnd(b, r, q) * s, rnd(b, q, c)) / math.sqrt(q)
        return {"g": (G * 1e-3).to(_TORCH[case["dtype"]]).contiguous()}
    T, E, k = case["T"], case["E"], case["k"]
    # token logits around a per-expert popularity
    full = torch.zeros(T, E + case["pad_cols"], device="cuda", dtype=torch.float32)
    full[:, :E] = 1.2 * rnd(T, E) + 0.6 * rnd(E)
    full = full.to(_TORCH[case["dtype"]])
    d = {"logits": full[:, :E], "bias": None, "mask": None}
    if case["bias"]:
        d["bias"] = 0.2 * (uni(E) - 0.5)
        if case["disabled"]:
            # spread over the groups, so that none loses all its experts
            d["bias"][[(i * (E // case["groups"] + 1)) % E for i in range(case["disabled"])]] = -INF
    if case["padded"] > 0:
        d["mask"] = (uni(T) >= case["padded"]).to(torch.uint8)
    if case["op"] == "route_bwd":
        d["idx"] = _plain_route(case, d)[0]
        d["dw"] = rnd(T, k)
    return d


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case
    if not own:
        return st
    from mixture_experts_ffn_bias_b200 import binding as B
    code = {F32: B.DTYPE_F32, BF16: B.DTYPE_BF16}
    if case["op"] == "ortho":
        st["cfg"] = B.make_ortho_config(case["batch"], case["rows"], case["cols"],
                                        in_dtype=code[case["dtype"]], out_dtype=code[case["out"]],
                                        steps=case["steps"], coeffs=COEFFS, eps=EPS)
        st["ws"] = torch.empty(max(256, B.moe_orthogonalize_workspace_size(st["cfg"])),
                               dtype=torch.uint8, device="cuda")
        st["out"] = torch.empty(st["g"].shape, dtype=_TORCH[case["out"]], device="cuda")
        return st
    T, E, k = case["T"], case["E"], case["k"]
    st["cfg"] = B.make_config(T, 128, E, 128, k, norm_topk_prob=int(case["norm"]),
                              gate=B.GATE_SIGMOID if case["gate"] == "sigmoid" else B.GATE_SOFTMAX)
    st["opts"] = B.make_group_opts(case["groups"], case["topk_group"], case["group_score"],
                                   bias_space=case["space"], scale=case["scale"],
                                   logits_dtype=code[case["dtype"]])
    if case["op"] == "route":
        st["idx"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
        st["w"] = torch.empty(T, k, dtype=torch.float32, device="cuda")
    else:
        st["dlogits"] = torch.empty(T, E, dtype=_TORCH[case["dtype"]], device="cuda")
    return st


# ------------------------------------------------------------- one pass each
def run(st):
    case = st["case"]
    if own:
        from mixture_experts_ffn_bias_b200 import binding as B
        if case["op"] == "ortho":
            B.moe_orthogonalize(st["cfg"], st["g"], st["out"], st["ws"])
            return st["out"]
        if case["op"] == "route":
            B.moe_route_groups(st["cfg"], st["opts"], st["logits"], st["bias"], st["mask"],
                               st["idx"], st["w"])
            return st["idx"], st["w"]
        B.moe_route_groups_backward(st["cfg"], st["opts"], st["logits"], st["idx"], st["dw"],
                                    st["dlogits"])
        return st["dlogits"]
    if case["op"] == "ortho":
        return _plain_ortho(case, st)
    if case["op"] == "route":
        return _plain_route(case, st)
    return _plain_route_bwd(case, st)


def _scores(l, gate):
    if gate == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    m = l.max(dim=1, keepdim=True).values
    e = torch.exp(l - torch.where(m == -INF, torch.zeros_like(m), m))
    return e / e.sum(dim=1, keepdim=True)


def _plain_route(case, st):
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    # keys in 64 bits: near a border 32 would order two experts wrongly
    l = st["logits"].double()
    s = _scores(l, case["gate"])
    key = s if case["space"] == 1 else l
    if st["bias"] is not None:
        key = key + st["bias"].double()
    ok = (l > -INF) & (s == s) & (key > -INF)
    if st["mask"] is not None:
        ok = ok & (st["mask"] != 0)[:, None]
    key = torch.where(ok, key, torch.full_like(key, -INF))
    if G > 1:
        best = torch.sort(key.view(T, G, E // G), dim=2, descending=True).values
        gs = best[:, :, 0]
        if case["group_score"] == 2:
            two = best[:, :, 1]
            gs = torch.where(two > -INF, gs + two, gs)
        order = torch.sort(gs, dim=1, descending=True, stable=True).indices
        use = torch.zeros(T, G, dtype=torch.bool, device=key.device)
        use.scatter_(1, order[:, :case["topk_group"]], True)
        key = torch.where(use.repeat_interleave(E // G, dim=1), key, torch.full_like(key, -INF))
    vals, idx = torch.sort(key, dim=1, descending=True, stable=True)
    vals, idx = vals[:, :k], idx[:, :k]
    hit = vals > -INF
    w = torch.where(hit, s.gather(1, idx), torch.zeros_like(vals)).float()
    if case["norm"]:
        w = w / (w.sum(dim=1, keepdim=True) + 1e-9)
    w = w * case["scale"]
    return torch.where(hit, idx, torch.full_like(idx, -1)).int(), w


def _plain_route_bwd(case, st):
    # in 64 bits: the renormalised weights' gradient cancels almost wholly for
    # one expert a token
    l = st["logits"].double()
    s = _scores(l, case["gate"])
    idx = st["idx"].long()
    hit = idx >= 0
    at = idx.clamp(min=0)
    sj = torch.where(hit, s.gather(1, at), torch.zeros((), dtype=s.dtype, device=s.device))
    dw = torch.where(hit, st["dw"].double(), torch.zeros((), dtype=s.dtype, device=s.device))
    c = float(np.float32(case["scale"]))
    if case["norm"]:
        D = sj.sum(dim=1, keepdim=True) + 1e-9
        ds = c * (dw - (dw * sj).sum(dim=1, keepdim=True) / D) / D
    else:
        ds = c * dw
    ds = torch.where(hit, ds, torch.zeros_like(ds))
    full = torch.zeros_like(s).scatter_add_(1, at, ds)
    if case["gate"] == "sigmoid":
        dl = full * s * (1.0 - s)
    else:
        dl = s * (full - (full * s).sum(dim=1, keepdim=True))
    return dl.to(st["logits"].dtype)


def _plain_ortho(case, st):
    X = st["g"].float()
    tall = case["rows"] > case["cols"]
    if tall:
        X = X.transpose(1, 2)
    norm = torch.sqrt((X * X).sum(dim=(1, 2), keepdim=True, dtype=torch.float64)).float()
    X = X / (norm + EPS)
    a, b, c = COEFFS
    for _ in range(case["steps"]):
        A = torch.matmul(X, X.transpose(1, 2))
        X = a * X + torch.matmul(b * A + c * torch.matmul(A, A), X)
    if tall:
        X = X.transpose(1, 2)
    return X.to(_TORCH[case["out"]]).contiguous()


# ------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "ortho":
        b, m = case["batch"], min(case["rows"], case["cols"])
        n = max(case["rows"], case["cols"])
        # X X^T and A A^T are symmetric: half of each is enough
        step = float(m) * m * n + float(m) ** 3 + 2.0 * m * m * n
        return {"bytes": b * m * n * (_SIZE[case["dtype"]] + _SIZE[case["out"]]),
                "flops": b * case["steps"] * step}
    T, E, k, es = case["T"], case["E"], case["k"], _SIZE[case["dtype"]]
    mask = T if case["padded"] > 0 else 0
    if case["op"] == "route":
        return {"bytes": T * E * es + T * k * 8 + mask + (4 * E if case["bias"] else 0),
                "flops": 12 * T * E}
    read = T * E * es if case["gate"] == "softmax" else T * k * es
    return {"bytes": read + T * k * 8 + T * E * es, "flops": 8 * T * E}


# --------------------------------------------- the definitions, in 64 bits
def _np_scores(l, gate):
    with np.errstate(all="ignore"):
        if gate == "sigmoid":
            return np.reciprocal(1.0 + np.exp(-l))
        e = np.exp(l - l.max(axis=1, keepdims=True))
        return e / e.sum(axis=1, keepdims=True)


def _exact_route(case, st):
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    l = st["logits"].double().cpu().numpy()
    s = _np_scores(l, case["gate"])
    key = (s if case["space"] == 1 else l).copy()
    if st["bias"] is not None:
        key += st["bias"].double().cpu().numpy()[None, :]
    if st["mask"] is not None:
        key[st["mask"].cpu().numpy() == 0] = -INF
    key[~((l > -INF) & (key > -INF))] = -INF
    per = E // G
    if G > 1:
        part = np.sort(key.reshape(T, G, per), axis=2)
        gs = part[:, :, -1].copy()
        if case["group_score"] == 2 and per > 1:
            second = part[:, :, -2]
            gs += np.where(second == -INF, 0.0, second)
        # rank of a group: how many come before it
        before = ((gs[:, None, :] > gs[:, :, None]) |
                  ((gs[:, None, :] == gs[:, :, None]) &
                   (np.arange(G)[None, :] < np.arange(G)[:, None])[None])).sum(axis=2)
        key[np.repeat(before >= case["topk_group"], per, axis=1)] = -INF
    idx = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    rows = np.arange(T)
    for j in range(k):
        e = key.argmax(axis=1)              # numpy: the first of equals
        live = key[rows, e] > -INF
        idx[live, j] = e[live]
        w[live, j] = s[rows, e][live]
        key[rows, e] = -INF
    if case["norm"]:
        w /= w.sum(axis=1, keepdims=True) + 1e-9
    return torch.from_numpy(idx), torch.from_numpy(w * float(np.float32(case["scale"])))


def _exact_route_bwd(case, st):
    l = st["logits"].double().cpu().numpy()
    idx = st["idx"].cpu().numpy()
    dw = st["dw"].double().cpu().numpy()
    s = _np_scores(l, case["gate"])
    T, k = idx.shape
    rows = np.arange(T)
    c = float(np.float32(case["scale"]))
    dl = np.zeros_like(s)
    sj = np.stack([np.where(idx[:, j] >= 0, s[rows, idx[:, j]], 0.0) for j in range(k)], axis=1)
    D = sj.sum(axis=1) + 1e-9
    mix = np.zeros(T)
    for j in range(k):
        on = idx[:, j] >= 0
        if case["norm"]:
            # sum_i s_i (dw_j - dw_i) + 1e-9 dw_j, over D^2
            num = 1e-9 * dw[:, j]
            for i in range(k):
                num = num + sj[:, i] * (dw[:, j] - dw[:, i]) * (idx[:, i] >= 0)
            ds = c * num / D ** 2
        else:
            ds = c * dw[:, j]
        ds = np.where(on, ds, 0.0)
        if case["gate"] == "sigmoid":
            lj = l[rows, idx[:, j]]
            ds = ds * np.exp(-np.abs(lj)) / (1.0 + np.exp(-np.abs(lj))) ** 2
        else:
            mix += ds * sj[:, j]
            ds = ds * sj[:, j]
        dl[rows[on], idx[on, j]] += ds[on]
    if case["gate"] == "softmax":
        dl -= s * mix[:, None]
    return torch.from_numpy(dl)


def _exact_ortho(case, st):
    outs = []
    a, b, c = COEFFS
    for G in st["g"]:
        X = G.double()
        X = X / (torch.linalg.vector_norm(X) + EPS)
        small = min(X.shape)
        for _ in range(case["steps"]):
            # the polynomial from the side with the smaller Gram matrix
            if X.shape[0] == small:
                S = X @ X.T
                X = (a * torch.eye(small, dtype=X.dtype, device=X.device) + S @
                     (b * torch.eye(small, dtype=X.dtype, device=X.device) + c * S)) @ X
            else:
                S = X.T @ X
                X = X @ (a * torch.eye(small, dtype=X.dtype, device=X.device) + S @
                         (b * torch.eye(small, dtype=X.dtype, device=X.device) + c * S))
        outs.append(X)
    return torch.stack(outs)


def exact(case, seed):
    st = _inputs(case, seed)
    if case["op"] == "ortho":
        return _exact_ortho(case, st)
    return _exact_route(case, st) if case["op"] == "route" else _exact_route_bwd(case, st)
