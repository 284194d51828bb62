"""The operators around the W4A4 linear layer in a decoder that serves with it:
the residual / gate / norm step that makes a layer's input, that step fused with
the layer's rotation and quantiser, and the low-rank adapters of many requests
beside a shared projection with the plan that groups their tokens.

``run`` computes each in plain torch (``own`` false) or through the package's
entry points (``own`` true); ``exact`` computes it in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
TILE = 64            # tokens of one adapter per tile of a plan
EPS = 1e-5


# ----------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of one request: the hidden size of the 4096-wide layers
        {"name": "norm decode M1", "op": "norm", "M": 1, "K": 4096, "xt": "f16", "wt": "f16", "post": False,
         "gate": "none", "alpha": 1.0, "offset": 0.0},
        # a prompt through a block with norms on both sides and a gate per token and channel
        {"name": "norm prompt sandwich", "op": "norm", "M": 4096, "K": 4096, "xt": "bf16", "wt": "bf16", "post": True,
         "gate": "token", "alpha": 1.0, "offset": 1.0},
        # fp32 residual stream, ragged batch, odd width, gate per channel, scaled residual
        {"name": "norm fp32 odd", "op": "norm", "M": 1537, "K": 5003, "xt": "f32", "wt": "bf16", "post": True,
         "gate": "channel", "alpha": 0.22, "offset": 0.0},
        # decode batch into 8-bit codes (the W4A8 layer)
        {"name": "norm+quant8 decode M16", "op": "normq", "M": 16, "K": 4096, "xt": "f16", "wt": "f16",
         "gate": "none", "alpha": 1.0, "offset": 0.0, "group": 128, "bits": 8, "want_x": False},
        # the attention projection's prompt: full-width rotation, 8-bit codes
        {"name": "norm+quant8 prompt g4096", "op": "normq", "M": 2048, "K": 4096, "xt": "bf16", "wt": "bf16",
         "gate": "none", "alpha": 1.0, "offset": 0.0, "group": 4096, "bits": 8, "want_x": False},
        # the 8192-wide layer's longest prompt, 4-bit codes, the normed rows kept for adapters
        {"name": "norm+quant4 prompt g256", "op": "normq", "M": 8192, "K": 8192, "xt": "bf16", "wt": "f32",
         "gate": "channel", "alpha": 0.5, "offset": 0.0, "group": 256, "bits": 4, "want_x": True},
        # plan of one decode step, and of a long mixed batch
        {"name": "plan decode M16", "op": "plan", "M": 16, "n": 64, "runs": 1, "bare": 8},
        {"name": "plan mixed M32768", "op": "plan", "M": 32768, "n": 256, "runs": 5, "bare": 8},
        # one request decoding with its adapter beside the up projection
        {"name": "lora decode M1", "op": "lora", "M": 1, "K": 4096, "N": 11008, "n": 8, "r": 16, "requests": 1,
         "xt": "f16", "yt": "f16", "ragged": False, "bare": 0},
        # sixteen requests of sixteen adapters with their own ranks, fp32 result
        {"name": "lora decode M16 ragged", "op": "lora", "M": 16, "K": 4096, "N": 11008, "n": 64, "r": 32,
         "requests": 16, "xt": "f16", "yt": "f32", "ragged": True, "bare": 8},
        # prompts of twelve requests, some without an adapter, beside the attention projection
        {"name": "lora prompts M2048", "op": "lora", "M": 2048, "K": 4096, "N": 4096, "n": 16, "r": 32,
         "requests": 12, "xt": "bf16", "yt": "bf16", "ragged": True, "bare": 6},
        # the 8192 -> 28672 layer's longest prompts at the highest rank here
        {"name": "lora prompts M8192", "op": "lora", "M": 8192, "K": 8192, "N": 28672, "n": 8, "r": 64,
         "requests": 8, "xt": "bf16", "yt": "bf16", "ragged": False, "bare": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "normq", "plan", "lora", "lora"])
    if op == "norm":
        return {"op": op, "M": _log(rng, 1, 6000), "K": _log(rng, 64, 8192), "xt": rng.choice(["f16", "bf16", "f32"]),
                "wt": rng.choice(["f16", "bf16", "f32"]), "post": rng.random() < 0.5,
                "gate": rng.choice(["none", "channel", "token"]), "alpha": rng.choice([1.0, 0.22, 0.5, 1.4]),
                "offset": rng.choice([0.0, 1.0])}
    if op == "normq":
        group = 8 << rng.randrange(10)
        step = max(group, 32)
        return {"op": op, "M": _log(rng, 1, 6000), "K": step * max(1, _log(rng, 128, 8192) // step),
                "xt": rng.choice(["f16", "bf16"]), "wt": rng.choice(["f16", "bf16", "f32"]),
                "gate": rng.choice(["none", "channel", "token"]), "alpha": rng.choice([1.0, 0.22, 0.5]),
                "offset": rng.choice([0.0, 1.0]), "group": group, "bits": rng.choice([4, 8]),
                "want_x": rng.random() < 0.3}
    if op == "plan":
        return {"op": op, "M": _log(rng, 1, 32768), "n": _log(rng, 1, 512), "runs": rng.choice([1, 3, 40, 500]),
                "bare": rng.choice([0, 4, 8])}
    M = _log(rng, 1, 4096)
    r = 8 * rng.choice([1, 2, 3, 4, 5, 8])
    n = _log(rng, 1, max(1, (512 if M >= 256 else 2048) // r))
    return {"op": op, "M": M, "K": 8 * _log(rng, 16, 1024), "N": 8 * _log(rng, 16, 2048), "n": n, "r": r,
            "requests": min(M, _log(rng, 1, 64)), "xt": rng.choice(["f16", "bf16"]),
            "yt": rng.choice(["f16", "bf16", "f32"]), "ragged": rng.random() < 0.5, "bare": rng.choice([0, 5])}


# ---------------------------------------------------------------------- inputs
def _request_adapter(case, i):
    """Request i's slot in the shuffled list of adapters; None without an adapter."""
    if case["bare"] and i % case["bare"] == case["bare"] - 1:
        return None
    return i % case["n"]


def _request_len(case, i):
    """Tokens of request i: the batch cut into runs of uneven length."""
    R, M = case["requests"], case["M"]
    cut = lambda k: (k * M + (k * (R - k) * M) // (2 * R * R)) // R if k < R else M  # noqa: E731
    return cut(i + 1) - cut(i)


def _rank(case, slot):
    return case["r"] if not case["ragged"] else max(1, case["r"] >> (slot % 3)) - (slot % 2 if case["r"] > 8 else 0)


def _stream(M, K, dt, g, scale):
    """Rows of a residual stream: a few channels far above the others, unit spread otherwise."""
    x = torch.randn(M, K, generator=g, device=DEV)
    out = torch.randint(0, K, (8,), generator=g, device=DEV)
    x[:, out] *= 30.0
    return x.mul_(scale).to(dt)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = {"case": case}
    op, M = case["op"], case["M"]
    if op in ("norm", "normq"):
        K, xt, wt = case["K"], TYPES[case["xt"]], TYPES[case["wt"]]
        # rows start on 16 bytes also where the width is odd
        pad = -(-K // 8) * 8
        rows = lambda scale: _stream(M, pad, xt, g, scale)[:, :K]  # noqa: E731
        norm_w = lambda: (1.0 - case["offset"] + 0.2 * torch.randn(K, generator=g, device=DEV)).to(wt)  # noqa: E731
        s["H"], s["Y"], s["w"] = rows(2.0), rows(0.5), norm_w()
        s["w_post"] = norm_w() if case.get("post") else None
        s["gate"] = None
        if case["gate"] == "channel":
            s["gate"] = (0.5 + 0.3 * torch.randn(K, generator=g, device=DEV)).to(xt)
        elif case["gate"] == "token":
            s["gate"] = (0.5 + 0.3 * torch.randn(M, pad, generator=g, device=DEV)).to(xt)[:, :K]
        s["H_out"] = torch.empty(M, pad, dtype=xt, device=DEV)[:, :K]
        s["X"] = torch.empty(M, pad, dtype=xt, device=DEV)[:, :K] if op == "norm" or case["want_x"] else None
        if op == "normq":
            d = torch.randint(0, 2, (case["group"],), generator=g, device=DEV) * 2 - 1
            d[0] = 1
            s["signs"] = d.to(torch.int8)
            s["Xq"] = (torch.empty(M, K, dtype=torch.int8, device=DEV) if case["bits"] == 8
                       else torch.empty(M, K // 2, dtype=torch.uint8, device=DEV))
            s["sx"] = torch.empty(M, dtype=torch.float32, device=DEV)
        return s
    if op == "plan":
        # runs of tokens of one adapter, as requests lie in a batch, then some without one
        n, runs = case["n"], case["runs"]
        ids = torch.randint(0, n, (-(-M // runs),), generator=g, device=DEV).repeat_interleave(runs)[:M]
        if case["bare"]:
            bare = torch.randint(0, case["bare"], (-(-M // runs),), generator=g, device=DEV).repeat_interleave(runs)[:M]
            ids = torch.where(bare == 0, -1, ids)
        s["ids"] = ids.to(torch.int32).contiguous()
        s["order"] = torch.empty(M, dtype=torch.int32, device=DEV)
        s["tiles"] = torch.empty(M // TILE + min(n + 1, M), 3, dtype=torch.int32, device=DEV)
        return s
    K, N, n, r, xt, yt = case["K"], case["N"], case["n"], case["r"], TYPES[case["xt"]], TYPES[case["yt"]]
    slots = torch.randperm(n, generator=g, device=DEV).tolist()
    ids, rank = [], [r] * n
    for i in range(case["requests"]):
        slot = _request_adapter(case, i)
        ids += [-1 if slot is None else slots[slot]] * _request_len(case, i)
    for slot in range(n):
        rank[slots[slot]] = _rank(case, slot)
    s["ids"] = torch.tensor(ids, dtype=torch.int32, device=DEV)
    s["X"] = _stream(M, K, xt, g, 1.0)
    s["A"] = (torch.randn(n, r, K, generator=g, device=DEV) / math.sqrt(K)).to(xt)
    s["B"] = (0.1 * torch.randn(n, N, r, generator=g, device=DEV)).to(xt)
    s["base"] = torch.randn(M, N, generator=g, device=DEV).to(yt)
    s["ranks"] = torch.tensor(rank, dtype=torch.int32, device=DEV) if case["ragged"] else None
    s["scales"] = 0.5 + torch.rand(n, generator=g, device=DEV)
    # the plan of this batch: every adapted layer of a step shares it
    s["order"], s["tiles"] = _plan_plain(s["ids"], n)
    s["out"] = torch.empty(M, N, dtype=yt, device=DEV)
    s["work"] = torch.empty(M, r, dtype=torch.float32, device=DEV)
    return s


# ----------------------------------------------------------------- plain forms
def _plan_plain(ids, n):
    """Tokens in the order of their adapter (-1, none, first), and that order cut
    into tiles (adapter, first position, tokens) of at most 64 tokens of one adapter."""
    M = ids.numel()
    order = torch.argsort(ids, stable=True).to(torch.int32)
    count = (ids[None, :] == torch.arange(-1, n, device=ids.device)[:, None]).sum(1) if M * (n + 1) <= 1 << 24 \
        else torch.zeros(n + 1, dtype=torch.int64, device=ids.device).index_add_(
            0, ids.long() + 1, torch.ones(M, dtype=torch.int64, device=ids.device))
    per = (count + TILE - 1) // TILE
    begin = torch.cumsum(count, 0) - count
    last = torch.cumsum(per, 0)
    rows = M // TILE + min(n + 1, M)
    t = torch.arange(rows, device=ids.device)
    a = torch.searchsorted(last, t, right=True)
    used = a <= n
    a = torch.where(used, a, 0)
    at = (t - (last[a] - per[a])) * TILE
    start = begin[a] + at
    here = torch.minimum(count[a] - at, torch.full_like(at, TILE))
    tiles = torch.stack((a - 1, start, here), 1)
    return order, torch.where(used[:, None], tiles, torch.tensor([-1, 0, 0], device=ids.device)).to(torch.int32)


def _residual(s):
    """The residual stream after the block, rounded to its type, and that as fp32."""
    case = s["case"]
    p = s["Y"].float()
    if s["w_post"] is not None:
        rstd = torch.rsqrt(p.square().mean(1, keepdim=True) + EPS)
        p = p * (s["w_post"].float() + case["offset"]) * rstd
    if s["gate"] is not None:
        p = s["gate"].float() * p
    h = (s["H"].float() + case["alpha"] * p).to(s["H"].dtype)
    return h, h.float()


def _norm_plain(s):
    h, f = _residual(s)
    v = f * (s["w"].float() + s["case"]["offset"])
    rstd = torch.rsqrt(f.square().mean(1, keepdim=True) + EPS)
    return {"h": h, "x": (v * rstd).to(h.dtype)}


def _butterfly(v, group):
    """v times the Sylvester matrix in each group: stages 1, 2, 4, ... of (a + b, a - b)."""
    M, K = v.shape
    h = 1
    while h < group:
        p = v.view(M, K // (2 * h), 2, h)
        v = torch.stack((p[:, :, 0] + p[:, :, 1], p[:, :, 0] - p[:, :, 1]), 2).view(M, K)
        h *= 2
    return v


def _normq_plain(s):
    case = s["case"]
    h, f = _residual(s)
    v = f * (s["w"].float() + case["offset"])
    rstd = torch.rsqrt(f.square().mean(1) + EPS)
    group = case["group"]
    u = _butterfly(v * s["signs"].float().repeat(case["K"] // group), group)
    # the codes are defined by this sequence of fp32 steps, with the division done as one
    top = torch.full_like(rstd, 127.0 if case["bits"] == 8 else 7.0)
    amax = u.abs().amax(1)
    inv = torch.where(amax > 0, top / amax, 0.0)
    q = torch.round(u * inv[:, None]).to(torch.int8)
    sx = (amax / top) * torch.tensor(1.0 / math.sqrt(group), dtype=torch.float32, device=u.device) * rstd
    out = {"h": h, "q": q, "sx": sx}
    if case["want_x"]:
        out["x"] = (v * rstd[:, None]).to(h.dtype)
    return out


def _lora_plain(s):
    """Every token against every adapter, the products of the other adapters masked out."""
    X, A, B, ids = s["X"], s["A"], s["B"], s["ids"].long()
    n, r, K = A.shape
    live = torch.ones(n, r, dtype=torch.bool, device=X.device)
    if s["ranks"] is not None:
        live = torch.arange(r, device=X.device)[None] < s["ranks"][:, None]
    mine = ids[:, None] == torch.arange(n, device=X.device)
    T = torch.matmul(X.float(), A.float().reshape(n * r, K).T).view(-1, n, r)
    T = torch.where(mine[:, :, None] & live[None], T * s["scales"][None, :, None], 0.0)
    Bt = torch.where(live[:, None, :], B.float(), 0.0).permute(0, 2, 1).reshape(n * r, -1)
    return (s["base"].float() + torch.matmul(T.view(-1, n * r), Bt)).to(s["base"].dtype)


def _signed(Xq):
    """The signed values of codes packed two per byte, the even one in the low half."""
    b = Xq.view(torch.int8)
    return (torch.stack((b << 4, b), 2) >> 4).view(b.shape[0], -1)


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        from w4a4_bit_gemm_hq_b200 import hq

        if op == "norm":
            h, x = hq.hq_residual_norm(s["H"], s["w"], EPS, Y=s["Y"], w_post=s["w_post"], gate=s["gate"],
                                       alpha=case["alpha"], w_offset=case["offset"], H_out=s["H_out"], X=s["X"])
            return {"h": h, "x": x}
        if op == "normq":
            Xq, sx, h, x = hq.hq_norm_rotate_quant(s["H"], s["w"], EPS, case["group"], s["signs"], Y=s["Y"],
                                                   gate=s["gate"], alpha=case["alpha"], w_offset=case["offset"],
                                                   bits=case["bits"], H_out=s["H_out"], X=s["X"], Xq=s["Xq"],
                                                   sx=s["sx"])
            out = {"h": h, "q": Xq if case["bits"] == 8 else _signed(Xq), "sx": sx}
            return {**out, "x": x} if case["want_x"] else out
        if op == "plan":
            return list(hq.hq_lora_plan(s["ids"], case["n"], s["order"], s["tiles"]))
        return hq.hq_lora_apply(s["X"], s["A"], s["B"], s["order"], s["tiles"], ranks=s["ranks"], scales=s["scales"],
                                base=s["base"], Y=s["out"], workspace=s["work"])
    if op == "norm":
        return _norm_plain(s)
    if op == "normq":
        return _normq_plain({**s, "w_post": None})
    if op == "plan":
        return list(_plan_plain(s["ids"], case["n"]))
    return _lora_plain(s)


# ------------------------------------------------------------------------ work
def work(case):
    op, M = case["op"], case["M"]
    size = {"f16": 2, "bf16": 2, "f32": 4}
    if op == "plan":
        return {"bytes": 8 * M + 12 * (M // TILE + min(case["n"] + 1, M)), "flops": 0}
    if op == "lora":
        K, N, e = case["K"], case["N"], size[case["xt"]]
        lens = [(_request_adapter(case, i), _request_len(case, i)) for i in range(case["requests"])]
        slots = {a for a, length in lens if a is not None and length}
        ranks = sum(_rank(case, a) for a in slots)
        adapted = sum(length for a, length in lens if a is not None)
        flops = sum(2.0 * length * _rank(case, a) * (K + N) for a, length in lens if a is not None)
        return {"bytes": e * adapted * K + e * ranks * (K + N) + 2 * size[case["yt"]] * M * N + 8 * M, "flops": flops}
    K, e = case["K"], size[case["xt"]]
    b = 3 * e * M * K + size[case["wt"]] * K * (2 if case.get("post") else 1)
    b += {"none": 0, "channel": e * K, "token": e * M * K}[case["gate"]]
    if op == "norm":
        return {"bytes": b + e * M * K, "flops": 12.0 * M * K}
    b += M * K * case["bits"] // 8 + 4 * M + (e * M * K if case["want_x"] else 0)
    return {"bytes": b, "flops": (8.0 + math.log2(case["group"])) * M * K}


# ------------------------------------------------------------- 64-bit reference
def exact(case, seed):
    op = case["op"]
    if op == "plan":
        return None
    s = prepare(case, seed)
    if op == "lora":
        out = s["base"].double()
        ids = s["ids"]
        for a in range(case["n"]):
            rows = torch.nonzero(ids == a).flatten()
            k = case["r"] if s["ranks"] is None else int(s["ranks"][a])
            if rows.numel() and k:
                t = torch.mm(s["X"][rows].double(), s["A"][a, :k].double().t())
                out[rows] += float(s["scales"][a]) * torch.mm(t, s["B"][a, :, :k].double().t())
        return out
    off, K = case["offset"], case["K"]
    block = s["Y"].double()
    if case.get("post"):
        block = (s["w_post"].double() + off) * block / ((block * block).sum(1, keepdim=True) / K + EPS).sqrt()
    if s["gate"] is not None:
        block = block * s["gate"].double()
    h = s["H"].double() + case["alpha"] * block
    kept = h.to(s["H"].dtype).double()               # what the next norm reads is the stored stream
    root = ((kept * kept).sum(1, keepdim=True) / K + EPS).sqrt()
    scaled = kept * (s["w"].double() + off)
    if op == "norm":
        return {"h": h, "x": scaled / root}
    g = case["group"]
    had = torch.ones(1, 1, dtype=torch.float64, device=DEV)
    while had.shape[0] < g:
        had = torch.cat((torch.cat((had, had), 1), torch.cat((had, -had), 1)), 0)
    turned = torch.matmul((scaled.view(-1, K // g, g) * s["signs"].double()), had).view(-1, K)
    top = 127.0 if case["bits"] == 8 else 7.0
    # the codes belong to their fp32 steps: a value on a rounding border has no 64-bit code
    out = {"h": h, "q": None, "sx": turned.abs().max(1).values / (top * math.sqrt(g)) / root[:, 0]}
    if case["want_x"]:
        out["x"] = scaled / root
    return out
