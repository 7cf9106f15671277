"""Cases of the operators that run before a dispatch, for measuring them: the
RMS norm with the residual's addition and an 8-bit output, the router's logits,
the choice of the experts, and the dispatch of rows that are in 8 bits already.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits, or in 64 for what decides between experts, rounded once at the end)
or, with ``own``, through the package's entry points.  ``exact`` computes the
same from the definitions in 64 bits.

Shapes: T tokens, H channels, E experts in G groups, K slots a token, P
destinations."""

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
FP8 = torch.float8_e4m3fn


def listed():
    return [
        # one decoded token of a large model: residual, bf16 row for the router, 8-bit row for
        # the experts; launch latency is all there is
        {"name": "norm_token", "op": "norm", "pass": "forward", "T": 1, "H": 7168,
         "residual": True, "fp8": True, "weight": "bf16"},
        # the rows of a long prompt on their way into the router and the dispatch
        {"name": "norm_prompt", "op": "norm", "pass": "forward", "T": 16384, "H": 7168,
         "residual": True, "fp8": True, "weight": "bf16"},
        # a fine-tuning step of a small model: odd rows, channels that are no multiple of 128
        {"name": "norm_step_odd", "op": "norm", "pass": "step", "T": 1237, "H": 2056,
         "residual": False, "fp8": False, "weight": "f32"},
        # the backward alone over a long batch, with the residual stream's gradient
        {"name": "norm_backward", "op": "norm", "pass": "backward", "T": 16384, "H": 4096,
         "residual": True, "fp8": False, "weight": "bf16"},
        # a few decoded tokens, a toy model's eight experts
        {"name": "route_tiny", "op": "route", "pass": "forward", "T": 5, "E": 8, "K": 2,
         "score": "softmax", "bias": False, "G": 1, "kept": 1, "top": 1, "renorm": True,
         "scale": 1.0},
        # a long prompt: sigmoid scores, the bias for balance, four of eight groups by the sum
        # of their two best, renormalised
        {"name": "route_groups", "op": "route", "pass": "forward", "T": 16384, "E": 256, "K": 8,
         "score": "sigmoid", "bias": True, "G": 8, "kept": 4, "top": 2, "renorm": True,
         "scale": 2.5},
        # a training step of softmax scores that are not renormalised: dense gradient, odd E
        {"name": "route_step_odd", "op": "route", "pass": "step", "T": 8195, "E": 60, "K": 4,
         "score": "softmax", "bias": False, "G": 1, "kept": 1, "top": 1, "renorm": False,
         "scale": 1.0},
        # the router of a small serving batch: the weights' bytes and latency
        {"name": "logits_few", "op": "logits", "pass": "forward", "T": 17, "E": 256, "H": 7168},
        # the router of a long prompt
        {"name": "logits_prompt", "op": "logits", "pass": "forward", "T": 16384, "E": 256,
         "H": 7168},
        # the router in a training step: forward, the rows' gradient and the weights'
        {"name": "logits_step", "op": "logits", "pass": "step", "T": 8195, "E": 64, "H": 4096},
        # 8-bit rows to eight destinations, a middling batch
        {"name": "rows_uniform", "op": "rows", "T": 4096, "H": 4096, "E": 64, "K": 6, "P": 8},
        # the largest: the rows of a long prompt to 32 destinations
        {"name": "rows_prompt", "op": "rows", "T": 32768, "H": 7168, "E": 256, "K": 8, "P": 32},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "route", "logits", "rows"])
    if op == "norm":
        fp8 = rng.random() < 0.5
        kind = "forward" if fp8 else rng.choice(["forward", "step", "backward"])
        return {"op": op, "pass": kind, "T": _log(rng, 1, 16384),
                "H": _log(rng, 256, 8192, 128 if fp8 else 8), "residual": rng.random() < 0.7,
                "fp8": fp8, "weight": rng.choice(["bf16", "f32"])}
    if op == "route":
        G = rng.choice([1, 1, 4, 8])
        E = G * _log(rng, max(2, 8 // G), 512 // G)
        kept = rng.randint(1, G)
        K = min(rng.randint(1, 8), kept * (E // G))
        return {"op": op, "pass": rng.choice(["forward", "step"]), "T": _log(rng, 1, 16384),
                "E": E, "K": K,
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "G": G,
                "kept": kept, "top": rng.choice([1, 2]),
                "renorm": K > 1 and rng.random() < 0.6,    # one slot's weight would be constant
                "scale": rng.choice([1.0, 2.5])}
    if op == "logits":
        return {"op": op, "pass": rng.choice(["forward", "step"]), "T": _log(rng, 1, 16384),
                "E": _log(rng, 8, 256), "H": _log(rng, 256, 7168, 8)}
    P = rng.choice([2, 8, 32])
    return {"op": op, "T": _log(rng, 1, 24000), "H": _log(rng, 256, 7168, 128), "E": 8 * P,
            "K": rng.randint(1, 8), "P": P}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op, T = case["op"], case["T"]
    st = {"case": case}

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, device=DEV, generator=g).to(dtype)

    if op == "norm":
        H = case["H"]
        dt = torch.bfloat16 if case["weight"] == "bf16" else torch.float32
        st["weight"] = (1.0 + 0.2 * normal(H)).to(dt)
        spread = torch.rand(T, 1, device=DEV, generator=g) * 3 + 0.1       # rows differ in size
        st["x"] = (normal(T, H) * spread).to(torch.bfloat16)
        if case["pass"] == "backward":      # x: the rows that the forward normalised
            st["rstd"] = (st["x"].double().square().mean(-1) + EPS).rsqrt().float()
        elif case["residual"]:
            st["residual"] = normal(T, H, dtype=torch.bfloat16)
        if case["pass"] != "forward":
            st["dy"] = normal(T, H, dtype=torch.bfloat16)
            if case["residual"]:
                st["d_residual"] = normal(T, H, dtype=torch.bfloat16)
    elif op == "route":
        E = case["E"]
        st["logits"] = normal(T, E) + 0.5 * normal(E)                      # some experts are liked
        if case["bias"]:
            st["bias"] = 0.1 * normal(E)
        if case["pass"] == "step":
            st["dw"] = normal(T, case["K"])
    elif op == "logits":
        E, H = case["E"], case["H"]
        st["x"] = normal(T, H, dtype=torch.bfloat16)
        st["w"] = (normal(E, H) * H ** -0.5).to(torch.bfloat16)
        if case["pass"] == "step":
            st["dlogits"] = normal(T, E) * T ** -0.5
    else:
        H, E, K, P = case["H"], case["E"], case["K"], case["P"]
        idx = torch.rand(T, E, device=DEV, generator=g).argsort(dim=1)[:, :K]
        # one row for each (destination, token) with a slot, destination-major
        key, inv = torch.unique(idx // (E // P) * T + torch.arange(T, device=DEV)[:, None],
                                return_inverse=True)
        st["token_row"], st["N"] = inv.to(torch.int32).contiguous(), key.numel()
        st["q"] = normal(T, H).clamp_(-3, 3).mul_(149.0).to(FP8)
        st["scale"] = torch.rand(T, H // 128, device=DEV, generator=g) * 0.02 + 0.001
        # buffers of the send layout's capacity; the rows past the pairs are spare
        cap = T * min(K, P)
        st["out"] = torch.zeros(cap, H, dtype=torch.uint8, device=DEV).view(FP8)
        st["out_scale"] = torch.zeros(cap, H // 128, device=DEV)
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _norm_plain(st):
    case = st["case"]
    x, w, out = st["x"].float(), st["weight"].float(), {}
    if case["pass"] != "backward":
        if "residual" in st:
            s = (x + st["residual"].float()).to(torch.bfloat16)
            out["residual"], x = s, s.float()
        rstd = 1.0 / torch.sqrt((x * x).mean(-1) + EPS)
        y = x * rstd[:, None] * w
        out["y"] = y.to(torch.bfloat16)
        if case["fp8"]:
            v = y.unflatten(-1, (-1, 128))
            out["scale"] = v.abs().amax(-1) / 448.0
            out["q"] = (v / out["scale"][..., None]).flatten(-2).to(FP8)
        if case["pass"] == "forward":
            return out
    else:
        rstd = st["rstd"]
    dy, n = st["dy"].float(), x * rstd[:, None]
    g = dy * w
    dx = (g - n * (g * n).mean(-1, keepdim=True)) * rstd[:, None]
    if "d_residual" in st:
        dx = dx + st["d_residual"].float()
    out["dx"], out["dw"] = dx.to(torch.bfloat16), (dy * n).sum(0)
    return out


def _scores(case, l):
    if case["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    e = torch.exp(l - l.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _route_plain(st):
    case = st["case"]
    T, E, G, K = case["T"], case["E"], case["G"], case["K"]
    l = st["logits"].double()           # scores that lie close decide between experts
    s = _scores(case, l)
    # without a bias the scores order as the logits do
    key = s + st["bias"].double() if case["bias"] else s if G > 1 and case["top"] == 2 else l
    if G > 1:
        by = key.view(T, G, E // G)
        best = by.sort(dim=-1, descending=True).values[..., :case["top"]].sum(-1)
        order = best.sort(dim=-1, descending=True, stable=True).indices[:, :case["kept"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=DEV).scatter_(1, order, True)
        key = by.masked_fill(~keep[..., None], -math.inf).flatten(1)
    idx = key.sort(dim=-1, descending=True, stable=True).indices[:, :K]
    p = s.gather(1, idx)
    total = p.sum(-1, keepdim=True) if case["renorm"] else torch.ones_like(p[:, :1])
    out = {"idx": idx, "w": (case["scale"] * p / total).float()}
    if case["pass"] == "step":
        dp = case["scale"] * st["dw"].double()
        if case["renorm"]:
            dp = (dp - (dp * p).sum(-1, keepdim=True) / total) / total
        ds = torch.zeros_like(s).scatter_(1, idx, dp)
        if case["score"] == "sigmoid":
            dl = ds * s * (1.0 - s)
        else:
            dl = s * (ds - (ds * s).sum(-1, keepdim=True))
        out["d_logits"] = dl.float()
    return out


def _logits_plain(st):
    x, w = st["x"].float(), st["w"].float()
    out = {"logits": x @ w.t()}
    if "dlogits" in st:
        out["dx"] = (st["dlogits"] @ w).to(torch.bfloat16)
        out["dw"] = st["dlogits"].t() @ x
    return out


def _rows_plain(st):
    N, row = st["N"], st["token_row"].long()
    tok = torch.empty(N, dtype=torch.long, device=DEV)
    tok[row] = torch.arange(row.shape[0], device=DEV)[:, None].expand_as(row)
    st["out"].view(torch.uint8)[:N] = st["q"].view(torch.uint8)[tok]
    st["out_scale"][:N] = st["scale"][tok]
    return {"q": st["out"], "scale": st["out_scale"]}


def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"norm": _norm_plain, "route": _route_plain, "logits": _logits_plain,
                "rows": _rows_plain}[op](st)
    import combine_ep_send_amd as ep

    out = {}
    if op == "norm":
        x, rstd = st["x"], st.get("rstd")
        if case["pass"] != "backward":
            n = ep.ep_rms_norm(x, st["weight"], EPS, residual=st.get("residual"),
                               fp8=case["fp8"], rstd=case["pass"] == "step")
            out["y"] = n.y
            if case["residual"]:
                out["residual"] = x = n.residual
            if case["fp8"]:
                out["q"], out["scale"] = n.q, n.scale
            rstd = n.rstd
        if case["pass"] != "forward":
            out["dx"], out["dw"] = ep.ep_rms_norm_backward(st["dy"], x, st["weight"], rstd,
                                                           d_residual=st.get("d_residual"))
    elif op == "route":
        how = {"score": case["score"], "renormalize": case["renorm"], "scale": case["scale"]}
        out["idx"], out["w"] = ep.ep_route(st["logits"], case["K"], bias=st.get("bias"),
                                           num_groups=case["G"], topk_groups=case["kept"],
                                           group_top=case["top"], **how)
        if case["pass"] == "step":
            out["d_logits"] = ep.ep_route_backward(st["dw"], st["logits"], out["idx"], **how)
    elif op == "logits":
        out["logits"] = ep.ep_router_logits(st["x"], st["w"])
        if case["pass"] == "step":
            out["dx"], out["dw"] = ep.ep_router_logits_backward(st["dlogits"], st["x"], st["w"])
    else:
        out["q"], out["scale"] = ep.ep_dispatch_permute_quantized(st["q"], st["scale"],
                                                                  st["token_row"],
                                                                  st["out"].shape[0],
                                                                  out=st["out"],
                                                                  out_scale=st["out_scale"])
    return out


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op, T = case["op"], case["T"]
    if op == "norm":
        H = case["H"]
        b = 0.0
        if case["pass"] != "backward":
            b += 4.0 * T * H + (4.0 * T * H if case["residual"] else 0.0)
            b += T * H * (1 + 4 / 128) if case["fp8"] else 0.0
        if case["pass"] != "forward":
            b += 6.0 * T * H + (2.0 * T * H if case["residual"] else 0.0) + 4.0 * H
        return {"bytes": b, "flops": 8.0 * T * H}
    if op == "route":
        E, K = case["E"], case["K"]
        both = 2 if case["pass"] == "step" else 1
        step = T * (4.0 * E + 12.0 * K) if case["pass"] == "step" else 0.0
        return {"bytes": T * (4.0 * E + 12.0 * K) + step, "flops": both * 10.0 * T * E}
    if op == "logits":
        E, H = case["E"], case["H"]
        both = 3 if case["pass"] == "step" else 1
        b = 2.0 * T * H + 2.0 * E * H + 4.0 * T * E
        if case["pass"] == "step":
            b += 4.0 * T * E + 2.0 * T * H + 2.0 * E * H + 2.0 * T * H + 4.0 * E * H
        return {"bytes": b, "flops": both * 2.0 * T * E * H}
    H, K, P = case["H"], case["K"], case["P"]
    # distinct destinations of K distinct experts, 8 (E / P) of them a destination
    E, own_share = case["E"], case["E"] // P
    rows = T * P * (1.0 - math.comb(E - own_share, K) / math.comb(E, K))
    return {"bytes": (T + rows) * H * (1 + 4 / 128) + 4.0 * T * K, "flops": 0.0}


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _norm_exact(case, st):
    out, x, w = {}, st["x"].double(), st["weight"].double()
    H = case["H"]
    if case["pass"] != "backward":
        if "residual" in st:
            x = (x + st["residual"].double()).float().to(torch.bfloat16).double()
            out["residual"] = x
        length = torch.linalg.vector_norm(x, dim=-1)
        rms = torch.sqrt(length ** 2 / H + EPS)
        out["y"] = x / rms[:, None] * w
        if case["fp8"]:
            blocks = out["y"].reshape(case["T"], H // 128, 128)
            top = torch.maximum(blocks.amax(-1), -blocks.amin(-1))
            out["scale"] = top / 448.0
            codes = blocks / out["scale"].float().double()[..., None]
            out["q"] = codes.float().to(FP8).reshape(case["T"], H)
    else:
        rms = 1.0 / st["rstd"].double()
    if case["pass"] != "forward":
        dy = st["dy"].double()
        gw = dy * w
        along = torch.einsum("th,th->t", gw, x) / (H * rms ** 3)
        out["dx"] = gw / rms[:, None] - along[:, None] * x
        if "d_residual" in st:
            out["dx"] += st["d_residual"].double()
        out["dw"] = torch.einsum("th,th,t->h", dy, x, 1.0 / rms)
    return out


def _route_exact(case, st):
    import numpy as np
    l = st["logits"].cpu().numpy().astype(np.float64)
    T, E, K, G = case["T"], case["E"], case["K"], case["G"]
    if case["score"] == "sigmoid":
        s = 0.5 * (1.0 + np.tanh(0.5 * l))
        slope = 0.25 * (1.0 - np.tanh(0.5 * l) ** 2)
    else:
        s = np.exp(l - np.logaddexp.reduce(l, axis=1, keepdims=True))
    key = s + (st["bias"].cpu().numpy().astype(np.float64) if case["bias"] else 0.0)
    if G > 1:
        best = -np.sort(-key.reshape(T, G, -1), axis=-1)[..., :case["top"]]
        rank = np.argsort(np.argsort(-best.sum(-1), axis=1, kind="stable"), axis=1)
        key = np.where(np.repeat(rank < case["kept"], E // G, axis=1), key, -np.inf)
    idx = np.argsort(-key, axis=1, kind="stable")[:, :K]
    p = np.take_along_axis(s, idx, 1)
    total = p.sum(1, keepdims=True) if case["renorm"] else 1.0
    out = {"idx": None, "w": case["scale"] * p / total}
    if case["pass"] == "step":
        # by the chain rule through w_j = scale * s_j / total
        g = case["scale"] * st["dw"].cpu().numpy().astype(np.float64)
        if case["renorm"]:
            g = g / total - ((g * p).sum(1, keepdims=True)) / total ** 2
        full = np.zeros((T, E))
        np.put_along_axis(full, idx, g, 1)
        full = full * slope if case["score"] == "sigmoid" else \
            full * s - s * (full * s).sum(1, keepdims=True)
        out["d_logits"] = full
    return {k: None if v is None else torch.from_numpy(v) for k, v in out.items()}


def _logits_exact(st):
    x, w = st["x"].double(), st["w"].double()
    out = {"logits": torch.mm(x, w.t())}
    if "dlogits" in st:
        d = st["dlogits"].double()
        out["dx"], out["dw"] = torch.mm(d, w), torch.mm(d.t(), x)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        return _norm_exact(case, st)
    if case["op"] == "route":
        return _route_exact(case, st)
    if case["op"] == "logits":
        return _logits_exact(st)
    # rows in the order of their numbers: sorting the slots' rows gives each row's token
    rows, at = torch.sort(st["token_row"].flatten().long(), stable=True)
    first = torch.ones_like(rows, dtype=torch.bool)
    first[1:] = rows[1:] != rows[:-1]
    tok = at[first] // case["K"]
    spare = st["out"].shape[0] - tok.numel()
    q = st["q"].view(torch.uint8).index_select(0, tok)
    scale = st["scale"].double().index_select(0, tok)
    return {"q": torch.cat((q, q.new_zeros(spare, q.shape[1]))).view(FP8),
            "scale": torch.cat((scale, scale.new_zeros(spare, scale.shape[1])))}
