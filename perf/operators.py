"""The operators of an expert layer at serving time, as calls to be timed and compared.

  linear_epilogue   Y = act(X W^T + bias) + residual, the W8A8 linear layer with its epilogue
  route_topk        scores of E experts -> the experts of each token and their weights
  moe_decode        a whole SwiGLU expert layer for a few tokens, from bf16 rows to the weighted sum

Each has a plain form (``own`` false: elementary torch operations in 32 bits, or in 64 where 32 lose what
matters) and the library's call (``own`` true).  The FP8 steps are part of the operators: activations are
quantized per token in 1x128 groups (scale = max(amax, 1e-4) / 448, or the smallest power of two not below
it), weights come as E4M3 codes with one scale per 128x128 block.
"""
import math

import torch

own = False

F32, UE8M0 = 0, 1
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
DEV = "cuda"


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # an attention output projection while one sequence decodes: latency alone
        dict(name="linear_decode_1", op="linear", M=1, N=4096, K=4096, fmt=F32, act="none", bias="", residual=True),
        # a batch of odd size through a wide projection with power-of-two scales: every weight is read once
        dict(name="linear_decode_37", op="linear", M=37, N=18432, K=7168, fmt=UE8M0, act="gelu_tanh", bias="bfloat16",
             residual=False),
        # a ragged prefill through a biased projection
        dict(name="linear_prefill_1000", op="linear", M=1000, N=4096, K=4096, fmt=F32, act="gelu", bias="float32",
             residual=True),
        # the feed-forward's gate-like projection of a prefill, power-of-two scales
        dict(name="linear_prefill_4096", op="linear", M=4096, N=14336, K=4096, fmt=UE8M0, act="silu", bias="bfloat16",
             residual=False),
        # the down projection of a long prefill, added to the residual stream
        dict(name="linear_down_8192", op="linear", M=8192, N=4096, K=14336, fmt=F32, act="none", bias="", residual=True),
        # one token's routing: latency alone
        dict(name="route_1", op="route", T=1, E=256, topk=8, score="sigmoid", groups=8, keep=4, bias=True, dtype="float32",
             masked=False),
        # a prefill's routing over groups of experts with a selection bias
        dict(name="route_8192", op="route", T=8192, E=256, topk=8, score="sigmoid", groups=8, keep=4, bias=True,
             dtype="float32", masked=False),
        # a prefill's softmax routing with padded tokens and experts that are switched off
        dict(name="route_softmax_20011", op="route", T=20011, E=160, topk=6, score="softmax", groups=1, keep=1, bias=False,
             dtype="bfloat16", masked=True),
        # a small expert layer: little to read, so launches and joins count
        dict(name="moe_small_5", op="moe", T=5, E=8, topk=2, K=1024, I=384, fmt=F32, residual=False, skew=0.0, holes=True),
        # one sequence decoding through the wide expert layer
        dict(name="moe_decode_1", op="moe", T=1, E=256, topk=8, K=7168, I=2048, fmt=UE8M0, residual=True, skew=0.0,
             holes=False),
        # a small batch: few experts see more than one token
        dict(name="moe_decode_7", op="moe", T=7, E=256, topk=8, K=7168, I=2048, fmt=F32, residual=True, skew=0.0,
             holes=False),
        # a full batch on one device's share of the experts, popularity skewed: some experts see most tokens
        dict(name="moe_decode_64", op="moe", T=64, E=32, topk=8, K=7168, I=2048, fmt=UE8M0, residual=True, skew=1.1,
             holes=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("linear", "linear", "route", "moe", "moe"))
    if op == "linear":
        while True:
            c = dict(op=op, M=_log_int(rng, 1, 8192), N=128 * _log_int(rng, 1, 144), K=128 * _log_int(rng, 1, 112))
            if c["M"] * c["N"] * c["K"] <= 8192 * 4096 * 14336 and c["N"] * c["K"] <= 18432 * 7168:
                break
        return dict(c, fmt=rng.choice((F32, UE8M0)), act=rng.choice(ACTS), bias=rng.choice(("", "bfloat16", "float32")),
                    residual=rng.random() < 0.5)
    if op == "route":
        groups = rng.choice((1, 1, 4, 8))
        E = groups * _log_int(rng, 8, 512 // groups)
        score = rng.choice(("softmax", "sigmoid"))
        return dict(op=op, T=_log_int(rng, 1, 20000), E=E, topk=rng.randint(1, 8), score=score, groups=groups,
                    keep=rng.randint((groups + 1) // 2, groups), bias=score == "sigmoid" and rng.random() < 0.5,
                    dtype=rng.choice(("float32", "bfloat16")), masked=rng.random() < 0.4)
    while True:
        c = dict(op=op, T=_log_int(rng, 1, 64), E=_log_int(rng, 4, 256), topk=rng.randint(1, 8),
                 K=128 * _log_int(rng, 2, 56), I=128 * _log_int(rng, 1, 16))
        c["topk"] = min(c["topk"], c["E"])
        if c["E"] * c["K"] * c["I"] <= 256 * 7168 * 2048 and _active(c) * c["K"] * c["I"] <= 32 * 7168 * 2048:
            break
    return dict(c, fmt=rng.choice((F32, UE8M0)), residual=rng.random() < 0.5, skew=rng.choice((0.0, 1.1)),
                holes=rng.random() < 0.3)


def _active(c):
    """Experts that T tokens meet when they choose evenly."""
    return c["E"] * (1.0 - (1.0 - c["topk"] / c["E"]) ** c["T"])


def work(case):
    c = case
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        ws = (N // 128) * (K // 128) * (4 if c["fmt"] == F32 else 1)
        nb = N * {"": 0, "bfloat16": 2, "float32": 4}[c["bias"]]
        return {"bytes": 2 * M * K + N * K + ws + nb + 2 * M * N * (2 if c["residual"] else 1), "flops": 2 * M * N * K}
    if c["op"] == "route":
        el = 4 if c["dtype"] == "float32" else 2
        return {"bytes": c["T"] * (c["E"] * el + c["topk"] * 8) + (4 * c["E"] if c["bias"] else 0),
                "flops": 4 * c["T"] * c["E"]}
    T, K, I = c["T"], c["K"], c["I"]
    a = _active(c)
    per = 3 * I * K + 3 * (I // 128) * (K // 128) * (4 if c["fmt"] == F32 else 1)
    return {"bytes": int(a * per) + 2 * T * K * (3 if c["residual"] else 2) + 8 * T * c["topk"],
            "flops": 6 * T * c["topk"] * I * K}


# ----------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _scale_of(amax, fmt):
    amax = torch.clamp(amax, min=1e-4)
    s = amax / torch.full_like(amax, 448.0)     # an IEEE quotient: a plain number would become a product with 1/448
    if fmt == UE8M0:
        m, e = torch.frexp(s)
        s = torch.ldexp(torch.ones_like(s), torch.where(m == 0.5, e - 1, e))
    return s


def _weight(N, K, fmt, g):
    """E4M3 codes u8 [N, K] and block scales [N/128, K/128] of a weight ~ N(0, 0.02), as a checkpoint holds them."""
    w = torch.empty(N, K, device=DEV).normal_(0.0, 0.02, generator=g).to(torch.bfloat16).float()
    w = w.view(N // 128, 128, K // 128, 128)
    s = _scale_of(w.abs().amax(dim=(1, 3)), fmt)
    q = (w / s[:, None, :, None]).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(N, K)
    if fmt == UE8M0:
        s = (torch.log2(s).round() + 127).to(torch.uint8)
    return q, s


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        X = torch.empty(M, K, device=DEV).normal_(generator=g)
        X = torch.where(torch.rand(M, K, device=DEV, generator=g) < 0.001, X * 50, X).to(torch.bfloat16)
        Wq, Ws = _weight(N, K, c["fmt"], g)
        bias = torch.randn(N, device=DEV, generator=g).to(getattr(torch, c["bias"])) if c["bias"] else None
        R = torch.randn(M, N, device=DEV, generator=g).to(torch.bfloat16) if c["residual"] else None
        return dict(c, X=X, Wq=Wq, Ws=Ws, bias=bias, R=R)
    if c["op"] == "route":
        T, E = c["T"], c["E"]
        z = torch.randn(T, E, device=DEV, generator=g)
        if c["masked"]:
            off = torch.rand(T, E, device=DEV, generator=g) < 0.1
            off |= torch.rand(T, 1, device=DEV, generator=g) < 0.05
            z = z.masked_fill(off, -math.inf)
        bias = 0.1 * torch.randn(E, device=DEV, generator=g) if c["bias"] else None
        return dict(c, logits=z.to(getattr(torch, c["dtype"])), b=bias)
    T, E, k, K, I = c["T"], c["E"], c["topk"], c["K"], c["I"]
    sd = torch.float32 if c["fmt"] == F32 else torch.uint8
    W13q = torch.empty(E, 2 * I, K, dtype=torch.uint8, device=DEV)
    W13s = torch.empty(E, 2 * I // 128, K // 128, dtype=sd, device=DEV)
    W2q = torch.empty(E, K, I, dtype=torch.uint8, device=DEV)
    W2s = torch.empty(E, K // 128, I // 128, dtype=sd, device=DEV)
    for e in range(E):
        W13q[e], W13s[e] = _weight(2 * I, K, c["fmt"], g)
        W2q[e], W2s[e] = _weight(K, I, c["fmt"], g)
    X = torch.randn(T, K, device=DEV, generator=g).to(torch.bfloat16)
    R = torch.randn(T, K, device=DEV, generator=g).to(torch.bfloat16) if c["residual"] else None
    u = torch.rand(T, E, device=DEV, generator=g, dtype=torch.float64).clamp_(1e-300, 1.0)
    z = -torch.log(-torch.log(u)) - c["skew"] * torch.log(torch.arange(1, E + 1, device=DEV, dtype=torch.float64))
    w, ids = torch.topk(z, k, dim=1)
    w = torch.softmax(w, dim=1).float()
    ids = ids.to(torch.int32)
    if c["holes"]:      # slots without an expert: padded tokens and experts that another device holds
        ids = torch.where(torch.rand(T, k, device=DEV, generator=g) < 0.2, torch.full_like(ids, -1), ids)
    return dict(c, X=X, W13q=W13q, W13s=W13s, W2q=W2q, W2s=W2s, ids=ids.contiguous(), w=w.contiguous(), R=R)


# ------------------------------------------------------------------------------------------ plain forms
def _act_hat(x, fmt):
    """What the 1x128 quantizer leaves of x (fp32 [..., K]): code * scale."""
    v = x.unflatten(-1, (-1, 128))
    s = _scale_of(v.abs().amax(dim=-1, keepdim=True), fmt)
    return ((v / s).clamp(-448, 448).to(torch.float8_e4m3fn).float() * s).flatten(-2)


def _w_hat(q, s, fmt):
    """fp32 weight [..., N, K] of codes and block scales."""
    if fmt == UE8M0:
        s = torch.ldexp(torch.ones(s.shape, device=s.device), s.int() - 127)
    w = q.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 128)).unflatten(-3, (-1, 128))
    return w.mul_(s[..., :, None, :, None]).flatten(-2).flatten(-3, -2)


def _act(y, act):
    if act == "relu":
        return torch.clamp(y, min=0)
    if act == "silu":
        return y / (1 + torch.exp(-y))
    if act == "gelu":
        return 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))
    return y


def _linear(s):
    y = _act_hat(s["X"].float(), s["fmt"]) @ _w_hat(s["Wq"], s["Ws"], s["fmt"]).T
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = _act(y, s["act"])
    if s["R"] is not None:
        y = y + s["R"].float()
    return y.to(torch.bfloat16)


def _route(s):
    z = s["logits"].double()                # in 64 bits: the k-th and the next score can lie close together
    T, E = z.shape
    p = torch.softmax(z, dim=1).nan_to_num(0.0) if s["score"] == "softmax" else 1 / (1 + torch.exp(-z))
    key = z if s["score"] == "softmax" else p
    if s["b"] is not None:
        key = key + s["b"].double()
    key = key.masked_fill(z == -math.inf, -math.inf)
    if s["groups"] > 1:
        per = key.view(T, s["groups"], -1)
        best = torch.sort(per, dim=2, descending=True, stable=True).values[:, :, :1 if s["score"] == "softmax" else 2]
        score = torch.where(torch.isinf(best[:, :, :1]), best[:, :, :1], best.nan_to_num(neginf=0.0)).sum(dim=2)
        kept = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :s["keep"]]
        on = torch.zeros_like(score, dtype=torch.bool).scatter_(1, kept, True)
        key = key.masked_fill(~on[:, :, None].expand_as(per).reshape(T, E), -math.inf)
    order = torch.sort(key, dim=1, descending=True, stable=True)
    ids, top = order.indices[:, :s["topk"]], order.values[:, :s["topk"]]
    empty = top == -math.inf
    w = p.gather(1, ids).masked_fill(empty, 0.0)
    w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-20)
    return ids.masked_fill(empty, -1).to(torch.int32), w.float()


def _moe(s):
    T, E, k, K, I = s["T"], s["E"], s["topk"], s["K"], s["I"]
    ids = s["ids"].long()
    share = torch.zeros(T, E + 1, device=ids.device).scatter_add_(1, torch.where(ids < 0, E, ids), s["w"])[:, :E]
    on = torch.unique(ids[ids >= 0])
    gu = _act_hat(s["X"].float(), s["fmt"]) @ _w_hat(s["W13q"][on], s["W13s"][on], s["fmt"]).flatten(0, 1).T
    gu = gu.view(T, -1, I // 128, 2, 128)
    g, u = gu[:, :, :, 0].flatten(-2), gu[:, :, :, 1].flatten(-2)
    h = _act_hat(g / (1 + torch.exp(-g)) * u, s["fmt"])                            # [T, experts, I]
    out = torch.bmm(h.transpose(0, 1), _w_hat(s["W2q"][on], s["W2s"][on], s["fmt"]).transpose(1, 2))
    y = (out * share[:, on].T[:, :, None]).sum(dim=0)
    if s["R"] is not None:
        y = y + s["R"].float()
    return y.to(torch.bfloat16)


# ---------------------------------------------------------------------------------------------- the run
def run(state):
    s = state
    if own:
        import fine_grained_fp8_token_b200 as fg
        if s["op"] == "linear":
            return fg.linear_epilogue(s["X"], s["Wq"], s["Ws"], s["fmt"], bias=s["bias"], act=s["act"], residual=s["R"])
        if s["op"] == "route":
            return fg.route_topk(s["logits"], s["topk"], score=s["score"], bias=s["b"], n_group=s["groups"],
                                 topk_group=s["keep"], renormalize=True)
        return fg.moe_decode(s["X"], s["ids"], s["w"], s["W13q"], s["W13s"], s["W2q"], s["W2s"], s["fmt"],
                             residual=s["R"])
    if s["op"] == "linear":
        return _linear(s)
    if s["op"] == "route":
        return _route(s)
    return _moe(s)


# -------------------------------------------------------------------------------- the definition in 64 bits
def _x64(x, fmt):
    """Codes and scales of the definition (each of its steps one rounding to fp32), multiplied in 64 bits."""
    M, K = x.shape
    v = x.double().reshape(M, K // 128, 128)
    amax = v.abs().max(dim=2).values
    amax = torch.where(amax < 1e-4, torch.full_like(amax, 1e-4), amax).float().double()
    s = (amax / 448).float().double()
    if fmt == UE8M0:
        s = torch.exp2(torch.ceil(torch.log2(s)))
    q = (v / s[:, :, None]).float()
    q = torch.maximum(torch.minimum(q, torch.full_like(q, 448.0)), torch.full_like(q, -448.0))
    return (q.to(torch.float8_e4m3fn).double() * s[:, :, None]).reshape(M, K)


def _w64(q, s, fmt):
    if fmt == UE8M0:
        s = torch.exp2(s.double() - 127)
    s = s.double().repeat_interleave(128, dim=0).repeat_interleave(128, dim=1)
    return q.view(torch.float8_e4m3fn).double() * s


def _exact_linear(s):
    X = _x64(s["X"], s["fmt"])
    y = torch.empty(s["M"], s["N"], dtype=torch.float64, device=DEV)
    for n in range(0, s["N"], 2048):
        rows = slice(n, min(n + 2048, s["N"]))
        blocks = slice(n // 128, (rows.stop + 127) // 128)
        y[:, rows] = X @ _w64(s["Wq"][rows], s["Ws"][blocks], s["fmt"]).T
    if s["bias"] is not None:
        y += s["bias"].double()
    a = s["act"]
    if a == "relu":
        y = torch.where(y > 0, y, torch.zeros_like(y))
    elif a == "silu":
        y = y * torch.sigmoid(y)
    elif a == "gelu":
        y = y * (0.5 * torch.erfc(-y / math.sqrt(2)))
    elif a == "gelu_tanh":
        y = y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y))
    return y if s["R"] is None else y + s["R"].double()


def _exact_route(s):
    z = s["logits"].double().cpu()
    T, E, G = s["T"], s["E"], s["groups"]
    soft = s["score"] == "softmax"
    if soft:
        m = z.max(dim=1, keepdim=True).values
        p = torch.exp(z - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    else:
        p = torch.sigmoid(z)
    key = (z if soft else p) + (0 if s["b"] is None else s["b"].double().cpu())
    dead = torch.isinf(z)
    key[dead] = -math.inf
    if G > 1:
        per = key.reshape(T, G, E // G)
        first = per.max(dim=2)
        score = first.values.clone()
        if not soft:
            rest = per.scatter(2, first.indices[:, :, None], -math.inf).max(dim=2).values
            score = torch.where(torch.isinf(rest), score, score + rest)
        alive = torch.zeros(T, G, dtype=torch.bool)
        for _ in range(s["keep"]):
            best = score.masked_fill(alive, -math.inf).max(dim=1, keepdim=True).indices
            alive.scatter_(1, best, True)
        key[~alive.repeat_interleave(E // G, dim=1)] = -math.inf
    w = torch.zeros(T, s["topk"], dtype=torch.float64)
    for j in range(s["topk"]):
        top = key.max(dim=1, keepdim=True)
        w[:, j:j + 1] = torch.where(torch.isinf(top.values), torch.zeros_like(top.values), p.gather(1, top.indices))
        key.scatter_(1, top.indices, -math.inf)
    total = w.sum(dim=1, keepdim=True)
    return None, torch.where(total > 0, w / total, w)


def _exact_moe(s):
    T, I, fmt = s["T"], s["I"], s["fmt"]
    X = _x64(s["X"], fmt)
    y = torch.zeros(T, s["K"], dtype=torch.float64, device=DEV) if s["R"] is None else s["R"].double()
    for e in sorted(set(s["ids"].flatten().tolist()) - {-1}):
        hit = s["ids"] == e
        rows = hit.any(dim=1).nonzero().flatten()
        gu = X[rows] @ _w64(s["W13q"][e], s["W13s"][e], fmt).T
        gu = gu.reshape(len(rows), I // 128, 256)
        g, u = gu[:, :, :128].reshape(-1, I), gu[:, :, 128:].reshape(-1, I)
        out = _x64(g * torch.sigmoid(g) * u, fmt) @ _w64(s["W2q"][e], s["W2s"][e], fmt).T
        y[rows] += out * (s["w"].double() * hit)[rows].sum(dim=1, keepdim=True)
    return y


def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _exact_linear, "route": _exact_route, "moe": _exact_moe}[s["op"]](s)
