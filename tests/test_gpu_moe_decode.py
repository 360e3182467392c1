"""GPU checks of the few-token expert layer (fgfp8_moe_decode) against its
formula in 64 bits.

Tolerance, before the run.  The sums g and u are within dg = 1e-4 S of the exact
ones (the GEMM's bound, S = sum |x_hat w_hat|), so h = silu(g) u is within
dh = 1.1 dg (|u| + du) + |silu(g)| du + 2^-20 |h| (silu's slope is at most 1.1).
The quantizer then divides by a scale that is within max(dh) / 448 of the
exact one.  Where h / s lies further than its error from the border of two E4M3
codes the code is the same, and only the scale's error remains; else the
code may be the neighbour's, one step (2^-3 of the value at most, 2^-9 below
2^-6) away.  For power-of-two scales a group whose amax / 448 lies within its
error of a power of two may take the other scale, which moves every value by
half a step (2^-4) on either side at most.  These sum over I with |W2 hat|, over
the experts with their weights, then the second GEMM's 1e-4 S, and half a bf16
step of the result."""
import numpy as np
import pytest
import torch

import fine_grained_fp8_token_b200 as fg
import oracle
import workloads
from parity import Guarded, bits16, require_gpu, to_np, y_to_f64

pytestmark = pytest.mark.gpu
F32, UE8M0 = 0, 1
TABLE = None


@pytest.fixture(scope="module")
def dev():
    d = require_gpu()
    fg.load()
    return d


def weights_for(dev, E, K, I, fmt, seed):
    W13q = torch.empty(E, 2 * I, K, dtype=torch.uint8, device=dev)
    W2q = torch.empty(E, K, I, dtype=torch.uint8, device=dev)
    sd = torch.float32 if fmt == F32 else torch.uint8
    W13s = torch.empty(E, 2 * I // 128, K // 128, dtype=sd, device=dev)
    W2s = torch.empty(E, K // 128, I // 128, dtype=sd, device=dev)
    for e in range(E):
        gate, up = (workloads.weights((I, K), seed=seed + 10 * e + j, device=dev) for j in (0, 1))
        fg.quant_weight(fg.interleave_gate_up(gate, up), fmt, W13q[e], W13s[e])
        fg.quant_weight(workloads.weights((K, I), seed=seed + 10 * e + 2, device=dev), fmt, W2q[e], W2s[e])
    return W13q, W13s, W2q, W2s


def quant64(h, dh, fmt):
    """What the 1x128 quantizer leaves of h [n, I], and by how much the result
    may differ when h is off by dh."""
    n, I = h.shape
    v, d = h.reshape(n, -1, 128), dh.reshape(n, -1, 128)
    amax = np.maximum(np.abs(v).max(axis=2, keepdims=True), 1e-4)
    damax = d.max(axis=2, keepdims=True)
    r = (amax / 448).astype(np.float32).astype(np.float64)
    dr = damax / 448 + 2.0 ** -22 * r
    if fmt == UE8M0:
        s = np.exp2(np.ceil(np.log2(r)))
        turns = (np.ceil(np.log2(r + dr)) != np.ceil(np.log2(np.maximum(r - dr, 1e-30))))
        ds = np.zeros_like(s)
    else:
        s, ds, turns = r, dr, np.zeros(r.shape, dtype=bool)
    q = v / s
    codes = oracle.e4m3_encode(q.astype(np.float32)).reshape(q.shape)
    global TABLE
    if TABLE is None:
        TABLE = oracle.e4m3_table()
    val = TABLE[codes]
    mag = np.abs(q)
    e = np.floor(np.log2(np.maximum(mag, 2.0 ** -6)))
    step = np.exp2(e - 3)
    dq = d / s + mag * ds / s + 2.0 ** -22 * mag
    off = np.abs(np.mod(mag / step, 1.0) - 0.5) * step
    err = np.abs(val) * ds + np.where(off <= dq, step * s, 0.0)
    # the other scale is a factor of two away: half a step of each
    err = np.where(turns, 2 * step * s, err)
    return (val * s).reshape(n, I), err.reshape(n, I)


def reference(X, ids, w, W, fmt, R):
    W13q, W13s, W2q, W2s = (to_np(t) for t in W)
    E, K, I = W2q.shape
    T = X.shape[0]
    Xq, Xs = oracle.quant_act(bits16(X), fmt)
    x = oracle.dequant_act(Xq, Xs, fmt)[:T]
    y = np.zeros((T, K)) if R is None else R.double().cpu().numpy()
    tol = np.zeros((T, K))
    for e in range(E):
        hit = ids == e
        rows = np.nonzero(hit.any(axis=1))[0]
        if not len(rows):
            continue
        wt = (w.astype(np.float64) * hit)[rows].sum(axis=1, keepdims=True)
        w13 = oracle.dequant_weight(W13q[e], W13s[e], fmt)
        w2 = oracle.dequant_weight(W2q[e], W2s[e], fmt)
        gu = (x[rows] @ w13.T).reshape(len(rows), I // 128, 2, 128)
        S = (np.abs(x[rows]) @ np.abs(w13).T).reshape(gu.shape)
        g, u = gu[:, :, 0].reshape(-1, I), gu[:, :, 1].reshape(-1, I)
        dg, du = 1e-4 * S[:, :, 0].reshape(-1, I), 1e-4 * S[:, :, 1].reshape(-1, I)
        sg = g / (1 + np.exp(-g))
        h = sg * u
        dh = 1.1 * dg * (np.abs(u) + du) + np.abs(sg) * du + 2.0 ** -20 * np.abs(h)
        hh, eh = quant64(h, dh, fmt)
        y[rows] += wt * (hh @ w2.T)
        tol[rows] += np.abs(wt) * (eh @ np.abs(w2).T + 1e-4 * (np.abs(hh) @ np.abs(w2).T))
    return y, tol + 2.0 ** -8 * np.abs(y) + 2.0 ** -20


def route(T, E, topk, seed, holes=0.0):
    g = torch.Generator().manual_seed(seed)
    ids = torch.stack([torch.randperm(E, generator=g)[:topk] for _ in range(T)]).to(torch.int32)
    ids = torch.where(torch.rand(T, topk, generator=g) < holes, torch.full_like(ids, -1), ids)
    w = torch.softmax(torch.randn(T, topk, generator=g), dim=1)
    return ids, w


def run(dev, X, ids, w, W, fmt, R=None, **kw):
    return fg.moe_decode(X.to(dev), ids.to(dev), w.to(dev), *W, fmt, residual=None if R is None else R.to(dev), **kw)


def check(Y, ref, tol, what=""):
    got = y_to_f64(Y)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][:3]} {ref[bad][:3]} {tol[bad][:3]}")


@pytest.mark.parametrize("fmt", [F32, UE8M0])
@pytest.mark.parametrize("T,E,topk,K,I", [(1, 4, 1, 128, 128), (1, 16, 8, 1024, 256), (2, 3, 3, 256, 384),
                                          (5, 8, 2, 640, 128), (16, 8, 4, 512, 256), (17, 8, 2, 384, 128),
                                          (31, 40, 8, 256, 128), (64, 4, 2, 512, 384), (64, 16, 16, 256, 128),
                                          (33, 512, 3, 128, 128), (1, 12, 8, 7168, 1024), (20, 3, 2, 4096, 1024)])
def test_against_the_formula(dev, T, E, topk, K, I, fmt):
    W = weights_for(dev, E, K, I, fmt, seed=T + E)
    X = workloads.activations((T, K), "normal", seed=T)
    ids, w = route(T, E, topk, seed=T + 1)
    R = workloads.activations((T, K), "normal", seed=T + 2) if T % 2 else None
    out = Guarded((T, K), torch.bfloat16, dev)
    n = fg.moe_workspace_bytes(T, topk, K, I)
    ws = Guarded((n,), torch.uint8, dev, fill=0xFF)          # NaN codes and scales: nothing stale is read
    Y = run(dev, X, ids, w, W, fmt, R, Y=out.t, workspace=ws.t)
    fg.check_device_status()
    check(Y, *reference(X, ids.numpy(), w.numpy(), W, fmt, R))
    out.check()
    ws.check("workspace")


@pytest.mark.parametrize("T", [6, 40])
def test_empty_slots_repeats_and_crowds(dev, T):
    """Empty slots, tokens without any expert, an expert named twice, every
    token at one expert, zero and negative weights."""
    E, topk, K, I, fmt = 6, 4, 256, 256, F32
    W = weights_for(dev, E, K, I, fmt, seed=77)
    X = workloads.activations((T, K), "normal", seed=1)
    R = workloads.activations((T, K), "normal", seed=2)
    ids, w = route(T, E, topk, seed=3, holes=0.4)
    ids[0] = -1
    ids[1] = torch.tensor([2, 2, -7, 2])
    ids[2] = torch.tensor([5, 0, 5, 0])
    w[3, 0], w[3, 1] = 0.0, -0.75
    for r in (None, R):
        check(run(dev, X, ids, w, W, fmt, r), *reference(X, ids.numpy(), w.numpy(), W, fmt, r))
    Y = run(dev, X, ids, w, W, fmt, R)
    assert torch.equal(Y[0].cpu(), R[0])                     # no expert: the residual as it was
    assert not run(dev, X, ids, w, W, fmt)[0].any()          # and zero without one
    one = torch.full((T, topk), -1, dtype=torch.int32)
    one[:, 2] = 4
    check(run(dev, X, one, w, W, fmt), *reference(X, one.numpy(), w.numpy(), W, fmt, None))
    none = torch.full((T, topk), -1, dtype=torch.int32)
    assert torch.equal(run(dev, X, none, w, W, fmt, R).cpu(), R)
    fg.check_device_status()


def test_bad_expert_is_reported(dev):
    E, topk, K, I = 4, 2, 128, 128
    W = weights_for(dev, E, K, I, F32, seed=5)
    X = workloads.activations((3, K), "normal", seed=1)
    ids, w = route(3, E, topk, seed=3)
    bad = ids.clone()
    bad[1, 0] = E
    Y = run(dev, X, bad, w, W, F32)
    with pytest.raises(fg.FGFP8Error) as err:
        fg.check_device_status()
    assert err.value.status == 7
    skipped = bad.clone()
    skipped[1, 0] = -1
    assert torch.equal(Y, run(dev, X, skipped, w, W, F32))
    fg.check_device_status()


def test_strides_in_place_stream_and_repeat(dev):
    """A strided X and residual, the residual being the output, a side stream,
    and the same bits from call to call."""
    T, E, topk, K, I, fmt = 9, 12, 3, 384, 256, UE8M0
    W = weights_for(dev, E, K, I, fmt, seed=8)
    X = workloads.activations((T, K), "normal", seed=4)
    R = workloads.activations((T, K), "normal", seed=5)
    ids, w = route(T, E, topk, seed=6)
    first = run(dev, X, ids, w, W, fmt, R)
    check(first, *reference(X, ids.numpy(), w.numpy(), W, fmt, R))
    wide = torch.full((T, K + 72), 3.0, dtype=torch.bfloat16, device=dev)
    wide[:, 24:24 + K] = X.to(dev)
    rwide = torch.full((T, K + 8), 3.0, dtype=torch.bfloat16, device=dev)
    rwide[:, 8:] = R.to(dev)
    args = (ids.to(dev), w.to(dev), *W, fmt)
    assert torch.equal(first, fg.moe_decode(wide[:, 24:24 + K], *args, residual=rwide[:, 8:]))
    Y = R.to(dev).clone()
    fg.moe_decode(X.to(dev), *args, residual=Y, Y=Y)
    assert torch.equal(first, Y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    Z = fg.moe_decode(X.to(dev), *args, residual=R.to(dev), stream=side)
    side.synchronize()
    assert torch.equal(first, Z)
    for _ in range(20):
        assert torch.equal(first, run(dev, X, ids, w, W, fmt, R))
    fg.check_device_status()


def test_graph_replays_with_other_routing(dev):
    T, E, topk, K, I, fmt = 8, 16, 4, 256, 128, F32
    W = weights_for(dev, E, K, I, fmt, seed=9)
    X = torch.zeros(T, K, dtype=torch.bfloat16, device=dev)
    ids = torch.full((T, topk), -1, dtype=torch.int32, device=dev)
    w = torch.zeros(T, topk, device=dev)
    Y = torch.empty(T, K, dtype=torch.bfloat16, device=dev)
    ws = torch.empty(fg.moe_workspace_bytes(T, topk, K, I), dtype=torch.uint8, device=dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fg.moe_decode(X, ids, w, *W, fmt, Y=Y, workspace=ws)
    for seed in range(3):
        x = workloads.activations((T, K), "normal", seed=seed)
        i, v = route(T, E, topk, seed=seed, holes=0.2 * seed)
        X.copy_(x), ids.copy_(i), w.copy_(v)
        graph.replay()
        assert torch.equal(Y, run(dev, x, i, v, W, fmt))
    fg.check_device_status()


def test_agrees_with_the_masked_path(dev):
    """The masked layout's layers (GEMM, SwiGLU in bf16, quantizer, GEMM) on the
    same routing: equal up to that path's bf16 roundings of g, u and h (2^-8
    each, which also move codes) and of its output."""
    T, E, topk, K, I, fmt = 12, 6, 2, 512, 256, F32
    W13q, W13s, W2q, W2s = W = weights_for(dev, E, K, I, fmt, seed=31)
    X = workloads.activations((T, K), "normal", seed=7).to(dev)
    ids, w = route(T, E, topk, seed=11)
    Y = run(dev, X, ids, w, W, fmt).float()
    cap = 128
    rows = torch.zeros(E * cap, K, dtype=torch.bfloat16, device=dev)
    counts = torch.zeros(E, dtype=torch.int32)
    where = {}
    for t in range(T):
        for j in range(topk):
            e = int(ids[t, j])
            where[t, j] = e * cap + int(counts[e])
            rows[where[t, j]] = X[t]
            counts[e] += 1
    cd = counts.to(dev)
    gu = fg.masked_linear(rows, W13q, W13s, cd, fmt).float().view(E * cap, I // 128, 2, 128)
    h = (torch.nn.functional.silu(gu[:, :, 0]) * gu[:, :, 1]).reshape(E * cap, I).to(torch.bfloat16)
    out = fg.masked_linear(h, W2q, W2s, cd, fmt).float()
    ref = torch.stack([sum(w[t, j].item() * out[where[t, j]] for j in range(topk)) for t in range(T)])
    fg.check_device_status()
    assert ((Y - ref).norm() / ref.norm()).item() < 0.03


def test_attention_output_router_and_experts_together(dev):
    """The decode step they serve: output projection + residual, router
    logits, routing, expert layer + residual; each stage against its own
    formula on the previous stage's output."""
    T, E, topk, K, I, fmt = 10, 128, 4, 512, 128, F32
    A = workloads.activations((T, K), "normal", seed=1)
    R = workloads.activations((T, K), "normal", seed=2)
    Wo = workloads.weights((K, K), seed=3)
    Wg = workloads.weights((E, K), seed=4, std=0.3)
    Woq, Wos = fg.quant_weight(Wo.to(dev), fmt)
    Wgq, Wgs = fg.quant_weight(Wg.to(dev), fmt)
    W = weights_for(dev, E, K, I, fmt, seed=100)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        x = fg.linear_epilogue(A.to(dev), Woq, Wos, fmt, residual=R.to(dev))
        logits = fg.linear_epilogue(x, Wgq, Wgs, fmt)
        ids, w = fg.route_topk(logits, topk, score="sigmoid", n_group=4, topk_group=2)
        Y = fg.moe_decode(x, ids, w, *W, fmt, residual=x)
    side.synchronize()
    fg.check_device_status()
    aq, asc = oracle.quant_act(bits16(A), fmt)
    acc, S = oracle.gemm(aq, asc, to_np(Woq), to_np(Wos), fmt)
    ref = acc + R.double().numpy()
    check(x, ref, 1e-4 * S + 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * np.abs(R.double().numpy()))
    from test_gpu_route import reference as route_reference
    ri, rw = route_reference(logits, topk, "sigmoid", None, 4, 2, True, 1.0)
    assert (ids.cpu().numpy() == ri).all()
    check(Y, *reference(x, ri, w.cpu().numpy(), W, fmt, x))


@pytest.mark.parametrize("T", [1, 12, 40])
def test_the_step_replayed_back_to_back(dev, T):
    """Output projection, router and two expert layers captured in one graph
    and replayed without a wait between the replays: each kernel may start
    while the one before it ends, and the results are those of the calls made
    one at a time."""
    E, topk, K, I, fmt = 128, 4, 512, 256, UE8M0
    Woq, Wos = fg.quant_weight(workloads.weights((K, K), seed=3).to(dev), fmt)
    Wgq, Wgs = fg.quant_weight(workloads.weights((E, K), seed=4, std=0.3).to(dev), fmt)
    W = weights_for(dev, E, K, I, fmt, seed=500)

    def step(a, r, wait):
        def after(x):
            if wait:
                torch.cuda.synchronize()
            return x
        x = after(fg.linear_epilogue(a, Woq, Wos, fmt, residual=r))
        for _ in range(2):
            logits = after(fg.linear_epilogue(x, Wgq, Wgs, fmt))
            ids, w = after(fg.route_topk(logits, topk, score="sigmoid"))
            x = after(fg.moe_decode(x, ids, w, *W, fmt, residual=x))
        return x
    inputs = [[workloads.activations((T, K), "normal", seed=10 * s + j).to(dev) for j in (0, 1)] for s in range(4)]
    alone = [step(a, r, True) for a, r in inputs]
    a, r = (torch.zeros_like(t) for t in inputs[0])
    step(a, r, True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(a, r, False)
    got = []
    for i in range(12):
        a.copy_(inputs[i % 4][0]), r.copy_(inputs[i % 4][1])
        graph.replay()
        got.append(out.clone())
    eager = [step(*inputs[i % 4], False) for i in range(8)]
    torch.cuda.synchronize()
    fg.check_device_status()
    for i, y in enumerate(got):
        assert torch.equal(y, alone[i % 4]), i
    for i, y in enumerate(eager):
        assert torch.equal(y, alone[i % 4]), i


def test_two_streams_with_workspaces_of_their_own(dev):
    """Two expert layers at once on two streams give what they give alone."""
    T, E, topk, K, I, fmt = 6, 16, 4, 512, 256, F32
    W = weights_for(dev, E, K, I, fmt, seed=600)
    calls = []
    for s in range(2):
        X = workloads.activations((T, K), "normal", seed=s).to(dev)
        ids, w = route(T, E, topk, seed=s)
        calls.append((X, ids.to(dev), w.to(dev)))
    alone = [fg.moe_decode(*c, *W, fmt) for c in calls]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for i in range(30):
        outs.append((i % 2, fg.moe_decode(*calls[i % 2], *W, fmt, stream=streams[i % 2])))
    torch.cuda.synchronize()
    fg.check_device_status()
    for i, y in outs:
        assert torch.equal(y, alone[i])


def test_zero_tokens(dev):
    W = weights_for(dev, 2, 128, 128, F32, seed=1)
    X = torch.empty(0, 128, dtype=torch.bfloat16, device=dev)
    Y = fg.moe_decode(X, torch.empty(0, 2, dtype=torch.int32, device=dev), torch.empty(0, 2, device=dev), *W, F32)
    assert Y.shape == (0, 128)


@pytest.mark.parametrize("fmt", [F32, UE8M0])
@pytest.mark.parametrize("T", [7, 40])
def test_tokens_that_are_not_finite_stay_alone(dev, T, fmt):
    """A token with a NaN, one with an infinity: not finite themselves, and the
    others' rows are as without them."""
    E, topk, K, I = 5, 3, 384, 256
    W = weights_for(dev, E, K, I, fmt, seed=6)
    X = workloads.activations((T, K), "normal", seed=1)
    R = workloads.activations((T, K), "normal", seed=2)
    ids, w = route(T, E, topk, seed=3)
    clean = run(dev, X, ids, w, W, fmt, R)
    X[1, 200], X[T - 2, 7] = float("nan"), float("inf")
    Y = run(dev, X, ids, w, W, fmt, R)
    fg.check_device_status()
    rest = [t for t in range(T) if t not in (1, T - 2)]
    assert torch.equal(Y[rest], clean[rest])
    assert not Y[1].isfinite().any() and not Y[T - 2].isfinite().any()


def test_long_rows(dev):
    """K and I far above the usual ones (hundreds of K blocks a piece), and
    the narrowest layer against them."""
    for T, K, I in ((2, 65536, 128), (20, 128, 32768)):
        E, topk, fmt = 2, 2, F32
        W = weights_for(dev, E, K, I, fmt, seed=2)
        X = workloads.activations((T, K), "normal", seed=1)
        ids, w = route(T, E, topk, seed=3)
        check(run(dev, X, ids, w, W, fmt), *reference(X, ids.numpy(), w.numpy(), W, fmt, None))
    fg.check_device_status()
