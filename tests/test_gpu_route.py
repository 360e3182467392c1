"""GPU checks of the expert router (fgfp8_route_topk) against the definition in
64 bits, written as loops over tokens: ids equal, weights within the fp32
arithmetic's error.  Each chosen p carries the errors of one exp (2 ulp), its
argument (|z - max| 2^-24 relative) and one division; the sum of up to 512 of
them adds 2^-24 each in a tree of depth 9 + 5: 2^-19 relative covers all of it
for |z| <= 16.  Beyond that the rounding of z - max counts: it is off by
|z - max| 2^-24, which moves exp(z - max) by that much relatively, so a weight
exp(-d) times the largest may be off by another d 2^-24; weights below fp32's
normal numbers are off by up to their step, 2^-149."""
import math

import numpy as np
import pytest
import torch

import fine_grained_fp8_token_b200 as fg
from parity import Guarded, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    d = require_gpu()
    fg.load()
    return d


def reference(z, topk, score, bias, G, keep, renorm, scale):
    z = z.double().cpu().numpy().copy()
    T, E = z.shape
    z[np.isnan(z)] = -np.inf
    b = np.zeros(E) if bias is None else bias.double().cpu().numpy()
    ids, w = np.full((T, topk), -1, dtype=np.int32), np.zeros((T, topk))
    for t in range(T):
        if score == "softmax":
            m = z[t].max()
            key = z[t].copy()
            if m == -np.inf:
                p = np.zeros(E)
            else:
                with np.errstate(invalid="ignore"):           # inf - inf where z is the maximum itself
                    p = np.where(z[t] == m, 1.0, np.exp(np.where(z[t] == m, 0.0, z[t] - m)))
                p = p / p.sum()
        else:
            with np.errstate(over="ignore"):
                p = 1 / (1 + np.exp(-z[t]))
            key = p + b
        key[z[t] == -np.inf] = -np.inf
        key[np.isnan(key)] = -np.inf
        per = E // G
        if G > 1:
            s = []
            for g in range(G):
                k = np.sort(key[g * per:(g + 1) * per])[::-1]
                two = score == "sigmoid" and per > 1 and k[1] > -np.inf
                s.append(k[0] + k[1] if two else k[0])
            best = sorted(range(G), key=lambda g: (-s[g], g))[:keep]
            for g in range(G):
                if g not in best:
                    key[g * per:(g + 1) * per] = -np.inf
        if bias is None:                             # the logits' order is the sigmoids' in exact arithmetic
            key = np.where(key > -np.inf, z[t], -np.inf)
        order = sorted(range(E), key=lambda e: (-key[e], e))[:topk]
        chosen = [e for e in order if key[e] > -np.inf]
        total = max(sum(p[e] for e in chosen), 1e-20) if renorm else 1.0
        for j, e in enumerate(chosen):
            ids[t, j], w[t, j] = e, p[e] / total * scale
    return ids, w


def check(dev, z, topk, score="softmax", bias=None, G=1, keep=1, renorm=True, scale=1.0):
    T = z.shape[0]
    i, w = Guarded((T, topk), torch.int32, dev), Guarded((T, topk), torch.float32, dev)
    zd = z.to(dev)
    bd = None if bias is None else bias.to(dev)
    fg.route_topk(zd, topk, score=score, bias=bd, n_group=G, topk_group=keep, renormalize=renorm, scale=scale,
                  ids=i.t, weights=w.t)
    fg.check_device_status()
    ri, rw = reference(z, topk, score, bias, G, keep, renorm, scale)
    gi, gw = i.t.cpu().numpy(), w.t.double().cpu().numpy()
    bad = np.argwhere(gi != ri)
    assert len(bad) == 0, f"{len(bad)} ids differ, first at {bad[0]}: {gi[bad[0][0]]} {ri[bad[0][0]]}"
    d = np.log(np.maximum(rw.max(axis=1, keepdims=True), 1e-300)) - np.log(np.maximum(rw, 1e-300))
    tol = (2.0 ** -19 + d * 2.0 ** -24) * np.abs(rw) + 2.0 ** -149
    assert (np.abs(gw - rw) <= tol).all(), np.abs(gw - rw).max()
    i.check()
    w.check()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,topk", [(1, 1, 1), (1, 256, 8), (3, 2, 2), (5, 31, 4), (130, 32, 1), (64, 33, 16),
                                      (257, 64, 6), (33, 160, 6), (50, 257, 8), (40, 512, 16)])
def test_softmax(dev, T, E, topk, dtype):
    z = torch.randn(T, E, generator=torch.Generator().manual_seed(T + E)).to(dtype)
    for renorm in (True, False):
        check(dev, z, topk, renorm=renorm, scale=1.0 if renorm else 2.5)


@pytest.mark.parametrize("T,E,topk,G,keep", [(1, 256, 8, 8, 4), (77, 256, 8, 8, 4), (40, 60, 6, 4, 3), (33, 512, 16, 32, 16),
                                             (20, 64, 4, 1, 1), (20, 8, 3, 8, 5), (9, 96, 2, 3, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_and_bias(dev, T, E, topk, G, keep, score):
    g = torch.Generator().manual_seed(E + G)
    z = torch.randn(T, E, generator=g) * 2
    b = torch.randn(E, generator=g) * 0.3 if score == "sigmoid" else None
    check(dev, z, topk, score=score, G=G, keep=keep)
    if b is not None:
        check(dev, z, topk, score=score, bias=b, G=G, keep=keep, renorm=False, scale=2.5)
        check(dev, z.bfloat16(), topk, score=score, bias=b * 100, G=G, keep=keep)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G,keep", [(1, 1), (4, 2)])
def test_masks_ties_and_infinities(dev, score, G, keep):
    E, topk = 64, 8
    g = torch.Generator().manual_seed(3)
    z = torch.randn(24, E, generator=g)
    z[0] = -math.inf                                 # nothing to choose
    z[1, 3:] = -math.inf                             # fewer than topk
    z[2] = torch.finfo(torch.float32).min            # the lowest finite value is still a score
    z[3, ::2] = float("nan")
    z[4] = 0.0                                       # all equal: lowest indexes
    z[5, 10:20] = 4.0
    z[6, 17:] = -math.inf
    z[7, :16] = -math.inf                            # a whole group off
    z[8] = (z[8] * 2).round() / 2                    # many ties
    z[9, 5] = 80.0
    z[10] = z[10] - 60
    z[13] = z[13] - 1000                             # sigmoids that vanish in 32 bits, and in 64
    z[14] = 0.0
    z[14, ::3] = -0.0                                # the two zeros are equal
    z[15] = z[15] * 0.01 + 40                        # sigmoids that are 1 in 64 bits
    check(dev, z, topk, score=score, G=G, keep=keep)
    if score == "sigmoid":
        b = torch.zeros(E)
        b[7] = -math.inf
        b[11] = float("nan")
        check(dev, z, topk, score=score, bias=b, G=G, keep=keep)
    else:
        z[11, 4] = math.inf
        z[12, 4] = z[12, 40] = math.inf
        check(dev, z, topk, score=score, G=G, keep=keep)


def test_near_ties_in_64_bits(dev):
    """Sigmoid keys that agree in 32 bits and differ in 64 keep their order:
    neighbouring logits near 15 (sigmoid steps of 3e-13), with a bias."""
    z = torch.full((4, 32), 15.0)
    step = 2.0 ** -20
    perm = torch.randperm(32, generator=torch.Generator().manual_seed(1))
    z[0] += perm * step
    z[1] += perm.flip(0) * step
    z[2, 16:] += step
    z[3, 5] += step
    check(dev, z, 8, score="sigmoid")
    check(dev, z, 8, score="sigmoid", bias=torch.full((32,), 0.25))
    check(dev, z, 8, score="sigmoid", bias=torch.full((32,), 0.25), G=4, keep=2)
    # more close keys than a warp has lanes, distinct and equal ones
    for E, G, keep in ((40, 1, 1), (256, 8, 4), (512, 4, 2)):
        z = torch.full((6, E), 14.0)
        for t in range(3):
            z[t] += torch.randperm(E, generator=torch.Generator().manual_seed(t)) * 2.0 ** -20
        z[4, 7:] = -math.inf
        z[5, ::2] = -1.0
        check(dev, z, 8, score="sigmoid", bias=torch.full((E,), 0.25))
        check(dev, z, 8, score="sigmoid", bias=torch.full((E,), 0.25), G=G, keep=keep)
        check(dev, z, 8, score="sigmoid", bias=torch.arange(E).flip(0) * 2.0 ** -40, G=G, keep=keep)
        check(dev, z, 8, score="sigmoid", G=G, keep=keep)


def test_strided_and_many_tokens(dev):
    wide = torch.randn(3000, 150, generator=torch.Generator().manual_seed(2))
    check(dev, wide[:, 11:139], 6)
    zd = wide.to(dev)[:, 11:139]
    i, w = fg.route_topk(zd, 6)
    ri, rw = reference(wide[:, 11:139], 6, "softmax", None, 1, 1, True, 1.0)
    assert (i.cpu().numpy() == ri).all()
    i0, _ = fg.route_topk(zd[:0], 6)
    assert i0.shape == (0, 6)
    fg.check_device_status()


def test_graph_replay(dev):
    z = torch.randn(50, 256, generator=torch.Generator().manual_seed(7)).to(dev)
    i, w = fg.route_topk(z, 8, score="sigmoid", n_group=8, topk_group=4)
    buf = torch.zeros_like(z)
    gi, gw = torch.empty_like(i), torch.empty_like(w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fg.route_topk(buf, 8, score="sigmoid", n_group=8, topk_group=4, ids=gi, weights=gw)
    buf.copy_(z)
    graph.replay()
    assert torch.equal(i, gi) and torch.equal(w, gw)
