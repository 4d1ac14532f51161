"""The behaviour-history tower: its operators together, as a program uses them,
against a plain 64-bit model of the same parameters."""
import math

import numpy as np
import pytest
import torch

import history_ref as R
from dlrm_cases import DEV, banner

pytestmark = pytest.mark.gpu

V, D, H, DK, DV, L = 500, 64, 2, 32, 32, 2


def _parameters(seed):
    g = torch.Generator().manual_seed(seed)
    bf = lambda t: t.to(torch.bfloat16).float()  # noqa: E731
    layers = []
    for _ in range(L):
        Wqkv = bf(torch.randn(H * (2 * DK + DV), D, generator=g) / math.sqrt(D))
        Wo = bf(torch.randn(D, H * DV, generator=g) / math.sqrt(H * DV))
        layers.append((1 + 0.2 * torch.randn(D, generator=g), Wqkv, Wo, torch.tensor([0.9, 0.97])))
    table = bf(torch.randn(V, D, generator=g) / math.sqrt(D))
    return table, layers, 1 + 0.2 * torch.randn(D, generator=g)


def _tower(params, **kw):
    from deep_learning_recommendation_amd import history as HT

    table, layers, w_out = params
    dt = torch.float32 if kw.get("train") else torch.bfloat16
    return HT.HistoryTower(table.to(dt).to(DEV), [HT.make_layer(*p) for p in layers], w_out.to(DEV), H, DK, DV, **kw)


def _histories(seed, lens):
    g = torch.Generator().manual_seed(seed)
    off = torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(torch.tensor(lens), 0)])
    tok = torch.randint(-1, V, (int(off[-1]),), generator=g)
    return tok, off


def _model(params, tok, off, keep, eps=1e-6):
    """The tower in fp64 torch on the CPU; keep[i]: branch i's mask and factor."""
    table, layers, w_out = params
    x = torch.where((tok >= 0)[:, None], table[tok.clamp(min=0)], 0.0) * math.sqrt(D)

    def norm(i, x, res, w):
        m, f = keep[i]
        h = torch.where(m, x * f, torch.zeros((), dtype=x.dtype))
        h = h if res is None else h + res
        return h, h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * w

    res = None
    for i, (w, Wqkv, Wo, lam) in enumerate(layers):
        res, y = norm(i, x, res, w)
        q, k, v = (y @ Wqkv.T).split([H * DK, H * DK, H * DV], 1)
        q, k, v = q.view(-1, H, DK), k.view(-1, H, DK), v.view(-1, H, DV)
        t = torch.arange(len(tok))
        hist = torch.bucketize(t, off[1:], right=True)
        D_ = torch.where((t[:, None] >= t) & (hist[:, None] == hist), 1.0, 0.0)
        dec = lam.double()[:, None, None] ** (t[:, None] - t).clamp(min=0).double() * D_
        o = torch.einsum("hti,ihd->thd", torch.einsum("thc,ihc->hti", q, k) * dec, v) * DK ** -0.5
        x = o.reshape(-1, H * DV) @ Wo.T
    _, y = norm(L, x, res, w_out)
    last = off[1:] - 1
    return torch.where((off[1:] > off[:-1])[:, None], y[last.clamp(min=0)], 0.0)


def _everything(n):
    return [(torch.ones((n, D), dtype=torch.bool), 1.0)] * (L + 1)


def _rel(a, b):
    return float((a.double().cpu() - b).norm() / b.norm())


def test_tower_forward_and_gradients():
    """fp32 activations around bf16 GEMMs: each GEMM rounds an operand to bf16
    (relative error at most 2^-8, 0.17% in norm), four in the forward pass of
    two layers and eight more operands in the backward pass, independent, with
    amplifications of a few through the norms and the attention: forward
    within 2e-2, gradients within 4e-2, in norm."""
    banner("history tower, training")
    params = _parameters(1)
    tok, off = _histories(2, [70, 0, 1, 130, 64])
    n, p = len(tok), 0.2
    tw = _tower(params, train=True, p=p)
    tw.seed(41)
    rng = tw.rng.cpu()
    keep = []
    for i in range(L + 1):
        m, f = R.keep_mask(n * D, p, int(rng[i, 0]), int(rng[i, 1]))
        keep.append((torch.from_numpy(m).view(n, D), f))
    out = torch.full((5, D), float("nan"), device=DEV)
    tw.forward(tok.to(DEV), off.to(DEV), 130, out, D)
    dbl = lambda t: t.double().requires_grad_(True)  # noqa: E731
    table, layers, w_out = params
    P = (dbl(table), [(dbl(w), dbl(a), dbl(b), lam) for w, a, b, lam in layers], dbl(w_out))
    ref = _model(P, tok, off, keep)
    assert _rel(out, ref.detach()) < 2e-2
    assert not out[1].any()
    g = torch.Generator().manual_seed(3)
    dout = torch.randn(5, D, generator=g)
    (ref * dout.double()).sum().backward()
    before = tw.rng.clone()
    got = tw.backward(dout.to(DEV), D)
    assert (tw.rng[:, 1] - before[:, 1] == (n * D + 7) // 8).all()
    assert _rel(got["table"], P[0].grad) < 4e-2
    assert _rel(got["w_out"], P[2].grad) < 4e-2
    for i in range(L):
        for name, var in zip(("w", "qkv", "out"), P[1][i]):
            assert _rel(got["layers"][i][name], var.grad) < 4e-2, (i, name)


def test_tower_serving_forward_then_steps():
    """bf16 activations: a rounding (0.17% in norm) at every buffer, about six
    a layer, amplified by a few: 3e-2 in norm against fp64.  A history taken
    in whole and then event by event through the state pools gives the vectors
    of the longer history; slots pick the users' pool entries."""
    banner("history tower, serving")
    import deep_learning_recommendation_amd as DL

    params = _parameters(5)
    lens = [100, 3, 64]
    tok, off = _histories(6, lens)
    tok[off[1:] - 1] = torch.tensor([5, 6, 7])  # the newest events name items
    tw = _tower(params)
    dbl = (params[0].double(), [tuple(t.double() for t in p) for p in params[1]], params[2].double())
    ref = _model(dbl, tok, off, _everything(len(tok)))
    out = torch.full((3, D), float("nan"), device=DEV)
    tw.forward(tok.to(DEV), off.to(DEV), 100, out, D)
    assert _rel(out, ref) < 3e-2
    # all but the last event in whole, the last one as a step
    keep = torch.ones(len(tok), dtype=torch.bool)
    keep[off[1:] - 1] = False
    off2 = off - torch.arange(4)
    slots = torch.tensor([4, 0, 2])
    tw.forward(tok[keep].to(DEV), off2.to(DEV), 99, torch.empty((3, D), device=DEV), D)
    pools = []
    for S in tw.states:
        pool = torch.full((6, H, DK, DV), float("nan"), device=DEV)
        pool[slots.to(DEV)] = S
        pools.append(pool)
    first = [p.clone() for p in pools]
    stepped = torch.empty((3, D), device=DEV)
    tw.step(tok[off[1:] - 1].to(DEV), pools, slots.to(DEV), stepped, D)
    assert _rel(stepped, ref) < 3e-2
    assert torch.isnan(pools[0][[1, 3, 5]]).all()
    # as int8 table rows: half a step of each row's scale beside the bf16 vector's own rounding
    rows = (torch.empty((3, D), dtype=torch.int8, device=DEV), torch.empty((3, 2), device=DEV))
    tw.step(tok[off[1:] - 1].to(DEV), first, slots.to(DEV), rows=rows)
    looked = torch.empty((3, D), device=DEV)
    DL.dlrm_embbag_fwd_lp(DL.device_pointer_array([rows[0]]), DL.DLRM_I8, DL.device_pointer_array([rows[1]]), 1, D,
                          torch.arange(3, device=DEV), torch.arange(4, device=DEV), 3, looked, D, nnz=3)
    step = rows[1][:, :1]
    assert ((looked - stepped).abs() <= 0.51 * step + 2 * R.U16 * stepped.abs()).all()


def test_tower_without_events():
    banner("history tower, empty histories")
    tw = _tower(_parameters(4))
    out = torch.full((3, D), 5.0, device=DEV)
    tw.forward(torch.empty(0, dtype=torch.int64, device=DEV), torch.zeros(4, dtype=torch.int64, device=DEV), 0, out, D)
    assert not out.any() and all(s.shape == (3, H, DK, DV) and not s.any() for s in tw.states)


def test_tower_refusals():
    banner("history tower refusals")
    params = _parameters(7)
    with pytest.raises(ValueError):
        _tower(params, p=0.1)
    with pytest.raises(ValueError):
        _tower(params).backward(torch.zeros((1, D), device=DEV), D)
    with pytest.raises(ValueError):
        _tower(params, train=True).step(torch.zeros(1, dtype=torch.int64, device=DEV), [], None)


def test_tower_under_a_captured_graph():
    """Serving steps replayed from a graph, with eager work between the
    replays, give what eager steps give."""
    banner("history tower graph")
    params = _parameters(8)
    tw = _tower(params)
    g = np.random.default_rng(9)
    B = 33
    toks = [torch.from_numpy(g.integers(0, V, B)).to(DEV) for _ in range(4)]
    pools = lambda: [torch.zeros((B, H, DK, DV), device=DEV) for _ in range(L)]  # noqa: E731
    eager, want = pools(), []
    for t in toks:
        o = torch.empty((B, D), device=DEV)
        tw.step(t, eager, None, o, D)
        want.append(o.clone())
    tok, live, out = toks[0].clone(), pools(), torch.empty((B, D), device=DEV)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):  # one run outside the capture
        tw.step(tok, pools(), None, out, D)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tw.step(tok, live, None, out, D)
    for t, w in zip(toks, want):
        tok.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)
        tw.step(t, pools(), None, torch.empty((B, D), device=DEV), D)
    for a, b in zip(live, eager):
        assert torch.equal(a, b)


@pytest.mark.parametrize("train", [False, True])
def test_tower_on_another_stream(train):
    """The same bits on a stream given to the calls while the current one is
    still busy with other work."""
    banner(f"history tower stream {train}")
    params = _parameters(10)
    tok, off = _histories(11, [70, 0, 9, 200])
    tok, off = tok.to(DEV), off.to(DEV)
    dout = torch.randn(4, D, generator=torch.Generator().manual_seed(1)).to(DEV)
    busy = torch.zeros(1 << 26, device=DEV)

    def run(stream):
        tw = _tower(params, train=train)
        out = torch.empty((4, D), device=DEV)
        torch.cuda.synchronize()
        for _ in range(60):
            busy.add_(1.0)
        tw.forward(tok, off, 200, out, D, stream=stream)
        if train:
            return out, tw.backward(dout, D, stream=stream), tw
        pools, stepped = tw.states, torch.empty((4, D), device=DEV)
        tw.step(tok[:4], pools, None, stepped, D, stream=stream)
        return out, {"table": stepped, "w_out": pools[0]}, tw

    want, got = run(None), run(torch.cuda.Stream())
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0])
    for name in ("table", "w_out"):
        assert torch.equal(got[1][name], want[1][name]), name
