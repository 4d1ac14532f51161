"""The behaviour-history operators against their 64-bit references.

Tolerances are elementwise bounds of the arithmetic, from the unit roundoffs
u32 = 2^-24 and u16 = 2^-8 (bf16) and the magnitudes that are summed; they are
stated at each test."""
import numpy as np
import pytest
import torch

import history_ref as R
from dlrm_cases import DEV, banner
from history_ref import U16, U32

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32


def _D():
    import deep_learning_recommendation_amd as D

    return D


def _rows(g, n, d, dtype, ld=None, lead=0, scale=1.0):
    """Rows of a wider, NaN-filled buffer; `lead` elements before the first."""
    ld = ld or d
    buf = torch.full((lead + n * ld + 8,), float("nan"), dtype=dtype)
    v = buf[lead:lead + n * ld].view(n, ld)[:, :d]
    v.copy_((torch.randn(n, d, generator=g) * scale).to(dtype))
    dev = buf.to(DEV)
    return dev[lead:lead + n * ld].view(n, ld)[:, :d]


def _out(n, d, dtype, ld=None):
    ld = ld or d
    fill = 77 if dtype == torch.int8 else float("nan")
    return torch.full((n, ld), fill, dtype=dtype, device=DEV)[:, :d]


def _ws(nbytes):
    return torch.full((max(nbytes, 256),), 0xFF, dtype=torch.uint8, device=DEV)


def _close(got, ref, tol, what=""):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), what
    bad = (got - ref).abs() > tol
    assert not bad.any(), (what, int(bad.sum()), float((got - ref).abs().max()), float((got - ref)[bad].abs().max()))


# ----------------------------------------------------------------- token embedding

@pytest.mark.parametrize("tin,tout", [(FP, FP), (BF, BF), (BF, FP), (FP, BF)])
@pytest.mark.parametrize("n,rows,d,ld", [(1, 1, 4, 4), (7, 5, 16, 16), (1003, 300, 100, 104), (513, 40, 128, 136),
                                         (65, 9, 1024, 1024), (40, 17, 132, 132)])
def test_token_embed_fwd(tin, tout, n, rows, d, ld):
    """fp32 output: the exact product rounded once.  bf16: the fp32 product
    rounded again.  Both bit for bit; padding tokens give +0."""
    banner(f"token_embed_fwd {tin} {tout} {n} {rows} {d} {ld}")
    g = torch.Generator().manual_seed(n + d)
    T = _rows(g, rows, d, tin)
    tok = torch.randint(-1, rows + 1, (n,), generator=g)
    out = _out(n, d, tout, ld)
    _D().dlrm_token_embed_fwd(T, rows, d, tok.to(DEV), n, 11.3, out, ld)
    ok = ((tok >= 0) & (tok < rows))[:, None]
    ref = torch.where(ok, T.cpu().float()[tok.clamp(0, rows - 1)] * torch.tensor(11.3), torch.zeros(())).to(tout)
    assert torch.equal(out.cpu().view(torch.int32 if tout == FP else torch.int16),
                       ref.view(torch.int32 if tout == FP else torch.int16))


def _bwd(tok, dout, rows, d, scale, dT, add):
    D = _D()
    n = tok.numel()
    ws = _ws(D.dlrm_token_embed_bwd_workspace_size(n, rows, d))
    D.dlrm_token_embed_bwd(tok.to(DEV), n, dout, dout.stride(0), rows, d, scale, dT, add, ws)
    return dT


def _token_list(kind, n, rows, g):
    if kind == "one row":
        return torch.full((n,), rows - 1)
    if kind == "all padding":
        return torch.full((n,), -1)
    if kind == "runs":  # run lengths around the chunk's 64 positions, in a random order
        t = torch.repeat_interleave(torch.arange(rows), torch.tensor([63, 64, 65, 127, 128, 129, 1, 191, 0, 2] * 20)[:rows])
        return t[torch.randperm(t.numel(), generator=g)][:n]
    if kind == "head":
        t = torch.randint(0, rows, (n,), generator=g)
        return torch.where(torch.rand(n, generator=g) < 0.4, torch.full_like(t, rows // 2), t)
    return torch.randint(-1, rows + 1, (n,), generator=g)


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("kind,n,rows,d,ld", [("random", 1, 1, 4, 4), ("random", 64, 3, 16, 16),
                                              ("random", 1003, 300, 100, 104), ("random", 5000, 70000, 128, 128),
                                              ("one row", 20000, 5, 64, 64), ("one row", 64, 2, 8, 8),
                                              ("all padding", 200, 7, 32, 32), ("runs", 1 << 20, 190, 136, 136),
                                              ("head", 30011, 999, 128, 144), ("head", 9001, 30, 1024, 1024),
                                              ("random", 4097, 1 << 20, 16, 16)])
@pytest.mark.parametrize("add", [False, True])
def test_token_embed_bwd(dtype, kind, n, rows, d, ld, add):
    """|err| <= (terms + 3) u32 * sum |terms| (at most `terms` additions on any
    path, the scale and the addition to what was there)."""
    banner(f"token_embed_bwd {dtype} {kind} {n} {rows} {d} {add}")
    g = torch.Generator().manual_seed(n + d)
    tok = _token_list(kind, n, rows, g)
    dout = _rows(g, tok.numel(), d, dtype, ld)
    first = torch.randn(rows, d, generator=g)
    dT = first.to(DEV) if add else torch.full((rows, d), float("nan"), device=DEV)
    _bwd(tok, dout, rows, d, 0.37, dT, add)
    ref, mag, cnt = R.embed_grad(tok, dout.cpu(), rows, float(np.float32(0.37)))
    if add:
        ref, mag = ref + first.double(), mag + first.double().abs()
        assert torch.equal(dT.cpu()[cnt == 0], first[cnt == 0])
    else:
        assert not dT.cpu()[cnt == 0].any()
    _close(dT, ref, (cnt[:, None] + 3) * U32 * mag)


def test_token_embed_bwd_exact_on_integers_and_repeatable():
    banner("token_embed_bwd integers")
    g = torch.Generator().manual_seed(5)
    n, rows, d = 40000, 211, 64
    tok = _token_list("head", n, rows, g)
    dout = torch.randint(-8, 9, (n, d), generator=g).float().to(DEV)
    a = _bwd(tok, dout, rows, d, 2.0, torch.empty((rows, d), device=DEV), False)
    b = _bwd(tok, dout, rows, d, 2.0, torch.empty((rows, d), device=DEV), False)
    assert torch.equal(a, b)
    assert torch.equal(a.cpu().double(), R.embed_grad(tok, dout.cpu(), rows, 2.0)[0])


@pytest.mark.parametrize("n", [63, 1024, 1025, 4096, 4097, 16384, 16385])
@pytest.mark.parametrize("rows", [1, 255, 256, 70001, 1 << 20])
def test_token_embed_bwd_sizes_of_the_sort(n, rows):
    """Every count of key bits and positions a thread at which the sort
    changes; sums of integers are exact."""
    banner(f"token_embed_bwd sort {n} {rows}")
    g = torch.Generator().manual_seed(n + rows)
    tok = torch.randint(0, rows + 2, (n,), generator=g) - 1  # the ends are out of range
    dout = torch.randint(-8, 9, (n, 8), generator=g).float().to(DEV)
    dT = _bwd(tok, dout, rows, 8, 2.0, torch.full((rows, 8), float("nan"), device=DEV), False)
    assert torch.equal(dT.cpu().double(), R.embed_grad(tok, dout.cpu(), rows, 2.0)[0])


def test_token_embed_empty():
    banner("token_embed empty")
    D = _D()
    dT = torch.full((6, 8), 3.0, device=DEV)
    none = torch.empty((0,), dtype=torch.int64, device=DEV)
    D.dlrm_token_embed_fwd(torch.ones((6, 8), device=DEV), 6, 8, none, 0, 1.0, torch.empty((0, 8), device=DEV), 8)
    ws = _ws(D.dlrm_token_embed_bwd_workspace_size(0, 6, 8))
    D.dlrm_token_embed_bwd(none, 0, torch.empty((0, 8), device=DEV), 8, 6, 8, 1.0, dT, True, ws)
    assert (dT == 3).all()
    D.dlrm_token_embed_bwd(none, 0, torch.empty((0, 8), device=DEV), 8, 6, 8, 1.0, dT, False, ws)
    assert not dT.any()


# ----------------------------------------------------------------- dropout

def _state(seed, offset):
    as_i64 = lambda v: v - (1 << 64) if v >= 1 << 63 else v  # noqa: E731
    return torch.tensor([as_i64(seed), as_i64(offset)], dtype=torch.int64, device=DEV)


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("n,d,ld,lead", [(1, 1, 1, 0), (3, 7, 7, 0), (33, 479, 512, 0), (33, 479, 479, 0), (64, 128, 128, 0),
                                         (17, 128, 136, 0), (17, 128, 131, 1), (5, 1000, 1000, 0), (9, 4, 4, 0),
                                         (300, 3, 5, 2), (257, 24, 24, 0)])
@pytest.mark.parametrize("p,seed,offset", [(0.3, 0x123456789ABCDEF, 5), (0.9, (1 << 64) - 3, (1 << 64) - 2),
                                           (0.0, 1, 2), (1.0, 1, 2)])
def test_dropout(dtype, n, d, ld, lead, p, seed, offset):
    """The mask bit for bit; kept values are one fp32 product, rounded to the
    type; dropped NaN and infinities give +0."""
    banner(f"dropout {dtype} {n} {d} {ld} {lead} {p}")
    g = torch.Generator().manual_seed(n * d)
    x = _rows(g, n, d, dtype, ld, lead)
    keep, f = R.keep_mask(n * d, p, seed, offset)
    keep = torch.from_numpy(keep).view(n, d)
    x[~keep.to(DEV)] = torch.tensor([float("nan"), float("inf")], dtype=dtype, device=DEV).repeat(n * d)[:int((~keep).sum())]
    y = _out(n, d, dtype, ld + 3)
    _D().dlrm_dropout(x, ld, y, ld + 3, n, d, p, _state(seed, offset))
    f32 = torch.tensor(np.float32(65536) / np.float32(max(65536 - int(p * 65536 + 0.5), 1)))
    ref = torch.where(keep, x.cpu().float() * f32, torch.zeros(())).to(dtype)
    i = torch.int32 if dtype == FP else torch.int16
    assert torch.equal(y.cpu().contiguous().view(i), ref.contiguous().view(i))
    _D().dlrm_dropout(x, ld, x, ld, n, d, p, _state(seed, offset))  # in place
    assert torch.equal(x.cpu().contiguous().view(i), ref.contiguous().view(i))


def test_dropout_writes_nothing_past_its_rows():
    banner("dropout padding columns")
    x = torch.ones((20, 64), device=DEV)
    y = torch.full((20, 64), 9.0, device=DEV)
    _D().dlrm_dropout(x, 64, y, 64, 20, 61, 0.5, _state(1, 1))
    assert (y[:, 61:] == 9).all() and not (y[:, :61] == 9).any()


# ----------------------------------------------------------------- residual + norm

SHAPES = [(1, 1, 1), (5, 8, 8), (33, 100, 100), (130, 128, 128), (129, 128, 136), (40, 479, 481), (17, 1000, 1000),
          (9, 1024, 1024), (3, 2048, 2056), (3, 5000, 5000), (2, 16384, 16384), (70, 64, 64), (31, 16, 24)]


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("n,d,ld", SHAPES)
@pytest.mark.parametrize("p,with_res,out", [(0.0, True, "same"), (0.25, True, "same"), (0.0, False, "i8"),
                                            (0.25, True, "i8")])
def test_add_rmsnorm_fwd(dtype, n, d, ld, p, with_res, out):
    """h: a product and an addition in fp32 (2 u32 of their magnitudes), and
    the type's rounding.  1/rms: the mean of squares errs by at most
    (d + 4) u32 relative (any order) plus the squares' 4 u32, half of that after
    the root, so y errs by (d/2 + 8) u32 relative plus the error of h carried
    over.  int8: the value is within half a scale step, and the scale within
    the error of the largest |y|."""
    banner(f"addnorm_fwd {dtype} {n} {d} {ld} {p} {with_res} {out}")
    g = torch.Generator().manual_seed(n + d)
    x = _rows(g, n, d, dtype, ld)
    res = _rows(g, n, d, dtype, ld, scale=3.0) if with_res else None
    w = (torch.randn(d, generator=g) * 0.3 + 1).to(DEV)
    keep, f = R.keep_mask(n * d, p, 77, 88)
    keep = torch.from_numpy(keep).view(n, d)
    h, rstd = _out(n, d, dtype, ld), torch.full((n,), float("nan"), device=DEV)
    y = _out(n, d, torch.int8 if out == "i8" else dtype, ld)
    sb = torch.full((n, 2), float("nan"), device=DEV) if out == "i8" else None
    eps = 1e-5
    _D().dlrm_add_rmsnorm_fwd(x, ld, res, ld, w, n, d, eps, p, _state(77, 88), h, ld, y, ld, sb, rstd)
    cpu = lambda t: None if t is None else t.cpu()  # noqa: E731
    rh, ry, rr = R.addnorm(cpu(x), cpu(res), cpu(w), eps, keep, f)
    unit = U16 if dtype == BF else 0.0
    mag = (x.cpu().double() * f).abs() + (0 if res is None else res.cpu().double().abs())
    eh = 2 * U32 * mag
    _close(h, rh, eh + unit * (rh.abs() + eh), "h")
    er = ((d / 2 + 8) * U32 + 2 * U32 * (mag.square().mean(1) / (rh.square().mean(1) + eps)).sqrt())
    _close(rstd, rr, er * rr, "rstd")
    ey = ry.abs() * er[:, None] * 2 + eh * (rr[:, None] * w.cpu().double().abs())
    if out != "i8":
        _close(y, ry, ey + unit * (ry.abs() + ey), "y")
        return
    s = sb[:, 0].cpu().double()
    top = ry.abs().amax(1)
    assert not sb[:, 1].any()
    assert ((s - top / 127).abs() <= (ey.amax(1) + 4 * U32 * top) / 127).all()
    _close(y.double() * sb[:, :1].double(), ry, 0.5 * s[:, None] * (1 + 512 * U32) + ey, "int8")
    assert int(y.abs().max()) <= 127


@pytest.mark.parametrize("dtype", [FP, BF])
def test_add_rmsnorm_int8_special_rows(dtype):
    """A zero row stands for zeros (s = 0), a row with a NaN has s = NaN and
    q = 0, and neither touches its neighbours; rows that the lookup of int8
    table rows decodes."""
    banner(f"addnorm int8 rows {dtype}")
    D = _D()
    for d in (64, 100, 1024):
        x = torch.randn(6, d, device=DEV).to(dtype)
        x[1] = 0
        x[3, 5] = float("nan")
        y, sb = _out(6, d, torch.int8), torch.empty((6, 2), device=DEV)
        w = torch.ones(d, device=DEV)
        D.dlrm_add_rmsnorm_fwd(x, d, None, 0, w, 6, d, 0.0 if d == 64 else 1e-6, 0.0, None, None, 0, y, d, sb, None)
        if d != 64:  # eps = 0 makes the zero row 0 * inf
            assert sb[1, 0] == 0 and not y[1].any()
        assert torch.isnan(sb[3, 0]) and not y[3].any()
        clean, sb2 = _out(6, d, torch.int8), torch.empty((6, 2), device=DEV)
        x[3] = 1
        D.dlrm_add_rmsnorm_fwd(x, d, None, 0, w, 6, d, 1e-6, 0.0, None, None, 0, clean, d, sb2, None)
        assert torch.equal(clean[[0, 2, 4, 5]], y[[0, 2, 4, 5]]) or d == 64
        pooled = torch.empty((6, d), device=DEV)
        tab, sbp = D.device_pointer_array([clean]), D.device_pointer_array([sb2])
        D.dlrm_embbag_fwd_lp(tab, D.DLRM_I8, sbp, 1, d, torch.arange(6, device=DEV), torch.arange(7, device=DEV), 6,
                             pooled, d, nnz=6)
        assert torch.equal(pooled, clean.float() * sb2[:, :1])


@pytest.mark.parametrize("d", [64, 100, 65, 1024])
@pytest.mark.parametrize("top", [2.0 ** 100, 1.0, 2.0 ** -112, 2.0 ** -114, 2.0 ** -121, 2.0 ** -126, 1e-40, 256 * 2.0 ** -149,
                                 190 * 2.0 ** -149, 71 * 2.0 ** -149, 40 * 2.0 ** -149])
def test_add_rmsnorm_int8_scales_down_to_the_smallest(d, top):
    """Rows of +-1 have r = 1, so y = +-w exactly, down to subnormal w: s is
    max |w| / 127 rounded once, q is w / s to the nearest step (the reciprocal
    and the product round, 2 u32 each of at most 127 steps), at most 127."""
    banner(f"addnorm int8 scales {d} {top}")
    g = torch.Generator().manual_seed(d)
    w = (torch.rand(d, generator=g, dtype=torch.float64) * top).float()
    w[3] = top
    x = torch.where(torch.rand(5, d, generator=g) < 0.5, -1.0, 1.0)
    y, sb = _out(5, d, torch.int8), torch.empty((5, 2), device=DEV)
    _D().dlrm_add_rmsnorm_fwd(x.to(DEV), d, None, 0, w.to(DEV), 5, d, 0.0, 0.0, None, None, 0, y, d, sb, None)
    s = np.float32(w.max().numpy()) / np.float32(127)
    assert (sb[:, 0].cpu().numpy() == s).all() and not sb[:, 1].any()
    if s == 0:
        assert not y.any()
        return
    want = (x.double() * w.double() / float(s)).clamp(-127, 127)
    assert bool(((y.cpu().double() - want).abs() <= 0.5 + 127 * 4 * U32).all())


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("n,d,ld", SHAPES + [(3000, 24, 24), (2500, 128, 128)])
@pytest.mark.parametrize("p,with_dh", [(0.0, True), (0.25, False), (0.25, True)])
def test_add_rmsnorm_bwd(dtype, n, d, ld, p, with_dh):
    """t: the mean of g h errs by (d + 6) u32 of the mean of |g h|; the three
    terms by a few u32 of their magnitudes.  dw: n + 6 roundings on any path."""
    banner(f"addnorm_bwd {dtype} {n} {d} {ld} {p} {with_dh}")
    D = _D()
    g = torch.Generator().manual_seed(n + d)
    dy, h = _rows(g, n, d, dtype, ld), _rows(g, n, d, dtype, ld, scale=2.0)
    dh = _rows(g, n, d, dtype, ld) if with_dh else None
    w = (torch.randn(d, generator=g) * 0.3 + 1).to(DEV)
    r = (torch.rand(n, generator=g) + 0.2).to(DEV)
    keep, f = R.keep_mask(n * d, p, 7, 1 << 40)
    keep = torch.from_numpy(keep).view(n, d)
    dx, dres, dw = _out(n, d, dtype, ld), _out(n, d, dtype, ld), torch.full((d,), float("nan"), device=DEV)
    ws = _ws(D.dlrm_add_rmsnorm_bwd_workspace_size(n, d))
    rng = _state(7, 1 << 40)
    D.dlrm_add_rmsnorm_bwd(dy, ld, dh, ld, h, ld, w, r, n, d, p, rng, dx, ld, dres, ld, dw, ws)
    cpu = lambda t: None if t is None else t.cpu()  # noqa: E731
    rx, rt, rw = R.addnorm_grad(cpu(dy), cpu(dh), cpu(h), cpu(w), cpu(r), keep, f)
    a = lambda t: t.cpu().double().abs()  # noqa: E731
    R3, G = a(r)[:, None] ** 3, a(dy) * a(w)
    mean = (G * a(h)).mean(1, keepdim=True)
    e = U32 * (6 * a(r)[:, None] * G + (d + 12) * a(h) * R3 * mean + (2 * a(dh) if with_dh else 0))
    unit = U16 if dtype == BF else 0.0
    _close(dres, rt, e + unit * (rt.abs() + e), "dres")
    ex = f * e + U32 * rx.abs()
    _close(dx, rx, ex + unit * (rx.abs() + ex), "dx")
    _close(dw, rw, (n + 6) * U32 * (a(dy) * a(h) * a(r)[:, None]).sum(0), "dw")
    # only one of the two outputs, and dres in dh's place
    only, dw2 = _out(n, d, dtype, ld), torch.empty_like(dw)
    D.dlrm_add_rmsnorm_bwd(dy, ld, dh, ld, h, ld, w, r, n, d, p, rng, only, ld, None, 0, dw2, ws)
    assert torch.equal(only, dx) and torch.equal(dw2, dw)
    if with_dh:
        D.dlrm_add_rmsnorm_bwd(dy, ld, dh, ld, h, ld, w, r, n, d, p, rng, None, 0, dh, ld, dw2, ws)
        assert torch.equal(dh, dres)


def test_add_rmsnorm_bwd_no_rows():
    banner("addnorm_bwd no rows")
    dw = torch.full((32,), 5.0, device=DEV)
    e = torch.empty((0, 32), device=DEV)
    _D().dlrm_add_rmsnorm_bwd(e, 32, None, 0, e, 32, dw, dw, 0, 32, 0.0, None, e, 32, None, 0, dw, _ws(256))
    assert not dw.any()


# ----------------------------------------------------------------- linear attention

def _decays(H, g):
    lam = 1 - torch.exp2(-1 - 7 * torch.rand(H, generator=g))
    lam[0] = 1.0
    if H > 1:
        lam[1] = 0.0
    return lam


class Attn:
    """Inputs on one packed buffer: NaN rows before, between strides and after."""

    def __init__(self, seed, lens, H, dk, dv, dtype, lead=3, packed=True, states=True):
        g = torch.Generator().manual_seed(seed)
        self.H, self.dk, self.dv, self.dtype = H, dk, dv, dtype
        self.off = torch.cat([torch.tensor([lead]), lead + torch.cumsum(torch.tensor(lens), 0)]).to(torch.int64)
        n = int(self.off[-1]) + 5
        self.n, self.B, self.max_len = n, len(lens), max(lens + [0])
        inside = torch.zeros(n, dtype=torch.bool)
        inside[lead:int(self.off[-1])] = True
        self.inside = inside

        def rows(width):
            t = torch.randn(n, H, width, generator=g)
            t[~inside] = float("nan")
            return t.to(dtype)

        q, k, v, do = rows(dk), rows(dk), rows(dv), rows(dv)
        if packed:  # q, k, v side by side, 8 more columns of NaN
            buf = torch.full((n, H * (2 * dk + dv) + 8), float("nan"), dtype=dtype)
            for t, a in ((q, 0), (k, H * dk), (v, 2 * H * dk)):
                buf[:, a:a + t[0].numel()] = t.reshape(n, -1)
            buf = buf.to(DEV)
            self.q = buf[:, :H * dk].unflatten(1, (H, dk))
            self.k = buf[:, H * dk:2 * H * dk].unflatten(1, (H, dk))
            self.v = buf[:, 2 * H * dk:2 * H * dk + H * dv].unflatten(1, (H, dv))
        else:  # heads outermost
            put = lambda t: t.transpose(0, 1).contiguous().to(DEV).transpose(0, 1)  # noqa: E731
            self.q, self.k, self.v = put(q), put(k), put(v)
        self.do = do.to(DEV)
        self.decay = _decays(H, g)
        st = lambda: torch.randn(self.B, H, dk, dv, generator=g) if states else None  # noqa: E731
        self.S0, self.dS = st(), st()
        self.scale = dk ** -0.5

    def dev(self, t):
        return None if t is None else t.to(DEV)

    def out(self, width):
        return torch.full((self.n, self.H, width), float("nan"), dtype=self.dtype, device=DEV)

    def clean(self, t):
        return torch.where(self.inside[:, None, None], t.cpu().double(), 0.0)

    def fwd(self, stream=None, in_place=False):
        D = _D()
        o = self.out(self.dv)
        S0 = self.dev(self.S0)
        S = S0 if in_place else torch.full((self.B, self.H, self.dk, self.dv), float("nan"), device=DEV)
        shape = (self.B, self.H, self.max_len, self.dk, self.dv)
        ws = _ws(D.dlrm_linattn_workspace_size(*shape))
        torch.cuda.synchronize()
        D.dlrm_linattn_fwd(self.q, self.k, self.v, self.off.to(DEV), *shape, self.decay.to(DEV), self.scale, S0, o, S,
                           ws, stream=stream)
        torch.cuda.synchronize()
        return o, S

    def bwd(self, stream=None):
        D = _D()
        dq, dk, dv = self.out(self.dk), self.out(self.dk), self.out(self.dv)
        dS0 = torch.full((self.B, self.H, self.dk, self.dv), float("nan"), device=DEV)
        shape = (self.B, self.H, self.max_len, self.dk, self.dv)
        ws = _ws(D.dlrm_linattn_bwd_workspace_size(*shape))
        torch.cuda.synchronize()
        D.dlrm_linattn_bwd(self.q, self.k, self.v, self.do, self.off.to(DEV), *shape, self.decay.to(DEV), self.scale,
                           self.dev(self.S0), self.dev(self.dS), dq, dk, dv, dS0, ws, stream=stream)
        torch.cuda.synchronize()
        return dq, dk, dv, dS0

    def tolerance(self, ref, mag, state=False):
        """fp32: at most max_len + 64 additions on any path, and decays within
        2^-18 (a power decay^n as 2^(n log2 decay) errs by at most
        |n log2 decay| u32 + 2 u32 relative, which matters while decay^n is not
        negligible: |n log2 decay| < 32).  bf16 operands: one rounding of
        each masked product or state (u16 of the magnitudes), and the
        output's own."""
        e = (2.0 ** -18 + (self.max_len + 64) * U32) * mag
        if self.dtype == BF and not state:
            e = e + U16 * mag
            e = e + U16 * (ref.abs() + e)
        return e + 1e-30

    def check_fwd(self, o, S):
        c = self.clean
        q, k, v = c(self.q), c(self.k), c(self.v)
        ro, rS = R.linattn(q, k, v, self.off, self.decay, self.scale, self.S0)
        ab = lambda t: None if t is None else t.abs()  # noqa: E731
        mo, mS = R.linattn(q.abs(), k.abs(), v.abs(), self.off, self.decay, self.scale, ab(self.S0))
        i = self.inside
        assert torch.isnan(o.cpu()[~i]).all()
        _close(o.cpu()[i], ro[i], self.tolerance(ro, mo)[i], "o")
        _close(S, rS, self.tolerance(rS, mS, True), "state")

    def check_bwd(self, got):
        c = self.clean
        args = c(self.q), c(self.k), c(self.v), c(self.do)
        ref = R.linattn_grad(*args, self.off, self.decay, self.scale, self.S0, self.dS)
        ab = lambda t: None if t is None else t.abs()  # noqa: E731
        mag = R.linattn_grad(*(t.abs() for t in args), self.off, self.decay, self.scale, ab(self.S0), ab(self.dS))
        i = self.inside
        for name, a, r, m in zip(("dq", "dk", "dv"), got, ref, mag):
            assert torch.isnan(a.cpu()[~i]).all(), name
            _close(a.cpu()[i], r[i], self.tolerance(r, m)[i], name)
        _close(got[3], ref[3], self.tolerance(ref[3], mag[3], True), "dstate0")


LENS = [[1], [0], [64], [65, 0, 63, 1, 128, 2], [129, 200], [0, 0, 31, 257]]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("H,dk,dv", [(1, 8, 8), (2, 64, 64), (1, 128, 128), (3, 32, 16), (2, 72, 40), (1, 40, 128),
                                     (2, 128, 64)])
@pytest.mark.parametrize("lens", LENS)
def test_linattn_fwd(dtype, H, dk, dv, lens):
    banner(f"linattn_fwd {dtype} {H} {dk} {dv} {lens}")
    a = Attn(sum(lens) + dk, lens, H, dk, dv, dtype, states=len(lens) != 2)
    a.check_fwd(*a.fwd())


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("H,dk,dv", [(1, 8, 8), (2, 64, 64), (1, 128, 128), (3, 32, 16), (2, 72, 40), (2, 40, 128),
                                     (2, 128, 64)])
@pytest.mark.parametrize("lens", LENS)
def test_linattn_bwd(dtype, H, dk, dv, lens):
    banner(f"linattn_bwd {dtype} {H} {dk} {dv} {lens}")
    a = Attn(sum(lens) + dv, lens, H, dk, dv, dtype, states=len(lens) != 2)
    a.check_bwd(a.bwd())


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("lens,H,d", [([3000], 2, 64), ([1, 2049], 3, 32), ([1500, 0, 700], 2, 128)])
def test_linattn_long(dtype, lens, H, d):
    """Few long histories: the length is cut into segments."""
    banner(f"linattn long {dtype} {lens} {H} {d}")
    a = Attn(7, lens, H, d, d, dtype)
    a.check_fwd(*a.fwd())
    a.check_fwd(*a.fwd(in_place=True))
    a.check_bwd(a.bwd())


@pytest.mark.parametrize("dtype", [BF, FP])
def test_linattn_bwd_many_ragged_histories(dtype):
    """Enough short histories for the gradient to start the longest first."""
    banner(f"linattn_bwd many histories {dtype}")
    g = np.random.default_rng(17)
    lens = [int(x) for x in g.integers(0, 40, 210)]
    lens[3], lens[100], lens[209] = 131, 0, 90
    a = Attn(18, lens, 2, 16, 16, dtype)
    a.check_bwd(a.bwd())
    a.check_fwd(*a.fwd())


@pytest.mark.parametrize("dtype", [BF, FP])
def test_linattn_max_len_may_be_loose(dtype):
    """max_len is an upper bound: segments that no history reaches stay empty."""
    banner(f"linattn loose max_len {dtype}")
    a = Attn(19, [300, 5, 0, 64], 1, 64, 32, dtype)
    a.max_len = 5000
    a.check_fwd(*a.fwd())
    a.check_bwd(a.bwd())


@pytest.mark.parametrize("dtype", [BF, FP])
def test_linattn_head_major_and_streams(dtype):
    """[heads][rows][width] storage, a stream other than the default one, and
    the same bits every time."""
    banner(f"linattn head-major {dtype}")
    a = Attn(11, [100, 0, 301], 2, 64, 72, dtype, packed=False)
    st = torch.cuda.Stream()
    one, two = a.fwd(), a.fwd(stream=st)
    a.check_fwd(*two)
    for x, y in zip(one + a.bwd(), two + a.bwd(stream=st)):
        assert torch.equal(torch.nan_to_num(x), torch.nan_to_num(y))


def test_linattn_one_bad_history_stays_alone():
    """NaN and infinity in one history reach no other."""
    banner("linattn bad history")
    a = Attn(12, [70, 64, 33], 2, 64, 64, BF)
    b, e = int(a.off[1]), int(a.off[2])
    o, S = a.fwd()
    a.v[b + 3], a.k[b + 9] = float("nan"), float("inf")
    o2, S2 = a.fwd()
    keep = [i for i in range(a.n) if not b <= i < e]
    assert torch.equal(torch.nan_to_num(o[keep]), torch.nan_to_num(o2[keep])) and torch.equal(S[[0, 2]], S2[[0, 2]])
    assert torch.isnan(o2[e - 1]).any()
    assert torch.equal(o[b:b + 3], o2[b:b + 3])  # causal: the rows before the bad one


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("B,H,dk,dv,pool", [(1, 1, 8, 8, 1), (5, 3, 64, 64, 9), (33, 2, 128, 128, 40), (7, 1, 72, 40, 7),
                                            (300, 2, 32, 16, 301), (2, 4, 16, 128, 2)])
@pytest.mark.parametrize("with_slots", [True, False])
def test_linattn_step(dtype, B, H, dk, dv, pool, with_slots):
    """One step of the recurrence in fp32: the state within 3 u32 of its two
    terms' magnitudes, o within (dk + 6) u32 of the sum's and the type's
    rounding; a negative slot gives +0 and leaves every state alone."""
    banner(f"linattn_step {dtype} {B} {H} {dk} {dv} {pool} {with_slots}")
    g = torch.Generator().manual_seed(B + dk)
    q, k, v = (torch.randn(B, H, w, generator=g).to(dtype) for w in (dk, dk, dv))
    S = torch.randn(pool, H, dk, dv, generator=g)
    slots = torch.randperm(pool, generator=g)[:B] if with_slots else None
    if with_slots and B > 4:
        slots[2] = -1
    lam = _decays(H, g)
    Sd = S.to(DEV)
    o = torch.full((B, H, dv), float("nan"), dtype=dtype, device=DEV)
    _D().dlrm_linattn_step(q.to(DEV), k.to(DEV), v.to(DEV), B, H, dk, dv, lam.to(DEV), 0.3, Sd,
                           None if slots is None else slots.to(DEV), o)
    at = torch.arange(B) if slots is None else slots
    on = at >= 0
    want, tol = S.double().clone(), torch.zeros(S.shape, dtype=torch.float64)
    kv = k.double()[..., None] * v.double()[:, :, None, :]
    l4 = lam.double().view(1, -1, 1, 1)
    want[at[on]] = (S[at[on]].double() * l4 + kv[on])
    tol[at[on]] = 3 * U32 * (S[at[on]].double().abs() * l4 + kv[on].abs())
    _close(Sd, want, tol, "state")
    ro = torch.where(on[:, None, None], (q.double()[..., None] * want[at]).sum(2) * 0.3, 0.0)
    mo = (q.double().abs()[..., None] * (S[at].double().abs() * l4 + kv.abs())).sum(2) * 0.3
    e = (dk + 6) * U32 * mo
    _close(o, ro, e + (U16 * (ro.abs() + e) if dtype == BF else 0), "o")


def test_linattn_steps_follow_the_histories():
    """A history fed event by event ends in the state of the whole-history call."""
    banner("linattn steps = histories")
    a = Attn(13, [40, 40], 2, 64, 64, FP)
    o, S = a.fwd()
    pool = a.S0.to(DEV)
    for t in range(40):
        rows = torch.tensor([int(a.off[0]) + t, int(a.off[1]) + t], device=DEV)
        ot = torch.empty((2, 2, 64), device=DEV)
        _D().dlrm_linattn_step(a.q[rows], a.k[rows], a.v[rows], 2, 2, 64, 64, a.decay.to(DEV), a.scale, pool, None, ot)
    c = a.clean
    mag = R.linattn(c(a.q).abs(), c(a.k).abs(), c(a.v).abs(), a.off, a.decay, a.scale, a.S0.abs())
    tol = 2 * a.tolerance(None, mag[1], True)
    _close(pool, S.cpu().double(), tol, "state")
    last = [int(a.off[1]) - 1, int(a.off[2]) - 1]
    _close(ot, o[last].cpu().double(), 2 * a.tolerance(None, mag[0][last], True), "o")


def test_linattn_step_pool_beyond_4_gib():
    """State offsets past 2^32 bytes."""
    banner("linattn_step large pool")
    H, d = 2, 128
    pool = (1 << 32) // (H * d * d * 4) + 3
    S = torch.zeros((pool, H, d, d), device=DEV)
    S[pool - 1] = 1.0
    x = torch.ones((1, H, d), device=DEV)
    o = torch.empty((1, H, d), device=DEV)
    _D().dlrm_linattn_step(x, x, x, 1, H, d, d, torch.full((H,), 0.5, device=DEV), 1.0, S,
                           torch.tensor([pool - 1], device=DEV), o)
    assert (S[pool - 1] == 1.5).all() and (o == 1.5 * d).all() and not S[0].any() and not S[pool - 2].any()


@pytest.mark.parametrize("dtype", [BF, FP])
def test_linattn_history_longer_than_its_bound(dtype):
    """max_len cuts the work, it does not bound it: a longer history is whole."""
    banner(f"linattn short max_len {dtype}")
    a = Attn(20, [1100, 40], 1, 64, 32, dtype)
    a.max_len = 600
    got, back = a.fwd(), a.bwd()
    a.max_len = 1100  # what the bounds of the sums go by
    a.check_fwd(*got)
    a.check_bwd(back)


# Launches of more blocks than one grid dimension takes (2^20 of them).

def test_token_embed_fwd_many_rows():
    banner("token_embed_fwd 2^26 rows")
    n, rows, d = (1 << 26) + 5, 1000, 68
    T = torch.randn(rows, d, generator=torch.Generator().manual_seed(3)).to(BF).to(DEV)
    tok = torch.randint(0, rows, (n,), device=DEV)
    out = torch.empty((n, d), dtype=BF, device=DEV)
    _D().dlrm_token_embed_fwd(T, rows, d, tok, n, 1.0, out, d)
    for i in range(0, n, 1 << 23):
        assert torch.equal(out[i:i + (1 << 23)], T[tok[i:i + (1 << 23)]])


def _two_steps(q, k, v, do, off, S0, dS, lam):
    """Histories of at most two rows, all at once: o, the states, dq, dk, dv and dS0."""
    len_ = off[1:] - off[:-1]
    S, states, o = S0, [], torch.zeros_like(v)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    rows = [(len_ > t, off[:-1] + t) for t in range(2)]
    for on, at in rows:
        i = at[on]
        S = S.clone()
        S[on] = lam * S[on] + k[i, :, None] * v[i, None, :]
        o[i] = (q[i, :, None] * S[on]).sum(1)
        dq[i] = (S[on] * do[i, None, :]).sum(2)
        states.append(S)
    W = dS
    for on, at in rows[::-1]:
        i = at[on]
        U = W[on] + q[i, :, None] * do[i, None, :]
        dk[i] = (U * v[i, None, :]).sum(2)
        dv[i] = (U * k[i, :, None]).sum(1)
        W = W.clone()
        W[on] = lam * U
    return o, S, dq, dk, dv, W


def test_linattn_many_histories():
    """Sums of at most 2 * 8 + 2 terms, whose weights (a power of the decay and
    its products) are within 8 u32: every output is within 32 u32 of its
    terms' magnitudes."""
    banner("linattn 2^20 histories")
    D, B, w = _D(), (1 << 20) + 5, 8
    g = torch.Generator().manual_seed(4)
    off = torch.zeros(B + 1, dtype=torch.int64)
    off[1:] = torch.randint(0, 3, (B,), generator=g).cumsum(0)
    n = int(off[-1])
    q, k, v, do = (torch.randn(n, 1, w, generator=g).to(DEV) for _ in range(4))
    S0, dS = (torch.randn(B, 1, w, w, generator=g).to(DEV) for _ in range(2))
    off, lam = off.to(DEV), torch.tensor([0.75], device=DEV)
    o, dq, dk, dv = (torch.empty_like(x) for x in (q, q, k, v))
    S, dS0 = torch.empty_like(S0), torch.empty_like(S0)
    D.dlrm_linattn_fwd(q, k, v, off, B, 1, 2, w, w, lam, 1.0, S0, o, S, _ws(D.dlrm_linattn_workspace_size(B, 1, 2, w, w)))
    D.dlrm_linattn_bwd(q, k, v, do, off, B, 1, 2, w, w, lam, 1.0, S0, dS, dq, dk, dv, dS0,
                       _ws(D.dlrm_linattn_bwd_workspace_size(B, 1, 2, w, w)))
    args = [x.double().squeeze(1) for x in (q, k, v, do)], [x.double().squeeze(1) for x in (S0, dS)]
    want = _two_steps(*args[0], off, *args[1], 0.75)
    mag = _two_steps(*[x.abs() for x in args[0]], off, *[x.abs() for x in args[1]], 0.75)
    for name, got, ref, m in zip("o S dq dk dv dS0".split(), (o, S, dq, dk, dv, dS0), want, mag):
        err = (got.squeeze(1).double() - ref).abs()
        assert bool((err <= 32 * U32 * m).all()), (name, float((err / m.clamp_min(1e-30)).max()))


@pytest.mark.parametrize("dtype", [FP, BF])
def test_linattn_step_many_users(dtype):
    """Small integers and a decay of 1/2: every sum is exact."""
    banner(f"linattn_step 2^20 users and heads {dtype}")
    B, H, w = (1 << 19) + 3, 2, 8
    g = torch.Generator().manual_seed(6)
    q, k, v = (torch.randint(-1, 2, (B, H, w), generator=g).to(dtype).to(DEV) for _ in range(3))
    S = torch.randint(-2, 3, (B, H, w, w), generator=g).float().to(DEV)
    want = 0.5 * S + k.float()[..., None] * v.float()[:, :, None, :]
    o = torch.empty((B, H, w), dtype=dtype, device=DEV)
    _D().dlrm_linattn_step(q, k, v, B, H, w, w, torch.full((H,), 0.5, device=DEV), 1.0, S, None, o)
    assert torch.equal(S, want)
    assert torch.equal(o, (q.float()[..., None] * want).sum(2).to(dtype))
