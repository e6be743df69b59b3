"""The norms in front of and behind the block and their gradients (moe_prenorm, moe_combine_norm and
their backward passes, moe_forward_norm) against fp64, element by element."""
from __future__ import annotations

import pytest
import torch

import token_permute_grouped_amd as tpg
from moe_synth import MoeConfig, generate
from tests._block import FP32, HALF, bf16, close, combine, dev, nan, rms, routing, tables, workspace
from tests._gpu import DEV, DeviceProblem

pytestmark = pytest.mark.gpu

EPS = 1e-5
# one row chunk per thread up to H = 8192, then 2, 4 and 8; 128 is half a wave, 65536 the widest row
WIDTHS = [(1, 128), (5, 256), (3, 640), (2, 1152), (4, 4096), (1, 7168), (2, 8320), (2, 16512), (1, 65536)]


def _problem(T, H, E=4, k=2, **kw):
    return tpg.make_problem(T, H, 256, E, k, **kw)


def _gen(*seed):
    return torch.Generator().manual_seed(sum(s * 7919 ** i for i, s in enumerate(seed)) % (1 << 31))


@pytest.mark.parametrize("T,H", WIDTHS + [(300, 384)])
@pytest.mark.parametrize("norm", ["weight", "ones", "none"])
def test_prenorm(T, H, norm):
    g = _gen(T, H)
    x = bf16(T, H, g=g) * torch.exp(torch.randn(T, 1, generator=g, dtype=torch.float64) * 2).to(torch.bfloat16)
    x[0, :128] = 0  # a block of zeros: its fp8 scale is 1
    w = bf16(H, g=g) if norm == "weight" else None
    p = _problem(T, H)
    n = None if norm == "none" else tpg.make_norm(dev(w), EPS)
    xn, q, sc = nan(T, H), nan(T, H).to(torch.float8_e4m3fn), nan(T, H // 128, dtype=torch.float32)
    tpg.moe_prenorm(dev(x), n, p, xn, q, sc)
    ref = x.double() if norm == "none" else rms(x.double(), None if w is None else w.double(), EPS)
    close(xn, ref, FP32 * ref.abs(), "xn")
    amax = ref.abs().reshape(T, -1, 128).amax(2)
    want = torch.where(amax == 0, 1.0, amax / 448)
    close(sc, want, FP32 * want, "scale", half=0.0)
    # a code stands for n / s rounded to e4m3: half a step is 2^-4 relative, 2^-10 among the subnormals
    s = sc.cpu().double().repeat_interleave(128, 1)
    close(q.float(), ref / s, (FP32 + 2.0 ** -4) * (ref / s).abs() + 2.0 ** -10, "codes", half=0.0)
    # each output on its own is the same
    xn2, q2, sc2 = nan(T, H), torch.zeros_like(q), torch.zeros_like(sc)
    tpg.moe_prenorm(dev(x), n, p, xn2)
    tpg.moe_prenorm(dev(x), n, p, None, q2, sc2)
    assert torch.equal(xn, xn2) and torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(sc, sc2)
    inplace = dev(x).clone()
    tpg.moe_prenorm(inplace, n, p, inplace)
    assert torch.equal(inplace, xn)


def test_prenorm_rows_of_zeros_and_of_tiny_values():
    x = torch.zeros(3, 256, dtype=torch.bfloat16)
    x[1] = 1e-30
    for eps in (1e-6, 1.2e-38):
        xn, q, sc = nan(3, 256), nan(3, 256).to(torch.float8_e4m3fn), nan(3, 2, dtype=torch.float32)
        tpg.moe_prenorm(dev(x), tpg.make_norm(None, eps), _problem(3, 256), xn, q, sc)
        assert (xn[0] == 0).all() and (xn[2] == 0).all() and (sc[0] == 1).all() and (q.float()[0] == 0).all()
        assert torch.isfinite(xn).all() and torch.isfinite(q.float()).all()
        dw, dx = nan(256, dtype=torch.float32), nan(3, 256)
        p = _problem(3, 256)
        ones = torch.ones(3, 256, dtype=torch.bfloat16, device=DEV)
        tpg.moe_prenorm_backward(None, None, ones, None, dev(x), tpg.make_norm(None, eps), p, dx, dw,
                                 workspace(p, tpg.MOE_WS_PRENORM_BACKWARD))
        assert torch.isfinite(dx).all() and torch.isfinite(dw).all()


@pytest.mark.parametrize("T,H,E,k,drop", [(1, 128, 4, 2, 0.0), (1, 7168, 8, 8, 0.0), (37, 640, 16, 3, 0.3),
                                          (700, 256, 8, 2, 0.1), (5, 8320, 12, 9, 0.2), (3, 16512, 4, 1, 0.0),
                                          (2, 65536, 20, 17, 0.2), (3000, 128, 4, 1, 0.5), (6, 384, 4, 2, 1.0)])
@pytest.mark.parametrize("form", ["norm", "ones", "none"])
def test_prenorm_backward(T, H, E, k, drop, form):
    g = _gen(T, H, k)
    offsets, slot_row, _ = routing(T, E, k, g, drop)
    R = int(offsets[-1])
    dxp, dxn, dres, x = (bf16(n, H, g=g) for n in (T * k, T, T, T))
    dxp[R:] = float("nan")  # rows behind the last are never read
    w = bf16(H, g=g) if form == "norm" else None
    p = _problem(T, H, E, k)
    norm = None if form == "none" else tpg.make_norm(dev(w), EPS)
    for use_perm, use_n, use_res in ((True, True, True), (True, False, False), (False, True, False)):
        dn, mag = (combine(dxp.double(), slot_row, torch.ones(T, k, dtype=torch.float64)) if use_perm else (0.0, 0.0))
        if use_n:
            dn, mag = dn + dxn.double(), mag + dxn.double().abs()
        if not torch.is_tensor(dn):
            continue
        xv = x.double().requires_grad_(True)
        wv = (torch.ones(H, dtype=torch.float64) if w is None else w.double()).requires_grad_(True)
        f = xv if form == "none" else rms(xv, wv, EPS)
        (f * dn).sum().backward()
        base = dres.double() if use_res else torch.zeros(T, H, dtype=torch.float64)
        hat = rms(x.double(), None, EPS)
        r = torch.rsqrt((x.double() ** 2).mean(1, keepdim=True) + EPS)
        if form == "none":
            size = mag
        else:
            a = mag * wv.detach().abs()
            size = r * (a + hat.abs() * (a * hat.abs()).mean(1, keepdim=True))
        dx = nan(T, H)
        dw = None if form == "none" else nan(H, dtype=torch.float32)
        ws = workspace(p, tpg.MOE_WS_PRENORM_BACKWARD)
        tpg.moe_prenorm_backward(dev(dxp) if use_perm else None, dev(slot_row) if use_perm else None,
                                 dev(dxn) if use_n else None, dev(dres) if use_res else None, dev(x), norm, p, dx, dw, ws)
        close(dx, xv.grad + base, FP32 * (size + base.abs()), "dx")
        if dw is not None:
            close(dw, wv.grad, FP32 * (mag * hat.abs()).sum(0), "dweight", half=0.0)
            only = nan(T, H)  # without dweight no workspace is needed, and dx is the same
            tpg.moe_prenorm_backward(dev(dxp) if use_perm else None, dev(slot_row) if use_perm else None,
                                     dev(dxn) if use_n else None, dev(dres) if use_res else None, dev(x), norm, p, only)
            assert torch.equal(only, dx)


def _end_problem(T, H, E, k, drop, gate, form, residual, seed=0):
    g = _gen(T, H, k, seed)
    offsets, slot_row, tw = routing(T, E, k, g, drop)
    y = bf16(T * k, H, g=g)
    y[int(offsets[-1]):] = float("nan")
    tw = torch.where(slot_row < 0, float("nan"), tw)  # a dropped slot's weight is never used
    w = bf16(H, g=g) if form == "norm" else None
    res = bf16(T, H, g=g) if residual else None
    gv = {"none": None, "channel": torch.randn(H, generator=g), "token": torch.randn(T, generator=g)}[gate]
    kind = {"none": tpg.MOE_GATE_NONE, "channel": tpg.MOE_GATE_CHANNEL, "token": tpg.MOE_GATE_TOKEN}[gate]
    keep = [dev(v) for v in (y, slot_row, tw, w, res, gv)]
    norm = None if form == "none" else tpg.make_norm(keep[3], EPS)
    rd = None if not residual and gate == "none" else tpg.make_residual(keep[4], -0.6, keep[5], kind)
    return dict(g=g, slot_row=slot_row, tw=tw, y=y, w=w, res=res, gate=gv, keep=keep, norm=norm, residual=rd,
                p=_problem(T, H, E, k), R=int(offsets[-1]))


def _end_forward(c, y, tw, w, res, gate, kind):
    """fp64 out and the magnitude of its terms"""
    s, mag = combine(y, c["slot_row"], tw)
    r = torch.rsqrt((s * s).mean(1, keepdim=True) + EPS) if c["norm"] is not None else 1.0
    f = r if w is None else r * w
    if gate is not None:
        f = f * (gate[:, None] if kind == "token" else gate)
    out = f * s
    size = (f.abs() if torch.is_tensor(f) else 1.0) * mag
    if res is not None:
        out, size = out - 0.6 * res, size + (0.6 * res).abs()
    return out, size.detach()


END_CASES = [(1, 128, 4, 2, 0.0), (1, 7168, 32, 8, 0.0), (37, 640, 16, 3, 0.3), (700, 256, 8, 2, 0.1),
             (5, 8320, 12, 9, 0.2), (3, 16512, 4, 1, 0.0), (2, 65536, 20, 17, 0.2), (2500, 128, 4, 1, 0.5),
             (6, 384, 4, 2, 1.0)]
FORMS = [("norm", "channel", True), ("norm", "token", True), ("ones", "none", True), ("none", "token", False),
         ("none", "channel", True), ("norm", "none", False), ("none", "none", False)]


@pytest.mark.parametrize("T,H,E,k,drop", END_CASES)
@pytest.mark.parametrize("form,gate,residual", FORMS)
def test_combine_norm(T, H, E, k, drop, form, gate, residual):
    c = _end_problem(T, H, E, k, drop, gate, form, residual)
    d = lambda t: None if t is None else t.double()  # noqa: E731
    ref, size = _end_forward(c, d(c["y"]), d(c["tw"]), d(c["w"]), d(c["res"]), d(c["gate"]), gate)
    y, slot_row, tw, _, res, _ = c["keep"]
    out = nan(T, H)
    tpg.moe_combine_norm(y, slot_row, tw, c["norm"], c["residual"], c["p"], out)
    close(out, ref, FP32 * size, "out")
    if residual:
        tpg.moe_combine_norm(y, slot_row, tw, c["norm"], c["residual"], c["p"], res)  # into the residual
        assert torch.equal(res, out)
    if form == gate == "none" and not residual:
        plain = nan(T, H)
        tpg.moe_unpermute_combine(y, slot_row, tw, c["p"], plain)
        assert torch.equal(plain, out)


@pytest.mark.parametrize("T,H,E,k,drop", END_CASES)
@pytest.mark.parametrize("form,gate,residual", FORMS)
def test_combine_norm_backward(T, H, E, k, drop, form, gate, residual):
    c = _end_problem(T, H, E, k, drop, gate, form, residual, seed=1)
    dout = bf16(T, H, g=c["g"])
    live = c["slot_row"] >= 0
    leaves = {n: None if c[n] is None else torch.nan_to_num(c[n].double()).requires_grad_(True)
              for n in ("y", "tw", "w", "res", "gate")}
    if form == "ones":
        leaves["w"] = torch.ones(H, dtype=torch.float64, requires_grad=True)
    out, _ = _end_forward(c, leaves["y"], leaves["tw"], leaves["w"], leaves["res"], leaves["gate"], gate)
    out.backward(dout.double())
    # magnitudes: dc and the sums over it
    with torch.no_grad():
        s, mag = combine(leaves["y"], c["slot_row"], leaves["tw"])
        on = form != "none"
        r = torch.rsqrt((s * s).mean(1, keepdim=True) + EPS) if on else torch.ones(T, 1, dtype=torch.float64)
        w = torch.ones(H, dtype=torch.float64) if leaves["w"] is None else leaves["w"].abs()
        gv = 1.0 if gate == "none" else leaves["gate"].abs()[:, None] if gate == "token" else leaves["gate"].abs()
        b = dout.double().abs() * gv * w
        dc = r * b + (r ** 3 * mag * (b * mag).mean(1, keepdim=True) if on else 0.0)
        twl = torch.where(live, leaves["tw"], 0.0).abs()
        dy_size = torch.zeros(T * k, H, dtype=torch.float64)
        dtw_size = torch.zeros(T, k, dtype=torch.float64)
        for j in range(k):
            m = live[:, j]
            rows = c["slot_row"][m, j].long()
            dy_size[rows] = dc[m] * twl[m, j:j + 1]
            dtw_size[m, j] = (dc[m] * leaves["y"][rows].abs()).sum(1)
    y, slot_row, tw, _, res, _ = c["keep"]
    p = c["p"]
    dy, dtw = nan(T * k, H), nan(T, k, dtype=torch.float32)
    dres = nan(T, H) if residual else None
    dw = nan(H, dtype=torch.float32) if on else None
    dgate = None if gate == "none" else nan(H if gate == "channel" else T, dtype=torch.float32)
    ws = workspace(p, tpg.MOE_WS_COMBINE_NORM_BACKWARD)
    tpg.moe_combine_norm_backward(dev(dout), y, slot_row, tw, c["norm"], c["residual"], p, dy, dtw, dres, dw, dgate, ws)
    R = c["R"]
    close(dy[:R], leaves["y"].grad[:R], FP32 * dy_size[:R], "dy")
    assert torch.isnan(dy[R:]).all()
    close(dtw, torch.where(live, leaves["tw"].grad, 0.0), FP32 * dtw_size, "dtopk_w", half=0.0)
    if residual:
        close(dres, leaves["res"].grad, FP32 * leaves["res"].grad.abs(), "dresidual")
    if on:
        close(dw, leaves["w"].grad, FP32 * (dout.double().abs() * gv * r * mag).sum(0), "dweight", half=0.0)
    if dgate is not None:
        close(dgate, leaves["gate"].grad, FP32 * (dout.double().abs() * w * r * mag).sum(1 if gate == "token" else 0),
              "dgate", half=0.0)
    # fewer outputs, and dy over y: the same values, no workspace
    again = y.clone()
    tpg.moe_combine_norm_backward(dev(dout), again, slot_row, tw, c["norm"], c["residual"], p, again)
    assert torch.equal(again[:R], dy[:R])


@pytest.mark.parametrize("scale", [float("nan"), float("inf")])
def test_scale_of_no_residual_is_not_used(scale):
    T, H = 9, 256
    c = _end_problem(T, H, 4, 2, 0.3, "token", "norm", False, seed=4)
    y, slot_row, tw, _, _, gate = c["keep"]
    out, want = nan(T, H), nan(T, H)
    for s, o in ((scale, out), (1.0, want)):
        tpg.moe_combine_norm(y, slot_row, tw, c["norm"], tpg.make_residual(None, s, gate, tpg.MOE_GATE_TOKEN), c["p"], o)
    assert torch.isfinite(want).all() and torch.equal(out, want)


@pytest.mark.parametrize("T,H,k", [(5, 640, 1), (40, 4096, 1), (33, 256, 3), (2, 16512, 1), (7, 384, 9)])
def test_weight_gradient_of_a_token_with_one_live_slot(T, H, k):
    """the norm takes a single weight out again but for eps: dtopk_w = r^3 eps (b . y), a difference of two numbers
    that agree to five digits and more if it is not computed as that"""
    g = _gen(T, H, k)
    idx = torch.full((T, k), -1)
    idx[torch.arange(T), torch.randint(0, k, (T,), generator=g)] = torch.randint(0, 4, (T,), generator=g)
    offsets, slot_row = tables(idx, 4)
    y, dout, w = bf16(T * k, H, g=g), bf16(T, H, g=g), bf16(H, g=g)
    tw = torch.rand(T, k, generator=g) + 0.1
    p = tpg.make_problem(T, H, 256, max(4, k), k)
    dtw = nan(T, k, dtype=torch.float32)
    keep = dev(w)
    tpg.moe_combine_norm_backward(dev(dout), dev(y), dev(slot_row), dev(tw), tpg.make_norm(keep, EPS), None, p,
                                  nan(T * k, H), dtw)
    live = slot_row >= 0
    rows = y.double()[slot_row[live].long()]
    c = rows * tw[live].double()[:, None]
    r = torch.rsqrt((c * c).mean(1) + EPS)
    by = dout.double() * w.double() * rows
    want, size = torch.zeros(T, k, dtype=torch.float64), torch.zeros(T, k, dtype=torch.float64)
    want[live], size[live] = r ** 3 * EPS * by.sum(1), r ** 3 * EPS * by.abs().sum(1)
    close(dtw, want, FP32 * size, "dtopk_w", half=0.0)


@pytest.mark.parametrize("prec,flags", [("bf16", 0), ("bf16", tpg.MOE_FLAG_SCATTER_Y), ("w4a8", 0),
                                        ("w4a8_mx", tpg.MOE_FLAG_SCATTER_Y), ("w4a8", tpg.MOE_FLAG_SCATTER_Y)])
@pytest.mark.parametrize("T", [1, 70, 1100])
def test_forward_norm_is_the_forward_with_the_norm_behind_it(prec, flags, T):
    cfg = MoeConfig("norm_fwd", T=T, H=512, I=256, E=8, k=2, prec=prec, drop_p=0.2)
    d = DeviceProblem(generate(cfg, seed=T), flags)
    g = _gen(T)
    w, res, gate = dev(bf16(512, g=g)), dev(bf16(T, 512, g=g)), dev(torch.randn(T, generator=g))
    norm, rd = tpg.make_norm(w, EPS), tpg.make_residual(res, 0.5, gate, tpg.MOE_GATE_TOKEN)
    idx, tw = d.route()
    offsets, row_src, slot_row, xp, xps = d.permute(idx)
    y = d.grouped_ffn(xp, xps, offsets)
    want, out = nan(T, 512), nan(T, 512)
    tpg.moe_combine_norm(y, slot_row, tw, norm, rd, d.p, want)
    tpg.moe_forward_norm(d.logits, d.drop, d.x, d.x_scale, d.weights, norm, rd, d.p, out,
                         d.workspace(tpg.MOE_WS_FORWARD, fill=0xEF))
    assert torch.isfinite(want).all() and torch.equal(out, want)
    tpg.moe_forward_norm(d.logits, d.drop, d.x, d.x_scale, d.weights, None, None, d.p, out,
                         d.workspace(tpg.MOE_WS_FORWARD, fill=0xEF))
    assert torch.equal(out.view(torch.int16), d.forward())


def test_prenorm_feeds_the_w4a8_forward():
    """prenorm's fp8 rows and scales are what the W4A8 forward takes"""
    cfg = MoeConfig("pre_w4", T=33, H=512, I=256, E=8, k=2, prec="w4a8")
    d = DeviceProblem(generate(cfg, seed=2))
    x = dev(bf16(33, 512, g=_gen(3)))
    q, sc = torch.empty(33, 512, dtype=torch.uint8, device=DEV), torch.empty(33, 4, device=DEV)
    tpg.moe_prenorm(x, tpg.make_norm(None, EPS), d.p, None, q, sc)
    d.x, d.x_scale = q, sc
    out = d.forward().view(torch.bfloat16)
    assert torch.isfinite(out).all()
    # the same layer on the rows the codes stand for, through bf16 products
    import oracle
    ref = oracle.moe_forward(dict(d.inp, x=q.cpu().numpy(), x_scale=sc.cpu().numpy()))
    err = (out.cpu().double() - torch.from_numpy(ref)).abs().max() / abs(ref).max()
    assert err <= 3e-2


def test_more_tokens_than_one_grid_dimension_holds():
    """2^20 + 3 tokens: the last ones are workgroups of the second grid row"""
    T, H = (1 << 20) + 3, 128
    p = tpg.make_problem(T, H, 128, 1, 1)
    x = torch.randn(T, H, device=DEV).to(torch.bfloat16)
    xn = nan(T, H)
    tpg.moe_prenorm(x, tpg.make_norm(None, EPS), p, xn)
    ref = x.double() * torch.rsqrt(x.double().square().mean(1, keepdim=True) + EPS)
    assert bool(((xn.double() - ref).abs() <= (HALF + FP32) * ref.abs()).all())
    slot_row = torch.arange(T - 1, -1, -1, dtype=torch.int32, device=DEV)
    w = torch.rand(T, 1, device=DEV) + 0.5
    out = nan(T, H)
    tpg.moe_combine_norm(x, slot_row, w, tpg.make_norm(None, EPS), None, p, out)
    c = x.double().flip(0) * w.double()
    ref = c * torch.rsqrt(c.square().mean(1, keepdim=True) + EPS)
    assert bool(((out.double() - ref).abs() <= (HALF + FP32) * ref.abs()).all())


@pytest.mark.parametrize("T,H,E,k", [(700, 384, 8, 2), (5, 7168, 12, 9), (3, 16512, 4, 2)])
def test_gradients_over_their_inputs(T, H, E, k):
    """dx may be dres, dxn or x; dresidual may be dout, with dy over y at the same time"""
    g = _gen(T, H, k, 2)
    p = _problem(T, H, E, k)
    _, slot_row, _ = routing(T, E, k, g, 0.1)
    dxp, dxn, dres, x = (dev(bf16(n, H, g=g)) for n in (T * k, T, T, T))
    sr, norm = dev(slot_row), tpg.make_norm(dev(bf16(H, g=g)), EPS)
    ws = workspace(p, tpg.MOE_WS_PRENORM_BACKWARD)
    want, dw = nan(T, H), nan(H, dtype=torch.float32)
    tpg.moe_prenorm_backward(dxp, sr, dxn, dres, x, norm, p, want, dw, ws)
    assert torch.isfinite(want).all()
    for i in range(3):
        a = [t.clone() for t in (dxn, dres, x)]
        dw2 = nan(H, dtype=torch.float32)
        tpg.moe_prenorm_backward(dxp, sr, *a, norm, p, a[i], dw2, ws)
        assert torch.equal(a[i], want) and torch.equal(dw2, dw), i

    c = _end_problem(T, H, E, k, 0.1, "channel", "norm", True, seed=2)
    dout = dev(bf16(T, H, g=g))
    y, slot_row, tw = c["keep"][:3]
    ws = workspace(p, tpg.MOE_WS_COMBINE_NORM_BACKWARD)

    def run(dout, y, dy, dres):
        o = [nan(T, k, dtype=torch.float32), nan(H, dtype=torch.float32), nan(H, dtype=torch.float32)]
        tpg.moe_combine_norm_backward(dout, y, slot_row, tw, c["norm"], c["residual"], p, dy, o[0], dres, o[1], o[2], ws)
        return [dy[:c["R"]], dres] + o

    want = run(dout, y, nan(T * k, H), nan(T, H))
    d2, y2 = dout.clone(), y.clone()
    for a, b in zip(run(d2, y2, y2, d2), want):
        assert torch.isfinite(b).all() and torch.equal(a, b)


@pytest.mark.parametrize("prec", ["bf16", "w4a8"])
@pytest.mark.parametrize("T", [3, 600])
def test_block_forward_in_place_and_in_a_graph(prec, T):
    """prenorm and the block behind it, out over the residual, on another stream and captured with the steps of
    another problem between the replays"""
    cfg = MoeConfig("norm_graph", T=T, H=512, I=256, E=8, k=2, prec=prec, drop_p=0.2)
    d = DeviceProblem(generate(cfg, seed=T))
    g = _gen(T, 9)
    w, gate = dev(bf16(512, g=g)), dev(torch.randn(512, generator=g))
    x0 = dev(bf16(T, 512, g=g))
    x = x0.clone()
    norm, rd = tpg.make_norm(w, EPS), tpg.make_residual(x, 0.5, gate, tpg.MOE_GATE_CHANNEL)
    ws = d.workspace(tpg.MOE_WS_FORWARD, fill=0xEF)
    bf = prec == "bf16"
    xn = nan(T, 512) if bf else torch.zeros(T, 512, dtype=torch.uint8, device=DEV)
    sc = None if bf else nan(T, 4, dtype=torch.float32)

    def run(out):
        tpg.moe_prenorm(x, norm, d.p, xn if bf else None, None if bf else xn, sc)
        tpg.moe_forward_norm(d.logits, d.drop, xn, sc, d.weights, norm, rd, d.p, out, ws)

    want = nan(T, 512)
    run(want)
    torch.cuda.synchronize()
    assert torch.isfinite(want).all() and torch.equal(x, x0)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run(x)
    torch.cuda.synchronize()
    assert torch.equal(x, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(x)
    other = nan(70, 640)
    for _ in range(4):
        x.copy_(x0)
        ws.fill_(0xEF)
        tpg.moe_prenorm(dev(bf16(70, 640, g=g)), None, _problem(70, 640), other)  # eager work between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, want)
