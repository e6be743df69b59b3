"""The gradients of the router and of the grouped FFN, and a whole training step of the block, against fp64.

The bounds are element-wise: an output is off by its own half step, by what the half steps of the
bf16 intermediates (h, dgu) make of it through the products, and by the fp32 accumulation."""
from __future__ import annotations

import pytest
import torch

import token_permute_grouped_amd as tpg
from tests._block import FP32, HALF, bf16, close, dev, glu, nan, rms, routing, stored_rows, workspace
from tests._gpu import DEV

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------------------------------------ router
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 4, 4), (3, 16, 2), (17, 32, 8), (50, 64, 6), (200, 128, 8),
                                   (33, 200, 40), (5, 256, 256), (1000, 8, 1)])
@pytest.mark.parametrize("drop", [0.0, 0.3])
def test_route_topk_backward(T, E, k, drop):
    g = _gen(T + E)
    logits = torch.randn(T, E, generator=g) * 3
    mask = (torch.rand(T, k, generator=g) < drop).to(torch.uint8)
    d = torch.randn(T, k, generator=g)
    lv = logits.double().requires_grad_(True)
    top, _ = torch.topk(lv, k)
    w = torch.softmax(top, 1)
    dm = torch.where(mask != 0, 0.0, d.double())
    (w * dm).sum().backward()
    d = torch.where(mask != 0, float("nan"), d)  # a dropped slot's gradient is not read
    out = nan(T, E, dtype=torch.float32)
    p = tpg.make_problem(T, 128, 128, E, k)
    tpg.moe_route_topk_backward(dev(logits), dev(mask) if drop else None, dev(d), p, out)
    # |dl| <= w (|d| + sum w |d|); k-term sums
    size = torch.zeros(T, E, dtype=torch.float64)
    idx = torch.topk(logits, k)[1]
    wd = w.detach()
    size.scatter_(1, idx, wd * (dm.abs() + (wd * dm.abs()).sum(1, keepdim=True)))
    close(out, lv.grad, FP32 * size, "dlogits", half=0.0)
    assert (out.cpu()[size == 0] == 0).all()


def test_route_topk_backward_ties_go_to_the_lower_expert():
    p = tpg.make_problem(2, 128, 128, 8, 2)
    logits = torch.zeros(2, 8)
    logits[1, 3:6] = 1.0
    out = nan(2, 8, dtype=torch.float32)
    tpg.moe_route_topk_backward(dev(logits), None, torch.tensor([[1.0, 3.0]] * 2, device=DEV), p, out)
    want = torch.zeros(2, 8)
    want[0, :2] = torch.tensor([-0.5, 0.5])
    want[1, 3:5] = torch.tensor([-0.5, 0.5])
    assert torch.equal(out.cpu(), want)


# ------------------------------------------------------------------------------------------------ grouped FFN
class Ffn:
    """rows of experts with the given counts, spare rows behind them full of NaN (one row is always spare where the
    bound on the tiles, S / 256 + min(E, S), has to pass 256)"""

    def __init__(self, counts, H, I, il=0, clamp=0.0, spare=3, seed=0, scale=1.0, experts=0):
        """experts: as many in all, those behind `counts` without rows"""
        g = _gen(seed + H + I)
        self.live_experts = len(counts)
        counts = counts + [0] * (experts - len(counts))
        E, R = len(counts), sum(counts)
        spare = max(spare, experts + 1 - R)
        self.counts, self.H, self.I, self.il, self.clamp, self.R, self.S = counts, H, I, il, clamp, R, R + spare
        self.off = [sum(counts[:e]) for e in range(E + 1)]
        self.p = tpg.make_problem(R + spare, H, I, E, 1, tpg.MOE_PREC_BF16, il, clamp)
        self.w1, self.w2 = bf16(E, 2 * I, H, g=g, std=H ** -0.5), bf16(E, H, I, g=g, std=I ** -0.5)
        self.x, self.dy, self.gu = bf16(self.S, H, g=g, std=scale), bf16(self.S, H, g=g), bf16(self.S, 2 * I, g=g, std=scale)
        for t in (self.x, self.dy, self.gu):
            t[R:] = float("nan")
        self.offsets = torch.tensor(self.off, dtype=torch.int32)
        self.dw1, self.dw2 = dev(self.w1), dev(self.w2)
        self.weights = tpg.make_weights(self.dw1, self.dw2)

    def backward(self, dx=True, dw1=True, dw2=True, ws=None):
        E = len(self.counts)
        o = [nan(self.S, self.H) if dx else None, nan(E, 2 * self.I, self.H) if dw1 else None,
             nan(E, self.H, self.I) if dw2 else None]
        tpg.moe_grouped_ffn_backward(dev(self.dy), dev(self.x) if dw1 else None, dev(self.gu), dev(self.offsets),
                                     self.weights, self.p, *o,
                                     workspace(self.p, tpg.MOE_WS_FFN_BACKWARD) if ws is None else ws)
        return o

    def reference(self):
        """(value, slack) of dx, dw1, dw2 by autograd of the fp64 forward"""
        E, H, I = self.live_experts, self.H, self.I
        dx, dxs = torch.zeros(self.R, H, dtype=torch.float64), torch.zeros(self.R, H, dtype=torch.float64)
        dw1, dw1s = (torch.zeros(E, 2 * I, H, dtype=torch.float64) for _ in range(2))
        dw2, dw2s = (torch.zeros(E, H, I, dtype=torch.float64) for _ in range(2))
        for e in range(E):
            a, b = self.off[e], self.off[e + 1]
            if a == b:
                continue
            x, dy, w1, w2 = (t.double() for t in (self.x[a:b], self.dy[a:b], self.w1[e], self.w2[e]))
            gu = self.gu[a:b].double().requires_grad_(True)
            h = glu(gu, I, self.il, self.clamp)
            dh = dy @ w2
            h.backward(dh)
            dgu, h = gu.grad, h.detach()
            # dgu = dh f: its half step, and dh's accumulation over H products through |f| <= |dgu / dh|
            gv = self.gu[a:b].double().requires_grad_(True)
            hv = glu(gv, I, self.il, self.clamp)
            hv.backward(torch.ones_like(hv))
            dh_mag = dy.abs() @ w2.abs()
            both = torch.cat([dh_mag, dh_mag], 1)[:, torch.argsort(stored_rows(I, self.il))]
            # the factor itself is a product of fp32 values with a sum 1 + g (1 - s) in it: |u| s (1 + |g|) at most
            gs, us = (self.gu[a:b].double()[:, stored_rows(I, self.il)][:, i * I:(i + 1) * I].abs() for i in (0, 1))
            fac = torch.cat([us * (1 + gs), gs], 1)[:, torch.argsort(stored_rows(I, self.il))]
            ddgu = HALF * dgu.abs() + FP32 * both * (gv.grad.abs() + fac)
            dh_ = HALF * h.abs() + FP32 * h.abs()
            dx[a:b], dxs[a:b] = dgu @ w1, ddgu @ w1.abs() + FP32 * (dgu.abs() @ w1.abs())
            dw1[e], dw1s[e] = dgu.T @ x, ddgu.T @ x.abs() + FP32 * (dgu.abs().T @ x.abs())
            dw2[e], dw2s[e] = dy.T @ h, dy.abs().T @ dh_ + FP32 * (dy.abs().T @ h.abs())
        return (dx, dxs), (dw1, dw1s), (dw2, dw2s)

    def check(self, o):
        R = self.R
        for (ref, slack), got, what in zip(self.reference(), o, ("dx", "dw1", "dw2")):
            if got is None:
                continue
            if what == "dx":
                assert torch.isnan(got[R:]).all()  # rows behind the last one stay
                got = got[:R]
            else:
                assert (got[self.live_experts:] == 0).all()
                got = got[:self.live_experts]
            close(got, ref, slack, what)


# counts around the sizes where the kernels change: 32-row stages of the weight gradients, 64-row sparse
# and 256-row full tiles of the others; empty experts at both ends; H and I of one and a half tiles
FFN_CASES = {
    "one_row": dict(counts=[1], H=128, I=128),
    "empty": dict(counts=[0, 0], H=128, I=256),
    "stages": dict(counts=[0, 31, 32, 33, 63, 64, 65, 0], H=256, I=128),
    "tiles": dict(counts=[255, 256, 257], H=128, I=384, il=32),
    "ragged": dict(counts=[5, 0, 300, 1, 170], H=384, I=384, clamp=0.7),
    "interleaved": dict(counts=[40, 129, 2], H=640, I=256, il=32, clamp=10.0),
    "many_experts": dict(counts=[(7 * e) % 5 for e in range(256)], H=128, I=128),
    "long": dict(counts=[2000], H=256, I=256),
    "wide": dict(counts=[70, 3], H=1152, I=640),
    "large_values": dict(counts=[50, 20], H=128, I=128, scale=60.0),
    "long_ragged": dict(counts=[1, 900, 129, 127], H=384, I=128, il=32),
}


@pytest.mark.parametrize("experts", [0, 256])
@pytest.mark.parametrize("name", FFN_CASES)
def test_grouped_ffn_backward(name, experts):
    """a small layer takes tiles of 128; with 256 experts (most of them empty) the bound on its tiles is above what
    fits the chip, and it takes tiles of 256"""
    f = Ffn(**FFN_CASES[name], experts=experts)
    f.check(f.backward())


@pytest.mark.parametrize("dx,dw1,dw2", [(True, False, False), (False, True, False), (False, False, True)])
def test_grouped_ffn_backward_of_some_gradients(dx, dw1, dw2):
    f = Ffn(counts=[30, 0, 70], H=256, I=128)
    part, whole = f.backward(dx, dw1, dw2), f.backward()
    for a, b in zip(part, whole):
        assert a is None or torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_clamp_gradient_on_the_border():
    """a pre-activation of exactly the clamp keeps its gradient, one step beyond it has none"""
    f = Ffn(counts=[8], H=128, I=128, clamp=1.0)
    f.gu[:8, :64], f.gu[:8, 64:128] = 1.0, -1.0
    f.gu[:8, 128:192], f.gu[:8, 192:] = 1.0078125, -1.0
    f.check(f.backward())


@pytest.mark.parametrize("experts", [0, 256])
@pytest.mark.parametrize("name", FFN_CASES)
def test_grouped_ffn_train(name, experts):
    """y is moe_grouped_ffn's, bit for bit, in small tiles and in the forward's own; gu is the first product"""
    f = Ffn(**FFN_CASES[name], experts=experts)
    gu, y, want = nan(f.S, 2 * f.I), nan(f.S, f.H), nan(f.S, f.H)
    x = dev(f.x)
    tpg.moe_grouped_ffn_train(x, dev(f.offsets), f.weights, f.p, gu, y, workspace(f.p, tpg.MOE_WS_GROUPED_FFN))
    tpg.moe_grouped_ffn(x, None, dev(f.offsets), f.weights, f.p, want, workspace(f.p, tpg.MOE_WS_GROUPED_FFN))
    assert torch.equal(y[:f.R], want[:f.R]) and torch.isfinite(want[:f.R]).all()
    assert torch.isnan(y[f.R:]).all() and torch.isnan(gu[f.R:]).all()
    for e in range(f.live_experts):
        a, b = f.off[e], f.off[e + 1]
        xe, we = f.x[a:b].double(), f.w1[e].double()
        close(gu[a:b], xe @ we.T, FP32 * (xe.abs() @ we.abs().T), f"gu of expert {e}")


# ------------------------------------------------------------------------------------------------ a training step
class Step:
    """forward and backward of the block through the library: x -> prenorm -> route -> permute -> FFN ->
    combine, norm, gate, residual; the router's product is the caller's"""

    def __init__(self, T=90, H=256, I=128, E=8, k=2, il=32, clamp=2.0, drop=0.15, seed=0):
        g = _gen(seed)
        self.T, self.H, self.I, self.E, self.k, self.il, self.clamp = T, H, I, E, k, il, clamp
        self.v = dict(x=bf16(T, H, g=g), wp=bf16(H, g=g, std=0.2) + 1, wq=bf16(H, g=g, std=0.2) + 1,
                      wr=bf16(E, H, g=g, std=H ** -0.5), w1=bf16(E, 2 * I, H, g=g, std=H ** -0.5),
                      w2=bf16(E, H, I, g=g, std=I ** -0.5), gate=torch.randn(H, generator=g))
        self.drop = (torch.rand(T, k, generator=g) < drop).to(torch.uint8)
        self.dout = bf16(T, H, g=g)
        self.p = tpg.make_problem(T, H, I, E, k, tpg.MOE_PREC_BF16, il, clamp)
        self.d = {n: dev(t) for n, t in self.v.items()}
        self.ddrop, self.ddout = dev(self.drop), dev(self.dout)
        self.norm, self.post = tpg.make_norm(self.d["wp"], 1e-5), tpg.make_norm(self.d["wq"], 1e-5)
        self.res = tpg.make_residual(self.d["x"], 0.9, self.d["gate"], tpg.MOE_GATE_CHANNEL)
        self.weights = tpg.make_weights(self.d["w1"], self.d["w2"])
        S, f32, i32 = T * k, torch.float32, torch.int32
        e = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device=DEV)  # noqa: E731
        self.b = dict(xn=e(T, H), logits=e(T, E, dtype=f32), idx=e(T, k, dtype=i32), tw=e(T, k, dtype=f32),
                      offsets=e(E + 1, dtype=i32), row_src=e(S, dtype=i32), slot_row=e(S, dtype=i32), xp=e(S, H),
                      gu=e(S, 2 * I), y=e(S, H), out=e(T, H), dy=e(S, H), dtw=e(T, k, dtype=f32), dres=e(T, H),
                      dwq=e(H, dtype=f32), dgate=e(H, dtype=f32), dxp=e(S, H), dw1=e(E, 2 * I, H), dw2=e(E, H, I),
                      dlogits=e(T, E, dtype=f32), dxn=e(T, H), dx=e(T, H), dwp=e(H, dtype=f32), dwr=e(E, H, dtype=f32))
        self.ws = {n: workspace(self.p, w) for n, w in dict(permute=tpg.MOE_WS_PERMUTE, ffn=tpg.MOE_WS_GROUPED_FFN,
                   ffn_b=tpg.MOE_WS_FFN_BACKWARD, pre=tpg.MOE_WS_PRENORM_BACKWARD,
                   end=tpg.MOE_WS_COMBINE_NORM_BACKWARD).items()}

    def run(self):
        b, p, ws, d = self.b, self.p, self.ws, self.d
        tpg.moe_prenorm(d["x"], self.norm, p, b["xn"])
        torch.mm(b["xn"].float(), d["wr"].float().T, out=b["logits"])
        tpg.moe_route_topk(b["logits"], self.ddrop, p, b["idx"], b["tw"])
        tpg.moe_permute(b["xn"], None, b["idx"], p, b["offsets"], b["row_src"], b["slot_row"], b["xp"], None, ws["permute"])
        tpg.moe_grouped_ffn_train(b["xp"], b["offsets"], self.weights, p, b["gu"], b["y"], ws["ffn"])
        tpg.moe_combine_norm(b["y"], b["slot_row"], b["tw"], self.post, self.res, p, b["out"])
        tpg.moe_combine_norm_backward(self.ddout, b["y"], b["slot_row"], b["tw"], self.post, self.res, p, b["dy"], b["dtw"],
                                      b["dres"], b["dwq"], b["dgate"], ws["end"])
        tpg.moe_grouped_ffn_backward(b["dy"], b["xp"], b["gu"], b["offsets"], self.weights, p, b["dxp"], b["dw1"], b["dw2"],
                                     ws["ffn_b"])
        tpg.moe_route_topk_backward(b["logits"], self.ddrop, b["dtw"], p, b["dlogits"])
        torch.mm(b["dlogits"].T, b["xn"].float(), out=b["dwr"])
        b["dxn"].copy_(b["dlogits"] @ d["wr"].float())
        tpg.moe_prenorm_backward(b["dxp"], b["slot_row"], b["dxn"], b["dres"], d["x"], self.norm, p, b["dx"], b["dwp"],
                                 ws["pre"])

    def loss(self, v, idx):
        """fp64 <out, dout> for leaves v, with the experts idx chosen and the sides of the clamp that the library's
        pre-activations took: both are steps, which rounding may put a value on the other side of.  (Near the
        clamp of 2 the pre-activations' density is 0.054 on either side; half a step of bf16 is 2^-7 there, and four
        borders (gate, up, +, -) put 4 * 0.054 * 2^-7 * E|error| / half step (1/2) = 0.08 % of the values across:
        alone sqrt(0.0008) = 2.9 % of the gradient's norm.)"""
        gu, slot_row = self.b["gu"].cpu().double(), self.b["slot_row"].cpu().reshape(self.T, self.k).long()
        xn = rms(v["x"], v["wp"], 1e-5)
        logits = xn @ v["wr"].T
        tw = torch.softmax(logits.gather(1, idx), 1)
        live = self.drop == 0
        c = torch.zeros(self.T, self.H, dtype=torch.float64)
        for e in range(self.E):
            t, j = ((idx == e) & live).nonzero(as_tuple=True)
            y = glu(xn[t] @ v["w1"][e].T, self.I, self.il, self.clamp, gu[slot_row[t, j]]) @ v["w2"][e].T
            c = c.index_add(0, t, tw[t, j][:, None] * y)
        out = 0.9 * v["x"] + v["gate"] * rms(c, v["wq"], 1e-5)
        return (out * self.dout.double()).sum()


GRADS = dict(x="dx", wp="dwp", wq="dwq", wr="dwr", w1="dw1", w2="dw2", gate="dgate")


def _choice(s):
    """the experts the library's logits choose (bf16 xn), dropped slots included"""
    return torch.sort(s.b["logits"].cpu(), dim=1, descending=True, stable=True)[1][:, :s.k]


def test_training_step_of_the_block():
    s = Step()
    s.run()
    torch.cuda.synchronize()
    idx = _choice(s)
    v = {n: t.double().requires_grad_(True) for n, t in s.v.items()}
    s.loss(v, idx).backward()
    for n, gname in GRADS.items():
        got, ref = s.b[gname].cpu().double(), v[n].grad
        rel = ((got - ref).norm() / ref.norm()).item()
        print(f"[step] {gname}: relative error {rel:.2e}", flush=True)
        # roundings to bf16 on the way: xn, gu, h, y, dy, dgu, dx rows, dxn and the output, each at most half a
        # step (2^-8) of a factor; nine of them in quadrature are 3 * 2^-8, doubled for the norms' projections
        assert rel <= 6 * HALF, (gname, rel)


def test_training_step_against_differences():
    """the gradients' product with a direction is the loss's difference quotient along it"""
    s = Step(seed=3)
    s.run()
    torch.cuda.synchronize()
    idx = _choice(s)
    g = _gen(11)
    base = {n: t.double() for n, t in s.v.items()}
    for n, gname in GRADS.items():
        grad = s.b[gname].cpu().double()
        # along the gradient itself, with a share of a random direction: no cancellation in the product
        dirn = grad / grad.norm() + torch.randn(grad.shape, generator=g, dtype=torch.float64) * (0.3 / grad.numel() ** 0.5)
        h = 1e-4 * base[n].norm()
        up, down = (s.loss(dict(base, **{n: base[n] + sign * h * dirn}), idx) for sign in (1, -1))
        want, got = ((up - down) / (2 * h)).item(), (grad * dirn).sum().item()
        print(f"[differences] {gname}: {got:.6g}, difference quotient {want:.6g}", flush=True)
        assert abs(got - want) <= 6 * HALF * abs(want), gname


def test_training_step_is_reproducible_captured_and_on_another_stream():
    s = Step(seed=5)
    s.run()
    torch.cuda.synchronize()
    want = {n: t.clone() for n, t in s.b.items()}

    def check(what, step=s):
        torch.cuda.synchronize()
        for n, t in want.items():
            same = torch.equal(step.b[n].reshape(-1).view(torch.uint8), t.reshape(-1).view(torch.uint8))
            assert same, f"{what}: {n} differs"

    def spoil():
        for t in s.b.values():
            t.zero_()
        for t in s.ws.values():
            t.fill_(0xFF)

    spoil()
    s.run()
    check("again")
    side = torch.cuda.Stream()
    spoil()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run()
    check("another stream")
    spoil()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    other = Step(seed=6)
    for i in range(4):
        spoil()
        other.run()  # eager work between the replays
        torch.cuda.synchronize()
        graph.replay()
        check(f"replay {i}")


@pytest.mark.parametrize("counts,H,I", [([600, 0, 300], 384, 256), ([40] * 200, 256, 128)])
def test_two_captured_backward_passes_share_a_workspace(counts, H, I):
    """small and large tiles; the passes follow one another on one stream, each writes what it reads of the workspace"""
    a, b = (Ffn(counts, H, I, il=32, clamp=3.0, seed=i) for i in range(2))
    ws = workspace(a.p, tpg.MOE_WS_FFN_BACKWARD)
    dev_in = [[dev(t) for t in (f.dy, f.x, f.gu, f.offsets)] for f in (a, b)]
    outs = [[nan(f.S, H), nan(len(counts), 2 * I, H), nan(len(counts), H, I)] for f in (a, b)]
    want = [f.backward() for f in (a, b)]
    torch.cuda.synchronize()
    graphs = []
    for f, i, o in zip((a, b), dev_in, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            tpg.moe_grouped_ffn_backward(*i, f.weights, f.p, *o, ws)
    for n in range(3):
        ws.fill_(0xFF)
        for o in outs[0] + outs[1]:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        for gr in graphs[::-1] if n == 1 else graphs:
            gr.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs[0] + outs[1], want[0] + want[1]):
            assert torch.equal(o.view(torch.int16), w.view(torch.int16)), n


def test_two_steps_at_once_on_two_streams():
    a, b = Step(seed=7), Step(T=150, H=384, seed=8)
    for s in (a, b):
        s.run()
    torch.cuda.synchronize()
    want = [{n: t.clone() for n, t in s.b.items()} for s in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for s, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                s.run()
    torch.cuda.synchronize()
    for s, w in zip((a, b), want):
        for n, t in w.items():
            assert torch.equal(s.b[n].reshape(-1).view(torch.uint8), t.reshape(-1).view(torch.uint8)), n


def test_sums_over_no_tokens_are_zero():
    p = tpg.make_problem(0, 128, 128, 3, 2)
    dw1, dw2, dw = nan(3, 256, 128), nan(3, 128, 128), nan(128, dtype=torch.float32)
    z = torch.zeros(0, 128, dtype=torch.bfloat16, device=DEV)
    w = tpg.make_weights(dw1, dw2)
    tpg.moe_grouped_ffn_backward(z, z, z, None, w, p, z, dw1, dw2, None)
    assert (dw1 == 0).all() and (dw2 == 0).all()
    n = tpg.make_norm(None, 1e-5)
    tpg.moe_prenorm_backward(z, None, None, None, z, n, p, z, dw, None)
    assert (dw == 0).all()
    dw, dg, gate = nan(128, dtype=torch.float32), nan(128, dtype=torch.float32), torch.ones(128, device=DEV)
    tpg.moe_combine_norm_backward(z, z, None, None, n, tpg.make_residual(None, 1.0, gate, tpg.MOE_GATE_CHANNEL), p, z,
                                  None, None, dw, dg, None)
    assert (dw == 0).all() and (dg == 0).all()
