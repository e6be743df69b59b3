"""The operators that train an MoE block and put its norms around it, as cases to measure.

Five groups: the grouped gated FFN's forward for training (``ffn``) and its backward pass (``ffn_bwd``), the norm in
front of the block (``prenorm``, ``prenorm_bwd``), the combine with the norm, gate and residual behind it
(``combine``, ``combine_bwd``) and the router's gradient (``route_bwd``).  Every group has a plain form in fp32 torch
operations (``own`` false), the library's calls (``own`` true), and the definition in fp64 (``exact``).

Layouts are the library's: rows in expert order with ``offsets`` [E+1], ``slot_row`` [T, k] with -1 for a dropped
slot, W1 [E, 2I, H] as [gate | up] or in 32-row blocks gate, up, gate, up, ..., W2 [E, H, I], bf16 activations.
"""
import math

import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # a training step's FFN forward on the mid-size layer: 24576 rows over 64 experts, about 384 each
        dict(name="ffn_mid", op="ffn", T=4096, H=2048, I=1408, E=64, k=6, il=0, clamp=0.0, zipf=0.0, drop=0.0),
        # a small micro-batch with odd sizes: interleaved gate/up rows, clamped SwiGLU, some slots routed elsewhere
        dict(name="ffn_odd", op="ffn", T=1000, H=896, I=640, E=8, k=2, il=32, clamp=10.0, zipf=0.0, drop=0.1),
        # the backward pass where launches count most: a unit-test-sized layer
        dict(name="ffn_bwd_tiny", op="ffn_bwd", T=64, H=128, I=256, E=8, k=2, il=0, clamp=0.0, zipf=0.0, drop=0.0),
        # the backward pass of the mid-size layer, experts of ragged sizes
        dict(name="ffn_bwd_mid", op="ffn_bwd", T=4096, H=2048, I=1408, E=64, k=6, il=32, clamp=1.0, zipf=0.0, drop=0.1),
        # the backward pass of the benchmark's layer: 131072 rows, Zipf-skewed experts of 1 to 16000 rows
        dict(name="ffn_bwd_skewed", op="ffn_bwd", T=16384, H=4096, I=2048, E=128, k=8, il=0, clamp=0.0, zipf=1.2,
             drop=0.0),
        # one decoded token in front of the W4A8 layer: bf16 row for the router, fp8 row and scales for the experts
        dict(name="prenorm_decode", op="prenorm", T=1, H=7168, fp8=True, bf16=True),
        # a long prompt in front of the bf16 layer
        dict(name="prenorm_long", op="prenorm", T=16384, H=4096, fp8=False, bf16=True),
        # the gradient of the norm in front, collecting a token's rows from the experts, some slots dropped
        dict(name="prenorm_bwd_long", op="prenorm_bwd", T=16384, H=4096, E=128, k=8, zipf=1.2, drop=0.1, router=True),
        # one decoded token behind the W4A8 layer
        dict(name="combine_decode", op="combine", T=1, H=7168, E=32, k=8, zipf=0.0, drop=0.0, gate="channel"),
        # the gradient of the combine, norm, gate and residual on the benchmark's layer
        dict(name="combine_bwd_long", op="combine_bwd", T=16384, H=4096, E=128, k=8, zipf=1.2, drop=0.1,
             gate="token"),
        # the router's gradient of a decode-sized batch, and of the benchmark's layer
        dict(name="route_bwd_small", op="route_bwd", T=256, E=32, k=8, zipf=0.0, drop=0.1),
        dict(name="route_bwd_long", op="route_bwd", T=16384, E=128, k=8, zipf=1.2, drop=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ffn", "ffn_bwd", "prenorm", "prenorm_bwd", "combine", "combine_bwd", "route_bwd"])
    T, H = _log(rng, 1, 16384), 128 * _log(rng, 1, 56)
    E = _log(rng, 1, 256)
    k = rng.randint(1, min(E, 8))
    zipf, drop = rng.choice([0.0, 1.2]), rng.choice([0.0, 0.1, 0.3])
    if op in ("ffn", "ffn_bwd"):
        T = _log(rng, 1, 8192)
        H, I, E = 128 * _log(rng, 1, 32), 128 * _log(rng, 1, 16), _log(rng, 1, 64)
        return dict(op=op, T=T, H=H, I=I, E=E, k=min(k, E), il=rng.choice([0, 32]), clamp=rng.choice([0.0, 1.0, 10.0]),
                    zipf=zipf, drop=drop)
    if op == "prenorm":
        fp8 = rng.random() < 0.5
        return dict(op=op, T=T, H=H, fp8=fp8, bf16=not fp8 or rng.random() < 0.5)
    if op == "prenorm_bwd":
        return dict(op=op, T=T, H=H, E=E, k=k, zipf=zipf, drop=drop, router=rng.random() < 0.5)
    if op == "route_bwd":
        return dict(op=op, T=T, E=E, k=k, zipf=zipf, drop=drop)
    return dict(op=op, T=T, H=H, E=E, k=k, zipf=zipf, drop=drop, gate=rng.choice(["none", "channel", "token"]))


# ------------------------------------------------------------------------------------------------ inputs
def _routing(c, g, dev):
    """A batch's routing: logits, dropped slots, weights, and the permutation tables of the chosen experts."""
    T, E, k = c["T"], c["E"], c["k"]
    logits = torch.randn(T, E, generator=g, device=dev)
    if c["zipf"]:
        rank = torch.randperm(E, generator=g, device=dev) + 1
        logits = logits - c["zipf"] * rank.log()
    top, idx = torch.sort(logits, dim=1, descending=True, stable=True)
    top, idx = top[:, :k], idx[:, :k]
    drop = torch.rand(T, k, generator=g, device=dev) < c["drop"]
    key = torch.where(drop, E, idx).reshape(-1)
    row_src = torch.sort(key, stable=True)[1]
    counts = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=dev)
    offsets[1:] = counts.cumsum(0)
    slot_row = torch.empty(T * k, dtype=torch.int64, device=dev)
    slot_row[row_src] = torch.arange(T * k, device=dev)
    slot_row = torch.where(drop.reshape(-1), -1, slot_row).reshape(T, k)
    return dict(logits=logits, slot_drop=drop.to(torch.uint8), topk_w=torch.softmax(top, 1),
                offsets=offsets.to(torch.int32), slot_row=slot_row.to(torch.int32), bounds=offsets.tolist())


def _gate_rows(I, il, dev):
    """Stored W1 rows of the gate and of the up projections."""
    c = torch.arange(I, device=dev)
    if il == 0:
        return c, I + c
    g = c // il * (2 * il) + c % il
    return g, g + il


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed * 2654435761 % (1 << 62))
    c, op = case, case["op"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).mul_(std)

    def bf16(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.bfloat16).mul_(std)

    s = dict(case=c)
    if op in ("ffn", "ffn_bwd"):
        T, H, I, E, k = (c[n] for n in ("T", "H", "I", "E", "k"))
        r = _routing(c, g, dev)
        s.update(offsets=r["offsets"], bounds=r["bounds"])
        s["w1"], s["w2"] = bf16(E, 2 * I, H, std=H ** -0.5), bf16(E, H, I, std=I ** -0.5)
        s["x"] = bf16(T * k, H)
        if op == "ffn_bwd":
            # what the forward kept, and the gradient that comes back through the combine (weights of about 1/k)
            s["gu"] = torch.empty(T * k, 2 * I, dtype=torch.bfloat16, device=dev)
            for e in range(E):
                a, b = r["bounds"][e], r["bounds"][e + 1]
                if b > a:
                    s["gu"][a:b] = s["x"][a:b] @ s["w1"][e].T
            s["dy"] = bf16(T * k, H, std=1.0 / k)
    elif op == "prenorm":
        s["x"] = bf16(c["T"], c["H"]) * (0.5 + normal(c["T"], 1).abs()).to(torch.bfloat16)
        s["w"] = (1 + normal(c["H"], std=0.1)).to(torch.bfloat16)
    elif op == "prenorm_bwd":
        r = _routing(c, g, dev)
        T, H, k = c["T"], c["H"], c["k"]
        s.update(slot_row=r["slot_row"], x=bf16(T, H), w=(1 + normal(H, std=0.1)).to(torch.bfloat16),
                 dx_perm=bf16(T * k, H, std=1.0 / k), dres=bf16(T, H), dxn=bf16(T, H, std=0.1) if c["router"] else None)
    elif op in ("combine", "combine_bwd"):
        r = _routing(c, g, dev)
        T, H, k = c["T"], c["H"], c["k"]
        s.update(slot_row=r["slot_row"], topk_w=r["topk_w"], y=bf16(T * k, H),
                 w=(1 + normal(H, std=0.1)).to(torch.bfloat16), res=bf16(T, H), scale=0.7,
                 gate={"none": lambda: None, "channel": lambda: normal(H, std=0.2) + 0.5,
                       "token": lambda: torch.sigmoid(normal(T))}[c["gate"]]())
        if op == "combine_bwd":
            s["dout"] = bf16(T, H)
    elif op == "route_bwd":
        r = _routing(c, g, dev)
        s.update(logits=r["logits"], slot_drop=r["slot_drop"], dw=normal(c["T"], c["k"]))
    if own:
        _plan(s, dev)
    return s


# ------------------------------------------------------------------------------------------------ the library's calls
def _plan(s, dev):
    """What a program keeps beside its inputs: the problem, descriptors, workspace and output buffers."""
    import token_permute_grouped_amd as tpg

    c, op = s["case"], s["case"]["op"]
    T, H, E, k = c["T"], c.get("H", 128), c.get("E", 1), c.get("k", 1)
    p = s["p"] = tpg.make_problem(T, H, c.get("I", 128), E, k, tpg.MOE_PREC_BF16, c.get("il", 0), c.get("clamp", 0.0))

    def empty(*shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device=dev)

    def rows(width):  # one row for each slot; those behind the last live row stay as they are
        return torch.zeros(T * k, width, dtype=torch.bfloat16, device=dev)

    def ws(which):
        s["ws"] = empty(max(1, tpg.moe_call_workspace_bytes(p, which)), dtype=torch.uint8)

    if op in ("ffn", "ffn_bwd"):
        I = c["I"]
        s["weights"] = tpg.make_weights(s["w1"], s["w2"])
        if op == "ffn":
            ws(tpg.MOE_WS_GROUPED_FFN)
            s["out"] = [rows(2 * I), rows(H)]
        else:
            ws(tpg.MOE_WS_FFN_BACKWARD)
            s["out"] = [rows(H), empty(E, 2 * I, H), empty(E, H, I)]
        return
    if op == "route_bwd":
        s["out"] = [empty(T, E, dtype=torch.float32)]
        return
    s["norm"] = tpg.make_norm(s["w"], EPS)
    if op == "prenorm":
        s["out"] = [empty(T, H) if c["bf16"] else None, empty(T, H, dtype=torch.float8_e4m3fn) if c["fp8"] else None,
                    empty(T, H // 128, dtype=torch.float32) if c["fp8"] else None]
    elif op == "prenorm_bwd":
        ws(tpg.MOE_WS_PRENORM_BACKWARD)
        s["out"] = [empty(T, H), empty(H, dtype=torch.float32)]
    else:
        kind = dict(none=tpg.MOE_GATE_NONE, channel=tpg.MOE_GATE_CHANNEL, token=tpg.MOE_GATE_TOKEN)[c["gate"]]
        s["residual"] = tpg.make_residual(s["res"], s["scale"], s["gate"], kind)
        if op == "combine":
            s["out"] = [empty(T, H)]
        else:
            ws(tpg.MOE_WS_COMBINE_NORM_BACKWARD)
            s["out"] = [rows(H), empty(T, k, dtype=torch.float32), empty(T, H), empty(H, dtype=torch.float32),
                        None if s["gate"] is None else torch.empty_like(s["gate"])]


def _own(s):
    import token_permute_grouped_amd as tpg

    op, p, o = s["case"]["op"], s["p"], s["out"]
    if op == "ffn":
        tpg.moe_grouped_ffn_train(s["x"], s["offsets"], s["weights"], p, o[0], o[1], s["ws"])
        return dict(gu=o[0], y=o[1])
    if op == "ffn_bwd":
        tpg.moe_grouped_ffn_backward(s["dy"], s["x"], s["gu"], s["offsets"], s["weights"], p, o[0], o[1], o[2], s["ws"])
        return dict(dx=o[0], dw1=o[1], dw2=o[2])
    if op == "prenorm":
        tpg.moe_prenorm(s["x"], s["norm"], p, o[0], o[1], o[2])
        return dict(xn=o[0], q=o[1], scale=o[2])
    if op == "prenorm_bwd":
        tpg.moe_prenorm_backward(s["dx_perm"], s["slot_row"], s["dxn"], s["dres"], s["x"], s["norm"], p, o[0], o[1],
                                 s["ws"])
        return dict(dx=o[0], dweight=o[1])
    if op == "combine":
        tpg.moe_combine_norm(s["y"], s["slot_row"], s["topk_w"], s["norm"], s["residual"], p, o[0])
        return dict(out=o[0])
    if op == "combine_bwd":
        tpg.moe_combine_norm_backward(s["dout"], s["y"], s["slot_row"], s["topk_w"], s["norm"], s["residual"], p,
                                      o[0], o[1], o[2], o[3], o[4], s["ws"])
        return dict(dy=o[0], dtopk_w=o[1], dres=o[2], dweight=o[3], dgate=o[4])
    tpg.moe_route_topk_backward(s["logits"], s["slot_drop"], s["dw"], p, o[0])
    return dict(dlogits=o[0])


# ------------------------------------------------------------------------------------------------ the plain forms
def _plain_ffn(s):
    c, b = s["case"], s["bounds"]
    gi, ui = _gate_rows(c["I"], c["il"], s["x"].device)
    y = torch.zeros_like(s["x"])
    gu = y.new_zeros(y.shape[0], 2 * c["I"])
    for e in range(c["E"]):  # ragged groups: one product for each expert that has rows
        if b[e + 1] > b[e]:
            a = s["x"][b[e]:b[e + 1]].float() @ s["w1"][e].float().T
            gu[b[e]:b[e + 1]] = a
            if c["clamp"]:
                a = a.clamp(-c["clamp"], c["clamp"])
            g, u = a[:, gi], a[:, ui]
            y[b[e]:b[e + 1]] = (g / (1 + torch.exp(-g)) * u) @ s["w2"][e].float().T
    return dict(gu=gu, y=y)


def _plain_ffn_bwd(s):
    c, b = s["case"], s["bounds"]
    gi, ui = _gate_rows(c["I"], c["il"], s["x"].device)
    dx, dw1, dw2 = torch.zeros_like(s["x"]), torch.zeros_like(s["w1"]), torch.zeros_like(s["w2"])
    for e in range(c["E"]):
        if b[e + 1] > b[e]:
            x, dy = s["x"][b[e]:b[e + 1]].float(), s["dy"][b[e]:b[e + 1]].float()
            a = s["gu"][b[e]:b[e + 1]].float()
            cl = a.clamp(-c["clamp"], c["clamp"]) if c["clamp"] else a
            g, u = cl[:, gi], cl[:, ui]
            sg = 1 / (1 + torch.exp(-g))
            dh = dy @ s["w2"][e].float()
            da = torch.empty_like(a)
            da[:, gi] = dh * u * sg * (1 + g * (1 - sg))
            da[:, ui] = dh * g * sg
            if c["clamp"]:
                da = da * (a.abs() <= c["clamp"])
            dx[b[e]:b[e + 1]] = da @ s["w1"][e].float()
            dw1[e] = da.T @ x
            dw2[e] = dy.T @ (g * sg * u)
    return dict(dx=dx, dw1=dw1, dw2=dw2)


def _plain_prenorm(s):
    c, x = s["case"], s["x"].float()
    n = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * s["w"].float()
    o = dict(xn=n.to(torch.bfloat16) if c["bf16"] else None, q=None, scale=None)
    if c["fp8"]:
        blk = n.reshape(c["T"], -1, 128)
        sc = blk.abs().amax(2) / 448
        sc = torch.where(sc == 0, 1.0, sc)
        o["scale"] = sc
        o["q"] = (blk / sc[:, :, None]).clamp(-448, 448).reshape(n.shape).to(torch.float8_e4m3fn)
    return o


def _rows(v, slot_row):
    """[T, k, H] rows of each slot in fp32, zero where the slot is dropped."""
    return torch.where((slot_row >= 0)[:, :, None], v[slot_row.clamp(min=0).long()].float(), 0.0)


def _plain_prenorm_bwd(s):
    x, w = s["x"].float(), s["w"].float()
    dn = _rows(s["dx_perm"], s["slot_row"]).sum(1)
    if s["dxn"] is not None:
        dn = dn + s["dxn"].float()
    r = torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
    a = dn * w
    dx = s["dres"].float() + r * a - x * r ** 3 * (a * x).mean(1, keepdim=True)
    return dict(dx=dx.to(torch.bfloat16), dweight=(dn * x * r).sum(0))


def _plain_combine(s):
    c = (_rows(s["y"], s["slot_row"]) * s["topk_w"][:, :, None]).sum(1)
    z = c * torch.rsqrt(c.square().mean(1, keepdim=True) + EPS) * s["w"].float()
    if s["gate"] is not None:
        z = z * (s["gate"] if s["case"]["gate"] == "channel" else s["gate"][:, None])
    return dict(out=(s["scale"] * s["res"].float() + z).to(torch.bfloat16))


def _plain_combine_bwd(s):
    kind, w, dout = s["case"]["gate"], s["w"].float(), s["dout"].float()
    y = _rows(s["y"], s["slot_row"])
    c = (y * s["topk_w"][:, :, None]).sum(1)
    r = torch.rsqrt(c.square().mean(1, keepdim=True) + EPS)
    dz, dgate = dout, None
    if kind != "none":
        dz = dout * (s["gate"] if kind == "channel" else s["gate"][:, None])
        dgate = (dout * c * r * w).sum(0 if kind == "channel" else 1)
    b = dz * w
    dc = r * b - c * r ** 3 * (b * c).mean(1, keepdim=True)
    dtopk_w = torch.where(s["slot_row"] >= 0, (dc[:, None, :] * y).sum(2), 0.0)
    live = s["slot_row"] >= 0
    dy = torch.zeros_like(s["y"])
    dy[s["slot_row"][live].long()] = (dc[:, None, :] * s["topk_w"][:, :, None]).to(torch.bfloat16)[live]
    return dict(dy=dy, dtopk_w=dtopk_w, dres=(s["scale"] * dout).to(torch.bfloat16), dweight=(dz * c * r).sum(0),
                dgate=dgate)


def _plain_route_bwd(s):
    k = s["case"]["k"]
    top, idx = torch.sort(s["logits"], dim=1, descending=True, stable=True)
    top, idx = top[:, :k], idx[:, :k]
    e = torch.exp(top - top[:, :1])
    w = e / e.sum(1, keepdim=True)
    d = torch.where(s["slot_drop"] != 0, 0.0, s["dw"])
    dl = torch.zeros_like(s["logits"])
    return dict(dlogits=dl.scatter_(1, idx, w * (d - (w * d).sum(1, keepdim=True))))


_PLAIN = dict(ffn=_plain_ffn, ffn_bwd=_plain_ffn_bwd, prenorm=_plain_prenorm, prenorm_bwd=_plain_prenorm_bwd,
              combine=_plain_combine, combine_bwd=_plain_combine_bwd, route_bwd=_plain_route_bwd)


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------ floors
def work(case):
    """Bytes and flops a pass cannot do without; live rows are T k (1 - drop) in expectation."""
    c, op = case, case["op"]
    T, H, E, k = c["T"], c.get("H", 0), c.get("E", 0), c.get("k", 0)
    R = T * k * (1 - c.get("drop", 0.0))
    if op in ("ffn", "ffn_bwd"):
        I = c["I"]
        used = min(E, max(1.0, R))  # experts with rows, at most
        wb = used * 3 * I * H * 2
        if op == "ffn":
            return dict(bytes=wb + R * (2 * H + 2 * I) * 2, flops=6 * R * H * I)
        return dict(bytes=wb + E * 3 * I * H * 2 + R * (3 * H + 2 * I) * 2, flops=12 * R * H * I)
    if op == "prenorm":
        out = (2 if c["bf16"] else 0) + (1 + 4 / 128 if c["fp8"] else 0)
        return dict(bytes=T * H * (2 + out) + 2 * H, flops=4 * T * H)
    if op == "prenorm_bwd":
        return dict(bytes=2 * H * (R + T * (3 + (1 if c["router"] else 0))) + 6 * H + 4 * T * k,
                    flops=H * (R + 8 * T))
    if op == "combine":
        return dict(bytes=2 * H * (R + 2 * T) + 6 * H + 8 * T * k, flops=H * (2 * R + 6 * T))
    if op == "combine_bwd":
        return dict(bytes=2 * H * (2 * R + 2 * T) + 10 * H + 12 * T * k, flops=H * (5 * R + 12 * T))
    return dict(bytes=8 * T * E + 5 * T * k, flops=8 * T * k + T * E)


# ------------------------------------------------------------------------------------------------ the definition in fp64
def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    f64 = {n: v.double() for n, v in s.items() if torch.is_tensor(v) and v.is_floating_point() and n not in ("w1", "w2")}
    if op in ("ffn", "ffn_bwd"):
        return _exact_ffn(c, s, f64)
    if op == "route_bwd":
        order = s["logits"].argsort(dim=1, descending=True, stable=True)[:, :c["k"]]
        w = torch.softmax(f64["logits"].gather(1, order), dim=1)
        d = f64["dw"].masked_fill(s["slot_drop"].bool(), 0)
        jac = torch.diag_embed(w) - w[:, :, None] * w[:, None, :]
        return dict(dlogits=torch.zeros_like(f64["logits"]).scatter(1, order, torch.matmul(jac, d[:, :, None])[:, :, 0]))
    if op == "prenorm":
        n = f64["x"] / torch.sqrt((f64["x"] ** 2).mean(-1, keepdim=True) + EPS) * f64["w"]
        sc = n.abs().reshape(c["T"], -1, 128).max(-1)[0] / 448
        sc[sc == 0] = 1
        q = n / sc.repeat_interleave(128, 1)
        return dict(xn=n if c["bf16"] else None, q=q if c["fp8"] else None, scale=sc if c["fp8"] else None)
    rows = s["slot_row"].long()
    if op == "prenorm_bwd":
        padded = torch.cat([f64["dx_perm"], f64["dx_perm"].new_zeros(1, c["H"])])
        rows = torch.where(rows < 0, c["T"] * c["k"], rows)
        dn = f64["dxn"].clone() if c["router"] else torch.zeros_like(f64["x"])
        for j in range(c["k"]):
            dn += padded[rows[:, j]]
        dx, dweight = _rms_gradient(f64["x"], f64["w"], dn)
        return dict(dx=dx + f64["dres"], dweight=dweight)
    live = rows >= 0
    pick = rows.clamp(min=0)
    comb = torch.zeros_like(f64["res"])
    for j in range(c["k"]):
        comb += (f64["topk_w"][:, j] * live[:, j])[:, None] * f64["y"][pick[:, j]]
    gate = torch.ones((), dtype=torch.float64, device=comb.device)
    if c["gate"] != "none":
        gate = f64["gate"][None, :] if c["gate"] == "channel" else f64["gate"][:, None]
    normed = comb / torch.sqrt((comb ** 2).mean(-1, keepdim=True) + EPS)
    if op == "combine":
        return dict(out=s["scale"] * f64["res"] + gate * (normed * f64["w"]))
    dcomb, dweight = _rms_gradient(comb, f64["w"], gate * f64["dout"])
    dgate = None
    if c["gate"] != "none":
        dgate = (f64["dout"] * normed * f64["w"]).sum(0 if c["gate"] == "channel" else 1)
    dy = torch.zeros_like(f64["y"])
    dtw = torch.zeros_like(f64["topk_w"])
    for j in range(c["k"]):
        m = live[:, j]
        dy[rows[m, j]] = dcomb[m] * f64["topk_w"][m, j:j + 1]
        dtw[m, j] = (dcomb[m] * f64["y"][rows[m, j]]).sum(1)
    return dict(dy=dy, dtopk_w=dtw, dres=s["scale"] * f64["dout"], dweight=dweight, dgate=dgate)


def _rms_gradient(v, w, dn):
    """Gradients of n = v / sqrt(mean(v^2) + eps) * w with respect to v and w."""
    root = torch.sqrt((v ** 2).mean(-1, keepdim=True) + EPS)
    hat = v / root
    t = dn * w
    return (t - hat * (t * hat).mean(-1, keepdim=True)) / root, (dn * hat).sum(0)


def _exact_ffn(c, s, f64):
    I, il, lim = c["I"], c["il"], c["clamp"] or math.inf
    R, dev = s["x"].shape[0], s["x"].device
    perm = torch.arange(2 * I, device=dev)  # perm[stored row] = row of [gate | up]
    if il:
        perm = perm.reshape(2, I // il, il).transpose(0, 1).reshape(-1)
    inv = torch.argsort(perm)
    out = [torch.zeros(R, 2 * I, dtype=torch.float64, device=dev) if c["op"] == "ffn" else None,
           torch.zeros(R, c["H"], dtype=torch.float64, device=dev)]
    if c["op"] == "ffn_bwd":
        dw1, dw2 = (torch.zeros(w.shape, dtype=torch.float64, device=dev) for w in (s["w1"], s["w2"]))
    for e in range(c["E"]):
        rows = slice(s["bounds"][e], s["bounds"][e + 1])
        if rows.start == rows.stop:
            continue
        w1, w2 = s["w1"][e].double(), s["w2"][e].double()
        a = f64["x"][rows].matmul(w1.T) if c["op"] == "ffn" else f64["gu"][rows]
        gate, up = a[:, inv].chunk(2, dim=1)
        inside = [(v >= -lim) & (v <= lim) for v in (gate, up)]
        gate, up = gate.clip(-lim, lim), up.clip(-lim, lim)
        sig = torch.sigmoid(gate)
        h = gate * sig * up
        if c["op"] == "ffn":
            out[0][rows], out[1][rows] = a, h.matmul(w2.T)
            continue
        dy = f64["dy"][rows]
        dh = dy.matmul(w2)
        dgate = dh * up * (sig + gate * sig * (1 - sig)) * inside[0]
        da = torch.cat([dgate, dh * gate * sig * inside[1]], 1)[:, perm]
        out[1][rows] = da.matmul(w1)
        dw1[e] = da.T.contiguous().matmul(f64["x"][rows])
        dw2[e] = dy.T.contiguous().matmul(h)
    return dict(gu=out[0], y=out[1]) if c["op"] == "ffn" else dict(dx=out[1], dw1=dw1, dw2=dw2)
