"""Host-side checks of the norm and training entry points (no GPU needed): every call below fails a check, or
has nothing to do, and returns before any HIP call."""
import ctypes

import pytest
import torch

import token_permute_grouped_amd as tpg

F = 0x1000     # never dereferenced
ODD = 0x1008   # not 16-byte aligned
BIG = 1 << 40
NULL, SHAPE, UNSUPPORTED, WORKSPACE = tpg.MOE_ERR_NULL, tpg.MOE_ERR_SHAPE, tpg.MOE_ERR_UNSUPPORTED, tpg.MOE_ERR_WORKSPACE


def _p(**kw):
    base = dict(T=64, H=128, I=256, E=8, k=2, prec=0, glu_interleave=0, swiglu_clamp=0.0)
    base.update(kw)
    return tpg.Problem(**base)


W = tpg.Weights(F, None, None, F, None, None)


def _refused(status, fn, *args):
    with pytest.raises(tpg.MoeError) as e:
        fn(*args, stream=F)
    assert e.value.status == status, (fn.__name__, e.value)


def _calls(p, norm=None, res=None, w=W):
    """every entry point with arguments that pass its checks, but for those given"""
    return [
        (tpg.moe_prenorm, [F, norm, p, F, F, F]),
        (tpg.moe_prenorm_backward, [F, F, F, F, F, norm, p, F, None, F, BIG]),
        (tpg.moe_combine_norm, [F, F, F, norm, res, p, F]),
        (tpg.moe_combine_norm_backward, [F, F, F, F, norm, res, p, F, F, None, None, None, F, BIG]),
        (tpg.moe_forward_norm, [F, None, F, None, w, norm, res, p, F, F, BIG]),
        (tpg.moe_route_topk_backward, [F, None, F, p, F]),
        (tpg.moe_grouped_ffn_train, [F, F, w, p, F, F, F, BIG]),
        (tpg.moe_grouped_ffn_backward, [F, F, F, F, w, p, F, F, F, F, BIG]),
    ]


@pytest.mark.parametrize("kw,status", [(dict(T=-1), SHAPE), (dict(H=100), SHAPE), (dict(I=64), SHAPE),
                                       (dict(E=257), SHAPE), (dict(k=9), SHAPE), (dict(prec=7), UNSUPPORTED),
                                       (dict(T=2 ** 30), SHAPE), (dict(swiglu_clamp=-1.0), UNSUPPORTED)])
def test_bad_problems(kw, status):
    for fn, args in _calls(_p(**kw)):
        _refused(status, fn, *args)
    for which in (tpg.MOE_WS_FFN_BACKWARD, tpg.MOE_WS_PRENORM_BACKWARD, tpg.MOE_WS_COMBINE_NORM_BACKWARD):
        assert tpg.moe_call_workspace_bytes(_p(**kw), which) == 0


@pytest.mark.parametrize("norm", [tpg.Norm(F, 0.0), tpg.Norm(F, -1e-6), tpg.Norm(F, float("nan")),
                                  tpg.Norm(F, float("inf")), tpg.Norm(F, 1e-40), tpg.Norm(ODD, 1e-6)])
def test_bad_norms(norm):
    for fn, args in _calls(_p(), norm=norm)[:5]:
        _refused(UNSUPPORTED, fn, *args)


@pytest.mark.parametrize("res,status", [(tpg.Residual(F, 1.0, F, 3), UNSUPPORTED), (tpg.Residual(F, 1.0, F, -1), UNSUPPORTED),
                                        (tpg.Residual(F, 1.0, None, tpg.MOE_GATE_TOKEN), NULL),
                                        (tpg.Residual(F, float("nan"), None, 0), UNSUPPORTED),
                                        (tpg.Residual(F, float("inf"), None, 0), UNSUPPORTED),
                                        (tpg.Residual(ODD, 1.0, None, 0), UNSUPPORTED),
                                        (tpg.Residual(F, 1.0, ODD, tpg.MOE_GATE_CHANNEL), UNSUPPORTED)])
def test_bad_residuals(res, status):
    for fn, args in _calls(_p(), res=res)[2:5]:
        _refused(status, fn, *args)


@pytest.mark.parametrize("call,missing", [(0, (0,)), (0, (3, 4, 5)), (0, (4,)), (0, (5,)), (1, (0, 2)), (1, (1,)), (1, (7,)),
                                          (2, (0,)), (2, (1,)), (2, (2,)), (2, (6,)), (3, (0,)), (3, (1,)), (3, (2,)),
                                          (3, (3,)), (3, (7,)), (4, (0,)), (4, (2,)), (4, (8,)), (4, (9,)), (5, (0,)),
                                          (5, (2,)), (5, (4,)), (6, (0,)), (6, (1,)), (6, (4,)), (6, (5,)), (6, (6,)),
                                          (7, (0,)), (7, (1,)), (7, (2,)), (7, (3,)), (7, (6, 7, 8)), (7, (9,))])
def test_missing_arrays(call, missing):
    fn, args = _calls(_p())[call]
    _refused(NULL, fn, *[None if i in missing else a for i, a in enumerate(args)])


@pytest.mark.parametrize("call,odd", [(0, 0), (0, 3), (0, 4), (1, 0), (1, 2), (1, 3), (1, 7), (2, 0), (2, 6), (3, 0), (3, 1),
                                      (3, 7), (4, 8), (6, 0), (6, 4), (6, 5), (6, 6), (7, 0), (7, 1), (7, 2), (7, 6), (7, 7),
                                      (7, 8), (7, 9)])
def test_misaligned_rows(call, odd):
    fn, args = _calls(_p())[call]
    _refused(UNSUPPORTED, fn, *[ODD if i == odd else a for i, a in enumerate(args)])


def test_misaligned_sums_over_tokens():
    p, norm, res = _p(), tpg.Norm(F, 1e-6), tpg.Residual(None, 1.0, F, tpg.MOE_GATE_CHANNEL)
    _refused(UNSUPPORTED, tpg.moe_prenorm_backward, F, F, None, None, F, norm, p, F, ODD, F, BIG)
    _refused(UNSUPPORTED, tpg.moe_prenorm_backward, F, F, None, None, F, norm, p, F, F, ODD, BIG)
    for dw, dg, ws in ((ODD, F, F), (F, ODD, F), (F, F, ODD)):
        _refused(UNSUPPORTED, tpg.moe_combine_norm_backward, F, F, F, F, norm, res, p, F, F, None, dw, dg, ws, BIG)


def test_gradients_of_what_is_not_there():
    p, norm, res = _p(), tpg.Norm(F, 1e-6), tpg.Residual(None, 1.0, None, 0)
    _refused(UNSUPPORTED, tpg.moe_prenorm_backward, F, F, None, None, F, None, p, F, F, F, BIG)
    back = lambda n, r, dres, dw, dg: (F, F, F, F, n, r, p, F, F, dres, dw, dg, F, BIG)  # noqa: E731
    _refused(UNSUPPORTED, tpg.moe_combine_norm_backward, *back(None, None, None, F, None))
    _refused(UNSUPPORTED, tpg.moe_combine_norm_backward, *back(norm, None, F, None, None))
    _refused(UNSUPPORTED, tpg.moe_combine_norm_backward, *back(norm, res, F, None, None))
    _refused(UNSUPPORTED, tpg.moe_combine_norm_backward, *back(norm, res, None, None, F))


def test_workspaces():
    p, norm = _p(T=5000, H=640), tpg.Norm(F, 1e-6)
    res = tpg.Residual(F, 1.0, F, tpg.MOE_GATE_CHANNEL)
    for which, fn, args in [
        (tpg.MOE_WS_FFN_BACKWARD, tpg.moe_grouped_ffn_backward, [F, F, F, F, W, p, F, F, F]),
        (tpg.MOE_WS_GROUPED_FFN, tpg.moe_grouped_ffn_train, [F, F, W, p, F, F]),
        (tpg.MOE_WS_PRENORM_BACKWARD, tpg.moe_prenorm_backward, [F, F, None, None, F, norm, p, F, F]),
        (tpg.MOE_WS_COMBINE_NORM_BACKWARD, tpg.moe_combine_norm_backward, [F, F, F, F, norm, res, p, F, F, F, F, None]),
        (tpg.MOE_WS_COMBINE_NORM_BACKWARD, tpg.moe_combine_norm_backward, [F, F, F, F, norm, res, p, F, F, F, None, F]),
        (tpg.MOE_WS_FORWARD, tpg.moe_forward_norm, [F, None, F, None, W, norm, res, p, F]),
    ]:
        n = tpg.moe_call_workspace_bytes(p, which)
        assert n > 0
        _refused(WORKSPACE, fn, *args, F, n - 1)
        _refused(NULL, fn, *args, None, n)
    # gradients of the W4A8 layers' FFN do not exist; its norms' do
    w4 = _p(H=256, prec=tpg.MOE_PREC_W4A8)
    assert tpg.moe_call_workspace_bytes(w4, tpg.MOE_WS_FFN_BACKWARD) == 0
    assert tpg.moe_call_workspace_bytes(w4, tpg.MOE_WS_PRENORM_BACKWARD) > 0
    full = tpg.Weights(*[F] * 6)
    _refused(UNSUPPORTED, tpg.moe_grouped_ffn_train, F, F, full, w4, F, F, F, BIG)
    _refused(UNSUPPORTED, tpg.moe_grouped_ffn_backward, F, F, F, F, full, w4, F, F, F, F, BIG)
    one = _p(H=1024, I=1024, prec=tpg.MOE_PREC_W4A8, flags=tpg.MOE_FLAG_SINGLE_LAUNCH)
    _refused(UNSUPPORTED, tpg.moe_forward_norm, F, None, F, F, full, norm, None, one, F, F, BIG)


def test_no_tokens_is_nothing_to_do():
    p = _p(T=0)
    w = tpg.Weights(*[None] * 6)
    for fn, args in _calls(p, w=w):
        fn(*[a if isinstance(a, ctypes.Structure) else None for a in args[:-1]], *([0] if args[-1] == BIG else [None]), stream=F)


def test_tensors_are_checked():
    p = _p(T=4)
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    for bad in (torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(128, 4, dtype=torch.bfloat16).T):
        with pytest.raises(ValueError):
            tpg.moe_prenorm(bad, None, p, x, stream=F)
    with pytest.raises(ValueError):
        tpg.moe_prenorm(x, tpg.make_norm(torch.zeros(64, dtype=torch.bfloat16), 1e-6), p, x, stream=F)
    gate = torch.zeros(4)
    with pytest.raises(ValueError):
        tpg.moe_combine_norm(F, F, F, None, tpg.make_residual(None, 1.0, gate, tpg.MOE_GATE_CHANNEL), p, F, stream=F)
    with pytest.raises(ValueError, match="not on a GPU"):
        tpg.moe_prenorm(x, None, p, x, stream=F)
