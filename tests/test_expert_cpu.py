"""The experts' calls without a GPU: pins of the oracle, and every argument
check of the C ABI and of the binding."""
import numpy as np
import pytest
import torch

import post_weight_quantization_16_amd as g
from oracle import moe
from post_weight_quantization_16_amd import _native as n

FAKE = 1 << 20   # never dereferenced: every call below returns before any HIP call
E4 = torch.float8_e4m3fn


# ---------------------------------------------------------------- oracle
def test_route_closed_forms():
    x = np.log(np.array([[1.0, 2.0, 4.0, 1.0]]))
    ids, w = moe.route(x, 2)
    assert ids.tolist() == [[2, 1]] and np.allclose(w, [[2 / 3, 1 / 3]])
    ids, w = moe.route(x, 3, renormalize=False, scale=8.0)
    assert ids.tolist() == [[2, 1, 0]] and np.allclose(w, [[4, 2, 1]])          # ties to the lowest index
    ids, w = moe.route(x, 1, bias=[0, 0, -1, 0], renormalize=False)
    assert ids.tolist() == [[1]] and np.allclose(w, [[0.25]])                   # the weight is without the bias
    ids, w = moe.route(x, 1, groups=2, top_groups=1, group_top=2)
    assert ids.tolist() == [[2]]
    y = np.array([[3.0, -9.0, 2.0, 2.0]])
    assert moe.route(y, 1, "sigmoid", groups=2, top_groups=1, group_top=1)[0].tolist() == [[0]]
    assert moe.route(y, 1, "sigmoid", groups=2, top_groups=1, group_top=2)[0].tolist() == [[2]]
    ids, w = moe.route([[-np.inf, 0, -np.inf, -np.inf], [0, np.nan, 0, 0], [0, 0, 0, 0]], 2, mask=[1, 1, 0])
    assert ids.tolist() == [[1, -1], [0, 1], [-1, -1]]
    assert w[0].tolist() == [1, 0] and np.isnan(w[1]).all() and w[2].tolist() == [0, 0]


def test_plan_closed_form():
    offsets, order = moe.plan([[2, 0], [0, -1], [2, 7]], 3)
    assert offsets.tolist() == [0, 2, 2, 4] and order.tolist() == [1, 2, 0, 4, -1, -1]


def test_products_of_experts():
    rng = np.random.default_rng(0)
    mats = lambda c, r, k, b: [(rng.integers(-8, 9, (r, k)) / 4.0, np.ones((-(-r // b), 1))) for _ in range(c)]
    (a,), gate, up = mats(1, 3, 20, 1), mats(4, 5, 20, 128), mats(4, 5, 20, 128)
    ids = np.array([[1, 3], [3, -1], [0, 1]])
    h, _ = moe.gated(a, ids, gate, up, "silu")
    c = a[0][2] @ gate[1][0].T
    assert h.shape == (5, 5) and np.allclose(h[2], c / (1 + np.exp(-c)) * (a[0][2] @ up[1][0].T))
    (q,), down = mats(1, 5, 20, 1), mats(4, 6, 20, 128)
    w = np.array([[0.5, 2.0], [1.0, 9.0], [3.0, 1.0]])
    y, _ = moe.combined(q, ids, w, down, np.ones((3, 6)))
    assert np.allclose(y[0], 0.5 * q[0][1] @ down[1][0].T + 2.0 * q[0][3] @ down[3][0].T + 1)
    assert np.allclose(y[1], q[0][4] @ down[3][0].T + 1)


# ---------------------------------------------------------------- C ABI
def test_linear_refusals():
    f = n.lib().gptq_fp8_linear

    def call(A=FAKE, sa=FAKE, M=4, K=256, lda=256, B=FAKE, sb=FAKE, N=64, ldb=256, bias=None, bdt=n.F32, act=-1, R=None,
             ldr=0, C=FAKE, dt=n.BF16, ldc=64, q=None, ldq=0, s=None, ws=None, wsb=0):
        return f(A, sa, M, K, lda, B, sb, N, ldb, bias, bdt, act, R, ldr, C, dt, ldc, q, ldq, s, ws, wsb, None)

    other = FAKE + (1 << 16)
    codes = dict(C=None, q=FAKE, ldq=64, s=FAKE)
    for kw in [dict(A=None), dict(sa=None), dict(B=None), dict(sb=None), dict(C=None), dict(M=-1), dict(K=0), dict(N=0),
               dict(K=70000, lda=70000, ldb=70000), dict(lda=255), dict(ldb=255), dict(ldc=63), dict(dt=5), dict(act=3), dict(act=-2),
               dict(bias=FAKE, bdt=9), dict(bias=FAKE + 1), dict(bias=FAKE + 1, bdt=n.BF16), dict(R=other, ldr=63), dict(R=other + 1, ldr=64),
               dict(R=FAKE, ldr=65), dict(sa=FAKE + 2), dict(C=FAKE + 1), dict(q=FAKE), dict(q=FAKE, ldq=64, s=FAKE),
               dict(codes, s=None), dict(codes, ldq=63), dict(codes, R=other, ldr=64), dict(codes, s=FAKE + 1)]:
        assert call(**kw) == n.ERR_INVALID_ARG, kw
        assert n.last_error()
    need = n.lib().gptq_workspace_bytes(n.WS_FP8_LINEAR, 64, 256, 4, None)
    assert need > 0 and need % 256 == 0
    assert call(ws=FAKE, wsb=need - 1) == n.ERR_WORKSPACE and call(ws=FAKE + 8, wsb=need) == n.ERR_WORKSPACE
    assert call(A=None, sa=None, C=None, M=0) == n.OK
    ws = n.lib().gptq_workspace_bytes
    assert ws(n.WS_FP8_LINEAR, 0, 256, 4, None) == 0 and ws(n.WS_FP8_LINEAR, 64, 256, 0, None) == 256


def test_route_and_plan_refusals():
    f, p = n.lib().gptq_moe_route, n.lib().gptq_moe_plan

    def call(X=FAKE, dt=n.F32, T=4, E=64, ld=64, bias=None, mask=None, sc=0, k=8, ng=1, tg=1, gt=1, rn=1, scale=1.0,
             ids=FAKE, w=FAKE, off=FAKE, order=FAKE, ws=None, wsb=0):
        return f(X, dt, T, E, ld, bias, mask, sc, k, ng, tg, gt, rn, scale, ids, w, off, order, ws, wsb, None)

    for kw in [dict(X=None), dict(ids=None), dict(w=None), dict(off=None), dict(order=None), dict(dt=4), dict(T=-1), dict(T=(1 << 24) + 1),
               dict(E=0), dict(E=1025, ld=1025), dict(ld=63), dict(sc=2), dict(sc=-1), dict(k=0), dict(k=65), dict(E=4, k=5),
               dict(E=128, ld=128, k=65), dict(ng=0), dict(ng=17), dict(ng=3), dict(ng=32), dict(ng=8, tg=0), dict(ng=8, tg=9),
               dict(ng=16, tg=1), dict(gt=0), dict(gt=3), dict(rn=2), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(X=FAKE + 2), dict(bias=FAKE + 2), dict(ids=FAKE + 1), dict(order=FAKE + 2), dict(T=1 << 24, E=128, ld=128, k=64 + 1)]:
        assert call(**kw) == n.ERR_INVALID_ARG, kw
    size = n.lib().gptq_expert_workspace_bytes
    need = size(n.WS_MOE, 1000, 8, 64, 0, 0)
    assert need >= 512 and need % 256 == 0
    assert call(T=1000) == n.ERR_WORKSPACE and call(T=1000, ws=FAKE, wsb=need - 1) == n.ERR_WORKSPACE
    assert call(T=1000, ws=FAKE + 4, wsb=need) == n.ERR_WORKSPACE
    assert call(T=0, X=None, ids=None, w=None, off=None, order=None) == n.OK
    plan = lambda ids=FAKE, T=1000, k=8, E=64, off=FAKE, order=FAKE, ws=FAKE, wsb=1 << 30: p(ids, T, k, E, off, order, ws, wsb, None)
    for kw in [dict(ids=None), dict(off=None), dict(order=None), dict(T=-1), dict(k=0), dict(k=65), dict(E=0), dict(E=1025), dict(ids=FAKE + 2)]:
        assert plan(**kw) == n.ERR_INVALID_ARG, kw
    assert plan(ws=None) == n.ERR_WORKSPACE and plan(wsb=need - 1) == n.ERR_WORKSPACE


def test_expert_product_refusals():
    f, h = n.lib().gptq_fp8_expert_gated_gemm, n.lib().gptq_fp8_expert_gemm

    def gated(A=FAKE, sa=FAKE, T=4, K=256, lda=256, k=2, off=FAKE, order=FAKE, E=8, G=FAKE, sg=FAKE, ldg=256, ng=1 << 14, U=FAKE,
              su=FAKE, ldu=256, nu=1 << 14, N=64, act=0, C=FAKE, dt=n.BF16, ldc=64, q=None, ldq=0, s=None, ws=None, wsb=0):
        return f(A, sa, T, K, lda, k, off, order, E, G, sg, ldg, ng, U, su, ldu, nu, N, act, C, dt, ldc, q, ldq, s, ws, wsb, None)

    codes = dict(C=None, q=FAKE, ldq=64, s=FAKE)
    for kw in [dict(A=None), dict(sa=None), dict(G=None), dict(sg=None), dict(U=None), dict(su=None), dict(off=None), dict(order=None),
               dict(T=-1), dict(K=0), dict(K=70000, lda=70000, ldg=70000, ldu=70000), dict(lda=255), dict(ldg=255), dict(ldu=255), dict(k=0),
               dict(k=9), dict(E=0), dict(E=1025), dict(ng=-1), dict(nu=-1), dict(N=0), dict(act=3), dict(act=-1), dict(C=None), dict(dt=7),
               dict(ldc=63), dict(q=FAKE, ldq=64, s=FAKE), dict(codes, s=None), dict(codes, ldq=63), dict(codes, s=FAKE + 2),
               dict(C=FAKE + 1), dict(sa=FAKE + 1), dict(off=FAKE + 2), dict(order=FAKE + 1)]:
        assert gated(**kw) == n.ERR_INVALID_ARG, kw
    size = n.lib().gptq_expert_workspace_bytes
    need = size(n.WS_EXPERT_GATED, 4, 2, 8, 64, 256)
    assert need and need % 256 == 0
    assert gated(ws=FAKE, wsb=need - 1) == n.ERR_WORKSPACE and gated(ws=FAKE + 8, wsb=need) == n.ERR_WORKSPACE
    assert gated(T=0, A=None, C=None) == n.OK

    def back(H=FAKE, sh=FAKE, T=100, K=256, ldh=256, k=2, ids=FAKE, w=FAKE, off=FAKE, order=FAKE, E=8, D=FAKE, sd=FAKE, ldd=256,
             nd=1 << 14, N=64, R=None, ldr=0, C=FAKE, dt=n.BF16, ldc=64, ws=FAKE, wsb=1 << 30):
        return h(H, sh, T, K, ldh, k, ids, w, off, order, E, D, sd, ldd, nd, N, R, ldr, C, dt, ldc, ws, wsb, None)

    for kw in [dict(H=None), dict(sh=None), dict(ids=None), dict(w=None), dict(off=None), dict(order=None), dict(D=None), dict(sd=None),
               dict(C=None), dict(T=-1), dict(K=0), dict(ldh=255), dict(ldd=255), dict(nd=-1), dict(N=0), dict(ldc=63), dict(dt=3), dict(k=0),
               dict(E=1), dict(R=FAKE + 4096, ldr=63), dict(R=FAKE, ldr=70), dict(R=FAKE + 1, ldr=64), dict(w=FAKE + 2), dict(C=FAKE + 1)]:
        assert back(**kw) == n.ERR_INVALID_ARG, kw
    need = size(n.WS_EXPERT_GEMM, 100, 2, 8, 64, 256)
    assert need > 256
    assert back(ws=None) == n.ERR_WORKSPACE and back(wsb=need - 1) == n.ERR_WORKSPACE and back(ws=FAKE + 16) == n.ERR_WORKSPACE
    assert back(T=0, H=None, C=None, ws=None, wsb=0) == n.OK
    for which in (n.WS_MOE, n.WS_EXPERT_GATED, n.WS_EXPERT_GEMM):
        assert size(which, -1, 2, 8, 64, 256) == 0 and size(which, 4, 9, 8, 64, 256) == 0 and size(which, 4, 2, 0, 64, 256) == 0
    for T, N in [(1000, 1), (999, 2), (70, 3), (500, 130), (40, 4096)]:    # fp16 terms and their powers of two, or fp32 terms
        assert size(n.WS_EXPERT_GEMM, T, 2, 8, N, 256) >= max(8 * T * N, 2 * -(-2 * T * N // 8) * 8 + 8 * T * -(-N // 128))
    assert size(n.WS_EXPERT_GEMM, 4, 2, 8, 0, 256) == 0 and size(n.WS_EXPERT_GATED, 4, 2, 8, 64, 0) == 0 and size(99, 4, 2, 8, 64, 256) == 0


# ---------------------------------------------------------------- binding
def _m(rows, cols, br=1):
    return g.Fp8Matrix(torch.zeros(rows, cols, dtype=torch.uint8).view(E4), torch.ones(-(-rows // br), -(-cols // 128)), br)


def _x(e, rows, cols):
    return g.Fp8Experts(torch.zeros(e, rows, cols, dtype=torch.uint8).view(E4), torch.ones(e, -(-rows // 128), -(-cols // 128)))


def _r(T, k, E):
    return g.Routing(torch.zeros(T, k, dtype=torch.int32), torch.zeros(T, k), torch.zeros(E + 1, dtype=torch.int32),
                     torch.zeros(T * k, dtype=torch.int32))


def _bad(f, *a, **kw):
    with pytest.raises(ValueError):
        f(*a, **kw)


def test_binding_refuses():
    a, b = _m(4, 200), _m(60, 200, 128)
    bf = torch.bfloat16
    for kw in [dict(bias=torch.zeros(61)), dict(bias=torch.zeros(60, dtype=torch.float64)), dict(bias=torch.zeros(120)[::2]),
               dict(activation="relu"), dict(residual=torch.zeros(4, 60)), dict(residual=torch.zeros(4, 61, dtype=bf)),
               dict(out=torch.zeros(4, 60, dtype=bf), out_dtype=torch.float32), dict(out=torch.zeros(5, 60, dtype=bf)),
               dict(out_dtype=torch.float64), dict(out_dtype=E4, residual=torch.zeros(4, 60, dtype=bf)), dict(out=_m(5, 60)),
               dict(out=_m(4, 60), out_dtype=bf), dict()]:      # the last: tensors of the host
        _bad(g.fp8_linear, a, b, **kw)
    _bad(g.fp8_linear, _m(4, 201), b)
    _bad(g.fp8_linear, b, a)
    x = torch.zeros(4, 16)
    for kw in [dict(scores="relu"), dict(bias=torch.zeros(15)), dict(bias=torch.zeros(16, dtype=bf)), dict(mask=torch.ones(4)),
               dict(mask=torch.ones(5, dtype=torch.bool)), dict(ws=torch.zeros(4)), dict()]:
        _bad(g.moe_route, x, 2, **kw)
    _bad(g.moe_route, x.double(), 2)
    _bad(g.moe_route, x.t(), 2)
    ids, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    for i, v in [(ids.long(), w), (ids, w[:, :1]), (ids, w.double()), (ids.reshape(-1), w), (ids.t(), w.t()), (ids, w)]:
        _bad(g.moe_plan, i, v, 8)
    r = _r(4, 2, 8)
    e = _x(8, 60, 200)
    f = g.fp8_expert_gated_gemm
    for args in [(_m(4, 201), r, e, e), (_m(5, 200), r, e, e), (_m(4, 200, 128), r, e, e), (a, _r(4, 2, 7), e, e), (a, r, e, _x(8, 61, 200)),
                 (a, r, e, _x(7, 60, 200)), (a, r, e, e, "relu"), (a, r, e, e)]:
        _bad(f, *args)
    broken = _r(4, 2, 8)
    broken.order = broken.order.long()
    _bad(f, a, broken, e, e)
    _bad(f, a, r, g.Fp8Experts(e.codes.transpose(1, 2), e.scales), e)
    _bad(f, a, r, g.Fp8Experts(e.codes, e.scales[:, :, :1]), e)
    _bad(f, a, r, g.Fp8Experts(e.codes[0], e.scales), e)
    for kw in [dict(out=_m(7, 60)), dict(out=_m(8, 60), out_dtype=bf), dict(out=torch.zeros(8, 61, dtype=bf)), dict(out_dtype=torch.float64)]:
        _bad(f, a, r, e, e, **kw)
    f, h = g.fp8_expert_gemm, _m(8, 200)
    for args in [(_m(7, 200), r, e), (_m(8, 201), r, e), (h, _r(3, 2, 8), e), (h, r, _x(9, 60, 200)), (h, r, e, torch.zeros(4, 60)), (h, r, e)]:
        _bad(f, *args)
    _bad(f, h, r, e, out=torch.zeros(4, 61, dtype=bf))
    _bad(g.fp8_quantize_experts, torch.zeros(4, 8))
    _bad(g.fp8_quantize_experts, torch.zeros(2, 4, 8), out=_x(2, 4, 9))
