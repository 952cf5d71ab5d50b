"""16-bit results of the experts' products and of the product with an epilogue:
as near as the fp8 instruction allows (what it cuts has a known spread), value
by value and as a whole, so that an element of K left out or taken twice shows."""
import numpy as np
import pytest

from oracle import fp8, moe
from parity_utils import gq, log, torch_mod
from test_expert_gpu import HALF, _check, _choice, _each, _experts, _matrix, _np, _randn, _t, _values

pytestmark = pytest.mark.gpu

SLOPE = 1.13   # of the activations, at most


def _whole(got, ref, spread, bound, dtype, what):
    """The error's norm: spreads and roundings (a rounding's mean square is a
    third of its largest) in squares, the fp32 part at its worst."""
    err = np.linalg.norm(_np(got) - ref)
    limit = np.sqrt(np.sum(spread ** 2 + (np.abs(ref) * HALF[dtype]) ** 2 / 3)) + np.linalg.norm(bound)
    log(f"{what}: error norm {err / np.linalg.norm(ref):.3e} of the result's, limit {limit / np.linalg.norm(ref):.3e}")
    assert err <= limit, what


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K,act", [(1, 1000, 4096, None), (37, 300, 4000, "silu"), (70, 500, 2704, None), (300, 4096, 640, "gelu"),
                                       (600, 2000, 2709, "gelu_tanh"), (2311, 4100, 400, None)])
def test_linear_16_bits(M, N, K, act, dtype):
    a, b = _matrix(M, K, 1, 1), _matrix(N, K, 128, 2, 0.05)
    bias, res = _randn(N, seed=3, std=0.5).cuda(), _randn(M, N, seed=4).to(_t(dtype)).cuda()
    ref, bound = moe.linear(_values(a), _values(b), _np(bias), act, _np(res))
    spread = (SLOPE if act else 1.0) * fp8.dropped_spread(_values(a), _values(b))
    C = gq().fp8_linear(a, b, bias, act, res, out_dtype=_t(dtype))
    what = f"LINEAR {M}x{N}x{K} {act} {dtype} tight"
    _check(C, ref, bound(False) + 8 * spread, dtype, what)
    _whole(C, ref, spread, bound(False), dtype, what)


GATED = [(1, 8, 2, 640, 2704), (30, 64, 8, 300, 1000), (61, 16, 4, 500, 2100), (700, 2, 1, 300, 2704), (1000, 8, 2, 640, 400)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,E,k,N,K", GATED)
def test_expert_gated_16_bits(T, E, k, N, K, dtype):
    act = ["silu", "gelu", "gelu_tanh"][T % 3]
    a, g_, u = _matrix(T, K, 1, 1), _experts(E, N, K, 2), _experts(E, N, K, 3)
    ids, w = _choice(T, E, k, T + E)
    r = gq().moe_plan(ids, w, E)
    A, G, U, I = _values(a), _each(g_), _each(u), ids.cpu().numpy()
    ref, bound = moe.gated(A, I, G, U, act)
    offsets, order = moe.plan(I, E)
    most, spread = np.zeros_like(ref), np.zeros_like(ref)
    for e in range(E):
        at, s = slice(offsets[e], offsets[e + 1]), order[offsets[e]:offsets[e + 1]] // k
        x = (A[0][s], A[1][s])
        cg, cu = np.abs(fp8.activation(fp8.matmul(x, G[e])[0], act)), np.abs(fp8.matmul(x, U[e])[0])
        sg, su = SLOPE * fp8.dropped_spread(x, G[e]), fp8.dropped_spread(x, U[e])
        most[at] = 8 * sg * (cu + 8 * su) + 8 * cg * su
        spread[at] = np.sqrt((sg * cu) ** 2 + (cg * su) ** 2 + (sg * su) ** 2)
    h = gq().fp8_expert_gated_gemm(a, r, g_, u, act, out_dtype=_t(dtype))
    what = f"GATED {T}x{E}x{k} {N}x{K} {act} {dtype} tight"
    _check(h, ref, bound + most, dtype, what)
    _whole(h, ref, spread, bound, dtype, what)


BACK = [(10, 8, 2, 640, 2704), (16, 16, 8, 300, 1000), (61, 64, 8, 500, 520), (300, 8, 2, 515, 2100), (700, 2, 1, 300, 2704),
        (1400, 4, 1, 515, 1000), (600, 4, 4, 700, 1100)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,E,k,N,K", BACK)
def test_expert_gemm_16_bits(T, E, k, N, K, dtype):
    h, d = _matrix(T * k, K, 1, 1), _experts(E, N, K, 2)
    ids, w = _choice(T, E, k, T + E)
    r = gq().moe_plan(ids, w, E)
    H, D, I, W = _values(h), _each(d), ids.cpu().numpy(), _np(w).reshape(-1)
    res = _randn(T, N, seed=5).to(_t(dtype)).cuda()
    half = dtype == "bf16" and T > 16
    ref, exact = moe.combined(H, I, _np(w), D, _np(res))
    most = moe.combined(H, I, _np(w), D, _np(res), half_terms=half)[1]
    offsets, order = moe.plan(I, E)
    cut, rounded = np.zeros((T, N)), np.zeros((T, N))
    for e in range(E):
        at, s = slice(offsets[e], offsets[e + 1]), order[offsets[e]:offsets[e + 1]]
        x, ws = (H[0][at], H[1][at]), W[s][:, None]
        np.add.at(cut, s // k, (ws * fp8.dropped_spread(x, D[e])) ** 2)
        if half:
            np.add.at(rounded, s // k, (ws * fp8.matmul(x, D[e])[0] * 2.0 ** -11) ** 2 / 3)
    y = gq().fp8_expert_gemm(h, r, d, res, out_dtype=_t(dtype))
    what = f"BACK {T}x{E}x{k} {N}x{K} {dtype} tight"
    _check(y, ref, most + 8 * np.sqrt(cut), dtype, what)
    _whole(y, ref, np.sqrt(cut + rounded), exact, dtype, what)
