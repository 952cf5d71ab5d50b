"""Terms of the experts' sums for bf16 results: fp16 on their way, whatever the
size of the codes and scales that they come from."""
import numpy as np
import pytest

from oracle import moe
from parity_utils import gq, log, torch_mod
from test_expert_gpu import HALF, _check, _choice, _each, _experts, _matrix, _np, _randn, _t, _values

pytestmark = pytest.mark.gpu


def _signs(rows, cols, seed, some=1.0):
    """±1, a share of `some` of them, the others 0."""
    torch = torch_mod()
    gen = torch.Generator().manual_seed(seed)
    x = torch.randint(0, 2, (rows, cols), generator=gen) * 2.0 - 1.0
    return x * (torch.rand(rows, cols, generator=gen) < some)


@pytest.mark.parametrize("code", [2.0 ** -6, 0.25, 448.0])
@pytest.mark.parametrize("K", [1024, 2704])
@pytest.mark.parametrize("T", [5, 40, 800, 1400])
def test_terms_keep_their_bits_whatever_the_codes(T, K, code):
    """Codes ± one size times one scale: every term is a whole number times its
    square, exact in fp32 (17 bits), rounded to 11 bits beyond 16 tokens and then
    to bf16, with codes that reach the last one and with small ones, as a matrix
    with one scale for all of it has."""
    torch = torch_mod()
    E, N = 4, 300
    ids, w = torch.arange(T, device="cuda").remainder(E).int()[:, None], torch.ones(T, 1, device="cuda")
    r = gq().moe_plan(ids, w, E)
    a, b = _signs(T, K, T + K), _signs(E * N, K, K, some=0.4).view(E, N, K)
    whole = torch.stack([a[t].double() @ b[t % E].double().t() for t in range(T)])
    assert whole.abs().max() < 2048
    slot = r.order.long().cpu()
    h = gq().Fp8Matrix((a[slot] * code).cuda().to(_t("fp8")), torch.ones(T, -(-K // 128), device="cuda"), 1)
    d = gq().Fp8Experts((b * code).cuda().to(_t("fp8")), torch.ones(E, -(-N // 128), -(-K // 128), device="cuda"))
    y = gq().fp8_expert_gemm(h, r, d).cpu()
    term = whole * code * code
    if T > 16:   # 11 bits: of 448² = 49·2^12 times a whole number not all are in them
        m, e = torch.frexp(term)
        term = torch.ldexp((m * 2048).round(), e - 11)
    assert torch.equal(y, term.to(torch.float32).to(torch.bfloat16))


@pytest.mark.parametrize("T,E,N,K", [(40, 4, 300, 520), (800, 4, 515, 400), (1400, 4, 515, 400), (800, 4, 300, 2704)])
def test_terms_of_blocks_and_columns_of_any_size(T, E, N, K):
    """Blocks of K whose scales are far apart, weights' rows far smaller than
    their neighbours, whole tokens of small codes: a term is off by half a step
    of fp16, 2^-11 of it, or of fp16's smallest numbers below a largest of 2^14,
    2^-39 of the largest term among its neighbours."""
    torch = torch_mod()
    k = 2
    ids, w = _choice(T, E, k, T)
    r = gq().moe_plan(ids, w, E)
    h, d = _matrix(T * k, K, 1, 1), _experts(E, N, K, 2)
    h.scales *= 2.0 ** torch.randint(-20, 21, h.scales.shape, generator=torch.Generator().manual_seed(1)).cuda()
    d.scales *= 2.0 ** torch.randint(-20, 21, d.scales.shape, generator=torch.Generator().manual_seed(2)).cuda()
    rows = h.codes.view(torch.uint8)
    rows[::3] = (rows[::3] & 0x80) | 0x08 + (rows[::3] & 7)             # codes of 2^-6 .. 2^-5
    cols = d.codes.view(torch.uint8)
    cols[:, 1::5] = (cols[:, 1::5] & 0x80) | 0x08 + (cols[:, 1::5] & 7)
    H, D, I = _values(h), _each(d), ids.cpu().numpy()
    ref, bound = moe.combined(H, I, _np(w), D, None, grouped=True, half_terms=True)
    y = gq().fp8_expert_gemm(h, r, d)
    _check(y, ref, bound, "bf16", f"TERMS {T}x{E}x{k} {N}x{K}")


@pytest.mark.parametrize("T", [40, 800, 1400])
def test_an_infinite_term_leaves_its_neighbours_their_values(T):
    """A sum past fp32's range, or NaN, beside ordinary ones of its row."""
    torch = torch_mod()
    E, N, K = 4, 300, 256
    ids, w = torch.arange(T, device="cuda").remainder(E).int()[:, None], torch.ones(T, 1, device="cuda")
    r = gq().moe_plan(ids, w, E)
    h = gq().Fp8Matrix(torch.zeros(T, K, device="cuda").to(_t("fp8")), torch.full((T, 2), 2.0 ** 60, device="cuda"), 1)
    h.codes[:, 3] = 256.0
    d = gq().Fp8Experts(torch.full((E, N, K), 2.0 ** -6, device="cuda").to(_t("fp8")), torch.full((E, 3, 2), 2.0 ** 60, device="cuda"))
    d.codes[2, 70, 3], d.codes[2, 71, 3] = 256.0, -256.0     # 2^136
    d.codes.view(torch.uint8)[2, 200, 3] = 0x7F
    y = gq().fp8_expert_gemm(h, r, d).double()
    want = torch.full((T, N), 2.0 ** 122, dtype=torch.float64, device="cuda")
    of = ids[:, 0] == 2
    want[of, 70], want[of, 71], want[of, 200] = float("inf"), float("-inf"), float("nan")
    assert torch.equal(y.isnan(), want.isnan()) and torch.equal(y.nan_to_num(0.0), want.nan_to_num(0.0))
