"""Tables that are not sorted slots: the outputs are undefined, but no count
passes 32 bits and nothing outside the operands is touched."""
import pytest

from parity_utils import gq, torch_mod
from test_expert_gpu import _choice, _experts, _matrix, _t

pytestmark = pytest.mark.gpu


def _tables(E, slots, how, gen):
    torch = torch_mod()
    i32 = torch.int32
    if how == "up and down":       # half of the experts claim all slots
        return (torch.arange(E + 1) % 2 * slots).to(i32), torch.zeros(slots, dtype=i32)
    if how == "outside":
        return (torch.randint(-2 ** 31, 2 ** 31, (E + 1,), generator=gen).to(i32),
                torch.randint(-2 ** 31, 2 ** 31, (slots,), generator=gen).to(i32))
    return torch.arange(E, -1, -1).to(i32) * (slots // E), torch.arange(slots - 1, -1, -1).to(i32)


@pytest.mark.parametrize("how", ["up and down", "outside", "backwards"])
@pytest.mark.parametrize("T,E,k,N,K", [(3, 16, 4, 100, 300), (61, 64, 8, 300, 260), (600, 6, 2, 520, 400), (2000, 4, 2, 300, 2704)])
def test_tables_of_another_form(T, E, k, N, K, how):
    torch = torch_mod()
    ids, w = _choice(T, E, k, 1)
    offsets, order = (t.cuda() for t in _tables(E, T * k, how, torch.Generator().manual_seed(T)))
    r = gq().Routing(ids, w, offsets, order)
    a, g_, h, d = _matrix(T, K, 1, 1), _experts(E, N, K, 2), _matrix(T * k, K, 1, 3), _experts(E, N, K, 4)
    for c in ("bf16", "f32"):
        for f, x, m, rows in ((gq().fp8_expert_gated_gemm, a, (g_, g_), T * k), (gq().fp8_expert_gemm, h, (d,), T)):
            wide = torch.full((rows + 2, N), 7.0, dtype=_t(c), device="cuda")
            f(x, r, *m, out=wide[1:-1])
            assert torch.all(wide[0] == 7) and torch.all(wide[-1] == 7)
    gq().fp8_expert_gated_gemm(a, r, g_, g_)
    torch.cuda.synchronize()


@pytest.mark.parametrize("c", ["bf16", "f32"])
def test_as_many_stretches_as_32_bits_cannot_count(c):
    torch = torch_mod()
    T, k, E = 1 << 24, 64, 1024
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("memory")
    offsets, order = _tables(E, T * k, "up and down", None)
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    w = torch.ones(T, k, device="cuda")
    r = gq().Routing(ids, w, offsets.cuda(), order.cuda())
    one = lambda rows: gq().Fp8Matrix(torch.ones(rows, 1, device="cuda").to(_t("fp8")), torch.ones(rows, 1, device="cuda"), 1)
    d = gq().Fp8Experts(torch.ones(E, 1, 1, device="cuda").to(_t("fp8")), torch.ones(E, 1, 1, device="cuda"))
    assert gq().fp8_expert_gated_gemm(one(T), r, d, d, out_dtype=_t(c)).shape == (T * k, 1)
    torch.cuda.synchronize()
    assert gq().fp8_expert_gemm(one(T * k), r, d, out_dtype=_t(c)).shape == (T, 1)
    torch.cuda.synchronize()
