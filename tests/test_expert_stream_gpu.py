"""The product back where a workgroup goes from tile to tile: whole numbers, so
that a scale, a row or a block of K from the tile before shows."""
import pytest

from parity_utils import gq, torch_mod
from test_expert_gpu import _same, _t

pytestmark = pytest.mark.gpu


def _ternary(shape, gen):
    """Codes -1, 0 and 1, rows at multiples of 16 bytes."""
    torch = torch_mod()
    wide = torch.zeros(*shape[:-1], (shape[-1] + 15) // 16 * 16, dtype=torch.float8_e4m3fn, device="cuda")
    x = torch.randint(-1, 2, shape, generator=gen, device="cuda").float()
    wide[..., :shape[-1]] = x.to(torch.float8_e4m3fn)
    return wide[..., :shape[-1]], x


def _powers(shape, most, gen):
    torch = torch_mod()
    return 2.0 ** torch.randint(0, most + 1, shape, generator=gen, device="cuda").float()


# rows of each expert: tiles of 32, 128 and (16-bit results) 256 rows, the last of
# an expert cut so that waves have no rows; columns for more tiles than workgroups
SHAPES = {"32": ([40] * 24, 1700), "128": ([168, 200, 232], 11300), "256": ([340, 300], 16700)}


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
# 8, 9, 16, 17, 20 and 24 blocks of K: one group of eight scales to three, whole and
# begun; rows that end with a block, between two pieces of 16 bytes and inside one
@pytest.mark.parametrize("K", [1024, 1100, 2048, 2100, 2512, 3000])
@pytest.mark.parametrize("rows", sorted(SHAPES))
def test_tiles_one_behind_the_other(rows, K, dtype):
    torch = torch_mod()
    counts, N = SHAPES[rows]
    E, k, kb, nb = len(counts), 2, -(-K // 128), -(-N // 128)
    gen = torch.Generator(device="cuda").manual_seed(K + E)
    ids = torch.cat([torch.full((c,), e) for e, c in enumerate(counts)] + [torch.full((10,), -1)])
    ids = ids[torch.randperm(ids.numel(), generator=torch.Generator().manual_seed(K))].view(-1, k).int().cuda()
    T = ids.shape[0]
    w = 0.5 * _powers((T, k), 2, gen)
    r = gq().moe_plan(ids, w, E)
    hc, h = _ternary((T * k, K), gen)
    dc, d = _ternary((E, N, K), gen)
    hs, ds = _powers((T * k, kb), 1, gen), 4.0 ** torch.randint(0, 2, (E, nb, kb), generator=gen, device="cuda").float()
    res = torch.randint(-50, 51, (T, N), generator=gen, device="cuda").to(_t(dtype))
    y = gq().fp8_expert_gemm(gq().Fp8Matrix(hc, hs, 1), r, gq().Fp8Experts(dc, ds), res, out_dtype=_t(dtype))
    want = res.double()
    order, off = r.order.long(), r.offsets.tolist()
    for e in range(E):
        at = slice(off[e], off[e + 1])
        a = h[at].double() * hs[at].double().repeat_interleave(128, 1)[:, :K]
        b = d[e].double() * ds[e].double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
        term = a @ b.t()
        if dtype == "bf16":   # 11 bits of a whole number
            assert term.abs().max() < 65504
            term = term.half().double()
        slot = order[at]
        want.index_add_(0, slot // k, term * w.reshape(-1)[slot].double()[:, None])
    assert want.abs().max() < 2 ** 20       # halves of whole numbers: exact in fp32
    assert _same(y, want.float().to(_t(dtype)))
