"""Routing to experts, the experts' products and the product with an epilogue
on the GPU, against the fp64 oracle."""
import numpy as np
import pytest

from oracle import fp8, moe
from parity_utils import gq, log, torch_mod

pytestmark = pytest.mark.gpu

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}   # half a step, relative
TINY = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -14}


def _t(name):
    torch = torch_mod()
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "fp8": torch.float8_e4m3fn}[name]


def _np(t):
    return t.double().cpu().numpy()


def _values(m):
    torch = torch_mod()
    return fp8.decode(m.codes.contiguous().view(torch.uint8).cpu().numpy()), m.scales.cpu().numpy()


def _randn(*shape, seed, std=1.0):
    torch = torch_mod()
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std


def _matrix(rows, cols, br, seed, std=1.0):
    x = _randn(rows, cols, seed=seed, std=std)
    if br == 1:
        x[:, ::37] *= 10
    return gq().fp8_quantize(x.cuda(), br)


def _experts(E, N, K, seed, std=0.05):
    return gq().fp8_quantize_experts(_randn(E, N, K, seed=seed, std=std).cuda())


def _each(m):
    """The experts' weights as the oracle takes them."""
    return [_values(m.expert(e)) for e in range(m.codes.shape[0])]


def _same(a, b):
    """Bitwise, NaN included; tensors or Fp8Matrix."""
    torch = torch_mod()
    if hasattr(a, "codes"):
        return _same(a.codes, b.codes) and _same(a.scales, b.scales)
    kind = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.contiguous().view(kind), b.contiguous().view(kind))


def _check(got, ref, bound, dtype, what):
    tol = bound + (np.abs(ref) + bound) * HALF[dtype] + TINY[dtype] * HALF[dtype]
    err = np.abs(_np(got) - ref)
    log(f"{what}: max err/tolerance {np.max(err / tol, initial=0):.3e}")
    assert np.all(err <= tol), what


def _check_codes(q, ref, bound, what):
    """Scales within the values' bound and a rounding, values within half a
    step of e4m3 (2^-4 relative, 2^-10 below its normal numbers)."""
    v, s = q
    rows, n = ref.shape
    kb = s.shape[1]
    pad = lambda x: np.pad(x, ((0, 0), (0, kb * 128 - n))).reshape(rows, kb, 128)
    amax, eb = pad(np.abs(ref)).max(2), pad(bound).max(2)
    assert np.all(np.abs(s - np.maximum(amax / 448, 2.0 ** -126)) <= eb / 448 + s * 2.0 ** -23), what
    e = fp8.expand(s, 1, rows, n)
    assert np.all(np.abs(v * e - ref) <= bound + (np.abs(ref) + bound) * 2.0 ** -4 + e * 2.0 ** -10), what


# ---------------------------------------------------------------- routing
def _check_route(r, logits, k, weights_of=None, **kw):
    ids, w = moe.route(_np(logits), k, **kw)
    E = logits.shape[1]
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    got = _np(r.weights)
    assert np.array_equal(np.isnan(got), np.isnan(w))
    ok = ~np.isnan(w)
    # one rounding of an fp64 value that is itself off by a few hundred units at most
    assert np.all(np.abs(got[ok] - w[ok]) <= np.abs(w[ok]) * (2.0 ** -24 + 2.0 ** -40) + 2.0 ** -150)
    offsets, order = moe.plan(ids, E)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.order.cpu().numpy(), order)


ROUTES = [  # T, E, k, dtype, options
    (1, 1, 1, "f32", {}),
    (1, 64, 8, "bf16", {}),
    (3, 5, 5, "f16", dict(kind="sigmoid", renormalize=False)),
    (7, 8, 2, "bf16", dict(renormalize=False, scale=0.5)),
    (16, 16, 4, "f32", dict(kind="sigmoid")),
    (17, 17, 3, "f32", dict(renormalize=False)),
    (63, 60, 6, "bf16", dict(groups=4, top_groups=2, scale=1.5)),
    (64, 100, 8, "f16", dict(groups=5, top_groups=2, group_top=2)),
    (65, 128, 8, "bf16", {}),
    (129, 256, 8, "f32", dict(kind="sigmoid", groups=8, top_groups=4, group_top=2, scale=2.5)),
    (200, 255, 64, "f32", dict(renormalize=False)),
    (33, 257, 8, "bf16", dict(groups=1)),
    (40, 512, 10, "f32", dict(kind="sigmoid", groups=16, top_groups=5, group_top=2)),
    (21, 1024, 64, "f16", dict(groups=16, top_groups=16)),
    (21, 1000, 32, "f32", dict(kind="sigmoid", renormalize=False)),
    (1025, 64, 6, "bf16", {}),
    (5000, 32, 4, "f32", dict(kind="sigmoid")),
    (4500, 130, 8, "bf16", dict(groups=2, top_groups=1)),
]


@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("T,E,k,dtype,kw", ROUTES)
def test_route(T, E, k, dtype, kw, with_bias):
    torch = torch_mod()
    logits = _randn(T, E, seed=T + E, std=2.0).to(_t(dtype)).cuda()
    bias = _randn(E, seed=E, std=0.1).cuda() if with_bias else None
    opts = {("scores" if n == "kind" else n): v for n, v in kw.items()}
    r = gq().moe_route(logits, k, bias=bias, **opts)
    _check_route(r, logits, k, bias=None if bias is None else _np(bias), **kw)
    again = gq().moe_route(logits, k, bias=bias, **opts)
    assert all(_same(getattr(r, n), getattr(again, n)) for n in ("ids", "weights", "offsets", "order"))
    p = gq().moe_plan(r.ids, r.weights, E)
    assert torch.equal(p.offsets, r.offsets) and torch.equal(p.order, r.order)


@pytest.mark.parametrize("T", [5, 300])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("groups,top_groups,group_top", [(1, 1, 1), (4, 2, 1), (4, 2, 2)])
def test_route_ties_masks_and_what_is_not_finite(T, kind, with_bias, groups, top_groups, group_top):
    """Rows of equal logits, rows that leave nothing or little, padding that is
    NaN, and infinities: a row decides for itself alone."""
    torch = torch_mod()
    E, k = 32, 6
    gen = torch.Generator().manual_seed(T)
    x = torch.randint(-3, 4, (T, E), generator=gen).float()      # ties everywhere
    x[0] = 1.0
    x[1] = float("-inf")
    x[2] = float("-inf")
    x[2, [3, 30]] = torch.tensor([-1.0, 2.0])
    x[3, 7] = float("nan")
    x[4, 9] = float("inf")
    x[T - 1] = torch.finfo(torch.float32).min
    if T > 5:
        x[6] = -800.0                                            # sigmoids that are 0
        x[7, ::2] = float("-inf")
        x[8] = torch.finfo(torch.float32).min
        x[8, 5:] = float("-inf")
        x[9:12] = float("nan")
    mask = torch.ones(T, dtype=torch.bool)
    mask[9:12] = False
    if T > 5:
        mask[13] = False
    bias = None
    if with_bias:
        # the same within a group: sums of two tie only where their terms do,
        # so that no tie hangs on a rounding
        bias = torch.tensor([0.0, 0.25, 0.0, 0.25]).repeat_interleave(8)
        bias[4] = float("-inf")
        bias = bias.cuda()
    x = x.cuda()
    kw = dict(groups=groups, top_groups=top_groups, group_top=group_top)
    for m in (None, mask.cuda()):
        r = gq().moe_route(x, k, scores=kind, bias=bias, mask=m, **kw)
        _check_route(r, x, k, kind=kind, bias=None if bias is None else _np(bias),
                     mask=None if m is None else mask.numpy(), **kw)


def test_route_strides_no_tokens_and_all_padding():
    torch = torch_mod()
    x = _randn(50, 40, seed=1).bfloat16().cuda()
    want = gq().moe_route(x, 4)
    wide = torch.full((50, 47), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 3:43] = x
    got = gq().moe_route(wide[:, 3:43], 4)
    assert all(_same(getattr(got, n), getattr(want, n)) for n in ("ids", "weights", "offsets", "order"))
    none = gq().moe_route(x[:0], 4)
    assert none.ids.shape == (0, 4) and none.offsets.tolist() == [0] * 41 and none.order.numel() == 0
    none = gq().moe_plan(none.ids, none.weights, 40)
    assert none.offsets.tolist() == [0] * 41
    for T in (50, 5):
        off = gq().moe_route(x[:T], 4, mask=torch.zeros(T, dtype=torch.bool, device="cuda"))
        assert torch.all(off.ids == -1) and torch.all(off.weights == 0) and torch.all(off.offsets == 0) and torch.all(off.order == -1)


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (3, 2, 9), (700, 8, 200), (2000, 8, 1024), (9000, 3, 7), (40000, 2, 64)])
def test_plan_of_any_ids(T, k, E):
    """Ids from everywhere: repeated within a token, negative, too large."""
    torch = torch_mod()
    gen = torch.Generator().manual_seed(T)
    ids = torch.randint(-2, E + 3, (T, k), generator=gen).int()
    ids[T // 2] = ids[T // 2, 0]
    if T > 10:
        ids[5], ids[6] = 2 ** 31 - 1, -2 ** 31
    r = gq().moe_plan(ids.cuda(), torch.zeros(T, k, device="cuda"), E)
    flat = ids.reshape(-1).numpy()
    live = (flat >= 0) & (flat < E)
    order = np.argsort(np.where(live, flat, E), kind="stable")
    order = np.where(live[order], order, -1)
    assert np.array_equal(r.order.cpu().numpy(), order)
    counts = np.bincount(flat[live], minlength=E)
    assert np.array_equal(r.offsets.cpu().numpy(), np.concatenate([[0], np.cumsum(counts)]))


# ---------------------------------------------------------------- product with an epilogue
LINEAR = [(1, 1, 1), (1, 4096, 1024), (2, 130, 300), (7, 257, 640), (16, 512, 2048), (33, 1100, 512), (37, 300, 4000),
          (64, 1024, 1000), (65, 640, 3968), (100, 129, 384), (130, 500, 256), (257, 770, 1280), (300, 4096, 640),
          (513, 1300, 777), (1025, 900, 520), (2100, 3300, 300), (54, 122, 204), (229, 129, 5362), (131, 5510, 3000)]


@pytest.mark.parametrize("i,M,N,K", [(i, *s) for i, s in enumerate(LINEAR)])
def test_linear(i, M, N, K):
    """Each size in each output form, with the bias, activation and residual
    that its number picks, split and unsplit, and twice the same."""
    torch = torch_mod()
    a, b = _matrix(M, K, 1, 1), _matrix(N, K, 128, 2, 0.05)
    A, B = _values(a), _values(b)
    acts = [None, "silu", "gelu", "gelu_tanh"]
    for j, c in enumerate(["bf16", "f16", "f32", "fp8"]):
        act = acts[(i + j) % 4]
        bias = [None, "f32", c if c != "fp8" else "bf16"][(i + j) % 3]
        bias = None if bias is None else _randn(N, seed=3, std=0.5).to(_t(bias)).cuda()
        res = _randn(M, N, seed=4, std=2.0).to(_t(c)).cuda() if c != "fp8" and (i + j) % 2 else None
        ref, bound = moe.linear(A, B, None if bias is None else _np(bias), act, None if res is None else _np(res))
        what = f"LINEAR {M}x{N}x{K} {c} {act}"
        C = gq().fp8_linear(a, b, bias, act, res, out_dtype=_t(c))
        assert _same(gq().fp8_linear(a, b, bias, act, res, out_dtype=_t(c)), C), what
        n = gq()._native
        D = gq().Fp8Matrix(torch.zeros_like(C.codes), torch.zeros_like(C.scales), 1) if c == "fp8" else torch.full_like(C, float("nan"))
        tag = {"f32": n.F32, "bf16": n.BF16, "f16": n.F16, "fp8": 0}
        q = c == "fp8"
        rc = n.lib().gptq_fp8_linear(
            a.codes.data_ptr(), a.scales.data_ptr(), M, K, a.codes.stride(0) if M > 1 else K, b.codes.data_ptr(),
            b.scales.data_ptr(), N, b.codes.stride(0) if N > 1 else K, None if bias is None else bias.data_ptr(),
            0 if bias is None else {torch.float32: n.F32, torch.bfloat16: n.BF16, torch.float16: n.F16}[bias.dtype],
            acts.index(act) - 1, None if res is None else res.data_ptr(), N, None if q else D.data_ptr(), tag[c], N,
            D.codes.data_ptr() if q else None, (D.codes.stride(0) if M > 1 else N) if q else 0,
            D.scales.data_ptr() if q else None, None, 0, torch.cuda.current_stream().cuda_stream)
        assert rc == n.OK, n.last_error()
        for got, how in ((C, what), (D, what + " unsplit")):
            if q:
                _check_codes(_values(got), ref, bound(False), how)
            else:
                _check(got, ref, bound(c != "f32"), c, how)


def test_linear_without_an_epilogue_is_the_product():
    for M, N, K in [(1, 300, 400), (50, 300, 400), (300, 600, 1000)]:
        a, b = _matrix(M, K, 1, 1), _matrix(N, K, 128, 2, 0.05)
        for c in ("bf16", "f32"):
            assert _same(gq().fp8_linear(a, b, out_dtype=_t(c)), gq().fp8_gemm(a, b, out_dtype=_t(c)))


@pytest.mark.parametrize("M,N,K", [(3, 45, 300), (40, 150, 400), (70, 150, 401), (300, 600, 130)])
def test_linear_in_place_strides_and_what_lies_behind(M, N, K):
    torch = torch_mod()
    a, b = _matrix(M, K, 1, 1), _matrix(N, K, 128, 2, 0.05)
    bias, res = _randn(N + 3, seed=1).bfloat16().cuda()[3:], _randn(M, N, seed=2).bfloat16().cuda()
    want = gq().fp8_linear(a, b, bias, "silu", res)
    wide = torch.full((M, N + 9), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 1:N + 1] = res
    got = gq().fp8_linear(a, b, bias, "silu", wide[:, 1:N + 1])
    assert _same(got, want)
    same = wide[:, 1:N + 1]
    assert gq().fp8_linear(a, b, bias, "silu", same, out=same) is same
    assert _same(same, want) and torch.all(wide[:, 0] == 7) and torch.all(wide[:, N + 1:] == 7)
    wq = gq().fp8_linear(a, b, bias, "gelu", out_dtype=_t("fp8"))
    cw = torch.full((M, N + 10), 0x55, dtype=torch.uint8, device="cuda")
    q = gq().Fp8Matrix(cw.view(_t("fp8"))[:, :N], torch.empty_like(wq.scales), 1)
    assert _same(gq().fp8_linear(a, b, bias, "gelu", out=q), wq) and torch.all(cw[:, N:] == 0x55)
    none = gq().Fp8Matrix(a.codes[:0], a.scales[:0], 1)
    assert gq().fp8_linear(none, b, bias).shape == (0, N)


@pytest.mark.parametrize("c", ["bf16", "f16", "f32"])
def test_linear_adds_a_residual_to_the_largest_tiles(c):
    """Many tiles of 256 rows, the last ones cut in both directions, with a
    residual from elsewhere and from the place of the result."""
    torch = torch_mod()
    M, N, K = 2311, 8197, 140
    a, b = _matrix(M, K, 1, 1), _matrix(N, K, 128, 2, 0.05)
    res = _randn(M, N, seed=4, std=2.0).to(_t(c)).cuda()
    ref, bound = moe.linear(_values(a), _values(b), None, None, _np(res))
    got = gq().fp8_linear(a, b, residual=res, out_dtype=_t(c))
    _check(got, ref, bound(c != "f32"), c, f"LINEAR {M}x{N}x{K} {c}")
    wide = torch.full((M, N + 2), 7.0, dtype=_t(c), device="cuda")
    wide[:, 1:N + 1] = res
    same = wide[:, 1:N + 1]
    assert gq().fp8_linear(a, b, residual=same, out=same) is same
    assert _same(same, got) and torch.all(wide[:, 0] == 7) and torch.all(wide[:, N + 1] == 7)


@pytest.mark.parametrize("M", [5, 70, 300])
def test_linear_keeps_what_is_not_finite_in_its_place(M):
    torch = torch_mod()
    N, K = 300, 300
    a, b = _matrix(M, K, 1, 1), _matrix(N, K, 128, 2, 0.05)
    bias, res = _randn(N, seed=1).cuda(), _randn(M, N, seed=2).cuda()
    want = gq().fp8_linear(a, b, bias, "gelu", res, out_dtype=torch.float32)
    wq = gq().fp8_linear(a, b, bias, "gelu", out_dtype=_t("fp8"))
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bias[9] = float("nan")
    bad[:, 9] = True
    q = gq().fp8_linear(a, b, bias, "gelu", out_dtype=_t("fp8"))
    blocks = torch.zeros_like(q.scales, dtype=torch.bool)
    blocks[:, 0] = True
    assert torch.equal(torch.isnan(q.scales), blocks)
    assert torch.equal(q.codes[:, 128:].float(), wq.codes[:, 128:].float())
    res[2, 77] = float("nan")
    bad[2, 77] = True
    a.scales[1, 0] = float("nan")
    bad[1] = True
    got = gq().fp8_linear(a, b, bias, "gelu", res, out_dtype=torch.float32)
    assert torch.equal(torch.isnan(got), bad) and torch.equal(got[~bad], want[~bad])


# ---------------------------------------------------------------- the experts' products
def _choice(T, E, k, seed, how="spread"):
    """ids [T, k] and weights: spread, all on one expert, few experts, with
    slots that have none, or the same expert twice in a token."""
    torch = torch_mod()
    gen = torch.Generator().manual_seed(seed)
    if how == "one":
        ids = torch.full((T, k), E - 1)
    elif how == "twice":
        ids = torch.randint(0, E, (T, k), generator=gen)
        ids[::2, -1] = ids[::2, 0]
    else:
        live = E if how != "few" else max(k, E // 3)
        ids = torch.rand(T, live, generator=gen).argsort(1)[:, :k]
    w = torch.rand(T, k, generator=gen) + 0.1
    if how == "gaps":
        ids[torch.rand(T, k, generator=gen) < 0.3] = -1
        ids[T // 2] = -1
        ids[T - 1, 0] = E + 5
        w[ids < 0] = float("nan")          # of slots without an expert: never read
    return ids.int().cuda(), w.cuda()


EXPERTS = [  # T, E, k, N, K, which experts
    (1, 1, 1, 1, 1, "spread"), (1, 8, 2, 1024, 512, "spread"), (1, 64, 8, 200, 300, "spread"), (2, 4, 2, 130, 129, "twice"),
    (3, 64, 6, 256, 640, "spread"), (5, 16, 4, 257, 1000, "gaps"), (8, 8, 2, 640, 384, "one"), (16, 60, 4, 384, 256, "spread"),
    (17, 256, 8, 128, 512, "spread"), (33, 8, 2, 500, 777, "few"), (61, 64, 8, 256, 512, "spread"), (64, 12, 3, 300, 140, "gaps"),
    (100, 4, 1, 700, 640, "one"), (130, 16, 4, 384, 520, "spread"), (200, 5, 2, 1000, 256, "spread"), (333, 128, 8, 136, 384, "few"),
    (500, 8, 2, 513, 300, "twice"), (700, 8, 2, 1280, 256, "gaps"), (1000, 2, 1, 640, 384, "spread"), (1500, 16, 4, 256, 300, "spread"),
    (300, 1024, 8, 64, 128, "spread"), (1024, 3, 3, 385, 129, "spread"), (40, 300, 16, 40, 200, "few"),
    # few columns and tokens, K cut between two pieces of 16; blocks that end in K = 1040 and 2704
    (2, 64, 8, 300, 400, "spread"), (1, 16, 1, 100, 1040, "spread"), (8, 32, 4, 60, 144, "gaps"), (30, 6, 2, 200, 2704, "spread"),
    # many tiles for each workgroup, products with and without a stream, short ones
    (300, 16, 1, 4500, 520, "spread"), (250, 12, 1, 5600, 300, "gaps"), (900, 8, 1, 7000, 400, "spread"), (900, 8, 1, 7000, 130, "spread"),
    (1000, 8, 2, 1, 200, "spread"), (300, 4, 2, 3, 130, "gaps"),      # terms beside as many bytes of powers of two
    (2000, 4, 1, 8500, 700, "spread"), (1300, 3, 1, 13000, 200, "spread"), (300, 4, 2, 200, 2704, "spread"), (700, 2, 1, 300, 2700, "spread"),
]


@pytest.mark.parametrize("T,E,k,N,K,how", EXPERTS)
def test_expert_gated(T, E, k, N, K, how):
    torch = torch_mod()
    act = ["silu", "gelu", "gelu_tanh"][T % 3]
    a, g_, u = _matrix(T, K, 1, 1), _experts(E, N, K, 2), _experts(E, N, K, 3)
    ids, w = _choice(T, E, k, T + E, how)
    r = gq().moe_plan(ids, w, E)
    A, G, U, I = _values(a), _each(g_), _each(u), ids.cpu().numpy()
    R = int(r.offsets[-1])
    ref, exact = moe.gated(A, I, G, U, act)
    for c in (["bf16", "f16"][T % 2], "f32"):
        out = torch.full((T * k, N), 7.0, dtype=_t(c), device="cuda")
        assert gq().fp8_expert_gated_gemm(a, r, g_, u, act, out=out) is out
        bound = exact if c == "f32" else moe.gated(A, I, G, U, act, grouped=True)[1]
        _check(out[:R], ref, bound, c, f"EXPERT GATED {T}x{E}x{k} {N}x{K} {c}")
        assert torch.all(out[R:] == 7)
        assert _same(gq().fp8_expert_gated_gemm(a, r, g_, u, act, out_dtype=_t(c))[:R], out[:R])
    q = gq().Fp8Matrix(torch.full((T * k, N), 0x55, dtype=torch.uint8, device="cuda").view(_t("fp8")),
                       torch.full((T * k, -(-N // 128)), 7.0, device="cuda"), 1)
    gq().fp8_expert_gated_gemm(a, r, g_, u, act, out=q)
    v, s = _values(q)
    _check_codes((v[:R], s[:R]), ref, exact, "codes")
    assert torch.all(q.codes[R:].view(torch.uint8) == 0x55) and torch.all(q.scales[R:] == 7)
    again = gq().fp8_expert_gated_gemm(a, r, g_, u, act)
    assert _same(again.codes[:R], q.codes[:R]) and _same(again.scales[:R], q.scales[:R])
    bare = gq().Fp8Matrix(torch.zeros_like(again.codes), torch.zeros_like(again.scales), 1)
    n = gq()._native                                        # without a workspace
    ld = lambda m, rows: m.codes.stride(-2) if rows > 1 else K
    rc = n.lib().gptq_fp8_expert_gated_gemm(
        a.codes.data_ptr(), a.scales.data_ptr(), T, K, ld(a, T), k, r.offsets.data_ptr(), r.order.data_ptr(), E,
        g_.codes.data_ptr(), g_.scales.data_ptr(), ld(g_, N), g_.codes.stride(0), u.codes.data_ptr(), u.scales.data_ptr(),
        ld(u, N), u.codes.stride(0), N, ["silu", "gelu", "gelu_tanh"].index(act), None, 0, 0, bare.codes.data_ptr(),
        bare.codes.stride(0) if T * k > 1 else N, bare.scales.data_ptr(), None, 0, torch.cuda.current_stream().cuda_stream)
    assert rc == n.OK, n.last_error()
    v, s = _values(bare)
    _check_codes((v[:R], s[:R]), ref, exact, "codes without a workspace")


@pytest.mark.parametrize("T,E,k,N,K,how", EXPERTS)
def test_expert_gemm(T, E, k, N, K, how):
    torch = torch_mod()
    ids, w = _choice(T, E, k, T + E, how)
    r = gq().moe_plan(ids, w, E)
    h, d = _matrix(T * k, K, 1, 1), _experts(E, N, K, 2)
    R = int(r.offsets[-1])
    h.codes.view(torch.uint8)[R:] = 0x7F                    # behind the last row: not read
    h.scales[R:] = float("nan")
    H, D, I = _values(h), _each(d), ids.cpu().numpy()
    for j, c in enumerate(["bf16", "f16", "f32"]):
        res = _randn(T, N, seed=5, std=2.0).to(_t(c)).cuda() if (T + j) % 2 else None
        ref, bound = moe.combined(H, I, np.nan_to_num(_np(w)), D, None if res is None else _np(res), grouped=c != "f32",
                                  half_terms=c == "bf16" and T > 16)      # up to 16 tokens: no terms leave the kernel
        y = gq().fp8_expert_gemm(h, r, d, res, out_dtype=_t(c))
        _check(y, ref, bound, c, f"EXPERT GEMM {T}x{E}x{k} {N}x{K} {c}")
        assert _same(gq().fp8_expert_gemm(h, r, d, res, out_dtype=_t(c)), y)
        if res is not None:
            assert gq().fp8_expert_gemm(h, r, d, res, out=res) is res and _same(res, y)


@pytest.mark.parametrize("T,E,k,N,K", [(3, 4, 2, 45, 300), (40, 8, 2, 150, 401), (300, 8, 2, 200, 130)])
def test_experts_take_any_stride_and_leave_the_rest(T, E, k, N, K):
    torch = torch_mod()
    F, X, E4 = gq().Fp8Matrix, gq().Fp8Experts, _t("fp8")
    ids, w = _choice(T, E, k, 1)
    r = gq().moe_plan(ids, w, E)
    a, g_, u = _matrix(T, K, 1, 1), _experts(E, N, K, 2), _experts(E, N, K, 3)
    h, d = _matrix(T * k, K, 1, 4), _experts(E, N, K, 5)
    want, wq = gq().fp8_expert_gated_gemm(a, r, g_, u, out_dtype=torch.bfloat16), gq().fp8_expert_gated_gemm(a, r, g_, u)
    wy = gq().fp8_expert_gemm(h, r, d)

    def rows(m, ld, off):
        flat = torch.full((m.codes.shape[0] * ld + off + 64,), 0x7F, dtype=torch.uint8, device="cuda")
        v = flat[off:off + m.codes.shape[0] * ld].view(-1, ld)[:, :K]
        v.copy_(m.codes.view(torch.uint8))
        return F(v.view(E4), m.scales, m.block_rows)

    def experts(m, ld, gap, off):
        flat = torch.full((E * (N * ld + gap) + off,), 0x7F, dtype=torch.uint8, device="cuda")
        v = torch.as_strided(flat, (E, N, K), (N * ld + gap, ld, 1), off)
        v.copy_(m.codes.view(torch.uint8))
        return X(v.view(E4), m.scales)

    for ld, gap, off in [(K + 1, 0, 0), ((K + 31) // 16 * 16, 5, 3), (512, 32, 16)]:
        aa, hh = rows(a, ld, off), rows(h, ld, off)
        gg, uu, dd = experts(g_, ld, gap, off), experts(u, ld, gap, off), experts(d, ld, gap, off)
        wide = torch.full((T * k, N + 9), 7.0, dtype=torch.bfloat16, device="cuda")
        assert _same(gq().fp8_expert_gated_gemm(aa, r, gg, uu, out=wide[:, :N]), want) and torch.all(wide[:, N:] == 7)
        cw = torch.full((T * k, N + 10), 0x55, dtype=torch.uint8, device="cuda")
        q = gq().fp8_expert_gated_gemm(aa, r, gg, uu, out=F(cw.view(E4)[:, :N], torch.empty_like(wq.scales), 1))
        assert _same(q, wq) and torch.all(cw[:, N:] == 0x55)
        wide = torch.full((T, N + 9), 7.0, dtype=torch.bfloat16, device="cuda")
        assert _same(gq().fp8_expert_gemm(hh, r, dd, out=wide[:, :N]), wy) and torch.all(wide[:, N:] == 7)


@pytest.mark.parametrize("T", [2, 40, 300])
def test_experts_take_rows_far_apart(T):
    """Offsets within a tile's rows past 32 bits: weights as [N, E, K], and
    activations that are columns of something wide."""
    torch = torch_mod()
    F, X, E4 = gq().Fp8Matrix, gq().Fp8Experts, _t("fp8")
    E, k, N, K, ld = 3, 2, 140, 260, (1 << 25) + 16
    ids, w = _choice(T, E, k, 1)
    r = gq().moe_plan(ids, w, E)
    a, g_, u = _matrix(T, K, 1, 1), _experts(E, N, K, 2), _experts(E, N, K, 3)
    h, d = _matrix(T * k, K, 1, 4), _experts(E, N, K, 5)
    want, wy = gq().fp8_expert_gated_gemm(a, r, g_, u), gq().fp8_expert_gemm(h, r, d)
    big = torch.empty((max(N, 2 * T) - 1) * ld + (1 << 20), dtype=torch.uint8, device="cuda")

    def far(m, at):
        shape = tuple(m.codes.shape)
        v = torch.as_strided(big, shape, ((4096,) if len(shape) == 3 else ()) + (ld, 1), at)
        v.copy_(m.codes.view(torch.uint8))
        return X(v.view(E4), m.scales) if len(shape) == 3 else F(v.view(E4), m.scales, 1)

    aa, hh, gg, uu, dd = far(a, 0), far(h, 1 << 15), far(g_, 1 << 16), far(u, 1 << 17), far(d, 1 << 18)
    assert gg.codes[0, N - 1].data_ptr() - gg.codes.data_ptr() > 1 << 32
    assert _same(gq().fp8_expert_gated_gemm(aa, r, gg, uu), want)
    assert _same(gq().fp8_expert_gated_gemm(aa, r, g_, u), want) and _same(gq().fp8_expert_gated_gemm(a, r, gg, uu), want)
    assert _same(gq().fp8_expert_gemm(hh, r, dd), wy) and _same(gq().fp8_expert_gemm(h, r, dd), wy)


@pytest.mark.parametrize("T", [3, 40, 300])
def test_experts_keep_what_is_not_finite_with_its_tokens(T):
    """A NaN token, a NaN expert and a NaN weight reach the outputs that they
    belong to, and no others."""
    torch = torch_mod()
    E, k, N, K = 6, 2, 200, 300
    ids, w = _choice(T, E, k, 1)
    a, g_, u = _matrix(T, K, 1, 1), _experts(E, N, K, 2), _experts(E, N, K, 3)
    h, d = _matrix(T * k, K, 1, 4), _experts(E, N, K, 5)
    r = gq().moe_plan(ids, w, E)
    want, wy = gq().fp8_expert_gated_gemm(a, r, g_, u, out_dtype=torch.float32), gq().fp8_expert_gemm(h, r, d)
    slot = r.order.long()
    token, expert = slot // k, ids.reshape(-1)[slot]
    a.scales[1, 1] = float("nan")
    g_.codes[4, 7].view(torch.uint8)[0] = 0x7F
    got = gq().fp8_expert_gated_gemm(a, r, g_, u, out_dtype=torch.float32)
    bad = (token == 1)[:, None].expand(-1, N).clone()
    bad[:, 7] |= expert == 4
    assert torch.equal(torch.isnan(got), bad) and torch.equal(got[~bad], want[~bad])
    q = gq().fp8_expert_gated_gemm(a, r, g_, u)
    assert torch.equal(torch.isnan(q.scales), torch.nn.functional.pad(bad, (0, 56)).view(T * k, -1, 128).any(2))
    d.scales[4, 0, 0] = float("nan")                        # the first 128 columns of expert 4
    w[2, 1] = float("nan")
    y = gq().fp8_expert_gemm(h, r, d)
    bad = torch.zeros(T, N, dtype=torch.bool, device="cuda")
    bad[:, :128] = (ids == 4).any(1)[:, None]
    bad[2] = True
    assert torch.equal(torch.isnan(y), bad) and torch.equal(y[~bad], wy[~bad])


def test_expert_sums_near_the_ends_of_fp32():
    """Terms for bf16 sums keep fp32's range: products just below 2^128, and
    scales whose products are tiny."""
    torch = torch_mod()
    T, E, k, N, K = 40, 2, 1, 130, 256
    ids, w = torch.arange(T, device="cuda").remainder(E).int()[:, None], torch.ones(T, k, device="cuda")
    r = gq().moe_plan(ids, w, E)
    for p, code in [(123, 24.0), (110, 3.0), (100, 1.0), (0, 1.0), (-100, 1.0), (-118, 2.0)]:
        h = gq().Fp8Matrix(torch.zeros(T, K, device="cuda").to(_t("fp8")), torch.full((T, 2), 2.0 ** (p - p // 2), device="cuda"), 1)
        h.codes[:, 5] = 1.0
        d = gq().Fp8Experts(torch.full((E, N, K), code, device="cuda").to(_t("fp8")), torch.full((E, 2, 2), 2.0 ** (p // 2), device="cuda"))
        y = gq().fp8_expert_gemm(h, r, d)
        assert torch.all(y.double() == code * 2.0 ** p), p


def test_experts_with_all_tokens_padding():
    torch = torch_mod()
    for T in (4, 90):
        a, g_, d = _matrix(T, 256, 1, 1), _experts(4, 130, 256, 2), _experts(4, 70, 130, 3)
        r = gq().moe_route(_randn(T, 4, seed=1).cuda(), 2, mask=torch.zeros(T, dtype=torch.bool, device="cuda"))
        h = gq().fp8_expert_gated_gemm(a, r, g_, g_)
        res = _randn(T, 70, seed=2).bfloat16().cuda()
        assert torch.all(gq().fp8_expert_gemm(h, r, d) == 0)
        assert _same(gq().fp8_expert_gemm(h, r, d, res), res)


# ---------------------------------------------------------------- together
def _block(g, x, r, gamma, router, bias, wg, wu, wd, sg, sd, mask=None):
    """A block of experts in 8 bits as a served model runs it: norm, router,
    routed experts, and a shared expert with an ungated activation beside them."""
    torch = torch_mod()
    n = g.rmsnorm_fp8(x, gamma, 1e-5, residual=r)
    logits = g.fp8_linear(n.q, router, out_dtype=torch.float32)
    route = g.moe_route(logits, 4, "sigmoid", bias=bias, groups=4, top_groups=2, group_top=2, scale=2.0, mask=mask)
    h = g.fp8_expert_gated_gemm(n.q, route, wg, wu)
    shared = g.fp8_linear(n.q, sg, activation="gelu", out_dtype=torch.float8_e4m3fn)
    s = g.fp8_linear(shared, sd, residual=n.h)
    return n, logits, route, h, shared, s, g.fp8_expert_gemm(h, route, wd, residual=s)


def _block_weights(d, f, E):
    torch = torch_mod()
    return (torch.ones(d, dtype=torch.bfloat16, device="cuda"), _matrix(E, d, 128, 3, 0.2), _randn(E, seed=4, std=0.1).cuda(),
            _experts(E, f, d, 5), _experts(E, f, d, 6), _experts(E, d, f, 7), _matrix(f, d, 128, 8, 0.05), _matrix(d, f, 128, 9, 0.05))


@pytest.mark.parametrize("T", [1, 7, 100, 300])
def test_block_of_experts(T):
    """Every step against the oracle on the step's own input."""
    torch = torch_mod()
    d, f, E = 512, 384, 16
    W = _block_weights(d, f, E)
    x, r = _randn(T, d, seed=1).bfloat16().cuda(), _randn(T, d, seed=2, std=2.0).bfloat16().cuda()
    mask = torch.ones(T, dtype=torch.bool, device="cuda")
    mask[T // 2 + 1:T // 2 + 3] = False
    n, logits, route, h, shared, s, y = _block(gq(), x, r, *W, mask=mask)
    q = _values(n.q)
    ref, bound = moe.linear(q, _values(W[1]), None, None, None)
    _check(logits, ref, bound(False), "f32", "router")
    _check_route(route, logits, 4, kind="sigmoid", bias=_np(W[2]), groups=4, top_groups=2, group_top=2, scale=2.0, mask=mask.cpu().numpy())
    I, R = route.ids.cpu().numpy(), int(route.offsets[-1])
    ref, bound = moe.gated(q, I, _each(W[3]), _each(W[4]), "silu")
    hv, hs = _values(h)
    _check_codes((hv[:R], hs[:R]), ref, bound, "experts")
    ref, bound = moe.linear(q, _values(W[6]), None, "gelu", None)
    _check_codes(_values(shared), ref, bound(False), "shared expert")
    ref, bound = moe.linear(_values(shared), _values(W[7]), None, None, _np(n.h))
    _check(s, ref, bound(True), "bf16", "shared expert back")
    ref, bound = moe.combined((hv[:R], hs[:R]), I, _np(route.weights), _each(W[5]), _np(s), grouped=True, half_terms=T > 16)
    _check(y, ref, bound, "bf16", f"BLOCK {T}")


def test_block_of_experts_in_a_graph_and_on_a_stream():
    torch = torch_mod()
    d, f, E = 512, 384, 16
    W = _block_weights(d, f, E)
    for T in (3, 150):
        xs = [(_randn(T, d, seed=i).bfloat16().cuda(), _randn(T, d, seed=50 + i).bfloat16().cuda()) for i in range(4)]
        want = [_block(gq(), x, r, *W) for x, r in xs]
        x, r = xs[0][0].clone(), xs[0][1].clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = _block(gq(), x, r, *W)
        side.synchronize()
        assert _same(got[-1], want[0][-1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            _, _, route, h, _, _, y = _block(gq(), x, r, *W)
        for i in (0, 1, 2, 3, 1):
            x.copy_(xs[i][0])
            r.copy_(xs[i][1])
            graph.replay()
            eager = _block(gq(), *xs[(i + 1) % 4], *W)
            torch.cuda.synchronize()
            assert _same(y, want[i][-1]) and torch.equal(route.ids, want[i][2].ids) and _same(h, want[i][3])
            assert _same(eager[-1], want[(i + 1) % 4][-1])


def test_two_streams_at_once():
    """Each with its own workspaces: the same bits as one after the other."""
    torch = torch_mod()
    d, f, E = 512, 384, 16
    W = _block_weights(d, f, E)
    xs = [(_randn(T, d, seed=T).bfloat16().cuda(), _randn(T, d, seed=T + 1).bfloat16().cuda()) for T in (2, 130)]
    want = [_block(gq(), x, r, *W)[-1] for x, r in xs]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(sides):
            with torch.cuda.stream(s):
                got[i].append(_block(gq(), *xs[i], *W)[-1])
    torch.cuda.synchronize()
    assert all(_same(y, want[i]) for i in range(2) for y in got[i])
