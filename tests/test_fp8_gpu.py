"""The 8-bit floating-point calls on the GPU, against the fp64 oracle."""
import numpy as np
import pytest

from oracle import fp8
from parity_utils import gq, log, torch_mod

pytestmark = pytest.mark.gpu

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}   # half a step, relative
TINY = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -14}


def _t(name):
    torch = torch_mod()
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def _np(t):
    return t.double().cpu().numpy()


def _codes(m):
    torch = torch_mod()
    return m.codes.contiguous().view(torch.uint8).cpu().numpy()


def _values(m):
    """What the oracle computes with: (values of the codes, scales)."""
    return fp8.decode(_codes(m)), m.scales.cpu().numpy()


def _rand(rows, cols, seed, dtype="f32", std=1.0):
    torch = torch_mod()
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=gen) * std
    x[:, torch.rand(cols, generator=gen) < 0.02] *= 15
    return x.to(_t(dtype)).cuda()


def _strided(t, ld, offset=0):
    """The same matrix with row stride ld, starting `offset` elements into its storage."""
    torch = torch_mod()
    rows, cols = t.shape
    flat = torch.zeros(rows * ld + offset + 64, dtype=t.dtype, device=t.device)
    out = flat[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    out.copy_(t)
    return out


def _same_codes(got, q, what):
    """Codes as the oracle's; one step off only where the quotient lies
    within 2^-22 of a border (a scale one unit off moves it that far)."""
    want = fp8.nearest(q)
    bad = got != want
    assert np.all(fp8.border_distance(q[bad]) <= 2.0 ** -22), what
    return int(bad.sum())


# ---------------------------------------------------------------- quantize
def test_every_border_is_kept():
    """Scale 1 (448 leads every block): each code, each border, and its
    neighbours one fp32 unit away, exactly as the oracle rounds them."""
    torch = torch_mod()
    mid = fp8._MID.astype(np.float32)
    v = np.concatenate([fp8.GRID.astype(np.float32), mid, np.nextafter(mid, np.float32(0)),
                        np.nextafter(mid, np.float32(1e9)), np.float32([1e-45, 1e-38, 2.0 ** -10, 0.0])])
    v = np.concatenate([v, -v])
    v = np.pad(v, (0, -v.size % 127)).reshape(-1, 127)
    x = np.concatenate([np.full((v.shape[0], 1), 448, np.float32), v], 1)
    m = gq().fp8_quantize(torch.from_numpy(x).cuda())
    assert np.all(m.scales.cpu().numpy() == 1)
    assert np.array_equal(fp8.decode(_codes(m)), fp8.nearest(x.astype(np.float64)))


@pytest.mark.parametrize("rows,cols,dtype,br", [
    (1, 1, "bf16", 1), (1, 4096, "bf16", 1), (3, 127, "f16", 1), (5, 129, "f32", 1), (17, 2056, "bf16", 1),
    (300, 1000, "f16", 1), (129, 11008, "bf16", 1), (1, 128, "f32", 128), (128, 128, "bf16", 128),
    (129, 131, "f16", 128), (300, 1000, "f32", 128), (1000, 520, "bf16", 128)])
def test_quantize_is_exact(rows, cols, dtype, br):
    """Scales and codes bit for bit: both are one rounding of an exact value."""
    x = _rand(rows, cols, rows * cols, dtype, 0.5)
    m = gq().fp8_quantize(x, br)
    v, s = fp8.quantize(_np(x), br)
    assert np.array_equal(m.scales.cpu().numpy(), s)
    assert np.array_equal(fp8.decode(_codes(m)), v)


def test_ties_between_codes_go_to_the_even_one():
    """bf16 values on a coarse grid whose blocks have scales with few bits
    (odd multiples of 2^-j): many quotients are exact ties."""
    torch = torch_mod()
    rng = np.random.default_rng(3)
    b = np.array([1, 3, 5, 9, 11, 13, 15, 17])
    x = rng.integers(-400, 401, (8, 128)) / 8 * b[:, None] / 4.0
    x[:, 0] = 448 / 8 * b / 4.0 * 8
    xt = torch.from_numpy(x).float().cuda()
    assert np.array_equal(_np(xt), x)
    m = gq().fp8_quantize(xt)
    v, s = fp8.quantize(x, 1)
    q = x / fp8.expand(s, 1, *x.shape)
    assert np.mean(fp8.border_distance(q) == 0) > 0.02   # ties are there
    assert np.array_equal(m.scales.cpu().numpy(), s) and np.array_equal(fp8.decode(_codes(m)), v)


@pytest.mark.parametrize("br", [1, 128])
def test_quantize_blocks_that_are_not_finite_or_are_zero(br):
    torch = torch_mod()
    x = _rand(260, 400, 5)
    x[0, 3], x[1, 130], x[2, 399] = float("nan"), float("inf"), float("-inf")
    x[3] = 0
    x[4, :128] = torch.randn(128, device="cuda") * 1e-42     # below fp32's normal numbers
    x[200:, 256:384] = 0
    x[5, 128:256] = 3e38
    m = gq().fp8_quantize(x, br)
    v, s = fp8.quantize(_np(x), br)
    assert np.array_equal(m.scales.cpu().numpy(), s, equal_nan=True)
    assert np.array_equal(fp8.decode(_codes(m)), v, equal_nan=True)


@pytest.mark.parametrize("br", [1, 128])
def test_quantize_strides_and_what_lies_behind(br):
    torch = torch_mod()
    x = _rand(150, 333, 6, "bf16")
    want = gq().fp8_quantize(x, br)
    for ld, off in [(333, 0), (336, 0), (340, 1), (401, 3)]:
        codes = torch.full((150, ld), 0x55, dtype=torch.uint8, device="cuda")
        scales = torch.empty_like(want.scales)
        out = gq().Fp8Matrix(codes.view(torch.float8_e4m3fn)[:, :333], scales, br)
        got = gq().fp8_quantize(_strided(x, ld, off), br, out=out)
        assert got is out and torch.equal(scales, want.scales)
        assert np.array_equal(_codes(got), _codes(want))
        assert torch.all(codes[:, 333:] == 0x55)
    assert gq().fp8_quantize(x[:0], br).codes.shape == (0, 333)


# ---------------------------------------------------------------- rmsnorm
@pytest.mark.parametrize("rows,cols,dtype,gd,res,y", [
    (1, 1, "f32", "f32", False, True), (1, 4096, "bf16", "bf16", True, False), (3, 100, "f16", "f32", True, True),
    (7, 513, "bf16", "f32", False, True), (33, 2048, "f16", "f16", True, True), (5, 2049, "f32", "f32", True, False),
    (4, 8190, "bf16", "bf16", True, True), (2, 16384, "f16", "f32", True, True), (3, 20000, "bf16", "bf16", False, True),
    (2, 40000, "f32", "f32", True, True), (2, 65536, "bf16", "f32", True, True)])
def test_rmsnorm(rows, cols, dtype, gd, res, y):
    torch = torch_mod()
    x, r = _rand(rows, cols, cols, dtype), _rand(rows, cols, cols + 1, dtype, 3.0)
    gamma = (1 + 0.1 * torch.randn(cols, generator=torch.Generator().manual_seed(1))).to(_t(gd)).cuda()
    out = gq().rmsnorm_fp8(x, gamma, 1e-5, residual=r if res else None, want_y=y)
    h = (x.double() + r.double()).to(_t(dtype)) if res else x
    assert torch.equal(out.h, h)
    ref = fp8.rmsnorm(_np(h), _np(gamma), 1e-5)
    _, s = fp8.quantize(ref, 1)
    got = out.q.scales.cpu().numpy()
    assert np.all(np.abs(got / s.astype(np.float64) - 1) <= 2.0 ** -23)   # one unit, where fp64 errors meet a border
    off = _same_codes(fp8.decode(_codes(out.q)), ref / fp8.expand(got, 1, rows, cols), "codes")
    log(f"RMSNORM {rows}x{cols} {dtype}: scales differing {int(np.sum(got != s))}, codes beside a border {off}")
    if y:
        assert np.all(np.abs(_np(out.y) - ref) <= np.abs(ref) * HALF[dtype] * (1 + 2.0 ** -12) + TINY[dtype] * HALF[dtype])
        only = gq().rmsnorm_fp8(x, gamma, 1e-5, residual=r if res else None, want_q=False, want_y=True)
        assert only.q is None and torch.equal(only.y, out.y)


def test_rmsnorm_in_place_and_strided():
    torch = torch_mod()
    x, r = _rand(9, 1000, 1, "bf16"), _rand(9, 1000, 2, "bf16")
    gamma = torch.rand(1000, device="cuda").bfloat16()
    want = gq().rmsnorm_fp8(x, gamma, residual=r)
    for xs, rs in [(x.clone(), r.clone()), (_strided(x, 1003, 1), _strided(r, 1024, 3))]:
        got = gq().rmsnorm_fp8(xs, gamma, residual=rs, h_out=rs)
        assert got.h is rs and torch.equal(rs, want.h) and torch.equal(got.q.scales, want.q.scales)
        assert np.array_equal(_codes(got.q), _codes(want.q))
        got = gq().rmsnorm_fp8(xs, gamma, residual=r, h_out=xs)
        assert torch.equal(xs, want.h) and np.array_equal(_codes(got.q), _codes(want.q))
    wide = torch.full((9, 1100), 7.0, dtype=torch.bfloat16, device="cuda")
    gq().rmsnorm_fp8(x, gamma, residual=r, h_out=wide[:, :1000])
    assert torch.equal(wide[:, :1000], want.h) and torch.all(wide[:, 1000:] == 7)
    assert gq().rmsnorm_fp8(x[:0], gamma, residual=r[:0], want_y=True).q.codes.shape == (0, 1000)


def test_rmsnorm_rows_that_are_zero_huge_or_not_finite():
    torch = torch_mod()
    x = torch.randn(6, 300, generator=torch.Generator().manual_seed(2)).cuda()
    x[0] = 0
    x[1] = 3e38
    x[2, 7] = float("nan")
    x[3, 7] = float("inf")
    x[4] = 1e-30
    gamma = torch.ones(300, device="cuda")
    out = gq().rmsnorm_fp8(x, gamma, 1e-6, want_y=True)
    with np.errstate(invalid="ignore"):
        ref = fp8.rmsnorm(_np(x), _np(gamma), 1e-6)
    v, s = fp8.quantize(ref, 1)
    got = out.q.scales.cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(s)) and np.isnan(s[2]).all() and np.isnan(s[3, 0]) and not np.isnan(s[3, 1:]).any()
    ok = ~np.isnan(s)
    assert np.all(np.abs(got[ok] / s[ok].astype(np.float64) - 1) <= 2.0 ** -23)
    assert np.array_equal(np.isnan(fp8.decode(_codes(out.q))), np.isnan(v))
    assert np.all(_codes(out.q)[0] & 0x7F == 0)
    assert np.array_equal(np.isnan(_np(out.y)), np.isnan(ref))


# ---------------------------------------------------------------- products
def _matrix(rows, cols, br, seed, std=1.0):
    return gq().fp8_quantize(_rand(rows, cols, seed, "f32", std), br)


def _check(C, ref, bound, dtype, what):
    got = _np(C)
    tol = bound + (np.abs(ref) + bound) * HALF[dtype] + TINY[dtype] * HALF[dtype]
    err = np.abs(got - ref)
    log(f"{what}: max err/tolerance {np.max(err / tol):.3e}")
    assert np.all(err <= tol), what


SHAPES = [(1, 1, 1), (1, 128, 128), (1, 4096, 4096), (2, 100, 300), (3, 1000, 1040), (7, 257, 4096), (16, 512, 2048),
          (17, 130, 640), (33, 4000, 1024), (37, 300, 11008), (64, 1024, 1000), (65, 640, 3968), (100, 129, 384),
          (128, 256, 256), (200, 1100, 513), (256, 512, 128), (257, 770, 1280), (300, 4096, 640), (513, 1300, 777),
          (1000, 2100, 256), (2048, 2304, 896), (2100, 6300, 300), (2000, 7000, 640)]


# every kernel the sizes choose between, split and unsplit
SHAPES = [(*s, ["f32", "bf16", "f16"][i % 3]) for i, s in enumerate(SHAPES)] + [
    (54, 122, 204, "bf16"), (51, 126, 2303, "f16"), (50, 122, 1384, "f32"), (229, 129, 5362, "bf16"),
    (480, 129, 1958, "f32"), (385, 7173, 211, "bf16"), (301, 6540, 200, "f32"), (66, 2803, 6309, "f16"),
    (65, 1350, 5633, "f32"), (1951, 6168, 203, "f16"), (131, 5510, 7906, "f32"), (3216, 1423, 7218, "bf16"),
    (20, 17000, 300, "bf16"), (47, 2000, 640, "bf16"), (16, 130, 65536, "bf16"), (49, 130, 65530, "f32"),
    (65, 128, 1291, "f32"), (20, 300, 700, "f32"), (8, 1000, 2000, "f16"), (9, 1000, 2000, "f32"),
    (33, 8324, 557, "bf16"), (1431, 30, 4875, "f16"), (65, 5740, 4516, "bf16"), (33, 30, 133, "f32"),
    (197, 6989, 137, "f32"), (1098, 66, 5606, "f32"), (65, 5671, 3143, "f32"), (471, 8371, 5355, "f32")]


@pytest.mark.parametrize("M,N,K,dtype", SHAPES)
def test_gemm(M, N, K, dtype):
    """Every size with and without a workspace, and twice the same."""
    torch = torch_mod()
    shape = (M, N, K)
    a, b = _matrix(M, K, 1, 1), _matrix(N, K, 128, 2, 0.05)
    ref, mag = fp8.matmul(_values(a), _values(b))
    bound = fp8.accumulation_bound(mag, K, grouped=dtype != "f32")
    C = gq().fp8_gemm(a, b, out_dtype=_t(dtype))
    _check(C, ref, bound, dtype, f"GEMM {shape} {dtype}")
    assert torch.equal(gq().fp8_gemm(a, b, out_dtype=_t(dtype)), C)
    n = gq()._native
    D = torch.full_like(C, float("nan"))
    rc = n.lib().gptq_fp8_gemm(a.codes.data_ptr(), a.scales.data_ptr(), M, K, a.codes.stride(0) if M > 1 else K,
                               b.codes.data_ptr(), b.scales.data_ptr(), N, b.codes.stride(0) if N > 1 else K,
                               D.data_ptr(), {"f32": n.F32, "bf16": n.BF16, "f16": n.F16}[dtype], N, None, 0,
                               torch.cuda.current_stream().cuda_stream)
    assert rc == n.OK, n.last_error()
    _check(D, ref, bound, dtype, f"GEMM {shape} {dtype} unsplit")


GATED = [(1, 1, 1, "silu"), (1, 4096, 1024, "silu"), (4, 1000, 4096, "gelu"), (9, 130, 300, "gelu_tanh"),
         (16, 384, 640, "silu"), (33, 1100, 1152, "silu"), (64, 256, 2048, "gelu"), (65, 300, 777, "silu"),
         (130, 500, 256, "gelu_tanh"), (256, 1280, 384, "silu"), (300, 2050, 512, "silu"), (1025, 900, 520, "gelu"),
         (2100, 3200, 300, "silu"), (1800, 4100, 256, "gelu_tanh")]


GATED = [(*s, ["f32", "bf16", "f16"][i % 3]) for i, s in enumerate(GATED)] + [
    (51, 126, 2303, "silu", "bf16"), (50, 122, 1384, "gelu", "f32"), (65, 2823, 202, "silu", "f16"),
    (67, 231, 5226, "silu", "bf16"), (66, 464, 1924, "gelu_tanh", "f32"), (213, 6510, 200, "silu", "bf16"),
    (165, 5605, 207, "silu", "f32"), (65, 3284, 5935, "silu", "f16"), (67, 1421, 3204, "silu", "f32"),
    (1282, 4452, 203, "silu", "bf16"), (135, 2942, 7038, "gelu", "f32"), (456, 4178, 6348, "silu", "bf16"),
    (20, 9000, 300, "gelu", "bf16"), (65, 120, 2194, "silu", "bf16"), (65, 121, 1484, "silu", "f32"),
    (396, 4716, 4274, "silu", "f32"), (166, 5484, 258, "gelu_tanh", "f32"), (20, 300, 700, "silu", "f32"),
    (40, 300, 700, "silu", "f32"), (8, 1000, 2000, "silu", "f32"), (64, 1000, 2000, "silu", "f32"),
    (17, 30, 136, "silu", "bf16"), (521, 36, 6938, "gelu", "f16"), (98, 6156, 137, "silu", "f32"),
    (1421, 68, 4327, "gelu_tanh", "f32"), (66, 2769, 3937, "silu", "f32"), (169, 8277, 5581, "silu", "f32"),
    (49, 32, 132, "gelu", "bf16")]


@pytest.mark.parametrize("M,N,K,act,dtype", GATED)
def test_gated(M, N, K, act, dtype):
    torch = torch_mod()
    shape = (M, N, K, act)
    a, g_, u = _matrix(M, K, 1, 1), _matrix(N, K, 128, 2, 0.05), _matrix(N, K, 128, 3, 0.05)
    ref, bound = fp8.gated(_values(a), _values(g_), _values(u), act)
    n = gq()._native

    def unsplit(C, dt, q):
        ld = lambda m, r: m.codes.stride(0) if r > 1 else K
        rc = n.lib().gptq_fp8_gated_gemm(
            a.codes.data_ptr(), a.scales.data_ptr(), M, K, ld(a, M), g_.codes.data_ptr(), g_.scales.data_ptr(), ld(g_, N),
            u.codes.data_ptr(), u.scales.data_ptr(), ld(u, N), N, {"silu": 0, "gelu": 1, "gelu_tanh": 2}[act],
            C.data_ptr() if C is not None else None, dt, N, q.codes.data_ptr() if q else None,
            (q.codes.stride(0) if M > 1 else N) if q else 0, q.scales.data_ptr() if q else None, None, 0,
            torch.cuda.current_stream().cuda_stream)
        assert rc == n.OK, n.last_error()

    wide = fp8.gated(_values(a), _values(g_), _values(u), act, grouped=dtype != "f32")[1]
    C = gq().fp8_gated_gemm(a, g_, u, act, out_dtype=_t(dtype))
    _check(C, ref, wide, dtype, f"GATED {shape} {dtype}")
    D = torch.full_like(C, float("nan"))
    unsplit(D, {"f32": n.F32, "bf16": n.BF16, "f16": n.F16}[dtype], None)
    _check(D, ref, wide, dtype, f"GATED {shape} {dtype} unsplit")
    q1 = gq().fp8_gated_gemm(a, g_, u, act)
    q2 = gq().Fp8Matrix(torch.zeros_like(q1.codes), torch.zeros_like(q1.scales), 1)
    unsplit(None, 0, q2)
    for q, how in [(q1, ""), (q2, " unsplit")]:
        v, s = _values(q)
        kb = s.shape[1]
        pad = lambda x: np.pad(x, ((0, 0), (0, kb * 128 - N))).reshape(M, kb, 128)
        amax, eb = pad(np.abs(ref)).max(2), pad(bound).max(2)
        assert np.all(np.abs(s - np.maximum(amax / 448, 2.0 ** -126)) <= eb / 448 + s * 2.0 ** -23), how
        e = fp8.expand(s, 1, M, N)
        tol = bound + (np.abs(ref) + bound) * 2.0 ** -4 + e * 2.0 ** -10
        assert np.all(np.abs(v * e - ref) <= tol), how


@pytest.mark.parametrize("M,N,K", [(70, 150, 400), (5, 150, 400), (30, 40, 401), (300, 600, 130), (3, 20, 9)])
def test_products_take_any_stride_and_leave_the_rest(M, N, K):
    torch = torch_mod()
    a, b, u = _matrix(M, K, 1, 1), _matrix(N, K, 128, 2, 0.05), _matrix(N, K, 128, 3, 0.05)
    want, wq = gq().fp8_gemm(a, b), gq().fp8_gated_gemm(a, b, u)
    F = gq().Fp8Matrix
    E4 = torch.float8_e4m3fn
    for ld, off in [(K + 1, 0), ((K + 31) // 16 * 16, 3), (512, 16)]:
        s = lambda m: F(_strided(m.codes.view(torch.uint8), ld, off).view(E4), m.scales, m.block_rows)
        for aa, bb, uu in [(s(a), b, u), (a, s(b), s(u)), (s(a), s(b), s(u))]:
            wide = torch.full((M, N + 9), 7.0, dtype=torch.bfloat16, device="cuda")
            assert torch.equal(gq().fp8_gemm(aa, bb, out=wide[:, :N]), want) and torch.all(wide[:, N:] == 7)
            cw = torch.full((M, N + 10), 0x55, dtype=torch.uint8, device="cuda")
            q = gq().fp8_gated_gemm(aa, bb, uu, out=F(cw.view(E4)[:, :N], torch.empty_like(wq.scales), 1))
            assert np.array_equal(_codes(q), _codes(wq)) and torch.equal(q.scales, wq.scales)
            assert torch.all(cw[:, N:] == 0x55)
    assert gq().fp8_gemm(F(a.codes[:0], a.scales[:0], 1), b).shape == (0, N)
    assert gq().fp8_gated_gemm(F(a.codes[:0], a.scales[:0], 1), b, u).codes.shape == (0, N)


@pytest.mark.parametrize("M,N,K", [(5, 300, 300), (70, 300, 300), (300, 600, 300)])
def test_what_is_not_finite_stays_in_its_row_and_column(M, N, K):
    """A NaN block of A makes its row NaN, one of B its 128 columns; a NaN
    code makes its row or column NaN; bytes behind K are NaN codes and stay out."""
    torch = torch_mod()
    F, E4 = gq().Fp8Matrix, torch.float8_e4m3fn
    a, b, u = _matrix(M, K, 1, 1), _matrix(N, K, 128, 2, 0.05), _matrix(N, K, 128, 3, 0.05)

    def behind(m):
        w = torch.full((m.codes.shape[0], 320), 0x7F, dtype=torch.uint8, device="cuda")
        w[:, :K] = m.codes.view(torch.uint8)
        return F(w.view(E4)[:, :K], m.scales.clone(), m.block_rows)

    want, wg = gq().fp8_gemm(a, b), gq().fp8_gated_gemm(a, b, u, out_dtype=torch.float32)
    a, b, u = behind(a), behind(b), behind(u)
    assert torch.equal(gq().fp8_gemm(a, b), want)
    assert torch.equal(gq().fp8_gated_gemm(a, b, u, out_dtype=torch.float32), wg)
    a.scales[1, 2] = float("nan")
    a.codes.view(torch.uint8)[3, 299] = 0x7F
    b.codes.view(torch.uint8)[7, 0] = 0xFF
    b.scales[1, 0] = float("nan")
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[1], bad[3], bad[:, 7], bad[:, 128:256] = True, True, True, True
    C = gq().fp8_gemm(a, b)
    assert torch.equal(torch.isnan(C), bad) and torch.equal(C[~bad], want[~bad])
    H = gq().fp8_gated_gemm(a, b, u, out_dtype=torch.float32)
    assert torch.equal(torch.isnan(H), bad) and torch.equal(H[~bad], wg[~bad])
    q = gq().fp8_gated_gemm(a, b, u)
    blocks = torch.nn.functional.pad(bad, (0, -N % 128)).view(M, -1, 128).any(2)
    assert torch.equal(torch.isnan(q.scales), blocks)
    nan = blocks.repeat_interleave(128, 1)[:, :N]
    assert torch.equal(torch.isnan(q.codes.float()), nan)


# ---------------------------------------------------------------- together
def _ffn(g, x, r, gamma, wg, wu, wd):
    """One feed-forward block in 8 bits, as a served model runs it."""
    n = g.rmsnorm_fp8(x, gamma, 1e-5, residual=r)
    h = g.fp8_gated_gemm(n.q, wg, wu)
    return n.h, h, g.fp8_gemm(h, wd)


@pytest.mark.parametrize("M", [1, 5, 100, 300])
def test_feed_forward_block(M):
    """norm -> gate and up -> down in 8 bits: every step against the oracle
    on the step's own input, and the whole against the same block with its
    tensors kept in fp64 (weights in 8 bits in both)."""
    torch = torch_mod()
    d, f = 512, 1400
    x, r = _rand(M, d, 1, "bf16"), _rand(M, d, 2, "bf16", 2.0)
    gamma = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    wg, wu, wd = _matrix(f, d, 128, 3, 0.05), _matrix(f, d, 128, 4, 0.05), _matrix(d, f, 128, 5, 0.03)
    h, q, C = _ffn(gq(), x, r, gamma, wg, wu, wd)
    assert torch.equal(h, (x.double() + r.double()).bfloat16())
    ref, mag = fp8.matmul(_values(q), _values(wd))
    _check(C, ref, fp8.accumulation_bound(mag, f, grouped=True), "bf16", f"FFN {M}")
    y = fp8.rmsnorm(_np(h), _np(gamma), 1e-5)
    mid = fp8.activation(y @ fp8.values(_values(wg), 128).T, "silu") * (y @ fp8.values(_values(wu), 128).T)
    whole = mid @ fp8.values(_values(wd), 128).T
    # each 8-bit rounding is off by at most 2^-4 of a value; independent
    # errors average over the sums, so the norm stays well under that bound
    rel = np.linalg.norm(_np(C) - whole) / np.linalg.norm(whole)
    log(f"FFN M={M}: 8-bit block off by {rel:.4f} of the fp64 block")
    assert rel <= 3 * 2.0 ** -4


def test_feed_forward_block_in_a_graph_and_on_a_stream():
    torch = torch_mod()
    d, f = 512, 1280
    gamma = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    wg, wu, wd = _matrix(f, d, 128, 3, 0.05), _matrix(f, d, 128, 4, 0.05), _matrix(d, f, 128, 5, 0.03)
    for M in (3, 150):
        xs = [(_rand(M, d, i, "bf16"), _rand(M, d, 50 + i, "bf16")) for i in range(4)]
        want = [_ffn(gq(), x, r, gamma, wg, wu, wd) for x, r in xs]
        x, r = xs[0][0].clone(), xs[0][1].clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = _ffn(gq(), x, r, gamma, wg, wu, wd)
        side.synchronize()
        assert torch.equal(got[2], want[0][2])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            h, q, C = _ffn(gq(), x, r, gamma, wg, wu, wd)
        for i in (0, 1, 2, 3, 1):
            x.copy_(xs[i][0])
            r.copy_(xs[i][1])
            graph.replay()
            eager = _ffn(gq(), *xs[(i + 1) % 4], gamma, wg, wu, wd)
            torch.cuda.synchronize()
            assert torch.equal(h, want[i][0]) and torch.equal(C, want[i][2])
            assert np.array_equal(_codes(q), _codes(want[i][1])) and torch.equal(q.scales, want[i][1].scales)
            assert torch.equal(eager[2], want[(i + 1) % 4][2])


def test_two_streams_at_once():
    """Split products on two streams, each with its own workspace, in turn
    and at once: the same bits."""
    torch = torch_mod()
    a, b, u = _matrix(100, 4096, 1, 1), _matrix(700, 4096, 128, 2, 0.05), _matrix(700, 4096, 128, 3, 0.05)
    want, wq = gq().fp8_gemm(a, b), gq().fp8_gated_gemm(a, b, u)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for st in (s, t):
        st.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(20):
        with torch.cuda.stream(s):
            got.append((gq().fp8_gemm(a, b), want))
        with torch.cuda.stream(t):
            got.append((gq().fp8_gated_gemm(a, b, u), wq))
    torch.cuda.synchronize()
    for x, y in got:
        if isinstance(x, torch.Tensor):
            assert torch.equal(x, y)
        else:
            assert torch.equal(x.scales, y.scales) and np.array_equal(_codes(x), _codes(y))


def test_a_workspace_of_ones_own_is_used_and_checked():
    torch = torch_mod()
    n = gq()._native
    a, b = _matrix(100, 4096, 1, 1), _matrix(700, 4096, 128, 2, 0.05)
    need = n.lib().gptq_workspace_bytes(n.WS_FP8_GEMM, 700, 4096, 100, None)
    assert need > 256
    ws = torch.full((need + 256,), 0x7F, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        assert torch.equal(gq().fp8_gemm(a, b, ws=ws[:need]), gq().fp8_gemm(a, b))
    assert torch.all(ws[need:] == 0x7F)
    with pytest.raises(gq().GPTQError):
        gq().fp8_gemm(a, b, ws=ws[:need - 256])
    with pytest.raises(ValueError):
        gq().fp8_gemm(a, b, ws=ws.cpu())


def test_gptq_weights_into_the_8_bit_product():
    """Ŵ of a quantized layer (fp32) as an 8-bit matrix: the layer's output
    against fp64 with the 8-bit weights."""
    torch = torch_mod()
    g = gq()
    W, X = _rand(256, 512, 1, "bf16", 0.02), _rand(1024, 512, 2, "bf16")
    q, _, _ = g.quantize(W, X, g.GPTQParams())
    b, a = g.fp8_quantize(q.W_hat, 128), g.fp8_quantize(X[:50])
    ref, mag = fp8.matmul(_values(a), _values(b))
    _check(g.fp8_gemm(a, b), ref, fp8.accumulation_bound(mag, 512, grouped=True), "bf16", "GPTQ")


def test_offsets_past_32_bits():
    """Matrices of more than 4 GiB: their last rows as the small matrix of the
    same rows gives them."""
    torch = torch_mod()
    rows, cols = (1 << 17) + 300, 32896
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-200:] = _rand(200, cols, 1, "bf16")
    for br in (1, 128):
        m = gq().fp8_quantize(x, br)
        tail = 300 if br == 128 else 200   # a whole number of 128-row blocks before it
        t = gq().fp8_quantize(x[-tail:], br)
        k = m.scales.shape[0] - t.scales.shape[0]
        assert rows % 128 == 300 % 128 and torch.equal(m.scales[k:], t.scales)
        assert torch.equal(m.codes[-tail:].view(torch.uint8), t.codes.view(torch.uint8))
    w = _matrix(130, cols, 128, 2, 0.05)
    a = gq().fp8_quantize(x, 1)
    t = gq().Fp8Matrix(a.codes[-256:], a.scales[-256:], 1)
    C, D = gq().fp8_gemm(a, w), gq().fp8_gemm(t, w, ws=None)
    ref, mag = fp8.matmul((fp8.decode(_codes(t))[-4:], t.scales.cpu().numpy()[-4:]), _values(w))
    _check(C[-4:], ref, fp8.accumulation_bound(mag, cols, grouped=True), "bf16", "PAST 32 BITS")
    _check(D[-4:], ref, fp8.accumulation_bound(mag, cols, grouped=True), "bf16", "PAST 32 BITS (tail)")
    assert torch.all(C[:256] == 0)
    n = gq().rmsnorm_fp8(x, torch.ones(cols, device="cuda"), 1e-6)
    s = gq().rmsnorm_fp8(x[-200:], torch.ones(cols, device="cuda"), 1e-6)
    assert torch.equal(n.q.scales[-200:], s.q.scales)
    assert torch.equal(n.q.codes[-200:].view(torch.uint8), s.q.codes.view(torch.uint8))


@pytest.mark.parametrize("M,N,K", [(1, 64, 8192), (2, 32, 4096), (16, 4, 2000)])
def test_codes_of_the_smallest_products_get_their_workspace(M, N, K):
    """The binding's own workspace and a caller's give the same bits, also
    where 256 bytes would hold the whole result."""
    torch = torch_mod()
    n = gq()._native
    a, g_, u = _matrix(M, K, 1, 1), _matrix(N, K, 128, 2, 0.05), _matrix(N, K, 128, 3, 0.05)
    ws = torch.empty(n.lib().gptq_workspace_bytes(n.WS_FP8_GATED, N, K, M, None), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 256
    x, y = gq().fp8_gated_gemm(a, g_, u), gq().fp8_gated_gemm(a, g_, u, ws=ws)
    assert torch.equal(x.scales, y.scales) and np.array_equal(_codes(x), _codes(y))


@pytest.mark.parametrize("eps", [1e-5, 1e-6, 3e-12])
def test_rmsnorm_rows_far_below_eps(eps):
    """eps counts in full: rows whose mean square is small beside it are
    x/sqrt(eps), rounded once, which eps in fp32 (up to 2^-25 off) would not
    give."""
    torch = torch_mod()
    x = torch.randn(16, 1000, generator=torch.Generator().manual_seed(3)).cuda()
    x *= (eps ** 0.5 * 2.0 ** -torch.arange(4, 20, device="cuda"))[:, None].float()
    gamma = torch.ones(1000, device="cuda")
    out = gq().rmsnorm_fp8(x, gamma, eps, want_y=True)
    ref = fp8.rmsnorm(_np(x), _np(gamma), eps)
    assert np.all(np.abs(_np(out.y) - ref) <= np.abs(ref) * HALF["f32"] * (1 + 2.0 ** -12))
    _, s = fp8.quantize(ref, 1)
    got = out.q.scales.cpu().numpy()
    # fp64 errors (below 2^-48) can move a scale over a border of fp32 in one of 2^23
    assert np.sum(got != s) <= 1 and np.all(np.abs(got / s.astype(np.float64) - 1) <= 2.0 ** -23)
    _same_codes(fp8.decode(_codes(out.q)), ref / fp8.expand(got, 1, 16, 1000), "codes")


# ---------------------------------------------------------------- exact sums
def _integers(rows, cols, br, seed, shift=0):
    """Codes -7..7 and scales 2^-shift and half of it: products of two such
    matrices are multiples of 2^-2 (times the shifts) below 2^24 of them for
    every K <= 65536, so all sums are exact in fp32 in any order, and an eight
    of products spans less than 2^13, so the fp8 instruction drops nothing."""
    torch = torch_mod()
    rng = np.random.default_rng(seed)
    v = rng.integers(-7, 8, (rows, cols)).astype(np.float32)
    s = 2.0 ** -(shift + rng.integers(0, 2, (-(-rows // br), -(-cols // 128))))
    codes = torch.zeros(rows, (cols + 15) // 16 * 16, dtype=torch.float8_e4m3fn, device="cuda")
    codes[:, :cols] = torch.from_numpy(v).cuda().to(torch.float8_e4m3fn)
    return gq().Fp8Matrix(codes[:, :cols], torch.from_numpy(s.astype(np.float32)).cuda(), br)


@pytest.mark.parametrize("M,N,K", sorted({s[:3] for s in SHAPES}))
def test_gemm_of_integers_is_exact(M, N, K):
    """Every type, every kernel and split: the exact result, rounded once.  A
    column of K that is left out, taken twice or scaled wrongly shows."""
    torch = torch_mod()
    a, b = _integers(M, K, 1, 1), _integers(N, K, 128, 2)
    ref = torch.from_numpy(fp8.values(_values(a), 1) @ fp8.values(_values(b), 128).T)
    n = gq()._native
    for dtype, code in [("f32", n.F32), ("bf16", n.BF16), ("f16", n.F16)]:
        want = ref.to(_t(dtype)).cuda()
        assert torch.equal(gq().fp8_gemm(a, b, out_dtype=_t(dtype)), want), dtype
        D = torch.full_like(want, float("nan"))
        rc = n.lib().gptq_fp8_gemm(a.codes.data_ptr(), a.scales.data_ptr(), M, K, (K + 15) // 16 * 16,
                                   b.codes.data_ptr(), b.scales.data_ptr(), N, (K + 15) // 16 * 16,
                                   D.data_ptr(), code, N, None, 0, torch.cuda.current_stream().cuda_stream)
        assert rc == n.OK and torch.equal(D, want), f"{dtype} unsplit"


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (16, 130, 65536), (37, 300, 11008), (66, 2803, 6309), (480, 129, 1958),
                                   (301, 6540, 200), (65, 5740, 4516), (300, 4096, 640)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gemm_16_bits_is_as_near_as_its_instruction_allows(M, N, K, dtype):
    """Beside the output's rounding, no value is further off than eight
    spreads of what the instruction drops, and the whole no further than one
    (a rounding's mean square is a third of its largest)."""
    a, b = _matrix(M, K, 1, 1), _matrix(N, K, 128, 2, 0.05)
    ref, mag = fp8.matmul(_values(a), _values(b))
    acc, sigma = fp8.accumulation_bound(mag, K), fp8.dropped_spread(_values(a), _values(b))
    C = gq().fp8_gemm(a, b, out_dtype=_t(dtype))
    _check(C, ref, acc + 8 * sigma, dtype, f"GEMM {(M, N, K)} {dtype} tight")
    err = np.linalg.norm(_np(C) - ref)
    limit = np.sqrt(np.sum(sigma ** 2 + (np.abs(ref) * HALF[dtype]) ** 2 / 3)) + np.linalg.norm(acc)
    log(f"GEMM {(M, N, K)} {dtype}: error norm {err / np.linalg.norm(ref):.3e} of the result's, limit "
        f"{limit / np.linalg.norm(ref):.3e}, spread {np.linalg.norm(sigma) / np.linalg.norm(ref):.3e}")
    assert err <= limit


# ---------------------------------------------------------------- codes of gated products
def _gated_null(a, g_, u, act, q):
    """Codes without a workspace."""
    torch = torch_mod()
    n = gq()._native
    (M, K), N = a.codes.shape, g_.codes.shape[0]
    ld = (K + 15) // 16 * 16
    rc = n.lib().gptq_fp8_gated_gemm(
        a.codes.data_ptr(), a.scales.data_ptr(), M, K, ld, g_.codes.data_ptr(), g_.scales.data_ptr(), ld,
        u.codes.data_ptr(), u.scales.data_ptr(), ld, N, {"silu": 0, "gelu": 1, "gelu_tanh": 2}[act], None, 0, 0,
        q.codes.data_ptr(), q.codes.stride(0) if M > 1 else (N + 15) // 16 * 16, q.scales.data_ptr(), None, 0,
        torch.cuda.current_stream().cuda_stream)
    assert rc == n.OK, n.last_error()


@pytest.mark.parametrize("M,N,K,act", sorted({s[:4] for s in GATED}))
def test_gated_of_integers(M, N, K, act):
    """With exact sums (gate values of about 2) h depends on neither kernel
    nor split.  fp32: the activation's own error alone.  Codes, with and
    without a workspace: scales of the computed h bit for bit, codes nearest
    to it but within 2^-22 of a border (1/s and the product round by 2^-24
    each).  16 bits: the product act·(A·Uᵀ) rounded once, to fp32 first or not
    (one instruction rounds a product of two floats straight to
    fp16).  With p that product, h is within 2^-24·|p| of it and the result
    within a half step of p or of h, so within a half step and 2·2^-24·|p| of
    h; 2·2^-24 is at most 2^-12 of fp16's half step 2^-11, and |p| at most
    |h|·(1 + 2^-23)."""
    torch = torch_mod()
    k = max(0, round(float(np.log2(14 * K ** 0.5))) - 1)
    a, g_, u = _integers(M, K, 1, 1), _integers(N, K, 128, 2, k), _integers(N, K, 128, 3, k)
    x = fp8.values(_values(a), 1)
    cg, cu = x @ fp8.values(_values(g_), 128).T, x @ fp8.values(_values(u), 128).T
    f = fp8.activation(cg, act)
    # the exponent of gelu_tanh, rounded before exp: |x| + |x|³/8 units more
    z = np.minimum(np.abs(cg) + np.abs(cg) ** 3 / 8, 100.0)
    h = gq().fp8_gated_gemm(a, g_, u, act, out_dtype=torch.float32)
    err = np.abs(_np(h) - f * cu)
    assert np.all(err <= np.abs(f * cu) * 2.0 ** -24 * (10 + 4 * z) + 1e-37 * (1 + np.abs(cu)))
    q1 = gq().fp8_gated_gemm(a, g_, u, act)
    q2 = gq().Fp8Matrix(torch.zeros_like(q1.codes), torch.zeros_like(q1.scales), 1)
    _gated_null(a, g_, u, act, q2)
    _, s = fp8.quantize(_np(h), 1)
    for q, how in [(q1, "workspace"), (q2, "none")]:
        assert np.array_equal(q.scales.cpu().numpy(), s), how
        _same_codes(fp8.decode(_codes(q)), _np(h) / fp8.expand(s, 1, M, N), how)
    for dtype in ("bf16", "f16"):
        C = gq().fp8_gated_gemm(a, g_, u, act, out_dtype=_t(dtype))
        assert np.all(np.abs(_np(C) - _np(h)) <= np.abs(_np(h)) * HALF[dtype] * (1 + 2.0 ** -11) + TINY[dtype] * HALF[dtype]), dtype


@pytest.mark.parametrize("M,N,K", [(8, 1000, 2000), (64, 1000, 2000), (67, 1421, 3204), (300, 2050, 512), (1025, 900, 520)])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gated_codes_beside_exact_sums(M, N, K, act):
    """On inputs with cancellation, through few rows, tiles, splits and with
    no workspace: a code differs from that of the exact sums only where a
    border lies within the error bound of the fp32 sums, and few do: with h
    off by 2^-20 of itself, a border is within reach of one in 2^15 values
    (steps are at least 1/16 of a value), given twice that for cancellation."""
    torch = torch_mod()
    a, g_, u = _matrix(M, K, 1, 1), _matrix(N, K, 128, 2, 0.05), _matrix(N, K, 128, 3, 0.05)
    ref, bound = fp8.gated(_values(a), _values(g_), _values(u), act)
    v, s = fp8.quantize(ref, 1)
    e = fp8.expand(s, 1, M, N)
    q1 = gq().fp8_gated_gemm(a, g_, u, act)
    q2 = gq().Fp8Matrix(torch.zeros_like(q1.codes), torch.zeros_like(q1.scales), 1)
    _gated_null(a, g_, u, act, q2)
    for q, how in [(q1, "workspace"), (q2, "none")]:
        got = fp8.decode(_codes(q))
        bad = got != v
        x = np.abs(ref[bad] / e[bad])
        far = fp8.border_distance(x) * np.maximum(x, 2.0 ** -10)
        # the scale's own error moves every quotient of its block
        top = np.pad(np.abs(ref), ((0, 0), (0, -N % 128))).reshape(M, -1, 128)
        ts = np.pad(bound, ((0, 0), (0, -N % 128))).reshape(M, -1, 128)
        ds = np.repeat(np.max(ts, 2) / np.max(top, 2), 128, 1)[:, :N]
        assert np.all(far <= bound[bad] / e[bad] + x * (ds[bad] + 2.0 ** -21)), how
        log(f"GATED {(M, N, K)} {act} codes, {how}: {bad.sum()} of {bad.size} beside a border, "
            f"scales differing {np.mean(q.scales.cpu().numpy() != s):.3f}")
        assert bad.sum() <= 2.0 ** -14 * bad.size + 4, how


# ---------------------------------------------------------------- the norm's y
def _rounded(x, dtype):
    """x (fp64) to the nearest of a 16-bit type, ties to even, in one step."""
    bits, low = {"bf16": (8, -126), "f16": (11, -14)}[dtype]
    step = 2.0 ** (np.maximum(np.frexp(x)[1] - 1, low) + 1 - bits)   # of the value's binade
    return np.rint(x / step) * step


@pytest.mark.parametrize("rows,cols,dtype", [(333, 8190, "f16"), (300, 8192, "bf16"), (70, 40000, "f16")])
def test_rmsnorm_y_is_rounded_once(rows, cols, dtype):
    """Bit for bit the fp64 result's nearest: by way of fp32, one value in 2^14
    (fp16) or 2^17 (bf16) would land on a border first and then on its wrong
    side."""
    torch = torch_mod()
    x = _rand(rows, cols, 7, dtype)
    gamma = (1 + 0.1 * torch.randn(cols, generator=torch.Generator().manual_seed(1))).cuda()
    y = _np(gq().rmsnorm_fp8(x, gamma, 1e-5, want_q=False, want_y=True).y)
    ref = _rounded(fp8.rmsnorm(_np(x), _np(gamma), 1e-5), dtype)
    assert np.array_equal(y, ref), f"{np.sum(y != ref)} of {y.size} differ"
