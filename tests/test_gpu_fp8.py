"""GPU tests of the block-scaled 8-bit quantizer and matrix product against
their definitions.

Quantizer: the definition is exact (one fp32 division per scale and per
element, one rounding to 8 bits), so codes and scales are compared bit for bit
with the same steps done by torch on the CPU.

Product: compared with the fp64 sum.  Bound per output, S = sum |a w| (scaled):
the result's rounding, half a step of y's type relative to y; the tensor
cores' sum of 128 exact products, at most one fp32 step (2^-23) of S per
addition, 128 * 2^-23 S; the blocks' scale products and additions in fp32,
(blocks + 3) * 2^-24 S.  fp16 results below 2^-14 are rounded to a step of
2^-24.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
LARGEST = {E4M3: 448.0, E5M2: 57344.0}


@pytest.fixture(scope="module")
def B():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from lut_dequant_gemv_b200 import binding, build

    build.build()
    binding.lib()
    return binding


def quantize_ref(x, block_rows, dtype):
    """The definition on the CPU in fp32: x [batch, rows, cols]."""
    z, r, c = x.shape
    p = torch.nn.functional.pad(x.float(), (0, -c % 128, 0, -r % block_rows))
    p = p.view(z, p.shape[1] // block_rows, block_rows, p.shape[2] // 128, 128)
    big = p.abs().amax(dim=(2, 4))
    scale = torch.where(big == 0, torch.ones_like(big), big / LARGEST[dtype])
    v = (p / scale[:, :, None, :, None]).clamp(-LARGEST[dtype], LARGEST[dtype])
    q = v.view(z, -1, p.shape[3] * 128)[:, :r, :c].contiguous().to(dtype)
    return q, scale


def same_codes(a, b):
    a, b = a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)
    return torch.equal(a, b)


def make_x(gen, shape, dtype, kind="normal"):
    x = torch.randn(shape, generator=gen)
    if kind == "wide":  # values over many binades, zeros among them
        x = x * torch.exp2(torch.randint(-20, 8, shape, generator=gen).float())
        x[torch.rand(shape, generator=gen) < 0.2] = 0
    return x.to(dtype)


@pytest.mark.parametrize("fmt", [E4M3, E5M2])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("batch,rows,cols,block_rows", [
    (1, 1, 1, 1), (1, 1, 4096, 1), (1, 3, 127, 1), (1, 5, 129, 1), (2, 7, 1000, 1), (1, 300, 777, 1),
    (1, 1, 1, 128), (1, 128, 128, 128), (1, 129, 255, 128), (3, 200, 300, 128), (2, 127, 1024, 128),
])
def test_quantize_is_the_definition(B, fmt, dtype, batch, rows, cols, block_rows):
    gen = torch.Generator().manual_seed(rows * 1000 + cols)
    for kind in ("normal", "wide"):
        x = make_x(gen, (batch, rows, cols), dtype, kind)
        q, s = B.sqz_fp8_quantize(x.cuda(), block_rows, fmt)
        q_ref, s_ref = quantize_ref(x, block_rows, fmt)
        assert torch.equal(s.cpu(), s_ref)
        assert same_codes(q.cpu(), q_ref)


def test_quantize_division_is_correctly_rounded(B):
    """Every quotient, over blocks whose scales span fp16's and bf16's range (the three-step quotient and, at
    the ends of the range, the division)."""
    gen = torch.Generator().manual_seed(5)
    for dtype, lo, hi in ((torch.float16, -22, 14), (torch.bfloat16, -130, 125)):
        e = torch.randint(lo, hi, (4096, 1), generator=gen).float()
        x = ((torch.rand((4096, 256), generator=gen) * 2 - 1) * torch.exp2(e)).to(dtype)
        q, s = B.sqz_fp8_quantize(x.cuda(), 1, E4M3)
        q_ref, s_ref = quantize_ref(x[None], 1, E4M3)
        assert torch.equal(s.cpu(), s_ref[0])
        assert same_codes(q.cpu(), q_ref[0])


def test_quantize_strides_alignment_and_edges(B):
    """x at every alignment and pitch; the codes' pitch padding and the scales' padding stay as they were."""
    gen = torch.Generator().manual_seed(6)
    for off, ldx in ((0, 200), (1, 201), (3, 240), (8, 208)):
        big = make_x(gen, (40 * 256,), torch.float16).cuda()
        x = big[off:off + 40 * ldx].view(40, ldx)[:, :193]
        qb = torch.full((40, 224), 7, dtype=torch.uint8, device="cuda").view(E4M3)
        sb = torch.full((40, 5), -1.0, device="cuda")
        B.sqz_fp8_quantize(x, 1, q=qb[:, :193], scale=sb[:, :2])
        q_ref, s_ref = quantize_ref(x.cpu()[None], 1, E4M3)
        assert same_codes(qb[:, :193].cpu(), q_ref[0]) and torch.equal(sb[:, :2].cpu(), s_ref[0])
        assert bool((qb.view(torch.uint8)[:, 193:] == 7).all()) and bool((sb[:, 2:] == -1).all())


def test_quantize_zeros_infinities_and_nan(B):
    x = torch.randn(6, 256).half()
    x[0] = 0
    x[1, 3] = float("inf")
    x[2, 130] = float("nan")
    x[3, 5], x[3, 6] = float("-inf"), float("nan")
    x[4] = -0.0
    x[5] = torch.finfo(torch.float16).smallest_normal / 1024  # the smallest subnormal
    q, s = B.sqz_fp8_quantize(x.cuda())
    v, s = q.cpu().float(), s.cpu()
    assert torch.equal(s[0], torch.ones(2)) and bool((v[0] == 0).all()) and bool((v[4] == 0).all())
    assert s[1, 0] == float("inf") and bool(v[1, 3].isnan()) and bool((v[1, :3] == 0).all())
    assert bool(s[2, 1].isnan()) and bool(v[2, 128:].isnan().all()) and not bool(v[2, :128].isnan().any())
    assert bool(s[3, 0].isnan()) and bool(v[3, :128].isnan().all())
    assert bool((v[5] == 448).all())


def random_matrix(gen, rows, k, fmt, block_rows, pitch_extra=0):
    spread = 100.0 if fmt == E4M3 else 10000.0
    ld = (k + 15) // 16 * 16 + pitch_extra
    # the bytes between k and the pitch are NaN codes: they must not be read
    q = torch.full((rows, ld), 0x7F, dtype=torch.uint8).view(fmt)
    q[:, :k] = (torch.randn((rows, k), generator=gen) * spread).clamp(-4 * spread, 4 * spread).to(fmt)
    s = (0.5 + torch.rand((-(-rows // block_rows), -(-k // 128)), generator=gen)) / spread
    q = q.cuda()[:, :k]
    return q, s.cuda()


def dense(q, s, block_rows):
    full = s.double().repeat_interleave(block_rows, 0)[: q.shape[0]].repeat_interleave(128, 1)[:, : q.shape[1]]
    return q.double() * full


def check_product(y, a, sa, w, sw):
    A, W = dense(a, sa, 1), dense(w, sw, 128)
    ref, S = A @ W.t(), A.abs() @ W.abs().t()
    blocks = sa.shape[1]
    fi = torch.finfo(y.dtype)
    tol = fi.eps / 2 * ref.abs() + (2.0 ** -16 + (blocks + 3) * 2.0 ** -24) * S * (1 + fi.eps)
    if y.dtype == torch.float16:
        tol = tol + 2.0 ** -25
    err = (y.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4].tolist(), float((err / tol).max()))


SIZES = [
    (1, 1, 1), (1, 8, 16), (1, 128, 128), (1, 4096, 4096), (2, 300, 1000), (16, 129, 513), (17, 128, 2048),
    (33, 1000, 300), (64, 640, 1152), (65, 200, 4100), (128, 257, 129), (129, 300, 130), (200, 64, 640),
    (257, 1111, 272), (500, 2050, 1000), (1000, 2048, 128), (300, 40, 5000),
    # every tile width: 160, 192 and 256 columns, the last ones partial, W's blocks ending inside a tile
    (300, 5000, 300), (290, 6900, 300), (70, 11000, 390), (200, 19000, 130), (256, 18000, 130),
]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_product_sizes_and_types(B, m, n, k, dtype):
    gen = torch.Generator().manual_seed(m * 7 + n * 3 + k)
    a, sa = random_matrix(gen, m, k, E4M3, 1)
    w, sw = random_matrix(gen, n, k, E4M3, 128, pitch_extra=16 if n % 2 else 0)
    y = torch.full((m, n), float("nan"), dtype=dtype, device="cuda")
    B.sqz_fp8_gemm(a, sa, w, sw, y)
    check_product(y, a, sa, w, sw)
    assert B.sqz_fp8_status() == 0


@pytest.mark.parametrize("fa", [E4M3, E5M2])
@pytest.mark.parametrize("fw", [E4M3, E5M2])
@pytest.mark.parametrize("m", [5, 300])
def test_product_formats(B, fa, fw, m):
    gen = torch.Generator().manual_seed(11)
    a, sa = random_matrix(gen, m, 700, fa, 1)
    w, sw = random_matrix(gen, 390, 700, fw, 128)
    y = torch.empty((m, 390), device="cuda")
    B.sqz_fp8_gemm(a, sa, w, sw, y)
    check_product(y, a, sa, w, sw)


@pytest.mark.parametrize("m", [3, 40, 150, 400])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_product_strides(B, m, dtype):
    """Pitches beyond the sizes, an unaligned y; what lies behind y's columns and last row stays."""
    gen = torch.Generator().manual_seed(12)
    n, k = 333, 400
    a, sa = random_matrix(gen, m, k, E4M3, 1, pitch_extra=48)
    w, sw = random_matrix(gen, n, k, E4M3, 128, pitch_extra=32)
    sa_wide = torch.full((m, 9), float("nan"), device="cuda")
    sa_wide[:, :4] = sa
    for off, ldy in ((0, 336), (0, 344), (4, 340), (2, 338), (1, 341)):  # rows aligned to 32 bytes .. one value
        buf = torch.full(((m + 2) * ldy + off,), -7.0, dtype=dtype, device="cuda")
        y = buf[off:].view(m + 2, ldy)
        B.sqz_fp8_gemm(a, sa_wide[:, :4], w, sw, y[:m, :n])
        check_product(y[:m, :n], a, sa, w, sw)
        assert bool((y[:m, n:] == -7).all()) and bool((y[m:] == -7).all()) and bool((buf[:off] == -7).all())


def test_product_equals_itself_bit_for_bit(B):
    gen = torch.Generator().manual_seed(13)
    for m, n, k in ((1, 1000, 4096), (100, 500, 3000), (300, 700, 3000)):
        a, sa = random_matrix(gen, m, k, E4M3, 1)
        w, sw = random_matrix(gen, n, k, E4M3, 128)
        ys = [torch.empty((m, n), device="cuda") for _ in range(3)]
        for y in ys:
            B.sqz_fp8_gemm(a, sa, w, sw, y)
        assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])


@pytest.mark.parametrize("m", [4, 260])
def test_product_with_nan_codes_and_scales(B, m):
    gen = torch.Generator().manual_seed(14)
    a, sa = random_matrix(gen, m, 384, E4M3, 1)
    w, sw = random_matrix(gen, 200, 384, E4M3, 128)
    a.view(torch.uint8)[2, 200] = 0x7F  # a NaN code: row 2
    w.view(torch.uint8)[77, 5] = 0xFF   # column 77
    sa[1, 0] = float("inf")             # row 1: infinite (or NaN) everywhere
    y = torch.empty((m, 200), device="cuda")
    B.sqz_fp8_gemm(a, sa, w, sw, y)
    assert bool(y[2].isnan().all()) and bool(y[:, 77].isnan().all()) and not bool(y[1].isfinite().any())
    keep = [r for r in range(m) if r not in (1, 2)]
    cols = [c for c in range(200) if c != 77]
    assert bool(y[keep][:, cols].isfinite().all())


def test_product_of_empty_sizes(B):
    f = dict(device="cuda")
    y = torch.full((3, 5), 9.0, **f)
    z = torch.empty((3, 0), dtype=E4M3, **f)
    B.sqz_fp8_gemm(z, torch.empty((3, 0), **f), torch.empty((5, 0), dtype=E4M3, **f), torch.empty((1, 0), **f), y)
    assert bool((y == 0).all())
    a = torch.zeros((0, 128), dtype=E4M3, **f)
    w = torch.zeros((5, 128), dtype=E4M3, **f)
    B.sqz_fp8_gemm(a, torch.empty((0, 1), **f), w, torch.ones((1, 1), **f), torch.empty((0, 5), **f))


@pytest.mark.parametrize("m", [2, 200])
def test_on_another_stream_and_in_a_graph(B, m):
    """Quantize then multiply on a side stream, and the pair captured and replayed on new inputs."""
    gen = torch.Generator().manual_seed(15)
    n, k = 512, 1024
    xs = [torch.randn((m, k), generator=gen).bfloat16().cuda() for _ in range(3)]
    w, sw = random_matrix(gen, n, k, E4M3, 128)
    want = []
    for x in xs:
        q, s = B.sqz_fp8_quantize(x)
        y = torch.empty((m, n), device="cuda")
        B.sqz_fp8_gemm(q, s, w, sw, y)
        check_product(y, q, s, w, sw)
        want.append(y)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    x_in, y_out = torch.empty_like(xs[0]), torch.empty((m, n), device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q, s = B.sqz_fp8_quantize(xs[0])
        B.sqz_fp8_gemm(q, s, w, sw, y_out)
    side.synchronize()
    assert torch.equal(y_out, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.sqz_fp8_quantize(x_in, q=q, scale=s)
        B.sqz_fp8_gemm(q, s, w, sw, y_out)
    for x, y in zip(xs, want):
        x_in.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y_out, y)


def test_prompt_through_a_lut_layer(B, orc):
    """A LUT layer's dense part, dequantized and requantized to 8 bits, for a prompt of more rows than sqz_gemv
    takes; its first rows against sqz_gemv within the error of the two 8-bit roundings (each off by at most
    half a step: 2^-4 of the value)."""
    import numpy as np
    import synth

    L = synth.make_layer(300, 1024, 3, 0.0, seed=4, key="prompt")
    layer = B.create_layer_from_numpy(L.n_out, L.k_in, L.bits, L.codes, L.lut, L.rowptr, L.col, L.val)
    dense_w = torch.empty((300, 1024), dtype=torch.float16, device="cuda")
    B.sqz_debug_dequant(layer, dense_w)
    w, sw = B.sqz_fp8_quantize(dense_w, 128)
    x = torch.from_numpy(synth.make_x(40, 1024, seed=1).view(np.float16).copy()).cuda()
    a, sa = B.sqz_fp8_quantize(x)
    y = torch.empty((40, 300), dtype=torch.float16, device="cuda")
    B.sqz_fp8_gemm(a, sa, w, sw, y)
    check_product(y, a, sa, w, sw)
    y16 = torch.empty((16, 300), dtype=torch.float16, device="cuda")
    B.sqz_gemv(layer, x[:16], y16)
    bound = x[:16].double().abs() @ dense_w.double().abs().t()
    # subnormal codes add an absolute error of half the smallest code (2^-10) times the scale
    slack = 2.0 ** -10 * (sa.double().repeat_interleave(128, 1)[:16] @ dense_w.double().abs().t()
                          + x[:16].double().abs() @ sw.double().repeat_interleave(128, 0)[:300].repeat_interleave(128, 1).t())
    assert bool(((y[:16].double() - y16.double()).abs() <= (2 * 2.0 ** -4 + 2.0 ** -7) * bound + 1.1 * slack).all())
    layer.close()


@pytest.mark.parametrize("m", [3, 200])
def test_offsets_beyond_32_bits(B, m):
    """Pitches that put rows of x, codes, scales and y more than 2^32 bytes apart."""
    gen = torch.Generator().manual_seed(16)
    n, k = 64, 300
    ld_x = (1 << 32) // 2 // m + 64  # the last rows of x lie beyond 2^32 bytes
    x_big = torch.empty((m + 1) * ld_x, dtype=torch.bfloat16, device="cuda")
    x = x_big.view(m + 1, ld_x)[:m, :k]
    x.copy_(torch.randn((m, k), generator=gen))
    ld_q = (1 << 32) // m // 16 * 16 + 64
    q = torch.empty((m + 1) * ld_q, dtype=torch.uint8, device="cuda").view(E4M3).view(m + 1, ld_q)[:m, :k]
    s = torch.empty((m + 1) * (ld_q // 4), device="cuda").view(m + 1, ld_q // 4)[:m, :3]
    B.sqz_fp8_quantize(x, q=q, scale=s)
    q_ref, s_ref = quantize_ref(x.cpu()[None], 1, E4M3)
    assert torch.equal(s.cpu(), s_ref[0]) and same_codes(q.cpu(), q_ref[0])
    w, sw = random_matrix(gen, n, k, E4M3, 128)
    y = torch.empty((m + 1) * (ld_q // 4), device="cuda").view(m + 1, ld_q // 4)[:m, :n]
    B.sqz_fp8_gemm(q, s, w, sw, y)
    check_product(y, q, s, w, sw)


def test_two_streams_at_once(B):
    gen = torch.Generator().manual_seed(17)
    jobs = []
    for m, n, k in ((5, 2000, 3000), (300, 1000, 3000), (64, 700, 1000), (1000, 800, 600)):
        a, sa = random_matrix(gen, m, k, E4M3, 1)
        w, sw = random_matrix(gen, n, k, E4M3, 128)
        want = torch.empty((m, n), device="cuda")
        B.sqz_fp8_gemm(a, sa, w, sw, want)
        check_product(want, a, sa, w, sw)
        jobs.append((a, sa, w, sw, torch.zeros_like(want), want, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for a, sa, w, sw, y, _, stream in jobs:
            B.sqz_fp8_gemm(a, sa, w, sw, y, stream=stream)
    torch.cuda.synchronize()
    for *_, y, want, _ in jobs:
        assert torch.equal(y, want)
    assert B.sqz_fp8_status() == 0


def test_binding_refusals(B):
    f = dict(device="cuda")
    a, w = torch.zeros((4, 256), dtype=E4M3, **f), torch.zeros((130, 256), dtype=E4M3, **f)
    sa, sw, y = torch.ones((4, 2), **f), torch.ones((2, 2), **f), torch.full((4, 130), 3.0, **f)
    for bad in (dict(a=a[:, :255]), dict(w=w[:, :128]), dict(sa=sa[:3]), dict(sw=sw[:1]), dict(sa=sa.half()),
                dict(y=y[:, :129]), dict(y=y.t()), dict(y=y.double()), dict(a=a.cpu()), dict(sw=sw.cpu()),
                dict(a=a.to(torch.float16)), dict(w=torch.zeros((256, 130), dtype=torch.uint8, **f).view(E4M3).t()),
                dict(a=torch.zeros((4, 260), dtype=torch.uint8, **f).view(E4M3)[:, 2:258])):
        v = dict(a=a, sa=sa, w=w, sw=sw, y=y)
        v.update(bad)
        with pytest.raises((ValueError, TypeError, B.SqzError)):
            B.sqz_fp8_gemm(v["a"], v["sa"], v["w"], v["sw"], v["y"])
    torch.cuda.synchronize()
    assert bool((y == 3).all())
    B.sqz_fp8_gemm(a[:1], sa[:1], w[:1], sw[:1], y[:1, :1])  # single rows: any pitch
    assert float(y[0, 0]) == 0


def test_status_refuses_a_capture_and_leaves_it_intact(B):
    x, y = torch.ones(4, device="cuda"), torch.zeros(4, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(B.SqzError) as e:
            B.sqz_fp8_status()
        assert e.value.status == B.SQZ_ERR_UNSUPPORTED
        y.add_(x)
    graph.replay()
    assert bool((y == 1).all())


# shapes for the few-row kernel's three tile sizes and the many-row kernel, in and across W's blocks of rows
SCALE_SHAPES = [(4, 333, 700), (20, 333, 700), (50, 333, 700), (700, 1000, 2200), (300, 5000, 2500)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n,k", SCALE_SHAPES)
def test_product_of_small_scales(B, m, n, k, dtype):
    """Scales about 2^-72, whose products are below fp32's normal numbers while the results are not."""
    gen = torch.Generator().manual_seed(18)
    a, sa = random_matrix(gen, m, k, E4M3, 1)
    w, sw = random_matrix(gen, n, k, E4M3, 128)
    for q in (a, w):  # of one sign, so that the products' errors do not average out
        q.view(torch.uint8).bitwise_and_(0x7F)
    sa, sw = sa * 2.0 ** -65, sw * 2.0 ** -65  # (random_matrix: about 1/100)
    y = torch.empty((m, n), dtype=dtype, device="cuda")
    B.sqz_fp8_gemm(a, sa, w, sw, y)
    check_product(y, a, sa, w, sw)


@pytest.mark.parametrize("m,n,k", SCALE_SHAPES)
def test_product_of_large_scales(B, m, n, k):
    """Scales about 2^65 with the smallest codes: the scales' products are beyond fp32, the results are not, and a
    row of zeros stays zero."""
    gen = torch.Generator().manual_seed(19)

    def few_codes(rows, block_rows):
        q, s = random_matrix(gen, rows, k, E4M3, block_rows)
        small = (torch.rand((rows, k), generator=gen) < 0.02) * torch.randint(1, 3, (rows, k), generator=gen)
        q.view(torch.uint8).copy_((small + 128 * torch.randint(0, 2, (rows, k), generator=gen)).to(torch.uint8))
        return q, s * 2.0 ** 71

    (a, sa), (w, sw) = few_codes(m, 1), few_codes(n, 128)
    a.view(torch.uint8)[1] = 0
    y = torch.empty((m, n), device="cuda")
    B.sqz_fp8_gemm(a, sa, w, sw, y)
    check_product(y, a, sa, w, sw)
    assert bool((y[1] == 0).all())


@pytest.mark.parametrize("m,n,k", SCALE_SHAPES)
def test_product_of_scales_of_every_size(B, m, n, k):
    """Each row of A and each block of rows of W at its own power of two, so that products inside and outside
    fp32's range stand side by side; a scale of zero makes its part zero."""
    gen = torch.Generator().manual_seed(20)
    a, sa = random_matrix(gen, m, k, E4M3, 1)
    w, sw = random_matrix(gen, n, k, E4M3, 128)
    for s in (sa, sw):
        s *= torch.exp2(torch.randint(-78, 45, (s.shape[0], 1), generator=gen).float()).cuda()
    sa[2, 1] = 0
    y = torch.empty((m, n), device="cuda")
    B.sqz_fp8_gemm(a, sa, w, sw, y)
    # results below fp32's normal numbers are rounded to a step of 2^-149, once for each block
    A, W = dense(a, sa, 1), dense(w, sw, 128)
    ref, S = A @ W.t(), A.abs() @ W.abs().t()
    blocks = sa.shape[1]
    tol = (2.0 ** -16 + (blocks + 4) * 2.0 ** -24) * S + blocks * 2.0 ** -149
    bad = ~((y.double() - ref).abs() <= tol)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4].tolist())


@pytest.mark.parametrize("m,n", [(5, 1000), (40, 4096), (600, 2000)])
def test_each_call_reads_what_the_call_before_it_wrote(B, m, n):
    """Product, quantizer of its result, product of that, over and over in the same buffers without a pause:
    the same bits as with every call waited for."""
    gen = torch.Generator().manual_seed(21)
    xs = [torch.randn((m, n), generator=gen).bfloat16().cuda() for _ in range(4)]
    w, sw = random_matrix(gen, n, n, E4M3, 128)
    sw *= n ** -0.5
    q = torch.empty((m, (n + 15) // 16 * 16), dtype=E4M3, device="cuda")[:, :n]
    s, y = torch.empty((m, -(-n // 128)), device="cuda"), torch.empty((m, n), dtype=torch.bfloat16, device="cuda")

    def chain(x, wait):
        for step in range(3):
            B.sqz_fp8_quantize(y if step else x, q=q, scale=s)
            wait()
            B.sqz_fp8_gemm(q, s, w, sw, y)
            wait()
        out = [y.clone(), q.clone(), s.clone()]
        wait()
        return out

    want = [chain(x, torch.cuda.synchronize) for x in xs]
    for _ in range(10):
        got = [chain(x, lambda: None) for x in xs]
        for a, b in zip(want, got):
            assert torch.equal(a[0], b[0]) and same_codes(a[1], b[1]) and torch.equal(a[2], b[2])


@pytest.mark.parametrize("dtype,fmt", [(torch.float16, E4M3), (torch.bfloat16, E5M2)])
@pytest.mark.parametrize("batch,rows,cols,extra", [
    (1, 20011, 100, 0),    # one block a row: a lane's next block is four rows on
    (1, 20011, 100, 1),
    (1, 5000, 777, 0),     # rows at odd offsets
    (1, 5000, 776, 2),     # rows on 4 bytes
    (3, 1700, 650, 6),     # ... of a batch with a pitch, a count of blocks that is no multiple of anything
    (1, 5000, 772, 0),     # on 8 bytes
    (1, 9601, 256, 0),     # whole blocks, an odd number of them
    (1, 4100, 13824, 0),   # more blocks than the grid takes in one step
    (2, 2050, 13700, 4),   # the same with edges
])
def test_quantize_of_more_blocks_than_the_sms_hold_at_once(B, batch, rows, cols, extra, dtype, fmt):
    """1 x 128 blocks beyond 128 for each SM take two blocks a lane and stride over the grid."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert batch * rows * -(-cols // 128) > 128 * sms
    gen = torch.Generator().manual_seed(rows + cols + extra)
    x = make_x(gen, (batch, rows, cols + extra), dtype, "wide")[:, :, :cols]
    qb = torch.full((batch, rows, (cols + 15) // 16 * 16 + 16), 7, dtype=torch.uint8, device="cuda").view(fmt)
    sb = torch.full((batch, rows, -(-cols // 128) + 1), -1.0, device="cuda")
    xd = torch.empty((batch, rows, cols + extra), dtype=dtype, device="cuda")[:, :, :cols]
    xd.copy_(x)
    B.sqz_fp8_quantize(xd, 1, q=qb[:, :, :cols], scale=sb[:, :, :-1])
    q_ref, s_ref = quantize_ref(x, 1, fmt)
    assert torch.equal(sb[:, :, :-1].cpu(), s_ref) and same_codes(qb[:, :, :cols].cpu(), q_ref)
    assert bool((qb.view(torch.uint8)[:, :, cols:] == 7).all()) and bool((sb[:, :, -1] == -1).all())


@pytest.mark.parametrize("fmt", [E4M3, E5M2])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_at_every_alignment_of_the_rows(B, block_rows, dtype, fmt):
    """Rows on 16, 8, 4 and 2 bytes, by their pitch and by their start, whole blocks and edges."""
    gen = torch.Generator().manual_seed(22)
    for cols in (256, 331):
        for off, ldx in ((0, 336), (8, 352), (0, 340), (4, 336), (0, 338), (2, 336), (6, 344), (0, 337), (1, 336), (3, 339)):
            big = make_x(gen, (off + 131 * ldx,), dtype, "wide")
            x = big.cuda()[off:].view(131, ldx)[:, :cols]
            q, s = B.sqz_fp8_quantize(x, block_rows, fmt)
            q_ref, s_ref = quantize_ref(big[off:].view(131, ldx)[:, :cols][None], block_rows, fmt)
            assert torch.equal(s.cpu(), s_ref[0]) and same_codes(q.cpu(), q_ref[0]), (cols, off, ldx)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("m,n,k", SCALE_SHAPES)
def test_product_with_one_scale_that_is_not_finite(B, m, n, k, value):
    """Finite codes under a scale that is NaN or infinite, in A and in W, next to scales of every size: NaN, or infinite
    (NaN where a block's sum is zero), in the outputs it enters, and the others as they are."""
    gen = torch.Generator().manual_seed(23)
    a, sa = random_matrix(gen, m, k, E4M3, 1)
    w, sw = random_matrix(gen, n, k, E4M3, 128)
    for big in (0, 60):  # products in range, and some that are not
        A, W = sa.clone(), sw.clone()
        A[0] *= 2.0 ** -big
        W[0] *= 2.0 ** -big
        A[2, 3], W[1, 4] = value, value
        y = torch.empty((m, n), device="cuda")
        B.sqz_fp8_gemm(a, A, w, W, y)
        hit = torch.zeros((m, n), dtype=torch.bool, device="cuda")
        hit[2], hit[:, 128:256] = True, True
        if value != value:
            assert bool(y[hit].isnan().all())
        else:
            assert not bool(y[hit].isfinite().any()) and bool(y[2, :128].isinf().any())
        assert bool(y[~hit].isfinite().all())
