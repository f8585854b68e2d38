"""GPU tests of the 8-bit product's kernel for many rows: every tile width with several runs of scales and a ring of
stages that goes round, formats, types, pitches and alignments, NaN, repetition, graphs, streams and offsets
beyond 32 bits.  Bound: tests/test_gpu_fp8.py.  tests/test_fp8_plan.py checks (without a GPU) that the shapes reach
the kernel."""
import pytest
import torch

from test_gpu_fp8 import E4M3, E5M2, check_product, quantize_ref, random_matrix, same_codes

pytestmark = pytest.mark.gpu

# width of the tiles, m, n, k
SHAPES = [
    (64, 700, 1000, 2200), (64, 2500, 301, 2200), (128, 1000, 2223, 4200), (160, 2000, 1337, 2500),
    (192, 290, 6901, 2200), (192, 2000, 5001, 2200), (256, 256, 18001, 2200), (256, 3000, 2500, 2200),
]
SMALLER = [s for s in SHAPES if s[1:] not in ((2500, 301, 2200), (2000, 5001, 2200), (3000, 2500, 2200))]  # one a width


@pytest.fixture(scope="module")
def B():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from lut_dequant_gemv_b200 import binding, build

    build.build()
    binding.lib()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for width, m, n, k in SHAPES:
        p = binding.sqz_fp8_plan_query(m, n, k, sms)
        assert p["many_rows"] == 1 and p["tile_cols"] == width
    return binding


def operands(seed, m, n, k, fa=E4M3, fw=E4M3, **pitch):
    gen = torch.Generator().manual_seed(seed)
    return (*random_matrix(gen, m, k, fa, 1, **pitch), *random_matrix(gen, n, k, fw, 128, **pitch))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("width,m,n,k", SHAPES)
def test_sizes_and_types(B, width, m, n, k, dtype):
    a, sa, w, sw = operands(31, m, n, k)
    y = torch.full((m, n), float("nan"), dtype=dtype, device="cuda")
    B.sqz_fp8_gemm(a, sa, w, sw, y)
    check_product(y, a, sa, w, sw)
    assert B.sqz_fp8_status() == 0


@pytest.mark.parametrize("fa,fw", [(E5M2, E4M3), (E4M3, E5M2), (E5M2, E5M2)])
@pytest.mark.parametrize("width,m,n,k", SMALLER)
def test_formats(B, width, m, n, k, fa, fw):
    a, sa, w, sw = operands(32, m, n, k, fa, fw)
    y = torch.empty((m, n), device="cuda")
    B.sqz_fp8_gemm(a, sa, w, sw, y)
    check_product(y, a, sa, w, sw)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("width,m,n,k", SMALLER)
def test_rows_of_y_at_every_alignment(B, width, m, n, k, dtype):
    """Rows of y on 32 and 16 bytes and on 8, 4 and 2 (stores of up to 4, 2 and 1 values), operands and scales with
    pitches of their own; what lies before y, between its rows and behind the last one stays."""
    a, sa, w, sw = operands(33, m, n, k, pitch_extra=48)
    wide = torch.full((m, sa.shape[1] + 3), float("nan"), device="cuda")
    wide[:, : sa.shape[1]] = sa
    up = -(-n // 16) * 16
    first = None
    for off, ldy in ((0, up + 16), (0, up + 8), (4, up + 4), (2, up + 2), (1, up + 1)):
        buf = torch.full(((m + 2) * ldy + off,), -7.0, dtype=dtype, device="cuda")
        y = buf[off:].view(m + 2, ldy)
        B.sqz_fp8_gemm(a, wide[:, : sa.shape[1]], w, sw, y[:m, :n])
        if first is None:
            first = y[:m, :n].clone()
            check_product(first, a, sa, w, sw)
        assert torch.equal(y[:m, :n], first), (off, ldy)
        assert bool((y[:m, n:] == -7).all()) and bool((y[m:] == -7).all()) and bool((buf[:off] == -7).all()), (off, ldy)


@pytest.mark.parametrize("width,m,n,k", SMALLER)
def test_nan_codes_and_scales(B, width, m, n, k):
    """In the second run of scales: a code of A, a code of W, a scale of each."""
    a, sa, w, sw = operands(34, m, n, k)
    a.view(torch.uint8)[2, 2100] = 0x7F
    w.view(torch.uint8)[200, 2150] = 0xFF
    sa[m - 1, 16] = float("inf")
    sw[1, 16] = float("nan")  # columns 128 .. 255
    y = torch.empty((m, n), device="cuda")
    B.sqz_fp8_gemm(a, sa, w, sw, y)
    assert bool(y[2].isnan().all()) and not bool(y[m - 1].isfinite().any()) and bool(y[:, 128:256].isnan().all())
    rest = torch.cat([y[:, :128], y[:, 256:]], dim=1)
    keep = torch.ones(m, dtype=torch.bool, device="cuda")
    keep[2] = keep[m - 1] = False
    assert bool(rest[keep].isfinite().all())


@pytest.mark.parametrize("width,m,n,k", SHAPES)
def test_the_same_bits_every_time(B, width, m, n, k):
    a, sa, w, sw = operands(35, m, n, k)
    ys = [torch.empty((m, n), device="cuda") for _ in range(6)]
    for y in ys:
        B.sqz_fp8_gemm(a, sa, w, sw, y)
    assert all(torch.equal(ys[0], y) for y in ys[1:])


def test_quantized_on_another_stream_and_replayed(B):
    m, n, k = 700, 1000, 2200
    gen = torch.Generator().manual_seed(36)
    xs = [torch.randn((m, k), generator=gen).bfloat16().cuda() for _ in range(3)]
    w, sw = random_matrix(gen, n, k, E4M3, 128)
    want = []
    for x in xs:
        q, s = B.sqz_fp8_quantize(x)
        y = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
        B.sqz_fp8_gemm(q, s, w, sw, y)
        check_product(y, q, s, w, sw)
        want.append(y)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        q, s = B.sqz_fp8_quantize(xs[0])
        y_out = torch.empty_like(want[0])
        B.sqz_fp8_gemm(q, s, w, sw, y_out)
    side.synchronize()
    assert torch.equal(y_out, want[0])
    x_in, graph = torch.empty_like(xs[0]), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.sqz_fp8_quantize(x_in, q=q, scale=s)
        B.sqz_fp8_gemm(q, s, w, sw, y_out)
    for x, y in zip(xs, want):
        x_in.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y_out, y)


def test_beside_other_products(B):
    """Every width on a stream of its own, at once, next to a product of few rows."""
    jobs = []
    for i, (m, n, k) in enumerate([s[1:] for s in SMALLER] + [(40, 3000, 4000)]):
        a, sa, w, sw = operands(37 + i, m, n, k)
        want = torch.empty((m, n), device="cuda")
        B.sqz_fp8_gemm(a, sa, w, sw, want)
        jobs.append((a, sa, w, sw, torch.zeros_like(want), want, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for a, sa, w, sw, y, _, stream in jobs:
            B.sqz_fp8_gemm(a, sa, w, sw, y, stream=stream)
    torch.cuda.synchronize()
    for *_, y, want, _ in jobs:
        assert torch.equal(y, want)
    assert B.sqz_fp8_status() == 0


def test_offsets_beyond_32_bits(B):
    """Pitches that put the last rows of codes, scales and y more than 2^32 bytes from the first."""
    m, n, k = 700, 1000, 2200
    gen = torch.Generator().manual_seed(43)
    x = torch.randn((m, k), generator=gen).bfloat16()
    ld = (1 << 32) // m // 16 * 16 + 64
    blocks = -(-k // 128)
    q = torch.empty((m + 1) * ld, dtype=torch.uint8, device="cuda").view(E4M3).view(m + 1, ld)[:m, :k]
    s = torch.empty((m + 1) * (ld // 4), device="cuda").view(m + 1, ld // 4)[:m, :blocks]
    B.sqz_fp8_quantize(x.cuda(), q=q, scale=s)
    q_ref, s_ref = quantize_ref(x[None], 1, E4M3)
    assert torch.equal(s.cpu(), s_ref[0]) and same_codes(q.cpu(), q_ref[0])
    w, sw = random_matrix(gen, n, k, E4M3, 128)
    ld_w = (1 << 32) // n // 16 * 16 + 64
    w_far = torch.empty((n + 1) * ld_w, dtype=torch.uint8, device="cuda").view(E4M3).view(n + 1, ld_w)[:n, :k]
    w_far.view(torch.uint8).copy_(w.view(torch.uint8))
    for odd in (0, 1):  # rows of y on 16 bytes, and turned
        ldy = ld // 4 + odd
        y = torch.empty((m + 1) * ldy, device="cuda").view(m + 1, ldy)[:m, :n]
        B.sqz_fp8_gemm(q, s, w_far, sw, y)
        check_product(y, q, s, w, sw)


def test_few_rows_of_a_matrix_wider_than_a_grid(B):
    """More blocks of 128 rows of W than a grid's second dimension has: the many-row kernel, with two rows of A."""
    m, n, k = 2, 65535 * 128 + 1, 20
    assert B.sqz_fp8_plan_query(m, n, k)["many_rows"] == 1 and B.sqz_fp8_plan_query(m, n - 1, k)["many_rows"] == 0
    a, sa, w, sw = operands(44, m, n, k)
    for cols in (n, n - 1):
        y = torch.full((m, cols), float("nan"), device="cuda")
        B.sqz_fp8_gemm(a, sa, w[:cols], sw[: -(-cols // 128)], y)
        check_product(y, a, sa, w[:cols], sw[: -(-cols // 128)])
