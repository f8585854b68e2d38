"""GPU tests of the mixture-of-experts layer against its definition in fp64.

Error bound per output, carried through the layer (all terms computed in fp64):
  * a product of K terms: 2^-16 S for the tensor cores' sums of 128 exact
    products (at most one fp32 step, 2^-23, per addition) and (blocks + 8) 2^-24
    S for the digits' joining, the scales and the blocks' additions, S = sum
    |w v|; the digits of an operand leave out at most 2^-29 of the largest
    value of its block of 128, so 2^-29 max|v| sum |w| more;
  * h = silu(gate) up: |silu'| <= 1.1, |silu(g)| <= |g|; exp, the division and
    the product are off by at most 2^-21 relative; four digits leave out at
    most 2^-18 of a value;
  * a logit is summed in fp32 by 32 lanes, hidden / 32 terms each and five
    joins: off by d <= (hidden / 32 + 5) 2^-24 S_l, S_l = sum |r x|.  A weight
    exp(l - top) / sum of such (and, renormalized, a quotient of two of them)
    is then off by at most 4 d relative, exp, sums and divisions adding 2^-20;
  * pieces joined: 200 additions, 200 * 2^-24; y's rounding: half a step.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def B():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from lut_dequant_gemv_b200 import binding, build

    build.build()
    binding.lib()
    return binding


def up(a, b):
    return -(-a // b)


class Case:
    def __init__(self, experts, hidden, inter, dtype, seed=0, router_scale=1.5):
        g = torch.Generator().manual_seed(seed + experts * 31 + hidden + inter)
        self.experts, self.hidden, self.inter, self.dtype = experts, hidden, inter, dtype

        def codes(*shape):
            return (torch.randn(shape, generator=g) * 100).clamp(-448, 448).to(E4M3).cuda()

        def scales(k, *shape):
            return ((0.5 + torch.rand(shape, generator=g)) * k ** -0.5 / 100).cuda()

        bi, bh = up(inter, 128), up(hidden, 128)
        self.router = (torch.randn((experts, hidden), generator=g) * router_scale * hidden ** -0.5).to(dtype).cuda()
        self.w13, self.s13 = codes(experts, 2 * inter, hidden), scales(hidden, experts, 2, bi, bh)
        self.w2, self.s2 = codes(experts, hidden, inter), scales(inter, experts, bh, bi)
        self.gen = g

    def x(self, tokens, scale=1.0):
        return (torch.randn((tokens, self.hidden), generator=self.gen) * scale).to(self.dtype).cuda()

    def handle(self, B, top_k, renormalize=True):
        return B.sqz_create_moe(self.router, self.w13, self.s13, self.w2, self.s2, top_k=top_k,
                                renormalize=renormalize)

    def weights(self, e):
        bi = torch.arange(self.inter, device="cuda") // 128
        bh = torch.arange(self.hidden, device="cuda") // 128
        w1 = self.w13[e, : self.inter].double() * self.s13[e, 0].double()[bi][:, bh]
        w3 = self.w13[e, self.inter:].double() * self.s13[e, 1].double()[bi][:, bh]
        return w1, w3, self.w2[e].double() * self.s2[e].double()[bh][:, bi]

    def reference(self, x, top_k, renormalize):
        x = x.double()
        logits = x @ self.router.double().t()
        order = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :top_k]
        g = torch.softmax(logits, dim=1).gather(1, order)
        if renormalize:
            g = g / g.sum(1, keepdim=True)
        S_l = (x.abs() @ self.router.double().abs().t()).amax(1, keepdim=True)
        self.weight_error = 4 * (self.hidden / 32 + 5) * 2.0 ** -24 * S_l + 2.0 ** -20  # relative, per token
        y, err = torch.zeros_like(x), torch.zeros_like(x)
        r1 = 2.0 ** -16 + (up(self.hidden, 128) + 8) * 2.0 ** -24
        r2 = 2.0 ** -16 + (up(self.inter, 128) + 8) * 2.0 ** -24
        for e in order.unique().tolist():
            tok, slot = (order == e).nonzero(as_tuple=True)
            w1, w3, w2 = self.weights(e)
            v = x[tok]
            big = v.abs().amax(1, keepdim=True) * 2.0 ** -29
            gate, upv = v @ w1.t(), v @ w3.t()
            eg = r1 * (v.abs() @ w1.abs().t()) + big * w1.abs().sum(1)
            eu = r1 * (v.abs() @ w3.abs().t()) + big * w3.abs().sum(1)
            silu = gate / (1 + torch.exp(-gate))
            h = silu * upv
            eh = 1.1 * eg * (upv.abs() + eu) + silu.abs() * eu + h.abs() * (2.0 ** -21 + 2.0 ** -18)
            eh = eh + 2.0 ** -29 * (h.abs() + eh).amax(1, keepdim=True)
            out = h @ w2.t()
            eo = eh @ w2.abs().t() + r2 * ((h.abs() + eh) @ w2.abs().t())
            wt = g[tok, slot, None]
            y.index_add_(0, tok, out * wt)
            ew = self.weight_error[tok]
            err.index_add_(0, tok, wt * (eo * (1 + ew) + (ew + 200 * 2.0 ** -24) * (h.abs() @ w2.abs().t())))
        return y, err, order, g


def check(B, case, x, top_k, renormalize=True, moe=None, ws=None):
    tokens = x.shape[0]
    moe = moe or case.handle(B, top_k, renormalize)
    ws = B.sqz_moe_workspace(moe, tokens) if ws is None else ws
    y = torch.full((tokens, case.hidden), float("nan"), dtype=case.dtype, device="cuda")
    ids = torch.full((tokens, top_k), -1, dtype=torch.int32, device="cuda")
    g = torch.full((tokens, top_k), -1.0, device="cuda")
    B.sqz_moe_forward(moe, x, y, ids=ids, weights=g, workspace=ws)
    assert B.sqz_moe_status(ws) == 0
    ref, err, order, g_ref = case.reference(x, top_k, renormalize)
    assert torch.equal(ids.long(), order)
    assert bool(((g.double() - g_ref).abs() <= case.weight_error * g_ref).all())
    fi = torch.finfo(case.dtype)
    tol = err + (ref.abs() + err) * fi.eps / 2 + (2.0 ** -25 if case.dtype == torch.float16 else 0)
    off = (y.double() - ref).abs()
    bad = ~(off <= tol)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4].tolist(), float((off / tol).max()))
    return y


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tokens,experts,top_k,hidden,inter", [
    (1, 1, 1, 16, 16), (1, 2, 1, 128, 128), (1, 4, 2, 256, 384), (2, 8, 2, 1040, 272), (1, 64, 6, 2048, 256),
    (4, 16, 4, 512, 1008), (5, 5, 5, 144, 400), (8, 128, 8, 1024, 128), (17, 8, 2, 640, 656), (32, 16, 4, 256, 512),
    (32, 1, 1, 512, 256), (31, 3, 3, 272, 144), (32, 1024, 16, 128, 16), (9, 40, 16, 384, 128),
])
def test_sizes(B, tokens, experts, top_k, hidden, inter, dtype):
    case = Case(experts, hidden, inter, dtype)
    check(B, case, case.x(tokens), top_k)


@pytest.mark.parametrize("renormalize", [False, True])
def test_weights_of_the_choice(B, renormalize):
    case = Case(12, 256, 128, torch.bfloat16, seed=3)
    check(B, case, case.x(7), 3, renormalize)


def test_equal_logits_go_to_the_lowest_expert(B):
    case = Case(40, 128, 64, torch.float16, seed=4)
    case.router.zero_()
    moe = case.handle(B, 4)
    x = case.x(3)
    check(B, case, x, 4, moe=moe)
    case.router[37] = case.router[5] = x[0]  # two experts tie for the first place of token 0
    ids = torch.empty((3, 4), dtype=torch.int32, device="cuda")
    B.sqz_moe_forward(moe, x, torch.empty_like(x), ids=ids, workspace=B.sqz_moe_workspace(moe, 3))
    assert ids[0].tolist() == [5, 37, 0, 1]


@pytest.mark.parametrize("dtype,scale", [(torch.float16, 1e-4), (torch.float16, 300.0), (torch.bfloat16, 1e-12),
                                         (torch.bfloat16, 1e4)])
def test_small_and_large_activations(B, dtype, scale):
    case = Case(4, 384, 256, dtype, seed=5, router_scale=0.5 / max(scale, 1.0))
    if scale > 1:  # keeps y inside the type's range
        case.s2 /= scale * scale
    check(B, case, case.x(3, scale), 2)


def test_one_large_value_among_small_ones(B):
    """The digits' error is relative to the largest of a block, within the bound."""
    case = Case(4, 384, 256, torch.float16, seed=6)
    x = case.x(2) * 0.01
    x[:, 70] = 500.0
    check(B, case, x.half(), 2)


def test_other_rows_strides_and_reuse_of_the_workspace(B):
    """One workspace for calls of fewer and more tokens; x and y with pitches, unaligned; rows around y stay."""
    case = Case(8, 272, 208, torch.bfloat16, seed=7)
    moe = case.handle(B, 3)
    ws = B.sqz_moe_workspace(moe, 32)
    for tokens in (32, 1, 7, 32, 2):
        check(B, case, case.x(tokens), 3, moe=moe, ws=ws)
    xb = torch.zeros((6 * 301 + 1,), dtype=torch.bfloat16, device="cuda")
    x = xb[1:].view(6, 301)[:, :272]
    x.copy_(case.x(6))
    yb = torch.full((8 * 303 + 1,), -3.0, dtype=torch.bfloat16, device="cuda")
    rows = yb[1:].view(8, 303)
    B.sqz_moe_forward(moe, x, rows[1:7, :272], workspace=ws)
    want = torch.empty((6, 272), dtype=torch.bfloat16, device="cuda")
    B.sqz_moe_forward(moe, x.contiguous(), want, workspace=ws)
    assert torch.equal(rows[1:7, :272], want)
    assert bool((rows[0] == -3).all()) and bool((rows[7] == -3).all()) and bool((rows[:, 272:] == -3).all())


def test_same_bits_every_time_and_alone_or_in_a_batch(B):
    case = Case(16, 512, 384, torch.float16, seed=8)
    moe = case.handle(B, 4)
    ws = B.sqz_moe_workspace(moe, 16)
    x = case.x(16)
    ys = [torch.empty_like(x) for _ in range(4)]
    for y in ys:
        B.sqz_moe_forward(moe, x, y, workspace=ws)
    assert all(torch.equal(ys[0], y) for y in ys[1:])


def test_not_finite_tokens_leave_the_others_alone(B):
    case = Case(8, 256, 256, torch.float16, seed=9)
    moe = case.handle(B, 2)
    x = case.x(5)
    want = check(B, case, x, 2, moe=moe)
    x2 = x.clone()
    x2[1, 7], x2[3, 200] = float("nan"), float("inf")
    ws = B.sqz_moe_workspace(moe, 5)
    y, ids = torch.empty_like(x), torch.full((5, 2), -1, dtype=torch.int32, device="cuda")
    B.sqz_moe_forward(moe, x2, y, ids=ids, workspace=ws)
    assert B.sqz_moe_status(ws) == 0
    assert bool(y[1].isnan().all()) and bool(y[3].isnan().all())
    assert bool(((ids >= 0) & (ids < 8)).all())
    fi = torch.finfo(torch.float16)
    for t in (0, 2, 4):  # the cut of the work may differ, so the last bits may
        assert bool(((y[t].double() - want[t].double()).abs() <= 4 * fi.eps * want[t].abs().max().double()).all())
    B.sqz_moe_forward(moe, x, y, workspace=ws)  # and the workspace is as good as new
    assert torch.equal(y, want)


def test_in_a_graph_and_on_two_streams(B):
    case = Case(16, 512, 384, torch.bfloat16, seed=10)
    moe = case.handle(B, 4)
    xs = [case.x(4) for _ in range(4)]
    want = [check(B, case, x, 4, moe=moe) for x in xs]
    ws = [B.sqz_moe_workspace(moe, 4) for _ in range(2)]
    ys = [torch.empty_like(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for rep in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                B.sqz_moe_forward(moe, xs[i], ys[i], workspace=ws[i])
    torch.cuda.synchronize()
    assert torch.equal(ys[0], want[0]) and torch.equal(ys[1], want[1])
    x_in, y_out = torch.empty_like(xs[0]), torch.empty_like(xs[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.sqz_moe_forward(moe, x_in, y_out, workspace=ws[0])
    for x, y in zip(xs, want):
        x_in.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y_out, y)
    assert B.sqz_moe_status(ws[0]) == 0


def test_quantized_experts_end_to_end(B):
    """fp16 experts quantized by sqz_fp8_quantize, one expert for every token, against the same MLP built from
    sqz_fp8_gemm calls on the same codes (which rounds its activations to 8 bits: half a step, 2^-4, each time)."""
    g = torch.Generator().manual_seed(11)
    hidden, inter, experts = 256, 272, 3
    w13f = (torch.randn((experts * 2, inter, hidden), generator=g) * hidden ** -0.5).half().cuda()
    w2f = (torch.randn((experts, hidden, inter), generator=g) * inter ** -0.5).half().cuda()
    w13, s13 = B.sqz_fp8_quantize(w13f, 128)
    w2, s2 = B.sqz_fp8_quantize(w2f, 128)
    router = torch.randn((experts, hidden), generator=g).half().cuda()
    moe = B.sqz_create_moe(router, w13.view(experts, 2 * inter, hidden), s13.view(experts, 2, 3, 2), w2, s2, top_k=1)
    x = torch.randn((6, hidden), generator=g).half().cuda()
    y, ids = torch.empty_like(x), torch.empty((6, 1), dtype=torch.int32, device="cuda")
    B.sqz_moe_forward(moe, x, y, ids=ids, workspace=B.sqz_moe_workspace(moe, 6))
    for t in range(6):
        e = int(ids[t, 0])
        a, sa = B.sqz_fp8_quantize(x[t:t + 1])
        gu = [torch.empty((1, inter), device="cuda") for _ in range(2)]
        for half in range(2):
            B.sqz_fp8_gemm(a, sa, w13.view(experts, 2, inter, hidden)[e, half], s13.view(experts, 2, 3, 2)[e, half], gu[half])
        h = (torch.nn.functional.silu(gu[0]) * gu[1]).half()
        q, sq = B.sqz_fp8_quantize(h)
        out = torch.empty((1, hidden), device="cuda")
        B.sqz_fp8_gemm(q, sq, w2[e], s2[e], out)
        rel = (out - y[t:t + 1].float()).norm() / y[t:t + 1].float().norm()
        # three 8-bit roundings meet (x in gate and up, h), each at most 2^-4 of its operand; norms of random
        # sums scale with the operands' relative error, |silu'| <= 1.1
        assert float(rel) <= (1.1 + 1 + 1) * 2.0 ** -4
    moe.close()


def test_forward_refusals(B):
    """Refused on the host: nothing is launched, y stays as it was."""
    import ctypes

    case = Case(4, 128, 64, torch.float16, seed=12)
    moe = case.handle(B, 2)
    x, y = case.x(2), torch.full((2, 128), 5.0, dtype=torch.float16, device="cuda")
    ws = B.sqz_moe_workspace(moe, 2)
    n = ctypes.c_int64()
    for tokens in (0, 33, -1):
        assert B.lib().sqz_moe_workspace_bytes(moe, tokens, ctypes.byref(n)) == B.SQZ_ERR_INVALID_ARG

    def call(**kw):
        a = dict(x=x.data_ptr(), tokens=2, ldx=128, y=y.data_ptr(), ldy=128, ws=ws.data_ptr(), size=ws.numel())
        a.update(kw)
        return B.lib().sqz_moe_forward(moe, a["x"], a["tokens"], a["ldx"], a["y"], a["ldy"], None, None, a["ws"],
                                       a["size"], None)

    for kw in (dict(x=None), dict(y=None), dict(ws=None), dict(tokens=33), dict(tokens=-1), dict(ldx=127),
               dict(ldy=100), dict(size=ws.numel() - 1), dict(ws=ws.data_ptr() + 16), dict(x=x.data_ptr() + 1)):
        assert call(**kw) == B.SQZ_ERR_INVALID_ARG, kw
    assert call(tokens=0) == B.SQZ_OK
    torch.cuda.synchronize()
    assert bool((y == 5).all())
    for bad in (dict(workspace=None), dict(workspace=ws[:100]), dict(workspace=ws, ids=torch.empty(2, 2, device="cuda")),
                dict(workspace=ws.cpu())):
        with pytest.raises((ValueError, B.SqzError)):
            B.sqz_moe_forward(moe, x, y, **bad)
    with pytest.raises(ValueError):
        B.sqz_moe_forward(moe, x.bfloat16(), y, workspace=ws)


def test_experts_beyond_32_bits(B):
    """Weights of more than 2^32 bytes: the last expert of many is the one expert of a small layer."""
    experts, hidden, inter = 70, 8192, 4096
    one = Case(1, hidden, inter, torch.bfloat16, seed=13)
    x = one.x(2)
    want = torch.empty_like(x)
    small = one.handle(B, 1)
    B.sqz_moe_forward(small, x, want, workspace=B.sqz_moe_workspace(small, 2))
    f = dict(device="cuda")
    w13 = torch.zeros((experts, 2 * inter, hidden), dtype=torch.uint8, **f).view(E4M3)
    w2 = torch.zeros((experts, hidden, inter), dtype=torch.uint8, **f).view(E4M3)
    s13 = torch.ones((experts, 2, inter // 128, hidden // 128), **f)
    s2 = torch.ones((experts, hidden // 128, inter // 128), **f)
    router = torch.zeros((experts, hidden), dtype=torch.bfloat16, **f)
    w13[-1], s13[-1], w2[-1], s2[-1] = one.w13[0], one.s13[0], one.w2[0], one.s2[0]
    router[-1] = x[0]
    x2 = x[:1].repeat(2, 1)
    big = B.sqz_create_moe(router, w13, s13, w2, s2, top_k=1)
    ws = B.sqz_moe_workspace(big, 2)
    y, ids = torch.empty_like(x2), torch.empty((2, 1), dtype=torch.int32, **f)
    B.sqz_moe_forward(big, x2, y, ids=ids, workspace=ws)
    assert B.sqz_moe_status(ws) == 0 and ids.flatten().tolist() == [experts - 1] * 2
    fi = torch.finfo(torch.bfloat16)
    for t in range(2):  # one rounding each; the sums are cut alike or not
        assert bool(((y[t].double() - want[0].double()).abs() <= 2 * fi.eps * want[0].double().abs() + 1e-5).all())


def test_padded_batch_and_repeated_rows(B):
    """Rows behind the tokens of a call stay as they are; equal rows give equal results."""
    case = Case(8, 256, 144, torch.float16, seed=14)
    moe = case.handle(B, 2)
    ws = B.sqz_moe_workspace(moe, 32)
    x = case.x(1).repeat(9, 1)
    y = torch.full((12, 256), 4.0, dtype=torch.float16, device="cuda")
    B.sqz_moe_forward(moe, x, y[:9], workspace=ws)
    assert bool((y[9:] == 4).all()) and all(torch.equal(y[0], y[t]) for t in range(1, 9))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tokens,hidden", [(1, 2048), (7, 272), (32, 4096)])
def test_near_equal_logits_go_to_the_larger(B, tokens, hidden, dtype):
    """Experts in pairs whose logits differ by 2^-24, less than fp32 holds of logits about 1: the later one of
    each pair is the larger."""
    case = Case(24, hidden, 32, dtype, seed=15)
    x = case.x(tokens)
    eps = torch.finfo(dtype).eps
    case.router[:, 40] = 1
    case.router[12:] = case.router[:12]
    case.router[12:, 40] += eps
    x[:, 40] = 2.0 ** -24 / eps
    moe = case.handle(B, 10)
    check(B, case, x, 10, moe=moe)
    case.router[12:, 40] -= eps  # and equal ones to the earlier
    check(B, case, x, 10, moe=moe)


@pytest.mark.parametrize("tokens", [1, 6, 32])
def test_scales_whose_products_leave_the_normal_numbers(B, tokens):
    """Weight scales so small (or, with weights of zero, so large) that their products with the activations' powers of
    two are not normal fp32 numbers, where the results are.  Everything is positive, so that errors add up."""
    case = Case(4, 512, 256, torch.bfloat16, seed=16)
    for codes in (case.w13, case.w2):
        codes.view(torch.uint8).bitwise_and_(0x7F)
    gate, up_ = case.s13[:, 0].clone(), case.s13[:, 1].clone()
    case.s13[:, 0], case.s13[:, 1] = gate * 2.0 ** -114, up_ * 2.0 ** 65 * 2.0 ** 65  # gate about 2^-124, up 2^120
    check(B, case, case.x(tokens, 2.0 ** -14).abs(), 2)
    case.s13[:, 0], case.s13[:, 1] = gate, up_ * 2.0 ** -108  # h about 2^-100, y about 2^-124
    case.s2 *= 2.0 ** -28
    check(B, case, case.x(tokens).abs(), 2)
    case.s13[:, 0], case.s13[:, 1] = gate * 2.0 ** -51, up_ * 2.0 ** 121  # gate about 2^-123, h 2^-75
    case.s2 *= 2.0 ** 68
    check(B, case, case.x(tokens, 2.0 ** -75).abs(), 2)
    case.w13.zero_()  # nothing times anything
    case.s13.fill_(2.0 ** 124)
    check(B, case, case.x(tokens, 2.0 ** 20), 2)


@pytest.mark.parametrize("tokens,aligned", [(1, True), (9, False), (32, True)])
def test_in_place(B, tokens, aligned):
    """y may be x."""
    case = Case(16, 512, 384, torch.bfloat16, seed=17)
    moe = case.handle(B, 4)
    ws = B.sqz_moe_workspace(moe, tokens)
    x = case.x(tokens)
    want = check(B, case, x, 4, moe=moe)
    at = 0 if aligned else 1
    buf = torch.zeros(tokens * 512 + at, dtype=torch.bfloat16, device="cuda")
    for _ in range(3):
        both = buf[at:].view(tokens, 512)
        both.copy_(x)
        B.sqz_moe_forward(moe, both, both, workspace=ws)
        assert torch.equal(both, want)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_each_token_alone_and_in_a_batch(B, dtype):
    """The work is cut over the SMs by the experts the whole batch reaches, so a token's sums are added in another order
    beside others: its row agrees within the bound, not bit for bit, and its routing is the same."""
    case = Case(16, 512, 384, dtype, seed=18)
    moe = case.handle(B, 4)
    ws = B.sqz_moe_workspace(moe, 32)
    x = case.x(20)
    y, ids = torch.empty_like(x), torch.empty((20, 4), dtype=torch.int32, device="cuda")
    weights = torch.empty((20, 4), device="cuda")
    B.sqz_moe_forward(moe, x, y, ids=ids, weights=weights, workspace=ws)
    ref, err, _, _ = case.reference(x, 4, True)
    eps = torch.finfo(dtype).eps
    tol = 2 * (err + (ref.abs() + err) * eps / 2 + (2.0 ** -25 if dtype == torch.float16 else 0))  # each side's
    for t in range(20):
        alone, i1, w1 = torch.empty_like(x[:1]), torch.empty_like(ids[:1]), torch.empty_like(weights[:1])
        B.sqz_moe_forward(moe, x[t:t + 1], alone, ids=i1, weights=w1, workspace=ws)
        assert torch.equal(i1, ids[t:t + 1]) and torch.equal(w1, weights[t:t + 1])
        assert bool(((alone[0].double() - y[t].double()).abs() <= tol[t]).all())
