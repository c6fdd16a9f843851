"""The 8-bit linear layer on the GPU against its definition in 64 bits.

Codes and row scales are compared for equality: in fp64 127 x is exact and the
quotient of two 24-bit numbers is at least 2^-34 away from a half-integer that
it does not equal, so rounding the fp64 quotient gives the definition's code.

Outputs: the sum of 8-bit products is exact, its conversion to fp32 and the
two scale products are off by half a step each (2^-24 relative), and so is the
last addition.  A dot product of n terms in fp32, in any order and with
truncating additions (a step each, 2^-23), is off by at most n 2^-23 times the
sum of the terms' magnitudes.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -24


@pytest.fixture(scope="module")
def lbq():
    from qlora_quantized_linear_b200 import lbq as m
    return m


def normal(shape, std, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def ref_rows(v):
    """(codes, fp32 scale) of the rows of v, in fp64."""
    v = v.double()
    amax = v.abs().amax(1, keepdim=True)
    bad = ~torch.isfinite(v).all(1, keepdim=True)
    safe = torch.where((amax == 0) | bad, torch.ones_like(amax), amax)
    codes = torch.where(bad, torch.zeros_like(v), torch.round(127.0 * v / safe))
    # the fp64 quotient rounded again is the correctly rounded fp32 quotient (53 >= 2 * 24 + 2 bits); torch's own
    # fp32 division by a Python number multiplies by a reciprocal
    scale = (torch.where(bad, torch.full_like(amax, float("nan")), amax) / 127.0).float()
    return codes, scale[:, 0]


def guarded(m, n):
    """An output [m, n] inside a buffer of a value that a stray write would change."""
    buf = torch.full((m * n + 2048,), 7.25, device="cuda")
    return buf, buf[1024:1024 + m * n].view(m, n)


def assert_guard(buf, m, n):
    assert bool((buf[:1024] == 7.25).all()) and bool((buf[1024 + m * n:] == 7.25).all()), "wrote outside the output"


def assert_close(got, ref, lim, what):
    got = got.double()
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    err = torch.where(nan, 0.0, (got - ref).abs())
    over = torch.where(nan, 0.0, err - lim).max().item()
    assert over <= 0, f"{what}: off by {err.max().item():.3e}, {over:.3e} over the bound"


def adapter_ref(x, P, Q, s):
    """(x P, bound) and (s x P Q, bound) in fp64: the adapter's saved product and its term."""
    x, P, Q = x.double(), P.double(), Q.double()
    t = x @ P
    tb = 2 * (x.shape[1] + 1) * STEP * (x.abs() @ P.abs())
    term = s * (t @ Q)
    r = P.shape[1]
    mag = abs(s) * ((t.abs() + tb) @ Q.abs())
    return t, tb, term, abs(s) * (tb @ Q.abs()) + (2 * r + 2) * STEP * mag, mag


def check_fwd(lbq, X, codes, scale, A, B, s, **kw):
    m, k = X.shape
    n = codes.shape[0]
    buf, Y = guarded(m, n)
    qw = lbq.Int8Weight(n, k, codes=codes, scale=scale)
    _, T = lbq.linear_i8_fwd(X, qw, A, B, s, Y=Y, **kw)
    torch.cuda.synchronize()
    assert lbq.device_status() == 0
    q, sx = ref_rows(X)
    main = (q @ codes.double().t()) * sx.double()[:, None] * scale.double()[None, :]
    lim = 4 * STEP * main.abs() + 1e-37
    ref = main
    if A is not None:
        t, tb, term, eb, mag = adapter_ref(X, A.t(), B.t(), s)
        assert_close(T, t, tb, "T")
        ref = main + term
        lim = lim + eb + 2 * STEP * mag
    assert_close(Y, ref, lim + STEP * ref.abs(), "Y")
    assert_guard(buf, m, n)
    return Y, T


def check_bwd(lbq, dY, codes, scale, A, B, s, **kw):
    m, n = dY.shape
    k = codes.shape[1]
    buf, dX = guarded(m, k)
    qw = lbq.Int8Weight(n, k, codes=codes, scale=scale)
    _, U = lbq.linear_i8_bwd(dY, qw, A, B, s, dX=dX, **kw)
    torch.cuda.synchronize()
    assert lbq.device_status() == 0
    q, sv = ref_rows(dY.float() * scale[None, :])
    main = (q @ codes.double()) * sv.double()[:, None]
    lim = 3 * STEP * main.abs() + 1e-37
    ref = main
    if A is not None:
        u, ub, term, eb, mag = adapter_ref(dY, B, A, s)
        assert_close(U, u, ub, "U")
        ref = main + term
        lim = lim + eb + 2 * STEP * mag
    assert_close(dX, ref, lim + STEP * ref.abs(), "dX")
    assert_guard(buf, m, k)
    return dX, U


def layer(n, k, rank, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    codes = torch.randint(-127, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    scale = torch.rand(n, generator=g, device="cuda") * 1e-2 + 1e-4
    A = normal((rank, k), 0.05, seed + 1) if rank else None
    B = normal((n, rank), 0.05, seed + 2) if rank else None
    return codes, scale, A, B


# --------------------------------------------------------------------------- rows to codes
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,k", [(1, 16), (3, 48), (5, 2048), (4, 2064), (3, 4112), (130, 4096), (2, 8208), (2, 16400),
                                    (2, 32784), (1, 131072)])
def test_quantize_rows_bit_exact(lbq, dtype, rows, k):
    X = normal((rows, k), 1.0, rows * 7 + k, dtype)
    codes, scale = lbq.quantize_i8(X)
    ref, rs = ref_rows(X)
    assert torch.equal(codes.double(), ref)
    assert torch.equal(scale, rs)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_quantize_rows_edges(lbq, dtype):
    """Ties, zero rows, the type's largest and smallest values, infinities and NaN."""
    info = torch.finfo(dtype)
    k = 512
    X = torch.zeros((12, k), device="cuda", dtype=torch.float64)
    X[0] = torch.linspace(-1, 1, k, device="cuda", dtype=torch.float64)
    X[1, :] = 0.5                                     # with amax 1 every value is the tie 63.5
    X[1, 3], X[1, 4] = 1.0, -0.5
    X[2, :254] = torch.arange(-127, 127, device="cuda", dtype=torch.float64) + 0.5
    X[2, 300] = 127.0                                 # the odd halves: -126.5 ... 126.5
    X[4] = normal((1, k), 1.0, 5, torch.float64)[0]
    X[4] *= info.max / X[4].abs().max()
    X[5] = normal((1, k), 1.0, 6, torch.float64)[0] * info.smallest_normal
    X[6, ::2] = info.smallest_normal * info.eps       # the smallest subnormal
    X[7] = X[0] * 1e-30 if dtype != torch.float16 else X[0] * 1e-6
    X[8, 9], X[8, 10] = float("inf"), 1.0
    X[9, 0], X[9, 11] = float("nan"), 2.0
    X[10, 1], X[10, 2] = float("-inf"), float("nan")
    X[11] = -1.0
    X = X.to(dtype)
    codes, scale = lbq.quantize_i8(X)
    ref, rs = ref_rows(X)
    assert torch.equal(codes.double(), ref)
    assert torch.equal(torch.isnan(scale), torch.isnan(rs)) and torch.equal(torch.nan_to_num(scale), torch.nan_to_num(rs))
    assert not codes[3].any() and scale[3] == 0
    assert set(codes[1].tolist()) == {64, -64, 127}


# --------------------------------------------------------------------------- products
SIZES = [
    # m, n, k, rank
    (1, 1, 16, 0), (1, 8, 16, 1), (1, 4096, 4096, 0), (2, 100, 48, 5), (7, 1001, 2064, 5), (15, 129, 144, 16),
    (16, 4096, 14336, 16), (17, 136, 128, 33), (32, 257, 272, 64), (33, 1000, 1040, 8), (64, 128, 4096, 0),
    (65, 4104, 160, 4), (77, 1001, 2064, 5), (128, 2048, 1024, 64), (129, 4096, 4096, 8), (300, 520, 784, 17),
    (513, 2000, 640, 16),
    # enough tiles for the paired kernel, ragged in both directions
    (2600, 2000, 160, 0), (2600, 2000, 160, 7), (2305, 2561, 1168, 16), (2305, 2568, 400, 64),
    # several waves of tiles
    (4200, 4208, 272, 0), (4110, 4368, 528, 16),
    # clusters of 3, 5, 6 and 7 parts in the forward
    (5, 12000, 2048, 8), (5, 6400, 4096, 0), (20, 6000, 4096, 4), (7, 5200, 4096, 16),
    # parts that the GPU's groups of SMs hold at the same time
    (8, 5100, 4096, 0), (300, 2304, 4096, 0), (2048, 2048, 2048, 16), (2155, 2000, 192, 33),
    # many tokens and few features: small token tiles, one part of the reduction
    (3913, 78, 64, 64), (1500, 40, 32, 0), (904, 1500, 224, 33), (1015, 300, 2000, 16), (260, 16, 1456, 64),
]


@pytest.mark.parametrize("m,n,k,rank", SIZES)
def test_forward(lbq, m, n, k, rank):
    codes, scale, A, B = layer(n, k, rank, n + k)
    X = normal((m, k), 1.0, m)
    check_fwd(lbq, X, codes, scale, A, B, 1.5)


@pytest.mark.parametrize("m,n,k,rank", SIZES)
def test_backward(lbq, m, n, k, rank):
    n = (n + 7) // 8 * 8
    codes, scale, A, B = layer(n, k, rank, n + k + 1)
    dY = normal((m, n), 0.1, m + 1) * torch.exp(normal((m, 1), 1.5, m + 2, torch.float32)).to(torch.bfloat16)
    check_bwd(lbq, dY, codes, scale, A, B, -0.75)


def test_largest_sums_do_not_wrap(lbq):
    """127^2 times 131072 terms is 2^31 less 33 million: both signs, both directions."""
    n, k = 16, 131072
    codes = torch.full((n, k), 127, dtype=torch.int8, device="cuda")
    codes[1::2] = -127
    scale = torch.ones(n, device="cuda")
    X = torch.ones((3, k), device="cuda", dtype=torch.bfloat16)
    X[1] = -1
    Y, _ = check_fwd(lbq, X, codes, scale, None, None, 0.0)
    assert Y[0, 0] > 0 and Y[1, 0] < 0 and Y[0, 1] < 0
    codes = codes.t().contiguous()
    dX, _ = check_bwd(lbq, X, codes, torch.ones(k, device="cuda"), None, None, 0.0)
    assert dX[0, 0] > 0 and dX[1, 0] < 0


@pytest.mark.parametrize("m", [5, 17, 130])
@pytest.mark.parametrize("rank", [3, 8, 16, 32, 33, 64])
def test_adapter_product_keeps_small_terms(lbq, m, rank):
    """A one and then 131071 products of 1.75 * 2^-28: sixteen of them are 7/8 of a step of fp32 at the sum, so a chain of
    tensor-core additions (a product of 16 terms each, truncated) loses as many steps as it is long after the one.  At
    most 16 such additions follow one another before the sum is taken to fp32 registers.  There every addition onto the
    one is off by half a step at most, and there are at most 144: 128 of a warp's products or 64 of a CTA's chains (the
    reduction is in 8 parts), 8 of the warps and 8 of the parts.  In all 16 + 72 steps of 2^-23."""
    red = 131072
    small = 1.75 * 2.0 ** -28
    P = torch.full((rank, red), small, device="cuda").to(torch.bfloat16)
    P[:, 0] = 1.0
    ones = torch.ones((m, red), device="cuda", dtype=torch.bfloat16)
    want, lim = 1.0 + (red - 1) * small, (16 + 72) * 2.0 ** -23
    other = torch.zeros((16, rank), device="cuda", dtype=torch.bfloat16)
    codes = torch.ones((16, red), dtype=torch.int8, device="cuda")
    T = lbq.linear_i8_fwd(ones, lbq.Int8Weight(16, red, codes=codes, scale=torch.ones(16, device="cuda")), P, other, 1.0)[1]
    assert (T.double() - want).abs().max().item() <= lim
    U = lbq.linear_i8_bwd(ones, lbq.Int8Weight(red, 16, codes=codes.t().contiguous(), scale=torch.ones(red, device="cuda")),
                          other.t().contiguous(), P.t().contiguous(), 1.0)[1]
    assert (U.double() - want).abs().max().item() <= lim


@pytest.mark.parametrize("m", [6, 40, 2600])
def test_rows_without_values(lbq, m):
    """Zero tokens give zeros (plus the adapter's zero); a token with an infinity or a NaN gives NaN and leaves the
    others alone; a zero channel and a NaN channel likewise."""
    n, k = 2000, 160
    codes, scale, A, B = layer(n, k, 4, 3)
    scale[5], scale[6] = 0.0, float("nan")
    X = normal((m, k), 1.0, 4)
    X[1] = 0
    X[3, 7] = float("inf")
    X[m - 1, 0] = float("nan")
    Y, _ = lbq.linear_i8_fwd(X, lbq.Int8Weight(n, k, codes=codes, scale=scale), A, B, 1.0)
    nan = torch.isnan(Y)
    assert nan[3].all() and nan[m - 1].all() and nan[:, 6].all()
    keep = [t for t in range(m) if t not in (3, m - 1)]
    cols = [j for j in range(n) if j != 6]
    assert not nan[keep][:, cols].any()
    assert not Y[1, cols].any()
    assert lbq.device_status() == 0


def shifted(t, count=1):
    """A copy of t that starts `count` times 16 bytes past a 256-byte boundary."""
    step = 16 * count // t.element_size()
    buf = torch.empty(t.numel() + step, dtype=t.dtype, device=t.device)
    out = buf[step:].view(t.shape)
    out.copy_(t)
    assert out.data_ptr() % 32 == 16 * (count % 2)
    return out


# every way that the row quantizer takes the channel scales: by the length of a row (pieces per thread, two passes) and
# the number of rows, then both products and both adapter kernels
@pytest.mark.parametrize("m,n,k,rank", [(1, 8, 16, 0), (3, 2048, 64, 8), (5, 4096, 32, 0), (5, 4104, 48, 3), (4, 8192, 32, 16),
                                        (2, 16384, 16, 0), (2, 32768, 16, 0), (2, 40000, 16, 4), (400, 2048, 48, 0),
                                        (300, 4096, 32, 8), (300, 8200, 16, 0), (300, 14336, 32, 16), (300, 16384, 16, 0),
                                        (300, 28672, 16, 64), (300, 30000, 16, 0), (2600, 2000, 160, 16)])
def test_pointers_on_16_byte_boundaries(lbq, m, n, k, rank):
    """16 bytes is all that is asked of a pointer: every tensor of a call, the channel scales among them (a slice of one
    buffer of scales), starts 16 bytes past a 32-byte boundary."""
    codes, scale, A, B = layer(n, k, rank, n + k)
    codes, scale = shifted(codes), shifted(scale)
    A, B = (shifted(A), shifted(B)) if rank else (None, None)
    X, dY = shifted(normal((m, k), 1.0, m)), shifted(normal((m, n), 0.1, m + 1))
    qw = lbq.Int8Weight(n, k, codes=codes, scale=scale)
    wf = shifted(lbq.linear_i8_fwd_workspace(m, qw, rank))
    wb = shifted(lbq.linear_i8_bwd_workspace(m, qw, rank))
    Y, dX = shifted(torch.zeros(m, n, device="cuda")), shifted(torch.zeros(m, k, device="cuda"))
    T, U = (shifted(torch.zeros(m, rank, device="cuda")) for _ in range(2)) if rank else (None, None)
    want = lbq.linear_i8_fwd(X.clone(), qw, A, B, 1.5), lbq.linear_i8_bwd(dY.clone(), qw, A, B, 1.5)
    got = (lbq.linear_i8_fwd(X, qw, A, B, 1.5, Y=Y, T=T, workspace=wf), lbq.linear_i8_bwd(dY, qw, A, B, 1.5, dX=dX, U=U, workspace=wb))
    for a, b in zip(want, got):
        assert torch.equal(a[0], b[0]) and (rank == 0 or torch.equal(a[1], b[1]))
    check_fwd(lbq, X, codes, scale, A, B, 1.5)
    check_bwd(lbq, dY, codes, scale, A, B, 1.5)
    W = shifted(normal((n, k), 0.02, 9, torch.float32))
    part = lbq.Int8Weight(n, k, codes=shifted(codes), scale=shifted(scale)).quantize(W)
    ref, rs = ref_rows(W)
    assert torch.equal(part.codes.double(), ref) and torch.equal(part.scale, rs)


@pytest.mark.parametrize("m", [6, 40, 2600])
@pytest.mark.parametrize("rank", [4, 33])
def test_an_infinite_factor_stays_with_its_feature(lbq, m, rank):
    """An infinite element of B (forward) or A (backward) makes its own output feature infinite or NaN and no other."""
    n, k = 2000, 2000 // 16 * 16
    codes, scale, A, B = layer(n, k, rank, 3)
    qw = lbq.Int8Weight(n, k, codes=codes, scale=scale)
    X, dY = normal((m, k), 1.0, 4), normal((m, n), 0.1, 5)
    Y0, dX0 = lbq.linear_i8_fwd(X, qw, A, B, 1.0)[0], lbq.linear_i8_bwd(dY, qw, A, B, 1.0)[0]
    A2, B2 = A.clone(), B.clone()
    A2[1, 17], B2[130, 1] = float("inf"), float("-inf")
    Y, dX = lbq.linear_i8_fwd(X, qw, A, B2, 1.0)[0], lbq.linear_i8_bwd(dY, qw, A2, B, 1.0)[0]
    for got, ref, j in ((Y, Y0, 130), (dX, dX0, 17)):
        assert not torch.isfinite(got[:, j]).any()
        got[:, j] = ref[:, j]
        assert torch.equal(got, ref)
    assert lbq.device_status() == 0


def test_quantized_weight_round_trip(lbq):
    W = normal((300, 528), 0.02, 8)
    qw = lbq.Int8Weight(300, 528).quantize(W)
    codes, scale = ref_rows(W)
    assert torch.equal(qw.codes.double(), codes) and torch.equal(qw.scale, scale)
    # half a code step, the scale's half step 127 times over, and the product's own
    lim = scale.double()[:, None] * (0.5 + 2 * 127 * STEP)
    assert bool(((qw.dequantize().double() - W.double()).abs() <= lim).all())


def test_gradient_against_differences(lbq):
    """dX is the gradient of sum dY * Y for the dequantized weight with the tokens' rounding passed through: along a
    direction D its product is the difference of that (linear) function, up to the rounding of V: sv / 2 per channel."""
    m, n, k, r, s = 24, 264, 320, 8, 2.0
    codes, scale, A, B = layer(n, k, r, 12)
    dY, X, D = normal((m, n), 0.1, 1), normal((m, k), 1.0, 2).double(), normal((m, k), 1.0, 3).double()
    dX, _ = lbq.linear_i8_bwd(dY, lbq.Int8Weight(n, k, codes=codes, scale=scale), A, B, s)
    W = codes.double() * scale.double()[:, None] + s * (B.double() @ A.double())

    def loss(x):
        return (dY.double() * (x @ W.t())).sum()

    h = 2.0 ** -10
    diff = (loss(X + h * D) - loss(X - h * D)) / (2 * h)
    sv = (dY.float() * scale).abs().amax(1).double() / 127
    lim = ((sv[:, None] / 2) * codes.double().abs().sum(0)[None, :] * D.abs()).sum()
    got = (dX.double() * D).sum()
    assert (got - diff).abs() <= lim + 1e-6 * diff.abs()
    # and it is not the bound that makes it pass: the rounding errors are spread, the gradient is not
    assert (got - diff).abs() <= 0.05 * (dX.double().norm() * D.norm())


# --------------------------------------------------------------------------- how it is called
@pytest.mark.parametrize("m", [1, 16, 129, 2600])
def test_same_bits_again_and_in_a_graph(lbq, m):
    n, k, r = 2000, 1040, 8
    codes, scale, A, B = layer(n, k, r, 20)
    qw = lbq.Int8Weight(n, k, codes=codes, scale=scale)
    X, dY = normal((m, k), 1.0, 21), normal((m, n), 0.1, 22)
    wf, wb = lbq.linear_i8_fwd_workspace(m, qw, r), lbq.linear_i8_bwd_workspace(m, qw, r)
    wf.fill_(0xAB)
    wb.fill_(0xCD)
    Y0, T0 = lbq.linear_i8_fwd(X, qw, A, B, 2.0, workspace=wf)
    dX0, U0 = lbq.linear_i8_bwd(dY, qw, A, B, 2.0, workspace=wb)
    Y, T, dX, U = (torch.zeros_like(t) for t in (Y0, T0, dX0, U0))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lbq.linear_i8_fwd(X, qw, A, B, 2.0, Y=Y, T=T, workspace=wf)
        lbq.linear_i8_bwd(dY, qw, A, B, 2.0, dX=dX, U=U, workspace=wb)
    for _ in range(3):
        for t in (Y, T, dX, U):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in ((Y, Y0), (T, T0), (dX, dX0), (U, U0)):
            assert torch.equal(a, b)
    # new inputs in the same buffers
    X.copy_(normal((m, k), 3.0, 23))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(Y, lbq.linear_i8_fwd(X, qw, A, B, 2.0)[0])
    assert lbq.device_status() == 0


def test_back_to_back_calls_and_streams(lbq):
    """Calls that follow one another without a wait, the weight quantized just before, and two streams at once with
    workspaces of their own."""
    n, k, m = 1024, 2048, 5
    W = [normal((n, k), 0.02, 30 + i) for i in range(4)]
    X = normal((m, k), 1.0, 40)
    want = [lbq.linear_i8_fwd(X, lbq.Int8Weight(n, k).quantize(w))[0].clone() for w in W]
    torch.cuda.synchronize()
    qw = lbq.Int8Weight(n, k)
    ws = lbq.linear_i8_fwd_workspace(m, qw)
    for _ in range(10):
        got = []
        for w in W:
            qw.quantize(w)                     # overwrites the codes that the call before has read
            got.append(lbq.linear_i8_fwd(X, qw, workspace=ws)[0])
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    streams = [torch.cuda.Stream() for _ in range(2)]
    qws = [lbq.Int8Weight(n, k).quantize(w) for w in W[:2]]
    spaces = [lbq.linear_i8_fwd_workspace(m, q) for q in qws]
    outs = [[torch.empty_like(want[0]) for _ in range(20)] for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(20):
        for j in range(2):
            lbq.linear_i8_fwd(X, qws[j], Y=outs[j][i], workspace=spaces[j], stream=streams[j])
    torch.cuda.synchronize()
    for j in range(2):
        for y in outs[j]:
            assert torch.equal(y, want[j])
    assert lbq.device_status() == 0


def test_inputs_written_by_the_kernel_just_before(lbq):
    """A kernel of this library may start while the one before it still writes: the channel scales of a weight that is
    quantized just before its backward, and an fp32 product that is quantized itself, are the new ones every time."""
    n, k, m = 2048, 512, 40
    W = [normal((n, k), 0.02 * 3 ** i, 60 + i) for i in range(4)]
    dY, X = normal((m, n), 0.1, 65), normal((m, k), 1.0, 66)
    qw = lbq.Int8Weight(n, k)
    Y = torch.empty(m, n, device="cuda")
    ws = lbq.linear_i8_bwd_workspace(m, qw)
    want = []
    for w in W:
        qw.quantize(w)
        torch.cuda.synchronize()
        dX = lbq.linear_i8_bwd(dY, qw)[0]
        lbq.linear_i8_fwd(X, qw, Y=Y)
        torch.cuda.synchronize()
        want.append((dX,) + lbq.quantize_i8(Y))
    for _ in range(10):
        got = []
        for w in W:
            qw.quantize(w)
            dX = lbq.linear_i8_bwd(dY, qw, workspace=ws)[0]
            lbq.linear_i8_fwd(X, qw, Y=Y)
            got.append((dX,) + lbq.quantize_i8(Y))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert lbq.device_status() == 0


def test_temporaries_on_another_stream(lbq):
    """Calls on a stream that is not the current one, with outputs and workspaces of the helpers' own, while the
    current stream takes and writes memory too."""
    n, k, m, r = 512, 4096, 24, 8
    codes, scale, A, B = layer(n, k, r, 31)
    qw = lbq.Int8Weight(n, k, codes=codes, scale=scale)
    X, dY, W = normal((m, k), 1.0, 32), normal((m, n), 0.1, 33), normal((64, k), 1.0, 34)
    want = [t.clone() for t in lbq.linear_i8_fwd(X, qw, A, B, 1.0) + lbq.linear_i8_bwd(dY, qw, A, B, 1.0) + lbq.quantize_i8(W)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got, other = [], []
    for _ in range(10):
        got.append(lbq.linear_i8_fwd(X, qw, A, B, 1.0, stream=side) + lbq.linear_i8_bwd(dY, qw, A, B, 1.0, stream=side) +
                   lbq.quantize_i8(W, stream=side))
        other.append(torch.full((m * k + 4096,), 0x7F, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, want):
            assert torch.equal(a, b)
    assert lbq.device_status() == 0


def test_helpers_refuse(lbq):
    n, k, m = 64, 32, 4
    qw = lbq.Int8Weight(n, k).quantize(normal((n, k), 1.0, 1))
    X, A, B = normal((m, k), 1.0, 2), normal((4, k), 1.0, 3), normal((n, 4), 1.0, 4)
    for bad in (lambda: lbq.linear_i8_fwd(X.float(), qw), lambda: lbq.linear_i8_fwd(X[:, :16], qw),
                lambda: lbq.linear_i8_fwd(X, qw, A), lambda: lbq.linear_i8_fwd(X, qw, B, A, 1.0),
                lambda: lbq.linear_i8_fwd(X, qw, Y=torch.empty((m, n), device="cuda", dtype=torch.bfloat16)),
                lambda: lbq.linear_i8_bwd(X, qw), lambda: lbq.quantize_i8(X.double()), lambda: lbq.quantize_i8(X.cpu()),
                lambda: lbq.quantize_i8(X.t()), lambda: lbq.Int8Weight(n, k, codes=qw.codes),
                lambda: lbq.linear_i8_fwd(X, qw, workspace=torch.empty(4096, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: lbq.linear_i8_fwd(X, qw, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
                lambda: lbq.quantize_i8(normal((2, 24), 1.0, 1)), lambda: lbq.linear_i8_fwd(X[:0], qw)):
        with pytest.raises(lbq.LbqError):
            bad()


# --------------------------------------------------------------------------- a step
def test_training_step_with_clipping(lbq):
    """Forward, input gradient, adapter gradients and clipping of two 8-bit layers, as the data-parallel step runs
    them; the clipped gradients are the unclipped ones times max_norm / norm."""
    from qlora_quantized_linear_b200.dp import AdapterLayer, DataParallelQLoRA
    m, s = 96, 2.0
    layers, shards = [], []
    for i, (n, k, r) in enumerate([(256, 512, 8), (384, 1024, 16)]):
        qw = lbq.Int8Weight(n, k).quantize(normal((n, k), 0.02, 50 + i))
        layers.append(AdapterLayer(qw, normal((r, k), 0.01, 60 + i), normal((n, r), 0.01, 70 + i), s))
        shards.append((normal((m, k), 1.0, 80 + i), normal((m, n), 0.1, 90 + i)))
    plain = DataParallelQLoRA(layers)
    outs = plain.step(shards)
    raw = plain.flat.clone()
    for L, (X, dY), (Y, dX) in zip(layers, shards, outs):
        Y2, T = lbq.linear_i8_fwd(X, L.qw, L.A, L.B, s)
        dX2, U = lbq.linear_i8_bwd(dY, L.qw, L.A, L.B, s)
        assert torch.equal(Y, Y2) and torch.equal(dX, dX2)
        t, tb, _, _, _ = adapter_ref(X, L.A.t(), L.B.t(), s)
        dB = s * (dY.double().t() @ t)
        # T is rounded to bf16 for the tensor cores (2^-8), beside its own error and the sum's
        lim = abs(s) * (dY.double().abs().t() @ (t.abs() * (2.0 ** -8 + 2 * (m + 2) * STEP) + 2 * tb))
        assert_close(L.dB, dB, lim, "dB")
    norm = raw.double().norm().item()
    clipped = DataParallelQLoRA(layers, max_grad_norm=norm / 4)
    clipped.step(shards)
    assert abs(clipped.grad_norm.item() - norm) <= 1e-6 * norm
    coef = torch.tensor(norm / 4 / (norm + 1e-6), dtype=torch.float64)
    assert bool(((clipped.flat.double() - raw.double() * coef).abs() <= 4 * STEP * raw.double().abs() + 1e-40).all())
    loose = DataParallelQLoRA(layers, max_grad_norm=norm * 4)
    loose.step(shards)
    assert torch.equal(loose.flat, raw)
    assert lbq.device_status() == 0


@pytest.mark.parametrize("eight", [True, False])
def test_training_step_on_a_side_stream(lbq, eight):
    """A step built behind queued work and run on another stream at once: the flat buffer, the clipping's workspace and
    every temporary are filled in that stream's order.  Same bits as on the current stream."""
    from qlora_quantized_linear_b200.dp import AdapterLayer, DataParallelQLoRA
    m, s = 24, 2.0
    layers, shards = [], []
    for i, (n, k, r) in enumerate([(256, 512, 8), (384, 1024, 16)]):
        W = normal((n, k), 0.02, 50 + i)
        qw = lbq.Int8Weight(n, k).quantize(W) if eight else lbq.QuantizedWeight(n, k, "minmax", 4).quantize(W)
        layers.append(AdapterLayer(qw, normal((r, k), 0.01, 60 + i), normal((n, r), 0.01, 70 + i), s))
        shards.append((normal((m, k), 1.0, 80 + i), normal((m, n), 0.1, 90 + i)))
    plain = DataParallelQLoRA(layers, max_grad_norm=0.5)
    want = [t.clone() for pair in plain.step(shards) for t in pair] + [plain.flat.clone(), plain.grad_norm.clone()]
    big = normal((1 << 26,), 1.0, 1, torch.float32)
    for _ in range(3):
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        dirt = [torch.full((1 << i,), 0x5A, dtype=torch.uint8, device="cuda") for i in range(8, 20) for _ in range(4)]
        for _ in range(20):
            big.mul_(1.0001)
        del dirt
        step = DataParallelQLoRA(layers, max_grad_norm=0.5)
        outs = step.step(shards, stream=side)
        torch.cuda.synchronize()
        got = [t for pair in outs for t in pair] + [step.flat, step.grad_norm]
        assert lbq.device_status() == 0
        for a, b in zip(got, want):
            assert torch.equal(a, b)
