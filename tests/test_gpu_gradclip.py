"""The gradient norm and clipping on the GPU against fp64.

The squares of a lane's four 16-byte pieces are added in fp32: chains of four
(4 roundings), the two halves of a 16-bit piece (1), the pieces in pairs (2), so
at most 7 roundings of 2^-24; all sums after that are in fp64.  The norm's square
root halves the relative error and the result is rounded once: 4.5 * 2^-24, and
5 * 2^-24 bounds it.  An output
is the fp32 product of the value with a coefficient that is off by as much and
rounded once (7 * 2^-24 in all), then rounded to its type.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -24
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def lbq():
    from qlora_quantized_linear_b200 import lbq as m
    return m


def normal(n, std, seed, dtype=torch.float32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(n, generator=g, device="cuda") * std).to(dtype)


def ref_norm(grads):
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


def norm_is(norm, want):
    """The definition rounds the norm to fp32: past its largest value that is infinity (the scaling is not affected)."""
    if want > torch.finfo(torch.float32).max * (1 + STEP):
        return norm == float("inf")
    return abs(norm - want) <= 5 * STEP * want + 2.0 ** -149


def check(lbq, grads, max_norm, outs=None, plan=None):
    raw = [g.clone() for g in grads]
    want = ref_norm(raw)
    plan = plan or lbq.GradClip(grads, outs)
    norm = plan.clip(max_norm)
    torch.cuda.synchronize()
    assert lbq.device_status() == 0
    assert norm_is(norm.item(), want)
    coef = min(1.0, max_norm / (want + 1e-6))
    for g, o, r in zip(grads, outs or grads, raw):
        eps = torch.finfo(o.dtype)
        ref = r.double() * coef
        # subnormal results are off by half the smallest step
        lim = ref.abs() * (7 * STEP + eps.eps / 2 * (o.dtype != torch.float32)) + eps.smallest_normal * eps.eps
        assert bool(((o.double() - ref).abs() <= lim).all())
        if outs is not None:
            assert torch.equal(g, r), "the gradient itself changed"
    return plan


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("sizes", [[1], [0, 3], [4096], [1024, 1025, 1023, 8], [65536 + 5, 7, 300001], [2_000_003]])
@pytest.mark.parametrize("inplace", [True, False])
def test_sizes_and_types(lbq, dtype, sizes, inplace):
    grads = [normal(n, 0.1, 7 + i, TYPES[dtype]) for i, n in enumerate(sizes)]
    check(lbq, grads, 0.05, None if inplace else [torch.zeros_like(g) for g in grads])


@pytest.mark.parametrize("max_norm", [0.0, 0.3, 1e9])
def test_limits(lbq, max_norm):
    grads = [normal(5000, 1.0, 1), normal(333, 1.0, 2, torch.bfloat16)]
    raw = [g.clone() for g in grads]
    check(lbq, grads, max_norm)
    if max_norm == 1e9:
        assert all(torch.equal(g, r) for g, r in zip(grads, raw))
    if max_norm == 0.0:
        assert not any(bool(g.any()) for g in grads)


def test_views_off_the_16_byte_grid(lbq):
    """Gradients and outputs that start anywhere in flat buffers, with guards between them."""
    for dtype in TYPES.values():
        flat, out = normal(40000, 0.3, 3, dtype), torch.full((40000,), 3.0, device="cuda", dtype=dtype)
        spans, at = [], 0
        for i, n in enumerate([1, 2, 3, 5, 8, 1000, 1021, 2048, 2047, 4099, 8193]):
            at += 1 + (i * 5) % 7
            spans.append((at, at + n))
            at += n
        shift = 11
        grads = [flat[a:b] for a, b in spans]
        outs = [out[a + shift:b + shift] for a, b in spans]
        check(lbq, grads, 0.7, outs)
        mask = torch.ones(40000, dtype=torch.bool, device="cuda")
        for a, b in spans:
            mask[a + shift:b + shift] = False
        assert bool((out[mask] == 3.0).all()), "wrote outside the outputs"
        check(lbq, grads, 0.7)


def test_many_tensors_of_all_types(lbq):
    """More tensors than one launch describes, some of them empty."""
    for count in (64, 65, 1000, 1001, 2300):
        grads = [normal((i * 37) % 611, 0.1, i, (torch.float32, torch.bfloat16, torch.float16)[i % 3])
                 for i in range(count)]
        check(lbq, grads, 0.2, [torch.zeros_like(g) for g in grads])
        plan = lbq.GradClip(grads)
        assert abs(plan.norm().item() - ref_norm(grads)) <= 5 * STEP * ref_norm(grads)


def test_many_small_tensors_in_one_range(lbq):
    """900 tensors of one element before a large one: the first CTA's equal share of the bytes meets all of them, more
    tensors than it has threads."""
    small = [torch.full((1,), 0.25 + 0.125 * (i % 7), device="cuda") for i in range(900)]
    large = torch.full((80_000_000,), 2.0 ** -10, device="cuda")
    want = math.sqrt(sum(float(t) ** 2 for t in small) + 80_000_000 * 2.0 ** -20)
    flat = torch.cat(small)
    norm = lbq.clip_grad_norm(small + [large], 1.0)
    torch.cuda.synchronize()
    assert norm_is(norm.item(), want)
    coef = 1.0 / (want + 1e-6)
    got = torch.cat(small).double()
    assert bool(((got - flat.double() * coef).abs() <= 7 * STEP * got).all())
    assert bool(((large.double() - 2.0 ** -10 * coef).abs() <= 7 * STEP * 2.0 ** -10 * coef).all())
    assert lbq.device_status() == 0


@pytest.mark.parametrize("scale", [1e-42, 1e-30, 1e-20, 1e-5, 1e15, 1e25, 1e37])
def test_magnitudes(lbq, scale):
    """Squares below and above the range of fp32."""
    g = normal(3001, 1.0, 4).double()
    grads = [(g * scale).clamp(-3e38, 3e38).float(), torch.zeros(50, device="cuda")]
    want = ref_norm(grads)
    assert norm_is(lbq.grad_norm(grads).item(), want)
    if 1e-30 < scale:
        check(lbq, grads, want / 3)


def test_all_zero(lbq):
    grads = [torch.zeros(1000, device="cuda"), torch.zeros(10, device="cuda", dtype=torch.bfloat16)]
    assert lbq.clip_grad_norm(grads, 1.0).item() == 0
    assert not any(bool(g.any()) for g in grads)


def test_infinity_and_nan(lbq):
    for bad, dtype in ((float("inf"), torch.float32), (float("-inf"), torch.bfloat16), (float("nan"), torch.float16)):
        grads = [normal(700, 1.0, 1), normal(901, 1.0, 2, dtype)]
        grads[1][5] = bad
        norm = lbq.clip_grad_norm(grads, 1.0)
        if math.isnan(bad):
            assert torch.isnan(norm).all() and all(bool(torch.isnan(g).all()) for g in grads)
        else:
            assert norm.item() == float("inf")
            assert not grads[0].any() and torch.isnan(grads[1][5]) and int(torch.isnan(grads[1]).sum()) == 1


def test_same_bits_and_reuse(lbq):
    """The same plan again and again, in a replayed graph, and with new values in the same tensors."""
    grads = [normal(100003, 0.1, 1), normal(4097, 0.1, 2, torch.bfloat16)]
    outs = [torch.empty_like(g) for g in grads]
    plan = check(lbq, grads, 0.5, outs)
    first = [o.clone() for o in outs]
    n0 = plan.total_norm.clone()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        plan.clip(0.5)
    for i in range(50):
        for o in outs:
            o.zero_()
        g.replay() if i % 2 else plan.clip(0.5)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, first)) and torch.equal(plan.total_norm, n0)
    grads[0].mul_(3)
    check(lbq, grads, 0.5, outs, plan)


def test_two_streams(lbq):
    """Two lists at once, each with its own workspace: both grids have to find room to meet."""
    lists = [[normal(500_000, 0.1, i), normal(77, 0.1, 9 + i)] for i in range(2)]
    outs = [[torch.empty_like(g) for g in gs] for gs in lists]
    plans = [lbq.GradClip(g, o) for g, o in zip(lists, outs)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for p, s in zip(plans, streams):
            p.clip(0.3, stream=s)
    torch.cuda.synchronize()
    for g, o, p in zip(lists, outs, plans):
        want = ref_norm(g)
        assert abs(p.total_norm.item() - want) <= 5 * STEP * want
        for a, b in zip(g, o):
            ref = a.double() * (0.3 / (want + 1e-6))
            assert bool(((b.double() - ref).abs() <= 7 * STEP * ref.abs()).all())
    assert lbq.device_status() == 0


def test_against_the_usual_clipping(lbq):
    """torch's own clipping of the same gradients (its norm is a tree of fp32 sums)."""
    params = [torch.nn.Parameter(torch.zeros(n, device="cuda")) for n in (1000, 70001, 3)]
    for i, p in enumerate(params):
        p.grad = normal(p.numel(), 0.2, i)
    mine = [p.grad.clone() for p in params]
    want = torch.nn.utils.clip_grad_norm_(params, 0.5)
    norm = lbq.clip_grad_norm(mine, 0.5)
    assert abs(norm.item() - want.item()) <= 1e-5 * want.item()
    for a, p in zip(mine, params):
        assert torch.allclose(a, p.grad, rtol=2e-5, atol=0)


def test_helpers_refuse(lbq):
    a, b = normal(100, 1.0, 1), normal(100, 1.0, 2)
    for bad in (lambda: lbq.grad_norm([]), lambda: lbq.grad_norm([a.double()]), lambda: lbq.grad_norm([a.cpu()]),
                lambda: lbq.GradClip([a], [b.half()]), lambda: lbq.GradClip([a], [b[:50]]),
                lambda: lbq.GradClip([a, b], [a]), lambda: lbq.grad_norm([normal(100, 1.0, 1).view(10, 10).t()])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: lbq.clip_grad_norm([a, a], 1.0),            # the same tensor scaled twice
                lambda: lbq.clip_grad_norm([a[:60], a[40:]], 1.0),
                lambda: lbq.clip_grad_norm([a, b], 1.0, [b, a]),    # an output over another's gradient
                lambda: lbq.clip_grad_norm([a[:50]], 1.0, [a[10:60]]),
                lambda: lbq.clip_grad_norm([a], -1.0), lambda: lbq.clip_grad_norm([a], float("nan")),
                lambda: lbq.clip_grad_norm([a], float("inf"))):
        with pytest.raises(lbq.LbqError):
            bad()
    assert abs(lbq.grad_norm([a, a]).item() - math.sqrt(2) * ref_norm([a])) <= 5 * STEP * 2 * ref_norm([a])


def test_helpers_own_the_order_on_another_stream(lbq):
    """clip_grad_norm and grad_norm on a stream that is not the current one, which is busy: their workspace is zeroed
    and given back in the order of the call's stream."""
    side = torch.cuda.Stream()
    grads = [normal(n, 0.5, n) for n in (70001, 33, 4096)]
    want = ref_norm(grads)
    copies = [[g.clone() for g in grads] for _ in range(6)]
    big = normal(1 << 26, 1.0, 1)
    dirt = torch.full((1 << 20,), 0x5A, dtype=torch.uint8, device="cuda")
    del dirt                                       # memory of the current stream that a workspace may take
    torch.cuda.synchronize()
    for _ in range(20):
        big.mul_(1.0001)                           # the current stream is milliseconds behind
    norms = [lbq.clip_grad_norm(c, 1.0, stream=side) for c in copies] + [lbq.grad_norm(grads, stream=side)]
    torch.cuda.synchronize()
    for n in norms:
        assert norm_is(n.item(), want)
    coef = 1.0 / (want + 1e-6)
    for c in copies:
        for g, o in zip(grads, c):
            assert bool(((o.double() - g.double() * coef).abs() <= 7 * STEP * g.double().abs() * coef).all())
    assert lbq.device_status() == 0


def test_some_in_place_some_not_and_nothing_to_clip(lbq):
    """Below max_norm the tensors in place keep their bits and the others are copied, also within one CTA's range."""
    grads = [normal(n, 0.01, n) for n in (3, 700_001, 40, 5000, 9)]
    outs = [g if i % 2 else torch.full_like(g, 7.0) for i, g in enumerate(grads)]
    before = [g.clone() for g in grads]
    lbq.clip_grad_norm(grads, 1e9, outs)
    torch.cuda.synchronize()
    for g, o, b in zip(grads, outs, before):
        assert torch.equal(g, b) and torch.equal(o, b)
    assert lbq.device_status() == 0


def test_a_plan_made_behind_queued_work_and_used_on_another_stream(lbq):
    """The plan's workspace is zeroed on the stream of its construction, which is milliseconds behind: the first call on
    another stream, clip or norm, waits for that, and the workspace is not given away under it."""
    grads = [normal(n, 0.5, n) for n in (300_001, 33, 4096)]
    want = ref_norm(grads)
    coef = 1.0 / (want + 1e-6)
    big = normal(1 << 26, 1.0, 1)
    for use in ("clip", "norm"):
        for _ in range(5):
            copies = [g.clone() for g in grads]
            dirt = [torch.full((1 << 12,), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(64)]
            side = torch.cuda.Stream()
            torch.cuda.synchronize()
            for _ in range(20):
                big.mul_(1.0001)
            del dirt
            plan = lbq.GradClip(copies)
            norm = plan.clip(1.0, stream=side) if use == "clip" else plan.norm(stream=side)
            again = plan.norm(stream=side).clone() if use == "norm" else None
            del plan
            rewrite = [torch.full((1 << 12,), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(64)]
            torch.cuda.synchronize()
            assert lbq.device_status() == 0
            assert norm_is(norm.item(), want) and len(rewrite) == 64
            if use == "norm":
                assert all(torch.equal(g, c) for g, c in zip(grads, copies)) and again.numel() == 1
            else:
                for g, c in zip(grads, copies):
                    assert bool(((c.double() - g.double() * coef).abs() <= 7 * STEP * g.double().abs() * coef).all())


def test_a_plan_in_a_graph_before_any_other_call(lbq):
    """Captured at its first use, then replayed, then called on the stream of its construction and on a third one."""
    grads = [normal(n, 0.5, n) for n in (70_001, 12)]
    outs = [torch.empty_like(g) for g in grads]
    plan = lbq.GradClip(grads, outs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.clip(0.25)
    g.replay()
    torch.cuda.synchronize()
    want = ref_norm(grads)
    assert norm_is(plan.total_norm.item(), want)
    first = [o.clone() for o in outs]
    side = torch.cuda.Stream()
    for stream in (None, side, side, None):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        assert norm_is(plan.clip(0.25, stream=stream).item(), want)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, first))
    assert lbq.device_status() == 0
