"""The dense product where arithmetic ends: infinities, sums far below zero, the last bits of fp32
operands, long reductions."""
import pytest
import torch

import mixture_experts_layer_31_b200 as moe
import ops_ref as ref
from test_gpu_linear import Product

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clear_flags():
    moe.moe_device_flags(clear=True)
    yield
    assert moe.moe_device_flags(clear=True) == 0


# K, N, M: the reduction split over several CTAs (few columns, more columns); one accumulator;
# several drained segments
SPLIT, LONG_SPLIT, WHOLE, SEGMENTS = (256, 96, 50), (2048, 96, 50), (128, 1100, 2500), (1664, 1100, 2500)


@pytest.mark.parametrize("wfmt,xfmt,yfmt,gated", [("f32", "f32", "f32", False), ("f32", "f32", "bf16", True),
                                                  ("f32", "bf16", "f32", False), ("bf16", "f32", "f32", False),
                                                  ("int8", "f32", "f32", False), ("int4", "f32", "f32", False),
                                                  ("int4", "bf16", "f32", False), ("int4", "bf16", "bf16", True),
                                                  ("int4b128", "bf16", "bf16", True)])
@pytest.mark.parametrize("K,N,M", [SPLIT, LONG_SPLIT, WHOLE, SEGMENTS])
def test_infinities_in_products_of_parts(wfmt, xfmt, yfmt, gated, K, N, M):
    """Operands that are multiplied in several bf16 parts: an infinity gives the signed infinity that
    the formula gives, and NaN only where that does (0 times infinity, infinities of both signs)."""
    p = Product(K, N, wfmt, xfmt, yfmt=yfmt, gated=gated)
    x = p.x(M)
    x[1, 3], x[M // 2, K - 1], x[M - 1, 0] = float("inf"), float("-inf"), float("nan")
    x[M - 2, 5], x[M - 2, 70] = float("inf"), float("-inf")
    if wfmt in ("f32", "bf16"):
        at = [(0, "W", 7, float("inf")), (N - 1, "W", 64, float("-inf"))] + ([(N // 2, "Wu", 9, float("-inf"))] if gated else [])
        for n, which, k, v in at:
            getattr(p, which)[n, k] = v
            p.dev.tensors["W" if which == "W" else "W_up"][n, k] = v
    y = p.dev(x.cuda()).cpu()
    rows = torch.tensor(sorted({0, 1, 2, M // 2, M - 3, M - 2, M - 1}))
    want, bound = ref.linear(x[rows], p.W, None, (p.Wu, None) if gated else None, "none", None, p.y_dtype, wfmt, 2 if gated else 0)
    got = y[rows].double()
    assert torch.equal(got.isnan(), want.isnan())
    inf = want.isinf()
    assert bool(inf.any()) and torch.equal(got[inf], want[inf])
    fine = want.isfinite()
    ref.check(got[fine], want[fine], bound[fine])


@pytest.mark.parametrize("wfmt,xfmt,M", [("bf16", "bf16", 5), ("bf16", "bf16", 20), ("bf16", "bf16", 150), ("int8", "bf16", 12),
                                         ("int8", "bf16", 60), ("int8", "bf16", 150), ("int4", "bf16", 12), ("int4", "bf16", 40),
                                         ("int4", "bf16", 150), ("int4b128", "bf16", 20), ("f32", "f32", 5), ("bf16", "f32", 16),
                                         ("int8", "f32", 9), ("int4", "f32", 5), ("f32", "bf16", 16)])
def test_infinities_in_the_other_forms(wfmt, xfmt, M):
    p = Product(384, 75, wfmt, xfmt)
    x = p.x(M)
    x[1, 3], x[M - 1, 380] = float("inf"), float("-inf")
    x[M - 2, 5], x[M - 2, 70] = float("inf"), float("-inf")
    y = p.dev(x.cuda()).cpu().double()
    want, bound = ref.linear(x, p.W, None, None, "none", None, p.y_dtype, wfmt, 1)
    assert torch.equal(y.isnan(), want.isnan())
    inf = want.isinf()
    assert bool(inf.any()) and torch.equal(y[inf], want[inf])
    fine = want.isfinite()
    ref.check(y[fine], want[fine], bound[fine])


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("yfmt", ["bf16", "f32"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("K,M", [(256, 8), (256, 100), (2048, 100)])
def test_activations_of_sums_far_below_zero(act, yfmt, gated, K, M):
    """Both activations are below |v| exp(-|v|) 2^-126 from v = -200 down, whatever rounding did to
    v: nothing is left of it beside the residual.  The largest v are their own activation."""
    low = [-200.0, -1e4, -1e30, -1e36, -3e38, torch.finfo(torch.bfloat16).min, torch.finfo(torch.float32).min]
    high = [3e4, 1e30, 3e38]
    p = Product(K, 96, "bf16", yfmt=yfmt, act=act, gated=gated, bias=True)
    for j, v in enumerate(low + high):
        p.b[5 * j] = v
        p.dev.tensors["b"][5 * j] = v
    p.W[5 * torch.arange(len(low))] *= 0.25  # products far smaller than 200
    p.dev.tensors["W"][5 * torch.arange(len(low))] *= 0.25
    x, r = p.x(M), p.residual(M)
    y = p.dev(x.cuda(), residual=r.cuda()).cpu()
    at = 5 * torch.arange(len(low))
    assert bool((x.double() @ p.W[at].T).abs().max() < 60)
    zero = p.dev(x.cuda()).cpu()[:, at].double()
    assert bool((zero.abs() <= ref.TINY).all())
    assert torch.equal(y[:, at], r[:, at])
    if not gated:
        at = 5 * (len(low) + torch.arange(len(high)))
        want = (x.double() @ p.W[at].T + p.b[at])
        ref.check(y[:, at], want, (2 * ref.HALF[p.y_dtype] + 2.0 ** -20) * want.abs() + 10)


def _all_bits(shape, gen):
    """fp32 values in [1, 2) whose three bf16 parts are as large as can be: the third is 63 2^-23 in
    all of them, so that leaving it out shifts every product the same way."""
    a = torch.randint(0, 127, shape, generator=gen).double()
    b = torch.randint(128, 251, shape, generator=gen).double() * (2 * torch.randint(0, 2, shape, generator=gen) - 1)
    v = 1 + a / 128 + b * 2.0 ** -16 + 63 * 2.0 ** -23
    assert torch.equal(v.float().double(), v)
    return v.float()


def _two_parts(v):
    h = v.to(torch.bfloat16).float()
    return (h + (v - h).to(torch.bfloat16).float()).double()


@pytest.mark.parametrize("wfmt,xfmt", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"), ("int8", "f32")])
@pytest.mark.parametrize("K", [16, 32])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** -100])
@pytest.mark.parametrize("M", [3, 40])
def test_every_bit_of_fp32_operands(wfmt, xfmt, K, scale, M):
    """Short reductions, whose worst rounding is smaller than what a third part brings."""
    gen, N = torch.Generator().manual_seed(K + M), 64
    x = _all_bits((M, K), gen).to(torch.bfloat16 if xfmt == "bf16" else torch.float32)
    x, s = x * scale if xfmt == "f32" else x, None
    if wfmt == "int8":
        W, s = torch.randint(64, 128, (N, K), generator=gen).to(torch.int8), torch.full((N,), 2.0 ** -6)
        Wd = W.double() * 2.0 ** -6
    else:
        W = _all_bits((N, K), gen).to(torch.bfloat16 if wfmt == "bf16" else torch.float32)
        W = W * scale if xfmt == "bf16" and scale != 1 else W
        Wd = W.double()
    y = moe.Linear(K=K, N=N, wfmt=wfmt, xfmt=xfmt, yfmt="f32", W=W, s=s)(x.cuda())
    want = x.double() @ Wd.T
    bound = ref.sum_error(K, x.double().abs() @ Wd.abs().T) + ref.HALF[torch.float32] * want.abs()
    ref.check(y, want, bound)
    # the oracle with a part left out is off by more than that everywhere
    if xfmt == "f32":
        assert bool(((_two_parts(x) @ Wd.T - want).abs() > bound).all())
    if wfmt == "f32":
        assert bool(((x.double() @ _two_parts(W).T - want).abs() > bound).all())


@pytest.mark.parametrize("fmt", ["bf16", "f32"])
def test_long_sums_of_one_sign_are_not_cut_off(fmt):
    """65,536 positive columns, fp32 output.  An accumulator is drained after 12 steps of 4
    instructions at full magnitude: were each of these 48 additions cut off by a whole unit of the
    last place, the sums would come out 48 x 2^-23 too small at most; the drained sums are added
    with rounding to nearest, whose errors are as often up as down.  4,096 additions in a
    row that cut off by half a unit each lose 4096 / 2 x 2^-24 = 1.2 x 10^-4."""
    dtype = torch.bfloat16 if fmt == "bf16" else torch.float32
    K, N, M = 65536, 1024, 2400  # tiles enough that the reduction is not split
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.empty((M, K), device="cuda").uniform_(1, 2, generator=gen).to(dtype)
    W = torch.empty((N, K), device="cuda").uniform_(1, 2, generator=gen).to(dtype)
    y = moe.Linear(K=K, N=N, wfmt=fmt, xfmt=fmt, yfmt="f32", W=W)(x)
    rows, cols = torch.arange(0, M, 149, device="cuda"), torch.arange(0, N, 31, device="cuda")
    want = x[rows].double() @ W[cols].double().T
    off = (y[rows][:, cols].double() - want) / want
    assert bool(off.abs().max() <= (K + ref.STEPS) * ref.U)
    assert abs(float(off.mean())) <= 48 * 2.0 ** -23
