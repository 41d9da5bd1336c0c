"""The whole layer for a few tokens against a 64-bit reference: formats, token counts,
masks, shared expert, residual, borders of the routing, capture, streams."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_31_b200 as moe
import ops_ref as ref
import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clear_flags(request):
    moe.moe_device_flags(clear=True)
    yield
    if "flags" not in request.keywords:
        assert moe.moe_device_flags(clear=True) == 0


class Layer:
    """A small layer: stored tensors, their 64-bit values, the device wrapper."""

    def __init__(self, H=256, I=128, E=16, k=4, router="sigmoid", scale=2.446, wfmt="bf16", xfmt="bf16", act="silu",
                 bias=True, active=None, shared=0, seed=1, W_r=None):
        self.__dict__.update(H=H, I=I, E=E, k=k, router=router, scale=scale, wfmt=wfmt, act=act, shared_I=shared)
        self.x_dtype = torch.bfloat16 if xfmt == "bf16" else torch.float32
        self.W_r = torch.from_numpy(synth.normal_f32((E, H), seed, 2, 0.0, 0.05)) if W_r is None else W_r
        self.b = torch.from_numpy(synth.normal_f32((E,), seed, 3, 0.0, 0.05)) if bias and router == "sigmoid" else None
        self.mask = None
        if active is not None:
            self.mask = torch.zeros(E, dtype=torch.uint8)
            self.mask[list(active)] = 1
        kw = {}
        self.experts = []
        for n, (part, r, c) in enumerate((("gate", I, H), ("up", I, H), ("down", H, I))):
            W, s, d = ref.weights(E * r, c, wfmt, seed * 100 + n)
            kw["W_" + part] = W.view(E, r, -1)
            kw["s_" + part] = None if s is None else (s.view(E, r) if s.dim() == 1 else s.view(E, r, -1))
            self.experts.append(d.view(E, r, c))
        self.shared = None
        if shared:
            self.shared = []
            for n, (part, r, c) in enumerate((("gate", shared, H), ("up", shared, H), ("down", H, shared))):
                kw["Ws_" + part], kw["ss_" + part], d = ref.weights(r, c, wfmt, seed * 100 + 50 + n)
                self.shared.append(d)
        self.dev = moe.MoELayer(H=H, I=I, E=E, k=k, router=router, scale=scale, wfmt=wfmt, xfmt=xfmt, act=act,
                                W_r=self.W_r, b=self.b, expert_mask=self.mask, I_s=shared, **kw)

    def x(self, T, seed=7):
        return torch.from_numpy(synth.normal_f32((T, self.H), seed, 9, 0.0, 1.0)).to(self.x_dtype)

    def compare(self, x, y, idx, w, residual=None, what=""):
        ri, rw = ref.route(x, self.W_r, self.b, self.mask, self.k, self.router, self.scale)
        assert torch.equal(idx.cpu(), ri), what
        # weights: one division and one product in 64 bits, one rounding to fp32
        assert bool(((w.cpu().double() - rw).abs() <= 2 * ref.U * rw.abs() + 1e-45).all()), what
        want, bound = ref.few(x, ri, rw, self.experts, self.act, self.shared, residual)
        ref.check(y, want, bound, what)

    def run(self, T, residual=False, seed=7):
        x = self.x(T, seed)
        r = self.x(T, seed + 1000) if residual else None
        y, idx, w = self.dev.few(x.cuda(), residual=None if r is None else r.cuda())
        torch.cuda.synchronize()
        self.compare(x, y, idx, w, r, "T=%d" % T)
        return x, y, idx, w


FORMATS = [("bf16", "bf16"), ("int8", "bf16"), ("int4", "bf16"), ("int4b128", "bf16"), ("f32", "f32"), ("f32", "bf16"),
           ("bf16", "f32"), ("int8", "f32"), ("int4", "f32"), ("int4b128", "f32")]


@pytest.mark.parametrize("wfmt,xfmt", FORMATS)
@pytest.mark.parametrize("T", [1, 3, 8, 16])
def test_formats(wfmt, xfmt, T):
    Layer(wfmt=wfmt, xfmt=xfmt).run(T, residual=T != 3)


@pytest.mark.parametrize("wfmt,xfmt", FORMATS)
def test_block_with_shared_expert(wfmt, xfmt):
    Layer(wfmt=wfmt, xfmt=xfmt, shared=384, act="gelu_tanh", I=256).run(5, residual=True)


@pytest.mark.parametrize("wfmt", ["bf16", "int8", "int4", "f32"])
@pytest.mark.parametrize("H,I", [(64, 64), (192, 320), (320, 64), (448, 832), (1088, 192)])
def test_widths_that_are_odd_multiples_of_64(wfmt, H, I):
    Layer(wfmt=wfmt, xfmt="f32" if wfmt == "f32" else "bf16", H=H, I=I, E=8, k=3).run(4, residual=True)


@pytest.mark.parametrize("T", range(1, 17))
def test_every_token_count(T):
    Layer(router="softmax", scale=1.0, E=24, k=6).run(T)


@pytest.mark.parametrize("T", [1, 9, 16])
@pytest.mark.parametrize("wfmt", ["bf16", "int8", "int4"])
def test_every_token_to_the_same_experts(T, wfmt):
    """k = E: each expert gets all tokens."""
    Layer(E=3, k=3, wfmt=wfmt).run(T, residual=True)
    Layer(E=1, k=1, wfmt=wfmt, router="softmax", shared=128).run(T)


def test_limits_of_experts_and_slots():
    Layer(H=64, I=64, E=1024, k=32, router="softmax").run(16)
    Layer(H=64, I=64, E=257, k=1).run(2)


@pytest.mark.parametrize("wfmt", ["bf16", "int8", "int4b128"])
def test_large_widths(wfmt):
    """The limit of the widths, each on one side."""
    Layer(H=8192, I=128, E=2, k=2, wfmt=wfmt).run(2)
    Layer(H=128, I=8192, E=2, k=2, wfmt=wfmt).run(16)


def test_workload_widths():
    """The int8 decode shape of the 256-expert layer with its shared expert, on fewer experts."""
    Layer(H=2304, I=2048, E=12, k=8, wfmt="int8", shared=2048).run(2, residual=True)
    Layer(H=2048, I=768, E=12, k=8, wfmt="int4", router="softmax", scale=1.0).run(3)


@pytest.mark.parametrize("wfmt,T,shared", [("bf16", 1, 2048), ("int8", 4, 512), ("int4", 16, 0), ("int4b128", 2, 1024)])
def test_many_calls_in_a_row_at_workload_widths(wfmt, T, shared):
    """Rings that go round many times: every call has the first one's bits, and no wait runs
    out (the fixture looks at the flags)."""
    layer = Layer(H=2304, I=2048, E=16, k=8, wfmt=wfmt, shared=shared)
    x = layer.x(T).cuda()
    first = [t.clone() for t in layer.dev.few(x, residual=x)]
    for _ in range(30):
        outs = [layer.dev.few(x, residual=x) for _ in range(5)]
        assert all(torch.equal(a, b) for o in outs for a, b in zip(o, first))
        assert moe.moe_device_flags() == 0


def test_mask_equals_slice():
    """Masked experts are never chosen; the result has the same bits as the sliced layer's."""
    full = Layer(E=16, k=4, active=[1, 3, 4, 8, 9, 15])
    x, y, idx, w = full.run(6)
    assert set(idx.unique().tolist()) <= {1, 3, 4, 8, 9, 15}
    keep = torch.tensor([1, 3, 4, 8, 9, 15])
    t = full.dev.tensors
    part = moe.MoELayer(H=256, I=128, E=6, k=4, router="sigmoid", scale=2.446, wfmt="bf16", xfmt="bf16",
                        W_r=t["W_r"].cpu()[keep], b=t["b"].cpu()[keep], W_gate=t["W_gate"].cpu()[keep],
                        W_up=t["W_up"].cpu()[keep], W_down=t["W_down"].cpu()[keep])
    y2, idx2, w2 = part.few(x.cuda())
    assert torch.equal(keep[idx2.cpu().long()].int(), idx.cpu()) and torch.equal(w2, w)
    assert torch.equal(y2.view(torch.int16), y.view(torch.int16))


@pytest.mark.flags
@pytest.mark.parametrize("active", [[], [5], [2, 11]])
def test_fewer_selectable_experts_than_slots(active):
    layer = Layer(active=active, shared=128)
    x = layer.x(3)
    y, idx, w = layer.dev.few(x.cuda(), residual=x.cuda())
    assert moe.moe_device_flags(clear=True) == 2  # MOE_FLAG_TOO_FEW_ACTIVE
    layer.compare(x, y, idx, w, x)
    assert bool((idx[:, len(active):] == -1).all()) and bool((w[:, len(active):] == 0).all())


@pytest.mark.flags
@pytest.mark.parametrize("wfmt", ["bf16", "int8", "int4"])
def test_infinity_and_nan_stay_in_their_token(wfmt):
    layer = Layer(wfmt=wfmt, shared=128)
    x = layer.x(4)
    clean = layer.dev.few(x.cuda())[0].clone()
    moe.moe_device_flags(clear=True)
    x[1, 5] = float("nan")
    x[3, 0] = float("inf")
    y, idx, w = layer.dev.few(x.cuda())
    assert moe.moe_device_flags(clear=True) & moe.MOE_FLAG_NONFINITE_LOGIT
    assert bool((idx[[1, 3]] == -1).all()) and bool((w[[1, 3]] == 0).all())
    assert torch.equal(y[[0, 2]].view(torch.int16), clean[[0, 2]].view(torch.int16))
    assert not bool(y[[1, 3]].isfinite().any())  # the shared expert still saw them


@pytest.mark.flags
def test_nonfinite_weights_of_masked_and_unchosen_experts_do_not_matter():
    layer = Layer(active=range(8))
    x, y, idx, w = layer.run(3)
    t = layer.dev.tensors
    unused = sorted(set(range(16)) - set(idx.unique().tolist()))
    for n, e in enumerate(unused):
        for part in ("W_gate", "W_up", "W_down"):
            t[part][e] = float("nan") if n % 2 else float("inf")
    y2, idx2, _ = layer.dev.few(x.cuda())
    assert torch.equal(y2.view(torch.int16), y.view(torch.int16)) and torch.equal(idx2, idx)


@pytest.mark.parametrize("wfmt", ["int8", "int4", "int4b128"])
@pytest.mark.parametrize("scale", [1e-30, 1e-6, 1e6, 1e18])
def test_tokens_of_any_magnitude(wfmt, scale):
    """Digits are relative to the token's largest value: its magnitude does not matter."""
    layer = Layer(wfmt=wfmt, bias=False)
    x = (layer.x(3).float() * torch.tensor([1.0, scale, 0.0])[:, None]).to(torch.bfloat16)
    y, idx, w = layer.dev.few(x.cuda())
    layer.compare(x, y, idx, w)


@pytest.mark.parametrize("wfmt", ["bf16", "int8", "int4"])
def test_outliers_in_a_token(wfmt):
    """A few columns thousands of times the others, as hidden states have them."""
    layer = Layer(wfmt=wfmt, shared=128)
    x = layer.x(5).float()
    x[:, 7] *= 4000
    x[1, 200] = -30000.0
    x = x.to(torch.bfloat16)
    y, idx, w = layer.dev.few(x.cuda())
    layer.compare(x, y, idx, w)


def test_beside_other_work():
    """CTAs that cannot start because other work holds their SMs: their units are taken over,
    and the results do not change."""
    layer = Layer(E=64, k=8, H=1024, I=1024, wfmt="int8", shared=512)
    xs = [layer.x(n, 60 + n).cuda() for n in (1, 4, 16)]
    want = [[t.clone() for t in layer.dev.few(x)] for x in xs]
    a = torch.randn(8192, 8192, device="cuda", dtype=torch.bfloat16)
    busy, mine = torch.cuda.Stream(), [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(15):
        with torch.cuda.stream(busy):
            a @ a
        for s in mine:
            with torch.cuda.stream(s):
                got += [(n, layer.dev.few(x)) for n, x in enumerate(xs)]
    torch.cuda.synchronize()
    for n, out in got:
        assert all(torch.equal(p, q) for p, q in zip(out, want[n]))


def test_large_activations_overflow_no_sooner_than_fp32():
    """Gate sums far out: SiLU ends at 0 on one side and at the identity on the other."""
    layer = Layer()
    x = layer.x(2) * 300
    y, idx, w = layer.dev.few(x.to(torch.bfloat16).cuda())
    layer.compare(x.to(torch.bfloat16), y, idx, w)


def test_ties_go_to_the_lower_expert():
    W_r = torch.from_numpy(synth.normal_f32((1, 256), 3, 2, 0.0, 0.05)).repeat(16, 1)
    layer = Layer(W_r=W_r, bias=False)
    x, y, idx, w = layer.run(5)
    assert torch.equal(idx.cpu(), torch.arange(4, dtype=torch.int32).repeat(5, 1))


@pytest.mark.parametrize("router", ["sigmoid", "softmax"])
def test_borders_closer_than_fp32_sums_resolve(router):
    """Experts whose logits differ by 2^-30 relative: every sum of 1,024 products in fp32
    would mix them up."""
    base = torch.from_numpy(synth.normal_f32((1, 1024), 5, 2, 0.0, 0.05))
    W_r = base.repeat(16, 1)
    order = [3, 14, 0, 7, 9, 1, 12, 5, 15, 8, 2, 11, 6, 13, 4, 10]
    x = torch.ones(2, 1024)
    for rank, e in enumerate(order):
        W_r[e, 100] = 2.0 ** -24 * (17 - rank)
    layer = Layer(H=1024, E=16, k=6, W_r=W_r, bias=False, router=router, scale=1.0)
    y, idx, w = layer.dev.few(x.to(torch.bfloat16).cuda())
    assert idx.cpu().tolist() == [order[:6]] * 2


def test_in_place_residual_and_untouched_neighbours():
    layer = Layer(shared=128)
    T, guard = 3, 5
    x = layer.x(T)
    r = layer.x(T, 99)
    y0, idx0, w0 = layer.dev.few(x.cuda(), residual=r.cuda())
    big_y = torch.full((T + guard, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    big_i = torch.full((T + guard, 4), 77, dtype=torch.int32, device="cuda")
    big_w = torch.full((T + guard, 4), 7.0, device="cuda")
    big_y[:T] = r.cuda()
    layer.dev.few(x.cuda(), residual=big_y[:T], out=(big_y[:T], big_i[:T], big_w[:T]))
    assert torch.equal(big_y[:T], y0) and torch.equal(big_i[:T], idx0) and torch.equal(big_w[:T], w0)
    assert bool((big_y[T:] == 7).all()) and bool((big_i[T:] == 77).all()) and bool((big_w[T:] == 7).all())


def test_same_call_same_bits_on_a_dirty_workspace():
    layer = Layer(wfmt="int8", shared=256, E=32, k=8)
    x = layer.x(16).cuda()
    first = [t.clone() for t in layer.dev.few(x)]
    for fill in (0, 255, 77):
        for _, ws in layer.dev._few_ws.values():
            ws.fill_(fill)
        again = layer.dev.few(x)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_matches_the_separate_entry_points():
    """Same formulas as moe_route + moe_forward_block: where both route alike, the outputs
    agree within the two calls' bounds."""
    layer = Layer(shared=128, seed=4)
    x, y, idx, w = layer.run(16, residual=True)
    i2, w2 = layer.dev.route(x.cuda())
    same = (i2 == idx).all(1)
    assert int(same.sum()) >= 15
    assert bool(((w2 - w)[same].abs() <= 1e-5 * w[same].abs()).all())


def test_captured_and_replayed_with_new_inputs():
    layer = Layer(shared=128, wfmt="int8")
    x = layer.x(4).cuda()
    out = tuple(t.clone() for t in layer.dev.few(x))  # first call: per-device setup
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.dev.few(x, out=out)
    for seed in (21, 22, 23):
        new = layer.x(4, seed)
        x.copy_(new)
        for t in out:
            t.zero_()
        g.replay()
        g.replay()
        torch.cuda.synchronize()
        layer.compare(new, *out)


@pytest.mark.parametrize("wfmt,xfmt", [("int8", "bf16"), ("f32", "f32")])
def test_graphs_keep_workspaces_of_their_own(wfmt, xfmt):
    """Two captured calls replayed at once, after the eager workspace was replaced by a larger one."""
    layer = Layer(E=64, k=8, H=512, I=512, wfmt=wfmt, xfmt=xfmt)
    xs = [layer.x(3, 60 + n).cuda() for n in range(2)]
    want = [[t.clone() for t in layer.dev.few(x)] for x in xs]
    outs, graphs = [tuple(torch.zeros_like(t) for t in w) for w in want], []
    for x, out in zip(xs, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            layer.dev.few(x, out=out)
    layer.dev.few(layer.x(16).cuda())
    other = [torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(16)]
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for out, w in zip(outs, want) for a, b in zip(out, w))
    assert all(bool((t == 255).all()) for t in other)


def test_two_streams_at_once():
    """Calls that overlap on the GPU, each stream with its own workspace: many at once."""
    layer = Layer(E=64, k=8, H=512, I=512, wfmt="bf16")
    xs = [layer.x(n + 1, 40 + n).cuda() for n in range(6)]
    want = [[t.clone() for t in layer.dev.few(x)] for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for s, x in zip(streams, xs):
            with torch.cuda.stream(s):
                got.append(layer.dev.few(x))
    torch.cuda.synchronize()
    for n, out in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(out, want[n % len(xs)]))


def test_wrapper_refusals():
    layer = Layer()
    x = layer.x(2).cuda()
    for bad in (x.float(), x[:, :128], x.T, x.cpu(), layer.x(17).cuda(), torch.stack((x, x), 1)[:, 0]):
        with pytest.raises(moe.MoeError):
            layer.dev.few(bad)
    with pytest.raises(moe.MoeError):
        layer.dev.few(x, residual=x[:1])
    y, idx, w = layer.dev.few(x[:0])
    assert y.shape == (0, 256) and idx.shape == (0, 4)


def test_dense_layer_then_routed_layers():
    """Two layers of a decoder's feed-forward stack as they are used: the dense first layer
    (gated product, then the product into the residual stream) and a routed layer with
    its shared expert on the result, captured as one graph and replayed."""
    H, F = 256, 640
    layer = Layer(H=H, I=128, E=16, k=4, wfmt="int8", shared=128)
    Wg, sg, dg = ref.weights(F, H, "int8", 61)
    Wu, su, du = ref.weights(F, H, "int8", 62)
    Wd, sd, dd = ref.weights(H, F, "int8", 63)
    up = moe.Linear(K=H, N=F, wfmt="int8", xfmt="bf16", W=Wg, s=sg, W_up=Wu, s_up=su, act="silu")
    down = moe.Linear(K=F, N=H, wfmt="int8", xfmt="bf16", W=Wd, s=sd)
    x = layer.x(5).cuda()

    def step():
        h = up(x)
        y = down(h, residual=x)
        return h, y, layer.dev.few(y, residual=y)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        h, y, (z, idx, w) = step()
    for seed in (71, 72):
        new = layer.x(5, seed)
        x.copy_(new)
        g.replay()
        torch.cuda.synchronize()
        # each step is compared on the inputs that it had
        want, bound = ref.linear(new, dg, None, (du, None), "silu", None, torch.bfloat16, "int8")
        ref.check(h, want, bound, "up")
        want, bound = ref.linear(h.cpu(), dd, None, None, "none", new, torch.bfloat16, "int8")
        ref.check(y, want, bound, "down")
        layer.compare(y.cpu(), z, idx, w, y.cpu(), "routed")


@pytest.mark.parametrize("wfmt,xfmt,tol", [("bf16", "bf16", 5e-3), ("int8", "bf16", 5e-3), ("int4", "bf16", 5e-3),
                                           ("int4b128", "bf16", 5e-3), ("f32", "f32", 1e-5)])
@pytest.mark.parametrize("T", [1, 16])
def test_outputs_are_those_of_the_separate_entry_points(wfmt, xfmt, tol, T):
    """moe_route + moe_forward_block on the tokens that both route alike: no further apart than the
    other calls' tolerance against 64 bits and this one's bound together."""
    layer = Layer(shared=128, seed=4, wfmt=wfmt, xfmt=xfmt)
    x, y, idx, w = layer.run(T, residual=True)
    r = layer.x(T, 7 + 1000)
    i2, w2 = layer.dev.route(x.cuda())
    y2 = layer.dev.block(x.cuda(), i2, w2, residual=r.cuda())
    same = (i2 == idx).all(1).cpu()
    assert int(same.sum()) >= T - 1
    ri, rw = ref.route(x, layer.W_r, layer.b, layer.mask, layer.k, layer.router, layer.scale)
    want, bound = ref.few(x, ri, rw, layer.experts, layer.act, layer.shared, r)
    off = (y.cpu().double() - y2.cpu().double())[same].norm()
    assert float(off) <= tol * float(want[same].norm()) + float(bound[same].norm())
