"""Host-side checks of the few-token layer and the dense product that need no GPU:
sizes, refusals with the documented status before anything is launched, no-ops."""
import ctypes

import pytest

import mixture_experts_layer_31_b200 as moe

FAKE = 1 << 20  # never dereferenced: validation and sizing only
INVALID, UNSUPPORTED, WORKSPACE = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE


def _few_desc(**kw):
    d = moe.moe_desc()
    d.H, d.I, d.E, d.k = 256, 128, 16, 4
    d.router, d.act, d.wfmt, d.xfmt, d.path, d.scale = 0, 0, moe.MOE_W_BF16, moe.MOE_X_BF16, 0, 2.446
    d.W_r = d.W_gate = d.W_up = d.W_down = FAKE
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def _shared(**kw):
    sh = moe.moe_shared_expert()
    sh.I, sh.wfmt = 256, moe.MOE_W_BF16
    sh.W_gate = sh.W_up = sh.W_down = FAKE
    for k, v in kw.items():
        setattr(sh, k, v)
    return sh


def _refused(status, call, *args):
    launches = moe.moe_launch_count()
    with pytest.raises(moe.MoeError) as ei:
        call(*args)
    assert ei.value.status == status, str(ei.value)
    assert moe.moe_last_error()
    assert moe.moe_launch_count() == launches


def test_few_workspace_covers_tokens_and_the_shared_expert():
    one, most = moe.moe_few_workspace_size(_few_desc(), None, 1), moe.moe_few_workspace_size(_few_desc(), None, 16)
    assert 0 < one < most and one % 256 == 0
    assert moe.moe_few_workspace_size(_few_desc(), _shared(), 16) > most


@pytest.mark.parametrize("T", [17, 32, 4096])
def test_few_refuses_more_tokens_than_it_is_for(T):
    _refused(UNSUPPORTED, moe.moe_few_workspace_size, _few_desc(), None, T)
    _refused(UNSUPPORTED, moe.moe_few_forward, _few_desc(), None, FAKE, T, FAKE, FAKE, None, FAKE, FAKE, 1 << 40)


@pytest.mark.parametrize("kw,status", [
    (dict(H=100), INVALID), (dict(k=17), INVALID), (dict(E=2048), UNSUPPORTED), (dict(act=moe.MOE_ACT_NONE), INVALID),
    (dict(router=3), INVALID), (dict(wfmt=moe.MOE_W_INT8_ROW), INVALID), (dict(W_r=None), INVALID),
    (dict(W_down=FAKE + 8), INVALID), (dict(scale=float("nan")), INVALID), (dict(H=8256), UNSUPPORTED),
])
def test_few_refuses_bad_descriptors(kw, status):
    _refused(status, moe.moe_few_workspace_size, _few_desc(**kw), None, 4)
    _refused(status, moe.moe_few_forward, _few_desc(**kw), None, FAKE, 4, FAKE, FAKE, None, FAKE, FAKE, 1 << 40)


def test_few_refuses_bad_shared_experts():
    for kw, status in ((dict(I=96), INVALID), (dict(wfmt=moe.MOE_W_F32), UNSUPPORTED), (dict(W_up=None), INVALID),
                       (dict(I=16384), UNSUPPORTED)):
        _refused(status, moe.moe_few_workspace_size, _few_desc(), _shared(**kw), 4)


def test_few_refuses_bad_buffers():
    d, T = _few_desc(), 4
    need = moe.moe_few_workspace_size(d, None, T)
    ok = dict(x=FAKE, idx=FAKE, w=FAKE, res=FAKE, y=FAKE, ws=FAKE, n=need)
    for kw, status in ((dict(x=None), INVALID), (dict(x=FAKE + 8), INVALID), (dict(y=None), INVALID),
                       (dict(y=FAKE + 2), INVALID), (dict(idx=None), INVALID), (dict(w=FAKE + 2), INVALID),
                       (dict(res=FAKE + 4), INVALID), (dict(ws=None), WORKSPACE), (dict(ws=FAKE + 128), WORKSPACE),
                       (dict(n=need - 1), WORKSPACE)):
        a = dict(ok, **kw)
        _refused(status, moe.moe_few_forward, d, None, a["x"], T, a["idx"], a["w"], a["res"], a["y"], a["ws"], a["n"])
    _refused(INVALID, moe.moe_few_forward, d, None, FAKE, -1, FAKE, FAKE, None, FAKE, FAKE, need)


def _linear_desc(**kw):
    d = moe.moe_linear_desc()
    d.K, d.N, d.act, d.wfmt, d.xfmt, d.yfmt = 256, 99, moe.MOE_ACT_NONE, moe.MOE_W_BF16, moe.MOE_X_BF16, moe.MOE_X_BF16
    d.W = FAKE
    for k, v in kw.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("kw,status", [
    (dict(K=0), INVALID), (dict(N=0), INVALID), (dict(K=-8), INVALID), (dict(K=260), INVALID), (dict(K=65544), UNSUPPORTED),
    (dict(N=(1 << 24) + 1), UNSUPPORTED), (dict(act=3), INVALID), (dict(wfmt=5), INVALID), (dict(xfmt=2), INVALID),
    (dict(yfmt=-1), INVALID), (dict(W=None), INVALID), (dict(W=FAKE + 8), INVALID), (dict(W_up=FAKE + 8), INVALID),
    (dict(b=FAKE + 2), INVALID), (dict(wfmt=moe.MOE_W_INT8_ROW), INVALID),
    (dict(wfmt=moe.MOE_W_INT8_ROW, s=FAKE, W_up=FAKE), INVALID),  # gated without the second scales
    (dict(wfmt=moe.MOE_W_INT8_ROW, s=FAKE, K=264), INVALID), (dict(wfmt=moe.MOE_W_INT4_B32, s=FAKE, K=272), INVALID),
    (dict(wfmt=moe.MOE_W_INT4_B128, s=FAKE, K=320), INVALID), (dict(wfmt=moe.MOE_W_F32, xfmt=moe.MOE_X_F32, K=258), INVALID),
])
def test_linear_refuses_bad_descriptors(kw, status):
    _refused(status, moe.moe_linear_workspace_size, _linear_desc(**kw), 4)
    d = _linear_desc(**kw)
    _refused(status, moe.moe_linear, d, FAKE, 1 << 17, 4, None, 0, FAKE, 1 << 25, FAKE, 1 << 40)


def test_linear_accepts_every_format():
    for wfmt in range(5):
        for act in (moe.MOE_ACT_NONE, moe.MOE_ACT_SILU, moe.MOE_ACT_GELU_TANH):
            for M in (0, 1, 100, 5000):
                assert moe.moe_linear_workspace_size(_linear_desc(wfmt=wfmt, s=FAKE, act=act), M) >= 0


def test_linear_refuses_bad_buffers():
    d, M = _linear_desc(), 4
    need = moe.moe_linear_workspace_size(d, M)
    ok = dict(x=FAKE, ldx=256, res=None, ldr=0, y=FAKE, ldy=99, ws=FAKE, n=max(need, 256))
    cases = [(dict(x=None), INVALID), (dict(x=FAKE + 8), INVALID), (dict(ldx=248), INVALID), (dict(ldx=260), INVALID),
             (dict(ldx=-256), INVALID), (dict(y=None), INVALID), (dict(y=FAKE + 1), INVALID), (dict(ldy=98), INVALID),
             (dict(res=FAKE, ldr=98), INVALID), (dict(res=FAKE + 1, ldr=99), INVALID),
             (dict(res=FAKE, ldr=99, ldy=100), INVALID)]  # in place with other row distances
    if need:
        cases += [(dict(ws=None), WORKSPACE), (dict(ws=FAKE + 128), WORKSPACE), (dict(n=need - 1), WORKSPACE)]
    for kw, status in cases:
        a = dict(ok, **kw)
        _refused(status, moe.moe_linear, d, a["x"], a["ldx"], M, a["res"], a["ldr"], a["y"], a["ldy"], a["ws"], a["n"])
    _refused(INVALID, moe.moe_linear, d, FAKE, 256, -1, None, 0, FAKE, 99, FAKE, 256)
    _refused(UNSUPPORTED, moe.moe_linear, d, FAKE, 256, (1 << 21) + 1, None, 0, FAKE, 99, FAKE, 1 << 60)


def test_no_tokens_launch_nothing():
    n = moe.moe_launch_count()
    moe.moe_few_forward(_few_desc(), None, None, 0, None, None, None, None, None, 0)
    moe.moe_linear(_linear_desc(), None, 256, 0, None, 0, None, 99, None, 0)
    assert moe.moe_launch_count() == n


def test_null_outputs_are_refused():
    for f, d in ((moe.lib().moe_few_workspace_size, _few_desc()),):
        assert f(ctypes.byref(d), None, 4, None) == INVALID
    assert moe.lib().moe_linear_workspace_size(ctypes.byref(_linear_desc()), 4, None) == INVALID
    assert moe.lib().moe_linear_workspace_size(None, 4, None) == INVALID


def test_wrappers_refuse_tensors_of_another_place_or_shape():
    """The convenience classes check tensors before any call into the library."""
    torch = pytest.importorskip("torch")
    lin = moe.Linear(K=64, N=5, wfmt="bf16", xfmt="bf16", W=torch.zeros(5, 64, dtype=torch.bfloat16), device="cpu")
    for x in (torch.zeros(3, 64, dtype=torch.bfloat16),  # not on a GPU
              torch.zeros(3, 64), torch.zeros(3, 32, dtype=torch.bfloat16),
              torch.zeros(64, 3, dtype=torch.bfloat16).T):
        with pytest.raises(moe.MoeError) as ei:
            lin(x)
        assert ei.value.status == INVALID


def _linear_tensors(**kw):
    torch = pytest.importorskip("torch")
    N, K = 6, 256
    t = dict(f32=dict(W=torch.zeros(N, K)), bf16=dict(W=torch.zeros(N, K, dtype=torch.bfloat16)),
             int8=dict(W=torch.zeros(N, K, dtype=torch.int8), s=torch.zeros(N)),
             int4=dict(W=torch.zeros(N, K // 2, dtype=torch.uint8), s=torch.zeros(N, K // 32)),
             int4b128=dict(W=torch.zeros(N, K // 2, dtype=torch.uint8), s=torch.zeros(N, K // 128)))[kw.pop("wfmt")]
    return dict(t, **kw)


@pytest.mark.parametrize("wfmt", ["f32", "bf16", "int8", "int4", "int4b128"])
def test_linear_refuses_tensors_that_its_kernels_would_read_out_of_range(wfmt):
    torch = pytest.importorskip("torch")
    make = lambda **kw: moe.Linear(K=256, N=6, wfmt=wfmt, xfmt="bf16", device="cpu", **_linear_tensors(wfmt=wfmt, **kw))
    good = _linear_tensors(wfmt=wfmt)
    make(b=torch.zeros(6), W_up=good["W"].clone(), s_up=good.get("s"), b_up=torch.zeros(6))
    bad = [dict(W=good["W"][:5]), dict(W=good["W"][:, :-1]), dict(W=good["W"].to(torch.float64)), dict(W=None),
           dict(W_up=good["W"][:5], s_up=good.get("s")), dict(b=torch.zeros(5)), dict(b=torch.zeros(6, dtype=torch.bfloat16)),
           dict(W_up=good["W"], s_up=good.get("s"), b_up=torch.zeros(12))]
    if "s" in good:
        bad += [dict(s=good["s"][:5]), dict(s=good["s"].to(torch.float16)), dict(W_up=good["W"], s_up=good["s"][1:])]
    for kw in bad:
        with pytest.raises(moe.MoeError) as ei:
            make(**kw)
        assert ei.value.status == INVALID


@pytest.mark.parametrize("bad", [None, "W_r", "b", "expert_mask", "W_gate", "W_up", "W_down", "s_gate", "s_up", "s_down", "Ws_gate",
                                 "Ws_up", "Ws_down", "ss_gate", "ss_up", "ss_down"])
@pytest.mark.parametrize("wfmt", ["f32", "bf16", "int8", "int4", "int4b128"])
def test_few_refuses_tensors_that_its_kernels_would_read_out_of_range(wfmt, bad):
    torch = pytest.importorskip("torch")
    H, I, E, Is = 256, 128, 4, 128
    kw = dict(W_r=torch.zeros(E, H), b=torch.zeros(E), expert_mask=torch.ones(E, dtype=torch.uint8))
    for prefix, lead, width in (("", (E,), I), ("s", (), Is)):
        for part, r, c in (("gate", width, H), ("up", width, H), ("down", H, width)):
            dtype, n, s = {"f32": (torch.float32, c, None), "bf16": (torch.bfloat16, c, None), "int8": (torch.int8, c, ()),
                           "int4": (torch.uint8, c // 2, (c // 32,)), "int4b128": (torch.uint8, c // 2, (c // 128,))}[wfmt]
            kw["W%s_%s" % (prefix, part)] = torch.zeros(lead + (r, n), dtype=dtype)
            kw["s%s_%s" % (prefix, part)] = None if s is None else torch.zeros(lead + (r,) + s)
    if bad is not None and kw[bad] is None:
        return  # the format has no scales
    if bad is not None:
        kw[bad] = kw[bad][:-1]
    x = torch.zeros(2, H, dtype=torch.bfloat16)
    layer = moe.MoELayer(H=H, I=I, E=E, k=2, router="sigmoid", scale=1.0, wfmt=wfmt, xfmt="bf16", I_s=Is, device="cpu", **kw)
    with pytest.raises(moe.MoeError) as ei:
        layer.few(x)
    assert ei.value.status == INVALID
    assert ("must hold" in str(ei.value)) == (bad is not None)  # else it is the place of x
