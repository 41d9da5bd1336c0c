"""How calls of the few-token layer and the dense product get on with one another: host threads on
one stream, programmatic launches, CTAs that start late."""
import threading

import pytest
import torch

import mixture_experts_layer_31_b200 as moe
from test_gpu_few import Layer
from test_gpu_linear import Product

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clear_flags():
    moe.moe_device_flags(clear=True)
    yield
    assert moe.moe_device_flags(clear=True) == 0


def _same_in_threads(call, inputs, rounds):
    """Each input from a thread of its own, all on one stream, gives what it gives alone."""
    want = [[t.clone() for t in call(x)] for x in inputs]
    torch.cuda.synchronize()
    got, errors, start = [[] for _ in inputs], [], threading.Barrier(len(inputs))

    def work(n):
        try:
            start.wait()
            for _ in range(rounds):
                got[n].append(call(inputs[n]))
        except Exception as e:  # shown by the assertion below
            errors.append(e)

    threads = [threading.Thread(target=work, args=(n,)) for n in range(len(inputs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for outs, w in zip(got, want):
        assert len(outs) == rounds
        assert all(torch.equal(a, b) for out in outs for a, b in zip(out, w))


@pytest.mark.parametrize("wfmt,xfmt", [("int8", "bf16"), ("bf16", "bf16"), ("f32", "f32")])
def test_few_from_several_threads_on_one_stream(wfmt, xfmt):
    layer = Layer(E=32, k=4, H=512, I=256, wfmt=wfmt, xfmt=xfmt)
    _same_in_threads(lambda x: layer.dev.few(x), [layer.x(4, 80 + n).cuda() for n in range(4)], 60)


@pytest.mark.parametrize("K,N,wfmt,xfmt,M", [
    (4608, 80, "int8", "bf16", 5),      # digits, product
    (2048, 320, "int8", "bf16", 130),   # widened weights, product, sum of the reduction's parts
    (1024, 320, "f32", "f32", 50),      # operands in parts, product, sum
])
def test_linear_from_several_threads_on_one_stream(K, N, wfmt, xfmt, M):
    p = Product(K, N, wfmt, xfmt)
    _same_in_threads(lambda x: [p.dev(x)], [p.x(M, 90 + n).cuda() for n in range(4)], 60)


@pytest.mark.parametrize("wfmt,T", [("bf16", 2), ("int8", 16), ("int4", 5)])
def test_lists_of_ctas_that_start_late_are_taken_over(wfmt, T):
    """A product that holds 80 SMs, with no shared memory left beside it, for a millisecond: calls that
    start meanwhile have CTAs that cannot, and their lists are taken over; the bits are the
    same, and the counter in the workspace says that it happened."""
    layer = Layer(E=64, k=8, H=1024, I=1024, wfmt=wfmt, shared=512)
    x = layer.x(T, 60).cuda()
    busy, mine = torch.cuda.Stream(), torch.cuda.Stream()
    K, N, M = 32768, 1024, 2400  # 40 tiles of the reduction's whole length, each on a pair of SMs
    W = torch.zeros((N, K), device="cuda")
    hold = moe.Linear(K=K, N=N, wfmt="f32", xfmt="f32", W=W)
    a = torch.zeros((M, K), device="cuda")
    with torch.cuda.stream(mine):
        want = [t.clone() for t in layer.dev.few(x, residual=x)]
        taken_over = layer.dev.few_workspace(T, mine.cuda_stream).view(torch.int32)[1]
    with torch.cuda.stream(busy):
        hold(a)
    torch.cuda.synchronize()
    got, counts = [], []
    for _ in range(3):
        with torch.cuda.stream(busy):
            hold(a)
        with torch.cuda.stream(mine):
            for _ in range(30):
                got.append(layer.dev.few(x, residual=x))
                counts.append(taken_over.clone())
    torch.cuda.synchronize()
    moe.release_workspaces()
    assert all(torch.equal(p, q) for out in got for p, q in zip(out, want))
    assert max(int(c) for c in counts) > 0


def test_programmatic_launches_do_not_change_results(tmp_path):
    """MOE_PDL=1 (read once per process, so in a child process): every first launch of a call may then
    start while the call before it ends.  Calls one after the other, whose workspaces are the
    same, give the same bits as in plain stream order."""
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    script = tmp_path / "calls.py"
    script.write_text(
        "import sys, torch\n"
        f"sys.path[:0] = [{os.path.dirname(here)!r}, {here!r}]\n"
        "import mixture_experts_layer_31_b200 as moe\n"
        "from test_gpu_few import Layer\n"
        "from test_gpu_linear import Product\n"
        "ops = []\n"
        "for wfmt, xfmt in (('bf16', 'bf16'), ('int8', 'bf16'), ('int4', 'bf16'), ('f32', 'f32')):\n"
        "    layer = Layer(wfmt=wfmt, xfmt=xfmt, shared=128)\n"
        "    ops += [(lambda x, f=layer.dev: torch.cat([t.flatten().float() for t in f.few(x, residual=x)]), layer.x(T).cuda())\n"
        "            for T in (1, 5)]\n"
        "    product = Product(2048, 96, wfmt, xfmt, bias=True, act='silu')\n"
        "    ops += [(product.dev, product.x(M).cuda()) for M in (1, 5, 20, 70)]\n"
        "out = [[f(x) for f, x in ops] for _ in range(20)]\n"
        "torch.cuda.synchronize()\n"
        "assert moe.moe_device_flags() == 0\n"
        "assert all(torch.equal(a, b) for o in out for a, b in zip(o, out[0]))\n"
        "torch.save([t.cpu() for t in out[0]], sys.argv[1])\n")
    runs = {}
    for pdl in ("0", "1"):
        dst = tmp_path / ("out_%s.pt" % pdl)
        subprocess.run([sys.executable, str(script), str(dst)], check=True, env=dict(os.environ, MOE_PDL=pdl), timeout=300)
        runs[pdl] = torch.load(dst)
    assert len(runs["0"]) == 24
    assert all(torch.equal(a, b) for a, b in zip(runs["0"], runs["1"]))
