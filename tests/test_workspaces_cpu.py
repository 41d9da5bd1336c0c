"""Workspaces that the wrappers of the few-token layer and the dense product keep: host logic,
with the library's launching calls replaced by ones that only take note of their arguments."""
import threading
import time
import types

import pytest
import torch

import mixture_experts_layer_31_b200 as moe


class _Calls:
    """The library, but for the calls that launch: those say which workspaces are in use at once."""

    def __init__(self, real, pause=0.0):
        self.real, self.pause = real, pause
        self.busy, self.overlaps, self.seen = set(), 0, []
        self.guard = threading.Lock()

    def __getattr__(self, name):
        return getattr(self.real, name)

    def _call(self, ws, n, stream):
        with self.guard:
            self.overlaps += ws in self.busy
            self.busy.add(ws)
            self.seen.append((ws, n, stream))
        time.sleep(self.pause)  # as a foreign call does, this lets other threads run
        with self.guard:
            self.busy.discard(ws)
        return 0

    def moe_few_forward(self, d, shared, x, T, idx, w, residual, y, ws, n, stream):
        return self._call(ws, n, stream)

    def moe_linear(self, d, x, ldx, M, residual, ldr, y, ldy, ws, n, stream):
        return self._call(ws, n, stream)


@pytest.fixture
def calls(monkeypatch):
    fake = _Calls(moe.lib())
    monkeypatch.setattr(moe, "lib", lambda: fake)
    monkeypatch.setattr(moe, "_require", lambda ok, message: None)  # tensors are on the CPU here
    monkeypatch.setattr(moe, "_capturing", lambda torch: False)
    fake.stream = 7
    monkeypatch.setattr(moe, "_raw_stream", lambda torch, device: fake.stream)
    return fake


def _without_gpu(op):
    op.torch = types.SimpleNamespace(**{n: getattr(torch, n) for n in ("empty", "uint8", "int32", "float32", "bfloat16")},
                                     _C=types.SimpleNamespace(_cuda_getDevice=lambda: None))
    return op


def _layer(H=128, I=64, E=8, k=2):
    bf = lambda *shape: torch.zeros(shape, dtype=torch.bfloat16)
    op = moe.MoELayer(H=H, I=I, E=E, k=k, router="softmax", scale=1.0, wfmt="bf16", xfmt="bf16", W_r=torch.zeros(E, H),
                      W_gate=bf(E, I, H), W_up=bf(E, I, H), W_down=bf(E, H, I), device="cpu")
    return _without_gpu(op), lambda T: op.few(bf(T, H))


def _linear(K=128, N=24, xfmt="f32"):
    op = moe.Linear(K=K, N=N, wfmt="f32", xfmt=xfmt, W=torch.zeros(N, K), device="cpu")
    dtype = torch.float32 if xfmt == "f32" else torch.bfloat16
    return _without_gpu(op), lambda M: op(torch.zeros(M, K, dtype=dtype))


@pytest.mark.parametrize("make,rows", [(_layer, 3), (_linear, 40)])
def test_threads_take_turns_with_a_workspace(calls, make, rows):
    """A call is several launches that hand results over in the workspace: two host threads on one
    stream must not interleave theirs."""
    calls.pause = 0.002
    _, call = make()
    start = threading.Barrier(3)

    def work():
        start.wait()
        for _ in range(5):
            call(rows)

    threads = [threading.Thread(target=work) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(calls.seen) == 15 and calls.overlaps == 0


@pytest.mark.parametrize("make,rows", [(_layer, 3), (_linear, 40)])
def test_threads_on_streams_of_their_own_do_not_wait_for_one_another(calls, monkeypatch, make, rows):
    """While one thread is inside a call on its stream, another's call on another stream goes through."""
    _, call = make()
    inside, go_on = threading.Event(), threading.Event()
    mine = threading.local()
    monkeypatch.setattr(moe, "_raw_stream", lambda torch, device: getattr(mine, "stream", 7))
    plain = calls._call

    def waiting(ws, n, stream):
        if stream == 8:
            inside.set()
            assert go_on.wait(20)
        return plain(ws, n, stream)

    calls._call = waiting

    def other():
        mine.stream = 8
        call(rows)

    t = threading.Thread(target=other)
    t.start()
    assert inside.wait(20)
    free = threading.Thread(target=call, args=(rows,))
    free.start()
    free.join(10)
    done = not free.is_alive()
    go_on.set()
    t.join()
    free.join()
    assert done and len({ws for ws, _, _ in calls.seen}) == 2


def test_products_share_a_workspace_for_each_stream(calls):
    """A workspace can hold the whole widened matrix: many objects keep the largest one, not one each."""
    moe.release_workspaces()
    (a, call_a), (b, call_b) = _linear(), _linear(K=256, N=40)
    call_b(40)
    call_a(40)
    call_b(20)
    assert len({ws for ws, _, _ in calls.seen}) == 1
    assert [n for _, n, _ in calls.seen] == 3 * [moe.moe_linear_workspace_size(b.desc, 40)]
    calls.stream = 8
    call_a(40)
    assert calls.seen[-1][0] != calls.seen[0][0]
    calls.stream = 7
    call_b(900)  # more than there is: replaced for all of them
    call_a(40)
    assert calls.seen[-1][:2] == calls.seen[-2][:2] and calls.seen[-1][1] >= moe.moe_linear_workspace_size(b.desc, 900)
    assert len(a._ws) == 2
    moe.release_workspaces()
    assert len(a._ws) == 0 and len(b._ws) == 0
    call_a(40)
    assert calls.seen[-1][1] == max(256, moe.moe_linear_workspace_size(a.desc, 40))
    moe.release_workspaces()


def test_threads_take_turns_with_a_workspace_of_several_products(calls):
    calls.pause = 0.002
    some = [_linear()[1], _linear(K=256)[1]]
    start = threading.Barrier(4)

    def work(call):
        start.wait()
        for _ in range(5):
            call(40)

    threads = [threading.Thread(target=work, args=(some[n % 2],)) for n in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(calls.seen) == 20 and calls.overlaps == 0
    moe.release_workspaces()
