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
