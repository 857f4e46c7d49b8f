"""The operators' binding with stand-ins for the library and CUDA (no GPU)."""
import contextlib
import types

import torch

from pretraining_optimizer_b200 import operators


def test_operator_status_reads_the_streams_device(monkeypatch):
    """The record is the device's: a stream of another device than the current one reads that device's."""
    current, seen = [0], []

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], torch.device(d).index
        yield
        current[0] = before

    def status(handle):
        seen.append((handle, current[0]))
        return 0

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda d=None: types.SimpleNamespace(device=torch.device("cuda", current[0]), cuda_stream=7))
    monkeypatch.setattr(operators, "library", lambda: types.SimpleNamespace(muonh_operator_status=status))
    operators.operator_status(types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=42))
    operators.operator_status()
    assert seen == [(42, 1), (7, 0)] and current == [0]


def test_which_stacks_are_apart():
    """Against the addresses themselves, for every small stack with unit column stride."""
    for batch in (1, 2, 3, 5):
        for rows in (1, 2, 4):
            for cols in (1, 3, 4):
                for ld in range(cols, 4 * cols + 2):
                    for stride in range(0, 40):
                        at = [b * stride + i * ld + j for b in range(batch) for i in range(rows) for j in range(cols)]
                        got = operators._apart(batch, rows, cols, stride, ld)
                        assert got == (len(set(at)) == len(at)), (batch, rows, cols, stride, ld)
