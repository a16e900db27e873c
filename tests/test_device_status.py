"""Which device a status call reads (no GPU needed)."""
import types

import torch

from block_sparse_full_b200 import ssa


def test_device_status_makes_the_device_current(monkeypatch):
    current, read = [0], []

    class Guard:
        def __init__(self, device):
            self.to = None if device is None else torch.device(device).index

        def __enter__(self):
            self.was = current[0]
            current[0] = self.was if self.to is None else self.to

        def __exit__(self, *_):
            current[0] = self.was

    monkeypatch.setattr(torch.cuda, "device", Guard)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda d=None: types.SimpleNamespace(cuda_stream=("stream of", d and str(d))))
    monkeypatch.setattr(ssa, "ssa_device_status", lambda stream: read.append((current[0], stream)) or ssa.SSA_OK)
    ssa.device_status("cuda:1")
    ssa.device_status()
    assert read == [(1, ("stream of", "cuda:1")), (0, ("stream of", None))] and current == [0]
