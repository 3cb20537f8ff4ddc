"""The binding's memory of workspace sizes (no GPU: the library answers for a
device without SMs)."""
import gc
import sys

import torch


def test_ragged_shapes_do_not_pile_up(monkeypatch):
    import q4_weight_only_gb300 as q4
    from q4_weight_only_gb300 import build
    build.build()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)

    def ask(rows):
        q4.attention_workspace_bytes(rows, 8, 2, 64, rows)   # 0 bytes without an SM

    for rows in range(1, 6000):
        ask(rows)
    gc.collect()
    before = sys.getallocatedblocks()
    for rows in range(6000, 36000):
        ask(rows)
    gc.collect()
    # a size kept for each of 30000 shapes would be several blocks a shape
    assert sys.getallocatedblocks() - before < 10000


def test_sizes_follow_the_arguments_and_the_device(monkeypatch):
    import q4_weight_only_gb300 as q4
    from q4_weight_only_gb300 import _lib, build
    build.build()
    asked = []

    class Library:
        def q4_0_attention_workspace_bytes(self, *args):
            asked.append(args)
            return len(asked)

    monkeypatch.setattr(_lib, "lib", Library)
    device = [1001]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: device[0])
    assert [q4.attention_workspace_bytes(r, 8, 2, 64, 1) for r in (1, 2, 1, 2)] == [1, 2, 1, 2]
    device[0] = 1002
    assert q4.attention_workspace_bytes(1, 8, 2, 64, 1) == 3
    assert asked == [(1, 8, 2, 64, 1), (2, 8, 2, 64, 1), (1, 8, 2, 64, 1)]
