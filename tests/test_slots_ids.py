"""Request ids of the slot table are any 64-bit numbers."""
import torch

import kv_cached_gqa_rope_gb300 as kv

IDS = (-1, -5, 0, 2 ** 63 - 1, -2 ** 63)


def test_negative_ids_hold_rows_of_their_own():
    t = kv.SlotTable(len(IDS), 8)
    assert [t.admit(r, 1) for r in IDS] == [0, 1, 2, 3, 4]
    assert t.query()["free"] == 0
    meta = torch.zeros(3, 8, dtype=torch.int32)
    t.step(list(IDS), [7, 8, 9, 10, 11], meta)
    assert meta[:, :5].tolist() == [[7, 8, 9, 10, 11], [1] * 5, [0, 1, 2, 3, 4]]
    t.release(-5)
    assert t.admit(3, 2) == 1 and t.admit(-1, 0) == 0
