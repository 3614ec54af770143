"""Corners of the eviction calls' contract: which protected slots a small budget keeps, and what the
calls write outside their own buffers' contents."""
import numpy as np
import pytest

import evictref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def kv():
    import bit_kv_cache_03_gb300 as k
    return k


@pytest.mark.parametrize("lens,keep,sink,recent,want", [
    ([6], [2], 0, 4, [2, 3]),       # the newest two of the last four go, whatever their weights
    ([6], [3], 1, 4, [0, 2, 3]),
    ([6], [5], 1, 4, [0, 2, 3, 4, 5]),
    ([6], [1], 9, 9, [0]),
    ([2000], [512], 4, 1024, [0, 1, 2, 3, *range(976, 1484)]),
])
@pytest.mark.parametrize("per_head", [True, False])
def test_protected_slots_rank_by_slot_alone(lens, keep, sink, recent, want, per_head):
    k = kv()
    w = np.zeros((1, 2, max(lens)), np.float32)
    w[..., :] = np.resize([1, 9, 2, 8, 3, 7], max(lens)) + np.arange(max(lens))  # later ones weigh more
    index = torch.full((1, 2 if per_head else 1, keep[0]), -7, dtype=torch.int32, device="cuda")
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    k.kv_nvfp4_evict_select(k.make_layout(2, 2), torch.from_numpy(w).cuda(), w.shape[2], dev(lens),
                            dev(keep), 1, per_head, sink, recent, index, keep[0], status)
    assert int(status.item()) == 0
    for row in index[0].cpu().numpy():
        assert row.tolist() == want
        assert row.tolist() == evictref.select(w[0, 0], lens[0], keep[0], sink, recent).tolist()
