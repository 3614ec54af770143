"""The lives of the workspaces that PagedNVFP4Cache keeps: over streams, plans and captured graphs."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HOLD = 400_000_000  # clock cycles of a kernel that only waits: 0.2 s and more


class Session:
    """One sequence whose slots are all in the pool's one page (zeros), with a short and a long plan.
    The short plan's weights workspace takes 13 MB: the allocator hands such a block out whole."""

    def __init__(self):
        import bit_kv_cache_03_gb300 as k
        self.c = k.PagedNVFP4Cache(1, np.zeros((1, 4096), np.int32), 64, 24, 4)
        self.c.pool.zero_()
        self.w = self.c.weight_accounts()
        self.qc, self.qs = self.c.quantized_q_buffers(1)
        self.qc.zero_(), self.qs.zero_()
        self.out = torch.empty(1, 24, 128, dtype=torch.bfloat16, device="cuda")
        self.plans = []
        for n in (131072, 262144):
            self.c.workspace = None
            self.plans.append((self.c.plan([n], 1), self.c.workspace))
        self.use(0)

    def use(self, i):
        self.c.plan_info, self.c.workspace = self.plans[i]

    def attend(self, stream=None):
        self.c.attend_weights(self.qc, self.qs, self.out, self.w, stream=stream)


def _overlaps(start, size, n=8):
    """Whether one of n further blocks of the current stream's memory lies in [start, start + size)."""
    blocks = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(n)]
    return any(b.data_ptr() < start + size and start < b.data_ptr() + size for b in blocks)


def test_the_weights_workspace_is_not_handed_out_under_a_call_of_another_stream():
    s = Session()
    s.attend()  # allocated for the current stream
    torch.cuda.synchronize()
    start, size = s.c.weights_workspace.data_ptr(), s.c.weights_workspace.numel()
    assert size > 12 << 20
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(HOLD)
        s.attend()
    s.use(1)
    s.attend(stream=side)  # grows
    assert s.c.weights_workspace.data_ptr() != start
    lent = _overlaps(start, size)
    assert not side.query()  # the first call on `side` has still to run
    assert not lent
    torch.cuda.synchronize()
    assert not s.out.any() and int(s.c.status.item()) == 0


def test_the_plan_workspace_is_not_handed_out_under_a_call_of_another_stream(monkeypatch):
    import bit_kv_cache_03_gb300.cache as cache
    s = Session()
    s.attend()
    torch.cuda.synchronize()
    start, size = s.c.workspace.data_ptr(), s.c.workspace.numel()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(HOLD)
        s.attend()
    # the buffers alone: a work list from pageable memory may wait for the stream
    monkeypatch.setattr(cache, "kv_nvfp4_plan", lambda *a: None)
    monkeypatch.setattr(cache, "kv_nvfp4_plan_workspace_bytes", lambda *a: size + 1)
    s.plans = None  # the cache alone holds its workspace
    s.c.plan([64], 1, stream=side)  # grows
    assert s.c.workspace.data_ptr() != start
    lent = _overlaps(start, size)
    assert not side.query()
    assert not lent
    torch.cuda.synchronize()
    assert not s.out.any() and int(s.c.status.item()) == 0


def test_a_plan_workspace_is_memory_of_the_stream_it_is_planned_on(monkeypatch):
    import bit_kv_cache_03_gb300.cache as cache
    s = Session()
    size = 64 << 20
    monkeypatch.setattr(cache, "kv_nvfp4_plan", lambda *a: None)
    monkeypatch.setattr(cache, "kv_nvfp4_plan_workspace_bytes", lambda *a: size)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(HOLD)
    x = torch.ones(size, dtype=torch.uint8, device="cuda")  # written when the wait is over
    start = x.data_ptr()
    del x  # free to the current stream, behind its work; not to another one
    s.plans = None
    s.c.plan([64], 1, stream=side)
    busy = not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert busy and not (start <= s.c.workspace.data_ptr() < start + size)


@pytest.mark.parametrize("given", [False, True])
def test_a_captured_call_keeps_its_workspaces(given):
    s = Session()
    s.plans = s.c.workspace = s.c.weights_workspace = None
    s.c.plan([640], 1)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream = side if given else None
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.attend(stream)
        want = s.w.clone(), s.out.clone()
        with torch.cuda.graph(graph, stream=side):
            s.attend(stream)
    torch.cuda.synchronize()
    held = [(b.data_ptr(), b.numel()) for b in (s.c.workspace, s.c.weights_workspace)]
    s.c.plan([262144], 1)
    s.attend()  # both grow
    torch.cuda.synchronize()
    assert all(b.data_ptr() != at for b, (at, _) in
               zip((s.c.workspace, s.c.weights_workspace), held))
    lent = [_overlaps(at, size, 64) for at, size in held]
    with torch.cuda.stream(side):
        lent += [_overlaps(at, size, 64) for at, size in held]
    assert not any(lent)
    s.w.zero_(), s.out.fill_(1)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(s.w, want[0]) and torch.equal(s.out, want[1])
    assert int(s.c.status.item()) == 0


def test_a_growing_sequence_seldom_needs_another_workspace(monkeypatch):
    import bit_kv_cache_03_gb300 as k
    s = Session()
    s.plans = s.c.workspace = None
    grown = []
    real = k.PagedNVFP4Cache._enlarge
    monkeypatch.setattr(k.PagedNVFP4Cache, "_enlarge",
                        lambda self, name, *a: (grown.append(name), real(self, name, *a))[1])
    for n in range(131072, 131072 + 64 * 64, 64):  # a page more each time
        s.c.plan([n], 1)
        s.attend()
        need = k.kv_nvfp4_weights_workspace_bytes(s.c.layout, s.c.plan_info)
        assert need <= s.c.weights_workspace.numel() <= need + need // 16
    assert grown.count("weights_workspace") == 2  # the first, and one with room for more
    torch.cuda.synchronize()
    assert int(s.c.status.item()) == 0


def test_capturing_is_asked_of_the_given_stream():
    import bit_kv_cache_03_gb300 as k
    side, other, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    x = torch.zeros(4, device="cuda")
    assert not k._capturing(side) and not k._capturing(0)
    with torch.cuda.graph(graph, stream=side):
        x += 1
        seen = [k._capturing(s) for s in (side, side.cuda_stream, other, other.cuda_stream)]
    assert seen == [True, True, False, False] and not k._capturing(side)
    graph.replay()
    torch.cuda.synchronize()
    assert x.tolist() == [1] * 4
