"""Which forks of a call are carried out, against the header's words."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def dev(x):
    return torch.tensor(np.ascontiguousarray(x), dtype=torch.int32, device="cuda")


def carried_out(src, dst, lens, held):
    """Indices of the forks that are, and whether a sequence, and whether a length, is refused."""
    S, done, bad_seq, bad_pos = len(held), [], False, False
    for i, (a, b, n) in enumerate(zip(src, dst, lens)):
        outside = not (0 <= a < S and 0 <= b < S)
        if outside or held[b] > 0 or b in dst[:i] or a in dst:
            bad_seq = True
        elif n < 0 or n > 64 * held[a]:
            bad_pos = True
        else:
            done.append(i)
    return done, bad_seq, bad_pos


CASES = [
    ([0, 1], [1, 3], [64, 64]),              # the first target holds pages; it is the second one's source
    ([0, 2], [2, 3], [64, 0]),               # a source that is filled by the call
    ([2, 0], [3, 2], [0, 64]),               # the same the other way round
    ([0, 0, 1], [2, 3, 0], [64, 10, 5]),     # a source as the target of a refused fork
    ([9, 0], [0, 3], [1, 1]),                # ... of one whose own source is none
    ([1, 1, 1], [2, 3, 2], [64, 1, 0]),
]


@pytest.mark.parametrize("case", range(30))
def test_forks(case):
    import bit_kv_cache_03_gb300 as kv
    rng = np.random.default_rng(case)
    S, P, N = (4, 4, 10) if case < len(CASES) else (12, 5, 60)
    if case < len(CASES):
        room = np.array([128, 64, 0, 0])
        src, dst, lens = CASES[case]
    else:
        room = np.where(rng.random(S) < 0.5, rng.integers(1, P * 64 + 1, S), 0)
        n = int(rng.integers(1, S + 1))
        src = rng.integers(-1, S + 1, n).tolist()
        dst = rng.choice(np.append(np.flatnonzero(room == 0), rng.integers(-1, S + 1, 2)), n).tolist()
        lens = rng.integers(-1, P * 64 + 1, n).tolist()
    c = kv.PagedNVFP4Cache(N, np.zeros((S, P), np.int32), 1, 4, 2, rot_dim=0)
    pages = c.page_accounts()
    c.resize(dev([0] * S), dev(room))
    table, held, refs, free, count, _ = pages.buffers
    t, h, r = (x.cpu().numpy().copy() for x in (table, held, refs))
    rest = free.clone(), count.clone()
    done, bad_seq, bad_pos = carried_out(src, dst, lens, h.tolist())
    before = t.copy()
    for i in done:
        n = (lens[i] + 63) // 64
        t[dst[i], :n] = before[src[i], :n]
        h[dst[i]] = n
        np.add.at(r, before[src[i], :n], 1)
    c.fork(dev(src), dev(dst), dev(lens))
    torch.cuda.synchronize()
    for got, want in ((table, t), (held, h), (refs, r)):
        assert np.array_equal(got.cpu().numpy(), want)
    assert torch.equal(free, rest[0]) and torch.equal(count, rest[1])
    assert int(c.status.item()) == kv.DEV_BAD_SEQ * bad_seq | kv.DEV_BAD_POS * bad_pos
