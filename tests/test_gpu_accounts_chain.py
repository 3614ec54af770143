"""Calls behind a resize without a wait in between: each kernel is launched while those before it run, and
must not read what they have yet to write."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def kv():
    import bit_kv_cache_03_gb300 as k
    return k


def dev(x, dtype=torch.int32):
    return torch.tensor(np.ascontiguousarray(x), dtype=dtype, device="cuda")


@pytest.mark.parametrize("Hq,H,q_len", [(24, 4, 3), (16, 8, 9), (24, 4, 1), (16, 8, 2)])
def test_weights_right_behind_a_resize(Hq, H, q_len):
    """Pages given back and taken anew in another order, then attention with weights, without an append
    in between, with and without a wait behind every call: the same bits. (More than 8 rows per KV head:
    the weight pass reads the table itself.)"""
    S, P, N, steps = 5, 60, 200, 16
    rng = np.random.default_rng(Hq + q_len)
    held = [900, 65, 2600, 129, 3000]
    pool = torch.tensor(rng.integers(0x20, 0x40, (N, 9216 * H), dtype=np.uint8), device="cuda")
    q_codes = dev(rng.integers(0, 256, S * q_len * Hq * 64), torch.uint8)
    q_scales = dev(rng.integers(0x28, 0x38, S * q_len * Hq * 8), torch.uint8)
    lens, none = dev(held), dev([0] * S)
    less = [dev(rng.integers(0, np.array(held) + 1)) for _ in range(steps)]

    def run(wait):
        def done():
            if wait:
                torch.cuda.synchronize()
        c = kv().PagedNVFP4Cache(N, np.zeros((S, P), np.int32), 1, Hq, H, 0)
        c.page_accounts()
        c.pool.copy_(pool.flatten())
        c.resize(none, lens)
        c.plan(held, q_len, causal=False, chunk_tokens=128)
        outs = [torch.empty(S * q_len, Hq, 128, dtype=torch.bfloat16, device="cuda")
                for _ in range(steps)]
        weights = [c.weight_accounts() for _ in range(steps)]
        torch.cuda.synchronize()
        for i in range(steps):
            c.resize(less[i], less[i])
            done()
            c.resize(less[i], lens)
            done()
            c.attend_weights(q_codes, q_scales, outs[i], weights[i])
            done()
        torch.cuda.synchronize()
        assert int(c.status.item()) == 0
        return outs + weights + [c.block_table]

    for i, (a, b) in enumerate(zip(run(True), run(False))):
        assert bool(torch.equal(a.view(torch.uint8), b.view(torch.uint8))), i
