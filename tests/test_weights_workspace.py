"""Size of the second workspace of the attention with per-key weights, from the lengths alone (CPU)."""
import pytest


@pytest.mark.parametrize("chunk", [64, 1024])
@pytest.mark.parametrize("Hq,Hkv,q_len", [
    (24, 4, 1), (8, 4, 4), (4, 1, 2), (9, 3, 2),     # the decode kernel, 6 and 8 rows
    (24, 4, 2), (9, 3, 3), (24, 4, 8), (16, 2, 40),  # 9 rows and more: no stored scores
    (32, 8, 1), (40, 5, 1), (24, 6, 2), (8, 8, 8),   # more than four KV heads, up to 8 rows
    (8, 8, 9), (45, 5, 1), (32, 8, 16),              # and 9 and more
])
@pytest.mark.parametrize("causal", [True, False])
def test_the_workspace_holds_statistics_row_sums_and_scores(Hq, Hkv, q_len, chunk, causal):
    import bit_kv_cache_03_gb300 as kv
    L = kv.make_layout(Hq, Hkv)
    lens = [40, 64, 65, 4000, 20001]
    info = kv.kv_nvfp4_plan_host(L, lens, q_len, causal, chunk, 152)[0]
    rows = Hq // Hkv * q_len  # of a KV head
    want = 8 * len(lens) * q_len * Hq                    # (m, 1 / l) of every row
    if rows > 8 or Hkv > 4:
        want += 4 * 128 * info.num_partials              # fp32 row sums of the split groups
    if rows <= 8:                                        # a score per row and slot of a page
        want += sum((n + 63) // 64 for n in lens) * 64 * Hkv * rows * 4
    got = kv.kv_nvfp4_weights_workspace_bytes(L, info)
    assert want <= got <= want + 2 * 256                 # two parts start at multiples of 256
