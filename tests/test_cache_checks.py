"""What PagedNVFP4Cache refuses before any launch, with the launches replaced by a record (CPU)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def calls(monkeypatch):
    """The library calls that come through, in the place of launches; memory on the CPU."""
    import bit_kv_cache_03_gb300.cache as cache
    seen = []
    for name in ("kv_nvfp4_decode_attn_weights", "kv_nvfp4_evict_select", "kv_nvfp4_evict_compact",
                 "kv_nvfp4_append_slots"):
        monkeypatch.setattr(cache, name, lambda *a, name=name: seen.append(name))
    monkeypatch.setattr(cache.PagedNVFP4Cache, "_check_current", lambda self: None)
    monkeypatch.setattr(cache.PagedNVFP4Cache, "_hold_captured", lambda self, stream: None)
    monkeypatch.setattr(cache.PagedNVFP4Cache, "_enlarge", lambda self, name, need, stream: setattr(
        self, name, torch.empty(need, dtype=torch.uint8)))
    return seen


def _cache(num_seqs=2, plan=(10, 10), q_len=1, Hq=4, H=2):
    import bit_kv_cache_03_gb300 as kv
    c = kv.PagedNVFP4Cache(2 * num_seqs, np.arange(2 * num_seqs, dtype=np.int32).reshape(-1, 2), 1,
                           Hq, H, rot_dim=0, device="cpu")
    c.plan_info = kv.kv_nvfp4_plan_host(c.layout, list(plan), q_len, True, 64, 8)[0]
    c.workspace = torch.empty(1, dtype=torch.uint8)
    out = torch.empty(len(plan) * q_len, Hq, 128, dtype=torch.bfloat16)
    return c, c.quantized_q_buffers(len(plan) * q_len), out, c.weight_accounts()


def test_attend_weights_wants_every_row_of_the_queries(calls):
    c, (codes, scales), out, w = _cache(q_len=3)
    c.attend_weights(codes, scales, out, w)
    c.attend_weights(torch.cat([codes, codes]), torch.cat([scales, scales]), out, w)  # room for more
    assert calls == ["kv_nvfp4_decode_attn_weights"] * 2
    wide = torch.empty(codes.numel(), 2, dtype=torch.uint8)[:, 0]
    for q, s in ((codes[:-1], scales), (codes, scales[:-1]), (codes[:0], scales), (wide, scales),
                 (codes, scales.view(-1, 8)[:, :4]), (codes.to("meta"), scales),
                 (codes, scales.to("meta"))):
        with pytest.raises(ValueError, match="q_codes"):
            c.attend_weights(q, s, out, w)
    assert len(calls) == 2


def test_attend_weights_refuses_a_plan_of_more_sequences(calls):
    c, (codes, scales), out, w = _cache(num_seqs=2, plan=(10, 10, 10))
    with pytest.raises(ValueError, match="sequences"):  # its third one has no table row and no accounts
        c.attend_weights(codes, scales, out, w)
    assert not calls
    c, (codes, scales), out, w = _cache(num_seqs=3, plan=(10, 10))
    c.attend_weights(codes, scales, out, w)  # the first two of three
    assert calls == ["kv_nvfp4_decode_attn_weights"]


def test_the_runtime_that_the_library_is_linked_with_is_reached():
    import bit_kv_cache_03_gb300 as kv
    assert kv.lib().cudaStreamIsCapturing
