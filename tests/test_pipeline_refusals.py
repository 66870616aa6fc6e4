"""Steps that cannot be run are refused before the first of their calls is issued (CPU only)."""
import pytest
import torch

from test_chunk_host import lib  # noqa: F401

CALLS = ("tree_mask_build", "tree_verify_attention", "chunk_attention_q8", "tree_logits_process", "logits_sample",
         "tree_accept", "token_counts_update", "kv_compact", "kv_compact_q8")


@pytest.fixture()
def issued(lib, monkeypatch):  # noqa: F811
    import eagle_speculative_decoding_parent_gb300.pipeline as pl
    calls = []
    for x in CALLS:
        monkeypatch.setattr(pl, x, lambda *a, _x=x, **k: calls.append(_x))
    for x in ("tree_verify_attention_workspace", "chunk_attention_q8_workspace", "tree_accept_workspace"):
        monkeypatch.setattr(pl, x, lambda *a: 0)
    return calls


def step(**kw):
    from eagle_speculative_decoding_parent_gb300.pipeline import VerifyStep
    return VerifyStep(B=1, N=2, Hq=2, Hkv=1, d=64, max_blocks=2, bs=16, dtype=torch.bfloat16, max_path=2, V=8,
                      device="cpu", **kw)


def args(**kw):
    t = torch.zeros(1)
    return dict(dict(parents=t, q=torch.zeros((1, 2, 2, 64)), k_cache=t, v_cache=t, block_table=t, prefix_lens=t,
                     draft_tokens=t, target=t), **kw)


def test_refused_before_anything_is_issued(issued):
    q8 = dict(cache_dtype=torch.float8_e4m3fn)
    t = torch.zeros(1)
    scales = dict(k_scale=t, v_scale=t)
    for make, run in ((q8, dict(scales, node_counts=t)), (q8, dict()), (q8, dict(k_scale=t)), (q8, dict(v_scale=t)),
                      (dict(), dict(sampling=dict())), (dict(mode=1, process=True), dict(mode=1, sampling=dict(top_k=t))),
                      (dict(process=True), dict(sampling=dict(min_p=t))),
                      (dict(mode=1, process=True, filters=True), dict(mode=0, sampling=dict(top_p=t)))):
        with pytest.raises(ValueError):
            step(**make).run(**args(**run))
        assert issued == [], (make, run)


def test_steps_that_run(issued):
    t = torch.zeros(1)
    step(cache_dtype=torch.float8_e4m3fn).run(**args(k_scale=t, v_scale=t))
    assert issued == ["tree_mask_build", "chunk_attention_q8", "tree_accept", "kv_compact_q8"]
    issued.clear()
    step(mode=1, process=True, filters=True).run(**args(mode=1, sampling=dict(top_k=t, counts=t), node_counts=t))
    assert issued == ["tree_mask_build", "tree_verify_attention", "tree_logits_process", "logits_sample", "tree_accept",
                      "token_counts_update", "kv_compact"]
