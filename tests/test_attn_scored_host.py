"""Refusals of the scored attention calls, without a GPU."""

import pytest

import megatron_tensor_sharded_b200 as tp

B = [0x100000000 * i for i in range(1, 16)]   # never dereferenced


def test_mask_refusals():
    n = tp.tp_attention_mask_size(300)
    assert n > 0 and tp.tp_attention_mask_size(-1) == 0 and tp.tp_attention_mask_size(2 ** 31) == 0

    def mask(**kw):
        a = dict(doc_offsets=B[0], n_docs=3, prefix=None, causal=True, mask=B[1], mask_bytes=n, T=300,
                 stream=0, check=False)
        a.update(kw)
        return tp.tp_attention_mask(**a)

    for kw, status in ((dict(T=-1), 1), (dict(T=2 ** 31), 4), (dict(n_docs=0), 1), (dict(doc_offsets=None), 1),
                       (dict(prefix=B[2], causal=False), 1), (dict(doc_offsets=B[0] + 2), 3),
                       (dict(prefix=B[2] + 1), 3), (dict(mask=None), 7), (dict(mask_bytes=n - 1), 7),
                       (dict(mask=B[1] + 16), 3), (dict(doc_offsets=B[1] + 64), 1)):
        assert mask(**kw) == status, kw
    assert mask(T=0, doc_offsets=None, mask=None) == 0


LAYOUT = [(dict(p=0), 1), (dict(T=-1), 1), (dict(n_heads=3), 2), (dict(n_kv_heads=3), 2),
          (dict(n_heads=4, n_kv_heads=8), 1), (dict(n_heads=0), 1), (dict(head_dim=64), 4),
          (dict(T=2 ** 31 - 1), 4)]
SCORES = [dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(softcap=-1.0),
          dict(softcap=float("nan"))]


def _scores():
    out = [(dict(score=tp.score_params(**kw)), 1) for kw in SCORES]
    out += [(dict(score=tp.score_params(slopes=B[9] + 2)), 3), (dict(score=tp.score_params(mask=B[9] + 8)), 3),
            (dict(score=tp.score_params(softcap=1e-5)), 4), (dict(score=tp.score_params(softcap=1e7)), 4)]
    return out


@pytest.mark.parametrize("kw,status", LAYOUT + _scores() + [
    (dict(Q=None), 1), (dict(K=None), 1), (dict(V=None), 1), (dict(O=None), 1), (dict(Q=B[0] + 8), 3),
    (dict(O=B[3] + 2), 3), (dict(LSE=B[4] + 2), 3), (dict(O=B[0]), 1), (dict(O=B[2] + 256), 1),
    (dict(LSE=B[3]), 1), (dict(LSE=B[9], score=tp.score_params(slopes=B[9])), 1)])
def test_forward_refusals(kw, status):
    a = dict(Q=B[0], K=B[1], V=B[2], O=B[3], LSE=B[4], T=300, p=2, n_heads=8, n_kv_heads=4, head_dim=128,
             score=None, stream=0, check=False)
    a.update(kw)
    assert tp.tp_attention_scored(**a) == status


@pytest.mark.parametrize("kw,status", LAYOUT + _scores() + [
    (dict(dO=None), 1), (dict(LSE=None), 1), (dict(dQ=None), 1), (dict(dV=B[8] + 8), 3), (dict(dQ=B[0]), 1),
    (dict(dK=B[8]), 1), (dict(workspace=None), 7), (dict(workspace_bytes=8), 7), (dict(workspace=B[10] + 16), 3),
    (dict(workspace=B[5]), 1), (dict(LSE=B[4] + 1), 3)])
def test_backward_refusals(kw, status):
    a = dict(Q=B[0], K=B[1], V=B[2], O=B[3], LSE=B[4], dO=B[5], dQ=B[6], dK=B[7], dV=B[8], workspace=B[10],
             workspace_bytes=tp.tp_attention_scored_backward_workspace_size(300, 2, 8, 4, 128), T=300, p=2,
             n_heads=8, n_kv_heads=4, head_dim=128, score=None, stream=0, check=False)
    a.update(kw)
    assert tp.tp_attention_scored_backward(**a) == status


def test_decode_refusals():
    size = tp.tp_attention_decode_workspace_size(3, 100, 2, 8, 4, 128)
    assert size > 0 and tp.tp_attention_decode_workspace_size(3, 0, 2, 8, 4, 128) == 0

    def call(**kw):
        a = dict(Q=B[0], K_new=B[1], V_new=B[2], K_cache=B[3], V_cache=B[4], lengths=B[5], O=B[6], LSE=B[7],
                 workspace=B[8], workspace_bytes=size, B=3, capacity=100, p=2, n_heads=8, n_kv_heads=4,
                 head_dim=128, score=None, stream=0, check=False)
        a.update(kw)
        return tp.tp_attention_decode(**a)

    for kw, status in [(dict(B=-1), 1), (dict(B=2 ** 31), 4), (dict(p=0), 1), (dict(n_heads=6, n_kv_heads=4), 1),
                       (dict(n_heads=7), 2), (dict(head_dim=96), 4), (dict(capacity=0), 1), (dict(capacity=2 ** 31), 4),
                       (dict(Q=None), 1), (dict(K_new=None), 1), (dict(V_new=None), 1), (dict(K_cache=None), 1),
                       (dict(V_cache=B[4] + 8), 3), (dict(lengths=None), 1), (dict(lengths=B[5] + 1), 3),
                       (dict(LSE=B[7] + 2), 3), (dict(workspace=None), 7), (dict(workspace_bytes=size - 1), 7),
                       (dict(workspace=B[8] + 128), 3), (dict(V_cache=B[3]), 1), (dict(O=B[0]), 1),
                       (dict(K_new=B[3] + 256), 1), (dict(score=tp.score_params(mask=B[9])), 4),
                       (dict(score=tp.score_params(softcap=-1.0)), 1)]:
        assert call(**kw) == status, kw
    assert call(B=0, Q=None, K_cache=None) == 0


def test_nothing_to_do():
    n0 = tp.tp_kernel_launch_count()
    assert tp.tp_attention_scored(None, None, None, None, None, 0, 1, 1, 1, 128, stream=0, check=False) == 0
    assert tp.tp_attention_scored_backward(None, None, None, None, None, None, None, None, None, None, 0, 0, 1, 1, 1,
                                           128, stream=0, check=False) == 0
    assert tp.tp_kernel_launch_count() == n0
    assert tp.tp_attention_scored_backward_workspace_size(0, 1, 1, 1, 128) > 0
    assert tp.tp_attention_scored_backward_workspace_size(10, 1, 1, 1, 64) == 0


@pytest.mark.parametrize("raw,device,agrees", [(lambda d: 70 + d, lambda: 1, True), (lambda d: 5, lambda: 1, False),
                                               (lambda: 71, lambda: 1, False), (None, lambda: 1, False)])
def test_the_short_way_to_the_current_stream_has_to_agree(monkeypatch, raw, device, agrees):
    import torch
    public = type("S", (), {"cuda_stream": 71})
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: public)
    for name, f in (("_cuda_getCurrentRawStream", raw), ("_cuda_getDevice", device)):
        if f is None:
            monkeypatch.delattr(torch._C, name, raising=False)
        else:
            monkeypatch.setattr(torch._C, name, f, raising=False)
    way = tp._find_raw_stream()
    assert way() == 71 and (way.__name__ == "short") == agrees


def test_sizes_past_what_a_block_counts():
    """Shares of steps, places among tiles and scores that would leave 32 bits."""
    huge = tp.score_params(scale=3e38)
    a = dict(Q=B[0], K=B[1], V=B[2], O=B[3], LSE=B[4], T=300, p=1, n_heads=1, n_kv_heads=1, head_dim=128, score=huge,
             stream=0, check=False)
    assert tp.tp_attention_scored(**a) == 4
    b = dict(a, dO=B[5], dQ=B[6], dK=B[7], dV=B[8], workspace=B[10], workspace_bytes=1 << 40)
    assert tp.tp_attention_scored_backward(**b) == 4
    # the steps of dK and dV: T^2 / 2^14 a head, shared by 148
    size = tp.tp_attention_scored_backward_workspace_size
    assert tp.tp_attention_scored_backward(**dict(b, T=2 ** 27, score=None)) == 4
    assert tp.tp_attention_scored_backward(**dict(b, T=2 ** 30, score=tp.score_params(causal=True))) == 4
    assert size(2 ** 26, 1, 1, 1, 128) > 0 and size(2 ** 30, 1, 1, 1, 128) == 0
    # a sequence's tiles of all its heads
    size = tp.tp_attention_decode_workspace_size
    assert size(1, 2 ** 30, 1, 64, 64, 128) > 0 and size(1, 2 ** 30, 1, 1024, 1024, 128) == 0
    assert size(1, 2 ** 30, 1, 1024, 64, 128) > 0
    c = dict(Q=B[0], K_new=None, V_new=None, K_cache=B[1], V_cache=B[1] << 13, lengths=B[2], O=B[3], LSE=None,
             workspace=B[4], workspace_bytes=1 << 30, B=1, capacity=2 ** 30, p=1, n_heads=1024, n_kv_heads=1024,
             head_dim=128, stream=0, check=False)
    assert tp.tp_attention_decode(**c) == 4
    assert tp.tp_attention_decode(**dict(c, capacity=64, n_heads=1, n_kv_heads=1, score=huge)) == 4
