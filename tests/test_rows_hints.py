"""The length that the split choices assume follows the tokens begun, evicted or given (host only)."""
import pytest
import torch

BF = torch.bfloat16


@pytest.fixture()
def hints(monkeypatch):
    from conftest import build_library
    build_library()
    from dynamic_sparse_kv_gb300 import _native
    given = []
    monkeypatch.setattr(_native, "fastocr_set_length_hint", lambda handle, n: given.append(n))
    monkeypatch.setattr(_native, "fastocr_evict", lambda *args, **kw: None)
    return given


def test_the_hint_of_a_decoder_follows_its_tokens(hints):
    from dynamic_sparse_kv_gb300 import DecodeAttention
    dec = object.__new__(DecodeAttention)
    dec.k_cache = dec.v_cache = torch.zeros(1, 4, 2, 16, 64, dtype=BF)
    dec.layers, dec.batch, dec.kv_heads, dec.handle, dec.kv = 1, 3, 2, None, [None]
    dec.hint, dec.weights, dec._tracked = 0, None, []
    dec.seq_len = torch.full((3,), 30, dtype=torch.int32)
    dec.begin_token()                    # nothing known: the capacity stays the assumption
    assert hints == [] and dec.seq_len.tolist() == [31] * 3
    dec.set_seq_len(30)
    dec.track_weights(64, torch.tensor([20, 24, 3]))
    for _ in range(5):
        dec.begin_token()
    assert hints == [30, 31, 32, 33, 34, 35]
    dec.weights["new_len"].fill_(30)
    dec.evict_step(8, 2)                 # at most 24 + 8 rows are left
    assert hints[6:] == [32]
    dec.begin_token()
    dec.evict_step(60, 2)                # no sequence is longer than that
    assert hints[7:] == [33]
    dec.track_weights(64, 0)
    dec.evict_step(1, 0)
    assert hints[8:] == [1]


def test_the_hint_of_cross_attention(hints, monkeypatch):
    """From lengths on the host, or given; none for lengths on the device, which may change."""
    from dynamic_sparse_kv_gb300 import CrossAttention, _native

    class OnDevice(torch.Tensor):        # a host tensor that says it is on the device
        is_cuda = True

    monkeypatch.setattr(_native, "fastocr_create", lambda *args: 0)
    monkeypatch.setattr(_native, "fastocr_rows_workspace", lambda *args: 16)
    k = torch.zeros(1, 4, 2, 16, 64, dtype=BF).as_subclass(OnDevice)
    table = torch.zeros(3, 2, dtype=torch.int32)
    on_device = torch.tensor([5, 0, 9], dtype=torch.int32).as_subclass(OnDevice)
    for state_len, most, want in ((7, None, 7), (0, None, 0), (torch.tensor([5, 0, 9]), None, 9), (on_device, None, 0),
                                  (on_device, 12, 12), (torch.tensor([5, 0, 9]), 30, 30),
                                  (torch.tensor([5, 1 << 40, -1]), None, 32)):
        CrossAttention(k, k, table, state_len, q_heads=4, max_states=most)
        assert hints[-1] == want
