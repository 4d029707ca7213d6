"""Tensors that the library would read or write wrongly are refused before any call of it:
wrong shape, type, strides or device. The library itself is replaced, so no GPU is needed."""
import pytest
import torch

BF = torch.bfloat16


@pytest.fixture()
def calls(monkeypatch):
    """Names of the library calls made."""
    from conftest import build_library
    build_library()
    from dynamic_sparse_kv_gb300 import _native
    made = []
    for name in ("cross_attend", "shared_attend", "weigh_attend", "evict"):
        monkeypatch.setattr(_native, "fastocr_" + name, lambda *args, name=name, **kw: made.append(name))
    return made


def spread(t):
    """The same values at other strides."""
    return torch.stack([t, t + 1], dim=-1)[..., 0]


def cross():
    from dynamic_sparse_kv_gb300 import CrossAttention
    ca = object.__new__(CrossAttention)
    ca.k_cache = ca.v_cache = torch.zeros(1, 4, 2, 16, 64, dtype=BF)
    ca.batch, ca.q_heads, ca.head_dim, ca.kv = 3, 4, 64, [None]
    ca.handle, ca.ws = None, torch.zeros(1, dtype=torch.uint8)
    return ca


def test_cross_attention_refuses_what_it_would_read_wrongly(calls):
    ca = cross()
    q = torch.zeros(5, 4, 64, dtype=BF)
    start = torch.tensor([0, 2, 2, 5], dtype=torch.int32)
    ca.attend(0, q, start, torch.empty_like(q))
    assert calls == ["cross_attend"]
    for bad in (spread(start), torch.zeros(1, dtype=torch.int32).expand(4), start.long(), start[:3],
                start.view(2, 2), start.to("meta")):
        with pytest.raises(ValueError, match="q_start"):
            ca.attend(0, q, bad, torch.empty_like(q))
    for bad in (spread(q), q.float(), q[:, :3], q.to("meta"), q[:, :1].expand(5, 4, 64), q.transpose(0, 1)):
        with pytest.raises(ValueError, match="q must"):
            ca.attend(0, bad, start, torch.empty(bad.shape, dtype=BF))
    for bad in (spread(q), q.float(), q[:4], q.to("meta"), q[:1].expand(5, 4, 64)):
        with pytest.raises(ValueError, match="out must"):
            ca.attend(0, q, start, bad)
    assert calls == ["cross_attend"]


def decoder():
    from dynamic_sparse_kv_gb300 import DecodeAttention
    dec = object.__new__(DecodeAttention)
    dec.k_cache = dec.v_cache = torch.zeros(1, 4, 2, 16, 64, dtype=BF)
    dec.layers, dec.batch, dec.q_heads, dec.head_dim, dec.kv = 1, 3, 4, 64, [None]
    dec.handle = None
    dec.groups = {"c": None, "ws": torch.zeros(1, dtype=torch.uint8)}
    dec.weights = {"c": [None]}
    return dec


def test_evict_refuses_lengths_it_would_write_wrongly(calls):
    dec = decoder()
    good = torch.zeros(3, dtype=torch.int32)
    dec.evict_layer(0, 2, 1)
    dec.evict_layer(0, 2, 1, good)
    assert calls == ["evict"] * 2
    for bad in (good.long(), good[:2], spread(good), good[:1].expand(3), good.to("meta"), good.view(3, 1)):
        with pytest.raises(ValueError, match="new_len"):
            dec.evict_layer(0, 2, 1, bad)
    assert calls == ["evict"] * 2


@pytest.mark.parametrize("kind", ["shared", "weigh"])
def test_shared_and_weighed_layers_refuse_what_they_would_read_wrongly(calls, kind):
    dec = decoder()
    layer = dec.shared_layer if kind == "shared" else dec.weigh_layer
    step = dec.shared_step if kind == "shared" else dec.weighed_step
    good = torch.zeros(3, 4, 64, dtype=BF)
    layer(0, good, torch.empty_like(good))
    step(good[None], torch.empty_like(good)[None])
    assert calls == [kind + "_attend"] * 2
    of_all = torch.zeros(3, 2, 4, 64, dtype=BF)          # [B, L, H_q, d]: a layer of it is strided
    for bad in (of_all[:, 0], good.float(), good[:2], good[:, :3], good.to("meta"), good.view(3, 256),
                good[:1].expand(3, 4, 64), good.transpose(0, 1)):
        with pytest.raises(ValueError, match="q must"):
            layer(0, bad, good)
        with pytest.raises(ValueError, match="out must"):
            layer(0, good, bad)
    with pytest.raises(ValueError):
        step(of_all.transpose(0, 1), torch.empty(2, 3, 4, 64, dtype=BF))
    assert calls == [kind + "_attend"] * 2


def test_cross_attention_refuses_lengths_of_another_batch(calls):
    from dynamic_sparse_kv_gb300 import CrossAttention
    k = torch.zeros(1, 4, 2, 16, 64, dtype=BF)
    table = torch.zeros(3, 2, dtype=torch.int32)
    for lengths in (torch.zeros(2), torch.zeros(1), torch.zeros(4), torch.zeros(3, 1), torch.tensor(5)):
        with pytest.raises(ValueError, match="state_len"):       # fewer were read past their end
            CrossAttention(k, k, table, lengths, q_heads=4)
    with pytest.raises(ValueError, match="block_table"):
        CrossAttention(k, k, table[0], torch.zeros(2), q_heads=4)


def test_caches_of_other_types_and_strides_are_refused(calls):
    from dynamic_sparse_kv_gb300 import CrossAttention, DecodeAttention
    k = torch.zeros(2, 4, 2, 16, 64, dtype=BF)
    table = torch.zeros(3, 2, dtype=torch.int32)
    half = k.half()                              # was read as fp32, past its end
    for kk, vv in ((half, half), (k, k.float()), (k.float(), k), (k, k[:, :3]), (k[0], k[0]),
                   (k.transpose(1, 2), k.transpose(1, 2)), (k, spread(k)),
                   (k[:, :1].expand(2, 4, 2, 16, 64), k), (k, k.to("meta"))):
        with pytest.raises(ValueError):
            CrossAttention(kk, vv, table, 5, q_heads=4)
        with pytest.raises(ValueError):
            DecodeAttention(kk, vv, table, q_heads=4)
    for good in (k, k.float(), torch.zeros(2, 6, 2, 16, 64, dtype=BF)[:, :4]):
        with pytest.raises(AssertionError):      # only for want of a GPU
            CrossAttention(good, good, table, 5, q_heads=4)
        with pytest.raises(AssertionError):
            DecodeAttention(good, good, table, q_heads=4)


def test_a_refused_checkpoint_changes_nothing(calls):
    dec = decoder()
    dec.stride, dec.tau, dec.max_img, dec.has_f_last = 4, 1.0, 8, False
    dec.focal, dec.sel = (0,), {0: (torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32))}
    st = {"batch": 3, "layers": 1, "stride": 4, "tau": 1.0, "max_img": 8, "focal": (0,), "has_f_last": True,
          "sel": {0: (torch.ones(3, 4, dtype=torch.int32), torch.ones(3, dtype=torch.int32))}, "warm": None,
          "weights": {"mass": torch.ones(1, 3, 2, 5), "pos": torch.ones(1, 3, 2, 5, dtype=torch.int32)}}
    small = {"mass": torch.zeros(1, 3, 2, 5), "pos": torch.zeros(1, 3, 2, 4, dtype=torch.int32)}
    for have in (None, small):
        dec.weights = have
        for focal in ((0,), ()):
            with pytest.raises(ValueError, match="track_weights"):
                dec.load_state_dict({**st, "focal": focal, "sel": st["sel"] if focal else {}})
            assert dec.focal == (0,) and not dec.sel[0][0].any() and not dec.has_f_last
    assert not small["mass"].any()
