"""Arguments of the cache's rows, 4-bit caches, rotary tables and pools that the library would
read or write wrongly are refused before any call of it. The library itself is replaced, so
no GPU is needed."""
import ctypes

import pytest
import torch

BF = torch.bfloat16
CALLS = ("write_rows", "read_rows", "pool_reserve", "pool_fork", "pool_release", "pool_trim", "pool_compact",
         "pool_copy")


@pytest.fixture()
def calls(monkeypatch):
    """Names and arguments of the library calls made."""
    from conftest import build_library
    build_library()
    from dynamic_sparse_kv_gb300 import _native
    made = []
    for name in CALLS:
        monkeypatch.setattr(_native, "fastocr_" + name, lambda *args, name=name, **kw: made.append((name, args)))
    monkeypatch.setattr(_native, "fastocr_pool_workspace", lambda *args: 64)
    return made


def decoder(cache=None):
    from dynamic_sparse_kv_gb300 import DecodeAttention
    dec = object.__new__(DecodeAttention)
    dec.k_cache = dec.v_cache = torch.zeros(2, 6, 2, 16, 64, dtype=BF) if cache is None else cache
    dec.layers, dec.num_pages, dec.batch, dec.q_heads, dec.kv_heads, dec.head_dim = 2, 6, 3, 4, 2, 64
    dec.kv, dec.handle = [None, None], None
    dec.block_table = torch.zeros(3, 4, dtype=torch.int32)
    dec.seq_len = torch.zeros(3, dtype=torch.int32)
    return dec


def spread(t):
    """The same values at other strides."""
    return torch.stack([t, t + 1], dim=-1)[..., 0]


def test_write_refuses_what_it_would_read_wrongly(calls):
    from dynamic_sparse_kv_gb300 import Rotary
    dec = decoder()
    q, k = torch.zeros(3, 4, 64, dtype=BF), torch.zeros(3, 2, 64, dtype=BF)
    pos, start = torch.zeros(2, 5, dtype=torch.int32), torch.tensor([0, 2, 2, 5], dtype=torch.int32)
    rot = Rotary(64, (16, 16), positions=10)
    dec.write_layer(0, k, k)
    dec.write_layer(1, k, k, q=q, out_q=q)
    q5, k5 = torch.zeros(5, 4, 64, dtype=BF), torch.zeros(5, 2, 64, dtype=BF)
    dec.write_layer(1, k5, k5, q=q5, out_q=torch.empty_like(q5), rotary=rot, pos=pos, q_start=start)
    dec.write_layer(1, k5[:0], k5[:0], q_start=start)       # nothing to do
    wide = torch.zeros(5, 4 * 64 + 2 * 2 * 64 + 8, dtype=BF)   # a projection's output
    parts = wide[:, :256].view(5, 4, 64), wide[:, 256:384].view(5, 2, 64), wide[:, 384:512].view(5, 2, 64)
    dec.write_layer(0, parts[1], parts[2], q=parts[0], out_q=torch.empty_like(q5), q_start=start)
    assert [n for n, _ in calls] == ["write_rows"] * 4
    t = calls[3][1][2]
    assert (t.q_stride, t.k_stride, t.tokens) == (520, 520, 5)
    del calls[:]
    for bad in (spread(k), k.float(), k[:, :1], k.to("meta"), k.transpose(0, 1), k[:1].expand(3, 2, 64), k[:2],
                torch.zeros(3, 2, 68, dtype=BF)[..., :64], torch.zeros(3, 132, dtype=BF)[:, :128].view(3, 2, 64),
                k.view(3, 128)):
        with pytest.raises(ValueError):
            dec.write_layer(0, bad, k)
        with pytest.raises(ValueError):
            dec.write_layer(0, k, bad)
    for bad in (q[:, :3], q.float(), q[:2], spread(q), q.to("meta")):
        with pytest.raises(ValueError):
            dec.write_layer(0, k, k, q=bad, out_q=q)
        with pytest.raises(ValueError):
            dec.write_layer(0, k, k, q=q, out_q=bad)
    for kw in (dict(q=q), dict(out_q=q), dict(rotary=rot), dict(rotary=rot, pos=pos), dict(rotary=rot, pos=pos[:1, :3]),
               dict(rotary=rot, pos=torch.zeros(2, 3)), dict(rotary=rot, pos=spread(pos[:, :3])),
               dict(rotary=Rotary(128, (64,), positions=4), pos=pos[:1, :3].contiguous()),
               dict(q_start=start[:3]), dict(q_start=start.long()), dict(q_start=start.to("meta"))):
        with pytest.raises(ValueError):
            dec.write_layer(0, k, k, **kw)
    with pytest.raises(ValueError, match="q_start"):
        dec.write_layer(0, k5, k5)
    assert not calls


def test_read_refuses_what_it_would_write_wrongly(calls):
    dec = decoder()
    start = torch.tensor([0, 2, 2, 5], dtype=torch.int32)
    out = torch.zeros(5, 2, 64)
    dec.read_layer(0, start, out, out.clone())
    dec.read_layer(0, start, out.to(BF), out.to(BF))
    dec.read_layer(0, start, out[:0], out[:0])
    assert [n for n, _ in calls] == ["read_rows"] * 2
    for a, b in ((out.half(), out.half()), (out, out.to(BF)), (out, out[:4]), (spread(out), out), (out, spread(out)),
                 (out[:, :1], out[:, :1]), (out.to("meta"), out), (out.view(5, 128), out)):
        with pytest.raises(ValueError):
            dec.read_layer(0, start, a, b)
    for bad in (start.long(), start[:3], start.to("meta"), spread(start)):
        with pytest.raises(ValueError, match="row_start"):
            dec.read_layer(0, bad, out, out)
    assert len(calls) == 2


def test_4_bit_caches_are_checked():
    from dynamic_sparse_kv_gb300 import DecodeAttention, Fp4Cache
    from dynamic_sparse_kv_gb300 import _native as N
    c = Fp4Cache(2, 6, 2, 16, 64)
    assert N.check_caches(c, Fp4Cache(2, 6, 2, 16, 64, gain=torch.full((2, 2), 0.5))) == N.FASTOCR_DTYPE_FP4
    assert c[1][0].shape == (6, 2, 16, 32) and c[1][1].shape == (6, 2, 16, 4) and c[1][2].shape == (2,)
    k = torch.zeros(2, 6, 2, 16, 64, dtype=BF)
    table = torch.zeros(3, 2, dtype=torch.int32)
    for a, b in ((c, k), (k, c), (c, Fp4Cache(2, 5, 2, 16, 64))):
        with pytest.raises(ValueError):
            N.check_caches(a, b)
    for name, t in (("codes", c.codes.int()), ("codes", c.codes[:, :5]), ("scales", c.scales.float()),
                    ("scales", c.scales.transpose(0, 1)), ("gain", c.gain[:1]), ("gain", c.gain.double())):
        d = Fp4Cache(2, 6, 2, 16, 64)
        setattr(d, name, t)
        with pytest.raises(ValueError, match=name):
            N.check_caches(c, d)
    for gain in (0.0, -1.0, float("inf"), float("nan"), torch.zeros(2, 2), torch.ones(2), torch.ones(2, 3)):
        with pytest.raises(ValueError, match="gain"):
            Fp4Cache(2, 6, 2, 16, 64, gain=gain)
    with pytest.raises(ValueError):
        Fp4Cache(2, 6, 2, 16, 72)
    with pytest.raises(AssertionError):      # only for want of a GPU
        DecodeAttention(c, c, table, q_heads=4)


def test_rotary_refuses_what_has_no_meaning(calls):
    from dynamic_sparse_kv_gb300 import Rotary
    for kw in (dict(axes=(16,)), dict(axes=(33,)), dict(axes=()), dict(axes=(32, 0)), dict(axes=(8, 8, 8, 4, 4)),
               dict(axes=(32,), positions=0), dict(axes=(32,), base=0.0), dict(axes=(8,), rotary_dim=16),
               dict(axes=(24,), rotary_dim=48), dict(axes=(48,), rotary_dim=96)):
        with pytest.raises(ValueError):
            Rotary(64, **{"positions": 4, **kw})


def test_pools_refuse_what_they_would_read_wrongly(calls):
    from dynamic_sparse_kv_gb300 import PagePool
    dec = decoder()
    good = torch.zeros(3, dtype=torch.int32), torch.zeros(6, dtype=torch.int32)
    for held, refs in ((good[0], None), (None, good[1]), (good[0].long(), good[1]), (good[0], good[1][:5]),
                       (good[0][:2], good[1]), (spread(good[0]), good[1]), (good[0].to("meta"), good[1])):
        with pytest.raises(ValueError):
            PagePool(dec, held=held, refs=refs)
    dec.seq_len.fill_(7)
    pool = PagePool(dec)
    assert bool((dec.block_table == -1).all()) and bool((dec.seq_len == 0).all())
    assert pool.c.k_layer == 6 * 2 * 16 * 64 * 2 and not pool.c.k_scale
    pool.reserve(5)
    pool.reserve(torch.tensor([1, 2, 3]))
    pool.reserve(extra=0)
    for args, kw in (((), {}), ((5,), dict(extra=1)), ((), dict(extra=-1)), ((), dict(extra=2**31)), ((torch.zeros(2),), {})):
        with pytest.raises(ValueError):
            pool.reserve(*args, **kw)
    pool.fork([0], [1])
    pool.fork([], [])
    pool.fork([0, 0], torch.tensor([1, 2], dtype=torch.int32))
    for src, dst in (([0, 0], [1, 1]), ([0, 1], [1, 2]), ([0], [3]), ([-1], [0]), ([0, 1], [2]), ([0.5], [1]),
                     ([[0]], [[1]]), ([0], torch.zeros(1, dtype=torch.int64, device="meta"))):
        with pytest.raises((ValueError, NotImplementedError)):
            pool.fork(src, dst)
    pool.release([2, 0, 2])
    pool.release([])
    for seqs in ([3], [-1], [True], torch.zeros(4, dtype=torch.int32), [0, 1, 2, 0]):
        with pytest.raises(ValueError):
            pool.release(seqs)
    pool.copy_pages([0, 0], [1, 5])
    for src, dst in (([0], [0]), ([0, 1], [2, 2]), ([6], [0])):
        with pytest.raises(ValueError):
            pool.copy_pages(src, dst)
    pool.trim()
    pool.compact()
    assert [n for n, _ in calls] == (["pool_reserve"] * 3 + ["pool_fork"] * 2 + ["pool_release", "pool_copy",
                                                                                "pool_trim", "pool_compact"])


def test_the_library_refuses_before_it_launches():
    """Host checks of the C entry points, with a handle that is not one: none gets as far as a device."""
    from conftest import build_library
    build_library()
    from dynamic_sparse_kv_gb300 import _native as N
    L = N.lib
    kv, tok, pool = N.fastocr_kv(), N.fastocr_tokens(), N.fastocr_pool()
    R = ctypes.byref
    assert L.fastocr_write_rows(None, R(kv), R(tok), None, None) == N.FASTOCR_ERR_NULL
    assert L.fastocr_read_rows(None, R(kv), None, 0, None, None, 0, None) == N.FASTOCR_ERR_NULL
    assert L.fastocr_pool_workspace(None, 5) == N.FASTOCR_ERR_NULL
    for call in (lambda: L.fastocr_pool_reserve(None, R(pool), None, 0, None, None),
                 lambda: L.fastocr_pool_fork(None, R(pool), None, None, 0, None),
                 lambda: L.fastocr_pool_release(None, R(pool), None, 0, None),
                 lambda: L.fastocr_pool_trim(None, R(pool), None),
                 lambda: L.fastocr_pool_compact(None, R(pool), None, None),
                 lambda: L.fastocr_pool_copy(None, R(pool), None, None, 0, None)):
        assert call() == N.FASTOCR_ERR_NULL
    # a noalloc call has no 4 bits
    dims = N.fastocr_dims(1, 4, 2, 64, N.FASTOCR_DTYPE_FP4, 16, 8, 64, 2)
    one = ctypes.c_void_p(256)
    kv = N.fastocr_kv(256, 256, 256, 256, 4)
    assert L.fastocr_focal_attend_noalloc(R(dims), one, R(kv), one, 0.5, one, one, 64, one, one,
                                          None) == N.FASTOCR_ERR_INVALID
