"""The pages of a pool against lists."""
import random

import pytest
import torch

from cache_harness import Pool

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


class Both:
    """A PagePool and the list model; page x's rows begin as x in every layer."""

    def __init__(self, batch, pages, page=16, cols=8, kind="bf16", layers=2, hkv=2, d=64):
        from dynamic_sparse_kv_gb300 import DecodeAttention, Fp4Cache, PagePool
        shape = (layers, pages, hkv, page, d)
        if kind == "fp4":
            self.caches = [Fp4Cache(*shape, device="cuda") for _ in range(2)]
            self.arrays = [t for c in self.caches for t in (c.codes, c.scales.view(torch.uint8))]
        else:
            self.caches = [torch.zeros(shape, dtype=BF if kind == "bf16" else F32, device="cuda") for _ in range(2)]
            self.arrays = self.caches
        mark = torch.arange(pages, device="cuda") % 250
        for i, a in enumerate(self.arrays):
            for l in range(layers):
                a[l] = (mark + i + 3 * l).to(a.dtype).view(-1, 1, 1, 1)
        table = torch.full((batch, cols), 5, dtype=torch.int32, device="cuda")
        self.dec = DecodeAttention(*self.caches, table, q_heads=hkv)
        self.dec.seq_len.fill_(99)
        self.pool = PagePool(self.dec)
        self.m = Pool(batch, pages, page, cols)
        self.layers, self.cols = layers, cols

    def set_len(self, n):
        self.m.len = list(n)
        self.dec.seq_len.copy_(torch.tensor(n, dtype=torch.int32))

    def check(self, status=0):
        m, dec, pool = self.m, self.dec, self.pool
        assert dec.block_table.tolist() == [r + [-1] * (self.cols - len(r)) for r in m.rows]
        assert pool.held.tolist() == [len(r) for r in m.rows]
        assert pool.refs.tolist() == m.refs()
        assert dec.seq_len.tolist() == m.len
        for i, a in enumerate(self.arrays):
            for l in range(self.layers):
                want = (torch.tensor(m.data) % 250 + i + 3 * l).to(a.dtype).view(-1, 1, 1, 1)
                got = a[l].cpu()
                # pages that nobody holds may keep what compact moved away
                for x, r in enumerate(m.refs()):
                    if r:
                        assert bool((got[x] == want[x]).all()), (i, l, x)
        assert dec.device_status() == status


@pytest.mark.parametrize("kind,page,hkv,d", [("bf16", 16, 2, 64), ("f32", 4, 1, 128), ("fp4", 16, 4, 128),
                                             ("fp4", 1, 1, 64), ("bf16", 64, 10, 128)])
def test_random_histories(kind, page, hkv, d):
    rng = random.Random(page)
    t = Both(6, 90, page, 10, kind, 2, hkv, d)
    for step in range(40):
        op = rng.choice(["grow", "grow", "grow", "fork", "release", "trim", "compact", "rows"])
        m = t.m
        if op == "grow":
            extra = rng.choice([1, 1, page, 2 * page + 1])
            extra = max(0, min(extra, min(10 * page - n for n in m.len)))
            short = m.reserve([n + extra for n in m.len])
            t.pool.reserve(extra=extra)
            assert int(t.pool.missing[0]) == short
            if short == 0:
                t.set_len([n + extra for n in m.len])
            t.dec.device_status()
        elif op == "rows":
            rows = [rng.randint(0, 10 * page) for _ in m.len]
            short = m.reserve(rows)
            t.pool.reserve(torch.tensor(rows))
            assert int(t.pool.missing[0]) == short
            t.dec.device_status()
        elif op == "fork":
            ids = rng.sample(range(6), rng.randint(2, 6))
            cut = rng.randint(1, len(ids) - 1)
            dst = ids[cut:]
            src = [rng.choice(ids[:cut]) for _ in dst]
            m.fork(src, dst)
            t.pool.fork(src, torch.tensor(dst, dtype=torch.int32, device="cuda"))
        elif op == "release":
            seqs = rng.sample(range(6), rng.randint(1, 2))
            m.release(seqs)
            t.pool.release(seqs + seqs[:1])
        elif op == "trim":
            t.set_len([rng.randint(max(0, n - 2 * page), n) for n in m.len])
            m.trim()
            t.pool.trim()
        else:
            used = m.compact()
            t.pool.compact()
            assert int(t.pool.used[0]) == used
        t.check()


def test_a_set_back_sequence_gets_pages_of_its_own():
    t = Both(3, 40)
    t.pool.reserve(100)
    assert t.m.reserve([100] * 3) == 0
    t.set_len([100] * 3)
    t.m.fork([0], [1])
    t.pool.fork([0], [1])
    t.set_len([40, 100, 100])       # sequence 0 goes back into pages that 1 reads
    t.pool.reserve([70, 100, 100])
    assert t.m.reserve([70, 100, 100]) == 0
    t.check()


def test_too_few_pages_change_nothing():
    from dynamic_sparse_kv_gb300 import _native as N
    t = Both(4, 10)
    t.pool.reserve([40, 16, 0, 1])
    assert t.m.reserve([40, 16, 0, 1]) == 0
    t.set_len([40, 16, 0, 1])
    t.check()
    t.pool.reserve([48, 64, 32, 1])
    assert t.m.reserve([48, 64, 32, 1]) == 0 and int(t.pool.missing[0]) == 0
    t.check()
    t.pool.reserve([48, 64, 48, 100])
    assert t.m.reserve([48, 64, 48, 100]) == 7 and int(t.pool.missing[0]) == 7
    t.check(N.DEV_NO_PAGES)


@pytest.mark.parametrize("page,pages,batch", [(1, 70000, 3), (16, 20000, 2000), (256, 3, 1)])
def test_many_pages_and_sequences(page, pages, batch):
    rng = random.Random(pages)
    cols = min(30000, 2 * pages // batch)
    t = Both(batch, pages, page, cols, layers=1, hkv=1)
    rows = [rng.randint(0, cols * page // 2) for _ in range(batch)]
    if batch == 1:
        rows = [page * 2 - 1]
    t.pool.reserve(torch.tensor(rows))
    assert t.m.reserve(rows) == 0
    t.set_len(rows)
    t.check()
    gone = rng.sample(range(batch), batch // 2)
    t.pool.release(torch.tensor(gone, dtype=torch.int32, device="cuda"))
    t.m.release(gone)
    t.pool.compact()
    assert int(t.pool.used[0]) == t.m.compact()
    t.pool.reserve(extra=1)
    assert t.m.reserve([n + 1 for n in t.m.len]) == 0
    t.check()


def test_bad_pairs_are_left_out_and_reported():
    from dynamic_sparse_kv_gb300 import _native as N
    t = Both(6, 40)
    rows = [20, 33, 0, 5, 64, 1]
    t.pool.reserve(rows)
    t.m.reserve(rows)
    t.set_len(rows)
    dev = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    t.pool.fork(dev(0, 0, 9, 3), dev(2, 2, 4, -1))      # 2 twice, 9 and -1 are nobody
    t.m.fork([0], [2])
    t.check(N.DEV_BAD_GROUP)
    t.pool.fork(dev(0, 3, 5), dev(3, 4, 5))             # 3 is both; 5 is its own
    t.check(N.DEV_BAD_GROUP)
    t.pool.release(dev(4, 77, 4))
    t.m.release([4])
    t.check(N.DEV_BAD_GROUP)


def test_state_that_does_not_fit_faults_nothing():
    from dynamic_sparse_kv_gb300 import _native as N
    t = Both(3, 20)
    t.pool.reserve([40, 40, 40])
    t.dec.block_table[0, 1] = 10 ** 6
    t.pool.held[1] = -7
    t.pool.refs[t.dec.block_table[2, 0].item()] = 0
    t.dec.seq_len.copy_(torch.tensor([-3, 10 ** 7, 40], dtype=torch.int32))
    t.pool.reserve(extra=1)
    t.pool.compact()
    t.pool.fork([0], [1])
    t.pool.trim()
    t.pool.release([0, 1, 2])
    torch.cuda.synchronize()
    assert t.dec.device_status() & (N.DEV_BAD_PAGE | N.DEV_BAD_POOL | N.DEV_BAD_SEQLEN)


@pytest.mark.parametrize("kind", ["bf16", "fp4"])
def test_copy_pages(kind):
    from dynamic_sparse_kv_gb300 import _native as N
    t = Both(2, 12, kind=kind)
    before = [a.clone() for a in t.arrays]
    t.pool.copy_pages([3, 3, 0], [7, 1, 11])
    for a, b in zip(t.arrays, before):
        b[:, [7, 1, 11]] = b[:, [3, 3, 0]]
        assert torch.equal(a, b)
    dev = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    t.pool.copy_pages(dev(0, 50, 2), dev(12, 2, 4))     # two of the pairs are nowhere
    for a, b in zip(t.arrays, before):
        b[:, 4] = b[:, 2]
        assert torch.equal(a, b)
    assert t.dec.device_status() == N.DEV_BAD_PAGE


def test_captured_and_replayed():
    t = Both(4, 60)
    t.pool.reserve([30, 16, 47, 1])
    t.m.reserve([30, 16, 47, 1])
    t.set_len([30, 16, 47, 1])
    t.m.fork([0], [3])
    t.pool.fork([0], [3])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.pool.reserve(extra=1)
        t.dec.begin_token()
    for _ in range(40):
        graph.replay()
        assert t.m.reserve([n + 1 for n in t.m.len]) == 0
        t.m.len = [n + 1 for n in t.m.len]
    t.check()


def test_pages_freed_by_an_eviction():
    from dynamic_sparse_kv_gb300 import DecodeAttention, PagePool
    g = torch.Generator().manual_seed(9)
    k, v = (torch.randn(1, 40, 2, 16, 64, generator=g).to(BF).cuda() for _ in range(2))
    dec = DecodeAttention(k, v, torch.zeros(3, 10, dtype=torch.int32, device="cuda"), q_heads=4)
    pool = PagePool(dec)
    rows = [150, 70, 33]
    pool.reserve(rows)
    dec.seq_len.copy_(torch.tensor(rows, dtype=torch.int32))
    dec.track_weights(160, 10)
    q = torch.randn(1, 3, 4, 64, generator=g).to(BF).cuda()
    dec.weighed_step(q, torch.empty_like(q))
    dec.evict_step(40, recent=8)
    pool.trim()
    assert dec.seq_len.tolist() == [50, 50, 33] and pool.held.tolist() == [4, 4, 3]
    table = dec.block_table.cpu()
    assert int((table >= 0).sum()) == 11 and int(pool.refs.sum()) == 11 and int(pool.refs.max()) == 1
    pool.reserve(extra=40)
    assert pool.held.tolist() == [6, 6, 5] and dec.device_status() == 0


@pytest.mark.parametrize("raw", [False, True])
def test_lists_and_numbers_on_another_stream(raw):
    """What a call makes of its arguments is made on the stream that it runs on."""
    t = Both(4, 60)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    given = s.cuda_stream if raw else s
    busy = torch.zeros(64 << 20, device="cuda")
    for rows in (40, 90, 100):
        for _ in range(20):
            busy.add_(1)                       # the current stream is late
        t.pool.reserve(rows, stream=given)
        t.pool.reserve(torch.tensor([rows, 0, rows, 1]), stream=given)
        t.m.reserve([rows] * 4)
    t.pool.release([1], stream=given)
    t.m.release([1])
    with torch.cuda.stream(s):
        t.set_len([100, 0, 77, 100])
    t.pool.fork([2], [1], stream=given)
    t.m.fork([2], [1])
    t.pool.trim(stream=given)
    t.m.trim()
    t.pool.compact(stream=given)
    t.m.compact()
    s.synchronize()
    t.check()
