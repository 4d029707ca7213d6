"""Tokens written to a paged cache with rotary positions, and rows read back, bit for bit
against float32 arithmetic in NumPy."""
import numpy as np
import pytest
import torch

from cache_harness import quantise, rotate, table, values

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


class Case:
    def __init__(self, kind, heads, page, tokens, rows, seed, layers=1, spare=2):
        from dynamic_sparse_kv_gb300 import DecodeAttention, Fp4Cache
        self.hq, self.hkv, self.d = heads
        self.kind, self.page, self.tokens, self.rows = kind, page, tokens, rows
        g = torch.Generator().manual_seed(seed)
        cols = max(1, -(-max(rows) // page))
        self.pages = len(rows) * cols + spare
        self.table = torch.randperm(self.pages, generator=g)[:len(rows) * cols].to(torch.int32).view(len(rows), cols)
        self.dt = F32 if kind == "f32" else BF
        shape = (layers, self.pages, self.hkv, page, self.d)
        self.gain = [(0.05 + torch.rand(layers, self.hkv, generator=g)) for _ in range(2)]
        if kind == "fp4":
            self.caches = [Fp4Cache(*shape, gain=x, device="cuda") for x in self.gain]
            for c in self.caches:
                c.codes.fill_(0x5a)
                c.scales.view(torch.uint8).fill_(0x33)
        else:
            self.caches = [torch.full(shape, 7.0, dtype=self.dt, device="cuda") for _ in range(2)]
        self.dec = DecodeAttention(*self.caches, self.table.cuda(), q_heads=self.hq)
        self.dec.set_seq_len(torch.tensor(rows, dtype=torch.int32, device="cuda"))
        t = sum(tokens)
        self.t = t
        # one projection's output, an odd multiple of 16 bytes from token to token
        wide = (self.hq + 2 * self.hkv) * self.d + 24
        self.qkv = torch.randn(max(t, 1), wide, generator=g)
        self.qkv *= torch.exp(torch.randn(wide, generator=g))
        self.qkv = self.qkv.to(self.dt).cuda()[:t]
        a, b = self.hq * self.d, (self.hq + self.hkv) * self.d
        self.q = self.qkv[:, :a].unflatten(1, (self.hq, self.d))
        self.k = self.qkv[:, a:b].unflatten(1, (self.hkv, self.d))
        self.v = self.qkv[:, b:b + self.hkv * self.d].unflatten(1, (self.hkv, self.d))
        self.start = torch.tensor(np.concatenate([[0], np.cumsum(tokens)]), dtype=torch.int32, device="cuda")
        self.g = g

    def positions(self, axes, top):
        return torch.randint(0, top, (axes, self.t), generator=self.g).to(torch.int32)

    def places(self):
        """(token, page, slot) of every token."""
        i = 0
        for b, (t, n) in enumerate(zip(self.tokens, self.rows)):
            for r in range(n - t, n):
                yield i, int(self.table[b, max(r, 0) // self.page]), r % self.page
                i += 1

    def check(self, before, k, v, skip=()):
        """The caches hold k, v [T, H_kv, d] float32 in the tokens' rows and elsewhere what was there."""
        for w, x in enumerate((k, v)):
            cache = self.caches[w]
            if self.kind == "fp4":
                want = [t.copy() for t in before[w]]
                for i, page, slot in self.places():
                    if i in skip:
                        continue
                    for h in range(self.hkv):
                        c, s = quantise(x[i, h], float(self.gain[w][0, h]))
                        want[0][0, page, h, slot], want[1][0, page, h, slot] = c, s
                assert np.array_equal(self.raw(w)[1], want[1])
                a, b = (self.values(z, want[1]) for z in (self.raw(w)[0], want[0]))
                assert np.array_equal(a, b, equal_nan=True)     # -0 is 0
            else:
                want = before[w].clone()
                x = torch.from_numpy(x).to(self.dt)
                for i, page, slot in self.places():
                    if i not in skip:
                        want[0, page, :, slot] = x[i]
                assert torch.equal(cache.cpu(), want)

    def raw(self, w):
        c = self.caches[w]
        return c.codes.cpu().numpy(), c.scales.view(torch.uint8).cpu().numpy()

    @staticmethod
    def values(codes, scales):
        return values(codes, scales, 1.0)

    def before(self):
        return [self.raw(w) if self.kind == "fp4" else self.caches[w].cpu() for w in range(2)]


def f32(t):
    return t.float().cpu().numpy()


KINDS = ["bf16", "f32", "fp4"]
HEADS = [(28, 4, 128), (10, 10, 128), (4, 2, 64), (7, 1, 128)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("page,tokens,rows,single", [
    (16, [1, 1, 1], [1, 17, 300], True),
    (16, [40, 0, 1, 131], [40, 9, 16, 200], False),
    (1, [3, 2], [3, 50], False),
    (256, [300], [300], False),
])
def test_write_and_read(kind, heads, adjacent, page, tokens, rows, single):
    from dynamic_sparse_kv_gb300 import Rotary
    c = Case(kind, heads, page, tokens, rows, 1)
    half = c.d // 2
    axes = (half // 4, 3 * half // 8, 3 * half // 8)
    rot = Rotary(c.d, axes, positions=5000, base=1e6, adjacent=adjacent, device="cuda")
    cos, sin = (rot.cos_sin[..., i].cpu().numpy() for i in range(2))
    assert max(abs(a - b).max() for a, b in zip((cos, sin), table(5000, c.d, 1e6))) <= 2.0 ** -23
    pos = c.positions(3, 5000)
    before = c.before()
    out_q = torch.full((c.t, c.hq, c.d), float("nan"), dtype=c.dt, device="cuda")
    c.dec.write_layer(0, c.k, c.v, q=c.q, out_q=out_q, rotary=rot, pos=pos.cuda(), q_start=None if single else c.start)
    axis = [0] * axes[0] + [1] * axes[1] + [2] * axes[2]
    turn = lambda x: rotate(f32(x), pos.numpy(), axis, cos, sin, adjacent)
    assert torch.equal(out_q.cpu(), torch.from_numpy(turn(c.q)).to(c.dt))
    k, v = turn(c.k), f32(c.v)
    c.check(before, k, v)
    # and back
    for dt in (F32, BF):
        back = [torch.full((c.t + 2, c.hkv, c.d), 3.0, dtype=dt, device="cuda") for _ in range(2)]
        c.dec.read_layer(0, c.start, *back)
        for w, x in enumerate((k, v)):
            want = torch.from_numpy(x).to(c.dt).float()
            if kind == "fp4":
                for h in range(c.hkv):
                    gain = float(c.gain[w][0, h])
                    codes, scales = quantise(x[:, h], gain)
                    want[:, h] = torch.from_numpy(values(codes, scales, 1.0).astype(np.float32)) * np.float32(gain)
            assert torch.equal(back[w][:c.t].cpu() + 0.0, want.to(dt) + 0.0)
            assert bool((back[w][c.t:] == 3.0).all())      # rows behind the last sequence
    assert c.dec.device_status() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads,tokens,adjacent", [((28, 4, 128), [700, 0, 333, 1], False), ((28, 4, 128), [499, 1], True),
                                                   ((20, 20, 64), [801], False), ((10, 10, 128), [5000, 3], True),
                                                   ((64, 8, 128), [600, 40], False), ((16, 16, 128), [5000], False)])
def test_many_tokens(kind, heads, tokens, adjacent):
    """Prompts, some of whose rows no sequence has: the last 8 tokens are behind the last sequence."""
    from dynamic_sparse_kv_gb300 import Rotary
    c = Case(kind, heads, 16, tokens, [t + 5 for t in tokens], 11)
    wide = torch.cat([c.qkv, c.qkv[:8]])
    c.t += 8
    a, b = c.hq * c.d, (c.hq + c.hkv) * c.d
    q, k, v = (x.unflatten(1, (-1, c.d)) for x in (wide[:, :a], wide[:, a:b], wide[:, b:b + c.hkv * c.d]))
    rot = Rotary(c.d, (c.d // 8, 3 * c.d // 8), positions=6000, adjacent=adjacent, device="cuda")
    cos, sin = (rot.cos_sin[..., i].cpu().numpy() for i in range(2))
    pos = c.positions(2, 6000)
    pos[:, -8:] = 10 ** 6                   # nobody's
    before = c.before()
    out_q = torch.full((c.t, c.hq, c.d), 5.0, dtype=c.dt, device="cuda")
    c.dec.write_layer(0, k, v, q=q, out_q=out_q, rotary=rot, pos=pos.cuda(), q_start=c.start)
    axis = [0] * (c.d // 8) + [1] * (3 * c.d // 8)
    n = c.t - 8
    turn = lambda x: rotate(f32(x[:n]), pos.numpy()[:, :n], axis, cos, sin, adjacent)
    assert torch.equal(out_q[:n].cpu(), torch.from_numpy(turn(q)).to(c.dt)) and bool((out_q[n:] == 5.0).all())
    c.check(before, turn(k), f32(v[:n]))
    # and in place
    same = q.contiguous()
    c.dec.write_layer(0, k, v, q=same, out_q=same, rotary=rot, pos=pos.cuda(), q_start=c.start)
    assert torch.equal(same[:n], out_q[:n]) and torch.equal(same[n:], q[n:])
    assert c.dec.device_status() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_many_tokens_without_rows_are_reported(kind):
    from dynamic_sparse_kv_gb300 import Rotary
    from dynamic_sparse_kv_gb300 import _native as N
    c = Case(kind, (28, 4, 128), 16, [600, 300], [600, 300], 12)
    rot = Rotary(128, (64,), positions=100, device="cuda")
    cos, sin = (rot.cos_sin[..., i].cpu().numpy() for i in range(2))
    pos = c.positions(1, 100)
    pos[0, 64] = -1
    c.dec.seq_len[0] = 590                  # ten tokens have no row
    c.dec.block_table[1, 3] = -1            # nor have rows 48 .. 63 of sequence 1
    before = c.before()
    c.rows[0] = 590
    out_q = torch.empty(c.t, c.hq, c.d, dtype=c.dt, device="cuda")
    c.dec.write_layer(0, c.k, c.v, q=c.q, out_q=out_q, rotary=rot, pos=pos.cuda(), q_start=c.start)
    assert c.dec.device_status() == N.DEV_BAD_GROUP | N.DEV_BAD_PAGE | N.DEV_BAD_POSITION
    turn = lambda x: rotate(f32(x), pos.numpy(), [0] * 64, cos, sin, False)
    assert torch.equal(out_q.cpu(), torch.from_numpy(turn(c.q)).to(c.dt))
    c.check(before, turn(c.k), f32(c.v), skip=[*range(10), *range(648, 664)])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rotary_dim,adjacent", [(32, False), (64, True), (96, False)])
def test_part_of_a_head_turns(kind, rotary_dim, adjacent):
    from dynamic_sparse_kv_gb300 import Rotary
    c = Case(kind, (6, 2, 128), 16, [5, 20], [7, 20], 2)
    rot = Rotary(128, (rotary_dim // 2,), positions=64, rotary_dim=rotary_dim, adjacent=adjacent, device="cuda")
    pos = c.positions(1, 64)
    before = c.before()
    out_q = torch.empty(c.t, c.hq, c.d, dtype=c.dt, device="cuda")
    c.dec.write_layer(0, c.k, c.v, q=c.q, out_q=out_q, rotary=rot, pos=pos.cuda(), q_start=c.start)
    cos, sin = (rot.cos_sin[..., i].cpu().numpy() for i in range(2))
    turn = lambda x: rotate(f32(x), pos.numpy(), [0] * (rotary_dim // 2), cos, sin, adjacent)
    assert torch.equal(out_q.cpu(), torch.from_numpy(turn(c.q)).to(c.dt))
    c.check(before, turn(c.k), f32(c.v))


@pytest.mark.parametrize("kind", KINDS)
def test_without_rotary_and_without_queries(kind):
    c = Case(kind, (4, 2, 64), 16, [1, 1], [1, 40], 3)
    before = c.before()
    c.dec.write_layer(0, c.k, c.v)
    c.check(before, f32(c.k), f32(c.v))
    q = c.q.contiguous()
    out = torch.empty_like(q)
    c.dec.write_layer(0, c.k, c.v, q=q, out_q=out)
    assert torch.equal(q, out)


def test_queries_turn_in_place():
    from dynamic_sparse_kv_gb300 import Rotary
    c = Case("bf16", (28, 4, 128), 16, [70], [70], 4)
    rot = Rotary(128, (64,), positions=100, device="cuda")
    pos = c.positions(1, 100).cuda()
    q = c.q.contiguous()
    out = torch.empty_like(q)
    c.dec.write_layer(0, c.k, c.v, q=q, out_q=out, rotary=rot, pos=pos, q_start=c.start)
    c.dec.write_layer(0, c.k, c.v, q=q, out_q=q, rotary=rot, pos=pos, q_start=c.start)
    assert torch.equal(q, out)


def test_axes_in_turn_and_with_frequencies_of_their_own():
    from dynamic_sparse_kv_gb300 import Rotary
    r = Rotary(64, (14, 9, 9), positions=50, interleaved=True, device="cuda")
    assert r.axis.tolist() == [0, 1, 2] * 9 + [0] * 5
    r = Rotary(64, (16, 16), positions=50, per_axis=True, base=100.0, device="cuda")
    f = np.concatenate([100.0 ** -(np.arange(16) / 16)] * 2)
    for i, x in enumerate(table(50, 64, f)):
        assert np.abs(r.cos_sin[..., i].cpu().numpy() - x).max() <= 2.0 ** -23


@pytest.mark.parametrize("kind", KINDS)
def test_tokens_without_a_row_are_left_out_and_reported(kind):
    from dynamic_sparse_kv_gb300 import Rotary
    from dynamic_sparse_kv_gb300 import _native as N
    c = Case(kind, (4, 2, 64), 16, [3, 3, 2, 2], [40, 3, 2, 60], 5)
    rot = Rotary(64, (32,), positions=30, device="cuda")
    cos, sin = (rot.cos_sin[..., i].cpu().numpy() for i in range(2))
    pos = c.positions(1, 30)
    pos[0, 0], pos[0, 9] = -4, 1000
    lens = torch.tensor([40, 2, -1, 60], dtype=torch.int32, device="cuda")   # two short of a row, one unusable
    c.dec.set_seq_len(lens)
    c.rows[1] = 2
    c.dec.block_table[0, 2] = 10 ** 6
    before = c.before()
    out_q = torch.empty(c.t, c.hq, c.d, dtype=c.dt, device="cuda")
    # tokens 0-2: rows 37-39, page 2: gone; 3: row -1; 4, 5: rows 0, 1; 6, 7: no length
    c.dec.write_layer(0, c.k, c.v, q=c.q, out_q=out_q, rotary=rot, pos=pos.cuda(), q_start=c.start)
    assert c.dec.device_status() == N.DEV_BAD_PAGE | N.DEV_BAD_GROUP | N.DEV_BAD_SEQLEN | N.DEV_BAD_POSITION
    turn = lambda x: rotate(f32(x), pos.numpy(), [0] * 32, cos, sin, False)
    assert torch.equal(out_q.cpu(), torch.from_numpy(turn(c.q)).to(c.dt))
    c.check(before, turn(c.k), f32(c.v), skip=(0, 1, 2, 3, 6, 7))
    back = [torch.full((c.t, 2, 64), 3.0, device="cuda") for _ in range(2)]
    c.dec.read_layer(0, c.start, *back)
    for x in back:
        assert [bool((x[i] == 0).all()) for i in range(c.t)] == [True] * 4 + [False] * 2 + [True] * 2 + [False] * 2
    assert c.dec.device_status() == N.DEV_BAD_PAGE | N.DEV_BAD_GROUP | N.DEV_BAD_SEQLEN


@pytest.mark.parametrize("start", [[0, 5, 3, 8], [-2, 3, 5, 8], [0, 3, 5, 100], [8, 5, 3, 0]])
def test_offsets_out_of_order_fault_nothing(start):
    c = Case("bf16", (4, 2, 64), 16, [3, 2, 3], [40, 16, 30], 6)
    mark = c.dec.block_table.clone()
    c.dec.write_layer(0, c.k, c.v, q_start=torch.tensor(start, dtype=torch.int32, device="cuda"))
    back = [torch.empty(8, 2, 64, device="cuda") for _ in range(2)]
    c.dec.read_layer(0, torch.tensor(start, dtype=torch.int32, device="cuda"), *back)
    torch.cuda.synchronize()
    assert torch.equal(mark, c.dec.block_table)
    free = sorted(set(range(c.pages)) - set(c.table.flatten().tolist()))
    assert bool((c.caches[0][0, free] == 7.0).all())
    c.dec.device_status()


def test_groups_at_the_ends_of_the_4_bit_range():
    c = Case("fp4", (4, 2, 64), 16, [8], [8], 7)
    inf, nan = float("inf"), float("nan")
    for w in range(2):
        c.gain[w].fill_(1.0)
        c.caches[w].gain.fill_(1.0)
    x = torch.randn(8, 2, 64, generator=c.g)
    x[0] = 0
    x[1, :, :16], x[1, :, 20], x[1, :, 40] = 5.0, inf, nan
    x[2] *= 1e30                # past 448 * 6: all at the largest value
    x[3] *= 1e-30               # below the smallest scale: zeros
    x[4] = 2.0 ** -9 * 6
    x[5] *= 2.0 ** -8           # scales among e4m3's smallest
    x[6] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 8)    # every tie, a scale of 1
    x[7] = -x[6]
    x = x.to(BF).cuda()
    before = c.before()
    c.dec.write_layer(0, x, -x, q_start=c.start)
    c.check(before, f32(x), -f32(x))
    s = c.raw(0)[1][0, int(c.table[0, 0]), 0]
    assert s[1].tolist()[1:3] == [0x7f, 0x7f] and s[1, 0] != 0x7f
    assert s[2].max() == 0x7e and s[3].max() == 0


def test_a_long_cache_is_written_past_4_gib():
    from dynamic_sparse_kv_gb300 import DecodeAttention
    pages, hkv, d, page = 8400, 8, 128, 256
    k = torch.zeros(1, pages, hkv, page, d, dtype=BF, device="cuda")
    v = torch.zeros_like(k)
    assert k.numel() * 2 > 2 ** 32
    t = torch.tensor([[0, pages - 1]], dtype=torch.int32)
    dec = DecodeAttention(k, v, t, q_heads=8)
    dec.set_seq_len(300)
    x = torch.randn(1, hkv, d, device="cuda").to(BF)
    dec.write_layer(0, x, -x)
    assert torch.equal(k[0, -1, :, 299 - 256], x[0]) and torch.equal(v[0, -1, :, 299 - 256], -x[0])
    assert int((k != 0).any(-1).sum()) == hkv
    out = [torch.empty(1, hkv, d, device="cuda") for _ in range(2)]
    dec.read_layer(0, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), *out)
    assert torch.equal(out[0], x.float())


def test_captured_and_replayed():
    from dynamic_sparse_kv_gb300 import Rotary
    c = Case("fp4", (28, 4, 128), 16, [1, 1], [20, 33], 8)
    rot = Rotary(128, (64,), positions=100, device="cuda")
    pos = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    out = torch.empty(2, 28, 128, dtype=BF, device="cuda")
    call = lambda: c.dec.write_layer(0, c.k, c.v, q=c.q, out_q=out, rotary=rot, pos=pos)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    c.rows = [21, 34]
    c.dec.seq_len.add_(1)
    pos.fill_(50)
    c.qkv.mul_(-0.5)
    before = c.before()
    graph.replay()
    cos, sin = (rot.cos_sin[..., i].cpu().numpy() for i in range(2))
    turn = lambda x: rotate(f32(x), pos.cpu().numpy(), [0] * 64, cos, sin, False)
    c.check(before, turn(c.k), f32(c.v))
    assert torch.equal(out.cpu(), torch.from_numpy(turn(c.q)).to(BF))
