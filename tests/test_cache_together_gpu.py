"""Pages reserved, tokens written with rotary positions, sequences forked, attended to,
released and moved together, as a decode loop uses them, against lists and 64 bits."""
import numpy as np
import pytest
import torch

from cache_harness import check_out4, quantise, rotate, values
from rows_harness import check_out, np64

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
HQ, HKV, D, PAGE, LAYERS = 28, 4, 128, 16, 2


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


class Loop:
    def __init__(self, kind, batch=4, pages=120, seed=3):
        from dynamic_sparse_kv_gb300 import DecodeAttention, Fp4Cache, PagePool, Rotary
        self.kind, self.batch = kind, batch
        self.g = torch.Generator().manual_seed(seed)
        shape = (LAYERS, pages, HKV, PAGE, D)
        self.gain = [0.05 + torch.rand(LAYERS, HKV, generator=self.g) for _ in range(2)]
        if kind == "fp4":
            caches = [Fp4Cache(*shape, gain=x, device="cuda") for x in self.gain]
        else:
            caches = [torch.full(shape, float("nan"), dtype=BF, device="cuda") for _ in range(2)]
        table = torch.zeros(batch, 30, dtype=torch.int32, device="cuda")
        self.dec = DecodeAttention(*caches, table, q_heads=HQ)
        self.pool = PagePool(self.dec)
        self.rot = Rotary(D, (16, 24, 24), positions=500, base=1e6, device="cuda")
        self.cos, self.sin = (self.rot.cos_sin[..., i].cpu().numpy() for i in range(2))
        self.axis = [0] * 16 + [1] * 24 + [2] * 24
        self.rows = [[[np.zeros((0, HKV, D))] * 2 for _ in range(batch)] for _ in range(LAYERS)]

    def tokens(self, counts):
        """q, k, v [L, T, ...] and positions of counts[b] new tokens."""
        t = sum(counts)
        x = [torch.randn(LAYERS, t, h, D, generator=self.g).to(BF) for h in (HQ, HKV, HKV)]
        pos = torch.randint(0, 500, (3, t), generator=self.g).to(torch.int32)
        return [y.cuda() for y in x], pos

    def held(self, x, w, l):
        """What layer l's cache w holds of rows x [T, H_kv, d] float32."""
        if self.kind != "fp4":
            return torch.from_numpy(x).to(BF).double().numpy()
        out = np.zeros(x.shape)
        for h in range(HKV):
            gain = float(self.gain[w][l, h])
            out[:, h] = values(*quantise(x[:, h], gain), gain)
        return out

    def note(self, counts, qkv, pos):
        """The model's rows; returns the turned queries."""
        turned = []
        for l in range(LAYERS):
            q, k, v = (y[l].float().cpu().numpy() for y in qkv)
            turn = lambda y: rotate(y, pos.numpy(), self.axis, self.cos, self.sin, False)
            turned.append(torch.from_numpy(turn(q)).to(BF))
            new = self.held(turn(k), 0, l), self.held(v, 1, l)
            at = 0
            for b, n in enumerate(counts):
                self.rows[l][b] = [np.concatenate([old, x[at:at + n]]) for old, x in zip(self.rows[l][b], new)]
                at += n
        return torch.stack(turned)

    def prompt(self, counts):
        (q, k, v), pos = self.tokens(counts)
        self.pool.reserve(torch.tensor(self.lens()) + torch.tensor(counts))
        self.dec.seq_len.add_(torch.tensor(counts, dtype=torch.int32, device="cuda"))
        start = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
        out = torch.empty_like(q)
        for l in range(LAYERS):
            self.dec.write_layer(l, k[l], v[l], q=q[l], out_q=out[l], rotary=self.rot, pos=pos.cuda(), q_start=start)
        assert torch.equal(out.cpu(), self.note(counts, (q, k, v), pos))

    def lens(self):
        return [len(r[0]) for r in self.rows[0]]

    def step(self, replay=None):
        """One token more in every sequence; returns and checks the outputs."""
        (q, k, v), pos = self.tokens([1] * self.batch)
        out, qt = torch.full_like(q, float("nan")), torch.empty_like(q)
        gpu_pos = pos.cuda()

        def write(l, before):
            if before:
                self.dec.write_layer(l, k[l], v[l], q=q[l], out_q=qt[l], rotary=self.rot, pos=gpu_pos)

        if replay is None:
            self.pool.reserve(extra=1)
            self.dec.begin_token()
            self.dec.dense_step(qt, out, hook=write)
        else:
            out = replay(q, k, v, gpu_pos)
        turned = self.note([1] * self.batch, (q, k, v), pos)
        for l in range(LAYERS):
            for b in range(self.batch):
                K, V = self.rows[l][b]
                where = f"layer {l} sequence {b}"
                if self.kind == "fp4":
                    check_out4(out[l, b:b + 1], np64(turned[l, b:b + 1]), K, V, where)
                else:
                    check_out(out[l, b:b + 1], np64(turned[l, b:b + 1]), K, V, BF, where)
        assert self.dec.device_status() == 0
        return out


@pytest.mark.parametrize("kind", ["bf16", "fp4"])
def test_prompt_fork_decode_release_compact(kind):
    t = Loop(kind)
    t.prompt([100, 33, 0, 0])
    t.prompt([40, 15, 0, 0])          # in two chunks; sequence 1 ends a page
    t.pool.fork([0, 1], [2, 3])
    for rows in t.rows:
        rows[2], rows[3] = list(rows[0]), list(rows[1])
    for _ in range(3):
        t.step()
    t.pool.release([0])
    t.pool.fork(torch.tensor([3], dtype=torch.int32, device="cuda"), torch.tensor([0], dtype=torch.int32, device="cuda"))
    for rows in t.rows:
        rows[0] = list(rows[3])
    t.pool.compact()
    used = len(set(t.dec.block_table[t.dec.block_table >= 0].tolist()))
    assert int(t.pool.used[0]) == used and int(t.dec.block_table.max()) == used - 1
    for _ in range(17):
        t.step()
    # two tokens are taken back: their page goes, and the next tokens are others
    t.dec.seq_len.sub_(2)
    t.pool.trim()
    for rows in t.rows:
        for b in range(t.batch):
            rows[b] = [x[:-2] for x in rows[b]]
    for _ in range(3):
        t.step()
    start = torch.tensor(np.concatenate([[0], np.cumsum(t.lens())]), dtype=torch.int32, device="cuda")
    back = [torch.empty(sum(t.lens()), HKV, D, device="cuda") for _ in range(2)]
    for l in range(LAYERS):
        t.dec.read_layer(l, start, *back)
        for w in range(2):
            assert np.array_equal(back[w].cpu().numpy(), np.concatenate([r[w] for r in t.rows[l]]).astype(np.float32))


@pytest.mark.parametrize("kind", ["bf16", "fp4"])
def test_a_captured_loop_replays(kind):
    t = Loop(kind, seed=5)
    t.prompt([30, 47, 5, 16])
    q, k, v = (torch.zeros(LAYERS, t.batch, h, D, dtype=BF, device="cuda") for h in (HQ, HKV, HKV))
    pos = torch.zeros(3, t.batch, dtype=torch.int32, device="cuda")
    qt, out = torch.empty_like(q), torch.empty_like(q)

    def write(l, before):
        if before:
            t.dec.write_layer(l, k[l], v[l], q=q[l], out_q=qt[l], rotary=t.rot, pos=pos)

    t.dec._set_hint(64)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.pool.reserve(extra=1)
        t.dec.seq_len.add_(1)
        t.dec.dense_step(qt, out, hook=write)

    def replay(*new):
        for mine, x in zip((q, k, v, pos), new):
            mine.copy_(x)
        graph.replay()
        return out

    for _ in range(20):
        t.step(replay)


def test_two_pools_on_two_streams():
    a, b = Loop("fp4", seed=7), Loop("bf16", seed=8)
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for x in s:
        x.wait_stream(torch.cuda.current_stream())
    for loop, stream, counts in ((a, s[0], [20, 31, 0, 1]), (b, s[1], [16, 2, 70, 9])):
        with torch.cuda.stream(stream):
            loop.prompt(counts)
    for _ in range(4):
        for loop, stream in ((a, s[0]), (b, s[1])):
            with torch.cuda.stream(stream):
                loop.step()
