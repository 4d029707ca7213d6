"""Shared-prefix attention, weighing, eviction and cross attention on the GPU
against the fp64 oracle, at the sizes and masks where they can go wrong."""
import numpy as np
import pytest
import torch

from oracle import rows as R
from rows_harness import Paged, check_out, np64

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def decoder(c, n, q_heads):
    from dynamic_sparse_kv_gb300 import DecodeAttention
    dec = DecodeAttention(c.k[None], c.v[None], c.gpu_table(), q_heads=q_heads)
    dec.set_seq_len(torch.tensor(n, dtype=torch.int32, device="cuda"))
    return dec


def shared_case(sizes, prefixes, tails, heads, page, dtype, seed):
    """Groups of `sizes` sequences; returns (cache, start, prefix [B], n [B], q)."""
    hq, hkv, d = heads
    start = np.concatenate([[0], np.cumsum(sizes)]).tolist()
    prefix = [p for s, p in zip(sizes, prefixes) for _ in range(s)]
    n = [p + t for p, t in zip(prefix, tails)]
    c = Paged(len(n), max(n), hkv, d, page, dtype, seed)
    g = torch.Generator().manual_seed(seed + 1)
    q = (2 * torch.randn(len(n), hq, d, generator=g)).to(dtype).cuda()
    return c, start, prefix, n, q


def check_shared(c, start, prefix, n, q, out):
    ps = []
    for i in range(len(start) - 1):
        for b in range(start[i], start[i + 1]):
            K0, V0 = c.rows(start[i], 0, prefix[b])
            K1, V1 = c.rows(b, prefix[b], n[b])
            K, V = np.concatenate([K0, K1]), np.concatenate([V0, V1])
            ps.append(check_out(out[b:b + 1], np64(q[b:b + 1]), K, V, q.dtype, f"sequence {b}"))
    return ps


HEADS = [(28, 4, 128), (10, 10, 128), (4, 2, 64), (8, 1, 64), (15, 3, 128)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("page,sizes,prefixes,tails", [
    (16, [3, 1, 2], [130, 17, 400], [1, 40, 7, 1, 16, 90]),
    (1, [2], [65], [3, 1]),
    (256, [1, 4], [511, 256], [2, 1, 300, 5, 6]),
    (4, [5], [1], [1, 2, 3, 4, 5]),
    (16, [2, 2], [0, 127], [1, 33, 2, 128]),
    (32, [40], [300], list(range(1, 41))),
])
def test_shared_prefix(dtype, heads, page, sizes, prefixes, tails):
    c, start, prefix, n, q = shared_case(sizes, prefixes, tails, heads, page, dtype, 3)
    dec = decoder(c, n, heads[0])
    dec.share_prefix(start, torch.tensor(prefix))
    dec.groups["ws"].fill_(127)       # whatever was in it: huge finite floats
    out = torch.full_like(q, float("nan"))
    dec.shared_layer(0, q, out)
    check_shared(c, start, prefix, n, q, out)
    assert dec.device_status() == 0


def test_shared_prefix_without_tail_and_with_empty_groups():
    heads = (4, 2, 64)
    c, _, prefix, n, q = shared_case([3], [70], [0, 0, 5], heads, 16, BF, 5)
    from dynamic_sparse_kv_gb300 import _native as N
    dec = decoder(c, n, 4)
    start = torch.tensor([0, 0, 3, 3], dtype=torch.int32, device="cuda")
    dec.share_prefix(start, torch.tensor(prefix))
    out = torch.full_like(q, float("nan"))
    dec.shared_layer(0, q, out)
    check_shared(c, [0, 3], prefix, n, q, out)
    assert dec.device_status() == 0
    g = dec.groups
    with pytest.raises(N.FastOCRError):
        N.fastocr_shared_attend(dec.handle, q, dec.kv[0], g["c"], out, g["ws"], g["ws"].numel() - 256)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("heads", HEADS[:3])
@pytest.mark.parametrize("splits", [0, 1, 5])
def test_weighed_attention(dtype, heads, splits):
    """Weights with and without a shared prefix; rows past the stride and protected ones get none."""
    hq, hkv, d = heads
    c, start, prefix, n, q = shared_case([2, 2], [40, 0], [30, 1, 200, 64], heads, 16, dtype, 7)
    from dynamic_sparse_kv_gb300 import _native as N
    for shared in (False, True):
        dec = decoder(c, n, hq)
        if splits:
            N.fastocr_set_splits(dec.handle, 0, splits)
        protect = [40, 40, 0, 70]       # sequence 3: nothing weighed yet but what follows
        rows = 200
        mass0 = torch.rand(1, 4, hkv, rows, generator=torch.Generator().manual_seed(1))
        pos0 = torch.arange(rows, dtype=torch.int32).expand(1, 4, hkv, rows).contiguous()
        seen = torch.tensor([100, 50, 900, 64], dtype=torch.int32, device="cuda")
        dec.track_weights(rows, torch.tensor(protect), mass=mass0.cuda(), pos=pos0.cuda(), seen=seen)
        out = torch.full_like(q, float("nan"))
        if shared:
            dec.share_prefix(start, torch.tensor(prefix))
            dec.shared_layer(0, q, out)
            full = [(start[0 if b < 2 else 1], prefix[b]) for b in range(4)]
        else:
            dec.weigh_layer(0, q, out)
            full = [(b, 0) for b in range(4)]
        mass, pos = np64(dec.weights["mass"][0]), dec.weights["pos"][0].cpu().numpy()
        for b in range(4):
            K0, V0 = c.rows(full[b][0], 0, full[b][1])
            K1, V1 = c.rows(b, full[b][1], n[b])
            K, V = np.concatenate([K0, K1]), np.concatenate([V0, V1])
            p, cb = check_out(out[b:b + 1], np64(q[b:b + 1]), K, V, dtype, f"sequence {b}")
            want, wpos = R.add_weights(np64(mass0[0, b]), pos0[0, b].numpy(), p[0], n[b], protect[b],
                                       int(seen[b]), hkv)
            # a sum of g probabilities, then one addition
            tol = (cb.max() + 9 * 2.0 ** -24) * np.abs(want) + 2.0 ** -24
            assert (np.abs(mass[b] - want) <= tol).all(), (b, np.abs(mass[b] - want).max())
            assert np.array_equal(pos[b], wpos)
        assert dec.device_status() == 0
        dec.close()


def run_evict(c, n, hq, mass, pos, seen, protect, budget, recent):
    dec = decoder(c, n, hq)
    dec.track_weights(mass.shape[-1], torch.tensor(protect), mass=mass.cuda()[None].contiguous(),
                      pos=pos.cuda()[None].contiguous(),
                      seen=torch.tensor(seen, dtype=torch.int32, device="cuda"))
    new_len = torch.full((len(n),), -7, dtype=torch.int32, device="cuda")
    dec.evict_layer(0, budget, recent, new_len)
    torch.cuda.synchronize()
    return dec, new_len


def check_evict(c, k0, v0, n, mass0, pos0, seen, protect, budget, recent, dec, new_len):
    """Every byte of K, V, mass and pos as the oracle's moves leave them."""
    k, v = k0.cpu().clone(), v0.cpu().clone()
    mass, pos = mass0.clone(), pos0.clone()
    hkv = mass0.shape[1]
    for b in range(len(n)):
        rows = max(0, n[b] - protect[b])
        assert int(new_len[b]) == min(n[b], protect[b]) + min(rows, budget), b
        for h in range(hkv):
            if rows <= budget:
                continue
            _, moves = R.evict_moves(mass0[b, h].tolist(), pos0[b, h].tolist(), rows, seen[b], budget, recent)
            for x, y in moves:
                mass[b, h, y], pos[b, h, y] = mass0[b, h, x], pos0[b, h, x]
                rx, ry = x + protect[b], y + protect[b]
                px, py = int(c.table[b, rx // c.page]), int(c.table[b, ry // c.page])
                k[py, h, ry % c.page] = k0.cpu()[px, h, rx % c.page]
                v[py, h, ry % c.page] = v0.cpu()[px, h, rx % c.page]
    w = dec.weights
    assert torch.equal(w["mass"][0].cpu().view(torch.int32), mass.view(torch.int32))
    assert torch.equal(w["pos"][0].cpu(), pos)
    assert torch.equal(c.k.cpu(), k) and torch.equal(c.v.cpu(), v)


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (F32, 64), (F32, 128)])
@pytest.mark.parametrize("page", [1, 16])
@pytest.mark.parametrize("rows,protect,stride,budget,recent", [
    ([9, 1, 0, 8], [0, 5, 3, 20], 9, 8, 3),
    ([300, 257, 256, 40], [17, 0, 1, 0], 300, 256, 100),
    ([1000, 999, 3, 700], [0, 0, 0, 31], 1024, 1, 0),
    ([1000, 64, 65, 513], [5, 5, 5, 5], 1000, 64, 64),
    ([600, 100, 100, 601], [0, 0, 0, 0], 601, 300, 0),
])
def test_evict(dtype, d, page, rows, protect, stride, budget, recent):
    hkv = 3
    n = [r + p for r, p in zip(rows, protect)]
    c = Paged(4, max(n), hkv, d, page, dtype, 11)
    k0, v0 = c.k.clone(), c.v.clone()
    g = torch.Generator().manual_seed(2)
    mass = torch.exp(2 * torch.randn(4, hkv, stride, generator=g))
    mass[:, 1] = (mass[:, 1] * 2).round() / 2          # many ties, zeros among them
    mass[0, 2, :3] = torch.tensor([float("nan"), float("inf"), -0.0])
    mass[3, 2] = -mass[3, 2]
    seen = [r + 50 for r in n]
    pos = torch.stack([torch.stack([s - 1 - torch.randperm(stride, generator=g) for _ in range(hkv)])
                       for s in seen]).to(torch.int32)
    dec, new_len = run_evict(c, n, 2 * hkv, mass, pos, seen, protect, budget, recent)
    check_evict(c, k0, v0, n, mass, pos, seen, protect, budget, recent, dec, new_len)
    assert dec.device_status() == 0


@pytest.mark.parametrize("batch,rows,budget,recent", [(1, 20000, 5000, 64), (2, 9000, 8999, 500),
                                                      (1, 40001, 1000, 0), (1, 70000, 60000, 1)])
def test_evict_over_a_cluster(batch, rows, budget, recent):
    """Rows over several CTAs; equal weights make the tie order count across them."""
    hkv = 2
    c = Paged(batch, rows + 3, hkv, 64, 16, BF, 12)
    k0, v0 = c.k.clone(), c.v.clone()
    g = torch.Generator().manual_seed(4)
    mass = torch.randint(0, 7, (batch, hkv, rows), generator=g).float()
    seen = [rows + 3] * batch
    pos = (torch.arange(rows, dtype=torch.int32) + 3).expand(batch, hkv, rows).contiguous()
    dec, new_len = run_evict(c, [rows + 3] * batch, 4, mass, pos, seen, [3] * batch, budget, recent)
    check_evict(c, k0, v0, [rows + 3] * batch, mass, pos, seen, [3] * batch, budget, recent, dec, new_len)
    assert dec.device_status() == 0


def cross_case(t, n, heads, page, dtype, seed, spare=3):
    hq, hkv, d = heads
    c = Paged(len(n), max(max(n), 1), hkv, d, page, dtype, seed)
    g = torch.Generator().manual_seed(seed + 1)
    start = np.concatenate([[0], np.cumsum(t)]).astype(np.int32)
    q = (2 * torch.randn(int(start[-1]) + spare, hq, d, generator=g)).to(dtype).cuda()
    return c, torch.from_numpy(start).cuda(), q


def check_cross(c, t, n, q, out, spare=3):
    at = 0
    for b in range(len(n)):
        K, V = c.rows(b, 0, n[b])
        if t[b]:
            check_out(out[at:at + t[b]], np64(q[at:at + t[b]]), K, V, q.dtype, f"sequence {b}")
        at += t[b]
    assert (out[at:at + spare].float() == 7.0).all(), "rows behind the last sequence were written"


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("page,t,n", [
    (16, [1, 1, 1], [300, 1, 0]),
    (16, [0, 37, 2, 0], [5, 700, 128, 9]),
    (1, [3], [129]),
    (256, [1, 130], [513, 255]),
    (8, [19], [1000]),
    (16, [1, 1, 1, 1], [700, 0, 1, 333]),       # a decode step
    (16, [0, 3, 0, 1, 0], [40, 50, 60, 700, 0]),  # few tokens, not one a sequence
    (4, [1, 0, 2], [129, 5, 64]),
])
@pytest.mark.parametrize("any_rows", [False, True])
def test_cross_attention(dtype, heads, page, t, n, any_rows):
    from dynamic_sparse_kv_gb300 import CrossAttention
    c, start, q = cross_case(t, n, heads, page, dtype, 21)
    ca = CrossAttention(c.k[None], c.v[None], c.gpu_table(), torch.tensor(n), q_heads=heads[0],
                        max_rows=None if any_rows else q.shape[0])
    ca.ws.fill_(127)
    out = torch.full_like(q, 7.0)
    ca.attend(0, q, start, out)
    check_cross(c, t, n, q, out)
    assert ca.device_status() == 0


def test_infinities_outside_the_attended_rows():
    """Rows past N_t, past the prefix in the leader's pages and in unused pages may hold anything."""
    heads = (8, 2, 128)
    c, start, prefix, n, q = shared_case([2, 1], [100, 37], [3, 1, 20], heads, 16, BF, 31)
    for x in (c.k, c.v):
        own = torch.ones(x.shape[0], x.shape[2], dtype=torch.bool)
        for i in range(2):
            for b in range(start[i], start[i + 1]):
                for r in range(n[b]):
                    lead = start[i] if r < prefix[b] else b
                    own[int(c.table[lead, r // 16]), r % 16] = False
        x.permute(0, 2, 1, 3)[own.cuda()] = float("nan")
    dec = decoder(c, n, 8)
    dec.share_prefix(start, torch.tensor(prefix))
    out = torch.full_like(q, float("nan"))
    dec.shared_layer(0, q, out)
    check_shared(c, start, prefix, n, q, out)
    out2 = torch.full((8, 8, 128), 7.0, dtype=BF, device="cuda")
    from dynamic_sparse_kv_gb300 import CrossAttention
    ca = CrossAttention(c.k[None], c.v[None], c.gpu_table(), torch.tensor([100, 0, 37]), q_heads=8,
                        max_rows=8)
    q2 = torch.randn(8, 8, 128, device="cuda").to(BF)
    ca.attend(0, q2, torch.tensor([0, 4, 5, 5], dtype=torch.int32, device="cuda"), out2)
    check_cross(c, [4, 1, 0], [100, 0, 37], q2, out2)


def test_bad_device_data_is_reported_and_masked():
    from dynamic_sparse_kv_gb300 import CrossAttention, _native as N
    heads = (4, 2, 64)
    c, start, prefix, n, q = shared_case([2, 1], [64, 20], [3, 1, 20], heads, 16, BF, 41)
    table = c.table.clone()
    c.table[0, 1] = 10 ** 6
    dec = decoder(c, n, 4)
    dec.share_prefix(start, torch.tensor(prefix))
    out = torch.full_like(q, float("nan"))
    dec.shared_layer(0, q, out)
    assert dec.device_status() == N.DEV_BAD_PAGE
    assert torch.isfinite(out.float()).all()
    # the masked page's rows are left out for the whole group
    c.table = table
    K0, V0 = c.rows(0, 0, 64)
    for b in (0, 1):
        K1, V1 = c.rows(b, 64, n[b])
        keep = np.r_[0:16, 32:64]
        check_out(out[b:b + 1], np64(q[b:b + 1]), np.concatenate([K0[keep], K1]),
                  np.concatenate([V0[keep], V1]), BF)
    dec.close()

    dec = decoder(c, n, 4)
    for start_bad, prefix_bad in (([0, 2, 5], prefix), ([0, 3, 2], prefix), ([-1, 2, 3], prefix),
                                  ([0, 1, 2], prefix), (start, [64, 60, 20]), (start, [900, 900, 20]),
                                  (start, [-1, -1, 20])):
        dec.share_prefix(torch.tensor(start_bad, dtype=torch.int32, device="cuda"),
                         torch.tensor(prefix_bad), max_prefix=64)
        dec.shared_layer(0, q, out)
        assert dec.device_status() == N.DEV_BAD_GROUP, (start_bad, prefix_bad)

    dec.track_weights(4, 0)
    dec.weigh_layer(0, q, out)
    assert dec.device_status() == N.DEV_BAD_WEIGHTS
    new_len = torch.zeros(3, dtype=torch.int32, device="cuda")
    k0 = c.k.clone()
    dec.evict_layer(0, 2, 1, new_len)      # more rows than weights: left as they are
    assert dec.device_status() == N.DEV_BAD_WEIGHTS
    assert new_len.tolist() == n and torch.equal(c.k, k0)

    ca = CrossAttention(c.k[None], c.v[None], c.gpu_table(), torch.tensor([64, 10 ** 6, -1]), q_heads=4,
                        max_rows=3)
    for qs, want in (([0, 1, 2, 3], N.DEV_BAD_SEQLEN), ([0, 1, 1, 9], N.DEV_BAD_GROUP | N.DEV_BAD_SEQLEN),
                     ([0, 1, 0, 1], N.DEV_BAD_GROUP | N.DEV_BAD_SEQLEN)):
        ca.attend(0, q, torch.tensor(qs, dtype=torch.int32, device="cuda"), out)
        got = ca.device_status()
        assert got & want and not got & ~want, (qs, got)


def simulate(steps, budget, recent, graph):
    """Two documents, five answers: every step appends a token, attends over the shared prefix
    with weights, and evicts; checked against the oracle after each step."""
    from dynamic_sparse_kv_gb300 import CapturedStep, DecodeAttention
    heads, page, dtype = (6, 2, 64), 8, BF
    sizes, prefixes = [3, 2], [50, 27]
    start = [0, 3, 5]
    prefix = [50] * 3 + [27] * 2
    protect = [p + 2 for p in prefix]          # two own tokens (a question) stay as well
    layers = 2
    cs = [Paged(5, 50 + 2 + budget + 4, 2, 64, page, dtype, 50 + l) for l in range(layers)]
    k, v = torch.stack([c.k for c in cs]), torch.stack([c.v for c in cs])
    for c in cs:
        c.table = cs[0].table
    dec = DecodeAttention(k, v, cs[0].gpu_table(), q_heads=6)
    n = list(protect)
    dec.set_seq_len(torch.tensor(n, dtype=torch.int32, device="cuda"))
    dec.share_prefix(start, torch.tensor(prefix))
    dec.track_weights(budget + 1, torch.tensor(protect))
    w = dec.weights
    mass, pos = np64(w["mass"]), w["pos"].cpu().numpy().astype(np.int64)
    seen = list(n)
    step = None
    g = torch.Generator().manual_seed(9)
    q = torch.empty(layers, 5, 6, 64, dtype=dtype, device="cuda")
    out = torch.empty_like(q)
    for t in range(steps):
        dec.begin_token()
        n = [x + 1 for x in n]
        seen = [x + 1 for x in seen]
        new = torch.randn(2, layers, 5, 2, 64, generator=g).to(dtype).cuda()
        table = cs[0].table
        for b in range(5):
            r = n[b] - 1
            k[:, int(table[b, r // page]), :, r % page] = new[0][:, b]
            v[:, int(table[b, r // page]), :, r % page] = new[1][:, b]
        q.copy_((2 * torch.randn(q.shape, generator=g)).to(dtype))
        if graph and t == 0:
            saved = {x: w[x].clone() for x in ("mass", "pos")}
            step = CapturedStep(dec, "shared")
            for x in saved:
                w[x].copy_(saved[x])
        if step is not None:
            step.q.copy_(q)
            step.replay()
            out.copy_(step.out)
        else:
            dec.shared_step(q, out)
        for l in range(layers):
            for b in range(5):
                lead = 0 if b < 3 else 3
                K0, V0 = cs[l].rows(lead, 0, prefix[b], k[l], v[l])
                K1, V1 = cs[l].rows(b, prefix[b], n[b], k[l], v[l])
                K, V = np.concatenate([K0, K1]), np.concatenate([V0, V1])
                p, cb = check_out(out[l, b:b + 1], np64(q[l, b:b + 1]), K, V, dtype, f"step {t} layer {l} seq {b}")
                want, wpos = R.add_weights(mass[l, b], pos[l, b], p[0], n[b], protect[b], seen[b], 2)
                got = np64(w["mass"][l, b])
                assert (np.abs(got - want) <= (cb.max() + 9 * 2.0 ** -24) * np.abs(want) + 2.0 ** -24).all()
                assert np.array_equal(w["pos"][l, b].cpu().numpy(), wpos)
                mass[l, b], pos[l, b] = got, wpos        # go on from the GPU's weights, checked above
        before = (k.cpu().clone(), v.cpu().clone())
        dec.evict_step(budget, recent)
        for l in range(layers):
            for b in range(5):
                rows = n[b] - protect[b]
                if rows <= budget:
                    continue
                for h in range(2):
                    _, moves = R.evict_moves(mass[l, b, h], pos[l, b, h], rows, seen[b], budget, recent)
                    for x, y in moves:
                        mass[l, b, h, y], pos[l, b, h, y] = mass[l, b, h, x], pos[l, b, h, x]
                        rx, ry = x + protect[b], y + protect[b]
                        for s, d in zip(before, (k, v)):
                            src = s[l, int(table[b, rx // page]), h, rx % page]
                            assert torch.equal(d[l, int(table[b, ry // page]), h, ry % page].cpu(), src)
                assert np.array_equal(w["pos"][l, b].cpu().numpy(), pos[l, b])
        n = [protect[b] + min(n[b] - protect[b], budget) for b in range(5)]
        assert dec.seq_len.tolist() == n
    assert dec.device_status() == 0
    # the recent tokens are all there
    for l in range(layers):
        for b in range(5):
            for h in range(2):
                have = set(pos[l, b, h, :n[b] - protect[b]].tolist())
                assert {seen[b] - 1 - i for i in range(min(recent, steps))} <= have


@pytest.mark.parametrize("graph", [False, True])
def test_shared_prefix_weights_and_eviction_together(graph):
    simulate(steps=20, budget=9, recent=3, graph=graph)


def test_on_another_stream_and_twice_at_once():
    """Two handles on two streams, each captured once and replayed in turn."""
    heads = (28, 4, 128)
    runs = []
    for seed in (61, 62):
        c, start, prefix, n, q = shared_case([4], [700], [9, 30, 1, 4], heads, 16, BF, seed)
        dec = decoder(c, n, 28)
        dec.share_prefix(start, torch.tensor(prefix))
        out = torch.full_like(q, float("nan"))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            dec.shared_layer(0, q, out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            dec.shared_layer(0, q, out)
        runs.append((c, start, prefix, n, q, out, s, graph, dec))
    torch.cuda.synchronize()
    for _, _, _, _, _, out, _, _, _ in runs:
        out.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(3):
        for r in runs:
            with torch.cuda.stream(r[6]):
                r[7].replay()
    torch.cuda.synchronize()
    for c, start, prefix, n, q, out, *_ in runs:
        check_shared(c, start, prefix, n, q, out)


def test_refusals():
    from dynamic_sparse_kv_gb300 import CrossAttention, _native as N
    heads = (4, 2, 64)
    c, start, prefix, n, q = shared_case([2, 1], [40, 20], [3, 1, 20], heads, 16, BF, 71)
    dec = decoder(c, n, 4)
    out = torch.full_like(q, 7.0)
    with pytest.raises(RuntimeError):
        dec.shared_layer(0, q, out)
    with pytest.raises(RuntimeError):
        dec.weigh_layer(0, q, out)
    with pytest.raises(RuntimeError):
        dec.evict_layer(0, 1, 0)
    with pytest.raises(RuntimeError):
        dec.evict_step(1, 0)
    for bad in ([0, 2], [1, 3], [0, 2, 1, 3], [0], [0, 1, 1, 2, 3, 3]):
        with pytest.raises(ValueError):
            dec.share_prefix(bad, torch.tensor(prefix))
    with pytest.raises(ValueError):
        dec.share_prefix(start, torch.tensor([40, 20]))
    with pytest.raises(ValueError):
        dec.track_weights(0, 0)
    with pytest.raises(ValueError):
        dec.track_weights(5, 0, mass=torch.zeros(1, 3, 2, 4, device="cuda"))
    with pytest.raises(ValueError):
        dec.track_weights(5, 0, seen=torch.zeros(3, dtype=torch.int64, device="cuda"))
    dec.share_prefix(start, torch.tensor(prefix))
    dec.track_weights(64, torch.tensor(prefix))
    g, w = dec.groups, dec.weights["c"][0]

    def status(call, *args):
        with pytest.raises(N.FastOCRError) as e:
            call(*args)
        return e.value.status

    ws = g["ws"]
    assert status(N.fastocr_shared_attend, dec.handle, q, dec.kv[0], g["c"], out, ws, ws.numel() - 1) \
        == N.FASTOCR_ERR_INVALID
    assert status(N.fastocr_shared_attend, dec.handle, q, dec.kv[0], g["c"], out, None, 0) == N.FASTOCR_ERR_NULL
    assert status(N.fastocr_shared_attend, dec.handle, q, dec.kv[0], g["c"], out, ws.data_ptr() + 4,
                  ws.numel()) == N.FASTOCR_ERR_ALIGN
    none = N.make_groups(g["start"], g["prefix_len"])
    none.n = 0
    assert status(N.fastocr_shared_attend, dec.handle, q, dec.kv[0], none, out, ws, ws.numel()) \
        == N.FASTOCR_ERR_INVALID
    none.n = 4
    assert status(N.fastocr_shared_attend, dec.handle, q, dec.kv[0], none, out, ws, ws.numel()) \
        == N.FASTOCR_ERR_INVALID
    for budget, recent in ((0, 0), (4, 5), (4, -1)):
        assert status(N.fastocr_evict, dec.handle, dec.kv[0], w, budget, recent) == N.FASTOCR_ERR_INVALID
    assert status(N.fastocr_evict, dec.handle, dec.kv[0], w, 4, 1, dec.seq_len) == N.FASTOCR_ERR_INVALID
    no_logits = N.make_weights(dec.weights["mass"][0], dec.weights["pos"][0], dec.weights["protect"],
                               dec.weights["seen"], None)
    assert status(N.fastocr_weigh_attend, dec.handle, q, dec.kv[0], no_logits, out) == N.FASTOCR_ERR_NULL
    no_logits.stride = 0
    assert status(N.fastocr_evict, dec.handle, dec.kv[0], no_logits, 4, 1) == N.FASTOCR_ERR_INVALID
    assert status(N.fastocr_rows_workspace, dec.handle, -1) == N.FASTOCR_ERR_INVALID
    assert status(N.fastocr_rows_workspace, dec.handle, 1 << 40) == N.FASTOCR_ERR_INVALID
    ca = CrossAttention(c.k[None], c.v[None], c.gpu_table(), 20, q_heads=4, max_rows=1)
    qs = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
    with pytest.raises(N.FastOCRError):      # more rows than the workspace is for
        ca.attend(0, q, qs, out)
    for args in ((q.float(), qs, out), (q, qs.long(), out), (q, qs[:3], out), (q, qs.cpu(), out),
                 (q, qs, out[:2]), (q.transpose(0, 1), qs, out.transpose(0, 1))):
        with pytest.raises(ValueError):
            ca.attend(0, *args)
    ca.attend(0, q[:0], torch.zeros(4, dtype=torch.int32, device="cuda"), out[:0])
    torch.cuda.synchronize()
    assert (out == 7.0).all() and dec.device_status() == 0 and ca.device_status() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_large_logits_and_a_rising_max(dtype):
    """Logits of hundreds that rise from tile to tile: the row's base has to move; and a first tile
    far above the rest."""
    heads = (2, 1, 64)
    from dynamic_sparse_kv_gb300 import CrossAttention
    n = 700
    for order in (1.0, -1.0):
        c, start, q = cross_case([3, 200], [n, n], heads, 16, dtype, 81)
        q[:] = 4.0
        level = order * torch.linspace(-20, 20, n)     # logit = 4 * 64 * level / 8 up to 640
        for b in range(2):
            r = torch.arange(n)
            rows = torch.full((n, 64), 1.0) * level[:, None] + 0.01 * torch.randn(n, 64)
            c.k[c.table[b][r // 16].long(), 0, r % 16] = rows.to(dtype).cuda()
        ca = CrossAttention(c.k[None], c.v[None], c.gpu_table(), n, q_heads=2)
        out = torch.full_like(q, 7.0)
        ca.attend(0, q, start, out)
        check_cross(c, [3, 200], [n, n], q, out)


def test_rows_past_4_gib():
    """Cache offsets that need more than 32 bits: shared prefix, weights and eviction."""
    hkv, page, d = 4, 16, 128
    pages = (5 << 30) // (hkv * page * d * 2)
    k = torch.empty(1, pages, hkv, page, d, dtype=BF, device="cuda")
    v = torch.empty_like(k)
    g = torch.Generator().manual_seed(3)
    cols = 12
    table = (pages - 1 - torch.randperm(2 * cols, generator=g)).to(torch.int32).view(2, cols)
    for x in (k, v):
        x[0, pages - 2 * cols:] = torch.randn(2 * cols, hkv, page, d, generator=g).to(BF).cuda()
    from dynamic_sparse_kv_gb300 import DecodeAttention
    dec = DecodeAttention(k, v, table, q_heads=8)
    n = [180, 170]
    dec.set_seq_len(torch.tensor(n, dtype=torch.int32, device="cuda"))
    dec.share_prefix([0, 2], 130)
    dec.track_weights(60, 130)

    class Cache:
        pass
    c = Cache()
    c.page, c.table = page, table - (pages - 2 * cols)
    c.k, c.v = k[0, pages - 2 * cols:], v[0, pages - 2 * cols:]
    c.rows = lambda b, lo, hi: Paged.rows(c, b, lo, hi)
    q = torch.randn(2, 8, d, generator=g).to(BF).cuda()
    out = torch.full_like(q, float("nan"))
    dec.shared_layer(0, q, out)
    check_shared(c, [0, 2], [130, 130], n, q, out)
    k0, v0 = c.k.clone(), c.v.clone()
    mass0, pos0 = dec.weights["mass"][0].cpu(), dec.weights["pos"][0].cpu()
    new_len = torch.zeros(2, dtype=torch.int32, device="cuda")
    dec.evict_layer(0, 20, 5, new_len)
    check_evict(c, k0, v0, n, mass0, pos0, n, [130, 130], 20, 5, dec, new_len)
    assert dec.device_status() == 0


def test_weights_are_part_of_a_checkpoint():
    heads = (4, 2, 64)
    c, _, _, n, q = shared_case([2], [0], [30, 21], heads, 16, BF, 91)
    out = torch.empty_like(q)
    dec = decoder(c, n, 4)
    dec.track_weights(40, 0)
    dec.weigh_layer(0, q, out)
    st = dec.state_dict()
    other = decoder(c, n, 4)
    with pytest.raises(ValueError):
        other.load_state_dict(st)
    other.track_weights(40, 0)
    other.load_state_dict(st)
    for x in ("mass", "pos", "seen", "protect"):
        assert torch.equal(other.weights[x], dec.weights[x])
    for d in (dec, other):
        d.weigh_layer(0, q, out)
    assert torch.equal(other.weights["mass"], dec.weights["mass"])


def test_weighed_step_captured():
    """A replay adds the step's weights once."""
    from dynamic_sparse_kv_gb300 import CapturedStep
    heads = (6, 2, 64)
    c, _, _, n, q = shared_case([3], [0], [90, 21, 300], heads, 16, BF, 95)
    runs = []
    for graph in (False, True):
        dec = decoder(c, n, 6)
        dec.track_weights(300, 0)
        out = torch.empty_like(q)[None]
        if graph:
            step = CapturedStep(dec, "weighed")
            assert step.launches == 1
            dec.weights["mass"].zero_()
            step.q.copy_(q[None])
            step.replay()
            step.replay()
        else:
            dec.weighed_step(q[None], out)
            dec.weighed_step(q[None], out)
        runs.append((dec.weights["mass"].clone(), dec.weights["pos"].clone()))
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("batch", [33, 700])
def test_many_groups(dtype, batch):
    """More groups than a warp's lanes and than a CTA's threads, empty ones among them."""
    heads = (4, 2, 64)
    g = np.random.default_rng(batch)
    sizes = [int(x) for x in g.integers(0, 3, batch)]
    sizes = [x for x in sizes if x] or [1]
    prefixes = [int(x) for x in g.integers(0, 300, len(sizes))]
    tails = [int(x) for x in g.integers(1, 20, sum(sizes))]
    c, start, prefix, n, q = shared_case(sizes, prefixes, tails, heads, 16, dtype, batch)
    dec = decoder(c, n, 4)
    dec.share_prefix(start, torch.tensor(prefix))
    dec.groups["ws"].fill_(127)
    out = torch.full_like(q, float("nan"))
    dec.shared_layer(0, q, out)
    some = sorted(set([0, 1, len(sizes) - 1] + [int(x) for x in g.integers(0, len(sizes), 12)]))
    for i in some:
        for b in range(start[i], start[i + 1]):
            K0, V0 = c.rows(start[i], 0, prefix[b])
            K1, V1 = c.rows(b, prefix[b], n[b])
            check_out(out[b:b + 1], np64(q[b:b + 1]), np.concatenate([K0, K1]), np.concatenate([V0, V1]),
                      dtype, f"sequence {b}")
    assert torch.isfinite(out.float()).all() and dec.device_status() == 0
    from dynamic_sparse_kv_gb300 import CrossAttention
    t = [int(x) for x in g.integers(0, 4, len(n))]
    cs = torch.from_numpy(np.concatenate([[0], np.cumsum(t)]).astype(np.int32)).cuda()
    qx = (2 * torch.randn(sum(t), 4, 64, generator=torch.Generator().manual_seed(1))).to(dtype).cuda()
    ca = CrossAttention(c.k[None], c.v[None], c.gpu_table(), torch.tensor(n), q_heads=4)
    ox = torch.full_like(qx, 7.0)
    ca.attend(0, qx, cs, ox)
    at = np.concatenate([[0], np.cumsum(t)])
    for b in some:
        if t[b]:
            K, V = c.rows(b, 0, n[b])
            check_out(ox[at[b]:at[b + 1]], np64(qx[at[b]:at[b + 1]]), K, V, dtype, f"cross {b}")
    assert torch.isfinite(ox.float()).all() and ca.device_status() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("batch", [5, 70, 700])
def test_disordered_offsets_leave_rows_alone(dtype, batch):
    """Offsets that run back and forth: every other group would have all rows."""
    from dynamic_sparse_kv_gb300 import CrossAttention, _native as N
    c, _, prefix, n, q = shared_case([1] * batch, [20] * batch, [3] * batch, (4, 2, 64), 16, dtype, batch)
    zigzag = torch.tensor([0, batch] * (batch // 2 + 1), dtype=torch.int32, device="cuda")[:batch + 1].contiguous()
    dec = decoder(c, n, 4)
    dec.share_prefix(zigzag, torch.tensor(prefix), max_prefix=20)
    dec.groups["ws"].fill_(255)
    dec.shared_layer(0, q, torch.empty_like(q))
    assert dec.device_status() == N.DEV_BAD_GROUP
    dec.share_prefix(list(range(batch + 1)), torch.tensor(prefix))   # and a good call after it
    out = torch.full_like(q, float("nan"))
    dec.shared_layer(0, q, out)
    assert torch.isfinite(out.float()).all() and dec.device_status() == 0
    qx = torch.cat([q, q])
    back = torch.tensor([0, 2 * batch] * (batch // 2 + 1), dtype=torch.int32, device="cuda")[:batch + 1].contiguous()
    ca = CrossAttention(c.k[None], c.v[None], c.gpu_table(), torch.tensor(n), q_heads=4)
    ox = torch.full_like(qx, 7.0)
    ca.attend(0, qx, back, ox)
    assert ca.device_status() == N.DEV_BAD_GROUP and (ox == 7.0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [4, 90])
def test_cross_attention_captured(dtype, rows):
    """A replay follows lengths, offsets, queries and states that changed on the device; 4 rows for
    4 sequences take the form for single tokens too."""
    from dynamic_sparse_kv_gb300 import CrossAttention
    heads = (4, 2, 64)
    g = np.random.default_rng(rows)
    c = Paged(4, 400, heads[1], heads[2], 16, dtype, rows)
    n = torch.zeros(4, dtype=torch.int32, device="cuda")
    qs = torch.zeros(5, dtype=torch.int32, device="cuda")
    q = torch.zeros(rows, 4, 64, dtype=dtype, device="cuda")
    out = torch.empty_like(q)
    ca = CrossAttention(c.k[None], c.v[None], c.gpu_table(), n, q_heads=4, max_rows=rows)
    ca.attend(0, q, qs, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ca.attend(0, q, qs, out)
    for step in range(4):
        t = [1] * 4 if step == 0 and rows == 4 else [int(x) for x in g.multinomial(rows, [0.25] * 4)]
        lens = [int(x) for x in g.integers(0, 400, 4)]
        n.copy_(torch.tensor(lens, dtype=torch.int32))
        qs.copy_(torch.from_numpy(np.concatenate([[0], np.cumsum(t)]).astype(np.int32)))
        q.copy_(torch.randn(rows, 4, 64, generator=torch.Generator().manual_seed(step)).to(dtype))
        out.fill_(float("nan"))
        graph.replay()
        check_cross(c, t, lens, q, out, spare=0)
        assert ca.device_status() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("page,t,n", [
    (16, [1, 1, 1, 1, 1], [700, 0, 1, 333, 128]),
    (1, [0, 2, 0, 1], [5, 300, 7, 129]),
    (256, [0, 0, 0, 3], [1, 1, 1, 513]),
    (4, [1] + [0] * 39 + [30] + [0] * 30, [9] * 40 + [257] + [3] * 30),
    (16, [0, 0], [20, 30]),
])
def test_cross_attention_of_no_more_tokens_than_sequences(dtype, heads, page, t, n):
    from dynamic_sparse_kv_gb300 import CrossAttention
    spare = len(t) - sum(t)
    c, start, q = cross_case(t, n, heads, page, dtype, 22, spare)
    ca = CrossAttention(c.k[None], c.v[None], c.gpu_table(), torch.tensor(n), q_heads=heads[0])
    out = torch.full_like(q, 7.0)
    ca.attend(0, q, start, out)
    check_cross(c, t, n, q, out, spare)
    assert ca.device_status() == 0


def test_captured_step_keeps_its_groups_and_weights():
    """share_prefix and track_weights again after a capture: the graph's own tensors stay alive."""
    from dynamic_sparse_kv_gb300 import CapturedStep
    heads = (4, 2, 64)
    c, start, prefix, n, q = shared_case([2, 1], [64, 20], [9, 11, 20], heads, 16, BF, 51)
    dec = decoder(c, n, 4)
    dec.share_prefix(start, torch.tensor(prefix))
    dec.track_weights(64, torch.tensor(prefix))
    step = CapturedStep(dec, "shared")
    old = dec.weights["mass"]
    dec.share_prefix([0, 1, 2, 3], 0)
    dec.track_weights(256, 0)
    junk = [torch.full((1 << 12,), -1, dtype=torch.int32, device="cuda") for _ in range(64)]
    old.zero_()
    step.q.copy_(q[None])
    step.replay()
    torch.cuda.synchronize()
    check_shared(c, start, prefix, n, q, step.out[0])
    assert old.sum() > 0 and dec.weights["mass"].sum() == 0
    assert all((x == -1).all() for x in junk) and dec.device_status() == 0
