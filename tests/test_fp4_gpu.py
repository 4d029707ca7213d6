"""Attention over a cache held in 4 bits against 64 bits, in every mode that reads it."""
import numpy as np
import pytest
import torch

import oracle.attention as A
from cache_harness import Fp4Paged, check_out4, logit_bound
from gpu_harness import check_selection
from rows_harness import np64

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
HEADS = [(28, 4, 128), (10, 10, 128), (4, 2, 64), (8, 1, 64), (15, 3, 128)]


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def queries(b, hq, d, seed, size=2.0):
    g = torch.Generator().manual_seed(seed)
    return (size * torch.randn(b, hq, d, generator=g)).to(BF).cuda()


def check(c, q, out, rows=None):
    """rows(b): positions that sequence b attends to (None: all)."""
    for b, (K, V) in enumerate(c.rows):
        at = slice(None) if rows is None else np.asarray(rows(b), dtype=int)
        check_out4(out[b:b + 1], np64(q[b:b + 1]), K[at], V[at], f"sequence {b}")


@pytest.mark.parametrize("splits", [0, 1, 2, 7, 16])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("page,n", [(16, [1, 16, 17, 130, 2000]), (1, [33, 7]), (256, [300, 256]), (4, [63])])
def test_full(heads, page, n, splits):
    hq, hkv, d = heads
    c = Fp4Paged(n, hkv, d, page, 1)
    dec = c.decoder(hq, splits={0: splits})
    q = queries(len(n), hq, d, 2)
    out = torch.full_like(q, float("nan"))
    dec.dense_step(q[None], out[None])
    check(c, q, out)
    assert dec.device_status() == 0


@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("heads", [(28, 4, 128), (4, 2, 64)])
@pytest.mark.parametrize("prefix,window", [(0, 5), (40, 1), (40, 0), (33, 64), (5000, 8), (0, 1)])
def test_rswa(heads, prefix, window, splits):
    hq, hkv, d = heads
    n = [1, 40, 41, 700]
    c = Fp4Paged(n, hkv, d, 16, 3)
    dec = c.decoder(hq, splits={2: splits}, rswa_prefix=prefix, rswa_window=window)
    q = queries(len(n), hq, d, 4)
    out = torch.full_like(q, float("nan"))
    dec.rswa_step(q[None], out[None])
    check(c, q, out, lambda b: [r for r in range(n[b]) if r < prefix or r >= max(prefix, n[b] - window)])


@pytest.mark.parametrize("flags", [0, 1, 2])
@pytest.mark.parametrize("heads", [(28, 4, 128), (8, 1, 64)])
def test_gather(heads, flags):
    from dynamic_sparse_kv_gb300 import _native as N
    hq, hkv, d = heads
    n = [400, 37, 900, 65]
    img = [(20, 300), (0, 37), (100, 700), (64, 0)]
    kept = [100, 1, 0, 0]
    c = Fp4Paged(n, hkv, d, 16, 5)
    dec = c.decoder(hq, img_range=torch.tensor(img), max_img=700)
    g = torch.Generator().manual_seed(6)
    idx = torch.full((4, 128), -5, dtype=torch.int32)
    for b in range(4):
        idx[b, :kept[b]] = img[b][0] + torch.randperm(max(img[b][1], 1), generator=g)[:kept[b]].to(torch.int32)
    q = queries(4, hq, d, 7)
    out = torch.full_like(q, float("nan"))
    k = torch.tensor(kept, dtype=torch.int32, device="cuda")
    gpu_idx = idx.cuda()
    torch.cuda.synchronize()
    N.fastocr_sparse_attend_ex(dec.handle, q, dec.kv[0], dec.img_range, gpu_idx, 128, k, out, flags)
    check(c, q, out, lambda b: list(range(img[b][0])) + idx[b, :kept[b]].tolist()
          + list(range(sum(img[b]), n[b])))
    assert dec.device_status() == 0


@pytest.mark.parametrize("splits", [0, 1])
def test_gather_of_a_list_in_several_rounds(splits):
    from dynamic_sparse_kv_gb300 import _native as N
    hq, hkv, d, n, kept = 8, 1, 64, 6100, 4600
    c = Fp4Paged([n], hkv, d, 16, 26)
    dec = c.decoder(hq, img_range=torch.tensor([[700, 5000]]), max_img=5000, splits={1: splits})
    idx = 700 + torch.randperm(5000, generator=torch.Generator().manual_seed(27))[:kept].to(torch.int32)
    q = queries(1, hq, d, 28)
    out = torch.full_like(q, float("nan"))
    N.fastocr_sparse_attend(dec.handle, q, dec.kv[0], dec.img_range, idx.cuda()[None], kept,
                            torch.full((1,), kept, dtype=torch.int32, device="cuda"), out)
    check(c, q, out, lambda b: [*range(700), *idx.tolist(), *range(5700, n)])
    assert dec.device_status() == 0


def test_steps_of_a_stack_hand_the_selection_on():
    """Three layers, the middle one focal: the last gathers its selection, the first the one of
    the step before (staged early, and found to be another when it is)."""
    from dynamic_sparse_kv_gb300 import DecodeAttention, Fp4Cache
    hq, hkv, d, n, start, n_img, tau = 28, 4, 128, 700, 30, 512, 0.1
    c = Fp4Paged([n, n], hkv, d, 16, 29)
    caches = []
    for w in range(2):
        p = c.codes[w].shape[0]
        x = Fp4Cache(3, p, hkv, 16, d, gain=torch.from_numpy(c.gain[w]).expand(3, -1), device="cuda")
        x.codes.copy_(torch.from_numpy(c.codes[w]).expand(3, -1, -1, -1, -1))
        x.scales.view(torch.uint8).copy_(torch.from_numpy(c.scales[w]).expand(3, -1, -1, -1, -1))
        caches.append(x)
    dec = DecodeAttention(*caches, c.table.cuda(), q_heads=hq, img_range=torch.tensor([[start, n_img]] * 2),
                          max_img=n_img, tau=tau)
    dec.set_focal_layers([1])
    last = None
    for t in range(4):
        dec.set_seq_len(n - 3 + t)
        q = torch.stack([queries(2, hq, d, 30 + 3 * t + l) for l in range(3)])
        out = torch.full_like(q, float("nan"))
        dec.step(q, out)
        sel = [dec.sel[1][0][b, :int(dec.sel[1][1][b])].tolist() for b in range(2)]
        text = [*range(start), *range(start + n_img, n - 3 + t)]
        every = list(range(n - 3 + t))
        check(c, q[0], out[0], lambda b: every if last is None else text + last[b])
        check(c, q[1], out[1], lambda b: every)
        check(c, q[2], out[2], lambda b: text + sel[b])
        last = sel
    assert dec.device_status() == 0


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("splits", [0, 1, 5])
def test_focal_selection_scores_and_profile(heads, splits):
    from dynamic_sparse_kv_gb300 import _native as N
    hq, hkv, d = heads
    n, start, n_img, tau = [333, 290], 21, 256, 0.1
    c = Fp4Paged(n, hkv, d, 16, 8)
    dec = c.decoder(hq, img_range=torch.tensor([[start, n_img]] * 2), max_img=n_img, tau=tau, splits={0: splits})
    dec.set_focal_layers([0])
    q = queries(2, hq, d, 9)
    out = torch.full_like(q, float("nan"))
    dec.step(q[None], out[None])
    check(c, q, out)
    sigma = torch.full((2, n_img), -1.0, device="cuda")
    N.fastocr_focal_scores(dec.handle, q, dec.kv[0], dec.img_range, out, sigma, n_img)
    N.fastocr_profiler_reset(dec.handle)
    N.fastocr_profile_attend(dec.handle, q, dec.kv[0], dec.img_range, out, 0)
    mass = N.fastocr_profiler_read(dec.handle, 1)[0]
    idx, k = dec.sel[0]
    want, slack = 0.0, 0.0
    for b, (K, V) in enumerate(c.rows):
        qb = np64(q[b])
        _, sel, s = A.focal_attend(qb, K, V, n[b], start, n_img, tau)
        check_selection(idx[b, :int(k[b])].cpu().numpy(), sel, s, start, f"sequence {b}")
        bound = logit_bound(qb[None], K).max()
        assert np.all(np.abs(np64(sigma[b]) - s) <= 2 * bound * s + hq * 2.0 ** -30)
        want += s.sum()
        slack += 2 * bound * s.sum() + hq * 2.0 ** -20
    assert abs(mass - want) <= slack
    assert dec.device_status() == 0


def test_large_logits_and_one_key_that_wins():
    hq, hkv, d = 28, 4, 128
    c = Fp4Paged([700, 5], hkv, d, 16, 10)
    K = c.rows[0][0]
    q = torch.zeros(2, hq, d)
    for h in range(hq):
        q[0, h] = torch.from_numpy(K[601, h // 7]) * 40      # logits of several thousand
        q[1, h] = 1e-30
    q = q.to(BF).cuda()
    out = torch.full_like(q, float("nan"))
    c.decoder(hq).dense_step(q[None], out[None])
    check(c, q, out)


@pytest.mark.parametrize("big", [2.0 ** 126, 2.0 ** -126, 0.0])
def test_queries_at_the_ends_of_their_range(big):
    hq, hkv, d = 8, 2, 64
    c = Fp4Paged([50], hkv, d, 16, 11, kv=lambda b, w, m: torch.full((m, hkv, d), 2.0 ** -5 if w == 0 else 1.5))
    q = torch.full((1, hq, d), big).to(BF).cuda()
    q[:, :, 1::2] *= -1          # the logits cancel
    out = torch.full_like(q, float("nan"))
    c.decoder(hq).dense_step(q[None], out[None])
    check(c, q, out)


def test_a_group_of_nan_reaches_those_that_attend_to_it_alone():
    hq, hkv, d = 4, 2, 64
    c = Fp4Paged([40, 40], hkv, d, 16, 12)
    at = int(c.table[1, 1]), 0, 3                           # row 19 of sequence 1, KV head 0
    c.scales[1][at[0], at[1], at[2], 2] = 0x7f
    q = queries(2, hq, d, 13)
    out = torch.zeros_like(q)
    c.decoder(hq).dense_step(q[None], out[None])
    bad = torch.isnan(out)
    assert bad[1, :2, 32:48].all() and int(bad.sum()) == 2 * 16
    check_out4(out[:1], np64(q[:1]), *c.rows[0])


def test_pages_out_of_range_are_masked_and_reported():
    from dynamic_sparse_kv_gb300 import _native as N
    hq, hkv, d = 4, 2, 64
    c = Fp4Paged([100, 64], hkv, d, 16, 14)
    good = c.table.clone()
    c.table[0, 2], c.table[1, 0] = 10 ** 6, -1
    dec = c.decoder(hq)
    q = queries(2, hq, d, 15)
    out = torch.full_like(q, float("nan"))
    dec.dense_step(q[None], out[None])
    c.table = good
    check(c, q, out, lambda b: [r for r in range(c.n[b]) if not ((b, r // 16) in ((0, 2), (1, 0)))])
    assert dec.device_status() == N.DEV_BAD_PAGE


def test_a_cache_past_4_gib():
    from dynamic_sparse_kv_gb300 import DecodeAttention, Fp4Cache
    hq, hkv, d, page, pages = 8, 8, 128, 256, 33000
    c = Fp4Paged([300], hkv, d, page, 23)
    caches = [Fp4Cache(1, pages, hkv, page, d, device="cuda", gain=torch.from_numpy(g)[None]) for g in c.gain]
    assert caches[0].codes.numel() > 2 ** 32
    table = torch.tensor([[0, pages - 1]], dtype=torch.int32)
    for w, x in enumerate(caches):
        for i, at in enumerate(c.table[0].tolist()):
            x.codes[0, table[0, i]].copy_(torch.from_numpy(c.codes[w][at]))
            x.scales.view(torch.uint8)[0, table[0, i]].copy_(torch.from_numpy(c.scales[w][at]))
    dec = DecodeAttention(*caches, table.cuda(), q_heads=hq)
    q = queries(1, hq, d, 24)
    out = torch.full_like(q, float("nan"))
    idx, k = torch.tensor([[299, 3, 260, 17]], dtype=torch.int32, device="cuda"), torch.full((1,), 4, dtype=torch.int32, device="cuda")
    img = torch.tensor([[0, 300]], dtype=torch.int32, device="cuda")
    dec.set_seq_len(300)
    dec.dense_step(q[None], out[None])
    check(c, q, out)
    from dynamic_sparse_kv_gb300 import fastocr_sparse_attend
    fastocr_sparse_attend(dec.handle, q, dec.kv[0], img, idx, 4, k, out)
    check(c, q, out, lambda b: idx[0].tolist())


def test_logits_of_any_size():
    """Logits far below any that a first running maximum could be taken for."""
    hq, hkv, d = 4, 2, 64
    c = Fp4Paged([40], hkv, d, 16, 25, kv=lambda b, w, m: torch.full((m, hkv, d), 2.0) if w == 0
                 else torch.arange(m * hkv * d).view(m, hkv, d) % 7 - 3.0)
    q = torch.full((1, hq, d), -2.0 ** 110).to(BF).cuda()      # every logit near -2^114: one value, no spread
    out = torch.full_like(q, float("nan"))
    c.decoder(hq).dense_step(q[None], out[None])
    want = c.rows[0][1].mean(0).repeat(hq // hkv, 0)
    assert np.abs(np64(out[0]) - want).max() <= (2.0 ** -8 + 2.0 ** -10) * 3


def test_captured_steps_replay_on_other_lengths_and_codes():
    from dynamic_sparse_kv_gb300 import CapturedStep
    hq, hkv, d = 28, 4, 128
    c = Fp4Paged([300, 90], hkv, d, 16, 16)
    dec = c.decoder(hq)
    steps = [CapturedStep(dec, "dense"), CapturedStep(dec, "dense")]
    other = Fp4Paged([17, 280], hkv, d, 16, 17, cap=300)
    other.table = c.table
    for s, cc in ((steps[0], c), (steps[1], c)):
        s.q.copy_(queries(2, hq, d, 18)[None])
        s.replay()
        check(cc, s.q[0], s.out[0])
    dec.set_seq_len(torch.tensor([17, 5], dtype=torch.int32, device="cuda"))
    steps[0].replay()
    for b, n in enumerate((17, 5)):
        check_out4(steps[0].out[0][b:b + 1], np64(steps[0].q[0][b:b + 1]), c.rows[b][0][:n], c.rows[b][1][:n])


def test_on_a_stream_of_its_own():
    hq, hkv, d = 28, 4, 128
    c = Fp4Paged([500, 90], hkv, d, 16, 19)
    dec = c.decoder(hq)
    q = queries(2, hq, d, 20)
    out = torch.full_like(q, float("nan"))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    dec.dense_step(q[None], out[None], stream=s)
    s.synchronize()
    check(c, q, out)


def test_calls_that_4_bits_do_not_have_are_refused():
    from dynamic_sparse_kv_gb300 import CrossAttention
    from dynamic_sparse_kv_gb300 import _native as N
    hq, hkv, d = 4, 2, 64
    c = Fp4Paged([40], hkv, d, 16, 21)
    dec = c.decoder(hq)
    q = queries(1, hq, d, 22)
    with pytest.raises(ValueError, match="4 bits"):
        dec.share_prefix([0, 1], 10)
    with pytest.raises(ValueError, match="4 bits"):
        dec.track_weights(10, 5)
    with pytest.raises(ValueError, match="4 bits"):
        CrossAttention(*c.caches(), c.table, 40, q_heads=hq)
    ints = torch.zeros(64, dtype=torch.int32, device="cuda")
    floats = torch.zeros(1, hkv, 8, 8, device="cuda")
    w = N.make_weights(floats[..., 0].contiguous(), ints.view(1, 1, 64), ints, ints, floats)
    start = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for call in (lambda: N.fastocr_weigh_attend(dec.handle, q, dec.kv[0], w, q),
                 lambda: N.fastocr_evict(dec.handle, dec.kv[0], w, 4, 1),
                 lambda: N.fastocr_shared_attend(dec.handle, q, dec.kv[0], N.make_groups(start, ints), q, ints, 256),
                 lambda: N.fastocr_cross_attend(dec.handle, q, dec.kv[0], start, 1, q, ints, 256)):
        with pytest.raises(N.FastOCRError) as e:
            call()
        assert e.value.status == N.FASTOCR_ERR_UNSUPPORTED
    kv = N.make_kv(*(x[0] for x in c.caches()), dec.block_table, dec.seq_len)
    kv.k_gain = None
    with pytest.raises(N.FastOCRError) as e:
        N.fastocr_full_attend(dec.handle, q, kv, q)
    assert e.value.status == N.FASTOCR_ERR_NULL
    with pytest.raises(N.FastOCRError) as e:
        N.fastocr_set_variant(dec.handle, 0, N.VARIANT_DEEP)
    assert e.value.status == N.FASTOCR_ERR_UNSUPPORTED
