"""Rows of weighed attention whose page is out of range: they are left out of the
attention, and no weight may come from what the logit scratch held before."""
import numpy as np
import pytest
import torch

from oracle import rows as R
from rows_harness import check_out, np64
from test_rows_gpu import decoder, shared_case

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("heads", [(28, 4, 128), (4, 2, 64)])
@pytest.mark.parametrize("splits", [0, 1, 5])
@pytest.mark.parametrize("shared", [False, True])
def test_rows_of_a_bad_page_get_no_weight(dtype, heads, splits, shared):
    """Bad pages before and behind protect, under the current token, and past one round of a CTA's list."""
    from dynamic_sparse_kv_gb300 import _native as N
    hq, hkv, d = heads
    page, prefix_rows = 16, 48
    c, start, prefix, n, q = shared_case([4], [prefix_rows], [70, 41, 100, 1900], heads, page, dtype, 17)
    dec = decoder(c, n, hq)
    if splits:
        N.fastocr_set_splits(dec.handle, 0, splits)
    # sequence: its bad own pages
    bad = {0: [5], 1: [(n[1] - 1) // page], 2: [3, 8], 3: [4, (n[3] - 5) // page]}
    for b, js in bad.items():
        for i, j in enumerate(js):
            dec.block_table[b, j] = -1 if i else c.k.shape[0]
    protect = [48, 60, 64, 48]
    rows = max(x - p for x, p in zip(n, protect))
    g = torch.Generator().manual_seed(2)
    mass0 = torch.rand(1, 4, hkv, rows, generator=g)
    pos0 = torch.randint(0, 9, (1, 4, hkv, rows), generator=g, dtype=torch.int32)
    seen = torch.tensor([100, 50, 900, 2000], dtype=torch.int32, device="cuda")
    dec.track_weights(rows, torch.tensor(protect), mass=mass0.cuda(), pos=pos0.cuda(), seen=seen)
    dec.weights["logits"].fill_(1e30)            # 2^1e30: what is read of it shows
    out = torch.full_like(q, float("nan"))
    if shared:
        dec.share_prefix(start, torch.tensor(prefix))
        dec.shared_layer(0, q, out)
    else:
        dec.weigh_layer(0, q, out)
    assert dec.device_status() == N.DEV_BAD_PAGE
    mass, pos = np64(dec.weights["mass"][0]), dec.weights["pos"][0].cpu().numpy()
    for b in range(4):
        lead = 0 if shared else b
        K0, V0 = c.rows(lead, 0, prefix_rows)
        K1, V1 = c.rows(b, prefix_rows, n[b])
        K, V = np.concatenate([K0, K1]), np.concatenate([V0, V1])
        gone = [r for r in range(n[b]) if r // page in bad[b] and r >= (prefix_rows if shared else 0)]
        left = np.setdiff1d(np.arange(n[b]), gone)
        p, cb = check_out(out[b:b + 1], np64(q[b:b + 1]), K[left], V[left], dtype, f"sequence {b}")
        full = np.zeros((hq, n[b]))
        full[:, left] = p[0]
        want, wpos = R.add_weights(np64(mass0[0, b]), pos0[0, b].numpy(), full, n[b], protect[b],
                                   int(seen[b]), hkv)
        # a sum of g probabilities, then one addition
        tol = (cb.max() + 9 * 2.0 ** -24) * np.abs(want) + 2.0 ** -24
        assert (np.abs(mass[b] - want) <= tol).all(), b
        for r in gone:                           # exactly: nothing was added, the current token starts at 0
            i = r - protect[b]
            if i >= 0:
                assert np.array_equal(mass[b, :, i], np.zeros(hkv) if r == n[b] - 1 else np64(mass0[0, b, :, i]))
        assert np.array_equal(pos[b], wpos)
    dec.close()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("splits", [1, 5])
def test_image_rows_of_a_bad_page_score_nothing(dtype, splits):
    """A focal layer's scores come from stored logits too; an earlier call left larger ones behind."""
    from dynamic_sparse_kv_gb300 import DecodeAttention, _native as N
    heads = (8, 2, 64)
    c, _, _, n, q = shared_case([1], [0], [300], heads, 16, dtype, 19)
    img = torch.tensor([[20, 200]], dtype=torch.int32)
    dec = DecodeAttention(c.k[None], c.v[None], c.gpu_table(), q_heads=8, img_range=img, max_img=200)
    N.fastocr_set_splits(dec.handle, 0, splits)
    dec.set_seq_len(torch.tensor(n, dtype=torch.int32, device="cuda"))
    out, sigma = torch.empty_like(q), torch.full((1, 200), float("nan"), device="cuda")
    N.fastocr_focal_scores(dec.handle, 30 * q, dec.kv[0], dec.img_range, out, sigma, 200)
    for j in (1, 5, 13):                         # rows 16-31 (half of them image), 80-95, 208-223
        dec.block_table[0, j] = c.k.shape[0]
    N.fastocr_focal_scores(dec.handle, q, dec.kv[0], dec.img_range, out, sigma, 200)
    assert dec.device_status() == N.DEV_BAD_PAGE
    left = np.array([r for r in range(n[0]) if r // 16 not in (1, 5, 13)])
    K, V = c.rows(0, 0, n[0])
    p, cb = check_out(out, np64(q), K[left], V[left], dtype)
    want = np.zeros(n[0])
    want[left] = p[0].sum(0)
    want = want[20:220]
    got = np64(sigma[0])
    assert (np.abs(got - want) <= (cb.max() + 9 * 2.0 ** -24) * want + 2.0 ** -24).all()
    assert (got[want == 0] == 0).all()
    dec.close()
