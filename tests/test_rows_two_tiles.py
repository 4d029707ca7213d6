"""The bf16 row kernel with two row tiles a CTA, an item of 129 to 256 rows: taken only where the
expected work is large, so the expected lengths are made long (a wide block table, or max_prefix)
and the real ones stay small. The CPU test shows that every case takes that form."""
import numpy as np
import pytest
import torch

from rows_harness import check_out, np64
from test_rows_gpu import check_shared, cross_case, decoder, shared_case
from test_rows_plan import BF16, plan  # noqa: F401  (a fixture)

BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _device(request):
    if request.node.get_closest_marker("gpu") and not torch.cuda.is_available():
        pytest.skip("no CUDA device")


WIDE = 16384     # tokens that the block tables have room for


def ragged(seed, count, lo, hi):
    return [int(x) for x in np.random.default_rng(seed).integers(lo, hi + 1, count)]


# heads (H_q, H_kv, d), page, query tokens and states of the sequences
CROSS = {
    # uncut items next to whole ones of one row tile, of no rows and of one key
    "g7": ((28, 4, 128), 16, [36, 20, 40, 5, 0, 73], [700, 333, 129, 900, 50, 1]),
    "g7_d64": ((28, 4, 64), 16, [36, 18, 19, 37, 90, 1], [640, 128, 127, 513, 300, 900]),
    "g8_one_head": ((8, 1, 64), 16, [32, 33, 31, 64, 16, 17, 1, 100], [640, 128, 127, 1000, 513, 5, 300, 257]),
    "g1": ((10, 10, 128), 16, [256, 257, 129, 128, 130, 60], [300, 129, 257, 500, 64, 0]),
    "g1_d64": ((10, 10, 64), 1, [300, 129, 128], [130, 300, 64]),
    "g5": ((15, 3, 64), 256, [51, 52, 26, 25, 103], [700, 255, 256, 257, 0]),
    "g3": ((15, 5, 128), 8, [85, 86, 43, 42], [401, 128, 1, 384]),
    # items cut over CTAs, each with its share
    "shares": ((28, 4, 128), 16, [36, 40, 25], [4100, 3000, 2]),
    "shares_d64": ((8, 2, 64), 16, [64, 33, 40, 70], [4100, 2900, 129, 3500]),
    # more items than CTAs: segments of both forms in one CTA, cut at both ends
    "dealt": ((16, 2, 128), 4, ragged(1, 48, 9, 60), ragged(2, 48, 1, 700)),
    "dealt_d64": ((28, 4, 64), 16, ragged(3, 40, 9, 60), ragged(4, 40, 0, 700)),
}
# heads, page, sizes and prefixes of the groups
SHARED = {
    "few": ((28, 4, 128), 16, [40, 20, 1, 30], [700, 300, 130, 2000]),
    "few_d64": ((8, 2, 64), 16, [33, 0, 70, 17], [513, 5, 1500, 128]),
    "dealt": ((15, 3, 64), 16, ragged(5, 30, 20, 51), ragged(6, 30, 0, 190)),
}


def tails(sizes):
    return [1 + (11 * i) % 40 for i in range(sum(sizes))]


def test_the_cases_take_two_row_tiles(plan):  # noqa: F811
    for heads, page, t, n in CROSS.values():
        g = heads[0] // heads[1]
        got = plan((len(t), *heads, BF16, WIDE // page, page), [f"t {sum(t)} {len(t)} 0"])[0][0]
        assert got == 256 // g and 128 < max(min(x, got) for x in t) * g, (heads, t)
    for heads, page, sizes, prefixes in SHARED.values():
        g = heads[0] // heads[1]
        got = plan((sum(sizes), *heads, BF16, WIDE // page, page), [f"t {sum(sizes)} {len(sizes)} {WIDE}"])[0][0]
        assert got == 256 // g and 128 < max(min(x, got) for x in sizes) * g, (heads, sizes)
    assert plan((2, 2, 1, 64, BF16, 4 * WIDE // 16, 16), ["t 303 2 0"])[0][0] == 128   # the large logits below


def wide_cross(c, n, q_heads, wide=WIDE):
    """A handle that expects long states; their real lengths are on the device."""
    from dynamic_sparse_kv_gb300 import CrossAttention
    table = torch.nn.functional.pad(c.gpu_table(), (0, wide // c.page - c.table.shape[1]), value=-1)
    ca = CrossAttention(c.k[None], c.v[None], table, torch.tensor(n, dtype=torch.int32, device="cuda"),
                        q_heads=q_heads)
    ca.ws.fill_(127)
    return ca


def check_cross(c, t, n, q, out):
    at = 0
    for b in range(len(n)):
        if t[b]:
            K, V = c.rows(b, 0, n[b])
            check_out(out[at:at + t[b]], np64(q[at:at + t[b]]), K, V, q.dtype, f"sequence {b}")
        at += t[b]
    assert (out[at:].float() == 7.0).all(), "rows behind the last sequence were written"


@pytest.mark.gpu
@pytest.mark.parametrize("case", CROSS)
def test_cross_attention(case):
    heads, page, t, n = CROSS[case]
    c, start, q = cross_case(t, n, heads, page, BF, 23)
    ca = wide_cross(c, n, heads[0])
    out = torch.full_like(q, 7.0)
    ca.attend(0, q, start, out)
    again = torch.full_like(q, 7.0)              # the same again, bit for bit, on the workspace it left
    ca.attend(0, q, start, again)
    assert torch.equal(out, again) and ca.device_status() == 0
    c.k, c.v = c.k.cpu(), c.v.cpu()              # read once for all sequences
    check_cross(c, t, n, q, out)
    ca.close()


@pytest.mark.gpu
@pytest.mark.parametrize("case", SHARED)
@pytest.mark.parametrize("weigh", [False, True])
def test_shared_prefix(case, weigh):
    heads, page, sizes, prefixes = SHARED[case]
    c, start, prefix, n, q = shared_case(sizes, prefixes, tails(sizes), heads, page, BF, 24)
    dec = decoder(c, n, heads[0])
    dec.share_prefix(start, torch.tensor(prefix), max_prefix=WIDE)
    dec.groups["ws"].fill_(127)
    if weigh:
        dec.track_weights(40, torch.tensor(prefix))
    out = torch.full_like(q, float("nan"))
    dec.shared_layer(0, q, out)
    c.k, c.v = c.k.cpu(), c.v.cpu()              # read once for all sequences
    ps = check_shared(c, start, prefix, n, q, out)
    if weigh:                                    # every own row has its weight: the rest of 1 is the prefix's
        mass = np64(dec.weights["mass"][0])
        g = heads[0] // heads[1]
        for b, (p, cb) in enumerate(ps):
            own = p[0, :, prefix[b]:].reshape(heads[1], g, -1).sum(1)
            got = mass[b][:, :own.shape[1]]
            assert (np.abs(got - own) <= (cb.max() + 9 * 2.0 ** -24) * own + 2.0 ** -24).all(), b
            assert not mass[b][:, own.shape[1]:].any()
    assert dec.device_status() == 0
    dec.close()


@pytest.mark.gpu
@pytest.mark.parametrize("order", [1.0, -1.0])
def test_large_logits_and_a_rising_max(order):
    """Logits up to 640 that rise from tile to tile: each turn moves its own rows' base while the
    other goes on; and a first tile far above the rest."""
    n, t, heads = [700, 700], [3, 300], (2, 1, 64)
    c, start, q = cross_case(t, n, heads, 16, BF, 81)
    q[:] = 4.0
    q[5::3] = -4.0                               # every third row sees them fall
    level = order * torch.linspace(-20, 20, 700)
    for b in range(2):
        r = torch.arange(700)
        rows = torch.full((700, 64), 1.0) * level[:, None] + 0.01 * torch.randn(
            700, 64, generator=torch.Generator().manual_seed(b))
        c.k[c.table[b][r // 16].long(), 0, r % 16] = rows.to(BF).cuda()
    ca = wide_cross(c, n, 2, 4 * WIDE)
    out = torch.full_like(q, 7.0)
    ca.attend(0, q, start, out)
    check_cross(c, t, n, q, out)
    assert ca.device_status() == 0
