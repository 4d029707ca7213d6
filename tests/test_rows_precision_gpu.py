"""Outputs of weighed attention and of single-token cross attention in bf16: their probabilities reach the second
product within 2^-15, so an output is off by its own rounding and fp32 arithmetic only."""
import numpy as np
import pytest
import torch

from oracle import rows as R
from rows_harness import U, np64, prob_bound
from test_rows_gpu import cross_case, decoder, shared_case

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def check_fine(got, q, K, V, where):
    """As rows_harness.check_out without the rounding of the probabilities. Their first part is cut
    off below 2^-7 of the value, the remainder rounded by 2^-8 of itself: 2^-15 of the value at
    most. The sums have twice as many terms."""
    out, _, mag = R.attend_all(q, K, V)
    c = prob_bound(q, K, q.shape[-1])
    tol = (c + 2.0 ** -15 + 2 * K.shape[0] * 2.0 ** -24)[..., None] * mag + U[BF] * np.abs(out)
    err = np.abs(np64(got) - out)
    assert (err <= tol).all(), f"{where}: error {err.max():.3g} is over its bound by {(err - tol).max():.3g}"


HEADS = [(28, 4, 128), (10, 10, 128), (8, 2, 64)]


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("splits", [0, 1, 5])
def test_weighed_attention(heads, splits):
    from dynamic_sparse_kv_gb300 import _native as N
    c, _, _, n, q = shared_case([3], [0], [700, 33, 2100], heads, 16, BF, 3)
    dec = decoder(c, n, heads[0])
    if splits:
        N.fastocr_set_splits(dec.handle, 0, splits)
    dec.track_weights(2100, 0)
    out = torch.empty_like(q)
    dec.weigh_layer(0, q, out)
    for b in range(3):
        check_fine(out[b:b + 1], np64(q[b:b + 1]), *c.rows(b, 0, n[b]), f"sequence {b}")
    dec.close()


@pytest.mark.parametrize("heads", HEADS)
def test_cross_attention_of_single_tokens(heads):
    from dynamic_sparse_kv_gb300 import CrossAttention
    t, n = [1, 2, 0, 1], [900, 1300, 50, 17]
    c, start, q = cross_case(t, n, heads, 16, BF, 5, 0)
    ca = CrossAttention(c.k[None], c.v[None], c.gpu_table(), torch.tensor(n), q_heads=heads[0])
    out = torch.empty_like(q)
    ca.attend(0, q, start, out)
    at = 0
    for b in range(4):
        if t[b]:
            check_fine(out[at:at + t[b]], np64(q[at:at + t[b]]), *c.rows(b, 0, n[b]), f"sequence {b}")
        at += t[b]
    ca.close()


@pytest.mark.parametrize("heads", HEADS)
def test_infinite_values_of_attended_rows_stay_infinite(heads):
    """Infinity times a probability is infinity, whatever the probability's parts; other dims are as before."""
    from dynamic_sparse_kv_gb300 import CrossAttention
    c, _, _, n, q = shared_case([2], [0], [150, 40], heads, 16, BF, 6)
    dec = decoder(c, n, heads[0])
    dec.track_weights(150, 0)
    start = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    ca = CrossAttention(c.k[None], c.v[None], c.gpu_table(), torch.tensor(n), q_heads=heads[0])
    outs = []
    for again in (False, True):
        if again:
            for b in range(2):
                for r, dim, x in ((0, 3, float("inf")), (17, 3, float("inf")), (n[b] - 1, 8, float("-inf")),
                                  (5, 20, float("inf")), (6, 20, float("-inf"))):
                    c.v[int(c.table[b, r // 16]), :, r % 16, dim] = x
        one, two = torch.empty_like(q), torch.empty_like(q)
        dec.weigh_layer(0, q, one)
        ca.attend(0, q, start, two)
        outs.append((one, two))
    for was, now in zip(*outs):
        assert (now[..., 3] == float("inf")).all() and (now[..., 8] == float("-inf")).all()
        assert now[..., 20].isnan().all()
        rest = [d for d in range(heads[2]) if d not in (3, 8, 20)]
        assert torch.equal(now[..., rest], was[..., rest])
    ca.close()
    dec.close()
