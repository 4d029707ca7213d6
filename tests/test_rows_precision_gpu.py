"""Outputs of the split-K forms of the row operators in bf16: their probabilities reach the second
product within 2^-16, so an output is off by its own rounding and fp32 arithmetic only."""
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
    """As rows_harness.check_out without the rounding of the probabilities: two parts leave 2^-8 of
    2^-8 of each, and the sums have twice as many terms."""
    out, _, mag = R.attend_all(q, K, V)
    c = prob_bound(q, K, q.shape[-1])
    tol = (c + 2.0 ** -16 + 2 * K.shape[0] * 2.0 ** -24)[..., None] * mag + U[BF] * np.abs(out)
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
def test_own_rows_of_a_shared_prefix_call(heads):
    """Without a prefix all rows are the tail kernel's."""
    c, start, prefix, n, q = shared_case([2, 1], [0, 0], [700, 33, 2100], heads, 16, BF, 4)
    dec = decoder(c, n, heads[0])
    dec.share_prefix(start, torch.tensor(prefix))
    out = torch.empty_like(q)
    dec.shared_layer(0, q, out)
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
