"""Sequences that the offsets of a shared-prefix call put into no group, on a workspace that an
earlier good call left: nothing of that call may come back."""
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
@pytest.mark.parametrize("batch", [6, 70, 600])     # groups for a warp's lanes, more, more than a CTA's threads
@pytest.mark.parametrize("kind", ["short", "late", "empty", "disordered"])
@pytest.mark.parametrize("weigh", [False, True])
def test_sequence_without_a_group_attends_to_its_own_rows(dtype, batch, kind, weigh):
    from dynamic_sparse_kv_gb300 import _native as N
    heads = (4, 2, 64)
    tails = [1 + (7 * b) % 23 for b in range(batch)]
    c, start, prefix, n, q = shared_case([1] * batch, [300 + b % 5 for b in range(batch)], tails, heads, 16,
                                         dtype, batch)
    dec = decoder(c, n, 4)
    dec.share_prefix(start, torch.tensor(prefix))
    out = torch.full_like(q, float("nan"))
    dec.shared_layer(0, 3 * q, out)                  # a good call: parts of every sequence, at other logits
    assert dec.device_status() == 0
    bad = list(range(batch + 1))
    if kind == "short":
        bad = [min(x, batch - 3) for x in bad]
        none = range(batch - 3, batch)
    elif kind == "late":
        bad[:3] = [2, 2, 2]
        none = range(0, 2)
    elif kind == "empty":
        bad = [batch] * (batch + 1)
        none = range(batch)
    else:
        bad[1], bad[2] = 4, 3
        none = range(batch)
    dec.share_prefix(torch.tensor(bad, dtype=torch.int32, device="cuda"), torch.tensor(prefix), max_prefix=304)
    mass0 = torch.rand(1, batch, 2, 32, generator=torch.Generator().manual_seed(3))
    if weigh:
        dec.track_weights(32, torch.tensor(prefix), mass=mass0.cuda())
    out.fill_(float("nan"))
    dec.shared_layer(0, q, out)
    assert dec.device_status() == N.DEV_BAD_GROUP
    none = set(none)
    for b in sorted(none)[:12] + sorted(none)[-3:]:
        K, V = c.rows(b, prefix[b], n[b])
        p, cb = check_out(out[b:b + 1], np64(q[b:b + 1]), K, V, dtype, f"sequence {b}")
        if weigh:
            full = np.zeros((4, n[b]))
            full[:, prefix[b]:] = p[0]
            want, _ = R.add_weights(np64(mass0[0, b]), np.zeros((2, 32), dtype=np.int64), full, n[b], prefix[b],
                                    n[b], 2)
            got = np64(dec.weights["mass"][0, b])
            assert (np.abs(got - want) <= (cb.max() + 9 * 2.0 ** -24) * np.abs(want) + 2.0 ** -24).all(), b
    for b in [x for x in range(batch) if x not in none][:6]:     # the others have their prefix
        K, V = c.rows(b, 0, n[b])
        check_out(out[b:b + 1], np64(q[b:b + 1]), K, V, dtype, f"sequence {b}")
    dec.close()
