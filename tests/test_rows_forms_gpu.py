"""Cross attention with no more query tokens than sequences, on both sides of the rule that
chooses between a token a unit and the row kernel; few tokens on a large handle."""
import numpy as np
import pytest
import torch

from rows_harness import check_out, np64
from test_rows_gpu import cross_case

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("heads", [(28, 4, 128), (4, 2, 64)])
@pytest.mark.parametrize("t", [[1] * 40, [0] * 39 + [40], [20, 0] * 2 + [0] * 36, [0] * 20 + [1] + [0] * 19])
@pytest.mark.parametrize("expected", [0, 300, 1 << 20])   # lengths unknown, known, and a wide table's
def test_cross_attention_on_both_sides_of_the_rule(dtype, heads, t, expected):
    from dynamic_sparse_kv_gb300 import CrossAttention
    r = np.random.default_rng(len(t) + sum(t))
    n = [int(x) for x in r.integers(0, 300, len(t))]
    spare = 1 if sum(t) < len(t) else 0
    c, start, q = cross_case(t, n, heads, 16, dtype, 31, spare)
    table = c.gpu_table()
    if expected > 300:                       # columns that no sequence reaches
        table = torch.nn.functional.pad(table, (0, expected // 16 - table.shape[1]), value=-1)
    ca = CrossAttention(c.k[None], c.v[None], table, torch.tensor(n, dtype=torch.int32, device="cuda"),
                        q_heads=heads[0], max_states=expected if expected == 300 else None)
    ca.ws.fill_(127)
    out = torch.full_like(q, 7.0)
    ca.attend(0, q, start, out)
    at = 0
    for b in range(len(n)):
        if t[b]:
            K, V = c.rows(b, 0, n[b])
            check_out(out[at:at + t[b]], np64(q[at:at + t[b]]), K, V, dtype, f"sequence {b}")
        at += t[b]
    assert (out[at:].float() == 7.0).all() and ca.device_status() == 0
    ca.close()
