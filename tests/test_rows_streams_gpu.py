"""Steps of the row operators on streams given in every form that the library takes."""
import pytest
import torch

from oracle import rows as R
from test_rows_gpu import decoder, shared_case

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("form", ["stream", "address", "default", "none"])
def test_a_weighed_step_and_an_eviction_on_a_stream(form):
    c, _, _, n, q = shared_case([2], [0], [30, 21], (4, 2, 64), 16, BF, 97)
    dec = decoder(c, n, 4)
    dec.track_weights(40, 4)
    out = torch.empty_like(q)[None]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    stream = {"stream": s, "address": s.cuda_stream, "default": 0, "none": None}[form]
    dec.weighed_step(q[None], out, stream)
    torch.cuda.synchronize()
    mass, pos = dec.weights["mass"][0].cpu().numpy(), dec.weights["pos"][0].cpu().numpy()
    dec.evict_step(9, 3, stream)
    torch.cuda.synchronize()
    assert dec.seq_len.tolist() == [13, 13]
    for b in range(2):
        for h in range(2):
            stay, moves = R.evict_moves(mass[b, h], pos[b, h], n[b] - 4, n[b], 9, 3)
            to = {y: x for x, y in moves}
            assert dec.weights["pos"][0, b, h, :9].tolist() == [int(pos[b, h, to.get(i, i)]) for i in range(9)]
    assert dec.device_status() == 0
