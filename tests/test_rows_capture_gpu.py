"""What a capture and a later track_weights do to the weights of captured steps."""
import pytest
import torch

from test_rows_gpu import decoder, shared_case

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def tracked(prefix_rows=20, rows=64):
    c, start, prefix, n, q = shared_case([2, 1], [prefix_rows] * 2, [9, 11, 20], (4, 2, 64), 16, BF, 52)
    dec = decoder(c, n, 4)
    dec.share_prefix(start, torch.tensor(prefix))
    g = torch.Generator().manual_seed(5)
    mass = torch.rand(1, 3, 2, rows, generator=g).cuda()
    pos = torch.randint(0, 9, (1, 3, 2, rows), generator=g, dtype=torch.int32).cuda()
    dec.track_weights(rows, torch.tensor(prefix), mass=mass, pos=pos)
    return dec, q


@pytest.mark.parametrize("kind", ["shared", "weighed"])
@pytest.mark.parametrize("host_io", [False, True])
def test_a_capture_leaves_the_weights_alone(kind, host_io):
    from dynamic_sparse_kv_gb300 import CapturedStep
    dec, q = tracked()
    before = {x: dec.weights[x].clone() for x in ("mass", "pos", "seen", "protect")}
    step = CapturedStep(dec, kind, host_io=host_io)
    torch.cuda.synchronize()
    for x, t in before.items():
        assert torch.equal(dec.weights[x], t), x
    # the first replay after it adds what the step itself adds
    if host_io:
        step.q_host.copy_(q[None])
    else:
        step.q.copy_(q[None])
    step.replay()
    torch.cuda.synchronize()
    once, where = dec.weights["mass"].clone(), dec.weights["pos"].clone()
    assert not torch.equal(once, before["mass"])
    for x in ("mass", "pos"):
        dec.weights[x].copy_(before[x])
    out = torch.empty_like(q)[None]
    (dec.shared_step if kind == "shared" else dec.weighed_step)(q[None], out)
    assert torch.equal(dec.weights["mass"], once) and torch.equal(dec.weights["pos"], where)
    assert torch.equal(step.out, out) and dec.device_status() == 0


def test_begin_token_advances_the_weights_of_every_captured_step():
    """An old capture goes on with its own weights, so the positions it writes must go on too."""
    from dynamic_sparse_kv_gb300 import CapturedStep
    dec, q = tracked()
    step = CapturedStep(dec, "shared")
    old = dec.weights
    dec.track_weights(64, 20)
    new = dec.weights
    first, second = old["seen"].tolist(), new["seen"].tolist()
    for t in range(1, 4):
        dec.begin_token()
        assert old["seen"].tolist() == [x + t for x in first]
        assert new["seen"].tolist() == [x + t for x in second]
        step.q.copy_(q[None])
        step.replay()
        for b, n in enumerate(dec.seq_len.tolist()):
            assert (old["pos"][0, b, :, n - 1 - 20] == first[b] + t - 1).all()
    # one counter given to both is advanced once, and weights that no step holds not at all
    del step
    loose = old["seen"]
    del old
    shared = new["seen"]
    keep = CapturedStep(dec, "weighed")
    dec.track_weights(64, 20, seen=shared)
    was, out_of_use = shared.tolist(), loose.tolist()
    dec.begin_token()
    assert shared.tolist() == [x + 1 for x in was] and loose.tolist() == out_of_use
    assert keep.launches == 1 and dec.device_status() == 0
