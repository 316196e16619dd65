"""Failure detection in the recurrence, without a fault: a message between the
blocks that share a sequence is withheld, or a block gives up (the
lose_scan_maps test setting), so bounded waits run out.  The call must end soon,
report FRNNT_STATUS_TIMEOUT, leave the sequences that had no part in it right,
and leave the context usable: the same calls made again give the same bits as
before."""

import time

import pytest
import torch

from oracle import ops_oracle as O
from rnn_joint_network_02_b200 import frnnt
from tests.test_logprob_gpu import close, host, ints
from tests.test_recurrence_gpu import make

pytestmark = pytest.mark.gpu
KEYS = ("dx", "dgate", "dh0")


@pytest.fixture
def lose_maps():
    frnnt.lose_scan_maps(0)
    yield frnnt.lose_scan_maps
    frnnt.lose_scan_maps(0)


def _times_out(call):
    start = time.monotonic()
    with pytest.raises(frnnt.FrnntStatusError) as e:
        call()
    torch.cuda.synchronize()
    assert e.value.bits == frnnt.STATUS_TIMEOUT
    assert frnnt.lose_scan_maps(0) == 0, "the setting is consumed by exactly one launch"
    return time.monotonic() - start


# sequences, steps, channels that clusters of blocks share, in one round (the first) or three and more
SHAPES = [(3, 300, 34, "plain", "bf16"), (1, 4200, 64, "plain", "bf16"), (30, 2100, 66, "plain", "bf16"),
          (40, 1300, 128, "plain", "bf16"), (3, 300, 34, "offset", "f32"), (1, 4200, 64, "offset", "f32"),
          (30, 2100, 66, "offset", "f32"), (30, 1300, 64, "offset", "f32")]


@pytest.mark.parametrize("quit", [False, True])
@pytest.mark.parametrize("B,T,D,layout,dtype,round", [(*shape, r) for shape in SHAPES for r in (0, 1, 2, -1)
                                                      if r <= 0 or shape[1] > 1000])
def test_lost_map_times_out_and_context_survives(cuda_ok, lose_maps, B, T, D, layout, dtype, round, quit):
    x, gate, lengths, h0, dh, dl = make(B, T, D, dtype, layout, seed=51)
    r = frnnt.recurrence(x, gate, lengths=lengths, h0=h0)
    d = frnnt.recurrence_bwd(x, gate, r, dh, lengths=lengths, dh_last=dl)
    want = [t.clone() for t in (r.h, r.h_last, *(d[k] for k in KEYS))]

    lose_maps(1, round, quit)
    assert _times_out(lambda: frnnt.recurrence(x, gate, lengths=lengths, h0=h0)) < 5
    lose_maps(1, round, quit)
    assert _times_out(lambda: frnnt.recurrence_bwd(x, gate, r, dh, lengths=lengths, dh_last=dl)) < 5

    # sequences without such a round (here: empty ones, and of one step where a later round is meant) take no harm
    lose_maps(1, round, quit)
    hurt = frnnt.recurrence(x, gate, lengths=lengths, h0=h0, check=False)
    short = [b for b, n in enumerate(lengths.tolist()) if n == 0 or (n == 1 and round > 0)]
    assert all(torch.equal(hurt.h[b], want[0][b]) and torch.equal(hurt.h_last[b], want[1][b]) for b in short)

    r = frnnt.recurrence(x, gate, lengths=lengths, h0=h0)
    d = frnnt.recurrence_bwd(x, gate, r, dh, lengths=lengths, dh_last=dl)
    assert all(torch.equal(a, b) for a, b in zip((r.h, r.h_last, *(d[k] for k in KEYS)), want))


def test_the_limit_itself(cuda_ok, lose_maps):
    """With the limit of ordinary calls (2 s a wait): the first wait in a round of many, each block's second one for
    what is on its way to it, and nothing else."""
    x, gate, _, _, _, _ = make(1, 20000, 64, "bf16", ragged=False, seed=52)
    want = frnnt.recurrence(x, gate).h.clone()
    lose_maps(1, 2, False, 20000)
    took = _times_out(lambda: frnnt.recurrence(x, gate))
    assert took < 15, took
    assert torch.equal(frnnt.recurrence(x, gate).h, want)


@pytest.mark.parametrize("B,T,D,layout,dtype", [(1, 4200, 64, "plain", "bf16"), (3, 700, 65, "offset", "f32")])
def test_refused_clusters_are_no_error(cuda_ok, B, T, D, layout, dtype):
    """Clusters that the runtime refuses are done without: the call succeeds, its results are those of one block a
    sequence, and no error is left for the next call."""
    x, gate, lengths, h0, dh, dl = make(B, T, D, dtype, layout, seed=53)
    run = lambda: frnnt.recurrence(x, gate, lengths=lengths, h0=h0)  # noqa: E731
    back = lambda r: frnnt.recurrence_bwd(x, gate, r, dh, lengths=lengths, dh_last=dl)  # noqa: E731
    assert not frnnt.refuse_clusters(True)
    try:
        r = run()
        d = back(r)
        assert frnnt.lose_scan_maps(1) == 0
        again = run()
        assert frnnt.lose_scan_maps(0) == 1, "no launch had clusters"
    finally:
        frnnt.refuse_clusters(False)
    assert torch.equal(r.h, again.h)
    torch.ones(1, device="cuda").add_(1).item()      # (would report an error that was left)
    ref = O.recurrence(host(x), host(gate), ints(lengths), host(h0), dtype)
    want = O.recurrence_bwd(host(x), host(gate), ref, host(dh), ints(lengths), host(dl), dtype)
    close(r.h, ref["h"], ref["h_tol"], "h")
    for k in KEYS:
        close(d[k], want[k], want[k + "_tol"], k)
    frnnt.lose_scan_maps(1)
    with pytest.raises(frnnt.FrnntStatusError):     # granted again
        run()
