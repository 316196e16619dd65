"""A loss call on a stream that is not the current one: its buffers come from
that stream's memory, memory that the current stream's queued work still reads
is left alone, its status is read behind its work, and its results are those of
the current stream."""

import pytest
import torch

from rnn_joint_network_02_b200 import frnnt, synth
from tests.helpers import to_device

pytestmark = pytest.mark.gpu
ARGS = ("f", "g", "W_f", "W_g", "W_o", "b_o", "labels", "T_len", "U_len")
DROP = frnnt.Dropout(0.2, 31)


def _stream_of(t):
    """The stream whose pool holds t's memory."""
    at = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= at < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in the caching allocator")


def _outputs(d, batch):
    dims = frnnt.dims_of(d["f"], d["g"], d["W_o"], "bf16", "untiled", "auto", 0, batch.blank)
    return frnnt.Outputs(*(d[k] for k in ARGS[:6]), dims)


@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("drop", [None, DROP])
def test_first_call_on_another_stream(cuda_ok, own, drop):
    batch = synth.workload("short")
    d = to_device(batch)
    args = [d[k] for k in ARGS]
    want, ref = frnnt.fwd_bwd(*args, mode="untiled", dropout=drop)
    want, df = want.clone(), ref["df"].clone()
    out = _outputs(d, batch) if own else None
    pending = [torch.full_like(t, 3.0) for t in (d["f"], d["g"], d["f"], d["g"])]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    # work that reads tensors which are freed before it has run: nothing of the call below may be put there
    torch.cuda._sleep(50_000_000)
    sums = [p.float().sum() for p in pending]
    sizes = [p.numel() for p in pending]
    del pending
    loss, grads = frnnt.fwd_bwd(*args, mode="untiled", out=out, stream=side, dropout=drop)
    assert torch.cuda.current_stream() != side
    side.synchronize()
    assert torch.allclose(loss, want, rtol=1e-5)
    # (fp32 atomic additions in another order, then a rounding to bf16)
    assert torch.equal(grads["df"] == 0, df == 0) and torch.allclose(grads["df"].float(), df.float(), rtol=0.05, atol=1e-4)
    torch.cuda.synchronize()
    assert [float(s) for s in sums] == [3.0 * n for n in sizes]
    if not own:
        assert _stream_of(loss) == _stream_of(grads["dW_o"]) == side.cuda_stream
    if own and drop:
        assert all(_stream_of(t) == side.cuda_stream for t in out.dropped)
        kept = out.dropped
        frnnt.fwd_bwd(*args, mode="untiled", out=out, stream=side, dropout=drop)
        assert out.dropped is kept


@pytest.mark.parametrize("entry", ["fwd_bwd", "noalloc", "pruned", "tdt"])
def test_status_is_read_behind_the_work(cuda_ok, entry):
    """The call waits for its own stream before it looks at the status."""
    batch = synth.workload("short")
    d = to_device(batch)
    args = [d[k] for k in ARGS]
    kw = dict(mode="untiled")
    call = dict(fwd_bwd=frnnt.fwd_bwd, noalloc=frnnt.fwd_bwd_noalloc, pruned=frnnt.fwd_bwd_pruned,
                tdt=frnnt.fwd_bwd_tdt)[entry]
    if entry == "pruned":
        args += [synth.diagonal_bounds(batch.T_len, batch.U_len, batch.f.shape[1], 6).cuda(), 6]
    if entry == "tdt":
        W_d, b_d = synth.duration_head(batch, len(synth.TDT_DURATIONS), seed=5)
        args[6:6] = [W_d.cuda(), b_d.cuda()]
        kw.update(durations=synth.TDT_DURATIONS)
    wrong = list(args)
    at = 8 if entry == "tdt" else 6
    wrong[at] = args[at].clone()
    wrong[at][0, 0] = -7
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    with pytest.raises(frnnt.FrnntStatusError) as e:
        call(*wrong, stream=side, **kw)
    assert e.value.bits == frnnt.STATUS_LABEL
    call(*args, stream=side, **kw)
