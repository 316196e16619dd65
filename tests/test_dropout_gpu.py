"""Dropout on the GPU: the mask bit for bit the oracle's, whatever the type,
shape and layout; the scale; in place; a generator state on the device."""

import numpy as np
import pytest
import torch

from oracle import ops_oracle as O
from rnn_joint_network_02_b200 import frnnt, synth
from tests.helpers import compare, run_oracle, to_device
from tests.test_logprob_gpu import TYPES, close, host

pytestmark = pytest.mark.gpu


def check(x, y, p, seed, offset, dtype):
    keep, scale = O.dropout_mask(x.numel(), p, seed, offset)
    want = np.where(keep.reshape(x.shape), host(x) * scale, 0.0)
    # the scale in fp32 and its product are rounded (2^-24 each), then the result to its type
    close(y, want, (2.0 ** -22 + O.HALF_STEP[dtype]) * np.abs(want) + 2.0 ** -133, "y")
    if scale:
        assert np.array_equal(host(y) != 0, keep.reshape(x.shape) & (host(x) != 0))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1,), (7,), (8,), (9,), (3, 5), (16, 640), (2, 3, 129), (255,), (257,), (2049,), (33, 1000)])
@pytest.mark.parametrize("p", [0.1, 0.5])
def test_mask_and_scale(cuda_ok, shape, p, dtype):
    x = torch.randn(shape, generator=torch.Generator().manual_seed(1)).to(TYPES[dtype]).cuda()
    seed, offset = 0xFEDCBA9876543210, 2 ** 33 + 5
    y = frnnt.dropout(x, p, seed, offset)
    check(x, y, p, seed, offset, dtype)
    assert torch.equal(frnnt.dropout(x, p, seed, offset), y)
    assert frnnt.dropout(x, p, seed, offset, out=x) is x and torch.equal(x, y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["rows", "odd_rows", "shifted", "steps"])
def test_layouts_share_the_mask(cuda_ok, layout, dtype):
    g = torch.Generator().manual_seed(2)
    wide = torch.randn(6, 50, 80, generator=g).to(TYPES[dtype]).cuda()
    x = {"rows": wide[0, :, :64], "odd_rows": wide[0, :, 3:40], "shifted": wide.view(-1)[1:20001],
         "steps": wide[:, :, 8:16]}[layout]
    want = frnnt.dropout(x.contiguous(), 0.3, 99, 7)
    check(x.contiguous(), want, 0.3, 99, 7, dtype)
    assert torch.equal(frnnt.dropout(x, 0.3, 99, 7), want)
    canvas = torch.full_like(wide, 5.0)
    out = canvas.as_strided(x.shape, x.stride(), x.storage_offset())
    assert torch.equal(frnnt.dropout(x, 0.3, 99, 7, out=out), want)
    assert torch.equal(frnnt.dropout(x.contiguous(), 0.3, 99, 7, out=out), want)
    out.fill_(5.0)
    assert bool((canvas == 5).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ends_of_p(cuda_ok, dtype):
    x = torch.randn(1000, device="cuda").to(TYPES[dtype])
    x[3], x[5] = float("nan"), float("inf")
    y = frnnt.dropout(x, 0.0, 1)
    assert torch.allclose(y, x, rtol=0, atol=0, equal_nan=True)
    assert bool((frnnt.dropout(x, 1.0, 1) == 0).all())
    y = frnnt.dropout(torch.full_like(x, float("nan")), 0.5, 1)
    keep, _ = O.dropout_mask(1000, 0.5, 1, 0)
    assert np.array_equal(torch.isnan(y).cpu().numpy(), keep) and bool((y[~torch.isnan(y)] == 0).all())


def test_counters_wrap_and_streams_follow_on(cuda_ok):
    x = torch.randn(100, device="cuda")
    check(x, frnnt.dropout(x, 0.5, 3, 2 ** 64 - 4), 0.5, 3, 2 ** 64 - 4, "f32")
    y = frnnt.dropout(x, 0.5, 3, 10)
    assert torch.equal(torch.cat([frnnt.dropout(x[:40], 0.5, 3, 10), frnnt.dropout(x[40:], 0.5, 3, 15)]), y)


def test_generator_state_on_the_device(cuda_ok):
    """A captured graph draws new numbers when the state it reads has moved on."""
    x = torch.randn(5000, device="cuda")
    rng = torch.tensor([-77, 5], dtype=torch.int64, device="cuda")       # seed 2^64 - 77
    assert torch.equal(frnnt.dropout(x, 0.4, rng, 3), frnnt.dropout(x, 0.4, 2 ** 64 - 77, 8))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            y = frnnt.dropout(x, 0.4, rng)
            rng[1] += 625
        for k in range(3):
            g.replay()
            stream.synchronize()
            assert torch.equal(y, frnnt.dropout(x, 0.4, 2 ** 64 - 77, 5 + 625 * k))


def test_offsets_past_32_bits(cuda_ok):
    """Elements past 2^32 keep their own numbers."""
    n = 2 ** 32 + 4096
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    frnnt.dropout(x, 0.5, 11, 0, out=x)
    tail = torch.ones(4096, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(x[2 ** 32:], frnnt.dropout(tail, 0.5, 11, 2 ** 29))
    assert not torch.equal(x[2 ** 32:], x[:4096])


# ------------------------------------------------------------------ the loss calls' own dropout
ARGS = ("f", "g", "W_f", "W_g", "W_o", "b_o", "labels", "T_len", "U_len")


def _dropped_batch(batch, drop):
    """The batch with f and g dropped as the call drops them (rounded once to its type), and the factors."""
    n = batch.f.numel()
    out, factors = dict(batch.__dict__), []
    for k, at in (("f", drop.offset), ("g", drop.offset + (n + 7) // 8)):
        t = getattr(batch, k)
        keep, scale = O.dropout_mask(t.numel(), drop.p, drop.seed, at)
        factors.append(torch.from_numpy(keep.reshape(t.shape) * scale))
        out[k] = (t.double() * factors[-1].float().double()).to(torch.float32).to(t.dtype)
    return synth.Batch(**out), factors


@pytest.mark.parametrize("entry", ["fwd_bwd", "noalloc", "pruned"])
def test_loss_with_dropout(cuda_ok, entry):
    """Loss and gradients of the dropped inputs against the oracle; df and dg
    masked alike (their tolerance is the contract's, on the oracle's masked
    gradient); the inputs themselves are left alone."""
    name = "tiny" if entry != "pruned" else "short"
    batch = synth.workload(name, **({} if name == "tiny" else dict(B=2, T=40, U=8, T_range=(20, 40), U_range=(4, 8))))
    d, drop = to_device(batch), frnnt.Dropout(0.3, 77, 5)
    f0 = d["f"].clone()
    args = [d[k] for k in ARGS]
    dropped, factors = _dropped_batch(batch, drop)
    if entry == "pruned":
        S = 5
        bounds = synth.diagonal_bounds(batch.T_len, batch.U_len, batch.f.shape[1], S)
        loss, grads = frnnt.fwd_bwd_pruned(*args, bounds.cuda(), S, dropout=drop)
        ref = run_oracle(dropped, bounds=bounds.numpy(), S=S)
    else:
        loss, grads = (frnnt.fwd_bwd if entry == "fwd_bwd" else frnnt.fwd_bwd_noalloc)(*args, dropout=drop)
        ref = run_oracle(dropped)
    ref.df, ref.dg = ref.df * factors[0].numpy(), ref.dg * factors[1].numpy()
    compare(loss, grads, ref, batch.dtype, extra_note=f"dropout {entry}")
    assert bool((grads["df"][factors[0].cuda() == 0] == 0).all())
    assert torch.equal(d["f"], f0)


def test_loss_with_dropout_uses_its_outputs_again_and_captures(cuda_ok):
    """With ``out`` nothing is allocated by the second call, and a captured call
    draws new numbers as the device state moves on."""
    batch = synth.workload("short")
    d = to_device(batch)
    args = [d[k] for k in ARGS]
    n = frnnt.Dropout.counters(d["f"], d["g"])
    want = [frnnt.fwd_bwd(*args, mode="untiled", dropout=frnnt.Dropout(0.2, 9, k * n))[0].clone() for k in range(3)]
    assert not torch.equal(want[0], want[1])
    rng = torch.tensor([9, 0], dtype=torch.int64, device="cuda")
    dims = frnnt.dims_of(d["f"], d["g"], d["W_o"], "bf16", "untiled", "auto", 0, batch.blank)
    out = frnnt.Outputs(*(d[k] for k in ARGS[:6]), dims)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        loss, _ = frnnt.fwd_bwd(*args, mode="untiled", out=out, stream=stream, dropout=frnnt.Dropout(0.2, rng))
        stream.synchronize()
        assert torch.allclose(loss, want[0], rtol=1e-5)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            frnnt.fwd_bwd(*args, mode="untiled", out=out, stream=stream, check=False, dropout=frnnt.Dropout(0.2, rng))
            rng[1] += n
        for k in range(3):
            g.replay()
            stream.synchronize()
            assert torch.allclose(out.loss, want[k], rtol=1e-5)


@pytest.mark.parametrize("entry", ["fwd_bwd", "tdt"])
def test_loss_with_dropout_is_the_calls_one_by_one(cuda_ok, entry):
    """The argument and the separate calls (dropout of f and g, loss, dropout of
    df and dg) give the same bits of the loss and the same zeros."""
    batch = synth.workload("short")
    d, drop = to_device(batch), frnnt.Dropout(0.15, 2 ** 63 + 11, 2 ** 40)
    args = [d[k] for k in ARGS]
    kw = {}
    if entry == "tdt":
        W_d, b_d = synth.duration_head(batch, len(synth.TDT_DURATIONS), seed=5)
        args[6:6] = [W_d.cuda(), b_d.cuda()]
        kw = dict(durations=synth.TDT_DURATIONS)
    call = frnnt.fwd_bwd_tdt if entry == "tdt" else frnnt.fwd_bwd
    loss, grads = call(*args, mode="untiled", dropout=drop, **kw)
    at = drop.offset + (d["f"].numel() + 7) // 8
    f, g = frnnt.dropout(d["f"], drop.p, drop.seed, drop.offset), frnnt.dropout(d["g"], drop.p, drop.seed, at)
    want, one = call(f, g, *args[2:], mode="untiled", **kw)
    assert torch.equal(loss, want)
    df = frnnt.dropout(one["df"], drop.p, drop.seed, drop.offset)
    assert torch.equal(grads["df"] == 0, df == 0) and torch.allclose(grads["df"].float(), df.float(), rtol=0.05, atol=1e-4)
