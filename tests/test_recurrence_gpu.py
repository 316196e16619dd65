"""The gated linear recurrence on the GPU against its fp64 oracle: forward,
backward and the one-step form, over types, lengths (zero, one, long, ragged),
odd sizes and strides."""

import subprocess
import sys
import threading
from pathlib import Path

import numpy as np
import pytest
import torch

from oracle import ops_oracle as O
from rnn_joint_network_02_b200 import frnnt
from tests.test_logprob_gpu import TYPES, close, host, ints

pytestmark = pytest.mark.gpu


def make(B, T, D, dtype, layout="plain", ragged=True, seed=0):
    g = torch.Generator().manual_seed(seed * 100 + B * 7 + T * 3 + D)
    t = TYPES[dtype]
    x, gate = torch.randn(B, T, D, generator=g), torch.randn(B, T, D, generator=g) * 2 + torch.linspace(-2, 6, D)
    dh = torch.randn(B, T, D, generator=g)
    if layout == "plain":
        x, gate, dh = (v.to(t).cuda() for v in (x, gate, dh))
    elif layout == "joined":             # the halves of one projection
        both = torch.cat([x, gate], 2).to(t).cuda()
        x, gate, dh = both[:, :, :D], both[:, :, D:], dh.to(t).cuda()
    elif layout == "step_major":         # [T, B, D] memory
        x, gate, dh = (v.transpose(0, 1).contiguous().to(t).cuda().transpose(0, 1) for v in (x, gate, dh))
    elif layout == "offset":             # rows that start at odd addresses
        wide = torch.zeros(B, T + 1, 2 * D + 3, dtype=t, device="cuda")
        wide[:, 1:, 1:1 + D], wide[:, 1:, D + 2:2 * D + 2] = x.to(t).cuda(), gate.to(t).cuda()
        x, gate, dh = wide[:, 1:, 1:1 + D], wide[:, 1:, D + 2:2 * D + 2], dh.to(t).cuda()
    elif layout == "shared":             # one gate for all sequences
        x, gate, dh = x.to(t).cuda(), gate[:1].to(t).cuda().expand(B, T, D), dh.to(t).cuda()
    lengths = None
    if ragged:
        lengths = torch.randint(0, T + 1, (B,), generator=g, dtype=torch.int32)
        lengths[0] = T
        if B > 1:
            lengths[1] = 0
        if B > 2:
            lengths[2] = 1
    h0, dh_last = torch.randn(B, D, generator=g).cuda(), torch.randn(B, D, generator=g).cuda()
    return x, gate, None if lengths is None else lengths.cuda(), h0, dh, dh_last


def check(x, gate, lengths, h0, dh, dh_last, dtype):
    ref = O.recurrence(host(x), host(gate), ints(lengths), host(h0), dtype)
    want = O.recurrence_bwd(host(x), host(gate), ref, host(dh), ints(lengths), host(dh_last), dtype)
    if lengths is not None:      # what lies past a sequence is not read
        for b, n in enumerate(ints(lengths)):
            dh[b, n:] = float("nan")
            if gate.stride(0) > 0:
                x[b, n:] = float("nan")
                gate[b, n:] = float("inf")
    r = frnnt.recurrence(x, gate, lengths=lengths, h0=h0)
    close(r.h, ref["h"], ref["h_tol"], "h")
    close(r.h_last, ref["h_last"], ref["h_last_tol"], "h_last")
    d = frnnt.recurrence_bwd(x, gate, r, dh, lengths=lengths, dh_last=dh_last)
    for k in ("dx", "dgate", "dh0"):
        close(d[k], want[k], want[k + "_tol"], k)
    return r, d


SHAPES = [(1, 1, 1), (3, 1, 8), (4, 2, 5), (3, 7, 64), (2, 15, 66), (3, 16, 128), (3, 17, 30), (2, 33, 256), (3, 81, 640),
          (2, 127, 33), (2, 128, 64), (3, 129, 72), (2, 257, 130), (1, 1000, 64), (3, 1500, 96), (1, 5003, 40),
          (20, 60, 16), (5, 300, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,D", SHAPES)
def test_forward_and_backward(cuda_ok, B, T, D, dtype):
    check(*make(B, T, D, dtype), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["joined", "step_major", "offset", "shared"])
@pytest.mark.parametrize("B,T,D", [(3, 150, 72), (2, 40, 33)])
def test_layouts(cuda_ok, layout, B, T, D, dtype):
    check(*make(B, T, D, dtype, layout, seed=1), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_without_lengths_start_or_end(cuda_ok, dtype):
    x, gate, _, _, dh, _ = make(2, 200, 48, dtype, ragged=False)
    check(x, gate, None, None, dh, None, dtype)


def test_long_sequence_few_channels(cuda_ok):
    check(*make(1, 20011, 24, "f32", ragged=False, seed=2), "f32")


def test_extreme_gates(cuda_ok):
    """Gates that are fully open, fully closed (also at +-inf), and slow
    memories whose 1 - a needs all its digits."""
    x, gate, _, h0, dh, dl = make(2, 300, 32, "f32", ragged=False, seed=3)
    gate[:, :, :4], gate[:, :, 4:8], gate[:, :, 8:16] = 1e4, -1e4, 14.0
    gate[:, ::5, 16:18], gate[:, ::7, 18:20] = float("inf"), float("-inf")
    check(x, gate, None, h0, dh, dl, "f32")


def test_chained_in_two_parts(cuda_ok):
    """h_last of a first part is the second part's h0, and dh0 the first part's dh_last."""
    x, gate, _, h0, dh, dl = make(2, 310, 40, "f32", ragged=False, seed=4)
    whole = frnnt.recurrence(x, gate, h0=h0)
    dw = frnnt.recurrence_bwd(x, gate, whole, dh, dh_last=dl)
    at = 130
    a = frnnt.recurrence(x[:, :at], gate[:, :at], h0=h0)
    b = frnnt.recurrence(x[:, at:], gate[:, at:], h0=a.h_last)
    db = frnnt.recurrence_bwd(x[:, at:], gate[:, at:], b, dh[:, at:], dh_last=dl)
    da = frnnt.recurrence_bwd(x[:, :at], gate[:, :at], a, dh[:, :at], dh_last=db["dh0"])
    ref = O.recurrence(host(x), host(gate), None, host(h0))
    close(torch.cat([a.h, b.h], 1), ref["h"], ref["h_tol"], "h")
    assert torch.allclose(torch.cat([da["dx"], db["dx"]], 1), dw["dx"], rtol=1e-4, atol=1e-5)
    assert torch.allclose(da["dh0"], dw["dh0"], rtol=1e-4, atol=1e-5)


def test_gradients_into_the_halves_of_one(cuda_ok):
    x, gate, lengths, h0, dh, dl = make(3, 90, 64, "bf16", "joined", seed=5)
    r = frnnt.recurrence(x, gate, lengths=lengths, h0=h0)
    want = frnnt.recurrence_bwd(x, gate, r, dh, lengths=lengths, dh_last=dl)
    both = torch.full((3, 92, 2 * 64 + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    out = dict(dx=both[:, 1:91, :64], dgate=both[:, 1:91, 64:128], dh0=torch.empty_like(h0))
    d = frnnt.recurrence_bwd(x, gate, r, dh, lengths=lengths, dh_last=dl, out=out)
    assert d is out and all(torch.equal(d[k], want[k]) for k in want)
    both[:, 1:91, :128] = 5.0
    assert bool((both == 5).all())


def test_bad_lengths_raise(cuda_ok):
    x, gate, lengths, h0, dh, _ = make(3, 20, 16, "f32", seed=6)
    r = frnnt.recurrence(x, gate, lengths=lengths)
    for bad in (-1, 21):
        lengths[1] = bad
        with pytest.raises(frnnt.FrnntStatusError) as e:
            frnnt.recurrence(x, gate, lengths=lengths)
        assert e.value.bits == frnnt.STATUS_LENGTH
        with pytest.raises(frnnt.FrnntStatusError):
            frnnt.recurrence_bwd(x, gate, r, dh, lengths=lengths)


def test_same_bits_every_time_and_captured(cuda_ok):
    x, gate, lengths, h0, dh, dl = make(2, 1200, 96, "bf16", seed=7)
    r = frnnt.recurrence(x, gate, lengths=lengths, h0=h0)
    d = frnnt.recurrence_bwd(x, gate, r, dh, lengths=lengths, dh_last=dl)
    want = [r.h.clone(), r.h_last.clone(), d["dx"].clone(), d["dgate"].clone(), d["dh0"].clone()]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            r2 = frnnt.recurrence(x, gate, lengths=lengths, h0=h0, check=False)
            d2 = frnnt.recurrence_bwd(x, gate, r2, dh, lengths=lengths, dh_last=dl, check=False)
        for _ in range(2):
            for t in (r2.h, d2["dx"]):
                t.zero_()
            g.replay()
            stream.synchronize()
            got = [r2.h, r2.h_last, d2["dx"], d2["dgate"], d2["dh0"]]
            assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_two_threads_two_streams(cuda_ok):
    """Calls from two host threads at once, each on its own stream, with blocks
    of several clusters waiting for their neighbours."""
    cases = [make(2, 1400, 100, "bf16", seed=s) for s in (21, 22)]
    want = []
    for x, gate, lengths, h0, dh, dl in cases:
        r = frnnt.recurrence(x, gate, lengths=lengths, h0=h0)
        want.append((r.h, frnnt.recurrence_bwd(x, gate, r, dh, lengths=lengths, dh_last=dl)))
    torch.cuda.synchronize()
    got, errors, start = [None, None], [], threading.Barrier(2)

    def worker(i):
        try:
            x, gate, lengths, h0, dh, dl = cases[i]
            s = torch.cuda.Stream()
            start.wait()
            for _ in range(10):
                r = frnnt.recurrence(x, gate, lengths=lengths, h0=h0, check=False, stream=s)
                d = frnnt.recurrence_bwd(x, gate, r, dh, lengths=lengths, dh_last=dl, check=False, stream=s)
            s.synchronize()
            got[i] = (r.h, d)
        except Exception as e:   # reported by the main thread
            errors.append(e)

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=120)
    assert not errors and all(g is not None for g in got), errors
    for (h, d), (wh, wd) in zip(got, want):
        assert torch.equal(h, wh) and all(torch.equal(d[k], wd[k]) for k in wd)


def test_offsets_past_32_bits(cuda_ok):
    B, T, D = 2, 40, 32
    x, gate, _, h0, dh, dl = make(B, T, D, "bf16", ragged=False, seed=8)
    r = frnnt.recurrence(x, gate, h0=h0)
    d = frnnt.recurrence_bwd(x, gate, r, dh, dh_last=dl)
    st = 56_000_000
    big = torch.empty(T * st, dtype=torch.bfloat16, device="cuda")
    spread = [big[64 * i:].as_strided((B, T, D), (D, st, 1)) for i in range(6)]      # step-major, 112 MB apart
    fx, fg, fh, fdh, fdx, fdg = spread
    fx.copy_(x), fg.copy_(gate), fdh.copy_(dh)
    out = frnnt.Recurrence(B, T, D, torch.bfloat16, "cuda")
    out.h = fh
    frnnt.recurrence(fx, fg, h0=h0, out=out)
    frnnt.recurrence_bwd(fx, fg, out, fdh, dh_last=dl, out=dict(dx=fdx, dgate=fdg, dh0=d["dh0"].clone()))
    assert torch.equal(fh, r.h) and torch.equal(fdx, d["dx"]) and torch.equal(fdg, d["dgate"])


# ------------------------------------------------------------------ one step
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,S,D", [(1, 1, 1), (1, 3, 640), (5, 2, 33), (64, 64, 640), (300, 300, 72), (33, 40, 1027)])
@pytest.mark.parametrize("form", ["plain", "beam"])
@pytest.mark.parametrize("gap", [0, 1])
def test_step(cuda_ok, N, S, D, dtype, form, gap):
    g = torch.Generator().manual_seed(N + D)
    t = TYPES[dtype]
    wide = (torch.randn(N, 2 * D + gap, generator=g) * 2).to(t).cuda()
    x, gate = wide[:, :D], wide[:, D + gap:]
    S = max(S, N) if form == "plain" else S
    state = torch.randn(S, D, generator=g).cuda()
    parent = advance = None
    if form == "beam":
        parent = torch.randint(0, S, (N,), generator=g, dtype=torch.int32).cuda()
        advance = (torch.rand(N, generator=g) < 0.6).cuda()
        gate[~advance] = float("nan")          # not read
    h, new = frnnt.recurrence_step(x, gate, state, parent=parent, advance=advance)
    want, err = O.recurrence_step(host(x), host(gate), host(state), ints(parent), ints(advance))
    close(new, want, err + 2.0 ** -24 * np.abs(want), "state")
    close(h, want, err + O.HALF_STEP[dtype] * (np.abs(want) + err), "h")
    if form == "beam":
        same = ~advance
        assert torch.equal(new[same], state[parent.long()][same])
    else:                                       # over the old state
        h2, new2 = frnnt.recurrence_step(x, gate, state, out=(torch.empty_like(h), state[:N]))
        assert torch.equal(h2, h) and torch.equal(new2, new)


def test_step_bad_parent_raises(cuda_ok):
    x = torch.randn(4, 16, device="cuda")
    state = torch.randn(3, 16, device="cuda")
    for bad in (-1, 3):
        parent = torch.tensor([0, 1, bad, 2], dtype=torch.int32, device="cuda")
        with pytest.raises(frnnt.FrnntStatusError) as e:
            frnnt.recurrence_step(x, x, state, parent=parent)
        assert e.value.bits == frnnt.STATUS_INDEX


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["plain", "offset"])
@pytest.mark.parametrize("B,T,D", [(1, 200, 64), (3, 300, 34), (2, 600, 128), (1, 700, 64), (1, 800, 64), (1, 1280, 70), (1, 4200, 64),
                                   (40, 1300, 128), (50, 700, 120), (30, 2100, 66), (60, 1000, 64)])
def test_cluster_sizes(cuda_ok, B, T, D, layout, dtype):
    """Chunk and tile counts that take each number of blocks a sequence, for one
    round and for several, the last one not full."""
    check(*make(B, T, D, dtype, layout, seed=9), dtype)


def test_few_and_many_sequences_agree(cuda_ok):
    """The blocks that share a sequence depend on the batch; the states they form agree to their rounding."""
    x, gate, _, h0, dh, dl = make(64, 900, 64, "f32", ragged=False, seed=10)
    many = frnnt.recurrence(x, gate, h0=h0)
    dm = frnnt.recurrence_bwd(x, gate, many, dh, dh_last=dl)
    ref = O.recurrence(host(x[:1]), host(gate[:1]), None, host(h0[:1]), "f32")
    want = O.recurrence_bwd(host(x[:1]), host(gate[:1]), ref, host(dh[:1]), None, host(dl[:1]), "f32")
    one = frnnt.recurrence(x[:1], gate[:1], h0=h0[:1])
    do = frnnt.recurrence_bwd(x[:1], gate[:1], one, dh[:1], dh_last=dl[:1])
    for r, d in ((many, dm), (one, do)):
        close(r.h[:1], ref["h"], ref["h_tol"], "h")
        for k in ("dx", "dgate", "dh0"):
            close(d[k][:1], want[k], want[k + "_tol"], k)


FIRST_CALL = """
import torch
from rnn_joint_network_02_b200 import frnnt
x, gate = (torch.randn(1, 1500, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2))
dh = torch.randn_like(x)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    r = frnnt.recurrence(x, gate, check=False)
    d = frnnt.recurrence_bwd(x, gate, r, dh, check=False)
graph.replay()
want = frnnt.recurrence(x, gate)
grads = frnnt.recurrence_bwd(x, gate, want, dh)
assert torch.equal(r.h, want.h) and all(torch.equal(d[k], grads[k]) for k in grads)
print("same")
"""


def test_first_call_of_a_process_is_captured(cuda_ok):
    """What a kernel asks of the runtime once may be asked during a capture."""
    done = subprocess.run([sys.executable, "-c", FIRST_CALL], capture_output=True, text=True, timeout=300,
                          cwd=Path(__file__).resolve().parent.parent)
    assert done.returncode == 0 and done.stdout.strip().endswith("same"), done.stderr[-2000:]
