"""Dropout on the GPU: the mask bit for bit the oracle's, whatever the type,
shape and layout; the scale; in place; a generator state on the device."""

import numpy as np
import pytest
import torch

from oracle import ops_oracle as O
from rnn_joint_network_02_b200 import frnnt
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
