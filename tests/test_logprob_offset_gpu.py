"""Rows of logits with a large common offset, up to rows that hold the type's
lowest or largest value only: log-probabilities, entropy and gradient go by the
differences of the logits, whichever kernel a row's length and layout choose."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import ops_oracle as O
from rnn_joint_network_02_b200 import frnnt
from tests.test_logprob_gpu import TYPES, check_backward, check_forward, host, ints

pytestmark = pytest.mark.gpu


def make(N, V, K, top, dtype, pad=0):
    """Rows in turn: an offset of -60000, of 2^20, the type's lowest value only, the same but for two columns, the
    largest value only, and one without offset.  Differences are steps of the type at the offset, so that rows have
    several columns of some probability."""
    g = torch.Generator().manual_seed(V + N)
    t, info = TYPES[dtype], torch.finfo(TYPES[dtype])
    z = torch.randn(N, V, generator=g) * 2
    for n in range(N):
        kind = n % 6
        if kind in (0, 1):
            at = (-60000.0, 2.0 ** 20)[kind]
            step = 2.0 ** np.floor(np.log2(abs(at))) * info.eps
            z[n] = torch.tensor(at).to(t).float() + (z[n] / step).round().clamp(-3, 0) * step
            z[n, V // 2] = z[n].max()
        elif kind == 2:
            z[n] = info.min
        elif kind == 3:
            z[n] = info.min
            z[n, 0] = z[n, V - 1] = 1.5
        elif kind == 4:
            z[n] = info.max
    wide = torch.zeros(N, V + pad, dtype=t)
    wide[:, :V] = z.to(t)
    z = wide.cuda()[:, :V]
    tokens = torch.randint(0, V, (N, K), generator=g, dtype=torch.int32).cuda()
    d = dict(dlogp=torch.randn(N, K, generator=g).cuda(), dentropy=torch.randn(N, generator=g).cuda(),
             dtop=torch.randn(N, top, generator=g).cuda() if top else None)
    return z, tokens, d


# short rows, rows of one and two chunks a warp, long rows of one and several warps, few and many coefficients
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,out_pad", [(0, 0), (3, 0), (0, 1)])
@pytest.mark.parametrize("N,V,K,top", [(12, 2, 1, 1), (12, 30, 2, 3), (12, 120, 2, 0), (12, 700, 2, 1), (12, 1900, 3, 8),
                                       (12, 2050, 1, 0), (6, 9001, 8, 4), (6, 70001, 2, 0)])
def test_gradient_goes_by_differences(cuda_ok, N, V, K, top, pad, out_pad, dtype):
    z, tokens, d = make(N, V, K, top, dtype, pad)
    r = frnnt.token_logprobs(z, tokens, top=top)
    ref = check_forward(z, tokens, top, r)
    out = torch.full((N, V + out_pad), 5.0, dtype=z.dtype, device="cuda")[:, :V]
    frnnt.token_logprobs_bwd(z, tokens, r, out=out, **d)
    check_backward(z, tokens, ref, d, out, dtype)
    frnnt.token_logprobs_bwd(z, tokens, r, out=z, **d)      # in place
    assert torch.equal(z, out)


@pytest.mark.parametrize("V", [48, 1024, 40001])
def test_two_parts_are_the_log_sum_exp(cuda_ok, V):
    z, tokens, _ = make(12, V, 1, 0, "f32")
    r = frnnt.token_logprobs(z, tokens)
    ref = O.token_logprobs(host(z), ints(tokens))
    off = (host(r.lse) - ref["max"]) + host(r.lse_rest) - ref["log_sum"]
    assert np.all(np.abs(off) <= 16 * O.UNIT + 2.0 ** -22 * np.log(V)), off


def test_result_of_an_empty_row_has_no_rest(cuda_ok):
    for V in (20, 1000, 30000):
        z = torch.full((3, V), -float("inf"), device="cuda")
        r = frnnt.token_logprobs(z)
        assert bool((r.lse == -float("inf")).all()) and bool((r.lse_rest == 0).all())
        assert bool((frnnt.token_logprobs_bwd(z, None, r, dentropy=torch.ones(3, device="cuda")) == 0).all())


def test_c_callers_without_the_second_part(cuda_ok):
    """lse_rest NULL: the forward call writes none, and the backward call's is 0."""
    N, V, K = 9, 1024, 2
    z, tokens, d = make(N, V, K, 0, "bf16")
    want = frnnt.token_logprobs(z, tokens)
    r = frnnt.LogProbs(N, K, 0, "cuda")
    r.lse_rest.zero_()
    dims = frnnt.LogprobDims(N, V, K, 0, frnnt.BF16, V, V)
    at, stream = lambda t: t.data_ptr(), torch.cuda.current_stream().cuda_stream  # noqa: E731
    L = frnnt.lib()
    assert L.frnnt_token_logprobs(ctypes.byref(dims), at(z), at(tokens), at(r.logp), at(r.entropy), at(r.lse), None, None,
                                  None, stream) == 0
    for k in ("logp", "entropy", "lse"):
        assert torch.equal(getattr(r, k), getattr(want, k))
    assert bool((r.lse_rest == 0).all())
    dz = torch.empty_like(z)
    assert L.frnnt_token_logprobs_bwd(ctypes.byref(dims), at(z), at(tokens), at(r.lse), at(r.entropy), None,
                                      at(d["dlogp"]), at(d["dentropy"]), None, at(dz), None, stream) == 0
    assert torch.equal(dz, frnnt.token_logprobs_bwd(z, tokens, r, dlogp=d["dlogp"], dentropy=d["dentropy"]))
