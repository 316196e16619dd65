"""The second part of the log-sum-exp, without a GPU: its checks."""

import ctypes

import pytest
import torch

from rnn_joint_network_02_b200 import frnnt


def test_misaligned_pointer_refused():
    fake = [ctypes.c_void_p(4096 * (i + 1)) for i in range(10)]
    dims = frnnt.LogprobDims(4, 100, 2, 3, frnnt.BF16, 100, 100, 4096 + 2)
    lib = frnnt.lib()
    assert lib.frnnt_token_logprobs(ctypes.byref(dims), *fake[:8], None) == 6
    assert lib.frnnt_token_logprobs_bwd(ctypes.byref(dims), *fake, None) == 6


def test_result_of_other_rows_refused():
    z, tokens = torch.zeros(4, 10), torch.zeros(4, 2, dtype=torch.int32)
    r = frnnt.LogProbs(4, 2, 0, "cpu")
    assert r.lse_rest.shape == (4,) and r.lse_rest.dtype == torch.float32
    r.lse_rest = torch.zeros(3)
    with pytest.raises(ValueError, match="lse_rest has shape"):
        frnnt.token_logprobs(z, tokens, out=r)
    with pytest.raises(ValueError, match="lse_rest has shape"):
        frnnt.token_logprobs_bwd(z, tokens, r)
