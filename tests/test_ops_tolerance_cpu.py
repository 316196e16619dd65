"""The tolerances that the oracle gives the log-probabilities: small where the
kernels' arithmetic is good, whatever value masks a column, so that a wrong
result is refused; and wide enough for a plain computation in fp32."""

import numpy as np
import pytest
import torch

from oracle import ops_oracle as O

LOWEST = {"f32": torch.finfo(torch.float32).min, "bf16": torch.finfo(torch.bfloat16).min}


def _masked(V, lowest, left):
    """One row of the type's lowest value but for the columns of `left`."""
    z = np.full((1, V), lowest)
    for j, v in left.items():
        z[0, j] = v
    return z


@pytest.mark.parametrize("dtype", LOWEST)
@pytest.mark.parametrize("V", [9, 1024, 50257])
@pytest.mark.parametrize("left", [{0: 2.0}, {0: 2.0, 3: 1.0, 7: -4.0}])
def test_rows_masked_by_the_lowest_value_are_held_to_account(dtype, V, left):
    z, tokens = _masked(V, LOWEST[dtype], left), np.array([[0, 1]])
    r = O.token_logprobs(z, tokens, top=2)
    few = np.array([v for v in left.values()])
    lp = few - np.log(np.exp(few).sum())
    assert np.allclose(r["lse"], 2.0 - lp[0]) and np.allclose(r["entropy"], -(np.exp(lp) * lp).sum())
    for k in ("lse_tol", "entropy_tol"):
        assert r[k][0] < 3e-5, (k, r[k])
    assert r["logp_tol"][0, 0] < 3e-5 and r["top_tol"][0, 0] < 3e-5
    # a masked column's log-probability is as large as the mask, and good to its own size
    assert r["logp_tol"][0, 1] < 2.0 ** -22 * abs(LOWEST[dtype])
    dz, tol = O.token_logprobs_bwd(z, tokens, r, np.array([[1.0, 0.5]]), np.array([0.7]), np.array([[0.2, -0.3]]), dtype)
    assert np.all(tol[0] <= O.HALF_STEP[dtype] * 1.01 * np.abs(dz[0]) + 1e-4), tol.max()
    # mistakes that such a row has to show: masked columns that count, ln V too much, a survivor that is left out
    wrong = np.log(np.exp(few).sum() + V - len(few))
    assert abs(wrong - r["lse"][0]) > r["lse_tol"][0]
    assert np.log(V) > r["entropy_tol"][0] and 1e-3 > r["logp_tol"][0, 0]
    p = np.exp(few[0] - wrong)
    assert abs(-1.4 * (p - np.exp(lp[0]))) > tol[0, 0]


@pytest.mark.parametrize("dtype", LOWEST)
def test_rows_of_the_lowest_value_only(dtype):
    """Nothing tells such a row's columns apart: they are equally likely."""
    r = O.token_logprobs(np.full((1, 64), LOWEST[dtype]), np.array([[5]]), top=3)
    assert np.allclose(r["logp"], -np.log(64)) and np.allclose(r["entropy"], np.log(64))
    assert r["logp_tol"][0, 0] < 3e-5 and r["entropy_tol"][0] < 3e-5 and r["top_tol"].max() < 3e-5
    assert r["lse_tol"][0] <= 2.0 ** -23 * abs(LOWEST[dtype])        # half a step of its value


def test_a_shift_of_all_logits_costs_log_probabilities_nothing():
    z = np.random.default_rng(1).normal(size=(1, 300)) * 3
    tokens = np.array([[3, 250]])
    near, far = (O.token_logprobs(z + c, tokens, top=4) for c in (0.0, 2.0 ** 20))
    for k in ("logp_tol", "entropy_tol", "top_tol"):
        assert np.allclose(near[k], far[k], rtol=1e-6), k
    assert far["lse_tol"][0] < 2.0 ** -3        # half a step of 2^20


def test_rows_without_a_value_have_no_room():
    """An infinite tolerance would let any value pass for -inf."""
    z = np.full((3, 5), -np.inf)
    z[1, 2], z[2, 4] = np.nan, np.inf
    r = O.token_logprobs(z, np.array([[0], [1], [2]]), top=2)
    assert all(np.all(np.isfinite(r[k])) for k in ("lse_tol", "entropy_tol", "logp_tol", "top_tol"))


@pytest.mark.parametrize("scale", [0.1, 3.0, 30.0])
@pytest.mark.parametrize("shift", [0.0, -60000.0])
@pytest.mark.parametrize("V", [2, 37, 1024, 20001])
def test_plain_fp32_is_within(V, shift, scale):
    """A computation in numpy's float32, a column after another in eight strands, keeps to the tolerances."""
    rng = np.random.default_rng(V)
    z = (rng.normal(size=(4, V)) * scale + shift).astype(np.float32)
    z[1, rng.random(V) < 0.5] = -np.inf
    z[1, 0], z[2, :] = shift, LOWEST["f32"]
    z[2, V // 2] = 2.0
    tokens = rng.integers(0, V, size=(4, 2))
    ref = O.token_logprobs(z.astype(np.float64), tokens, 2)
    dlogp, dent = rng.normal(size=(4, 2)).astype(np.float32), rng.normal(size=4).astype(np.float32)
    want, tol = O.token_logprobs_bwd(z.astype(np.float64), tokens, ref, dlogp.astype(np.float64), dent.astype(np.float64))
    f = np.float32
    for n in range(4):
        row = z[n]
        m = row.max()
        with np.errstate(over="ignore", invalid="ignore", under="ignore"):
            d = np.maximum((row - m) * f(1.4426950408889634), f(-160))
            e = np.exp2(d)
            pad = (-V) % 8
            s = np.concatenate([e, np.zeros(pad, f)]).reshape(-1, 8).cumsum(0, dtype=f)[-1].sum(dtype=f)
            w = np.concatenate([e * d, np.zeros(pad, f)]).reshape(-1, 8).cumsum(0, dtype=f)[-1].sum(dtype=f)
            ls = np.log(s)
            lse, entropy = f(m + ls), f(ls - f(0.6931471805599453) * (w / s))
            rest = (m - (lse - (lse - m))) + (ls - (lse - m))
            logp = (row[tokens[n]] - m) - ls
            q = np.maximum(((row - lse) - rest) * f(1.4426950408889634), f(-160))
            grad = np.exp2(q) * (f(-dent[n] * f(0.6931471805599453)) * q - (dent[n] * entropy + dlogp[n].sum(dtype=f)))
        for t, c in zip(tokens[n], dlogp[n]):
            grad[t] += c
        assert abs(lse - ref["lse"][n]) <= ref["lse_tol"][n], (n, lse)
        assert abs(entropy - ref["entropy"][n]) <= ref["entropy_tol"][n], (n, entropy)
        same = logp == ref["logp"][n]
        assert np.all(same | (np.abs(np.where(same, 0.0, logp) - np.where(same, 0.0, ref["logp"][n])) <= ref["logp_tol"][n])), (n, logp)
        assert np.all(np.abs(grad - want[n]) <= tol[n]), n
