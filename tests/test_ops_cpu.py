"""The operators beside the loss, without a GPU: pins of their fp64 oracle
(closed forms, finite differences, known answers of the generator) and the
refusals of the C entry points and of the binding."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import ops_oracle as O
from rnn_joint_network_02_b200 import frnnt


# ------------------------------------------------------------------ oracle pins
def test_logprobs_closed_forms():
    r = O.token_logprobs(np.zeros((1, 8)), np.array([[3, 3, -1]]), top=3)
    assert np.allclose(r["logp"], [[-np.log(8), -np.log(8), 0.0]])
    assert np.allclose(r["entropy"], np.log(8)) and np.allclose(r["lse"], np.log(8))
    assert r["top_ids"].tolist() == [[0, 1, 2]]
    z = np.full((2, 5), -np.inf)
    z[1, 2] = 7.0
    r = O.token_logprobs(z, np.array([[1], [2]]), top=5)
    assert r["lse"].tolist() == [-np.inf, 7.0] and r["entropy"].tolist() == [0.0, 0.0]
    assert r["logp"].tolist() == [[-np.inf], [0.0]]
    assert r["top_ids"].tolist() == [[0, 1, 2, 3, 4], [2, 0, 1, 3, 4]]


def test_logprobs_match_torch_double():
    g = torch.Generator().manual_seed(1)
    z = torch.randn(5, 37, generator=g, dtype=torch.float64) * 4
    r = O.token_logprobs(z.numpy(), np.array([[k, 36 - k] for k in range(5)]), top=6)
    lp = torch.log_softmax(z, 1)
    assert np.allclose(r["logp"], torch.stack([lp[:, :5].diagonal(), torch.stack([lp[k, 36 - k] for k in range(5)])], 1))
    assert np.allclose(r["entropy"], -(lp.exp() * lp).sum(1))
    assert np.allclose(r["top_logp"], lp.topk(6, 1).values)


def test_logprobs_gradient_against_differences():
    rng = np.random.default_rng(2)
    z, tokens = rng.normal(size=(3, 9)) * 2, np.array([[1, 1], [0, 8], [-1, 4]])
    dlogp, dent, dtop = rng.normal(size=(3, 2)), rng.normal(size=3), rng.normal(size=(3, 4))

    def loss(z):
        r = O.token_logprobs(z, tokens, top=4)
        return (r["logp"] * dlogp).sum() + (r["entropy"] * dent).sum() + (r["top_logp"] * dtop).sum()

    dz, _ = O.token_logprobs_bwd(z, tokens, O.token_logprobs(z, tokens, top=4), dlogp, dent, dtop)
    for n in range(3):
        for j in range(9):
            e = np.zeros_like(z)
            e[n, j] = 1e-5
            assert abs((loss(z + e) - loss(z - e)) / 2e-5 - dz[n, j]) < 1e-7
    assert np.allclose(dz.sum(1), 0.0)      # a shift of all logits changes nothing


def test_recurrence_closed_forms():
    # constant gate and input from zero: h_t = x (1 - a^(t+1))
    x, gate = np.full((1, 6, 2), 3.0), np.full((1, 6, 2), 0.4)
    a = 1 / (1 + np.exp(-0.4))
    h = O.recurrence(x, gate)["h"]
    assert np.allclose(h[0, :, 0], 3 * (1 - a ** np.arange(1, 7)))
    # open gate copies the input, closed gate keeps the state
    r = O.recurrence(x, np.full_like(x, -800.0), h0=np.ones((1, 2)))
    assert np.allclose(r["h"], x)
    r = O.recurrence(x, np.full_like(x, 800.0), h0=np.ones((1, 2)))
    assert np.allclose(r["h"], 1.0) and np.allclose(r["h_last"], 1.0)


def test_recurrence_gradients_against_differences():
    rng = np.random.default_rng(3)
    B, T, D, lengths = 3, 5, 2, np.array([5, 3, 0])
    v = dict(x=rng.normal(size=(B, T, D)), gate=rng.normal(size=(B, T, D)), h0=rng.normal(size=(B, D)))
    dh, dl = rng.normal(size=(B, T, D)), rng.normal(size=(B, D))

    def loss(v):
        r = O.recurrence(v["x"], v["gate"], lengths, v["h0"])
        return (r["h"] * dh).sum() + (r["h_last"] * dl).sum()

    g = O.recurrence_bwd(v["x"], v["gate"], O.recurrence(v["x"], v["gate"], lengths, v["h0"]), dh, lengths, dl)
    for k in v:
        num = np.zeros_like(v[k])
        for i in np.ndindex(v[k].shape):
            up, down = {m: a.copy() for m, a in v.items()}, {m: a.copy() for m, a in v.items()}
            up[k][i] += 1e-6
            down[k][i] -= 1e-6
            num[i] = (loss(up) - loss(down)) / 2e-6
        assert np.allclose(num, g["d" + k], atol=1e-8), k


def test_recurrence_step_is_the_recurrence():
    rng = np.random.default_rng(4)
    x, gate, h0 = rng.normal(size=(2, 4, 3)), rng.normal(size=(2, 4, 3)), rng.normal(size=(2, 3))
    state = h0
    for t in range(4):
        state, _ = O.recurrence_step(x[:, t], gate[:, t], state)
    assert np.allclose(state, O.recurrence(x, gate, h0=h0)["h_last"])
    moved, _ = O.recurrence_step(x[:, 0], gate[:, 0], h0, parent=[1, 1], advance=[True, False])
    assert np.allclose(moved[1], h0[1])


def test_philox_known_answers():
    """The known answers published with the generator for all-zero words, all-one
    words and the digits of pi."""
    ones = 0xFFFFFFFF
    assert O.philox4x32_10([0] * 4, [0] * 2) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]
    assert O.philox4x32_10([ones] * 4, [ones] * 2) == [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]
    assert O.philox4x32_10([0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344], [0xa4093822, 0x299f31d0]) == \
        [0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1]


def test_dropout_mask_share():
    keep, scale = O.dropout_mask(20000, 0.25, 0x123456789ABCDEF, 2 ** 40)
    # 20,000 independent draws: the share that stays is within five standard deviations of 0.75
    assert abs(keep.mean() - 0.75) < 5 * (0.75 * 0.25 / 20000) ** 0.5
    assert scale == 4 / 3
    assert O.dropout_mask(64, 0.0, 1, 0)[0].all() and not O.dropout_mask(64, 1.0, 1, 0)[0].any()


# ------------------------------------------------------------------ refusals of the C entry points
FAKE = [ctypes.c_void_p(4096 * (i + 1)) for i in range(16)]


def _logprob_dims(**kw):
    d = frnnt.LogprobDims(4, 100, 2, 3, frnnt.BF16, 100, 100)
    for k, v in kw.items():
        setattr(d, k, v)
    return ctypes.byref(d)


@pytest.mark.parametrize("kw,code", [
    (dict(N=0), 2), (dict(V=0), 2), (dict(K=-1), 2), (dict(K=33), 2), (dict(top=33), 2), (dict(top=-1), 2),
    (dict(V=2, top=3), 2), (dict(ld=99), 2), (dict(ld=1 << 41), 2), (dict(dtype=2), 4)])
def test_token_logprobs_dims_refused(kw, code):
    lib = frnnt.lib()
    assert lib.frnnt_token_logprobs(_logprob_dims(**kw), *FAKE[:8], None) == code
    assert lib.frnnt_token_logprobs_bwd(_logprob_dims(**kw), *FAKE[:10], None) == code


def test_token_logprobs_pointers_refused():
    lib = frnnt.lib()
    assert lib.frnnt_token_logprobs(None, *FAKE[:8], None) == 1
    for i in range(7):      # logits, tokens, logp, entropy, lse, top_logp, top_ids
        args = list(FAKE[:8])
        args[i] = None
        assert lib.frnnt_token_logprobs(_logprob_dims(), *args, None) == 1, i
    for i in range(8):
        args = list(FAKE[:8])
        args[i] = ctypes.c_void_p(4096 + 1)
        assert lib.frnnt_token_logprobs(_logprob_dims(), *args, None) == 6, i
    # backward: logits, tokens, lse, entropy, top_ids, dlogp, dentropy, dtop, dlogits, status
    for i in (0, 1, 2, 3, 4, 8):
        args = list(FAKE[:10])
        args[i] = None
        assert lib.frnnt_token_logprobs_bwd(_logprob_dims(), *args, None) == 1, i
    for i in range(10):
        args = list(FAKE[:10])
        args[i] = ctypes.c_void_p(4096 + 1)
        assert lib.frnnt_token_logprobs_bwd(_logprob_dims(), *args, None) == 6, i
    assert lib.frnnt_token_logprobs_bwd(_logprob_dims(ldd=99), *FAKE[:10], None) == 2
    args = list(FAKE[:10])
    args[8] = args[0]       # in place needs the same rows
    assert lib.frnnt_token_logprobs_bwd(_logprob_dims(ldd=108), *args, None) == 2


def _rec_dims(**kw):
    v = dict(B=2, T=10, D=8, dtype=frnnt.F32)
    for k in ("x", "gate", "h", "dh", "dx", "dgate"):
        v[k + "_sb"], v[k + "_st"] = 80, 8
    v.update(kw)
    d = frnnt.RecurrenceDims()
    for k, x in v.items():
        setattr(d, k, x)
    return ctypes.byref(d)


@pytest.mark.parametrize("kw,fwd,bwd", [
    (dict(B=0), 2, 2), (dict(T=0), 2, 2), (dict(D=0), 2, 2), (dict(B=65536), 2, 2), (dict(dtype=3), 4, 4),
    (dict(x_sb=-1), 2, 2), (dict(gate_st=-8), 2, 2), (dict(h_st=7), 2, 1), (dict(h_sb=79), 2, 1),
    (dict(dx_sb=0), 1, 2), (dict(dgate_st=0), 1, 2), (dict(dh_st=-1), 1, 2),
    # step-major outputs are as good as sequence-major ones, and inputs may repeat
    (dict(h_sb=8, h_st=16, dx_sb=8, dx_st=16, x_sb=0, x_st=0), 1, 1)])
def test_recurrence_dims_refused(kw, fwd, bwd):
    """(the calls that pass the size checks are refused for a missing pointer)"""
    lib = frnnt.lib()
    args = list(FAKE[:8])
    args[5] = None          # h_last
    assert lib.frnnt_recurrence_fwd(_rec_dims(**kw), *args, None) == fwd
    args = list(FAKE[:10])
    args[3] = None          # saved
    assert lib.frnnt_recurrence_bwd(_rec_dims(**kw), *args, None) == bwd


def test_recurrence_pointers_refused():
    lib = frnnt.lib()
    for i in (0, 1, 4, 5):      # x, gate, h, h_last
        args = list(FAKE[:8])
        args[i] = None
        assert lib.frnnt_recurrence_fwd(_rec_dims(), *args, None) == 1, i
    for i in range(8):
        args = list(FAKE[:8])
        args[i] = ctypes.c_void_p(4096 + 2)
        assert lib.frnnt_recurrence_fwd(_rec_dims(), *args, None) == 6, i
    for i in (0, 1, 3, 4, 6, 7):  # x, gate, saved, dh, dx, dgate
        args = list(FAKE[:10])
        args[i] = None
        assert lib.frnnt_recurrence_bwd(_rec_dims(), *args, None) == 1, i
    for i in range(10):
        args = list(FAKE[:10])
        args[i] = ctypes.c_void_p(4096 + 2)
        assert lib.frnnt_recurrence_bwd(_rec_dims(), *args, None) == 6, i


def test_step_refused():
    lib = frnnt.lib()

    def call(args=None, **kw):
        d = frnnt.StepDims(4, 4, 8, frnnt.BF16, 8, 8)
        for k, v in kw.items():
            setattr(d, k, v)
        return lib.frnnt_recurrence_step(ctypes.byref(d), *(args or FAKE[:8]), None)

    for kw, code in ((dict(N=0), 2), (dict(S=0), 2), (dict(D=0), 2), (dict(x_sn=-1), 2), (dict(dtype=9), 4)):
        assert call(**kw) == code
    for i in (0, 1, 2, 5, 6):
        args = list(FAKE[:8])
        args[i] = None
        assert call(args) == 1
    args = list(FAKE[:8])
    args[3] = None              # no parents: row n of state, so no more rows than states
    assert call(args, N=5) == 2
    args = list(FAKE[:8])
    args[6] = args[2]           # in place with parents: rows would read what others wrote
    assert call(args) == 2
    args = list(FAKE[:8])
    args[2] = ctypes.c_void_p(4096 + 2)
    assert call(args) == 6


@pytest.mark.parametrize("kw,code", [(dict(R=0), 2), (dict(C=0), 2), (dict(p=-0.1), 2), (dict(p=1.1), 2),
                                     (dict(p=float("nan")), 2), (dict(x_ld=7), 2), (dict(y_ld=7), 2),
                                     (dict(R=1 << 40), 2), (dict(dtype=5), 4)])
def test_dropout_refused(kw, code):
    d = frnnt.DropoutDims(4, 8, frnnt.F32, 8, 8, 0.5, 1, 0)
    for k, v in kw.items():
        setattr(d, k, v)
    lib = frnnt.lib()
    assert lib.frnnt_dropout(ctypes.byref(d), FAKE[0], FAKE[1], None, None) == code


def test_dropout_pointers_refused():
    lib = frnnt.lib()
    d = ctypes.byref(frnnt.DropoutDims(4, 8, frnnt.F32, 8, 8, 0.5, 1, 0))
    assert lib.frnnt_dropout(None, FAKE[0], FAKE[1], None, None) == 1
    assert lib.frnnt_dropout(d, None, FAKE[1], None, None) == 1
    assert lib.frnnt_dropout(d, FAKE[0], None, None, None) == 1
    assert lib.frnnt_dropout(d, ctypes.c_void_p(4098), FAKE[1], None, None) == 6
    assert lib.frnnt_dropout(d, FAKE[0], FAKE[1], ctypes.c_void_p(4100), None) == 6


# ------------------------------------------------------------------ refusals of the binding
Z, TOK = torch.zeros(4, 10), torch.zeros(4, 2, dtype=torch.int32)
X3, X2 = torch.zeros(2, 5, 8), torch.zeros(4, 8)


@pytest.mark.parametrize("call,msg", [
    (lambda: frnnt.token_logprobs(Z[0]), "logits must be"),
    (lambda: frnnt.token_logprobs(Z.double()), "float32 or bfloat16"),
    (lambda: frnnt.token_logprobs(Z.half()), "float32 or bfloat16"),
    (lambda: frnnt.token_logprobs(Z.t()), "columns of logits"),
    (lambda: frnnt.token_logprobs(Z, TOK.long()), "tokens is torch.int64"),
    (lambda: frnnt.token_logprobs(Z, TOK[:3]), "tokens has shape"),
    (lambda: frnnt.token_logprobs(Z, TOK[:, 0]), "tokens must be"),
    (lambda: frnnt.token_logprobs(Z, top=11), "at most"),
    (lambda: frnnt.token_logprobs(Z, top=-1), "at most"),
    (lambda: frnnt.token_logprobs(Z, torch.zeros(4, 33, dtype=torch.int32)), "at most"),
    (lambda: frnnt.token_logprobs(Z, TOK, out=frnnt.LogProbs(4, 1, 0, "cpu")), "logp has shape"),
    (lambda: frnnt.token_logprobs(Z, TOK, out=frnnt.LogProbs(4, 0, 0, "cpu")), "no logp"),
    (lambda: frnnt.token_logprobs(Z, TOK), "CUDA tensors"),
    (lambda: frnnt.token_logprobs_bwd(Z, TOK, frnnt.LogProbs(4, 2, 0, "cpu"), dlogp=torch.zeros(4, 1)), "dlogp has shape"),
    (lambda: frnnt.token_logprobs_bwd(Z, TOK, frnnt.LogProbs(4, 2, 0, "cpu"), dtop=torch.zeros(4, 1)), "dtop has shape"),
    (lambda: frnnt.token_logprobs_bwd(Z, TOK, frnnt.LogProbs(3, 2, 0, "cpu")), "logp has shape"),
    (lambda: frnnt.token_logprobs_bwd(Z, TOK, frnnt.LogProbs(4, 2, 0, "cpu"), out=Z.bfloat16()), "out is"),
    (lambda: frnnt.recurrence(X2, X2), r"\[B, T, D\]"),
    (lambda: frnnt.recurrence(X3, X3[:, :4]), "gate has shape"),
    (lambda: frnnt.recurrence(X3, X3.bfloat16()), "gate is"),
    (lambda: frnnt.recurrence(X3.transpose(1, 2), X3.transpose(1, 2)), "channels of x"),
    (lambda: frnnt.recurrence(X3, X3, lengths=torch.zeros(2)), "lengths is"),
    (lambda: frnnt.recurrence(X3, X3, h0=torch.zeros(2, 7)), "h0 has shape"),
    (lambda: frnnt.recurrence(X3, X3), "CUDA tensors"),
    (lambda: frnnt.recurrence_bwd(X3, X3, frnnt.Recurrence(2, 5, 8, X3.dtype, "cpu", save=False), X3), "kept no states"),
    (lambda: frnnt.recurrence_bwd(X3, X3, frnnt.Recurrence(2, 200, 8, X3.dtype, "cpu"), X3), "saved has shape"),
    (lambda: frnnt.recurrence_bwd(X3, X3, frnnt.Recurrence(2, 5, 8, X3.dtype, "cpu"), X3.bfloat16()), "dh is"),
    (lambda: frnnt.recurrence_step(X3, X3, X2), r"\[N, D\]"),
    (lambda: frnnt.recurrence_step(X2, X2, X2.bfloat16()), "state is"),
    (lambda: frnnt.recurrence_step(X2, X2, X2[:3]), "need parents"),
    (lambda: frnnt.recurrence_step(X2, X2, X2, parent=torch.zeros(4)), "parent is"),
    (lambda: frnnt.recurrence_step(X2, X2, X2, advance=torch.zeros(4)), "advance is"),
    (lambda: frnnt.recurrence_step(X2, X2, X2, parent=torch.zeros(4, dtype=torch.int32), out=(X2.clone(), X2)), "overlaps"),
    (lambda: frnnt.recurrence_step(X2, X2, X2), "CUDA tensors"),
    (lambda: frnnt.dropout(X2.half(), 0.5, 1), "float32 or bfloat16"),
    (lambda: frnnt.dropout(X2, 1.5, 1), r"p must be"),
    (lambda: frnnt.dropout(X2, float("nan"), 1), r"p must be"),
    (lambda: frnnt.dropout(X2[:0], 0.5, 1), "no elements"),
    (lambda: frnnt.dropout(X2.t(), 0.5, 1), "constant distance"),
    (lambda: frnnt.dropout(X2, 0.5, torch.zeros(2)), "seed is"),
    (lambda: frnnt.dropout(X2, 0.5, 1, out=X2.bfloat16()), "out is"),
    (lambda: frnnt.dropout(X2, 0.5, 1), "CUDA tensors"),
])
def test_binding_refuses(call, msg):
    with pytest.raises(ValueError, match=msg):
        call()


def test_calls_go_to_the_tensors_device_and_stream(monkeypatch):
    """The context that a call is made in: none on the current device's current
    stream, the tensors' device where that is another one, a given stream where
    it belongs to that device."""
    monkeypatch.setattr(frnnt, "_current_device", lambda: 0)
    first, second = torch.device("cuda", 0), torch.device("cuda", 1)
    assert frnnt._elsewhere(first, None) is None
    there = frnnt._elsewhere(second, None)
    assert isinstance(there, torch.cuda.device) and there.idx == 1

    class Stream:
        device = first

    assert isinstance(frnnt._elsewhere(first, Stream()), torch.cuda.StreamContext)
    with pytest.raises(ValueError, match="the stream is on"):
        frnnt._elsewhere(second, Stream())
    with pytest.raises(ValueError, match="CUDA tensors"):
        frnnt._elsewhere(torch.device("cpu"), None)
