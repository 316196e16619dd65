"""The operators as they are used together: a prediction network in front of
the transducer loss, and one decoding step behind it."""

import numpy as np
import pytest
import torch

import oracle
from oracle import ops_oracle as O
from rnn_joint_network_02_b200 import frnnt, synth
from tests.helpers import rel_l2

pytestmark = pytest.mark.gpu


def _predictor(B, U, D, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(B, U + 1, 2 * D, generator=g)


def test_training_step(cuda_ok):
    """projection -> recurrence -> dropout -> transducer loss and back, against
    the same chain of fp64 oracles and against differences of it."""
    b = synth.workload("tiny")
    B, U, D = b.g.shape[0], b.g.shape[1] - 1, b.g.shape[2]
    proj, seed, p = _predictor(B, U, D, 1), 1234567, 0.25
    dev = {k: getattr(b, k).cuda() for k in ("f", "W_f", "W_g", "W_o", "b_o", "labels", "T_len", "U_len")}
    both = proj.cuda()
    x, gate = both[:, :, :D], both[:, :, D:]
    steps = dev["U_len"] + 1
    r = frnnt.recurrence(x, gate, lengths=steps)
    g = frnnt.dropout(r.h, p, seed)
    loss, grads = frnnt.fwd_bwd(dev["f"], g, dev["W_f"], dev["W_g"], dev["W_o"], dev["b_o"], dev["labels"],
                                dev["T_len"], dev["U_len"])
    dh = frnnt.dropout(grads["dg"], p, seed)
    d = frnnt.recurrence_bwd(x, gate, r, dh, lengths=steps)

    f, _, W_f, W_g, W_o, b_o = (t.numpy() for t in b.float64())
    keep, scale = O.dropout_mask(B * (U + 1) * D, p, seed, 0)
    factor = keep.reshape(B, U + 1, D) * scale
    n = (b.U_len + 1).numpy()

    def chain(pr):
        h = O.recurrence(pr[:, :, :D], pr[:, :, D:], n)
        return h, oracle.fwd_bwd(f, h["h"] * factor, W_f, W_g, W_o, b_o, b.labels.numpy(), b.T_len.numpy(), b.U_len.numpy())

    pr = proj.double().numpy()
    h, ref = chain(pr)
    want = O.recurrence_bwd(pr[:, :, :D], pr[:, :, D:], h, ref.dg * factor, n)
    assert np.allclose(loss.cpu().numpy(), ref.loss, rtol=1e-4)
    for k in ("dx", "dgate"):
        assert rel_l2(d[k].cpu().numpy(), want[k]) <= 1e-4, k
    step = np.random.default_rng(2).normal(size=pr.shape)
    num = (chain(pr + 1e-5 * step)[1].loss.sum() - chain(pr - 1e-5 * step)[1].loss.sum()) / 2e-5
    got = (torch.cat([d["dx"], d["dgate"]], 2).double().cpu().numpy() * step).sum()
    assert abs(got - num) <= 2e-4 * np.linalg.norm(step) * np.linalg.norm(np.concatenate([want["dx"], want["dgate"]], 2))


def test_cell_logprobs_give_the_loss(cuda_ok):
    """Blank and label log-probabilities of every lattice cell, and the alpha
    recursion over them, are the loss that frnnt.fwd_bwd returns."""
    b = synth.workload("tiny")
    d = {k: getattr(b, k).cuda() for k in ("f", "g", "W_f", "W_g", "W_o", "b_o", "labels", "T_len", "U_len")}
    B, T, U = b.f.shape[0], b.f.shape[1], b.g.shape[1] - 1
    h = torch.tanh((d["f"] @ d["W_f"])[:, :, None] + (d["g"] @ d["W_g"])[:, None])
    z = (h @ d["W_o"].t() + d["b_o"]).reshape(B * T * (U + 1), -1)
    label = torch.cat([d["labels"], torch.full((B, 1), frnnt.NO_TOKEN, dtype=torch.int32, device="cuda")], 1)
    tokens = torch.stack([torch.zeros_like(label), label], 2)[:, None].expand(B, T, U + 1, 2).reshape(-1, 2).contiguous()
    lp = frnnt.token_logprobs(z, tokens).logp.view(B, T, U + 1, 2).double().cpu().numpy()
    loss, _ = frnnt.fwd_bwd(*(d[k] for k in ("f", "g", "W_f", "W_g", "W_o", "b_o", "labels", "T_len", "U_len")))
    for i in range(B):
        n, u = int(b.T_len[i]), int(b.U_len[i])
        alpha = oracle.alpha_lattice(lp[i, :, :, 0], lp[i, :, :, 1], n, u)
        assert abs(-(alpha[n - 1, u] + lp[i, n - 1, u, 0]) - float(loss[i])) <= 1e-4 * abs(float(loss[i]))


def test_decoding_steps_follow_the_sequence(cuda_ok):
    """A beam that is reordered at each label keeps, for each surviving
    hypothesis, the states of its own history: the same as the sequence form
    over that history."""
    N, D, V, U = 6, 64, 50, 5
    g = torch.Generator().manual_seed(3)
    table = torch.randn(V, 2 * D, generator=g).to(torch.bfloat16).cuda()
    W = torch.randn(V, D, generator=g).to(torch.bfloat16).cuda()
    state, history = torch.zeros(N, D, device="cuda"), torch.zeros(N, 0, dtype=torch.long, device="cuda")
    token = torch.arange(N, device="cuda")
    parent = torch.arange(N, dtype=torch.int32, device="cuda")
    for _ in range(U):
        both = table[token]
        h, state = frnnt.recurrence_step(both[:, :D], both[:, D:], state, parent=parent)
        history = torch.cat([history[parent.long()], token[:, None]], 1)
        r = frnnt.token_logprobs(h @ W.t(), top=2)
        flat = r.top_logp.reshape(-1)
        best = torch.argsort(flat, descending=True)[:N]
        parent = (best // 2).to(torch.int32)
        token = r.top_ids.reshape(-1)[best].long()
    both = table[history]
    seq = frnnt.recurrence(both[:, :, :D], both[:, :, D:])
    ref = O.recurrence(both[:, :, :D].double().cpu().numpy(), both[:, :, D:].double().cpu().numpy())
    assert np.all(np.abs(state.double().cpu().numpy() - ref["h_last"]) <= ref["h_last_tol"])
    assert np.all(np.abs(seq.h_last.double().cpu().numpy() - ref["h_last"]) <= ref["h_last_tol"])


def test_a_chain_on_a_side_stream(cuda_ok):
    """Every call takes the stream it is given, for its work and its outputs, and
    the chain's results are those of the current stream."""
    g = torch.Generator().manual_seed(5)
    both = torch.randn(4, 300, 96, generator=g).cuda()
    z = torch.randn(64, 3000, generator=g).cuda()
    tokens, one = torch.randint(0, 3000, (64, 1), generator=g, dtype=torch.int32).cuda(), torch.ones(64, 1).cuda()

    def chain(stream):
        x, gate = both[:, :, :48], both[:, :, 48:]
        r = frnnt.recurrence(x, gate, stream=stream)
        y = frnnt.dropout(r.h, 0.3, 17, stream=stream)
        d = frnnt.recurrence_bwd(x, gate, r, y, stream=stream)
        step, _ = frnnt.recurrence_step(both[:, 0, :48], both[:, 0, 48:], r.h_last, stream=stream)
        lp = frnnt.token_logprobs(z, tokens, top=4, stream=stream)
        dz = frnnt.token_logprobs_bwd(z, tokens, lp, dlogp=one, stream=stream)
        return [r.h, y, d["dx"], d["dgate"], d["dh0"], step, lp.logp, lp.top_ids, dz]

    want = chain(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = chain(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
