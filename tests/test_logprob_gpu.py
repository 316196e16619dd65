"""Token log-probabilities on the GPU against their fp64 oracle: values,
entropy, alternatives and the gradient of the logits, over types, row lengths
and layouts, with masked, empty, tied, NaN and infinite rows."""

import threading

import numpy as np
import pytest
import torch

from oracle import ops_oracle as O
from rnn_joint_network_02_b200 import frnnt

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(N, V, K, top, dtype, seed=0, pad=0, shift=0, special=True):
    """Rows of logits on the device (a view `shift` elements into rows of V +
    pad), tokens, and gradients of the outputs."""
    g = torch.Generator().manual_seed(seed * 1000 + N * 7 + V)
    z = torch.randn(N, V, generator=g) * 3
    z[torch.rand(N, V, generator=g) < 0.2] = -float("inf")
    if special and N > 4:
        z[0] = -float("inf")                                  # nothing left
        z[1] = 1.5                                            # all equal
        z[2, V // 2] = float("nan")
        z[3, V - 1] = float("inf")
        z[4] = -float("inf")
        z[4, V // 3] = -60000.0                               # one candidate, far down
    if special and N > 6:
        z[5] = torch.finfo(TYPES[dtype]).min                  # masked by the type's lowest value, but for one
        z[5, 0] = 2.0
        z[6] = z[6].nan_to_num(neginf=-1.0).round()           # many ties
    wide = torch.full((N, V + pad + shift), 777.0).to(TYPES[dtype])
    wide[:, shift:shift + V] = z.to(TYPES[dtype])
    z = wide.cuda()[:, shift:shift + V]
    tokens = None
    if K:
        tokens = torch.randint(0, V, (N, K), generator=g, dtype=torch.int32)
        tokens[torch.rand(N, K, generator=g) < 0.15] = frnnt.NO_TOKEN
        if K > 1:
            tokens[::3, 1] = tokens[::3, 0]                   # the same token twice
        tokens = tokens.cuda()
    d = dict(dlogp=torch.randn(N, K, generator=g).cuda() if K else None, dentropy=torch.randn(N, generator=g).cuda(),
             dtop=torch.randn(N, top, generator=g).cuda() if top else None)
    return z, tokens, d


def host(t):
    return None if t is None else t.double().cpu().numpy()


def ints(t):
    return None if t is None else t.cpu().numpy()


def close(got, want, tol, what):
    got = host(got)
    assert got.shape == want.shape, what
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN in other places"
    same = (got == want) | np.isnan(want)
    with np.errstate(invalid="ignore"):
        bad = ~same & ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} values off, the first at {np.argwhere(bad)[0]}: " \
                          f"{got[bad][0]!r} for {want[bad][0]!r} +- {np.broadcast_to(tol, want.shape)[bad][0]!r}"


def check_forward(z, tokens, top, r):
    ref = O.token_logprobs(host(z), ints(tokens), top)
    close(r.lse, ref["lse"], ref["lse_tol"], "lse")
    close(r.entropy, ref["entropy"], ref["entropy_tol"], "entropy")
    if tokens is not None:
        close(r.logp, ref["logp"], ref["logp_tol"], "logp")
    if top:
        assert np.array_equal(ints(r.top_ids), ref["top_ids"])
        close(r.top_logp, ref["top_logp"], ref["top_tol"], "top_logp")
    return ref


def check_backward(z, tokens, ref, d, dz, dtype):
    want, tol = O.token_logprobs_bwd(host(z), ints(tokens), ref, host(d["dlogp"]), host(d["dentropy"]),
                                     host(d["dtop"]), dtype)
    close(dz, want, tol, "dlogits")


SHAPES = [
    # N, V, K, top
    (9, 1, 1, 1), (9, 2, 2, 2), (9, 7, 1, 7), (9, 8, 2, 4), (9, 31, 3, 5), (9, 33, 1, 32), (9, 128, 2, 1),
    (9, 255, 0, 8), (9, 257, 2, 0), (9, 1000, 4, 20), (9, 1024, 2, 8), (9, 1025, 32, 32), (40, 1024, 2, 0),
    (1, 1024, 1, 8), (7, 4096, 1, 16), (7, 4099, 2, 3), (3, 50257, 1, 20), (2, 131071, 2, 32), (1, 131072, 1, 4),
    (700, 130, 2, 4), (2500, 24, 1, 2),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,K,top", SHAPES)
def test_forward_and_backward(cuda_ok, N, V, K, top, dtype):
    z, tokens, d = make(N, V, K, top, dtype)
    r = frnnt.token_logprobs(z, tokens, top=top)
    ref = check_forward(z, tokens, top, r)
    dz = frnnt.token_logprobs_bwd(z, tokens, r, **d)
    check_backward(z, tokens, ref, d, dz, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,K,top", [(80, 9001, 2, 8), (40, 17000, 1, 20), (1200, 3001, 2, 8), (1900, 9000, 6, 4),
                                       (9000, 1000, 3, 2), (40000, 48, 2, 3)])
def test_many_rows(cuda_ok, N, V, K, top, dtype):
    """The row counts that choose other ways through the kernels, against the
    definition in torch's float64 (with the oracle's tolerances)."""
    z, tokens, d = make(N, V, K, top, dtype, seed=20, special=False)
    r = frnnt.token_logprobs(z, tokens, top=top)
    dz = frnnt.token_logprobs_bwd(z, tokens, r, **d)
    w = z.double()
    lse = torch.logsumexp(w, 1, keepdim=True)
    lp, p = w - lse, torch.exp(w - lse)
    entropy = -torch.where(p > 0, p * lp, 0.0).sum(1)
    near = 4 * O.UNIT + 2.0 ** -23 * (float(w[w > -float("inf")].abs().max()) + np.log(V) + 1)
    none = tokens == frnnt.NO_TOKEN
    at = tokens.clamp(min=0).long()

    def check(got, want, tol, what):
        want = torch.as_tensor(want, dtype=torch.float64, device="cuda")
        bad = ~((got.double() == want) | ((got.double() - want).abs() <= tol))
        assert not bool(bad.any()), f"{what}: {int(bad.sum())} values off"

    check(r.lse, lse[:, 0], near, "lse")
    check(r.entropy, entropy, near * (np.log(V) + 2), "entropy")
    check(r.logp, torch.where(none, 0.0, lp.gather(1, at)), near, "logp")
    values, ids = torch.sort(w, dim=1, descending=True, stable=True)
    assert torch.equal(r.top_ids.long(), ids[:, :top])
    check(r.top_logp, values[:, :top] - lse, near, "top_logp")
    coef = torch.where(none, 0.0, d["dlogp"].double())
    size = coef.abs().sum(1, keepdim=True) + d["dtop"].double().abs().sum(1, keepdim=True)
    want = -p * (coef.sum(1, keepdim=True) + d["dtop"].double().sum(1, keepdim=True))
    want.scatter_add_(1, at, coef)
    want.scatter_add_(1, ids[:, :top], d["dtop"].double())
    de = d["dentropy"].double()[:, None]
    safe = torch.where(p > 0, lp, 0.0)
    want -= de * p * (safe + entropy[:, None])
    rel = 2 * near
    tol = 2 * rel * p * (size + de.abs() * (safe.abs() + entropy[:, None] + 1)) + de.abs() * p * near * (np.log(V) + 2)
    hit = torch.zeros_like(w).scatter_(1, at, 1.0).scatter_(1, ids[:, :top], 1.0)
    tol = tol + hit * 2.0 ** -21 * size
    tol = tol + O.HALF_STEP[dtype] * (want.abs() + tol) + 2.0 ** -126
    check(dz, want, tol, "dlogits")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,shift,out_pad,out_shift", [(8, 0, 8, 0), (3, 0, 0, 0), (0, 1, 0, 0), (1, 2, 5, 3),
                                                         (24, 5, 24, 5), (0, 0, 1, 0)])
@pytest.mark.parametrize("V", [9, 1024, 2051])
def test_strided_and_unaligned_rows(cuda_ok, V, pad, shift, out_pad, out_shift, dtype):
    """Rows at any distance and alignment; elements around the output rows stay."""
    N, K, top = 8, 2, 5
    z, tokens, d = make(N, V, K, top, dtype, seed=3, pad=pad, shift=shift)
    r = frnnt.token_logprobs(z, tokens, top=min(top, V))
    ref = check_forward(z, tokens, top, r)
    wide = torch.full((N, out_shift + V + out_pad), 5.0, dtype=z.dtype, device="cuda")
    out = wide[:, out_shift:out_shift + V]
    dz = frnnt.token_logprobs_bwd(z, tokens, r, **d, out=out)
    assert dz.data_ptr() == out.data_ptr()
    check_backward(z, tokens, ref, d, out, dtype)
    assert bool((wide[:, :out_shift] == 5).all()) and bool((wide[:, out_shift + V:] == 5).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("terms", [("dlogp",), ("dentropy",), ("dtop",), ("dlogp", "dtop"), ()])
def test_backward_terms_one_by_one(cuda_ok, terms, dtype):
    z, tokens, d = make(12, 300, 2, 4, dtype, seed=5)
    d = {k: (v if k in terms else None) for k, v in d.items()}
    r = frnnt.token_logprobs(z, tokens, top=4)
    ref = O.token_logprobs(host(z), ints(tokens), 4)
    check_backward(z, tokens, ref, d, frnnt.token_logprobs_bwd(z, tokens, r, **d), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,pad", [(1024, 0), (20001, 7)])
def test_backward_in_place(cuda_ok, V, pad, dtype):
    z, tokens, d = make(10, V, 3, 6, dtype, seed=6, pad=pad)
    r = frnnt.token_logprobs(z, tokens, top=6)
    apart = frnnt.token_logprobs_bwd(z, tokens, r, **d)
    frnnt.token_logprobs_bwd(z, tokens, r, **d, out=z)
    assert torch.equal(apart.nan_to_num(nan=-99.0), z.nan_to_num(nan=-99.0))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V", [(3, 70000), (300, 1024)])
def test_same_bits_every_time(cuda_ok, N, V, dtype):
    z, tokens, d = make(N, V, 4, 8, dtype, seed=7)
    first = None
    for _ in range(3):
        r = frnnt.token_logprobs(z, tokens, top=8)
        dz = frnnt.token_logprobs_bwd(z, tokens, r, **d)
        bits = [t.contiguous().view(torch.uint8).clone() for t in (r.logp, r.entropy, r.lse, r.top_logp, r.top_ids, dz)]
        first = first or bits
        assert all(torch.equal(a, b) for a, b in zip(first, bits))


@pytest.mark.parametrize("bad", [-2, 300, 2 ** 31 - 1])
def test_bad_tokens_raise_and_touch_nothing_else(cuda_ok, bad):
    z, tokens, d = make(6, 300, 2, 0, "f32", special=False)
    good = frnnt.token_logprobs(z, tokens)
    wrong = tokens.clone()
    wrong[4, 1] = bad
    with pytest.raises(frnnt.FrnntStatusError) as e:
        frnnt.token_logprobs(z, wrong)
    assert e.value.bits == frnnt.STATUS_LABEL
    r = frnnt.token_logprobs(z, wrong, check=False)
    rows = [0, 1, 2, 3, 5]
    assert torch.equal(r.logp[rows], good.logp[rows]) and torch.equal(r.entropy, good.entropy)
    with pytest.raises(frnnt.FrnntStatusError):
        frnnt.token_logprobs_bwd(z, wrong, good, dlogp=d["dlogp"])


def test_offsets_past_32_bits(cuda_ok):
    """Rows that start more than 2^32 bytes (and 2^31 elements) into the array."""
    V, ld = 1000, 1_100_000_000
    z, tokens, d = make(3, V, 1, 4, "bf16", special=False)
    big = torch.empty(2 * ld + V, dtype=torch.bfloat16, device="cuda")
    far = big.as_strided((3, V), (ld, 1))
    far.copy_(z)
    a, b = frnnt.token_logprobs(z, tokens, top=4), frnnt.token_logprobs(far, tokens, top=4)
    assert torch.equal(a.logp, b.logp) and torch.equal(a.top_ids, b.top_ids) and torch.equal(a.entropy, b.entropy)
    want = frnnt.token_logprobs_bwd(z, tokens, a, **d)
    frnnt.token_logprobs_bwd(far, tokens, a, **d, out=far)
    assert torch.equal(want, far)


def test_result_used_again_and_other_stream(cuda_ok):
    z, tokens, _ = make(20, 512, 2, 4, "bf16", seed=8)
    want = frnnt.token_logprobs(z, tokens, top=4)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    r = frnnt.token_logprobs(z, tokens, top=4, stream=side)
    again = frnnt.token_logprobs(z, tokens, top=4, out=r, stream=side)
    side.synchronize()
    assert again is r
    assert torch.equal(r.top_ids, want.top_ids) and torch.equal(r.logp.nan_to_num(), want.logp.nan_to_num())


def test_captured_and_replayed(cuda_ok):
    """Two captured graphs and an eager call share nothing but their inputs."""
    z, tokens, d = make(16, 40000, 2, 8, "bf16", seed=9, special=False)
    other = make(16, 40000, 2, 8, "bf16", seed=10, special=False)[0]
    want = [(r.logp.clone(), r.top_ids.clone(), frnnt.token_logprobs_bwd(t, tokens, r, **d))
            for t in (z, other) for r in [frnnt.token_logprobs(t, tokens, top=8)]]
    buf, graphs, outs = [z.clone(), z.clone()], [], []
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        for i in range(2):
            stream.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                r = frnnt.token_logprobs(buf[i], tokens, top=8, check=False)
                dz = frnnt.token_logprobs_bwd(buf[i], tokens, r, **d, check=False)
            graphs.append(g)
            outs.append((r.logp, r.top_ids, dz))
        buf[1].copy_(other)
        for g in (graphs[0], graphs[1], graphs[0]):
            g.replay()
        stream.synchronize()
    for got, ref in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_two_threads(cuda_ok):
    cases = [make(30, 5000, 2, 8, "bf16", seed=s, special=False) for s in (11, 12)]
    want = [frnnt.token_logprobs(z, t, top=8) for z, t, _ in cases]
    torch.cuda.synchronize()
    got, errors, start = [None, None], [], threading.Barrier(2)

    def worker(i):
        try:
            s = torch.cuda.Stream()
            start.wait()
            for _ in range(20):
                r = frnnt.token_logprobs(cases[i][0], cases[i][1], top=8, stream=s)
            s.synchronize()
            got[i] = r
        except Exception as e:   # reported by the main thread
            errors.append(e)

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=120)
    assert not errors and all(g is not None for g in got), errors
    for g, w in zip(got, want):
        assert torch.equal(g.logp, w.logp) and torch.equal(g.top_ids, w.top_ids)


SHORT = [
    # N, V, K, top: short rows, one below and one above every change of the lanes a row takes; row counts that end
    # inside a warp; more tokens than lanes a row; every column an alternative
    (1, 1, 0, 0), (37, 3, 32, 0), (37, 12, 5, 12), (35, 16, 3, 0), (35, 17, 2, 17), (33, 32, 8, 32), (33, 33, 2, 1),
    (31, 64, 20, 0), (31, 65, 2, 32), (130, 128, 17, 0), (17, 128, 16, 1), (130, 129, 2, 20), (19, 256, 2, 0),
    (19, 256, 6, 32), (19, 257, 2, 20), (11, 511, 32, 0), (11, 512, 2, 0), (11, 513, 2, 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,K,top", SHORT)
def test_short_rows(cuda_ok, N, V, K, top, dtype):
    z, tokens, d = make(N, V, K, top, dtype, seed=30, pad=3, shift=1)
    r = frnnt.token_logprobs(z, tokens, top=top)
    ref = check_forward(z, tokens, top, r)
    wide = torch.full((N, V + 5), 5.0, dtype=z.dtype, device="cuda")
    frnnt.token_logprobs_bwd(z, tokens, r, out=wide[:, 2:2 + V], **d)
    check_backward(z, tokens, ref, d, wide[:, 2:2 + V], dtype)
    assert bool((wide[:, :2] == 5).all()) and bool((wide[:, 2 + V:] == 5).all())
    kept = wide[:, 2:2 + V].clone()
    frnnt.token_logprobs_bwd(z, tokens, r, out=z, **d)   # in place
    assert torch.equal(z.isnan(), kept.isnan()) and torch.equal(z.nan_to_num(), kept.nan_to_num())


@pytest.mark.parametrize("V", [5, 40, 120])
def test_short_rows_with_bad_tokens(cuda_ok, V):
    z, tokens, d = make(6, V, 2, 0, "bf16", special=False)
    good = frnnt.token_logprobs(z, tokens)
    wrong = tokens.clone()
    wrong[4, 1] = V
    r = frnnt.token_logprobs(z, wrong, check=False)
    assert r.logp[4, 1] == 0
    assert torch.equal(r.logp[:4], good.logp[:4]) and torch.equal(r.entropy, good.entropy)
    with pytest.raises(frnnt.FrnntStatusError) as e:
        frnnt.token_logprobs(z, wrong)
    assert e.value.bits == frnnt.STATUS_LABEL
    with pytest.raises(frnnt.FrnntStatusError) as e:
        frnnt.token_logprobs_bwd(z, wrong, good, dlogp=d["dlogp"])
    assert e.value.bits == frnnt.STATUS_LABEL


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,K,top", [(5, 523, 2, 0), (8000, 1027, 2, 0), (7500, 1500, 1, 2), (6, 1030, 5, 3),
                                       (3, 40001, 2, 0), (4, 1, 1, 1), (4, 7, 2, 0)])
@pytest.mark.parametrize("pad,shift,out_pad,out_shift", [(3, 0, 0, 0), (0, 0, 3, 1), (1, 2, 5, 3), (4, 4, 0, 0)])
def test_gradient_elsewhere_in_its_16_bytes(cuda_ok, N, V, K, top, pad, shift, out_pad, out_shift, dtype):
    """Rows of logits and of the gradient that start at different places of their 16 bytes: the bits are those of
    dense rows, and nothing around the gradient's rows is written."""
    z, tokens, d = make(N, V, K, top, dtype, seed=40, pad=pad, shift=shift)
    r = frnnt.token_logprobs(z, tokens, top=top)
    want = frnnt.token_logprobs_bwd(z.contiguous(), tokens, r, **d)
    wide = torch.full((N, out_shift + V + out_pad), 5.0, dtype=z.dtype, device="cuda")
    got = frnnt.token_logprobs_bwd(z, tokens, r, out=wide[:, out_shift:out_shift + V], **d)
    raw = torch.int16 if dtype == "bf16" else torch.int32
    assert torch.equal(got.contiguous().view(raw), want.view(raw))
    assert bool((wide[:, :out_shift] == 5).all()) and bool((wide[:, out_shift + V:] == 5).all())
