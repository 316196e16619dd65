"""Operators beside the transducer loss, as they are measured: token log-probabilities of logit rows with
entropy and top alternatives (and their gradient), the gated linear recurrence of a prediction network or
encoder layer (training, and one step of a beam of hypotheses), and dropout from a counter-based generator.

``own`` false: the plain form of each, elementary torch operations in 32 bits.  ``own`` true: the calls a
user makes of the package.
"""

import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # Log-probabilities of rows in hand.  One step of a beam search with four hypotheses over 1,024 word
        # pieces: every hypothesis's own token, its entropy and the eight best continuations (latency).
        dict(name="beam_step_4x1024", op="logprobs", N=4, V=1024, K=1, top=8, dtype="bf16", pad=0, masked=0.0),
        # The same for a batch of beams over 4,096 characters, 32-bit logits, a quarter of them forbidden
        # (prefix or grammar constraints set those to -inf).
        dict(name="beams_64x4096_f32", op="logprobs", N=64, V=4096, K=1, top=16, dtype="f32", pad=0, masked=0.25),
        # Few rows of a very large, odd vocabulary: one step of a few requests.
        dict(name="step_7x131071", op="logprobs", N=7, V=131071, K=1, top=20, dtype="bf16", pad=0, masked=0.0),
        # Training: blank and label log-probabilities of the 400 x 81 cells of a medium utterance, with
        # entropy regularisation, and the gradient of the logits.
        dict(name="cells_32400x1024_train", op="logprobs_train", N=32400, V=1024, K=2, dtype="bf16", pad=0),
        # Scoring and distillation of a large batch over a large vocabulary: the largest case.
        dict(name="rows_8190x32768_train", op="logprobs_train", N=8190, V=32768, K=1, dtype="bf16", pad=128),
        # Gated linear recurrence, forward and backward.  The prediction network of a small batch (21 label
        # positions), of an ordinary ragged one in 32 bits, an encoder layer over 1,500 frames, and two very
        # long sequences of odd length.
        dict(name="predict_8x21x256_train", op="recurrence_train", B=8, T=21, D=256, dtype="bf16", ragged=True, joined=False),
        dict(name="predict_16x81x640_f32", op="recurrence_train", B=16, T=81, D=640, dtype="f32", ragged=True, joined=False),
        dict(name="encode_8x1500x512_train", op="recurrence_train", B=8, T=1500, D=512, dtype="bf16", ragged=True, joined=True),
        dict(name="long_2x32749x1024_train", op="recurrence_train", B=2, T=32749, D=1024, dtype="bf16", ragged=False, joined=True),
        # One label of 64 hypotheses: each continues its parent's state, or keeps it where it emitted blank.
        dict(name="step_64x640", op="recurrence_step", N=64, D=640, dtype="bf16"),
        # Dropout and its gradient: the prediction rows of a medium batch, and an encoder batch of the
        # largest workload, 32 bits.
        dict(name="dropout_1296x640", op="dropout", R=1296, D=640, dtype="bf16", p=0.1),
        dict(name="dropout_32000x1024_f32", op="dropout", R=32000, D=1024, dtype="f32", p=0.25),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "logprobs_train", "recurrence_train", "recurrence_train", "recurrence_step", "dropout"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "logprobs":
        V = _spread(rng, 8, 131072)
        N = _spread(rng, 1, max(1, min(40000, (1 << 26) // V)))
        return dict(op=op, N=N, V=V, K=rng.choice([0, 1, 2, 5]), top=min(V, rng.choice([0, 1, 4, 8, 20, 32])), dtype=dtype,
                    pad=rng.choice([0, 0, 8, 5]), masked=rng.choice([0.0, 0.0, 0.3]))
    if op == "logprobs_train":
        V = _spread(rng, 8, 131072)
        N = _spread(rng, 1, max(1, min(60000, (1 << 26) // V)))
        return dict(op=op, N=N, V=V, K=rng.choice([1, 2, 4]), dtype=dtype, pad=rng.choice([0, 0, 128, 3]))
    if op == "recurrence_train":
        D = _spread(rng, 16, 2048) // 8 * 8 + rng.choice([0, 0, 0, 8, 3])
        T = _spread(rng, 1, 32768)
        B = _spread(rng, 1, max(1, min(64, (1 << 25) // (T * D))))
        return dict(op=op, B=B, T=T, D=D, dtype=dtype, ragged=rng.random() < 0.6, joined=rng.random() < 0.5)
    if op == "recurrence_step":
        return dict(op=op, N=_spread(rng, 1, 4096), D=_spread(rng, 16, 4096) // 8 * 8 + rng.choice([0, 0, 0, 5]), dtype=dtype)
    D = _spread(rng, 16, 4096)
    return dict(op=op, R=_spread(rng, 1, max(1, (1 << 25) // D)), D=D, dtype=dtype, p=round(rng.uniform(0.02, 0.6), 3))


# ------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(1_000_003 * (seed % 1_000_000) + 17)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _logits(g, N, V, pad, dtype):
    """Rows of a trained output layer: a flat part and a few strong candidates; a view of wider rows where `pad` is set."""
    z = torch.empty(N, V + pad, device="cuda", dtype=TYPES[dtype])
    step = max(1, (1 << 26) // (V + pad))
    for n in range(0, N, step):
        z[n:n + step] = _randn(g, min(step, N - n), V + pad) * 2.5
    # three different columns of each row
    away = torch.randint(0, V // 2 - 1, (N, 3), generator=g, device="cuda") + torch.tensor([0, 1, V // 2], device="cuda")
    away[:, 0] = 0
    best = (torch.randint(0, V, (N, 1), generator=g, device="cuda") + away) % V
    z.scatter_(1, best, (_randn(g, N, 3) * 2 + 10).to(z.dtype))
    return z[:, :V], best


def prepare(case, seed):
    g, op = _generator(seed), case["op"]
    s = dict(case)
    if op in ("logprobs", "logprobs_train"):
        N, V, K = case["N"], case["V"], case["K"]
        s["logits"], best = _logits(g, N, V, case["pad"], case["dtype"])
        other = torch.randint(0, V, (N, K), generator=g, device="cuda")
        pick = torch.rand(N, K, generator=g, device="cuda") < 0.7
        tokens = torch.where(pick, best[:, torch.arange(K, device="cuda") % 3], other)
        if case.get("masked"):
            # forbidden entries: -inf, never a row's given tokens or its first candidate
            hit = torch.rand(N, V, generator=g, device="cuda") < case["masked"]
            hit.scatter_(1, torch.cat([tokens, best], 1), False)
            s["logits"].masked_fill_(hit, -math.inf)
        s["tokens"] = tokens.to(torch.int32) if K else None
        if op == "logprobs_train":
            s["dlogp"] = -torch.rand(N, K, generator=g, device="cuda")
            s["dentropy"] = _randn(g, N) * 0.1
        return s
    if op == "recurrence_train":
        B, T, D, t = case["B"], case["T"], case["D"], TYPES[case["dtype"]]
        # memories from a step to some hundreds of steps, by channel
        bias = torch.linspace(-1.0, 5.5, D, device="cuda")
        if case["joined"]:   # the two halves of one projection
            both = torch.empty(B, T, 2 * D, device="cuda", dtype=t)
            s["x"], s["gate"] = both[:, :, :D], both[:, :, D:]
        else:
            s["x"], s["gate"] = (torch.empty(B, T, D, device="cuda", dtype=t) for _ in range(2))
        s["x"].copy_(_randn(g, B, T, D))
        s["gate"].copy_(_randn(g, B, T, D) + bias)
        s["h0"] = _randn(g, B, D) * 0.5
        s["dh"] = _randn(g, B, T, D).to(t)
        s["dh_last"] = _randn(g, B, D)
        s["lengths"] = torch.randint((T + 1) // 2, T + 1, (B,), generator=g, device="cuda").to(torch.int32) if case["ragged"] else None
        return s
    if op == "recurrence_step":
        N, D, t = case["N"], case["D"], TYPES[case["dtype"]]
        s["x"], s["gate"] = _randn(g, N, D).to(t), (_randn(g, N, D) + torch.linspace(-1.0, 5.5, D, device="cuda")).to(t)
        s["state"] = _randn(g, N, D)
        s["parent"] = torch.randint(0, N, (N,), generator=g, device="cuda").to(torch.int32)
        s["advance"] = torch.rand(N, generator=g, device="cuda") < 0.6
        return s
    R, D, t = case["R"], case["D"], TYPES[case["dtype"]]
    s["x"], s["dy"] = _randn(g, R, D).to(t), _randn(g, R, D).to(t)
    s["seed"], s["offset"] = 0x5DEECE66D1234567 ^ (seed * 0x9E3779B1 % 2**62), (seed % 1000) * 1_000_003
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    return {"logprobs": _logprobs, "logprobs_train": _logprobs_train, "recurrence_train": _recurrence_train,
            "recurrence_step": _recurrence_step, "dropout": _dropout_both}[s["op"]](s)


def _run_own(s):
    from rnn_joint_network_02_b200 import frnnt
    op = s["op"]
    if op == "logprobs":
        r = frnnt.token_logprobs(s["logits"], s["tokens"], top=s["top"], check=False)
        return dict(logp=r.logp, entropy=r.entropy, lse=r.lse, top_logp=r.top_logp, top_ids=r.top_ids)
    if op == "logprobs_train":
        r = frnnt.token_logprobs(s["logits"], s["tokens"], check=False)
        d = frnnt.token_logprobs_bwd(s["logits"], s["tokens"], r, dlogp=s["dlogp"], dentropy=s["dentropy"], check=False)
        return dict(logp=r.logp, entropy=r.entropy, dlogits=d)
    if op == "recurrence_train":
        r = frnnt.recurrence(s["x"], s["gate"], lengths=s["lengths"], h0=s["h0"], check=False)
        d = frnnt.recurrence_bwd(s["x"], s["gate"], r, s["dh"], lengths=s["lengths"], dh_last=s["dh_last"], check=False)
        return dict(h=r.h, h_last=r.h_last, dx=d["dx"], dgate=d["dgate"], dh0=d["dh0"])
    if op == "recurrence_step":
        h, state = frnnt.recurrence_step(s["x"], s["gate"], s["state"], parent=s["parent"], advance=s["advance"], check=False)
        return dict(h=h, state=state)
    return dict(y=frnnt.dropout(s["x"], s["p"], s["seed"], offset=s["offset"]),
                dx=frnnt.dropout(s["dy"], s["p"], s["seed"], offset=s["offset"]))


def _softmax_parts(logits):
    z = logits.float()
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    lse = m + torch.log(total)
    lp = z - lse
    p = e / total
    entropy = -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(1)
    return lse, lp, p, entropy


def _logprobs(s):
    lse, lp, _, entropy = _softmax_parts(s["logits"])
    out = dict(logp=lp.gather(1, s["tokens"].long()) if s["tokens"] is not None else None, entropy=entropy, lse=lse[:, 0],
               top_logp=None, top_ids=None)
    if s["top"]:
        values, ids = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True)   # ties: the lowest index first
        out["top_logp"] = values[:, :s["top"]] - lse
        out["top_ids"] = ids[:, :s["top"]].to(torch.int32)
    return out


def _logprobs_train(s):
    _, lp, p, entropy = _softmax_parts(s["logits"])
    tokens = s["tokens"].long()
    d = -p * s["dlogp"].sum(1, keepdim=True) - s["dentropy"][:, None] * p * (lp + entropy[:, None])
    d.scatter_add_(1, tokens, s["dlogp"])
    return dict(logp=lp.gather(1, tokens), entropy=entropy, dlogits=d.to(s["logits"].dtype))


def _sigmoids(gate):
    """sigmoid(gate) and sigmoid(-gate), each to full relative precision."""
    u = torch.exp(-gate.abs())
    big, small = 1 / (1 + u), u / (1 + u)
    return torch.where(gate >= 0, big, small), torch.where(gate >= 0, small, big)


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t from h_{-1} = 0 along dim 1, by doubling: after each round step t holds 2x as many steps' effect."""
    step, T = 1, a.shape[1]
    while step < T:
        b = torch.cat([b[:, :step], b[:, step:] + a[:, step:] * b[:, :-step]], 1)
        a = torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], 1)
        step *= 2
    return b


def _recurrence_train(s):
    x, gate = s["x"].float(), s["gate"].float()
    B, T, D = x.shape
    keep, take = _sigmoids(gate)
    if s["lengths"] is not None:
        live = (torch.arange(T, device=x.device)[None, :] < s["lengths"][:, None])[:, :, None]
    else:
        live = torch.ones(B, T, 1, dtype=torch.bool, device=x.device)
    a = torch.where(live, keep, torch.ones_like(keep))
    b = torch.where(live, take * x, torch.zeros_like(x))
    b[:, 0] += a[:, 0] * s["h0"]
    h = _scan(a, b)
    before = torch.cat([s["h0"][:, None], h[:, :-1]], 1)
    g = torch.where(live, s["dh"].float(), torch.zeros_like(x))
    g[:, -1] += s["dh_last"]
    after = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    g = _scan(after.flip(1), g.flip(1)).flip(1)
    zero = torch.zeros((), device=x.device)
    t = s["x"].dtype
    return dict(h=torch.where(live, h, zero).to(t), h_last=h[:, -1], dx=torch.where(live, g * take, zero).to(t),
                dgate=torch.where(live, g * (before - x) * keep * take, zero).to(t), dh0=a[:, 0] * g[:, 0])


def _recurrence_step(s):
    keep, take = _sigmoids(s["gate"].float())
    before = s["state"][s["parent"].long()]
    state = torch.where(s["advance"][:, None], keep * before + take * s["x"].float(), before)
    return dict(h=state.to(s["x"].dtype), state=state)


def _philox_words(n, seed, offset):
    """Philox4x32-10 (Salmon et al., "Parallel Random Numbers: As Easy as 1, 2, 3"): four 32-bit words of each of n counters offset, offset + 1, ..."""
    low = 0xFFFFFFFF
    c = torch.arange(n, dtype=torch.int64, device="cuda") + offset
    c0, c1, c2, c3 = c & low, (c >> 32) & low, torch.zeros_like(c), torch.zeros_like(c)
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        p, q = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((q >> 32) & low) ^ c1 ^ k0, q & low, ((p >> 32) & low) ^ c3 ^ k1, p & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack([c0, c1, c2, c3], 1)


def _kept(shape, p, seed, offset):
    """Which elements stay: 16 random bits each, eight elements a counter, against p in 65536ths; and the scale of what stays."""
    n = math.prod(shape)
    w = _philox_words((n + 7) // 8, seed, offset)
    bits = torch.stack([w & 0xFFFF, w >> 16], 2).reshape(-1)[:n].view(shape)
    limit = int(p * 65536 + 0.5)
    return bits >= limit, 65536 / (65536 - limit)


def _dropout_both(s):
    stay, scale = _kept(s["x"].shape, s["p"], s["seed"], s["offset"])
    zero = torch.zeros((), device="cuda")
    return {k: torch.where(stay, s[i].float() * scale, zero).to(s[i].dtype) for k, i in (("y", "x"), ("dx", "dy"))}


# ------------------------------------------------------------------ what it cannot do without
def work(case):
    op, e = case["op"], SIZE[case["dtype"]]
    if op == "logprobs":
        N, V, K, top = case["N"], case["V"], case["K"], case["top"]
        return dict(bytes=N * V * e + N * (8 * K + 8 * top + 8), flops=5 * N * V)
    if op == "logprobs_train":
        N, V, K = case["N"], case["V"], case["K"]
        return dict(bytes=2 * N * V * e + N * (12 * K + 8), flops=11 * N * V)
    if op == "recurrence_train":
        B, T, D = case["B"], case["T"], case["D"]
        full, some = B * T * D, B * T * D * (0.75 if case["ragged"] else 1.0)
        return dict(bytes=int(3 * e * some + 3 * e * full) + 16 * B * D, flops=int(24 * some))
    if op == "recurrence_step":
        N, D = case["N"], case["D"]
        return dict(bytes=N * D * (3 * e + 8) + 5 * N, flops=8 * N * D)
    n = case["R"] * case["D"]
    return dict(bytes=4 * e * n, flops=4 * n)


# ------------------------------------------------------------------ the definition, in 64 bits
def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("logprobs", "logprobs_train"):
        return _exact_logprobs(s, op)
    if op == "recurrence_train":
        return _exact_recurrence(s)
    if op == "recurrence_step":
        x, w, old = s["x"].double(), s["gate"].double().neg().exp(), s["state"].double()
        new = torch.stack([(old[j] + w[n] * x[n]) / (1 + w[n]) if go else old[j]
                           for n, (j, go) in enumerate(zip(s["parent"].tolist(), s["advance"].tolist()))])
        return dict(h=new, state=new)
    return _exact_dropout(s)


def _exact_logprobs(s, op):
    N, V = s["logits"].shape
    keys = ["logp", "entropy", "lse", "top_logp"] if op == "logprobs" else ["logp", "entropy", "dlogits"]
    got = {k: [] for k in keys}
    step = max(1, (1 << 25) // V)
    for n in range(0, N, step):
        at = slice(n, min(N, n + step))
        z = s["logits"][at].double()
        lse = torch.logsumexp(z, 1)
        p = torch.exp(z - lse[:, None])
        entropy = lse - torch.nansum(p * z, 1)        # 0 * -inf of a forbidden entry counts nothing
        got["entropy"].append(entropy)
        if s["tokens"] is not None:
            tok = s["tokens"][at].long()
            got["logp"].append(torch.gather(z, 1, tok) - lse[:, None])
        if op == "logprobs":
            got["lse"].append(lse)
            if s["top"]:
                got["top_logp"].append(torch.topk(z, s["top"], 1).values - lse[:, None])
        else:
            d = torch.zeros_like(z)
            for k in range(tok.shape[1]):
                one = torch.zeros_like(z)
                one[torch.arange(tok.shape[0], device=z.device), tok[:, k]] = 1
                d += s["dlogp"][at, k, None].double() * (one - p)
            d += s["dentropy"][at, None].double() * p * (lse[:, None] - z - entropy[:, None])
            got["dlogits"].append(d)
    out = {k: torch.cat(v) if v else None for k, v in got.items()}
    if op == "logprobs":
        out["top_ids"] = None
    return out


def _exact_recurrence(s):
    x, w = s["x"].double(), s["gate"].double()
    B, T, D = x.shape
    ends = s["lengths"].tolist() if s["lengths"] is not None else [T] * B
    live = torch.tensor([[float(t < e) for e in ends] for t in range(T)], device=x.device, dtype=torch.float64)[:, :, None]
    a = torch.sigmoid(w)
    h, past = s["h0"].double(), torch.empty_like(x)
    hs = torch.empty_like(x)
    for t in range(T):
        past[:, t] = h
        h = h + live[t] * (1 - a[:, t]) * (x[:, t] - h)
        hs[:, t] = h * live[t]
    g, dx, dgate = s["dh_last"].double(), torch.empty_like(x), torch.empty_like(x)
    for t in range(T - 1, -1, -1):
        on = live[t]
        g = g + on * s["dh"][:, t].double()
        dx[:, t] = on * g * (1 - a[:, t])
        dgate[:, t] = on * g * (past[:, t] - x[:, t]) * a[:, t] * (1 - a[:, t])
        g = torch.where(on > 0, g * a[:, t], g)
    return dict(h=hs, h_last=h, dx=dx, dgate=dgate, dh0=g)


def _exact_dropout(s):
    shape = tuple(s["x"].shape)
    n = math.prod(shape)
    m = np.uint64(0xFFFFFFFF)
    half = np.uint64(32)
    at = np.arange((n + 7) // 8, dtype=np.uint64) + np.uint64(s["offset"])
    v = [at & m, at >> half, np.zeros_like(at), np.zeros_like(at)]
    key = [s["seed"] % 2**32, s["seed"] // 2**32 % 2**32]
    for turn in range(10):
        a, b = v[0] * np.uint64(0xD2511F53), v[2] * np.uint64(0xCD9E8D57)
        k = [np.uint64((key[i] + turn * w) % 2**32) for i, w in ((0, 0x9E3779B9), (1, 0xBB67AE85))]
        v = [(b >> half) ^ v[1] ^ k[0], b & m, (a >> half) ^ v[3] ^ k[1], a & m]
    words = np.stack(v, 1).astype("<u4")
    r = np.ascontiguousarray(words).view("<u2").reshape(-1)[:n].reshape(shape)
    limit = math.floor(s["p"] * 65536 + 0.5)
    factor = torch.from_numpy((r >= limit) * (65536.0 / (65536 - limit))).to("cuda")
    return dict(y=s["x"].double() * factor, dx=s["dy"].double() * factor)
