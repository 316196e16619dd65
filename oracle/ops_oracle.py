"""fp64 CPU oracle for the operators beside the loss: token log-probabilities,
the gated linear recurrence, and dropout from a counter-based generator.

TEST INFRASTRUCTURE ONLY, like ``rnnt_oracle``: nothing on the product path may
import, call or execute it, and it shares no code with the CUDA library.  The
definitions are written out, a row or a time step at a time.

Beside each value these functions also return how far an implementation may be
off that computes in fp32 and rounds the result once (``*_tol``, same shape).
The fp32 part follows the computation: every elementary operation is charged
``UNIT`` relative to what it produces, and errors already made are carried
through the same formulas.
"""

from __future__ import annotations

import numpy as np

NO_TOKEN = -1
# Relative error charged to one elementary function in fp32: a hardware exp2,
# reciprocal or logarithm is good to 2^-22, its scaled argument and the
# roundings of two products and a sum around it are 2^-24 each; 2^-20 covers
# them with the two orders in which sums may be taken.
UNIT = 2.0 ** -20
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


# ------------------------------------------------------------------ token log-probabilities
def _row_tolerances(row, m, ls, V):
    """Of a row's lse, entropy, and log-probabilities (an array, one a column).
    Magnitudes count where they carry probability: a value that masks a column
    (-inf, or the type's lowest) enters no sum, and a shift of all logits enters
    none either, since their differences from the maximum are formed first."""
    if not np.isfinite(m):    # an empty row's values are exact, one with NaN or +inf has none
        return 0.0, 0.0, np.zeros_like(row)
    d, p = np.where(row > -np.inf, m - row, 0.0), np.exp((row - m) - ls)
    # A term of the sum, exp(-d): the difference, its product with log2 e and that constant are rounded, 3 * 2^-24 d in
    # the exponent; the function itself, and the orders of summing, are UNIT each.  The sum's relative error is the
    # terms' mean error (at 1000 and more, where p is 0, d is cut off so that 0 times it is 0).
    near = np.minimum(d, 1000.0)
    term = 4 * UNIT + 2.0 ** -22 * near
    total = (p * term).sum()
    # its logarithm, and the sum of the maximum and that, rounded once each
    lse_tol = total + 2.0 ** -23 * np.log(V) + 2.0 ** -24 * abs(m + ls) + 2.0 ** -126
    # difference from the maximum, logarithm, and their difference; of columns of any probability
    log_p = total + 2.0 ** -23 * (d + np.log(V) + 1.0)
    # H = log(sum) + sum p d: the terms' errors against d, d's own, the quotient by the sum, and roundings
    mean = (p * near).sum()
    entropy_tol = total * (1 + mean) + (p * near * (term + 2.0 ** -22)).sum() + 2.0 ** -22 * (np.log(V) + mean + 1)
    return lse_tol, entropy_tol, log_p


def token_logprobs(z, tokens=None, top=0):
    """z [N, V] float64 (-inf allowed), tokens [N, K] ints.  Returns a dict: logp
    [N, K], entropy [N], lse [N], top_logp, top_ids [N, top] and logp_tol,
    entropy_tol, lse_tol, top_tol; and lse in two parts, max and log_sum [N],
    since their sum loses the second one where the logits are huge (even in 64
    bits: rows of the type's lowest value)."""
    N, V = z.shape
    K = 0 if tokens is None else tokens.shape[1]
    out = dict(logp=np.zeros((N, K)), entropy=np.zeros(N), lse=np.zeros(N), top_logp=np.zeros((N, top)),
               top_ids=np.zeros((N, top), dtype=np.int64), max=np.zeros(N), log_sum=np.zeros(N))
    tol = dict(logp_tol=np.zeros((N, K)), entropy_tol=np.zeros(N), lse_tol=np.zeros(N), top_tol=np.zeros((N, top)))
    for n in range(N):
        row = z[n]
        # equal values: lowest column first; NaN last
        order = sorted(range(V), key=lambda j: (np.isnan(row[j]), -row[j] if not np.isnan(row[j]) else 0.0, j))
        ids = order[:top]
        given = [] if K == 0 else [int(t) for t in tokens[n]]
        if np.isnan(row).any() or np.isposinf(row).any():
            m, ls, entropy = np.nan, 0.0, np.nan
        elif np.isneginf(row).all():
            m, ls, entropy = -np.inf, 0.0, 0.0
        else:
            m = row.max()
            ls = np.log(np.exp(row - m).sum())
            lp = (row[row > -np.inf] - m) - ls
            entropy = -(np.exp(lp) * lp).sum()
        lse = m + ls
        one = (lambda t: -np.inf if np.isneginf(m) else (row[t] - m) - ls)
        out["lse"][n], out["entropy"][n], out["max"][n], out["log_sum"][n] = lse, entropy, m, ls
        out["top_ids"][n] = ids
        out["top_logp"][n] = [one(j) for j in ids]
        out["logp"][n] = [0.0 if t == NO_TOKEN else one(t) for t in given]
        with np.errstate(invalid="ignore", over="ignore", under="ignore"):
            tol["lse_tol"][n], tol["entropy_tol"][n], near = _row_tolerances(row, m, ls, V)
            tol["logp_tol"][n] = [0.0 if t == NO_TOKEN else near[t] for t in given]
            tol["top_tol"][n] = [near[j] for j in ids]
    out.update(tol)
    return out


def token_logprobs_bwd(z, tokens, fwd, dlogp=None, dentropy=None, dtop=None, dtype="f32"):
    """dz [N, V] and dz_tol [N, V]: sum of the formula's terms, one given token
    and one alternative at a time."""
    N, V = z.shape
    dz, tol = np.zeros((N, V)), np.zeros((N, V))
    for n in range(N):
        lse = fwd["lse"][n]
        if np.isneginf(lse):
            continue
        with np.errstate(invalid="ignore"):
            lp = (z[n] - fwd["max"][n]) - fwd["log_sum"][n]
            p = np.exp(lp)
        safe = np.where(p > 0, lp, 0.0) if not np.isnan(lse) else lp
        # of p, where it is not 0: its exponent's absolute error.  The sum's logarithm has the sum's relative error
        # (that of the log-probability of the maximum, with its roundings); z - lse is rounded at its own size, which
        # is within log(sum) <= ln V of log p's; and two products at theirs
        with np.errstate(invalid="ignore", over="ignore"):
            of_sum = _row_tolerances(z[n], fwd["max"][n], fwd["log_sum"][n], V)[2].min()
            rel = 4 * UNIT + of_sum + 2.0 ** -22 * (np.where(p > 0, np.abs(lp), 0.0) + np.log(V) + 1)
        coef = []
        if dlogp is not None:
            coef += [(int(tokens[n, k]), dlogp[n, k]) for k in range(dlogp.shape[1]) if int(tokens[n, k]) != NO_TOKEN]
        if dtop is not None:
            coef += [(int(fwd["top_ids"][n, i]), dtop[n, i]) for i in range(dtop.shape[1])]
        size = sum(abs(c) for _, c in coef)
        for j, c in coef:
            dz[n, j] += c
            dz[n] -= c * p
            tol[n, j] += 2.0 ** -22 * (abs(c) + size)
        tol[n] += 2 * rel * p * size
        if dentropy is not None:
            H, d = fwd["entropy"][n], dentropy[n]
            dz[n] -= d * p * (safe + H)
            tol[n] += abs(d) * p * (2 * rel * (np.abs(safe) + abs(H) + 1) + fwd["entropy_tol"][n])
        # a p below 2^-126 may count as 0
        gone = 2.0 ** -126 * (1 + size + (0.0 if dentropy is None else 200 * abs(dentropy[n])))
        tol[n] += HALF_STEP[dtype] * (np.abs(dz[n]) + tol[n]) + gone
    return dz, tol


# ------------------------------------------------------------------ gated linear recurrence
def sigmoid(g):
    return np.exp(-np.logaddexp(0.0, -g))


def recurrence(x, gate, lengths=None, h0=None, dtype="f32"):
    """x, gate [B, T, D] -> h, h_last and their tolerances, and past [B, T, D]:
    the state before every step (with past_err, its fp32 error)."""
    B, T, D = x.shape
    h, h_tol = np.zeros((B, T, D)), np.zeros((B, T, D))
    past, past_err = np.zeros((B, T, D)), np.zeros((B, T, D))
    last, last_tol = np.zeros((B, D)), np.zeros((B, D))
    for b in range(B):
        v = np.zeros(D) if h0 is None else h0[b].astype(np.float64).copy()
        e = np.zeros(D)
        for t in range(T if lengths is None else int(lengths[b])):
            a, s = sigmoid(gate[b, t]), sigmoid(-gate[b, t])
            past[b, t], past_err[b, t] = v, e
            e = a * e + UNIT * (a * np.abs(v) + s * np.abs(x[b, t]))
            v = a * v + s * x[b, t]
            h[b, t] = v
            h_tol[b, t] = e + HALF_STEP[dtype] * (np.abs(v) + e)
        last[b], last_tol[b] = v, e + 2.0 ** -24 * np.abs(v)
    return dict(h=h, h_tol=h_tol, h_last=last, h_last_tol=last_tol, past=past, past_err=past_err)


def recurrence_bwd(x, gate, fwd, dh, lengths=None, dh_last=None, dtype="f32"):
    """dx, dgate, dh0 of sum(h dh) + sum(h_last dh_last), each with its _tol."""
    B, T, D = x.shape
    r = {k: np.zeros((B, T, D)) for k in ("dx", "dx_tol", "dgate", "dgate_tol")}
    r.update(dh0=np.zeros((B, D)), dh0_tol=np.zeros((B, D)))
    for b in range(B):
        q = np.zeros(D) if dh_last is None else dh_last[b].astype(np.float64).copy()
        e = np.zeros(D)
        for t in range((T if lengths is None else int(lengths[b])) - 1, -1, -1):
            a, s = sigmoid(gate[b, t]), sigmoid(-gate[b, t])
            g, size = q + dh[b, t], np.abs(q) + np.abs(dh[b, t])
            e = e + UNIT * size
            diff = fwd["past"][b, t] - x[b, t]
            r["dx"][b, t] = s * g
            ex = s * e + UNIT * s * size
            r["dx_tol"][b, t] = ex + HALF_STEP[dtype] * (np.abs(s * g) + ex)
            r["dgate"][b, t] = a * s * diff * g
            ed = fwd["past_err"][b, t] + UNIT * (np.abs(fwd["past"][b, t]) + np.abs(x[b, t]))
            eg = a * s * (np.abs(diff) * (e + UNIT * size) + ed * (np.abs(g) + e))
            r["dgate_tol"][b, t] = eg + HALF_STEP[dtype] * (np.abs(r["dgate"][b, t]) + eg)
            q = a * g
            e = a * e + UNIT * a * size
        r["dh0"][b], r["dh0_tol"][b] = q, e + 2.0 ** -24 * np.abs(q)
    return r


def recurrence_step(x, gate, state, parent=None, advance=None):
    """New state [N, D] of one step and its fp32 error."""
    N = x.shape[0]
    new, err = np.zeros(x.shape), np.zeros(x.shape)
    for n in range(N):
        v = state[n if parent is None else int(parent[n])].astype(np.float64)
        if advance is None or advance[n]:
            a, s = sigmoid(gate[n]), sigmoid(-gate[n])
            err[n] = UNIT * (a * np.abs(v) + s * np.abs(x[n]))
            v = a * v + s * x[n]
        new[n] = v
    return new, err


# ------------------------------------------------------------------ dropout
def philox4x32_10(counter, key):
    """One block: counter and key as sequences of four and two 32-bit words
    ("Parallel Random Numbers: As Easy as 1, 2, 3")."""
    c, k = [int(v) for v in counter], [int(v) for v in key]
    low = 0xFFFFFFFF
    for _ in range(10):
        p, q = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(q >> 32) ^ c[1] ^ k[0], q & low, (p >> 32) ^ c[3] ^ k[1], p & low]
        k = [(k[0] + 0x9E3779B9) & low, (k[1] + 0xBB67AE85) & low]
    return c


def dropout_mask(n, p, seed, offset):
    """Which of n elements stay, and the scale of those that do."""
    limit = int(p * 65536 + 0.5)
    keep = np.zeros(n, dtype=bool)
    for g in range((n + 7) // 8):
        at = (offset + g) % 2 ** 64
        w = philox4x32_10((at & 0xFFFFFFFF, at >> 32, 0, 0), (seed & 0xFFFFFFFF, seed >> 32))
        for j in range(8):
            if g * 8 + j < n:
                keep[g * 8 + j] = ((w[j // 2] >> (16 * (j % 2))) & 0xFFFF) >= limit
    return keep, (65536.0 / (65536 - limit) if limit < 65536 else 0.0)
