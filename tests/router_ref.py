"""Plain 64-bit references (numpy, no code of the library) of the linear layer, the
scored router and the gradients of the router, and the error bounds of the kernels.

Bounds.  One rounding to a type is off by at most half a step of it relative to the
value: 2^-8 (bf16), 2^-24 (fp32).  A product accumulated in fp32 over K terms by the
tensor cores is off by at most K 2^-23 sum|a b| (each addition may truncate instead of
rounding: one step, 2^-23, of a partial sum that is at most sum|a b|)."""
import math

import numpy as np

BF16, F32 = 2.0 ** -8, 2.0 ** -24


def act(kind, u):
    if kind == 1:
        return np.maximum(u, 0)
    if kind == 2:
        return u * sigmoid(u)
    if kind == 3:
        return 0.5 * u * (1 + erf(u / math.sqrt(2)))
    return u


def dact(kind, u):
    if kind == 1:
        return (u > 0).astype(np.float64)
    if kind == 2:
        p = sigmoid(u)
        return p * (1 + u * (1 - p))
    if kind == 3:
        return 0.5 * (1 + erf(u / math.sqrt(2))) + u * np.exp(-0.5 * u * u) / math.sqrt(2 * math.pi)
    return np.ones_like(u)


erf = np.vectorize(math.erf, otypes=[np.float64])


def sigmoid(u):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-u))


def linear(x, W, bias, residual, kind, out_step):
    """(out, u, bound of out, bound of u before its own rounding)."""
    u = x @ W
    err = x.shape[1] * 2.0 ** -23 * (np.abs(x) @ np.abs(W))
    if bias is not None:
        u = u + bias
        err = err + F32 * np.abs(u)
    h = act(kind, u)
    # |act'| <= 1.13 for every kind; the function itself in fp32: a few roundings of
    # values up to |u| (8 of them bounds exp, a division and two products)
    e = 1.13 * err + (8 * F32 * np.abs(u) if kind else 0)
    out = h if residual is None else h + residual
    e = e + F32 * np.abs(out)
    return out, u, e * (1 + out_step) + out_step * np.abs(out), err


def linear_backward(dout, x, W, pre, kind, du_step):
    """du, dx, dW, dbias and the bounds of dx, dW, dbias before their own rounding.
    du_step: the relative rounding of the bf16 terms that du goes in as."""
    M, K = x.shape
    N = W.shape[1]
    du = dout * (dact(kind, pre) if kind else 1.0)
    # act' in fp32: values up to 1.13 (1 + |pre|), 10 roundings
    e = 10 * F32 * np.abs(dout) * (1 + np.abs(pre)) if kind else 0.0 * du
    e = e + du_step * np.abs(du)
    terms = 3                                     # du's terms are products of their own
    dx, dW = du @ W.T, x.T @ du
    bx = e @ np.abs(W).T + terms * N * 2.0 ** -23 * (np.abs(du) @ np.abs(W).T)
    bW = np.abs(x).T @ e + terms * M * 2.0 ** -23 * (np.abs(x).T @ np.abs(du))
    bb = (10 * F32 * np.abs(dout) * (1 + np.abs(pre)) if kind else 0.0 * du).sum(0) + M * F32 * np.abs(du).sum(0)
    return dict(du=du, dx=dx, dW=dW, dbias=du.sum(0), bx=bx, bW=bW, bb=bb)


def scores(z, kind):
    """p [E] of one token, masked experts 0, and which are live."""
    z = np.asarray(z, np.float64)
    live = ~(np.isnan(z) | (z == -np.inf))
    z = np.minimum(z, float(np.finfo(np.float32).max))
    p = np.zeros(len(z))
    if not live.any():
        return p, live
    if kind == 1:
        p[live] = sigmoid(z[live])
    else:
        e = np.exp(z[live] - z[live].max())
        p[live] = e / e.sum()
    return p, live


def route(logits, k, kind=0, bias=None, n_groups=1, topk_groups=0, top2=False, renorm=True, scale=1.0):
    """Token by token, by sorting lists: (idx, gate)."""
    T, E = logits.shape
    topk_groups = topk_groups or n_groups
    S = E // n_groups
    idx, gate = np.zeros((T, k), np.int32), np.zeros((T, k))
    for t in range(T):
        p, live = scores(logits[t], kind)
        biased = p if bias is None else p + np.asarray(bias, np.float64)
        key = biased if bias is not None else np.minimum(logits[t].astype(np.float64), 3.4028234663852886e38)
        groups = list(range(n_groups))
        if topk_groups < n_groups:
            value = []
            for g in groups:
                of = sorted((float((biased if top2 else key)[e]) for e in range(g * S, g * S + S) if live[e]),
                            reverse=True)
                value.append(sum(of[:2 if top2 else 1]) if of else -np.inf)
            groups = sorted(groups, key=lambda g: (-value[g], g))[:topk_groups]
        open_ = [e for g in groups for e in range(g * S, g * S + S)]
        order = sorted(open_, key=lambda e: (0, -key[e], e) if live[e] else (1, 0, e))[:k]
        w = p[order]
        if renorm:
            s = w.sum()
            w = w / s if s > 0 else 0 * w
        idx[t], gate[t] = order, scale * w
    return idx, gate


def route_backward(dgate, logits, idx, kind=0, renorm=True, scale=1.0):
    """(dlogits, bound): by the formula, token by token."""
    T, E = logits.shape
    dz, bound = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        p, _ = scores(logits[t], kind)
        sel = [j for j in range(idx.shape[1]) if 0 <= idx[t, j] < E]
        c = np.array([scale * float(dgate[t, j]) for j in sel])
        e = np.array([idx[t, j] for j in sel], int)
        size = np.abs(c).sum()
        if renorm:
            S = p[e].sum()
            dp = (c - (c * p[e]).sum() / S) / S if S > 0 else 0 * c
            size = 2 * size / S if S > 0 else 0.0
        else:
            dp = c
        full = np.zeros(E)
        full[e] = dp
        dz[t] = full * p * (1 - p) if kind == 1 else p * (full - (p * full).sum())
        # E + 32 roundings of values up to 2 size p_e
        bound[t] = (E + 32) * 2 * F32 * 2 * size * p
    return dz, bound


def combine_backward(dout, y, row_of, gate, dy):
    """(dy, dgate, bound of dgate); dy: the buffer's values before the call."""
    T, k = gate.shape
    dy, dgate, bound = dy.copy(), np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = row_of[t * k + j]
            if 0 <= r < T * k:
                dy[r] = gate[t, j] * dout[t]
                dgate[t, j] = (dout[t] * y[r]).sum()
                bound[t, j] = dout.shape[1] * F32 * np.abs(dout[t] * y[r]).sum()
    return dy, dgate, bound
