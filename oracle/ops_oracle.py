"""float64 CPU reference of the operators on logits and on a solved layer
(test infrastructure only), row by row from their definitions."""
from __future__ import annotations

import math

import numpy as np


# ------------------------------------------------------------------ logits

def token_logprobs(z, tokens, top):
    """z: t x V float64.  dict(lse, logprob, entropy, top_ids, top_logprobs)."""
    t, V = z.shape
    out = dict(lse=np.empty(t), logprob=np.empty(t), entropy=np.empty(t), top_ids=np.full((t, top), -1, np.int64),
               top_logprobs=np.full((t, top), -np.inf))
    for i in range(t):
        row = z[i]
        if np.isnan(row).any() or np.isposinf(row).any():
            for k in ("lse", "logprob", "entropy"):
                out[k][i] = np.nan
            if tokens[i] < 0:
                out["logprob"][i] = 0.0
            out["top_logprobs"][i] = np.nan
            continue
        alive = np.flatnonzero(row > -np.inf)
        if alive.size == 0:
            lse, H = -np.inf, 0.0
        else:
            x = row[alive]
            m = x.max()
            s = np.exp(x - m).sum()
            lse = m + math.log(s)
            q = np.exp(x - lse)
            H = float(-(q * (x - lse)).sum())
        out["lse"][i], out["entropy"][i] = lse, H
        tok = int(tokens[i])
        out["logprob"][i] = 0.0 if tok < 0 else np.nan if tok >= V else (
            -np.inf if row[tok] == -np.inf else row[tok] - lse)
        order = alive[np.lexsort((alive, -row[alive]))][:top]
        out["top_ids"][i, :order.size] = order
        out["top_logprobs"][i, :order.size] = row[order] - lse
    return out


def distill(z, ids, teacher, T=1.0, tail=False, weights=None):
    """(loss, grad, scale): scale[i, j] = weight / T (q_j + the mass the teacher gives j), which
    rounding errors of the gradient are measured against."""
    t, V = z.shape
    loss, grad, scale = np.zeros(t), np.zeros((t, V)), np.zeros((t, V))
    for i in range(t):
        w = 1.0 if weights is None else float(weights[i])
        if w == 0.0:
            continue
        a = z[i] / T
        a = a - a.max()
        q = np.exp(a) / np.exp(a).sum()
        lq = a - math.log(np.exp(a).sum())
        keep = [(int(j), float(v) / T) for j, v in zip(ids[i], teacher[i]) if 0 <= j < V]
        if not tail:
            keep = [(j, v) for j, v in keep if v > -np.inf]
        p = np.zeros(V)
        if tail:
            kl = 0.0
            for j, v in keep:
                p[j] += math.exp(v)
                if v > -np.inf:
                    kl += math.exp(v) * (v - lq[j])
            rest = 1.0 - p.sum()
            listed = np.zeros(V, bool)
            listed[[j for j, _ in keep]] = True
            if rest < 2.0 ** -20 or listed.all():
                rest = 0.0
            g = np.where(listed, q - p, q)
            share = 0.0
            if rest > 0:
                # the unlisted mass by its own maximum: it may be far below what float64 holds about the row's
                top = lq[~listed].max()
                if top == -np.inf:
                    kl, share = np.inf, 0.0   # nothing to move: no gradient but the listed tokens'
                else:
                    e = np.exp(np.where(listed, -np.inf, lq - top))
                    kl += rest * (math.log(rest) - top - math.log(e.sum()))
                    share = rest * (e / e.sum())
                g = np.where(listed, g, q - share)
        elif not keep:
            continue
        else:
            m = max(v for _, v in keep)
            tot = sum(math.exp(v - m) for _, v in keep)
            kl = 0.0
            for j, v in keep:
                lp = v - m - math.log(tot)
                p[j] += math.exp(lp)
                kl += math.exp(lp) * (lp - lq[j])
            g, share = q - p, 0.0
        loss[i] = w * kl
        grad[i] = w / T * g
        scale[i] = w / T * (q + share + p)
    return loss, grad, scale


# ------------------------------------------------------------------ a solved layer's product

def layer_entries(codes, E, group):
    """Entries (m x n) and each column's group."""
    E = np.asarray(E, np.float64)
    m = codes.shape[0]
    e = E[codes].reshape(m, -1)
    n = e.shape[1]
    g = group if 0 < group < n else n
    return e, np.arange(n) // g


def layer_weights(codes, E, scale, offset, group=0):
    e, col = layer_entries(codes, E, group)
    a = np.asarray(scale, np.float64).reshape(e.shape[0], -1)[:, col]
    w = a * e
    if offset is not None:
        w = w + np.asarray(offset, np.float64).reshape(e.shape[0], -1)[:, col]
    return w


def act(name, u):
    if name is None:
        return u
    if name == "relu":
        return np.where(u < 0, 0.0, u)
    if name == "silu":
        return u / (1 + np.exp(-u))
    if name == "gelu":
        return 0.5 * u * (1 + np.vectorize(math.erf)(u / math.sqrt(2)))
    return 0.5 * u * (1 + np.tanh(math.sqrt(2 / math.pi) * (u + 0.044715 * u ** 3)))


def act_slope(name, u):
    if name is None:
        return np.ones_like(u)
    if name == "relu":
        return (u > 0).astype(np.float64)
    if name == "silu":
        q = 1 / (1 + np.exp(-u))
        return q * (1 + u * (1 - q))
    if name == "gelu":
        return 0.5 * (1 + np.vectorize(math.erf)(u / math.sqrt(2))) + u * np.exp(-0.5 * u * u) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    th = np.tanh(c * (u + 0.044715 * u ** 3))
    return 0.5 * (1 + th) + 0.5 * u * (1 - th * th) * c * (1 + 3 * 0.044715 * u * u)


def linear(x, w, bias=None, name=None, residual=None):
    """(y, pre)"""
    u = x @ w.T
    if bias is not None:
        u = u + bias
    y = act(name, u)
    return (y if residual is None else y + residual), u


def linear_backward(dy, x, codes, E, scale, offset, group=0, pre=None, name=None):
    du = dy * (act_slope(name, pre) if name is not None else 1.0)
    w = layer_weights(codes, E, scale, offset, group)
    e, col = layer_entries(codes, E, group)
    dW = du.T @ x
    G = int(col[-1]) + 1
    da, do = np.zeros((w.shape[0], G)), np.zeros((w.shape[0], G))
    for g in range(G):
        da[:, g] = (dW * e)[:, col == g].sum(1)
        do[:, g] = dW[:, col == g].sum(1)
    return dict(dx=du @ w, dscale=da.reshape(np.shape(scale)), doffset=do.reshape(np.shape(scale)), dbias=du.sum(0))
