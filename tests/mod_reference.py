"""Plain float64 attention with modified scores, one head at a time, for the tests of the
_mod calls: the definition written out row by row from the mask's words."""
import numpy as np


def visible(Nq, Nk, causal, prefix=None, doc_ids=None):
    """[Nq, Nk] truth values: key j is visible to query row i at position i + Nk - Nq."""
    p = np.arange(Nq)[:, None] + (Nk - Nq)
    j = np.arange(Nk)[None, :]
    seen = np.ones((Nq, Nk), dtype=bool)
    if causal:
        seen = j <= p
        if prefix is not None:
            seen = seen | (j < prefix)
    if doc_ids is not None:
        doc_ids = np.asarray(doc_ids)
        # a run number per token: equal ids apart from each other are different documents
        run = np.concatenate([[0], np.cumsum(doc_ids[1:] != doc_ids[:-1])]) if Nk else doc_ids
        run = np.where(doc_ids < 0, -1, run)
        at = np.arange(Nq) + (Nk - Nq)
        mine = np.where(at >= 0, run[np.maximum(at, 0)], -1)
        seen = seen & (mine[:, None] == run[None, :]) & (run[None, :] >= 0)
    return seen


def scores(Q, K, scale, softcap=0.0, slope=None):
    """(x, dx/dz): the modified scores and the cap's derivative."""
    Nq, Nk = Q.shape[0], K.shape[0]
    z = scale * (Q @ K.T)
    dz = np.ones_like(z)
    if softcap:
        t = np.tanh(z / softcap)
        z, dz = softcap * t, 1 - t * t
    if slope is not None:
        p = np.arange(Nq)[:, None] + (Nk - Nq)
        z = z - slope * np.abs(p - np.arange(Nk)[None, :])
    return z, dz


def forward(Q, K, V, scale, seen, softcap=0.0, slope=None):
    """(O, LSE, P) of one head; rows that see nothing: O = 0, LSE = -inf."""
    x, _ = scores(Q, K, scale, softcap, slope)
    x = np.where(seen, x, -np.inf)
    m = x.max(axis=1, initial=-np.inf)
    e = np.exp(x - np.where(np.isfinite(m), m, 0.0)[:, None])
    l = e.sum(axis=1)
    P = e / np.where(l == 0, 1.0, l)[:, None]
    with np.errstate(divide="ignore"):
        return P @ V, np.where(l == 0, -np.inf, m + np.log(l)), P


def backward(Q, K, V, dO, scale, seen, softcap=0.0, slope=None, O=None):
    """(dQ, dK, dV) of one head; O, if given, is the rounded output D is formed from."""
    x, dz = scores(Q, K, scale, softcap, slope)
    O_exact, _, P = forward(Q, K, V, scale, seen, softcap, slope)
    D = (dO * (O_exact if O is None else O)).sum(axis=1, keepdims=True)
    dS = P * (dO @ V.T - D) * dz
    return scale * dS @ K, scale * dS.T @ Q, P.T @ dO
