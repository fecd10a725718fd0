"""Plain 64-bit attention over an element mask: the definition, on the CPU, for the tests of the masked forms.

``forward(q, k, v, visible, scale)`` takes ``q [B,Hq,Sq,D]``, ``k``/``v [B,Hkv,Sk,D]`` and a bool ``visible`` that
broadcasts to ``[B,Hq,Sq,Sk]``, and returns fp64 ``(o, lse)``; rows without keys are 0 and -inf.  ``backward`` adds
an upstream gradient and returns ``(dq, dk, dv)`` by the formulas of the softmax's Jacobian.
"""
import numpy as np
import torch


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def window_mask(Sq, Sk, causal, window, sinks):
    """bool [Sq, Sk]: j <= p and (p - j < window or j < sinks), p = i + Sk - Sq (causal 1) or i (causal 2)."""
    p = np.arange(Sq)[:, None] + (Sk - Sq if causal == 1 else 0)
    j = np.arange(Sk)[None, :]
    return (j <= p) & ((p - j < window) | (j < sinks))


def _logits(q, k, visible, scale):
    G = q.shape[1] // k.shape[1]
    s = np.einsum("bhid,bhjd->bhij", q, np.repeat(k, G, axis=1)) * scale
    return np.where(np.broadcast_to(visible, s.shape), s, -np.inf)


def _softmax(s):
    top = s.max(-1, keepdims=True, initial=-np.inf)
    top = np.where(np.isinf(top), 0.0, top)
    e = np.exp(s - top)
    z = e.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (top + np.log(z))[..., 0]
    return e / np.where(z > 0, z, 1.0), lse


def forward(q, k, v, visible, scale):
    q, k, v = f64(q), f64(k), f64(v)
    p, lse = _softmax(_logits(q, k, visible, scale))
    return p @ np.repeat(v, q.shape[1] // k.shape[1], axis=1), lse


def backward(q, k, v, do, visible, scale):
    q, k, v, do = f64(q), f64(k), f64(v), f64(do)
    B, Hq, Sq, D = q.shape
    Hkv, Sk = k.shape[1:3]
    G = Hq // Hkv
    p, _ = _softmax(_logits(q, k, visible, scale))
    kk, vv = np.repeat(k, G, axis=1), np.repeat(v, G, axis=1)
    dp = do @ vv.swapaxes(-1, -2)
    ds = p * (dp - (p * dp).sum(-1, keepdims=True)) * scale
    shared = lambda x: x.reshape(B, Hkv, G, Sk, D).sum(2)  # noqa: E731
    return ds @ kk, shared(ds.swapaxes(-1, -2) @ q), shared(p.swapaxes(-1, -2) @ do)
