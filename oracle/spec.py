"""Oracle for a step that checks drafted tokens (speculative decoding).

TEST INFRASTRUCTURE ONLY (see the package docstring): plain, slow, float64.

* ``tree_attention_request``: every node of a tree sees the cached prefix, its
  ancestors and itself (scale 1/sqrt(hd), q head h reads KV head h // group).
* ``layer_step_tree``: the layer of ``oracle.layer`` over a batch whose
  requests are trees: node i of a request with c cached tokens is rotated for
  position c + depth(i), stored at position c + i, and attends as above.
* ``verify``: acceptance of the drafted tokens from given uniform numbers,
  literally: a refusal replaces the target's distribution p by
  norm(max(0, p - q)), or, for a token proposed for certain, takes the token
  out of p (Leviathan et al., "Fast Inference from Transformers via
  Speculative Decoding", 2023; Miao et al., "SpecInfer", 2024).
* ``compact``: the accepted path's cache entries move behind the prefix.
"""

from __future__ import annotations

import math

import numpy as np

from .layer import gather_kv, linear, page_slot, rms_norm, rope, silu


def ancestors(parent) -> np.ndarray:
    """[n, n] bool: node i sees node j (itself or an ancestor)."""
    n = len(parent)
    see = np.zeros((n, n), dtype=bool)
    for i in range(n):
        j = i
        while j >= 0:
            see[i, j] = True
            j = int(parent[j])
    return see


def depths(parent) -> np.ndarray:
    d = np.zeros(len(parent), dtype=np.int64)
    for i, up in enumerate(parent):
        d[i] = 0 if up < 0 else d[up] + 1
    return d


def tree_attention_request(q: np.ndarray, K: np.ndarray, V: np.ndarray, parent):
    """q [n, Hq, hd]; K, V [kv, Hkv, hd], the last n of them the nodes' own.
    Returns (o [n, Hq, hd], A, B): the output, A = sum_j p_ij |v_j| and B =
    max_j sum_d |q_id k_jd| / sqrt(hd) over visible j (for error bounds)."""
    n, Hq, hd = q.shape
    kv, Hkv, _ = K.shape
    see = np.ones((n, kv), dtype=bool)
    see[:, kv - n:] = ancestors(parent)
    o, A, B = np.empty((n, Hq, hd)), np.empty((n, Hq, hd)), np.empty((n, Hq))
    for h in range(Hq):
        k, v = K[:, h // (Hq // Hkv)], V[:, h // (Hq // Hkv)]
        for i in range(n):
            kk, vv = k[see[i]], v[see[i]]
            s = kk @ q[i, h] / math.sqrt(hd)
            e = np.exp(s - s.max())
            p = e / e.sum()
            o[i, h], A[i, h] = p @ vv, p @ np.abs(vv)
            B[i, h] = np.max(np.abs(kk) @ np.abs(q[i, h])) / math.sqrt(hd)
    return o, A, B


def layer_step_tree(shape, w, pool, qo_indptr, kv_len, bt_indptr, bt, parent, x):
    """oracle.layer.layer_step for trees; ``parent`` [T], within each request."""
    Hq, Hkv, hd, F, eps = (shape[k] for k in ("n_q_heads", "n_kv_heads", "head_dim", "d_ff", "rms_eps"))
    T = int(qo_indptr[-1])
    qkv = linear(rms_norm(x, w["g_attn"], eps), w["w_qkv"])
    q = qkv[:, :Hq * hd].reshape(T, Hq, hd)
    k = qkv[:, Hq * hd:(Hq + Hkv) * hd].reshape(T, Hkv, hd)
    v = qkv[:, (Hq + Hkv) * hd:].reshape(T, Hkv, hd)
    if shape["qk_norm"]:
        q, k = rms_norm(q, w["g_q"], eps), rms_norm(k, w["g_k"], eps)
    o, written = np.empty((T, Hq, hd)), []
    for r in range(len(kv_len)):
        a, b = int(qo_indptr[r]), int(qo_indptr[r + 1])
        n, c = b - a, int(kv_len[r]) - (b - a)
        par = [int(x) for x in parent[a:b]]
        pos = c + depths(par)
        qr, kr = rope(q[a:b], pos[:, None], shape["rope_theta"]), rope(k[a:b], pos[:, None], shape["rope_theta"])
        table = bt[bt_indptr[r]:bt_indptr[r + 1]]
        for i in range(n):
            page, slot = page_slot(table, c + i)
            pool[page, 0, :, slot], pool[page, 1, :, slot] = kr[i], v[a + i]
            written.append((page, slot))
        K, V = gather_kv(pool, table, c + n)
        o[a:b] = tree_attention_request(qr, K, V, par)[0]
    h = x + linear(o.reshape(T, Hq * hd), w["w_o"])
    gu = linear(rms_norm(h, w["g_ffn"], eps), w["w_gate_up"])
    return {"y": h + linear(silu(gu[:, :F]) * gu[:, F:], w["w_down"]), "o": o.reshape(T, -1), "written": written}


def target_row(logits: np.ndarray, temperature: float) -> np.ndarray:
    """softmax(logits / temperature); NaN and -inf have probability 0, +inf
    entries share everything; all zero if there is nothing else."""
    z = np.where(np.isnan(logits), -np.inf, logits.astype(np.float64))
    top = z.max()
    if top == -np.inf:
        return np.zeros_like(z)
    below = z != top
    e = np.ones_like(z)
    e[below] = np.exp((z[below] - top) / temperature)
    return e / e.sum()


def verify(logits, tokens, probs, parent, temperature, u_accept, u_final, max_path):
    """One request: logits [n, V] float64, tokens [n], probs [n, V] or None.
    Returns (path, next token, margins): the smallest distances, in
    probability, of an acceptance test from its border and of the last draw
    from the borders of its token."""
    n, V = logits.shape
    path, margin, last = [0], np.inf, np.inf
    while True:
        cur = path[-1]
        kids = [i for i in range(1, n) if parent[i] == cur] if len(path) < max_path else []
        if temperature == 0:
            z = np.where(np.isnan(logits[cur]), -np.inf, logits[cur])
            top = int(np.argmax(z))
            hit = [i for i in kids if tokens[i] == top]
            if not hit:
                return path, top, (margin, last)
            path.append(hit[0])
            continue
        p = target_row(logits[cur], temperature)
        left, hit = p.copy(), None
        for i in kids:
            x = int(tokens[i])
            if not 0 <= x < V:
                continue
            qx = 1.0 if probs is None else float(probs[cur, x])
            margin = min(margin, abs(left[x] - u_accept[i] * qx)) if left[x] > 0 else margin
            if u_accept[i] * qx < left[x]:
                hit = i
                break
            if probs is None:
                left[x] = 0.0
            else:
                left = np.maximum(0.0, left - probs[cur])
            left = left / left.sum() if left.sum() > 0 else left
        if hit is not None:
            path.append(hit)
            continue
        left = left if left.sum() > 0 else p
        if left.sum() == 0:
            return path, 0, (margin, last)
        cum = np.cumsum(left)
        t = u_final * cum[-1]
        tok = int(np.argmax(cum > t))
        last = min(abs(cum[tok] - t), abs(t - cum[tok - 1]) if tok else np.inf)
        return path, tok, (margin, last)


def compact(pool, qo_indptr, kv_len, bt_indptr, bt, path):
    """pool [P][2][Hkv][16][hd], in place; path: one list of node indices per
    request.  Returns the new lengths."""
    new = []
    for r, nodes in enumerate(path):
        c = int(kv_len[r]) - int(qo_indptr[r + 1] - qo_indptr[r])
        table = bt[bt_indptr[r]:bt_indptr[r + 1]]
        moved = [pool[page_slot(table, c + f)[0], :, :, page_slot(table, c + f)[1]].copy() for f in nodes]
        for k, x in enumerate(moved):
            page, slot = page_slot(table, c + k)
            pool[page, :, :, slot] = x
        new.append(c + len(nodes))
    return np.array(new, dtype=np.int32)
