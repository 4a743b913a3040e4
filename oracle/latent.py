"""Float64 oracle of the latent cache's operators and of the descriptors built
from lengths: plain NumPy, written from the definitions in include/mb.h."""

import numpy as np

PAGE = 16
ROPE = 64


def rope64(x, pos, theta):
    """Rotate-half RoPE of the last axis (64 numbers) at position `pos`."""
    half = ROPE // 2
    angle = pos * theta ** (-2.0 * np.arange(half) / ROPE)
    a, b = x[..., :half], x[..., half:]
    return np.concatenate([a * np.cos(angle) - b * np.sin(angle), b * np.cos(angle) + a * np.sin(angle)], axis=-1)


def append_row(ckv, gain, pos, eps, theta):
    """A token's cache row: normalised vector, rotated key."""
    rank = len(gain)
    c = ckv[:rank]
    return np.concatenate([c / np.sqrt(np.mean(c * c) + eps) * gain, rope64(ckv[rank:rank + ROPE], pos, theta)])


def attention_request(q, q_rope, w_kv, rows, scale):
    """q [n][H][hd], q_rope [n][H][64], w_kv [H][2 hd][rank], rows [kv][rank +
    64]; token i sees keys 0 .. kv - n + i.  Returns o [n][H][hd], the
    probabilities [H][n][kv] and the logits."""
    n, H, hd = q.shape
    kv, rank = len(rows), w_kv.shape[2]
    c, kr = rows[:, :rank], rows[:, rank:]
    hidden = np.arange(kv)[None, :] > (kv - n + np.arange(n))[:, None]
    o = np.zeros((n, H, hd))
    ps, zs = np.zeros((H, n, kv)), np.zeros((H, n, kv))
    for h in range(H):
        K, V = c @ w_kv[h, :hd].T, c @ w_kv[h, hd:].T
        z = scale * (q[:, h] @ K.T + q_rope[:, h] @ kr.T)
        z = np.where(hidden, -np.inf, z)
        e = np.exp(z - z.max(axis=1, keepdims=True))
        p = e / e.sum(axis=1, keepdims=True)
        o[:, h], ps[h], zs[h] = p @ V, p, z
    return o, ps, zs


def batch_tables(slots, cached, new, T, bt_cap, tables, owned, ring, head, count, num_pages):
    """Request by request.  Changes `tables` and `owned` in place; returns the
    outputs of mb_batch_tables (bt without what is behind its last page), the
    ring's head and count, and whether an error is recorded."""
    max_slots, max_pages = tables.shape
    bad = not (0 <= head < num_pages and 0 <= count <= num_pages)
    ring_ok = not bad
    asked, plan, taken = 0, [], 0
    for s, c, m in zip(slots, cached, new):
        s, c, m = int(s), int(c), int(m)
        ok = ring_ok and 0 <= s < max_slots and list(slots).count(s) == 1
        ok = ok and c >= 0 and m >= 0 and 0 <= owned[s] <= max_pages and c <= owned[s] * PAGE
        ok = ok and c + m <= max_pages * PAGE
        if not ok:
            bad = True
            plan.append((s, 0, 0, []))
            continue
        need = max(0, -(-(c + m) // PAGE) - int(owned[s]))
        asked += need
        if need and asked > count:
            m = need = 0
        fresh = [int(ring[(head + taken + i) % num_pages]) for i in range(need)]
        taken += need
        plan.append((s, c, m, fresh))
    total = sum(m for _, _, m, _ in plan)
    pages = sum(-(-(c + m) // PAGE) for _, c, m, _ in plan)
    if total > T or pages > bt_cap:
        n = len(plan)
        none = np.full(T, -1, np.int64)
        return (np.zeros(n + 1), np.zeros(n), np.zeros(n + 1), np.zeros(0), none, none, none), head, count, True
    qo, kv, bti, bt, req, pos, slot = [0], [], [0], [], [], [], []
    for r, (s, c, m, fresh) in enumerate(plan):
        for page in fresh:
            tables[s, owned[s]] = page
            owned[s] += 1
        mine = [int(x) for x in tables[s, :-(-(c + m) // PAGE)]] if c + m else []
        bt += mine
        bad |= any(not 0 <= page < num_pages for page in mine)
        kv.append(c + m)
        for p in range(c, c + m):
            req.append(r)
            pos.append(p)
            page = mine[p // PAGE]
            good = 0 <= page < num_pages
            bad |= not good
            slot.append(page * PAGE + p % PAGE if good else -1)
        qo.append(qo[-1] + m)
        bti.append(bti[-1] + len(mine))
    rest = [-1] * (T - total)
    out = tuple(np.asarray(x) for x in (qo, kv, bti, bt, req + rest, pos + rest, slot + rest))
    if taken:
        head, count = (head + taken) % num_pages, count - taken
    return out, head, count, bad


def tables_release(slots, tables, owned, ring, head, count, num_pages):
    """Changes `owned` and `ring` in place; returns the new count and whether
    an error is recorded."""
    max_slots, max_pages = tables.shape
    if not (0 <= head < num_pages and 0 <= count <= num_pages):
        return count, True
    good = [0 <= s < max_slots and list(slots).count(s) == 1 and 0 <= owned[s] <= max_pages for s in slots]
    pages = [int(x) for s, ok in zip(slots, good) if ok for x in tables[s, :owned[s]]]
    if count + len(pages) > num_pages:
        return count, True
    for i, page in enumerate(pages):
        ring[(head + count + i) % num_pages] = page
    for s, ok in zip(slots, good):
        if ok:
            owned[s] = 0
    return count + len(pages), not all(good)
