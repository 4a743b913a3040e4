"""Cases for the speculative-decoding operators over the paged KV cache.

A step that checks drafted tokens runs, per request, a small tree of drafted
tokens against the request's cached prefix, keeps the accepted path and puts
its keys and values where the next step looks for them:

* ``tree``     mb_tree_attention: every drafted token attends to the whole
               cached prefix, to its ancestors in the tree and to itself;
* ``verify``   mb_verify_tree: the drafted tokens against the target's
               probabilities, from given random numbers;
* ``compact``  mb_kv_compact: the accepted path's keys and values move to the
               positions behind the prefix, in every layer's pool;
* ``copy``     mb_kv_copy_pages: a fork of requests (pages copied in every
               layer's pool).

``run`` computes the plain form (elementary torch operations in 32 bits, in 64
for the probabilities, where a comparison at a border decides) or, with
``own`` set, calls the framework.
"""

import functools
import math

import numpy as np
import torch

own = False

PAGE = 16
DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one user, a short draft of 5 tokens behind an 1,125-token context: latency
        dict(name="tree_one", op="tree", n=1, kv_lo=1125, kv_hi=1125, nodes_lo=6, nodes_hi=6, hkv=8, g=4, hd=128,
             shape="chain"),
        # the 64 decodes at 1,125 tokens of the Llama-3-8B-shaped layer, 8 drafted tokens each
        dict(name="tree_64x1125", op="tree", n=64, kv_lo=1125, kv_hi=1125, nodes_lo=8, nodes_hi=8, hkv=8, g=4, hd=128,
             shape="wide"),
        # the 96 running decodes of the Qwen3-14B-shaped stack, ragged contexts and ragged trees
        dict(name="tree_96_ragged", op="tree", n=96, kv_lo=1024, kv_hi=8192, nodes_lo=1, nodes_hi=25, hkv=8, g=5,
             hd=128, shape="wide"),
        # its 16 long decodes with trees of 64 tokens: 320 rows a KV head, where arithmetic counts as much as bytes
        dict(name="tree_16x8192_big", op="tree", n=16, kv_lo=8192, kv_hi=8192, nodes_lo=64, nodes_hi=64, hkv=8, g=5,
             hd=128, shape="wide"),
        # a small model without shared heads (head 64), odd lengths up to 32,768
        dict(name="tree_hd64_long", op="tree", n=7, kv_lo=33, kv_hi=32768, nodes_lo=3, nodes_hi=33, hkv=4, g=1, hd=64,
             shape="wide"),
        # one request, greedy, a chain of 5 drafts: latency
        dict(name="verify_greedy_one", op="verify", n=1, nodes=6, vocab=32000, mode="greedy", children=1),
        # 64 requests, a chain of 5 drafts each with the draft model's probabilities
        dict(name="verify_chain_64", op="verify", n=64, nodes=6, vocab=128256, mode="probs", children=1),
        # 16 requests with trees of 25 tokens from a deterministic draft (its best tokens), odd vocabulary
        dict(name="verify_tree_16", op="verify", n=16, nodes=25, vocab=50264, mode="points", children=4),
        # one request on a 32-layer cache: 4 accepted tokens of 8
        dict(name="compact_one", op="compact", n=1, layers=32, kv_lo=500, kv_hi=600, nodes=8, accept=4, hkv=8, hd=128),
        # 64 requests on the 40-layer cache, trees of 25 tokens, 5 accepted
        dict(name="compact_64", op="compact", n=64, layers=40, kv_lo=64, kv_hi=512, nodes=25, accept=5, hkv=8, hd=128),
        # copy of one request's last page before its fork, 32 layers
        dict(name="copy_one", op="copy", layers=32, pages=64, pairs=1, hkv=8, hd=128),
        # fork of whole requests: 256 pages (4,096 tokens) of the 40-layer cache
        dict(name="copy_256", op="copy", layers=40, pages=640, pairs=256, hkv=8, hd=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "verify", "verify", "compact", "copy"])
    if op == "tree":
        hkv, g = rng.choice([(8, 4), (8, 5), (4, 1), (2, 4), (2, 5), (8, 8), (1, 7), (4, 2)])
        hd = rng.choice([64, 128])
        n = _log(rng, 1, 64)
        hi = min(32768, max(64, 131072 // n))
        kv_hi = _log(rng, 40, hi)
        nodes_hi = _log(rng, 1, 64)
        return dict(op=op, n=n, kv_lo=max(nodes_hi, kv_hi // rng.choice([1, 2, 8])), kv_hi=max(kv_hi, nodes_hi),
                    nodes_lo=max(1, nodes_hi // rng.choice([1, 3])), nodes_hi=nodes_hi, hkv=hkv, g=g, hd=hd,
                    shape=rng.choice(["chain", "wide"]))
    if op == "verify":
        mode = rng.choice(["greedy", "probs", "points"])
        nodes = _log(rng, 1, 32)
        n = _log(rng, 1, max(1, 384 // nodes))
        return dict(op=op, n=n, nodes=nodes, vocab=8 * _log(rng, 12, 16032), mode=mode, children=rng.choice([1, 2, 4]))
    if op == "compact":
        nodes = _log(rng, 2, 64)
        return dict(op=op, n=_log(rng, 1, 64), layers=rng.choice([1, 32, 40]), kv_lo=nodes + rng.randrange(1, 40),
                    kv_hi=nodes + rng.randrange(40, 400), nodes=nodes, accept=rng.randrange(1, min(nodes, 9) + 1),
                    hkv=rng.choice([2, 4, 8]), hd=rng.choice([64, 128]))
    pages = _log(rng, 8, 512)
    return dict(op=op, layers=rng.choice([1, 8, 32, 40]), pages=pages, pairs=_log(rng, 1, pages // 2),
                hkv=rng.choice([2, 4, 8]), hd=rng.choice([64, 128]))


# ----------------------------------------------------------------- inputs
def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=np.int32))).to(DEV)


def _parents(rs, nodes, shape, children=4):
    """Parents of one request's tokens: token 0 is the last sampled one (its
    parent -1: the cached prefix), the others its drafted descendants, each
    token with at most `children` children, parents before children."""
    idx = np.arange(nodes)
    if shape == "chain" or children == 1:
        return idx - 1
    back = rs.randint(0, 3, size=nodes)
    return np.where(idx == 0, -1, np.maximum(0, (idx - 1) // children - back % 2))


def _lengths(rs, c):
    """Context lengths log-uniform over the case's range: its n quantiles, in an order of the seed."""
    lo, hi = c["kv_lo"], c["kv_hi"]
    at = (np.arange(c["n"]) + 0.5) / c["n"]
    kv = np.exp(math.log(lo) + at * (math.log(hi + 0.999) - math.log(lo))).astype(np.int64)
    return rs.permutation(np.clip(kv, lo, hi))


def _tables(rs, kv):
    """Block tables over a pool with a few spare pages, pages scattered."""
    per = (kv + PAGE - 1) // PAGE
    total = int(per.sum())
    perm = rs.permutation(total + 3)[:total]
    return total + 3, np.concatenate([[0], np.cumsum(per)]), perm


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(gen, *shape):
    """bf16 normal numbers, drawn a slice at a time along the first axis."""
    out = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    step = max(1, (1 << 27) // max(1, math.prod(shape[1:])))
    for a in range(0, shape[0], step):
        part = out[a:a + step]
        part.copy_(torch.randn(part.shape, generator=gen, device=DEV))
    return out


def prepare(case, seed):
    return {"tree": _prepare_tree, "verify": _prepare_verify, "compact": _prepare_compact,
            "copy": _prepare_copy}[case["op"]](case, seed)


def _prepare_tree(c, seed):
    rs, gen = np.random.RandomState(seed), _gen(seed)
    n = c["n"]
    nodes = rs.permutation(c["nodes_lo"] + np.arange(n) * (c["nodes_hi"] + 1 - c["nodes_lo"]) // n)
    kv = _lengths(rs, c)
    num_pages, bt_indptr, bt = _tables(rs, kv)
    qo = np.concatenate([[0], np.cumsum(nodes)])
    parent = np.concatenate([_parents(rs, int(m), c["shape"]) for m in nodes])
    T, hq = int(qo[-1]), c["hkv"] * c["g"]
    s = dict(case=c, op="tree", n=n, T=T, num_pages=num_pages, hq=hq, hkv=c["hkv"], hd=c["hd"],
             max_nodes=int(nodes.max()), max_pages=int((bt_indptr[1:] - bt_indptr[:-1]).max()),
             qo=_i32(qo), kv=_i32(kv), bti=_i32(bt_indptr), bt=_i32(bt), parent=_i32(parent))
    # keys and queries of unit variance give logits of unit variance; a few
    # queries are longer, so that some rows attend to few keys
    s["q"] = _randn(gen, T, hq, c["hd"]) * (1.0 + 3.0 * torch.rand(T, hq, 1, generator=gen, device=DEV) ** 4).to(
        torch.bfloat16)
    s["pool"] = _randn(gen, num_pages, 2, c["hkv"], PAGE, c["hd"])
    s["o"] = torch.empty(T, hq * c["hd"], dtype=torch.bfloat16, device=DEV)
    # the caller's workspace, its size from mb_tree_attention_workspace_bytes()
    # (which is at most this on any shape)
    s["work"] = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    return s


def _prepare_verify(c, seed):
    rs, gen = np.random.RandomState(seed), _gen(seed)
    n, m, V = c["n"], c["nodes"], c["vocab"]
    parent = np.concatenate([_parents(rs, m, "wide", c["children"]) for _ in range(n)])
    qo = np.arange(n + 1) * m
    T = n * m
    up = _i32(np.where(parent < 0, 0, parent) + np.repeat(qo[:-1], m)).long()
    logits = _randn(gen, T, V) * 2.0
    temp = 0.6 + 0.6 * torch.rand(n, generator=gen, device=DEV)
    row_temp = temp.repeat_interleave(m)[:, None]
    # the draft proposes tokens that the target often agrees with: the k-th
    # child of a token carries the row's k-th favourite, whose logit is raised
    # to about the size of all others together
    sib = torch.zeros(T, dtype=torch.long, device=DEV)
    for k in range(1, T):
        if parent[k] >= 0 and k % m:
            first = (k // m) * m
            sib[k] = int(np.sum(parent[first:k] == parent[k]))
    most = int(sib.max()) + 1
    fav = torch.randint(0, V, (T, most), generator=gen, device=DEV)
    tok_sib = torch.where(torch.rand(T, generator=gen, device=DEV) < 0.2,
                          torch.randint(0, V, (T,), generator=gen, device=DEV), fav[up, sib])   # one in five a miss
    lse = torch.logsumexp(logits.float() / row_temp, dim=1, keepdim=True) * row_temp
    raised = lse + 2.0 * torch.rand(T, most, generator=gen, device=DEV) - 0.7 * torch.arange(most, device=DEV)
    logits.scatter_(1, fav, raised.to(torch.bfloat16))
    s = dict(case=c, op="verify", n=n, T=T, vocab=V, mode=c["mode"], m=m, qo=_i32(qo), parent=_i32(parent),
             logits=logits, max_path=min(m, 16), most=most, sib=sib.to(torch.int32))
    s["probs"] = None
    if c["mode"] == "probs":
        # the draft's own distribution: the target's logits with noise; its
        # tokens are drawn from it
        q = (logits.float() + 0.5 * torch.randn(T, V, generator=gen, device=DEV)) / row_temp
        s["probs"] = torch.softmax(q, dim=1)
        race = s["probs"][up] / -torch.log(torch.rand(T, V, generator=gen, device=DEV).clamp_min(1e-30))
        tok_sib = torch.argmax(race, dim=1)
    s["tokens"] = tok_sib.to(torch.int32)
    s["temp"] = None if c["mode"] == "greedy" else temp
    s["u_accept"] = torch.rand(T, generator=gen, device=DEV)
    s["u_final"] = torch.rand(n, generator=gen, device=DEV)
    for k, size in (("count", (n,)), ("path", (n, s["max_path"])), ("next", (n,))):
        s[k] = torch.empty(size, dtype=torch.int32, device=DEV)
    return s


def _prepare_compact(c, seed):
    rs, gen = np.random.RandomState(seed), _gen(seed)
    n, m = c["n"], c["nodes"]
    kv = _lengths(rs, c)
    num_pages, bt_indptr, bt = _tables(rs, kv)
    path = np.full((n, 16), -1)
    count = np.minimum(m, 1 + rs.randint(0, 2 * c["accept"] - 1, size=n)) if n > 1 else np.array([c["accept"]])
    count = np.minimum(count, 16)
    for r in range(n):
        path[r, :count[r]] = np.concatenate([[0], np.sort(rs.permutation(m - 1)[:count[r] - 1]) + 1])
    s = dict(case=c, op="compact", n=n, num_pages=num_pages, hkv=c["hkv"], hd=c["hd"], max_path=16,
             qo=_i32(np.arange(n + 1) * m), kv=_i32(kv), bti=_i32(bt_indptr), bt=_i32(bt), count=_i32(count),
             path=_i32(path), new_kv=torch.empty(n, dtype=torch.int32, device=DEV))
    s["pools"] = _randn(gen, c["layers"], num_pages, 2, c["hkv"], PAGE, c["hd"])
    s["list"] = list(s["pools"].unbind(0))
    return s


def _prepare_copy(c, seed):
    rs, gen = np.random.RandomState(seed), _gen(seed)
    perm = rs.permutation(c["pages"]).astype(np.int32)
    s = dict(case=c, op="copy", num_pages=c["pages"], hkv=c["hkv"], hd=c["hd"], src=perm[:c["pairs"]].copy(),
             dst=perm[c["pairs"]:2 * c["pairs"]].copy())
    s["pools"] = _randn(gen, c["layers"], c["pages"], 2, c["hkv"], PAGE, c["hd"])
    s["list"] = list(s["pools"].unbind(0))
    return s


# -------------------------------------------------------------------- run
def run(s):
    return {"tree": _run_tree, "verify": _run_verify, "compact": _run_compact, "copy": _run_copy}[s["op"]](s)


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _closure(parent):
    """[n, N] parents -> [n, N, N]: token i sees token j (itself or an ancestor)."""
    N = parent.shape[1]
    idx = torch.arange(N, device=parent.device)
    edge = ((parent[:, :, None] == idx) | (idx[:, None] == idx)).float()
    return functools.reduce(lambda a, _: ((a @ a) > 0).float(), range(max(1, (N - 1).bit_length())), edge) > 0


def _run_tree(s):
    if own:
        from mixed_prefill_decode_gb300 import binding as mb
        mb.mb_tree_attention(s["q"], s["pool"], s["o"], s["num_pages"], s["hq"], s["hkv"], s["hd"], s["n"], s["T"],
                             s["qo"], s["kv"], s["bti"], s["bt"], s["parent"], s["work"], _stream())
        return s["o"]
    n, N, hkv, hd, T = s["n"], s["max_nodes"], s["hkv"], s["hd"], s["T"]
    g, L = s["hq"] // hkv, s["max_pages"] * PAGE
    qo, kv, bti = s["qo"].long(), s["kv"].long(), s["bti"].long()
    nodes = qo[1:] - qo[:-1]
    cached = kv - nodes
    # keys and values, gathered by the block tables and padded
    col = torch.arange(s["max_pages"], device=DEV)
    at = bti[:-1, None] + col
    page = torch.where(col < (bti[1:] - bti[:-1])[:, None], s["bt"].long()[at.clamp_max(s["bt"].numel() - 1)], 0)
    kvs = s["pool"][page]                                             # [n, pages, 2, hkv, 16, hd]
    pos = torch.arange(L, device=DEV)
    K = kvs[:, :, 0].permute(0, 2, 1, 3, 4).reshape(n, hkv, L, hd).float()
    V = kvs[:, :, 1].permute(0, 2, 1, 3, 4).reshape(n, hkv, L, hd).float()
    V = torch.where((pos < kv[:, None])[:, None, :, None], V, 0.0)
    # queries by request and token, padded
    node = torch.arange(N, device=DEV)
    tok = (qo[:-1, None] + node).clamp_max(T - 1)
    q = s["q"][tok].float().reshape(n, N, hkv, g, hd).permute(0, 2, 1, 3, 4).reshape(n, hkv, N * g, hd)
    par = torch.where(node < nodes[:, None], s["parent"].long()[tok], -1)
    sees = _closure(par)
    rel = pos - cached[:, None]                                       # [n, L]: index in the tree
    tree = torch.gather(sees, 2, rel.clamp(0, N - 1)[:, None, :].expand(n, N, L))
    see = (rel < 0)[:, None, :] | (tree & (rel < nodes[:, None])[:, None, :] & (rel >= 0)[:, None, :])
    see = see[:, None, :, None, :].expand(n, 1, N, g, L).reshape(n, 1, N * g, L)
    S = torch.where(see, (q @ K.transpose(2, 3)) * (1.0 / math.sqrt(hd)), float("-inf"))
    P = torch.exp(S - S.amax(dim=3, keepdim=True).clamp_min(-1e30))
    O = (P @ V) / P.sum(dim=3, keepdim=True)
    O = O.reshape(n, hkv, N, g, hd).permute(0, 2, 1, 3, 4).reshape(n, N, hkv * g * hd)
    t = torch.arange(T, device=DEV)
    r = torch.searchsorted(qo[1:].contiguous(), t, right=True)
    s["o"].copy_(O[r, t - qo[r]])
    return s["o"]


def _run_verify(s):
    if own:
        from mixed_prefill_decode_gb300 import binding as mb
        mb.mb_verify_tree(s["logits"], s["vocab"], s["tokens"], s["probs"], s["n"], s["T"], s["qo"], s["parent"],
                          s["temp"], s["u_accept"], s["u_final"], s["max_path"], s["count"], s["path"], s["next"],
                          _stream())
        return s["count"], s["path"], s["next"]
    n, m, T, V, most = s["n"], s["m"], s["T"], s["vocab"], s["most"]
    parent = s["parent"].long().reshape(n, m)
    base = torch.arange(n, device=DEV)[:, None] * m
    up = (parent.clamp_min(0) + base).reshape(T)
    tok = s["tokens"].long()
    drafted = (parent >= 0).reshape(T)
    logits = s["logits"].double()
    best = torch.argmax(logits, dim=1)
    sib = s["sib"].long()                 # how many earlier children the token's parent has
    if s["mode"] == "greedy":
        ok = tok == best[up]
    else:
        x = (logits - logits.amax(dim=1, keepdim=True)) / s["temp"].double().repeat_interleave(m)[:, None]
        e = torch.exp(x)
        e = e / e.sum(dim=1, keepdim=True)
        u = s["u_accept"].double()
        px = e[up, tok]
        same = (up[:, None] == up[None, :]) & drafted[:, None] & drafted[None, :]
        before = same & (torch.arange(T, device=DEV)[None, :] < torch.arange(T, device=DEV)[:, None])
        if s["mode"] == "points":
            # after earlier siblings were refused, their tokens are out and
            # the rest is scaled up: p(x) / (1 - sum of the refused)
            twice = before & (tok[:, None] == tok[None, :])
            first = ~twice.any(dim=1)
            gone = (before & first[None, :]).double() @ px
            ok = first & (u * (1.0 - gone) < px)
        else:
            # refused once, the target becomes norm(max(0, p - q)); k times,
            # max(0, p - a q) / c with a' = a + c, c' = sum max(0, p - a' q)
            q = s["probs"].double()

            def refuse(ac, _):
                a = ac[0][-1] + ac[1][-1]
                return ac[0] + [a], ac[1] + [(e - a[:, None] * q).clamp_min(0).sum(dim=1)]

            zero = torch.zeros(T, dtype=torch.float64, device=DEV)
            A, C = functools.reduce(refuse, range(most), ([zero], [zero + 1]))
            A, C = torch.stack(A, dim=1), torch.stack(C, dim=1)       # [T, most + 1]
            qx = q[up, tok]
            ok = u * C[up, sib] * qx < px - A[up, sib] * qx
    # the first accepted child of each token, and the path from the root
    ok = ok & drafted
    code = torch.where(ok, torch.arange(T, device=DEV), T)
    first_child = torch.full((T + 1,), T, dtype=torch.long, device=DEV).scatter_reduce(
        0, torch.where(drafted, up, T), code, "amin")[:T]
    step = torch.cat([first_child, torch.full((1,), T, device=DEV)])
    walk = functools.reduce(lambda w, _: w + [step[w[-1]]], range(s["max_path"] - 1), [base[:, 0]])
    walk = torch.stack(walk, dim=1)                                   # [n, max_path], T past the end
    count = (walk < T).sum(dim=1)
    last = torch.gather(walk, 1, (count - 1)[:, None])[:, 0]
    s["count"].copy_(count)
    s["path"].copy_(torch.where(walk < T, walk - base, -1))
    if s["mode"] == "greedy":
        s["next"].copy_(best[last])
        return s["count"], s["path"], s["next"]
    # a token of what is left of the last row: the refused children's share is out
    kids = torch.where(drafted[None, :] & (up[None, :] == last[:, None]), 1, 0)          # [n, T]
    left = e[last]
    if s["mode"] == "points":
        cut = torch.zeros(n, V + 1, dtype=torch.float64, device=DEV).scatter_add(
            1, torch.where(kids > 0, tok[None, :].expand(n, T), V), torch.ones(n, T, dtype=torch.float64, device=DEV))
        full = torch.where(count == s["max_path"], 0, 1)[:, None]
        w = torch.where((cut[:, :V] > 0) & (full > 0), 0.0, left)
    else:
        refused = torch.where(count == s["max_path"], 0, kids.sum(dim=1))
        w = (left - A[last, refused][:, None] * s["probs"].double()[last]).clamp_min(0)
        w = torch.where(refused[:, None] > 0, w, left)
    w = torch.where(w.sum(dim=1, keepdim=True) > 0, w, left)
    total = w.sum(dim=1, keepdim=True)
    over = w.cumsum(dim=1) > s["u_final"].double()[:, None] * total
    s["next"].copy_(torch.argmax(over.to(torch.int32), dim=1))
    return s["count"], s["path"], s["next"]


def _run_compact(s):
    if own:
        from mixed_prefill_decode_gb300 import binding as mb
        mb.mb_kv_compact(s["list"], s["num_pages"], s["hkv"], s["hd"], s["n"], s["qo"], s["kv"], s["bti"], s["bt"],
                         s["count"], s["path"], s["max_path"], s["new_kv"], _stream())
        return s["pools"], s["new_kv"]
    qo, kv, bti, count = s["qo"].long(), s["kv"].long(), s["bti"].long(), s["count"].long()
    cached = kv - (qo[1:] - qo[:-1])
    k = torch.arange(s["max_path"], device=DEV)
    live = k < count[:, None]
    frm = cached[:, None] + torch.where(live, s["path"].long(), 0)
    to = cached[:, None] + torch.where(live, k, 0)
    last = s["bt"].numel() - 1
    page_f = s["bt"].long()[(bti[:-1, None] + frm // PAGE).clamp_max(last)].reshape(-1)
    page_t = s["bt"].long()[(bti[:-1, None] + to // PAGE).clamp_max(last)].reshape(-1)
    # entries past the path move the first token onto itself (path[0] is 0)
    s["pools"][:, page_t, :, :, to.reshape(-1) % PAGE] = s["pools"][:, page_f, :, :, frm.reshape(-1) % PAGE]
    s["new_kv"].copy_(cached + count)
    return s["pools"], s["new_kv"]


def _run_copy(s):
    if own:
        from mixed_prefill_decode_gb300 import binding as mb
        mb.mb_kv_copy_pages(s["list"], s["num_pages"], s["hkv"], s["hd"], s["src"], s["dst"], _stream())
        return s["pools"]
    src = torch.from_numpy(s["src"]).to(DEV, non_blocking=True).long()
    dst = torch.from_numpy(s["dst"]).to(DEV, non_blocking=True).long()
    s["pools"][:, dst] = s["pools"][:, src]
    return s["pools"]


# ------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "tree":
        mean = c["kv_lo"] if c["kv_hi"] == c["kv_lo"] else (c["kv_hi"] - c["kv_lo"]) / math.log(c["kv_hi"] / c["kv_lo"])
        nodes = (c["nodes_lo"] + c["nodes_hi"]) / 2
        keys = c["n"] * max(mean, nodes)
        rows = nodes * c["g"] * c["hkv"]
        return {"bytes": int(keys * c["hkv"] * c["hd"] * 4 + 2 * c["n"] * rows * c["hd"] * 2),
                "flops": int(4 * keys * rows * c["hd"])}
    if c["op"] == "verify":
        # the rows on the accepted path (about two drafts a request), read once
        rows = c["n"] * min(c["nodes"], 3)
        each = c["vocab"] * (2 + (4 if c["mode"] == "probs" else 0) / 3)
        return {"bytes": int(rows * each), "flops": int(4 * rows * c["vocab"])}
    if c["op"] == "compact":
        moved = c["n"] * max(1, min(c["nodes"], c["accept"]) - 1)
        return {"bytes": int(2 * moved * c["layers"] * 2 * c["hkv"] * c["hd"] * 2), "flops": 0}
    return {"bytes": int(2 * c["pairs"] * c["layers"] * 2 * c["hkv"] * PAGE * c["hd"] * 2), "flops": 0}


# ------------------------------------------------------------------ exact
def exact(case, seed):
    s = prepare(case, seed)
    return {"tree": _exact_tree, "verify": _exact_verify, "compact": _exact_compact, "copy": _exact_copy}[s["op"]](s)


def _exact_tree(s):
    qo, kv, bti = (s[k].cpu().numpy() for k in ("qo", "kv", "bti"))
    bt, parent = s["bt"].cpu().numpy(), s["parent"].cpu().numpy()
    g, out = s["hq"] // s["hkv"], torch.empty(s["T"], s["hq"], s["hd"], dtype=torch.float64, device=DEV)
    for r in range(s["n"]):
        a, b, k = int(qo[r]), int(qo[r + 1]), int(kv[r])
        c = k - (b - a)
        see = np.zeros((b - a, k), dtype=bool)
        see[:, :c] = True
        for i in range(b - a):
            j = i
            while j >= 0:
                see[i, c + j] = True
                j = int(parent[a + j])
        see = torch.from_numpy(see).to(DEV)
        pages = torch.from_numpy(bt[bti[r]:bti[r] + -(-k // PAGE)].astype(np.int64)).to(DEV)
        mine = s["pool"][pages]
        for h in range(s["hkv"]):
            key = mine[:, 0, h].reshape(-1, s["hd"])[:k].double()
            val = mine[:, 1, h].reshape(-1, s["hd"])[:k].double()
            for x in range(h * g, h * g + g):
                z = (s["q"][a:b, x].double() @ key.T) / math.sqrt(s["hd"])
                out[a:b, x] = torch.softmax(z.masked_fill(~see, float("-inf")), dim=1) @ val
    return out.reshape(s["T"], -1)


def _exact_verify(s):
    """Whole numbers only: the walk itself, token by token."""
    parent, tok, m = s["parent"].cpu().numpy(), s["tokens"].cpu().numpy(), s["m"]
    u, last_u = s["u_accept"].cpu().numpy().astype(np.float64), s["u_final"].cpu().numpy().astype(np.float64)
    counts, paths, nexts = [], [], []
    for r in range(s["n"]):
        path = [0]
        while True:
            row = r * m + path[-1]
            z = s["logits"][row].double().cpu().numpy()
            kids = [] if len(path) == s["max_path"] else [i for i in range(m) if parent[r * m + i] == path[-1]]
            if s["mode"] == "greedy":
                top = int(np.argmax(z))
                hit = [i for i in kids if tok[r * m + i] == top]
                if not hit:
                    nexts.append(top)
                    break
                path.append(hit[0])
                continue
            p = np.exp((z - z.max()) / float(s["temp"][r].double()))
            p /= p.sum()
            left, hit = p.copy(), None
            q = s["probs"][row].double().cpu().numpy() if s["mode"] == "probs" else None
            for i in kids:
                x = int(tok[r * m + i])
                good = u[r * m + i] * (q[x] if q is not None else 1.0) < left[x]
                if good:
                    hit = i
                    break
                if q is not None:
                    left = np.maximum(0.0, left - q)
                else:
                    left[x] = 0.0
                left = left / left.sum() if left.sum() > 0 else left
            if hit is None:
                left = left if left.sum() > 0 else p
                cum = np.cumsum(left)
                nexts.append(int(np.argmax(cum > last_u[r] * cum[-1])))
                break
            path.append(hit)
        counts.append(len(path))
        paths.append(path + [-1] * (s["max_path"] - len(path)))
    return np.array(counts, np.int32), np.array(paths, np.int32), np.array(nexts, np.int32)


def _exact_compact(s):
    qo, kv, bti, bt = (s[k].cpu().numpy() for k in ("qo", "kv", "bti", "bt"))
    count, path = s["count"].cpu().numpy(), s["path"].cpu().numpy()
    pools, new = s["pools"], []
    for r in range(s["n"]):
        c = int(kv[r] - (qo[r + 1] - qo[r]))
        for k in range(int(count[r])):   # ascending: a token moves to a lower place or stays
            f, t = c + int(path[r, k]), c + k
            if f != t:
                pools[:, int(bt[bti[r] + t // PAGE]), :, :, t % PAGE] = pools[:, int(bt[bti[r] + f // PAGE]), :, :, f % PAGE]
        new.append(c + int(count[r]))
    return pools, np.array(new, np.int32)


def _exact_copy(s):
    for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
        s["pools"][:, b] = s["pools"][:, a].clone()
    return s["pools"]
