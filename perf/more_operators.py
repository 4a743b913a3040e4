"""Cases for the latent-cache operators and the descriptors built on the GPU.

A layer with latent attention caches one vector per token (``rank`` numbers,
normalised) and one rotated key of 64 numbers that all heads share; every
head's keys and values are linear maps of the vector.  A serving step is

* ``tables``   mb_batch_tables: the batch's descriptor, its block tables and
               the place of every new token, from the requests' lengths;
* ``append``   mb_latent_append: the new tokens' vectors normalised, their keys
               and the queries rotated, vectors and keys into the paged cache;
* ``absorbed`` mb_latent_attention: attention of single tokens (or a few)
               against the cached vectors themselves, the maps applied to
               queries and outputs instead;
* ``expanded`` mb_latent_prefill: attention of prompt chunks, keys and values
               of every head made from the cached vectors first.

``run`` computes the plain form (elementary torch operations in 32 bits, in 64
for the angles of rotations) or, with ``own`` set, calls the framework.
"""

import math

import numpy as np
import torch

own = False

PAGE = 16
ROPE = 64
THETA = 10000.0
EPS = 1e-6
DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a step of 64 decodes at 1,125 tokens: latency
        dict(name="tables_64", op="tables", n=64, chunks=0, chunk=0, kv_lo=1125, kv_hi=1125, slots=256, max_pages=512,
             left=1.0),
        # 256 decodes with contexts up to 32,768 tokens beside two prompts' chunks, in all 8,192 tokens; odd lengths
        dict(name="tables_256_mixed", op="tables", n=258, chunks=2, chunk=3967, kv_lo=512, kv_hi=32768, slots=1024,
             max_pages=2560, left=1.0),
        # 64 decodes of a layer with 32 heads: latency
        dict(name="append_64", op="append", T=64, heads=32, hd=128, rank=512, pos_hi=1200),
        # a chunk of 2,048 tokens with 96 decodes, 40 heads
        dict(name="append_2144", op="append", T=2144, heads=40, hd=128, rank=512, pos_hi=32768),
        # one user's next token behind 1,125: latency
        dict(name="absorbed_one", op="absorbed", n=1, qo_lo=1, qo_hi=1, kv_lo=1125, kv_hi=1125, heads=32, hd=128,
             rank=512),
        # 64 decodes at 1,125 tokens, 32 heads
        dict(name="absorbed_64x1125", op="absorbed", n=64, qo_lo=1, qo_hi=1, kv_lo=1125, kv_hi=1125, heads=32, hd=128,
             rank=512),
        # 96 decodes with contexts log-uniform in 1,024 to 8,192, 40 heads
        dict(name="absorbed_96_ragged", op="absorbed", n=96, qo_lo=1, qo_hi=1, kv_lo=1024, kv_hi=8192, heads=40, hd=128,
             rank=512),
        # 16 long decodes of a layer with 128 heads, where arithmetic counts as much as bytes
        dict(name="absorbed_16x8192", op="absorbed", n=16, qo_lo=1, qo_hi=1, kv_lo=8192, kv_hi=8192, heads=128, hd=128,
             rank=512),
        # a small model (head 64, rank 256) with two to five drafted tokens each, odd lengths up to 32,768
        dict(name="absorbed_drafts_small", op="absorbed", n=9, qo_lo=2, qo_hi=5, kv_lo=33, kv_hi=32768, heads=8, hd=64,
             rank=256),
        # one prompt of 512 tokens, nothing cached, 32 heads
        dict(name="expanded_512", op="expanded", n=1, qo_lo=512, qo_hi=512, pre_lo=0, pre_hi=0, heads=32, hd=128,
             rank=512),
        # five chunks of a small model, odd lengths, behind odd prefixes
        dict(name="expanded_ragged_small", op="expanded", n=5, qo_lo=33, qo_hi=1025, pre_lo=0, pre_hi=4001, heads=8,
             hd=64, rank=256),
        # a chunk of 2,048 tokens behind 6,144, 40 heads
        dict(name="expanded_2048_8192", op="expanded", n=1, qo_lo=2048, qo_hi=2048, pre_lo=6144, pre_hi=6144, heads=40,
             hd=128, rank=512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng, hd):
    return rng.choice([1, 4, 8, 20, 32, 40, 64, 128] if hd == 128 else [2, 5, 8, 16, 32, 40])


def draw(rng):
    op = rng.choice(["tables", "append", "absorbed", "absorbed", "absorbed", "expanded", "expanded"])
    hd = rng.choice([64, 128, 128])
    rank = rng.choice([256, 512, 512])
    if op == "tables":
        n = _log(rng, 1, 1024)
        chunks = rng.choice([0, 0, 1, 2, 5])
        hi = _log(rng, 40, max(41, min(32768, 2000000 // n)))
        return dict(op=op, n=n + chunks, chunks=chunks, chunk=_log(rng, 2, 8192 // max(1, chunks)) if chunks else 0,
                    kv_lo=max(1, hi // rng.choice([1, 2, 64])), kv_hi=hi, slots=n + chunks + _log(rng, 1, 500),
                    max_pages=2600, left=rng.choice([1.0, 1.0, 0.6]))
    if op == "append":
        return dict(op=op, T=_log(rng, 1, 2144), heads=rng.choice([1, 4, 8, 20, 32, 40]), hd=hd, rank=rank,
                    pos_hi=_log(rng, 100, 100000))
    if op == "absorbed":
        heads = _heads(rng, hd)
        n = _log(rng, 1, 96)
        qo_hi = rng.choice([1, 1, 1, 3, 6])
        room = 96 * 3500 * 40 // (max(heads, 40) * qo_hi * n)
        hi = _log(rng, 40, max(41, min(32768, room)))
        return dict(op=op, n=n, qo_lo=1, qo_hi=qo_hi, kv_lo=max(qo_hi, hi // rng.choice([1, 2, 8])), kv_hi=hi,
                    heads=heads, hd=hd, rank=rank)
    heads = rng.choice([1, 4, 8, 20, 32, 40])
    n = _log(rng, 1, 8)
    qo_hi = _log(rng, 2, max(3, 2048 // n))
    pre_hi = _log(rng, 1, max(2, 6000 // n))
    return dict(op=op, n=n, qo_lo=max(1, qo_hi // rng.choice([1, 3, 20])), qo_hi=qo_hi,
                pre_lo=rng.choice([0, pre_hi // 2, pre_hi]), pre_hi=pre_hi, heads=heads, hd=hd, rank=rank)


# ----------------------------------------------------------------- inputs
def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=np.int32))).to(DEV)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(gen, *shape, scale=1.0):
    """bf16 normal numbers, drawn a slice at a time along the first axis."""
    out = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    step = max(1, (1 << 27) // max(1, math.prod(shape[1:])))
    for a in range(0, shape[0], step):
        part = out[a:a + step]
        part.copy_(torch.randn(part.shape, generator=gen, device=DEV) * scale)
    return out


def _spread(rs, n, lo, hi):
    """n whole numbers log-uniform in [lo, hi]: the quantiles, in an order of the seed."""
    at = (np.arange(n) + 0.5) / n
    a = math.log(lo + 0.5)
    v = np.round(np.exp(a + at * (math.log(hi + 0.5) - a))).astype(np.int64)
    return rs.permutation(np.clip(v, lo, hi))


def prepare(case, seed):
    return {"tables": _prepare_tables, "append": _prepare_append, "absorbed": _prepare_attention,
            "expanded": _prepare_attention}[case["op"]](case, seed)


def _prepare_tables(c, seed):
    rs = np.random.RandomState(seed)
    n, k = c["n"], c["chunks"]
    cached = _spread(rs, n, c["kv_lo"], c["kv_hi"])
    new = np.ones(n, np.int64)
    at = rs.permutation(n)[:k]
    new[at] = c["chunk"]
    cached[at] = np.minimum(cached[at], 4096)   # a prompt part of the way through
    slots = rs.permutation(c["slots"])[:n]
    owned = np.zeros(c["slots"], np.int64)
    owned[slots] = -(-cached // PAGE)
    need = int(np.maximum(0, -(-(cached + new) // PAGE) - owned[slots]).sum())
    free = max(1, int(c["left"] * need)) + (n // 4 if c["left"] >= 1.0 else 0)
    # room for every request at its longest, whichever of them are the prompts
    cap = int((-(-_spread(rs, n, c["kv_lo"], c["kv_hi"]) // PAGE)).sum()) + n + k * (-(-c["chunk"] // PAGE))
    num_pages = cap + n // 4 + 1
    perm = rs.permutation(num_pages)
    tables = np.zeros((c["slots"], c["max_pages"]), np.int64)
    used = 0
    for s in slots:
        tables[s, :owned[s]] = perm[used:used + owned[s]]
        used += owned[s]
    # the free pages stand in a ring, from some place of it on
    ring = np.zeros(num_pages, np.int64)
    head = int(rs.randint(num_pages))
    ring[(head + np.arange(free)) % num_pages] = perm[used:used + free]
    T = int(new.sum())
    s = dict(case=c, op="tables", n=n, T=T, cap=cap, num_pages=num_pages, max_slots=c["slots"],
             max_pages=c["max_pages"], slots=_i32(slots), cached=_i32(cached), new=_i32(new), tables=_i32(tables),
             owned=_i32(owned), ring=_i32(ring), state=_i32([head, free, 0, 0]))
    for key, size in (("qo", n + 1), ("kv", n), ("bti", n + 1), ("bt", cap), ("req", T), ("pos", T), ("slot", T)):
        s[key] = torch.zeros(size, dtype=torch.int32, device=DEV)
    return s


def _prepare_append(c, seed):
    rs, gen = np.random.RandomState(seed), _gen(seed)
    T, rank = c["T"], c["rank"]
    num_pages = -(-T // PAGE) + 5
    s = dict(case=c, op="append", T=T, heads=c["heads"], hd=c["hd"], rank=rank, num_pages=num_pages)
    # what the down-projections of queries and of keys and values gave lies in one row
    s["ld"] = rank + ROPE + 256
    s["ckv"] = _randn(gen, T, s["ld"])[:, 256:]
    s["q"] = _randn(gen, T, c["heads"], c["hd"] + ROPE)
    s["gain"] = (1.0 + 0.1 * torch.randn(rank, generator=gen, device=DEV)).to(torch.bfloat16)
    s["pos"] = _i32(rs.randint(0, c["pos_hi"], size=T))
    s["slot"] = _i32(rs.permutation(num_pages * PAGE)[:T])
    s["pool"] = _randn(gen, num_pages, PAGE, rank + ROPE)
    s["q_rope"] = torch.zeros(T, c["heads"], ROPE, dtype=torch.bfloat16, device=DEV)
    return s


def _prepare_attention(c, seed):
    rs, gen = np.random.RandomState(seed), _gen(seed)
    n, H, hd, rank = c["n"], c["heads"], c["hd"], c["rank"]
    nodes = rs.permutation(c["qo_lo"] + np.arange(n) * (c["qo_hi"] + 1 - c["qo_lo"]) // n)
    if c["op"] == "absorbed":
        kv = np.maximum(_spread(rs, n, c["kv_lo"], c["kv_hi"]), nodes)
    else:
        kv = _spread(rs, n, c["pre_lo"], c["pre_hi"]) + nodes
    per = -(-kv // PAGE)
    total = int(per.sum())
    qo = np.concatenate([[0], np.cumsum(nodes)])
    T = int(qo[-1])
    s = dict(case=c, op=c["op"], n=n, T=T, heads=H, hd=hd, rank=rank, num_pages=total + 3,
             scale=1.0 / math.sqrt(hd + ROPE), kv_tokens=int(kv.sum()), max_new=int(nodes.max()),
             max_pages=int(per.max()), qo=_i32(qo), kv=_i32(kv), bti=_i32(np.concatenate([[0], np.cumsum(per)])),
             bt=_i32(rs.permutation(total + 3)[:total]))
    # vectors, keys and queries of unit variance give logits of about unit
    # variance; a few queries are longer, so that some rows attend to few keys
    far = (1.0 + 3.0 * torch.rand(T, H, 1, generator=gen, device=DEV) ** 4).to(torch.bfloat16)
    s["q"] = _randn(gen, T, H, hd + ROPE) * far
    s["q_rope"] = _randn(gen, T, H, ROPE) * far
    s["w_kv"] = _randn(gen, H, 2 * hd, rank, scale=1.0 / math.sqrt(rank))
    s["pool"] = _randn(gen, total + 3, PAGE, rank + ROPE)
    s["o"] = torch.zeros(T, H * hd, dtype=torch.bfloat16, device=DEV)
    return s


# -------------------------------------------------------------------- run
def run(s):
    return {"tables": _run_tables, "append": _run_append, "absorbed": _run_absorbed, "expanded": _run_expanded}[
        s["op"]](s)


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _scan(x):
    """0, x0, x0 + x1, ..."""
    return torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), torch.cumsum(x, 0)])


def _run_tables(s):
    keys = ("qo", "kv", "bti", "bt", "req", "pos", "slot", "tables", "owned", "state")
    if own:
        from mixed_prefill_decode_gb300 import binding as mb
        mb.mb_batch_tables(s["slots"], s["cached"], s["new"], s["n"], s["T"], s["cap"], s["tables"], s["owned"],
                           s["max_slots"], s["max_pages"], s["ring"], s["state"], s["num_pages"], s["qo"], s["kv"],
                           s["bti"], s["bt"], s["req"], s["pos"], s["slot"], _stream())
        return tuple(s[k] for k in keys)
    n, T, P = s["n"], s["T"], s["num_pages"]
    row, cached, new = s["slots"].long(), s["cached"].long(), s["new"].long()
    have, head, count = s["owned"].long()[row], s["state"].long()[0], s["state"].long()[1]
    need = (torch.div(cached + new + PAGE - 1, PAGE, rounding_mode="floor") - have).clamp_min(0)
    upto = torch.cumsum(need, 0)
    ok = (need == 0) | (upto <= count)
    new, need = torch.where(ok, new, 0), torch.where(ok, need, 0)
    kv = cached + new
    pages = torch.div(kv + PAGE - 1, PAGE, rounding_mode="floor")
    qo, bti, first = _scan(new), _scan(pages), _scan(need)
    # the new pages, from the ring into the requests' rows
    i = torch.arange(P, device=DEV)
    r = torch.searchsorted(first[1:].contiguous(), i, right=True)
    live, r = r < n, r.clamp_max(n - 1)
    place = row[r] * s["max_pages"] + have[r] + (i - first[r])
    flat = torch.cat([s["tables"].view(-1), s["tables"].new_zeros(1)])
    flat[torch.where(live, place, flat.numel() - 1)] = s["ring"][(head + i) % P]
    s["tables"].view(-1).copy_(flat[:-1])
    s["owned"][row] = (have + need).to(torch.int32)
    taken = first[-1]
    s["state"][0] = ((head + taken) % P).to(torch.int32)
    s["state"][1] = (count - taken).to(torch.int32)
    # the rows' pages one after another, and the tokens' places
    j = torch.arange(s["cap"], device=DEV)
    r = torch.searchsorted(bti[1:].contiguous(), j, right=True)
    live, r = r < n, r.clamp_max(n - 1)
    s["bt"].copy_(torch.where(live, s["tables"].view(-1).long()[row[r] * s["max_pages"] + (j - bti[r]).clamp_min(0)
                                                                .clamp_max(s["max_pages"] - 1)], s["bt"].long()))
    t = torch.arange(T, device=DEV)
    r = torch.searchsorted(qo[1:].contiguous(), t, right=True)
    live, r = r < n, r.clamp_max(n - 1)
    pos = (cached[r] + t - qo[r]).clamp_min(0)
    col = torch.div(pos, PAGE, rounding_mode="floor").clamp_max(s["max_pages"] - 1)
    page = s["tables"].view(-1).long()[row[r] * s["max_pages"] + col]
    s["req"].copy_(torch.where(live, r, -1))
    s["pos"].copy_(torch.where(live, pos, -1))
    s["slot"].copy_(torch.where(live, page * PAGE + pos % PAGE, -1))
    s["qo"].copy_(qo)
    s["kv"].copy_(kv)
    s["bti"].copy_(bti)
    return tuple(s[k] for k in keys)


def _rotate(x, pos):
    """RoPE of the last 64 numbers, pairs (i, i + 32), x in 32 bits."""
    i = torch.arange(ROPE // 2, device=DEV, dtype=torch.float64)
    angle = pos.double()[:, None] * torch.exp(i * (-2.0 / ROPE * math.log(THETA)))
    shape = (x.shape[0],) + (1,) * (x.dim() - 2) + (ROPE // 2,)
    c, d = torch.cos(angle).float().reshape(shape), torch.sin(angle).float().reshape(shape)
    a, b = x[..., :ROPE // 2], x[..., ROPE // 2:]
    return torch.cat([a * c - b * d, b * c + a * d], dim=-1)


def _run_append(s):
    if own:
        from mixed_prefill_decode_gb300 import binding as mb
        mb.mb_latent_append(s["ckv"], s["ld"], s["q"], s["gain"], s["pool"], s["q_rope"], s["pos"], s["slot"], s["T"],
                            s["num_pages"], s["heads"], s["hd"], s["rank"], EPS, THETA, _stream())
        return s["pool"], s["q_rope"]
    rank = s["rank"]
    x = s["ckv"].float()
    c = x[:, :rank]
    c = c * torch.rsqrt((c * c).mean(dim=1, keepdim=True) + EPS) * s["gain"].float()
    row = torch.cat([c, _rotate(x[:, rank:rank + ROPE], s["pos"])], dim=1)
    s["pool"].view(-1, rank + ROPE)[s["slot"].long()] = row.to(torch.bfloat16)
    s["q_rope"].copy_(_rotate(s["q"][..., s["hd"]:].float(), s["pos"]))
    return s["pool"], s["q_rope"]


def _work(s, size):
    if "work" not in s:   # the caller's workspace, kept from call to call
        s["work"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    return s["work"]


def _padded(s):
    """Cached rows [n, L, rank + 64], queries' token indices [n, N], and which of the keys each token sees [n, N, L]."""
    n, T, L = s["n"], s["T"], s["max_pages"] * PAGE
    qo, kv, bti = s["qo"].long(), s["kv"].long(), s["bti"].long()
    col = torch.arange(s["max_pages"], device=DEV)
    at = bti[:-1, None] + col
    page = torch.where(col < (bti[1:] - bti[:-1])[:, None], s["bt"].long()[at.clamp_max(s["bt"].numel() - 1)], 0)
    pos = torch.arange(L, device=DEV)
    rows = s["pool"][page].reshape(n, L, -1).float()
    rows = torch.where((pos < kv[:, None])[:, :, None], rows, 0.0)
    node = torch.arange(s["max_new"], device=DEV)
    tok = (qo[:-1, None] + node).clamp_max(T - 1)
    last = (kv - (qo[1:] - qo[:-1]))[:, None] + node          # the last key that a token sees
    return rows, tok, pos <= last[:, :, None]


def _unpad(s, o):
    """[n, N, heads, hd] -> the rows of o."""
    qo = s["qo"].long()
    t = torch.arange(s["T"], device=DEV)
    r = torch.searchsorted(qo[1:].contiguous(), t, right=True)
    s["o"].copy_(o[r, t - qo[r]].reshape(s["T"], -1))
    return s["o"]


def _softmax(z):
    p = torch.exp(z - z.amax(dim=-1, keepdim=True).clamp_min(-1e30))
    return p / p.sum(dim=-1, keepdim=True)


def _run_absorbed(s):
    if own:
        from mixed_prefill_decode_gb300 import binding as mb
        mb.mb_latent_attention(s["q"], s["q_rope"], s["w_kv"], s["pool"], s["o"], s["num_pages"], s["heads"], s["hd"],
                               s["rank"], s["scale"], s["n"], s["T"], s["qo"], s["kv"], s["bti"], s["bt"],
                               _work(s, mb.mb_latent_attention_workspace_bytes(s["T"], s["heads"], s["rank"])),
                               _stream())
        return s["o"]
    n, H, hd, rank = s["n"], s["heads"], s["hd"], s["rank"]
    rows, tok, see = _padded(s)
    N = tok.shape[1]
    w = s["w_kv"].float()
    q = torch.cat([torch.einsum("thd,hdr->thr", s["q"][..., :hd].float(), w[:, :hd]), s["q_rope"].float()], dim=2)
    q = q[tok].reshape(n, N * H, rank + ROPE)
    z = ((q @ rows.transpose(1, 2)) * s["scale"]).reshape(n, N, H, -1)
    p = _softmax(torch.where(see[:, :, None, :], z, float("-inf")))
    o = (p.reshape(n, N * H, -1) @ rows[..., :rank]).reshape(n, N, H, rank)
    return _unpad(s, torch.einsum("nthr,hdr->nthd", o, w[:, hd:]))


def _run_expanded(s):
    if own:
        from mixed_prefill_decode_gb300 import binding as mb
        mb.mb_latent_prefill(s["q"], s["q_rope"], s["w_kv"], s["pool"], s["o"], s["num_pages"], s["heads"], s["hd"],
                             s["rank"], s["scale"], s["n"], s["T"], s["qo"], s["kv"], s["bti"], s["bt"],
                             s["kv_tokens"],
                             _work(s, mb.mb_latent_prefill_workspace_bytes(s["kv_tokens"], s["n"], s["heads"], s["hd"],
                                                                           s["rank"])), _stream())
        return s["o"]
    n, H, hd, rank = s["n"], s["heads"], s["hd"], s["rank"]
    rows, tok, see = _padded(s)
    w = s["w_kv"].float()
    kv = torch.einsum("nlr,hdr->nhld", rows[..., :rank], w)
    k = torch.cat([kv[..., :hd], rows[:, None, :, rank:].expand(-1, H, -1, -1)], dim=3)
    q = torch.cat([s["q"][..., :hd], s["q_rope"]], dim=2)[tok].float().transpose(1, 2)     # [n, H, N, hd + 64]
    z = (q @ k.transpose(2, 3)) * s["scale"]
    p = _softmax(torch.where(see[:, None], z, float("-inf")))
    return _unpad(s, (p @ kv[..., hd:]).transpose(1, 2))


# ------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "tables":
        mean = c["kv_lo"] if c["kv_hi"] == c["kv_lo"] else (c["kv_hi"] - c["kv_lo"]) / math.log(c["kv_hi"] / c["kv_lo"])
        tokens = c["n"] - c["chunks"] + c["chunks"] * c["chunk"]
        pages = (c["n"] * mean + tokens) / PAGE
        return {"bytes": int(8 * pages + 12 * tokens + 28 * c["n"]), "flops": 0}
    H, rank, hd = c["heads"], c["rank"], c["hd"]
    if c["op"] == "append":
        return {"bytes": int(c["T"] * (4 * (rank + ROPE) + 4 * H * ROPE + 8)), "flops": int(c["T"] * 6 * H * ROPE)}
    new = c["n"] * (c["qo_lo"] + c["qo_hi"]) / 2
    if c["op"] == "absorbed":
        mean = c["kv_lo"] if c["kv_hi"] == c["kv_lo"] else (c["kv_hi"] - c["kv_lo"]) / math.log(c["kv_hi"] / c["kv_lo"])
        keys = c["n"] * mean
        pairs = new * mean
        flops = 2 * pairs * H * (2 * rank + ROPE) + 4 * new * H * hd * rank
    else:
        lo, hi = c["pre_lo"] + 0.5, c["pre_hi"] + 0.5
        mean = lo if hi == lo else (hi - lo) / math.log(hi / lo)
        keys = c["n"] * mean + new
        pairs = new * (mean + new / c["n"] / 2)
        flops = 2 * pairs * H * (2 * hd + ROPE) + 4 * keys * H * hd * rank
    bytes_ = 2 * (keys * (rank + ROPE) + 2 * H * hd * rank + new * H * (2 * hd + ROPE))
    return {"bytes": int(bytes_), "flops": int(flops)}


# ------------------------------------------------------------------ exact
def exact(case, seed):
    s = prepare(case, seed)
    return {"tables": _exact_tables, "append": _exact_append, "absorbed": _exact_attention,
            "expanded": _exact_attention}[s["op"]](s)


def _exact_tables(s):
    """Whole numbers only: request by request, page by page."""
    a = {k: s[k].cpu().numpy().astype(np.int64) for k in ("slots", "cached", "new", "tables", "owned", "ring", "state",
                                                          "bt")}
    head, count, asked = int(a["state"][0]), int(a["state"][1]), 0
    qo, bti, kvs, bt, req, pos, slot = [0], [0], [], [], [], [], []
    left = count
    for r in range(s["n"]):
        at, c, m = int(a["slots"][r]), int(a["cached"][r]), int(a["new"][r])
        need = max(0, -(-(c + m) // PAGE) - int(a["owned"][at]))
        asked += need
        if need and asked > count:
            m = need = 0
        for _ in range(need):
            a["tables"][at, a["owned"][at]] = a["ring"][head]
            a["owned"][at] += 1
            head, left = (head + 1) % s["num_pages"], left - 1
        pages = a["tables"][at, :-(-(c + m) // PAGE)]
        bt.extend(pages.tolist())
        kvs.append(c + m)
        p = np.arange(c, c + m)
        req.extend([r] * m)
        pos.extend(p.tolist())
        slot.extend((pages[p // PAGE] * PAGE + p % PAGE).tolist())
        qo.append(qo[-1] + m)
        bti.append(bti[-1] + len(pages))
    rest = s["T"] - len(req)
    full = a["bt"].copy()
    full[:len(bt)] = bt
    return tuple(np.asarray(x, np.int32) for x in (
        qo, kvs, bti, full, req + [-1] * rest, pos + [-1] * rest, slot + [-1] * rest, a["tables"], a["owned"],
        [head, left, 0, 0]))


def _exact_append(s):
    rank, half = s["rank"], ROPE // 2
    freq = THETA ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
    turn = torch.polar(torch.ones(s["T"], half, dtype=torch.float64, device=DEV), s["pos"].double()[:, None] * freq)
    x = s["ckv"].double()
    pool = s["pool"].double().view(-1, rank + ROPE)
    k = torch.complex(x[:, rank:rank + half], x[:, rank + half:rank + ROPE]) * turn
    c = x[:, :rank] / torch.sqrt(x[:, :rank].square().sum(dim=1, keepdim=True) / rank + EPS) * s["gain"].double()
    for t, at in enumerate(s["slot"].tolist()):
        pool[at, :rank] = c[t]
        pool[at, rank:rank + half] = k[t].real
        pool[at, rank + half:] = k[t].imag
    q = s["q"].double()[:, :, s["hd"]:]
    q = torch.complex(q[..., :half].contiguous(), q[..., half:].contiguous()) * turn[:, None]
    return pool.view(s["num_pages"], PAGE, -1), torch.cat([q.real, q.imag], dim=2)


def _exact_attention(s):
    qo, kv, bti = (s[k].cpu().numpy() for k in ("qo", "kv", "bti"))
    hd, rank = s["hd"], s["rank"]
    out = torch.empty(s["T"], s["heads"], hd, dtype=torch.float64, device=DEV)
    for r in range(s["n"]):
        a, b, k = int(qo[r]), int(qo[r + 1]), int(kv[r])
        rows = s["pool"][s["bt"][int(bti[r]):int(bti[r]) + -(-k // PAGE)].long()].reshape(-1, rank + ROPE)[:k].double()
        hidden = torch.arange(k, device=DEV)[None, :] > torch.arange(k - (b - a), k, device=DEV)[:, None]
        for h in range(s["heads"]):
            w = s["w_kv"][h].double()
            if b - a < 64:   # the same numbers either way; the cheaper order
                z = (s["q"][a:b, h, :hd].double() @ w[:hd]) @ rows[:, :rank].T
            else:
                z = s["q"][a:b, h, :hd].double() @ (rows[:, :rank] @ w[:hd].T).T
            z = (z + s["q_rope"][a:b, h].double() @ rows[:, rank:].T) * s["scale"]
            p = torch.softmax(z.masked_fill(hidden, float("-inf")), dim=1)
            out[a:b, h] = (p @ rows[:, :rank]) @ w[hd:].T
    return out.reshape(s["T"], -1)
