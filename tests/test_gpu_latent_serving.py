"""The latent-cache operators together, as a serving loop uses them: each
step builds its descriptor on the GPU, appends the new tokens' rows, attends
(chunks expanded, single tokens absorbed), and the next one goes on from its
lengths; steps of single tokens run as one captured graph.

Every row of the cache is compared with the oracle's (its bounds are those of
the append test), every step's output with the exact attention over the rows
that the cache holds (bounds as in test_gpu_latent)."""

import numpy as np
import pytest
import torch

from oracle import latent as OL
from gpu_util import f64, from_dev, to_dev
from test_gpu_latent import U, _bf16, _i32, all_elements, near_exact

pytestmark = pytest.mark.gpu
EPS, THETA = 1e-6, 10000.0


class Server:
    """Rows of tables and one layer's latent cache; `tokens` keeps what each
    request was given, to follow it on the host."""

    def __init__(self, mb, H, hd, rank, slots, pages, max_pages, most, seed):
        self.mb, self.H, self.hd, self.rank, self.S, self.P, self.M, self.most = mb, H, hd, rank, slots, pages, max_pages, most
        rng = self.rng = np.random.default_rng(seed)
        self.w, self.gain, self.scale = _bf16(rng, H, 2 * hd, rank, scale=rank ** -0.5), _bf16(rng, rank), (hd + 64) ** -0.5
        self.d = dict(tables=_i32(np.zeros((slots, max_pages))), owned=_i32(np.zeros(slots)), ring=_i32(rng.permutation(pages)),
                      state=_i32([5 % pages, pages, 0, 0]), w=to_dev(self.w), gain=to_dev(self.gain))
        self.pool = torch.full((pages, 16, rank + 64), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.ckv = torch.zeros(most, rank + 64, dtype=torch.bfloat16, device="cuda")
        self.q = torch.zeros(most, H, hd + 64, dtype=torch.bfloat16, device="cuda")
        self.q_rope = torch.zeros(most, H, 64, dtype=torch.bfloat16, device="cuda")
        self.o = torch.zeros(most, H * hd, dtype=torch.bfloat16, device="cuda")
        self.work = torch.empty(mb.mb_latent_attention_workspace_bytes(most, H, rank), dtype=torch.uint8, device="cuda")
        self.given = {}

    def batch(self, slots, cached, new):
        """The step's own arrays (a graph keeps them)."""
        n, cap = len(slots), self.P
        b = dict(n=n, slots=_i32(slots), cached=_i32(cached), new=_i32(new))
        for k, size in (("qo", n + 1), ("kv", n), ("bti", n + 1), ("bt", cap), ("req", self.most), ("pos", self.most), ("slot", self.most)):
            b[k] = torch.zeros(size, dtype=torch.int32, device="cuda")
        return b

    def issue(self, b, chunks, kv_tokens):
        """One step on the current stream; the first `chunks` requests attend in
        the expanded form, the others in the absorbed one."""
        mb, st, n = self.mb, torch.cuda.current_stream().cuda_stream, b["n"]
        mb.mb_batch_tables(b["slots"], b["cached"], b["new"], n, self.most, self.P, self.d["tables"], self.d["owned"], self.S,
                           self.M, self.d["ring"], self.d["state"], self.P, b["qo"], b["kv"], b["bti"], b["bt"], b["req"],
                           b["pos"], b["slot"], st)
        mb.mb_latent_append(self.ckv, self.rank + 64, self.q, self.d["gain"], self.pool, self.q_rope, b["pos"], b["slot"],
                            self.most, self.P, self.H, self.hd, self.rank, EPS, THETA, st)
        common = [self.q, self.q_rope, self.d["w"], self.pool, self.o, self.P, self.H, self.hd, self.rank, self.scale]
        if chunks:
            size = mb.mb_latent_prefill_workspace_bytes(kv_tokens, chunks, self.H, self.hd, self.rank)
            mb.mb_latent_prefill(*common, chunks, self.most, b["qo"], b["kv"], b["bti"], b["bt"], kv_tokens,
                                 torch.empty(size, dtype=torch.uint8, device="cuda"), st)
        if n > chunks:
            mb.mb_latent_attention(*common, n - chunks, self.most, b["qo"][chunks:], b["kv"][chunks:], b["bti"][chunks:],
                                   b["bt"], self.work, st)

    def draw(self):
        ckv, q = _bf16(self.rng, self.most, self.rank + 64, scale=2.0), _bf16(self.rng, self.most, self.H, self.hd + 64)
        self.ckv.copy_(to_dev(ckv))
        self.q.copy_(to_dev(q))
        return f64(ckv), f64(q)

    def follow(self, b, slots, cached, new, ckv, q, chunks):
        """What the step must have done."""
        torch.cuda.synchronize()
        self.mb.mb_device_status(None, torch.cuda.current_stream().cuda_stream)
        qo, kv, bti, bt = (b[k].cpu().numpy() for k in ("qo", "kv", "bti", "bt"))
        assert np.array_equal(np.diff(qo), new) and np.array_equal(kv, np.add(cached, new))
        pool, q_rope = f64(from_dev(self.pool)), f64(from_dev(self.q_rope))
        got, parts = f64(from_dev(self.o)).reshape(self.most, self.H, self.hd), []
        seen = set()
        for r, s in enumerate(slots):
            pages = bt[bti[r]:bti[r + 1]]
            assert len(pages) == -(-int(kv[r]) // 16) and not seen & set(pages.tolist())
            seen |= set(pages.tolist())
            rows = pool[pages].reshape(-1, self.rank + 64)[:kv[r]]
            mine = self.given.setdefault(int(s), [])[:cached[r]] + [ckv[t] for t in range(qo[r], qo[r + 1])]
            self.given[int(s)] = mine
            assert len(mine) == kv[r]
            for p, x in enumerate(mine):
                want = OL.append_row(x, f64(self.gain), p, EPS, THETA)
                tol = np.abs(want) * (U + (self.rank + 4) * 2.0 ** -24) * 1.01 + 1e-30
                pair = np.abs(x[self.rank:self.rank + 32]) + np.abs(x[self.rank + 32:])
                tol[self.rank:] += np.tile(pair, 2) * 2.0 ** -18
                assert np.all(np.abs(rows[p] - want) <= tol), (r, p)
            a, e = int(qo[r]), int(qo[r + 1])
            if e > a:
                parts.append(near_exact(got[a:e], q[a:e, :, :self.hd], q_rope[a:e], f64(self.w), rows, self.scale,
                                        "expanded" if r < chunks else "absorbed"))
        if parts:
            all_elements(parts)


@pytest.mark.parametrize("H,hd,rank", [(8, 64, 256), (5, 128, 512)])
def test_a_serving_loop(mb, H, hd, rank):
    s = Server(mb, H, hd, rank, slots=6, pages=40, max_pages=20, most=200, seed=H)
    slots = [4, 1, 3, 0]
    # prompts of three requests in chunks, beside the first single tokens of one that is through
    cached = np.zeros(4, np.int64)
    for new, chunks in (([60, 37, 5, 17], 4), ([33, 1, 64, 1], 4), ([50, 7, 1, 1], 2)):
        b = s.batch(slots, cached, new)
        ckv, q = s.draw()
        s.issue(b, chunks, kv_tokens=int(np.sum(cached + new)))
        s.follow(b, slots, cached, new, ckv, q, chunks)
        cached = cached + new
    # three drafted tokens each, of which two are kept
    b = s.batch(slots, cached, [3] * 4)
    ckv, q = s.draw()
    s.issue(b, 0, 0)
    s.follow(b, slots, cached, [3] * 4, ckv, q, 0)
    cached = cached + 2
    # one request ends, another takes its row and its pages
    mb.mb_tables_release(_i32([3]), 1, s.d["tables"], s.d["owned"], s.S, s.M, s.d["ring"], s.d["state"], s.P,
                         torch.cuda.current_stream().cuda_stream)
    cached[2] = 0
    s.given[3] = []
    new = [1, 1, 90, 1]
    order = [2, 0, 1, 3]       # the chunk first
    slots, cached, new = [slots[i] for i in order], cached[order], [new[i] for i in order]
    b = s.batch(slots, cached, new)
    ckv, q = s.draw()
    s.issue(b, 1, 90)
    s.follow(b, slots, cached, new, ckv, q, 1)
    cached = cached + new
    # single tokens, captured once and replayed: the lengths go on by themselves
    b = s.batch(slots, cached, [1] * 4)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        s.issue(b, 0, 0)
        b["cached"].copy_(b["kv"])
    for _ in range(18):
        ckv, q = s.draw()
        graph.replay()
        s.follow(b, slots, cached, [1] * 4, ckv, q, 0)
        cached = cached + 1


def test_a_batch_that_does_not_fit_waits(mb):
    """Two requests, pages for one: the other's turn comes when the first ends."""
    s = Server(mb, 4, 64, 256, slots=2, pages=3, max_pages=8, most=64, seed=3)
    b = s.batch([0, 1], [0, 0], [30, 20])
    ckv, q = s.draw()
    s.issue(b, 2, 50)
    torch.cuda.synchronize()
    assert b["qo"].tolist() == [0, 30, 30] and b["kv"].tolist() == [30, 0]
    s.follow(b, [0, 1], [0, 0], [30, 0], ckv, q, 2)
    mb.mb_tables_release(_i32([0]), 1, s.d["tables"], s.d["owned"], s.S, s.M, s.d["ring"], s.d["state"], s.P,
                         torch.cuda.current_stream().cuda_stream)
    s.given = {}
    b = s.batch([1], [0], [20])
    ckv, q = s.draw()
    s.issue(b, 0, 0)
    s.follow(b, [1], [0], [20], ckv, q, 0)
