"""GPU parity of the drafted-token operators against the float64 oracle.

Tree attention, elementwise.  With p the exact probabilities, A = sum_j p_j
|v_j| and B = max_j sum_d |q_d k_jd| / sqrt(hd), a kernel that keeps logits,
maxima, sums and o in fp32, rounds its probabilities to bf16 for the product
with V and o to bf16 at the end is off by at most
  2^-8 |o|                     the output's rounding (half a step)
+ 2^-8 A                       the probabilities' rounding
+ 2 d A                        d = relative error of an unrounded probability:
                               (hd + 4) 2^-24 B from the fp32 dot product and its scaling, plus
                               2^-21 from the exponential and the running reference; twice, as
                               the same errors sit in the sum that divides
+ 2^-20 A                      fp32 accumulation of o and the merge of key splits
(products of these terms are below 2^-14 A and covered by 1 % on top).

Verification: whole numbers, equal to the oracle's.  The cases keep clear of
borders closer than the kernel resolves: 1e-6 in probability for the
acceptance tests (fp32 sums and exponentials, 2^-21), 4e-9 for the last draw
(each weight off by at most 2^-29 of itself, in the sum below the border and in
the total: 2 2^-29).

Page operations: bit-exact."""

import numpy as np
import pytest
import torch

from oracle import layer as OL
from oracle import spec as OS
from mixed_prefill_decode_gb300 import workload as W
from gpu_util import f64, from_dev, to_dev

pytestmark = pytest.mark.gpu
SENT = 0x7FC1   # a NaN: what stale slots and unwritten rows hold


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=np.int32))).cuda()


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _parents(rng, n, kind):
    if kind == "chain":
        return np.arange(n) - 1
    if kind == "forest":          # several nodes hang on the prefix
        return np.array([rng.integers(-1, i) if i else -1 for i in range(n)], dtype=np.int64)
    if kind == "star":
        return np.where(np.arange(n) == 0, -1, 0)
    return np.array([rng.integers(max(0, (i - 1) // 3 - 1), i) if i else -1 for i in range(n)], dtype=np.int64)


class Trees:
    """A batch of trees: (cached, nodes) per request; stale slots hold NaN."""

    def __init__(self, reqs, hkv, g, hd, seed, kind="wide", spare_rows=3):
        rng = np.random.default_rng(seed)
        self.reqs, self.hkv, self.g, self.hd = reqs, hkv, g, hd
        need = [(c + n + 15) // 16 for c, n in reqs]
        self.P = sum(need) + 5
        perm = rng.permutation(self.P)
        self.qo = np.concatenate([[0], np.cumsum([n for _, n in reqs])]).astype(np.int32)
        self.kv = np.array([c + n for c, n in reqs], np.int32)
        self.bti = np.concatenate([[0], np.cumsum(need)]).astype(np.int32)
        self.bt = perm[:sum(need)].astype(np.int32) if sum(need) else np.zeros(1, np.int32)
        self.parent = np.concatenate([_parents(rng, n, kind) for _, n in reqs] + [np.zeros(spare_rows)]).astype(np.int32)
        self.rows = int(self.qo[-1])
        self.T = self.rows + spare_rows
        self.q = W.f32_to_bf16_bits(rng.standard_normal((self.T, hkv * g, hd), dtype=np.float32) *
                                    (1.0 + 3.0 * rng.random((self.T, 1, 1), dtype=np.float32)))
        self.pool = np.full((self.P, 2, hkv, 16, hd), SENT, np.uint16)
        for r, (c, n) in enumerate(reqs):
            for p in range(c + n):
                self.pool[self.bt[self.bti[r] + p // 16], :, :, p % 16] = W.f32_to_bf16_bits(
                    rng.standard_normal((2, hkv, hd), dtype=np.float32))

    def run(self, mb, work=None, **over):
        a = dict(qo=self.qo, kv=self.kv, bti=self.bti, bt=self.bt, parent=self.parent)
        a.update(over)
        self.dq, self.dpool = to_dev(self.q), to_dev(self.pool)
        self.dev = {k: _i32(v) for k, v in a.items()}
        if work is None:
            work = torch.full((mb.mb_tree_attention_workspace_bytes(),), 0xFF, dtype=torch.uint8, device="cuda")
        self.work = work
        self.o = to_dev(np.full((self.T, self.hkv * self.g * self.hd), SENT, np.uint16))
        self.call(mb)
        return self

    def call(self, mb, o=None, stream=None):
        d = self.dev
        mb.mb_tree_attention(self.dq, self.dpool, self.o if o is None else o, self.P, self.hkv * self.g, self.hkv,
                             self.hd, len(self.reqs), self.T, d["qo"], d["kv"], d["bti"], d["bt"], d["parent"],
                             self.work, _stream() if stream is None else stream)

    def check(self, bits, skip=()):
        got = bits.reshape(self.T, self.hkv * self.g, self.hd)
        assert np.all(got[self.rows:] == SENT), "rows behind the last request were written"
        pool = f64(self.pool)
        for r, (c, n) in enumerate(self.reqs):
            if n == 0:
                continue
            a, b = self.qo[r], self.qo[r + 1]
            if r in skip:
                assert np.all(got[a:b] == SENT)
                continue
            K, V = OL.gather_kv(pool, self.bt[self.bti[r]:self.bti[r + 1]], c + n)
            o, A, B = OS.tree_attention_request(f64(self.q[a:b]), K, V, self.parent[a:b])
            d = (self.hd + 4) * 2.0 ** -24 * B[..., None] + 2.0 ** -21
            bound = 1.01 * (2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2 * d + 2.0 ** -20) * A) + 1e-30
            err = np.abs(f64(got[a:b]) - o)
            assert np.all(err <= bound), (r, c, n, float(np.max(err / bound)))


CASES = {
    "one_token": ([(0, 1)], 2, 4, 128, "chain"),
    "no_prefix": ([(0, 5), (0, 17), (0, 128)], 2, 4, 128, "forest"),
    "page_edges": ([(15, 1), (16, 1), (14, 3), (1, 16), (31, 2)], 1, 8, 128, "wide"),
    "block_edges": ([(127, 1), (128, 1), (126, 4), (100, 64), (255, 2), (120, 128), (256, 128)], 2, 1, 128, "wide"),
    "empty_requests": ([(0, 0), (40, 7), (9, 0), (300, 3), (0, 0)], 2, 2, 64, "wide"),
    "group5_big": ([(700, 64), (33, 26), (511, 51)], 2, 5, 128, "wide"),
    "group8_big": ([(200, 128), (1000, 33)], 1, 8, 128, "forest"),
    "group7": ([(150, 37), (20, 19)], 2, 7, 64, "wide"),
    "group3_star": ([(64, 100), (5, 43)], 3, 3, 64, "star"),
    "chains_hd64": ([(77, 9), (400, 128)], 4, 1, 64, "chain"),
    "group6": ([(129, 22), (1, 21)], 1, 6, 128, "wide"),
    "long_splits": ([(5000, 6), (3, 2), (2047, 13)], 2, 4, 128, "wide"),
    "long_hd64": ([(9001, 40)], 1, 4, 64, "forest"),
}


@pytest.mark.parametrize("name", list(CASES))
def test_tree_attention_matches_oracle(mb, name):
    reqs, hkv, g, hd, kind = CASES[name]
    t = Trees(reqs, hkv, g, hd, 100 + len(name), kind).run(mb)
    mb.mb_device_status(None, _stream())
    t.check(from_dev(t.o))


@pytest.mark.parametrize("seed", range(6))
def test_tree_attention_random_batches(mb, seed):
    rng = np.random.default_rng(900 + seed)
    g, hd = [(1, 64), (2, 128), (4, 128), (5, 64), (8, 64), (3, 128)][seed]
    reqs = [(int(rng.integers(0, 900)), int(rng.integers(0, 40))) for _ in range(int(rng.integers(1, 40)))]
    t = Trees(reqs, 2, g, hd, seed, "forest").run(mb)
    mb.mb_device_status(None, _stream())
    t.check(from_dev(t.o))


def test_tree_attention_many_requests(mb):
    """More requests than threads of a CTA, most of them tiny."""
    rng = np.random.default_rng(77)
    reqs = [(int(rng.integers(0, 40)), int(rng.integers(0, 4))) for _ in range(700)]
    t = Trees(reqs, 1, 2, 64, 5).run(mb)
    mb.mb_device_status(None, _stream())
    t.check(from_dev(t.o))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("which", ["k", "v", "both"])
def test_tree_attention_hidden_nodes_may_hold_anything(mb, bad, which):
    """Non-finite keys and values of nodes reach only the nodes that see them."""
    t = Trees([(130, 24), (60, 70), (0, 20)], 2, 4, 128, 11)
    bits = np.uint16(W.f32_to_bf16_bits(np.array([bad], np.float32))[0])
    clean = Trees([(130, 24), (60, 70), (0, 20)], 2, 4, 128, 11).run(mb)
    blind = {}
    for r, node in ((0, 5), (1, 9), (1, 66), (2, 3)):
        pos = t.kv[r] - (t.qo[r + 1] - t.qo[r]) + node
        page, slot = t.bt[t.bti[r] + pos // 16], pos % 16
        if which in ("k", "both"):
            t.pool[page, 0, :, slot, 3:70] = bits
        if which in ("v", "both"):
            t.pool[page, 1, :, slot, 1::2] = bits
        see = OS.ancestors(t.parent[t.qo[r]:t.qo[r + 1]])[:, node]
        for i in np.nonzero(see)[0]:
            blind[t.qo[r] + i] = True
    t.run(mb)
    mb.mb_device_status(None, _stream())
    got, ref = f64(from_dev(t.o)), f64(from_dev(clean.o))
    keep = np.array([i not in blind for i in range(t.rows)])
    assert keep.sum() > 40 and np.array_equal(got[:t.rows][keep], ref[:t.rows][keep])
    if which != "k":
        seen = f64(from_dev(t.o))[np.array(sorted(blind))][:, 1::2]
        assert not np.any(np.isfinite(seen))


def test_tree_attention_is_deterministic_and_ignores_the_workspaces_contents(mb):
    reqs = [(4000, 20), (12, 3), (900, 64)]
    t = Trees(reqs, 2, 4, 128, 21).run(mb)
    first = from_dev(t.o)
    t.work.fill_(0x5A)
    o2 = torch.empty_like(t.o)
    o2.copy_(t.o)
    t.call(mb, o2)
    assert np.array_equal(first, from_dev(o2))
    # the plain order of requests does not matter to a request's numbers beyond rounding: checked by the oracle
    t.check(first)


def test_tree_attention_in_a_graph_and_on_two_streams(mb):
    """A captured call replayed with other contents, and two calls at once with workspaces of their own."""
    t = Trees([(2500, 12), (77, 30)], 2, 4, 128, 31).run(mb)
    u = Trees([(1800, 40)], 2, 4, 128, 32).run(mb)
    mb.mb_device_status(None, _stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        t.call(mb)
    q2 = torch.randn_like(t.dq.float()).to(torch.bfloat16)
    t.dq.copy_(q2)
    t.q = from_dev(q2)
    t.o.view(torch.int16).fill_(SENT)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        with torch.cuda.stream(s1):
            g.replay()
        u.call(mb, stream=s2.cuda_stream)
    torch.cuda.synchronize()
    mb.mb_device_status(None, _stream())
    t.check(from_dev(t.o))
    u.check(from_dev(u.o))


def test_tree_attention_descriptor_faults_are_reported_and_harmless(mb):
    """Requests that break a rule are skipped, the others computed."""
    reqs = [(50, 4), (20, 6), (30, 5), (64, 3)]
    for what in ("kv_below_nodes", "short_table", "negative_kv", "too_many"):
        t = Trees(reqs, 2, 4, 128, 41)
        kv, bti, qo = t.kv.copy(), t.bti.copy(), t.qo.copy()
        if what == "kv_below_nodes":
            kv[1] = 5
        elif what == "negative_kv":
            kv[1] = -3
        elif what == "short_table":
            kv[1] = 16 * (bti[2] - bti[1]) + 1
        else:
            t = Trees([(50, 4), (20, 129), (30, 5), (64, 3)], 2, 4, 128, 41)
            kv, bti, qo = t.kv.copy(), t.bti.copy(), t.qo.copy()
        t.run(mb, kv=kv, bti=bti, qo=qo)
        with pytest.raises(mb.MbError) as e:
            mb.mb_device_status(None, _stream())
        assert e.value.status == mb.MB_EDEVICE
        t.check(from_dev(t.o), skip=(1,))
    # a parent out of range counts as -1, a page out of range as page 0
    t = Trees(reqs, 2, 4, 128, 43)
    par = t.parent.copy()
    par[t.qo[2] + 2] = 4
    t.run(mb, parent=par)
    t.parent[t.qo[2] + 2] = -1
    with pytest.raises(mb.MbError):
        mb.mb_device_status(None, _stream())
    t.check(from_dev(t.o))
    t = Trees(reqs, 2, 4, 128, 44)
    bt = t.bt.copy()
    bt[t.bti[1]] = t.P + 7
    t.run(mb, bt=bt)
    with pytest.raises(mb.MbError):
        mb.mb_device_status(None, _stream())
    t.check_others = [0, 2, 3]
    got = from_dev(t.o).reshape(t.T, -1)
    keep = Trees(reqs, 2, 4, 128, 44).run(mb)
    ref = from_dev(keep.o).reshape(t.T, -1)
    for r in (0, 2, 3):
        assert np.array_equal(got[t.qo[r]:t.qo[r + 1]], ref[t.qo[r]:t.qo[r + 1]])


# ------------------------------------------------------------ verification
class Drafts:
    def __init__(self, sizes, vocab, mode, seed, kind="wide", temps=None, agree=0.7):
        rng = np.random.default_rng(seed)
        self.sizes, self.V, self.mode = sizes, vocab, mode
        self.qo = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
        T = self.T = int(self.qo[-1])
        self.parent = np.concatenate([_parents(rng, m, kind) for m in sizes] or [np.zeros(0)]).astype(np.int32)
        self.temp = np.asarray(temps if temps is not None else 0.5 + rng.random(len(sizes)), np.float32)
        logits = 2.0 * rng.standard_normal((T, vocab))
        self.tokens = rng.integers(0, vocab, size=T).astype(np.int32)
        self.probs = None
        if mode == "probs":
            q = np.exp(logits + 0.7 * rng.standard_normal((T, vocab)))
            self.probs = (q / q.sum(1, keepdims=True)).astype(np.float32)
        for r in range(len(sizes)):
            for i in range(1, sizes[r]):
                t, up = self.qo[r] + i, self.qo[r] + max(0, self.parent[self.qo[r] + i])
                if mode == "probs":
                    self.tokens[t] = rng.choice(vocab, p=self.probs[up].astype(np.float64) / self.probs[up].sum(dtype=np.float64))
                if rng.random() < agree:
                    logits[up, self.tokens[t]] += (0.8 if mode == "probs" else 1.3) * np.log(vocab)
        self.logits = W.f32_to_bf16_bits(logits.astype(np.float32))
        self.u_accept = rng.random(T, dtype=np.float32)
        self.u_final = rng.random(len(sizes), dtype=np.float32)

    def run(self, mb, max_path=16, sampling=True):
        n = len(self.sizes)
        d = self.dev = dict(logits=to_dev(self.logits), tokens=_i32(self.tokens), qo=_i32(self.qo), parent=_i32(self.parent),
                            probs=None if self.probs is None else torch.from_numpy(self.probs).cuda(),
                            temp=torch.from_numpy(self.temp).cuda() if sampling else None,
                            ua=torch.from_numpy(self.u_accept).cuda() if sampling else None,
                            uf=torch.from_numpy(self.u_final).cuda() if sampling else None)
        out = [torch.full(s, -7, dtype=torch.int32, device="cuda") for s in ((n,), (n, max_path), (n,))]
        mb.mb_verify_tree(d["logits"], self.V, d["tokens"], d["probs"], n, self.T, d["qo"], d["parent"], d["temp"],
                          d["ua"], d["uf"], max_path, *out, _stream())
        return [x.cpu().numpy() for x in out]

    def expect(self, max_path=16, sampling=True):
        lg = f64(self.logits)
        want = []
        for r in range(len(self.sizes)):
            a, b = self.qo[r], self.qo[r + 1]
            if a == b:
                want.append(([], -1, (np.inf, np.inf)))
                continue
            want.append(OS.verify(lg[a:b], self.tokens[a:b], None if self.probs is None else self.probs[a:b].astype(np.float64),
                                  self.parent[a:b], float(self.temp[r]) if sampling else 0.0,
                                  self.u_accept[a:b].astype(np.float64), float(self.u_final[r]), max_path))
        return want

    def check(self, got, max_path=16, sampling=True):
        count, path, nxt = got
        for r, (p, tok, (tests, last)) in enumerate(self.expect(max_path, sampling)):
            assert tests > 1e-6 and last > 4e-9, "the case sits on a border"
            assert list(path[r]) == p + [-1] * (max_path - len(p)) and count[r] == len(p) and nxt[r] == tok, \
                (r, p, tok, list(path[r]), count[r], nxt[r])


@pytest.mark.parametrize("mode", ["points", "probs"])
@pytest.mark.parametrize("vocab", [8, 96, 1000, 32000])
@pytest.mark.parametrize("kind", ["chain", "wide", "star"])
def test_verify_matches_oracle(mb, mode, vocab, kind):
    d = Drafts([1, 6, 13, 2, 0, 25, 5, 9], vocab, mode, 7 * vocab + len(kind), kind)
    got = d.run(mb)
    mb.mb_device_status(None, _stream())
    d.check(got)


@pytest.mark.parametrize("mode,n,vocab", [("points", 1, 128256), ("probs", 2, 151936), ("probs", 70, 4096), ("points", 200, 2048)])
def test_verify_sizes(mb, mode, n, vocab):
    d = Drafts([4] * n if vocab > 100000 else [1 + (i % 7) for i in range(n)], vocab, mode, 3, "wide")
    got = d.run(mb)
    mb.mb_device_status(None, _stream())
    d.check(got)


@pytest.mark.parametrize("vocab", [8, 32000])
def test_verify_greedy(mb, vocab):
    d = Drafts([1, 6, 13, 128, 25], vocab, "points", 5, "wide")
    lg = f64(d.logits)
    for r in range(5):   # most nodes carry their parent's argmax
        for i in range(1, d.sizes[r]):
            if (i * 7 + r) % 3:
                d.tokens[d.qo[r] + i] = int(np.argmax(lg[d.qo[r] + d.parent[d.qo[r] + i]]))
    got = d.run(mb, sampling=False)
    d.check(got, sampling=False)
    d.temp[:] = 0.0   # the same, asked for by temperature 0 beside a sampling request
    d.temp[2] = 0.9
    d.check(d.run(mb))
    mb.mb_device_status(None, _stream())


def test_verify_path_limit(mb):
    d = Drafts([40, 40], 64, "points", 9, "chain", agree=1.0)
    d.u_accept[:] = 0.0
    for lim in (1, 2, 7, 40, 64):
        got = d.run(mb, max_path=lim)
        assert got[0].max() == min(lim, 40)
        d.check(got, lim)


def test_verify_long_chain_all_accepted(mb):
    d = Drafts([128], 256, "probs", 10, "chain")
    d.u_accept[:] = 0.0
    got = d.run(mb, max_path=128)
    assert got[0][0] == 128 and list(got[1][0]) == list(range(128))
    d.check(got, 128)


def test_verify_special_logits(mb):
    """-inf and NaN logits have no chance, +inf takes everything, a row of
    nothing gives token 0, ties go to the lowest index."""
    V = 64
    d = Drafts([2, 2, 1, 1, 2, 1], V, "points", 12, "chain", temps=[1, 1, 1, 1, 0, 1e-3])
    lg = f64(d.logits).astype(np.float32)
    d.tokens[:] = 3
    lg[0, 3] = -np.inf                       # the draft has no chance
    lg[2, 3] = np.nan
    lg[4, :] = -np.inf
    lg[5, :] = -np.inf
    lg[5, [7, 9]] = np.inf
    lg[6, :] = 1.0                            # greedy tie: token 0
    d.logits = W.f32_to_bf16_bits(lg)
    d.logits[2, 3] = SENT
    d.logits[8, 20] = SENT
    got = d.run(mb)
    assert list(got[0]) == [1, 1, 1, 1, 1, 1]
    assert got[2][2] == 0 and got[2][3] in (7, 9) and got[2][4] == 0
    d.check(got)


def test_verify_reports_bad_descriptors(mb):
    d = Drafts([3, 4], 64, "points", 13, "star")
    good = d.run(mb)
    d.tokens[5] = 64
    d.run(mb)
    with pytest.raises(mb.MbError) as e:
        mb.mb_device_status(None, _stream())
    assert e.value.status == mb.MB_EDEVICE
    d = Drafts([3, 4], 64, "points", 13, "star")
    d.qo[2] = 300          # rows past T
    d.T = 7
    got = d.run(mb)
    with pytest.raises(mb.MbError):
        mb.mb_device_status(None, _stream())
    assert got[0][0] == good[0][0] and got[0][1] == 0 and got[2][1] == -1 and np.all(got[1][1] == -1)
    d = Drafts([3, 4], 64, "points", 13, "star", temps=[-1.0, float("nan")])
    d.run(mb)
    with pytest.raises(mb.MbError):
        mb.mb_device_status(None, _stream())


@pytest.mark.parametrize("mode", ["points", "probs"])
@pytest.mark.parametrize("sizes,vocab,kind,seed", [([128, 70, 33], 96, "star", 21), ([90], 40000, "star", 22),
                                                   ([3], 1 << 19, "chain", 23), ([2, 3], 262144, "star", 24),
                                                   ([5, 5], 65536, "wide", 25)])
def test_verify_many_children_and_large_vocabularies(mb, mode, sizes, vocab, kind, seed):
    """More children than a warp has lanes; every cluster size up to the largest row."""
    d = Drafts(sizes, vocab, mode, seed, kind, agree=0.1 if sizes[0] > 30 else 0.7)
    got = d.run(mb)
    mb.mb_device_status(None, _stream())
    d.check(got)


def test_verify_draft_equal_to_the_target_and_useless_drafts(mb):
    """q = p: a refusal leaves nothing or next to nothing, and the draw still has
    a token.  A q of 1 on the child, 0 elsewhere, and not a number elsewhere: no
    weight becomes negative."""
    V = 4096
    d = Drafts([2, 2, 2, 2], V, "probs", 26, "chain", temps=[1, 1, 1, 1])
    p = np.exp(f64(d.logits) - f64(d.logits).max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    d.probs[:] = p.astype(np.float32)
    for r in (1, 2, 3):
        d.probs[2 * r] = 0.0
        d.probs[2 * r, d.tokens[2 * r + 1]] = 1.0
    d.probs[6, :7] = np.nan
    d.u_accept[:] = 1.0 - 2.0 ** -24
    got = d.run(mb)
    mb.mb_device_status(None, _stream())
    assert np.all(got[0] >= 1) and np.all((got[2] >= 0) & (got[2] < V))
    for r in (1, 2):
        p_child = p[2 * r, d.tokens[2 * r + 1]]
        if got[0][r] == 1:
            assert d.u_accept[2 * r + 1] >= p_child * (1 - 1e-6) and got[2][r] != d.tokens[2 * r + 1]
    if got[0][3] == 1:
        assert got[2][3] >= 7   # a q that is not a number takes the token away


def test_rows_given_by_words_that_wrap_around_are_refused(mb):
    """qo_indptr words whose difference overflows to a valid size."""
    t = Trees([(50, 40)], 2, 4, 128, 45)
    wrap = np.array([2 ** 31 - 21, -2 ** 31 + 19], np.int32)   # 40 rows by subtraction in 32 bits
    t.run(mb, qo=wrap)
    with pytest.raises(mb.MbError) as e:
        mb.mb_device_status(None, _stream())
    assert e.value.status == mb.MB_EDEVICE
    assert np.all(t.o.view(torch.int16).cpu().numpy().view(np.uint16) == SENT)
    d = Drafts([40], 64, "points", 27, "wide")
    d.qo = wrap
    count, path, nxt = d.run(mb)
    with pytest.raises(mb.MbError):
        mb.mb_device_status(None, _stream())
    assert count[0] == 0 and nxt[0] == -1 and np.all(path == -1)
    pool = torch.zeros((4, 2, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    new = torch.full((1,), -7, dtype=torch.int32, device="cuda")
    mb.mb_kv_compact([pool], 4, 2, 64, 1, _i32(wrap), _i32([60]), _i32([0, 4]), _i32([0, 1, 2, 3]), _i32([1]),
                     _i32([[0]]), 1, new, _stream())
    with pytest.raises(mb.MbError):
        mb.mb_device_status(None, _stream())
    assert new.item() == -7


def test_verify_and_compact_in_a_graph_beside_another_stream(mb):
    """Verification and compaction captured together follow new logits, numbers
    and paths, while eager calls run on another stream."""
    sizes, V, hkv, hd = [6, 9, 1, 13], 8192, 2, 64
    d = Drafts(sizes, V, "points", 28, "wide")
    e = Drafts(sizes, V, "points", 29, "wide")
    other = Drafts([7, 3], 32000, "probs", 30, "wide")
    n, L = len(sizes), 16
    kv = np.array([20 + s for s in sizes], np.int32)
    need = (kv + 15) // 16
    bti = np.concatenate([[0], np.cumsum(need)]).astype(np.int32)
    bt = np.arange(bti[-1]).astype(np.int32)[::-1].copy()
    rng = np.random.default_rng(31)
    pools = rng.integers(0, 1 << 16, size=(2, int(bti[-1]), 2, hkv, 16, hd)).astype(np.uint16)
    d.run(mb)
    v = d.dev
    dev = [to_dev(p) for p in pools]
    out = [torch.full(s, -7, dtype=torch.int32, device="cuda") for s in ((n,), (n, L), (n,))]
    dkv, dbti, dbt = _i32(kv), _i32(bti), _i32(bt)
    new = torch.zeros_like(dkv)

    def step():
        s = _stream()
        mb.mb_verify_tree(v["logits"], V, v["tokens"], v["probs"], n, d.T, v["qo"], v["parent"], v["temp"], v["ua"], v["uf"],
                          L, *out, s)
        mb.mb_kv_compact(dev, int(bti[-1]), hkv, hd, n, v["qo"], dkv, dbti, dbt, out[0], out[1], L, new, s)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    s2 = torch.cuda.Stream()
    s2.wait_stream(torch.cuda.current_stream())
    for case in (e, d):
        for k, a in (("logits", to_dev(case.logits)), ("tokens", _i32(case.tokens)), ("parent", _i32(case.parent)),
                     ("temp", torch.from_numpy(case.temp).cuda()), ("ua", torch.from_numpy(case.u_accept).cuda()),
                     ("uf", torch.from_numpy(case.u_final).cuda())):
            v[k].copy_(a)
        for x, p in zip(dev, pools):
            x.copy_(to_dev(p))
        torch.cuda.synchronize()
        g.replay()
        with torch.cuda.stream(s2):
            beside = other.run(mb)
        torch.cuda.synchronize()
        mb.mb_device_status(None, _stream())
        got = [x.cpu().numpy() for x in out]
        case.check(got, L)
        other.check(beside)
        paths = [list(got[1][r, :got[0][r]]) for r in range(n)]
        for x, p in zip(dev, pools):
            want = p.copy()
            lens = OS.compact(want, case.qo, kv, bti, bt, paths)
            assert np.array_equal(from_dev(x), want)
        assert np.array_equal(new.cpu().numpy(), lens)


# --------------------------------------------------------- page operations
@pytest.mark.parametrize("hkv,hd,layers", [(2, 64, 1), (8, 128, 3), (1, 128, 130), (3, 40, 2)])
def test_compact_moves_the_path_and_nothing_else(mb, hkv, hd, layers):
    rng = np.random.default_rng(hkv + layers)
    reqs = [(33, 8), (0, 20), (15, 1), (40, 0), (100, 64), (7, 128), (16, 16)]
    need = [(c + n + 15) // 16 for c, n in reqs]
    P = sum(need) + 2
    perm = rng.permutation(P).astype(np.int32)
    qo = np.concatenate([[0], np.cumsum([n for _, n in reqs])]).astype(np.int32)
    kv = np.array([c + n for c, n in reqs], np.int32)
    bti = np.concatenate([[0], np.cumsum(need)]).astype(np.int32)
    paths = [[0, 2, 3, 7], [0], [0], [], [0, 1, 2, 10, 11, 40, 41, 42, 43, 63], list(range(0, 128, 9)), list(range(16))]
    path = np.full((len(reqs), 16), -1, np.int32)
    for r, x in enumerate(paths):
        path[r, :len(x)] = x
    pools = rng.integers(0, 1 << 16, size=(layers, P, 2, hkv, 16, hd)).astype(np.uint16)
    dev = [to_dev(p) for p in pools]
    new = torch.full((len(reqs),), -7, dtype=torch.int32, device="cuda")
    mb.mb_kv_compact(dev, P, hkv, hd, len(reqs), _i32(qo), _i32(kv), _i32(bti), _i32(perm), _i32([len(x) for x in paths]),
                     _i32(path), 16, new, _stream())
    mb.mb_device_status(None, _stream())
    for i in range(layers):
        want = pools[i].copy()
        lens = OS.compact(want, qo, kv, bti, perm, paths)
        assert np.array_equal(from_dev(dev[i]), want)
    assert np.array_equal(new.cpu().numpy(), lens)


def test_compact_refuses_bad_paths_on_the_device(mb):
    hkv, hd, reqs = 2, 64, [(20, 6)] * 5
    rng = np.random.default_rng(4)
    qo, kv = np.arange(0, 31, 6).astype(np.int32), np.full(5, 26, np.int32)
    bti, perm = np.arange(0, 11, 2).astype(np.int32), rng.permutation(10).astype(np.int32)
    pool = rng.integers(0, 1 << 16, size=(10, 2, hkv, 16, hd)).astype(np.uint16)
    path = np.array([[0, 2, 1], [0, 6, -1], [0, 3, 5], [0, 0, 1], [1, 2, 3]], np.int32)
    count = np.array([3, 2, 3, 3, 9], np.int32)
    d, new = to_dev(pool), torch.full((5,), -7, dtype=torch.int32, device="cuda")
    mb.mb_kv_compact([d], 10, hkv, hd, 5, _i32(qo), _i32(kv), _i32(bti), _i32(perm), _i32(count), _i32(path), 3, new,
                     _stream())
    with pytest.raises(mb.MbError) as e:
        mb.mb_device_status(None, _stream())
    assert e.value.status == mb.MB_EDEVICE
    want = pool.copy()
    OS.compact(want, qo, kv, bti, perm, [[], [], [0, 3, 5], [], []])
    assert np.array_equal(from_dev(d), want)
    assert list(new.cpu().numpy()) == [-7, -7, 23, -7, -7]


@pytest.mark.parametrize("hkv,hd,layers,pages,pairs", [(8, 128, 3, 40, 1), (2, 64, 1, 64, 20), (1, 8, 131, 9, 4),
                                                       (1, 64, 2, 5000, 2300)])
def test_copy_pages(mb, hkv, hd, layers, pages, pairs):
    rng = np.random.default_rng(pages)
    perm = rng.permutation(pages)
    dst, src = perm[:pairs], rng.choice(perm[pairs:], size=pairs)   # sources may repeat
    pools = rng.integers(0, 1 << 16, size=(layers, pages, 2, hkv, 16, hd)).astype(np.uint16)
    dev = [to_dev(p) for p in pools]
    mb.mb_kv_copy_pages(dev, pages, hkv, hd, src, dst, _stream())
    mb.mb_device_status(None, _stream())
    pools[:, dst] = pools[:, src]
    for i in range(layers):
        assert np.array_equal(from_dev(dev[i]), pools[i])


def test_pages_beyond_32_bit_offsets(mb):
    """The same pages at the far end of a pool of more than 2^32 bytes (and of
    2^32 elements): the same attention, the same moves, the same copies."""
    t = Trees([(300, 9), (5, 20), (1200, 3)], 8, 4, 128, 51).run(mb)
    small = from_dev(t.o)
    t.check(small)
    far = 140000                                  # pages of 64 KB: 9.2 GB
    big = torch.empty((far + t.P, 2, 8, 16, 128), dtype=torch.bfloat16, device="cuda")
    assert big.numel() > 2 ** 32
    big[far:].copy_(t.dpool)
    o = to_dev(np.full((t.T, 8 * 4 * 128), SENT, np.uint16))
    d = t.dev
    bt = _i32(t.bt + far)
    mb.mb_tree_attention(t.dq, big, o, far + t.P, 32, 8, 128, 3, t.T, d["qo"], d["kv"], d["bti"], bt, d["parent"], t.work,
                         _stream())
    mb.mb_device_status(None, _stream())
    assert np.array_equal(from_dev(o), small)
    n, path = np.array([3, 4, 2], np.int32), np.array([[0, 4, 8, -1], [0, 1, 7, 19], [0, 2, -1, -1]], np.int32)
    new = torch.zeros(3, dtype=torch.int32, device="cuda")
    mb.mb_kv_compact([big], far + t.P, 8, 128, 3, d["qo"], d["kv"], d["bti"], bt, _i32(n), _i32(path), 4, new, _stream())
    want = t.pool.copy()
    lens = OS.compact(want, t.qo, t.kv, t.bti, t.bt, [list(path[r, :n[r]]) for r in range(3)])
    assert np.array_equal(from_dev(big[far:]), want) and np.array_equal(new.cpu().numpy(), lens)
    mb.mb_kv_copy_pages([big], far + t.P, 8, 128, [far + 1, far + 2], [far + 4, 3], _stream())
    mb.mb_device_status(None, _stream())
    want[4] = want[1]
    assert np.array_equal(from_dev(big[far:]), want) and np.array_equal(from_dev(big[3]), want[2])


def test_tree_attention_on_another_stream_than_its_tensors(mb):
    """A call on a side stream behind the tensors' own, and a batch of the most
    nodes in every request at once with one that has none."""
    t = Trees([(700, 128), (0, 0), (129, 128), (15, 128)], 1, 8, 64, 52, kind="star")
    s = torch.cuda.Stream()
    t.run(mb)
    first = from_dev(t.o)
    t.check(first)
    t.o.view(torch.int16).fill_(SENT)
    s.wait_stream(torch.cuda.current_stream())
    t.call(mb, stream=s.cuda_stream)
    torch.cuda.current_stream().wait_stream(s)
    assert np.array_equal(from_dev(t.o), first)
    mb.mb_device_status(None, s.cuda_stream)
