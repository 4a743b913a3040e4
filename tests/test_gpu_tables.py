"""mb_batch_tables and mb_tables_release against the oracle: whole numbers,
equal."""

import numpy as np
import pytest
import torch

from oracle import latent as OL

pytestmark = pytest.mark.gpu
OUT = ("qo", "kv", "bti", "bt", "req", "pos", "slot")


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=np.int32))).cuda()


def _host(t):
    return t.cpu().numpy().astype(np.int64)


def _stream():
    return torch.cuda.current_stream().cuda_stream


class Cache:
    """Rows of tables, a ring of free pages, on both sides."""

    def __init__(self, num_pages, max_slots, max_pages, seed, head=0):
        rng = np.random.default_rng(seed)
        self.P, self.S, self.M, self.rng = num_pages, max_slots, max_pages, rng
        self.ring = np.roll(rng.permutation(num_pages), head)
        self.head, self.count = head % num_pages, num_pages
        self.tables, self.owned = np.full((max_slots, max_pages), -7, np.int64), np.zeros(max_slots, np.int64)
        self.d = {k: _i32(getattr(self, k)) for k in ("ring", "tables", "owned")}
        self.d["state"] = _i32([self.head, self.count, 0, 0])

    def step(self, mb, slots, cached, new, T, cap=None, err=False, stream=None):
        n = len(slots)
        cap = 4096 if cap is None else cap
        o = {k: torch.full((size,), -99, dtype=torch.int32, device="cuda")
             for k, size in zip(OUT, (n + 1, n, n + 1, cap, T, T, T))}
        args = [_i32(x) for x in (slots, cached, new)]
        mb.mb_batch_tables(*args, n, T, cap, self.d["tables"], self.d["owned"], self.S, self.M, self.d["ring"],
                           self.d["state"], self.P, *(o[k] for k in OUT), _stream() if stream is None else stream)
        want, self.head, self.count, bad = OL.batch_tables(slots, cached, new, T, cap, self.tables, self.owned,
                                                           self.ring, self.head, self.count, self.P)
        assert bad == err
        if err:
            with pytest.raises(mb.MbError) as e:
                mb.mb_device_status(None, _stream())
            assert e.value.status == mb.MB_EDEVICE
        else:
            mb.mb_device_status(None, _stream())
        got = {k: _host(o[k]) for k in OUT}
        for k, w in zip(OUT, want):
            assert np.array_equal(got[k][:len(w)], w), k
        assert np.all(got["bt"][len(want[3]):] == -99)   # behind the last page: as it was
        self.same()
        return got

    def release(self, mb, slots, err=False):
        mb.mb_tables_release(_i32(slots), len(slots), self.d["tables"], self.d["owned"], self.S, self.M, self.d["ring"],
                             self.d["state"], self.P, _stream())
        self.count, bad = OL.tables_release(slots, self.tables, self.owned, self.ring, self.head, self.count, self.P)
        assert bad == err
        if err:
            with pytest.raises(mb.MbError):
                mb.mb_device_status(None, _stream())
        else:
            mb.mb_device_status(None, _stream())
        self.same()

    def same(self):
        assert np.array_equal(_host(self.d["state"]), [self.head, self.count, 0, 0])
        assert np.array_equal(_host(self.d["owned"]), self.owned)
        assert np.array_equal(_host(self.d["tables"]), self.tables)
        assert np.array_equal(_host(self.d["ring"]), self.ring)


@pytest.mark.parametrize("n,P,S,M,head", [(1, 8, 1, 8, 0), (3, 40, 5, 40, 39), (37, 900, 64, 64, 500),
                                          (600, 9000, 700, 40, 8999)])
def test_a_run_of_steps_with_requests_coming_and_going(mb, n, P, S, M, head):
    c = Cache(P, S, M, seed=n, head=head)
    rng = c.rng
    slots = rng.permutation(S)[:n]
    cached = np.zeros(n, np.int64)
    for step in range(9):
        room = M * 16 - cached
        new = np.minimum(rng.choice([0, 1, 1, 1, 15, 16, 17, 33, 200], size=n), room)
        got = c.step(mb, slots, cached, new, T=int(new.sum()) + int(rng.integers(0, 9)), cap=P + n)
        again = c.step(mb, slots, cached, np.diff(got["qo"]), T=int(new.sum()) + 3, cap=P + n)
        for k in ("qo", "kv", "bti"):
            assert np.array_equal(got[k], again[k])
        # some keep fewer tokens than they brought (drafts refused), some end
        cached = got["kv"] - (rng.integers(0, 2, size=n) * (np.diff(got["qo"]) > 1))
        gone = np.flatnonzero(rng.random(n) < 0.25)
        if len(gone):
            c.release(mb, slots[gone])
            cached[gone] = 0


def test_pages_run_out_in_request_order(mb):
    # needs 2, 3, 0, 1 with 4 pages: granted, not, granted (needs none), not (2 + 3 + 1 > 4)
    c = Cache(7, 4, 16, seed=1, head=5)
    c.step(mb, [0, 1, 2, 3], [0, 0, 0, 0], [0, 0, 33, 0], T=40)     # row 2 takes 3
    got = c.step(mb, [0, 1, 2, 3], [0, 0, 33, 0], [32, 48, 15, 1], T=96)
    assert np.diff(got["qo"]).tolist() == [32, 0, 15, 0]
    assert got["kv"].tolist() == [32, 0, 48, 0]


def test_empty_batch_and_no_tokens(mb):
    c = Cache(8, 4, 8, seed=2)
    got = c.step(mb, [], [], [], T=5)
    assert got["slot"].tolist() == [-1] * 5
    c.step(mb, [3, 1], [0, 0], [0, 0], T=0)


@pytest.mark.parametrize("slots,cached,new", [
    ([0, 4, 1], [0, 0, 0], [5, 5, 5]), ([0, -1, 1], [0, 0, 0], [5, 5, 5]), ([0, 2, 2], [0, 0, 0], [5, 6, 7]),
    ([0, 1, 2], [0, -1, 0], [5, 5, 5]), ([0, 1, 2], [0, 0, 0], [5, -5, 5]), ([0, 1, 2], [0, 1, 0], [5, 5, 5]),
    ([0, 1, 2], [0, 0, 0], [5, 129, 5]), ([0, 1, 2], [0, 2**31 - 1, 0], [5, 2**31 - 1, 5])])
def test_a_bad_request_counts_as_empty(mb, slots, cached, new):
    Cache(16, 4, 8, seed=3).step(mb, slots, cached, new, T=20, err=True)


@pytest.mark.parametrize("T,cap", [(9, 64), (64, 2), (0, 64), (64, 0)])
def test_arrays_too_short_leave_everything(mb, T, cap):
    Cache(16, 4, 8, seed=4).step(mb, [1, 2], [0, 0], [5, 17], T=T, cap=cap, err=True)


@pytest.mark.parametrize("head,count", [(-1, 3), (16, 3), (0, -1), (0, 17)])
def test_a_bad_ring_gives_an_empty_batch(mb, head, count):
    c = Cache(16, 4, 8, seed=5)
    c.head, c.count = head, count
    c.d["state"].copy_(_i32([head, count, 0, 0]))
    c.step(mb, [1, 2], [0, 0], [5, 17], T=32, err=True)


def test_a_page_out_of_range_gives_no_place(mb):
    c = Cache(16, 4, 8, seed=6)
    c.ring[1] = 16
    c.d["ring"].copy_(_i32(c.ring))
    got = c.step(mb, [1, 2], [0, 0], [5, 17], T=32, err=True)
    assert got["slot"][5:21].tolist() == [-1] * 16 and got["slot"][21] >= 0


def test_release_refuses_what_the_ring_cannot_hold_and_rows_given_twice(mb):
    c = Cache(16, 4, 8, seed=7)
    c.step(mb, [0, 1, 2], [0, 0, 0], [40, 20, 1], T=64)
    c.release(mb, [1, 4, 1], err=True)      # row 4 is none, row 1 comes twice
    c.release(mb, [2, -1], err=True)
    c.count = 15
    c.d["state"].copy_(_i32([c.head, 15, 0, 0]))
    c.release(mb, [0, 1], err=True)


def test_the_largest_sizes(mb):
    n, S, M = 8192, 65536, 70
    c = Cache(40000, S, M, seed=8, head=39990)
    slots = c.rng.permutation(S)[:n]
    new = c.rng.integers(0, 70, size=n)
    got = c.step(mb, slots, np.zeros(n, np.int64), new, T=int(new.sum()) + 5, cap=60000)
    c.step(mb, slots, got["kv"], np.full(n, 16), T=16 * n, cap=60000)


def test_captured_and_replayed_the_step_follows_the_lengths(mb):
    """One graph, replayed: each replay brings every request one token."""
    n, P = 5, 64
    c = Cache(P, 8, 16, seed=9, head=60)
    slots = [6, 0, 3, 7, 2]
    got = c.step(mb, slots, [0] * n, [15, 16, 17, 1, 40], T=89, cap=P)
    d = dict(slots=_i32(slots), cached=_i32(got["kv"]), new=_i32([1] * n))
    o = {k: torch.full((s,), -99, dtype=torch.int32, device="cuda") for k, s in zip(OUT, (n + 1, n, n + 1, P, 8, 8, 8))}

    def call():
        mb.mb_batch_tables(d["slots"], d["cached"], d["new"], n, 8, P, c.d["tables"], c.d["owned"], c.S, c.M,
                           c.d["ring"], c.d["state"], P, *(o[k] for k in OUT), _stream())
        d["cached"].copy_(o["kv"])

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    cached = got["kv"]
    for _ in range(20):
        graph.replay()
        want, c.head, c.count, bad = OL.batch_tables(slots, cached, [1] * n, 8, P, c.tables, c.owned, c.ring, c.head,
                                                     c.count, P)
        assert not bad
        torch.cuda.synchronize()
        for k, w in zip(OUT, want):
            assert np.array_equal(_host(o[k])[:len(w)], w), k
        cached = want[1]
        c.same()
    mb.mb_device_status(None, _stream())


@pytest.mark.parametrize("page", [16, -1, 2 ** 31 - 1])
def test_a_listed_page_out_of_range_is_recorded(mb, page):
    """A page of cached tokens only, in a row: no token's place needs it, but the
    descriptor lists it."""
    c = Cache(16, 4, 8, seed=10)
    c.step(mb, [1, 2], [0, 0], [40, 17], T=64)
    c.tables[1, 0] = page
    c.d["tables"].copy_(_i32(c.tables))
    got = c.step(mb, [1, 2], [40, 17], [1, 1], T=64, err=True)
    assert np.all(got["slot"][:2] >= 0)
    c.step(mb, [2], [18], [1], T=64)             # not among these requests' pages


def test_an_unlisted_page_out_of_range_is_not(mb):
    """A row may hold more pages than the batch lists, and the ring any number."""
    c = Cache(16, 4, 8, seed=11)
    c.step(mb, [1], [0], [60], T=64)
    c.tables[1, 3] = 99
    c.ring[(c.head + c.count - 1) % 16] = -5
    c.d["tables"].copy_(_i32(c.tables))
    c.d["ring"].copy_(_i32(c.ring))
    c.step(mb, [1], [40], [3], T=64)
