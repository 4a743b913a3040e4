"""GPU parity of the latent cache's operators against the float64 oracle.

Append.  A bf16 output is off by its rounding, 2^-8 of the value (half a
step), and by the fp32 arithmetic before it: the sum of rank squares and the
reciprocal root, at most (rank + 4) 2^-24 relative; for a rotated number
a cos - b sin, 2^-22 (|a| + |b|) from products and sines and 2^-19 (|a| + |b|) from
the angle (good to 2^-20 rad up to 2^24: the reduction's constants leave 2^-47 a
turn, of 2^21.4 turns, the products 2^-48 of the angle, and the two steps round
numbers below 8 by 2^-22 each).

Attention.  Let p be the exact probabilities, y = sum_j p_j c_j, o = W_uv y,
S the largest standard deviation of a row's logits, and let every rounding to
bf16 be off by at most u = 2^-8 of the value.

Every element: with E = u scale max_j sum_r |q'_r| |c_jr| (q' = W_uk^T q; the
fp32 sums add less than 2^-10 of that) a logit is off by at most E, a probability
by a factor within e^(2 E), and
  |do| <= W_abs (sum_j p_j |c_j| (e^(2 E) (1 + u) - 1) + u e^(2 E) (1 + u) |y|_max part) + u |o|
bounded here by  (e^(2E) (1 + u)^2 - 1) |W_uv| sum_j p_j |c_j| + u |o|, with 1 % for
products of small terms.  In the expanded form the keys and values are rounded
instead: E = u scale max_j sum_d |q_d| |K_jd|, and the values' error is within
the same (1 + u)^2 of |W_uv| sum_j p_j |c_j|.

All elements: those worst cases add up what in truth is independent.  With
independent roundings of root mean square at most u / sqrt(3) each, the error's
root mean square relative to o's is at most u / sqrt(3) times the root of S^2 (the
logits' error is that share of a logit, a probability's that of the error) + 1
(probabilities) + 1 (y, or the values) + 1 (o).  The inputs are independent
random numbers, so it is asserted with twice that."""

import numpy as np
import pytest
import torch

from oracle import latent as OL
from mixed_prefill_decode_gb300 import workload as W
from gpu_util import f64, from_dev, to_dev

pytestmark = pytest.mark.gpu
SENT = 0x7FC1   # a NaN: what stale slots and unwritten rows hold
U = 2.0 ** -8


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=np.int32))).cuda()


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _bf16(rng, *shape, scale=1.0):
    return W.f32_to_bf16_bits(rng.standard_normal(shape, dtype=np.float32) * np.float32(scale))


def _status(mb, err):
    if err:
        with pytest.raises(mb.MbError) as e:
            mb.mb_device_status(None, _stream())
        assert e.value.status == mb.MB_EDEVICE
    else:
        mb.mb_device_status(None, _stream())


# ----------------------------------------------------------------- append
@pytest.mark.parametrize("T,H,hd,rank,ld,far", [
    (1, 1, 64, 256, 320, 5), (3, 5, 64, 512, 584, 70), (17, 40, 128, 512, 832, 100000), (33, 128, 128, 256, 320, 40000),
    (700, 32, 128, 512, 576, 33000), (9, 2, 64, 256, 320, 1 << 24)])
def test_append(mb, T, H, hd, rank, ld, far):
    rng = np.random.default_rng(T)
    P, eps, theta = T // 16 + 4, 1e-6, 10000.0
    ckv, q, gain = _bf16(rng, T + 1, ld, scale=3.0), _bf16(rng, T, H, hd + 64), _bf16(rng, rank)
    pool = np.full((P * 16, rank + 64), SENT, np.uint16)
    pos, slot = rng.integers(0, far + 1, size=T), rng.permutation(P * 16)[:T]
    pos[0] = far
    skipped = [t for t in range(T) if T > 3 and t % 7 == 2]
    slot[skipped] = -1
    dp, dq = to_dev(pool), torch.full((T, H, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    mb.mb_latent_append(to_dev(ckv), ld, to_dev(q), to_dev(gain), dp, dq, _i32(pos), _i32(slot), T, P, H, hd, rank, eps,
                        theta, _stream())
    _status(mb, False)
    got_pool, got_q = f64(from_dev(dp)).reshape(P * 16, rank + 64), f64(from_dev(dq)).reshape(T, H, 64)
    untouched = np.ones(P * 16, bool)
    untouched[slot[slot >= 0]] = False
    assert np.all(from_dev(dp).reshape(P * 16, -1)[untouched] == SENT)
    for t in range(T):
        if slot[t] < 0:
            assert np.all(np.isnan(got_q[t]))
            continue
        row, x = f64(ckv[t]), f64(q[t])[:, hd:]
        want = OL.append_row(row, f64(gain), pos[t], eps, theta)
        tol = np.abs(want) * (U + (rank + 4) * 2.0 ** -24) * 1.01
        pair = np.abs(row[rank:rank + 32]) + np.abs(row[rank + 32:rank + 64])
        tol[rank:] += np.tile(pair, 2) * 2.0 ** -18
        assert np.all(np.abs(got_pool[slot[t]] - want) <= tol + 1e-30)
        want = OL.rope64(x, pos[t], theta)
        tol = np.abs(want) * U * 1.01 + np.tile(np.abs(x[:, :32]) + np.abs(x[:, 32:]), 2) * 2.0 ** -18
        assert np.all(np.abs(got_q[t] - want) <= tol)


@pytest.mark.parametrize("slot,pos", [(64, 0), (-2, 0), (2**31 - 1, 0), (3, -1), (3, 2**24 + 1)])
def test_append_passes_bad_places_over(mb, slot, pos):
    rng = np.random.default_rng(1)
    pool = to_dev(np.full((4 * 16, 320), SENT, np.uint16))
    q_rope = torch.full((2, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    mb.mb_latent_append(to_dev(_bf16(rng, 2, 320)), 320, to_dev(_bf16(rng, 2, 2, 128)), to_dev(_bf16(rng, 256)), pool,
                        q_rope, _i32([pos, 9]), _i32([slot, 5]), 2, 4, 2, 64, 256, 1e-6, 1e4, _stream())
    _status(mb, True)
    bits = from_dev(pool).reshape(64, 320)
    assert np.all(bits[5] != SENT) and np.all(np.delete(bits, 5, axis=0) == SENT)
    assert np.all(from_dev(q_rope)[0] == from_dev(q_rope)[0, 0, 0]) and not torch.any(q_rope[1] == 7.0).item()


# -------------------------------------------------------------- attention
class Batch:
    """(cached, new) per request over a latent cache; stale slots hold NaN."""

    def __init__(self, reqs, H, hd, rank, seed, lead=0, tail=2):
        rng = np.random.default_rng(seed)
        self.reqs, self.H, self.hd, self.rank, self.rng = reqs, H, hd, rank, rng
        need = [(c + n + 15) // 16 for c, n in reqs]
        self.P = sum(need) + 3
        perm = rng.permutation(self.P)
        self.qo = (lead + np.concatenate([[0], np.cumsum([n for _, n in reqs])])).astype(np.int32)
        self.kv = np.array([c + n for c, n in reqs], np.int32)
        self.bti = np.concatenate([[0], np.cumsum(need)]).astype(np.int32)
        self.bt = perm[:sum(need)].astype(np.int32) if sum(need) else np.zeros(1, np.int32)
        self.T, self.scale = int(self.qo[-1]) + tail, float((hd + 64) ** -0.5)
        self.q, self.q_rope = _bf16(rng, self.T, H, hd + 64), _bf16(rng, self.T, H, 64)
        self.w = _bf16(rng, H, 2 * hd, rank, scale=rank ** -0.5)
        self.pool = np.full((self.P, 16, rank + 64), SENT, np.uint16)
        for r, (c, n) in enumerate(reqs):
            for p in range(0, c + n, 16):
                m = min(16, c + n - p)
                self.pool[self.bt[self.bti[r] + p // 16], :m] = _bf16(rng, m, rank + 64)

    def dev(self):
        return dict(q=to_dev(self.q), q_rope=to_dev(self.q_rope), w=to_dev(self.w), pool=to_dev(self.pool),
                    qo=_i32(self.qo), kv=_i32(self.kv), bti=_i32(self.bti), bt=_i32(self.bt))

    def call(self, mb, form, d, o, work, stream=None, n=None, at=0, P=None):
        """`form` on requests at .. at + n of the batch."""
        n = len(self.reqs) - at if n is None else n
        args = [d["q"], d["q_rope"], d["w"], d["pool"], o, self.P if P is None else P, self.H, self.hd, self.rank,
                self.scale, n, self.T, d["qo"][at:], d["kv"][at:], d["bti"][at:], d["bt"]]
        if form == "expanded":
            args.append(self.room())
        (mb.mb_latent_attention if form == "absorbed" else mb.mb_latent_prefill)(
            *args, work, _stream() if stream is None else stream)

    def room(self):
        return max(1, int(self.kv.sum()))

    def work(self, mb, form):
        size = (mb.mb_latent_attention_workspace_bytes(self.T, self.H, self.rank) if form == "absorbed" else
                mb.mb_latent_prefill_workspace_bytes(self.room(), len(self.reqs), self.H, self.hd, self.rank))
        return torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")   # all NaN, whatever the type

    def out(self):
        return torch.full((self.T, self.H * self.hd), float("nan"), dtype=torch.bfloat16, device="cuda")

    def run(self, mb, form, err=False, d=None):
        o = self.out()
        self.call(mb, form, self.dev() if d is None else d, o, self.work(mb, form))
        _status(mb, err)
        return f64(from_dev(o)).reshape(self.T, self.H, self.hd)

    def rows(self, r):
        k = int(self.kv[r])
        pages = self.bt[self.bti[r]:self.bti[r] + (k + 15) // 16]
        return f64(self.pool[pages].reshape(-1, self.rank + 64)[:k])

    def check(self, got, form, only=None):
        """Returns the largest share of the bound on all elements that was used."""
        parts, touched = [], np.zeros(self.T, bool)
        for r, (c, n) in enumerate(self.reqs):
            if n == 0 or (only is not None and r not in only):
                continue
            a = int(self.qo[r])
            touched[a:a + n] = True
            parts.append(near_exact(got[a:a + n], f64(self.q[a:a + n])[:, :, :self.hd], f64(self.q_rope[a:a + n]),
                                    f64(self.w), self.rows(r), self.scale, form))
        assert np.all(np.isnan(got[~touched])), "a row outside the requests was written"
        return all_elements(parts)


def near_exact(got, q, q_rope, w, rows, scale, form):
    """Every element of a request's rows within its bound; returns the squares
    of the errors and of the exact values, and the logits' largest deviation."""
    n, H, hd = q.shape
    rank = w.shape[2]
    o, p, z = OL.attention_request(q, q_rope, w, rows, scale)
    lat, most = np.abs(rows[:, :rank]), 0.0
    for h in range(H):
        wk, wv = w[h, :hd], w[h, hd:]
        if form == "absorbed":
            E = U * scale * np.max(np.abs(q[:, h] @ wk) @ lat.T, axis=1)
        else:
            E = U * scale * np.max(np.abs(q[:, h]) @ np.abs(rows[:, :rank] @ wk.T).T, axis=1)
        E = E * 1.01 + 2.0 ** -18
        A = (p[h] @ lat) @ np.abs(wv).T
        tol = 1.01 * ((np.exp(2 * E) * (1 + U) ** 2 - 1)[:, None] * A + U * np.abs(o[:, h]))
        d = np.abs(got[:, h] - o[:, h])
        assert np.all(d <= tol), (h, float(np.max(d / tol)))
        most = max(most, max(float(np.std(z[h, i][np.isfinite(z[h, i])])) for i in range(n)))
    return float(np.sum((got - o) ** 2)), float(np.sum(o ** 2)), most


def all_elements(parts):
    err, ref = sum(x[0] for x in parts), sum(x[1] for x in parts)
    share = np.sqrt(err / ref) / (U / np.sqrt(3.0) * np.sqrt(max(x[2] for x in parts) ** 2 + 3))
    assert share <= 2.0, share
    return share


SHAPES = [(1, 64, 256), (5, 64, 512), (8, 128, 512), (20, 128, 256), (32, 128, 512), (40, 128, 512), (64, 64, 256),
          (65, 64, 512), (100, 128, 256), (128, 128, 512)]
EDGES = [(0, 1), (14, 1), (15, 1), (16, 1), (62, 1), (63, 1), (64, 1), (127, 1), (128, 1), (300, 1)]


@pytest.mark.parametrize("H,hd,rank", SHAPES)
def test_absorbed_single_tokens_at_block_and_page_edges(mb, H, hd, rank):
    b = Batch(EDGES, H, hd, rank, seed=H, lead=3)
    b.check(b.run(mb, "absorbed"), "absorbed")


@pytest.mark.parametrize("H,hd,rank", [(1, 64, 256), (8, 64, 256), (20, 128, 512), (40, 128, 512), (72, 128, 512)])
def test_absorbed_several_tokens_and_requests_without(mb, H, hd, rank):
    reqs = [(0, 0), (100, 2), (0, 3), (7, 0), (61, 7), (1, 1), (250, 0), (90, 130 if H == 1 else 17), (0, 0)]
    b = Batch(reqs, H, hd, rank, seed=H + 1)
    b.check(b.run(mb, "absorbed"), "absorbed")


@pytest.mark.parametrize("reqs,H,hd,rank", [([(9000, 1)], 32, 128, 512), ([(20011, 3), (5, 1), (3001, 1)], 8, 64, 256),
                                            ([(4000, 1), (8191, 1)], 128, 128, 512)])
def test_absorbed_long_caches_cut_over_many_ctas(mb, reqs, H, hd, rank):
    b = Batch(reqs, H, hd, rank, seed=len(reqs))
    b.check(b.run(mb, "absorbed"), "absorbed")


@pytest.mark.parametrize("H,hd,rank", [(128, 128, 512), (97, 64, 512), (100, 128, 256), (80, 64, 256)])
def test_absorbed_many_rows(mb, H, hd, rank):
    """More rows than the merge's warps, outputs by tiles of 128 tokens, the
    first of them of no request."""
    reqs = [(int(k), 1 + int(k) % 5 // 4) for k in np.random.default_rng(8).integers(0, 200, size=40)] + [(2500, 1)]
    b = Batch(reqs, H, hd, rank, seed=H + 40, lead=130, tail=70)
    b.check(b.run(mb, "absorbed"), "absorbed")


@pytest.mark.parametrize("form,reqs,H", [("absorbed", [(300, 1)] * 40 + [(0, 130)], 128), ("absorbed", [(300, 1), (70, 2)], 8),
                                         ("expanded", [(0, 400), (300, 20), (64, 1)], 8),
                                         ("expanded", [(5000, 40)], 2)])
def test_arrays_on_16_byte_boundaries(mb, form, reqs, H):
    """Inputs and outputs that begin 16 bytes behind a boundary of 256: the same
    bits, and nothing around them."""
    b = Batch(reqs, H, 64, 256, seed=50)
    want = b.out()
    b.call(mb, form, b.dev(), want, b.work(mb, form))
    d = b.dev()
    for k in ("q", "q_rope", "w"):
        buf = torch.empty(d[k].numel() + 8, dtype=d[k].dtype, device="cuda")
        buf[8:] = d[k].reshape(-1)
        d[k] = buf[8:]
        assert d[k].data_ptr() % 32 == 16
    buf = torch.full((b.T * H * 64 + 16,), float("nan"), dtype=torch.bfloat16, device="cuda")
    b.call(mb, form, d, buf[8:-8], b.work(mb, form))
    _status(mb, False)
    assert torch.equal(buf[8:-8].view(torch.int16), want.reshape(-1).view(torch.int16))
    assert torch.all(torch.isnan(buf[:8])).item() and torch.all(torch.isnan(buf[-8:])).item()


def test_absorbed_more_requests_than_threads(mb):
    reqs = [(int(k) % 90, int(k) % 3) for k in np.random.default_rng(5).integers(0, 1000, size=700)]
    b = Batch(reqs, 4, 64, 256, seed=6)
    b.check(b.run(mb, "absorbed"), "absorbed")


@pytest.mark.parametrize("H,hd,rank", [(1, 64, 256), (3, 128, 256), (8, 64, 512), (5, 128, 512), (40, 128, 512)])
def test_expanded_chunks(mb, H, hd, rank):
    """Chunks at tile, block and page edges, behind prefixes at theirs, with
    single tokens and requests without any."""
    reqs = [(0, 1), (0, 127), (0, 129), (5, 0), (128, 128), (127, 1), (3, 300)]
    if H < 8:
        reqs += [(0, 256), (0, 257), (15, 16), (500, 513), (0, 0), (1000, 2), (255, 130)]
    b = Batch(reqs, H, hd, rank, seed=H + 20, lead=5)
    b.check(b.run(mb, "expanded"), "expanded")


@pytest.mark.parametrize("reqs,H,hd,rank", [([(9000, 40)], 3, 128, 512), ([(0, 2500)], 2, 64, 256), ([(3001, 700), (77, 5)], 2, 128, 256)])
def test_expanded_long_caches_cut_over_many_ctas(mb, reqs, H, hd, rank):
    b = Batch(reqs, H, hd, rank, seed=len(reqs) + 30)
    b.check(b.run(mb, "expanded"), "expanded")


def test_expanded_groups_of_heads(mb):
    """Keys of 26,000 tokens, 6.7 MB a head: 100 heads are two groups of 50."""
    b = Batch([(25990, 10)], 100, 64, 256, seed=33)
    got = b.run(mb, "expanded")
    heads = [0, 49, 50, 99]
    b.q, b.q_rope, b.w, b.H = b.q[:, heads], b.q_rope[:, heads], b.w[heads], len(heads)
    b.check(got[:, heads], "expanded")


def test_expanded_more_requests_than_threads(mb):
    reqs = [(int(k) % 90, int(k) % 4) for k in np.random.default_rng(6).integers(0, 1000, size=700)]
    b = Batch(reqs, 2, 64, 256, seed=7)
    b.check(b.run(mb, "expanded"), "expanded")


def test_expanded_room_too_small_leaves_the_requests_behind(mb):
    b = Batch([(100, 28), (0, 128), (300, 20), (7, 3)], 2, 64, 256, seed=34)
    b.room = lambda: 128 * 2 - 1     # with four requests: 1 + 4 blocks, and 1 + 1 + 3 + 1 are asked for
    b.check(b.run(mb, "expanded", err=True), "expanded", only=[0, 1, 2])
    b.room = lambda: 0               # four blocks: the third request does not fit any more, nor does what follows
    b.check(b.run(mb, "expanded", err=True), "expanded", only=[0, 1])


def test_the_forms_agree_on_a_mixed_batch(mb):
    """Decodes and chunks of one descriptor, each form on its part: as each
    form on the whole."""
    b = Batch([(900, 1), (64, 1), (0, 1), (200, 150), (0, 33)], 8, 128, 512, seed=35)
    d, o = b.dev(), b.out()
    b.call(mb, "absorbed", d, o, b.work(mb, "absorbed"), n=3)
    b.call(mb, "expanded", d, o, b.work(mb, "expanded"), n=2, at=3)
    _status(mb, False)
    got = f64(from_dev(o)).reshape(b.T, 8, 128)
    b.check(np.where(np.arange(b.T)[:, None, None] < 3, got, np.nan), "absorbed", only=[0, 1, 2])
    b.check(np.where(np.arange(b.T)[:, None, None] >= 3, got, np.nan), "expanded", only=[3, 4])


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
def test_rows_do_not_depend_on_what_they_do_not_see(mb, form):
    """A vector that is not finite makes the rows that see it NaN; the others'
    bits stay."""
    b = Batch([(40, 6), (70, 1), (130, 5)], 8, 64, 256, seed=8)
    clean = b.run(mb, form)
    for r, p, col, bits in ((0, 43, 5, 0x7F80), (2, 134, 300, 0x7FC0), (2, 131, 17, 0xFF80)):
        b.pool[b.bt[b.bti[r] + p // 16], p % 16, col] = bits
    got = b.run(mb, form)
    sees = np.zeros(b.T, bool)
    sees[int(b.qo[0]) + 3:int(b.qo[1])] = True      # positions 43 .. 45
    sees[int(b.qo[2]) + 1:int(b.qo[3])] = True      # positions 131 .. 134
    rows = np.zeros(b.T, bool)
    rows[:int(b.qo[-1])] = True
    assert np.all(np.isnan(got[sees])) and np.array_equal(got[rows & ~sees], clean[rows & ~sees])


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
def test_large_logits(mb, form):
    """Maxima that rise by hundreds from block to block."""
    b = Batch([(400, 3)], 8, 64, 256, seed=9)
    rows = f64(b.pool).astype(np.float32)
    for p in range(403):
        rows[b.bt[p // 16], p % 16] *= np.float32(1 + p / 20)
    stale = b.pool == SENT
    b.pool = np.where(stale, SENT, W.f32_to_bf16_bits(rows)).astype(np.uint16)
    got = b.run(mb, form)
    for h in range(8):
        o, _, _ = OL.attention_request(f64(b.q[:3])[:, h:h + 1, :64], f64(b.q_rope[:3])[:, h:h + 1], f64(b.w)[h:h + 1],
                                       b.rows(0), b.scale)
        assert np.all(np.isfinite(got[:3, h])) and np.max(np.abs(o)) > 5
    # two runs agree to the bit
    assert np.array_equal(got[:3], b.run(mb, form)[:3])


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
@pytest.mark.parametrize("what", ["kv_short", "kv_huge", "table_short", "rows_behind", "rows_back", "negative"])
def test_a_bad_request_is_left_alone(mb, form, what):
    b = Batch([(30, 2), (40, 2), (50, 1)], 8, 64, 256, seed=10, tail=0)
    d = b.dev()
    only = [0, 2]
    if what == "kv_short":
        d["kv"][1] = 1
    elif what == "kv_huge":
        d["kv"][1] = 2 ** 31 - 1
    elif what == "table_short":
        d["kv"][1] = 16 * int(b.bti[2] - b.bti[1]) + 1
    elif what == "rows_behind":
        d["qo"][3] = 2 ** 31 - 1
        only = [0, 1]
    elif what == "rows_back":
        d["qo"][2] = 1
        only = [0]
    else:
        d["qo"][0] = -5
        only = [1, 2]
    got = b.run(mb, form, err=True, d=d)
    if what == "rows_back":     # request 2 now begins inside request 0
        assert np.all(np.isnan(got[5:]))
    else:
        b.check(got, form, only=only)


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
@pytest.mark.parametrize("page", [-1, 2 ** 31 - 1, "P"])
def test_a_page_out_of_range_is_read_as_page_0(mb, form, page):
    b = Batch([(30, 2), (40, 2)], 8, 64, 256, seed=11)
    b.pool[0] = _bf16(b.rng, 16, 320)
    d = b.dev()
    b.bt[1] = 0                                   # the second page of request 0
    d["bt"][1] = b.P if page == "P" else page
    b.check(b.run(mb, form, err=True, d=d), form)


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
def test_pages_beyond_32_bit_offsets(mb, form):
    b = Batch([(200, 3), (33, 1)], 8, 128, 512, seed=12)
    P = (1 << 31) // (16 * 576) + 400
    pool = torch.empty(P, 16, 576, dtype=torch.bfloat16, device="cuda")
    high = P - 1 - np.arange(len(b.bt))
    pool[torch.from_numpy(high).cuda()] = to_dev(b.pool)[torch.from_numpy(b.bt.astype(np.int64)).cuda()]
    d = b.dev()
    d["pool"], d["bt"] = pool, _i32(high)
    o = b.out()
    b.call(mb, form, d, o, b.work(mb, form), P=P)
    _status(mb, False)
    b.check(f64(from_dev(o)).reshape(b.T, b.H, b.hd), form)


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
def test_two_calls_at_once_and_a_graph(mb, form):
    """Calls on two side streams with a workspace each; then one captured and
    replayed with another batch's contents."""
    a, b = Batch([(500, 2), (40, 1)], 20, 128, 512, seed=13), Batch([(3000, 1), (90, 4)], 20, 128, 512, seed=14)
    da, db, oa, ob = a.dev(), b.dev(), a.out(), b.out()
    wa, wb = a.work(mb, form), b.work(mb, form)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a.call(mb, form, da, oa, wa, stream=sa.cuda_stream)
        b.call(mb, form, db, ob, wb, stream=sb.cuda_stream)
    torch.cuda.synchronize()
    _status(mb, False)
    ga, gb = (f64(from_dev(o)).reshape(x.T, 20, 128) for o, x in ((oa, a), (ob, b)))
    a.check(ga, form)
    b.check(gb, form)
    # same shapes, other lengths: the graph reads what the arrays hold then
    c, e = Batch([(500, 2), (40, 1)], 20, 128, 512, seed=15), Batch([(77, 1), (465, 2)], 20, 128, 512, seed=16)
    assert c.T == e.T and c.P == e.P
    dc, oc, wc = c.dev(), c.out(), c.work(mb, form)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=sa):
        c.call(mb, form, dc, oc, wc, stream=sa.cuda_stream)
    for x in (c, e, c):
        for k, v in x.dev().items():
            dc[k].copy_(v)
        oc.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        _status(mb, False)
        x.check(f64(from_dev(oc)).reshape(x.T, 20, 128), form)


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
def test_runs_repeat_to_the_bit(mb, form):
    b = Batch([(2500, 1), (33, 2), (700, 1)], 40, 128, 512, seed=17)
    first = b.run(mb, form)
    for _ in range(20):
        assert np.array_equal(b.run(mb, form), first, equal_nan=True)


# -------------------------------------------------------------- workspace
class Guarded:
    """A workspace of `size` bytes, all NaN, with a known pattern behind it."""

    def __init__(self, size):
        self.size, self.buf = size, torch.full((size + 65536,), 0xFF, dtype=torch.uint8, device="cuda")
        self.buf[size:] = 0x5A

    def check(self):
        assert torch.all(self.buf[self.size:] == 0x5A).item(), "written behind the workspace"


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
def test_one_workspace_for_calls_of_all_sizes(mb, form):
    """The workspace of the largest batch, for it, for smaller ones, and for it again."""
    H, hd, rank = 20, 128, 512
    batches = [Batch(reqs, H, hd, rank, seed=60 + i, tail=0) for i, reqs in enumerate(
        ([(700, 40), (0, 130), (2000, 1), (64, 1)], [(0, 1)], [(0, 300)], [(60, 4), (0, 0), (127, 1)], [(3000, 5)]))]
    batches.append(batches[0])
    T, kv, n = (max(f(b) for b in batches) for f in (lambda b: b.T, lambda b: b.room(), lambda b: len(b.reqs)))
    w = Guarded(mb.mb_latent_attention_workspace_bytes(T, H, rank) if form == "absorbed" else
                mb.mb_latent_prefill_workspace_bytes(kv, n, H, hd, rank))
    for b in batches:
        o = b.out()
        b.call(mb, form, b.dev(), o, w.buf)
        _status(mb, False)
        w.check()
        b.check(f64(from_dev(o)).reshape(b.T, H, hd), form)


def test_one_expanded_workspace_on_both_sides_of_the_groups(mb):
    """128 heads of 128: their keys and values are one group up to 8,191 tokens of
    one request, two behind.  The workspace of the largest call, for all."""
    H, hd, rank, heads = 128, 128, 256, [0, 63, 64, 127]
    w = Guarded(mb.mb_latent_prefill_workspace_bytes(8400, 2, H, hd, rank))
    for reqs in ([(8390, 10)], [(8000, 5)], [(8060, 3), (100, 30)], [(70, 60)], [(8390, 10)]):
        b = Batch(reqs, H, hd, rank, seed=70 + reqs[0][1], tail=0)
        o = b.out()
        b.call(mb, "expanded", b.dev(), o, w.buf)
        _status(mb, False)
        w.check()
        got = f64(from_dev(o)).reshape(b.T, H, hd)
        b.q, b.q_rope, b.w, b.H = b.q[:, heads], b.q_rope[:, heads], b.w[heads], len(heads)
        b.check(got[:, heads], "expanded")


# ------------------------------------------- values that are not finite, pieces
@pytest.mark.parametrize("form", ["absorbed", "expanded"])
@pytest.mark.parametrize("n,H,hd,rank", [(1, 8, 64, 256), (3, 128, 64, 512)])
def test_a_vector_that_is_not_finite_in_a_piece_without_weight(mb, form, n, H, hd, rank):
    """The last key is a block, and in so short a batch a piece, of its own.  An
    infinite number in its vector gives about half of the heads a logit of minus
    infinity, so the piece's weight is 0, but a vector that is not finite makes
    its rows NaN whatever its weight."""
    b = Batch([(192, 1)] * n, H, hd, rank, seed=80 + n)
    clean = b.run(mb, form)
    assert np.all(np.isfinite(clean[:n]))
    for r in range(n):
        b.pool[b.bt[b.bti[r] + 12], 0, 7] = 0x7F80
    towards = np.einsum("thd,hd->th", f64(b.q[:n])[:, :, :hd], f64(b.w)[:, :hd, 7])
    assert np.any(towards < 0) and np.any(towards > 0)
    got = b.run(mb, form)
    assert np.all(np.isnan(got[:n]))


def test_a_vector_that_is_not_finite_far_below_the_others(mb):
    """The same with a logit so low that the piece's weight is 0 in fp32 beside the
    rest: its key alone is far down, its vector's product with q' is 0 times infinity
    or of either sign."""
    b = Batch([(192, 1)], 8, 64, 256, seed=90)
    b.q_rope[:, :, 1:] = 0
    b.q_rope[:, :, 0] = 0x4080                                # 4
    b.pool[b.bt[12], 0, 256] = 0xC47A                         # -1,000: 500 powers of two below
    want = b.run(mb, "absorbed")
    b.check(want, "absorbed")
    b.pool[b.bt[12], 0, 7] = 0x7F80
    assert np.all(np.isnan(b.run(mb, "absorbed")[:1]))


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
def test_few_requests_with_tokens_among_many_without(mb, form):
    reqs = [(0, 0)] * 20000
    for r, x in ((0, (70, 1)), (255, (0, 2)), (256, (300, 1)), (9999, (100, 3)), (19999, (130, 2))):
        reqs[r] = x
    b = Batch(reqs, 2, 64, 256, seed=95)
    b.check(b.run(mb, form), form)
