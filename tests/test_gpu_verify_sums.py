"""How exact the verification's decisions are, against float64.

A weight 2^((l - m) k) is off by at most 2^-29 of itself and is rounded to a
multiple of 2^-41 of the reference's, so by 2^-42 of that more; a sum S over a
row (reference 1) of V tokens by 2^-29 S + V 2^-42.  A child of probability p'
in what is left of a row (S = the tokens left) passes for u < p', so with u and
p' apart by more than
  2^-28 + V 2^-42 / S     relative to p'
(2^-29 of the child's weight, the sum's error) the decision is the exact one,
and it is the same whatever the batch, hence the number of CTAs, the row is
summed in.  Without draft probabilities the reference is the largest weight or
the largest left, whichever gives S >= 1; a border of the draw, a partial sum
over S, is off by at most 2 (2^-29 + V 2^-42).  The logits here are 0 or at least 2^-16 of a row's largest, so that
l - m is exact."""

import numpy as np
import pytest
import torch

from mixed_prefill_decode_gb300 import workload as W
from gpu_util import f64, to_dev

pytestmark = pytest.mark.gpu


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=np.int32))).cuda()


def _f32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=np.float32))).cuda()


class Stars:
    """Requests of a root and its children, 1 + k nodes; only the roots' logits are random."""

    def __init__(self, n, vocab, children, seed):
        self.rng = rng = np.random.default_rng(seed)
        self.n, self.V, self.m = n, vocab, 1 + children
        self.temp = (0.6 + 0.6 * rng.random(n)).astype(np.float32)
        self.root = 2.0 * rng.standard_normal((n, vocab))
        self.tokens = np.zeros((n, self.m), np.int32)
        for r in range(n):
            self.tokens[r, 1:] = rng.choice(vocab, size=children, replace=False)
        self.u = np.full((n, self.m), 1.0 - 2.0 ** -24, np.float32)
        self.u_final = rng.random(n, dtype=np.float32)
        self.probs = None

    def settle(self):
        """Round the logits; their float64 values."""
        top = np.abs(self.root).max(1, keepdims=True)
        self.bits = W.f32_to_bf16_bits(np.where(np.abs(self.root) < top * 2.0 ** -12, 0.0, self.root).astype(np.float32))
        return f64(self.bits)

    def weights(self, r, logits):
        z = logits[r] / np.float64(self.temp[r])
        return np.exp(z - z.max())

    def run(self, mb, rows, max_path=4, check=True):
        """The requests `rows` as a batch of their own: (n_accepted, path, next token)."""
        k, m, V = len(rows), self.m, self.V
        lg = np.zeros((k, m, V), np.uint16)
        lg[:, 0] = self.bits[rows]
        q = None
        if self.probs is not None:
            q = torch.zeros((k, m, V), dtype=torch.float32, device="cuda")
            q[:, 0] = _f32(self.probs[rows])
        parent = np.tile(np.array([-1] + [0] * (m - 1)), k)
        out = [torch.full(s, -7, dtype=torch.int32, device="cuda") for s in ((k,), (k, max_path), (k,))]
        s = torch.cuda.current_stream().cuda_stream
        mb.mb_verify_tree(to_dev(lg.reshape(k * m, V)), V, _i32(self.tokens[rows].reshape(-1)), q, k, k * m,
                          _i32(np.arange(k + 1) * m), _i32(parent), _f32(self.temp[rows]), _f32(self.u[rows].reshape(-1)),
                          _f32(self.u_final[rows]), max_path, *out, s)
        if check:
            mb.mb_device_status(None, s)
        return [x.cpu().numpy() for x in out]


def _after_refusal(lefts, per, vocab, seed):
    """Two children: the first holds 1 - left of the row and is refused, the second about half of what is left."""
    s = Stars(len(lefts) * per, vocab, 2, seed)
    for r in range(s.n):
        left, T = lefts[r // per], np.float64(s.temp[r])
        h, x = s.tokens[r, 1:]
        s.root[r, [h, x]] = -np.inf
        rest = T * np.log(np.sum(np.exp(s.root[r] / T)))
        s.root[r, x] = rest + T * np.log(0.5 + s.rng.random())
        rest = T * np.log(np.sum(np.exp(s.root[r] / T)))
        s.root[r, h] = rest + T * np.log((1 - left) / left)
    return s


def _check_second_child(mb, s, tolerance):
    """u of the second child on either side of its border, at three times the tolerance."""
    lg, sides = s.settle(), []
    for r in range(s.n):
        w = s.weights(r, lg)
        h, x = s.tokens[r, 1:]
        left = 1.0 - w[h] / w.sum() if w[h] < 0.5 * w.sum() else (w.sum() - w[h]) / w.sum()
        p = w[x] / (np.sum(np.delete(w, h)))
        tol = max(tolerance(left), 2.0 ** -23)   # (u is a float: half a step is 2^-25 of it)
        s.u[r, 2] = np.float32(p * (1 + (3 if r % 2 else -3) * tol))
        assert left > 2.0 ** -22 and abs(s.u[r, 2] / p - 1) > 2 * tol
        sides.append(s.u[r, 2] < p)
    count, path, _ = s.run(mb, np.arange(s.n))
    assert np.array_equal(count, 1 + np.array(sides)) and np.array_equal(path[:, 1], np.where(sides, 2, -1))


@pytest.mark.parametrize("vocab", [1000, 4096, 32000, 128256])
def test_a_child_behind_a_likely_one_that_was_refused(mb, vocab):
    _check_second_child(mb, _after_refusal([0.3, 1e-1, 1e-2, 1e-3, 1e-4], 12, vocab, vocab),
                        lambda left: 2.0 ** -28 + vocab * 2.0 ** -42 / left)


@pytest.mark.parametrize("mode", ["points", "probs"])
def test_a_decision_does_not_depend_on_the_batch(mb, mode):
    """u on the border of the first child's test, or of the second's, to half a
    step of the float: the same answer alone (16 CTAs a row), in 70 (8) and in 200 (4)."""
    n, V = 200, 65536
    s = Stars(n, V, 2, 31 + len(mode))
    for r in range(n):
        T = np.float64(s.temp[r])
        rest = T * np.log(np.sum(np.exp(s.root[r] / T)))
        s.root[r, s.tokens[r, 1:]] = rest + T * np.log(0.2 + 2.0 * s.rng.random(2))
    lg = s.settle()
    if mode == "probs":
        s.probs = np.empty((n, V), np.float32)
    sure = {}
    for r in range(n):
        w = s.weights(r, lg)
        p = w / w.sum()
        a, b = s.tokens[r, 1:]
        if mode == "probs":
            q = p * np.exp(0.5 * s.rng.standard_normal(V))
            s.probs[r] = q / q.sum()
            for x in (a, b):   # the draft likes its children more than the target does: the test can fail
                s.probs[r, x] = p[x] * (1.2 + s.rng.random())
            q = s.probs[r].astype(np.float64)
            left = np.maximum(0.0, p - q)
            border = p[a] / q[a] if r % 2 else None
        else:
            left = p.copy()
            left[a] = 0.0
            border = p[a] if r % 2 else left[b] / left.sum()
        if border is not None:
            u = np.float32(border)
            s.u[r, 1 if r % 2 else 2] = u
            if r % 2 and abs(u / border - 1) > 2.0 ** -28 + V * 2.0 ** -42:
                sure[r] = u < border
    full = s.run(mb, np.arange(n))
    for r, passes in sure.items():
        assert (full[1][r, 1] == 1) == passes, r
    assert len(sure) > 20
    some = s.run(mb, np.arange(70))
    alone = [s.run(mb, np.array([r])) for r in range(24)]
    for a, b in zip(full, some):
        assert np.array_equal(a[:70], b)
    for k in range(3):
        assert np.array_equal(full[k][:24], np.concatenate([x[k] for x in alone]))


@pytest.mark.parametrize("vocab", [1000, 4096, 128256])   # (1, 2 and 8 CTAs a row)
def test_a_child_behind_one_that_took_nearly_everything(mb, vocab):
    """What is left is measured by itself, however little it is."""
    _check_second_child(mb, _after_refusal([1e-3, 1e-5, 1e-6, 4e-7], 12, vocab, 9 + vocab), lambda left: 2.0 ** -28 + vocab * 2.0 ** -42)


@pytest.mark.parametrize("children", [1, 3])
@pytest.mark.parametrize("vocab", [1000, 4096, 128256])
def test_the_draw_behind_a_refused_child_that_took_nearly_everything(mb, vocab, children):
    """u_final a tenth of a token's width inside it, from either side.  Three
    children: the others hold 0.9 of what the first left and are refused too."""
    lefts, per = [0.6, 1e-2, 1e-4, 1e-5, 1e-6, 4e-7], 10
    s = Stars(len(lefts) * per, vocab, children, 77 + vocab + children)
    s.u[:, 2:] = 1.0 - 2.0 ** -24
    for r in range(s.n):
        T, kids, scale = np.float64(s.temp[r]), s.tokens[r, 1:], 1.0
        s.root[r, kids] = -np.inf
        for k, out in zip(kids[::-1], ([0.3, 0.9] if children > 1 else []) + [1 - lefts[r // per]]):
            rest = T * np.log(np.sum(np.exp(s.root[r] / T)))
            s.root[r, k] = rest + T * np.log(out / (1 - out))
    lg, want = s.settle(), []
    tol = 2.0 ** -28 + vocab * 2.0 ** -41
    for r in range(s.n):
        w = s.weights(r, lg)
        w[s.tokens[r, 1:]] = 0.0
        cum = np.concatenate([[0.0], np.cumsum(w / w.sum())])
        width = np.diff(cum)
        t = s.rng.choice(np.nonzero(width > max(60 * tol, 2.0 ** -20))[0])   # (u is a float, to 2^-25)
        s.u_final[r] = np.float32(cum[t] + (0.1 if r % 2 else 0.9) * width[t])
        assert cum[t] + 3 * tol < s.u_final[r] < cum[t + 1] - 3 * tol
        want.append(t)
    count, path, nxt = s.run(mb, np.arange(s.n))
    assert np.all(count == 1) and np.array_equal(nxt, want)


def test_nothing_or_one_token_is_left(mb):
    """A second child that is all that is left is certain, whatever u; u = 1 (not
    below 1, as it should be) refuses it too, and the draw is from p itself."""
    s = Stars(40, 64, 2, 5)
    s.root[:] = -np.inf
    for r in range(s.n):
        s.root[r, s.tokens[r, 1:]] = [3.0, 1.0]
    s.bits = W.f32_to_bf16_bits(s.root.astype(np.float32))
    count, path, nxt = s.run(mb, np.arange(s.n))
    assert np.all(count == 2) and np.all(path[:, 1] == 2)
    s.u[:] = 1.0
    count, path, nxt = s.run(mb, np.arange(s.n))
    lg = f64(s.bits)
    for r in range(s.n):
        w = s.weights(r, lg)
        assert abs(s.u_final[r] - w[:s.tokens[r, 1:].max()].sum() / w.sum()) > 1e-6
        assert count[r] == 1 and nxt[r] == np.argmax(np.cumsum(w / w.sum()) > s.u_final[r])
