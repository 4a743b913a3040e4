"""The softmax of latent attention where its reference has to move: logits that
rise from block to block, inside one, in steps, at the last key, and pieces
of a cut request whose maxima lie far apart.  The absorbed form rescales when a
row rises more than 8 (in powers of two) above its reference, the expanded one
when half a block's probabilities sum to more than 2^14.

So that nothing else limits the comparison, the logits are exact: q_nope is 0 and
each row of q_rope has one number, a power of two, so a logit is one product of
two bf16 numbers.  Column i of the rotated keys holds profile i, which the heads
i, i + 16, ... attend by.  And so that every key counts, however low its logit:
those heads' W_uv reads 16 columns of the vectors only, and there the vector of
a key whose logit lies d below the profile's highest is 2^min(d, 60) times as
long.  A key's share in o is then about the same for all keys, and a block that
is scaled once too often, too little or not at all is off by as much as it
counts.

Bound: with exact logits the exponents are off by the rounding of scale log2(e)
(3 2^-24 of a difference of at most 60 that counts: 2^-16) and of
the differences (2^-18), a power by 2^-22, and each of at most 80 moves of the
reference by 2^-22 + 2^-24 * 60: together below 2^-11 of a probability.  What is
left are roundings to bf16, off by at most U = 2^-8: the probabilities (up to U
and alike where the logits are, so their root mean square is at most U), the
vectors' sum or the values, and o (at most U / sqrt(3) each, of independent
numbers).  The error's root mean square relative to that of o is then at most
sqrt(1 + 1/3 + 1/3) U + 2^-11 = 1.42 U; asserted with 2 U, head by head."""

import numpy as np
import pytest

from oracle import latent as OL
from mixed_prefill_decode_gb300 import workload as W
from gpu_util import f64
from test_gpu_latent import SENT, U, Batch

pytestmark = pytest.mark.gpu
NP, CLIP = 16, 60


def profiles(kv):
    """[16][kv]: logits in powers of two."""
    j = np.arange(kv)
    rise = lambda at, by: np.where(j >= at, float(by), 0.0)   # noqa: E731
    x = [np.zeros(kv),
         9.0 * (j // 64),                                # above the absorbed form's limit at every block
         7.5 * (j // 64),                                # below it each time
         15.0 * (j // 128),                              # above the expanded form's at every block
         0.3 * j,                                        # inside a block
         -0.5 * j,
         rise(kv - 1, 40),                               # the last key alone
         np.where(j % 128 == 100, 20.0, 0.0),            # single keys, in the second half of a block
         np.where(j % 128 == 20, 20.0, 0.0),             # and in the first
         rise(128 + 64, 8.5),                            # sums of halves near 2^14
         rise(192, 200) - rise(320, 150),                # up and down again
         rise(64, 300),                                  # a reference that is of no use
         -rise(64, 300),                                 # blocks that count nothing
         rise(300, 31) + rise(301, 31) + rise(500, 31),
         np.where(j % 3 == 0, 12.0, 0.0) * (j // 64 % 2),
         0.02 * j]
    return np.stack(x)


class Rising(Batch):
    def __init__(self, reqs, H, hd, rank, seed, tail=2):
        super().__init__(reqs, H, hd, rank, seed, tail=tail)
        rng, q = self.rng, 4.0
        unit = self.scale * np.log2(np.e) * q            # a key's number x is the logit unit * x
        self.q[:, :, :hd] = 0
        self.q_rope[:] = 0
        self.w = np.zeros_like(self.w)
        bits = W.f32_to_bf16_bits(np.full(1, q, np.float32))[0]
        wide = rank // NP
        for h in range(H):
            i = h % NP
            self.q_rope[:, h, i] = bits
            self.w[h, :, wide * i:wide * (i + 1)] = W.f32_to_bf16_bits(rng.standard_normal((2 * hd, wide), dtype=np.float32))
        for r, (c, n) in enumerate(reqs):
            kv = c + n
            level = profiles(kv)
            row = np.zeros((kv, rank + 64), np.float32)
            # (a tenth of a power of two at random, so that probabilities differ)
            keys = W.f32_to_bf16_bits(((level + 0.1 * rng.standard_normal(level.shape)) / unit).astype(np.float32).T)
            up = np.exp2(np.minimum(level.max(axis=1, keepdims=True) - level, CLIP)).astype(np.float32)
            vec = rng.standard_normal((kv, NP, wide), dtype=np.float32) * up.T[:, :, None]
            row[:, :rank] = vec.reshape(kv, rank)
            out = W.f32_to_bf16_bits(row)
            out[:, rank:rank + NP] = keys
            for p in range(0, kv, 16):
                m = min(16, kv - p)
                self.pool[self.bt[self.bti[r] + p // 16], :m] = out[p:p + m]

    def compare(self, got, heads=None):
        for r, (c, n) in enumerate(self.reqs):
            a = int(self.qo[r])
            rows = self.rows(r)
            for h in range(self.H) if heads is None else heads:
                o, _, _ = OL.attention_request(f64(self.q[a:a + n])[:, h:h + 1, :self.hd], f64(self.q_rope[a:a + n])[:, h:h + 1],
                                               f64(self.w)[h:h + 1], rows, self.scale)
                err = np.sqrt(np.sum((got[a:a + n, h] - o[:, 0]) ** 2) / np.sum(o ** 2))
                assert err <= 2 * U, (r, h % NP, float(err / U))
        assert np.all(np.isnan(got[int(self.qo[-1]):])), "a row outside the requests was written"


def test_the_profiles_move_the_references():
    """(What the cases are for: of the sixteen, how many rise as the two forms'
    limits ask.)"""
    x = profiles(800)
    blocks = x[:, :768].reshape(NP, 12, 64).max(axis=2)
    assert np.sum(np.any(np.diff(np.maximum.accumulate(blocks, axis=1), axis=1) > 8.2, axis=1)) >= 8
    first = x[:, :128].max(axis=1)
    sums = np.exp2(np.minimum(x - first[:, None], 100))[:, :768].reshape(NP, 12, 64).sum(axis=2)
    assert np.sum(np.any(sums[:, 2::2] > 2 ** 14.5, axis=1)) >= 6 and np.sum(np.any(sums[:, 3::2] > 2 ** 14.5, axis=1)) >= 6


@pytest.mark.parametrize("reqs,H,hd,rank", [
    ([(800, 1), (321, 1), (65, 1)], 16, 64, 256),            # several requests a CTA or several CTAs a request
    ([(798, 3), (190, 7), (100, 70)], 16, 64, 256),          # four tokens a unit
    ([(799, 1)], 64, 128, 512), ([(511, 1), (512, 2)], 80, 128, 512),
    ([(4999, 1)], 16, 128, 512),                             # a piece a block
    ([(700, 1)] * 40, 32, 64, 512),                          # cut units, a warp a row in the merge
    ([(500, 1)] * 300, 16, 64, 256)])                        # whole units
def test_absorbed(mb, reqs, H, hd, rank):
    b = Rising(reqs, H, hd, rank, seed=H + len(reqs))
    if len(reqs) < 20:
        b.compare(b.run(mb, "absorbed"))
        return
    got = b.run(mb, "absorbed")
    keep = list(range(0, len(reqs), len(reqs) // 8))
    part = [(int(b.qo[r]), b.reqs[r]) for r in keep]
    for (a, (c, n)), r in zip(part, keep):
        rows = b.rows(r)
        for h in range(NP):
            o, _, _ = OL.attention_request(f64(b.q[a:a + n])[:, h:h + 1, :hd], f64(b.q_rope[a:a + n])[:, h:h + 1],
                                           f64(b.w)[h:h + 1], rows, b.scale)
            assert np.sqrt(np.sum((got[a:a + n, h] - o[:, 0]) ** 2) / np.sum(o ** 2)) <= 2 * U, (r, h)


@pytest.mark.parametrize("reqs,H,hd,rank", [
    ([(798, 3)], 16, 64, 256), ([(798, 3), (120, 100)], 16, 128, 512),    # one query tile: two groups take turns at its blocks
    ([(0, 128), (500, 128)], 16, 64, 512),
    ([(0, 600), (77, 257)], 16, 64, 256), ([(300, 256)], 16, 128, 256),   # two query tiles, and tails
    ([(4000, 150)], 16, 64, 256), ([(2500, 40)], 16, 128, 512)])          # cut over many CTAs
def test_expanded(mb, reqs, H, hd, rank):
    b = Rising(reqs, H, hd, rank, seed=H + len(reqs))
    b.compare(b.run(mb, "expanded"))


def test_the_forms_agree_on_stale_slots(mb):
    """(The rising cache keeps the base class's stale slots.)"""
    b = Rising([(70, 2)], 16, 64, 256, seed=1)
    assert np.any(b.pool == SENT)
    b.compare(b.run(mb, "absorbed"))
    b.compare(b.run(mb, "expanded"))
