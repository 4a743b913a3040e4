"""Host-side checks of the drafted-token entry points (no GPU): every refusal
comes back before any device work, and the oracle of the verification keeps
the target's distribution."""

import numpy as np
import pytest

from oracle import spec as OS

A = 1 << 12   # a non-null, aligned address; no call below gets as far as using it


def _tree(mb, **over):
    a = dict(q=A, pool=A, o=2 * A, num_pages=8, n_q_heads=8, n_kv_heads=2, head_dim=128, num_reqs=1, T=4, qo_indptr=A,
             kv_len=A, bt_indptr=A, bt=A, parent=A, workspace=A)
    a.update(over)
    mb.mb_tree_attention(**a)


@pytest.mark.parametrize("over,status", [
    (dict(q=None), "MB_EINVAL"), (dict(pool=None), "MB_EINVAL"), (dict(o=None), "MB_EINVAL"),
    (dict(workspace=None), "MB_EINVAL"), (dict(parent=None), "MB_EINVAL"), (dict(kv_len=None), "MB_EINVAL"),
    (dict(q=A, o=A), "MB_EINVAL"), (dict(q=A + 8), "MB_EINVAL"), (dict(o=A + 4), "MB_EINVAL"),
    (dict(pool=A + 64), "MB_EINVAL"), (dict(workspace=A + 128), "MB_EINVAL"), (dict(num_pages=0), "MB_EINVAL"),
    (dict(T=-1), "MB_EINVAL"), (dict(num_reqs=-1), "MB_EINVAL"), (dict(n_q_heads=7), "MB_EINVAL"),
    (dict(n_q_heads=18), "MB_EUNSUPPORTED"), (dict(head_dim=96), "MB_EUNSUPPORTED"),
    (dict(head_dim=256), "MB_EUNSUPPORTED"), (dict(num_pages=1 << 30), "MB_EUNSUPPORTED")])
def test_tree_attention_refuses(mb, over, status):
    with pytest.raises(mb.MbError) as e:
        _tree(mb, **over)
    assert e.value.status == getattr(mb, status)


def test_empty_calls_do_nothing(mb):
    _tree(mb, num_reqs=0, T=0)
    _tree(mb, T=0)
    mb.mb_verify_tree(A, 64, A, None, 0, 0, A, A, None, None, None, 4, A, A, A)
    mb.mb_kv_compact([A], 8, 2, 64, 0, A, A, A, A, A, A, 4, 2 * A)
    mb.mb_kv_copy_pages([A], 8, 2, 64, [], [])


def _verify(mb, **over):
    a = dict(logits=A, vocab=64, tokens=A, draft_probs=None, num_reqs=1, T=4, qo_indptr=A, parent=A, temperature=A,
             u_accept=A, u_final=A, max_path=4, n_accepted=A, path=A, next_token=A)
    a.update(over)
    mb.mb_verify_tree(**a)


@pytest.mark.parametrize("over,status", [
    (dict(logits=None), "MB_EINVAL"), (dict(tokens=None), "MB_EINVAL"), (dict(path=None), "MB_EINVAL"),
    (dict(u_accept=None), "MB_EINVAL"), (dict(u_final=None), "MB_EINVAL"), (dict(max_path=0), "MB_EINVAL"),
    (dict(vocab=0), "MB_EINVAL"), (dict(T=-1), "MB_EINVAL"), (dict(logits=A + 2), "MB_EINVAL"),
    (dict(draft_probs=A + 4), "MB_EINVAL"), (dict(vocab=60), "MB_EUNSUPPORTED"),
    (dict(vocab=1 << 24), "MB_EUNSUPPORTED")])
def test_verify_refuses(mb, over, status):
    with pytest.raises(mb.MbError) as e:
        _verify(mb, **over)
    assert e.value.status == getattr(mb, status)


def _compact(mb, **over):
    a = dict(pools=[A, 2 * A], num_pages=8, n_kv_heads=2, head_dim=64, num_reqs=1, qo_indptr=A, kv_len=A, bt_indptr=A,
             bt=A, n_accepted=A, path=A, max_path=4, new_kv_len=2 * A)
    a.update(over)
    mb.mb_kv_compact(**a)


@pytest.mark.parametrize("over,status", [
    (dict(pools=[]), "MB_EINVAL"), (dict(pools=[A, None]), "MB_EINVAL"), (dict(pools=[A, A]), "MB_EINVAL"),
    (dict(pools=[A + 8]), "MB_EINVAL"), (dict(num_pages=0), "MB_EINVAL"), (dict(max_path=0), "MB_EINVAL"),
    (dict(new_kv_len=A), "MB_EINVAL"), (dict(n_accepted=None), "MB_EINVAL"), (dict(num_reqs=-1), "MB_EINVAL"),
    (dict(head_dim=60), "MB_EUNSUPPORTED")])
def test_compact_refuses(mb, over, status):
    with pytest.raises(mb.MbError) as e:
        _compact(mb, **over)
    assert e.value.status == getattr(mb, status)


@pytest.mark.parametrize("src,dst", [([0], [8]), ([8], [0]), ([-1], [1]), ([0], [-1]), ([0, 1], [2, 2]),
                                     ([0, 1], [1, 2]), ([3], [3])])
def test_copy_pages_refuses(mb, src, dst):
    with pytest.raises(mb.MbError) as e:
        mb.mb_kv_copy_pages([A], 8, 2, 64, src, dst)
    assert e.value.status == mb.MB_EINVAL


def test_copy_pages_refuses_uneven_lists(mb):
    with pytest.raises(ValueError):
        mb.mb_kv_copy_pages([A], 8, 2, 64, [1, 2], [3])


# ------------------------------------------------------- the oracle's pins
def _empirical(parent, tokens_of, probs, logits, trials, seed, V):
    """Distribution of the first emitted token over many draws."""
    rng = np.random.default_rng(seed)
    n = len(parent)
    got = np.zeros(V)
    for _ in range(trials):
        tokens = tokens_of(rng)
        path, nxt, _ = OS.verify(logits, tokens, probs, parent, 1.0, rng.random(n), rng.random(), n)
        got[tokens[path[1]] if len(path) > 1 else nxt] += 1
    return got / trials


@pytest.mark.parametrize("kind", ["probs", "points"])
def test_oracle_verification_keeps_the_targets_distribution(kind):
    """Three children of the root, drawn from the draft's distribution (probs)
    or fixed (points): the first emitted token is distributed as the target.
    20,000 draws: the standard deviation of a frequency is at most
    sqrt(1/4/20000) = 0.0035; 4.5 of them."""
    V, rng = 6, np.random.default_rng(1)
    logits = np.tile(rng.standard_normal(V), (4, 1))
    parent = [-1, 0, 0, 0]
    q = rng.random(V) + 0.05
    q /= q.sum()
    probs = np.tile(q, (4, 1)) if kind == "probs" else None
    draw = (lambda g: [0, *g.choice(V, size=3, p=q)]) if kind == "probs" else (lambda g: [0, 4, 1, 4])
    got = _empirical(parent, draw, probs, logits, 20000, 2, V)
    assert np.max(np.abs(got - OS.target_row(logits[0], 1.0))) < 4.5 * 0.0035


def test_oracle_tree_attention_of_a_chain_is_causal_attention():
    from oracle.layer import attention_request
    rng = np.random.default_rng(3)
    q, K, V = rng.standard_normal((5, 4, 8)), rng.standard_normal((12, 2, 8)), rng.standard_normal((12, 2, 8))
    o, _, _ = OS.tree_attention_request(q, K, V, np.arange(5) - 1)
    assert np.allclose(o, attention_request(q, K, V, 7), atol=1e-12)
