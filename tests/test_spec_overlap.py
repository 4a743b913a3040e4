"""Host-side refusals of the drafted-token calls whose arguments lie over one
another (no GPU): requests and pools run side by side, so one would read or
overwrite what another has written."""

import pytest

G = 1 << 30   # arguments this far apart do not overlap


def _args(names, **over):
    a = {n: (i + 1) * G for i, n in enumerate(names)}
    return {**a, **over}


def _refused(mb, call, text):
    with pytest.raises(mb.MbError) as e:
        call()
    assert e.value.status == mb.MB_EINVAL and "overlap" in str(e.value) and all(t in str(e.value) for t in text)


TREE = ["q", "pool", "o", "qo_indptr", "kv_len", "bt_indptr", "bt", "parent", "workspace"]
TREE_BYTES = dict(q=7 * 8 * 128 * 2, pool=8 * 2 * 2 * 16 * 128 * 2, o=7 * 8 * 128 * 2, qo_indptr=16, kv_len=12,
                  bt_indptr=16, bt=4, parent=28)


def _tree(mb, **over):
    mb.mb_tree_attention(num_pages=8, n_q_heads=8, n_kv_heads=2, head_dim=128, num_reqs=3, T=7, **_args(TREE, **over))


@pytest.mark.parametrize("name", [n for n in TREE if n not in ("o", "workspace")])
def test_tree_attention_refuses_an_output_over_an_input(mb, name):
    at = _args(TREE)[name]
    last = (at + TREE_BYTES[name] - 1) & ~15
    _refused(mb, lambda: _tree(mb, o=last), ("o ", name))
    first = at - TREE_BYTES["o"] + 16
    _refused(mb, lambda: _tree(mb, o=first), ("o ", name))
    _refused(mb, lambda: _tree(mb, workspace=at), ("workspace", name))


def test_tree_attention_refuses_its_workspace_over_the_output(mb):
    _refused(mb, lambda: _tree(mb, workspace=3 * G - (1 << 20)), ("o", "workspace"))


VERIFY_IN = dict(logits=5 * 64 * 2, tokens=20, draft_probs=5 * 64 * 4, qo_indptr=12, parent=20, temperature=8, u_accept=20,
                 u_final=8)
VERIFY_OUT = dict(n_accepted=8, path=2 * 4 * 4, next_token=8)


def _verify(mb, **over):
    a = _args([*VERIFY_IN, *VERIFY_OUT], **over)
    mb.mb_verify_tree(vocab=64, num_reqs=2, T=5, max_path=4, **a)


@pytest.mark.parametrize("out", list(VERIFY_OUT))
@pytest.mark.parametrize("other", [*VERIFY_IN, *VERIFY_OUT])
def test_verify_refuses_an_output_over_anything_else(mb, out, other):
    if out == other:
        return
    at = _args([*VERIFY_IN, *VERIFY_OUT])[other]
    size = {**VERIFY_IN, **VERIFY_OUT}[other]
    _refused(mb, lambda: _verify(mb, **{out: at + size - 4}), (out, other))
    _refused(mb, lambda: _verify(mb, **{out: at - VERIFY_OUT[out] + 4}), (out, other))


COMPACT_IN = dict(qo_indptr=16, kv_len=12, bt_indptr=16, bt=4, n_accepted=12, path=3 * 4 * 4)


@pytest.mark.parametrize("other", list(COMPACT_IN))
def test_compact_refuses_new_lengths_over_an_input(mb, other):
    a = _args(COMPACT_IN)
    for at in (a[other] + COMPACT_IN[other] - 4, a[other] - 8):
        _refused(mb, lambda: mb.mb_kv_compact([64 * G, 65 * G], 8, 2, 64, 3, a["qo_indptr"], a["kv_len"], a["bt_indptr"],
                                              a["bt"], a["n_accepted"], a["path"], 4, at), ("new_kv_len", other))


POOL = 8 * 2 * 2 * 16 * 64 * 2   # bytes of a pool of 8 pages, 2 heads of 64


@pytest.mark.parametrize("pools", [[G, G + POOL - 16], [3 * G, G, 3 * G - POOL + 16], [G, 2 * G, G + 16]])
def test_page_operations_refuse_pools_over_one_another(mb, pools):
    _refused(mb, lambda: mb.mb_kv_copy_pages(pools, 8, 2, 64, [1], [2]), ())
    a = _args(COMPACT_IN)
    _refused(mb, lambda: mb.mb_kv_compact(pools, 8, 2, 64, 3, *(16 * G + a[k] for k in COMPACT_IN), 4, 64 * G), ())


def test_page_operations_take_pools_side_by_side(mb):
    mb.mb_kv_copy_pages([G, G + POOL, G - POOL], 8, 2, 64, [], [])
