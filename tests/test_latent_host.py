"""Host-side refusals of the latent-cache calls and of the descriptors built on
the GPU (no GPU): each comes back before any device work."""

import numpy as np
import pytest

from oracle import latent as OL

G = 1 << 30   # arguments this far apart do not overlap


def _args(names, over):
    return {**{n: (i + 1) * G for i, n in enumerate(names)}, **over}


def _refused(mb, call, status, text=()):
    with pytest.raises(mb.MbError) as e:
        call()
    assert e.value.status == getattr(mb, status) and all(t in str(e.value) for t in text)


TAB = ["slots", "cached", "new_tokens", "tables", "owned", "ring", "state", "qo_indptr", "kv_len", "bt_indptr", "bt",
       "tok_req", "tok_pos", "tok_slot"]
TAB_BYTES = dict(slots=12, cached=12, new_tokens=12, tables=4 * 8 * 6, owned=32, ring=80, state=16, qo_indptr=16, kv_len=12,
                 bt_indptr=16, bt=36, tok_req=28, tok_pos=28, tok_slot=28)


def _tables(mb, **over):
    mb.mb_batch_tables(**{**_args(TAB, {}), "num_reqs": 3, "T": 7, "bt_cap": 9, "max_slots": 8, "max_pages": 6,
                          "num_pages": 20, **over})


@pytest.mark.parametrize("over,status", [
    *[({n: None}, "MB_EINVAL") for n in TAB], (dict(num_reqs=-1), "MB_EINVAL"), (dict(T=-1), "MB_EINVAL"),
    (dict(bt_cap=-1), "MB_EINVAL"), (dict(max_slots=0), "MB_EINVAL"), (dict(max_pages=0), "MB_EINVAL"),
    (dict(num_pages=0), "MB_EINVAL"), (dict(num_reqs=8193), "MB_EUNSUPPORTED"),
    (dict(max_slots=65537), "MB_EUNSUPPORTED"), (dict(max_pages=(1 << 20) + 1), "MB_EUNSUPPORTED"),
    (dict(num_pages=1 << 27), "MB_EUNSUPPORTED"), (dict(T=1 << 30), "MB_EUNSUPPORTED"),
    (dict(bt_cap=1 << 30), "MB_EUNSUPPORTED")])
def test_batch_tables_refuses(mb, over, status):
    _refused(mb, lambda: _tables(mb, **over), status)


OUTS = ("tables", "owned", "state", "qo_indptr", "kv_len", "bt_indptr", "bt", "tok_req", "tok_pos", "tok_slot")


@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("other", TAB)
def test_batch_tables_refuses_an_output_over_anything_else(mb, out, other):
    if out == other:
        return
    at = _args(TAB, {})[other]
    for x in (at + TAB_BYTES[other] - 4, at - TAB_BYTES[out] + 4):
        _refused(mb, lambda: _tables(mb, **{out: x}), "MB_EINVAL", ("overlap", out, other))


def _release(mb, **over):
    mb.mb_tables_release(**{**_args(["slots", "tables", "owned", "ring", "state"], {}), "n": 3, "max_slots": 8,
                            "max_pages": 6, "num_pages": 20, **over})


@pytest.mark.parametrize("over,status", [
    *[({n: None}, "MB_EINVAL") for n in ("slots", "tables", "owned", "ring", "state")], (dict(n=-1), "MB_EINVAL"),
    (dict(max_slots=0), "MB_EINVAL"), (dict(n=8193), "MB_EUNSUPPORTED"), (dict(owned=G + 8), "MB_EINVAL"),
    (dict(ring=2 * G + 188), "MB_EINVAL"), (dict(state=4 * G + 76), "MB_EINVAL")])
def test_tables_release_refuses(mb, over, status):
    _refused(mb, lambda: _release(mb, **over), status)


def test_empty_calls_do_nothing(mb):
    _release(mb, n=0)
    _append(mb, T=0)
    for form in FORMS:
        _attention(mb, form, T=0)
        _attention(mb, form, num_reqs=0)


def test_arrays_of_no_elements_may_have_no_address(mb):
    _append(mb, T=0, **{n: None for n in ("ckv", "q", "q_rope", "tok_pos", "tok_slot")})
    for form in FORMS:
        _attention(mb, form, T=0, **{n: None for n in ("q", "q_rope", "o", "bt")})
        _attention(mb, form, T=0, num_reqs=0, **{n: None for n in ("q", "q_rope", "o", "bt", "kv_len")})
        _refused(mb, lambda: _attention(mb, form, T=0, kv_len=None), "MB_EINVAL")


APP = ["ckv", "q", "gain", "pool", "q_rope", "tok_pos", "tok_slot"]
APP_BYTES = dict(ckv=2 * (2 * 832 + 576), q=3 * 8 * 192 * 2, gain=1024, pool=4 * 16 * 576 * 2, q_rope=3 * 8 * 64 * 2,
                 tok_pos=12, tok_slot=12)


def _append(mb, **over):
    mb.mb_latent_append(**{**_args(APP, {}), "ld": 832, "T": 3, "num_pages": 4, "n_heads": 8, "head_dim": 128, "rank": 512,
                           "rms_eps": 1e-6, "rope_theta": 1e4, **over})


@pytest.mark.parametrize("over,status", [
    *[({n: None}, "MB_EINVAL") for n in APP], *[({n: G + 8}, "MB_EINVAL") for n in APP[:5]], (dict(T=-1), "MB_EINVAL"),
    (dict(ld=575), "MB_EINVAL"), (dict(ld=568), "MB_EINVAL"), (dict(ld=580), "MB_EINVAL"), (dict(num_pages=0), "MB_EINVAL"),
    (dict(n_heads=0), "MB_EINVAL"), (dict(rms_eps=-1.0), "MB_EINVAL"), (dict(rms_eps=float("nan")), "MB_EINVAL"),
    (dict(rope_theta=0.0), "MB_EINVAL"), (dict(rope_theta=float("inf")), "MB_EINVAL"), (dict(rank=384), "MB_EUNSUPPORTED"),
    (dict(head_dim=96), "MB_EUNSUPPORTED"), (dict(n_heads=129), "MB_EUNSUPPORTED"),
    (dict(num_pages=1 << 27), "MB_EUNSUPPORTED"), (dict(T=(1 << 20) + 1), "MB_EUNSUPPORTED")])
def test_append_refuses(mb, over, status):
    _refused(mb, lambda: _append(mb, **over), status)


@pytest.mark.parametrize("out", ["pool", "q_rope"])
@pytest.mark.parametrize("other", APP)
def test_append_refuses_an_output_over_anything_else(mb, out, other):
    if out == other:
        return
    at = _args(APP, {})[other]
    for x in ((at + APP_BYTES[other] - 1) & ~15, (at - APP_BYTES[out] + 16) & ~15):
        _refused(mb, lambda: _append(mb, **{out: x}), "MB_EINVAL", ("overlap", out, other))


ATT = ["q", "q_rope", "w_kv", "pool", "o", "qo_indptr", "kv_len", "bt_indptr", "bt", "workspace"]
ATT_BYTES = dict(q=7 * 8 * 192 * 2, q_rope=7 * 8 * 64 * 2, w_kv=8 * 256 * 512 * 2, pool=4 * 16 * 576 * 2, o=7 * 8 * 128 * 2,
                 qo_indptr=16, kv_len=12, bt_indptr=16, bt=4)


def _attention(mb, form="absorbed", **over):
    a = {**_args(ATT, {}), "num_pages": 4, "n_heads": 8, "head_dim": 128, "rank": 512, "scale": 0.07, "num_reqs": 3, "T": 7,
         **over}
    if form == "absorbed":
        mb.mb_latent_attention(**a)
    else:
        mb.mb_latent_prefill(**{"kv_tokens": 100, **a})


FORMS = ["absorbed", "expanded"]
BAD = [*[({n: None}, "MB_EINVAL") for n in ATT], *[({n: G + 8}, "MB_EINVAL") for n in ("q", "q_rope", "w_kv", "o")],
       (dict(pool=4 * G + 64), "MB_EINVAL"), (dict(workspace=20 * G + 128), "MB_EINVAL"), (dict(T=-1), "MB_EINVAL"),
       (dict(num_reqs=-1), "MB_EINVAL"), (dict(num_pages=0), "MB_EINVAL"), (dict(n_heads=0), "MB_EINVAL"),
       (dict(scale=0.0), "MB_EINVAL"), (dict(scale=float("nan")), "MB_EINVAL"), (dict(scale=float("inf")), "MB_EINVAL"),
       (dict(rank=128), "MB_EUNSUPPORTED"), (dict(head_dim=192), "MB_EUNSUPPORTED"),
       (dict(n_heads=129), "MB_EUNSUPPORTED"), (dict(num_pages=1 << 27), "MB_EUNSUPPORTED"),
       (dict(T=(1 << 20) + 1), "MB_EUNSUPPORTED")]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("over,status", BAD)
def test_attention_refuses(mb, form, over, status):
    _refused(mb, lambda: _attention(mb, form, **over), status)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("other", [n for n in ATT if n not in ("o", "workspace")])
def test_attention_refuses_an_output_over_an_input(mb, form, other):
    at = _args(ATT, {})[other]
    for x in ((at + ATT_BYTES[other] - 1) & ~15, at - ATT_BYTES["o"] + 16):
        _refused(mb, lambda: _attention(mb, form, o=x), "MB_EINVAL", ("overlap", "o ", other))
    _refused(mb, lambda: _attention(mb, form, workspace=at), "MB_EINVAL", ("overlap", "workspace", other))


@pytest.mark.parametrize("over,status", [(dict(kv_tokens=-1), "MB_EINVAL"), (dict(kv_tokens=(1 << 27) + 1), "MB_EUNSUPPORTED"),
                                         (dict(num_reqs=(1 << 20) + 1), "MB_EUNSUPPORTED")])
def test_expanded_refuses(mb, over, status):
    _refused(mb, lambda: _attention(mb, "expanded", **over), status)


# ------------------------------------------------------- the oracle's pins
def test_oracle_attention_is_the_absorbed_form_too():
    rng = np.random.default_rng(1)
    n, H, hd, rank, kv = 3, 2, 8, 16, 11
    q, qr, w = rng.standard_normal((n, H, hd)), rng.standard_normal((n, H, 64)), rng.standard_normal((H, 2 * hd, rank))
    rows = rng.standard_normal((kv, rank + 64))
    o, p, _ = OL.attention_request(q, qr, w, rows, 0.1)
    for h in range(H):
        full = np.concatenate([q[:, h] @ w[h, :hd], qr[:, h]], axis=1)
        z = 0.1 * full @ rows.T
        z[np.arange(kv)[None, :] > kv - n + np.arange(n)[:, None]] = -np.inf
        e = np.exp(z)
        y = (e / e.sum(axis=1, keepdims=True)) @ rows[:, :rank]
        assert np.allclose(o[:, h], y @ w[h, hd:].T, atol=1e-12)
    assert np.allclose(p.sum(axis=2), 1.0) and np.all(p[:, 0, -2:] == 0) and np.all(p[:, 1, -1] == 0)


def test_oracle_rope_turns_pairs_and_keeps_relative_positions():
    rng = np.random.default_rng(2)
    a, b = rng.standard_normal(64), rng.standard_normal(64)
    assert np.allclose(OL.rope64(a, 0, 1e4), a)
    assert np.allclose(OL.rope64(a, 7, 1e4) @ OL.rope64(b, 12, 1e4), OL.rope64(a, 107, 1e4) @ OL.rope64(b, 112, 1e4))
    one = np.zeros(64)
    one[0] = 1.0
    assert np.allclose(OL.rope64(one, 2, 1e4)[[0, 32]], [np.cos(2.0), np.sin(2.0)])


def test_oracle_tables_hand_trace():
    tables, owned, ring = np.zeros((3, 4), np.int64), np.zeros(3, np.int64), np.array([9, 8, 7, 6, 5])
    out, head, count, bad = OL.batch_tables([2, 0], [0, 0], [17, 3], 24, 9, tables, owned, ring, 3, 4, 10 // 2)
    qo, kv, bti, bt, req, pos, slot = out
    assert qo.tolist() == [0, 17, 20] and kv.tolist() == [17, 3] and bti.tolist() == [0, 2, 3]
    assert bt.tolist() == [6, 5, 9] and (head, count) == (1, 1) and bad   # pages of 5 and more are out of range
    assert req.tolist() == [0] * 17 + [1] * 3 + [-1] * 4 and pos.tolist()[:17] == list(range(17))
    assert slot.tolist() == [-1] * 24
    assert owned.tolist() == [1, 0, 2]
    count, bad = OL.tables_release([2], tables, owned, ring, head, count, 5)
    assert count == 3 and not bad and ring.tolist() == [9, 8, 6, 5, 5] and owned.tolist() == [1, 0, 0]


# ---------------------------------------------------------- workspace sizes
def _never_falls(size, axes, fixed):
    """`size` over every axis, the others at each of `fixed`'s values."""
    for at in fixed:
        for axis, values in axes.items():
            sizes = [size(**{**at, axis: v}) for v in values]
            assert sizes == sorted(sizes), (at, axis, values[int(np.argmin(np.diff(sizes)))])


def test_expanded_workspace_never_falls_as_a_batch_grows(mb):
    """A workspace of the largest call does for every smaller one, across the
    sizes where the heads begin to be taken in groups (512 MB of keys and values:
    8,192 keys of 128 heads of 128)."""
    axes = dict(kv_tokens=[0, 1, 127, 128, 4000, 8000, 8063, 8064, 8191, 8192, 8320, 13000, 16384, 26000, 26112, 32768, 52000,
                           1 << 20, (1 << 20) + 128, 1 << 21, 1 << 22, 1 << 24, 1 << 27],
                num_reqs=[0, 1, 2, 8, 33, 64, 65, 128, 129, 1000, 4096, 8192, 1 << 14, 1 << 17, 1 << 20],
                n_heads=list(range(1, 129)), head_dim=[64, 128], rank=[256, 512])
    fixed = [dict(kv_tokens=kv, num_reqs=n, n_heads=H, head_dim=hd, rank=512)
             for kv in (1, 8000, 8320, 26000, 1 << 20, 1 << 27) for n in (1, 8, 64, 1 << 20) for H in (1, 40, 128) for hd in (64, 128)]
    _never_falls(mb.mb_latent_prefill_workspace_bytes, axes, fixed)


@pytest.mark.parametrize("kv,n,H,hd", [(26000, 1, 40, 128), (26112, 1, 40, 128), (8320, 1, 128, 128), (26000, 1, 100, 64),
                                       (1 << 21, 1, 3, 64), (1 << 27, 1, 128, 128), (0, 1, 1, 64)])
def test_expanded_workspace_holds_what_a_group_takes(mb, kv, n, H, hd):
    """The groups' keys and values (4 bytes a number of a head's keys), evenly
    spread, and the rotated keys, by blocks of 128 keys."""
    blocks = kv // 128 + n
    most = max(1, min(H, (512 << 20) // (blocks * 128 * 4 * hd)))
    group = -(-H // -(-H // most))
    part = 2 * 160 * 256 * (hd + 2) * 4 + 8192 + 20480
    assert mb.mb_latent_prefill_workspace_bytes(kv, n, H, hd, 256) >= blocks * 128 * (4 * hd * group + 128) + part


def test_absorbed_workspace_never_falls_as_a_batch_grows(mb):
    axes = dict(T=[0, 1, 2, 63, 64, 65, 1000, 1 << 20], n_heads=list(range(1, 129)), rank=[256, 512])
    _never_falls(mb.mb_latent_attention_workspace_bytes, axes,
                 [dict(T=T, n_heads=H, rank=r) for T in (0, 7, 1 << 20) for H in (1, 40, 128) for r in (256, 512)])


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("n", [(1 << 20) + 1, 2 ** 31 - 1])
def test_attention_refuses_more_requests_than_it_counts(mb, form, n):
    _refused(mb, lambda: _attention(mb, form, num_reqs=n, T=0, **{k: (i + 1) << 40 for i, k in enumerate(ATT)}),
             "MB_EUNSUPPORTED", ("num_reqs",))
