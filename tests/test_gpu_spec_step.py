"""GPU parity of the layer step over batches with drafted trees, and the
drafted-token operators together as a speculative decoding loop.

Layer outputs are compared with the float64 oracle within the acceptance
tolerance of the other step tests (max|d| <= 2e-2 max|ref|); placement of keys
and values, and whatever must be the same computation, bit-exactly."""

import numpy as np
import pytest
import torch

from oracle import layer as OL
from oracle import spec as OS
from mixed_prefill_decode_gb300 import workload as W
from gpu_util import assert_close, f64, from_dev, to_dev

pytestmark = pytest.mark.gpu


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=np.int32))).cuda()


def _tree(rng, n):
    return [-1] + [int(rng.integers(max(0, (i - 1) // 2 - 1), i)) for i in range(1, n)]


def _setup(shape, reqs, trees, seed):
    """reqs: (cached, tokens); trees: which requests bring a tree."""
    wl = W.Workload("spec", shape, reqs, seed)
    weights, x, batch, pool = W.materialize(wl)
    rng = np.random.default_rng(seed + 50)
    parent = np.concatenate([_tree(rng, q) if r in trees else np.arange(q) - 1 for r, (_, q) in enumerate(reqs)])
    return wl, weights, x, batch, pool, parent.astype(np.int32)


MIXED = [(130, 1), (17, 9), (77, 200), (0, 12), (300, 64), (255, 2), (5, 1), (640, 30)]


@pytest.mark.parametrize("shape,seed", [(W.TINY, 1), (W.SMALL_GQA, 2), (W.SMALL_G5_QKN, 3)])
def test_step_with_trees_matches_oracle(mb, shape, seed):
    """Decodes, a prefill chunk and trees in one batch."""
    wl, weights, x, batch, pool, parent = _setup(shape, MIXED, {1, 3, 4, 7}, seed)
    dpool = to_dev(pool.reshape(-1))
    L = mb.Layer(shape.as_dict(), {k: to_dev(v) for k, v in weights.items()}, batch.num_tokens, pool.shape[0], kv_buf=dpool)
    dx = to_dev(x)
    y = torch.full_like(dx, float("nan"))
    mb.mb_step_tree(L.handle, L.kv, mb.Batch.of(batch), parent, dx, y, _stream())
    mb.mb_device_status(L.handle, _stream())
    ref = OS.layer_step_tree(shape.as_dict(), OL.weights_to_f64(weights), f64(pool), batch.qo_indptr, batch.kv_len,
                             batch.bt_indptr, batch.bt, parent, f64(x))
    assert_close("y", f64(from_dev(y)), ref["y"])
    after = from_dev(dpool).reshape(pool.shape)
    changed = np.any(after != pool, axis=(1, 2, 4)).reshape(-1)
    expect = np.zeros_like(changed)
    for page, slot in ref["written"]:
        expect[page * 16 + slot] = True
    assert np.array_equal(changed, expect), "keys or values outside this step's places"
    L.close()


def test_step_with_chains_is_the_plain_step(mb):
    """Chains take the ordinary path: bit for bit mb_step, also with parent None."""
    shape = W.SMALL_GQA
    wl, weights, x, batch, pool, parent = _setup(shape, MIXED, set(), 4)
    out = []
    for par in (None, parent):
        dpool = to_dev(pool.reshape(-1))
        L = mb.Layer(shape.as_dict(), {k: to_dev(v) for k, v in weights.items()}, batch.num_tokens, pool.shape[0], kv_buf=dpool)
        dx = to_dev(x)
        y = torch.empty_like(dx)
        L.step(mb.Batch.of(batch), dx, y, _stream(), parent=par)
        mb.mb_device_status(L.handle, _stream())
        out.append((from_dev(y), from_dev(dpool)))
        L.close()
    assert np.array_equal(out[0][0], out[1][0]) and np.array_equal(out[0][1], out[1][1])


def test_step_tree_refuses_bad_parents(mb):
    shape = W.SMALL_GQA
    wl, weights, x, batch, pool, parent = _setup(shape, [(5, 3), (4, 130)], {0}, 5)
    L = mb.Layer(shape.as_dict(), {k: to_dev(v) for k, v in weights.items()}, batch.num_tokens, pool.shape[0],
                 kv_buf=to_dev(pool.reshape(-1)))
    dx = to_dev(x)
    y = torch.empty_like(dx)
    for at, value, status in ((1, 1, "MB_EINVAL"), (2, -2, "MB_EINVAL"), (3 + 100, 50, "MB_EUNSUPPORTED")):
        bad = parent.copy()
        bad[at] = value
        with pytest.raises(mb.MbError) as e:
            mb.mb_step_tree(L.handle, L.kv, mb.Batch.of(batch), bad, dx, y, _stream())
        assert e.value.status == getattr(mb, status)
    with pytest.raises(ValueError):
        mb.mb_step_tree(L.handle, L.kv, mb.Batch.of(batch), parent[:-1], dx, y, _stream())
    L.close()


def test_stack_graphs_follow_new_trees(mb):
    """One captured graph serves batches of one geometry: other trees, other
    tables, and a step without trees in between."""
    shape = W.SMALL_GQA
    reqs = [(200, 1), (60, 20), (33, 40), (500, 7)]
    wl, weights, x, batch, pool, parent = _setup(shape, reqs, {1, 2, 3}, 6)
    rng = np.random.default_rng(60)
    per = [W.make_weights(shape, 70 + i) for i in range(2)]
    res = []
    steps = [np.concatenate([_tree(rng, q) if r else [-1] for r, (_, q) in enumerate(reqs)]) for _ in range(3)]
    for graphs in (True, False):
        pools = [to_dev(pool.reshape(-1)) for _ in range(2)]
        layers = [mb.Layer(shape.as_dict(), {k: to_dev(v) for k, v in per[i].items()}, batch.num_tokens, pool.shape[0],
                           kv_buf=pools[i]) for i in range(2)]
        S = mb.mb_stack_create([l.handle for l in layers], graphs)
        dx, out = to_dev(x), []
        y = torch.empty_like(dx)
        for par in (steps[0], steps[1], None, steps[2], steps[0]):
            mb.mb_stack_step_tree(S, [l.kv for l in layers], mb.Batch.of(batch), par, dx, y, _stream())
            mb.mb_device_status(layers[0].handle, _stream())
            out.append(from_dev(y))
        res.append((out, [from_dev(p) for p in pools]))
        mb.mb_stack_destroy(S)
        for l in layers:
            l.close()
    for a, b in zip(res[0][0], res[1][0]):
        assert np.array_equal(a, b)
    assert all(np.array_equal(a, b) for a, b in zip(res[0][1], res[1][1]))
    assert np.array_equal(res[0][0][0], res[0][0][4]) and not np.array_equal(res[0][0][0], res[0][0][1])


def _chain_kv(shape, weights, pool, table, c, x):
    """Keys and values that the oracle's layer stores for x after c cached tokens."""
    p = pool.copy()
    n = x.shape[0]
    OL.layer_step(shape.as_dict(), OL.weights_to_f64(weights), p, [0, n], [c + n], [0, len(table)], np.asarray(table), x)
    return OL.gather_kv(p, np.asarray(table), c + n)


@pytest.mark.parametrize("mode", ["greedy", "points", "probs"])
def test_speculative_decoding_loop(mb, mode):
    """Rounds of draft, step with trees, logits, verification and compaction
    on one layer.  Each round's decision equals the oracle's on the kernel's own
    logits, the accepted tokens' keys and values end up behind the prefix
    bit-exactly, and what the cache then holds is what a plain prefill of the
    accepted tokens stores."""
    shape, vocab, nodes, max_path = W.SMALL_G5_QKN, 512, 9, 8
    reqs = [(c, nodes) for c in (40, 95, 16, 130, 7)]
    n, d = len(reqs), shape.d_model
    rng = np.random.default_rng(200)
    weights = W.make_weights(shape, 201)
    batch, P = W.make_batch([(c + 60, nodes) for c, _ in reqs], 202)   # tables with room for every round
    pool = np.full((P, 2, shape.n_kv_heads, 16, shape.head_dim), W.KV_SENTINEL, np.uint16)
    for r, (c, _) in enumerate(reqs):
        for p in range(c):
            pool[batch.bt[batch.bt_indptr[r] + p // 16], :, :, p % 16] = W.f32_to_bf16_bits(
                rng.standard_normal((2, shape.n_kv_heads, shape.head_dim), dtype=np.float32))
    table = W.f32_to_bf16_bits(rng.standard_normal((vocab, d), dtype=np.float32))
    w_lm = W.f32_to_bf16_bits(0.1 * rng.standard_normal((vocab, d), dtype=np.float32))
    g_f = W.f32_to_bf16_bits(np.ones(d, np.float32))
    dpool, dt, dlm, dg = to_dev(pool.reshape(-1)), to_dev(table), to_dev(w_lm), to_dev(g_f)
    T = n * nodes
    L = mb.Layer(shape.as_dict(), {k: to_dev(v) for k, v in weights.items()}, T, P, kv_buf=dpool)
    x = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
    y, yw = torch.empty_like(x), torch.empty_like(x)
    logits = torch.empty((T, vocab), dtype=torch.bfloat16, device="cuda")
    ids = torch.empty(T, dtype=torch.int32, device="cuda")
    rows = torch.arange(T, dtype=torch.int32, device="cuda")
    qo = np.arange(0, T + 1, nodes).astype(np.int32)
    dqo, dbti, dbt = _i32(qo), _i32(batch.bt_indptr), _i32(batch.bt)
    cached = np.array([c for c, _ in reqs])
    start = cached.copy()
    emitted = [[int(rng.integers(vocab))] for _ in reqs]   # token 0 of the next round
    done = [[] for _ in reqs]                              # tokens whose keys are in the cache behind `start`
    longest = 0
    for step in range(4):
        parent = np.concatenate([_tree(rng, nodes) for _ in reqs]).astype(np.int32)
        kv = (cached + nodes).astype(np.int32)
        b = mb.Batch(qo, kv, batch.bt_indptr, batch.bt)
        tokens = rng.integers(0, vocab, size=T).astype(np.int32)
        for r in range(n):
            tokens[qo[r]] = emitted[r][-1]

        def run_layer():
            mb.mb_embed(dt, vocab, d, _i32(tokens), T, x, _stream())
            mb.mb_step_tree(L.handle, L.kv, b, parent, x, y, _stream())
            mb.mb_sample_greedy(y, T, rows, T, d, shape.rms_eps, dg, dlm, vocab, yw, logits, ids, _stream())

        # drafts that the target likes: most nodes take the favourite of their parent's row, level by level
        for _ in range(4):
            run_layer()
            fav = ids.cpu().numpy()
            for t in range(T):
                if parent[t] >= 0 and (t * 5 + step) % 4:
                    tokens[t] = fav[(t // nodes) * nodes + parent[t]]
        probs = None
        if mode == "probs":
            q = rng.random((T, vocab)).astype(np.float32) ** 8
            for t in range(T):
                if parent[t] >= 0:
                    q[(t // nodes) * nodes + parent[t], tokens[t]] += q.sum(1).mean()
            probs = q / q.sum(1, keepdims=True)
        run_layer()
        before = from_dev(dpool).reshape(pool.shape)
        temp = None if mode == "greedy" else np.full(n, 0.7, np.float32)
        ua, uf = rng.random(T, dtype=np.float32), rng.random(n, dtype=np.float32)
        cnt, nxt, new_kv = (torch.full((n,), -7, dtype=torch.int32, device="cuda") for _ in range(3))
        path = torch.full((n, max_path), -7, dtype=torch.int32, device="cuda")
        dev = [None if a is None else torch.from_numpy(a).cuda() for a in (probs, temp, ua, uf)]
        mb.mb_verify_tree(logits, vocab, _i32(tokens), dev[0], n, T, dqo, _i32(parent), dev[1], dev[2], dev[3], max_path, cnt,
                          path, nxt, _stream())
        mb.mb_kv_compact([dpool], P, shape.n_kv_heads, shape.head_dim, n, dqo, _i32(kv), dbti, dbt, cnt, path, max_path,
                         new_kv, _stream())
        mb.mb_device_status(L.handle, _stream())
        mb.mb_device_status(None, _stream())
        lg, cnt, path, nxt = f64(from_dev(logits)), cnt.cpu().numpy(), path.cpu().numpy(), nxt.cpu().numpy()
        after = from_dev(dpool).reshape(pool.shape)
        want = before.copy()
        paths = []
        for r in range(n):
            a, e = qo[r], qo[r + 1]
            p, tok, _ = OS.verify(lg[a:e], tokens[a:e], None if probs is None else probs[a:e].astype(np.float64),
                                  parent[a:e], 0.0 if temp is None else float(temp[r]), ua[a:e].astype(np.float64),
                                  float(uf[r]), max_path)
            assert list(path[r, :cnt[r]]) == p and nxt[r] == tok and np.all(path[r, cnt[r]:] == -1)
            paths.append(p)
            longest = max(longest, len(p))
        lens = OS.compact(want, qo, kv, batch.bt_indptr, batch.bt, paths)
        assert np.array_equal(after, want)
        assert np.array_equal(new_kv.cpu().numpy(), lens) and np.array_equal(lens, cached + cnt)
        for r in range(n):
            done[r] += [int(tokens[qo[r] + i]) for i in paths[r]]
            emitted[r].append(int(nxt[r]))
        cached = lens.astype(np.int64)
    assert longest > 2, "no draft was accepted beyond the root's child: the loop tests nothing"
    final = f64(from_dev(dpool)).reshape(pool.shape)
    for r in range(n):
        tab = batch.bt[batch.bt_indptr[r]:batch.bt_indptr[r + 1]]
        K, V = OL.gather_kv(final, tab, int(cached[r]))
        Kr, Vr = _chain_kv(shape, weights, f64(pool), tab, int(start[r]), f64(table)[done[r]])
        assert_close(f"keys of request {r}", K[start[r]:], Kr[start[r]:])
        assert_close(f"values of request {r}", V[start[r]:], Vr[start[r]:])
    L.close()
