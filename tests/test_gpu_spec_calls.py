"""Calls of the drafted-token operators at the edge of what they are given."""

import numpy as np
import pytest
import torch

from oracle import spec as OS
from mixed_prefill_decode_gb300 import workload as W
from gpu_util import f64, from_dev, to_dev
from test_gpu_verify_sums import Stars

pytestmark = pytest.mark.gpu


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _with_drafts(n, vocab, children, seed):
    """Requests whose children are drawn from draft probabilities near the target's."""
    s = Stars(n, vocab, children, seed)
    lg = s.settle()
    s.probs = np.empty((n, vocab), np.float32)
    for r in range(n):
        q = s.weights(r, lg) * np.exp(0.7 * s.rng.standard_normal(vocab))
        s.probs[r] = q / q.sum()
        q = s.probs[r].astype(np.float64)
        s.tokens[r, 1:] = s.rng.choice(vocab, size=children, p=q / q.sum())
    s.u = s.rng.random(s.u.shape, dtype=np.float32)
    return s


def _expect(s, max_path=4):
    """The oracle's answers; a case at a border is not one to ask about."""
    lg, out = f64(s.bits), []
    for r in range(s.n):
        rows = np.zeros((s.m, s.V))
        rows[0] = lg[r]
        q = None
        if s.probs is not None:
            q = np.zeros((s.m, s.V))
            q[0] = s.probs[r]
        path, nxt, (test, last) = OS.verify(rows, s.tokens[r], q, [-1] + [0] * (s.m - 1), float(s.temp[r]),
                                            s.u[r].astype(np.float64), float(s.u_final[r]), max_path)
        assert test > 1e-6 and last > 1e-7
        out.append((len(path), path + [-1] * (max_path - len(path)), nxt))
    return out


def _same(got, want):
    for r, (n, path, nxt) in enumerate(want):
        assert (got[0][r], list(got[1][r]), got[2][r]) == (n, path, nxt), r


@pytest.mark.parametrize("drafts", [False, True])
@pytest.mark.parametrize("token", [-1, 4096, 2 ** 31 - 1, -2 ** 31])
def test_a_child_with_no_token_of_the_vocabulary_is_passed_over(mb, drafts, token):
    """Whichever child it is, the others and the draw are as without it."""
    s = _with_drafts(48, 4096, 3, 11)
    if not drafts:
        s.probs = None
    for r in range(s.n):
        s.tokens[r, 1 + r % 3] = token
    got = s.run(mb, np.arange(s.n), check=False)
    with pytest.raises(mb.MbError) as e:
        mb.mb_device_status(None, _stream())
    assert e.value.status == mb.MB_EDEVICE
    _same(got, _expect(s))


def test_negative_draft_probabilities_count_as_zero(mb):
    """Small ones, and ones that are no probabilities at all, the children's own among them."""
    s = _with_drafts(40, 4096, 2, 12)
    s.probs[0, 0] = 0.25   # (of request 0 only: so that a sum above 1 is among them)
    at = s.rng.random(s.probs.shape) < 0.3
    for r in range(s.n):
        at[r, s.tokens[r, 1 + r % 2]] = r % 4 == 0
    clean = np.where(at, np.float32(0.0), s.probs)
    bad = np.array([-1e-6, -0.3, -1.0, -3e38, -np.inf], np.float32)[s.rng.integers(0, 5, size=s.probs.shape)]
    s.probs = clean
    want = s.run(mb, np.arange(s.n))
    _same(want, _expect(s))
    s.probs = np.where(at, bad, clean)
    for a, b in zip(s.run(mb, np.arange(s.n)), want):
        assert np.array_equal(a, b)


def test_a_temperature_that_is_none_is_greedy(mb):
    """Below 0 or not a number: as 0, and reported."""
    s = Stars(4, 4096, 2, 13)
    lg = s.settle()
    s.tokens[:, 2] = np.argmax(lg, 1)
    s.temp[:] = [-1.0, np.nan, -np.inf, 0.0]
    got = s.run(mb, np.arange(4), check=False)
    with pytest.raises(mb.MbError):
        mb.mb_device_status(None, _stream())
    assert np.all(got[0] == 2) and np.all(got[1][:, 1] == 2) and np.all(got[2] == 0)   # (the child's row is all zeros: token 0)


def _tree_layers(mb, count, seed=3):
    """Layers of one shape with their pools and a batch of trees for each."""
    shape, reqs = W.SMALL_GQA, [(700, 24), (90, 5), (1500, 60), (33, 1)]
    wl = W.Workload("spec", shape, reqs, seed)
    weights, x, batch, pool = W.materialize(wl)
    rng = np.random.default_rng(seed)
    parent = np.concatenate([[-1] + [int(rng.integers(0, i)) for i in range(1, q)] for _, q in reqs]).astype(np.int32)
    dw = {k: to_dev(v) for k, v in weights.items()}
    layers = []
    for i in range(count):
        dx = to_dev(x) * (1.0 + 0.25 * i)
        layers.append((mb.Layer(shape.as_dict(), dw, batch.num_tokens, pool.shape[0], kv_buf=to_dev(pool.reshape(-1))), dx,
                       torch.empty_like(dx)))
    return layers, mb.Batch.of(batch), parent


def test_layers_that_step_in_order_share_a_workspace(mb):
    """The first step with trees of each further layer costs no 43 MB."""
    layers, batch, parent = _tree_layers(mb, 5)
    for L, x, y in layers:
        L.step(batch, x, y, _stream())
    L, x, y = layers[0]
    L.step(batch, x, y, _stream(), parent=parent)
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    for L, x, y in layers[1:]:
        L.step(batch, x, y, _stream(), parent=parent)
        mb.mb_device_status(L.handle, _stream())
    assert free - torch.cuda.mem_get_info()[0] < mb.mb_tree_attention_workspace_bytes()
    for L, _, _ in layers:
        L.close()


def test_layers_that_step_at_once_have_workspaces_of_their_own(mb):
    """Two layers with GEMM workspaces of their own on two streams, each as alone."""
    layers, batch, parent = _tree_layers(mb, 3)
    alone = []
    for L, x, y in layers:
        L.step(batch, x, y, _stream(), parent=parent)
        mb.mb_device_status(L.handle, _stream())
        alone.append(from_dev(y))
    ws, streams = [], [torch.cuda.Stream() for _ in layers]
    for i, (L, x, y) in enumerate(layers):
        if i > 0:   # (layer 0 keeps the device's)
            ws.append(torch.zeros(mb.mb_gemm_workspace_bytes(), dtype=torch.uint8, device="cuda"))
            mb.mb_layer_set_gemm_workspace(L.handle, ws[-1])
        mb.mb_layer_set_gemm_sms(L.handle, 48)   # (3 x 48 CTAs fit the GPU together)
        L.step(batch, x, y, _stream(), parent=parent)
    torch.cuda.synchronize()
    want = [from_dev(y) for _, _, y in layers]
    for _ in range(20):
        for (L, x, y), s in zip(layers, streams):
            L.step(batch, x, y, s.cuda_stream, parent=parent)
    torch.cuda.synchronize()
    for (L, _, y), w, a in zip(layers, want, alone):
        mb.mb_device_status(L.handle, _stream())
        assert np.array_equal(from_dev(y), w)
        assert np.max(np.abs(f64(w) - f64(a))) <= 2e-2 * np.max(np.abs(f64(a)))   # (fewer CTAs: other K splits)
        L.close()
