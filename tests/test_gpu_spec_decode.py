"""Speculative decoding with trees against decoding token by token.

Two stacks of the same layers, each with pools of its own, continue the same
prompts: one decodes greedily, a token a step; the other checks trees of
drafted tokens (mb_stack_step_tree, mb_verify_tree, mb_kv_compact).  Both emit
the same tokens: with more than one layer a node's keys and values depend on
what it saw, so a wrong mask, position or cache slot shows in what follows.

The two compute the same logits in different kernels.  Two tokens whose logits
are closer than both sides' tolerance, 2 x 2e-2 of the largest logit (the step
tests' tolerance), may change places; a request is followed up to there."""

import numpy as np
import pytest
import torch

from mixed_prefill_decode_gb300 import workload as W
from gpu_util import TOL, f64, from_dev, to_dev

pytestmark = pytest.mark.gpu

PROMPTS = [4, 9, 1, 17, 33, 12, 2, 26]
STEPS, NODES, VOCAB, ROOM = 20, 9, 512, 80


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=np.int32))).cuda()


class Model:
    """A stack with its pools, embeddings and head, and the requests' tables (room for every step)."""

    def __init__(self, mb, shape, n_layers, graphs, seed):
        rng = np.random.default_rng(seed)
        self.mb, self.shape, self.n = mb, shape, len(PROMPTS)
        batch, self.P = W.make_batch([(ROOM, p) for p in PROMPTS], seed)
        self.bti, self.bt = batch.bt_indptr, batch.bt
        pool = np.full((self.P, 2, shape.n_kv_heads, 16, shape.head_dim), W.KV_SENTINEL, np.uint16)
        self.pools = [to_dev(pool.reshape(-1)) for _ in range(n_layers)]
        self.rows = max(sum(PROMPTS), self.n * NODES)
        self.layers = [mb.Layer(shape.as_dict(), {k: to_dev(v) for k, v in W.make_weights(shape, seed + 1 + i).items()},
                                self.rows, self.P, kv_buf=self.pools[i]) for i in range(n_layers)]
        self.stack = mb.mb_stack_create([l.handle for l in self.layers], graphs)
        d = shape.d_model
        # (small embeddings: what the attention adds weighs as much as the token itself)
        self.table = to_dev(W.f32_to_bf16_bits(0.1 * rng.standard_normal((VOCAB, d), dtype=np.float32)))
        self.head = to_dev(W.f32_to_bf16_bits(0.1 * rng.standard_normal((VOCAB, d), dtype=np.float32)))
        self.gain = to_dev(W.f32_to_bf16_bits(np.ones(d, np.float32)))
        self.x = torch.empty((self.rows, d), dtype=torch.bfloat16, device="cuda")
        self.y, self.work = torch.empty_like(self.x), torch.empty_like(self.x)
        self.logits = torch.empty((self.rows, VOCAB), dtype=torch.bfloat16, device="cuda")
        self.ids = torch.empty(self.rows, dtype=torch.int32, device="cuda")

    def step(self, tokens, qo, kv, parent=None):
        """One pass; the logits' argmax of every row."""
        mb, T, d = self.mb, int(qo[-1]), self.shape.d_model
        mb.mb_embed(self.table, VOCAB, d, _i32(tokens), T, self.x, _stream())
        mb.mb_stack_step_tree(self.stack, [l.kv for l in self.layers], mb.Batch(qo, kv, self.bti, self.bt), parent, self.x,
                              self.y, _stream())
        rows = torch.arange(T, dtype=torch.int32, device="cuda")
        mb.mb_sample_greedy(self.y, T, rows, T, d, self.shape.rms_eps, self.gain, self.head, VOCAB, self.work, self.logits,
                            self.ids, _stream())
        mb.mb_device_status(self.layers[0].handle, _stream())
        mb.mb_device_status(None, _stream())
        return self.ids[:T].cpu().numpy()

    def prompt(self, tokens):
        qo = np.concatenate([[0], np.cumsum(PROMPTS)]).astype(np.int32)
        return self.step(tokens, qo, np.array(PROMPTS, np.int32))[qo[1:] - 1]

    def close(self):
        self.mb.mb_stack_destroy(self.stack)
        for l in self.layers:
            l.close()


def _draft(rng, last, future):
    """A tree behind `last`: a random path of it carries the coming tokens
    `future` as far as it reaches, all others a token at random."""
    parent = [-1] + [int(rng.integers(max(0, (i - 1) // 2 - 1), i)) for i in range(1, NODES)]
    tokens = rng.integers(0, VOCAB, size=NODES)
    tokens[0] = last
    node = int(rng.integers(1, NODES)) if rng.random() < 0.9 else 0
    path = []
    while node > 0:
        path.append(node)
        node = parent[node]
    for node, tok in zip(path[::-1], future):
        tokens[node] = tok
    return parent, tokens


@pytest.mark.parametrize("shape,n_layers,graphs,seed", [(W.SMALL_GQA, 3, True, 40), (W.SMALL_G5_QKN, 2, False, 50),
                                                        (W.TINY, 4, True, 60)])
def test_trees_give_the_tokens_of_plain_decoding(mb, shape, n_layers, graphs, seed):
    rng = np.random.default_rng(seed)
    prompt = rng.integers(0, VOCAB, size=sum(PROMPTS))
    n = len(PROMPTS)
    # token by token
    plain = Model(mb, shape, n_layers, False, seed)
    out, gap, kv = [plain.prompt(prompt)], [], np.array(PROMPTS, np.int32)
    for _ in range(STEPS):
        kv = kv + 1
        out.append(plain.step(out[-1], np.arange(n + 1, dtype=np.int32), kv))
        top = torch.topk(plain.logits[:n].float(), 2, dim=1).values.cpu().numpy()
        gap.append((top[:, 0] - top[:, 1]) / np.abs(f64(from_dev(plain.logits[:n]))).max(1))
    out, gap = np.array(out).T, np.array(gap).T   # token t + 1 of a request was chosen by a margin of gap[t]
    plain.close()
    # trees
    m = Model(mb, shape, n_layers, graphs, seed)
    first = m.prompt(prompt)
    live = [r for r in range(n) if first[r] == out[r, 0]]
    done, kv = [[int(t)] for t in first], np.array(PROMPTS, np.int32)
    qo = np.arange(0, n * NODES + 1, NODES).astype(np.int32)
    dqo, dbti, dbt = _i32(qo), _i32(m.bti), _i32(m.bt)
    path = torch.full((n, NODES), -7, dtype=torch.int32, device="cuda")
    count, nxt, new = (torch.full((n,), -7, dtype=torch.int32, device="cuda") for _ in range(3))
    rounds = 0
    while any(len(done[r]) < STEPS for r in live) and kv.max() + NODES <= min(p + ROOM for p in PROMPTS):
        drafts = [_draft(rng, done[r][-1], out[r, len(done[r]):]) for r in range(n)]
        parent, tokens = (np.concatenate([d[k] for d in drafts]).astype(np.int32) for k in (0, 1))
        m.step(tokens, qo, kv + NODES, parent)
        mb.mb_verify_tree(m.logits, VOCAB, _i32(tokens), None, n, n * NODES, dqo, _i32(parent), None, None, None, NODES, count,
                          path, nxt, _stream())
        mb.mb_kv_compact(m.pools, m.P, shape.n_kv_heads, shape.head_dim, n, dqo, _i32(kv + NODES), dbti, dbt, count, path,
                         NODES, new, _stream())
        mb.mb_device_status(None, _stream())
        kv, c, p, x = (t.cpu().numpy() for t in (new, count, path, nxt))
        for r in range(n):
            done[r] += [int(tokens[qo[r] + i]) for i in p[r, 1:c[r]]] + [int(x[r])]
        rounds += 1
    m.close()
    same = 0
    for r in live:
        for t in range(min(len(done[r]) - 1, STEPS)):
            if done[r][t + 1] != out[r, t + 1]:
                assert gap[r, t] <= 2 * TOL, (r, t)
                break
            same += 1
    assert same >= n * STEPS // 2, "too few tokens were compared"
    assert rounds < STEPS, "no draft was taken"
