"""Pins of the oracle's drafted-tree functions: none compares it with itself."""
import numpy as np
import pytest
import torch

from oracle import impl as O

SCALE = dict(lora_scale=2.0, softmax_scale=0.125, rope_base=10000.0)


def _inputs(n, C, seed, A=2, kv=2, g=2, d=64, r=8, trees=1):
    rng = np.random.default_rng(seed)
    L = C + trees * n
    f = lambda *s: rng.standard_normal(s)  # noqa: E731
    return dict(k_base=f(1, kv, L, d), v_base=f(1, kv, L, d), lr=f(1, L, 2 * r),
                B_k=0.2 * f(A, r, kv * d), B_v=0.2 * f(A, r, kv * d), q=f(1, A, n, kv * g, d))


def _run(i, C, parent, tree_len=None, n_trees=1, **kw):
    a = {**i, **kw}
    return O.tree_attention(a["k_base"], a["v_base"], a["lr"], a["B_k"], a["B_v"], a["q"], [C],
                            parent, tree_len, n_trees=n_trees, **SCALE)


def test_chain_is_the_prefill():
    n, C = 5, 11
    i = _inputs(n, C, 0)
    ref = O.lora_attention(i["k_base"], i["v_base"], i["lr"], i["B_k"], i["B_v"], i["q"],
                           np.array([C + n]), mode="prefill", q_pos0=C, **SCALE)
    for parent in (None, np.array([[[-1, 0, 1, 2, 3]]])):
        for s, a, out, _, _, _ in _run(i, C, parent):
            np.testing.assert_allclose(out, ref[s, a], rtol=0, atol=1e-12)


def test_every_branch_equals_its_own_chain():
    """A node's output is that of a plain prefill of its branch alone."""
    n, C = 7, 6
    parent = [-1, 0, 0, 1, -1, 4, 3]
    i = _inputs(n, C, 1)
    res = _run(i, C, np.array([[parent]]))
    for j in range(n):
        c = [j]
        while parent[c[0]] >= 0:
            c.insert(0, parent[c[0]])
        rows = list(range(C)) + [C + k for k in c]
        ref = O.lora_attention(i["k_base"][:, :, rows], i["v_base"][:, :, rows], i["lr"][:, rows],
                               i["B_k"], i["B_v"], i["q"][:, :, c], np.array([len(rows)]),
                               mode="prefill", q_pos0=C, **SCALE)
        for s, a, out, _, _, _ in res:
            np.testing.assert_allclose(out[j], ref[s, a, -1], rtol=0, atol=1e-12)


def test_per_agent_rows_and_lengths():
    """Agent a's tree lies n rows behind agent a - 1's; its length cuts it."""
    n, C = 3, 4
    i = _inputs(n, C, 2, trees=2)
    parent = np.array([[[-1, 0, 0], [-1, -1, 1]]])
    res = _run(i, C, parent, np.array([[3, 2]]), n_trees=2)
    assert [r[2].shape[0] for r in res] == [3, 2]
    rows = list(range(C)) + [C + n, C + n + 1, C + n + 2]
    alone = _run({**i, "k_base": i["k_base"][:, :, rows], "v_base": i["v_base"][:, :, rows],
                  "lr": i["lr"][:, rows]}, C, parent[:, 1:], np.array([[2]]))
    np.testing.assert_allclose(res[1][2], alone[1][2], rtol=0, atol=1e-12)


def test_single_root_without_context_returns_its_value():
    i = _inputs(1, 0, 3)
    for s, a, out, pv, _, _ in _run(i, 0, None):
        for h in range(4):
            V = O.agent_values(i["v_base"][s, h // 2], i["lr"][s][:, 8:],
                               i["B_v"][a][:, (h // 2) * 64:(h // 2 + 1) * 64], 2.0)
            np.testing.assert_allclose(out[0, h], V[0], atol=1e-13)
            np.testing.assert_allclose(pv[0, h], np.abs(V[0]), atol=1e-13)


def test_no_key_delta_equals_zero_up_projection():
    i = _inputs(4, 9, 4)
    parent = np.array([[[-1, 0, 0, -1]]])
    a, b = _run(i, 9, parent, B_k=None), _run(i, 9, parent, B_k=np.zeros_like(i["B_k"]))
    for x, y in zip(a, b):
        np.testing.assert_array_equal(x[2], y[2])


@pytest.mark.parametrize("d", [64, 128])
def test_head_norm_against_torch(d):
    x, w = torch.randn(5, 3, d, dtype=torch.float64), torch.randn(d, dtype=torch.float64)
    ref = torch.nn.functional.rms_norm(x, (d,), w, eps=1e-5)
    np.testing.assert_allclose(O.head_norm(x, w, 1e-5), ref.numpy(), rtol=1e-12)
    assert O.head_norm(x, None, 1e-5) is not None
    np.testing.assert_array_equal(O.head_norm(x, None, 1e-5), x.numpy())


def test_grouped_delta_row_by_row():
    rng = np.random.default_rng(5)
    T, H, N, r, A = 9, 16, 8, 8, 3
    x, y = rng.standard_normal((T, H)), rng.standard_normal((T, N))
    Am, B = rng.standard_normal((A, H, r)), rng.standard_normal((A, r, N))
    start, agent = [1, 3, 3, 6, 8], [2, 0, -1, 0]
    out = O.grouped_delta(x, Am, B, y, start, agent, 0.5)
    who = {1: 2, 2: 2, 6: 0, 7: 0}
    for t in range(T):
        ref = y[t].copy()
        if t in who:
            for c in range(N):
                ref[c] += 0.5 * sum(sum(x[t, k] * Am[who[t], k, j] for k in range(H)) * B[who[t], j, c]
                                    for j in range(r))
        np.testing.assert_allclose(out[t], ref, atol=1e-12)
