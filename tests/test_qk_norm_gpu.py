"""lora_qk_norm_rope against the fp64 oracle.

A rotated element is x1 c - x2 s of normed values: its fp32 error is at most
(|x1| + |x2|) (d + 24) 2^-24 (the mean of squares: d products and sums, halved
by the root; weight, turn and the rounded cos and sin, each a few half steps),
then the output type's rounding."""
import numpy as np
import pytest
import torch

from oracle import impl as O
from tests.helpers import to_np
from tests.test_tree_gpu import parents

pytestmark = pytest.mark.gpu
DEV = "cuda"
SENT = -77.0


@pytest.fixture(scope="module")
def la():
    from rank_attention_b200 import lora_attn
    return lora_attn


def depth(parent, j):
    return len(O.tree_chain(parent, j)) - 1


def run(la, dtype=torch.bfloat16, S=1, A=2, kv=2, hq=8, d=128, n=5, ctx=(40,), per_agent=False,
        tree=True, lens=None, weights=True, fused=False, inplace=False, values=True, seed=0,
        base=500000.0, std=1.28, eps=1e-6):
    gen = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    T = A if per_agent else 1
    ctx = [ctx[s % len(ctx)] for s in range(S)]
    mx = max(ctx) + T * n
    f = lambda *sh: (torch.randn(*sh, generator=gen) * std).to(dtype)  # noqa: E731
    if fused:   # q, k, v as slices of one projection's output
        assert T == A
        buf = f(S, A, n, (hq + 2 * kv) * d).to(DEV)
        q = buf[..., :hq * d].view(S, A, n, hq, d)
        k = buf[..., hq * d:(hq + kv) * d].unflatten(-1, (kv, d))
        v = buf[..., (hq + kv) * d:].unflatten(-1, (kv, d))
        q = buf[..., :hq * d].unflatten(-1, (hq, d))
    else:
        q, k, v = f(S, A, n, hq, d).to(DEV), f(S, T, n, kv, d).to(DEV), f(S, T, n, kv, d).to(DEV)
    qh, kh, vh = q.cpu(), k.cpu(), v.cpu()
    w_q = (1 + 0.2 * torch.randn(d, generator=gen)).to(dtype) if weights else None
    w_k = (1 + 0.2 * torch.randn(d, generator=gen)).to(dtype) if weights else None
    cache = lambda: torch.full((S, kv, mx + 3, d), SENT, dtype=dtype, device=DEV)  # noqa: E731
    kb, vb = cache(), cache()
    q_out = q if inplace else torch.full((S, A, n, hq, d), SENT, dtype=dtype, device=DEV)
    par = parents(rng, S, T, n) if tree else None
    tl = None if lens is None else np.array([[lens[(s * T + t) % len(lens)] for t in range(T)]
                                             for s in range(S)], dtype=np.int32)
    ptd = None if par is None else torch.from_numpy(par).to(DEV)
    tld = None if tl is None else torch.from_numpy(tl).to(DEV)
    dev = lambda x: None if x is None else x.to(DEV)  # noqa: E731
    wqd, wkd, kl = dev(w_q), dev(w_k), torch.tensor(ctx, dtype=torch.int32, device=DEV)
    args = la.make_qk_args(q, k, v if values else None, wqd, wkd, q_out, kb, vb if values else None,
                           kl, rope_base=base, max_kv_len=mx, eps=eps)
    la.lora_qk_norm_rope(args, la.make_tree_args(ptd, tld, n_trees=T))
    torch.cuda.synchronize()
    assert la.la_device_check() == la.LA_OK
    uo = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24

    def close(got, x, w, pos):   # got, x [m, heads, d] at positions pos [m]
        nx = O.head_norm(x, w, eps)
        ref = O.rope(nx.transpose(1, 0, 2), pos, base).transpose(1, 0, 2)
        h = d // 2
        mag = np.abs(nx[..., :h]) + np.abs(nx[..., h:])
        tol = uo * np.abs(ref) + np.concatenate([mag, mag], -1) * (d + 24) * 2.0 ** -24
        assert (np.abs(to_np(got) - ref) <= tol).all(), (np.abs(to_np(got) - ref) / tol).max()

    want_v = torch.full_like(vb, SENT).cpu()
    dead = torch.ones(S, mx + 3, dtype=torch.bool)
    for s in range(S):
        for t in range(T):
            m = n if tl is None else int(tl[s, t])
            pos = np.array([ctx[s] + (depth(par[s, t], j) if tree else j) for j in range(m)])
            lo = ctx[s] + t * n
            dead[s, lo:lo + m] = False
            close(kb[s, :, lo:lo + m].transpose(0, 1), kh[s, t, :m], w_k, pos)
            want_v[s, :, lo:lo + m] = vh[s, t, :m].transpose(0, 1)
            for a in ([t] if per_agent else range(A)):
                close(q_out[s, a, :m], qh[s, a, :m], w_q, pos)
                rest = qh[s, a, m:] if inplace else torch.full_like(qh[s, a, m:], SENT)
                assert torch.equal(q_out[s, a, m:].cpu(), rest)
        assert (kb[s][:, dead[s].to(DEV)] == SENT).all()
    assert torch.equal(vb.cpu(), want_v if values else torch.full_like(want_v, SENT))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kw", [
    dict(),
    dict(n=1, ctx=(0,)),
    dict(n=64, A=3, S=2, ctx=(40, 0), lens=(64, 33)),
    dict(d=64, hq=6, kv=2, n=7, per_agent=True, lens=(7, 0)),
    dict(tree=False, n=133, S=2, ctx=(5, 90000), lens=(133, 70)),
    dict(tree=False, n=1, A=5, hq=7, kv=1, S=3, ctx=(9, 8, 131000)),
    dict(weights=False, n=9),
    dict(values=False, n=9),
    dict(fused=True, A=1, n=6),
    dict(fused=True, A=3, n=6, per_agent=True, d=64),
    dict(inplace=True, n=20, tree=False, lens=(11,)),
    dict(tree=False, n=601, A=4, hq=32, kv=8, ctx=(100,)),
])
def test_parity(la, dtype, kw):
    run(la, dtype=dtype, **kw)


def test_extreme_magnitudes(la):
    """Zero heads stay zero (eps in the root); large ones do not overflow."""
    run(la, std=1e-12, n=3)
    run(la, std=1e15, n=3, dtype=torch.float32)
    run(la, std=0.0, n=3)


def test_only_queries_or_only_keys(la):
    q = torch.randn(2, 3, 4, 8, 128, device=DEV).to(torch.bfloat16)
    out, kl = torch.empty_like(q), torch.tensor([5, 70], dtype=torch.int32, device=DEV)
    w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    la.lora_qk_norm_rope(la.make_qk_args(q, None, None, w, None, out, None, None, kl,
                                         rope_base=10000.0, max_kv_len=80))
    k = torch.randn(2, 1, 4, 2, 128, device=DEV).to(torch.bfloat16)
    kb = torch.zeros(2, 2, 80, 128, dtype=torch.bfloat16, device=DEV)
    la.lora_qk_norm_rope(la.make_qk_args(None, k, None, None, None, None, kb, None, kl,
                                         rope_base=10000.0, max_kv_len=80))
    torch.cuda.synchronize()
    for s in range(2):
        pos = int(kl[s]) + np.arange(4)
        ref = O.rope(O.head_norm(to_np(q[s]).transpose(0, 2, 1, 3), np.ones(128), 1e-6), pos, 10000.0)
        assert np.abs(to_np(out[s]).transpose(0, 2, 1, 3) - ref).max() <= 2.0 ** -8 * np.abs(ref).max()
        rk = O.rope(to_np(k[s, 0]).transpose(1, 0, 2), pos, 10000.0)
        got = to_np(kb[s, :, int(kl[s]):int(kl[s]) + 4])
        assert np.abs(got - rk).max() <= 2.0 ** -8 * np.abs(rk).max()


def test_bad_lengths_are_reported(la):
    for what, bit in (("kv", la.LA_DEV_KV_LEN), ("len", la.LA_DEV_TREE), ("parent", la.LA_DEV_TREE)):
        q = torch.randn(2, 1, 3, 4, 128, device=DEV).to(torch.bfloat16)
        k = torch.randn(2, 1, 3, 2, 128, device=DEV).to(torch.bfloat16)
        kb = torch.full((2, 2, 20, 128), SENT, dtype=torch.bfloat16, device=DEV)
        vb, out = kb.clone(), torch.full_like(q, SENT)
        kl = torch.tensor([4, 18 if what == "kv" else 5], dtype=torch.int32, device=DEV)
        tl = torch.tensor([[3], [4 if what == "len" else 3]], dtype=torch.int32, device=DEV)
        par = torch.tensor([[[-1, 0, 1]], [[-1, 1 if what == "parent" else 0, 0]]],
                           dtype=torch.int32, device=DEV)
        la.lora_qk_norm_rope(la.make_qk_args(q, k, k, None, None, out, kb, vb, kl, rope_base=1e4,
                                             max_kv_len=20), la.make_tree_args(par, tl))
        assert la.la_device_check_word() == (la.LA_ERR_DEVICE_CHECK, bit)
        assert (out[1] == SENT).all() and (kb[1] == SENT).all() and (vb[1] == SENT).all()
        assert (out[0] != SENT).all()
