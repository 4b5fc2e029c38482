"""One layer of a verification step, its calls in a row as a server makes them:
grouped query deltas, norm and rotation with the cache rows, the LR rows, tree
attention, grouped output deltas.  Every stage is checked against the fp64 oracle
on what that stage read (the bounds are the stages' own tests'), eagerly and
replayed from one captured graph with other lengths, trees and tokens."""
import numpy as np
import pytest
import torch

from oracle import impl as O
from tests import test_tree_gpu as T
from tests.helpers import to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def la():
    from rank_attention_b200 import lora_attn
    return lora_attn


def grouped_tol(ref, mag, y, hidden, r):
    """The bound of the grouped products' own test, bf16."""
    return 2.0 ** -8 * np.abs(ref) + mag * ((hidden + r + 8) * 2.0 ** -24 + 2.0 ** -16) + 2.0 ** -24 * np.abs(y)


class Layer:
    """A = 3 agents on one sequence, each with a tree of up to n nodes."""

    def __init__(self, la, keys, per_agent, H=256, kv=2, g=4, d=128, r=16, L=512, n=11, seed=0):
        gen = torch.Generator().manual_seed(seed)
        f = lambda *s, std=1.0: (torch.randn(*s, generator=gen) * std).to(torch.bfloat16).to(DEV)  # noqa: E731
        A = self.A = 3
        self.la, self.keys, self.n, self.r, self.d, self.kv, self.g, self.H = la, keys, n, r, d, kv, g, H
        self.T = A if per_agent else 1
        hq = kv * g
        self.W_q, self.W_k, self.W_v = f(H, hq * d, std=H ** -0.5), f(H, kv * d, std=H ** -0.5), f(H, kv * d, std=H ** -0.5)
        self.W_o = f(hq * d, H, std=(hq * d) ** -0.5)
        self.A_q, self.B_q = f(H, r, std=H ** -0.5), f(A, r, hq * d, std=0.05)     # shared down-projection
        self.A_o, self.B_o = f(A, hq * d, r, std=(hq * d) ** -0.5), f(A, r, H, std=0.05)
        self.A_kv = f(H, 2 * r, std=H ** -0.5)
        self.B_k, self.B_v = (f(A, r, kv * d, std=0.05) if keys else None), f(A, r, kv * d, std=0.05)
        self.w_q = self.w_k = None
        if not keys:   # a norm does not split into base and delta: keys shared outright
            self.w_q, self.w_k = 1 + f(d, std=0.1), 1 + f(d, std=0.1)
        self.k, self.v, self.lr = f(1, kv, L, d, std=T.STD), f(1, kv, L, d, std=T.STD), f(1, L, 2 * r, std=T.STD)
        z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
        rows = A * n
        self.x, self.xt = z(rows, H), z(self.T * n, H)
        self.q, self.qr, self.o = z(rows, hq * d), z(1, A, n, hq, d), z(1, A, n, hq, d)
        self.kvn = z(self.T * n, 2 * kv * d)     # k and v of the drafted tokens side by side
        self.y, self.out = z(rows, H), z(rows, H)
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)  # noqa: E731
        self.C, self.parent, self.tl = i32(1), i32(1, self.T, n), i32(1, self.T)
        self.seg, self.who = i32(A + 1), i32(A)
        self.L = L
        kn = self.kvn.view(1, self.T, n, 2 * kv, d)
        self.tree = la.make_tree_args(self.parent, self.tl)
        self.a_q = la.make_grouped_args(self.x, self.A_q, self.B_q, self.q, self.q, self.seg, self.who, lora_scale=2.0)
        self.a_n = la.make_qk_args(self.q.view(1, A, n, hq, d), kn[:, :, :, :kv], kn[:, :, :, kv:], self.w_q, self.w_k,
                                   self.qr, self.k, self.v, self.C, rope_base=10000.0, max_kv_len=L)
        self.a_t = la.make_args(self.k, self.v, self.lr, self.B_k, self.B_v, self.qr, self.o, lora_scale=2.0,
                                rope_base=10000.0, kv_len=self.C, max_kv_len=L)
        self.a_o = la.make_grouped_args(self.o.view(rows, hq * d), self.A_o, self.B_o, self.y, self.out, self.seg,
                                        self.who, lora_scale=2.0)

    def feed(self, C, lens, seed):
        """New tokens, trees and lengths in the same buffers."""
        gen, rng = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
        self.x.copy_(torch.randn(self.x.shape, generator=gen).to(torch.bfloat16))
        self.xt.copy_(self.x[:self.T * self.n])
        self.parent.copy_(torch.from_numpy(T.parents(rng, 1, self.T, self.n)))
        self.tl.copy_(torch.tensor([lens[:self.T]], dtype=torch.int32))
        self.C.fill_(C)
        self.c = C
        # a segment is an agent's n rows, the unused ones behind its tree included
        cuts = [a * self.n for a in range(self.A)] + [self.A * self.n]
        self.seg.copy_(torch.tensor(cuts, dtype=torch.int32))
        self.who.copy_(torch.arange(self.A, dtype=torch.int32))
        for t in (self.o, self.out):
            t.zero_()

    def step(self):
        la = self.la
        torch.mm(self.x, self.W_q, out=self.q)
        torch.mm(self.xt, self.W_k, out=self.kvn[:, :self.kv * self.d])
        torch.mm(self.xt, self.W_v, out=self.kvn[:, self.kv * self.d:])
        la.lora_grouped_delta(self.a_q)
        la.lora_qk_norm_rope(self.a_n, self.tree)
        la.lr_cache_append(self.xt.view(1, -1, self.H), self.A_kv, self.lr, self.c)
        la.lora_attn_tree(self.a_t, self.tree)
        torch.mm(self.o.view(self.A * self.n, -1), self.W_o, out=self.y)
        la.lora_grouped_delta(self.a_o)

    def check(self):
        la, A, n, d = self.la, self.A, self.n, self.d
        assert la.la_device_check() == la.LA_OK
        # queries: delta, then norm and rotation; the projection itself is the library product's
        q0 = to_np(torch.mm(self.x, self.W_q))
        cuts, who = self.seg.tolist(), self.who.tolist()
        ref = O.grouped_delta(self.x.cpu(), self.A_q.cpu(), self.B_q.cpu(), q0, cuts, who, 2.0)
        got = to_np(self.q)
        mag = O.grouped_delta(self.x.abs().cpu(), self.A_q.abs().cpu(), self.B_q.abs().cpu(), 0 * q0, cuts, who, 2.0)
        assert (np.abs(got - ref) <= grouped_tol(ref, mag, q0, self.H, self.r)).all()
        par, tl, C = self.parent.cpu().numpy(), self.tl.cpu().numpy(), self.c
        for a in range(A):
            t = a if self.T > 1 else 0
            m = int(tl[0, t])
            pos = C + np.array([len(O.tree_chain(par[0, t], j)) - 1 for j in range(m)])
            for src, w, dst in ((got.reshape(A, n, -1, d)[a, :m], self.w_q, self.qr[0, a, :m]),
                                (to_np(self.kvn).reshape(self.T, n, -1, d)[t, :m, :self.kv], self.w_k,
                                 self.k[0, :, C + t * n: C + t * n + m].transpose(0, 1))):
                nx = O.head_norm(src, None if w is None else w.cpu(), 1e-6)
                rot = O.rope(nx.transpose(1, 0, 2), pos, 10000.0).transpose(1, 0, 2)
                mag = np.abs(nx[..., :d // 2]) + np.abs(nx[..., d // 2:])
                tol = 2.0 ** -8 * np.abs(rot) + np.concatenate([mag, mag], -1) * (d + 24) * 2.0 ** -24
                assert (np.abs(to_np(dst) - rot) <= tol).all()
        # attention over the caches as the step left them
        cpu = lambda x: None if x is None else x.cpu()  # noqa: E731
        T.check(la, dict(k_base=cpu(self.k), v_base=cpu(self.v), lr=cpu(self.lr), B_k=cpu(self.B_k), B_v=cpu(self.B_v),
                         q=cpu(self.qr), kv_len=self.C.cpu(), parent=par, tree_len=tl, n_trees=self.T,
                         max_kv_len=self.L, base=10000.0), self._unwritten(), torch.bfloat16)
        y = to_np(self.y)
        o = self.o.view(A * n, -1)
        ref = O.grouped_delta(o.cpu(), self.A_o.cpu(), self.B_o.cpu(), y, cuts, who, 2.0)
        mag = O.grouped_delta(o.abs().cpu(), self.A_o.abs().cpu(), self.B_o.abs().cpu(), 0 * y, cuts, who, 2.0)
        assert (np.abs(to_np(self.out) - ref) <= grouped_tol(ref, mag, y, self.kv * self.g * d, self.r)).all()

    def _unwritten(self):
        """The attention's outputs, rows of nodes past tree_len marked as T.check expects."""
        o = self.o.clone()
        for a in range(self.A):
            m = int(self.tl[0, a if self.T > 1 else 0])
            assert (o[0, a, m:] == 0).all()
            o[0, a, m:] = T.SENT
        return o


@pytest.mark.parametrize("keys,per_agent", [(True, True), (True, False), (False, True), (False, False)])
def test_a_layer_of_a_verification_step(la, keys, per_agent):
    layer = Layer(la, keys, per_agent)
    layer.feed(300, [11, 4, 7], 1)
    layer.step()
    torch.cuda.synchronize()
    layer.check()
    # one graph of the step (the committed length of the LR append is an argument: the
    # graph's is 300), replayed with another tree and other tokens
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer.step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.step()
    layer.feed(300, [9, 11, 1], 2)
    g.replay()
    torch.cuda.synchronize()
    layer.check()
