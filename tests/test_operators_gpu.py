"""Calls of the drafted-tree operators that their documentation allows and no other test
makes, against the fp64 oracle within the operators' own bounds."""
import threading
from pathlib import Path

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


def grouped_tol(ref, mag, y, hidden, r, bf):
    """The bound of the grouped products' own tests."""
    return (2.0 ** -8 if bf else 2.0 ** -24) * np.abs(ref) + \
        mag * ((hidden + r + 8) * 2.0 ** -24 + (2.0 ** -16 if bf else 0)) + 2.0 ** -24 * np.abs(y)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_grouped_over_a_million_tokens(la, dtype):
    """More tokens than 65535 tiles of 16 rows: the kernel's own tile height counts."""
    T, H, N, r = 1100003, 64, 64, 8
    gen = torch.Generator(device=DEV).manual_seed(1)
    f = lambda *s, std=1.0: (torch.randn(*s, generator=gen, device=DEV) * std).to(dtype)  # noqa: E731
    x, y, A, B = f(T, H), f(T, N), f(2, H, r, std=0.05), f(2, r, N, std=0.05)
    out = torch.zeros_like(y)
    cuts, who = [0, 70001, T - 1], [1, 0]
    ss, sa = (torch.tensor(v, dtype=torch.int32, device=DEV) for v in (cuts, who))
    la.lora_grouped_delta(la.make_grouped_args(x, A, B, y, out, ss, sa, lora_scale=2.0))
    torch.cuda.synchronize()
    assert la.la_device_check() == la.LA_OK
    for lo, hi, a in ((0, 200, 1), (69900, 70001, 1), (70001, 70200, 0), (1048500, 1048700, 0), (T - 300, T - 1, 0)):
        xs, ys = x[lo:hi].cpu(), to_np(y[lo:hi])
        ref = O.grouped_delta(xs, A.cpu(), B.cpu(), ys, [0, hi - lo], [a], 2.0)
        mag = O.grouped_delta(xs.abs(), A.abs().cpu(), B.abs().cpu(), 0 * ys, [0, hi - lo], [a], 2.0)
        err = np.abs(to_np(out[lo:hi]) - ref)
        assert (err <= grouped_tol(ref, mag, ys, H, r, dtype == torch.bfloat16)).all(), (lo, a)
    assert (out[T - 1] == 0).all(), "the row in no segment was written"


@pytest.mark.parametrize("keys", [True, False])
def test_kernels_with_tensor_memory_on_streams_of_their_own(la, keys):
    """Trees of head_dim 64 (all TMEM columns), grouped products and LR appends (some of
    them), each a grid of clusters, in flight together: the same bits as alone."""
    i = T.make(S=4, A=3, kv=4, d=64, r=16, ctx=(1500, 900, 2048, 30), n=9, per_agent=True, keys=keys, garbage=False, seed=31)
    args, tree, out, keep = T.launch(la, i)
    gen = torch.Generator(device=DEV).manual_seed(2)
    f = lambda *s, std=1.0: (torch.randn(*s, generator=gen, device=DEV) * std).to(torch.bfloat16)  # noqa: E731
    x, y, A, B = f(3000, 2048), f(3000, 1024), f(3, 2048, 64, std=0.05), f(3, 64, 1024, std=0.05)
    o = torch.zeros_like(y)
    ss, sa = (torch.tensor(v, dtype=torch.int32, device=DEV) for v in ([0, 700, 1600, 3000], [2, 0, 1]))
    ga = la.make_grouped_args(x, A, B, y, o, ss, sa, lora_scale=2.0)
    X, A_kv, lr = f(2, 700, 2048), f(2048, 64, std=0.02), torch.zeros(2, 800, 64, dtype=torch.bfloat16, device=DEV)
    calls = [(lambda: la.lora_attn_tree(args, tree), out), (lambda: la.lora_grouped_delta(ga), o),
             (lambda: la.lr_cache_append(X, A_kv, lr, 17), lr)]
    alone = []
    for call, res in calls:
        call()
        torch.cuda.synchronize()
        alone.append(res.clone())
        res.zero_()
    T.check(la, i, alone[0], torch.bfloat16)
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (call, _) in zip(streams, calls):
            with torch.cuda.stream(s):
                call()
    torch.cuda.synchronize()
    assert la.la_device_check() == la.LA_OK
    for (_, res), ref in zip(calls, alone):
        assert torch.equal(torch.where(ref == T.SENT, ref, res), ref)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("s,b_std", [(1.1e-5, 2e4), (3e5, 1e-6), (-0.75, 0.05), (2.0 ** -20, 3e5), (7e9, 3e-11), (0.0, 1.0)])
def test_tree_takes_any_scale_the_delta_fits(la, d, s, b_std):
    """Only K^a and the scaled delta have to lie in fp16's range, neither s nor LRk B_k^a
    alone: deltas of about one from a small s and products beyond 65504, and the reverse.
    (The bound of the trees' tests, on up-projections that carry s.)"""
    i = T.make(d=d, r=16, ctx=(300,), n=7, garbage=False, seed=32)
    s = float(np.float32(s))
    gen = torch.Generator().manual_seed(33)
    for k in ("B_k", "B_v"):
        i[k] = (torch.randn(i[k].shape, generator=gen) * b_std).to(torch.bfloat16)
    args, tree, out, keep = T.launch(la, i, torch.float32)
    args.lora_scale = s
    la.lora_attn_tree(args, tree)
    torch.cuda.synchronize()
    assert la.la_device_check() == la.LA_OK
    T.check(la, {**i, **{k: i[k].double() * (s / 2.0) for k in ("B_k", "B_v")}}, out, torch.float32)   # its scale is 2


def in_threads(*works):
    """Run every function in a host thread of its own, all at once; their errors."""
    errors = []

    def run(f):
        try:
            f()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(f,)) for f in works]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return errors


def test_threads_with_different_ranks(la):
    """Two host threads call at once, each with a rank (a shared-memory size) of its own."""
    runs = []
    for r in (8, 64):
        i = T.make(dtype=torch.float32, d=64, r=r, ctx=(90,), n=4, garbage=False, seed=r)
        runs.append((i, torch.cuda.Stream(), *T.launch(la, i, torch.float32)))
    torch.cuda.synchronize()

    def work(s, args, tree):
        for _ in range(2000):
            la.lora_attn_tree(args, tree, stream=s)

    assert in_threads(*(lambda x=x: work(*x[1:4]) for x in runs)) == []
    for i, s, args, tree, out, keep in runs:
        T.check(la, i, out, torch.float32)


def test_threads_with_different_shapes_of_prefill_and_decode(la):
    """The same for the prefill and decode kernels whose shared memory goes by the call."""
    def prepared(decode, **kw):
        i = T.make(ctx=(90,), n=1 if decode else 4, garbage=False, **kw)
        d = {k: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in i.items()}
        out = torch.zeros(d["q"].shape, dtype=torch.float32, device=DEV)
        args = la.make_args(d["k_base"], d["v_base"], d["lr"], d["B_k"], d["B_v"], d["q"], out, lora_scale=2.0,
                            rope_base=i["base"], kv_len=d["kv_len"] + 1, max_kv_len=91, q_pos0=90)
        ws, s = la.decode_workspace(args, DEV) if decode else None, torch.cuda.Stream()

        def work(n=1000):
            for _ in range(n):
                la.lora_attn_decode(args, ws, stream=s) if decode else la.lora_attn_prefill(args, stream=s)

        work(1)
        torch.cuda.synchronize()
        return work, out, out.clone()

    f32 = torch.float32
    for decode, kws in ((False, (dict(dtype=f32, d=64, r=8, A=1, g=1), dict(dtype=f32, d=64, r=64, A=2, g=4))),
                        (True, (dict(dtype=f32, d=64, r=8, A=1, g=1), dict(dtype=f32, d=64, r=64, A=2, g=4))),
                        (True, (dict(r=16, A=1, g=4), dict(r=16, A=3, g=4))),      # tensor-core decode
                        (True, (dict(r=8, A=1, g=4), dict(r=8, A=2, g=4)))):       # bf16, r = 8
        runs = [prepared(decode, seed=40 + j, **kw) for j, kw in enumerate(kws)]
        assert in_threads(*(w for w, _, _ in runs)) == [], (decode, kws)
        for _, out, ref in runs:
            assert (out - ref).abs().max() <= 1e-5 * ref.abs().max()
    assert la.la_device_check() == la.LA_OK


def test_first_cuda_call_of_a_thread(la):
    """A host thread that has made no CUDA call before calls an entry point with tensor
    maps: the thread has no context of its own yet."""
    i = T.make(ctx=(90,), n=4, garbage=False, seed=34)
    args, tree, out, keep = T.launch(la, i)
    d = keep[0]
    ref = torch.zeros_like(out)
    pre = la.make_args(d["k_base"], d["v_base"], d["lr"], d["B_k"], d["B_v"], d["q"], ref, lora_scale=2.0,
                       rope_base=i["base"], q_pos0=90)
    q1 = d["q"][:, :, :1].contiguous()
    dec = la.make_args(d["k_base"], d["v_base"], d["lr"], d["B_k"], d["B_v"], q1, torch.zeros_like(q1), lora_scale=2.0,
                       rope_base=i["base"], kv_len=d["kv_len"], max_kv_len=94)
    ws = la.decode_workspace(dec, DEV)
    z = lambda *s: torch.ones(*s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    ss, sa = (torch.tensor(v, dtype=torch.int32, device=DEV) for v in ([0, 9], [0]))
    ga = la.make_grouped_args(z(9, 64), z(64, 16), z(1, 16, 64), z(9, 64), z(9, 64), ss, sa, lora_scale=1.0)
    X, A_kv, lr = z(1, 40, 256), z(256, 64), z(1, 40, 64)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for call in (lambda: la.lora_attn_tree(args, tree, stream=s), lambda: la.lora_attn_prefill(pre, stream=s),
                 lambda: la.lora_attn_decode(dec, ws, stream=s), lambda: la.lora_grouped_delta(ga, stream=s),
                 lambda: la.lr_cache_append(X, A_kv, lr, 0, stream=s)):
        assert in_threads(call) == []
    assert la.la_device_check() == la.LA_OK
    T.check(la, i, out, torch.bfloat16)
    assert (lr == 256).all() and (ga.keep[4] == 1 + 64 * 16).all()


# ---- forms that no other test runs
@pytest.mark.parametrize("r", [8, 16, 32, 64])
@pytest.mark.parametrize("keys", [True, False])
@pytest.mark.parametrize("n", [13, 27])   # folded, and with two warps a row
def test_tree_head_dim_64_many_tiles(la, r, keys, n):
    """head_dim 64 over long unsplit runs of tiles: both dK buffers, every K, V and LR stage
    refilled many times, partial context tiles and drafted ones at their end."""
    T.run(la, S=3, A=4, kv=8, g=4, d=64, r=r, ctx=(2999, 1777, 2421), n=n, per_agent=True, lens=(13, 9, 2, 7, 12),
          keys=keys, seed=r + n)


def test_tree_of_one_node_is_the_decode(la):
    """Committed length C in front of one node is the decode of kv_len = C + 1, and a chain the
    prefill: row and position conventions of three entry points, within the bf16 bound of the
    library's paths (1e-2 of the largest output), over ranks and lengths off the tile."""
    for r, ctx in ((16, (200, 77)), (64, (383, 1)), (32, (128, 1290))):
        for n in (1, 9):
            i = T.make(S=2, A=2, r=r, ctx=ctx, n=n, extra=0, garbage=False, seed=r + n)
            i["parent"] = None
            args, tree, out, keep = T.launch(la, i, torch.float32)
            la.lora_attn_tree(args, tree)
            d = keep[0]
            caches = (d["k_base"], d["v_base"], d["lr"], d["B_k"], d["B_v"])
            ref = torch.zeros_like(out)
            if n == 1:
                dec = la.make_args(*caches, d["q"], ref, lora_scale=2.0, rope_base=i["base"], kv_len=d["kv_len"] + 1,
                                   max_kv_len=i["max_kv_len"])
                la.lora_attn_decode(dec, la.decode_workspace(dec, DEV))
            for s in range(2 if n > 1 else 0):   # one prefill a sequence: its first position is the host's
                one = [x[s:s + 1] for x in caches[:3]]
                la.lora_attn_prefill(la.make_args(*one, *caches[3:], d["q"][s:s + 1], ref[s:s + 1], lora_scale=2.0,
                                                  rope_base=i["base"], q_pos0=ctx[s]))
            torch.cuda.synchronize()
            assert la.la_device_check() == la.LA_OK
            T.check(la, i, out, torch.float32)
            assert (out - ref).abs().max() <= 1e-2 * ref.abs().max(), (r, ctx, n)


def test_tree_launches_in_a_row_over_every_form(la):
    """Thirty launches give the same bits, head_dim 64 and rank 8 among them."""
    for kw in (dict(d=64, r=16, n=13), dict(d=64, r=64, n=27), dict(d=64, r=32, n=27, keys=False), dict(d=128, r=8, n=13),
               dict(d=64, r=8, n=5, lr_agents=True)):
        i = T.make(S=4, A=3, kv=2, g=3, ctx=(1450, 700, 1101, 481), per_agent=True, garbage=False, seed=35, **kw)
        args, tree, out, keep = T.launch(la, i)
        la.lora_attn_tree(args, tree)
        torch.cuda.synchronize()
        T.check(la, i, out, torch.bfloat16)
        first = out.clone()
        for _ in range(30):
            out.fill_(T.SENT)
            la.lora_attn_tree(args, tree)
            assert torch.equal(out, first), kw
    assert la.la_device_check() == la.LA_OK


def test_readme_layer_runs(la):
    """README's layer of a verification step, word for word, over a batch of two lengths."""
    text = (Path(__file__).resolve().parent.parent / "README.md").read_text()
    part = text.split("## Verifying drafted tokens")[1].split("\n## ")[0]
    code = "\n".join(ln[4:] for ln in part.splitlines() if ln.startswith("    "))
    assert "lora_attn_tree" in code and code.count("lora_grouped_delta") == 2
    i = T.make(S=2, A=2, kv=2, g=2, d=64, r=16, ctx=(90, 41), n=5, lens=(5, 3), extra=0, garbage=False, seed=36, base=1e4)
    args, tree, o, (dd, _, par, tl) = T.launch(la, i)
    gen = torch.Generator(device=DEV).manual_seed(37)
    f = lambda *s, std=1.0: (torch.randn(*s, generator=gen, device=DEV) * std).to(torch.bfloat16)  # noqa: E731
    H, r, n, n_q, d, rows = 128, 16, 5, 4, 64, 20
    seg_start, seg_agent = (torch.tensor(v, dtype=torch.int32, device=DEV) for v in ([0, 5, 10, 15, 20], [0, 1, 0, 1]))
    env = dict(la=la, parent=par, tree_len=tl, n_q=n_q, d=d, x=f(rows, H), q=f(2, 2, n, n_q, d), A_q=f(H, r, std=H ** -0.5),
               B_q=f(2, r, n_q * d, std=0.05), seg_start=seg_start, seg_agent=seg_agent, s=2.0, base=1e4, L=i["max_kv_len"],
               k=f(2, 1, n, 2, d), v=f(2, 1, n, 2, d), w_q=None, w_k=None, q_rot=torch.zeros_like(dd["q"]),
               k_base=dd["k_base"], v_base=dd["v_base"], kv_len=dd["kv_len"], lengths=i["kv_len"].tolist(),
               x_tree=f(2, n, H), A_kv=f(H, 2 * r, std=H ** -0.5), lr_cache=dd["lr"], B_k=dd["B_k"], B_v=dd["B_v"], o=o,
               A_o=f(2, n_q * d, r, std=0.05), B_o=f(2, r, H, std=0.05), y=f(rows, H), out=torch.zeros(rows, H, dtype=torch.bfloat16, device=DEV))
    q0, lr0 = env["q"].clone(), dd["lr"].clone()
    exec(code, env)
    torch.cuda.synchronize()
    assert la.la_device_check() == la.LA_OK
    cuts, who = seg_start.tolist(), seg_agent.tolist()

    def products(x, A, B, y, got):
        ref = O.grouped_delta(x.cpu(), A.cpu(), B.cpu(), to_np(y), cuts, who, 2.0)
        mag = O.grouped_delta(x.abs().cpu(), A.abs().cpu(), B.abs().cpu(), 0 * to_np(y), cuts, who, 2.0)
        assert (np.abs(to_np(got) - ref) <= grouped_tol(ref, mag, to_np(y), x.shape[1], r, True)).all()

    products(env["x"], env["A_q"], env["B_q"], q0.view(rows, -1), env["q"].view(rows, -1))
    for s in range(2):   # the LR rows: at their places, the others as they were
        C = env["lengths"][s]
        want = env["x_tree"][s].double() @ env["A_kv"].double()
        mag = env["x_tree"][s].abs().double() @ env["A_kv"].abs().double()
        assert ((dd["lr"][s, C:C + n].double() - want).abs() <= 2.0 ** -8 * want.abs() + mag * (H + 8) * 2.0 ** -24).all()
        assert torch.equal(dd["lr"][s, :C], lr0[s, :C]) and torch.equal(dd["lr"][s, C + n:], lr0[s, C + n:])
    T.check(la, {**i, **{k: dd[k].cpu() for k in ("k_base", "v_base", "lr")}, "q": env["q_rot"].cpu()}, o, torch.bfloat16)
    products(o.view(rows, -1), env["A_o"], env["B_o"], env["y"], env["out"])
