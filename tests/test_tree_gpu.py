"""lora_attn_tree against the fp64 oracle, with tolerances from the roundings.

|out - ref| <= uo |ref| + (u_P + 2 delta) (P |V^a|), where uo is the output
type's half step, u_P the rounding of a softmax weight, and delta a bound on a
score's error (a weight's relative change, in numerator and denominator):
  tensor cores: u_P = 2^-8 (bf16 P) + 2^-13 (the polynomial 2^x, 7.5e-5);
    with a key delta, delta = scale (2^-11 |q||K^a| + 12 2^-11 |q||dK|): K^a
    rounded once to fp16, and of the delta alone the conversion, two turns with
    fp16 (cos, sin) and their sums (each at most sqrt 2 times 2^-11);
    without one, delta = scale d 2^-24 |q||K| (fp32 accumulation).
  CUDA cores: u_P = 4 2^-24 + L 2^-24 (a sequential sum over L keys),
    delta = scale (d 2^-24 |q||K^a| + (r + 16) 2^-24 |q||dK|)."""
import numpy as np
import pytest
import torch

from oracle import impl as O
from rank_attention_b200 import workloads as W
from tests.helpers import to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"
STD = W.CACHE_STD
SENT = -77.0
U = 2.0 ** -24


@pytest.fixture(scope="module")
def la():
    from rank_attention_b200 import lora_attn
    return lora_attn


def parents(rng, S, T, n):
    p = np.full((S, T, n), -1, dtype=np.int32)
    for s in range(S):
        for t in range(T):
            for j in range(1, n):
                p[s, t, j] = -1 if rng.random() < 0.2 else rng.integers(0, j)
    return p


def make(dtype=torch.bfloat16, S=1, A=2, kv=2, g=4, d=128, r=16, ctx=(300,), n=5, per_agent=False,
         keys=True, lens=None, lr_agents=False, tok_major=False, extra=7, garbage=True, seed=0,
         base=500000.0):
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    T = A if per_agent else 1
    ctx = [ctx[s % len(ctx)] for s in range(S)]
    max_len = max(ctx) + T * n
    L = max_len + extra
    f = lambda *sh, std=STD: (torch.randn(*sh, generator=gen) * std).to(dtype)  # noqa: E731
    i = dict(k_base=f(S, kv, L, d), v_base=f(S, kv, L, d), q=f(S, A, n, kv * g, d),
             lr=f(A, S, L, 2 * r) if lr_agents else f(S, L, 2 * r),
             B_k=f(A, r, kv * d, std=0.02 * (1 if r >= 16 else 2)) if keys else None,
             B_v=f(A, r, kv * d, std=0.02))
    tl = None if lens is None else np.array([[lens[(s * T + t) % len(lens)] for t in range(T)]
                                             for s in range(S)], dtype=np.int32)
    if garbage:   # rows no node may see: anything, NaN and infinities included
        for s in range(S):
            dead = torch.ones(L, dtype=torch.bool)
            dead[:ctx[s]] = False
            for t in range(T):
                m = n if tl is None else tl[s, t]
                dead[ctx[s] + t * n: ctx[s] + t * n + m] = False
            junk = torch.tensor([float("nan"), float("inf"), -float("inf")], dtype=dtype)
            for x in (i["k_base"][s], i["v_base"][s]):
                x[:, dead] = junk[torch.arange(d) % 3]
            for x in ([i["lr"][a, s] for a in range(A)] if lr_agents else [i["lr"][s]]):
                x[dead] = junk[torch.arange(2 * r) % 3]
    i.update(kv_len=torch.tensor(ctx, dtype=torch.int32), parent=parents(rng, S, T, n), tree_len=tl,
             n_trees=T, max_kv_len=max_len, tok_major=tok_major, base=base)
    return i


def launch(la, i, out_dtype=torch.bfloat16, stream=None, softmax_scale=None):
    d = {k: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in i.items()}
    if i["tok_major"]:   # [n_seqs, L, n_kv, d] storage
        d["k_base"], d["v_base"] = (x.transpose(1, 2).contiguous().transpose(1, 2)
                                    for x in (d["k_base"], d["v_base"]))
    out = torch.full(i["q"].shape, SENT, dtype=out_dtype, device=DEV)
    args = la.make_args(d["k_base"], d["v_base"], d["lr"], d["B_k"], d["B_v"], d["q"], out,
                        lora_scale=2.0, rope_base=i["base"], kv_len=d["kv_len"],
                        max_kv_len=i["max_kv_len"], softmax_scale=softmax_scale)
    par = None if i["parent"] is None else torch.from_numpy(i["parent"]).to(DEV)
    tl = None if i["tree_len"] is None else torch.from_numpy(i["tree_len"]).to(DEV)
    tree = la.make_tree_args(par, tl, n_trees=i["n_trees"])
    keep = (d, out, par, tl)
    return args, tree, out, keep


def check(la, i, out, out_dtype, softmax_scale=None):
    scale = softmax_scale or i["q"].shape[-1] ** -0.5
    d, r, dt = i["q"].shape[-1], i["lr"].shape[-1] // 2, i["q"].dtype
    L = i["max_kv_len"]
    uo = 2.0 ** -8 if out_dtype == torch.bfloat16 else U
    got = to_np(out)
    tc = dt == torch.bfloat16
    for s, a, ref, pv, qk, qd in O.tree_attention(
            i["k_base"], i["v_base"], i["lr"], i["B_k"], i["B_v"], i["q"], i["kv_len"], i["parent"],
            i["tree_len"], n_trees=i["n_trees"], lora_scale=2.0, softmax_scale=scale,
            rope_base=i["base"]):
        m = ref.shape[0]
        if tc:
            u_p = 2.0 ** -8 + 2.0 ** -13 + L * U
            delta = scale * ((2.0 ** -11 * qk + 12 * 2.0 ** -11 * qd) if i["B_k"] is not None
                             else d * U * qk)
        else:
            u_p = 4 * U + L * U
            delta = scale * (d * U * qk + (r + 16) * U * qd)
        tol = uo * np.abs(ref) + (u_p + 2 * delta)[..., None] * pv + 1e-30
        assert np.isfinite(got[s, a, :m]).all(), (s, a)
        worst = (np.abs(got[s, a, :m] - ref) / tol).max() if m else 0.0
        assert worst <= 1.0, (s, a, worst)
        assert (got[s, a, m:] == SENT).all(), "a node past tree_len was written"


def run(la, out_dtype=torch.bfloat16, **kw):
    i = make(**kw)
    args, tree, out, keep = launch(la, i, out_dtype)
    la.lora_attn_tree(args, tree)
    torch.cuda.synchronize()
    assert la.la_device_check() == la.LA_OK
    check(la, i, out, out_dtype)


F32 = dict(dtype=torch.float32)


@pytest.mark.parametrize("kw", [
    dict(F32, d=64, r=8, g=2, ctx=(256,), n=8, base=10000.0),
    dict(F32, d=128, r=64, g=1, ctx=(0,), n=1),
    dict(F32, d=64, r=16, g=3, ctx=(33, 0, 1), S=3, n=33, lens=(33, 0, 20)),
    dict(F32, d=128, r=32, g=7, ctx=(700,), n=9, per_agent=True, lens=(9, 4)),
    dict(F32, d=128, r=16, g=8, ctx=(95,), n=64, keys=False),
    dict(F32, d=128, r=16, g=4, ctx=(128, 127), S=2, n=17, lr_agents=True, tok_major=True),
    dict(F32, d=64, r=8, g=64, kv=1, A=1, ctx=(40,), n=2),
])
def test_fp32(la, kw):
    run(la, out_dtype=torch.float32, **kw)


@pytest.mark.parametrize("r", [8, 16, 32, 64])
@pytest.mark.parametrize("keys", [True, False])
def test_bf16_ranks(la, r, keys):
    run(la, r=r, keys=keys, ctx=(300,), n=13, seed=r)


@pytest.mark.parametrize("ctx", [0, 1, 127, 128, 129, 255, 256, 257, 641])
def test_bf16_context_lengths(la, ctx):
    run(la, ctx=(ctx,), n=3, seed=ctx)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64])
def test_bf16_node_counts(la, n):
    run(la, ctx=(190,), n=n, seed=n)


@pytest.mark.parametrize("g", [1, 2, 3, 5, 7, 8, 16])
def test_bf16_groups(la, g):
    run(la, g=g, kv=2, A=1, ctx=(200,), n=21, seed=g)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("r", [8, 32])
def test_bf16_head_dims(la, d, r):
    run(la, d=d, r=r, ctx=(333,), n=11, seed=d + r)


@pytest.mark.parametrize("keys", [True, False])
def test_bf16_ragged_batch_of_own_trees(la, keys):
    run(la, S=3, A=4, r=64, ctx=(401, 0, 130), n=13, per_agent=True, lens=(13, 1, 0, 7, 12),
        keys=keys, seed=3)


def test_bf16_own_lr_caches_and_token_major_strides(la):
    run(la, S=2, A=3, r=16, ctx=(259, 77), n=6, lr_agents=True, tok_major=True, seed=4)
    run(la, S=2, A=3, r=32, ctx=(259, 77), n=6, per_agent=True, lr_agents=True, seed=5)


def test_bf16_long_context_many_splits(la):
    run(la, A=1, kv=1, ctx=(6001,), n=9, seed=6)
    run(la, A=1, kv=1, ctx=(6001,), n=40, keys=False, seed=7)


@pytest.mark.parametrize("r", [16, 32, 64])
@pytest.mark.parametrize("n", [8, 32])
def test_bf16_repeats_are_identical(la, r, n):
    """The merge's up-projection takes the place of the key's one only once every
    read of that is over: thirty launches in a row give the same bits."""
    i = make(S=4, A=3, kv=2, g=3, r=r, ctx=(1450, 700, 1101, 481), n=n, per_agent=True, garbage=False, seed=r + n)
    args, tree, out, keep = launch(la, i)
    la.lora_attn_tree(args, tree)
    torch.cuda.synchronize()
    check(la, i, out, torch.bfloat16)
    first = out.clone()
    for _ in range(30):
        out.fill_(SENT)
        la.lora_attn_tree(args, tree)
        assert torch.equal(out, first)


@pytest.mark.parametrize("n", [13, 27])   # folded, and with two warps a row
def test_bf16_one_value_stage_many_tiles(la, n):
    """r = 64 leaves one V stage: a long unsplit run of tiles ends in a partial
    context tile and the drafted one, whose dead rows are cleared in that stage."""
    for seed in range(2):
        run(la, S=3, A=4, kv=8, r=64, ctx=(2999, 1777, 2421), n=n, per_agent=True, lens=(13, 9, 2, 7, 12), seed=seed)


def test_bf16_fp32_out(la):
    run(la, out_dtype=torch.float32, ctx=(300,), n=5, seed=8)


def test_growing_scores(la):
    """Later keys outweigh earlier ones by far: the running maximum moves in every tile."""
    for keys in (True, False):
        i = make(ctx=(900,), n=5, keys=keys, seed=9)
        ramp = torch.linspace(0.02, 6.0, i["k_base"].shape[2]).view(1, 1, -1, 1)
        i["k_base"] = torch.where(torch.isfinite(i["k_base"]), i["k_base"] * ramp, i["k_base"]).to(i["q"].dtype)
        args, tree, out, keep = launch(la, i)
        la.lora_attn_tree(args, tree)
        torch.cuda.synchronize()
        check(la, i, out, torch.bfloat16)


def test_chain_agrees_with_prefill_and_decode(la):
    """A chain is the prefill of its tokens, one node the decode of a token: the
    library's own paths, within their 1e-2 of the largest output."""
    i = make(ctx=(200,), n=9, extra=0, garbage=False, seed=10)
    i["parent"] = None
    args, tree, out, keep = launch(la, i, torch.float32)
    la.lora_attn_tree(args, tree)
    ref = torch.empty_like(out)
    d = keep[0]
    pre = la.make_args(d["k_base"], d["v_base"], d["lr"], d["B_k"], d["B_v"], d["q"], ref,
                       lora_scale=2.0, rope_base=i["base"], q_pos0=200)
    la.lora_attn_prefill(pre)
    torch.cuda.synchronize()
    assert (out - ref).abs().max() <= 1e-2 * ref.abs().max()


def test_bad_trees_are_reported(la):
    """Host-checked lengths and parents out of range: caught before any access."""
    for what, bit in (("parent", la.LA_DEV_TREE), ("self", la.LA_DEV_TREE), ("len", la.LA_DEV_TREE),
                      ("kv", la.LA_DEV_KV_LEN), ("kv_neg", la.LA_DEV_KV_LEN)):
        for dt in (torch.bfloat16, torch.float32):
            i = make(dtype=dt, S=2, ctx=(60, 50), n=4, lens=(4,), garbage=False, seed=11)
            if what == "parent":
                i["parent"][1, 0, 2] = -2
            elif what == "self":
                i["parent"][1, 0, 2] = 2
            elif what == "len":
                i["tree_len"][1, 0] = 5
            else:
                i["kv_len"][1] = i["max_kv_len"] - 3 if what == "kv" else -1
            args, tree, out, keep = launch(la, i, dt)
            la.lora_attn_tree(args, tree)
            st, word = la.la_device_check_word()
            assert (st, word) == (la.LA_ERR_DEVICE_CHECK, bit), (what, dt)
            assert (out[1] == SENT).all() and (out[0] != SENT).all()


def test_graph_stream_and_repeat(la):
    """Captured and replayed, on a stream of its own, with lengths, parents and
    queries that change between replays; repeated runs are bit-identical."""
    i = make(S=2, A=3, ctx=(500, 300), n=8, lens=(8, 5), garbage=False, seed=12)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        args, tree, out, keep = launch(la, i)
        la.lora_attn_tree(args, tree)
    s.synchronize()
    check(la, i, out, torch.bfloat16)
    first = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        la.lora_attn_tree(args, tree)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    i2 = make(S=2, A=3, ctx=(340, 499), n=8, lens=(3, 8), garbage=False, seed=13)
    i2["max_kv_len"] = i["max_kv_len"]
    d, _, par, tl = keep
    for k in ("k_base", "v_base", "lr"):
        L = min(d[k].shape[-2], i2[k].shape[-2])
        d[k][..., :L, :].copy_(i2[k][..., :L, :])
        i2[k] = d[k].cpu()
    for k in ("q", "kv_len", "B_k", "B_v"):
        d[k].copy_(i2[k])
    par.copy_(torch.from_numpy(i2["parent"]))
    tl.copy_(torch.from_numpy(i2["tree_len"]))
    out.fill_(SENT)
    g.replay()
    torch.cuda.synchronize()
    check(la, i2, out, torch.bfloat16)


def test_offsets_past_32_bits(la):
    """Rows beyond 2^31 elements of one cache: 17 sequences of 2^20 rows."""
    kv, d, r, L, S, n = 1, 128, 16, 1 << 20, 17, 2
    k = torch.zeros(S, kv, L, d, dtype=torch.bfloat16, device=DEV)
    i = make(S=S, A=1, kv=kv, g=1, ctx=(150,), n=n, garbage=False, extra=0, seed=14)
    v, lr = torch.zeros_like(k), torch.zeros(S, L, 2 * r, dtype=torch.bfloat16, device=DEV)
    for big, x in ((k, i["k_base"]), (v, i["v_base"])):
        big[:, :, :x.shape[2]] = x.to(DEV)
    lr[:, :i["lr"].shape[1]] = i["lr"].to(DEV)
    dd = {x: i[x].to(DEV) for x in ("B_k", "B_v", "q", "kv_len")}
    out = torch.full(i["q"].shape, SENT, dtype=torch.bfloat16, device=DEV)
    args = la.make_args(k, v, lr, dd["B_k"], dd["B_v"], dd["q"], out, lora_scale=2.0,
                        rope_base=i["base"], kv_len=dd["kv_len"], max_kv_len=i["max_kv_len"])
    par = torch.from_numpy(i["parent"]).to(DEV)
    la.lora_attn_tree(args, la.make_tree_args(par))
    torch.cuda.synchronize()
    check(la, i, out, torch.bfloat16)


def test_wide_group_own_lr_without_key_delta_and_chains_of_every_agent(la):
    run(la, S=1, A=1, kv=1, g=64, ctx=(150,), n=3, seed=15)                          # 192 rows: two blocks
    run(la, S=1, A=1, kv=1, g=64, d=64, ctx=(20,), n=64, keys=False, seed=16)        # 32 blocks
    run(la, S=2, A=3, ctx=(259, 77), n=6, lr_agents=True, keys=False, seed=17)
    run(la, S=1, A=2, r=8, ctx=(140,), n=20, per_agent=True, lr_agents=True, keys=False, d=64, seed=18)
    run(la, dtype=torch.float32, out_dtype=torch.bfloat16, ctx=(130,), n=5, seed=19)
    for dt in (torch.bfloat16, torch.float32):   # neither parents nor lengths: a chain an agent
        i = make(dtype=dt, A=3, ctx=(201,), n=7, per_agent=True, garbage=False, seed=20)
        i["parent"] = None
        args, tree, out, keep = launch(la, i, dt)
        la.lora_attn_tree(args, tree)
        torch.cuda.synchronize()
        check(la, i, out, dt)


def test_two_streams_at_once(la):
    """Nothing is shared between calls: two of different shapes in flight together."""
    cases = [make(S=2, A=3, ctx=(1500, 900), n=8, garbage=False, seed=21),
             make(S=1, A=2, r=32, ctx=(2100,), n=40, per_agent=True, garbage=False, seed=22)]
    runs = [(torch.cuda.Stream(), *launch(la, i)) for i in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, args, tree, out, keep in runs:
            with torch.cuda.stream(s):
                la.lora_attn_tree(args, tree)
    torch.cuda.synchronize()
    for i, (s, args, tree, out, keep) in zip(cases, runs):
        check(la, i, out, torch.bfloat16)


FIRST_IN_CAPTURE = """
import torch
from tests import test_tree_gpu as T
from rank_attention_b200 import lora_attn as la
i = T.make(ctx=(300,), n=5, garbage=False, seed=23)
args, tree, out, keep = T.launch(la, i)
x, y = torch.randn(40, 128, device="cuda").bfloat16(), torch.randn(40, 64, device="cuda").bfloat16()
A, B = torch.randn(128, 16, device="cuda").bfloat16(), torch.randn(2, 16, 64, device="cuda").bfloat16()
o = torch.zeros_like(y)
ss, sa = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 9, 40], [1, 0]))
ga = la.make_grouped_args(x, A, B, y, o, ss, sa, lora_scale=1.0)
q = torch.randn(1, 2, 5, 8, 128, device="cuda").bfloat16()
qo, kl = torch.zeros_like(q), torch.tensor([7], dtype=torch.int32, device="cuda")
qa = la.make_qk_args(q, None, None, None, None, qo, None, None, kl, rope_base=1e4, max_kv_len=20)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    la.lora_attn_tree(args, tree)
    la.lora_grouped_delta(ga)
    la.lora_qk_norm_rope(qa)
g.replay()
torch.cuda.synchronize()
T.check(la, i, out, torch.bfloat16)
assert (o != 0).any() and (qo != 0).any() and la.la_device_check() == 0
print("captured")
"""


def test_first_call_of_a_process_may_be_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_IN_CAPTURE], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
