"""lora_grouped_delta against the fp64 oracle.

|out - ref| <= uo |ref| + s (|x||A||B|) u: uo the output type's half step; u =
(hidden + r + 8) 2^-24 for fp32 sums, plus 2^-16 where the tensor cores take
x A as two bf16 terms (each 2^-8: the second of the first's remainder)."""
import numpy as np
import pytest
import torch

from oracle import impl as O
from tests.helpers import to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"
SENT = -77.0


@pytest.fixture(scope="module")
def la():
    from rank_attention_b200 import lora_attn
    return lora_attn


def run(la, start, agent, dtype=torch.bfloat16, H=256, N=256, r=16, A=3, T=None, shared=False,
        inplace=False, pad=0, zero_y=False, seed=0):
    gen = torch.Generator().manual_seed(seed)
    T = (start[-1] + 5) if T is None else T   # rows behind the last segment
    f = lambda *sh, std=1.0: (torch.randn(*sh, generator=gen) * std).to(dtype)  # noqa: E731
    x, y = f(T, H + pad), f(T, N + pad)
    Am, B = f(*((H, r) if shared else (A, H, r)), std=0.05), f(A, r, N, std=0.05)
    if zero_y:
        y.zero_()
    xd, yd, Ad, Bd = x.to(DEV), y.to(DEV), Am.to(DEV), B.to(DEV)
    xv, yv = xd[:, :H], yd[:, :N]
    out = yv if inplace else torch.full((T, N + pad), SENT, dtype=dtype, device=DEV)[:, :N]
    ss = torch.tensor(start, dtype=torch.int32, device=DEV)
    sa = torch.tensor(agent, dtype=torch.int32, device=DEV)
    la.lora_grouped_delta(la.make_grouped_args(xv, Ad, Bd, yv, out, ss, sa, lora_scale=2.0))
    torch.cuda.synchronize()
    assert la.la_device_check() == la.LA_OK
    xn, yn = to_np(x[:, :H]), to_np(y[:, :N])
    ref = O.grouped_delta(xn, Am, B, yn, start, agent, 2.0)
    mag = O.grouped_delta(np.abs(xn), np.abs(to_np(Am)), np.abs(to_np(B)), 0 * yn, start, agent, 2.0)
    bf = dtype == torch.bfloat16
    tol = (2.0 ** -8 if bf else 2.0 ** -24) * np.abs(ref) + \
        mag * ((H + r + 8) * 2.0 ** -24 + (2.0 ** -16 if bf else 0)) + 2.0 ** -24 * np.abs(yn)
    got = to_np(out)
    lo, hi = start[0], start[-1]
    err = np.abs(got[lo:hi] - ref[lo:hi])
    assert np.isfinite(got[lo:hi]).all() and (err <= tol[lo:hi]).all(), (err / np.maximum(tol[lo:hi], 1e-30)).max()
    rest = np.r_[0:lo, hi:T]
    assert (got[rest] == (yn[rest] if inplace else SENT)).all(), "a row in no segment was written"
    if pad and inplace:
        assert torch.equal(yd[:, N:].cpu(), y[:, N:])


CASES = [
    dict(start=[0, 1], agent=[0], A=1),
    dict(start=[0, 16, 32, 48], agent=[0, 1, 2]),
    dict(start=[3, 3, 20, 20, 151, 152], agent=[2, 0, 1, -1, 0]),      # empty ones, one agent twice
    dict(start=[0, 127, 255, 384, 640], agent=[1, -1, 2, 0]),
    dict(start=[0, 129, 130], agent=[-1, 1]),
    dict(start=[5, 5], agent=[0]),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("r", [8, 16, 32, 64])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_segments(la, dtype, r, case):
    run(la, dtype=dtype, r=r, seed=case, **CASES[case])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,N", [(8, 8), (64, 4096), (4096, 64), (72, 1000), (1000, 72), (2056, 264), (4096, 4096)])
def test_sizes(la, dtype, H, N):
    run(la, [0, 30, 77], [1, 0], dtype=dtype, H=H, N=N, r=16, seed=H + N)
    run(la, [0, 30, 177], [1, 0], dtype=dtype, H=H, N=N, r=64, seed=H + N)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_shared_inplace_strided_and_zero_y(la, dtype):
    c = dict(start=[2, 40, 40, 300], agent=[0, 2, 1], dtype=dtype)
    run(la, shared=True, **c)
    run(la, inplace=True, **c)
    run(la, pad=24, **c)
    run(la, pad=8, inplace=True, shared=True, **c)
    run(la, zero_y=True, r=64, **c)


def test_many_segments(la):
    """More segments than a warp has lanes, most of them short or empty."""
    rng = np.random.default_rng(1)
    start = np.concatenate([[0], np.cumsum(rng.integers(0, 5, 300))]).tolist()
    agent = rng.integers(-1, 7, 300).tolist()
    run(la, start, agent, A=7, H=128, N=136, r=16)
    run(la, start, agent, A=7, H=128, N=136, r=32, dtype=torch.float32)


def test_infinities_stay_in_their_rows(la):
    """A token's infinities and NaN reach its own row only."""
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.randn(40, 128, device=DEV).to(dtype)
        x[3, 5], x[20, 7] = float("inf"), float("nan")
        A = torch.randn(2, 128, 16, device=DEV).to(dtype)
        B = torch.randn(2, 16, 128, device=DEV).to(dtype)
        y = torch.randn(40, 128, device=DEV).to(dtype)
        out = torch.empty_like(y)
        ss = torch.tensor([0, 18, 40], dtype=torch.int32, device=DEV)
        sa = torch.tensor([1, 0], dtype=torch.int32, device=DEV)
        la.lora_grouped_delta(la.make_grouped_args(x, A, B, y, out, ss, sa, lora_scale=1.0))
        bad = ~torch.isfinite(out).all(1)
        assert bad.nonzero().flatten().tolist() == [3, 20]


def test_bad_segments_are_reported(la):
    x = torch.randn(40, 128, device=DEV).to(torch.bfloat16)
    A = torch.randn(2, 128, 16, device=DEV).to(torch.bfloat16)
    B = torch.randn(2, 16, 128, device=DEV).to(torch.bfloat16)
    for start, agent in (([0, 41], [0]), ([-1, 4], [0]), ([0, 9, 8], [0, 1]), ([0, 4], [2]), ([0, 4], [-2])):
        for dt in (torch.bfloat16, torch.float32):
            out = torch.full((40, 128), SENT, device=DEV, dtype=dt)
            ss = torch.tensor(start, dtype=torch.int32, device=DEV)
            sa = torch.tensor(agent, dtype=torch.int32, device=DEV)
            la.lora_grouped_delta(la.make_grouped_args(x.to(dt), A.to(dt), B.to(dt), out.clone(), out, ss, sa,
                                                       lora_scale=1.0))
            assert la.la_device_check_word() == (la.LA_ERR_DEVICE_CHECK, la.LA_DEV_SEGMENT)
            assert (out == SENT).all()


def test_graph_with_changing_segments(la):
    """One captured call serves other cuts of the same tokens; repeats are bit-identical."""
    T, H, N, r = 300, 512, 384, 32
    gen = torch.Generator().manual_seed(3)
    x, y = torch.randn(T, H, generator=gen).to(torch.bfloat16), torch.randn(T, N, generator=gen).to(torch.bfloat16)
    A, B = (0.05 * torch.randn(2, H, r, generator=gen)).to(torch.bfloat16), (0.05 * torch.randn(2, r, N, generator=gen)).to(torch.bfloat16)
    xd, yd, Ad, Bd = (t.to(DEV) for t in (x, y, A, B))
    out = torch.zeros(T, N, dtype=torch.bfloat16, device=DEV)
    ss = torch.tensor([0, 100, 300], dtype=torch.int32, device=DEV)
    sa = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    args = la.make_grouped_args(xd, Ad, Bd, yd, out, ss, sa, lora_scale=2.0)
    la.lora_grouped_delta(args)
    first = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        la.lora_grouped_delta(args)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, out)
    for start, agent in (([0, 300, 300], [1, 0]), ([0, 1, 299], [-1, 0])):
        ss.copy_(torch.tensor(start, dtype=torch.int32))
        sa.copy_(torch.tensor(agent, dtype=torch.int32))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        ref = O.grouped_delta(x, A, B, y, start, agent, 2.0)
        ref[start[-1]:] = 0
        assert np.abs(to_np(out) - ref).max() <= 2.0 ** -8 * np.abs(ref).max() + 1e-3


def test_two_streams_at_once_and_one_agent_expanded(la):
    gen = torch.Generator().manual_seed(5)
    f = lambda *s, std=1.0: (torch.randn(*s, generator=gen) * std).to(torch.bfloat16).to(DEV)  # noqa: E731
    runs = []
    for T, H, N, r, start, agent in ((700, 512, 256, 32, [0, 300, 700], [0, 1]), (90, 1024, 512, 16, [0, 1, 90], [1, 0])):
        x, y, A, B = f(T, H), f(T, N), f(H, r, std=0.05), f(2, r, N, std=0.05)
        out = torch.zeros_like(y)
        ss, sa = (torch.tensor(v, dtype=torch.int32, device=DEV) for v in (start, agent))
        args = la.make_grouped_args(x, A.expand(2, H, r), B, y, out, ss, sa, lora_scale=2.0)   # stride 0: one A
        runs.append((torch.cuda.Stream(), args, (x, A, B, y, start, agent), out, (ss, sa)))
    torch.cuda.synchronize()
    for _ in range(10):
        for s, args, *_rest in runs:
            with torch.cuda.stream(s):
                la.lora_grouped_delta(args)
    torch.cuda.synchronize()
    for s, args, (x, A, B, y, start, agent), out, keep in runs:
        ref = O.grouped_delta(x.cpu(), A.cpu(), B.cpu(), to_np(y), start, agent, 2.0)
        mag = O.grouped_delta(x.abs().cpu(), A.abs().cpu(), B.abs().cpu(), 0 * to_np(y), start, agent, 2.0)
        tol = 2.0 ** -8 * np.abs(ref) + mag * ((x.shape[1] + B.shape[1] + 8) * 2.0 ** -24 + 2.0 ** -16) + \
            2.0 ** -24 * np.abs(to_np(y))
        assert (np.abs(to_np(out) - ref) <= tol).all()
