"""Refusals of the drafted-tree entry points, before any launch: every call
carries at least one invalid argument or nothing to do (no GPU needed)."""
import ctypes
import os
import subprocess

import pytest
import torch

from rank_attention_b200 import lora_attn as la

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000   # 16-byte aligned, never dereferenced
BAD, UNS, CAP = la.LA_ERR_INVALID_ARG, la.LA_ERR_UNSUPPORTED, la.LA_ERR_CAPACITY


@pytest.mark.parametrize("cname,cls", [("la_tree_args", la.TreeArgs), ("la_qk_args", la.QkArgs),
                                       ("la_grouped_args", la.GroupedArgs)])
def test_struct_layouts_match_the_header(tmp_path, cname, cls):
    fields = [f[0] for f in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "lora_attn.h"\nint main(void){' +
                   "\n".join(f'printf("{f} %zu\\n", offsetof({cname}, {f}));' for f in fields) +
                   f'printf("sizeof %zu\\n", sizeof({cname})); return 0;}}\n')
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = dict(l.split() for l in subprocess.run([str(exe)], capture_output=True, text=True,
                                                 check=True).stdout.splitlines())
    for f in fields:
        assert int(got[f]) == getattr(cls, f).offset, f
    assert int(got["sizeof"]) == ctypes.sizeof(cls)


def attn(**kw):
    a = la.AttnArgs()
    a.n_seqs, a.n_agents, a.n_q_heads, a.n_kv_heads, a.head_dim, a.r = 1, 2, 4, 2, 64, 8
    a.lora_scale, a.softmax_scale, a.rope_base, a.L_max = 2.0, 0.125, 10000.0, 256
    a.k_base = a.v_base = a.lr_cache = a.B_k = a.B_v = a.q = a.out = a.kv_len = FAKE
    a.kv_seq_stride, a.kv_head_stride, a.kv_tok_stride = 2 * 256 * 64, 256 * 64, 64
    a.lr_seq_stride, a.max_kv_len, a.n_q_tokens = 256 * 16, 256, 4
    a.io_dtype = a.out_dtype = la.LA_F32
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def tree(**kw):
    t = la.TreeArgs()
    t.parent, t.tree_len, t.n_trees = FAKE, FAKE, 1
    for k, v in kw.items():
        setattr(t, k, v)
    return t


@pytest.mark.parametrize("akw,tkw,status", [
    (dict(head_dim=96), {}, UNS), (dict(r=24), {}, UNS), (dict(n_q_heads=5), {}, BAD),
    (dict(n_q_heads=130, n_kv_heads=2), {}, UNS), (dict(k_base=0), {}, BAD), (dict(B_v=0), {}, BAD),
    (dict(q=FAKE + 8), {}, BAD), (dict(kv_tok_stride=32), {}, BAD), (dict(kv_len=0), {}, BAD),
    (dict(kv_len=FAKE + 2), {}, BAD), (dict(max_kv_len=0), {}, BAD), (dict(max_kv_len=257), {}, CAP),
    (dict(n_q_tokens=0), {}, BAD), (dict(n_q_tokens=65), {}, BAD), (dict(value_path=2), {}, UNS),
    (dict(value_path=9), {}, BAD), (dict(key_pos0=4), {}, UNS), (dict(row_stats=FAKE), {}, UNS),
    (dict(softmax_scale=0.0), {}, BAD), (dict(io_dtype=4), {}, BAD),
    ({}, dict(n_trees=0), BAD), ({}, dict(n_trees=3), BAD), ({}, dict(parent=FAKE + 1), BAD),
    ({}, dict(tree_len=FAKE + 2), BAD), (dict(max_kv_len=3), {}, CAP),
    (dict(max_kv_len=7), dict(n_trees=2), CAP),
])
def test_tree_attention_refuses(akw, tkw, status):
    assert la.lib.lora_attn_tree(ctypes.byref(attn(**akw)), ctypes.byref(tree(**tkw)), None) == status


def test_tree_attention_null_structs_and_empty_batch():
    assert la.lib.lora_attn_tree(None, ctypes.byref(tree()), None) == BAD
    assert la.lib.lora_attn_tree(ctypes.byref(attn()), None, None) == BAD
    assert la.lib.lora_attn_tree(ctypes.byref(attn(n_seqs=0)), ctypes.byref(tree()), None) == la.LA_OK


def test_other_paths_still_need_B_k():
    a = attn(B_k=0, q_pos0=0)
    assert la.lib.lora_attn_prefill(ctypes.byref(a), None) == BAD
    a.n_q_tokens = 1
    assert la.lib.lora_attn_decode(ctypes.byref(a), FAKE, 1 << 20, None) == BAD


def qk(**kw):
    a = la.QkArgs()
    a.n_seqs, a.n_agents, a.n_tokens, a.n_q_heads, a.n_kv_heads, a.head_dim = 2, 2, 4, 4, 2, 64
    a.eps, a.rope_base = 1e-6, 10000.0
    a.q = a.q_out = a.k = a.v = a.w_q = a.w_k = a.k_base = a.v_base = a.kv_len = FAKE
    a.q_tok_stride, a.q_agent_stride, a.q_seq_stride = 256, 1024, 2048
    a.kv_in_tok_stride, a.kv_in_tree_stride, a.kv_in_seq_stride = 128, 512, 512
    a.L_max, a.kv_seq_stride, a.kv_head_stride, a.kv_tok_stride = 256, 2 * 256 * 64, 256 * 64, 64
    a.max_kv_len, a.dtype = 256, la.LA_BF16
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("akw,tkw,status", [
    (dict(head_dim=32), {}, UNS), (dict(dtype=2), {}, BAD), (dict(n_agents=0), {}, BAD),
    (dict(eps=-1.0), {}, BAD), (dict(eps=float("nan")), {}, BAD), (dict(rope_base=1.0), {}, BAD),
    (dict(q=0), {}, BAD), (dict(q_out=0), {}, BAD), (dict(k=0), {}, BAD), (dict(k_base=0), {}, BAD),
    (dict(v_base=0), {}, BAD), (dict(q=FAKE + 2), {}, BAD), (dict(w_k=FAKE + 2), {}, BAD),
    (dict(q_tok_stride=255), {}, BAD), (dict(q_tok_stride=248), {}, BAD), (dict(kv_in_tok_stride=64), {}, BAD),
    (dict(kv_tok_stride=60), {}, BAD), (dict(kv_len=0), {}, BAD), (dict(max_kv_len=257), {}, CAP),
    (dict(max_kv_len=3), {}, CAP), (dict(n_tokens=65), {}, UNS), ({}, dict(n_trees=3), BAD),
    ({}, dict(parent=FAKE + 2), BAD), (dict(q=0, q_out=0, k=0, k_base=0, v=0, v_base=0), {}, BAD),
    (dict(k=0, k_base=0), {}, BAD),
])
def test_norm_refuses(akw, tkw, status):
    assert la.lib.lora_qk_norm_rope(ctypes.byref(qk(**akw)), ctypes.byref(tree(**tkw)), None) == status


def test_norm_with_nothing_to_do():
    for kw in (dict(n_seqs=0), dict(n_tokens=0)):
        assert la.lib.lora_qk_norm_rope(ctypes.byref(qk(**kw)), None, None) == la.LA_OK
    assert la.lib.lora_qk_norm_rope(None, None, None) == BAD


def grouped(**kw):
    a = la.GroupedArgs()
    a.n_tokens, a.hidden, a.n_out, a.r, a.n_agents, a.n_segs = 10, 64, 64, 16, 2, 2
    a.lora_scale = 1.0
    a.x = a.A = a.B = a.y = a.out = a.seg_start = a.seg_agent = FAKE
    a.ldx = a.ldy = a.ldo = 64
    a.a_agent_stride, a.dtype = 64 * 16, la.LA_BF16
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=5), BAD), (dict(hidden=0), BAD), (dict(hidden=12), BAD), (dict(n_out=4), BAD),
    (dict(r=24), UNS), (dict(n_agents=0), BAD), (dict(n_segs=-1), BAD), (dict(lora_scale=float("inf")), BAD),
    (dict(x=0), BAD), (dict(B=0), BAD), (dict(seg_start=0), BAD), (dict(seg_agent=FAKE + 2), BAD),
    (dict(y=FAKE + 8), BAD), (dict(ldx=56), BAD), (dict(ldy=68), BAD), (dict(ldo=72), BAD),
    (dict(a_agent_stride=1016), BAD), (dict(n_tokens=1 << 20, n_segs=1 << 16), UNS),
])
def test_grouped_refuses(kw, status):
    assert la.lib.lora_grouped_delta(ctypes.byref(grouped(**kw)), None) == status


def test_grouped_with_nothing_to_do():
    for kw in (dict(n_tokens=0), dict(n_segs=0)):
        assert la.lib.lora_grouped_delta(ctypes.byref(grouped(**kw)), None) == la.LA_OK
    assert la.lib.lora_grouped_delta(None, None) == BAD


def test_binding_refuses():
    i32 = torch.int32
    p = torch.zeros(1, 1, 3, dtype=i32)
    with pytest.raises(ValueError):
        la.make_tree_args(p.long())
    with pytest.raises(ValueError):
        la.make_tree_args(p, torch.zeros(1, 2, dtype=i32))
    with pytest.raises(ValueError):
        la.make_tree_args(p)                       # not on a CUDA device
    q, k = torch.zeros(1, 2, 3, 4, 64), torch.zeros(1, 1, 3, 2, 64)
    kb, kl = torch.zeros(1, 2, 8, 64), torch.zeros(1, dtype=i32)
    kw = dict(rope_base=1e4, max_kv_len=8)
    for bad in ((None, None, None, None, None, None, None, None, kl),
                (q, k, None, None, None, None, kb, None, kl),
                (q, k, None, None, None, q[..., :32], kb, None, kl),
                (q.transpose(3, 4), k, None, None, None, q, kb, None, kl),
                (q, k, None, torch.zeros(32), None, q, kb, None, kl),
                (q, k, None, None, None, q, kb[:, :1], None, kl),
                (q, k, k, None, None, q, kb, kb[:, :, :4], kl),
                (q, k, None, None, None, q, kb, None, kl.long()),
                (q, k, None, None, None, q, kb, None, kl)):     # not on a CUDA device
        with pytest.raises(ValueError):
            la.make_qk_args(*bad, **kw)
    with pytest.raises(TypeError):
        la.make_qk_args(q, k.double(), None, None, None, q, kb, None, kl, **kw)
    x, y, A, B = torch.zeros(5, 16), torch.zeros(5, 8), torch.zeros(16, 8), torch.zeros(2, 8, 8)
    ss, sa = torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32)
    for bad in ((x, A, B, y[:4], y, ss, sa), (x, A.T, B, y, y, ss, sa), (x, A, B, y, y, ss[:2], sa),
                (x, A, B, y, y, ss.long(), sa), (x.T.contiguous().T, A, B, y, y, ss, sa),
                (x, A, B, y, y, ss, sa)):                       # not on a CUDA device
        with pytest.raises(ValueError):
            la.make_grouped_args(*bad, lora_scale=1.0)
    with pytest.raises(TypeError):
        la.make_grouped_args(x, A.double(), B, y, y, ss, sa, lora_scale=1.0)
