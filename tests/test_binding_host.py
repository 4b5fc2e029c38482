"""The Python binding's argument structs, on the CPU: tensors stand in for CUDA
ones (the device check is replaced), nothing is launched."""
import ctypes
import gc
import weakref

import pytest
import torch

from rank_attention_b200 import lora_attn as la

I32 = torch.int32


@pytest.fixture
def any_device(monkeypatch):
    monkeypatch.setattr(la, "_same_device", lambda ts: 0)


def _structs():
    """name -> (function of fresh tensors, those tensors' makers)."""
    z = torch.zeros
    S, A, n, kv, hq, d, r, L = 1, 2, 3, 2, 4, 64, 8, 16
    return {
        "tree": (lambda p, t: la.make_tree_args(p, t), [z(S, 1, n, dtype=I32), z(S, 1, dtype=I32)]),
        "qk": (lambda *t: la.make_qk_args(*t, rope_base=1e4, max_kv_len=L),
               [z(S, A, n, hq, d), z(S, 1, n, kv, d), z(S, 1, n, kv, d), z(d), z(d), z(S, A, n, hq, d),
                z(S, kv, L, d), z(S, kv, L, d), z(S, dtype=I32)]),
        "grouped": (lambda *t: la.make_grouped_args(*t, lora_scale=1.0),
                    [z(5, 16), z(A, 16, r), z(A, r, 8), z(5, 8), z(5, 8), z(3, dtype=I32), z(2, dtype=I32)]),
        "attn": (lambda kl, *t: la.make_args(*t, lora_scale=1.0, rope_base=1e4, kv_len=kl, max_kv_len=L),
                 [z(S, dtype=I32), z(S, kv, L, d), z(S, kv, L, d), z(S, L, 2 * r), z(A, r, kv * d),
                  z(A, r, kv * d), z(S, A, n, hq, d), z(S, A, n, hq, d)]),
    }


@pytest.mark.parametrize("name", ["tree", "qk", "grouped", "attn"])
def test_structs_keep_their_tensors(any_device, name):
    """A struct holds addresses, so a tensor made in the call that fills it must live
    as long as the struct: freed, its memory is handed out again before the launch."""
    make, tensors = _structs()[name]
    refs = [weakref.ref(t) for t in tensors]
    args = make(*tensors)
    del tensors
    gc.collect()
    assert all(x() is not None for x in refs)
    del args
    gc.collect()
    assert all(x() is None for x in refs)


def odd(t, dim):
    """t with a meaningless stride in a dimension of one entry (as views of slices have)."""
    st = list(t.stride())
    assert t.shape[dim] == 1
    st[dim] = 7
    return t.as_strided(t.shape, st)


def status(fn, args, *rest):
    return getattr(la.lib, fn)(ctypes.byref(args), *rest)


def test_strides_of_single_entries_are_not_looked_at(any_device):
    """A stride of a dimension of one entry is never used, so it refuses nothing: the call
    gets as far as a max_kv_len beyond L_max (nothing launches)."""
    z = torch.zeros
    kl = z(1, dtype=I32)
    q, k, kb = z(1, 1, 1, 4, 64), z(1, 1, 1, 2, 64), z(1, 2, 16, 64)
    for dim in range(3):
        for t in (odd(q, dim),):
            a = la.make_qk_args(t, k, k.clone(), None, None, z(1, 1, 1, 4, 64), kb, kb.clone(), kl, rope_base=1e4, max_kv_len=17)
            assert status("lora_qk_norm_rope", a, None, None) == la.LA_ERR_CAPACITY
        for kk, vv in ((odd(k, dim), odd(k, dim)), (k, odd(k, dim)), (odd(k, dim), k)):
            a = la.make_qk_args(q, kk, vv, None, None, z(1, 1, 1, 4, 64), kb, kb.clone(), kl, rope_base=1e4, max_kv_len=17)
            assert status("lora_qk_norm_rope", a, None, None) == la.LA_ERR_CAPACITY
    for kc, vc in ((odd(kb, 0), kb.clone()), (kb, odd(kb, 0)), (odd(z(1, 1, 16, 64), 1), z(1, 1, 16, 64))):
        a = la.make_qk_args(q, k[:, :, :, :kc.shape[1]], k[:, :, :, :kc.shape[1]].clone(), None, None,
                            z(1, 1, 1, 4, 64), kc, vc, kl, rope_base=1e4, max_kv_len=17)
        assert status("lora_qk_norm_rope", a, None, None) == la.LA_ERR_CAPACITY
    x, A, B, y = z(5, 16), z(1, 16, 8), z(1, 8, 8), z(5, 8)
    a = la.make_grouped_args(x, odd(A, 0), B, y, y, z(2, dtype=I32), z(1, dtype=I32), lora_scale=1.0)
    assert a.a_agent_stride == 0   # one agent, one A


def test_strides_of_several_entries_count(any_device):
    z = torch.zeros
    q, kb, kl = z(2, 1, 1, 4, 64), z(2, 2, 16, 64), z(2, dtype=I32)
    k = z(2, 1, 1, 2, 64)
    with pytest.raises(ValueError):
        la.make_qk_args(q, k, z(2, 2, 1, 2, 64)[:, :1], None, None, z(2, 1, 1, 4, 64), kb, kb.clone(), kl,
                        rope_base=1e4, max_kv_len=16)


@pytest.mark.parametrize("change,error", [
    (dict(), None),
    (dict(q=torch.bfloat16), TypeError), (dict(lr=torch.bfloat16), TypeError), (dict(B_v=torch.bfloat16), TypeError),
    (dict(v_base=torch.bfloat16), TypeError), (dict(B_k=torch.bfloat16), TypeError),
    (dict(kv_len=torch.int64), ValueError), (dict(kv_len=(0,)), ValueError), (dict(kv_len=None), ValueError),
    (dict(q=(1, 2, 3, 4, 32)), ValueError), (dict(q=(2, 2, 3, 4, 64)), ValueError), (dict(out=(1, 2, 2, 4, 64)), ValueError),
    (dict(lr=(1, 15, 16)), ValueError), (dict(B_v=(2, 8, 64)), ValueError), (dict(B_k=(1, 8, 128)), ValueError),
])
def test_tree_attention_looks_at_its_tensors(monkeypatch, change, error):
    """make_args' struct shows neither types nor shapes: a float32 call's bfloat16 queries, or
    lengths in 64 bits, would be read as what they are not, past their end."""
    shapes = dict(k_base=(1, 2, 16, 64), v_base=(1, 2, 16, 64), lr=(1, 16, 16), B_k=(2, 8, 128), B_v=(2, 8, 128),
                  q=(1, 2, 3, 4, 64), out=(1, 2, 3, 4, 64))
    t = {k: torch.zeros(change[k] if isinstance(change.get(k), tuple) else s,
                        dtype=change[k] if isinstance(change.get(k), torch.dtype) else torch.float32)
         for k, s in shapes.items()}
    c = change.get("kv_len", I32)
    kl = None if c is None else torch.zeros(c if isinstance(c, tuple) else 1, dtype=c if isinstance(c, torch.dtype) else I32)
    args = la.make_args(**t, lora_scale=1.0, rope_base=1e4, kv_len=kl, max_kv_len=17)   # beyond L_max: nothing launches
    with pytest.raises(ValueError if error is None else error):
        la.lora_attn_tree(args, la.make_tree_args(None))    # not on a CUDA device, or the change
    if error is None:
        monkeypatch.setattr(la, "_same_device", lambda ts: 0)
        with pytest.raises(la.LoraAttnError) as e:
            la.lora_attn_tree(args, la.make_tree_args(None), stream=0)
        assert e.value.status == la.LA_ERR_CAPACITY
