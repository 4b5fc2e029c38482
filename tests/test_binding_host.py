"""The Python binding's argument structs, on the CPU: tensors stand in for CUDA
ones (the device check is replaced), nothing is launched."""
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
