"""More refusals of the drafted-tree operators, before any launch: every call carries
at least one invalid argument (no GPU needed; the addresses are never dereferenced)."""
import ctypes

import pytest

from rank_attention_b200 import lora_attn as la
from tests.test_tree_host import BAD, FAKE, UNS, grouped, qk

OTHER = FAKE + 0x10000


def norm(**kw):
    """The status of a call with 4 query heads of 64, 2 agents, 4 tokens and 2 sequences
    whose max_kv_len lies beyond L_max: strides that pass end there, nothing launches."""
    return la.lib.lora_qk_norm_rope(ctypes.byref(qk(max_kv_len=257, **kw)), None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q_out=FAKE), la.LA_ERR_CAPACITY),                                  # dense
    (dict(q_out=FAKE, q_tok_stride=512, q_agent_stride=2048, q_seq_stride=4096), BAD),   # a fused projection's slice
    (dict(q_out=FAKE, q_agent_stride=2048, q_seq_stride=4096), BAD),
    (dict(q_out=FAKE, q_seq_stride=4096), BAD),
    (dict(q_out=FAKE, q_agent_stride=0), BAD),
    # a stride whose extent is one is not used
    (dict(q_out=FAKE, n_seqs=1, q_seq_stride=4096), la.LA_ERR_CAPACITY),
    (dict(q_out=FAKE, n_agents=1, q_agent_stride=4096, q_seq_stride=1024), la.LA_ERR_CAPACITY),
    (dict(q_out=FAKE, n_tokens=1, q_tok_stride=512, q_agent_stride=256, q_seq_stride=512), la.LA_ERR_CAPACITY),
    # another buffer: strides as before
    (dict(q_out=OTHER, q_tok_stride=512, q_agent_stride=2048, q_seq_stride=4096), la.LA_ERR_CAPACITY),
])
def test_queries_in_place_must_be_dense(kw, status):
    """q_out is written densely: over a strided q, a head's row would land on rows that
    another block has yet to read, or on its neighbours' columns."""
    assert norm(**kw) == status


@pytest.mark.parametrize("kw", [
    dict(n_tokens=(1 << 31) - 1, dtype=la.LA_BF16), dict(n_tokens=(1 << 31) - 1, dtype=la.LA_F32),
    dict(n_tokens=(1 << 31) - 1, n_segs=(1 << 31) - 1),
    # one tile more than the grid holds: 128 rows a tile in bf16, 64 in fp32 (16 where segments are short)
    dict(n_tokens=65533 * 128 + 1, dtype=la.LA_BF16), dict(n_tokens=65533 * 64 + 1, dtype=la.LA_F32),
    dict(n_tokens=16 * 32768 + 1, n_segs=32767, dtype=la.LA_F32),
])
def test_grouped_refuses_more_tiles_than_the_grid_holds(kw):
    assert la.lib.lora_grouped_delta(ctypes.byref(grouped(**kw)), None) == UNS


@pytest.mark.parametrize("kw", [dict(x=FAKE), dict(A=FAKE), dict(B=FAKE)])
def test_grouped_refuses_out_over_an_input(kw):
    """Only y may be out: the others are still read when the first columns are written."""
    base = dict(x=OTHER, A=OTHER, B=OTHER, y=OTHER, out=FAKE)
    assert la.lib.lora_grouped_delta(ctypes.byref(grouped(**{**base, **kw})), None) == BAD
