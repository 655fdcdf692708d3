"""A step that is short of blocks: a request that got none is released by the
tokens it holds, and every block comes back. On the GPU the README's example is
run as it stands."""

import os
import re

import numpy as np
import pytest

import oracle
from table_cases import pool_state

torch = pytest.importorskip("torch")

B, HQ, HKV, D = 16, 4, 2, 64


def short_step():
    """Four requests; the queue covers the first, and the last two (of whom one
    needs no block)."""
    c, n = np.array([0, 50, 33, 17]), np.array([20, 40, 1, 2])
    table, ref, queue, state = pool_state(c, c + n, B, spare=0, seed=1)
    state = np.array([state[0], 2], np.int32)  # the rest of the ring is held elsewhere
    return c, n, table, ref, queue, state


def test_release_by_seq_lens_leaks_and_by_the_held_tokens_does_not():
    c, n, table, ref, queue, state = short_step()
    out = oracle.build_step_tables(table, c, n, queue, state, ref, B)
    assert out["denied"].tolist() == [False, True, False, False]
    assert out["seq_lens"].tolist() == [20, 0, 34, 19]
    for held, left in ((out["seq_lens"], 4), (np.where(out["seq_lens"] > 0, out["seq_lens"], c), 0)):
        back = oracle.release_blocks(out["block_table"], range(4), held, queue, out["free_state"],
                                     out["ref_cnt"], B)
        assert (back["ref_cnt"] > 0).sum() == left  # ceil(50 / 16)


def example():
    """The README's block with the step's tables made on the GPU."""
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md"),
              encoding="utf-8") as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    found = [b for b in blocks if "pkv_release_blocks" in b]
    assert len(found) == 1
    return found[0]


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")
def test_the_readmes_example_under_shortage():
    from paged_kv_cache_hkv_gb300 import binding
    binding.pkv_get_device_errors(clear=True)
    c, n, table, ref, queue, state = short_step()
    R, T, blocks = len(c), int(n.sum()), len(queue)
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    rows = lambda h: torch.randn(T, h, D, device="cuda").to(torch.bfloat16)  # noqa: E731
    kv_cache = torch.zeros(blocks, 2, B, HKV, D, dtype=torch.bfloat16, device="cuda")
    names = dict(
        torch=torch, binding=binding, block_table=i32(table), query_start_loc=i32(np.zeros(R + 1)),
        seq_lens=i32(np.zeros(R)), slots=torch.zeros(T, dtype=torch.int64, device="cuda"),
        num_computed=i32(c), query_lens=i32(n), free_queue=i32(queue), free_state=i32(state),
        ref_cnt=i32(ref), kv_cache=kv_cache, q=rows(HQ), k=rows(HKV), v=rows(HKV), out=rows(HQ),
        max_q=int(n.max()), max_s=int((c + n).max()), D=D, document_start=i32(np.zeros(T)),
        finished_rows=i32(np.arange(R)), release_ws=None,
        ws=torch.empty(binding.pkv_attention_workspace_size(R, HQ, kv_cache), dtype=torch.uint8,
                       device="cuda"))
    exec(example(), names)
    torch.cuda.synchronize()
    assert binding.pkv_get_device_errors(clear=True) == (
        binding.DEVERR_NO_BLOCKS | binding.DEVERR_LENGTHS | binding.DEVERR_BLOCK_RANGE)
    assert (names["ref_cnt"] == 0).all()
    held = sum(-(-int(x) // B) for x in c)
    free = oracle.ring(names["free_queue"].tolist(), names["free_state"].tolist())
    assert len(free) == len(set(free)) == state[1] + held  # two were taken and given back too
