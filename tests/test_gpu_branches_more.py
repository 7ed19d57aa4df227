"""Branches of rollouts that begin where others do not: without history, on a
stream of their own, from a restored or a fused-Q parent."""
import numpy as np
import pytest
import torch

from chunk_causal_attention_block_b200 import wf
from chunk_causal_attention_block_b200.rollout import BranchRollout, Rollout
from tests.test_gpu_branches import SMALL, check_round

pytestmark = pytest.mark.gpu
ROWS = np.arange(SMALL.R * SMALL.C)


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    wf.lib()
    yield


def test_branches_without_history():
    ro = Rollout(SMALL, first_n0=0)
    ro.prefill()
    br = BranchRollout(ro, branches=2, rounds=3, page_tokens=16)
    assert br.prefix_tokens == 0
    for r in range(3):
        br.run_round(r)
        check_round(br, r, [0, 1], ROWS)


def test_branches_on_a_stream_that_is_not_the_current_one():
    side = torch.cuda.Stream()
    ro = Rollout(SMALL, stream=side)
    ro.prefill()
    ro.run_round(0)
    br = BranchRollout(ro, branches=2, rounds=2, page_tokens=32)
    for r in range(2):
        br.run_round(r)
        side.synchronize()
        check_round(br, r, [0, 1], ROWS)
    assert br.device_status()[0] == wf.WF_OK


def test_branches_of_a_restored_parent():
    ro = Rollout(SMALL)
    ro.prefill()
    ro.run_round(0)
    state = ro.checkpoint()
    again = Rollout(SMALL, seed=1, fused_q_rope=True)
    again.restore(state)
    outs = []
    for parent in (ro, again):
        br = BranchRollout(parent, branches=2, page_tokens=8)
        br.run_round(0)
        check_round(br, 0, [0, 1], ROWS)
        outs.append(br.out.clone())
    assert torch.equal(*outs)


def test_pages_are_taken_once_and_kept():
    ro = Rollout(SMALL)
    ro.prefill()
    br = BranchRollout(ro, branches=3, rounds=3, page_tokens=16)
    held = [0] * 3
    for r in range(3):
        br.run_round(r)
        tokens = (r + SMALL.R) * SMALL.C
        held = [max(h, -(-tokens // 16)) for h in held]
        assert br.held[0].tolist() == held
        table = br.block_table.cpu().numpy()
        mine = [p for b in range(3) for p in table[b, :held[b]]] + br.prefix_table.flatten().tolist()
        assert len(set(mine)) == len(mine) and min(mine) >= 0 and max(mine) < br.desc.pool_pages
