"""Branches of a rollout: several continuations of one history, denoised
together over a shared prefix, against the fp64 oracle and the ring path."""
import dataclasses

import numpy as np
import pytest
import torch

from chunk_causal_attention_block_b200 import wf
from chunk_causal_attention_block_b200.rollout import CONFIGS, BranchRollout, Rollout, RoundConfig
from tests import gpu_common as gc

pytestmark = pytest.mark.gpu

SMALL = RoundConfig("branches", H=2, D=128, fh=10, fw=10, F=3, Wc=3, R=3, noise_t=(250, 500, 750))


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    wf.lib()
    yield


def expected(br: BranchRollout, b: int, r: int, heads, rows):
    """The oracle's round r of branch b: the parent's chunks below n0 (its seed), the branch's own from n0 on."""
    cfg, ro, seed = br.cfg, br.parent, br.seed + b
    window = min(cfg.Wc, br.n0) + r  # a branch keeps all of the history it started from
    grown = dataclasses.replace(cfg, Wc=window, S=0)
    n0 = br.n0 + r
    q, k, v, kc, vc = gc.oracle_inputs(grown, n0, ro.first_n0, heads, seed)
    _, _, _, kc0, vc0 = gc.oracle_inputs(grown, n0, ro.first_n0, heads, br.seed)
    old = window - r
    kc[:old], vc[:old] = kc0[:old], vc0[:old]
    return gc.oracle_call(grown, n0, (q, k, v, kc, vc), rows)


def check_round(br, r, heads, rows):
    n = br.cfg.R * br.cfg.C
    for b in range(br.branches):
        ref = expected(br, b, r, heads, rows)
        gc.assert_bf16_close(gc.to_np(br.out[b * n + rows][:, heads]), ref["O"], f"branch {b} round {r}")
        lse = br.lse[heads][:, b * n + rows].t().cpu().numpy()
        np.testing.assert_allclose(lse, ref["LSE"], rtol=0, atol=2e-3 * max(1.0, np.abs(ref["LSE"]).max()))
    assert br.device_status()[0] == wf.WF_OK


@pytest.mark.parametrize("first_n0,after,page", [(3, 0, 64), (3, 2, 16), (1, 0, 128), (5, 4, 8)])
def test_branches_follow_the_oracle(first_n0, after, page):
    ro = Rollout(SMALL, first_n0=first_n0)
    ro.prefill()
    for r in range(after):
        ro.run_round(r)
    br = BranchRollout(ro, branches=3, rounds=3, page_tokens=page)
    rows = np.arange(SMALL.R * SMALL.C)
    for r in range(3):
        br.run_round(r)
        check_round(br, r, [0, 1], rows)
    # the ring is untouched: the parent goes on as if nothing had been
    ro.run_round(after)
    gc.check_attention(ro, after, [0, 1], rows, "parent")
    with pytest.raises(ValueError):
        br.run_round(3)


def test_branch_zero_continues_as_the_parent():
    ro = Rollout(SMALL)
    ro.prefill()
    br = BranchRollout(ro, branches=2)
    br.run_round(0)
    ro.run_round(0)
    n = SMALL.R * SMALL.C
    # same keys and queries but for the rotation's fp32 arithmetic: the two stay within two bf16 roundings
    gc.assert_bf16_close(gc.to_np(br.out[:n]), gc.to_np(ro.out[:n]), "branch 0")
    assert not torch.equal(br.out[:n], br.out[n:])


def test_full_size_branches_sampled():
    cfg = CONFIGS["wan13b_round"]
    ro = Rollout(cfg)
    ro.prefill()
    br = BranchRollout(ro, branches=2)
    br.run_round(0)
    check_round(br, 0, [0, 7], gc.sample_rows(cfg, extra=4))


def test_branches_refuse_what_they_cannot_continue():
    with pytest.raises(ValueError):
        BranchRollout(Rollout(CONFIGS["tiny_f32"]), 2)
    ro = Rollout(SMALL)
    ro.prefill()
    with pytest.raises(ValueError):
        BranchRollout(ro, 0)
    br = BranchRollout(ro, 1)
    with pytest.raises(ValueError):
        br.run_round(1)
