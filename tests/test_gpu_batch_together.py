"""Batch calls beside one another: threads, graphs and plans that a program may
share between them."""
import threading

import pytest
import torch

from chunk_causal_attention_block_b200 import wf
from tests.batch_common import SENTINEL, Step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    wf.lib()
    yield


@pytest.mark.parametrize("kw", [dict(), dict(D=64, H=6, Hkv=3, num_ctas=23)])
def test_two_threads_on_one_stream_and_workspace(kw):
    # the stream keeps the calls apart, so one workspace serves both; each call's two kernels have to stay together
    s = Step([900, 20, 4], [1, 30, 300], prefix=1500, **kw)
    s.run()
    s.check_attention()
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    work = []
    for _ in range(3):
        q = torch.randn(s.q.shape, generator=g, device="cuda").to(torch.bfloat16)
        out, lse = torch.full_like(s.out, SENTINEL), torch.full_like(s.lse, SENTINEL)
        attend(s, q, out, lse)
        work.append((q, out.clone(), lse.clone()))
    torch.cuda.synchronize()
    failed = []

    def loop(q, want, want_lse):
        try:
            torch.cuda.set_device(0)
            outs = [(torch.empty_like(s.out), torch.empty_like(s.lse)) for _ in range(40)]
            with torch.cuda.stream(s.stream):
                for _ in range(5):
                    for out, lse in outs:
                        attend(s, q, out, lse)
                    s.stream.synchronize()
                    for out, lse in outs:
                        assert torch.equal(out[:s.T], want[:s.T]) and torch.equal(lse[:, :s.T], want_lse[:, :s.T])
        except BaseException as e:  # noqa: BLE001 (seen by the test below)
            failed.append(e)

    threads = [threading.Thread(target=loop, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


def attend(s, q, out, lse):
    wf.wf_batch_attn(s.desc, s.d["plan"], s.d["block_table"], s.prefix_dev, q, s.k_pool, s.v_pool, out, lse,
                     workspace=s.ws, stream=s.stream)


def test_an_item_may_run_longer_than_the_wait_limit(monkeypatch):
    # ten units of 256 rows on one block, each some 15 ms long: a slot of the block's eight items comes free only
    # when the oldest is done, and what waits for it may not take that for a stall
    s = Step([0], [2560], prefix=1 << 21, H=1, Hkv=1, D=64, page=128, num_ctas=1, poison=0.0)
    s.run()
    assert wf.wf_attn_workspace_status(s.ws, s.stream)[0] == wf.WF_OK
    out, lse = s.out.clone(), s.lse.clone()
    assert not (out[:s.T] == SENTINEL).any()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    s.attend()
    end.record()
    end.synchronize()
    assert start.elapsed_time(end) > 10 * 6.0  # each unit well above the limit set below
    s.out.fill_(SENTINEL)
    monkeypatch.setenv("WF_WAIT_TIMEOUT_MS", "3")
    s.attend()
    monkeypatch.delenv("WF_WAIT_TIMEOUT_MS")
    code, detail = wf.wf_attn_workspace_status(s.ws, s.stream)
    assert code == wf.WF_OK, detail
    assert torch.equal(s.out, out) and torch.equal(s.lse, lse)
