"""Batch calls beside one another: threads, graphs and plans that a program may
share between them."""
import os
import subprocess
import sys
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


@pytest.mark.parametrize("before", ["nothing", "a copy", "a fill"])
@pytest.mark.parametrize("call", ["tables", "append", "attend"])
def test_a_call_is_the_first_of_a_graph(call, before):
    # alone, or right behind a copy of one of its inputs (which holds something else till then) or a fill of a result
    s = Step([200, 3, 40], [1, 9, 130], prefix=500)
    start = dict(k=s.k_pool.clone(), v=s.v_pool.clone(), table=s.d["block_table"].clone())
    s.run()
    s.check_attention()
    want = dict(out=s.out[:s.T].clone(), lse=s.lse[:, :s.T].clone(), q_rot=s.q_rot[:s.T].clone(),
                k=s.k_pool.clone(), v=s.v_pool.clone())
    given = dict(tables=s.d["fresh"], append=s.k, attend=s.q_rot)[call]
    result = dict(tables=s.d["slot_map"], append=s.q_rot, attend=s.out)[call]
    host, fill = given.cpu().pin_memory(), -9 if call == "tables" else SENTINEL
    side = torch.cuda.Stream()
    s.stream = side
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        if before == "a copy":
            given.copy_(host, non_blocking=True)
        elif before == "a fill":
            result.fill_(fill)
        getattr(s, call)()
    for _ in range(3):
        # nothing of an earlier run is left for the graph to agree with
        if call == "tables":
            s.d["block_table"].copy_(start["table"])
            for name in ("token_start", "free_head_out"):
                s.d[name].fill_(-1)
            for name in ("slot_map", "positions"):
                s.d[name].fill_(-9)
            s.d["plan"].zero_()
        elif call == "append":
            s.k_pool.copy_(start["k"])
            s.v_pool.copy_(start["v"])
            s.q_rot.fill_(SENTINEL)
        else:
            s.out.fill_(SENTINEL)
            s.lse.fill_(SENTINEL)
        if before == "a copy":
            given.fill_(0)
        elif before == "a fill":
            result.fill_(1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        if call == "tables":
            s.check_tables()
            s.stream = torch.cuda.current_stream()
            s.append()
            s.attend()
            s.stream = side
            torch.cuda.synchronize()
        elif call == "append":
            assert torch.equal(s.q_rot[:s.T], want["q_rot"])
            for name in ("k", "v"):
                assert torch.equal(getattr(s, name + "_pool").view(torch.int16), want[name].view(torch.int16))
            continue
        assert torch.equal(s.out[:s.T], want["out"]) and torch.equal(s.lse[:, :s.T], want["lse"])
        assert (s.out[s.T:] == SENTINEL).all()


def test_first_calls_of_a_process_may_come_from_many_threads():
    # what a device's first call finds out and keeps (its size, the kernels' shared memory, the map encoder)
    code = """
import threading, torch
from chunk_causal_attention_block_b200 import wf
from tests.batch_common import Step
kws = [dict(D=d, H=h, Hkv=h, seed=i) for i, (d, h) in enumerate([(64, 1), (128, 2)] * 4)]
steps = [Step([40, 0] + [1] * 2600, [3, 150] + [0] * 2600, prefix=200, **kw) for kw in kws]
torch.cuda.synchronize()
failed, gate = [], threading.Barrier(len(steps))
def work(s):
    try:
        s.stream = torch.cuda.Stream()
        gate.wait()
        s.run()
        s.stream.synchronize()
    except BaseException as e:
        failed.append(e)
threads = [threading.Thread(target=work, args=(s,)) for s in steps]
[t.start() for t in threads]
[t.join() for t in threads]
assert not failed, failed
for s in steps:
    s.check_tables()
    s.check_attention()
print("all right")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.endswith("all right\n"), r.stderr[-2000:]
