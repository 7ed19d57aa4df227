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
