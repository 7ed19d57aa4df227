"""Values that the batched attention's documentation speaks of: keys that the
mask hides and that are not finite."""
import pytest
import torch

from chunk_causal_attention_block_b200 import wf
from tests.batch_common import Step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    wf.lib()
    yield


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("D", [64, 128])
def test_hidden_keys_that_are_not_finite(D, bad):
    # a token's own key is hidden from the tokens of its request before it; requests of every kind of unit
    cached, fresh = [30, 200, 7, 0], [6, 40, 1, 300]
    s = Step(cached, fresh, prefix=300, D=D, H=4, Hkv=2, num_ctas=11)
    s.run()
    s.check_attention()
    out, lse = s.out.clone(), s.lse.clone()
    first = 0
    for f in fresh:
        if f > 1:
            t = first + f - 2  # hidden from the request's tokens first .. t-1, seen by t and t+1
            slot, hkv, dim = int(s.d["slot_map"][t]), 1, 5
            rows = torch.zeros(s.T, dtype=torch.bool, device="cuda")
            rows[first:first + f] = True
            hidden = rows.clone()
            hidden[t:] = False
            other_heads = torch.tensor([0, 1], device="cuda")  # of key head 0
            for pool in (s.k_pool, s.v_pool):
                was = pool[slot, hkv, dim].clone()
                pool[slot, hkv, dim] = bad
                s.attend()
                pool[slot, hkv, dim] = was
                assert wf.wf_attn_workspace_status(s.ws, s.stream)[0] == wf.WF_OK
                # no other request's row, no other key head's
                assert torch.equal(s.out[:s.T][~rows], out[:s.T][~rows])
                assert torch.equal(s.lse[:, :s.T][:, ~rows], lse[:, :s.T][:, ~rows])
                assert torch.equal(s.out[:s.T, other_heads], out[:s.T, other_heads])
                # a hidden key has no part in the scores
                assert torch.equal(s.lse[:, :s.T][:, hidden], lse[:, :s.T][:, hidden])
                if pool is s.k_pool:
                    assert torch.equal(s.out[:s.T][hidden], out[:s.T][hidden])
                else:
                    # of O, only the value's own column may be touched
                    keep = torch.arange(D, device="cuda") != dim
                    assert torch.equal(s.out[:s.T][:, :, keep], out[:s.T][:, :, keep])
                    assert torch.equal(s.lse[:, :s.T], lse[:, :s.T])
                    assert not torch.isfinite(s.out[t:t + 2, 2:, dim].float()).any()
        first += f
    s.attend()
    assert torch.equal(s.out, out) and torch.equal(s.lse, lse)
