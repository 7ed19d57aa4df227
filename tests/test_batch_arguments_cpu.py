"""What the batch calls' binding makes of tensors, by the reason it gives: each
refusal names the argument and what is wrong with it, so that one check cannot
stand in for another.  The plan is a raw address here (a tensor would have to
be on a GPU), and nothing is ever launched: all memory is the host's."""
import pytest
import torch

from chunk_causal_attention_block_b200 import wf

D = dict(H=4, Hkv=2, D=64, page_tokens=16, pool_pages=10, max_requests=3, max_tokens=40, max_request_pages=5,
         max_prefix_pages=2, num_ctas=8)
AT = 1 << 20


def desc():
    a = dict(D)
    return wf.make_batch_desc(a.pop("H"), a.pop("Hkv"), a.pop("D"), a.pop("page_tokens"), a.pop("pool_pages"), **a)


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def f32(*shape):
    return torch.zeros(*shape, dtype=torch.float32)


# every tensor argument, well formed but for its device
TABLES = dict(cached=i32(3), fresh=i32(3), prefix_len=i32(1), held=i32(3), free_pages=i32(9), free_head=i32(1),
              free_head_out=i32(1), held_out=i32(3), block_table=i32(3, 5), token_start=i32(4), slot_map=i32(40),
              positions=i32(40))
APPEND = dict(slot_map=i32(40), rope=f32(40, 32, 2), q=bf16(40, 4, 64), k=bf16(40, 2, 64), v=bf16(40, 2, 64),
              q_rot=bf16(40, 4, 64), k_pool=bf16(160, 2, 64), v_pool=bf16(160, 2, 64))
ATTN = dict(block_table=i32(3, 5), prefix_table=i32(2), q=bf16(40, 4, 64), k_pool=bf16(160, 2, 64),
            v_pool=bf16(160, 2, 64), out=bf16(40, 4, 64), lse=f32(4, 40),
            workspace=torch.zeros(1 << 20, dtype=torch.uint8))
CALLS = dict(tables=(wf.wf_batch_tables, TABLES), append=(wf.wf_batch_append, APPEND), attn=(wf.wf_batch_attn, ATTN))
EVERY = [(call, name) for call, (_, args) in CALLS.items() for name in args]


def reason(call, **change):
    """Why the call with raw addresses but for `change` was refused."""
    f, args = CALLS[call]
    a = {name: AT * (2 + i) for i, name in enumerate(args)}
    a["plan"] = AT
    if call == "tables":
        a.update(num_free=9, plan_bytes=1 << 20)
    if call == "attn":
        a["workspace_bytes"] = 1 << 30
    with pytest.raises(wf.WfError) as e:
        f(desc(), **{**a, **change})
    assert e.value.code == wf.WF_ERR_INVALID_ARG
    return str(e.value)


@pytest.mark.parametrize("call,name", EVERY)
def test_a_tensor_of_another_type_is_refused_for_its_type(call, name):
    good = CALLS[call][1][name]
    assert f"{name} has " in reason(call, **{name: good}) and "on cpu" in reason(call, **{name: good})
    # other types of the same element size, and of another
    others = {torch.int32: (torch.float32, torch.uint32, torch.int64), torch.float32: (torch.int32, torch.float64),
              torch.bfloat16: (torch.float16, torch.int16, torch.float32), torch.uint8: (torch.int16,)}[good.dtype]
    for t in others:
        assert f"{name} is of type" in reason(call, **{name: good.to(t)}), t
