"""What the batch calls' binding makes of tensors, by the reason it gives: each
refusal names the argument and what is wrong with it, so that one check cannot
stand in for another.  The plan is a raw address here (a tensor would have to
be on a GPU), and nothing is ever launched: all memory is the host's."""
import os
import shutil
import subprocess

import pytest
import torch

from chunk_causal_attention_block_b200 import build as wfbuild
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


@pytest.mark.parametrize("call,name,shape", [
    *[(call, "block_table", s) for call in ("tables", "attn") for s in ((3, 6), (4, 4), (5, 3), (1, 3, 6))],
    *[("attn", "lse", s) for s in ((4, 41), (5, 36), (40, 4), (2, 2, 80))],
    *[(call, n, s) for call, n in (("append", "q"), ("append", "q_rot"), ("attn", "q"), ("attn", "out"))
      for s in ((40, 5, 64), (40, 64, 4), (40, 320), (20, 8, 64), (4, 40, 64), (40, 2, 128), (20, 512))],
    *[("append", n, s) for n in ("k", "v") for s in ((40, 4, 64), (40, 64, 2), (40, 1, 128 * 2), (2, 40, 64))],
    *[(call, n, s) for call in ("append", "attn") for n in ("k_pool", "v_pool")
      for s in ((160, 3, 64), (160, 64, 2), (2, 160, 64), (10, 2, 16, 64), (80, 256), (10, 16, 3, 64))],
    *[("append", "rope", s) for s in ((40, 32, 3), (40, 2, 32), (40, 65), (40, 33, 2), (40, 64, 2))],
])
def test_rows_of_another_length_are_refused(call, name, shape):
    good = CALLS[call][1][name]
    assert f"{name} is of shape" in reason(call, **{name: torch.zeros(shape, dtype=good.dtype)})


@pytest.mark.parametrize("call,name,shape", [
    *[(call, "block_table", s) for call in ("tables", "attn") for s in ((15,), (20,), (4, 5), (1, 3, 5), (3, 5, 1))],
    ("attn", "prefix_table", (1, 2)), ("attn", "prefix_table", (2, 1)), ("attn", "prefix_table", (7,)),
    *[("attn", "lse", s) for s in ((160,), (5, 40), (2, 2, 40))],
    *[(call, n, s) for call, n in (("append", "q"), ("append", "q_rot"), ("attn", "q"), ("attn", "out"))
      for s in ((41, 4, 64), (40, 256), (40 * 256,), (40, 2, 2, 64), (2, 20, 4, 64))],
    *[("append", n, s) for n in ("k", "v") for s in ((44, 2, 64), (40, 128), (2, 20, 2, 64), (5120,))],
    *[(call, n, s) for call in ("append", "attn") for n in ("k_pool", "v_pool")
      for s in ((10, 16, 2, 64), (160, 128), (10, 2048), (11, 2048), (10, 16, 128), (20480,))],
    *[("append", "rope", s) for s in ((40, 64), (1, 40, 32, 2), (2560,))],
])
def test_shapes_of_the_documented_rows_are_not(call, name, shape):
    # (what is wrong with them is where they lie)
    good = CALLS[call][1][name]
    assert "on cpu" in reason(call, **{name: torch.zeros(shape, dtype=good.dtype)})


def test_the_end_of_a_single_row_does_not_matter():
    one = wf.make_batch_desc(1, 1, 64, 16, 10, max_requests=1, max_tokens=1, max_request_pages=5, num_ctas=8)
    for shape in ((1, 9), (2, 3), (5, 1)):
        with pytest.raises(wf.WfError, match="on cpu"):
            wf.wf_batch_attn(one, AT, i32(*shape), None, 2 * AT, 3 * AT, 4 * AT, 5 * AT, f32(1, 1), workspace=6 * AT,
                             workspace_bytes=1 << 30)


def test_a_size_above_the_tensors_is_refused():
    small = torch.zeros(100, dtype=torch.uint8)
    for n in (101, 1 << 30):
        assert "plan_bytes is more than plan holds" in reason("tables", plan=small, plan_bytes=n)
        assert "num_free is more than free_pages holds" in reason("tables", free_pages=i32(100), num_free=n)
    # not more: what is wrong is where they lie
    assert "on cpu" in reason("tables", plan=small, plan_bytes=99)
    assert "on cpu" in reason("tables", free_pages=i32(100), num_free=100)


def test_every_plan_holds_what_is_read_of_it_before_it_is_known_to_be_the_calls():
    # 256 bytes of header and 8 for each of the up to 256 blocks of a call
    head = 256 + 256 * 8
    for ctas in (1, 2, 256):
        assert wf.wf_batch_plan_bytes(wf.make_batch_desc(1, 1, 64, 8, 1, max_requests=1, max_tokens=1,
                                                         max_request_pages=1, num_ctas=ctas)) >= head
    for call in ("tables", "append", "attn"):
        short = torch.zeros(head - 1, dtype=torch.uint8)
        extra = dict(plan_bytes=None) if call == "tables" else {}
        assert f"where {head} are needed" in reason(call, plan=short, **extra)


def test_what_counts_as_shared_memory(tmp_path):
    if not shutil.which("g++"):
        pytest.skip("no C++ compiler")
    exe = str(tmp_path / "overlap")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", wfbuild.INCLUDE, "-I", wfbuild.CSRC,
                    os.path.join(os.path.dirname(__file__), "c", "overlap.cpp"), "-o", exe], check=True)
    assert subprocess.run([exe], capture_output=True, text=True, check=True).stdout == "0 wrong\n"


@pytest.mark.parametrize("call,name", EVERY)
def test_tensors_beside_a_plan_by_address_have_to_be_on_the_current_device(call, name):
    # (an address says nothing of the device that the other tensors have to be on)
    assert "on the current GPU" in reason(call, **{name: CALLS[call][1][name]})
