"""Host checks of the batched-request calls: sizes, refusals and the oracle's own pins."""
import ctypes

import numpy as np
import pytest

from chunk_causal_attention_block_b200 import wf
from oracle import batch_oracle as orc

GOOD = dict(H=8, Hkv=2, D=128, page_tokens=16, pool_pages=100, max_requests=4, max_tokens=64, max_request_pages=9,
            max_prefix_pages=3, block_tokens=1, num_ctas=8)


def desc(**kw):
    a = {**GOOD, **kw}
    return wf.make_batch_desc(a.pop("H"), a.pop("Hkv"), a.pop("D"), a.pop("page_tokens"), a.pop("pool_pages"), **a)


@pytest.mark.parametrize("kw,code", [
    (dict(H=0), wf.WF_ERR_INVALID_ARG), (dict(Hkv=0), wf.WF_ERR_INVALID_ARG), (dict(Hkv=3), wf.WF_ERR_INVALID_ARG),
    (dict(D=0), wf.WF_ERR_INVALID_ARG), (dict(D=96), wf.WF_ERR_UNSUPPORTED), (dict(D=256), wf.WF_ERR_UNSUPPORTED),
    (dict(dtype=wf.WF_F32), wf.WF_ERR_UNSUPPORTED), (dict(dtype=5), wf.WF_ERR_INVALID_ARG),
    (dict(H=258, Hkv=2), wf.WF_ERR_UNSUPPORTED), (dict(page_tokens=0), wf.WF_ERR_INVALID_ARG),
    (dict(page_tokens=4), wf.WF_ERR_INVALID_ARG), (dict(page_tokens=48), wf.WF_ERR_INVALID_ARG),
    (dict(page_tokens=256), wf.WF_ERR_INVALID_ARG), (dict(pool_pages=0), wf.WF_ERR_INVALID_ARG),
    (dict(pool_pages=2 ** 27), wf.WF_ERR_CAPACITY), (dict(max_requests=0), wf.WF_ERR_INVALID_ARG),
    (dict(max_requests=8193), wf.WF_ERR_CAPACITY), (dict(max_tokens=0), wf.WF_ERR_INVALID_ARG),
    (dict(max_tokens=2 ** 22 + 1), wf.WF_ERR_CAPACITY), (dict(max_request_pages=0), wf.WF_ERR_INVALID_ARG),
    (dict(max_request_pages=2 ** 24), wf.WF_ERR_CAPACITY), (dict(max_prefix_pages=-1), wf.WF_ERR_INVALID_ARG),
    (dict(max_prefix_pages=2 ** 24), wf.WF_ERR_CAPACITY), (dict(block_tokens=0), wf.WF_ERR_INVALID_ARG),
    (dict(num_ctas=-1), wf.WF_ERR_INVALID_ARG), (dict(num_ctas=257), wf.WF_ERR_CAPACITY),
    (dict(H=300, Hkv=300), wf.WF_ERR_CAPACITY),
])
def test_bad_descriptions_are_refused_everywhere(kw, code):
    d = desc(**kw)
    assert wf.wf_batch_plan_bytes(d) == 0 and wf.wf_batch_workspace_bytes(d) == 0
    p = 1 << 20  # an address that is never used: the description is looked at first
    for call in (lambda: wf.wf_batch_tables(d, *[p + 4096 * i for i in range(11)], num_free=5, plan_bytes=1 << 20),
                 lambda: wf.wf_batch_append(d, p, p, p, p, 2 * p, 3 * p),
                 lambda: wf.wf_batch_attn(d, p, p, p, p, p, p, p, workspace=p, workspace_bytes=1 << 30)):
        with pytest.raises(wf.WfError) as e:
            call()
        assert e.value.code == code


def test_sizes_grow_with_the_capacities():
    base = wf.wf_batch_plan_bytes(desc()), wf.wf_batch_workspace_bytes(desc())
    assert base[0] > 256 and base[1] > 256
    assert wf.wf_batch_plan_bytes(desc(max_tokens=4096)) > base[0]
    # partial rows: 4 per (token, head) of what may need merging, 512 per CTA
    assert wf.wf_batch_workspace_bytes(desc(num_ctas=9)) - base[1] >= 4 * 128 * (128 * 4 + 4)
    # tokens beyond one tile per request need none
    assert wf.wf_batch_workspace_bytes(desc(max_tokens=4 * 32)) == wf.wf_batch_workspace_bytes(desc(max_tokens=4096))


ARGS = dict(cached=1, fresh=2, prefix_len=3, free_pages=4, free_head=5, free_head_out=6, block_table=7, token_start=8,
            slot_map=9, positions=10, plan=11)


def tables_with(**kw):
    d = desc()
    a = {k: (v << 20) for k, v in ARGS.items()}
    a.update({k: v for k, v in kw.items()})
    wf.wf_batch_tables(d, **{"num_free": 5, "plan_bytes": wf.wf_batch_plan_bytes(d), **a})


@pytest.mark.parametrize("kw,code", [
    *[({k: None}, wf.WF_ERR_INVALID_ARG) for k in ARGS],
    (dict(num_free=-1), wf.WF_ERR_INVALID_ARG), (dict(held=12 << 20), wf.WF_ERR_INVALID_ARG),
    (dict(held_out=12 << 20), wf.WF_ERR_INVALID_ARG), (dict(free_head_out=5 << 20), wf.WF_ERR_INVALID_ARG),
    (dict(held=12 << 20, held_out=12 << 20), wf.WF_ERR_INVALID_ARG), (dict(slot_map=1 << 20), wf.WF_ERR_INVALID_ARG),
    (dict(cached=(1 << 20) + 2), wf.WF_ERR_ALIGNMENT), (dict(plan=(11 << 20) + 8), wf.WF_ERR_ALIGNMENT),
    (dict(plan_bytes=100), wf.WF_ERR_WORKSPACE),
])
def test_tables_refuse(kw, code):
    with pytest.raises(wf.WfError) as e:
        tables_with(**kw)
    assert e.value.code == code


def append_with(**kw):
    a = dict(plan=1 << 20, slot_map=2 << 20, k=3 << 20, v=4 << 20, k_pool=5 << 20, v_pool=6 << 20, q=7 << 20, rope=8 << 20,
             q_rot=9 << 20)
    a.update(kw)
    wf.wf_batch_append(desc(), **a)


@pytest.mark.parametrize("kw,code", [
    *[({k: None}, wf.WF_ERR_INVALID_ARG) for k in ("plan", "slot_map", "k", "v", "k_pool", "v_pool", "q", "q_rot", "rope")],
    (dict(rope=None, q_rot=None), wf.WF_ERR_INVALID_ARG), (dict(rope=None, q=None), wf.WF_ERR_INVALID_ARG),
    (dict(k=5 << 20), wf.WF_ERR_INVALID_ARG), (dict(v_pool=5 << 20), wf.WF_ERR_INVALID_ARG),
    *[({k: (3 << 24) + 8}, wf.WF_ERR_ALIGNMENT) for k in ("plan", "k", "v", "k_pool", "v_pool", "q", "rope", "q_rot")],
    (dict(slot_map=(3 << 24) + 2), wf.WF_ERR_ALIGNMENT),
])
def test_append_refuses(kw, code):
    with pytest.raises(wf.WfError) as e:
        append_with(**kw)
    assert e.value.code == code


def attn_with(**kw):
    a = dict(plan=1 << 20, block_table=2 << 20, prefix_table=3 << 20, q=4 << 20, k_pool=5 << 20, v_pool=6 << 20,
             out=7 << 20, lse=8 << 20, workspace=9 << 20, workspace_bytes=1 << 40)
    a.update(kw)
    wf.wf_batch_attn(desc(), **a)


@pytest.mark.parametrize("kw,code", [
    *[({k: None}, wf.WF_ERR_INVALID_ARG) for k in ("plan", "block_table", "prefix_table", "q", "k_pool", "v_pool", "out",
                                                   "workspace")],
    *[({k: (3 << 24) + 8}, wf.WF_ERR_ALIGNMENT) for k in ("plan", "q", "k_pool", "v_pool", "out", "workspace")],
    *[({k: (3 << 24) + 2}, wf.WF_ERR_ALIGNMENT) for k in ("block_table", "prefix_table", "lse")],
    (dict(workspace_bytes=1000), wf.WF_ERR_WORKSPACE), (dict(softmax_scale=-1.0), wf.WF_ERR_INVALID_ARG),
    (dict(softmax_scale=float("nan")), wf.WF_ERR_INVALID_ARG), (dict(softmax_scale=float("inf")), wf.WF_ERR_INVALID_ARG),
])
def test_attention_refuses(kw, code):
    with pytest.raises(wf.WfError) as e:
        attn_with(**kw)
    assert e.value.code == code


def test_the_binding_refuses_small_or_strided_tensors():
    torch = pytest.importorskip("torch")
    d = desc()
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    good = dict(cached=i32(4), fresh=i32(4), prefix_len=i32(1), free_pages=i32(9), free_head=i32(1), free_head_out=i32(1),
                block_table=i32(36), token_start=i32(5), slot_map=i32(64), positions=i32(64),
                plan=torch.zeros(wf.wf_batch_plan_bytes(d), dtype=torch.uint8))
    for name, bad in (("cached", i32(3)), ("token_start", i32(4)), ("slot_map", i32(63)), ("block_table", i32(72)[::2]),
                      ("fresh", torch.zeros(4, dtype=torch.int64)), ("free_head_out", i32(0))):
        with pytest.raises(wf.WfError) as e:
            wf.wf_batch_tables(d, **{**good, name: bad})
        assert e.value.code == wf.WF_ERR_INVALID_ARG


# ---------------------------------------------------------------- the oracle, by hand
def test_oracle_tables_by_hand():
    table = [[3, 0, 0], [5, 6, 0], [0, 0, 0]]
    got = orc.tables([4, 7, 0], [1, 2, 0], 10, 4, [9, 8, 7, 2], 1, table)
    assert got[0].tolist() == [[3, 8, 0], [5, 6, 7], [0, 0, 0]]
    assert got[1].tolist() == [0, 1, 3, 3]
    assert got[2].tolist() == [32, 27, 28] and got[3].tolist() == [14, 17, 18]
    assert got[4] == 3 and got[5].tolist() == [2, 3, 0]
    held = orc.tables([1, 2], [1, 6], 0, 4, [9, 8], 0, [[4, 1], [5, 0]], held=[2, 1])
    assert held[0].tolist() == [[4, 1], [5, 9]] and held[4] == 1 and held[5].tolist() == [2, 2]


def test_oracle_rotation_by_hand():
    x = np.array([[[1.0, 0.0, 3.0, 4.0]]])
    cs = np.array([[[0.0, 1.0], [-1.0, 0.0]]])
    assert orc.rotate(x, cs).tolist() == [[[0.0, 1.0, -3.0, -4.0]]]


def test_oracle_attention_by_hand():
    # one head, D = 2, pages of 2: prefix key on page 2, own keys on page 0; equal scores, so plain means
    v = np.zeros((6, 1, 2))
    v[4, 0], v[0, 0], v[1, 0] = [6.0, 0.0], [0.0, 2.0], [3.0, 4.0]
    k = np.zeros((6, 1, 2))
    q = np.ones((2, 1, 2))
    r = orc.attention(q, k, v, [0], [2], 1, [[0]], [2], 2, 1)
    np.testing.assert_allclose(r["O"][:, 0], [[3.0, 1.0], [3.0, 2.0]])
    np.testing.assert_allclose(r["LSE"][0], np.log([2.0, 3.0]))
    r = orc.attention(q, k, v, [0], [2], 1, [[0]], [2], 2, 2)  # blocks of two: both rows see both
    np.testing.assert_allclose(r["O"][:, 0], [[3.0, 2.0], [3.0, 2.0]])


def test_struct_sizes_match_the_header():
    assert ctypes.sizeof(wf.BatchDesc) == 48


@pytest.mark.parametrize("name", ["q", "k_pool", "v_pool"])
def test_attention_does_not_write_over_what_it_reads(name):
    # other thread blocks may still read the rows that one of them stores
    with pytest.raises(wf.WfError) as e:
        attn_with(**{name: 7 << 20})
    assert e.value.code == wf.WF_ERR_INVALID_ARG


@pytest.mark.parametrize("a,b", [("slot_map", "positions"), ("token_start", "slot_map"), ("plan", "block_table"),
                                 ("free_head_out", "token_start")])
def test_tables_need_a_buffer_for_each_result(a, b):
    with pytest.raises(wf.WfError) as e:
        tables_with(**{a: ARGS[b] << 20})
    assert e.value.code == wf.WF_ERR_INVALID_ARG


def test_memory_that_is_not_the_devices_is_refused():
    # every argument is well formed, but the plan is no memory of the current device (here: of none at all)
    d = desc()
    for call in (tables_with, append_with, attn_with):
        with pytest.raises(wf.WfError) as e:
            call()
        assert e.value.code == wf.WF_ERR_INVALID_ARG
    torch = pytest.importorskip("torch")
    host = torch.zeros(wf.wf_batch_plan_bytes(d), dtype=torch.uint8)
    x = torch.zeros(64, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(wf.WfError) as e:
        wf.wf_batch_append(d, host, torch.zeros(64, dtype=torch.int32), x, x, x, x)
    assert e.value.code == wf.WF_ERR_INVALID_ARG


@pytest.mark.parametrize("a,b", [("q_rot", "k"), ("q_rot", "v"), ("q_rot", "rope"), ("q_rot", "k_pool"), ("v_pool", "k"),
                                 ("k_pool", "q"), ("k_pool", "rope")])
def test_append_does_not_write_over_what_it_reads(a, b):
    at = dict(k=3 << 20, v=4 << 20, k_pool=5 << 20, q=7 << 20, rope=8 << 20)
    with pytest.raises(wf.WfError) as e:
        append_with(**{a: at[b]})
    assert e.value.code == wf.WF_ERR_INVALID_ARG


def test_arguments_of_other_types_are_refused():
    torch = pytest.importorskip("torch")
    d = desc()
    at = 1 << 20
    for call in (lambda: tables_with(cached=np.zeros(4, np.int32)), lambda: tables_with(num_free="5"),
                 lambda: tables_with(num_free=None), lambda: tables_with(num_free=2 ** 40), lambda: tables_with(fresh=2.0),
                 lambda: append_with(k=[1, 2]), lambda: attn_with(softmax_scale="1"), lambda: attn_with(workspace_bytes=None),
                 lambda: attn_with(q=2 ** 70), lambda: attn_with(lse=torch.zeros(10 ** 4)),
                 lambda: attn_with(q=torch.zeros(64, 8, 128, dtype=torch.bfloat16).to_sparse())):
        with pytest.raises(wf.WfError) as e:
            call()
        assert e.value.code == wf.WF_ERR_INVALID_ARG
    for other in (wf.RoundDesc(), b"12", None):
        with pytest.raises(TypeError):
            wf.wf_batch_append(other, at, at, at, at, 2 * at, 3 * at)
    assert bytes(d) == bytes(desc())
