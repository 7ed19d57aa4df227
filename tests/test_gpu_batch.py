"""Batched requests on the GPU: block tables, cache append and attention over a
shared prefix against the fp64 oracle, at the lengths, pages, groups and cuts
where they can go wrong."""
import numpy as np
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


def whole(**kw):
    s = Step(**kw)
    s.tables()
    s.check_tables()
    k, v = s.k_pool.clone(), s.v_pool.clone()
    s.append()
    s.check_append(k, v)
    s.attend()
    s.check_attention(str(kw))
    return s


# ---------------------------------------------------------------- tables and append
@pytest.mark.parametrize("page", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("cached,fresh", [
    ([0], [1]), ([0], [0]), ([5, 0, 16, 17], [0, 0, 0, 0]), ([0, 127, 128, 129, 15, 16], [1, 1, 1, 1, 1, 1]),
    ([3, 0, 40, 0, 7], [130, 0, 1, 257, 0]),
])
def test_tables_and_append(page, cached, fresh):
    s = Step(cached, fresh, prefix=37, page=page)
    s.tables()
    s.check_tables()
    k, v = s.k_pool.clone(), s.v_pool.clone()
    s.append()
    s.check_append(k, v)


@pytest.mark.parametrize("B", [1, 31, 1023, 1024, 1025, 2100])
def test_tables_of_many_requests(B):
    rng = np.random.default_rng(B)
    s = Step(rng.integers(0, 90, B), rng.integers(0, 4, B), prefix=5, H=2, Hkv=2, D=64)
    s.tables()
    s.check_tables()


def test_tables_of_the_most_requests():
    rng = np.random.default_rng(3)
    s = Step(rng.integers(0, 20, 8192), rng.integers(0, 3, 8192), H=1, Hkv=1, D=64, page=8)
    s.tables()
    s.check_tables()


def test_tables_keep_pages_that_were_held():
    # cached lengths fell back: pages taken before are used again, none is taken twice
    s = Step([10, 64, 0], [30, 1, 100], held=[5, 6, 2], page=16, prefix=20)
    s.tables()
    s.check_tables()
    s.append()
    s.attend()
    s.check_attention()


def test_append_without_angles_copies():
    s = Step([3, 18], [20, 1], rope=False)
    s.tables()
    k, v = s.k_pool.clone(), s.v_pool.clone()
    s.append()
    s.check_append(k, v)


def test_append_turns_q_in_place():
    s = Step([3, 18], [20, 1])
    s.run()
    want = s.q_rot[:s.T].clone()
    wf.wf_batch_append(s.desc, s.d["plan"], s.d["slot_map"], s.k, s.v, s.k_pool, s.v_pool, q=s.q, rope=s.rope, q_rot=s.q,
                       stream=s.stream)
    assert torch.equal(s.q[:s.T], want)


# ---------------------------------------------------------------- attention
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cached,fresh,prefix", [
    ([0], [1], 0), ([0], [1], 1), ([300], [1], 0), ([127], [1], 128), ([128], [1], 129),
    ([5, 0, 250], [1, 1, 1], 0), ([5, 0, 250], [1, 1, 1], 1), ([5, 0, 250], [1, 1, 1], 700),
    ([0, 9, 0, 40], [0, 1, 0, 2], 130), ([0, 0], [0, 0], 50),
    ([0], [129], 0), ([0, 77], [300, 1], 260), ([33, 0, 500], [64, 700, 3], 127),
])
def test_lengths(D, cached, fresh, prefix):
    whole(cached=cached, fresh=fresh, prefix=prefix, D=D)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 3), (10, 2), (7, 1), (14, 2), (16, 1), (32, 2), (65, 1), (128, 1)])
def test_groups(H, Hkv):
    whole(cached=[40, 0, 130, 9], fresh=[1, 33, 2, 5], prefix=200, H=H, Hkv=Hkv)
    whole(cached=[40, 0], fresh=[150, 1], prefix=0, H=H, Hkv=Hkv, D=64)


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
def test_pages_that_end_inside_a_tile(page, D):
    whole(cached=[1, 135, 60], fresh=[1, 2, 200], prefix=143, page=page, D=D)


@pytest.mark.parametrize("block", [1, 2, 37, 128, 300, 1 << 30])
def test_block_masks(block):
    whole(cached=[0, 74, 10], fresh=[333, 111, 1], prefix=65, block=block)


@pytest.mark.parametrize("num_ctas", [1, 2, 5, 37, 148, 256])
def test_cuts_of_the_work(num_ctas):
    whole(cached=[900, 20, 0], fresh=[1, 1, 280], prefix=1500, num_ctas=num_ctas)
    whole(cached=[900], fresh=[3], prefix=1500, num_ctas=num_ctas, D=64)
    whole(cached=[10] * 40, fresh=[1] * 40, prefix=900, num_ctas=num_ctas, H=8, Hkv=8)


@pytest.mark.parametrize("n", [2, 63, 64, 65, 127, 128, 129, 200])
def test_many_small_requests_fill_row_tiles(n):
    rng = np.random.default_rng(n)
    whole(cached=rng.integers(0, 300, n), fresh=rng.integers(0, 3, n), prefix=333, H=3, Hkv=3)


def test_requests_around_the_sharing_threshold():
    # group 2: up to 32 tokens share the prefix tiles, more run them alone
    whole(cached=[0] * 6, fresh=[31, 32, 33, 1, 64, 65], prefix=400, H=4, Hkv=2)


@pytest.mark.parametrize("scale", [1e-3, 0.5, 4.0])
def test_scales(scale):
    whole(cached=[40, 300], fresh=[1, 150], prefix=200, scale=scale)


def test_a_late_key_dominates():
    # the maximum grows by far more than 2^8 after many keys: O and the sums are rescaled
    s = Step([600, 5], [1, 1], prefix=500, rope=False)
    s.tables()
    s.append()
    slot = s.d["slot_map"][0]
    s.k_pool[slot] = 8 * s.q[0, ::2]
    s.attend()
    s.check_attention()


def test_masked_keys_may_be_anything():
    for poison in (float("nan"), float("inf"), -3.0e38):
        whole(cached=[1, 130, 60], fresh=[1, 1, 40], prefix=143, page=128, poison=poison)


def test_pools_beyond_32_bit_offsets():
    # pages at 4.3 GB and more into each pool
    whole(cached=[100, 3], fresh=[1, 150], prefix=200, page=128, H=1, Hkv=1, far_pages=131072)


def test_a_long_prefix_is_shared_out():
    whole(cached=[0, 700], fresh=[1, 1], prefix=60000, H=2, Hkv=1, page=128)


# ---------------------------------------------------------------- steps together
def test_results_do_not_depend_on_timing():
    s = Step([900, 20, 0] * 9, [1, 1, 30] * 9, prefix=1500).run()
    out, lse = s.out.clone(), s.lse.clone()
    for _ in range(5):
        s.attend()
        assert torch.equal(s.out, out) and torch.equal(s.lse, lse)


def test_a_captured_graph_follows_the_lengths():
    s = Step([100, 0, 40], [8, 20, 0], prefix=200, spare_tokens=64, spare_cols=4)
    s.free_pages = np.concatenate([s.free_pages])
    side = torch.cuda.Stream()
    s.stream = side
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run()
    side.synchronize()
    s.check_attention("before the capture")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        s.run()
    for cached, fresh in (([100, 0, 40], [8, 20, 0]), ([100, 0, 40], [1, 1, 2]), ([100, 0, 40], [0, 0, 0]),
                          ([100, 0, 40], [1, 30, 3])):
        s.cached, s.fresh, s.T = cached, fresh, sum(fresh)
        s.d["fresh"].copy_(torch.tensor(fresh, dtype=torch.int32))
        for name in ("slot_map", "positions"):
            s.d[name].fill_(-9)
        s.d["block_table"].copy_(torch.tensor(s.table, dtype=torch.int32))
        for t in (s.out, s.lse, s.q_rot):
            t.fill_(SENTINEL)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        s.check_tables()
        s.check_attention(str(fresh))


def test_steps_in_a_row_take_pages_one_after_another():
    s = Step([0, 30, 7], [5, 1, 0], prefix=40, spare_tokens=40, spare_cols=6)
    s.tables()
    s.check_tables()
    head, table, cached = int(s.d["free_head_out"]), s.d["block_table"].clone(), [5, 31, 7]
    assert torch.equal(table.cpu(), s.d["block_table"].cpu())
    s2_fresh = [13, 0, 2]
    s.cached, s.fresh, s.T, s.free_head, s.table = cached, s2_fresh, 15, head, table.cpu().numpy()
    s.free_pages = np.concatenate([s.free_pages, np.arange(9)])
    s.d.update(free_pages=torch.tensor(s.free_pages, dtype=torch.int32, device="cuda"))
    s.d["cached"].copy_(torch.tensor(cached, dtype=torch.int32))
    s.d["fresh"].copy_(torch.tensor(s2_fresh, dtype=torch.int32))
    head_in = s.d["free_head_out"].clone()
    s.d["slot_map"].fill_(-9)
    s.d["positions"].fill_(-9)
    s.tables(free_head=head_in)
    s.check_tables()


def test_two_steps_at_once_on_two_streams():
    one, two = Step([900, 20], [1, 30], prefix=1500), Step([5, 60, 7], [200, 1, 2], prefix=300, D=64, H=6, Hkv=3)
    for s in (one, two):
        s.run()
        s.check_attention()
    outs = [s.out.clone() for s in (one, two)]
    torch.cuda.synchronize()
    one.stream, two.stream = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        one.run()
        two.run()
    torch.cuda.synchronize()
    for s, o in zip((one, two), outs):
        assert torch.equal(s.out, o)


def test_writes_stay_inside_their_buffers():
    s = Step([20, 3, 128], [2, 300, 1], prefix=150, H=6, Hkv=3)
    guards = []

    def guard(t):
        pad = 4096
        raw = torch.full((t.numel() * t.element_size() + 2 * pad,), 0x5A, dtype=torch.uint8, device="cuda")
        mid = raw[pad:pad + t.numel() * t.element_size()]
        mid.copy_(t.contiguous().view(torch.uint8).reshape(-1))
        guards.append((raw, pad))
        return mid.view(t.dtype).view(t.shape)

    for name in ("free_head_out", "block_table", "token_start", "slot_map", "positions", "plan"):
        s.d[name] = guard(s.d[name])
    for name in ("k_pool", "v_pool", "q_rot", "out", "lse", "ws"):
        setattr(s, name, guard(getattr(s, name)))
    s.run()
    torch.cuda.synchronize()
    s.check_tables()
    s.check_attention()
    for raw, pad in guards:
        assert (raw[:pad] == 0x5A).all() and (raw[-pad:] == 0x5A).all()


def test_expired_wait_reports_timeout_and_context_stays_usable(monkeypatch):
    # CTA 0's first K tile is never loaded: every role has to leave within the limit
    for kw in (dict(cached=[300, 20], fresh=[1, 40], prefix=700), dict(cached=[0], fresh=[900], D=64)):
        s = Step(**kw)
        s.tables()
        s.append()
        monkeypatch.setenv("WF_WAIT_TIMEOUT_MS", "100")
        monkeypatch.setenv("WF_DEBUG_STALL_FIRST_LOAD", "1")
        s.attend()
        code, detail = wf.wf_attn_workspace_status(s.ws, s.stream)
        monkeypatch.delenv("WF_DEBUG_STALL_FIRST_LOAD")
        monkeypatch.delenv("WF_WAIT_TIMEOUT_MS")
        assert code == wf.WF_ERR_DEVICE_TIMEOUT and detail[2] == 0, (code, detail)
        wf.wf_attn_workspace_init(s.ws, s.stream)
        s.attend()
        s.check_attention()


# ---------------------------------------------------------------- what does not fit
@pytest.mark.parametrize("change,code", [
    (dict(cached=[-1, 3]), wf.WF_ERR_INVALID_ARG), (dict(fresh=[2, -5]), wf.WF_ERR_INVALID_ARG),
    (dict(fresh=[2, 1000]), wf.WF_ERR_CAPACITY), (dict(cached=[2 ** 31 - 1, 3]), wf.WF_ERR_CAPACITY),
    (dict(free_head=[-1]), wf.WF_ERR_INVALID_ARG), (dict(free_head=[10 ** 6]), wf.WF_ERR_CAPACITY),
    (dict(prefix_len=[-1]), wf.WF_ERR_INVALID_ARG), (dict(prefix_len=[10 ** 6]), wf.WF_ERR_CAPACITY),
    (dict(fresh=[2 ** 31 - 1, 2 ** 31 - 1]), wf.WF_ERR_CAPACITY),
])
def test_lengths_that_do_not_fit_void_the_step(change, code):
    s = Step([20, 3], [2, 30], prefix=50)
    for name, v in change.items():
        s.d[name].copy_(torch.tensor(v, dtype=torch.int32))
    head = int(s.d["free_head"])
    k = s.k_pool.clone()
    s.run()
    assert wf.wf_batch_status(s.d["plan"], s.stream) == code
    assert int(s.d["free_head_out"]) == head
    assert s.d["token_start"].tolist() == [0, 0, 0]
    assert torch.equal(s.d["block_table"].cpu(), torch.tensor(s.table, dtype=torch.int32))
    assert (s.d["slot_map"] == -9).all() and (s.q_rot == SENTINEL).all()
    assert torch.equal(s.k_pool.view(torch.int16), k.view(torch.int16))
    assert (s.out == SENTINEL).all() and (s.lse == SENTINEL).all()
    assert wf.wf_attn_workspace_status(s.ws, s.stream)[0] == wf.WF_OK
    # the same plan buffer serves the next good step
    s2 = Step([20, 3], [2, 30], prefix=50)
    s2.d["plan"] = s.d["plan"]
    s2.run()
    s2.check_tables()
    s2.check_attention()


def test_a_plan_of_another_description_does_nothing():
    s = Step([20, 3], [2, 30], prefix=50)
    k = s.k_pool.clone()
    s.append()   # no plan built yet
    s.attend()
    assert wf.wf_attn_workspace_status(s.ws, s.stream)[0] == wf.WF_ERR_PLAN
    assert (s.out == SENTINEL).all() and torch.equal(s.k_pool.view(torch.int16), k.view(torch.int16))


def test_pages_outside_the_pool_are_not_touched():
    s = Step([20, 3], [2, 30], prefix=50)
    s.d["free_pages"].copy_(torch.where(torch.arange(len(s.free_pages)).cuda() % 2 == 0, 2 ** 31 - 1, -3))
    s.run()
    torch.cuda.synchronize()
    slots = s.d["slot_map"][:s.T]
    assert ((slots == -1) | (slots < s.k_pool.shape[0])).all()
    assert (slots == -1).any()
    assert wf.wf_attn_workspace_status(s.ws, s.stream)[0] == wf.WF_OK
    assert not torch.isnan(s.out[:s.T].float()).any()


def test_host_memory_is_refused():
    s = Step([20, 3], [2, 30], prefix=50).run()
    for name in ("cached", "block_table", "positions"):
        with pytest.raises(wf.WfError) as e:
            s.tables(**{name: s.d[name].cpu()})
        assert e.value.code == wf.WF_ERR_INVALID_ARG
    with pytest.raises(wf.WfError) as e:
        s.tables(plan=s.d["plan"].cpu().pin_memory().data_ptr(), plan_bytes=s.d["plan"].numel())
    assert e.value.code == wf.WF_ERR_INVALID_ARG
    with pytest.raises(wf.WfError) as e:
        wf.wf_batch_attn(s.desc, s.d["plan"], s.d["block_table"], s.prefix_dev, s.q_rot.cpu(), s.k_pool, s.v_pool, s.out,
                         s.lse, workspace=s.ws, stream=s.stream)
    assert e.value.code == wf.WF_ERR_INVALID_ARG
    s.check_attention()  # nothing of it ran


@pytest.mark.parametrize("D", [64, 128])
def test_a_row_of_nans_stays_one_and_alone(D):
    # rows of every kind of unit: narrow, shared, whole tiles, merged parts
    s = Step([200, 3, 900, 0], [1, 9, 1, 300], prefix=500, H=4, Hkv=2, D=D, num_ctas=23)
    s.run()
    s.check_attention()
    out, lse = s.out.clone(), s.lse.clone()
    bad = torch.zeros(s.q_rot.shape[:2], dtype=torch.bool, device="cuda")
    for t, h in ((0, 1), (4, 0), (10, 3), (11, 2), (150, 0), (310, 1)):
        bad[t, h] = True
        s.q_rot[t, h, 5] = float("nan")
    s.attend()
    assert wf.wf_attn_workspace_status(s.ws, s.stream)[0] == wf.WF_OK
    assert torch.isnan(s.out[bad].float()).all() and torch.isnan(s.lse.T[bad]).all()
    assert torch.equal(s.out[~bad], out[~bad]) and torch.equal(s.lse.T[~bad], lse.T[~bad])


def test_an_expired_wait_in_a_fresh_workspace_leaves_other_rows_alone(monkeypatch):
    # whatever the workspace held behind its first 256 bytes, nothing outside the step's rows is written
    for kw in (dict(cached=[0, 7], fresh=[900, 300], num_ctas=23), dict(cached=[300, 20], fresh=[1, 40], prefix=700)):
        s = Step(**kw, spare_tokens=400)
        s.tables()
        s.append()
        s.ws[256:] = 1
        monkeypatch.setenv("WF_WAIT_TIMEOUT_MS", "100")
        monkeypatch.setenv("WF_DEBUG_STALL_FIRST_LOAD", "1")
        s.attend()
        code, _ = wf.wf_attn_workspace_status(s.ws, s.stream)
        monkeypatch.delenv("WF_DEBUG_STALL_FIRST_LOAD")
        monkeypatch.delenv("WF_WAIT_TIMEOUT_MS")
        assert code == wf.WF_ERR_DEVICE_TIMEOUT
        assert (s.out[s.T:] == SENTINEL).all() and (s.lse[:, s.T:] == SENTINEL).all()


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("D,num_ctas", [(128, 0), (64, 23)])
def test_calls_wait_for_what_is_before_them_in_the_stream(D, num_ctas, captured):
    # kernels, copies, fills and a join with another stream stand right before each call, and a reader right behind
    s = Step([200, 3, 900], [1, 9, 300], prefix=500, D=D, num_ctas=num_ctas)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    s.stream = side
    table = s.d["block_table"].clone()
    inputs, want = [], []
    for i in range(2):
        g = torch.Generator(device="cuda")
        g.manual_seed(100 + i)
        inputs.append([torch.randn(x.shape, generator=g, device="cuda").to(torch.bfloat16) for x in (s.q, s.k, s.v)] +
                      [torch.tensor([[1, 9, 300], [5, 0, 130]][i], dtype=torch.int32, device="cuda")])
    busy, pool = torch.zeros(1 << 24, device="cuda"), (s.k_pool.clone(), s.v_pool.clone())

    def step(new, results):
        for dst, src in zip((s.k_pool, s.v_pool), pool):
            dst.copy_(src)
        busy.add_(1)
        s.out.fill_(SENTINEL)
        for name, x in zip(("q", "k", "v"), new):
            getattr(s, name).copy_(x)
        s.d["block_table"].copy_(table)
        s.d["slot_map"].zero_()
        s.d["fresh"].copy_(new[3])
        s.tables()
        results.append(s.d["slot_map"].clone())
        s.k.copy_(new[1])
        s.append()
        other.wait_stream(side)
        with torch.cuda.stream(other):
            busy.mul_(0.5)
            s.lse.fill_(SENTINEL)
        side.wait_stream(other)
        s.attend()
        results.append(s.out.clone())
        results.append(s.lse.clone())
        s.q_rot.zero_()
        s.d["plan"][256:].zero_()  # the next step builds another

    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for i in range(2):
            want.append([])
            step(inputs[i], want[i])
            torch.cuda.synchronize()
            assert not torch.isnan(want[i][1].float()).any() and not torch.equal(want[i][1], torch.full_like(s.out, SENTINEL))
        assert not torch.equal(want[0][1], want[1][1])
        got = [[] for _ in range(8)]
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                for i in range(8):
                    step(inputs[i % 2], got[i])
            for _ in range(3):
                graph.replay()
        else:
            for i in range(8):
                step(inputs[i % 2], got[i])
    torch.cuda.synchronize()
    for i in range(8):
        for a, b in zip(got[i], want[i % 2]):
            assert torch.equal(a, b), i


def test_a_call_may_be_the_first_of_a_graph_and_follow_a_copy_alone():
    s = Step([200, 3], [1, 9], prefix=500).run()
    s.check_attention()
    out, host = s.out.clone(), s.q_rot.cpu().pin_memory()
    side = torch.cuda.Stream()
    s.stream = side
    for before in (lambda: None, lambda: s.q_rot.copy_(host, non_blocking=True), lambda: s.out.zero_()):
        for call in (s.tables, s.append, s.attend):
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                before()
                call()
            if call == s.attend:
                graph.replay()
            torch.cuda.synchronize()
        assert torch.equal(s.out[:s.T], out[:s.T])


def test_a_step_that_needs_no_page_runs_without_free_ones():
    s = Step([20, 3], [2, 5], prefix=50, held=[2, 1])
    s.d["free_pages"] = torch.zeros(0, dtype=torch.int32, device="cuda")
    s.free_head = 0
    s.d["free_head"].zero_()
    s.run()
    s.check_tables()
    s.check_attention()
    s.d["held"].copy_(torch.tensor([2, 0], dtype=torch.int32))
    s.tables()
    assert wf.wf_batch_status(s.d["plan"], s.stream) == wf.WF_ERR_INVALID_ARG  # fewer held than the cached tokens fill
    s.d["held"].copy_(torch.tensor([2, 1], dtype=torch.int32))
    s.d["fresh"].copy_(torch.tensor([2, 14], dtype=torch.int32))
    s.tables()
    assert wf.wf_batch_status(s.d["plan"], s.stream) == wf.WF_ERR_CAPACITY


def test_two_threads_call_at_once():
    import threading
    steps = [Step([900, 20], [1, 30], prefix=1500), Step([5, 60, 7], [200, 1, 2], prefix=300, D=64, H=6, Hkv=3)]
    want = []
    for s in steps:
        s.run()
        s.check_attention()
        want.append((s.out.clone(), s.lse.clone(), s.d["slot_map"].clone()))
    torch.cuda.synchronize()
    failed = []

    def work(s):
        try:
            torch.cuda.set_device(0)
            s.stream = torch.cuda.Stream()
            for _ in range(200):
                s.run()
            s.stream.synchronize()
        except Exception as e:  # noqa: BLE001 (seen by the test below)
            failed.append(e)

    threads = [threading.Thread(target=work, args=(s,)) for s in steps]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for s, w in zip(steps, want):
        for got, x in zip((s.out, s.lse, s.d["slot_map"]), w):
            assert torch.equal(got, x)
