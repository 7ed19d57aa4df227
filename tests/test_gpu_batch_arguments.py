"""Refusals of the batch calls, each from a call that is first seen to succeed
and of which one argument is then changed: a check that was missing would let
the changed call through (or refuse it for another reason than the one named)."""
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


class Calls:
    """The three calls of a step, argument by argument."""

    def __init__(self, **kw):
        s = self.step = Step([20, 3, 0], [2, 30, 1], prefix=50, held=[2, 1, 0], **kw)
        self.f = dict(tables=wf.wf_batch_tables, append=wf.wf_batch_append, attn=wf.wf_batch_attn)
        self.args = dict(
            tables=dict(s.d),
            append=dict(plan=s.d["plan"], slot_map=s.d["slot_map"], k=s.k, v=s.v, k_pool=s.k_pool, v_pool=s.v_pool, q=s.q,
                        rope=s.rope, q_rot=s.q_rot),
            attn=dict(plan=s.d["plan"], block_table=s.d["block_table"], prefix_table=s.prefix_dev, q=s.q_rot,
                      k_pool=s.k_pool, v_pool=s.v_pool, out=s.out, lse=s.lse, workspace=s.ws))

    def __call__(self, call, **change):
        self.f[call](self.step.desc, **{**self.args[call], "stream": self.step.stream, **change})

    def good(self):
        for call in self.f:
            self(call)
        return self.step

    def refused(self, call, code=wf.WF_ERR_INVALID_ARG, **change):
        with pytest.raises(wf.WfError) as e:
            self(call, **change)
        assert e.value.code == code, str(e.value)
        return str(e.value)

    def check(self):
        """The step's results are those of the good calls: no refused one ran."""
        self.step.check_tables()
        self.step.check_attention()


OTHERS = {torch.int32: (torch.float32, torch.uint32, torch.int64), torch.float32: (torch.int32, torch.float64),
          torch.bfloat16: (torch.float16, torch.int16, torch.float32), torch.uint8: (torch.int16, torch.float32)}


def test_tensors_of_other_types_are_refused():
    c = Calls()
    c.good()
    for call, args in c.args.items():
        for name, x in args.items():
            for t in OTHERS[x.dtype]:
                other = torch.zeros(x.shape, dtype=t, device="cuda")
                assert f"{name} is of type" in c.refused(call, **{name: other}), (call, name, t)
    c.check()


def test_rows_of_another_length_are_refused():
    c = Calls()
    c.good()
    cols, cap = c.step.desc.max_request_pages, c.step.desc.max_tokens
    zeros = lambda t, *shape: torch.zeros(*shape, dtype=t, device="cuda")  # noqa: E731
    for call, name, x in (("tables", "block_table", zeros(torch.int32, 3, cols + 1)),
                          ("attn", "block_table", zeros(torch.int32, 3, cols + 1)),
                          ("attn", "lse", zeros(torch.float32, 4, cap + 1)),
                          ("attn", "q", zeros(torch.bfloat16, cap, 5, 128)),
                          ("attn", "out", zeros(torch.bfloat16, cap, 128, 4)),
                          ("append", "k_pool", zeros(torch.bfloat16, c.step.k_pool.shape[0], 3, 128)),
                          ("append", "rope", zeros(torch.float32, cap, 2, 64))):
        assert f"{name} is of shape" in c.refused(call, **{name: x}), (call, name)
    # flattened, the same memory is taken
    pool = lambda x: x.view(-1, c.step.page, 2, 128)  # noqa: E731
    for call in ("append", "attn"):
        c(call, q=c.step.q.view(cap, -1) if call == "append" else c.step.q_rot.flatten(),
          k_pool=pool(c.step.k_pool), v_pool=pool(c.step.v_pool))
    c.check()


def test_a_size_above_the_tensors_is_refused():
    c = Calls()
    c.good()
    plan, ws = c.step.d["plan"], c.step.ws
    c("tables", plan_bytes=plan.numel())
    c("attn", workspace_bytes=ws.numel())
    for n in (plan.numel() + 1, 1 << 40):
        assert "plan_bytes is more" in c.refused("tables", plan_bytes=n)
    for n in (ws.numel() + 1, 1 << 40):
        assert "workspace_bytes is more" in c.refused("attn", workspace_bytes=n)
    assert "num_free is more" in c.refused("tables", num_free=c.step.d["free_pages"].numel() + 1)
    c.refused("tables", wf.WF_ERR_WORKSPACE, plan_bytes=plan.numel() - 257)
    c.refused("attn", wf.WF_ERR_WORKSPACE, workspace_bytes=ws.numel() - 257)
    c.check()


@pytest.mark.parametrize("change", [dict(block=2), dict(page=32), dict(H=8, Hkv=4), dict(spare_tokens=4),
                                    dict(num_ctas=255), dict(D=64), dict(spare_cols=2), dict(smallest=True)])
def test_a_plan_built_for_another_description_does_nothing(change):
    # 256 blocks, more than any other plan here has shares
    s = Step([20, 3], [2, 30], prefix=50, num_ctas=256)
    other = Step([0], [1], H=1, Hkv=1, D=64, page=8, num_ctas=1, spare_tokens=0, spare_cols=0) \
        if change.pop("smallest", False) else Step([20, 3], [2, 30], prefix=50, **{"num_ctas": 256, **change})
    # (in a buffer of its own, so that the room of a plan of the call's description meets none of its results)
    buffer = torch.zeros(other.d["plan"].numel() + s.d["plan"].numel(), dtype=torch.uint8, device="cuda")
    other.d["plan"] = buffer[:other.d["plan"].numel()]
    other.tables()
    s.tables()  # (the slots; its own plan stays unused)
    k, v = s.k_pool.clone(), s.v_pool.clone()
    wf.wf_batch_append(s.desc, other.d["plan"], s.d["slot_map"], s.k, s.v, s.k_pool, s.v_pool, q=s.q, rope=s.rope,
                       q_rot=s.q_rot, stream=s.stream)
    wf.wf_batch_attn(s.desc, other.d["plan"], s.d["block_table"], s.prefix_dev, s.q, s.k_pool, s.v_pool, s.out, s.lse,
                     workspace=s.ws, stream=s.stream)
    assert wf.wf_attn_workspace_status(s.ws, s.stream)[0] == wf.WF_ERR_PLAN
    assert (s.out == SENTINEL).all() and (s.lse == SENTINEL).all() and (s.q_rot == SENTINEL).all()
    for now, before in ((s.k_pool, k), (s.v_pool, v)):
        assert torch.equal(now.view(torch.int16), before.view(torch.int16))
    # nothing is left of it: the step's own plan still serves
    wf.wf_attn_workspace_init(s.ws, s.stream)
    s.append()
    s.attend()
    s.check_attention()


INPUTS = dict(tables=("cached", "fresh", "prefix_len", "held", "free_pages", "free_head"),
              append=("plan", "slot_map", "rope", "q", "k", "v"),
              attn=("plan", "block_table", "prefix_table", "q", "k_pool", "v_pool"))
OUTPUTS = dict(tables=("free_head_out", "held_out", "block_table", "token_start", "slot_map", "positions", "plan"),
               append=("q_rot", "k_pool", "v_pool"), attn=("out", "lse", "workspace"))


@pytest.mark.parametrize("call", ["tables", "append", "attn"])
def test_results_that_share_memory_are_refused(call):
    c = Calls()
    c.good()
    args = c.args[call]
    nbytes = {name: x.numel() * x.element_size() for name, x in args.items()}
    why = f"wf_batch_{call}: {wf.status_string(wf.WF_ERR_INVALID_ARG)}"  # the library's own, not the binding's
    for o in OUTPUTS[call]:
        for i in INPUTS[call] + OUTPUTS[call][:OUTPUTS[call].index(o)]:
            # b begins where a does, or in a's last 16 (or 4) bytes
            for a, b in ((o, i), (i, o)):
                for at in (0, nbytes[a] - (16 if nbytes[a] % 16 == 0 else 4)):
                    if at == 0 and {a, b} == {"q", "q_rot"}:
                        continue  # in place
                    raw = torch.zeros(nbytes[a] + nbytes[b], dtype=torch.uint8, device="cuda")
                    views = {a: raw[:nbytes[a]], b: raw[at:at + nbytes[b]]}
                    views = {n: x.view(args[n].dtype).view(args[n].shape) for n, x in views.items()}
                    assert c.refused(call, **views) == why, (a, b, at)
    c.check()


def test_buffers_right_behind_one_another_are_taken():
    c = Calls()
    s = c.step
    tensors = [(s.d, n) for n in s.d] + [(s.__dict__, n) for n in ("k_pool", "v_pool", "q", "k", "v", "rope", "q_rot", "out",
                                                                   "lse", "ws", "prefix_dev")]
    sizes = [-(-where[n].numel() * where[n].element_size() // 16) * 16 for where, n in tensors]
    arena = torch.zeros(sum(sizes), dtype=torch.uint8, device="cuda")
    for (where, n), size in zip(tensors, sizes):
        x, (part, arena) = where[n], arena.split([size, arena.numel() - size])
        where[n] = part[:x.numel() * x.element_size()].view(x.dtype).view(x.shape)
        where[n].copy_(x)
    k, v = s.k_pool.clone(), s.v_pool.clone()
    s.tables()
    s.append()
    s.attend()
    s.check_tables()
    s.check_append(k, v)
    s.check_attention()


def test_a_plan_may_be_an_address_beside_tensors():
    c = Calls()
    plan = c.step.d["plan"]
    c("tables", plan=plan.data_ptr(), plan_bytes=plan.numel())
    c("append", plan=plan.data_ptr())
    c("attn", plan=plan.data_ptr())
    c.check()
    for call, name in (("tables", "fresh"), ("append", "k"), ("attn", "out")):
        extra = dict(plan_bytes=plan.numel()) if call == "tables" else {}
        assert "on the current GPU" in c.refused(call, plan=plan.data_ptr(), **{name: c.args[call][name].cpu()}, **extra)
    if torch.cuda.device_count() > 1:
        with torch.cuda.device(1):
            for call in c.args:
                extra = dict(plan_bytes=plan.numel()) if call == "tables" else {}
                assert "on the current GPU" in c.refused(call, plan=plan.data_ptr(), **extra)
    c.check()


# ---------------------------------------------------------------- the library's own refusals
def own(call, code):
    return f"wf_batch_{call}: {wf.status_string(code)}"


NEEDED = dict(tables=("cached", "fresh", "prefix_len", "free_pages", "free_head", "free_head_out", "block_table",
                      "token_start", "slot_map", "positions", "plan"),
              append=("plan", "slot_map", "k", "v", "k_pool", "v_pool", "q", "rope", "q_rot"),
              attn=("plan", "block_table", "prefix_table", "q", "k_pool", "v_pool", "out", "workspace"))


@pytest.mark.parametrize("call,change", [
    *[(call, {name: None}) for call, names in NEEDED.items() for name in names],
    ("tables", dict(held=None)), ("tables", dict(held_out=None)), ("tables", dict(num_free=-1)),
    ("append", dict(rope=None, q_rot=None)), ("append", dict(rope=None, q=None)),
    ("append", dict(q=None, q_rot=None)),
    *[("attn", dict(softmax_scale=x)) for x in (-1.0, -0.5, float("nan"), float("inf"), float("-inf"))],
])
def test_the_library_refuses(call, change):
    c = Calls()
    c.good()
    extra = {}
    if change.get("free_pages", 0) is None:
        extra["num_free"] = c.step.d["free_pages"].numel()
    if call == "tables" and change.get("plan", 0) is None:
        extra["plan_bytes"] = c.step.d["plan"].numel()
    if change.get("workspace", 0) is None:
        extra["workspace_bytes"] = c.step.ws.numel()
    # (a number for the missing buffer is not what is refused: with the buffer the call goes through)
    c(call, **extra)
    assert c.refused(call, **change, **extra) == own(call, wf.WF_ERR_INVALID_ARG)
    c.check()


def test_what_may_be_left_out():
    c = Calls()
    c.good()
    c("attn", lse=None)
    c("tables", held=None, held_out=None)
    s = Step([20, 3], [2, 30], rope=False)  # no prefix, no angles
    s.d["prefix_len"] = None
    s.run()
    s.check_attention()


@pytest.mark.parametrize("call,name", [(call, n) for call, names in dict(
    tables=("plan",), append=("plan", "k", "v", "k_pool", "v_pool", "q", "rope", "q_rot"),
    attn=("plan", "q", "k_pool", "v_pool", "out", "workspace")).items() for n in names])
def test_buffers_off_their_boundary_are_refused(call, name):
    c = Calls()
    c.good()
    x = c.args[call][name]
    n = x.numel() * x.element_size()
    raw = torch.zeros(n + 64, dtype=torch.uint8, device="cuda")
    at = lambda by: raw[by:by + n].view(x.dtype).view(x.shape)  # noqa: E731
    at(16).copy_(x)
    if name not in ("q_rot", "out"):  # (on its boundary it is taken)
        c(call, **{name: at(16)})
    for by in (4, 8, 24):
        assert c.refused(call, wf.WF_ERR_ALIGNMENT, **{name: at(by)}) == own(call, wf.WF_ERR_ALIGNMENT)
    c.check()


@pytest.mark.parametrize("call,name", [("tables", n) for n in INPUTS["tables"] + OUTPUTS["tables"][:-1]] +
                         [("append", "slot_map"), ("attn", "block_table"), ("attn", "prefix_table"), ("attn", "lse")])
def test_addresses_off_a_word_are_refused(call, name):
    # (no tensor of 4-byte elements lies so: addresses)
    c = Calls()
    c.good()
    args = {n: x.data_ptr() for n, x in c.args[call].items()}
    if call == "tables":
        args.update(num_free=c.step.d["free_pages"].numel(), plan_bytes=c.step.d["plan"].numel())
    if call == "attn":
        args["workspace_bytes"] = c.step.ws.numel()
    c(call, **args)
    # into the middle of a buffer of its own, as long twice
    raw = torch.zeros(2 * c.args[call][name].numel() * 4 + 64, dtype=torch.uint8, device="cuda")
    for by in (1, 2, 3):
        assert c.refused(call, wf.WF_ERR_ALIGNMENT, **{**args, name: raw.data_ptr() + 16 + by}) == \
            own(call, wf.WF_ERR_ALIGNMENT)
    c.check()


# ---------------------------------------------------------------- room and layout
@pytest.mark.parametrize("call", ["tables", "append", "attn"])
def test_tensors_too_small_or_strided_are_refused(call):
    c = Calls()
    c.good()
    for name, x in c.args[call].items():
        short = x.flatten()[:x.numel() - 1].clone()
        wide = torch.zeros(2 * x.numel(), dtype=x.dtype, device="cuda")[::2]
        if name in ("plan", "workspace"):
            # (their sizes are the library's to judge; of a plan that is only read, what every plan holds is asked for)
            if call == "tables" or name == "workspace":
                assert c.refused(call, wf.WF_ERR_WORKSPACE, **{name: short}) == own(call, wf.WF_ERR_WORKSPACE)
            if name == "plan":
                assert "2304 are needed" in c.refused(call, plan=x[:2303])
        elif name == "free_pages":
            assert "num_free is more" in c.refused(call, free_pages=short, num_free=x.numel())
        else:
            why = c.refused(call, **{name: short})
            assert f"{name} has {x.numel() - 1} elements" in why and f"{x.numel()} are needed" in why, why
        if x.numel() > 1:
            assert f"{name} has {x.numel()} elements on cuda:0, not dense" in c.refused(call, **{name: wide})
    c.check()


@pytest.mark.parametrize("call", ["tables", "append", "attn"])
def test_host_tensors_are_refused(call):
    c = Calls()
    c.good()
    for name, x in c.args[call].items():
        for host in (x.cpu(), x.cpu().pin_memory()):
            assert f"{name} has {x.numel()} elements on cpu" in c.refused(call, **{name: host}), name
    pinned = c.step.d["plan"].cpu().pin_memory()
    extra = dict(plan_bytes=pinned.numel()) if call == "tables" else {}
    assert c.refused(call, plan=pinned.data_ptr(), **extra) == own(call, wf.WF_ERR_INVALID_ARG)
    c.check()
