"""One step of a batch of requests on the GPU, built from lists of lengths, and
the error bounds that its results are held to."""
from __future__ import annotations

import numpy as np
import torch

from chunk_causal_attention_block_b200 import wf
from oracle import batch_oracle as orc

HALF_BF16 = 2.0 ** -8  # half a step of bf16, relative
SENTINEL = -123.0


class Step:
    """Buffers of one step.  The pool holds `poison` wherever no token of the step's requests or of the prefix lies."""

    def __init__(self, cached, fresh, prefix=0, H=4, Hkv=2, D=128, page=16, block=1, num_ctas=0, seed=0, spare_tokens=3,
                 spare_cols=1, poison=float("nan"), held=None, scale=0.0, rope=True, far_pages=0):
        self.cached, self.fresh, self.prefix = list(cached), list(fresh), prefix
        self.H, self.Hkv, self.D, self.page, self.block, self.scale = H, Hkv, D, page, block, scale
        self.far_pages = far_pages
        rng = np.random.default_rng(seed)
        B, self.T = len(cached), sum(fresh)
        have = [-(-c // page) for c in cached] if held is None else list(held)
        self.held = None if held is None else list(held)
        need = [max(h, -(-(c + f) // page)) for h, c, f in zip(have, cached, fresh)]
        cols = max(1, max(need)) + spare_cols
        pp = -(-prefix // page)
        # far_pages: that many pages lie unused before the first
        pool_pages = far_pages + pp + sum(need) + 5
        order = far_pages + rng.permutation(pool_pages - far_pages)
        self.prefix_table = order[:pp]
        at = pp
        self.table = np.full((B, cols), -7)
        for b, h in enumerate(have):
            self.table[b, :h] = order[at:at + h]
            at += h
        self.free_head = 2
        self.free_pages = np.concatenate([[-1, -1], order[at:]])
        self.desc = wf.make_batch_desc(H, Hkv, D, page, pool_pages, max_requests=B, max_tokens=max(1, self.T + spare_tokens),
                                       max_request_pages=cols, max_prefix_pages=pp, block_tokens=block, num_ctas=num_ctas)
        cap = self.desc.max_tokens
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + 1)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
        i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
        self.d = dict(cached=i32(cached), fresh=i32(fresh), prefix_len=i32([prefix]), free_pages=i32(self.free_pages),
                      free_head=i32([self.free_head]), free_head_out=i32([-1]), block_table=i32(self.table),
                      token_start=i32([-1] * (B + 1)), slot_map=i32([-9] * cap), positions=i32([-9] * cap),
                      plan=torch.zeros(wf.wf_batch_plan_bytes(self.desc), dtype=torch.uint8, device="cuda"))
        if held is not None:
            self.d.update(held=i32(held), held_out=i32([-1] * B))
        self.prefix_dev = i32(self.prefix_table) if pp else None
        tokens = pool_pages * page
        self.k_pool = torch.full((tokens, Hkv, D), poison, dtype=torch.bfloat16, device="cuda")
        self.v_pool = torch.full((tokens, Hkv, D), poison, dtype=torch.bfloat16, device="cuda")
        stored = [orc.page_tokens(self.prefix_table, prefix, page)]
        stored += [orc.page_tokens(self.table[b], c, page) for b, c in enumerate(cached)]
        stored = torch.tensor(np.concatenate(stored).astype(np.int64), device="cuda")
        self.k_pool[stored], self.v_pool[stored] = rand(len(stored), Hkv, D), rand(len(stored), Hkv, D)
        self.q, self.k, self.v = rand(cap, H, D), rand(cap, Hkv, D), rand(cap, Hkv, D)
        self.rope = None
        if rope:
            angle = torch.rand(cap, D // 2, generator=g, device="cuda", dtype=torch.float64) * 6.3
            self.rope = torch.stack([angle.cos(), angle.sin()], -1).float().contiguous()
        self.q_rot = torch.full_like(self.q, SENTINEL) if rope else None
        self.out = torch.full_like(self.q, SENTINEL)
        self.lse = torch.full((H, cap), SENTINEL, dtype=torch.float32, device="cuda")
        self.ws = torch.zeros(wf.wf_batch_workspace_bytes(self.desc), dtype=torch.uint8, device="cuda")
        self.stream = torch.cuda.current_stream()

    # ------------------------------------------------------------- calls
    def tables(self, **kw):
        wf.wf_batch_tables(self.desc, stream=self.stream, **{**self.d, **kw})

    def append(self):
        wf.wf_batch_append(self.desc, self.d["plan"], self.d["slot_map"], self.k, self.v, self.k_pool, self.v_pool,
                           q=self.q if self.rope is not None else None, rope=self.rope, q_rot=self.q_rot,
                           stream=self.stream)

    def attend(self):
        wf.wf_batch_attn(self.desc, self.d["plan"], self.d["block_table"], self.prefix_dev,
                         self.q if self.rope is None else self.q_rot, self.k_pool, self.v_pool, self.out, self.lse,
                         softmax_scale=self.scale, workspace=self.ws, stream=self.stream)

    def run(self):
        self.tables()
        self.append()
        self.attend()
        return self

    # ------------------------------------------------------------- checks
    def check_tables(self):
        table, start, slots, pos, head, held = orc.tables(self.cached, self.fresh, self.prefix, self.page,
                                                          self.free_pages, self.free_head, self.table, self.held)
        got = {k: self.d[k].cpu().numpy() for k in ("block_table", "token_start", "slot_map", "positions", "free_head_out")}
        np.testing.assert_array_equal(got["block_table"], table)
        np.testing.assert_array_equal(got["token_start"], start)
        np.testing.assert_array_equal(got["slot_map"][:self.T], slots)
        np.testing.assert_array_equal(got["positions"][:self.T], pos)
        assert (got["slot_map"][self.T:] == -9).all() and (got["positions"][self.T:] == -9).all()
        assert got["free_head_out"].tolist() == [head]
        if self.held is not None:
            np.testing.assert_array_equal(self.d["held_out"].cpu().numpy(), held)
        assert wf.wf_batch_status(self.d["plan"], self.stream) == wf.WF_OK

    def check_append(self, k_before, v_before):
        slots = self.d["slot_map"][:self.T].long()
        keep = torch.ones(self.k_pool.shape[0], dtype=torch.bool, device="cuda")
        keep[slots] = False
        for now, before in ((self.k_pool, k_before), (self.v_pool, v_before)):
            assert torch.equal(now[keep].view(torch.int16), before[keep].view(torch.int16)), "another slot was written"
        assert torch.equal(self.v_pool[slots], self.v[:self.T])
        if self.rope is None:
            assert torch.equal(self.k_pool[slots], self.k[:self.T])
            return
        assert (self.q_rot[self.T:] == SENTINEL).all()
        cs = self.rope[:self.T].cpu().numpy()
        for got, raw in ((self.k_pool[slots], self.k[:self.T]), (self.q_rot[:self.T], self.q[:self.T])):
            raw = raw.double().cpu().numpy()
            want = orc.rotate(raw, cs)
            # two products and a sum in fp32 (half a step each, of at most |x| + |y|), then one rounding to bf16
            size = np.repeat(np.abs(raw[..., 0::2]) + np.abs(raw[..., 1::2]), 2, axis=-1)
            err32 = 3 * 2.0 ** -24 * size
            bound = HALF_BF16 * (np.abs(want) + err32) + err32
            assert (np.abs(got.double().cpu().numpy() - want) <= bound).all()

    def check_attention(self, what=""):
        code, detail = wf.wf_attn_workspace_status(self.ws, self.stream)
        assert code == wf.WF_OK, (what, code, detail)
        assert (self.out[self.T:] == SENTINEL).all() and (self.lse[:, self.T:] == SENTINEL).all(), what
        if self.T == 0:
            return
        q = self.q if self.rope is None else self.q_rot
        skip = self.far_pages * self.page
        k, v = (x[skip:].double().cpu().numpy() for x in (self.k_pool, self.v_pool))
        ref = orc.attention(q[:self.T].double().cpu().numpy(), k, v, self.cached, self.fresh, self.prefix,
                            self.d["block_table"].cpu().numpy() - self.far_pages, self.prefix_table - self.far_pages,
                            self.page, self.block, self.scale or None)
        out = self.out[:self.T].double().cpu().numpy()
        lse = self.lse[:, :self.T].double().cpu().numpy()
        # scores: D products added in fp32, at most a whole step each (the tensor cores may truncate)
        score = 2.0 ** -23 * self.D * ref["Z"]
        # log2 domain: the scaled score, the maximum and exp2's argument are each rounded once (of at most
        # 1.5 |s| + 8), exp2 and log2 are good to 2^-21, sums of the keys' fp32 values to 2^-20
        approx = 2.0 ** -23 * (1.5 * np.maximum(ref["Z"], np.abs(ref["LSE"])) + 8) * 3 + 2.0 ** -19
        lse_bound = score + approx
        assert (np.abs(lse - ref["LSE"]) <= lse_bound).all(), (what, np.abs(lse - ref["LSE"]).max(), lse_bound.max())
        # O: P rounded to bf16 (half a step of every p |v|), weights off by the scores' errors (numerator and sum),
        # then one rounding of O
        soft = (HALF_BF16 + 2 * lse_bound.T[..., None] + 2.0 ** -18) * ref["A"]
        bound = soft + HALF_BF16 * (np.abs(ref["O"]) + soft)
        err = np.abs(out - ref["O"])
        assert (err <= bound).all(), (what, err.max(), np.argwhere(~(err <= bound))[:4].tolist())
