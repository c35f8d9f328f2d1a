"""A serving loop from request lengths to outputs: page tables (PageTable), the writer
(hpa_store_qkv) and attention (decode_step) in turn, with sessions that begin, grow, draft and
end, against the definitions in 64 bits (oracle/paging.py, oracle/qkv.py, oracle/bounded.py)."""
import random
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import load_balanced_split_gb300 as hpa
from bounded_helpers import check_attention
from oracle import bounded, paging
from test_gpu_store_qkv import POOL, Case

pytestmark = pytest.mark.gpu

HQ, HKV, ROWS, STRIDE, P = 16, 2, 9, 12, 70


class Loop:
    def __init__(self, kv, q_len, window, seed):
        self.kv, self.q_len, self.window = kv, q_len, window
        self.rng, self.g = random.Random(seed), torch.Generator().manual_seed(seed)
        self.pt = hpa.PageTable(P, ROWS, STRIDE, max_tokens=900)
        self.state = ([[0] * STRIDE for _ in range(ROWS)], [0] * ROWS, list(range(P - 1, -1, -1)))
        dtype, shape = POOL[kv]
        self.kp = torch.zeros((P, HKV, *shape), dtype=dtype, device="cuda")
        self.vp = torch.zeros_like(self.kp)
        a = torch.arange(1000, dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(0, 128, 2, dtype=torch.float64) / 128)
        self.cos_sin = torch.cat([a.cos(), a.sin()], 1).float().cuda()
        self.qn, self.kn = ((1 + 0.2 * torch.randn(128, generator=self.g)).cuda() for _ in "qk")
        s = (0.5 + torch.rand(2, HKV, generator=self.g)) / 64
        self.ks, self.vs = (None, None) if kv == "bf16" else (s[0].cuda(), s[1].cuda())

    def store(self, rows, lens, new):
        """One step of tables and writer for these sessions; the queries of their new tokens."""
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.lens, self.rows = i32(lens), i32(rows)
        self.pt.assign(self.lens, i32(new), rows=self.rows)
        self.state, (indptr, ix), (slots, pos), status = paging.assign(
            lens, new, *self.state, P, rows, None, 900)
        assert status == 0 and self.pt.status.item() == 0
        n = 900                                          # the writer takes the whole buffer
        x = torch.randn(n, HQ + 2 * HKV, 128, generator=self.g).to(torch.bfloat16).cuda()
        q = torch.full((n, HQ, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        hpa.hpa_store_qkv(x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], self.pt.positions,
                          self.pt.slots, self.cos_sin, self.kp, self.vp, q, self.qn, self.kn,
                          use_hadamard=True, k_scale=self.ks, v_scale=self.vs, status=self.pt.status)
        assert self.pt.status.item() == 0
        self.check_rows(x, q, slots, pos, sum(new))
        self.indptr, self.ix = indptr, ix
        return q[:sum(new)]

    def check_rows(self, x, q, slots, pos, n):
        """Some of the tokens' queries and cache rows, as the writer's own tests check them."""
        c = Case.__new__(Case)
        c.n, c.hq, c.hkv, c.kv, c.x, c.q_out = len(slots), HQ, HKV, self.kv, x, q
        c.slots, c.positions = torch.tensor(slots), torch.tensor(pos)
        c.cos_sin, c.qn, c.kn, c.ks, c.vs, c.kp, c.vp = (self.cos_sin, self.qn, self.kn, self.ks,
                                                         self.vs, self.kp.clone(), self.vp.clone())
        c.how, c.eps = dict(norm_after=False, interleaved=False, use_hadamard=True), 1e-6
        used = torch.zeros(P * 64, dtype=torch.bool)
        used[slots[:n]] = True
        for pool in (c.kp, c.vp):                        # what other tokens wrote is not this step's
            free = (~used).view(P, 64).cuda()
            if self.kv == "e2m1":
                pool[..., :4096].unflatten(-1, (64, 64)).permute(0, 2, 1, 3)[free] = 0x11
                pool[..., 4096:].unflatten(-1, (64, 8)).permute(0, 2, 1, 3)[free] = 0x11
            else:
                pool.permute(0, 2, 1, 3)[free] = 7.0 if self.kv == "bf16" else 0x11
        c.check(tokens=sorted({0, n - 1, n // 2}))

    def attend(self, q):
        B = self.lens.numel()
        kv = dict(bf16=hpa.KV_BF16, e4m3=hpa.KV_E4M3, e2m1=hpa.KV_E2M1)[self.kv]
        more = dict(window=self.window, sinks=3) if self.window else {}
        count = hpa.hpa_default_num_ctas_window if self.window else hpa.hpa_default_num_ctas
        ws = hpa.Workspace(B, self.q_len, HQ, 128, Hkv=HKV,
                           num_ctas=count(HKV, self.q_len, kv, HQ), **more)
        out = torch.empty((B, self.q_len, HQ, 128), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((B, self.q_len, HQ), device="cuda")
        q = q.view(B, self.q_len, HQ, 128)
        hpa.decode_step(ws, q, self.kp, self.vp, self.lens, self.pt.page_indptr,
                        self.pt.page_indices, out, lse, self.ks, self.vs)
        assert ws.status() == 0
        host = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
        b = SimpleNamespace(B=B, q_len=self.q_len, Hq=HQ, Hkv=HKV, d=128, kv_dtype=self.kv,
                            seq_lens=host(self.lens), page_indptr=np.array(self.indptr),
                            page_indices=np.array(self.ix), q=q.cpu(), k_pool=self.kp.cpu(),
                            v_pool=self.vp.cpu(), k_scale=host(self.ks), v_scale=host(self.vs))
        check_attention(b, out, lse, bounded.attention_rows(b, self.window, 3 if self.window else 0),
                        self.kv)


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("q_len,window", [(1, None), (2, None), (1, 90)])
def test_serving(kv, q_len, window):
    loop = Loop(kv, q_len, window, seed=q_len + (window or 0))
    length = {}
    for step in range(9):
        # sessions end, others begin with a prompt, in one batch of tables and rows
        for r in list(length):
            if loop.rng.random() < 0.15:
                loop.pt.assign(torch.zeros(1, dtype=torch.int32, device="cuda"),
                               rows=torch.tensor([r], dtype=torch.int32, device="cuda"))
                loop.state = paging.assign([0], None, *loop.state, P, [r])[0]
                del length[r]
        start = [r for r in range(ROWS) if r not in length][:2 if step else 4]
        prompts = [loop.rng.choice([1, 63, 64, 65, loop.rng.randint(1, 300)]) for _ in start]
        if start:
            loop.store(start, prompts, prompts)
            length.update(zip(start, prompts))
        # then every session decodes, in any order
        rows = loop.rng.sample(sorted(length), len(length))
        for r in rows:
            length[r] += q_len
        q = loop.store(rows, [length[r] for r in rows], [q_len] * len(rows))
        loop.attend(q)
        if q_len > 1 and step % 2:                       # a draft token is rejected
            for r in rows[::2]:
                length[r] -= 1
