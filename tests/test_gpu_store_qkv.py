"""hpa_store_qkv against the 64-bit definition (oracle/qkv.py, oracle/fourbit.py).

Bounds.  fp32 arithmetic: the row's factor is off by at most 2^-20 of itself (a sum of 128 squares
in a tree, a reciprocal square root and three products), an element by two or three roundings and,
through the transform, seven additions of at most M each: 2^-19 M covers both, with M the
magnitude that the oracle gives.  A rounded result then lies between the roundings of the value
less and plus that error; values are only scaled, by a factor off by 2^-23."""
import numpy as np
import pytest
import torch

import load_balanced_split_gb300 as hpa
from oracle import fourbit, qkv
from oracle.feeder import encode_e4m3_value

pytestmark = pytest.mark.gpu

ERR = 2.0 ** -19
POOL = {"bf16": (torch.bfloat16, (64, 128)), "e4m3": (torch.uint8, (64, 128)),
        "e2m1": (torch.uint8, (hpa.E2M1_PAGE_BYTES,))}


def bf16(x):
    """fp64 to bf16, one rounding (to nearest even), as fp64."""
    x = np.asarray(x, np.float64)
    e = np.floor(np.log2(np.where(x == 0, 1.0, np.abs(x))))
    step = 2.0 ** (np.maximum(e, -126) - 7)
    return np.round(x / step) * step


class Case:
    def __init__(self, n, hq, hkv, kv, rot=128, seed=0, norm=True, pages=None, skip=(), packed=True,
                 scale=None):
        g = torch.Generator().manual_seed(seed)
        self.n, self.hq, self.hkv, self.kv = n, hq, hkv, kv
        P = pages or (n + 63) // 64 + 2
        x = torch.randn(n, hq + 2 * hkv, 128, generator=g)
        x = (x * torch.exp(torch.randn(hq + 2 * hkv, 128, generator=g))).to(torch.bfloat16)
        self.x = x.cuda()
        self.q, self.k, self.v = self.x[:, :hq], self.x[:, hq:hq + hkv], self.x[:, hq + hkv:]
        if not packed:
            self.q, self.k, self.v = (t.contiguous() for t in (self.q, self.k, self.v))
        slots = torch.randperm(P * 64, generator=g)[:n]
        slots[list(skip)] = -1
        self.slots = slots.cuda()
        self.positions = torch.randint(0, 5000, (n,), generator=g, dtype=torch.int32).cuda()
        self.cos_sin = None
        if rot:
            a = torch.arange(5000, dtype=torch.float64)[:, None] * 10000.0 ** (
                -torch.arange(0, rot, 2, dtype=torch.float64) / rot)
            self.cos_sin = torch.cat([a.cos(), a.sin()], 1).float().cuda()
        self.qn = (1 + 0.2 * torch.randn(128, generator=g)).cuda() if norm else None
        self.kn = (1 + 0.2 * torch.randn(128, generator=g)).cuda() if norm else None
        self.ks = self.vs = None
        if kv != "bf16":
            s = (0.5 + torch.rand(2, hkv, generator=g)) / 64 if scale is None else torch.full(
                (2, hkv), scale)
            self.ks, self.vs = s[0].cuda(), s[1].cuda()
        dtype, shape = POOL[kv]
        fill = 0x11 if dtype == torch.uint8 else 7.0
        self.kp = torch.full((P, hkv, *shape), fill, dtype=dtype, device="cuda")
        self.vp = self.kp.clone()
        self.q_out = torch.full((n, hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, eps=1e-6, stream=None, **kw):
        self.how = dict(norm_after=kw.get("norm_after", False),
                        interleaved=kw.get("interleaved", False),
                        use_hadamard=kw.get("use_hadamard", False))
        self.eps = eps
        a = dict(q=self.q, k=self.k, v=self.v, positions=self.positions, slots=self.slots,
                 cos_sin=self.cos_sin, k_pool=self.kp, v_pool=self.vp, q_out=self.q_out,
                 q_norm=self.qn, k_norm=self.kn, eps=eps, k_scale=self.ks, v_scale=self.vs,
                 status=self.status, stream=stream)
        a.update(kw)
        hpa.hpa_store_qkv(**a)
        return self

    def check(self, tokens=None, live=None):
        """The rows of `tokens` (default all) and, exactly, everything that no token writes."""
        torch.cuda.synchronize()
        np_ = lambda t: None if t is None else t.float().cpu().double().numpy()  # noqa: E731
        x, cs = np_(self.x), np_(self.cos_sin)
        slots, pos = self.slots.tolist(), self.positions.tolist()
        live = [t for t in range(self.n) if slots[t] >= 0] if live is None else live
        q_out = np_(self.q_out)
        dead = np.ones(self.n, bool)
        dead[live] = False
        assert (q_out[dead] == 7.0).all()
        how = self.how.values()
        for t in live if tokens is None else tokens:
            for h in range(self.hq):
                y, m = qkv.head(x[t, h], pos[t], cs, np_(self.qn), self.eps, *how)
                self.between(q_out[t, h], y, ERR * m, bf16, ("q", t, h))
        for name, at, pool, scale in (("k", self.hq, self.kp, self.ks),
                                      ("v", self.hq + self.hkv, self.vp, self.vs)):
            raw = pool.cpu()
            used = np.zeros(pool.shape[0] * 64, bool)
            used[[slots[t] for t in live]] = True
            used = used.reshape(-1, 64)
            if self.kv == "e2m1":
                codes, sb = fourbit.unpack(raw.numpy())
                free = np.broadcast_to(~used[:, None, :, None], codes.shape)
                assert (codes[free] == 1).all()
                assert (sb[np.broadcast_to(~used[:, None, :, None], sb.shape)] == 0x11).all()
            else:
                vals = raw.float().numpy() if self.kv == "bf16" else raw.numpy()
                free = np.broadcast_to(~used[:, None, :, None], vals.shape)
                assert (vals[free] == (7.0 if self.kv == "bf16" else 0x11)).all()
                vals = vals.astype(np.float64) if self.kv == "bf16" else raw.view(
                    torch.float8_e4m3fn).double().numpy()
            for t in live if tokens is None else tokens:
                p, s = divmod(slots[t], 64)
                for h in range(self.hkv):
                    if name == "k":
                        y, m = qkv.head(x[t, at + h], pos[t], cs, np_(self.kn), self.eps, *how)
                        e = ERR * m
                    else:
                        y = x[t, at + h]
                        e = np.zeros(128)
                    if scale is not None:
                        r = float(scale[h])
                        y, e = y / r, e / r
                        if np.log2(r) % 1:
                            e = e + 2.0 ** -23 * np.abs(y)
                    what = (name, t, h)
                    if self.kv == "bf16":
                        self.between(vals[p, h, s], y, e, bf16, what)
                    elif self.kv == "e4m3":
                        self.between(vals[p, h, s], y, e, encode_e4m3_value, what)
                    else:
                        self.check_4bit(codes[p, h, s], sb[p, h, s], y, e, what)

    @staticmethod
    def between(got, y, e, rnd, what):
        lo, hi = rnd(y - e), rnd(y + e)
        bad = ~((got >= lo) & (got <= hi))
        assert not bad.any(), (what, np.nonzero(bad)[0][:5], got[bad][:5], y[bad][:5])

    @classmethod
    def check_4bit(cls, codes, sb, y, e, what):
        b = fourbit.e4m3_value(sb)
        yb, eb = np.abs(y).reshape(8, 16), e.reshape(8, 16)
        step = 1 + 2.0 ** -24                            # the rounding of the division by six
        lo = encode_e4m3_value((yb - eb).max(-1).clip(0) / 6 / step)
        hi = encode_e4m3_value((yb + eb).max(-1) / 6 * step)
        assert ((b >= lo) & (b <= hi)).all(), (what, b, lo, hi)
        got = fourbit.decode_e2m1(codes)
        b = np.repeat(b, 16)
        zero = b == 0
        assert (codes[zero] == 0).all()
        b = np.where(zero, 1.0, b)

        def code(v):
            return np.where(zero, 0.0, fourbit.decode_e2m1(fourbit.encode_e2m1(v / b)))
        cls.between(got, y, e, code, what)


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("rot,interleaved", [(128, False), (128, True), (64, False), (64, True),
                                             (32, False), (32, True), (16, False), (16, True),
                                             (0, False)])
@pytest.mark.parametrize("norm_after,use_hadamard", [(False, False), (True, True)])
def test_forms(kv, rot, interleaved, norm_after, use_hadamard):
    Case(9, 6, 3, kv, rot, seed=rot + interleaved, skip=(4,)).run(
        norm_after=norm_after, interleaved=interleaved, use_hadamard=use_hadamard).check()


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 8), (9, 1), (64, 8), (17, 17), (40, 5), (12, 3)])
@pytest.mark.parametrize("n", [1, 5])
def test_head_layouts(kv, hq, hkv, n):
    c = Case(n, hq, hkv, kv, seed=hq, packed=n == 5)
    c.run(norm_after=hq % 2 == 0, use_hadamard=hq > 8).check()
    assert c.status.item() == 0


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "e2m1"])
def test_without_norms(kv):
    Case(20, 4, 2, kv, norm=False, seed=2).run(use_hadamard=True).check()
    c = Case(20, 4, 2, kv, seed=3)
    c.kn = None
    c.run().check()


@pytest.mark.parametrize("n,kv", [(5000, "e4m3"), (20001, "e2m1"), (3001, "bf16")])
def test_many_tokens(n, kv):
    g = np.random.default_rng(n)
    c = Case(n, 16, 4, kv, seed=n, skip=g.integers(0, n, 50))
    c.run(use_hadamard=kv == "e2m1")
    live = set(np.nonzero((c.slots >= 0).cpu().numpy())[0])
    c.check(tokens=sorted(live & (set(g.integers(0, n, 60)) | set(range(n - 8, n)) | {0, 1})))


def test_parts_alone():
    c = Case(30, 10, 2, "e2m1", seed=6)
    c.run(k=None, v=None, k_pool=None, v_pool=None, k_scale=None, v_scale=None, num_pages=3)
    q = c.q_out.clone()
    assert (c.kp == 0x11).all()
    c.q_out.fill_(7.0)
    c.run(q=None, q_out=None)
    assert (c.q_out == 7.0).all()
    c.q_out.copy_(q)
    c.check()


def test_in_place_and_strided_out():
    c = Case(33, 6, 2, "e4m3", seed=7)
    keep, tail = c.x.clone(), c.x[:, 6:].clone()
    c.run(q_out=None)                                 # over the queries of the packed projection
    assert torch.equal(c.x[:, 6:], tail)
    c.q_out.copy_(c.x[:, :6])
    c.x.copy_(keep)
    c.check()
    wide = torch.full((33, 9, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    ref = c.q_out.clone()
    c.run(q_out=wide[:, 2:8])
    assert torch.equal(wide[:, 2:8], ref) and (wide[:, :2] == 5).all() and (wide[:, 8:] == 5).all()


def test_bad_places_are_reported_and_passed_over():
    for kv in ("bf16", "e2m1"):
        for slot, pos, bit in ((-2, 5, 4), (3 * 64, 5, 4), (1 << 40, 5, 4), (-(1 << 62), 5, 4),
                               (7, -1, 1), (7, 5000, 1), (7, 2 ** 31 - 1, 1), (-1, -1, 0)):
            c = Case(6, 3, 1, kv, seed=8, pages=3)
            keep = c.slots.clone()
            keep[keep == 7] = 3 * 64 - 1
            c.slots.copy_(keep)
            c.slots[2], c.positions[2] = slot, pos
            c.run()
            torch.cuda.synchronize()
            assert c.status.item() == bit, (slot, pos)
            c.slots[2] = -1
            c.check(live=[0, 1, 3, 4, 5])


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -6])
def test_ties_and_special_values(scale):
    """Values on the borders between codes, tiny blocks, infinities and NaN, at exact scales."""
    c = Case(16, 1, 1, "e2m1", seed=9, norm=False, rot=0, scale=scale)
    v = torch.zeros(16, 128)
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    for t in range(8):                    # amax 6 b, so the scale is b itself
        b = [1.0, 1.125, 1.25, 1.875, 2.0 ** -9, 2.0 ** -6, 448.0, 13.0][t]
        v[t] = torch.cat([border, -border]).repeat(8) * b * scale
    v[8] = 1e-4 * scale                   # scales that round to zero
    v[9, ::16] = 5000.0 * scale           # beyond the largest scale
    v[9, 1::16] = 3000.0 * scale
    v[10, 5] = float("inf")
    v[10, 6] = 1.0
    v[11, 17] = float("nan")
    v[12] = -0.0
    for t in range(13, 16):
        v[t] = torch.randn(128, generator=torch.Generator().manual_seed(t)) * 10.0 ** (t - 14)
    c.v.copy_(v[:, None].to(torch.bfloat16))
    c.run()
    torch.cuda.synchronize()
    codes, sb = fourbit.unpack(c.vp.cpu().numpy())
    b = fourbit.e4m3_value(sb)
    x = c.v[:, 0].float().cpu().double().numpy() / scale
    for t, slot in enumerate(c.slots.tolist()):
        p, s = divmod(slot, 64)
        got_c, got_b = codes[p, 0, s], b[p, 0, s]
        if t == 10:
            assert got_b[0] == 448 and (got_b[1:] == 0).all()
            assert got_c[5] == 7 and (np.delete(got_c, [5]) == 0).all()
        elif t == 11:
            assert np.isnan(got_b[1]) and not np.isnan(np.delete(got_b, 1)).any()
        else:
            ref_c, ref_b = fourbit.encode(x[t])
            assert (got_b == ref_b).all() and (got_c == ref_c).all(), t


def test_long_pool_offsets():
    """Rows past 2^31 and 2^32 bytes of a pool."""
    P = 70000                                        # 8 heads: 2.58 GB of 4-bit, 4.6 GB of E4M3
    for kv, rowb in (("e2m1", 4608), ("e4m3", 8192)):
        c = Case(4, 1, 8, kv, seed=11, pages=P)
        far = torch.tensor([64 * (P - 1) + 63, 64 * ((1 << 31) // (8 * rowb)) + 1,
                            64 * min(P - 2, (1 << 32) // (8 * rowb)) + 2, 0])
        c.slots.copy_(far)
        c.run()
        torch.cuda.synchronize()
        small = Case(4, 1, 8, kv, seed=11, pages=4)
        for name in ("q", "k", "v", "positions", "qn", "kn", "ks", "vs"):
            setattr(small, name, getattr(c, name))
        small.slots.copy_(torch.tensor([63, 64 + 1, 128 + 2, 192]))
        small.run()
        for i, slot in enumerate(far.tolist()):
            for a, b in ((c.kp, small.kp), (c.vp, small.vp)):
                if kv == "e4m3":
                    assert torch.equal(a[slot // 64, :, slot % 64], b[i, :, (63, 1, 2, 0)[i]])
                else:
                    assert torch.equal(a[slot // 64], b[i])


def test_captured_on_a_stream():
    c = Case(40, 8, 2, "e2m1", seed=12)
    c.run()
    torch.cuda.synchronize()
    kp, vp, q = c.kp.clone(), c.vp.clone(), c.q_out.clone()
    c.kp.fill_(0x11), c.vp.fill_(0x11), c.q_out.fill_(7.0)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        c.run()
    assert (c.q_out == 7.0).all()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(kp, c.kp) and torch.equal(vp, c.vp) and torch.equal(q, c.q_out)
    c.slots[10:] = -1                                # fewer tokens in the same graph
    c.kp.fill_(0x11), c.vp.fill_(0x11), c.q_out.fill_(7.0)
    graph.replay()
    c.check()


def test_no_tokens():
    c = Case(1, 2, 1, "bf16")
    e = c.q[:0]
    hpa.hpa_store_qkv(e, c.k[:0], c.v[:0], c.positions[:0], c.slots[:0], c.cos_sin, c.kp, c.vp)
    torch.cuda.synchronize()
    assert (c.kp == 7).all()


def test_binding_shapes():
    c = Case(8, 4, 2, "e2m1", seed=13)
    for kw, text in ((dict(q=c.q[:7]), "tokens"), (dict(k=c.k[..., :64]), "128"),
                     (dict(q=c.x[:, ::2][:, :4]), "contiguous"), (dict(slots=c.slots[:7]), "per token"),
                     (dict(v=c.x[:, 5:8]), "same heads"), (dict(k_pool=c.kp[:, :1].contiguous()), "match"),
                     (dict(q_norm=c.qn[:64]), "128"), (dict(k_scale=c.ks[:1]), "k_scale"),
                     (dict(v_scale=None), "CUDA tensor"), (dict(k_pool=None), "pools"),
                     (dict(k_pool=c.kp[..., :4096].contiguous(), v_pool=c.vp[..., :4096].contiguous()),
                      "match"), (dict(slots=c.slots.int()), "int64"), (dict(q=c.q.float()), "bfloat16"),
                     (dict(cos_sin=c.cos_sin[:, :0]), "cos_sin"), (dict(cos_sin=c.cos_sin[:, :96].contiguous()),
                                                                    "failed")):
        with pytest.raises(hpa.HpaError, match=text):
            c.run(**kw)
    assert (c.kp == 0x11).all()
