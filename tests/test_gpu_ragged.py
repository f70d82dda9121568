"""The ragged-step calls (GPU) against their definitions in 64 bits: the plan of
pages and slots, the normalised append, the query norm and rotation, and the
attention of every request's new tokens over its paged cache.

Tolerances.  A rounding to a type is off by at most half a step, u =
finfo.eps / 2 of the value (bf16 2^-8, fp32 2^-24).  The attention rounds its
weights and its output once each (bf16); its scores are fp32 sums of d products,
off by at most d 2^-24 sum |q k|, which scales every weight by at most
exp(2 s d 2^-24 sum |q k|); the exponentials and sums add a few 2^-22.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
DEV = "cuda"


@pytest.fixture(scope="module")
def mla():
    from head_latent_attention_append_b200 import mla as m
    return m


def dims_of(mla, dtype, n_h, d_h, d_c, d_r, d_cq=0, **kw):
    return mla.make_dims(n_h, d_h, d_h, d_c, d_r, 256, d_cq, dtype=mla.BF16 if dtype == "bf16" else mla.F32, **kw)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------------- plan
def plan_reference(new, past, free, table, num_pages, rows):
    """Request by request, token by token."""
    B, width = table.shape
    table = table.copy()
    q_start, kv, seq, pos, slot = [0], [], [], [], []
    admitted = taken = 0
    err, open_ = 0, True
    for b in range(B):
        n, p = int(new[b]), int(past[b])
        if n < 0 or p < 0 or n + p > 64 * width:
            err = 1
            n, p = 0, 0
            have = need = 0
        else:
            have, need = -(-p // 64), -(-(n + p) // 64) - -(-p // 64)
        open_ = open_ and q_start[-1] + n <= rows and taken + need <= len(free)
        if open_:
            admitted += 1
            for i in range(need):
                table[b, have + i] = free[taken + i]
            taken += need
            for i in range(n):
                page = int(table[b, (p + i) // 64])
                seq.append(b)
                pos.append(p + i)
                slot.append(page * 64 + (p + i) % 64 if 0 <= page < num_pages else -1)
                err |= not 0 <= page < num_pages
        q_start.append(q_start[-1] + (n if open_ else 0))
        kv.append(p + (n if open_ else 0))
    total = len(seq)
    seq += [-1] * (rows - total)
    pos += [0] * (rows - total)
    slot += [-1] * (rows - total)
    return dict(page_table=table, q_start=q_start, kv_len=kv, seq_idx=seq, pos=pos, slot=slot,
                counts=[admitted, total, taken]), int(err)


def run_plan(mla, new, past, free, table, num_pages, rows, stream=None):
    B = len(new)
    t = dict(page_table=i32(table), q_start=i32([7] * (B + 1)), kv_len=i32([7] * B), seq_idx=i32([7] * rows),
             pos=i32([7] * rows), slot=torch.full((rows,), 7, dtype=torch.int64, device=DEV), counts=i32([7] * 3))
    err = i32([0])
    mla.plan_step(i32(new), i32(past), i32(free), t["page_table"], num_pages, t["q_start"], t["kv_len"], t["seq_idx"],
                  t["pos"], t["slot"], t["counts"], err, stream=stream)
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in t.items()}, int(err.item())


def plan_case(seed, B, new_max, past_max, free_share=1.0):
    r = np.random.default_rng(seed)
    new = r.integers(0, new_max + 1, B)
    past = r.integers(0, past_max + 1, B)
    have, want = -(-past // 64), -(-(past + new) // 64)
    width = max(1, int(want.max()))
    n_free = int((want - have).sum() * free_share)
    num_pages = int(have.sum()) + n_free
    ids = r.permutation(num_pages)
    table = np.full((B, width), -1)
    at = 0
    for b in range(B):
        table[b, :have[b]] = ids[at:at + have[b]]
        at += have[b]
    return new, past, ids[at:], table, num_pages


def check_plan(mla, new, past, free, table, num_pages, rows):
    got, err = run_plan(mla, new, past, free, table, num_pages, rows)
    ref, want_err = plan_reference(new, past, free, np.asarray(table), num_pages, rows)
    for k, v in ref.items():
        np.testing.assert_array_equal(got[k], np.asarray(v), err_msg=k)
    assert err == want_err


@pytest.mark.parametrize("B,new_max,past_max", [(1, 1, 0), (1, 700, 63), (2, 0, 5), (7, 3, 64), (64, 1, 8192),
                                                (513, 40, 300), (1000, 129, 1000), (5000, 2, 100)])
def test_plan_matches_a_walk_over_requests_and_tokens(mla, B, new_max, past_max):
    case = plan_case(B + new_max, B, new_max, past_max)
    check_plan(mla, *case, rows=int(case[0].sum()) + 5)


@pytest.mark.parametrize("budget", [0, 1, 17, 100, 399])
def test_plan_admits_in_order_until_the_rows_run_out(mla, budget):
    check_plan(mla, *plan_case(3, 40, 20, 200), rows=budget)


@pytest.mark.parametrize("share", [0.0, 0.3, 0.8])
def test_plan_admits_in_order_until_the_pages_run_out(mla, share):
    case = plan_case(4, 60, 150, 90, free_share=share)
    check_plan(mla, *case, rows=int(case[0].sum()))


def test_plan_largest_number_of_requests(mla):
    case = plan_case(5, 16384, 3, 130)
    check_plan(mla, *case, rows=int(case[0].sum()))
    with pytest.raises(mla.MlaError) as e:
        run_plan(mla, [0] * 16385, [0] * 16385, [0], [[0]] * 16385, 1, 1)
    assert e.value.code == -2


def test_plan_reports_lengths_and_pages_that_make_no_sense(mla):
    new, past, free, table, num_pages = plan_case(6, 9, 70, 200)
    for at, (n, p) in ((2, (-1, 5)), (4, (3, -2)), (6, (2 ** 31 - 1, 2 ** 31 - 1)), (7, (1, 64 * table.shape[1]))):
        bad_new, bad_past = new.copy(), past.copy()
        bad_new[at], bad_past[at] = n, p
        check_plan(mla, bad_new, bad_past, free, table, num_pages, 400)
    bad = free.copy()
    bad[0], bad[1] = num_pages, -3
    check_plan(mla, new, past, bad, table, num_pages, 700)


def test_plan_again_on_its_own_output_changes_nothing(mla):
    new, past, free, table, num_pages = plan_case(8, 30, 90, 300)
    rows = int(new.sum())
    got, _ = run_plan(mla, new, past, free, table, num_pages, rows)
    again, _ = run_plan(mla, new, past, free, got["page_table"], num_pages, rows)
    for k in got:
        np.testing.assert_array_equal(got[k], again[k])


# ------------------------------------------------------------ norms, rotation
def rms64(x, gamma, eps):
    x = x.double()
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gamma.double()


def turn64(x, pos, base=10000.0):
    d = x.shape[-1]
    theta = base ** (-torch.arange(0, d, 2, dtype=torch.float64, device=DEV) / d)
    a = (pos.double()[:, None] * theta).view(-1, *([1] * (x.dim() - 2)), d // 2)
    c, s = torch.cos(a), torch.sin(a)
    e, o = x.double()[..., 0::2], x.double()[..., 1::2]
    return torch.stack([e * c - o * s, e * s + o * c], -1).flatten(-2)


def close_norm(got, ref, dtype, n):
    # The mean of n squares in fp32 is off by at most n 2^-24 of itself, half of that after the root, and the
    # root, the two products and the rounding add 4 steps of 2^-24 and one of the type.
    tol = (U[dtype] + (n / 2 + 4) * 2.0 ** -24) * ref.abs() + 1e-30
    assert ((got.double() - ref).abs() <= tol).all()


def close_turn(got, ref, x, dtype):
    # The angle is within 2^-24 turns' rounding (|half turns| <= 1: 2^-24 pi), sine and cosine within 2 steps, the
    # two products and the sum within one each: 8 steps of the pair's length; then the type's rounding.
    length = torch.hypot(x.double()[..., 0::2], x.double()[..., 1::2]).repeat_interleave(2, -1)
    assert ((got.double() - ref).abs() <= U[dtype] * ref.abs() + 8 * 2.0 ** -24 * length + 1e-30).all()


NORM_DIMS = [  # dtype, d_c, d_r, d_cq, per head keys (n_h), offset of the rows in a wider one
    ("bf16", 512, 64, 1536, 0, 0), ("bf16", 128, 16, 8, 0, 8), ("bf16", 256, 32, 0, 16, 0), ("bf16", 384, 48, 24, 0, 3),
    ("f32", 64, 16, 96, 0, 0), ("f32", 5, 2, 7, 0, 0), ("f32", 511, 62, 513, 0, 1), ("f32", 512, 64, 4100, 0, 4),
    ("f32", 33, 6, 0, 5, 0), ("bf16", 512, 64, 9000, 0, 0)]


@pytest.mark.parametrize("dtype,d_c,d_r,d_cq,heads,offset", NORM_DIMS)
@pytest.mark.parametrize("T", [1, 2, 67])
def test_append_normed_matches_the_formula(mla, dtype, d_c, d_r, d_cq, heads, offset, T):
    g = gen(T + d_c)
    dims = dims_of(mla, dtype, heads or 4, 32, d_c, d_r, d_cq, rope_key_per_head=int(heads > 0))
    keys = max(heads, 1) * d_r
    wide = randn(g, T, offset + d_cq + d_c + keys + 2 * offset, dtype=DT[dtype], scale=2.0)
    cq = wide[:, offset:offset + d_cq] if d_cq else None
    kv = wide[:, offset + d_cq:offset + d_cq + d_c + keys]
    gk = randn(g, d_c, dtype=DT[dtype])
    gq = randn(g, d_cq, dtype=DT[dtype]) if d_cq else None
    pos = torch.randint(0, 200000, (T,), generator=g, device=DEV).to(torch.int32)
    pages = -(-T // 64) + 2
    before = randn(g, pages, 64, d_c + keys, dtype=DT[dtype])
    cache = before.clone()
    slot = torch.randperm(pages * 64, generator=g, device=DEV)[:T].contiguous()
    out = torch.empty(T, d_cq, dtype=DT[dtype], device=DEV) if d_cq else None
    err = i32([0])
    mla.append_normed(dims, kv, gk, pos, slot, cache, 1e-5, cq, gq, out, err)
    torch.cuda.synchronize()
    assert err.item() == 0
    rows = cache.view(-1, d_c + keys)
    close_norm(rows[slot, :d_c], rms64(kv[:, :d_c], gk, 1e-5), dtype, d_c)
    key = kv[:, d_c:].reshape(T, -1, d_r)
    close_turn(rows[slot, d_c:].view(T, -1, d_r), turn64(key, pos), key, dtype)
    if d_cq:
        close_norm(out, rms64(cq, gq, 1e-5), dtype, d_cq)
    rest = torch.ones(pages * 64, dtype=torch.bool, device=DEV)
    rest[slot] = False
    assert torch.equal(rows[rest], before.view(-1, d_c + keys)[rest])


def test_append_normed_skips_padding_and_reports_bad_slots(mla):
    g = gen(1)
    dims = dims_of(mla, "bf16", 16, 32, 128, 16, 64)
    kv, cq = randn(g, 6, 144, dtype=DT["bf16"]), randn(g, 6, 64, dtype=DT["bf16"])
    cache = torch.full((2, 64, 144), 7.0, dtype=DT["bf16"], device=DEV)
    out = torch.zeros_like(cq)
    err = i32([0])
    pos = i32(range(6))

    def run(slots):
        mla.append_normed(dims, kv, None, pos, torch.tensor(slots, device=DEV), cache, 1e-6, cq, None, out, err)
        torch.cuda.synchronize()
        return int(err.item())

    assert run([-1, 3, -1, 127, -1, -1]) == 0
    assert torch.equal(out, cq)                       # no gamma: copied
    assert torch.equal(cache.view(-1, 144)[[3, 127], :128], kv[[1, 3], :128])
    assert int((cache.view(-1, 144) != 7).any(1).sum()) == 2
    assert run([128, 5, -1, -1, -1, -1]) == 1 and int((cache.view(-1, 144) != 7).any(1).sum()) == 3
    err.zero_()
    assert run([-2, -1, -1, 2 ** 40, -1, -1]) == 1 and int((cache.view(-1, 144) != 7).any(1).sum()) == 3


@pytest.mark.parametrize("x", [0.0, 1e-30, 3e18, float("nan"), float("inf")])
def test_norm_of_extreme_rows(mla, x):
    dims = dims_of(mla, "f32", 2, 32, 64, 16)
    kv = torch.full((1, 80), x, device=DEV)
    kv[0, 64:] = 1
    cache = torch.zeros(1, 64, 80, device=DEV)
    mla.append_normed(dims, kv, torch.ones(64, device=DEV), i32([0]), torch.tensor([9], device=DEV), cache, 1e-6)
    y = cache[0, 9, :64]
    if x == 0:
        assert (y == 0).all()
    elif math.isfinite(x) and x > 1:
        assert torch.allclose(y, torch.ones_like(y), rtol=1e-5)
    elif math.isfinite(x):
        assert torch.allclose(y, torch.full_like(y, x * 1e3), rtol=1e-5)   # 1 / sqrt(eps)
    else:
        assert torch.isnan(y).all()


QUERY_DIMS = [("bf16", 128, 128, 64), ("bf16", 16, 128, 32), ("bf16", 1, 8, 16), ("bf16", 5, 96, 48), ("bf16", 3, 1504, 16),
              ("f32", 4, 32, 16), ("f32", 3, 5, 2), ("f32", 2, 131, 62), ("f32", 128, 64, 64), ("f32", 1, 1028, 4)]


@pytest.mark.parametrize("dtype,n_h,d_h,d_r", QUERY_DIMS)
@pytest.mark.parametrize("T,form", [(1, "dense"), (9, "dense"), (9, "absorbed"), (9, "odd"), (9, "in place")])
def test_query_norm_rope_matches_the_formula(mla, dtype, n_h, d_h, d_r, T, form):
    g = gen(n_h + d_h)
    dims = dims_of(mla, dtype, n_h, d_h, 128, d_r)
    pad = 3 if form == "odd" else 0
    wide = randn(g, T, n_h * (d_h + d_r) + pad, dtype=DT[dtype], scale=1.5)
    q = wide[:, pad:].view(T, n_h, d_h + d_r) if not pad else torch.as_strided(
        wide, (T, n_h, d_h + d_r), (wide.shape[1], d_h + d_r, 1), pad)
    keep = q.clone()
    gamma = randn(g, d_h, dtype=DT[dtype])
    pos = torch.randint(0, 200000, (T,), generator=g, device=DEV).to(torch.int32)
    if form == "in place":
        qc, qr = q[..., :d_h], q[..., d_h:]
    elif form == "absorbed":
        qc, qr = torch.empty(T, n_h, d_h, dtype=DT[dtype], device=DEV), torch.zeros(
            T, n_h, 128 + d_r, dtype=DT[dtype], device=DEV)[..., 128:]
    else:
        qc = torch.empty(T, n_h, d_h + pad, dtype=DT[dtype], device=DEV)[..., pad:]
        qr = torch.empty(T, n_h, d_r + pad, dtype=DT[dtype], device=DEV)[..., pad:]
    mla.query_norm_rope(dims, q, gamma, pos, qc, qr, 1e-5)
    torch.cuda.synchronize()
    close_norm(qc, rms64(keep[..., :d_h], gamma, 1e-5), dtype, d_h)
    close_turn(qr, turn64(keep[..., d_h:], pos), keep[..., d_h:], dtype)
    mla.query_norm_rope(dims, keep, None, pos, qc, qr)
    assert torch.equal(qc, keep[..., :d_h])


# ------------------------------------------------------------------ attention
class Step:
    """Inputs of one attention over a packed batch; everything no query sees is NaN."""

    def __init__(self, mla, dtype, n_h, d_c, d_r, lens, seed=0, d_h=32, head=0, tail=0, qscale=1.0, softmax_scale=0.0):
        g = gen(seed)
        self.mla, self.dtype, self.n_h, self.d_c, self.d_r = mla, dtype, n_h, d_c, d_r
        self.dims = dims_of(mla, dtype, n_h, d_h, d_c, d_r, softmax_scale=softmax_scale)
        self.scale = softmax_scale or 1 / math.sqrt(d_h + d_r)
        self.new, self.kv = [n for n, _ in lens], [k for _, k in lens]
        self.B, self.head = len(lens), head
        self.T = head + sum(self.new) + tail
        starts = [head]
        for n in self.new:
            starts.append(starts[-1] + n)
        self.starts = starts
        self.q = randn(g, self.T, n_h, d_c + d_r, dtype=DT[dtype], scale=qscale)
        pages = [max(0, -(-k // 64)) for k in self.kv]
        width = max(1, max(pages)) + 1
        n_pages = sum(pages) + 3
        ids = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
        self.table = torch.full((self.B, width), -1, dtype=torch.int32, device=DEV)
        self.cache = torch.full((n_pages, 64, d_c + d_r), float("nan"), dtype=DT[dtype], device=DEV)
        at = 0
        for b, k in enumerate(self.kv):
            self.table[b, :pages[b]] = ids[at:at + pages[b]]
            if k > 0:
                rows = (ids[at:at + pages[b]].long()[:, None] * 64 + torch.arange(64, device=DEV)).flatten()[:k]
                self.cache.view(-1, d_c + d_r)[rows] = randn(g, k, d_c + d_r, dtype=DT[dtype])
            at += pages[b]
        self.ws = torch.empty(mla.attend_ragged_workspace_bytes(self.dims, self.B, self.T), dtype=torch.uint8, device=DEV)

    def keys(self, b):
        k = self.kv[b]
        pages = self.table[b, :-(-k // 64)].long()
        return self.cache[pages].flatten(0, 1)[:k].double()

    def run(self, q=None, lse=True, ws=None, fill=7.0):
        out = torch.full((self.T, self.n_h, self.d_c), fill, dtype=DT[self.dtype], device=DEV)
        l = torch.full((self.T, self.n_h), fill, device=DEV) if lse else None
        self.mla.attend_ragged(self.dims, self.q if q is None else q, i32(self.starts), i32(self.kv), self.table,
                               self.cache, out, l, self.ws if ws is None else ws)
        return out, l

    def check(self, out, lse, only=None):
        torch.cuda.synchronize()
        assert self.mla.get_error(self.ws) == 0
        u, off, norm = U[self.dtype], 0.0, 0.0
        for b in range(self.B) if only is None else only:
            keys = self.keys(b)
            for i in range(self.new[b]):
                t, sees = self.starts[b] + i, self.kv[b] - self.new[b] + i + 1
                if sees <= 0:
                    assert (out[t] == 0).all() and (lse[t] == -math.inf).all()
                    continue
                q, k = self.q[t].double(), keys[:sees]
                a = self.scale * (q @ k.t())
                z = torch.logsumexp(a, -1, keepdim=True)
                alpha = torch.exp(a - z)
                ref, mag = alpha @ k[:, :self.d_c], alpha @ k[:, :self.d_c].abs()
                d = self.d_c + self.d_r
                ds = self.scale * d * 2.0 ** -24 * (q.abs() @ k.abs().t()).max()
                weight = (u if self.dtype == "bf16" else 0) + 2 * float(ds) + 16 * 2.0 ** -22 + sees * 2.0 ** -24
                err = (out[t].double() - ref).abs()
                assert (err <= 1.05 * weight * mag + u * ref.abs() + 1e-30).all(), (b, i, float((err / mag).max()))
                assert ((lse[t].double() - z[:, 0] / math.log(2)).abs() <= 1.5 * (weight + 2.0 ** -22 * z.abs().max())).all()
                off += float(err.square().sum())
                norm += float(ref.square().sum())
        if norm:
            # Random roundings of weights and output: their root mean square is u / sqrt(3) of the value at most.
            assert math.sqrt(off / norm) <= (2 * u if self.dtype == "bf16" else 1e-5)
        for t in list(range(self.starts[0])) + list(range(self.starts[-1], self.T)):
            assert (out[t] == 7).all() and (lse[t] == 7).all()


LENS = {
    "one": [(1, 1)],
    "edges": [(1, 63), (1, 64), (1, 65), (2, 64), (2, 65), (3, 2), (0, 10), (65, 65), (64, 129)],
    "chunks": [(37, 37), (0, 0), (129, 300), (1, 513), (5, 70), (64, 64)],
    "long": [(3, 2500), (1, 5)],
    "empty": [(0, 5), (0, 0), (0, 700)],
    "nothing seen": [(3, 0), (5, 2), (1, 0), (2, 66)],
}
BF16_DIMS = [(16, 256, 32), (128, 512, 64), (3, 128, 16), (1, 384, 48), (40, 512, 32), (128, 128, 64)]
F32_DIMS = [(4, 64, 16), (16, 256, 32), (5, 5, 2), (7, 131, 62), (64, 512, 64), (1, 300, 8)]


@pytest.mark.parametrize("name", list(LENS))
@pytest.mark.parametrize("dtype,n_h,d_c,d_r", [("bf16", *d) for d in BF16_DIMS] + [("f32", *d) for d in F32_DIMS])
def test_attend_ragged_matches_the_softmax(mla, dtype, n_h, d_c, d_r, name):
    s = Step(mla, dtype, n_h, d_c, d_r, LENS[name], head=2, tail=3)
    s.check(*s.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend_ragged_many_requests_and_few_heads(mla, dtype):
    r = np.random.default_rng(3)
    lens = [(int(n), int(n + p)) for n, p in zip(r.integers(0, 4, 300), r.integers(0, 200, 300))]
    s = Step(mla, dtype, 2, 128, 16, lens)
    s.check(*s.run())


@pytest.mark.parametrize("dtype,n_h", [("bf16", 128), ("bf16", 16), ("f32", 16)])
def test_attend_ragged_peaked_and_flat_scores(mla, dtype, n_h):
    for qscale in (0.0, 8.0):
        s = Step(mla, dtype, n_h, 256, 32, [(4, 400), (33, 90)], qscale=qscale)
        s.check(*s.run())
    s = Step(mla, dtype, n_h, 256, 32, [(4, 400)], softmax_scale=0.01)
    s.check(*s.run())


@pytest.mark.parametrize("dtype,n_h", [("bf16", 128), ("bf16", 16), ("f32", 5)])
def test_attend_ragged_rising_scores_rescale_the_sums(mla, dtype, n_h):
    """Later pages hold ever larger scores, so every page moves the running maximum."""
    s = Step(mla, dtype, n_h, 128, 16, [(2, 700), (70, 400)])
    for b in range(2):
        pages = s.table[b, :-(-s.kv[b] // 64)].long()
        for i, p in enumerate(pages.tolist()):
            s.cache[p, :, 128:] *= 1 + 2 * i
    s.check(*s.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend_ragged_strided_queries_and_no_lse(mla, dtype):
    s = Step(mla, dtype, 6, 128, 16, LENS["chunks"], tail=1)
    want, lse = s.run()
    for pad_h, pad_t in ((8, 0), (0, 16), (24, 40)) + (((1, 3),) if dtype == "f32" else ()):
        hs = 144 + pad_h
        buf = torch.full((s.T, 6 * hs + pad_t), float("nan"), dtype=DT[dtype], device=DEV)
        q = torch.as_strided(buf, (s.T, 6, 144), (buf.shape[1], hs, 1))
        q.copy_(s.q)
        got, l2 = s.run(q)
        assert torch.equal(got, want) and torch.equal(l2, lse)
    heads_first = s.q.transpose(0, 1).contiguous().transpose(0, 1)
    with pytest.raises(mla.MlaError):
        s.run(heads_first)      # a token's heads are not one behind the other
    got, _ = s.run(lse=False)
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype,n_h", [("bf16", 128), ("bf16", 16), ("f32", 16)])
def test_attend_ragged_bitwise_properties(mla, dtype, n_h):
    s = Step(mla, dtype, n_h, 256, 32, [(5, 900), (40, 333), (1, 64)])
    out, lse = s.run()
    again, lse2 = s.run(fill=3.0)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    # Another order of the pages in memory.
    perm = torch.randperm(s.cache.shape[0], device=DEV)
    s.cache = s.cache[perm].contiguous()
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(perm.numel(), device=DEV)
    s.table = torch.where(s.table >= 0, inv[s.table.clamp(min=0).long()].int(), s.table)
    moved, lse3 = s.run()
    assert torch.equal(out, moved) and torch.equal(lse, lse3)


@pytest.mark.parametrize("dtype,n_h", [("bf16", 128), ("bf16", 16), ("bf16", 3), ("f32", 16)])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_attend_ragged_keys_behind_a_query_do_not_reach_it(mla, dtype, n_h, what):
    s = Step(mla, dtype, n_h, 128, 16, [(7, 71), (30, 100)])
    want, lse = s.run()
    first = [s.starts[0] + 4, s.starts[1] + 20]      # the tokens whose own key is spoilt
    for b, i in ((0, 4), (1, 20)):
        p = s.kv[b] - s.new[b] + i
        s.cache[int(s.table[b, p // 64]), p % 64] = what
    got, l2 = s.run()
    for b in range(2):
        clean = slice(s.starts[b], first[b])
        assert torch.equal(got[clean], want[clean]) and torch.equal(l2[clean], lse[clean])
        spoilt = got[first[b]:s.starts[b + 1]]
        if math.isnan(what):
            assert torch.isnan(spoilt).all() and torch.isnan(l2[first[b]:s.starts[b + 1]]).all()


def test_attend_ragged_reports_what_it_cannot_use(mla):
    s = Step(mla, "bf16", 16, 128, 16, [(5, 200), (3, 80), (4, 100)])
    want, _ = s.run()
    table = s.table.clone()
    s.table[1, 0] = s.cache.shape[0]
    out, _ = s.run()
    assert mla.get_error(s.ws) == -5
    keep = [t for t in range(s.T) if not s.starts[1] <= t < s.starts[2]]
    assert torch.equal(out[keep], want[keep])
    s.table = table
    s.run()
    assert mla.get_error(s.ws) == 0          # the word is the last call's
    starts, kv = s.starts, s.kv
    for bad in ([0, 5, 3, 12], [0, 5, 8, 13], [-1, 5, 8, 12]):
        s.starts = bad
        out, _ = s.run()
        assert mla.get_error(s.ws) == -5 and (out == 7).all()
    s.starts = starts
    for bad in ([200, 64 * s.table.shape[1] + 1, 100], [200, -1, 100]):
        s.kv = bad
        out, _ = s.run()
        assert mla.get_error(s.ws) == -5
        keep = [t for t in range(s.T) if not s.starts[1] <= t < s.starts[2]]
        assert torch.equal(out[keep], want[keep])
    s.kv = kv


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend_ragged_in_a_graph_on_another_stream(mla, dtype):
    s = Step(mla, dtype, 16, 128, 16, [(9, 300), (1, 65)])
    want, lse = s.run()
    starts, kv = i32(s.starts), i32(s.kv)
    out, l2 = torch.zeros_like(want), torch.zeros_like(lse)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        mla.attend_ragged(s.dims, s.q, starts, kv, s.table, s.cache, out, l2, s.ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(l2, lse)
    # New lengths in the same buffers: the captured call reads them when it runs.
    kv[0] -= 64
    s.kv = [236, 65]
    graph.replay()
    torch.cuda.synchronize()
    s.check(out, l2)


def test_a_ragged_step_from_lengths_to_outputs(mla):
    """Plan, normalised append, query norm, absorption, attention over three steps of changing requests, against the
    definition on unpaged data."""
    n_h, d_h, d_c, d_r, eps = 16, 128, 256, 32, 1e-6
    dims = dims_of(mla, "bf16", n_h, d_h, d_c, d_r)
    g = gen(11)
    B, width, num_pages = 4, 6, 20
    gk, gq = randn(g, d_c, dtype=DT["bf16"]), randn(g, d_h, dtype=DT["bf16"])
    w_uk = randn(g, n_h, d_h, d_c, dtype=DT["bf16"], scale=d_c ** -0.5)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    cache = torch.full((num_pages, 64, d_c + d_r), float("nan"), dtype=DT["bf16"], device=DEV)
    free = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32)
    taken, past = 0, [0] * B
    history = [torch.zeros(0, d_c + d_r, dtype=torch.float64, device=DEV) for _ in range(B)]
    for new in ([70, 1, 0, 130], [1, 1, 40, 3], [4, 64, 1, 1]):
        total = sum(new)
        rows = total + 9
        q_start, kv_len = i32([0] * (B + 1)), i32([0] * B)
        seq, pos, slot = i32([0] * rows), i32([0] * rows), torch.zeros(rows, dtype=torch.int64, device=DEV)
        counts = i32([0] * 3)
        mla.plan_step(i32(new), i32(past), free[taken:], table, num_pages, q_start, kv_len, seq, pos, slot, counts)
        kv = randn(g, rows, d_c + d_r, dtype=DT["bf16"], scale=1.5)
        q = randn(g, rows, n_h, d_h + d_r, dtype=DT["bf16"], scale=1.5)
        mla.append_normed(dims, kv, gk, pos, slot, cache, eps)
        absorbed = torch.empty(rows, n_h, d_c + d_r, dtype=DT["bf16"], device=DEV)
        qc = torch.empty(rows, n_h, d_h, dtype=DT["bf16"], device=DEV)
        mla.query_norm_rope(dims, q, gq, pos, qc, absorbed[..., d_c:], eps)
        absorbed[..., :d_c] = torch.einsum("thd,hdc->thc", qc.float(), w_uk.float()).to(DT["bf16"])
        out = torch.full((rows, n_h, d_c), 7.0, dtype=DT["bf16"], device=DEV)
        ws = torch.empty(mla.attend_ragged_workspace_bytes(dims, B, rows), dtype=torch.uint8, device=DEV)
        mla.attend_ragged(dims, absorbed, q_start, kv_len, table, cache, out, None, ws)
        assert mla.get_error(ws) == 0
        c = counts.tolist()
        assert c[:2] == [B, total]
        taken += c[2]
        assert (out[total:] == 7).all()
        row = 0
        for b in range(B):
            p = torch.arange(past[b], past[b] + new[b], device=DEV)
            x = kv[row:row + new[b]]
            history[b] = torch.cat([history[b], torch.cat([rms64(x[:, :d_c], gk, eps), turn64(x[:, d_c:], p)], 1)])
            qx = q[row:row + new[b]]
            qa = torch.cat([torch.einsum("thd,hdc->thc", rms64(qx[..., :d_h], gq, eps), w_uk.double()),
                            turn64(qx[..., d_h:], p)], -1)
            for i in range(new[b]):
                k = history[b][:past[b] + i + 1]
                alpha = torch.softmax(qa[i] @ k.t() / math.sqrt(d_h + d_r), -1)
                ref = alpha @ k[:, :d_c]
                # Six roundings of bf16 on the way (latent, q_C, q~, q_R, weights, output), each at most u of its value;
                # those of queries and keys move a score of standard deviation ~2 by a few u.
                assert (out[row + i].double() - ref).norm() <= 6 * U["bf16"] * ref.norm()
            past[b] += new[b]
            row += new[b]


@pytest.mark.parametrize("dtype,dims_", [("bf16", (16, 128, 128, 256, 32, 512, 0)), ("bf16", (128, 64, 64, 512, 64, 256, 128)),
                                         ("f32", (4, 32, 32, 64, 16, 128, 0)), ("f32", (3, 16, 24, 40, 6, 64, 48))])
def test_ragged_step_matches_oracle_over_several_steps(mla, dtype, dims_):
    """Requests that grow by different numbers of tokens, planned on the GPU, against the oracle's decode of each."""
    import oracle as O
    from head_latent_attention_append_b200 import synth, workload
    n_h, d_h, d_v, d_c, d_r, d_model, d_cq = dims_
    wl = synth.Workload("ragged", 21, n_h, d_h, d_v, d_c, d_r, d_model, d_cq, dtype, "decode", 5, 1, 0)
    hw = synth.make_weights(wl, 5)
    weights = mla.Weights(workload.dims_of(wl), workload.upload_weights(wl, hw, torch.device(DEV)))
    odims, ow = O.Dims(n_h, d_h, d_v, d_c, d_r, d_model, d_cq, wl.rope_base), O.Weights(**hw.as_dict())
    steps = [[70, 1, 0, 130, 5], [1, 3, 64, 1, 1], [0, 2, 1, 0, 40]]
    H = [synth.make_hidden(wl, b, sum(s[b] for s in steps), 5) for b in range(5)]
    num_pages, width = 24, 5
    table = torch.full((5, width), -1, dtype=torch.int32, device=DEV)
    free = torch.randperm(num_pages, generator=gen(2), device=DEV).to(torch.int32)
    cache = torch.full((num_pages, 64, d_c + d_r), float("nan"), dtype=DT[dtype], device=DEV)
    taken, past = 0, [0] * 5
    for new in steps:
        total, rows = sum(new), sum(new) + 4
        q_start, kv_len, seq, pos = i32([0] * 6), i32([0] * 5), i32([0] * rows), i32([0] * rows)
        counts, slot = i32([0] * 3), torch.zeros(rows, dtype=torch.int64, device=DEV)
        mla.plan_step(i32(new), i32(past), free[taken:], table, num_pages, q_start, kv_len, seq, pos, slot, counts)
        h = torch.from_numpy(np.concatenate([H[b][past[b]:past[b] + new[b]] for b in range(5)]
                                            + [np.zeros((4, d_model), np.float32)])).to(DEV, DT[dtype])
        out = torch.empty(rows, n_h, d_v, device=DEV)
        ws = torch.empty(mla.ragged_step_workspace_bytes(weights.dims, 5, rows), dtype=torch.uint8, device=DEV)
        mla.ragged_step(weights, h, q_start, kv_len, seq, pos, table, num_pages, cache, out, ws)
        assert mla.get_error(ws) == mla.MLA_OK
        taken += int(counts[2])
        got, row = out.cpu().numpy(), 0
        for b in range(5):
            past[b] += new[b]
            if new[b]:
                ref = O.mla_decode(odims, ow, H[b][:past[b]], new[b])
                # The bounds of the library's other paths (their intermediates are rounded alike).
                err = np.abs(got[row:row + new[b]] - ref).max() / np.abs(ref).max()
                assert err <= {"f32": 1e-4, "bf16": 2e-2}[dtype], (b, err)
            row += new[b]


def test_ragged_step_reports_rows_that_belong_nowhere(mla):
    from head_latent_attention_append_b200 import synth, workload
    wl = synth.Workload("ragged", 22, 4, 32, 32, 64, 16, 128, 0, "f32", "decode", 2, 1, 0)
    weights = mla.Weights(workload.dims_of(wl), workload.upload_weights(wl, synth.make_weights(wl, 5), torch.device(DEV)))
    h = torch.zeros(3, 128, device=DEV)
    cache, out = torch.zeros(4, 64, 80, device=DEV), torch.empty(3, 4, 32, device=DEV)
    ws = torch.empty(mla.ragged_step_workspace_bytes(weights.dims, 2, 3), dtype=torch.uint8, device=DEV)

    def run(seq, pos, kv, table):
        mla.ragged_step(weights, h, i32([0, 2, 3]), i32(kv), i32(seq), i32(pos), i32(table), 4, cache, out, ws)
        return mla.get_error(ws)

    good = [[0, 1], [2, 3]]
    assert run([0, 0, 1], [0, 1, 0], [2, 1], good) == 0
    assert run([0, 0, -1], [0, 1, 0], [2, 1], good) == 0          # a row of no request
    assert run([0, 0, 2], [0, 1, 0], [2, 1], good) == -5
    assert run([0, 0, -2], [0, 1, 0], [2, 1], good) == -5
    assert run([0, 0, 1], [0, 128, 0], [2, 1], good) == -5
    assert run([0, 0, 1], [0, 1, 0], [2, 129], good) == -5
    assert run([0, 0, 1], [0, 1, 0], [2, 1], [[0, 1], [9, 3]]) == -5
    assert run([0, 0, 1], [0, 1, 0], [2, 1], good) == 0


# --------------------------------------------------- sizes and uses at the edges
@pytest.mark.parametrize("dtype,n_h,B,most", [("bf16", 16, 700, 3), ("f32", 4, 520, 2), ("bf16", 128, 40, 60), ("f32", 64, 40, 60)])
def test_attend_ragged_schedules_of_many_requests_and_row_blocks(mla, dtype, n_h, B, most):
    r = np.random.default_rng(B)
    lens = [(int(n), int(n + p)) for n, p in zip(r.integers(0, most + 1, B), r.integers(0, 150, B))]
    s = Step(mla, dtype, n_h, 128, 16, lens)
    out, lse = s.run()
    s.check(out, lse, only=list(r.choice(B, 12, replace=False)) + [0, B - 1])


@pytest.mark.parametrize("by", ["requests", "row blocks"])
@pytest.mark.parametrize("dtype,most", [("bf16", 384), ("bf16", 385), ("bf16", 1024), ("bf16", 1025), ("f32", 256),
                                        ("f32", 257), ("f32", 1024), ("f32", 1025)])
def test_attend_ragged_at_the_limits_of_each_way_to_schedule(mla, dtype, most, by):
    """At one more than these numbers another kernel, or another part of it, makes the schedule."""
    r = np.random.default_rng(most)
    if by == "requests":                       # most of them without a token, the longest ones at both ends
        n_h, lens = 4, [(0, int(k)) for k in r.integers(0, 100, most)]
        for b in r.choice(most, 30, replace=False):
            lens[b] = (int(r.integers(1, 4)), int(r.integers(3, 200)))
        lens[0], lens[-1] = (2, 1900), (1, 2100)
    else:                                      # one row block per token, and two requests
        n_h = 128 if dtype == "bf16" else 64
        lens = [(most - 2 - 7, most + 40), (7, 900)]
    s = Step(mla, dtype, n_h, 128, 16, lens)
    only = [0, s.B - 1] + ([b for b in range(s.B) if s.new[b]][1:8] if by == "requests" else [])
    first = s.run()
    s.check(*first, only=only)
    good = s.table.clone()
    s.table[-1, 1] = 10 ** 6                   # a page that is not there: reported, and by this call alone
    s.run()
    torch.cuda.synchronize()
    assert mla.get_error(s.ws) == -5
    s.table.copy_(good)
    again = s.run()
    s.check(*again, only=only)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    s.kv[-1] += 64 * s.table.shape[1]          # a length behind the table
    s.run()
    torch.cuda.synchronize()
    assert mla.get_error(s.ws) == -5
    s.starts[1], s.starts[2] = s.starts[2] + 1, s.starts[1]
    out, lse = s.run()
    torch.cuda.synchronize()
    assert mla.get_error(s.ws) == -5 and (out == 7).all() and (lse == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend_ragged_schedule_that_does_not_fit_shared_memory(mla, dtype):
    """16,000 requests of one token and 64 heads or more are more row blocks than the schedule keeps on chip."""
    r = np.random.default_rng(7)
    B, n_h = 16000, 128 if dtype == "bf16" else 64
    lens = [(1, int(k)) for k in r.integers(1, 4, B)]
    s = Step(mla, dtype, n_h, 128, 16, lens)
    out, lse = s.run()
    s.check(out, lse, only=list(r.choice(B, 30, replace=False)) + [0, B - 1])
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()


def test_attend_ragged_offsets_past_32_bits(mla):
    """Queries and outputs of more than 2^31 elements and a cache of more than 4 GiB."""
    n_h, d_c, d_r = 128, 512, 64
    dims = dims_of(mla, "bf16", n_h, 32, d_c, d_r)
    B, n = 330, 100
    T, num_pages = B * n, 70000
    assert T * n_h * d_c > 2 ** 31 and num_pages * 64 * 576 * 2 > 2 ** 32
    g = gen(3)
    q = torch.empty(T, n_h, d_c + d_r, dtype=DT["bf16"], device=DEV)
    q.normal_(generator=g)
    cache = torch.full((num_pages, 64, d_c + d_r), float("nan"), dtype=DT["bf16"], device=DEV)
    table = torch.randperm(num_pages, generator=g, device=DEV)[:2 * B].view(B, 2).to(torch.int32)
    table[-1] = torch.tensor([num_pages - 1, num_pages - 2])
    table[0, 0] = num_pages - 3
    for b in range(B):
        for j in range(2):
            cache[table[b, j].long()].normal_(generator=g)
    starts, kv = i32([n * b for b in range(B + 1)]), i32([n + 7] * B)
    out = torch.empty(T, n_h, d_c, dtype=DT["bf16"], device=DEV)
    lse = torch.empty(T, n_h, device=DEV)
    ws = torch.empty(mla.attend_ragged_workspace_bytes(dims, B, T), dtype=torch.uint8, device=DEV)
    mla.attend_ragged(dims, q, starts, kv, table, cache, out, lse, ws)
    assert mla.get_error(ws) == 0
    for t in (0, 99, T // 2, T - 101, T - 100, T - 1):
        b, sees = t // n, 7 + t % n + 1
        k = cache[table[b].long()].flatten(0, 1)[:sees].double()
        a = q[t].double() @ k.t() / math.sqrt(32 + d_r)
        alpha = torch.softmax(a, -1)
        ref = alpha @ k[:, :d_c]
        # As in Step.check: weights and output rounded once each, scores fp32 sums of 576 products.
        ds = 576 * 2.0 ** -24 * float((q[t].double().abs() @ k.abs().t()).max()) / math.sqrt(32 + d_r)
        tol = 1.05 * (U["bf16"] + 2 * ds + 1e-5) * (alpha @ k[:, :d_c].abs()) + U["bf16"] * ref.abs()
        assert ((out[t].double() - ref).abs() <= tol).all(), t
    assert torch.isfinite(lse).all()


def test_norm_calls_offsets_past_32_bits(mla):
    T, width = 300000, 8000                       # 2.4e9 elements of rows, of which slices are read
    wide = torch.empty(T, width, dtype=DT["bf16"], device=DEV)
    rows = torch.tensor([0, 1, T // 2, T - 2, T - 1], device=DEV)
    wide[:, 7000:].normal_(generator=gen(4))
    dims = dims_of(mla, "bf16", 2, 128, 512, 64, 16)
    kv = wide[:, 7000:7576]
    cache = torch.zeros(T // 64 + 1, 64, 576, dtype=DT["bf16"], device=DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    slot = torch.arange(T - 1, -1, -1, device=DEV)
    ones = torch.ones(512, dtype=DT["bf16"], device=DEV)
    mla.append_normed(dims, kv, ones, pos, slot, cache, 1e-6)
    flat = cache.view(-1, 576)
    close_norm(flat[slot[rows], :512], rms64(kv[rows, :512], ones, 1e-6), "bf16", 512)
    close_turn(flat[slot[rows], 512:], turn64(kv[rows, 512:], pos[rows]), kv[rows, 512:], "bf16")
    q = torch.as_strided(wide, (T, 2, 192), (width, 192, 1), 7600)
    qc, qr = torch.as_strided(wide, (T, 2, 128), (width, 128, 1), 0), torch.as_strided(wide, (T, 2, 64), (width, 64, 1), 256)
    mla.query_norm_rope(dims, q, ones[:128], pos, qc, qr, 1e-6)
    close_norm(qc[rows], rms64(q[rows][..., :128], ones[:128], 1e-6), "bf16", 128)
    close_turn(qr[rows], turn64(q[rows][..., 128:], pos[rows]), q[rows][..., 128:], "bf16")


def test_calls_on_two_streams_at_once(mla):
    """Each with its own workspace; the norm and plan calls have none."""
    a = Step(mla, "bf16", 16, 256, 32, [(40, 3000), (3, 500)], seed=1)
    b = Step(mla, "bf16", 16, 256, 32, [(1, 2000)] * 20, seed=2)
    want = [a.run(), b.run()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(6):
        for i, s in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i].append(s.run())
    torch.cuda.synchronize()
    for i in range(2):
        for out, lse in got[i]:
            assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


def test_a_whole_step_in_one_graph(mla):
    """Plan to attention captured once and replayed with other lengths."""
    n_h, d_c, d_r, B, rows, num_pages = 16, 256, 32, 3, 80, 12
    dims = dims_of(mla, "bf16", n_h, 32, d_c, d_r)
    g = gen(9)
    kv, q = randn(g, rows, d_c + d_r, dtype=DT["bf16"]), randn(g, rows, n_h, 32 + d_r, dtype=DT["bf16"])
    absorbed = randn(g, rows, n_h, d_c + d_r, dtype=DT["bf16"])
    gk = torch.ones(d_c, dtype=DT["bf16"], device=DEV)
    new, past, free = i32([5, 1, 30]), i32([0, 0, 0]), torch.arange(num_pages, dtype=torch.int32, device=DEV)
    table = torch.full((B, 4), -1, dtype=torch.int32, device=DEV)
    q_start, kv_len, seq, pos = i32([0] * 4), i32([0] * 3), i32([0] * rows), i32([0] * rows)
    slot, counts = torch.zeros(rows, dtype=torch.int64, device=DEV), i32([0] * 3)
    cache = torch.zeros(num_pages, 64, d_c + d_r, dtype=DT["bf16"], device=DEV)
    qc, out = torch.empty(rows, n_h, 32, dtype=DT["bf16"], device=DEV), torch.empty(rows, n_h, d_c, dtype=DT["bf16"], device=DEV)
    ws = torch.empty(mla.attend_ragged_workspace_bytes(dims, B, rows), dtype=torch.uint8, device=DEV)

    def step():
        mla.plan_step(new, past, free, table, num_pages, q_start, kv_len, seq, pos, slot, counts)
        mla.append_normed(dims, kv, gk, pos, slot, cache)
        mla.query_norm_rope(dims, q, None, pos, qc, absorbed[..., d_c:])
        mla.attend_ragged(dims, absorbed, q_start, kv_len, table, cache, out, None, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([5, 1, 30], [64, 1, 15], [1, 1, 1], [0, 80, 0], [2, 70, 40]):
        new.copy_(i32(lens))
        table.fill_(-1)
        out.fill_(7)
        graph.replay()
        got, rows_used = out.clone(), int(counts[1])
        assert rows_used == (72 if lens == [2, 70, 40] else sum(lens))      # the last request does not fit
        out.fill_(7)
        step()
        assert torch.equal(got, out) and (out[rows_used:] == 7).all() and torch.isfinite(out.float()).all()
        assert mla.get_error(ws) == 0
