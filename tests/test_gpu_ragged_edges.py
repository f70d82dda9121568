"""More uses of the ragged-step calls (GPU) that their documentation allows,
against the definitions in 64 bits; tolerances as in test_gpu_ragged.py."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_ragged import (DEV, DT, Step, close_norm, close_turn, dims_of, gen, i32, mla, randn, rms64,  # noqa: E402,F401
                             turn64)


# ------------------------------------------------------------------ attention
def segments_behind_keyless_blocks(lens, n_h, workers, rows=64, surcharge=1):
    """How many times a worker of the fp32 schedule (equal shares of all tiles, a row block counting one more) goes
    from a row block that sees no key to one that does."""
    keys, start = [], 0
    for new, kv in lens:
        end = start + new
        for r in range(start * n_h, end * n_h, rows):
            keys.append(max(0, kv - end + (min(r + rows, end * n_h) - 1) // n_h + 1))
        start = end
    size = [max(1, -(-k // 64)) + surcharge for k in keys]
    workers = min(workers, sum(size))
    share, rest = divmod(sum(size), workers)
    owner = lambda x: x // (share + 1) if x < rest * (share + 1) else rest + (x - rest * (share + 1)) // share
    mine, at = [[] for _ in range(workers)], 0
    for k, n in zip(keys, size):
        for w in range(owner(at + surcharge), owner(at + n - 1) + 1):
            mine[w].append(k)
        at += n
    return sum(a == 0 and b > 0 for m in mine for a, b in zip(m, m[1:]))


@pytest.mark.parametrize("n_h,d_c,d_r", [(64, 512, 64), (64, 256, 32), (64, 61, 6)])
@pytest.mark.parametrize("B", [80, 300, 600])        # one for each way to schedule
def test_attend_ragged_row_blocks_without_keys_between_others(mla, B, n_h, d_c, d_r):
    """Requests of two tokens over one key: every other row block (a token's 64 heads) sees nothing."""
    lens = [(2, 1)] * B
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert segments_behind_keyless_blocks(lens, n_h, min(160, sms)) > 0
    s = Step(mla, "f32", n_h, d_c, d_r, lens)
    first = s.run()
    s.check(*first)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, s.run()))


# ---------------------------------------------------------------------- norms
# Widths that the threads hold in registers, longer ones, odd ones: dtype, d_c, d_cq, d_h.
NORM_WIDTHS = [("bf16", 512, 1536, 128), ("bf16", 128, 9000, 1504), ("f32", 64, 96, 32), ("f32", 512, 4100, 1028),
               ("f32", 5, 513, 131)]


def check_norms(mla, dtype, d_c, d_cq, d_h, scales, eps):
    """Both norm calls on rows (and, in the query call, heads) of these scales, one behind the other."""
    g, T, n_h, d_r = gen(d_c), len(scales), 3, 16 if dtype == "bf16" else 2
    dims = dims_of(mla, dtype, n_h, d_h, d_c, d_r, d_cq)
    factor = torch.tensor(scales, device=DEV)[:, None]
    rows = lambda n: (torch.rand(T, n, generator=g, device=DEV) * 2 - 1).mul(factor).to(DT[dtype])
    kv, cq = rows(d_c + d_r), rows(d_cq)
    gk, gq, gh = (randn(g, n, dtype=DT[dtype]) for n in (d_c, d_cq, d_h))
    assert all(torch.isfinite(x).all() for x in (kv, cq))
    pos = i32(range(T))
    cache, out = torch.zeros(1, 64, d_c + d_r, dtype=DT[dtype], device=DEV), torch.empty_like(cq)
    mla.append_normed(dims, kv, gk, pos, torch.arange(T, device=DEV), cache, eps, cq, gq, out)
    close_norm(cache[0, :T, :d_c], rms64(kv[:, :d_c], gk, eps), dtype, d_c)
    close_norm(out, rms64(cq, gq, eps), dtype, d_cq)
    # Heads of different scales share a warp.
    q = torch.stack([rows(d_h + d_r).roll(h, 0) for h in range(n_h)], 1).contiguous()
    qc, qr = torch.empty(T, n_h, d_h, dtype=DT[dtype], device=DEV), torch.empty(T, n_h, d_r, dtype=DT[dtype], device=DEV)
    mla.query_norm_rope(dims, q, gh, pos, qc, qr, eps)
    close_norm(qc, rms64(q[..., :d_h], gh, eps), dtype, d_h)


@pytest.mark.parametrize("dtype,d_c,d_cq,d_h", NORM_WIDTHS)
def test_norms_of_rows_whose_squares_pass_32_bits(mla, dtype, d_c, d_cq, d_h):
    check_norms(mla, dtype, d_c, d_cq, d_h, [1.0, 3e18, 1e37, 1e38, 3.3e38, 1e-3, 2e19, 3.3e38], 1e-6)


@pytest.mark.parametrize("dtype,d_c,d_cq,d_h", NORM_WIDTHS)
def test_norms_of_rows_of_the_largest_value(mla, dtype, d_c, d_cq, d_h):
    """Every value of the row as large as the type holds: outputs of +-gamma."""
    most, d_r = torch.finfo(DT[dtype]).max, 16 if dtype == "bf16" else 2
    dims = dims_of(mla, dtype, 1, d_h, d_c, d_r, d_cq)
    ones = lambda n: torch.ones(n, dtype=DT[dtype], device=DEV)
    kv, cq, q = (torch.full((1, n), most, dtype=DT[dtype], device=DEV) for n in (d_c + d_r, d_cq, d_h + d_r))
    kv[0, 1::2] = -most
    cache, out = torch.zeros(1, 64, d_c + d_r, dtype=DT[dtype], device=DEV), torch.empty_like(cq)
    mla.append_normed(dims, kv, ones(d_c), i32([0]), torch.tensor([5], device=DEV), cache, 1e-6, cq, ones(d_cq), out)
    close_norm(cache[0, 5:6, :d_c], rms64(kv[:, :d_c], ones(d_c), 1e-6), dtype, d_c)
    close_norm(out, rms64(cq, ones(d_cq), 1e-6), dtype, d_cq)
    qc, qr = torch.empty(1, 1, d_h, dtype=DT[dtype], device=DEV), torch.empty(1, 1, d_r, dtype=DT[dtype], device=DEV)
    mla.query_norm_rope(dims, q.view(1, 1, -1), ones(d_h), i32([0]), qc, qr)
    close_norm(qc, rms64(q[:, None, :d_h], ones(d_h), 1e-6), dtype, d_h)


@pytest.mark.parametrize("eps", [0.0, 1e-35])
@pytest.mark.parametrize("dtype,d_c,d_cq,d_h", NORM_WIDTHS)
def test_norms_of_rows_whose_squares_fall_below_32_bits(mla, dtype, d_c, d_cq, d_h, eps):
    """A small or no eps: what the squares lose of their bits shows.  Rows of ordinary size beside them."""
    check_norms(mla, dtype, d_c, d_cq, d_h, [1e-18, 1.0, 1e-25, 1e-30, 3e-20, 1e-34, 1e38, 1e-16], eps)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 3, 700])
def test_append_writes_the_query_latent_over_itself_beside_the_rows_of_the_cache(mla, dtype, T):
    """One wide row holds c_Q, the latent and the key: in place, and into another part of the same rows."""
    g, d_c, d_r, d_cq = gen(T), 128, 16, 200
    dims = dims_of(mla, dtype, 2, 32, d_c, d_r, d_cq)
    ones = lambda n: torch.ones(n, dtype=DT[dtype], device=DEV)
    pos, slot = i32(range(T)), torch.randperm(-(-T // 64) * 64, generator=g, device=DEV)[:T].contiguous()
    for place in (0, d_cq + d_c + d_r):                       # over itself; behind the key
        wide = randn(g, T, 2 * d_cq + d_c + d_r, dtype=DT[dtype])
        keep = wide.clone()
        cq, kv, out = wide[:, :d_cq], wide[:, d_cq:d_cq + d_c + d_r], wide[:, place:place + d_cq]
        cache = torch.zeros(-(-T // 64), 64, d_c + d_r, dtype=DT[dtype], device=DEV)
        mla.append_normed(dims, kv, ones(d_c), pos, slot, cache, 1e-6, cq, ones(d_cq), out)
        close_norm(out, rms64(keep[:, :d_cq], ones(d_cq), 1e-6), dtype, d_cq)
        close_norm(cache.view(-1, d_c + d_r)[slot, :d_c], rms64(keep[:, d_cq:d_cq + d_c], ones(d_c), 1e-6), dtype, d_c)
        same = torch.ones(wide.shape[1], dtype=torch.bool, device=DEV)
        same[place:place + d_cq] = False
        assert torch.equal(wide[:, same], keep[:, same])
        if T > 1:
            with pytest.raises(mla.MlaError) as e:            # c_Q's rows, packed: where other rows still are
                mla.append_normed(dims, kv, ones(d_c), pos, slot, cache, 1e-6, cq, ones(d_cq),
                                  torch.as_strided(wide, (T, d_cq), (d_cq, 1)))
            assert e.value.code == -1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,n_h", [(1, 1), (1, 5), (40, 1), (40, 7)])
def test_query_outputs_in_other_parts_of_the_rows_of_q(mla, dtype, T, n_h):
    """Rows [q_C | q_R of all heads | room for the outputs]: head strides differ, token strides do not."""
    g, d_h, d_r = gen(T + n_h), 32, 16
    dims, dq = dims_of(mla, dtype, n_h, d_h, 128, d_r), d_h + d_r
    gamma, pos = randn(g, d_h, dtype=DT[dtype]), i32([5 * i for i in range(T)])
    wide = randn(g, T, 2 * n_h * dq, dtype=DT[dtype])
    keep = wide.clone().view(T, 2, n_h, dq)[:, 0]
    view = lambda n, at, hs: torch.as_strided(wide, (T, n_h, n), (wide.shape[1], hs, 1), at)
    q, qc, qr = view(dq, 0, dq), view(d_h, n_h * dq, d_h), view(d_r, n_h * (dq + d_h), d_r)
    mla.query_norm_rope(dims, q, gamma, pos, qc, qr, 1e-6)
    close_norm(qc, rms64(keep[..., :d_h], gamma, 1e-6), dtype, d_h)
    close_turn(qr, turn64(keep[..., d_h:], pos), keep[..., d_h:], dtype)
    assert torch.equal(q, keep)
    if n_h > 1:
        for bad in (dict(qc_out=view(d_h, 0, d_h)), dict(qr_out=view(d_r, d_h, d_r)), dict(qr_out=qc[..., :d_r])):
            with pytest.raises(mla.MlaError) as e:
                mla.query_norm_rope(dims, q, gamma, pos, **{"qc_out": qc, "qr_out": qr, **bad})
            assert e.value.code == -1


# ------------------------------------------------------------------ refusals
def spoilt(t, axes, packed=True):
    """Tensors that cannot stand for `t` (checked along `axes`); each has at least the memory of `t` behind its address."""
    yield "type", t.to(torch.float64 if t.dtype == torch.int64 else torch.int64)
    yield "axes", t[None]
    yield "axes", t.flatten() if t.dim() > 1 else t[:, None].contiguous()
    yield "device", t.cpu()
    for axis in axes:
        if t.shape[axis] > 1:
            less = t.narrow(axis, 0, t.shape[axis] - 1)
            # A contiguous tensor of the smaller shape at the start of as much memory.
            yield f"shorter axis {axis}", t.flatten()[:less.numel()].view(less.shape)
        size = list(t.shape)
        size[axis] += 1
        yield f"longer axis {axis}", t.new_zeros(size)
    if t.shape[-1] > 1:
        yield "strided last axis", torch.stack([t, t], -1)[..., 0]
    if packed and t.dim() > 1 and t.shape[0] > 1:
        wide = torch.cat([t, t], 1)
        yield "rows apart", wide[:, :t.shape[1]]


def check_refusals(mla, call, tensors, others=(), loose=()):
    """`tensors`: name -> (tensor, the axes whose size the call knows); `loose`: names that may have rows apart."""
    good = {k: t for k, (t, _) in tensors.items()}
    call(**good)
    torch.cuda.synchronize()
    for name, (t, axes) in tensors.items():
        for what, bad in spoilt(t, axes, name not in loose):
            with pytest.raises(mla.MlaError) as e:
                call(**{**good, name: bad})
            assert e.value.code == -1 and f"({name}" in str(e.value), (name, what, str(e.value))
    for kw in others:
        with pytest.raises(mla.MlaError) as e:
            call(**{**good, **kw})
        assert e.value.code == -1, kw
    call(**good)
    torch.cuda.synchronize()


def step_tensors(T, B, pages, width):
    z = lambda *n, dtype=torch.int32: torch.zeros(n, dtype=dtype, device=DEV)
    return z, dict(q_start=(i32([0] * B + [T]), (0,)), kv_len=(i32([0] * (B - 1) + [T]), ()),
                   page_table=(z(B, width) % pages, (0,)))


@pytest.mark.parametrize("rows", [5, 1])
def test_plan_refuses_tensors_that_are_not_the_calls(mla, rows):
    B = 3
    z = lambda *n, dtype=torch.int32: torch.zeros(n, dtype=dtype, device=DEV)
    t = dict(new_len=(z(B), ()), past_len=(z(B), (0,)), free_pages=(z(4), ()), page_table=(z(B, 2), (0,)),
             q_start=(z(B + 1), (0,)), kv_len=(z(B), (0,)), seq_idx=(z(rows), ()), pos=(z(rows), (0,)),
             slot=(z(rows, dtype=torch.int64), (0,)), counts=(z(3), (0,)), device_error=(z(1), (0,)))

    def call(num_pages=8, stream=None, **kw):
        mla.plan_step(num_pages=num_pages, stream=stream, **kw)

    check_refusals(mla, call, t, others=(dict(num_pages=0), dict(num_pages=2 ** 40), dict(num_pages="8"), dict(slot=None),
                                         dict(counts=None), dict(new_len=t["kv_len"][0], past_len=t["kv_len"][0])))
    call(**{k: v for k, (v, _) in t.items() if k != "device_error"})


@pytest.mark.parametrize("dtype,per_head", [("bf16", 0), ("f32", 0), ("bf16", 1)])
def test_append_refuses_tensors_that_are_not_the_calls(mla, dtype, per_head):
    T, n_h, d_c, d_r, d_cq = 5, 3, 128, 16, 24
    dims = dims_of(mla, dtype, n_h, 32, d_c, d_r, d_cq, rope_key_per_head=per_head)
    row = d_c + (n_h if per_head else 1) * d_r
    z = lambda *n, dtype=DT[dtype]: torch.zeros(n, dtype=dtype, device=DEV)
    t = dict(kv=(z(T, row), (1,)), kv_gamma=(z(d_c), (0,)), pos=(z(T, dtype=torch.int32), (0,)),
             slot=(z(T, dtype=torch.int64) - 1, (0,)), cache=(z(2, 64, row), (1, 2)), cq=(z(T, d_cq), (0, 1)),
             cq_gamma=(z(d_cq), (0,)), cq_out=(z(T, d_cq), (0, 1)), device_error=(z(1, dtype=torch.int32), (0,)))

    def call(eps=1e-6, stream=None, **kw):
        mla.append_normed(dims, eps=eps, stream=stream, **kw)

    check_refusals(mla, call, t, loose=("kv", "cq", "cq_out"),
                   others=(dict(cq=None), dict(cq_out=None), dict(cq=None, cq_out=None), dict(eps="x"), dict(eps=-1.0),
                           dict(slot=None), dict(cache=None), dict(pos=None)))
    call(**{**{k: v for k, (v, _) in t.items() if "cq" not in k}, "kv_gamma": None})


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_query_refuses_tensors_that_are_not_the_calls(mla, dtype):
    T, n_h, d_h, d_r = 5, 3, 32, 16
    dims = dims_of(mla, dtype, n_h, d_h, 128, d_r)
    z = lambda *n, dtype=DT[dtype]: torch.zeros(n, dtype=dtype, device=DEV)
    t = dict(q=(z(T, n_h, d_h + d_r), (1, 2)), gamma=(z(d_h), (0,)), pos=(z(T, dtype=torch.int32), (0,)),
             qc_out=(z(T, n_h, d_h), (0, 1, 2)), qr_out=(z(T, n_h, d_r), (0, 1, 2)))

    def call(eps=1e-6, stream=None, **kw):
        mla.query_norm_rope(dims, eps=eps, stream=stream, **kw)

    apart = torch.zeros(T, n_h, d_h + d_r + 8, dtype=DT[dtype], device=DEV)[..., :d_h + d_r]
    check_refusals(mla, call, t, loose=("q", "qc_out", "qr_out"),
                   others=(dict(q=apart), dict(pos=None), dict(qc_out=None), dict(qr_out=None), dict(eps=None)))
    call(**{**{k: v for k, (v, _) in t.items()}, "gamma": None})


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend_refuses_tensors_that_are_not_the_calls(mla, dtype):
    T, B, pages, n_h, d_c, d_r = 5, 3, 4, 3, 128, 16
    dims = dims_of(mla, dtype, n_h, 32, d_c, d_r)
    z, t = step_tensors(T, B, pages, 2)
    t.update(q=(z(T, n_h, d_c + d_r, dtype=DT[dtype]), (1, 2)), cache=(z(pages, 64, d_c + d_r, dtype=DT[dtype]), (1, 2)),
             out=(z(T, n_h, d_c, dtype=DT[dtype]), (0, 1, 2)), lse=(z(T, n_h, dtype=torch.float32), (0, 1)))
    ws = z(mla.attend_ragged_workspace_bytes(dims, B, T), dtype=torch.uint8)

    def call(workspace=ws, stream=None, **kw):
        mla.attend_ragged(dims, workspace=workspace, stream=stream, **kw)

    check_refusals(mla, call, t, loose=("q",),
                   others=(dict(workspace=None), dict(workspace=ws.cpu()), dict(workspace=ws[::2]), dict(out=None),
                           dict(cache=None), dict(kv_len=None)))
    call(**{**{k: v for k, (v, _) in t.items()}, "lse": None})
    assert mla.get_error(ws) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ragged_step_refuses_tensors_that_are_not_the_calls(mla, dtype):
    from head_latent_attention_append_b200 import synth, workload
    wl = synth.Workload("ragged", 22, 4, 32, 32, 128, 16, 128, 0, dtype, "decode", 2, 1, 0)
    weights = mla.Weights(workload.dims_of(wl), workload.upload_weights(wl, synth.make_weights(wl, 5), torch.device(DEV)))
    T, B, pages = 5, 3, 4
    z, t = step_tensors(T, B, pages, 2)
    t.update(h=(z(T, 128, dtype=DT[dtype]), (1,)), seq_idx=(i32([B - 1] * T), (0,)), pos=(i32(range(T)), (0,)),
             cache=(z(pages, 64, 144, dtype=DT[dtype]), (1, 2)), out=(z(T, 4, 32, dtype=torch.float32), (0, 1, 2)))
    ws = z(mla.ragged_step_workspace_bytes(weights.dims, B, T), dtype=torch.uint8)

    def call(num_pages=pages, workspace=ws, stream=None, w=weights, **kw):
        mla.ragged_step(w, kw["h"], kw["q_start"], kw["kv_len"], kw["seq_idx"], kw["pos"], kw["page_table"], num_pages,
                        kw["cache"], kw["out"], workspace, stream)

    check_refusals(mla, call, t, others=(dict(num_pages=pages + 1), dict(num_pages=0), dict(num_pages=None),
                                         dict(workspace=None), dict(workspace=ws.cpu()), dict(h=None), dict(out=None)))
    assert mla.get_error(ws) == 0
    with pytest.raises(mla.MlaError) as e:
        call(workspace=ws[:-256].contiguous(), **{k: v for k, (v, _) in t.items()})
    assert e.value.code == -3
    call(num_pages=pages - 1, **{k: v for k, (v, _) in t.items()})          # fewer than the cache has: allowed
    weights.close()
    with pytest.raises(mla.MlaError) as e:
        call(**{k: v for k, (v, _) in t.items()})
    assert e.value.code == -1


def test_a_stream_that_is_none_is_refused(mla):
    """Not run on the legacy stream, which is what a failed conversion to an address gives."""
    class Stream:
        def __init__(self, handle):
            self.cuda_stream = handle

    t = dict(q=torch.ones(1, 1, 48, device=DEV), gamma=None, pos=i32([0]))
    dims = dims_of(mla, "f32", 1, 32, 64, 16)
    qc, qr = torch.zeros(1, 1, 32, device=DEV), torch.zeros(1, 1, 16, device=DEV)
    for bad in ("0", 0.5, 2 ** 70, Stream("0"), Stream(None), Stream(2 ** 70), object()):
        with pytest.raises(mla.MlaError) as e:
            mla.query_norm_rope(dims, **t, qc_out=qc, qr_out=qr, stream=bad)
        assert e.value.code == -1
        torch.cuda.synchronize()
        assert not qc.any() and not qr.any()
    for good in (None, 0, torch.cuda.current_stream(), torch.cuda.Stream(), Stream(0)):
        qc.zero_()
        torch.cuda.synchronize()
        mla.query_norm_rope(dims, **t, qc_out=qc, qr_out=qr, stream=good)
        torch.cuda.synchronize()
        assert (qc == 1).all()


# ---------------------------------------------------------------- ragged step
def small_model(mla, dtype, seed=31):
    from head_latent_attention_append_b200 import synth, workload
    wl = synth.Workload("ragged", seed, 8, 64, 64, 128, 32, 256, 64, dtype, "decode", 2, 1, 0)
    return mla.Weights(workload.dims_of(wl), workload.upload_weights(wl, synth.make_weights(wl, 5), torch.device(DEV)))


class Serving:
    """Plan and step of up to B requests on buffers of `rows` rows."""

    def __init__(self, mla, w, B, rows, num_pages, width, seed):
        d, dt = w.dims, DT["bf16" if w.dims.dtype == mla.BF16 else "f32"]
        self.mla, self.w, self.num_pages = mla, w, num_pages
        self.new, self.past, self.free = i32([0] * B), i32([0] * B), torch.randperm(num_pages, generator=gen(seed), device=DEV).int()
        self.table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
        self.q_start, self.kv_len, self.counts = i32([0] * (B + 1)), i32([0] * B), i32([0] * 3)
        self.seq, self.pos = i32([0] * rows), i32([0] * rows)
        self.slot = torch.zeros(rows, dtype=torch.int64, device=DEV)
        self.h = randn(gen(seed + 1), rows, d.d_model, dtype=dt)
        self.cache = torch.full((num_pages, 64, d.d_c + d.d_r), float("nan"), dtype=dt, device=DEV)
        self.out = torch.zeros(rows, d.n_h, d.d_v, device=DEV)
        self.ws = torch.empty(mla.ragged_step_workspace_bytes(d, B, rows), dtype=torch.uint8, device=DEV)

    def step(self):
        self.mla.plan_step(self.new, self.past, self.free, self.table, self.num_pages, self.q_start, self.kv_len, self.seq,
                           self.pos, self.slot, self.counts)
        self.mla.ragged_step(self.w, self.h, self.q_start, self.kv_len, self.seq, self.pos, self.table, self.num_pages,
                             self.cache, self.out, self.ws)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ragged_step_in_a_graph_on_another_stream(mla, dtype):
    """Captured with the plan, replayed with other lengths: bit for bit what the calls give one by one."""
    s = Serving(mla, small_model(mla, dtype), B=4, rows=150, num_pages=12, width=4, seed=3)
    s.new.copy_(i32([1, 2, 3, 4]))
    s.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        s.step()
    for lens in ([1, 2, 3, 4], [150, 0, 0, 0], [64, 65, 1, 20], [0, 0, 0, 0], [0, 1, 0, 0], [100, 60, 0, 1]):
        got = []
        for go in (graph.replay, s.step):
            s.new.copy_(i32(lens))
            s.table.fill_(-1)
            s.cache.fill_(float("nan"))
            s.out.fill_(7)
            go()
            used = int(s.counts[1])
            assert mla.get_error(s.ws) == 0
            got.append((used, s.out[:used].clone(), s.cache.clone(), s.table.clone()))
        used = got[0][0]
        assert used == (100 if lens[:2] == [100, 60] else sum(lens)) == got[1][0]
        assert torch.equal(got[0][1], got[1][1]) and torch.isfinite(got[0][1]).all() and torch.equal(got[0][3], got[1][3])
        assert torch.equal(got[0][2].nan_to_num(9.0), got[1][2].nan_to_num(9.0))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ragged_steps_on_two_streams_at_once(mla, dtype):
    w = small_model(mla, dtype)
    sides = [Serving(mla, w, B=3, rows=90, num_pages=9, width=3, seed=5), Serving(mla, w, B=40, rows=64, num_pages=50, width=2, seed=6)]
    sides[0].new.copy_(i32([70, 1, 12]))
    sides[1].new.copy_(i32([1] * 39 + [20]))
    want = []
    for s in sides:
        s.step()
        want.append(s.out[:int(s.counts[1])].clone())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for s, st in zip(sides, streams):
            with torch.cuda.stream(st):
                s.out.fill_(7)
                s.step()
        torch.cuda.synchronize()
        for s, x in zip(sides, want):
            assert torch.equal(s.out[:x.shape[0]], x)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ragged_step_of_no_token_and_of_a_workspace_for_more(mla, dtype):
    w = small_model(mla, dtype)
    big = torch.empty(mla.ragged_step_workspace_bytes(w.dims, 30, 700), dtype=torch.uint8, device=DEV)
    for B, rows in ((1, 1), (2, 5), (30, 700), (30, 699), (5, 64), (29, 513)):
        s = Serving(mla, w, B=B, rows=rows, num_pages=60, width=13, seed=B)
        s.new.copy_(i32([rows - (B - 1)] + [1] * (B - 1)))
        s.step()
        want, own = s.out.clone(), s.ws
        s.ws = big
        s.step()
        assert mla.get_error(own) == 0 and mla.get_error(big) == 0 and torch.equal(s.out, want) and torch.isfinite(want).all()
    s = Serving(mla, w, B=2, rows=0, num_pages=2, width=1, seed=1)
    s.ws = big
    s.step()
    assert s.kv_len.tolist() == [0, 0]


@pytest.mark.parametrize("dtype,n_h,d_c,d_r", [("bf16", 16, 256, 32), ("bf16", 128, 128, 64), ("f32", 8, 64, 16), ("f32", 5, 61, 6)])
def test_steps_one_behind_the_other_on_the_same_buffers(mla, dtype, n_h, d_c, d_r):
    """Each kernel of a step starts while the one before it ends and reads what that one has written, into buffers that
    the step before read: three steps in one graph, against the same calls with the GPU waited for after each."""
    B, rows, num_pages, width, d_h = 6, 120, 40, 6, 32
    dims, dt, g = dims_of(mla, dtype, n_h, d_h, d_c, d_r), DT[dtype], gen(8)
    plans = [([40, 1, 30, 2, 0, 17], [0] * 6), ([1, 1, 1, 70, 5, 3], [40, 1, 30, 2, 0, 17]),
             ([3, 64, 1, 1, 1, 40], [41, 2, 31, 72, 5, 20])]
    plans = [(i32(n), i32(p)) for n, p in plans]
    free = torch.randperm(num_pages, generator=g, device=DEV).int().view(4, 10)
    kv, q = [randn(g, rows, d_c + d_r, dtype=dt) for _ in plans], [randn(g, rows, n_h, d_h + d_r, dtype=dt) for _ in plans]
    gk, gq = randn(g, d_c, dtype=dt), randn(g, d_h, dtype=dt)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    q_start, kv_len, seq, pos = i32([0] * (B + 1)), i32([0] * B), i32([0] * rows), i32([0] * rows)
    slot, counts = torch.zeros(rows, dtype=torch.int64, device=DEV), i32([0] * 3)
    cache = torch.zeros(num_pages, 64, d_c + d_r, dtype=dt, device=DEV)
    absorbed, qc = randn(g, rows, n_h, d_c + d_r, dtype=dt), torch.empty(rows, n_h, d_h, dtype=dt, device=DEV)
    outs = [torch.zeros(rows, n_h, d_c, dtype=dt, device=DEV) for _ in plans]
    lses = [torch.zeros(rows, n_h, device=DEV) for _ in plans]
    ws = torch.empty(mla.attend_ragged_workspace_bytes(dims, B, rows), dtype=torch.uint8, device=DEV)

    def steps(after=lambda: None):
        for i, (new, past) in enumerate(plans):
            mla.plan_step(new, past, free[i], table, num_pages, q_start, kv_len, seq, pos, slot, counts)
            after()
            mla.append_normed(dims, kv[i], gk, pos, slot, cache)
            after()
            mla.query_norm_rope(dims, q[i], gq, pos, qc, absorbed[..., d_c:])
            after()
            mla.attend_ragged(dims, absorbed, q_start, kv_len, table, cache, outs[i], lses[i], ws)
            after()

    def begin():
        table.fill_(-1)
        cache.zero_()
        for t in outs + lses:
            t.fill_(7)
        torch.cuda.synchronize()

    begin()
    steps(torch.cuda.synchronize)
    want = [t.clone() for t in outs + lses + [cache, table]]
    assert mla.get_error(ws) == 0 and all(torch.isfinite(t.float()).all() for t in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        steps()
    for go in [graph.replay, steps] * 10:
        begin()
        go()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs + lses + [cache, table], want))
