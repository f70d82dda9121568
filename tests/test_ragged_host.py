"""The ragged-step calls without a GPU: sizes, refusals of the C ABI before any
CUDA call, and the binding's checks of its tensors."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

FAKE = 0x100000  # aligned, never dereferenced: every call below returns before any CUDA call
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3


@pytest.fixture(scope="module")
def mla():
    from head_latent_attention_append_b200 import build
    build.build()
    from head_latent_attention_append_b200 import mla as m
    return m


def dims(mla, **kw):
    d = dict(n_h=16, d_h=128, d_v=128, d_c=256, d_r=32, d_model=2048, d_cq=1536)
    d.update(kw)
    return mla.make_dims(**d)


def call(fn, defaults, **kw):
    assert set(kw) <= set(defaults), kw
    return fn(*{**defaults, **kw}.values())


def test_plan_refusals(mla):
    out = FAKE + 4096
    ok = dict(new_len=FAKE, past_len=FAKE, B=4, free_pages=FAKE, n_free=9, page_table=out, max_pages=8, num_pages=99,
              q_start=out, kv_len=out, seq_idx=out, pos=out, slot=out, rows=5, counts=out, err=None, stream=None)
    f = mla.lib.mla_plan_step
    for bad in ("new_len", "past_len", "page_table", "q_start", "kv_len", "counts", "free_pages", "seq_idx", "pos", "slot"):
        assert call(f, ok, **{bad: None}) == INVALID, bad
        assert call(f, ok, **{bad: FAKE + 2}) == INVALID, bad
    for bad in (dict(B=0), dict(B=-1), dict(n_free=-1), dict(max_pages=0), dict(num_pages=0), dict(rows=-1),
                dict(slot=FAKE + 4), dict(err=FAKE + 1)):
        assert call(f, ok, **bad) == INVALID, bad
    # Outputs in the place of lengths or free pages that other CTAs still read.
    for bad in (dict(kv_len=FAKE), dict(q_start=FAKE + 12), dict(page_table=FAKE - 4), dict(seq_idx=FAKE + 32),
                dict(slot=FAKE - 32), dict(counts=FAKE), dict(pos=FAKE)):
        assert call(f, ok, **bad) == INVALID, bad
    for bad in (dict(B=16385), dict(rows=2 ** 31 - 1), dict(rows=2 ** 30 + 1), dict(n_free=2 ** 31 - 1), dict(max_pages=2 ** 25)):
        assert call(f, ok, **bad) == UNSUPPORTED, bad


def test_append_normed_refusals(mla):
    d = dims(mla)
    ok = dict(dims=ctypes.byref(d), kv=FAKE, kv_stride=288, kv_gamma=FAKE, cq=FAKE, cq_stride=1536, cq_gamma=FAKE,
              cq_out=FAKE, cq_out_stride=1536, eps=1e-6, pos=FAKE, slot=FAKE, cache=FAKE, num_pages=4, T=3, err=None,
              stream=None)
    f = mla.lib.mla_append_normed
    for bad in (dict(dims=None), dict(kv=None), dict(pos=None), dict(slot=None), dict(cache=None), dict(kv_stride=287),
                dict(cq=None), dict(cq_out=None), dict(cq_stride=1535), dict(cq_out_stride=8), dict(eps=-1.0),
                dict(eps=float("nan")), dict(num_pages=0), dict(T=-1), dict(kv=FAKE + 1), dict(cache=FAKE + 8),
                dict(slot=FAKE + 4), dict(kv_gamma=FAKE + 1), dict(err=FAKE + 2),
                dict(cq=None, cq_out=None)):           # a gamma without its latent
        assert call(f, ok, **bad) == INVALID, bad
    assert call(f, ok, T=0) == 0
    plain = dims(mla, d_cq=0)
    assert call(f, ok, dims=ctypes.byref(plain)) == INVALID
    odd = dims(mla, d_r=15)
    assert call(f, ok, dims=ctypes.byref(odd)) == UNSUPPORTED


def test_query_norm_rope_refusals(mla):
    d = dims(mla)
    ok = dict(dims=ctypes.byref(d), q=FAKE, q_stride=16 * 160, gamma=FAKE, eps=1e-6, pos=FAKE, qc=FAKE, qc_ts=16 * 128,
              qc_hs=128, qr=FAKE, qr_ts=16 * 32, qr_hs=32, T=2, stream=None)
    f = mla.lib.mla_query_norm_rope
    for bad in (dict(dims=None), dict(q=None), dict(pos=None), dict(qc=None), dict(qr=None), dict(q_stride=2559),
                dict(qc_ts=2047), dict(qc_hs=127), dict(qr_ts=511), dict(qr_hs=31), dict(T=-1), dict(eps=-1.0),
                dict(q=FAKE + 1), dict(gamma=FAKE + 1), dict(qr=FAKE + 1)):
        assert call(f, ok, **bad) == INVALID, bad
    assert call(f, ok, T=0) == 0


def test_attend_ragged_refusals_and_sizes(mla):
    d = dims(mla)
    need = mla.attend_ragged_workspace_bytes(d, 4, 70)
    assert need > 2 * 160 * 64 * 256 * 4
    out = FAKE + 2 * 70 * 16 * 288
    ok = dict(dims=ctypes.byref(d), q=FAKE, q_ts=16 * 288, q_hs=288, q_start=FAKE, kv_len=FAKE, table=FAKE, max_pages=8,
              num_pages=99, cache=FAKE, out=out, lse=FAKE, B=4, T=70, ws=FAKE, ws_bytes=need, stream=None)
    f = mla.lib.mla_attend_ragged
    for bad in (dict(dims=None), dict(q=None), dict(q_start=None), dict(kv_len=None), dict(table=None), dict(cache=None),
                dict(out=None), dict(ws=None), dict(B=0), dict(T=-1), dict(max_pages=0), dict(num_pages=0),
                dict(num_pages=2 ** 26), dict(max_pages=2 ** 26), dict(q_hs=280), dict(q_ts=16 * 288 - 8),
                dict(q_hs=289, q_ts=16 * 289), dict(q_ts=16 * 288 + 4), dict(q=FAKE + 8), dict(out=out + 8), dict(out=out - 16), dict(out=FAKE),
                dict(ws=FAKE + 64), dict(lse=FAKE + 2)):
        assert call(f, ok, **bad) == INVALID, bad
    assert call(f, ok, ws_bytes=need - 1) == WORKSPACE
    assert call(f, ok, T=0) == 0
    for bad in (dict(B=16385), dict(T=2 ** 28)):
        assert call(f, ok, **bad) == UNSUPPORTED, bad
    per_head = dims(mla, rope_key_per_head=1, d_c=128)
    assert call(f, ok, dims=ctypes.byref(per_head)) == UNSUPPORTED
    assert mla.attend_ragged_workspace_bytes(per_head, 4, 70) == 0
    assert mla.attend_ragged_workspace_bytes(d, 0, 70) == 0
    # More tokens never need less.
    sizes = [mla.attend_ragged_workspace_bytes(d, 4, t) for t in (1, 70, 1000, 100000)]
    assert sizes == sorted(sizes)


def test_rows_past_32_bits_are_refused(mla):
    """A warp of the normalised append counts on from its row by a whole grid: T leaves room for that."""
    f = mla.lib.mla_append_normed
    for d in (dims(mla), dims(mla, dtype=mla.F32), dims(mla, dtype=mla.F32, d_c=16, d_r=2)):
        ok = dict(dims=ctypes.byref(d), kv=FAKE, kv_stride=288, kv_gamma=None, cq=None, cq_stride=0, cq_gamma=None,
                  cq_out=None, cq_out_stride=0, eps=1e-6, pos=FAKE, slot=FAKE, cache=FAKE, num_pages=4, T=0, err=None,
                  stream=None)
        assert call(f, ok) == 0
        for T in (2 ** 31 - 1, 2 ** 30 + 1):
            assert call(f, ok, T=T) == UNSUPPORTED


def test_the_binding_refuses_tensors_it_could_not_pass_on(mla):
    """Shapes, types and devices are checked before the library sees an address; tensors on the CPU never get there."""
    d = dims(mla, d_cq=0)
    bf, i32 = torch.bfloat16, torch.int32
    q, out = torch.zeros(5, 16, 288, dtype=bf), torch.zeros(5, 16, 256, dtype=bf)
    starts, kv, table = torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(2, 4, dtype=i32)
    cache, lse, ws = torch.zeros(3, 64, 288, dtype=bf), torch.zeros(5, 16), torch.zeros(64, dtype=torch.uint8)
    ok = dict(q=q, q_start=starts, kv_len=kv, page_table=table, cache=cache, out=out, lse=lse, workspace=ws)
    for name, t in (("q", q.float()), ("q", q[..., :256]), ("q", q[:, :15]), ("q_start", starts[:2]),
                    ("q_start", starts.long()), ("kv_len", kv.float()), ("page_table", table[:1]),
                    ("page_table", table.t().contiguous().t()), ("cache", cache[:, :32]), ("cache", cache.float()),
                    ("cache", cache[:, :, :280]), ("out", out[:4]), ("out", out.float()), ("lse", lse[:, :3]),
                    ("lse", lse.to(bf)), ("q", q.transpose(1, 2).contiguous().transpose(1, 2)), ("kv_len", kv.to("meta")),
                    ("workspace", ws)):
        with pytest.raises(mla.MlaError) as e:
            mla.attend_ragged(d, **{**ok, name: t})
        assert e.value.code == INVALID and (name in str(e.value) or name == "workspace")
    kvr, pos, slot = torch.zeros(5, 288, dtype=bf), torch.zeros(5, dtype=i32), torch.zeros(5, dtype=torch.int64)
    gamma = torch.ones(256, dtype=bf)
    ok = dict(kv=kvr, kv_gamma=gamma, pos=pos, slot=slot, cache=cache)
    for name, t in (("kv", kvr[:, :256]), ("kv", kvr.float()), ("kv_gamma", gamma[:8]), ("pos", pos[:4]), ("pos", pos.long()),
                    ("slot", slot.int()), ("cache", cache[..., :256]), ("cq", kvr), ("cq_out", kvr), ("kv", kvr)):
        with pytest.raises(mla.MlaError):
            mla.append_normed(d, **{**ok, name: t})
    qq, qc, qr = torch.zeros(5, 16, 160, dtype=bf), torch.zeros(5, 16, 128, dtype=bf), torch.zeros(5, 16, 32, dtype=bf)
    ok = dict(q=qq, gamma=None, pos=pos, qc_out=qc, qr_out=qr)
    for name, t in (("q", qq[:, :, :128]), ("q", qq[:, :8]), ("gamma", gamma), ("qc_out", qr), ("qr_out", qc), ("pos", slot),
                    ("qc_out", qc.float()), ("q", torch.zeros(5, 16, 200, dtype=bf)[..., :160]), ("q", qq)):
        with pytest.raises(mla.MlaError):
            mla.query_norm_rope(d, **{**ok, name: t})
    v = torch.zeros(2, dtype=i32)
    ok = dict(new_len=v, past_len=v, free_pages=v, page_table=table, num_pages=9, q_start=starts, kv_len=v,
              seq_idx=pos, pos=pos, slot=slot, counts=starts)
    for name, t in (("past_len", starts), ("page_table", table[:1]), ("q_start", v), ("kv_len", starts), ("pos", v),
                    ("slot", pos), ("counts", v), ("free_pages", slot), ("new_len", v)):
        with pytest.raises(mla.MlaError):
            mla.plan_step(**{**ok, name: t})


def test_ragged_step_refusals_and_sizes(mla):
    d = dims(mla)
    need = mla.ragged_step_workspace_bytes(d, 4, 70)
    assert need >= mla.attend_ragged_workspace_bytes(d, 4, 70) + 2 * 70 * 16 * (128 + 288 + 256) + 2 * 70 * 1536
    assert mla.ragged_step_workspace_bytes(d, 0, 70) == 0 and mla.ragged_step_workspace_bytes(d, 4, -1) == 0
    assert mla.ragged_step_workspace_bytes(dims(mla, rope_key_per_head=1, d_c=128), 4, 70) == 0
    # A null handle is refused before anything else is looked at.
    assert mla.lib.mla_ragged_step(None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 4, 9, FAKE, FAKE, 4, 70, FAKE, need, None) == INVALID


def test_append_and_query_refuse_outputs_over_their_inputs(mla):
    """An output row may be its own input row, at the same addresses and strides; every other overlap would be read half
    written."""
    d = dims(mla)
    at = lambda i: FAKE + (i << 24)
    ok = dict(dims=ctypes.byref(d), kv=at(0), kv_stride=288, kv_gamma=at(1), cq=at(2), cq_stride=1600, cq_gamma=at(3),
              cq_out=at(4), cq_out_stride=1536, eps=1e-6, pos=at(5), slot=at(6), cache=at(7), num_pages=4, T=5, err=None,
              stream=None)
    f = mla.lib.mla_append_normed
    row = 2 * 1600
    for bad in (dict(cq_out=at(2)),                                        # c_Q's rows with another stride
                dict(cq_out=at(2) + 16, cq_out_stride=1600), dict(cq_out=at(2) + row, cq_out_stride=1600),
                dict(cq_out=at(2) - row, cq_out_stride=1600), dict(cq_out=at(2) + 2 * 1535, cq_out_stride=1600),
                dict(cq_out=at(0)), dict(cq_out=at(0) + 4 * 2 * 288 + 2 * 287), dict(cq_out=at(1)), dict(cq_out=at(3)),
                dict(cq_out=at(5)), dict(cq_out=at(6)), dict(cq_out=at(7)), dict(cache=at(0)), dict(cache=at(2)),
                dict(cache=at(4)), dict(cache=at(6)), dict(cache=at(5) - 4 * 64 * 288 * 2 + 16), dict(cache=at(1)),
                dict(kv=at(2) + 2 * 1500, kv_stride=1600, cq_out=at(2), cq_out_stride=1600)):
        assert call(f, ok, **bad) == INVALID, bad
    ok = dict(dims=ctypes.byref(d), q=at(0), q_stride=16 * 160, gamma=at(1), eps=1e-6, pos=at(2), qc=at(3), qc_ts=16 * 128,
              qc_hs=128, qr=at(4), qr_ts=16 * 32, qr_hs=32, T=2, stream=None)
    f = mla.lib.mla_query_norm_rope
    own = dict(q_stride=16 * 160, qc_ts=16 * 160, qc_hs=160, qr_ts=16 * 160, qr_hs=160)
    for bad in (dict(qc=at(0)), dict(qr=at(0)), dict(qr=at(0) + 2 * 128), dict(qc=at(1)), dict(qr=at(1)), dict(qc=at(2)),
                dict(qr=at(2)), dict(qr=at(3)), dict(qc=at(4) - 2 * 16 * 128 + 2), {**own, "qc": at(0) + 2},
                {**own, "qc": at(0), "qr": at(0) + 2 * 126}, {**own, "qc": at(0) + 2 * 160}, {**own, "qr": at(0)},
                {**own, "qr": at(0) + 2 * (128 + 16 * 160)}, {**own, "qc": at(0) - 2 * 16 * 160}):
        assert call(f, ok, **bad) == INVALID, bad


def test_arguments_that_are_no_tensors_are_named(mla):
    """The calls' own error, whichever argument is not a tensor."""
    d = dims(mla, d_cq=0)
    t = torch.zeros(2, 3, 4)
    calls = {
        "plan_step": (mla.plan_step, ("new_len", "past_len", "free_pages", "page_table", "q_start", "kv_len", "seq_idx", "pos",
                                      "slot", "counts"), dict(num_pages=4)),
        "append_normed": (lambda **kw: mla.append_normed(d, **kw), ("kv", "kv_gamma", "pos", "slot", "cache"), {}),
        "query_norm_rope": (lambda **kw: mla.query_norm_rope(d, **kw), ("q", "gamma", "pos", "qc_out", "qr_out"), {}),
        "attend_ragged": (lambda **kw: mla.attend_ragged(d, **kw), ("q", "q_start", "kv_len", "page_table", "cache", "out",
                                                                     "lse", "workspace"), {}),
    }
    for fn, (call_, names, more) in calls.items():
        for name in names:
            for bad in (None, [1, 2], 3, "x", t[0, 0, 0]):
                with pytest.raises(mla.MlaError) as e:
                    call_(**{**dict.fromkeys(names, t), **more, name: bad})
                assert e.value.code == INVALID and fn in str(e.value), (fn, name, bad)
        # The argument that gives the call its size.
        for bad in (None, [1, 2], 3):
            with pytest.raises(mla.MlaError, match=rf"\({names[0]}: a tensor is expected"):
                call_(**{**dict.fromkeys(names, t), **more, names[0]: bad})


def test_a_workspace_that_is_missing_is_refused(mla):
    """Everything else as the call wants it, on the CPU."""
    d = dims(mla, d_cq=0)
    bf, i32 = torch.bfloat16, torch.int32
    with pytest.raises(mla.MlaError) as e:
        mla.attend_ragged(d, torch.zeros(5, 16, 288, dtype=bf), torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32),
                          torch.zeros(2, 4, dtype=i32), torch.zeros(3, 64, 288, dtype=bf), torch.zeros(5, 16, 256, dtype=bf),
                          None, None)
    assert e.value.code == INVALID
