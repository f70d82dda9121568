"""More uses of the ragged-step calls (GPU) that their documentation allows,
against the definitions in 64 bits; tolerances as in test_gpu_ragged.py."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_ragged import DEV, DT, Step, close_norm, dims_of, gen, i32, mla, randn, rms64  # noqa: E402,F401


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
