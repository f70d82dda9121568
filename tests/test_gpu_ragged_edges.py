"""More uses of the ragged-step calls (GPU) that their documentation allows,
against the definitions in 64 bits; tolerances as in test_gpu_ragged.py."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_ragged import Step, mla  # noqa: E402,F401  (the fixture)


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
