"""Cases and plain forms of the ragged-step operators: what a serving loop runs
around the attention when every request brings its own number of new tokens.

  plan     lengths -> page-table entries, slots, positions (mla_plan_step)
  append   RMS-norm of the two latents, rotation of the position key and the
           write into the paged cache (mla_append_normed)
  query    RMS-norm of every query head and rotation of its position part
           (mla_query_norm_rope)
  attend   attention of every request's new tokens over its paged latent
           cache (mla_attend_ragged)

`run` computes them from elementary torch operations in 32 bits (angles in 64)
while `own` is false, and through this repository's library when it is true.
"""
import math
import random

import torch

own = False

PAGE = 64
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
ROPE_BASE = 10000.0
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    dsv2 = {"n_h": 128, "d_h": 128, "d_c": 512, "d_r": 64}
    page = {"n_h": 16, "d_h": 128, "d_c": 256, "d_r": 32}
    tiny = {"n_h": 4, "d_h": 32, "d_c": 64, "d_r": 16}
    return [
        # One decode step of 64 requests, one new token each: the plan is pure latency.
        {"name": "plan_decode", "op": "plan", "B": 64, "new_max": 1, "past_max": 8192, "budget": 1.0},
        # A large engine step: 1024 requests, most of them decoding, some with a chunk of their prompt; the
        # token budget cuts the last ones off.
        {"name": "plan_mixed", "op": "plan", "B": 1024, "new_max": 512, "past_max": 32768, "budget": 0.9},
        # The new tokens of a decode step: both latents of 64 rows, latency again.
        {"name": "append_decode", "op": "append", "dtype": "bf16", "T": 64, "past_max": 8192, "d_cq": 1536, **dsv2},
        # A 32-bit model without a query latent, an odd number of rows.
        {"name": "append_f32", "op": "append", "dtype": "f32", "T": 1001, "past_max": 4096, "d_cq": 0, **page},
        # A whole prefill's tokens (4 x 4096): bound by memory.
        {"name": "append_prefill", "op": "append", "dtype": "bf16", "T": 16384, "past_max": 0, "d_cq": 1536, **dsv2},
        # The 128 query heads of a decode step's 64 tokens.
        {"name": "query_decode", "op": "query", "dtype": "bf16", "T": 64, "past_max": 8192, **dsv2},
        # 32-bit queries of a small model.
        {"name": "query_f32", "op": "query", "dtype": "f32", "T": 777, "past_max": 32768, **tiny},
        # The query heads of one prefill chunk: 400 MB through memory.
        {"name": "query_prefill", "op": "query", "dtype": "bf16", "T": 4096, "past_max": 8192, **dsv2},
        # 32-bit chunks over short histories, down to single keys.
        {"name": "attend_f32", "op": "attend", "dtype": "f32", "B": 3, "q_max": 37, "kv_max": 517, **page},
        # Single-token decode of eight requests of a 16-head model.
        {"name": "attend_decode", "op": "attend", "dtype": "bf16", "B": 8, "q_max": 1, "kv_max": 4097, **page},
        # A mixed step: requests with one or a few new tokens beside chunks of their prompt.
        {"name": "attend_mixed", "op": "attend", "dtype": "bf16", "B": 12, "q_max": 96, "kv_max": 4171, **dsv2},
        # Two long chunks over long histories: bound by the tensor cores.
        {"name": "attend_chunk", "op": "attend", "dtype": "bf16", "B": 2, "q_max": 512, "kv_max": 16001, **dsv2},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "query", "attend", "attend"])
    if op == "plan":
        return {"op": op, "B": _log(rng, 1, 1024), "new_max": _log(rng, 1, 512), "past_max": _log(rng, 1, 32768),
                "budget": rng.choice([1.0, 1.0, 0.5, 0.9])}
    dtype = rng.choice(["bf16", "bf16", "f32"])
    dims = {"n_h": _log(rng, 1, 128), "d_h": 8 * rng.randint(2, 16), "d_c": 128 * rng.randint(1, 4),
            "d_r": 16 * rng.randint(1, 4)}
    if dtype == "f32" and rng.random() < 0.5:
        dims.update(d_h=rng.randint(3, 130), d_c=rng.randint(5, 512), d_r=2 * rng.randint(1, 32))
    if op == "append":
        return {"op": op, "dtype": dtype, "T": _log(rng, 1, 16384 if dtype == "bf16" else 8192),
                "past_max": _log(rng, 1, 100000), "d_cq": rng.choice([0, 8 * rng.randint(8, 192)]), **dims}
    if op == "query":
        most = 4096 * 128 // dims["n_h"] // (2 if dtype == "f32" else 1)
        return {"op": op, "dtype": dtype, "T": _log(rng, 1, min(16384, most)), "past_max": _log(rng, 1, 100000), **dims}
    if dtype == "f32":
        return {"op": op, "dtype": dtype, "B": rng.randint(1, 6), "q_max": _log(rng, 1, 64), "kv_max": _log(rng, 64, 1500),
                **{**dims, "n_h": min(dims["n_h"], 32)}}
    case = {"op": op, "dtype": dtype, "B": rng.randint(1, 16), "q_max": _log(rng, 1, 512), "kv_max": _log(rng, 512, 16001),
            **dims}
    while case["B"] * case["q_max"] * case["n_h"] * case["kv_max"] > 1.2e9:  # the padded score tensor of the plain form
        case["B"] = max(1, case["B"] // 2)
        case["q_max"] = max(1, case["q_max"] * 2 // 3)
    return case


def _lengths(case):
    """(new tokens, cached tokens) of every request, from the case alone."""
    r = random.Random("%(B)d %(new)d %(past)d" % {"B": case["B"], "new": case.get("new_max", case.get("q_max")),
                                                  "past": case.get("past_max", case.get("kv_max"))})
    if case["op"] == "plan":
        new = [1 if r.random() < 0.75 else _log(r, 1, case["new_max"]) for _ in range(case["B"])]
        return new, [r.randint(0, case["past_max"]) for _ in new]
    # The first request is the longest of both kinds; the others fall anywhere, some of them empty.
    new, past = [case["q_max"]], [case["kv_max"] - case["q_max"]]
    for _ in range(case["B"] - 1):
        q = 0 if r.random() < 0.05 else _log(r, 1, case["q_max"])
        new.append(q)
        past.append(r.randint(0, case["kv_max"] - q))
    return new, past


def _plan_rows(case):
    new, _ = _lengths(case)
    return max(1, int(sum(new) * case["budget"]))


def work(case):
    op = case["op"]
    if op == "plan":
        new, past = _lengths(case)
        rows, pages, tokens = _plan_rows(case), 0, 0
        for n, p in zip(new, past):
            if tokens + n > rows:
                break
            tokens += n
            pages += -(-(p + n) // PAGE) - -(-p // PAGE)
        b = case["B"]
        return {"bytes": 8 * b + 4 * b + 8 * pages + 4 * (2 * b + 1) + 16 * rows, "flops": 4 * rows}
    e = 2 if case["dtype"] == "bf16" else 4
    if op == "append":
        width = case["d_c"] + case["d_r"] + case["d_cq"]
        return {"bytes": case["T"] * (2 * e * width + 12) + e * (case["d_c"] + case["d_cq"]), "flops": 4 * case["T"] * width}
    if op == "query":
        width = case["n_h"] * (case["d_h"] + case["d_r"])
        return {"bytes": case["T"] * (2 * e * width + 4) + e * case["d_h"], "flops": 4 * case["T"] * width}
    new, past = _lengths(case)
    row, rows = case["d_c"] + case["d_r"], sum(new)
    pairs = sum(n * p + n * (n + 1) // 2 for n, p in zip(new, past))
    keys = sum(n + p for n, p in zip(new, past) if n)
    return {"bytes": e * row * keys + rows * case["n_h"] * (e * (row + case["d_c"]) + 4),
            "flops": pairs * case["n_h"] * (2 * row + 2 * case["d_c"])}


# ----------------------------------------------------------------- the inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _dims(case):
    from head_latent_attention_append_b200 import mla
    return mla.make_dims(case["n_h"], case["d_h"], case["d_h"], case["d_c"], case["d_r"], 2048, case.get("d_cq", 0),
                         ROPE_BASE, page_size=PAGE, dtype=mla.BF16 if case["dtype"] == "bf16" else mla.F32)


def prepare(case, seed):
    s = {"op": case["op"], "case": case}
    g = _gen(seed)
    if case["op"] == "plan":
        new, past = _lengths(case)
        b, rows = case["B"], _plan_rows(case)
        have = [-(-p // PAGE) for p in past]
        want = [-(-(p + n) // PAGE) for n, p in zip(new, past)]
        width, n_free = max(1, max(want)), sum(want) - sum(have) + 7
        num_pages = sum(have) + n_free
        ids = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
        table = torch.full((b, width), -1, dtype=torch.int32, device="cuda")
        held = torch.arange(width, device="cuda")[None, :] < torch.tensor(have, device="cuda")[:, None]
        table[held] = ids[:sum(have)]
        s.update(new_len=_i32(new), past_len=_i32(past), page_table=table, free_pages=ids[sum(have):].contiguous(),
                 num_pages=num_pages, rows=rows, q_start=_i32([0] * (b + 1)), kv_len=_i32([0] * b),
                 seq_idx=_i32([0] * rows), pos=_i32([0] * rows), counts=_i32([0] * 3),
                 slot=torch.zeros(rows, dtype=torch.int64, device="cuda"))
        return s
    dt = DTYPE[case["dtype"]]
    n_h, d_h, d_c, d_r = (case[k] for k in ("n_h", "d_h", "d_c", "d_r"))
    s["dims"] = _dims(case)
    if case["op"] in ("append", "query"):
        t = case["T"]
        s["pos"] = (torch.randint(0, case["past_max"] + 1, (t,), generator=g, device="cuda") if case["past_max"]
                    else torch.arange(t, device="cuda") % 4096).to(torch.int32)
    if case["op"] == "append":
        # One down-projection gives [query latent | latent | position key]: the operator reads slices of its rows.
        x = _normal(g, t, case["d_cq"] + d_c + d_r, dtype=dt, scale=1.5)
        num_pages = -(-t // PAGE) + 3
        s.update(kv=x[:, case["d_cq"]:], kv_gamma=_normal(g, d_c, dtype=dt, scale=0.1) + 1,
                 slot=torch.randperm(num_pages * PAGE, generator=g, device="cuda")[:t].contiguous(),
                 cache=_normal(g, num_pages, PAGE, d_c + d_r, dtype=dt), cq=None, cq_gamma=None, cq_out=None)
        if case["d_cq"]:
            s.update(cq=x[:, :case["d_cq"]], cq_gamma=_normal(g, case["d_cq"], dtype=dt, scale=0.1) + 1,
                     cq_out=torch.empty(t, case["d_cq"], dtype=dt, device="cuda"))
    elif case["op"] == "query":
        # The position part goes straight into the rows that the attention reads, [absorbed content | position].
        s.update(q=_normal(g, t, n_h, d_h + d_r, dtype=dt, scale=1.5), gamma=_normal(g, d_h, dtype=dt, scale=0.1) + 1,
                 qc_out=torch.empty(t, n_h, d_h, dtype=dt, device="cuda"),
                 qr_out=torch.zeros(t, n_h, d_c + d_r, dtype=dt, device="cuda")[..., d_c:])
    else:
        new, past = _lengths(case)
        total, kv = sum(new), [n + p for n, p in zip(new, past)]
        pages = [-(-k // PAGE) for k in kv]
        width = max(1, max(pages))
        ids = torch.randperm(sum(pages) + 2, generator=g, device="cuda").to(torch.int32)
        held = torch.arange(width, device="cuda")[None, :] < torch.tensor(pages, device="cuda")[:, None]
        table = torch.full((case["B"], width), -1, dtype=torch.int32, device="cuda")
        table[held] = ids[:sum(pages)]
        starts = [0]
        for n in new:
            starts.append(starts[-1] + n)
        s.update(q=_normal(g, total, n_h, d_c + d_r, dtype=dt), q_start=_i32(starts), kv_len=_i32(kv), page_table=table,
                 cache=_normal(g, sum(pages) + 2, PAGE, d_c + d_r, dtype=dt), q_most=max(new), kv_most=max(kv),
                 out=torch.empty(total, n_h, d_c, dtype=dt, device="cuda"),
                 lse=torch.empty(total, n_h, dtype=torch.float32, device="cuda"), workspace=None)
    return s


# -------------------------------------------------------------- the plain forms
def _plain_plan(s):
    new, past, table, free = s["new_len"].long(), s["past_len"].long(), s["page_table"], s["free_pages"]
    width = table.shape[1]
    ok = (new >= 0) & (past >= 0) & (past + new <= width * PAGE)
    new = torch.where(ok, new, 0)
    have = torch.where(ok, (past + PAGE - 1) // PAGE, 0)
    need = torch.where(ok, (past + new + PAGE - 1) // PAGE, 0) - have
    pages = torch.cumsum(need, 0)
    fits = (torch.cumsum(new, 0) <= s["rows"]) & (pages <= free.shape[0])
    new, need = torch.where(fits, new, 0), torch.where(fits, need, 0)
    ends = torch.cumsum(new, 0)
    q_start = torch.cat([torch.zeros_like(ends[:1]), ends])
    kv_len = torch.where(ok, past + new, 0)
    col = torch.arange(width, device="cuda")[None, :] - have[:, None]
    fresh = (col >= 0) & (col < need[:, None])
    at = (torch.cumsum(need, 0) - need)[:, None] + col
    table = torch.where(fresh, free[torch.where(fresh, at, 0)], table)
    row = torch.arange(s["rows"], device="cuda")
    live = row < ends[-1]
    seq = torch.where(live, torch.searchsorted(ends, row, right=True), 0)
    pos = torch.where(live, past[seq] + row - q_start[seq], 0)
    page = table[seq, pos // PAGE].long()
    slot = torch.where(live & (page >= 0) & (page < s["num_pages"]), page * PAGE + pos % PAGE, -1)
    counts = torch.stack([fits.sum(), ends[-1], need.sum()])
    return {"page_table": table, "q_start": q_start.int(), "kv_len": kv_len.int(), "slot": slot, "pos": pos.int(),
            "seq_idx": torch.where(live, seq, -1).int(), "counts": counts.int()}


def _rms(x, gamma):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gamma.float()


def _rotate(x, pos):
    """Pairs (2i, 2i+1) of the last axis by pos * base^(-2i/d): x [T, ..., d], the angle in 64 bits."""
    d = x.shape[-1]
    theta = ROPE_BASE ** (-torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d)
    angle = (pos.double()[:, None] * theta).view(-1, *([1] * (x.dim() - 2)), d // 2)
    c, n = torch.cos(angle).float(), torch.sin(angle).float()
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * c - b * n, a * n + b * c], -1).flatten(-2)


def _plain_append(s):
    d_c, dt = s["case"]["d_c"], s["kv"].dtype
    x = s["kv"].float()
    rows = torch.cat([_rms(x[:, :d_c], s["kv_gamma"]), _rotate(x[:, d_c:], s["pos"])], 1)
    s["cache"].view(-1, rows.shape[1])[s["slot"]] = rows.to(dt)
    return {"cache": s["cache"], "cq": None if s["cq"] is None else _rms(s["cq"].float(), s["cq_gamma"]).to(dt)}


def _plain_query(s):
    d_h, dt, x = s["case"]["d_h"], s["q"].dtype, s["q"].float()
    return {"qc": _rms(x[..., :d_h], s["gamma"]).to(dt), "qr": _rotate(x[..., d_h:], s["pos"]).to(dt)}


def _plain_attend(s):
    case, q, starts, kv_len = s["case"], s["q"], s["q_start"].long(), s["kv_len"].long()
    b, n_h, d_c, width, most = case["B"], case["n_h"], case["d_c"], s["kv_most"], s["q_most"]
    row = d_c + case["d_r"]
    pages = s["page_table"][:, :-(-width // PAGE)].long().clamp(0)
    key = torch.arange(width, device="cuda")
    k = s["cache"][pages].view(b, -1, row)[:, :width].float()
    k = torch.where((key < kv_len[:, None])[..., None], k, 0)
    at = starts[:-1, None] + torch.arange(most, device="cuda")
    x = q[at.clamp(max=q.shape[0] - 1)].float().view(b, most * n_h, row)
    scale = 1.0 / math.sqrt(case["d_h"] + case["d_r"])
    a = torch.matmul(x, k.transpose(1, 2)).mul_(scale).view(b, most, n_h, width)
    seen = (kv_len - (starts[1:] - starts[:-1]))[:, None] + torch.arange(1, most + 1, device="cuda")
    a.masked_fill_((key >= seen[..., None])[:, :, None], -math.inf)
    m = a.amax(-1, keepdim=True).clamp(min=-3e38)
    a.sub_(m).exp_()
    l = a.sum(-1, keepdim=True)
    o = torch.matmul(a.view(b, most * n_h, width), k[..., :d_c]).view(b, most, n_h, d_c) / l
    lse = ((m + torch.log(l)) / math.log(2.0))[..., 0]
    token = torch.arange(q.shape[0], device="cuda")
    seq = torch.searchsorted(starts[1:].contiguous(), token, right=True)
    return {"out": o[seq, token - starts[seq]].to(q.dtype), "lse": lse[seq, token - starts[seq]]}


def run(s):
    op = s["op"]
    if own:
        from head_latent_attention_append_b200 import mla
        if op == "plan":
            mla.plan_step(s["new_len"], s["past_len"], s["free_pages"], s["page_table"], s["num_pages"], s["q_start"],
                          s["kv_len"], s["seq_idx"], s["pos"], s["slot"], s["counts"])
            return {k: s[k] for k in ("page_table", "q_start", "kv_len", "slot", "pos", "seq_idx", "counts")}
        if op == "append":
            mla.append_normed(s["dims"], s["kv"], s["kv_gamma"], s["pos"], s["slot"], s["cache"], EPS, s["cq"],
                              s["cq_gamma"], s["cq_out"])
            return {"cache": s["cache"], "cq": s["cq_out"]}
        if op == "query":
            mla.query_norm_rope(s["dims"], s["q"], s["gamma"], s["pos"], s["qc_out"], s["qr_out"], EPS)
            return {"qc": s["qc_out"], "qr": s["qr_out"]}
        if s["workspace"] is None:  # kept from one step to the next, as a serving loop keeps it
            s["workspace"] = torch.empty(mla.attend_ragged_workspace_bytes(s["dims"], s["case"]["B"], s["q"].shape[0]),
                                         dtype=torch.uint8, device="cuda")
        mla.attend_ragged(s["dims"], s["q"], s["q_start"], s["kv_len"], s["page_table"], s["cache"], s["out"],
                          s["lse"], s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    return {"plan": _plain_plan, "append": _plain_append, "query": _plain_query, "attend": _plain_attend}[op](s)


# ------------------------------------------------ the definition, in 64 bits
def _exact_rows(x, gamma):
    x = x.double()
    return x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS) * gamma.double()


def _exact_turn(x, pos):
    """The same rotation as a product of complex numbers."""
    d = x.shape[-1]
    rate = torch.exp(-math.log(ROPE_BASE) * torch.arange(d // 2, dtype=torch.float64, device="cuda") * 2 / d)
    angle = torch.outer(pos.double(), rate).reshape(x.shape[0], *([1] * (x.dim() - 2)), d // 2)
    z = torch.view_as_complex(x.double().unflatten(-1, (d // 2, 2)).contiguous())
    return torch.view_as_real(z * torch.polar(torch.ones_like(angle), angle)).flatten(-2)


def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    if case["op"] == "append":
        d_c = case["d_c"]
        cache = s["cache"].double()
        flat = cache.view(-1, cache.shape[-1])
        flat[s["slot"], :d_c] = _exact_rows(s["kv"][:, :d_c], s["kv_gamma"])
        flat[s["slot"], d_c:] = _exact_turn(s["kv"][:, d_c:], s["pos"])
        return {"cache": cache, "cq": None if s["cq"] is None else _exact_rows(s["cq"], s["cq_gamma"])}
    if case["op"] == "query":
        return {"qc": _exact_rows(s["q"][..., :case["d_h"]], s["gamma"]),
                "qr": _exact_turn(s["q"][..., case["d_h"]:], s["pos"])}
    new, past = _lengths(case)
    n_h, d_c = case["n_h"], case["d_c"]
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device="cuda")
    token = 0
    for b in range(case["B"]):
        pages = s["page_table"][b, :-(-(new[b] + past[b]) // PAGE)].long()
        keys = s["cache"][pages].flatten(0, 1)[:new[b] + past[b]].double()
        for first in range(0, new[b], 32):  # a few of the request's tokens at a time
            n = min(32, new[b] - first)
            x = s["q"][token + first:token + first + n].double().flatten(0, 1)
            a = x @ keys.t() / math.sqrt(case["d_h"] + case["d_r"])
            sees = past[b] + first + torch.arange(n, device="cuda").repeat_interleave(n_h)
            a = a.masked_fill(torch.arange(keys.shape[0], device="cuda")[None, :] > sees[:, None], -math.inf)
            z = torch.logsumexp(a, -1)
            out[token + first:token + first + n] = (torch.exp(a - z[:, None]) @ keys[:, :d_c]).view(n, n_h, d_c)
            lse[token + first:token + first + n] = (z / math.log(2.0)).view(n, n_h)
        token += new[b]
    return {"out": out, "lse": lse}
