"""The paged KV cache: writing a batch's new rows into it (per-head norms of queries and keys, the position rotation and the
store in one pass), attention of a chunk of new tokens over it, and the same with a sliding window and a few first tokens
that stay visible; each as a case list with a plain form in elementary torch operations and the calls a user makes of
this package.

The pool of a layer is [pages, kv_heads, page_rows, head_dim], K and V apart; row j of sequence i lies in page
table[i, j // page_rows] at j % page_rows.  New rows are packed by sequence: those of sequence i are starts[i] ..
starts[i + 1] - 1 and take the places lengths[i] - n_i .. lengths[i] - 1.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


def listed():
    drafter = dict(heads=16, kv_heads=16, head_dim=128)    # FlashMap-4B's heads
    mtp = dict(heads=24, kv_heads=4, head_dim=256)         # the MTP head's
    tiny = dict(heads=4, kv_heads=4, head_dim=64)          # the tiny drafter's
    small = dict(heads=32, kv_heads=8, head_dim=64)        # grouped heads of 64
    rope = dict(rot=128, half=False, theta=1e4, scaling="none", factor=1.0)
    part = dict(rot=64, half=True, theta=1e7, scaling="none", factor=1.0)
    far = dict(rot=64, half=True, theta=1e4, scaling="parts", factor=8.0)
    every = dict(window=0, sinks=0)
    return [
        # one token of one sequence enters the cache: the smallest write
        dict(name="write_token", op="write", seqs=1, new_lo=1, new_hi=1, past_lo=4160, past_hi=4160, page=64, lens=1, dtype="bf16",
             rows="bf16", norm=True, **mtp, **part),
        # a batched verify round hands 1..17 rows of each of 32 sequences to the cache
        dict(name="write_round_32seq", op="write", seqs=32, new_lo=1, new_hi=17, past_lo=512, past_hi=8192, page=16, lens=5, dtype="f16",
             rows="f32", norm=True, **drafter, **rope),
        # a 32768-row prompt enters the cache, positions scaled for a long context
        dict(name="write_prompt_32k", op="write", seqs=1, new_lo=32768, new_hi=32768, past_lo=65536, past_hi=65536, page=64, lens=2,
             dtype="bf16", rows="bf16", norm=True, **mtp, **far),
        # the smallest attention: one token of the tiny drafter's heads over 81 rows
        dict(name="attend_token_81", op="attend", seqs=1, new_lo=1, new_hi=1, past_lo=80, past_hi=80, page=16, lens=1, dtype="f16",
             **tiny, **every),
        # one token of each of 32 sequences, grouped heads
        dict(name="attend_token_32seq", op="attend", seqs=32, new_lo=1, new_hi=1, past_lo=0, past_hi=8192, page=64, lens=7, dtype="bf16",
             **mtp, **every),
        # a draft block's 16 rows over one long context, one query head a KV head
        dict(name="attend_block_64k", op="attend", seqs=1, new_lo=16, new_hi=16, past_lo=65521, past_hi=65521, page=128, lens=3,
             dtype="bf16", **drafter, **every),
        # a verify round: 1..17 rows of each of 32 sequences over 512..8192 rows
        dict(name="attend_verify_32seq", op="attend", seqs=32, new_lo=1, new_hi=17, past_lo=512, past_hi=8192, page=16, lens=5,
             dtype="f16", **drafter, **every),
        # the pending rows and drafts of one sequence, grouped heads
        dict(name="attend_rows_8", op="attend", seqs=1, new_lo=8, new_hi=8, past_lo=4153, past_hi=4153, page=32, lens=3, dtype="f16",
             **mtp, **every),
        # a chunk of a long prompt over what is there already
        dict(name="attend_chunk_2k", op="attend", seqs=1, new_lo=2048, new_hi=2048, past_lo=32768, past_hi=32768, page=64, lens=3,
             dtype="bf16", **drafter, **every),
        # ragged prompts that enter an empty cache together
        dict(name="attend_prompts", op="attend", seqs=8, new_lo=33, new_hi=4001, past_lo=0, past_hi=0, page=64, lens=11, dtype="bf16",
             **mtp, **every),
        # one token of each of 32 sequences with a window over long contexts
        dict(name="window_token_32seq", op="attend", seqs=32, new_lo=1, new_hi=1, past_lo=500, past_hi=16384, page=32, lens=9,
             dtype="bf16", **small, window=1024, sinks=4),
        # a long prompt's chunk with a window
        dict(name="window_chunk_8k", op="attend", seqs=1, new_lo=8191, new_hi=8191, past_lo=8200, past_hi=8200, page=128, lens=3,
             dtype="f16", **small, window=1024, sinks=16),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["write", "attend", "attend", "attend"])
    kv_heads, group, head_dim = rng.choice([(16, 1, 128), (8, 1, 128), (4, 1, 64), (4, 6, 256), (2, 4, 64), (8, 4, 64), (8, 4, 128),
                                            (1, 16, 128)])
    case = dict(op=op, heads=kv_heads * group, kv_heads=kv_heads, head_dim=head_dim, page=rng.choice([16, 32, 64, 128]),
                lens=rng.randrange(1000), dtype=rng.choice(["f16", "bf16", "bf16"]))
    seqs = _spread(rng, 1, 64)
    new = _spread(rng, 1, max(1, 4096 // seqs)) if rng.random() < 0.6 else rng.choice([1, 1, 2, 5, 16, 17])
    pairs = 2 ** 33 // (case["heads"] * head_dim)   # (row, key) pairs of a drawn case: below the largest listed one's
    past = _spread(rng, 1, max(1, min(65536 // seqs, pairs * 16 // (seqs * new), 33554432 // (seqs * kv_heads * head_dim) * 16)))
    case.update(seqs=seqs, new_lo=rng.choice([1, new]), new_hi=new, past_lo=rng.choice([0, past // 4, past]), past_hi=past)
    if op == "write":
        rot = rng.choice([r for r in (16, 32, 64, 128, 256) if r <= head_dim])
        scaling = rng.choice(["none", "none", "linear", "parts"])
        case.update(rows=rng.choice(["f32", case["dtype"]]), norm=rng.random() < 0.7, rot=rot, half=rng.random() < 0.5,
                    theta=rng.choice([1e4, 5e5, 1e7]), scaling=scaling, factor=1.0 if scaling == "none" else rng.choice([2.0, 8.0]))
    else:
        window = _spread(rng, 1, 4096) if rng.random() < 0.4 else 0
        case.update(window=window, sinks=rng.choice([0, 1, 4, 16, 130]) if window else 0)
    return case


def _counts(case):
    """New rows of each sequence, and the rows that were there before."""
    r = random.Random(case["lens"])
    return ([r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["seqs"])],
            [r.randint(case["past_lo"], case["past_hi"]) for _ in range(case["seqs"])])


def _rope(case):
    """The rotation's parameters as the framework takes them."""
    gain = 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "parts" else 1.0
    return dict(rot_dims=case["rot"], theta=case["theta"], factor=case["factor"], original_rows=8192, low=1.0, high=32.0, gain=gain)


def _inputs(case, seed):
    """New rows, cut out of one projection's output as they lie there; the pool; the pages of each sequence, in any order."""
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    new, past = _counts(case)
    heads, kv, hd, page, t = case["heads"], case["kv_heads"], case["head_dim"], case["page"], DTYPES[case["dtype"]]
    n, lengths = sum(new), [a + b for a, b in zip(new, past)]
    held = [-(-v // page) for v in lengths]
    pages = sum(held) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((case["seqs"], max(held)), dtype=torch.int32, device="cuda")
    there = torch.arange(max(held), device="cuda")[None] < torch.tensor(held, device="cuda")[:, None]
    table[there] = order[:sum(held)]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    x = {"table": table, "starts": torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32),
         "lengths": torch.tensor(lengths, dtype=torch.int32, device="cuda")}
    if case["op"] == "write":
        rows = normal(n, heads + 2 * kv, hd).to(DTYPES[case["rows"]])
        x.update(q=rows[:, :heads], k=rows[:, heads:heads + kv], v=rows[:, heads + kv:])
        x["q_norm"], x["k_norm"] = (1.0 + 0.1 * normal(hd) for _ in "qk")
        x["k_pool"], x["v_pool"] = (torch.zeros((1, pages, kv, page, hd), dtype=t, device="cuda") for _ in "kv")
    else:   # keys as they leave a per-head norm, a few channels four times the others' size; queries with some peaks
        channel = torch.where(torch.rand((kv, 1, hd), generator=g, device="cuda") < 0.03, 4.0, 1.0)
        x["k_pool"] = (normal(1, pages, kv, page, hd) * channel).to(t)
        x["v_pool"] = (0.5 * normal(1, pages, kv, page, hd)).to(t)
        x["q"] = (1.5 * normal(n, heads, hd) / channel[:, 0].repeat_interleave(heads // kv, 0)).to(t)
    return x


def prepare(case, seed):
    x = _inputs(case, seed)
    new, past = _counts(case)
    state = dict(case=case, x=x, new=new, out=torch.empty(x["q"].shape, dtype=DTYPES[case["dtype"]], device="cuda"))
    state["longest"] = max(a + b for a, b in zip(new, past))
    state["at"] = torch.cat([torch.arange(a, device="cuda") + b for a, b in zip(new, past)])      # each row's position
    state["seq"] = torch.repeat_interleave(torch.arange(case["seqs"], device="cuda"), torch.tensor(new, device="cuda"))
    if own:
        import block_speculative_decoding_fm_gb300 as fm
        rope = dict(rot_dims=0)
        if case["op"] == "write":
            kind = {"none": fm.FM_ROPE_PLAIN, "linear": fm.FM_ROPE_LINEAR, "parts": fm.FM_ROPE_BY_PARTS}[case["scaling"]]
            rope = dict(_rope(case), scaling=kind, layout=fm.FM_ROPE_HALF if case["half"] else fm.FM_ROPE_INTERLEAVED)
        state["cache"] = fm.fm_paged_create(x["k_pool"], x["v_pool"], case["heads"], eps=EPS, **rope)
        state["batch"] = fm.fm_paged_batch(state["cache"], x["starts"], x["lengths"], x["table"], sum(new), max(new))
    return state


def run(state):
    case, x = state["case"], state["x"]
    if own:
        import block_speculative_decoding_fm_gb300 as fm
        if case["op"] == "write":
            norms = (x["q_norm"], x["k_norm"]) if case["norm"] else (None, None)
            fm.fm_paged_write(state["cache"], 0, state["batch"], x["q"], x["k"], x["v"], state["out"], *norms)
            return {"q": state["out"], "k_pool": x["k_pool"], "v_pool": x["v_pool"]}
        fm.fm_paged_attend(state["cache"], 0, state["batch"], x["q"], state["out"], window=case["window"], sinks=case["sinks"])
        return {"out": state["out"]}
    return _plain_write(state) if case["op"] == "write" else _plain_attend(state)


def _frequencies(case):
    """The angle a position of each pair, in 64 bits."""
    r = _rope(case)
    f = r["theta"] ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64) / case["rot"])
    if case["scaling"] == "linear":
        return f / r["factor"]
    if case["scaling"] == "parts":   # pairs that turn often keep their angle, slow ones are stretched
        keep = ((r["original_rows"] * f / (2 * math.pi) - r["low"]) / (r["high"] - r["low"])).clamp(0.0, 1.0)
        return f * (keep + (1.0 - keep) / r["factor"])
    return f


def _plain_rows(case, rows, weight, at):
    y = rows.float()
    if case["norm"]:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * weight
    angle, gain = at.double()[:, None, None] * _frequencies(case), _rope(case)["gain"]
    cos, sin = gain * torch.cos(angle).float(), gain * torch.sin(angle).float()
    turned, rest = y[..., :case["rot"]], y[..., case["rot"]:]
    a, b = turned.chunk(2, -1) if case["half"] else (turned[..., 0::2], turned[..., 1::2])
    pair = (a * cos - b * sin, a * sin + b * cos)
    turned = torch.cat(pair, -1) if case["half"] else torch.stack(pair, -1).flatten(-2)
    return torch.cat((turned, rest), -1).to(DTYPES[case["dtype"]])


def _plain_write(state):
    case, x, at, page = state["case"], state["x"], state["at"], state["case"]["page"]
    where = x["table"][state["seq"], at // page].long()
    x["k_pool"][0][where, :, at % page] = _plain_rows(case, x["k"], x["k_norm"], at)
    x["v_pool"][0][where, :, at % page] = x["v"].to(DTYPES[case["dtype"]])
    return {"q": _plain_rows(case, x["q"], x["q_norm"], at), "k_pool": x["k_pool"], "v_pool": x["v_pool"]}


def _plain_attend(state):
    case, x, at, seq = state["case"], state["x"], state["at"], state["seq"]
    n, most, kv, hd, group = case["seqs"], max(state["new"]), case["kv_heads"], case["head_dim"], case["heads"] // case["kv_heads"]
    k, v = (x[s][0][x["table"].long()].transpose(2, 3).flatten(1, 2)[:, :state["longest"]].transpose(1, 2).float()
            for s in ("k_pool", "v_pool"))                                              # [seqs, kv_heads, L, hd]
    row = torch.arange(at.shape[0], device="cuda") - x["starts"][seq]
    q = torch.zeros((n, most, case["heads"], hd), device="cuda")
    q[seq, row] = x["q"].float()
    last = torch.full((n, most), -1, device="cuda")                                       # a row's position; padding sees nothing
    last[seq, row] = at
    key = torch.arange(k.shape[2], device="cuda")
    seen = key <= last[..., None]
    if case["window"]:
        seen = seen & ((key > last[..., None] - case["window"]) | (key < case["sinks"]))
    q = q.view(n, most, kv, group, hd).permute(0, 2, 3, 1, 4)                             # [seqs, kv_heads, group, rows, hd]
    s = (q @ k[:, :, None].transpose(-1, -2)) / math.sqrt(hd)
    s = torch.where(seen[:, None, None], s, -torch.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(-1, keepdim=True)
    out = (p @ v[:, :, None]) / torch.where(total == 0, 1.0, total)
    return {"out": out.permute(0, 3, 1, 2, 4).reshape(n, most, case["heads"], hd)[seq, row].to(x["q"].dtype)}


def _seen(case, position):
    """Rows that the row at a position sees."""
    if not case["window"]:
        return position + 1
    first = max(0, position + 1 - case["window"])
    return position + 1 - first + min(case["sinks"], first)


def work(case):
    new, past = _counts(case)
    kv, hd, size, n = case["kv_heads"], case["head_dim"], DTYPES[case["dtype"]].itemsize, sum(new)
    if case["op"] == "write":   # rows in; queries and the pages' rows out
        values = n * (case["heads"] + 2 * kv) * hd
        return {"bytes": values * (DTYPES[case["rows"]].itemsize + size), "flops": 8 * values}
    pairs = sum(_seen(case, p) for a, b in zip(new, past) for p in range(b, b + a))
    rows = sum(a - 1 + _seen(case, b) if not case["window"] else
               min(a + b, a - 1 + case["window"] + min(case["sinks"], max(0, b + 1 - case["window"]))) for a, b in zip(new, past))
    return {"bytes": 2 * rows * kv * hd * size + 2 * n * case["heads"] * hd * size, "flops": 4 * pairs * case["heads"] * hd}


def _exact_turn(case, rows, weight, at):
    y = rows.double().clone()
    if case["norm"]:
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + EPS) * weight.double()
    r, half = _rope(case), case["rot"] // 2
    out = y.clone()
    for i in range(half):   # pair by pair
        f = math.exp(-2.0 * i / case["rot"] * math.log(r["theta"]))
        if case["scaling"] == "linear":
            f /= r["factor"]
        if case["scaling"] == "parts":
            turns = r["original_rows"] * f / (2 * math.pi)
            share = min(1.0, max(0.0, (turns - r["low"]) / (r["high"] - r["low"])))
            f = share * f + (1.0 - share) * f / r["factor"]
        one, two = (i, i + half) if case["half"] else (2 * i, 2 * i + 1)
        z = torch.polar(torch.full(at.shape, r["gain"], dtype=torch.float64, device="cuda"), at.double() * f)[:, None]
        z = z * torch.complex(y[..., one], y[..., two])
        out[..., one], out[..., two] = z.real, z.imag
    return out


def exact(case, seed):
    x = _inputs(case, seed)
    new, past = _counts(case)
    page, group, hd, first = case["page"], case["heads"] // case["kv_heads"], case["head_dim"], 0
    if case["op"] == "write":
        at = torch.cat([torch.arange(b, b + a, device="cuda") for a, b in zip(new, past)])
        q, k = _exact_turn(case, x["q"], x["q_norm"], at), _exact_turn(case, x["k"], x["k_norm"], at)
        pools = {s: x[s].double() for s in ("k_pool", "v_pool")}
        for i, (a, b) in enumerate(zip(new, past)):
            j = torch.arange(b, b + a, device="cuda")
            to = x["table"][i].long()[torch.div(j, page, rounding_mode="floor")]
            pools["k_pool"][0, to, :, j % page] = k[first:first + a]
            pools["v_pool"][0, to, :, j % page] = x["v"][first:first + a].double()
            first += a
        return {"q": q, **pools}
    out = torch.zeros(x["q"].shape, dtype=torch.float64, device="cuda")
    for i, (a, b) in enumerate(zip(new, past)):
        n = a + b
        k, v = (x[s][0][x["table"][i, :-(-n // page)].long()].double().permute(1, 0, 2, 3).reshape(case["kv_heads"], -1, hd)[:, :n]
                for s in ("k_pool", "v_pool"))
        step = max(1, 2 ** 26 // n)   # rows a turn
        for r in range(0, a, step):
            rows = torch.arange(r, min(a, r + step), device="cuda")
            j, p = torch.arange(n, device="cuda")[None], (b + rows)[:, None]
            hidden = j > p
            if case["window"]:
                hidden |= (j <= p - case["window"]) & (j >= case["sinks"])
            for h in range(case["heads"]):
                s = x["q"][first + rows, h].double() @ k[h // group].T * hd ** -0.5
                out[first + rows, h] = torch.softmax(s.masked_fill(hidden, -math.inf), -1) @ v[h // group]
        first += a
    return {"out": out}
