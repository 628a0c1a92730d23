"""The KV cache held in 4 bits: appending rows to it, attention over it, eviction from it by accumulated attention
weight, and reading rows back, each as a case list with a plain form in elementary torch operations and the
calls a user makes of this package.

Format of the cache: a row of a KV head is cut into groups of 32 values; a group holds an f16 scale d and codes
c in 0..15 and stands for d (c - 8).  d = f16(m / -8), m the group's value of largest magnitude (the negative one
where +m and -m tie); c = clamp(rint(x / d) + 8, 0, 15), 8 where d = 0.
"""
import math
import random

import torch

own = False

GROUP = 32
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    flashmap = dict(heads=16, kv_heads=16, head_dim=128)   # FlashMap-4B cross-attention
    mtp = dict(heads=24, kv_heads=4, head_dim=256)         # the MTP head: grouped heads
    tiny = dict(heads=4, kv_heads=4, head_dim=64)          # the tiny drafter
    return [
        # a batched verify round hands 1..17 context rows of each of 32 sequences to the cache
        dict(name="append_round_32seq", op="append", seqs=32, lo=1, hi=17, start=1003, lens=5, dtype="bf16", **flashmap),
        # a 32768-row prompt enters the cache
        dict(name="append_prompt_32k", op="append", seqs=1, lo=32768, hi=32768, start=0, lens=0, dtype="f16", **flashmap),
        # the smallest call: the tiny drafter's 16 slots over an 81-row context
        dict(name="attend_tiny", op="attend", seqs=1, lo=81, hi=81, rows=16, causal=False, weights=False, lens=0,
             dtype="f32", **tiny),
        # the drafter's cross-attention in the default workload: 16 slots over 1042 rows
        dict(name="attend_draft_1k", op="attend", seqs=1, lo=1042, hi=1042, rows=16, causal=False, weights=False,
             lens=0, dtype="f32", **flashmap),
        # the same over a long context
        dict(name="attend_draft_32k", op="attend", seqs=1, lo=32769, hi=32769, rows=16, causal=False, weights=False,
             lens=0, dtype="bf16", **flashmap),
        # 32 sequences draft together over contexts of 512..8192 rows
        dict(name="attend_draft_32seq", op="attend", seqs=32, lo=512, hi=8192, rows=16, causal=False, weights=False,
             lens=5, dtype="f16", **flashmap),
        # one token of each of 32 sequences, grouped heads
        dict(name="attend_token_32seq", op="attend", seqs=32, lo=1, hi=4160, rows=1, causal=True, weights=False,
             lens=7, dtype="bf16", **mtp),
        # the MTP head takes its 8 pending rows over 4161 positions
        dict(name="attend_mtp_rows", op="attend", seqs=1, lo=4161, hi=4161, rows=8, causal=True, weights=False, lens=0,
             dtype="f32", **mtp),
        # decoding that keeps each row's attention weight for a later eviction
        dict(name="attend_weights_16seq", op="attend", seqs=16, lo=1000, hi=8192, rows=1, causal=True, weights=True,
             lens=9, dtype="bf16", **mtp),
        # a draft over a long context that keeps the weights
        dict(name="attend_weights_32k", op="attend", seqs=1, lo=32769, hi=32769, rows=16, causal=False, weights=True,
             lens=0, dtype="bf16", **flashmap),
        # 32 sequences brought down to 2048 rows a head
        dict(name="evict_32seq", op="evict", seqs=32, lo=512, hi=8192, keep=2048, recent=256, ties=False, lens=5,
             dtype="bf16", **flashmap),
        # a long context of the MTP head halved twice
        dict(name="evict_64k", op="evict", seqs=1, lo=65535, hi=65535, keep=16384, recent=1001, ties=True, lens=0,
             dtype="bf16", **mtp),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "evict"])
    kv_heads, group, head_dim = rng.choice([(16, 1, 128), (8, 1, 128), (4, 1, 64), (4, 6, 256), (2, 4, 64), (8, 4, 128)])
    seqs = _spread(rng, 1, 32)
    wide = kv_heads * head_dim
    hi = _spread(rng, 16, max(16, min(65536, (32 * 4096 * 1024) // (seqs * wide))))
    case = dict(op=op, seqs=seqs, lo=rng.choice([1, max(1, hi // 8), hi]), hi=hi, lens=rng.randrange(1000),
                heads=kv_heads * group, kv_heads=kv_heads, head_dim=head_dim, dtype=rng.choice(["f32", "f16", "bf16", "bf16"]))
    if op == "append":
        case.update(hi=min(hi, 32768), lo=min(case["lo"], 32768), start=rng.choice([0, rng.randrange(1, 4000)]))
    elif op == "attend":
        case.update(rows=rng.choice([1, 1, 2, 5, 8, 16, 17]), causal=rng.random() < 0.6, weights=rng.random() < 0.4)
    else:
        keep = _spread(rng, 1, hi)
        case.update(keep=keep, recent=rng.randrange(0, keep + 1), ties=rng.random() < 0.5)
    return case


def _lengths(case):
    """Rows of each sequence: the cache's length, or for append the rows that arrive."""
    r = random.Random(case["lens"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]


def _inputs(case, seed):
    """Rows packed by sequence: k, v [N, kv_heads, head_dim]; q [seqs * rows, heads, head_dim]; weights
    [seqs, kv_heads, longest].  Keys as they leave a per-head norm, a few channels four times the others' size;
    queries wide enough that the attention has peaks."""
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    n, hd, t = sum(_lengths(case)), case["head_dim"], DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    channel = torch.where(torch.rand((case["kv_heads"], hd), generator=g, device="cuda") < 0.03, 4.0, 1.0)
    x = {"k": (normal(n, case["kv_heads"], hd) * channel).to(t), "v": (0.5 * normal(n, case["kv_heads"], hd)).to(t)}
    if case["op"] == "attend":
        x["q"] = (2.0 * normal(case["seqs"] * case["rows"], case["heads"], hd) / channel.repeat_interleave(
            case["heads"] // case["kv_heads"], 0)).to(t)
    if case["op"] == "evict":
        w = torch.exp(2.0 * normal(case["seqs"], case["kv_heads"], max(_lengths(case))))
        x["weights"] = torch.floor(8.0 * w) / 8.0 if case["ties"] else w
    return x


def _quantize(x):
    """Codes (uint8) and f16 scales of groups along the last axis; in 64 bits, where the border between two codes matters."""
    g = x.double().unflatten(-1, (-1, GROUP))
    hi, lo = g.amax(-1), g.amin(-1)
    m = torch.where(hi > -lo, hi, lo)
    d = (m / -8.0).clamp(-65504.0, 65504.0).half()
    dd = d.double().unsqueeze(-1)
    c = torch.where(dd == 0, 8.0, torch.round(g / torch.where(dd == 0, 1.0, dd)) + 8.0).clamp(0.0, 15.0)
    return c.to(torch.uint8).flatten(-2), d


def _values(codes, scales):
    """The f32 values that codes and scales stand for."""
    return ((codes.float() - 8.0).unflatten(-1, (-1, GROUP)) * scales.float().unsqueeze(-1)).flatten(-2)


def _pack(codes):
    """Two codes a byte."""
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _unpack(packed):
    return torch.stack((packed & 15, packed >> 4), -1).flatten(-2)


def _padded(x, lengths):
    """Rows packed by sequence -> [seqs, longest, ...], zeros behind each sequence's end."""
    out = x.new_zeros((len(lengths), max(lengths)) + x.shape[1:])
    out[_inside(lengths, max(lengths))] = x
    return out


def _inside(lengths, longest):
    return torch.arange(longest, device="cuda")[None, :] < torch.tensor(lengths, device="cuda")[:, None]


def prepare(case, seed):
    lengths, x, t = _lengths(case), _inputs(case, seed), DTYPES[case["dtype"]]
    hkv, hd, n = case["kv_heads"], case["head_dim"], case["seqs"]
    state = dict(case=case, lengths=lengths, inputs=x, ids=list(range(n)))
    longest = max(lengths)
    if case["op"] == "append":
        state["k_out"], state["v_out"] = torch.empty_like(x["k"]), torch.empty_like(x["v"])
        state["starts"] = [case["start"]] * n
    if case["op"] == "attend":
        state["out"] = torch.empty_like(x["q"])
        state["weights"] = torch.zeros((n, hkv, longest), device="cuda") if case["weights"] else None
        state["rows"] = [case["rows"]] * n
        state["inside"] = _inside(lengths, longest)
    if case["op"] == "evict":
        state["kept"] = torch.full((n, hkv, case["keep"]), -1, dtype=torch.int32, device="cuda")
        state["left"] = [min(case["keep"], v) for v in lengths]
        total = sum(state["left"])
        state["k_out"], state["v_out"] = (torch.empty((total, hkv, hd), dtype=t, device="cuda") for _ in "kv")
        state["weights"] = torch.zeros((n, hkv, max(state["left"])), device="cuda")
        state["inside"] = _inside(lengths, longest)
        state["inside_left"] = _inside(state["left"], max(state["left"]))
    if own:
        import block_speculative_decoding_fm_gb300 as fm
        rows = case["start"] + longest if case["op"] == "append" else longest
        slots = 2 * n if case["op"] == "evict" else n
        cache = state["cache"] = fm.fm_kvq_create(1, slots, hkv, hd, rows)
        if case["op"] == "append":
            if case["start"]:   # the rows that are there already
                old = torch.zeros((n * case["start"], hkv, hd), dtype=t, device="cuda")
                fm.fm_kvq_append(cache, 0, state["ids"], old, old, [case["start"]] * n, [0] * n)
        else:
            fm.fm_kvq_append(cache, 0, state["ids"], x["k"], x["v"], lengths, [0] * n)
        if case["op"] == "evict":
            fm.fm_kvq_set_weights(cache, 0, state["ids"], x["weights"])
            state["to"] = list(range(n, 2 * n))   # the slots that the kept rows go to
    elif case["op"] != "append":
        (kc, state["kd"]), (vc, state["vd"]) = (_quantize(_padded(x[s], lengths)) for s in "kv")
        state["kc"], state["vc"] = _pack(kc), _pack(vc)
    return state


def run(state):
    case, x = state["case"], state["inputs"]
    if own:
        import block_speculative_decoding_fm_gb300 as fm
        cache, ids, lengths = state["cache"], state["ids"], state["lengths"]
        if case["op"] == "append":
            fm.fm_kvq_append(cache, 0, ids, x["k"], x["v"], lengths, state["starts"])
            fm.fm_kvq_read(cache, 0, ids, state["starts"], lengths, state["k_out"], state["v_out"])
            return {"k": state["k_out"], "v": state["v_out"]}
        if case["op"] == "attend":
            if not case["weights"]:
                fm.fm_kvq_attend(cache, 0, ids, x["q"], state["rows"], state["out"], causal=case["causal"])
                return {"out": state["out"]}
            fm.fm_kvq_attend(cache, 0, ids, x["q"], state["rows"], state["out"], causal=case["causal"], decay=0.0,
                             weights=state["weights"])
            return {"out": state["out"], "weights": state["weights"]}
        fm.fm_kvq_evict(cache, 0, ids, state["to"], case["keep"], case["recent"], state["kept"])
        fm.fm_kvq_read(cache, 0, state["to"], [0] * len(ids), state["left"], state["k_out"], state["v_out"],
                       state["weights"])
        return {"kept": state["kept"], "k": state["k_out"], "v": state["v_out"], "weights": state["weights"]}
    if case["op"] == "append":
        return _plain_append(state)
    return _plain_attend(state) if case["op"] == "attend" else _plain_evict(state)


def _plain_append(state):
    x = state["inputs"]
    return {s: _values(*_quantize(x[s])).to(x[s].dtype) for s in "kv"}


def _plain_attend(state):
    case, q, inside = state["case"], state["inputs"]["q"], state["inside"]
    n, rows, hkv, hd, group = case["seqs"], case["rows"], case["kv_heads"], case["head_dim"], case["heads"] // case["kv_heads"]
    k, v = (_values(_unpack(state[s + "c"]), state[s + "d"]).transpose(1, 2) for s in "kv")   # [seqs, kv_heads, L, hd]
    qf = q.float().view(n, rows, hkv, group, hd).permute(0, 2, 1, 3, 4).reshape(n, hkv, rows * group, hd)
    s = (qf @ k.transpose(-1, -2)) / math.sqrt(hd)
    seen = inside[:, None, :].expand(n, rows, -1)
    if case["causal"]:   # row t of the last `rows` rows sees the cache up to its own
        end = inside.sum(-1)[:, None] - rows + 1 + torch.arange(rows, device="cuda")[None, :]
        seen = seen & (torch.arange(k.shape[2], device="cuda") < end[..., None])
    seen = seen.repeat_interleave(group, 1)[:, None]
    s = torch.where(seen, s, -torch.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(s - torch.where(torch.isinf(top), 0.0, top)), 0.0)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    out = (p @ v).view(n, hkv, rows, group, hd).permute(0, 2, 1, 3, 4).reshape(q.shape).to(q.dtype)
    return {"out": out, "weights": p.sum(2)} if case["weights"] else {"out": out}


def _plain_evict(state):
    case, inside, w = state["case"], state["inside"], state["inputs"]["weights"]
    longest, keep, recent = inside.shape[1], case["keep"], case["recent"]
    row, length = torch.arange(longest, device="cuda"), inside.sum(-1)[:, None, None]
    recently = inside[:, None] & (row >= length - recent)
    rank = torch.where(recently, torch.inf, torch.where(inside[:, None], w, -torch.inf))
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :keep]   # ties: the lowest row first
    left = torch.clamp(length, max=keep)
    there = torch.arange(order.shape[-1], device="cuda") < left
    rows = torch.sort(torch.where(there, order, longest), dim=-1).values
    kept = torch.full_like(state["kept"], -1)
    kept[..., : order.shape[-1]] = torch.where(there, rows, -1)
    most = state["inside_left"].shape[1]
    at = torch.where(there, rows, 0)[..., :most]   # [seqs, kv_heads, rows]
    weights = torch.where(there[..., :most], torch.gather(w, 2, at), 0.0)
    at = at.transpose(1, 2)[..., None]
    res = {"kept": kept, "weights": weights}
    for s in "kv":
        codes = torch.gather(state[s + "c"], 1, at.expand(-1, -1, -1, state[s + "c"].shape[-1]))
        scales = torch.gather(state[s + "d"], 1, at.expand(-1, -1, -1, state[s + "d"].shape[-1]))
        res[s] = _values(_unpack(codes), scales)[state["inside_left"]].to(state["k_out"].dtype)
    return res


def work(case):
    lengths, hkv, hd, size = _lengths(case), case["kv_heads"], case["head_dim"], DTYPES[case["dtype"]].itemsize
    values = 2 * hkv * hd                      # of a row, keys and values
    held = values // 2 + 2 * values // GROUP   # its bytes in the cache
    if case["op"] == "append":   # rows in, the cache's rows written, the values they stand for out
        n = sum(lengths)
        return {"bytes": n * (2 * values * size + held), "flops": 10 * n * values}
    if case["op"] == "attend":
        q = case["seqs"] * case["rows"] * case["heads"] * hd
        rows = sum(lengths)
        return {"bytes": rows * (held + (4 * hkv if case["weights"] else 0)) + 2 * q * size,
                "flops": 4 * rows * case["rows"] * case["heads"] * hd}
    left = sum(min(case["keep"], v) for v in lengths)
    # weights in; kept rows in, out to their slot, and out as values; their weights moved and out; their places out
    return {"bytes": 4 * hkv * sum(lengths) + left * (2 * held + values * size + 12 * hkv), "flops": 2 * left * values}


def _exact_cache(x):
    """The values in 64 bits, group by group from the definition."""
    f = x.double().reshape(-1, GROUP)
    big = f.abs().max(1).values
    m = torch.where((f == -big[:, None]).any(1), -big, big)
    d = torch.clip(-m / 8, -65504, 65504).to(torch.float16).to(torch.float64)
    out = torch.zeros_like(f)
    some = d != 0
    steps = torch.clip(torch.round(f[some] / d[some, None]), -8, 7)
    out[some] = steps * d[some, None]
    return out.reshape(x.shape)


def exact(case, seed):
    x, lengths = _inputs(case, seed), _lengths(case)
    k, v = _exact_cache(x["k"]), _exact_cache(x["v"])
    if case["op"] == "append":
        return {"k": k, "v": v}
    first = [sum(lengths[:i]) for i in range(len(lengths))]
    hkv, hd = case["kv_heads"], case["head_dim"]
    if case["op"] == "attend":
        rows, group = case["rows"], case["heads"] // case["kv_heads"]
        q = x["q"].double()
        out = torch.zeros_like(q)
        weights = torch.zeros((case["seqs"], hkv, max(lengths)), dtype=torch.float64, device="cuda")
        for i, (at, n) in enumerate(zip(first, lengths)):
            for t in range(rows):
                end = n - rows + t + 1 if case["causal"] else n
                if end <= 0:
                    continue
                qt = q[i * rows + t].reshape(hkv, group, hd)
                s = torch.einsum("hgd,lhd->hgl", qt, k[at:at + end]) * hd ** -0.5
                p = torch.softmax(s, -1)
                out[i * rows + t] = torch.einsum("hgl,lhd->hgd", p, v[at:at + end]).reshape(-1, hd)
                weights[i, :, :end] += p.sum(1)
        return {"out": out, "weights": weights} if case["weights"] else {"out": out}
    keep, recent = case["keep"], case["recent"]
    most = max(min(keep, n) for n in lengths)
    weights = torch.zeros((case["seqs"], hkv, most), dtype=torch.float64, device="cuda")
    ks, vs = [], []
    for i, (at, n) in enumerate(zip(first, lengths)):
        left = min(keep, n)
        w = x["weights"][i, :, :n].double()
        old = max(0, n - recent)
        chosen = torch.ones((hkv, n), dtype=torch.bool, device="cuda")
        if n > keep:   # a row's place among the older ones: by weight, then by row
            place = torch.argsort(torch.argsort(-w[:, :old], dim=-1, stable=True), dim=-1)
            chosen[:, :old] = place < keep - recent
        weights[i, :, :left] = w[chosen].reshape(hkv, left)
        for src, dst in ((k, ks), (v, vs)):
            dst.append(src[at:at + n].transpose(0, 1)[chosen].reshape(hkv, left, hd).transpose(0, 1))
    return {"kept": None, "weights": weights, "k": torch.cat(ks), "v": torch.cat(vs)}
