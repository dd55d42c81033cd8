"""Cases of the operators that choose: what is timed, and their plain forms.

A decoder layer of this library makes two kinds of choice, each with the numbers
that the choice goes by:

* ``route``: the experts of a token, from scores (softmax or sigmoid), a bias for
  balance, groups of experts, and the weights of the chosen;
* ``prompt_weigh`` and ``kv_weigh``: the attention weight that every cached token
  has received, summed over queries: of whole prompts, and of a token or a few per
  sequence over the paged 4-bit cache;
* ``kv_evict``: the tokens that a cache of bounded size keeps by these sums, moved
  together in place, in their order.

Sums ("totals") are fp32 ``[n_pages, n_kv_heads, page_size]``, found by the same page
table as the cache's tokens.  A token that a call queries is new: its total begins
at 0 with that call.  The cache's pages are those of ``kv_append``: per key/value head
tiles of 32 tokens, a tile of head width D being ``36 D`` bytes: key codes
``[D/32][32 tokens][16 bytes]``, key scales ``[32 tokens][D/32]`` fp16, then the values'
codes and scales likewise; 32 values of a head are one block, ``(q - 8) d``, with the low
nibbles of its 16 bytes holding values 0..15 and the high ones 16..31.
"""
import random

import torch

own = False

F32, F64 = torch.float32, torch.float64
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one token's router logits, the decode workload's (128 experts, 8 chosen): launch latency counts
        dict(name="route_one", op="route", tokens=1, experts=128, k=8, score="softmax", bias=False, groups=1, kept=1,
             group_score="max", renorm=False, scale=1.0, dtype="f32"),
        # a served batch's decode step, grouped sigmoid routing with a bias
        dict(name="route_batch_64", op="route", tokens=64, experts=256, k=8, score="sigmoid", bias=True, groups=8, kept=4,
             group_score="top2", renorm=True, scale=2.5, dtype="f32"),
        # a prefill batch, the same in bf16
        dict(name="route_prompt", op="route", tokens=16384, experts=256, k=8, score="sigmoid", bias=True, groups=8,
             kept=4, group_score="top2", renorm=True, scale=2.5, dtype="bf16"),
        # a short question's weights: latency counts
        dict(name="weigh_prompt_37", op="prompt", seqs=1, longest=37, shortest=37, prefix=0, hq=16, hkv=8, d=128, page=64,
             window=0, dtype="bf16"),
        # one prefill batch: prompts packed one after another, odd lengths, fp16 and narrow heads
        dict(name="weigh_packed_d64", op="prompt", seqs=12, longest=1500, shortest=3, prefix=0, hq=24, hkv=8, d=64,
             page=128, window=0, dtype="f16"),
        # a long document in one call
        dict(name="weigh_8192", op="prompt", seqs=1, longest=8192, shortest=8192, prefix=0, hq=32, hkv=8, d=128, page=64,
             window=0, dtype="bf16"),
        # one user early in a conversation: a few hundred cached tokens
        dict(name="weigh_short", op="decode", seqs=1, longest=333, shortest=333, q_tokens=1, hq=16, hkv=8, d=128, page=64,
             window=0, dtype="bf16"),
        # one user with a very long context
        dict(name="weigh_long", op="decode", seqs=1, longest=131071, shortest=131071, q_tokens=1, hq=32, hkv=8, d=128,
             page=64, window=0, dtype="bf16"),
        # the largest served batch, ragged contexts
        dict(name="weigh_batch_128", op="decode", seqs=128, longest=8192, shortest=64, q_tokens=1, hq=32, hkv=8, d=128,
             page=64, window=0, dtype="bf16"),
        # one user's cache a little over its budget
        dict(name="evict_one", op="evict", seqs=1, longest=1100, shortest=1100, budget=1024, first=4, recent=128, hkv=8,
             d=128, page=64),
        # a served batch, ragged, most over budget, wide heads and small pages
        dict(name="evict_batch_32", op="evict", seqs=32, longest=12000, shortest=3000, budget=4096, first=4, recent=512,
             hkv=4, d=256, page=32),
        # a very long context halved
        dict(name="evict_long", op="evict", seqs=1, longest=131071, shortest=131071, budget=65536, first=4, recent=1024,
             hkv=8, d=128, page=64),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["route", "prompt", "decode", "evict"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8, 16])
        size = rng.choice([1, 2, 3, 5, 8, 10, 16, 20, 32, 40, 64, 100, 128])
        experts = min(1024 // groups, size * (1 if groups > 1 else rng.choice([1, 2, 4]))) * groups
        kept = rng.randrange(1, groups + 1)
        k = rng.randrange(1, min(32, experts // groups * kept) + 1)
        return dict(op="route", tokens=_log_int(rng, 1, max(1, min(16384, 16384 * 256 // experts))), experts=experts, k=k,
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups, kept=kept,
                    group_score=rng.choice(["max", "top2"]), renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5, 16.0]),
                    dtype=rng.choice(["f32", "f32", "bf16", "f16"]))
    d = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    page = rng.choice([32, 64, 96, 128, 256])
    if op == "evict":
        seqs = _log_int(rng, 1, 64)
        longest = _log_int(rng, 1, max(1, min(131072, 131072 * 8 * 128 // (seqs * hkv * d))))
        budget = max(1, int(longest * rng.choice([0.05, 0.25, 0.5, 0.8, 0.97, 1.1])))
        first = min(budget, rng.choice([0, 0, 1, 4, 64]))
        return dict(op="evict", seqs=seqs, longest=longest,
                    shortest=longest if rng.random() < 0.3 else rng.randrange(0, longest + 1), budget=budget, first=first,
                    recent=rng.choice([0, (budget - first) // 8, (budget - first) // 2, budget - first]), hkv=hkv, d=d,
                    page=page)
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16])
    c = dict(hq=hkv * group, hkv=hkv, d=d, page=page, dtype=rng.choice(["bf16", "bf16", "f16"]))
    if op == "decode":
        seqs = _log_int(rng, 1, 128)
        longest = _log_int(rng, 1, max(1, min(131072, 128 * 4100 * 8 * 128 // (seqs * hkv * d))))
        return dict(c, op="decode", seqs=seqs, longest=longest,
                    shortest=longest if rng.random() < 0.3 else rng.randrange(0, longest + 1),
                    q_tokens=rng.choice([1, 1, 1, 2, 3, 5, 8]) if group <= 8 else 1,
                    window=rng.choice([0, 0, 0, 128, 1000, 4096]))
    seqs = _log_int(rng, 1, 24)
    longest = _log_int(rng, 1, max(1, 8192 // seqs))
    prefix = rng.choice([0, 0, 0, rng.randrange(1, 2000)]) if longest <= 2000 else 0
    # no more work than the largest listed case
    while seqs * longest * (longest + prefix) * c["hq"] * max(d, 128) > 8192 * 8192 * 32 * 128:
        longest //= 2
    return dict(c, op="prompt", seqs=seqs, longest=longest,
                shortest=longest if rng.random() < 0.3 else rng.randrange(0, longest + 1), prefix=prefix,
                window=rng.choice([0, 0, 0, 1, 200, 1024]))


def _lengths(case):
    """Tokens per sequence, by the case alone (its work depends on them): spread evenly from shortest to longest, in a
    shuffled order."""
    n, hi, lo = case["seqs"], case["longest"], case["shortest"]
    lens = [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]
    random.Random(n * 1000003 + hi).shuffle(lens)
    return lens


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _pairs(case):
    """(query, key) pairs that a head of one call looks at."""
    w, total = case["window"], 0
    for n in _lengths(case):
        rows, keys = (case["q_tokens"], n) if case["op"] == "decode" else (n, n + case["prefix"])
        last = [keys - rows + j + 1 for j in range(rows)]
        total += sum(max(0, min(x, w) if w else x) for x in last)
    return total


def work(case):
    if case["op"] == "route":
        t, e, k = case["tokens"], case["experts"], case["k"]
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": t * e * size + t * k * 8 + (e * 4 if case["bias"] else 0), "flops": t * e * 8}
    lens, d, hkv = _lengths(case), case["d"], case["hkv"]
    if case["op"] == "evict":
        over = [n for n in lens if n > case["budget"]]
        moved = len(over) * case["budget"] * hkv
        return {"bytes": 2 * moved * d * 36 // 32 + 4 * hkv * sum(over) + 8 * moved + 8 * case["seqs"],
                "flops": 4 * hkv * sum(over)}
    hq, w = case["hq"], case["window"]
    flops = 2 * hq * d * _pairs(case)
    if case["op"] == "decode":
        j = case["q_tokens"]
        keys = sum(min(n, w + j - 1) if w else n for n in lens)
        return {"bytes": keys * hkv * (d * 18 // 32 + 8) + case["seqs"] * j * hq * (2 * d + 4), "flops": flops}
    t, p = sum(lens), case["prefix"]
    keys = sum(min(n + p, n + w - 1) if w else n + p for n in lens if n)
    return {"bytes": t * hq * (2 * d + 4) + keys * hkv * (2 * d + 8), "flops": flops}


# ------------------------------------------------------------------- the cache's blocks
def _quantise(x):
    """fp32 [..., D] -> codes uint8 [..., D/32, 16], scales fp16 [..., D/32]: the value of largest magnitude is -8 d."""
    x = x.unflatten(-1, (-1, 32))
    hi, lo = x.amax(-1, keepdim=True), x.amin(-1, keepdim=True)
    d = torch.where(hi >= -lo, hi, lo) / -8.0
    q = torch.where(d == 0, torch.full_like(x, 8.0), (x / d + 8.5).clamp(0.0, 15.0)).to(torch.uint8)
    return q[..., :16] | (q[..., 16:] << 4), d.squeeze(-1).to(torch.float16)


def _views(pages, hkv, d):
    """The page planes: codes [page, head, tile, D/32, 32, 16] and scale bytes [page, head, tile, 32, D/32, 2]."""
    t = pages.unflatten(1, (hkv, -1, 36 * d))
    return (t[..., :16 * d].unflatten(-1, (d // 32, 32, 16)), t[..., 16 * d:18 * d].unflatten(-1, (32, d // 32, 2)),
            t[..., 18 * d:34 * d].unflatten(-1, (d // 32, 32, 16)), t[..., 34 * d:].unflatten(-1, (32, d // 32, 2)))


def _values(codes, scales):
    """codes [..., D/32, 16] and scale bytes [..., D/32, 2] -> values [..., D]."""
    q = torch.cat([codes & 15, codes >> 4], -1).to(F32) - 8
    return (q * scales.contiguous().view(torch.float16).to(F32)).flatten(-2)


# ------------------------------------------------------------------- inputs
def _heads(t, h, d, dtype, g, spread=False):
    x = torch.randn(t, h, d, generator=g, device="cuda", dtype=F32)
    if spread:  # keys have a few channels that are much larger than the others
        x[..., ::17] *= 4.0
    return x.to(dtype)


def _table(case, lens, g):
    """A page table and its pool's size: pages in the order that a program which has been serving for a while hands them
    out; unused entries are -1."""
    page = case["page"]
    width = max(1, -(-max(lens) // page))
    used = torch.tensor([-(-n // page) for n in lens], device="cuda")
    n_pages = int(used.sum()) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((case["seqs"], width), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(width, device="cuda")[None, :] < used[:, None]] = order[:n_pages - 3]
    return table, n_pages


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(op=case["op"])
    if case["op"] == "route":
        x = torch.randn(case["tokens"], case["experts"], generator=g, device="cuda", dtype=F32)
        s.update(logits=(x * 1.5).to(DTYPES[case["dtype"]]), k=case["k"], score=case["score"], groups=case["groups"],
                 kept=case["kept"], group_score=case["group_score"], renorm=case["renorm"], scale=case["scale"], bias=None)
        if case["bias"]:
            s["bias"] = torch.randn(case["experts"], generator=g, device="cuda", dtype=F32) * 0.1
        return s

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    d, hkv, page = case["d"], case["hkv"], case["page"]
    lens = _lengths(case)
    keys = [n + case["prefix"] for n in lens] if case["op"] == "prompt" else lens
    table, n_pages = _table(case, keys, g)
    s.update(d=d, hkv=hkv, page=page, table=table)
    if case["op"] == "prompt":
        hq, dt, t = case["hq"], DTYPES[case["dtype"]], sum(lens)
        s.update(hq=hq, window=case["window"], scale=d ** -0.5, n_tokens=t, max_q=max(lens), max_k=max(keys),
                 cu=i32(_cu(lens)), cu_k=i32(_cu(keys)), q=_heads(t, hq, d, dt, g), k=_heads(sum(keys), hkv, d, dt, g, True))
        s["totals"] = torch.rand(n_pages, hkv, page, generator=g, device="cuda", dtype=F32)
        # what the prompt's attention gave beside its result
        scores = _prompt_scores(s)
        lse = torch.logsumexp(scores, -1).unflatten(2, (-1, s["max_q"])).permute(0, 3, 1, 2).flatten(2, 3)
        s["lse"] = lse[_prompt_place(s)].contiguous()
        return s
    # whole pages of keys (and, to be moved, values)
    pages = torch.empty(n_pages, hkv * page * d * 9 // 8, dtype=torch.uint8, device="cuda")
    kc, ks, vc, vs = _views(pages, hkv, d)
    for c, sc, spread in ((kc, ks, True), (vc, vs, False)):
        x = torch.randn(n_pages, hkv, page // 32, 32, d, generator=g, device="cuda", dtype=F32)
        if spread:
            x[..., ::17] *= 4.0
        codes, scale = _quantise(x)
        c.copy_(codes.transpose(-2, -3))
        sc.copy_(scale.view(torch.uint8).unflatten(-1, (-1, 2)))
        del x, codes, scale
    s.update(pages=pages, lens=i32(lens))
    if case["op"] == "evict":
        s.update(budget=case["budget"], first=case["first"], recent=case["recent"])
        # a few tokens have most of the weight; some none at all
        x = torch.randn(n_pages, hkv, page, generator=g, device="cuda", dtype=F32)
        s["totals"] = torch.where(x < -1.5, torch.zeros_like(x), torch.exp(1.7 * x))
        return s
    hq, j = case["hq"], case["q_tokens"]
    s.update(hq=hq, q_tokens=j, window=case["window"], scale=d ** -0.5,
             q=_heads(case["seqs"] * j, hq, d, DTYPES[case["dtype"]], g))
    s["totals"] = torch.rand(n_pages, hkv, page, generator=g, device="cuda", dtype=F32) * (4.0 * j / max(1, max(lens)))
    lse = torch.logsumexp(_decode_scores(s), -1)                                        # [b, hkv, group x j]
    s["lse"] = lse.unflatten(2, (-1, j)).permute(0, 3, 1, 2).reshape(-1, hq).contiguous()
    return s


# ------------------------------------------------------------------- one pass
def run(s):
    return {"route": _run_route, "prompt": _run_prompt, "decode": _run_decode, "evict": _run_evict}[s["op"]](s)


def _run_route(s):
    """The experts of every token, and their weights."""
    if own:
        import router_softmax_top_gb300 as moe
        ids, w = moe.route(s["logits"], s["k"], score=s["score"], bias=s["bias"], n_groups=s["groups"],
                           top_groups=s["kept"], group_score=s["group_score"], renormalise=s["renorm"], scale=s["scale"])
        return {"ids": ids, "weights": w}
    x = s["logits"].to(F64)  # (values next to each other decide)
    p = torch.softmax(x, -1) if s["score"] == "softmax" else 1.0 / (1.0 + torch.exp(-x))
    # without a bias scores are in the order of the logits
    c = p + s["bias"].to(F64) if s["bias"] is not None else x
    if s["groups"] > 1:
        by = (c if s["group_score"] == "max" else p if s["bias"] is None else c).unflatten(-1, (s["groups"], -1))
        most = 1 if s["group_score"] == "max" else min(2, by.shape[-1])
        by = torch.sort(by, dim=-1, descending=True).values[..., :most].sum(-1)
        best = torch.sort(by, dim=-1, descending=True, stable=True).indices[..., :s["kept"]]
        open_ = torch.zeros_like(by, dtype=torch.bool).scatter_(-1, best, True)
        c = c.masked_fill(~open_.repeat_interleave(x.shape[-1] // s["groups"], -1), float("-inf"))
    ids = torch.sort(c, dim=-1, descending=True, stable=True).indices[..., :s["k"]]
    w = p.gather(-1, ids)
    if s["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return {"ids": ids.to(torch.int32), "weights": (w * s["scale"]).to(F32)}


def _seen(at, n_keys, window, width):
    """at [..., rows]: key positions of the rows; n_keys broadcasts against it.  -> [..., rows, width]"""
    key = torch.arange(width, device=at.device)
    at = at[..., None]
    seen = (key <= at) & (key < n_keys[..., None])
    return seen & (key > at - window) if window else seen


def _prompt_place(s):
    """Per token: its sequence and its place in that."""
    cu = s["cu"].long()
    t = torch.arange(s["n_tokens"], device=cu.device)
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return seq, t - cu[seq]


def _prompt_scores(s):
    """[b, hkv, group x max_q, max_k], -inf where a row sees nothing or there is none."""
    hkv, dev = s["hkv"], s["q"].device
    cu, cu_k = s["cu"].long(), s["cu_k"].long()
    n, n_keys = cu.diff(), cu_k.diff()
    i, j = torch.arange(s["max_q"], device=dev), torch.arange(s["max_k"], device=dev)
    q = s["q"][(cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)].to(F32)              # [b, max_q, hq, d]
    k = s["k"][(cu_k[:-1, None] + j).clamp(max=s["k"].shape[0] - 1)].to(F32).transpose(1, 2)
    q = q.unflatten(2, (hkv, -1)).permute(0, 2, 3, 1, 4).flatten(2, 3)                  # [b, hkv, group x max_q, d]
    at = torch.where(i < n[:, None], (n_keys - n)[:, None] + i, -1)                     # [b, max_q]
    at = at.repeat(1, s["hq"] // hkv)[:, None]
    seen = _seen(at, n_keys[:, None, None], s["window"], s["max_k"])
    return ((q @ k.transpose(-1, -2)).mul_(s["scale"])).masked_fill_(~seen, float("-inf"))


def _add(s, got, n, new):
    """Adds got [b, hkv, width] to the totals of the sequences' first n [b] tokens, those from `new` [b] on beginning at 0."""
    i = torch.arange(got.shape[2], device=got.device)
    seq, tok = (i < n[:, None]).nonzero(as_tuple=True)
    page = s["table"][seq, tok // s["page"]].long()
    before = s["totals"][page, :, tok % s["page"]] * (tok < new[seq])[:, None]
    s["totals"][page, :, tok % s["page"]] = before + got[seq, :, tok]
    return s["totals"]


def _run_prompt(s):
    """The weight that every token of the prompts has received from the prompts' queries."""
    if own:
        import router_softmax_top_gb300 as moe
        return moe.prompt_weigh(s["q"], s["k"], s["lse"], s["cu"], s["cu_k"], totals=s["totals"], page_table=s["table"],
                                scale=s["scale"], window=s["window"])
    i = torch.arange(s["max_q"], device=s["q"].device)
    cu, cu_k = s["cu"].long(), s["cu_k"].long()
    lse = s["lse"][(cu[:-1, None] + i).clamp(max=s["lse"].shape[0] - 1)]                # [b, max_q, hq]
    lse = lse.unflatten(2, (s["hkv"], -1)).permute(0, 2, 3, 1).flatten(2, 3)[..., None]
    scores = _prompt_scores(s)
    unseen = scores == float("-inf")
    got = scores.sub_(lse).exp_().masked_fill_(unseen, 0.0).sum(2)                      # [b, hkv, max_k]
    n_keys = cu_k.diff()
    return _add(s, got, n_keys, n_keys - cu.diff())


def _decode_scores(s):
    """[b, hkv, group x j, keys]"""
    b, j, hkv, d = s["table"].shape[0], s["q_tokens"], s["hkv"], s["d"]
    held = s["pages"][s["table"].clamp(min=0).long()].flatten(0, 1)
    kc, ks, _, _ = _views(held, hkv, d)
    k = _values(kc.transpose(-2, -3), ks).unflatten(0, (b, -1)).transpose(1, 2).flatten(2, 4)
    q = s["q"].to(F32).reshape(b, j, hkv, -1, d).permute(0, 2, 3, 1, 4).flatten(2, 3)
    lens = s["lens"].long()
    at = (lens[:, None] - j + torch.arange(j, device=lens.device)).repeat(1, s["hq"] // hkv)[:, None]
    seen = _seen(at, lens[:, None, None], s["window"], k.shape[2])
    return ((q @ k.transpose(-1, -2)) * s["scale"]).masked_fill(~seen, float("-inf"))


def _run_decode(s):
    """The weight that every cached token receives from the sequences' last tokens, added to what it had."""
    if own:
        import router_softmax_top_gb300 as moe
        return moe.kv_weigh(s["q"], s["pages"], s["table"], s["lens"], s["lse"], totals=s["totals"], page_size=s["page"],
                            n_kv_heads=s["hkv"], q_tokens=s["q_tokens"], scale=s["scale"], window=s["window"])
    b, j = s["table"].shape[0], s["q_tokens"]
    lse = s["lse"].reshape(b, j, s["hkv"], -1).permute(0, 2, 3, 1).flatten(2, 3)[..., None]
    scores = _decode_scores(s)
    got = torch.exp(scores - lse).masked_fill(scores == float("-inf"), 0.0).sum(2)
    return _add(s, got, s["lens"].long(), (s["lens"] - j).long())


def _run_evict(s):
    """Keeps what has most weight of every sequence that is over its budget."""
    totals = s["totals"].clone()  # (a pass changes them: the next one has the same to do)
    if own:
        import router_softmax_top_gb300 as moe
        lens, kept = moe.kv_evict(s["pages"], s["table"], s["lens"], s["budget"], totals=totals, page_size=s["page"],
                                  n_kv_heads=s["hkv"], head_dim=s["d"], first=s["first"], recent=s["recent"])
        return {"lens": lens, "kept": kept, "totals": totals, "pages": s["pages"]}
    lens, page, width = s["lens"].long(), s["page"], s["table"].shape[1] * s["page"]
    tok = torch.arange(width, device=lens.device)
    at = s["table"].clamp(min=0).long()
    of = totals[at].transpose(1, 2).flatten(2)                                          # [b, hkv, width]
    n = lens[:, None]
    over = n > s["budget"]
    free = (tok >= s["first"]) & (tok < n - s["recent"]) & over
    rank = torch.sort(of.masked_fill(~free[:, None], float("-inf")), dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(rank).scatter_(-1, rank, tok.expand_as(rank))
    keep = (tok < n) & ~free
    keep = keep[:, None] | (free[:, None] & (rank < s["budget"] - s["first"] - s["recent"]))
    kept = torch.where(keep, tok, width).sort(-1).values[..., :s["budget"]]
    kept = torch.where(kept < width, kept, -1)
    if kept.shape[2] < s["budget"]:
        kept = torch.nn.functional.pad(kept, (0, s["budget"] - kept.shape[2]), value=-1)
    seq, head, to = (over[..., None] & (kept >= 0)).nonzero(as_tuple=True)
    src = kept[seq, head, to]
    src_page, dst_page = at[seq, src // page], at[seq, to // page]
    for c, scale in (_views(s["pages"], s["hkv"], s["d"])[:2], _views(s["pages"], s["hkv"], s["d"])[2:]):
        held, held_scale = (c[src_page, head, src % page // 32, :, src % 32], scale[src_page, head, src % page // 32, src % 32])
        c[dst_page, head, to % page // 32, :, to % 32] = held
        scale[dst_page, head, to % page // 32, to % 32] = held_scale
    held = totals[src_page, head, src % page]
    seq_all, tok_all = ((tok < n) & (tok >= s["budget"])).nonzero(as_tuple=True)
    totals[at[seq_all, tok_all // page], :, tok_all % page] = 0.0
    totals[dst_page, head, to % page] = held
    return {"lens": lens.clamp(max=s["budget"]).to(torch.int32), "kept": kept.to(torch.int32), "totals": totals,
            "pages": s["pages"]}


# ------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "prompt": _exact_prompt, "decode": _exact_decode, "evict": _exact_evict}[case["op"]](case, s)


def _exact_route(case, s):
    x = s["logits"].double()
    top = x.max(1, keepdim=True).values
    score = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.exp(x - top) / torch.exp(x - top).sum(1, keepdim=True)
    value = score + (0.0 if s["bias"] is None else s["bias"].double())
    size = case["experts"] // case["groups"]
    closed = torch.zeros(value.shape, dtype=torch.bool, device="cuda")
    if case["groups"] > 1:
        parts = value.reshape(case["tokens"], case["groups"], size)
        worth = parts.max(2).values
        if case["group_score"] == "top2" and size > 1:
            at = parts.argmax(2, keepdim=True)
            worth = worth + parts.scatter(2, at, -1e300).max(2).values
        open_ = torch.zeros(worth.shape, dtype=torch.bool, device="cuda")
        for _ in range(case["kept"]):
            best = worth.argmax(1, keepdim=True)
            open_.scatter_(1, best, True)
            worth = worth.scatter(1, best, -1e300)
        closed = ~open_.repeat_interleave(size, 1)
    value = value.masked_fill(closed, -1e300)
    # the k largest by value, whichever of equal ones: their scores in descending order of value
    best = value.topk(case["k"], 1).indices
    w = score.gather(1, best)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": None, "weights": w * case["scale"]}


def _exact_prompt(case, s):
    out = s["totals"].double()
    group, page = case["hq"] // case["hkv"], case["page"]
    a = b = 0
    for i, n in enumerate(_lengths(case)):
        m = n + case["prefix"]
        got = torch.zeros(case["hkv"], m, dtype=F64, device="cuda")
        for h in range(case["hq"]):
            k = s["k"][b:b + m, h // group].double()
            for lo in range(0, n, 2048):
                hi = min(n, lo + 2048)
                z = s["q"][a + lo:a + hi, h].double() @ k.t() * s["scale"] - s["lse"][a + lo:a + hi, h, None].double()
                row = torch.arange(m - n + lo, m - n + hi, device="cuda")[:, None]
                col = torch.arange(m, device="cuda")[None]
                hide = col > row
                if case["window"]:
                    hide |= col <= row - case["window"]
                got[h // group] += z.exp().masked_fill(hide, 0.0).sum(0)
        tok = torch.arange(m, device="cuda")
        at = s["table"][i, tok // page].long()
        old = out[at, :, tok % page]
        old[case["prefix"]:] = 0.0
        out[at, :, tok % page] = old + got.t()
        a, b = a + n, b + m
    return out


def _exact_decode(case, s):
    if case["seqs"] * case["longest"] * case["hkv"] * case["d"] > 1 << 30:
        return None
    d, j, page, group = case["d"], case["q_tokens"], case["page"], case["hq"] // case["hkv"]
    raw = s["pages"].view(s["pages"].shape[0], case["hkv"], page // 32, 36 * d)
    out = s["totals"].double()
    for b, n in enumerate(_lengths(case)):
        if n == 0:
            continue
        mine = s["table"][b, :-(-n // page)].long()
        tok = torch.arange(n, device="cuda")
        row = torch.arange(n - j, n, device="cuda")[:, None, None]
        hide = (tok > row) | (row < 0)
        if case["window"]:
            hide |= tok <= row - case["window"]
        for h in range(case["hkv"]):
            x = raw[mine, h].reshape(-1, 36 * d)[:, :18 * d]
            code = x[:, :16 * d].reshape(-1, d // 32, 32, 16).permute(0, 2, 1, 3)
            step = x[:, 16 * d:].reshape(-1, 2).contiguous().view(torch.float16).double().reshape(-1, 32, d // 32, 1)
            w = torch.stack([(code % 16).double(), (code // 16).double()], 3).reshape(code.shape[:3] + (32,))
            k = ((w - 8.0) * step).reshape(-1, d)[:n]
            q = s["q"][b * j:(b + 1) * j, h * group:(h + 1) * group].double()
            z = q @ k.t() * s["scale"] - s["lse"][b * j:(b + 1) * j, h * group:(h + 1) * group, None].double()
            got = z.exp().masked_fill(hide, 0.0).sum((0, 1))
            old = out[mine, h].reshape(-1)
            old[max(0, n - j):n] = 0.0
            old[:n] += got
            out[mine, h] = old.reshape(len(mine), page)
    return out


def _exact_evict(case, s):
    out = s["totals"].double()
    page = case["page"]
    for b, n in enumerate(_lengths(case)):
        if n <= case["budget"]:
            continue
        mine = s["table"][b, :-(-n // page)].long()
        for h in range(case["hkv"]):
            old = out[mine, h].reshape(-1)
            mid = old[case["first"]:n - case["recent"]]
            quota = case["budget"] - case["first"] - case["recent"]
            chosen = torch.sort(torch.sort(-mid, stable=True).indices[:quota]).values
            new = torch.cat([old[:case["first"]], mid[chosen], old[n - case["recent"]:n]])
            old[:n] = 0.0
            old[:case["budget"]] = new
            out[mine, h] = old.reshape(len(mine), page)
    return {"lens": None, "kept": None, "totals": out, "pages": None}
