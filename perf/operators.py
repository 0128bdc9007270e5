"""Serving and training cases of the packed and 4-bit-cache attention operators.

Four groups of calls, in the order in which a program that serves or trains a
decoder makes them:

* ``prompt``  causal attention over a packed batch of whole prompts of different
  lengths, grouped heads;
* ``train``   the same with its backward pass (o, lse, dq, dk, dv);
* ``store``   quantise new keys and values into a paged cache of 4-bit codes and
  read the stored values back;
* ``step``    one query token per sequence attends to its 4-bit cache, with or
  without adding each key's attention weight to a running sum;
* ``evict``   keep the keys with the largest accumulated weight and the latest
  ones, moved in order to fresh pages, and read the kept values back.

A cached key (or value) vector of D elements is held as D/32 groups of 32 codes of
4 bits with a bf16 minimum and a bf16 scale per group:

    mn = min(x),  scale = bf16((max(x) - mn) / 15),
    code = clamp(round((x - mn) / scale), 0, 15)  (0 where scale is 0),
    value = mn + scale * code

``own`` selects the framework's operators; otherwise the plain forms below run.
"""
import math
import random

import torch

own = False

GROUP = 32  # elements that share a minimum and a scale


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a handful of short chat turns prefilled together: launch latency counts
        dict(name="prompt_short", op="prompt", Hq=4, Hkv=2, D=64, tokens=437, max_len=200,
             shape_seed=3),
        # a full prefill batch of a grouped-head model: 16384 tokens of mixed prompts
        dict(name="prompt_16k", op="prompt", Hq=32, Hkv=8, D=128, tokens=16384, max_len=8192,
             shape_seed=11),
        # one training step's attention over packed documents, one head per kv head
        dict(name="train_16k", op="train", Hq=16, Hkv=16, D=128, tokens=16384, max_len=8192,
             deterministic=False, shape_seed=23),
        # a small packed step with head dimension 64 and bit-reproducible gradients
        dict(name="train_d64_det", op="train", Hq=16, Hkv=4, D=64, tokens=4099, max_len=1500,
             deterministic=True, shape_seed=5),
        # a decoding step's store: one new token in each of 64 running sequences
        dict(name="store_step", op="store", B=64, Hkv=8, D=128, page=64, lo=1, hi=1, past=2048,
             shape_seed=7),
        # the store after a prefill: a batch of whole prompts
        dict(name="store_prompt", op="store", B=9, Hkv=8, D=128, page=64, lo=1024, hi=4096, past=0,
             shape_seed=13),
        # one short conversation: a single step's latency
        dict(name="step_one", op="step", B=1, Hq=32, Hkv=8, D=128, page=16, lo=300, hi=300,
             weights=False, shape_seed=1),
        # a busy server: 64 sequences of mixed lengths, weights kept for eviction
        dict(name="step_b64", op="step", B=64, Hq=32, Hkv=8, D=128, page=64, lo=512, hi=8192,
             weights=True, shape_seed=17),
        # few long contexts, head dimension 64, one query head per kv head
        dict(name="step_long_d64", op="step", B=2, Hq=16, Hkv=16, D=64, page=128, lo=30001,
             hi=32768, weights=False, shape_seed=19),
        # long contexts cut to half: the usual eviction after long prompts
        dict(name="evict_half", op="evict", B=16, Hkv=8, D=128, page=64, lo=6000, hi=8192,
             budget=4096, recent=512, shape_seed=29),
        # two short conversations kept within a small budget
        dict(name="evict_small", op="evict", B=2, Hkv=4, D=64, page=16, lo=257, hi=700,
             budget=250, recent=33, shape_seed=31),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "train", "store", "step", "evict"])
    D = rng.choice([64, 128])
    seed = rng.randrange(1 << 30)
    if op in ("prompt", "train"):
        Hq, Hkv = rng.choice([(2, 2), (4, 2), (8, 1), (16, 4), (16, 16), (32, 8)])
        if op == "train" and Hq == 32:
            Hq, Hkv = 14, 2
        tokens = _log_int(rng, 60, 16384)
        case = dict(op=op, Hq=Hq, Hkv=Hkv, D=D, tokens=tokens,
                    max_len=_log_int(rng, 20, min(tokens, 4096)), shape_seed=seed)
        if op == "train":
            case["deterministic"] = rng.random() < 0.5
        return case
    page = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    if op == "store":
        hi = rng.choice([1, _log_int(rng, 2, 2048)])
        return dict(op=op, B=_log_int(rng, 1, 64 if hi < 256 else 8), Hkv=Hkv, D=D, page=page,
                    lo=1, hi=hi, past=rng.choice([0, _log_int(rng, 1, 4096)]), shape_seed=seed)
    if op == "step":
        B = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, 131072 // max(B, 4))
        return dict(op=op, B=B, Hq=Hkv * rng.choice([1, 2, 4, 5, 8, 12]), Hkv=Hkv, D=D,
                    page=page, lo=_log_int(rng, 1, hi), hi=hi, weights=rng.random() < 0.5,
                    shape_seed=seed)
    B = _log_int(rng, 1, 16)
    hi = _log_int(rng, 20, 8192)
    budget = _log_int(rng, 4, hi // 2)
    return dict(op=op, B=B, Hkv=Hkv, D=D, page=page, lo=_log_int(rng, 1, hi), hi=hi,
                budget=budget, recent=rng.randrange(0, budget + 1), shape_seed=seed)


def lengths(case):
    """Tokens of each sequence: a part of the case, the same for every seed."""
    rng = random.Random(case["shape_seed"])
    if "tokens" in case:
        left, out = case["tokens"], []
        while left > 0:
            n = min(left, _log_int(rng, max(1, case["max_len"] // 16), case["max_len"]))
            out.append(n)
            left -= n
        return out
    return [_log_int(rng, case["lo"], case["hi"]) for _ in range(case["B"])]


def past_lengths(case):
    """Tokens already held by each sequence of a store case."""
    rng = random.Random(case["shape_seed"] + 1)
    return [rng.randrange(case["past"] + 1) for _ in range(case["B"])]


# ------------------------------------------------------------------ work

def _cached_bytes(D):
    """Bytes of a cached key and value: codes, minima and scales."""
    return 2 * (D // 2 + D // GROUP * 4)


def work(case):
    D, Hkv, lens = case["D"], case["Hkv"], lengths(case)
    n = sum(lens)
    if case["op"] in ("prompt", "train"):
        Hq = case["Hq"]
        pairs = sum(x * (x + 1) // 2 for x in lens)
        flops = 4 * pairs * Hq * D
        nbytes = n * D * 2 * (2 * Hq + 2 * Hkv) + n * Hq * 4
        if case["op"] == "train":
            flops += 10 * pairs * Hq * D
            nbytes += n * D * 2 * (2 * Hq + 2 * Hkv)  # dO in, dq, dk, dv out
        return {"bytes": nbytes, "flops": flops}
    if case["op"] == "store":
        per = 2 * D * 2 + 2 * _cached_bytes(D) + 2 * D * 2  # k, v in; store; load; values out
        return {"bytes": n * Hkv * per, "flops": 0}
    if case["op"] == "step":
        Hq, B = case["Hq"], case["B"]
        nbytes = n * Hkv * _cached_bytes(D) + B * Hq * (2 * D * 2 + 4)
        if case["weights"]:
            nbytes += n * Hkv * 8
        return {"bytes": nbytes, "flops": 4 * n * Hq * D}
    kept = sum(min(x, case["budget"]) for x in lens)
    per = 3 * _cached_bytes(D) + 2 * D * 2  # load, store, load again; values out
    return {"bytes": kept * Hkv * (per + 8) + n * Hkv * 4, "flops": 0}


# ------------------------------------------------------------------ quantiser (plain form)

def quantise(x):
    """bf16 [..., D] -> codes uint8 [..., D], minima and scales fp32 [..., D/32]."""
    g = x.float().unflatten(-1, (-1, GROUP))
    mn = g.amin(-1)
    scale = ((g.amax(-1) - mn) / 15).to(torch.bfloat16).float()
    safe = torch.where(scale > 0, scale, torch.ones_like(scale))
    code = ((g - mn[..., None]) / safe[..., None]).round().clamp(0, 15)
    code = torch.where(scale[..., None] > 0, code, torch.zeros_like(code))
    return code.flatten(-2).to(torch.uint8), mn, scale


def pack(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def dequantise(packed, mn, scale):
    """Packed codes -> the fp32 values they stand for."""
    code = torch.stack((packed & 15, packed >> 4), -1).flatten(-2)
    g = code.float().unflatten(-1, (-1, GROUP))
    return (mn[..., None] + scale[..., None] * g).flatten(-2)


# ------------------------------------------------------------------ inputs

def _randn(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(torch.bfloat16)


def _keys(gen, *shape):
    """Keys as a projection gives them: some channels with an offset of their own."""
    off = torch.randn(shape[-2:], generator=gen, device="cuda") * 2
    return (torch.randn(*shape, generator=gen, device="cuda") + off).to(torch.bfloat16)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cu(lens):
    return _i32([0] + [sum(lens[:i + 1]) for i in range(len(lens))])


def _page_table(gen, lens, page, first=0):
    """Pages of each sequence, scattered over a pool: (table [B, width], pool size)."""
    width = max(1, max(-(-x // page) for x in lens))
    n = len(lens) * width
    perm = torch.randperm(n, generator=gen, device="cuda").to(torch.int32) + first
    return perm.view(len(lens), width).contiguous(), n


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lens, D, Hkv = lengths(case), case["D"], case["Hkv"]
    n = sum(lens)
    s = {"case": case, "lens": lens}
    if case["op"] in ("prompt", "train"):
        s["q"] = _randn(gen, n, case["Hq"], D)
        s["k"] = _randn(gen, n, Hkv, D)
        s["v"] = _randn(gen, n, Hkv, D)
        s["cu"] = _cu(lens)
        if case["op"] == "train":
            s["do"] = _randn(gen, n, case["Hq"], D)
        return s
    # packed new keys and values, as prefill or a decoding step hands them over
    s["k"], s["v"] = _keys(gen, n, Hkv, D), _randn(gen, n, Hkv, D)
    s["cu"], page = _cu(lens), case["page"]
    if case["op"] == "store":
        past = past_lengths(case)
        s["width"] = max(lens)
        total = [a + b for a, b in zip(past, lens)]
        table, pages = _page_table(gen, total, page)
        s["past"] = _i32(past)
        s["count"] = _i32(lens)
        if own:
            import exact_attention_blackwell_tiled_gb300 as fa
            s["table"] = table
            s["cache"] = fa.cache4_empty(pages, Hkv, D, page, device="cuda")
        else:
            tok, seq = _token_slots(lens)
            s["seq"], s["tok"] = seq, tok
            slots = max(total)
            s["codes"] = torch.zeros(2, len(lens), Hkv, slots, D // 2, dtype=torch.uint8,
                                     device="cuda")
            s["mn"] = torch.zeros(2, len(lens), Hkv, slots, D // GROUP, device="cuda")
            s["scale"] = torch.zeros_like(s["mn"])
        return s
    s["len"] = _i32(lens)
    slots = max(lens)
    if case["op"] == "step":
        s["q"] = _randn(gen, len(lens), case["Hq"], D)
    if case["op"] == "evict" or case["weights"]:
        # sums of softmax weights: most keys near nothing, a few large, ties at the bottom
        w = torch.rand(len(lens), Hkv, slots, generator=gen, device="cuda") ** 6
        w = torch.where(w < 1e-3, torch.zeros_like(w), w)
        s["w"] = w * (torch.arange(slots, device="cuda") < s["len"][:, None, None])
        s["w_out"] = torch.zeros_like(s["w"])
    table, pages = _page_table(gen, lens, page)
    if own:
        import exact_attention_blackwell_tiled_gb300 as fa
        s["table"] = table
        extra = 0
        if case["op"] == "evict":
            s["table_out"], extra = _page_table(gen, [min(x, case["budget"]) for x in lens], page,
                                                first=pages)
        s["cache"] = fa.cache4_empty(pages + extra, Hkv, D, page, device="cuda")
        fa.cache4_append(s["cache"], s.pop("k"), s.pop("v"), s["table"], torch.zeros_like(s["len"]),
                         cu_seqlens=s["cu"])
        if case["op"] == "step":
            s["ws"] = torch.empty(fa.cache4_attend_workspace_bytes(
                len(lens), case["Hq"], Hkv, D, slots if case["weights"] else 0),
                dtype=torch.uint8, device="cuda")
    else:
        tok, seq = _token_slots(lens)
        codes, mn, scale = [], [], []
        for x in (s.pop("k"), s.pop("v")):
            c, m, sc = quantise(x)
            for dst, src in ((codes, pack(c)), (mn, m), (scale, sc)):
                full = torch.zeros(len(lens), Hkv, slots, src.shape[-1], dtype=src.dtype,
                                   device="cuda")
                full[seq, :, tok] = src
                dst.append(full)
        s["codes"], s["mn"], s["scale"] = torch.stack(codes), torch.stack(mn), torch.stack(scale)
    return s


def _token_slots(lens):
    """Packed token -> (index inside its sequence, sequence)."""
    tok = torch.cat([torch.arange(x) for x in lens]).cuda()
    seq = torch.cat([torch.full((x,), i) for i, x in enumerate(lens)]).cuda()
    return tok, seq


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"prompt": _own_prompt, "train": _own_train, "store": _own_store,
                "step": _own_step, "evict": _own_evict}[op](s)
    return {"prompt": _plain_prompt, "train": _plain_train, "store": _plain_store,
            "step": _plain_step, "evict": _plain_evict}[op](s)


def _own_prompt(s):
    import exact_attention_blackwell_tiled_gb300 as fa
    return fa.fwd_varlen(s["q"], s["k"], s["v"], s["cu"], causal=True)


def _own_train(s):
    import exact_attention_blackwell_tiled_gb300 as fa
    o, lse = fa.fwd_varlen(s["q"], s["k"], s["v"], s["cu"], causal=True)
    grads = fa.bwd_varlen(s["q"], s["k"], s["v"], o, s["do"], lse, s["cu"], causal=True,
                          deterministic=s["case"]["deterministic"])
    return (o, lse, *grads)


def _own_store(s):
    import exact_attention_blackwell_tiled_gb300 as fa
    fa.cache4_append(s["cache"], s["k"], s["v"], s["table"], s["past"], cu_seqlens=s["cu"])
    return fa.cache4_read(s["cache"], s["table"], s["past"], s["count"], s["width"],
                          s["case"]["D"])


def _own_step(s):
    import exact_attention_blackwell_tiled_gb300 as fa
    kw = dict(weights=s["w"], weights_out=s["w_out"]) if s["case"]["weights"] else {}
    o, lse = fa.cache4_attend(s["q"], s["cache"], s["table"], s["len"], workspace=s["ws"], **kw)
    return (o, lse, s["w_out"]) if s["case"]["weights"] else (o, lse)


def _own_evict(s):
    import exact_attention_blackwell_tiled_gb300 as fa
    c = s["case"]
    src, w, n = fa.cache4_evict(s["cache"], s["table"], s["len"], s["w"], s["table_out"],
                                c["D"], budget=c["budget"], recent=c["recent"])
    k, v = fa.cache4_read(s["cache"], s["table_out"], torch.zeros_like(n), n, c["budget"], c["D"])
    return src, w, n, k, v


def _plain_heads(s, b0, n):
    """q [Hkv, group, n, D], k and v [Hkv, n, D] of the sequence at token b0, in fp32."""
    c = s["case"]
    q = s["q"][b0:b0 + n].float().view(n, c["Hkv"], -1, c["D"]).permute(1, 2, 0, 3)
    k = s["k"][b0:b0 + n].float().transpose(0, 1)
    v = s["v"][b0:b0 + n].float().transpose(0, 1)
    return q, k, v


def _plain_softmax(q, k, scale, mask):
    """Causal weights and log-sum-exp of one kv head: q [group, n, D], k [n, D]."""
    sc = (q @ k.T) * scale
    sc = torch.where(mask, sc, torch.full_like(sc, -math.inf))
    m = sc.amax(-1, keepdim=True)
    p = (sc - m).exp()
    total = p.sum(-1, keepdim=True)
    return p / total, (m + total.log())[..., 0]


def _plain_prompt(s):
    o, lse, _ = _plain_forward(s)
    return o.to(torch.bfloat16), lse


def _plain_forward(s, visit=None):
    c = s["case"]
    scale = 1 / math.sqrt(c["D"])
    o = torch.empty(s["q"].shape, device="cuda")
    lse = torch.empty(c["Hq"], s["q"].shape[0], device="cuda")
    group, b0 = c["Hq"] // c["Hkv"], 0
    for n in s["lens"]:
        q, k, v = _plain_heads(s, b0, n)
        pos = torch.arange(n, device="cuda")
        mask = pos[:, None] >= pos
        for h in range(c["Hkv"]):
            p, l = _plain_softmax(q[h], k[h], scale, mask)
            out = p @ v[h]
            o[b0:b0 + n, h * group:(h + 1) * group] = out.transpose(0, 1)
            lse[h * group:(h + 1) * group, b0:b0 + n] = l
            if visit:
                visit(b0, n, h, q[h], k[h], v[h], p, out)
        b0 += n
    return o, lse, scale


def _plain_train(s):
    c = s["case"]
    group, scale = c["Hq"] // c["Hkv"], 1 / math.sqrt(c["D"])
    dq = torch.empty(s["q"].shape, device="cuda")
    dk = torch.empty(s["k"].shape, device="cuda")
    dv = torch.empty(s["v"].shape, device="cuda")

    def visit(b0, n, h, q, k, v, p, out):
        heads = slice(h * group, (h + 1) * group)
        do = s["do"][b0:b0 + n, heads].float().transpose(0, 1)
        dv[b0:b0 + n, h] = (p.transpose(1, 2) @ do).sum(0)
        ds = p * (do @ v.T - (do * out).sum(-1, keepdim=True))
        dq[b0:b0 + n, heads] = ((ds @ k) * scale).transpose(0, 1)
        dk[b0:b0 + n, h] = (ds.transpose(1, 2) @ q).sum(0) * scale

    o, lse, _ = _plain_forward(s, visit)
    bf = torch.bfloat16
    return o.to(bf), lse, dq.to(bf), dk.to(bf), dv.to(bf)


def _plain_store(s):
    c = s["case"]
    out = []
    slot = s["past"].long()[s["seq"]] + s["tok"]
    for i, x in enumerate((s["k"], s["v"])):
        code, mn, scale = quantise(x)
        s["codes"][i][s["seq"], :, slot] = pack(code)
        s["mn"][i][s["seq"], :, slot] = mn
        s["scale"][i][s["seq"], :, slot] = scale
        val = torch.zeros(c["B"], c["Hkv"], s["width"], c["D"], dtype=torch.bfloat16,
                          device="cuda")
        val[s["seq"], :, s["tok"]] = dequantise(
            s["codes"][i][s["seq"], :, slot], s["mn"][i][s["seq"], :, slot],
            s["scale"][i][s["seq"], :, slot]).to(torch.bfloat16)
        out.append(val)
    return tuple(out)


def _plain_step(s):
    c = s["case"]
    k = dequantise(s["codes"][0], s["mn"][0], s["scale"][0])
    v = dequantise(s["codes"][1], s["mn"][1], s["scale"][1])
    q = s["q"].float().view(c["B"], c["Hkv"], -1, c["D"])
    sc = (q @ k.transpose(2, 3)) * (1 / math.sqrt(c["D"]))
    live = torch.arange(sc.shape[-1], device="cuda") < s["len"][:, None, None, None]
    sc = torch.where(live, sc, torch.full_like(sc, -math.inf))
    m = sc.amax(-1, keepdim=True)
    p = (sc - m).exp()
    total = p.sum(-1, keepdim=True)
    p = p / total
    o = (p @ v).view(c["B"], c["Hq"], c["D"]).to(torch.bfloat16)
    lse = (m + total.log()).view(c["B"], c["Hq"])
    if not c["weights"]:
        return o, lse
    return o, lse, s["w"] + p.sum(2)


def _plain_evict(s):
    c = s["case"]
    budget, recent = c["budget"], c["recent"]
    n = s["len"].long()[:, None, None]
    idx = torch.arange(s["w"].shape[-1], device="cuda").expand(s["w"].shape)
    # the latest keys rank above every weight; a stable sort sends ties to the lowest index
    rank = torch.where(idx >= n - recent, torch.full_like(s["w"], math.inf), s["w"])
    rank = torch.where(idx < n, rank, torch.full_like(rank, -math.inf))
    order = rank.sort(dim=-1, descending=True, stable=True).indices[..., :budget]
    if order.shape[-1] < budget:
        order = torch.cat((order, order.new_full((*order.shape[:2], budget - order.shape[-1]),
                                                 s["w"].shape[-1])), -1)
    kept = torch.where(torch.arange(budget, device="cuda") < n, order,
                       torch.full_like(order, 1 << 30)).sort(-1).values
    live = kept < n
    at = torch.where(live, kept, torch.zeros_like(kept))
    w = torch.where(live, s["w"].gather(-1, at), torch.zeros((), device="cuda"))
    src = torch.where(live, kept, torch.full_like(kept, -1)).to(torch.int32)
    vals = []
    for i in range(2):
        take = [x[i].gather(2, at[..., None].expand(-1, -1, -1, x.shape[-1]))
                for x in (s["codes"], s["mn"], s["scale"])]
        val = dequantise(*take)
        vals.append(torch.where(live[..., None], val, torch.zeros_like(val)).to(torch.bfloat16))
    return src, w, torch.clamp(s["len"], max=budget), vals[0], vals[1]


# ------------------------------------------------------------------ the definitions in 64 bits

def _stored(x):
    """The values a cache of 4-bit codes holds for x [..., D], from the definition."""
    d = x.double().reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    low, high = d.min(-1, keepdim=True)[0], d.max(-1, keepdim=True)[0]
    step = ((high - low) / 15.0).float().bfloat16().double()
    ratio = torch.where(step > 0, (d - low) / step.clamp_min(1e-300), torch.zeros_like(d))
    return (low + step * ratio.round().clamp(0.0, 15.0)).reshape(x.shape)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        return _exact(case, seed)
    finally:
        own = was


def _exact(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lens, D, Hkv, op = lengths(case), case["D"], case["Hkv"], case["op"]
    n = sum(lens)
    if op in ("prompt", "train"):
        Hq = case["Hq"]
        q, k, v = (_randn(gen, n, h, D).double() for h in (Hq, Hkv, Hkv))
        do = _randn(gen, n, Hq, D).double() if op == "train" else None
        outs = [torch.empty(n, Hq, D, dtype=torch.float64, device="cuda"),
                torch.empty(Hq, n, dtype=torch.float64, device="cuda")]
        grads = [torch.zeros_like(x) for x in (q, k, v)] if op == "train" else []
        start = 0
        for m in lens:
            rows = slice(start, start + m)
            above = torch.ones(m, m, dtype=torch.bool, device="cuda").triu(1)
            for h in range(Hq):
                kv = h * Hkv // Hq
                qh, kh, vh = q[rows, h], k[rows, kv], v[rows, kv]
                logits = (torch.einsum("id,jd->ij", qh, kh) / math.sqrt(D)).masked_fill_(
                    above, -math.inf)
                lse = torch.logsumexp(logits, 1)
                prob = logits.sub_(lse[:, None]).exp_()
                out = torch.einsum("ij,jd->id", prob, vh)
                outs[0][rows, h], outs[1][h, rows] = out, lse
                if op == "train":
                    g = do[rows, h]
                    grads[2][rows, kv] += torch.einsum("ij,id->jd", prob, g)
                    dlog = torch.einsum("id,jd->ij", g, vh).sub_((g * out).sum(1)[:, None])
                    dlog.mul_(prob).div_(math.sqrt(D))
                    grads[0][rows, h] = torch.einsum("ij,jd->id", dlog, kh)
                    grads[1][rows, kv] += torch.einsum("ij,id->jd", dlog, qh)
            start += m
        return (*outs, *grads)
    k, v = _keys(gen, n, Hkv, D), _randn(gen, n, Hkv, D)
    ends = [sum(lens[:i + 1]) for i in range(len(lens))]
    if op == "store":
        width = max(lens)
        out = torch.zeros(2, case["B"], Hkv, width, D, dtype=torch.float64, device="cuda")
        for i, x in enumerate((k, v)):
            for b, m in enumerate(lens):
                out[i, b, :, :m] = _stored(x[ends[b] - m:ends[b]]).transpose(0, 1)
        return out[0], out[1]
    s = prepare(case, seed)
    slots = max(lens)
    if op == "step":
        Hq = case["Hq"]
        group = Hq // Hkv
        o = torch.empty(case["B"], Hq, D, dtype=torch.float64, device="cuda")
        lse = torch.empty(case["B"], Hq, dtype=torch.float64, device="cuda")
        w = s["w"].double() if case["weights"] else None
        for b, m in enumerate(lens):
            kb, vb = (_stored(x[ends[b] - m:ends[b]]) for x in (k, v))
            qb = s["q"][b].double().view(Hkv, group, D)
            logits = torch.einsum("hgd,jhd->hgj", qb, kb) / math.sqrt(D)
            lse[b] = torch.logsumexp(logits, -1).view(Hq)
            prob = torch.softmax(logits, -1)
            o[b] = torch.einsum("hgj,jhd->hgd", prob, vb).reshape(Hq, D)
            if w is not None:
                w[b, :, :m] += prob.sum(1)
        return (o, lse) if w is None else (o, lse, w)
    budget, recent = case["budget"], case["recent"]
    src = torch.full((case["B"], Hkv, budget), -1, dtype=torch.int32, device="cuda")
    w = torch.zeros(case["B"], Hkv, budget, dtype=torch.float64, device="cuda")
    vals = torch.zeros(2, case["B"], Hkv, budget, D, dtype=torch.float64, device="cuda")
    weights = s["w"].cpu()
    for b, m in enumerate(lens):
        late = min(recent, m)
        kb, vb = (_stored(x[ends[b] - m:ends[b]]) for x in (k, v))
        for h in range(Hkv):
            if m <= budget:
                keep = list(range(m))
            else:
                early = weights[b, h, :m - late].tolist()
                best = sorted(range(m - late), key=lambda i: (-early[i], i))[:budget - late]
                keep = sorted(best) + list(range(m - late, m))
            at = torch.tensor(keep, dtype=torch.int64, device="cuda")
            c = len(keep)
            src[b, h, :c] = at.to(torch.int32)
            w[b, h, :c] = s["w"][b, h, at].double()
            vals[0, b, h, :c], vals[1, b, h, :c] = kb[at, h], vb[at, h]
    counts = torch.tensor([min(m, budget) for m in lens], dtype=torch.int32, device="cuda")
    return src, w, counts, vals[0], vals[1]
