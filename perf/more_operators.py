"""Cases of the sliding window with sinks, of the norms and rotation of queries and keys,
and of the page tables of a paged cache.

Five groups of calls around a decoder's attention:

* ``prompt``  causal attention over packed prompts in which a query sees the latest
  ``window`` tokens before it and the first ``sinks`` tokens of its sequence;
* ``train``   the same with its backward pass (o, lse, dq, dk, dv);
* ``step``    one query token per sequence attends to its 4-bit cache in that window;
* ``rope``    RMS norms of every query and key head and the rotation by position in one
  pass, or that with its backward pass and the norm weights' gradients;
* ``pages``   page tables brought up to date for the lengths to come: new pages from the
  pool, pages behind the window and of ended sequences back to it, and the position and
  cache slot of every new token.

Visible to query i of a sequence: keys j <= i with j >= i - window or j < sinks.

``own`` selects the framework's operators; otherwise the plain forms below run.
"""
import math
import random

import torch

own = False

GROUP = 32   # elements of a cached vector that share a minimum and a scale
EPS = 1e-6   # of the norms
BASE = 10000.0
BLOCK = 512  # query rows the plain form takes at a time


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a handful of short chat turns prefilled together: launch latency counts
        dict(name="prompt_short", op="prompt", Hq=4, Hkv=2, D=64, tokens=437, max_len=200,
             window=63, sinks=4, shape_seed=3),
        # a full prefill batch of a grouped-head model with a window of 1024 tokens
        dict(name="prompt_16k", op="prompt", Hq=32, Hkv=8, D=128, tokens=16384, max_len=8192,
             window=1023, sinks=4, shape_seed=11),
        # one training step over long packed documents, one head per kv head
        dict(name="train_16k", op="train", Hq=16, Hkv=16, D=128, tokens=16384, max_len=8192,
             window=1023, sinks=16, deterministic=False, shape_seed=23),
        # a small packed step with head dimension 64 and bit-reproducible gradients
        dict(name="train_d64_det", op="train", Hq=16, Hkv=4, D=64, tokens=4099, max_len=1500,
             window=300, sinks=7, deterministic=True, shape_seed=5),
        # one long conversation: a single step's latency
        dict(name="step_one", op="step", B=1, Hq=32, Hkv=8, D=128, page=16, lo=5000, hi=5000,
             window=511, sinks=4, weights=False, shape_seed=1),
        # a busy server: 64 sequences of mixed lengths, weights kept for eviction
        dict(name="step_b64", op="step", B=64, Hq=32, Hkv=8, D=128, page=64, lo=512, hi=16384,
             window=4095, sinks=4, weights=True, shape_seed=17),
        # a decoding step's queries and keys, slices of the fused projection
        dict(name="rope_step", op="rope", T=64, Hq=32, Hkv=8, D=128, rot=128, interleaved=False,
             max_pos=131072, run=1, train=False, wtype="bfloat16", shape_seed=37),
        # a prefill batch's, far into long contexts
        dict(name="rope_prompt", op="rope", T=16384, Hq=32, Hkv=8, D=128, rot=128,
             interleaved=False, max_pos=131072, run=2048, train=False, wtype="bfloat16",
             shape_seed=41),
        # a training step's forward and backward pass, weights in 32 bits
        dict(name="rope_train", op="rope", T=16384, Hq=16, Hkv=16, D=128, rot=128,
             interleaved=False, max_pos=8192, run=8192, train=True, wtype="float32",
             shape_seed=43),
        # an odd number of tokens, half of each head rotated in adjacent pairs
        dict(name="rope_train_odd", op="rope", T=4099, Hq=14, Hkv=2, D=64, rot=32,
             interleaved=True, max_pos=2000, run=1500, train=True, wtype="bfloat16",
             shape_seed=47),
        # a decoding step's page tables: a new page every 64 tokens, one behind the window back
        dict(name="pages_step", op="pages", B=64, page=64, lo=512, hi=16384, grow_lo=1, grow_hi=1,
             finish=0.05, window=4095, sinks=4, shape_seed=53),
        # a large server takes in prompts: some sequences start, some end, the rest step
        dict(name="pages_prompt", op="pages", B=1024, page=16, lo=1, hi=8192, grow_lo=1,
             grow_hi=2048, finish=0.1, window=-1, sinks=0, shape_seed=59),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "train", "step", "rope", "pages"])
    seed = rng.randrange(1 << 30)
    if op == "pages":
        B = _log_int(rng, 1, 1024)
        hi = _log_int(rng, 1, 16384)
        grow = rng.choice([1, _log_int(rng, 1, max(1, 400000 // B) if B > 200 else 2048)])
        return dict(op=op, B=B, page=rng.choice([16, 32, 64, 128]), lo=_log_int(rng, 1, hi), hi=hi,
                    grow_lo=1, grow_hi=min(grow, 2048), finish=rng.choice([0.0, 0.1, 0.5]),
                    window=rng.choice([-1, _log_int(rng, 1, 8192)]),
                    sinks=rng.choice([0, 1, 4, 64]), shape_seed=seed)
    D = rng.choice([64, 128])
    if op == "rope":
        Hq, Hkv = rng.choice([(1, 1), (4, 2), (8, 1), (14, 2), (16, 16), (32, 8)])
        T = _log_int(rng, 1, 16384)
        train = rng.random() < 0.5
        if train and Hq == 32:
            T = min(T, 8192)
        return dict(op=op, T=T, Hq=Hq, Hkv=Hkv, D=D, rot=rng.choice([16, D // 2, D, D]),
                    interleaved=rng.random() < 0.5, max_pos=_log_int(rng, 2, 131072),
                    run=_log_int(rng, 1, 4096), train=train,
                    wtype=rng.choice(["bfloat16", "float32"]), shape_seed=seed)
    window, sinks = _log_int(rng, 1, 4095), rng.choice([1, 2, 4, 4, 7, 16, 33, 64, 128])
    if op in ("prompt", "train"):
        Hq, Hkv = rng.choice([(2, 2), (4, 2), (8, 1), (16, 4), (16, 16), (32, 8)])
        if op == "train" and Hq == 32:
            Hq, Hkv = 14, 2
        tokens = _log_int(rng, 60, 12000)
        case = dict(op=op, Hq=Hq, Hkv=Hkv, D=D, tokens=tokens,
                    max_len=_log_int(rng, max(20, tokens // 24), min(tokens, 8192)),
                    window=min(window, 1023), sinks=sinks, shape_seed=seed)
        if op == "train":
            case["deterministic"] = rng.random() < 0.5
        return case
    B = _log_int(rng, 1, 64)
    Hkv = rng.choice([1, 2, 4, 8])
    hi = _log_int(rng, 1, 262144 // max(B, 16))
    return dict(op=op, B=B, Hq=Hkv * rng.choice([1, 2, 4, 5, 8, 12]), Hkv=Hkv, D=D,
                page=rng.choice([16, 32, 64, 128]), lo=_log_int(rng, 1, hi), hi=hi, window=window,
                sinks=sinks, weights=rng.random() < 0.5, shape_seed=seed)


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


def next_lengths(case):
    """Tokens held before and after the new ones, of each sequence of a pages case."""
    rng = random.Random(case["shape_seed"] + 1)
    old, new = [], []
    for n in lengths(case):
        if rng.random() < case["finish"]:
            old.append(n)
            new.append(0)
        else:
            n = 0 if case["grow_hi"] > 1 and rng.random() < 0.5 else n  # a sequence that starts
            old.append(n)
            new.append(n + _log_int(rng, case["grow_lo"], case["grow_hi"]))
    return old, new


def positions(case):
    """Positions of the tokens of a rope case: runs of consecutive ones."""
    rng = random.Random(case["shape_seed"])
    out = []
    while len(out) < case["T"]:
        n = min(case["max_pos"], _log_int(rng, max(1, case["run"] // 4), case["run"]))
        first = rng.randrange(case["max_pos"] - n + 1)
        out += range(first, first + n)
    return out[:case["T"]]


# ------------------------------------------------------------------ work

def _cached_bytes(D):
    """Bytes of a cached key and value: codes, minima and scales."""
    return 2 * (D // 2 + D // GROUP * 4)


def _visible(i, window, sinks):
    """Keys that query i sees."""
    return min(i, window) + 1 + min(sinks, max(0, i - window))


def work(case):
    op = case["op"]
    if op == "pages":
        old, new = next_lengths(case)
        T = sum(max(0, n - o) for o, n in zip(old, new))
        page = case["page"]
        moved = sum(abs(-(-n // page) - -(-o // page)) for o, n in zip(old, new))
        return {"bytes": 12 * case["B"] + 12 * T + 12 * moved, "flops": 0}
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    if op == "rope":
        n = case["T"] * (Hq + Hkv) * D
        rows = len(set(positions(case)))
        per, flops = (4, 12) if not case["train"] else (10, 42)
        return {"bytes": per * n + 4 * case["T"] + 4 * rows * case["rot"], "flops": flops * n}
    lens, window, sinks = lengths(case), case["window"], case["sinks"]
    n = sum(lens)
    if op in ("prompt", "train"):
        pairs = sum(_visible(i, window, sinks) for m in lens for i in range(m))
        flops = 4 * pairs * Hq * D
        nbytes = n * D * 2 * (2 * Hq + 2 * Hkv) + n * Hq * 4
        if op == "train":
            flops += 10 * pairs * Hq * D
            nbytes += n * D * 2 * (2 * Hq + 2 * Hkv)  # dO in, dq, dk, dv out
        return {"bytes": nbytes, "flops": flops}
    B = case["B"]
    seen = sum(_visible(m - 1, window, sinks) for m in lens)
    nbytes = seen * Hkv * _cached_bytes(D) + B * Hq * (2 * D * 2 + 4)
    if case["weights"]:
        nbytes += n * Hkv * 8
    return {"bytes": nbytes, "flops": 4 * seen * Hq * D}


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
    out = [0]
    for x in lens:
        out.append(out[-1] + x)
    return _i32(out)


def _projections(case, gen):
    """The fused projection [T, Hq + 2 Hkv, D] and the norms' weights."""
    T, Hq, Hkv, D = (case[x] for x in ("T", "Hq", "Hkv", "D"))
    channel = torch.rand(Hq + 2 * Hkv, D, generator=gen, device="cuda") * 2 + 0.25
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=gen, device="cuda")
    qkv = (qkv * channel).to(torch.bfloat16)
    w = 1 + 0.2 * torch.randn(2, D, generator=gen, device="cuda")
    w = w.to(getattr(torch, case["wtype"]))
    grads = [_randn(gen, T, h, D) for h in (Hq, Hkv)] if case["train"] else []
    return qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], w[0], w[1], grads


def _angles(case, dtype):
    """cos and sin [max_pos, rot/2], the angles taken in 64 bits."""
    half = case["rot"] // 2
    rate = BASE ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    at = torch.arange(case["max_pos"], dtype=torch.float64, device="cuda")[:, None] * rate
    return at.cos().to(dtype), at.sin().to(dtype)


def _pool(case, gen):
    """Tables and free pages in mid-service: one buffer [tables | stack of free pages | its height]."""
    old, new = next_lengths(case)
    B, page, window, sinks = case["B"], case["page"], case["window"], case["sinks"]
    width = max(-(-max(a, b) // page) for a, b in zip(old, new)) + 1
    e = torch.arange(width, device="cuda")
    o = _i32(old).long()[:, None]
    held = e * page < o
    if window >= 0:
        held &= ~(((e + 1) * page <= o - 1 - window) & (e * page >= sinks))
    n_held = int(held.sum())
    wanted = sum(max(0, -(-b // page) - -(-a // page)) for a, b in zip(old, new))
    pages = n_held + wanted + (n_held + wanted) // 8 + 64
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    table[held] = order[:n_held]
    free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    free[:pages - n_held] = order[n_held:]
    buf = torch.cat((table.flatten(), free, _i32([pages - n_held])))
    return buf, _i32(old), _i32(new), width, pages


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op == "pages":
        s["saved"], s["old"], s["new"], width, pages = _pool(case, gen)
        s["buf"] = torch.empty_like(s["saved"])  # a pass starts from the same tables
        n = case["B"] * width
        s["table"] = s["buf"][:n].view(case["B"], width)
        s["free"], s["height"] = s["buf"][n:n + pages], s["buf"][n + pages:]
        old, new = next_lengths(case)
        s["T"] = sum(max(0, b - a) for a, b in zip(old, new))
        return s
    if op == "rope":
        s["q"], s["k"], s["qw"], s["kw"], s["grads"] = _projections(case, gen)
        s["pos"] = _i32(positions(case))
        if own:
            import exact_attention_blackwell_tiled_gb300 as fa
            s["cos"], s["sin"] = fa.rope_table(case["max_pos"], case["rot"], BASE)
        else:
            s["cos"], s["sin"] = _angles(case, torch.float32)
        return s
    lens, D, Hkv = lengths(case), case["D"], case["Hkv"]
    n = sum(lens)
    s["lens"] = lens
    if op in ("prompt", "train"):
        s["q"] = _randn(gen, n, case["Hq"], D)
        s["k"] = _randn(gen, n, Hkv, D)
        s["v"] = _randn(gen, n, Hkv, D)
        s["cu"] = _cu(lens)
        if op == "train":
            s["do"] = _randn(gen, n, case["Hq"], D)
        return s
    k, v = _keys(gen, n, Hkv, D), _randn(gen, n, Hkv, D)
    s["len"], slots = _i32(lens), max(lens)
    s["q"] = _randn(gen, len(lens), case["Hq"], D)
    if case["weights"]:
        # sums of softmax weights: most keys near nothing, a few large
        w = torch.rand(len(lens), Hkv, slots, generator=gen, device="cuda") ** 6
        s["w"] = w * (torch.arange(slots, device="cuda") < s["len"][:, None, None])
        s["w_out"] = torch.zeros_like(s["w"])
    if own:
        import exact_attention_blackwell_tiled_gb300 as fa
        page = case["page"]
        width = -(-slots // page)
        order = torch.randperm(len(lens) * width, generator=gen, device="cuda").to(torch.int32)
        table = order.view(len(lens), width).contiguous()
        s["cache"] = fa.cache4_empty(order.numel(), Hkv, D, page, device="cuda")
        fa.cache4_append(s["cache"], k, v, table, torch.zeros_like(s["len"]), cu_seqlens=_cu(lens))
        # the pages behind the window are other sequences' by now
        e = torch.arange(width, device="cuda")
        gone = ((e + 1) * page <= s["len"][:, None] - 1 - case["window"]) & (
            e * page >= case["sinks"])
        s["table"] = torch.where(gone, torch.full_like(table, -1), table)
        s["ws"] = torch.empty(fa.cache4_attend_workspace_bytes(
            len(lens), case["Hq"], Hkv, D, slots if case["weights"] else 0),
            dtype=torch.uint8, device="cuda")
    else:
        tok = torch.cat([torch.arange(x) for x in lens]).cuda()
        seq = torch.cat([torch.full((x,), i) for i, x in enumerate(lens)]).cuda()
        codes, mn, scale = [], [], []
        for x in (k, v):
            c, m, sc = quantise(x)
            for dst, src in ((codes, c[..., 0::2] | (c[..., 1::2] << 4)), (mn, m), (scale, sc)):
                full = torch.zeros(len(lens), Hkv, slots, src.shape[-1], dtype=src.dtype,
                                   device="cuda")
                full[seq, :, tok] = src
                dst.append(full)
        s["codes"], s["mn"], s["scale"] = codes, mn, scale
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    c = s["case"]
    if own:
        return {"prompt": _own_prompt, "train": _own_train, "step": _own_step, "rope": _own_rope,
                "pages": _own_pages}[c["op"]](s, c)
    return {"prompt": _plain_prompt, "train": _plain_train, "step": _plain_step,
            "rope": _plain_rope, "pages": _plain_pages}[c["op"]](s, c)


def _own_prompt(s, c):
    import exact_attention_blackwell_tiled_gb300 as fa
    return fa.fwd_varlen(s["q"], s["k"], s["v"], s["cu"], window=(c["window"], 0),
                         sinks=c["sinks"])


def _own_train(s, c):
    import exact_attention_blackwell_tiled_gb300 as fa
    kw = dict(window=(c["window"], 0), sinks=c["sinks"])
    o, lse = fa.fwd_varlen(s["q"], s["k"], s["v"], s["cu"], **kw)
    grads = fa.bwd_varlen(s["q"], s["k"], s["v"], o, s["do"], lse, s["cu"],
                          deterministic=c["deterministic"], **kw)
    return (o, lse, *grads)


def _own_step(s, c):
    import exact_attention_blackwell_tiled_gb300 as fa
    kw = dict(weights=s["w"], weights_out=s["w_out"]) if c["weights"] else {}
    o, lse = fa.cache4_attend(s["q"], s["cache"], s["table"], s["len"], window_left=c["window"],
                              sinks=c["sinks"], workspace=s["ws"], **kw)
    return (o, lse, s["w_out"]) if c["weights"] else (o, lse)


def _own_rope(s, c):
    import exact_attention_blackwell_tiled_gb300 as fa
    args = (s["q"], s["k"], s["qw"], s["kw"], s["cos"], s["sin"], s["pos"])
    kw = dict(eps=EPS, interleaved=c["interleaved"])
    out = fa.norm_rope_fwd(*args, **kw)
    if not c["train"]:
        return out
    return (*out, *fa.norm_rope_bwd(*args, *s["grads"], **kw))


def _own_pages(s, c):
    import exact_attention_blackwell_tiled_gb300 as fa
    s["buf"].copy_(s["saved"])
    cu, pos, slots = fa.page_update(s["table"], s["free"], s["height"], s["old"], s["new"],
                                    c["page"], s["T"], window_left=c["window"], sinks=c["sinks"])
    return s["table"], s["free"], s["height"], cu, pos, slots


def _blocks(s, c):
    """(rows, keys, mask) of the plain form's steps: query rows, the rows of the keys that
    any of them sees, and which sees which."""
    b0 = 0
    for n in s["lens"]:
        for i0 in range(0, n, BLOCK):
            i1 = min(n, i0 + BLOCK)
            lo = max(0, i0 - c["window"])
            first = min(lo, c["sinks"])  # sinks in front of the window
            i = torch.arange(i0, i1, device="cuda")[:, None]
            j = torch.cat((torch.arange(first, device="cuda"), torch.arange(lo, i1, device="cuda")))
            mask = (j <= i) & ((j >= i - c["window"]) | (j < c["sinks"]))
            yield slice(b0 + i0, b0 + i1), b0 + j, mask
        b0 += n


def _plain_forward(s, c, visit=None):
    Hkv, D = c["Hkv"], c["D"]
    scale = 1 / math.sqrt(D)
    o = torch.empty(s["q"].shape, device="cuda")
    lse = torch.empty(c["Hq"], s["q"].shape[0], device="cuda")
    for rows, keys, mask in _blocks(s, c):
        # q [Hkv, group, rows, D], k and v [Hkv, 1, keys, D]
        q = s["q"][rows].float().unflatten(1, (Hkv, -1)).permute(1, 2, 0, 3)
        k, v = (s[x][keys].float().transpose(0, 1)[:, None] for x in ("k", "v"))
        sc = (q @ k.transpose(2, 3)) * scale
        sc = torch.where(mask, sc, torch.full_like(sc, -math.inf))
        m = sc.amax(-1, keepdim=True)
        p = (sc - m).exp()
        total = p.sum(-1, keepdim=True)
        p = p / total
        out = p @ v
        o[rows] = out.permute(2, 0, 1, 3).flatten(1, 2)
        lse[:, rows] = (m + total.log())[..., 0].flatten(0, 1)
        if visit:
            visit(rows, keys, q, k, v, p, out)
    return o.to(torch.bfloat16), lse


def _plain_prompt(s, c):
    return _plain_forward(s, c)


def _plain_train(s, c):
    Hkv, scale = c["Hkv"], 1 / math.sqrt(c["D"])
    dq = torch.empty(s["q"].shape, device="cuda")
    dk = torch.zeros(s["k"].shape, device="cuda")
    dv = torch.zeros(s["v"].shape, device="cuda")

    def visit(rows, keys, q, k, v, p, out):
        do = s["do"][rows].float().unflatten(1, (Hkv, -1)).permute(1, 2, 0, 3)
        ds = p * (do @ v.transpose(2, 3) - (do * out).sum(-1, keepdim=True))
        dq[rows] = ((ds @ k) * scale).permute(2, 0, 1, 3).flatten(1, 2)
        dv.index_add_(0, keys, (p.transpose(2, 3) @ do).sum(1).transpose(0, 1))
        dk.index_add_(0, keys, ((ds.transpose(2, 3) @ q) * scale).sum(1).transpose(0, 1))

    o, lse = _plain_forward(s, c, visit)
    bf = torch.bfloat16
    return o, lse, dq.to(bf), dk.to(bf), dv.to(bf)


def _plain_step(s, c):
    B, Hq, Hkv, D, window, sinks = (c[x] for x in ("B", "Hq", "Hkv", "D", "window", "sinks"))
    n = s["len"].long()[:, None]
    slots = s["codes"][0].shape[2]
    # slots in sight, sinks first; behind the last one: not live
    lo = torch.clamp(n - 1 - window, min=0)
    front = torch.clamp(lo, max=sinks)
    x = torch.arange(min(slots, window + 1 + sinks), device="cuda")
    at = torch.where(x < front, x.expand(B, -1), lo + x - front)
    live = at < n
    at = torch.where(live, at, torch.zeros_like(at))

    def values(i):
        take = [y[i].gather(2, at[:, None, :, None].expand(-1, Hkv, -1, y[i].shape[-1]))
                for y in (s["codes"], s["mn"], s["scale"])]
        return dequantise(*take)

    q = s["q"].float().view(B, Hkv, -1, D)
    sc = (q @ values(0).transpose(2, 3)) * (1 / math.sqrt(D))
    sc = torch.where(live[:, None, None], sc, torch.full_like(sc, -math.inf))
    m = sc.amax(-1, keepdim=True)
    p = (sc - m).exp()
    total = p.sum(-1, keepdim=True)
    p = p / total
    o = (p @ values(1)).view(B, Hq, D).to(torch.bfloat16)
    lse = (m + total.log()).view(B, Hq)
    if not c["weights"]:
        return o, lse
    # (slots that are not live add 0 to slot 0)
    return o, lse, s["w"].scatter_add(2, at[:, None].expand(-1, Hkv, -1), p.sum(2))


def _turn(x, cos, sin, c):
    """Rotates the pairs of the first rot elements of x [T, H, D]; cos and sin [T, 1, rot/2]."""
    rot = c["rot"]
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _plain_rope(s, c):
    cos, sin = (s[x][s["pos"].long()][:, None] for x in ("cos", "sin"))
    out, dx, dw = [], [], []
    for i, (x, w) in enumerate(((s["q"], s["qw"]), (s["k"], s["kw"]))):
        x, w = x.float(), w.float()
        r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
        unit = x * r
        out.append(_turn(unit * w, cos, sin, c).to(torch.bfloat16))
        if c["train"]:
            g = _turn(s["grads"][i].float(), cos, -sin, c)
            h = g * w
            dx.append((r * (h - unit * (h * unit).mean(-1, keepdim=True))).to(torch.bfloat16))
            dw.append((g * unit).double().sum((0, 1)).float())
    return (*out, *dx, *dw)


def _plain_pages(s, c):
    s["buf"].copy_(s["saved"])
    table, free, height, page = s["table"], s["free"], s["height"].long(), c["page"]
    B, width = table.shape
    pages = free.numel()
    old, new = s["old"].long()[:, None], s["new"].long()[:, None]
    e = torch.arange(width, device="cuda")
    n0, n1 = (old + page - 1) // page, (new + page - 1) // page
    hidden = torch.zeros(B, width, dtype=torch.bool, device="cuda")
    if c["window"] >= 0:
        hidden = ((e + 1) * page <= new - 1 - c["window"]) & (e * page >= c["sinks"])
    released = (e < n0) & (table >= 0) & (table < pages) & (hidden | (e >= n1))
    taken = (e >= n0) & (e < n1) & ~hidden
    back = released.flatten().long().cumsum(0)
    out = taken.flatten().long().cumsum(0)
    # the pages that come back on top of the stack; what is not one goes behind its end
    to = torch.where(released.flatten(), height + back - 1, torch.full_like(back, pages))
    stack = torch.cat((free, free.new_zeros(1))).scatter(0, to, table.flatten())
    top = height + back[-1]
    at = (top - out).view(B, width)
    got = torch.where(at >= 0, stack[at.clamp(0, pages)], torch.full_like(table, -1))
    table = torch.where(released, torch.full_like(table, -1), torch.where(taken, got, table))
    s["table"].copy_(table)
    free.copy_(stack[:pages])
    s["height"].copy_(torch.clamp(top - out[-1], min=0))
    # the new tokens
    cu = torch.cat((old.new_zeros(1), torch.clamp(new - old, min=0)[:, 0].cumsum(0)))
    i = torch.arange(s["T"], device="cuda")
    b = (cu[1:] <= i[:, None]).sum(1) if B <= 64 else torch.searchsorted(cu[1:], i, right=True)
    pos = old[b, 0] + i - cu[b]
    held = table[b, pos // page].long()
    slot = torch.where(held >= 0, held * page + pos % page, torch.full_like(held, -1))
    return s["table"], free, s["height"], cu.to(torch.int32), pos.to(torch.int32), slot


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        gen = torch.Generator(device="cuda").manual_seed(seed)
        return {"prompt": _exact_attention, "train": _exact_attention, "step": _exact_step,
                "rope": _exact_rope, "pages": _exact_pages}[case["op"]](case, seed, gen)
    finally:
        own = was


def _exact_attention(case, seed, gen):
    lens, D, Hkv, Hq = lengths(case), case["D"], case["Hkv"], case["Hq"]
    window, sinks, train = case["window"], case["sinks"], case["op"] == "train"
    n = sum(lens)
    q, k, v = (_randn(gen, n, h, D).double() for h in (Hq, Hkv, Hkv))
    do = _randn(gen, n, Hq, D).double() if train else None
    o = torch.empty(n, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.empty(Hq, n, dtype=torch.float64, device="cuda")
    grads = [torch.zeros_like(x) for x in (q, k, v)] if train else []
    start = 0
    for m in lens:
        for r0 in range(0, m, 768):
            r1 = min(m, r0 + 768)
            rows = torch.arange(r0, r1, device="cuda")
            cols = torch.arange(r1, device="cuda")
            cols = cols[(cols < sinks) | (cols + window >= r0)]
            gap = rows[:, None] - cols
            unseen = (gap < 0) | ((gap > window) & (cols >= sinks))
            for h in range(Hq):
                kv = h * Hkv // Hq
                qh, kh, vh = q[start + rows, h], k[start + cols, kv], v[start + cols, kv]
                logits = (torch.einsum("id,jd->ij", qh, kh) / math.sqrt(D)).masked_fill_(
                    unseen, -math.inf)
                z = torch.logsumexp(logits, 1)
                prob = logits.sub_(z[:, None]).exp_()
                out = torch.einsum("ij,jd->id", prob, vh)
                o[start + rows, h], lse[h, start + rows] = out, z
                if train:
                    g = do[start + rows, h]
                    grads[2][start + cols, kv] += torch.einsum("ij,id->jd", prob, g)
                    dlog = torch.einsum("id,jd->ij", g, vh).sub_((g * out).sum(1)[:, None])
                    dlog.mul_(prob).div_(math.sqrt(D))
                    grads[0][start + rows, h] = torch.einsum("ij,jd->id", dlog, kh)
                    grads[1][start + cols, kv] += torch.einsum("ij,id->jd", dlog, qh)
        start += m
    return (o, lse, *grads)


def _stored(x):
    """The values a cache of 4-bit codes holds for x [..., D], from the definition."""
    d = x.double().reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    low, high = d.min(-1, keepdim=True)[0], d.max(-1, keepdim=True)[0]
    step = ((high - low) / 15.0).float().bfloat16().double()
    ratio = torch.where(step > 0, (d - low) / step.clamp_min(1e-300), torch.zeros_like(d))
    return (low + step * ratio.round().clamp(0.0, 15.0)).reshape(x.shape)


def _exact_step(case, seed, gen):
    lens, D, Hkv, Hq, B = lengths(case), case["D"], case["Hkv"], case["Hq"], case["B"]
    n = sum(lens)
    k, v = _keys(gen, n, Hkv, D), _randn(gen, n, Hkv, D)
    q = _randn(gen, B, Hq, D)
    w = None
    if case["weights"]:
        w = (torch.rand(B, Hkv, max(lens), generator=gen, device="cuda") ** 6).double()
    o = torch.empty(B, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.empty(B, Hq, dtype=torch.float64, device="cuda")
    start = 0
    for b, m in enumerate(lens):
        j = torch.arange(m, device="cuda")
        j = j[(j < case["sinks"]) | (j >= m - 1 - case["window"])]
        kb, vb = _stored(k[start + j]), _stored(v[start + j])
        logits = torch.einsum("hgd,jhd->hgj", q[b].double().view(Hkv, -1, D), kb) / math.sqrt(D)
        lse[b] = torch.logsumexp(logits, -1).view(Hq)
        prob = torch.softmax(logits, -1)
        o[b] = torch.einsum("hgj,jhd->hgd", prob, vb).reshape(Hq, D)
        if w is not None:
            w[b, :, m:] = 0
            w[b][:, j] += prob.sum(1)
        start += m
    return (o, lse) if w is None else (o, lse, w)


def _exact_rope(case, seed, gen):
    q, k, qw, kw, grads = _projections(case, gen)
    rot, half = case["rot"], case["rot"] // 2
    cos, sin = (x[_i32(positions(case)).long()] for x in _angles(case, torch.float64))
    if case["interleaved"]:
        first = torch.arange(0, rot, 2, device="cuda")
        second = first + 1
    else:
        first = torch.arange(half, device="cuda")
        second = first + half
    out, dx, dw = [], [], []
    for i, (x, w) in enumerate(((q, qw), (k, kw))):
        x, w = x.double(), w.double()
        size = (x.square().sum(-1) / case["D"] + EPS).sqrt()
        u = torch.einsum("thd,th->thd", x, 1 / size)
        y = u * w
        a, b = y[..., first], y[..., second]
        z = y.clone()
        z[..., first] = torch.einsum("thd,td->thd", a, cos) - torch.einsum("thd,td->thd", b, sin)
        z[..., second] = torch.einsum("thd,td->thd", a, sin) + torch.einsum("thd,td->thd", b, cos)
        out.append(z)
        if case["train"]:
            g = grads[i].double()
            a, b = g[..., first], g[..., second]
            t = g.clone()
            t[..., first] = torch.einsum("thd,td->thd", a, cos) + torch.einsum("thd,td->thd", b, sin)
            t[..., second] = torch.einsum("thd,td->thd", b, cos) - torch.einsum("thd,td->thd", a, sin)
            dw.append(torch.einsum("thd,thd->d", t, u))
            t = t * w
            along = torch.einsum("thd,thd->th", t, u) / case["D"]
            dx.append((t - u * along[..., None]) / size[..., None])
    return (*out, *dx, *dw)


def _exact_pages(case, seed, gen):
    buf, old, new, width, pages = _pool(case, gen)
    old, new, page = old.tolist(), new.tolist(), case["page"]
    flat = buf.tolist()
    B = case["B"]
    table = [flat[b * width:(b + 1) * width] for b in range(B)]
    stack, height = flat[B * width:B * width + pages], flat[-1]
    wanted, cu, pos, slot = [], [0], [], []
    for b in range(B):
        had, has = -(-old[b] // page), -(-new[b] // page)
        for e in range(max(had, has)):
            out_of_sight = (case["window"] >= 0 and e * page >= case["sinks"]
                            and e * page + page - 1 < new[b] - 1 - case["window"])
            if e >= had:
                if not out_of_sight:
                    wanted.append((b, e))
            elif (out_of_sight or e >= has) and 0 <= table[b][e] < pages:
                stack[height] = table[b][e]
                height += 1
                table[b][e] = -1
    for b, e in wanted:
        height -= 1
        table[b][e] = stack[height] if height >= 0 else -1
    for b in range(B):
        for i in range(old[b], new[b]):
            p = table[b][i // page]
            pos.append(i)
            slot.append(p * page + i % page if p >= 0 else -1)
        cu.append(len(pos))
    return (_i32(table), _i32(stack), _i32([max(height, 0)]), _i32(cu), _i32(pos),
            torch.tensor(slot, dtype=torch.int64, device="cuda"))
