"""What the second set of operators is measured on: cases, inputs, plain forms.

Around the attention of packed sequences and of a paged cache:

  axes    queries and keys rotated by positions with several axes (time, height, width), either
          way round;
  slots   new keys and values into the cache rows that a slot map names, keys and queries rotated
          by such positions on the way;
  pages   block table, slot map and positions of one step from the requests' lengths and the
          list of free pages;
  prompt  attention of packed sequences (forward) whose scores are capped by a tanh, get a
          bias that grows with distance, or see a whole prefix of their sequence;
  train   the same with its gradients: output, log-sum-exp, dQ, dK, dV;
  paged   the same for the newest tokens of each sequence over its paged cache.

With s_ij = scale * q_i . k_j a capped score is cap * tanh(s_ij / cap), and a head's bias is
-slope * |i - j|, added behind the cap. Position i of a sequence sees the positions j that it
holds with j <= i or j < prefix. With ``own`` false ``run`` computes the plain form, in elementary
torch operations; with ``own`` true it calls this repository's package.
"""
import math
import random

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_THETA = 1e6
_ATTENTION = ("prompt", "train", "paged")


# ---- cases -----------------------------------------------------------------------------------

def _lengths(lo, hi, count, order, spread):
    """`count` lengths between lo and hi: "even" (uniform), "log" (uniform in the
    logarithm) or "mix" (four of five from the lowest eighth of the range, as batches
    of mostly short and some long samples have them)."""
    rng = random.Random(order)
    out = []
    for _ in range(count):
        if spread == "log":
            n = round(lo * (hi / lo) ** rng.random())
        elif spread == "mix" and rng.random() < 0.8:
            n = rng.randint(lo, lo + (hi - lo) // 8)
        else:
            n = rng.randint(lo, hi)
        out.append(min(hi, max(lo, n)))
    return out


def _new(case):
    """New tokens of each sequence. Over a cache the first `chunks` take `chunk` tokens each,
    the others one; a page step leaves every eleventh sequence out."""
    if case["kind"] in ("prompt", "train", "axes"):
        return _lengths(case["lo"], case["hi"], case["seqs"], case["order"], case["spread"])
    new = [case["chunk"] if s < case["chunks"] else 1 for s in range(case["seqs"])]
    if case["kind"] == "pages":
        new = [0 if s % 11 == 10 else n for s, n in enumerate(new)]
    return new


def _before(case):
    """Tokens that each sequence held before the new ones."""
    if case["kind"] in ("prompt", "train", "axes"):
        return [0] * case["seqs"]
    return _lengths(case["lo"], case["hi"], case["seqs"], case["order"], case["spread"])


def _held(case):
    """Tokens that each sequence holds with the new ones."""
    return [b + n for b, n in zip(_before(case), _new(case))]


def _prefixes(case):
    """Of each sequence the prefix that all of it sees: about the given percentage of what it
    holds, none for every fifth sequence."""
    rng = random.Random(case["order"] + 1)
    return [0 if s % 5 == 4 else min(m, round(m * case["prefix"] / 100 * (0.5 + rng.random())))
            for s, m in enumerate(_held(case))]


def _axes(name, dtype, heads, kv_heads, size, seqs, lo, hi, spread, sections, layout, direction, order=1):
    return dict(name=name, kind="axes", dtype=dtype, Hq=heads, Hkv=kv_heads, D=size, seqs=seqs, lo=lo, hi=hi,
                spread=spread, sections=sections, layout=layout, direction=direction, order=order)


def _slots(name, dtype, heads, kv_heads, size, seqs, lo, hi, spread, sections, layout, chunks, chunk, page, order=1):
    return dict(_axes(name, dtype, heads, kv_heads, size, seqs, lo, hi, spread, sections, layout, 1, order),
                kind="slots", chunks=chunks, chunk=chunk, page=page)


def _pages(name, seqs, lo, hi, spread, chunks, chunk, page, short, order=1):
    return dict(name=name, kind="pages", seqs=seqs, lo=lo, hi=hi, spread=spread, chunks=chunks, chunk=chunk,
                page=page, short=short, order=order)


def _attn(name, kind, dtype, heads, kv_heads, size, seqs, lo, hi, spread, cap, slopes, prefix, order=1,
          chunks=0, chunk=1, page=0):
    return dict(name=name, kind=kind, dtype=dtype, Hq=heads, Hkv=kv_heads, D=size, seqs=seqs, lo=lo, hi=hi,
                spread=spread, cap=cap, slopes=slopes, prefix=prefix, order=order, chunks=chunks, chunk=chunk,
                page=page)


def listed():
    return [
        # a tiny packed batch of text and images: latency alone
        _axes("axes_tiny", "f32", 4, 2, 16, 3, 3, 39, "even", "4+2+2", "sections", 1),
        # a packed batch of text with images in it, 32 + 8 heads of 128
        _axes("axes_packed", "bf16", 32, 8, 128, 22, 32, 4096, "mix", "24+20+20", "interleaved", 1),
        # gradients of an image encoder's patches: height and width, a ladder of frequencies each
        _axes("axes_patches", "f16", 16, 16, 80, 9, 500, 1500, "even", "20+20", "separate", -1),
        # one decode step of a serving batch
        _slots("slots_decode", "bf16", 32, 8, 128, 64, 100, 8000, "log", "16+24+24", "sections", 0, 1, 16),
        # prompts with images going into the cache
        _slots("slots_prompt", "bf16", 32, 8, 128, 4, 1, 1000, "log", "24+20+20", "interleaved", 4, 4001, 64),
        # one decode step's block table and slot map, a batch of 64
        _pages("pages_decode", 64, 100, 8000, "log", 0, 1, 16, 0),
        # a long queue: prompts of 1100 tokens for some, one token for the others, too few free pages
        _pages("pages_queue", 4000, 1, 6000, "log", 300, 1100, 64, 1),
        # a packed training batch of eight samples, capped scores, 32 + 8 heads of 128
        _attn("train_capped", "train", "bf16", 32, 8, 128, 8, 256, 2048, "even", 50.0, 0, 0),
        # short ragged samples with a bias by distance, head size and group that are no power of two
        _attn("train_biased", "train", "f16", 6, 2, 80, 61, 1, 301, "log", 0.0, 1, 0),
        # images and questions that are seen as a whole, answers causal
        _attn("prompt_prefix", "prompt", "bf16", 32, 8, 128, 16, 300, 4096, "even", 0.0, 0, 60),
        # a decode step of a serving batch with contexts of 512 to 16384 tokens, capped scores
        _attn("paged_capped", "paged", "bf16", 32, 8, 128, 64, 512, 16384, "log", 30.0, 0, 0, 1, 0, 1, 16),
        # chunks of long prompts among decoding sequences, a bias by distance and a prefix
        _attn("paged_chunk", "paged", "f16", 16, 4, 64, 24, 33, 9001, "log", 0.0, 1, 30, 1, 4, 1025, 48),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(lo * (hi / lo) ** rng.random())))


def _split(rng, half):
    """Sections of `half` frequencies and a layout that takes them."""
    layout = rng.choice(["sections", "sections", "interleaved", "separate"])
    axes = rng.choice([2, 3, 3]) if half >= 6 else 2
    if layout == "interleaved":  # the first axis keeps what the turns of the others leave
        each = half // axes
        rest = [rng.randint(max(1, each // 2), each) for _ in range(axes - 1)]
        return "+".join(str(n) for n in [half - sum(rest)] + rest), layout
    cuts = sorted(rng.sample(range(1, half), axes - 1))
    return "+".join(str(b - a) for a, b in zip([0] + cuts, cuts + [half])), layout


def draw(rng):
    kind = rng.choice(["axes", "slots", "pages", "prompt", "train", "train", "paged"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    size = rng.choice([16, 32, 40, 64, 64, 72, 80, 96, 112, 128, 128, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 5, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8])
    order = rng.randrange(1 << 30)
    spread = rng.choice(["even", "log", "mix"])
    page = rng.choice([8, 16, 16, 32, 48, 64, 128, 256])
    if kind == "axes":
        dtype = rng.choice([dtype, dtype, "f32"])
        seqs, hi = _log(rng, 1, 64), _log(rng, 2, 8192)
        while seqs * hi * (heads + kv_heads) * size > (1 << 27):
            seqs, hi = max(1, seqs // 2), max(2, hi * 3 // 4)
        sections, layout = _split(rng, size // 2)
        return _axes("", dtype, heads, kv_heads, size, seqs, _log(rng, 1, hi), hi, spread, sections, layout,
                     rng.choice([1, -1]), order)
    if kind == "pages":
        seqs, hi, chunk = _log(rng, 1, 4000), _log(rng, 2, 16384), _log(rng, 1, 2048)
        chunks = rng.choice([0, rng.randint(0, seqs), seqs])
        while chunks * chunk > 300000:
            chunks = chunks // 2
        return _pages("", seqs, _log(rng, 1, hi), hi, spread, chunks, chunk, max(page, 16), rng.choice([0, 0, 1]), order)
    cap = rng.choice([0.0, 30.0, 50.0, round(2.0 ** rng.uniform(2, 8), 2)])
    slopes = rng.choice([0, 1])
    prefix = rng.choice([0, 0, rng.randint(1, 100)])
    if cap == 0.0 and slopes == 0 and prefix == 0:
        cap = 20.0
    if kind in ("prompt", "train"):
        seqs, hi = _log(rng, 1, 64), _log(rng, 2, 8192)
        lo = _log(rng, 1, hi)
        # the plain form's scores stay below those of the largest listed cases
        most = 1 << 30
        while seqs * heads * hi * hi > most:
            seqs, hi = max(1, seqs // 2), max(2, hi * 3 // 4)
        return _attn("", kind, dtype, heads, kv_heads, size, seqs, min(lo, hi), hi, spread, cap, slopes, prefix, order)
    seqs, hi = _log(rng, 1, 128), _log(rng, 2, 16384)
    lo = _log(rng, 1, hi)
    chunk = _log(rng, 1, 2048)
    chunks = rng.choice([0, rng.randint(0, seqs), seqs])
    if kind == "slots":
        dtype = rng.choice([dtype, "f32"])
        while seqs * heads * chunk * size > (1 << 26):
            seqs, chunk = max(1, seqs // 2), max(1, chunk * 3 // 4)
    while kind == "paged" and seqs * heads * (chunk if chunks else 1) * (hi + chunk) > (1 << 30):
        seqs, chunk, hi = max(1, seqs * 3 // 4), max(1, chunk * 3 // 4), max(2, hi * 3 // 4)
    while seqs * (hi + chunk) * kv_heads * size > (1 << 29):
        seqs, hi = max(1, seqs // 2), max(2, hi * 3 // 4)
    if kind == "slots":
        sections, layout = _split(rng, size // 2)
        return _slots("", dtype, heads, kv_heads, size, seqs, min(lo, hi), hi, spread, sections, layout,
                      min(chunks, seqs), chunk, page, order)
    return _attn("", kind, dtype, heads, kv_heads, size, seqs, min(lo, hi), hi, spread, cap, slopes, prefix, order,
                 min(chunks, seqs), chunk, page)


# ---- inputs ----------------------------------------------------------------------------------

def _grid(length, axes, rng):
    """Positions [axes, length] of one sequence: runs of text, whose axes go on together, and
    images of rows x columns, whose first axis stands still; with two axes images alone."""
    out = np.empty((axes, length), dtype=np.int32)
    at, pos = 0, 0
    while at < length:
        if axes >= 3 and rng.random() < 0.5:
            n = min(length - at, rng.randint(1, 200))
            out[:, at:at + n] = pos + np.arange(n)
            at, pos = at + n, pos + n
            continue
        rows, cols = rng.randint(1, 40), rng.randint(1, 40)
        n = min(length - at, rows * cols)
        cell = np.arange(n)
        base = 0 if axes == 2 else pos
        out[:, at:at + n] = base
        out[-2, at:at + n] = base + cell // cols
        out[-1, at:at + n] = base + cell % cols
        at, pos = at + n, pos + max(rows, cols)
    return out


def _positions(case, before, new, seed):
    axes = case["sections"].count("+") + 1
    rng = random.Random(seed)
    parts = []
    for b, n in zip(before, new):
        if case["kind"] == "slots" and n == 1:  # an answer's token: its axes go on together
            parts.append(np.full((axes, 1), max(1, b - rng.randint(0, b // 2 + 1)), dtype=np.int32))
        else:
            parts.append(_grid(n, axes, rng) + (b if axes >= 3 else 0))
    return np.concatenate(parts, 1)


def _running(values, dev):
    out = [0]
    for n in values:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    if case["kind"] == "pages":
        return _prepare_pages(case, dev, gen)
    dtype, kind = _TYPES[case["dtype"]], case["kind"]
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    new, held = _new(case), _held(case)
    T, B = sum(new), len(new)

    def normal(*shape, size=1.0):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).mul_(size).to(dtype)

    state = dict(case=case, dtype=dtype, scale=D ** -0.5, most_new=max(new), most_held=max(held),
                 cu=_running(new, dev), held=torch.tensor(held, dtype=torch.int32, device=dev))
    if kind in ("axes", "slots"):
        state["sections"] = tuple(int(n) for n in case["sections"].split("+"))
        state["positions"] = torch.from_numpy(_positions(case, _before(case), new, seed)).to(dev)
    # scores under a cap are some times larger than they come from new weights
    wide = 4.0 if kind in _ATTENTION and case["cap"] else 1.0
    if kind == "paged":
        state["q"] = normal(T, Hq, D, size=wide)
    elif kind == "axes" and case["direction"] < 0:  # gradients come as two tensors
        state.update(q=normal(T, Hq, D), k=normal(T, Hkv, D))
    else:
        # the three parts of one fused projection
        qkv = normal(T, Hq + 2 * Hkv, D)
        if wide != 1.0:
            qkv[:, :Hq] *= wide
        state.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:])
    if kind == "train":
        state["dout"] = normal(T, Hq, D)
    if kind in ("slots", "paged"):
        page = case["page"]
        per = -(-max(held) // page)
        used = [-(-m // page) for m in held]
        pages = sum(used) + 3
        # pages in the order in which a pool that has been in use hands them out
        order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
        table = torch.full((B, per), -1, dtype=torch.int32, device=dev)
        at = 0
        for s, n in enumerate(used):
            table[s, :n] = order[at:at + n]
            at += n
        state.update(k_cache=normal(pages, page, Hkv, D), v_cache=normal(pages, page, Hkv, D), table=table)
    if kind == "slots":
        seq, _, pos = _places(state, T)
        state["slots"] = state["table"].long()[seq, pos // page] * page + pos % page
    if kind in _ATTENTION:
        state["slopes"] = state["prefixes"] = None
        if case["slopes"]:  # falling from head to head, as a geometric series
            state["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], dtype=torch.float32,
                                           device=dev)
        if case["prefix"]:
            state["prefixes"] = torch.tensor(_prefixes(case), dtype=torch.int32, device=dev)
        if own:
            # a batch's plan is made once and serves every layer of the model
            import packed_varlen_rotary_rope_amd as rope
            if kind == "paged":
                state["plan"] = rope.paged_plan(state["cu"], state["held"], T, Hq, Hkv,
                                                prefix_lens=state["prefixes"])
            else:
                state["plan"] = rope.attn_plan(state["cu"], T, Hq, Hkv, prefix_lens=state["prefixes"])
    return state


def _prepare_pages(case, dev, gen):
    page, new, before = case["page"], _new(case), _before(case)
    has = [-(-b // page) for b in before]
    wants = [-(-(b + n) // page) - h for b, n, h in zip(before, new, has)]
    per = max(h + w for h, w in zip(has, wants)) + 1
    free = sum(wants) * 3 // 4 if case["short"] else sum(wants) + 5
    total = sum(has) + free
    order = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
    # each sequence's pages in a row of the table, the free ones in a ring that has turned
    count = torch.tensor(has, device=dev)
    table = torch.full((len(new), per), -1, dtype=torch.int32, device=dev)
    table[torch.arange(per, device=dev) < count[:, None]] = order[:sum(has)]
    first = int(torch.randint(total, (1,), generator=gen, device=dev))
    ring = torch.full((total,), -1, dtype=torch.int32, device=dev)
    ring[(first + torch.arange(free, device=dev)) % total] = order[sum(has):]
    int32 = dict(dtype=torch.int32, device=dev)
    state = dict(case=case, T=sum(new), table=table, ring=ring, ring_state=torch.tensor([first, free], **int32),
                 new=torch.tensor(new, **int32), before=torch.tensor(before, **int32))
    if own:
        import packed_varlen_rotary_rope_amd as rope
        state["pool"] = rope.PagePool(ring, state["ring_state"])
    return state


# ---- one pass --------------------------------------------------------------------------------

def run(state):
    kind = state["case"]["kind"]
    if own:
        return _own(kind, state)
    if kind == "pages":
        return _plain_pages(state)
    if kind == "axes":
        turned = _plain_rotation(state)
        return {"q": turned(state["q"]), "k": turned(state["k"])}
    if kind == "slots":
        return _plain_slots(state)
    return _plain_attention(kind, state)


def _own(kind, s):
    import packed_varlen_rotary_rope_amd as rope
    case = s["case"]
    if kind == "pages":
        step = rope.page_step(s["pool"], s["table"], s["before"], s["new"], s["T"], case["page"])
        return {"table": s["table"], "cu": step.cu_seqlens, "kv_lens": step.kv_lens, "held": step.held,
                "positions": step.positions, "slots": step.slots, "ring_state": step.state}
    if kind == "axes":
        q, k = rope.qk_apply_axes(s["q"], s["k"], s["positions"], s["sections"], _THETA, case["direction"],
                                  layout=case["layout"])
        return {"q": q, "k": k}
    if kind == "slots":
        q = rope.kv_append_slots_(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], s["positions"], _THETA,
                                  sections=s["sections"], layout=case["layout"], q=s["q"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    more = dict(softcap=case["cap"] or None, slopes=s["slopes"])
    if kind == "paged":
        out, lse = rope.attn_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["plan"], s["scale"], **more)
        return {"out": out, "lse": lse}
    out, lse = rope.attn_fwd(s["q"], s["k"], s["v"], s["plan"], s["scale"], **more)
    if kind == "prompt":
        return {"out": out, "lse": lse}
    dq, dk, dv = rope.attn_bwd(s["dout"], s["q"], s["k"], s["v"], out, lse, s["plan"], s["scale"], **more)
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def _places(s, T):
    """Of each packed token its sequence, its number among the sequence's new tokens
    and its position."""
    cu = s["cu"].long()
    t = torch.arange(T, device=cu.device)
    seq = torch.searchsorted(cu, t, right=True) - 1
    row = t - cu[seq]
    return seq, row, s["held"].long()[seq] - (cu[1:] - cu[:-1])[seq] + row


def _ladder(sections, layout):
    """Of each frequency its axis, its number and the size of its ladder."""
    half, axes = sum(sections), len(sections)
    if layout == "interleaved":
        axis = [j % axes if j < axes * sections[j % axes] else 0 for j in range(half)]
        return axis, list(range(half)), [half] * half
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    if layout == "sections":
        return axis, list(range(half)), [half] * half
    return axis, [j for n in sections for j in range(n)], [n for n in sections for _ in range(n)]


def _plain_rotation(s):
    axis, number, size = _ladder(s["sections"], s["case"]["layout"])
    dev = s["q"].device
    # angles are single-precision products of the position and the frequency
    number, size = (torch.tensor(x, dtype=torch.float64, device=dev) for x in (number, size))
    freq = (_THETA ** (-number / size)).float()
    angle = (s["positions"][torch.tensor(axis, device=dev)].float().t() * freq).double()[:, None]
    cos, sin = angle.cos().float(), (angle.sin() * s["case"]["direction"]).float()

    def turned(x):
        a, b = x.float().chunk(2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(s["dtype"])

    return turned


def _plain_slots(s):
    turned = _plain_rotation(s)
    page = s["case"]["page"]
    where = s["slots"] // page, s["slots"] % page
    s["k_cache"][where] = turned(s["k"])
    s["v_cache"][where] = s["v"]
    return {"q": turned(s["q"]), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_pages(s):
    page, T, table, ring = s["case"]["page"], s["T"], s["table"], s["ring"]
    dev, N = table.device, ring.numel()
    new, before = s["new"].long(), s["before"].long()
    first, count = s["ring_state"].long()
    has = (before + page - 1) // page
    wants = (before + new + page - 1) // page - has
    upto = wants.cumsum(0)
    served = (wants == 0) | (upto <= count)
    wants = torch.where(served, wants, 0)
    place = upto - wants
    # the new entries of the table
    entry = torch.arange(table.shape[1], device=dev) - has[:, None]
    fresh = ring[(first + place[:, None] + entry.clamp_min(0)) % N]
    table.copy_(torch.where((entry >= 0) & (entry < wants[:, None]), fresh, table))
    cu = torch.zeros(new.numel() + 1, dtype=torch.int32, device=dev)
    cu[1:] = new.cumsum(0)
    t = torch.arange(T, device=dev)
    seq = torch.searchsorted(cu.long(), t, right=True) - 1
    pos = before[seq] + t - cu.long()[seq]
    slot = table.long()[seq, (pos // page).clamp_max(table.shape[1] - 1)] * page + pos % page
    on = served[seq]
    used = wants.sum()
    return {"table": table, "cu": cu, "kv_lens": torch.where(served, before + new, 0).int(),
            "held": torch.where(served, before + new, before).int(), "positions": torch.where(on, pos, -1).int(),
            "slots": torch.where(on, slot, -1), "ring_state": torch.stack([(first + used) % N, count - used]).int()}


def _plain_attention(kind, s):
    case = s["case"]
    Hq, Hkv, D, B = case["Hq"], case["Hkv"], case["D"], case["seqs"]
    G, N, M = Hq // Hkv, s["most_new"], s["most_held"]
    seq, row, pos = _places(s, s["q"].shape[0])
    dev = seq.device

    def padded(x, heads):  # [T, heads, D] -> float [B, heads, N, D]
        full = torch.zeros((B, N, heads, D), dtype=torch.float32, device=dev)
        full[seq, row] = x.float()
        return full.transpose(1, 2)

    q = padded(s["q"], Hq).reshape(B, Hkv, G * N, D)
    if kind == "paged":
        table = s["table"].long().clamp_min(0)
        k = s["k_cache"][table].reshape(B, -1, Hkv, D)[:, :M].float().transpose(1, 2).contiguous()
        v = s["v_cache"][table].reshape(B, -1, Hkv, D)[:, :M].float().transpose(1, 2).contiguous()
    else:
        k, v = padded(s["k"], Hkv).contiguous(), padded(s["v"], Hkv).contiguous()
    at = torch.full((B, N), M, dtype=torch.int64, device=dev)  # rows of padding see every key
    at[seq, row] = pos
    last = at
    if s["prefixes"] is not None:
        last = torch.maximum(at, torch.minimum(s["prefixes"], s["held"]).long()[:, None] - 1)
    key = torch.arange(M, device=dev)
    seen = key <= last[:, :, None]
    p = torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(s["scale"])
    slope = None
    if case["cap"]:
        p.div_(case["cap"]).tanh_()
        if kind == "train":
            slope = 1 - p * p
        p.mul_(case["cap"])
    p = p.view(B, Hkv, G, N, M)
    if s["slopes"] is not None:
        p.sub_(s["slopes"].view(1, Hkv, G, 1, 1) * (at[:, :, None] - key).abs().float()[:, None, None])
    p = p.masked_fill_(~seen[:, None, None], float("-inf")).view(B, Hkv, G * N, M)
    top = p.amax(-1, keepdim=True)
    p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(total)
    lse = (top + total.log()).view(B, Hq, N)
    o = torch.matmul(p, v)

    def packed(x, heads):  # float [B, heads, N, D] -> [T, heads, D]
        return x.reshape(B, heads, N, D)[seq, :, row].to(s["dtype"])

    out = {"out": packed(o, Hq), "lse": lse[seq, :, row]}
    if kind == "train":
        do = padded(s["dout"], Hq).reshape(B, Hkv, G * N, D)
        dv = torch.matmul(p.transpose(-1, -2).contiguous(), do)
        ds = torch.matmul(do, v.transpose(-1, -2).contiguous())
        ds.sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(s["scale"])
        if slope is not None:
            ds.mul_(slope)
        dq = torch.matmul(ds, k)
        dk = torch.matmul(ds.transpose(-1, -2).contiguous(), q)
        out.update(dq=packed(dq, Hq), dk=packed(dk, Hkv), dv=packed(dv, Hkv))
    return out


# ---- what a pass cannot do without -----------------------------------------------------------

def work(case):
    new, held = _new(case), _held(case)
    T, M = sum(new), sum(held)
    if case["kind"] == "pages":
        fresh = sum(-(-m // case["page"]) - -(-(m - n) // case["page"]) for m, n in zip(held, new))
        # lengths in and out, free pages read and written to the table, positions and slots out
        return {"bytes": 4 * 5 * case["seqs"] + 2 * 4 * fresh + 12 * T, "flops": 8 * T}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    size = 4 if case["dtype"] == "f32" else 2
    rows = T * Hq * D * size
    if case["kind"] in ("axes", "slots"):
        where = 4 * T * (case["sections"].count("+") + 1)
        keys = T * Hkv * D * size
        if case["kind"] == "slots":
            return {"bytes": 2 * rows + 4 * keys + where + 8 * T, "flops": 3 * T * (Hq + Hkv) * D}
        return {"bytes": 2 * rows + 2 * keys + where, "flops": 3 * T * (Hq + Hkv) * D}
    prefixes = _prefixes(case) if case["prefix"] else [0] * len(new)
    # pairs of a query token and a key that it sees; below the prefix all of it is seen
    pairs = 0
    for n, m, pre in zip(new, held, prefixes):
        pairs += n * (m - n) + n * (n + 1) // 2
        short = max(0, min(pre - (m - n), n))  # new tokens inside of the prefix
        pairs += short * (short - 1) // 2
    keys = (M if case["kind"] == "paged" else T) * Hkv * D * size
    forward = {"bytes": 2 * rows + 2 * keys + 4 * T * Hq, "flops": 4 * pairs * Hq * D}
    if case["kind"] != "train":
        return forward
    # the step as a whole: q, k, v, dout in; out, lse, dq, dk, dv out
    return {"bytes": 4 * rows + 4 * keys + 4 * T * Hq, "flops": 14 * pairs * Hq * D}


# ---- the definitions in 64 bits --------------------------------------------------------------

def exact(case, seed):
    if case["kind"] == "pages":
        return _exact_pages(case, prepare(case, seed))
    if case["kind"] in ("axes", "slots"):
        return _exact_rotation(case, prepare(case, seed))
    if work(case)["flops"] > 1e13:
        return None
    return _exact_attention(case, prepare(case, seed))


def _exact_attention(case, s):
    """Sequence by sequence and head by head."""
    new, held = _new(case), _held(case)
    prefixes = _prefixes(case) if case["prefix"] else [0] * len(new)
    Hq, Hkv = case["Hq"], case["Hkv"]
    G, dev = Hq // Hkv, s["q"].device
    q = s["q"].double()
    out = torch.zeros(q.shape, dtype=torch.float64, device=dev)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=dev)
    grads = {}
    if case["kind"] == "train":
        do = s["dout"].double()
        grads = {"dq": torch.zeros_like(q), "dk": torch.zeros_like(s["k"], dtype=torch.float64),
                 "dv": torch.zeros_like(s["v"], dtype=torch.float64)}
    t0 = 0
    for b, (n, m) in enumerate(zip(new, held)):
        t1 = t0 + n
        j = torch.arange(m, device=dev)
        if case["kind"] == "paged":
            page = s["table"][b].long()[j // case["page"]]
            k, v = s["k_cache"][page, j % case["page"]], s["v_cache"][page, j % case["page"]]
        else:
            k, v = s["k"][t0:t1], s["v"][t0:t1]
        i = torch.arange(m - n, m, device=dev)[:, None]
        hidden = (j[None] > i) & (j[None] >= prefixes[b])
        far = (i - j[None]).abs().double()
        for h in range(Hq):
            kh, vh = k[:, h // G].double(), v[:, h // G].double()
            score = (q[t0:t1, h] @ kh.T) * s["scale"]
            rise = 1.0
            if case["cap"]:
                bent = torch.tanh(score / case["cap"])
                score, rise = case["cap"] * bent, 1 - bent ** 2
            if case["slopes"]:
                score = score - s["slopes"][h].double() * far
            score = score.masked_fill(hidden, -math.inf)
            lse[t0:t1, h] = torch.logsumexp(score, -1)
            p = torch.exp(score - lse[t0:t1, h, None])
            out[t0:t1, h] = p @ vh
            if grads:
                dp = do[t0:t1, h] @ vh.T
                ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * rise * s["scale"]
                grads["dv"][t0:t1, h // G] += p.T @ do[t0:t1, h]
                grads["dq"][t0:t1, h] = ds @ kh
                grads["dk"][t0:t1, h // G] += ds.T @ q[t0:t1, h]
        t0 = t1
    return {"out": out, "lse": lse, **grads}


def _exact_rotation(case, s):
    """Axis by axis of every section."""
    D, half, dev = case["D"], case["D"] // 2, s["q"].device
    axes = len(s["sections"])
    angle = torch.zeros((s["q"].shape[0], half), dtype=torch.float32, device=dev)
    begin = 0
    for a, n in enumerate(s["sections"]):
        if case["layout"] == "interleaved":
            if a == 0:  # what the others leave
                taken = {b + axes * i for b in range(1, axes) for i in range(s["sections"][b])}
                mine = [j for j in range(half) if j not in taken]
            else:
                mine = [a + axes * i for i in range(n)]
        else:
            mine = list(range(begin, begin + n))
        for at, j in enumerate(mine):
            # the frequencies and angles are rounded to single precision by definition
            power = -at / n if case["layout"] == "separate" else -2.0 * j / D
            freq = torch.tensor(_THETA ** power, dtype=torch.float64).to(torch.float32).to(dev)
            angle[:, j] = s["positions"][a].to(torch.float32) * freq
        begin += n
    c, z = angle.double().cos()[:, None], case["direction"] * angle.double().sin()[:, None]

    def turn(x):
        x = x.double()
        y = torch.empty_like(x)
        y[..., :half] = x[..., :half] * c - x[..., half:] * z
        y[..., half:] = x[..., half:] * c + x[..., :half] * z
        return y

    if case["kind"] == "axes":
        return {"q": turn(s["q"]), "k": turn(s["k"])}
    caches = {}
    for name, rows in (("k_cache", turn(s["k"])), ("v_cache", s["v"].double())):
        full = s[name].double()
        full.view(-1, *full.shape[2:])[s["slots"]] = rows
        caches[name] = full
    return {"q": turn(s["q"]), **caches}


def _exact_pages(case, s):
    """Request by request, on the host."""
    page = case["page"]
    table, ring = s["table"].cpu().numpy().copy(), s["ring"].cpu().numpy()
    first, count = (int(x) for x in s["ring_state"].cpu())
    cu, kv_lens, after, positions, slots = [0], [], [], [], []
    used, asked = 0, 0
    for b, (held, n) in enumerate(zip(_before(case), _new(case))):
        cu.append(cu[-1] + n)
        have = -(-held // page)
        need = -(-(held + n) // page) - have
        asked += need
        if need > 0 and asked > count:
            kv_lens.append(0)
            after.append(held)
            positions.extend([-1] * n)
            slots.extend([-1] * n)
            continue
        for x in range(need):
            table[b, have + x] = ring[(first + used) % len(ring)]
            used += 1
        kv_lens.append(held + n)
        after.append(held + n)
        for p in range(held, held + n):
            positions.append(p)
            slots.append(int(table[b, p // page]) * page + p % page)

    def whole(x, dtype=torch.int32):
        return torch.tensor(x, dtype=dtype, device=s["table"].device)

    return {"table": torch.from_numpy(table).to(s["table"].device), "cu": whole(cu), "kv_lens": whole(kv_lens),
            "held": whole(after), "positions": whole(positions), "slots": whole(slots, torch.int64),
            "ring_state": whole([(first + used) % len(ring), count - used])}
