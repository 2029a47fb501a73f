"""What the attention operators are measured on: cases, inputs, plain forms.

Four operators around one softmax attention with grouped heads (query head h reads
key/value head h // (Hq / Hkv)):

  prompt  causal attention over packed sequences of different lengths (forward);
  train   the same with its gradients: output, log-sum-exp, dQ, dK, dV;
  append  new keys and values written into a paged cache, keys rotated on the way,
          the new queries rotated with them;
  paged   attention of the newest tokens of each sequence (one, or a chunk) over the
          paged cache that holds all its tokens.

Token i of the n new tokens of a sequence that then holds m tokens sits at position
m - n + i, and sees the keys of the positions up to its own (for prompt and train
m = n). With ``own`` false ``run`` computes the plain form, in elementary torch
operations on a padded batch; with ``own`` true it calls this repository's package.
"""
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_THETA = 1e6


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
    """New tokens of each sequence: of a paged batch the first `chunks` take `chunk`
    tokens each and the others one."""
    if case["kind"] in ("prompt", "train"):
        return _lengths(case["lo"], case["hi"], case["seqs"], case["order"], case["spread"])
    return [case["chunk"] if s < case["chunks"] else 1 for s in range(case["seqs"])]


def _held(case):
    """Tokens that each sequence holds with the new ones."""
    new = _new(case)
    if case["kind"] in ("prompt", "train"):
        return new
    before = _lengths(case["lo"], case["hi"], case["seqs"], case["order"], case["spread"])
    return [b + n for b, n in zip(before, new)]


def _packed(name, kind, dtype, heads, kv_heads, size, seqs, lo, hi, spread, order=1):
    return dict(name=name, kind=kind, dtype=dtype, Hq=heads, Hkv=kv_heads, D=size, seqs=seqs,
                lo=lo, hi=hi, spread=spread, order=order)


def _cached(name, kind, dtype, heads, kv_heads, size, seqs, lo, hi, spread, chunks, chunk, page,
            order=1):
    return dict(_packed(name, kind, dtype, heads, kv_heads, size, seqs, lo, hi, spread, order),
                chunks=chunks, chunk=chunk, page=page)


def listed():
    return [
        # four short samples of the tiny packed batch's sizes: latency alone
        _packed("prompt_tiny", "prompt", "f16", 4, 2, 16, 4, 3, 39, "even"),
        # a packed batch of mostly short and some long samples, 32 + 8 heads of 128
        _packed("prompt_mixed", "prompt", "bf16", 32, 8, 128, 22, 32, 4096, "mix"),
        # one long document
        _packed("prompt_long", "prompt", "bf16", 32, 8, 128, 1, 16384, 16384, "even"),
        # a packed training batch of eight samples of 256 to 2048 tokens
        _packed("train_packed", "train", "bf16", 32, 8, 128, 8, 256, 2048, "even"),
        # short ragged samples, head size and head group that are no power of two
        _packed("train_ragged", "train", "f16", 6, 2, 80, 61, 1, 301, "log"),
        # one long sample, 64-wide heads in large groups
        _packed("train_long", "train", "bf16", 16, 2, 64, 1, 8192, 8192, "even"),
        # one decode step of a serving batch: one token each
        _cached("append_decode", "append", "bf16", 32, 8, 128, 64, 100, 8000, "log", 0, 1, 16),
        # prompts of four sequences going into the cache
        _cached("append_prompt", "append", "bf16", 32, 8, 128, 4, 1, 1000, "log", 4, 4001, 64),
        # a single user's decode step
        _cached("paged_single", "paged", "bf16", 32, 8, 128, 1, 4099, 4099, "even", 0, 1, 16),
        # a decode step of a serving batch with contexts of 512 to 16384 tokens
        _cached("paged_decode", "paged", "bf16", 32, 8, 128, 64, 512, 16384, "log", 0, 1, 16),
        # chunks of long prompts over what is cached of them
        _cached("paged_chunk", "paged", "bf16", 32, 8, 128, 4, 8000, 24000, "even", 4, 1024, 64),
        # two prompt chunks among decoding sequences, 64-wide heads, pages of no power of two
        _cached("paged_mixed", "paged", "f16", 64, 8, 64, 16, 33, 7001, "log", 2, 257, 48),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    kind = rng.choice(["prompt", "train", "append", "paged"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    size = rng.choice([16, 32, 40, 64, 64, 72, 80, 96, 112, 128, 128, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 5, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8])
    order = rng.randrange(1 << 30)
    spread = rng.choice(["even", "log", "mix"])
    if kind in ("prompt", "train"):
        seqs, hi = _log(rng, 1, 64), _log(rng, 2, 8192)
        lo = _log(rng, 1, hi)
        # the plain form's scores stay below those of the largest listed cases
        most = (1 << 31) if kind == "prompt" else (1 << 29)
        while seqs * heads * hi * hi > most:
            seqs, hi = max(1, seqs // 2), max(2, hi * 3 // 4)
        return _packed("", kind, dtype, heads, kv_heads, size, seqs, min(lo, hi), hi, spread, order)
    seqs, hi = _log(rng, 1, 128), _log(rng, 2, 16384)
    lo = _log(rng, 1, hi)
    page = rng.choice([8, 16, 16, 32, 48, 64, 128, 256])
    chunk = _log(rng, 1, 2048)
    chunks = rng.choice([0, rng.randint(0, seqs), seqs])
    if kind == "append":
        dtype = rng.choice([dtype, "f32"])
        while seqs * heads * chunk * size > (1 << 26):
            seqs, chunk = max(1, seqs // 2), max(1, chunk * 3 // 4)
    while kind == "paged" and seqs * heads * (chunk if chunks else 1) * (hi + chunk) > (1 << 31):
        seqs, chunk, hi = max(1, seqs * 3 // 4), max(1, chunk * 3 // 4), max(2, hi * 3 // 4)
    while seqs * (hi + chunk) * kv_heads * size > (1 << 29):
        seqs, hi = max(1, seqs // 2), max(2, hi * 3 // 4)
    return _cached("", kind, dtype, heads, kv_heads, size, seqs, min(lo, hi), hi, spread,
                   min(chunks, seqs), chunk, page, order)


def prepare(case, seed):
    dev, dtype = torch.device("cuda"), _TYPES[case["dtype"]]
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    new, held = _new(case), _held(case)
    T, B = sum(new), len(new)
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)

    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    state = dict(case=case, dtype=dtype, scale=D ** -0.5, most_new=max(new), most_held=max(held),
                 cu=torch.tensor(starts, dtype=torch.int32, device=dev),
                 held=torch.tensor(held, dtype=torch.int32, device=dev))
    if case["kind"] in ("prompt", "train", "append"):
        # the three parts of one fused projection
        qkv = normal(T, Hq + 2 * Hkv, D)
        state.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:])
    else:
        state["q"] = normal(T, Hq, D)
    if case["kind"] == "train":
        state["dout"] = normal(T, Hq, D)
    if case["kind"] in ("append", "paged"):
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
        state.update(k_cache=normal(pages, page, Hkv, D), v_cache=normal(pages, page, Hkv, D),
                     table=table)
    if own:
        # a batch's plan is made once and serves every layer of the model
        import packed_varlen_rotary_rope_amd as rope
        if case["kind"] in ("prompt", "train"):
            state["plan"] = rope.attn_plan(state["cu"], T, Hq, Hkv)
        elif case["kind"] == "paged":
            state["plan"] = rope.paged_plan(state["cu"], state["held"], T, Hq, Hkv)
    return state


def run(state):
    kind = state["case"]["kind"]
    if own:
        return _own(kind, state)
    if kind == "append":
        return _plain_append(state)
    return _plain_attention(kind, state)


def _own(kind, s):
    import packed_varlen_rotary_rope_amd as rope
    if kind == "append":
        q = rope.kv_append_(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["cu"],
                            s["held"], _THETA, q=s["q"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if kind == "paged":
        out, lse = rope.attn_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["plan"],
                                   s["scale"])
        return {"out": out, "lse": lse}
    out, lse = rope.attn_fwd(s["q"], s["k"], s["v"], s["plan"], s["scale"])
    if kind == "prompt":
        return {"out": out, "lse": lse}
    dq, dk, dv = rope.attn_bwd(s["dout"], s["q"], s["k"], s["v"], out, lse, s["plan"], s["scale"])
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def _places(s):
    """Of each packed token its sequence, its number among the sequence's new tokens
    and its position."""
    cu, T = s["cu"].long(), s["q"].shape[0]
    t = torch.arange(T, device=cu.device)
    seq = torch.searchsorted(cu, t, right=True) - 1
    row = t - cu[seq]
    return seq, row, s["held"].long()[seq] - (cu[1:] - cu[:-1])[seq] + row


def _plain_attention(kind, s):
    case = s["case"]
    Hq, Hkv, D, B = case["Hq"], case["Hkv"], case["D"], case["seqs"]
    G, N, M = Hq // Hkv, s["most_new"], s["most_held"]
    seq, row, pos = _places(s)
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
    last = torch.full((B, N), M, dtype=torch.int64, device=dev)  # rows of padding see every key
    last[seq, row] = pos
    seen = torch.arange(M, device=dev) <= last[:, :, None]
    p = torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(s["scale"])
    p.view(B, Hkv, G, N, M).masked_fill_(~seen[:, None, None], float("-inf"))
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
        dq = torch.matmul(ds, k)
        dk = torch.matmul(ds.transpose(-1, -2).contiguous(), q)
        out.update(dq=packed(dq, Hq), dk=packed(dk, Hkv), dv=packed(dv, Hkv))
    return out


def _plain_append(s):
    case = s["case"]
    D, page = case["D"], case["page"]
    seq, row, pos = _places(s)
    # angles are single-precision products of the position and the frequency
    freq = (_THETA ** (-torch.arange(0, D, 2, device=pos.device, dtype=torch.float64) / D)).float()
    angle = (pos.float()[:, None] * freq).double()[:, None]
    cos, sin = angle.cos().float(), angle.sin().float()

    def rotated(x):
        a, b = x.float().chunk(2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(s["dtype"])

    where = s["table"].long()[seq, pos // page], pos % page
    s["k_cache"][where] = rotated(s["k"])
    s["v_cache"][where] = s["v"]
    return {"q": rotated(s["q"]), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def work(case):
    new, held = _new(case), _held(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    size = 4 if case["dtype"] == "f32" else 2
    T, M = sum(new), sum(held)
    # pairs of a query token and a key that it sees
    pairs = sum(n * (m - n) + n * (n + 1) // 2 for n, m in zip(new, held))
    rows = T * Hq * D * size
    if case["kind"] == "append":
        return {"bytes": 2 * rows + 4 * T * Hkv * D * size, "flops": 3 * T * (Hq + Hkv) * D}
    keys = (M if case["kind"] == "paged" else T) * Hkv * D * size
    forward = {"bytes": 2 * rows + 2 * keys + 4 * T * Hq, "flops": 4 * pairs * Hq * D}
    if case["kind"] != "train":
        return forward
    # the step as a whole: q, k, v, dout in; out, lse, dq, dk, dv out
    return {"bytes": 4 * rows + 4 * keys + 4 * T * Hq, "flops": 14 * pairs * Hq * D}


def exact(case, seed):
    """The definition in 64 bits, sequence by sequence and head by head."""
    if work(case)["flops"] > 1e13:
        return None
    s = prepare(case, seed)
    new, held = _new(case), _held(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    G, dev = Hq // Hkv, s["q"].device
    q = s["q"].double()
    if case["kind"] == "append":
        return _exact_append(case, s, new, held)
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
        if case["kind"] == "paged":
            at = torch.arange(m, device=dev)
            page = s["table"][b].long()[at // case["page"]]
            k, v = s["k_cache"][page, at % case["page"]], s["v_cache"][page, at % case["page"]]
        else:
            k, v = s["k"][t0:t1], s["v"][t0:t1]
        hidden = torch.ones((n, m), dtype=torch.bool, device=dev).triu(m - n + 1)
        for h in range(Hq):
            kh, vh = k[:, h // G].double(), v[:, h // G].double()
            score = (q[t0:t1, h] @ kh.T) * s["scale"]
            score[hidden] = float("-inf")
            lse[t0:t1, h] = torch.logsumexp(score, -1)
            p = torch.exp(score - lse[t0:t1, h, None])
            out[t0:t1, h] = p @ vh
            if grads:
                dp = do[t0:t1, h] @ vh.T
                ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * s["scale"]
                grads["dv"][t0:t1, h // G] += p.T @ do[t0:t1, h]
                grads["dq"][t0:t1, h] = ds @ kh
                grads["dk"][t0:t1, h // G] += ds.T @ q[t0:t1, h]
        t0 = t1
    return {"out": out, "lse": lse, **grads}


def _exact_append(case, s, new, held):
    D, half, page = case["D"], case["D"] // 2, case["page"]
    dev = s["q"].device
    # the frequencies and angles are rounded to single precision by definition
    freq = torch.tensor([_THETA ** (-2.0 * j / D) for j in range(half)], device=dev).float()
    q = s["q"].double()
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    t0 = 0
    for b, (n, m) in enumerate(zip(new, held)):
        pos = torch.arange(m - n, m, device=dev)
        angle = (pos.float()[:, None] * freq[None]).double()
        c, z = torch.cos(angle)[:, None, :], torch.sin(angle)[:, None, :]
        turned = []
        for x in (s["q"][t0:t0 + n].double(), s["k"][t0:t0 + n].double()):
            lo, hi = x[..., :half], x[..., half:]
            turned.append(torch.cat([lo * c - hi * z, hi * c + lo * z], -1))
        q[t0:t0 + n] = turned[0]
        pages = s["table"][b].long()[pos // page]
        k_cache[pages, pos % page] = turned[1]
        v_cache[pages, pos % page] = s["v"][t0:t0 + n].double()
        t0 += n
    return {"q": q, "k_cache": k_cache, "v_cache": v_cache}
