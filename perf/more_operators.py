"""Cases of the operators around a rotated and a 4-bit paged cache, with their
plain forms.

They stand where a serving loop's layer has its position rotation, its cache
append and its attention:

  rotate     ``api.paged_append_rotary``: queries and keys are rotated by their
             positions, keys and values go to their slots of a 16-bit cache;
  append4    ``api.paged_append_fp4``: the same into a cache of 4 bits (groups
             of 16 values with a scale of 8 bits), and ``api.paged_read_fp4``,
             which gives back the whole cache as the values it stands for;
  attention4 ``api.paged_attention_fp4``: the new tokens (one per request, K + 1
             drafted ones to verify, a chunk of a prompt) attend to a 4-bit
             cache, causally, with grouped heads.

A case fixes the lengths of all its requests (they follow from its numbers);
the seed makes the tensors and the order of the pages.
"""
import math

import torch

own = False

DEV = "cuda:0"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)   # what the codes 0 .. 7 stand for; 8 more is the sign
GROUP = 16                                        # values that share a scale

# The largest listed cases, which bound the drawn ones: elements moved by an
# append, cached elements read by one attention call, its causal products.
MAX_APPEND_ELEMENTS = 32768 * 48 * 128
MAX_CACHE_ELEMENTS = 256 * 6144 * 8 * 128
MAX_ATTENTION_FLOPS = 4.0e11


def listed():
    return [
        # the verify step of one user, K = 4: latency only
        dict(name="rotate_one", op="rotate", T=5, run=5, Hq=32, Hk=8, D=128, rot=128, pairs="halves", page=16,
             dtype="bf16", far=4000),
        # ragged requests of small heads, half of each rotated, neighbours as pairs, far positions, padding
        dict(name="rotate_ragged", op="rotate", T=4099, run=111, Hq=28, Hk=4, D=64, rot=32, pairs="neighbours", page=8,
             dtype="f16", far=131072),
        # a batch of prompts: queries, keys and values of 32768 tokens
        dict(name="rotate_prompts", op="rotate", T=32768, run=1111, Hq=32, Hk=8, D=128, rot=128, pairs="halves", page=64,
             dtype="bf16", far=8192),
        # the verify step of a batch of 64, K = 4, into a 4-bit cache
        dict(name="append4_verify", op="append4", T=320, run=5, Hq=32, Hk=8, D=128, rot=128, pairs="halves", page=16,
             dtype="bf16", far=4099, k_gain=1.0, v_gain=1.0),
        # ragged requests as above
        dict(name="append4_ragged", op="append4", T=4099, run=111, Hq=28, Hk=4, D=64, rot=64, pairs="neighbours", page=8,
             dtype="f16", far=131072, k_gain=0.5, v_gain=0.03125),
        # a batch of prompts
        dict(name="append4_prompts", op="append4", T=32768, run=1111, Hq=32, Hk=8, D=128, rot=128, pairs="halves", page=64,
             dtype="bf16", far=8192, k_gain=1.0, v_gain=1.0),
        # one request, one token, a short context: the smallest call of a decode loop
        dict(name="token_one", op="attention4", B=1, ctx_min=1000, ctx_max=1000, n_min=1, n_max=1,
             Hq=32, Hk=8, D=128, page=16, dtype="bf16", holes=False, k_gain=1.0, v_gain=1.0),
        # the verify step's attention: K = 4 drafted tokens and the last one, batch of 64
        dict(name="verify", op="attention4", B=64, ctx_min=203, ctx_max=4099, n_min=5, n_max=5,
             Hq=32, Hk=8, D=128, page=16, dtype="bf16", holes=False, k_gain=1.0, v_gain=1.0),
        # long contexts, few requests, one token each: the cache is split over the GPU
        dict(name="token_long", op="attention4", B=4, ctx_min=60001, ctx_max=131072, n_min=1, n_max=1,
             Hq=64, Hk=8, D=128, page=64, dtype="bf16", holes=False, k_gain=0.5, v_gain=0.25),
        # long drafts (K = 8) verified for a batch of 256: the most cache read by one call
        dict(name="verify_long_draft", op="attention4", B=256, ctx_min=2000, ctx_max=10240, n_min=9, n_max=9,
             Hq=64, Hk=8, D=128, page=32, dtype="bf16", holes=False, k_gain=1.0, v_gain=1.0),
        # ragged chunks with finished and failed requests among them, an odd group, small heads and pages
        dict(name="ragged_chunks", op="attention4", B=37, ctx_min=0, ctx_max=3001, n_min=1, n_max=167,
             Hq=28, Hk=4, D=64, page=8, dtype="f16", holes=True, k_gain=1.0, v_gain=0.5),
        # a chunk of 2048 prompt tokens over a context of about 6000, two requests: the most arithmetic
        dict(name="chunk_prompt", op="attention4", B=2, ctx_min=5000, ctx_max=7001, n_min=2048, n_max=2048,
             Hq=32, Hk=8, D=128, page=128, dtype="bf16", holes=False, k_gain=1.0, v_gain=1.0),
    ]


def _log_int(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["rotate", "append4", "attention4", "attention4", "attention4"])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    Hk, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    case = dict(op=op, Hq=Hk * G, Hk=Hk, D=D, page=page, dtype=dtype)
    if op != "rotate":
        case.update(k_gain=rng.choice([1.0, 1.0, 0.5, 0.0625]), v_gain=rng.choice([1.0, 1.0, 0.25, 0.1015625]))
    if op != "attention4":
        T = _log_int(rng, 1, min(65536, MAX_APPEND_ELEMENTS // ((G + 2) * Hk * D)))
        return dict(case, T=T, run=_log_int(rng, 1, T), rot=rng.choice([r for r in (32, 64, 96, 128) if r <= D]),
                    pairs=rng.choice(["halves", "neighbours"]), far=_log_int(rng, 1000, 131072))
    if rng.random() < 0.6:  # single tokens and drafts
        B = _log_int(rng, 1, 256)
        n_max = _log_int(rng, 1, 17)
        ctx_max = _log_int(rng, 1, max(1, min(131072, MAX_CACHE_ELEMENTS // (B * Hk * D))))
        ctx_min = rng.randint(0, ctx_max)
    else:  # chunks of prompts, and whole ones
        B = _log_int(rng, 1, 8)
        ctx_max = rng.choice([0, _log_int(rng, 1, 16384)])
        ctx_min = rng.randint(0, ctx_max)
        n_max = _log_int(rng, 18, 8192)
        while 4 * D * Hk * G * B * n_max * (ctx_max + n_max) > MAX_ATTENTION_FLOPS:
            n_max = n_max * 3 // 4
    return dict(case, B=B, ctx_min=ctx_min, ctx_max=ctx_max, n_min=rng.randint(1, n_max), n_max=n_max,
                holes=rng.random() < 0.3)


# ------------------------------------------------------------------ lengths

def _spread(low, high, count, step):
    """`count` whole numbers of [low, high], in a fixed scattered order."""
    return [low + (b * step % 1009) * (high - low) // 1008 for b in range(count)]


def _lengths(case):
    """(new tokens, kv lengths) of a case's requests.  With holes, some
    requests bring no token and some have failed (no key visible)."""
    B = case["B"]
    ctx = _spread(case["ctx_min"], case["ctx_max"], B, 613) if B > 1 else [case["ctx_max"]]
    new = _spread(case["n_min"], case["n_max"], B, 389) if B > 1 else [case["n_max"]]
    if B > 1:
        ctx[-1], new[-1] = case["ctx_max"], case["n_max"]
    kv = [c + n for c, n in zip(ctx, new)]
    if case.get("holes"):
        for b in range(B):
            if b % 7 == 3:
                new[b], kv[b] = 0, ctx[b]
            if b % 7 == 5:
                kv[b] = 0
    return new, kv


def _slots(case):
    """How many slots the cache of an append has, and its pages per request."""
    each = (case["run"] + case["page"] - 2) // case["page"] + 1
    return (-(-case["T"] // case["run"]) * each + 2) * case["page"], each


def work(case):
    D, Hk, Hq = case["D"], case["Hk"], case["Hq"]
    packed = D // 2 + D // GROUP   # bytes of a 4-bit key or value
    if case["op"] != "attention4":
        T, rot = case["T"], case["rot"]
        # the new tokens are read, the rotated queries written; positions, slots, and a table row per token
        moved = T * ((2 * Hq + 2 * Hk) * D * 2 + 8 + 4 * rot)
        flops = 3.0 * T * (Hq + Hk) * rot
        if case["op"] == "rotate":
            return {"bytes": float(moved + T * 2 * Hk * D * 2), "flops": flops}
        n_slots, _ = _slots(case)
        return {"bytes": float(moved + T * 2 * Hk * packed + n_slots * (4 + 2 * Hk * (packed + 2 * D))), "flops": flops}
    new, kv = _lengths(case)
    pairs = 0
    for n, L in zip(new, kv):
        first = L - n + 1  # keys visible to the request's first token
        k = max(0, 1 - first)  # tokens that see none
        pairs += (n - k) * (2 * (first + k) + n - k - 1) // 2
    read = sum(L for n, L in zip(new, kv) if n) * Hk * packed * 2
    pages = sum(-(-L // case["page"]) for n, L in zip(new, kv) if n)
    return {"bytes": float(read + sum(new) * (2 * Hq * D * 2 + 4 * Hq) + 4 * pages + 8 * case["B"]),
            "flops": 4.0 * D * Hq * pairs}


# ------------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _coded(shape, g):
    """Codes and scales of normal numbers [..., D], a piece at a time."""
    rows, D = math.prod(shape[:-1]), shape[-1]
    codes = torch.empty(rows, D // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(rows, D // GROUP, dtype=torch.float8_e4m3fn, device=DEV)
    step = 1 << 20
    for i in range(0, rows, step):
        n = min(step, rows - i)
        codes[i:i + n], scales[i:i + n] = _encode(torch.randn(n, D, generator=g, device=DEV), 1.0)
    return codes.view(*shape[:-1], D // 2), scales.view(*shape[:-1], D // GROUP)


def prepare(case, seed):
    g = _generator(seed)
    page, dt, Hq, Hk, D = case["page"], DTYPES[case["dtype"]], case["Hq"], case["Hk"], case["D"]
    if case["op"] != "attention4":
        T, length, far, rot = case["T"], case["run"], case["far"], case["rot"]
        n_slots, each = _slots(case)
        n_pages = n_slots // page
        # the projection's output holds queries, keys and values of a token side by side
        qkv = torch.randn((T, Hq + 2 * Hk, D), generator=g, device=DEV).to(dt)
        token = torch.arange(T, device=DEV)
        request = token // length
        start = request * 7919 % max(1, far - length)   # cached tokens of the request
        positions = (start + token % length).to(torch.int32)
        at = start % page + token % length              # requests begin anywhere in a page
        slots = (torch.randperm(n_pages, generator=g, device=DEV)[request * each + at // page] * page + at % page).to(torch.int32)
        slots[T // 2: T // 2 + T // 64] = -1             # tokens of a request that got no pages
        positions[T - T // 100:], slots[T - T // 100:] = -1, -1   # padding
        angles = torch.arange(far + 1, dtype=torch.float64, device=DEV)[:, None] * 10000.0 ** (
            -torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
        s = dict(case=case, q=qkv[:, :Hq], k_new=qkv[:, Hq:Hq + Hk], v_new=qkv[:, Hq + Hk:], slot_map=slots, positions=positions,
                 cos_sin=torch.cat([angles.cos(), angles.sin()], 1).float(), neighbours=case["pairs"] == "neighbours")
        if case["op"] == "rotate":
            for name in ("k_cache", "v_cache"):
                s[name] = torch.randn((n_pages, Hk, page, D), generator=g, device=DEV).to(dt)
        else:
            s["k"], s["k_scale"] = _coded((n_pages, Hk, page, D), g)
            s["v"], s["v_scale"] = _coded((n_pages, Hk, page, D), g)
            s["every_slot"] = torch.arange(n_slots, dtype=torch.int32, device=DEV)
        return s
    new, kv = _lengths(case)
    pages = [-(-L // page) for L in kv]
    n_pages, width = sum(pages) + 8, max(max(pages), 1)
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    count = torch.tensor(pages, device=DEV)
    column = torch.arange(width, device=DEV)
    at = ((torch.cumsum(count, 0) - count)[:, None] + column).clamp(max=n_pages - 1)
    table = torch.where(column < count[:, None], order[at], torch.zeros_like(order[at]))
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    qkv = torch.randn((cu[-1], Hq + 2 * Hk, D), generator=g, device=DEV).to(dt)
    k, k_scale = _coded((n_pages, Hk, page, D), g)
    v, v_scale = _coded((n_pages, Hk, page, D), g)
    return dict(case=case, q=qkv[:, :Hq], k=k, k_scale=k_scale, v=v, v_scale=v_scale, block_table=table,
                cu_new=_ints(cu), kv_len=_ints(kv), scale=1.0 / math.sqrt(D), most_new=max(new), most_kv=max(kv))


# ---------------------------------------------------------------- operators

def run(state):
    return RUN[state["case"]["op"]](state)


def _run_rotate(s):
    if own:
        from speculative_decoding_verification_25_gb300 import api
        q = api.paged_append_rotary(s["q"], s["k_new"], s["v_new"], s["positions"], s["cos_sin"], s["slot_map"],
                                    s["k_cache"], s["v_cache"], interleaved=s["neighbours"])
        return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])
    page, dt = s["case"]["page"], s["q"].dtype
    good = s["slot_map"] >= 0
    slot = s["slot_map"][good].long()
    k = _rotated(s["k_new"].float(), s["positions"], s["cos_sin"], s["neighbours"])
    s["k_cache"][slot // page, :, slot % page] = k[good].to(dt)
    s["v_cache"][slot // page, :, slot % page] = s["v_new"][good]
    q = _rotated(s["q"].float(), s["positions"], s["cos_sin"], s["neighbours"]).to(dt)
    return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])


def _run_append4(s):
    c, dt = s["case"], s["q"].dtype
    if own:
        from speculative_decoding_verification_25_gb300 import api
        cache = api.PagedCacheFp4(s["k"], s["k_scale"], s["v"], s["v_scale"])
        q = api.paged_append_fp4(s["q"], s["k_new"], s["v_new"], s["positions"], s["cos_sin"], s["slot_map"], cache,
                                 k_gain=c["k_gain"], v_gain=c["v_gain"], interleaved=s["neighbours"])
        k, v = api.paged_read_fp4(cache, s["every_slot"], dt, k_gain=c["k_gain"], v_gain=c["v_gain"])
        return dict(q=q, k=k, v=v)
    page = c["page"]
    good = s["slot_map"] >= 0
    slot = s["slot_map"][good].long()
    # in 64 bits: a rotated key may lie next to the border of two codes
    k = _rotated(s["k_new"][good].double(), s["positions"][good], s["cos_sin"].double(), s["neighbours"])
    out = {}
    for name, x in (("k", k), ("v", s["v_new"][good].double())):
        codes, scales = _encode(x, c[name + "_gain"])
        s[name][slot // page, :, slot % page] = codes
        s[name + "_scale"].view(torch.uint8)[slot // page, :, slot % page] = scales.view(torch.uint8)
        values = _decode(s[name], s[name + "_scale"]) * c[name + "_gain"]
        out[name] = values.transpose(1, 2).flatten(0, 1).to(dt)
    out["q"] = _rotated(s["q"].float(), s["positions"], s["cos_sin"], s["neighbours"]).to(dt)
    return out


def _run_attention4(s):
    c = s["case"]
    if own:
        from speculative_decoding_verification_25_gb300 import api
        r = api.paged_attention_fp4(s["q"], api.PagedCacheFp4(s["k"], s["k_scale"], s["v"], s["v_scale"]), s["block_table"],
                                    s["cu_new"], s["kv_len"], scale=s["scale"], k_gain=c["k_gain"], v_gain=c["v_gain"],
                                    want_lse=True)
        return dict(out=r.out, lse=r.lse)
    return _plain_attention(s, c)


RUN = {"rotate": _run_rotate, "append4": _run_append4, "attention4": _run_attention4}


def _rotated(x, positions, cos_sin, neighbours):
    """x [T, heads, D] with its first columns rotated, in x's type; zeros where
    there is no position."""
    rot = cos_sin.shape[1]
    row = cos_sin[positions.clamp(min=0).long()][:, None]   # [T, 1, rot]
    cos, sin = row[..., :rot // 2], row[..., rot // 2:]
    turned = x[..., :rot]
    a, b = (turned[..., 0::2], turned[..., 1::2]) if neighbours else (turned[..., :rot // 2], turned[..., rot // 2:])
    a, b = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([a, b], -1).flatten(-2) if neighbours else torch.cat([a, b], -1)
    y = torch.cat([turned, x[..., rot:]], -1)
    return torch.where((positions >= 0)[:, None, None], y, torch.zeros_like(y))


def _encode(x, gain):
    """Codes [..., D / 2] (the even element in the low half) and scales [...,
    D / 16] of x [..., D].  A group's scale is its largest magnitude over 6
    gain, rounded to 8 bits; its codes are the nearest to x over scale and
    gain, ties to the even one."""
    groups = x.unflatten(-1, (-1, GROUP))
    want = groups.abs().amax(-1) / torch.full((), 6.0 * gain, dtype=x.dtype, device=x.device)
    _, e = torch.frexp(want)
    step = torch.exp2((e - 4).clamp(min=-9).to(x.dtype))   # of an e4m3 number of that size
    scale = (torch.round(want / step) * step).clamp(max=448.0)
    unit = (scale * gain)[..., None]
    y = torch.where(unit > 0, groups.abs() / unit, torch.zeros_like(groups))
    code = torch.zeros_like(y, dtype=torch.uint8)
    for border, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (y >= border) if up else (y > border)
    code += 8 * (torch.signbit(groups) & (unit > 0))
    code = code.flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, scale.float().to(torch.float8_e4m3fn)


def _decode(codes, scales):
    """Values [..., D] in 32 bits: exact."""
    table = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=codes.device)
    both = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    values = table[both.int()].unflatten(-1, (-1, GROUP))
    return values.mul_(scales.float()[..., None]).flatten(-2)


def _plain_attention(s, c):
    """Every request padded to the longest, products and softmax in 32 bits."""
    q, table, cu, kv_len, most_new, most_kv = s["q"], s["block_table"], s["cu_new"].long(), s["kv_len"].long(), s["most_new"], s["most_kv"]
    T, Hq, D = q.shape
    Hk, page = c["Hk"], c["page"]
    B, G = kv_len.numel(), Hq // Hk
    dev = q.device
    if most_kv == 0:
        return dict(out=torch.zeros(T, Hq, D, dtype=q.dtype, device=dev), lse=torch.full((T, Hq), -math.inf, device=dev))
    blocks = table[:, :-(-most_kv // page)].long()
    key = torch.arange(blocks.shape[1] * page, device=dev)
    inside = key < kv_len[:, None]  # [B, L]
    k, v = (_decode(s[n][blocks], s[n + "_scale"].view(torch.uint8)[blocks].view(torch.float8_e4m3fn))
            .transpose(1, 2).reshape(B, Hk, -1, D).mul_(c[n + "_gain"]) for n in ("k", "v"))
    v = torch.where(inside[:, None, :, None], v, 0.0)
    new = cu[1:] - cu[:-1]
    i = torch.arange(most_new, device=dev)
    real = i < new[:, None]  # [B, n]
    rows = (cu[:-1, None] + i).clamp(max=T - 1)
    qs = q[rows].float().reshape(B, most_new, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, most_new * G, D)
    seen = (key <= (kv_len - new)[:, None, None] + i[:, None]) & inside[:, None]  # [B, n, L]
    x = torch.matmul(qs, k.transpose(-1, -2)).reshape(B, Hk, most_new, G, -1).mul_(s["scale"])
    x = x.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(B, Hk, most_new * G, -1), v).reshape(B, Hk, most_new, G, D)
    o = torch.where(total > 0, o / total.clamp(min=1e-30), 0.0)
    lse = (top + total.log()).squeeze(-1)  # -inf where nothing is visible
    o = o.permute(0, 2, 1, 3, 4).reshape(B, most_new, Hq, D)[real]
    lse = lse.permute(0, 2, 1, 3).reshape(B, most_new, Hq)[real]
    return dict(out=o.to(q.dtype), lse=lse)


# ---------------------------------------------------------------- in 64 bits

def _nearest(y, values):
    """Index of the nearest of ascending `values`, of two the even one."""
    low = (torch.searchsorted(values, y.contiguous(), right=True) - 1).clamp(0, len(values) - 2)
    below, above = y - values[low], values[low + 1] - y
    return low + ((above < below) | ((above == below) & (low % 2 == 1)))


def _stored(x, gain):
    """The values that x [n, heads, D] is held as, in 64 bits."""
    eights = torch.arange(127, dtype=torch.uint8, device=x.device).view(torch.float8_e4m3fn).double()
    fours = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    y = x.reshape(*x.shape[:-1], -1, GROUP)
    scale = eights[_nearest(y.abs().amax(-1) / (6.0 * gain), eights)][..., None] * gain
    ratio = y.abs() / torch.where(scale == 0, math.inf, scale)
    return (fours[_nearest(ratio, fours)] * scale * torch.sign(y)).reshape(x.shape)


def _turned(x, s):
    """x with columns turned as complex numbers, in 64 bits."""
    rot, table = s["case"]["rot"], s["cos_sin"].double()
    turn = torch.complex(table[:, :rot // 2], table[:, rot // 2:])[s["positions"].clamp(min=0).long()][:, None]
    first = x[..., :rot]
    first = first.unflatten(-1, (rot // 2, 2) if s["neighbours"] else (2, rot // 2))
    if not s["neighbours"]:
        first = first.transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(first.contiguous()) * turn)
    if not s["neighbours"]:
        z = z.transpose(-1, -2)
    y = torch.cat([z.flatten(-2), x[..., rot:]], -1)
    return y * (s["positions"] >= 0)[:, None, None]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] != "attention4":
        at = torch.nonzero(s["slot_map"] >= 0).squeeze(1)
        slots = s["slot_map"][at].long()
        want = {"q": _turned(s["q"].double(), s)}
        for name, x in (("k", _turned(s["k_new"].double(), s)), ("v", s["v_new"].double())):
            if case["op"] == "rotate":
                tokens = s[name + "_cache"].double().transpose(1, 2).flatten(0, 1)   # [slots, Hk, D]
                tokens = tokens.index_copy(0, slots, x.index_select(0, at))
                want[name + "_cache"] = tokens.unflatten(0, (-1, case["page"])).transpose(1, 2)
            else:
                before = _values(s, name).transpose(1, 2).flatten(0, 1)
                want[name] = before.index_copy(0, slots, _stored(x.index_select(0, at), case[name + "_gain"]))
        return want
    q = s["q"]
    T, Hq, D = q.shape
    Hk, page = case["Hk"], case["page"]
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=DEV)
    new, kv = _lengths(case)
    first = 0
    for b, (n, L) in enumerate(zip(new, kv)):
        if n and L:
            ids = s["block_table"][b, :-(-L // page)].long()
            K, V = (_values(s, name, ids).transpose(1, 2).flatten(0, 1)[:L] for name in ("k", "v"))   # [L, Hk, D]
            for h in range(Hk):
                heads = slice(h * (Hq // Hk), (h + 1) * (Hq // Hk))
                for t in range(0, n, 1024):
                    m = min(1024, n - t)
                    x = torch.einsum("tgd,ld->tgl", q[first + t:first + t + m, heads].double(), K[:, h]) * case["D"] ** -0.5
                    last = torch.arange(t, t + m, device=DEV) + (L - n)
                    x[(torch.arange(L, device=DEV)[None] > last[:, None])[:, None].expand_as(x)] = -math.inf
                    z = torch.logsumexp(x, -1)
                    w = torch.exp(x - torch.where(z.isinf(), 0.0, z)[..., None])
                    out[first + t:first + t + m, heads] = torch.einsum("tgl,ld->tgd", w, V[:, h])
                    lse[first + t:first + t + m, heads] = z
        first += n
    return dict(out=out, lse=lse)


def _values(s, name, pages=slice(None)):
    """What the cache's pages stand for, in 64 bits."""
    codes, scales = s[name][pages].long(), s[name + "_scale"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).double()
    signed = torch.tensor([w * x for w in (1.0, -1.0) for x in E2M1], dtype=torch.float64, device=DEV)
    pair = torch.stack([signed[codes % 16], signed[codes // 16]], -1).flatten(-2)
    return pair * scales.repeat_interleave(GROUP, -1) * s["case"][name + "_gain"]
