"""Cases of the paged key/value cache operators, with their plain forms.

The three operators are the target model's side of a speculative decoding
step, in the order in which a serving loop calls them:

  plan       ``api.paged_plan``: from the request lengths on the device, the
             block tables, slot map, positions and packed offsets of the step;
  append     ``api.paged_append``: the new tokens' keys and values go to
             their slots of the paged cache;
  attention  ``api.paged_attention``: the new tokens (one per request, K + 1
             drafted ones to verify, a chunk of a prompt or all of it) attend
             to the cache, causally, with grouped heads.

A case fixes the lengths of all its requests (they follow from its numbers);
the seed makes the tensors and the order of the pages.
"""
import math

import torch

own = False

DEV = "cuda:0"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}

# The largest listed cases, which bound the drawn ones: cached elements read
# by one attention call, its causal products, and tokens of a plan or append.
MAX_CACHE_ELEMENTS = 256 * 6144 * 8 * 128
MAX_ATTENTION_FLOPS = 1.0e12
MAX_PLAN_TOKENS = 1 << 19
MAX_APPEND_ELEMENTS = 32768 * 8 * 128


def listed():
    return [
        # one short request between two steps of a single-user loop: latency only
        dict(name="plan_one", op="plan", B=1, ctx_min=1000, ctx_max=1000, n_min=5, n_max=5, page=16),
        # the verify step of a batch of 64, K = 4: five new tokens each, odd contexts
        dict(name="plan_verify", op="plan", B=64, ctx_min=203, ctx_max=4099, n_min=5, n_max=5, page=16),
        # a large service admits prompts: many rows, ragged chunks, half a million tokens
        dict(name="plan_prompts", op="plan", B=1024, ctx_min=0, ctx_max=2048, n_min=1, n_max=1001, page=32),
        # keys and values of the verify step of a batch of 64
        dict(name="append_verify", op="append", T=320, run=5, Hk=8, D=128, page=16, dtype="bf16"),
        # keys and values of a batch of prompts
        dict(name="append_prompts", op="append", T=32768, run=1111, Hk=8, D=128, page=64, dtype="bf16"),
        # one request, one token, a short context: the smallest call of a decode loop
        dict(name="token_one", op="attention", B=1, ctx_min=1000, ctx_max=1000, n_min=1, n_max=1,
             Hq=32, Hk=8, D=128, page=16, dtype="bf16", holes=False),
        # the verify step's attention: K = 4 drafted tokens and the last one, batch of 64
        dict(name="verify", op="attention", B=64, ctx_min=203, ctx_max=4099, n_min=5, n_max=5,
             Hq=32, Hk=8, D=128, page=16, dtype="bf16", holes=False),
        # long contexts, few requests, one token each: the cache is split over the GPU
        dict(name="token_long", op="attention", B=4, ctx_min=60001, ctx_max=131072, n_min=1, n_max=1,
             Hq=64, Hk=8, D=128, page=64, dtype="bf16", holes=False),
        # long drafts (K = 8) verified for a batch of 256: the most cache read by one call
        dict(name="verify_long_draft", op="attention", B=256, ctx_min=2000, ctx_max=10240, n_min=9, n_max=9,
             Hq=64, Hk=8, D=128, page=32, dtype="bf16", holes=False),
        # ragged chunks with finished and failed requests among them, an odd group, small heads and pages
        dict(name="ragged_chunks", op="attention", B=37, ctx_min=0, ctx_max=3001, n_min=1, n_max=167,
             Hq=28, Hk=4, D=64, page=8, dtype="f16", holes=True),
        # a chunk of 2048 prompt tokens over a context of about 6000, two requests
        dict(name="chunk_prompt", op="attention", B=2, ctx_min=5000, ctx_max=7001, n_min=2048, n_max=2048,
             Hq=32, Hk=8, D=128, page=128, dtype="bf16", holes=False),
        # whole prompts of different lengths, no context: the most arithmetic
        dict(name="whole_prompts", op="attention", B=3, ctx_min=0, ctx_max=0, n_min=4000, n_max=8192,
             Hq=32, Hk=8, D=128, page=16, dtype="bf16", holes=False),
    ]


def _log_int(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "attention", "attention", "attention", "attention"])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    if op == "plan":
        B = _log_int(rng, 1, 2048)
        n_max = _log_int(rng, 1, max(1, min(8192, MAX_PLAN_TOKENS // B)))
        ctx_max = _log_int(rng, 1, 16384)
        return dict(op=op, B=B, ctx_min=rng.randint(0, ctx_max), ctx_max=ctx_max,
                    n_min=rng.randint(1, n_max), n_max=n_max, page=page)
    dtype = rng.choice(["bf16", "bf16", "f16"])
    Hk, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    if op == "append":
        T = _log_int(rng, 1, MAX_APPEND_ELEMENTS // (Hk * D))
        return dict(op=op, T=T, run=_log_int(rng, 1, T), Hk=Hk, D=D, page=page, dtype=dtype)
    G = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    case = dict(op=op, Hq=Hk * G, Hk=Hk, D=D, page=page, dtype=dtype)
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
    """(contexts, new tokens, kv lengths) of a case's requests.  With holes,
    some requests bring no token and some have failed (no key visible)."""
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
    return ctx, new, kv


def _held(case):
    """Pages that each request of a plan holds before the step: those of its
    context; one request in four one more (rejected drafts), one in sixteen
    has finished and gives all of its pages back."""
    ctx, new, _ = _lengths(case)
    page = case["page"]
    seq = list(ctx)
    held = [-(-c // page) for c in ctx]
    for b in range(case["B"]):
        if b % 4 == 1:
            held[b] = -(-(ctx[b] + new[b]) // page) + 1
        if b % 16 == 7:
            seq[b], new[b] = 0, 0
    return seq, new, held


def work(case):
    if case["op"] == "plan":
        seq, new, held = _held(case)
        want = [-(-(s + n) // case["page"]) for s, n in zip(seq, new)]
        moved = sum(abs(w - h) for w, h in zip(want, held))
        looked = sum(min(w, h) - s // case["page"] for w, h, s in zip(want, held, seq) if min(w, h) > s // case["page"])
        rows = case["B"] * 4 * (3 + 3) + 16  # lengths and page counts in; offsets, lengths and page counts out
        return {"bytes": float(rows + 8 * sum(new) + 8 * moved + 4 * looked), "flops": 0.0}
    elt = 2
    if case["op"] == "append":
        return {"bytes": 4.0 * elt * case["T"] * case["Hk"] * case["D"] + 4.0 * case["T"], "flops": 0.0}
    _, new, kv = _lengths(case)
    pairs = 0
    for n, L in zip(new, kv):
        first = L - n + 1  # keys visible to the request's first token
        k = max(0, 1 - first)  # tokens that see none
        pairs += (n - k) * (2 * (first + k) + n - k - 1) // 2
    row = case["Hq"] * case["D"] * elt
    read = sum(L for n, L in zip(new, kv) if n) * case["Hk"] * case["D"] * elt * 2
    pages = sum(-(-L // case["page"]) for n, L in zip(new, kv) if n)
    return {"bytes": float(read + sum(new) * (2 * row + 4 * case["Hq"]) + 4 * pages + 8 * case["B"]),
            "flops": 4.0 * case["D"] * case["Hq"] * pairs}


# ------------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(shape, dtype, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32 if math.prod(shape) < 1 << 28 else dtype).to(dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _tables(pages, width, n_pages, g):
    """Block tables of requests that hold `pages` pages each, scattered over a
    pool of `n_pages`, and the pages left over."""
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    count = torch.tensor(pages, device=DEV)
    start = torch.cumsum(count, 0) - count
    column = torch.arange(width, device=DEV)
    at = (start[:, None] + column).clamp(max=n_pages - 1)
    table = torch.where(column < count[:, None], order[at], torch.zeros_like(order[at]))
    return table, order[sum(pages):].contiguous()


def prepare(case, seed):
    g = _generator(seed)
    page = case["page"]
    if case["op"] == "plan":
        seq, new, held = _held(case)
        want = [-(-(s + n) // page) for s, n in zip(seq, new)]
        width = max(max(want), max(held)) + 1
        n_pages = sum(held) + sum(max(0, w - h) for w, h in zip(want, held)) + 7
        table, free = _tables(held, width, n_pages, g)
        stack = torch.full((n_pages,), -1, dtype=torch.int32, device=DEV)
        stack[:free.numel()] = free
        return dict(case=case, seq_len=_ints(seq), num_new=_ints(new), page_count=_ints(held), block_table=table,
                    free_pages=stack, free_count=_ints([free.numel()]), max_tokens=sum(new) + 3)
    dt, Hk, D = DTYPES[case["dtype"]], case["Hk"], case["D"]
    if case["op"] == "append":
        T, length = case["T"], case["run"]  # requests of `length` tokens each, begun anywhere in a page
        each = (length + page - 2) // page + 1
        n_pages = -(-T // length) * each + 8
        # the projection's output holds queries, keys and values of a token side by side
        qkv = _normal((T, 3 * Hk, D), dt, g)
        token = torch.arange(T, device=DEV)
        request, at = token // length, token % length + token // length * 7 % page
        slots = (torch.randperm(n_pages, generator=g, device=DEV)[request * each + at // page] * page + at % page).to(torch.int32)
        slots[T // 2: T // 2 + T // 64] = -1  # tokens of a request that got no pages
        cache = [_normal((n_pages, Hk, page, D), dt, g) for _ in range(2)]
        return dict(case=case, k_new=qkv[:, Hk:2 * Hk], v_new=qkv[:, 2 * Hk:], slot_map=slots, k_cache=cache[0], v_cache=cache[1])
    _, new, kv = _lengths(case)
    pages = [-(-L // page) for L in kv]
    n_pages = sum(pages) + 8
    table, _ = _tables(pages, max(max(pages), 1), n_pages, g)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    qkv = _normal((cu[-1], case["Hq"] + 2 * Hk, D), dt, g)
    cache = [_normal((n_pages, Hk, page, D), dt, g) for _ in range(2)]
    return dict(case=case, q=qkv[:, :case["Hq"]], k_cache=cache[0], v_cache=cache[1], block_table=table,
                cu_new=_ints(cu), kv_len=_ints(kv), scale=1.0 / math.sqrt(D), most_new=max(new), most_kv=max(kv))


# ---------------------------------------------------------------- operators

def run(state):
    return RUN[state["case"]["op"]](state)


def _run_plan(s):
    if own:
        from speculative_decoding_verification_25_gb300 import api
        p = api.paged_plan(s["seq_len"], s["num_new"], s["page_count"], s["block_table"], s["free_pages"], s["free_count"],
                           page_size=s["case"]["page"], max_tokens=s["max_tokens"])
        return dict(cu_new=p.cu_new, kv_len=p.kv_len, slot_map=p.slot_map, positions=p.positions, page_count=p.page_count,
                    free_count=p.free_count, block_table=s["block_table"], free_pages=s["free_pages"])
    return _plain_plan(s["seq_len"].long(), s["num_new"].long(), s["page_count"].long(), s["block_table"], s["free_pages"],
                       s["free_count"].long(), s["case"]["page"], s["max_tokens"])


def _run_append(s):
    if own:
        from speculative_decoding_verification_25_gb300 import api
        api.paged_append(s["k_new"], s["v_new"], s["slot_map"], s["k_cache"], s["v_cache"])
    else:
        page = s["case"]["page"]
        good = s["slot_map"] >= 0
        slot = s["slot_map"][good].long()
        s["k_cache"][slot // page, :, slot % page] = s["k_new"][good]
        s["v_cache"][slot // page, :, slot % page] = s["v_new"][good]
    return dict(k_cache=s["k_cache"], v_cache=s["v_cache"])


def _run_attention(s):
    if own:
        from speculative_decoding_verification_25_gb300 import api
        r = api.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["cu_new"], s["kv_len"],
                                scale=s["scale"], want_lse=True)
        return dict(out=r.out, lse=r.lse)
    return _plain_attention(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["cu_new"].long(), s["kv_len"].long(),
                            s["scale"], s["most_new"], s["most_kv"])


RUN = {"plan": _run_plan, "append": _run_append, "attention": _run_attention}


def _plain_plan(seq, new, have, table, stack, free, page, max_tokens):
    """Requests in their order; pages given back are taken first, the last
    free page next."""
    B, width = table.shape
    dev = table.device
    valid = (seq >= 0) & (new >= 0) & (have >= 0) & (have <= width) & (seq + new <= width * page)
    new = torch.where(valid, new, 0)
    ends = torch.cumsum(new, 0)
    fits = valid & ((ends <= max_tokens) | (new == 0))
    new = torch.where(fits, new, 0)
    ends = torch.cumsum(new, 0)
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), ends])
    want = torch.where(fits, (seq + new + page - 1) // page, have)
    back, need = (have - want).clamp(min=0), (want - have).clamp(min=0)
    back_at, need_at = torch.cumsum(back, 0), torch.cumsum(need, 0)
    served = fits & ((need == 0) | (need_at <= free + back_at[-1]))
    need = torch.where(served, need, 0)
    need_at = torch.cumsum(need, 0)

    # pages in the order in which they are taken: those given back, then the stack from its top
    column = torch.arange(width, device=dev)
    given = table[(column >= want[:, None]) & (column < have[:, None])]
    top = torch.arange(stack.numel(), device=dev)
    pool = torch.cat([given, stack.flip(0)[top >= stack.numel() - free]])
    taken = (need_at - need)[:, None] + column - have[:, None]
    grown = (column >= have[:, None]) & (column < (have + need)[:, None])
    table.copy_(torch.where(grown, pool[taken.clamp(0, pool.numel() - 1)] if pool.numel() else table, table))
    held = torch.where(served, want, have)
    total = need_at[-1:]
    left = free + back_at[-1:] - total
    rest = pool.flip(0)  # the whole stack, bottom first
    keep = (top < left) & (top >= free)
    if rest.numel():
        stack.copy_(torch.where(keep, rest[top.clamp(max=rest.numel() - 1)], stack))

    token = torch.arange(max_tokens, device=dev)
    row = torch.searchsorted(cu[1:], token, right=True).clamp(max=B - 1)
    real = token < cu[-1]
    at = seq[row] + token - cu[row]
    block = table[row, (at // page).clamp(0, width - 1)].long()
    slot = torch.where(real & served[row], block * page + at % page, -1)
    kv = torch.where(served, seq + new, 0)
    i32 = torch.int32
    return dict(cu_new=cu.to(i32), kv_len=kv.to(i32), slot_map=slot.to(i32), positions=torch.where(real, at, -1).to(i32),
                page_count=held.to(i32), free_count=left.to(i32), block_table=table, free_pages=stack)


def _plain_attention(q, k_cache, v_cache, table, cu, kv_len, scale, most_new, most_kv):
    """Every request padded to the longest, products and softmax in 32 bits."""
    T, Hq, D = q.shape
    n_pages, Hk, page, _ = k_cache.shape
    B, G = kv_len.numel(), Hq // Hk
    dev = q.device
    if most_kv == 0:
        return dict(out=torch.zeros(T, Hq, D, dtype=q.dtype, device=dev), lse=torch.full((T, Hq), -math.inf, device=dev))
    blocks = table[:, :-(-most_kv // page)].long()
    key = torch.arange(blocks.shape[1] * page, device=dev)
    inside = key < kv_len[:, None]  # [B, L]
    k = k_cache[blocks].transpose(1, 2).reshape(B, Hk, -1, D).float()
    v = v_cache[blocks].transpose(1, 2).reshape(B, Hk, -1, D).float()
    v = torch.where(inside[:, None, :, None], v, 0.0)
    new = cu[1:] - cu[:-1]
    i = torch.arange(most_new, device=dev)
    real = i < new[:, None]  # [B, n]
    rows = (cu[:-1, None] + i).clamp(max=T - 1)
    qs = q[rows].float().reshape(B, most_new, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, most_new * G, D)
    seen = (key <= (kv_len - new)[:, None, None] + i[:, None]) & inside[:, None]  # [B, n, L]
    s = torch.matmul(qs, k.transpose(-1, -2)).reshape(B, Hk, most_new, G, -1).mul_(scale)
    s = s.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = s.amax(-1, keepdim=True).clamp(min=-3e38)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(B, Hk, most_new * G, -1), v).reshape(B, Hk, most_new, G, D)
    o = torch.where(total > 0, o / total.clamp(min=1e-30), 0.0)
    lse = (top + total.log()).squeeze(-1)  # -inf where nothing is visible
    o = o.permute(0, 2, 1, 3, 4).reshape(B, most_new, Hq, D)[real]
    lse = lse.permute(0, 2, 1, 3).reshape(B, most_new, Hq)[real]
    return dict(out=o.to(q.dtype), lse=lse)


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return None  # whole numbers: equal or wrong
    if case["op"] == "append":
        cells = torch.nonzero(s["slot_map"] >= 0).squeeze(1)
        at = s["slot_map"][cells].long()
        want = {}
        for name in ("k", "v"):
            tokens = s[name + "_cache"].double().transpose(1, 2).flatten(0, 1)  # [slots, Hk, D]
            tokens = tokens.index_copy(0, at, s[name + "_new"].double().index_select(0, cells))
            want[name + "_cache"] = tokens.unflatten(0, (-1, case["page"])).transpose(1, 2)
        return want
    q, kc, vc = s["q"], s["k_cache"], s["v_cache"]
    T, Hq, D = q.shape
    Hk, page = kc.shape[1], case["page"]
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=DEV)
    _, new, kv = _lengths(case)
    first = 0
    for b, (n, L) in enumerate(zip(new, kv)):
        if n and L:
            ids = s["block_table"][b, :-(-L // page)].long()
            for h in range(Hk):
                K = kc[ids, h].reshape(-1, D)[:L].double()
                V = vc[ids, h].reshape(-1, D)[:L].double()
                heads = slice(h * (Hq // Hk), (h + 1) * (Hq // Hk))
                for t in range(0, n, 1024):
                    m = min(1024, n - t)
                    x = torch.einsum("tgd,ld->tgl", q[first + t:first + t + m, heads].double(), K) * case["D"] ** -0.5
                    last = torch.arange(t, t + m, device=DEV) + (L - n)
                    x[(torch.arange(L, device=DEV)[None] > last[:, None])[:, None].expand_as(x)] = -math.inf
                    z = torch.logsumexp(x, -1)
                    w = torch.exp(x - torch.where(z.isinf(), 0.0, z)[..., None])
                    out[first + t:first + t + m, heads] = torch.einsum("tgl,ld->tgd", w, V)
                    lse[first + t:first + t + m, heads] = z
        first += n
    return dict(out=out, lse=lse)
