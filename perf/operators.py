"""Cases of the paged decoding step's operators: the tables of the paged cache, rotary positions
with the cache write, and the attention of a batch over a shared prefix.

`run` computes each of them in elementary torch operations (`own` false) or through the
framework's entry points (`own` true); `exact` gives the same outputs from the definitions in 64
bits. A case is a dict with an "op" of
  tables   page tables, slots and positions of a step's new tokens, from request lengths
  rope     rotary positions of Q and K
  write    rotary positions of Q and K, K and V rows written into the E4M3 cache
  prefix   attention of drafted tokens over a prefix shared by the batch and their own suffixes
"""
import math

import torch

own = False

HEAD_DIM = 256
E4M3_MAX = 448.0
# (query heads, KV heads): one tensor-parallel rank of the drafted-block shape, and all its heads
RANK, MODEL = (6, 1), (24, 4)


# ---------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step of a small batch: eight drafted tokens each, the call is all latency
        dict(name="tables_step_b4_q8", op="tables", batch=4, new="draft", max_new=8, page=16,
             max_context=32768, prefix=0),
        # the same step of a loaded server with long rows
        dict(name="tables_step_b1000_q8", op="tables", batch=1000, new="draft", max_new=8, page=16,
             max_context=32768, prefix=0),
        # prompts of very different lengths admitted at once behind one shared system prompt
        dict(name="tables_prompts_b93", op="tables", batch=93, new="prompt", max_new=8191, page=64,
             max_context=65536, prefix=2048),
        # Q and K of a few drafted blocks, no cache behind them
        dict(name="rope_b5_q8_interleaved", op="rope", tokens=40, heads="model", rotary=256,
             layout="interleaved", scaling="none", dtype="fp16", far=262144, fused_qkv=False),
        # Q and K of long prompts in bf16, a quarter of the head, positions past the trained length
        dict(name="rope_prompt_part", op="rope", tokens=24571, heads="model", rotary=64,
             layout="half", scaling="yarn", dtype="bf16", far=1048576, fused_qkv=True),
        # the drafted block of one sequence on one rank
        dict(name="write_rank_b1_q8", op="write", tokens=8, heads="rank", rotary=256, layout="half",
             scaling="none", dtype="fp16", far=262144, fused_qkv=False, page=16),
        # drafted blocks of 64 sequences, all heads, a stretched context, interleaved pairs
        dict(name="write_b64_q8", op="write", tokens=512, heads="model", rotary=128,
             layout="interleaved", scaling="linear", dtype="fp16", far=262144, fused_qkv=True,
             page=16),
        # a packed prompt batch of odd length out of one fused projection, with padding tokens
        dict(name="write_prompt_packed", op="write", tokens=16381, heads="model", rotary=256,
             layout="half", scaling="yarn", dtype="fp16", far=131072, fused_qkv=True, page=64),
        # three short continuations of one prompt on one rank: latency
        dict(name="prefix_rank_b3_q8", op="prefix", batch=3, q_len=8, heads="rank", prefix=4099,
             suffix=200, page=16, peaked=False, empty=False),
        # single-token decoding of 32 requests behind one long document
        dict(name="prefix_b32_q1", op="prefix", batch=32, q_len=1, heads="model", prefix=65536,
             suffix=1000, page=16, peaked=False, empty=False),
        # drafted blocks of 16 requests, a padded batch slot among them, peaked scores
        dict(name="prefix_b16_q8", op="prefix", batch=16, q_len=8, heads="model", prefix=32768,
             suffix=2048, page=16, peaked=True, empty=True),
        # the largest: 40 requests, 131000 shared tokens, pages that do not divide them
        dict(name="prefix_b40_q8", op="prefix", batch=40, q_len=8, heads="model", prefix=131000,
             suffix=4000, page=64, peaked=False, empty=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "rope", "write", "prefix", "prefix"])
    if op == "tables":
        page = rng.choice([16, 32, 48, 64])
        if rng.random() < 0.5:
            return dict(op=op, batch=_log(rng, 1, 1000), new="draft", max_new=rng.randint(1, 16),
                        page=page, max_context=_log(rng, 2048, 32768),
                        prefix=rng.choice([0, _log(rng, 17, 1500)]))
        return dict(op=op, batch=_log(rng, 1, 93), new="prompt", max_new=_log(rng, 100, 8191),
                    page=page, max_context=_log(rng, 16384, 65536),
                    prefix=rng.choice([0, _log(rng, 17, 4096)]))
    if op in ("rope", "write"):
        case = dict(op=op, tokens=_log(rng, 1, 16381), heads=rng.choice(["rank", "model"]),
                    rotary=16 * rng.randint(1, 16), layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn", "wavelength"]),
                    dtype=rng.choice(["fp16", "bf16"]), far=_log(rng, 20000, 1048576),
                    fused_qkv=rng.random() < 0.5)
        if op == "write":
            case["page"] = rng.choice([16, 32, 48, 64])
        return case
    return dict(op=op, batch=_log(rng, 2, 40), q_len=rng.choice([1, 2, 4, 5, 8]),
                heads=rng.choice(["rank", "model"]), prefix=_log(rng, 300, 120000),
                suffix=_log(rng, 16, 3500), page=rng.choice([16, 32, 48, 64]),
                peaked=rng.random() < 0.3, empty=rng.random() < 0.3)


def _heads(case):
    return RANK if case["heads"] == "rank" else MODEL


def _dtype(case):
    return torch.bfloat16 if case.get("dtype") == "bf16" else torch.float16


# --------------------------------------------------------------------------- what a user has

# Rotary frequencies. theta_i = base^(-2i/d) for pair i of d rotated elements, and for contexts
# longer than the trained one: all divided by the factor (linear); a larger base (ntk); divided
# only where a pair turns few times over the trained length, with a ramp between and the cosine
# and sine scaled by 0.1 ln(factor) + 1 (yarn); or the same by wavelength, no scaling (wavelength).
ROPE = dict(base=500000.0, factor=8.0, trained=32768, beta_fast=32.0, beta_slow=1.0, low=1.0,
            high=4.0)


def _frequencies(d, scaling):
    p = ROPE
    i = torch.arange(d // 2, dtype=torch.float64)
    base, s, trained = p["base"], p["factor"], p["trained"]
    if scaling == "ntk":
        base = base * s ** (d / (d - 2)) if d > 2 else base
    theta = base ** (-2.0 * i / d)
    if scaling == "linear":
        theta = theta / s
    elif scaling == "yarn":
        def pair(turns):  # the pair that turns so often over the trained length
            return d * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))
        low = max(math.floor(pair(p["beta_fast"])), 0)
        high = min(math.ceil(pair(p["beta_slow"])), d - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        theta = theta / s * ramp + theta * (1 - ramp)
    elif scaling == "wavelength":
        turns = trained * theta / (2 * math.pi)
        mix = ((turns - p["low"]) / (p["high"] - p["low"])).clamp(0, 1)
        theta = theta / s * (1 - mix) + theta * mix
    return theta, (0.1 * math.log(s) + 1.0 if scaling == "yarn" else 1.0)


def _rotary_handle(case, num_pages, page):
    from speculative_verify_paged_e4m3_gb300 import binding
    Hq, Hkv = _heads(case)
    return binding.Rotary(Hq, Hkv, HEAD_DIM, case["rotary"], layout=case["layout"],
                          dtype=_dtype(case), base=ROPE["base"], scaling=case["scaling"],
                          factor=ROPE["factor"], trained_context=ROPE["trained"],
                          beta_fast=ROPE["beta_fast"], beta_slow=ROPE["beta_slow"],
                          low_turns=ROPE["low"], high_turns=ROPE["high"], page_size=page,
                          num_pages=num_pages)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _ints(g, lo, hi, n):
    """n int32 in [lo, hi]."""
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)


def prepare(case, seed):
    return dict(tables=_prepare_tables, rope=_prepare_rope, write=_prepare_rope,
                prefix=_prepare_prefix)[case["op"]](case, _gen(seed))


def _prepare_tables(case, g):
    B, P, prefix = case["batch"], case["page"], case["prefix"]
    max_pages = -(-case["max_context"] // P)
    max_ctx = max_pages * P
    if case["new"] == "draft":  # running requests: cached tokens, one drafted block each
        room = max_ctx - case["max_new"]
        cached = _ints(g, min(prefix, room), room, B)
        new = torch.full((B,), case["max_new"], dtype=torch.int32, device="cuda")
        held = (cached + P - 1) // P + _ints(g, 0, 1, B)  # a rejected draft may leave a page
        held = held.clamp(max=max_pages)
    else:  # fresh prompts behind the shared prefix (whole pages of it); some are long
        shared = min(prefix, max_ctx // 2) // P * P
        cached = torch.full((B,), shared, dtype=torch.int32, device="cuda")
        top = min(case["max_new"], max_ctx - shared)
        u = torch.rand((B,), generator=g, device="cuda")
        new = (top * u * u).to(torch.int32).clamp(min=1)
        held = torch.zeros((B,), dtype=torch.int32, device="cuda")
    max_tokens = B * case["max_new"]
    n_free = B * (-(-case["max_new"] // P) + 1) + 5
    num_pages = B * max_pages + n_free
    order = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    table = order[:B * max_pages].view(B, max_pages).clone()
    lp = torch.arange(max_pages, device="cuda", dtype=torch.int32)
    table = torch.where(lp < held[:, None], table, -1)
    i32 = dict(dtype=torch.int32, device="cuda")
    state = dict(case=case, cached=cached, new=new, held=held, table=table,
                 free=order[B * max_pages:].contiguous(),
                 head=torch.tensor([3], **i32),
                 prefix_table=order[:max(1, prefix // P)].contiguous(),
                 prefix_pages=torch.tensor([prefix // P], **i32),
                 max_tokens=max_tokens, max_ctx=max_ctx)
    if own:
        from speculative_verify_paged_e4m3_gb300 import binding
        state["tables"] = binding.PagedTables(B, P, max_pages, num_pages, max_ctx, max_tokens)
        state["out"] = state["tables"].empty()
    return state


def _prepare_rope(case, g):
    (Hq, Hkv), T, D, dt = _heads(case), case["tokens"], HEAD_DIM, _dtype(case)
    if case["fused_qkv"]:  # slices of one projection's output
        qkv = torch.randn((T, (Hq + 2 * Hkv), D), generator=g, device="cuda").to(dt)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        q, k, v = (torch.randn((T, h, D), generator=g, device="cuda").to(dt)
                   for h in (Hq, Hkv, Hkv))
    pos = _ints(g, 0, case["far"] - 1, T)
    state = dict(case=case, q=q, k=k, v=v, pos=pos, q_out=torch.empty((T, Hq, D), dtype=dt,
                                                                      device="cuda"))
    theta, amp = _frequencies(case["rotary"], case["scaling"])
    state.update(theta=theta.cuda(), amp=amp)
    if case["op"] == "rope":
        state["k_out"] = torch.empty((T, Hkv, D), dtype=dt, device="cuda")
        num_pages, page = 1, 16
    else:
        page = case["page"]
        num_pages = -(-T // page) + 3
        slots = torch.randperm(num_pages * page, generator=g, device="cuda")[:T]
        if T > 64:  # padding tokens of a packed batch: nothing of theirs is written
            pad = torch.rand((T,), generator=g, device="cuda") < 0.01
            slots = torch.where(pad, -1, slots)
            state["q_out"].zero_()
        scale = 4.5 / E4M3_MAX  # calibrated once: a few values saturate
        shape = (num_pages, page, Hkv, D)
        for n in ("k_pool", "v_pool"):
            x = torch.randn(shape, generator=g, device="cuda") / scale
            state[n] = x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        state.update(slots=slots, k_scale=torch.full((1,), scale, device="cuda"),
                     v_scale=torch.full((1,), 1.25 * scale, device="cuda"))
    if own:
        state["rotary"] = _rotary_handle(case, num_pages, page)
    return state


def _prepare_prefix(case, g):
    (Hq, Hkv), D, P = _heads(case), HEAD_DIM, case["page"]
    B, q_len, prefix = case["batch"], case["q_len"], case["prefix"]
    lens = prefix + q_len + _ints(g, 0, case["suffix"], B)
    lens[0] = prefix + q_len + case["suffix"]
    if case["empty"]:
        lens[B // 2] = 0  # a slot of the batch that holds no request
    shared = prefix // P
    max_ctx = prefix + q_len + case["suffix"]
    max_pages = -(-max_ctx // P)
    private = max_pages - shared
    num_pages = shared + B * private
    order = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.empty((B, max_pages), dtype=torch.int32, device="cuda")
    table[:, :shared] = order[:shared]
    table[:, shared:] = order[shared:].view(B, private)
    # the page that the prefix ends in is every request's own copy: equal keys and values
    pools, scales = [], []
    for peaked in (case["peaked"], False):
        scale = (16.0 if peaked else 5.2) / E4M3_MAX
        x = torch.randn((num_pages, P, Hkv, D), generator=g, device="cuda")
        if peaked:  # some keys that draw most of the attention
            u = torch.rand((num_pages, P, 1, 1), generator=g, device="cuda")
            x = torch.where(u < 0.05, 4.0 * x, x)
        x = (x / scale).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        if prefix % P:
            x[table[:, shared].long(), :prefix % P] = x[table[0, shared].long(), :prefix % P]
        pools.append(x)
        scales.append(torch.full((1,), scale, device="cuda"))
    q = torch.randn((B, q_len, Hq, D), generator=g, device="cuda").to(torch.float16)
    one = dict(dtype=torch.int32, device="cuda")
    state = dict(case=case, q=q, k_pool=pools[0], v_pool=pools[1], table=table,
                 prefix_table=order[:max(1, shared)].contiguous(), max_ctx=max_ctx,
                 prefix_len=torch.tensor([prefix], **one), lens=lens,
                 k_scale=scales[0], v_scale=scales[1],
                 out=torch.empty((B, q_len, Hq, D), dtype=torch.float16, device="cuda"),
                 lse=torch.empty((B, q_len, Hq), dtype=torch.float32, device="cuda"))
    if own:
        from speculative_verify_paged_e4m3_gb300 import binding
        state["att"] = binding.SharedPrefixAttention(B, q_len, Hq, Hkv, D, P, max_pages, num_pages,
                                                     max_ctx, max_prefix=prefix)
    return state


# ------------------------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return dict(tables=_own_tables, rope=_own_rope, write=_own_write,
                    prefix=_own_prefix)[op](state)
    return dict(tables=_plain_tables, rope=_plain_rope, write=_plain_write,
                prefix=_plain_prefix)[op](state)


def _own_tables(s):
    shared = s["case"]["prefix"] > 0
    out = s["tables"](s["cached"], s["new"], s["held"], s["free"], s["head"], s["table"],
                      prefix_table=s["prefix_table"] if shared else None,
                      prefix_pages=s["prefix_pages"] if shared else None, out=s["out"])
    return dict(table=s["table"], context_lens=out.context_lens, held=out.held_pages,
                head=out.free_head, starts=out.token_starts, positions=out.positions,
                slots=out.slots)


def _own_rope(s):
    s["rotary"].apply(s["q"], s["k"], s["pos"], q_out=s["q_out"], k_out=s["k_out"])
    return dict(q=s["q_out"], k=s["k_out"])


def _own_write(s):
    s["rotary"].kv_write(s["q"], s["k"], s["v"], s["pos"], s["slots"], s["k_scale"], s["v_scale"],
                         s["k_pool"], s["v_pool"], q_out=s["q_out"])
    return dict(q=s["q_out"], k_pool=s["k_pool"].view(torch.float8_e4m3fn),
                v_pool=s["v_pool"].view(torch.float8_e4m3fn))


def _own_prefix(s):
    s["att"](s["q"], s["k_pool"], s["v_pool"], s["prefix_table"], s["prefix_len"], s["table"],
             s["lens"], s["k_scale"], s["v_scale"], out=s["out"], lse=s["lse"])
    return dict(out=s["out"], lse=s["lse"])


def _plain_tables(s):
    """Pages [held, need) of each row come from the shared prefix's table, then from the free
    list in request order; token i of request b sits at position cached + i."""
    P, max_pages = s["case"]["page"], s["table"].shape[1]
    cached, new, held = s["cached"].long(), s["new"].long(), s["held"].long()
    ctx = cached + new
    need = torch.maximum((ctx + P - 1) // P, held)
    shared = s["prefix_pages"].long() if s["case"]["prefix"] > 0 else torch.zeros_like(cached[:1])
    first = torch.minimum(torch.maximum(held, shared), need)  # first page off the free list
    take = need - first
    before = torch.cumsum(take, 0) - take
    lp = torch.arange(max_pages, device="cuda")
    at = (s["head"].long() + before)[:, None] + lp - first[:, None]
    fresh = s["free"][at.clamp(0, s["free"].numel() - 1)]
    pre = s["prefix_table"][lp.clamp(max=s["prefix_table"].numel() - 1)]
    fill = torch.where(lp < shared, pre, fresh)
    mine = (lp >= held[:, None]) & (lp < need[:, None])
    s["table"].copy_(torch.where(mine, fill, s["table"]))
    starts = torch.cat([torch.zeros_like(new[:1]), torch.cumsum(new, 0)])
    t = torch.arange(s["max_tokens"], device="cuda")
    b = (torch.searchsorted(starts, t, right=True) - 1).clamp(max=new.numel() - 1)
    live = t < starts[-1]
    pos = cached[b] + t - starts[b]
    pos = torch.where(live, pos, 0)
    page = s["table"][b, (pos // P).clamp(max=max_pages - 1)].long()
    # shared pages are read only: their tokens have no slot
    slots = torch.where(live & (pos >= shared * P), page * P + pos % P, -1)
    i32 = torch.int32
    return dict(table=s["table"], context_lens=ctx.to(i32), held=need.to(i32),
                head=(s["head"].long() + take.sum()).to(i32), starts=starts.to(i32),
                positions=pos.to(i32), slots=slots)


def _rotated(x, cos, sin, d, layout):
    """x [T, H, D] in fp32 with its first d elements rotated; cos, sin [T, 1, d / 2]."""
    r, rest = x[..., :d], x[..., d:]
    if layout == "half":
        a, b = r[..., :d // 2], r[..., d // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([r, rest], -1)


def _turned(s):
    """Q and K of the state rotated, in fp32; angles of far positions need 64 bits."""
    c = s["case"]
    angle = s["pos"].double()[:, None, None] * s["theta"]
    cos, sin = (f(angle).float() * s["amp"] for f in (torch.cos, torch.sin))
    return tuple(_rotated(s[n].float(), cos, sin, c["rotary"], c["layout"]) for n in ("q", "k"))


def _plain_rope(s):
    q, k = _turned(s)
    s["q_out"].copy_(q)
    s["k_out"].copy_(k)
    return dict(q=s["q_out"], k=s["k_out"])


def _plain_write(s):
    q, k = _turned(s)
    live = s["slots"] >= 0
    s["q_out"].copy_(torch.where(live[:, None, None], q.to(s["q_out"].dtype), s["q_out"]))
    rows = s["k_pool"].shape[0] * s["k_pool"].shape[1]
    at = torch.where(live, s["slots"], rows)  # padding goes to a row behind the pool
    res = dict(q=s["q_out"])
    for name, x, scale in (("k_pool", k, s["k_scale"]), ("v_pool", s["v"].float(), s["v_scale"])):
        code = (x / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        pool = s[name].view((rows,) + tuple(code.shape[1:]))
        grown = torch.cat([pool, pool[:1]])
        grown[at] = code
        pool.copy_(grown[:rows])
        res[name] = s[name].view(torch.float8_e4m3fn)
    return res


def _plain_prefix(s):
    c, q = s["case"], s["q"]
    (Hq, Hkv), P, D = _heads(c), c["page"], HEAD_DIM
    B, q_len, G = c["batch"], c["q_len"], Hq // Hkv
    n_shared = c["prefix"] // P  # whole pages; the prefix's last tokens are in the rows' own
    own_pages = s["table"].shape[1] - n_shared

    def rows(pool, pages, scale):  # [..., pages] -> [..., pages * P, Hkv, D]
        x = pool.view(torch.float8_e4m3fn)[pages.long()].float() * scale
        return x.flatten(-4, -3)

    qf = q.float().view(B, q_len, Hkv, G, D) / math.sqrt(D)
    pre, suf = s["prefix_table"][:n_shared], s["table"][:, n_shared:]
    sc = torch.cat([
        torch.einsum("bihgd,jhd->bihgj", qf, rows(s["k_pool"], pre, s["k_scale"])),
        torch.einsum("bihgd,bjhd->bihgj", qf, rows(s["k_pool"], suf, s["k_scale"]))], -1)
    j = torch.arange((n_shared + own_pages) * P, device="cuda")
    last = s["lens"][:, None] - q_len + torch.arange(q_len, device="cuda")  # last visible key
    seen = j <= last[..., None]
    sc = torch.where(seen[:, :, None, None], sc, -math.inf)
    top = sc.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(sc - top)
    total = p.sum(-1)
    cut = n_shared * P
    o = torch.einsum("bihgj,jhd->bihgd", p[..., :cut], rows(s["v_pool"], pre, s["v_scale"]))
    o += torch.einsum("bihgj,bjhd->bihgd", p[..., cut:], rows(s["v_pool"], suf, s["v_scale"]))
    o = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
    s["out"].copy_(o.view(B, q_len, Hq, D))
    s["lse"].copy_((top[..., 0] + torch.log(total)).view(B, q_len, Hq))
    return dict(out=s["out"], lse=s["lse"])


# ------------------------------------------------------------------------------------ its work

def work(case):
    op, D = case["op"], HEAD_DIM
    if op == "tables":
        B, P = case["batch"], case["page"]
        # three lengths in, two lengths and the token starts out, page entries in and out, a
        # position and a slot per new token (about a third of max_new on average for prompts)
        new = B * case["max_new"] if case["new"] == "draft" else B * case["max_new"] // 3
        return dict(bytes=B * 24 + 8 * (new // P + B) + 4 * B * case["max_new"]
                    + 8 * B * case["max_new"], flops=10 * B * case["max_new"])
    if op in ("rope", "write"):
        (Hq, Hkv), T = _heads(case), case["tokens"]
        turned = 6 * T * (Hq + Hkv) * case["rotary"] // 2
        if op == "rope":
            return dict(bytes=T * (4 + 4 * (Hq + Hkv) * D), flops=turned)
        return dict(bytes=T * (12 + 4 * Hq * D + 2 * Hkv * D * 3),
                    flops=turned + 2 * T * Hkv * D)
    (Hq, Hkv), B, q_len = _heads(case), case["batch"], case["q_len"]
    rows = B * q_len * Hq
    private = case["suffix"] / 2 + q_len
    keys = case["prefix"] + B * private
    return dict(bytes=2 * keys * Hkv * D + rows * (4 * D + 4) + 4 * keys / case["page"],
                flops=4 * D * rows * (case["prefix"] + private))


# --------------------------------------------------------------------- the definitions, 64 bits

def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers
    s = prepare(case, seed)
    return _exact_prefix(s) if case["op"] == "prefix" else _exact_rope(s)


def _exact_rope(s):
    """Pair (x, y) as the complex number x + iy, turned by amp e^(i pos theta)."""
    c = s["case"]
    d, half = c["rotary"], c["rotary"] // 2
    angle = torch.outer(s["pos"].double(), s["theta"])
    turn = torch.polar(torch.full_like(angle, s["amp"]), angle)[:, None]
    first = torch.arange(half, device="cuda") * (1 if c["layout"] == "half" else 2)
    second = first + (half if c["layout"] == "half" else 1)
    res = {}
    for name in ("q", "k"):
        x = s[name].double()
        z = torch.complex(x[..., first], x[..., second]) * turn
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        res[name] = y
    if c["op"] == "rope":
        return res
    out = dict(q=s["q_out"].double())
    live = s["slots"] >= 0
    out["q"][live] = res["q"][live]
    for name, x, scale in (("k_pool", res["k"], s["k_scale"]), ("v_pool", s["v"].double(),
                                                                s["v_scale"])):
        pool = s[name].view(torch.float8_e4m3fn).double()
        flat = pool.view(-1, *pool.shape[2:])
        flat[s["slots"][live]] = (x[live] / scale.double()).clamp(-E4M3_MAX, E4M3_MAX)
        out[name] = pool
    return out


def _exact_prefix(s):
    """Request by request over its whole row of pages, the prefix like any other keys."""
    c, D, P = s["case"], HEAD_DIM, s["case"]["page"]
    Hq, Hkv = _heads(c)
    G, q_len = Hq // Hkv, c["q_len"]
    out, lse = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), torch.full(
        s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    kp, vp = (s[n].view(torch.float8_e4m3fn) for n in ("k_pool", "v_pool"))
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        pages = s["table"][b, :-(-n // P)].long()
        k, v = ((p[pages].flatten(0, 1)[:n].double() * sc.double()).transpose(0, 1)
                for p, sc in ((kp, s["k_scale"]), (vp, s["v_scale"])))  # [Hkv, n, D]
        q = s["q"][b].double().view(q_len, Hkv, G, D).permute(1, 0, 2, 3).reshape(Hkv, -1, D)
        x = torch.bmm(q, k.transpose(1, 2)) / 16.0
        last = n - q_len + torch.arange(q_len, device="cuda").repeat_interleave(G)
        x.masked_fill_(torch.arange(n, device="cuda") > last[:, None], -math.inf)
        z = torch.logsumexp(x, -1)
        o = torch.bmm(torch.exp(x - z[..., None]), v).view(Hkv, q_len, G, D)
        out[b] = o.permute(1, 0, 2, 3).reshape(q_len, Hq, D)
        lse[b] = z.view(Hkv, q_len, G).permute(1, 0, 2).reshape(q_len, Hq)
    return dict(out=out, lse=lse)
