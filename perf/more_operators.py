"""Cases of a decoding step over a cache held in 4 bits: norms of the heads of Q and K with the
rotary positions in the same pass, keys and values appended to the cache, cached tokens read back,
and the attention of drafted tokens over the cache.

`run` computes each of them in elementary torch operations (`own` false) or through the
framework's entry points (`own` true); `exact` gives the same outputs from the definitions in 64
bits. A case is a dict with an "op" of
  norm    head norms and rotary positions of Q and K
  write   the same, K and V rows written into the paged cache ("cache": mx4, or e4m3)
  read    tokens of the 4-bit cache as numbers
  attn    attention of drafted tokens over the 4-bit cache

The 4-bit format: 32 elements of a head share a power of two 2^e, the smallest with max |x| <= 7 * 2^e,
and each is the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 times it (ties to the even code), with its
sign. A pool is [pages, page_size / 16, KV heads, 2176 bytes]: 16 tokens' codes (2048) and scale
bytes e + 127 (16 x 8).
"""
import math

import torch

own = False

HEAD_DIM = 256
E4M3_MAX = 448.0
CHUNK, CHUNK_BYTES, CODE_BYTES = 16, 2176, 2048
# (query heads, KV heads): one tensor-parallel rank of the drafted-block shape, and all its heads
RANK, MODEL = (6, 1), (24, 4)
ROPE_BASE = 500000.0
EPS = 1e-6


# ---------------------------------------------------------------------------------------- cases

def listed():
    return [
        # Q and K of a few drafted blocks, no cache behind them: the call is all latency
        dict(name="norm_b5_q8_interleaved", op="norm", tokens=40, heads="model", rotary=256,
             layout="interleaved", dtype="fp16", offset=0.0, fused_qkv=False, far=262144),
        # Q and K of long prompts in bf16, a quarter of the head turned, weights kept about zero
        dict(name="norm_prompt_part", op="norm", tokens=24571, heads="model", rotary=64,
             layout="half", dtype="bf16", offset=1.0, fused_qkv=True, far=1048576),
        # drafted blocks of 64 sequences into the 8-bit cache
        dict(name="write_e4m3_b64_q8", op="write", cache="e4m3", tokens=512, heads="model",
             rotary=128, layout="interleaved", dtype="fp16", offset=1.0, fused_qkv=True,
             far=262144, page=16),
        # the drafted block of one sequence on one rank
        dict(name="write_mx4_rank_b1_q8", op="write", cache="mx4", tokens=8, heads="rank",
             rotary=256, layout="half", dtype="fp16", offset=0.0, fused_qkv=False, far=262144,
             page=16),
        # one new token of each of 61 requests, all heads
        dict(name="write_mx4_b61_q1", op="write", cache="mx4", tokens=61, heads="model", rotary=64,
             layout="half", dtype="bf16", offset=1.0, fused_qkv=True, far=262144, page=64),
        # a packed prompt batch of odd length out of one fused projection, with padding tokens
        dict(name="write_mx4_prompt_packed", op="write", cache="mx4", tokens=16381, heads="model",
             rotary=256, layout="half", dtype="fp16", offset=0.0, fused_qkv=True, far=131072,
             page=64),
        # a few pages of one rank, to be looked at or sent on
        dict(name="read_rank_pages", op="read", tokens=83, heads="rank", page=16, dtype="fp16"),
        # the whole context of a request that moves to another server
        dict(name="read_context", op="read", tokens=65521, heads="model", page=64, dtype="bf16"),
        # three short sequences of one rank: latency
        dict(name="attn_rank_b3_q8", op="attn", batch=3, q_len=8, heads="rank", context=4107,
             page=16, peaked=False, empty=False),
        # the longest context on one rank, one drafted block
        dict(name="attn_rank_b1_q8_long", op="attn", batch=1, q_len=8, heads="rank",
             context=261888, page=16, peaked=False, empty=False),
        # single-token decoding of a loaded server, ragged lengths, one padded slot
        dict(name="attn_b32_q1", op="attn", batch=32, q_len=1, heads="model", context=16384,
             page=16, peaked=False, empty=True),
        # the largest: drafted blocks of four long requests, peaked scores, pages of 64
        dict(name="attn_b4_q8", op="attn", batch=4, q_len=8, heads="model", context=65536,
             page=64, peaked=True, empty=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "write", "write", "read", "attn", "attn", "attn"])
    heads = rng.choice(["rank", "model"])
    if op == "read":
        return dict(op=op, tokens=_log(rng, 1, 65521), heads=heads,
                    page=rng.choice([16, 32, 48, 64]), dtype=rng.choice(["fp16", "bf16"]))
    if op in ("norm", "write"):
        case = dict(op=op, tokens=_log(rng, 1, 16381), heads=heads, rotary=16 * rng.randint(1, 16),
                    layout=rng.choice(["half", "interleaved"]),
                    dtype=rng.choice(["fp16", "bf16"]), offset=rng.choice([0.0, 1.0]),
                    fused_qkv=rng.random() < 0.5, far=_log(rng, 20000, 1048576))
        if op == "write":
            case.update(cache=rng.choice(["mx4", "mx4", "e4m3"]), page=rng.choice([16, 32, 48, 64]))
        return case
    batch = _log(rng, 1, 32)
    keys = rng.choice([262144, 262144 // 4])  # the batch's at most: a drawn case costs no more
    return dict(op=op, batch=batch, q_len=rng.choice([1, 2, 3, 4, 5, 8]), heads=heads,
                context=_log(rng, 40, max(80, keys // batch)), page=rng.choice([16, 32, 48, 64]),
                peaked=rng.random() < 0.3, empty=batch > 1 and rng.random() < 0.3)


def _heads(case):
    return RANK if case["heads"] == "rank" else MODEL


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float16


# ------------------------------------------------------------------------------ the 4-bit format

def _codes(x):
    """x [..., 256] as 4-bit codes [..., 256] and scale bytes [..., 8] (uint8 both)."""
    blocks = x.unflatten(-1, (8, 32))
    top = blocks.abs().amax(-1)
    mant, expo = torch.frexp(top)  # top = mant 2^expo, mant in [0.5, 1)
    e = torch.where(top > 0, expo - 3 + (mant > 0.875), -127).clamp(-127, 127)
    y = torch.ldexp(blocks.abs(), -e[..., None])
    code = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5)
            + (y >= 3.5) + (y > 5.0)).to(torch.uint8)
    code = code + 8 * (blocks < 0).to(torch.uint8)
    return code.flatten(-2), (e + 127).to(torch.uint8)


def _packed(code, scale, of_v):
    """The 136 bytes of each row of codes: a token's in a chunk, in the order of _offsets."""
    if of_v:  # elements e and e + 128 in a byte
        b = code[..., :128] | (code[..., 128:] << 4)
    else:  # elements 2i and 2i + 1
        b = code[..., 0::2] | (code[..., 1::2] << 4)
    return torch.cat([b, scale], -1)


def _offsets(slot, of_v):
    """Where in its chunk the 136 bytes of each slot's token lie: [..., 136]."""
    tok = (slot % CHUNK)[..., None]
    i = torch.arange(128, device=slot.device)
    j = torch.arange(8, device=slot.device)
    at = i * CHUNK + tok if of_v else i // 16 * 256 + tok * 16 + i % 16
    return torch.cat([at, CODE_BYTES + tok * 8 + j], -1)


def _whole_pool(code, scale, num_pages, page, of_v):
    """A pool from codes [tokens, Hkv, 256] and scales [tokens, Hkv, 8] of all its slots in order."""
    T, H = code.shape[:2]
    rows = _packed(code, scale, of_v).view(T // CHUNK, CHUNK, H, 136).transpose(1, 2)
    b, s = rows[..., :128], rows[..., 128:]  # [chunks, H, 16, .]
    if of_v:
        b = b.transpose(2, 3)
    else:
        b = b.unflatten(-1, (8, 16)).transpose(2, 3)
    pool = torch.cat([b.flatten(2), s.flatten(2)], -1)
    return pool.view(num_pages, page // CHUNK, H, CHUNK_BYTES).contiguous()


def _numbers(chunks, of_v, dtype):
    """The numbers of chunks [..., 2176] (uint8): [..., 16 tokens, 256]."""
    b = chunks[..., :CODE_BYTES]
    s = chunks[..., CODE_BYTES:].unflatten(-1, (CHUNK, 8)).to(torch.int32)
    if of_v:
        b = b.unflatten(-1, (128, CHUNK)).transpose(-1, -2)
        code = torch.cat([b & 15, b >> 4], -1)
    else:
        b = b.unflatten(-1, (8, CHUNK, 16)).transpose(-2, -3).flatten(-2)
        code = torch.stack([b & 15, b >> 4], -1).flatten(-2)
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6],
                        device=chunks.device, dtype=dtype)
    x = grid[code.int()].unflatten(-1, (8, 32))
    power = (s.clamp(1, 254) << 23).view(torch.float32).to(dtype)  # 2^(s - 127)
    return (x * power[..., None]).flatten(-2)


# --------------------------------------------------------------------------- what a user has

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _ints(g, lo, hi, n):
    """n int32 in [lo, hi]."""
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)


def prepare(case, seed):
    return dict(norm=_prepare_rows, write=_prepare_rows, read=_prepare_read,
                attn=_prepare_attn)[case["op"]](case, _gen(seed))


def _prepare_rows(case, g):
    (Hq, Hkv), T, D, dt = _heads(case), case["tokens"], HEAD_DIM, _dtype(case)
    if case["fused_qkv"]:  # slices of one projection's output
        qkv = (3.0 * torch.randn((T, Hq + 2 * Hkv, D), generator=g, device="cuda")).to(dt)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        q, k, v = ((3.0 * torch.randn((T, h, D), generator=g, device="cuda")).to(dt)
                   for h in (Hq, Hkv, Hkv))
    w = 1.0 + 0.3 * torch.randn((2, D), generator=g, device="cuda") - case["offset"]
    theta = ROPE_BASE ** (-2.0 * torch.arange(case["rotary"] // 2, dtype=torch.float64)
                          / case["rotary"])
    state = dict(case=case, q=q, k=k, v=v, pos=_ints(g, 0, case["far"] - 1, T),
                 q_weight=w[0].to(dt), k_weight=w[1].to(dt), theta=theta.cuda(),
                 q_out=torch.zeros((T, Hq, D), dtype=dt, device="cuda"))
    num_pages, page = 1, 16
    if case["op"] == "norm":
        state["k_out"] = torch.empty((T, Hkv, D), dtype=dt, device="cuda")
    else:
        page = case["page"]
        num_pages = -(-T // page) + 3
        n = num_pages * page
        # a token's slot is the one after the last one's until its page ends; pages in any order
        order = torch.randperm(num_pages, generator=g, device="cuda")
        at = torch.arange(T, device="cuda") + 5
        slots = order[at // page] * page + at % page
        if T > 64:  # padding tokens of a packed batch: nothing of theirs is written
            pad = torch.rand((T,), generator=g, device="cuda") < 0.01
            slots = torch.where(pad, -1, slots)
        state["slots"] = slots
        old = [torch.randn((n, Hkv, D), generator=g, device="cuda") for _ in range(2)]
        if case["cache"] == "e4m3":
            scale = 4.5 / E4M3_MAX  # calibrated once: a few values saturate
            state["k_pool"], state["v_pool"] = (
                (x / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
                .view(num_pages, page, Hkv, D) for x in old)
            state.update(k_scale=torch.full((1,), scale, device="cuda"),
                         v_scale=torch.full((1,), 3.0 * scale, device="cuda"))
        else:
            state["k_pool"] = _whole_pool(*_codes(old[0]), num_pages, page, False)
            state["v_pool"] = _whole_pool(*_codes(old[1]), num_pages, page, True)
            e5m2 = dict(dtype=torch.float8_e5m2, device="cuda")
            state.update(all_slots=torch.arange(n, device="cuda"),
                         k_held=torch.empty((n, Hkv, D), **e5m2),
                         v_held=torch.empty((n, Hkv, D), **e5m2))
    if own:
        from speculative_verify_paged_e4m3_gb300 import binding
        state["rotary"] = binding.Rotary(Hq, Hkv, D, case["rotary"], layout=case["layout"],
                                         dtype=dt, base=ROPE_BASE, page_size=page,
                                         num_pages=num_pages)
        state["norm"] = binding.HeadNorm(state["q_weight"], state["k_weight"], EPS, case["offset"])
        state["cache"] = binding.Mx4Cache(Hkv, D, page, num_pages)
    return state


def _prepare_read(case, g):
    (_, Hkv), T, D, page = _heads(case), case["tokens"], HEAD_DIM, case["page"]
    num_pages = -(-T // page) + 3
    order = torch.randperm(num_pages, generator=g, device="cuda")
    at = torch.arange(T, device="cuda")
    state = dict(case=case, slots=order[at // page] * page + at % page)
    for name, of_v in (("k_pool", False), ("v_pool", True)):
        x = torch.randn((num_pages * page, Hkv, D), generator=g, device="cuda")
        state[name] = _whole_pool(*_codes(x), num_pages, page, of_v)
    for name in ("k_out", "v_out"):
        state[name] = torch.empty((T, Hkv, D), dtype=_dtype(case), device="cuda")
    if own:
        from speculative_verify_paged_e4m3_gb300 import binding
        state["cache"] = binding.Mx4Cache(Hkv, D, page, num_pages)
    return state


def _prepare_attn(case, g):
    (Hq, Hkv), D, P = _heads(case), HEAD_DIM, case["page"]
    B, q_len, ctx = case["batch"], case["q_len"], max(case["context"], case["q_len"])
    lens = _ints(g, max(q_len, ctx // 3), ctx, B)
    lens[0] = ctx
    if case["empty"]:
        lens[B // 2] = 0  # a slot of the batch that holds no request
    max_pages = -(-ctx // P)
    num_pages = B * max_pages + 2
    order = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    state = dict(case=case, lens=lens, max_ctx=ctx,
                 table=order[:B * max_pages].view(B, max_pages).contiguous())
    channel = torch.exp(0.4 * torch.randn((Hkv, D), generator=g, device="cuda"))
    for name, of_v in (("k_pool", False), ("v_pool", True)):
        x = torch.randn((num_pages * P, Hkv, D), generator=g, device="cuda")
        if not of_v:  # keys have strong channels; of peaked ones some draw most of the attention
            x *= channel
            if case["peaked"]:
                u = torch.rand((num_pages * P, 1, 1), generator=g, device="cuda")
                x = torch.where(u < 0.05, 4.0 * x, x)
        state[name] = _whole_pool(*_codes(x), num_pages, P, of_v)
    state.update(q=torch.randn((B, q_len, Hq, D), generator=g, device="cuda").to(torch.float16),
                 out=torch.empty((B, q_len, Hq, D), dtype=torch.float16, device="cuda"),
                 lse=torch.empty((B, q_len, Hq), dtype=torch.float32, device="cuda"))
    if own:
        from speculative_verify_paged_e4m3_gb300 import binding
        state["att"] = binding.Mx4Attention(B, q_len, Hq, Hkv, D, P, max_pages, num_pages, ctx)
    return state


# ------------------------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return dict(norm=_own_norm, write=_own_write, read=_own_read, attn=_own_attn)[op](state)
    return dict(norm=_plain_norm, write=_plain_write, read=_plain_read,
                attn=_plain_attn)[op](state)


def _own_norm(s):
    s["rotary"].apply(s["q"], s["k"], s["pos"], q_out=s["q_out"], k_out=s["k_out"],
                      norm=s["norm"])
    return dict(q=s["q_out"], k=s["k_out"])


def _own_write(s):
    if s["case"]["cache"] == "e4m3":
        s["rotary"].kv_write(s["q"], s["k"], s["v"], s["pos"], s["slots"], s["k_scale"],
                             s["v_scale"], s["k_pool"], s["v_pool"], q_out=s["q_out"],
                             norm=s["norm"])
        return dict(q=s["q_out"], k_pool=s["k_pool"].view(torch.float8_e4m3fn),
                    v_pool=s["v_pool"].view(torch.float8_e4m3fn))
    s["rotary"].mx4_write(s["q"], s["k"], s["v"], s["pos"], s["slots"], s["k_pool"], s["v_pool"],
                          q_out=s["q_out"], norm=s["norm"])
    # what the cache holds now, as numbers (8 bits hold any of them)
    s["cache"].read(s["k_pool"], s["v_pool"], s["all_slots"], k_out=s["k_held"],
                    v_out=s["v_held"])
    return dict(q=s["q_out"], k_pool=s["k_held"], v_pool=s["v_held"])


def _own_read(s):
    s["cache"].read(s["k_pool"], s["v_pool"], s["slots"], k_out=s["k_out"], v_out=s["v_out"])
    return dict(k=s["k_out"], v=s["v_out"])


def _own_attn(s):
    s["att"](s["q"], s["k_pool"], s["v_pool"], s["table"], s["lens"], out=s["out"], lse=s["lse"])
    return dict(out=s["out"], lse=s["lse"])


def _turned(s, name, dtype):
    """Q or K of the state, each head normed and turned to its position, in this type."""
    c, x = s["case"], s[name].to(dtype)
    w = s[name + "_weight"].to(dtype) + c["offset"]
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    angle = s["pos"].double()[:, None, None] * s["theta"]  # angles of far positions need 64 bits
    cos, sin = torch.cos(angle).to(dtype), torch.sin(angle).to(dtype)
    d = c["rotary"]
    r, rest = x[..., :d], x[..., d:]
    if c["layout"] == "half":
        a, b = r[..., :d // 2], r[..., d // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([r, rest], -1)


def _plain_norm(s):
    s["q_out"].copy_(_turned(s, "q", torch.float32))
    s["k_out"].copy_(_turned(s, "k", torch.float32))
    return dict(q=s["q_out"], k=s["k_out"])


def _put_8(s, name, x, scale):
    """Rows x at the state's slots of an 8-bit pool; padding goes to a row behind it."""
    pool = s[name].flatten(0, 1)
    code = (x / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    grown = torch.cat([pool, pool[:1]])
    grown[torch.where(s["slots"] >= 0, s["slots"], pool.shape[0])] = code
    pool.copy_(grown[:-1])
    return s[name].view(torch.float8_e4m3fn)


def _put_4(s, name, x, of_v):
    """Rows x [T, Hkv, 256] at the state's slots of a 4-bit pool; padding goes to a byte behind it.
    Returns the numbers that the pool holds."""
    pool, slots = s[name].flatten(), s["slots"]
    H = x.shape[1]
    head = torch.arange(H, device=x.device)[:, None]
    at = ((slots // CHUNK)[:, None, None] * H + head) * CHUNK_BYTES + _offsets(slots, of_v)[:, None]
    at = torch.where(slots[:, None, None] >= 0, at, pool.numel())
    grown = torch.cat([pool, pool[:1]])
    grown[at] = _packed(*_codes(x), of_v)
    pool.copy_(grown[:-1])
    x = _numbers(s[name].flatten(0, 1), of_v, torch.float32)  # [chunks, H, 16, 256]
    return x.transpose(1, 2).flatten(0, 1).to(torch.float8_e5m2)


def _plain_write(s):
    live = s["slots"] >= 0
    q = _turned(s, "q", torch.float32)
    s["q_out"].copy_(torch.where(live[:, None, None], q.to(s["q_out"].dtype), s["q_out"]))
    # next to the border of two codes 32 bits are not enough
    k, v = _turned(s, "k", torch.float64), s["v"].double()
    if s["case"]["cache"] == "e4m3":
        return dict(q=s["q_out"], k_pool=_put_8(s, "k_pool", k.float(), s["k_scale"]),
                    v_pool=_put_8(s, "v_pool", v.float(), s["v_scale"]))
    return dict(q=s["q_out"], k_pool=_put_4(s, "k_pool", k, False),
                v_pool=_put_4(s, "v_pool", v, True))


def _read(pool, slots, of_v, dtype):
    x = _numbers(pool.flatten(0, 1)[slots // CHUNK], of_v, dtype)  # [T, H, 16, 256]
    tok = (slots % CHUNK)[:, None, None, None].expand(-1, x.shape[1], 1, HEAD_DIM)
    return x.gather(2, tok).squeeze(2)


def _plain_read(s):
    s["k_out"].copy_(_read(s["k_pool"], s["slots"], False, torch.float32))
    s["v_out"].copy_(_read(s["v_pool"], s["slots"], True, torch.float32))
    return dict(k=s["k_out"], v=s["v_out"])


def _rows(pool, table, of_v, dtype):
    """The keys or values of each request's pages in order: [B, pages * P, Hkv, 256]."""
    x = _numbers(pool[table.long()], of_v, dtype)  # [B, pages, P / 16, Hkv, 16, 256]
    return x.transpose(3, 4).flatten(1, 3)


def _plain_attn(s):
    c, q = s["case"], s["q"]
    (Hq, Hkv), D = _heads(c), HEAD_DIM
    B, q_len = q.shape[:2]
    G = Hq // Hkv
    qf = q.float().view(B, q_len, Hkv, G, D) / math.sqrt(D)
    sc = torch.einsum("bihgd,bjhd->bihgj", qf, _rows(s["k_pool"], s["table"], False, torch.float32))
    j = torch.arange(sc.shape[-1], device=q.device)
    last = s["lens"][:, None] - q_len + torch.arange(q_len, device=q.device)  # last visible key
    sc = torch.where((j <= last[..., None])[:, :, None, None], sc, -math.inf)
    top = sc.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(sc - top)
    total = p.sum(-1)
    o = torch.einsum("bihgj,bjhd->bihgd", p, _rows(s["v_pool"], s["table"], True, torch.float32))
    o = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
    s["out"].copy_(o.view(B, q_len, Hq, D))
    s["lse"].copy_((top[..., 0] + torch.log(total)).view(B, q_len, Hq))
    return dict(out=s["out"], lse=s["lse"])


# ------------------------------------------------------------------------------------ its work

def work(case):
    op, D = case["op"], HEAD_DIM
    Hq, Hkv = _heads(case)
    if op == "read":
        T = case["tokens"]
        return dict(bytes=T * (8 + 2 * Hkv * (136 + 2 * D)), flops=2 * T * Hkv * D)
    if op in ("norm", "write"):
        T = case["tokens"]
        # a sum of squares, two products an element, and six operations a turned pair
        flops = T * (Hq + Hkv) * (4 * D + 3 * case["rotary"])
        if op == "norm":
            return dict(bytes=T * (4 + 4 * (Hq + Hkv) * D) + 4 * D, flops=flops)
        held = D if case["cache"] == "e4m3" else 136
        moved = T * (12 + 4 * Hq * D + 2 * Hkv * (2 * D + held)) + 4 * D
        if case["cache"] == "mx4":  # the pools' numbers go out too
            n = (-(-T // case["page"]) + 3) * case["page"]
            moved += n * 2 * Hkv * D + (n - T) * 2 * Hkv * held
        return dict(bytes=moved, flops=flops + 2 * T * Hkv * D)
    B, q_len = case["batch"], case["q_len"]
    ctx = max(case["context"], q_len)
    rows = q_len * Hq
    keys = ctx + (B - 1 - (1 if case["empty"] else 0)) * (ctx + max(q_len, ctx // 3)) / 2
    return dict(bytes=keys * Hkv * 2 * 136 + B * rows * (4 * D + 4) + 4 * keys / case["page"],
                flops=4 * D * rows * keys)


# --------------------------------------------------------------------- the definitions, 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return dict(norm=_exact_rows, write=_exact_rows, read=_exact_read,
                attn=_exact_attn)[case["op"]](s)


def _decoded(pool, of_v):
    """Every number of a pool, [slots, Hkv, 256], code by code."""
    chunks = pool.flatten(0, 1)
    C, H = chunks.shape[:2]
    res = torch.empty((C, CHUNK, H, HEAD_DIM), dtype=torch.float64, device=pool.device)
    for e in range(HEAD_DIM):
        if of_v:
            b = chunks[..., e % 128 * 16:e % 128 * 16 + 16] >> (4 * (e // 128))
        else:
            first = e // 32 * 256 + e % 32 // 2
            b = chunks[..., first:first + 256:16] >> (4 * (e % 2))
        m = (b & 7).double()
        # codes 0 and 1 are halves; from 2 on, 1.5 or 1 times a power of two
        size = torch.where(m < 2, m / 2, (1 + (m % 2) / 2) * 2.0 ** (torch.floor(m / 2) - 1))
        power = chunks[..., CODE_BYTES + e // 32::8].double() - 127
        res[..., e] = (torch.where((b & 8) > 0, -size, size) * 2.0 ** power).transpose(1, 2)
    return res.flatten(0, 1)


def _nearest(x):
    """x [..., 256] on the 4-bit grid of its blocks of 32."""
    b = x.unflatten(-1, (8, 32))
    top = b.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top.clamp(min=1e-60) / 7))
    e = torch.where(top > 7 * 2.0 ** e, e + 1, torch.where(top <= 3.5 * 2.0 ** e, e - 1, e))
    y = b / 2.0 ** e.clamp(min=-127)
    step = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0))
    y = (torch.round(y / step) * step).clamp(-6, 6)  # (torch rounds halves to even)
    return (y * 2.0 ** e.clamp(min=-127)).flatten(-2)


def _exact_rows(s):
    """Pair (x, y) as the complex number x + iy, turned by e^(i pos theta)."""
    c = s["case"]
    half = c["rotary"] // 2
    angle = torch.outer(s["pos"].double(), s["theta"])
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    first = torch.arange(half, device="cuda") * (1 if c["layout"] == "half" else 2)
    second = first + (half if c["layout"] == "half" else 1)
    res = {}
    for name in ("q", "k"):
        x = s[name].double()
        y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / HEAD_DIM + EPS)
        y = y * (s[name + "_weight"].double() + c["offset"])
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        res[name] = y
    if c["op"] == "norm":
        return res
    live = s["slots"] >= 0
    out = dict(q=s["q_out"].double())
    out["q"][live] = res["q"][live]
    for name, x, of_v in (("k", res["k"], False), ("v", s["v"].double(), True)):
        if c["cache"] == "mx4" and not of_v:
            # the code of a key next to a border goes by the last bits of its norm and its angle
            out["k_pool"] = None
            continue
        if c["cache"] == "e4m3":
            held = s[name + "_pool"].view(torch.float8_e4m3fn).double()
            new = (x / s[name + "_scale"].double()).clamp(-E4M3_MAX, E4M3_MAX)
            held.flatten(0, 1)[s["slots"][live]] = new[live]
        else:
            held = _decoded(s[name + "_pool"], of_v)
            held[s["slots"][live]] = _nearest(x)[live]
        out[name + "_pool"] = held
    return out


def _exact_read(s):
    return dict(k=_decoded(s["k_pool"], False)[s["slots"]],
                v=_decoded(s["v_pool"], True)[s["slots"]])


def _exact_attn(s):
    """Request by request over its row of pages, a KV head at a time."""
    c, D, P = s["case"], HEAD_DIM, s["case"]["page"]
    Hq, Hkv = _heads(c)
    B, q_len = s["q"].shape[:2]
    G = Hq // Hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        pages = s["table"][b, :-(-n // P)].long()
        k, v = (_decoded(s[x][pages], of_v)[:n] for x, of_v in (("k_pool", False),
                                                                ("v_pool", True)))
        last = n - q_len + torch.arange(q_len, device="cuda").repeat_interleave(G)
        hidden = torch.arange(n, device="cuda") > last[:, None]
        for h in range(Hkv):
            q = s["q"][b, :, h * G:(h + 1) * G].double().reshape(-1, D)
            x = (q @ k[:, h].T / 16.0).masked_fill_(hidden, -math.inf)
            z = torch.logsumexp(x, -1)
            out[b, :, h * G:(h + 1) * G] = (torch.exp(x - z[:, None]) @ v[:, h]).view(q_len, G, D)
            lse[b, :, h * G:(h + 1) * G] = z.view(q_len, G)
    return dict(out=out, lse=lse)
