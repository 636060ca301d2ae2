"""What the 8-bit cache operators are measured on: the cases, their inputs, the
operators in plain torch operations, and their definition in 64 bits.

The operators serve the softmax layers that stand between the lightning layers of
a hybrid stack.  Their keys and values are kept in pages of 8-bit floating point
codes (e4m3) with one power-of-two scale for each page (a block of tokens) and kv
head:

    scale = 2^e, the least e >= -126 with max |x| <= 448 * 2^e over the block
    code  = x / scale, rounded to e4m3;   the cache then holds code * scale

  write   stores new tokens; a page that already holds tokens keeps its scale, or
          grows it to fit the new ones and rounds the older codes to it
  read    gives tokens of the cache back as bf16, fp16 or fp32
  token   attention of one or a few new tokens over the cache
  prompt  attention of a prompt, or of a later piece of one, over the cache

Sequence b has kv_len[b] tokens in the pages table[b]; its q_len[b] queries are the
last of them, and each sees the tokens up to its own.
"""
import math

import torch

own = False

LOW = -126    # least exponent of a scale
TOP = 448.0   # largest e4m3 number
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# --------------------------------------------------------------------- cases
def listed():
    return [
        # the prompt of the GQA prefill workload, 32768 tokens of 32 kv heads, as it enters a cache
        dict(name="write prompt 32K", op="write", B=1, Hkv=32, N=32768, held=0, ragged=False, d=128,
             page=64, type="bf16"),
        # the decode workload's 256 sequences, each adding one token to a page that holds others
        dict(name="write token B256", op="write", B=256, Hkv=16, N=1, held=512, ragged=True, d=128,
             page=64, type="bf16"),
        # pieces of prompts of several users, of different lengths, starting inside a page
        dict(name="write ragged pieces", op="write", B=5, Hkv=3, N=777, held=901, ragged=True, d=64,
             page=16, type="fp16"),
        # a stored conversation brought back for a layer that wants whole numbers of its own type
        dict(name="read 128K", op="read", B=1, Hkv=8, N=131072, held=0, ragged=False, d=128,
             page=128, type="bf16"),
        # a look at parts of several short sequences in fp32
        dict(name="read ragged fp32", op="read", B=7, Hkv=2, N=1000, held=300, ragged=True, d=64,
             page=32, type="fp32"),
        # one user in a short conversation: the latency of a single token
        dict(name="token B1 short", op="token", B=1, Hq=16, Hkv=16, N=1, held=332, ragged=False, d=128,
             page=64, type="bf16", lse=False),
        # the decode workload's batch: 256 sequences of up to 2048 tokens, 64 query heads on 16
        dict(name="token B256", op="token", B=256, Hq=64, Hkv=16, N=1, held=2047, ragged=True, d=128,
             page=64, type="bf16", lse=False),
        # one sequence of a million tokens, 8 heads (the long workload), next token
        dict(name="token 1M", op="token", B=1, Hq=8, Hkv=8, N=1, held=1048575, ragged=False, d=128,
             page=128, type="bf16", lse=False),
        # four drafted tokens for each of 32 sequences, joined with other attention by the row's logarithm
        dict(name="tokens 4 x B32", op="token", B=32, Hq=64, Hkv=16, N=4, held=8188, ragged=True, d=128,
             page=16, type="fp16", lse=True),
        # whole prompts without a past: the MHA prefill workload
        dict(name="prompt B4 8K", op="prompt", B=4, Hq=16, Hkv=16, N=8192, held=0, ragged=False, d=128,
             page=64, type="bf16", lse=False),
        # the last piece of a 32K prompt, 128 query heads on 32
        dict(name="prompt piece at 32K", op="prompt", B=1, Hq=128, Hkv=32, N=1024, held=31744,
             ragged=False, d=128, page=64, type="bf16", lse=False),
        # prompts of several users padded to one length, groups of three heads
        dict(name="prompt ragged", op="prompt", B=6, Hq=12, Hkv=4, N=777, held=600, ragged=True, d=64,
             page=32, type="fp16", lse=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "token", "token", "prompt", "prompt"])
    case = dict(op=op, d=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]),
                ragged=rng.random() < 0.6)
    if op in ("write", "read"):
        Hkv, B = rng.choice([1, 2, 3, 4, 8, 16, 32]), _log(rng, 1, 256)
        most = 2 ** 20 // (B * Hkv)               # tokens of one sequence: a GQA 32K prompt in all
        N = 1 if op == "write" and rng.random() < 0.3 else _log(rng, 1, max(2, most * 3 // 4))
        case |= dict(B=B, Hkv=Hkv, N=N, held=rng.randint(0, max(1, most - N)),
                     type=rng.choice(["bf16", "fp16", "fp32"]))
    elif op == "token":
        Hkv, G, B = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 2, 3, 4, 6, 8, 16]), _log(rng, 1, 256)
        N = 1 if rng.random() < 0.6 else rng.randint(1, max(1, 32 // G))
        case |= dict(B=B, Hq=Hkv * G, Hkv=Hkv, N=N, held=_log(rng, 1, 4 * 2 ** 20 // (B * Hkv)) - 1,
                     type=rng.choice(["bf16", "fp16"]), lse=rng.random() < 0.3)
    else:
        Hkv, G, B = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 6, 8]), _log(rng, 1, 16)
        N = _log(rng, 9, 8192)
        pairs = 2 ** 31 // (B * Hkv * G)          # query-key pairs of one head, half the largest case's
        N = max(9, min(N, int(math.sqrt(pairs))))
        case |= dict(B=B, Hq=Hkv * G, Hkv=Hkv, N=N,
                     held=0 if rng.random() < 0.4 else _log(rng, 1, max(2, min(65536, pairs // N - N))),
                     type=rng.choice(["bf16", "fp16"]), lse=rng.random() < 0.3)
    return case


def _lengths(case):
    """For each sequence the tokens held before the call and the call's own; spread over the range, by the case alone."""
    B, held, N = case["B"], case["held"], case["N"]
    if not case["ragged"]:
        return [held] * B, [N] * B
    part = [0.125 + 0.875 * ((0.618033988749895 * b + 0.93) % 1.0) for b in range(B)]
    return [int(held * p) for p in part], [max(1, int(N * part[-1 - b])) for b in range(B)]


# -------------------------------------------------------------------- inputs
def _quantised(x):
    """Codes (as e4m3) and scales of blocks x [..., page, d]."""
    part, e = torch.frexp(x.abs().amax((-2, -1)).double() / TOP)
    e = torch.where(part > 0, torch.where(part > 0.5, e, e - 1).clamp(min=LOW), LOW)
    scale = torch.ldexp(torch.ones_like(part), e).float()
    return (x / scale[..., None, None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    B, Hkv, N, d, page, dtype = (case[k] for k in ("B", "Hkv", "N", "d", "page", "type"))
    dtype = TYPES[dtype]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    # channels of keys differ in size as they do after training; blocks of tokens differ too
    channel = torch.exp(0.5 * normal(Hkv, 1, d))
    held, count = _lengths(case)
    pages = [-(-(h + c) // page) for h, c in zip(held, count)]
    total = sum(pages)
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, max(pages) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    # one page more than the tables name: nobody's
    cache = {}
    for name, size in (("k", channel), ("v", 1.0)):
        codes = torch.empty(total + 1, Hkv, page, d, dtype=torch.float8_e4m3fn, device="cuda")
        scales = torch.empty(total + 1, Hkv, device="cuda")
        step = max(1, 2 ** 27 // (Hkv * page * d))
        for i in range(0, total + 1, step):
            n = min(step, total + 1 - i)
            x = normal(n, Hkv, page, d) * size * torch.exp(0.4 * normal(n, Hkv, 1, 1))
            codes[i:i + n], scales[i:i + n] = _quantised(x)
        cache[name], cache[name + "_scale"] = codes, scales
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    state = dict(case=dict(case), **cache, table=table, held=ints(held), count=ints(count),
                 kv_len=ints([h + c for h, c in zip(held, count)]),
                 longest=max(h + c for h, c in zip(held, count)))
    if case["op"] == "write":
        state["new_k"] = (normal(B, Hkv, N, d) * channel).to(dtype)
        state["new_v"] = (normal(B, Hkv, N, d) * torch.exp(0.4 * normal(B, Hkv, N, 1))).to(dtype)
    elif case["op"] == "read":
        state["to"] = [torch.zeros(B, Hkv, N, d, dtype=dtype, device="cuda") for _ in "kv"]
    else:
        state["q"] = normal(B, case["Hq"], N, d).to(dtype)
        state["o"] = torch.zeros_like(state["q"])
        state["lse"] = torch.zeros(B, case["Hq"], N, device="cuda") if case["lse"] else None
    return state


# ------------------------------------------------------------ the operators
def run(state):
    op = state["case"]["op"]
    if own:
        import linear_attention_11_b200 as la
        cache = la.la_cache(state["k"], state["v"], state["k_scale"], state["v_scale"])
        ragged = state["case"]["ragged"]
        if op == "write":
            la.la_cache_write(state["new_k"], state["new_v"], cache, state["table"], state["held"],
                              count=state["count"] if ragged else None)
            return list(cache)
        if op == "read":
            return la.la_cache_read(cache, state["table"], state["held"], *state["to"],
                                    count=state["count"] if ragged else None)
        o = la.la_cache_attend(state["q"], cache, state["table"], state["kv_len"],
                               q_len=state["count"] if ragged else None, o=state["o"], lse=state["lse"])
        return [o, state["lse"]]
    if op == "write":
        return _write(state)
    if op == "read":
        return [_read(state, "k"), _read(state, "v")]
    return _attend(state)


def _write_one(state, x, name):
    """The pages of the new tokens, with those, in place; nobody's page stands in for the ones a sequence does not touch."""
    codes, scales, table = state[name], state[name + "_scale"], state["table"]
    start, count = state["held"].long(), state["count"].long()
    B, Hkv, N, d = x.shape
    page, nobody = codes.shape[2], codes.shape[0] - 1
    span = torch.arange(-(-N // page) + 1, device=x.device)
    block = start[:, None] // page + span                                     # [B, S] pages of a sequence
    token = block[:, :, None] * page + torch.arange(page, device=x.device)    # [B, S, page]
    new = (token >= start[:, None, None]) & (token < (start + count)[:, None, None])
    older = token < start[:, None, None]
    touched = new.any(2)
    at = table.long().gather(1, block.clamp(max=table.shape[1] - 1))
    at = torch.where(touched, at, nobody)
    row = (token - start[:, None, None]).clamp(0, N - 1).reshape(B, 1, -1, 1).expand(B, Hkv, -1, d)
    x = x.gather(2, row).float().reshape(B, Hkv, -1, page, d).transpose(1, 2)  # [B, S, Hkv, page, d]
    new, older = new[:, :, None, :, None], older[:, :, None, :, None]
    before, old = codes.view(torch.uint8)[at].view(codes.dtype).float(), scales[at]
    part, e = torch.frexp(torch.where(new, x.abs(), 0).amax((3, 4)).double() / TOP)
    e = torch.where(part > 0, torch.where(part > 0.5, e, e - 1).clamp(min=LOW), LOW)
    scale = torch.ldexp(torch.ones_like(part), e).float()
    scale = torch.where(older.any(3).squeeze(3), torch.maximum(scale, old), scale)
    both = torch.where(new, x / scale[..., None, None], before * (old / scale)[..., None, None])
    both = torch.where(new | older, both, before)
    both = torch.where(touched[:, :, None, None, None], both, before).to(codes.dtype)
    codes.view(torch.uint8)[at] = both.view(torch.uint8)
    scales[at] = torch.where(touched[:, :, None], scale, old)


def _write(state):
    _write_one(state, state["new_k"], "k")
    _write_one(state, state["new_v"], "v")
    return [state["k"], state["v"], state["k_scale"], state["v_scale"]]


def _tokens(state, name, token):
    """Tokens token [B, L] of each sequence as fp32 [B, Hkv, L, d]."""
    codes, table = state[name], state["table"]
    page = codes.shape[2]
    at = table.long().gather(1, (token // page).clamp(max=table.shape[1] - 1)).clamp(min=0)
    x = codes.view(torch.uint8)[at, :, token % page].view(codes.dtype).float()
    return (x * state[name + "_scale"][at][..., None]).transpose(1, 2)


def _read(state, name):
    to = state["to"]["kv".index(name)]
    i = torch.arange(to.shape[2], device="cuda")
    x = _tokens(state, name, state["held"].long()[:, None] + i)
    return torch.where((i < state["count"][:, None])[:, None, :, None], x, 0).to(to.dtype)


def _attend(state):
    q, kv_len, count = state["q"], state["kv_len"].long(), state["count"].long()
    B, Hq, N, d = q.shape
    Hkv = state["k"].shape[1]
    token = torch.arange(state["longest"], device="cuda")
    inside = token < kv_len[:, None]
    every = token.expand(B, -1)
    s = torch.matmul(q.float().view(B, Hkv, -1, d), _tokens(state, "k", every).transpose(2, 3))
    s = s.view(B, Hq, N, -1).mul_(1 / math.sqrt(d))
    i = torch.arange(N, device="cuda")
    sees = (token <= ((kv_len - count)[:, None] + i)[:, :, None]) & inside[:, None]
    s.masked_fill_(~sees[:, None], -math.inf)
    top = s.amax(3, keepdim=True)
    s.sub_(torch.where(top > -math.inf, top, 0)).exp_()
    total = s.sum(3, keepdim=True)
    v = torch.where(inside[:, None, :, None], _tokens(state, "v", every), 0)
    o = torch.matmul(s.view(B, Hkv, -1, s.shape[3]), v).view(B, Hq, N, d) / torch.where(total > 0, total, 1)
    there = (i < count[:, None])[:, None]
    o = torch.where(there[..., None], o, 0).to(q.dtype)
    if state["lse"] is None:
        return [o, None]
    return [o, torch.where(there, (top + total.log()).squeeze(3), 0)]


# --------------------------------------------------------------------- work
def work(case):
    d, Hkv = case["d"], case["Hkv"]
    held, count = _lengths(case)
    size = {"bf16": 2, "fp16": 2, "fp32": 4}[case["type"]]
    if case["op"] in ("write", "read"):
        n, page = sum(count), case["page"]
        blocks = sum(-(-(h + c) // page) - h // page for h, c in zip(held, count))
        return {"bytes": 2 * Hkv * (n * d * (size + 1) + blocks * 4), "flops": 2 * Hkv * n * d}
    blocks = sum(-(-(h + c) // case["page"]) for h, c in zip(held, count))
    pairs = sum(c * h + c * (c + 1) // 2 for h, c in zip(held, count))
    out = sum(count) * case["Hq"]
    return {"bytes": 2 * Hkv * (sum(h + c for h, c in zip(held, count)) * d + blocks * 4)
            + out * (2 * d * size + (4 if case["lse"] else 0)),
            "flops": 4 * case["Hq"] * d * pairs}


# -------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    state = prepare(case, seed)
    held, count = _lengths(case)
    page, d, table = case["page"], case["d"], state["table"].tolist()

    def sequence(name, b, h, first, last):
        """Tokens first..last of kv head h of sequence b."""
        ids = table[b][first // page:-(-last // page)]
        ids = torch.tensor(ids, device="cuda")
        x = state[name][ids, h].double() * state[name + "_scale"][ids, h].double()[:, None, None]
        return x.reshape(-1, d)[first % page:first % page + last - first]

    if case["op"] == "write":
        out = []
        powers = torch.tensor([2.0 ** e for e in range(LOW, 128)], dtype=torch.float64, device="cuda")
        for name in ("k", "v"):
            codes, scales, new = state[name].double(), state[name + "_scale"].double(), state["new_" + name]
            for b, (h, c) in enumerate(zip(held, count)):
                for p in range(h // page, -(-(h + c) // page)):
                    lo, hi = max(h, p * page), min(h + c, (p + 1) * page)
                    x = new[b, :, lo - h:hi - h].double()
                    least = torch.searchsorted(TOP * powers, x.abs().amax((1, 2)))
                    scale, at = powers[least], table[b][p]
                    if lo > p * page:
                        old = scales[at].clone()
                        scale = torch.maximum(scale, old)
                        codes[at, :, :lo - p * page] *= (old / scale)[:, None, None]
                    codes[at, :, lo - p * page:hi - p * page] = x / scale[:, None, None]
                    scales[at] = scale
            out.append((codes, scales))
        return [out[0][0], out[1][0], out[0][1], out[1][1]]
    if case["op"] == "read":
        out = [torch.zeros(t.shape, dtype=torch.float64, device="cuda") for t in state["to"]]
        for name, to in zip("kv", out):
            for b, (first, c) in enumerate(zip(held, count)):
                for h in range(case["Hkv"]):
                    to[b, h, :c] = sequence(name, b, h, first, first + c)
        return out
    q = state["q"].double()
    o, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], dtype=torch.float64, device="cuda")
    G = case["Hq"] // case["Hkv"]
    for b, (past, c) in enumerate(zip(held, count)):
        for h in range(case["Hkv"]):
            k, v = (sequence(name, b, h, 0, past + c) for name in ("k", "v"))
            mine = slice(h * G, (h + 1) * G)
            s = (q[b, mine, :c] @ k.T) / math.sqrt(d)
            if c > 1:
                s += torch.full((c, past + c), -math.inf, dtype=s.dtype, device="cuda").triu_(past + 1)
            o[b, mine, :c] = torch.softmax(s, -1) @ v
            lse[b, mine, :c] = torch.logsumexp(s, -1)
    return [o, lse if case["lse"] else None]
