"""Cases and plain forms of the rotary-append and sliding-window attention operators.

Three operators of one layer of a windowed model:
  rotary_append   rotary positions (half or adjacent pairs, part of the head, scaled for long
                  contexts) of the new tokens' q and k, with k and v written to their cache slots
  decode_window   one query per sequence over the last `window` tokens and the first `sinks`
  prefill_window  chunks of causal queries, each row over its own window and the sinks
With `own` false, `run` computes them with elementary torch operations in 32 bits (angles in 64);
with `own` true it makes the package's calls.
"""
import math
import random

import torch

own = False

PAGE = 4224  # bytes of an fp8 page: 16 tokens of one KV head, K and V codes and their scales


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the one new token of a chat with a small fp32 model (12 heads of 64): latency
        dict(name="rotary_one", op="rotary", dtype="f32", hq=12, hkv=12, d=64, layout="half", rot=64, scaling="none",
             factor=1.0, chunks=0, chunk=0, single=1, far=1023, block=16, lens=1),
        # a decode step of 64 sequences far into a context extended by parts
        dict(name="rotary_decode", op="rotary", dtype="bf16", hq=32, hkv=8, d=128, layout="half", rot=128,
             scaling="parts", factor=8.0, chunks=0, chunk=0, single=64, far=131071, block=16, lens=2),
        # the mixed step of the benchmark: 16 chunks of 512 prompt tokens and 128 single tokens
        dict(name="rotary_mixed", op="rotary", dtype="bf16", hq=32, hkv=8, d=128, layout="half", rot=128,
             scaling="parts", factor=8.0, chunks=16, chunk=512, single=128, far=8192, block=16, lens=3),
        # ragged prompts of a multi-head model that rotates half of each head, adjacent pairs
        dict(name="rotary_partial", op="rotary", dtype="bf16", hq=32, hkv=32, d=128, layout="adjacent", rot=64,
             scaling="base", factor=4.0, chunks=5, chunk=1021, single=0, far=4096, block=16, lens=4),
        # one sequence, a short window: latency
        dict(name="decode_one", op="decode", dtype="bf16", hq=32, hkv=8, d=128, batch=1, least=2000, most=4096,
             window=128, sinks=4, block=16, lens=5),
        # 8 sequences of a small fp32 model in a contiguous cache, some shorter than the window
        dict(name="decode_contiguous", op="decode", dtype="f32", hq=12, hkv=12, d=64, batch=8, least=1, most=1025,
             window=256, sinks=1, block=0, lens=6),
        # a full serving batch of long sequences: the whole window is read, the rest was freed
        dict(name="decode_batch", op="decode", dtype="bf16", hq=32, hkv=8, d=128, batch=256, least=1024, most=131072,
             window=4096, sinks=16, block=16, lens=7),
        # groups of 8 query heads over the 8-bit cache
        dict(name="decode_fp8", op="decode", dtype="fp8", hq=64, hkv=8, d=128, batch=64, least=1, most=32768,
             window=1024, sinks=4, block=16, lens=8),
        # a short prompt of a small model: latency
        dict(name="prefill_small", op="prefill", dtype="bf16", hq=12, hkv=12, d=64, chunks=1, chunk=100, ragged=False,
             far=0, window=128, sinks=0, block=16, lens=9),
        # the benchmark's 16 chunks of 512 queries with a window of 1024
        dict(name="prefill_mixed", op="prefill", dtype="bf16", hq=32, hkv=8, d=128, chunks=16, chunk=512, ragged=False,
             far=8192, window=1024, sinks=4, block=16, lens=10),
        # long documents: ragged chunks far in, a window of 4096
        dict(name="prefill_long", op="prefill", dtype="bf16", hq=32, hkv=8, d=128, chunks=16, chunk=512, ragged=True,
             far=32768, window=4096, sinks=16, block=16, lens=11),
        # chunks over the 8-bit cache
        dict(name="prefill_fp8", op="prefill", dtype="fp8", hq=32, hkv=8, d=128, chunks=8, chunk=512, ragged=False,
             far=8192, window=1024, sinks=4, block=16, lens=12),
    ]


HEADS = [(12, 12), (16, 8), (32, 8), (8, 1), (32, 32), (64, 8)]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.5)))))))


def draw(rng):
    cost = {c["name"]: work(c) for c in listed()}
    most = {"rotary": cost["rotary_mixed"]["bytes"], "decode": cost["decode_batch"]["bytes"],
            "prefill": cost["prefill_long"]["flops"]}
    while True:
        op = rng.choice(["rotary", "decode", "prefill"])
        hq, hkv = rng.choice(HEADS)
        case = dict(op=op, hq=hq, hkv=hkv, d=rng.choice([64, 128]), block=rng.choice([16, 16, 32, 128]),
                    lens=rng.randrange(1 << 30))
        if op == "rotary":
            dtype = rng.choice(["bf16", "bf16", "f32"])
            case |= dict(dtype=dtype, layout=rng.choice(["half", "adjacent"]),
                         rot=rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= case["d"]]),
                         scaling=rng.choice(["none", "linear", "base", "parts"]), factor=rng.choice([2.0, 4.0, 8.0]),
                         chunks=rng.choice([0, 1, 4, 16]), chunk=_log(rng, 1, 1024), single=_log(rng, 1, 256),
                         far=_log(rng, 64, 131071))
            key = "bytes"
        elif op == "decode":
            dtype = rng.choice(["bf16", "bf16", "f32", "fp8"])
            case |= dict(dtype=dtype, batch=_log(rng, 1, 256), least=rng.choice([0, 1, 100]),
                         most=_log(rng, 128, 131072), window=_log(rng, 16, 8192), sinks=rng.choice([0, 1, 4, 16, 63]))
            if rng.random() < 0.2 and dtype != "fp8":  # a contiguous cache: one row per sequence
                case |= dict(block=0, most=min(case["most"], 4096))
            if dtype == "fp8":
                case |= dict(d=128)
            key = "bytes"
        else:
            dtype = rng.choice(["bf16", "bf16", "fp8"])
            case |= dict(dtype=dtype, chunks=_log(rng, 1, 16), chunk=_log(rng, 1, 512), ragged=rng.random() < 0.5,
                         far=_log(rng, 1, 32768), window=_log(rng, 16, 8192), sinks=rng.choice([0, 1, 4, 16, 63]))
            if dtype == "fp8":
                case |= dict(d=128)
            key = "flops"
        if case["dtype"] == "fp8" and hq // hkv not in (4, 8):
            continue  # the 8-bit cache is read in groups of 4 or 8 query heads
        if op != "prefill" or _prefill_scores(case) <= _prefill_scores(listed()[10]):
            if work(case)[key] <= most[op]:
                return case


def _prefill_scores(case):
    n = min(case["sinks"] + case["window"] - 1, case["far"]) + case["chunk"]
    return case["chunks"] * case["hq"] * case["chunk"] * n


def _tokens(case):
    """Start position and length of every run of new tokens of a rotary case: one run per sequence."""
    r = random.Random(case["lens"])
    runs = [(r.randint(0, case["far"]), case["chunk"] - (r.randint(0, case["chunk"] // 2) if case["lens"] % 2 == 0 else 0))
            for _ in range(case["chunks"])]
    return runs + [(r.randint(0, case["far"]), 1) for _ in range(case["single"])]


def _lengths(case):
    """Cached tokens of every sequence of a decode case, the new one among them."""
    r = random.Random(case["lens"])
    return [r.randint(case["least"], case["most"]) for _ in range(case["batch"])]


def _chunks(case):
    """(prefix, queries) of every chunk of a prefill case."""
    r = random.Random(case["lens"])
    return [(r.randint(0, case["far"]), r.randint(1, case["chunk"]) if case["ragged"] else case["chunk"])
            for _ in range(case["chunks"])]


def _seen(p, window, sinks):
    """Keys that the row at position p sees."""
    low = max(0, p - window + 1)
    return p + 1 - low + min(sinks, low)


def _element(case):
    return {"f32": 4.0, "bf16": 2.0, "fp8": 1.0 + 4.0 / case["d"]}[case["dtype"]]


def work(case):
    hq, hkv, d, e = case["hq"], case["hkv"], case["d"], _element(case)
    if case["op"] == "rotary":
        t = sum(n for _, n in _tokens(case))
        return {"bytes": t * (2 * (hq + 2 * hkv) * d * e + 12), "flops": 3 * t * (hq + hkv) * case["rot"]}
    io = 4.0 if case["dtype"] == "f32" else 2.0
    w, s = case["window"], case["sinks"]
    if case["op"] == "decode":
        keys = sum(_seen(n - 1, w, s) for n in _lengths(case) if n)
        return {"bytes": keys * 2 * hkv * d * e + case["batch"] * (2 * hq * d * io + 4), "flops": 4 * d * hq * keys}
    keys = pairs = rows = 0
    for p, n in _chunks(case):
        low = max(0, p - w + 1)
        keys += p + n - low + min(s, low)
        pairs += sum(_seen(p + i, w, s) for i in range(n))
        rows += n
    return {"bytes": keys * 2 * hkv * d * e + 2 * rows * hq * d * io, "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------ inputs

BASE = 10000.0
ORIGINAL, LOW, HIGH = 4096.0, 1.0, 32.0  # `parts`: the original context, and the turns over it between which the speeds pass over
AMPLITUDE = {"none": 1.0, "linear": 1.0, "base": 1.0, "parts": 1.1875}


def _table(case, spans, rng, keep):
    """A block table with a block for every (sequence, column) that keep(sequence, column) names, -1 elsewhere,
    and the number of blocks of the pool: those, in a random order, and a few that nobody owns."""
    if not case["block"]:
        ids = list(range(len(spans) + 1))
        rng.shuffle(ids)
        return [[i] for i in ids[:len(spans)]], len(ids)
    block = case["block"]
    width = max(1, max((n + block - 1) // block for n in spans))
    cells = [(r, c) for r, n in enumerate(spans) for c in keep(r, (n + block - 1) // block)]
    ids = list(range(len(cells) + 3))
    rng.shuffle(ids)
    table = [[-1] * width for _ in spans]
    for (r, c), i in zip(cells, ids):
        table[r][c] = i
    return table, len(ids)


def _seen_columns(case, spans, firsts):
    """Columns of each row that hold a key some query sees: firsts[r] is the position of its first query."""
    block, w, s = case["block"] or 1, case["window"], case["sinks"]

    def keep(r, n):
        lead = min(n, (s + block - 1) // block)
        return list(range(lead)) + list(range(max(lead, max(0, firsts[r] - w + 1) // block), n))
    return keep


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _swizzle():
    """[16, 8]: which 16-dim chunk of K is held in place j of token r's row of an fp8 page."""
    r = torch.arange(16)
    return (torch.arange(8)[None, :] ^ ((r & 1) | ((r >> 1) & 6))[:, None]).cuda()


def _fp8_pool(gen, blocks, hkv, block):
    """Pages of e4m3 codes with a scale for each (slot, head), as an append leaves them."""
    pages = blocks * hkv * (block // 16)
    pool = torch.empty((pages, PAGE), dtype=torch.uint8, device="cuda")
    place = _swizzle()
    step = 1 << 14
    for a in range(0, pages, step):
        n = min(step, pages - a)
        x = _normal(gen, (2, n, 16, 128), torch.bfloat16).float()
        amax = x.abs().amax(-1, keepdim=True)
        scale = amax / 448.0
        code = (x * (448.0 / amax)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        k = code[0].view(n, 16, 8, 16)
        k = torch.gather(k, 2, place[None, :, :, None].expand(n, 16, 8, 16))
        pool[a:a + n, :2048] = k.reshape(n, 2048)
        pool[a:a + n, 2048:4096] = code[1].transpose(1, 2).reshape(n, 2048)
        pool[a:a + n, 4096:4160] = scale[0].reshape(n, 16).contiguous().view(torch.uint8)
        pool[a:a + n, 4160:] = scale[1].reshape(n, 16).contiguous().view(torch.uint8)
    return pool.view(blocks, hkv, block // 16, PAGE)


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _inputs(case, seed):
    rng = random.Random("%d %d" % (seed, case["lens"]))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(rng.randrange(1 << 60))
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    dtype = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    st = dict(case=case)
    if case["op"] == "rotary":
        runs = _tokens(case)
        block = case["block"]
        table, blocks = _table(case, [p + n for p, n in runs], rng, lambda r, n: range(runs[r][0] // block, n))
        order = list(range(len(runs)))
        rng.shuffle(order)
        st["positions"] = _int([p + i for r in order for p, n in [runs[r]] for i in range(n)])
        st["seq_ids"] = _int([r for r in order for _ in range(runs[r][1])])
        t = st["positions"].numel()
        st["qkv"] = _normal(gen, (t, (hq + 2 * hkv) * d), dtype)
        st["q_out"] = torch.empty((t, hq, d), dtype=dtype, device="cuda")
        st["speeds"] = _speeds(case)
    elif case["op"] == "decode":
        spans = _lengths(case)
        table, blocks = _table(case, spans, rng, _seen_columns(case, spans, [n - 1 for n in spans]))
        st["seq_lens"] = _int(spans)
        st["max_len"] = max(spans)
        st["q"] = _normal(gen, (case["batch"], hq, d), dtype)
        st["out"] = torch.empty_like(st["q"])
    else:
        chunks = _chunks(case)
        spans = [p + n for p, n in chunks]
        table, blocks = _table(case, spans, rng, _seen_columns(case, spans, [p for p, _ in chunks]))
        cu = [0]
        for _, n in chunks:
            cu.append(cu[-1] + n)
        st["cu"], st["prefix"] = _int(cu), _int([p for p, _ in chunks])
        st["max_q"] = max(n for _, n in chunks)
        st["max_len"] = max(spans)
        st["q"] = _normal(gen, (cu[-1], hq, d), dtype)
        st["out"] = torch.empty_like(st["q"])
    st["table"] = _int(table)
    block = case["block"] or case["most"]
    if case["dtype"] == "fp8":
        st["pool"] = _fp8_pool(gen, blocks, hkv, block)
    else:
        st["k_pool"] = _normal(gen, (blocks, hkv, block, d), dtype)
        st["v_pool"] = _normal(gen, (blocks, hkv, block, d), dtype)
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        import kv_cache_attention_rope_gb300 as kv

        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        st["kv"] = kv
        st["cfg"] = kv.make_config(hq, hkv, d, kv.F32 if case["dtype"] == "f32" else kv.BF16, rope_base=BASE)
        if case["dtype"] == "fp8":
            st["cache"] = kv.CacheFP8(st["pool"], case["block"])
        else:
            st["cache"] = kv.Cache(st["k_pool"], st["v_pool"])
        size = 0
        if case["op"] == "rotary":
            st["rotary"] = kv.make_rotary(case["layout"], case["rot"], case["scaling"], factor=case["factor"],
                                          original_len=ORIGINAL, low=LOW, high=HIGH,
                                          amplitude=AMPLITUDE[case["scaling"]])
            st["split"] = kv.split_qkv(st["qkv"], hq, hkv, d)
        elif case["op"] == "decode":
            size = kv.decode_window_workspace_size(st["cfg"], case["batch"], st["max_len"], case["window"],
                                                   case["sinks"])
        elif case["dtype"] == "fp8":
            size = kv.prefill_window_fp8_workspace_size(st["cfg"], case["block"], st["table"].shape[1], case["chunks"],
                                                        st["max_q"], case["window"], case["sinks"])
        st["workspace"] = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------ plain forms

def _speeds(case):
    """Speed of every pair in radians per position, in 64 bits."""
    r, f = case["rot"], case["factor"]
    i = torch.arange(r // 2, dtype=torch.float64, device="cuda")
    if case["scaling"] == "base":
        return (BASE * f ** (r / (r - 2))) ** (-2.0 * i / r)
    speed = BASE ** (-2.0 * i / r)
    if case["scaling"] == "linear":
        return speed / f
    if case["scaling"] == "parts":
        turns = ORIGINAL * speed / (2 * math.pi)
        share = ((turns - LOW) / (HIGH - LOW)).clamp(0.0, 1.0)
        return speed * (share + (1 - share) / f)
    return speed


def _rotate(x, cos, sin, case):
    """x [T, H, D] in 32 bits, the first rot dims of each head turned."""
    n = case["rot"] // 2
    y = x.clone()
    if case["layout"] == "half":
        a, b = x[..., :n], x[..., n:2 * n]
        y[..., :n] = a * cos - b * sin
        y[..., n:2 * n] = a * sin + b * cos
    else:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y[..., 0:2 * n:2] = a * cos - b * sin
        y[..., 1:2 * n:2] = a * sin + b * cos
    return y


def _plain_rotary(st):
    case = st["case"]
    hq, hkv, d, block = case["hq"], case["hkv"], case["d"], case["block"]
    t = st["qkv"].shape[0]
    dtype = st["qkv"].dtype
    x = st["qkv"].view(t, hq + 2 * hkv, d)
    angle = st["positions"].double()[:, None] * st["speeds"]
    amplitude = AMPLITUDE[case["scaling"]]
    cos = (angle.cos() * amplitude).float()[:, None, :]
    sin = (angle.sin() * amplitude).float()[:, None, :]
    turned = _rotate(x[:, :hq + hkv].float(), cos, sin, case).to(dtype)
    st["q_out"].copy_(turned[:, :hq])
    column = (st["positions"] // block).long()
    slot = (st["positions"] % block).long()
    ids = st["table"].long()[st["seq_ids"].long(), column]
    st["k_pool"][ids, :, slot] = turned[:, hq:]
    st["v_pool"][ids, :, slot] = x[:, hq + hkv:]
    return {"q": st["q_out"], "k_pool": st["k_pool"], "v_pool": st["v_pool"]}


def _read(st, tokens):
    """K and V [rows, n, Hkv, D] in 32 bits of the tokens [rows, n] of the table's rows."""
    case = st["case"]
    block = case["block"] or case["most"]
    width = st["table"].shape[1]
    ids = st["table"].long().gather(1, (tokens // block).clamp(max=width - 1)).clamp(min=0)
    slot = tokens % block
    if case["dtype"] != "fp8":
        return st["k_pool"][ids, :, slot].float(), st["v_pool"][ids, :, slot].float()
    page, r = slot // 16, slot % 16
    pool = st["pool"]
    rows, n = tokens.shape
    hkv = pool.shape[1]
    head = torch.arange(hkv, device="cuda")
    where = (ids[:, :, None], head[None, None, :], page[:, :, None])
    # token r's K chunk c stands in place c ^ swizzle(r); dim d of its V at 2048 + 16 d + r
    lane = torch.arange(128, device="cuda")
    at = r[:, :, None] * 128 + ((lane // 16) ^ ((r & 1) | ((r >> 1) & 6))[:, :, None]) * 16 + lane % 16
    k = pool[where[0][..., None], where[1][..., None], where[2][..., None], at[:, :, None, :]]
    v = pool[where[0][..., None], where[1][..., None], where[2][..., None], (2048 + 16 * lane + r[:, :, None])[:, :, None, :]]
    scales = pool[..., 4096:].contiguous().view(torch.float32)
    ks = scales[where[0], where[1], where[2], r[:, :, None]]
    vs = scales[where[0], where[1], where[2], 16 + r[:, :, None]]
    return (k.view(torch.float8_e4m3fn).float() * ks[..., None], v.view(torch.float8_e4m3fn).float() * vs[..., None])


def _attend(q, k, v, seen):
    """q [b, rows, Hq, D], k and v [b, n, Hkv, D], seen [b, rows, n]; a row that sees nothing gives zeros."""
    b, rows, hq, d = q.shape
    n, hkv = k.shape[1], k.shape[2]
    g = hq // hkv
    q = q.view(b, rows, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * rows, d)
    s = q @ k.permute(0, 2, 3, 1) * (1.0 / math.sqrt(d))
    s = s.view(b, hkv, g, rows, n).masked_fill(~seen[:, None, None], -math.inf)
    p = (s - s.amax(-1, keepdim=True).clamp(min=-3e38)).exp()
    total = p.sum(-1, keepdim=True)
    o = (p.view(b, hkv, g * rows, n) @ v.permute(0, 2, 1, 3)).view(b, hkv, g, rows, d)
    o = o / total.clamp(min=1e-37)
    return o.permute(0, 3, 1, 2, 4).reshape(b, rows, hq, d)


def _plain_decode(st):
    case = st["case"]
    w, s = case["window"], case["sinks"]
    n = max(1, min(st["max_len"], s + w))
    count = st["seq_lens"].long()[:, None]
    v = torch.arange(n, device="cuda")[None]
    tokens = torch.where(v < s, v, v - s + (count - w).clamp(min=s))
    seen = tokens < count
    k, val = _read(st, tokens.clamp(max=max(0, st["max_len"] - 1)))
    out = _attend(st["q"].float()[:, None], k, val, seen[:, None])
    st["out"].copy_(out[:, 0])
    return st["out"]


def _plain_prefill(st):
    case = st["case"]
    w, s = case["window"], case["sinks"]
    n = min(st["max_len"], s + w - 1 + st["max_q"])
    first = st["prefix"].long()[:, None]
    cu = st["cu"].long()
    total = cu[1:, None] - cu[:-1, None] + first
    v = torch.arange(n, device="cuda")[None]
    tokens = torch.where(v < s, v, v - s + (first - w + 1).clamp(min=s))
    r = torch.arange(st["max_q"], device="cuda")[None]
    p = (first + r)[:, :, None]
    j = tokens[:, None, :]
    seen = (j <= p) & ((j < s) | (j > p - w)) & (j < total[:, :, None])
    rows = st["q"].shape[0]
    q = st["q"].float()[(cu[:-1, None] + r).clamp(max=rows - 1)]
    k, val = _read(st, tokens.clamp(max=st["max_len"] - 1))
    out = _attend(q, k, val, seen)
    row = torch.arange(rows, device="cuda")
    chunk = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    st["out"].copy_(out[chunk, row - cu[chunk]])
    return st["out"]


def run(st):
    case = st["case"]
    if not own:
        return {"rotary": _plain_rotary, "decode": _plain_decode, "prefill": _plain_prefill}[case["op"]](st)
    kv, cfg, cache = st["kv"], st["cfg"], st["cache"]
    if case["op"] == "rotary":
        q, k, v = st["split"]
        kv.rotary_append(cfg, st["rotary"], cache, q, k, v, st["positions"], st["seq_ids"], st["table"],
                         q_out=st["q_out"])
        return {"q": st["q_out"], "k_pool": st["k_pool"], "v_pool": st["v_pool"]}
    fp8 = case["dtype"] == "fp8"
    if case["op"] == "decode":
        call = kv.decode_window_fp8 if fp8 else kv.decode_window
        return call(cfg, cache, st["q"], st["table"], st["seq_lens"], st["max_len"], case["window"], case["sinks"],
                    out=st["out"], workspace=st["workspace"])
    if fp8:
        return kv.prefill_window_fp8(cfg, cache, st["q"], st["cu"], st["prefix"], st["table"], st["max_q"],
                                     case["window"], case["sinks"], out=st["out"], workspace=st["workspace"])
    return kv.prefill_window(cfg, cache, st["q"], st["cu"], st["prefix"], st["table"], st["max_q"], case["window"],
                             case["sinks"], out=st["out"])


# ------------------------------------------------------------------ 64 bits

def _exact_rotary(case, st):
    """As complex numbers: a pair is a point, turned by e^(i m f)."""
    hq, hkv, d, r = case["hq"], case["hkv"], case["d"], case["rot"]
    base, factor = BASE, case["factor"]
    if case["scaling"] == "base":
        base = base * factor ** (r / (r - 2))
    speeds = []
    for i in range(r // 2):
        f = base ** (-2.0 * i / r)
        if case["scaling"] == "linear":
            f = f / factor
        elif case["scaling"] == "parts":
            share = min(1.0, max(0.0, (ORIGINAL * f / (2 * math.pi) - LOW) / (HIGH - LOW)))
            f = share * f + (1 - share) * f / factor
        speeds.append(f)
    angle = torch.outer(st["positions"].double(), torch.tensor(speeds, dtype=torch.float64, device="cuda"))
    turn = torch.polar(torch.full_like(angle, AMPLITUDE[case["scaling"]]), angle)[:, None]
    x = st["qkv"].double().view(-1, hq + 2 * hkv, d)
    head, rest = x[:, :hq + hkv, :r], x[:, :hq + hkv, r:]
    pairs = head.unflatten(-1, (2, r // 2)).transpose(-1, -2) if case["layout"] == "half" else head.unflatten(-1, (r // 2, 2))
    y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    if case["layout"] == "half":
        y = y.transpose(-1, -2)
    y = torch.cat([y.flatten(-2), rest], -1)
    k_pool, v_pool = st["k_pool"].double(), st["v_pool"].double()
    column = (st["positions"] // case["block"]).long()
    slot = (st["positions"] % case["block"]).long()
    ids = st["table"][st["seq_ids"].long(), column].long()
    k_pool[ids, :, slot] = y[:, hq:]
    v_pool[ids, :, slot] = x[:, hq + hkv:]
    return {"q": y[:, :hq].contiguous(), "k_pool": k_pool, "v_pool": v_pool}


def _exact_cache(case, st, row, tokens):
    """K and V [n, Hkv, D] in 64 bits of one sequence's tokens."""
    block = case["block"] or case["most"]
    ids = st["table"][row].long()[tokens // block]
    slot = tokens % block
    if case["dtype"] != "fp8":
        return st["k_pool"][ids, :, slot].double(), st["v_pool"][ids, :, slot].double()
    page = st["pool"][ids, :, slot // 16]  # [n, Hkv, PAGE]
    n, hkv, r = len(tokens), case["hkv"], slot % 16
    pick = torch.arange(n, device="cuda")
    k = page[..., :2048].reshape(n, hkv, 16, 8, 16)[pick, :, r]
    k = k.gather(2, _swizzle()[r][:, None, :, None].expand(n, hkv, 8, 16)).reshape(n, hkv, 128)
    v = page[..., 2048:4096].reshape(n, hkv, 128, 16)[pick, :, :, r]
    ks = page[..., 4096:4160].contiguous().view(torch.float32)[pick, :, r]
    vs = page[..., 4160:].contiguous().view(torch.float32)[pick, :, r]
    return (k.contiguous().view(torch.float8_e4m3fn).double() * ks.double()[..., None],
            v.contiguous().view(torch.float8_e4m3fn).double() * vs.double()[..., None])


def exact(case, seed):
    st = _inputs(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(case, st)
    w, s, hq, hkv, d = case["window"], case["sinks"], case["hq"], case["hkv"], case["d"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    if case["op"] == "decode":
        queries = [(b, b, b + 1, n - 1) for b, n in enumerate(_lengths(case)) if n]
    else:
        starts = st["cu"].tolist()
        queries = [(c, starts[c], starts[c + 1], p) for c, (p, _) in enumerate(_chunks(case))]
    for row, a, b, p in queries:
        low = max(0, p - w + 1)
        keys = sorted(set(range(min(s, low))) | set(range(low, p + b - a)))
        tokens = torch.tensor(keys, device="cuda")
        k, v = _exact_cache(case, st, row, tokens)
        at = torch.arange(p, p + b - a, device="cuda")[:, None]
        hidden = (tokens > at) | ((tokens >= s) & (tokens <= at - w))
        q = st["q"][a:b].double().view(b - a, hkv, hq // hkv, d)
        score = torch.einsum("rhgd,nhd->hgrn", q, k) / math.sqrt(d)
        weight = torch.softmax(score.masked_fill(hidden, -math.inf), -1)
        out[a:b] = torch.einsum("hgrn,nhd->rhgd", weight, v).reshape(b - a, hq, d)
    return out
