"""Cases and plain forms of the operators of a batch that shares prompts: samples of one prompt, chats under one
system prompt, questions about one document, image or video.

Four operators that act on one paged cache:
  decode_shared       one query per sequence; the prefix that a group of sequences has in common is read once for all
  compact_tokens      a sequence's kept tokens move together in its cache (rejected drafts and evicted tokens leave)
  copy_blocks         whole blocks of an 8-bit cache copied, as a fork's partial block is before it is written to
  rotary_append_axes  rotary positions of several axes (time, height, width), k and v written to slots of their own
With `own` false, `run` computes them with elementary torch operations in 32 bits (angles in 64); with `own` true it
makes the package's calls.
"""
import math
import random

import torch

own = False

PAGE = 4224  # bytes of an fp8 page: 16 tokens of one KV head, K and V codes and their scales
BLOCK = 16


# ------------------------------------------------------------------ cases

def listed():
    return [
        # four samples of one short prompt with a small model (12 heads of 64): latency
        dict(name="shared_small", op="shared", dtype="bf16", hq=12, hkv=12, d=64, batch=4, groups=1, shared=512,
             ragged=False, tail=64, lens=1),
        # 64 chats under one system prompt
        dict(name="shared_chats", op="shared", dtype="bf16", hq=32, hkv=8, d=128, batch=64, groups=1, shared=2048,
             ragged=False, tail=512, lens=2),
        # 32 questions about one long document
        dict(name="shared_document", op="shared", dtype="bf16", hq=32, hkv=8, d=128, batch=32, groups=1, shared=65536,
             ragged=False, tail=256, lens=3),
        # a serving batch: twelve prompts of many lengths with few to many samples each, long answers
        dict(name="shared_groups", op="shared", dtype="bf16", hq=32, hkv=8, d=128, batch=192, groups=12, shared=8191,
             ragged=True, tail=1024, lens=4),
        # groups of 8 query heads over the 8-bit cache
        dict(name="shared_fp8", op="shared", dtype="fp8", hq=64, hkv=8, d=128, batch=64, groups=1, shared=16384,
             ragged=False, tail=1024, lens=5),
        # after the check of 24 drafted tokens of each of 64 sequences: the accepted ones move up, in all layers
        dict(name="compact_drafts", op="compact", dtype="bf16", hq=12, hkv=12, d=64, layers=12, batch=64, most=1024,
             drafts=24, share=0.2, lens=6),
        # half of the tokens of 16 long sequences evicted
        dict(name="compact_evict", op="compact", dtype="bf16", hq=32, hkv=8, d=128, layers=1, batch=16, most=32768,
             drafts=0, share=0.5, lens=7),
        # a quarter of the tokens evicted from the 8-bit cache
        dict(name="compact_fp8", op="compact", dtype="fp8", hq=32, hkv=8, d=128, layers=1, batch=32, most=8192,
             drafts=0, share=0.75, lens=8),
        # the partial block of each of 64 new samples: latency
        dict(name="copy_fork", op="copy", dtype="fp8", hq=32, hkv=8, d=128, blocks=64, lens=9),
        # long sequences copied whole
        dict(name="copy_many", op="copy", dtype="fp8", hq=32, hkv=8, d=128, blocks=8192, lens=10),
        # a decode step of 64 sequences after images: the slot is not the position
        dict(name="axes_decode", op="axes", dtype="bf16", hq=32, hkv=8, d=128, layout="half", rot=128, order="sections",
             axes=3, prompts=0, images=0, side=0, words=0, single=64, lens=11),
        # prompts of text around images (a grid of side x side tokens each), axes taking turns over the pairs
        dict(name="axes_images", op="axes", dtype="bf16", hq=32, hkv=8, d=128, layout="half", rot=128, order="cyclic",
             axes=3, prompts=8, images=2, side=20, words=200, single=128, lens=12),
    ]


HEADS = [(12, 12), (16, 8), (32, 8), (8, 1), (32, 32), (64, 8)]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.5)))))))


def draw(rng):
    cost = {c["name"]: work(c) for c in listed()}
    most = {"shared": max(cost["shared_groups"]["bytes"], cost["shared_document"]["bytes"]),
            "compact": cost["compact_evict"]["bytes"], "copy": cost["copy_many"]["bytes"],
            "axes": cost["axes_images"]["bytes"]}
    flops = max(cost["shared_document"]["flops"], cost["shared_fp8"]["flops"])
    while True:
        op = rng.choice(["shared", "shared", "compact", "copy", "axes"])
        hq, hkv = rng.choice(HEADS)
        case = dict(op=op, hq=hq, hkv=hkv, d=rng.choice([64, 128]), lens=rng.randrange(1 << 30))
        if op == "shared":
            batch = _log(rng, 2, 256)
            case |= dict(dtype=rng.choice(["bf16", "bf16", "fp8"]), batch=batch,
                         groups=min(batch, rng.choice([1, 1, _log(rng, 1, 24)])), shared=_log(rng, 48, 65536),
                         ragged=rng.random() < 0.5, tail=_log(rng, 1, 2048))
            # (the plain form holds every group's scores at the longest prefix)
            if case["groups"] * case["shared"] > 131072 or batch * case["groups"] * case["shared"] * hq > 1 << 28:
                continue
        elif op == "compact":
            case |= dict(dtype=rng.choice(["bf16", "bf16", "f32", "fp8"]), batch=_log(rng, 1, 128),
                         layers=rng.choice([1, 1, 4]), most=_log(rng, 64, 32768),
                         drafts=rng.choice([0, 0, _log(rng, 2, 64)]), share=rng.choice([0.1, 0.5, 0.75, 0.9]))
        elif op == "copy":
            case |= dict(dtype="fp8", blocks=_log(rng, 1, 8192))
        else:
            case |= dict(dtype=rng.choice(["bf16", "bf16", "f32"]), layout=rng.choice(["half", "adjacent"]),
                         rot=rng.choice([r for r in (32, 64, 96, 128) if r <= case["d"]]),
                         order=rng.choice(["sections", "cyclic"]), axes=rng.choice([1, 2, 3, 4]),
                         prompts=_log(rng, 1, 8), images=rng.choice([0, 1, 2]), side=_log(rng, 2, 20),
                         words=_log(rng, 1, 400), single=_log(rng, 1, 256))
        if case["dtype"] == "fp8":
            case |= dict(d=128)
            if op == "compact":
                case |= dict(layers=1)
            if op == "shared" and hq // hkv not in (4, 8):
                continue  # the 8-bit cache is read in groups of 4 or 8 query heads
        if op == "compact" and (case["batch"] * case["most"] * case["layers"] * 2 * hkv * case["d"] * _element(case) > 3e9
                                or case["batch"] * case["most"] > 1 << 20):
            continue
        w = work(case)
        if 0 < w["bytes"] <= most[op] and w["flops"] <= flops:
            return case


def _groups(case):
    """(sequences, shared tokens) of every group, and the cached tokens of every sequence (0: a place of the batch
    that no sequence has; one in sixteen)."""
    r = random.Random(case["lens"])
    cuts = sorted(r.sample(range(1, case["batch"]), case["groups"] - 1)) + [case["batch"]]
    groups, lengths, at = [], [], 0
    for cut in cuts:
        shared = r.randint(case["shared"] // 16, case["shared"]) if case["ragged"] else case["shared"]
        groups.append((cut - at, shared))
        for _ in range(cut - at):
            lengths.append(0 if case["ragged"] and r.randrange(16) == 0 else shared + r.randint(1, case["tail"]))
        at = cut
    return groups, lengths


def _kept(case):
    """(cached tokens, first place, kept positions from there on) of every sequence of a compaction."""
    r = random.Random(case["lens"])
    out = []
    for _ in range(case["batch"]):
        n = r.randint(max(1, case["most"] // 4), case["most"])
        start = n if case["drafts"] else r.randint(0, 4)
        stop = n + case["drafts"]
        keep = [p for p in range(min(start, stop), stop) if r.random() < case["share"]]
        out.append((stop, min(start, stop), keep))
    return out


def _tokens(case):
    """(sequence, slot, positions on the axes) of every new token: prompts (words, then images of side x side tokens
    with words after each: text counts on all axes alike, an image's rows and columns on their own and its time stands
    still), then single tokens of sequences further on."""
    r = random.Random(case["lens"])
    out = []
    for s in range(case["prompts"]):
        slot = at = 0
        for part in range(case["images"] + 1):
            for _ in range(r.randint((case["words"] + 1) // 2, case["words"])):
                out.append((s, slot, [at] * 4))
                slot += 1
                at += 1
            if part < case["images"]:
                for y in range(case["side"]):
                    for x in range(case["side"]):
                        out.append((s, slot, [at, at + y, at + x, at + x + y]))
                        slot += 1
                at += case["side"]
    for s in range(case["single"]):
        at = r.randint(0, 8192)
        out.append((case["prompts"] + s, at + r.randint(0, 4096), [at] * 4))
    return out


def _sections(case):
    """Pairs of each axis: of three, a quarter for the first and the rest shared by the others."""
    n, a = case["rot"] // 2, case["axes"]
    if a == 1:
        return [n]
    if case["order"] == "cyclic":
        rest = [n // a - (1 if n // a > 4 else 0)] * (a - 1)
    else:
        rest = [(n - n // 4) // (a - 1)] * (a - 1)
    return [n - sum(rest)] + rest


def _element(case):
    return {"f32": 4.0, "bf16": 2.0, "fp8": 1.0 + 4.0 / case["d"]}[case["dtype"]]


def work(case):
    hq, hkv, d, e = case["hq"], case["hkv"], case["d"], _element(case)
    if case["op"] == "shared":
        groups, lengths = _groups(case)
        keys, at = 0, 0
        for n, shared in groups:
            used = [x for x in lengths[at:at + n] if x]
            keys += (shared if used else 0) + sum(x - shared for x in used)
            at += n
        return {"bytes": keys * 2 * hkv * d * e + case["batch"] * (2 * hq * d * 2 + 4), "flops": 4 * d * hq * sum(lengths)}
    if case["op"] == "compact":
        moved = sum(sum(p != start + j for j, p in enumerate(keep)) for _, start, keep in _kept(case))
        kept = sum(len(keep) for _, _, keep in _kept(case))
        return {"bytes": case["layers"] * moved * 2 * 2 * hkv * d * e + 4 * kept, "flops": 0}
    if case["op"] == "copy":
        return {"bytes": case["blocks"] * (2 * hkv * PAGE + 8), "flops": 0}
    t = len(_tokens(case))
    return {"bytes": t * (2 * (hq + 2 * hkv) * d * e + 4 * (case["axes"] + 2)), "flops": 3 * t * (hq + hkv) * case["rot"]}


# ------------------------------------------------------------------ inputs

BASE = 10000.0


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _swizzle():
    """[16, 8]: which 16-dim chunk of K is held in place j of token r's row of an fp8 page."""
    r = torch.arange(16)
    return (torch.arange(8)[None, :] ^ ((r & 1) | ((r >> 1) & 6))[:, None]).cuda()


def _fp8_pool(gen, blocks, hkv):
    """Pages of e4m3 codes with a scale for each (slot, head), as an append leaves them."""
    pages = blocks * hkv
    pool = torch.empty((pages, PAGE), dtype=torch.uint8, device="cuda")
    place = _swizzle()
    step = 1 << 14
    for a in range(0, pages, step):
        n = min(step, pages - a)
        x = _normal(gen, (2, n, 16, 128), torch.bfloat16).float()
        amax = x.abs().amax(-1, keepdim=True)
        code = (x * (448.0 / amax)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        k = torch.gather(code[0].view(n, 16, 8, 16), 2, place[None, :, :, None].expand(n, 16, 8, 16))
        pool[a:a + n, :2048] = k.reshape(n, 2048)
        pool[a:a + n, 2048:4096] = code[1].transpose(1, 2).reshape(n, 2048)
        scale = (amax / 448.0).reshape(2, n, 16).contiguous().view(torch.uint8)
        pool[a:a + n, 4096:4160], pool[a:a + n, 4160:] = scale[0], scale[1]
    return pool.view(blocks, hkv, 1, PAGE)


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _blocks_of(n):
    return -(-n // BLOCK)


def _inputs(case, seed):
    rng = random.Random("%d %d" % (seed, case["lens"]))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(rng.randrange(1 << 60))
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    dtype = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    st = dict(case=case)
    if case["op"] == "shared":
        groups, lengths = _groups(case)
        width = max(1, max(map(_blocks_of, lengths)))
        table, copies, cu, blocks = [], [], [0], 0
        for n, shared in groups:
            whole, first = shared // BLOCK, blocks
            blocks += whole
            for b in range(cu[-1], cu[-1] + n):
                row = list(range(first, first + whole))
                more = max(0, _blocks_of(lengths[b]) - whole)
                row += range(blocks, blocks + more)
                table.append(row + [-1] * (width - len(row)))
                blocks += more
                if shared % BLOCK and lengths[b]:  # a copy of the block that the prompt ends in
                    copies.append((cu[-1] + n, row[whole]))
            cu.append(cu[-1] + n)
        order = list(range(blocks + 3))
        rng.shuffle(order)
        st["table"] = _int([[order[i] if i >= 0 else -1 for i in row] for row in table])
        st["cu"], st["shared"] = _int(cu), _int([s for _, s in groups])
        st["most_shared"], st["max_len"] = max(s for _, s in groups), max(1, max(lengths))
        st["seq_lens"] = _int(lengths)
        st["q"] = _normal(gen, (case["batch"], hq, d), dtype)
        st["out"] = torch.empty_like(st["q"])
        blocks += 3
        st["same"] = [(order[b], order[next(x for g, x in copies if g == group)]) for group, b in copies]
        # where the padded plain form finds the sequences of a group
        st["most_in_group"] = max(n for n, _ in groups)
    elif case["op"] == "compact":
        kept = _kept(case)
        blocks = sum(_blocks_of(n) for n, _, _ in kept)
        order = list(range(blocks + 3))
        rng.shuffle(order)
        width, at, table, cu = max(_blocks_of(n) for n, _, _ in kept), 0, [], [0]
        for n, _, keep in kept:
            table.append(order[at:at + _blocks_of(n)] + [-1] * (width - _blocks_of(n)))
            at += _blocks_of(n)
            cu.append(cu[-1] + len(keep))
        st["table"], st["cu"] = _int(table), _int(cu)
        st["starts"] = _int([s for _, s, _ in kept])
        st["keep"] = _int([p for _, _, keep in kept for p in keep])
        blocks += 3
    elif case["op"] == "copy":
        blocks = 2 * case["blocks"] + 3
        order = list(range(blocks))
        rng.shuffle(order)
        st["src"], st["dst"] = _int(order[:case["blocks"]]), _int(order[case["blocks"]:2 * case["blocks"]])
    else:
        tokens = _tokens(case)
        rows = case["prompts"] + case["single"]
        last = [0] * rows
        for s, slot, _ in tokens:
            last[s] = max(last[s], slot)
        # (of the single tokens' sequences only the block that is written to is here)
        cells = [(s, c) for s in range(rows)
                 for c in (range(last[s] // BLOCK + 1) if s < case["prompts"] else [last[s] // BLOCK])]
        blocks = len(cells) + 3
        order = list(range(blocks))
        rng.shuffle(order)
        table = [[-1] * (max(last) // BLOCK + 1) for _ in range(rows)]
        for (s, c), i in zip(cells, order):
            table[s][c] = i
        st["table"] = _int(table)
        st["seq_ids"], st["slots"] = _int([t[0] for t in tokens]), _int([t[1] for t in tokens])
        st["positions"] = _int([[t[2][a] for t in tokens] for a in range(case["axes"])])
        st["qkv"] = _normal(gen, (len(tokens), (hq + 2 * hkv) * d), dtype)
        st["q_out"] = torch.empty((len(tokens), hq, d), dtype=dtype, device="cuda")
        n = case["rot"] // 2
        st["speeds"] = BASE ** (-2.0 * torch.arange(n, dtype=torch.float64, device="cuda") / case["rot"])
        st["axis"] = torch.tensor(_axis_of_pairs(case), device="cuda")
    if case["dtype"] == "fp8":
        st["pool"] = _fp8_pool(gen, blocks, hkv)
    elif case["op"] == "compact":
        st["pools"] = torch.empty((case["layers"], 2, blocks, hkv, BLOCK, d), dtype=dtype, device="cuda")
        for layer in st["pools"]:
            layer.copy_(_normal(gen, layer.shape, dtype))
    else:
        st["k_pool"] = _normal(gen, (blocks, hkv, BLOCK, d), dtype)
        st["v_pool"] = _normal(gen, (blocks, hkv, BLOCK, d), dtype)
    if case["op"] == "shared" and st["same"]:
        to, of = (torch.tensor(x, device="cuda") for x in zip(*st["same"]))
        for pool in ([st["pool"]] if case["dtype"] == "fp8" else [st["k_pool"], st["v_pool"]]):
            pool[to] = pool[of]  # (the tokens after the prompt's may be alike too)
    return st


def _axis_of_pairs(case):
    n, sections = case["rot"] // 2, _sections(case)
    if case["order"] == "sections":
        return [a for a, k in enumerate(sections) for _ in range(k)]
    return [i % len(sections) if i < len(sections) * sections[i % len(sections)] else 0 for i in range(n)]


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        import kv_cache_attention_rope_gb300 as kv

        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        st["kv"] = kv
        st["cfg"] = kv.make_config(hq, hkv, d, kv.F32 if case["dtype"] == "f32" else kv.BF16, rope_base=BASE)
        if case["dtype"] == "fp8":
            st["cache"] = kv.CacheFP8(st["pool"], BLOCK)
        elif case["op"] == "compact":
            st["cache"] = (kv.LayeredCache(st["cfg"], st["pools"]) if case["layers"] > 1
                           else kv.Cache(st["pools"][0, 0], st["pools"][0, 1]))
        else:
            st["cache"] = kv.Cache(st["k_pool"], st["v_pool"])
        if case["op"] == "shared":
            size = kv.decode_shared_workspace_size(st["cfg"], case["batch"], st["max_len"], case["groups"],
                                                   st["most_shared"])
            st["workspace"] = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
        elif case["op"] == "axes":
            st["rotary"] = kv.make_rotary(case["layout"], case["rot"])
            st["axes"] = kv.make_axes(_sections(case), case["order"])
            st["split"] = kv.split_qkv(st["qkv"], hq, hkv, d)
    return st


# ------------------------------------------------------------------ plain forms

def _read(st, ids, slot):
    """K and V [..., Hkv, D] in 32 bits of the slots [...] of the blocks ids [...]."""
    if st["case"]["dtype"] != "fp8":
        return st["k_pool"][ids, :, slot].float(), st["v_pool"][ids, :, slot].float()
    pool = st["pool"][:, :, 0]
    head = torch.arange(pool.shape[1], device="cuda")[:, None]
    ids, slot = ids[..., None, None], slot[..., None, None]
    # token r's K chunk c stands in place c ^ swizzle(r); dim d of its V at 2048 + 16 d + r
    lane = torch.arange(128, device="cuda")
    k = pool[ids, head, slot * 128 + ((lane // 16) ^ ((slot & 1) | ((slot >> 1) & 6))) * 16 + lane % 16]
    v = pool[ids, head, 2048 + 16 * lane + slot]
    scales = pool[..., 4096:].contiguous().view(torch.float32)
    return (k.view(torch.float8_e4m3fn).float() * scales[ids, head, slot],
            v.view(torch.float8_e4m3fn).float() * scales[ids, head, 16 + slot])


def _plain_shared(st):
    case = st["case"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    g, scale = hq // hkv, 1.0 / math.sqrt(d)
    cu, shared, table = st["cu"].long(), st["shared"].long(), st["table"].long()
    count = st["seq_lens"].long()
    batch, groups = case["batch"], case["groups"]
    group = torch.searchsorted(cu[1:].contiguous(), torch.arange(batch, device="cuda"), right=True)
    first = shared[group]
    # the prefixes, each read through a row of its group that has a sequence; groups padded to one size
    place = torch.arange(batch, device="cuda") - cu[group]
    leader = torch.zeros(groups, dtype=torch.long, device="cuda").scatter_reduce_(
        0, group, torch.where(count > 0, torch.arange(batch, device="cuda"), 0), "amax")
    tokens = torch.arange(st["most_shared"], device="cuda")
    k, v = _read(st, table[leader][:, (tokens // BLOCK).clamp(max=table.shape[1] - 1)].clamp(min=0),
                 (tokens % BLOCK).expand(groups, -1))
    n, q = st["most_in_group"], st["q"].float()
    padded = torch.zeros((groups, n, hq, d), device="cuda")
    padded[group, place] = q
    padded = padded.view(groups, n, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(groups, hkv, n * g, d)
    s = padded @ k.permute(0, 2, 3, 1) * scale
    s = s.masked_fill((tokens >= shared[:, None])[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = (s - top).exp()
    total, o = p.sum(-1, keepdim=True), p @ v.permute(0, 2, 1, 3)
    top, total, o = (x.view(groups, hkv, n, g, -1).permute(0, 2, 1, 3, 4)[group, place] for x in (top, total, o))
    # each sequence's own tokens
    tokens = first[:, None] + torch.arange(case["tail"], device="cuda")
    k, v = _read(st, table.gather(1, (tokens // BLOCK).clamp(max=table.shape[1] - 1)).clamp(min=0), tokens % BLOCK)
    s = q.view(batch, hkv, g, d) @ k.permute(0, 2, 3, 1) * scale
    s = s.masked_fill((tokens >= count[:, None])[:, None, None], -math.inf)
    both = torch.maximum(top, s.amax(-1, keepdim=True))
    p, old = (s - both).exp(), (top - both).exp()
    out = (o * old + p @ v.permute(0, 2, 1, 3)) / (total * old + p.sum(-1, keepdim=True))
    st["out"].copy_(out.reshape(batch, hq, d).masked_fill((count == 0)[:, None, None], 0.0))
    return st["out"]


def _plain_compact(st):
    case = st["case"]
    cu, keep, table = st["cu"].long(), st["keep"].long(), st["table"].long()
    at = torch.arange(keep.numel(), device="cuda")
    seq = torch.searchsorted(cu[1:].contiguous(), at, right=True)
    to = st["starts"].long()[seq] + at - cu[seq]
    src, dst = table[seq, keep // BLOCK], table[seq, to // BLOCK]
    r0, r1 = keep % BLOCK, to % BLOCK
    if case["dtype"] != "fp8":
        pools = st["pools"]
        pools[:, :, dst, :, r1] = pools[:, :, src, :, r0]
        return {"pools": pools}
    pool = st["pool"][:, :, 0]
    lane = torch.arange(128, device="cuda")
    four = torch.arange(4, device="cuda")

    def places(r):  # bytes of a token's K codes, V codes and scales in its page
        r = r[:, None]
        k = r * 128 + ((lane // 16) ^ ((r & 1) | ((r >> 1) & 6))) * 16 + lane % 16
        return torch.cat([k, 2048 + 16 * lane + r, 4096 + 4 * r + four, 4160 + 4 * r + four], 1)[:, None]

    head = torch.arange(pool.shape[1], device="cuda")[:, None]
    pool[dst[:, None, None], head, places(r1)] = pool[src[:, None, None], head, places(r0)]
    return _pages(st)


def _pages(st):
    """An 8-bit pool as the values that its bytes stand for: codes and scales."""
    return {"codes": st["pool"].view(torch.float8_e4m3fn)[..., :4096], "scales": st["pool"].view(torch.float32)[..., 1024:]}


def _plain_copy(st):
    st["pool"][st["dst"].long()] = st["pool"][st["src"].long()]
    return _pages(st)


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


def _plain_axes(st):
    case = st["case"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    t, dtype = st["qkv"].shape[0], st["qkv"].dtype
    x = st["qkv"].view(t, hq + 2 * hkv, d)
    angle = st["positions"].double()[st["axis"]].t() * st["speeds"]
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    turned = _rotate(x[:, :hq + hkv].float(), cos, sin, case).to(dtype)
    st["q_out"].copy_(turned[:, :hq])
    slots = st["slots"].long()
    ids = st["table"].long()[st["seq_ids"].long(), slots // BLOCK]
    st["k_pool"][ids, :, slots % BLOCK] = turned[:, hq:]
    st["v_pool"][ids, :, slots % BLOCK] = x[:, hq + hkv:]
    return {"q": st["q_out"], "k_pool": st["k_pool"], "v_pool": st["v_pool"]}


def run(st):
    case = st["case"]
    if not own:
        return {"shared": _plain_shared, "compact": _plain_compact, "copy": _plain_copy, "axes": _plain_axes}[case["op"]](st)
    kv, cfg, cache = st["kv"], st["cfg"], st["cache"]
    if case["op"] == "shared":
        call = kv.decode_shared_fp8 if case["dtype"] == "fp8" else kv.decode_shared
        return call(cfg, cache, st["q"], st["table"], st["seq_lens"], st["max_len"], st["cu"], st["shared"],
                    st["most_shared"], out=st["out"], workspace=st["workspace"])
    if case["op"] == "compact":
        kv.compact_tokens(cfg, cache, st["table"], st["starts"], st["cu"], st["keep"])
        return _pages(st) if case["dtype"] == "fp8" else {"pools": st["pools"]}
    if case["op"] == "copy":
        kv.copy_blocks(cfg, cache, st["src"], st["dst"])
        return _pages(st)
    q, k, v = st["split"]
    kv.rotary_append_axes(cfg, st["rotary"], st["axes"], cache, q, k, v, st["positions"], st["slots"], st["seq_ids"],
                          st["table"], q_out=st["q_out"])
    return {"q": st["q_out"], "k_pool": st["k_pool"], "v_pool": st["v_pool"]}


# ------------------------------------------------------------------ 64 bits

def _exact_cache(case, st, row, tokens):
    """K and V [n, Hkv, D] in 64 bits of one sequence's tokens."""
    ids, slot = st["table"][row].long()[tokens // BLOCK], tokens % BLOCK
    if case["dtype"] != "fp8":
        return st["k_pool"][ids, :, slot].double(), st["v_pool"][ids, :, slot].double()
    page = st["pool"][ids, :, 0]  # [n, Hkv, PAGE]
    n, hkv = len(tokens), case["hkv"]
    pick = torch.arange(n, device="cuda")
    k = page[..., :2048].reshape(n, hkv, 16, 8, 16)[pick, :, slot]
    k = k.gather(2, _swizzle()[slot][:, None, :, None].expand(n, hkv, 8, 16)).reshape(n, hkv, 128)
    v = page[..., 2048:4096].reshape(n, hkv, 128, 16)[pick, :, :, slot]
    ks = page[..., 4096:4160].contiguous().view(torch.float32)[pick, :, slot]
    vs = page[..., 4160:].contiguous().view(torch.float32)[pick, :, slot]
    return (k.contiguous().view(torch.float8_e4m3fn).double() * ks.double()[..., None],
            v.contiguous().view(torch.float8_e4m3fn).double() * vs.double()[..., None])


def _exact_shared(case, st):
    """Every sequence by itself, through its own row of the table."""
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_groups(case)[1]):
        if n:
            k, v = _exact_cache(case, st, b, torch.arange(n, device="cuda"))
            q = st["q"][b].double().view(hkv, hq // hkv, d)
            weight = torch.softmax(torch.einsum("hgd,nhd->hgn", q, k) / math.sqrt(d), -1)
            out[b] = torch.einsum("hgn,nhd->hgd", weight, v).reshape(hq, d)
    return out


def _exact_compact(case, st):
    """Sequence by sequence: its tokens in order of their places, and those that stay, written over them."""
    kept, table = _kept(case), st["table"].long()
    if case["dtype"] != "fp8":
        pools = st["pools"].double()
        for s, (n, start, keep) in enumerate(kept):
            rows = table[s, :_blocks_of(n)]
            # [layers, 2, blocks, Hkv, 16, D] -> tokens in the third place
            line = pools[:, :, rows].permute(0, 1, 2, 4, 3, 5).flatten(2, 3).clone()
            line[:, :, start:start + len(keep)] = line[:, :, torch.tensor(keep, dtype=torch.long, device="cuda")]
            pools[:, :, rows] = line.unflatten(2, (-1, BLOCK)).permute(0, 1, 2, 4, 3, 5)
        return {"pools": pools}
    pool = st["pool"].clone()
    inverse = _swizzle()
    turn = inverse[:, :, None].expand(16, 8, 16)
    for s, (n, start, keep) in enumerate(kept):
        rows, keep = table[s, :_blocks_of(n)], torch.tensor(keep, dtype=torch.long, device="cuda")
        page = pool[rows, :, 0]  # [blocks, Hkv, PAGE]
        b, hkv = page.shape[:2]
        k = page[..., :2048].reshape(b, hkv, 16, 8, 16).gather(3, turn.expand(b, hkv, 16, 8, 16))
        v = page[..., 2048:4096].reshape(b, hkv, 128, 16).transpose(2, 3)
        scale = page[..., 4096:].reshape(b, hkv, 2, 16, 4).transpose(2, 3)
        line = torch.cat([k.reshape(b, hkv, 16, 128), v, scale.reshape(b, hkv, 16, 8)], -1)
        line = line.transpose(1, 2).reshape(b * 16, hkv, 264).clone()
        line[start:start + len(keep)] = line[keep]
        line = line.view(b, 16, hkv, 264).transpose(1, 2)
        k = line[..., :128].reshape(b, hkv, 16, 8, 16).gather(3, turn.expand(b, hkv, 16, 8, 16))
        scale = line[..., 256:].reshape(b, hkv, 16, 2, 4).transpose(2, 3)
        pool[rows, :, 0] = torch.cat([k.reshape(b, hkv, 2048), line[..., 128:256].transpose(2, 3).reshape(b, hkv, 2048),
                                      scale.reshape(b, hkv, 128)], -1)
    return {"codes": pool.view(torch.float8_e4m3fn)[..., :4096].double(), "scales": pool.view(torch.float32)[..., 1024:].double()}


def _exact_axes(case, st):
    """As complex numbers: pair i is a point, turned by e^(i m f) with m the position on its axis."""
    hq, hkv, d, r = case["hq"], case["hkv"], case["d"], case["rot"]
    sections, angle = _sections(case), []
    left, axis = list(sections), 0
    for i in range(r // 2):
        if case["order"] == "cyclic":
            a = i % len(sections)
            a = a if i // len(sections) < sections[a] else 0
        else:
            while left[axis] == 0:
                axis += 1
            left[axis] -= 1
            a = axis
        angle.append(st["positions"][a].double() * BASE ** (-2.0 * i / r))
    angle = torch.stack(angle, 1)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    x = st["qkv"].double().view(-1, hq + 2 * hkv, d)
    head, rest = x[:, :hq + hkv, :r], x[:, :hq + hkv, r:]
    half = case["layout"] == "half"
    pairs = head.unflatten(-1, (2, r // 2)).transpose(-1, -2) if half else head.unflatten(-1, (r // 2, 2))
    y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    y = torch.cat([(y.transpose(-1, -2) if half else y).flatten(-2), rest], -1)
    k_pool, v_pool = st["k_pool"].double(), st["v_pool"].double()
    for t, (s, slot, _) in enumerate(_tokens(case)):
        blk = int(st["cells"][s][slot // BLOCK])
        k_pool[blk, :, slot % BLOCK] = y[t, hq:]
        v_pool[blk, :, slot % BLOCK] = x[t, hq + hkv:]
    return {"q": y[:, :hq].contiguous(), "k_pool": k_pool, "v_pool": v_pool}


def exact(case, seed):
    st = _inputs(case, seed)
    if case["op"] == "shared":
        return _exact_shared(case, st)
    if case["op"] == "compact":
        return _exact_compact(case, st)
    if case["op"] == "copy":
        pool = st["pool"].clone()
        for src, dst in zip(st["src"].tolist(), st["dst"].tolist()):
            pool[dst] = st["pool"][src]
        return {"codes": pool.view(torch.float8_e4m3fn)[..., :4096].double(),
                "scales": pool.view(torch.float32)[..., 1024:].double()}
    st["cells"] = st["table"].tolist()
    return _exact_axes(case, st)
