"""What a step with drafted tokens needs around the model, with what it is measured on.

A narrow child of the nested weights drafts a few tokens for each sequence and a wider one
checks them all in one step.  Three operators, over the paged key-value cache:

  reserve  from the sequences' lengths: pages taken from a free list and given back to it, the
           table of pages brought up to date, and for each new token its position and slot
  shared   attention of each sequence's new tokens over its cached ones, where groups of
           sequences share a long prefix that is attended to once for all of them
  verify   which drafted tokens the target's probabilities accept, and the token after them,
           from given random numbers

``run`` computes them in elementary torch operations, or, with ``own`` set, by the
calls that a user of this package makes.  ``exact`` is the same mathematics in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

FP8_MAX = 448.0  # the largest finite value of the 8-bit type (4 exponent bits, 3 of mantissa)


# ---------------------------------------------------------------------------
# cases

def _reserve(name, rows, longest, new, page, heads=8, shared=False, short=False, first=False):
    return {"name": name, "op": "reserve", "rows": rows, "longest": longest, "new": new, "page": page, "kv": heads,
            "shared": shared, "short": short, "first": first}


def _shared(name, groups, rows, prefix, tail, new, heads, kv, dim=128, page=64, dtype="bf16", ragged=True):
    return {"name": name, "op": "shared", "groups": groups, "rows": rows, "prefix": prefix, "tail": tail, "new": new,
            "heads": heads, "kv": kv, "dim": dim, "page": page, "dtype": dtype, "ragged": ragged}


def _verify(name, rows, drafts, vocab, dtype="fp32", ragged=True, sampled=True):
    return {"name": name, "op": "verify", "rows": rows, "drafts": drafts, "vocab": vocab, "dtype": dtype, "ragged": ragged,
            "sampled": sampled}


def listed():
    return [
        # one conversation asks for the place of its next token: a call whose latency counts
        _reserve("reserve-one", 1, 333, 1, 16),
        # an ordinary serving step: a few drafted tokens each, some rows give pages back, some have ended
        _reserve("reserve-step", 256, 8192, 6, 64, shared=True),
        # prompts of many lengths arrive at once, more than the pool has pages for
        _reserve("reserve-prompts", 96, 0, 8192, 16, short=True, first=True),
        # a few answers to one short question, sampled side by side: latency
        _shared("shared-few", 1, 4, 500, 40, 1, 32, 8, page=16),
        # a serving batch behind one system prompt, the Llama-3.1-8B heads
        _shared("shared-64", 1, 64, 8192, 600, 1, 32, 8),
        # several system prompts, the 70B layer's heads over an 8-bit cache
        _shared("shared-groups-fp8", 6, 48, 4001, 900, 1, 64, 8, page=128, dtype="fp8"),
        # drafted tokens of unrelated conversations: nothing is shared but each one's own past
        _shared("shared-drafts", 16, 16, 0, 4096, 5, 32, 8),
        # a long document that many are asked about, with drafted tokens: the arithmetic counts
        _shared("shared-document", 1, 96, 32767, 500, 5, 32, 8),
        # short prompts that follow the same long instructions, narrow heads, small pages
        _shared("shared-prompts", 2, 8, 4096, 300, 300, 12, 12, dim=64, page=16),
        # one conversation with four drafted tokens
        _verify("verify-one", 1, 4, 32000, ragged=False),
        # an ordinary batch, a larger vocabulary
        _verify("verify-64", 64, 5, 128000),
        # a full batch, probabilities of 16 bits, drafts looked up in the text instead of sampled
        _verify("verify-256-lookup", 256, 7, 160001, dtype="bf16", sampled=False),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        b, f = most.get(c["op"], (0, 0))
        most[c["op"]] = max(b, w["bytes"]), max(f, w["flops"])
    while True:
        op = rng.choice(["reserve", "shared", "shared", "verify"])
        if op == "reserve":
            first = rng.random() < 0.4
            c = _reserve("", _log(rng, 1, 1024), 0 if first else _log(rng, 1, 16384), _log(rng, 1, 8192) if first else
                         rng.randint(1, 9), rng.choice([1, 8, 16, 32, 64, 128, 256]), 1, rng.random() < 0.3, rng.random() < 0.3,
                         first)
            # tables of a drawn case stay small beside the card too
            slots = c["rows"] * (c["longest"] + 2 * c["new"])
            fits = slots // c["page"] <= 1 << 21 and slots <= 1 << 24
        elif op == "shared":
            kv = rng.choice([1, 2, 4, 8, 8, 8, 10])
            rows = _log(rng, 1, 128)
            new = rng.choice([1, 1, rng.randint(2, 9), _log(rng, 10, 512)])
            c = _shared("", rng.choice([1, 1, min(rows, rng.randint(2, 12)), rows]), rows,
                        rng.choice([0, _log(rng, 1, 32768), _log(rng, 64, 32768)]), new + _log(rng, 1, 4096) - 1, new,
                        kv * rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16]), kv, rng.choice([64, 128, 128, 128, 256]),
                        rng.choice([8, 16, 32, 64, 128, 256]), rng.choice(["bf16", "bf16", "fp8"]), rng.random() < 0.75)
            # scores of the plain form stay small beside the card too
            lines = rows * new * c["heads"]
            fits = lines * (c["prefix"] + c["tail"]) <= 1 << 30 and rows * kv * c["dim"] * (c["prefix"] + c["tail"]) <= 1 << 31
        else:
            c = _verify("", _log(rng, 1, 256), rng.randint(0, 9), _log(rng, 500, 200000), rng.choice(["fp32", "fp32", "bf16"]),
                        rng.random() < 0.6, rng.random() < 0.6)
            fits = c["rows"] * (c["drafts"] + 1) * c["vocab"] <= 1 << 28
        del c["name"]
        w = work(c)
        if fits and w["bytes"] <= most[op][0] and w["flops"] <= most[op][1]:
            return c


def _spread(n, longest, ragged, salt, least=1):
    """n numbers: the longest one, the others spread below it."""
    if not ragged or n == 1 or longest <= least:
        return [longest] * n
    r = random.Random(n * 1000003 + longest * 101 + salt)
    return [longest] + [max(least, int(longest * r.uniform(0.1, 1.0))) for _ in range(n - 1)]


def _reserve_sizes(case):
    """For every row: slots in use, tokens asked for, pages held; pages that the rows share; free pages."""
    rows, page = case["rows"], case["page"]
    r = random.Random(rows * 1000003 + case["longest"] * 101 + case["new"])
    lens = [0] * rows if case["first"] else _spread(rows, case["longest"], True, 1)
    new = _spread(rows, case["new"], True, 2)
    # the last step's drafts, some of them taken back, are still covered by the pages held
    held = [0 if case["first"] else -(-(n + r.randint(0, case["new"])) // page) for n in lens]
    for i in range(3, rows, 8):
        lens[i] = new[i] = 0  # ended, or an idle place
    own = 0
    if case["shared"]:
        own = min(held) // 2
    wanted = sum(max(0, -(-(n + t) // page) - h) for n, t, h in zip(lens, new, held))
    back = sum(max(0, h - max(-(-(n + t) // page), own if i else 0)) for i, (n, t, h) in enumerate(zip(lens, new, held)))
    spare = max(0, int(wanted * 0.7) - back) if case["short"] else wanted + 64
    return lens, new, held, own, spare


def _shared_sizes(case):
    """(first row of every group and the end, prefix of every group, lengths, new tokens of every row)."""
    rows, groups = case["rows"], case["groups"]
    r = random.Random(rows * 1000003 + case["prefix"] * 101 + groups)
    cuts = sorted(r.sample(range(1, rows), groups - 1)) if groups < rows else list(range(1, rows))
    cuts = [0] + cuts + [rows]
    prefix = _spread(groups, case["prefix"], case["ragged"], 3, least=0)
    new = _spread(rows, case["new"], case["ragged"], 4)
    tail = [max(t, n) for t, n in zip(_spread(rows, case["tail"], case["ragged"], 5), new)]
    if case["ragged"] and rows >= 4:
        new[2] = 0  # waits for its turn
    lens = [prefix[g] + tail[i] for g in range(groups) for i in range(cuts[g], cuts[g + 1])]
    return cuts, prefix, lens, new


def _verify_counts(case):
    """Tokens of every row: the last one that is certain and the drafts behind it."""
    counts = [n + 1 for n in _spread(case["rows"], case["drafts"], case["ragged"], 6, least=0)]
    if case["ragged"] and case["rows"] >= 4:
        counts[2] = 1  # nothing drafted
    return counts


def work(case):
    if case["op"] == "reserve":
        lens, new, held, own, spare = _reserve_sizes(case)
        page, rows, tokens = case["page"], case["rows"], sum(new)
        moved = sum(abs(max(-(-(n + t) // page), own if i else 0) - h) for i, (n, t, h) in enumerate(zip(lens, new, held)))
        touched = sum(-(-(n + t) // page) - n // page for n, t in zip(lens, new))
        # lengths, counts, pages held in and out; pages taken and given back; positions and slots
        return {"bytes": rows * 4 * 7 + moved * 8 + touched * 4 + tokens * 12 + 8, "flops": rows * 8 + tokens * 4}
    if case["op"] == "shared":
        cuts, prefix, lens, new = _shared_sizes(case)
        kv, heads, dim = case["kv"], case["heads"], case["dim"]
        row = dim * (2 if case["dtype"] == "bf16" else 1)  # one head's key, or value, of one token
        slots = flops = 0
        for g, p in enumerate(prefix):
            mine = range(cuts[g], cuts[g + 1])
            if any(new[i] for i in mine):
                slots += p
            for i in mine:
                if new[i]:
                    slots += lens[i] - p
                    # token j of n sees all but the n - 1 - j slots after its own
                    flops += 4 * heads * dim * (new[i] * lens[i] - new[i] * (new[i] - 1) // 2)
        return {"bytes": slots * kv * 2 * row + slots // case["page"] * 4 + 2 * sum(new) * heads * dim * 2, "flops": flops}
    # Each row's next token needs one line of the vocabulary, and after a refused draft the
    # draft's line beside it if that was sampled; about three rows in four have one.
    each = case["vocab"] * (4 if case["dtype"] == "fp32" else 2)
    refused = 0.75 * sum(n > 1 for n in _verify_counts(case)) if case["sampled"] else 0
    tokens = sum(_verify_counts(case))
    return {"bytes": int((case["rows"] + refused) * each + tokens * 16), "flops": int(2 * (case["rows"] + refused) * case["vocab"])}


# ---------------------------------------------------------------------------
# inputs

def prepare(case, seed):
    return _PREPARE[case["op"]](case, torch.Generator(device="cuda").manual_seed(seed), torch.device("cuda"))


def _ints(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def _running(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def _prepare_reserve(c, g, dev):
    lens, new, held, share, spare = _reserve_sizes(c)
    rows, page, kv = c["rows"], c["page"], c["kv"]
    width = max([-(-(n + t) // page) for n, t in zip(lens, new)] + held + [1])
    mine = [h if i == 0 else h - min(h, share) for i, h in enumerate(held)]
    pages = sum(mine) + spare
    order = torch.randperm(max(pages, 1), generator=g, device=dev).to(torch.int32).cpu().numpy()
    table = np.full((rows, width), -1, dtype=np.int32)
    at = 0
    for i, h in enumerate(held):
        of = h - mine[i]
        table[i, :of] = table[0, :of]
        table[i, of:h] = order[at:at + mine[i]]
        at += mine[i]
    free = np.full(max(pages, 1), -1, dtype=np.int32)
    free[:spare] = order[at:at + spare]
    s = {"case": c, "page": page, "pages": max(pages, 1), "table": torch.from_numpy(table).to(dev), "lens": _ints(lens, dev),
         "new": _ints(new, dev), "held": _ints(held, dev), "free": torch.from_numpy(free).to(dev), "count": _ints([spare], dev),
         "kept": _ints([0 if i == 0 else min(h, share) for i, h in enumerate(held)], dev) if c["shared"] else None,
         "most": max(sum(new), 1)}
    # a sequence that has lost tokens to its budget has seen more than it holds
    s["seen"] = s["lens"] + torch.randint(0, 50, (rows,), generator=g, device=dev, dtype=torch.int32)
    for name, shape, dtype in (("cu", rows + 1, torch.int32), ("positions", s["most"], torch.int32), ("slots", s["most"], torch.int64),
                               ("granted", rows, torch.int32), ("held_out", rows, torch.int32), ("count_out", 1, torch.int32)):
        s[name] = torch.zeros(shape, dtype=dtype, device=dev)
    if own:
        import nested_bit_weight_amd as nbw
        # the table is what counts here: the layers' pools are beside it
        pool = torch.zeros(s["pages"], kv, page, 64, dtype=torch.bfloat16, device=dev)
        s["cache"] = nbw.KVCache(pool, pool, s["table"])
    return s


def _prepare_shared(c, g, dev):
    def normal(*shape, by=1.0, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).mul_(by).to(dtype)

    cuts, prefix, lens, new = _shared_sizes(c)
    rows, kv, dim, page = c["rows"], c["kv"], c["dim"], c["page"]
    whole = [p // page for p in prefix]  # pages that hold nothing but the prefix are shared
    need = [-(-n // page) for n in lens]
    group = [k for k in range(c["groups"]) for _ in range(cuts[k], cuts[k + 1])]
    pages = sum(whole) + sum(n - whole[k] for n, k in zip(need, group)) + 1  # the last page belongs to nobody
    order = torch.randperm(pages - 1, generator=g, device=dev).to(torch.int32).cpu().numpy()
    table = np.full((rows, max(need + [1])), -1, dtype=np.int32)
    at = 0
    for k, w in enumerate(whole):
        table[cuts[k]:cuts[k + 1], :w] = order[at:at + w]
        at += w
    for i, n in enumerate(need):
        w = whole[group[i]]
        table[i, w:n] = order[at:at + n - w]
        at += n - w
    s = {"case": c, "page": page, "table": torch.from_numpy(table).to(dev), "k_scale": None, "v_scale": None}
    if c["dtype"] == "fp8":
        # one factor a head, as calibration leaves them: 8-bit value times factor is the key (the value)
        s["k_scale"] = torch.rand(kv, generator=g, device=dev) * 0.01 + 0.01
        s["v_scale"] = torch.rand(kv, generator=g, device=dev) * 0.01 + 0.01
    kind = torch.float8_e4m3fn if c["dtype"] == "fp8" else torch.bfloat16
    for name in ("k", "v"):
        pool = normal(pages, kv, page, dim, dtype=torch.float32)
        if c["dtype"] == "fp8":
            pool = (pool / s[name + "_scale"][None, :, None, None]).clamp_(-FP8_MAX, FP8_MAX)
        s[name] = pool.to(kind)
    # where a page holds the prefix's last slots and each row's first ones, all rows have the prefix's
    for k, p in enumerate(prefix):
        if p % page:
            mine = torch.from_numpy(table[cuts[k]:cuts[k + 1], whole[k]]).long().to(dev)
            for name in ("k", "v"):
                raw = s[name].view(torch.uint8)
                raw[mine, :, :p % page] = raw[mine[:1], :, :p % page].clone()
    tokens = sum(new)
    s["q"] = normal(tokens, c["heads"], dim, by=2.0)
    s["out"] = torch.empty_like(s["q"])
    s["lens"], s["prefix"], s["groups"] = _ints(lens, dev), _ints(prefix, dev), _ints(cuts, dev)
    s["cu"] = torch.from_numpy(_running(new)).to(dev)
    if own:
        import nested_bit_weight_amd as nbw
        s["cache"] = nbw.KVCache(s["k"], s["v"], s["table"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return s


def _prepare_verify(c, g, dev):
    counts = _verify_counts(c)
    rows, vocab, tokens = c["rows"], c["vocab"], sum(counts)
    kind = torch.float32 if c["dtype"] == "fp32" else torch.bfloat16
    # a few tokens have most of the probability; the narrow child's logits are a little off
    logits = torch.randn(tokens, vocab, generator=g, device=dev).mul_(6.0)
    target = torch.softmax(logits, dim=1).to(kind)
    draft = None
    if c["sampled"]:
        logits.add_(torch.randn(tokens, vocab, generator=g, device=dev), alpha=0.8)
        draft = torch.softmax(logits, dim=1).to(kind)
    del logits
    cu = _running(counts)
    # the drafts: sampled from the child, or what a lookup proposes, often the likeliest token
    last = torch.rand(tokens, 1, generator=g, device=dev)
    if c["sampled"]:
        total = draft.float().cumsum(dim=1)
        pick = torch.searchsorted(total, last * total[:, -1:]).clamp_(max=vocab - 1)[:, 0]
        del total
    else:
        pick = torch.where(last[:, 0] < 0.9, target.float().argmax(dim=1), torch.randint(0, vocab, (tokens,), generator=g, device=dev))
    ids = torch.randint(0, vocab, (tokens,), generator=g, device=dev, dtype=torch.int32)
    ids[1:] = pick[:-1].to(torch.int32)  # the draft at a place follows from the line before it
    return {"case": c, "target": target, "draft": draft, "ids": ids, "u": torch.rand(tokens, generator=g, device=dev),
            "cu": torch.from_numpy(cu).to(dev), "accepted": torch.zeros(rows, dtype=torch.int32, device=dev),
            "next": torch.zeros(rows, dtype=torch.int32, device=dev)}


_PREPARE = {"reserve": _prepare_reserve, "shared": _prepare_shared, "verify": _prepare_verify}


# ---------------------------------------------------------------------------
# one pass

def run(state):
    return _PASSES[state["case"]["op"]](state)


def _reserve_pass(s):
    if own:
        import nested_bit_weight_amd as nbw
        nbw.kv_reserve(s["cache"], s["lens"], s["new"], s["held"], s["free"], s["count"], s["most"], shared=s["kept"],
                       seen=s["seen"], cu=s["cu"], positions=s["positions"], slots=s["slots"], granted=s["granted"],
                       held_out=s["held_out"], count_out=s["count_out"])
    else:
        page, table, free, most = s["page"], s["table"], s["free"], s["most"]
        rows, width = table.shape
        lens, held = s["lens"].long(), s["held"].long()
        keep = held.new_zeros(rows) if s["kept"] is None else s["kept"].long()
        new = torch.where(lens + s["new"] > width * page, 0, s["new"].long())
        pages = torch.maximum((lens + new + page - 1) // page, keep)
        back, take = (held - pages).clamp(min=0), (pages - held).clamp(min=0)
        count = s["count"].long()
        # in order, as long as pages and places for tokens last
        served = (take.cumsum(0) <= count + back.sum()) & (new.cumsum(0) <= most)
        new, take = torch.where(served, new, 0), torch.where(served, take, 0)
        s["granted"].copy_(new)
        s["cu"].copy_(torch.cat([new.new_zeros(1), new.cumsum(0)]))
        s["held_out"].copy_(torch.where(take > 0, pages, held - back))
        s["count_out"].copy_(count + back.sum() - take.sum())
        # pages given back, in the order of rows, are the first to be taken again
        gone_to, taken_at, end = back.cumsum(0) - back, take.cumsum(0) - take, free.numel()
        j = torch.arange(width, device=table.device)[None, :]
        gone = (j >= pages[:, None]) & (j < held[:, None])
        given = free.new_zeros(end + 1)
        given[torch.where(gone, gone_to[:, None] + j - pages[:, None], end)] = table
        nth = taken_at[:, None] + j - held[:, None]
        fresh = torch.where(nth < back.sum(), given[nth.clamp(0, end)], free[(count + back.sum() - 1 - nth).clamp(0, end - 1)])
        table.copy_(torch.where((j >= held[:, None]) & (j < (held + take)[:, None]), fresh, table))
        place = torch.arange(end, device=table.device)
        kept = given[(count + back.sum() - 1 - place).clamp(0, end)]
        free.copy_(torch.where((place >= count) & (place < s["count_out"]), kept, free))
        token = torch.arange(most, device=table.device)
        row = torch.searchsorted(s["cu"][1:], token.to(torch.int32), right=True)
        there = row < rows
        row = row.clamp(max=rows - 1)
        nth = token - s["cu"][row]
        slot = torch.where(there, lens[row] + nth, 0)
        s["positions"].copy_(torch.where(there, s["seen"][row] + nth, 0))
        s["slots"].copy_(torch.where(there, table[row, slot // page].long() * page + slot % page, -1))
    return {name: s[name] for name in ("table", "free", "cu", "positions", "slots", "granted", "held_out", "count_out")}


def _rows_of(s, pool, scale, rows, first, last):
    """Slots first .. last - 1 of some rows in 32 bits, [rows][kv][last - first][dim]."""
    slot = torch.arange(first, max(last, first), device=pool.device)
    page = s["table"][rows].long()[:, slot // s["page"]]
    got = pool[torch.where(page < 0, pool.shape[0] - 1, page), :, slot % s["page"]].float()  # [rows][slots][kv][dim]
    got = got.permute(0, 2, 1, 3)
    return (got if scale is None else got * scale[None, :, None, None]).contiguous()


def _shared_pass(s):
    c = s["case"]
    if own:
        import nested_bit_weight_amd as nbw
        groups, prefix = (s["groups"], s["prefix"]) if c["prefix"] else (None, None)
        nbw.kv_attend_shared(s["cache"], s["q"], s["lens"], cu=s["cu"], groups=groups, prefix=prefix, out=s["out"])
        return {"out": s["out"]}
    cuts, prefix, lens, new = _shared_sizes(c)
    kv, dim, group = c["kv"], c["dim"], c["heads"] // c["kv"]
    cu = _running(new)
    for g, p in enumerate(prefix):
        r0, r1, t0, t1 = cuts[g], cuts[g + 1], int(cu[cuts[g]]), int(cu[cuts[g + 1]])
        n, most, far = t1 - t0, max(new[r0:r1]), max(lens[r0:r1])
        if n == 0:
            continue
        q = s["q"][t0:t1].float().view(n, kv, group, dim).permute(1, 0, 2, 3)  # [kv][n][group][dim]
        token = torch.arange(t0, t1, device=q.device)
        row = torch.searchsorted(s["cu"][1:], token.to(torch.int32), right=True)
        nth = token - s["cu"][row]
        sees = s["lens"][row] - (s["cu"][row + 1] - s["cu"][row]) + 1 + nth  # slots that the token attends to
        # the prefix, once for the group
        k, v = (_rows_of(s, s[x], s[x + "_scale"], slice(r0, r0 + 1), 0, p)[0] for x in ("k", "v"))
        score = [torch.matmul(q.reshape(kv, n * group, dim), k.transpose(1, 2)).view(kv, n, group, p)]
        # each row's own slots, its tokens side by side
        ko, vo = (_rows_of(s, s[x], s[x + "_scale"], slice(r0, r1), p, far) for x in ("k", "v"))
        side = torch.zeros(r1 - r0, kv, most, group, dim, device=q.device)
        side[row - r0, :, nth] = q.permute(1, 0, 2, 3)
        own_score = torch.matmul(side.view(r1 - r0, kv, most * group, dim), ko.transpose(2, 3))
        own_score = own_score.view(r1 - r0, kv, most, group, far - p)
        score.append(own_score[row - r0, :, nth].permute(1, 0, 2, 3))
        score = torch.cat(score, dim=3).div_(math.sqrt(dim))
        slot = torch.arange(far, device=q.device)
        score = torch.where(slot < sees[None, :, None, None], score, -math.inf)
        top = score.amax(dim=3, keepdim=True)
        w = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
        del score
        total = w.sum(dim=3, keepdim=True)
        w = w / torch.where(total == 0, 1.0, total)
        out = torch.matmul(w[..., :p].reshape(kv, n * group, p), v).view(kv, n, group, dim)
        side = torch.zeros(r1 - r0, kv, most, group, far - p, device=q.device)
        side[row - r0, :, nth] = w[..., p:].permute(1, 0, 2, 3)
        there = torch.arange(p, far, device=q.device)[None, :] < s["lens"][r0:r1, None]
        vo = torch.where(there[:, None, :, None], vo, 0.0)
        rest = torch.matmul(side.view(r1 - r0, kv, most * group, far - p), vo).view(r1 - r0, kv, most, group, dim)
        out = out + rest[row - r0, :, nth].permute(1, 0, 2, 3)
        s["out"][t0:t1] = out.permute(1, 0, 2, 3).reshape(n, c["heads"], dim).to(torch.bfloat16)
    return {"out": s["out"]}


def _verify_pass(s):
    if own:
        import nested_bit_weight_amd as nbw
        nbw.verify_drafts(s["target"], s["ids"], s["u"], draft=s["draft"], cu=s["cu"], accepted=s["accepted"], next=s["next"])
        return {"accepted": s["accepted"], "next": s["next"]}
    cu, target, draft = s["cu"].long(), s["target"], s["draft"]
    tokens, vocab = target.shape
    rows = cu.numel() - 1
    token = torch.arange(tokens, device=target.device)
    row = torch.searchsorted(cu[1:], token, right=True)
    ids = torch.cat([s["ids"][1:], s["ids"][:1]]).long()[:, None]  # the draft that follows from each line
    # 64 bits: the product of two numbers of 24 is exact, and so is the comparison
    p = target.gather(1, ids)[:, 0].double()
    q = torch.ones_like(p) if draft is None else draft.gather(1, ids)[:, 0].double()
    refused = ~(s["u"].double() * q < p) | (token == cu[row + 1] - 1)
    at = torch.where(refused, token, tokens)
    stop = torch.full((rows,), tokens, device=target.device).scatter_reduce(0, row, at, "amin")
    s["accepted"].copy_(stop - cu[:-1])
    end = cu[1:] - 1
    line = target[stop].double()
    less = torch.zeros_like(line).scatter_(1, ids[stop], 1.0) if draft is None else draft[stop].double()
    rest = (line - torch.where((stop < end)[:, None], less, 0.0)).clamp_(min=0.0)
    rest = torch.where(rest.sum(dim=1, keepdim=True) > 0, rest, line)
    upto = rest.cumsum(dim=1)
    nth = (upto <= s["u"][end].double()[:, None] * upto[:, -1:]).sum(dim=1)
    last = torch.where(rest > 0, torch.arange(vocab, device=rest.device), -1).amax(dim=1)
    s["next"].copy_(torch.minimum(nth, last))
    return {"accepted": s["accepted"], "next": s["next"]}


_PASSES = {"reserve": _reserve_pass, "shared": _shared_pass, "verify": _verify_pass}


# ---------------------------------------------------------------------------
# the same in 64 bits, one sequence after the other

def exact(case, seed):
    return _EXACT[case["op"]](case, prepare(case, seed))


def _reserve_exact(c, s):
    lens, new, held, kept, seen = ([0] * c["rows"] if s[x] is None else s[x].tolist() for x in ("lens", "new", "held", "kept", "seen"))
    table, free, page = s["table"].tolist(), s["free"].tolist(), c["page"]
    count, most, width = int(s["count"]), s["most"], s["table"].shape[1]
    asked = [t if n + t <= width * page else 0 for n, t in zip(lens, new)]
    stack = free[:count]
    given = []
    for i, n in enumerate(lens):
        stays = max(-(-(n + asked[i]) // page), kept[i])
        given += table[i][stays:held[i]]
        held[i] = min(held[i], max(stays, 0)) if held[i] > stays else held[i]
    stack += given[::-1]
    full, granted, places = False, [], 0
    for i, n in enumerate(lens):
        lacks = max(0, max(-(-(n + asked[i]) // page), kept[i]) - held[i])
        full = full or lacks > len(stack) or places + asked[i] > most
        granted.append(0 if full else asked[i])
        if not full:
            for _ in range(lacks):
                table[i][held[i]] = stack.pop()
                held[i] += 1
            places += asked[i]
    free[count:max(count, len(stack))] = stack[count:]
    positions, slots = np.zeros(most, dtype=np.int32), np.full(most, -1, dtype=np.int64)
    cu = _running(granted)
    for i, n in enumerate(granted):
        nth = np.arange(n)
        positions[cu[i]:cu[i + 1]] = seen[i] + nth
        slots[cu[i]:cu[i + 1]] = np.array(table[i], dtype=np.int64)[(lens[i] + nth) // page] * page + (lens[i] + nth) % page
    got = {"table": table, "free": free, "cu": cu, "positions": positions, "slots": slots, "granted": granted, "held_out": held,
           "count_out": [len(stack)]}
    return {k: torch.from_numpy(np.array(v, dtype=np.int64 if k == "slots" else np.int32)) for k, v in got.items()}


def _shared_exact(c, s):
    cuts, prefix, lens, new = _shared_sizes(c)
    kv, dim, group, page = c["kv"], c["dim"], c["heads"] // c["kv"], c["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    t = 0
    for i, (n, m) in enumerate(zip(lens, new)):
        at = s["table"][i, :-(-n // page)].long()
        for h in range(kv if m else 0):
            k, v = (s[x][at, h].reshape(-1, dim)[:n].double() for x in ("k", "v"))
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            q = s["q"][t:t + m, h * group:(h + 1) * group].double().reshape(m * group, dim)
            score = (q @ k.t().contiguous()) * dim ** -0.5
            behind = torch.arange(n, device="cuda")[None, :] > n - m + torch.arange(m, device="cuda")[:, None]
            score.view(m, group, n).masked_fill_(behind[:, None, :], -math.inf)
            out[t:t + m, h * group:(h + 1) * group] = (torch.softmax(score, dim=1) @ v).view(m, group, dim)
        t += m
    return {"out": out}


def _verify_exact(c, s):
    accepted, after, t = [], [], 0
    ids, u = s["ids"].cpu().numpy(), s["u"].cpu().numpy().astype(np.float64)

    def line(of, i):
        return s[of][i].float().cpu().numpy().astype(np.float64)

    for n in _verify_counts(c):
        i = 0
        while i + 1 < n:
            x = int(ids[t + i + 1])
            q = 1.0 if s["draft"] is None else float(s["draft"][t + i, x])
            if not u[t + i] * q < float(s["target"][t + i, x]):
                break
            i += 1
        rest = line("target", t + i)
        if i + 1 < n:
            less = np.zeros(c["vocab"])
            if s["draft"] is None:
                less[ids[t + i + 1]] = 1.0
            else:
                less = line("draft", t + i)
            more = np.maximum(rest - less, 0.0)
            rest = more if more.any() else rest
        upto = np.cumsum(rest)
        nth = int(np.searchsorted(upto, u[t + n - 1] * upto[-1], side="right"))
        accepted.append(i)
        after.append(min(nth, int(np.flatnonzero(rest).max())))
        t += n
    return {"accepted": torch.tensor(accepted, dtype=torch.int32), "next": torch.tensor(after, dtype=torch.int32)}


_EXACT = {"reserve": _reserve_exact, "shared": _shared_exact, "verify": _verify_exact}
