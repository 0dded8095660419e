"""The paged key-value cache operators, as cases that can be timed and compared.

Five operators around one verify step of a serving loop, each reached through the package's
public calls:

* ``attention``  spec_paged_attention: the attention of a verify block (each stream's N_b drafts
                 and the token before them; N_b = 0 is plain decoding) over a paged cache;
* ``window``     the same call with a sliding window and first tokens that stay visible;
* ``append``     spec_cache_append: the block's keys and values written into their pages;
* ``resize``     spec_cache_resize: room for the next block reserved, and the accepted part of a
                 block kept while the pages of the rest are freed;
* ``fork``       spec_cache_fork followed by spec_cache_resize: a prompt's pages shared with
                 several continuations, and the page that each will write copied for it.

``run`` computes them in elementary torch operations in 32 bits (``own`` false) or calls the
package (``own`` true).  Lengths and draft counts are part of a case (drawn from its sizes alone);
page numbers and contents come from the seed.
"""

import math
import random

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def _att(name, op, streams, drafts, q_heads, kv_heads, head, page, short, long, window=0, sinks=0, type="bf16"):
    return dict(name=name, op=op, streams=streams, drafts=drafts, q_heads=q_heads, kv_heads=kv_heads, head=head,
                page=page, short=short, long=long, window=window, sinks=sinks, type=type)


def listed():
    return [
        # one user, plain decoding, a short context: latency alone
        _att("token_1x1003", "attention", 1, 0, 16, 4, 64, 16, 1003, 1003),
        # the batch-64 verify step: up to 5 drafts a stream, contexts from a question to a document
        _att("verify_64", "attention", 64, 5, 64, 8, 128, 16, 200, 8000),
        # two long documents, 5 drafts: few rows, the context split over the whole GPU
        _att("verify_long", "attention", 2, 5, 64, 8, 128, 64, 100001, 131072),
        # the longest blocks that a verify call takes (32 drafts): the most arithmetic per byte read
        _att("verify_wide", "attention", 16, 32, 64, 8, 128, 32, 500, 4000),
        # the batch-64 verify step of a layer with a window of 1,024 tokens and 4 sinks
        _att("window_64", "window", 64, 5, 64, 8, 128, 16, 500, 16000, window=1024, sinks=4),
        # a float32 model under test, odd window, a few streams
        _att("window_f32", "window", 8, 5, 32, 8, 128, 32, 300, 5000, window=509, sinks=16, type="f32"),
        # one stream's block of up to 6 tokens
        dict(name="append_1", op="append", streams=1, drafts=5, kv_heads=8, head=128, page=16, short=777, long=777,
             type="bf16"),
        # 256 streams with up to 33 tokens each
        dict(name="append_256", op="append", streams=256, drafts=32, kv_heads=8, head=128, page=16, short=20,
             long=2000, type="bf16"),
        # a decode batch's bookkeeping: reserve, then keep what was accepted
        dict(name="resize_64", op="resize", streams=64, drafts=5, kv_heads=8, head=128, page=16, short=100, long=4000,
             layers=2),
        # a large batch over a pool of several hundred thousand pages
        dict(name="resize_1024", op="resize", streams=1024, drafts=9, kv_heads=1, head=64, page=16, short=100,
             long=8000, layers=1),
        # one prompt, eight continuations
        dict(name="fork_8", op="fork", prompts=1, children=8, drafts=5, kv_heads=4, head=64, page=16, short=1000,
             long=1000, layers=4),
        # 16 prompts with 15 continuations each, 16 layers: the copies of the written pages dominate
        dict(name="fork_240", op="fork", prompts=16, children=15, drafts=5, kv_heads=8, head=128, page=16, short=500,
             long=3000, layers=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "window", "window", "append", "resize", "fork"])
    if op in ("attention", "window"):
        kv = rng.choice([1, 2, 4, 8])
        c = _att("", op, _log(rng, 1, 128), rng.choice([0, 1, 2, 3, 5, 7, 9, 16, 32]), kv * rng.choice([1, 2, 3, 4, 7, 8]),
                 kv, rng.choice([64, 128, 128, 128, 80, 256]), rng.choice([8, 16, 32, 64, 128]), 0, 0,
                 type=rng.choice(["bf16", "bf16", "bf16", "f32"]))
        budget = 300000 * 8 * 128 // (kv * c["head"])  # tokens of all streams together
        budget = min(budget, 300000 * 64 * 6 // (c["q_heads"] * (c["drafts"] + 1)))
        if c["type"] == "f32":
            budget //= 8
        top = max(40, min(100000, budget // c["streams"]))
        c["long"] = _log(rng, 40, top)
        c["short"] = rng.randint(max(1, c["long"] // 20), c["long"])
        if op == "window":
            c["window"] = _log(rng, 1, 4000)
            c["sinks"] = rng.choice([0, 1, 4, 17, 128])
    elif op == "append":
        c = dict(op=op, streams=_log(rng, 1, 256), drafts=rng.choice([0, 1, 3, 5, 9, 32]), kv_heads=rng.choice([1, 2, 4, 8]),
                 head=rng.choice([64, 80, 128]), page=rng.choice([8, 16, 32, 64]), type=rng.choice(["bf16", "bf16", "f32"]))
        c["long"] = _log(rng, 30, 1500)
        c["short"] = rng.randint(1, c["long"])
    elif op == "resize":
        c = dict(op=op, streams=_log(rng, 1, 1024), drafts=rng.choice([0, 1, 3, 5, 9, 32]), kv_heads=1, head=64,
                 page=rng.choice([8, 16, 32, 64]), layers=1)
        c["long"] = _log(rng, 70, 6000)
        c["short"] = rng.randint(40, c["long"])
    else:
        c = dict(op=op, prompts=_log(rng, 1, 16), children=_log(rng, 1, 12), drafts=rng.choice([0, 3, 5, 9]),
                 kv_heads=rng.choice([1, 2, 4]), head=rng.choice([64, 128]), page=rng.choice([8, 16, 32]),
                 layers=rng.choice([1, 2, 4, 8]))
        c["long"] = _log(rng, 30, 3000)
        c["short"] = rng.randint(1, c["long"])
    c.pop("name", None)
    return c


def _sizes(case, streams):
    """(length, drafts) of each stream, from the case's sizes alone: lengths spread over their
    logarithm, the longest among them; draft counts from 0 to the most, the most among them."""
    rng = random.Random("%d %d %d %d" % (streams, case["drafts"], case["short"], case["long"]))
    length = [_log(rng, case["short"], case["long"]) for _ in range(streams)]
    length[0] = case["long"]
    drafts = [rng.randint((case["drafts"] + 1) // 2, case["drafts"]) for _ in range(streams)]
    drafts[-1] = case["drafts"]
    return np.array(length, np.int64), np.array(drafts, np.int64)


def _ceil(a, b):
    return -(-a // b)


# ---------------------------------------------------------------------------------------------
# what a program has in hand
# ---------------------------------------------------------------------------------------------
def _cache(g, dev, held, width, spare, layers, kv_heads, page, head, dtype):
    """A pool of pages and the table of streams that hold `held` pages each, page numbers at random."""
    total = int(held.sum())
    pages = total + spare
    order = torch.randperm(pages, generator=g, device=dev)[:total].to(torch.int32)
    h = torch.from_numpy(held).to(dev)
    col = torch.arange(width, device=dev)
    mine = col[None, :] < h[:, None]
    table = torch.full((len(held), width), -1, dtype=torch.int32, device=dev)
    table[mine] = order
    refs = torch.zeros(pages, dtype=torch.int32, device=dev)
    refs[order.long()] = 1
    shape = (layers, pages, kv_heads, page, head)
    k = torch.randn(shape, generator=g, device=dev, dtype=dtype)
    v = torch.randn(shape, generator=g, device=dev, dtype=dtype)
    return k, v, table, h.to(torch.int32), refs


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op, P = case["op"], case["page"]
    s = dict(op=op, page=P, kmax=case["drafts"])
    if op in ("attention", "window", "append"):
        dtype = TYPES[case["type"]]
        length, drafts = _sizes(case, case["streams"])
        held = _ceil(length + drafts + 1, P)
        k, v, s["table"], s["held"], _ = _cache(g, dev, held, int(held.max()) + 1, 7, 1, case["kv_heads"], P,
                                                case["head"], dtype)
        s["k"], s["v"] = k[0], v[0]
        s["length"] = torch.from_numpy(length).to(dev, torch.int32)
        s["cu"] = torch.from_numpy(np.concatenate([[0], np.cumsum(drafts)])).to(dev, torch.int32)
        rows = int(drafts.sum()) + len(drafts)
        if op == "append":
            s["new_k"] = torch.randn((rows, case["kv_heads"], case["head"]), generator=g, device=dev, dtype=dtype)
            s["new_v"] = torch.randn((rows, case["kv_heads"], case["head"]), generator=g, device=dev, dtype=dtype)
        else:
            # queries longer than keys: scores spread as in a trained head (a few keys carry a row)
            q = torch.randn((rows, case["q_heads"], case["head"]), generator=g, device=dev, dtype=torch.float32)
            s["q"] = (2.5 * q).to(dtype)
            s["scale"] = 1.0 / math.sqrt(case["head"])
            s["window"], s["sinks"] = case["window"], case["sinks"]
    elif op == "resize":
        length, drafts = _sizes(case, case["streams"])
        held = _ceil(length, P)
        k, v, s["table"], s["held"], s["refs"] = _cache(
            g, dev, held, int(_ceil(length + 2 * (drafts + 1), P).max()), int(_ceil(2 * (drafts + 1), P).sum()) + 64,
            case["layers"], case["kv_heads"], P, case["head"], torch.bfloat16)
        s["k"], s["v"] = k, v
        s["length"] = torch.from_numpy(length).to(dev, torch.int32)
        s["room"] = torch.from_numpy(drafts + 1).to(dev, torch.int32)
        # tokens kept by the verify step; the next pass takes the same ones back (a stream that is
        # rolled back), so that passes can follow one another without end
        kept = 1 + (torch.rand(len(drafts), generator=g, device=dev) * (s["room"] - 0.5)).to(torch.int32)
        s["advance"] = [torch.minimum(kept, s["room"]).contiguous(), (-torch.minimum(kept, s["room"])).contiguous()]
        s["turn"] = 0
    else:
        n, m = case["prompts"], case["children"]
        length, drafts = _sizes(case, n)
        streams = n * (1 + m)
        held = np.zeros(streams, np.int64)
        held[:n] = _ceil(length, P)
        grown = _ceil(length + case["drafts"] + 1, P)
        k, v, s["table"], s["held"], s["refs"] = _cache(
            g, dev, held, int(grown.max()), int(((1 + m) * (grown - length // P)).sum()) + 64, case["layers"],
            case["kv_heads"], P, case["head"], torch.bfloat16)
        s["k"], s["v"] = k, v
        s["length"] = torch.zeros(streams, dtype=torch.int32, device=dev)
        s["length"][:n] = torch.from_numpy(length).to(dev, torch.int32)
        s["src"] = torch.arange(n, device=dev, dtype=torch.int32).repeat_interleave(m)
        s["dst"] = (n + torch.arange(n * m, device=dev)).to(torch.int32)
        s["room"] = torch.full((streams,), case["drafts"] + 1, dtype=torch.int32, device=dev)
    return s


# ---------------------------------------------------------------------------------------------
# the operators in elementary torch operations
# ---------------------------------------------------------------------------------------------
def _rows(s, rows):
    """(stream, token of its block, position) of each packed row."""
    cu = s["cu"].long()
    B = cu.numel() - 1
    n = cu[1:] - cu[:-1] + 1
    stream = torch.repeat_interleave(torch.arange(B, device=cu.device), n, output_size=rows)
    i = torch.arange(rows, device=cu.device) - cu[stream] - stream
    return stream, i, s["length"].long()[stream] + i


def _plain_attention(s):
    q, kp, vp, table = s["q"], s["k"], s["v"], s["table"]
    rows, Hq, D = q.shape
    Hkv, P = kp.shape[1], kp.shape[2]
    B, n, G = table.shape[0], s["kmax"] + 1, Hq // kp.shape[1]
    stream, i, pos = _rows(s, rows)
    qp = torch.zeros((B, n, Hkv, G, D), dtype=torch.float32, device=q.device)
    qp[stream, i] = q.float().view(rows, Hkv, G, D)
    qp = qp.permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D)
    t = table.long().clamp(min=0)
    S = t.shape[1] * P
    k = kp[t].permute(0, 2, 1, 3, 4).reshape(B, Hkv, S, D).float()
    w = torch.matmul(qp, k.transpose(2, 3)) * s["scale"]
    del k
    j = torch.arange(S, device=q.device)
    at = s["length"].long()[:, None] + torch.arange(n, device=q.device)
    sees = j <= at[:, :, None]
    if s["window"]:
        sees &= (j > at[:, :, None] - s["window"]) | (j < s["sinks"])
    sees = sees[:, None, :, None, :].expand(B, 1, n, G, S).reshape(B, 1, n * G, S)
    w = w.masked_fill_(~sees, float("-inf"))
    w = torch.exp(w - w.amax(dim=-1, keepdim=True))
    total = w.sum(dim=-1, keepdim=True)
    v = vp[t].permute(0, 2, 1, 3, 4).reshape(B, Hkv, S, D).float()
    o = (torch.matmul(w, v) / total).view(B, Hkv, n, G, D).permute(0, 2, 1, 3, 4).reshape(B, n, Hq, D)
    return {"out": o[stream, i].to(q.dtype), "status": torch.zeros(B, dtype=torch.int32, device=q.device)}


def _plain_append(s):
    rows, P = s["new_k"].shape[0], s["page"]
    stream, _, pos = _rows(s, rows)
    page = s["table"][stream, pos // P].long()
    s["k"][page, :, pos % P] = s["new_k"]
    s["v"][page, :, pos % P] = s["new_v"]
    return {"k": s["k"], "v": s["v"], "status": torch.zeros(s["table"].shape[0], dtype=torch.int32, device=s["k"].device)}


def _plain_resize(s, advance, room):
    table, held, length, refs, P = s["table"], s["held"], s["length"], s["refs"], s["page"]
    B, width = table.shape
    col = torch.arange(width, device=table.device)
    n = length.long() + (0 if advance is None else advance.long())
    room = torch.zeros_like(n) if room is None else room.long()
    have = held.long()
    want = (n + room + P - 1) // P
    full = (n + P - 1) // P
    # pages past the kept tokens that another stream holds too are given up from the first one on
    shared = (col >= full[:, None]) & (col < torch.minimum(want, have)[:, None]) & (refs[table.clamp(min=0).long()] > 1)
    first = torch.where(shared, col, width).amin(dim=1)
    keep = torch.minimum(torch.minimum(want, have), first)
    drop = (col >= keep[:, None]) & (col < have[:, None])
    refs.index_add_(0, table.clamp(min=0).long().reshape(-1), -drop.to(torch.int32).reshape(-1))
    table.masked_fill_(drop, -1)
    # the page that holds both kept tokens and room, where another stream holds it too
    tail = n // P
    page = table.gather(1, tail.clamp(max=width - 1)[:, None])[:, 0].long().clamp(min=0)
    asks = (n % P != 0) & (room > 0) & (tail < keep) & (refs[page] > 1)
    askers = torch.zeros_like(refs).index_add_(0, page, asks.to(torch.int32))
    index = torch.arange(B, device=table.device)
    lowest = torch.full(refs.shape, B, dtype=torch.int64, device=table.device)
    lowest.scatter_reduce_(0, page, torch.where(asks, index, B), "amin")
    copy = asks & ~((askers[page] == refs[page]) & (lowest[page] == index))
    # the lowest pages that nobody holds, in the order of the streams
    need = want - keep + copy.long()
    begin = torch.cumsum(need, 0) - need
    free = torch.nonzero(refs == 0)[:, 0]
    fits = (begin + need <= free.numel()) | (need == 0)
    copy &= fits
    got = torch.where(fits, want, keep)
    new = free[begin[copy]]
    old = page[copy]
    refs.index_add_(0, old, torch.full_like(old, -1, dtype=torch.int32))
    s["k"][:, new] = s["k"][:, old]
    s["v"][:, new] = s["v"][:, old]
    table[index[copy], tail[copy]] = new.to(torch.int32)
    refs[new] = 1
    grow = (col >= keep[:, None]) & (col < got[:, None])
    nth = (begin + copy.long())[:, None] + col - keep[:, None]
    taken = free[nth[grow]]
    table[grow] = taken.to(torch.int32)
    refs[taken] = 1
    held.copy_(got)
    length.copy_(n)
    return torch.where(fits, 0, 8).to(torch.int32)


def _plain_fork(s):
    table, held, length, refs, P = s["table"], s["held"], s["length"], s["refs"], s["page"]
    src, dst = s["src"].long(), s["dst"].long()
    col = torch.arange(table.shape[1], device=table.device)
    old, gives = table[dst], col < held[dst][:, None]
    refs.index_add_(0, old.clamp(min=0).long().reshape(-1), -gives.to(torch.int32).reshape(-1))
    n = length[src]
    pages = (n + P - 1) // P
    takes = col < pages[:, None]
    row = torch.where(takes, table[src], -1)
    refs.index_add_(0, row.clamp(min=0).long().reshape(-1), takes.to(torch.int32).reshape(-1))
    table[dst] = row
    held[dst] = pages
    length[dst] = n
    return torch.zeros(src.numel(), dtype=torch.int32, device=src.device)


def _book(s, *status):
    return {"table": s["table"], "held": s["held"], "length": s["length"], "refs": s["refs"], "status": list(status)}


def run(s):
    if own:
        return _run_own(s)
    if s["op"] in ("attention", "window"):
        return _plain_attention(s)
    if s["op"] == "append":
        return _plain_append(s)
    if s["op"] == "resize":
        advance = s["advance"][s["turn"]]
        s["turn"] ^= 1
        return _book(s, _plain_resize(s, None, s["room"]), _plain_resize(s, advance, None))
    return dict(_book(s, _plain_fork(s), _plain_resize(s, None, s["room"])), k=s["k"], v=s["v"])


def _run_own(s):
    import speculative_decoding_block_verify_gb300 as sv

    if s["op"] in ("attention", "window"):
        s["out"] = r = sv.spec_paged_attention(s["q"], s["k"], s["v"], s["table"], s["length"], s["cu"], s["kmax"],
                                               s["scale"], window=s["window"], sinks=s["sinks"], out=s.get("out"))
        return {"out": r["out"], "status": r["status"]}
    if s["op"] == "append":
        s["out"] = r = sv.spec_cache_append(s["new_k"], s["new_v"], s["k"], s["v"], s["table"], s["length"], s["cu"],
                                            s["kmax"], out=s.get("out"))
        return {"k": s["k"], "v": s["v"], "status": r["status"]}
    book = (s["table"], s["held"], s["length"], s["refs"])
    if s["op"] == "resize":
        advance = s["advance"][s["turn"]]
        s["turn"] ^= 1
        s["out"] = a = sv.spec_cache_resize(s["k"], s["v"], *book, room=s["room"], out=s.get("out"))
        s["out2"] = b = sv.spec_cache_resize(s["k"], s["v"], *book, advance=advance, out=s.get("out2"))
        return _book(s, a["status"], b["status"])
    s["out"] = a = sv.spec_cache_fork(s["src"], s["dst"], *book, s["page"], out=s.get("out"))
    s["out2"] = b = sv.spec_cache_resize(s["k"], s["v"], *book, room=s["room"], out=s.get("out2"))
    return dict(_book(s, a["status"], b["status"]), k=s["k"], v=s["v"])


# ---------------------------------------------------------------------------------------------
# work and definition
# ---------------------------------------------------------------------------------------------
def _visible(n, window, sinks):
    """How many of the positions 0..n-1 the token at position n - 1 sees."""
    if not window or n <= window:
        return n
    return window + min(sinks, n - window)


def work(case):
    op, P = case["op"], case["page"]
    if op in ("attention", "window"):
        length, drafts = _sizes(case, case["streams"])
        size = 2 if case["type"] == "bf16" else 4
        W, S = case["window"], case["sinks"]
        read = pairs = 0
        for n, d in zip(length.tolist(), drafts.tolist()):
            last = n + d + 1
            low = max(0, n + 1 - W) if W else 0   # the first row's window begins here
            read += last - low + min(S, low)
            pairs += sum(_visible(n + i + 1, W, S) for i in range(d + 1))
        rows = int((drafts + 1).sum())
        return {"bytes": (read * case["kv_heads"] + rows * case["q_heads"]) * 2 * case["head"] * size
                + 4 * read // P + 12 * len(drafts),
                "flops": 4 * pairs * case["q_heads"] * case["head"]}
    if op == "append":
        length, drafts = _sizes(case, case["streams"])
        size = 2 if case["type"] == "bf16" else 4
        rows = int((drafts + 1).sum())
        return {"bytes": 4 * rows * case["kv_heads"] * case["head"] * size + 4 * rows + 12 * len(drafts), "flops": 0}
    token = 2 * 2 * case["kv_heads"] * case["head"] * case["layers"]   # bytes of one token's keys and values
    if op == "resize":
        length, drafts = _sizes(case, case["streams"])
        new = int((_ceil(length + drafts + 1, P) - _ceil(length, P)).sum())
        # both calls: lengths, held counts (read and written), one input, status; the new pages'
        # table entries and counts, given out and taken back; counts looked through for the new pages
        return {"bytes": 2 * 24 * len(length) + 2 * new * 12 + 4 * 2 * int(_ceil(length, P).sum()), "flops": 0}
    length, _ = _sizes(case, case["prompts"])
    m = case["children"]
    pages = _ceil(length, P)
    book = m * int(pages.sum()) * (4 + 4 + 4 + 8 + 8)   # old entries, new entries (read, written), counts twice
    copies = m * int((length % P != 0).sum()) * P * token * 2
    return {"bytes": book + copies + 40 * (1 + m) * len(length), "flops": 0}


def exact(case, seed):
    """What run() returns, from the definitions, one row (one page) after the other."""
    if case["op"] == "resize":
        return None   # whole numbers only
    s = prepare(case, seed)

    def attention():
        length, drafts = _sizes(case, case["streams"])
        q = s["q"]
        G, P = case["q_heads"] // case["kv_heads"], s["page"]
        out = torch.empty(q.shape, dtype=torch.float64, device=q.device)
        at = 0
        for b in range(len(length)):
            L, n = int(length[b]), int(drafts[b]) + 1
            pages = s["table"][b, :_ceil(L + n, P)].long()
            for h in range(case["kv_heads"]):
                k = s["k"][pages, h].double().reshape(-1, case["head"])[:L + n]
                v = s["v"][pages, h].double().reshape(-1, case["head"])[:L + n]
                for i in range(n):
                    p = L + i
                    low = max(0, p + 1 - case["window"]) if case["window"] else 0
                    first = min(case["sinks"], low)
                    kk = torch.cat([k[:first], k[low:p + 1]]) if low else k[:p + 1]
                    vv = torch.cat([v[:first], v[low:p + 1]]) if low else v[:p + 1]
                    x = kk @ q[at + i, h * G:(h + 1) * G].double().T * s["scale"]
                    out[at + i, h * G:(h + 1) * G] = torch.softmax(x, dim=0).T @ vv
            at += n
        return {"out": out, "status": None}

    def append():
        length, drafts = _sizes(case, case["streams"])
        k, v, table = s["k"].double(), s["v"].double(), s["table"].tolist()
        r = 0
        for b in range(len(length)):
            for p in range(int(length[b]), int(length[b] + drafts[b]) + 1):
                k[table[b][p // s["page"]], :, p % s["page"]] = s["new_k"][r].double()
                v[table[b][p // s["page"]], :, p % s["page"]] = s["new_v"][r].double()
                r += 1
        return {"k": k, "v": v, "status": None}

    def fork():
        """One fork and the resize after it, page by page: where each written page is copied to."""
        P, room = s["page"], case["drafts"] + 1
        n, m = case["prompts"], case["children"]
        length, _ = _sizes(case, n)
        k, v = s["k"].double(), s["v"].double()
        refs, table = s["refs"].tolist(), s["table"].tolist()
        free = (p for p in range(len(refs)) if refs[p] == 0)
        for b in range(n * (1 + m)):   # the streams in order; the lowest holder of a shared page keeps it
            parent = b if b < n else (b - n) // m
            L = int(length[parent])
            if L % P and b >= n:
                page = next(free)
                k[:, page] = k[:, table[parent][L // P]]
                v[:, page] = v[:, table[parent][L // P]]
            for _ in range(_ceil(L + room, P) - _ceil(L, P)):
                next(free)
        return {"table": None, "held": None, "length": None, "refs": None, "status": [None, None], "k": k, "v": v}

    return {"append": append, "fork": fork}.get(case["op"], attention)()
