"""What a prompt goes through on its way into the paged cache, as cases that can be timed and compared.

Three operators, each reached through the package's public calls:

* ``prompt``  spec_prompt_attention: causal attention over whole prompts, packed one behind the other, with
              grouped heads and an optional sliding window with first tokens that stay visible;
* ``rotate``  spec_rotate: rotary positions of packed rows (halves or interleaved pairs, all of the head or
              its first elements, frequencies scaled for long contexts);
* ``append``  spec_cache_append_rotated: a block's or a whole prompt's keys rotated into their pages, its
              values beside them, and the queries rotated on the way.

``run`` computes them in elementary torch operations in 32 bits (``own`` false; the angles, which grow with the position,
in 64) or calls the package (``own`` true).  Lengths and row counts are part of a case (drawn from its sizes alone);
contents, page numbers and far positions come from the seed.
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
def _prompt(name, prompts, short, long, q_heads, kv_heads, head, window=0, sinks=0, type="bf16"):
    return dict(name=name, op="prompt", streams=prompts, short=short, long=long, q_heads=q_heads, kv_heads=kv_heads,
                head=head, window=window, sinks=sinks, type=type)


def _turn(dim, base=10000.0, scaling="none", factor=1.0, original=4096, interleaved=False):
    return dict(dim=dim, base=base, scaling=scaling, factor=factor, original=original, interleaved=interleaved)


def listed():
    return [
        # one user's question: latency alone
        _prompt("prompt_1x333", 1, 333, 333, 16, 4, 64),
        # a batch of questions, a few tokens to two thousand each: ragged, most of it short
        _prompt("prompts_24", 24, 17, 2000, 64, 8, 128),
        # one long document: the most arithmetic
        _prompt("prompt_16001", 1, 16001, 16001, 64, 8, 128),
        # documents through a layer with a window of 1,024 tokens and 4 sinks
        _prompt("prompts_window", 6, 2000, 9000, 64, 8, 128, window=1024, sinks=4),
        # a float32 model under test
        _prompt("prompts_f32", 5, 100, 1500, 32, 8, 128, type="f32"),
        # one verify block's queries and keys, as they lie beside each other in a projection
        dict(_turn(64, interleaved=True), name="rotate_6", op="rotate", rows=6, heads=20, beside=4, head=64, far=2000, type="bf16"),
        # a long prompt's queries and keys, positions scaled for a long context
        dict(_turn(128, base=500000.0, scaling="yarn", factor=16.0, original=8192), name="rotate_8191", op="rotate", rows=8191,
             heads=72, beside=8, head=128, far=131072, type="bf16"),
        # a float32 model whose heads turn in part
        dict(_turn(32, scaling="linear", factor=4.0, interleaved=True), name="rotate_part_f32", op="rotate", rows=2047, heads=40,
             beside=8, head=80, far=16384, type="f32"),
        # one stream's verify block of up to 6 tokens
        dict(_turn(64), name="turn_append_1", op="append", streams=1, least=6, most=6, q_heads=16, kv_heads=4, head=64, page=16,
             short=777, long=777, keep=False, type="bf16"),
        # the batch-64 verify step, contexts from a question to a document
        dict(_turn(128, base=500000.0, scaling="yarn", factor=16.0, original=8192), name="turn_append_64", op="append", streams=64,
             least=3, most=6, q_heads=64, kv_heads=8, head=128, page=16, short=200, long=16384, keep=False, type="bf16"),
        # a batch of prompts into an empty cache; the turned keys are kept for spec_prompt_attention
        dict(_turn(128, scaling="ntk", factor=8.0), name="turn_append_prompts", op="append", streams=24, least=17, most=2000, q_heads=64,
             kv_heads=8, head=128, page=16, short=0, long=0, keep=True, type="bf16"),
        # float32, second turns of conversations behind what is cached, heads that turn in part
        dict(_turn(32), name="turn_append_f32", op="append", streams=9, least=1, most=500, q_heads=32, kv_heads=8, head=80, page=32,
             short=1, long=3000, keep=True, type="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_turn(rng, head):
    dim = rng.choice([head, head, head, head // 2, head // 4, head - 2 * rng.randint(1, head // 4), 2 * rng.randint(2, head // 2)])
    return _turn(dim, base=rng.choice([10000.0, 500000.0, 1000000.0]), scaling=rng.choice(["none", "none", "linear", "ntk", "yarn", "yarn"]),
                 factor=rng.choice([1.0, 2.0, 3.5, 8.0, 32.0]), original=rng.choice([2048, 4096, 8192, 32768]),
                 interleaved=rng.choice([False, False, True]))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt", "rotate", "append", "append"])
    head = rng.choice([64, 128, 128, 128, 80, 96])
    kv = rng.choice([1, 2, 4, 8])
    q = kv * rng.choice([1, 2, 3, 4, 7, 8])
    type = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "prompt":
        c = _prompt("", _log(rng, 1, 64), 0, 0, q, kv, head, type=type)
        budget = 16001 * 16001 * 64 * 128 / (q * head)   # pairs of positions of all prompts together
        if type == "f32":
            budget /= 16
        if rng.random() < 0.35:
            c["window"], c["sinks"] = _log(rng, 1, 4000), rng.choice([0, 1, 4, 17, 300])
        c["long"] = _log(rng, 2, min(20000, math.sqrt(budget / c["streams"])))
        c["short"] = rng.randint(1, max(1, c["long"] // 3))
    elif op == "rotate":
        c = dict(_draw_turn(rng, head), op=op, rows=_log(rng, 1, 8191), heads=q + kv, beside=rng.choice([0, 0, kv, 1]), head=head,
                 far=_log(rng, 100, 1000000), type=type)
    else:
        c = dict(_draw_turn(rng, head), op=op, streams=_log(rng, 1, 128), q_heads=q, kv_heads=kv, head=head,
                 page=rng.choice([8, 16, 32, 64, 128]), keep=rng.choice([False, True]), type=type)
        c["most"] = _log(rng, 1, min(3000, 20000 // c["streams"]))
        c["least"] = rng.randint(1, c["most"])
        c["long"] = rng.choice([0, _log(rng, 10, min(100000, 300000 * 8 * 128 // (c["streams"] * kv * head)))])
        c["short"] = rng.randint(0, c["long"])
    c.pop("name", None)
    return c


def _counts(case):
    """(length, rows) of each stream, from the case's sizes alone, spread over their logarithm: `length` is what is cached before
    (0 for a prompt), `rows` what comes.  The most are among them, and with several streams the least too."""
    n = case["streams"]
    rng = random.Random("%d %d %d" % (n, case["short"], case["long"]))
    if case["op"] == "prompt":
        length, lo, hi = np.zeros(n, np.int64), case["short"], case["long"]
    else:
        length = np.array([_log(rng, case["short"] + 1, case["long"] + 1) - 1 for _ in range(n)], np.int64)
        length[0] = case["long"]
        lo, hi = case["least"], case["most"]
    rows = np.array([_log(rng, lo, hi) for _ in range(n)], np.int64)
    rows[-1] = lo
    rows[n // 2] = hi
    return length, rows


def _ceil(a, b):
    return -(-a // b)


# ---------------------------------------------------------------------------------------------
# what a program has in hand
# ---------------------------------------------------------------------------------------------
def _frequencies(c):
    """Radians a position of each pair (64 bits), and the factor of the turned elements."""
    d, s = c["dim"], c["factor"]
    j = np.arange(d // 2, dtype=np.float64)
    base = c["base"]
    if c["scaling"] == "ntk" and d > 2:
        base = base * s ** (d / (d - 2))
    f = base ** (-2 * j / d)
    if c["scaling"] == "linear":
        f = f / s
    if c["scaling"] == "yarn":   # pairs that turn less than once in the original context are stretched, those above 32 left
        turns = c["original"] * f / (2 * math.pi)
        g = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        f = f * g + f / s * (1 - g)
    return f, (0.1 * math.log(s) + 1.0 if c["scaling"] == "yarn" else 1.0)


def _rotary(s, case, dev):
    f, s["magnitude"] = _frequencies(case)
    s["frequency"] = torch.from_numpy(f).to(dev)
    s["dim"], s["interleaved"] = case["dim"], case["interleaved"]
    if own:
        import speculative_decoding_block_verify_gb300 as sv

        s["rotary"] = sv.RotaryTable(case["dim"], base=case["base"], scaling=case["scaling"], factor=case["factor"],
                                     original=case["original"], interleaved=case["interleaved"])


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dtype, D = TYPES[case["type"]], case["head"]
    s = dict(op=case["op"])
    if case["op"] == "rotate":
        # the turned heads are the first of a wider projection (`beside`: the values' heads)
        wide = torch.randn((case["rows"], case["heads"] + case["beside"], D), generator=g, device=dev, dtype=torch.float32).to(dtype)
        s["x"] = wide[:, :case["heads"]]
        s["positions"] = torch.randint(0, case["far"], (case["rows"],), generator=g, device=dev, dtype=torch.int32)
        _rotary(s, case, dev)
        return s
    length, rows = _counts(case)
    n, H, G = int(rows.sum()), case["q_heads"], case["kv_heads"]
    # queries, keys and values as they lie in one projection; queries longer than keys: scores spread as in a trained head
    wide = torch.randn((n, H + 2 * G, D), generator=g, device=dev, dtype=torch.float32)
    wide[:, :H] *= 2.5
    wide = wide.to(dtype)
    s["q"], s["k"], s["v"] = wide[:, :H], wide[:, H:H + G], wide[:, H + G:]
    s["rows"] = rows.tolist()
    s["cu"] = torch.from_numpy(np.concatenate([[0], np.cumsum(rows)])).to(dev, torch.int32)
    if case["op"] == "prompt":
        s["scale"], s["window"], s["sinks"] = 1.0 / math.sqrt(D), case["window"], case["sinks"]
        return s
    P = case["page"]
    held = _ceil(length + rows, P)
    total = int(held.sum())
    pages = total + 7
    order = torch.randperm(pages, generator=g, device=dev)[:total].to(torch.int32)
    col = torch.arange(int(held.max()) + 1, device=dev)
    mine = col[None, :] < torch.from_numpy(held).to(dev)[:, None]
    s["table"] = torch.full(mine.shape, -1, dtype=torch.int32, device=dev)
    s["table"][mine] = order
    s["page"], s["keep"] = P, case["keep"]
    s["length"] = torch.from_numpy(length).to(dev, torch.int32)
    s["k_pages"] = torch.zeros((pages, G, P, D), dtype=dtype, device=dev)
    s["v_pages"] = torch.zeros_like(s["k_pages"])
    _rotary(s, case, dev)
    return s


# ---------------------------------------------------------------------------------------------
# the operators in elementary torch operations
# ---------------------------------------------------------------------------------------------
def _plain_turn(s, x, positions):
    angle = positions.double()[:, None] * s["frequency"]
    c = (torch.cos(angle) * s["magnitude"]).float()[:, None, :]
    n = (torch.sin(angle) * s["magnitude"]).float()[:, None, :]
    d = s["dim"]
    y = x.float()
    a, b = (y[..., 0:d:2], y[..., 1:d:2]) if s["interleaved"] else (y[..., :d // 2], y[..., d // 2:d])
    a, b = a * c - b * n, b * c + a * n
    turned = torch.stack([a, b], dim=-1).flatten(-2) if s["interleaved"] else torch.cat([a, b], dim=-1)
    return torch.cat([turned, y[..., d:]], dim=-1).to(x.dtype)


def _plain_prompt(s):
    q, k, v = s["q"], s["k"], s["v"]
    H, G, D = q.shape[1], k.shape[1], q.shape[2]
    out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    at = 0
    for n in s["rows"]:
        kk = k[at:at + n].float().permute(1, 2, 0)   # [G, D, n]
        vv = v[at:at + n].float().permute(1, 0, 2)   # [G, n, D]
        step = max(16, min(n, (1 << 28) // (n * H)))
        for i0 in range(0, n, step):
            i1 = min(n, i0 + step)
            qq = q[at + i0:at + i1].float().view(i1 - i0, G, H // G, D).permute(1, 2, 0, 3)
            w = torch.matmul(qq.reshape(G, -1, D), kk[:, :, :i1]) * s["scale"]
            w = w.view(G, H // G, i1 - i0, i1)
            i, j = torch.arange(i0, i1, device=q.device)[:, None], torch.arange(i1, device=q.device)[None, :]
            sees = j <= i
            if s["window"]:
                sees &= (j > i - s["window"]) | (j < s["sinks"])
            w = w.masked_fill_(~sees, float("-inf"))
            w = w.sub_(w.amax(dim=-1, keepdim=True)).exp_()
            total = w.sum(dim=-1, keepdim=True)
            o = torch.matmul(w.view(G, -1, i1), vv[:, :i1]).view(G, H // G, i1 - i0, D) / total
            out[at + i0:at + i1] = o.permute(2, 0, 1, 3).reshape(i1 - i0, H, D).to(q.dtype)
        at += n
    return {"out": out, "status": torch.zeros(len(s["rows"]), dtype=torch.int32, device=q.device)}


def _plain_append(s):
    rows, B, P = s["q"].shape[0], s["table"].shape[0], s["page"]
    cu = s["cu"].long()
    stream = torch.repeat_interleave(torch.arange(B, device=cu.device), cu[1:] - cu[:-1], output_size=rows)
    at = s["length"].long()[stream] + torch.arange(rows, device=cu.device) - cu[stream]
    q, k = _plain_turn(s, s["q"], at), _plain_turn(s, s["k"], at)
    page = s["table"][stream, at // P].long()
    s["k_pages"][page, :, at % P] = k
    s["v_pages"][page, :, at % P] = s["v"]
    out = {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"], "status": torch.zeros(B, dtype=torch.int32, device=cu.device)}
    if s["keep"]:
        out["k"] = k
    return out


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "prompt":
        return _plain_prompt(s)
    if s["op"] == "rotate":
        return {"out": _plain_turn(s, s["x"], s["positions"])}
    return _plain_append(s)


def _run_own(s):
    import speculative_decoding_block_verify_gb300 as sv

    if s["op"] == "prompt":
        s["out"] = r = sv.spec_prompt_attention(s["q"], s["k"], s["v"], s["cu"], s["scale"], window=s["window"], sinks=s["sinks"],
                                                out=s.get("out"))
        return {"out": r["out"], "status": r["status"]}
    if s["op"] == "rotate":
        s["out"] = r = sv.spec_rotate(s["x"], s["positions"], s["rotary"], out=s.get("out"))
        return {"out": r}
    s["out"] = r = sv.spec_cache_append_rotated(s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["length"], s["rotary"],
                                                cu_rows=s["cu"], keep_keys=s["keep"], out=s.get("out"))
    out = {"q": r["q"], "k_pages": s["k_pages"], "v_pages": s["v_pages"], "status": r["status"]}
    if s["keep"]:
        out["k"] = r["k"]
    return out


# ---------------------------------------------------------------------------------------------
# work and definition
# ---------------------------------------------------------------------------------------------
def _pairs(n, window, sinks):
    """Pairs (i, j) of a prompt of n tokens where token i sees token j."""
    if not window or n <= window:
        return n * (n + 1) // 2
    total = window * (window + 1) // 2 + (n - window) * window
    # beyond the window, min(sinks, i + 1 - window) of the first tokens
    m = n - window
    few = min(m, sinks)
    return total + few * (few + 1) // 2 + (m - few) * sinks


def work(case):
    size, D = (2 if case["type"] == "bf16" else 4), case["head"]
    if case["op"] == "rotate":
        return {"bytes": 2 * case["rows"] * case["heads"] * D * size + 4 * case["rows"] + 8 * (case["dim"] // 2),
                "flops": 6 * case["rows"] * case["heads"] * (case["dim"] // 2)}
    length, rows = _counts(case)
    n, H, G = int(rows.sum()), case["q_heads"], case["kv_heads"]
    if case["op"] == "prompt":
        pairs = sum(_pairs(int(r), case["window"], case["sinks"]) for r in rows)
        return {"bytes": 2 * n * (H + G) * D * size + 4 * len(rows), "flops": 4 * pairs * H * D}
    pages = int((_ceil(length + rows, case["page"]) - length // case["page"]).sum())
    return {"bytes": n * (2 * H + (5 if case["keep"] else 4) * G) * D * size + 4 * pages + 12 * len(rows) + 8 * (case["dim"] // 2),
            "flops": 6 * n * (H + G) * (case["dim"] // 2)}


def exact(case, seed):
    """What run() returns, from the definitions in 64 bits."""
    s = prepare(case, seed)

    def turned(x, positions):
        # a pair is a complex number, multiplied by magnitude e^(i position frequency)
        f, m = _frequencies(case)
        y = x.double().clone()
        z = torch.polar(torch.full_like(positions, m, dtype=torch.float64)[:, None].expand(-1, len(f)).contiguous(),
                        torch.outer(positions.double(), torch.from_numpy(f).to(x.device)))
        for j in range(len(f)):
            a, b = (2 * j, 2 * j + 1) if case["interleaved"] else (j, j + len(f))
            w = torch.complex(y[:, :, a], y[:, :, b]) * z[:, j, None]
            y[:, :, a], y[:, :, b] = w.real, w.imag
        return y

    if case["op"] == "rotate":
        return {"out": turned(s["x"], s["positions"])}
    if case["op"] == "append":
        length, rows = _counts(case)
        at = torch.cat([torch.arange(int(a), int(a + n), device=s["q"].device) for a, n in zip(length, rows)])
        q, k = turned(s["q"], at), turned(s["k"], at)
        kp, vp, r = s["k_pages"].double(), s["v_pages"].double(), 0
        for b in range(len(rows)):
            p, end = int(length[b]), int(length[b] + rows[b])
            while p < end:   # page by page
                n = min(end, (p // s["page"] + 1) * s["page"]) - p
                page, o = int(s["table"][b, p // s["page"]]), p % s["page"]
                kp[page, :, o:o + n] = k[r:r + n].transpose(0, 1)
                vp[page, :, o:o + n] = s["v"][r:r + n].double().transpose(0, 1)
                p, r = p + n, r + n
        out = {"q": q, "k_pages": kp, "v_pages": vp, "status": None}
        if case["keep"]:
            out["k"] = k
        return out
    if work(case)["flops"] > 6e12:   # at about a TFLOP/s
        return None
    q, k, v = s["q"], s["k"], s["v"]
    G = case["q_heads"] // case["kv_heads"]
    out = torch.empty(q.shape, dtype=torch.float64, device=q.device)
    at = 0
    for n in s["rows"]:
        for h in range(case["q_heads"]):
            kk, vv = k[at:at + n, h // G].double(), v[at:at + n, h // G].double()
            for i0 in range(0, n, 2048):
                i1 = min(n, i0 + 2048)
                low = max(0, i0 + 1 - case["window"]) if case["window"] else 0
                first = min(case["sinks"], low)
                j = torch.cat([torch.arange(first, device=q.device), torch.arange(low, i1, device=q.device)])
                i = torch.arange(i0, i1, device=q.device)[:, None]
                hidden = j > i
                if case["window"]:
                    hidden |= (j <= i - case["window"]) & (j >= case["sinks"])
                x = (q[at + i0:at + i1, h].double() @ kk[j].T) * s["scale"]
                out[at + i0:at + i1, h] = torch.softmax(x.masked_fill(hidden, -math.inf), dim=1) @ vv[j]
        at += n
    return {"out": out, "status": None}
