"""A decode loop over the paged key-value cache, with every call of the library that one step takes.

    python -m speculative_decoding_block_verify_gb300.decode_example [--streams 8] [--steps 32]

One prompt is prefilled into stream 0 and forked to the other streams (their pages are shared until they are
written into).  Each step then
  1. drafts N tokens per stream (dspark_markov_walk: a low-rank previous-token drafter),
  2. runs the target over the block of N + 1 tokens: per layer the new keys and values go into the pages
     (spec_cache_append) and the block attends over the whole context (spec_paged_attention),
  3. verifies the block (spec_verify_block), and
  4. keeps the emitted tokens' pages and reserves room for the next block (spec_cache_resize).
With ``--rotary`` the target has rotary positions instead of learned ones: every step's append turns keys and queries on the way
(spec_cache_append_rotated), and the prompt goes through in one piece (the same call, and spec_prompt_attention over its packed rows).
Nothing is read back to the host inside a step: what a call reports for a stream goes into the next one on the device.  A
stream that finds no page in step 4 is passed over by the next step's append, keeps nothing of that step and asks again.  The target is a small random transformer whose projections
are plain torch products: it stands for a user's model.
"""

import argparse

import speculative_decoding_block_verify_gb300 as sv


class Target:
    """A random decoder: embeddings, ``layers`` blocks of attention with a residual, and logits of a head plus a
    low-rank table of the token before (the part that the drafter knows, and most of them)."""

    def __init__(self, torch, V=512, width=256, layers=2, q_heads=8, kv_heads=2, head=64, positions=4096, seed=0,
                 dtype=None, device="cuda", rotary=False):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.dtype = torch.float32 if dtype is None else dtype
        r = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
        self.rotary = sv.RotaryTable(head, device=device) if rotary else None
        self.V, self.layers, self.q_heads, self.kv_heads, self.head = V, layers, q_heads, kv_heads, head
        self.embedding = r(V, width).to(self.dtype)
        self.position = (0.3 * r(positions, width)).to(self.dtype)
        out = (q_heads + 2 * kv_heads) * head
        self.qkv = [(r(width, out) * width ** -0.5).to(self.dtype) for _ in range(layers)]
        self.logits = (2 * r(width, V) * width ** -0.5).to(self.dtype)
        self.table = (1.2 * r(V, 16), 1.2 * r(16, V))
        self.o = [(r(q_heads * head, width) * (q_heads * head) ** -0.5).to(self.dtype) for _ in range(layers)]


class Cache:
    """Pages, table and counts of ``streams`` streams of up to ``tokens`` tokens."""

    def __init__(self, torch, target, streams, tokens, page=16, spare=0, device="cuda"):
        width = -(-tokens // page)
        pages = streams * width + spare
        shape = (target.layers, pages, target.kv_heads, page, target.head)
        self.page = page
        self.k = torch.zeros(shape, dtype=target.dtype, device=device)
        self.v = torch.zeros_like(self.k)
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=device)  # noqa: E731
        self.table, self.held, self.length, self.refs = i32(streams, width) - 1, i32(streams), i32(streams), i32(pages)
        self._resize = self._fork = None
        self.reserved = None   # the status of the resize that made the room for the next block

    def resize(self, advance=None, room=None):
        self._resize = sv.spec_cache_resize(self.k, self.v, self.table, self.held, self.length, self.refs, advance=advance,
                                            room=room, out=self._resize)
        self.reserved = self._resize["status"]
        return self.reserved

    def fork(self, src, dst):
        self._fork = sv.spec_cache_fork(src, dst, self.table, self.held, self.length, self.refs, self.page)
        return self._fork["status"]


def first_of(torch, *statuses):
    """Per stream, the first status that is not OK."""
    worst = statuses[0].clone()
    for s in statuses[1:]:
        worst = torch.where(worst == 0, s, worst)
    return worst


def forward(torch, target, cache, tokens, cu, kmax, state):
    """Logits [rows, V] of the packed block rows ``tokens``; their keys and values are appended.  ``state["status"]`` is
    what the block's calls report for each stream, that of the resize before them included."""
    if target.rotary is None and cache.table.shape[1] * cache.page > target.position.shape[0]:
        raise ValueError(f"the cache has room for {cache.table.shape[1] * cache.page} tokens a stream, the model for "
                         f"{target.position.shape[0]}")
    rows, H, G = tokens.numel(), target.q_heads, target.kv_heads
    x = target.embedding[tokens.long()]
    if target.rotary is None:
        stream = torch.searchsorted(cu + torch.arange(cu.numel(), device=cu.device), torch.arange(rows, device=cu.device), right=True) - 1
        at = cache.length[stream] + torch.arange(rows, device=cu.device) - cu[stream] - stream
        # a block that does not fit its stream's table row is refused by the calls below, and its rows stand for nothing
        x = x + target.position[at.clamp(max=target.position.shape[0] - 1)]

    def block(i, qkv):
        # slices of the projection go in as they lie
        q, k, v = qkv[:, :H], qkv[:, H:H + G], qkv[:, H + G:]
        pool = (cache.k[i], cache.v[i], cache.table, cache.length)
        turn = ("append", rows)
        if target.rotary is None:
            a = sv.spec_cache_append(k, v, *pool, cu, kmax, out=state.get(turn), reserved=cache.reserved)
        else:
            a = sv.spec_cache_append_rotated(q, k, v, *pool, target.rotary, cu_drafts=cu, kmax=kmax, out=state.get(turn), reserved=cache.reserved)
            q = a["q"]
        state[turn] = a
        key = ("attention", rows, kmax)
        state[key] = o = sv.spec_paged_attention(q, *pool, cu, kmax, target.head ** -0.5, out=state.get(key))
        return o["out"], a["status"], o["status"]

    return layers(torch, target, tokens, x, cache.reserved, block, state)


def layers(torch, target, tokens, x, status, attend, state):
    """Logits of the rows ``x``; ``attend(layer, projections)`` returns the layer's attention and what its calls report."""
    rows, H, G, D = tokens.numel(), target.q_heads, target.kv_heads, target.head
    for i in range(target.layers):
        out, *seen = attend(i, (x @ target.qkv[i]).view(rows, H + 2 * G, D))
        status = first_of(torch, status, *seen)
        x = x + out.view(rows, H * D) @ target.o[i]
        x = x * torch.rsqrt((x.float() ** 2).mean(dim=1, keepdim=True)).to(x.dtype)
    state["status"] = status
    W1, W2 = target.table
    return (x @ target.logits).float() + W1[tokens.long()] @ W2


def prefill_whole(torch, target, cache, tokens, counts, state):
    """Whole prompts into a cache that holds none of their streams yet: ``tokens`` [rows] packed, counts[b] of them for stream b (0 for
    one that takes no part).  Returns the logits [rows, V]; ``state["status"]`` [B] is what the calls report."""
    H, G, dev = target.q_heads, target.kv_heads, tokens.device
    counts = torch.as_tensor(counts, dtype=torch.int32, device=dev)
    cu = torch.zeros(counts.numel() + 1, dtype=torch.int32, device=dev)
    cu[1:] = torch.cumsum(counts, 0)
    reserved = cache.resize(room=counts)

    def whole(i, qkv):
        a = sv.spec_cache_append_rotated(qkv[:, :H], qkv[:, H:H + G], qkv[:, H + G:], cache.k[i], cache.v[i], cache.table, cache.length,
                                         target.rotary, cu_rows=cu, keep_keys=True, reserved=reserved)
        o = sv.spec_prompt_attention(a["q"], a["k"], qkv[:, H + G:], cu, target.head ** -0.5)
        return o["out"], a["status"], o["status"]

    logits = layers(torch, target, tokens, target.embedding[tokens.long()], reserved, whole, state)
    cache.resize(advance=torch.where(state["status"] == 0, counts, 0))
    return logits


def prefill(torch, target, cache, prompt, state, kmax=sv.MAX_DRAFTS):
    """The prompt but its last token into stream 0's pages, a block of kmax + 1 tokens at a time.  Returns the first
    status [1] that is not OK."""
    B, dev = cache.length.numel(), prompt.device
    n = prompt.numel() - 1
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    for at in range(0, n, kmax + 1):
        part = prompt[at:min(n, at + kmax + 1)]
        one = torch.zeros(B, dtype=torch.int32, device=dev)
        one[0] = part.numel()
        cache.resize(room=one)
        # the other streams have no tokens yet: the block belongs to stream 0 alone
        view = _OneStream(cache)
        cu = torch.tensor([0, part.numel() - 1], dtype=torch.int32, device=dev)
        mine = {}
        forward(torch, target, view, part, cu, kmax, mine)
        status = first_of(torch, status, mine["status"])
        one[0] = torch.where(status[0] == 0, one[0], 0)
        cache.resize(advance=one)
    return status


class _OneStream:
    """Stream 0 of a cache."""

    def __init__(self, cache):
        self.k, self.v, self.table, self.length, self.reserved = cache.k, cache.v, cache.table[:1], cache.length[:1], cache.reserved[:1]
        self.page = cache.page


def decode(torch, target, cache, anchor, steps, drafts, temperature, drafter, seed=0):
    """``steps`` verify steps from the tokens ``anchor`` [B].  Returns (tokens [B, steps * (drafts + 1)] with
    -1 past the emitted ones, emitted counts [steps, B], statuses [steps, B]): 0 tokens and the first status of the step's calls
    that is not OK where a stream could not take part."""
    dev, B, N = anchor.device, anchor.numel(), drafts
    # resize leaves a stream whose next block does not fit its row as it was, kept tokens and all: rows are long enough
    most = int(cache.length.max()) + (steps + 1) * (N + 1)
    if most > cache.table.shape[1] * cache.page:
        raise ValueError(f"{steps} steps may need {most} tokens a stream, the cache has room for {cache.table.shape[1] * cache.page}")
    W1, W2 = drafter
    cu = torch.arange(B + 1, dtype=torch.int32, device=dev) * N
    room = torch.full((B,), N + 1, dtype=torch.int32, device=dev)
    base = torch.zeros((B, N, target.V), dtype=torch.float32, device=dev)
    state, walk, out = {}, None, None
    tokens = torch.full((B, steps * (N + 1)), -1, dtype=torch.int32, device=dev)
    counts = torch.zeros((steps, B), dtype=torch.int32, device=dev)
    status = torch.zeros((steps, B), dtype=torch.int32, device=dev)
    ends = torch.zeros(B, dtype=torch.int64, device=dev)
    cache.resize(room=room)
    for step in range(steps):
        if N > 0:
            walk = sv.dspark_markov_walk(base, anchor, W1, W2, temperature, seed, step, out=walk)
            x, q = walk["tokens"].view(-1), walk["logits"].view(B * N, -1)
        else:
            x, q = torch.zeros(0, dtype=torch.int32, device=dev), base.view(0, target.V)
        block = torch.cat([anchor[:, None], x.view(B, N)], dim=1).view(-1)
        logits = forward(torch, target, cache, block, cu, N, state)
        out = sv.spec_verify_block(cu, q, logits, x, temperature, N, seed, step, out=out)
        status[step] = first_of(torch, state["status"], out["status"])
        kept = torch.where(status[step] == 0, out["n_emitted"], 0)
        cache.resize(advance=kept, room=room)
        n = kept.long()
        last = out["out_tokens"].gather(1, (n - 1).clamp(min=0)[:, None])[:, 0]
        anchor = torch.where(n > 0, last, anchor).contiguous()
        col = torch.arange(N + 1, device=dev)
        here = col < n[:, None]
        where = torch.where(here, ends[:, None] + col, tokens.shape[1] - 1)
        tokens.scatter_(1, where, torch.where(here, out["out_tokens"], tokens.gather(1, where)))
        ends += n
        counts[step] = kept
    return tokens, counts, status


def main():
    import torch

    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--streams", type=int, default=8)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--drafts", type=int, default=5)
    ap.add_argument("--prompt", type=int, default=100)
    ap.add_argument("--temperature", type=float, default=0.8)
    ap.add_argument("--rotary", action="store_true", help="rotary positions, and the prompt in one piece")
    a = ap.parse_args()
    tokens = a.prompt + (a.steps + 1) * (a.drafts + 1)
    target = Target(torch, positions=-(-tokens // 16) * 16, rotary=a.rotary)
    cache = Cache(torch, target, a.streams, tokens)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    prompt = torch.randint(0, target.V, (a.prompt,), generator=g, device="cuda", dtype=torch.int32)
    if a.rotary:
        state = {}
        prefill_whole(torch, target, cache, prompt[:-1], [a.prompt - 1] + [0] * (a.streams - 1), state)
        seen = [state["status"]]
    else:
        seen = [prefill(torch, target, cache, prompt, {})]
    if a.streams > 1:
        others = torch.arange(1, a.streams, dtype=torch.int32, device="cuda")
        seen.append(cache.fork(torch.zeros_like(others), others))
    temperature = torch.full((a.streams,), a.temperature, device="cuda")
    tokens, counts, status = decode(torch, target, cache, prompt[-1:].repeat(a.streams), a.steps, a.drafts, temperature, target.table)
    torch.cuda.synchronize()
    print(f"{a.streams} streams, {a.steps} steps of {a.drafts} drafts: {counts.float().mean().item():.2f} tokens a step, "
          f"statuses {sorted(set(torch.cat(seen + [status.view(-1)]).tolist()))}, pages held {int(cache.held.sum())} of {cache.refs.numel()}")
    for b in range(min(3, a.streams)):
        print(" ", tokens[b, :16].tolist())


if __name__ == "__main__":
    main()
