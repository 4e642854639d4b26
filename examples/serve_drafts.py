"""Disaggregated serving on one GPU: a prompt's cache is weighed, evicted,
compressed and sent; the receiver decodes drafted trees of tokens over it.

    python examples/serve_drafts.py

One layer, random projections. The sender appends a prompt to a paged cache
chunk by chunk (rotary positions applied), lets the prompt's last tokens weigh
it, keeps an eighth of it packed, and encodes that with the lossless codec. The
receiver decodes the stream and runs steps of a drafted tree: append, attend,
accept a path, add its weights. Because the codec is lossless, the receiver's
outputs are bit for bit those of the same steps on the sender's packed copy;
the script checks that."""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import lossless_bf16_exponent_gb300 as uz  # noqa: E402

B, Q_HEADS, KV_HEADS, DIM, PAGE = 2, 32, 8, 128, 64
PROMPT, CHUNK, WINDOW, KEEP, STEPS = 2048, 512, 32, 256, 3
PARENTS = [-1, 0, 0, 1, 1, 2, 3, 3]  # a drafted tree: node t continues node PARENTS[t]


def project(g: torch.Generator, tokens: int):
    """Queries, keys and values of new tokens, side by side as a fused projection gives them."""
    x = torch.randn((B, tokens, Q_HEADS + 2 * KV_HEADS, DIM), generator=g, device="cuda").bfloat16()
    return x[:, :, :Q_HEADS], x[:, :, Q_HEADS:Q_HEADS + KV_HEADS], x[:, :, Q_HEADS + KV_HEADS:]


def span(first: torch.Tensor, tokens: int) -> torch.Tensor:
    return (first[:, None] + torch.arange(tokens, device="cuda")).to(torch.int32)


def prefill(g: torch.Generator, plan: uz.RotaryPlan):
    """The prompt's cache, and the attention weight its last tokens give each token."""
    per = PROMPT // PAGE
    pool = torch.empty((B * per, 2, KV_HEADS, PAGE, DIM), dtype=torch.bfloat16, device="cuda")
    table = torch.randperm(B * per, generator=g, device="cuda").view(B, per).to(torch.int32)
    cache = uz.KVCache(pool[:, 0], pool[:, 1], table, torch.zeros(B, dtype=torch.int32, device="cuda"))
    for _ in range(PROMPT // CHUNK):
        q, k, v = project(g, CHUNK)
        q = uz.rotary_append(q, k, v, span(cache.lengths, CHUNK), plan, cache)
        cache.lengths += CHUNK
    window = q[:, -WINDOW:].contiguous()  # the chunk's last queries see the cache before them and, as a chain, themselves
    cache.lengths -= WINDOW
    _, lse = uz.tree_attention(window, cache)
    mass = uz.attention_mass(window, cache, lse)
    cache.lengths += WINDOW
    return cache, mass


def receive(packed: torch.Tensor, lengths: torch.Tensor):
    """A cache of whole-sequence pages around [K/V, sequences, heads, keep, dim], with room for new tokens."""
    room = torch.zeros((2, B, KV_HEADS, KEEP + 64, DIM), dtype=torch.bfloat16, device="cuda")
    room[:, :, :, :KEEP] = packed
    return uz.KVCache(room[0], room[1], torch.arange(B, dtype=torch.int32, device="cuda")[:, None], lengths.clone())


def decode_steps(cache: uz.KVCache, mass: torch.Tensor, plan: uz.RotaryPlan, seed: int):
    """Steps of a drafted tree; returns their outputs and the masses after them."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    mask = uz.tree_mask([PARENTS], device="cuda")
    depth = [0] * len(PARENTS)
    for t, u in enumerate(PARENTS):
        depth[t] = depth[u] + 1 if u >= 0 else 0
    deep = torch.tensor(depth, dtype=torch.int32, device="cuda")
    path = [len(PARENTS) - 1]  # the accepted path: the deepest node and its ancestors
    while PARENTS[path[0]] >= 0:
        path.insert(0, PARENTS[path[0]])
    weights = torch.zeros((B, len(PARENTS)), device="cuda")
    weights[:, path] = 1.0
    wide = torch.zeros((B, KV_HEADS, cache.capacity), device="cuda")
    wide[:, :, :KEEP] = mass
    position = torch.full((B,), PROMPT, device="cuda")
    outs = []
    for _ in range(STEPS):
        q, k, v = project(g, len(PARENTS))
        where = (position[:, None] + deep).to(torch.int32)
        rotated = uz.rotary_append(q, k, v, where, plan, cache)
        out, lse = uz.tree_attention(rotated, cache, mask)
        weighed = uz.attention_mass(rotated, cache, lse, mask, weights=weights, mass=wide, decay=0.99)
        outs.append(out)
        # The accepted tokens' rows move to the front of the new ones: append them again, as a chain.
        uz.rotary_append(q[:, path], k[:, path], v[:, path], where[:, path].contiguous(), plan, cache)
        at = cache.lengths.long()[:, None, None]
        rows = torch.arange(len(path), device="cuda")[None, None] + at
        taken = weighed.gather(2, (at + torch.tensor(path, device="cuda")).expand(B, KV_HEADS, -1))
        wide = torch.where(torch.arange(cache.capacity, device="cuda") < at, weighed, 0.0)
        wide.scatter_(2, rows.expand(B, KV_HEADS, -1), taken)
        cache.lengths += len(path)
        position += len(path)
    return outs, wide


def main() -> dict:
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    plan = uz.rotary_plan(DIM, base=1e6, layout="half", scaling="ramp", factor=4.0, original_length=32768)
    cache, mass = prefill(g, plan)
    both = torch.empty((2, B, KV_HEADS, KEEP, DIM), dtype=torch.bfloat16, device="cuda")
    packed = uz.evict(cache, mass, KEEP, sink=4, recent=64, out_k=both[0], out_v=both[1])

    codebook = uz.calibrate(both)
    stream, nbytes = uz.encode(both, codebook)
    sent = torch.zeros_like(stream)
    uz.stream_copy(stream, sent)  # the link
    got = uz.decode(sent, both.numel(), stream_bytes=nbytes).view(both.shape)

    mine, masses = decode_steps(receive(both, packed.lengths), packed.mass, plan, 11)
    theirs, their_masses = decode_steps(receive(got, packed.lengths), packed.mass, plan, 11)
    same = all(torch.equal(a, b) for a, b in zip(mine, theirs)) and torch.equal(masses, their_masses)
    raw = 2 * 2 * B * KV_HEADS * PROMPT * DIM
    return {"bit_identical": same, "finite": all(bool(torch.isfinite(o).all()) for o in theirs),
            "prompt_bytes": raw, "kept_bytes": 2 * both.numel(), "sent_bytes": nbytes,
            "mass_kept": float(packed.mass.sum() / mass.sum())}


if __name__ == "__main__":
    result = main()
    print(", ".join(f"{k} {v}" for k, v in result.items()))
    sys.exit(0 if result["bit_identical"] and result["finite"] else 1)
