"""Timed cases of the prompt, draft-tree and cache-writing operators.

Each case is one call (or the plain torch form of it) over a paged KV cache:

  prefill : causal attention of packed prompt chunks over the cache that holds
            their tokens, grouped heads (pkv.attn_prefill)
  tree    : attention of drafted token trees over the cached context and the
            drafts' own keys and values (pkv.attn_tree)
  write   : per-head norms of queries and keys, rotary positions and the
            append of keys and values to their slots (pkv.qk_norm_rope_append)

With `own` false, run() computes the operators in elementary torch operations
in 32 bits, rounded once at the end; with `own` true it makes the library's
calls. exact() is the definition in 64 bits, written apart from both.
"""
import math
import random

import torch

own = False

HEAD_DIM = 128
NORM_EPS = 1e-6
# Scores held at once by the plain form, in elements (1 GB in 32 bits).
PLAIN_SCORES = 1 << 28
EXACT_SCORES = 1 << 27

HEADS = [(32, 8), (64, 8), (16, 8), (8, 8), (8, 1)]


# ---------------------------------------------------------------------------
# cases


def _attend_case(kind, name, seqs, new_median, new_sigma, new_max, cached_median, cached_sigma, cached_max,
                 q_heads, kv_heads, block_tokens, shape_seed):
    case = {"kind": kind, "seqs": seqs, "new_median": new_median, "new_sigma": new_sigma, "new_max": new_max,
            "cached_median": cached_median, "cached_sigma": cached_sigma, "cached_max": cached_max,
            "q_heads": q_heads, "kv_heads": kv_heads, "block_tokens": block_tokens, "shape_seed": shape_seed}
    if name:
        case["name"] = name
    return case


def _write_case(name, tokens, padding, q_heads, kv_heads, head_dim, rotary_dim, norm, interleaved, block_tokens,
                max_position):
    case = {"kind": "write", "tokens": tokens, "padding": padding, "q_heads": q_heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "rotary_dim": rotary_dim, "norm": norm, "interleaved": interleaved,
            "block_tokens": block_tokens, "max_position": max_position}
    if name:
        case["name"] = name
    return case


def listed():
    return [
        # one short prompt on an idle server: what a user waits for is latency
        _attend_case("prefill", "prefill_one_prompt", 1, 37, 0.0, 37, 0, 0.0, 0, 32, 8, 16, 1),
        # a packed batch of chat prompts of different lengths, nothing cached
        _attend_case("prefill", "prefill_packed", 16, 512, 0.8, 2048, 0, 0.0, 0, 32, 8, 16, 2),
        # chunked prefill: about a thousand new tokens each on long cached contexts
        _attend_case("prefill", "prefill_chunks", 5, 1000, 0.2, 2048, 9000, 0.7, 65536, 64, 8, 16, 3),
        # one long document
        _attend_case("prefill", "prefill_long", 1, 16411, 0.0, 16411, 0, 0.0, 0, 64, 8, 16, 4),
        # one query head per KV head, larger blocks, ragged: decode rows ride along with prompts
        _attend_case("prefill", "prefill_ragged_mha", 24, 40, 2.0, 4001, 300, 1.5, 5003, 8, 8, 32, 5),
        # one user's speculative step
        _attend_case("tree", "tree_one", 1, 8, 0.0, 8, 417, 0.0, 417, 32, 8, 16, 6),
        # a serving batch, each sequence with a tree of about sixteen drafts
        _attend_case("tree", "tree_batch", 64, 16, 0.3, 32, 1024, 1.0, 8192, 32, 8, 16, 7),
        # long contexts, wide trees up to the largest
        _attend_case("tree", "tree_long", 24, 24, 0.8, 64, 16000, 0.8, 131072, 64, 8, 16, 8),
        # one KV head, many sequences, small blocks
        _attend_case("tree", "tree_mqa", 200, 5, 0.8, 24, 700, 0.8, 5000, 8, 1, 8, 9),
        # one decode step's tokens, padded to a batch bucket
        _write_case("write_decode", 64, 3, 32, 8, 128, 128, True, False, 16, 131072),
        # a prefill step's tokens
        _write_case("write_prompt", 16411, 0, 64, 8, 128, 128, True, False, 16, 131072),
        # interleaved pairs on a part of a smaller head, no norms
        _write_case("write_partial", 5003, 0, 8, 8, 64, 32, False, True, 64, 8192),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    kind = rng.choice(["prefill", "prefill", "tree", "tree", "write"])
    if kind == "write":
        head_dim = rng.choice([64, 128, 128, 256])
        rotary = rng.choice([head_dim, head_dim, head_dim // 2, head_dim // 4])
        q_heads, kv_heads = rng.choice(HEADS)
        return _write_case(None, _log_int(rng, 1, 16411 * 128 // head_dim // 2), rng.choice([0, 0, 1, 5]), q_heads,
                           kv_heads, head_dim, rotary, rng.random() < 0.7, rng.random() < 0.3,
                           rng.choice([8, 16, 16, 32, 64]), _log_int(rng, 2048, 131072))
    # no more operations than the largest listed case of its kind, no more bytes than the largest listed case
    works = [(c["kind"], work(c)) for c in listed()]
    most_flops = max(w["flops"] for k, w in works if k == kind)
    most_bytes = max(w["bytes"] for _, w in works)
    while True:
        q_heads, kv_heads = rng.choice(HEADS)
        block_tokens = rng.choice([8, 16, 16, 16, 32, 64])
        shape_seed = rng.randrange(1 << 30)
        if kind == "prefill":
            new = _log_int(rng, 1, 16411)
            cached = rng.choice([0, 0, _log_int(rng, 1, 65536)])
            case = _attend_case("prefill", None, _log_int(rng, 1, 64), new, rng.uniform(0.0, 1.5), 16411, cached,
                                rng.uniform(0.0, 1.0), 65536, q_heads, kv_heads, block_tokens, shape_seed)
        else:
            case = _attend_case("tree", None, _log_int(rng, 1, 256), _log_int(rng, 1, 64), rng.uniform(0.0, 1.0), 64,
                                _log_int(rng, 1, 65536), rng.uniform(0.0, 1.2), 131072, q_heads, kv_heads,
                                block_tokens, shape_seed)
        w = work(case)
        if w["flops"] <= most_flops and w["bytes"] <= most_bytes:
            return case


def _lengths(case):
    """(new tokens, cached tokens) of each sequence."""
    r = random.Random(case["shape_seed"])

    def one(median, sigma, top, low):
        if median <= 0:
            return 0
        return int(min(top, max(low, round(median * math.exp(sigma * r.gauss(0.0, 1.0))))))

    new = [one(case["new_median"], case["new_sigma"], case["new_max"], 1) for _ in range(case["seqs"])]
    cached = [one(case["cached_median"], case["cached_sigma"], case["cached_max"], 0) for _ in range(case["seqs"])]
    return new, cached


def _trees(case, new):
    """One list of parents a sequence: a draft's parent is an earlier draft, or -1."""
    r = random.Random(case["shape_seed"] + 1)
    return [[-1 if j == 0 else r.randrange(-1, j) for j in range(n)] for n in new]


def _tree_masks(parents):
    """Bit j of row i: draft i sees draft j (its ancestors and itself)."""
    rows = []
    for i, p in enumerate(parents):
        rows.append((rows[p] if p >= 0 else 0) | (1 << i))
    return rows


def work(case):
    """Bytes and operations of one pass: inputs read once, outputs written once."""
    hq, hkv = case["q_heads"], case["kv_heads"]
    if case["kind"] == "write":
        t, d = case["tokens"], case["head_dim"]
        rows = t * (hq + 2 * hkv) * d * 2
        return {"bytes": 2 * rows + t * (case["rotary_dim"] * 4 + 4 + 8) + (4 * d if case["norm"] else 0),
                "flops": t * (hq + hkv) * d * (6 if case["norm"] else 3)}
    new, cached = _lengths(case)
    entries = tokens = pairs = 0
    if case["kind"] == "prefill":
        for n, c in zip(new, cached):
            tokens += n + c
            pairs += n * c + n * (n + 1) // 2
            entries += -(-(n + c) // case["block_tokens"])
        extra = 0
    else:
        for n, c, parents in zip(new, cached, _trees(case, new)):
            tokens += c + n
            pairs += n * c + sum(bin(m).count("1") for m in _tree_masks(parents))
            entries += -(-c // case["block_tokens"])
        extra = 8 * sum(new)
    nbytes = tokens * hkv * HEAD_DIM * 4 + 2 * sum(new) * hq * HEAD_DIM * 2 + 4 * entries + 8 * case["seqs"] + 4 + extra
    return {"bytes": nbytes, "flops": 4 * HEAD_DIM * hq * pairs}


# ---------------------------------------------------------------------------
# inputs


def _randn(gen, shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _pool(gen, blocks, hkv, block_tokens, dim):
    pool = torch.empty((blocks, hkv, block_tokens, dim), device="cuda", dtype=torch.bfloat16)
    step = max(1, (1 << 26) // (hkv * block_tokens * dim))
    for lo in range(0, blocks, step):
        hi = min(blocks, lo + step)
        pool[lo:hi] = _randn(gen, (hi - lo, hkv, block_tokens, dim))
    return pool


def _rope_table(max_positions, rotary_dim):
    """cos and sin of every position's angles, [positions, rotary_dim] in 32 bits."""
    half = rotary_dim // 2
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") * 2.0 / rotary_dim)
    angle = torch.arange(max_positions, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], dim=1).float().contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    r = random.Random(seed)
    hq, hkv, bt = case["q_heads"], case["kv_heads"], case["block_tokens"]
    state = {"case": case}
    if case["kind"] == "write":
        t, d = case["tokens"], case["head_dim"]
        blocks = -(-t // bt) + 2
        # the fused projection's output: q, k and v are views of it
        fused = _randn(gen, (t, (hq + 2 * hkv) * d))
        state["q"] = fused[:, : hq * d].view(t, hq, d)
        state["k"] = fused[:, hq * d : (hq + hkv) * d].view(t, hkv, d)
        state["v"] = fused[:, (hq + hkv) * d :].view(t, hkv, d)
        state["q_weight"] = state["k_weight"] = None
        if case["norm"]:
            state["q_weight"] = (1.0 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(torch.bfloat16)
            state["k_weight"] = (1.0 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(torch.bfloat16)
        state["cos_sin"] = _rope_table(case["max_position"], case["rotary_dim"])
        state["positions"] = torch.randint(0, case["max_position"], (t,), generator=gen, device="cuda",
                                           dtype=torch.int32)
        order = torch.randperm(blocks, generator=gen, device="cuda")
        pos = torch.arange(t, device="cuda")
        slots = order[pos // bt] * bt + pos % bt
        padding = min(case["padding"], t - 1)
        if padding:
            slots[t - padding :] = -1
        state["slots"] = slots.contiguous()
        state["k_cache"] = torch.zeros((blocks, hkv, bt, d), device="cuda", dtype=torch.bfloat16)
        state["v_cache"] = torch.zeros_like(state["k_cache"])
        if own:
            import paged_kv_cache_49_gb300 as pkv
            state["errors"] = pkv.new_error_word()
            state["q_out"] = torch.empty((t, hq, d), device="cuda", dtype=torch.bfloat16)
        return state

    new, cached = _lengths(case)
    in_cache = [n + c for n, c in zip(new, cached)] if case["kind"] == "prefill" else cached
    per_seq = [-(-n // bt) for n in in_cache]
    blocks = sum(per_seq) + sum(per_seq) // 10 + 1
    order = list(range(blocks))
    r.shuffle(order)
    width = max(1, max(per_seq))
    rows, at = [], 0
    for n in per_seq:
        rows.append(order[at : at + n] + [-1] * (width - n))
        at += n
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    state["new"], state["in_cache"], state["starts"], state["rows"] = new, in_cache, starts, rows
    state["tables"] = torch.tensor(rows, dtype=torch.int32, device="cuda")
    state["context_lens"] = torch.tensor(in_cache, dtype=torch.int32, device="cuda")
    state["query_starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    state["scale"] = 1.0 / math.sqrt(HEAD_DIM)
    state["k_cache"] = _pool(gen, blocks, hkv, bt, HEAD_DIM)
    state["v_cache"] = _pool(gen, blocks, hkv, bt, HEAD_DIM)
    state["q"] = _randn(gen, (starts[-1], hq, HEAD_DIM))
    if case["kind"] == "tree":
        state["k_draft"] = _randn(gen, (starts[-1], hkv, HEAD_DIM))
        state["v_draft"] = _randn(gen, (starts[-1], hkv, HEAD_DIM))
        masks = [m for parents in _trees(case, new) for m in _tree_masks(parents)]
        state["masks"] = torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks], dtype=torch.int64,
                                      device="cuda")
    if own:
        import paged_kv_cache_49_gb300 as pkv
        state["workspace"] = pkv.PrefillWorkspace()
        state["out"] = torch.empty_like(state["q"])
    return state


# ---------------------------------------------------------------------------
# one pass


def run(state):
    kind = state["case"]["kind"]
    if own:
        import paged_kv_cache_49_gb300 as pkv
        if kind == "prefill":
            return pkv.attn_prefill(state["q"], state["k_cache"], state["v_cache"], state["tables"],
                                    state["context_lens"], state["query_starts"], state["scale"], out=state["out"],
                                    workspace=state["workspace"])
        if kind == "tree":
            return pkv.attn_tree(state["q"], state["k_draft"], state["v_draft"], state["masks"], state["k_cache"],
                                 state["v_cache"], state["tables"], state["context_lens"], state["query_starts"],
                                 state["scale"], out=state["out"], workspace=state["workspace"])
        q_out = pkv.qk_norm_rope_append(state["q"], state["k"], state["v"], state["cos_sin"], state["positions"],
                                        state["slots"], state["k_cache"], state["v_cache"],
                                        q_weight=state["q_weight"], k_weight=state["k_weight"], eps=NORM_EPS,
                                        interleaved=state["case"]["interleaved"], q_out=state["q_out"],
                                        device_error=state["errors"])
        return q_out, state["k_cache"], state["v_cache"]
    if kind == "write":
        return _plain_write(state)
    return _plain_attention(state)


def _gather(cache, row, tokens):
    """[Hkv, tokens, D] in 32 bits, read through one sequence's table row."""
    bt = cache.shape[2]
    blocks = cache[row[: -(-tokens // bt)].long()]
    return blocks.permute(1, 0, 2, 3).reshape(cache.shape[1], -1, cache.shape[3])[:, :tokens].float()


def _plain_attention(state):
    case = state["case"]
    tree = case["kind"] == "tree"
    hq, hkv = case["q_heads"], case["kv_heads"]
    group = hq // hkv
    out = torch.empty_like(state["q"])
    for s, (n, held) in enumerate(zip(state["new"], state["in_cache"])):
        lo = state["starts"][s]
        keys = _gather(state["k_cache"], state["tables"][s], held)
        values = _gather(state["v_cache"], state["tables"][s], held)
        if tree:
            keys = torch.cat([keys, state["k_draft"][lo : lo + n].float().transpose(0, 1)], dim=1)
            values = torch.cat([values, state["v_draft"][lo : lo + n].float().transpose(0, 1)], dim=1)
        total = keys.shape[1]
        at = torch.arange(total, device="cuda")
        step = max(1, min(n, PLAIN_SCORES // (hq * total)))
        for first in range(0, n, step):
            m = min(step, n - first)
            q = state["q"][lo + first : lo + first + m].float()
            q = q.view(m, hkv, group, HEAD_DIM).permute(1, 2, 0, 3).reshape(hkv, group * m, HEAD_DIM)
            scores = torch.matmul(q, keys.transpose(1, 2)) * state["scale"]
            if tree:
                bits = state["masks"][lo + first : lo + first + m]
                among = (bits[:, None] >> torch.arange(n, device="cuda")) & 1
                seen = torch.cat([torch.ones((m, held), dtype=torch.bool, device="cuda"), among == 1], dim=1)
            else:
                position = held - n + first + torch.arange(m, device="cuda")
                seen = at[None, :] <= position[:, None]
            scores = scores.view(hkv, group, m, total).masked_fill(~seen, float("-inf"))
            weights = torch.exp(scores - scores.amax(dim=-1, keepdim=True))
            total_weight = weights.sum(dim=-1, keepdim=True)
            o = torch.matmul(weights.view(hkv, group * m, total), values).view(hkv, group, m, HEAD_DIM) / total_weight
            out[lo + first : lo + first + m] = o.permute(2, 0, 1, 3).reshape(m, hq, HEAD_DIM).to(out.dtype)
    return out


def _plain_write(state):
    case = state["case"]
    rot = case["rotary_dim"]
    half = rot // 2
    angles = state["cos_sin"][state["positions"].long()][:, None, :]
    cos, sin = angles[..., :half], angles[..., half:]

    def turn(x, weight):
        y = x.float()
        if weight is not None:
            y = y / torch.sqrt((y * y).mean(dim=-1, keepdim=True) + NORM_EPS) * weight.float()
        part = y[..., :rot]
        if case["interleaved"]:
            a, b = part[..., 0::2], part[..., 1::2]
            turned = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
        else:
            a, b = part[..., :half], part[..., half:]
            turned = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
        return torch.cat([turned, y[..., rot:]], dim=-1).to(torch.bfloat16)

    q_out = turn(state["q"], state["q_weight"])
    k = turn(state["k"], state["k_weight"])
    bt = case["block_tokens"]
    kept = state["case"]["tokens"] - min(case["padding"], state["case"]["tokens"] - 1)
    slots = state["slots"][:kept]
    state["k_cache"][slots // bt, :, slots % bt] = k[:kept]
    state["v_cache"][slots // bt, :, slots % bt] = state["v"][:kept]
    return q_out, state["k_cache"], state["v_cache"]


# ---------------------------------------------------------------------------
# the definition in 64 bits


def exact(case, seed):
    state = prepare(case, seed)
    if case["kind"] == "write":
        return _exact_write(case, state)
    group = case["q_heads"] // case["kv_heads"]
    bt = case["block_tokens"]
    result = torch.zeros(state["q"].shape, dtype=torch.float64, device="cuda")
    for s in range(case["seqs"]):
        held, n, lo = state["in_cache"][s], state["new"][s], state["starts"][s]
        token = torch.arange(held, device="cuda")
        physical = torch.tensor(state["rows"][s], device="cuda")[token // bt] if held else token
        if case["kind"] == "tree":
            words = state["masks"][lo : lo + n].tolist()
            sight = torch.ones(n, held + n, dtype=torch.bool)
            sight[:, held:] = torch.tensor([[bool(w >> j & 1) for j in range(n)] for w in words])
            sight = sight.cuda()
        for g in range(case["kv_heads"]):
            key = state["k_cache"][physical, g, token % bt].double()
            value = state["v_cache"][physical, g, token % bt].double()
            if case["kind"] == "tree":
                key = torch.vstack([key, state["k_draft"][lo : lo + n, g].double()])
                value = torch.vstack([value, state["v_draft"][lo : lo + n, g].double()])
            for first in range(0, n, max(1, EXACT_SCORES // key.shape[0])):
                last = min(n, first + max(1, EXACT_SCORES // key.shape[0]))
                # a prompt row sees nothing behind the chunk's last row
                reach = key.shape[0] if case["kind"] == "tree" else held - n + last
                for h in range(g * group, (g + 1) * group):
                    x = state["q"][lo + first : lo + last, h].double() @ key[:reach].T * state["scale"]
                    if case["kind"] == "tree":
                        x[~sight[first:last]] = -math.inf
                    else:
                        x += torch.full_like(x, -math.inf).triu(held - n + first + 1)
                    result[lo + first : lo + last, h] = torch.softmax(x, dim=1) @ value[:reach]
    return result


def _exact_write(case, state):
    rot, d = case["rotary_dim"], case["head_dim"]
    half = rot // 2
    table = state["cos_sin"].double()[state["positions"].long()]

    def rotated(x, weight):
        y = x.double()
        if weight is not None:
            y = y * torch.rsqrt(y.square().sum(-1, keepdim=True) / d + NORM_EPS) * weight.double()
        result = y.clone()
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
            c, s = table[:, i, None], table[:, half + i, None]
            result[..., a] = y[..., a] * c - y[..., b] * s
            result[..., b] = y[..., b] * c + y[..., a] * s
        return result

    keys = torch.zeros(state["k_cache"].shape, dtype=torch.float64, device="cuda")
    values = torch.zeros_like(keys)
    written = state["slots"] >= 0
    slots = state["slots"][written]
    bt = case["block_tokens"]
    keys[slots // bt, :, slots % bt] = rotated(state["k"], state["k_weight"])[written]
    values[slots // bt, :, slots % bt] = state["v"].double()[written]
    return rotated(state["q"], state["q_weight"]), keys, values
