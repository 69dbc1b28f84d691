"""Timed cases of the 4-bit cache's operators and of beam selection.

Each case is one pass (or the plain torch form of it):

  write  : new tokens' keys and values into a cache held in 4 bits, and the
           touched pages read back as the values they stand for
           (pkv.append_int4, pkv.load_int4)
  load   : pages of cached contexts as bf16 pages, for the attention of a
           prompt's next chunk (pkv.load_int4)
  decode : decode attention over a paged 4-bit cache (pkv.attn_decode_int4)
  beams  : the best continuations of groups of beams over the vocabulary, and
           their token histories (pkv.beam_select)

A row of 128 values is held as groups of `group_dims` values with a scale s and
a minimum m in fp16 and a code c of 4 bits each: s = fp16((max - min) / 15),
m = fp16(min), c = rint((x - m) / s) in 0 .. 15, the value s c + m.

With `own` false, run() computes the operators in elementary torch operations
in 32 bits (beam scores in 64), rounded once at the end; with `own` true it
makes the library's calls. exact() is the definition in 64 bits, written apart
from both.
"""
import math
import random

import torch

own = False

HEAD_DIM = 128
FP16_MAX = 65504.0
HEADS = [(32, 8), (64, 8), (16, 8), (8, 8), (8, 1)]
# Elements made, quantised or read at once (fp32 copies of 1 GB).
CHUNK = 1 << 28


# ---------------------------------------------------------------------------
# cases


def _write_case(name, tokens, padding, kv_heads, block_tokens, group_dims):
    case = {"kind": "write", "tokens": tokens, "padding": padding, "kv_heads": kv_heads, "block_tokens": block_tokens,
            "group_dims": group_dims}
    return {"name": name, **case} if name else case


def _context_case(kind, name, seqs, median, sigma, top, longest, q_heads, kv_heads, block_tokens, group_dims, shape_seed):
    """`longest` of the sequences have `top` tokens, the others are lognormal."""
    case = {"kind": kind, "seqs": seqs, "median": median, "sigma": sigma, "top": top, "longest": longest,
            "q_heads": q_heads, "kv_heads": kv_heads, "block_tokens": block_tokens, "group_dims": group_dims,
            "shape_seed": shape_seed}
    return {"name": name, **case} if name else case


def _beam_case(name, groups, beams, candidates, vocab, dtype, finished, first, history):
    case = {"kind": "beams", "groups": groups, "beams": beams, "candidates": candidates, "vocab": vocab, "dtype": dtype,
            "finished": finished, "first": first, "history": history}
    return {"name": name, **case} if name else case


def listed():
    return [
        # one decode step's tokens, padded to a batch bucket
        _write_case("write_decode", 64, 3, 8, 16, 64),
        # a prefill step's tokens
        _write_case("write_prompt", 16411, 0, 8, 16, 64),
        # small groups, large blocks, an odd number of tokens
        _write_case("write_groups", 5003, 5, 16, 64, 32),
        # the pages of one short conversation
        _context_case("load", "load_one", 1, 417, 0.0, 417, 0, 8, 8, 16, 64, 1),
        # the cached contexts of a batch of prompt chunks
        _context_case("load", "load_chunks", 5, 9000, 0.7, 65536, 0, 64, 8, 16, 64, 2),
        # one user's decode step: what counts is latency
        _context_case("decode", "decode_one", 1, 417, 0.0, 417, 0, 32, 8, 16, 64, 3),
        # a serving batch
        _context_case("decode", "decode_batch", 64, 1024, 1.0, 8192, 0, 32, 8, 16, 64, 4),
        # a large batch, some of its contexts very long
        _context_case("decode", "decode_long", 256, 4096, 1.2, 131072, 4, 64, 8, 16, 64, 5),
        # one KV head, many sequences, small blocks, one group a row
        _context_case("decode", "decode_mqa", 200, 700, 0.8, 5000, 0, 8, 1, 8, 128, 6),
        # one request's beams
        _beam_case("beams_one", 1, 4, 8, 32000, "bf16", 0.0, False, 97),
        # a batch of requests, some beams finished
        _beam_case("beams_batch", 64, 4, 8, 131072, "bf16", 0.1, False, 512),
        # many beams, logits in 32 bits, an odd vocabulary
        _beam_case("beams_wide", 12, 16, 32, 100003, "fp32", 0.05, False, 1000),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    works = [(c["kind"], work(c)) for c in listed()]
    while True:
        kind = rng.choice(["write", "load", "decode", "decode", "beams"])
        _, kv_heads = heads = rng.choice(HEADS)
        block_tokens, group_dims = rng.choice([8, 16, 16, 32, 64]), rng.choice([32, 64, 64, 128])
        if kind == "write":
            case = _write_case(None, _log_int(rng, 1, 16411), rng.choice([0, 0, 1, 5]), kv_heads, block_tokens, group_dims)
        elif kind == "beams":
            beams = _log_int(rng, 1, 16)
            case = _beam_case(None, _log_int(rng, 1, 64), beams, rng.choice([beams, 2 * beams]), _log_int(rng, 1000, 131072),
                              rng.choice(["bf16", "fp32"]), rng.choice([0.0, 0.1, 0.5]), rng.random() < 0.2,
                              _log_int(rng, 1, 1000))
        else:
            seqs = _log_int(rng, 1, 256)
            case = _context_case(kind, None, seqs, _log_int(rng, 1, 65536), rng.uniform(0.0, 1.2), 131072,
                                 rng.choice([0, 0, 0, 1]), *heads, block_tokens, group_dims, rng.randrange(1 << 30))
        w = work(case)
        if all(w[x] <= max(v[x] for k, v in works if k == kind) for x in ("bytes", "flops")):
            return case


def _lengths(case):
    r = random.Random(case["shape_seed"])
    drawn = [int(min(case["top"], max(1, round(case["median"] * math.exp(case["sigma"] * r.gauss(0.0, 1.0))))))
             for _ in range(case["seqs"])]
    return [case["top"]] * min(case["longest"], case["seqs"]) + drawn[case["longest"]:]


def _row_bytes(case):
    """Key and value of one token and head: codes, and a scale and a minimum a group."""
    return 2 * (HEAD_DIM // 2 + HEAD_DIM // case["group_dims"] * 4)


def work(case):
    """Bytes and operations of one pass: inputs read once, outputs written once."""
    if case["kind"] == "beams":
        rows, n = case["groups"] * case["beams"], case["groups"] * case["candidates"]
        values = rows * case["vocab"]
        return {"bytes": values * (2 if case["dtype"] == "bf16" else 4) + rows * 9 + n * 17 + 4 * n * case["history"],
                "flops": 4 * values}
    if case["kind"] == "write":
        rows, pages = case["tokens"] * case["kv_heads"], -(-case["tokens"] // case["block_tokens"])
        held = pages * case["block_tokens"] * case["kv_heads"]
        return {"bytes": rows * (4 * HEAD_DIM + _row_bytes(case)) + 8 * case["tokens"] + held * 4 * HEAD_DIM,
                "flops": 2 * rows * HEAD_DIM * 6 + 2 * held * HEAD_DIM * 2}
    lengths = _lengths(case)
    entries = sum(-(-n // case["block_tokens"]) for n in lengths)
    if case["kind"] == "load":
        rows = entries * case["block_tokens"] * case["kv_heads"]
        return {"bytes": rows * (4 * HEAD_DIM + _row_bytes(case)) + 8 * entries, "flops": 2 * rows * HEAD_DIM * 2}
    return {"bytes": sum(lengths) * case["kv_heads"] * _row_bytes(case) + 4 * case["seqs"] * case["q_heads"] * HEAD_DIM
            + 4 * entries + 4 * case["seqs"], "flops": 4 * HEAD_DIM * case["q_heads"] * sum(lengths)}


# ---------------------------------------------------------------------------
# inputs


def _kv_source(seed, kv_heads):
    """A generator of keys and values [n, heads, 128] in bf16: channels of keys differ in
    their means and widths, as they do behind a projection."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    mean = torch.randn((kv_heads, HEAD_DIM), generator=gen, device="cuda")
    width = torch.exp(0.4 * torch.randn((kv_heads, HEAD_DIM), generator=gen, device="cuda"))

    def rows(n):
        k = torch.randn((n, kv_heads, HEAD_DIM), generator=gen, device="cuda").mul_(width).add_(mean).to(torch.bfloat16)
        v = torch.randn((n, kv_heads, HEAD_DIM), generator=gen, device="cuda").mul_(0.5).to(torch.bfloat16)
        return k, v

    return gen, rows


def _pool_chunks(blocks, kv_heads, block_tokens):
    step = max(1, CHUNK // 8 // (kv_heads * block_tokens * HEAD_DIM))
    return [(lo, min(blocks, lo + step)) for lo in range(0, blocks, step)]


def _paged(x, blocks, block_tokens):
    """[blocks * block_tokens, heads, ...] -> [blocks, heads, block_tokens, ...]"""
    return x.view(blocks, block_tokens, *x.shape[1:]).transpose(1, 2)


def _quantise(x, group_dims):
    """(codes, scales, minima) of rows of 128 values."""
    x = x.float().unflatten(-1, (-1, group_dims))
    lo = x.amin(dim=-1, keepdim=True).clamp(-FP16_MAX, FP16_MAX)
    hi = x.amax(dim=-1, keepdim=True).clamp(-FP16_MAX, FP16_MAX)
    m = lo.half()
    s = ((hi - lo) / 15).half()
    c = torch.round((x - m.float()) / torch.where(s > 0, s, torch.ones_like(s)).float()).clamp(0, 15)
    c = torch.where(s > 0, c, torch.zeros_like(c))
    return c.to(torch.uint8).flatten(-2), s.squeeze(-1), m.squeeze(-1)


def _values(codes, scales, minima):
    """What codes stand for, in 32 bits."""
    per_group = codes.unflatten(-1, (scales.shape[-1], -1)).float()
    return (per_group * scales[..., None].float() + minima[..., None].float()).flatten(-2)


def _prepare_pool(case, state, blocks, rows):
    """The cache in hand before the call: the library's, or the plain form's codes."""
    hkv, bt, gd = case["kv_heads"], case["block_tokens"], case["group_dims"]
    if own:
        import paged_kv_cache_49_gb300 as pkv
        state["cache"] = pkv.Int4Cache(blocks, hkv, bt, gd)
    else:
        kinds = ((HEAD_DIM, torch.uint8), (HEAD_DIM // gd, torch.float16), (HEAD_DIM // gd, torch.float16))
        state["k"], state["v"] = ([torch.zeros((blocks, hkv, bt, n), dtype=t, device="cuda") for n, t in kinds]
                                  for _ in range(2))
    if rows is None:
        return
    for lo, hi in _pool_chunks(blocks, hkv, bt):
        k, v = rows((hi - lo) * bt)
        if own:
            slots = torch.arange(lo * bt, hi * bt, device="cuda")
            pkv.append_int4(k, v, slots, state["cache"])
        else:
            for held, x in ((state["k"], k), (state["v"], v)):
                for dst, src in zip(held, _quantise(x, gd)):
                    dst[lo:hi] = _paged(src, hi - lo, bt)


def _prepare_beams(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    g, k, vocab, room = case["groups"], case["beams"], case["vocab"], case["history"]
    rand = lambda *shape: torch.rand(shape, generator=gen, device="cuda")
    logits = torch.randn((g * k, vocab), generator=gen, device="cuda").mul_(1.5)
    # a few tokens stand out in each row, some are barred everywhere
    likely = torch.randint(0, vocab, (g * k, 12), generator=gen, device="cuda")
    logits.scatter_add_(1, likely, 4.0 + 4.0 * rand(g * k, 12))
    logits[:, torch.randint(0, vocab, (37,), generator=gen, device="cuda")] = -math.inf
    state = {"case": case, "logits": logits.to(torch.bfloat16) if case["dtype"] == "bf16" else logits, "eos": 2}
    state["scores"] = torch.sort(-3.0 - 9.0 * rand(g, k), dim=1, descending=True).values
    state["finished"] = rand(g, k) < case["finished"]
    state["lengths"] = (1 + rand(g, k) * (room - 1)).to(torch.int32).clamp(max=max(room - 1, 0))
    if case["first"]:  # the beams of a group are alike before the first step: one of them counts
        state["scores"][:, 1:] = -math.inf
        state["finished"][:] = False
    state["history"] = torch.randint(0, vocab, (g, k, room), generator=gen, device="cuda", dtype=torch.int32)
    if own:
        import paged_kv_cache_49_gb300 as pkv
        state["out"] = pkv.BeamBuffers(g, case["candidates"], room)
        state["workspace"] = pkv.BeamWorkspace(g, k, case["candidates"], vocab)
    else:
        state["history_out"] = torch.zeros((g, case["candidates"], room), dtype=torch.int32, device="cuda")
    return state


def _tables(case, r):
    """Each sequence's pages, in an order without order, and the pool's blocks."""
    per_seq = [-(-n // case["block_tokens"]) for n in _lengths(case)]
    blocks = sum(per_seq) + sum(per_seq) // 10 + 1
    order = list(range(blocks))
    r.shuffle(order)
    rows, at = [], 0
    for n in per_seq:
        rows.append(order[at:at + n])
        at += n
    return rows, blocks


def prepare(case, seed):
    if case["kind"] == "beams":
        return _prepare_beams(case, seed)
    gen, rows = _kv_source(seed, case["kv_heads"])
    r = random.Random(seed)
    hkv, bt = case["kv_heads"], case["block_tokens"]
    state = {"case": case}
    if case["kind"] == "write":
        t = case["tokens"]
        pages = -(-t // bt)
        # the fused projection's output: k and v are views of it
        fused = torch.empty((t, 4 * hkv, HEAD_DIM), dtype=torch.bfloat16, device="cuda")
        state["new_k"], state["new_v"] = fused[:, 2 * hkv:3 * hkv], fused[:, 3 * hkv:]
        for dst, src in zip((state["new_k"], state["new_v"]), rows(t)):
            dst.copy_(src)
        order = torch.randperm(pages, generator=gen, device="cuda")
        at = torch.arange(t, device="cuda")
        state["slots"] = order[at // bt] * bt + at % bt
        state["kept"] = t - min(case["padding"], t - 1)
        state["slots"][state["kept"]:] = -1
        _prepare_pool(case, state, pages, None)
        if own:
            state["pairs"] = torch.arange(pages, dtype=torch.int32, device="cuda")[:, None].repeat(1, 2).contiguous()
    else:
        tables, blocks = _tables(case, r)
        state["lengths"] = _lengths(case)
        _prepare_pool(case, state, blocks, rows)
        if case["kind"] == "load":
            pages = sum(len(x) for x in tables)
            state["blocks"] = torch.tensor([b for row in tables for b in row], dtype=torch.int32, device="cuda")
            state["pairs"] = torch.stack([state["blocks"], torch.arange(pages, dtype=torch.int32, device="cuda")], dim=1)
        else:
            width = max(len(x) for x in tables)
            state["tables"] = torch.tensor([x + [-1] * (width - len(x)) for x in tables], dtype=torch.int32, device="cuda")
            state["context_lens"] = torch.tensor(state["lengths"], dtype=torch.int32, device="cuda")
            state["q"] = torch.randn((case["seqs"], case["q_heads"], HEAD_DIM), generator=gen, device="cuda").to(torch.bfloat16)
            state["scale"] = 1.0 / math.sqrt(HEAD_DIM)
            if own:
                import paged_kv_cache_49_gb300 as pkv
                state["workspace"] = pkv.AttentionWorkspace(case["seqs"], hkv)
                state["out"] = torch.empty_like(state["q"])
    if own and case["kind"] != "decode":
        import paged_kv_cache_49_gb300 as pkv
        state["errors"] = pkv.new_error_word()
        shape = (state["pairs"].shape[0], hkv, bt, HEAD_DIM)
        state["k_pages"], state["v_pages"] = (torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    return state


# ---------------------------------------------------------------------------
# one pass


def run(state):
    kind = state["case"]["kind"]
    if own:
        import paged_kv_cache_49_gb300 as pkv
        if kind == "beams":
            out = pkv.beam_select(state["logits"], state["scores"], state["finished"], state["eos"], state["history"],
                                  state["lengths"], out=state["out"], workspace=state["workspace"])
            return out.scores, out.tokens, out.parents, out.finished, out.lengths, out.history
        if kind == "decode":
            return pkv.attn_decode_int4(state["q"], state["cache"], state["tables"], state["context_lens"], state["scale"],
                                        out=state["out"], workspace=state["workspace"])
        if kind == "write":
            pkv.append_int4(state["new_k"], state["new_v"], state["slots"], state["cache"], state["errors"])
        pkv.load_int4(state["cache"], state["pairs"], state["k_pages"], state["v_pages"], state["errors"])
        return state["k_pages"], state["v_pages"]
    if kind == "beams":
        return _plain_beams(state)
    if kind == "decode":
        return _plain_decode(state)
    if kind == "load":
        blocks = state["blocks"].long()
        return tuple(_values(*(x[blocks] for x in state[name])).to(torch.bfloat16) for name in "kv")
    return _plain_write(state)


def _plain_write(state):
    bt = state["case"]["block_tokens"]
    slots = state["slots"][:state["kept"]]
    for name in "kv":
        for dst, src in zip(state[name], _quantise(state["new_" + name][:state["kept"]], state["case"]["group_dims"])):
            dst[slots // bt, :, slots % bt] = src
    return tuple(_values(*state[name]).to(torch.bfloat16) for name in "kv")


def _plain_decode(state):
    case = state["case"]
    hkv, group = case["kv_heads"], case["q_heads"] // case["kv_heads"]
    out = torch.empty_like(state["q"])
    for s, n in enumerate(state["lengths"]):
        blocks = state["tables"][s, :-(-n // case["block_tokens"])].long()
        keys, values = (_values(*(x[blocks] for x in state[name])).transpose(0, 1).reshape(hkv, -1, HEAD_DIM)[:, :n]
                        for name in "kv")
        q = state["q"][s].float().view(hkv, group, HEAD_DIM)
        scores = torch.matmul(q, keys.transpose(1, 2)) * state["scale"]
        weights = torch.exp(scores - scores.amax(dim=-1, keepdim=True))
        o = torch.matmul(weights, values) / weights.sum(dim=-1, keepdim=True)
        out[s] = o.view(-1, HEAD_DIM).to(out.dtype)
    return out


def _plain_beams(state):
    """Scores in 64 bits: neighbours of the last one taken may differ by little."""
    case = state["case"]
    g, k, n, vocab = case["groups"], case["beams"], case["candidates"], case["vocab"]
    device = state["logits"].device
    x = state["logits"].view(g, k, vocab).double()
    top = x.amax(dim=-1, keepdim=True)
    x = x - (top + torch.log(torch.exp(x - top).sum(dim=-1, keepdim=True))) + state["scores"].double()[..., None]
    # a finished beam goes on as it is
    done = state["finished"][..., None]
    only = torch.arange(vocab, device=device) == state["eos"]
    x = torch.where(done, torch.where(only, state["scores"].double()[..., None], -math.inf), x).view(g, k * vocab)
    x = torch.where(torch.isnan(x), -math.inf, x)
    scores, at = torch.sort(x, dim=1, descending=True, stable=True)
    scores, at = scores[:, :n], at[:, :n]
    some = scores > -math.inf
    tokens = torch.where(some, at % vocab, -1).to(torch.int32)
    parents = torch.where(some, at // vocab, -1).to(torch.int32)
    p = parents.long().clamp(min=0)
    was = torch.gather(state["finished"], 1, p) & some
    finished = was | (tokens == state["eos"])
    held = torch.where(some, torch.gather(state["lengths"], 1, p), 0)
    lengths = held + (some & ~was).to(torch.int32)
    position = torch.arange(case["history"], device=device)
    history = torch.gather(state["history"], 1, p[..., None].expand(-1, -1, case["history"]))
    history = torch.where(position < held[..., None], history, state["history_out"])
    history = torch.where((position == held[..., None]) & (some & ~was)[..., None], tokens[..., None], history)
    return scores.float(), tokens, parents, finished, lengths, history


# ---------------------------------------------------------------------------
# the definition in 64 bits


def _exact_rows(x, group_dims):
    """Rows of 128 values as a 4-bit cache gives them back."""
    rows = x.double().reshape(*x.shape[:-1], HEAD_DIM // group_dims, group_dims)
    least, most = (x.clamp(-FP16_MAX, FP16_MAX) for x in (rows.min(-1)[0], rows.max(-1)[0]))
    span = most - least
    m = least.float().half().double()[..., None]
    s = (span / 15).float().half().double()[..., None]
    code = torch.clamp(((rows - m) / s).round(), 0, 15)
    code[s.expand_as(code) == 0] = 0
    return (s * code + m).reshape(x.shape)


def exact(case, seed):
    if case["kind"] == "beams":
        return _exact_beams(case, seed)
    state = _exact_inputs(case, seed)
    hkv, bt, gd = case["kv_heads"], case["block_tokens"], case["group_dims"]
    if case["kind"] == "write":
        pages = []
        for x in state["kv"]:
            page = torch.zeros((-(-case["tokens"] // bt) * bt, hkv, HEAD_DIM), dtype=torch.float64, device="cuda")
            page[state["slots"]] = _exact_rows(x, gd)
            pages.append(page.view(-1, bt, hkv, HEAD_DIM).permute(0, 2, 1, 3).contiguous())
        return tuple(pages)
    if case["kind"] == "load":
        at = torch.tensor([b for row in state["tables"] for b in row], device="cuda")
        return tuple(_exact_rows(x[at], gd) for x in state["kv"])
    result = torch.empty(state["q"].shape, dtype=torch.float64, device="cuda")
    group = case["q_heads"] // hkv
    for s, n in enumerate(_lengths(case)):
        token = torch.arange(n, device="cuda")
        page = torch.tensor(state["tables"][s], device="cuda")[token // bt]
        for g in range(hkv):
            key, value = (_exact_rows(x[page, g, token % bt], gd) for x in state["kv"])
            w = torch.softmax(state["q"][s, g * group:(g + 1) * group].double() @ key.T / math.sqrt(HEAD_DIM), dim=1)
            result[s, g * group:(g + 1) * group] = w @ value
    return result


def _exact_inputs(case, seed):
    """The inputs of prepare() as they are before they are quantised."""
    gen, rows = _kv_source(seed, case["kv_heads"])
    bt = case["block_tokens"]
    if case["kind"] == "write":
        kv, pages = rows(case["tokens"]), -(-case["tokens"] // bt)
        order = torch.randperm(pages, generator=gen, device="cuda").tolist()
        kept = case["tokens"] - min(case["padding"], case["tokens"] - 1)
        return {"kv": [x[:kept] for x in kv],
                "slots": torch.tensor([order[i // bt] * bt + i % bt for i in range(kept)], device="cuda")}
    tables, blocks = _tables(case, random.Random(seed))
    kv = [torch.empty((blocks, case["kv_heads"], bt, HEAD_DIM), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for lo, hi in _pool_chunks(blocks, case["kv_heads"], bt):
        for dst, src in zip(kv, rows((hi - lo) * bt)):
            dst[lo:hi] = _paged(src, hi - lo, bt)
    state = {"kv": kv, "tables": tables}
    if case["kind"] == "decode":
        state["q"] = torch.randn((case["seqs"], case["q_heads"], HEAD_DIM), generator=gen, device="cuda").to(torch.bfloat16)
    return state


def _exact_beams(case, seed):
    state = _prepare_beams(case, seed)
    g, k, n, vocab, eos = case["groups"], case["beams"], case["candidates"], case["vocab"], state["eos"]
    scores = torch.full((g, n), -math.inf, dtype=torch.float64)
    tokens, parents = (torch.full((g, n), -1, dtype=torch.int32) for _ in range(2))
    finished, lengths = torch.zeros((g, n), dtype=torch.bool), torch.zeros((g, n), dtype=torch.int32)
    history = torch.zeros((g, n, case["history"]), dtype=torch.int32)
    before, held, done = state["history"].cpu(), state["lengths"].tolist(), state["finished"].tolist()
    for b in range(g):
        total = torch.log_softmax(state["logits"][b * k:(b + 1) * k].double(), dim=1)
        total += state["scores"][b].double()[:, None]
        for i in range(k):
            if done[b][i]:
                total[i] = -math.inf
                total[i, eos] = state["scores"][b, i].double()
        total = torch.nan_to_num(total, nan=-math.inf, neginf=-math.inf).flatten()
        for j in range(n):
            best = total.max()
            if not best > -math.inf:
                break
            at = int((total == best).nonzero()[0])
            total[at] = -math.inf
            i, token = divmod(at, vocab)
            scores[b, j], tokens[b, j], parents[b, j] = best, token, i
            finished[b, j] = done[b][i] or token == eos
            kept = held[b][i]
            history[b, j, :kept] = before[b, i, :kept]
            if not done[b][i]:
                history[b, j, kept] = token
            lengths[b, j] = kept + (0 if done[b][i] else 1)
    return tuple(x.cuda() for x in (scores, tokens, parents, finished, lengths, history))
