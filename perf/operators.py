"""Cases of the operators that serve a compressed KV cache with a bounded
memory: attention over a sliding window with a few first tokens that stay
visible (one new token per sequence, and prompt chunks), and the pages behind
it (advanced by a step, forked, compacted, copied).

`own` chooses between the operators' plain form (elementary torch operations)
and the framework's calls. A container holds one token's K or V head vector:
an fp16 norm, a 24-bit rANS state and its renormalisation bytes; a block is 32
containers, byte-interleaved. The vector is norm * D * H * y / 128, with y the
decoded levels, H the Walsh-Hadamard matrix and D the head's signs.
"""
import math

import torch

own = False

DEV = "cuda"
K_LEVELS, V_LEVELS = 8, 6
# Frequencies (of 4096), levels and thresholds of the upper half of the
# symmetric tables, by (levels, container bytes): 1.96, 2.26 and 3.0 bits.
TABLES = {
    (8, 31): ([1745, 297, 5, 1], [0.6075646877288818, 1.8666375875473022, 3.269965648651123, 4.947254657745361],
              [1.4465693235397339, 2.9871561527252197, 4.7523064613342285]),
    (8, 36): ([1518, 485, 44, 1], [0.507427990436554, 1.5356272459030151, 2.6062002182006836, 3.759296417236328],
              [1.1290714740753174, 2.2868895530700684, 3.5083816051483154]),
    (8, 48): ([928, 677, 346, 97], [0.2922300100326538, 0.8892105221748352, 1.5375365018844604, 2.3568990230560303],
              [0.6024525165557861, 1.2363989353179932, 1.9815667867660522]),
    (6, 31): ([1745, 297, 6], [0.6075502038002014, 1.866613507270813, 3.271406412124634],
              [1.446516752243042, 2.987417459487915]),
    (6, 36): ([1514, 489, 45], [0.5056282877922058, 1.532261610031128, 2.631152629852295],
              [1.123993158340454, 2.28859543800354]),
    (6, 48): ([1004, 741, 303], [0.3177163600921631, 1.0001060962677002, 1.8935948610305786],
              [0.6589112281799316, 1.4468504190444946]),
}
BITS = {31: 1.96, 36: 2.26, 48: 3.0}


def listed():
    return [
        # One user at an 8K context: the latency of a single decode step.
        dict(name="decode_b1_8k", op="decode", B=1, Hkv=8, G=4, T=8192, window=1024, sinks=4, C=36, paged=False, half=True, spread=0),
        # fp32 queries and outputs, one query head per KV head, an odd window, ragged lengths down to none, a page table.
        dict(name="decode_b19_f32", op="decode", B=19, Hkv=8, G=1, T=4001, window=1001, sinks=5, C=31, paged=True, half=False, spread=4001),
        # The serving batch at an 8K context, behind page tables whose middle has been given back.
        dict(name="decode_b128_8k", op="decode", B=128, Hkv=8, G=4, T=8192, window=2048, sinks=64, C=36, paged=True, half=True, spread=900),
        # The ragged tail of one prompt.
        dict(name="prefill_b1_n77", op="prefill", B=1, Hkv=8, G=4, T=2111, n_q=77, window=500, sinks=4, C=36, paged=True, half=True, spread=0),
        # A chunk of 512 tokens for a batch of prompts.
        dict(name="prefill_b16_n512", op="prefill", B=16, Hkv=8, G=4, T=8192, n_q=512, window=1024, sinks=4, C=36, paged=False, half=True, spread=1000),
        # Long prompts in large chunks, eight query heads per KV head, fp32 queries.
        dict(name="prefill_b4_64k", op="prefill", B=4, Hkv=4, G=8, T=65536, n_q=2048, window=4096, sinks=128, C=48, paged=False, half=False, spread=777),
        # The page bookkeeping of one decode step of the serving batch.
        dict(name="advance_b128", op="advance", B=128, max_pages=256, num_pages=8192, window=1024, sinks=4),
        # Long contexts without a window, prompts joining and leaving, a large pool of an odd size.
        dict(name="advance_b500", op="advance", B=500, max_pages=2048, num_pages=600011, window=0, sinks=0),
        # A beam step of a small batch, one layer's pools.
        dict(name="fork_b16", op="fork", B_in=16, B_out=16, max_pages=65, num_pages=1100, layers=1, Hkv=8, C=36),
        # Prompts forked into four samples each, all layers' pools in one tensor.
        dict(name="fork_b256", op="fork", B_in=64, B_out=256, max_pages=256, num_pages=17000, layers=4, Hkv=8, C=36),
        # A small uneven pool defragmented.
        dict(name="compact_777", op="compact", B=9, max_pages=100, num_pages=777, layers=1, Hkv=3, C=31),
        # A serving pool defragmented in all layers.
        dict(name="compact_8k", op="compact", B=48, max_pages=256, num_pages=8192, layers=8, Hkv=8, C=36),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["decode", "decode", "prefill", "prefill", "advance", "fork", "compact"])
    C = rng.choice([31, 36, 48])
    if op in ("decode", "prefill"):
        Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
        window, sinks = log(1, 4096), rng.choice([0, 1, 4, 33, 128])
        c = dict(op=op, Hkv=Hkv, G=G, window=window, sinks=sinks, C=C, paged=rng.random() < 0.5, half=rng.random() < 0.6)
        if op == "decode":
            T = log(1, 16384)
            B = log(1, min(128, max(1, 128 * 8 * 2000 // (min(T, window + sinks + 32) * Hkv))))
            return dict(c, B=B, T=T, spread=rng.choice([0, T // 3, T]))
        T = log(1, 32768)
        n_q = log(1, min(T, 2048))
        B = log(1, min(16, max(1, 4 * 32 * 2048 * 4096 // (n_q * Hkv * G * (min(T, window + n_q) + sinks + 64)))))
        return dict(c, B=B, T=T, n_q=n_q, spread=rng.choice([0, (T - n_q) // 2, T - n_q]))
    if op == "advance":
        B, max_pages = log(1, 512), log(1, 1024)
        return dict(op=op, B=B, max_pages=max_pages, num_pages=max(16, int(B * max_pages * rng.uniform(0.2, 1.0))),
                    window=rng.choice([0, log(1, 32 * max_pages)]), sinks=rng.choice([0, 4, 40]))
    max_pages, Hkv = log(1, 256), rng.choice([1, 3, 8])
    layers = rng.choice([1, 2, 4])
    B = log(1, 48)
    if op == "fork":
        return dict(op=op, B_in=B, B_out=log(1, 256), max_pages=max_pages, num_pages=B * max_pages + log(1, 200), layers=layers, Hkv=Hkv, C=C)
    return dict(op=op, B=B, max_pages=max_pages, num_pages=B * max_pages + log(1, 200), layers=layers, Hkv=Hkv, C=C)


# ---- inputs ---------------------------------------------------------------


def _full_table(n, C):
    """Frequencies, their running sums, levels and thresholds of a symmetric table."""
    f, y, t = TABLES[n, C]
    freq = f[::-1] + f
    cum = [sum(freq[:i]) for i in range(n)]
    return freq, cum, [-v for v in y[::-1]] + y, [-v for v in t[::-1]] + [0.0] + t


def _signs(heads):
    """Rotation signs [heads, 128] from splitmix64 with seed 0: two 64-bit words per head, a set bit is -1."""
    rows = []
    for i in range(1, 2 * heads + 1):
        z = (i * 0x9E3779B97F4A7C15) & (2**64 - 1)
        z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & (2**64 - 1)
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & (2**64 - 1)
        z ^= z >> 31
        rows.append([-1.0 if z >> b & 1 else 1.0 for b in range(64)])
    return torch.tensor(rows, device=DEV).reshape(heads, 128)


def _containers(gen, count, n, C):
    """`count` containers [count, C] of normal vectors: quantised, rANS-coded from the last symbol to the first."""
    freq, cum, _, thr = _full_table(n, C)
    F, S = torch.tensor(freq, device=DEV, dtype=torch.int32), torch.tensor(cum, device=DEV, dtype=torch.int32)
    u = torch.randn(count, 128, device=DEV, generator=gen)
    sym = torch.bucketize(u, torch.tensor(thr, device=DEV), right=True)
    x = torch.full((count,), 65536, device=DEV, dtype=torch.int32)
    pushed = torch.zeros(count, 260, device=DEV, dtype=torch.uint8)
    at = torch.zeros(count, 1, device=DEV, dtype=torch.int64)
    for i in range(127, -1, -1):
        f = F[sym[:, i]]
        for _ in range(2):
            full = x >= 4096 * f
            pushed.scatter_(1, at, (x & 255).to(torch.uint8)[:, None])
            at += full[:, None]
            x = torch.where(full, x >> 8, x)
        x = (torch.div(x, f, rounding_mode="floor") << 12) + x % f + S[sym[:, i]]
    norm = (11.3 * torch.exp(0.25 * torch.randn(count, device=DEV, generator=gen))).half().view(torch.int16).to(torch.int32)
    out = torch.zeros(count, C, device=DEV, dtype=torch.uint8)
    for j, v in enumerate((norm & 255, (norm >> 8) & 255, x & 255, (x >> 8) & 255, x >> 16)):
        out[:, j] = v.to(torch.uint8)
    back = at - 1 - torch.arange(C - 5, device=DEV)
    out[:, 5:] = torch.where(back >= 0, pushed.gather(1, back.clamp(min=0)), torch.zeros_like(out[:, 5:]))
    fits = torch.nonzero(at[:, 0] <= C - 5)[:, 0]  # the few that are too long give way to others
    return out[fits[torch.arange(count, device=DEV) % fits.numel()]]


def _blocks(gen, shape, n, C):
    """Random blocks [*shape, C, 32] of valid containers, drawn from 2048 different blocks."""
    bank = _containers(gen, 2048 * 32, n, C).reshape(2048, 32, C).transpose(1, 2).contiguous()
    return bank[torch.randint(2048, shape, device=DEV, generator=gen)]


def _lens(case):
    """Tokens in each sequence: T, less a part of `spread` that differs from one to the next."""
    return [case["T"] - (b * 7919 * 31) % (case["spread"] + 1) for b in range(case["B"])]


def _attention_state(case, gen):
    B, Hkv, G, C, T = (case[k] for k in ("B", "Hkv", "G", "C", "T"))
    nb = (T + 31) // 32
    lens = _lens(case)
    n_q = case.get("n_q")
    s = {"lens": torch.tensor(lens, dtype=torch.int32, device=DEV), "table": None}
    if case["paged"]:
        pages = B * nb + 3
        perm = torch.randperm(pages, device=DEV, generator=gen)[:B * nb].reshape(B, nb)
        first = s["lens"].long() - (n_q or 1) - case["window"] + 1  # what no query sees has been given back
        j = torch.arange(nb, device=DEV)
        kept = (j * 32 < case["sinks"]) | (j * 32 + 32 > first[:, None])
        kept &= j * 32 < s["lens"][:, None]
        s["table"] = torch.where(kept, perm, -1).to(torch.int32).contiguous()
        shape = (pages, Hkv)
    else:
        shape = (B, Hkv, nb)
    s["k"], s["v"] = _blocks(gen, shape, K_LEVELS, C), _blocks(gen, shape, V_LEVELS, C)
    if not case["paged"]:
        s["k"], s["v"] = s["k"].reshape(B, Hkv, nb * 32, C), s["v"].reshape(B, Hkv, nb * 32, C)
    dt = torch.bfloat16 if case["half"] else torch.float32
    qshape = (B, Hkv * G, 128) if n_q is None else (B, n_q, Hkv * G, 128)
    s["q"] = torch.randn(qshape, device=DEV, generator=gen).to(dt)
    # The chunk kernels' key levels are fp16: a chunk's outputs are bf16, a decode step's of the query's type.
    s["out"] = torch.empty(qshape, device=DEV, dtype=dt if n_q is None else torch.bfloat16)
    if n_q is not None:
        s["start"] = s["lens"] - n_q
    return s


def _pages_state(case, gen):
    """A table of shuffled pages, lengths and reference counts; some rows share their first pages."""
    op, P, mp = case["op"], case["num_pages"], case["max_pages"]
    B = case["B_in"] if op == "fork" else case["B"]
    cap = 32 * mp
    j = torch.arange(mp, device=DEV)
    lens = torch.randint(0, cap + 1, (B,), device=DEV, generator=gen)
    if op == "advance":  # about a tenth of the pool is free
        budget = max(1, (P * 9 // 10) // B)
        if not case["window"] or (case["window"] + case["sinks"]) // 32 + 3 > budget:
            lens = lens.clamp(max=32 * budget)
    has = j * 32 < lens[:, None]
    if op == "advance" and case["window"]:  # the state that the last step left
        has &= (j * 32 < case["sinks"]) | (j * 32 + 32 > (lens - case["window"])[:, None])
    ids = torch.randperm(P, device=DEV, generator=gen)
    rank = torch.cumsum(has.reshape(-1), 0).reshape(B, mp) - 1
    table = torch.where(has & (rank < P), ids[rank.clamp(0, P - 1)], -1)
    if B > 1:  # every fourth row holds the prefix of the row before it
        both = (j < mp // 3) & (torch.arange(B, device=DEV)[:, None] % 4 == 1) & (table >= 0) & (table.roll(1, 0) >= 0)
        both &= (j * 32 + 32 <= lens[:, None]) & (j * 32 + 32 <= lens.roll(1)[:, None])
        table = torch.where(both, table.roll(1, 0), table)
    refs = torch.bincount(table[table >= 0], minlength=P)
    s = {"table": table.to(torch.int32), "lens": lens.to(torch.int32), "refs": refs.to(torch.int32),
         "refs_out": torch.empty(P, dtype=torch.int32, device=DEV), "counts": torch.zeros(8, dtype=torch.int32, device=DEV)}
    B_out = case.get("B_out", B)
    s["table_out"] = torch.empty(B_out, mp, dtype=torch.int32, device=DEV)
    if op == "advance":
        kind = torch.rand(B, device=DEV, generator=gen)
        more = torch.where(kind < 0.04, -1, torch.where(kind > 0.97, torch.randint(1, 2049, (B,), device=DEV, generator=gen), 1))
        s["n_new"] = more.to(torch.int32)
        s["lens_out"] = torch.empty(B, dtype=torch.int32, device=DEV)
        return s
    if op == "fork":
        parent = torch.randint(-1, B, (B_out,), device=DEV, generator=gen)
        stay = torch.rand(B_out, device=DEV, generator=gen) < 0.5
        at = torch.arange(B_out, device=DEV)
        s["parent"] = torch.where(stay & (at < B), at, parent).to(torch.int32)
        s["lens_out"] = torch.empty(B_out, dtype=torch.int32, device=DEV)
        s["pairs"] = torch.empty(B_out, 2, dtype=torch.int32, device=DEV)
    else:
        s["pairs"] = torch.empty(max(1, P // 2), 2, dtype=torch.int32, device=DEV)
    shape = (case["layers"], P, case["Hkv"], case["C"], 32)
    s["k"] = torch.randint(0, 256, shape, dtype=torch.uint8, device=DEV, generator=gen)
    s["v"] = torch.randint(0, 256, shape, dtype=torch.uint8, device=DEV, generator=gen)
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed) * 2654435761 % (2**63))
    attends = case["op"] in ("decode", "prefill")
    s = _attention_state(case, gen) if attends else _pages_state(case, gen)
    s["case"] = case
    if own:
        _plan(s)
    elif attends:
        s["signs"] = _signs(case["Hkv"])
        s["hadamard"] = _hadamard(torch.float32)
        s["k_lut"], s["v_lut"] = _lut(K_LEVELS, case["C"]), _lut(V_LEVELS, case["C"])
    return s


def _plan(s):
    """What a user's program keeps between calls of the framework: tables and workspaces."""
    import decode_attention_dq_b200 as dq

    c = s["case"]
    bits = BITS[c.get("C", 36)]
    s["tab"] = dq.dq_build_tables(n_kv_heads=c.get("Hkv", 1), k_bits_per_value=bits, v_bits_per_value=bits)
    if c["op"] == "decode":
        need = dq.dq_decode_workspace_bytes(s["tab"], c["B"], c["Hkv"] * c["G"], c["Hkv"], c["T"])
    elif c["op"] == "prefill":
        need = dq.dq_prefill_window_workspace_bytes(s["tab"], c["B"], c["Hkv"], -(-c["T"] // 32) * 32, c["n_q"], c["window"], c["sinks"])
    else:
        need = dq.dq_pages_workspace_bytes(s["tab"], c["num_pages"], max(c.get("B", 0), c.get("B_in", 0), c.get("B_out", 0)), c["max_pages"])
    s["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV)


# ---- one pass -------------------------------------------------------------


def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(s)
    if op == "decode":
        return _plain_decode(s)
    if op == "prefill":
        return _plain_prefill(s)
    if op == "advance":
        return _plain_advance(s)
    if op == "fork":
        return _plain_fork(s)
    return _plain_compact(s)


def _run_own(s):
    import decode_attention_dq_b200 as dq

    c = s["case"]
    if c["op"] == "decode":
        if c["paged"]:
            dq.dq_decode_attention_window_paged(s["tab"], s["q"], s["k"], s["v"], s["table"], s["lens"], c["T"], c["window"], c["sinks"],
                                                s["out"], s["workspace"])
        else:
            dq.dq_decode_attention_window(s["tab"], s["q"], s["k"], s["v"], s["lens"], c["T"], c["window"], c["sinks"], s["out"], s["workspace"])
        return s["out"]
    if c["op"] == "prefill":
        if c["paged"]:
            dq.dq_prefill_attention_window_paged(s["tab"], s["q"], s["k"], s["v"], s["table"], s["start"], c["window"], c["sinks"], s["out"],
                                                 s["workspace"])
        else:
            dq.dq_prefill_attention_window(s["tab"], s["q"], s["k"], s["v"], s["start"], c["window"], c["sinks"], s["out"], s["workspace"])
        return s["out"]
    if c["op"] == "advance":
        dq.dq_pages_advance(s["tab"], s["refs"], s["table"], s["lens"], s["n_new"], s["refs_out"], s["table_out"], s["lens_out"], s["counts"],
                            s["workspace"], window=c["window"], sinks=c["sinks"])
        return {k: s[k] for k in ("refs_out", "table_out", "lens_out", "counts")}
    if c["op"] == "fork":
        dq.dq_pages_fork(s["tab"], s["refs"], s["table"], s["lens"], s["parent"], s["refs_out"], s["table_out"], s["lens_out"], s["pairs"], s["counts"],
                         s["workspace"])
    else:
        dq.dq_pages_compact(s["tab"], s["refs"], s["table"], s["refs_out"], s["table_out"], s["pairs"], s["counts"], s["workspace"])
    dq.dq_pages_copy(s["tab"], s["k"], s["v"], s["pairs"], s["counts"])
    return {k: s[k] for k in ("refs_out", "table_out", "lens_out", "counts", "pairs", "k", "v") if k in s}


# ---- the plain form -------------------------------------------------------


def _hadamard(dtype):
    h = torch.ones(1, 1, device=DEV, dtype=dtype)
    while h.shape[0] < 128:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h


def _lut(n, C):
    """By slot of 4096: the symbol's frequency, the slot's place in it, the level."""
    freq, cum, lev, _ = _full_table(n, C)
    f = torch.tensor(freq, device=DEV)
    rep = lambda v, d: torch.tensor(v, device=DEV, dtype=d).repeat_interleave(f)  # noqa: E731
    return rep(freq, torch.int32), torch.arange(4096, device=DEV, dtype=torch.int32) - rep(cum, torch.int32), rep(lev, torch.float32)


def _decoded(cont, lut):
    """Containers [n, C] -> levels [n, 128] and norms [n]."""
    freq, place, level = lut
    n, C = cont.shape
    b = [cont[:, j].to(torch.int32) for j in range(5)]
    norm = (b[0] | (b[1] << 8)).to(torch.int16).view(torch.float16).float()
    x = b[2] | (b[3] << 8) | (b[4] << 16)
    at = torch.full((n, 1), 5, device=DEV, dtype=torch.int64)
    y = torch.empty(128, n, device=DEV)
    for i in range(128):  # the coder's state is a chain through the symbols
        slot = (x & 4095).long()
        y[i] = level[slot]
        x = freq[slot] * (x >> 12) + place[slot]
        for _ in range(2):
            low = x < 65536
            x = torch.where(low, (x << 8) + cont.gather(1, at.clamp(max=C - 1))[:, 0], x)
            at += low[:, None]
    return y.t(), norm


def _gathered(s, blocks):
    """Containers of the token blocks [B, M] of every KV head: K and V as [B * Hkv * M * 32, C]."""
    c = s["case"]
    got = []
    for cache in (s["k"], s["v"]):
        if c["paged"]:
            page = torch.gather(s["table"].long(), 1, blocks).clamp(min=0)
            x = cache[page].transpose(1, 2)  # [B, Hkv, M, C, 32]
        else:
            x = cache.reshape(c["B"], c["Hkv"], -1, c["C"], 32)
            x = x[torch.arange(c["B"], device=DEV)[:, None], :, blocks].transpose(1, 2)
        got.append(x.transpose(-1, -2).reshape(-1, c["C"]))
    return got


def _visible_blocks(s, lo, hi, width):
    """The blocks that hold the first tokens and positions lo..hi-1 [B], and the tokens' positions
    [B, M * 32], with -1 for a token that is there already or beyond hi."""
    c = s["case"]
    nb = (c["T"] + 31) // 32
    first = min(nb, (c["sinks"] + 31) // 32)
    a = torch.arange(first, device=DEV).expand(c["B"], first)
    b = (lo.clamp(min=0) // 32)[:, None] + torch.arange(min(nb, (width + 31) // 32 + 1), device=DEV)
    late = torch.where((b >= first) & (b < nb), b, -1)
    blocks = torch.cat([a, late], 1)
    pos = blocks[:, :, None] * 32 + torch.arange(32, device=DEV)
    pos = torch.where((blocks[:, :, None] >= 0) & (pos < hi[:, None, None]), pos, -1).reshape(c["B"], -1)
    return blocks.clamp(min=0), pos


def _rotated(s, q):
    """q [.., Hkv, G, 128] in the containers' domain, scaled for the scores."""
    return (q.float() * s["signs"][:, None, :]) @ s["hadamard"] / (128.0 * math.sqrt(128.0))


def _softmax(a):
    """Softmax over the last axis, 0 for a row with nothing in it."""
    m = a.amax(-1, keepdim=True)
    p = torch.exp(a - torch.where(m == -math.inf, 0.0, m))
    z = p.sum(-1, keepdim=True)
    return p / torch.where(z == 0, 1.0, z)


def _plain_decode(s):
    c = s["case"]
    B, Hkv, G = c["B"], c["Hkv"], c["G"]
    lens = s["lens"].long()
    blocks, pos = _visible_blocks(s, lens - c["window"], lens, c["window"])
    k, v = _gathered(s, blocks)
    yk, nk = _decoded(k, s["k_lut"])
    yv, nv = _decoded(v, s["v_lut"])
    shape = (B, Hkv, pos.shape[1])
    seen = (pos >= 0) & ((pos < c["sinks"]) | (pos >= (lens - c["window"])[:, None]))
    a = _rotated(s, s["q"].reshape(B, Hkv, G, 128)) @ yk.reshape(*shape, 128).transpose(-1, -2) * nk.reshape(*shape)[:, :, None]
    p = _softmax(torch.where(seen[:, None, None], a, -math.inf)) * nv.reshape(*shape)[:, :, None]
    o = (p @ yv.reshape(*shape, 128)) @ s["hadamard"] / 128.0 * s["signs"][:, None, :]
    return o.reshape(B, Hkv * G, 128).to(s["out"].dtype)


def _plain_prefill(s):
    c = s["case"]
    B, Hkv, G, n = c["B"], c["Hkv"], c["G"], c["n_q"]
    start = s["start"].long()
    blocks, pos = _visible_blocks(s, start - c["window"] + 1, start + n, c["window"] + n)
    k, v = _gathered(s, blocks)
    yk, nk = _decoded(k, s["k_lut"])
    yv, nv = _decoded(v, s["v_lut"])
    M = pos.shape[1]
    q = _rotated(s, s["q"].reshape(B, n, Hkv, G, 128)).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, 128)
    at = start[:, None] + torch.arange(n, device=DEV)
    out = torch.empty(B, n, Hkv * G, 128, device=DEV, dtype=s["out"].dtype)
    yk, yv, nk, nv = yk.reshape(B, Hkv, M, 128), yv.reshape(B, Hkv, M, 128), nk.reshape(B, Hkv, 1, M), nv.reshape(B, Hkv, 1, M)
    for b in range(B):  # one sequence at a time: the scores are large
        t, i = pos[b], at[b][:, None]
        seen = (t >= 0) & (t <= i) & ((t < c["sinks"]) | (t > i - c["window"]))
        a = torch.where(seen.repeat_interleave(G, 0), q[b] @ yk[b].transpose(-1, -2) * nk[b], -math.inf)
        o = ((_softmax(a) * nv[b]) @ yv[b]) @ s["hadamard"] / 128.0
        o = o.reshape(Hkv, n, G, 128) * s["signs"][:, None, None]
        out[b] = o.transpose(0, 1).reshape(n, Hkv * G, 128).to(out.dtype)
    return out


def _counts(refs, **named):
    order = ("free", "taken", "released", "short", "bad", "clamped", "pairs")
    named["free"] = (refs == 0).sum()
    zero = torch.zeros((), dtype=torch.int64, device=DEV)
    return torch.stack([named.get(k, zero) for k in order] + [zero]).to(torch.int32)


def _free_list(refs):
    """The free pages in ascending order, then -1, one entry more than there are pages."""
    free = refs == 0
    at = torch.where(free, torch.cumsum(free, 0) - 1, refs.numel())
    got = torch.full((refs.numel() + 1,), -1, dtype=torch.int64, device=DEV)
    got[at] = torch.where(free, torch.arange(refs.numel(), device=DEV), -1)
    got[-1] = -1
    return got


def _hand_out(refs, need):
    """The lowest free pages for the places where `need` is set, in their order; -1 where none is left."""
    rank = torch.cumsum(need.reshape(-1), 0).reshape(need.shape) - 1
    page = torch.where(need, _free_list(refs)[rank.clamp(0, refs.numel())], -1)
    taken = (page >= 0).reshape(-1)
    refs = refs + torch.zeros_like(refs).index_add_(0, page.reshape(-1).clamp(min=0), taken.to(refs.dtype))
    return refs, page, taken.sum(), need.sum() - taken.sum()


def _plain_advance(s):
    c = s["case"]
    P, mp = c["num_pages"], c["max_pages"]
    table, lens, n = s["table"].long(), s["lens"].long(), s["n_new"].long()
    j = torch.arange(mp, device=DEV)
    ends = n < 0
    want = torch.where(ends, 0, lens + n)
    new = want.clamp(max=32 * mp)
    gone = ends[:, None].expand(-1, mp)
    if c["window"]:
        gone = gone | ((j * 32 >= c["sinks"]) & (j * 32 + 32 <= (lens + 1 - c["window"])[:, None]))
    held = (table >= 0) & (table < P)
    drop = gone & held
    refs = s["refs"].long()
    refs = refs - torch.zeros_like(refs).index_add_(0, table.clamp(0, P - 1).reshape(-1), drop.reshape(-1).long())
    table2 = torch.where(gone | ~held, -1, table)
    need = (j >= (lens // 32)[:, None]) & (j < ((new + 31) // 32)[:, None]) & (table2 < 0)
    refs, page, taken, short = _hand_out(refs, need)
    table2 = torch.where(need, page, table2)
    counts = _counts(refs, taken=taken, released=drop.sum(), short=short, bad=(~held & (table != -1)).sum(), clamped=(want != new).sum())
    return {"refs_out": refs.to(torch.int32), "table_out": table2.to(torch.int32), "lens_out": new.to(torch.int32), "counts": counts}


def _plain_fork(s):
    c = s["case"]
    P, mp, B, B_out = c["num_pages"], c["max_pages"], c["B_in"], c["B_out"]
    table, lens, parent = s["table"].long(), s["lens"].long(), s["parent"].long()
    real = (parent >= 0) & (parent < B)
    p = parent.clamp(0, B - 1)
    out = torch.where(real[:, None], table[p], -1)
    new_lens = torch.where(real, lens[p], 0)
    # The last page, where it is not full, stays with a row's first child if nobody else holds it; the other children get a copy.
    part = (new_lens % 32 != 0) & real
    col = (new_lens // 32).clamp(max=mp - 1)
    tail = torch.gather(out, 1, col[:, None])[:, 0]
    part &= tail >= 0
    at = torch.arange(B_out, device=DEV)
    first = torch.full((B + 1,), B_out, device=DEV).scatter_reduce_(0, torch.where(real, p, B), at, "amin")[p] == at
    need = part & ~(first & (s["refs"].long()[tail.clamp(min=0)] == 1))
    old = s["refs"].long()
    refs, page, taken, short = _hand_out(old, need)
    out = torch.where(need[:, None] & (torch.arange(mp, device=DEV) == col[:, None]), page[:, None], out)
    count = lambda t: torch.zeros(P, dtype=torch.int64, device=DEV).index_add_(0, t.clamp(min=0).reshape(-1), (t >= 0).reshape(-1).long())  # noqa: E731
    refs = old - count(table) + count(out)
    copied = need & (page >= 0)
    rank = torch.where(copied, torch.cumsum(copied, 0) - 1, B_out)
    pairs = torch.full((B_out + 1, 2), -1, dtype=torch.int64, device=DEV)
    pairs[rank] = torch.stack([tail, page], 1)
    pairs[-1] = -1
    _plain_copy(s, pairs[:-1])
    counts = _counts(refs, taken=taken, short=short, pairs=copied.sum(), bad=(parent >= B).sum())
    return {"refs_out": refs.to(torch.int32), "table_out": out.to(torch.int32), "lens_out": new_lens.to(torch.int32), "counts": counts,
            "pairs": pairs[:-1].to(torch.int32), "k": s["k"], "v": s["v"]}


def _plain_compact(s):
    P = s["case"]["num_pages"]
    refs, table = s["refs"].long(), s["table"].long()
    live = refs > 0
    n = live.sum()
    ids = torch.arange(P, device=DEV)
    cap = s["pairs"].shape[0]
    pairs = torch.full((cap + 1, 2), -1, dtype=torch.int64, device=DEV)
    moved, hole = live & (ids >= n), ~live & (ids < n)
    to = torch.where(live, ids, -1)
    mrank, hrank = torch.cumsum(moved, 0) - 1, torch.cumsum(hole, 0) - 1
    pairs[torch.where(moved, mrank, cap), 0] = ids
    pairs[torch.where(hole, hrank, cap), 1] = ids
    pairs[-1] = -1
    to = torch.where(moved, pairs[mrank.clamp(0, cap), 1], to)
    held = (table >= 0) & (table < P)
    out = torch.where(held, to[table.clamp(0, P - 1)], -1)
    refs2 = torch.zeros(P + 1, dtype=torch.int64, device=DEV)
    refs2[torch.where(live, to, P)] = refs
    refs2 = refs2[:-1]
    _plain_copy(s, pairs[:-1])
    counts = _counts(refs2, pairs=moved.sum(), bad=(~held & (table != -1)).sum())
    return {"refs_out": refs2.to(torch.int32), "table_out": out.to(torch.int32), "counts": counts, "pairs": pairs[:-1].to(torch.int32),
            "k": s["k"], "v": s["v"]}


def _plain_copy(s, pairs):
    got = pairs[pairs[:, 0] >= 0]
    for pool in (s["k"], s["v"]):
        pool[:, got[:, 1]] = pool[:, got[:, 0]]


# ---- what a pass cannot do without ----------------------------------------


def _seen_tokens(case):
    """Tokens that some query of a sequence sees, and (query, token) pairs, summed over the sequences."""
    W, S, n = case["window"], case["sinks"], case.get("n_q", 1)
    tokens = pairs = 0
    for L in _lens(case):
        lo = max(0, L - n + 1 - W)
        tokens += max(0, L - max(lo, 0)) + min(S, lo)
        for p in range(L - n, L):
            if p >= 0:
                w0 = max(0, p - W + 1)
                pairs += p + 1 - w0 + min(S, w0)
    return tokens, pairs


def work(case):
    op = case["op"]
    if op in ("decode", "prefill"):
        tokens, pairs = _seen_tokens(case)
        rows = case["B"] * case.get("n_q", 1) * case["Hkv"] * case["G"]
        out = 4 if op == "decode" and not case["half"] else 2
        moved = tokens * case["Hkv"] * 2 * case["C"] + rows * 128 * ((2 if case["half"] else 4) + out)
        return {"bytes": moved, "flops": pairs * case["Hkv"] * case["G"] * 4 * 128}
    B = case.get("B", case.get("B_in"))
    B_out = case.get("B_out", B)
    # Counts and tables in and out; a copied page is read and written in every layer.
    moved = 8 * case["num_pages"] + 4 * (B + B_out) * (case["max_pages"] + 1)
    page = 2 * case.get("Hkv", 0) * case.get("C", 0) * 32 * case.get("layers", 0)
    if op == "fork":
        # Nearly every row ends inside a page; half of the rows stay, the others choose a parent or none.
        moved += 2 * page * max(0, int(0.5 * B_out))
    elif op == "compact":
        held = min(case["num_pages"], B * case["max_pages"] // 2)
        moved += 2 * page * int(held * (1 - held / case["num_pages"]))
    return {"bytes": moved, "flops": 0}


# ---- the definition in 64 bits --------------------------------------------


def _unpacked(cont, n, C):
    """Containers [m, C] -> vectors' levels [m, 128] and norms [m] in 64 bits, symbol by symbol from the running sums."""
    freq, cum, lev, _ = _full_table(n, C)
    F, S = torch.tensor(freq, device=DEV), torch.tensor(cum, device=DEV)
    Y = torch.tensor(lev, device=DEV, dtype=torch.float64)
    wide = torch.cat([cont.long(), torch.zeros(cont.shape[0], 300, dtype=torch.long, device=DEV)], 1)
    half = (wide[:, 0] + 256 * wide[:, 1])
    e, m = (half >> 10) & 31, half & 1023
    norm = torch.where(e == 0, m * 2.0**-24, (1024 + m).double() * torch.exp2(e.double() - 25))
    x = wide[:, 2] + 256 * wide[:, 3] + 65536 * wide[:, 4]
    nxt = torch.full_like(x, 5)
    cols = []
    for _ in range(128):
        r = x % 4096
        sym = torch.searchsorted(S, r, right=True) - 1
        cols.append(sym.to(torch.uint8))
        x = F[sym] * torch.div(x, 4096, rounding_mode="floor") + r - S[sym]
        while True:
            low = x < 65536
            if not bool(low.any()):
                break
            x = torch.where(low, x * 256 + wide.gather(1, nxt[:, None])[:, 0], x)
            nxt = nxt + low.long()
    return Y[torch.stack(cols, 1).long()], norm


def exact(case, seed):
    if case["op"] not in ("decode", "prefill"):
        return None
    tokens, pairs = _seen_tokens(case)
    if tokens * case["Hkv"] > 3_000_000 or pairs * case["Hkv"] * case["G"] > 3_000_000_000:
        return None
    gen = torch.Generator(device=DEV).manual_seed(int(seed) * 2654435761 % (2**63))
    s = _attention_state(case, gen)
    C, Hkv, G, W, S = case["C"], case["Hkv"], case["G"], case["window"], case["sinks"]
    n = case.get("n_q", 1)
    H, D = _hadamard(torch.float64), _signs(Hkv).double()
    out = torch.zeros(case["B"], n, Hkv * G, 128, dtype=torch.float64, device=DEV)
    q = s["q"].double().reshape(case["B"], n, Hkv, G, 128)
    for b, L in enumerate(_lens(case)):
        first = L - n
        lo = max(0, first + 1 - W)
        t = torch.cat([torch.arange(min(S, lo), device=DEV), torch.arange(lo, max(lo, L), device=DEV)])
        if not t.numel():
            continue
        rows = []
        for cache in (s["k"], s["v"]):
            if case["paged"]:
                x = cache[s["table"][b, t // 32].long(), :, :, t % 32]
            else:
                x = cache.reshape(case["B"], Hkv, -1, C, 32)[b][:, t // 32, :, t % 32]
            rows.append(x.reshape(t.numel() * Hkv, C))
        vec = []
        for x, levels in zip(rows, (K_LEVELS, V_LEVELS)):
            y, norm = _unpacked(x, levels, C)
            vec.append((norm[:, None] * (y @ H) / 128).reshape(t.numel(), Hkv, 128) * D)
        i = (first + torch.arange(n, device=DEV))[:, None]
        seen = (t <= i) & ((t > i - W) | (t < S))
        for h in range(Hkv):
            a = torch.einsum("igd,td->git", q[b, :, h], vec[0][:, h]) / math.sqrt(128.0)
            a = a.masked_fill(~seen, -math.inf)
            p = torch.softmax(a, -1)
            p = torch.where(seen.any(-1)[:, None], p, torch.zeros_like(p))
            out[b, :, h * G:(h + 1) * G] = torch.einsum("git,td->igd", p, vec[1][:, h])
    return out[:, 0] if case["op"] == "decode" else out
