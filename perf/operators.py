"""Timing cases of the ragged serving step over a paged TQ4 cache.

Four operators that a serving program calls one after the other, with the plain
torch form of each beside the library's call:

  plan     block tables and slot maps from the requests' lengths
  rope     rotary positions (one or three axes) on q and k, then encode + append of k, v
  decode   one to four query tokens per request, sliding window and sinks, over the pages
  ragged   chunks of new tokens of several requests at once, over their paged prefixes

A pool page holds 256 positions of one layer: K words [4 heads][256][32 u32] (eight
4-bit indices each), V words, K norms [4][256] fp16, V norms. A stored vector stands for
norm * R^T c[idx], R = H diag(signs) / 16, c the 16-level Lloyd-Max codebook of
N(0, 1/256).
"""
import math
import random

import numpy as np
import torch

own = False

D, PAGE, H_KV, H_Q, GROUP = 256, 256, 4, 24, 6
PAGE_BYTES, PAGE_WORDS, PAGE_HALVES = 266_240, 66_560, 133_120
SCALE = 1.0 / 16.0
NO_WINDOW = 1 << 30
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- the format's constants
def _codebook():
    """The 16-level Lloyd-Max quantiser of N(0, 1/256) in 64 bits: (centroids, boundaries)."""
    pdf = lambda z: math.exp(-0.5 * z * z) / math.sqrt(2 * math.pi) if math.isfinite(z) else 0.0  # noqa: E731
    cdf = lambda z: 0.5 * math.erfc(-z / math.sqrt(2))  # noqa: E731
    c = [-2.5 + 5.0 * j / 15 for j in range(16)]
    for _ in range(20_000):
        b = [-math.inf] + [0.5 * (c[j] + c[j + 1]) for j in range(15)] + [math.inf]
        n = [(pdf(b[j]) - pdf(b[j + 1])) / (cdf(b[j + 1]) - cdf(b[j])) for j in range(16)]
        moved = max(abs(x - y) for x, y in zip(c, n))
        c = n
        if moved < 1e-16:
            break
    c = np.array([0.5 * (c[j] - c[15 - j]) for j in range(16)]) / 16.0   # symmetric about 0
    return c, 0.5 * (c[1:] + c[:-1])


CENTROIDS, BOUNDARIES = _codebook()
# share of a Gaussian coordinate's mass in each cell, as a 256-entry table byte -> index
_MASS = np.array([0.5 * math.erfc(-16.0 * b / math.sqrt(2)) for b in BOUNDARIES])
INDEX_OF_BYTE = np.searchsorted(_MASS, (np.arange(256) + 0.5) / 256).astype(np.uint8)


def _signs(seed):
    return np.random.default_rng([seed, 7]).integers(0, 2, D) * 2 - 1


def _rotation(signs, dtype):
    """R = H diag(signs) / 16 with the Sylvester Hadamard matrix H."""
    h = np.ones((1, 1))
    while h.shape[0] < D:
        h = np.block([[h, h], [h, -h]])
    return torch.from_numpy(h * signs[None, :] / 16.0).to("cuda", dtype)


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of eight requests: the smallest plan
        {"name": "plan_8_decode", "op": "plan", "n_req": 8, "chunks": 0, "chunk": 1, "max_past": 33_792, "pad": 0, "scarce": False},
        # a busy step: 256 requests, 24 of them prefilling; the free list runs out at the end
        {"name": "plan_256_mixed", "op": "plan", "n_req": 256, "chunks": 24, "chunk": 512, "max_past": 32_768, "pad": 61, "scarce": True},
        # a prefill burst of 64 requests over a long table
        {"name": "plan_64_prefill", "op": "plan", "n_req": 64, "chunks": 64, "chunk": 2048, "max_past": 212_992, "pad": 0, "scarce": False},
        # one decode step of eight requests at far positions
        {"name": "rope_8_decode", "op": "rope", "n_tok": 8, "pad": 0, "in": "bf16", "rot": 64, "axes": 1, "interleaved": False,
         "pairs": "halves", "k_out": False, "far": 229_376},
        # a prefill chunk with image tokens: three interleaved axes
        {"name": "rope_2048_3axes", "op": "rope", "n_tok": 2048, "pad": 0, "in": "bf16", "rot": 64, "axes": 3, "interleaved": True,
         "pairs": "halves", "k_out": True, "far": 34_816},
        # a large odd batch of fp32 projections with padded rows, adjacent pairs, three axes in blocks
        {"name": "rope_8191_f32", "op": "rope", "n_tok": 8191, "pad": 37, "in": "f32", "rot": 128, "axes": 3, "interleaved": False,
         "pairs": "adjacent", "k_out": True, "far": 65_536},
        # one request decoding with a window: latency
        {"name": "decode_1x32k_w4096", "op": "decode", "n_req": 1, "n_q": 1, "min_len": 32_768, "max_len": 32_768, "window": 4096,
         "sinks": 4, "out": "bf16", "empty": 0},
        # a batch of 64 ragged requests, two of them padding: throughput
        {"name": "decode_64_w4096", "op": "decode", "n_req": 64, "n_q": 1, "min_len": 300, "max_len": 32_768, "window": 4096,
         "sinks": 4, "out": "bf16", "empty": 2},
        # a verify step of four tokens per request, fp32 results
        {"name": "decode_16x4_w8192", "op": "decode", "n_req": 16, "n_q": 4, "min_len": 1000, "max_len": 65_536, "window": 8192,
         "sinks": 130, "out": "f32", "empty": 0},
        # a few short chunks: the smallest ragged call
        {"name": "ragged_5_short", "op": "ragged", "n_req": 5, "min_new": 1, "max_new": 65, "max_past": 2_000, "window": 1024,
         "sinks": 4, "out": "bf16", "pad": 3, "empty": 1},
        # one prefill chunk with a window
        {"name": "ragged_2k_on_32k_w4096", "op": "ragged", "n_req": 1, "min_new": 2048, "max_new": 2048, "max_past": 32_768, "window": 4096,
         "sinks": 4, "out": "bf16", "pad": 0, "empty": 0},
        # a mixed step without a window: chunks of 17 to 1,024 tokens over histories up to 16,384
        {"name": "ragged_8_mixed_full", "op": "ragged", "n_req": 8, "min_new": 17, "max_new": 1024, "max_past": 16_384, "window": NO_WINDOW,
         "sinks": 0, "out": "bf16", "pad": 0, "empty": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "decode", "decode", "ragged", "ragged"])
    if op == "plan":
        n = _log(rng, 1, 1024)
        return {"op": op, "n_req": n, "chunks": rng.randint(0, min(n, 64)), "chunk": _log(rng, 1, 2048), "max_past": _log(rng, 1, 65_536),
                "pad": rng.choice([0, rng.randint(1, 300)]), "scarce": rng.random() < 0.3}
    if op == "rope":
        n = _log(rng, 1, 8191)
        return {"op": op, "n_tok": n, "pad": rng.choice([0, rng.randint(0, n - 1)]) if n > 1 else 0, "in": rng.choice(["bf16", "bf16", "f32"]),
                "rot": 16 * rng.randint(1, 16), "axes": rng.choice([1, 2, 3]), "interleaved": rng.random() < 0.5,
                "pairs": rng.choice(["halves", "adjacent"]), "k_out": rng.random() < 0.6, "far": _log(rng, 16_384, 229_376)}
    if op == "decode":
        n, hi, window = _log(rng, 1, 64), _log(rng, 8, 32_768), _log(rng, 1, 4096)
        return {"op": op, "n_req": n, "n_q": rng.choice([1, 1, 2, 3, 4]) if n <= 32 else 1, "min_len": rng.randint(4, hi), "max_len": hi,
                "window": window, "sinks": rng.choice([0, 4, rng.randint(1, 300)]), "out": rng.choice(["bf16", "bf16", "f32"]),
                "empty": rng.choice([0, rng.randint(0, n - 1)]) if n > 1 else 0}
    n, hi = _log(rng, 1, 8), _log(rng, 1, 1024)
    return {"op": op, "n_req": n, "min_new": rng.randint(1, hi), "max_new": hi, "max_past": _log(rng, 1, 16_384),
            "window": rng.choice([_log(rng, 1, 4096), _log(rng, 64, 4096), NO_WINDOW]), "sinks": rng.choice([0, 4, rng.randint(1, 300)]),
            "out": rng.choice(["bf16", "bf16", "f32"]), "pad": rng.choice([0, rng.randint(1, 70)]),
            "empty": rng.choice([0, rng.randint(0, n - 1)]) if n > 1 else 0}


def _spread(n, lo, hi):
    """n whole numbers from lo to hi, spread over their logarithm (hi is always among them)."""
    if n == 1:
        return [hi]
    return [int(round(math.exp(math.log(lo + 1) + (math.log(hi + 1) - math.log(lo + 1)) * i / (n - 1)))) - 1 for i in range(n)]


def _plan_lens(case):
    """(past, new) per request: one new token each, the first `chunks` requests a chunk; every 16th is idle."""
    n = case["n_req"]
    past = _spread(n, 0, case["max_past"])
    past = past[::2] + past[1::2]
    chunk = _spread(max(case["chunks"], 1), 1, case["chunk"])
    new = [chunk[i] if i < case["chunks"] else 0 if i % 16 == 15 else 1 for i in range(n)]
    return past, new


def _decode_lens(case):
    n, e = case["n_req"], case["empty"]
    return _spread(n - e, max(case["min_len"], case["n_q"]), max(case["max_len"], case["n_q"])) + [0] * e


def _ragged_lens(case):
    n, e = case["n_req"], case["empty"]
    new = _spread(n - e, case["min_new"], case["max_new"])
    past = _spread(n - e, 0, case["max_past"])
    return past[::2] + past[1::2] + [0] * e, new + [0] * e


def _visible(end, window, sinks):
    """Positions that the query at `end` - 1 sees: its window and the sinks before it."""
    lo = max(0, end - window)
    return end - lo + min(sinks, lo)


def work(case):
    op = case["op"]
    if op == "plan":
        past, new = _plan_lens(case)
        tok = sum(new)
        fresh = sum(-(-(p + n) // PAGE) - -(-p // PAGE) for p, n in zip(past, new))
        # lengths in, offsets and lengths out, position and slot per token, each fresh page id read and written
        return {"bytes": len(past) * 16 + (tok + case["pad"]) * 12 + fresh * 8, "flops": 0}
    if op == "rope":
        n, size = case["n_tok"] - case["pad"], 2 if case["in"] == "bf16" else 4
        rows = 32 * D * size + H_Q * D * 2 + (H_KV * D * 2 if case["k_out"] else 0) + case["rot"] * 4 + 8 + 4 * case["axes"]
        # the projections in, q (and k) out, the packed vectors written, read back and returned
        return {"bytes": n * (rows + 2 * 8 * 130 + 2 * H_KV * D * size), "flops": n * 16 * D * 16}
    if op == "decode":
        lens, n_q, w, s = _decode_lens(case), case["n_q"], case["window"], case["sinks"]
        read = sum(_visible(t, w + n_q - 1, s) for t in lens)
        seen = sum(_visible(t - i, w, s) for t in lens if t for i in range(n_q))
        rows = len(lens) * n_q * H_Q * D
        return {"bytes": read * 1040 + rows * (2 + (2 if case["out"] == "bf16" else 4)), "flops": seen * H_Q * D * 4}
    past, new = _ragged_lens(case)
    w, s = case["window"], case["sinks"]
    read, seen = 0, 0
    for p, n in zip(past, new):
        if n:
            lo = max(0, p + 1 - w)
            read += max(0, p - lo) + min(s, lo, p)
            ends = np.arange(p + 1, p + n + 1)
            los = np.maximum(0, ends - w)
            seen += int((ends - los + np.minimum(s, los)).sum())
    rows = sum(new) * D
    return {"bytes": read * 1040 + rows * (H_Q * 2 + 2 * H_KV * 2 + H_Q * (2 if case["out"] == "bf16" else 4)), "flops": seen * H_Q * D * 4}


# ---------------------------------------------------------------- what a program has in hand
def _generator(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _pool(g, pages):
    """A pool of encoded Gaussian vectors: indices with their cells' masses, norms 16 s, s in [0.5, 2]."""
    pool = torch.empty((pages, PAGE_BYTES), dtype=torch.uint8, device="cuda")
    lut = torch.from_numpy(INDEX_OF_BYTE).cuda()
    for a in range(0, pages, 128):
        n = min(128, pages - a)
        r = lut[torch.randint(0, 256, (n, 262_144, 2), generator=g, device="cuda", dtype=torch.int32)]
        pool[a:a + n, :262_144] = r[..., 0] | (r[..., 1] << 4)
        norms = 16.0 * (0.5 + 1.5 * torch.rand((n, 2048), generator=g, device="cuda"))
        pool[a:a + n, 262_144:] = norms.half().view(torch.uint8)
    return pool.view(-1)


def _tables(rng, lens, cover=None):
    """A scattered page table for these lengths, -1 past each request's pages: (table [n_req][max_pages], pages used)."""
    need = [-(-t // PAGE) for t in lens]
    total = max(1, sum(need))
    ids = rng.permutation(total)
    tab = np.full((len(lens), max(1, max(cover or need))), -1, np.int32)
    at = 0
    for r, n in enumerate(need):
        tab[r, :n] = ids[at:at + n]
        at += n
    return tab, total


def _context(signs):
    if not own:
        return None
    from compressed_paged_kv_tq4_b200 import tq4
    return tq4.Context(signs)


def prepare(case, seed):
    rng, g, op = np.random.default_rng(seed), _generator(seed), case["op"]
    s = {"case": case, "ctx": _context(_signs(seed)), "seed": seed}
    if op == "plan":
        past, new = (np.array(x) for x in _plan_lens(case))
        order = rng.permutation(len(past))
        past, new = past[order], new[order]
        need = -(-(past + new) // PAGE)
        tab, used = _tables(rng, list(past), cover=list(need))
        fresh = int((need - -(-past // PAGE)).sum())
        free = max(1, int(fresh * 0.8) if case["scarce"] else fresh + 5)
        n_tok = int(new.sum()) + case["pad"]
        s |= {"past": _i32(past), "new": _i32(new), "tables": _i32(tab), "free": _i32(used + rng.permutation(free)), "pages": used + free,
              "n_tok": n_tok, "cu": _i32(np.zeros(len(past) + 1)), "lens": _i32(np.zeros(len(past))), "pos": _i32(np.zeros(n_tok)),
              "slot": torch.zeros(n_tok, dtype=torch.int64, device="cuda"), "taken": _i32([0])}
    elif op == "rope":
        n, dt, half, far = case["n_tok"], DTYPES[case["in"]], case["rot"] // 2, case["far"]
        live = n - case["pad"]
        qkv = torch.randn((n, (H_Q + 2 * H_KV) * D), generator=g, device="cuda")
        qkv *= 0.5 + 1.5 * torch.rand((n, 1), generator=g, device="cuda")
        qkv = qkv.to(dt)   # one projection's rows: q, k and v are slices of it
        freq = 1e6 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
        angle = torch.arange(far, dtype=torch.float64, device="cuda")[:, None] * freq
        p0 = int(rng.integers(0, far - n))
        pos = np.tile(p0 + np.arange(n), (case["axes"], 1))
        if case["axes"] > 1:   # a grid of image patches in the middle: time stands still, height and width run
            a, b = n // 4, n // 2
            side = max(1, int(math.sqrt(b - a)))
            for axis in range(case["axes"]):
                pos[axis, a:b] = p0 + a + (0 if axis == 0 else np.arange(b - a) // side if axis == 1 else np.arange(b - a) % side)
        pages = -(-n // PAGE) + 2
        start = int(rng.integers(0, PAGE))
        at = start + np.arange(n)
        slot = rng.permutation(pages)[at // PAGE].astype(np.int64) * PAGE + at % PAGE
        slot[live:] = -1
        third = half // 3
        s |= {"qkv": qkv, "table": torch.stack([angle.cos(), angle.sin()], -1).float().contiguous(), "pos": _i32(pos),
              "sections": {1: [half], 2: [half - half // 2, half // 2], 3: [half - 2 * third, third, third]}[case["axes"]],
              "slot": torch.from_numpy(slot).cuda(), "live": live, "pool": torch.zeros(pages * PAGE_BYTES, dtype=torch.uint8, device="cuda"),
              "q_out": torch.zeros((n, H_Q, D), dtype=torch.bfloat16, device="cuda"),
              "k_out": torch.zeros((n, H_KV, D), dtype=torch.bfloat16, device="cuda") if case["k_out"] else None}
        if not own:
            s |= {"R": _rotation(_signs(seed), torch.float64)}
    else:
        if op == "decode":
            lens = rng.permutation(_decode_lens(case))
            tab, pages = _tables(rng, list(lens))
            s |= {"q": torch.randn((len(lens), case["n_q"], H_Q, D), generator=g, device="cuda").bfloat16()}
        else:
            past, new = (np.array(x) for x in _ragged_lens(case))
            order = rng.permutation(len(past))
            past, new = past[order], new[order]
            lens, cu = past + new, np.concatenate([[0], np.cumsum(new)])
            tab, pages = _tables(rng, list(lens))
            n = int(cu[-1]) + case["pad"]
            s |= {"q": torch.randn((n, H_Q, D), generator=g, device="cuda").bfloat16(), "cu": _i32(cu),
                  "k": torch.randn((n, H_KV, D), generator=g, device="cuda").bfloat16(),
                  "v": torch.randn((n, H_KV, D), generator=g, device="cuda").bfloat16()}
        s |= {"lens": _i32(lens), "tables": _i32(tab), "pool": _pool(g, pages), "top": int(max(lens)),
              "out": torch.zeros(s["q"].shape, dtype=DTYPES[case["out"]], device="cuda")}
        if own and op == "decode":
            s["workspace"] = s["ctx"].decode_window_workspace(len(lens), case["n_q"], tab.shape[1], case["window"], case["sinks"])
        elif own:
            s["workspace"] = s["ctx"].prefill_ragged_workspace(len(lens), s["q"].shape[0], tab.shape[1], case["window"], case["sinks"])
        else:
            s["R"] = _rotation(_signs(seed), torch.float32)
    if not own:
        s |= {"c": torch.from_numpy(CENTROIDS).cuda(), "b": torch.from_numpy(BOUNDARIES).cuda()}
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    return {"plan": _plan, "rope": _rope, "decode": _decode, "ragged": _ragged}[s["case"]["op"]](s)


def _plan(s):
    if own:
        s["ctx"].plan_step(s["past"], s["new"], s["free"], s["tables"], s["pages"], cu_tok=s["cu"], seq_lens=s["lens"], tok_pos=s["pos"],
                           tok_slot=s["slot"], taken=s["taken"])
        return {"tables": s["tables"], "cu": s["cu"], "lens": s["lens"], "pos": s["pos"], "slot": s["slot"], "taken": s["taken"]}
    past, new, free, tab, n_tok = s["past"].long(), s["new"].long(), s["free"], s["tables"], s["n_tok"]
    has, need = (past + PAGE - 1) // PAGE, (past + new + PAGE - 1) // PAGE
    fresh = need - has
    start = fresh.cumsum(0) - fresh
    fits = (start + fresh <= free.numel()) | (fresh == 0)
    ends = new.cumsum(0)
    col = torch.arange(tab.shape[1], device="cuda")
    take = (start[:, None] + col - has[:, None]).clamp(0, free.numel() - 1)
    tables = torch.where((col >= has[:, None]) & (col < need[:, None]) & fits[:, None], free[take], tab)
    i = torch.arange(n_tok, device="cuda")
    r = torch.searchsorted(ends, i, right=True)
    live = i < ends[-1]
    r = r.clamp(max=past.numel() - 1)
    p = torch.where(live, past[r] + i - (ends - new)[r], 0)
    slot = torch.where(live & fits[r], tables[r, p // PAGE].long() * PAGE + p % PAGE, -1)
    return {"tables": tables, "cu": torch.cat([ends.new_zeros(1), ends]).int(), "lens": torch.where(fits, past + new, 0).int(), "pos": p.int(),
            "slot": slot, "taken": torch.where(fits, fresh, 0).sum().reshape(1).int()}


def _split(s):
    """q, k and v as slices of the projection's rows."""
    x = s["qkv"]
    n = x.shape[0]
    return (x[:, :H_Q * D].view(n, H_Q, D), x[:, H_Q * D:(H_Q + H_KV) * D].view(n, H_KV, D), x[:, (H_Q + H_KV) * D:].view(n, H_KV, D))


def _axis_of(case, sections):
    """The axis whose position turns each frequency: sections in blocks, or dealt out in turn."""
    half = case["rot"] // 2
    if not case["interleaved"]:
        return np.repeat(np.arange(len(sections)), sections)
    i, k = np.arange(half), len(sections)
    axis = np.zeros(half, np.int64)
    for a in range(1, k):
        axis[(i % k == a) & (i < k * sections[a])] = a
    return axis


def _turn(x, cos, sin, case):
    """Rotate the first `rot` dims of x [n][heads][256] by the angles [n][rot / 2]."""
    rot, half = case["rot"], case["rot"] // 2
    cos, sin = cos[:, None, :], sin[:, None, :]
    if case["pairs"] == "halves":
        a, b = x[..., :half], x[..., half:rot]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], -1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., rot:]], -1)


def _half(x):
    """64-bit values to the nearest fp16 in one rounding (a cast goes through 32 bits)."""
    h = x.half()
    around = torch.stack([h, (h.view(torch.int16) - 1).clamp(min=0).view(torch.float16), (h.view(torch.int16) + 1).view(torch.float16)])
    off = (around.double() - x).abs()
    odd = (around.view(torch.int16) & 1).double()
    best = (off[1:] < off[:1]) | ((off[1:] == off[:1]) & (odd[1:] < odd[:1]))
    return torch.where(best[0], around[1], torch.where(best[1], around[2], h))


def _rope(s):
    case, pool, slot, n = s["case"], s["pool"], s["slot"], s["live"]
    q, k, v = _split(s)
    if own:
        s["ctx"].rope_append(pool, q, k, v, s["pos"], s["table"], slot, sections=s["sections"], interleaved=case["interleaved"],
                             pairs=case["pairs"], q_out=s["q_out"], k_out=s["k_out"])
        kh, vh = s["ctx"].reconstruct_slots(pool, slot, out_dtype=DTYPES[case["in"]])
        return {"q": s["q_out"], "k": s["k_out"], "k_hat": kh, "v_hat": vh}
    axis = torch.from_numpy(_axis_of(case, s["sections"])).to("cuda")
    angle = s["table"][s["pos"][axis].T.long(), torch.arange(case["rot"] // 2, device="cuda")]
    cos, sin = angle[:n, :, 0], angle[:n, :, 1]
    s["q_out"][:n] = _turn(q[:n].float(), cos, sin, case).bfloat16()
    x = torch.stack([_turn(k[:n].double(), cos.double(), sin.double(), case), v[:n].double()], 1)   # [n][2][4][256], next to borders: 64 bits
    if s["k_out"] is not None:
        s["k_out"][:n] = x[:, 0].float().bfloat16()
    norm = x.square().sum(-1, keepdim=True).sqrt()
    y = (x / norm.clamp(min=1e-300)) @ s["R"].T
    index = torch.bucketize(y, s["b"]) * (norm > 0)
    norm = _half(norm[..., 0])
    shift = 4 * torch.arange(8, device="cuda")
    words = (index.view(n, 2, H_KV, 32, 8) << shift).sum(-1)
    words = torch.where(words >= 1 << 31, words - (1 << 32), words).int()
    page, off = slot[:n, None, None] // PAGE, slot[:n, None, None] % PAGE
    kv, head = torch.arange(2, device="cuda")[:, None], torch.arange(H_KV, device="cuda")
    pool.view(torch.int32).view(-1, PAGE_WORDS)[:, :65_536].view(-1, 2, H_KV, PAGE, 32)[page, kv, head, off] = words
    pool.view(torch.float16).view(-1, PAGE_HALVES)[:, 131_072:].view(-1, 2, H_KV, PAGE)[page, kv, head, off] = norm
    hat = (norm.float()[..., None] * (s["c"].float()[index] @ s["R"].float())).to(DTYPES[case["in"]])
    full = hat.new_zeros((2, case["n_tok"], H_KV, D))
    full[:, :n] = hat.transpose(0, 1)
    return {"q": s["q_out"], "k": s["k_out"], "k_hat": full[0], "v_hat": full[1]}


def _stored(s, pos):
    """The vectors that stand at positions pos [n_req][P] of each request: two tensors [n_req][P][4][256]."""
    pool, tab = s["pool"], s["tables"].long()
    page = tab.gather(1, (pos // PAGE).clamp(0, tab.shape[1] - 1)).clamp(min=0)[..., None]
    off, head = (pos % PAGE)[..., None], torch.arange(H_KV, device="cuda")
    words = pool.view(torch.int32).view(-1, PAGE_WORDS)[:, :65_536].view(-1, 2, H_KV, PAGE, 32)
    norms = pool.view(torch.float16).view(-1, PAGE_HALVES)[:, 131_072:].view(-1, 2, H_KV, PAGE)
    shift = 4 * torch.arange(8, device="cuda", dtype=torch.int32)
    c = s["c"].float()

    def one(kv):
        index = (words[page, kv, head, off][..., None] >> shift) & 15
        return norms[page, kv, head, off].float()[..., None] * (c[index].flatten(-2) @ s["R"])

    return one(0), one(1)


def _attend(q, k, v, ok):
    """softmax(q k / 16) v in 32 bits: q [r][n][24][256], k, v [r][P][4][256], ok [r][n][P]; rows that see nothing are 0."""
    r, n = q.shape[:2]
    q = q.float().view(r, n, H_KV, GROUP, D).permute(0, 2, 3, 1, 4).reshape(r, H_KV, GROUP * n, D)
    x = q @ k.permute(0, 2, 3, 1) * SCALE
    x = x.view(r, H_KV, GROUP, n, -1).masked_fill_(~ok[:, None, None], -math.inf)
    x = (x - x.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    total = x.sum(-1)
    o = (x.view(r, H_KV, GROUP * n, -1) @ v.permute(0, 2, 1, 3)).view(r, H_KV, GROUP, n, D)
    o = o / total.clamp(min=1e-30)[..., None]
    return o.permute(0, 3, 1, 2, 4).reshape(r, n, H_Q, D)


def _span(s, first, top_new):
    """The positions that the tokens [first, length) of each request may see, sinks first: (pos [n_req][P], usable)."""
    case = s["case"]
    width = min(s["top"], case["window"] + top_new - 1)
    sinks = min(case["sinks"], s["top"])
    lo = (first - case["window"] + 1).clamp(min=0)[:, None]
    head = torch.arange(sinks, device="cuda").expand(lo.shape[0], -1)
    body = lo + torch.arange(width, device="cuda")
    return torch.cat([head, body], 1), torch.cat([head < lo, body < s["lens"].long()[:, None]], 1)


def _decode(s):
    case, n_q = s["case"], s["case"]["n_q"]
    if own:
        return s["ctx"].decode_attention_window(s["pool"], s["q"], s["tables"], s["lens"], case["window"], case["sinks"], SCALE, out=s["out"],
                                                workspace=s["workspace"])
    first = s["lens"].long() - n_q
    pos, usable = _span(s, first, n_q)
    k, v = _stored(s, pos)
    at = (first[:, None] + torch.arange(n_q, device="cuda"))[..., None]   # [n_req][n_q][1]
    ok = usable[:, None] & (pos[:, None] <= at) & ((pos[:, None] > at - case["window"]) | (pos[:, None] < case["sinks"]))
    return _attend(s["q"], k, v, ok).to(DTYPES[case["out"]])


def _ragged(s):
    case = s["case"]
    if own:
        return s["ctx"].prefill_attention_ragged(s["pool"], s["q"], s["k"], s["v"], s["cu"], s["lens"], s["tables"], case["window"],
                                                 case["sinks"], SCALE, out=s["out"], workspace=s["workspace"])
    cu, top = s["cu"].long(), case["max_new"]
    new = cu[1:] - cu[:-1]
    first = s["lens"].long() - new
    pos, usable = _span(s, first, top)
    k, v = _stored(s, pos)
    rows = s["q"].shape[0]
    own_row = (cu[:-1, None] + pos - first[:, None]).clamp(0, rows - 1)
    fresh = (pos >= first[:, None])[..., None, None]
    k, v = torch.where(fresh, s["k"][own_row].float(), k), torch.where(fresh, s["v"][own_row].float(), v)
    i = torch.arange(top, device="cuda")
    at = (first[:, None] + i)[..., None]
    ok = usable[:, None] & (pos[:, None] <= at) & ((pos[:, None] > at - case["window"]) | (pos[:, None] < case["sinks"]))
    o = _attend(s["q"][(cu[:-1, None] + i).clamp(0, rows - 1)], k, v, ok)
    j = torch.arange(rows, device="cuda")
    r = torch.searchsorted(cu[1:], j, right=True).clamp(max=new.numel() - 1)
    live = (j < cu[-1])[:, None, None]
    return torch.where(live, o[r, (j - cu[r]).clamp(0, top - 1)], 0).to(DTYPES[case["out"]])


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    if case["op"] == "plan":
        return None   # whole numbers only
    global own
    mine, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = mine
    rot = _rotation(_signs(seed), torch.float64)
    c = s["c"]
    if case["op"] == "rope":
        return _exact_rope(s, rot, c)
    words = s["pool"].view(torch.int32).view(-1, PAGE_WORDS)
    norms = s["pool"].view(torch.float16).view(-1, PAGE_HALVES).double()
    lens, tab = s["lens"].tolist(), s["tables"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for r, t in enumerate(lens):
        if t == 0:
            continue
        n_new = case["n_q"] if case["op"] == "decode" else int(s["cu"][r + 1] - s["cu"][r])
        if n_new == 0:
            continue
        pages = torch.tensor(tab[r][:-(-t // PAGE)], device="cuda")
        lo = max(0, t - n_new - case["window"] + 1)
        keep = torch.cat([torch.arange(min(case["sinks"], lo), device="cuda"), torch.arange(lo, t, device="cuda")])
        page, off = pages[keep // PAGE], keep % PAGE
        kv = []
        for side in range(2):
            x = torch.empty((keep.numel(), H_KV, D), dtype=torch.float64, device="cuda")
            for h in range(H_KV):
                w = words.view(words.shape[0], -1)[page[:, None], side * 32_768 + h * 8_192 + off[:, None] * 32 + torch.arange(32, device="cuda")].long()
                for e in range(8):
                    x[:, h, e::8] = c[(w >> (4 * e)) & 15]
                x[:, h] *= norms[page, 131_072 + side * 1024 + h * PAGE + off][:, None]
            kv.append(x @ rot)
        if case["op"] == "ragged":
            a = int(s["cu"][r])
            tail = keep >= t - n_new
            kv[0][tail], kv[1][tail] = s["k"][a:a + n_new].double()[keep[tail] - t + n_new], s["v"][a:a + n_new].double()[keep[tail] - t + n_new]
            q, dst = s["q"][a:a + n_new].double(), out[a:a + n_new]
        else:
            q, dst = s["q"][r].double(), out[r]
        at = torch.arange(t - n_new, t, device="cuda")[:, None]
        see = (keep <= at) & ((keep > at - case["window"]) | (keep < case["sinks"]))
        for h in range(H_Q):
            x = (q[:, h] @ kv[0][:, h // GROUP].T * SCALE).masked_fill(~see, -math.inf)
            dst[:, h] = torch.nan_to_num(torch.softmax(x, -1)) @ kv[1][:, h // GROUP]
    return out


def _exact_rope(s, rot, c):
    case, n, half = s["case"], s["live"], s["case"]["rot"] // 2
    x = s["qkv"].double().view(case["n_tok"], H_Q + 2 * H_KV, D)[:n].clone()
    axis = _axis_of(case, s["sections"])
    for i in range(half):
        a, b = (i, i + half) if case["pairs"] == "halves" else (2 * i, 2 * i + 1)
        cs = s["table"][s["pos"][int(axis[i]), :n].long(), i].double()
        lo, hi = x[:, :H_Q + H_KV, a].clone(), x[:, :H_Q + H_KV, b].clone()
        x[:, :H_Q + H_KV, a] = lo * cs[:, :1] - hi * cs[:, 1:]
        x[:, :H_Q + H_KV, b] = hi * cs[:, :1] + lo * cs[:, 1:]
    pad = lambda t: torch.cat([t, t.new_zeros((case["pad"],) + t.shape[1:])])  # noqa: E731
    hats = []
    for kv in (x[:, H_Q:H_Q + H_KV], x[:, H_Q + H_KV:]):
        norm = torch.linalg.vector_norm(kv, dim=-1, keepdim=True)
        y = torch.nan_to_num(kv / norm) @ rot.T
        index = (y[..., None] > s["b"]).sum(-1)
        hats.append(pad(_half(norm).double() * (c[index * (norm > 0)] @ rot)))
    return {"q": pad(x[:, :H_Q]), "k": pad(x[:, H_Q:H_Q + H_KV]) if case["k_out"] else None, "k_hat": hats[0], "v_hat": hats[1]}
