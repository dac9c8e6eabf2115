"""The operators around the top-k of a sparse-attention indexer, as cases to be measured.

Rotary positions of queries and keys, quantising rows to e4m3 with a scale for each
block of 128 columns (on their own, or as they are written into a paged cache),
reading a cache back at selected slots, and the indexer's scores over the paged
8-bit cache. ``run`` computes them in plain torch, or (``own``) with the
framework's entry points; ``exact`` from their definitions in 64 bits.
"""

import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -64
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of 48 sequences: the indexer's query heads, half of each head rotated
        {"name": "rotary_decode", "op": "rotary", "tokens": 48, "heads": 64, "dim": 128, "rot": 64,
         "start": 64, "layout": "half", "dtype": "bf16", "far": 262144, "factor": 4.0, "train": False},
        # a training step on a prompt of odd length: forward and the gradient, whole head, interleaved
        {"name": "rotary_train", "op": "rotary", "tokens": 8191, "heads": 64, "dim": 128, "rot": 128,
         "start": 0, "layout": "interleaved", "dtype": "bf16", "far": 8191, "factor": 1.0, "train": True},
        # the same in 32 bits over one shared key head, part of a wider row, far positions
        {"name": "rotary_key_fp32", "op": "rotary", "tokens": 32768, "heads": 1, "dim": 192, "rot": 64,
         "start": 128, "layout": "interleaved", "dtype": "fp32", "far": 1048576, "factor": 40.0, "train": True},
        # queries of a decode step, their scales folded into the heads' weights
        {"name": "quantise_decode", "op": "quantise", "tokens": 48, "heads": 64, "dim": 128,
         "dtype": "bf16", "format": "fp32", "fold": True},
        # queries of a prompt chunk
        {"name": "quantise_prompt", "op": "quantise", "tokens": 8192, "heads": 64, "dim": 128,
         "dtype": "bf16", "format": "fp32", "fold": True},
        # the keys of one decode step of 256 sequences
        {"name": "write_decode", "op": "write", "tokens": 256, "dim": 128, "page_size": 64,
         "dtype": "bf16", "format": "pow2"},
        # a long prompt's wide rows (four whole blocks and a half one), some tokens without a slot
        {"name": "write_prompt_wide", "op": "write", "tokens": 65535, "dim": 576, "page_size": 64,
         "dtype": "bf16", "format": "fp32"},
        # what the selection of one row picked
        {"name": "read_one_row", "op": "read", "rows": 1, "k": 1024, "dim": 128, "page_size": 64,
         "pool": 32768, "dtype": "bf16"},
        # what the selections of 256 rows picked, wide rows
        {"name": "read_wide", "op": "read", "rows": 256, "k": 2048, "dim": 512, "page_size": 64,
         "pool": 2097152, "dtype": "bf16"},
        # one sequence's decode step, the shortest context of the unit test
        {"name": "scores_b1_n2048", "op": "scores", "batch": 1, "queries": 1, "heads": 64,
         "row_len": 2048, "page_size": 64, "ragged": False},
        # the decode sweep's largest batch at 128k context, 4x compressed
        {"name": "scores_b256_n32768", "op": "scores", "batch": 256, "queries": 1, "heads": 64,
         "row_len": 32768, "page_size": 64, "ragged": False},
        # a chunk of a prompt, each query seeing the keys up to its own
        {"name": "scores_prompt", "op": "scores", "batch": 1, "queries": 2048, "heads": 64,
         "row_len": 32768, "page_size": 64, "ragged": False},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["rotary", "quantise", "write", "read", "scores", "scores"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "rotary":
        dim = rng.choice([64, 80, 128, 128, 192, 576])
        rot = rng.choice([dim, 64, 32, 2 * rng.randint(1, dim // 2)])
        rot = min(rot, dim)
        heads = rng.choice([1, 2, 7, 32, 64, 128])
        tokens = _log(rng, 1, max(1, min(65536, (1 << 26) // (heads * dim))))
        return {"op": op, "tokens": tokens, "heads": heads, "dim": dim, "rot": rot,
                "start": rng.choice([0, dim - rot]), "layout": rng.choice(["half", "interleaved"]),
                "dtype": dtype, "far": _log(rng, 1024, 1 << 20), "factor": rng.choice([1.0, 4.0, 40.0]),
                "train": rng.random() < 0.5}
    if op == "quantise":
        dim = rng.choice([128, 128, 128, 512, 576, 200, 63])
        heads = rng.choice([1, 8, 64, 33])
        tokens = _log(rng, 1, max(1, min(16384, (1 << 26) // (heads * dim))))
        return {"op": op, "tokens": tokens, "heads": heads, "dim": dim, "dtype": dtype,
                "format": rng.choice(["fp32", "pow2"]), "fold": dim <= BLOCK and rng.random() < 0.5}
    if op == "write":
        dim = rng.choice([128, 128, 512, 576, 200])
        return {"op": op, "tokens": _log(rng, 1, 65536), "dim": dim,
                "page_size": rng.choice([1, 16, 64, 128, 48]), "dtype": dtype,
                "format": rng.choice(["fp32", "pow2"])}
    if op == "read":
        dim = rng.choice([128, 128, 512, 576, 200])
        return {"op": op, "rows": _log(rng, 1, 256), "k": rng.choice([1, 64, 500, 1024, 2048]), "dim": dim,
                "page_size": rng.choice([1, 16, 64, 128, 48]), "pool": _log(rng, 4096, 1 << 20),
                "dtype": dtype}
    heads = rng.choice([64, 64, 32, 8, 24, 1, 128])
    queries = rng.choice([1, 1, 2, 4, 7, _log(rng, 16, 1024)])
    row_len = _log(rng, 1, 262144)
    most = min((1 << 32) // (queries * heads * row_len), (1 << 23) // row_len)
    return {"op": "scores", "batch": _log(rng, 1, max(1, min(256, most))), "queries": queries, "heads": heads,
            "row_len": row_len, "page_size": rng.choice([64, 64, 64, 128, 16, 1, 48]),
            "ragged": rng.random() < 0.6}


def work(case):
    op = case["op"]
    if op == "rotary":
        size = 4 if case["dtype"] == "fp32" else 2
        n = case["tokens"] * case["heads"] * case["dim"]
        passes = 2 if case["train"] else 1
        return {"bytes": passes * (2 * n * size + case["tokens"] * 4),
                "flops": passes * 3 * case["tokens"] * case["heads"] * case["rot"]}
    if op in ("quantise", "write"):
        size = 4 if case["dtype"] == "fp32" else 2
        rows = case["tokens"] * case.get("heads", 1)
        blocks = -(-case["dim"] // BLOCK)
        return {"bytes": rows * (case["dim"] * (size + 1) + 4 * blocks + 4 * (op == "write" or case["fold"])),
                "flops": rows * case["dim"] * 2}
    if op == "read":
        size = 4 if case["dtype"] == "fp32" else 2
        rows = case["rows"] * case["k"]
        return {"bytes": rows * (case["dim"] * (size + 1) + 4 * -(-case["dim"] // BLOCK) + 4),
                "flops": rows * case["dim"]}
    seen, cached = _seen(case)
    rows = case["batch"] * case["queries"]
    return {"bytes": cached * (BLOCK + 4) + rows * case["heads"] * (BLOCK + 4) + rows * case["row_len"] * 4
            + case["batch"] * 4 * -(-case["row_len"] // case["page_size"]),
            "flops": seen * case["heads"] * (2 * BLOCK + 3)}


def _seen(case):
    """(query, key) pairs scored, and keys read: of a ragged case, what its lengths' distribution expects."""
    b, n, w = case["batch"], case["queries"], case["row_len"]
    if case["ragged"]:
        return b * n * (w + 1) // 2, b * (w + 1) // 2
    return b * sum(max(0, w - n + 1 + i) for i in range(n)), b * w


# ------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _frequencies(case):
    """Radians per position of each pair; past factor 1, the slow pairs are slowed down by it
    and those between are blended, as for a context longer than the trained one."""
    rot = case["rot"]
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = 10000.0 ** (-2.0 * i / rot)
    if case["factor"] > 1.0:
        turns = 4096.0 * f / (2.0 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        f = f * keep + f / case["factor"] * (1.0 - keep)
    return f.cuda()


def _activations(g, shape, dtype):
    """Normal values whose rows differ in size, a few of them with outlying columns."""
    x = torch.randn(shape, generator=g, device="cuda")
    x = x * torch.exp2(torch.randint(-3, 4, shape[:-1] + (1,), generator=g, device="cuda").float())
    x[..., :: 61] *= 8.0
    return x.to(DTYPES[dtype])


def _cache(g, pages, page_size, dim):
    """A cache as it stands after many writes: codes over the whole range of e4m3, a scale for each block."""
    codes = torch.empty((pages, page_size, dim), dtype=torch.float8_e4m3fn, device="cuda")
    flat = codes.view(torch.uint8).view(-1)
    step = 1 << 28
    for at in range(0, flat.numel(), step):
        part = flat[at:at + step]
        part.copy_((torch.randn(part.numel(), generator=g, device="cuda") * 100.0).clamp(-448.0, 448.0)
                   .to(torch.float8_e4m3fn).view(torch.uint8))
    scales = torch.rand((pages, page_size, -(-dim // BLOCK)), generator=g, device="cuda") * 0.02 + 0.001
    return codes, scales


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    s = dict(case)
    if op == "rotary":
        shape = (case["tokens"], case["heads"], case["dim"])
        s["x"] = torch.randn(shape, generator=g, device="cuda").to(DTYPES[case["dtype"]])
        top = max(case["far"], 1)
        s["positions"] = torch.randint(0, top, (case["tokens"],), generator=g, device="cuda", dtype=torch.int32)
        s["freqs"] = _frequencies(case)
        s["scale"] = 0.1 * math.log(case["factor"]) + 1.0
        if case["train"]:
            s["x"].requires_grad_(True)
            s["grad"] = torch.randn(shape, generator=g, device="cuda").to(DTYPES[case["dtype"]])
    elif op == "quantise":
        s["x"] = _activations(g, (case["tokens"], case["heads"], case["dim"]), case["dtype"])
        s["weights"] = (torch.randn((case["tokens"], case["heads"]), generator=g, device="cuda")
                        * case["heads"] ** -0.5 if case["fold"] else None)
    elif op == "write":
        s["x"] = _activations(g, (case["tokens"], case["dim"]), case["dtype"])
        pages = -(-case["tokens"] * 5 // (4 * case["page_size"])) + 1
        s["codes"], s["scales"] = _cache(g, pages, case["page_size"], case["dim"])
        s["slots"] = torch.randperm(pages * case["page_size"], generator=g, device="cuda")[:case["tokens"]].int()
        s["slots"][13::97] = -1
    elif op == "read":
        pages = -(-case["pool"] // case["page_size"])
        s["codes"], s["scales"] = _cache(g, pages, case["page_size"], case["dim"])
        shape = (case["rows"], case["k"])
        s["slots"] = torch.randint(0, pages * case["page_size"], shape, generator=g, device="cuda", dtype=torch.int32)
        if case["rows"] > 1:  # rows shorter than k end in -1
            short = torch.randint(1, 8 * case["k"], (case["rows"], 1), generator=g, device="cuda")
            s["slots"][torch.arange(case["k"], device="cuda")[None, :] >= short] = -1
    else:
        b, n, h, w, ps = (case[k] for k in ("batch", "queries", "heads", "row_len", "page_size"))
        pages = -(-w // ps)
        s["codes"], s["scales"] = _cache(g, b * pages, ps, BLOCK)
        s["page_table"] = torch.randperm(b * pages, generator=g, device="cuda").view(b, pages).int()
        s["q"] = (torch.randn((b, n, h, BLOCK), generator=g, device="cuda") * 100.0).clamp(-448.0, 448.0).to(
            torch.float8_e4m3fn)
        s["weights"] = torch.randn((b, n, h), generator=g, device="cuda") * (0.01 * (h * BLOCK) ** -0.5)
        last = (torch.randint(1, w + 1, (b, 1), generator=g, device="cuda") if case["ragged"]
                else torch.full((b, 1), w, device="cuda"))
        # the last of a sequence's queries sees all of its keys, each one before it one fewer
        s["seq_lens"] = (last - (n - 1) + torch.arange(n, device="cuda")[None, :]).clamp(min=0).int()
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return _run_own(s) if own else _PLAIN[s["op"]](s)


def _run_own(s):
    import sparse_attention_indexer_sm_gb300 as fw
    op = s["op"]
    if op == "rotary":
        y = fw.indexer_rotary(s["x"], s["positions"], s["freqs"], layout=s["layout"], start=s["start"],
                              scale=s["scale"])
        if not s["train"]:
            return y
        return {"out": y.detach(), "grad": torch.autograd.grad(y, s["x"], s["grad"])[0]}
    if op == "quantise":
        codes, scales = fw.indexer_quantise(s["x"], scale_format=s["format"], weights=s["weights"])
        return {"codes": codes, "scales": scales}
    if op == "write":
        fw.indexer_cache_write(s["x"], s["slots"], s["codes"], s["scales"], scale_format=s["format"])
        return {"codes": s["codes"], "scales": s["scales"]}
    if op == "read":
        return fw.indexer_cache_read(s["codes"], s["scales"], s["slots"], dtype=DTYPES[s["dtype"]])
    return fw.indexer_scores(s["q"], s["weights"], s["codes"], s["scales"], s["page_table"], s["seq_lens"],
                             s["row_len"])


def _pairs(x, s):
    r = x[..., s["start"]:s["start"] + s["rot"]]
    if s["layout"] == "half":
        return r[..., :s["rot"] // 2], r[..., s["rot"] // 2:]
    return r[..., 0::2], r[..., 1::2]


def _rotate(x, s, sign):
    angle = s["positions"].double()[:, None, None] * s["freqs"]
    c, d = (angle.cos() * s["scale"]).float(), (angle.sin() * (sign * s["scale"])).float()
    a, b = _pairs(x.float(), s)
    y = x.clone()
    u, v = _pairs(y, s)
    u.copy_(a * c - b * d)
    v.copy_(a * d + b * c)
    return y


def _plain_rotary(s):
    x = s["x"].detach()
    y = _rotate(x, s, 1.0)
    return {"out": y, "grad": _rotate(s["grad"], s, -1.0)} if s["train"] else y


def _blocks(x):
    pad = -x.shape[-1] % BLOCK
    x = torch.nn.functional.pad(x, (0, pad)) if pad else x
    return x.view(x.shape[:-1] + (-1, BLOCK))


def _power(e):
    """2**e in 64 bits, exactly: e goes into the exponent's bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _quantised(x, how):
    dim = x.shape[-1]
    x = _blocks(x.float())
    amax = x.abs().amax(-1).clamp(min=AMAX_FLOOR)
    if how == "pow2":
        m, e = torch.frexp(amax)
        scale = _power(torch.where(m <= 0.875, e - 9, e - 8)).float()
    else:
        scale = (amax.double() / E4M3_MAX).float()  # in 64 bits: an ulp of it moves values across a border
    y = x.double() / scale.double()[..., None]
    step = _power(torch.frexp(y)[1].clamp(min=-5) - 4)
    y = (torch.round(y / step) * step).float().to(torch.float8_e4m3fn)
    return y.flatten(-2)[..., :dim], scale


def _plain_quantise(s):
    codes, scale = _quantised(s["x"], s["format"])
    if s["fold"]:
        scale = scale[..., 0] * s["weights"]
    return {"codes": codes.contiguous(), "scales": scale}


def _plain_write(s):
    codes, scale = _quantised(s["x"], s["format"])
    keep = s["slots"] >= 0
    at = s["slots"][keep].long()
    dim = codes.shape[-1]
    s["codes"].view(torch.uint8).view(-1, dim)[at] = codes.view(torch.uint8)[keep]
    s["scales"].view(-1, scale.shape[-1])[at] = scale[keep]
    return {"codes": s["codes"], "scales": s["scales"]}


def _plain_read(s):
    dim = s["codes"].shape[-1]
    at = s["slots"].clamp(min=0).long()
    x = s["codes"].view(torch.uint8).view(-1, dim)[at].view(torch.float8_e4m3fn).float()
    f = s["scales"].view(-1, s["scales"].shape[-1])[at].repeat_interleave(BLOCK, -1)[..., :dim]
    x = torch.where((s["slots"] >= 0)[..., None], x * f, torch.zeros((), device=x.device))
    return x.to(DTYPES[s["dtype"]])


def _plain_scores(s):
    b, n, h, w = s["batch"], s["queries"], s["heads"], s["row_len"]
    at = (s["page_table"].long()[:, :, None] * s["page_size"]
          + torch.arange(s["page_size"], device="cuda")).flatten(1)[:, :w]
    keys = s["codes"].view(torch.uint8).view(-1, BLOCK)[at].view(torch.float8_e4m3fn).float()
    dots = torch.bmm(s["q"].float().view(b, n * h, BLOCK), keys.transpose(1, 2)).relu_()
    y = torch.bmm(s["weights"].view(b * n, 1, h), dots.view(b * n, h, w)).view(b, n, w)
    y = y * s["scales"].view(-1)[at][:, None, :]
    seen = torch.arange(w, device="cuda") < s["seq_lens"][:, :, None]
    return torch.where(seen, y, -math.inf).view(b * n, w)


_PLAIN = {"rotary": _plain_rotary, "quantise": _plain_quantise, "write": _plain_write, "read": _plain_read,
          "scores": _plain_scores}


# ------------------------------------------------------------------ from the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rotary":
        y = _exact_rotary(s["x"].detach(), s, 1)
        return {"out": y, "grad": _exact_rotary(s["grad"], s, -1)} if case["train"] else y
    if op in ("quantise", "write"):
        codes, scales = _exact_quantised(s["x"], case["format"])
        if op == "quantise":
            return {"codes": codes, "scales": scales[..., 0] * s["weights"].double() if case["fold"] else scales}
        c = s["codes"].float().double().view(-1, case["dim"])
        f = s["scales"].double().view(-1, scales.shape[-1])
        for slots, row, scale in zip(s["slots"].split(4096), codes.split(4096), scales.split(4096)):
            here = (slots >= 0).nonzero()[:, 0]
            c.index_copy_(0, slots[here].long(), row[here])
            f.index_copy_(0, slots[here].long(), scale[here])
        return {"codes": c.view(s["codes"].shape), "scales": f.view(s["scales"].shape)}
    if op == "read":
        flat = s["slots"].view(-1)
        y = torch.zeros((flat.numel(), case["dim"]), dtype=torch.float64, device="cuda")
        c, f = s["codes"].view(torch.uint8).view(-1, case["dim"]), s["scales"].view(-1, s["scales"].shape[-1])
        i = (flat >= 0).nonzero()[:, 0]
        j = flat[i].long()
        for k in range(f.shape[-1]):
            part = slice(k * BLOCK, min((k + 1) * BLOCK, case["dim"]))
            y[i, part] = c[j, part].view(torch.float8_e4m3fn).float().double() * f[j, k, None].double()
        return y.view(s["slots"].shape + (case["dim"],))
    return _exact_scores(s)


def _exact_rotary(x, s, sign):
    y = x.double()
    turns = torch.remainder(s["positions"].double()[:, None] * s["freqs"], 2.0 * math.pi)
    by = torch.polar(torch.full_like(turns, s["scale"]), sign * turns)[:, None, :]
    i = torch.arange(s["rot"] // 2, device="cuda")
    first = s["start"] + (i if s["layout"] == "half" else 2 * i)
    second = first + (s["rot"] // 2 if s["layout"] == "half" else 1)
    z = torch.complex(y[..., first], y[..., second]) * by
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_quantised(x, how):
    dim = x.shape[-1]
    grid = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).float().double()
    between = (grid[1:] + grid[:-1]) / 2
    codes = torch.empty(x.shape, dtype=torch.float64, device="cuda")
    scales = []
    for at in range(0, dim, BLOCK):
        v = x[..., at:at + BLOCK].double()
        top = v.abs().amax(-1).clamp(min=AMAX_FLOOR)
        if how == "pow2":
            powers = torch.tensor([2.0 ** k for k in range(-80, 124)], dtype=torch.float64, device="cuda")
            scale = powers[torch.searchsorted(powers * E4M3_MAX, top)]
        else:
            scale = (top / E4M3_MAX).float().double()  # the stored scale is a 32-bit number
        y = v.abs() / scale[..., None]
        i = torch.bucketize(y, between)
        tie = (y == between[i.clamp(max=125)]) & (i % 2 == 1) & (i < 126)
        codes[..., at:at + BLOCK] = torch.copysign(grid[i + tie.long()], v)
        scales.append(scale)
    return codes, torch.stack(scales, -1)


def _exact_scores(s):
    b, n, h, w = s["batch"], s["queries"], s["heads"], s["row_len"]
    flat, scale = s["codes"].view(torch.uint8).view(-1, BLOCK), s["scales"].view(-1).double()
    j = torch.arange(w, device="cuda")
    y = torch.full((b, n, w), -math.inf, dtype=torch.float64, device="cuda")
    few = max(1, (1 << 28) // (h * w))
    for i in range(b):
        slot = s["page_table"][i, j // s["page_size"]].long() * s["page_size"] + j % s["page_size"]
        keys = flat[slot].view(torch.float8_e4m3fn).float().double() * scale[slot, None]
        for at in range(0, n, few):
            q = s["q"][i, at:at + few].float().double()
            dots = torch.einsum("qhd,jd->qhj", q, keys)
            part = (dots.clamp(min=0.0) * s["weights"][i, at:at + few].double()[:, :, None]).sum(1)
            part[j[None, :] >= s["seq_lens"][i, at:at + few, None]] = -math.inf
            y[i, at:at + few] = part
    return y.view(b * n, w)
