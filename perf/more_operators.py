"""Workloads of the operators that carry a step's activations into and out of the paged cache,
with their plain forms.

Three families, each as a model runner calls it within one layer of a step:

* ``append`` - this step's queries and keys are rotated by their positions and keys and values
  appended to the paged cache, in 16 bits or (``"bits": 4``) in 4 bits with a scale for every 16
  values, whose rows are then read back;
* ``attention`` - causal attention of a mixed batch over a paged cache held in 4 bits;
* ``norm`` - the residual's addition and the root-mean-square norm, with an output in 16 bits or
  in 8 bits with scales.

``own`` selects the library's kernels; otherwise ``run`` computes the same with elementary
torch operations in 32 bits.

A page of the 4-bit cache holds, for each kv head, 16 tokens of ``hd`` values: ``hd / 2`` bytes of
codes a token (the even value in a byte's low half), then the scales, ``[16, hd / 16]`` for keys and
``[hd / 16, 16]`` for values.  A code is a sign, two bits of exponent and one of mantissa (0, 0.5, 1,
1.5, 2, 3, 4, 6), a scale four bits of exponent and three of mantissa.
"""
import math
import random

import torch

own = False

PAGE = 16   # tokens of a page
BLOCK = 16  # values that share a scale in the 4-bit cache
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # The tokens of a small decode step: latency.
        _append("append_decode_small", layout=1, tokens=8, runs=8, bits=16),
        # A chunked-prefill step with a full token budget, q, k and v parts of one projection's
        # output, some rows of padding.
        _append("append_prompt_fused", layout=2, tokens=8192, runs=132, bits=16, fused=True,
                padding=37),
        # A full decode batch into a 4-bit cache.
        _append("append4_decode_batch", layout=3, tokens=256, runs=256, bits=4),
        # Prompts into a 4-bit cache: adjacent pairs rotated, half of each head left as it is,
        # heads and lengths that divide nothing.
        _append("append4_prompt_odd", layout=4, tokens=4099, runs=5, bits=4, nh=12, nkv=3,
                rotary=64, interleaved=True, padding=5, scaled=True),
        # Six decodes of a step that has nothing else to do: latency of one token.
        _attention("attention4_decode_small", layout=5, decodes=6, dec_min=1000, dec_max=4000),
        # A full decode batch over long caches: every cached key is read once.
        _attention("attention4_decode_batch", layout=6, decodes=256, dec_min=512, dec_max=8192),
        # A chunked-prefill step: prompts with cached parts among decodes.
        _attention("attention4_mixed", layout=7, decodes=128, dec_min=256, dec_max=32768,
                   chunks=4, chunk_min=1024, chunk_max=2048, hist_max=16384, scaled=True),
        # Prompts of odd lengths, a head group that does not divide a tile, padded rows.
        _attention("attention4_prompts_odd", layout=8, nh=12, nkv=2, hd=64, decodes=5, dec_min=1,
                   dec_max=777, chunks=9, chunk_min=1, chunk_max=1501, hist_max=700, padding=11),
        # A decode step's hidden states, 16-bit output.
        _norm("norm_decode", rows=64, hidden=4096, dtype="bf16", bits=16),
        # A token budget's hidden states into an 8-bit product, one scale a row.
        _norm("norm_prompt_rows", rows=8192, hidden=4096, dtype="bf16", bits=8),
        # Odd numbers of rows and a row distance, a scale for every 128 values.
        _norm("norm_prompt_groups", rows=2047, hidden=5120, dtype="fp16", bits=8, group=128,
              gap=64),
        # A row that is no whole number of vectors, in 32 bits, without a residual.
        _norm("norm_odd_width", rows=513, hidden=2889, dtype="fp32", bits=16, residual=False),
    ]


def _append(name, layout, tokens, runs, bits, nh=32, nkv=8, hd=128, rotary=0, interleaved=False,
            fused=False, padding=0, scaled=False):
    return {"name": name, "op": "append", "layout": layout, "tokens": tokens, "runs": runs,
            "bits": bits, "nh": nh, "nkv": nkv, "hd": hd, "rotary": rotary or hd,
            "interleaved": interleaved, "fused": fused, "padding": padding, "scaled": scaled}


def _attention(name, layout, nh=32, nkv=8, hd=128, decodes=0, dec_min=1, dec_max=1, chunks=0,
               chunk_min=1, chunk_max=1, hist_max=0, padding=0, scaled=False):
    return {"name": name, "op": "attention", "layout": layout, "nh": nh, "nkv": nkv, "hd": hd,
            "decodes": decodes, "dec_min": dec_min, "dec_max": dec_max, "chunks": chunks,
            "chunk_min": chunk_min, "chunk_max": chunk_max, "hist_max": hist_max,
            "padding": padding, "scaled": scaled}


def _norm(name, rows, hidden, dtype, bits, group=0, gap=0, residual=True):
    return {"name": name, "op": "norm", "rows": rows, "hidden": hidden, "dtype": dtype,
            "bits": bits, "group": group, "gap": gap, "residual": residual}


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "attention", "attention", "attention", "norm", "norm"])
    if op == "append":
        nh, nkv = rng.choice([(32, 8), (64, 8), (16, 16), (12, 3), (28, 4), (16, 1), (7, 1)])
        hd = rng.choice([64, 128])
        tokens = min(_log_uniform(rng, 1, 8192), 8192 * 40 * 128 // ((nh + nkv) * hd))
        runs = rng.randint(1, min(tokens, 300))
        return _append("", layout=rng.randrange(1 << 30), tokens=tokens, runs=runs,
                       bits=rng.choice([4, 16]), nh=nh, nkv=nkv, hd=hd,
                       rotary=rng.choice([hd, hd, hd // 2, hd // 4]),
                       interleaved=rng.random() < 0.4, fused=rng.random() < 0.5,
                       padding=rng.choice([0, 0, 1, 9, 40]), scaled=rng.random() < 0.3)
    if op == "attention":
        nh, nkv = rng.choice([(32, 8), (64, 8), (16, 16), (12, 2), (28, 4), (16, 1), (7, 1),
                              (8, 2)])
        hd = rng.choice([64, 128])
        kinds = rng.choice(["decode", "prefill", "mixed"])
        hist = _log_uniform(rng, 16, 16384)
        chunk = _log_uniform(rng, 2, 2048)
        dec = _log_uniform(rng, 16, 32768)
        # no more keys or (query, key) pairs than the largest listed case has
        most = 600_000 * 8 * 128 // (nkv * hd * dec)
        decodes = min(_log_uniform(rng, 1, 256), max(1, most)) if kinds != "prefill" else 0
        most = 25_000_000 * 32 * 128 // (nh * hd * chunk * (hist // 2 + chunk // 2 + 1))
        chunks = min(_log_uniform(rng, 1, 9), max(1, most)) if kinds != "decode" else 0
        return _attention("", layout=rng.randrange(1 << 30), nh=nh, nkv=nkv, hd=hd,
                          decodes=decodes, dec_min=max(1, dec // 8), dec_max=dec, chunks=chunks,
                          chunk_min=max(1, chunk // 2), chunk_max=chunk, hist_max=hist,
                          padding=rng.choice([0, 0, 3, 60]), scaled=rng.random() < 0.3)
    bits = rng.choice([8, 8, 16])
    group = rng.choice([0, 0, 128, 64]) if bits == 8 else 0
    hidden = _log_uniform(rng, 32, 16384)
    if group or rng.random() < 0.7:
        hidden = -(-hidden // 128) * 128
    rows = max(1, min(_log_uniform(rng, 1, 8192), 8192 * 4096 // hidden))
    return _norm("", rows=rows, hidden=hidden, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                 bits=bits, group=group, gap=rng.choice([0, 0, 8, 61]),
                 residual=rng.random() < 0.7)


# ------------------------------------------------------------------------------- 4-bit values
def _encode(x, scale):
    """Codes [..., hd] and scale bytes [..., hd / 16] of values [..., hd]."""
    y = (x.float() / scale).unflatten(-1, (-1, BLOCK))
    size = y.abs()
    e4m3 = (size.amax(-1, keepdim=True) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = e4m3.float()
    t = torch.where(s > 0, size / s, torch.zeros_like(size))
    # a half-way value goes to the code whose last bit is 0
    code = (t > 0.25).byte() + (t >= 0.75).byte() + (t > 1.25).byte() + (t >= 1.75).byte() + \
        (t > 2.5).byte() + (t >= 3.5).byte() + (t > 5.0).byte()
    return (code + 8 * torch.signbit(y).byte()).flatten(-2), e4m3.squeeze(-1).view(torch.uint8)


def _levels():
    return torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0,
                         -3.0, -4.0, -6.0], device="cuda")


def _parts(cache, hd, values):
    """Views of a cache [pages, nkv, 9 hd]: codes [pages, nkv, 16, hd / 2] and scales [pages, nkv,
    16, hd / 16]."""
    codes = cache[:, :, :8 * hd].unflatten(2, (PAGE, hd // 2))
    scales = cache[:, :, 8 * hd:]
    if values:
        return codes, scales.unflatten(2, (hd // BLOCK, PAGE)).transpose(2, 3)
    return codes, scales.unflatten(2, (PAGE, hd // BLOCK))


def _decode(codes, scales, scale):
    """The fp32 values [..., hd] of codes [..., hd / 2] and scales [..., hd / 16]."""
    both = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()
    value = _levels()[both].unflatten(-1, (-1, BLOCK))
    s = scales.contiguous().view(torch.float8_e4m3fn).float()
    return (value * s[..., None] * scale).flatten(-2)


def _random_cache(g, pages, nkv, hd, scale, values):
    """A 4-bit cache of normally distributed values whose channels differ in size."""
    cache = torch.empty(pages, nkv, 9 * hd, dtype=torch.uint8, device="cuda")
    gain = torch.exp(0.3 * torch.randn(nkv, 1, hd, generator=g, device="cuda"))
    codes, scales = _parts(cache, hd, values)
    step = max(1, (1 << 25) // (nkv * hd * PAGE))
    for lo in range(0, pages, step):
        n = min(step, pages - lo)
        x = torch.randn(n, nkv, PAGE, hd, generator=g, device="cuda") * gain * scale
        code, s = _encode(x.to(torch.bfloat16), scale)
        codes[lo:lo + n] = code[..., ::2] + 16 * code[..., 1::2]
        scales[lo:lo + n] = s
    return cache


# ------------------------------------------------------------------------------------ append
def _append_layout(case):
    """Position and slot of each token: runs of consecutive positions, each of them a request,
    whose pages are scattered over the pool; the padding tokens come last and have no slot."""
    rng = random.Random(case["layout"])
    real = max(1, case["tokens"] - case["padding"])
    cuts = sorted(rng.sample(range(1, real), min(case["runs"], real) - 1)) if real > 1 else []
    positions, places, pages = [], [], 0
    for a, b in zip([0] + cuts, cuts + [real]):
        start = _log_uniform(rng, 1, 30000) - 1
        for t in range(b - a):
            p = start + t
            if t == 0 or p % PAGE == 0:
                pages += 1
            positions.append(p)
            places.append((pages - 1, p % PAGE))
    spare = 3
    ids = rng.sample(range(1, pages + 1 + spare), pages)  # page 0 is the null page
    slots = [ids[i] * PAGE + o for i, o in places]
    extra = case["tokens"] - real
    return positions + [0] * extra, slots + [-1] * extra, pages + 1 + spare


def _prepare_append(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    nh, nkv, hd, tokens = case["nh"], case["nkv"], case["hd"], case["tokens"]
    positions, slots, pages = _append_layout(case)
    i32 = lambda xs: torch.tensor(xs, dtype=torch.int32).cuda()
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)
    if case["fused"]:
        q, k, v = randn(tokens, nh + 2 * nkv, hd).split([nh, nkv, nkv], 1)
    else:
        q, k, v = randn(tokens, nh, hd), randn(tokens, nkv, hd), randn(tokens, nkv, hd)
    half = case["rotary"] // 2
    # cosines, then sines, of every position's angles, which are taken in 64 bits
    step = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    angle = torch.arange(max(positions) + 1, dtype=torch.float64, device="cuda")[:, None] * step
    s = {"op": "append", "case": case, "q": q, "k": k, "v": v, "positions": i32(positions),
         "slots": i32(slots), "pages": pages,
         "table": torch.cat((torch.cos(angle), torch.sin(angle)), 1).float(),
         "k_scale": 0.25 if case["scaled"] else 1.0, "v_scale": 3.0 if case["scaled"] else 1.0}
    if case["bits"] == 4:
        s["k_cache"] = _random_cache(g, pages, nkv, hd, s["k_scale"], False)
        s["v_cache"] = _random_cache(g, pages, nkv, hd, s["v_scale"], True)
    else:
        s["k_cache"], s["v_cache"] = randn(pages * PAGE, nkv, hd), randn(pages * PAGE, nkv, hd)
    s["q_out"] = torch.empty(tokens, nh, hd, dtype=torch.bfloat16, device="cuda")
    s["error"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if own:
        import ragged_mixed_paged_gb300 as rb

        s["dims"] = rb.Dims(block_size=PAGE, num_q_heads=nh, num_kv_heads=nkv, head_dim=hd,
                            max_num_reqs=1, max_model_len=PAGE, max_blocks_per_req=1,
                            num_blocks=pages)
        s["rotation"] = rb.Rotation(s["table"], interleaved=case["interleaved"])
        s["rows"] = tuple(torch.empty(tokens, nkv, hd, dtype=torch.bfloat16, device="cuda")
                          for _ in range(2))
    return s


def _rotate(x, cos, sin, interleaved):
    """Heads [tokens, heads, hd] with their first 2 * cos.shape[1] values rotated, in bf16."""
    n = 2 * cos.shape[1]
    y, rest = x[..., :n].float(), x[..., n:].float()
    a, b = (y[..., ::2], y[..., 1::2]) if interleaved else (y[..., :n // 2], y[..., n // 2:])
    cos, sin = cos[:, None], sin[:, None]
    c, d = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((c, d), -1).flatten(-2) if interleaved else torch.cat((c, d), -1)
    return torch.cat((turned, rest), -1).to(torch.bfloat16)


def _run_append(s):
    case = s["case"]
    if own:
        import ragged_mixed_paged_gb300 as rb

        if case["bits"] == 16:
            rb.kv_append(s["dims"], s["q"], s["k"], s["v"], s["slots"], s["k_cache"],
                         s["v_cache"], positions=s["positions"], rotation=s["rotation"],
                         q_out=s["q_out"], error_word=s["error"])
            return s["q_out"], s["k_cache"], s["v_cache"]
        rb.kv4_append(s["dims"], s["q"], s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"],
                      positions=s["positions"], rotation=s["rotation"], k_scale=s["k_scale"],
                      v_scale=s["v_scale"], q_out=s["q_out"], error_word=s["error"])
        return (s["q_out"],) + rb.kv4_read(
            s["dims"], s["slots"], s["k_cache"], s["v_cache"], k_scale=s["k_scale"],
            v_scale=s["v_scale"], out=s["rows"], error_word=s["error"])
    turn = s["table"][s["positions"].long()]
    cos, sin = turn.chunk(2, 1)
    q = _rotate(s["q"], cos, sin, case["interleaved"])
    k = _rotate(s["k"], cos, sin, case["interleaved"])
    slots = s["slots"].long()
    real = torch.nonzero(slots >= 0).flatten()
    slots = slots[real]
    if case["bits"] == 16:
        s["k_cache"][slots] = k[real]
        s["v_cache"][slots] = s["v"][real]
        return q, s["k_cache"], s["v_cache"]
    page, place = slots // PAGE, slots % PAGE
    rows = []
    for name, x, scale in (("k_cache", k, s["k_scale"]), ("v_cache", s["v"], s["v_scale"])):
        codes, scales = _parts(s[name], case["hd"], name == "v_cache")
        code, e4m3 = _encode(x[real], scale)
        codes[page, :, place] = code[..., ::2] + 16 * code[..., 1::2]
        scales[page, :, place] = e4m3
        row = torch.zeros_like(x, memory_format=torch.contiguous_format)
        row[real] = _decode(codes[page, :, place], scales[page, :, place], scale).to(row.dtype)
        rows.append(row)
    return q, rows[0], rows[1]


def _exact_append(case, seed):
    s = _prepare_append(case, seed)
    half, hd = case["rotary"] // 2, case["hd"]
    pos = s["positions"].long()
    cs, sn = s["table"].double()[pos, :half], s["table"].double()[pos, half:]

    def turn(x):
        x = x.double()
        first = torch.arange(half, device="cuda")
        i, j = (2 * first, 2 * first + 1) if case["interleaved"] else (first, first + half)
        z = torch.complex(x[..., i], x[..., j]) * torch.complex(cs, sn)[:, None]
        x = x.clone()
        x[..., i], x[..., j] = z.real, z.imag
        return x

    q, k = turn(s["q"]), turn(s["k"])
    at = s["slots"].long()
    here = at >= 0
    if case["bits"] == 16:
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        kc[at[here]], vc[at[here]] = k[here], s["v"][here].double()
        return q, kc, vc

    def held(x, scale):
        """The nearest value that each block of a 16-bit row can hold, 0 without a slot."""
        x = x.to(torch.bfloat16).double().unflatten(-1, (hd // BLOCK, BLOCK)) / scale
        grid = torch.tensor([m * 2.0 ** -9 for m in range(8)] +
                            [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)],
                            dtype=torch.float64, device="cuda")[:127]
        s8 = _nearest(x.abs().amax(-1, keepdim=True) / 6, grid)
        small = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
        t = torch.where(s8 > 0, x.abs() / torch.where(s8 > 0, s8, 1.0), 0.0)
        y = torch.copysign(_nearest(t, small), x) * s8 * scale
        return torch.where(here[:, None, None], y.flatten(-2), 0.0)

    return q, held(k, s["k_scale"]), held(s["v"], s["v_scale"])


def _nearest(x, grid):
    """The nearest of ascending `grid` values, the even one of two that are as near."""
    hi = torch.searchsorted(grid, x).clamp(1, len(grid) - 1)
    below, above = x - grid[hi - 1], grid[hi] - x
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return torch.where(up, grid[hi], grid[hi - 1])


def _append_work(case):
    nh, nkv, hd, tokens = case["nh"], case["nkv"], case["hd"], case["tokens"]
    real = max(1, tokens - case["padding"])
    positions, _, _ = _append_layout(case)
    turn = 4 * case["rotary"] * len(set(positions[:real]))
    row = 2 * nkv * hd  # K and V values of one token
    cache = real * (2 * row if case["bits"] == 16 else row * 9 // 16)
    back = 0 if case["bits"] == 16 else real * row * 9 // 16 + tokens * 2 * row
    # a rotated pair is four products and two sums; a quantised value is a comparison, a quotient
    # and a rounding, a value read back a product
    flops = tokens * (nh + nkv) * case["rotary"] * 3
    flops += real * row * 4 if case["bits"] == 4 else 0
    return {"bytes": tokens * (4 * nh * hd + 8) + real * 2 * row + turn + cache + back,
            "flops": flops}


# --------------------------------------------------------------------------------- attention
def _requests(case):
    """(cached, new) tokens of the batch's requests."""
    rng = random.Random(case["layout"])
    reqs = [(_log_uniform(rng, case["dec_min"], case["dec_max"]), 1)
            for _ in range(case["decodes"])]
    for _ in range(case["chunks"]):
        q = rng.randint(case["chunk_min"], case["chunk_max"])
        reqs.append((rng.randint(0, case["hist_max"]), q))
    rng.shuffle(reqs)
    return reqs


def _prepare_attention(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    reqs = _requests(case)
    nh, nkv, hd = case["nh"], case["nkv"], case["hd"]
    pages = [-(-(c + q) // PAGE) for c, q in reqs]
    num_pages = sum(pages) + 1
    tokens = sum(q for _, q in reqs)
    width = max(pages)
    ids = (1 + torch.randperm(num_pages - 1, generator=g, device="cuda")).to(torch.int32).cpu()
    table = torch.full((len(reqs), width), -1, dtype=torch.int32)
    loc, at = [0], 0
    for i, n in enumerate(pages):
        table[i, :n] = ids[at:at + n]
        at += n
        loc.append(loc[-1] + reqs[i][1])
    i32 = lambda xs: torch.tensor(xs, dtype=torch.int32).cuda()
    s = {"op": "attention", "case": case, "tokens": tokens, "width": width,
         "num_pages": num_pages, "table": table.cuda(), "loc": i32(loc),
         "lens": i32([c + q for c, q in reqs]),
         "k_scale": 0.25 if case["scaled"] else 1.0, "v_scale": 3.0 if case["scaled"] else 1.0}
    s["q"] = 3.0 * torch.randn(tokens + case["padding"], nh, hd, generator=g, device="cuda",
                               dtype=torch.bfloat16) / s["k_scale"]
    s["k"] = _random_cache(g, num_pages, nkv, hd, s["k_scale"], False)
    s["v"] = _random_cache(g, num_pages, nkv, hd, s["v_scale"], True)
    s["out"] = torch.empty_like(s["q"])
    s["error"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    # the order in which the plain form takes the requests: sixteen of one new token and about the
    # same length at a time, the others alone
    length = lambda i: sum(reqs[i])
    order = sorted((i for i, (_, q) in enumerate(reqs) if q == 1), key=length)
    groups = [order[a:a + 16] for a in range(0, len(order), 16)]
    groups += [[i] for i, (_, q) in enumerate(reqs) if q > 1]
    s["groups"] = [(torch.tensor(x).cuda(),
                    torch.tensor([list(range(loc[i], loc[i + 1])) for i in x]).cuda(),
                    length(x[-1])) for x in groups]
    if own:
        import ragged_mixed_paged_gb300 as rb

        s["dims"] = rb.Dims(block_size=PAGE, num_q_heads=nh, num_kv_heads=nkv, head_dim=hd,
                            max_num_reqs=len(reqs), max_model_len=width * PAGE,
                            max_blocks_per_req=width, num_blocks=num_pages)
        s["workspace"] = torch.empty(rb.workspace_size(s["dims"], len(reqs), tokens),
                                     dtype=torch.uint8, device="cuda")
    return s


def _run_attention(s):
    case = s["case"]
    nh, nkv, hd = case["nh"], case["nkv"], case["hd"]
    if own:
        import ragged_mixed_paged_gb300 as rb

        return rb.paged_attention_kv4(s["dims"], s["lens"].shape[0], s["tokens"], s["q"], s["k"],
                                      s["v"], s["table"], s["loc"], s["lens"],
                                      k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["out"],
                                      workspace=s["workspace"], error_word=s["error"])
    out = torch.zeros_like(s["q"])
    for rows, tokens, length in s["groups"]:
        ids = s["table"][rows, :-(-length // PAGE)].long().clamp(min=0)
        k = _decode(*_parts(s["k"][ids].flatten(0, 1), hd, False), s["k_scale"])
        v = _decode(*_parts(s["v"][ids].flatten(0, 1), hd, True), s["v_scale"])
        # [requests, nkv, keys, hd]
        k = k.unflatten(0, ids.shape).transpose(1, 2).flatten(2, 3)[:, :, :length]
        v = v.unflatten(0, ids.shape).transpose(1, 2).flatten(2, 3)[:, :, :length]
        n = tokens.shape[1]
        q = s["q"][tokens].float().view(-1, n, nkv, nh // nkv, hd).permute(0, 2, 3, 1, 4)
        x = torch.matmul(q.flatten(2, 3), k.transpose(2, 3)) / math.sqrt(hd)
        x = x.unflatten(2, (nh // nkv, n))
        pos = tokens - s["loc"][rows + 1].long()[:, None] + s["lens"][rows].long()[:, None]
        hidden = torch.arange(length, device="cuda") > pos[:, :, None]
        x = x.masked_fill(hidden[:, None, None], -math.inf)
        p = torch.exp(x - x.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
        o = torch.matmul(p.flatten(2, 3), v).unflatten(2, (nh // nkv, n))
        out[tokens] = o.permute(0, 3, 1, 2, 4).flatten(2, 3).to(out.dtype)
    return out


def _exact_attention(case, seed):
    if _attention_work(case)["flops"] > 4e12:
        return None
    s = _prepare_attention(case, seed)
    nh, nkv, hd = case["nh"], case["nkv"], case["hd"]
    group = nh // nkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")

    def held(page, scales, scale):
        """Values [keys, hd] in 64 bits of bytes [pages, 8 hd] and scale bytes [keys, hd / 16]."""
        b = page.reshape(-1, hd // 2).long()
        c = torch.stack([b % 16, b // 16], 2).reshape(-1, hd // BLOCK, BLOCK)
        e, m = (c // 2) % 4, (c % 2).double()
        size = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e.double() - 1))
        sb = scales.long()
        se, sm = sb // 8, (sb % 8).double()
        by = torch.where(se == 0, sm / 512, (1 + sm / 8) * torch.exp2(se.double() - 7))
        return (torch.where(c >= 8, -size, size) * (by * scale)[:, :, None]).reshape(-1, hd)

    first = 0
    for i, (c, q) in enumerate(_requests(case)):
        length = c + q
        ids = s["table"][i, :-(-length // PAGE)].long()
        for h in range(nkv):
            kp, vp = s["k"][ids, h], s["v"][ids, h]
            kk = held(kp[:, :8 * hd], kp[:, 8 * hd:].reshape(-1, hd // BLOCK), s["k_scale"])
            vs = vp[:, 8 * hd:].reshape(-1, hd // BLOCK, PAGE).permute(0, 2, 1)
            vv = held(vp[:, :8 * hd], vs.reshape(-1, hd // BLOCK), s["v_scale"])
            kk, vv = kk[:length], vv[:length]
            rows = max(1, (1 << 26) // (length * group))
            for a in range(0, q, rows):
                b = min(q, a + rows)
                x = s["q"][first + a:first + b, h * group:(h + 1) * group].double()
                y = torch.einsum("qhd,kd->hqk", x, kk) * hd ** -0.5
                ahead = torch.ones(b - a, length, dtype=torch.bool, device="cuda")
                y[:, ahead.triu(c + a + 1)] = -math.inf
                o = torch.einsum("hqk,kd->qhd", torch.softmax(y, 2), vv)
                out[first + a:first + b, h * group:(h + 1) * group] = o
        first += q
    return out


def _attention_work(case):
    nh, nkv, hd = case["nh"], case["nkv"], case["hd"]
    reqs = _requests(case)
    keys = sum(c + q for c, q in reqs)
    tokens = sum(q for _, q in reqs)
    pairs = sum(q * c + q * (q + 1) // 2 for c, q in reqs)
    return {"bytes": 2 * (2 * tokens + case["padding"]) * nh * hd + 2 * keys * nkv * hd * 9 // 16 +
            4 * -(-keys // PAGE) + 8 * len(reqs), "flops": 4 * hd * nh * pairs}


# -------------------------------------------------------------------------------------- norm
EPS = 1e-5


def _prepare_norm(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows, hidden, dtype = case["rows"], case["hidden"], TYPES[case["dtype"]]
    wide = hidden + case["gap"]
    # a few channels far larger than the others, as hidden states have
    gain = torch.exp(torch.randn(wide, generator=g, device="cuda"))
    state = lambda: (torch.randn(rows, wide, generator=g, device="cuda") * gain).to(dtype)
    s = {"op": "norm", "case": case, "x": state()[:, :hidden],
         "weight": (1.0 + 0.2 * torch.randn(hidden, generator=g, device="cuda")).to(dtype),
         "residual": state()[:, :hidden] if case["residual"] else None}
    if case["residual"]:
        s["sum"] = torch.empty(rows, hidden, dtype=dtype, device="cuda")
    if case["bits"] == 8:
        s["out"] = torch.empty(rows, hidden, dtype=torch.float8_e4m3fn, device="cuda")
        s["scales"] = torch.empty(rows, hidden // case["group"] if case["group"] else 1,
                                  dtype=torch.float32, device="cuda")
    else:
        s["out"] = torch.empty(rows, hidden, dtype=dtype, device="cuda")
    return s


def _run_norm(s):
    case = s["case"]
    if own:
        import ragged_mixed_paged_gb300 as rb

        if case["bits"] == 8:
            rb.add_rms_norm_fp8(s["x"], s["weight"], EPS, residual=s["residual"],
                                residual_out=s.get("sum"), group=case["group"], out=s["out"],
                                scales=s["scales"])
            got = (s["out"], s["scales"])
        else:
            rb.add_rms_norm(s["x"], s["weight"], EPS, residual=s["residual"],
                            residual_out=s.get("sum"), out=s["out"])
            got = (s["out"],)
        return got + (s["sum"],) if case["residual"] else got
    x = s["x"].float()
    if case["residual"]:
        total = (x + s["residual"].float()).to(s["x"].dtype)
        x = total.float()
    y = x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS) * s["weight"].float()
    if case["bits"] == 8:
        y = y.unflatten(1, (-1, case["group"] or case["hidden"]))
        scales = y.abs().amax(2, keepdim=True) / 448.0
        code = torch.where(scales > 0, y / scales, torch.zeros_like(y)).clamp(-448.0, 448.0)
        got = (code.to(torch.float8_e4m3fn).flatten(1), scales.squeeze(2))
    else:
        got = (y.to(s["x"].dtype),)
    return got + (total,) if case["residual"] else got


def _exact_norm(case, seed):
    s = _prepare_norm(case, seed)
    z = s["x"].double()
    if case["residual"]:
        z = (z + s["residual"].double()).to(s["x"].dtype).double()
        after = (z,)
    else:
        after = ()
    size = torch.linalg.vector_norm(z, dim=1).square() / case["hidden"] + EPS
    y = s["weight"].double() * z / size.sqrt()[:, None]
    if case["bits"] != 8:
        return (y,) + after
    n = case["group"] or case["hidden"]
    blocks = y.reshape(case["rows"], -1, n)
    top = torch.maximum(blocks.amax(2), -blocks.amin(2)) / 448
    grid = torch.tensor([m * 2.0 ** -9 for m in range(8)] +
                        [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)],
                        dtype=torch.float64, device="cuda")[:127]
    t = blocks / torch.where(top > 0, top, 1.0)[:, :, None]
    code = torch.copysign(_nearest(t.abs().contiguous(), grid), t)
    return (code.reshape(case["rows"], -1), top) + after


def _norm_work(case):
    n, wide = case["rows"] * case["hidden"], 4 if case["dtype"] == "fp32" else 2
    moved = n * wide * (3 if case["residual"] else 1) + case["hidden"] * wide
    if case["bits"] == 8:
        moved += n + 4 * (n // case["group"] if case["group"] else case["rows"])
    else:
        moved += n * wide
    # the sum, its square and their sum, two products; the size, a quotient and the rounding
    return {"bytes": moved, "flops": n * (5 if case["bits"] == 16 else 8)}


# --------------------------------------------------------------------------------- interface
_PREPARE = {"append": _prepare_append, "attention": _prepare_attention, "norm": _prepare_norm}
_RUN = {"append": _run_append, "attention": _run_attention, "norm": _run_norm}
_EXACT = {"append": _exact_append, "attention": _exact_attention, "norm": _exact_norm}
_WORK = {"append": _append_work, "attention": _attention_work, "norm": _norm_work}


def prepare(case, seed):
    return _PREPARE[case["op"]](case, seed)


def run(state):
    return _RUN[state["op"]](state)


def exact(case, seed):
    return _EXACT[case["op"]](case, seed)


def work(case):
    return _WORK[case["op"]](case)
