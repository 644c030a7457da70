"""Workloads of the serving operators around the paged cache, with their plain forms.

Three families, each as a server calls it between two steps of a model runner:

* ``attention`` - attention of a mixed batch through the page table whose scores are capped by
  a tanh, biased by the distance of query and key, or masked by documents, windows and
  bidirectional prefixes;
* ``copy``, ``fork`` and ``compact`` - page management of the paged cache: copying pages,
  forking requests (shared full pages, the partial page copied), and freeing finished requests
  followed by compacting the pool;
* ``logprobs`` - log probability, rank and entropy of given tokens with the top alternatives.

``own`` selects the library's kernels; otherwise ``run`` computes the same with elementary
torch operations in 32 bits or more.
"""
import math
import random

import torch

own = False

PAGE = 16  # tokens of a page
LOG_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # Six decodes of a serving step that has nothing else to do: latency of one token with
        # capped scores.
        _attention("attention_decode_small", layout=1, decodes=6, dec_min=1000, dec_max=4000,
                   softcap=30.0),
        # A full decode batch over long caches with a bias that falls with distance: every
        # cached key is read once.
        _attention("attention_decode_batch", layout=2, decodes=256, dec_min=512, dec_max=8192,
                   slopes=True),
        # A chunked-prefill step: packed documents in the prompts, a window for the decodes,
        # capped scores, some tokens that may see nothing.
        _attention("attention_mixed_documents", layout=3, decodes=128, dec_min=256,
                   dec_max=32768, dec_window=4096, chunks=4, chunk_min=1024, chunk_max=2048,
                   hist_max=16384, doc_len=12000, softcap=50.0, blanks=True),
        # Prompts whose first part is read in both directions, odd lengths, a head group that
        # does not divide a tile.
        _attention("attention_prefix_odd", layout=4, nh=12, nkv=2, hd=64, decodes=5, dec_min=1,
                   dec_max=777, chunks=9, chunk_min=1, chunk_max=1501, hist_max=700,
                   slopes=True, prefix=True),
        # Copy-on-write of four pages at one step.
        {"name": "copy_few_pages", "op": "copy", "nkv": 8, "hd": 128, "pages": 4096, "pairs": 4},
        # Moving a preempted request's worth of pages many times over: the bandwidth case.
        {"name": "copy_many_pages", "op": "copy", "nkv": 8, "hd": 128, "pages": 24576,
         "pairs": 8191},
        # Four samples drawn from one prompt.
        {"name": "fork_samples", "op": "fork", "nkv": 8, "hd": 128, "layout": 11, "rows": 8,
         "forks": 4, "sources": 1, "c_min": 900, "c_max": 1100, "spare": 64},
        # Every request of a full batch forks once, beams of two.
        {"name": "fork_batch", "op": "fork", "nkv": 8, "hd": 128, "layout": 12, "rows": 512,
         "forks": 256, "sources": 256, "c_min": 512, "c_max": 4096, "spare": 700},
        # A few requests of a small pool finish.
        {"name": "compact_small", "op": "compact", "nkv": 2, "hd": 64, "layout": 13, "rows": 24,
         "free": 9, "c_min": 1, "c_max": 500, "spare": 100},
        # Half of a full batch finishes and the pool is packed.
        {"name": "compact_batch", "op": "compact", "nkv": 8, "hd": 128, "layout": 14,
         "rows": 200, "free": 100, "c_min": 512, "c_max": 5000, "spare": 5000},
        # One decode step's sampled tokens, logits in 16 bits, padded rows.
        _logprobs("logprobs_decode", rows=64, vocab=32000, stride=32064, dtype="bf16", top=5),
        # The prompt tokens of a chunk, logits in 32 bits, grammar-masked tokens among them.
        _logprobs("logprobs_prompt", rows=2047, vocab=100003, stride=100003, dtype="fp32",
                  top=20, banned=True),
    ]


def _attention(name, layout, nh=32, nkv=8, hd=128, decodes=0, dec_min=1, dec_max=1,
               dec_window=0, chunks=0, chunk_min=1, chunk_max=1, hist_max=0, doc_len=0,
               softcap=0.0, slopes=False, prefix=False, blanks=False):
    return {"name": name, "op": "attention", "layout": layout, "nh": nh, "nkv": nkv, "hd": hd,
            "decodes": decodes, "dec_min": dec_min, "dec_max": dec_max,
            "dec_window": dec_window, "chunks": chunks, "chunk_min": chunk_min,
            "chunk_max": chunk_max, "hist_max": hist_max, "doc_len": doc_len,
            "softcap": softcap, "slopes": slopes, "prefix": prefix, "blanks": blanks}


def _logprobs(name, rows, vocab, stride, dtype, top, banned=False):
    return {"name": name, "op": "logprobs", "rows": rows, "vocab": vocab, "stride": stride,
            "dtype": dtype, "top": top, "banned": banned}


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "copy", "fork", "compact",
                     "logprobs", "logprobs"])
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
        return _attention(
            "", layout=rng.randrange(1 << 30), nh=nh, nkv=nkv, hd=hd, decodes=decodes,
            dec_min=max(1, dec // 8), dec_max=dec, dec_window=rng.choice([0, 0, 100, 1024]),
            chunks=chunks, chunk_min=max(1, chunk // 2), chunk_max=chunk, hist_max=hist,
            doc_len=rng.choice([0, 0, 37, 1500]), softcap=rng.choice([0.0, 0.0, 20.0, 50.0]),
            slopes=rng.random() < 0.5, prefix=rng.random() < 0.3, blanks=rng.random() < 0.2)
    nkv, hd = rng.choice([(8, 128), (2, 64), (1, 128), (16, 64), (3, 128)])
    if op == "copy":
        pairs = _log_uniform(rng, 1, 8000)
        return {"name": "", "op": "copy", "nkv": nkv, "hd": hd,
                "pages": 2 * pairs + rng.randrange(1, 2000), "pairs": pairs}
    if op == "fork":
        sources = _log_uniform(rng, 1, 200)
        forks = _log_uniform(rng, 1, 250)
        c_max = _log_uniform(rng, 4, 4000)
        return {"name": "", "op": "fork", "nkv": nkv, "hd": hd, "layout": rng.randrange(1 << 30),
                "rows": sources + forks + rng.randrange(0, 60), "forks": forks,
                "sources": sources, "c_min": rng.randrange(0, c_max), "c_max": c_max,
                "spare": forks + rng.randrange(0, 500)}
    if op == "compact":
        rows = _log_uniform(rng, 1, 200)
        c_max = _log_uniform(rng, 4, 4900)
        return {"name": "", "op": "compact", "nkv": nkv, "hd": hd,
                "layout": rng.randrange(1 << 30), "rows": rows, "free": rng.randrange(0, rows + 1),
                "c_min": rng.randrange(0, c_max), "c_max": c_max,
                "spare": rng.randrange(1, 5000)}
    vocab = _log_uniform(rng, 50, 200000)
    rows = max(1, min(_log_uniform(rng, 1, 4096), 200_000_000 // vocab))
    return _logprobs("", rows=rows, vocab=vocab, stride=vocab + rng.choice([0, 0, 1, 8, 61]),
                     dtype=rng.choice(["bf16", "fp16", "fp32"]), top=rng.choice([0, 1, 5, 20, 32]),
                     banned=rng.random() < 0.3)


# ----------------------------------------------------------------------------- attention: layout
def _requests(case):
    """The batch's requests: cached and new tokens, bidirectional prefix, window, and the
    first position of the document that each new token belongs to."""
    rng = random.Random(case["layout"])
    reqs = []
    for _ in range(case["decodes"]):
        c = _log_uniform(rng, case["dec_min"], case["dec_max"])
        reqs.append((c, 1, case["dec_window"], False))
    for _ in range(case["chunks"]):
        q = rng.randint(case["chunk_min"], case["chunk_max"])
        c = rng.randint(0, case["hist_max"])
        reqs.append((c, q, 0, case["doc_len"] > 0))
    rng.shuffle(reqs)
    out = []
    for i, (c, q, window, docs) in enumerate(reqs):
        length = c + q
        prefix = rng.randint(0, length) if case["prefix"] else 0
        starts = []
        bounds = [0]
        if docs:
            while bounds[-1] < length:
                bounds.append(bounds[-1] + rng.randint(1, 2 * case["doc_len"]))
        b = 0
        for j in range(q):
            p = c + j
            while docs and b + 1 < len(bounds) and bounds[b + 1] <= p:
                b += 1
            s = bounds[b]
            if window:
                s = max(s, p - window + 1)
            if case["blanks"] and (31 * i + j) % 97 == 13:
                s = length + 5  # a token that may see no key
            starts.append(max(s, 0))
        out.append({"c": c, "q": q, "prefix": prefix, "starts": starts})
    return out


def _uses_starts(case):
    return bool(case["doc_len"] or case["dec_window"] or case["blanks"])


def _visible(req):
    """(first, past-the-last) visible key of each new token of a request."""
    length = req["c"] + req["q"]
    return [(s, min(length, max(req["c"] + j + 1, req["prefix"])))
            for j, s in enumerate(req["starts"])]


def _prepare_attention(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    reqs = _requests(case)
    nh, nkv, hd = case["nh"], case["nkv"], case["hd"]
    pages = [-(-(r["c"] + r["q"]) // PAGE) for r in reqs]
    num_pages = sum(pages) + 1
    tokens = sum(r["q"] for r in reqs)
    width = max(pages)
    ids = 1 + torch.randperm(num_pages - 1, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(reqs), width), -1, dtype=torch.int32)
    ids = ids.cpu()
    at = 0
    for i, n in enumerate(pages):
        table[i, :n] = ids[at:at + n]
        at += n
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)
    loc, total = [0], 0
    for r in reqs:
        total += r["q"]
        loc.append(total)
    i32 = lambda xs: torch.tensor(xs, dtype=torch.int32).cuda()
    s = {"op": "attention", "case": case, "reqs": reqs, "tokens": tokens, "num_pages": num_pages,
         "q": 3.0 * randn(tokens, nh, hd), "k": randn(num_pages * PAGE, nkv, hd),
         "v": randn(num_pages * PAGE, nkv, hd), "table": table.cuda(), "loc": i32(loc),
         "lens": i32([r["c"] + r["q"] for r in reqs]), "width": width,
         "slopes": None, "starts": None, "prefix": None}
    if case["slopes"]:
        s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / nh) for h in range(nh)],
                                   dtype=torch.float32).cuda()
    if _uses_starts(case):
        s["starts"] = i32([x for r in reqs for x in r["starts"]])
    if case["prefix"]:
        s["prefix"] = i32([r["prefix"] for r in reqs])
    # the order in which the plain form takes the requests
    length = lambda i: reqs[i]["c"] + reqs[i]["q"]
    order = sorted((i for i, r in enumerate(reqs) if r["q"] == 1), key=length)
    groups = [order[a:a + 16] for a in range(0, len(order), 16)]
    s["singles"] = [(torch.tensor(x).cuda(), torch.tensor([[loc[i]] for i in x]).cuda(),
                     length(x[-1])) for x in groups]
    s["chunks"] = [(torch.tensor([i]).cuda(), loc[i], r["q"], length(i))
                   for i, r in enumerate(reqs) if r["q"] > 1]
    if own:
        import ragged_mixed_paged_gb300 as rb

        s["dims"] = rb.Dims(block_size=PAGE, num_q_heads=nh, num_kv_heads=nkv, head_dim=hd,
                            max_num_reqs=len(reqs), max_model_len=width * PAGE,
                            max_blocks_per_req=width, num_blocks=num_pages)
        s["rules"] = rb.ScoreRules(softcap=case["softcap"], head_slopes=s["slopes"],
                                   key_start=s["starts"], prefix_lens=s["prefix"])
        s["workspace"] = torch.empty(rb.workspace_size(s["dims"], len(reqs), tokens),
                                     dtype=torch.uint8, device="cuda")
        s["out"] = torch.empty_like(s["q"])
        s["error"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


def _run_attention(s):
    case = s["case"]
    nh, nkv, hd = case["nh"], case["nkv"], case["hd"]
    if own:
        import ragged_mixed_paged_gb300 as rb

        return rb.paged_attention_scored(s["dims"], len(s["reqs"]), s["tokens"], s["q"], s["k"],
                                         s["v"], s["table"], s["loc"], s["lens"], s["rules"],
                                         out=s["out"], workspace=s["workspace"],
                                         error_word=s["error"])
    out = torch.empty_like(s["q"])
    kp = s["k"].view(s["num_pages"], PAGE, nkv, hd)
    vp = s["v"].view(s["num_pages"], PAGE, nkv, hd)

    def attend(rows, tokens, length):
        """Requests `rows` (a tensor of B of them) with n new tokens each, whose flat indices
        are `tokens` [B, n]; keys [0, length) of each."""
        ids = s["table"][rows, :-(-length // PAGE)].long().clamp(min=0)
        k = kp[ids].flatten(1, 2)[:, :length].float().permute(0, 2, 3, 1)  # [B, nkv, hd, L]
        v = vp[ids].flatten(1, 2)[:, :length].float().permute(0, 2, 1, 3)  # [B, nkv, L, hd]
        n = tokens.shape[1]
        q = s["q"][tokens].float().view(-1, n, nkv, nh // nkv, hd).permute(0, 2, 3, 1, 4)
        x = torch.matmul(q.flatten(2, 3), k) / math.sqrt(hd)
        x = x.view(len(rows), nh, n, length)
        if case["softcap"]:
            x = case["softcap"] * torch.tanh(x / case["softcap"])
        lens = s["lens"][rows].long()[:, None]
        pos = tokens - s["loc"][rows + 1].long()[:, None] + lens  # position of each new token
        key = torch.arange(length, device="cuda")
        if s["slopes"] is not None:
            dist = (pos[:, :, None] - key).abs().float()
            x = x - s["slopes"].view(nh, 1, 1) * dist[:, None]
        upper = pos + 1
        if s["prefix"] is not None:
            upper = torch.minimum(torch.maximum(upper, s["prefix"][rows].long()[:, None]), lens)
        keep = key < upper[:, :, None]
        if s["starts"] is not None:
            keep &= key >= s["starts"][tokens].long()[:, :, None]
        x = x.masked_fill(~keep[:, None], -math.inf)
        m = x.amax(-1, keepdim=True)
        e = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
        total = e.sum(-1, keepdim=True)
        p = e / torch.where(total > 0, total, torch.ones_like(total))
        o = torch.matmul(p.view(len(rows), nkv, -1, length), v)
        o = o.view(len(rows), nh, n, hd).transpose(1, 2)
        out[tokens] = o.to(out.dtype)

    # requests with one new token, sixteen of about the same length at a time
    for rows, tokens, length in s["singles"]:
        attend(rows, tokens, length)
    for row, first, q, length in s["chunks"]:
        step = max(1, (1 << 29) // (nh * length))
        for lo in range(first, first + q, step):
            attend(row, torch.arange(lo, min(first + q, lo + step), device="cuda")[None], length)
    return out


def _exact_attention(case, seed):
    s = _prepare_attention(case, seed)
    nh, nkv, hd = case["nh"], case["nkv"], case["hd"]
    if _attention_work(case)["flops"] > 4e12:
        return None
    out = torch.zeros(s["tokens"], nh, hd, dtype=torch.float64, device="cuda")
    first = 0
    for i, r in enumerate(s["reqs"]):
        length = r["c"] + r["q"]
        where = torch.arange(length, device="cuda")
        slot = s["table"][i].long()[where // PAGE] * PAGE + where % PAGE
        seen = _visible(r)
        for h in range(nh):
            kk = s["k"][slot, h * nkv // nh].double()
            vv = s["v"][slot, h * nkv // nh].double()
            rows = max(1, (1 << 27) // length)
            for a in range(0, r["q"], rows):
                b = min(r["q"], a + rows)
                y = s["q"][first + a:first + b, h].double() @ kk.t() / math.sqrt(hd)
                if case["softcap"]:
                    y = torch.tanh(y / case["softcap"]) * case["softcap"]
                lo = torch.tensor([x for x, _ in seen[a:b]], device="cuda").unsqueeze(1)
                hi = torch.tensor([x for _, x in seen[a:b]], device="cuda").unsqueeze(1)
                if case["slopes"]:
                    own_pos = torch.arange(r["c"] + a, r["c"] + b, device="cuda").unsqueeze(1)
                    y -= float(s["slopes"][h]) * torch.abs(where - own_pos)
                w = torch.where((where >= lo) & (where < hi), y,
                                torch.full((), -math.inf, dtype=torch.float64, device="cuda"))
                w = torch.nan_to_num(torch.softmax(w, 1), nan=0.0)  # a row without keys is zero
                out[first + a:first + b, h] = w @ vv
        first += r["q"]
    return out


def _attention_work(case):
    reqs = _requests(case)
    nh, nkv, hd = case["nh"], case["nkv"], case["hd"]
    pairs = keys = tokens = 0
    for r in reqs:
        seen = _visible(r)
        tokens += r["q"]
        pairs += sum(max(0, hi - lo) for lo, hi in seen)
        some = [(lo, hi) for lo, hi in seen if hi > lo]
        if some:
            keys += max(hi for _, hi in some) - min(lo for lo, _ in some)
    rules = 4 * tokens * _uses_starts(case) + 4 * len(reqs) * case["prefix"] + \
        4 * nh * case["slopes"]
    return {"bytes": 2 * 2 * tokens * nh * hd + 2 * 2 * keys * nkv * hd + 4 * -(-keys // PAGE) +
            8 * len(reqs) + rules, "flops": 4 * hd * nh * pairs}


# ------------------------------------------------------------------------------------- pages
def _rows(case):
    """Cached tokens of each row of the page table (0: the row holds no request), the forks or
    the freed rows, and the pages that rows share."""
    rng = random.Random(case["layout"])
    rows = case["rows"]
    if case["op"] == "fork":
        order = list(range(rows))
        rng.shuffle(order)
        src = order[:case["sources"]]
        dst = order[case["sources"]:case["sources"] + case["forks"]]
        cached = [0] * rows
        for r in src:
            cached[r] = rng.randint(case["c_min"], case["c_max"])
        return cached, [src[i % len(src)] for i in range(len(dst))], dst
    cached = [rng.randint(case["c_min"], case["c_max"]) for _ in range(rows)]
    return cached, rng.sample(range(rows), case["free"]), []


def _prepare_pages(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    nkv, hd = case["nkv"], case["hd"]
    s = {"op": case["op"], "case": case}
    i32 = lambda xs: torch.tensor(xs, dtype=torch.int32).cuda()
    if case["op"] == "copy":
        pages, n, width, rows = case["pages"], case["pairs"], 1, 1
        ids = 1 + torch.randperm(pages - 1, generator=host)
        s["src"] = ids[:n].to(torch.int32)
        s["src"][n // 2:n // 2 + n // 8] = s["src"][0]  # one page copied to many
        s["src"], s["dst"] = s["src"].cuda(), ids[n:2 * n].to(torch.int32).cuda()
    else:
        cached, first, second = _rows(case)
        rows = case["rows"]
        entries = [-(-c // PAGE) for c in cached]
        width = max(1, max(entries))
        shared = case["op"] == "compact"
        pages = 1 + sum(entries) + case["spare"]
        ids = (1 + torch.randperm(pages - 1, generator=host)).to(torch.int32)
        table = torch.full((rows, width), -1, dtype=torch.int32)
        at = 0
        for r, n in enumerate(entries):
            table[r, :n] = ids[at:at + n]
            if shared and r % 3 == 1:  # every third row shares the full pages of the row before
                common = min(cached[r - 1], cached[r]) // PAGE
                table[r, :common] = table[r - 1, :common]
            at += n
        count = torch.zeros(pages, dtype=torch.int32)
        held = table[table >= 0].long()
        count.scatter_add_(0, held, torch.ones_like(held, dtype=torch.int32))
        s["saved"] = torch.cat([table.flatten(), torch.tensor(entries, dtype=torch.int32),
                                count]).cuda()
        live = s["live"] = s["saved"].clone()
        s["table"] = live[:rows * width].view(rows, width)
        s["entries"] = live[rows * width:rows * width + rows]
        s["count"] = live[rows * width + rows:]
        s["cached"] = i32(cached)
        if case["op"] == "fork":
            s["src"], s["dst"] = i32(first), i32(second)
        else:
            s["free"] = i32(first)
            s["map"] = torch.empty(pages, dtype=torch.int32, device="cuda")
            s["totals"] = torch.zeros(2, dtype=torch.int32, device="cuda")
    s["num_pages"] = pages
    for name in ("k", "v"):
        s[name] = torch.randn(pages * PAGE, nkv, hd, generator=g, device="cuda",
                              dtype=torch.bfloat16)
    if own:
        import ragged_mixed_paged_gb300 as rb

        dims = rb.Dims(block_size=PAGE, num_q_heads=nkv, num_kv_heads=nkv, head_dim=hd,
                       max_num_reqs=rows, max_model_len=width * PAGE, max_blocks_per_req=width,
                       num_blocks=pages)
        s["pool"] = rb.PagePool(dims, s["k"], s["v"], s.get("table"), s.get("entries"),
                                ref_count=s.get("count"))
    return s


def _run_copy(s):
    if own:
        s["pool"].copy(s["src"], s["dst"])
        return s["k"], s["v"]
    for name in ("k", "v"):
        page = s[name].view(s["num_pages"], -1)
        page[s["dst"].long()] = page[s["src"].long()]
    return s["k"], s["v"]


def _run_fork(s):
    s["live"].copy_(s["saved"])  # the tables as they stand before the call
    if own:
        s["pool"].fork(s["src"], s["dst"], s["cached"])
        return s["table"], s["entries"], s["count"], s["k"], s["v"]
    src, dst = s["src"].long(), s["dst"].long()
    table, count = s["table"], s["count"]
    c = s["cached"][src].long()
    full, tail = c // PAGE, c % PAGE
    column = torch.arange(table.shape[1], device="cuda")
    old = table[src].long()
    # lowest free pages, one for each fork that ends inside a page
    number = torch.arange(s["num_pages"], device="cuda")
    free = torch.nonzero((count == 0) & (number != 0)).flatten()
    needs = tail > 0
    fresh = free[(torch.cumsum(needs, 0) - 1).clamp(0, max(free.numel() - 1, 0))]
    share = column[None, :] < full[:, None]
    last = (column[None, :] == full[:, None]) & needs[:, None]
    table[dst] = torch.where(share, old, torch.where(last, fresh[:, None],
                                                     table[dst].long())).to(torch.int32)
    s["entries"][dst] = (full + needs).to(torch.int32)
    held = torch.where(share, old, torch.where(last, fresh[:, None], torch.zeros_like(old)))
    count.scatter_add_(0, held.flatten(), (share | last).flatten().to(torch.int32))
    row = torch.arange(PAGE, device="cuda")
    at = torch.nonzero(needs).flatten()
    origin = old[at, full[at]] * PAGE
    target = fresh[at] * PAGE
    keep = row[None, :] < tail[at][:, None]
    a = (origin[:, None] + row)[keep]
    b = (target[:, None] + row)[keep]
    for name in ("k", "v"):
        s[name][b] = s[name][a]
    return table, s["entries"], count, s["k"], s["v"]


def _run_compact(s):
    s["live"].copy_(s["saved"])
    if own:
        s["pool"].free(s["free"], num_freed=s["totals"][:1])
        s["pool"].compact(page_map=s["map"], num_live=s["totals"][1:])
        return (s["table"], s["entries"], s["count"], s["map"], s["totals"], s["k"], s["v"])
    table, count = s["table"], s["count"]
    rows = s["free"].long()
    column = torch.arange(table.shape[1], device="cuda")
    held = column[None, :] < s["entries"][rows].long()[:, None]
    ids = table[rows].long()
    before = count > 0
    count.scatter_add_(0, torch.where(held, ids, torch.zeros_like(ids)).flatten(),
                       -held.flatten().to(torch.int32))
    table[rows] = torch.where(held, torch.full_like(ids, -1), ids).to(torch.int32)
    s["entries"][rows] = 0
    s["totals"][0] = (before & (count == 0)).sum()
    number = torch.arange(s["num_pages"], device="cuda")
    live = (count > 0) & (number != 0)
    n = live.sum()
    s["totals"][1] = n
    low = (number >= 1) & (number <= n)  # where the live pages end up
    movers = torch.nonzero(live & ~low).flatten()
    holes = torch.nonzero(low & ~live).flatten()
    page_map = torch.where(live, number, torch.full_like(number, -1))
    page_map[0] = 0
    page_map[movers] = holes
    for name in ("k", "v"):
        page = s[name].view(s["num_pages"], -1)
        page[holes] = page[movers]
    count[holes] = count[movers]
    count[movers] = 0
    held = column[None, :] < s["entries"].long()[:, None]
    table.copy_(torch.where(held, page_map[table.long().clamp(min=0)], table.long()))
    s["map"].copy_(page_map)
    return (table, s["entries"], count, s["map"], s["totals"], s["k"], s["v"])


def _exact_pages(case, seed):
    """The page operators by their definition, one request and one page at a time."""
    s = _prepare_pages(case, seed)
    pools = [s[name].view(s["num_pages"], PAGE, -1) for name in ("k", "v")]
    if case["op"] == "copy":
        src, dst = s["src"].tolist(), s["dst"].tolist()
        origin = list(range(s["num_pages"]))
        for a, b in zip(src, dst):
            origin[b] = a
        pick = torch.tensor(origin, device="cuda")
        return tuple(p[pick].view(-1, case["nkv"], case["hd"]).double() for p in pools)
    table = s["table"].tolist()
    entries, count = s["entries"].tolist(), s["count"].tolist()
    i32 = lambda xs: torch.tensor(xs, dtype=torch.int32, device="cuda")
    flat = lambda p: p.view(-1, case["nkv"], case["hd"])
    if case["op"] == "fork":
        cached = s["cached"].tolist()
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            full, tail = divmod(cached[a], PAGE)
            for j in range(full):
                table[b][j] = table[a][j]
                count[table[a][j]] += 1
            if tail:
                page = next(i for i in range(1, len(count)) if count[i] == 0)
                count[page] = 1
                table[b][full] = page
                for p in pools:
                    p[page, :tail] = p[table[a][full], :tail]
            entries[b] = full + (tail > 0)
        return (i32(table), i32(entries), i32(count)) + tuple(flat(p).double() for p in pools)
    freed = 0
    for r in s["free"].tolist():
        for j in range(entries[r]):
            count[table[r][j]] -= 1
            freed += count[table[r][j]] == 0
            table[r][j] = -1
        entries[r] = 0
    live = [i for i in range(1, len(count)) if count[i] > 0]
    holes = [i for i in range(1, len(live) + 1) if count[i] == 0]
    page_map = [0] + [i if count[i] > 0 else -1 for i in range(1, len(count))]
    origin = list(range(len(count)))
    for a, b in zip([i for i in live if i > len(live)], holes):
        page_map[a] = b
        origin[b] = a
        count[b], count[a] = count[a], 0
    for r, n in enumerate(entries):
        for j in range(n):
            table[r][j] = page_map[table[r][j]]
    pick = torch.tensor(origin, device="cuda")
    return (i32(table), i32(entries), i32(count), i32(page_map), i32([freed, len(live)])) + \
        tuple(flat(p[pick]).double() for p in pools)


def _pages_work(case):
    page = 2 * PAGE * case["nkv"] * case["hd"] * 2  # K and V of one page
    if case["op"] == "copy":
        n = case["pairs"]
        return {"bytes": page * (2 * n - n // 8) + 8 * n, "flops": 0}
    cached, first, second = _rows(case)
    entries = [-(-c // PAGE) for c in cached]
    rows = case["rows"]
    if case["op"] == "fork":
        tails = sum(cached[a] % PAGE for a in first)
        shared = sum(-(-cached[a] // PAGE) for a in first)
        read = sum(cached[a] % PAGE for a in set(first))
        table = sum(entries[a] for a in set(first))
        return {"bytes": (page // PAGE) * (tails + read) + 4 * (table + 3 * shared) +
                16 * len(first), "flops": 0}
    # pages that are live after the frees, and how many of them lie above the packed region:
    # page ids are a random permutation, so the expected share is that of the free pages below
    pages = 1 + sum(entries) + case["spare"]
    freed = set(first)
    owner = {}
    at = 0
    table = []
    for r, n in enumerate(entries):
        line = list(range(at, at + n))
        if r % 3 == 1:
            common = min(cached[r - 1], cached[r]) // PAGE
            line[:common] = table[r - 1][:common]
        table.append(line)
        at += n
        if r not in freed:
            owner.update(dict.fromkeys(line))
    live = len(owner)
    moved = live * (pages - 1 - live) // (pages - 1)
    left = sum(entries[r] for r in range(rows) if r not in freed)
    gone = sum(entries[r] for r in freed)
    return {"bytes": 2 * page * moved + 4 * (2 * left + 2 * gone + 3 * pages + 2 * rows),
            "flops": 0}


# ---------------------------------------------------------------------------------- logprobs
def _prepare_logprobs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows, vocab, stride = case["rows"], case["vocab"], case["stride"]
    x = torch.randn(rows, stride, generator=g, device="cuda")
    # flat rows and sharp ones, as a model's logits are
    x *= 0.5 + 3.0 * torch.rand(rows, 1, generator=g, device="cuda")
    tokens = torch.randint(vocab, (rows,), generator=g, device="cuda")
    best = x[:, :vocab].argmax(1)
    pick = torch.rand(rows, generator=g, device="cuda") < 0.6  # mostly likely tokens
    tokens = torch.where(pick, best, tokens).to(torch.int32)
    if case["banned"]:
        for lo in range(0, rows, 256):
            part = x[lo:lo + 256]
            ban = torch.rand(part.shape, generator=g, device="cuda") < 0.3
            ban[::2] = False  # every other row is free
            part.masked_fill_(ban, -math.inf)
    x = x.to(LOG_DTYPES[case["dtype"]])
    s = {"op": "logprobs", "case": case, "logits": x[:, :vocab], "tokens": tokens}
    if own:
        import ragged_mixed_paged_gb300 as rb

        s["out"] = rb.TokenLogprobs.allocate(rows, case["top"], "cuda")
        s["error"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


def _run_logprobs(s):
    top = s["case"]["top"]
    if own:
        import ragged_mixed_paged_gb300 as rb

        o = rb.token_logprobs(s["logits"], s["tokens"], top, out=s["out"],
                              error_word=s["error"])
        return o.logprobs, o.ranks, o.entropy, o.top_ids, o.top_logprobs
    vocab = s["case"]["vocab"]
    step = max(1, (1 << 28) // vocab)
    parts = []
    for lo in range(0, s["case"]["rows"], step):
        x = s["logits"][lo:lo + step].float()
        t = s["tokens"][lo:lo + step].long()[:, None]
        m = x.amax(1, keepdim=True)
        d = x - m
        e = torch.exp(d)
        total = e.sum(1, keepdim=True, dtype=torch.float64)
        log_total = torch.log(total)
        mine = torch.gather(x, 1, t)
        logprob = (mine - m) - log_total
        rank = 1 + (x > mine).sum(1)
        mean = torch.where(e > 0, e * d, torch.zeros_like(e)).sum(1, dtype=torch.float64)
        entropy = log_total.flatten() - mean / total.flatten()
        if top:
            order = torch.sort(x, dim=1, descending=True, stable=True)
            ids = order.indices[:, :top]
            best = (order.values[:, :top] - m) - log_total
        else:
            ids = torch.zeros(x.shape[0], 0, device="cuda")
            best = ids
        if ids.shape[1] < top:
            ids = torch.nn.functional.pad(ids, (0, top - ids.shape[1]), value=-1)
            best = torch.nn.functional.pad(best, (0, top - best.shape[1]), value=-math.inf)
        parts.append((logprob.flatten().float(), rank.to(torch.int32), entropy.float(),
                      ids.to(torch.int32), best.float()))
    return tuple(torch.cat(x) for x in zip(*parts))


def _exact_logprobs(case, seed):
    s = _prepare_logprobs(case, seed)
    rows, vocab, top = case["rows"], case["vocab"], case["top"]
    if rows * vocab > 400_000_000:
        return None
    out = [[], [], [], [], []]
    block = max(1, (1 << 26) // vocab)
    for a in range(0, rows, block):
        x = s["logits"][a:a + block].double()
        t = s["tokens"][a:a + block].long()
        lse = torch.logsumexp(x, 1)
        lp = x - lse[:, None]
        mine = lp[torch.arange(lp.shape[0], device="cuda"), t]
        xm = x[torch.arange(lp.shape[0], device="cuda"), t]
        out[0].append(mine)
        out[1].append(((x > xm[:, None]).sum(1) + 1).to(torch.int32))
        out[2].append(-torch.special.xlogy(torch.exp(lp), torch.exp(lp)).sum(1))
        ids = torch.full((x.shape[0], top), -1, dtype=torch.int32, device="cuda")
        best = torch.full((x.shape[0], top), -math.inf, dtype=torch.float64, device="cuda")
        rest = x.clone()
        index = torch.arange(vocab, device="cuda")
        taken = torch.zeros_like(rest, dtype=torch.bool)
        for j in range(min(top, vocab)):  # repeatedly the largest left, lowest index first
            high = torch.where(taken, -math.inf, rest).amax(1, keepdim=True)
            at = torch.where((rest == high) & ~taken, index, vocab).amin(1)
            ids[:, j] = at.to(torch.int32)
            best[:, j] = torch.gather(lp, 1, at[:, None]).flatten()
            taken.scatter_(1, at[:, None], True)
        out[3].append(ids)
        out[4].append(best)
    return tuple(torch.cat(o) for o in out)


def _logprobs_work(case):
    rows, vocab, top = case["rows"], case["vocab"], case["top"]
    size = 4 if case["dtype"] == "fp32" else 2
    # one exponential, its sum, the sum weighted by the logit (a product) and the comparisons
    # with the token and with the top alternatives' threshold: 6 operations an element
    return {"bytes": rows * vocab * size + 4 * rows + rows * (12 + 8 * top),
            "flops": 6 * rows * vocab}


# --------------------------------------------------------------------------------- interface
_PREPARE = {"attention": _prepare_attention, "copy": _prepare_pages, "fork": _prepare_pages,
            "compact": _prepare_pages, "logprobs": _prepare_logprobs}
_RUN = {"attention": _run_attention, "copy": _run_copy, "fork": _run_fork,
        "compact": _run_compact, "logprobs": _run_logprobs}
_EXACT = {"attention": _exact_attention, "copy": _exact_pages, "fork": _exact_pages,
          "compact": _exact_pages, "logprobs": _exact_logprobs}
_WORK = {"attention": _attention_work, "copy": _pages_work, "fork": _pages_work,
         "compact": _pages_work, "logprobs": _logprobs_work}


def prepare(case, seed):
    return _PREPARE[case["op"]](case, seed)


def run(state):
    return _RUN[state["op"]](state)


def exact(case, seed):
    return _EXACT[case["op"]](case, seed)


def work(case):
    return _WORK[case["op"]](case)
