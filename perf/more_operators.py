"""Operators of a serving step around the scaled GEMMs and the paged cache: cases, plain forms, 64-bit values.

norm     a residual's addition, root-mean-square norm and quantisation to the codes and scales that the
         next scaled GEMM reads (ptpc, blockscale, mxfp8; bf16: no codes).
chunk    attention of chunks of new tokens, as many for each sequence as there are, over the paged e4m3 cache
         that holds them and what came before.
fork     pages of that cache among sequences: finished sequences are released, others forked (whole pages are
         shared, the last one is copied where it is not full), and all grow by some tokens.
compact  the pages in use are moved to the lowest numbers and the block tables follow.

The cache is [pages][Hk][page][D] codes and [pages][Hk][page / 16] e8m0 scales, in each layer; a
sequence's pages are listed in its row of the block table, and refs counts the rows that list a page.

``own`` False: elementary torch operations in fp32.  ``own`` True: the calls of
``fp8_scaled_gemm_sm_gb300``.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 16      # tokens that share a scale
NAN_CODE = 0x7F
EPS = 1e-6


# --------------------------------------------------------------------------- cases


def listed():
    return [
        # the norm before a projection in a decode step of one sequence: a launch and little else
        dict(name="norm_token", op="norm", mode="ptpc", rows=1, cols=7168, dtype="bf16", lens=1),
        # ragged tokens of a mixed step, a residual stream in fp32
        dict(name="norm_step_777", op="norm", mode="mxfp8", rows=777, cols=2048, dtype="f32", lens=2),
        # a whole prompt
        dict(name="norm_prompt_32768", op="norm", mode="blockscale", rows=32768, cols=7168, dtype="bf16", lens=3),
        # one short question behind a shared prompt
        dict(name="chunk_question", op="chunk", B=1, q_lo=24, q_hi=24, ctx_lo=900, ctx_hi=900, idle=0, hq=32, hk=8, d=128, page=64, lens=4),
        # a step of a server that mixes single tokens, drafts and pieces of prompts; small pages, five heads a group
        dict(name="chunk_mixed_40", op="chunk", B=40, q_lo=1, q_hi=300, ctx_lo=0, ctx_hi=9000, idle=2, hq=40, hk=8, d=128, page=16, lens=5),
        # few questions to very long documents: the work has to be split along the keys
        dict(name="chunk_documents_2", op="chunk", B=2, q_lo=101, q_hi=256, ctx_lo=120001, ctx_hi=130000, idle=0, hq=64, hk=8, d=128, page=128, lens=6),
        # ungrouped 64-wide heads
        dict(name="chunk_ungrouped_24", op="chunk", B=24, q_lo=5, q_hi=700, ctx_lo=1, ctx_hi=4000, idle=0, hq=16, hk=16, d=64, page=32, lens=7),
        # pieces of long prompts
        dict(name="chunk_prompts_4", op="chunk", B=4, q_lo=1000, q_hi=2048, ctx_lo=4000, ctx_hi=24000, idle=0, hq=32, hk=8, d=128, page=64, lens=8),
        # beams of one prompt: some end, others branch
        dict(name="fork_beams", op="fork", rows=16, keep=4, drop=4, children=8, len_lo=300, len_hi=2000, add_hi=1, spare=40, hk=8, d=128,
             page=64, layers=4, lens=9),
        # many answers to each of some prompts, in a model's every layer
        dict(name="fork_answers", op="fork", rows=160, keep=8, drop=70, children=96, len_lo=40, len_hi=2500, add_hi=40, spare=400, hk=8,
             d=128, page=128, layers=12, lens=10),
        # a small pool after its sequences ended
        dict(name="compact_small", op="compact", rows=12, len_lo=10, len_hi=300, used=0.6, hk=4, d=64, page=16, layers=2, lens=11),
        # a large one with holes all over
        dict(name="compact_large", op="compact", rows=300, len_lo=100, len_hi=6000, used=0.5, hk=8, d=128, page=64, layers=3, lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "chunk", "chunk", "fork", "compact"])
    c = dict(op=op, lens=rng.randrange(1 << 20))
    if op == "norm":
        mode = rng.choice(["ptpc", "blockscale", "mxfp8", "bf16"])
        cols = max(1, _log(rng, 128, 16384) // 128) * 128
        if mode in ("ptpc", "bf16"):
            cols += rng.choice([0, 16, 112])
        c.update(mode=mode, rows=_log(rng, 1, min(40000, 200_000_000 // cols)), cols=cols, dtype=rng.choice(["bf16", "bf16", "f32"]))
        return c
    hk = rng.choice([1, 2, 4, 8, 16])
    c.update(hk=hk, d=rng.choice([64, 96, 128, 128]), page=rng.choice([16, 32, 64, 128]))
    if op == "chunk":
        c["hq"] = hk * rng.choice([1, 2, 3, 4, 5, 7, 8, 16] if hk <= 4 else [1, 2, 4, 5, 7])
        B = _log(rng, 1, 100)
        q_hi = min(_log(rng, 1, 4000), int((1.5e9 / (B * c["hq"])) ** 0.5))
        ctx_hi = min(_log(rng, 16, 131072), int(1.5e9 / (B * c["hq"] * q_hi)), int(4e8 / (B * hk * c["d"])))
        c.update(B=B, q_lo=max(1, q_hi // rng.choice([1, 4, 60])), q_hi=q_hi, ctx_lo=ctx_hi // rng.choice([1, 3, 50]), ctx_hi=ctx_hi,
                 idle=rng.choice([0, 0, 1]) if B > 1 else 0)
        return c
    layers, rows = rng.choice([1, 2, 5, 8]), _log(rng, 4, 150)
    bytes_ = 2 * layers * hk * c["d"]                          # of a token
    hi = max(20, min(_log(rng, 20, 20000), int(2.5e9 / (bytes_ * rows))))
    c.update(rows=rows, layers=layers, len_lo=max(1, hi // rng.choice([2, 10, 100])), len_hi=hi)
    if op == "compact":
        c["used"] = rng.choice([0.3, 0.6, 0.9])
    else:
        keep = max(1, rows // rng.choice([3, 8]))
        drop = rng.randint(0, rows - keep - 1)
        c.update(keep=keep, drop=drop, children=rng.randint(1, rows - keep), add_hi=rng.choice([1, 7, 200]),
                 spare=rng.choice([rows // 2 + 1, rows * (2 + 200 // c["page"])]))  # the first may run out
    return c


def _lens(case, n, lo, hi, salt):
    """n lengths spread over their logarithm; the first is the longest."""
    rng = random.Random(case["lens"] * 8 + salt)
    if n == 0:
        return []
    return [hi] + [lo if lo == hi else (_log(rng, max(lo, 1), hi) if lo else rng.randint(lo, hi)) for _ in range(n - 1)]


def _chunk_lens(case):
    """New tokens of each sequence, and all of its tokens in the cache; some slots idle."""
    new = _lens(case, case["B"], case["q_lo"], case["q_hi"], 1)
    ctx = _lens(case, case["B"], case["ctx_lo"], case["ctx_hi"], 2)
    for i in range(1, 1 + case["idle"]):
        new[i] = 0
    return new, [a + b for a, b in zip(new, ctx)]


def _rows_of(case):
    """Of a fork: lengths of all rows, then the kept, dropped, source and destination rows and what each row grows by."""
    rng = random.Random(case["lens"] * 8 + 3)
    order = list(range(case["rows"]))
    rng.shuffle(order)
    keep, drop, empty = order[:case["keep"]], order[case["keep"]:case["keep"] + case["drop"]], order[case["keep"] + case["drop"]:]
    lens = [0] * case["rows"]
    for r, n in zip(keep + drop, _lens(case, len(keep + drop), case["len_lo"], case["len_hi"], 4)):
        lens[r] = n
    dst = (drop + empty)[:case["children"]]
    rng.shuffle(dst)
    src = [keep[0]] + [rng.choice(keep) for _ in dst[1:]]
    live = keep + dst
    return lens, drop, src, dst, live, [rng.randint(1, case["add_hi"]) for _ in live]


# --------------------------------------------------------------------------- inputs


def _ints(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def _cum(lens, dev):
    return _ints(np.concatenate([[0], np.cumsum(lens)]).tolist(), dev)


def _table(lens, page, width, pages, gen, dev):
    """A block table over shuffled pages, unused entries -1."""
    need = [-(-n // page) for n in lens]
    ids = torch.randperm(pages, generator=gen, device=dev)[:sum(need)].to(torch.int32)
    at = torch.arange(width, device=dev)[None, :] < torch.tensor(need, device=dev)[:, None]
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=dev)
    table[at] = ids
    return table


def _bytes(shape, gen, dev):
    """Codes of all values but NaN."""
    x = torch.randint(0, 256, shape, generator=gen, device=dev, dtype=torch.uint8)
    return torch.where((x & 127) == NAN_CODE, torch.zeros_like(x), x)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev)
    gen.manual_seed(seed * 1000003 + case["lens"])
    s = {"norm": _prepare_norm, "chunk": _prepare_chunk, "fork": _prepare_fork, "compact": _prepare_compact}[case["op"]](case, gen, dev)
    s["case"] = case
    if own and case["op"] != "norm":
        from fp8_scaled_gemm_sm_gb300 import KVCache, PagedAttention, PagePool

        s["plan"] = PagedAttention(case.get("hq", case["hk"]), case["hk"], case["d"], page_size=case["page"])
        if case["op"] == "chunk":
            s["cache"] = KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        else:
            layers = [KVCache(*(s[n][i] for n in ("k", "v", "k_scale", "v_scale"))) for i in range(case["layers"])]
            s["pool"] = PagePool(s["plan"], layers, s["table"], s["lens"], s["refs"])
    return s


def _prepare_norm(case, gen, dev):
    """A projection's output and the residual stream, some channels of which are far larger than others; rows of different sizes."""
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    R, C = case["rows"], case["cols"]
    wide = torch.exp(0.8 * torch.randn(C, generator=gen, device=dev))
    rows = torch.exp(0.5 * torch.randn(R, 1, generator=gen, device=dev))
    x = (torch.randn(R, C, generator=gen, device=dev) * rows).to(dt)
    r = (torch.randn(R, C, generator=gen, device=dev) * (3 * wide)).to(dt)
    w = (1 + 0.3 * torch.randn(C, generator=gen, device=dev)).to(dt)
    return dict(x=x, residual=r, weight=w)


def _prepare_chunk(case, gen, dev):
    """The cache after the new tokens were appended: normal values at their blocks' scales, stale bytes of all kinds behind the sequences."""
    new, lens = _chunk_lens(case)
    hk, page, d = case["hk"], case["page"], case["d"]
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 3
    table = _table(lens, page, max(max(need), 1), pages, gen, dev)
    scales = [torch.randint(115, 123, (pages, hk, page // BLOCK), generator=gen, device=dev, dtype=torch.uint8) for _ in range(2)]
    rows = torch.arange(case["B"], device=dev)
    last = torch.tensor([max(n - 1, 0) for n in lens], device=dev)
    live = torch.tensor([n > 0 for n in lens], device=dev)
    end = table[rows, last // page].long()[live]
    dead = (torch.arange(page, device=dev)[None, :] > (last % page)[:, None])[live]
    codes = []
    for _ in range(2):
        c = torch.empty((pages, hk, page, d), dtype=torch.uint8, device=dev)
        for i in range(0, pages, 4096):
            x = torch.randn(c[i:i + 4096].shape, generator=gen, device=dev) * 110
            c[i:i + 4096] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        c[end] = c[end].masked_fill(dead[:, None, :, None], NAN_CODE)
        codes.append(c)
    q = (torch.randn(sum(new), case["hq"], d, generator=gen, device=dev) * 2).to(torch.bfloat16)
    return dict(q=q, k=codes[0], v=codes[1], k_scale=scales[0], v_scale=scales[1], table=table, lens=_ints(lens, dev), cu=_cum(new, dev),
                max_q=max(new))


def _pool(case, lens, pages, width, gen, dev):
    """Layers of a cache whose sequences hold `lens` tokens."""
    hk, page, d, layers = case["hk"], case["page"], case["d"], case["layers"]
    s = dict(k=_bytes((layers, pages, hk, page, d), gen, dev), v=_bytes((layers, pages, hk, page, d), gen, dev))
    for n in ("k_scale", "v_scale"):
        s[n] = torch.randint(100, 140, (layers, pages, hk, page // BLOCK), generator=gen, device=dev, dtype=torch.uint8)
    s["table0"] = _table(lens, page, width, pages, gen, dev)
    s["lens0"] = _ints(lens, dev)
    s["refs0"] = torch.zeros(pages, dtype=torch.int32, device=dev)
    s["refs0"][s["table0"][s["table0"] >= 0].long()] = 1
    for n in ("table", "lens", "refs"):
        s[n] = s[n + "0"].clone()
    return s


def _prepare_fork(case, gen, dev):
    lens, drop, src, dst, live, add = _rows_of(case)
    page = case["page"]
    pages = sum(-(-n // page) for n in lens) + case["spare"]
    width = -(-(max(lens) + case["add_hi"]) // page)
    s = _pool(case, lens, pages, width, gen, dev)
    s.update(drop=_ints(drop, dev), src=_ints(src, dev), dst=_ints(dst, dev), live=_ints(live, dev), add=_ints(add, dev))
    return s


def _prepare_compact(case, gen, dev):
    lens = _lens(case, case["rows"], case["len_lo"], case["len_hi"], 5)
    need = [-(-n // case["page"]) for n in lens]
    return _pool(case, lens, int(sum(need) / case["used"]) + 1, max(need), gen, dev)


# --------------------------------------------------------------------------- one pass


def run(s):
    case = s["case"]
    op = case["op"]
    if op in ("fork", "compact"):
        for n in ("table", "lens", "refs"):  # the state before the pass
            s[n].copy_(s[n + "0"])
    if not own:
        return {"norm": _plain_norm, "chunk": _plain_chunk, "fork": _plain_fork, "compact": _plain_compact}[op](s)
    if op == "norm":
        from fp8_scaled_gemm_sm_gb300 import norm_quantize

        return _norm_out(case, *norm_quantize(case["mode"], s["x"], s["weight"], EPS, residual=s["residual"]))
    if op == "chunk":
        out, lse = s["plan"].chunk(s["q"], s["cache"], s["table"], s["lens"], s["cu"])
        return dict(out=out, lse=lse)
    if op == "fork":
        s["pool"].release(s["drop"])
        forked = s["pool"].fork(s["src"], s["dst"])
        return _pool_out(s, forked=forked, grown=s["pool"].grow(s["live"], s["add"]))
    return _pool_out(s, in_use=s["pool"].compact())


def _norm_out(case, codes, scale, r):
    if case["mode"] == "bf16":
        return dict(y=codes, residual=r)
    return dict(codes=codes.view(torch.float8_e4m3fn), scale=scale, residual=r)


def _pool_out(s, **more):
    e4m3 = torch.float8_e4m3fn
    return dict(table=s["table"], lens=s["lens"], refs=s["refs"], k=s["k"].view(e4m3), v=s["v"].view(e4m3), k_scale=s["k_scale"],
                v_scale=s["v_scale"], **more)


def _pow2(code):
    """2^(code - 127) of e8m0 codes below 255."""
    code = code.to(torch.int32)
    return torch.where(code > 0, code << 23, 0x00400000).view(torch.float32)


def _e4m3(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_norm(s):
    """The norm is that of the residual as it is kept.  Its mean square is formed in 64 bits: a scale of mxfp8 goes by which side of a
    power of two the largest value of 32 lies."""
    case, x = s["case"], s["x"]
    r = (x.float() + s["residual"].float()).to(x.dtype)
    mean = r.double().square_().mean(-1, keepdim=True)
    y = r.float() * (1.0 / (mean + EPS).sqrt()).float() * s["weight"].float()
    R, C = y.shape
    if case["mode"] == "bf16":
        return _norm_out(case, y.to(torch.bfloat16), None, r)
    b = y.view(R, -1, {"ptpc": C, "blockscale": 128, "mxfp8": 32}[case["mode"]])
    amax = b.abs().amax(-1)
    if case["mode"] == "mxfp8":
        m, e = torch.frexp(amax)
        code = torch.where(amax > 0, torch.where(m <= 0.875, e - 9, e - 8) + 127, 127).clamp(0, 254)
        codes, scale = _e4m3(b * _pow2(254 - code)[..., None]), code.to(torch.uint8).t().contiguous()
    else:
        sc = torch.where(amax > 0, amax / 448.0, 1.0)
        codes, scale = _e4m3(b / sc[..., None]), (sc.view(R) if case["mode"] == "ptpc" else sc.t().contiguous())
    return _norm_out(case, codes.view(R, C), scale, r)


def _plain_chunk(s):
    case = s["case"]
    B, hq, hk, d, page = (case[x] for x in ("B", "hq", "hk", "d", "page"))
    g, table, lens, cu = hq // hk, s["table"].long(), s["lens"].long(), s["cu"].long()
    L = table.shape[1] * page
    pg, at = table.clamp(min=0), torch.arange(L, device=table.device)
    there = (at[None, :] < lens[:, None])[:, None, :, None]

    def values(codes, scale):
        x = codes[pg].view(torch.float8_e4m3fn).float()            # [B, P, Hk, page, D]
        x *= _pow2(scale[pg]).repeat_interleave(BLOCK, -1)[..., None]
        return x.transpose(1, 2).reshape(B, hk, L, d).masked_fill_(~there, 0.0)

    n = cu.diff()
    i = torch.arange(s["max_q"], device=table.device)
    rows = i[None, :] < n[:, None]
    q = s["q"][(cu[:-1, None] + i).clamp(max=max(s["q"].shape[0] - 1, 0))].float()      # [B, Q, Hq, D]
    q = q.view(B, len(i), hk, g, d).permute(0, 2, 3, 1, 4).reshape(B, hk, g * len(i), d)
    sc = torch.matmul(q * d ** -0.5, values(s["k"], s["k_scale"]).transpose(2, 3)).view(B, hk, g, len(i), L)
    see = lens[:, None] - n[:, None] + 1 + i[None, :]
    sc.masked_fill_((at[None, None, :] >= see[..., None])[:, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    base = torch.where(torch.isinf(m), 0.0, m)
    p = sc.sub_(base).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, hk, g * len(i), L), values(s["v"], s["v_scale"])).view(B, hk, g, len(i), d)
    o = o / torch.where(total == 0, 1.0, total)
    lse = (base + total.log()).squeeze(-1)
    return dict(out=o.permute(0, 3, 1, 2, 4).reshape(B, len(i), hq, d)[rows].to(torch.bfloat16),
                lse=lse.permute(0, 3, 1, 2).reshape(B, len(i), hq)[rows])


def _free_pages(refs):
    """All pages, the free ones first, in order."""
    return torch.argsort((refs > 0).to(torch.int32), stable=True)


def _granted(need, refs):
    """Which requests get the pages that they need, in order; and the first page's number among the free ones."""
    upto = need.cumsum(0)
    return (need == 0) | (upto <= (refs == 0).sum()), upto - need


def _plain_fork(s):
    case, page = s["case"], s["case"]["page"]
    table, lens, refs = s["table"], s["lens"], s["refs"]
    entry = torch.arange(table.shape[1], device=table.device)[None, :]
    # release
    drop = s["drop"].long()
    gone = table[drop]
    refs.index_add_(0, gone.clamp(min=0).flatten().long(), -(gone >= 0).flatten().to(torch.int32))
    table[drop], lens[drop] = -1, 0
    # fork
    src, dst = s["src"].long(), s["dst"].long()
    n = lens[src]
    full, part = (n // page)[:, None], (n % page > 0).to(torch.int32)
    ok, first = _granted(part, refs)
    ok &= lens[dst] == 0
    copy = ok & (part > 0)
    new = _free_pages(refs)[first.clamp(max=len(refs) - 1)]
    old = torch.gather(table[src], 1, full.clamp(max=table.shape[1] - 1).long())[:, 0].long()
    rows = torch.where(entry < full, table[src], -1)
    rows = torch.where((entry == full) & copy[:, None], new[:, None].to(torch.int32), rows)
    rows = torch.where(ok[:, None], rows, table[dst])
    refs.index_add_(0, rows.clamp(min=0).flatten().long(), ((rows >= 0) & ok[:, None]).flatten().to(torch.int32))
    table[dst] = rows
    lens[dst] = torch.where(ok, n, lens[dst])
    for t in (s["k"], s["v"], s["k_scale"], s["v_scale"]):
        t[:, new[copy]] = t[:, old[copy]]
    # grow
    live = s["live"].long()
    n, add = lens[live], s["add"]
    have = (n + page - 1) // page
    need = (n + add + page - 1) // page - have
    fits = n + add <= table.shape[1] * page
    grown, first = _granted(torch.where(fits, need, 0), refs)
    grown &= fits
    which = (entry >= have[:, None]) & (entry < (have + need)[:, None]) & grown[:, None]
    pages = _free_pages(refs)[(first[:, None] + entry - have[:, None]).clamp(0, len(refs) - 1)].to(torch.int32)
    rows = torch.where(which, pages, table[live])
    refs.index_add_(0, pages.flatten().long(), which.flatten().to(torch.int32))
    table[live] = rows
    lens[live] = torch.where(grown, n + add, n)
    return _pool_out(s, forked=ok.to(torch.int32), grown=grown.to(torch.int32))


def _plain_compact(s):
    table, refs = s["table"], s["refs"]
    used = refs > 0
    total = used.sum()
    at = torch.arange(len(refs), device=refs.device)
    to = torch.nonzero(~used & (at < total))[:, 0]
    frm = torch.nonzero(used & (at >= total))[:, 0]
    moved = at.to(torch.int32)
    moved[frm] = to.to(torch.int32)
    table.copy_(torch.where(table >= 0, moved[table.clamp(min=0).long()], table))
    refs[to] = refs[frm]
    refs[frm] = 0
    for t in (s["k"], s["v"], s["k_scale"], s["v_scale"]):
        t[:, to] = t[:, frm]
    return _pool_out(s, in_use=total.to(torch.int32).view(1))


# --------------------------------------------------------------------------- work


def work(case):
    op = case["op"]
    if op == "norm":
        n, R = case["rows"] * case["cols"], case["rows"]
        size = 2 if case["dtype"] == "bf16" else 4
        out = {"ptpc": n + 4 * R, "blockscale": n + n // 32, "mxfp8": n + n // 32, "bf16": 2 * n}[case["mode"]]
        return dict(bytes=3 * size * n + size * case["cols"] + out, flops=7 * n)
    page = case["page"]
    if op == "chunk":
        new, lens = _chunk_lens(case)
        seen = sum(b * a - a * (a - 1) // 2 for a, b in zip(new, lens))
        kv = sum(n for a, n in zip(new, lens) if a)
        return dict(bytes=kv * case["hk"] * 2 * (case["d"] + 1 / BLOCK) + sum(new) * case["hq"] * (4 * case["d"] + 4),
                    flops=4 * seen * case["hq"] * case["d"])
    page_bytes = 2 * case["layers"] * case["hk"] * (page * case["d"] + page // BLOCK)
    if op == "fork":
        lens, drop, src, dst, live, add = _rows_of(case)
        copies = sum(1 for r in src if lens[r] % page)
        entries = sum(-(-lens[r] // page) for r in drop + src)
        return dict(bytes=2 * copies * page_bytes + 12 * entries, flops=0)
    lens = _lens(case, case["rows"], case["len_lo"], case["len_hi"], 5)
    used = sum(-(-n // page) for n in lens)
    pages = int(used / case["used"]) + 1
    # pages in use are spread evenly: what lies past the first `used` has to move
    moves = used * (pages - used) // pages
    return dict(bytes=2 * moves * page_bytes + 4 * pages + 8 * used, flops=0)


# --------------------------------------------------------------------------- 64 bits


def _e4m3_values(dev):
    """The 256 values of e4m3 by its definition."""
    v = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.nan if (c & 127) == 127 else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        v.append(-x if c & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device=dev)


def exact(case, seed):
    """Pages are moved, not computed: no values for those."""
    global own
    if case["op"] in ("fork", "compact"):
        return None
    mine, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = mine
    return (_exact_norm if case["op"] == "norm" else _exact_chunk)(case, s)


def _exact_norm(case, s):
    total = s["x"].double() + s["residual"].double()
    r = total.to(s["x"].dtype).double()              # what the norm is of
    y = r / torch.sqrt((r * r).sum(1) / case["cols"] + EPS)[:, None] * s["weight"].double()
    if case["mode"] == "bf16":
        return dict(y=y, residual=total)
    width = {"ptpc": case["cols"], "blockscale": 128, "mxfp8": 32}[case["mode"]]
    blocks = y.unflatten(1, (-1, width))
    top = blocks.abs().max(-1).values
    if case["mode"] == "mxfp8":
        e = torch.ceil(torch.log2(top / 448)).clamp(-127, 127)
        return dict(codes=(blocks / torch.exp2(e)[..., None]).flatten(1).clamp(-448, 448), scale=None, residual=total)
    scale = top / 448
    return dict(codes=(blocks / scale[..., None]).flatten(1), scale=scale[:, 0] if case["mode"] == "ptpc" else scale.T.contiguous(), residual=total)


def _exact_chunk(case, s):
    hq, hk, d, page = case["hq"], case["hk"], case["d"], case["page"]
    new, lens = _chunk_lens(case)
    if sum(a * b for a, b in zip(new, lens)) * hq * d * 4 > 4e12 or case["B"] * hq > 4000:
        return None
    lut = _e4m3_values(s["q"].device)
    outs, lses, t0 = [], [], 0
    for b, (n, m) in enumerate(zip(new, lens)):
        q = s["q"][t0:t0 + n].double()
        t0 += n
        o = torch.zeros(n, hq, d, dtype=torch.float64, device=q.device)
        lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device=q.device)
        pages = s["table"][b, :-(-m // page)].long()
        sees = torch.arange(m, device=q.device)[None, :] <= (m - n + torch.arange(n, device=q.device))[:, None]
        for h in range(hk if n else 0):
            kv = [(lut[s[c][pages, h].long()] * torch.exp2(s[e][pages, h].double() - 127).repeat_interleave(BLOCK, 1)[..., None])
                  .reshape(-1, d)[:m] for c, e in (("k", "k_scale"), ("v", "v_scale"))]
            for x in range(h * (hq // hk), (h + 1) * (hq // hk)):
                sc = (q[:, x] @ kv[0].T / math.sqrt(d)).masked_fill(~sees, -math.inf)
                lse[:, x] = torch.logsumexp(sc, 1)
                o[:, x] = torch.softmax(sc, 1) @ kv[1]
        outs.append(o)
        lses.append(lse)
    return dict(out=torch.cat(outs), lse=torch.cat(lses))
