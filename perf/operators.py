"""The paged 8-bit cache's operators: what is measured, and their plain forms.

The cache holds K and V as E4M3 codes in pages of 16 tokens, with one power-of-two scale
per page and KV head for each of K and V.  Operators:

  plan    block tables, slot maps, positions and packed row starts from request lengths,
          all on the GPU; pages are popped from a free stack
  append  quantise new tokens into their slots; a page's scale grows when a token needs
          it, and the page's other codes are then rounded to the new scale
  gather  the values of the tokens at given slots
  attend  grouped-query attention over the pages for packed ragged queries: single
          tokens (optionally with each block's mass: the max over query heads of the
          weight in the block), a few tokens each, or prompt chunks; causal, optionally
          within a window

Shapes are this repository's decode stacks (32/4 and 64/8 heads of 128, contexts of
4096, 32768 and 131072, ragged U[1024, 32768]) and generic smaller ones.
"""

import math
import random

import numpy as np
import torch

own = False

PAGE = 16
E_MIN, E_MAX = -100, 119          # exponents a page scale can have

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    base = {"hq": 32, "hkv": 4, "d": 128, "dtype": "bf16", "window": 0, "scored": False, "lens_seed": 1}

    def case(name, op, n, lo, hi, q_lo, q_hi, **kw):
        return {"name": name, "op": op, "n": n, "lo": lo, "hi": hi, "q_lo": q_lo, "q_hi": q_hi, **base, **kw}

    # n requests; lo..hi: tokens cached before the call; q_lo..q_hi: new tokens of each request
    return [
        # one decode step of a serving batch: the page bookkeeping alone, latency only
        case("plan-decode-b16", "plan", 16, 32000, 32768, 1, 1),
        # a ragged batch of prompts admitted in one step
        case("plan-admit-b64", "plan", 64, 0, 0, 1024, 32768),
        # the decode step's store: one token per request into a partly filled page
        case("append-decode-b16", "append", 16, 32000, 32768, 1, 1),
        # prompts of odd lengths stored in one call, some behind a cached prefix
        case("append-prompts-b6", "append", 6, 0, 500, 900, 8192),
        # one short context read back in 32 bits
        case("gather-f32-b1", "gather", 1, 1000, 1000, 0, 0, dtype="f32"),
        # sixteen windows' worth of context read back
        case("gather-b16", "gather", 16, 4000, 4096, 0, 0),
        # the smallest decode call: one short chat
        case("attend-decode-b1-ctx700", "attend", 1, 700, 700, 1, 1),
        # a decode step of the repository's 16-sequence stack without its window
        case("attend-decode-b16-ctx32768", "attend", 16, 32000, 32768, 1, 1),
        # the ragged 64-sequence stack, with the block masses that selection needs
        case("attend-scored-b64-ragged", "attend", 64, 1024, 32768, 1, 1, scored=True),
        # one very long context on the 64/8 stack: work has to be split over the context
        case("attend-decode-b1-ctx131072", "attend", 1, 131000, 131071, 1, 1, hq=64, hkv=8),
        # chunked prefill: ragged chunks behind ragged contexts
        case("attend-chunks-b5", "attend", 5, 0, 8192, 100, 2048),
        # one whole prompt
        case("attend-prompt-b1-8192", "attend", 1, 0, 0, 8192, 8192),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    hq, hkv, d = rng.choice([(32, 4, 128), (32, 4, 128), (64, 8, 128), (32, 8, 128), (8, 8, 128), (16, 2, 64), (12, 4, 64)])
    case = {"hq": hq, "hkv": hkv, "d": d, "dtype": "bf16", "window": 0, "scored": False,
            "lens_seed": rng.randrange(1 << 30)}
    kind = rng.choice(["plan", "append", "gather", "decode", "decode", "few", "prompt"])
    if kind == "plan":
        n = _log(rng, 1, 300)
        if rng.random() < 0.5:
            case.update(op="plan", n=n, lo=0, hi=_log(rng, 1, 32768), q_lo=1, q_hi=_log(rng, 1, 8))
        else:
            hi = max(2, min(32768, 1000000 // n))
            case.update(op="plan", n=n, lo=0, hi=_log(rng, 1, 4096), q_lo=0 if n > 8 else 1, q_hi=_log(rng, 2, hi))
    elif kind in ("append", "gather"):
        n = _log(rng, 1, 64)
        top = _log(rng, 1, max(2, 40000 // n))
        if kind == "append":
            case.update(op="append", n=n, lo=0, hi=_log(rng, 1, 2000), q_lo=max(1, top // 3), q_hi=top)
        else:
            case.update(op="gather", n=n, lo=max(1, top // 2), hi=top, q_lo=0, q_hi=0)
        case["dtype"] = rng.choice(["bf16", "bf16", "f32"])
    elif kind == "decode":
        n = _log(rng, 1, 128)
        hi = min(131072, _log(rng, 1, max(2, 500000 // n)))
        case.update(op="attend", n=n, lo=0, hi=hi, q_lo=1, q_hi=1, scored=rng.random() < 0.3)
        if rng.random() < 0.3:
            case["window"] = _log(rng, 1, 8192)
        if n * hi < 40000 and rng.random() < 0.3:
            case["dtype"] = "f32"
    elif kind == "few":
        n = _log(rng, 1, 32)
        case.update(op="attend", n=n, lo=0, hi=_log(rng, 1, max(2, 200000 // n)), q_lo=1, q_hi=rng.randint(2, 9))
    else:
        n = _log(rng, 1, 8)
        q = _log(rng, 16, 5000 // n)
        pairs = 30000000 * 32 // (hq * n)            # of a query and an entry, for each request
        case.update(op="attend", n=n, lo=0, hi=_log(rng, 1, max(2, min(16000 // n, pairs // q - q))),
                    q_lo=max(1, q // 2), q_hi=q)
        if rng.random() < 0.3:
            case["window"] = _log(rng, 16, 8192)
    return case


def _lens(case):
    """The requests' cached lengths and new lengths: part of the case, not of the seed."""
    r = random.Random(case["lens_seed"])
    ctx = [r.randint(case["lo"], case["hi"]) for _ in range(case["n"])]
    new = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["n"])]
    return ctx, new


def _visible(c, q, window):
    """Entries that the q queries behind c cached tokens see in all."""
    if not window:
        return q * c + q * (q + 1) // 2
    return sum(min(window, c + i + 1) for i in range(q))


def work(case):
    ctx, new = _lens(case)
    es = 2 if case["dtype"] == "bf16" else 4
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    t = sum(new)
    if case["op"] == "plan":
        taken = sum((c + q + PAGE - 1) // PAGE - (c + PAGE - 1) // PAGE for c, q in zip(ctx, new))
        # lengths in, starts and lengths out; a popped page read and written; slot and position of each token
        return {"bytes": 4 * (4 * case["n"] + 2 * taken + 2 * t), "flops": 0}
    if case["op"] == "append":
        # new rows in, and the values of the written pages' tokens back out of their codes
        back = sum(q + c % PAGE for c, q in zip(ctx, new))
        return {"bytes": 2 * hkv * d * (t * (es + 1) + back * (1 + es)), "flops": 0}
    if case["op"] == "gather":
        return {"bytes": 2 * hkv * d * sum(ctx) * (1 + es), "flops": 0}
    w = case["window"]
    read = sum(min(c + q, w + q - 1) if w else c + q for c, q in zip(ctx, new))
    mass = 4 * sum((c + q + PAGE - 1) // PAGE for c, q in zip(ctx, new)) if case["scored"] else 0
    return {"bytes": 2 * hkv * d * read + 8 * hkv * (read // PAGE) + 2 * t * hq * d * es + mass,
            "flops": 4 * hq * d * sum(_visible(c, q, w) for c, q in zip(ctx, new))}


# ------------------------------------------------------------------ inputs
class _State:
    pass


def _keys_values(g, rows, hkv, d, dtype):
    """K with a few strong channels and heavy tokens, V plain: what makes a page's scale grow."""
    k = torch.randn((rows, hkv, d), generator=g, device="cuda")
    k *= torch.exp(0.5 * torch.randn((1, hkv, d), generator=g, device="cuda"))
    k *= 1 + 3 * (torch.rand((rows, 1, 1), generator=g, device="cuda") < 0.02)
    v = torch.randn((rows, hkv, d), generator=g, device="cuda")
    return k.to(dtype), v.to(dtype)


def _inputs(case, seed):
    """Everything that both forms and the 64-bit one start from."""
    s = _State()
    s.case = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    ctx, new = _lens(case)
    n, hkv, d = case["n"], case["hkv"], case["d"]
    dt = _DT[case["dtype"]]
    total = [c + q for c, q in zip(ctx, new)]
    s.n, s.hq, s.hkv, s.d, s.dt = n, case["hq"], hkv, d, dt
    s.max_len, s.max_new, s.t = max(total), max(new), sum(new)
    s.stride = max(1, -(-s.max_len // PAGE))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    s.ctx, s.new, s.kv_len = i32(ctx), i32(new), i32(total)
    start = [0]
    for q in new:
        start.append(start[-1] + q)
    s.q_start = i32(start)
    blocks = [-(-x // PAGE) for x in total]
    s.num_pages = sum(blocks) + 7
    perm = torch.randperm(s.num_pages, generator=g, device="cuda").to(torch.int32)
    if case["op"] == "plan":
        # the cached blocks' pages are in the table, the others on the free stack
        held = [-(-x // PAGE) for x in ctx]
        s.table = torch.full((n, s.stride), -1, dtype=torch.int32, device="cuda")
        h = i32(held).long()
        col = torch.arange(s.stride, device="cuda")
        at = (torch.cumsum(h, 0) - h)[:, None] + col
        s.table = torch.where(col < h[:, None], perm[at.clamp(max=s.num_pages - 1)], s.table).contiguous()
        s.free = perm[sum(held):].contiguous()
        s.free_count = i32([s.free.numel()])
        return s
    # every block's page, in random order
    b = i32(blocks).long()
    col = torch.arange(s.stride, device="cuda")
    at = (torch.cumsum(b, 0) - b)[:, None] + col
    s.table = torch.where(col < b[:, None], perm[at.clamp(max=s.num_pages - 1)], torch.full_like(perm[:1], -1)).contiguous()

    def slots(lo, ln):
        """Slots of positions lo[r] .. lo[r] + ln[r] of every request, packed."""
        ln_t = torch.tensor(ln, device="cuda")
        rows = sum(ln)
        req = torch.repeat_interleave(torch.arange(n, device="cuda"), ln_t, output_size=rows)
        pos = torch.arange(rows, device="cuda") - (torch.cumsum(ln_t, 0) - ln_t)[req] + torch.tensor(lo, device="cuda")[req]
        return (s.table[req, pos // PAGE] * PAGE + pos % PAGE).to(torch.int32), req, pos

    if case["op"] == "append":
        # the partly filled pages that the new tokens join
        lo = [c - c % PAGE for c in ctx]
        s.old_slots = slots(lo, [c % PAGE for c in ctx])[0]
        s.old_k, s.old_v = _keys_values(g, s.old_slots.numel(), hkv, d, dt)
        s.slots = slots(ctx, new)[0]
        s.k, s.v = _keys_values(g, s.t, hkv, d, dt)
        s.read = slots(lo, [c % PAGE + q for c, q in zip(ctx, new)])[0]
        s.runs = s.t // PAGE + 2 * n
    else:
        s.old_slots = slots([0] * n, total)[0]
        s.old_k, s.old_v = _keys_values(g, s.old_slots.numel(), hkv, d, dt)
        s.read = s.old_slots
        if case["op"] == "attend":
            s.q = torch.randn((s.t, s.hq, d), generator=g, device="cuda").to(dt)
            _, s.row_req, pos = slots(ctx, new)
            s.row_i = pos - s.ctx[s.row_req]
    s.old_runs = s.old_slots.numel() // PAGE + 2 * n
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import attention_scored_kv_gb300 as kvs
        s.cache = kvs.PagedCache(kvs.paged_config_init(
            num_layers=1, num_q_heads=s.hq, num_kv_heads=s.hkv, head_dim=s.d, num_pages=s.num_pages,
            in_dtype=kvs.BF16 if s.dt == torch.bfloat16 else kvs.F32))
        if case["op"] == "plan":
            s.free_left = torch.zeros_like(s.free_count)
        elif s.old_slots.numel():
            s.cache.append(0, s.old_k, s.old_v, s.old_slots)
        if case["scored"]:
            s.mass = torch.zeros((s.n, s.stride), dtype=torch.float32, device="cuda")
    elif case["op"] != "plan":
        # one page more than the pool has: where runs that do not exist are written
        shape = (s.num_pages + 1, PAGE, s.hkv, s.d)
        s.codes = [torch.zeros(shape, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
        s.scales = [torch.full((s.num_pages + 1, s.hkv), 2.0 ** E_MIN, device="cuda") for _ in range(2)]
        if s.old_slots.numel():
            _append(s, s.old_k, s.old_v, s.old_slots, s.old_runs)
    if case["op"] != "append":
        s.old_k = s.old_v = None
    return s


# ------------------------------------------------------------------ plain forms
def _needed_scale(absmax):
    """The smallest power of two s with absmax <= 448 * s."""
    f, e = torch.frexp(absmax)                       # absmax = f * 2^e, f in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(f <= 0.875, e - 9, e - 8)
    e = torch.where(absmax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)
    return ((e + 127) << 23).view(torch.float32)     # 2^e to the bit, which pow() does not give


def _append(s, k, v, slots, runs):
    """Tokens of one page are neighbours in a call: a run.  A run that starts a page empties it first."""
    slots = slots.long()
    page, off = slots // PAGE, slots % PAGE
    leads = torch.ones_like(page, dtype=torch.bool)
    leads[1:] = page[1:] != page[:-1]
    run = torch.cumsum(leads.long(), 0) - 1
    run_page = torch.full((runs,), s.num_pages, dtype=torch.long, device="cuda").scatter_(0, run, page)
    fresh = torch.zeros((runs,), device="cuda").scatter_reduce_(0, run, (off == 0).float(), "amax") > 0
    for which, x in ((0, k), (1, v)):
        x = x.float()
        absmax = x.abs().amax(-1)
        top = torch.zeros((runs, s.hkv), device="cuda").scatter_reduce_(0, run[:, None].expand(-1, s.hkv), absmax, "amax")
        old = s.scales[which][run_page]
        scale = torch.maximum(_needed_scale(top), torch.where(fresh[:, None], torch.full_like(old, 2.0 ** E_MIN), old))
        kept = s.codes[which][run_page].float() * torch.where(fresh[:, None], torch.zeros_like(old), old / scale)[:, None, :, None]
        kept[run, off] = x / scale[run][:, :, None]
        s.codes[which][run_page] = kept.to(torch.float8_e4m3fn)
        s.scales[which][run_page] = scale


def _read(s, slots):
    slots = slots.long()
    page, off = slots // PAGE, slots % PAGE
    return [(c[page, off].float() * z[page][:, :, None]).to(s.dt) for c, z in zip(s.codes, s.scales)]


def _plan(s):
    ctx, new = s.ctx.long(), s.new.long()
    kv_len = ctx + new
    held, need = (ctx + PAGE - 1) // PAGE, (kv_len + PAGE - 1) // PAGE
    take = need - held
    upto = torch.cumsum(take, 0)
    col = torch.arange(s.stride, device="cuda")
    j = (upto - take)[:, None] + col - held[:, None]
    fills = (col >= held[:, None]) & (col < need[:, None])
    popped = s.free[(s.free_count.long() - 1 - j).clamp(0, s.free.numel() - 1)]
    table = torch.where(fills, popped, s.table)
    q_start = torch.cat([torch.zeros_like(upto[:1]), torch.cumsum(new, 0)])
    t = torch.arange(s.t, device="cuda")
    req = torch.searchsorted(q_start[1:], t, right=True)
    pos = t - q_start[req] + ctx[req]
    slots = table[req, pos // PAGE] * PAGE + pos % PAGE
    return {"table": table, "q_start": q_start.int(), "kv_len": kv_len.int(), "slots": slots.int(),
            "positions": pos.int(), "free": s.free_count - upto[-1:].int()}


def _attend(s):
    n, hkv, g, d, qm, w = s.n, s.hkv, s.hq // s.hkv, s.d, s.max_new, s.case["window"]
    table = s.table.long().clamp(min=0)
    length = s.stride * PAGE
    k, v = ((c[table].float() * z[table][:, :, None, :, None]).view(n, length, hkv, d).transpose(1, 2)
            for c, z in zip(s.codes, s.scales))                                       # [n, hkv, length, d]
    i = torch.arange(qm, device="cuda")
    rows = (s.q_start[:-1].long()[:, None] + i).clamp(max=s.t - 1)
    q = s.q[rows].float().view(n, qm, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, g * qm, d)
    logits = (q @ k.transpose(2, 3)).view(n, hkv, g, qm, length) / math.sqrt(d)
    at = (s.kv_len - s.new).long()[:, None] + i                                        # query positions [n, qm]
    j = torch.arange(length, device="cuda")
    seen = (j <= at[:, :, None]) & (i < s.new[:, None])[:, :, None]
    if w:
        seen &= j > at[:, :, None] - w
    logits = logits.masked_fill_(~seen[:, None, None], -math.inf)
    top = logits.amax(-1, keepdim=True)
    p = logits.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    p = p.div_(p.sum(-1, keepdim=True).clamp(min=1e-30))
    o = (p.view(n, hkv, g * qm, length) @ v).view(n, hkv, g, qm, d)
    out = o.permute(0, 3, 1, 2, 4)[s.row_req, s.row_i].reshape(s.t, s.hq, d).to(s.dt)
    if not s.case["scored"]:
        return out
    return {"out": out, "mass": p.view(n, s.hq, s.stride, PAGE).sum(-1).amax(1)}


def run(s):
    op = s.case["op"]
    if own:
        if op == "plan":
            p = s.cache.plan(s.ctx, s.new, s.table, s.free, s.free_count, s.t, free_count_out=s.free_left)
            return {"table": s.table, "q_start": p.q_start, "kv_len": p.kv_len, "slots": p.slots,
                    "positions": p.positions, "free": s.free_left}
        if op == "append":
            s.cache.append(0, s.k, s.v, s.slots)
            return s.cache.gather(0, s.read)
        if op == "gather":
            return s.cache.gather(0, s.read)
        if s.case["scored"]:
            return {"out": s.cache.attend(0, s.q, s.table, s.kv_len, window=s.case["window"], block_mass=s.mass),
                    "mass": s.mass}
        if s.max_new == 1:
            return s.cache.attend(0, s.q, s.table, s.kv_len, window=s.case["window"])
        return s.cache.attend(0, s.q, s.table, s.kv_len, q_start=s.q_start, max_q_len=s.max_new,
                              window=s.case["window"])
    if op == "plan":
        return _plan(s)
    if op == "append":
        _append(s, s.k, s.v, s.slots, s.runs)
        return _read(s, s.read)
    if op == "gather":
        return _read(s, s.read)
    return _attend(s)


# ------------------------------------------------------------------ the definitions in 64 bits
def _two_to(e):
    """2^e in 64 bits, to the bit."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3(x):
    """x rounded to the nearest E4M3 value, ties to even, in 64 bits."""
    a = x.abs()
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -20))).clamp(min=-6)
    e = torch.where(_two_to(e + 1) <= a, e + 1, e)
    step = _two_to(e - 3)
    return torch.sign(x) * torch.round(a / step) * step


def _exact_scale(absmax):
    e = torch.ceil(torch.log2(absmax.clamp(min=2.0 ** -200) / 448)).clamp(E_MIN, E_MAX)
    s = _two_to(e)
    s = torch.where(absmax > 448 * s, 2 * s, s)
    return torch.where((absmax <= 224 * s) & (e > E_MIN), s / 2, s)


def _exact_pages(x, slots, pages, codes=None, scale=None):
    """The pages [pages, 16, hkv, d] after the tokens x are stored at slots: their code values and scales."""
    x = x.double()
    slots = slots.long()
    new = torch.zeros((pages * PAGE,) + x.shape[1:], dtype=torch.float64, device="cuda")
    new[slots] = x
    written = torch.zeros((pages * PAGE,), dtype=torch.bool, device="cuda")
    written[slots] = True
    new, written = new.view(pages, PAGE, *x.shape[1:]), written.view(pages, PAGE)
    first = torch.full((pages, x.shape[1]), 2.0 ** E_MIN, dtype=torch.float64, device="cuda")
    if codes is None:
        codes, scale = torch.zeros_like(new), first
    fresh = written[:, 0]
    scale_old = torch.where(fresh[:, None], first, scale)
    codes = torch.where(fresh[:, None, None, None], torch.zeros_like(codes), codes)
    top = _exact_scale(new.abs().amax(dim=(1, 3)))
    scale_new = torch.where(written.any(1)[:, None], torch.maximum(scale_old, top), scale_old)
    kept = codes * (scale_old / scale_new)[:, None, :, None]
    return _e4m3(torch.where(written[:, :, None, None], new / scale_new[:, None, :, None], kept)), scale_new


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "plan":
        # in plain integers, one request after the other
        ctx, new = (x.cpu().numpy().astype(np.int64) for x in (s.ctx, s.new))
        table, free = s.table.cpu().numpy().copy(), s.free.cpu().numpy()
        left, slots, positions, start = int(s.free_count), [], [], [0]
        for r in range(s.n):
            for b in range(-(-int(ctx[r]) // PAGE), -(-int(ctx[r] + new[r]) // PAGE)):
                left -= 1
                table[r, b] = free[left]
            p = np.arange(ctx[r], ctx[r] + new[r])
            slots.append(table[r, p // PAGE] * PAGE + p % PAGE)
            positions.append(p)
            start.append(start[-1] + len(p))
        return {"table": table, "q_start": np.array(start, np.int32), "kv_len": (ctx + new).astype(np.int32),
                "slots": np.concatenate(slots).astype(np.int32), "positions": np.concatenate(positions).astype(np.int32),
                "free": np.array([left], np.int32)}
    both = []
    for x, y in ((s.old_k, s.k if case["op"] == "append" else None), (s.old_v, s.v if case["op"] == "append" else None)):
        codes = scale = None
        if s.old_slots.numel():
            codes, scale = _exact_pages(x, s.old_slots, s.num_pages)
        if y is not None:
            codes, scale = _exact_pages(y, s.slots, s.num_pages, codes, scale)
        both.append(codes * scale[:, None, :, None])
        del codes, scale
    if case["op"] in ("append", "gather"):
        at = s.read.long()
        return [x.view(-1, s.hkv, s.d)[at] for x in both]
    out = torch.zeros((s.t, s.hq, s.d), dtype=torch.float64, device="cuda")
    mass = torch.zeros((s.n, s.stride), dtype=torch.float64, device="cuda")
    ctx, new = _lens(case)
    g, at = s.hq // s.hkv, 0
    for r in range(s.n):
        total = ctx[r] + new[r]
        pages = s.table[r, :-(-total // PAGE)].long()
        for h in range(s.hkv):
            k, v = (x[pages, :, h].reshape(-1, s.d)[:total] for x in both)
            for lo in range(0, new[r], 1024):
                q = s.q[at + lo:at + min(lo + 1024, new[r]), h * g:(h + 1) * g].double()
                p = torch.einsum("ihd,jd->hij", q, k) / math.sqrt(s.d)
                i = ctx[r] + lo + torch.arange(q.shape[0], device="cuda")[:, None]
                j = torch.arange(total, device="cuda")[None]
                hidden = (j > i) | ((j <= i - case["window"]) if case["window"] else torch.zeros_like(j > i))
                p = torch.softmax(p.masked_fill(hidden, -math.inf), -1)
                out[at + lo:at + lo + q.shape[0], h * g:(h + 1) * g] = torch.einsum("hij,jd->ihd", p, v)
                if case["scored"]:
                    sums = torch.nn.functional.pad(p[:, 0], (0, -total % PAGE)).view(g, -1, PAGE).sum(-1)
                    mass[r, :sums.shape[1]] = torch.maximum(mass[r, :sums.shape[1]], sums.amax(0))
        at += new[r]
    return {"out": out, "mass": mass} if case["scored"] else out
