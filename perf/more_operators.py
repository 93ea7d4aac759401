"""Cases for a serving step over an 8-bit cache with a scale for each block of tokens and head: pages
and slots of a batch from its lengths, the new tokens' rows into the cache (and cached tokens back
out), attention over it, and the draw of the next tokens from logits.

``run`` computes a case in plain torch operations (float32, or float64 where float32 loses what
matters) when ``own`` is false, and through the package's entry points when it is true; ``exact``
computes it from the definition in float64.

Batches are ragged and follow the package's conventions: request b owns rows
qo_indptr[b] .. qo_indptr[b+1]-1 of the new tokens, which are the last ones of its seq_lens[b]
cached tokens; token j of request b is in page page_table[b][j // P], slot j % P.  The scale of
KV head h for the S tokens of a page from slot t S on is scales[page][h][t].
"""
import math
import random

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step of 256 requests: one token each, every 64th request needs a page; a few
        # requests have ended and give theirs back (where latency counts)
        dict(name="pages_decode", op="pages", batch=256, page=64, hist_lo=512, hist_hi=16384, new_lo=1, new_hi=1,
             ended=6, shape=1),
        # prompts of up to 8k tokens for 96 requests, in place of as many that ended
        dict(name="pages_prompts", op="pages", batch=192, page=16, hist_lo=0, hist_hi=0, new_lo=200, new_hi=8192,
             ended=96, shape=2),
        # one new token for each of 64 decoding requests: most fall inside a block that holds older
        # tokens, whose codes change when the scale has to grow
        dict(name="append_decode", op="append", rows="bf16", batch=64, heads=8, dim=128, page=64, block=64,
             hist_lo=1024, hist_hi=16384, new_lo=1, new_hi=1, shape=3),
        # prefill chunks of up to 4k tokens, K and V sliced out of one fused projection (strided
        # rows), blocks of 16 tokens
        dict(name="append_prefill", op="append", rows="bf16", batch=8, heads=8, dim=128, page=64, block=16,
             hist_lo=1, hist_hi=4096, new_lo=1500, new_hi=4096, shape=4),
        # short ragged requests read back as float32
        dict(name="gather_short", op="gather", rows="f32", batch=12, heads=8, dim=128, page=64, block=16,
             hist_lo=1, hist_hi=700, new_lo=1, new_hi=5, shape=5),
        # eight long requests read back as bf16 rows (moving a request to another cache)
        dict(name="gather_long", op="gather", rows="bf16", batch=8, heads=8, dim=128, page=64, block=64,
             hist_lo=8192, hist_hi=24576, new_lo=1, new_hi=1, shape=6),
        # one decoding request of 64 query heads over 8 KV heads: the smallest attention call
        dict(name="attend_single", op="attend", batch=1, heads=8, group=8, page=64, block=16, hist_lo=4000, hist_hi=4200,
             new_lo=1, new_hi=1, shape=7),
        # a decode batch at 32,768 tokens a request, 128 query heads over 8 KV heads
        dict(name="attend_decode", op="attend", batch=32, heads=8, group=16, page=64, block=64, hist_lo=32767,
             hist_hi=32767, new_lo=1, new_hi=1, shape=8),
        # chunks of new tokens after long histories, one scale per page of 128
        dict(name="attend_chunk", op="attend", batch=2, heads=8, group=8, page=128, block=128, hist_lo=12000,
             hist_hi=20000, new_lo=900, new_hi=2048, shape=9),
        # one request's next token from a vocabulary of 32,000, temperature and top-p
        dict(name="sample_single", op="sample", rows=1, vocab=32000, logits="f32", flat=0.0, probs=False,
             use="tp", shape=10),
        # the next tokens of 128 requests with settings of their own (greedy ones among them), some
        # distributions flat, bf16 logits (many ties) over 128,000 tokens
        dict(name="sample_batch", op="sample", rows=128, vocab=128000, logits="bf16", flat=0.2, probs=False,
             use="tkpm", shape=11),
        # the target's distributions that draft verification takes: 48 requests of 16 rows
        dict(name="sample_probs", op="sample", rows=768, vocab=32000, logits="f32", flat=0.1, probs=True,
             use="tkp", shape=12),
    ]


def _log_int(rng, lo, hi):
    if hi <= lo:
        return lo
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(max(1, lo)), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["pages", "append", "gather", "attend", "attend", "sample", "sample"])
    shape = rng.randrange(1 << 30)
    page = rng.choice([64, 128])
    if op == "pages":
        batch = _log_int(rng, 1, 512)
        fresh = rng.random() < 0.5
        return dict(op=op, batch=batch, page=rng.choice([16, 64, 128]), hist_lo=0 if fresh else 1,
                    hist_hi=0 if fresh else _log_int(rng, 16, 32768), new_lo=1,
                    new_hi=_log_int(rng, 1, max(1, 400000 // batch)), ended=rng.randint(0, batch // 2), shape=shape)
    if op in ("append", "gather"):
        batch, heads = _log_int(rng, 1, 96), rng.choice([1, 2, 4, 8])
        tokens = _log_int(rng, batch, 20000 if op == "append" else 60000)     # about so many rows
        most = max(1, 2 * tokens // batch)
        hist, new = (_log_int(rng, 1, 4096), most) if op == "append" else (most, 4)
        page = rng.choice([16, 64, 128])
        return dict(op=op, rows=rng.choice(["bf16", "f32"]), batch=batch, heads=heads, dim=rng.choice([64, 128]), page=page,
                    block=rng.choice([s for s in (16, 32, 64, 128) if s <= page]), hist_lo=1, hist_hi=hist, new_lo=1,
                    new_hi=min(new, 8192), shape=shape)
    if op == "attend":
        heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 4, 8, 16])
        batch = _log_int(rng, 1, 32)
        hist, new = _log_int(rng, 1, 32767), rng.choice([1, 1, 1, rng.randint(2, 8), _log_int(rng, 16, 2048)])
        case = dict(op=op, batch=batch, heads=heads, group=group, page=page,
                    block=rng.choice([s for s in (16, 32, 64, 128) if s <= page]),
                    hist_lo=max(1, hist // 8), hist_hi=hist, new_lo=max(1, new // 8), new_hi=new, shape=shape)
        while work(case)["flops"] > 1.5e12:              # no more than the listed chunks
            if case["batch"] > 1:
                case["batch"] //= 2
            else:
                case["new_hi"] //= 2
                case["new_lo"] = max(1, case["new_hi"] // 8)
        return case
    vocab = _log_int(rng, 500, 160000)
    return dict(op=op, rows=min(_log_int(rng, 1, 512), max(1, 16000000 // vocab)), vocab=vocab,
                logits=rng.choice(["f32", "bf16"]), flat=rng.choice([0.0, 0.1, 0.3]), probs=rng.random() < 0.3,
                use=rng.choice(["", "t", "tk", "tp", "tm", "tkp", "tkpm"]), shape=shape)


def _lengths(case):
    """(seq_lens, q_lens) of a case: histories log-uniform, new tokens log-uniform."""
    rng = random.Random(case["shape"])
    q = [_log_int(rng, case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    h = [_log_int(rng, case["hist_lo"], case["hist_hi"]) if case["hist_hi"] else 0 for _ in range(case["batch"])]
    return [a + b for a, b in zip(h, q)], q


def _pages_plan(case):
    """Per request of a page case: (seq_len, new tokens, pages held before the call).  The first
    `ended` ones (in a shuffled order) have ended; they hold the pages of a past length."""
    seq, q = _lengths(case)
    rng = random.Random(case["shape"] + 1)
    gone = set(rng.sample(range(case["batch"]), case["ended"]))
    held = []
    for b in range(case["batch"]):
        if b in gone:
            held.append(-(-max(1, seq[b]) // case["page"]))
            seq[b] = q[b] = 0
        else:
            held.append(-(-(seq[b] - q[b]) // case["page"]))
    return seq, q, held


def _pairs(case):
    """(query, key) pairs that the causal rule lets meet."""
    return sum(t * (n - t) + t * (t + 1) // 2 for n, t in zip(*_lengths(case)))


def work(case):
    op = case["op"]
    if op == "pages":
        seq, q, held = _pages_plan(case)
        need = [-(-n // case["page"]) for n in seq]
        moved = sum(abs(a - b) for a, b in zip(need, held))       # an id read and written each
        return dict(bytes=len(seq) * 16 + moved * 8 + sum(q) * 8, flops=sum(q) + moved)
    if op == "sample":
        n = case["rows"] * case["vocab"]
        return dict(bytes=n * ((4 if case["logits"] == "f32" else 2) + (4 if case["probs"] else 0)) + case["rows"] * 24,
                    flops=n * 3)
    seq, q = _lengths(case)
    if op in ("append", "gather"):
        n = (sum(q) if op == "append" else sum(seq)) * case["heads"] * case["dim"] * 2
        scales = n // (case["block"] * case["dim"]) * 4
        return dict(bytes=n * ((4 if case["rows"] == "f32" else 2) + 1) + scales, flops=n)
    H, Hq, D = case["heads"], case["heads"] * case["group"], 128
    return dict(bytes=sum(seq) * H * 2 * (D + 4 / case["block"]) + sum(q) * Hq * (D * 4 + 4), flops=4 * D * Hq * _pairs(case))


# ------------------------------------------------------------------ inputs
def _normal(gen, shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32) * scale).to(dtype)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _indptr(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return at


def _paging(case, seed):
    """Lengths and a shuffled page table on the device, and their host copies."""
    seq, q = _lengths(case)
    pages = [-(-n // case["page"]) for n in seq]
    perm = torch.randperm(sum(pages), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)
    table = torch.full((len(seq), max(pages)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
    qo = _indptr(q)
    return dict(page_table=table.to(DEV), seq_lens=_i32(seq), qo_indptr=_i32(qo), seq=seq, new=q, qo=qo, pages=sum(pages))


def _codes(gen, shape):
    """E4M3 codes of normal values, their largest near the format's."""
    return (_normal(gen, shape, torch.float32) * 120.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case=case)
    op = case["op"]
    if op == "pages":
        seq, q, held = _pages_plan(case)
        need = [-(-n // case["page"]) for n in seq]
        grow = sum(max(0, a - b) for a, b in zip(need, held))
        back = sum(max(0, b - a) for a, b in zip(need, held))
        spare = grow + 100 + sum(held) // 4                       # free pages before the call
        total = sum(held) + spare
        perm = torch.randperm(total, generator=torch.Generator().manual_seed(seed), dtype=torch.int32)
        table = torch.full((case["batch"], max(max(need), max(held)) + 1), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(held):
            table[b, :n] = perm[at:at + n]
            at += n
        stack = torch.full((total,), -1, dtype=torch.int32)
        stack[:spare] = perm[at:]
        qo = _indptr(q)
        s.update(page_table=table.to(DEV), free_pages=stack.to(DEV), free_count=_i32([spare]), held=_i32(held),
                 seq_lens=_i32(seq), qo_indptr=_i32(qo), slots=torch.empty(qo[-1], dtype=torch.int64, device=DEV),
                 held_out=_i32(held), free_count_out=_i32([spare]), tokens=qo[-1], grow=grow, back=back)
        return s
    if op == "sample":
        R, V = case["rows"], case["vocab"]
        # a model's next-token distribution has a tail like a power of the rank: exponential logits
        # under a slope, steep in most rows and flat in some
        slope = torch.rand(R, 1, generator=gen, device=DEV) * 1.4 + 1.2
        slope = torch.where(torch.rand(R, 1, generator=gen, device=DEV) < case["flat"], 0.7, slope)
        x = -torch.log1p(-torch.rand(R, V, generator=gen, device=DEV)) * slope
        s["logits"] = (x + torch.randn(R, V, generator=gen, device=DEV) * 0.3 - 4.0).to(_DT[case["logits"]])
        s["u"] = torch.rand(R, generator=gen, device=DEV)
        pick = lambda values: torch.tensor(values, device=DEV)[  # noqa: E731
            torch.randint(0, len(values), (R,), generator=gen, device=DEV)].contiguous()
        s["temperature"] = pick([0.0, 0.6, 0.7, 0.8, 1.0, 1.0, 1.2]) if "t" in case["use"] else None
        s["top_k"] = pick([0, 20, 50, 64, 200]).to(torch.int32) if "k" in case["use"] else None
        s["top_p"] = pick([0.8, 0.9, 0.95, 1.0]) if "p" in case["use"] else None
        s["min_p"] = pick([0.0, 0.02, 0.05, 0.1]) if "m" in case["use"] else None
        s["tokens"] = torch.empty(R, dtype=torch.int32, device=DEV)
        s["probs"] = torch.empty(R, V, device=DEV) if case["probs"] else None
        return s
    s.update(_paging(case, seed))
    T, P, N, H, S = s["qo"][-1], case["page"], s["pages"], case["heads"], case["block"]
    D = case.get("dim", 128)
    s["k_cache"], s["v_cache"] = _codes(gen, (N, H, P, D)), _codes(gen, (N, H, P, D))
    shape = (N, H, P // S)
    if op == "attend":        # scales as a calibration leaves them
        s["k_scales"] = torch.exp2(_normal(gen, shape, torch.float32, 0.4)) / 120.0
        s["v_scales"] = torch.exp2(_normal(gen, shape, torch.float32, 0.7)) / 120.0
        s["q"] = _normal(gen, (T, H * case["group"], D))
        s["scale"] = 1.0 / math.sqrt(D)
        s["out"] = torch.empty(T, H * case["group"], D, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(T, H * case["group"], device=DEV)
    else:                     # powers of two, as the append writes them
        s["k_scales"] = torch.exp2(torch.randint(-8, -5, shape, generator=gen, device=DEV).float())
        s["v_scales"] = torch.exp2(torch.randint(-9, -6, shape, generator=gen, device=DEV).float())
    if op == "append":        # one fused projection's output: queries, keys and values side by side
        # tokens differ in size, so that some raise their block's scale
        size = torch.exp2(_normal(gen, (T, 1, 1), torch.float32))
        fused = (_normal(gen, (T, 3 * H, D), torch.float32) * size).to(_DT[case["rows"]])
        s["k_new"], s["v_new"] = fused[:, H:2 * H], fused[:, 2 * H:]
    if op == "gather":
        rows = sum(s["seq"])
        s["kv_indptr"] = _i32(_indptr(s["seq"]))
        s["k_out"] = torch.empty(rows, H, D, dtype=_DT[case["rows"]], device=DEV)
        s["v_out"] = torch.empty_like(s["k_out"])
    if own:
        import long_context_split_gb300 as skv
        group = case.get("group", 1)
        q = s["q"] if op == "attend" else torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV)
        s["problem"] = skv.AttentionProblem(
            q=q, k_cache=s["k_cache"], v_cache=s["v_cache"], page_table=s["page_table"], seq_lens=s["seq_lens"],
            qo_indptr=s["qo_indptr"], num_q_heads=H * group, num_kv_heads=H, head_dim_qk=D, head_dim_v=D, page_size=P,
            scale=s.get("scale", 1.0), seq_lens_host=s["seq"], qo_indptr_host=s["qo"],
            k_scale=s["k_scales"], v_scale=s["v_scales"])
        if op == "attend":
            s["attention"] = skv.SplitKVAttention(s["problem"])
    return s


# ------------------------------------------------------------------ plain forms
def _owner(indptr, rows):
    """The request of each row."""
    return torch.searchsorted(indptr, torch.arange(rows, device=DEV, dtype=torch.int32), right=True) - 1


def _pages(s):
    P = s["case"]["page"]
    need = (s["seq_lens"].long() + P - 1) // P
    held, n = s["held"].long(), s["free_count"].long()
    grow, back = (need - held).clamp(min=0), (held - need).clamp(min=0)
    grow_at, back_at = torch.cumsum(grow, 0), torch.cumsum(back, 0)
    # ended requests' pages go on the stack, in order
    i = torch.arange(s["back"], device=DEV)
    b = torch.searchsorted(back_at, i, right=True)
    s["free_pages"][n + i] = s["page_table"][b, need[b] + i - (back_at - back)[b]]
    # and the growing ones take from its top, in order
    i = torch.arange(s["grow"], device=DEV)
    b = torch.searchsorted(grow_at, i, right=True)
    s["page_table"][b, held[b] + i - (grow_at - grow)[b]] = s["free_pages"][n + s["back"] - 1 - i]
    s["held_out"].copy_(need)
    s["free_count_out"].copy_(n + s["back"] - s["grow"])
    T = s["tokens"]
    b = _owner(s["qo_indptr"], T)
    pos = s["seq_lens"][b].long() - s["qo_indptr"][b + 1] + torch.arange(T, device=DEV)
    s["slots"].copy_(s["page_table"][b, pos // P].long() * P + pos % P)


def _values(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _e4m3(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _pow2_scale(amax):
    """The smallest power of two (from 2^-126) whose 448-fold is not below amax."""
    frac, exp = torch.frexp(amax)                                  # amax = frac 2^exp, frac in [0.5, 1)
    e = torch.where(frac <= 0.875, exp - 9, exp - 8)               # 448 = 0.875 2^9
    return torch.exp2(torch.where(amax > 0, e, -126).clamp(min=-126).double()).float()


def _append(s):
    case, P, S = s["case"], s["case"]["page"], s["case"]["block"]
    T, per = s["qo"][-1], P // S
    b = _owner(s["qo_indptr"], T)
    pos = s["seq_lens"][b] - s["qo_indptr"][b + 1] + torch.arange(T, device=DEV)
    page, slot = s["page_table"][b, pos // P].long(), (pos % P).long()
    # each request's first block may hold older tokens: those before its first new one (every
    # request of a case has new tokens)
    first = (s["seq_lens"] - (s["qo_indptr"][1:] - s["qo_indptr"][:-1])).long()
    old_n, fblk = first % S, first % P // S
    fpage = s["page_table"].gather(1, (first // P)[:, None])[:, 0].long()
    flat, fflat = page * per + slot // S, fpage * per + fblk
    inside = (fblk * S)[:, None] + torch.arange(S, device=DEV)                                    # [B, S]
    older = torch.arange(S, device=DEV) < old_n[:, None]
    for new, cache, scales in ((s["k_new"], s["k_cache"], s["k_scales"]), (s["v_new"], s["v_cache"], s["v_scales"])):
        N, H = scales.shape[:2]
        x = new.float()
        amax = torch.where(x.isfinite(), x.abs(), 0.0).amax(-1)                                   # [T, H]
        top = torch.zeros(N * per, H, device=DEV).index_reduce_(0, flat, amax, "amax")
        was = scales[fpage, :, fblk]                                                              # [B, H]
        old = torch.zeros(N * per, H, device=DEV)
        old[fflat] = torch.where(old_n[:, None] > 0, was, 0.0)
        scale = torch.where((old > 0) & (top <= E4M3_MAX * old), old, _pow2_scale(top))           # [N per, H]
        # older tokens of a block whose scale has grown
        now = scale[fflat]
        codes = cache[fpage[:, None], :, inside]                                                  # [B, S, H, D]
        again = _e4m3(_values(codes) * was[:, None, :, None] / now[:, None, :, None])
        cache[fpage[:, None], :, inside] = torch.where((older[:, :, None] & (now != was)[:, None])[..., None], again, codes)
        cache[page, :, slot] = _e4m3(x / scale[flat][:, :, None])
        scales[page, :, slot // S] = scale[flat]


def _gather(s):
    case, P, S = s["case"], s["case"]["page"], s["case"]["block"]
    rows = s["k_out"].shape[0]
    b = _owner(s["kv_indptr"], rows)
    pos = torch.arange(rows, device=DEV) - s["kv_indptr"][b]
    page, slot = s["page_table"][b, pos // P].long(), pos % P
    for cache, scales, out in ((s["k_cache"], s["k_scales"], s["k_out"]), (s["v_cache"], s["v_scales"], s["v_out"])):
        out.copy_(_values(cache[page, :, slot]) * scales[page, :, slot // S][..., None])


def _cached(cache, scales, pages, length, S, h):
    """Head h of a request's cached values in float32, [length, D]."""
    P, D = cache.shape[2:]
    x = _values(cache[pages, h]).view(len(pages), P // S, S, D) * scales[pages, h][:, :, None, None]
    return x.view(-1, D)[:length]


def _attend(s):
    case, P, S, g = s["case"], s["case"]["page"], s["case"]["block"], s["case"]["group"]
    for b, (L, T) in enumerate(zip(s["seq"], s["new"])):
        pages = s["page_table"][b, :-(-L // P)].long()
        lo = s["qo"][b]
        visible = torch.arange(L, device=DEV)[None] <= L - T + torch.arange(T, device=DEV)[:, None]
        for h in range(case["heads"]):
            k = _cached(s["k_cache"], s["k_scales"], pages, L, S, h)
            v = _cached(s["v_cache"], s["v_scales"], pages, L, S, h)
            q = s["q"][lo:lo + T, h * g:(h + 1) * g].float()
            x = (q.reshape(T * g, -1) @ k.T).mul_(s["scale"]).view(T, g, L)
            x.masked_fill_(~visible[:, None], -math.inf)
            m = x.amax(-1, keepdim=True)
            e = x.sub_(m).exp_()
            total = e.sum(-1, keepdim=True)
            s["out"][lo:lo + T, h * g:(h + 1) * g] = ((e.view(T * g, L) @ v).view(T, g, -1) / total).to(torch.bfloat16)
            s["lse"][lo:lo + T, h * g:(h + 1) * g] = (m + total.log())[..., 0]


def _sample(s):
    # float64: a cut or a draw next to its border, and sums over the vocabulary
    x = s["logits"].double()
    R, V = x.shape
    ones = torch.ones(R, 1, dtype=torch.float64, device=DEV)
    t = ones if s["temperature"] is None else s["temperature"].double()[:, None]
    top = x.amax(1, keepdim=True)
    greedy = t == 0
    z = torch.where(greedy, torch.where(x == top, 0.0, -math.inf), (x - top) / torch.where(greedy, 1.0, t))
    keep = torch.ones(R, V, dtype=torch.bool, device=DEV)
    if s["min_p"] is not None:
        m = s["min_p"].double()[:, None]
        keep &= (x - top >= t * torch.log(torch.where(m > 0, m, 1.0))) | (m <= 0)
    # equal values in the order of their tokens
    z_sorted, order = torch.sort(torch.where(keep, z, -math.inf), dim=1, descending=True, stable=True)
    w = torch.exp(z_sorted)
    rank = torch.arange(V, device=DEV)[None]
    stay = torch.ones(R, V, dtype=torch.bool, device=DEV)
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        stay &= (rank < k) | (k <= 0)
    w = torch.where(stay | greedy, w, 0.0)
    stay = (w > 0) & (~greedy | (rank == 0))
    w = torch.where(stay, w, 0.0)
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        cum = torch.cumsum(w, 1)
        stay &= (cum - w < p * cum[:, -1:]) | (p >= 1)
    w = torch.zeros_like(w).scatter_(1, order, torch.where(stay, w, 0.0))
    cum = torch.cumsum(w, 1)
    v = torch.arange(V, device=DEV)
    hit = torch.where((cum > s["u"].double()[:, None] * cum[:, -1:]) & (w > 0), v, V).amin(1)
    last = torch.where(w > 0, v, -1).amax(1)
    s["tokens"].copy_(torch.where(hit < V, hit, last))
    if s["probs"] is not None:
        s["probs"].copy_(w / cum[:, -1:])


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        import long_context_split_gb300 as skv
        if op == "pages":
            skv.assign_pages(s["page_table"], s["held"], s["seq_lens"], s["free_pages"], s["free_count"],
                             page_size=s["case"]["page"], held_out=s["held_out"], free_count_out=s["free_count_out"],
                             qo_indptr=s["qo_indptr"], slots=s["slots"])
        elif op == "append":
            skv.kv_append(s["problem"], s["k_new"], s["v_new"])
        elif op == "gather":
            skv.kv_gather(s["problem"], s["kv_indptr"], s["k_out"], s["v_out"])
        elif op == "attend":
            s["attention"].decode(s["out"], s["lse"])
        else:
            skv.sample_tokens(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                              min_p=s["min_p"], out_tokens=s["tokens"], probs_out=s["probs"])
    else:
        {"pages": _pages, "append": _append, "gather": _gather, "attend": _attend, "sample": _sample}[op](s)
    if op == "pages":
        return [s["page_table"], s["held_out"], s["free_pages"], s["free_count_out"], s["slots"]]
    if op == "append":
        return [s["k_cache"].view(torch.float8_e4m3fn), s["v_cache"].view(torch.float8_e4m3fn), s["k_scales"], s["v_scales"]]
    if op == "gather":
        return [s["k_out"], s["v_out"]]
    if op == "attend":
        return [s["out"], s["lse"]]
    return [s["tokens"]] if s["probs"] is None else [s["tokens"], s["probs"]]


# ------------------------------------------------------------------ float64, from the definitions
def _nearest_e4m3(x):
    """The E4M3 number nearest to each x (ties to the even one), saturated."""
    x = x.clamp(-E4M3_MAX, E4M3_MAX)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3.0)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_append(s, cache, scales, new):
    case, P, S = s["case"], s["case"]["page"], s["case"]["block"]
    full, sc = cache.view(torch.float8_e4m3fn).double(), scales.double()
    for b in range(case["batch"]):
        at = s["seq"][b] - s["new"][b]
        while at < s["seq"][b]:
            # one block at a time: tokens lo .. hi-1 of it are there, at .. end-1 are new
            lo, end = at // S * S, min(at // S * S + S, s["seq"][b])
            page, t = int(s["table_host"][b, lo // P]), lo % P // S
            r = s["qo"][b] + at - (s["seq"][b] - s["new"][b])
            x = new[r:r + end - at].double().transpose(0, 1)                                      # [H, n, D]
            amax = x.abs().amax((1, 2))
            was = sc[page, :, t].clone()
            least = torch.exp2(torch.ceil(torch.log2(amax / E4M3_MAX) - 0.5).clamp(min=-126.0))   # or twice that
            least = torch.where(amax <= E4M3_MAX * least, least, 2.0 * least)
            now = least if lo == at else torch.where(amax <= E4M3_MAX * was, was, least)
            here = full[page, :, lo % P:lo % P + at - lo]
            full[page, :, lo % P:lo % P + at - lo] = torch.where(
                (now == was)[:, None, None], here, _nearest_e4m3(here * (was / now)[:, None, None]))
            full[page, :, at % P:at % P + end - at] = _nearest_e4m3(x / now[:, None, None])
            sc[page, :, t] = now
            at = end
    return full, sc


def exact(case, seed):
    op = case["op"]
    if op == "pages" or (op == "sample" and not case["probs"]):
        return None                                    # whole numbers only
    s = prepare(case, seed)
    if op == "append":
        s["table_host"] = s["page_table"].cpu()
        k, ks = _exact_append(s, s["k_cache"], s["k_scales"], s["k_new"])
        v, vs = _exact_append(s, s["v_cache"], s["v_scales"], s["v_new"])
        return [k, v, ks, vs]
    if op == "sample":
        out = torch.zeros(case["rows"], case["vocab"], dtype=torch.float64, device=DEV)
        host = {n: None if s[n] is None else s[n].tolist() for n in ("temperature", "top_k", "top_p", "min_p")}
        for r in range(case["rows"]):
            get = lambda n, off: off if host[n] is None else host[n][r]  # noqa: E731
            x, t = s["logits"][r].double(), get("temperature", 1.0)
            x, order = torch.sort(x, descending=True, stable=True)
            if t == 0:
                out[r, order[0]] = 1.0
                continue
            z = (x - x[0]) / t
            if get("min_p", 0.0) > 0:
                z = z[z >= math.log(get("min_p", 0.0))]
            if get("top_k", 0) > 0:
                z = z[:get("top_k", 0)]
            p = torch.softmax(z, 0)
            if get("top_p", 1.0) < 1:
                before = torch.cumsum(p, 0) - p
                p = p[before < get("top_p", 1.0)]
                p = p / p.sum()
            out[r, order[:p.numel()]] = p
        return [None, out]
    P, S = case["page"], case["block"]
    wide = lambda c, sc: (c.view(torch.float8_e4m3fn).double().view(*c.shape[:2], P // S, S, -1)  # noqa: E731
                          * sc.double()[..., None, None]).view(c.shape)
    if op == "gather":
        out = []
        for cache, scales in ((s["k_cache"], s["k_scales"]), (s["v_cache"], s["v_scales"])):
            full, rows = wide(cache, scales).transpose(1, 2), []
            for b in range(case["batch"]):
                pages = s["page_table"][b, :-(-s["seq"][b] // P)].long()
                rows.append(full[pages].flatten(0, 1)[:s["seq"][b]])
            out.append(torch.cat(rows))
        return out
    H, g = case["heads"], case["group"]
    out = torch.empty(s["qo"][-1], H * g, 128, dtype=torch.float64, device=DEV)
    lse = torch.empty(s["qo"][-1], H * g, dtype=torch.float64, device=DEV)
    for b in range(case["batch"]):
        pages = s["page_table"][b, :-(-s["seq"][b] // P)].long()
        lo, hi, L = s["qo"][b], s["qo"][b + 1], s["seq"][b]
        hide = torch.arange(L, device=DEV)[None] > L - (hi - lo) + torch.arange(hi - lo, device=DEV)[:, None]
        for h in range(H):
            k = wide(s["k_cache"][pages, h:h + 1], s["k_scales"][pages, h:h + 1]).reshape(-1, 128)[:L]
            v = wide(s["v_cache"][pages, h:h + 1], s["v_scales"][pages, h:h + 1]).reshape(-1, 128)[:L]
            for j in range(h * g, h * g + g):
                a = (s["q"][lo:hi, j].double() @ k.T * s["scale"]).masked_fill(hide, -math.inf)
                lse[lo:hi, j] = torch.logsumexp(a, 1)
                out[lo:hi, j] = torch.softmax(a, 1) @ v
    return [out, lse]
