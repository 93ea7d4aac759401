"""Cases for the operators that surround split-KV attention: writing a paged KV cache (with E4M3
quantisation), reading it back, latent attention from queries of the model's own width in its
expanded and absorbed forms, and the verification of drafted tokens.

``run`` computes a case in plain torch operations (float32, or float64 where float32 loses what
matters) when ``own`` is false, and through the package's entry points when it is true; ``exact``
computes it from the definition in float64.

Batches are ragged and follow the package's conventions: request b owns rows
qo_indptr[b] .. qo_indptr[b+1]-1 of the new tokens, which are the last ones of its seq_lens[b]
cached tokens; token j of request b is in page page_table[b][j // P], slot j % P.
"""
import math
import random

import torch

own = False

NOPE, ROPE, LATENT, VDIM = 128, 64, 512, 128       # latent attention's widths (512 + 64 per token)
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new token for each of 64 decoding requests, written to an E4M3 cache (8 KV heads of
        # 128): the call that a decode step makes in every layer, where latency counts
        dict(name="append_decode_e4m3", op="append", kind="gqa", cache="e4m3", rows="bf16", batch=64, heads=8, dim=128,
             page=64, hist_lo=1024, hist_hi=16384, new_lo=1, new_hi=1, shape=1),
        # prefill chunks of up to 4k tokens, K and V sliced out of one fused projection (strided
        # rows), quantised into an E4M3 cache
        dict(name="append_prefill_e4m3", op="append", kind="gqa", cache="e4m3", rows="bf16", batch=8, heads=8, dim=128,
             page=64, hist_lo=1, hist_hi=4096, new_lo=1500, new_hi=4096, shape=2),
        # latent rows of a ragged batch (512 latent + 64 rotary columns from two tensors) into
        # a bf16 latent cache
        dict(name="append_latent_bf16", op="append", kind="mla", cache="bf16", rows="bf16", batch=24, heads=1, dim=576,
             page=64, hist_lo=1, hist_hi=8192, new_lo=1, new_hi=2048, shape=3),
        # an E4M3 cache of eight long requests read back as bf16 rows (moving a request to
        # another cache layout or another machine)
        dict(name="gather_e4m3", op="gather", kind="gqa", cache="e4m3", rows="bf16", batch=8, heads=8, dim=128,
             page=64, hist_lo=8192, hist_hi=24576, new_lo=1, new_hi=1, shape=4),
        # latent rows of short ragged requests, read back as float32
        dict(name="gather_latent", op="gather", kind="mla", cache="bf16", rows="f32", batch=12, heads=1, dim=576,
             page=64, hist_lo=1, hist_hi=700, new_lo=1, new_hi=5, shape=5),
        # short fresh prompts, ragged (a serving batch's smallest prefill)
        dict(name="expanded_short", op="expanded", cache="bf16", batch=5, heads=128, page=64,
             hist_lo=0, hist_hi=0, new_lo=33, new_hi=300, shape=6),
        # two long fresh prompts
        dict(name="expanded_prompt", op="expanded", cache="bf16", batch=2, heads=128, page=64,
             hist_lo=0, hist_hi=0, new_lo=3500, new_hi=4096, shape=7),
        # a chunk of new tokens after a long history in an E4M3 latent cache, 32 of the heads
        dict(name="expanded_chunk_e4m3", op="expanded", cache="e4m3", batch=2, heads=32, page=64,
             hist_lo=12000, hist_hi=20000, new_lo=900, new_hi=2048, shape=8),
        # one decoding request: one token, the smallest latent-attention call
        dict(name="absorbed_single", op="absorbed", cache="bf16", batch=1, heads=128, page=64,
             hist_lo=4000, hist_hi=4200, new_lo=1, new_hi=1, shape=9),
        # a decode batch of 64 requests, log-uniform histories
        dict(name="absorbed_batch", op="absorbed", cache="bf16", batch=64, heads=128, page=64,
             hist_lo=1024, hist_hi=16384, new_lo=1, new_hi=1, shape=10),
        # three drafts for each of four requests (vocabulary of 32,000, all probabilities positive)
        dict(name="verify_small", op="verify", batch=4, vocab=32000, new_lo=4, new_hi=4, nucleus=False, shape=11),
        # 15 drafts for each of 48 requests (16 query tokens each) over 128,000 tokens, the
        # distributions truncated to their most likely tokens
        dict(name="verify_batch", op="verify", batch=48, vocab=128000, new_lo=16, new_hi=16, nucleus=True, shape=12),
    ]


def _log_int(rng, lo, hi):
    if hi <= lo:
        return lo
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(max(1, lo)), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "gather", "expanded", "absorbed", "verify"])
    shape = rng.randrange(1 << 30)
    if op in ("append", "gather"):
        kind = rng.choice(["gqa", "gqa", "mla"])
        batch = _log_int(rng, 1, 96)
        heads, dim = (rng.choice([1, 2, 4, 8]), rng.choice([64, 128])) if kind == "gqa" else (1, LATENT + ROPE)
        tokens = _log_int(rng, batch, 20000 if op == "append" else 60000)     # about so many rows
        most = max(1, 2 * tokens // batch)
        hist, new = (_log_int(rng, 1, 4096), most) if op == "append" else (most, 4)
        return dict(op=op, kind=kind, cache=rng.choice(["bf16", "e4m3", "e4m3", "f32"]), rows=rng.choice(["bf16", "f32"]),
                    batch=batch, heads=heads, dim=dim, page=rng.choice([16, 64, 128]),
                    hist_lo=1, hist_hi=hist, new_lo=1, new_hi=min(new, 8192), shape=shape)
    if op == "expanded":
        batch, heads = rng.randint(1, 4), rng.choice([8, 16, 32, 64, 128])
        new = _log_int(rng, 16, 2048)
        hist = rng.choice([0, _log_int(rng, 64, 8192)])
        case = dict(op=op, cache=rng.choice(["bf16", "bf16", "e4m3"]), batch=batch, heads=heads, page=rng.choice([16, 64, 128]),
                    hist_lo=0 if hist == 0 else max(1, hist // 4), hist_hi=hist, new_lo=max(1, new // 8), new_hi=new, shape=shape)
        while work(case)["flops"] > 1e12:              # no more than the longest listed prompts
            case["heads"] //= 2
        return case
    if op == "absorbed":
        return dict(op=op, cache=rng.choice(["bf16", "bf16", "e4m3"]), batch=_log_int(rng, 1, 48), heads=128, page=64,
                    hist_lo=64, hist_hi=_log_int(rng, 128, 12000), new_lo=1, new_hi=rng.choice([1, 1, 2, 4]), shape=shape)
    return dict(op=op, batch=_log_int(rng, 1, 48), vocab=_log_int(rng, 1000, 128000), new_lo=1, new_hi=rng.randint(1, 12),
                nucleus=rng.random() < 0.5, shape=shape)


def _lengths(case):
    """(seq_lens, q_lens) of a case: histories log-uniform, new tokens log-uniform."""
    rng = random.Random(case["shape"])
    q = [_log_int(rng, case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    h = [_log_int(rng, case["hist_lo"], case["hist_hi"]) if case.get("hist_hi") else 0 for _ in range(case["batch"])]
    return [a + b for a, b in zip(h, q)], q


_ESIZE = {"bf16": 2, "f32": 4, "e4m3": 1}


def _pairs(case):
    """(query, key) pairs that the causal rule lets meet."""
    return sum(t * (n - t) + t * (t + 1) // 2 for n, t in zip(*_lengths(case)))


def work(case):
    if case["op"] == "verify":
        _, q = _lengths(dict(case, hist_lo=1, hist_hi=1))
        rows = sum(1 for t in q if t > 0)
        # two entries per draft, then one row of the target's and the draft's distribution
        return dict(bytes=rows * case["vocab"] * 8 + sum(q) * 24, flops=rows * case["vocab"] * 3)
    seq, q = _lengths(case)
    if case["op"] in ("append", "gather"):
        per = case["heads"] * case["dim"] * (2 if case["kind"] == "gqa" else 1)
        n = sum(q) if case["op"] == "append" else sum(seq)
        return dict(bytes=n * per * (_ESIZE[case["rows"]] + _ESIZE[case["cache"]]), flops=n * per)
    H, T, L = case["heads"], sum(q), sum(seq)
    moved = L * (LATENT + ROPE) * _ESIZE[case["cache"]] + T * H * (NOPE + ROPE + VDIM) * 2 + H * (NOPE + VDIM) * LATENT * 2
    if case["op"] == "expanded":
        flops = 2 * H * (L * LATENT * (NOPE + VDIM) + _pairs(case) * (NOPE + ROPE + VDIM))
    else:
        flops = 2 * H * (T * LATENT * (NOPE + VDIM) + _pairs(case) * (2 * LATENT + ROPE))
    return dict(bytes=moved, flops=flops)


# ------------------------------------------------------------------ inputs
_DT = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.uint8}
DEV = "cuda"


def _normal(gen, shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32) * scale).to(dtype)


def _cache(gen, shape, kind, scale):
    """A cache full of values: E4M3 codes of N(0, 1) / scale, or N(0, 1) itself."""
    if kind == "e4m3":
        return (_normal(gen, shape, torch.float32) / scale).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    return _normal(gen, shape, _DT[kind])


def _paging(case, seed):
    """Lengths and a shuffled page table on the device, and their host copies."""
    seq, q = _lengths(case)
    P = case["page"]
    pages = [-(-n // P) for n in seq]
    gen = torch.Generator().manual_seed(seed)
    perm = torch.randperm(sum(pages), generator=gen, dtype=torch.int32)
    table = torch.full((len(seq), max(pages)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
    qo = [0]
    for t in q:
        qo.append(qo[-1] + t)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    return dict(page_table=table.to(DEV), seq_lens=i32(seq), qo_indptr=i32(qo), seq=seq, new=q, qo=qo, pages=sum(pages))


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "verify":
        _, q = _lengths(dict(case, hist_lo=1, hist_hi=1))
        qo = [0]
        for t in q:
            qo.append(qo[-1] + t)
        T, V = qo[-1], case["vocab"]
        logits = torch.randn(T, V, generator=gen, device=DEV) * 2.5
        draft = logits + torch.randn(T, V, generator=gen, device=DEV) * 0.5
        p, d = torch.softmax(logits, 1), torch.softmax(draft, 1)
        if case["nucleus"]:                            # tokens far below the row's most likely one are cut
            p = torch.where(p < p.amax(1, keepdim=True) * 1e-3, 0.0, p)
            d = torch.where(d < d.amax(1, keepdim=True) * 1e-3, 0.0, d)
            p, d = p / p.sum(1, keepdim=True), d / d.sum(1, keepdim=True)
        picks = torch.multinomial(d, 1, generator=gen).view(-1).to(torch.int32)    # the token drawn after row r
        tokens = torch.cat([torch.zeros(1, dtype=torch.int32, device=DEV), picks[:-1]])
        s.update(target=p, draft=d, tokens=tokens, qo_indptr=torch.tensor(qo, dtype=torch.int32, device=DEV),
                 accept_u=torch.rand(T, generator=gen, device=DEV), sample_u=torch.rand(case["batch"], generator=gen, device=DEV),
                 seq_lens=torch.tensor(q, dtype=torch.int32, device=DEV) + 100,
                 out_tokens=torch.empty(T, dtype=torch.int32, device=DEV),
                 accepted=torch.empty(case["batch"], dtype=torch.int32, device=DEV),
                 new_lens=torch.empty(case["batch"], dtype=torch.int32, device=DEV))
        return s
    s.update(_paging(case, seed))
    T, P, N = s["qo"][-1], case["page"], s["pages"]
    e4m3 = case["cache"] == "e4m3"
    s["k_scale"], s["v_scale"] = (0.0625, 0.05) if e4m3 else (1.0, 1.0)
    s["scales"] = dict(k_scale=s["k_scale"], v_scale=s["v_scale"]) if e4m3 else {}
    if case["op"] in ("append", "gather"):
        H, D, gqa = case["heads"], case["dim"], case["kind"] == "gqa"
        shape = (N, H, P, D) if gqa else (N, P, D)
        s["k_cache"] = _cache(gen, shape, case["cache"], s["k_scale"])
        s["v_cache"] = _cache(gen, shape, case["cache"], s["v_scale"]) if gqa else None
        rdt = _DT[case["rows"]]
        if case["op"] == "append":
            if gqa:       # one fused projection's output: queries, keys and values side by side
                fused = _normal(gen, (T, 3 * H, D), rdt)
                s["k_new"], s["v_new"] = fused[:, H:2 * H], fused[:, 2 * H:]
            else:
                s["k_new"], s["v_new"] = _normal(gen, (T, LATENT), rdt), _normal(gen, (T, ROPE), rdt)
        else:
            rows = sum(s["seq"])
            at = [0]
            for n in s["seq"]:
                at.append(at[-1] + n)
            s["kv_indptr"] = torch.tensor(at, dtype=torch.int32, device=DEV)
            wide = (lambda w: (rows, H, D)) if gqa else (lambda w: (rows, w))
            s["k_out"] = torch.empty(wide(LATENT), dtype=rdt, device=DEV)
            s["v_out"] = torch.empty(wide(ROPE), dtype=rdt, device=DEV)
        if own:
            import long_context_split_gb300 as skv
            q = torch.empty(T, H, D, dtype=torch.bfloat16 if e4m3 else _DT[case["cache"]], device=DEV)
            s["problem"] = skv.AttentionProblem(
                q=q, k_cache=s["k_cache"], v_cache=s["v_cache"], page_table=s["page_table"], seq_lens=s["seq_lens"],
                qo_indptr=s["qo_indptr"], num_q_heads=H, num_kv_heads=H, head_dim_qk=D, head_dim_v=D if gqa else LATENT,
                page_size=P, scale=1.0 / math.sqrt(D), kind=case["kind"], seq_lens_host=s["seq"], qo_indptr_host=s["qo"],
                **s["scales"])
        return s
    H = case["heads"]
    s["k_cache"] = _cache(gen, (N, P, LATENT + ROPE), case["cache"], s["k_scale"])
    s["w_kv_b"] = _normal(gen, (H, NOPE + VDIM, LATENT), scale=1.0 / math.sqrt(LATENT))
    s["q"] = _normal(gen, (T, H, NOPE + ROPE))
    s["out"] = torch.empty(T, H, VDIM, dtype=torch.bfloat16, device=DEV)
    s["scale"] = 1.0 / math.sqrt(NOPE + ROPE)
    if own:
        import long_context_split_gb300 as skv
        s["attention"] = skv.LatentAttention(
            k_cache=s["k_cache"], w_kv_b=s["w_kv_b"], page_table=s["page_table"], seq_lens=s["seq_lens"],
            qo_indptr=s["qo_indptr"], scale=s["scale"], form=case["op"], seq_lens_host=s["seq"], qo_indptr_host=s["qo"],
            k_scale=s["k_scale"] if e4m3 else None)
    return s


# ------------------------------------------------------------------ plain forms
def _values(codes, kind, scale):
    """The float32 values that a cache's entries stand for."""
    return codes.view(torch.float8_e4m3fn).float() * scale if kind == "e4m3" else codes.float()


def _shown(codes, kind):
    """A cache as values (E4M3 codes as the numbers they encode; the scale is the caller's)."""
    return codes.view(torch.float8_e4m3fn) if kind == "e4m3" and codes is not None else codes


def _encode(x, kind, scale):
    if kind != "e4m3":
        return x.to(_DT[kind])
    return (x.float() / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _owner(indptr, rows):
    """The request of each row."""
    return torch.searchsorted(indptr, torch.arange(rows, device=DEV, dtype=torch.int32), right=True) - 1


def _append(s):
    case, P = s["case"], s["case"]["page"]
    T = s["qo"][-1]
    b = _owner(s["qo_indptr"], T)
    pos = s["seq_lens"][b] - s["qo_indptr"][b + 1] + torch.arange(T, device=DEV)
    page, slot = s["page_table"][b, pos // P].long(), pos % P
    if case["kind"] == "gqa":
        s["k_cache"][page, :, slot] = _encode(s["k_new"], case["cache"], s["k_scale"])
        s["v_cache"][page, :, slot] = _encode(s["v_new"], case["cache"], s["v_scale"])
    else:
        s["k_cache"][page, slot] = _encode(torch.cat([s["k_new"], s["v_new"]], 1), case["cache"], s["k_scale"])


def _gather(s):
    case, P = s["case"], s["case"]["page"]
    rows = s["k_out"].shape[0]
    b = _owner(s["kv_indptr"], rows)
    pos = torch.arange(rows, device=DEV) - s["kv_indptr"][b]
    page, slot = s["page_table"][b, pos // P].long(), pos % P
    if case["kind"] == "gqa":
        s["k_out"].copy_(_values(s["k_cache"][page, :, slot], case["cache"], s["k_scale"]))
        s["v_out"].copy_(_values(s["v_cache"][page, :, slot], case["cache"], s["v_scale"]))
    else:
        x = _values(s["k_cache"][page, slot], case["cache"], s["k_scale"])
        s["k_out"].copy_(x[:, :LATENT])
        s["v_out"].copy_(x[:, LATENT:])


def _padded(s):
    """Latent rows [B, Lmax, 576] and queries [B, Tmax, H, 192] in float32, padded, with the
    positions of the padded queries' rows and the mask of visible keys [B, Tmax, Lmax]."""
    P = s["case"]["page"]
    seq, qo = s["seq_lens"].long(), s["qo_indptr"].long()
    ql = qo[1:] - qo[:-1]
    lmax, tmax = max(s["seq"]), max(s["new"])
    j = torch.arange(lmax, device=DEV)
    page = s["page_table"].long()[:, j // P].clamp(min=0)
    rows = _values(s["k_cache"].view(-1, LATENT + ROPE)[page * P + j % P], s["case"]["cache"], s["k_scale"])
    i = torch.arange(tmax, device=DEV)
    at = (qo[:-1, None] + i).clamp(max=qo[-1] - 1)
    visible = j <= (seq - ql)[:, None, None] + i[None, :, None]
    return rows, s["q"][at].float(), visible & (j < seq[:, None])[:, None], i < ql[:, None]


def _softmax(scores, visible):
    """Softmax over the last axis of scores [B, H, T, L]; masked keys weigh nothing."""
    scores = scores.masked_fill_(~visible[:, None], -math.inf)
    scores = scores.sub_(scores.amax(-1, keepdim=True)).exp_()
    return scores.div_(scores.sum(-1, keepdim=True))


def _expanded(s):
    rows, q, visible, real = _padded(s)
    B, L, _ = rows.shape
    T, H = q.shape[1:3]
    w = s["w_kv_b"].float()
    kv = (rows[..., :LATENT].reshape(B * L, LATENT) @ w.reshape(-1, LATENT).T).view(B, L, H, NOPE + VDIM)
    k = torch.cat([kv[..., :NOPE], rows[:, :, None, LATENT:].expand(B, L, H, ROPE)], -1)
    scores = torch.matmul(q.transpose(1, 2), k.permute(0, 2, 3, 1)).mul_(s["scale"])
    p = _softmax(scores, visible)
    out = torch.matmul(p, kv[..., NOPE:].transpose(1, 2)).transpose(1, 2)
    s["out"].copy_(out[real])


def _absorbed(s):
    rows, q, visible, real = _padded(s)
    B, T, H, _ = q.shape
    w = s["w_kv_b"].float()
    q_lat = torch.matmul(q[..., :NOPE].reshape(B * T, H, NOPE).transpose(0, 1), w[:, :NOPE])      # [H, BT, 512]
    q_all = torch.cat([q_lat.transpose(0, 1).reshape(B, T, H, LATENT), q[..., NOPE:]], -1)
    scores = torch.matmul(q_all.view(B, T * H, -1), rows.transpose(1, 2)).mul_(s["scale"])
    p = _softmax(scores.view(B, T, H, -1).transpose(1, 2), visible)
    o = torch.matmul(p.transpose(1, 2).reshape(B, T * H, -1), rows[..., :LATENT])                  # [B, TH, 512]
    out = torch.matmul(o.view(B * T, H, LATENT).transpose(0, 1), w[:, NOPE:].transpose(1, 2))
    s["out"].copy_(out.transpose(0, 1).reshape(B, T, H, VDIM)[real])


def _verify(s):
    # float64: an acceptance test next to its border, and sums over the vocabulary
    qo, V = s["qo_indptr"].long(), s["case"]["vocab"]
    first, n = qo[:-1], qo[1:] - qo[:-1] - 1                                   # drafts per request
    T, most = s["tokens"].numel(), s["case"]["new_hi"]
    i = torch.arange(most, device=DEV)
    r = (first[:, None] + i).clamp(max=T - 1)
    nxt = s["tokens"][(r + 1).clamp(max=T - 1)].long()
    take = s["accept_u"][r].double() * s["draft"][r, nxt].double() < s["target"][r, nxt].double()
    take = take & (i < n[:, None])
    a = torch.cumprod(take.int(), 1).sum(1)                                    # accepted drafts
    row = first + a
    p = s["target"][row].double()
    w = torch.where((a < n)[:, None], p - s["draft"][row].double(), p).clamp_(min=0.0)
    w = torch.where(w.sum(1, keepdim=True) > 0, w, p)
    cdf = torch.cumsum(w, 1)
    v = torch.arange(V, device=DEV)
    hit = torch.where((cdf > s["sample_u"].double()[:, None] * cdf[:, -1:]) & (w > 0), v, V).amin(1)
    last = torch.where(w > 0, v, -1).amax(1)
    new = torch.where(hit < V, hit, last)
    b = _owner(s["qo_indptr"], T)
    at = torch.arange(T, device=DEV) - first[b]
    kept = s["tokens"][(torch.arange(T, device=DEV) + 1).clamp(max=T - 1)].long()
    s["out_tokens"].copy_(torch.where(at < a[b], kept, torch.where(at == a[b], new[b], -1)))
    s["accepted"].copy_(a)
    s["new_lens"].copy_(s["seq_lens"] - n + a)


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        import long_context_split_gb300 as skv
        if op == "append":
            skv.kv_append(s["problem"], s["k_new"], s["v_new"])
        elif op == "gather":
            skv.kv_gather(s["problem"], s["kv_indptr"], s["k_out"], s["v_out"])
        elif op == "verify":
            skv.verify_drafts(s["tokens"], s["qo_indptr"], s["target"], s["draft"], s["accept_u"], s["sample_u"],
                              s["out_tokens"], s["accepted"], seq_lens=s["seq_lens"], seq_lens_out=s["new_lens"])
        else:
            s["attention"](s["q"], out=s["out"])
    else:
        {"append": _append, "gather": _gather, "expanded": _expanded, "absorbed": _absorbed, "verify": _verify}[op](s)
    if op == "append":
        return [_shown(s["k_cache"], case["cache"]), _shown(s["v_cache"], case["cache"])]
    if op == "gather":
        return [s["k_out"], s["v_out"]]
    if op == "verify":
        return [s["out_tokens"], s["accepted"], s["new_lens"]]
    return s["out"]


# ------------------------------------------------------------------ float64, from the definitions
def _e4m3_of(x):
    """The E4M3 number nearest to each x (ties to the even one), saturated."""
    x = x.clamp(-E4M3_MAX, E4M3_MAX)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3.0)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _token_rows(s, cache, b, lo, hi):
    """Tokens lo .. hi-1 of request b in a cache, as stored."""
    P = s["case"]["page"]
    t = s["page_table"][b].long()
    j = torch.arange(lo, hi, device=DEV)
    return cache[t[j // P], :, j % P] if s["case"].get("kind") == "gqa" else cache[t[j // P], j % P]


def exact(case, seed):
    if case["op"] == "verify":
        return None                                    # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "append":
        out = []
        for cache, new, scale in (("k_cache", s["k_new"], s["k_scale"]), ("v_cache", s["v_new"], s["v_scale"])):
            if s[cache] is None:
                out.append(None)
                continue
            if case["kind"] == "mla":
                new = torch.cat([s["k_new"], s["v_new"]], 1)
            full = _shown(s[cache], case["cache"]).double()
            x = new.double() / scale if case["cache"] == "e4m3" else new.double()
            x = _e4m3_of(x) if case["cache"] == "e4m3" else x.to(_DT[case["cache"]]).double()
            for b in range(case["batch"]):
                j = torch.arange(s["seq"][b] - s["new"][b], s["seq"][b], device=DEV)
                page = s["page_table"][b].long()[j // case["page"]]
                mine = x[s["qo"][b]:s["qo"][b + 1]]
                if case["kind"] == "gqa":
                    full[page, :, j % case["page"]] = mine
                else:
                    full[page, j % case["page"]] = mine
            out.append(full)
        return out
    if case["op"] == "gather":
        k, v = [], []
        for b in range(case["batch"]):
            rows = _shown(_token_rows(s, s["k_cache"], b, 0, s["seq"][b]), case["cache"]).double() * s["k_scale"]
            if case["kind"] == "gqa":
                k.append(rows)
                v.append(_shown(_token_rows(s, s["v_cache"], b, 0, s["seq"][b]), case["cache"]).double() * s["v_scale"])
            else:
                k.append(rows[:, :LATENT])
                v.append(rows[:, LATENT:])
        return [torch.cat(k), torch.cat(v)]
    # latent attention, one request at a time: few query rows meet the latent rows themselves, many
    # meet one head's expanded keys and values at a time
    out = torch.empty(s["qo"][-1], case["heads"], VDIM, dtype=torch.float64, device=DEV)
    for b in range(case["batch"]):
        c = _shown(_token_rows(s, s["k_cache"], b, 0, s["seq"][b]), case["cache"]).double() * s["k_scale"]
        lo, hi = s["qo"][b], s["qo"][b + 1]
        hide = torch.arange(s["seq"][b], device=DEV)[None, :] > s["seq"][b] - (hi - lo) + torch.arange(hi - lo, device=DEV)[:, None]
        if hi - lo <= 8:
            w, q = s["w_kv_b"].double(), s["q"][lo:hi].double()
            a = torch.einsum("thd,hdc->htc", q[..., :NOPE], w[:, :NOPE]) @ c[:, :LATENT].T
            a = (a + q[..., NOPE:].transpose(0, 1) @ c[:, LATENT:].T) * s["scale"]
            a = torch.softmax(a.masked_fill(hide, -math.inf), 2)
            out[lo:hi] = torch.einsum("htc,hvc->thv", a @ c[:, :LATENT], w[:, NOPE:])
            continue
        for h in range(case["heads"]):
            w, q = s["w_kv_b"][h].double(), s["q"][lo:hi, h].double()
            kv = c[:, :LATENT] @ w.T
            a = (q[:, :NOPE] @ kv[:, :NOPE].T + q[:, NOPE:] @ c[:, LATENT:].T) * s["scale"]
            a = torch.softmax(a.masked_fill(hide, -math.inf), 1)
            out[lo:hi, h] = a @ kv[:, NOPE:]
    return out
