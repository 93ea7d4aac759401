"""A serving loop over a cache with block scales, all on the GPU: pages from lengths, the new tokens' rows into the cache,
attention of drafted blocks over it, the targets' distributions from logits, verification of the drafts, pages of
refused ones back.  Cached values are read back with kv_gather (exact, its own test) and attention over them is
checked against float64 with the bounds of ``block_util``; pages are counted; the verified tokens are
checked against a restatement of the whole step from the same random numbers."""
import math

import numpy as np
import pytest
import torch

import long_context_split_gb300 as skv
from tests.block_util import BlockBatch, check_attention
from tests.test_gpu_sample import reference

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("page,block,heads,group", [(64, 16, 2, 8), (128, 64, 1, 4)])
def test_drafted_blocks_from_pages_to_tokens(page, block, heads, group):
    B, D, V, drafts, rounds = 4, 128, 700, 3, 4
    g = torch.Generator().manual_seed(page)
    total = 30
    k = torch.full((total, heads, page, D), 0x7F, dtype=torch.uint8, device="cuda")          # NaN everywhere
    v = k.clone()
    ks = torch.full((total, heads, page // block), float("nan"), device="cuda")
    vs = ks.clone()
    table, held = torch.full((B, 8), -1, dtype=torch.int32, device="cuda"), i32([0] * B)
    free, count = torch.randperm(total, generator=g).int().cuda(), i32([total])
    err = i32([0])
    lens = [0] * B
    prompts = [100, 61, 7, 300]
    for step in range(rounds + 1):
        new = prompts if step == 0 else [1 + drafts] * B
        if step == rounds:
            new[2], lens[2] = 0, 0                   # request 2 has ended: its pages come back
        seq = [n + t for n, t in zip(lens, new)]
        qo = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        T = int(qo[-1])
        slots = torch.empty(T, dtype=torch.int64, device="cuda")
        seq_dev = i32(seq)
        skv.assign_pages(table, held, seq_dev, free, count, page_size=page, qo_indptr=i32(qo.tolist()), slots=slots, dev_error_word=err)
        need = [-(-n // page) for n in seq]
        t_host, n_free = table.cpu().numpy(), int(count)
        assert held.tolist() == need and n_free == total - sum(need)
        ids = [int(x) for b in range(B) for x in t_host[b, :need[b]]] + free[:n_free].tolist()
        assert sorted(ids) == list(range(total))     # every page once: with a request or free
        want = [t_host[b, p // page] * page + p % page for b in range(B) for p in range(seq[b] - new[b], seq[b])]
        assert slots.tolist() == want
        live = [b for b in range(B) if seq[b] > 0]
        qo_l = np.concatenate([[0], np.cumsum([new[b] for b in live])]).astype(np.int32)
        q = torch.randn(T, heads * group, D, generator=g).bfloat16()
        problem = skv.AttentionProblem(
            q=q.cuda(), k_cache=k, v_cache=v, page_table=table[live].contiguous(), seq_lens=i32([seq[b] for b in live]),
            qo_indptr=i32(qo_l.tolist()), num_q_heads=heads * group, num_kv_heads=heads, head_dim_qk=D, head_dim_v=D, page_size=page,
            scale=1 / math.sqrt(D), k_scale=ks, v_scale=vs)
        rows = [(torch.randn(T, heads, D, generator=g) * torch.exp2(torch.randn(T, 1, 1, generator=g))).bfloat16() for _ in range(2)]
        skv.kv_append(problem, rows[0].cuda(), rows[1].cuda(), dev_error_word=err)
        # the new tokens' values: within half a step of E4M3 of their block's largest
        at = i32(np.concatenate([[0], np.cumsum([seq[b] for b in live])]).tolist())
        ko, vo = (torch.empty(int(at[-1]), heads, D, device="cuda") for _ in range(2))
        skv.kv_gather(problem, at, ko, vo, dev_error_word=err)
        for i, b in enumerate(live):
            n0, n1 = int(at[i]) + seq[b] - new[b], int(at[i + 1])
            for got, x in ((ko, rows[0]), (vo, rows[1])):
                mine = x[qo[b]:qo[b + 1]].float()
                # a scale is below twice the largest / 448: 2^-4 of a value, or half a subnormal step (2^-10 scales)
                top = got[int(at[i]):n1].abs().amax().cpu()
                assert ((got[n0:n1].cpu() - mine).abs() <= mine.abs() * 2.0 ** -4 + 2 * top / 448 * 2.0 ** -10).all()
        att = skv.SplitKVAttention(problem)
        out, lse = att.decode()
        att.check_device_error()
        host = BlockBatch([seq[b] for b in live], [new[b] for b in live], heads=heads, group=group, dim=D, page=page, block=block, dev="cpu")
        host.table, host.q, host.qo = t_host[live], q, qo_l
        check_attention(host, out, lse, ref=host.attention(tuple(x.cpu().numpy() for x in (k, ks, v, vs))))
        if step == 0:
            lens = seq
            continue
        # targets and drafts from logits, then the verification
        logits = torch.randn(T, V, generator=g) * 3
        near = logits + 0.5 * torch.randn(T, V, generator=g)
        settings = dict(temperature=torch.full((T,), 0.8, device="cuda"), top_k=torch.full((T,), 40, dtype=torch.int32, device="cuda"),
                        top_p=torch.full((T,), 0.9, device="cuda"))
        probs, dprobs = (torch.empty(T, V, device="cuda") for _ in range(2))
        u = torch.rand(T, generator=g)
        drawn = skv.sample_tokens(near.cuda(), u.cuda(), probs_out=dprobs, dev_error_word=err, **settings).cpu()
        skv.sample_tokens(logits.cuda(), None, probs_out=probs, dev_error_word=err, **settings)
        for r in range(T):
            assert int(drawn[r]) == reference(near[r].numpy(), float(np.float32(0.8)), 40, float(np.float32(0.9)), u=float(u[r]))[1]
        tokens = torch.cat([torch.zeros(1, dtype=torch.int32), drawn[:-1]])                  # row r + 1 fed the draft drawn after row r
        accept, sample = torch.rand(T, generator=g), torch.rand(len(live), generator=g)
        new_lens = i32([seq[b] for b in live])
        got, acc = skv.verify_drafts(tokens.cuda(), i32(qo_l.tolist()), probs, dprobs, accept.cuda(), sample.cuda(), seq_lens=new_lens,
                                     seq_lens_out=new_lens, dev_error_word=err)
        p, d = probs.double().cpu(), dprobs.double().cpu()
        for i, b in enumerate(live):
            r0, a = int(qo_l[i]), 0
            while a < drafts and accept[r0 + a].double() * d[r0 + a, tokens[r0 + a + 1]] < p[r0 + a, tokens[r0 + a + 1]]:
                a += 1
            w = (p[r0 + a] - d[r0 + a]).clamp(min=0) if a < drafts else p[r0 + a]
            cum = torch.cumsum(w, 0)
            token = int(torch.nonzero((cum > sample[i].double() * cum[-1]) & (w > 0))[0])
            assert int(acc[i]) == a and got[r0:r0 + a + 1].tolist() == tokens[r0 + 1:r0 + 1 + a].tolist() + [token]
            lens[b] = seq[b] - drafts + a
        assert new_lens.tolist() == [lens[b] for b in live]
    assert skv.read_device_error(err)[0] == skv.OK


def test_a_captured_step_follows_its_lengths():
    """Pages, append and sampling of one new token per request in a graph: replays follow the lengths on the device, and
    equal the same calls made one by one."""
    B, heads, D, page, block, V = 6, 2, 128, 64, 16, 5000
    g = torch.Generator().manual_seed(9)

    def state():
        z = dict(k=torch.zeros(60, heads, page, D, dtype=torch.uint8, device="cuda"), v=torch.zeros(60, heads, page, D, dtype=torch.uint8, device="cuda"),
                 ks=torch.ones(60, heads, page // block, device="cuda"), vs=torch.ones(60, heads, page // block, device="cuda"),
                 table=torch.full((B, 10), -1, dtype=torch.int32, device="cuda"), held=i32([0] * B), free=torch.arange(60, dtype=torch.int32, device="cuda"),
                 count=i32([60]), seq=i32([1] * B), slots=torch.zeros(B, dtype=torch.int64, device="cuda"), tokens=i32([0] * B),
                 kn=torch.zeros(B, heads, D, dtype=torch.bfloat16, device="cuda"), vn=torch.zeros(B, heads, D, dtype=torch.bfloat16, device="cuda"),
                 logits=torch.zeros(B, V, dtype=torch.bfloat16, device="cuda"), u=torch.zeros(B, device="cuda"), p=torch.full((B,), 0.9, device="cuda"),
                 qo=torch.arange(B + 1, dtype=torch.int32, device="cuda"))
        z["problem"] = skv.AttentionProblem(
            q=torch.zeros(B, heads, D, dtype=torch.bfloat16, device="cuda"), k_cache=z["k"], v_cache=z["v"], page_table=z["table"], seq_lens=z["seq"],
            qo_indptr=z["qo"], num_q_heads=heads, num_kv_heads=heads, head_dim_qk=D, head_dim_v=D, page_size=page, scale=1.0,
            seq_lens_host=[1] * B, k_scale=z["ks"], v_scale=z["vs"])
        return z

    def call(z):
        skv.assign_pages(z["table"], z["held"], z["seq"], z["free"], z["count"], page_size=page, qo_indptr=z["qo"], slots=z["slots"])
        skv.kv_append(z["problem"], z["kn"], z["vn"])
        skv.sample_tokens(z["logits"], z["u"], top_p=z["p"], out_tokens=z["tokens"])

    a, b = state(), state()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(a)
    call(b)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(a)
    lens = [1] * B
    for _ in range(8):
        lens = [n + int(torch.randint(1, 70, (1,), generator=g)) for n in lens]
        inputs = dict(seq=torch.tensor(lens, dtype=torch.int32), kn=torch.randn(B, heads, D, generator=g).bfloat16(),
                      vn=torch.randn(B, heads, D, generator=g).bfloat16(), logits=(torch.randn(B, V, generator=g) * 3).bfloat16(),
                      u=torch.rand(B, generator=g))
        for z in (a, b):
            for name, x in inputs.items():
                z[name].copy_(x)
        graph.replay()
        call(b)
        torch.cuda.synchronize()
        for name in ("table", "held", "free", "count", "slots", "k", "v", "ks", "vs", "tokens"):
            assert torch.equal(a[name], b[name]), name
        assert a["held"].tolist() == [-(-n // page) for n in lens] and (a["tokens"] >= 0).all()
