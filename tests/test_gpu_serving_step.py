"""The cache, attention and verification calls run together, as a serving loop runs them.

GQA: prompts' K/V are appended to an E4M3 cache, a drafted block is appended and attended by
splitkv_decode, the drafts are verified, and the next block is appended over the refused
drafts' slots; every attention is checked against float64 over the values that the cache must
hold by then.  Latent: prompt rows are appended and attended in the expanded form, then single
tokens in the absorbed form.

The attention tolerances are those of the parity tests (bf16 outputs: 2e-3 + 1e-2 |ref|); the
quantised values are restated exactly, so they add nothing."""
import math

import numpy as np
import pytest
import torch

import long_context_split_gb300 as skv
from tests.gpu_util import check_output
from tests.test_gpu_cache_rows import K_SCALE, V_SCALE, decode, encode

pytestmark = pytest.mark.gpu


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _attend(q, k, v, pos, scale):
    """float64 attention of rows q [T, Hq, D] at positions pos over k, v [L, Hkv, D]."""
    out = torch.zeros(q.shape[0], q.shape[1], v.shape[2], dtype=torch.float64)
    g = q.shape[1] // k.shape[1]
    for h in range(q.shape[1]):
        s = q[:, h].double() @ k[:, h // g].double().T * scale
        s = s.masked_fill(torch.arange(k.shape[0])[None] > pos[:, None], -math.inf)
        out[:, h] = torch.softmax(s, 1) @ v[:, h // g].double()
    return out.numpy()


def test_speculative_decoding_over_an_e4m3_cache():
    Hq, Hkv, D, P, V, drafts = 8, 2, 128, 64, 1000, 3
    gen = torch.Generator().manual_seed(3)
    prompts = [100, 61, 7]
    B, pages = len(prompts), 4
    table = torch.randperm(B * pages, generator=gen, dtype=torch.int32).view(B, pages).cuda()
    k_cache = torch.full((B * pages, Hkv, P, D), 0x7F, dtype=torch.uint8, device="cuda")     # NaN everywhere
    v_cache = k_cache.clone()
    scale = 1 / math.sqrt(D)
    held = [[torch.zeros(0, Hkv, D), torch.zeros(0, Hkv, D)] for _ in range(B)]             # the caches' values

    def step(seq, new, k, v, q=None):
        """Append rows and attend q; seq holds the lengths with the new tokens."""
        qo = np.concatenate([[0], np.cumsum(new)])
        prob = skv.AttentionProblem(
            q=(torch.zeros(int(qo[-1]), Hq, D) if q is None else q).bfloat16().cuda(), k_cache=k_cache, v_cache=v_cache,
            page_table=table, seq_lens=_i32(seq), qo_indptr=_i32(qo.tolist()), num_q_heads=Hq, num_kv_heads=Hkv, head_dim_qk=D,
            head_dim_v=D, page_size=P, scale=scale, k_scale=K_SCALE, v_scale=V_SCALE)
        skv.kv_append(prob, k.cuda(), v.cuda())
        for b in range(B):
            lo = seq[b] - new[b]
            rows = slice(qo[b], qo[b + 1])
            for i, (x, sc) in enumerate(((k, K_SCALE), (v, V_SCALE))):
                held[b][i] = torch.cat([held[b][i][:lo], decode(encode(x[rows], "e4m3", sc), "e4m3", sc, "f32")])
        if q is None:
            return None
        att = skv.SplitKVAttention(prob, skv.plan_params("uniform", uniform_splits=2))
        out, _ = att.decode()
        torch.cuda.synchronize()
        att.check_device_error()
        got = out.float().cpu().numpy()
        for b in range(B):
            pos = torch.arange(seq[b] - new[b], seq[b])
            ref = _attend(q[qo[b]:qo[b + 1]].bfloat16(), *held[b], pos, scale)
            check_output(got[qo[b]:qo[b + 1]], ref, "bf16", f"request {b}")
        return prob

    def rows(n):
        return torch.randn(n, Hkv, D, generator=gen).bfloat16()

    step(prompts, prompts, rows(sum(prompts)), rows(sum(prompts)))
    lens, accepted_any = list(prompts), 0
    for it in range(3):
        new = [1 + drafts] * B
        T = sum(new)
        seq = [n + t for n, t in zip(lens, new)]
        q = torch.randn(T, Hq, D, generator=gen)
        prob = step(seq, new, rows(T), rows(T), q)
        # verification: the draft distribution a perturbation of the target's
        logits = torch.randn(T, V, generator=gen) * 2
        target, draft = torch.softmax(logits, 1), torch.softmax(logits + 0.3 * torch.randn(T, V, generator=gen), 1)
        tokens = torch.zeros(T, dtype=torch.int32)
        tokens[1:] = torch.multinomial(draft, 1, generator=gen).view(-1)[:-1].int()
        seq_dev = _i32(seq)
        out, acc = skv.verify_drafts(tokens.cuda(), prob.qo_indptr, target.cuda(), draft.cuda(),
                                     torch.rand(T, generator=gen).cuda(), torch.rand(B, generator=gen).cuda(),
                                     seq_lens=seq_dev, seq_lens_out=seq_dev)
        a = acc.cpu().tolist()
        accepted_any += sum(a)
        for b in range(B):
            r0 = b * (1 + drafts)
            kept = tokens[r0 + 1:r0 + 1 + a[b]].tolist()
            assert out[r0:r0 + a[b]].tolist() == kept
            assert 0 <= int(out[r0 + a[b]]) < V and (out[r0 + a[b] + 1:r0 + 1 + drafts] == -1).all()
        lens = seq_dev.cpu().tolist()                # the next block goes over the refused drafts' slots
        assert lens == [s - drafts + x for s, x in zip(seq, a)]
    assert accepted_any > 0
    # what the caches hold, read back
    prob = skv.AttentionProblem(
        q=torch.zeros(B, Hq, D).bfloat16().cuda(), k_cache=k_cache, v_cache=v_cache, page_table=table, seq_lens=_i32(lens),
        qo_indptr=_i32([0, 1, 2, 3]), num_q_heads=Hq, num_kv_heads=Hkv, head_dim_qk=D, head_dim_v=D, page_size=P, scale=scale,
        k_scale=K_SCALE, v_scale=V_SCALE)
    at = np.concatenate([[0], np.cumsum(lens)])
    ko, vo = (torch.zeros(int(at[-1]), Hkv, D, device="cuda") for _ in range(2))
    skv.kv_gather(prob, _i32(at.tolist()), ko, vo)
    torch.cuda.synchronize()
    for b in range(B):
        assert torch.equal(ko[at[b]:at[b + 1]].cpu(), held[b][0][:lens[b]])
        assert torch.equal(vo[at[b]:at[b + 1]].cpu(), held[b][1][:lens[b]])


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_a_latent_prompt_and_its_decode_steps(cache):
    H, P, L0 = 128, 64, [70, 200]
    gen = torch.Generator().manual_seed(4)
    table = torch.randperm(10, generator=gen, dtype=torch.int32).view(2, 5).cuda()
    nan = torch.full((10, P, 576), float("nan"))
    cache_t = (nan.to(torch.float8_e4m3fn).view(torch.uint8) if cache == "e4m3" else nan.bfloat16()).cuda()
    k_scale = K_SCALE if cache == "e4m3" else None
    w = (torch.randn(H, 256, 512, generator=gen) / math.sqrt(512)).bfloat16()
    held = [torch.zeros(0, 576), torch.zeros(0, 576)]
    scale = 1 / math.sqrt(192)

    def step(seq, new, form):
        qo = np.concatenate([[0], np.cumsum(new)])
        T = int(qo[-1])
        att = skv.LatentAttention(k_cache=cache_t, w_kv_b=w.cuda(), page_table=table, seq_lens=_i32(seq), qo_indptr=_i32(qo.tolist()),
                                  scale=scale, k_scale=k_scale)
        assert att.form == form
        latent, rope = torch.randn(T, 512, generator=gen).bfloat16(), torch.randn(T, 64, generator=gen).bfloat16()
        q = torch.randn(T, H, 192, generator=gen).bfloat16()
        skv.kv_append(att.problem, latent.cuda(), rope.cuda())
        out = att(q.cuda())
        torch.cuda.synchronize()
        att.check_device_error()
        rows = torch.cat([latent, rope], 1)
        for b in range(2):
            x = encode(rows[qo[b]:qo[b + 1]], cache, K_SCALE)
            held[b] = torch.cat([held[b], decode(x, cache, K_SCALE, "f32")])
            c = held[b].double()
            pos = torch.arange(seq[b] - new[b], seq[b])
            for h in (0, 77, 127):
                kn, v = c[:, :512] @ w[h, :128].double().T, c[:, :512] @ w[h, 128:].double().T
                k = torch.cat([kn, c[:, 512:]], 1)
                ref = _attend(q[qo[b]:qo[b + 1], h:h + 1].double(), k[:, None], v[:, None], pos, scale)
                got = out[qo[b]:qo[b + 1], h:h + 1].float().cpu().numpy()
                # the tests of each form bound every element; together they are held to their norm
                assert np.linalg.norm(got - ref) <= 6e-3 * np.linalg.norm(ref), (form, b, h)

    step(L0, L0, "expanded")
    step([n + 1 for n in L0], [1, 1], "absorbed")
    step([n + 4 for n in L0], [3, 3], "absorbed")
