"""Verify steps whose layers attend over a paged cache: every stage against the
oracle on the GPU's own inputs (the attention within the tolerance of
test_gpu_attention, the linears within G1), the step's acceptance against the
oracle's on its own target ids, several blocks in a row with rejected drafts
overwritten, and the whole step captured in a graph."""
import numpy as np
import pytest

import gen
from oracle import attention as oa, gemm as og, verify as over
from tests.gpu_util import check_gemm, dev, host
from tests.test_gpu_attention import check_attention

pytestmark = pytest.mark.gpu

LAYERS, HQ, HKV, D, HIDDEN, INTER, VOCAB = 2, 8, 2, 64, 256, 384, 640
WIDTHS = [(HIDDEN, (HQ + 2 * HKV) * D), (HQ * D, HIDDEN), (HIDDEN, 2 * INTER), (INTER, HIDDEN)]


def build(rng, batch, k, page=16, max_ctx=900, prompt=(700, 40, 333)):
    """(step, mixer, host linears): random W4A16 layers, caches holding random prompts."""
    from w4a16_speculative_verify_amd.step import DeviceLinear, PagedMixer, VerifyStep
    pages = -(-max_ctx // page)
    mixer = PagedMixer(LAYERS, batch, k + 1, HQ, HKV, D, batch * pages, page, max_ctx)
    mixer.block_table.copy_(dev(rng.permutation(batch * pages).astype(np.int32).reshape(batch, pages)))
    for c in mixer.k_cache + mixer.v_cache:
        c.copy_(dev(rng.standard_normal(tuple(c.shape)).astype(np.float16)))
    mixer.ctx_lens.copy_(dev(np.asarray(prompt[:batch], np.int32) + k + 1))
    lins, dl = [], []
    for _ in range(LAYERS):
        for kin, n in WIDTHS:
            q = gen.qlinear(rng, kin, n)
            a = gen.chain_alpha(kin)
            lins.append((q, kin, a))
            dl.append(DeviceLinear(dev(q.qweight), dev(q.scales), dev(q.qzeros), kin, n, a))
    w, s = gen.lmhead_weights(rng, VOCAB, HIDDEN), gen.lmhead_scales(rng, VOCAB)
    return VerifyStep(dl, dev(w), dev(s), batch * (k + 1), batch, k, mixer=mixer), mixer, lins


def test_each_stage_matches_the_oracle(lib):
    import torch
    rng = np.random.default_rng(1)
    batch, k = 3, 7
    step, mixer, lins = build(rng, batch, k)
    h = dev(rng.standard_normal((batch * (k + 1), HIDDEN)).astype(np.float16))
    for i, (lin, kin, a) in enumerate(lins):
        y = lib.w4a16_gemm(h[:, :kin], step.linears[i].qweight, step.linears[i].scales,
                           step.linears[i].qzeros, alpha=a, workspace=step.workspace)
        torch.cuda.synchronize()
        check_gemm(host(y), og.w4a16_gemm(host(h[:, :kin]), lin.qweight, lin.scales, lin.qzeros, a),
                   f"linear {i}")
        h = y
        if i % 4 == 0:
            n = i // 4
            kc, vc = host(mixer.k_cache[n]).copy(), host(mixer.v_cache[n]).copy()
            h = mixer(n, y, step.workspace)
            torch.cuda.synchronize()
            cu, ctx, table = host(mixer.cu), host(mixer.ctx_lens), host(mixer.block_table)
            q_ref, k_ref, v_ref = oa.rope_append(host(y), kc, vc, table, cu, ctx, host(mixer.inv_freq), HQ)
            kg, vg, qg = host(mixer.k_cache[n]), host(mixer.v_cache[n]), host(mixer.q)
            assert np.allclose(qg, q_ref, rtol=2**-10, atol=2**-16)
            assert np.allclose(kg, k_ref, rtol=2**-10, atol=2**-16) and np.array_equal(vg, v_ref)
            ref = oa.attention(qg, kg, vg, table, cu, ctx, D ** -0.5)
            check_attention(host(h).reshape(-1, HQ, D), qg, ref, D, D ** -0.5, f"layer {n}")
    torch.cuda.synchronize()


def test_blocks_in_a_row_and_captured(lib):
    """Three blocks, each from where the one before was accepted, eagerly and as replays of one
    captured step (with eager work between): the same tokens, caches and lengths, and the
    acceptance that the oracle gives on the step's target ids."""
    import torch
    rng = np.random.default_rng(2)
    batch, k = 3, 7
    seed = int(rng.integers(1 << 30))
    eager, me, _ = build(np.random.default_rng(seed), batch, k)
    graph, mg, _ = build(np.random.default_rng(seed), batch, k)
    x = torch.empty((batch * (k + 1), HIDDEN), dtype=torch.float16, device="cuda")
    drafts = torch.empty((batch, k), dtype=torch.int32, device="cuda")
    x.copy_(dev(rng.standard_normal(tuple(x.shape)).astype(np.float16)))
    drafts.fill_(-1)
    first = mg.ctx_lens.clone()
    graph(x, drafts)                                          # warm: everything is allocated
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = graph(x, drafts)
        mg.advance(graph.accepted_len)
    mg.ctx_lens.copy_(first)
    for a, b in zip(mg.k_cache + mg.v_cache, me.k_cache + me.v_cache):
        a.copy_(b)
    for block in range(3):
        xs = rng.standard_normal(tuple(x.shape)).astype(np.float16)
        x.copy_(dev(xs))
        # drafts around what the target will say: its ids for these rows, some of them wrong
        drafts.fill_(-1)
        keep = [c.clone() for c in me.k_cache + me.v_cache]
        t, _, _, _ = eager(x, drafts)
        ids = host(t).reshape(batch, k + 1)
        for c, old in zip(me.k_cache + me.v_cache, keep):
            c.copy_(old)
        d = np.stack([gen.drafts_with_prefix(rng, ids[b], k, VOCAB, int(rng.integers(0, k + 1)))
                      for b in range(batch)])
        drafts.copy_(dev(d))
        t, _, acc, toks = eager(x, drafts)
        me.advance(eager.accepted_len)
        g.replay()
        torch.cuda.synchronize()
        a_o, out_o = over.greedy_verify(host(t).reshape(batch, -1), d, VOCAB)
        assert np.array_equal(host(acc), a_o) and np.array_equal(host(toks), out_o)
        assert torch.equal(out[0], t) and torch.equal(out[2], acc) and torch.equal(out[3], toks)
        assert torch.equal(mg.ctx_lens, me.ctx_lens)
        for a, b in zip(mg.k_cache + mg.v_cache, me.k_cache + me.v_cache):
            assert torch.equal(a, b)
    assert np.array_equal(host(graph.out[-1]), host(eager.out[-1]))


def test_a_step_refuses_what_does_not_fit(lib):
    from w4a16_speculative_verify_amd.step import PagedMixer, VerifyStep
    rng = np.random.default_rng(3)
    step, mixer, _ = build(rng, 2, 3, prompt=(10, 20))
    args = (step.linears, step.lm_w, step.lm_s)
    with pytest.raises(ValueError):
        VerifyStep(*args, 8, 2, 3, mixer=mixer, chain=True)
    with pytest.raises(ValueError):
        VerifyStep(*args, 6, 2, 2, mixer=mixer)               # another number of rows
    with pytest.raises(ValueError):
        VerifyStep(step.linears[:6], *args[1:], 8, 2, 3, mixer=mixer)
    with pytest.raises(ValueError):                           # heads wider than the QKV linear
        VerifyStep(*args, 8, 2, 3, mixer=PagedMixer(LAYERS, 2, 4, 16, 2, D, 4, 16, 64))
