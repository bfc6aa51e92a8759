"""The token mixers of a verify step, measured: rotary positions with the append to a paged
key/value cache, attention of a chunk of new tokens over that cache, and the gated delta rule.

``run`` computes them in plain torch where ``own`` is false and through the library's calls
where it is true.  Every case is a dict with the operator in ``"op"``:

  rope   rows of a fused QKV projection: q and k rotated, k and v written to their pages
  attn   softmax attention of the new rows over all cached tokens at or before them
  gdn    S <- alpha S (I - beta k k^T) + beta v k^T,  o = scale S q

Sequences are ragged: ``t`` is the longest sequence's count of new tokens, ``ctx`` the longest
context (new tokens included), and ``spread`` how far the others fall behind.
"""
import math

import numpy as np
import torch

own = False

CHUNK = 64          # most tokens the plain gated delta rule takes at a time


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a verify block (K = 15 drafts) of the 4B-class target at 8 sequences: latency
        dict(name="rope_verify_8x16", op="rope", b=8, t=16, ctx=2048, spread=0.5, hq=32, hkv=8, d=128,
             rot=128, pairs="half", factor=1.0, page=16),
        # an 8,192-token prompt in one pass; half of the head rotated, interleaved, frequencies
        # divided for a long context
        dict(name="rope_prompt_8192", op="rope", b=1, t=8192, ctx=8192, spread=0.0, hq=32, hkv=8, d=128,
             rot=64, pairs="interleaved", factor=4.0, page=64),
        # one sequence, one token, a short odd context: the smallest call of a decode
        dict(name="attn_decode_1_ctx1001", op="attn", b=1, t=1, ctx=1001, spread=0.0, hq=32, hkv=8,
             d=128, page=16),
        # the verify block of one sequence behind an 8,192-token prompt
        dict(name="attn_verify_1x16_ctx8208", op="attn", b=1, t=16, ctx=8208, spread=0.0, hq=32, hkv=8,
             d=128, page=64),
        # the batched verify block with K = 20 (168 rows), ragged contexts
        dict(name="attn_verify_8x21_ctx8213", op="attn", b=8, t=21, ctx=8213, spread=0.6, hq=32, hkv=8,
             d=128, page=16),
        # a full decode batch on long ragged contexts: bound by the cache's bytes
        dict(name="attn_decode_64_ctx16384", op="attn", b=64, t=1, ctx=16384, spread=0.7, hq=32, hkv=8,
             d=128, page=32),
        # chunks of prompts behind long contexts, narrow heads, eight query heads a key head
        dict(name="attn_chunk_2x500_ctx32500", op="attn", b=2, t=500, ctx=32500, spread=0.3, hq=32,
             hkv=4, d=64, page=128),
        # an 8,192-token prompt attending to itself: bound by the matrix cores
        dict(name="attn_prompt_8192", op="attn", b=1, t=8192, ctx=8192, spread=0.0, hq=32, hkv=8, d=128,
             page=64),
        # one decoded token of one sequence through one layer's 16 heads
        dict(name="gdn_decode_1", op="gdn", b=1, t=1, spread=0.0, hk=16, h=16, d=128, kind="f32",
             update=True),
        # the batched verify block: outputs of every position, the state left for the commit
        dict(name="gdn_verify_8x21", op="gdn", b=8, t=21, spread=0.0, hk=16, h=16, d=128, kind="f16",
             update=False),
        # ragged prompts of four sequences, two value heads a key head, narrow heads
        dict(name="gdn_prompt_4x2048", op="gdn", b=4, t=2048, spread=0.6, hk=8, h=16, d=64, kind="f16",
             update=True),
        # an 8,192-token prompt
        dict(name="gdn_prompt_8192", op="gdn", b=1, t=8192, spread=0.0, hk=16, h=16, d=128, kind="f16",
             update=True),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "attn", "attn", "gdn", "gdn"))
    spread = rng.choice((0.0, rng.uniform(0.1, 0.9)))
    if op == "gdn":
        t = _log_uniform(rng, 1, 6000)
        return dict(op=op, b=_log_uniform(rng, 1, max(1, min(64, 8192 // t))), t=t, spread=spread,
                    **dict(rng.choice((dict(hk=16, h=16), dict(hk=8, h=16), dict(hk=4, h=12)))),
                    d=rng.choice((64, 128)), kind=rng.choice(("f16", "f32")) if t <= 64 else "f16",
                    update=rng.random() < 0.7)
    d = rng.choice((64, 128, 256))
    hkv = rng.choice((1, 2, 4, 8))
    hq = hkv * rng.choice((1, 2, 4, 5, 8))
    page = rng.choice((16, 32, 64, 128, 256))
    if op == "rope":
        t = _log_uniform(rng, 1, 8000)
        b = _log_uniform(rng, 1, max(1, min(64, 8192 // t)))
        rot = rng.choice((d, d // 2, d // 4))
        return dict(op=op, b=b, t=t, ctx=t + _log_uniform(rng, 1, max(2, 100000 // b)), spread=spread, hq=hq,
                    hkv=hkv, d=d, rot=rot, pairs=rng.choice(("half", "interleaved")),
                    factor=rng.choice((1.0, 8.0)), page=page)
    t = rng.choice((1, _log_uniform(rng, 2, 32), _log_uniform(rng, 33, 2048)))
    ctx = t + _log_uniform(rng, 1, 32768)
    most = max(1, min(64, 200000 // ctx, int(1.2e9 // (hq * t * ctx))))
    return dict(op=op, b=_log_uniform(rng, 1, most), t=t, ctx=ctx, spread=spread, hq=hq, hkv=hkv, d=d,
                page=page)


def _lengths(case):
    """(new tokens, context) of each sequence, from the case alone: the first is the longest."""
    f = [1.0 - case["spread"] * ((0.6180339887 * i) % 1.0) for i in range(case["b"])]
    t = [max(1, int(case["t"] * (x if case["t"] > 32 else 1.0))) for x in f]
    ctx = [max(n, int(case.get("ctx", case["t"]) * x)) for n, x in zip(t, f)]
    return t, ctx


def work(case):
    t, ctx = _lengths(case)
    n, d = sum(t), case["d"]
    if case["op"] == "gdn":
        size = 2 if case["kind"] == "f16" else 4
        h, hk = case["h"], case["hk"]
        state = case["b"] * h * d * d * 4
        return {"bytes": n * (2 * hk + 2 * h) * d * size + n * h * 8 + state * (2 if case["update"] else 1),
                "flops": 8.0 * n * h * d * d}
    hq, hkv = case["hq"], case["hkv"]
    if case["op"] == "rope":
        return {"bytes": 2 * n * (hq + 2 * hkv) * d * 2, "flops": 3.0 * n * (hq + hkv) * case["rot"]}
    seen = sum(m * c - m * (m - 1) // 2 for m, c in zip(t, ctx))
    return {"bytes": 2 * n * hq * d * 2 + sum(ctx) * hkv * d * 2 * 2, "flops": 4.0 * d * hq * seen}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def normal(*shape, dtype=torch.float16):
        x = torch.empty(shape, dtype=dtype, device=dev)
        return x.normal_(generator=g)

    t, ctx = _lengths(case)
    b, d, n = case["b"], case["d"], sum(t)
    cu = torch.tensor([0] + list(np.cumsum(t)), dtype=torch.int32, device=dev)
    s = dict(case=case, n=n, max_t=max(t), cu=cu)
    # the row that token i of sequence b has, and whether it has one: the plan of a padded batch
    i = torch.arange(max(t), device=dev)
    live = i[None, :] < torch.tensor(t, device=dev)[:, None]
    s["live"], s["rows"] = live, torch.where(live, cu[:-1, None].long() + i[None, :], 0)
    if case["op"] == "gdn":
        dt = torch.float16 if case["kind"] == "f16" else torch.float32
        hk, h = case["hk"], case["h"]
        q, k = (normal(n, hk, d, dtype=torch.float32) for _ in range(2))
        s["q"], s["k"] = ((x / x.norm(dim=-1, keepdim=True)).to(dt) for x in (q, k))
        s["v"] = normal(n, h, d, dtype=dt)
        s["alpha"] = 1.0 - 0.1 * torch.rand((n, h), generator=g, device=dev)
        s["beta"] = torch.rand((n, h), generator=g, device=dev)
        s["state"] = normal(b, h, d, d, dtype=torch.float32)
        s["new_state"] = torch.empty_like(s["state"]) if case["update"] else None
        return s
    hq, hkv, page = case["hq"], case["hkv"], case["page"]
    pages = [-(-c // page) for c in ctx]
    total, width = sum(pages), max(pages)
    # pages were handed out in no order; entries behind a sequence's last page hold none
    order = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    first = torch.tensor([0] + list(np.cumsum(pages))[:-1], device=dev)
    j = torch.arange(width, device=dev)
    has = j[None, :] < torch.tensor(pages, device=dev)[:, None]
    s["table"] = torch.where(has, order[torch.where(has, first[:, None] + j[None, :], 0)], -1).contiguous()
    s["ctx"], s["max_ctx"] = torch.tensor(ctx, dtype=torch.int32, device=dev), max(ctx)
    s["k_cache"], s["v_cache"] = (normal(total, hkv, page, d) for _ in range(2))
    s["scale"] = d ** -0.5
    if case["op"] == "rope":
        s["qkv"] = normal(n, (hq + 2 * hkv) * d)
        e = torch.arange(0, case["rot"], 2, dtype=torch.float64, device=dev) / case["rot"]
        s["inv_freq"] = (10000.0 ** -e / case["factor"]).to(torch.float32)
        s["mscale"] = 1.0 + 0.1 * math.log(case["factor"])
    else:
        s["q"] = normal(n, hq, d)
    return s


# ------------------------------------------------------------------ plain forms
def _positions(s):
    """Position of every row, and its sequence."""
    t = s["cu"][1:] - s["cu"][:-1]
    seq = torch.repeat_interleave(torch.arange(t.numel(), device=t.device), t.long(), output_size=s["n"])
    i = torch.arange(s["n"], device=t.device)
    return (s["ctx"].long() - s["cu"][1:].long())[seq] + i, seq


def _rope_plain(s):
    c = s["case"]
    hq, hkv, d, rot, page = c["hq"], c["hkv"], c["d"], c["rot"], c["page"]
    p, seq = _positions(s)
    x = s["qkv"].view(s["n"], hq + 2 * hkv, d)
    angle = p[:, None].double() * s["inv_freq"].double()
    cos = (angle.cos() * s["mscale"]).float()[:, None, :]
    sin = (angle.sin() * s["mscale"]).float()[:, None, :]
    y = x[:, :hq + hkv].float()
    a, b = (y[..., :rot // 2], y[..., rot // 2:rot]) if c["pairs"] == "half" else (y[..., 0:rot:2], y[..., 1:rot:2])
    pair = (a * cos - b * sin, b * cos + a * sin)
    turned = torch.cat(pair, -1) if c["pairs"] == "half" else torch.stack(pair, -1).flatten(-2)
    y = torch.cat((turned, y[..., rot:]), -1).half()
    where, slot = s["table"][seq, p // page].long(), p % page
    s["k_cache"][where, :, slot] = y[:, hq:]
    s["v_cache"][where, :, slot] = x[:, hq + hkv:]
    return {"q": y[:, :hq].contiguous(), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _gathered(s, cache):
    """[B, Hkv, tokens, D] of a cache, by the page table."""
    b, width = s["table"].shape
    x = cache[s["table"].clamp(min=0).long()]                       # [B, pages, Hkv, page, D]
    return x.transpose(1, 2).reshape(b, cache.shape[1], width * cache.shape[2], cache.shape[3])


def _attn_plain(s):
    c = s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    g, b, t = hq // hkv, c["b"], s["max_t"]
    k, v = _gathered(s, s["k_cache"]).float(), _gathered(s, s["v_cache"]).float()
    q = s["q"].float()[s["rows"]].view(b, t, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, t * g, d)
    sc = (q @ k.transpose(2, 3).contiguous()).mul_(s["scale"]).view(b, hkv, t, g, -1)
    new = s["cu"][1:] - s["cu"][:-1]
    p = (s["ctx"] - new)[:, None] + torch.arange(t, device=q.device)[None, :]
    hidden = torch.arange(k.shape[2], device=q.device)[None, None, :] > p[:, :, None]
    sc.masked_fill_(hidden[:, None, :, None, :], -math.inf)
    sc.sub_(sc.amax(-1, keepdim=True)).exp_()
    o = (sc.view(b, hkv, t * g, -1) @ v).view(b, hkv, t, g, d) / sc.sum(-1, keepdim=True)
    return o.permute(0, 2, 1, 3, 4).reshape(b, t, hq, d)[s["live"]].half()


def _gdn_plain(s):
    """Chunks of up to CHUNK tokens: inside one, the tokens' updates solve a unit lower triangular
    system; from one to the next, the state is carried."""
    c = s["case"]
    b, h, d, t = c["b"], c["h"], c["d"], s["max_t"]
    size = min(CHUNK, t)
    m = -(-t // size)
    rows = torch.nn.functional.pad(s["rows"], (0, m * size - t))
    live = torch.nn.functional.pad(s["live"], (0, m * size - t))

    def chunked(x, fill):                              # [N, H, ...] -> [B, H, chunks, size, ...]
        x = x.float().repeat_interleave(h // x.shape[1], 1)[rows]
        x = torch.where(live.view(b, -1, *[1] * (x.dim() - 2)), x, fill)
        return x.transpose(1, 2).reshape(b, h, m, size, *x.shape[3:])

    q, k, v = (chunked(s[x], 0.0) for x in "qkv")
    alpha, beta = chunked(s["alpha"], 1.0), chunked(s["beta"], 0.0)
    logs = alpha.double().log().cumsum(-1)
    low = torch.ones(size, size, dtype=torch.bool, device=q.device).tril()
    decay = torch.where(low, (logs[..., :, None] - logs[..., None, :]), -math.inf).exp().float()
    since = logs.exp().float()[..., None]              # decay since the chunk's start
    kt = k.transpose(-1, -2).contiguous()
    mix = (beta[..., None] * decay * (k @ kt)).tril(-1)
    solve = torch.eye(size, device=q.device).expand_as(mix).clone()
    for i in range(1, size):                          # rows of the inverse, each from those above it
        solve[..., i, :i] = -(mix[..., i:i + 1, :i] @ solve[..., :i, :i])[..., 0, :]
    w = solve @ (k * since * beta[..., None])
    u0 = solve @ (v * beta[..., None])
    att = decay * (q @ kt)
    left = decay[..., -1, :, None]                     # decay from each token to the chunk's end
    state, out = s["state"], torch.empty_like(v)
    for i in range(m):
        st = state.transpose(-1, -2).contiguous()
        u = u0[:, :, i] - w[:, :, i] @ st
        out[:, :, i] = since[:, :, i] * (q[:, :, i] @ st) + att[:, :, i] @ u
        state = since[:, :, i, -1:] * state + (u * left[:, :, i]).transpose(-1, -2).contiguous() @ k[:, :, i]
    o = out.reshape(b, h, m * size, d).transpose(1, 2)[live] * d ** -0.5
    o = o.to(s["v"].dtype)
    return {"o": o, "state": state} if c["update"] else {"o": o}


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if not own:
        return {"rope": _rope_plain, "attn": _attn_plain, "gdn": _gdn_plain}[op](state)
    import w4a16_speculative_verify_amd as w4v
    s, c = state, state["case"]
    if op == "rope":
        q = w4v.rope_kv_append(s["qkv"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["ctx"],
                               s["inv_freq"], c["hq"], interleaved=c["pairs"] == "interleaved",
                               mscale=s["mscale"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "attn":
        if "workspace" not in s:         # kept from call to call, as a serving loop keeps it
            s["workspace"] = w4v.new_workspace(w4v.paged_attention_workspace_size(
                c["b"], s["max_t"], s["max_ctx"], c["hq"], c["hkv"], c["d"]))
        return w4v.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["ctx"],
                                   s["max_t"], max_ctx=s["max_ctx"], workspace=s["workspace"])
    if "workspace" not in s:
        s["workspace"] = w4v.new_workspace(w4v.gdn_forward_workspace_size(
            s["n"], c["b"], s["max_t"], c["hk"], c["h"], c["d"], s["q"].dtype))
    o = w4v.gdn_forward(s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["cu"], s["state"], s["max_t"],
                        state_out=s["new_state"], workspace=s["workspace"])
    return {"o": o, "state": s["new_state"]} if c["update"] else {"o": o}


# ------------------------------------------------------------------ the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    t, ctx = _lengths(case)
    start = [0] + list(np.cumsum(t))
    d = case["d"]
    if case["op"] == "gdn":
        # token by token, as the rule is written
        h, b = case["h"], case["b"]
        q, k, v = (s[x].double().repeat_interleave(h // s[x].shape[1], 1) for x in "qkv")
        alpha, beta = s["alpha"].double(), s["beta"].double()
        state, o = s["state"].double(), torch.zeros_like(v)
        order = sorted(range(b), key=lambda i: -t[i])
        for j in range(max(t)):
            on = torch.tensor([i for i in order if t[i] > j], device="cuda")
            at = torch.tensor([start[i] + j for i in order if t[i] > j], device="cuda")
            m = state if len(on) == b and order == list(range(b)) else state[on]
            e = v[at] - alpha[at][..., None] * (m * k[at][:, :, None, :]).sum(-1)
            m = alpha[at][..., None, None] * m + (beta[at][..., None] * e)[..., None] * k[at][:, :, None, :]
            o[at] = (m * q[at][:, :, None, :]).sum(-1) * d ** -0.5
            state[on] = m
        return {"o": o, "state": state} if case["update"] else {"o": o}
    hq, hkv, page = case["hq"], case["hkv"], case["page"]
    table = s["table"].cpu().long()
    if case["op"] == "rope":
        rot = case["rot"]
        x = s["qkv"].double().view(s["n"], hq + 2 * hkv, d)
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        out = x.clone()
        for b in range(case["b"]):
            p = torch.arange(ctx[b] - t[b], ctx[b], device="cuda")
            turn = torch.polar(torch.full((t[b], rot // 2), s["mscale"], dtype=torch.float64, device="cuda"),
                               p.double()[:, None] * s["inv_freq"].double()[None, :])
            y = out[start[b]:start[b + 1], :hq + hkv]
            re, im = ((slice(0, rot // 2), slice(rot // 2, rot)) if case["pairs"] == "half"
                      else (slice(0, rot, 2), slice(1, rot, 2)))
            z = torch.complex(y[..., re], y[..., im]) * turn[:, None, :]
            y[..., re], y[..., im] = z.real, z.imag
            where, slot = table[b].cuda()[p // page], p % page
            kc[where, :, slot] = out[start[b]:start[b + 1], hq:hq + hkv]
            vc[where, :, slot] = x[start[b]:start[b + 1], hq + hkv:]
        return {"q": out[:, :hq].contiguous(), "k_cache": kc, "v_cache": vc}
    out = torch.empty(s["n"], hq, d, dtype=torch.float64, device="cuda")
    g = hq // hkv
    for b in range(case["b"]):
        ids = table[b, :-(-ctx[b] // page)].cuda()
        at = torch.arange(ctx[b], device="cuda")
        for n in range(hkv):
            k = s["k_cache"][ids, n].reshape(-1, d)[:ctx[b]].double()
            v = s["v_cache"][ids, n].reshape(-1, d)[:ctx[b]].double()
            for lo in range(0, t[b], 2048):
                hi = min(t[b], lo + 2048)
                p = torch.arange(ctx[b] - t[b] + lo, ctx[b] - t[b] + hi, device="cuda")
                mask = torch.where(at[None, :] > p[:, None], -math.inf, 0.0)
                for j in range(n * g, n * g + g):
                    q = s["q"][start[b] + lo:start[b] + hi, j].double()
                    w = torch.softmax(torch.addmm(mask.double(), q, k.t(), alpha=s["scale"]), -1)
                    out[start[b] + lo:start[b] + hi, j] = w @ v
    return out
