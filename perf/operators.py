"""The attention-side operators of a transformer block served on the FP4 linear layer, as cases.

Between the QKV projection's output and the next preparation a served model rotates q and k, keeps k and v
in a paged cache of FP4 codes, attends over that cache, and adds each block's output to the residual stream:

  append   rotation (and optional per-head RMSNorm) of q and k, k and v quantised into the paged cache; the rows
           just written are read back as the values they stand for
  read     whole prefixes read back out of the cache
  attn     attention over the cache: single tokens, several tokens per sequence, whole prompts
  norm     norms before and after a block with its gate and the scaled residual stream

`run` computes a case in plain torch operations, or through the library where `own` is true.
"""
import math

import torch

own = False

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one new token for each of 32 running conversations, Llama-3.1-8B's heads, small pages
        dict(name="append_decode", op="append", fmt="nvfp4", seqs=32, new_lo=1, new_hi=1, ctx_lo=100, ctx_hi=4000,
             q_heads=32, kv_heads=8, dim=128, page=16, rot=128, inter=False, qk_norm=False),
        # four prompts of uneven length entering the cache, with per-head norms, heads of a mixture-of-experts model
        dict(name="append_prompts", op="append", fmt="mxfp4", seqs=4, new_lo=1100, new_hi=2900, ctx_lo=0, ctx_hi=500,
             q_heads=32, kv_heads=4, dim=128, page=64, rot=128, inter=False, qk_norm=True),
        # cached prefixes of eight conversations taken out of the cache
        dict(name="read_prefixes", op="read", fmt="nvfp4", seqs=8, new_lo=2000, new_hi=6000, ctx_lo=0, ctx_hi=0,
             q_heads=32, kv_heads=8, dim=128, page=64, rot=128, inter=False, qk_norm=False),
        # one conversation, one token: latency
        dict(name="decode_one", op="attn", fmt="nvfp4", seqs=1, new_lo=1, new_hi=1, ctx_lo=776, ctx_hi=776,
             q_heads=32, kv_heads=8, dim=128, page=16, causal=True, window=0),
        # a full decode batch with uneven contexts
        dict(name="decode_batch", op="attn", fmt="nvfp4", seqs=64, new_lo=1, new_hi=1, ctx_lo=33, ctx_hi=8191,
             q_heads=32, kv_heads=8, dim=128, page=16, causal=True, window=0),
        # two long documents, one token each
        dict(name="decode_long", op="attn", fmt="mxfp4", seqs=2, new_lo=1, new_hi=1, ctx_lo=120000, ctx_hi=131071,
             q_heads=32, kv_heads=8, dim=128, page=64, causal=True, window=0),
        # five drafted tokens a sequence checked at once, Qwen2.5-7B's heads (seven queries share a key head)
        dict(name="verify_drafts", op="attn", fmt="nvfp4", seqs=16, new_lo=3, new_hi=5, ctx_lo=1500, ctx_hi=6000,
             q_heads=28, kv_heads=4, dim=128, page=32, causal=True, window=0),
        # one whole prompt
        dict(name="prompt", op="attn", fmt="nvfp4", seqs=1, new_lo=8192, new_hi=8192, ctx_lo=0, ctx_hi=0,
             q_heads=32, kv_heads=8, dim=128, page=64, causal=True, window=0),
        # pieces of long prompts against what is cached, a sliding window, small heads of their own
        dict(name="chunks_window", op="attn", fmt="mxfp4", seqs=4, new_lo=301, new_hi=1024, ctx_lo=9000, ctx_hi=15000,
             q_heads=16, kv_heads=16, dim=64, page=32, causal=True, window=4096),
        # every video token over a cached text prompt: no causal order, the DiT's 40 heads
        dict(name="cross_text", op="attn", fmt="nvfp4", seqs=2, new_lo=4680, new_hi=4680, ctx_lo=512, ctx_hi=512,
             q_heads=40, kv_heads=40, dim=128, page=64, causal=False, window=0),
        # one decode step's rows between two blocks
        dict(name="norm_decode", op="norm", tokens=16, k=4096, post=True, gates=0, rows_per_gate=0, alpha=1.0, pre=True),
        # the video DiT's rows, gated by sample
        dict(name="norm_video", op="norm", tokens=32760, k=5120, post=True, gates=2, rows_per_gate=16380, alpha=1.0, pre=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "read", "attn", "attn", "attn", "attn", "norm", "norm"])
    if op == "norm":
        k = 8 * _log(rng, 64, 1024)
        tokens = min(_log(rng, 1, 32760), (32760 * 5120) // k)
        gates = rng.choice([0, 0, 1, 3])
        rows = 0 if gates < 2 else -(-tokens // gates)
        return dict(op="norm", tokens=tokens, k=k, post=rng.random() < 0.6, gates=gates if rows != 1 else 0,
                    rows_per_gate=rows if rows != 1 else 0, alpha=rng.choice([1.0, 1.0, 0.5, 0.87]), pre=rng.random() < 0.7)
    fmt = rng.choice(["nvfp4", "mxfp4"])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 5, 7, 8])
    dim = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    heads = dict(fmt=fmt, q_heads=kv_heads * group, kv_heads=kv_heads, dim=dim, page=page)
    if op in ("append", "read"):
        seqs = _log(rng, 1, 64)
        most = max(1, 8000 // seqs)
        hi = _log(rng, 1, most)
        lo = max(1, int(hi * rng.uniform(0.3, 1.0)))
        return dict(op=op, seqs=seqs, new_lo=lo, new_hi=hi, ctx_lo=0, ctx_hi=rng.randint(0, 3000),
                    rot=rng.choice([dim, dim, dim // 2]), inter=rng.random() < 0.3, qk_norm=rng.random() < 0.4, **heads)
    kind = rng.choice(["decode", "decode", "several", "prompt"])
    if kind == "decode":
        seqs = _log(rng, 1, 64)
        hi = _log(rng, 1, min(131071, 500000 // seqs))
        return dict(op="attn", seqs=seqs, new_lo=1, new_hi=1, ctx_lo=int(hi * rng.uniform(0.0, 1.0)), ctx_hi=hi, causal=True,
                    window=rng.choice([0, 0, 0, 1000]), **heads)
    if kind == "several":
        seqs = _log(rng, 1, 24)
        new = rng.randint(2, 40)
        hi = _log(rng, 10, min(20000, 150000 // seqs))
        return dict(op="attn", seqs=seqs, new_lo=max(1, new // 2), new_hi=new, ctx_lo=hi // 3, ctx_hi=hi, causal=True,
                    window=rng.choice([0, 0, 0, 513]), **heads)
    seqs = rng.choice([1, 1, 2, 4])
    new = _log(rng, 60, 4500 // seqs)
    hi = _log(rng, 1, 9000 // seqs)
    causal = rng.random() < 0.8
    while 4.0 * seqs * new * (hi + new / 2) * kv_heads * group * dim > 5e11:
        new = new * 2 // 3
    return dict(op="attn", seqs=seqs, new_lo=max(1, int(new * rng.uniform(0.4, 1.0))), new_hi=new, ctx_lo=hi // 2, ctx_hi=hi,
                causal=causal, window=rng.choice([0, 0, 700]) if causal else 0, **heads)


def _block(fmt):
    return 16 if fmt == "nvfp4" else 32


def _group_bytes(case):
    d = case["dim"]
    return 16 * d + 32 * (d // _block(case["fmt"]))


def _lengths(case):
    """New tokens and cached tokens of each sequence, uneven and the same for every seed: a scheduler's host values."""
    n, span_new, span_ctx = case["seqs"], case["new_hi"] - case["new_lo"] + 1, case["ctx_hi"] - case["ctx_lo"] + 1
    g = torch.Generator().manual_seed(1000 * n + 7 * span_new + span_ctx)
    new = case["new_lo"] + torch.randint(0, span_new, (n,), generator=g)
    ctx = case["ctx_lo"] + torch.randint(0, span_ctx, (n,), generator=g)
    return new.tolist(), ctx.tolist()


# --------------------------------------------------------------------------------------- the cache's bytes
# A page of one key head is page/16 groups of 16 tokens. A group is 16 x dim/2 bytes of K codes (row by row, the
# lower element in the low nibble), as many of V codes in the order below, 16 x dim/B K scales row by row, and the V
# scales. V codes: a token r = 8h + 2t + j and a run g of dim/8 elements have dim/16 bytes at
# (64h + 2(4g + t) + j) * 8 for dim 128 and ((4g + t) * 4 + 2h + j) * 4 for dim 64; the V scale of block b is byte
# (4b + t) * 4 + 2h + j.
def _v_places(dim, device):
    r = torch.arange(16, device=device)
    h, t, j = r // 8, (r // 2) % 4, r % 2
    g = torch.arange(8, device=device)
    cell = 4 * g[None, :] + t[:, None]
    if dim == 128:
        return (64 * h[:, None] + 2 * cell + j[:, None]) * 8
    return (4 * cell + 2 * h[:, None] + j[:, None]) * 4


def _v_scale_places(blocks, device):
    r = torch.arange(16, device=device)
    b = torch.arange(blocks, device=device)
    return (4 * b[None, :] + ((r // 2) % 4)[:, None]) * 4 + (2 * (r // 8) + r % 2)[:, None]


def _row_places(dim, fmt, device):
    """Offsets within a group of each row's K codes, V codes, K scales and V scales: [16, n] each."""
    half, blocks = dim // 2, dim // _block(fmt)
    r = torch.arange(16, device=device)[:, None]
    kc = r * half + torch.arange(half, device=device)[None, :]
    unit = dim // 16
    vc = 16 * half + (_v_places(dim, device)[:, :, None] + torch.arange(unit, device=device)).reshape(16, half)
    ks = 32 * half + r * blocks + torch.arange(blocks, device=device)[None, :]
    vs = 32 * half + 16 * blocks + _v_scale_places(blocks, device)
    return kc, vc, ks, vs


def _encode(x):
    """E2M1 codes of float32 values: nearest, ties to the even code, saturating."""
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    a = x.abs().contiguous()
    up = torch.bucketize(a, edges, right=True)     # a tie goes up here
    down = torch.bucketize(a, edges, right=False)  # and down here
    code = torch.where(up % 2 == 0, up, down)
    return (code + 8 * torch.signbit(x)).to(torch.uint8)


def _quantise(x, fmt, scale):
    """float32 rows [..., heads, dim] -> (codes two a byte, block scale bytes); scale [heads, 1] float32."""
    b = _block(fmt)
    blocks = x.reshape(*x.shape[:-1], x.shape[-1] // b, b)
    amax = blocks.abs().amax(-1)
    if fmt == "nvfp4":
        gain = 1.0 / (6.0 * scale)
        sb = (amax * gain).clamp(max=448.0).to(torch.float8_e4m3fn)
        d = sb.float() * scale
        inv = torch.where(d == 0, torch.zeros_like(d), 1.0 / d)
        byte = sb.view(torch.uint8)
    else:
        e = torch.frexp(amax)[1] - 3  # floor(log2 amax) - 2
        e = torch.where(amax == 0, torch.full_like(e, -23), e.clamp(-23, 13))
        inv = torch.ldexp(torch.ones_like(amax), -e)
        byte = (e + 127).to(torch.uint8)
    codes = _encode(blocks * inv.unsqueeze(-1)).reshape(x.shape)
    return codes[..., 0::2] | (codes[..., 1::2] << 4), byte


def _values(codes, scales, fmt, scale):
    """The float32 values of codes [..., heads, dim/2] with block scales [..., heads, blocks]."""
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=codes.device)
    pair = torch.stack((table.repeat(16), table.repeat_interleave(16)), -1)
    v = pair[codes.int()].reshape(*codes.shape[:-1], scales.shape[-1], -1)
    s = scales.view(torch.float8_e4m3fn).float() if fmt == "nvfp4" else torch.ldexp(torch.ones_like(scales, dtype=torch.float32), scales.int() - 127)
    v = v * s.unsqueeze(-1)
    v = v.reshape(*codes.shape[:-1], -1)
    return v * scale if fmt == "nvfp4" else v


def _heads_view(case, pages):
    return pages.view(-1, case["kv_heads"], case["page"] // 16, _group_bytes(case))


def _fill(case, s, gen):
    """Every page of the cache with quantised random keys and values (a few key channels much larger, as in served models)."""
    dev, n, h, p, d = "cuda", s["num_pages"], case["kv_heads"], case["page"], case["dim"]
    view = _heads_view(case, s["pages"])
    kc, vc, ks, vs = _row_places(d, case["fmt"], dev)
    big = torch.ones(h, d, device=dev)
    big[:, torch.randperm(d, generator=gen, device=dev)[: d // 32]] = 4.0
    step = max(1, (1 << 25) // (h * p * d))
    for a in range(0, n, step):
        m = min(step, n - a)
        for which, cp, sp in (("k", kc, ks), ("v", vc, vs)):
            x = torch.randn(m, p, h, d, generator=gen, device=dev)
            x = x * big if which == "k" else x * 0.7
            codes, byte = _quantise(x, case["fmt"], s["scales"][which])
            view[a:a + m][..., cp.reshape(-1)] = codes.view(m, p // 16, 16, h, -1).permute(0, 3, 1, 2, 4).reshape(m, h, p // 16, -1)
            view[a:a + m][..., sp.reshape(-1)] = byte.view(m, p // 16, 16, h, -1).permute(0, 3, 1, 2, 4).reshape(m, h, p // 16, -1)


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    rand = lambda *n: torch.randn(*n, generator=gen, device=dev)  # noqa: E731
    if case["op"] == "norm":
        t, k = case["tokens"], case["k"]
        s = dict(case=case, y=(0.8 * rand(t, k)).bfloat16(), residual=(2.0 * rand(t, k)).bfloat16())
        s["post"] = (1 + 0.2 * rand(k)).bfloat16() if case["post"] else None
        s["pre"] = (1 + 0.2 * rand(k)).bfloat16() if case["pre"] else None
        s["gate"] = (0.5 * rand(case["gates"], k)).bfloat16() if case["gates"] else None
        return s
    new, ctx = _lengths(case)
    h, d, hq, page = case["kv_heads"], case["dim"], case["q_heads"], case["page"]
    # kv lengths: cached tokens and, where the order is causal, the call's own tokens after them
    length = [c + n for c, n in zip(ctx, new)] if case.get("causal", True) else [max(1, c) for c in ctx]
    need = [-(-x // page) for x in length]
    spare = 3
    num_pages = sum(need) + spare
    order = torch.randperm(num_pages, generator=gen, device=dev).int()
    most = max(need)
    table = torch.full((case["seqs"], most), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s = dict(case=case, new=new, length=length, num_pages=num_pages, tokens=cu[-1], max_q=max(new), max_kv=max(length),
             cu_q=torch.tensor(cu, dtype=torch.int32, device=dev), kv_len=torch.tensor(length, dtype=torch.int32, device=dev),
             table=table, pages=torch.zeros(num_pages * h * (page // 16) * _group_bytes(case), dtype=torch.uint8, device=dev))
    # second-level scales by head, from calibration: the largest value over 6 * 448
    s["scales"] = {"k": (0.8 + 0.4 * torch.rand(h, 1, generator=gen, device=dev)) * (20.0 / 2688), "v": (0.8 + 0.4 * torch.rand(h, 1, generator=gen, device=dev)) * (4.0 / 2688)}
    _fill(case, s, gen)
    if case["op"] == "attn":
        s["q"] = rand(s["tokens"], hq, d).bfloat16()
        return s
    rows = rand(s["tokens"], (hq + 2 * h) * d)
    s["qkv"] = rows.bfloat16()
    s["q_gamma"] = (1 + 0.2 * rand(d)).bfloat16() if case["qk_norm"] else None
    s["k_gamma"] = (1 + 0.2 * rand(d)).bfloat16() if case["qk_norm"] else None
    half = case["rot"] // 2
    s["inv_freq"] = (500000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)).float()
    return s


# ------------------------------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    if own:
        return _library(s)
    if case["op"] == "norm":
        return _plain_norm(s)
    if case["op"] == "read":
        return _plain_read(s)
    if case["op"] == "append":
        q = _plain_append(s)
        return (q, *_plain_read(s))
    return _plain_attention(s)


def _library(s):
    import fp4_activation_sparse_b200 as S
    case = s["case"]
    if case["op"] == "norm":
        r, h = S.sharq_norm_residual(s["y"], s["residual"], post_gamma=s["post"], gate=s["gate"], rows_per_gate=case["rows_per_gate"],
                                     alpha=case["alpha"], pre_gamma=s["pre"], eps=1e-6)
        return (r, h) if h is not None else (r,)
    if "plan" not in s:  # a served model keeps its cache, its batch tables and its workspace
        nv = case["fmt"] == "nvfp4"
        cache = S.KVCache(s["pages"], s["num_pages"], case["page"], case["kv_heads"], case["dim"], case["fmt"],
                          s["scales"]["k"] if nv else None, s["scales"]["v"] if nv else None)
        batch = S.KVBatch(s["cu_q"], s["kv_len"], s["table"], s["max_q"], s["tokens"])
        ws = S.alloc_attention_workspace(cache, batch, case["q_heads"]) if case["op"] == "attn" else None
        s["plan"] = (cache, batch, ws)
    cache, batch, ws = s["plan"]
    if case["op"] == "attn":
        return S.sharq_attention(s["q"], cache, batch, causal=case["causal"], window=case["window"], return_lse=True, workspace=ws)
    if case["op"] == "read":
        return S.sharq_kv_read(cache, batch)
    q = S.sharq_kv_append(s["qkv"], cache, batch, case["q_heads"], inv_freq=s["inv_freq"], interleaved=case["inter"],
                          q_gamma=s["q_gamma"], k_gamma=s["k_gamma"], eps=1e-6)
    return (q, *S.sharq_kv_read(cache, batch))


def _rms(x, gamma, eps):
    """RMSNorm of float32 rows, the sum of squares in 64 bits."""
    mean = (x.double().square().sum(-1, keepdim=True) / x.shape[-1]).float()
    return x * (1.0 / torch.sqrt(mean + eps)) * gamma.float()


def _plain_norm(s):
    case = s["case"]
    z = s["y"].float()
    if s["post"] is not None:
        z = _rms(z, s["post"], 1e-6)
    if s["gate"] is not None:
        t = torch.arange(case["tokens"], device=z.device)
        z = z * s["gate"].float()[t // case["rows_per_gate"] if case["rows_per_gate"] else torch.zeros_like(t)]
    r = (case["alpha"] * s["residual"].float() + z).bfloat16()
    return (r, _rms(r.float(), s["pre"], 1e-6).bfloat16()) if s["pre"] is not None else (r,)


def _token_places(s):
    """Sequence, position and (page, group, row) of every new token."""
    t = torch.arange(s["tokens"], device="cuda")
    b = torch.searchsorted(s["cu_q"].long(), t, right=True) - 1
    pos = s["kv_len"][b].long() - s["cu_q"][b + 1].long() + t
    page = s["table"][b, pos // s["case"]["page"]].long()
    return pos, page, pos % s["case"]["page"] // 16, pos % 16


def _plain_append(s):
    case = s["case"]
    hq, h, d, rot = case["q_heads"], case["kv_heads"], case["dim"], case["rot"]
    pos, page, group, row = _token_places(s)
    x = s["qkv"].float().view(s["tokens"], hq + 2 * h, d)
    q, k, v = x[:, :hq], x[:, hq:hq + h], x[:, hq + h:]
    if s["q_gamma"] is not None:
        q, k = _rms(q, s["q_gamma"], 1e-6), _rms(k, s["k_gamma"], 1e-6)
    angle = pos.double()[:, None, None] * s["inv_freq"].double()
    c, n = angle.cos().float(), angle.sin().float()

    def rotated(y):
        if case["inter"]:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            r = torch.stack((a * c - b * n, b * c + a * n), -1).flatten(-2)
        else:
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            r = torch.cat((a * c - b * n, b * c + a * n), -1)
        return torch.cat((r, y[..., rot:]), -1)

    view = _heads_view(case, s["pages"])
    kc, vc, ks, vs = _row_places(d, case["fmt"], x.device)
    heads = torch.arange(h, device=x.device)
    at = (page[:, None, None], heads[None, :, None], group[:, None, None])
    for y, cp, sp, which in ((rotated(k), kc, ks, "k"), (v, vc, vs, "v")):
        codes, byte = _quantise(y, case["fmt"], s["scales"][which])
        view[(*at, cp[row][:, None, :])] = codes
        view[(*at, sp[row][:, None, :])] = byte
    return rotated(q).bfloat16()


def _plain_read(s):
    case = s["case"]
    _, page, group, row = _token_places(s)
    view = _heads_view(case, s["pages"])
    kc, vc, ks, vs = _row_places(case["dim"], case["fmt"], page.device)
    heads = torch.arange(case["kv_heads"], device=page.device)
    at = (page[:, None, None], heads[None, :, None], group[:, None, None])
    out = [_values(view[(*at, cp[row][:, None, :])], view[(*at, sp[row][:, None, :])], case["fmt"], s["scales"][which]).bfloat16()
           for cp, sp, which in ((kc, ks, "k"), (vc, vs, "v"))]
    return out[0], out[1]


def _plain_attention(s):
    """Padded to the longest: scores of every query and every cached position, masked, softmax, product."""
    case = s["case"]
    hq, h, d, p, n = case["q_heads"], case["kv_heads"], case["dim"], case["page"], case["seqs"]
    dev = s["q"].device
    chunks = _heads_view(case, s["pages"])[s["table"].clamp(min=0).long()]  # [seq, page, head, group, bytes]
    kc, vc, ks, vs = _row_places(d, case["fmt"], dev)

    def cached(cp, sp, which):
        codes, byte = chunks[..., cp.reshape(-1)], chunks[..., sp.reshape(-1)]
        shape = lambda x: x.view(n, -1, h, p // 16, 16, x.shape[-1] // 16).permute(0, 2, 1, 3, 4, 5).reshape(n, h, -1, x.shape[-1] // 16)  # noqa: E731
        return _values(shape(codes), shape(byte), case["fmt"], s["scales"][which][:, :, None])

    k, v = cached(kc, ks, "k"), cached(vc, vs, "v")  # [seq, head, position, dim]
    t = torch.arange(s["tokens"], device=dev)
    b = torch.searchsorted(s["cu_q"].long(), t, right=True) - 1
    i = t - s["cu_q"][b]
    q = torch.zeros(n, s["max_q"], hq, d, device=dev)
    q[b, i] = s["q"].float()
    q = q.view(n, s["max_q"], h, hq // h, d).permute(0, 2, 3, 1, 4).reshape(n, h, -1, d)
    scores = (q @ k.transpose(-1, -2)).view(n, h, hq // h, s["max_q"], -1)
    scores *= d ** -0.5
    j = torch.arange(scores.shape[-1], device=dev)
    length = s["kv_len"].long()[:, None, None]
    seen = j < length
    if case["causal"]:
        pos = length - (s["cu_q"][1:] - s["cu_q"][:-1]).long()[:, None, None] + torch.arange(s["max_q"], device=dev)[None, :, None]
        seen = seen & (j <= pos)
        if case["window"]:
            seen = seen & (j > pos - case["window"])
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    scores -= top
    w = scores.exp_()
    total = w.sum(-1, keepdim=True)
    o = (w.view(n, h, -1, w.shape[-1]) @ v).view(n, h, hq // h, s["max_q"], d) / total.clamp(min=1e-38)
    lse = (top + total.log()).squeeze(-1)
    y = o.permute(0, 3, 1, 2, 4).reshape(n, s["max_q"], hq, d)[b, i]
    return y.bfloat16(), lse.permute(0, 3, 1, 2).reshape(n, s["max_q"], hq)[b, i]


# ------------------------------------------------------------------------------------------ the work
def work(case):
    if case["op"] == "norm":
        t, k = case["tokens"], case["k"]
        extra = (case["post"] + case["pre"] + case["gates"]) * k * 2
        return {"bytes": t * k * 2 * (3 + case["pre"]) + extra, "flops": t * k * 10}
    hq, h, d = case["q_heads"], case["kv_heads"], case["dim"]
    row = 2 * h * (d / 2 + d / _block(case["fmt"]))  # cache bytes of one token
    each, ctx = _lengths(case)
    new = sum(each)
    if case["op"] == "read":
        return {"bytes": new * (row + 4 * h * d), "flops": new * 4 * h * d}
    if case["op"] == "append":
        return {"bytes": new * (2 * (hq + 2 * h) * d + 2 * hq * d + 2 * row + 4 * h * d), "flops": new * d * (6 * (hq + h) + 8 * h)}
    pairs = keys = 0  # (query, key) pairs that see each other, and cached tokens that any query sees
    for m, c in zip(each, ctx):
        if not case["causal"]:
            pairs, keys = pairs + m * max(1, c), keys + max(1, c)
        elif not case["window"]:
            pairs, keys = pairs + m * c + m * (m + 1) / 2, keys + c + m
        else:
            w = case["window"]
            short = min(m, max(0, w - c))  # queries whose window reaches the sequence's start
            pairs, keys = pairs + short * c + short * (short + 1) / 2 + (m - short) * w, keys + min(c + m, w + m - 1)
    return {"bytes": keys * row + new * hq * (4 * d + 4), "flops": 4.0 * pairs * hq * d}


# ------------------------------------------------------------- the definition in 64 bits, written apart
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    return _exact_cache(s)


def _exact_norm(s):
    case = s["case"]
    y, r = s["y"].double(), s["residual"].double()
    if s["post"] is not None:
        y = y / torch.sqrt((y * y).mean(1, keepdim=True) + 1e-6) * s["post"].double()[None]
    if s["gate"] is not None:
        if case["rows_per_gate"]:
            y = y * s["gate"].double().repeat_interleave(case["rows_per_gate"], 0)[: case["tokens"]]
        else:
            y = y * s["gate"].double()[0]
    r = case["alpha"] * r + y
    if s["pre"] is None:
        return (r,)
    stored = r.bfloat16().double()  # the next block sees the residual stream as it is stored
    return r, stored / torch.sqrt((stored * stored).mean(1, keepdim=True) + 1e-6) * s["pre"].double()[None]


def _e4m3_value(byte):
    b = byte.long()
    e, m = (b >> 3) & 15, b & 7
    v = torch.where(e == 0, m.double() / 8 * 2.0 ** -6, (1 + m.double() / 8) * torch.pow(2.0, (e - 7).double()))
    return torch.where(b >= 128, -v, v)


def _exact_sequence(s, b, first, last):
    """Keys and values of positions first..last of one sequence, float64 [positions, heads, dim]."""
    case = s["case"]
    h, d, p, fmt = case["kv_heads"], case["dim"], case["page"], case["fmt"]
    blk = _block(fmt)
    gb = _group_bytes(case)
    pos = torch.arange(first, last, device="cuda")
    base = s["table"][b].long()[pos // p]
    raw = s["pages"].view(-1, h, (p // 16) * gb)[base]  # [positions, heads, page bytes]
    g0 = ((pos % p) // 16 * gb)[:, None]
    r = pos % 16
    hh, t, j = r // 8, (r // 2) % 4, r % 2
    e = torch.arange(d, device="cuda")[None]
    run, inside = e // (d // 8), e % (d // 8)
    where_k = g0 + r[:, None] * (d // 2) + e // 2
    cell = 4 * run + t[:, None]
    unit = (64 * hh[:, None] + 2 * cell + j[:, None]) * 8 if d == 128 else (4 * cell + 2 * hh[:, None] + j[:, None]) * 4
    where_v = g0 + 8 * d + unit + inside // 2
    nb = d // blk
    scale_k = g0 + 16 * d + r[:, None] * nb + e // blk
    scale_v = g0 + 16 * d + 16 * nb + (4 * (e // blk) + t[:, None]) * 4 + (2 * hh + j)[:, None]
    out = []
    for code_at, scale_at, which in ((where_k, scale_k, "k"), (where_v, scale_v, "v")):
        take = lambda at: raw.gather(2, at[:, None, :].expand(-1, h, -1))  # noqa: E731
        c = (take(code_at).long() >> (4 * (e % 2))[:, None]) & 15
        ex, m = (c >> 1) & 3, c & 1
        v = torch.where(ex == 0, m.double() / 2, (1 + m.double() / 2) * torch.pow(2.0, (ex - 1).double()))
        v = torch.where(c >= 8, -v, v)
        sc = take(scale_at)
        v = v * (_e4m3_value(sc) if fmt == "nvfp4" else torch.pow(2.0, (sc.long() - 127).double()))
        out.append(v * s["scales"][which].double()[None] if fmt == "nvfp4" else v)
    return out


def _exact_quantised(x, fmt, scale):
    """float64 rows [tokens, heads, dim] as the values that their codes stand for."""
    blk = _block(fmt)
    y = x.reshape(*x.shape[:2], -1, blk)
    top = y.abs().amax(-1, keepdim=True)
    if fmt == "nvfp4":
        sc = scale.double()[None, :, :, None]
        sb = _e4m3_value((top / (6 * sc)).clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8)) * sc
    else:
        sb = torch.pow(2.0, (torch.floor(torch.log2(top.clamp(min=1e-30))) - 2).clamp(-23, 13))
    u = torch.where(sb > 0, y / sb.clamp(min=1e-300), torch.zeros_like(y))
    grid = torch.tensor(_E2M1, dtype=torch.float64, device=x.device)
    far = (u.abs().clamp(max=6).unsqueeze(-1) - grid).abs()
    best = far.amin(-1, keepdim=True)
    even = torch.arange(8, device=x.device) % 2 == 0
    code = torch.where(far == best, even.double() + 1, torch.zeros_like(far)).argmax(-1)  # of two, the even one
    return (torch.sign(u) * grid[code] * sb).reshape(x.shape)


def _exact_cache(s):
    case = s["case"]
    hq, h, d = case["q_heads"], case["kv_heads"], case["dim"]
    parts, start = [], 0
    if case["op"] == "attn" and 4.0 * sum(n * c for n, c in zip(s["new"], s["length"])) * hq * d > 4e12:
        return None
    for b, (n, length) in enumerate(zip(s["new"], s["length"])):
        first = length - n
        if case["op"] == "read":
            parts.append(_exact_sequence(s, b, first, length))
        elif case["op"] == "append":
            x = s["qkv"][start:start + n].double().view(n, hq + 2 * h, d)
            q, k, v = x.split((hq, h, h), 1)
            if s["q_gamma"] is not None:
                q, k = [y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6) * g.double() for y, g in ((q, s["q_gamma"]), (k, s["k_gamma"]))]
            turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                               torch.arange(first, length, device=x.device).double()[:, None] * s["inv_freq"].double()[None])[:, None]
            half = case["rot"] // 2
            both = []
            for y in (q, k):
                z = y[..., :2 * half].reshape(n, -1, half, 2) if case["inter"] else y[..., :2 * half].reshape(n, -1, 2, half).transpose(2, 3)
                z = torch.view_as_real(torch.complex(z[..., 0].contiguous(), z[..., 1].contiguous()) * turn)
                z = z if case["inter"] else z.transpose(2, 3)
                both.append(torch.cat((z.reshape(n, -1, 2 * half), y[..., 2 * half:]), -1))
            parts.append((both[0], _exact_quantised(both[1], case["fmt"], s["scales"]["k"]), _exact_quantised(v, case["fmt"], s["scales"]["v"])))
        else:
            k, v = _exact_sequence(s, b, 0, length)
            q = s["q"][start:start + n].double()
            y, lse = [], []
            for head in range(hq):
                w = q[:, head] @ k[:, head * h // hq].T / math.sqrt(d)
                if case["causal"]:
                    ahead = torch.arange(length, device=w.device)[None] - torch.arange(first, length, device=w.device)[:, None]
                    w = w.masked_fill(ahead > 0, -math.inf)
                    if case["window"]:
                        w = w.masked_fill(ahead <= -case["window"], -math.inf)
                lse.append(torch.logsumexp(w, -1))
                y.append(torch.exp(w - lse[-1][:, None]) @ v[:, head * h // hq])
            parts.append((torch.stack(y, 1), torch.stack(lse, 1)))
        start += n
    return tuple(torch.cat(x) for x in zip(*parts))
